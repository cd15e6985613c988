"""Quantising to 4 bits where the scale overflows its type, against the
definition in 64 bits (GPU tests)."""

import numpy as np
import pytest
import torch

import dense_fp32_matrix_sgemm_amd as sg
from tests.test_parity_w4 import quantised

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sg.load_library()


@pytest.mark.parametrize("group", [32, 96, 256])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("dtype,stype", [("f32", "f16"), ("bf16", "f16"), ("f32", "f32"), ("f32", "bf16")])
def test_scales_that_overflow(dtype, stype, zeros, group):
    # Groups whose scale is infinite (in f16 from 7 * 65520 on; in float32 where hi - lo is), next to ones whose is not.
    rows = np.linspace(-1.0, 1.0, 5 * 300).reshape(5, 300)
    rows[0] *= 1e6
    rows[1] *= 7 * 65504.0       # without zeros just within f16
    rows[2, 40:] = np.where(np.arange(260) % 3 == 0, -3e38, 3e38)
    rows[3, 100:140] = 2e38      # one sign
    rows[4, ::7] = -3.2e38
    with np.errstate(all="ignore"):
        quantised(rows.astype(np.float32), group, zeros, stype, dtype, f"{dtype} {stype} group {group}")

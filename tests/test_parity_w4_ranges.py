"""The product with a matrix held in 4 bits at the ends of float32's range and
over long sums, against its definition in 64 bits (GPU tests)."""

import numpy as np
import pytest
import torch

import dense_fp32_matrix_sgemm_amd as sg
from tests import lowbit_ref as ref
from tests.test_parity_w4 import TYPES

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sg.load_library()


# Few rows (with A in LDS, straight to registers, K shorter than a step), and each tile.
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,N,K", [(3, 70, 600), (1, 20, 100), (13, 48, 4100), (20, 96, 600), (50, 96, 600), (257, 8200, 300), (1030, 4100, 300)])
def test_the_largest_scales(M, N, K, dtype):
    # A is small: sums of whole numbers times 2^125 * 2^-22, finite and exact. A row of W that is zero gives 0.
    g = torch.Generator().manual_seed(M)
    A = torch.randint(-4, 5, (M, K), generator=g).float()
    codes = torch.randint(0, 256, (N, -(-K // 2)), generator=g, dtype=torch.uint8)
    codes[5] = 0x88
    q = torch.from_numpy(ref.codes_of(codes.numpy(), K)).float() - 8
    want = (A @ q.t()).double() * 2.0**103  # the sum is below 2^18: exact
    # f16 has no number below 2^-24: there the 2^-22 is split between A and alpha.
    a, alpha = (A * 2.0**-11, 2.0**-11) if dtype == "f16" else (A * 2.0**-22, 1.0)
    assert (want.abs() < 2.0**(128 - 11)).all()
    for stype in ("f32", "bf16"):
        S = torch.full((N, -(-K // 32)), 2.0**125).to(TYPES[stype]).cuda()
        for zeros in (None, torch.full(S.shape, 8, dtype=torch.uint8).cuda()):
            W = sg.W4(codes.cuda(), S, zeros, K, 32)
            C = sg.gemm_w4(a.to(TYPES[dtype]).cuda(), W, alpha=alpha).cpu().double()
            assert torch.equal(C, want), (stype, zeros is not None)

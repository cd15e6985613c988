"""Arguments of a serving step's helpers that are of no use at all, and that are
refused as such (GPU tests)."""

import pytest
import torch

import dense_fp32_matrix_sgemm_amd as sg

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sg.load_library()


def test_outputs_that_are_no_tensors():
    Q, K = torch.ones(4, 2, 64, device="cuda"), torch.ones(4, 1, 64, device="cuda")
    positions, freqs = torch.arange(4, dtype=torch.int32).cuda(), sg.rope_frequencies(64)[0]
    for key, out in ((None, (Q,)), (None, [Q, K]), (None, 5), (None, "Q"), (K, 5), (K, (Q, 5)), (K, (5, K)), (K, (None, K)), (K, (Q, K, K))):
        with pytest.raises(TypeError):
            sg.rope(Q, key, positions, freqs, out=out)
        with pytest.raises(TypeError):
            sg.rope(Q, key, positions, freqs, dtype=torch.float32, out=out)
    assert (Q == 1).all() and (K == 1).all()

"""The tile kernels of the product with a matrix held in 4 bits, at sizes that
reach each of their shapes (GPU tests)."""

import pytest
import torch

import dense_fp32_matrix_sgemm_amd as sg
from tests.test_parity_w4 import TYPES

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sg.load_library()


# Tiles whose waves divide K and each hold A's slab in LDS of their own: 32 x
# 32, 64 x 32 and 64 x 64. K gives each wave many slabs, or fewer slabs than
# there are waves; whole numbers, so that a stale or torn slab changes the
# result by a whole number.
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,N", [(20, 96), (50, 96), (257, 8200)])
def test_slabs_of_a_wave_of_its_own(M, N, dtype):
    g = torch.Generator().manual_seed(M)
    for K, group in ((4096 + 77, 128), (2048, 32), (640, 64), (300, 32)):
        print(f"[w4 tiles] {M}x{N}x{K} {dtype} group={group}", flush=True)
        A = torch.randint(-4, 5, (M, K), generator=g).float()
        codes = torch.randint(0, 256, (N, -(-K // 2)), generator=g, dtype=torch.uint8)
        q = torch.stack((codes & 15, codes >> 4), dim=2).flatten(1)[:, :K].float() - 8
        W = sg.W4(codes.cuda(), torch.ones(N, -(-K // group)).cuda(), None, K, group)
        C = sg.gemm_w4(A.to(TYPES[dtype]).cuda(), W)
        # Sums below 2^24: exact in float32 in any order.
        assert torch.equal(C.cpu(), A @ q.t()), (K, group)

"""The tile kernels of the product with a matrix held in 4 bits, at sizes that
reach each of their shapes (GPU tests)."""

import numpy as np
import pytest
import torch

import dense_fp32_matrix_sgemm_amd as sg
from oracle.check import assert_within
from tests.test_parity_w4 import TYPES, check, operands

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


# (M, N): shape of 16-bit rows, of float32 rows: rows and columns of a work-group, waves along N and K.
TILES = {(1030, 4100): ((64, 256, 4, 1), (64, 256, 4, 1)), (257, 8200): ((64, 64, 1, 4), (32, 32, 1, 4)),
         (50, 100): ((64, 32, 1, 8), (32, 32, 1, 4)), (20, 100): ((32, 32, 1, 8), (32, 32, 1, 4))}
# Less than a slab of 128 k, slabs and one k, ends inside a slab and a group, groups inside, across and of whole slabs.
DEPTHS = [(33, 32), (129, 64), (300, 96), (385, 128), (512, 256), (643, 32), (200, 128)]


def shape_of(dtype, M, N, K):
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    code = {"f32": sg.SGEMM_F32, "bf16": sg.SGEMM_LP_BF16, "f16": sg.SGEMM_LP_F16}[dtype]
    if cus != 256:
        pytest.skip("sizes chosen for 256 compute units")
    return sg.sgemm_w4_shape(code, M, N, K, cus)[:4]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("size", TILES)
def test_each_tile(size, zeros, dtype):
    M, N = size
    for i, (K, group) in enumerate(DEPTHS):
        print(f"[w4 tiles] {M}x{N}x{K} {dtype} zeros={zeros} group={group}", flush=True)
        assert shape_of(dtype, M, N, K) == TILES[size][dtype == "f32"]
        A, W, dense = operands(K + M, M, N, K, group, dtype, ("f32", "bf16", "f16")[i % 3], zeros, pad=i % 4)
        check(A, W, dense, what=f"K={K} group={group}", pad=i % 4)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("size", TILES)
def test_alpha_and_beta_of_each_tile(size, dtype):
    M, N = size
    A, W, dense = operands(8, M, N, 200, 64, dtype, "f32", True, pad=3)
    C0 = torch.randn(M, N, generator=torch.Generator().manual_seed(9))
    check(A, W, dense, C0, -0.75, 1.5, "alpha, beta", pad=3)
    check(A, W, dense, torch.full((M, N), float("nan")), 0.5, 0.0, "C not read")


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("size", TILES)
def test_what_is_not_finite_stays_in_its_row_and_column(size, dtype):
    M, N, K = *size, 200
    A, W, dense = operands(12, M, N, K, 32, dtype, "f32", True)
    A[3, 190], A[M - 1, 5] = float("nan"), float("nan")
    W.scales[7, 6], W.scales[N - 1, 0] = float("nan"), float("nan")  # k 192 to 199; 0 to 31
    C = sg.gemm_w4(A.cuda(), W).cpu().numpy()
    rows, cols = np.ones(M, bool), np.ones(N, bool)
    rows[[3, M - 1]], cols[[7, N - 1]] = False, False
    assert np.isnan(C[~rows]).all() and np.isnan(C[:, ~cols]).all()
    a = A.double().numpy()[rows]
    assert_within(C[rows][:, cols], a @ dense[cols].T, np.abs(a) @ np.abs(dense[cols]).T, "the rest")

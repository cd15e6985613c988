"""The product with a matrix held in 4 bits, and the quantising and reading
back of such a matrix, against their definitions in 64 bits (GPU tests)."""

import numpy as np
import pytest
import torch

import dense_fp32_matrix_sgemm_amd as sg
from oracle.check import assert_within
from tests import lowbit_ref as ref

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sg.load_library()


def padded(t, pad, fill):
    """t (on the GPU) as a view whose rows lie `pad` elements further apart, the padding holding `fill`."""
    rows, cols = t.shape
    buf = torch.full((rows, cols + pad), 0, dtype=t.dtype).fill_(fill)
    buf[:, :cols] = t
    return buf.cuda()[:, :cols]


def operands(seed, M, N, K, group, dtype, stype, zeros, pad=0):
    g = torch.Generator().manual_seed(seed)
    G = -(-K // group)
    A = torch.randn(M, K, generator=g).to(TYPES[dtype])
    codes = torch.randint(0, 256, (N, -(-K // 2)), generator=g, dtype=torch.uint8)
    S = (torch.rand(N, G, generator=g) * 0.02 + 0.001).to(TYPES[stype])
    Z = torch.randint(0, 16, (N, G), generator=g, dtype=torch.uint8) if zeros else None
    nan = float("nan")
    W = sg.W4(padded(codes, pad, 0xA7), padded(S, pad, nan), None if Z is None else padded(Z, pad, 0xFF), K, group)
    return A, W, ref.w4_matrix(codes.numpy(), S.double().numpy(), None if Z is None else Z.numpy(), K, group)


def check(A, W, dense, C0=None, alpha=1.0, beta=0.0, what="", pad=0):
    M, N = A.shape[0], dense.shape[0]
    buf = torch.full((M + 1, N + 1 + pad), -12345.0)
    if C0 is not None:
        buf[:M, :N] = C0
    dev = buf.cuda()
    C = dev[:M, :N]
    sg.gemm_w4(padded(A, pad, float("nan")) if pad else A.cuda(), W, C, alpha, beta)
    torch.cuda.synchronize()
    a = A.double().numpy()
    exact, size = alpha * (a @ dense.T), abs(alpha) * (np.abs(a) @ np.abs(dense).T)
    if beta:
        exact, size = exact + beta * C0.double().numpy(), size + abs(beta) * np.abs(C0.double().numpy())
    got = dev.cpu().numpy()
    assert_within(got[:M, :N], exact, size, what)
    buf[:M, :N] = torch.from_numpy(got[:M, :N])
    assert np.array_equal(got, buf.numpy()), "written outside C"


# Sizes at and around the steps of the kernels: 16 rows and columns, 32, 128
# and 256 k, odd k, groups that end inside a row, one of each.
SHAPES = [(1, 1, 1), (1, 16, 128), (1, 17, 129), (2, 15, 127), (3, 33, 31), (5, 40, 32), (16, 16, 33), (17, 31, 255),
          (1, 100, 2049), (33, 65, 300), (64, 48, 513), (65, 130, 384), (100, 129, 641), (128, 256, 96), (200, 300, 257),
          (15, 64, 1024), (31, 257, 1000), (129, 64, 64)]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_product(shape, zeros, dtype):
    M, N, K = shape
    for i, group in enumerate((32, 64, 96, 128, 256)):
        stype = ("f32", "bf16", "f16")[(i + M) % 3]
        print(f"[w4] {shape} {dtype} zeros={zeros} group={group} {stype}", flush=True)
        A, W, dense = operands(100 * M + K + i, M, N, K, group, dtype, stype, zeros, pad=i)
        check(A, W, dense, what=f"group {group}", pad=i)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M,N,K", [(1, 4096, 4096), (7, 1000, 8200), (40, 2047, 1500), (300, 1024, 1024), (513, 640, 2050)])
def test_larger_products(M, N, K, dtype):
    print(f"[w4] {M}x{N}x{K} {dtype}", flush=True)
    A, W, dense = operands(M, M, N, K, 128, dtype, "f16", M % 2 == 1)
    check(A, W, dense, what="larger")


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M", [3, 150])
def test_alpha_beta(M, dtype):
    A, W, dense = operands(5, M, 70, 200, 64, dtype, "f32", True, pad=3)
    C0 = torch.randn(M, 70, generator=torch.Generator().manual_seed(6))
    check(A, W, dense, C0, -0.75, 1.5, "alpha, beta", pad=3)
    check(A, W, dense, torch.full((M, 70), float("nan")), 0.5, 0.0, "C not read")
    # Nothing but C: alpha 0.
    C = C0.cuda()
    sg.gemm_w4(A.cuda(), W, C, 0.0, 2.0)
    assert torch.equal(C.cpu(), 2 * C0)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M", [1, 16, 40, 100, 200])
def test_small_whole_numbers_are_exact(M, dtype):
    g = torch.Generator().manual_seed(M)
    N, K, group = 50, 700, 64
    A = torch.randint(-8, 9, (M, K), generator=g).to(TYPES[dtype])
    codes = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8)
    S = torch.tensor([0.5, 1.0, 2.0])[torch.randint(0, 3, (N, -(-K // group)), generator=g)]
    Z = torch.randint(0, 16, S.shape, generator=g, dtype=torch.uint8)
    for z in (None, Z):
        dense = ref.w4_matrix(codes.numpy(), S.numpy(), None if z is None else z.numpy(), K, group)
        C = sg.gemm_w4(A.cuda(), sg.W4(codes.cuda(), S.cuda(), None if z is None else z.cuda(), K, group))
        assert np.array_equal(C.cpu().double().numpy(), A.double().numpy() @ dense.T)


@pytest.mark.parametrize("M", [2, 130])
def test_float32_rows_keep_their_bits(M):
    # One element of A against one code each: the product is a * s * (q - z) with a's 24 bits.
    K, N = 64, 16
    g = torch.Generator().manual_seed(3)
    A = torch.zeros(M, K)
    A[:, 5] = torch.randn(M, generator=g) * 10.0 ** torch.randint(-20, 20, (M,), generator=g)
    codes = torch.randint(0, 256, (N, K // 2), generator=g, dtype=torch.uint8)
    W = sg.W4(codes.cuda(), torch.ones(N, 1).cuda(), None, K, 64)
    dense = ref.w4_matrix(codes.numpy(), np.ones((N, 1)), None, K, 64)
    C = sg.gemm_w4(A.cuda(), W).cpu().double().numpy()
    exact = A.double().numpy() @ dense.T
    # three exact parts, two additions: two roundings of at most 2^-24 each
    assert (np.abs(C - exact) <= 2.0**-23 * np.abs(exact)).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("M", [4, 160])
def test_infinities_nan_and_zero_groups(M, zeros, dtype):
    A, W, dense = operands(9, M, 40, 256, 32, dtype, "f32", zeros)
    # A group whose codes are all its zero point is zero, exactly.
    zero = 8 if W.zeros is None else int(W.zeros[3, 2].item() & 15)
    W.codes[3, 32:48] = zero * 17
    dense[3, 64:96] = 0.0
    A[:] = 0
    A[:, 64:96] = torch.randn(M, 32).to(A.dtype)
    C = sg.gemm_w4(A.cuda(), W).cpu()
    assert (C[:, 3] == 0).all()
    # Infinity times the matrix: infinities of the weights' signs, NaN where the weight is 0.
    A[:] = 0
    A[0, 70], A[1, 7] = float("inf"), float("nan")
    C = sg.gemm_w4(A.cuda(), W).cpu().numpy()
    with np.errstate(invalid="ignore"):
        want = np.float64("inf") * dense[:, 70]
    assert np.array_equal(C[0], want.astype(np.float32), equal_nan=True)
    assert np.isnan(C[1]).all() and np.isfinite(C[2:]).all()


# More of A than a compute unit's LDS holds: in slabs, or (few columns) straight to registers.
@pytest.mark.parametrize("M,N,K,group,zeros,dtype", [
    (13, 200, 4093, 32, True, "f32"), (16, 48, 4096, 128, False, "f32"), (3, 17, 20001, 64, True, "f32"),
    (8, 40, 12000, 96, True, "bf16"), (8, 33, 16384, 128, False, "f16"), (1, 5, 90000, 128, True, "bf16"),
    (13, 4200, 4093, 64, False, "f32"), (8, 4100, 11000, 128, True, "bf16")])
def test_rows_longer_than_lds(M, N, K, group, zeros, dtype):
    A, W, dense = operands(11, M, N, K, group, dtype, "f16", zeros)
    a = A.double().numpy()
    assert_within(sg.gemm_w4(A.cuda(), W).cpu().numpy(), a @ dense.T, np.abs(a) @ np.abs(dense).T)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("M", [4, 40])
def test_infinite_and_nan_scales_of_a_short_last_group(M, dtype):
    # K ends 8 into its last group (and inside a slab of 128): only real products see its scale.
    A, W, dense = operands(10, M, 40, 136, 32, dtype, "f32", False)
    W.codes[:, -4:] = 0x99
    W.scales[0, -1], W.scales[1, -1] = float("inf"), float("nan")
    A[:, -8:] = A[:, -8:].abs() + 1
    C = sg.gemm_w4(A.cuda(), W).cpu()
    assert (C[:, 0] == float("inf")).all() and torch.isnan(C[:, 1]).all() and torch.isfinite(C[:, 2:]).all()


def test_two_runs_are_the_same():
    for M in (1, 9, 77, 300):
        A, W, _ = operands(M, M, 333, 2000, 64, "bf16", "bf16", True)
        A = A.cuda()
        first = sg.gemm_w4(A, W)
        for _ in range(3):
            assert torch.equal(sg.gemm_w4(A, W), first)


# ------------------------------------------------- quantising, reading back


def to_type(stype):
    return lambda x: torch.tensor(x, dtype=torch.float32).to(TYPES[stype]).double().item()


def quantised(W, group, zeros, stype, dtype, what):
    t = torch.from_numpy(W).to(TYPES[dtype])
    q, S, Z = ref.w4_quantize(t.double().numpy(), group, zeros, to_type(stype))
    src = padded(t, 5, float("nan"))
    got = sg.quantize_w4(src, group, zeros, TYPES[stype])
    torch.cuda.synchronize()
    K = W.shape[1]
    assert np.array_equal(got.scales.cpu().double().numpy(), S, equal_nan=True), what
    if zeros:
        assert np.array_equal(got.zeros.cpu().numpy(), Z), what
    assert np.array_equal(ref.codes_of(got.codes.cpu().numpy(), K), q), what
    for out in ("f32", "bf16", "f16"):
        back = sg.dequantize_w4(got, TYPES[out]).cpu()
        with np.errstate(all="ignore"):
            z = 8 if Z is None else Z[:, np.arange(K) // group]
            exact = torch.from_numpy(((q - z) * S[:, np.arange(K) // group]).astype(np.float32)).to(TYPES[out])
        assert torch.equal(torch.nan_to_num(back, 7.0), torch.nan_to_num(exact, 7.0)), (what, out)


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("dtype,stype", [("f32", "f32"), ("f32", "f16"), ("bf16", "bf16"), ("bf16", "f16"), ("f16", "f32")])
@pytest.mark.parametrize("N,K", [(1, 1), (3, 31), (5, 33), (7, 200), (4, 257), (2, 1030)])
def test_quantise_and_read_back(N, K, dtype, stype, zeros):
    rng = np.random.default_rng(N * 1000 + K)
    for group in (32, 64, 96, 128, 288):
        W = rng.standard_normal((N, K)) * np.exp2(rng.integers(-6, 6, (N, 1)))
        quantised(W, group, zeros, stype, dtype, f"group {group}")


@pytest.mark.parametrize("zeros", [False, True])
def test_quantise_borders(zeros):
    # Quotients on and next to a half, all-zero groups, one sign only, values at the ends of float32, not finite ones.
    s = 0.25
    ties = np.array([7 * s] + [s * (k + 0.5) for k in range(-7, 7)] + [np.nextafter(np.float32(s * 2.5), np.float32(9)),
                    np.nextafter(np.float32(s * 2.5), np.float32(-9)), -7 * s], np.float64)
    rows = np.zeros((9, 64))
    rows[0, :len(ties)] = ties
    rows[1, 32:] = 3.0
    rows[2, :32] = -np.linspace(0, 5, 32)
    rows[3] = np.linspace(1, 2, 64)
    rows[4] = 1e-45
    rows[5] = np.linspace(-1e-40, 1e-38, 64)
    rows[6] = np.linspace(-1e38, 1e38, 64)
    rows[7, 3], rows[7, 40] = np.inf, np.nan
    rows[8] = np.linspace(-1e-6, 1e-6, 64)
    with np.errstate(all="ignore"):
        quantised(rows.astype(np.float32), 32, zeros, "f32", "f32", "borders")
        quantised(rows[[0, 1, 2, 3, 7, 8]].astype(np.float32), 32, zeros, "f16", "f32", "borders f16")


def test_codes_of_a_quantised_matrix_multiply():
    W = torch.randn(96, 320, generator=torch.Generator().manual_seed(1))
    A = torch.randn(6, 320, generator=torch.Generator().manual_seed(2))
    for zeros in (False, True):
        Q = sg.quantize_w4(W.cuda(), 64, zeros)
        dense = sg.dequantize_w4(Q).cpu().double().numpy()
        C = sg.gemm_w4(A.cuda(), Q).cpu().numpy()
        a = A.double().numpy()
        assert_within(C, a @ dense.T, np.abs(a) @ np.abs(dense).T, "quantised")
        # Half a step of a group's scale (its rounding to float32 aside).
        step = Q.scales.cpu().double().numpy()[:, np.arange(320) // 64]
        clipped = 1.0 if zeros else 0.5  # zeros: the zero point is rounded too
        assert (np.abs(dense - W.double().numpy()) <= (clipped + 1e-6) * step).all()

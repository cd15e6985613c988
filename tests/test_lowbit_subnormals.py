"""The products held in few bits on every code and on operands below their
type's normal numbers, brought back into sight by large scales (GPU tests)."""

import numpy as np
import pytest
import torch

import dense_fp32_matrix_sgemm_amd as sg
from tests import lowbit_ref as ref
from tests.test_parity_kv8 import TYPES, Case, close

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sg.load_library()


# Each kernel: few rows, the tiles whose waves divide K, the shared slab.
SIZES = [(3, 70, 600), (13, 48, 4100), (20, 96, 600), (50, 96, 600), (257, 8200, 300), (1030, 4100, 300)]


@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("dtype,low", [("f16", -24), ("bf16", -133)])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_subnormal_rows_multiply(M, N, K, dtype, low, zeros):
    # A holds whole multiples of the type's least number; sums of whole numbers, exact.
    g = torch.Generator().manual_seed(M)
    A = torch.randint(-4, 5, (M, K), generator=g).float()
    codes = torch.randint(0, 256, (N, -(-K // 2)), generator=g, dtype=torch.uint8)
    Z = torch.randint(0, 16, (N, -(-K // 32)), generator=g, dtype=torch.uint8) if zeros else None
    q = torch.from_numpy(ref.codes_of(codes.numpy(), K)).float()
    q = q - (8.0 if Z is None else Z[:, torch.arange(K) // 32].float())
    up = 20 if dtype == "f16" else 110
    W = sg.W4(codes.cuda(), torch.full((N, -(-K // 32)), 2.0**up).cuda(), None if Z is None else Z.cuda(), K, 32)
    a = (A.double() * 2.0**low).to(TYPES[dtype])
    assert torch.equal(a.double(), A.double() * 2.0**low)
    C = sg.gemm_w4(a.cuda(), W).cpu().double()
    assert torch.equal(C, (A @ q.t()).double() * 2.0**(low + up))


@pytest.mark.parametrize("M,N,K", SIZES)
def test_small_float32_rows_keep_their_bits(M, N, K):
    # One element of 24 bits near 2^-109 a row: its three parts are there to the last bit.
    g = torch.Generator().manual_seed(M)
    A = torch.zeros(M, K)
    A[:, 37] = (torch.rand(M, generator=g) + 1) * 2.0**-109
    codes = torch.randint(0, 256, (N, -(-K // 2)), generator=g, dtype=torch.uint8)
    q = torch.from_numpy(ref.codes_of(codes.numpy(), K)).double()[:, 37] - 8
    W = sg.W4(codes.cuda(), torch.full((N, -(-K // 32)), 2.0**100).cuda(), None, K, 32)
    C = sg.gemm_w4(A.cuda(), W).cpu().double()
    exact = A[:, 37].double()[:, None] * q[None, :] * 2.0**100
    # three exact parts, two additions: two roundings of at most 2^-24 each
    assert ((C - exact).abs() <= 2.0**-23 * exact.abs()).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("heads,new", [(1, 1), (256, 128)])
def test_every_code_of_a_value(heads, new, dtype):
    # A window of one token takes all: the output is its values, code by code.
    dim = 256
    case = Case(51, [max(new, 1)], [new], heads, 128, dim)
    page = case.table[0, 0]
    every = np.where((np.arange(256) & 0x7F) == 0x7F, 0, np.arange(256)).astype(np.uint8)
    for t in range(128):
        case.ref.codes[1][page, :, t] = np.roll(every, t)
    Q = case.normal(heads, dtype)
    got = sg.kv8_attend(Q.cuda(), case.device(), *case.args(), window=1, max_new=new).cpu().double().numpy()
    for i in range(new):
        want = ref.E4M3[case.ref.codes[1][page][:, i]] * case.ref.scales[1][page][:, None]
        assert np.array_equal(got[i], want), i


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("heads,new,dim", [(1, 3, 64), (2, 40, 128), (256, 128, 64)])
def test_every_code_of_a_key(heads, new, dim, dtype):
    case = Case(52, [max(new, 150)], [new], heads, 16, dim)
    codes = case.rng.integers(0, 256, case.ref.codes[0].shape).astype(np.uint8)
    small = case.rng.integers(0, 2, codes.shape).astype(bool)
    codes = np.where(small, codes & 0x8F, codes)  # half of them among the two least exponents
    case.ref.codes[0][...] = np.where((codes & 0x7F) == 0x7F, codes & 0x87, codes)
    Q = case.normal(heads, dtype)
    O, bound = case.ref.attend(Q.double().numpy(), case.table, case.lens, case.starts, 0.05, True, 0)
    got = sg.kv8_attend(Q.cuda(), case.device(), *case.args(), scale=0.05, max_new=new).cpu().double().numpy()
    close(got, O, bound, dtype)


@pytest.mark.parametrize("dtype,low", [("f16", -24), ("bf16", -133), ("f32", -109)])
@pytest.mark.parametrize("heads,new", [(1, 3), (256, 128)])
def test_small_queries_meet_large_scales(heads, new, dtype, low):
    # Multiples of the least number (float32: 24 bits near 2^-109) against keys whose scale brings the scores to about 1.
    case = Case(53, [max(new, 90)], [new], heads, 16, 64)
    case.ref.scales[0][...] = 2.0**(-low - 8)
    Q = case.rng.standard_normal((case.rows, heads, 64))
    Q = torch.from_numpy((np.rint(Q * 2) if dtype != "f32" else Q) * 2.0**low).to(TYPES[dtype])
    O, bound = case.ref.attend(Q.double().numpy(), case.table, case.lens, case.starts, 0.5, True, 0)
    got = sg.kv8_attend(Q.cuda(), case.device(), *case.args(), scale=0.5, max_new=new).cpu().double().numpy()
    close(got, O, bound, dtype)


@pytest.mark.parametrize("heads,new", [(1, 3), (256, 128)])
def test_small_value_scales(heads, new):
    # Values whose page scale is 2^-100: weights from 2^-110 on keep their bits.
    case = Case(54, [max(new, 90)], [new], heads, 16, 64)
    case.ref.scales[1][...] = 2.0**-100
    Q = case.normal(heads, "f32")
    O, bound = case.ref.attend(Q.double().numpy(), case.table, case.lens, case.starts, 0.01, True, 0)
    bound = (bound - 1e-30) + 2.0**-140  # the reference's own allowance is far above these results
    got = sg.kv8_attend(Q.cuda(), case.device(), *case.args(), scale=0.01, max_new=new).cpu().double().numpy()
    close(got, O, np.maximum(bound, 0), "small values")


@pytest.mark.parametrize("dtype,low", [("f16", -24), ("bf16", -133), ("f32", -149)])
def test_subnormal_rows_are_written(dtype, low):
    case = Case(55, [20], [20], 1, 32, 64)
    x = torch.from_numpy(np.rint(case.rng.standard_normal((20, 1, 64)) * 3) * 2.0**low).to(TYPES[dtype])
    cache = case.device()
    case.ref.write([x.double().numpy()] * 2, case.table, case.lens, case.starts)
    sg.kv8_write(cache, x.cuda(), x.cuda(), *case.args())
    page = case.table[0, 0]
    assert np.array_equal(cache.K.view(torch.uint8).cpu().numpy()[page, 0, :20] & 0x7F, case.ref.codes[0][page, 0, :20] & 0x7F)
    assert cache.Ks[page, 0].item() == case.ref.scales[0][page, 0]

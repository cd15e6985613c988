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


def dense_of(codes, zeros, scales, K, group):
    """The matrix in 64 bits, on the GPU."""
    g = torch.arange(K, device="cuda") // group
    q = torch.stack((codes & 15, codes >> 4), dim=2).flatten(1)[:, :K].double()
    return (q - (8.0 if zeros is None else zeros.double()[:, g])) * scales.double()[:, g]


# K in pieces: ends inside groups, groups longer than a piece, every kernel, float32's three parts, an odd end.
@pytest.mark.parametrize("M,N,K,group,zeros,dtype", [
    (1030, 4100, 65536 + 305, 96, True, "bf16"), (1030, 4100, 140001, 131072, True, "f16"), (1030, 4100, 131072 + 33, 32, False, "f32"),
    (1030, 4100, 3 * 65536, 64, False, "bf16"), (257, 8200, 4 * 65536 + 97, 128, True, "f16"), (50, 40, 8 * 65536 + 500, 160, False, "bf16"),
    (20, 40, 8 * 65536 + 31, 2**20, True, "f16"), (20, 40, 4 * 65536 + 1001, 32, True, "f32"), (2, 16, 16 * 65536 + 777, 64, True, "bf16"),
    (16, 20, 16 * 65536 + 1001, 128, False, "f32")])
def test_k_in_pieces(M, N, K, group, zeros, dtype):
    print(f"[w4 ranges] {M}x{N}x{K} group={group} zeros={zeros} {dtype}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(K)
    A = torch.randint(-4, 5, (M, K), generator=g, device="cuda", dtype=torch.int8).to(TYPES[dtype])
    codes = torch.randint(0, 256, (N, -(-K // 2)), generator=g, device="cuda", dtype=torch.uint8)
    S = torch.tensor([0.5, 1.0, 2.0], device="cuda")[torch.randint(0, 3, (N, -(-K // group)), generator=g, device="cuda")]
    Z = torch.randint(6, 10, S.shape, generator=g, device="cuda", dtype=torch.uint8) if zeros else None
    C0 = torch.randint(-9, 10, (M, N), generator=g, device="cuda").float()
    want = -0.5 * torch.matmul(A.double(), dense_of(codes, Z, S, K, group).t()) + 2.0 * C0.double()
    assert want.abs().max() < 2**21  # quarters below 2^22: float32 holds every partial sum
    W = sg.W4(codes, S, Z, K, group)
    C = C0.clone()
    sg.gemm_w4(A, W, C, -0.5, 2.0)
    assert torch.equal(C.double(), want)
    C.fill_(float("nan"))
    assert torch.equal(sg.gemm_w4(A, W, C, -0.5, 0.0).double(), want - 2.0 * C0.double())


# Terms of one sign, the same everywhere: the roundings of a long sum all go one way.
@pytest.mark.parametrize("M,N,K,dtype", [(1030, 4100, 65536, "bf16"), (1030, 4100, 2**20, "bf16"), (1030, 4100, 2**18, "f32"), (20, 96, 2**24, "f16"),
                                         (2, 16, 2**25, "bf16"), (16, 20, 2**24, "f32")])
def test_long_sums_of_one_sign(M, N, K, dtype):
    print(f"[w4 ranges] one sign {M}x{N}x{K} {dtype}", flush=True)
    A = torch.full((M, K), 0.7, dtype=TYPES[dtype], device="cuda")
    S = torch.full((N, K // 32), 0.013, dtype=torch.bfloat16, device="cuda")
    W = sg.W4(torch.full((N, K // 2), 0xFF, dtype=torch.uint8, device="cuda"), S, None, K, 32)
    exact = K * A[0, 0].double().item() * 7 * S[0, 0].double().item()
    C = sg.gemm_w4(A, W).double()
    worst = ((C - exact).abs().max() / exact).item()
    print(f"[w4 ranges] worst {worst:.2e}", flush=True)
    assert worst <= 1e-5 + 2.0**-29 * min(K, 65536) + 2.0**-40 * K


@pytest.mark.parametrize("M,N,K", [(20, 40, 8 * 65536 + 500), (1030, 4100, 65536 + 300)])
def test_pieces_in_a_captured_graph(M, N, K):
    # Several launches that follow from one another through C: every replay on new inputs agrees with the call itself.
    g = torch.Generator(device="cuda").manual_seed(M)
    A = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    codes = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    W = sg.W4(codes, torch.rand(N, -(-K // 128), generator=g, device="cuda"), None, K, 128)
    out, eager = torch.empty(M, N, device="cuda"), torch.empty(M, N, device="cuda")
    A.normal_(generator=g)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        sg.gemm_w4(A, W, out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sg.gemm_w4(A, W, out)
    for replay in range(3):
        A.normal_(generator=g)
        out.fill_(float("nan"))
        torch.cuda.synchronize()
        graph.replay()
        sg.gemm_w4(A, W, eager)
        torch.cuda.synchronize()
        assert torch.equal(out, eager) and torch.isfinite(out).all(), replay
    del graph

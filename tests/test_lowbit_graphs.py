"""The products held in few bits as a program runs them: together, on streams
of its own, captured and replayed, two at once (GPU tests)."""

import numpy as np
import pytest
import torch

import dense_fp32_matrix_sgemm_amd as sg
from oracle.check import assert_within
from tests import lowbit_ref as ref
from tests.test_parity_kv8 import Case, close, same_cache

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sg.load_library()


class Block:
    """The attention half of a block: x -> q, k, v (4-bit products) -> cache
    -> attention -> 4-bit product added to x. Everything float32 in between."""

    def __init__(self, seed, width, heads, ratio, dim, zeros):
        g = torch.Generator().manual_seed(seed)
        self.heads, self.ratio, self.dim = heads, ratio, dim
        self.w = {}
        for name, n, k in (("q", heads * ratio * dim, width), ("k", heads * dim, width), ("v", heads * dim, width),
                           ("o", width, heads * ratio * dim)):
            W = (torch.randn(n, k, generator=g) / k**0.5).cuda()
            self.w[name] = sg.quantize_w4(W, 64, zeros, torch.float16)

    def __call__(self, x, cache, args, max_new):
        rows = x.shape[0]
        q, k, v = (sg.gemm_w4(x, self.w[n]) for n in "qkv")
        sg.kv8_write(cache, k.view(rows, self.heads, self.dim), v.view(rows, self.heads, self.dim), *args, max_new=max_new)
        o = sg.kv8_attend(q.view(rows, -1, self.dim), cache, *args, max_new=max_new)
        return q, k, v, o, sg.gemm_w4(o.view(rows, -1), self.w["o"], x.clone(), beta=1.0)

    def check(self, x, outs, case, what):
        """Each output against its definition on the inputs that the library's call had."""
        q, k, v, o, y = (t.cpu() for t in outs)
        x = x.cpu().double().numpy()
        dense = {n: sg.dequantize_w4(w).cpu().double().numpy() for n, w in self.w.items()}
        for name, got in (("q", q), ("k", k), ("v", v)):
            assert_within(got.numpy(), x @ dense[name].T, np.abs(x) @ np.abs(dense[name]).T, f"{what} {name}")
        rows = x.shape[0]
        kv = [t.double().numpy().reshape(rows, self.heads, self.dim) for t in (k, v)]
        case.ref.write(kv, case.table, case.lens, case.starts)
        O, bound = case.ref.attend(q.double().numpy().reshape(rows, -1, self.dim), case.table, case.lens, case.starts,
                                   self.dim**-0.5, True, 0)
        close(o.double().numpy(), O, bound, f"{what} attention")
        a = o.double().numpy().reshape(rows, -1)
        assert_within(y.numpy(), x + a @ dense["o"].T, np.abs(x) + np.abs(a) @ np.abs(dense["o"]).T, f"{what} y")


@pytest.mark.parametrize("zeros", [False, True])
def test_prompt_then_tokens(zeros):
    block = Block(1, 256, 2, 3, 64, zeros)
    g = torch.Generator().manual_seed(2)
    case = Case(3, [20, 7, 33], [20, 7, 33], 2, 16, 64, columns=4)
    # Room for the tokens to come: pages of their own behind each sequence's last.
    used = {int(p) for p in case.table.reshape(-1) if p >= 0}
    free = [p for p in range(case.ref.pages) if p not in used]
    for b in range(3):
        case.table[b, -(-int(case.lens[b]) // 16)] = free[b]
    cache = case.device()
    x = torch.randn(case.rows, 256, generator=g).cuda()
    outs = block(x, cache, case.args(), 33)
    block.check(x, outs, case, "prompt")
    for step in range(3):
        case.lens = case.lens + 1
        case.starts = np.arange(4, dtype=np.int32)
        x = torch.randn(3, 256, generator=g).cuda() * 2.0**step
        outs = block(x, cache, case.args(), 1)
        block.check(x, outs, case, f"token {step}")
    same_cache(cache, case.ref, "after the tokens")


def test_a_captured_step_replayed():
    # One token for two long sequences: split attention with its workspace inside the graph.
    block = Block(5, 128, 1, 4, 128, True)
    case = Case(7, [4500, 3000], [1, 1], 1, 32, 128)
    cache, args = case.device(), case.args()
    x = torch.zeros(2, 128, device="cuda")
    codes = [t.clone() for t in (cache.K.view(torch.uint8), cache.V.view(torch.uint8), cache.Ks, cache.Vs)]
    before = [c.copy() for c in case.ref.codes + case.ref.scales]

    def restore():
        for t, c in zip((cache.K.view(torch.uint8), cache.V.view(torch.uint8), cache.Ks, cache.Vs), codes):
            t.copy_(c)
        case.ref.codes, case.ref.scales = [c.copy() for c in before[:2]], [c.copy() for c in before[2:]]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        block(x, cache, args, 1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = block(x, cache, args, 1)
    for replay in range(3):
        restore()
        x.copy_(torch.randn(2, 128, generator=torch.Generator().manual_seed(replay)))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        block.check(x, outs, case, f"replay {replay}")
        same_cache(cache, case.ref, f"replay {replay}")
        torch.matmul(x, x.t()).sum().item()  # eager work between replays
    del graph


def test_two_graphs_and_two_streams_do_not_share_scratch():
    # Each captured call and each stream has its own workspace: replays that overlap agree with eager results.
    cases = [Case(20 + i, [5000 - 700 * i], [1], 1, 32, 128) for i in range(2)]
    caches, args = [c.device() for c in cases], [c.args() for c in cases]
    Q = [c.normal(8, "bf16").cuda() for c in cases]
    want = [sg.kv8_attend(q, c, *a, max_new=1) for q, c, a in zip(Q, caches, args)]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for q, c, a in zip(Q, caches, args):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(sg.kv8_attend(q, c, *a, max_new=1))
        graphs.append(graph)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(4):
        for s, graph, o in zip(streams, graphs, outs):
            with torch.cuda.stream(s):
                o.zero_()
                graph.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w)
    for _ in range(4):
        eager = []
        for s, q, c, a in zip(streams, Q, caches, args):
            with torch.cuda.stream(s):
                eager.append(sg.kv8_attend(q, c, *a, max_new=1))
        torch.cuda.synchronize()
        for o, w in zip(eager, want):
            assert torch.equal(o, w)
    del graphs


def test_a_given_workspace_gives_the_same_bits():
    case = Case(31, [3000, 2000], [2, 2], 2, 32, 64)
    cache, args = case.device(), case.args()
    Q = case.normal(4, "f32").cuda()
    want = sg.kv8_attend(Q, cache, *args, max_new=2)
    batch = sg.KV8Batch(*[t.data_ptr() for t in args], 2, args[0].shape[1], 4, 2)
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    need = sg.sgemm_kv8_attend_workspace_size(cache._struct, batch, 4, 0, cus)
    assert need > 0
    ws = torch.full((need + 64,), 0x7F, dtype=torch.uint8, device="cuda")
    out = sg.kv8_attend(Q, cache, *args, max_new=2, workspace=ws[:need])
    assert torch.equal(out, want)
    assert (ws[need:] == 0x7F).all()
    # One that is too small, or not 16-byte aligned, is not used: the tokens are not split.
    plain = sg.kv8_attend(Q, cache, *args, max_new=2, workspace=torch.empty(0, device="cuda"))
    for small in (ws[:need - 1], ws[1:need + 1]):
        small.fill_(0x55)
        assert torch.equal(sg.kv8_attend(Q, cache, *args, max_new=2, workspace=small), plain)
        assert (small == 0x55).all()


def test_offsets_past_31_bits():
    # A cache of more than 2^31 code bytes, with a sequence in its last pages.
    pages, heads, block, dim = 4200, 8, 256, 256
    cache = sg.KV8.empty(pages, heads, block, dim)
    assert cache.K.numel() > 2**31
    g = torch.Generator().manual_seed(4)
    n = 300
    K, V, Q = (torch.randn(n, heads, dim, generator=g) for _ in range(3))
    table = torch.tensor([[pages - 1, pages - 3]], dtype=torch.int32).cuda()
    lens, starts = torch.tensor([n], dtype=torch.int32).cuda(), torch.tensor([0, n], dtype=torch.int32).cuda()
    sg.kv8_write(cache, K.cuda(), V.cuda(), table, lens, starts)
    small = ref.Cache(*[np.zeros((2, heads, block, dim), np.uint8) for _ in range(2)], *[np.zeros((2, heads)) for _ in range(2)])
    t = np.array([[1, 0]], np.int32)
    small.write([K.double().numpy(), V.double().numpy()], t, [n], [0, n])
    outs = sg.kv8_read(cache, table, lens, starts, rows=n)
    for i in range(2):
        assert np.array_equal(outs[i].cpu().double().numpy(), small.tokens(t, 0, n, i))
    last = torch.tensor([0, 4], dtype=torch.int32).cuda()
    O, bound = small.attend(Q[:4].double().numpy(), t, [n], [0, 4], dim**-0.5, True, 0)
    got = sg.kv8_attend(Q[:4].cuda(), cache, table, lens, last).cpu().double().numpy()
    close(got, O, bound, "last pages")


def test_large_matrix_offsets():
    # Codes and results past 2^31 bytes: the last columns of a tall matrix.
    N, K = 36000, 131072
    codes = torch.zeros((N, K // 2), dtype=torch.uint8, device="cuda")
    assert codes.numel() > 2**31
    codes.fill_(0x88)  # all zero
    g = torch.Generator().manual_seed(1)
    tail = torch.randint(0, 256, (4, K // 2), generator=g, dtype=torch.uint8)
    codes[-4:] = tail.cuda()
    scales = torch.full((N, K // 128), 0.01, device="cuda")
    W = sg.W4(codes, scales, None, K, 128)
    dense = ref.w4_matrix(tail.numpy(), np.full((4, K // 128), np.float32(0.01)), None, K, 128)
    for M in (1, 40):
        A = torch.randn(M, K, generator=g).bfloat16()
        C = sg.gemm_w4(A.cuda(), W)
        assert (C[:, :-4] == 0).all()
        a = A.double().numpy()
        assert_within(C[:, -4:].cpu().numpy(), a @ dense.T, np.abs(a) @ np.abs(dense).T, f"{M} rows")


def test_the_helpers_refuse():
    # Wrong kinds, types, sizes, strides and places of every tensor; nothing is launched.
    case = Case(41, [40, 20], [2, 1], 2, 16, 64)
    cache, (table, lens, starts) = case.device(), case.args()
    K, Q = case.normal(2, "f32").cuda(), case.normal(4, "bf16").cuda()
    W = sg.quantize_w4(torch.randn(32, 64, device="cuda"), 32, True)
    A, C = torch.randn(3, 64, device="cuda"), torch.zeros(3, 32, device="cuda")
    wide = torch.randn(3, 4, 128, device="cuda")
    bad = {
        TypeError: [
            lambda: sg.kv8_write(cache, K.double(), K, table, lens, starts), lambda: sg.kv8_write(cache, K, K.half(), table, lens, starts),
            lambda: sg.kv8_write(cache, K, K, table.long(), lens, starts), lambda: sg.kv8_write(cache, K, K, table, lens.float(), starts),
            lambda: sg.kv8_write(cache, K, K, table[0], lens, starts), lambda: sg.kv8_write(cache, K[0], K, table, lens, starts),
            lambda: sg.kv8_read(cache, table, lens, starts, rows=3, dtype=torch.float64),
            lambda: sg.kv8_attend(Q, cache, table, lens, starts, out=torch.zeros(Q.shape, device="cuda").half()),
            lambda: sg.kv8_attend(Q.int(), cache, table, lens, starts), lambda: sg.kv8_attend(Q, W, table, lens, starts),
            lambda: sg.gemm_w4(A.double(), W), lambda: sg.gemm_w4(A, W, C.half()), lambda: sg.gemm_w4(A, W.codes),
            lambda: sg.dequantize_w4(W, torch.int32), lambda: sg.dequantize_w4(W, torch.float16, torch.zeros(32, 64, device="cuda")),
            lambda: sg.W4(W.codes.int(), W.scales, None, 64, 32), lambda: sg.W4(W.codes, W.scales, W.scales, 64, 32),
            lambda: sg.KV8(cache.K.view(torch.uint8), cache.V, cache.Ks, cache.Vs), lambda: sg.KV8(cache.K, cache.V, cache.Ks.half(), cache.Vs),
        ],
        ValueError: [
            lambda: sg.kv8_write(cache, K.cpu(), K, table, lens, starts), lambda: sg.kv8_write(cache, K, K, table.cpu(), lens, starts),
            lambda: sg.kv8_write(cache, K, K[:2], table, lens, starts), lambda: sg.kv8_write(cache, K[:, :, :32], K, table, lens, starts),
            lambda: sg.kv8_write(cache, K, K, table, lens[:1], starts), lambda: sg.kv8_write(cache, K, K, table, lens, starts[:2]),
            lambda: sg.kv8_write(cache, K, K, table.t().contiguous().t(), lens, starts), lambda: sg.kv8_write(cache, Q.float(), K, table, lens, starts),
            lambda: sg.kv8_write(cache, K.transpose(1, 2).contiguous().transpose(1, 2), K, table, lens, starts),
            lambda: sg.kv8_read(cache, table, lens, starts), lambda: sg.kv8_read(cache, table, lens, starts, K=K),
            lambda: sg.kv8_read(cache, table, lens, starts, rows=4, K=K, V=K.clone()),
            lambda: sg.kv8_attend(wide, cache, table, lens, starts), lambda: sg.kv8_attend(Q, cache, table, lens, starts, out=K),
            lambda: sg.kv8_attend(Q, cache, table, lens, starts, workspace=torch.zeros(8)),
            lambda: sg.gemm_w4(A.cpu(), W), lambda: sg.gemm_w4(A[:, :63], W), lambda: sg.gemm_w4(A, W, C[:2]), lambda: sg.gemm_w4(A, W, beta=1.0),
            lambda: sg.gemm_w4(A.t().contiguous().t(), W), lambda: sg.gemm_w4(A[:1].expand(3, 64), W),
            lambda: sg.dequantize_w4(W, out=torch.zeros(32, 63, device="cuda")), lambda: sg.quantize_w4(A, 48),
            lambda: sg.W4(W.codes, W.scales, None, 66, 32), lambda: sg.W4(W.codes, W.scales[:, :1], None, 64, 32),
            lambda: sg.W4(W.codes.cpu(), W.scales, None, 64, 32), lambda: sg.KV8(cache.K.cpu(), cache.V.cpu(), cache.Ks.cpu(), cache.Vs.cpu()),
            lambda: sg.KV8(cache.K, cache.V, cache.Ks[:1], cache.Vs), lambda: sg.KV8(cache.K[:, :, :12], cache.V[:, :, :12], cache.Ks, cache.Vs),
        ],
        sg.SgemmError: [
            lambda: sg.kv8_attend(Q[:, :3].contiguous(), cache, table, lens, starts), lambda: sg.kv8_attend(Q, cache, table, lens, starts, causal=False, window=4),
            lambda: sg.kv8_attend(K[:1].expand(3, 2, 64), cache, table, lens, starts), lambda: sg.kv8_read(cache, table, lens, starts, K=K, V=K),
            lambda: sg.gemm_w4(A, W, A[:, :32]), lambda: sg.kv8_attend(K, cache, table, lens, starts, out=K),
        ],
    }
    before = [t.clone() for t in (cache.K.view(torch.uint8), cache.Ks, A, K)]
    for error, calls in bad.items():
        for i, call in enumerate(calls):
            with pytest.raises(error):
                call()
                pytest.fail(f"{error.__name__} {i} was not refused")
    assert all(torch.equal(x, y) for x, y in zip(before, (cache.K.view(torch.uint8), cache.Ks, A, K)))


def test_calls_with_nothing_to_do():
    case = Case(42, [40, 20], [0, 0], 2, 16, 64)
    cache, args = case.device(), case.args()
    none = torch.empty(0, 2, 64, device="cuda")
    sg.kv8_write(cache, none, none, *args)
    assert [t.shape for t in sg.kv8_read(cache, *args, rows=0)] == [none.shape] * 2 and sg.kv8_attend(none, cache, *args).shape == none.shape
    empty = [args[0][:0], args[1][:0], args[2][:1]]
    out = torch.full((3, 2, 64), 2.5, device="cuda")
    sg.kv8_write(cache, out, out, *empty)
    assert (sg.kv8_attend(torch.zeros_like(out), cache, *empty, out=out) == 2.5).all()
    same_cache(cache, case.ref, "nothing written")
    for N, K in ((0, 64), (5, 0)):
        W = sg.quantize_w4(torch.empty(N, K, device="cuda"), 32, True)
        assert sg.dequantize_w4(W).shape == (N, K)
        assert (sg.gemm_w4(torch.empty(2, K, device="cuda"), W) == torch.zeros(2, N, device="cuda")).all()
        assert (sg.gemm_w4(torch.empty(2, K, device="cuda"), W, torch.full((2, N), 3.0, device="cuda"), beta=0.5) == 1.5).all()
    W = sg.quantize_w4(torch.randn(32, 64, device="cuda"), 32)
    assert sg.gemm_w4(torch.empty(0, 64, device="cuda"), W).shape == (0, 32)

"""A serving step as a program runs it: page tables, rotary positions, the 4-bit
cache and attention together, captured and replayed, on two streams (GPU
tests)."""

import numpy as np
import pytest
import torch

import dense_fp32_matrix_sgemm_amd as sg
from oracle.check import assert_within
from tests import step_ref as ref
from tests.test_parity_kv4 import Case4, close, same_cache
from tests.test_parity_rope import check as check_rope

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sg.load_library()


class Server:
    """Sequences that grow step by step, and the attention half of a block: x
    -> q, k, v (4-bit products) -> turned by their positions -> cache ->
    attention -> 4-bit product. All of a step's tables are made on the GPU."""

    def __init__(self, seed, seqs, pages, columns, width=256, heads=2, ratio=3, dim=64, block=16, interleaved=False):
        g = torch.Generator().manual_seed(seed)
        self.seqs, self.heads, self.ratio, self.dim, self.block, self.interleaved = seqs, heads, ratio, dim, block, interleaved
        self.w = {}
        for name, n, k in (("q", heads * ratio * dim, width), ("k", heads * dim, width), ("v", heads * dim, width), ("o", width, heads * ratio * dim)):
            self.w[name] = sg.quantize_w4((torch.randn(n, k, generator=g) / k**0.5).cuda(), 64, True, torch.float16)
        self.cache = sg.KV4.empty(pages, heads, block, dim)
        self.freqs, self.amplitude = sg.rope_frequencies(dim, stretch=4.0, original=64)
        self.pool = torch.randperm(pages, generator=g).to(torch.int32)
        self.state = {"pool": self.pool.cuda(), "taken": torch.zeros(1, dtype=torch.int32).cuda(),
                      "table": torch.full((seqs, columns), -1, dtype=torch.int32).cuda(), "lens": torch.zeros(seqs, dtype=torch.int32).cuda()}
        zeros = np.zeros((pages, heads, block, dim // 2), np.uint8), np.zeros((pages, heads, block))
        self.ref = ref.Cache(zeros[0], zeros[0], zeros[1], zeros[1])
        self.host = {"taken": 0, "table": np.full((seqs, columns), -1, np.int32), "lens": np.zeros(seqs, np.int64)}

    def step(self, x, new, max_new):
        """One step of x.shape[0] rows, new of them for each sequence (both on the GPU)."""
        s, rows = self.state, x.shape[0]
        s["lens"] += new
        tables = sg.kv_tables(s["table"], s["lens"], new, s["pool"], s["taken"], self.block, rows, taken_after=s["taken"])
        starts, positions = tables[:2]
        q, k, v = (sg.gemm_w4(x, self.w[n]).view(rows, -1, self.dim) for n in "qkv")
        Q, K = sg.rope(q, k, positions, self.freqs, interleaved=self.interleaved, amplitude=self.amplitude)
        sg.kv4_write(self.cache, K, v, s["table"], s["lens"], starts, max_new=max_new)
        o = sg.kv4_attend(Q, self.cache, s["table"], s["lens"], starts, max_new=max_new)
        return (*tables, q, k, v, Q, K, o, sg.gemm_w4(o.view(rows, -1), self.w["o"]))

    def check(self, x, new, outs, what):
        """Each output against its definition on the inputs that the library's call had."""
        starts, positions, slots, taken, q, k, v, Q, K, o, y = (t.cpu() for t in outs)
        h, rows = self.host, x.shape[0]
        h["lens"] = h["lens"] + new
        want = ref.tables(h["table"], h["lens"], new, self.pool.numpy(), h["taken"], self.block, rows)
        h["taken"], h["table"] = want[3], want[4]
        for got, w, name in zip((starts, positions, slots), want, ("starts", "positions", "slots")):
            assert np.array_equal(got.numpy()[:len(w)], w), (what, name)
        assert int(taken) == h["taken"] and np.array_equal(self.state["table"].cpu().numpy(), h["table"]), what
        check_rope(q, k, want[1], self.freqs.cpu().numpy(), (Q, K), "f32", self.interleaved, self.amplitude, what=what)
        self.ref.write([K.double().numpy(), v.double().numpy()], h["table"], h["lens"], want[0])
        O, bound = self.ref.attend(Q.double().numpy(), h["table"], h["lens"], want[0], self.dim**-0.5, True, 0)
        close(o.double().numpy(), O, bound, f"{what} attention")
        a, dense = o.double().numpy().reshape(rows, -1), sg.dequantize_w4(self.w["o"]).cpu().double().numpy()
        assert_within(y.numpy(), a @ dense.T, np.abs(a) @ np.abs(dense).T, f"{what} y")


def gpu(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


@pytest.mark.parametrize("interleaved", [False, True])
def test_prompts_then_tokens(interleaved):
    server = Server(1, 4, 40, 8, interleaved=interleaved)
    g = torch.Generator().manual_seed(2)
    for step, new in enumerate(([20, 7, 0, 33], [1, 1, 40, 1], [1, 1, 1, 1], [0, 9, 1, 1], [1, 1, 1, 15])):
        x = torch.randn(sum(new), 256, generator=g).cuda()
        outs = server.step(x, gpu(new), max(new))
        server.check(x, np.array(new), outs, f"step {step}")
    same_cache(server.cache, server.ref, "after the steps")


def test_a_captured_step_replayed():
    # The whole step in one graph: lengths, table and counter go on from replay to replay.
    server = Server(5, 2, 400, 150, ratio=4, dim=128, heads=1, block=32)
    g = torch.Generator().manual_seed(6)
    prompt = torch.randn(4700, 256, generator=g).cuda()
    outs = server.step(prompt, gpu([2600, 2100]), 2600)
    # Only the tables and the cache of the prompt are checked; its attention would take the reference long.
    h = server.host
    h["lens"] = np.array([2600, 2100])
    want = ref.tables(h["table"], h["lens"], [2600, 2100], server.pool.numpy(), 0, 32, 4700)
    h["taken"], h["table"] = want[3], want[4]
    assert np.array_equal(server.state["table"].cpu().numpy(), h["table"])
    server.ref.write([outs[8].cpu().double().numpy(), outs[6].cpu().double().numpy()], h["table"], h["lens"], want[0])
    same_cache(server.cache, server.ref, "prompt")
    x, new = torch.zeros(2, 256, device="cuda"), gpu([1, 1])
    saved = {k: t.clone() for k, t in server.state.items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        server.step(x, new, 1)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = server.step(x, new, 1)
    for k, t in saved.items():  # what the trial took is given back
        server.state[k].copy_(t)
    for replay in range(4):
        x.copy_(torch.randn(2, 256, generator=torch.Generator().manual_seed(replay)))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        server.check(x, np.array([1, 1]), outs, f"replay {replay}")
        same_cache(server.cache, server.ref, f"replay {replay}")
        torch.matmul(x, x.t()).sum().item()  # eager work between replays
    del graph


def test_two_graphs_and_two_streams_do_not_share_scratch():
    cases = [Case4(20 + i, [5000 - 700 * i], [1], 1, 32, 128) for i in range(2)]
    caches, args = [c.device() for c in cases], [c.args() for c in cases]
    Q = [c.normal(8, "bf16").cuda() for c in cases]
    want = [sg.kv4_attend(q, c, *a, max_new=1) for q, c, a in zip(Q, caches, args)]
    torch.cuda.synchronize()
    graphs, outs = [], []
    for q, c, a in zip(Q, caches, args):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(sg.kv4_attend(q, c, *a, max_new=1))
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
                eager.append(sg.kv4_attend(q, c, *a, max_new=1))
        torch.cuda.synchronize()
        for o, w in zip(eager, want):
            assert torch.equal(o, w)
    del graphs


def test_a_given_workspace_gives_the_same_bits():
    case = Case4(31, [3000, 2000], [2, 2], 2, 32, 64)
    cache, args = case.device(), case.args()
    Q = case.normal(4, "f32").cuda()
    want = sg.kv4_attend(Q, cache, *args, max_new=2)
    batch = sg.KV8Batch(*[t.data_ptr() for t in args], 2, args[0].shape[1], 4, 2)
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    need = sg.sgemm_kv4_attend_workspace_size(cache._struct, batch, 4, 0, cus)
    assert need > 0
    ws = torch.full((need + 64,), 0x7F, dtype=torch.uint8, device="cuda")
    out = sg.kv4_attend(Q, cache, *args, max_new=2, workspace=ws[:need])
    assert torch.equal(out, want)
    assert (ws[need:] == 0x7F).all()
    # One that is too small, or not 16-byte aligned, is not used: the tokens are not split.
    plain = sg.kv4_attend(Q, cache, *args, max_new=2, workspace=torch.empty(0, device="cuda"))
    for small in (ws[:need - 1], ws[1:need + 1]):
        small.fill_(0x55)
        assert torch.equal(sg.kv4_attend(Q, cache, *args, max_new=2, workspace=small), plain)
        assert (small == 0x55).all()


def test_offsets_past_31_bits():
    # A cache of more than 2^31 code bytes, with a sequence in its last pages.
    pages, heads, block, dim = 8400, 8, 256, 256
    cache = sg.KV4.empty(pages, heads, block, dim)
    assert cache.K.numel() > 2**31
    g = torch.Generator().manual_seed(4)
    n = 300
    K, V, Q = (torch.randn(n, heads, dim, generator=g) for _ in range(3))
    table = torch.tensor([[pages - 1, pages - 3]], dtype=torch.int32).cuda()
    lens, starts = torch.tensor([n], dtype=torch.int32).cuda(), torch.tensor([0, n], dtype=torch.int32).cuda()
    sg.kv4_write(cache, K.cuda(), V.cuda(), table, lens, starts)
    small = ref.Cache(*[np.zeros((2, heads, block, dim // 2), np.uint8) for _ in range(2)], *[np.zeros((2, heads, block)) for _ in range(2)])
    t = np.array([[1, 0]], np.int32)
    small.write([K.double().numpy(), V.double().numpy()], t, [n], [0, n])
    outs = sg.kv4_read(cache, table, lens, starts, rows=n)
    for i in range(2):
        assert np.array_equal(outs[i].cpu().double().numpy(), small.tokens(t, 0, n, i))
    last = torch.tensor([0, 4], dtype=torch.int32).cuda()
    O, bound = small.attend(Q[:4].double().numpy(), t, [n], [0, 4], dim**-0.5, True, 0)
    got = sg.kv4_attend(Q[:4].cuda(), cache, table, lens, last).cpu().double().numpy()
    close(got, O, bound, "last pages")


def test_the_helpers_refuse():
    # Wrong kinds, types, sizes, strides and places of every tensor; nothing is launched.
    case = Case4(41, [40, 20], [2, 1], 2, 16, 64)
    cache, (table, lens, starts) = case.device(), case.args()
    K, Q = case.normal(2, "f32").cuda(), case.normal(4, "bf16").cuda()
    other = sg.KV8.empty(2, 2, 16, 64)
    bad = {
        TypeError: [
            lambda: sg.kv4_write(cache, K.double(), K, table, lens, starts), lambda: sg.kv4_write(cache, K, K.half(), table, lens, starts),
            lambda: sg.kv4_write(cache, K, K, table.long(), lens, starts), lambda: sg.kv4_write(other, K, K, table, lens, starts),
            lambda: sg.kv4_read(cache, table, lens, starts, rows=3, dtype=torch.float64), lambda: sg.kv8_attend(Q, cache, table, lens, starts),
            lambda: sg.kv4_attend(Q, cache, table, lens, starts, out=torch.zeros(Q.shape, device="cuda").half()),
            lambda: sg.kv4_attend(Q.int(), cache, table, lens, starts), lambda: sg.kv4_attend(Q, other, table, lens, starts),
            lambda: sg.KV4(cache.K.view(torch.int8), cache.V, cache.Ks, cache.Vs), lambda: sg.KV4(cache.K, cache.V, cache.Ks.float(), cache.Vs),
        ],
        ValueError: [
            lambda: sg.kv4_write(cache, K.cpu(), K, table, lens, starts), lambda: sg.kv4_write(cache, K, K[:2], table, lens, starts),
            lambda: sg.kv4_write(cache, K[:, :, :32], K, table, lens, starts), lambda: sg.kv4_write(cache, K, K, table, lens[:1], starts),
            lambda: sg.kv4_write(cache, Q.float(), K, table, lens, starts), lambda: sg.kv4_read(cache, table, lens, starts),
            lambda: sg.kv4_read(cache, table, lens, starts, K=K), lambda: sg.kv4_read(cache, table, lens, starts, rows=4, K=K, V=K.clone()),
            lambda: sg.kv4_attend(Q, cache, table, lens, starts, out=K), lambda: sg.kv4_attend(Q, cache, table, lens, starts, workspace=torch.zeros(8)),
            lambda: sg.KV4(cache.K, cache.V, cache.Ks[:1], cache.Vs), lambda: sg.KV4(cache.K[:, :, :12], cache.V[:, :, :12], cache.Ks[:, :, :12], cache.Vs[:, :, :12]),
            lambda: sg.KV4(cache.K[..., :12].contiguous(), cache.V[..., :12].contiguous(), cache.Ks, cache.Vs),
            lambda: sg.KV4(*(torch.zeros(2 * 2 * 16 * 32 + 8, dtype=torch.uint8, device="cuda")[8:].view(2, 2, 16, 32) for _ in range(2)), cache.Ks[:2], cache.Vs[:2]),
        ],
        sg.SgemmError: [
            lambda: sg.kv4_attend(Q[:, :3].contiguous(), cache, table, lens, starts), lambda: sg.kv4_attend(Q, cache, table, lens, starts, causal=False, window=4),
            lambda: sg.kv4_attend(K[:1].expand(3, 2, 64), cache, table, lens, starts), lambda: sg.kv4_read(cache, table, lens, starts, K=K, V=K),
            lambda: sg.kv4_attend(K, cache, table, lens, starts, out=K),
            lambda: sg.kv4_write(sg.KV4(cache.K, cache.K, cache.Ks, cache.Vs), K, K, table, lens, starts),
            lambda: sg.kv4_write(sg.KV4(cache.K, cache.V, cache.Ks, cache.Ks), K, K, table, lens, starts),
        ],
    }
    before = [t.clone() for t in (cache.K, cache.V, cache.Ks, cache.Vs, K)]
    for error, calls in bad.items():
        for i, call in enumerate(calls):
            with pytest.raises(error):
                call()
                pytest.fail(f"{error.__name__} {i} was not refused")
    assert all(torch.equal(x, y) for x, y in zip(before, (cache.K, cache.V, cache.Ks, cache.Vs, K)))


def test_keys_that_are_the_values():
    # One tensor for both may be read and attended over.
    case = Case4(43, [100, 20], [1, 4], 2, 16, 64)
    case.ref.codes[1], case.ref.scales[1] = case.ref.codes[0], case.ref.scales[0]
    K, Ks = torch.from_numpy(case.ref.codes[0]).cuda(), torch.from_numpy(case.ref.scales[0]).cuda().to(torch.bfloat16)
    cache, Q = sg.KV4(K, K, Ks, Ks), case.normal(4, "f32")
    O, bound = case.ref.attend(Q.double().numpy(), case.table, case.lens, case.starts, 0.2, True, 0)
    close(sg.kv4_attend(Q.cuda(), cache, *case.args(), scale=0.2).cpu().double().numpy(), O, bound, "shared")
    k, v = sg.kv4_read(cache, *case.args(), rows=case.rows)
    assert torch.equal(k, v)


def test_calls_with_nothing_to_do():
    case = Case4(42, [40, 20], [0, 0], 2, 16, 64)
    cache, args = case.device(), case.args()
    none = torch.empty(0, 2, 64, device="cuda")
    sg.kv4_write(cache, none, none, *args)
    assert [t.shape for t in sg.kv4_read(cache, *args, rows=0)] == [none.shape] * 2 and sg.kv4_attend(none, cache, *args).shape == none.shape
    empty = [args[0][:0], args[1][:0], args[2][:1]]
    out = torch.full((3, 2, 64), 2.5, device="cuda")
    sg.kv4_write(cache, out, out, *empty)
    assert (sg.kv4_attend(torch.zeros_like(out), cache, *empty, out=out) == 2.5).all()
    same_cache(cache, case.ref, "nothing written")

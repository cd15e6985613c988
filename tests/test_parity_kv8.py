"""The 8-bit cache of keys and values: writing, reading back and attending,
against their definitions in 64 bits (GPU tests)."""

import numpy as np
import pytest
import torch

import dense_fp32_matrix_sgemm_amd as sg
from tests import lowbit_ref as ref

pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sg.load_library()


class Case:
    """A cache with random pages, a table of distinct pages in random order
    (-1 behind each sequence's last), on both sides."""

    def __init__(self, seed, lens, new, heads, block, dim, spare=3, columns=None, before=0, behind=0):
        self.rng = np.random.default_rng(seed)
        self.heads, self.block, self.dim, self.new = heads, block, dim, new
        used = [-(-max(l, 0) // block) for l in lens]
        pages = sum(used) + spare
        columns = max(used + [1]) if columns is None else columns
        ids = self.rng.permutation(pages)
        self.table = np.full((len(lens), columns), -1, np.int32)
        at = 0
        for b, u in enumerate(used):
            self.table[b, :u] = ids[at:at + u][:columns]
            at += u
        self.lens = np.array(lens, np.int32)
        self.starts = (before + np.concatenate([[0], np.cumsum(new)])).astype(np.int32)
        self.rows = int(self.starts[-1]) + behind
        shape = (pages, heads, block, dim)
        K, V = (ref.e4m3(np.clip(self.rng.standard_normal(shape) * 64, -448, 448)) for _ in range(2))
        Ks, Vs = (np.exp2(self.rng.integers(-8, -4, (pages, heads))).astype(np.float32) for _ in range(2))
        self.ref = ref.Cache(K, V, Ks, Vs)

    def device(self):
        f8 = [torch.from_numpy(x).cuda().view(torch.float8_e4m3fn) for x in self.ref.codes]
        scales = [torch.from_numpy(x.astype(np.float32)).cuda() for x in self.ref.scales]
        return sg.KV8(*f8, *scales)

    def args(self):
        return [torch.from_numpy(x).cuda() for x in (self.table, self.lens, self.starts)]

    def normal(self, heads, dtype, scale=1.0):
        return torch.from_numpy(self.rng.standard_normal((self.rows, heads, self.dim)) * scale).to(TYPES[dtype])


def views(t, layout):
    """t on the GPU with rows x heads x dim strides of another layout, NaN between the elements."""
    rows, heads, dim = t.shape
    if layout == "packed":
        return t.cuda()
    if layout == "padded":
        buf = torch.full((rows, heads + 1, dim + 8), float("nan"), dtype=t.dtype)
        buf[:, :heads, :dim] = t
        return buf.cuda()[:, :heads, :dim]
    buf = torch.full((heads, rows + 2, dim), float("nan"), dtype=t.dtype)  # heads outermost
    buf[:, :rows] = t.transpose(0, 1)
    return buf.cuda()[:, :rows].transpose(0, 1)


def same_cache(cache, want, what):
    for name, got, codes in (("K", cache.K, want.codes[0]), ("V", cache.V, want.codes[1])):
        got = got.view(torch.uint8).cpu().numpy()
        nan = (codes & 0x7F) == 0x7F
        assert np.array_equal((got & 0x7F) == 0x7F, nan), (what, name, "NaN")
        assert np.array_equal(np.where(nan, 0, got), np.where(nan, 0, codes)), (what, name)
    for got, scales in ((cache.Ks, want.scales[0]), (cache.Vs, want.scales[1])):
        assert np.array_equal(got.cpu().double().numpy(), scales), (what, "scales")


# (lens, new rows): one token, none, a page filled exactly, a page begun,
# rows over several pages, whole prompts, an empty sequence between others.
BATCHES = [([1], [1]), ([16, 17, 33], [1, 1, 1]), ([0, 40, 0, 7], [0, 5, 0, 7]), ([130, 64, 31], [130, 20, 1]),
           ([16, 32, 48, 300], [16, 32, 1, 47])]


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("block,dim,heads", [(16, 64, 2), (32, 128, 1), (64, 80, 3), (16, 256, 1), (128, 16, 2)])
@pytest.mark.parametrize("batch", BATCHES)
def test_write_and_read(batch, block, dim, heads, dtype):
    lens, new = batch
    print(f"[kv8] write {lens} {new} block={block} dim={dim} heads={heads} {dtype}", flush=True)
    for i, layout in enumerate(("packed", "padded", "heads")):
        case = Case(len(lens) + i, lens, new, heads, block, dim, before=i, behind=2 * i)
        cache, args = case.device(), case.args()
        # Some rows larger than their page's scale allows, so that scales rise.
        size = torch.from_numpy(np.exp2(case.rng.integers(-3, 5, (case.rows, 1, 1)))).float()
        K, V = (case.normal(heads, dtype) * size.to(TYPES[dtype]) for _ in range(2))
        for t in (K, V):
            t[:, :, dim // 2] = 0
        case.ref.write([K.double().numpy(), V.double().numpy()], case.table, case.lens, case.starts)
        sg.kv8_write(cache, views(K, layout), views(V, layout), *args, max_new=max(new) if i else 1)
        torch.cuda.synchronize()
        same_cache(cache, case.ref, layout)
        # Everything read back, into every layout and type; rows outside the sequences stay.
        starts = (i + np.concatenate([[0], np.cumsum(lens)])).astype(np.int32)
        rows = int(starts[-1]) + i
        for out in ("f32", "bf16", "f16"):
            outs = [views(torch.full((rows, heads, dim), 3.25, dtype=TYPES[out]), layout) for _ in range(2)]
            sg.kv8_read(cache, args[0], args[1], torch.from_numpy(starts).cuda(), K=outs[0], V=outs[1])
            for j in range(2):
                want = np.full((rows, heads, dim), 3.25)
                for b, l in enumerate(lens):
                    want[starts[b]:starts[b + 1]] = case.ref.tokens(case.table, b, l, j)
                want = torch.from_numpy(want).float().to(TYPES[out])
                assert torch.equal(outs[j].cpu(), want), (layout, out, j)


def test_scales_rise_and_keep_what_was_written():
    # A page filled token by token holds what it holds when written at once, but for subnormals.
    heads, block, dim = 2, 32, 64
    whole, single = (Case(7, [32], [32], heads, block, dim) for _ in range(2))
    x = torch.randn(32, heads, dim, generator=torch.Generator().manual_seed(8)).abs() * 0.5 + 0.5
    x = x * torch.exp2(torch.arange(32).float() / 8)[:, None, None]  # 16 times larger at the end: no subnormals
    a, b = whole.device(), single.device()
    sg.kv8_write(a, x.cuda(), x.cuda(), *whole.args())
    one = torch.tensor([0, 1], dtype=torch.int32).cuda()
    for t in range(32):
        lens = torch.tensor([t + 1], dtype=torch.int32).cuda()
        row = x[t:t + 1].cuda()
        sg.kv8_write(b, row, row, torch.from_numpy(single.table).cuda(), lens, one, max_new=1)
    page = int(whole.table[0, 0])
    assert torch.equal(a.Ks[page], b.Ks[page]) and torch.equal(a.K.view(torch.uint8)[page], b.K.view(torch.uint8)[page])
    assert torch.equal(a.Vs[page], b.Vs[page]) and torch.equal(a.V.view(torch.uint8)[page], b.V.view(torch.uint8)[page])


def test_write_borders():
    # Zeros, values at a power's border, the ends of float32, infinities and NaN.
    heads, block, dim = 1, 16, 64
    rows = [torch.zeros(dim) for _ in range(7)]
    rows[1][0] = 448.0
    rows[2][0] = float(np.nextafter(np.float32(448), np.float32(1000)))
    rows[3][:4] = torch.tensor([1e-45, -1e-44, 1e-40, 0.0])
    rows[4][:3] = torch.tensor([3.0e38, -1.0, 1e-3])
    rows[5][:4] = torch.tensor([float("inf"), -float("inf"), 2.0, -3.0])
    rows[6][:3] = torch.tensor([float("nan"), 448 * 2.0**-9, 17.0])
    for i, row in enumerate(rows):
        case = Case(i, [18], [1], heads, block, dim)
        cache = case.device()
        x = row.view(1, 1, dim)
        case.ref.write([x.double().numpy(), -x.double().numpy()], case.table, case.lens, case.starts)
        sg.kv8_write(cache, x.cuda(), -x.cuda(), *case.args())
        same_cache(cache, case.ref, i)


def test_bad_tables_are_not_followed():
    # Pages that are not the cache's, columns that are not the table's, lengths
    # below 0, rows before token 0, starts that fall or lie outside.
    heads, block, dim = 2, 16, 64
    case = Case(3, [40, 40, 20, -5, 3, 70], [40, 24, 20, 4, 5, 10], heads, block, dim, columns=3)
    case.table[0, 1], case.table[1, 2], case.table[2, 0] = 10**6, -7, case.ref.pages
    K, V = case.normal(heads, "f32"), case.normal(heads, "f32")
    cache, args = case.device(), case.args()
    case.ref.write([K.double().numpy(), V.double().numpy()], case.table, case.lens, case.starts)
    sg.kv8_write(cache, K.cuda(), V.cuda(), *args)
    same_cache(cache, case.ref, "bad pages")
    outs = sg.kv8_read(cache, *args, K=torch.full((case.rows, heads, dim), 3.25).cuda(), V=torch.full((case.rows, heads, dim), 3.25).cuda())
    for j in range(2):
        want = np.full((case.rows, heads, dim), 3.25)
        for b in range(6):
            n, l = int(case.starts[b + 1] - case.starts[b]), max(0, int(case.lens[b]))
            t = case.ref.tokens(case.table, b, l, j)[max(0, l - n):]
            want[case.starts[b + 1] - len(t):case.starts[b + 1]] = t
        assert np.array_equal(outs[j].cpu().double().numpy(), want, equal_nan=True)
    Q = case.normal(2 * heads, "f32")
    for causal in (True, False):
        O, bound = case.ref.attend(Q.double().numpy(), case.table, case.lens, case.starts, 0.2, causal, 0)
        got = sg.kv8_attend(Q.cuda(), cache, *args, scale=0.2, causal=causal).cpu().double().numpy()
        close(got, O, bound, f"bad pages causal={causal}")
    for starts in ([5, 2, 9, 9, 200, 300, 7], [-4, 3, 2, -1, 8, 8, 2**31 - 1]):
        case.starts = np.array(starts, np.int32)
        args[2] = torch.from_numpy(case.starts).cuda()
        case.lens = np.array([10, 40, 16, 2, 3, 48], np.int32)
        args[1] = torch.from_numpy(case.lens).cuda()
        got = sg.kv8_attend(Q.cuda(), cache, *args, scale=0.2, out=torch.full(Q.shape, 3.25).cuda()).cpu().double().numpy()
        # Ranges may meet here: only rows of one range are checked, and those of none.
        cover = np.zeros(case.rows, int)
        for b in range(6):
            first, end = np.clip(case.starts[b:b + 2].astype(np.int64), 0, case.rows)
            cover[first:max(first, end)] += 1
        O, bound = case.ref.attend(Q.double().numpy(), case.table, case.lens, case.starts, 0.2, True, 0)
        close(got[cover == 1], O[cover == 1], bound[cover == 1], f"starts {starts}")
        assert (got[cover == 0] == 3.25).all()


# ------------------------------------------------------------- attention


def close(got, want, bound, what):
    assert np.array_equal(np.isnan(got), np.isnan(want)), (what, "NaN")
    ok = ~np.isnan(want)
    off = np.abs(got[ok] - want[ok])
    assert (off <= bound[ok]).all(), (what, float((off / bound[ok]).max()))


def attends(case, ratio, dtype, causal=True, window=0, scale=None, layout="packed", max_new=None, workspace=None, what=""):
    cache, args = case.device(), case.args()
    Q = case.normal(case.heads * ratio, dtype)
    scale_ = case.dim**-0.5 if scale is None else scale
    O, bound = case.ref.attend(Q.double().numpy(), case.table, case.lens, case.starts, scale_, causal, window)
    out = views(torch.full(Q.shape, 3.25), layout)
    sg.kv8_attend(views(Q, layout), cache, *args, scale=scale, causal=causal, window=window, out=out, max_new=max_new,
                  workspace=workspace)
    got = out.cpu().double().numpy()
    inside = np.zeros(case.rows, bool)
    inside[case.starts[0]:case.starts[-1]] = True
    assert (got[~inside] == 3.25).all(), (what, "rows outside the sequences")
    close(got[inside], O[inside], bound[inside], what)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("dim,block", [(16, 16), (64, 32), (80, 16), (128, 64), (208, 16), (256, 128)])
@pytest.mark.parametrize("ratio", [1, 4, 7])
def test_next_token(ratio, dim, block, dtype):
    print(f"[kv8] next token ratio={ratio} dim={dim} block={block} {dtype}", flush=True)
    case = Case(dim + ratio, [1, 15, 16, 17, 0, 33, 127, 129, 300], [1, 1, 1, 1, 0, 1, 1, 1, 1], 2, block, dim, before=1, behind=2)
    for i, layout in enumerate(("packed", "padded", "heads")):
        attends(case, ratio, dtype, layout=layout, max_new=1 if i else None, what=layout)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 1), (True, 40), (True, 1000)])
@pytest.mark.parametrize("heads,ratio,dim,block", [(1, 1, 64, 16), (2, 3, 128, 32), (1, 8, 96, 64), (1, 2, 256, 16)])
def test_several_rows(heads, ratio, dim, block, causal, window, dtype):
    print(f"[kv8] rows heads={heads} ratio={ratio} dim={dim} causal={causal} window={window} {dtype}", flush=True)
    # Prompts whole and behind a cache, rows before token 0, sequences without rows.
    case = Case(dim + window, [70, 200, 31, 50, 3, 260], [70, 9, 31, 0, 5, 130], heads, block, dim)
    attends(case, ratio, dtype, causal, window, what="all rows at once")
    attends(case, ratio, dtype, causal, window, max_new=3, layout="heads", what="a hint that is too small")


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("seqs,length,new,ratio,dim", [(1, 5000, 1, 8, 128), (2, 3000, 4, 4, 128), (1, 9000, 1, 1, 64), (1, 2500, 40, 2, 256), (1, 700, 500, 1, 128)])
def test_long_sequences(seqs, length, new, ratio, dim, dtype):
    print(f"[kv8] long {seqs}x{length} new={new} ratio={ratio} dim={dim} {dtype}", flush=True)
    case = Case(length, [length - 37 * b for b in range(seqs)], [new] * seqs, 1, 32, dim)
    attends(case, ratio, dtype, max_new=new, what="split")
    attends(case, ratio, dtype, max_new=new, workspace=torch.empty(0, device="cuda"), what="not split")
    attends(case, ratio, dtype, max_new=new, window=length // 2, what="split window")
    # A table laid out for far longer sequences.
    case.table = np.concatenate([case.table, np.full((seqs, 2000), -1, np.int32)], axis=1)
    attends(case, ratio, dtype, max_new=new, what="wide table")


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_large_scores(dtype):
    # Softmax of scores up to thousands: one token takes all, or none moves far from the maximum.
    case = Case(11, [300, 64], [5, 64], 2, 16, 64)
    attends(case, 2, dtype, scale=30.0, what="large")
    attends(case, 2, dtype, scale=-2.0, what="negative")
    attends(case, 2, dtype, scale=0.0, what="mean")


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 20), (False, 0)])
def test_nan_reaches_only_rows_that_see_it(causal, window, dtype):
    case = Case(13, [90, 64, 200], [40, 64, 3], 2, 16, 96)
    for b, t, comp in ((0, 60, 5), (1, 33, 95), (2, 100, 0), (0, 88, 17)):
        page = case.table[b, t // 16]
        case.ref.codes[1][page, 1, t % 16, comp] = 0xFF
    case.ref.codes[0][case.table[1, 2], 0, 7, 3] = 0x7F  # a key
    # Behind the last token of a sequence: seen by nobody.
    page = case.table[0, 5]
    case.ref.codes[0][page, :, 10:] = 0x7F
    case.ref.codes[1][page, :, 10:] = 0x7F
    with np.errstate(invalid="ignore"):
        attends(case, 2, dtype, causal, window, what="nan")


def test_two_runs_are_the_same():
    case = Case(17, [3000, 500], [2, 2], 2, 32, 128)
    Q = case.normal(8, "bf16").cuda()
    cache, args = case.device(), case.args()
    first = sg.kv8_attend(Q, cache, *args, max_new=2)
    for _ in range(3):
        assert torch.equal(sg.kv8_attend(Q, cache, *args, max_new=2), first)


@pytest.mark.parametrize("ratio,columns", [(1, 1), (1, 2), (2, 3), (70, 3), (70, 4), (3, 7)])
@pytest.mark.parametrize("window", [0, 5, 40])
def test_rows_past_a_short_table(window, ratio, columns):
    # Lengths behind the table's last column: rows that see only its tokens are
    # as ever, the others NaN, rows before token 0 zero; nothing behind is read.
    block, dim = 16, 64
    case = Case(12, [16 * columns] * 4, [9, 3, 8, 2], 1, block, dim)
    case.lens = np.array([16 * columns + 3, 16 * columns + 200, 6, 2**31 - 1], np.int32)
    cache, args = case.device(), case.args()
    Q = case.normal(ratio, "bf16")
    for max_new in (1, 9):
        O, bound = case.ref.attend(Q.double().numpy(), case.table, case.lens, case.starts, 0.2, True, window)
        assert np.isfinite(O[:6]).all() and np.isnan(O[6:12]).all() and (O[12:14] == 0).all() and np.isnan(O[20:]).all()
        got = sg.kv8_attend(Q.cuda(), cache, *args, scale=0.2, window=window, max_new=max_new).cpu().double().numpy()
        close(got, O, bound, f"columns {columns} window {window} max_new {max_new}")


def test_splits_past_a_short_table():
    # The same where sequences are split over work-groups and joined.
    case = Case(13, [4096, 4096], [4, 3], 1, 64, 128)
    case.lens = np.array([4098, 5000], np.int32)
    cache, args = case.device(), case.args()
    Q = case.normal(2, "bf16")
    for window in (0, 100, 3000):
        O, bound = case.ref.attend(Q.double().numpy(), case.table, case.lens, case.starts, 0.2, True, window)
        assert np.isfinite(O[:2]).all() and np.isnan(O[2:]).all()
        close(sg.kv8_attend(Q.cuda(), cache, *args, scale=0.2, window=window, max_new=4).cpu().double().numpy(), O, bound, f"window {window}")


def test_positions_up_to_31_bits():
    # The last tokens of a sequence of 2^31 - 1, whose table repeats a few pages, through a window.
    block, dim, n, window = 1024, 16, 20, 50
    case = Case(14, [2 * block - 1], [n], 1, block, dim, spare=0)
    cache = case.device()
    K, V, Q = (case.normal(1, "f32") for _ in range(3))
    case.ref.write([K.double().numpy(), V.double().numpy()], case.table, case.lens, case.starts)
    O, bound = case.ref.attend(Q.double().numpy(), case.table, case.lens, case.starts, 0.3, True, window)
    table = torch.full((1, 2**21), -1, dtype=torch.int32)
    table[0, -2:] = torch.from_numpy(case.table[0])
    args = [table.cuda(), torch.tensor([2**31 - 1], dtype=torch.int32).cuda(), torch.from_numpy(case.starts).cuda()]
    sg.kv8_write(cache, K.cuda(), V.cuda(), *args)
    same_cache(cache, case.ref, "last tokens")
    for max_new in (1, n):
        got = sg.kv8_attend(Q.cuda(), cache, *args, scale=0.3, window=window, max_new=max_new).cpu().double().numpy()
        close(got, O, bound, f"last tokens, max_new {max_new}")
    outs = sg.kv8_read(cache, *args, rows=n)
    for i in range(2):
        assert np.array_equal(outs[i].cpu().double().numpy(), case.ref.tokens(case.table, 0, 2 * block - 1, i)[-n:])

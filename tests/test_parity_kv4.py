"""The 4-bit cache of keys and values: writing, reading back and attending,
against their definitions in 64 bits (GPU tests)."""

import numpy as np
import pytest
import torch

import dense_fp32_matrix_sgemm_amd as sg
from tests import step_ref as ref
from tests.test_parity_kv8 import BATCHES, TYPES, Case, close, views

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sg.load_library()


class Case4(Case):
    """The cases of the 8-bit cache's tests, with a 4-bit cache of random codes."""

    def __init__(self, *args, **kw):
        super().__init__(*args, **kw)
        pages = self.ref.pages
        K, V = (self.rng.integers(0, 256, (pages, self.heads, self.block, self.dim // 2)).astype(np.uint8) for _ in range(2))
        Ks, Vs = (ref.bf16(np.exp2(self.rng.uniform(-3, 1, (pages, self.heads, self.block)))) for _ in range(2))
        self.ref = ref.Cache(K, V, Ks, Vs)

    def device(self):
        return sg.KV4(*[torch.from_numpy(x).cuda() for x in self.ref.codes],
                      *[torch.from_numpy(x).cuda().to(torch.bfloat16) for x in self.ref.scales])


def same_cache(cache, want, what):
    """Codes (but for the sign of zeros) and scales."""
    for name, got, codes in (("K", cache.K, want.codes[0]), ("V", cache.V, want.codes[1])):
        assert np.array_equal(ref.values(got.cpu().numpy()), ref.values(codes)), (what, name)
    for got, scales in ((cache.Ks, want.scales[0]), (cache.Vs, want.scales[1])):
        assert np.array_equal(got.cpu().double().numpy(), scales, equal_nan=True), (what, "scales")


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("block,dim,heads", [(16, 64, 2), (32, 128, 1), (64, 80, 3), (16, 256, 1), (128, 16, 2), (16, 48, 35)])
@pytest.mark.parametrize("batch", BATCHES)
def test_write_and_read(batch, block, dim, heads, dtype):
    lens, new = batch
    print(f"[kv4] write {lens} {new} block={block} dim={dim} heads={heads} {dtype}", flush=True)
    for i, layout in enumerate(("packed", "padded", "heads")):
        case = Case4(len(lens) + i, lens, new, heads, block, dim, before=i, behind=2 * i)
        cache, args = case.device(), case.args()
        size = torch.from_numpy(np.exp2(case.rng.integers(-3, 5, (case.rows, 1, 1)))).float()
        K, V = (case.normal(heads, dtype) * size.to(TYPES[dtype]) for _ in range(2))
        for t in (K, V):
            t[:, :, dim // 2] = 0
        case.ref.write([K.double().numpy(), V.double().numpy()], case.table, case.lens, case.starts)
        sg.kv4_write(cache, views(K, layout), views(V, layout), *args, max_new=max(new) if i else 1)
        torch.cuda.synchronize()
        same_cache(cache, case.ref, layout)
        # Everything read back, into every layout and type; rows outside the sequences stay.
        starts = (i + np.concatenate([[0], np.cumsum(lens)])).astype(np.int32)
        rows = int(starts[-1]) + i
        for out in ("f32", "bf16", "f16"):
            outs = [views(torch.full((rows, heads, dim), 3.25, dtype=TYPES[out]), layout) for _ in range(2)]
            sg.kv4_read(cache, args[0], args[1], torch.from_numpy(starts).cuda(), K=outs[0], V=outs[1], max_new=max(lens) if i else 2)
            for j in range(2):
                want = np.full((rows, heads, dim), 3.25)
                for b, l in enumerate(lens):
                    want[starts[b]:starts[b + 1]] = case.ref.tokens(case.table, b, l, j)
                want = torch.from_numpy(want).float().to(TYPES[out])
                assert torch.equal(outs[j].cpu(), want), (layout, out, j)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_rounding_next_to_every_midpoint(dtype):
    # Rows whose largest value fixes the scale, and the numbers of the type on, below and above each midpoint of it.
    block, dim = 16, 64
    rows = []
    for top in (6.0, 1.0, 0.37, 5.99, 250.0, 2.0**-14):
        t = torch.tensor(top).to(TYPES[dtype])
        s = float(ref.scale_of(np.array([[float(t)]]))[0])
        row = [t]
        for m in ref.MIDPOINTS:
            v = torch.tensor(m * s, dtype=torch.float64).to(TYPES[dtype])
            for x in (v, torch.nextafter(v, torch.tensor(0.0, dtype=TYPES[dtype])), torch.nextafter(v, torch.tensor(1e4, dtype=TYPES[dtype]))):
                if float(x) <= float(t):
                    row += [x, -x]
        row = torch.stack(row)[:dim]
        rows.append(torch.cat([row, torch.zeros(dim - len(row), dtype=TYPES[dtype])]))
    x = torch.stack(rows)[:, None]
    case = Case4(2, [len(rows)], [len(rows)], 1, block, dim)
    cache = case.device()
    case.ref.write([x.double().numpy(), -x.double().numpy()], case.table, case.lens, case.starts)
    sg.kv4_write(cache, x.cuda(), -x.cuda(), *case.args())
    same_cache(cache, case.ref, dtype)


def test_write_borders():
    # Zeros, the least scale, the ends of float32, infinities and NaN, subnormals.
    heads, block, dim = 2, 16, 32
    rows = [torch.zeros(heads, dim) for _ in range(8)]
    rows[1][0, 0] = 3.0e38
    rows[1][0, 1:4] = torch.tensor([-2.0e38, 1e30, 1.5e37])
    rows[2][0, 0] = 2.0**-99
    rows[2][1, :3] = torch.tensor([2.0**-101, 2.0**-102, -(2.0**-100)])
    rows[3][:, :4] = torch.tensor([1e-45, -1e-44, 1e-40, 0.0])
    rows[4][0, :4] = torch.tensor([float("inf"), 1.0, 2.0, -3.0])
    rows[4][1, 5] = 7.0
    rows[5][1, :3] = torch.tensor([float("nan"), 4.0, 17.0])
    rows[6][0, :2] = torch.tensor([-float("inf"), float("nan")])
    rows[7][:] = -0.0
    x = torch.stack(rows)
    case = Case4(4, [40], [8], heads, block, dim)
    cache = case.device()
    y = x.flip(0)
    case.ref.write([x.double().numpy(), y.double().numpy()], case.table, case.lens, case.starts)
    sg.kv4_write(cache, x.cuda(), y.cuda(), *case.args())
    same_cache(cache, case.ref, "borders")
    outs = sg.kv4_read(cache, *case.args(), rows=8)
    for j in range(2):
        assert np.array_equal(outs[j].cpu().double().numpy(), case.ref.tokens(case.table, 0, 40, j)[-8:], equal_nan=True)


def test_new_tokens_change_no_older_ones():
    heads, block, dim = 2, 32, 64
    case = Case4(7, [50], [1], heads, block, dim)
    cache = case.device()
    before = [t.clone() for t in (cache.K, cache.V, cache.Ks, cache.Vs)]
    x = (torch.randn(1, heads, dim, generator=torch.Generator().manual_seed(1)) * 1000).cuda()
    sg.kv4_write(cache, x, x, *case.args())
    page, place = int(case.table[0, 1]), 49 % 32
    for a, b in zip(before, (cache.K, cache.V, cache.Ks, cache.Vs)):
        changed = (a != b).flatten(3).any(3) if a.dim() == 4 else a != b
        assert changed[page, :, place].all() and int(changed.sum()) == heads


def test_bad_tables_are_not_followed():
    # Pages that are not the cache's, columns that are not the table's, lengths
    # below 0, rows before token 0, starts that fall or lie outside.
    heads, block, dim = 2, 16, 64
    case = Case4(3, [40, 40, 20, -5, 3, 70], [40, 24, 20, 4, 5, 10], heads, block, dim, columns=3)
    case.table[0, 1], case.table[1, 2], case.table[2, 0] = 10**6, -7, case.ref.pages
    K, V = case.normal(heads, "f32"), case.normal(heads, "f32")
    cache, args = case.device(), case.args()
    case.ref.write([K.double().numpy(), V.double().numpy()], case.table, case.lens, case.starts)
    sg.kv4_write(cache, K.cuda(), V.cuda(), *args)
    same_cache(cache, case.ref, "bad pages")
    outs = sg.kv4_read(cache, *args, K=torch.full((case.rows, heads, dim), 3.25).cuda(), V=torch.full((case.rows, heads, dim), 3.25).cuda())
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
        got = sg.kv4_attend(Q.cuda(), cache, *args, scale=0.2, causal=causal).cpu().double().numpy()
        close(got, O, bound, f"bad pages causal={causal}")
    for starts in ([5, 2, 9, 9, 200, 300, 7], [-4, 3, 2, -1, 8, 8, 2**31 - 1]):
        case.starts = np.array(starts, np.int32)
        args[2] = torch.from_numpy(case.starts).cuda()
        case.lens = np.array([10, 40, 16, 2, 3, 48], np.int32)
        args[1] = torch.from_numpy(case.lens).cuda()
        got = sg.kv4_attend(Q.cuda(), cache, *args, scale=0.2, out=torch.full(Q.shape, 3.25).cuda()).cpu().double().numpy()
        # Ranges may meet here: only rows of one range are checked, and those of none.
        cover = np.zeros(case.rows, int)
        for b in range(6):
            first, end = np.clip(case.starts[b:b + 2].astype(np.int64), 0, case.rows)
            cover[first:max(first, end)] += 1
        O, bound = case.ref.attend(Q.double().numpy(), case.table, case.lens, case.starts, 0.2, True, 0)
        close(got[cover == 1], O[cover == 1], bound[cover == 1], f"starts {starts}")
        assert (got[cover == 0] == 3.25).all()


# ------------------------------------------------------------- attention


def attends(case, ratio, dtype, causal=True, window=0, scale=None, layout="packed", max_new=None, workspace=None, Q=None, what=""):
    cache, args = case.device(), case.args()
    Q = case.normal(case.heads * ratio, dtype) if Q is None else Q
    scale_ = case.dim**-0.5 if scale is None else scale
    O, bound = case.ref.attend(Q.double().numpy(), case.table, case.lens, case.starts, scale_, causal, window)
    out = views(torch.full(Q.shape, 3.25), layout)
    sg.kv4_attend(views(Q, layout), cache, *args, scale=scale, causal=causal, window=window, out=out, max_new=max_new,
                  workspace=workspace)
    got = out.cpu().double().numpy()
    inside = np.zeros(case.rows, bool)
    inside[case.starts[0]:case.starts[-1]] = True
    assert (got[~inside] == 3.25).all(), (what, "rows outside the sequences")
    close(got[inside], O[inside], bound[inside], what)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("dim,block", [(16, 16), (48, 16), (64, 32), (80, 16), (128, 64), (208, 16), (256, 128)])
@pytest.mark.parametrize("ratio", [1, 4, 7])
def test_next_token(ratio, dim, block, dtype):
    print(f"[kv4] next token ratio={ratio} dim={dim} block={block} {dtype}", flush=True)
    case = Case4(dim + ratio, [1, 15, 16, 17, 0, 33, 127, 129, 300], [1, 1, 1, 1, 0, 1, 1, 1, 1], 2, block, dim, before=1, behind=2)
    for i, layout in enumerate(("packed", "padded", "heads")):
        attends(case, ratio, dtype, layout=layout, max_new=1 if i else None, what=layout)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 1), (True, 40), (True, 1000)])
@pytest.mark.parametrize("heads,ratio,dim,block", [(1, 1, 64, 16), (2, 3, 128, 32), (1, 8, 96, 64), (1, 2, 256, 16), (1, 33, 32, 16)])
def test_several_rows(heads, ratio, dim, block, causal, window, dtype):
    print(f"[kv4] rows heads={heads} ratio={ratio} dim={dim} causal={causal} window={window} {dtype}", flush=True)
    # Prompts whole and behind a cache, rows before token 0, sequences without rows.
    case = Case4(dim + window, [70, 200, 31, 50, 3, 260], [70, 9, 31, 0, 5, 130], heads, block, dim)
    attends(case, ratio, dtype, causal, window, what="all rows at once")
    attends(case, ratio, dtype, causal, window, max_new=3, layout="heads", what="a hint that is too small")


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("seqs,length,new,ratio,dim", [(1, 5000, 1, 8, 128), (2, 3000, 4, 4, 128), (1, 9000, 1, 1, 64), (1, 2500, 40, 2, 256), (1, 700, 500, 1, 128)])
def test_long_sequences(seqs, length, new, ratio, dim, dtype):
    print(f"[kv4] long {seqs}x{length} new={new} ratio={ratio} dim={dim} {dtype}", flush=True)
    case = Case4(length, [length - 37 * b for b in range(seqs)], [new] * seqs, 1, 32, dim)
    attends(case, ratio, dtype, max_new=new, what="split")
    attends(case, ratio, dtype, max_new=new, workspace=torch.empty(0, device="cuda"), what="not split")
    attends(case, ratio, dtype, max_new=new, window=length // 2, what="split window")
    # A table laid out for far longer sequences.
    case.table = np.concatenate([case.table, np.full((seqs, 2000), -1, np.int32)], axis=1)
    attends(case, ratio, dtype, max_new=new, what="wide table")


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_large_scores(dtype):
    # Softmax of scores up to thousands: one token takes all, or none moves far from the maximum.
    case = Case4(11, [300, 64], [5, 64], 2, 16, 64)
    attends(case, 2, dtype, scale=30.0, what="large")
    attends(case, 2, dtype, scale=-2.0, what="negative")
    attends(case, 2, dtype, scale=0.0, what="mean")


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("scales", ["small", "large", "wide", "rising", "zero", "negative"])
def test_scales_of_every_size(scales, dtype):
    # Values' scales far from 1, far from one another, growing along the tokens, zero, and of either sign.
    case = Case4(19, [700, 90, 33], [3, 40, 1], 2, 16, 64)
    s = case.ref.scales[1]
    if scales == "small":
        s *= 2.0**-80
    elif scales == "large":
        s *= 2.0**80
    elif scales == "wide":
        s[:] = ref.bf16(s * np.exp2(case.rng.integers(-30, 30, s.shape)))
    elif scales == "rising":
        for b in range(3):
            for t in range(int(case.lens[b])):
                s[case.table[b, t // 16], :, t % 16] = 2.0**(-40 + 80 * t / case.lens[b])
        s[:] = ref.bf16(s)
    elif scales == "zero":
        s[case.rng.random(s.shape) < 0.7] = 0
        case.ref.scales[0][case.rng.random(s.shape) < 0.5] = 0
    else:
        s[case.rng.random(s.shape) < 0.5] *= -1
        case.ref.scales[0][case.rng.random(s.shape) < 0.5] *= -1
    attends(case, 3, dtype, what=scales)
    attends(case, 3, dtype, max_new=40, window=70, what=scales + " window")


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 20), (False, 0)])
def test_scales_that_are_not_finite_reach_only_rows_that_see_them(causal, window, dtype):
    case = Case4(13, [90, 64, 200], [40, 64, 3], 2, 16, 96)
    for b, t, bad in ((0, 60, np.nan), (1, 33, np.inf), (2, 100, -np.inf), (0, 88, np.nan)):
        case.ref.scales[1][case.table[b, t // 16], 1, t % 16] = bad
    case.ref.scales[0][case.table[1, 2], 0, 7] = np.inf  # keys
    case.ref.scales[0][case.table[2, 11], 0, 3] = np.nan
    # Behind the last token of a sequence: seen by nobody.
    page = case.table[0, 5]
    case.ref.scales[0][page, :, 10:] = np.nan
    case.ref.scales[1][page, :, 10:] = np.inf
    with np.errstate(invalid="ignore"):
        attends(case, 2, dtype, causal, window, what="not finite")


# One work-group a row tile; tokens split and joined; row tiles a wave (prompts).
LAYOUTS = {"tokens": ([1, 40, 130], [1, 9, 130], 1), "split": ([3000, 700], [3, 2], 1), "rows": ([150] + [20] * 31, [130] + [2] * 31, 8)}


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 7)])
@pytest.mark.parametrize("layout", LAYOUTS)
def test_infinite_queries(layout, causal, window, dtype):
    lens, new, heads = LAYOUTS[layout]
    print(f"[kv4 inf] {layout} causal={causal} window={window} {dtype}", flush=True)
    case = Case4(31, lens, new, heads, 16, 64)
    # Component 0 of every key is positive, component 1 of either sign.
    case.ref.codes[0][..., 0] = (case.ref.codes[0][..., 0] & 0xF7) | 1
    Q = case.normal(heads, dtype)
    last = case.rows - 1
    Q[0, :, 0], Q[last, :, 0] = -float("inf"), float("inf")   # every score -inf; every score +inf
    Q[case.rows // 2, 0, 1] = -float("inf")                   # scores of both signs, or one
    cache, args = case.device(), case.args()
    with np.errstate(invalid="ignore"):
        O, bound = case.ref.attend(Q.double().numpy(), case.table, case.lens, case.starts, 0.2, causal, window)
    assert np.isnan(O[0]).all() and np.isnan(O[last]).all() and np.isfinite(O[1]).all()
    got = sg.kv4_attend(Q.to(TYPES[dtype]).cuda(), cache, *args, scale=0.2, causal=causal, window=window, max_new=max(new))
    close(got.cpu().double().numpy(), O, bound, f"{layout} {dtype}")


def test_queries_of_every_size():
    # Rows of float32 queries far from 1 and far from one another, some components tiny beside others.
    case = Case4(23, [200, 90], [30, 20], 2, 16, 80)
    case.ref.scales[0] *= 2.0**-3
    Q = case.normal(4, "f32")
    Q = Q * torch.exp2(torch.from_numpy(case.rng.integers(-12, 6, (case.rows, 4, 1)))).float()
    Q = Q * torch.exp2(torch.from_numpy(case.rng.integers(-20, 1, (1, 1, 80)))).float()
    attends(case, 2, "f32", Q=Q, scale=0.3, what="spread")
    attends(case, 2, "f32", Q=Q * 2.0**60, scale=0.3 * 2.0**-60, what="large")
    attends(case, 2, "f32", Q=Q * 2.0**-60, scale=0.3 * 2.0**60, what="small")
    Q[:, 1] = 0
    attends(case, 2, "f32", Q=Q, what="zero heads")


def test_two_runs_are_the_same():
    case = Case4(17, [3000, 500], [2, 2], 2, 32, 128)
    Q = case.normal(8, "bf16").cuda()
    cache, args = case.device(), case.args()
    first = sg.kv4_attend(Q, cache, *args, max_new=2)
    for _ in range(3):
        assert torch.equal(sg.kv4_attend(Q, cache, *args, max_new=2), first)


@pytest.mark.parametrize("ratio,columns", [(1, 1), (1, 2), (2, 3), (70, 3), (70, 4), (3, 7)])
@pytest.mark.parametrize("window", [0, 5, 40])
def test_rows_past_a_short_table(window, ratio, columns):
    # Lengths behind the table's last column: rows that see only its tokens are
    # as ever, the others NaN, rows before token 0 zero; nothing behind is read.
    block, dim = 16, 64
    case = Case4(12, [16 * columns] * 4, [9, 3, 8, 2], 1, block, dim)
    case.lens = np.array([16 * columns + 3, 16 * columns + 200, 6, 2**31 - 1], np.int32)
    cache, args = case.device(), case.args()
    Q = case.normal(ratio, "bf16")
    for max_new in (1, 9):
        O, bound = case.ref.attend(Q.double().numpy(), case.table, case.lens, case.starts, 0.2, True, window)
        assert np.isfinite(O[:6]).all() and np.isnan(O[6:12]).all() and (O[12:14] == 0).all() and np.isnan(O[20:]).all()
        got = sg.kv4_attend(Q.cuda(), cache, *args, scale=0.2, window=window, max_new=max_new).cpu().double().numpy()
        close(got, O, bound, f"columns {columns} window {window} max_new {max_new}")


def test_positions_up_to_31_bits():
    # The last tokens of a sequence of 2^31 - 1, whose table repeats a few pages, through a window.
    block, dim, n, window = 1024, 16, 20, 50
    case = Case4(14, [2 * block - 1], [n], 1, block, dim, spare=0)
    cache = case.device()
    K, V, Q = (case.normal(1, "f32") for _ in range(3))
    case.ref.write([K.double().numpy(), V.double().numpy()], case.table, case.lens, case.starts)
    O, bound = case.ref.attend(Q.double().numpy(), case.table, case.lens, case.starts, 0.3, True, window)
    table = torch.full((1, 2**21), -1, dtype=torch.int32)
    table[0, -2:] = torch.from_numpy(case.table[0])
    args = [table.cuda(), torch.tensor([2**31 - 1], dtype=torch.int32).cuda(), torch.from_numpy(case.starts).cuda()]
    sg.kv4_write(cache, K.cuda(), V.cuda(), *args)
    same_cache(cache, case.ref, "last tokens")
    for max_new in (1, n):
        got = sg.kv4_attend(Q.cuda(), cache, *args, scale=0.3, window=window, max_new=max_new).cpu().double().numpy()
        close(got, O, bound, f"last tokens, max_new {max_new}")
    outs = sg.kv4_read(cache, *args, rows=n)
    for i in range(2):
        assert np.array_equal(outs[i].cpu().double().numpy(), case.ref.tokens(case.table, 0, 2 * block - 1, i)[-n:])


# 32 sequences of 8 heads are one work-group's heads for each of 256 compute
# units; two sequences have many rows, the others few or none.
def prompts(seed, block, dim, **kw):
    lens = [300, 150] + [(37 * b) % 90 for b in range(2, 32)]
    new = [300, 130] + [min(l, b % 5) for b, l in enumerate(lens[2:])]
    lens[5], new[5] = 3, 9  # rows before token 0
    return Case4(seed, lens, new, 8, block, dim, before=1, behind=2, **kw)


def queries(case, ratio):
    """Doubles that every type holds exactly: multiples of 1/32 below 4."""
    x = case.rng.standard_normal((case.rows, case.heads * ratio, case.dim))
    return np.clip(np.rint(x * 32), -127, 127) / 32


def prompt_runs(case, Q, ratio, dtype, causal, window, want, what, hints=(130, 300, None)):
    O, bound = want
    cache, args = case.device(), case.args()
    q = torch.from_numpy(Q).to(TYPES[dtype])
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    inside = np.zeros(case.rows, bool)
    inside[case.starts[0]:case.starts[-1]] = True
    for i, max_new in enumerate(hints):  # the first: fewer than the first sequence has
        if cus == 256:
            batch = sg.lowbit._batch(cache, *args, case.rows, max_new)
            shape = sg.sgemm_kv4_attend_shape(cache._struct, batch, 8 * ratio, window, cus)
            assert shape[1] == 4 and shape[3] == 0
        layout = ("packed", "padded", "heads")[i]
        out = views(torch.full(Q.shape, 3.25), layout)
        sg.kv4_attend(views(q, layout), cache, *args, scale=0.11, causal=causal, window=window, out=out, max_new=max_new)
        got = out.cpu().double().numpy()
        assert (got[~inside] == 3.25).all(), (what, "rows outside the sequences")
        close(got[inside], O[inside], bound[inside], f"{what} {dtype} max_new={max_new}")


@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 1), (True, 40)])
@pytest.mark.parametrize("dim,block,ratio", [(64, 16, 1), (128, 32, 1), (80, 64, 2), (16, 16, 1), (208, 16, 1), (256, 32, 1)])
def test_prompts(dim, block, ratio, causal, window):
    print(f"[kv4 prompts] dim={dim} block={block} ratio={ratio} causal={causal} window={window}", flush=True)
    case = prompts(dim + window, block, dim)
    Q = queries(case, ratio)
    want = case.ref.attend(Q, case.table, case.lens, case.starts, 0.11, causal, window)
    for dtype in ("f32", "bf16", "f16"):
        prompt_runs(case, Q, ratio, dtype, causal, window, want, "prompts")


@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 20)])
@pytest.mark.parametrize("dim", [64, 96, 144])
def test_prompts_with_bad_pages_and_short_tables(dim, causal, window):
    print(f"[kv4 prompts] bad pages dim={dim} causal={causal} window={window}", flush=True)
    case = prompts(7 + dim, 16, dim, columns=18)  # the first sequence has 300 tokens, the table names 288
    for b, t, bad in ((0, 100, np.nan), (0, 250, np.inf), (1, 0, np.nan), (1, 149, -np.inf)):
        case.ref.scales[1][case.table[b, t // 16], 1, t % 16] = bad
    case.ref.scales[0][case.table[1, 5], 2, 7] = np.nan
    last = int(case.lens[1]) % 16
    case.ref.scales[0][case.table[1, 9], :, last:] = np.nan
    case.ref.scales[1][case.table[1, 9], :, last:] = np.nan
    case.table[0, 9], case.table[3, 0], case.table[8, 1] = 10**6, -7, case.ref.pages
    Q = queries(case, 1)
    with np.errstate(invalid="ignore"):
        want = case.ref.attend(Q, case.table, case.lens, case.starts, 0.11, causal, window)
    for dtype in ("f32", "bf16", "f16"):
        prompt_runs(case, Q, 1, dtype, causal, window, want, "bad pages")


def test_prompts_with_rising_scales():
    case = prompts(5, 16, 128)
    s = case.ref.scales[1]
    for t in range(300):
        s[case.table[0, t // 16], :, t % 16] = 2.0**(-30 + 60 * t / 300)
    s[:] = ref.bf16(s)
    Q = queries(case, 1)
    want = case.ref.attend(Q, case.table, case.lens, case.starts, 0.11, True, 0)
    for dtype in ("f32", "bf16", "f16"):
        prompt_runs(case, Q, 1, dtype, True, 0, want, "rising")


def test_prompts_whose_tiles_go_both_ways():
    # Tiles of sequences and heads that begin in one round of work-groups and end in the next.
    lens = [500, 420, 390, 17, 333, 470, 128, 256, 64]
    case = Case4(51, lens, lens, 7, 16, 64)
    Q = queries(case, 3)
    q = torch.from_numpy(Q).to(torch.bfloat16)
    cache, args = case.device(), case.args()
    got = sg.kv4_attend(q.cuda(), cache, *args, max_new=500).cpu().double().numpy()
    first = 0
    for b, l in enumerate(lens):  # the last rows of each sequence, and its first: every tile has one of them or lies between
        for part in (slice(0, min(l, 40)), slice(max(0, l - 90), l)):
            rows = np.arange(l)[part]
            one = np.array([0, len(rows)])
            O, bound = case.ref.attend(Q[first + rows], case.table[b:b + 1], [int(rows[-1]) + 1], one, 64**-0.5, True, 0)
            close(got[first + rows], O, bound, f"sequence {b}")
        first += l
    # And all rows against the same by tiles of one work-group each.
    again = torch.zeros(q.shape, device="cuda")
    for b in range(len(lens)):
        a, e = int(case.starts[b]), int(case.starts[b + 1])
        again[a:e] = sg.kv4_attend(q[a:e].cuda(), cache, args[0][b:b + 1], args[1][b:b + 1], torch.tensor([0, e - a], dtype=torch.int32).cuda(), max_new=1)
    assert np.allclose(got, again.cpu().double().numpy(), rtol=1e-4, atol=1e-5)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("layout", LAYOUTS)
def test_equal_scores_of_every_size(layout, dtype):
    # Every token has the same score, however large: the mean of the values seen. The
    # weights are then equal to the bit, so that what is left are the roundings of a
    # weight's parts (2^-22), of its product with a scale and of float32 sums over the
    # tokens (2^-24 each a term). Where one token's key is twice the others', it takes
    # all the weight of positive scores.
    lens, new, heads = LAYOUTS[layout]
    print(f"[kv4 equal] {layout} {dtype}", flush=True)
    case = Case4(61, lens, new, heads, 16, 64)
    case.ref.codes[0][:] = 0x22
    case.ref.scales[0][:] = 0.75
    Q = torch.ones((case.rows, heads, 64)).to(TYPES[dtype]).cuda()
    V = [case.ref.tokens(case.table, b, lens[b], 1) for b in range(len(lens))]
    args = case.args()
    for twice in (None, 11):
        if twice is not None:
            for b in range(len(lens)):
                if lens[b] > twice:
                    case.ref.scales[0][case.table[b, twice // 16], :, twice % 16] = 1.5
        cache = case.device()
        for size in (0, 7, 13, 14, 15, 20, 22, 23, 24, 26, 30, 40, 100):
            for sign in (1, -1) if twice is None else (1,):
                got = sg.kv4_attend(Q, cache, *args, scale=sign * 2.0**size, max_new=max(new)).cpu().double().numpy()
                for b in range(len(lens)):
                    for i in range(new[b]):
                        seen = V[b][:lens[b] - new[b] + i + 1]
                        if twice is not None and len(seen) > twice:
                            seen = seen[twice:twice + 1]
                        close(got[case.starts[b] + i], seen.mean(axis=0), (len(seen) + 16) * 2.0**-22 * np.abs(seen).mean(axis=0) + 2.0**-37 * np.abs(seen).max(),
                              f"{layout} {dtype} 2^{size} sign {sign} sequence {b} row {i}")


@pytest.mark.parametrize("heads,ratio,dim", [(1, 2, 64), (2, 5, 80)])
def test_many_sequences_share_their_tokens(heads, ratio, dim):
    # More sequences than lanes of a wave, from empty to long, whose tokens are shared
    # out together; parts that end within a sequence, and work-groups without one.
    rng = np.random.default_rng(dim)
    lens = [int(x) for x in rng.integers(0, 60, 150)]
    for b in (0, 63, 64, 70, 149):
        lens[b] = int(rng.integers(1500, 3000))
    new = [min(l, int(n)) for l, n in zip(lens, rng.integers(0, 4, 150))]
    new[64], new[149] = 9, 9
    case = Case4(71, lens, new, heads, 16, dim)
    shape = sg.sgemm_kv4_attend_shape(case.device()._struct, sg.KV8Batch(None, None, None, 150, case.table.shape[1], case.rows, 3), heads * ratio, 0)
    assert shape[3] > 64
    for max_new in (9, 3, 1):
        attends(case, ratio, "bf16", max_new=max_new, what=f"max_new {max_new}")
        attends(case, ratio, "f32", max_new=max_new, window=900, what=f"window, max_new {max_new}")
    attends(case, ratio, "f16", causal=False, max_new=9, what="not causal")


@pytest.mark.parametrize("dtype", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("dim,layout", [(128, "packed"), (48, "padded"), (80, "heads")])
def test_reading_back_more_than_the_caches_hold(dim, layout, dtype):
    print(f"[kv4] large read dim={dim} {layout} {dtype}", flush=True)
    lens = [5000, 3001, 17, 2500]
    case = Case4(81, lens, [4990, 3001, 0, 2499], 6, 16, dim, before=2, behind=3)
    assert case.rows * 6 * dim * 2 >= 4 << 20 or dim == 48
    cache, args = case.device(), case.args()
    outs = [views(torch.full((case.rows, 6, dim), 3.25).to(TYPES[dtype]), layout) for _ in range(2)]
    if layout != "packed":  # rows that begin at an odd element
        outs = [torch.full((case.rows, 7, dim + 1), 3.25, device="cuda").to(TYPES[dtype])[:, :6, 1:] for _ in range(2)]
    sg.kv4_read(cache, *args, K=outs[0], V=outs[1])
    for j in range(2):
        got = outs[j].cpu().double().numpy()
        for b in range(4):
            n = int(case.new[b])
            want = torch.from_numpy(case.ref.tokens(case.table, b, lens[b], j)[lens[b] - n:]).to(torch.float32).to(TYPES[dtype]).double().numpy()
            assert np.array_equal(got[case.starts[b]:case.starts[b] + n], want), (b, j)
        assert (got[:2] == 3.25).all() and (got[-3:] == 3.25).all()

"""How exact attention over the 4-bit cache is: weights at values' scales of
every size, and a bound for each row from what that row sees (GPU tests)."""

import numpy as np
import pytest
import torch

import dense_fp32_matrix_sgemm_amd as sg
from tests import lowbit_ref, step_ref as ref
from tests.test_parity_kv4 import LAYOUTS, Case4, prompts
from tests.test_parity_kv8 import TYPES, close

pytestmark = pytest.mark.gpu

U = 2.0**-24


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sg.load_library()


def page_of(case, b, t):
    return case.table[b, t // case.block], t % case.block


# Two tokens of a sequence share its weight, all others have a score 384 below
# and weigh nothing. Query components 0 to 7 are one-hot and meet codes of 1, so
# that a score is K's scale itself, 1/8 to 1. In powers of two it is at most 1.45 and,
# with log2(e) and its product with the scale rounded, off by 2 * 1.45 u; what the
# exponential takes lies within 6 of 0 and is rounded by 4 u: 14 u for both tokens,
# ln 2 of it in their weights, and the exponential's own 2 u each: 14 u of their
# ratio, 10 u of the smaller share (0.3 at least). The product with V's scale (a
# power of two) is exact, its two parts hold it to 2 u, the two sums of them take 2 u,
# those of the normaliser and of waves and parts and their factors 7 u, the quotient
# and what follows it 2 u: 23 u of the outcome, 24 are allowed.
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("e", [0, -7, -40, -80, 13, 60, 100])
def test_weights_at_scales_of_every_size(e, layout, dtype):
    lens, new, heads = LAYOUTS[layout]
    print(f"[kv4 weights] 2^{e} {layout} {dtype}", flush=True)
    case = Case4(100 + e, lens, new, heads, 16, 64)
    rng = case.rng
    codes = ref.e2m1(np.full(case.ref.codes[0].shape[:-1] + (64,), -6.0))
    case.ref.codes[0][:] = ref.pack(codes)
    case.ref.scales[0][:] = 64.0
    case.ref.codes[1][:] = 0x22          # 1
    case.ref.scales[1][:] = 2.0**e
    share = {}                           # of the token whose value counts in odd components
    for b, l in enumerate(lens):
        seen = l - new[b] + 1            # what the first new row sees
        if seen < 2:
            continue
        ts = rng.choice(seen, 2, replace=False)
        for h in range(heads):
            s = ref.bf16(np.array([rng.uniform(1 / 8, 1 / 4), rng.uniform(3 / 4, 1)]))
            for k, t in enumerate(ts):
                page, place = page_of(case, b, t)
                case.ref.codes[0][page, h, place] = 0x22
                case.ref.scales[0][page, h, place] = s[k]
            page, place = page_of(case, b, ts[1])
            case.ref.codes[1][page, h, place] = 0x02     # 1 in even components, 0 in odd ones
            share[b, h] = 1 / (1 + np.exp(s[1] - s[0]))
    Q = torch.zeros(case.rows, heads, 64)
    for r in range(case.rows):
        Q[r, :, r % 8] = 1
    got = sg.kv4_attend(Q.to(TYPES[dtype]).cuda(), case.device(), *case.args(), scale=1.0, max_new=max(new)).cpu().double().numpy()
    worst = 0.0
    for (b, h), p in share.items():
        o = got[case.starts[b]:case.starts[b + 1], h] * 2.0**-e
        worst = max(worst, np.abs(o[:, 0::2] - 1).max(), np.abs(o[:, 1::2] / p - 1).max())
    print(f"[kv4 weights] off by {worst / U:.1f} units", flush=True)
    assert worst <= 24 * U


def row_bound(case, Q, scale, causal, window):
    """(O, bound): each row's from the tokens that it sees, head by head.

    As lowbit_ref.Cache.attend has it, and what the two parts of a weight and of a
    query may hold less than float32: 2^-38 of the row's largest product of a weight
    and a scale for each token seen, with codes of up to 6."""
    O, bound = lowbit_ref.Cache.attend(case.ref, Q, case.table, case.lens, case.starts, scale, causal, window)
    ratio = Q.shape[1] // case.heads
    for b in range(len(case.lens)):
        n, length = int(case.starts[b + 1] - case.starts[b]), int(case.lens[b])
        K = case.ref.tokens(case.table, b, length, 0)
        s = np.array([case.ref.scales[1][page_of(case, b, t)[0], :, t % case.block] for t in range(length)])
        for i in range(n):
            p = length - n + i
            hi, lo = (p + 1 if causal else length), max(0, p + 1 - window) if window else 0
            if hi <= lo:
                continue
            for h in range(Q.shape[1]):
                z = K[lo:hi, h // ratio] @ Q[case.starts[b] + i, h] * scale
                w = np.exp(z - z.max())
                bound[case.starts[b] + i, h] += (hi - lo) * 2.0**-38 * 6 * (w / w.sum() * np.abs(s[lo:hi, h // ratio])).max()
    return O, bound


def held(case, Q, dtype, causal, window, max_new, what):
    scale = case.dim**-0.5
    O, bound = row_bound(case, Q, scale, causal, window)
    inside = np.zeros(case.rows, bool)
    inside[case.starts[0]:case.starts[-1]] = True
    for b in range(len(case.lens)):  # rows before token 0
        inside[case.starts[b]:case.starts[b] + max(0, int(case.starts[b + 1] - case.starts[b]) - int(case.lens[b]))] = False
    # The bound says something of every row: it is far below the row's largest component.
    assert (bound[inside].max(axis=2) <= 2.0**-8 * np.abs(O[inside]).max(axis=2)).all(), what
    got = sg.kv4_attend(torch.from_numpy(Q).to(TYPES[dtype]).cuda(), case.device(), *case.args(), scale=scale, causal=causal, window=window, max_new=max_new)
    close(got.cpu().double().numpy()[inside], O[inside], bound[inside], what)


def coarse(case, heads):
    """Queries that every type holds exactly."""
    return np.clip(np.rint(case.rng.standard_normal((case.rows, heads, case.dim)) * 32), -127, 127) / 32


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("kind", ["rising", "falling", "wide", "unseen"])
def test_rows_by_what_they_see(kind, dtype):
    # Scales that differ by 2^80 along the tokens, or from token to token; large ones that no row sees.
    case = Case4(19, [700, 90, 33], [3, 40, 1], 2, 16, 64)
    s = case.ref.scales[1]
    if kind == "wide":
        s[:] = ref.bf16(s * np.exp2(case.rng.integers(-30, 30, s.shape)))
    elif kind == "unseen":
        s[:] = 2.0**100
    for b in range(3):
        for t in range(int(case.lens[b])):
            page, place = page_of(case, b, t)
            if kind in ("rising", "falling"):
                s[page, :, place] = ref.bf16(2.0**((-40 + 80 * t / case.lens[b]) * (1 if kind == "rising" else -1)))
            elif kind == "unseen":
                s[page, :, place] = 2.0**-60 if t > case.lens[b] - 70 else 2.0**90
    Q = coarse(case, 6)
    for causal, window, max_new in ((True, 0, 3), (True, 30, 40), (False, 0, 40)):
        if kind == "unseen" and not window:
            continue
        held(case, Q, dtype, causal, window, max_new, f"{kind} {causal} {window} {dtype}")


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 40), (False, 0)])
@pytest.mark.parametrize("kind", ["rising", "falling", "wide"])
def test_prompt_rows_by_what_they_see(kind, causal, window, dtype):
    case = prompts(5, 16, 64)
    s = case.ref.scales[1]
    if kind == "wide":
        s[:] = ref.bf16(s * np.exp2(case.rng.integers(-30, 30, s.shape)))
    else:
        for b in range(len(case.lens)):
            for t in range(int(case.lens[b])):
                page, place = page_of(case, b, t)
                s[page, :, place] = ref.bf16(2.0**((-30 + 60 * t / 300) * (1 if kind == "rising" else -1)))
    held(case, coarse(case, 8), dtype, causal, window, 130, f"prompts {kind} {causal} {window} {dtype}")


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("layout", LAYOUTS)
def test_the_largest_product_changes_with_the_largest_score(layout, dtype):
    # Scores that rise along the tokens while their values' scales fall, and the
    # other way round: each new largest score makes the products before it small.
    lens, new, heads = LAYOUTS[layout]
    for sign in (1, -1):
        case = Case4(37, lens, new, heads, 16, 64)
        case.ref.codes[0][:] = 0x22
        for b, l in enumerate(lens):
            for t in range(l):
                page, place = page_of(case, b, t)
                case.ref.scales[0][page, :, place] = ref.bf16(max(t, 1) / l)
                case.ref.scales[1][page, :, place] = ref.bf16(2.0**(-sign * 60 * t / l))
        Q = np.zeros((case.rows, heads, 64))
        Q[..., 0] = sign * 100.0  # scores up to 12.5 log2(e) = 18 binary digits apart
        Q[:, :, 1] = 4.0
        held(case, Q, dtype, True, 0, max(new), f"{layout} {sign} {dtype}")


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("layout", LAYOUTS)
def test_powers_of_two_pass_through(layout, dtype):
    # Values' scales times 2^k give the same rows times 2^k, to the bit: products are
    # held relative to their row's largest, and weights do not know of the scales.
    lens, new, heads = LAYOUTS[layout]
    case = Case4(41, lens, new, heads, 16, 96)
    Q = case.normal(3 * heads, dtype).cuda()
    s = case.ref.scales[1].copy()
    want = sg.kv4_attend(Q, case.device(), *case.args(), max_new=max(new))
    for k in (-80, -30, 1, 30, 90, 124):
        case.ref.scales[1] = s * 2.0**k
        got = sg.kv4_attend(Q, case.device(), *case.args(), max_new=max(new))
        assert torch.equal(got.double() * 2.0**-k, want.double()), (layout, dtype, k)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_one_token_is_read_as_it_is(dtype):
    # A window of one: the weight is its own normaliser, up to a rounding of each of product, parts and quotient.
    for layout in LAYOUTS:
        lens, new, heads = LAYOUTS[layout]
        case = Case4(43, lens, new, heads, 16, 64)
        Q = case.normal(heads, dtype).cuda()
        got = sg.kv4_attend(Q, case.device(), *case.args(), window=1, max_new=max(new)).cpu().double().numpy()
        for b, l in enumerate(lens):
            v = case.ref.tokens(case.table, b, l, 1)[l - new[b]:]
            o = got[case.starts[b]:case.starts[b + 1]]
            assert (np.abs(o - v) <= 6 * U * np.abs(v)).all(), (layout, b)

"""Attention over the 8-bit cache where the waves of a work-group take row
tiles of their own (prompts), against its definition in 64 bits (GPU tests)."""

import numpy as np
import pytest
import torch

import dense_fp32_matrix_sgemm_amd as sg
from tests.test_parity_kv8 import TYPES, Case, close, views

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sg.load_library()


def queries(case, ratio):
    """Doubles that every type holds exactly: multiples of 1/32 below 4."""
    x = case.rng.standard_normal((case.rows, case.heads * ratio, case.dim))
    return np.clip(np.rint(x * 32), -127, 127) / 32


# 32 sequences of 8 heads are one work-group's heads for each of 256 compute
# units; two sequences have many rows, the others few or none.
def prompts(seed, block, dim, **kw):
    lens = [300, 150] + [(37 * b) % 90 for b in range(2, 32)]
    new = [300, 130] + [min(l, b % 5) for b, l in enumerate(lens[2:])]
    lens[5], new[5] = 3, 9  # rows before token 0
    return Case(seed, lens, new, 8, block, dim, before=1, behind=2, **kw)


def runs(case, Q, ratio, dtype, causal, window, want, what, hints=(130, 300, None)):
    O, bound = want
    cache, args = case.device(), case.args()
    q = torch.from_numpy(Q).to(TYPES[dtype])
    assert np.array_equal(q.double().numpy(), Q)
    cus = torch.cuda.get_device_properties(0).multi_processor_count
    inside = np.zeros(case.rows, bool)
    inside[case.starts[0]:case.starts[-1]] = True
    for i, max_new in enumerate(hints):  # the first: fewer than the first sequence has
        if cus == 256:
            batch = sg.lowbit._batch(cache, *args, case.rows, max_new)
            shape = sg.sgemm_kv8_attend_shape(cache._struct, batch, 8 * ratio, window, cus)
            assert shape[:2] == (32 if case.dim <= 128 else 16, 4) and shape[3] == 1
        layout = ("packed", "padded", "heads")[i]
        out = views(torch.full(Q.shape, 3.25), layout)
        sg.kv8_attend(views(q, layout), cache, *args, scale=0.11, causal=causal, window=window, out=out, max_new=max_new)
        got = out.cpu().double().numpy()
        assert (got[~inside] == 3.25).all(), (what, "rows outside the sequences")
        close(got[inside], O[inside], bound[inside], f"{what} {dtype} max_new={max_new}")


@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 1), (True, 40)])
@pytest.mark.parametrize("dim,block,ratio", [(64, 16, 1), (128, 32, 1), (80, 64, 2), (16, 16, 1), (208, 16, 1), (256, 32, 1)])
def test_prompts(dim, block, ratio, causal, window):
    print(f"[kv8 prompts] dim={dim} block={block} ratio={ratio} causal={causal} window={window}", flush=True)
    case = prompts(dim + window, block, dim)
    Q = queries(case, ratio)
    want = case.ref.attend(Q, case.table, case.lens, case.starts, 0.11, causal, window)
    for dtype in ("f32", "bf16", "f16"):
        runs(case, Q, ratio, dtype, causal, window, want, "prompts")


@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 20)])
@pytest.mark.parametrize("dim", [64, 96, 144])
def test_nan_bad_pages_and_short_tables(dim, causal, window):
    print(f"[kv8 prompts] nan and bad pages dim={dim} causal={causal} window={window}", flush=True)
    case = prompts(7 + dim, 16, dim, columns=18)  # the first sequence has 300 tokens, the table names 288
    for b, t, comp in ((0, 100, 5), (0, 250, dim - 1), (1, 0, 0), (1, 149, 17)):
        case.ref.codes[1][case.table[b, t // 16], 1, t % 16, comp] = 0xFF
    case.ref.codes[0][case.table[1, 5], 2, 7, 3] = 0x7F  # a key
    # Behind the last token of a sequence: seen by nobody.
    last = int(case.lens[1]) % 16
    case.ref.codes[0][case.table[1, 9], :, last:] = 0x7F
    case.ref.codes[1][case.table[1, 9], :, last:] = 0x7F
    case.ref.scales[0][case.table[4, 2], 3] = np.nan  # scales of a page
    case.ref.scales[1][case.table[6, 1], 4] = np.nan
    case.table[0, 9], case.table[3, 0], case.table[8, 1] = 10**6, -7, case.ref.pages
    Q = queries(case, 1)
    with np.errstate(invalid="ignore"):
        want = case.ref.attend(Q, case.table, case.lens, case.starts, 0.11, causal, window)
    for dtype in ("f32", "bf16", "f16"):
        runs(case, Q, 1, dtype, causal, window, want, "nan and bad pages")


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_two_runs_are_the_same(dtype):
    case = prompts(3, 32, 128)
    cache, args = case.device(), case.args()
    q = case.normal(16, dtype).cuda()
    first = sg.kv8_attend(q, cache, *args, max_new=300, out=torch.zeros(q.shape).cuda())
    for _ in range(3):
        assert torch.equal(sg.kv8_attend(q, cache, *args, max_new=300, out=torch.zeros(q.shape).cuda()), first)

"""Attention over the 8-bit cache with scores that are not finite, against its
definition in 64 bits (GPU tests)."""

import numpy as np
import pytest
import torch

import dense_fp32_matrix_sgemm_amd as sg
from tests.test_parity_kv8 import TYPES, Case, close

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sg.load_library()


# One work-group a row tile; tokens split and joined; row tiles a wave (prompts).
LAYOUTS = {"tokens": ([1, 40, 130], [1, 9, 130], 1), "split": ([3000, 700], [3, 2], 1), "rows": ([150] + [20] * 31, [130] + [2] * 31, 8)}


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 7)])
@pytest.mark.parametrize("layout", LAYOUTS)
def test_infinite_queries(layout, causal, window, dtype):
    lens, new, heads = LAYOUTS[layout]
    print(f"[kv8 inf] {layout} causal={causal} window={window} {dtype}", flush=True)
    case = Case(31, lens, new, heads, 16, 64)
    # Component 0 of every key is positive, component 1 of either sign.
    case.ref.codes[0][..., 0] = np.where((case.ref.codes[0][..., 0] & 0x7F) == 0, 0x38, case.ref.codes[0][..., 0] & 0x7F)
    Q = case.normal(heads, dtype)
    last = case.rows - 1
    Q[0, :, 0], Q[last, :, 0] = -float("inf"), float("inf")   # every score -inf; every score +inf
    Q[case.rows // 2, 0, 1] = -float("inf")                   # scores of both signs, or one
    cache, args = case.device(), case.args()
    if torch.cuda.get_device_properties(0).multi_processor_count == 256:
        batch = sg.lowbit._batch(cache, *args, case.rows, max(new))
        shape = sg.sgemm_kv8_attend_shape(cache._struct, batch, heads, window, 256)
        assert (shape[1] == 4) == (layout == "rows") and (shape[3] > 1) == (layout == "split" and not window)
    with np.errstate(invalid="ignore"):
        O, bound = case.ref.attend(Q.double().numpy(), case.table, case.lens, case.starts, 0.2, causal, window)
    assert np.isnan(O[0]).all() and np.isnan(O[last]).all() and np.isfinite(O[1]).all()
    got = sg.kv8_attend(Q.to(TYPES[dtype]).cuda(), cache, *args, scale=0.2, causal=causal, window=window, max_new=max(new))
    close(got.cpu().double().numpy(), O, bound, f"{layout} {dtype}")


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_one_finite_score_among_minus_infinities(dtype):
    # Token 0 alone has a finite score: it takes all. The window's rows that do not see it have no finite score.
    case = Case(33, [90], [5], 1, 16, 64)
    case.ref.codes[0][..., 0] = 0x38  # 1 in component 0 of every key but token 0's
    case.ref.codes[0][case.table[0, 0], :, 0, 0] = 0
    Q = torch.zeros(5, 1, 64)
    Q[:, :, 0] = -1e4
    cache, args = case.device(), case.args()
    got = sg.kv8_attend(Q.to(TYPES[dtype]).cuda(), cache, *args, scale=1e38).cpu().double().numpy()
    V = case.ref.tokens(case.table, 0, 1, 1)[0]
    assert np.array_equal(got, np.broadcast_to(V, got.shape))
    assert torch.isnan(sg.kv8_attend(Q.to(TYPES[dtype]).cuda(), cache, *args, scale=1e38, window=30)).all()


@pytest.mark.parametrize("heads,new", [(1, 40), (1, 100), (256, 128)])
def test_a_nan_scale_meets_scores_of_minus_infinity(heads, new):
    # Scores of page 0 are 0, all others -inf. A row that sees page 2 gets 0 * NaN from its values' scale, also where
    # another of its row tile does not see all of that page.
    case = Case(35, [130], [new], heads, 16, 64)
    case.ref.codes[0][..., 0] = 0x38
    case.ref.codes[0][case.table[0, 0], :, :, 0] = 0
    case.ref.scales[1][case.table[0, 2]] = np.nan
    Q = torch.zeros(case.rows, heads, 64)
    Q[:, :, 0] = -1e4
    got = sg.kv8_attend(Q.cuda(), case.device(), *case.args(), scale=1e38).cpu().double().numpy()
    V = case.ref.tokens(case.table, 0, 16, 1)
    for i in range(case.rows):
        position = 130 - new + i
        if position >= 32:
            assert np.isnan(got[i]).all(), i
        else:
            seen = V[:min(position + 1, 16)]
            # equal weights of 1: a float32 sum of up to 16 values and a division
            assert (np.abs(got[i] - seen.mean(axis=0)) <= 20 * 2.0**-24 * np.abs(seen).mean(axis=0)).all(), i


@pytest.mark.parametrize("causal,window", [(True, 0), (True, 400), (False, 0)])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_rows_that_see_nothing_beside_split_sequences(dtype, causal, window):
    # Long sequences are split over work-groups; the short ones between them have rows before token 0, or no token at all.
    case = Case(37, [3000, 3, 0, 2500, 1], [4, 9, 5, 1, 2], 1, 32, 128)
    cache, args = case.device(), case.args()
    Q = case.normal(3, dtype)
    if torch.cuda.get_device_properties(0).multi_processor_count == 256:
        batch = sg.lowbit._batch(cache, *args, case.rows, 9)
        assert sg.sgemm_kv8_attend_shape(cache._struct, batch, 3, window, 256)[3] == (1 if window else 11)
    O, bound = case.ref.attend(Q.double().numpy(), case.table, case.lens, case.starts, 0.1, causal, window)
    if causal:
        assert (O[4:10] == 0).all() and (O[13:18] == 0).all() and (O[19] == 0).all()
    for workspace in (None, torch.empty(0, device="cuda")):
        got = sg.kv8_attend(Q.cuda(), cache, *args, scale=0.1, causal=causal, window=window, max_new=9, workspace=workspace)
        close(got.cpu().double().numpy(), O, bound, f"{dtype} workspace={workspace is None}")

"""Writing into pages whose scale the caller set to something that is not a
power of two (GPU tests)."""

import numpy as np
import pytest
import torch

import dense_fp32_matrix_sgemm_amd as sg
from tests import lowbit_ref as ref
from tests.test_parity_kv8 import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sg.load_library()


@pytest.mark.parametrize("scale", [0.3, 0.7, 1.1, 3.0, 1e-3, 7e5, 1.5 * 2.0**-126, 1.9 * 2.0**126])
def test_quotients_next_to_a_tie(scale):
    # New values a few float32 steps around scale * (a tie of e4m3): x / scale in float32, ties to even after that.
    s = np.float32(scale)
    heads, block, dim = 1, 64, 256
    ties = np.array([(8.5 + k) * 2.0**e for k in range(8) for e in range(-5, 5)] + [(k + 0.5) * 2.0**-9 for k in range(8)])
    ties = ties[ties * np.float64(s) < 3.4e38]  # what float32 can hold
    x = (ties * np.float64(s)).astype(np.float32)
    rows = []
    for step in range(-3, 4):
        rows.append((x.view(np.int32) + step).view(np.float32))
    x = np.concatenate(rows + [-r for r in rows])
    x = np.resize(x, (len(x) // dim + 1, 1, dim)).astype(np.float32)
    assert np.abs(x / s).max() < 448 and len(x) < 60
    case = Case(3, [64], [len(x)], heads, block, dim)
    page = case.table[0, 0]
    case.ref.scales[0][page], case.ref.scales[1][page] = s, s
    cache, args = case.device(), case.args()
    sg.kv8_write(cache, torch.from_numpy(x).cuda(), torch.from_numpy(-x).cuda(), *args)
    want = ref.e4m3((x / s).astype(np.float64))
    for got, sign in ((cache.K, 0), (cache.V, 0x80)):
        got = got.view(torch.uint8).cpu().numpy()[page, 0]
        assert np.array_equal(got[-len(x):], want[:, 0] ^ sign)
    for got, codes in ((cache.K, case.ref.codes[0]), (cache.V, case.ref.codes[1])):  # the scale stands, and what was there
        assert np.array_equal(got.view(torch.uint8).cpu().numpy()[page, 0, :-len(x)], codes[page, 0, :-len(x)])
    assert cache.Ks[page, 0].item() == s and cache.Vs[page, 0].item() == s


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_a_scale_below_the_normal_numbers_and_zeros(dtype):
    # 1 / scale is infinite; zeros have the code 0 all the same, and what is not finite is NaN.
    case = Case(4, [17], [1], 1, 32, 64)
    page = case.table[0, 0]
    case.ref.scales[0][page] = case.ref.scales[1][page] = 2.0**-140
    cache = case.device()
    x = torch.zeros(1, 1, 64, dtype=dtype)
    x[..., 1], x[..., 2] = -0.0, float("inf")
    sg.kv8_write(cache, x.cuda(), x.cuda(), *case.args())
    got = cache.K.view(torch.uint8)[page, 0, 16].cpu().numpy()
    assert got[0] == 0 and got[1] == 0x80 and (got[2] & 0x7F) == 0x7F and (got[3:] == 0).all()
    assert cache.Ks[page, 0].item() == 2.0**-140


def test_a_scale_that_rises_from_one_that_is_no_power():
    # Larger values come: the earlier codes go to the new power of two by old / new.
    case = Case(5, [40], [8], 2, 64, 64)
    page = case.table[0, 0]
    case.ref.scales[0][page], case.ref.scales[1][page] = np.float32(0.013), np.float32(0.9)
    x = case.normal(2, "f32") * 900
    cache = case.device()
    before = [c.copy() for c in case.ref.codes]
    sg.kv8_write(cache, x.cuda(), x.cuda(), *case.args())
    for i, (got, scales) in enumerate(((cache.K, cache.Ks), (cache.V, cache.Vs))):
        old = np.float32((0.013, 0.9)[i])
        for h in range(2):
            s = np.float32(ref.scale_for(x[:, h].double().numpy()))
            assert s > old and scales[page, h].item() == s
            codes = got.view(torch.uint8).cpu().numpy()[page, h]
            with np.errstate(invalid="ignore"):
                moved = (ref.E4M3[before[i][page, h, :32]].astype(np.float32) * (old / s)).astype(np.float64)
            assert np.array_equal(codes[:32], ref.e4m3(moved))
            assert np.array_equal(codes[32:40], ref.e4m3(x[:, h].double().numpy() / s))

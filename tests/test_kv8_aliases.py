"""A cache whose arrays overlap: refused where it is written (no GPU needed),
taken where it is read (GPU test)."""

import numpy as np
import pytest
import torch

import dense_fp32_matrix_sgemm_amd as sg
from tests.test_lowbit_host import A, F, K8, KS, LEN, ST, TAB, V8, W, att, batch, cache

ROWS = (F, A, 128, 64, W, 128, 64)
CODES = 10 * 2 * 16 * 64  # bytes of K (and of V) in cache(): pages, heads, tokens, components


@pytest.mark.parametrize("c", [cache(V=K8), cache(V=K8 + CODES - 16), cache(K=V8 + 16), cache(Vs=KS), cache(Vs=KS + 76), cache(Ks=K8),
                               cache(Vs=V8 + CODES - 4), cache(Ks=TAB), cache(Vs=LEN + 8), cache(K=ST)])
def test_write_refuses_a_cache_that_overlaps_itself_or_the_batch(c):
    assert sg.sgemm_kv8_write(c, batch(), *ROWS, None) == sg.SGEMM_ERR_ALIAS
    # Reading and attending write neither; nothing to write is nothing to refuse.
    assert sg.sgemm_kv8_check_args(c, batch(), *ROWS) == sg.SGEMM_OK
    assert sg.sgemm_kv8_attend_check_args(c, batch(), *att()) == sg.SGEMM_OK
    assert sg.sgemm_kv8_write(c, batch(rows=0), *ROWS, None) == sg.SGEMM_OK


@pytest.mark.parametrize("c", [cache(), cache(V=K8 + CODES), cache(Vs=KS + 80), cache(Ks=K8 + CODES)])
def test_arrays_that_only_touch_are_taken(c):
    if torch.cuda.is_available():
        pytest.skip("fake addresses: only where the call ends at the missing device")
    assert sg.sgemm_kv8_write(c, batch(), *ROWS, None) == sg.SGEMM_ERR_DEVICE


@pytest.mark.gpu
def test_keys_that_are_the_values():
    from tests.test_parity_kv8 import Case, close

    case = Case(41, [70, 33], [3, 33], 2, 16, 64)
    case.ref.codes[1], case.ref.scales[1] = case.ref.codes[0], case.ref.scales[0]
    codes = torch.from_numpy(case.ref.codes[0]).cuda().view(torch.float8_e4m3fn)
    scales = torch.from_numpy(case.ref.scales[0].astype(np.float32)).cuda()
    one, args = sg.KV8(codes, codes, scales, scales), case.args()
    q = case.normal(4, "bf16")
    want, bound = case.ref.attend(q.double().numpy(), case.table, case.lens, case.starts, 0.2, True, 0)
    close(sg.kv8_attend(q.cuda(), one, *args, scale=0.2).cpu().double().numpy(), want, bound, "one tensor")
    K, V = sg.kv8_read(one, *args, rows=case.rows)
    assert torch.equal(K, V) and torch.equal(K[:3].cpu().double(), torch.from_numpy(case.ref.tokens(case.table, 0, 70, 0)[-3:]))
    x = case.normal(2, "bf16").cuda()
    before = codes.view(torch.uint8).clone()
    with pytest.raises(sg.SgemmError) as e:
        sg.kv8_write(one, x, x, *args)
    assert e.value.status == sg.SGEMM_ERR_ALIAS and torch.equal(codes.view(torch.uint8), before)

"""The entry points of a serving step on the host: what they refuse, in which
order, before any GPU call (no GPU needed)."""

import ctypes
import os
import shutil

import pytest
import torch

import dense_fp32_matrix_sgemm_amd as sg
from tests.test_lowbit_host import batch
from tests.test_sanitizers import CSRC, HERE, ROOT, SAN, _build_and_run

A, W, Q, O, WS, POS, FR = (0x10000000 * i for i in range(1, 8))  # distinct fake addresses, never touched
K4, V4, KS, VS = (0x10000000 * i for i in range(16, 20))
TAB, LEN, ST = (0x10000000 * i for i in range(10, 13))  # as in batch()
F, BF, H = sg.SGEMM_F32, sg.SGEMM_LP_BF16, sg.SGEMM_LP_F16


def cache(K=K4, V=V4, Ks=KS, Vs=VS, pages=10, heads=2, block=16, dim=64):
    return sg.KV4Cache(K, V, Ks, Vs, pages, heads, block, dim)


CACHE_CASES = [
    (cache(), batch(), sg.SGEMM_OK),
    (cache(pages=0), batch(), sg.SGEMM_ERR_DIM), (cache(heads=0), batch(), sg.SGEMM_ERR_DIM),
    (cache(heads=65537), batch(), sg.SGEMM_ERR_DIM), (cache(), batch(seqs=-1), sg.SGEMM_ERR_DIM), (cache(), batch(table_ld=-1), sg.SGEMM_ERR_DIM),
    (cache(), batch(rows=-1), sg.SGEMM_ERR_DIM), (cache(), batch(max_new=-1), sg.SGEMM_ERR_DIM),
    (cache(block=8), batch(), sg.SGEMM_ERR_CACHE), (cache(block=48), batch(), sg.SGEMM_ERR_CACHE), (cache(block=2048), batch(), sg.SGEMM_ERR_CACHE),
    (cache(dim=0), batch(), sg.SGEMM_ERR_CACHE), (cache(dim=72), batch(), sg.SGEMM_ERR_CACHE), (cache(dim=272), batch(), sg.SGEMM_ERR_CACHE),
    (cache(K=K4 + 8), batch(), sg.SGEMM_ERR_CACHE), (cache(V=V4 + 1), batch(), sg.SGEMM_ERR_CACHE),
    (cache(Ks=KS + 8), batch(), sg.SGEMM_ERR_CACHE), (cache(Vs=VS + 2), batch(), sg.SGEMM_ERR_CACHE),
    (cache(K=None), batch(), sg.SGEMM_ERR_NULL), (cache(Vs=None), batch(), sg.SGEMM_ERR_NULL),
    (cache(), batch(table=None), sg.SGEMM_ERR_NULL), (cache(), batch(lens=None), sg.SGEMM_ERR_NULL), (cache(), batch(starts=None), sg.SGEMM_ERR_NULL),
    (cache(), batch(table=None, table_ld=0), sg.SGEMM_OK),
    (cache(K=None), batch(seqs=0), sg.SGEMM_OK), (cache(K=None), batch(rows=0), sg.SGEMM_OK),
]


@pytest.mark.parametrize("c,b,want", CACHE_CASES)
def test_kv4_cache_and_batch(c, b, want):
    rows = (F, A, 128, 64, W, 128, 64)
    assert sg.sgemm_kv4_check_args(c, b, *rows) == want
    attend = (F, 4, Q, 256, 64, 0.125, 1, 0, O, 256, 64, None, 0)
    assert sg.sgemm_kv4_attend_check_args(c, b, *attend) == want
    if want != sg.SGEMM_OK:
        assert sg.sgemm_kv4_write(c, b, *rows, None) == want
        assert sg.sgemm_kv4_read(c, b, *rows, None) == want
        assert sg.sgemm_kv4_attend(c, b, *attend, None) == want
    if want in (sg.SGEMM_ERR_DIM, sg.SGEMM_ERR_CACHE):
        assert sg.sgemm_kv4_attend_workspace_size(c, b, 4, 0, 256) == 0
        with pytest.raises(sg.SgemmError) as e:
            sg.sgemm_kv4_attend_shape(c, b, 4)
        assert e.value.status == want


def test_kv4_null_structures():
    none = ctypes.POINTER(sg.KV4Cache)()
    assert sg.sgemm_kv4_check_args(none, batch(), F, A, 128, 64, W, 128, 64) == sg.SGEMM_ERR_NULL
    assert sg.sgemm_kv4_check_args(cache(), None, F, A, 128, 64, W, 128, 64) == sg.SGEMM_ERR_NULL
    assert sg.sgemm_kv4_attend_workspace_size(none, batch(), 4, 0, 256) == 0


ROW_CASES = [
    ((3, A, 128, 64, W, 128, 64), sg.SGEMM_ERR_DTYPE),
    ((F, A, 127, 64, W, 128, 64), sg.SGEMM_ERR_LD), ((F, A, 128, 63, W, 128, 64), sg.SGEMM_ERR_LD),
    ((F, A, 128, 64, W, 64, 64), sg.SGEMM_ERR_LD), ((F, A, 64, 320, W, 65, 400), sg.SGEMM_OK),  # heads outermost
    ((F, A, 64, 319, W, 128, 64), sg.SGEMM_ERR_LD), ((F, A, -128, 64, W, 128, 64), sg.SGEMM_ERR_LD),
    ((F, None, 128, 64, W, 128, 64), sg.SGEMM_ERR_NULL), ((F, A, 128, 64, None, 128, 64), sg.SGEMM_ERR_NULL),
    # 10 pages of 2 heads of 16 tokens: 32 bytes of codes and 2 of a scale each.
    ((F, K4 + 20 * 512 - 4, 128, 64, W, 128, 64), sg.SGEMM_ERR_ALIAS), ((F, K4 + 20 * 512, 128, 64, W, 128, 64), sg.SGEMM_OK),
    ((F, A, 128, 64, VS + 638, 128, 64), sg.SGEMM_ERR_ALIAS), ((F, A, 128, 64, VS + 640, 128, 64), sg.SGEMM_OK),
    ((F, A, 128, 64, A, 128, 64), sg.SGEMM_OK),  # the same keys and values may be written
]


@pytest.mark.parametrize("args,want", ROW_CASES)
def test_kv4_rows(args, want):
    assert sg.sgemm_kv4_check_args(cache(), batch(), *args) == want
    if want != sg.SGEMM_OK:
        assert sg.sgemm_kv4_write(cache(), batch(), *args, None) == want


def test_kv4_write_refuses_a_cache_that_overlaps():
    rows = (F, A, 128, 64, W, 128, 64, None)
    for c in (cache(V=K4), cache(V=K4 + 16), cache(Vs=KS), cache(Ks=K4 + 512), cache(Ks=LEN), cache(K=TAB), cache(V=ST)):
        assert sg.sgemm_kv4_check_args(c, batch(), *rows[:-1]) == sg.SGEMM_OK
        assert sg.sgemm_kv4_write(c, batch(), *rows) == sg.SGEMM_ERR_ALIAS


def test_kv4_read_outputs_must_not_meet():
    for other in (A, A + 4, TAB, LEN + 8, ST):
        assert sg.sgemm_kv4_read(cache(), batch(), F, A, 128, 64, other, 128, 64, None) == sg.SGEMM_ERR_ALIAS
    if not torch.cuda.is_available():  # the halves of one buffer's rows do not meet
        assert sg.sgemm_kv4_read(cache(), batch(), F, A, 256, 64, A + 512, 256, 64, None) == sg.SGEMM_ERR_DEVICE
        assert sg.sgemm_kv4_read(cache(), batch(), F, A + 512, 256, 64, A, 256, 64, None) == sg.SGEMM_ERR_DEVICE
    assert sg.sgemm_kv4_read(cache(), batch(), F, A, 256, 64, A + 508, 256, 64, None) == sg.SGEMM_ERR_ALIAS
    assert sg.sgemm_kv4_read(cache(), batch(), F, A, 256, 64, A + 516, 256, 64, None) == sg.SGEMM_ERR_ALIAS
    assert sg.sgemm_kv4_read(cache(), batch(), F, A, 256, 64, A + 512, 257, 64, None) == sg.SGEMM_ERR_ALIAS


def att(dtype=F, heads_q=4, Q=Q, ldq=256, hsq=64, scale=0.125, causal=1, window=0, O=O, ldo=256, hso=64, ws=None, n=0):
    return dtype, heads_q, Q, ldq, hsq, scale, causal, window, O, ldo, hso, ws, n


ATTEND_CASES = [
    (att(), sg.SGEMM_OK), (att(dtype=5), sg.SGEMM_ERR_DTYPE), (att(heads_q=0), sg.SGEMM_ERR_HEADS), (att(heads_q=3), sg.SGEMM_ERR_HEADS),
    (att(heads_q=-2), sg.SGEMM_ERR_HEADS), (att(causal=2), sg.SGEMM_ERR_MASK), (att(window=-1), sg.SGEMM_ERR_MASK),
    (att(causal=0, window=4), sg.SGEMM_ERR_MASK), (att(window=4), sg.SGEMM_OK), (att(ldq=255), sg.SGEMM_ERR_LD), (att(hso=63), sg.SGEMM_ERR_LD),
    (att(Q=None), sg.SGEMM_ERR_NULL), (att(O=None), sg.SGEMM_ERR_NULL), (att(O=Q), sg.SGEMM_ERR_ALIAS), (att(O=K4), sg.SGEMM_ERR_ALIAS),
    (att(O=TAB), sg.SGEMM_ERR_ALIAS), (att(ws=WS, n=64), sg.SGEMM_OK), (att(ws=O + 5 * 1024 - 4, n=64), sg.SGEMM_ERR_ALIAS),
    (att(ws=V4, n=1), sg.SGEMM_ERR_ALIAS), (att(ws=KS, n=1), sg.SGEMM_ERR_ALIAS), (att(ws=Q, n=1), sg.SGEMM_ERR_ALIAS), (att(ws=Q, n=0), sg.SGEMM_OK),
]


@pytest.mark.parametrize("args,want", ATTEND_CASES)
def test_kv4_attend_check_args(args, want):
    assert sg.sgemm_kv4_attend_check_args(cache(), batch(), *args) == want
    if want != sg.SGEMM_OK:
        assert sg.sgemm_kv4_attend(cache(), batch(), *args, None) == want


def test_kv4_attend_shapes():
    def shape(seqs, rows, max_new, columns, heads=8, dim=128, heads_q=32, window=0, cus=256):
        return sg.sgemm_kv4_attend_shape(cache(heads=heads, dim=dim, block=64), batch(seqs=seqs, rows=rows, max_new=max_new, table_ld=columns),
                                         heads_q, window, cus)

    # Few rows: copies in the columns of a tile, and the tokens of all sequences shared out.
    assert shape(32, 32, 1, 128)[:3] == (4, 1, 1) and shape(32, 32, 1, 128, heads_q=64)[:3] == (8, 1, 1)
    assert shape(32, 32, 1, 128, heads_q=72)[:3] == (16, 1, 1) and shape(31, 31, 1, 128, heads_q=160)[:3] == (16, 1, 2)
    assert shape(200, 200, 1, 128, heads_q=160)[:3] == (16, 1, 2) and shape(200, 200, 1, 128, heads_q=160, dim=256)[:3] == (16, 1, 2)
    assert shape(32, 32, 1, 128)[3] == 96 and shape(32, 32, 1, 128, dim=256)[3] == 64
    assert shape(1000, 1000, 1, 128)[3] == 0 and shape(1025, 1025, 1, 128, heads=1, heads_q=4)[3] == 0   # sequences enough
    assert shape(1, 1, 1, 1)[3] == 0 and shape(1, 1, 1, 128, window=64)[3] == 0                         # few tokens to see
    assert shape(1, 1, 1, 2**20, heads=1, heads_q=1)[3] == 64                                           # not all for one sequence
    assert shape(2, 2048, 1024, 80)[:2] == (32, 4) and shape(2, 2048, 1024, 80)[3] == 0                 # prompts: row tiles a wave
    for s in ((32, 32, 1, 128), (2, 2048, 1024, 80), (1, 1, 1, 1)):
        b = batch(seqs=s[0], rows=s[1], max_new=s[2], table_ld=s[3])
        assert (sg.sgemm_kv4_attend_workspace_size(cache(heads=8, dim=128, block=64), b, 32, 0, 256) > 0) == (shape(*s)[3] > 0)


def rows_of(X=Q, Y=O, heads=2, ldx=128, hsx=64, ldy=128, hsy=64):
    return sg.RopeRows(X, Y, heads, ldx, hsx, ldy, hsy)


def turn(dtype=F, otype=F, rows=5, dim=64, rot=64, interleaved=0, inverse=0, amplitude=1.0, positions=POS, freqs=FR, first=None, second=None):
    return dtype, otype, rows, dim, rot, interleaved, inverse, amplitude, positions, freqs, first or rows_of(), second


ROPE_CASES = [
    (turn(), sg.SGEMM_OK), (turn(second=rows_of(A, W)), sg.SGEMM_OK), (turn(dtype=3), sg.SGEMM_ERR_DTYPE), (turn(otype=-1), sg.SGEMM_ERR_DTYPE),
    (turn(rows=-1), sg.SGEMM_ERR_DIM), (turn(dim=0), sg.SGEMM_ERR_DIM), (turn(dim=1025, rot=0), sg.SGEMM_ERR_DIM), (turn(rot=66), sg.SGEMM_ERR_DIM),
    (turn(rot=63), sg.SGEMM_ERR_DIM), (turn(rot=-2), sg.SGEMM_ERR_DIM), (turn(first=rows_of(heads=0)), sg.SGEMM_ERR_DIM),
    (turn(second=rows_of(A, W, heads=65537)), sg.SGEMM_ERR_DIM), (turn(interleaved=2), sg.SGEMM_ERR_MASK), (turn(inverse=-1), sg.SGEMM_ERR_MASK),
    (turn(first=rows_of(ldx=127)), sg.SGEMM_ERR_LD), (turn(first=rows_of(hsy=63)), sg.SGEMM_ERR_LD), (turn(second=rows_of(A, W, ldy=0)), sg.SGEMM_ERR_LD),
    (turn(first=rows_of(ldx=64, hsx=320)), sg.SGEMM_OK), (turn(rows=0, positions=None, freqs=None, first=rows_of(None, None)), sg.SGEMM_OK),
    (turn(positions=None), sg.SGEMM_ERR_NULL), (turn(freqs=None), sg.SGEMM_ERR_NULL), (turn(freqs=None, rot=0), sg.SGEMM_OK),
    (turn(first=rows_of(X=None)), sg.SGEMM_ERR_NULL), (turn(second=rows_of(A, None)), sg.SGEMM_ERR_NULL),
    # In place: the same place, strides and type, and nothing else.
    (turn(first=rows_of(Q, Q)), sg.SGEMM_OK), (turn(first=rows_of(Q, Q), otype=BF), sg.SGEMM_ERR_ALIAS), (turn(first=rows_of(Q, Q + 4)), sg.SGEMM_ERR_ALIAS),
    (turn(first=rows_of(Q, Q, ldy=192)), sg.SGEMM_ERR_ALIAS), (turn(first=rows_of(Q, Q), second=rows_of(A, Q)), sg.SGEMM_ERR_ALIAS),
    (turn(first=rows_of(Q, O), second=rows_of(A, O)), sg.SGEMM_ERR_ALIAS), (turn(first=rows_of(Q, O), second=rows_of(Q, W)), sg.SGEMM_OK),
    (turn(first=rows_of(Q, A), second=rows_of(A, W)), sg.SGEMM_ERR_ALIAS), (turn(first=rows_of(Q, O), second=rows_of(A, Q)), sg.SGEMM_ERR_ALIAS),
    # Parts of one buffer: rows side by side.
    (turn(first=rows_of(Q, Q, ldx=256, ldy=256), second=rows_of(Q + 512, Q + 512, ldx=256, ldy=256)), sg.SGEMM_OK),
    (turn(first=rows_of(Q + 512, Q + 512, ldx=256, ldy=256), second=rows_of(Q, Q, ldx=256, ldy=256)), sg.SGEMM_OK),
    (turn(first=rows_of(Q, Q, ldx=256, ldy=256), second=rows_of(Q + 508, Q + 508, ldx=256, ldy=256)), sg.SGEMM_ERR_ALIAS),
    (turn(first=rows_of(Q, Q, ldx=256, ldy=256), second=rows_of(Q + 516, Q + 516, ldx=256, ldy=256)), sg.SGEMM_ERR_ALIAS),
    (turn(first=rows_of(Q, POS + 16)), sg.SGEMM_ERR_ALIAS), (turn(first=rows_of(Q, FR + 8 * 31)), sg.SGEMM_ERR_ALIAS), (turn(first=rows_of(Q, FR + 8 * 32)), sg.SGEMM_OK),
]


@pytest.mark.parametrize("args,want", ROPE_CASES)
def test_rope_check_args(args, want):
    assert sg.sgemm_rope_check_args(*args) == want
    if want != sg.SGEMM_OK:
        assert sg.sgemm_rope(*args, None) == want


def test_rope_null_structure():
    args = turn()[:10]
    assert sg.sgemm_rope_check_args(*args, None, rows_of()) == sg.SGEMM_ERR_NULL


STEP = dict(lens=A, news=W, pool=Q, taken=O, table=TAB, starts=ST, positions=POS, slots=KS, taken_after=VS, seqs=3, table_ld=4, block=16,
            pool_size=10, rows=5)
STEP_CASES = [
    ({}, sg.SGEMM_OK), ({"taken_after": O}, sg.SGEMM_OK), ({"seqs": -1}, sg.SGEMM_ERR_DIM), ({"table_ld": -1}, sg.SGEMM_ERR_DIM),
    ({"pool_size": -1}, sg.SGEMM_ERR_DIM), ({"rows": -1}, sg.SGEMM_ERR_DIM), ({"block": 8}, sg.SGEMM_ERR_CACHE), ({"block": 24}, sg.SGEMM_ERR_CACHE),
    ({"block": 2048}, sg.SGEMM_ERR_CACHE), ({"block": 8, "rows": -1}, sg.SGEMM_ERR_DIM),
    *[({k: None}, sg.SGEMM_ERR_NULL) for k in ("lens", "news", "pool", "taken", "table", "starts", "positions", "slots", "taken_after")],
    ({"seqs": 0, "lens": None, "news": None, "table": None}, sg.SGEMM_OK), ({"pool": None, "pool_size": 0}, sg.SGEMM_OK),
    ({"table": None, "table_ld": 0}, sg.SGEMM_OK), ({"rows": 0, "positions": None, "slots": None}, sg.SGEMM_OK),
    ({"table": A + 8}, sg.SGEMM_ERR_ALIAS), ({"starts": W - 12}, sg.SGEMM_ERR_ALIAS), ({"starts": W - 16}, sg.SGEMM_OK),
    ({"positions": Q + 36}, sg.SGEMM_ERR_ALIAS), ({"slots": O}, sg.SGEMM_ERR_ALIAS), ({"slots": TAB + 44}, sg.SGEMM_ERR_ALIAS),
    ({"slots": TAB + 48}, sg.SGEMM_OK), ({"taken_after": ST + 12}, sg.SGEMM_ERR_ALIAS), ({"taken_after": A}, sg.SGEMM_ERR_ALIAS),
    ({"taken_after": O + 2}, sg.SGEMM_ERR_ALIAS), ({"positions": KS + 39}, sg.SGEMM_ERR_ALIAS),
]


@pytest.mark.parametrize("change,want", STEP_CASES)
def test_kv_tables_check_args(change, want):
    step = sg.KVStep(**{**STEP, **change})
    assert sg.sgemm_kv_tables_check_args(step) == want
    if want != sg.SGEMM_OK:
        assert sg.sgemm_kv_tables(step, None) == want


def test_no_device_is_reported_not_crashed():
    assert sg.sgemm_kv_tables_check_args(None) == sg.SGEMM_ERR_NULL
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert sg.sgemm_kv4_write(cache(), batch(), F, A, 128, 64, W, 128, 64, None) == sg.SGEMM_ERR_DEVICE
    assert sg.sgemm_kv4_read(cache(), batch(), F, A, 128, 64, W, 128, 64, None) == sg.SGEMM_ERR_DEVICE
    assert sg.sgemm_kv4_attend(cache(), batch(), *att(), None) == sg.SGEMM_ERR_DEVICE
    assert sg.sgemm_rope(*turn(), None) == sg.SGEMM_ERR_DEVICE
    assert sg.sgemm_kv_tables(sg.KVStep(**STEP), None) == sg.SGEMM_ERR_DEVICE


def test_the_binding_refuses():
    cpu, codes, ints = torch.zeros(4, 2, 64), torch.zeros(2, 1, 16, 32, dtype=torch.uint8), torch.zeros(4, dtype=torch.int32)
    scales = torch.zeros(2, 1, 16, dtype=torch.bfloat16)
    for call in (lambda: sg.KV4(codes, codes, scales, scales), lambda: sg.KV4.empty(2, 1, 16, 63, device="cpu"),
                 lambda: sg.rope(cpu, None, ints, torch.zeros(32, dtype=torch.float64)), lambda: sg.rope_frequencies(7, device="cpu"),
                 lambda: sg.rope_frequencies(0, device="cpu"), lambda: sg.rope_frequencies(8, base=0, device="cpu"),
                 lambda: sg.rope_frequencies(8, stretch=4, original=0, device="cpu"),
                 lambda: sg.kv_tables(ints.view(2, 2), ints[:2], ints[:2], ints, ints[:1], 16, 3)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: sg.kv4_write(cpu, cpu, cpu, ints, ints, ints), lambda: sg.kv4_read(cpu, ints, ints, ints),
                 lambda: sg.kv4_attend(cpu, cpu, ints, ints, ints), lambda: sg.KV4(codes.float(), codes, scales, scales),
                 lambda: sg.rope(cpu[0], None, ints, ints), lambda: sg.kv_tables(cpu, ints, ints, ints, ints, 16, 3)):
        with pytest.raises(TypeError):
            call()


def test_frequencies():
    f, amplitude = sg.rope_frequencies(8, device="cpu")
    assert f.dtype == torch.float64 and torch.allclose(f, torch.tensor([1, 0.1, 0.01, 0.001], dtype=torch.float64)) and amplitude == 1
    g, _ = sg.rope_frequencies(8, stretch=4, device="cpu")
    assert torch.equal(g, f / 4)
    h, amplitude = sg.rope_frequencies(8, stretch=4, original=1000, device="cpu")
    assert h[0] == f[0] and h[3] == f[3] / 4 and (h < f)[1:].all() and (h > f / 4)[1:3].all() and amplitude > 1


@pytest.mark.skipif(shutil.which("g++") is None, reason="no g++")
def test_checks_under_sanitizers(tmp_path):
    exe = str(tmp_path / "step_checks")
    cmd = ["g++", "-std=c++17", *SAN, f"-I{os.path.join(ROOT, 'include')}", f"-I{CSRC}", os.path.join(HERE, "step_checks.cpp"),
           os.path.join(CSRC, "args_step.cpp"), os.path.join(CSRC, "args_lowbit.cpp"), "-o", exe]
    assert "step checks ok" in _build_and_run(cmd, exe, tmp_path)

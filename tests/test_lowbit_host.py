"""The entry points of the products held in few bits on the host: what they
refuse, in which order, before any GPU call (no GPU needed)."""

import ctypes
import os
import shutil

import pytest
import torch

import dense_fp32_matrix_sgemm_amd as sg
from tests.test_sanitizers import CSRC, HERE, ROOT, SAN, _build_and_run

A, W, S, Z, C = (0x10000000 * i for i in range(1, 6))  # distinct fake addresses, never touched
F, BF, H = sg.SGEMM_F32, sg.SGEMM_LP_BF16, sg.SGEMM_LP_F16


def w4(dtype=F, stype=F, M=4, N=6, K=100, group=32, alpha=1.0, A=A, lda=100, W=W, ldw=50, S=S, lds=4, Z=Z, ldz=4,
       beta=0.0, C=C, ldc=6):
    return dtype, stype, M, N, K, group, alpha, A, lda, W, ldw, S, lds, Z, ldz, beta, C, ldc


W4_CASES = [
    (w4(), sg.SGEMM_OK),
    (w4(dtype=3), sg.SGEMM_ERR_DTYPE), (w4(stype=-1), sg.SGEMM_ERR_DTYPE), (w4(dtype=BF, stype=H), sg.SGEMM_OK),
    (w4(M=-1), sg.SGEMM_ERR_DIM), (w4(N=-1), sg.SGEMM_ERR_DIM), (w4(K=-1), sg.SGEMM_ERR_DIM),
    (w4(group=0), sg.SGEMM_ERR_GROUP), (w4(group=-32), sg.SGEMM_ERR_GROUP), (w4(group=48), sg.SGEMM_ERR_GROUP),
    (w4(group=2**31 - 32), sg.SGEMM_OK),
    (w4(lda=99), sg.SGEMM_ERR_LD), (w4(ldw=49), sg.SGEMM_ERR_LD), (w4(K=101, lda=101, ldw=50), sg.SGEMM_ERR_LD),
    (w4(lds=3), sg.SGEMM_ERR_LD), (w4(ldz=3), sg.SGEMM_ERR_LD), (w4(Z=None, ldz=0), sg.SGEMM_OK), (w4(ldc=5), sg.SGEMM_ERR_LD),
    (w4(M=-1, dtype=7), sg.SGEMM_ERR_DTYPE), (w4(M=-1, group=1), sg.SGEMM_ERR_DIM), (w4(group=1, lda=1), sg.SGEMM_ERR_GROUP),
    (w4(M=0, A=None, W=None, S=None, C=None), sg.SGEMM_OK), (w4(N=0, C=None), sg.SGEMM_OK),
    (w4(C=None), sg.SGEMM_ERR_NULL), (w4(A=None), sg.SGEMM_ERR_NULL), (w4(W=None), sg.SGEMM_ERR_NULL), (w4(S=None), sg.SGEMM_ERR_NULL),
    (w4(K=0, A=None, W=None, S=None), sg.SGEMM_OK), (w4(alpha=0.0, A=None, W=None, S=None), sg.SGEMM_OK),
    (w4(C=A + 4 * 399), sg.SGEMM_ERR_ALIAS), (w4(C=A + 4 * 400), sg.SGEMM_OK), (w4(C=W + 296), sg.SGEMM_ERR_ALIAS),
    (w4(C=S + 92), sg.SGEMM_ERR_ALIAS), (w4(C=Z + 20), sg.SGEMM_ERR_ALIAS), (w4(C=Z + 24), sg.SGEMM_OK),
    (w4(K=2**30 + 1, lda=2**31 - 1, ldw=2**31 - 1, lds=2**31 - 1, ldz=2**31 - 1), sg.SGEMM_ERR_DIM),
    (w4(M=2**31 - 1, N=2**31 - 1, K=2**30, lda=2**31 - 1, ldw=2**31 - 1, lds=2**31 - 1, ldz=2**31 - 1, ldc=2**31 - 1), sg.SGEMM_ERR_ALIAS),
]


@pytest.mark.parametrize("args,want", W4_CASES)
def test_w4_check_args(args, want):
    assert sg.sgemm_w4_check_args(*args) == want
    if want != sg.SGEMM_OK:
        assert sg.sgemm_w4(*args, None) == want


def pack(dtype=F, stype=F, N=6, K=100, group=32, B=A, ldb=100, W=W, ldw=50, S=S, lds=4, Z=Z, ldz=4):
    return dtype, stype, N, K, group, B, ldb, W, ldw, S, lds, Z, ldz


PACK_CASES = [
    (pack(), sg.SGEMM_OK), (pack(dtype=9), sg.SGEMM_ERR_DTYPE), (pack(N=-1), sg.SGEMM_ERR_DIM), (pack(K=-1), sg.SGEMM_ERR_DIM),
    (pack(K=2**30 + 1, ldb=2**31 - 1, ldw=2**31 - 1, lds=2**31 - 1, ldz=2**31 - 1), sg.SGEMM_ERR_DIM),
    (pack(group=31), sg.SGEMM_ERR_GROUP), (pack(ldb=99), sg.SGEMM_ERR_LD), (pack(ldw=49), sg.SGEMM_ERR_LD),
    (pack(lds=3), sg.SGEMM_ERR_LD), (pack(ldz=3), sg.SGEMM_ERR_LD), (pack(Z=None, ldz=0), sg.SGEMM_OK),
    (pack(N=0, B=None, W=None, S=None), sg.SGEMM_OK), (pack(K=0, B=None, W=None, S=None), sg.SGEMM_OK),
    (pack(B=None), sg.SGEMM_ERR_NULL), (pack(W=None), sg.SGEMM_ERR_NULL), (pack(S=None), sg.SGEMM_ERR_NULL),
    (pack(W=A), sg.SGEMM_ERR_ALIAS), (pack(S=W + 299), sg.SGEMM_ERR_ALIAS), (pack(Z=S), sg.SGEMM_ERR_ALIAS),
]


@pytest.mark.parametrize("args,want", PACK_CASES)
def test_w4_pack_check_args(args, want):
    assert sg.sgemm_w4_pack_check_args(*args) == want
    if want != sg.SGEMM_OK:
        assert sg.sgemm_w4_quantize(*args, None) == want
        d, s, N, K, g, B, ldb, *rest = args
        assert sg.sgemm_w4_dequantize(d, s, N, K, g, *rest, B, ldb, None) == want


K8, V8, KS, VS, TAB, LEN, ST, Q, O, WS = (0x10000000 * i for i in range(6, 16))


def cache(K=K8, V=V8, Ks=KS, Vs=VS, pages=10, heads=2, block=16, dim=64):
    return sg.KV8Cache(K, V, Ks, Vs, pages, heads, block, dim)


def batch(table=TAB, lens=LEN, starts=ST, seqs=3, table_ld=4, rows=5, max_new=2):
    return sg.KV8Batch(table, lens, starts, seqs, table_ld, rows, max_new)


CACHE_CASES = [
    (cache(), batch(), sg.SGEMM_OK),
    (cache(pages=0), batch(), sg.SGEMM_ERR_DIM), (cache(heads=0), batch(), sg.SGEMM_ERR_DIM),
    (cache(heads=65537), batch(), sg.SGEMM_ERR_DIM), (cache(), batch(seqs=-1), sg.SGEMM_ERR_DIM), (cache(), batch(table_ld=-1), sg.SGEMM_ERR_DIM),
    (cache(), batch(rows=-1), sg.SGEMM_ERR_DIM), (cache(), batch(max_new=-1), sg.SGEMM_ERR_DIM),
    (cache(block=8), batch(), sg.SGEMM_ERR_CACHE), (cache(block=48), batch(), sg.SGEMM_ERR_CACHE), (cache(block=2048), batch(), sg.SGEMM_ERR_CACHE),
    (cache(dim=0), batch(), sg.SGEMM_ERR_CACHE), (cache(dim=72), batch(), sg.SGEMM_ERR_CACHE), (cache(dim=272), batch(), sg.SGEMM_ERR_CACHE),
    (cache(K=K8 + 8), batch(), sg.SGEMM_ERR_CACHE), (cache(V=V8 + 1), batch(), sg.SGEMM_ERR_CACHE),
    (cache(K=None), batch(), sg.SGEMM_ERR_NULL), (cache(Vs=None), batch(), sg.SGEMM_ERR_NULL),
    (cache(), batch(table=None), sg.SGEMM_ERR_NULL), (cache(), batch(lens=None), sg.SGEMM_ERR_NULL), (cache(), batch(starts=None), sg.SGEMM_ERR_NULL),
    (cache(), batch(table=None, table_ld=0), sg.SGEMM_OK),
    (cache(K=None), batch(seqs=0), sg.SGEMM_OK), (cache(K=None), batch(rows=0), sg.SGEMM_OK),
]


@pytest.mark.parametrize("c,b,want", CACHE_CASES)
def test_kv8_cache_and_batch(c, b, want):
    rows = (F, A, 128, 64, W, 128, 64)
    assert sg.sgemm_kv8_check_args(c, b, *rows) == want
    attend = (F, 4, Q, 256, 64, 0.125, 1, 0, O, 256, 64, None, 0)
    assert sg.sgemm_kv8_attend_check_args(c, b, *attend) == want
    if want != sg.SGEMM_OK:
        assert sg.sgemm_kv8_write(c, b, *rows, None) == want
        assert sg.sgemm_kv8_read(c, b, *rows, None) == want
        assert sg.sgemm_kv8_attend(c, b, *attend, None) == want
    if want in (sg.SGEMM_ERR_DIM, sg.SGEMM_ERR_CACHE):
        assert sg.sgemm_kv8_attend_workspace_size(c, b, 4, 0, 256) == 0


def test_kv8_null_structures():
    none = ctypes.POINTER(sg.KV8Cache)()
    assert sg.sgemm_kv8_check_args(none, batch(), F, A, 128, 64, W, 128, 64) == sg.SGEMM_ERR_NULL
    assert sg.sgemm_kv8_check_args(cache(), None, F, A, 128, 64, W, 128, 64) == sg.SGEMM_ERR_NULL
    assert sg.sgemm_kv8_attend_workspace_size(none, batch(), 4, 0, 256) == 0


ROW_CASES = [
    ((3, A, 128, 64, W, 128, 64), sg.SGEMM_ERR_DTYPE),
    ((F, A, 127, 64, W, 128, 64), sg.SGEMM_ERR_LD), ((F, A, 128, 63, W, 128, 64), sg.SGEMM_ERR_LD),
    ((F, A, 128, 64, W, 64, 64), sg.SGEMM_ERR_LD), ((F, A, 64, 320, W, 65, 400), sg.SGEMM_OK),  # heads outermost
    ((F, A, 64, 319, W, 128, 64), sg.SGEMM_ERR_LD), ((F, A, -128, 64, W, 128, 64), sg.SGEMM_ERR_LD),
    ((F, None, 128, 64, W, 128, 64), sg.SGEMM_ERR_NULL), ((F, A, 128, 64, None, 128, 64), sg.SGEMM_ERR_NULL),
    ((F, K8 + 20 * 1024 - 4, 128, 64, W, 128, 64), sg.SGEMM_ERR_ALIAS), ((F, A, 128, 64, VS + 76, 128, 64), sg.SGEMM_ERR_ALIAS),
    ((F, A, 128, 64, A, 128, 64), sg.SGEMM_OK),  # the same keys and values may be written
]


@pytest.mark.parametrize("args,want", ROW_CASES)
def test_kv8_rows(args, want):
    assert sg.sgemm_kv8_check_args(cache(), batch(), *args) == want
    if want != sg.SGEMM_OK:
        assert sg.sgemm_kv8_write(cache(), batch(), *args, None) == want


def test_kv8_read_outputs_must_not_meet():
    for other in (A, A + 4, TAB, LEN + 8, ST):
        assert sg.sgemm_kv8_read(cache(), batch(), F, A, 128, 64, other, 128, 64, None) == sg.SGEMM_ERR_ALIAS


def att(dtype=F, heads_q=4, Q=Q, ldq=256, hsq=64, scale=0.125, causal=1, window=0, O=O, ldo=256, hso=64, ws=None, n=0):
    return dtype, heads_q, Q, ldq, hsq, scale, causal, window, O, ldo, hso, ws, n


ATTEND_CASES = [
    (att(), sg.SGEMM_OK), (att(dtype=5), sg.SGEMM_ERR_DTYPE), (att(heads_q=0), sg.SGEMM_ERR_HEADS), (att(heads_q=3), sg.SGEMM_ERR_HEADS),
    (att(heads_q=-2), sg.SGEMM_ERR_HEADS), (att(causal=2), sg.SGEMM_ERR_MASK), (att(window=-1), sg.SGEMM_ERR_MASK),
    (att(causal=0, window=4), sg.SGEMM_ERR_MASK), (att(window=4), sg.SGEMM_OK), (att(ldq=255), sg.SGEMM_ERR_LD), (att(hso=63), sg.SGEMM_ERR_LD),
    (att(Q=None), sg.SGEMM_ERR_NULL), (att(O=None), sg.SGEMM_ERR_NULL), (att(O=Q), sg.SGEMM_ERR_ALIAS), (att(O=K8), sg.SGEMM_ERR_ALIAS),
    (att(O=TAB), sg.SGEMM_ERR_ALIAS), (att(ws=WS, n=64), sg.SGEMM_OK), (att(ws=O + 5 * 1024 - 4, n=64), sg.SGEMM_ERR_ALIAS),
    (att(ws=V8, n=1), sg.SGEMM_ERR_ALIAS), (att(ws=Q, n=1), sg.SGEMM_ERR_ALIAS), (att(ws=Q, n=0), sg.SGEMM_OK),
]


@pytest.mark.parametrize("args,want", ATTEND_CASES)
def test_kv8_attend_check_args(args, want):
    assert sg.sgemm_kv8_attend_check_args(cache(), batch(), *args) == want
    if want != sg.SGEMM_OK:
        assert sg.sgemm_kv8_attend(cache(), batch(), *args, None) == want


def test_no_device_is_reported_not_crashed():
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert sg.sgemm_w4(*w4(), None) == sg.SGEMM_ERR_DEVICE
    assert sg.sgemm_w4_quantize(*pack(), None) == sg.SGEMM_ERR_DEVICE
    assert sg.sgemm_kv8_write(cache(), batch(), F, A, 128, 64, W, 128, 64, None) == sg.SGEMM_ERR_DEVICE
    assert sg.sgemm_kv8_read(cache(), batch(), F, A, 128, 64, W, 128, 64, None) == sg.SGEMM_ERR_DEVICE
    assert sg.sgemm_kv8_attend(cache(), batch(), *att(), None) == sg.SGEMM_ERR_DEVICE


def test_status_strings_of_these_entry_points():
    codes = (sg.SGEMM_ERR_GROUP, sg.SGEMM_ERR_CACHE, sg.SGEMM_ERR_HEADS, sg.SGEMM_ERR_MASK, sg.SGEMM_ERR_DTYPE)
    texts = [sg.sgemm_status_string(c) for c in codes]
    assert len(set(texts)) == len(codes) and "unknown status" not in texts


def test_the_binding_refuses():
    cpu = torch.zeros(4, 64)
    for call in (lambda: sg.quantize_w4(cpu), lambda: sg.W4(torch.zeros(4, 32, dtype=torch.uint8), cpu, None, 64, 64),
                 lambda: sg.KV8(*[torch.zeros(2, 1, 16, 64, dtype=torch.uint8).view(torch.float8_e4m3fn)] * 2, cpu, cpu)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: sg.gemm_w4(cpu, cpu), lambda: sg.dequantize_w4(cpu), lambda: sg.kv8_write(cpu, cpu, cpu, cpu, cpu, cpu),
                 lambda: sg.kv8_read(cpu, cpu, cpu, cpu), lambda: sg.kv8_attend(cpu, cpu, cpu, cpu, cpu),
                 lambda: sg.quantize_w4(torch.zeros(4)), lambda: sg.quantize_w4(cpu.double())):
        with pytest.raises(TypeError):
            call()


@pytest.mark.skipif(shutil.which("g++") is None, reason="no g++")
def test_checks_under_sanitizers(tmp_path):
    exe = str(tmp_path / "lowbit_checks")
    cmd = ["g++", "-std=c++17", *SAN, f"-I{os.path.join(ROOT, 'include')}", f"-I{CSRC}",
           os.path.join(HERE, "lowbit_checks.cpp"), os.path.join(CSRC, "args_lowbit.cpp"), "-o", exe]
    assert "lowbit checks ok" in _build_and_run(cmd, exe, tmp_path)

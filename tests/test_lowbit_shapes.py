"""How the products held in few bits are laid out over the device, on the host
(no GPU needed)."""

import ctypes
import os
import shutil

import pytest

import dense_fp32_matrix_sgemm_amd as sg
from tests.test_lowbit_host import batch, cache
from tests.test_sanitizers import CSRC, HERE, ROOT, SAN, _build_and_run

F, BF, H = sg.SGEMM_F32, sg.SGEMM_LP_BF16, sg.SGEMM_LP_F16


def test_w4_shapes():
    # Few rows: columns over waves with many of them, K over waves else; A in slabs, or straight to registers.
    assert sg.sgemm_w4_shape(H, 1, 1024, 1024) == (16, 16, 1, 4, 1)
    assert sg.sgemm_w4_shape(BF, 1, 16384, 4096) == (16, 64, 4, 4, 1)
    assert sg.sgemm_w4_shape(BF, 8, 4096, 100) == (16, 16, 1, 1, 1)       # less than one step of 256 k
    assert sg.sgemm_w4_shape(F, 16, 8192, 8192) == (16, 32, 2, 8, 5)
    assert sg.sgemm_w4_shape(F, 13, 2047, 4093) == (16, 16, 1, 16, 0)
    # More rows: the larger tile as soon as every compute unit has one, then K over waves.
    for dtype in (BF, H):
        assert sg.sgemm_w4_shape(dtype, 9, 100, 500) == (32, 32, 1, 8, 1)
        assert sg.sgemm_w4_shape(dtype, 33, 100, 500) == (64, 32, 1, 8, 1)
        assert sg.sgemm_w4_shape(dtype, 257, 8200, 500) == (64, 64, 1, 4, 1)
        assert sg.sgemm_w4_shape(dtype, 2048, 4096, 4096) == (64, 256, 4, 1, 1)
        assert sg.sgemm_w4_shape(dtype, 2048, 2048, 4096, cus=128) == (64, 256, 4, 1, 1)
    assert sg.sgemm_w4_shape(F, 17, 100, 500) == (32, 32, 1, 4, 1)
    assert sg.sgemm_w4_shape(F, 257, 8200, 500) == (32, 32, 1, 4, 1)
    assert sg.sgemm_w4_shape(F, 2048, 2048, 4096) == (64, 256, 4, 1, 1)
    assert sg.sgemm_w4_shape(F, 0, 0, 0)[0] == 16


def test_w4_shape_refuses():
    for args in ((3, 4, 4, 4), (F, -1, 4, 4), (F, 4, -1, 4), (F, 4, 4, -1), (F, 4, 4, 2**30 + 1)):
        with pytest.raises(sg.SgemmError) as e:
            sg.sgemm_w4_shape(*args)
        assert e.value.status == (sg.SGEMM_ERR_DTYPE if args[0] == 3 else sg.SGEMM_ERR_DIM)
    assert sg.load_library().sgemm_w4_shape(F, 4, 4, 4, 0, None) == sg.SGEMM_ERR_NULL


def test_kv8_attend_shapes():
    def shape(seqs, heads, ratio, new, dim=128, columns=64, block=64, window=0, cus=0):
        b = batch(seqs=seqs, table_ld=columns, rows=seqs * new, max_new=new)
        return sg.sgemm_kv8_attend_shape(cache(pages=9, heads=heads, block=block, dim=dim), b, heads * ratio, window, cus)

    # One token: 16 rows, split over as many work-groups as the compute units hold.
    assert shape(1, 1, 8, 1) == (16, 1, 1, 16)
    assert shape(32, 8, 4, 1, columns=128) == (16, 1, 1, 3)
    assert shape(1, 1, 8, 1, window=200) == (16, 1, 1, 1)
    assert shape(512, 8, 4, 1) == (16, 1, 1, 1)
    # Some rows, and prompts: two groups of 16 a wave but for the longest heads; four tiles a work-group once they fill the device.
    assert shape(1, 2, 4, 10)[:2] == (32, 1)
    assert shape(1, 2, 4, 10, dim=256)[:2] == (16, 1)
    assert shape(2, 8, 4, 1024) == (32, 4, 32, 1)
    assert shape(2, 8, 4, 1024, dim=144) == (16, 4, 64, 1)
    assert shape(32, 8, 1, 128) == (32, 4, 1, 1)
    assert shape(32, 8, 1, 127)[1] == 1


def test_kv8_attend_shape_refuses():
    none = ctypes.POINTER(sg.KV8Cache)()
    for c, b, heads_q, window, want in ((none, batch(), 4, 0, sg.SGEMM_ERR_NULL), (cache(pages=0), batch(), 4, 0, sg.SGEMM_ERR_DIM),
                                        (cache(dim=8), batch(), 4, 0, sg.SGEMM_ERR_CACHE), (cache(), batch(), 3, 0, sg.SGEMM_ERR_HEADS),
                                        (cache(), batch(), 4, -1, sg.SGEMM_ERR_MASK)):
        with pytest.raises(sg.SgemmError) as e:
            sg.sgemm_kv8_attend_shape(c, b, heads_q, window)
        assert e.value.status == want
    assert sg.load_library().sgemm_kv8_attend_shape(cache(), batch(), 4, 0, 0, None) == sg.SGEMM_ERR_NULL


@pytest.mark.skipif(shutil.which("g++") is None, reason="no g++")
def test_shapes_under_sanitizers(tmp_path):
    exe = str(tmp_path / "lowbit_shapes")
    cmd = ["g++", "-std=c++17", *SAN, f"-I{os.path.join(ROOT, 'include')}", f"-I{CSRC}",
           os.path.join(HERE, "lowbit_shapes.cpp"), os.path.join(CSRC, "args_lowbit.cpp"), "-o", exe]
    assert "lowbit shapes ok" in _build_and_run(cmd, exe, tmp_path)

"""Which sequence a row or a work-group of a serving step falls to, at counts of
sequences next to 2^31 (no GPU needed)."""

import os
import shutil

import pytest

from tests.test_sanitizers import CSRC, HERE, ROOT, SAN, _build_and_run


@pytest.mark.skipif(shutil.which("g++") is None, reason="no g++")
def test_sequences_up_to_31_bits(tmp_path):
    exe = str(tmp_path / "step_search")
    cmd = ["g++", "-std=c++17", *SAN, f"-I{os.path.join(ROOT, 'include')}", f"-I{CSRC}", os.path.join(HERE, "step_search.cpp"), "-o", exe]
    assert "step search ok" in _build_and_run(cmd, exe, tmp_path)

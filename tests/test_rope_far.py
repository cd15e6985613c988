"""cos and sin of far positions: good to 2^-22 for angles up to 2^30 (GPU
tests)."""

import numpy as np
import pytest
import torch

import dense_fp32_matrix_sgemm_amd as sg

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sg.load_library()


def worst(positions, freqs, inverse=False):
    """The largest error of cos and sin, in units of 2^-22: what unit vectors are turned to.

    The angle is formed in extended precision (64 bits: off by 2^-34 at 2^30)."""
    rows, half = len(positions), len(freqs)
    x = torch.zeros(rows, 1, 2 * half, device="cuda")
    x[..., :half] = 1
    y = sg.rope(x, None, torch.from_numpy(positions).cuda(), torch.from_numpy(freqs).cuda(), inverse=inverse)
    y = y[:, 0].cpu().numpy().astype(np.longdouble)
    angle = positions.astype(np.longdouble)[:, None] * freqs.astype(np.longdouble)[None, :]
    sine = -np.sin(angle) if inverse else np.sin(angle)
    return float(max(np.abs(y[:, :half] - np.cos(angle)).max(), np.abs(y[:, half:] - sine).max())) * 2**22


# What is left of the angle, at most pi / 4, becomes float32 (u = 2^-24 of it) and is
# multiplied (u, and 0.5 u for the rounded pi / 2): 2.5 u pi / 4 of an angle, 1.4 u of
# cos or sin. Their polynomials end in values below 1 (0.5 u), after roundings of y
# and of the terms before of another u at most: 3 u.
LIMIT = 3 / 4

# Angles at which the roundings of position times frequency and of 2 / pi add up.
FAR = [(1040586219, "0x1.f9625e955e379p-1"), (1063987612, "0x1.eb653263db716p-1"), (1060660240, "0x1.f7ce4bc6a6fa4p-1"),
       (1056496415, "0x1.f93cbb303703cp-1"), (1056203933, "0x1.fb0ac7512de9bp-1"), (1070009864, "0x1.e523f8d14b7b8p-1"),
       (1071021006, "0x1.c80346c531389p-1"), (1062324160, "0x1.e9065cf7f0a3dp-1"), (1011764651, "0x1.f27494476e6ccp-1"),
       (1040894897, "0x1.fe9fc99ea5d22p-1"), (1053929980, "0x1.d0ca1076a0fa1p-1"), (1064468139, "0x1.e103996c770aap-1")]


@pytest.mark.parametrize("inverse", [False, True])
def test_angles_whose_roundings_add_up(inverse):
    got = [worst(np.array([p], np.int32), np.array([float.fromhex(f)]), inverse) for p, f in FAR]
    print("[far]", [round(x, 3) for x in got], flush=True)
    assert max(got) <= LIMIT


@pytest.mark.parametrize("bits", [0, 4, 10, 17, 24, 28, 30])
def test_angles_of_every_size(bits):
    rng = np.random.default_rng(bits)
    positions = rng.integers(2**30 // 2, 2**30, 3000, dtype=np.int32)
    positions[::2] *= -1
    freqs = rng.uniform(0.5, 1, 300) * 2.0**(bits - 30)
    got = worst(positions, freqs)
    print("[far]", bits, got, flush=True)
    assert got <= LIMIT

"""Operands of a serving step that lie between one another in one buffer: which
calls are refused (no GPU needed), and that the others give what separate
tensors give (GPU tests)."""

import itertools
import random

import pytest
import torch

import dense_fp32_matrix_sgemm_amd as sg
from tests.test_lowbit_host import batch
from tests.test_step_host import FR, POS, Q, cache

F, BF, H = sg.SGEMM_F32, sg.SGEMM_LP_BF16, sg.SGEMM_LP_F16
SIZE = {F: 4, BF: 2, H: 2}
AT = 2**44  # far from positions and frequencies, whatever the operand spans


def turn(rows, dim, first, second, dtype=F, otype=F):
    return sg.sgemm_rope_check_args(dtype, otype, rows, dim, dim - dim % 2, 0, 0, 1.0, POS, FR, first, second)


def in_place(at, heads, ld, hs):
    return sg.RopeRows(at, at, heads, ld, hs, ld, hs)


@pytest.mark.parametrize("rows", [1, 2, 4, 1000])
@pytest.mark.parametrize("heads,parts,dim", [(2, 2, 64), (8, 3, 128), (1, 3, 64), (40, 3, 80), (65536, 2, 64)])
def test_heads_side_by_side(rows, heads, parts, dim):
    # One buffer, rows x heads x parts x dim; padded rows too, and heads outermost.
    hs = parts * dim
    for pad in (0, 8, dim):
        ld = heads * hs + pad
        for a, b in itertools.permutations(range(parts), 2):
            qa, qb = in_place(AT + 4 * a * dim, heads, ld, hs), in_place(AT + 4 * b * dim, heads, ld, hs)
            assert turn(rows, dim, qa, qb) == sg.SGEMM_OK, (pad, a, b)
            if abs(a - b) == 1:  # one element towards its neighbour
                one = in_place(AT + 4 * b * dim + (-4 if a < b else 4), heads, ld, hs)
                assert turn(rows, dim, qa, one) == sg.SGEMM_ERR_ALIAS, (pad, a, b)
    outer = [in_place(AT + 4 * a * dim, heads, parts * dim, rows * parts * dim) for a in range(parts)]
    if heads * rows * parts * dim < 2**31:
        for a, b in itertools.permutations(range(parts), 2):
            assert turn(rows, dim, outer[a], outer[b]) == sg.SGEMM_OK


def taken(at, rows, heads, dim, ld, hs, elem):
    """The bytes that an operand holds."""
    return {at + (r * ld + h * hs) * elem + x for r in range(rows) for h in range(heads) for x in range(dim * elem)}


def nested(rng, rows, heads, dim):
    """Strides of which elements share no places, heads inside rows or rows inside heads."""
    if rng.random() < 0.6:
        hs = dim * rng.randint(1, 4) + rng.randint(0, 2)
        return (heads - 1) * hs + dim + rng.randint(0, 3 * dim), hs
    ld = dim * rng.randint(1, 4) + rng.randint(0, 2)
    return ld, (rows - 1) * ld + dim + rng.randint(0, 3 * dim)


def test_every_byte_of_small_operands():
    # Queries and keys of equal strides are refused exactly where they share a byte.
    rng = random.Random(1)
    seen = {True: 0, False: 0}
    for i in range(4000):
        rows, dim, dtype = rng.randint(1, 4), rng.randint(1, 5), rng.choice([F, BF])
        heads = [rng.randint(1, 4), rng.randint(1, 4)]
        ld, hs = nested(rng, rows, max(heads), dim)
        elem = SIZE[dtype]
        at = [2**20, 2**20 + elem * rng.randint(-2 * dim * 4, 2 * dim * 4)]
        # Strides of one row or one head mean nothing.
        strides = [(ld if rows > 1 else rng.randint(-9, 99), hs if heads[k] > 1 else rng.randint(-9, 99)) for k in range(2)]
        meet = bool(taken(at[0], rows, heads[0], dim, ld, hs, elem) & taken(at[1], rows, heads[1], dim, ld, hs, elem))
        got = turn(rows, dim, *(in_place(at[k], heads[k], *strides[k]) for k in range(2)), dtype=dtype, otype=dtype)
        assert got == (sg.SGEMM_ERR_ALIAS if meet else sg.SGEMM_OK), (i, rows, heads, dim, ld, hs, at)
        seen[meet] += 1
    assert min(seen.values()) > 500


def test_equal_strides_in_bytes():
    # A float32 operand and a 16-bit output of half the stride that lie in the gaps of each other.
    x, y = sg.RopeRows(Q, Q + 4 * 64, 2, 512, 192, 1024, 384), sg.RopeRows(Q, Q + 4 * 63, 2, 512, 192, 1024, 384)
    assert turn(5, 64, x, None, F, BF) == sg.SGEMM_OK and turn(5, 64, y, None, F, BF) == sg.SGEMM_ERR_ALIAS
    # Other strides: refused where the ranges meet, as the header says.
    assert turn(5, 64, sg.RopeRows(Q, Q + 4 * 64, 2, 512, 192, 1536, 384), None, F, BF) == sg.SGEMM_ERR_ALIAS


def test_outputs_read_back_side_by_side():
    c, b = cache(heads=2, dim=64), batch(rows=5)
    for ld, hs, off in ((256, 128, 64), (320, 128, 64), (128, 1280, 64)):
        for at, other in ((Q, Q + 4 * off), (Q + 4 * off, Q)):
            if not torch.cuda.is_available():
                assert sg.sgemm_kv4_read(c, b, F, at, ld, hs, other, ld, hs, None) == sg.SGEMM_ERR_DEVICE, (ld, hs)
        assert sg.sgemm_kv4_read(c, b, F, Q, ld, hs, Q + 4 * off - 4, ld, hs, None) == sg.SGEMM_ERR_ALIAS


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,heads,dim,rot", [(1, 2, 64, 64), (5, 3, 80, 48), (700, 32, 128, 128)])
def test_rope_in_place_in_a_buffer_of_heads(rows, heads, dim, rot, dtype):
    buf = torch.randn(rows, heads, 3, dim, generator=torch.Generator().manual_seed(rows)).to(dtype).cuda()
    positions = torch.arange(rows, dtype=torch.int32, device="cuda") * 77
    freqs = sg.rope_frequencies(rot)[0]
    q, k, v = (buf[:, :, i].clone() for i in range(3))
    want = sg.rope(q, k, positions, freqs)
    got = sg.rope(buf[:, :, 0], buf[:, :, 1], positions, freqs, out=(buf[:, :, 0], buf[:, :, 1]))
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(buf[:, :, 2], v)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_read_back_into_a_buffer_of_heads(dtype):
    from tests.test_parity_kv4 import Case4

    case = Case4(3, [700, 45], [650, 20], 6, 16, 80)
    args, c = case.args(), case.device()
    K, V = sg.kv4_read(c, *args, rows=case.rows, dtype=dtype)
    buf = torch.full((case.rows, 6, 2, 80), 3.25, dtype=dtype, device="cuda")
    sg.kv4_read(c, *args, K=buf[:, :, 1], V=buf[:, :, 0])
    assert torch.equal(buf[:, :, 1], K) and torch.equal(buf[:, :, 0], V)

"""Rotary positions against their definition in extended precision (GPU
tests)."""

import numpy as np
import pytest
import torch

import dense_fp32_matrix_sgemm_amd as sg
from tests import step_ref as ref
from tests.test_parity_kv8 import TYPES, views

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sg.load_library()


def bound(x, positions, freqs, interleaved, amplitude, want, otype):
    """cos and sin each within 3.5 u (u = 2^-24: the argument, the polynomial
    and its rounding, the amplitude's product), the amplitude's own rounding u,
    the angle's in float64, two products and a sum: (7 u + |angle| 2^-51) of
    amplitude (|a| + |b|). The result is rounded to its type, by half a unit of
    float16's least one where it falls among its subnormals."""
    half = len(freqs)
    angle = np.abs(positions.astype(np.float64)[:, None] * freqs[None, :])[:, None]
    y = np.zeros_like(x)
    ia = np.arange(half) * 2 if interleaved else np.arange(half)
    ib = ia + 1 if interleaved else ia + half
    pair = (7 * 2.0**-24 + angle * 2.0**-51) * abs(amplitude) * (np.abs(x[..., ia]) + np.abs(x[..., ib]))
    y[..., ia], y[..., ib] = pair, pair
    eps = torch.finfo(TYPES[otype]).eps / 2 if otype != "f32" else 0.0
    return y + (np.abs(want) + y) * eps + (2.0**-25 if otype == "f16" else 1e-37)


def check(Q, K, positions, freqs, got, otype, interleaved=False, amplitude=1.0, inverse=False, what=""):
    for name, x, y in (("Q", Q, got[0]), ("K", K, got[1])):
        x, y = x.double().cpu().numpy(), y.double().cpu().numpy()
        want = ref.rope(x, positions, freqs, interleaved, amplitude, inverse)
        b = bound(x, positions, freqs, interleaved, amplitude, want, otype)
        off = np.abs(y - want)
        assert (off <= b).all(), (what, name, float((off / b).max()))


def operands(seed, rows, heads, kv_heads, dim, dtype):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(rows, heads, dim, generator=g).to(TYPES[dtype]), torch.randn(rows, kv_heads, dim, generator=g).to(TYPES[dtype])


@pytest.mark.parametrize("otype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dim,rot", [(64, 64), (128, 128), (80, 32), (96, 18), (1, 0), (2, 2), (7, 6), (50, 0), (256, 254), (33, 16), (1024, 1024)])
def test_every_shape(dim, rot, interleaved, dtype, otype):
    print(f"[rope] dim={dim} rot={rot} interleaved={interleaved} {dtype} to {otype}", flush=True)
    freqs = sg.rope_frequencies(rot)[0].cpu().numpy() if rot else np.zeros(0)
    f = torch.from_numpy(freqs).cuda()
    for i, (rows, heads, kv_heads, layout) in enumerate(((1, 1, 1, "packed"), (5, 6, 2, "padded"), (37, 3, 3, "heads"))):
        Q, K = operands(i + dim, rows, heads, kv_heads, dim, dtype)
        positions = torch.randint(0, 5000, (rows,), generator=torch.Generator().manual_seed(i), dtype=torch.int32)
        outs = [views(torch.full(t.shape, 3.25, dtype=TYPES[otype]), layout) for t in (Q, K)]
        got = sg.rope(views(Q, layout), views(K, layout), positions.cuda(), f, interleaved=interleaved, out=outs)
        assert got[0] is outs[0] and got[1] is outs[1]
        check(Q, K, positions.numpy(), freqs, got, otype, interleaved, what=layout)
        new = sg.rope(Q.cuda(), K.cuda(), positions.cuda(), f, interleaved=interleaved, dtype=TYPES[otype])
        assert all(torch.equal(a.cpu(), b.cpu()) for a, b in zip(got, new))
        one = sg.rope(Q.cuda(), None, positions.cuda(), f, interleaved=interleaved, dtype=TYPES[otype])
        assert torch.equal(one, new[0])
        # Components behind the turned ones are copied, rounded to the type.
        assert torch.equal(new[0][..., rot:].cpu(), Q[..., rot:].float().to(TYPES[otype]))


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows", [1, 255, 4099])
def test_rows_and_the_place_they_go_to(rows, dtype):
    # Enough rows for several at once a work-group; queries, keys and values in one buffer, turned in place.
    heads, kv_heads, dim = 4, 2, 64
    g = torch.Generator().manual_seed(rows)
    qkv = torch.randn(rows, heads + 2 * kv_heads, dim, generator=g).to(TYPES[dtype])
    positions = torch.randint(0, 100000, (rows,), generator=g, dtype=torch.int32)
    freqs, _ = sg.rope_frequencies(dim)
    buf = qkv.cuda()
    Q, K = buf[:, :heads], buf[:, heads:heads + kv_heads]
    want = sg.rope(Q, K, positions.cuda(), freqs)
    check(qkv[:, :heads], qkv[:, heads:heads + kv_heads], positions.numpy(), freqs.cpu().numpy(), want, dtype)
    got = sg.rope(Q, K, positions.cuda(), freqs, out=(Q, K))
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert torch.equal(buf[:, heads + kv_heads:].cpu(), qkv[:, heads + kv_heads:])
    # Part of each head in place: the rest stays.
    buf = qkv.cuda()
    sg.rope(buf[:, :heads], None, positions.cuda(), freqs[:8], out=buf[:, :heads])
    assert torch.equal(buf[..., 16:].cpu(), qkv[..., 16:])
    check(qkv[:, :heads], qkv[:, :0], positions.numpy(), freqs[:8].cpu().numpy(), (buf[:, :heads], buf[:, :0]), dtype)


@pytest.mark.parametrize("dtype,otype", [("bf16", "bf16"), ("f16", "f16"), ("f32", "bf16"), ("bf16", "f16"), ("f16", "f32")])
@pytest.mark.parametrize("dim,rot", [(128, 128), (80, 48), (72, 40)])
def test_more_rows_than_the_caches_hold(dim, rot, dtype, otype):
    print(f"[rope] large dim={dim} rot={rot} {dtype} to {otype}", flush=True)
    rows = 4099
    Q, K = operands(dim, rows, 6, 3, dim, dtype)
    positions = torch.randint(0, 100000, (rows,), generator=torch.Generator().manual_seed(dim), dtype=torch.int32)
    freqs, _ = sg.rope_frequencies(rot)
    got = sg.rope(Q.cuda(), K.cuda(), positions.cuda(), freqs, dtype=TYPES[otype])
    check(Q, K, positions.numpy(), freqs.cpu().numpy(), got, otype)
    # Rows that begin at an odd element, and in place.
    wide = [torch.full((rows, t.shape[1] + 1, dim + 1), 3.25, device="cuda").to(TYPES[otype]) for t in (Q, K)]
    outs = [w[:, :-1, 1:] for w in wide]
    sg.rope(Q.cuda(), K.cuda(), positions.cuda(), freqs, out=outs)
    assert all(torch.equal(a, b) for a, b in zip(outs, got))
    assert all((w[:, -1] == 3.25).all() and (w[..., 0] == 3.25).all() for w in wide)
    if dtype == otype:
        q, k = Q.cuda(), K.cuda()
        sg.rope(q, k, positions.cuda(), freqs, out=(q, k))
        assert torch.equal(q, got[0]) and torch.equal(k, got[1])


@pytest.mark.parametrize("interleaved", [False, True])
def test_positions_from_end_to_end(interleaved):
    # Angles of every quadrant and next to its borders, far positions, negative ones.
    dim = 32
    freqs = np.concatenate([sg.rope_frequencies(dim)[0].cpu().numpy()[:8], np.pi / 2 * np.array([1, 0.5, 1 / 3, 2, 0.25, 1e-9, 0.0, 3.0])])
    positions = np.array([0, 1, 2, 3, 4, 5, 6, 7, 8, -1, -2, -3, 1000, 10**6, 10**6 + 1, 2**24 + 1, 2**30, 2**31 - 1, -(2**31)], np.int32)
    Q, K = operands(5, len(positions), 3, 1, dim, "f32")
    got = sg.rope(Q.cuda(), K.cuda(), torch.from_numpy(positions).cuda(), torch.from_numpy(freqs).cuda(), interleaved=interleaved)
    check(Q, K, positions, freqs, got, "f32", interleaved)


@pytest.mark.parametrize("kind", ["linear", "parts", "other base"])
def test_stretched_contexts(kind):
    dim = 64
    freqs, amplitude = {"linear": lambda: sg.rope_frequencies(dim, stretch=8.0),
                        "parts": lambda: sg.rope_frequencies(dim, stretch=16.0, original=4096),
                        "other base": lambda: sg.rope_frequencies(dim, base=500000.0)}[kind]()
    f = freqs.cpu().numpy()
    plain = 10000.0 ** (-np.arange(32) / 32)
    if kind == "linear":
        assert np.allclose(f, plain / 8, rtol=1e-14) and amplitude == 1
    elif kind == "parts":
        turns = plain * 4096 / (2 * np.pi)
        assert np.allclose(f[turns >= 32], plain[turns >= 32], rtol=1e-14) and np.allclose(f[turns <= 1], plain[turns <= 1] / 16, rtol=1e-14)
        assert (np.diff(f) < 0).all() and abs(amplitude - (0.1 * np.log(16) + 1)) < 1e-15
    else:
        assert np.allclose(f, 500000.0 ** (-np.arange(32) / 32), rtol=1e-14)
    positions = np.arange(0, 65536, 997, dtype=np.int32)
    Q, K = operands(6, len(positions), 2, 1, dim, "f32")
    got = sg.rope(Q.cuda(), K.cuda(), torch.from_numpy(positions).cuda(), freqs, amplitude=amplitude)
    check(Q, K, positions, f, got, "f32", amplitude=amplitude)


@pytest.mark.parametrize("interleaved", [False, True])
def test_the_gradient(interleaved):
    # The matrix of the map by differences (it is linear: its values on unit vectors), and the gradient's as its transpose.
    dim, rot, rows = 12, 10, 12
    freqs = sg.rope_frequencies(rot)[0]
    unit = torch.eye(dim).view(rows, 1, dim).cuda()
    for position in (0, 3, 77777):
        positions = torch.full((rows,), position, dtype=torch.int32).cuda()
        J = sg.rope(unit, None, positions, freqs, interleaved=interleaved, amplitude=1.25)[:, 0].double()
        G = sg.rope(unit, None, positions, freqs, interleaved=interleaved, amplitude=1.25, inverse=True)[:, 0].double()
        # Both are rounded products of the same cos, sin and amplitude.
        assert torch.equal(J, G.t())
        h = 0.5
        x = torch.randn(1, 1, dim, generator=torch.Generator().manual_seed(1)).cuda().expand(rows, 1, dim).contiguous()
        up, down = (sg.rope(x + s * h * unit, None, positions, freqs, interleaved=interleaved, amplitude=1.25)[:, 0].double() for s in (1, -1))
        # x +- h is rounded (2^-24 of at most 4), each value of the map within 7 u of its pair's size (at most 8).
        assert (((up - down) / (2 * h) - J).abs() <= (2 * 4 * 2.0**-24 + 2 * 7 * 2.0**-24 * 1.25 * 8) / (2 * h)).all()
    g = torch.randn(5, 3, dim, generator=torch.Generator().manual_seed(2))
    positions = np.array([0, 1, 50, 4000, 123456], np.int32)
    got = sg.rope(g.cuda(), g.cuda(), torch.from_numpy(positions).cuda(), freqs, interleaved=interleaved, amplitude=1.25, inverse=True)
    check(g, g, positions, freqs.cpu().numpy(), got, "f32", interleaved, 1.25, inverse=True)
    # The gradient of sum(g * rope(x)) by automatic differentiation of the formula.
    x = torch.randn(5, 3, dim, dtype=torch.float64, generator=torch.Generator().manual_seed(3), requires_grad=True)
    angle = torch.from_numpy(positions).double()[:, None, None] * freqs.cpu()
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    ga, gb = (g[..., 0:rot:2], g[..., 1:rot:2]) if interleaved else (g[..., :rot // 2], g[..., rot // 2:rot])
    y = 1.25 * ((a * angle.cos() - b * angle.sin()) * ga + (b * angle.cos() + a * angle.sin()) * gb)
    (y.sum() + (x[..., rot:] * g[..., rot:]).sum()).backward()
    limit = bound(g.double().numpy(), positions, freqs.cpu().numpy(), interleaved, 1.25, x.grad.numpy(), "f32")
    assert (np.abs(got[0].double().cpu().numpy() - x.grad.numpy()) <= limit + 1e-12).all()


def test_numbers_that_are_not_finite_stay_in_their_pair():
    dim = 32
    Q, K = operands(8, 4, 2, 1, dim, "f32")
    Q[1, 0, 3], Q[2, 1, 20] = float("nan"), float("inf")
    freqs = sg.rope_frequencies(dim)[0]
    positions = torch.tensor([1, 2, 3, 4], dtype=torch.int32).cuda()
    got, _ = sg.rope(Q.cuda(), K.cuda(), positions, freqs)
    bad = ~torch.isfinite(got.cpu())
    want = torch.zeros_like(bad)
    want[1, 0, [3, 19]] = True
    want[2, 1, [4, 20]] = True
    assert torch.equal(bad, want)


def test_many_rows_and_offsets_past_31_bits():
    # A buffer of more than 2^31 elements of which the last rows are turned, by a stride of its own.
    rows, dim, ld = 9, 64, 2**28
    buf = torch.zeros(rows * ld, dtype=torch.bfloat16, device="cuda")
    x = torch.as_strided(buf, (rows, 2, dim), (ld, 128, 1))
    Q, _ = operands(9, rows, 2, 1, dim, "bf16")
    x.copy_(Q.cuda())
    freqs = sg.rope_frequencies(dim)[0]
    positions = np.arange(rows, dtype=np.int32) * 1000
    sg.rope(x, None, torch.from_numpy(positions).cuda(), freqs, out=x)
    check(Q, Q[:, :0], positions, freqs.cpu().numpy(), (x, x[:, :0]), "bf16")


def test_the_helper_refuses():
    Q, K = (t.cuda() for t in operands(1, 4, 2, 1, 64, "f32"))
    pos = torch.arange(4, dtype=torch.int32).cuda()
    f = sg.rope_frequencies(64)[0]
    bad = {
        TypeError: [lambda: sg.rope(Q.double(), None, pos, f), lambda: sg.rope(Q, K.half(), pos, f), lambda: sg.rope(Q, K, pos.long(), f),
                    lambda: sg.rope(Q, K, pos, f.float()), lambda: sg.rope(Q[0], None, pos, f), lambda: sg.rope(Q, K, pos, f, dtype=torch.int32),
                    lambda: sg.rope(Q, K, pos, f, out=Q), lambda: sg.rope(Q, K, pos, f, out=(Q, None)),
                    lambda: sg.rope(Q, K, pos, f, dtype=torch.float16, out=(Q, K)), lambda: sg.rope(Q, K, pos, f, out=(Q, K.half()))],
        ValueError: [lambda: sg.rope(Q.cpu(), None, pos, f), lambda: sg.rope(Q, K, pos[:3], f), lambda: sg.rope(Q, K[:3], pos, f),
                     lambda: sg.rope(Q[..., :32], None, pos, f), lambda: sg.rope(Q, K[..., :32], pos, f), lambda: sg.rope(Q, None, pos, f, out=K),
                     lambda: sg.rope(Q.transpose(1, 2), None, pos, f), lambda: sg.rope(Q, None, pos.repeat(2)[::2], f),
                     lambda: sg.rope(Q, None, pos.cpu(), f), lambda: sg.rope_frequencies(63), lambda: sg.rope_frequencies(64, stretch=0.5)],
        sg.SgemmError: [lambda: sg.rope(Q, Q, pos, f, out=(Q, Q)), lambda: sg.rope(Q[:1].expand(4, 2, 64), None, pos, f),
                        lambda: sg.rope(Q, None, pos, f, out=Q.flatten().view(2, 4, 64).transpose(0, 1)),
                        lambda: sg.rope(torch.zeros(2, 1, 1026, device="cuda"), None, pos[:2], f)],
    }
    before = Q.clone(), K.clone()
    for error, calls in bad.items():
        for i, call in enumerate(calls):
            with pytest.raises(error):
                call()
                pytest.fail(f"{error.__name__} {i} was not refused")
    assert torch.equal(before[0], Q) and torch.equal(before[1], K)


def test_calls_with_nothing_to_do():
    none = torch.empty(0, 2, 64, device="cuda")
    f = sg.rope_frequencies(64)[0]
    q, k = sg.rope(none, none, torch.empty(0, dtype=torch.int32, device="cuda"), f)
    assert q.shape == none.shape and k.shape == none.shape

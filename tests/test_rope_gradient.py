"""The gradient of rotary positions by automatic differentiation, against that
of the formula in 64 bits and against differences (GPU tests)."""

import numpy as np
import pytest
import torch

import dense_fp32_matrix_sgemm_amd as sg
from tests.test_parity_kv8 import TYPES
from tests.test_parity_rope import bound, operands

pytestmark = pytest.mark.gpu

POSITIONS = [0, 1, 50, 4000, 123456, 7, 9]


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    sg.load_library()


def formula(x, freqs, interleaved, amplitude, inverse):
    """The map in 64 bits, of elementary operations."""
    rot = 2 * len(freqs)
    angle = torch.tensor(POSITIONS, dtype=torch.float64)[:, None, None] * freqs.cpu()
    c, s = angle.cos(), angle.sin() * (-1 if inverse else 1)
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    a, b = amplitude * (a * c - b * s), amplitude * (b * c + a * s)
    turned = torch.stack((a, b), dim=-1).flatten(-2) if interleaved else torch.cat((a, b), dim=-1)
    return torch.cat((turned, x[..., rot:]), dim=-1)


@pytest.mark.parametrize("inverse", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype,out", [("f32", None), ("bf16", None), ("f16", "f32"), ("f32", "bf16"), ("bf16", "f16")])
def test_the_gradient_reaches_queries_and_keys(dtype, out, interleaved, inverse):
    dim, rot, amplitude = 24, 20, 1.25
    freqs, positions = sg.rope_frequencies(rot)[0], torch.tensor(POSITIONS, dtype=torch.int32).cuda()
    Q, K = operands(3, len(POSITIONS), 6, 2, dim, dtype)
    q, k = (t.cuda().requires_grad_() for t in (Q, K))
    got = sg.rope(q, k, positions, freqs, interleaved=interleaved, amplitude=amplitude, inverse=inverse, dtype=TYPES[out] if out else None)
    with torch.no_grad():
        plain = sg.rope(q, k, positions, freqs, interleaved=interleaved, amplitude=amplitude, inverse=inverse, dtype=TYPES[out] if out else None)
    assert all(y.requires_grad and torch.equal(y, p) and not p.requires_grad for y, p in zip(got, plain))
    g = [torch.randn(y.shape, generator=torch.Generator().manual_seed(i)).to(y.dtype) for i, y in enumerate(got)]
    torch.autograd.backward(got, [t.cuda() for t in g])
    for x, d, leaf in ((Q, g[0], q), (K, g[1], k)):
        y = x.double().requires_grad_()
        formula(y, freqs, interleaved, amplitude, inverse).backward(d.double())
        limit = bound(d.double().numpy(), np.array(POSITIONS, np.int32), freqs.cpu().numpy(), interleaved, amplitude, y.grad.numpy(), dtype)
        assert leaf.grad.dtype == x.dtype
        # Components behind the turned ones come as they are, rounded to the type.
        eps = torch.finfo(x.dtype).eps / 2
        assert (np.abs(leaf.grad.double().cpu().numpy() - y.grad.numpy()) <= limit + eps * np.abs(y.grad.numpy())).all()


def test_the_gradient_against_differences():
    # sum(g * rope(x)) is linear in x: its difference over x +- h is the gradient, but for roundings.
    dim, rot, h = 12, 10, 0.5
    freqs, positions = sg.rope_frequencies(rot)[0], torch.tensor(POSITIONS, dtype=torch.int32).cuda()
    x, _ = operands(4, len(POSITIONS), 1, 1, dim, "f32")
    x = (x * 8).round() / 8  # x +- h are exact, and below 8
    g = torch.randn(x.shape, generator=torch.Generator().manual_seed(5))
    leaf = x.cuda().requires_grad_()
    (sg.rope(leaf, None, positions, freqs) * g.cuda()).sum().backward()
    for i in range(dim):
        step = torch.zeros(dim)
        step[i] = h
        up, down = ((sg.rope((x + s * step).cuda(), None, positions, freqs).double().cpu() * g).sum((1, 2)) for s in (1, -1))
        # Each component of the map within 7 u of its pair's |a| + |b| <= 16; the gradient itself within 7 u of its pair's.
        limit = (2 * 7 * 2.0**-24 * 16 * g.abs().sum((1, 2))) / (2 * h) + 7 * 2.0**-24 * 2 * g.abs().amax()
        assert (((up - down) / (2 * h) - leaf.grad.double().cpu()[:, 0, i]).abs() <= limit).all()


def test_which_operands_get_a_gradient():
    dim = 16
    freqs, positions = sg.rope_frequencies(dim)[0], torch.tensor(POSITIONS, dtype=torch.int32).cuda()
    Q, K = (t.cuda() for t in operands(6, len(POSITIONS), 4, 2, dim, "f32"))
    want = sg.rope(torch.ones_like(Q), torch.ones_like(K), positions, freqs, inverse=True)
    # One of the two, either.
    for i in range(2):
        x = [Q.clone(), K.clone()]
        x[i].requires_grad_()
        y = sg.rope(*x, positions, freqs)
        assert y[i].requires_grad and not y[1 - i].requires_grad
        y[i].sum().backward()  # a gradient that is one element, expanded
        assert torch.equal(x[i].grad, want[i]) and x[1 - i].grad is None
    # Both, of which one output alone is used.
    for i in range(2):
        x = [Q.clone().requires_grad_(), K.clone().requires_grad_()]
        sg.rope(*x, positions, freqs)[i].sum().backward()
        assert torch.equal(x[i].grad, want[i]) and x[1 - i].grad is None
    # Through a view of a buffer that holds both, head by head.
    buf = torch.stack((Q[:, :2], K), dim=2).requires_grad_()
    y = sg.rope(buf[:, :, 0], buf[:, :, 1], positions, freqs)
    (y[0].sum() + y[1].sum()).backward()
    assert torch.equal(buf.grad[:, :, 0], want[0][:, :2]) and torch.equal(buf.grad[:, :, 1], want[1])
    # No rows, and none where nothing asks for it.
    none = torch.zeros(0, 2, dim, device="cuda", requires_grad=True)
    sg.rope(none, None, positions[:0], freqs).sum().backward()
    assert none.grad.shape == none.shape
    assert not sg.rope(Q, K, positions, freqs)[0].requires_grad


def test_the_gradient_of_the_gradient():
    dim = 16
    freqs, positions = sg.rope_frequencies(dim)[0], torch.tensor(POSITIONS, dtype=torch.int32).cuda()
    x = operands(7, len(POSITIONS), 2, 1, dim, "f32")[0].cuda().requires_grad_()
    w = torch.ones_like(x).requires_grad_()
    g, = torch.autograd.grad((sg.rope(x, None, positions, freqs) * w).sum(), x, create_graph=True)
    v = torch.randn(x.shape, generator=torch.Generator().manual_seed(8)).cuda()
    h, = torch.autograd.grad((g * v).sum(), w)
    assert torch.equal(h, sg.rope(v, None, positions, freqs))


def test_what_has_no_gradient_is_refused():
    dim = 16
    freqs, positions = sg.rope_frequencies(dim)[0], torch.tensor(POSITIONS, dtype=torch.int32).cuda()
    Q, K = (t.cuda() for t in operands(9, len(POSITIONS), 2, 1, dim, "f32"))
    q, k, f = Q.clone().requires_grad_(), K.clone().requires_grad_(), freqs.clone().requires_grad_()
    out = torch.empty_like(Q), torch.empty_like(K)
    for call in (lambda: sg.rope(q, K, positions, freqs, out=out), lambda: sg.rope(Q, k, positions, freqs, out=out), lambda: sg.rope(Q, K, positions, f),
                 lambda: sg.rope(q, None, positions, freqs, out=q), lambda: sg.rope(Q, K, positions, freqs, out=(q, K))):
        with pytest.raises(ValueError):
            call()
    assert torch.equal(q, Q) and torch.equal(k, K)
    with torch.no_grad():  # in place where no gradient is asked for
        sg.rope(q, k, positions, f, out=(q, k))
    assert torch.equal(q, sg.rope(Q, None, positions, freqs))
    # Positions that change between the pass and its gradient are told.
    x = Q.clone().requires_grad_()
    y = sg.rope(x, None, positions, freqs)
    positions.add_(1)
    with pytest.raises(RuntimeError):
        y.sum().backward()


def test_a_pass_and_its_gradient_captured_together():
    dim, rows = 64, 33
    freqs = sg.rope_frequencies(dim)[0]
    positions = torch.arange(rows, dtype=torch.int32).cuda() * 100
    x = torch.zeros(rows, 4, dim, device="cuda", requires_grad=True)
    d = torch.zeros(rows, 4, dim, device="cuda")

    def step():
        y = sg.rope(x, None, positions, freqs)
        return y.detach(), torch.autograd.grad(y, x, d)[0]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, g = step()
    for replay in range(4):
        gen = torch.Generator().manual_seed(replay)
        a, b = (torch.randn(rows, 4, dim, generator=gen).cuda() for _ in range(2))
        with torch.no_grad():
            x.copy_(a)
        d.copy_(b)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, sg.rope(a, None, positions, freqs)) and torch.equal(g, sg.rope(b, None, positions, freqs, inverse=True))
    del graph

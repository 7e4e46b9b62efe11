"""nn.gated_linear on the GPU against its definition in float64 (bounds derived in
step_helpers), at the sizes where tiles, steps and slices end."""

import pytest
import torch

from precision_optimizer_state_amd import binding as B
from precision_optimizer_state_amd import nn
from step_helpers import TYPES, U, Gated, check, generator, normal

pytestmark = pytest.mark.gpu


def make(seed, rows, cols, features, dtype, pad=0, lead=0):
    gen = generator(seed)
    dt = TYPES[dtype]
    x = normal(gen, rows, cols, dtype=dt, pad=pad, lead=lead)
    gate, up = (normal(gen, features, cols, scale=cols ** -0.5, dtype=dt) for _ in range(2))
    return x, gate, up, normal(gen, rows, features, dtype=dt)


def run(x, gate, up, dy, act="silu"):
    leaves = [a.detach().requires_grad_(True) for a in (x, gate, up)]
    y = nn.gated_linear(*leaves, act)
    return (y,) + torch.autograd.grad(y, leaves, dy)


def against(name, x, gate, up, dy, act="silu"):
    got = run(x, gate, up, dy, act)
    want = Gated(x, gate, up, act, dy)
    for part, g in zip(("y", "dx", "dgate", "dup"), got):
        assert g.dtype == x.dtype
        check(f"{name} {part}", g, getattr(want, part), getattr(want, "d_" + part))
    with torch.no_grad():
        assert torch.equal(nn.gated_linear(x, gate, up, act), got[0].detach())


SIZES = [(1, 1, 1), (1, 64, 2), (2, 7, 3), (31, 64, 31), (32, 64, 32), (33, 65, 33), (64, 32, 63), (65, 96, 64), (63, 63, 65),
         (127, 128, 127), (128, 100, 128), (129, 192, 129), (1, 768, 1000), (1, 4096, 70), (17, 40, 500), (257, 33, 70), (600, 72, 300)]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("rows, cols, features", SIZES)
def test_sizes(rows, cols, features, dtype):
    against(f"{rows}x{cols}x{features}", *make(rows + cols + features, rows, cols, features, dtype))


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("rows, cols, features", [(4095, 64, 2049), (2050, 520, 1030), (300, 1024, 1500)])
def test_larger_tiles(rows, cols, features, dtype):
    against("large", *make(3, rows, cols, features, dtype))


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_activations(act, dtype):
    x, gate, up, dy = make(4, 100, 64, 90, dtype)
    against(act, x * 3, gate, up, dy, act)              # gates of a few units either way


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
def test_far_gates(act):
    """Gates whose sigmoid has reached 0 or 1, and whose square passes float32's range."""
    g = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 20.0, -20.0, 90.0, -90.0, 200.0, -200.0, 1e10, -1e10, 1e20, -1e20], device="cuda")
    x = g[:, None].clone()
    one = torch.ones(1, 1, device="cuda")
    y, dx, dgate, dup = run(x, one, one, torch.ones(14, 1, device="cuda"), act)
    pos = g > 10
    # far out act(g) is g or 0, its slope 1 or 0: y = g act(g), dx = g act' + act
    assert torch.isfinite(y).all() == (g.abs() < 1e19).all()
    fin = g.abs() < 1e19
    assert torch.equal(y[fin & pos], (x * x)[fin & pos]) and torch.equal(dx[fin & pos], 2 * x[fin & pos])
    neg = g <= -200
    assert not y[neg].any() and not dx[neg].any() and not dx.isnan().any() and not y.isnan().any()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("pad, lead", [(1, 0), (0, 3), (8, 0), (8, 8), (61, 2)])
def test_slices(pad, lead, dtype):
    x, gate, up, _ = make(5, 90, 64, 70, dtype, pad=pad, lead=lead)
    dy = normal(generator(6), 90, 70, dtype=TYPES[dtype], pad=pad, lead=lead)
    wide = torch.zeros(70, 64 + pad + lead, device="cuda", dtype=TYPES[dtype])
    wide[:, lead:lead + 64] = up
    against("slices", x, gate, wide[:, lead:lead + 64], dy)      # one weight packed, one not


def test_layouts():
    x, gate, up, dy = make(7, 24, 64, 40, "bf16")
    against("three dimensions", x.view(2, 12, 64), gate, up, dy.view(2, 12, 40))
    against("transposed", x.view(2, 12, 64).transpose(0, 1), gate, up, dy.view(12, 2, 40))
    against("one vector", x[0], gate, up, dy[0])
    against("expanded", x[0].expand(24, 64), gate, up, dy[0].expand(24, 40))
    against("columns", x.t().contiguous().t(), gate.t().contiguous().t(), up, dy)
    # a gate and an up projection side by side in one matrix
    both = torch.cat([gate, up]).view(2, 40, 64)
    against("one matrix", x, both[0], both[1], dy)
    both = torch.stack([gate, up], 1)
    against("alternating rows", x, both[:, 0], both[:, 1], dy)


@pytest.mark.parametrize("rows", [1, 100, 300])
def test_long_float32_sums_are_kept_in_two_levels(rows):
    # 512 terms at a time, then 16 sums of those: of positive terms each product is off by
    # at most 2 U (512 + 16 + 4) of itself (2 U per addition, should the instruction
    # truncate), where one chain could be off by 2 U 8192.  y = g u for g far above 0,
    # where gelu is the identity; 20 U for the activation and the last products.
    gen = generator(16)
    x, gate, up = (0.5 + 0.5 * torch.rand(n, 8192, generator=gen, device="cuda") for n in (rows, 70, 70))
    y = nn.gated_linear(x, gate, up, "gelu").double()
    want = (x.double() @ gate.double().t()) * (x.double() @ up.double().t())
    check("y", y, want, (2 * 2 * (512 + 16 + 4) + 20) * U * want)


def test_one_weight_for_both():
    x, gate, _, dy = make(8, 50, 64, 40, "bf16")
    a = gate.detach().requires_grad_(True)
    nn.gated_linear(x, a, a).backward(dy)
    want = Gated(x, gate, gate, "silu", dy)
    check("both", a.grad, want.dgate + want.dup, want.d_dgate + want.d_dup + 2.0 ** -8 * (want.dgate + want.dup).abs())


def test_empty():
    gate = torch.randn(10, 64, device="cuda", requires_grad=True)
    up = torch.randn(10, 64, device="cuda", requires_grad=True)
    x = torch.randn(0, 64, device="cuda", requires_grad=True)
    y = nn.gated_linear(x, gate, up)
    assert y.shape == (0, 10)
    y.sum().backward()
    assert x.grad.shape == (0, 64) and not gate.grad.any() and not up.grad.any()
    assert nn.gated_linear(torch.randn(3, 0, 64, device="cuda"), gate, up).shape == (3, 0, 10)


def test_only_the_gradients_that_are_needed():
    args = make(9, 70, 64, 50, "bf16")
    want = run(*args)
    for need in range(1, 8):
        leaves = [a.detach().requires_grad_(bool(need >> i & 1)) for i, a in enumerate(args[:3])]
        nn.gated_linear(*leaves).backward(args[3])
        for i, a in enumerate(leaves):
            assert (a.grad is None) != bool(need >> i & 1)
            assert a.grad is None or torch.equal(a.grad, want[1 + i])


def test_gradients_against_differences():
    x, gate, up, dy = make(10, 40, 64, 30, "f32")
    gen = generator(11)
    dirs = [normal(gen, *a.shape, scale=float(a.std())) for a in (x, gate, up)]
    h = 2.0 ** -7
    _, *grads = run(x, gate, up, dy)
    ref = Gated(x, gate, up, "silu", dy)
    ends, exact = [], []
    for sign in (1, -1):
        args = [a + sign * h * d for a, d in zip((x, gate, up), dirs)]
        ends.append(float((nn.gated_linear(*args).double() * dy).sum()))
        exact.append(Gated(*args))
    slope = sum(float((g.double() * d).sum()) for g, d in zip(grads, dirs))
    true = sum(float((g * d).sum()) for g, d in zip((ref.dx, ref.dgate, ref.dup), dirs))
    curve = abs(float(((exact[0].y - exact[1].y) * dy).sum()) / (2 * h) - true)
    room = float(((exact[0].d_y + exact[1].d_y) * dy.abs()).sum()) / (2 * h) + curve + \
        sum(float((b * d.abs()).sum()) for b, d in zip((ref.d_dx, ref.d_dgate, ref.d_dup), dirs))
    assert abs((ends[0] - ends[1]) / (2 * h) - slope) <= room
    # less than a wrong gradient of this size is off by
    size = sum(float((g * g).sum()) for g in (ref.dx, ref.dgate, ref.dup)) ** 0.5 * sum(float((d * d).sum()) for d in dirs) ** 0.5
    assert room < size / sum(d.numel() for d in dirs) ** 0.5


def test_nothing_behind_the_outputs_is_written():
    x, gate, up, dy = make(12, 37, 72, 131, "bf16")
    n = 37 * 131
    buf = torch.full((n + 128,), 7.0, device="cuda", dtype=torch.bfloat16)
    fb = torch.full((2 * n + 192,), 7.0, device="cuda")
    y, g, u = buf[64:64 + n].view(37, 131), fb[64:64 + n].view(37, 131), fb[128 + n:128 + 2 * n].view(37, 131)
    B.fo_gated_forward(x, gate, up, y, g, u)
    assert torch.equal(y, nn.gated_linear(x, gate, up))
    for s in (buf[:64], buf[64 + n:], fb[:64], fb[64 + n:128 + n], fb[128 + 2 * n:]):
        assert (s == 7).all()
    out = torch.full((37 * 72 + 2 * 131 * 72 + 256,), 7.0, device="cuda", dtype=torch.bfloat16)
    m = 131 * 72
    dx, dgate, dup = out[64:64 + 37 * 72].view(37, 72), out[128 + 37 * 72:128 + 37 * 72 + m].view(131, 72), \
        out[192 + 37 * 72 + m:192 + 37 * 72 + 2 * m].view(131, 72)
    B.fo_gated_backward(x, gate, up, g, u, dy, dx, dgate, dup)
    for a, b in zip((dx, dgate, dup), run(x, gate, up, dy)[1:]):
        assert torch.equal(a, b)
    for s in (out[:64], out[64 + 37 * 72:128 + 37 * 72], out[128 + 37 * 72 + m:192 + 37 * 72 + m], out[192 + 37 * 72 + 2 * m:]):
        assert (s == 7).all()


def test_refusals():
    x, gate, up, dy = make(13, 8, 64, 30, "bf16")
    for args, match in (((x, gate.half(), up), "agree"), ((x, gate, up[:20]), "agree"), ((x, gate[:, :32], up), "shape"),
                        ((x, gate[:0], up[:0]), "shape"), ((x.double(), gate.double(), up.double()), "not supported"),
                        ((x, gate.cpu(), up), "GPU"), ((x, gate, up, "relu"), "activation")):
        with pytest.raises(ValueError, match=match):
            nn.gated_linear(*args)
    a = x.detach().requires_grad_(True)
    g = torch.autograd.grad(nn.gated_linear(a, gate, up), a, dy, create_graph=True)[0]
    with pytest.raises(RuntimeError, match="second derivatives"):
        g.float().sum().backward()
    with pytest.raises(NotImplementedError, match="forward-mode"), torch.autograd.forward_ad.dual_level():
        nn.gated_linear(torch.autograd.forward_ad.make_dual(x, x), gate, up)

"""Linear cross entropy, the gated block, gradient clipping, the norms and the optimizer in
one training step; captured steps; two streams."""

import pytest
import torch

from precision_optimizer_state_amd import FlashAdamW, clip_grad_norm_, clip_grads, grad_norm, nn
from step_helpers import TYPES, Gated, Loss, check, generator, normal

pytestmark = pytest.mark.gpu


class Block(torch.nn.Module):
    """Embedding, one gated block with its norm, and a head."""

    def __init__(self, vocab, width, features, seed=0):
        super().__init__()
        gen = generator(seed)
        p = torch.nn.Parameter
        self.embed = p(normal(gen, vocab, width))
        self.norm = nn.FlashRMSNorm(width, device="cuda")
        self.gate, self.up = (p(normal(gen, features, width, scale=width ** -0.5)) for _ in range(2))
        self.down = p(normal(gen, width, features, scale=features ** -0.5))
        self.head = p(normal(gen, vocab, width, scale=width ** -0.5))

    def forward(self, tokens, target):
        x = self.embed[tokens]
        y = nn.gated_linear(self.norm(x), self.gate, self.up)
        x = x + torch.matmul(y, self.down.t())
        return nn.linear_cross_entropy(x, self.head, target)

    def plain(self, tokens, target, params):
        """The same step in float64 from given parameters."""
        x = params["embed"][tokens]
        h = x / torch.sqrt(x.square().mean(-1, keepdim=True) + 1e-6) * params["norm.weight"]
        g, u = h @ params["gate"].t(), h @ params["up"].t()
        x = x + (g * torch.sigmoid(g) * u) @ params["down"].t()
        z = x @ params["head"].t()
        return torch.nn.functional.cross_entropy(z.flatten(0, -2), target.flatten(), ignore_index=-100)


def batch(gen, vocab, shape=(4, 33)):
    tokens = torch.randint(vocab, shape, generator=gen, device="cuda")
    target = torch.roll(tokens, -1, 1)
    target[:, -1] = -100
    return tokens, target


def test_a_training_step_against_float64():
    """Gradients of a whole step in float32 against float64, clipped, and fed to the
    optimizer, which steps.  Errors pass through four layers: 1e-4 of each gradient's
    largest element is some hundred float32 roundings of terms of that size."""
    model = Block(300, 64, 96)
    gen = generator(1)
    tokens, target = batch(gen, 300)
    loss = model(tokens, target)
    loss.backward()
    params = {k: v.detach().double().requires_grad_(True) for k, v in model.named_parameters()}
    want = model.plain(tokens, target, params)
    want.backward()
    assert abs(float(loss) - float(want)) < 1e-5 * float(want)
    for k, v in model.named_parameters():
        check(k, v.grad, params[k].grad, 1e-4 * params[k].grad.abs().max())
    total = torch.sqrt(sum(p.grad.square().sum() for p in params.values()))
    norm = clip_grad_norm_(model.parameters(), 0.1)
    check("norm", norm, total, 1e-4 * total)
    check("clipped", grad_norm([p.grad for p in model.parameters()]), torch.tensor(0.1, device="cuda"), 1e-5)


@pytest.mark.parametrize("wfmt", ["bf16", "fp16"])
def test_training_with_the_optimizer(wfmt):
    """16-bit parameters, gradients summed over micro-batches in float32, clipped into the
    parameters' gradients, stepped.  Each step's gradients are those of the same
    parameters in float64 within what 16-bit activations, gradients and weights allow;
    the parameters move by what the optimizer makes of the clipped gradients."""
    model = Block(200, 64, 128, seed=2)
    opt = FlashAdamW(model.parameters(), lr=1e-3, wfmt=wfmt)
    gen = generator(3)
    for _ in range(3):
        sums = [torch.zeros_like(p, dtype=torch.float32) for p in model.parameters()]
        exact = {k: v.detach().double().requires_grad_(True) for k, v in model.named_parameters()}
        for _ in range(2):
            tokens, target = batch(gen, 200)
            opt.zero_grad()
            model(tokens, target).backward()
            for s, p in zip(sums, model.parameters()):
                s.add_(p.grad)
            model.plain(tokens, target, exact).backward()
        for (k, p), s in zip(model.named_parameters(), sums):
            off = float((s.double() - exact[k].grad).norm() / exact[k].grad.norm())
            assert off < 12 * torch.finfo(p.dtype).eps, (k, off)
        _, norm = clip_grads(sums, 0.2, out=[p.grad for p in model.parameters()])
        c = min(1.0, 0.2 / (float(norm) + 1e-6))
        for s, p in zip(sums, model.parameters()):
            assert p.grad.dtype == TYPES[wfmt]
            check("clipped", p.grad, s.double() * c, torch.finfo(p.dtype).eps / 2 * (s.double() * c).abs() * 1.01 + 2.0 ** -25)
        before = [p.detach().clone() for p in model.parameters()]
        opt.step()
        assert all(torch.isfinite(p).all() for p in model.parameters())
        assert any(not torch.equal(a, p) for a, p in zip(before, model.parameters()))


def test_checkpointed_block():
    model = Block(100, 64, 64, seed=4)
    gen = generator(5)
    x = normal(gen, 50, 64).requires_grad_(True)

    def block(t):
        return nn.gated_linear(model.norm(t), model.gate, model.up)

    dy = normal(gen, 50, 64)
    want = torch.autograd.grad(block(x), (x, model.gate), dy)
    for reentrant in (True, False):
        y = torch.utils.checkpoint.checkpoint(block, x, use_reentrant=reentrant)
        x.grad = model.gate.grad = None
        y.backward(dy)
        assert torch.equal(x.grad, want[0]) and torch.equal(model.gate.grad, want[1])


def test_captured_step():
    """Forward, backward and clipping in one graph; every replay on new inputs equals the
    eager step, with eager work of the same operators between replays."""
    gen = generator(6)
    dt = torch.bfloat16
    x0, gate0, up0, head0 = (normal(gen, *s, scale=k, dtype=dt) for s, k in
                             (((70, 64), 1), ((96, 64), 0.1), ((96, 64), 0.1), ((500, 96), 0.1)))
    target = torch.randint(500, (70,), generator=gen, device="cuda")

    def step(x, leaves, target, grads):
        y = nn.gated_linear(x, *leaves[:2])
        loss = nn.linear_cross_entropy(y, leaves[2], target)
        for g, d in zip(grads, torch.autograd.grad(loss, leaves)):
            g.copy_(d)
        norm = clip_grads(grads, 0.05)[1]
        return loss.detach(), norm

    def fresh():
        leaves = [a.clone().requires_grad_(True) for a in (gate0, up0, head0)]
        return leaves, [torch.empty_like(a) for a in leaves]

    x, (leaves, grads), t = x0.clone(), fresh(), target.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(x, leaves, t, grads)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    leaves, grads = fresh()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(x, leaves, t, grads)
    for r in range(4):
        new = normal(gen, 70, 64, dtype=dt)
        x.copy_(new)
        t.copy_(torch.roll(target, r))
        t[:r] = -100
        graph.replay()
        eager, eg = fresh()
        want = step(new, eager, t.clone(), eg)
        torch.cuda.synchronize()
        for a, b in zip((*out, *grads), (*want, *eg)):
            assert torch.equal(a, b), r


def test_two_graphs_and_an_eager_call_between():
    gen = generator(7)
    shapes = [(40, 64, 300), (300, 128, 1000)]
    made = []
    for rows, cols, vocab in shapes:
        x, w = normal(gen, rows, cols, dtype=torch.bfloat16), normal(gen, vocab, cols, scale=0.1, dtype=torch.bfloat16)
        t = torch.randint(vocab, (rows,), generator=gen, device="cuda")
        made.append((x, w, t))

    def call(x, w, t):
        x, w = x.detach().requires_grad_(True), w.detach().requires_grad_(True)
        loss = nn.linear_cross_entropy(x, w, t)
        return (loss.detach(),) + torch.autograd.grad(loss, (x, w))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        for m in made:
            call(*m)
    torch.cuda.current_stream().wait_stream(side)
    graphs, outs = [], []
    for m in made:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(call(*m))
        graphs.append(g)
    want = [call(*m) for m in made]
    for _ in range(3):
        for g in graphs:
            g.replay()
        again = call(*made[0])
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert all(torch.equal(a, b) for a, b in zip(o, w))
        assert all(torch.equal(a, b) for a, b in zip(again, want[0]))


def test_capture_refuses_leaves_of_a_living_eager_graph():
    w = normal(generator(8), 100, 64).requires_grad_(True)
    x = normal(generator(9), 10, 64)
    t = torch.zeros(10, dtype=torch.int64, device="cuda")
    loss = nn.linear_cross_entropy(x, w, t)
    gated = nn.gated_linear(x, w, w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        with pytest.raises(RuntimeError, match="captured"):
            nn.linear_cross_entropy(x, w, t)
        with pytest.raises(RuntimeError, match="captured"):
            nn.gated_linear(x, w, w)
        kept = nn.linear_cross_entropy(x, w.detach(), t)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(kept, loss.detach()) and gated.shape == (10, 100)


def test_two_streams_at_once():
    gen = generator(10)
    sets = []
    for i in range(2):
        x, w = normal(gen, 200, 128, dtype=torch.bfloat16), normal(gen, 3000, 128, scale=0.1, dtype=torch.bfloat16)
        sets.append((x, w, torch.randint(3000, (200,), generator=gen, device="cuda"), normal(gen, 200, 3000, dtype=torch.bfloat16)))

    def call(x, w, t, dy):
        a, b = x.detach().requires_grad_(True), w.detach().requires_grad_(True)
        out = torch.autograd.grad(nn.linear_cross_entropy(a, b, t), (a, b))
        y = nn.gated_linear(a, b, b)
        out += torch.autograd.grad(y, (a, b), dy)
        return out + (clip_grads([g.clone() for g in out], 0.01)[1],)

    want = [call(*s) for s in sets]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            s.wait_stream(torch.cuda.default_stream())
            with torch.cuda.stream(s):
                got[i].append(call(*sets[i]))
    torch.cuda.synchronize()
    for i in range(2):
        for g in got[i]:
            assert all(torch.equal(a, b) for a, b in zip(g, want[i]))


def test_tracers_are_refused():
    from torch.fx.experimental.proxy_tensor import make_fx
    x, w = normal(generator(12), 5, 64), normal(generator(13), 70, 64)
    t = torch.zeros(5, dtype=torch.int64, device="cuda")
    for f in (lambda a: nn.linear_cross_entropy(a, w, t), lambda a: nn.gated_linear(a, w, w)):
        for pre in (False, True):
            with pytest.raises(NotImplementedError, match="traced"):
                make_fx(f, pre_dispatch=pre)(x)
        with pytest.raises(NotImplementedError, match="traced"):
            torch.jit.trace(f, x, check_trace=False)
        a = x.clone().requires_grad_(True)
        y = f(a)
        with pytest.raises(NotImplementedError, match="traced"):
            make_fx(lambda dy: torch.autograd.grad(y, a, dy, retain_graph=True)[0])(torch.ones_like(y))


def test_negated_views():
    gen = generator(14)
    x, w, u = normal(gen, 20, 64), normal(gen, 70, 64), normal(gen, 70, 64)
    t = torch.randint(70, (20,), generator=gen, device="cuda")
    neg = [torch._neg_view(-a) for a in (x, w, u)]
    assert torch.equal(nn.linear_cross_entropy(neg[0], neg[1], t), nn.linear_cross_entropy(x, w, t))
    assert torch.equal(nn.linear_cross_entropy(x, w, torch._neg_view(-t)), nn.linear_cross_entropy(x, w, t))
    assert torch.equal(nn.gated_linear(*neg), nn.gated_linear(x, w, u))
    a = x.clone().requires_grad_(True)
    dy = normal(gen, 20, 70)
    y = nn.gated_linear(a, w, u)
    plain = torch.autograd.grad(y, a, dy, retain_graph=True)[0]
    assert torch.equal(torch.autograd.grad(y, a, torch._neg_view(-dy))[0], plain)


def test_inference_mode():
    gen = generator(11)
    x, w = normal(gen, 5, 64), normal(gen, 70, 64)
    t = torch.zeros(5, dtype=torch.int64, device="cuda")
    with torch.inference_mode():
        a, y = nn.linear_cross_entropy(x, w, t), nn.gated_linear(x, w, w)
        g = torch.ones(5, device="cuda")
        clip_grads([g], 1.0)
    assert torch.equal(a, nn.linear_cross_entropy(x, w, t)) and torch.equal(y, nn.gated_linear(x, w, w))
    ref = Loss(x, w, t)
    check("loss", a, ref.loss, ref.d_loss)
    check("y", y, Gated(x, w, w).y, Gated(x, w, w).d_y)

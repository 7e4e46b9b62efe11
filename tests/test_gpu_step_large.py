"""Clipping, linear cross entropy and the gated block where offsets pass 32 bits, on the
GPU: a few rows at both ends against float64 (bounds derived in step_helpers), the others
without a part in what is compared."""

import math

import pytest
import torch

from precision_optimizer_state_amd import clip_grads, grad_norm, nn
from step_helpers import U, Gated, Loss, check, generator, half_step

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def give_memory_back():
    yield
    torch.cuda.empty_cache()


def bf16(gen, *shape, scale=1.0):
    return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.bfloat16) * scale


def test_a_tensor_past_2_32_elements():
    n, at = (1 << 32) + 12345, torch.tensor([0, (1 << 32) - 1, 1 << 32, -2, -1], device="cuda")
    t = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    t[1 << 32], t[-1] = 5, 3
    few = t[at].double()
    want = math.sqrt(n - 2 + 25 + 9)
    check("norm", grad_norm([t]), torch.tensor(want, device="cuda"), 2 * U * want)
    assert grad_norm([t], math.inf) == 5 and grad_norm([t], 1) == float(torch.tensor(n - 2 + 5 + 3, dtype=torch.float32))
    scaled = few / (want + 1e-6)
    bound = half_step(torch.bfloat16, scaled) * (1 + 2.0 ** -7) + 4 * U * scaled
    out = torch.zeros_like(t)
    clip_grads([t], 1.0, out=[out])
    check("into another", out[at], scaled, bound)
    assert torch.equal(t[at].double(), few) and bool((out[(1 << 32) + 1:-1] == out[0]).all())
    clip_grads([t], 1.0)
    check("in place", t[at], scaled, bound)
    assert torch.equal(t, out)


def test_outputs_of_the_gated_block_past_2_32_elements():
    gen, rows, features = generator(71), (1 << 18) + 37, 16384 + 8
    x, gate, up = bf16(gen, rows, 64), bf16(gen, features, 64, scale=0.1), bf16(gen, features, 64, scale=0.1)
    few = torch.tensor([0, 1, rows // 2, rows - 38, rows - 2, rows - 1], device="cuda")
    leaves = [a.requires_grad_(True) for a in (x, gate, up)]
    y = nn.gated_linear(*leaves)
    assert y.numel() > 1 << 32
    dy = torch.zeros_like(y)
    dy[few] = bf16(gen, len(few), features)
    dx, dgate, dup = torch.autograd.grad(y, leaves, dy)
    # (the sums over rows have zeros besides: no error of their own)
    want = Gated(x[few], gate, up, "silu", dy[few])
    check("y", y[few], want.y, want.d_y)
    check("dx", dx[few], want.dx, want.d_dx)
    check("dgate", dgate, want.dgate, want.d_dgate)
    check("dup", dup, want.dup, want.d_dup)
    dx[few] = 0
    assert not dx.any()


def test_tokens_past_2_32_elements():
    gen, rows, cols, vocab = generator(72), (1 << 20) + 5, 4160, 40
    x, w = bf16(gen, rows, cols), bf16(gen, vocab, cols, scale=0.05)
    t = torch.randint(vocab, (rows,), generator=gen, device="cuda")
    few = torch.cat([torch.arange(5, device="cuda"), rows - 1 - torch.arange(40, device="cuda")])
    masked = torch.full_like(t, -100)
    masked[few] = t[few]
    x.requires_grad_(True), w.requires_grad_(True)
    loss = nn.linear_cross_entropy(x, w, masked, reduction="none")
    dloss = torch.ones_like(loss)
    dx, dw = torch.autograd.grad(loss, (x, w), dloss)
    want = Loss(x[few], w, t[few], "none", dloss=dloss[few])
    check("loss", loss[few], want.loss, want.d_loss)
    check("dx", dx[few], want.dx, want.d_dx)
    check("dw", dw, want.dw, want.d_dw)
    dx[few] = 0
    assert not dx.any() and loss.count_nonzero() == len(few)


def test_a_vocabulary_past_2_32_elements():
    gen, cols, vocab = generator(73), 1032, (1 << 22) + 77
    x, w = bf16(gen, 3, cols), bf16(gen, vocab, cols, scale=0.05)
    t = torch.tensor([0, vocab - 1, vocab - 70], device="cuda")
    x.requires_grad_(True), w.requires_grad_(True)
    loss = nn.linear_cross_entropy(x, w, t, reduction="none")
    dx, dw = torch.autograd.grad(loss, (x, w), torch.ones_like(loss))
    want = Loss(x, w, t, "none", dloss=torch.ones_like(loss))
    check("loss", loss, want.loss, want.d_loss)
    check("dx", dx, want.dx, want.d_dx)
    check("dw", dw, want.dw, want.d_dw)

"""nn.linear_cross_entropy of logits whose log-sum-exp does not fit one float32, against
the definition in float64.

The logits of these tests are exact: every sum has at most two terms besides zeros, and
each of those is representable.  What is left is the softmax's own arithmetic.  With U =
2^-24 and D the distance of a logit from its token's largest: a term e^-D of the sum has
an exponent off by 2 U (1.45 D + 4) (the fused operation, the constant, the hardware's
exponential); D e^-D is at most 0.4, and a sum of V places adds (V / 4096 + 200) U;
logarithm and joining add 4 U (1 + ln V).  Together E, whatever the logits' size.  A
probability exp((z - lse) - rest) adds 2 U (1.45 D + 4) again.  A loss, a sum of a
difference of logits and ln of that sum, has E and three roundings of its own value."""

import math

import pytest
import torch

from precision_optimizer_state_amd import binding as B
from precision_optimizer_state_amd import nn
from step_helpers import TYPES, U, check, generator, half_step, normal, product_bound
from test_gpu_loss import make, run

pytestmark = pytest.mark.gpu


def exact(x, w, t, dloss):
    """loss, dx, dw in float64 and their bounds, of no reduction."""
    dtype, V = x.dtype, w.shape[0]
    x, w = x.double(), w.double()
    z = x @ w.t()
    low = z - z.max(1, keepdim=True).values
    lse = torch.logsumexp(low, 1)
    loss = lse - low.gather(1, t[:, None])[:, 0]
    E = (2 * (1.45 * 0.4 + 4) + V / 4096 + 200 + 4 * (1 + math.log(V))) * U
    d_loss = E + 8 * U * loss.abs()
    p = torch.softmax(z, 1)
    y = torch.zeros_like(p).scatter_(1, t[:, None], 1.0)
    f = dloss.double()
    top = f.abs().max()
    P = (p - y) * (f / top)[:, None]
    d_p = p * (E + 2 * U * (1.45 * -low + 4)) + 4 * U * (p + y)
    half = torch.finfo(dtype).eps / 2
    if dtype != torch.float32:
        d_p = d_p * (1 + half) + half * P.abs()
    if dtype == torch.float16:
        d_p = d_p + 2.0 ** -40
    out = [loss, d_loss]
    for a, da, b in ((P, d_p, w), (P.t(), d_p.t(), x)):
        got = a @ b * top
        inner = (da @ b.abs() + 2 * (a.shape[1] + 40) * U * (a.abs() @ b.abs())) * top * (1 + half) + 8 * U * got.abs()
        out += [got, inner + half_step(dtype, got) * (1 + 2.0 ** -7)]
    return out


def compare(x, w, t, dloss):
    loss, dx, dw, _ = run(x, w, t, "none", dloss=dloss)
    want = exact(x, w, t, dloss)
    check("loss", loss, want[0], want[1])
    check("dx", dx, want[2], want[3])
    check("dw", dw, want[4], want[5])
    return loss, dx, dw


def sizes(gen, n, low, high, dtype, unit):
    """`n` numbers spread over [low, high] by their logarithm, whole multiples of `unit`
    that the type holds."""
    r = torch.rand(n, generator=gen, device="cuda", dtype=torch.float64)
    s = torch.exp(math.log(low) + r * math.log(high / low))
    return (torch.round(s / unit) * unit).to(TYPES[dtype])


@pytest.mark.parametrize("rows", [17, 200, 700])
@pytest.mark.parametrize("dtype", list(TYPES))
def test_softmax_of_neighbours_at_any_height(dtype, rows):
    """Logits s + d with s from 2^8 to 2^22, the same for all places of a token but those far
    below, and d of a few halves: the softmax is that of d, on both sides of 2^20."""
    gen = generator(40)
    V = 300
    x = torch.zeros(rows, 64, device="cuda", dtype=TYPES[dtype])
    w = torch.zeros(V, 64, device="cuda", dtype=TYPES[dtype])
    # 64 times the rows' first column is whole, of 8 (bf16), 11 (fp16) or 22 bits (float32)
    x[:, 0] = sizes(gen, rows, 2.0 ** 2, 2.0 ** 15.9, dtype, 2.0 ** -6)
    x[:, 1] = 1.0
    w[:, 0] = 32.0                                      # half of s below
    w[::3, 0] = 64.0
    w[:, 1] = -0.5 * torch.randint(24, (V,), generator=gen, device="cuda").to(w.dtype)
    t = 3 * torch.randint(V // 3, (rows,), generator=gen, device="cuda")
    t[0] = 4                                            # a target half of s below
    f = torch.ones(rows, device="cuda")
    if dtype == "fp16":
        f *= 2.0 ** -11                                 # (sums of 700 rows of up to 61000 would not fit)
    loss, _, _ = compare(x, w, t, f)
    compare(x, w, t, f * (0.5 + torch.rand(rows, generator=gen, device="cuda")))
    # the height has no part in the result: the same softmax without it, both off by less
    # than E + 8 U loss, 22e-6
    x0, w0 = x.clone(), w.clone()
    x0[:, 0] = 0.0
    w0[w[:, 0] == 32.0, 1] = -200.0
    flat = nn.linear_cross_entropy(x0, w0, t, reduction="none")
    assert (flat[1:] - loss[1:]).abs().max() <= 44e-6


@pytest.mark.parametrize("places", [(7,), (7, 205)])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_one_place_or_two_that_dominate(dtype, places):
    """Logits from 2^17 to 2^100, of any bits: one place has all of the probability, or two
    have half each."""
    gen = generator(41)
    x = torch.zeros(500, 64, device="cuda", dtype=TYPES[dtype])
    w = torch.zeros(300, 64, device="cuda", dtype=TYPES[dtype])
    r = torch.rand(500, generator=gen, device="cuda", dtype=torch.float64)
    x[:, 0] = torch.exp2(17 + r * torch.where(torch.arange(500, device="cuda") < 400, 15, 83)).to(x.dtype)
    w[:, 0] = -torch.exp2(-torch.randint(6, (300,), generator=gen, device="cuda").float()).to(w.dtype)
    w[list(places), 0] = 1.0
    t = torch.full((500,), 7, device="cuda")
    one = torch.ones(500, device="cuda")
    loss, _, _ = compare(x, w, t, one)
    assert (loss - math.log(len(places))).abs().max() <= 2 ** -16
    t[::5] = places[-1] if len(places) == 2 else 3
    compare(x, w, t, one)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_logits_that_depend_on_their_order_of_summation(dtype):
    """Sums of many large terms differ by whole numbers between two ways of adding them.
    Gradients of logits stay in [-1, 1] all the same."""
    gen = generator(42)
    for rows in (20, 100, 400):
        x = (1e5 * torch.randn(rows, 256, generator=gen, device="cuda")).to(TYPES[dtype])
        w = (1e3 * torch.randn(160, 256, generator=gen, device="cuda")).to(TYPES[dtype])
        w[:, 255] = 0.0
        w[11, 255] = 1.0                                # dx there is the gradient of place 11's logit
        x[:, 255] = 0.0
        t = torch.randint(160, (rows,), generator=gen, device="cuda")
        x[1], w[12, :255] = x[0], w[11, :255]           # a tie of two places
        _, dx, dw, _ = run(x, w, t, "none")
        assert torch.isfinite(dx).all() and torch.isfinite(dw).all()
        assert dx[:, 255].abs().max() <= 1.0
        total = x.double().abs().sum(0)
        assert (dw.double().abs() <= total * (1 + 2 ** -7)).all()


def test_confident_tokens():
    """A token whose target has all but e of the probability, e from 1e-2 to 1e-5, at logits
    of 500 to 1000: the gradient of its logit is -e, off by roundings of numbers next to 1, U
    or an exponential's 2 U each: the largest term, at most 14 additions, 3 of bringing the
    sum to its reference, 5 of the logarithm, the rest and the probability."""
    gen = generator(43)
    rows, V = 64, 40
    x = torch.zeros(rows, 64, device="cuda")
    w = torch.zeros(V, 64, device="cuda")
    x[:, 0] = 500 + 500 * torch.rand(rows, generator=gen, device="cuda")
    w[5, 0], w[5, 2] = 1.0, 1.0                         # (x[:, 2] is 0: dx there is the target's gradient)
    gap = 8 + 7 * torch.rand(rows, generator=gen, device="cuda")
    x[:, 1] = x[:, 0] - gap
    w[:, 1] = torch.where(torch.arange(V, device="cuda") == 5, 0.0, 1.0)
    t = torch.full((rows,), 5, device="cuda")
    loss, dx, _, _ = run(x, w, t, "none")
    z = x.double() @ w.double().t()
    e = -torch.expm1(z[:, 5] - torch.logsumexp(z, 1))
    far = (z - z.max(1, keepdim=True).values).abs()[:, 0]
    room = 24 * U + 2 * e * (2 * U * (1.45 * far + 4) + 40 * U)
    check("dx", dx[:, 2], -e, room)
    check("loss", loss, -torch.log1p(-e), room)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("rows, cols, vocab", [(1, 64, 300), (33, 65, 1000), (300, 128, 4500)])
def test_the_library_with_and_without_the_rest(rows, cols, vocab, dtype):
    """fo_loss_backward finds what lse's rounding left by itself: the same gradients, to the
    bit, as with the array that the forward call can give."""
    x, w, t = make(44, rows, cols, vocab, dtype, ignored=0.2 if rows > 1 else 0.0)
    lo, lse, rest, cnt, one = (torch.full((n,), 7.0, device="cuda") for n in (1, rows, rows, 1, 1))
    B.fo_loss_forward(x, w, t, lo, lse, cnt, rest_out=rest)
    # half a step of lse, and together log sum exp to less than that
    z = x.double() @ w.double().t()
    want, counted = torch.logsumexp(z, 1), t != -100
    assert (rest.abs() <= U * lse.abs())[counted].all()
    check("lse + rest", (lse.double() + rest)[counted], want[counted],
          (product_bound(x.double(), w.double()).max(1).values + (2 * (1.45 * z.abs().max(1).values + 4) + 250) * U)[counted])
    grads = [[torch.empty_like(x), torch.empty_like(w)] for _ in range(3)]
    B.fo_loss_backward(x, w, t, lse, one, cnt, *grads[0], rest=rest)
    B.fo_loss_backward(x, w, t, lse, one, cnt, *grads[1])
    a, b = x.detach().clone().requires_grad_(True), w.detach().clone().requires_grad_(True)
    loss = nn.linear_cross_entropy(a, b, t)
    loss.backward(one[0])
    assert torch.equal(loss, lo[0])
    for g in (grads[1], [a.grad, b.grad]):
        assert torch.equal(g[0], grads[0][0]) and torch.equal(g[1], grads[0][1])


@pytest.mark.parametrize("cols", [32, 64])
def test_the_library_finds_the_rest_over_several_pieces(cols):
    """... of weights that are copied (32 columns of bf16) and read as they lie."""
    x, w, t = make(45, 8192, cols, 40001, "bf16", ignored=0.1)
    n = 8192
    lo, lse, rest, cnt, one = (torch.full((k + 2,), 7.0, device="cuda") for k in (1, n, n, 1, 1))
    B.fo_loss_forward(x, w, t, lo[1:2], lse[1:-1], cnt[1:2], rest_out=rest[1:-1])
    plain = torch.full_like(lse, 7.0)
    B.fo_loss_forward(x, w, t, lo[1:2], plain[1:-1], cnt[1:2])
    assert torch.equal(lse, plain) and (rest[::n + 1] == 7).all()
    grads = [[torch.empty_like(x), torch.empty_like(w)] for _ in range(2)]
    B.fo_loss_backward(x, w, t, lse[1:-1], one[1:2], cnt[1:2], *grads[0], rest=rest[1:-1])
    B.fo_loss_backward(x, w, t, lse[1:-1], one[1:2], cnt[1:2], *grads[1])
    assert torch.equal(grads[0][0], grads[1][0]) and torch.equal(grads[0][1], grads[1][1])


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("rows", [20, 3000])
def test_losses_are_not_negative(rows, dtype):
    """log of a sum whose largest term is 1, and the target's distance from the largest logit:
    0 at least, and 0 where nothing else counts."""
    gen = generator(46)
    x = torch.zeros(rows, 64, device="cuda", dtype=TYPES[dtype])
    w = torch.zeros(300, 64, device="cuda", dtype=TYPES[dtype])
    x[:, 0] = (1 + 999 * torch.rand(rows, generator=gen, device="cuda")).to(x.dtype)
    w[5, 0] = 1.0
    t = torch.full((rows,), 5, device="cuda")
    loss = nn.linear_cross_entropy(x, w, t, reduction="none")
    assert (loss >= 0).all()
    assert (loss[x[:, 0] > 128] <= 24 * U).all()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("smoothing", [0.0, 0.25, 1.0])
@pytest.mark.parametrize("rows", [1, 19, 324])
def test_a_vocabulary_of_one_place(rows, smoothing, dtype):
    """The softmax of one logit is 1, whatever the logit: no loss and no gradients, exactly."""
    x, w, t = make(47, rows, 80, 1, dtype)
    loss, dx, dw, _ = run(x, w, t, "none", smoothing)
    assert not loss.any() and not dx.any() and not dw.any()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("rows, vocab", [(1, 50), (20, 13), (32, 2000), (33, 300), (100, 5000), (400, 700), (1100, 5001)])
def test_probabilities_add_up_to_one(rows, vocab, dtype):
    """The backward pass makes the forward pass's logits to the bit, so that the roundings of
    sums of many large terms cancel: a column of ones in the weight gives the sum of a
    token's gradients of logits, which is 0.  It is off by E and 2 U (1.45 D + 4) for the
    probabilities (D e^-D is at most 0.4), their roundings to the type, and the product's
    own, of at most 2 in absolute values."""
    gen = generator(48)
    cols, E = 513, (2 * (2 * (1.45 * 0.4 + 4)) + vocab / 4096 + 200 + 4 * (1 + math.log(vocab)))
    x = normal(gen, rows, cols, dtype=TYPES[dtype], scale=60.0)
    w = normal(gen, vocab, cols, dtype=TYPES[dtype])
    x[:, 512], w[:, 512] = 0.0, 1.0
    t = torch.randint(vocab, (rows,), generator=gen, device="cuda")
    _, dx, _, _ = run(x, w, t, "none")
    half = 0.0 if dtype == "f32" else torch.finfo(TYPES[dtype]).eps / 2
    # (float32 sums of V terms of at most 2 in all, in matrix instructions: 2 (V + 40) U of that, of which
    # the terms that are not 0 are a few)
    room = (E + 2 * 64 * 2) * U + 2 * half + 2.0 ** -24
    assert dx[:, 512].abs().max() <= room

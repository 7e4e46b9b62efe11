"""nn.linear_cross_entropy on the GPU against its definition in float64 (bounds derived in
step_helpers), at the sizes where tiles, steps, slices and pieces end, and under masks."""

import pytest
import torch

from precision_optimizer_state_amd import binding as B
from precision_optimizer_state_amd import nn
from step_helpers import TYPES, Loss, check, generator, normal

pytestmark = pytest.mark.gpu


def make(seed, rows, cols, vocab, dtype, ignored=0.0, scale=None, pad=0, lead=0, peaked=True):
    gen = generator(seed)
    x = normal(gen, rows, cols, dtype=TYPES[dtype], pad=pad, lead=lead)
    w = normal(gen, vocab, cols, scale=(scale or cols ** -0.5), dtype=TYPES[dtype])
    t = torch.randint(vocab, (rows,), generator=gen, device="cuda")
    t = torch.where(torch.rand(rows, generator=gen, device="cuda") < ignored, -100, t)
    return x, w, t


def run(x, w, t, reduction="mean", smoothing=0.0, ignore=-100, dloss=None):
    x, w = x.detach().requires_grad_(True), w.detach().requires_grad_(True)
    loss = nn.linear_cross_entropy(x, w, t, ignore_index=ignore, reduction=reduction, label_smoothing=smoothing)
    if dloss is None:
        dloss = torch.ones_like(loss)
    dx, dw = torch.autograd.grad(loss, (x, w), dloss)
    return loss, dx, dw, dloss


def against(name, x, w, t, reduction="mean", smoothing=0.0, ignore=-100, dloss=None):
    loss, dx, dw, dloss = run(x, w, t, reduction, smoothing, ignore, dloss)
    want = Loss(x, w, t, reduction, smoothing, ignore, dloss)
    assert loss.dtype == torch.float32 and dx.dtype == x.dtype and dw.dtype == w.dtype
    check(name + " loss", loss, want.loss, want.d_loss)
    check(name + " dx", dx, want.dx.view(x.shape), want.d_dx.view(x.shape))
    check(name + " dw", dw, want.dw, want.d_dw)
    with torch.no_grad():
        again = nn.linear_cross_entropy(x, w, t, ignore_index=ignore, reduction=reduction, label_smoothing=smoothing)
    assert torch.equal(again, loss.detach())


# rows: narrow tiles end at 32; columns: a step is 64 elements (32 floats); vocabulary: tiles of 64, 128, 256
SIZES = [(1, 1, 1), (1, 64, 2), (2, 7, 3), (31, 64, 63), (32, 64, 64), (33, 65, 65), (64, 32, 127), (65, 96, 128), (63, 63, 129),
         (127, 128, 255), (128, 100, 256), (129, 192, 257), (1, 768, 5000), (17, 40, 1000), (255, 64, 513), (257, 33, 70), (1000, 72, 300)]


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("rows, cols, vocab", SIZES)
def test_sizes(rows, cols, vocab, dtype):
    against(f"{rows}x{cols}x{vocab}", *make(rows * 7 + cols + vocab, rows, cols, vocab, dtype))


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("rows, cols, vocab", [(4095, 64, 4100), (4097, 128, 4353), (300, 1024, 2000), (2048, 300, 700)])
def test_larger_tiles(rows, cols, vocab, dtype):
    """Wide and middle tiles, several of them, with ragged ends."""
    against("large", *make(3, rows, cols, vocab, dtype))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
def test_several_pieces_of_the_vocabulary(dtype):
    x, w, t = make(4, 8192, 32, 40001, dtype, ignored=0.1)
    a = B.Loss(x=x.data_ptr(), weight=w.data_ptr(), rows=8192, cols=32, vocab=40001, x_ld=32, weight_ld=32,
               dtype=B._dtype(x), reduction=1, dx=1 << 40)
    n = B.c_int64(0)
    B._check(B._load_step().fo_loss_backward_workspace(a, n))
    assert n.value < 8192 * 40001 * 2                  # fewer bytes than the logits' gradients have
    against("pieces", x, w, t)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("reduction", ["mean", "sum", "none"])
@pytest.mark.parametrize("smoothing", [0.0, 0.1, 1.0])
def test_reductions_and_smoothing(reduction, smoothing, dtype):
    x, w, t = make(5, 100, 64, 200, dtype, ignored=0.3)
    gen = generator(6)
    dloss = None
    if reduction == "none":
        dloss = torch.randn(100, generator=gen, device="cuda")
        dloss[3] = 0.0
    elif dtype == "fp16":
        dloss = torch.tensor(1024.0, device="cuda")
    against(reduction, x, w, t, reduction, smoothing, dloss=dloss)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("reduction", ["mean", "sum", "none"])
def test_no_token_counts(reduction, dtype):
    x, w, t = make(7, 40, 64, 100, dtype)
    t[:] = -100
    loss, dx, dw, _ = run(x, w, t, reduction)
    if reduction == "mean":
        assert loss.isnan()
    else:
        assert not loss.any()
    assert not dx.any() and not dw.any()


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("value", [float("nan"), float("inf"), -float("inf")])
def test_masked_tokens_may_hold_anything(value, dtype):
    x, w, t = make(8, 70, 96, 150, dtype, ignored=0.4)
    t[-1], t[0] = -100, 5                               # the last row is read for the padding's steps
    clean = x.clone()
    x[t == -100] = value
    got, want = run(x, w, t), run(clean, w, t)
    assert (t == -100).any()
    for a, b in zip(got[:3], want[:3]):
        assert torch.equal(a, b)
    assert not got[1][t == -100].any()


@pytest.mark.parametrize("ignore", [0, 7, -1, 10 ** 12, -2 ** 63])
def test_any_ignore_index(ignore):
    x, w, t = make(9, 64, 64, 90, "bf16")
    t[::3] = ignore
    against("ignore", x, w, t, ignore=ignore)


@pytest.mark.parametrize("bad", [-1, 90, 127, 2 ** 40, -2 ** 63, 2 ** 63 - 1])
def test_targets_out_of_range_give_nan(bad):
    x, w, t = make(10, 40, 64, 90, "bf16")
    t[7] = bad
    loss, dx, dw, _ = run(x, w, t, "none")
    assert loss[7].isnan() and loss.isnan().sum() == 1
    assert dx[7].isnan().all() and not dx[:7].isnan().any() and not dx[8:].isnan().any()
    assert dw.isnan().all()


@pytest.mark.parametrize("dtype", list(TYPES))
def test_logits_of_minus_infinity_and_of_the_types_lowest(dtype):
    """Whole tiles of places that are masked out by their logits."""
    x, w, t = make(11, 50, 64, 400, dtype)
    x[:, 0], w[:, 0] = 1.0, 0.0
    for low in (-float("inf"), torch.finfo(TYPES[dtype]).min):
        v = w.clone()
        v[:260, 0] = low
        v[390:, 0] = low
        t2 = 260 + t % 130
        loss = nn.linear_cross_entropy(x, v, t2, reduction="none")
        z = x.double() @ v.double().t()
        want = torch.logsumexp(z, 1) - z.gather(1, t2[:, None])[:, 0]
        ref = Loss(x, w[260:390], t2 - 260, "none")
        assert torch.isfinite(loss).all()
        check("masked places", loss, want, ref.d_loss + 1e-6)
    # nothing left: 0 / 0
    v = w.clone()
    v[:, 0] = -float("inf")
    assert nn.linear_cross_entropy(x, v, t, reduction="none").isnan().all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [1e5, 1e9, 1e30])
def test_logits_past_the_integers_of_float32(scale, dtype):
    """Logits whose product with log2(e) rounds by more than exponentials can take: the
    probabilities of an exact tie are halves, other places have none."""
    x = torch.full((40, 64), scale, device="cuda", dtype=TYPES[dtype])
    w = torch.zeros(300, 64, device="cuda", dtype=TYPES[dtype])
    w[:, 0] = torch.linspace(-0.5, 0.5, 300, device="cuda").to(w.dtype)
    w[7, 0], w[205, 0] = 1.0, 1.0
    t = torch.full((40,), 7, device="cuda")
    t[1] = 3
    loss, dx, dw, _ = run(x, w, t, "none")
    z = float(x[0, 0])
    ulp = z * 2.0 ** -23                                # the logits' own spacing, or less
    assert (loss[2:] >= -ulp).all() and (loss[2:] <= ulp + 1).all()
    assert abs(float(loss[1]) - 1.5 * z) < 0.02 * z + 2
    assert torch.isfinite(dx).all() and torch.isfinite(dw).all()
    # softmax is a half at places 7 and 205, within e to the spacing's power
    if ulp < 0.01:
        check("dx", dx[2:, 0], torch.zeros(38, device="cuda"), 1e-2)
        check("dw", dw[205], 40 * 0.5 * x[0].double(), 0.02 * 40 * 0.5 * x[0].double())


def test_an_infinite_gradient_of_one_token():
    x, w, t = make(21, 30, 64, 90, "bf16")
    dloss = torch.ones(30, device="cuda")
    want = run(x, w, t, "none", dloss=dloss)
    for bad in (float("inf"), float("nan")):
        dloss[4] = bad
        _, dx, dw, _ = run(x, w, t, "none", dloss=dloss)
        keep = torch.arange(30, device="cuda") != 4
        assert torch.equal(dx[keep], want[1][keep]) and not torch.isfinite(dx[4]).any()
        assert not torch.isfinite(dw).any()


def test_large_logits_neither_overflow_nor_vanish():
    x, w, t = make(12, 40, 64, 300, "f32")
    x = x * 3000.0                                      # logits of tens of thousands
    against("large logits", x, w, t, "none", dloss=torch.ones(40, device="cuda"))


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("pad, lead", [(1, 0), (0, 3), (8, 0), (8, 8), (61, 2)])
def test_slices(pad, lead, dtype):
    x, _, t = make(13, 90, 64, 130, dtype, pad=pad, lead=lead)
    _, w, _ = make(14, 1, 64, 130, dtype)
    wide = torch.zeros(130, 64 + pad + lead, device="cuda", dtype=TYPES[dtype])
    wide[:, lead:lead + 64] = w
    against("slices", x, wide[:, lead:lead + 64], t)


def test_layouts():
    gen = generator(15)
    x = normal(gen, 3, 5, 64, dtype=torch.bfloat16)
    w = normal(gen, 100, 64, scale=0.1, dtype=torch.bfloat16)
    t = torch.randint(100, (3, 5), generator=gen, device="cuda")
    against("three dimensions", x, w, t, "none", dloss=torch.ones(3, 5, device="cuda"))
    against("transposed", x.transpose(0, 1), w, t.t())
    against("one vector", x[0, 0], w, t[0, 0])
    against("columns", normal(gen, 64, 20, dtype=torch.bfloat16).t(), normal(gen, 64, 100, dtype=torch.bfloat16).t() * 0.1,
            t.reshape(-1).repeat(2)[:20])
    y = x[0, 0].expand(40, 64)                          # one row, 40 times
    against("expanded", y, w, t.reshape(-1).repeat(3)[:40])
    # an expanded gradient, as .sum() makes it, and a negated view
    a, b = x.detach().clone().requires_grad_(True), w.detach().clone().requires_grad_(True)
    nn.linear_cross_entropy(a, b, t, reduction="none").sum().backward()
    want = Loss(x, w, t, "sum", 0.0, -100, torch.ones((), device="cuda"))
    check("sum", a.grad, want.dx.view(x.shape), want.d_dx.view(x.shape))
    c = torch.complex(torch.zeros(6, 64), torch.randn(6, 64)).cuda().conj().imag
    assert c.is_neg()
    got = nn.linear_cross_entropy(c, w.float(), t.reshape(-1)[:6])
    assert torch.equal(got, nn.linear_cross_entropy(c.resolve_neg().clone(), w.float(), t.reshape(-1)[:6]))


def test_empty():
    w = torch.randn(10, 64, device="cuda", requires_grad=True)
    x = torch.randn(0, 64, device="cuda", requires_grad=True)
    t = torch.zeros(0, dtype=torch.int64, device="cuda")
    loss = nn.linear_cross_entropy(x, w, t, reduction="sum")
    loss.backward()
    assert loss == 0 and w.grad.shape == (10, 64) and not w.grad.any() and x.grad.shape == (0, 64)
    assert nn.linear_cross_entropy(x, w, t).isnan()
    assert nn.linear_cross_entropy(x, w, t, reduction="none").shape == (0,)
    assert nn.linear_cross_entropy(torch.randn(2, 0, 64, device="cuda"), w, t.view(2, 0), reduction="none").shape == (2, 0)


def test_only_the_gradients_that_are_needed():
    x, w, t = make(16, 50, 64, 80, "bf16")
    loss, dx, dw, _ = run(x, w, t)
    a = x.detach().requires_grad_(True)
    nn.linear_cross_entropy(a, w, t).backward()
    assert torch.equal(a.grad, dx)
    b = w.detach().requires_grad_(True)
    nn.linear_cross_entropy(x, b, t).backward()
    assert torch.equal(b.grad, dw)
    # one weight, two uses of it
    b = w.detach().requires_grad_(True)
    (nn.linear_cross_entropy(x, b, t) + nn.linear_cross_entropy(x, b, t)).backward()
    check("twice", b.grad, 2 * dw.double(), 2.0 ** -8 * 2 * dw.double().abs())


def test_gradients_against_differences():
    """A directional difference quotient of the operator's own losses: off the gradient's
    product with the direction by the losses' bounds over h, by the quotient's own
    distance from the derivative (taken in 64 bits) and by the gradients' bounds."""
    x, w, t = make(17, 60, 64, 100, "f32", ignored=0.2)
    gen = generator(18)
    dirs = normal(gen, 60, 64), normal(gen, 100, 64, scale=0.1)
    h = 2.0 ** -7
    _, dx, dw, one = run(x, w, t, "sum")
    ref = Loss(x, w, t, "sum", 0.0, -100, one)
    ends, exact = [], []
    for sign in (1, -1):
        args = x + sign * h * dirs[0], w + sign * h * dirs[1]
        ends.append(float(nn.linear_cross_entropy(*args, t, reduction="sum").double()))
        exact.append(Loss(*args, t, "sum"))
    slope = float((dx.double() * dirs[0]).sum() + (dw.double() * dirs[1]).sum())
    true = float((ref.dx * dirs[0]).sum() + (ref.dw * dirs[1]).sum())
    quotient = (ends[0] - ends[1]) / (2 * h)
    curve = abs(float(exact[0].loss - exact[1].loss) / (2 * h) - true)
    room = float(exact[0].d_loss + exact[1].d_loss) / (2 * h) + curve + \
        float((ref.d_dx * dirs[0].abs()).sum() + (ref.d_dw * dirs[1].abs()).sum())
    assert abs(quotient - slope) <= room
    # the comparison says something: less than a wrong gradient of this size is off by
    size = sum(float((g * g).sum()) for g in (ref.dx, ref.dw)) ** 0.5 * sum(float((d * d).sum()) for d in dirs) ** 0.5
    assert room < size / sum(d.numel() for d in dirs) ** 0.5


def test_nothing_behind_the_outputs_is_written():
    x, w, t = make(19, 37, 72, 131, "bf16")
    buf = torch.full((40 * 72 + 140 * 72 + 512,), 7.0, device="cuda", dtype=torch.bfloat16)
    dx, dw = buf[64:64 + 37 * 72].view(37, 72), buf[64 + 37 * 72 + 64:64 + 37 * 72 + 64 + 131 * 72].view(131, 72)
    lo, lse, cnt = (torch.full((n + 2,), 7.0, device="cuda") for n in (1, 37, 1))
    B.fo_loss_forward(x, w, t, lo[1:2], lse[1:38], cnt[1:2])
    B.fo_loss_backward(x, w, t, lse[1:38], torch.ones(1, device="cuda"), cnt[1:2], dx, dw)
    loss, gx, gw, _ = run(x, w, t)
    assert torch.equal(dx, gx) and torch.equal(dw, gw) and lo[1] == loss
    for s in (buf[:64], buf[64 + 37 * 72:128 + 37 * 72], buf[128 + 168 * 72:], lo[::2], lse[::38], cnt[::2]):
        assert (s == 7).all()


def test_refusals():
    x, w, t = make(20, 8, 64, 30, "bf16")
    for args, match in (((x, w.half(), t), "agree"), ((x, w[:, :32], t), "shape"), ((x, w, t[:4]), "shape"),
                        ((x, w, t.int()), "int64"), ((x, w[0], t), "shape"), ((x, w[:0], t), "shape"),
                        ((x.double(), w.double(), t), "not supported"), ((x, w.cpu(), t), "GPU"), ((x, w, t.cpu()), "GPU")):
        with pytest.raises(ValueError, match=match):
            nn.linear_cross_entropy(*args)
    a = x.detach().requires_grad_(True)
    g = torch.autograd.grad(nn.linear_cross_entropy(a, w, t), a, create_graph=True)[0]
    with pytest.raises(RuntimeError, match="second derivatives"):
        g.float().sum().backward()
    with pytest.raises(NotImplementedError, match="forward-mode"), torch.autograd.forward_ad.dual_level():
        nn.linear_cross_entropy(torch.autograd.forward_ad.make_dual(x, x), w, t)
    a = x.detach().requires_grad_(True)
    b = a * 1
    loss = nn.linear_cross_entropy(b, w, t)
    with torch.no_grad():
        b.add_(1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        loss.backward()

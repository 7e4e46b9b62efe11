"""grads.grad_norm, clip_grads, clip_grad_norm_ and the optimizers' clip_grad_norm_ on the
GPU against their definition in float64.

A norm is summed in float64 (n terms: relative n 2^-53, far below 2^-24), and rounded to
float32 once: off by 2^-24 of itself, twice that with the square root's and the sum's own
errors.  The factor c = min(1, max / (norm + 1e-6)) is rounded to float32 once, each
product once to float32 and once to the outputs' type."""

import math

import pytest
import torch

from precision_optimizer_state_amd import FlashAdam, FlashAdamW, FlashSGD, FoError
from precision_optimizer_state_amd import binding as B
from precision_optimizer_state_amd import clip_grad_norm_, clip_grads, grad_norm
from step_helpers import TYPES, U, check, generator, half_step

pytestmark = pytest.mark.gpu

# tiles are of 16384 elements, accesses of 8 and of 4; one launch's table has 196 or 140 tensors
LISTS = {"one": [1], "few": [7, 1, 16384, 16385, 16383, 3, 8, 100003], "empty ones": [0, 5, 0, 17, 0],
         "tables": [13] * 150 + [40000] + [5] * 400, "large": [3_000_001, 1 << 20]}


def make(sizes, dtype, seed=0, scale=1.0):
    gen = generator(seed)
    return [(scale * torch.randn(n, generator=gen, device="cuda")).to(TYPES[dtype]) for n in sizes]


def norm64(gs, p):
    flat = torch.cat([g.double().reshape(-1) for g in gs]) if gs else torch.zeros(0, device="cuda", dtype=torch.float64)
    if flat.numel() == 0:
        return torch.zeros((), device="cuda", dtype=torch.float64)
    return flat.abs().max() if p == math.inf else flat.abs().sum() if p == 1 else flat.square().sum().sqrt()


def factor64(norm, max_norm):
    return min(1.0, max_norm / (float(norm) + 1e-6))


def check_clipped(name, got, gs, c):
    for i, (o, g) in enumerate(zip(got, gs)):
        want = g.double() * c
        check(f"{name} {i}", o, want, half_step(o.dtype, want) * (1 + 2.0 ** -7) + 4 * U * want.abs())


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("p", [2.0, 1.0, math.inf])
@pytest.mark.parametrize("sizes", list(LISTS))
def test_norms(sizes, p, dtype):
    gs = make(LISTS[sizes], dtype, 1)
    norm = grad_norm(gs, p)
    assert norm.dtype == torch.float32 and norm.shape == () and norm.is_cuda
    want = norm64(gs, p)
    check(sizes, norm, want, 2 * U * want)
    assert torch.equal(grad_norm(iter(gs), p), norm)


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("out", list(TYPES))
@pytest.mark.parametrize("sizes", list(LISTS))
def test_clipping_into_other_tensors(sizes, out, dtype):
    gs = make(LISTS[sizes], dtype, 2)
    before = [g.clone() for g in gs]
    outs = [torch.full_like(g, 7, dtype=TYPES[out]) for g in gs]
    want = norm64(gs, 2)
    got, norm = clip_grads(gs, 0.37, out=outs)
    assert all(a is b for a, b in zip(got, outs))
    check("norm", norm, want, 2 * U * want)
    check_clipped(sizes, outs, gs, factor64(want, 0.37))
    assert all(torch.equal(a, b) for a, b in zip(gs, before))
    clip_grads(gs, 1e9, out=outs)                       # the bound holds: a conversion
    assert all(torch.equal(o, g.to(o.dtype)) for o, g in zip(outs, gs))


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("p", [2.0, 1.0, math.inf])
@pytest.mark.parametrize("sizes", list(LISTS))
def test_clipping_in_place(sizes, p, dtype):
    gs = make(LISTS[sizes], dtype, 3)
    before = [g.clone() for g in gs]
    want = norm64(gs, p)
    params = [torch.nn.Parameter(torch.empty_like(g)) for g in gs] + [torch.nn.Parameter(torch.ones(3, device="cuda"))]
    for q, g in zip(params, gs):
        q.grad = g                                      # (the last parameter has no gradient)
    bound = 0.37 * float(want)
    norm = clip_grad_norm_(params, bound, p)
    check("norm", norm, want, 2 * U * want)
    check_clipped(sizes, [q.grad for q in params[:-1]], before, factor64(want, bound))
    assert all(q.grad is g for q, g in zip(params, gs))
    after = [g.clone() for g in gs]
    clip_grad_norm_(iter(params), 2 * float(want), p)
    assert all(torch.equal(a, b) for a, b in zip(gs, after))


@pytest.mark.parametrize("dtype,out", [("f32", "bf16"), ("bf16", "f32"), ("fp16", "fp16")])
def test_large_lists_into_other_tensors(dtype, out):
    # past 4096 tiles (2^26 elements) a workgroup has half a tile; tensors that end in a
    # first half, at its end and in a second, behind guards
    sizes = [16384 * 4096, 3, 16384 + 8192, 16384 + 8193, 8191, 1, 2 * 16384 - 1]
    gs = make(sizes, dtype, 4)
    buffer = torch.full((sum(sizes) + 8 * len(sizes),), 7, dtype=TYPES[out], device="cuda")
    outs, at = [], 0
    for n in sizes:
        outs.append(buffer[at:at + n])
        at += n + 8
    inside = make([1000], dtype, 5)[0]
    before, want = inside.clone(), norm64(gs + [inside], 2)
    norm = clip_grads(gs + [inside], 0.37, out=outs + [inside])[1]
    check("norm", norm, want, 2 * U * want)
    check_clipped("large", outs + [inside], gs + [before], factor64(want, 0.37))
    again = clip_grads(gs, 1e9, out=outs)[1]            # the bound holds: a conversion
    assert all(torch.equal(o, g.to(o.dtype)) for o, g in zip(outs, gs))
    check("again", again, norm64(gs, 2), 2 * U * norm64(gs, 2))
    at = 0
    for n in sizes:
        at += n + 8
        assert (buffer[at - 8:at] == 7).all()


def test_types_in_one_list():
    gs = [make([1000 + i], d, i)[0] for i, d in enumerate(list(TYPES) * 3)]
    before = [g.clone() for g in gs]
    want = norm64(gs, 2)
    outs, norm = clip_grads(gs, 1.0)
    assert outs is not None and all(o is g for o, g in zip(outs, gs))
    check("norm", norm, want, 2 * U * want)
    check_clipped("mixed", gs, before, factor64(want, 1.0))
    # some in place, some into other tensors
    gs = [b.clone() for b in before]
    outs = [g if i % 2 else torch.empty_like(g, dtype=torch.float32) for i, g in enumerate(gs)]
    clip_grads(gs, 1.0, out=outs)
    check_clipped("both", outs, before, factor64(want, 1.0))


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("lead", [1, 2, 3, 5])
def test_any_alignment(lead, dtype):
    buf = make([50000], dtype, 4)[0]
    keep = buf.clone()
    g = buf[lead:lead + 40001]
    want = norm64([g], 2)
    check("norm", grad_norm([g]), want, 2 * U * want)
    clip_grads([g], 1.0)
    check_clipped("view", [g], [keep[lead:lead + 40001]], factor64(want, 1.0))
    assert torch.equal(buf[:lead], keep[:lead]) and torch.equal(buf[lead + 40001:], keep[lead + 40001:])


def test_layouts():
    gen = generator(5)
    base = torch.randn(6, 8, 10, 12, generator=gen, device="cuda")
    for g in (base.clone().permute(0, 3, 1, 2), base.clone().to(memory_format=torch.channels_last), base.clone()[:, ::2],
              base.clone()[:, :, 1:, 3:], base.clone().transpose(1, 2)[1]):
        keep, want = g.clone(), norm64([g], 2)
        strides = g.stride()
        check("norm", grad_norm([g]), want, 2 * U * want)
        out = torch.empty(g.shape, device="cuda", dtype=torch.bfloat16)
        clip_grads([g], 1.0, out=[out])
        check_clipped("out", [out], [keep], factor64(want, 1.0))
        assert torch.equal(g, keep)
        clip_grads([g], 1.0)
        check_clipped("in place", [g], [keep], factor64(want, 1.0))
        assert g.stride() == strides
        outs = torch.zeros(g.shape[::-1], device="cuda").permute(*range(g.dim())[::-1])
        clip_grads([keep], 1.0, out=[outs])
        check_clipped("other strides", [outs], [keep], factor64(want, 1.0))
    e = torch.randn(1, 5, device="cuda").expand(4, 5)
    check("expanded", grad_norm([e]), norm64([e], 2), 4 * U * norm64([e], 2))
    with pytest.raises(RuntimeError, match="single memory location"):
        clip_grads([e], 0.1)
    c = torch.complex(torch.zeros(6, 64), torch.randn(6, 64)).cuda().conj().imag
    keep = c.clone()
    clip_grads([c], 0.5)
    check_clipped("negated", [c], [keep], factor64(norm64([keep], 2), 0.5))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [1e30, 1e-30])
def test_squares_past_the_range_of_float32(scale, dtype):
    gs = make([5000, 40001], dtype, 6, scale)
    before = [g.clone() for g in gs]
    want = norm64(gs, 2)
    bound = 0.1 * float(want)
    check("norm", clip_grads(gs, bound)[1], want, 2 * U * want)
    check_clipped("far", gs, before, factor64(want, bound))


@pytest.mark.parametrize("dtype", list(TYPES))
@pytest.mark.parametrize("p", [2.0, 1.0, math.inf])
def test_infinities_and_nans(p, dtype):
    for value, norm_is in ((math.inf, math.isinf), (-math.inf, math.isinf), (math.nan, math.isnan)):
        for place in (0, 70000):
            gs = make([70001, 30], dtype, 7)
            gs[0][place] = value
            assert norm_is(float(grad_norm(gs, p)))
            norm = clip_grads(gs, 1.0, p)[1]
            assert norm_is(float(norm))
            if math.isnan(value):
                assert all(g.isnan().all() for g in gs)
            else:                                       # everything finite is scaled by 0
                assert gs[0][place].isnan() and gs[0].isnan().sum() == 1
                assert not gs[0][torch.arange(70001, device="cuda") != place].any() and not gs[1].any()
    gs = make([50], dtype, 8)
    gs[0][3], gs[0][4] = math.inf, math.nan
    assert grad_norm(gs, p).isnan()


def test_no_bound_and_a_bound_of_zero():
    gs = make([100], "f32", 9)
    keep = gs[0].clone()
    clip_grads(gs, math.inf)
    assert torch.equal(gs[0], keep)
    gs[0][5] = math.inf
    clip_grads(gs, math.inf)
    assert gs[0][5] == math.inf and torch.equal(gs[0][6:], keep[6:])
    gs = [keep.clone()]
    clip_grads(gs, 0.0)
    assert not gs[0].any()
    z = [torch.zeros(70, device="cuda")]
    assert clip_grads(z, 0.0)[1] == 0 and not z[0].any()


def test_error_if_nonfinite_leaves_gradients():
    p = torch.nn.Parameter(torch.zeros(20, device="cuda"))
    p.grad = torch.ones(20, device="cuda")
    p.grad[3] = math.nan
    keep = p.grad.clone()
    with pytest.raises(RuntimeError, match="norm"):
        clip_grad_norm_([p], 1.0, error_if_nonfinite=True)
    assert torch.equal(p.grad.nan_to_num(5), keep.nan_to_num(5))
    p.grad[3] = 1.0
    assert abs(float(clip_grad_norm_(p, 1.0, error_if_nonfinite=True)) - 20 ** 0.5) < 1e-5


def test_empty_lists():
    assert grad_norm([]) == 0
    outs, norm = clip_grads([], 1.0)
    assert outs == [] and norm == 0
    assert clip_grad_norm_([torch.nn.Parameter(torch.ones(3, device="cuda"))], 1.0) == 0


def test_refusals():
    g = torch.randn(100, device="cuda")
    with pytest.raises(FoError, match="overlap"):
        clip_grads([g, g], 1.0)
    with pytest.raises(FoError, match="overlap"):
        clip_grads([g[:60], g[50:]], 1.0)
    with pytest.raises(FoError, match="overlap"):
        clip_grads([g[:50]], 1.0, out=[g[1:51]])
    assert abs(float(grad_norm([g, g])) - 2 ** 0.5 * float(g.norm())) < 1e-4       # reading twice is fine
    with pytest.raises(ValueError, match="shape"):
        clip_grads([g], 1.0, out=[g[:50]])
    with pytest.raises(ValueError, match="not supported"):
        grad_norm([g.double()])
    with pytest.raises(ValueError, match="dense"):
        grad_norm([torch.eye(3, device="cuda").to_sparse()])
    with pytest.raises(ValueError, match="GPU"):
        grad_norm([g, g.cpu()])


def test_a_strided_tensor_listed_twice_is_refused():
    # such tensors are clipped through copies, which would hide it
    buffer = torch.randn(8, 10, device="cuda")
    before = buffer.clone()
    with pytest.raises(ValueError, match="listed twice"):
        clip_grads([buffer[:, :3], buffer[:, 5:], buffer[:, :3]], 1.0)
    assert torch.equal(buffer, before)
    norm = clip_grads([buffer[:, :5], buffer[:, 5:]], 1.0)[1]      # its halves may be
    check("norm", norm, norm64([before], 2), 2 * U * norm64([before], 2))
    check_clipped("halves", [buffer], [before], factor64(norm64([before], 2), 1.0))


def test_a_graph_that_saved_a_clipped_gradient_is_refused():
    g = torch.randn(10, device="cuda")
    a = torch.randn(10, device="cuda", requires_grad=True)
    y = (a * g).sum()
    clip_grads([g], 0.1)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.backward()


def test_the_norm_has_no_derivative():
    w = torch.randn(10, device="cuda", requires_grad=True)
    norm = grad_norm([w, torch.ones(3, device="cuda")])
    assert abs(float(norm.detach()) - float((w.detach().square().sum() + 3).sqrt())) < 1e-5
    with pytest.raises(RuntimeError, match="no derivative"):
        norm.backward()
    with torch.no_grad():
        assert not grad_norm([w]).requires_grad
    assert not grad_norm([w.detach()]).requires_grad
    with torch.autograd.forward_ad.dual_level(), pytest.raises(NotImplementedError, match="forward-mode"):
        grad_norm([torch.autograd.forward_ad.make_dual(w.detach(), w.detach())])


def test_tracers_are_refused():
    from torch.fx.experimental.proxy_tensor import make_fx
    g = torch.randn(10, device="cuda")
    for f in (lambda t: grad_norm([t]), lambda t: clip_grads([t], 1.0)[1]):
        with pytest.raises(NotImplementedError, match="traced"):
            make_fx(f)(g)


def test_nothing_behind_the_norm_is_written():
    gs = make([100, 5], "f32", 10)
    norm = torch.full((3,), 7.0, device="cuda")
    B.fo_grad_norm(gs, norm[1:2])
    assert torch.equal(norm[1], grad_norm(gs))
    B.fo_grad_clip(gs, gs, 1.0, norm[1:2])
    assert norm[0] == 7 and norm[2] == 7


def test_order_of_the_list_and_repeats_do_not_change_results():
    gs = make([30011, 5, 100000], "bf16", 11)
    a = grad_norm(gs)
    assert all(torch.equal(grad_norm(gs), a) for _ in range(5))
    check("order", grad_norm(gs[::-1]), a.double(), 4 * U * a.double())


@pytest.mark.parametrize("cls", [FlashAdamW, FlashAdam, FlashSGD])
def test_optimizers_clip_every_group(cls):
    gen = generator(12)
    ws = [torch.nn.Parameter(torch.randn(n, generator=gen, device="cuda")) for n in (50, 33, 7)]
    opt = cls([{"params": ws[:2]}, {"params": ws[2:], "lr": 1e-2}], lr=1e-3)
    for w in ws:
        w.grad = torch.randn(w.shape, generator=gen, device="cuda").to(w.dtype)
    before = [w.grad.clone() for w in ws]
    want = norm64(before, 2)
    norm = opt.clip_grad_norm_(0.5)
    check("norm", norm, want, 2 * U * want)
    check_clipped("groups", [w.grad for w in ws], before, factor64(want, 0.5))
    opt.step()
    release = cls([torch.nn.Parameter(torch.randn(8, device="cuda"))], grad_release=True)
    with pytest.raises(RuntimeError, match="grad_release"):
        release.clip_grad_norm_(1.0)

"""Row operators on the GPU (dropout, layer norm, RMS norm, dropout + residual
+ norm) against the float64 oracle, with the a-priori bounds of
rows_helpers.py."""

import numpy as np
import pytest
import torch

from oracle import rows as R
from precision_optimizer_state_amd import binding as B
from precision_optimizer_state_amd import nn
from rows_helpers import DTYPES, U, check, check_backward, check_forward, half_step, host, matrix

pytestmark = pytest.mark.gpu

# around every boundary a launch shape may have: chunks of 8, lanes of a wave, a
# workgroup's reach, and past the longest rows kept in registers
COLS = [1, 2, 7, 8, 9, 31, 64, 65, 127, 128, 129, 250, 256, 257, 511, 512, 513, 768, 1000, 1024, 1025, 1601, 2047,
        2048, 2049, 4095, 4096, 4100, 8191, 8192, 8200, 16383, 16384, 16385, 20000, 40001]
SEED, OFFSET = 0xDEADBEEF12345678, 0x123456789A


def rng_of(*key):
    return np.random.default_rng(np.random.SeedSequence([hash(k) % 2 ** 32 if not isinstance(k, str)
                                                         else sum(map(ord, k)) for k in key]))


# ---------------------------------------------------------------------------
# dropout
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", [(1, 1), (1, 7), (3, 8), (5, 9), (64, 1), (33, 100), (7, 1024), (1000, 768),
                                   (2, 100001), (70000, 3)])
def test_dropout_values_and_gradient(shape, dtype):
    rng, dt, p = rng_of(*shape, dtype), DTYPES[dtype], 0.3
    x = matrix(rng, *shape, dt).requires_grad_(True)
    dy = matrix(rng, *shape, dt)
    y = nn.dropout(x, p, SEED, OFFSET)
    dx, = torch.autograd.grad(y, x, dy)
    for name, got, src in (("y", y, x), ("dx", dx, dy)):
        want = R.dropout(host(src), p, SEED, OFFSET)
        check(name, got, want, dt, 2 * U * np.abs(want))
        assert np.array_equal(host(got) == 0, ~R.keep(*shape, p, SEED, OFFSET) | (host(src) == 0)), name


@pytest.mark.parametrize("p", [2.0 ** -32, 1e-6, 0.1, 0.5, 1 - 2.0 ** -16, 1 - 2.0 ** -32])
def test_dropout_decisions_are_exact(p):
    # the second generator call decides where the first half-word is the threshold's: enough
    # elements for that to happen some tens of times
    shape = (1500, 1111)
    ones = torch.ones(shape, device="cuda")
    for seed, offset in ((0, 0), (2 ** 64 - 1, 2 ** 64 - 1), (SEED, 7)):
        got = nn.dropout(ones, p, seed, offset) != 0
        assert np.array_equal(got.cpu().numpy(), R.keep(*shape, p, seed, offset)), (p, seed)


def test_dropout_open_decisions_occur():
    u = R.uniforms(1500, 1111, SEED, 7)
    t = R.threshold(0.1)
    assert (u >> 16 == t >> 16).sum() >= 10          # the case above covers both sides of the second half-word
    tied = u[u >> 16 == t >> 16]
    assert (tied >= t).any() and (tied < t).any()


def test_dropout_of_everything_and_of_nothing():
    x = torch.full((9, 31), float("nan"), device="cuda", requires_grad=True)
    y = nn.dropout(x, 1.0, 1, 2)
    assert (y == 0).all() and not torch.signbit(y).any()
    dx, = torch.autograd.grad(y, x, torch.full_like(y, float("inf")))
    assert (dx == 0).all()
    assert nn.dropout(x, 0.0, 1, 2) is x


def test_dropped_infinities_and_nan_are_zero():
    shape = (64, 40)
    x = torch.full(shape, float("inf"), device="cuda", dtype=torch.bfloat16)
    x[::2] = float("nan")
    y = nn.dropout(x, 0.5, SEED, 3)
    k = torch.from_numpy(R.keep(*shape, 0.5, SEED, 3)).cuda()
    assert (y[~k] == 0).all()
    assert torch.isinf(y[1::2][k[1::2]]).all() and torch.isnan(y[::2][k[::2]]).all()


@pytest.mark.parametrize("layout", ["slice", "transposed", "expanded", "rows of a permutation", "0-d", "empty"])
def test_dropout_layouts(layout):
    base = torch.randn(6, 10, 24, device="cuda")
    x = {"slice": base[:, :, 3:20], "transposed": base.transpose(1, 2), "expanded": base[:1, :1].expand(6, 10, 24),
         "rows of a permutation": base.permute(1, 0, 2), "0-d": base[0, 0, 0], "empty": base[:, :0]}[layout]
    x = x.detach().requires_grad_(True)
    y = nn.dropout(x, 0.4, SEED, 1)
    assert y.shape == x.shape and y.is_contiguous()
    if x.numel():
        flat = host(x).reshape(-1, x.shape[-1] if x.dim() else 1)
        want = R.dropout(flat, 0.4, SEED, 1).reshape(tuple(x.shape))
        check("y", y, want, torch.float32, 2 * U * np.abs(want))
    y.sum().backward()                               # an expanded gradient
    want = np.where(host(y) != 0, R.scale(0.4), 0.0)
    check("dx", x.grad, want, torch.float32, 2 * U * want)


def test_dropout_past_32_bits():
    # more than 2^32 elements, compared at both ends; the chunk index passes 2^29 and the
    # element offset 2^32
    rows, cols = (1 << 17) + 9, 1 << 15
    x = torch.ones(rows, cols, dtype=torch.bfloat16, device="cuda")
    y = nn.dropout(x, 0.25, SEED, OFFSET)
    for first in (0, 1 << 16, (1 << 17) - 3, rows - 5):
        got = (y[first:first + 5] != 0).cpu().numpy()
        assert np.array_equal(got, R.keep(5, cols, 0.25, SEED, OFFSET, first)), first
    del x, y


def test_dropout_of_more_chunks_than_one_launch_covers():
    # 2^32 chunks of one element each and some more: the grid covers 2^32 chunks and loops for the rest
    rows = (1 << 32) + 601
    x = torch.ones(rows, 1, dtype=torch.bfloat16, device="cuda")
    y = nn.dropout(x, 0.3, SEED, OFFSET)
    for first in (0, (1 << 31) - 300, (1 << 32) - 300, rows - 600):
        got = (y[first:first + 600] != 0).cpu().numpy()
        assert np.array_equal(got, R.keep(600, 1, 0.3, SEED, OFFSET, first)), first
    del x, y


# ---------------------------------------------------------------------------
# norms
# ---------------------------------------------------------------------------
def run_norm(kind, rows, cols, dtype, wdtype, join=False, p=0.0, affine=True, pad=0, lead=0, seed_key=0, loc=0.3):
    rng = rng_of(kind, rows, cols, dtype, wdtype, seed_key)
    dt, wdt, eps = DTYPES[dtype], DTYPES[wdtype], 1e-5
    x = matrix(rng, rows, cols, dt, loc, 1.5, pad, lead).detach().requires_grad_(True)
    res = matrix(rng, rows, cols, dt, -0.2, 2.0).requires_grad_(True) if join else None
    w = (matrix(rng, 1, cols, wdt, 1.0, 0.3)[0]).detach().requires_grad_(True) if affine else None
    b = (matrix(rng, 1, cols, wdt, 0.0, 0.3)[0]).detach().requires_grad_(True) if affine and kind == "layer" else None
    dy, dh = matrix(rng, rows, cols, dt, 0.0, 1.0, pad, lead), matrix(rng, rows, cols, dt) if join else None
    key = dict(p=p, seed=SEED, offset=OFFSET) if join else {}
    fn = {("layer", False): lambda: nn.layer_norm(x, w, b, eps),
          ("rms", False): lambda: nn.rms_norm(x, w, eps),
          ("layer", True): lambda: nn.dropout_add_layer_norm(x, res, w, b, eps, **key),
          ("rms", True): lambda: nn.dropout_add_rms_norm(x, res, w, eps, **key)}[kind, join]
    tag = f"{kind} {rows}x{cols} {dtype}/{wdtype} join={join} p={p}"
    with torch.no_grad():
        inference = fn()
    out = fn()
    leaves = {k: t for k, t in (("x", x), ("residual", res), ("weight", w), ("bias", b)) if t is not None}
    if join:
        h, y = out
        assert torch.equal(inference[0], h) and torch.equal(inference[1], y)
        want = host(res) + (R.dropout(host(x), p, SEED, OFFSET) if p else host(x))
        check(tag + " h", h, want, dt, 3 * U * (np.abs(host(x)) * max(1.0, R.scale(p)) + np.abs(host(res))))
        grads = torch.autograd.grad([h, y], list(leaves.values()), [dh, dy])
    else:
        y = out
        assert torch.equal(inference, y)
        h = x
        grads = torch.autograd.grad(y, list(leaves.values()), dy)
    grads = dict(zip(leaves, grads))
    hw, hb = None if w is None else host(w), None if b is None else host(b)
    check_forward(tag + " y", y, host(h), hw, hb, eps, kind)
    got = {"d": grads["residual" if join else "x"], "dx": grads["x"] if join and p else None,
           "dweight": grads.get("weight"), "dbias": grads.get("bias")}
    check_backward(tag, got, host(dy), host(h), hw, eps, kind, None if dh is None else host(dh), (p, SEED, OFFSET))
    if join and not p:
        assert torch.equal(grads["x"], grads["residual"])


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_norm_every_width(kind, cols):
    for i, (rows, dtype, wdtype) in enumerate([(1, "bf16", "bf16"), (5, "fp16", "f32"), (37, "f32", "f32")]):
        run_norm(kind, rows, cols, dtype, wdtype, seed_key=i)


@pytest.mark.parametrize("cols", COLS)
@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_join_every_width(kind, cols):
    for i, (rows, dtype, wdtype, p) in enumerate([(3, "bf16", "bf16", 0.1), (17, "fp16", "fp16", 0.5),
                                                  (2, "f32", "f32", 0.25), (9, "bf16", "f32", 0.0)]):
        run_norm(kind, rows, cols, dtype, wdtype, join=True, p=p, seed_key=i)


@pytest.mark.parametrize("rows", [1, 2, 3, 8, 63, 64, 65, 255, 257, 1023, 2049, 5000, 20011])
@pytest.mark.parametrize("cols", [33, 128, 768, 1500])
def test_norm_row_counts(rows, cols):
    run_norm("layer", rows, cols, "bf16", "bf16")
    run_norm("rms", rows, cols, "f32", "f32", join=True, p=0.2)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("wdtype", DTYPES)
def test_norm_type_pairs(dtype, wdtype):
    run_norm("layer", 19, 300, dtype, wdtype, join=True, p=0.1)
    run_norm("rms", 19, 300, dtype, wdtype)


@pytest.mark.parametrize("pad, lead", [(8, 0), (3, 0), (0, 1), (16, 8), (5, 5)])
@pytest.mark.parametrize("dtype", DTYPES)
def test_norm_of_row_slices(pad, lead, dtype):
    for cols in (40, 999, 1024, 5000):
        run_norm("layer", 13, cols, dtype, "f32", pad=pad, lead=lead)
        run_norm("rms", 13, cols, dtype, dtype, join=True, p=0.3, pad=pad, lead=lead)


def test_norm_without_parameters():
    run_norm("layer", 21, 333, "bf16", "bf16", affine=False)
    run_norm("rms", 21, 333, "f32", "f32", join=True, p=0.1, affine=False)


def test_norm_of_rows_far_from_zero():
    # mean 1000 times the spread: variances taken from squares less the squared mean would
    # lose everything here (the bound carries mean|h| * rstd)
    run_norm("layer", 11, 768, "f32", "f32", loc=1500.0)
    run_norm("layer", 11, 5000, "f32", "f32", loc=-1500.0)


def test_more_rows_than_one_launch_covers():
    # 2^31 threads hold 2^28 rows of 8 columns; both ends and the seam against the oracle
    rows, cols = (1 << 28) + 37, 8
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda").normal_()
    with torch.no_grad():
        y = nn.layer_norm(x)
    for at in (0, (1 << 28) - 16, rows - 16):
        check_forward(f"rows from {at}", y[at:at + 16], host(x[at:at + 16]), None, None, 1e-5, "layer")
    del x, y


def test_very_long_rows():
    run_norm("layer", 2, 3_000_017, "bf16", "f32", join=True, p=0.1)
    run_norm("rms", 3, 1_000_000, "f32", "bf16")


def test_join_that_drops_everything():
    run_norm("layer", 7, 100, "bf16", "bf16", join=True, p=1.0)


@pytest.mark.parametrize("shape", [(0, 16), (4, 0, 16)])
def test_norm_of_no_rows(shape):
    x = torch.zeros(shape, device="cuda", requires_grad=True)
    w = torch.ones(16, device="cuda", requires_grad=True)
    b = torch.ones(16, device="cuda", requires_grad=True)
    h, y = nn.dropout_add_layer_norm(x, x, w, b, p=0.1, seed=1)
    assert h.shape == y.shape == shape
    gx, gw, gb = torch.autograd.grad([h, y], [x, w, b], [torch.zeros_like(h), torch.zeros_like(y)])
    assert gx.shape == shape and (gw == 0).all() and (gb == 0).all()


def test_constant_rows_and_one_column():
    # no spread: y is the bias, the gradient of the rows 0 up to eps' share
    x = torch.full((5, 96), 3.0, device="cuda", requires_grad=True)
    w, b = torch.full((96,), 2.0, device="cuda"), torch.full((96,), 0.5, device="cuda")
    y = nn.layer_norm(x, w, b)
    assert torch.equal(y, torch.full_like(y, 0.5))
    one = torch.randn(7, 1, device="cuda", requires_grad=True)
    y1 = nn.layer_norm(one)
    dx, = torch.autograd.grad(y1, one, torch.ones_like(y1))
    assert (y1 == 0).all() and (dx == 0).all()


def test_nan_and_infinite_rows_stay_alone():
    x = torch.randn(9, 500, device="cuda", dtype=torch.bfloat16)
    clean = nn.layer_norm(x)
    x[3, 17], x[6, 400] = float("nan"), float("inf")
    y = nn.layer_norm(x)
    assert torch.isnan(y[3]).all() and torch.isnan(y[6]).all()
    rest = [0, 1, 2, 4, 5, 7, 8]
    assert torch.equal(y[rest], clean[rest])


def test_norm_layouts_and_broadcast_inputs():
    base = torch.randn(4, 6, 40, device="cuda")
    for x in (base.transpose(0, 1), base.transpose(1, 2), base[:, ::2], base[:1].expand(4, 6, 40), base[:, :, 1:33],
              base[0, 0]):
        x = x.detach().requires_grad_(True)
        y = nn.rms_norm(x)
        flat = host(x).reshape(-1, x.shape[-1])
        check_forward("y", y.reshape(flat.shape), flat, None, None, 1e-6, "rms")
        dx, = torch.autograd.grad(y, x, torch.ones_like(y))
        check_backward("dx", {"d": dx.reshape(flat.shape)}, np.ones_like(flat), flat, None, 1e-6, "rms")
    # a residual broadcast over the batch: autograd sums the gradient of the expanded one
    pos = torch.randn(6, 40, device="cuda", requires_grad=True)
    h, y = nn.dropout_add_layer_norm(base, pos.expand(4, 6, 40))
    gpos, = torch.autograd.grad([h, y], pos, [torch.ones_like(h), torch.ones_like(y)])
    hh = host(h).reshape(-1, 40)
    d, _, _ = R.norm_backward(np.ones_like(hh), hh, dh=np.ones_like(hh))
    np.testing.assert_allclose(host(gpos), d.reshape(4, 6, 40).sum(0), atol=1e-4)


def test_only_some_gradients():
    x, r = torch.randn(33, 72, device="cuda"), torch.randn(33, 72, device="cuda")
    w, b = torch.randn(72, device="cuda"), torch.randn(72, device="cuda")
    dy, dh = torch.randn(33, 72, device="cuda"), torch.randn(33, 72, device="cuda")
    full = {}
    for want in (("x", "r", "w", "b"), ("x",), ("r",), ("w",), ("b",), ("x", "b"), ("r", "w")):
        t = {"x": x.clone(), "r": r.clone(), "w": w.clone(), "b": b.clone()}
        leaves = [t[k].requires_grad_(True) for k in want]
        h, y = nn.dropout_add_layer_norm(t["x"], t["r"], t["w"], t["b"], p=0.2, seed=5)
        outs, grads = ([h, y], [dh, dy]) if h.requires_grad and set(want) & {"x", "r"} else ([y], [dy])
        got = dict(zip(want, torch.autograd.grad(outs, leaves, grads)))
        full = full or got
        for k in got:
            assert torch.equal(got[k], full[k]), (want, k)


def test_unused_outputs():
    def fresh():
        return [torch.randn(12, 50, device="cuda", requires_grad=True) for _ in range(2)]
    dy = torch.randn(12, 50, device="cuda")
    x, r = fresh()
    h, y = nn.dropout_add_layer_norm(x, r, p=0.3, seed=9)
    gx, gr = torch.autograd.grad(h, [x, r], dy)                    # the norm unused
    assert torch.equal(gr, dy)
    check("dx", gx, R.dropout(host(dy), 0.3, 9, 0), torch.float32, 4 * U * np.abs(host(dy)))
    x, r = fresh()
    h, y = nn.dropout_add_layer_norm(x, r, p=0.3, seed=9)
    gx, gr = torch.autograd.grad(y, [x, r], dy)                    # the sum used by the norm alone
    check_backward("y only", {"d": gr, "dx": gx}, host(dy), host(h), None, 1e-5, "layer", None, (0.3, 9, 0))


@pytest.mark.parametrize("kind", ["layer", "rms"])
@pytest.mark.parametrize("cols", [24, 768, 20000])
def test_gradient_against_differences(kind, cols):
    """Directional central differences of the float32 kernel's own output.  The
    oracle's differences at the same step give what the step's truncation makes
    of the derivative; the kernel may differ from them by its output bounds
    over the step."""
    rng = rng_of(kind, cols, "differences")
    x, v, c, w = (rng.normal(size=s) for s in ((6, cols), (6, cols), (6, cols), (cols,)))
    step = 2.0 ** -6

    def f32(a):
        return torch.from_numpy(a.astype(np.float32)).cuda()

    x, v, c, w = (host(f32(a)) for a in (x, v, c, w))
    fn = (lambda t: nn.layer_norm(t, f32(w))) if kind == "layer" else (lambda t: nn.rms_norm(t, f32(w), 1e-5))
    xp, xm = host(f32(x + step * v)), host(f32(x - step * v))
    got = (c * (host(fn(f32(xp))) - host(fn(f32(xm))))).sum() / (2 * step)
    yp, ym = (R.norm_forward(t, w, None, 1e-5, kind) for t in (xp, xm))
    want = (c * (yp[0] - ym[0])).sum() / (2 * step)
    err = 0.0
    for t, (y, mean, rstd) in ((xp, yp), (xm, ym)):
        u, big = np.abs(t - mean) * rstd, np.abs(t).mean(1, keepdims=True) * rstd
        err += (np.abs(c * w) * U * (cols / 256 + 42) * (u + big) + np.abs(c) * U * np.abs(y)).sum() / (2 * step)
    assert abs(got - want) <= err
    # and the kernel's gradient along v is the oracle's exact one
    xt = f32(x).requires_grad_(True)
    dx, = torch.autograd.grad(fn(xt), xt, f32(c))
    d, _, _ = R.norm_backward(c, x, w, 1e-5, kind)
    check_backward("dx", {"d": dx}, c, x, w, 1e-5, kind)
    # the differences approach that derivative: their distance is the truncation, step^2 / 6
    # times the third derivative along v, a few times |c w v| for rows of unit spread
    assert abs(want - (d * v).sum()) <= 40 * step ** 2 * np.abs(c * w).sum()


def test_weight_gradients_repeat_bitwise():
    x = torch.randn(9001, 768, device="cuda", dtype=torch.bfloat16)
    w = torch.ones(768, device="cuda", requires_grad=True)
    b = torch.zeros(768, device="cuda", requires_grad=True)
    dy = torch.randn(9001, 768, device="cuda", dtype=torch.bfloat16)
    first = torch.autograd.grad(nn.layer_norm(x, w, b), [w, b], dy)
    for _ in range(3):
        again = torch.autograd.grad(nn.layer_norm(x, w, b), [w, b], dy)
        assert all(torch.equal(p, q) for p, q in zip(first, again))


def test_outputs_end_where_they_should():
    """Rows behind the last one, and the memory around every output, stay as they were."""
    for rows, cols in ((3, 5), (7, 100), (2, 1000), (5, 4097), (2, 16391)):
        for dt in DTYPES.values():
            def guarded(shape, dtype):
                n = int(np.prod(shape))
                buf = torch.full((n + 128,), 77.0, dtype=dtype, device="cuda")
                return buf, buf[64:64 + n].view(shape)
            x, r, dy = (torch.randn(rows, cols, device="cuda").to(dt) for _ in range(3))
            key = B.dropout_key(0.4, 3)
            bufs = {k: guarded((rows, cols), dt) for k in ("h", "y", "d", "dx", "z")}
            bufs.update({k: guarded((rows,), torch.float32) for k in ("mean", "rstd")})
            bufs.update({k: guarded((cols,), torch.float32) for k in ("dw", "db")})
            o = {k: v[1] for k, v in bufs.items()}
            w = torch.ones(cols, device="cuda")
            B.fo_dropout(x, o["z"], key)
            B.fo_norm_forward(x, o["y"], "layer", w, None, 1e-5, r, o["h"], o["mean"], o["rstd"], key)
            B.fo_norm_backward(dy, o["h"], o["rstd"], "layer", o["mean"], w, None, o["d"], o["dx"], o["dw"], o["db"],
                               drop=key)
            for k, (buf, view) in bufs.items():
                assert (buf[:64] == 77).all() and (buf[64 + view.numel():] == 77).all(), (rows, cols, dt, k)
                assert not (view == 77).all(), k


# ---------------------------------------------------------------------------
# streams, graphs, devices, modules, and a training step
# ---------------------------------------------------------------------------
def test_on_a_side_stream():
    x, r = torch.randn(512, 768, device="cuda"), torch.randn(512, 768, device="cuda")
    want = nn.dropout_add_layer_norm(x, r, p=0.1, seed=4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        x2, r2 = (x * 1).requires_grad_(True), r * 1
        got = nn.dropout_add_layer_norm(x2, r2, p=0.1, seed=4)
        g, = torch.autograd.grad(got, x2, [r2, r2])
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    check_backward("side", {"dx": g}, host(r), host(want[0]), None, 1e-5, "layer", host(r), (0.1, 4, 0))


def test_two_streams_at_once():
    """Backward passes with weight gradients on two streams, unordered: each has its
    own workspace, so both give what they give alone."""
    gen = torch.Generator(device="cuda").manual_seed(8)
    data = [[torch.randn(4000, 1024, device="cuda", generator=gen) for _ in range(2)] for _ in range(2)]
    w = torch.ones(1024, device="cuda", requires_grad=True)
    alone = [torch.autograd.grad(nn.layer_norm(h, w), w, dy)[0] for h, dy in data]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        got = []
        for stream, (h, dy) in zip(streams, data):
            with torch.cuda.stream(stream):
                leaf = w.detach().requires_grad_(True)
                got.append(torch.autograd.grad(nn.layer_norm(h, leaf), leaf, dy)[0])
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, alone))


def test_one_tensor_as_both_inputs_and_backward_twice():
    x = torch.randn(30, 200, device="cuda", requires_grad=True)
    dh, dy = torch.randn(30, 200, device="cuda"), torch.randn(30, 200, device="cuda")
    h, y = nn.dropout_add_rms_norm(x, x, p=0.3, seed=np.int64(6))
    first, = torch.autograd.grad([h, y], x, [dh, dy], retain_graph=True)
    again, = torch.autograd.grad([h, y], x, [dh, dy])
    assert torch.equal(first, again)
    d, _, _ = R.norm_backward(host(dy), host(h), None, 1e-6, "rms", host(dh))
    want = d + np.where(R.keep(30, 200, 0.3, 6, 0), d * R.scale(0.3), 0.0)
    # two gradients within the bound of check_backward, below 2^-15 of values of order 1, and one sum
    np.testing.assert_allclose(host(first), want, rtol=2.0 ** -15, atol=2.0 ** -15)
    with pytest.raises(RuntimeError, match="second time"):
        torch.autograd.grad([h, y], x, [dh, dy])


def test_an_output_changed_before_the_backward_pass_is_refused():
    x, r = (torch.randn(4, 16, device="cuda", requires_grad=True) for _ in range(2))
    h, y = nn.dropout_add_layer_norm(x, r)
    with torch.no_grad():
        h.add_(1.0)
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()


def test_checkpointed_recomputation_finds_the_same_mask():
    from torch.utils.checkpoint import checkpoint
    counter = nn.DropoutCounter(seed=4)
    x, r = (torch.randn(16, 64, device="cuda", requires_grad=True) for _ in range(2))
    w = torch.ones(64, device="cuda", requires_grad=True)
    key = counter.next()

    def block(x, r):
        h, y = nn.dropout_add_rms_norm(x, r, w, p=0.4, **key)
        return h * y

    want = torch.autograd.grad(block(x, r).sum(), [x, r, w])
    got = torch.autograd.grad(checkpoint(block, x, r, use_reentrant=False).sum(), [x, r, w])
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_explicit_stream_needs_its_own_workspace():
    h, dy = torch.randn(8, 16, device="cuda"), torch.randn(8, 16, device="cuda")
    rstd, dw = torch.ones(8, device="cuda"), torch.empty(16, device="cuda")
    stream = torch.cuda.current_stream().cuda_stream
    with pytest.raises(ValueError, match="workspace"):
        B.fo_norm_backward(dy, h, rstd, "rms", dweight_out=dw, stream=stream)
    ws = torch.empty(B.fo_norm_backward_workspace(8, 16), dtype=torch.uint8, device="cuda")
    B.fo_norm_backward(dy, h, rstd, "rms", dweight_out=dw, workspace=ws, stream=stream)
    torch.cuda.synchronize()
    check("dw", dw, (host(dy) * host(h)).sum(0), torch.float32, 100 * U * np.abs(host(dy) * host(h)).sum(0))


def test_captured_step_draws_new_masks():
    """A forward and backward pass in one HIP graph: every replay equals the eager
    step with the offsets the counter has reached, with eager work between."""
    rows, cols, p = 300, 768, 0.1
    counter = nn.DropoutCounter(seed=77, device="cuda")
    x, r = torch.randn(rows, cols, device="cuda"), torch.randn(rows, cols, device="cuda")
    w, b = torch.ones(cols, device="cuda"), torch.zeros(cols, device="cuda")
    dy, dh = torch.randn(rows, cols, device="cuda"), torch.randn(rows, cols, device="cuda")
    args = [counter.next(), counter.next()]

    def step(state_args):
        leaves = [t.detach().requires_grad_(True) for t in (x, r, w, b)]
        z = nn.dropout(leaves[0], p, **state_args[0])
        h, y = nn.dropout_add_layer_norm(z, leaves[1], leaves[2], leaves[3], p=p, **state_args[1])
        return [h, y, *torch.autograd.grad([h, y], leaves, [dh, dy])]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(args)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(args)
        counter.advance()
    # the capture ran nothing: the state still stands at its start
    masks = []
    for replay in range(4):
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        eager = [dict(a, offset=a["offset"] + replay * nn.DropoutCounter._STRIDE, state=None) for a in args]
        want = step(eager)
        for i, (g, e) in enumerate(zip(got, want)):
            assert torch.equal(g, e), (replay, i)
        masks.append(got[0])
        x.normal_()
        torch.cuda.synchronize()
    assert not torch.equal(masks[0], masks[1])
    assert counter.state.tolist() == [0, 4 * nn.DropoutCounter._STRIDE]


def test_two_graphs_do_not_share_a_workspace():
    def make(seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        h, dy = (torch.randn(3000, 512, device="cuda", generator=g) for _ in range(2))
        w = torch.ones(512, device="cuda", requires_grad=True)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            want = torch.autograd.grad(nn.rms_norm(h, w), w, dy)[0].clone()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            leaf = w.detach().requires_grad_(True)
            out, = torch.autograd.grad(nn.rms_norm(h, leaf), leaf, dy)
        return graph, out, want, (h, dy, w, leaf)

    made = [make(s) for s in (1, 2)]
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(3):
        torch.cuda.synchronize()
        for s, m in ((s1, made[0]), (s2, made[1])):
            with torch.cuda.stream(s):
                m[0].replay()
        torch.cuda.synchronize()
        for m in made:
            assert torch.equal(m[1], m[2])


def test_capture_refuses_leaves_of_a_living_eager_graph():
    x = torch.randn(8, 32, device="cuda", requires_grad=True)
    w = torch.ones(32, device="cuda", requires_grad=True)
    alive = nn.rms_norm(x, w)                        # made on the default stream, still alive
    torch.cuda.synchronize()
    for call in (lambda: nn.rms_norm(x, w), lambda: nn.dropout(x, 0.5, 1),
                 lambda: nn.dropout_add_layer_norm(x.detach(), x.detach(), w)):
        with pytest.raises(RuntimeError, match="default stream"):
            with torch.cuda.graph(torch.cuda.CUDAGraph()):
                call()
    del alive
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):                    # the eager graph is gone
        y = nn.rms_norm(x, w)
        gx, gw = torch.autograd.grad(y, [x, w], y.detach())
    graph.replay()
    torch.cuda.synchronize()
    check_backward("captured", {"d": gx, "dweight": gw}, host(y), host(x), host(w), 1e-6, "rms")


def test_state_changed_before_the_backward_pass_is_refused():
    counter = nn.DropoutCounter(seed=1, device="cuda")
    x = torch.randn(4, 8, device="cuda", requires_grad=True)
    y = nn.dropout(x, 0.5, **counter.next())
    counter.advance()
    with pytest.raises(RuntimeError, match="modified by an inplace operation"):
        y.sum().backward()
    h, y = nn.dropout_add_rms_norm(x, x, p=0.0, **counter.next())
    counter.advance()                                # no mask came from it
    y.sum().backward()


def test_modules_follow_torch():
    torch.manual_seed(0)
    x = torch.randn(4, 9, 200, device="cuda")
    ln, fl = torch.nn.LayerNorm(200, device="cuda"), nn.FlashLayerNorm(200, device="cuda")
    rn, fr = torch.nn.RMSNorm(200, eps=1e-6, device="cuda"), nn.FlashRMSNorm(200, device="cuda")
    for ours, theirs in ((fl, ln), (fr, rn)):
        with torch.no_grad():
            for q in theirs.parameters():
                q.normal_()
        ours.load_state_dict(theirs.state_dict())
        torch.testing.assert_close(ours(x), theirs(x), rtol=1e-5, atol=1e-5)
    counter = nn.DropoutCounter(seed=3)
    drop = nn.FlashDropout(0.25, counter)
    a, b = drop(x), drop(x)
    assert counter.offset == 2 and not torch.equal(a, b)
    assert torch.equal(a, nn.dropout(x, 0.25, 3, 0)) and torch.equal(b, nn.dropout(x, 0.25, 3, 1))
    drop.eval()
    assert drop(x) is x and counter.offset == 2


@pytest.mark.parametrize("release", [False, True])
def test_training_steps_with_the_optimizer(release):
    """Blocks of linear -> dropout + residual + norm trained by FlashAdamW: the
    norm's weight gradients arrive in theta' type, every gradient is that of the
    float64 model with the same masks, and parameters move."""
    from precision_optimizer_state_amd import FlashAdamW
    torch.manual_seed(1)
    dim, rows, layers, p = 96, 40, 2, 0.2
    counter = nn.DropoutCounter(seed=21)
    params = []
    for _ in range(layers):
        params.append({"lin": torch.nn.Parameter(torch.randn(dim, dim, device="cuda") / 10),
                       "w": torch.nn.Parameter(1 + torch.randn(dim, device="cuda") / 10),
                       "b": torch.nn.Parameter(torch.randn(dim, device="cuda") / 10)})
    flat = [q for layer in params for q in layer.values()]
    opt = FlashAdamW(flat, lr=1e-2, grad_release=release)
    assert all(q.dtype == torch.bfloat16 for q in flat)
    x0 = torch.randn(rows, dim, device="cuda").bfloat16()
    seen = {}
    if release:
        for i, q in enumerate(flat):
            q.register_hook(lambda g, i=i: seen.__setitem__(i, g.clone()))
    for _ in range(2):
        keys = [counter.next() for _ in range(layers)]
        before = [q.detach().clone() for q in flat]
        h = nn.dropout(x0, p, 5, 5)
        y = h
        for layer, key in zip(params, keys):
            h, y = nn.dropout_add_layer_norm(y @ layer["lin"], h, layer["w"], layer["b"], p=p, **key)
        loss = (h.float() * y.float()).mean()
        loss.backward()
        grads = [seen[i] for i in range(len(flat))] if release else [q.grad.clone() for q in flat]
        assert all(g.dtype == torch.bfloat16 for g in grads)
        # the same model in float64 with torch's operations and the oracle's masks
        ref = [q.cpu().double().requires_grad_(True) for q in before]
        def drop(t, key):
            k = torch.from_numpy(R.keep(rows, dim, p, key["seed"], key["offset"]))
            return torch.where(k, t * R.scale(p), torch.zeros_like(t))
        hr = drop(x0.cpu().double(), {"seed": 5, "offset": 5})
        yr = hr
        for i, key in enumerate(keys):
            lin, w, b = ref[3 * i:3 * i + 3]
            hr = hr + drop(yr @ lin, key)
            yr = torch.nn.functional.layer_norm(hr, (dim,), w, b, 1e-5)
        (hr * yr).mean().backward()
        for i, (g, want) in enumerate(zip(grads, ref)):
            # about ten bf16 roundings (each 2^-8 relative) in a row on the way forward and
            # back, in quadrature over the elements of a gradient: 12 * 2^-8 of its norm
            err = (g.cpu().double() - want.grad).norm() / want.grad.norm()
            assert err < 12 * 2.0 ** -8, (i, float(err))
        if not release:
            opt.step()
            opt.zero_grad()
        assert all(not torch.equal(q, o) for q, o in zip(flat, before) if q.dim() == 2)


def test_modules_under_the_optimizer():
    """The modules as layers of a model FlashAdamW owns: their weights become theta',
    every gradient has its type, and the weights move against the gradient."""
    from precision_optimizer_state_amd import FlashAdamW
    torch.manual_seed(2)
    counter = nn.DropoutCounter(seed=5)
    model = torch.nn.Sequential(torch.nn.Linear(48, 80, device="cuda"), nn.FlashLayerNorm(80, device="cuda"),
                                nn.FlashDropout(0.1, counter), torch.nn.Linear(80, 24, device="cuda"),
                                nn.FlashRMSNorm(24, device="cuda"))
    opt = FlashAdamW(model.parameters(), lr=1e-2, weight_decay=0.0)
    x, target = torch.randn(64, 48, device="cuda").bfloat16(), torch.randn(64, 24, device="cuda")
    before = [opt.master_weights(q) for q in model.parameters()]
    (model(x).float() - target).square().mean().backward()
    grads = [q.grad.float() for q in model.parameters()]
    assert counter.offset == 1
    opt.step()
    for q, old, g in zip(model.parameters(), before, grads):
        assert q.dtype == q.grad.dtype == torch.bfloat16
        # the first step of AdamW moves every weight by lr against its gradient's sign
        step = opt.master_weights(q) - old
        sure = g.abs() > 1e-6
        assert sure.any() and (torch.sign(step[sure]) == -torch.sign(g[sure])).all()


def test_device_state_is_added_to_the_key():
    x = torch.ones(40, 100, device="cuda")
    state = torch.tensor([3, -1], dtype=torch.int64, device="cuda")          # -1: the offset wraps
    y = torch.empty_like(x)
    B.fo_dropout(x, y, B.dropout_key(0.5, 7, 10, state))
    assert np.array_equal((y != 0).cpu().numpy(), R.keep(40, 100, 0.5, 10, 9))
    assert torch.equal(nn.dropout(x, 0.5, 7, 10, state), y)
    h, _ = nn.dropout_add_rms_norm(x, torch.zeros_like(x), p=0.5, seed=7, offset=10, state=state)
    assert torch.equal(h, y)


# ---------------------------------------------------------------------------
# refusals that need a device tensor
# ---------------------------------------------------------------------------
def test_refusals():
    x = torch.randn(4, 8, device="cuda")
    w = torch.ones(8, device="cuda")
    with pytest.raises(ValueError, match="probability"):
        nn.dropout(x, 1.5, 0)
    with pytest.raises(ValueError, match="probability"):
        nn.dropout(x, float("nan"), 0)
    with pytest.raises(ValueError, match="not supported"):
        nn.dropout(x.double(), 0.5, 0)
    with pytest.raises(ValueError, match="GPU"):
        nn.layer_norm(x.cpu())
    with pytest.raises(ValueError, match="weight has shape"):
        nn.layer_norm(x, w[:4])
    with pytest.raises(ValueError, match="must agree"):
        nn.layer_norm(x, w, w.bfloat16())
    with pytest.raises(ValueError, match="residual must be"):
        nn.dropout_add_rms_norm(x, x.bfloat16(), w)
    with pytest.raises(ValueError, match="residual must be"):
        nn.dropout_add_rms_norm(x, x[:1], w)
    with pytest.raises(ValueError, match="last dimension"):
        nn.rms_norm(x[:, :0])
    with pytest.raises(ValueError, match="2 int64"):
        nn.dropout(x, 0.5, 0, state=torch.zeros(3, dtype=torch.int64, device="cuda"))
    with pytest.raises(B.FoError, match="eps") as e:
        nn.layer_norm(x, w, eps=-1.0)
    assert e.value.code == B.FO_EINVAL
    with pytest.raises(B.FoError) as e:
        B.fo_dropout(x, x, B.dropout_key(0.5, 0))
    assert e.value.code == B.FO_EALIAS
    with pytest.raises(ValueError, match="last dimension"):
        nn.FlashLayerNorm((4, 8))
    with pytest.raises(ValueError, match="expected a last dimension"):
        nn.FlashRMSNorm(8, device="cuda")(x[:, :4])
    x.requires_grad_(True)
    y = nn.rms_norm(x)
    g, = torch.autograd.grad(y, x, torch.ones_like(y).requires_grad_(True), create_graph=True)
    with pytest.raises(RuntimeError, match="second derivatives"):
        (g.sum() + x.sum()).backward()

"""The training-step operators next to the optimizer, as timed workloads.

Four operators work on rows of activations and share one mask generator:

  dropout              y = keep * x / (1 - p), the keep decisions recomputed
                       from a counter wherever they are needed
  layer_norm           y = (x - mean) / sqrt(var + eps) * weight + bias
  rms_norm             y = x / sqrt(mean(x^2) + eps) * weight
  dropout_add_norm     h = residual + dropout(x), rounded to its type;
                       y = layer_norm(h) or rms_norm(h); both are outputs

A "forward" case is one call without gradients (inference).  A "train" case is
the call and its gradients for given output gradients, as one training step
makes them.

With `own` false, run() computes the plain form from elementary torch
operations; with `own` true it calls precision_optimizer_state_amd.nn.

Keep decisions.  An activation tensor is a matrix of R rows and C columns (the
last dimension).  Element (r, c) belongs to block b = r * ceil(C / 8) + c // 8.
W(b, 0) and W(b, 1) are the four 32-bit words of Philox4x32-10 (Salmon, Moraes,
Dror, Shaw: Parallel random numbers: as easy as 1, 2, 3; SC 2011) at counter
(b mod 2^32, b div 2^32 + 2^31 * which, offset mod 2^32, offset div 2^32) under
key (seed mod 2^32, seed div 2^32).  Element c takes half j = c mod 8 of each
(word j // 2, low half first): u = 2^16 * half(W(b, 0)) + half(W(b, 1)).  It is
kept where u >= T, T = round(2^32 * p); kept values are scaled by
1 / (1 - T / 2^32).
"""

import math

import numpy as np
import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "f32": torch.float32}
_SIZE = {"bf16": 2, "fp16": 2, "f32": 4}


def _case(name, op, rows, cols, dtype, mode, norm="", p=0.0, wdtype="", pad=0):
    return {"name": name, "op": op, "norm": norm, "rows": rows, "cols": cols, "dtype": dtype,
            "wdtype": wdtype or dtype, "mode": mode, "p": p, "pad": pad}


def listed():
    return [
        # a short sequence on its way into the first block of a GPT-2-small (width 768)
        _case("dropout_short_sequence", "dropout", 17, 768, "bf16", "train", p=0.1),
        # the embedding dropout of 8 sequences of 1024 tokens
        _case("dropout_embedding", "dropout", 8192, 768, "bf16", "train", p=0.1),
        # attention probabilities: 8 sequences, 12 heads, 1024 x 1024; the largest call
        _case("dropout_attention_map", "dropout", 98304, 1024, "fp16", "train", p=0.1),
        # one token through a layer norm while a text is generated; the smallest call
        _case("layer_norm_one_token", "layer_norm", 1, 768, "bf16", "forward", "layer"),
        # a layer norm of a GPT-2-small training step
        _case("layer_norm_gpt2", "layer_norm", 8192, 768, "bf16", "train", "layer"),
        # single precision, odd sizes, rows that are slices of a wider buffer
        _case("layer_norm_f32_slice", "layer_norm", 1021, 1601, "f32", "train", "layer", pad=7),
        # a handful of sequences generating with a Llama-3.1-8B (width 4096)
        _case("rms_norm_five_tokens", "rms_norm", 5, 4096, "fp16", "forward", "rms"),
        # a norm of a Llama-3.1-8B training step on 8192 tokens
        _case("rms_norm_llama", "rms_norm", 8192, 4096, "bf16", "train", "rms"),
        # queries normalised head by head: 4096 tokens, 32 heads of 128
        _case("rms_norm_heads", "rms_norm", 131072, 128, "bf16", "train", "rms"),
        # the end of a GPT-2-small block: dropout, residual sum, the next block's norm
        _case("dropout_add_norm_gpt2", "dropout_add_norm", 8192, 768, "bf16", "train", "layer", p=0.1),
        # the same place in a Llama-3.1-8B step (which has no dropout)
        _case("dropout_add_norm_llama", "dropout_add_norm", 4096, 4096, "bf16", "train", "rms"),
        # a small single-precision model with odd sizes
        _case("dropout_add_norm_f32_odd", "dropout_add_norm", 129, 1001, "f32", "train", "layer", p=0.25),
    ]


def draw(rng):
    op = rng.choice(["dropout", "layer_norm", "rms_norm", "dropout_add_norm", "dropout_add_norm"])
    budget = 1 << (26 if op == "dropout" else 24)       # elements
    cols = int(round(math.exp(rng.uniform(math.log(1.0), math.log(16384.0)))))
    rows = int(round(math.exp(rng.uniform(0.0, math.log(131072.0)))))
    rows = max(1, min(rows, budget // cols))
    dtype = rng.choice(["bf16", "bf16", "fp16", "f32"])
    norm = {"dropout": "", "layer_norm": "layer", "rms_norm": "rms"}.get(op) if op != "dropout_add_norm" \
        else rng.choice(["layer", "rms"])
    p = 0.0
    if op == "dropout" or (op == "dropout_add_norm" and rng.random() < 0.75):
        p = rng.choice([0.1, 0.5, rng.uniform(0.001, 0.9)])
    case = _case("", op, rows, cols, dtype, rng.choice(["forward", "train", "train"]), norm, p,
                 rng.choice([dtype, "f32"]), rng.choice([0, 0, 8, rng.randrange(1, 64)]))
    del case["name"]
    return case


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rows, cols, dt, wdt = case["rows"], case["cols"], _DT[case["dtype"]], _DT[case["wdtype"]]
    train = case["mode"] == "train"

    def normal(r, c):
        return torch.randn(r, c, generator=gen, device="cuda", dtype=torch.float32)

    # activations: unit spread around a per-channel mean, one channel in 64 far larger
    def activations(pad):
        width = cols + pad
        scale = torch.where(torch.rand(width, generator=gen, device="cuda") < 1 / 64, 12.0, 1.0)
        x = torch.addcmul(0.3 * normal(1, width), normal(rows, width), scale).to(dt)[:, :cols]
        return x.detach()

    # output gradients: heavier tails than a normal distribution's, of a scaled loss
    def gradient():
        return (0.2 * normal(rows, cols) * (0.2 + normal(rows, 1).square())).to(dt)

    st = {"case": case, "x": activations(case["pad"])}
    if case["op"] == "dropout_add_norm":
        st["residual"] = activations(0)
    if case["norm"]:
        st["weight"] = (1.0 + 0.1 * normal(1, cols)[0]).to(wdt)
        st["eps"] = 1e-5 if case["norm"] == "layer" else 1e-6
    if case["norm"] == "layer":
        st["bias"] = (0.1 * normal(1, cols)[0]).to(wdt)
    if train:
        st["dy"] = gradient()
        if case["op"] == "dropout_add_norm":
            st["dh"] = gradient()
        for key in ("x", "residual", "weight", "bias"):
            if key in st:
                st[key].requires_grad_(True)
    st["seed"] = (seed * 0x9E3779B97F4A7C15 + 0x1234567) % (1 << 64)
    st["offset"] = (seed * 11400714819 + 5) % (1 << 40)
    return st


# ---------------------------------------------------------------------------
# plain form
# ---------------------------------------------------------------------------
_LOW = 0xFFFFFFFF


def _plain_words(rows, cols, seed, offset, which):
    """The four 32-bit words of every block, in int64 (products wrap; their bits are right)."""
    blocks = -(-cols // 8)
    b = torch.arange(rows * blocks, dtype=torch.int64, device="cuda")
    c0, c1 = b & _LOW, (b >> 32) + (which << 31)
    c2, c3 = torch.full_like(b, offset & _LOW), torch.full_like(b, (offset >> 32) & _LOW)
    k0, k1 = seed & _LOW, seed >> 32
    for _ in range(10):
        p0, p1 = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = (((p1 >> 32) & _LOW) ^ c1) ^ k0, p1 & _LOW, (((p0 >> 32) & _LOW) ^ c3) ^ k1, p0 & _LOW
        k0, k1 = (k0 + 0x9E3779B9) & _LOW, (k1 + 0xBB67AE85) & _LOW
    return torch.stack((c0, c1, c2, c3), dim=-1).view(rows, blocks, 4)


def _plain_keep(rows, cols, p, seed, offset):
    halves = []
    for which in (0, 1):
        w = _plain_words(rows, cols, seed, offset, which)
        halves.append(torch.stack((w & 0xFFFF, w >> 16), dim=-1).view(rows, -1)[:, :cols])
    return ((halves[0] << 16) | halves[1]) >= round(p * 2.0 ** 32)


def _plain_dropped(v, keep, p):
    threshold = round(p * 2.0 ** 32)
    scale = 2.0 ** 32 / (2.0 ** 32 - threshold)
    return torch.where(keep, v * scale, torch.zeros_like(v))


def _plain(st):
    case = st["case"]
    dt, p, train = _DT[case["dtype"]], case["p"], case["mode"] == "train"
    rows, cols = case["rows"], case["cols"]
    x = st["x"].float()
    keep = _plain_keep(rows, cols, p, st["seed"], st["offset"]) if p else None
    if case["op"] == "dropout":
        out = {"y": _plain_dropped(x, keep, p).to(dt)}
        if train:
            out["dx"] = _plain_dropped(st["dy"].float(), keep, p).to(dt)
        return out
    out = {}
    h = x
    if case["op"] == "dropout_add_norm":
        out["h"] = (st["residual"].float() + (_plain_dropped(x, keep, p) if p else x)).to(dt)
        h = out["h"].float()
    w = st["weight"].float()
    if case["norm"] == "layer":
        centred = h - h.mean(dim=1, keepdim=True)
    else:
        centred = h
    rstd = 1.0 / torch.sqrt((centred * centred).mean(dim=1, keepdim=True) + st["eps"])
    xhat = centred * rstd
    y = xhat * w
    if case["norm"] == "layer":
        y = y + st["bias"].float()
    out["y"] = y.to(dt)
    if train:
        dy = st["dy"].float()
        g = dy * w
        d = g - xhat * (g * xhat).mean(dim=1, keepdim=True)
        if case["norm"] == "layer":
            d = d - g.mean(dim=1, keepdim=True)
        d = d * rstd
        if case["op"] == "dropout_add_norm":
            d = d + st["dh"].float()
            out["dx"] = (_plain_dropped(d, keep, p) if p else d).to(dt)
            out["dresidual"] = d.to(dt)
        else:
            out["dx"] = d.to(dt)
        out["dweight"] = (dy * xhat).sum(dim=0).to(st["weight"].dtype)
        if case["norm"] == "layer":
            out["dbias"] = dy.sum(dim=0).to(st["bias"].dtype)
    return out


def _own(st):
    from precision_optimizer_state_amd import nn
    case, p, train = st["case"], st["case"]["p"], st["case"]["mode"] == "train"
    leaves = [k for k in ("x", "residual", "weight", "bias") if k in st]
    with torch.set_grad_enabled(train):
        if case["op"] == "dropout":
            out = {"y": nn.dropout(st["x"], p, st["seed"], st["offset"])}
        elif case["op"] == "layer_norm":
            out = {"y": nn.layer_norm(st["x"], st["weight"], st["bias"], st["eps"])}
        elif case["op"] == "rms_norm":
            out = {"y": nn.rms_norm(st["x"], st["weight"], st["eps"])}
        elif case["norm"] == "layer":
            h, y = nn.dropout_add_layer_norm(st["x"], st["residual"], st["weight"], st["bias"], st["eps"],
                                             p=p, seed=st["seed"], offset=st["offset"])
            out = {"h": h, "y": y}
        else:
            h, y = nn.dropout_add_rms_norm(st["x"], st["residual"], st["weight"], st["eps"],
                                           p=p, seed=st["seed"], offset=st["offset"])
            out = {"h": h, "y": y}
    if train:
        grads = torch.autograd.grad(list(out.values()), [st[k] for k in leaves],
                                    [st["d" + k] for k in out])
        out = {k: v.detach() for k, v in out.items()}
        out.update(("d" + k, g) for k, g in zip(leaves, grads))
    return out


def run(state):
    if own:
        return _own(state)
    with torch.no_grad():
        return _plain(state)


def work(case):
    n, e, we = case["rows"] * case["cols"], _SIZE[case["dtype"]], _SIZE[case["wdtype"]]
    train = case["mode"] == "train"
    if case["op"] == "dropout":
        return {"bytes": n * e * (4 if train else 2), "flops": n * (2 if train else 1)}
    params = case["cols"] * (2 if case["norm"] == "layer" else 1)
    arrays = {False: 2, True: 4}[train]                 # x, y; dy, dx
    flops = 8 * n + (14 * n if train else 0)
    if case["op"] == "dropout_add_norm":
        arrays += 2 + (2 if train else 0)               # residual, h; dh, dresidual
        if train and not case["p"]:
            arrays -= 1                                 # dx and dresidual are one array
        flops += n * (4 if train else 2)
    return {"bytes": n * e * arrays + params * we * (2 if train else 1), "flops": flops}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def _exact_keep(rows, cols, p, seed, offset):
    """The keep decisions with NumPy's unsigned arithmetic, a range of blocks at a time;
    the second set of words only where the first leaves the decision open."""
    threshold = round(p * 2.0 ** 32)
    per_row = (cols + 7) // 8
    mask32, sh = np.uint64(0xFFFFFFFF), np.uint64(32)

    def generator(index, which):
        ctr = [index & mask32, (index >> sh) | np.uint64(which << 31),
               np.full(index.shape, offset % 2 ** 32, np.uint64), np.full(index.shape, offset // 2 ** 32, np.uint64)]
        for i in range(10):
            ka = np.uint64((seed % 2 ** 32 + i * 0x9E3779B9) % 2 ** 32)
            kb = np.uint64((seed // 2 ** 32 + i * 0xBB67AE85) % 2 ** 32)
            a = ctr[0] * np.uint64(0xD2511F53)
            b = ctr[2] * np.uint64(0xCD9E8D57)
            ctr = [(b >> sh) ^ ctr[1] ^ ka, b & mask32, (a >> sh) ^ ctr[3] ^ kb, a & mask32]
        return np.stack(ctr, axis=1).astype("<u4").view("<u2")          # low half first

    keep = np.empty((rows * per_row, 8), bool)
    step = 1 << 16
    for lo in range(0, rows * per_row, step):
        index = np.arange(lo, min(lo + step, rows * per_row), dtype=np.uint64)
        u = generator(index, 0).astype(np.int64)
        part = u > threshold // 65536
        open_rows = np.nonzero((u == threshold // 65536).any(axis=1))[0]
        if open_rows.size:
            full = u[open_rows] * 65536 + generator(index[open_rows], 1)
            part[open_rows] = full >= threshold
        keep[lo:lo + step] = part
    return torch.from_numpy(keep.reshape(rows, per_row * 8)[:, :cols].copy()).cuda()


def exact(case, seed):
    st = prepare(case, seed)
    dt = _DT[case["dtype"]]
    v = {k: t.detach().double() for k, t in st.items() if torch.is_tensor(t)}
    rows, cols, p = case["rows"], case["cols"], case["p"]
    n = float(cols)
    factor = 1.0
    if p:
        factor = _exact_keep(rows, cols, p, st["seed"], st["offset"]).double()
        factor *= 1.0 / (1.0 - round(p * 2.0 ** 32) / 2.0 ** 32)
    if case["op"] == "dropout":
        res = {"y": v["x"] * factor}
        if "dy" in v:
            res["dx"] = v["dy"] * factor
        return res
    res = {}
    inp = v["x"]
    if "residual" in v:
        res["h"] = v["x"] * factor + v["residual"]
        inp = res["h"].to(dt).double()                  # the norm is that of h as it is handed on
    mu = inp.sum(1, keepdim=True) / n if case["norm"] == "layer" else 0.0
    sigma = ((inp - mu).pow(2).sum(1, keepdim=True) / n + st["eps"]).sqrt()
    unit = (inp - mu) / sigma
    res["y"] = unit * v["weight"] + v.get("bias", 0.0)
    if "dy" in v:
        gw = v["dy"] * v["weight"]
        grad = gw * n - unit * (gw * unit).sum(1, keepdim=True)
        if case["norm"] == "layer":
            grad = grad - gw.sum(1, keepdim=True)
        grad = grad / (n * sigma)
        if "residual" in v:
            grad = grad + v["dh"]
        res["dx"] = grad * factor
        if "residual" in v:
            res["dresidual"] = grad
        res["dweight"] = (v["dy"] * unit).sum(0)
        if case["norm"] == "layer":
            res["dbias"] = v["dy"].sum(0)
    return res

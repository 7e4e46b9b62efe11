"""More operators of the training step around the optimizer, as timed workloads.

  gradient clipping       the norm of a model's gradients taken together, and the
                          gradients scaled down where it passes a bound
  linear_cross_entropy    loss = softmax cross entropy of the logits x W^T against
                          target tokens, and the gradients of x and W, without an
                          array of logits
  gated_linear            y = act(x Wg^T) * (x Wu^T), the first half of a gated
                          feed-forward block, and the gradients of x, Wg and Wu

With `own` false, run() computes the plain form from elementary torch
operations; with `own` true it calls precision_optimizer_state_amd.

Formulas.

  norm     (sum |g|^2)^(1/2) over every element of every tensor, or sum |g|, or
           max |g|.  Clipping multiplies by c = min(1, max_norm / (norm + 1e-6)).
  loss     z = W x for each row x; l = log sum_v exp(z_v);
           loss = l - (1 - s) z_t - (s / V) sum_v z_v  with target t, smoothing s;
           0 for rows whose target is -100.  "mean" divides by the other rows' number.
  dz       (softmax(z) - (1 - s) [v = t] - s / V) * dloss; dx = dz W, dW = dz^T x.
  gated    g = Wg x, u = Wu x, y = act(g) u; dg = dy u act'(g), du = dy act(g);
           dx = dg Wg + du Wu, dWg = dg^T x, dWu = du^T x.
           silu(g) = g / (1 + exp(-g)); gelu(g) = g (1 + erf(g / sqrt 2)) / 2; gelu_tanh(g) =
           g (1 + tanh(k (g + 0.044715 g^3))) / 2 with k = sqrt(2 / pi).
"""

import math
import random

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "f32": torch.float32}
_SIZE = {"bf16": 2, "fp16": 2, "f32": 4}
_IGNORE = -100


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _clip(name, tensors, dtype, mode, norm="2", out="", max_norm=1.0, list_seed=0, largest=0):
    """mode "norm": the norm alone; "in_place": clipping of .grad by a bound that holds, as in most steps of a
    run (the call can be made again on the same gradients); "out": clipped gradients into other tensors."""
    return {"name": name, "op": "clip", "list": tensors, "list_seed": list_seed, "largest": largest, "dtype": dtype,
            "out": out or dtype, "mode": mode, "norm": norm, "max_norm": max_norm}


def _loss(name, rows, cols, vocab, dtype, mode, reduction="mean", smoothing=0.0, ignored=0.0, pad=0):
    return {"name": name, "op": "loss", "rows": rows, "cols": cols, "vocab": vocab, "dtype": dtype, "mode": mode,
            "reduction": reduction, "smoothing": smoothing, "ignored": ignored, "pad": pad}


def _gated(name, rows, cols, features, dtype, mode, act="silu", pad=0):
    return {"name": name, "op": "gated", "rows": rows, "cols": cols, "features": features, "dtype": dtype,
            "mode": mode, "act": act, "pad": pad}


def listed():
    return [
        # a small classifier's six gradients; the smallest call
        _clip("norm_small_model", "mlp", "f32", "norm"),
        # GPT-2-small, 148 tensors, after each backward pass; the bound holds
        _clip("clip_gpt2_within_bound", "gpt2", "bf16", "in_place", max_norm=1000.0),
        # ResNet-50, 161 tensors of a loss-scaled half-precision step: the largest element
        _clip("norm_resnet50_largest", "resnet50", "fp16", "norm", norm="inf"),
        # 8 blocks of a Llama-3.1-8B: gradients summed over micro-batches in single precision,
        # clipped into the 16-bit ones that the optimizer reads
        _clip("clip_llama_accumulated", "llama_blocks", "f32", "out", out="bf16"),
        # the loss of one generated token, GPT-2-small's head
        _loss("loss_one_token", 1, 768, 50257, "bf16", "forward", "none"),
        # 512 tokens scored by a Llama-3.1-8B
        _loss("loss_score_llama", 512, 4096, 128256, "bf16", "forward", "none"),
        # a GPT-2-small training step: 8 sequences of 1024 tokens, the ends of some are padding
        _loss("loss_gpt2", 8192, 768, 50257, "bf16", "train", ignored=0.1),
        # a Llama-3.1-8B training step on 8192 tokens; the largest call
        _loss("loss_llama", 8192, 4096, 128256, "bf16", "train"),
        # half precision with a scaled loss, smoothing, odd sizes, rows that are slices of a wider buffer
        _loss("loss_fp16_odd", 1021, 801, 10007, "fp16", "train", "sum", 0.1, 0.25, pad=7),
        # one token through a Llama-3.1-8B's block while a text is generated
        _gated("gated_one_token", 1, 4096, 14336, "bf16", "forward"),
        # the same block in a training step on 8192 tokens
        _gated("gated_llama", 8192, 4096, 14336, "bf16", "train"),
        # a small single-precision model with odd sizes
        _gated("gated_f32_odd", 333, 521, 1365, "f32", "train", "gelu_tanh"),
    ]


def _log_int(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["clip", "loss", "loss", "gated"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "f32"])
    if op == "clip":
        mode = rng.choice(["norm", "in_place", "out"])
        case = _clip("", "drawn", dtype, mode, rng.choice(["2", "2", "2", "1", "inf"]),
                     rng.choice([dtype, "bf16", "fp16"]) if mode == "out" else dtype,
                     1e12 if mode == "in_place" else rng.choice([1.0, 0.1, rng.uniform(0.01, 10.0)]),
                     rng.randrange(1 << 30), _log_int(rng, 1, 1 << 26))
    elif op == "loss":
        cols, vocab, rows = _log_int(rng, 1, 4096), _log_int(rng, 1, 131072), _log_int(rng, 1, 8192)
        if rng.random() < 0.5:
            cols = -(-cols // 64) * 64
        rows = max(1, min(rows, (1 << 40) // (cols * vocab * (4 if dtype == "f32" else 1))))
        case = _loss("", rows, cols, vocab, dtype, rng.choice(["forward", "train", "train"]),
                     rng.choice(["mean", "sum", "none"]), rng.choice([0.0, 0.0, 0.1, rng.uniform(0.01, 0.5)]),
                     rng.choice([0.0, 0.0, 0.1, 0.5]), rng.choice([0, 0, 8, rng.randrange(1, 64)]))
    else:
        cols, features, rows = _log_int(rng, 1, 4096), _log_int(rng, 1, 14336), _log_int(rng, 1, 8192)
        if rng.random() < 0.5:
            cols, features = -(-cols // 64) * 64, -(-features // 64) * 64
        rows = max(1, min(rows, (1 << 38) // (cols * features * (4 if dtype == "f32" else 1))))
        case = _gated("", rows, cols, features, dtype, rng.choice(["forward", "train", "train"]),
                      rng.choice(["silu", "silu", "gelu", "gelu_tanh"]), rng.choice([0, 0, 8, rng.randrange(1, 64)]))
    del case["name"]
    return case


def _shapes(case):
    """The shapes of a list of gradients."""
    kind = case["list"]
    if kind == "mlp":
        return [(256, 784), (256,), (256, 256), (256,), (10, 256), (10,)]
    if kind == "gpt2":
        d, v, ctx, layers = 768, 50257, 1024, 12
        block = [(d,), (d,), (d, 3 * d), (3 * d,), (d, d), (d,), (d,), (d,), (d, 4 * d), (4 * d,), (4 * d, d), (d,)]
        return [(v, d), (ctx, d)] + block * layers + [(d,), (d,)]
    if kind == "llama_blocks":
        d, ff, kv, layers = 4096, 14336, 1024, 8
        return [(d, d), (kv, d), (kv, d), (d, d), (ff, d), (ff, d), (d, ff), (d,), (d,)] * layers
    if kind == "resnet50":
        out, cin = [(64, 3, 7, 7), (64,), (64,)], 64
        for blocks, width in zip([3, 4, 6, 3], [64, 128, 256, 512]):
            for b in range(blocks):
                for shape in ((width, cin, 1, 1), (width, width, 3, 3), (4 * width, width, 1, 1)):
                    out += [shape, (shape[0],), (shape[0],)]
                if b == 0:
                    out += [(4 * width, cin, 1, 1), (4 * width,), (4 * width,)]
                cin = 4 * width
        return out + [(1000, 2048), (1000,)]
    rng = random.Random(case["list_seed"])
    shapes, left = [], 1 << 28                          # elements in all
    for _ in range(_log_int(rng, 1, 400)):
        n = min(left, _log_int(rng, 1, case["largest"]))
        if n:
            shapes.append((n,))
        left -= n
    return shapes


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32)

    # rows as a norm leaves them: unit spread, one channel in 64 far larger; `pad`: slices of a wider buffer
    def activations(rows, cols, dt, pad):
        scale = torch.where(torch.rand(cols + pad, generator=gen, device="cuda") < 1 / 64, 6.0, 1.0)
        return (normal(rows, cols + pad) * scale).to(dt)

    st, dt = {"case": case}, _DT[case["dtype"]]
    if case["op"] == "clip":
        # heavier tails than a normal distribution's; a loss scale on half-precision gradients;
        # a model's gradients lie one after another in one buffer, as buckets of them do
        unit, shapes = 1.0 if case["dtype"] == "fp16" else 1e-3, _shapes(case)
        counts = [math.prod(s) for s in shapes]

        def views(flat):
            return [v.view(s) for v, s in zip(flat.split(counts), shapes)]

        st["flat"] = torch.empty(sum(counts), dtype=dt, device="cuda")
        st["grads"] = views(st["flat"])
        for g in st["grads"]:
            f = normal(*g.shape)
            g.copy_(f.mul_(f.square().add_(0.2)).mul_(unit))
        if case["mode"] == "in_place":
            st["params"] = [torch.empty_like(g).requires_grad_(True) for g in st["grads"]]
            for p, g in zip(st["params"], st["grads"]):
                p.grad = g
        if case["mode"] == "out":
            st["flat"] = torch.empty(sum(counts), dtype=_DT[case["out"]], device="cuda")
            st["out"] = views(st["flat"])
        return st

    rows, cols, train = case["rows"], case["cols"], case["mode"] == "train"
    x = activations(rows, cols, dt, case["pad"])
    if case["op"] == "loss":
        vocab = case["vocab"]
        st["weight"] = (0.02 * normal(vocab, cols)).to(dt)
        target = torch.randint(vocab, (rows,), generator=gen, device="cuda")
        # a trained model is sure of some of its tokens: the target's logit is raised by 0 to 12
        pick = st["weight"][target].float()
        boost = 12.0 * torch.rand(rows, 1, generator=gen, device="cuda")
        x[:, :cols] += (boost * pick / (pick.square().sum(1, keepdim=True) + 0.05)).to(dt)
        lost = torch.rand(rows, generator=gen, device="cuda") < case["ignored"]
        st["target"] = torch.where(lost, _IGNORE, target)
        if train:
            # the loss's own gradient: a loss scale in half precision, a weight per row for "none"
            st["dloss"] = (0.5 + torch.rand(rows, generator=gen, device="cuda")) if case["reduction"] == "none" \
                else torch.ones((), device="cuda")
            if case["dtype"] == "fp16":
                st["dloss"] = st["dloss"] * (1024.0 if case["reduction"] == "mean" else 8.0)
        leaves = ("x", "weight")
    else:
        features = case["features"]
        st["gate"] = (0.02 * normal(features, cols)).to(dt)
        st["up"] = (0.02 * normal(features, cols)).to(dt)
        if train:
            st["dy"] = (0.2 * normal(rows, features) * (0.2 + normal(rows, 1).square())).to(dt)
        leaves = ("x", "gate", "up")
    st["x"] = x[:, :cols].detach()
    if train:
        for key in leaves:
            st[key].requires_grad_(True)
    return st


# ---------------------------------------------------------------------------
# plain form
# ---------------------------------------------------------------------------
def _plain_norm(grads, kind):
    if kind == "inf":
        return torch.stack([g.float().abs().max() for g in grads]).max().double()
    if kind == "1":
        return torch.stack([g.float().abs().sum(dtype=torch.float64) for g in grads]).sum()
    return torch.stack([g.float().square().sum(dtype=torch.float64) for g in grads]).sum().sqrt()


def _plain_clip(st):
    case = st["case"]
    norm = _plain_norm(st["grads"], case["norm"])
    if case["mode"] == "norm":
        return {"norm": norm.float()}
    c = (case["max_norm"] / (norm + 1e-6)).clamp(max=1.0).float()
    out = st["grads"] if case["mode"] == "in_place" else st["out"]
    [o.copy_(g.float() * c) for o, g in zip(out, st["grads"])]
    return {"norm": norm.float(), "grads": st["flat"]}


def _plain_loss(st):
    case = st["case"]
    s, vocab, dt = case["smoothing"], case["vocab"], _DT[case["dtype"]]
    x, weight, target = st["x"].float(), st["weight"].float(), st["target"]
    logits = torch.matmul(x, weight.t())
    valid = target != _IGNORE
    index = torch.where(valid, target, 0)[:, None]
    top = logits.max(dim=1, keepdim=True).values
    probs = torch.exp(logits - top)
    total = probs.sum(dim=1, keepdim=True)
    loss = (top + torch.log(total))[:, 0] - (1.0 - s) * logits.gather(1, index)[:, 0]
    if s:
        loss = loss - s * logits.mean(dim=1)
    loss = torch.where(valid, loss, 0.0)
    count = valid.sum().float()
    out = {"none": loss, "sum": loss.sum(), "mean": loss.sum() / count}[case["reduction"]]
    if case["mode"] != "train":
        return {"loss": out}
    scale = torch.where(valid, st["dloss"] / count if case["reduction"] == "mean" else st["dloss"], 0.0)
    dlogits = probs / total
    dlogits.scatter_add_(1, index, torch.full_like(index, s - 1.0, dtype=torch.float32))
    dlogits = (dlogits - s / vocab) * scale[:, None]
    return {"loss": out, "dx": torch.matmul(dlogits, weight).to(dt), "dweight": torch.matmul(dlogits.t(), x).to(dt)}


def _plain_gated(st):
    case = st["case"]
    dt = _DT[case["dtype"]]
    x, wg, wu = st["x"].float(), st["gate"].float(), st["up"].float()
    g, u = torch.matmul(x, wg.t()), torch.matmul(x, wu.t())
    if case["act"] == "silu":
        sig = 1.0 / (1.0 + torch.exp(-g))
        act, slope = g * sig, sig * (1.0 + g * (1.0 - sig))
    elif case["act"] == "gelu":
        cdf = 0.5 * (1.0 + torch.erf(g * math.sqrt(0.5)))
        act, slope = g * cdf, cdf + g * torch.exp(-0.5 * g * g) * math.sqrt(0.5 / math.pi)
    else:
        k = math.sqrt(2.0 / math.pi)
        th = torch.tanh(k * (g + 0.044715 * g * g * g))
        act = 0.5 * g * (1.0 + th)
        slope = 0.5 * (1.0 + th) + 0.5 * g * (1.0 - th * th) * k * (1.0 + 3.0 * 0.044715 * g * g)
    y = (act * u).to(dt)
    if case["mode"] != "train":
        return {"y": y}
    dy = st["dy"].float()
    dg, du = dy * u * slope, dy * act
    return {"y": y, "dx": (torch.matmul(dg, wg) + torch.matmul(du, wu)).to(dt),
            "dgate": torch.matmul(dg.t(), x).to(dt), "dup": torch.matmul(du.t(), x).to(dt)}


def _own(st):
    case = st["case"]
    if case["op"] == "clip":
        from precision_optimizer_state_amd import grads
        kind = float(case["norm"])
        if case["mode"] == "norm":
            return {"norm": grads.grad_norm(st["grads"], kind)}
        if case["mode"] == "in_place":
            norm = grads.clip_grad_norm_(st["params"], case["max_norm"], kind)
        else:
            _, norm = grads.clip_grads(st["grads"], case["max_norm"], kind, out=st["out"])
        return {"norm": norm, "grads": st["flat"]}
    from precision_optimizer_state_amd import nn
    train = case["mode"] == "train"
    with torch.set_grad_enabled(train):
        if case["op"] == "loss":
            key, leaves = "loss", ("x", "weight")
            y = nn.linear_cross_entropy(st["x"], st["weight"], st["target"], ignore_index=_IGNORE,
                                        reduction=case["reduction"], label_smoothing=case["smoothing"])
        else:
            key, leaves = "y", ("x", "gate", "up")
            y = nn.gated_linear(st["x"], st["gate"], st["up"], activation=case["act"])
    out = {key: y.detach()}
    if train:
        grads = torch.autograd.grad(y, [st[k] for k in leaves], st["d" + key])
        out.update(("d" + k, g) for k, g in zip(leaves, grads))
    return out


def run(state):
    if own:
        return _own(state)
    with torch.no_grad():
        return {"clip": _plain_clip, "loss": _plain_loss, "gated": _plain_gated}[state["case"]["op"]](state)


def work(case):
    e = _SIZE[case["dtype"]]
    if case["op"] == "clip":
        n = sum(math.prod(s) for s in _shapes(case))
        written = 0 if case["mode"] != "out" else _SIZE[case["out"]]       # a bound that holds changes nothing
        return {"bytes": n * (e + written), "flops": n * (2 if case["mode"] != "out" else 3)}
    rows, cols, train = case["rows"], case["cols"], case["mode"] == "train"
    if case["op"] == "loss":
        product, weights = 2 * rows * cols * case["vocab"], case["vocab"] * cols
        row_bytes = 8 + (4 if case["reduction"] == "none" else 0) * (2 if train else 1)
        return {"bytes": (rows * cols + weights) * e * (2 if train else 1) + rows * row_bytes,
                "flops": product * (3 if train else 1)}
    product, weights, mid = 4 * rows * cols * case["features"], 2 * case["features"] * cols, rows * case["features"]
    return {"bytes": ((rows * cols + weights) * (2 if train else 1) + mid * (2 if train else 1)) * e,
            "flops": product * (3 if train else 1)}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------
def _exact_clip(case, st):
    p = float(case["norm"])
    flat = [g.reshape(-1) for g in st["grads"]]
    if p == math.inf:
        norm = max(float(t.abs().max()) for t in flat)
    else:
        norm = math.fsum(float(t.double().abs().pow(p).sum()) for t in flat) ** (1.0 / p)
    norm_out = torch.tensor(norm, dtype=torch.float64, device="cuda")
    if case["mode"] == "norm":
        return {"norm": norm_out}
    factor = min(1.0, case["max_norm"] / (norm + 1e-6))
    return {"norm": norm_out, "grads": torch.cat(flat).double() * factor}


def _exact_loss(case, st):
    """Row by row through log-probabilities, a few rows at a time."""
    rows, cols, vocab, s = case["rows"], case["cols"], case["vocab"], case["smoothing"]
    w = st["weight"].detach().double()
    labels = st["target"].cpu()
    counted = int((labels != _IGNORE).sum())
    losses = torch.zeros(rows, dtype=torch.float64, device="cuda")
    train = case["mode"] == "train"
    dx = torch.zeros(rows, cols, dtype=torch.float64, device="cuda")
    dw = torch.zeros(vocab, cols, dtype=torch.float64, device="cuda") if train else None
    step = max(1, (1 << 28) // vocab)
    for lo in range(0, rows, step):
        mine = torch.nonzero(labels[lo:lo + step] != _IGNORE)[:, 0].cuda() + lo
        if mine.numel() == 0:
            continue
        xs = st["x"].detach()[mine].double()
        wanted = torch.full((mine.numel(), vocab), s / vocab, dtype=torch.float64, device="cuda")
        wanted[torch.arange(mine.numel(), device="cuda"), st["target"][mine]] += 1.0 - s
        logp = xs @ w.T
        logp -= torch.logsumexp(logp, dim=1, keepdim=True)
        losses[mine] = -(wanted * logp).sum(1)
        if train:
            dz = logp.exp_().sub_(wanted)
            if case["reduction"] == "none":
                dz *= st["dloss"][mine].double()[:, None]
            else:
                dz *= float(st["dloss"]) / (counted if case["reduction"] == "mean" else 1)
            dx[mine] = dz @ w
            dw += dz.T @ xs
    if case["reduction"] != "none":
        losses = losses.sum()
    if case["reduction"] == "mean":
        losses = losses / counted if counted else losses / 0.0
    return {"loss": losses, "dx": dx, "dweight": dw} if train else {"loss": losses}


def _exact_gated(case, st):
    """The product by torch's double arithmetic; slopes by the quotient and chain rules written out."""
    x, wg, wu = (st[k].detach().double() for k in ("x", "gate", "up"))
    g, u = x @ wg.T, x @ wu.T
    if case["act"] == "silu":
        e = torch.exp(-g)
        act, slope = g / (1 + e), (1 + e + g * e) / (1 + e) ** 2
    elif case["act"] == "gelu":
        act = g * 0.5 * torch.erfc(-g / math.sqrt(2.0))
        slope = 0.5 * torch.erfc(-g / math.sqrt(2.0)) + g * torch.exp(-g.pow(2) / 2) / math.sqrt(2 * math.pi)
    else:
        # (1 + tanh a) / 2 = 1 / (1 + exp(-2a))
        a2 = 2 * math.sqrt(2 / math.pi) * (g + 0.044715 * g.pow(3))
        half = 1 / (1 + torch.exp(-a2))
        act = g * half
        slope = half + g * half * (1 - half) * 2 * math.sqrt(2 / math.pi) * (1 + 0.134145 * g.pow(2))
    res = {"y": act * u}
    if case["mode"] == "train":
        dy = st["dy"].double()
        dact = dy * u * slope
        dup = dy * act
        res["dx"] = dact @ wg + dup @ wu
        res["dgate"] = dact.T @ x
        res["dup"] = dup.T @ x
    return res


def exact(case, seed):
    st = prepare(case, seed)
    return {"clip": _exact_clip, "loss": _exact_loss, "gated": _exact_gated}[case["op"]](case, st)

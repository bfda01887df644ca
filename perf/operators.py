"""Measured cases of the training operators: the vocabulary cross entropy with
its gradient, the router's gradient with its balance and z losses, and the
global gradient norm with clipping.

Where ``own`` is false ``run`` computes them in their plain form (elementary
torch operations in 32 bits, rounded once at the end); where it is true it
makes the calls a user makes of this package.  Both take what ``prepare`` gives.
"""
import math
import random

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
IGNORE = -100


# ---------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------
def _ce(name, mode, T, H, V, dtype="bf16", reduction="mean", ignored=0.0, pad=0):
    c = dict(op="ce", mode=mode, T=T, H=H, V=V, dtype=dtype, reduction=reduction,
             ignored=ignored, pad=pad)
    if name:
        c["name"] = name
    return c


def _router(name, T, H, E, k, norm, gate, dtype="bf16", balance=0.01, z=0.001):
    c = dict(op="router", T=T, H=H, E=E, k=k, norm=norm, gate=gate, dtype=dtype, balance=balance,
             z=z)
    if name:
        c["name"] = name
    return c


def _clip(name, kind, n, total, bf16, clips, layout=0):
    c = dict(op="clip", kind=kind, n=n, total=total, bf16=bf16, clips=clips, layout=layout)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # the log-probability of one sampled token
        _ce("ce-score-T1", "score", 1, 2048, 50257, reduction="none"),
        # a batch scored for its perplexity: no gradient
        _ce("ce-score-T2048", "score", 2048, 4096, 128000, reduction="none"),
        # one training step's loss of a model with a large vocabulary
        _ce("ce-train-T4096", "train", 4096, 2048, 131072),
        # the widest layer of the workloads, a packed batch with some padding
        _ce("ce-train-T8192", "train", 8192, 7168, 65536, ignored=0.05),
        # fine-tuning: half the tokens are prompt and not learned, each token
        # with a weight of its own; odd sizes
        _ce("ce-train-odd", "train", 777, 2816, 50257, reduction="none", ignored=0.5, pad=8),
        # fp32 training of a small model
        _ce("ce-train-f32", "train", 1000, 1024, 32001, dtype="f32", reduction="sum", ignored=0.1),
        # a micro batch through the 60-expert router with its shared gate
        _router("router-T64", 64, 3584, 60, 4, False, True),
        # the 128-expert prefill shape, weights renormalised
        _router("router-T4096", 4096, 2048, 128, 8, True, False),
        # the 256-expert shape, full softmax
        _router("router-T8192", 8192, 7168, 256, 8, False, False),
        # the gradients of a tiny fp32 layer with its norms and biases
        _clip("clip-tiny", "ragged", 48, 800_000, 0.0, True, layout=3),
        # one layer of 128 experts in bf16: three large tensors, router, norm
        _clip("clip-layer", "layer", 5, 0, 1.0, True),
        # a whole model's list: many tensors of all sizes, both types, at any
        # element offset of two flat buffers
        _clip("clip-model", "ragged", 1500, 200_000_000, 0.6, True, layout=1),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    pick = rng.random()
    if pick < 0.55:
        mode = rng.choice(["score", "train", "train"])
        dtype = "f32" if rng.random() < 0.2 else "bf16"
        T = _log_int(rng, 1, 8192)
        H = 8 * _log_int(rng, 32, 512)
        V = _log_int(rng, 1000, 131072)
        if dtype == "f32":
            T, H, V = min(T, 2048), min(H, 2048), min(V, 50000)
        return _ce(None, mode, T, H, V, dtype=dtype,
                   reduction=rng.choice(["none", "sum", "mean"]),
                   ignored=rng.choice([0.0, 0.1, 0.5, 0.9]), pad=rng.choice([0, 0, 8, 24]))
    if pick < 0.8:
        E = rng.choice([8, 16, 60, 61, 64, 128, 160, 256, 384])
        return _router(None, _log_int(rng, 1, 8192), 8 * _log_int(rng, 32, 896), E,
                       rng.randint(1, 8), rng.random() < 0.5, rng.random() < 0.3,
                       dtype="f32" if rng.random() < 0.2 else "bf16",
                       balance=rng.choice([0.0, 0.01, 0.1]), z=rng.choice([0.0, 0.001]))
    n = _log_int(rng, 1, 2000)
    return _clip(None, "ragged", n, max(n, _log_int(rng, 1000, 300_000_000)),
                 rng.choice([0.0, 0.5, 1.0]), rng.random() < 0.7, layout=rng.randint(0, 10**6))


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _gen(seed, k):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + k)
    return g


def _randn(shape, g, dtype=torch.float32, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=dtype) * std).to(dtype)


def _rows(T, ignored):
    """Tokens that count."""
    return T - int(T * ignored)


def _prepare_ce(c, seed):
    T, H, V, dt = c["T"], c["H"], c["V"], DT[c["dtype"]]
    w = _randn((V, H), _gen(seed, 1), dt, 1.0 / math.sqrt(H))
    # frequent tokens are the low ids, as in a frequency-ordered vocabulary
    u = torch.rand((T,), generator=_gen(seed, 2), device="cuda", dtype=torch.float64)
    target = (torch.exp(u * math.log(V + 1.0)) - 1.0).long().clamp_(0, V - 1).to(torch.int32)
    # hidden rows of unit variance that lean towards their target's row, so
    # the probabilities run from the uninformed to the nearly certain
    lean = 8.0 * torch.rand((T, 1), generator=_gen(seed, 4), device="cuda")
    x = (_randn((T, H), _gen(seed, 3)) + lean * w[target.long()].float()).to(dt)
    if c["pad"]:   # rows of a wider buffer
        wide = torch.zeros((T, H + c["pad"]), device="cuda", dtype=dt)
        wide[:, :H] = x
        x = wide[:, :H]
    skip = T - _rows(T, c["ignored"])
    if skip:
        order = torch.randperm(T, generator=_gen(seed, 5), device="cuda")
        target[order[:skip]] = IGNORE
    s = dict(case=c, x=x, w=w, target=target)
    if c["mode"] == "train":
        s["dloss"] = (torch.rand((T,), generator=_gen(seed, 6), device="cuda") + 0.5) / T \
            if c["reduction"] == "none" else None
    if own:
        import mixture_experts_ffn_04_gb300 as m
        s["op"] = m.LinearCrossEntropy(T, H, V, dtype=dt, reduction=c["reduction"],
                                       ignore_index=IGNORE)
    return s


def _prepare_router(c, seed):
    T, H, E, k, dt = c["T"], c["H"], c["E"], c["k"], DT[c["dtype"]]
    rows = E + int(c["gate"])
    x = _randn((T, H), _gen(seed, 1), dt)
    w = _randn((rows, H), _gen(seed, 2), dt, 0.02)
    logits = x.float() @ w[:E].float().t()
    s = dict(case=c, x=x, w=w, idx=logits.topk(k, dim=1).indices.to(torch.int32).contiguous(),
             d_w=_randn((T, k), _gen(seed, 3), std=0.1),
             d_gate=_randn((T,), _gen(seed, 4), std=0.1) if c["gate"] else None,
             dx_experts=_randn((T, H), _gen(seed, 5), dt, 0.1))
    if own:
        import mixture_experts_ffn_04_gb300 as m
        s["op"] = m.RouterGrad(T, H, E, k, norm_topk=c["norm"], shared_gate=c["gate"], dtype=dt,
                               balance_coef=c["balance"], z_coef=c["z"])
    return s


def _clip_sizes(c):
    """Numbers of elements and types of the list's tensors."""
    if c["kind"] == "layer":
        big = 128 * 768 * 2048
        return [(128 * 2048, "bf16"), (big, "bf16"), (big, "bf16"), (big, "bf16"), (2048, "bf16")]
    rng = random.Random(c["layout"])
    part = [math.exp(rng.uniform(0.0, 9.0)) for _ in range(c["n"])]
    scale = c["total"] / sum(part)
    return [(max(1, int(p * scale)), "bf16" if rng.random() < c["bf16"] else "f32") for p in part]


def _prepare_clip(c, seed):
    sizes = _clip_sizes(c)
    need = {"f32": 0, "bf16": 0}
    for n, t in sizes:
        need[t] += n
    # gradients live in one flat buffer for each type
    flat = {t: _randn((n,), _gen(seed, i), DT[t], 1e-3) for i, (t, n) in enumerate(need.items()) if n}
    out = {t: torch.zeros_like(v) for t, v in flat.items()}
    at = {t: 0 for t in flat}
    grads, outs = [], []
    for n, t in sizes:
        grads.append(flat[t][at[t]: at[t] + n])
        outs.append(out[t][at[t]: at[t] + n])
        at[t] += n
    norm = 1e-3 * math.sqrt(sum(need.values()))
    s = dict(case=c, grads=grads, outs=outs, flat_out=[out[t] for t in sorted(out)],
             max_norm=norm * (0.3 if c["clips"] else 3.0))
    if own:
        import mixture_experts_ffn_04_gb300 as m
        s["op"] = m.GradClip(grads, out=outs)
    return s


def prepare(case, seed):
    return {"ce": _prepare_ce, "router": _prepare_router, "clip": _prepare_clip}[case["op"]](case, seed)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _run_ce(s):
    c, x, w, target = s["case"], s["x"], s["w"], s["target"]
    if own:
        loss = s["op"].forward(x, w, target)
        if c["mode"] == "score":
            return [loss, s["op"].lse]
        dx, dw = s["op"].backward(x, w, target, s["dloss"])
        return [loss, dx, dw]
    T, dt = c["T"], DT[c["dtype"]]
    row = (target != IGNORE).nonzero().flatten()
    t = target[row].long()
    xf, wf = x[row].float(), w.float()
    z = xf @ wf.t()
    top = z.amax(dim=1, keepdim=True)
    zt = z.gather(1, t[:, None])[:, 0]
    z -= top
    z.exp_()
    total = z.sum(dim=1, keepdim=True)
    each = (total.log() + top)[:, 0]
    lse = torch.zeros(T, device=x.device)
    lse[row] = each
    each = each - zt
    count = max(row.numel(), 1)
    if c["reduction"] == "none":
        loss = torch.zeros(T, device=x.device)
        loss[row] = each
    else:
        loss = each.sum(dtype=torch.float64)
        loss = (loss / count if c["reduction"] == "mean" else loss).float().reshape(1)
    if c["mode"] == "score":
        return [loss, lse]
    if c["reduction"] == "none":
        g = s["dloss"][row]
    else:
        g = torch.full_like(each, 1.0 / count if c["reduction"] == "mean" else 1.0)
    z *= g[:, None] / total
    z[torch.arange(row.numel(), device=x.device), t] -= g
    dx = torch.zeros((T, c["H"]), device=x.device, dtype=dt)
    dx[row] = (z @ wf).to(dt)
    dw = (z.t() @ xf).to(dt)
    return [loss, dx, dw]


def _run_router(s):
    c, x, w, idx, d_w = s["case"], s["x"], s["w"], s["idx"], s["d_w"]
    if own:
        dx, dw, aux = s["op"].backward(x, w, idx, d_w, d_gate=s["d_gate"], dx_add=s["dx_experts"])
        return [dx, dw, aux]
    T, E, k, dt = c["T"], c["E"], c["k"], DT[c["dtype"]]
    xf, wf = x.float(), w.float()
    z = xf @ wf.t()
    ze, at = z[:, :E], idx.long()
    top = ze.amax(dim=1, keepdim=True)
    e = (ze - top).exp()
    total = e.sum(dim=1, keepdim=True)
    p = e / total
    lse = (total.log() + top)[:, 0]
    dz = torch.zeros_like(z)
    if c["norm"]:
        sel = e.gather(1, at)
        pw = sel / sel.sum(dim=1, keepdim=True)
        dz.scatter_add_(1, at, pw * (d_w - (pw * d_w).sum(dim=1, keepdim=True)))
    else:
        pw = p.gather(1, at)
        dz.scatter_add_(1, at, pw * d_w)
        dz[:, :E] -= p * (pw * d_w).sum(dim=1, keepdim=True)
    n = torch.zeros(E, device=x.device).index_add_(0, at.flatten(), torch.ones(T * k, device=x.device))
    pn = (p * n).sum(dim=1, keepdim=True)
    dz[:, :E] += (c["balance"] * E / (T * float(T) * k)) * p * (n - pn)
    dz[:, :E] += (2.0 * c["z"] / T) * lse[:, None] * p
    if c["gate"]:
        sg = 1.0 / (1.0 + (-z[:, E]).exp())
        dz[:, E] = s["d_gate"] * sg * (1.0 - sg)
    balance = c["balance"] * E / (T * float(T) * k) * pn.sum(dtype=torch.float64)
    zloss = c["z"] * lse.double().square().mean()
    dx = (s["dx_experts"].float() + dz @ wf).to(dt)
    return [dx, (dz.t() @ xf).to(dt), torch.stack([balance, zloss]).float()]


def _run_clip(s):
    if own:
        return [s["op"].clip(s["max_norm"])] + s["flat_out"]
    total = torch.zeros((), device="cuda", dtype=torch.float64)
    for g in s["grads"]:
        total += g.float().square().sum(dtype=torch.float64)
    norm = total.sqrt()
    coef = (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0).float()
    coef = torch.where(norm.isfinite(), coef, torch.ones_like(coef))
    for g, o in zip(s["grads"], s["outs"]):
        o.copy_(g.float() * coef)
    return [norm.float().reshape(1)] + s["flat_out"]


def run(state):
    return {"ce": _run_ce, "router": _run_router, "clip": _run_clip}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def work(c):
    size = {"bf16": 2, "f32": 4}
    if c["op"] == "ce":
        n, b = _rows(c["T"], c["ignored"]), size[c["dtype"]]
        data = b * c["H"] * (n + c["V"]) + 4 * c["T"]
        flops = 2 * n * c["H"] * c["V"]
        if c["mode"] == "score":
            return dict(bytes=data + 8 * c["T"], flops=flops)
        return dict(bytes=data + b * c["H"] * (c["T"] + c["V"]) + 4, flops=3 * flops)
    if c["op"] == "router":
        b, rows = size[c["dtype"]], c["E"] + int(c["gate"])
        return dict(bytes=b * c["H"] * (3 * c["T"] + 2 * rows) + 8 * c["T"] * c["k"],
                    flops=6 * c["T"] * c["H"] * rows)
    sizes = _clip_sizes(c)
    # the norm needs every gradient before the first can be scaled; a list
    # that fits on the chip need not be read a second time
    return dict(bytes=sum(2 * n * size[t] for n, t in sizes), flops=sum(3 * n for n, _ in sizes))


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "ce":
        if float(c["T"]) * c["H"] * c["V"] > 1.3e12:
            return None
        train = c["mode"] == "train"
        x = s["x"].double().requires_grad_(train)
        w = s["w"].double().requires_grad_(train)
        t = s["target"].long()
        z = x @ w.t()
        loss = torch.nn.functional.cross_entropy(z, t, ignore_index=IGNORE,
                                                 reduction=c["reduction"])
        if not train:
            return [loss.reshape(-1), torch.logsumexp(z, 1).masked_fill(t == IGNORE, 0.0)]
        up = s["dloss"].double() if c["reduction"] == "none" else None
        dx, dw = torch.autograd.grad(loss, [x, w], up)
        return [loss.detach().reshape(-1), dx, dw]
    if c["op"] == "router":
        x = s["x"].double().requires_grad_(True)
        w = s["w"].double().requires_grad_(True)
        z = x @ w.t()
        ze, at, E, T, k = z[:, : c["E"]], s["idx"].long(), c["E"], c["T"], c["k"]
        p = torch.softmax(ze, 1)
        weights = torch.softmax(ze.gather(1, at), 1) if c["norm"] else p.gather(1, at)
        share = torch.bincount(at.flatten(), minlength=E).double() / (T * k)
        balance = c["balance"] * E * (share * p.mean(0)).sum()
        zloss = c["z"] * torch.logsumexp(ze, 1).square().mean()
        obj = (weights * s["d_w"].double()).sum() + balance + zloss
        if c["gate"]:
            obj = obj + (torch.sigmoid(z[:, E]) * s["d_gate"].double()).sum()
        dx, dw = torch.autograd.grad(obj, [x, w])
        return [dx + s["dx_experts"].double(), dw, torch.stack([balance, zloss]).detach()]
    norm = torch.stack([torch.linalg.vector_norm(g.double()) for g in s["grads"]])
    norm = torch.linalg.vector_norm(norm)
    coef = min(1.0, s["max_norm"] / (float(norm) + 1e-6))
    flat = {}
    for g in s["grads"]:
        flat.setdefault("bf16" if g.dtype == torch.bfloat16 else "f32", []).append(g)
    return [norm.reshape(1)] + [torch.cat(flat[t]).double() * coef for t in sorted(flat)]

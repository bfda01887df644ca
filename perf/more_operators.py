"""Measured cases of the operators of a training step around the layer: the
token embedding with its gradient, the norms before and after a block with its
gate and residual, and the orthogonalised update of weight matrices.

Where ``own`` is false ``run`` computes them in their plain form (elementary
torch operations in 32 bits, rounded once at the end); where it is true it
makes the calls a user makes of this package.  Both take what ``prepare`` gives.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EPS_NORM = 1e-6                       # of the block norms
EPS_ORTH = 1e-7                       # added to the Frobenius norm
COEFS = (3.4445, -4.7750, 2.0315)     # a x + b x^3 + c x^5, applied STEPS times
STEPS = 5
LR, BETA, DECAY = 0.02, 0.95, 0.1


# ---------------------------------------------------------------------------
# the cases
# ---------------------------------------------------------------------------
def _emb(name, mode, T, H, V, dtype="bf16", scale=1.0, pad=False, add=False):
    c = dict(op="emb", mode=mode, T=T, H=H, V=V, dtype=dtype, scale=scale, pad=pad, add=add)
    if name:
        c["name"] = name
    return c


def _norm(name, mode, T, H, dtype="bf16", gate="none", pre=True, post=True, offset=False,
          residual=1.0):
    c = dict(op="norm", mode=mode, T=T, H=H, dtype=dtype, gate=gate, pre=pre, post=post,
             offset=offset, residual=residual)
    if name:
        c["name"] = name
    return c


def _muon(name, batch, rows, cols, dtype="bf16", kind="layer", nesterov=True):
    """kind "layer": gate, up [batch, rows, cols] and down [batch, cols, rows] of one layer's
    experts; "one": a single [batch, rows, cols] parameter; "direction": only the
    orthogonalised matrices."""
    c = dict(op="muon", kind=kind, batch=batch, rows=rows, cols=cols, dtype=dtype,
             nesterov=nesterov)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # the embedding of the one token just sampled
        _emb("emb-lookup-T1", "lookup", 1, 2048, 50257),
        # the embedding of a prefill at the widest layer, scaled by sqrt(H)
        _emb("emb-lookup-T8192", "lookup", 8192, 7168, 65536, scale=math.sqrt(7168.0)),
        # a training step's lookup and gradient, added to the gradient of the
        # classifier that shares the table
        _emb("emb-train-tied-T4096", "train", 4096, 2048, 131072, add=True),
        # packed batches of a small fp32 model with padding tokens, odd sizes
        _emb("emb-train-f32-odd", "train", 60001, 1000, 32001, dtype="f32", pad=True),
        # one token between two sublayers: both norms and the residual
        _norm("norm-decode-T1", "forward", 1, 2048),
        # the 2816-wide prefill with its four-norm block and (1 + w) weights
        _norm("norm-prefill-T4096", "forward", 4096, 2816, offset=True),
        # training of the widest layer, a learned gate for each channel
        _norm("norm-train-T8192", "train", 8192, 7168, gate="channel"),
        # a small fp32 model whose gate is a value for each token; odd sizes
        _norm("norm-train-f32-odd", "train", 777, 1000, dtype="f32", gate="token", residual=0.5),
        # the router's weight alone: one small matrix
        _muon("muon-router", 1, 128, 2048, kind="one"),
        # the experts of one 704 x 2816 layer (a quarter of its 128), three parameters
        _muon("muon-layer-E32", 32, 704, 2816),
        # the wide experts, tall orientation (down projections)
        _muon("muon-wide", 4, 7168, 2048, kind="one", nesterov=False),
        # directions alone of fp32 matrices with odd sizes
        _muon("muon-direction-f32-odd", 3, 777, 1001, dtype="f32", kind="direction"),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    pick = rng.random()
    if pick < 0.34:
        mode = rng.choice(["lookup", "train", "train"])
        dtype = "f32" if rng.random() < 0.3 else "bf16"
        H = 8 * _log_int(rng, 8, 896)
        T = min(_log_int(rng, 1, 65536), 8192 * 7168 // H)
        V = min(_log_int(rng, 16, 131072), 131072 * 2048 // H)
        return _emb(None, mode, T, H, V, dtype=dtype, scale=rng.choice([1.0, 0.5, math.sqrt(H)]),
                    pad=rng.random() < 0.3, add=rng.random() < 0.4)
    if pick < 0.67:
        dtype = "f32" if rng.random() < 0.3 else "bf16"
        H = 8 * _log_int(rng, 8, 1024)
        T = min(_log_int(rng, 1, 32768), (8192 if dtype == "bf16" else 4096) * 7168 // H)
        pre, post = rng.choice([(True, True), (True, True), (True, False), (False, True)])
        return _norm(None, rng.choice(["forward", "train", "train"]), T, H, dtype=dtype,
                     gate=rng.choice(["none", "channel", "token"]), pre=pre, post=post,
                     offset=rng.random() < 0.3, residual=rng.choice([1.0, 1.0, 0.5]))
    kind = rng.choice(["layer", "one", "direction"])
    dtype = "f32" if rng.random() < 0.3 else "bf16"
    rows, cols = _log_int(rng, 16, 4096), _log_int(rng, 16, 8192)
    each = _orth_flops(rows, cols) * (3 if kind == "layer" else 1)
    # at most the work of the largest listed case
    batch = max(1, min(_log_int(rng, 1, 32), int(1.2e12 / each)))
    if each > 1.2e12:
        cols = min(cols, 2048)
    return _muon(None, batch, rows, cols, dtype=dtype, kind=kind, nesterov=rng.random() < 0.7)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _gen(seed, k):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 1000003 + k)
    return g


def _randn(shape, g, dtype=torch.float32, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda", dtype=torch.float32) * std).to(dtype)


def _prepare_emb(c, seed):
    T, H, V, dt = c["T"], c["H"], c["V"], DT[c["dtype"]]
    # frequent tokens are the low ids, as in a frequency-ordered vocabulary
    u = torch.rand((T,), generator=_gen(seed, 1), device="cuda", dtype=torch.float64)
    ids = (torch.exp(u * math.log(V + 1.0)) - 1.0).long().clamp_(0, V - 1).to(torch.int32)
    s = dict(case=c, w=_randn((V, H), _gen(seed, 2), dt, 1.0 / math.sqrt(H)), ids=ids)
    if c["pad"]:   # an eighth of the tokens are padding, with an id of its own
        order = torch.randperm(T, generator=_gen(seed, 3), device="cuda")
        ids[order[: T // 8]] = V - 1
    if c["mode"] == "train":
        s["dy"] = _randn((T, H), _gen(seed, 4), dt, 1e-2)
        s["dw_add"] = _randn((V, H), _gen(seed, 5), dt, 1e-2) if c["add"] else None
    if own:
        import mixture_experts_ffn_04_gb300 as m
        s["op"] = m.TokenEmbedding(T, H, V, dtype=dt, scale=c["scale"],
                                   padding_idx=V - 1 if c["pad"] else None)
    return s


def _prepare_norm(c, seed):
    T, H, dt = c["T"], c["H"], DT[c["dtype"]]
    mid = 0.0 if c["offset"] else 1.0

    def weight(k):
        return (_randn((H,), _gen(seed, k), std=0.1) + mid).to(dt)

    s = dict(case=c, x=_randn((T, H), _gen(seed, 1), dt, 2.0), y=_randn((T, H), _gen(seed, 2), dt, 0.5),
             w_post=weight(3) if c["post"] else None, w_pre=weight(4) if c["pre"] else None, gate=None)
    if c["gate"] == "channel":
        s["gate"] = _randn((H,), _gen(seed, 5), dt, 0.5)
    elif c["gate"] == "token":
        s["gate"] = torch.rand((T,), generator=_gen(seed, 5), device="cuda")
    if c["mode"] == "train":
        s["ds"] = _randn((T, H), _gen(seed, 6), dt, 1e-2)
        s["dh"] = _randn((T, H), _gen(seed, 7), dt, 1e-2) if c["pre"] else None
    if own:
        import mixture_experts_ffn_04_gb300 as m
        s["op"] = m.BlockNorm(T, H, dtype=dt, gate=c["gate"], residual_scale=c["residual"],
                              eps=EPS_NORM, unit_offset=c["offset"])
    return s


def _shapes(c):
    b, r, n = c["batch"], c["rows"], c["cols"]
    return [(b, r, n), (b, r, n), (b, n, r)] if c["kind"] == "layer" else [(b, r, n)]


def _gradient(shape, g, dtype):
    """Gradients as sums over a few hundred tokens have them: some strong
    directions over a broad floor, another size for each matrix."""
    b, r, n = shape
    k = min(r, n, 64)
    fall = (1.0 + torch.arange(k, device="cuda")).rsqrt()
    strong = (_randn((b, r, k), g) * fall) @ _randn((b, k, n), g)
    size = torch.rand((b, 1, 1), generator=g, device="cuda") + 0.1
    return ((strong + 0.3 * _randn((b, r, n), g)) * size * 1e-3).to(dtype)


def _prepare_muon(c, seed):
    dt = DT[c["dtype"]]
    s = dict(case=c, grads=[], params=[], momenta=[])
    for i, shape in enumerate(_shapes(c)):
        s["grads"].append(_gradient(shape, _gen(seed, 3 * i), dt))
        if c["kind"] != "direction":
            s["params"].append(_randn(shape, _gen(seed, 3 * i + 1), dt, 1.0 / math.sqrt(shape[2])))
            s["momenta"].append(_gradient(shape, _gen(seed, 3 * i + 2), torch.float32))
    if own:
        import mixture_experts_ffn_04_gb300 as m
        if c["kind"] == "direction":
            b, r, n = _shapes(c)[0]
            s["op"] = m.Orthogonalize(b, r, n, dtype=dt, coefficients=COEFS, steps=STEPS, eps=EPS_ORTH)
        else:
            s["op"] = m.Muon(s["params"], s["grads"], momenta=s["momenta"], lr=LR, momentum=BETA,
                             nesterov=c["nesterov"], weight_decay=DECAY, scale="spectral",
                             coefficients=COEFS, steps=STEPS, eps=EPS_ORTH)
    return s


def prepare(case, seed):
    return {"emb": _prepare_emb, "norm": _prepare_norm, "muon": _prepare_muon}[case["op"]](case, seed)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def _run_emb(s):
    c, w, ids = s["case"], s["w"], s["ids"]
    if own:
        y = s["op"].forward(w, ids)
        if c["mode"] == "lookup":
            return [y]
        return [y, s["op"].backward(ids, s["dy"], dw_add=s["dw_add"])]
    at, dt = ids.long(), DT[c["dtype"]]
    y = (w[at].float() * c["scale"]).to(dt)
    if c["mode"] == "lookup":
        return [y]
    dy = s["dy"].float() * c["scale"]
    if c["pad"]:
        dy = torch.where((ids == c["V"] - 1)[:, None], torch.zeros_like(dy), dy)
    if c["dtype"] == "f32":   # long sums of frequent tokens
        dw = torch.zeros((c["V"], c["H"]), device=dy.device, dtype=torch.float64)
        dw.index_add_(0, at, dy.double())
    else:
        dw = torch.zeros((c["V"], c["H"]), device=dy.device).index_add_(0, at, dy)
    if c["add"]:
        dw += s["dw_add"]
    return [y, dw.to(dt)]


def _run_norm(s):
    c, x, y, gate = s["case"], s["x"], s["y"], s["gate"]
    train = c["mode"] == "train"
    if own:
        op = s["op"]
        s_out, h = op.forward(x, y, w_post=s["w_post"], gate=gate, w_pre=s["w_pre"])
        if not train:
            return [t for t in (s_out, h) if t is not None]
        d = op.backward(s["ds"], s["dh"], x, y, w_post=s["w_post"], gate=gate, w_pre=s["w_pre"])
        return [t for t in (s_out, h, d.dx, d.dy, d.dw_post, d.dgate, d.dw_pre) if t is not None]
    dt, H = DT[c["dtype"]], c["H"]
    off = 1.0 if c["offset"] else 0.0
    xf, yf = x.float(), y.float()
    g = 1.0
    if gate is not None:
        g = gate.float() if c["gate"] == "channel" else gate[:, None]
    u = yf
    if c["post"]:
        r1 = torch.rsqrt(yf.square().mean(dim=1, keepdim=True) + EPS_NORM)
        yn = yf * r1
        wp = s["w_post"].float() + off
        u = yn * wp
    t = c["residual"] * xf + g * u
    out = [t.to(dt)]
    if c["pre"]:
        r2 = torch.rsqrt(t.square().mean(dim=1, keepdim=True) + EPS_NORM)
        tn = t * r2
        wq = s["w_pre"].float() + off
        out.append((tn * wq).to(dt))
    if not train:
        return out
    d = s["ds"].float()
    if c["pre"]:
        dh = s["dh"].float()
        a = dh * wq
        d = d + r2 * (a - tn * (a * tn).mean(dim=1, keepdim=True))
    du = g * d
    dy = du
    if c["post"]:
        b = du * wp
        dy = r1 * (b - yn * (b * yn).mean(dim=1, keepdim=True))
    out += [(c["residual"] * d).to(dt), dy.to(dt)]
    if c["post"]:
        out.append((du * yn).sum(dim=0).to(dt))
    if c["gate"] == "channel":
        out.append((d * u).sum(dim=0).to(dt))
    elif c["gate"] == "token":
        out.append((d * u).sum(dim=1))
    if c["pre"]:
        out.append((dh * tn).sum(dim=0).to(dt))
    return out


def _orthogonal(u):
    """The polynomial of u's singular values, u [batch, rows, cols] in fp32."""
    tall = u.shape[1] > u.shape[2]
    x = u.transpose(1, 2) if tall else u
    x = x / (x.square().sum(dim=(1, 2), keepdim=True, dtype=torch.float64).sqrt().float() + EPS_ORTH)
    a, b, c = COEFS
    for _ in range(STEPS):
        p = x @ x.transpose(1, 2)
        x = a * x + (b * p + c * (p @ p)) @ x
    return x.transpose(1, 2) if tall else x


def _run_muon(s):
    c = s["case"]
    if own:
        if c["kind"] == "direction":
            return [s["op"].forward(s["grads"][0])]
        s["op"].step()
        return s["params"] + s["momenta"]
    if c["kind"] == "direction":
        return [_orthogonal(s["grads"][0].float()).to(DT[c["dtype"]])]
    for w, g, v in zip(s["params"], s["grads"], s["momenta"]):
        gf = g.float()
        v.copy_(BETA * v + (1.0 - BETA) * gf)
        u = BETA * v + (1.0 - BETA) * gf if c["nesterov"] else v
        size = LR * math.sqrt(max(1.0, w.shape[1] / w.shape[2]))
        w.copy_((1.0 - LR * DECAY) * w.float() - size * _orthogonal(u))
    return s["params"] + s["momenta"]


def run(state):
    return {"emb": _run_emb, "norm": _run_norm, "muon": _run_muon}[state["case"]["op"]](state)


# ---------------------------------------------------------------------------
# what a pass cannot do without
# ---------------------------------------------------------------------------
def _orth_flops(rows, cols):
    """One matrix: of X X^T and its square half is enough (both are symmetric)."""
    m, n = min(rows, cols), max(rows, cols)
    return STEPS * (1.0 * m * m * n + 1.0 * m * m * m + 2.0 * m * m * n)


def work(c):
    size = {"bf16": 2, "f32": 4}[c["dtype"]]
    if c["op"] == "emb":
        T, H, V = c["T"], c["H"], c["V"]
        rows = min(T, V)
        data = size * H * (rows + T) + 4 * T
        if c["mode"] == "lookup":
            return dict(bytes=data, flops=T * H)
        data += size * H * (T + V + (V if c["add"] else 0))
        return dict(bytes=data, flops=3 * T * H)
    if c["op"] == "norm":
        T, H = c["T"], c["H"]
        rows = 3 + int(c["pre"])                   # x, y; s, h
        per = 10
        if c["mode"] == "train":
            rows += 5 + int(c["pre"])              # x, y again, ds, dh; dx, dy
            per += 30
        vectors = int(c["pre"]) + int(c["post"]) + int(c["gate"] == "channel")
        data = size * H * (rows * T + vectors * (3 if c["mode"] == "train" else 1))
        if c["gate"] == "token":
            data += 4 * T * (3 if c["mode"] == "train" else 1)
        return dict(bytes=data, flops=per * T * H)
    flops = nbytes = 0
    for b, r, n in _shapes(c):
        flops += b * _orth_flops(r, n)
        # gradient in, and either the direction out or parameter and momentum both ways
        nbytes += b * r * n * (2 * size if c["kind"] == "direction" else 3 * size + 8)
    return dict(bytes=nbytes, flops=int(flops))


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_emb(c, s):
    w = s["w"].double().requires_grad_(True)
    ids = s["ids"].long()
    y = torch.nn.functional.embedding(ids, w, padding_idx=c["V"] - 1 if c["pad"] else None) * c["scale"]
    if c["mode"] == "lookup":
        return [y.detach()]
    (dw,) = torch.autograd.grad(y, [w], s["dy"].double())
    return [y.detach(), dw + s["dw_add"].double() if c["add"] else dw]


def _exact_norm(c, s):
    leaf = {k: s[k].double().requires_grad_(True) for k in ("x", "y", "w_post", "gate", "w_pre")
            if s.get(k) is not None}
    off = 1.0 if c["offset"] else 0.0

    def rms(v, w):
        return v / torch.sqrt((v * v).sum(1, keepdim=True) / c["H"] + EPS_NORM) * (w + off)

    u = rms(leaf["y"], leaf["w_post"]) if c["post"] else leaf["y"]
    if c["gate"] != "none":
        u = u * (leaf["gate"] if c["gate"] == "channel" else leaf["gate"].reshape(-1, 1))
    t = leaf["x"] * c["residual"] + u
    out = [t] + ([rms(t, leaf["w_pre"])] if c["pre"] else [])
    if c["mode"] == "forward":
        return [v.detach() for v in out]
    up = [s["ds"].double()] + ([s["dh"].double()] if c["pre"] else [])
    names = [k for k in ("x", "y", "w_post", "gate", "w_pre") if k in leaf]
    return [v.detach() for v in out] + list(torch.autograd.grad(out, [leaf[k] for k in names], up))


def _exact_direction(u):
    """u [batch, rows, cols] in 64 bits, by products from the smaller side."""
    u = u / (torch.linalg.matrix_norm(u, keepdim=True) + EPS_ORTH)
    eye = torch.eye(min(u.shape[1:]), device=u.device, dtype=u.dtype)
    left = u.shape[1] <= u.shape[2]
    for _ in range(STEPS):
        p = torch.bmm(u, u.mT) if left else torch.bmm(u.mT, u)
        q = COEFS[0] * eye + torch.bmm(p, COEFS[1] * eye + COEFS[2] * p)
        u = torch.bmm(q, u) if left else torch.bmm(u, q)
    return u


def _exact_muon(c, s):
    if sum(b * _orth_flops(r, n) for b, r, n in _shapes(c)) > 6e12:
        return None
    if c["kind"] == "direction":
        return [_exact_direction(s["grads"][0].double())]
    params, momenta = [], []
    for w, g, v in zip(s["params"], s["grads"], s["momenta"]):
        m = torch.lerp(v.double(), g.double(), 1.0 - BETA)
        u = torch.lerp(g.double(), m, BETA) if c["nesterov"] else m
        rows, cols = w.shape[1:]
        step = LR * max(1.0, rows / cols) ** 0.5
        params.append(w.double() * (1.0 - LR * DECAY) - step * _exact_direction(u))
        momenta.append(m)
    return params + momenta


def exact(case, seed):
    s = prepare(case, seed)
    return {"emb": _exact_emb, "norm": _exact_norm, "muon": _exact_muon}[case["op"]](case, s)

"""Norms before and after a block with gate and residual, and their gradients,
against one float64 autograd graph.

Bounds (derived).  u is half a step of the output's type (bf16 2^-8, fp32 2^-24), e =
2^-24.  A row's sum runs over at most 32 columns a thread, then 5 shuffles and 32
warps: depth 72, so a norm is within 40 e of its value (half the sum's error and
four roundings), and every fp32 intermediate within 64 e of the sum of the
magnitudes that enter it; where row sums of sums enter (D, dy) 256 e.  Columns: terms
within 256 e of their magnitudes, at most 128 in a row of one sum, then the groups'
sums, n of them: (384 + n) e of the sum of magnitudes, n at most T and 4096.  Each output
is rounded once: u |exact| more.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu
U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
E24 = 2.0 ** -24


@pytest.fixture(scope="module")
def m():
    import mixture_experts_ffn_04_gb300 as m
    return m


def inputs(T, H, dt, gate, post, pre, with_y, seed=0, offset=0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def r(*shape, std=1.0, mid=0.0, dtype=dt):
        return (torch.randn(shape, generator=g, device="cuda") * std + mid).to(dtype)

    return dict(x=r(T, H, std=2.0), y=r(T, H, std=0.5) if with_y else None,
                w_post=r(H, std=0.1, mid=1.0 - offset) if post else None,
                gate={None: None, "channel": r(H, std=0.5),
                      "token": r(T, std=0.5, dtype=torch.float32)}[gate],
                w_pre=r(H, std=0.1, mid=1.0 - offset) if pre else None,
                ds=r(T, H), dh=r(T, H) if pre else None)


def reference(a, gate, res, off, eps):
    """Outputs and gradients in float64, each with the magnitudes that bound it."""
    d = {k: (None if t is None else t.double()) for k, t in a.items()}
    leaf = {k: d[k].requires_grad_(True) for k in ("x", "y", "w_post", "gate", "w_pre") if d[k] is not None}
    rms = lambda v: torch.rsqrt(v.square().mean(1, keepdim=True) + eps)
    one = torch.ones((), dtype=torch.float64, device="cuda")
    g = one if gate is None else (d["gate"] if gate == "channel" else d["gate"][:, None])
    s = res * d["x"]
    if d["y"] is not None:
        r1 = rms(d["y"]) if d["w_post"] is not None else one
        wp = d["w_post"] + off if d["w_post"] is not None else one
        yn = d["y"] * r1
        s = s + g * yn * wp
    out, mag = {"s": s}, {}
    ups = [d["ds"]] if d["ds"] is not None else []
    outs = [s] if d["ds"] is not None else []
    if d["w_pre"] is not None:
        r2 = rms(s)
        out["h"] = s * r2 * (d["w_pre"] + off)
        outs.append(out["h"])
        ups.append(d["dh"])
    grads = dict(zip(leaf, torch.autograd.grad(outs, list(leaf.values()), ups, allow_unused=True)))
    with torch.no_grad():
        ab = (res * d["x"]).abs()
        if d["y"] is not None:
            ab = ab + (g * yn * wp).abs()
        mag["s"] = ab
        D = d["ds"].abs() if d["ds"] is not None else torch.zeros_like(ab)
        if d["w_pre"] is not None:
            wq = (d["w_pre"] + off).abs()
            mag["h"] = ab * r2 * wq
            aa, sn = d["dh"].abs() * wq, ab * r2
            D = D + r2 * (aa + sn * (aa * sn).mean(1, keepdim=True))
            mag["dw_pre"] = (d["dh"].abs() * sn).sum(0)
        mag["dx"] = abs(res) * D
        if d["y"] is not None:
            ga, wa, ya = g.abs() * one, wp.abs() * one, yn.abs()
            b = D * ga * wa
            mag["dy"] = r1 * (b + ya * (b * ya).mean(1, keepdim=True)) if d["w_post"] is not None else b
            mag["dw_post"] = (D * ga * ya).sum(0)
            mag["dgate"] = (D * ya * wa).sum(0 if gate == "channel" else 1)
    names = {"x": "dx", "y": "dy", "w_post": "dw_post", "gate": "dgate", "w_pre": "dw_pre"}
    out.update({names[k]: v for k, v in grads.items()})
    return out, mag


def check(name, got, want, mag, T):
    want = want.detach()
    k = {"s": 64, "h": 128, "dx": 256, "dy": 512}.get(name, 384 + 256 + min(T, 4096))
    bound = U[got.dtype] * want.abs() + k * E24 * mag[name]
    err = (got.double() - want).abs()
    assert bool((err <= bound).all()), (name, float((err / (bound + 1e-300)).max()))


CASES = [  # T, H, dtype, gate, post, pre, y, offset, residual scale
    (1, 8, "f32", None, True, True, True, 0, 1.0), (1, 2048, "bf16", None, True, True, True, 0, 1.0),
    (3, 16, "bf16", "token", True, True, True, 1, 0.5), (70, 24, "f32", "channel", True, True, True, 0, 1.0),
    (130, 200, "bf16", "channel", True, True, True, 1, 1.0), (777, 1000, "f32", "token", True, True, True, 0, 0.5),
    (33, 256, "f32", None, False, True, True, 0, 1.0), (50, 264, "bf16", "token", False, False, True, 0, 2.0),
    (50, 2816, "bf16", None, True, False, True, 1, 1.0), (40, 2816, "f32", None, False, True, False, 0, 1.0),
    (65, 4096, "bf16", "channel", True, True, True, 0, 1.0), (20, 7168, "f32", "channel", True, True, True, 0, 1.0),
    (700, 7168, "bf16", "token", True, True, True, 0, 1.0), (9, 8200, "f32", "token", True, True, True, 0, 1.0),
    (5, 32768, "bf16", "channel", True, True, True, 0, 1.0), (3, 32768, "f32", None, True, True, True, 0, 0.0),
    (40000, 64, "bf16", "channel", True, True, True, 0, 1.0), (50001, 8, "f32", "channel", True, True, True, 0, 1.0)]


@pytest.mark.parametrize("T,H,dtype,gate,post,pre,with_y,offset,res", CASES)
def test_forward_and_gradients(m, T, H, dtype, gate, post, pre, with_y, offset, res):
    dt = torch.float32 if dtype == "f32" else torch.bfloat16
    a = inputs(T, H, dt, gate, post, pre, with_y, seed=T + H, offset=offset)
    want, mag = reference(a, gate, res, offset, 1e-6)
    op = m.BlockNorm(T, H, dtype=dt, gate=gate, residual_scale=res, unit_offset=bool(offset))
    kw = {k: a[k] for k in ("w_post", "gate", "w_pre")}
    s, h = op.forward(a["x"], a["y"], **kw)
    d = op.backward(a["ds"], a["dh"], a["x"], a["y"], **kw)
    for name, got in [("s", s), ("h", h)] + list(d._asdict().items()):
        assert (got is None) == (want.get(name) is None), name
        if got is not None:
            check(name, got, want[name], mag, T)
    again = op.backward(a["ds"], a["dh"], a["x"], a["y"], **kw)
    assert all(torch.equal(p, q) for p, q in zip(d, again) if p is not None)


def test_gradients_against_differences(m):
    """The gradient formulas themselves, by central differences of the kernel's own fp32
    forward: a step of 2^-6 and values of order one leave an error below 1e-3 of the
    largest gradient (third derivatives times 2^-12 / 6) plus 2 * 64 e / 2^-6 * H."""
    T, H = 2, 16
    a = inputs(T, H, torch.float32, "channel", True, True, True, seed=3)
    op = m.BlockNorm(T, H, dtype=torch.float32, gate="channel")

    def objective():
        s, h = op.forward(a["x"], a["y"], w_post=a["w_post"], gate=a["gate"], w_pre=a["w_pre"])
        return float((s.double() * a["ds"].double()).sum() + (h.double() * a["dh"].double()).sum())

    objective()
    d = op.backward(a["ds"], a["dh"], a["x"], a["y"], w_post=a["w_post"], gate=a["gate"], w_pre=a["w_pre"])
    step = 2.0 ** -6
    for name, grad in (("x", d.dx), ("y", d.dy), ("w_post", d.dw_post), ("gate", d.dgate), ("w_pre", d.dw_pre)):
        t = a[name].view(-1)
        top = float(grad.abs().max())
        for i in range(0, t.numel(), 5):
            keep = float(t[i])
            t[i] = keep + step
            up = objective()
            t[i] = keep - step
            down = objective()
            t[i] = keep
            assert abs((up - down) / (2 * step) - float(grad.view(-1)[i])) <= 2e-3 * top + 2e-3, (name, i)


def test_only_some_gradients_and_in_place(m):
    T, H = 100, 512
    a = inputs(T, H, torch.bfloat16, "token", True, True, True)
    op = m.BlockNorm(T, H, gate="token")
    kw = {k: a[k] for k in ("w_post", "gate", "w_pre")}
    op.forward(a["x"], a["y"], **kw)
    full = op.backward(a["ds"], a["dh"], a["x"], a["y"], **kw)
    ref = (a["w_post"], a["gate"], a["w_pre"])
    only = torch.empty_like(a["x"])
    m.moe_block_norm_backward(op.shape, a["ds"], a["dh"], a["x"], a["y"], *ref, op.rstd, None, only, None, None, None, op.ws)
    assert torch.equal(only, full.dy)
    col = torch.empty_like(a["w_pre"])
    m.moe_block_norm_backward(op.shape, a["ds"], a["dh"], a["x"], a["y"], *ref, op.rstd, None, None, None, None, col, op.ws)
    assert torch.equal(col, full.dw_pre)
    ds, y = a["ds"].clone(), a["y"].clone()
    m.moe_block_norm_backward(op.shape, ds, a["dh"], a["x"], y, *ref, op.rstd, ds, y, None, None, None, op.ws)
    assert torch.equal(ds, full.dx) and torch.equal(y, full.dy)
    x = a["x"].clone()
    s, h = op.forward(x, a["y"], **kw, s=x)
    want, _ = op.forward(a["x"], a["y"], **kw)
    assert torch.equal(x, want)


def test_no_gradient_of_s(m):
    a = inputs(64, 256, torch.float32, None, True, True, True)
    op = m.BlockNorm(64, 256, dtype=torch.float32)
    kw = {k: a[k] for k in ("w_post", "w_pre")}
    op.forward(a["x"], a["y"], **kw)
    d = op.backward(None, a["dh"], a["x"], a["y"], **kw)
    zero = op.backward(torch.zeros_like(a["ds"]), a["dh"], a["x"], a["y"], **kw)
    assert all(torch.equal(p, q) for p, q in zip(d, zero) if p is not None)


def test_no_tokens_and_rows_of_zeros(m):
    op = m.BlockNorm(0, 64, gate="channel")
    e = torch.empty((0, 64), device="cuda", dtype=torch.bfloat16)
    w = torch.ones(64, device="cuda", dtype=torch.bfloat16)
    s, h = op.forward(e, e, w_post=w, gate=w, w_pre=w)
    d = op.backward(e, e, e, e, w_post=w, gate=w, w_pre=w)
    assert s.shape == h.shape == (0, 64)
    assert all(float(t.abs().max()) == 0.0 for t in (d.dw_post, d.dgate, d.dw_pre))
    z = torch.zeros((5, 64), device="cuda", dtype=torch.bfloat16)
    op = m.BlockNorm(5, 64)
    s, h = op.forward(z, z, w_post=w, w_pre=w)
    d = op.backward(z, z + 1, z, z, w_post=w, w_pre=w)
    assert float(s.abs().max()) == float(h.abs().max()) == 0.0
    assert all(bool(torch.isfinite(t).all()) for t in (d.dx, d.dy))   # 1 / sqrt(eps) times 1


def test_a_bad_row_stays_in_its_row(m):
    a = inputs(40, 520, torch.bfloat16, None, True, True, True)
    op = m.BlockNorm(40, 520)
    kw = {k: a[k] for k in ("w_post", "w_pre")}
    s0, h0 = (t.clone() for t in op.forward(a["x"], a["y"], **kw))
    a["y"][7, 3] = float("nan")
    a["x"][9, 5] = float("inf")
    s, h = op.forward(a["x"], a["y"], **kw)
    ok = torch.ones(40, dtype=torch.bool, device="cuda")
    ok[[7, 9]] = False
    assert torch.equal(s[ok], s0[ok]) and torch.equal(h[ok], h0[ok])
    assert bool(s[7].isnan().all()) and bool(h[9].isnan().any())


def test_stream_and_graph(m):
    T, H = 300, 1024
    a = inputs(T, H, torch.bfloat16, "channel", True, True, True)
    op = m.BlockNorm(T, H, gate="channel")
    kw = {k: a[k] for k in ("w_post", "gate", "w_pre")}

    def both(stream=None):
        out = op.forward(a["x"], a["y"], **kw, stream=stream)
        return list(out) + list(op.backward(a["ds"], a["dh"], a["x"], a["y"], **kw, stream=stream))

    want = [t.clone() for t in both()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = both(side)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both()
    for t in out:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(out, want))


MANY = [  # rows enough for several steps of every ring, in both directions
    (5000, 1024, "bf16", "channel", True, True, True, 0, 1.0), (4001, 1000, "f32", "token", True, True, True, 1, 0.5),
    (3001, 2816, "bf16", None, True, True, True, 1, 1.0), (3001, 512, "f32", "token", False, True, True, 0, 1.0),
    (4000, 520, "bf16", "channel", True, False, True, 0, 1.0), (6001, 264, "bf16", None, False, True, False, 0, 2.0),
    (3000, 640, "f32", "channel", False, False, True, 0, 1.0), (9001, 136, "bf16", "token", True, True, True, 0, 1.0),
    (2000, 7168, "bf16", "channel", True, True, True, 0, 1.0), (1500, 7168, "f32", None, True, True, True, 0, 1.0)]


@pytest.mark.parametrize("T,H,dtype,gate,post,pre,with_y,offset,res", MANY)
def test_many_rows(m, T, H, dtype, gate, post, pre, with_y, offset, res):
    test_forward_and_gradients(m, T, H, dtype, gate, post, pre, with_y, offset, res)


@pytest.mark.parametrize("T,H,dt", [(6000, 512, torch.bfloat16), (4001, 72, torch.float32), (3000, 4096, torch.bfloat16)])
def test_many_rows_in_place(m, T, H, dt):
    a = inputs(T, H, dt, "token", True, True, True)
    op = m.BlockNorm(T, H, dtype=dt, gate="token")
    kw = {k: a[k] for k in ("w_post", "gate", "w_pre")}
    s, h = op.forward(a["x"], a["y"], **kw)
    full = op.backward(a["ds"], a["dh"], a["x"], a["y"], **kw)
    ds, y = a["ds"].clone(), a["y"].clone()
    got = op.backward(ds, a["dh"], a["x"], y, **kw, dx=ds, dy=y)
    assert all(torch.equal(p, q) for p, q in zip(got, full))
    x = a["x"].clone()
    again = op.forward(x, a["y"], **kw, s=x)
    assert torch.equal(again[0], s) and torch.equal(again[1], h)
    zero = op.backward(torch.zeros_like(a["ds"]), a["dh"], a["x"], a["y"], **kw)
    none = op.backward(None, a["dh"], a["x"], a["y"], **kw)
    assert all(torch.equal(p, q) for p, q in zip(none, zero))
    # a bad row stays in its row (what is summed over rows apart)
    a["y"][T // 3, 3], a["x"][T // 2, 5] = float("nan"), float("inf")
    s2, h2 = op.forward(a["x"], a["y"], **kw)
    d = op.backward(a["ds"], a["dh"], a["x"], a["y"], **kw)
    ok = torch.ones(T, dtype=torch.bool, device="cuda")
    ok[[T // 3, T // 2]] = False
    assert torch.equal(s2[ok], s[ok]) and torch.equal(h2[ok], h[ok])
    assert torch.equal(d.dx[ok], full.dx[ok]) and torch.equal(d.dy[ok], full.dy[ok])
    assert torch.equal(d.dgate[ok], full.dgate[ok])

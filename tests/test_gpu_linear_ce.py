"""The vocabulary cross entropy and its gradients on the GPU against the
definition in float64.

Bounds (derived, not fitted).  u = eps / 2 of the input type, f = 2^-24.
 * logits: fp32 sums of exact products, |error| <= 2 H f * sum |x w| at worst;
   the random walk of the rounding gives sqrt(H) f |x||w|.  The bound taken is
   8 sqrt(H) f |x||w| + 8 f |z|, absolute, for lse and loss (lse and z_target
   each, so twice), plus 8 f |lse| for the exponentials and the final rounding.
 * gradients: every d_tv is rounded once (u, relative; fp32: three planes,
   2^-24) and carries the logit's error as a relative one; each output is
   rounded once (u).  Sums of n such terms: relative L2 error at most
   u (rounding of d, independent) + u (output) + logit error.  The bound taken is
   2 u + 4 * the logit bound + 16 f, on the relative L2 of the matrix.
"""
import math

import pytest
import torch

import mixture_experts_ffn_04_gb300 as m

pytestmark = pytest.mark.gpu
IGNORE = -100
F = 2.0 ** -24
U = {torch.bfloat16: 2.0 ** -8, torch.float32: F}


def make(T, H, V, dtype, ignored=0.0, pad=0, wpad=0, seed=0, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn((T, H + pad), generator=g, device="cuda").mul_(scale).to(dtype)[:, :H]
    w = (torch.randn((V, H + wpad), generator=g, device="cuda") / math.sqrt(H)).to(dtype)[:, :H]
    t = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    if ignored:
        t[torch.rand((T,), generator=g, device="cuda") < ignored] = IGNORE
    return x, w, t


def reference(x, w, t, reduction, dloss, V):
    """Loss, lse, dx, dw in float64 over the rows that count."""
    ok = (t >= 0) & (t < V) & (t != IGNORE)
    rows = ok.nonzero().flatten()
    xd, wd = x[rows].double(), w.double()
    z = xd @ wd.t()
    lse = torch.full((len(t),), 0.0, device=x.device, dtype=torch.float64)
    loss = torch.zeros_like(lse)
    p = torch.zeros_like(z)
    if len(rows):
        lse[rows] = torch.logsumexp(z, 1)
        loss[rows] = lse[rows] - z[torch.arange(len(rows)), t[rows].long()]
        p = torch.softmax(z, 1)
        p[torch.arange(len(rows)), t[rows].long()] -= 1.0
    n = max(len(rows), 1)
    if reduction == "none":
        out, g = loss, dloss.double()[rows]
    else:
        up = 1.0 if dloss is None else float(dloss)
        k = n if reduction == "mean" else 1
        out = loss.sum().reshape(1) / k
        g = torch.full((len(rows),), up / k, device=x.device, dtype=torch.float64)
    d = p * g[:, None]
    dx = torch.zeros(tuple(x.shape), device=x.device, dtype=torch.float64)
    dx[rows] = d @ wd
    dw = d.t() @ xd
    zb = 8 * math.sqrt(x.shape[1]) * F * float((xd.norm(dim=1).max() if len(rows) else 0.0) * wd.norm(dim=1).max())
    zb += 16 * F * (float(z.abs().max()) if z.numel() else 0.0)
    return out, lse, dx, dw, zb


def rel(a, b):
    n = float(b.norm())
    return float((a.double() - b).norm()) / n if n else float(a.double().norm())


def check(x, w, t, dtype, reduction="mean", dloss=None, V=None):
    T, H = x.shape
    V = w.shape[0]
    op = m.LinearCrossEntropy(T, H, V, dtype=dtype, reduction=reduction, ignore_index=IGNORE)
    loss = op.forward(x, w, t)
    dx, dw = op.backward(x, w, t, dloss)
    out, lse, rdx, rdw, zb = reference(x, w, t, reduction, dloss, V)
    assert torch.isfinite(loss).all() and torch.isfinite(dx.float()).all() and torch.isfinite(dw.float()).all()
    tol = 2 * zb + 8 * F * float(lse.abs().max() if T else 0.0)
    many = 1 if reduction != "sum" else max(T, 1)
    assert (op.lse.double() - lse).abs().max() <= tol if T else True
    assert (loss.double() - out).abs().max() <= tol * many + 2 * F * float(out.abs().max()) if T else True
    gt = 2 * U[dtype] + 4 * zb + 16 * F
    assert rel(dx, rdx) <= gt, (rel(dx, rdx), gt)
    assert rel(dw, rdw) <= gt, (rel(dw, rdw), gt)
    # rows that do not count have exactly zero gradients
    off = ~((t >= 0) & (t < V) & (t != IGNORE))
    assert (dx[off] == 0).all() and (op.lse[off] == 0).all()
    return op, loss, dx, dw


SHAPES = [(1, 256, 257), (2, 64, 1000), (63, 72, 255), (64, 264, 256), (65, 512, 511),
          (127, 8, 5), (129, 1032, 3001), (256, 256, 1), (257, 2048, 4099), (1000, 320, 2049),
          (300, 4096, 700)]


@pytest.mark.parametrize("T,H,V", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_shapes(T, H, V, dtype):
    x, w, t = make(T, H, V, dtype, seed=T + V)
    check(x, w, t, dtype)


@pytest.mark.parametrize("reduction", ["none", "sum", "mean"])
@pytest.mark.parametrize("ignored", [0.3, 0.97])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_reductions_and_ignored(reduction, ignored, dtype):
    T, H, V = 333, 264, 1111
    x, w, t = make(T, H, V, dtype, ignored=ignored, pad=8, wpad=16, seed=7)
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    dloss = torch.randn(T if reduction == "none" else 1, generator=g, device="cuda")
    check(x, w, t, dtype, reduction, dloss)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rows_that_do_not_count_may_hold_anything(dtype):
    T, H, V = 200, 128, 600
    x, w, t = make(T, H, V, dtype, ignored=0.4, seed=1)
    off = t == IGNORE
    a = check(x, w, t, dtype)
    for bad in (float("nan"), float("inf"), torch.finfo(dtype).min):
        xb = x.clone()
        xb[off] = bad
        b = check(xb, w, t, dtype)
        for p, q in zip(a[1:], b[1:]):
            assert torch.equal(p, q)


@pytest.mark.parametrize("reduction", ["none", "sum", "mean"])
def test_no_row_counts(reduction):
    T, H, V = 70, 64, 300
    x, w, t = make(T, H, V, torch.bfloat16)
    t.fill_(IGNORE)
    dloss = torch.ones(T, device="cuda") if reduction == "none" else None
    op, loss, dx, dw = check(x, w, t, torch.bfloat16, reduction, dloss)
    assert (loss == 0).all() and (dx == 0).all() and (dw == 0).all()
    assert op.device_status() == (m.MOE_OK, 0)


def test_no_tokens():
    x, w, t = make(0, 64, 300, torch.bfloat16)
    op = m.LinearCrossEntropy(0, 64, 300)
    assert float(op.forward(x, w, t)) == 0.0
    dx, dw = op.backward(x, w, t)
    assert dx.shape == (0, 64) and (dw == 0).all()


def test_target_out_of_range_is_dropped_and_flagged():
    x, w, t = make(40, 64, 300, torch.bfloat16)
    t[3], t[17] = 300, -1
    op, *_ = check(x, w, t, torch.bfloat16)
    st, bits = op.device_status()
    assert st == m.MOE_ERR_TARGET and bits == 16
    assert op.device_status() == (m.MOE_OK, 0)


def test_large_logits_and_masked_columns():
    """Logits of several hundred: nothing overflows; and rows of w at the type's
    lowest value only push their columns' probabilities to 0."""
    T, H, V = 96, 64, 515
    x, w, t = make(T, H, V, torch.bfloat16, scale=40.0, seed=5)
    check(x, (w * 8), t, torch.bfloat16)
    x = x.abs()
    w = w.clone()
    w[100:110] = -torch.finfo(torch.bfloat16).max / 1e6
    t[(t >= 100) & (t < 110)] = 0
    op = m.LinearCrossEntropy(T, H, V, reduction="none")
    loss = op.forward(x, w, t)
    keep = torch.ones(V, dtype=torch.bool, device="cuda")
    keep[100:110] = False
    z = x.double() @ w[keep].double().t()
    lse = torch.logsumexp(z, 1)
    assert torch.allclose(op.lse.double(), lse, rtol=1e-5, atol=1e-3)
    assert torch.isfinite(loss).all()


def test_pieces_of_the_vocabulary():
    """More rows x columns than one piece of the backward holds."""
    T, H, V = 2100, 128, 70001
    x, w, t = make(T, H, V, torch.bfloat16, ignored=0.1, seed=11)
    check(x, w, t, torch.bfloat16)


def test_one_of_the_gradients():
    x, w, t = make(130, 128, 900, torch.bfloat16)
    op, loss, dx, dw = check(x, w, t, torch.bfloat16)
    a, b = torch.empty_like(dx), torch.empty_like(dw)
    m.moe_linear_ce_backward(op.shape, x, w, t, op.stats, None, a, None, op.ws)
    m.moe_linear_ce_backward(op.shape, x, w, t, op.stats, None, None, b, op.ws)
    assert torch.equal(a, dx) and torch.equal(b, dw)


def test_gradient_against_differences():
    """Central differences of the float64 loss along a random direction, and
    the kernel's own forward for a direction large enough to see in fp32."""
    T, H, V = 50, 64, 400
    x, w, t = make(T, H, V, torch.float32, seed=2)
    op, loss, dx, dw = check(x, w, t, torch.float32)
    g = torch.Generator(device="cuda")
    g.manual_seed(9)
    vx = torch.randn((T, H), generator=g, device="cuda")
    vw = torch.randn((V, H), generator=g, device="cuda") / math.sqrt(H)
    h = 2.0 ** -6
    up = float(op.forward(x + h * vx, w + h * vw, t))
    dn = float(op.forward(x - h * vx, w - h * vw, t))
    want = float((dx.double() * vx).sum() + (dw.double() * vw).sum())
    # truncation h^2/6 f''' with f''' of order 1..10, rounding 2^-22 / h
    assert abs((up - dn) / (2 * h) - want) <= 10 * h * h + 2.0 ** -20 / h


def test_repeatable_other_stream_and_graph():
    T, H, V = 500, 256, 5000
    x, w, t = make(T, H, V, torch.bfloat16, ignored=0.2, seed=21)
    op, loss, dx, dw = check(x, w, t, torch.bfloat16)
    for _ in range(3):
        a = op.forward(x, w, t)
        b = op.backward(x, w, t)
        assert torch.equal(a, loss) and torch.equal(b[0], dx) and torch.equal(b[1], dw)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        a = op.forward(x, w, t)
        b = op.backward(x, w, t)
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(a, loss) and torch.equal(b[0], dx) and torch.equal(b[1], dw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a = op.forward(x, w, t)
        b = op.backward(x, w, t)
    x2, _, t2 = make(T, H, V, torch.bfloat16, ignored=0.6, seed=22)
    x.copy_(x2)
    t.copy_(t2)
    graph.replay()
    c = check(x, w, t, torch.bfloat16)
    assert torch.equal(a, c[1]) and torch.equal(b[0], c[2]) and torch.equal(b[1], c[3])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_outputs_on_16_byte_boundaries(dtype):
    """dx and dw that start 16 bytes past a 32-byte boundary."""
    T, H, V = 200, 256, 700
    x, w, t = make(T, H, V, dtype, ignored=0.2, seed=4)
    op, loss, dx, dw = check(x, w, t, dtype)
    o = 16 // x.element_size()
    bx = torch.full((T * H + 2 * o,), 3.0, device="cuda", dtype=dtype)
    bw = torch.full((V * H + 2 * o,), 3.0, device="cuda", dtype=dtype)
    vx, vw = bx[o: o + T * H].view(T, H), bw[o: o + V * H].view(V, H)
    op.backward(x, w, t, dx=vx, dw=vw)
    assert torch.equal(vx, dx) and torch.equal(vw, dw)
    for b in (bx, bw):
        assert (b[:o] == 3).all() and (b[-o:] == 3).all()


@pytest.mark.parametrize("a,b", [(1e-12, 1e12), (1e15, 1e-15), (2.0 ** -60, 2.0 ** 60)])
def test_fp32_of_any_magnitude(a, b):
    """The fp16 planes of fp32 inputs follow the matrices' own magnitudes."""
    T, H, V = 150, 128, 500
    x, w, t = make(T, H, V, torch.float32, ignored=0.2, seed=6)
    check(x * a, w * b, t, torch.float32)
    dl = torch.rand(T, device="cuda") * a
    check(x, w, t, torch.float32, "none", dl)


def test_fp32_rows_of_different_magnitude():
    """Rows of x, rows of w and the tokens' weights over six decades each: every
    row of dx and dw is as exact as its own magnitude allows (22 bits down to
    2^-29 of the largest)."""
    T, H, V = 120, 64, 300
    x, w, t = make(T, H, V, torch.float32, seed=8)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    ten = lambda n: 10.0 ** (-6.0 * torch.rand(n, generator=g, device="cuda"))
    x, w, dl = x * ten(T)[:, None], w * ten(V)[:, None], ten(T)
    op, loss, dx, dw = check(x, w, t, torch.float32, "none", dl)
    _, _, rdx, rdw, zb = reference(x, w, t, "none", dl, V)
    tol = 2.0 ** -21 + 4 * zb + 16 * F
    for got, want in ((dx, rdx), (dw, rdw)):
        # a row's terms cancel (each token's weight is p - 1 at its target): the
        # bound is on the row's own norm where it is not below its largest term
        err = (got.double() - want).norm(dim=1)
        size = want.norm(dim=1)
        assert (err <= 16 * tol * torch.maximum(size, 2.0 ** -20 * size.max())).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_many_tokens(dtype):
    """Several tokens a warp in the packing; dW's rows (K) split in parts."""
    T, H, V = 40001, 64, 300
    x, w, t = make(T, H, V, dtype, ignored=0.3, seed=12)
    check(x, w, t, dtype)


@pytest.mark.parametrize("T,V", [(263001, 70), (70, 263001)])
def test_offsets_past_31_bits(T, V):
    """x and dx, or w and dw, of more than 2^31 elements: the first and last rows
    against float64 on those rows."""
    H = 8200
    g = torch.Generator(device="cuda")
    g.manual_seed(0)
    x = torch.randn((T, H), generator=g, device="cuda", dtype=torch.bfloat16)
    w = torch.randn((V, H), generator=g, device="cuda", dtype=torch.bfloat16).mul_(H ** -0.5)
    t = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    t[-3], t[1] = V - 1, IGNORE
    op = m.LinearCrossEntropy(T, H, V, reduction="none", ignore_index=IGNORE)
    dl = torch.rand(T, generator=g, device="cuda")
    loss = op.forward(x, w, t)
    dx, dw = op.backward(x, w, t, dl)
    keep = (t != IGNORE).float()
    if V < T:   # a few rows of dx
        rows = torch.tensor([0, 1, 2, 131072, T - 3, T - 1], device="cuda")
        z = x[rows].double() @ w.double().t()
        lse = torch.logsumexp(z, 1) * keep[rows]
        p = torch.softmax(z, 1)
        p[torch.arange(len(rows)), t[rows].long().clamp(min=0)] -= 1.0
        want = (p * (dl * keep)[rows, None].double()) @ w.double()
        got = dx[rows]
        assert ((op.lse[rows].double() - lse).abs() <= 1e-4).all()
    else:       # a few rows of dw: p of those columns needs every column's lse
        cols = torch.tensor([0, 1, 131072, V - 2, V - 1], device="cuda")
        z = torch.cat([x.double() @ c.double().t() for c in w.split(32768)], 1)
        lse = torch.logsumexp(z, 1)
        assert ((op.lse.double() - lse * keep).abs() <= 1e-4).all()
        p = torch.exp(z[:, cols] - lse[:, None]) - (t.long()[:, None] == cols[None]).double()
        want = (p * (dl * keep)[:, None].double()).t() @ x.double()
        got = dw[cols]
    err = (got.double() - want).norm(dim=1) / want.norm(dim=1).clamp(min=1e-30)
    # two roundings of bf16 and, on sums of few terms, what the logits' fp32 sums
    # leave (1e-4 on a probability)
    assert (err <= 2 * U[torch.bfloat16] + 1e-3).all(), err


@pytest.mark.parametrize("T", [2, 60])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_nearly_certain_targets(T, dtype):
    """Targets whose probability is 1 - 1e-2 .. 1 - 1e-5 (logits 20 above the rest):
    the loss and d = p - 1 keep their digits although lse is near 24.  The bound is
    relative: the chunked fp32 sums' error of the logits' difference (zb, absolute)
    plus a few f, against a loss and a gradient of size 1 - p."""
    H, V = 64, 400
    x, w, t = make(T, H, V, dtype, seed=9)
    x = torch.nn.functional.normalize(w[t.long()].float(), dim=1) * 22
    x = x.to(dtype)
    op = m.LinearCrossEntropy(T, H, V, dtype=dtype, reduction="sum", ignore_index=IGNORE)
    loss = op.forward(x, w, t)
    dx, dw = op.backward(x, w, t)
    out, lse, rdx, rdw, zb = reference(x, w, t, "sum", None, V)
    assert abs(float(loss) - float(out)) <= (2 * zb + 64 * F) * T
    tol = 2 * U[dtype] + 4 * zb + 16 * F
    # each token's row of dx is (p - 1) w_t + ...: size 1 - p, error 8 f + zb (1 - p)
    size = rdx.norm(dim=1)
    err = (dx.double() - rdx).norm(dim=1)
    assert (err <= tol * size + 8 * F * float(w.double().norm(dim=1).max())).all()

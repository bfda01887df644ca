"""The training operators where their state, ranges and inputs are unusual: one
workspace for several shapes, logits far from zero, fp32 matrices whose rows and
columns differ by more than half precision can hold, dropped routes with any value
in their slots, very many tokens, lists given as generators, outputs made on
another stream.

Bounds (derived).  f = 2^-24, u = f or 2^-8 (bf16).
 * logits: zb = 8 sqrt(H) f max|x| max|w| + 16 f max|z|, the bound of a product in
   fp32, over the columns that are not masked (a masked column's probability is
   exactly 0 on both sides).  lse and loss: 2 zb + 8 f |lse|.
 * gradients: 2 u (the operand's and the result's rounding) + 4 zb (the
   probabilities' relative error) + 16 f, relative, of the matrix or row named.
"""
import math

import pytest
import torch

import mixture_experts_ffn_04_gb300 as m
from mixture_experts_ffn_04_gb300 import workloads as W

pytestmark = pytest.mark.gpu
IGNORE = -100
F = 2.0 ** -24
BF, FP = torch.bfloat16, torch.float32


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def make(T, H, V, seed):
    g = gen(seed)
    x = torch.randn((T, H), generator=g, device="cuda")
    w = torch.randn((V, H), generator=g, device="cuda") / math.sqrt(H)
    t = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
    return x, w, t, torch.rand(T, generator=g, device="cuda") + 0.5


# ---------------------------------------------------------------------------
# cross entropy in fp32: magnitudes that differ within a matrix
# ---------------------------------------------------------------------------
def compare(x, w, t, dl, columns, rows):
    """Loss, lse, dx and dw with weights per token; `columns` of w are not masked,
    `rows` of x have ordinary logits."""
    T, H = x.shape
    V = w.shape[0]
    op = m.LinearCrossEntropy(T, H, V, dtype=FP, reduction="none", ignore_index=IGNORE)
    loss = op.forward(x, w, t)
    dx, dw = op.backward(x, w, t, dl)
    xd, wd = x[rows].double(), w[columns].double()
    z = xd @ wd.t()
    at = torch.full((V,), -1, device="cuda")
    at[columns] = torch.arange(len(columns), device="cuda")
    tt = at[t[rows].long()]
    assert (tt >= 0).all()
    one = torch.nn.functional.one_hot(tt, len(columns)).double()
    lse = torch.logsumexp(z, 1)
    d = (torch.softmax(z, 1) - one) * dl[rows].double()[:, None]
    # entries that meet zeros on the other side add nothing to a logit
    live = (wd != 0).any(0), (xd != 0).any(0)
    zb = 8 * math.sqrt(H) * F * float((xd * live[0]).norm(dim=1).max() * (wd * live[1]).norm(dim=1).max())
    zb += 16 * F * float(z.abs().max())
    tol = 2 * zb + 8 * F * float(lse.abs().max())
    assert float((op.lse[rows].double() - lse).abs().max()) <= tol
    assert float((loss[rows].double() - (lse - (z * one).sum(1))).abs().max()) <= tol
    gt = 2 * F + 4 * zb + 16 * F
    assert torch.isfinite(dx[rows]).all() and torch.isfinite(dw).all()
    return d, dx, dw, xd, wd, gt


@pytest.mark.parametrize("value", [1e9, 1e15, 1e30, -torch.finfo(FP).min])
@pytest.mark.parametrize("T", [2, 5, 60, 300])
def test_fp32_masked_rows_of_w(T, value):
    """Rows of w that send their column's logit to -value through one feature."""
    H, V = 72, 700
    x, w, t, dl = make(T, H, V, 31)
    x[:, 3] = 1.0
    columns = torch.ones(V, dtype=torch.bool, device="cuda")
    columns[torch.tensor([0, 100, 101, 255, 256, 699], device="cuda")] = False
    columns[384:512] = False         # all the columns of a half tile
    w[~columns] = 0.0
    w[~columns, 3] = -value
    columns = columns.nonzero().flatten()
    t = columns[t.long() % len(columns)].to(torch.int32)
    rows = torch.arange(T, device="cuda")
    d, dx, dw, xd, wd, gt = compare(x, w, t, dl, columns, rows)
    want = d @ wd
    assert float((dx.double() - want).norm()) <= gt * float(want.norm())
    want = d.t() @ xd
    assert float((dw[columns].double() - want).norm()) <= gt * float(want.norm())
    gone = torch.ones(V, dtype=torch.bool, device="cuda")
    gone[columns] = False
    assert (dw[gone] == 0).all()


@pytest.mark.parametrize("value", [1e9, 1e15, 1e30])
@pytest.mark.parametrize("T", [5, 130])
def test_fp32_row_and_feature_of_x_far_above_the_rest(T, value):
    """A token of huge magnitude that is not learned from (weight 0), and a huge
    feature that no row of w reads: the other tokens keep their digits."""
    H, V = 136, 515
    x, w, t, dl = make(T, H, V, 32)
    x[3] *= value
    dl[3] = 0.0
    x[:, 7] = value
    w[:, 7] = 0.0
    rows = torch.arange(T, device="cuda") != 3
    rows = rows.nonzero().flatten()
    d, dx, dw, xd, wd, gt = compare(x, w, t, dl, torch.arange(V, device="cuda"), rows)
    want = d @ wd
    assert float((dx[rows].double() - want).norm()) <= gt * float(want.norm())
    assert (dx[3] == 0).all()
    # the huge feature's own gradients are huge: the others by themselves
    keep = torch.arange(H, device="cuda") != 7
    want = (d.t() @ xd)[:, keep]
    assert float((dw[:, keep].double() - want).norm()) <= gt * float(want.norm())


@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 8, 9, 16, 17])
def test_fp32_few_rows_over_several_pieces(T):
    """Few rows have kernels of their own in both directions (up to 16 at this size);
    w's planes take more than one piece here; one of the tokens does not count."""
    H, V = 4096, 40001
    x, w, t, dl = make(T, H, V, 37)
    t[T - 1] = 39999
    if T > 1:
        t[0] = IGNORE
        x[0] = math.nan
        rows = torch.arange(1, T, device="cuda")
    else:
        rows = torch.arange(1, device="cuda")
    d, dx, dw, xd, wd, gt = compare(x, w, t, dl, torch.arange(V, device="cuda"), rows)
    want = d @ wd
    assert float((dx[rows].double() - want).norm()) <= gt * float(want.norm())
    want = d.t() @ xd
    assert float((dw.double() - want).norm()) <= gt * float(want.norm())
    if T > 1:
        assert (dx[0] == 0).all()


@pytest.mark.parametrize("H,T", [(520, 7), (520, 12), (520, 16), (520, 17), (520, 31), (520, 32), (520, 33),
                                 (4000, 15), (4000, 17), (8200, 6), (8200, 8), (8200, 9), (14080, 3), (14088, 3)])
def test_fp32_rows_in_groups(H, T):
    """Rows that fill one or two groups of the few-row kernels (16, 8 or 4 rows, by H)
    or miss them by one; a third of the tokens do not count and hold anything."""
    V = 777
    x, w, t, dl = make(T, H, V, 38)
    skip = torch.arange(T, device="cuda") % 3 == 1
    t[skip] = IGNORE
    x[skip] = math.inf
    rows = (~skip).nonzero().flatten()
    d, dx, dw, xd, wd, gt = compare(x, w, t, dl, torch.arange(V, device="cuda"), rows)
    want = d @ wd
    assert float((dx[rows].double() - want).norm()) <= gt * float(want.norm())
    want = d.t() @ xd
    assert float((dw.double() - want).norm()) <= gt * float(want.norm())
    assert (dx[skip] == 0).all()
    for reduction in ("sum", "mean"):
        op = m.LinearCrossEntropy(T, H, V, dtype=FP, reduction=reduction, ignore_index=IGNORE)
        got = float(op.forward(x, w, t))
        z = xd @ wd.t()
        each = torch.logsumexp(z, 1) - z.gather(1, t[rows].long()[:, None])[:, 0]
        ref = float(each.sum() if reduction == "sum" else each.mean())
        assert abs(got - ref) <= gt * abs(ref)


def test_fp32_gradient_of_rare_columns():
    """A column whose probability is about 1e-13 at every token: its row of dw has
    all its digits, not those that are left next to 1."""
    T, H, V = 64, 64, 300
    x, w, t, dl = make(T, H, V, 33)
    x[:, 5] = 1.0
    w[200, 5] -= 30.0
    t[t == 200] = 7
    rows = torch.arange(T, device="cuda")
    d, dx, dw, xd, wd, gt = compare(x, w, t, dl, torch.arange(V, device="cuda"), rows)
    want = (d.t() @ xd)[200]
    assert 0 < float(want.norm()) < 1e-9
    assert float((dw[200].double() - want).norm()) <= gt * float(d[:, 200].norm() * torch.linalg.matrix_norm(xd, 2))


# ---------------------------------------------------------------------------
# logits far from zero
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("value", [1e4, 1e8, 1e12, 1e25])
@pytest.mark.parametrize("T", [2, 60, 300])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_masked_half_tiles(T, value, dtype):
    """All of 128 and of 256 neighbouring columns at logits of -value (a padded
    vocabulary): the exponentials of such a group's own differences from its
    maximum must not leave the range."""
    H, V = 64, 1000
    x, w, t, dl = make(T, H, V, 34)
    x, w = x.to(dtype), w.to(dtype)
    x[:, 3] = 1.0
    columns = torch.ones(V, dtype=torch.bool, device="cuda")
    columns[128:256] = False
    columns[512:768] = False
    w[~columns, 3] = -value
    keep = columns.nonzero().flatten()
    t = keep[t.long() % len(keep)].to(torch.int32)
    op = m.LinearCrossEntropy(T, H, V, dtype=dtype, reduction="none", ignore_index=IGNORE)
    loss = op.forward(x, w, t)
    dx, dw = op.backward(x, w, t, dl)
    z = x.double() @ w[keep].double().t()
    at = torch.cumsum(columns.long(), 0)[t.long()] - 1
    one = torch.nn.functional.one_hot(at, len(keep)).double()
    lse = torch.logsumexp(z, 1)
    zb = 8 * math.sqrt(H) * F * float(x.double().norm(dim=1).max() * w[keep].double().norm(dim=1).max())
    zb += 16 * F * float(z.abs().max())
    tol = 2 * zb + 8 * F * float(lse.abs().max())
    assert float((op.lse.double() - lse).abs().max()) <= tol
    assert float((loss.double() - (lse - (z * one).sum(1))).abs().max()) <= tol
    d = (torch.softmax(z, 1) - one) * dl.double()[:, None]
    gt = (2.0 ** -7 if dtype == BF else 2 * F) + 4 * zb + 16 * F
    want = d @ w[keep].double()
    assert float((dx.double() - want).norm()) <= gt * float(want.norm())
    want = d.t() @ x.double()
    assert float((dw[keep].double() - want).norm()) <= gt * float(want.norm())
    assert (dw[~columns] == 0).all()


@pytest.mark.parametrize("value", [300.0, 1e4, 1e8, 1e12, 1e25])
@pytest.mark.parametrize("T", [2, 60, 300])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_huge_logits(T, value, dtype):
    """Rows of x of norm value sqrt(H): every probability is 0 or 1 where the two
    largest logits are further apart than the sums' error."""
    H, V = 2048, 500
    x, w, t, dl = make(T, H, V, 35)
    x, w = (x * value).to(dtype), w.to(dtype)
    op = m.LinearCrossEntropy(T, H, V, dtype=dtype, reduction="none", ignore_index=IGNORE)
    loss = op.forward(x, w, t)
    dx, dw = op.backward(x, w, t, dl)
    z = x.double() @ w.double().t()
    one = torch.nn.functional.one_hot(t.long(), V).double()
    lse = torch.logsumexp(z, 1)
    zb = 8 * math.sqrt(H) * F * (x.double().norm(dim=1) * float(w.double().norm(dim=1).max()))
    zb += 16 * F * z.abs().amax(dim=1)
    tol = 2 * zb + 8 * F * lse.abs()
    assert ((op.lse.double() - lse).abs() <= tol).all()
    assert ((loss.double() - (lse - (z * one).sum(1))).abs() <= tol).all()
    assert torch.isfinite(dx.float()).all() and torch.isfinite(dw.float()).all()
    top = z.topk(2, dim=1).values
    sure = (top[:, 0] - top[:, 1]) > 2 * zb + 100.0
    sure &= z.argmax(dim=1) != t          # (p - 1 of a certain target is 0)
    assert T < 60 or int(sure.sum()) >= T // 20
    d = (torch.softmax(z, 1) - one) * dl.double()[:, None]
    want = (d @ w.double())[sure]
    gt = (2.0 ** -7 if dtype == BF else 2 * F) + 16 * F
    err = (dx[sure].double() - want).norm(dim=1)
    assert (err <= gt * want.norm(dim=1)).all()


# ---------------------------------------------------------------------------
# the objective's gradient
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("T", [2, 64, 300])
@pytest.mark.parametrize("up", [1 + 2.0 ** -8, 1 / 129.0, 3.0e-30, 65504.0 * 3])
def test_bf16_gradients_follow_the_objectives_gradient(T, up):
    """One gradient of the reduced loss scales every entry: the same factor must not be
    rounded to bf16 in each of them.  Against the gradients at 1, projected on them, the
    factor is off by the results' own roundings (at most 2^-8 each, independent) alone:
    6 sigma of their mean."""
    H, V = 256, 3000
    x, w, t, _ = make(T, H, V, 42)
    x, w = x.bfloat16(), w.bfloat16()
    op = m.LinearCrossEntropy(T, H, V, reduction="sum", ignore_index=IGNORE)
    op.forward(x, w, t)
    one = [g.double() for g in op.backward(x, w, t)]
    got = op.backward(x, w, t, torch.tensor([up], device="cuda"))
    factor = float(torch.tensor(up, dtype=FP))
    for a, b in zip(got, one):
        ratio = float((a.double() * b).sum() / (b * b).sum()) / factor
        weight = float((b ** 4).sum().sqrt() / (b * b).sum())   # of independent errors
        assert abs(ratio - 1) <= 6 * 2.0 ** -8 * weight + 4 * F, (ratio, weight)


@pytest.mark.parametrize("T", [1, 2, 3, 8, 31, 32])
def test_bf16_gradients_of_few_rows(T):
    """Up to 32 tokens the logit gradient keeps 16 bits: beside the results' rounding
    (of the exact result itself) only 2^-16 of it and the logits' error are left."""
    H, V = 264, 1500
    x, w, t, dl = make(T, H, V, 43)
    x, w = x.bfloat16(), w.bfloat16()
    op = m.LinearCrossEntropy(T, H, V, reduction="none", ignore_index=IGNORE)
    op.forward(x, w, t)
    dx, dw = op.backward(x, w, t, dl)
    xd, wd = x.double(), w.double()
    z = xd @ wd.t()
    d = (torch.softmax(z, 1) - torch.nn.functional.one_hot(t.long(), V)) * dl.double()[:, None]
    zb = 8 * math.sqrt(H) * F * float(xd.norm(dim=1).max() * wd.norm(dim=1).max()) + 16 * F * float(z.abs().max())
    for got, want in ((dx, d @ wd), (dw, d.t() @ xd)):
        own = float((want.bfloat16().double() - want).norm())
        left = (4 * zb + 2.0 ** -16 + 16 * F) * float(want.norm())
        assert float((got.double() - want).norm()) <= 1.05 * own + left


# ---------------------------------------------------------------------------
# one workspace for several shapes and operators
# ---------------------------------------------------------------------------
def router_shape(T, H, E, k, dtype=BF):
    s = m.MoEShape()
    s.tokens, s.hidden, s.moe_inter, s.topk_shape = T, H, 8, m.moe_topk_pack(E, k)
    s.norm_topk, s.dtype, s.norm_eps = 1, m.MOE_F32 if dtype == FP else m.MOE_BF16, 1e-6
    return s


def workspace(n):
    ws = torch.empty(n + 256, dtype=torch.uint8, device="cuda")
    ws.fill_(0xFF)   # NaN in whatever is read without having been written
    off = (-ws.data_ptr()) % 256
    ws = ws[off: off + n]
    m.moe_workspace_init(ws)
    return ws


def router_call(shape, ws, dtype, seed):
    T, H = shape.tokens, shape.hidden
    E, k = m.moe_topk_unpack(shape.topk_shape)
    g = gen(seed)
    x = torch.randn((T, H), generator=g, device="cuda").to(dtype)
    w = (torch.randn((E, H), generator=g, device="cuda") / math.sqrt(H)).to(dtype)
    idx = torch.randint(0, E, (T, k), generator=g, device="cuda").to(torch.int32)
    d_w = torch.randn((T, k), generator=g, device="cuda")
    dx, dw, aux = torch.empty_like(x), torch.empty_like(w), torch.empty(2, device="cuda")
    m.moe_router_backward(shape, x, w, idx, d_w, None, 0.02, 0.003, None, dx, dw, aux, ws)
    return dx, dw, aux


def ce_call(T, H, V, dtype, ws, seed):
    s = m.MoECeShape()
    s.tokens, s.hidden, s.vocab, s.dtype = T, H, V, m.MOE_F32 if dtype == FP else m.MOE_BF16
    s.reduction, s.ignore_index = m.MOE_CE_MEAN, IGNORE
    x, w, t, _ = make(T, H, V, seed)
    x, w = x.to(dtype), w.to(dtype)
    stats, total = torch.empty((T, 4), device="cuda"), torch.empty(1, device="cuda")
    dx, dw = torch.empty_like(x), torch.empty_like(w)
    ws = workspace(m.moe_linear_ce_workspace_bytes(s)) if ws is None else ws
    m.moe_linear_ce_forward(s, x, w, t, None, None, stats, total, ws)
    m.moe_linear_ce_backward(s, x, w, t, stats, None, dx, dw, ws)
    return total, dx, dw


# the kernels of a router call depend on its columns, slots and type: wide, few
# slots, many slots, many slots a token
ROUTERS = [(300, 128, 700, 5, BF), (64, 256, 60, 4, BF), (257, 64, 32, 40, BF), (16, 1024, 16, 2, BF),
           (600, 256, 64, 8, BF), (64, 128, 600, 3, FP), (64, 256, 60, 4, FP), (40, 512, 8, 1, BF)]


def test_one_workspace_for_routers_of_any_shape():
    shapes = [router_shape(*r) for r in ROUTERS]
    ws = workspace(max(m.moe_router_backward_workspace_bytes(s) for s in shapes))
    fresh = [router_call(s, workspace(m.moe_router_backward_workspace_bytes(s)), r[4], i)
             for i, (s, r) in enumerate(zip(shapes, ROUTERS))]
    order = [0, 1, 2, 3, 0, 3, 5, 1, 4, 2, 7, 6, 0, 7, 5, 3, 1]
    for i in order:
        got = router_call(shapes[i], ws, ROUTERS[i][4], i)
        for a, b in zip(got, fresh[i]):
            assert torch.isfinite(a.float()).all(), i
            assert torch.equal(a, b), i
    assert m.moe_get_device_status(ws)[0] == m.MOE_OK


def test_one_workspace_for_the_layer_and_the_training_operators():
    wl = W.small(W.QWEN3_30B_A3B, T=64, H=256, I=128, E=16, k=2)
    dev = W.make_inputs(wl, seed=0, device="cuda")
    layer = m.MoELayer(wl, dev)
    shapes = [router_shape(*r) for r in ROUTERS[:4]]
    ces = [(1, 256, 900, BF), (300, 128, 2000, BF), (3, 64, 500, FP), (70, 64, 500, FP)]
    n = max([layer.ws.numel()] + [m.moe_router_backward_workspace_bytes(s) for s in shapes] + [64 << 20])
    y = layer.forward(dev["x"])
    ce = [ce_call(*c, None, i) for i, c in enumerate(ces)]
    ro = [router_call(s, workspace(m.moe_router_backward_workspace_bytes(s)), BF, i) for i, s in enumerate(shapes)]
    layer.ws = workspace(n)
    for i in [0, 1, 2, 3, 0, 1, 3, 2]:
        assert torch.equal(layer.forward(dev["x"]), y)
        assert all(torch.equal(a, b) for a, b in zip(ce_call(*ces[i], layer.ws, i), ce[i])), i
        assert all(torch.equal(a, b) for a, b in zip(router_call(shapes[i], layer.ws, BF, i), ro[i])), i
    assert layer.device_status()[0] == m.MOE_OK


# ---------------------------------------------------------------------------
# dropped routes
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("E,k", [(16, 3), (16, 33), (700, 3)])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
def test_a_dropped_route_may_hold_any_gradient(E, k, norm, bad):
    """k = 3 and E = 16 take the kernel for few columns, the others the general one."""
    T, H = 90, 128
    g = gen(5)
    x = torch.randn((T, H), generator=g, device="cuda").bfloat16()
    w = (torch.randn((E, H), generator=g, device="cuda") / math.sqrt(H)).bfloat16()
    idx = torch.randint(0, E, (T, k), generator=g, device="cuda").to(torch.int32)
    d_w = torch.randn((T, k), generator=g, device="cuda")
    idx[4, 1], idx[7, 0], idx[9], idx[80, 2] = E, -1, -7, 2 ** 31 - 1
    gone = (idx < 0) | (idx >= E)
    out = []
    for v in (0.0, bad):
        d_w[gone] = v
        op = m.RouterGrad(T, H, E, k, norm_topk=norm, balance_coef=0.01, z_coef=0.001)
        out.append(op.backward(x, w, idx, d_w))
        assert op.device_status()[0] == m.MOE_ERR_DEVICE_ROUTE
    for a, b in zip(*out):
        assert torch.isfinite(b.float()).all()
        assert torch.equal(a, b)


# ---------------------------------------------------------------------------
# very many tokens
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [BF, FP])
def test_packing_of_several_hundred_thousand_tokens(dtype):
    """Above 2^18 tokens: losses per token, and dx and dw, against float64.  bf16
    gradients: 2^-8 twice; the fp32 sums over the rows (586 chunks of 512, in each 32
    truncated steps) add at worst 650 f, 2^-14."""
    T, H, V = 300011, 16, 40
    x, w, t, dl = make(T, H, V, 41)
    x, w = x.to(dtype), w.to(dtype)
    t[torch.rand(T, generator=gen(2), device="cuda") < 0.3] = IGNORE
    t[:300] = IGNORE
    t[-1] = 3
    op = m.LinearCrossEntropy(T, H, V, dtype=dtype, reduction="none", ignore_index=IGNORE)
    loss = op.forward(x, w, t)
    dx, dw = op.backward(x, w, t, dl)
    ok = t != IGNORE
    z = x.double() @ w.double().t()
    one = torch.nn.functional.one_hot(t.long().clamp(min=0), V).double()
    lse = torch.logsumexp(z, 1)
    want = (lse - (z * one).sum(1)) * ok
    zb = 8 * math.sqrt(H) * F * float(x.double().norm(dim=1).max() * w.double().norm(dim=1).max())
    zb += 16 * F * float(z.abs().max())
    assert float((loss.double() - want).abs().max()) <= 2 * zb + 8 * F * float(lse.abs().max())
    d = (torch.softmax(z, 1) - one) * (dl * ok).double()[:, None]
    tol = (2.0 ** -7 if dtype == BF else 2 * F) + 4 * zb + 16 * F + 2.0 ** -14
    for got, ref in ((dx, d @ w.double()), (dw, d.t() @ x.double())):
        assert float((got.double() - ref).norm()) <= tol * float(ref.norm())
    assert (dx[~ok] == 0).all()


def test_packing_time_grows_with_the_tokens():
    """Eight times the tokens cost about eight times the time (the packing must not
    count every token in every block): at most sixteen are allowed."""
    def time(T):
        x = torch.randn((T, 8), device="cuda").bfloat16()
        w = torch.randn((2, 8), device="cuda").bfloat16()
        t = torch.zeros(T, device="cuda", dtype=torch.int32)
        op = m.LinearCrossEntropy(T, 8, 2, reduction="sum")
        total = torch.empty(1, device="cuda")
        best = math.inf
        for _ in range(6):
            a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
            a.record()
            op.forward(x, w, t, total=total)
            b.record()
            b.synchronize()
            best = min(best, a.elapsed_time(b))
        return best
    assert time(1 << 22) <= 16 * time(1 << 19)


# ---------------------------------------------------------------------------
# the Python classes
# ---------------------------------------------------------------------------
def test_clip_of_a_generator():
    grads = [torch.randn(1000, device="cuda") for _ in range(3)]
    want = math.sqrt(sum(float(g.double().square().sum()) for g in grads))
    op = m.GradClip(g for g in grads)
    keep = [g.clone() for g in grads]
    assert abs(float(op.clip(1.0)) - want) <= 64 * F * want
    for g, k in zip(grads, keep):
        assert torch.allclose(g, k / want, rtol=1e-5, atol=0)


def test_outputs_are_made_on_the_stream_that_writes_them():
    """A block that the current stream has just freed may still be in use there, so
    an output for another stream must not come from it."""
    T, H, V, E, k = 512, 512, 2048, 16, 2
    x, w, t, _ = make(T, H, V, 3)
    x, w = x.bfloat16(), w.bfloat16()
    wr = w[:E].contiguous()
    idx = torch.randint(0, E, (T, k), device="cuda").to(torch.int32)
    d_w = torch.randn((T, k), device="cuda")
    ce = m.LinearCrossEntropy(T, H, V, reduction="none")
    ro = m.RouterGrad(T, H, E, k)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()

    def freed(numel, dtype):
        b = torch.empty(numel, dtype=dtype, device="cuda")
        return b.data_ptr()

    calls = [(T, FP, lambda s: ce.forward(x, w, t, stream=s)),
             (V * H, BF, lambda s: ce.backward(x, w, t, d_w[:, 0].contiguous(), stream=s)[1]),
             (T * H, BF, lambda s: ro.backward(x, wr, idx, d_w, stream=s)[0])]
    for numel, dtype, call in calls:
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        at = freed(numel, dtype)
        assert freed(numel, dtype) == at        # the current stream takes it again
        for s in (side, side.cuda_stream):
            out = call(s)
            torch.cuda.synchronize()
            assert not at <= out.data_ptr() < at + numel * out.element_size()
            del out
    layer_ws = m.GradClip([d_w], stream=side)
    torch.cuda.synchronize()
    assert float(layer_ws.clip(math.inf, stream=side)) > 0

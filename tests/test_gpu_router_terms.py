"""The router's gradient on the GPU, one term of the objective at a time, so that no
other term's size hides it: the balance loss, the z loss, the routing weights and the
shared gate, each against its formula in float64, without dx_add, and each test's
tolerance shown to be far below the term itself.

Bounds (derived).  f = 2^-24, u = 2^-8 (bf16) or f.
 * logits: zb = 8 sqrt(H) f max|x| max|w| + 2 f (H / 16) max|z| (fp32 sums; the tensor
   cores cut off at each of H / 16 steps).
 * dz against U, the sum of the absolute values it is made of: each of p, w and lse
   carries two logits' errors, a term at most two of them: 4 zb, 32 f for exponentials,
   quotients and sums, and what the planes leave (bf16: two of them, 2^-16; fp32: f).
 * the products: |E B| <= |E| s(B) in the Frobenius norm, s the largest singular value;
   their sums are cut off at each K / 16 step: 2 f (K / 16 + 8) |U| s(B).
 * the result is rounded once: u of its norm.
"""
import math

import pytest
import torch

import mixture_experts_ffn_04_gb300 as m

F = 2.0 ** -24
U = {torch.bfloat16: 2.0 ** -8, torch.float32: F}

# few slots (the dz kernel counts them itself), many slots with the histogram of one
# block and of a cluster, more columns than the small kernel takes, more slots a token
SHAPES = [(64, 264, 60, 4), (600, 256, 32, 4), (257, 1032, 128, 8), (1000, 256, 256, 8), (300, 128, 700, 5),
          (120, 64, 64, 40)]
TERMS = ["balance", "z", "weights", "gate"]


def make(T, H, E, k, dtype, device, seed=0):
    g = torch.Generator()
    g.manual_seed(seed + T + E)
    x = torch.randn((T, H), generator=g).to(dtype)
    w = (torch.randn((E + 1, H), generator=g) / math.sqrt(H)).to(dtype)
    idx = (x.float() @ w[:E].float().t()).topk(k, dim=1).indices.to(torch.int32).contiguous()
    d_w, d_gate = torch.randn((T, k), generator=g), torch.randn((T,), generator=g)
    return [t.to(device) for t in (x, w, idx, d_w, d_gate)]


def term(name, x, w, idx, d_w, d_gate, norm, E, coef):
    """dz of one term, U, the losses, and the router's rows that it uses."""
    T, k = idx.shape
    xd, at = x.double(), idx.long()
    z = xd @ w.double().t()
    ze = z[:, :E]
    p, lse = torch.softmax(ze, 1), torch.logsumexp(ze, 1)
    dz, ab = torch.zeros_like(z), torch.zeros_like(z)
    aux = torch.zeros(2, dtype=torch.float64, device=x.device)
    if name == "balance":
        n = torch.bincount(at.flatten(), minlength=E).double()
        pn = (p * n).sum(1, keepdim=True)
        cb = coef * E / (T * T * k)
        dz[:, :E], ab[:, :E] = cb * p * (n - pn), cb * p * (n + pn)
        aux[0] = cb * pn.sum()
    elif name == "z":
        dz[:, :E] = 2 * coef / T * lse[:, None] * p
        ab = dz.abs()
        aux[1] = coef * lse.square().mean()
    elif name == "gate":
        s = torch.sigmoid(z[:, E])
        dz[:, E] = d_gate.double() * s * (1 - s)
        ab = dz.abs()
    else:
        D = d_w.double()
        wt = torch.softmax(ze.gather(1, at), 1) if norm else p.gather(1, at)
        dot = (wt * D).sum(1, keepdim=True)
        add = (wt * D.abs()).sum(1, keepdim=True)
        zero = torch.zeros_like(ze)
        if norm:
            dz[:, :E] = zero.scatter_add(1, at, wt * (D - dot))
            ab[:, :E] = zero.scatter_add(1, at, wt * (D.abs() + add))
        else:
            dz[:, :E] = zero.scatter_add(1, at, wt * D) - p * dot
            ab[:, :E] = zero.scatter_add(1, at, wt * D.abs()) + p * add
    return dz, ab, aux, z


def expected(name, x, w, idx, d_w, d_gate, norm, E, coef):
    """(dx, tolerance), (dw, tolerance), losses and their tolerances."""
    T, H = x.shape
    dz, ab, aux, z = term(name, x, w, idx, d_w, d_gate, norm, E, coef)
    xd, wd = x.double(), w.double()
    zb = 8 * math.sqrt(H) * F * float(xd.norm(dim=1).max() * wd.norm(dim=1).max())
    zb += H / 16 * 2 * F * float(z.abs().max())
    e = 4 * zb + 32 * F + (2.0 ** -16 if x.dtype == torch.bfloat16 else F)
    out = []
    for want, K, B in ((dz @ wd, w.shape[0], wd), (dz.t() @ xd, T, xd)):
        size = float(ab.norm()) * float(torch.linalg.matrix_norm(B, 2))
        out.append((want, (e + 2 * F * (K / 16 + 8)) * size + U[x.dtype] * float(want.norm())))
    return out[0], out[1], aux, (4 * zb + 32 * F) * aux


def resolved(want, tol):
    """Leaving the term out, or a tenth of it, would be seen."""
    return tol <= 0.1 * float(want.norm())


@pytest.mark.parametrize("T,H,E,k", SHAPES)
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("name", TERMS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_the_bounds_resolve_each_term(T, H, E, k, norm, name, dtype):
    """On the CPU: the GPU test below would notice the term's absence."""
    x, w, idx, d_w, d_gate = make(T, H, E, k, dtype, "cpu")
    (dx, tx), (dw, tw), _, _ = expected(name, x, w, idx, d_w, d_gate, norm, E, 0.5)
    assert resolved(dx, tx) and resolved(dw, tw), (tx / float(dx.norm()), tw / float(dw.norm()))


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,E,k", SHAPES)
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("name", TERMS)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_one_term_alone(T, H, E, k, norm, name, dtype):
    x, w, idx, d_w, d_gate = make(T, H, E, k, dtype, "cuda")
    rdx, rdw, raux, taux = expected(name, x, w, idx, d_w, d_gate, norm, E, 0.5)
    op = m.RouterGrad(T, H, E, k, norm_topk=norm, shared_gate=True, dtype=dtype,
                      balance_coef=0.5 if name == "balance" else 0.0, z_coef=0.5 if name == "z" else 0.0)
    gate = d_gate if name == "gate" else torch.zeros_like(d_gate)
    dx, dw, aux = op.backward(x, w, idx, d_w if name == "weights" else None, d_gate=gate)
    for got, (want, tol) in ((dx, rdx), (dw, rdw)):
        assert torch.isfinite(got.float()).all()
        assert float((got.double() - want).norm()) <= tol
    assert ((aux.double() - raux).abs() <= taux + 1e-30).all()


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,E,k", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_dx_add_of_the_terms_own_size(T, H, E, k, dtype):
    """dx_add as large as the router's part, so that neither hides the other."""
    x, w, idx, d_w, d_gate = make(T, H, E, k, dtype, "cuda", seed=1)
    (want, tol), _, _, _ = expected("weights", x, w, idx, d_w, d_gate, True, E, 0.0)
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    add = (torch.randn((T, H), generator=g, device="cuda") * float(want.norm()) / math.sqrt(T * H)).to(dtype)
    op = m.RouterGrad(T, H, E, k, norm_topk=True, shared_gate=True, dtype=dtype)
    dx, _, _ = op.backward(x, w, idx, d_w, d_gate=torch.zeros_like(d_gate), dx_add=add)
    whole = want + add.double()
    # the sum is rounded instead of the part; its K / 16 steps start from the addend
    tol += U[dtype] * float(whole.norm()) + 2 * F * ((E + 1) / 16 + 8) * float(add.double().norm())
    assert float((dx.double() - whole).norm()) <= tol
    assert tol <= 0.1 * float(want.norm()) and tol <= 0.1 * float(add.double().norm())

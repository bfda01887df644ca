"""The router's gradient on the GPU against the definition in float64 (autograd
of the weights, the gate and both losses).

Bounds (derived): u = eps / 2 of the layer's type, f = 2^-24.
 * logits: fp32 sums, |error| <= zb = 8 sqrt(H) f max|x| max|w| (2-norms of rows);
   tensor cores cut the accumulator off at each of H / 16 steps: + H / 16 * 2 f
   max|z|.
 * dz carries relative errors of a few zb (each p and w is an exponential of
   differences of logits) and one rounding u (fp32: three planes, below f); the
   products round once more: relative L2 of dx and dw at most 2 u + 8 zb + 32 f,
   the 32 f for the exponentials, quotients and sums.  The differences n_e - sum
   n p and w (D - dot) may cancel, so errors count against the uncancelled sizes:
   the test adds their matrices' norms instead of the result's where larger.
 * losses: sums of positive terms: relative 2 zb (lse^2: an absolute zb in lse,
   |lse| >= 1 here) + 16 f.
"""
import math

import pytest
import torch

import mixture_experts_ffn_04_gb300 as m

pytestmark = pytest.mark.gpu
F = 2.0 ** -24
U = {torch.bfloat16: 2.0 ** -8, torch.float32: F}


def make(T, H, E, k, gate, dtype, seed=0, dup=False):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda")
    x, w = rnd(T, H).to(dtype), (rnd(E + int(gate), H) / math.sqrt(H)).to(dtype)
    if dup:
        idx = torch.randint(0, E, (T, k), generator=g, device="cuda").to(torch.int32)
    else:
        idx = (x.float() @ w[:E].float().t()).topk(k, dim=1).indices.to(torch.int32).contiguous()
    return x, w, idx, rnd(T, k), (rnd(T) if gate else None), rnd(T, H).to(dtype)


def reference(x, w, idx, d_w, d_gate, dx_add, norm, bal, zc, E):
    T, k = idx.shape
    xd, wd = x.double().requires_grad_(True), w.double().requires_grad_(True)
    z = xd @ wd.t()
    ze, ok = z[:, :E], (idx >= 0) & (idx < E)
    at = idx.long().clamp(0, E - 1)
    sel = ze.gather(1, at).masked_fill(~ok, -math.inf)
    p = torch.softmax(ze, 1)
    if norm:
        full = sel - sel.amax(1, keepdim=True).clamp(min=-1e30)
        wts = torch.exp(full) / torch.exp(full).sum(1, keepdim=True).clamp(min=1e-300)
    else:
        wts = p.gather(1, at) * ok
    n = torch.bincount(at[ok], minlength=E).double()
    lb = bal * E * (n / (T * k) * p.mean(0)).sum()
    lz = zc * torch.logsumexp(ze, 1).square().mean()
    obj = lb + lz
    if d_w is not None:
        obj = obj + (wts * d_w.double() * ok).sum()
    if d_gate is not None:
        obj = obj + (torch.sigmoid(z[:, E]) * d_gate.double()).sum()
    dx, dw = torch.autograd.grad(obj, [xd, wd])
    if dx_add is not None:
        dx = dx + dx_add.double()
    H = x.shape[1]
    zb = 8 * math.sqrt(H) * F * float(x.double().norm(dim=1).max() * w.double().norm(dim=1).max())
    zb += H / 16 * 2 * F * float(z.detach().abs().max())
    return dx, dw, torch.stack([lb, lz]).detach(), zb


def check(x, w, idx, d_w, d_gate, dx_add, E, k, norm, bal=0.02, zc=0.003):
    T, H = x.shape
    op = m.RouterGrad(T, H, E, k, norm_topk=norm, shared_gate=d_gate is not None, dtype=x.dtype,
                      balance_coef=bal, z_coef=zc)
    dx, dw, aux = op.backward(x, w, idx, d_w, d_gate=d_gate, dx_add=dx_add)
    rdx, rdw, raux, zb = reference(x, w, idx, d_w, d_gate, dx_add, norm, bal, zc, E)
    tol = 2 * U[x.dtype] + 8 * zb + 32 * F
    for got, want in ((dx, rdx), (dw, rdw)):
        assert torch.isfinite(got.float()).all()
        big = float(want.norm())
        if d_w is not None:   # uncancelled size of the slots' terms
            big = max(big, float(d_w.double().norm()) * 0.05)
        assert float((got.double() - want).norm()) <= tol * big
    assert ((aux.double() - raux).abs() <= (2 * zb + 16 * F) * raux.abs() + 1e-12).all()
    return op, dx, dw, aux


@pytest.mark.parametrize("T,H,E,k", [(1, 64, 8, 2), (3, 256, 16, 1), (63, 264, 60, 4), (65, 512, 61, 8),
                                     (257, 1032, 128, 8), (1000, 256, 256, 8), (300, 128, 700, 5),
                                     (64, 64, 1, 1)])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_shapes(T, H, E, k, norm, gate, dtype):
    x, w, idx, d_w, d_gate, add = make(T, H, E, k, gate, dtype, seed=T + E)
    check(x, w, idx, d_w, d_gate, add, E, k, norm)


@pytest.mark.parametrize("norm", [True, False])
def test_repeated_routes(norm):
    x, w, idx, d_w, _, add = make(200, 128, 8, 6, False, torch.float32, dup=True)
    idx[5] = 3
    check(x, w, idx, d_w, None, add, 8, 6, norm)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_optional_inputs(dtype):
    x, w, idx, d_w, _, add = make(130, 192, 32, 4, False, dtype)
    check(x, w, idx, None, None, add, 32, 4, True)
    check(x, w, idx, d_w, None, None, 32, 4, False, bal=0.0, zc=0.0)
    check(x, w, idx, d_w, None, None, 32, 4, False, bal=0.0, zc=0.01)


def test_dx_add_in_place():
    x, w, idx, d_w, _, add = make(300, 256, 64, 4, False, torch.bfloat16)
    op, dx, dw, aux = check(x, w, idx, d_w, None, add, 64, 4, True)
    buf = add.clone()
    out = op.backward(x, w, idx, d_w, dx_add=buf, dx=buf)
    assert out[0] is buf and torch.equal(buf, dx) and torch.equal(out[1], dw)


def test_routes_out_of_range_are_dropped_and_flagged():
    x, w, idx, d_w, _, add = make(90, 128, 16, 3, False, torch.float32)
    idx[4, 1], idx[7, 0], idx[9] = 16, -1, -1
    op, *_ = check(x, w, idx, d_w, None, add, 16, 3, False)
    assert op.device_status()[0] == m.MOE_ERR_DEVICE_ROUTE


def test_no_tokens():
    op = m.RouterGrad(0, 64, 8, 2)
    x = torch.empty((0, 64), device="cuda", dtype=torch.bfloat16)
    w = torch.randn((8, 64), device="cuda").bfloat16()
    idx = torch.empty((0, 2), device="cuda", dtype=torch.int32)
    dx, dw, aux = op.backward(x, w, idx, torch.empty((0, 2), device="cuda"))
    assert (dw == 0).all() and (aux == 0).all()


def test_many_experts():
    """More router columns than eight warps' shared memory holds."""
    x, w, idx, d_w, _, add = make(40, 64, 9000, 4, False, torch.float32)
    check(x, w, idx, d_w, None, add, 9000, 4, True)


def test_against_the_layers_own_routing_and_graph():
    """idx and weights from moe_route; the same bits on replay and repetition."""
    T, H, E, k = 500, 256, 32, 4
    x, w, idx, d_w, d_gate, add = make(T, H, E, k, True, torch.bfloat16)
    op, dx, dw, aux = check(x, w, idx, d_w, d_gate, add, E, k, True)
    for _ in range(2):
        o = op.backward(x, w, idx, d_w, d_gate=d_gate, dx_add=add)
        assert all(torch.equal(p, q) for p, q in zip(o, (dx, dw, aux)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = op.backward(x, w, idx, d_w, d_gate=d_gate, dx_add=add)
    d_w.mul_(-2.0)
    graph.replay()
    c = check(x, w, idx, d_w, d_gate, add, E, k, True)
    assert all(torch.equal(p, q) for p, q in zip(o, c[1:]))

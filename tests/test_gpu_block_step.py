"""The step of one block from token ids, with every operator together, against one
float64 autograd graph of it.

Bounds (derived): u = 2^-8.  The step around the layer (test_gpu_train_step.py) has at
most 12 roundings of u on a path; the embedding, the two norms and their gradients add
x, h, s, z, dz, dy, dx (twice) and the table's gradient (twice): 22 in all, independent, so
sqrt(22) u, plus the forward's roundings acting through the gradients' own inputs, another
sqrt(9) u: 8 u in all, relative to each gradient's norm.  The loss: each logit moves by at
most 2 u |z| |w| / sqrt(H) in random directions; averaged over the tokens
8 u / sqrt(T) |z| |w|.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -8


def reference(s, k, bal, zc, padding_idx):
    """Loss and gradients in float64, with the routes the layer took."""
    p = {n: t.double().requires_grad_(True) for n, t in s.params.items()}
    F = torch.nn.functional
    rms = lambda v, w: v * torch.rsqrt(v.square().mean(1, keepdim=True) + 1e-6) * w
    x = F.embedding(s.ids.long(), p["table"], padding_idx=padding_idx) * s.scale
    T, H = x.shape
    E = p["gate"].shape[0]
    idx = s.topk_idx.long()
    h = rms(x, p["norm_in"])
    zr = h @ p["router"].t()
    wts = torch.softmax(zr.gather(1, idx), 1)
    a = torch.einsum("th,eih->tei", h, p["gate"])
    b = torch.einsum("th,eih->tei", h, p["up"])
    o = torch.einsum("tei,ehi->teh", F.silu(a) * b, p["down"])
    y = (wts[:, :, None] * o.gather(1, idx[:, :, None].expand(-1, -1, H))).sum(1)
    z = rms(x + p["channel_gate"] * rms(y, p["norm_post"]), p["norm_out"])
    loss = F.cross_entropy(z @ p["table"].t(), s.target.long(), ignore_index=-100)
    share = torch.bincount(idx.flatten(), minlength=E).double() / (T * k)
    lb = bal * E * (share * torch.softmax(zr, 1).mean(0)).sum()
    lz = zc * torch.logsumexp(zr, 1).square().mean()
    (loss + lb + lz).backward()
    return loss.detach(), {n: t.grad for n, t in p.items()}, z.detach()


@pytest.mark.parametrize("padding", [None, 3])
def test_step_against_autograd(padding):
    from mixture_experts_ffn_04_gb300.train_step import BlockStep
    s = BlockStep(T=200, H=128, I=64, E=8, k=2, V=300, max_norm=1e9, padding_idx=padding)
    if padding is not None:
        s.ids[::9] = padding
    s.gradients()
    assert all(st == (0, 0) for st in s.device_status())
    loss, g, z = reference(s, 2, 0.01, 0.001, padding)
    zw = float(z.norm(dim=1).max() * s.params["table"].double().norm(dim=1).max())
    assert abs(float(s.loss) - float(loss)) <= 8 * U / math.sqrt(200) * zw
    for n, want in g.items():
        err = float((s.grads[n].double() - want).norm() / want.norm())
        assert err <= 8 * U, (n, err)


def test_steps_and_replay_in_a_graph():
    """The step runs, stays finite, moves every parameter, and its gradients and the
    experts' update are the same bits from a graph."""
    from mixture_experts_ffn_04_gb300.train_step import BlockStep
    s, q = BlockStep(seed=1), BlockStep(seed=1)
    before = {n: p.clone() for n, p in s.params.items()}
    s.step(0.5)
    assert math.isfinite(float(s.loss)) and all(st == (0, 0) for st in s.device_status())
    for n, p in s.params.items():
        assert bool(torch.isfinite(p).all()) and not torch.equal(p, before[n]), n
    q.gradients()     # first calls outside the capture
    q.muon.step()
    for n, p in q.params.items():
        p.copy_(before[n])
    for v in q.muon.momenta:
        v.zero_()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        q.gradients()
        q.muon.step()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(q.loss, s.loss)
    for n in ("gate", "up", "down"):
        assert torch.equal(q.params[n], s.params[n]) and torch.equal(q.grads[n], s.grads[n])
    assert torch.equal(q.grads["table"], s.grads["table"])

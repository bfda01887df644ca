"""The training step with every operator together, against one float64 autograd
graph of the whole step.

Bounds (derived): u = 2^-8.  The layer rounds h, y_perm, y and, in the backward,
grad_fc2, d_fc1, dx_perm and dx to bf16 (at most 8 roundings on a path, each u
relative to its own vector), the cross entropy its logit gradient and dy, the
router its results: at most 12 roundings of u on the longest path, independent, so
relative L2 errors below sqrt(12) u plus the effect of the forward's rounding on
the gradients' own inputs, another sqrt(4) u: 6 u in all.  The loss: an fp32 sum
over y, whose rounding moves each logit by at most u |y| |w| / sqrt(H) in random
directions; averaged over the tokens 4 u / sqrt(T) |y||w|.
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu
U = 2.0 ** -8


def reference(s, k, bal, zc):
    """Loss and gradients in float64, with the routes the layer took."""
    p = {n: t.double().requires_grad_(True) for n, t in s.params.items()}
    x = s.x.double().requires_grad_(True)
    T, H = x.shape
    E = p["gate"].shape[0]
    idx = s.topk_idx.long()
    z = x @ p["router"].t()
    wts = torch.softmax(z.gather(1, idx), 1)
    a = torch.einsum("th,eih->tei", x, p["gate"])
    b = torch.einsum("th,eih->tei", x, p["up"])
    o = torch.einsum("tei,ehi->teh", torch.nn.functional.silu(a) * b, p["down"])
    pick = o.gather(1, idx[:, :, None].expand(-1, -1, H))
    y = x + (wts[:, :, None] * pick).sum(1)
    loss = torch.nn.functional.cross_entropy(y @ p["vocab"].t(), s.target.long(), ignore_index=-100)
    share = torch.bincount(idx.flatten(), minlength=E).double() / (T * k)
    lb = bal * E * (share * torch.softmax(z, 1).mean(0)).sum()
    lz = zc * torch.logsumexp(z, 1).square().mean()
    (loss + lb + lz).backward()
    return loss.detach(), lb.detach(), lz.detach(), x.grad, {n: t.grad for n, t in p.items()}


def test_step_against_autograd():
    from mixture_experts_ffn_04_gb300.train_step import TrainStep
    s = TrainStep(T=200, H=128, I=64, E=8, k=2, V=700, max_norm=1e9)
    s.gradients()
    assert all(st == (0, 0) for st in s.device_status())
    loss, lb, lz, dx, g = reference(s, 2, 0.01, 0.001)
    yw = float(s.y.double().norm(dim=1).max() * s.w_vocab.double().norm(dim=1).max())
    assert abs(float(s.loss) - float(loss)) <= 4 * U / math.sqrt(200) * yw
    assert abs(float(s.aux[0]) - float(lb)) <= 1e-5 and abs(float(s.aux[1]) - float(lz)) <= 1e-5
    norm = math.sqrt(sum(float(t.square().sum()) for t in g.values()))
    assert abs(float(s.norm) - norm) <= 6 * U * norm
    for n, want in [("dx", dx)] + list(g.items()):
        got = s.dx if n == "dx" else s.grads[n]
        err = float((got.double() - want).norm() / want.norm())
        assert err <= 6 * U, (n, err)


def test_steps_lower_the_loss_and_replay_in_a_graph():
    from mixture_experts_ffn_04_gb300.train_step import TrainStep
    s = TrainStep()
    s.step(2.0)
    first = float(s.loss)
    for _ in range(15):
        s.step(2.0)
    assert float(s.loss) < first - 0.2
    # the same step as a graph: the same bits
    s.gradients()
    keep = [t.clone() for t in [s.loss, s.norm, s.dx] + list(s.grads.values())]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s.gradients()
    for t in [s.loss, s.norm, s.dx] + list(s.grads.values()):
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(keep, [s.loss, s.norm, s.dx] + list(s.grads.values())))

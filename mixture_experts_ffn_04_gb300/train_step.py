"""A training step around one MoE layer, with every operator of the library that
takes part in it:

    y = x + MoE(x)                       moe_layer_forward (train)
    loss = cross entropy(y . w^T)        moe_linear_ce_forward
    dy, dw                               moe_linear_ce_backward
    dx, d_topk_w, expert gradients       moe_layer_backward
    dx += router's part, dw_router       moe_router_backward (+ balance, z loss)
    norm, clipped gradients              moe_grad_clip
    parameters -= lr * gradient          (plain SGD, torch)

    python -m mixture_experts_ffn_04_gb300.train_step --steps 20

trains the layer, its router and a vocabulary on one synthetic batch (random
rows, random targets) and prints loss, balance loss and gradient norm.  With
--block the step goes from token ids to the same table as classifier, through the
norms around the layer, and the experts are updated by their orthogonalised momentum:

    x = scale * table[id]                moe_embed_forward
    h = norm(x)                          moe_block_norm_forward
    y = MoE(h)
    s = x + gate * norm(y), z = norm(s)  moe_block_norm_forward
    loss = cross entropy(z . table^T)
    ...                                  and back, dtable from both of its uses
    experts                              moe_muon_step
"""
from __future__ import annotations

import argparse
import math

import torch

import mixture_experts_ffn_04_gb300 as m
from mixture_experts_ffn_04_gb300 import workloads as W


class TrainStep:
    """Parameters, gradients and operators of the step; all tensors stay where
    they are, so step() can be captured in a CUDA graph."""

    def __init__(self, T=512, H=256, I=128, E=16, k=4, V=5000, seed=0, balance_coef=0.01,
                 z_coef=0.001, max_norm=1.0, ignore_index=-100):
        wl = W.small(W.QWEN3_30B_A3B, T=T, H=H, I=I, E=E, k=k)
        inp = W.make_inputs(wl, seed=seed, device="cpu")
        dev = {n: (t.cuda() if t is not None else None) for n, t in inp.items()}
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        self.max_norm = max_norm
        self.x = dev["x"]
        self.target = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
        self.target[::7] = ignore_index
        self.w_vocab = (torch.randn((V, H), generator=g, device="cuda") / math.sqrt(H)).bfloat16()
        self.layer = m.MoELayer(wl, dev, train=True)
        self.layer.shape.residual = 1
        self.params = {"gate": dev["w_gate"], "up": dev["w_up"], "down": dev["w_down"],
                       "router": dev["w_router"], "vocab": self.w_vocab}
        self.grads = {n: torch.empty_like(p) for n, p in self.params.items()}
        self.ce = m.LinearCrossEntropy(T, H, V, reduction="mean", ignore_index=ignore_index)
        self.router = m.RouterGrad(T, H, E, k, norm_topk=bool(wl.norm_topk),
                                   balance_coef=balance_coef, z_coef=z_coef)
        self.clip = m.GradClip(list(self.grads.values()))
        self.y, self.dy = torch.empty_like(self.x), torch.empty_like(self.x)
        self.dx = torch.empty_like(self.x)
        self.d_topk_w = torch.empty((T, k), device="cuda")
        self.loss = torch.empty(1, device="cuda")
        self.aux = torch.empty(2, device="cuda")
        self.norm = torch.empty(1, device="cuda")
        self.topk_idx = self.layer.views()["topk_idx"]

    def gradients(self):
        """Loss, gradients of every parameter and of x, clipped."""
        g = self.grads
        self.layer.forward(self.x, y=self.y)
        self.ce.forward(self.y, self.w_vocab, self.target, total=self.loss)
        self.ce.backward(self.y, self.w_vocab, self.target, dx=self.dy, dw=g["vocab"])
        self.layer.backward(self.dy, self.dx, self.d_topk_w,
                            m.grads_for(g["gate"], g["up"], g["down"]))
        self.router.backward(self.x, self.params["router"], self.topk_idx, self.d_topk_w,
                             dx_add=self.dx, dx=self.dx, dw_router=g["router"], aux=self.aux)
        self.clip.clip(self.max_norm, norm=self.norm)

    def step(self, lr: float):
        self.gradients()
        for n, p in self.params.items():
            p.add_(self.grads[n], alpha=-lr)

    def device_status(self):
        return [o.device_status() for o in (self.layer, self.ce, self.router)]


class BlockStep:
    """The step of a model of one block between a token embedding and the classifier
    that shares its table; tensors stay where they are, as in TrainStep."""

    def __init__(self, T=512, H=256, I=128, E=16, k=4, V=5000, seed=0, balance_coef=0.01,
                 z_coef=0.001, max_norm=1.0, ignore_index=-100, padding_idx=None, lr=0.02):
        wl = W.small(W.QWEN3_30B_A3B, T=T, H=H, I=I, E=E, k=k)
        inp = W.make_inputs(wl, seed=seed, device="cpu")
        dev = {n: (t.cuda() if t is not None else None) for n, t in inp.items()}
        g = torch.Generator(device="cuda")
        g.manual_seed(seed)
        bf16 = torch.bfloat16
        self.max_norm, self.lr, self.scale = max_norm, lr, math.sqrt(H)
        self.ids = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
        self.target = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
        self.target[::7] = ignore_index
        self.layer = m.MoELayer(wl, dev, train=True)
        self.params = {"gate": dev["w_gate"], "up": dev["w_up"], "down": dev["w_down"],
                       "router": dev["w_router"],
                       "table": (torch.randn((V, H), generator=g, device="cuda") / math.sqrt(H)).to(bf16)}
        for n in ("norm_in", "norm_post", "norm_out", "channel_gate"):
            self.params[n] = (1.0 + 0.1 * torch.randn(H, generator=g, device="cuda")).to(bf16)
        self.grads = {n: torch.empty_like(p) for n, p in self.params.items()}
        self.emb = m.TokenEmbedding(T, H, V, scale=self.scale, padding_idx=padding_idx)
        self.before = m.BlockNorm(T, H)
        self.after = m.BlockNorm(T, H, gate="channel")
        self.ce = m.LinearCrossEntropy(T, H, V, reduction="mean", ignore_index=ignore_index)
        self.router = m.RouterGrad(T, H, E, k, norm_topk=bool(wl.norm_topk),
                                   balance_coef=balance_coef, z_coef=z_coef)
        self.clip = m.GradClip(list(self.grads.values()))
        experts = ("gate", "up", "down")
        self.muon = m.Muon([self.params[n] for n in experts], [self.grads[n] for n in experts], lr=lr)
        self.rest = [n for n in self.params if n not in experts]

        def rows():
            return torch.empty((T, H), device="cuda", dtype=bf16)

        self.x, self.h, self.y, self.s, self.z = rows(), rows(), rows(), rows(), rows()
        self.dx, self.dh, self.dy, self.dz = rows(), rows(), rows(), rows()
        self.d_topk_w = torch.empty((T, k), device="cuda")
        self.loss = torch.empty(1, device="cuda")
        self.aux = torch.empty(2, device="cuda")
        self.norm = torch.empty(1, device="cuda")
        self.topk_idx = self.layer.views()["topk_idx"]

    def gradients(self):
        """Loss and gradients of every parameter, clipped."""
        p, g = self.params, self.grads
        self.emb.forward(p["table"], self.ids, y=self.x)
        m.moe_block_norm_forward(self.before.shape, self.x, None, None, None, p["norm_in"], None, self.h,
                                 self.before.rstd)
        self.layer.forward(self.h, y=self.y)
        after = dict(w_post=p["norm_post"], gate=p["channel_gate"], w_pre=p["norm_out"])
        self.after.forward(self.x, self.y, **after, s=self.s, h=self.z)
        self.ce.forward(self.z, p["table"], self.target, total=self.loss)
        self.ce.backward(self.z, p["table"], self.target, dx=self.dz, dw=g["table"])
        self.after.backward(None, self.dz, self.x, self.y, **after, dx=self.dx, dy=self.dy,
                            dw_post=g["norm_post"], dgate=g["channel_gate"], dw_pre=g["norm_out"])
        self.layer.backward(self.dy, self.dh, self.d_topk_w, m.grads_for(g["gate"], g["up"], g["down"]))
        self.router.backward(self.h, p["router"], self.topk_idx, self.d_topk_w, dx_add=self.dh, dx=self.dh,
                             dw_router=g["router"], aux=self.aux)
        self.before.backward(self.dx, self.dh, self.x, w_pre=p["norm_in"], dx=self.dx, dw_pre=g["norm_in"])
        self.emb.backward(self.ids, self.dx, dw_add=g["table"], dw=g["table"])
        self.clip.clip(self.max_norm, norm=self.norm)

    def step(self, lr: float):
        """lr of the parameters outside the experts, which have the constructor's."""
        self.gradients()
        self.muon.step()
        for n in self.rest:
            self.params[n].add_(self.grads[n], alpha=-lr)

    def device_status(self):
        return [o.device_status() for o in (self.layer, self.ce, self.router, self.emb, self.before,
                                            self.after, self.muon)]


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--lr", type=float, default=2.0)
    ap.add_argument("--block", action="store_true", help="from token ids, with norms and the experts' Muon")
    a = ap.parse_args()
    s = BlockStep() if a.block else TrainStep()
    for i in range(a.steps):
        s.step(a.lr)
        print("step %3d  loss %.4f  balance %.5f  z %.5f  gradient norm %.4f"
              % (i, float(s.loss), float(s.aux[0]), float(s.aux[1]), float(s.norm)))


if __name__ == "__main__":
    main()

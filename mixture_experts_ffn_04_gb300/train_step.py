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
rows, random targets) and prints loss, balance loss and gradient norm.
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


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--steps", type=int, default=20)
    ap.add_argument("--lr", type=float, default=2.0)
    a = ap.parse_args()
    s = TrainStep()
    for i in range(a.steps):
        s.step(a.lr)
        print("step %3d  loss %.4f  balance %.5f  z %.5f  gradient norm %.4f"
              % (i, float(s.loss), float(s.aux[0]), float(s.aux[1]), float(s.norm)))


if __name__ == "__main__":
    main()

#!/usr/bin/env python
"""A low-rank adapter on every expert of a frozen layer, trained with the router.

The layer's experts run on their tokens in expert order, so that something of
each expert's own can stand beside them:

  router (exl3_router_forward) -> tokens in expert order (exl3_dispatch_plan, exl3_dispatch)
  -> frozen experts, one route a row (exl3_moe_forward with topk = 1)
  -> + the expert's adapter (exl3_lora_forward, adapter = expert)
  -> back to the tokens with the route weights (exl3_combine)

and backward through the same steps; one AdamW step (exl3_adamw) moves the
adapters (float16 with float32 masters and 8-bit states, rounded at random),
another the router.

  python examples/expert_adapters.py          # a short fine-tuning run
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import trellis_quantized_moe_gb300 as X  # noqa: E402
from workloads import MoEWorkload, config  # noqa: E402

DT = torch.float16


def _buffer(n):
    return torch.empty(n, dtype=torch.uint8, device="cuda")


class ExpertAdapted:
    """Frozen experts with a router and an adapter for each of them, every buffer of a step and its optimisers."""

    def __init__(self, tokens, rank, generator, spread=0.5):
        spec = config(0, M=tokens)
        self.M, self.H, self.E, self.k, self.capacity = tokens, spec.hidden, spec.E, spec.topk, spec.capacity
        M, H, E, R = self.M, self.H, self.E, tokens * spec.topk
        self.experts = X.DeviceExperts.from_workload(MoEWorkload(spec))
        rnd = lambda *s: torch.randn(*s, generator=generator, device="cuda")
        e = lambda *s, dt=torch.float32: torch.empty(s, dtype=dt, device="cuda")
        self.router = rnd(H, E) * (spread * H ** -0.5)
        masters = [rnd(rank, H) * H ** -0.5 for _ in range(E)] + [rnd(rank, H) * (0.1 * spread) for _ in range(E)]
        params = [p.to(DT) for p in masters]
        grads = [torch.empty_like(p) for p in params]
        self.adapters = X.DeviceAdapters(params[:E], params[E:], [1.0] * E)
        self.grads = X.DeviceAdapters(grads[:E], grads[E:], [1.0] * E)
        # activations and gradients
        self.ids, self.rw, self.stats = e(M, self.k, dt=torch.int32), e(M, self.k), e(M, 2)
        self.counts, self.loss, self.d_logits = e(E + 1, dt=torch.int32), e(1), e(M, E)
        self.offsets, self.slots = e(E + 1, dt=torch.int32), e(M, self.k, dt=torch.int32)
        self.packed, self.expert_of = e(R, dt=torch.int32), e(R, dt=torch.int32)
        self.xp, self.frozen, self.y, self.dy = (e(R, H, dt=DT) for _ in range(4))
        self.ones = torch.ones((R, 1), device="cuda")
        self.h, self.out, self.d_rw = e(R, self.adapters.h_cols, dt=DT), e(M, H, dt=DT), e(M, self.k)
        self.d_router = e(H, E)
        # workspaces
        self.ws_router = _buffer(X.exl3_router_workspace_bytes(M, E))
        self.ws_plan = _buffer(X.exl3_dispatch_workspace_bytes(M, self.k, E))
        self.plan = _buffer(X.exl3_lora_plan_bytes(R, E))
        self.ws_moe = _buffer(X.exl3_moe_workspace_bytes(R, 1, E, H, spec.inter, self.capacity))
        self.ws_lora = _buffer(X.exl3_lora_workspace_bytes(R, E, H, H, rank))
        # optimisers: fresh states are zeros
        codes = lambda: [torch.zeros(p.numel(), device="cuda").to(torch.float8_e4m3fn) for p in params]
        scales = lambda: [torch.zeros(-(-p.numel() // 256), device="cuda") for p in params]
        flat = lambda ts: [t.view(-1) for t in ts]
        self.opt = X.DeviceAdamW(flat(params), flat(grads), codes(), codes(), m_scale=scales(), v_scale=scales(),
                                 master=flat(masters), rounding="random")
        zero = lambda: [torch.zeros(H * E, device="cuda")]
        self.opt_router = X.DeviceAdamW(flat([self.router]), flat([self.d_router]), zero(), zero())
        self.step, self.step_router = (torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(2))
        self.ws_opt, self.ws_opt_router = _buffer(X.exl3_adamw_workspace_bytes()), _buffer(X.exl3_adamw_workspace_bytes())
        self.balance = torch.empty(1, device="cuda")

    def forward(self, x):
        self.logits = x.float() @ self.router
        X.exl3_router_forward(self.logits, self.ids, self.rw, renorm=True, stats=self.stats, counts=self.counts,
                              loss=self.loss, workspace=self.ws_router)
        X.exl3_dispatch_plan(self.ids, self.E, self.offsets, self.packed, self.slots, self.ws_plan,
                             experts=self.expert_of)
        X.exl3_dispatch(x, self.slots, self.xp)
        X.exl3_moe_forward(self.xp, self.expert_of.view(-1, 1), self.ones, self.experts, self.capacity, self.ws_moe,
                           self.frozen)
        X.exl3_lora_plan(self.expert_of, self.E, self.plan)
        X.exl3_lora_forward(self.xp, self.plan, self.adapters, self.y, self.ws_lora, base=self.frozen, h=self.h)
        X.exl3_combine(self.y, self.slots, self.out, rw=self.rw)
        return self.out

    def backward(self, x, d_out):
        """Gradients of adapters and router (self.grads, self.d_router) from that of the output."""
        X.exl3_combine_backward(d_out, self.y, self.slots, self.rw, dy=self.dy, d_rw=self.d_rw)
        X.exl3_lora_backward(self.dy, self.xp, self.h, self.plan, self.adapters, self.grads, self.ws_lora)
        X.exl3_router_backward(self.logits, self.ids, self.stats, self.d_logits, renorm=True, d_rw=self.d_rw,
                               counts=self.counts, d_loss=self.balance)
        torch.mm(x.float().T, self.d_logits, out=self.d_router)

    def update(self, lr):
        X.exl3_adamw(self.opt, self.step, self.ws_opt, lr=lr, weight_decay=0.0)
        X.exl3_adamw(self.opt_router, self.step_router, self.ws_opt_router, lr=lr, weight_decay=0.0)

    def train_step(self, x, target, lr=3e-3, balance=0.01):
        """Squared error / 2 summed over the tokens, and the balance loss per token."""
        self.balance.fill_(balance * self.M)
        diff = self.forward(x).float() - target
        self.error = (diff ** 2).mean()
        self.backward(x, diff.to(DT))
        self.update(lr)


def finetune(tokens=512, steps=60, seed=0):
    """Losses of the steps (mean squared error, balance loss) against a teacher of the same form."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(tokens, config(0).hidden, generator=gen, device="cuda").to(DT)
    target = ExpertAdapted(tokens, 4, gen, spread=2.0).forward(x).float()
    student = ExpertAdapted(tokens, 8, gen)
    history = []
    for _ in range(steps):
        student.train_step(x, target)
        history.append((float(student.error), float(student.loss)))
    return history


if __name__ == "__main__":
    losses = finetune()
    for i in range(0, len(losses), 10):
        print(f"step {i:3d}: error {losses[i][0]:.5f}, balance loss {losses[i][1]:.4f}")
    print(f"last    : error {losses[-1][0]:.5f}, balance loss {losses[-1][1]:.4f}")

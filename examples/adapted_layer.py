#!/usr/bin/env python
"""The routed-expert layer with a trainable router and adapters, end to end.

A layer of frozen trellis weights: routed experts (exl3_moe_forward) plus one
shared projection (exl3_linear).  What is trained around them is the router
(exl3_router_forward / _backward, with its balance loss) and low-rank adapters
beside the shared projection (exl3_lora_forward / _backward).

  python examples/adapted_layer.py            # a short fine-tuning run, then a decode batch

finetune() fits both to a teacher of the same form: one adapter per half of the
tokens, mean squared error plus 0.01 of the balance loss, plain SGD.  serve()
runs a decode batch in which every request brings its own adapter, or none, and
replays it as a CUDA graph.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import trellis_quantized_moe_gb300 as X  # noqa: E402
from workloads import CB_MCG, LinearWorkload, MoEWorkload, config  # noqa: E402

DT = torch.float16


def _buffer(n):
    return torch.empty(n, dtype=torch.uint8, device="cuda")


class FrozenLayer:
    """Experts and shared projection of one layer, with the buffers their calls take."""

    def __init__(self, tokens):
        spec = config(0, M=tokens)
        self.M, self.hidden, self.E, self.topk = tokens, spec.hidden, spec.E, spec.topk
        self.experts = X.DeviceExperts.from_workload(MoEWorkload(spec))
        self.shared = X.DeviceProjection(
            LinearWorkload(tokens, spec.hidden, spec.hidden, K=4, cb=CB_MCG, act="f16", seed=9).proj)
        self.capacity = spec.capacity
        self.ws_moe = _buffer(X.exl3_moe_workspace_bytes(tokens, spec.topk, spec.E, spec.hidden, spec.inter,
                                                         spec.capacity))
        self.ws_linear = _buffer(X.exl3_linear_workspace_bytes(tokens, spec.hidden, spec.hidden))
        self.base = torch.empty((tokens, spec.hidden), dtype=DT, device="cuda")

    def routed(self, x, ids, rw, out):
        X.exl3_moe_forward(x, ids, rw, self.experts, self.capacity, self.ws_moe, out)

    def project(self, x):
        X.exl3_linear(x, self.shared, self.base, self.ws_linear)
        return self.base


class Adapted:
    """Router weight and adapters of a FrozenLayer, their gradients and buffers."""

    def __init__(self, layer, ids, ranks, scales, generator, spread):
        M, H, E, k = layer.M, layer.hidden, layer.E, layer.topk
        rnd = lambda *s: torch.randn(*s, generator=generator, device="cuda")
        self.layer = layer
        self.router = rnd(H, E) * (spread * H ** -0.5)
        A = [(rnd(r, H) * H ** -0.5).to(DT) for r in ranks]
        B = [(rnd(r, H) * 0.1 * spread).to(DT) for r in ranks]
        self.adapters = X.DeviceAdapters(A, B, scales)
        self.grads = X.DeviceAdapters([torch.empty_like(a) for a in A], [torch.empty_like(b) for b in B], scales)
        self.plan = _buffer(X.exl3_lora_plan_bytes(M, len(ranks)))
        X.exl3_lora_plan(ids, len(ranks), self.plan)       # once per batch, for every adapted projection
        self.ws_lora = _buffer(X.exl3_lora_workspace_bytes(M, len(ranks), H, H, self.adapters.max_rank))
        self.ws_router = _buffer(X.exl3_router_workspace_bytes(M, E))
        e = lambda *s, **kw: torch.empty(s, device="cuda", **kw)
        self.ids, self.rw = e(M, k, dtype=torch.int32), e(M, k)
        self.stats, self.counts, self.loss = e(M, 2), e(E + 1, dtype=torch.int32), e(1)
        self.d_logits = e(M, E)
        self.h = e(M, self.adapters.h_cols, dtype=DT)
        self.mixed, self.y = e(M, H, dtype=DT), e(M, H, dtype=DT)

    def forward(self, x):
        self.logits = x.float() @ self.router
        X.exl3_router_forward(self.logits, self.ids, self.rw, renorm=True, stats=self.stats, counts=self.counts,
                              loss=self.loss, workspace=self.ws_router)
        self.layer.routed(x, self.ids, self.rw, self.mixed)
        X.exl3_lora_forward(x, self.plan, self.adapters, self.y, self.ws_lora, base=self.layer.project(x), h=self.h)
        return self.mixed.float() + self.y.float()

    def backward(self, x, d_out, balance):
        """Gradients of the adapters (self.grads) and of the router weight (returned)."""
        # d rw_j = <d_out, output of the token's j-th expert>: the layer on one route at a time
        d_rw = torch.empty_like(self.rw)
        one = torch.ones((self.layer.M, 1), device="cuda")
        out = torch.empty_like(self.mixed)
        for j in range(self.layer.topk):
            self.layer.routed(x, self.ids[:, j:j + 1].contiguous(), one, out)
            d_rw[:, j] = (d_out * out.float()).sum(dim=1)
        X.exl3_router_backward(self.logits, self.ids, self.stats, self.d_logits, renorm=True, d_rw=d_rw,
                               counts=self.counts, d_loss=torch.full((1,), balance, device="cuda"))
        X.exl3_lora_backward(d_out.to(DT), x, self.h, self.plan, self.adapters, self.grads, self.ws_lora)
        return x.float().T @ self.d_logits


def finetune(tokens=512, steps=60, rate=0.1, balance=0.01, seed=0):
    """Losses of the steps (mean squared error, balance loss)."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    layer = FrozenLayer(tokens)
    ids = (torch.arange(tokens, device="cuda") * 2 // tokens).int()
    x = torch.randn(tokens, layer.hidden, generator=gen, device="cuda").to(DT)
    teacher = Adapted(layer, ids, [4, 4], [1.0, 1.0], gen, spread=3.0)
    target = teacher.forward(x).clone()
    student = Adapted(layer, ids, [8, 4], [1.0, 1.0], gen, spread=0.5)
    history = []
    for _ in range(steps):
        diff = student.forward(x) - target
        history.append((float((diff ** 2).mean()), float(student.loss)))
        # of the sum over tokens (squared error / 2, and the balance loss per
        # token): a mean's gradients would be small for 16 bits; the step divides
        d_router = student.backward(x, diff, balance * tokens)
        student.router -= rate / tokens * d_router
        for params, grads in ((student.adapters.A, student.grads.A), (student.adapters.B, student.grads.B)):
            for p, g in zip(params, grads):
                p -= (rate / tokens * g.float()).to(DT)
    torch.cuda.synchronize()
    return history


def serve(seed=1):
    """One decode step of 24 requests over 6 adapters of mixed ranks; some have none.
    Returns the step's output and the output of its graph replay."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    tokens = 24
    layer = FrozenLayer(tokens)
    ids = torch.tensor([i % 7 - 1 for i in range(tokens)], dtype=torch.int32, device="cuda")
    model = Adapted(layer, ids, [8, 16, 4, 32, 8, 64], [1.0] * 6, gen, spread=1.0)
    x = torch.randn(tokens, layer.hidden, generator=gen, device="cuda").to(DT)
    logits = torch.empty((tokens, layer.E), device="cuda")

    def step():
        torch.mm(x.float(), model.router, out=logits)
        X.exl3_router_forward(logits, model.ids, model.rw)
        layer.routed(x, model.ids, model.rw, model.mixed)
        X.exl3_lora_forward(x, model.plan, model.adapters, model.y, model.ws_lora, base=layer.project(x))

    step()
    torch.cuda.synchronize()
    eager = (model.mixed.clone(), model.y.clone())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    model.mixed.zero_()
    model.y.zero_()
    graph.replay()
    torch.cuda.synchronize()
    return eager, (model.mixed, model.y)


if __name__ == "__main__":
    losses = finetune()
    for i in range(0, len(losses), 10):
        print(f"step {i:3d}: error {losses[i][0]:.5f}, balance loss {losses[i][1]:.4f}")
    print(f"last    : error {losses[-1][0]:.5f}, balance loss {losses[-1][1]:.4f}")
    eager, replayed = serve()
    print("decode step and its graph replay agree:", all(torch.equal(a, b) for a, b in zip(eager, replayed)))

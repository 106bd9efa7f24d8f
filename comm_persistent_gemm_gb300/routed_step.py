"""Training steps of an expert layer with its own router.

    python -m comm_persistent_gemm_gb300.routed_step [--steps N] [--lr R] [--tokens T] [--hidden H] [--experts E]
                                                     [--topk K] [--inter I] [--ranks P] [--score sigmoid]

One step, the way a training program runs it:

    logits = x W_r                               (torch, fp32)
    route            -> experts, gates, tokens per expert
    moe_fwd_routed   -> y
    loss = mean over tokens of |y - target|^2 / 2
    moe_bwd          -> dx (the experts' part), dW_gate / dW_up / dW_down, dgate
    route_bwd        -> dlogits;  dW_r = x^T dlogits;  dx += dlogits W_r^T
    grad_clip        over every gradient of the layer, then the update
    bias[e] += rate * sign(mean load - load[e])  (balance without a loss)

The inputs are synthetic: tokens around a few centres, so that some experts
are popular, and the targets of a fixed random layer."""
from __future__ import annotations

import argparse
import math

import comm_persistent_gemm_gb300 as K


class RoutedLayer:
    """Weights, router, workspaces and gradients of one layer on P emulated
    ranks."""

    def __init__(self, P, tokens, hidden, experts, topk, inter, score=K.SCORE_SIGMOID, n_groups=1, topk_groups=1,
                 scale=1.0, seed=0, device="cuda"):
        import torch
        self.P, self.T, self.H, self.E, self.k, self.I = P, tokens, hidden, experts, topk, inter
        g = torch.Generator(device=device).manual_seed(seed)

        def randn(*shape, std):
            return torch.randn(*shape, generator=g, device=device) * std

        per = experts // P
        # fp32 masters; the layer's weights are their bf16 roundings
        self.w_router = randn(hidden, experts, std=1.0 / math.sqrt(hidden))
        self.masters = {"gate": [randn(per, hidden, inter, std=hidden ** -0.5) for _ in range(P)],
                        "up": [randn(per, hidden, inter, std=hidden ** -0.5) for _ in range(P)],
                        "down": [randn(per, inter, hidden, std=inter ** -0.5) for _ in range(P)]}
        self.weights = {n: [w.bfloat16() for w in ws] for n, ws in self.masters.items()}
        self.bias = torch.zeros(experts, device=device)
        self.router = K.router(topk=topk, score=score, n_groups=n_groups, topk_groups=topk_groups,
                               group_top=2 if n_groups > 1 else 1, scale=scale)
        f32, i32, bf16 = torch.float32, torch.int32, torch.bfloat16

        def empty(*shape, dtype):
            return torch.empty(*shape, dtype=dtype, device=device)

        self.idx, self.gate = empty(tokens, topk, dtype=i32), empty(tokens, topk, dtype=f32)
        self.load, self.counts = empty(experts, dtype=i32), empty(experts, dtype=i32)
        self.pos = empty(tokens, topk, dtype=i32)
        self.y = [empty(tokens // P, hidden, dtype=bf16) for _ in range(P)]
        self.dx = [empty(tokens // P, hidden, dtype=bf16) for _ in range(P)]
        self.dlogits = empty(tokens, experts, dtype=f32)
        self.grads = {n: [torch.empty_like(w) for w in ws] for n, ws in self.weights.items()}
        self.dw_router = empty(hidden, experts, dtype=f32)
        # the fused backward's own router part is not this layer's router: zeros in, ignored out
        self.no_router = torch.zeros(hidden, experts, dtype=bf16, device=device)
        self.no_dw_router = empty(hidden, experts, dtype=f32)
        self.norm = empty(1, dtype=f32)
        self.route_ws = K.route_workspace(experts, device)
        self.fwd_ws = K.moe_workspace(P, tokens, hidden, experts, topk, inter, device=device)
        self.bwd_ws = K.moe_bwd_workspace(P, tokens, hidden, experts, topk, inter, device=device)
        # every gradient of the layer, marshalled once
        self.grad_set = K.GradSet([g for n in ("gate", "up", "down") for g in self.grads[n]] + [self.dw_router])
        self.grad_ws = K.grad_workspace(self.grad_set, device)

    def forward(self, x_shards):
        """y of the layer for bf16 token shards [tokens / P, hidden]."""
        import torch
        self.x = torch.cat(x_shards).float()
        self.logits = self.x @ self.w_router
        K.route(self.logits, self.router, self.idx, self.gate, bias=self.bias, expert_counts=self.load,
                ws=self.route_ws)
        w = self.weights
        K.moe_fwd_routed(x_shards, w["gate"], w["up"], w["down"], self.y, self.idx, self.gate, self.counts, self.pos,
                         self.fwd_ws)
        return self.y

    def backward(self, x_shards, dy_shards):
        """Every gradient from dy; returns dx [tokens, hidden] fp32."""
        import torch
        w, g = self.weights, self.grads
        K.moe_bwd(x_shards, self.no_router, w["gate"], w["up"], w["down"], self.idx, self.gate, self.fwd_ws, dy_shards,
                  self.dx, self.no_dw_router, g["gate"], g["up"], g["down"], self.bwd_ws)
        dgate = K.moe_bwd_debug_view(K.MOE_BWD_VIEW_DGATE, self.P, self.T, self.H, self.E, self.k, self.I,
                                     self.bwd_ws).view(torch.float32).view(self.T, self.k)
        K.route_bwd(self.logits, self.router, self.idx, self.gate, dgate, self.dlogits)
        torch.mm(self.x.t(), self.dlogits, out=self.dw_router)
        return torch.cat(self.dx).float() + self.dlogits @ self.w_router.t()

    def update(self, lr, max_norm, bias_rate):
        """Clips, steps, and moves the balance bias towards an even load."""
        import torch
        K.grad_clip(self.grad_set, max_norm, self.norm, self.grad_ws)
        for n, ws in self.masters.items():
            for m, w, g in zip(ws, self.weights[n], self.grads[n]):
                m.sub_(g.float(), alpha=lr)
                w.copy_(m)
        self.w_router.sub_(self.dw_router, alpha=lr)
        load = self.load.float()
        self.bias += bias_rate * torch.sign(load.mean() - load)

    def check(self):
        """Raises on a status that a kernel left behind."""
        K.check(self.fwd_ws, "moe_fwd_routed")
        K.check(self.bwd_ws, "moe_bwd")
        K.check(self.grad_ws, "grad_clip")


def inputs(layer, seed):
    """(token shards, targets): tokens around 8 centres, targets of a random
    linear map of them."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    centres = torch.randn(8, layer.H, generator=g, device="cuda")
    x = centres[torch.randint(0, 8, (layer.T,), generator=g, device="cuda")]
    x = (0.7 * x + 0.7 * torch.randn(layer.T, layer.H, generator=g, device="cuda")).bfloat16()
    a = torch.randn(layer.H, layer.H, generator=g, device="cuda") * layer.H ** -0.5
    return [s.contiguous() for s in x.chunk(layer.P)], x.float() @ a


def train(layer, steps, lr=0.5, max_norm=1.0, bias_rate=0.01, seed=1, report=None):
    """Runs steps of training; returns the losses."""
    import torch
    x, target = inputs(layer, seed)
    losses = []
    for i in range(steps):
        y = torch.cat(layer.forward(x)).float()
        diff = y - target
        loss = 0.5 * (diff * diff).sum(1).mean()
        dy = [s.contiguous() for s in (diff / layer.T).bfloat16().chunk(layer.P)]
        layer.backward(x, dy)
        layer.update(lr, max_norm, bias_rate)
        layer.check()
        losses.append(float(loss))
        if report:
            load = layer.load.float()
            report(f"step {i}: loss {losses[-1]:.4f}  gradient norm {float(layer.norm):.4f}  "
                   f"busiest expert {float(load.max() / load.mean()):.2f} x the mean load")
    return losses


def main():
    a = argparse.ArgumentParser(description=__doc__.split("\n")[0])
    a.add_argument("--steps", type=int, default=20)
    a.add_argument("--lr", type=float, default=0.5)
    a.add_argument("--ranks", type=int, default=8)
    a.add_argument("--tokens", type=int, default=2048)
    a.add_argument("--hidden", type=int, default=1024)
    a.add_argument("--experts", type=int, default=128)
    a.add_argument("--topk", type=int, default=8)
    a.add_argument("--inter", type=int, default=512)
    a.add_argument("--groups", type=int, default=8)
    a.add_argument("--open-groups", type=int, default=4)
    a.add_argument("--score", choices=["softmax", "sigmoid"], default="sigmoid")
    o = a.parse_args()
    K.build()
    layer = RoutedLayer(o.ranks, o.tokens, o.hidden, o.experts, o.topk, o.inter,
                        K.SCORE_SIGMOID if o.score == "sigmoid" else K.SCORE_SOFTMAX, o.groups, o.open_groups)
    train(layer, o.steps, o.lr, report=print)


if __name__ == "__main__":
    main()

"""A gated delta rule layer, trained and then served, on the framework's operators:

  train   project -> qk_norm_rope_train -> gated_delta_rule -> project, its backward, clip_grad_norm
  serve   project -> qk_norm_rope -> gdr_prefill (ragged prompts), then gdr_decode a token at a time

Run:  python examples/delta_rule_layer.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from state_summary_scan_gb300 import api  # noqa: E402


class Layer:
    """x [B,T,width] -> [B,T,width]: heads of 64, unit keys (an l2 norm) with rotated positions.
    Parameters are fp32; the matrices are used in bf16."""

    def __init__(self, width: int, heads: int, max_positions: int, seed: int = 0, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        self.heads, self.dim = heads, 64
        n = heads * self.dim

        def matrix(rows, cols):
            return (torch.randn(rows, cols, generator=g) / rows ** 0.5).to(device).requires_grad_(True)

        self.w_qkv, self.w_gates, self.w_out = matrix(width, 3 * n), matrix(width, 2 * heads), matrix(n, width)
        # queries and keys end up with norms near 1: the delta rule's keys are unit vectors
        self.q_weight = torch.ones(self.dim, device=device, requires_grad=True)
        self.k_weight = torch.ones(self.dim, device=device, requires_grad=True)
        self.table = api.make_rope_table(max_positions, self.dim, device=device)

    def parameters(self):
        return [self.w_qkv, self.w_gates, self.w_out, self.q_weight, self.k_weight]

    def project(self, x):
        """q, k (slices of one projection), v, and the gates g = log sigmoid, beta = sigmoid in fp32."""
        n = self.heads * self.dim
        qkv = x @ self.w_qkv.to(x.dtype)
        q, k, v = (qkv[..., i * n: (i + 1) * n].unflatten(-1, (self.heads, self.dim)) for i in range(3))
        g, beta = (x @ self.w_gates.to(x.dtype)).float().split(self.heads, -1)
        return q, k, v, torch.nn.functional.logsigmoid(g + 4), torch.sigmoid(beta)

    def train_forward(self, x, num_segments: int):
        q, k, v, g, beta = self.project(x)
        q, k = api.qk_norm_rope_train(q, k, self.table, None, self.q_weight, self.k_weight, norm="l2")
        o = api.gated_delta_rule(q, k, v, g, beta, num_segments, chunk=64)
        return o.flatten(2) @ self.w_out.to(x.dtype)

    def serving_plan(self, max_prompts: int, max_tokens: int, slots: int):
        plan = api.make_gdr_state_plan(max_prompts, max_tokens, self.heads, self.dim, self.dim, num_slots=slots)
        return plan, api.make_gdr_state(plan)

    @torch.no_grad()
    def prefill(self, plan, state, x, cu_seqlens, positions, slots):
        """Packed prompts x [N,width], positions [N]; leaves each prompt's state in its slot."""
        q, k, v, g, beta = self.project(x)
        q, k = api.qk_norm_rope(q[None], k[None], self.table, positions[None], self.q_weight.detach(), self.k_weight.detach(), norm="l2")
        fresh = torch.ones(len(slots), dtype=torch.uint8, device=x.device)
        o = api.gdr_prefill(plan, q[0], k[0], v, g.contiguous(), beta.contiguous(), state, cu_seqlens, slots=slots, fresh=fresh)
        return o.flatten(1) @ self.w_out.to(x.dtype)

    @torch.no_grad()
    def decode(self, plan, state, x, positions, slots):
        """One token of each sequence, x [S,width], positions [S]."""
        q, k, v, g, beta = (y[:, None] for y in self.project(x))
        q, k = api.qk_norm_rope(q, k, self.table, positions[:, None], self.q_weight.detach(), self.k_weight.detach(), norm="l2")
        o = api.gdr_decode(plan, q, k, v, g.contiguous(), beta.contiguous(), state, slots=slots)
        return o.flatten(1) @ self.w_out.to(x.dtype)


def train(layer: Layer, steps: int = 20, B: int = 2, T: int = 256, lr: float = 0.3, max_norm: float = 1.0):
    """Learns to give each token its own input back, through the state; returns the losses (squared
    error a token).  Gradients are far above max_norm at first: every step has that norm."""
    g = torch.Generator("cuda").manual_seed(1)
    x = torch.randn(B, T, layer.w_qkv.shape[0], generator=g, device="cuda").to(torch.bfloat16)
    plan = api.make_clip_plan(len(layer.parameters()))
    losses = []
    for _ in range(steps):
        loss = (layer.train_forward(x, num_segments=4).float() - x.float()).square().sum(-1).mean()
        grads = torch.autograd.grad(loss, layer.parameters())
        api.clip_grad_norm(plan, grads, max_norm)
        with torch.no_grad():
            for p, d in zip(layer.parameters(), grads):
                p -= lr * d
        losses.append(loss.detach())
    return torch.stack(losses).tolist()


def serve(layer: Layer, lens=(100, 37, 64), generate: int = 8):
    """Prefills ragged prompts, then decodes `generate` more tokens of each.  Returns each sequence's
    inputs and the layer's outputs for all of its tokens."""
    g = torch.Generator("cuda").manual_seed(2)
    width = layer.w_qkv.shape[0]
    xs = [torch.randn(n + generate, width, generator=g, device="cuda").to(torch.bfloat16) for n in lens]
    plan, state = layer.serving_plan(len(lens), sum(lens), len(lens) + 1)
    slots = torch.arange(len(lens), dtype=torch.int32, device="cuda").flip(0).contiguous()
    cu = torch.tensor([0, *lens], device="cuda").cumsum(0).to(torch.int32)
    positions = torch.cat([torch.arange(n, device="cuda", dtype=torch.int32) for n in lens])
    y = layer.prefill(plan, state, torch.cat([x[:n] for x, n in zip(xs, lens)]), cu, positions, slots)
    outs = [[part] for part in y.split(list(lens))]
    at = torch.tensor(lens, dtype=torch.int32, device="cuda")
    for t in range(generate):
        y = layer.decode(plan, state, torch.stack([x[n + t] for x, n in zip(xs, lens)]), at + t, slots)
        for i in range(len(lens)):
            outs[i].append(y[i: i + 1])
    return xs, [torch.cat(o) for o in outs]


def main():
    layer = Layer(width=256, heads=4, max_positions=4096)
    losses = train(layer)
    print("loss: " + " ".join(f"{x:.4f}" for x in losses[:: max(1, len(losses) // 5)]))
    xs, outs = serve(layer)
    for x, y in zip(xs, outs):
        # the training forward over the same tokens, padded to whole segments
        T = (x.shape[0] + 255) // 256 * 256
        padded = torch.cat([x, torch.zeros(T - x.shape[0], x.shape[1], dtype=x.dtype, device=x.device)])
        with torch.no_grad():
            want = layer.train_forward(padded[None], num_segments=4)[0, : x.shape[0]]
        err = float((y.float() - want.float()).norm() / want.float().norm())
        print(f"served {x.shape[0]} tokens, {err:.1e} from the training forward")


if __name__ == "__main__":
    main()

"""A block of gated linear attention, trained and then served, on the framework's operators:

  train   rms_norm_train (with the residual's addition) -> project -> qk_norm_rope_train -> chunkwise_gla ->
          rms_norm_train with a gate -> project, its backward, clip_grad_norm
  serve   rms_norm or rms_norm_quant -> project -> qk_norm_rope -> gla_prefill (ragged prompts), then gla_decode
          a token at a time -> the gated norm -> project

Run:  python examples/linear_attention_layer.py
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
from state_summary_scan_gb300 import api  # noqa: E402


class Block:
    """(x, stream) [B,T,width] -> (y, stream): the stream takes x in before the norm, and y is what the block adds to
    it next.  Heads of 128 with rotated positions and a decay for each token and head.  Parameters are fp32; the
    matrices are used in bf16."""

    def __init__(self, width: int, heads: int, max_positions: int, seed: int = 0, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        self.heads, self.dim = heads, 128
        n = heads * self.dim

        def matrix(rows, cols):
            return (torch.randn(rows, cols, generator=g) / rows ** 0.5).to(device).requires_grad_(True)

        self.w_in, self.w_decay, self.w_out = matrix(width, 4 * n), matrix(width, heads), matrix(n, width)
        self.norm, self.out_norm = (torch.ones(m, device=device, requires_grad=True) for m in (width, self.dim))
        self.table = api.make_rope_table(max_positions, self.dim, device=device)

    def parameters(self):
        return [self.w_in, self.w_decay, self.w_out, self.norm, self.out_norm]

    def project(self, x):
        """q, k, v and the output's gate as slices of one projection, and the log-decays in fp32."""
        n = self.heads * self.dim
        wide = x @ self.w_in.to(x.dtype)
        q, k, v, z = (wide[..., i * n: (i + 1) * n].unflatten(-1, (self.heads, self.dim)) for i in range(4))
        return q, k, v, z, torch.nn.functional.logsigmoid((x @ self.w_decay.to(x.dtype)).float() + 4)

    def train_forward(self, x, stream, num_segments: int):
        h, stream = api.rms_norm_train(x, self.norm, stream)
        q, k, v, z, g = self.project(h)
        q, k = api.qk_norm_rope_train(q, k, self.table, norm="l2")
        o = api.chunkwise_gla(q, k, v, g, num_segments, chunk=64)
        y, _ = api.rms_norm_train(o, self.out_norm, gate=z)
        return y.flatten(2) @ self.w_out.to(x.dtype), stream

    def serving_plan(self, max_prompts: int, max_tokens: int, slots: int):
        plan = api.make_gla_state_plan(max_prompts, max_tokens, self.heads, self.dim, self.dim, num_slots=slots)
        return plan, api.make_gla_state(plan)

    @torch.no_grad()
    def _serve(self, x, stream, positions, mix, eight_bits):
        """x, stream [N,width], positions [N]; mix(q, k, v, g) -> o [N,heads,128].  The stream is updated in place.
        eight_bits: the projections' inputs in 8 bits with a scale for each 128 elements (multiplied out here; a product in
        8 bits would take them as they are)."""
        if eight_bits:
            h = self._values(*api.rms_norm_quant(x, self.norm.detach(), stream, group=128, h=stream)[:2], x.dtype)
        else:
            h, _ = api.rms_norm(x, self.norm.detach(), stream, h=stream)
        q, k, v, z, g = self.project(h)
        q, k = api.qk_norm_rope(q[None], k[None], self.table, positions[None], norm="l2")
        o = mix(q[0], k[0], v, g.contiguous())
        if eight_bits:
            y = self._values(*api.rms_norm_quant(o, self.out_norm.detach(), gate=z, group=128)[:2], x.dtype)
        else:
            y, _ = api.rms_norm(o, self.out_norm.detach(), gate=z)
        return y.flatten(1) @ self.w_out.to(x.dtype)

    @staticmethod
    def _values(y8, scales, dtype):
        return (y8.float().unflatten(-1, (scales.shape[-1], -1)) * scales[..., None]).flatten(-2).to(dtype)

    def prefill(self, plan, state, x, stream, cu_seqlens, positions, slots, eight_bits=False):
        """Packed prompts; leaves each prompt's state in its slot."""
        fresh = torch.ones(len(slots), dtype=torch.uint8, device=x.device)
        return self._serve(x, stream, positions, lambda q, k, v, g: api.gla_prefill(plan, q, k, v, g, state, cu_seqlens, slots=slots, fresh=fresh),
                           eight_bits)

    def decode(self, plan, state, x, stream, positions, slots, eight_bits=False):
        """One token of each sequence."""
        one = lambda t: t[:, None]  # noqa: E731
        return self._serve(x, stream, positions, lambda q, k, v, g: api.gla_decode(plan, one(q), one(k), one(v), one(g), state, slots=slots)[:, 0],
                           eight_bits)


def train(block: Block, steps: int = 20, B: int = 2, T: int = 256, lr: float = 0.2, max_norm: float = 1.0):
    """Learns to give each token its own input back; returns the losses (squared error a token)."""
    gen = torch.Generator("cuda").manual_seed(1)
    x, stream = (torch.randn(B, T, block.w_in.shape[0], generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2))
    plan = api.make_clip_plan(len(block.parameters()))
    losses = []
    for _ in range(steps):
        y, _ = block.train_forward(x, stream, num_segments=4)
        loss = (y.float() - x.float()).square().sum(-1).mean()
        grads = torch.autograd.grad(loss, block.parameters())
        api.clip_grad_norm(plan, grads, max_norm)
        with torch.no_grad():
            for p, d in zip(block.parameters(), grads):
                p -= lr * d
        losses.append(loss.detach())
    return torch.stack(losses).tolist()


def serve(block: Block, lens=(100, 37, 64), generate: int = 8, eight_bits=False):
    """Prefills ragged prompts, then decodes `generate` more tokens of each.  Returns each sequence's inputs
    and streams, and the block's outputs for all of its tokens."""
    gen = torch.Generator("cuda").manual_seed(2)
    width = block.w_in.shape[0]
    xs, streams = ([torch.randn(n + generate, width, generator=gen, device="cuda").to(torch.bfloat16) for n in lens] for _ in range(2))
    plan, state = block.serving_plan(len(lens), sum(lens), len(lens) + 1)
    slots = torch.arange(len(lens), dtype=torch.int32, device="cuda").flip(0).contiguous()
    cu = torch.tensor([0, *lens], device="cuda").cumsum(0).to(torch.int32)
    positions = torch.cat([torch.arange(n, device="cuda", dtype=torch.int32) for n in lens])
    first = [torch.cat([t[:n] for t, n in zip(ts, lens)]) for ts in (xs, streams)]
    outs = [[part] for part in block.prefill(plan, state, *first, cu, positions, slots, eight_bits).split(list(lens))]
    at = torch.tensor(lens, dtype=torch.int32, device="cuda")
    for t in range(generate):
        now = [torch.stack([r[n + t] for r, n in zip(rows, lens)]) for rows in (xs, streams)]
        for i, y in enumerate(block.decode(plan, state, *now, at + t, slots, eight_bits).split(1)):
            outs[i].append(y)
    return xs, streams, [torch.cat(o) for o in outs]


def trained_outputs(block: Block, x, stream):
    """The training forward over one sequence, padded to whole segments."""
    n, T = x.shape[0], (x.shape[0] + 255) // 256 * 256
    pad = lambda t: torch.cat([t, torch.zeros(T - n, t.shape[1], dtype=t.dtype, device=t.device)])[None]  # noqa: E731
    with torch.no_grad():
        return block.train_forward(pad(x), pad(stream), num_segments=4)[0][0, :n]


def main():
    block = Block(width=256, heads=2, max_positions=4096)
    losses = train(block)
    print("loss: " + " ".join(f"{x:.3f}" for x in losses[:: max(1, len(losses) // 5)]))
    for eight_bits in (False, True):
        for x, stream, y in zip(*serve(block, eight_bits=eight_bits)):
            want = trained_outputs(block, x, stream)
            err = float((y.float() - want.float()).norm() / want.float().norm())
            print(f"served {x.shape[0]} tokens{' in 8 bits' if eight_bits else ''}, {err:.1e} from the training forward")


if __name__ == "__main__":
    main()

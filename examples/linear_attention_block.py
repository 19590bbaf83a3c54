"""A linear-attention block from the library's operators, serving packed prompts and single tokens.

    python examples/linear_attention_block.py

Per block: norm of the residual stream -> projections -> short convolution with SiLU -> linear
attention with a decay for each head -> gated norm of the heads -> output projection; the block's
output joins the stream in the next block's norm, which is one call.  A `Cache` holds, per block, the
recurrence's float32 states and the convolution's last inputs; a decode step updates both in place.
"""
from __future__ import annotations

import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import chunked_kda_gb300 as kda  # noqa: E402


class Block:
    def __init__(self, width, heads, head_dim, taps=4, device="cuda", dtype=torch.bfloat16, seed=0):
        gen = torch.Generator(device=device).manual_seed(seed)
        r = lambda *s, std: torch.randn(s, generator=gen, device=device) * std  # noqa: E731
        self.H, self.D, inner = heads, head_dim, heads * head_dim
        self.pre_weight = 1 + r(width, std=0.1)
        self.w_qkv = r(width, 3 * inner, std=width ** -0.5).to(dtype)
        self.w_gate = r(width, inner, std=width ** -0.5).to(dtype)
        self.w_decay = r(width, heads, std=width ** -0.5).to(dtype)
        self.decay_rate = torch.exp(r(heads, std=1.0) - 2.0)
        self.conv = r(3 * inner, taps, std=taps ** -0.5)
        self.head_weight = 1 + r(head_dim, std=0.1)
        self.w_out = r(inner, width, std=inner ** -0.5).to(dtype)

    def new_cache(self, n_seqs):
        device, taps = self.conv.device, self.conv.shape[1]
        return {"state": torch.zeros(n_seqs, self.H, self.D, self.D, device=device),
                "conv": torch.zeros(n_seqs, taps - 1, self.conv.shape[0], device=device, dtype=self.w_qkv.dtype)}

    def __call__(self, x, cache, cu_seqlens, single):
        """x [1, T, width], normalised; the block's output before it joins the stream."""
        T = x.shape[1]
        qkv, _ = kda.kda_short_conv_fwd(x @ self.w_qkv, self.conv, initial_state=cache["conv"],
                                        final_state=cache["conv"], cu_seqlens=cu_seqlens)
        q, k, v = (t.contiguous() for t in qkv.view(1, T, 3, self.H, self.D).unbind(2))
        q, k = (torch.nn.functional.normalize(t.float(), dim=-1).to(t.dtype) for t in (q, k))
        decay = -self.decay_rate * torch.nn.functional.softplus((x @ self.w_decay).float())
        recurrence = kda.kda_decay_recurrent_fwd if single else kda.kda_decay_chunk_fwd
        o, _ = recurrence(q, k, v, decay, initial_state=cache["state"], final_state=cache["state"], cu_seqlens=cu_seqlens)
        gate = (x @ self.w_gate).view(1, T, self.H, self.D)
        o = kda.kda_gated_norm_fwd(o, gate, self.head_weight, act=kda.ACT_SILU, out=o)
        return o.view(1, T, -1) @ self.w_out


class Model:
    """Blocks over a float32 residual stream."""

    def __init__(self, n_blocks=2, width=512, heads=4, head_dim=128, device="cuda"):
        self.blocks = [Block(width, heads, head_dim, device=device, seed=i) for i in range(n_blocks)]
        self.last_weight = torch.ones(width, device=device)

    def new_cache(self, n_seqs):
        return [b.new_cache(n_seqs) for b in self.blocks]

    def __call__(self, x, cache, cu_seqlens, single=False):
        """x [1, T, width] bf16, the packed sequences' embeddings; their last hidden rows, normalised."""
        h, y = kda.kda_block_norm_fwd(x, residual=torch.zeros_like(x, dtype=torch.float32),
                                      pre_weight=self.blocks[0].pre_weight)
        for i, block in enumerate(self.blocks):
            out = block(y, cache[i], cu_seqlens, single)
            last = i + 1 == len(self.blocks)
            h, y = kda.kda_block_norm_fwd(out, residual=h, residual_out=h,
                                          pre_weight=self.last_weight if last else self.blocks[i + 1].pre_weight)
        return y


def main(lengths=(150, 1, 77, 300), n_new=8):
    """Prompts at once, then single tokens; against the whole sequences at once.  Returns the relative
    2-norm of the difference of the tokens' rows."""
    torch.manual_seed(0)
    model, width = Model(), 512
    rows = [torch.randn(n + n_new, width, device="cuda").bfloat16() for n in lengths]
    offsets = lambda ns: torch.tensor([0, *torch.tensor(ns).cumsum(0).tolist()], dtype=torch.int32, device="cuda")  # noqa: E731

    whole = model(torch.cat(rows)[None], model.new_cache(len(rows)), offsets([len(r) for r in rows]))[0]
    ends = offsets([len(r) for r in rows])[1:].tolist()
    want = torch.stack([whole[e - n_new:e] for e in ends], 1)

    cache = model.new_cache(len(rows))
    model(torch.cat([r[:n] for r, n in zip(rows, lengths)])[None], cache, offsets(list(lengths)))
    each = offsets([1] * len(rows))
    got = torch.stack([model(torch.stack([r[n + t] for r, n in zip(rows, lengths)])[None], cache, each, single=True)[0]
                       for t in range(n_new)])
    off = float((got - want).double().norm() / want.double().norm())
    print(f"{len(rows)} prompts of {list(lengths)} tokens, then {n_new} single tokens each: "
          f"relative difference to the whole sequences at once {off:.2e}")
    return off


if __name__ == "__main__":
    main()

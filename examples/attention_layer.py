"""The attention half of a decoder layer on 4-bit weights: one fused q/k/v product, norms + rotation + store into the
paged cache, attention, output product. A batch of prompts of different lengths is prefilled at once, then every
sequence decodes token by token; at the end the decoded tokens are prefilled again in one go and both ways are compared.

    python examples/attention_layer.py [--batch 4] [--prompt 500] [--steps 16] [--cache fp8] [--window 256 --sinks 4]

Random weights and inputs; needs an MI355X and the built library.
"""

from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bit_weight_quantized_qgemm_amd as qg  # noqa: E402


class Linear:
    """A W4A16 linear layer with random codes, scaled to keep its input's variance."""

    def __init__(self, K: int, N: int, gen, device):
        self.K, self.N = K, N
        codes = torch.randint(-2 ** 31, 2 ** 31 - 1, (K // 8, N), generator=gen, device=device, dtype=torch.int64)
        # uniform codes q - 8 deviate by sqrt(255 / 12)
        scales = torch.full((K // 128, N), (12 / 255 / K) ** 0.5, dtype=torch.float16, device=device)
        self.blob = qg.repack_w4a16(codes.to(torch.int32), scales)

    def __call__(self, x):
        return qg.w4a16(x, self.blob, self.K, self.N)


class Attention:
    """One layer's attention: weights, and the cache of `pages` pages."""

    def __init__(self, hidden, heads, kv_heads, dim, pages, page, cache_dtype, max_len, window, sinks, gen, device):
        self.heads, self.kv_heads, self.dim, self.window, self.sinks = heads, kv_heads, dim, window, sinks
        self.qkv = Linear(hidden, (heads + 2 * kv_heads) * dim, gen, device)
        self.out = Linear(heads * dim, hidden, gen, device)
        self.q_norm, self.k_norm = (torch.ones(dim, dtype=torch.float16, device=device) for _ in range(2))
        self.rope = qg.rope_table(max_len, dim, device=device)
        scale = 1 / 16 if cache_dtype == torch.float8_e4m3fn else 1.0
        self.cache = qg.KVCache.empty(pages, page, kv_heads, dim, cache_dtype, device, scale, scale)

    def _append(self, x, positions, table, token_seq):
        H, KV, D = self.heads, self.kv_heads, self.dim
        q, k, v = (t.unflatten(-1, (-1, D)) for t in self.qkv(x).split([H * D, KV * D, KV * D], dim=-1))
        return qg.qk_rope_append(q, k, v, positions, self.cache, table, self.rope, q_norm=self.q_norm,
                                 k_norm=self.k_norm, token_seq=token_seq)

    def prefill(self, x, positions, token_seq, table, starts, lens, max_q, max_len):
        """x [tokens][hidden]: the new tokens of all sequences, one after another."""
        q = self._append(x, positions, table, token_seq)
        o = qg.attn_prefill(q, self.cache, table, starts, lens, max_q, max_len, window=self.window, sinks=self.sinks)
        return self.out(o.flatten(1))

    def decode(self, x, positions, table, lens, max_len):
        """x [sequences][hidden]: one new token each."""
        q = self._append(x, positions, table, None)
        o = qg.attn_decode(q, self.cache, table, lens, max_len, window=self.window, sinks=self.sinks)
        return self.out(o.flatten(1))


def _packed(lens, device, first=0):
    """Positions, sequence numbers and row starts of tokens first..first+n-1 of each sequence, packed."""
    firsts = first if isinstance(first, list) else [first] * len(lens)
    positions = torch.cat([torch.arange(f, f + n, dtype=torch.int32) for f, n in zip(firsts, lens)]).to(device)
    seq = torch.repeat_interleave(torch.arange(len(lens), dtype=torch.int32), torch.tensor(lens)).to(torch.int32)
    starts = torch.tensor([0] + lens, dtype=torch.int32).cumsum(0, dtype=torch.int32)
    return positions, seq.to(device), starts.to(device)


def run(batch=4, prompt=500, steps=16, hidden=4096, heads=32, kv_heads=8, dim=128, page=16, cache="f16", window=0,
        sinks=0, seed=0, device="cuda:0"):
    """Returns (relative difference of the two ways, prefill ms, ms of a decode step), the times after a warm-up."""
    device = torch.device(device)
    torch.cuda.set_device(device)
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)
    lens = [max(1, prompt - prompt * i // (2 * batch)) for i in range(batch)]
    max_len = max(lens) + steps
    columns = -(-max_len // page)
    order = torch.randperm(batch * columns, generator=gen, device=device).to(torch.int32)
    table = order.view(batch, columns).contiguous()   # every sequence owns its pages from the start
    dtype = {"f16": torch.float16, "fp8": torch.float8_e4m3fn}[cache]
    layer = Attention(hidden, heads, kv_heads, dim, batch * columns, page, dtype, max_len, window, sinks, gen, device)

    positions, seq, starts = _packed(lens, device)
    now = torch.tensor(lens, dtype=torch.int32, device=device)
    x = torch.randn((sum(lens), hidden), generator=gen, device=device).to(torch.float16)
    new = torch.randn((steps, batch, hidden), generator=gen, device=device).to(torch.float16)

    def prefill():
        return layer.prefill(x, positions, seq, table, starts, now, max(lens), max_len)

    prefill()
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    prefill()
    torch.cuda.synchronize()
    prefill_ms = (time.perf_counter() - t0) * 1e3

    # twice: the second time, which stores the same keys and values again, is timed
    for _ in range(2):
        outs, cur = [], now.clone()
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        for s in range(steps):
            at = cur.clone()   # the new token's position: the cache's length so far
            cur += 1
            outs.append(layer.decode(new[s], at, table, cur, max_len))
        torch.cuda.synchronize()
        step_ms = (time.perf_counter() - t0) * 1e3 / max(1, steps)

    # the same tokens as one chunk after the prompts
    positions, seq, starts = _packed([steps] * batch, device, first=lens)
    chunk = layer.prefill(new.transpose(0, 1).reshape(batch * steps, hidden).contiguous(), positions, seq, table, starts,
                          now + steps, steps, max_len)
    one_by_one = torch.stack(outs, dim=1).reshape(batch * steps, hidden)
    diff = float((chunk.float() - one_by_one.float()).norm() / one_by_one.float().norm())
    return diff, prefill_ms, step_ms


def main():
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, default in (("batch", 4), ("prompt", 500), ("steps", 16), ("hidden", 4096), ("heads", 32),
                          ("kv-heads", 8), ("dim", 128), ("page", 16), ("window", 0), ("sinks", 0)):
        p.add_argument("--" + name, type=int, default=default)
    p.add_argument("--cache", choices=["f16", "fp8"], default="f16")
    a = p.parse_args()
    diff, prefill_ms, step_ms = run(a.batch, a.prompt, a.steps, a.hidden, a.heads, a.kv_heads, a.dim, a.page, a.cache,
                                    a.window, a.sinks)
    print(f"prefill {prefill_ms:.3f} ms, decode {step_ms * 1e3:.1f} us per step of {a.batch} tokens, "
          f"decoded against prefilled: relative difference {diff:.2e}")
    if not diff < 0.02:
        raise SystemExit("the two ways disagree")


if __name__ == "__main__":
    main()

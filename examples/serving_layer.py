"""One attention layer on 4-bit weights serving many requests at once: they begin with the same prompt, which lies in the
paged cache once, and each has an adapter of its own on the queries and on the output product. The prompt is prefilled
once, then every request's own question behind it, then all decode token by token. At the end every request is computed
again alone, with a cache of its own, and both ways are compared.

    python examples/serving_layer.py [--requests 32] [--prompt 2000] [--question 40] [--steps 16] [--cache fp8]

(An adapter on keys or values would give every request another cache of the same prompt: only requests of one adapter
could share it then.) Random weights and inputs; needs an MI355X and the built library.
"""

from __future__ import annotations

import argparse
import os
import sys
import time

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import bit_weight_quantized_qgemm_amd as qg  # noqa: E402
from attention_layer import Linear  # noqa: E402


def _pool(n, K, N, rank, gen, device):
    """n random adapters of a K x N projection, whose product is a fraction of the projection's own."""
    a = torch.randn((n, rank, K), generator=gen, device=device) * K ** -0.5
    b = torch.randn((n, N, rank), generator=gen, device=device) * 0.3 * rank ** -0.5
    return qg.LoraAdapters(a.half(), b.half(), scales=torch.rand((n,), generator=gen, device=device) + 0.5)


class Layer:
    def __init__(self, hidden, heads, kv_heads, dim, adapters, rank, max_len, gen, device):
        self.heads, self.kv_heads, self.dim, self.adapters = heads, kv_heads, dim, adapters
        self.qkv = Linear(hidden, (heads + 2 * kv_heads) * dim, gen, device)
        self.out = Linear(heads * dim, hidden, gen, device)
        self.q_adapters = _pool(adapters, hidden, heads * dim, rank, gen, device)
        self.out_adapters = _pool(adapters, heads * dim, hidden, rank, gen, device)
        self.rope = qg.rope_table(max_len, dim, device=device)

    def __call__(self, x, batch, cache, positions, table, token_seq, attend):
        """x [tokens][hidden]; batch: the adapters of its rows; attend(q): attention over the cache."""
        H, KV, D = self.heads, self.kv_heads, self.dim
        qkv = self.qkv(x)
        q = qkv[:, :H * D]
        qg.lora(x, self.q_adapters, batch, base=q, out=q)   # into the fused product's columns of the queries
        q, k, v = (t.unflatten(-1, (-1, D)) for t in qkv.split([H * D, KV * D, KV * D], dim=-1))
        q = qg.qk_rope_append(q, k, v, positions, cache, table, self.rope, token_seq=token_seq)
        o = attend(q).flatten(1)
        y = self.out(o)
        return qg.lora(o, self.out_adapters, batch, base=y, out=y)


def run(requests=32, prompt=2000, question=40, steps=16, hidden=4096, heads=32, kv_heads=8, dim=128, page=16, cache="f16",
        adapters=5, rank=16, seed=0, device="cuda:0"):
    """Returns (relative difference of the two ways, ms of the questions' prefill, ms of a decode step)."""
    device = torch.device(device)
    torch.cuda.set_device(device)
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)
    own = [max(1, question - question * i // (2 * requests)) for i in range(requests)]
    shared = prompt // page * page   # whole pages; the rest of the prompt is part of every question
    own = [n + prompt - shared for n in own]
    lens = [shared + n for n in own]
    max_len = max(lens) + steps
    dtype = {"f16": torch.float16, "fp8": torch.float8_e4m3fn}[cache]
    scale = 1 / 16 if cache == "fp8" else 1.0
    layer = Layer(hidden, heads, kv_heads, dim, adapters, rank, max_len, gen, device)
    ids = torch.arange(requests, dtype=torch.int32) % (adapters + 1)
    ids = torch.where(ids == adapters, -1, ids)   # some requests without an adapter
    x0 = torch.randn((shared, hidden), generator=gen, device=device).half()
    xs = [torch.randn((n, hidden), generator=gen, device=device).half() for n in own]
    new = torch.randn((steps, requests, hidden), generator=gen, device=device).half()

    def int32(t):
        return torch.as_tensor(t, dtype=torch.int32).to(device)

    # ---- together: the prompt's pages once, then each request's own
    first, each = shared // page, -(-(max(own) + steps) // page)
    pages = torch.randperm(first + requests * each, generator=gen, device=device).to(torch.int32)
    table = torch.cat([pages[:first].expand(requests, -1), pages[first:].view(requests, each)], dim=1).contiguous()
    store = qg.KVCache.empty(len(pages), page, kv_heads, dim, dtype, device, scale, scale)
    no_adapter = qg.LoraBatch(torch.full((shared,), -1, dtype=torch.int32, device=device), adapters)
    group_start, shared_lens = int32([0, requests]), int32([shared])
    layer(x0, no_adapter, store, torch.arange(shared, dtype=torch.int32, device=device), table, no_ids(shared, device),
          lambda q: qg.attn_prefill(q, store, table[:1].contiguous(), int32([0, shared]), int32([shared]), shared, shared))
    token_seq = torch.repeat_interleave(torch.arange(requests), torch.tensor(own))
    starts = int32([0] + own).cumsum(0, dtype=torch.int32)
    positions = int32(torch.cat([torch.arange(shared, n) for n in lens]))
    token_batch = qg.LoraBatch(int32(ids[token_seq]), adapters)
    now = int32(lens)

    def questions():
        return layer(torch.cat(xs), token_batch, store, positions, table, int32(token_seq),
                     lambda q: qg.attn_prefill_shared(q, store, table, starts, now, max(own), max(lens), group_start,
                                                      shared_lens, shared))

    batch = qg.LoraBatch(int32(ids), adapters)   # one for every step and projection

    def decode():
        outs, cur = [], now.clone()
        for s in range(steps):
            at = cur.clone()
            cur += 1
            outs.append(layer(new[s], batch, store, at, table, None,
                              lambda q: qg.attn_decode_shared(q, store, table, cur, max_len, group_start, shared_lens, shared)))
        return outs

    def timed(f):
        f()   # a warm-up, which stores the same keys and values
        torch.cuda.synchronize()
        t0 = time.perf_counter()
        out = f()
        torch.cuda.synchronize()
        return out, (time.perf_counter() - t0) * 1e3

    asked, question_ms = timed(questions)
    outs, decode_ms = timed(decode)

    # ---- each request alone: its whole context in one sequence, one adapter for all rows
    worst = 0.0
    table1 = torch.arange(first + each, dtype=torch.int32, device=device)[None]
    at = 0
    for r in range(requests):
        n = lens[r]
        alone = qg.KVCache.empty(first + each, page, kv_heads, dim, dtype, device, scale, scale)

        def rows(count):
            return qg.LoraBatch(torch.full((count,), int(ids[r]), dtype=torch.int32, device=device), adapters)

        y = layer(torch.cat([x0, xs[r]]), rows(n), alone, torch.arange(n, dtype=torch.int32, device=device), table1,
                  no_ids(n, device), lambda q: qg.attn_prefill(q, alone, table1, int32([0, n]), int32([n]), n, n))
        pairs = [(asked[at:at + own[r]], y[shared:])]
        at += own[r]
        for s in range(steps):
            length = int32([n + s + 1])
            y = layer(new[s, r:r + 1].contiguous(), rows(1), alone, length - 1, table1, None,
                      lambda q: qg.attn_decode(q, alone, table1, length, max_len))
            pairs.append((outs[s][r:r + 1], y))
        worst = max([worst] + [float((a.float() - b.float()).norm() / b.float().norm()) for a, b in pairs])
    return worst, question_ms, decode_ms / max(1, steps)


def no_ids(n, device):
    """Sequence 0 for n tokens."""
    return torch.zeros((n,), dtype=torch.int32, device=device)


def main():
    p = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    for name, default in (("requests", 32), ("prompt", 2000), ("question", 40), ("steps", 16), ("hidden", 4096),
                          ("heads", 32), ("kv-heads", 8), ("dim", 128), ("page", 16), ("adapters", 5), ("rank", 16)):
        p.add_argument("--" + name, type=int, default=default)
    p.add_argument("--cache", choices=["f16", "fp8"], default="f16")
    a = p.parse_args()
    diff, question_ms, step_ms = run(a.requests, a.prompt, a.question, a.steps, a.hidden, a.heads, a.kv_heads, a.dim, a.page,
                                     a.cache, a.adapters, a.rank)
    print(f"questions {question_ms:.3f} ms, decode {step_ms * 1e3:.1f} us per step of {a.requests} tokens, "
          f"together against each alone: relative difference {diff:.2e}")
    if not diff < 0.02:
        raise SystemExit("the two ways disagree")


if __name__ == "__main__":
    main()

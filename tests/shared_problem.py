"""Paged-cache problems whose sequences share pages: NumPy inputs as bit patterns, device tensors, oracle outputs."""

import numpy as np
import torch

import bit_weight_quantized_qgemm_amd as qg
from attn_problem import NAN, Paged
from oracle import attention as oa


class SharedPaged(Paged):
    """A Paged cache in which the sequences of group g have their first pages in common.

    groups: per group (sequences, shared pages, tokens said to be shared: up to that many pages); before: sequences in
    front of the first group; the rest follow the last. A shared page holds the same tokens for all; what a sequence
    does not reach of it is still there (and finite)."""

    def __init__(self, rng, lens, groups, kv_heads, dim, fmt, page, dev, layout="heads", scales=(1.0, 1.0), before=0,
                 missing=()):
        self.lens, self.kv_heads, self.dim, self.fmt, self.page, self.scales = lens, kv_heads, dim, fmt, page, scales
        of = np.full(len(lens), -1)
        at = before
        for g, (n, _, _) in enumerate(groups):
            of[at:at + n] = g
            at += n
        assert at <= len(lens)
        self.of = of
        need = [-(-n // page) for n in lens]
        shared_pages = [p for _, p, _ in groups]
        pool = sum(shared_pages) + sum(need) + 2
        order = rng.permutation(pool).astype(np.int32)
        cols = max(need + shared_pages + [0]) + 1
        self.table = np.full((len(lens), cols), -1, dtype=np.int32)
        self.table[:, -1] = np.iinfo(np.int32).max
        at, heads_of = 0, []
        for p in shared_pages:
            heads_of.append(order[at:at + p])
            at += p
        for b, n in enumerate(need):
            first = shared_pages[of[b]] if of[b] >= 0 else 0
            if first:
                self.table[b, :first] = heads_of[of[b]]
            if n > first:
                self.table[b, first:n] = order[at:at + n - first]
                at += n - first
        dtype = np.uint8 if fmt == "fp8" else np.uint16
        self.bits = [np.full((pool, page, kv_heads, dim), NAN[fmt], dtype=dtype) for _ in range(2)]
        values = [np.full((pool, page, kv_heads, dim), np.nan) for _ in range(2)]

        def fill(pages, tokens):
            for i in range(2):
                x = rng.standard_normal((tokens, kv_heads, dim)) + (0.25 if i else 0.0)
                bits = oa.encode(x / scales[i], fmt)
                val = oa.decode(bits, fmt) * scales[i]
                for j in range(tokens):
                    self.bits[i][pages[j // page], j % page] = bits[j]
                    values[i][pages[j // page], j % page] = val[j]

        for pages in heads_of:
            fill(pages, len(pages) * page)
        for b, n in enumerate(lens):
            first = shared_pages[of[b]] if of[b] >= 0 else 0
            if n > first * page:
                fill(self.table[b, first:], n - first * page)
        self.tokens = []
        for b, n in enumerate(lens):
            j = np.arange(n)
            self.tokens.append([v[self.table[b, j // page], j % page] for v in values])
        self.lost = np.zeros((len(lens), max(list(lens) + [1])), dtype=bool)
        for b, col, entry in missing:
            self.table[b, col] = entry if entry < 0 else pool + entry
            self.lost[b, col * page:(col + 1) * page] = True
        self.k, self.v = (self._place(x, layout, dev) for x in self.bits)
        self.cache = qg.KVCache(self.k, self.v, *scales)
        self.table_dev = torch.from_numpy(self.table).to(dev)
        self.lens_dev = torch.tensor(lens, dtype=torch.int32, device=dev)
        starts = before + np.concatenate([[0], np.cumsum([n for n, _, _ in groups])])
        self.group_start = torch.tensor(starts, dtype=torch.int32, device=dev)
        self.shared_lens = torch.tensor([s for _, _, s in groups], dtype=torch.int32, device=dev)
        self.max_shared = max([s for _, _, s in groups] + [0])

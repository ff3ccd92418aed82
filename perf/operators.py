"""Cases, plain forms and exact values of the attention operators around a paged key-value cache.

Three operators that stand between the quantized linear layers of a decoder layer:

* ``append``: norms of queries and keys per head, position rotation, and the store of keys and
  values into a paged cache, in one pass over the output of the fused q/k/v product;
* ``decode``: attention of one new token per sequence over that cache;
* ``prefill``: attention of many new tokens per sequence (a prompt, a chunk of one, a few
  speculated tokens) over that cache, causal.

Both attentions know a sliding window with a few first tokens that stay visible (sinks), groups of
query heads that share a key-value head, and a cache in the activations' type or in 8 bits (e4m3).
``own`` selects the framework's kernels; otherwise the operators are computed by elementary torch
operations in 32 bits.
"""

import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn}
FP8_MAX = 448.0
EPS = 1e-6
THETA = 10000.0


# ------------------------------------------------------------------------------------------ cases
def _append(name, T, heads, kv_heads, dim, dtype, cache, seqs, page=16, rot=0, norm=True, interleaved=False):
    return {"name": name, "op": "append", "tokens": T, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "dtype": dtype, "cache": cache, "seqs": seqs, "page": page, "rot": rot or dim, "norm": norm,
            "interleaved": interleaved}


def _attend(name, op, seqs, q_len, kv_len, heads, kv_heads, dim, dtype, cache, page=16, window=0, sinks=0,
            ragged=False):
    return {"name": name, "op": op, "seqs": seqs, "q_len": q_len, "kv_len": kv_len, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "dtype": dtype, "cache": cache, "page": page, "window": window,
            "sinks": sinks, "ragged": ragged}


def listed():
    return [
        # one sequence's next token, heads of a 4096-wide layer: a call whose latency counts
        _append("append 1 token, 32/32 heads", 1, 32, 32, 128, "f16", "f16", 1),
        # a decoding batch, heads of an 8192-wide layer, 8-bit cache
        _append("append 128 tokens, 64/8 heads, fp8 cache", 128, 64, 8, 128, "bf16", "fp8", 128, page=32),
        # a ragged batch of prompts, head length 80, half of each head rotated, interleaved pairs, no norms
        _append("append 1003 tokens, 32/32 heads of 80, interleaved", 1003, 32, 32, 80, "f16", "f16", 5, rot=32,
                norm=False, interleaved=True),
        # one long prompt
        _append("append 8192 tokens, 64/8 heads", 8192, 64, 8, 128, "bf16", "bf16", 1),
        # one sequence decoding at a short context: latency
        _attend("decode 1 x 1000, 32/32 heads", "decode", 1, 1, 1000, 32, 32, 128, "f16", "f16"),
        # an ordinary serving batch with ragged contexts, eight query heads to a key-value head
        _attend("decode 32 x 4096 ragged, 64/8 heads", "decode", 32, 1, 4096, 64, 8, 128, "bf16", "bf16", ragged=True),
        # one very long context in an 8-bit cache: few rows, the cache's length has to be split
        _attend("decode 1 x 131072, 64/8 heads, fp8 cache", "decode", 1, 1, 131072, 64, 8, 128, "f16", "fp8", page=64),
        # long contexts of which a window and a few first tokens are visible; heads of 64
        _attend("decode 64 x 16384, window 1024 and 4 sinks", "decode", 64, 1, 16384, 32, 8, 64, "bf16", "bf16",
                window=1024, sinks=4, ragged=True),
        # a few speculated tokens on a long context: few rows, split
        _attend("prefill 2 x 5 on 6001, 64/8 heads", "prefill", 2, 5, 6001, 64, 8, 128, "bf16", "bf16"),
        # a ragged batch of prompts
        _attend("prefill 4 x 2048 ragged, 32/32 heads", "prefill", 4, 2048, 2048, 32, 32, 128, "f16", "f16", ragged=True),
        # one long prompt with a window and sinks, 8-bit cache
        _attend("prefill 1 x 8192, window 1024 and 4 sinks, fp8 cache", "prefill", 1, 8192, 8192, 32, 8, 128, "bf16",
                "fp8", page=32, window=1024, sinks=4),
        # one long prompt
        _attend("prefill 1 x 8192, 64/8 heads", "prefill", 1, 8192, 8192, 64, 8, 128, "bf16", "bf16"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "decode", "prefill"])
    heads, kv_heads = rng.choice([(32, 32), (32, 8), (64, 8), (28, 4), (40, 8), (16, 1), (8, 2), (20, 20)])
    dim = rng.choice([64, 80, 96, 128, 128, 128, 256])
    dtype = rng.choice(["f16", "bf16"])
    cache = rng.choice([dtype, dtype, "fp8"])
    page = rng.choice([16, 32, 64, 128, 256, 48])
    if op == "append":
        T = _log(rng, 1, 8192 * 64 * 128 // max(64 * 128, heads * dim))
        rot = rng.choice([dim, dim, 32])
        c = _append("", T, heads, kv_heads, dim, dtype, cache, rng.randint(1, min(T, 16)), page, rot,
                    rng.random() < 0.7, rng.random() < 0.4)
    else:
        window, sinks = rng.choice([(0, 0), (0, 0), (rng.randint(1, 4096), rng.choice([0, 1, 4, 37]))])
        ragged = rng.random() < 0.6
        if op == "decode":
            seqs = _log(rng, 1, 128)
            most = 131072 * 8 * 128 // (seqs * kv_heads * dim)
            kv_len, q_len = _log(rng, 1, max(1, min(131072, most))), 1
        else:
            seqs = rng.choice([1, 1, 2, 3, 5, 8])
            share = min(1.0, 64 * 128 / (seqs * heads * dim))    # of the largest listed case's scores
            q_len = _log(rng, 1, int(8192 * math.sqrt(share)))
            most = min(16384, int(8192 * 8192 * share / 2) // q_len)
            kv_len = q_len + (0 if rng.random() < 0.5 or most <= q_len else rng.randint(0, most - q_len))
        c = _attend("", op, seqs, q_len, kv_len, heads, kv_heads, dim, dtype, cache, page, window, sinks, ragged)
    del c["name"]
    return c


# --------------------------------------------------------------------------------- a case's lengths
def _spread(n, most, ragged):
    """Lengths of n sequences: all `most`, or spread over 1..most with `most` among them."""
    if not ragged:
        return [most] * n
    return [most if i == 0 else max(1, int(most * ((i * 0.6180339887) % 1.0))) for i in range(n)]


def _lengths(case):
    """(new tokens, cache length with them) of each sequence."""
    if case["op"] == "append":
        n, T = case["seqs"], case["tokens"]
        q = [T // n + (1 if i < T % n else 0) for i in range(n)]
        before = [0 if T > 4 * n else 100 + 97 * i % 400 for i in range(n)]    # prompts, or decoding
        return q, [a + b for a, b in zip(q, before)]
    kv = _spread(case["seqs"], case["kv_len"], case["ragged"])
    if case["op"] == "decode":
        return [1] * len(kv), kv
    return [min(case["q_len"], n) for n in kv], kv


def _visible(first, last, window, sinks):
    """Number of (query, key) pairs of the queries at positions first..last-1."""
    if not window:
        return (first + 1 + last) * (last - first) // 2
    total = 0
    for i in range(first, last):
        low = max(0, i + 1 - window)
        total += i + 1 - low + min(sinks, low)
    return total


def work(case):
    H, KV, D = case["heads"], case["kv_heads"], case["dim"]
    cb = 1 if case["cache"] == "fp8" else 2
    if case["op"] == "append":
        T, norms = case["tokens"], 2 * 2 * D * case["norm"]
        rope = 4 * case["rot"] * min(T, max(_lengths(case)[1]))
        return {"bytes": T * (2 * H * D * 2 + 2 * KV * D * (2 + cb) + 8) + rope + norms,
                "flops": T * (H + KV) * (4 * D * case["norm"] + 3 * case["rot"])}
    q, kv = _lengths(case)
    pairs = sum(_visible(n - m, n, case["window"], case["sinks"]) for m, n in zip(q, kv))
    keys = 0
    for m, n in zip(q, kv):    # tokens that at least one query sees
        low = max(0, n - m + 1 - case["window"]) if case["window"] else 0
        keys += n - low + min(case["sinks"], low)
    return {"bytes": 2 * sum(q) * H * D * 2 + 2 * keys * KV * D * cb, "flops": 4 * pairs * H * D}


# ------------------------------------------------------------------------------------------ inputs
def _pages(case, gen, dev):
    """A block table over a shuffled pool of pages with some to spare, and the pool's size."""
    lens, page = _lengths(case)[1], case["page"]
    need = [-(-n // page) for n in lens]
    pool = sum(need) + 3
    order = torch.randperm(pool, generator=gen, device=dev).to(torch.int32)
    table = torch.full((len(lens), max(need)), -1, dtype=torch.int32, device=dev)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    return table, pool


def _cache(case, pool, gen, dev):
    """Keys and values of earlier tokens, [pages][heads][page][dim] in memory, seen as [pages][page][heads][dim]."""
    dt, got = DTYPES[case["cache"]], []
    for _ in range(2):
        shape = (pool, case["kv_heads"], case["page"], case["dim"])
        t = torch.empty(shape, dtype=torch.float16 if dt == DTYPES["fp8"] else dt, device=dev).normal_(generator=gen)
        if dt == DTYPES["fp8"]:
            out = torch.empty(shape, dtype=dt, device=dev)
            step = max(1, (1 << 27) // t[0].numel())
            for i in range(0, pool, step):
                out[i:i + step] = (t[i:i + step] * 32).to(dt)    # the scale below is 1/32
            t = out
        got.append(t.transpose(1, 2))
    return got


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dt, D = DTYPES[case["dtype"]], case["dim"]
    H, KV = case["heads"], case["kv_heads"]
    q_lens, kv_lens = _lengths(case)
    T = sum(q_lens)
    s = {"case": case, "max_q": max(q_lens), "max_len": max(kv_lens)}
    s["table"], pool = _pages(case, gen, dev)
    s["k"], s["v"] = _cache(case, pool, gen, dev)
    s["scales"] = (1 / 32, 1 / 32) if case["cache"] == "fp8" else (1.0, 1.0)
    s["lens"] = torch.tensor(kv_lens, dtype=torch.int32, device=dev)
    if case["op"] == "append":
        # the fused product's output, its three parts seen per head
        qkv = torch.randn((T, (H + 2 * KV) * D), generator=gen, device=dev).to(dt)
        s["q"], s["new_k"], s["new_v"] = (x.unflatten(-1, (-1, D)) for x in qkv.split([H * D, KV * D, KV * D], dim=-1))
        s["positions"] = torch.cat([torch.arange(n - m, n, dtype=torch.int32) for m, n in zip(q_lens, kv_lens)]).to(dev)
        s["token_seq"] = torch.repeat_interleave(torch.arange(len(q_lens), dtype=torch.int32),
                                                 torch.tensor(q_lens)).to(torch.int32).to(dev)
        rows, half = max(kv_lens), case["rot"] // 2
        angle = torch.arange(rows, dtype=torch.float64)[:, None] * THETA ** (-torch.arange(half, dtype=torch.float64) / half)
        s["rope"] = torch.cat([angle.cos(), angle.sin()], dim=1).to(torch.float32).to(dev)
        if case["norm"]:
            s["q_norm"], s["k_norm"] = ((1 + 0.1 * torch.randn((D,), generator=gen, device=dev)).to(dt) for _ in range(2))
        else:
            s["q_norm"] = s["k_norm"] = None
    else:
        s["q"] = torch.randn((T, H, D), generator=gen, device=dev).to(dt)
        starts = [0]
        for m in q_lens:
            starts.append(starts[-1] + m)
        s["starts"] = torch.tensor(starts, dtype=torch.int32, device=dev)
    if own:
        import bit_weight_quantized_qgemm_amd as qg

        s["cache"] = qg.KVCache(s["k"], s["v"], *s["scales"])
    return s


# --------------------------------------------------------------------------------------- the passes
def run(state):
    op = state["case"]["op"]
    if own:
        return _run_own(state, op)
    if op == "append":
        return _plain_append(state)
    return _plain_attend(state)


def _run_own(s, op):
    import bit_weight_quantized_qgemm_amd as qg

    c = s["case"]
    if op == "append":
        q = qg.qk_rope_append(s["q"], s["new_k"], s["new_v"], s["positions"], s["cache"], s["table"], s["rope"],
                              q_norm=s["q_norm"], k_norm=s["k_norm"], eps=EPS, token_seq=s["token_seq"],
                              interleaved=c["interleaved"])
        return q, s["k"], s["v"]
    if op == "decode":
        return qg.attn_decode(s["q"], s["cache"], s["table"], s["lens"], s["max_len"], window=c["window"],
                              sinks=c["sinks"])
    return qg.attn_prefill(s["q"], s["cache"], s["table"], s["starts"], s["lens"], s["max_q"], s["max_len"],
                           window=c["window"], sinks=c["sinks"])


def _plain_rotate(x, s):
    """Rotates the first `rot` values of each head by its token's angles; x: fp32 [T][heads][dim]."""
    rot, half = s["case"]["rot"], s["case"]["rot"] // 2
    row = s["rope"][s["positions"].long()][:, None, :]
    cos, sin = row[..., :half], row[..., half:]
    if s["case"]["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([turned, x[..., rot:]], dim=-1)


def _plain_append(s):
    c = s["case"]

    def normed(x, w):
        x = x.float()
        if w is None:
            return x
        return x * torch.rsqrt((x * x).mean(dim=-1, keepdim=True) + EPS) * w.float()

    q = _plain_rotate(normed(s["q"], s["q_norm"]), s).to(s["q"].dtype)
    k = _plain_rotate(normed(s["new_k"], s["k_norm"]), s)
    v = s["new_v"].float()
    at = s["positions"].long()
    page = s["table"][s["token_seq"].long(), at // c["page"]].long()
    for buf, x, scale in ((s["k"], k, s["scales"][0]), (s["v"], v, s["scales"][1])):
        if c["cache"] == "fp8":
            x = (x / scale).clamp(-FP8_MAX, FP8_MAX).to(buf.dtype)
            buf.view(torch.uint8)[page, at % c["page"]] = x.view(torch.uint8)
        else:
            buf[page, at % c["page"]] = x.to(buf.dtype)
    return q, s["k"], s["v"]


def _gathered(buf, table, scale):
    """A sequence's cache in order, fp32 [seqs][tokens][heads][dim]."""
    at = table.clamp(min=0).long()
    if buf.dtype == torch.float8_e4m3fn:
        return buf.view(torch.uint8)[at].view(torch.float8_e4m3fn).flatten(1, 2).float() * scale
    return buf[at].flatten(1, 2).float()


def _plain_attend(s):
    c = s["case"]
    H, KV, D = c["heads"], c["kv_heads"], c["dim"]
    B, S, L, G = c["seqs"], s["max_q"], s["max_len"], c["heads"] // c["kv_heads"]
    dev = s["q"].device
    lens, starts = s["lens"].long(), s["starts"].long()
    new = starts[1:] - starts[:-1]
    slot = torch.arange(S, device=dev)
    live = slot[None, :] < new[:, None]                                   # [B][S]
    row = (starts[:-1, None] + slot[None, :]).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][row].float()                                               # [B][S][H][D]
    q = q.view(B, S, KV, G, D).permute(0, 2, 3, 1, 4).reshape(B * KV, G * S, D)
    token = torch.arange(L, device=dev)
    there = token[None, :] < lens[:, None]                                # [B][L]
    k = _gathered(s["k"], s["table"], s["scales"][0])[:, :L].permute(0, 2, 3, 1).reshape(B * KV, D, L).contiguous()
    v = _gathered(s["v"], s["table"], s["scales"][1])[:, :L]
    v = torch.where(there[:, :, None, None], v, 0.0).permute(0, 2, 1, 3).reshape(B * KV, L, D).contiguous()
    where = (lens - new)[:, None] + slot[None, :]                         # a query's position
    seen = there[:, None, :] & (token[None, None, :] <= where[:, :, None])
    if c["window"]:
        seen &= (token[None, None, :] > where[:, :, None] - c["window"]) | (token[None, None, :] < c["sinks"])
    seen = seen[:, None, None]                                            # [B][1][1][S][L]
    score = torch.matmul(q, k).view(B, KV, G, S, L).mul_(1 / math.sqrt(D)).masked_fill_(~seen, float("-inf"))
    top = score.amax(dim=-1, keepdim=True)
    p = score.sub_(torch.where(top == float("-inf"), 0.0, top)).exp_()
    total = p.sum(dim=-1, keepdim=True)
    out = torch.matmul(p.view(B * KV, G * S, L), v).view(B, KV, G, S, D)
    out = torch.where(total > 0, out / total, 0.0)
    out = out.permute(0, 3, 1, 2, 4).reshape(B, S, H, D)
    return out[live].to(s["q"].dtype)


# -------------------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "append":
        return _exact_append(case, s)
    return _exact_attend(case, s)


def _exact_append(case, s):
    D, half, rot = case["dim"], case["rot"] // 2, case["rot"]
    turn = torch.complex(s["rope"][:, :half].double(), s["rope"][:, half:].double())[s["positions"].long()][:, None]

    def rotated(x, w):
        x = x.double()
        if w is not None:
            x = x / (x.pow(2).sum(-1, keepdim=True) / D + EPS).sqrt() * w.double()
        if case["interleaved"]:
            pairs = torch.view_as_complex(x[..., :rot].unflatten(-1, (half, 2)).contiguous())
        else:
            pairs = torch.complex(x[..., :half].contiguous(), x[..., half:rot].contiguous())
        pairs = pairs * turn
        out = x.clone()
        if case["interleaved"]:
            out[..., :rot] = torch.view_as_real(pairs).flatten(-2)
        else:
            out[..., :half], out[..., half:rot] = pairs.real, pairs.imag
        return out

    q, k = rotated(s["q"], s["q_norm"]), rotated(s["new_k"], s["k_norm"])
    # the caches hold other tokens too, and in 8 bits a rounded value: no exact value of their own
    if case["cache"] == "fp8":
        return q, None, None
    kc, vc = s["k"].double(), s["v"].double()
    n = torch.arange(q.shape[0], device=q.device)
    pos = s["positions"].long()
    page = s["table"].long()[s["token_seq"].long()[n], torch.div(pos, case["page"], rounding_mode="floor")]
    kc[page, torch.remainder(pos, case["page"])] = k
    vc[page, torch.remainder(pos, case["page"])] = s["new_v"].double()
    return q, kc, vc


def _exact_attend(case, s):
    q_lens, kv_lens = _lengths(case)
    H, KV, D, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    dev = s["q"].device
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=dev)
    first = 0
    for b, (m, n) in enumerate(zip(q_lens, kv_lens)):
        ids = s["table"][b, :-(-n // page)].long()
        j = torch.arange(n, device=dev)
        for h in range(KV):
            # pages are picked as whole numbers of the same width: an index over 8-bit floats is not there everywhere
            kk, vv = (buf.view(torch.uint8 if buf.itemsize == 1 else torch.int16)[ids, :, h].reshape(-1, D)[:n]
                      .view(buf.dtype).double() * scale for buf, scale in zip((s["k"], s["v"]), s["scales"]))
            kt = kk.t().contiguous()
            step = max(1, (1 << 28) // n)
            for g in range(h * (H // KV), (h + 1) * (H // KV)):
                for r in range(0, m, step):
                    e = min(m, r + step)
                    i = torch.arange(n - m + r, n - m + e, device=dev)[:, None]
                    hide = j[None] > i
                    if case["window"]:
                        hide = hide | ((j[None] <= i - case["window"]) & (j[None] >= case["sinks"]))
                    z = s["q"][first + r:first + e, g].double() @ kt / math.sqrt(D)
                    w = torch.softmax(z.masked_fill(hide, float("-inf")), dim=-1)
                    out[first + r:first + e, g] = w @ vv
        first += m
    return out

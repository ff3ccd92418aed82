"""Cases, plain forms and exact values of the operators for many requests at once.

Two kinds of operator that a layer needs when its requests differ in some things and share others:

* ``lora``: low-rank adapters beside a shared projection. Each row of a batch adds the product with its own
  request's pair of low-rank matrices to the shared product's output; the projection may be a fused one (several
  column ranges, each with a first matrix of its own), adapters may differ in rank, rows may have none;
* ``decode`` and ``prefill``: attention over a paged key-value cache, one or several new tokens per sequence, for a
  batch whose sequences begin with the same long prefix, group by group: the prefix lies in the cache once and is
  computed once for all rows of its group.

``own`` selects the framework's kernels; otherwise the operators are computed by elementary torch operations in 32 bits.
"""

import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn}


# ------------------------------------------------------------------------------------------ cases
def _lora(name, T, K, widths, rank, used, dtype, pool=0, prompts=False, mixed=False, none=False):
    return {"name": name, "op": "lora", "tokens": T, "k": K, "widths": ",".join(map(str, widths)), "rank": rank,
            "used": used, "pool": pool or used + 2, "dtype": dtype, "prompts": prompts, "mixed": mixed, "none": none}


def _attend(name, op, seqs, groups, q_len, shared, own_len, heads, kv_heads, dim, dtype, cache, page=16, window=0,
            sinks=0, ragged=False, loners=0):
    return {"name": name, "op": op, "seqs": seqs, "groups": groups, "q_len": q_len, "shared": shared,
            "own_len": own_len, "heads": heads, "kv_heads": kv_heads, "dim": dim, "dtype": dtype, "cache": cache,
            "page": page, "window": window, "sinks": sinks, "ragged": ragged, "loners": loners}


def listed():
    return [
        # one request's next token through a square projection: a call whose latency counts
        _lora("lora 1 token 4096 to 4096 rank 16", 1, 4096, [4096], 16, 1, "f16", pool=8),
        # a decoding batch in which every request has its own adapter, on the fused q/k/v product
        _lora("lora 64 tokens of 64 adapters fused q/k/v rank 16", 64, 8192, [8192, 1024, 1024], 16, 64, "bf16"),
        # a decoding batch of adapters of different ranks, in no order, some requests without one, on a wide projection
        _lora("lora 128 tokens of 24 adapters ranks to 64", 128, 8192, [28672], 64, 24, "f16", mixed=True, none=True),
        # a ragged batch of prompts
        _lora("lora 1003 tokens of 5 prompts 4096 to 11008", 1003, 4096, [11008], 64, 5, "f16", prompts=True),
        # long prompts
        _lora("lora 8192 tokens of 3 prompts 8192 to 8192", 8192, 8192, [8192], 16, 3, "bf16", prompts=True),
        # a few short requests behind one short prompt: latency
        _attend("decode 4 on 768 shared 32/32 heads", "decode", 4, 1, 1, 768, 130, 32, 32, 128, "f16", "f16"),
        # a serving batch behind one long system prompt, eight query heads to a key-value head
        _attend("decode 64 on 8192 shared 64/8 heads", "decode", 64, 1, 1, 8192, 512, 64, 8, 128, "bf16", "bf16",
                ragged=True),
        # several system prompts of different lengths at once, some requests without one, 8-bit cache
        _attend("decode 96 in 4 groups 32/8 heads fp8 cache", "decode", 96, 4, 1, 4096, 700, 32, 8, 128, "bf16", "fp8",
                page=32, ragged=True, loners=5),
        # unshared heads: every sequence's cache is large, one row of it for each
        _attend("decode 128 on 2048 shared 32/32 heads", "decode", 128, 1, 1, 2048, 256, 32, 32, 128, "f16", "f16",
                ragged=True),
        # a few speculated tokens per sequence
        _attend("prefill 16 x 5 on 6000 shared 64/8 heads", "prefill", 16, 1, 5, 6000, 100, 64, 8, 128, "bf16", "bf16",
                ragged=True),
        # ragged questions behind one prompt, heads of 80
        _attend("prefill 24 ragged on 2048 shared 32/32 heads of 80", "prefill", 24, 1, 200, 2048, 200, 32, 32, 80,
                "f16", "f16", ragged=True),
        # chunks of 128 tokens behind a very long document, 8-bit cache
        _attend("prefill 32 x 128 on 16384 shared fp8 cache", "prefill", 32, 1, 128, 16384, 128, 32, 8, 128, "bf16",
                "fp8", page=64),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    if rng.random() < 0.45:
        T = _log(rng, 1, 4096)
        K = rng.choice([1024, 4096, 8192, 8 * _log(rng, 16, 1024)])
        widths = rng.choice([[1024], [4096], [8192], [11008], [4096, 1024, 1024], [1024, 1024, 1024], [11008, 11008],
                             [8 * _log(rng, 16, 1024)]])
        rank = rng.choice([8, 16, 16, 32, 64, 128, 40])
        used = _log(rng, 1, min(T, 64))
        c = _lora("", T, K, widths, rank, used, rng.choice(["f16", "bf16"]), prompts=T > 300 and rng.random() < 0.8,
                  mixed=rng.random() < 0.4, none=rng.random() < 0.3, pool=used + rng.randint(0, 9))
    else:
        op = rng.choice(["decode", "decode", "prefill"])
        heads, kv_heads = rng.choice([(32, 32), (32, 8), (64, 8), (28, 4), (40, 8), (16, 1), (8, 2), (20, 20)])
        dim = rng.choice([64, 80, 96, 128, 128, 128, 256])
        dtype = rng.choice(["f16", "bf16"])
        window, sinks = rng.choice([(0, 0), (0, 0), (0, 0), (rng.randint(1, 6000), rng.choice([0, 1, 4, 37]))])
        seqs = _log(rng, 2, 128 if op == "decode" else 48)
        q_len = 1 if op == "decode" else _log(rng, 1, 160)
        groups = rng.choice([1, 1, 1, 2, 3, 5])
        loners = rng.choice([0, 0, 1, 3])
        c = _attend("", op, seqs, min(groups, seqs), q_len, _log(rng, 64, 16384), q_len + _log(rng, 1, 400), heads,
                    kv_heads, dim, dtype, rng.choice([dtype, dtype, "fp8"]), rng.choice([16, 32, 64, 128, 48]), window,
                    sinks, rng.random() < 0.7, loners)
        # no more rows than the largest listed case has
        most = 32 * 128 * 32 * 128 // (q_len * heads * dim)
        c["seqs"] = max(c["groups"], min(seqs, most))
    del c["name"]
    return c


# --------------------------------------------------------------------------------- a case's structure
def _spread(n, most, ragged):
    """Lengths of n sequences: all `most`, or spread over 1..most with `most` among them."""
    if not ragged:
        return [most] * n
    return [most if i == 0 else max(1, int(most * ((i * 0.6180339887) % 1.0))) for i in range(n)]


def _widths(case):
    return [int(w) for w in case["widths"].split(",")]


def _users(case):
    """The adapter in use (0..used-1, or -1) of each row, and each one's rank."""
    T, used = case["tokens"], case["used"]
    if case["prompts"]:
        share = [0.5 + (i * 0.6180339887) % 1.0 for i in range(used)]
        ends = [round(T * sum(share[:i + 1]) / sum(share)) for i in range(used)]
        ids = [next(i for i, e in enumerate(ends) if t < e) for t in range(T)]
    else:
        ids = [(t * 7919) % used for t in range(T)]
    if case["none"]:
        ids = [-1 if t % 8 == 5 else i for t, i in enumerate(ids)]
    ranks = [8 * max(1, case["rank"] // 8 >> i % 4) if case["mixed"] else case["rank"] for i in range(used)]
    return ids, ranks


def _groups(case):
    """Per sequence (loners last) the group, -1 for none; per group the shared length, whole pages."""
    n, g, page = case["seqs"], case["groups"], case["page"]
    of = [i * g // n for i in range(n)] + [-1] * case["loners"]
    most = max(1, case["shared"] // page)
    return of, [max(1, int(most * (1 - 0.22 * i))) * page for i in range(g)]


def _lengths(case):
    """(new tokens, cache length with them, shared tokens) of each sequence."""
    of, shared = _groups(case)
    mine = _spread(len(of), case["own_len"], case["ragged"])
    base = [shared[g] if g >= 0 else 0 for g in of]
    return [min(case["q_len"], n) for n in mine], [b + n for b, n in zip(base, mine)], base


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
    if case["op"] == "lora":
        ids, ranks = _users(case)
        K, widths = case["k"], _widths(case)
        N, S = sum(widths), len(widths)
        live = [ranks[i] for i in ids if i >= 0]
        weights = sum(ranks[i] for i in set(ids) if i >= 0) * (S * K + N)
        return {"bytes": 2 * (len(live) * K + weights + 2 * len(ids) * N) + 4 * len(ids),
                "flops": 2 * sum(live) * (S * K + N)}
    H, KV, D = case["heads"], case["kv_heads"], case["dim"]
    window, sinks = case["window"], case["sinks"]
    q, kv, base = _lengths(case)
    of, shared = _groups(case)
    pairs = sum(_visible(n - m, n, window, sinks) for m, n in zip(q, kv))
    keys, first = 0, list(shared)    # tokens that some query sees; a group's first shared token behind the sinks
    for m, n, s, g in zip(q, kv, base, of):
        low = max(0, n - m + 1 - window) if window else 0
        keys += n - max(s, low) + (min(sinks, low) - s if sinks > s and low > s else 0)
        if g >= 0:
            first[g] = min(first[g], low)
    for s, low in zip(shared, first):
        keys += s - low + min(sinks, low)
    cb = 1 if case["cache"] == "fp8" else 2
    return {"bytes": 2 * sum(q) * H * D * 2 + 2 * keys * KV * D * cb, "flops": 4 * pairs * H * D}


# ------------------------------------------------------------------------------------------ inputs
def _prepare_lora(case, gen, dev):
    T, K, R, pool = case["tokens"], case["k"], case["rank"], case["pool"]
    widths, dt = _widths(case), DTYPES[case["dtype"]]
    S, N = len(widths), sum(widths)
    logical, ranks = _users(case)
    place = torch.randperm(pool, generator=gen, device=dev)[:case["used"]]    # where the adapters in use lie
    ids = torch.tensor(logical, device=dev)
    ids = torch.where(ids >= 0, place[ids.clamp(min=0)], -1).to(torch.int32)
    rank = torch.full((pool,), R, dtype=torch.int32, device=dev)
    rank[place] = torch.tensor(ranks, dtype=torch.int32, device=dev)

    def normal(shape, dev_of):
        return (torch.randn(shape, generator=gen, device=dev) * dev_of).to(dt)

    s = {"x": normal((T, K), 1.0), "a": normal((pool, S, R, K), K ** -0.5), "b": normal((pool, N, R), 0.3 * R ** -0.5),
         "base": normal((T, N), 1.0), "ids": ids, "ranks": rank if case["mixed"] else None, "widths": widths,
         "scales": 0.5 + torch.rand((pool,), generator=gen, device=dev)}
    if own:
        import bit_weight_quantized_qgemm_amd as qg

        s["adapters"] = qg.LoraAdapters(s["a"], s["b"], scales=s["scales"], ranks=s["ranks"], widths=widths)
        s["batch"] = qg.LoraBatch(ids, pool)    # one for all layers of a step
    return s


def _prepare_attend(case, gen, dev):
    dt, ct, D, page = DTYPES[case["dtype"]], DTYPES[case["cache"]], case["dim"], case["page"]
    H, KV = case["heads"], case["kv_heads"]
    q_lens, kv_lens, base = _lengths(case)
    of, shared = _groups(case)
    B, T = len(q_lens), sum(q_lens)
    # pages: a group's shared ones once, then each sequence's own
    need = [-(-n // page) for n in kv_lens]
    total = sum(s // page for s in shared) + sum(n - b // page for n, b in zip(need, base))
    pool = total + 3
    order = torch.randperm(pool, generator=gen, device=dev).to(torch.int32).cpu()
    table = torch.full((B, max(need)), -1, dtype=torch.int32)
    at, head = 0, []
    for s in shared:
        head.append(order[at:at + s // page])
        at += s // page
    for b, (n, g) in enumerate(zip(need, of)):
        first = len(head[g]) if g >= 0 else 0
        if g >= 0:
            table[b, :first] = head[g]
        table[b, first:n] = order[at:at + n - first]
        at += n - first
    buffers = []
    for _ in range(2):
        shape = (pool, KV, page, D)
        t = torch.empty(shape, dtype=torch.float16 if ct == DTYPES["fp8"] else ct, device=dev).normal_(generator=gen)
        if ct == DTYPES["fp8"]:
            t = (t * 32).to(ct)    # the scale below is 1/32
        buffers.append(t.transpose(1, 2))
    starts = torch.tensor([0] + q_lens).cumsum(0)
    seq = torch.repeat_interleave(torch.arange(B), torch.tensor(q_lens))
    group_start = [of.index(g) for g in range(case["groups"])] + [case["seqs"]]

    def int32(x):
        return torch.as_tensor(x).to(torch.int32).to(dev)

    s = {"q": torch.randn((T, H, D), generator=gen, device=dev).to(dt), "k": buffers[0], "v": buffers[1],
         "table": table.to(dev), "lens": int32(kv_lens), "starts": int32(starts), "group_start": int32(group_start),
         "shared": int32(shared), "max_q": max(q_lens), "max_len": max(kv_lens), "max_shared": max(shared),
         "scales": (1 / 32, 1 / 32) if case["cache"] == "fp8" else (1.0, 1.0),
         # which sequence and group each token is of, and its position
         "seq": seq.to(dev), "of": torch.tensor(of, device=dev), "base": torch.tensor(base, device=dev),
         "pos": (torch.tensor(kv_lens)[seq] - torch.tensor(q_lens)[seq] + torch.arange(T) - starts[seq]).to(dev)}
    if own:
        import bit_weight_quantized_qgemm_amd as qg

        s["cache"] = qg.KVCache(s["k"], s["v"], *s["scales"])
    return s


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    s = _prepare_lora(case, gen, dev) if case["op"] == "lora" else _prepare_attend(case, gen, dev)
    s["case"] = case
    return s


# --------------------------------------------------------------------------------------- the passes
def run(state):
    if own:
        return _run_own(state)
    return _plain_lora(state) if state["case"]["op"] == "lora" else _plain_attend(state)


def _run_own(s):
    import bit_weight_quantized_qgemm_amd as qg

    c = s["case"]
    if c["op"] == "lora":
        return qg.lora(s["x"], s["adapters"], s["batch"], base=s["base"])
    if c["op"] == "decode":
        return qg.attn_decode_shared(s["q"], s["cache"], s["table"], s["lens"], s["max_len"], s["group_start"],
                                     s["shared"], s["max_shared"], window=c["window"], sinks=c["sinks"])
    return qg.attn_prefill_shared(s["q"], s["cache"], s["table"], s["starts"], s["lens"], s["max_q"], s["max_len"],
                                  s["group_start"], s["shared"], s["max_shared"], window=c["window"],
                                  sinks=c["sinks"])


def _plain_lora(s):
    """Every row with every adapter in two dense products, all but its own one masked in between."""
    a, b, ids = s["a"], s["b"], s["ids"].long()
    pool, S, R, K = a.shape
    T = ids.shape[0]
    y = torch.matmul(s["x"].float(), a.float().view(-1, K).t()).view(T, pool, S, R)
    mine = (ids[:, None] == torch.arange(pool, device=ids.device)) * s["scales"]
    keep = mine[:, :, None].expand(T, pool, R)
    if s["ranks"] is not None:
        keep = keep * (torch.arange(R, device=ids.device) < s["ranks"][:, None])
    y = y * keep[:, :, None]
    parts = [torch.matmul(y[:, :, i].reshape(T, pool * R), w.float().transpose(1, 2).reshape(pool * R, -1))
             for i, w in enumerate(b.split(s["widths"], dim=1))]
    return (s["base"].float() + torch.cat(parts, dim=1)).to(s["x"].dtype)


def _rows(buf, page, place, scale):
    """Cached heads by page and place in it, fp32."""
    if buf.dtype == torch.float8_e4m3fn:
        return buf.view(torch.uint8)[page, place].view(torch.float8_e4m3fn).float() * scale
    return buf[page, place].float()


def _partial(s, q, live, pos, token, there, table):
    """Attention of batches of rows over one run of tokens each, before the joint division.

    q fp32 [n][rows][H][D] at positions pos [n][rows], token and there [n][L], table [n][columns]; returns the
    rows' largest score, sum of weights and weighted sum of values, [n][rows][H](, D)."""
    c = s["case"]
    n, rows, H, D = q.shape
    KV, page = c["kv_heads"], c["page"]
    col = torch.div(token, page, rounding_mode="floor").clamp(max=table.shape[1] - 1)
    at = torch.gather(table.long(), 1, col).clamp(min=0)
    k, v = (_rows(s[x], at, token % page, f) for x, f in zip("kv", s["scales"]))    # [n][L][KV][D]
    L = token.shape[1]
    q = q.view(n, rows, KV, H // KV, D).permute(0, 2, 1, 3, 4).reshape(n * KV, rows * (H // KV), D)
    seen = there[:, None] & (token[:, None] <= pos[:, :, None]) & live[:, :, None]
    if c["window"]:
        seen &= (token[:, None] > pos[:, :, None] - c["window"]) | (token[:, None] < c["sinks"])
    seen = seen[:, None, :, None]                                             # [n][1][rows][1][L]
    k = k.permute(0, 2, 3, 1).reshape(n * KV, D, L).contiguous()
    score = torch.matmul(q, k).view(n, KV, rows, H // KV, L).mul_(1 / math.sqrt(D)).masked_fill_(~seen, float("-inf"))
    top = score.amax(dim=-1, keepdim=True)
    p = score.sub_(torch.where(top == float("-inf"), 0.0, top)).exp_()
    total = p.sum(dim=-1, keepdim=True)
    v = torch.where(there[:, :, None, None], v, 0.0).permute(0, 2, 1, 3).reshape(n * KV, L, D).contiguous()
    out = torch.matmul(p.view(n * KV, -1, L), v).view(n, KV, rows, H // KV, D)
    return [x.permute(0, 2, 1, 3, 4).reshape(n, rows, H, -1) for x in (top, total, out)]


def _plain_attend(s):
    """The shared tokens once for all rows of a group, each sequence's own ones for its rows, joined."""
    seq, pos, q = s["seq"], s["pos"], s["q"]
    dev = q.device
    of, base, lens = s["of"], s["base"], s["lens"].long()
    T, groups = seq.shape[0], s["shared"].shape[0]
    # rows of each group and of each sequence, padded to the longest
    token_group = of[seq]
    first_of = torch.searchsorted(torch.where(token_group < 0, groups, token_group).contiguous(),
                                  torch.arange(groups + 1, device=dev))
    most = int(s["case"]["q_len"] * -(-s["case"]["seqs"] // groups))
    slot = torch.arange(most, device=dev)
    row = first_of[:-1, None] + slot
    live = row < first_of[1:, None]
    row = row.clamp(max=T - 1)
    token = torch.arange(s["max_shared"], device=dev).expand(groups, -1)
    there = token < s["shared"][:, None]
    table = s["table"][s["group_start"][:-1].long()]
    shared = _partial(s, q[row].float(), live, pos[row], token, there, table)
    slot = torch.arange(s["max_q"], device=dev)
    starts = s["starts"].long()
    own_row = starts[:-1, None] + slot
    own_live = own_row < starts[1:, None]
    own_row = own_row.clamp(max=T - 1)
    token = base[:, None] + torch.arange(s["case"]["own_len"], device=dev)
    there = token < lens[:, None]
    mine = _partial(s, q[own_row].float(), own_live, pos[own_row], token, there, s["table"])
    H, D = q.shape[1:]
    top, total, out = (torch.zeros((T, H, x.shape[-1]), device=dev).index_put((own_row[own_live],), x[own_live])
                       for x in mine)
    # rows without a group keep nothing of the shared part
    top2 = torch.full((T, H, 1), float("-inf"), device=dev).index_put((row[live],), shared[0][live])
    total2, out2 = (torch.zeros((T, H, x.shape[-1]), device=dev).index_put((row[live],), x[live]) for x in shared[1:])
    m = torch.maximum(top, top2)
    m = torch.where(m == float("-inf"), 0.0, m)
    f, f2 = (top - m).exp(), (top2 - m).exp()
    total = total * f + total2 * f2
    return torch.where(total > 0, (out * f + out2 * f2) / total, 0.0).to(q.dtype)


# -------------------------------------------------------------------------------------- 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    return _exact_lora(case, s) if case["op"] == "lora" else _exact_attend(case, s)


def _exact_lora(case, s):
    out = s["base"].double()
    for i in s["ids"].unique().tolist():
        if i < 0:
            continue
        rows = (s["ids"] == i).nonzero()[:, 0]
        r = case["rank"] if s["ranks"] is None else int(s["ranks"][i])
        x, at = s["x"][rows].double(), 0
        for j, w in enumerate(s["widths"]):
            low = x @ s["a"][i, j, :r].double().t()
            out[rows, at:at + w] += float(s["scales"][i]) * (low @ s["b"][i, at:at + w, :r].double().t())
            at += w
    return out


def _exact_attend(case, s):
    q_lens, kv_lens, _ = _lengths(case)
    H, KV, D, page = case["heads"], case["kv_heads"], case["dim"], case["page"]
    dev = s["q"].device
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=dev)
    first = 0
    for b, (m, n) in enumerate(zip(q_lens, kv_lens)):
        ids = s["table"][b, :-(-n // page)].long()
        i, j = torch.arange(n - m, n, device=dev)[:, None], torch.arange(n, device=dev)[None]
        hide = j > i
        if case["window"]:
            hide = hide | ((j <= i - case["window"]) & (j >= case["sinks"]))
        # pages are picked as whole numbers of the same width: an index over 8-bit floats is not there everywhere
        kk, vv = (buf.view(torch.uint8 if buf.itemsize == 1 else torch.int16)[ids].flatten(0, 1)[:n].view(buf.dtype)
                  .double().transpose(0, 1).contiguous() * scale for buf, scale in zip((s["k"], s["v"]), s["scales"]))
        q = s["q"][first:first + m].double().view(m, KV, H // KV, D).permute(1, 2, 0, 3).reshape(KV, -1, D)
        for h in range(KV):
            z = (q[h] @ kk[h].t() / math.sqrt(D)).view(H // KV, m, n)
            w = torch.softmax(z.masked_fill(hide, float("-inf")), dim=-1)
            out[first:first + m, h * (H // KV):(h + 1) * (H // KV)] = (w @ vv[h]).transpose(0, 1)
        first += m
    return out

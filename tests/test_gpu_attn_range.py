"""GPU parity of the attention operators at the ends of what their arguments may be, against the fp64 oracle as in
tests/test_gpu_attn.py: masks beyond the context, weights far below the
largest, contexts of several groups of pages and parts, calls of more workgroups than one launch
holds."""

import numpy as np
import pytest
import torch

import bit_weight_quantized_qgemm_amd as qg
from oracle import attention as oa

from attn_problem import Paged, check, to_bits, to_torch
from test_gpu_attn import DECODE_WEIGHTS, DEV, PREFILL_WEIGHTS, _decode, _decode_refs, _prefill, _prefill_refs, _say, _values

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _automatic_splits():
    qg.set_attn_splits(0)
    yield
    qg.set_attn_splits(0)


@pytest.mark.parametrize("window,sinks", [(2 ** 63 - 1, 0), (2 ** 63 - 30, 2 ** 31 - 1), (1000, 5), (64, 2 ** 31 - 1),
                                          (1, 2 ** 31 - 15), (64, 1000)])
def test_masks_beyond_the_context(window, sinks):
    _say("masks beyond the context", window, sinks)
    rng = np.random.default_rng(40)
    H, KV, D, act, lens, new = 4, 1, 128, "f16", [1000, 77], [9, 40]
    pg = Paged(rng, lens, KV, D, act, 16, DEV)
    bits, q = _values(rng, (sum(new), H, D), act)
    qd = to_torch(bits, act, DEV)
    scale = np.float32(D ** -0.5).astype(np.float64)
    # every token is visible: the window covers all of them, or the sinks do
    dec, pre = _decode_refs(pg, q, scale), _prefill_refs(pg, q, new, scale)
    for splits in (0, 1, 3):
        qg.set_attn_splits(splits)
        one = _decode(pg, qd[:2], window=window, sinks=sinks)
        many = _prefill(pg, qd, new, window=window, sinks=sinks)
        torch.cuda.synchronize()
        check(oa.decode(to_bits(one), act), dec, act, DECODE_WEIGHTS[act], splits)
        check(oa.decode(to_bits(many), act), pre, act, PREFILL_WEIGHTS[act], splits)


# Weights far below a row's largest one. In fp16 (fp16 and e4m3 caches) they carry 2^11 and the largest may pass the
# reference by 2^4: a rounding moves a weight by half a last place, or, in the format's last bits, by 2^-25 / 2^11 of
# the reference's weight, and the weights sum to at least that.
WEIGHT_FLOOR = {"f16": 2.0 ** -36, "bf16": 0.0}


@pytest.mark.parametrize("act,cache", [("f16", "f16"), ("f16", "fp8"), ("bf16", "fp8"), ("bf16", "bf16")])
def test_a_first_token_far_above_the_rest(act, cache):
    _say("first token far above the rest", act, cache)
    rng = np.random.default_rng(41)
    n, D, gaps, page = 20000, 128, [10, 13, 16, 18, 20, 22], 16
    H, dtype = len(gaps), {"f16": torch.float16, "bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn}[cache]
    k = rng.standard_normal((n, 1, D))
    k[:, :, 0] = 0.0
    k[0, :, 0] = 1.0
    v = 1.0 + 0.5 * rng.standard_normal((n, 1, D))
    v[0] = 0.0   # only the others show
    kb, vb = oa.encode(k, cache), oa.encode(v, cache)
    k, v = oa.decode(kb, cache), oa.decode(vb, cache)
    q = 0.05 * rng.standard_normal((1, H, D))
    q[0, :, 0] = gaps
    bits = oa.encode(q, act)
    q = oa.decode(bits, act)[0]
    place = [to_torch(x.reshape(n // page, page, 1, D), cache, DEV) for x in (kb, vb)]
    assert place[0].dtype is dtype
    pg = qg.KVCache(*place)
    table = torch.arange(n // page, dtype=torch.int32, device=DEV)[None]
    lens, start = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([n], [0, 1]))
    qd = to_torch(bits, act, DEV)
    ks, vs = (np.repeat(x, H, axis=1) for x in (k, v))
    ref, mag, err = oa.attend(q, ks, vs, np.ones(n, dtype=bool), 1.0)
    s = np.einsum("hd,nhd->hn", q, ks)
    total = np.exp(s - s.max(axis=1, keepdims=True)).sum(axis=1)[:, None]
    kind = "f16" if cache == "fp8" else act
    floor = WEIGHT_FLOOR[kind] * (np.abs(vs).sum(axis=0) + n * np.abs(ref)) / total
    for splits in (1, 5, 0):
        qg.set_attn_splits(splits)
        one = qg.attn_decode(qd, pg, table, lens, n, scale=1.0)
        many = qg.attn_prefill(qd, pg, table, start, lens, 1, n, scale=1.0)
        torch.cuda.synchronize()
        for out, weights in ((one, DECODE_WEIGHTS[kind]), (many, PREFILL_WEIGHTS[kind])):
            got = oa.decode(to_bits(out), act)[0]
            bound = oa.attention_bound(ref, mag, err, n, act, weights) + floor
            off = (np.abs(got - ref) / bound).max(axis=1)
            print([f"{x:.3f}" for x in off], flush=True)
            assert np.all(off <= 1), (splits, off)


# A part of the prefill kernel looks its pages up for 64 blocks (1024 tokens) at a time: contexts of two and three such
# groups, windows that begin inside one, and pages lost on both sides of each change.
# heads, kv heads, dim, act, cache, page, layout, window, sinks
GROUPS = [
    (4, 2, 128, "f16", "f16", 16, "heads", 0, 0), (2, 1, 64, "bf16", "bf16", 16, "padded", 0, 0),
    (2, 1, 256, "f16", "f16", 32, "heads", 0, 0), (2, 2, 192, "bf16", "bf16", 16, "tokens", 0, 0),
    (2, 1, 96, "f16", "f16", 16, "heads", 0, 0), (4, 2, 128, "bf16", "fp8", 16, "tokens", 0, 0),
    (2, 1, 64, "f16", "fp8", 16, "heads", 0, 0), (2, 1, 256, "bf16", "fp8", 16, "heads", 0, 0),
    (4, 2, 128, "bf16", "bf16", 16, "heads", 1500, 37), (2, 1, 256, "f16", "f16", 16, "heads", 1111, 5),
    (2, 1, 128, "f16", "fp8", 16, "padded", 1300, 200),
]


@pytest.mark.parametrize("lost", [False, True], ids=["whole", "lost pages"])
@pytest.mark.parametrize("H,KV,D,act,cache,page,layout,window,sinks", GROUPS)
def test_contexts_of_several_page_groups(H, KV, D, act, cache, page, layout, window, sinks, lost):
    _say("page groups", H, KV, D, act, cache, page, layout, window, sinks, lost)
    rng = np.random.default_rng(42 + D)
    lens, new = [1100, 2300, 1024, 3200], [40, 5, 33, 2]
    at = [1024 // page - 1, 1024 // page]   # the pages before and after the change
    missing = [(0, at[0], 0), (1, at[0], -7), (1, at[1], 3), (1, 2 * at[1], 0), (3, 2 * at[1] - 1, -1), (3, 3 * at[1], 5)]
    pg = Paged(rng, lens, KV, D, cache, page, DEV, layout, (0.25, 0.125) if cache == "fp8" else (1.0, 1.0),
               missing=missing if lost else ())
    bits, q = _values(rng, (sum(new), H, D), act, 2.0)
    qd = to_torch(bits, act, DEV)
    scale = np.float32(D ** -0.5).astype(np.float64)
    kind = "f16" if cache == "fp8" else act
    refs = _prefill_refs(pg, q, new, scale, window, sinks)
    one = _decode_refs(pg, q, scale, window, sinks)
    for splits in (0, 1, 2):
        qg.set_attn_splits(splits)
        out = _prefill(pg, qd, new, window=window, sinks=sinks)
        last = _decode(pg, qd[:4], window=window, sinks=sinks)
        torch.cuda.synchronize()
        check(oa.decode(to_bits(out), act), refs, act, PREFILL_WEIGHTS[kind], ("prefill", splits))
        check(oa.decode(to_bits(last), act), one, act, DECODE_WEIGHTS[kind], ("decode", splits))


def _set_key(pg, b, j, head, x):
    """Token j of sequence b gets the key x (values) in one head."""
    bits = oa.encode(np.asarray(x) / pg.scales[0], pg.fmt)
    pg.k[int(pg.table[b, j // pg.page]), j % pg.page, head] = to_torch(bits, pg.fmt, DEV)
    pg.tokens[b][0][j, head] = oa.decode(bits, pg.fmt) * pg.scales[0]


# Joins read 16 parts at a time: parts in the second and third such batch, of which some sequences have none, and
# scores that pass all earlier ones there (or in the first part).
@pytest.mark.parametrize("peaks", [(4400, 2250, 650, 10), (3, 100, 680, 0)], ids=["late", "early"])
@pytest.mark.parametrize("H,KV,D,act,cache", [(4, 2, 128, "f16", "f16"), (3, 1, 256, "bf16", "bf16"),
                                              (2, 1, 64, "bf16", "bf16"), (4, 1, 80, "bf16", "fp8")])
def test_joins_of_many_parts(H, KV, D, act, cache, peaks):
    _say("many parts", H, KV, D, act, cache, peaks)
    rng = np.random.default_rng(43 + D)
    lens, new = [4500, 2300, 700, 20], [3, 9, 40, 2]
    pg = Paged(rng, lens, KV, D, cache, 16, DEV, "heads", (0.25, 0.125) if cache == "fp8" else (1.0, 1.0))
    bits, q = _values(rng, (sum(new), H, D), act)
    qd = to_torch(bits, act, DEV)
    scale = np.float32(D ** -0.5).astype(np.float64)
    kind = "f16" if cache == "fp8" else act
    ends = np.cumsum(new)
    for b, j in enumerate(peaks):
        # about 1.5 sqrt(D) nats for the last row's first head, and the same for the decoded row's
        _set_key(pg, b, j, 0, 1.5 * q[ends[b] - 1, 0])
        _set_key(pg, b, j + 1, KV - 1, 1.5 * q[b, H - 1])
    refs, one = _prefill_refs(pg, q, new, scale), _decode_refs(pg, q, scale)
    for splits in (17, 40, 1024):
        qg.set_attn_splits(splits)
        out, again = (_prefill(pg, qd, new) for _ in range(2))
        last, once_more = (_decode(pg, qd[:4]) for _ in range(2))
        torch.cuda.synchronize()
        assert torch.equal(out, again) and torch.equal(last, once_more)
        check(oa.decode(to_bits(out), act), refs, act, PREFILL_WEIGHTS[kind], ("prefill", splits))
        check(oa.decode(to_bits(last), act), one, act, DECODE_WEIGHTS[kind], ("decode", splits))


# -------------------------------------------------------------- more workgroups than one launch holds (2^24 and above)
def _pages(rng, pages, KV, D):
    kv = [to_torch(_values(rng, (pages, 16, KV, D), "f16")[0], "f16", DEV) for _ in range(2)]
    return qg.KVCache(*kv)


def test_prefill_of_many_row_tiles():
    _say("prefill of 2^24 row tiles")
    rng = np.random.default_rng(44)
    # 1024 sequences, 128 heads to one key-value head: up to 16384 new tokens are 16384 row tiles of each sequence
    B, H, D, most, pages = 1024, 128, 16, 16384, 1100
    cache = _pages(rng, pages, 1, D)
    lens = rng.integers(1, 60, B)
    long = 700
    lens[long] = most
    new = np.minimum(lens, rng.integers(1, 4, B))
    new[long] = most
    table = torch.from_numpy(rng.integers(0, pages, (B, most // 16)).astype(np.int32)).to(DEV)
    starts = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device=DEV)
    lens = torch.from_numpy(lens.astype(np.int32)).to(DEV)
    T, at = int(new.sum()), int(new[:long].sum())
    q = torch.randn((T, H, D), dtype=torch.float32, device=DEV).to(torch.float16)
    out = torch.full_like(q, float("nan"))
    qg.set_attn_splits(1)
    qg.attn_prefill(q, cache, table, starts, lens, most, most, out=out)
    # the same sequences in two calls of few row tiles: the long one, and the others
    alone = qg.attn_prefill(q[at:at + most], cache, table[long:long + 1], starts[:2] * 0 + torch.tensor(
        [0, most], dtype=torch.int32, device=DEV), lens[long:long + 1], most, most)
    rest = torch.full_like(q, float("nan"))
    qg.attn_prefill(q, cache, table, starts, lens, 3, most, out=rest)
    torch.cuda.synchronize()
    assert not bool(out.isnan().any())
    assert torch.equal(out[at:at + most], alone)
    rest[at:at + most] = alone
    assert torch.equal(out, rest)


def test_decode_of_many_tiles():
    _say("decode of 65535 x 256 tiles")
    rng = np.random.default_rng(45)
    B, H, D, pages = 65535, 256, 16, 40
    cache = _pages(rng, pages, H, D)
    table = torch.from_numpy(rng.integers(0, pages, (B, 2)).astype(np.int32)).to(DEV)
    lens = torch.from_numpy(rng.integers(0, 33, B).astype(np.int32)).to(DEV)
    q = torch.randn((B, H, D), dtype=torch.float32, device=DEV).to(torch.float16)
    out = qg.attn_decode(q, cache, table, lens, 32, out=torch.full_like(q, float("nan")))
    torch.cuda.synchronize()
    for a in range(0, B, 16384):   # calls of one launch each
        e = min(B, a + 16384)
        assert torch.equal(out[a:e], qg.attn_decode(q[a:e], cache, table[a:e], lens[a:e], 32)), a


def test_append_of_many_heads():
    _say("append of 2^20 x 1026 heads")
    T, H, D = 1 << 20, 342, 16
    gen = torch.Generator(device=DEV)
    gen.manual_seed(46)
    q = torch.empty((T, H, D), dtype=torch.float16, device=DEV).normal_(generator=gen)
    k, v = (torch.randn((1, H, D), generator=gen, device=DEV).to(torch.float16).expand(T, H, D) for _ in range(2))
    cache = qg.KVCache.empty(2, 16, H, D, torch.float16, DEV)
    table = torch.tensor([[-1], [1]], dtype=torch.int32, device=DEV)
    pos = torch.zeros(T, dtype=torch.int32, device=DEV)
    seq = torch.zeros(T, dtype=torch.int32, device=DEV)   # whose page is out of range: rotated, not stored
    kept = {0: 3, T // 2 + 1: 7, T - 1: 12}
    for t, p in kept.items():
        seq[t], pos[t] = 1, p
    pos[5] = -1
    out = torch.full_like(q, float("nan"))
    qg.qk_rope_append(q, k, v, pos, cache, table, token_seq=seq, out=out)
    torch.cuda.synchronize()
    q[5] = 0
    assert all(torch.equal(out[a:a + (T >> 4)], q[a:a + (T >> 4)]) for a in range(0, T, T >> 4))
    del q, out
    torch.cuda.empty_cache()
    for buf, new in ((cache.k, k), (cache.v, v)):
        assert not bool(buf[0].any())
        for p in range(16):
            assert torch.equal(buf[1, p], new[0] if p in kept.values() else torch.zeros_like(new[0])), p


def test_strides_along_one_token_or_head():
    _say("odd strides of single tokens and heads")
    rng = np.random.default_rng(47)
    D, act = 64, "f16"
    pg = Paged(rng, [37], 1, D, act, 16, DEV)
    bits, q = _values(rng, (1, 1, D), act)
    plain = to_torch(bits, act, DEV)
    odd = plain.as_strided((1, 1, D), (3, 1, 1))
    out = torch.zeros(D, dtype=torch.float16, device=DEV).as_strided((1, 1, D), (5, 7, 1))
    ref = _decode_refs(pg, q, np.float32(1 / 8).astype(np.float64))
    start = torch.tensor([0, 1], dtype=torch.int32, device=DEV)
    for got in (_decode(pg, odd), _decode(pg, odd, out=out),
                qg.attn_prefill(odd, pg.cache, pg.table_dev, start, pg.lens_dev, 1, 37)):
        torch.cuda.synchronize()
        check(oa.decode(to_bits(got), act), ref, act, PREFILL_WEIGHTS[act], "odd")
    pos = torch.tensor([20], dtype=torch.int32, device=DEV)
    got = qg.qk_rope_append(odd, odd, odd, pos, pg.cache, pg.table_dev, out=out)
    torch.cuda.synchronize()
    page, place = int(pg.table[0, 1]), 4
    assert torch.equal(got, plain) and torch.equal(pg.k[page, place], plain[0]) and torch.equal(pg.v[page, place], plain[0])


def test_a_cache_object_is_fixed():
    _say("fixed cache")
    cache = qg.KVCache.empty(2, 16, 1, 64, torch.float8_e4m3fn, DEV, 0.5, 0.25)
    for name, value in (("k_scale", 1.0), ("v_scale", 1.0), ("k", cache.v), ("v", cache.k), ("num_pages", 1)):
        with pytest.raises(AttributeError):
            setattr(cache, name, value)
    assert (cache.k_scale, cache.v_scale) == (0.5, 0.25)


@pytest.mark.parametrize("act,cache", [("f16", "f16"), ("f16", "fp8"), ("bf16", "bf16")])
def test_scores_that_fp32_hardly_tells_apart(act, cache):
    _say("scores of 2^24", act, cache)
    # about 2^24.7 in log2 units and within 20 of one another: which token wins is up to fp32, but every output is a
    # mean of the values
    rng = np.random.default_rng(48)
    n, H, D = 512, 4, 128
    k = np.full((n, 1, D), 96.0)
    k[:, 0, 0] = np.arange(n) * 9 // n   # scores that creep past the first ones
    v = rng.standard_normal((n, 1, D))
    q = np.full((1, H, D), 1024.0)
    q[0, :, 0] = [1, 1.5, -1, 0.75]
    kb, vb = oa.encode(k, cache), oa.encode(v, cache)
    v = oa.decode(vb, cache)[:, 0]
    place = [to_torch(x.reshape(n // 16, 16, 1, D), cache, DEV) for x in (kb, vb)]
    pg = qg.KVCache(*place)
    table = torch.arange(n // 16, dtype=torch.int32, device=DEV)[None]
    lens, start = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([n], [0, 1]))
    qd = to_torch(oa.encode(q, act), act, DEV)
    slop = 2 * oa.ROUNDOFF[act] * np.abs(v).max(axis=0)
    for splits in (1, 3):
        qg.set_attn_splits(splits)
        for out in (qg.attn_decode(qd, pg, table, lens, n, scale=1.5),
                    qg.attn_prefill(qd, pg, table, start, lens, 1, n, scale=1.5)):
            torch.cuda.synchronize()
            got = oa.decode(to_bits(out), act)[0]
            assert np.isfinite(got).all(), splits
            assert np.all(got <= v.max(axis=0) + slop) and np.all(got >= v.min(axis=0) - slop), splits

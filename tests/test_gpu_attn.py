"""GPU parity of the attention operators (qgemm_qk_rope_append, qgemm_attn_decode, qgemm_attn_prefill) against the
fp64 oracle, each output within the bound derived from the number formats (oracle/attention.py). Memory that holds no
token is NaN in every cache, and table entries past a sequence's end are out of range."""

import ctypes
import sys

import numpy as np
import pytest
import torch

import bit_weight_quantized_qgemm_amd as qg
from oracle import attention as oa

from attn_problem import NAN, Paged, check, to_bits, to_torch

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")

# rounding of the softmax weights: two 16-bit terms (the rest of the rounded weight, rounded again), or one
DECODE_WEIGHTS = {"f16": 2.0 ** -22, "bf16": 2.0 ** -16}
PREFILL_WEIGHTS = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8}


def _say(*a):
    print("[case]", *a, flush=True)
    sys.stdout.flush()


@pytest.fixture(autouse=True)
def _automatic_splits():
    qg.set_attn_splits(0)
    yield
    qg.set_attn_splits(0)


def _weights(table, act, cache):
    return table["f16" if cache == "fp8" else act]


def _values(rng, shape, fmt, scale=1.0):
    bits = oa.encode(rng.standard_normal(shape) * scale, fmt)
    return bits, oa.decode(bits, fmt)


# ------------------------------------------------------------------------------------------ append
APPEND = [
    # tokens, q heads, kv heads, dim, rot, act, cache, norm, interleaved, page, layout, fused
    (1, 32, 32, 128, 128, "f16", "f16", True, False, 16, "heads", True),
    (7, 8, 2, 64, 64, "bf16", "bf16", True, True, 16, "tokens", True),
    (33, 5, 1, 80, 32, "f16", "f16", False, True, 48, "padded", True),
    (20, 6, 3, 96, 96, "bf16", "fp8", True, False, 32, "heads", False),
    (19, 4, 2, 256, 128, "f16", "fp8", True, True, 16, "padded", True),
    (9, 3, 3, 16, 16, "f16", "f16", True, False, 16, "heads", False),
    (130, 4, 4, 112, 48, "bf16", "bf16", False, False, 64, "tokens", True),
    (5, 2, 1, 240, 0, "bf16", "bf16", True, False, 16, "heads", True),
    (6, 2, 2, 32, 16, "f16", "f16", False, False, 16, "heads", True),
]


def _append_problem(rng, T, H, KV, D, rot, act, cache, norm, page, layout, scales):
    n_seq = 3 if T > 3 else T
    seq = rng.integers(0, n_seq, T).astype(np.int32)
    lens = [0] * n_seq
    pos = np.zeros(T, dtype=np.int32)
    start = rng.integers(0, 2 * page, n_seq)
    for t in range(T):
        pos[t] = start[seq[t]] + lens[seq[t]]
        lens[seq[t]] += 1
    full = [int(s + n) for s, n in zip(start, lens)]
    pg = Paged(rng, full, KV, D, cache, page, DEV, layout, scales)
    qkv_bits, qkv = _values(rng, (T, (H + 2 * KV) * D), act, 3.0)
    wq, wk = (_values(rng, (D,), act) for _ in range(2)) if norm else ((None, None), (None, None))
    return pg, seq, pos, qkv_bits, qkv, wq, wk


def _split(x, T, H, KV, D):
    return (x[:, :H * D].reshape(T, H, D), x[:, H * D:(H + KV) * D].reshape(T, KV, D),
            x[:, (H + KV) * D:].reshape(T, KV, D))


def _check_append(got_q, pg, before, seq, pos, qkv, rope, H, KV, D, rot, act, wq, wk, eps, interleaved, stored=None):
    T = len(pos)
    q, k, v = _split(qkv, T, H, KV, D)
    expect = [x.copy() for x in before]
    written = [np.zeros(x.shape[:2], dtype=bool) for x in before]
    after = [to_bits(pg.k), to_bits(pg.v)]
    for t in range(T):
        row = rope[pos[t]].astype(np.float64) if rot else np.zeros(0)
        angles = (row[:rot // 2], row[rot // 2:])
        ref, err = oa.norm_rotate(q[t], wq, eps, angles, interleaved)
        assert np.all(np.abs(got_q[t] - ref) <= oa.rounding_bound(ref, err, act)), t
        if stored is not None and not stored[t]:
            continue
        page, place = pg.table[seq[t], pos[t] // pg.page], pos[t] % pg.page
        ref, err = oa.norm_rotate(k[t], wk, eps, angles, interleaved)
        ref, err = ref / pg.scales[0], err / pg.scales[0] + oa.FP32 * np.abs(ref / pg.scales[0])
        if pg.fmt == "fp8":
            ref = np.clip(ref, -oa.FP8_MAX, oa.FP8_MAX)
        got = oa.decode(after[0][page, place], pg.fmt)
        assert np.all(np.abs(got - ref) <= oa.rounding_bound(ref, err, pg.fmt)), t
        # values are copied (or rounded once; the scale is a power of two)
        expect[1][page, place] = oa.encode(v[t] / pg.scales[1], pg.fmt)
        written[0][page, place] = True
    assert np.array_equal(after[1], expect[1])
    assert np.array_equal(after[0][~written[0]], expect[0][~written[0]])   # nothing else was touched


@pytest.mark.parametrize("T,H,KV,D,rot,act,cache,norm,interleaved,page,layout,fused", APPEND)
def test_append(T, H, KV, D, rot, act, cache, norm, interleaved, page, layout, fused):
    _say("append", T, H, KV, D, rot, act, cache, norm, interleaved, page, layout, fused)
    rng = np.random.default_rng(T * 7 + D)
    scales = (2.0 ** -4, 2.0 ** -3) if cache == "fp8" else (1.0, 1.0)
    pg, seq, pos, bits, qkv, wq, wk = _append_problem(rng, T, H, KV, D, rot, act, cache, norm, page, layout, scales)
    before = [to_bits(pg.k), to_bits(pg.v)]
    rows = int(pos.max()) + 1
    table = qg.rope_table(rows, rot, device=DEV) if rot else None
    fused_dev = to_torch(bits, act, DEV)
    parts = [x.unflatten(-1, (-1, D)) for x in fused_dev.split([H * D, KV * D, KV * D], dim=-1)]
    if not fused:
        parts = [x.contiguous() for x in parts]
    eps = 1e-5
    out = qg.qk_rope_append(*parts, torch.from_numpy(pos).to(DEV), pg.cache, pg.table_dev, table,
                            q_norm=None if wq[0] is None else to_torch(wq[0], act, DEV),
                            k_norm=None if wk[0] is None else to_torch(wk[0], act, DEV), eps=eps,
                            token_seq=torch.from_numpy(seq).to(DEV), interleaved=interleaved)
    torch.cuda.synchronize()
    got = oa.decode(to_bits(out), act)
    rope = table.cpu().numpy() if rot else None
    _check_append(got, pg, before, seq, pos, qkv, rope, H, KV, D, rot, act, wq[1], wk[1], eps, interleaved)


def test_append_in_place_one_norm_and_default_sequences():
    _say("append in place")
    rng = np.random.default_rng(3)
    T, H, KV, D, rot, act = 4, 8, 2, 128, 64, "bf16"
    pg = Paged(rng, [40, 1, 17, 16], KV, D, act, 16, DEV)
    pos = np.array([39, 0, 16, 15], dtype=np.int32)
    bits, qkv = _values(rng, (T, (H + 2 * KV) * D), act)
    wk = _values(rng, (D,), act)
    before = [to_bits(pg.k), to_bits(pg.v)]
    fused = to_torch(bits, act, DEV)
    q, k, v = (x.unflatten(-1, (-1, D)) for x in fused.split([H * D, KV * D, KV * D], dim=-1))
    table = qg.rope_table(64, rot, device=DEV)
    out = qg.qk_rope_append(q, k, v, torch.from_numpy(pos).to(DEV), pg.cache, pg.table_dev, table,
                            k_norm=to_torch(wk[0], act, DEV), eps=1e-6, out=q)
    torch.cuda.synchronize()
    assert out.data_ptr() == fused.data_ptr()
    after = to_bits(fused)
    assert np.array_equal(after[:, H * D:], bits[:, H * D:])   # k and v of the product stay
    _check_append(oa.decode(to_bits(out), act), pg, before, np.arange(T), pos, qkv, table.cpu().numpy(), H, KV, D, rot,
                  act, None, wk[1], 1e-6, False)


def test_append_padding_and_places_out_of_range():
    _say("append padding")
    rng = np.random.default_rng(4)
    H, KV, D, act = 4, 2, 64, "f16"
    pg = Paged(rng, [16, 30, 5], KV, D, act, 16, DEV, missing=[(1, 1, 7)])
    #       stored, padding, past the rope table, page out of range, past the table, bad sequences, stored
    pos = np.array([3, -1, 48, 20, 40, 2, 2, 4], dtype=np.int32)
    seq = np.array([0, 0, 1, 1, 0, -1, 3, 2], dtype=np.int32)
    stored = [True, False, False, False, False, False, False, True]
    T = len(pos)
    bits, qkv = _values(rng, (T, (H + 2 * KV) * D), act)
    before = [to_bits(pg.k), to_bits(pg.v)]
    fused = to_torch(bits, act, DEV)
    q, k, v = (x.unflatten(-1, (-1, D)) for x in fused.split([H * D, KV * D, KV * D], dim=-1))
    table = qg.rope_table(48, D, device=DEV)
    out = qg.qk_rope_append(q, k, v, torch.from_numpy(pos).to(DEV), pg.cache, pg.table_dev, table,
                            token_seq=torch.from_numpy(seq).to(DEV))
    torch.cuda.synchronize()
    got = oa.decode(to_bits(out), act)
    assert not got[1].any() and not got[2].any()
    live = [t for t in range(T) if t not in (1, 2)]
    _check_append(got[live], pg, before, seq[live], pos[live], qkv[live], table.cpu().numpy(), H, KV, D, D, act, None,
                  None, 0.0, False, stored=[stored[t] for t in live])


def test_append_e4m3_saturates_and_keeps_nan():
    _say("append e4m3 range")
    D = 16
    pg = Paged(np.random.default_rng(5), [1], 1, D, "fp8", 16, DEV, scales=(0.5, 2.0))
    k = torch.tensor([[[1e4, -1e4, 224.0, 232.0, 240.0, float("nan"), float("inf"), -float("inf")] + [0.0] * 8]],
                     dtype=torch.float16, device=DEV)
    q = torch.ones((1, 1, D), dtype=torch.float16, device=DEV)
    qg.qk_rope_append(q, k, k, torch.zeros(1, dtype=torch.int32, device=DEV), pg.cache, pg.table_dev)
    torch.cuda.synchronize()
    page = pg.table[0, 0]
    for buf, scale in ((pg.k, 0.5), (pg.v, 2.0)):
        got = to_bits(buf)[page, 0, 0]
        want = oa.encode(k[0, 0].double().cpu().numpy() / scale, "fp8")
        assert got[5] & 0x7F == 0x7F
        assert np.array_equal(np.delete(got, 5), np.delete(want, 5))


def test_append_offsets_beyond_32_bits():
    _say("append far pages")
    KV, D, page, pages, step = 2, 64, 16, 450, 10 << 20
    k, v = (torch.zeros(pages * step, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    shape, stride = (pages, page, KV, D), (step, D, page * D, 1)
    cache = qg.KVCache(k.as_strided(shape, stride), v.as_strided(shape, stride))
    rng = np.random.default_rng(14)
    fused = to_torch(_values(rng, (3, 3 * KV, D), "bf16")[0], "bf16", DEV)
    table = torch.tensor([[449, 3, 420]], dtype=torch.int32, device=DEV)
    pos = torch.tensor([5, 20, 47], dtype=torch.int32, device=DEV)
    q = qg.qk_rope_append(fused[:, :KV], fused[:, KV:2 * KV], fused[:, 2 * KV:], pos, cache, table,
                          token_seq=torch.zeros(3, dtype=torch.int32, device=DEV))
    torch.cuda.synchronize()
    assert torch.equal(q, fused[:, :KV])
    for t, (pg, place) in enumerate([(449, 5), (3, 4), (420, 15)]):
        assert torch.equal(cache.k[pg, place], fused[t, KV:2 * KV])
        assert torch.equal(cache.v[pg, place], fused[t, 2 * KV:])


def test_append_without_tokens():
    _say("append of nothing")
    pg = Paged(np.random.default_rng(6), [3], 2, 64, "f16", 16, DEV)
    e = torch.empty((0, 2, 64), dtype=torch.float16, device=DEV)
    assert qg.qk_rope_append(e, e, e, torch.empty(0, dtype=torch.int32, device=DEV), pg.cache,
                             pg.table_dev).shape == (0, 2, 64)


# ------------------------------------------------------------------------------------------ decode
DECODE = [
    # lens, q heads, kv heads, dim, act, cache, page, layout, window, sinks
    ([1000], 4, 4, 128, "f16", "f16", 16, "heads", 0, 0),
    ([0, 1, 15, 16, 17, 31, 32, 33, 127, 128, 129, 500], 8, 1, 128, "bf16", "bf16", 16, "tokens", 0, 0),
    ([77, 300], 10, 2, 64, "bf16", "bf16", 48, "padded", 0, 0),
    ([77, 300, 0, 2], 6, 2, 256, "f16", "f16", 32, "heads", 0, 0),
    ([260, 31], 20, 1, 80, "f16", "f16", 16, "padded", 0, 0),
    ([100, 47], 33, 1, 16, "bf16", "bf16", 16, "heads", 0, 0),
    ([1, 200, 513], 7, 1, 128, "f16", "fp8", 64, "heads", 0, 0),
    ([1, 200, 513], 7, 7, 128, "bf16", "fp8", 16, "padded", 0, 0),
    ([90, 300], 4, 2, 64, "f16", "fp8", 16, "tokens", 0, 0),
    ([90, 300], 4, 2, 96, "bf16", "fp8", 16, "heads", 0, 0),
    ([90, 300], 4, 2, 208, "bf16", "fp8", 16, "heads", 0, 0),
    # windows: none seen beyond, whole, ending inside blocks, of one token; sinks that meet the window or overlap it
    ([0, 1, 5, 40, 47, 48, 49, 200, 333], 4, 2, 128, "bf16", "bf16", 16, "heads", 33, 4),
    ([3, 64, 65, 500], 4, 2, 128, "f16", "f16", 16, "heads", 1, 0),
    ([3, 64, 65, 500], 4, 2, 64, "f16", "f16", 16, "heads", 1, 1),
    ([20, 100, 640], 4, 2, 128, "f16", "f16", 32, "padded", 64, 16),
    ([20, 100, 640], 4, 2, 128, "f16", "fp8", 32, "heads", 50, 37),
    ([70, 640], 4, 2, 256, "bf16", "bf16", 16, "heads", 600, 50),
    ([70, 640], 4, 2, 128, "bf16", "bf16", 16, "heads", 100000, 3),
]


def _decode(pg, q, max_len=None, **kw):
    return qg.attn_decode(q, pg.cache, pg.table_dev, pg.lens_dev, max_len if max_len is not None else max(pg.lens), **kw)


def _decode_refs(pg, q, scale, window=0, sinks=0, lens=None):
    return [pg.attend(b, q[b], (lens or pg.lens)[b] - 1, scale, window, sinks) for b in range(len(pg.lens))]


@pytest.mark.parametrize("lens,H,KV,D,act,cache,page,layout,window,sinks", DECODE)
def test_decode(lens, H, KV, D, act, cache, page, layout, window, sinks):
    _say("decode", lens, H, KV, D, act, cache, page, layout, window, sinks)
    rng = np.random.default_rng(sum(lens) + D)
    pg = Paged(rng, lens, KV, D, cache, page, DEV, layout, (0.25, 0.125) if cache == "fp8" else (1.0, 1.0))
    bits, q = _values(rng, (len(lens), H, D), act, 2.0)
    qd = to_torch(bits, act, DEV)
    scale = 1 / np.sqrt(D)
    refs = _decode_refs(pg, q, np.float32(scale).astype(np.float64), window, sinks)
    for splits in (0, 1, 2, 7):
        qg.set_attn_splits(splits)
        out = _decode(pg, qd, scale=scale, window=window, sinks=sinks)
        again = _decode(pg, qd, scale=scale, window=window, sinks=sinks)
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), again.view(torch.int16))
        check(oa.decode(to_bits(out), act), refs, act, _weights(DECODE_WEIGHTS, act, cache), splits)


def test_decode_strided_rows_and_guards():
    _say("decode strided")
    rng = np.random.default_rng(8)
    H, KV, D = 6, 2, 64
    pg = Paged(rng, [50, 200, 7], KV, D, "f16", 16, DEV)
    bits, q = _values(rng, (3, H, D), "f16")
    big = torch.full((3, H + 1, D + 8), float("nan"), dtype=torch.float16, device=DEV)
    big[:, :H, :D] = to_torch(bits, "f16", DEV)
    out = torch.full((3, H + 1, D + 8), 7.0, dtype=torch.float16, device=DEV)
    for splits in (1, 4):
        qg.set_attn_splits(splits)
        _decode(pg, big[:, :H, :D], out=out[:, :H, :D])
        torch.cuda.synchronize()
        check(oa.decode(to_bits(out[:, :H, :D]), "f16"), _decode_refs(pg, q, np.float32(1 / 8.0)), "f16",
              DECODE_WEIGHTS["f16"], "strided")
        assert bool((out[:, H:] == 7.0).all()) and bool((out[:, :, D:] == 7.0).all())


def test_decode_large_scores_move_the_maximum():
    _say("decode large scores")
    rng = np.random.default_rng(9)
    H, KV, D = 4, 1, 128
    pg = Paged(rng, [700], KV, D, "bf16", 16, DEV)
    bits, q = _values(rng, (1, H, D), "bf16", 12.0)
    for splits in (1, 3):
        qg.set_attn_splits(splits)
        out = _decode(pg, to_torch(bits, "bf16", DEV), scale=0.25)
        torch.cuda.synchronize()
        check(oa.decode(to_bits(out), "bf16"), _decode_refs(pg, q, 0.25), "bf16", DECODE_WEIGHTS["bf16"], splits)


def test_decode_pages_out_of_range_are_masked():
    _say("decode missing pages")
    rng = np.random.default_rng(10)
    H, KV, D = 4, 2, 128
    pg = Paged(rng, [100, 40, 20], KV, D, "f16", 16, DEV, missing=[(0, 2, -5), (0, 6, 0), (1, 0, 3), (2, 0, -1), (2, 1, 9)])
    bits, q = _values(rng, (3, H, D), "f16")
    refs = _decode_refs(pg, q, np.float32(D ** -0.5))
    assert refs[2][3] == 0
    for splits in (1, 3):
        qg.set_attn_splits(splits)
        out = _decode(pg, to_torch(bits, "f16", DEV))
        torch.cuda.synchronize()
        check(oa.decode(to_bits(out), "f16"), refs, "f16", DECODE_WEIGHTS["f16"], splits)


def test_decode_lengths_are_bounded():
    _say("decode length bounds")
    rng = np.random.default_rng(11)
    H, KV, D = 2, 1, 64
    pg = Paged(rng, [64, 64, 64], KV, D, "f16", 16, DEV)
    bits, q = _values(rng, (3, H, D), "f16")
    lens = torch.tensor([-3, 1 << 30, 20], dtype=torch.int32, device=DEV)
    out = qg.attn_decode(to_torch(bits, "f16", DEV), pg.cache, pg.table_dev, lens, 50)
    torch.cuda.synchronize()
    check(oa.decode(to_bits(out), "f16"), _decode_refs(pg, q, np.float32(1 / 8), lens=[0, 50, 20]), "f16",
          DECODE_WEIGHTS["f16"], "bounds")


def test_decode_nan_in_a_visible_place_shows():
    _say("decode visible NaN")
    rng = np.random.default_rng(12)
    pg = Paged(rng, [40, 40], 1, 64, "f16", 16, DEV)
    pg.k[int(pg.table[0, 1]), 3] = float("nan")
    bits, _ = _values(rng, (2, 2, 64), "f16")
    for splits in (1, 2):
        qg.set_attn_splits(splits)
        out = _decode(pg, to_torch(bits, "f16", DEV))
        torch.cuda.synchronize()
        assert bool(out[0].isnan().all()) and not bool(out[1].isnan().any())


def test_decode_offsets_beyond_32_bits():
    _say("decode far pages")
    # pages 20 MiB apart: the last lies past 2^32 elements and bytes
    H, KV, D, page = 8, 1, 128, 16
    pages, step = 450, 10 << 20
    k, v = (torch.full((pages * step,), float("nan"), dtype=torch.float16, device=DEV) for _ in range(2))
    shape, stride = (pages, page, KV, D), (step, D, D, 1)
    k, v = k.as_strided(shape, stride), v.as_strided(shape, stride)
    rng = np.random.default_rng(13)
    n = 40
    kb, kx = _values(rng, (n, KV, D), "f16")
    vb, vx = _values(rng, (n, KV, D), "f16")
    table = np.array([[449, 3, 420]], dtype=np.int32)
    for j in range(n):
        k[int(table[0, j // page]), j % page] = to_torch(kb[j], "f16", DEV)
        v[int(table[0, j // page]), j % page] = to_torch(vb[j], "f16", DEV)
    bits, q = _values(rng, (1, H, D), "f16")
    cache = qg.KVCache(k, v)
    table_dev, lens = torch.from_numpy(table).to(DEV), torch.tensor([n], dtype=torch.int32, device=DEV)
    qd = to_torch(bits, "f16", DEV)
    out = qg.attn_decode(qd, cache, table_dev, lens, n)
    many = qg.attn_prefill(qd, cache, table_dev, torch.tensor([0, 1], dtype=torch.int32, device=DEV), lens, 1, n)
    torch.cuda.synchronize()
    ref = (*oa.attend(q[0], np.repeat(kx, H, axis=1), np.repeat(vx, H, axis=1), np.ones(n, dtype=bool),
                      np.float32(D ** -0.5).astype(np.float64)), n)
    check(oa.decode(to_bits(out), "f16"), [ref], "f16", DECODE_WEIGHTS["f16"], "far")
    check(oa.decode(to_bits(many), "f16"), [ref], "f16", PREFILL_WEIGHTS["f16"], "far")


# ----------------------------------------------------------------------------------------- prefill
PREFILL = [
    # new tokens, cached with them, q heads, kv heads, dim, act, cache, page, layout, window, sinks
    ([1], [1], 1, 1, 128, "f16", "f16", 16, "heads", 0, 0),
    ([130], [130], 4, 4, 128, "f16", "f16", 16, "heads", 0, 0),
    ([5, 0, 1, 33, 70], [200, 17, 64, 33, 71], 8, 1, 128, "bf16", "bf16", 16, "tokens", 0, 0),
    ([40, 77], [40, 90], 10, 2, 64, "bf16", "bf16", 48, "padded", 0, 0),
    ([40, 9], [300, 9], 6, 2, 256, "f16", "f16", 32, "heads", 0, 0),
    ([65, 20], [65, 260], 5, 1, 80, "f16", "f16", 16, "padded", 0, 0),
    ([11], [100], 33, 1, 16, "bf16", "bf16", 16, "heads", 0, 0),
    ([50, 3], [50, 129], 7, 1, 128, "f16", "fp8", 64, "heads", 0, 0),
    ([50, 3], [50, 129], 4, 4, 128, "bf16", "fp8", 16, "padded", 0, 0),
    ([50, 3], [64, 129], 4, 2, 64, "f16", "fp8", 16, "tokens", 0, 0),
    ([20, 3], [64, 129], 4, 2, 96, "bf16", "fp8", 16, "heads", 0, 0),
    ([20, 3], [64, 129], 4, 2, 192, "bf16", "fp8", 16, "heads", 0, 0),
    # more new tokens than cached ones: the first rows see nothing
    ([20, 5, 3], [12, 0, 3], 4, 2, 128, "f16", "f16", 16, "heads", 0, 0),
    # windows
    ([150, 9], [150, 333], 4, 2, 128, "bf16", "bf16", 16, "heads", 33, 4),
    ([70, 70], [70, 500], 4, 2, 128, "f16", "f16", 16, "heads", 1, 0),
    ([70, 70], [70, 500], 4, 2, 64, "f16", "f16", 16, "heads", 1, 1),
    ([100, 40], [100, 640], 4, 2, 128, "f16", "f16", 32, "padded", 64, 16),
    ([100, 40], [100, 640], 4, 2, 128, "f16", "fp8", 32, "heads", 50, 37),
    ([70], [640], 2, 1, 256, "bf16", "bf16", 16, "heads", 500, 50),
    ([70], [140], 2, 1, 128, "bf16", "bf16", 16, "heads", 100000, 3),
]


def _prefill(pg, q, new, max_q=None, **kw):
    start = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device=DEV)
    return qg.attn_prefill(q, pg.cache, pg.table_dev, start, pg.lens_dev, max_q if max_q is not None else max(new),
                           max(pg.lens), **kw)


def _prefill_refs(pg, q, new, scale, window=0, sinks=0):
    refs, row = [], 0
    for b, m in enumerate(new):
        for i in range(m):
            refs.append(pg.attend(b, q[row], pg.lens[b] - m + i, scale, window, sinks))
            row += 1
    return refs


@pytest.mark.parametrize("new,lens,H,KV,D,act,cache,page,layout,window,sinks", PREFILL)
def test_prefill(new, lens, H, KV, D, act, cache, page, layout, window, sinks):
    _say("prefill", new, lens, H, KV, D, act, cache, page, layout, window, sinks)
    rng = np.random.default_rng(sum(lens) + D)
    pg = Paged(rng, lens, KV, D, cache, page, DEV, layout, (0.25, 0.125) if cache == "fp8" else (1.0, 1.0))
    bits, q = _values(rng, (sum(new), H, D), act, 2.0)
    qd = to_torch(bits, act, DEV)
    scale = 1 / np.sqrt(D)
    refs = _prefill_refs(pg, q, new, np.float32(scale).astype(np.float64), window, sinks)
    for splits in (0, 1, 2, 7):
        qg.set_attn_splits(splits)
        out = _prefill(pg, qd, new, scale=scale, window=window, sinks=sinks)
        again = _prefill(pg, qd, new, scale=scale, window=window, sinks=sinks)
        torch.cuda.synchronize()
        assert torch.equal(out.view(torch.int16), again.view(torch.int16))
        check(oa.decode(to_bits(out), act), refs, act, _weights(PREFILL_WEIGHTS, act, cache), splits)


# head sizes on both sides of every limit at which the products widen
@pytest.mark.parametrize("D", [32, 80, 96, 112, 144, 160, 192, 208])
@pytest.mark.parametrize("act,cache", [("f16", "f16"), ("bf16", "bf16"), ("bf16", "fp8")])
def test_prefill_head_sizes(D, act, cache):
    test_prefill([45, 70], [45, 333], 6, 2, D, act, cache, 16, "padded" if D % 32 else "heads", 0, 0)
    test_prefill([70], [400], 3, 1, D, act, cache, 32, "tokens", 77, 5)


def test_prefill_strided_rows_bounds_and_guards():
    _say("prefill strided and bounded")
    rng = np.random.default_rng(21)
    H, KV, D, new = 6, 2, 64, [50, 20]
    pg = Paged(rng, [60, 20], KV, D, "f16", 16, DEV)
    bits, q = _values(rng, (sum(new), H, D), "f16")
    big = torch.full((sum(new), H + 1, D + 8), float("nan"), dtype=torch.float16, device=DEV)
    big[:, :H, :D] = to_torch(bits, "f16", DEV)
    refs = _prefill_refs(pg, q, new, np.float32(1 / 8.0))
    for splits in (1, 3):
        qg.set_attn_splits(splits)
        out = torch.full((sum(new), H + 1, D + 8), 7.0, dtype=torch.float16, device=DEV)
        _prefill(pg, big[:, :H, :D], new, out=out[:, :H, :D])
        torch.cuda.synchronize()
        check(oa.decode(to_bits(out[:, :H, :D]), "f16"), refs, "f16", PREFILL_WEIGHTS["f16"], "strided")
        assert bool((out[:, H:] == 7.0).all()) and bool((out[:, :, D:] == 7.0).all())
        # starts outside the rows of q: nothing beyond them is read or written
        out = torch.full((sum(new), H, D), 7.0, dtype=torch.float16, device=DEV)
        start = torch.tensor([60, 1 << 30, -4], dtype=torch.int32, device=DEV)
        qg.attn_prefill(big[:, :H, :D], pg.cache, pg.table_dev, start, pg.lens_dev, 70, 60, out=out)
        torch.cuda.synchronize()
        assert bool((out[:60] == 7.0).all()) and not bool((out[60:] == 7.0).all())


def test_prefill_large_scores_move_the_maximum():
    _say("prefill large scores")
    rng = np.random.default_rng(22)
    H, KV, D, new = 4, 1, 128, [70]
    pg = Paged(rng, [500], KV, D, "bf16", 16, DEV)
    bits, q = _values(rng, (70, H, D), "bf16", 12.0)
    refs = _prefill_refs(pg, q, new, 0.25)
    for splits in (1, 3):
        qg.set_attn_splits(splits)
        out = _prefill(pg, to_torch(bits, "bf16", DEV), new, scale=0.25)
        torch.cuda.synchronize()
        check(oa.decode(to_bits(out), "bf16"), refs, "bf16", PREFILL_WEIGHTS["bf16"], splits)


def test_prefill_pages_out_of_range_are_masked():
    _say("prefill missing pages")
    rng = np.random.default_rng(23)
    H, KV, D, new = 4, 2, 128, [30, 20]
    pg = Paged(rng, [100, 20], KV, D, "f16", 16, DEV, missing=[(0, 2, -5), (0, 6, 0), (1, 0, 3)])
    bits, q = _values(rng, (sum(new), H, D), "f16")
    refs = _prefill_refs(pg, q, new, np.float32(D ** -0.5))
    for splits in (1, 3):
        qg.set_attn_splits(splits)
        out = _prefill(pg, to_torch(bits, "f16", DEV), new)
        torch.cuda.synchronize()
        check(oa.decode(to_bits(out), "f16"), refs, "f16", PREFILL_WEIGHTS["f16"], splits)


# ------------------------------------------------------------------------- streams, graphs, steps
def test_decode_steps_on_a_side_stream_and_in_a_graph():
    _say("append + decode: side stream and graph")
    rng = np.random.default_rng(31)
    B, H, KV, D, act = 5, 8, 2, 128, "bf16"
    lens = [200, 1, 64, 333, 17]
    pg = Paged(rng, [n + 8 for n in lens], KV, D, act, 16, DEV)
    table = qg.rope_table(512, D, device=DEV)
    fused = to_torch(_values(rng, (B, (H + 2 * KV) * D), act)[0], act, DEV)
    cur = torch.tensor(lens, dtype=torch.int32, device=DEV)
    pos = cur - 1
    ws = qg.Workspace()

    def step(out):
        q, k, v = (x.unflatten(-1, (-1, D)) for x in fused.split([H * D, KV * D, KV * D], dim=-1))
        qo = qg.qk_rope_append(q, k, v, pos, pg.cache, pg.table_dev, table)
        return qg.attn_decode(qo, pg.cache, pg.table_dev, cur, 352, out=out, workspace=ws)

    qg.set_attn_splits(4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        first = step(None)
    side.synchronize()
    plain = step(None)
    torch.cuda.synchronize()
    assert torch.equal(first, plain)
    out = torch.empty_like(plain)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        step(out)
    for i in range(4):
        cur += 1
        pos += 1
        fused.copy_(to_torch(_values(rng, tuple(fused.shape), act)[0], act, DEV))
        out.zero_()
        g.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert torch.equal(got, step(None)), i
        torch.cuda.synchronize()


def test_prefill_then_decode_equals_one_prefill():
    _say("prefill in chunks, then tokens one by one")
    rng = np.random.default_rng(32)
    H, KV, D, act, n = 8, 2, 128, "f16", 150
    pg = Paged(rng, [n], KV, D, act, 16, DEV)
    bits, q = _values(rng, (n, H, D), act)
    qd = to_torch(bits, act, DEV)
    refs = _prefill_refs(pg, q, [n], np.float32(D ** -0.5))
    one = torch.tensor([0], dtype=torch.int32, device=DEV)
    done, rows = 0, []
    for m in (64, 37, 48):
        start = torch.tensor([0, m], dtype=torch.int32, device=DEV)
        rows.append(qg.attn_prefill(qd[done:done + m], pg.cache, pg.table_dev, start, one + done + m, m, n))
        done += m
    while done < n:
        rows.append(qg.attn_decode(qd[done:done + 1], pg.cache, pg.table_dev, one + done + 1, n))
        done += 1
    torch.cuda.synchronize()
    check(oa.decode(to_bits(torch.cat(rows)), act), refs, act, PREFILL_WEIGHTS[act], "chunks")


def test_calls_by_argument_equal_the_binding():
    _say("flat entry points")
    rng = np.random.default_rng(33)
    H, KV, D, act, lens, new = 8, 2, 64, "bf16", [70, 33], [5, 2]
    pg = Paged(rng, lens, KV, D, act, 16, DEV)
    L, scale = qg.lib(), 0.125
    T = sum(new)
    fused = to_torch(_values(rng, (T, H + 2 * KV, D), act)[0], act, DEV)
    q, k, v = fused[:, :H], fused[:, H:H + KV], fused[:, H + KV:]
    rope = qg.rope_table(80, D, device=DEV)
    pos = torch.tensor([lens[0] - 5 + i for i in range(5)] + [31, 32], dtype=torch.int32, device=DEV)
    seq = torch.tensor([0] * 5 + [1] * 2, dtype=torch.int32, device=DEV)
    start = torch.tensor([0, 5, 7], dtype=torch.int32, device=DEV)
    n = torch.tensor(lens, dtype=torch.int32, device=DEV)
    c, cols = pg.cache, pg.table_dev.shape[1]
    ref = ctypes.byref(c._struct)
    rotated = qg.qk_rope_append(q, k, v, pos, c, pg.table_dev, rope, token_seq=seq)
    stored = c.k.clone(), c.v.clone()
    out = torch.zeros_like(rotated)
    assert L.qgemm_qk_rope_append(q.data_ptr(), q.stride(0), D, k.data_ptr(), k.stride(0), D, v.data_ptr(),
                                  v.stride(0), D, None, None, 1e-6, rope.data_ptr(), 80, D, 0, pos.data_ptr(),
                                  seq.data_ptr(), pg.table_dev.data_ptr(), cols, 2, T, H, qg.DT_BF16, ref,
                                  out.data_ptr(), H * D, D, None) == 0
    torch.cuda.synchronize()
    assert torch.equal(out, rotated)
    for a, b in zip((c.k, c.v), stored):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    ws = torch.zeros(1 << 22, dtype=torch.uint8, device=DEV)
    for splits in (1, 3):
        qg.set_attn_splits(splits)
        got = torch.zeros_like(rotated)
        assert L.qgemm_attn_prefill(rotated.data_ptr(), H * D, D, ref, pg.table_dev.data_ptr(), cols, start.data_ptr(),
                                    n.data_ptr(), 2, T, 5, 80, H, qg.DT_BF16, scale, 0, 0, got.data_ptr(), H * D, D,
                                    ws.data_ptr(), ws.numel(), None) == 0
        torch.cuda.synchronize()
        assert torch.equal(got, qg.attn_prefill(rotated, c, pg.table_dev, start, n, 5, 80, scale=scale))
        got = torch.zeros_like(rotated[:2])
        assert L.qgemm_attn_decode(rotated.data_ptr(), H * D, D, ref, pg.table_dev.data_ptr(), cols, n.data_ptr(), 2,
                                   80, H, qg.DT_BF16, scale, 0, 0, got.data_ptr(), H * D, D, ws.data_ptr(), ws.numel(),
                                   None) == 0
        torch.cuda.synchronize()
        assert torch.equal(got, qg.attn_decode(rotated[:2], c, pg.table_dev, n, 80, scale=scale))

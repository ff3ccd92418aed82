"""Attention over tokens that sequences share (qgemm_attn_decode_shared, qgemm_attn_prefill_shared) against the fp64
oracle, each output within the bound derived from the number formats. Memory that holds no token is NaN, and table
entries past a sequence's end are out of range."""

import numpy as np
import pytest
import torch

import bit_weight_quantized_qgemm_amd as qg
from attn_problem import check, to_bits, to_torch
from oracle import attention as oa
from shared_problem import SharedPaged
from test_gpu_attn import DEV, PREFILL_WEIGHTS, _say, _values, _weights

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _modes():
    qg.set_attn_splits(0)
    qg.set_attn_sharing(1)
    yield
    qg.set_attn_splits(0)
    qg.set_attn_sharing(0)


def _decode(rng, pg, H, act, window=0, sinks=0, max_shared=None, max_len=None, what=""):
    B, D = len(pg.lens), pg.dim
    scale = D ** -0.5
    bits, q = _values(rng, (B, H, D), act)
    out = qg.attn_decode_shared(to_torch(bits, act, DEV), pg.cache, pg.table_dev, pg.lens_dev, max_len or max(pg.lens),
                                pg.group_start, pg.shared_lens, pg.max_shared if max_shared is None else max_shared,
                                window=window, sinks=sinks)
    torch.cuda.synchronize()
    refs = [pg.attend(b, q[b], n - 1, scale, window, sinks) for b, n in enumerate(pg.lens)]
    # the shared tokens' weights are rounded to one 16-bit term
    check(oa.decode(to_bits(out), act), refs, act, _weights(PREFILL_WEIGHTS, act, pg.fmt), what)
    return out


def _prefill(rng, pg, new, H, act, window=0, sinks=0, max_shared=None, what=""):
    D = pg.dim
    T = sum(new)
    bits, q = _values(rng, (T, H, D), act)
    start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
    out = qg.attn_prefill_shared(to_torch(bits, act, DEV), pg.cache, pg.table_dev, torch.from_numpy(start).to(DEV),
                                 pg.lens_dev, max(new), max(pg.lens), pg.group_start, pg.shared_lens,
                                 pg.max_shared if max_shared is None else max_shared, window=window, sinks=sinks)
    torch.cuda.synchronize()
    refs = [pg.attend(b, q[start[b] + i], n - m + i, D ** -0.5, window, sinks)
            for b, (m, n) in enumerate(zip(new, pg.lens)) for i in range(m)]
    check(oa.decode(to_bits(out), act), refs, act, _weights(PREFILL_WEIGHTS, act, pg.fmt), what)
    return out


# groups: (sequences, shared pages, shared tokens); lens of all sequences; before: sequences in front of the first group
DECODE = [
    # one group of short contexts; a shared run that ends inside a page, inside a block, and one of no whole block
    ([40, 33, 64, 50], [(4, 2, 32)], 0, 4, 4, 64, "f16", "f16", 16, "heads", 0, 0),
    ([100, 129, 96, 97, 200], [(5, 3, 96)], 0, 8, 2, 128, "bf16", "bf16", 32, "tokens", 0, 0),
    ([100, 129, 96, 97, 200], [(5, 3, 90)], 0, 8, 2, 128, "f16", "f16", 32, "heads", 0, 0),
    ([40, 41], [(2, 1, 15)], 0, 2, 1, 80, "f16", "f16", 16, "padded", 0, 0),
    # several groups, empty ones, sequences in none before and after
    ([70, 300, 310, 500, 20, 40, 41, 17, 260], [(2, 16, 256), (0, 3, 48), (1, 20, 320), (3, 1, 16), (0, 1, 16)], 1, 6, 2, 96,
     "bf16", "fp8", 16, "heads", 0, 0),
    # sequences shorter than what is said to be shared; of no tokens; all tokens shared
    ([100, 5, 0, 64, 63, 65, 1], [(7, 6, 96)], 0, 4, 2, 64, "f16", "f16", 16, "heads", 0, 0),
    ([128, 128, 128], [(3, 4, 128)], 0, 4, 1, 128, "bf16", "bf16", 32, "heads", 0, 0),
    # many rows: several tiles of 128
    ([300 + 7 * i % 90 for i in range(40)], [(40, 16, 256)], 0, 16, 2, 64, "f16", "f16", 16, "heads", 0, 0),
    ([150 + i for i in range(70)], [(30, 8, 128), (39, 4, 64)], 1, 40, 8, 128, "bf16", "bf16", 16, "heads", 0, 0),
    # groups of heads above one workgroup's 16
    ([90, 70, 80], [(3, 4, 64)], 0, 40, 2, 64, "f16", "f16", 16, "heads", 0, 0),
    ([90, 70, 80], [(3, 4, 64)], 0, 128, 1, 32, "bf16", "fp8", 16, "heads", 0, 0),
    # windows: over part of the shared run, past it, all of it; sinks inside it, past it
    ([200, 150, 170, 260], [(4, 8, 128)], 0, 4, 2, 64, "f16", "f16", 16, "heads", 100, 0),
    ([200, 150, 170, 260], [(4, 8, 128)], 0, 4, 2, 64, "bf16", "bf16", 16, "heads", 20, 3),
    ([200, 150, 170, 260], [(4, 8, 128)], 0, 4, 2, 128, "f16", "fp8", 16, "heads", 300, 5),
    ([200, 150, 170, 260], [(4, 8, 128)], 0, 4, 2, 64, "f16", "f16", 16, "heads", 10, 140),
    ([1000, 700, 400, 600], [(4, 20, 320)], 0, 4, 2, 64, "f16", "f16", 16, "heads", 333, 37),
    ([40, 500, 330, 100], [(4, 20, 320)], 0, 4, 4, 96, "bf16", "bf16", 16, "heads", 64, 17),
    # head sizes
    ([90, 70, 80], [(3, 4, 64)], 0, 4, 2, 16, "f16", "f16", 16, "heads", 0, 0),
    ([90, 70, 80], [(3, 4, 64)], 0, 4, 2, 192, "bf16", "bf16", 16, "heads", 0, 0),
    ([90, 70, 80], [(3, 4, 64)], 0, 4, 2, 256, "f16", "fp8", 16, "heads", 0, 0),
    ([90, 70, 80], [(3, 4, 64)], 0, 4, 2, 240, "f16", "f16", 16, "padded", 0, 0),
]


@pytest.mark.parametrize("splits", [0, 1, 3])
@pytest.mark.parametrize("lens,groups,before,H,KV,D,act,cache,page,layout,window,sinks", DECODE)
def test_decode(lens, groups, before, H, KV, D, act, cache, page, layout, window, sinks, splits):
    _say("decode", lens[:8], groups, before, H, KV, D, act, cache, page, layout, window, sinks, splits)
    rng = np.random.default_rng(len(lens) + D + window)
    scales = (2.0 ** -4, 2.0 ** -3) if cache == "fp8" else (1.0, 1.0)
    pg = SharedPaged(rng, lens, groups, KV, D, cache, page, DEV, layout, scales, before)
    qg.set_attn_splits(splits)
    _decode(rng, pg, H, act, window, sinks, what=(lens[:8], splits))


PREFILL = [
    ([3, 1, 5, 2], [40, 33, 64, 50], [(4, 2, 32)], 0, 4, 4, 64, "f16", "f16", 16, "heads", 0, 0),
    ([5, 5, 5], [200, 170, 140], [(3, 8, 128)], 0, 8, 1, 128, "bf16", "bf16", 16, "tokens", 0, 0),
    # new tokens that are themselves shared (whole prompts alike), partly and all
    ([70, 100, 20], [70, 100, 20], [(3, 4, 64)], 0, 4, 2, 64, "f16", "f16", 16, "heads", 0, 0),
    ([64, 60, 33], [64, 64, 64], [(3, 4, 64)], 0, 2, 2, 80, "bf16", "bf16", 16, "padded", 0, 0),
    # sequences without new tokens, groups of several tiles, sequences in no group
    ([0, 9, 0, 30, 1, 0, 44, 2], [100, 90, 80, 130, 66, 64, 110, 50], [(2, 2, 32), (5, 4, 64)], 0, 8, 2, 96, "f16", "fp8",
     16, "heads", 0, 0),
    ([50, 60, 70, 3, 200], [114, 100, 71, 3, 300], [(2, 2, 32), (2, 0, 0)], 1, 16, 2, 128, "bf16", "bf16", 16, "heads", 0, 0),
    # more new tokens than lengths: rows at negative positions
    ([5, 4], [3, 40], [(2, 2, 32)], 0, 2, 1, 64, "f16", "f16", 16, "heads", 0, 0),
    # windows and sinks
    ([20, 33, 8], [200, 150, 260], [(3, 8, 128)], 0, 4, 2, 64, "f16", "f16", 16, "heads", 100, 0),
    ([20, 33, 8], [200, 150, 260], [(3, 8, 128)], 0, 4, 2, 64, "bf16", "bf16", 16, "heads", 24, 3),
    ([20, 100, 8], [200, 150, 260], [(3, 8, 128)], 0, 4, 2, 128, "f16", "fp8", 32, "heads", 70, 20),
    ([2, 3], [700, 400], [(2, 20, 320)], 0, 4, 2, 64, "f16", "f16", 16, "heads", 333, 37),
    # many sequences of few tokens: a wave's rows are of many sequences
    ([i % 3 for i in range(150)], [40 + i % 9 for i in range(150)], [(149, 2, 32)], 1, 2, 2, 32, "f16", "f16", 16, "heads", 0, 0),
    # head sizes
    ([9, 4], [90, 70], [(2, 4, 64)], 0, 4, 2, 16, "f16", "f16", 16, "heads", 0, 0),
    ([9, 4], [90, 70], [(2, 4, 64)], 0, 4, 2, 192, "bf16", "bf16", 16, "heads", 0, 0),
    ([9, 4], [90, 70], [(2, 4, 64)], 0, 4, 2, 256, "f16", "fp8", 16, "heads", 0, 0),
]


@pytest.mark.parametrize("splits", [0, 1, 3])
@pytest.mark.parametrize("new,lens,groups,before,H,KV,D,act,cache,page,layout,window,sinks", PREFILL)
def test_prefill(new, lens, groups, before, H, KV, D, act, cache, page, layout, window, sinks, splits):
    _say("prefill", new[:8], lens[:8], groups, before, H, KV, D, act, cache, page, layout, window, sinks, splits)
    rng = np.random.default_rng(len(lens) + D + window)
    scales = (2.0 ** -4, 2.0 ** -3) if cache == "fp8" else (1.0, 1.0)
    pg = SharedPaged(rng, lens, groups, KV, D, cache, page, DEV, layout, scales, before)
    qg.set_attn_splits(splits)
    _prefill(rng, pg, new, H, act, window, sinks, what=(lens[:8], splits))


def test_many_groups():
    _say("many groups")
    rng = np.random.default_rng(5)
    # more than 64 groups
    lens = [20 + i % 7 for i in range(200)]
    pg = SharedPaged(rng, lens, [(i % 4, 1, 16) for i in range(120)], 1, 32, "f16", 16, DEV, before=5)
    _decode(rng, pg, 2, "f16")
    new = [1 + i % 3 for i in range(200)]
    _prefill(rng, pg, new, 2, "f16")


def test_thousands_of_groups():
    """More groups than one look at 64 x 64 of them finds, and more than one run of lanes holds."""
    _say("thousands of groups")
    rng = np.random.default_rng(20)
    n = 4500
    pg = SharedPaged(rng, [17 + i % 3 for i in range(2 * n)], [(2, 1, 16)] * n, 1, 16, "f16", 16, DEV)
    _decode(rng, pg, 1, "f16")
    _prefill(rng, pg, [1] * (2 * n), 1, "f16")


LONG = [
    # shared and own runs of more pages than a wave holds the places of; lost pages in both
    ([2400, 3700, 2110, 2200], [(3, 132, 2112)], 4, 2, 128, "f16", "f16", 16, [(0, 70, -1), (1, 70, -1), (2, 70, -1), (1, 200, -1)]),
    ([2400, 3700, 2110, 2200], [(3, 132, 2112)], 4, 2, 64, "bf16", "fp8", 16, []),
    ([2400, 3700, 1500, 2200], [(3, 33, 2112)], 2, 1, 96, "bf16", "bf16", 64, [(3, 20, 5)]),
    ([1300, 1700, 1110], [(3, 66, 1056)], 2, 1, 256, "f16", "f16", 16, [(0, 40, -1), (1, 40, -1), (2, 40, -1)]),
]


@pytest.mark.parametrize("splits", [0, 1, 2])
@pytest.mark.parametrize("lens,groups,H,KV,D,act,cache,page,missing", LONG)
def test_long_runs(lens, groups, H, KV, D, act, cache, page, missing, splits):
    _say("long", lens, groups, H, KV, D, act, cache, page, missing, splits)
    rng = np.random.default_rng(D)
    scales = (2.0 ** -4, 2.0 ** -3) if cache == "fp8" else (1.0, 1.0)
    pg = SharedPaged(rng, lens, groups, KV, D, cache, page, DEV, scales=scales, missing=missing)
    qg.set_attn_splits(splits)
    for window, sinks in ((0, 0), (1500, 5)):
        _decode(rng, pg, H, act, window, sinks, what=(lens, splits))
        _prefill(rng, pg, [3, 40, 7, 1][:len(lens)], H, act, window, sinks, what=(lens, splits))


@pytest.mark.parametrize("sharing", [0, 1])
@pytest.mark.parametrize("splits", [0, 2])
def test_one_long_prompt_among_single_tokens(splits, sharing):
    """Most of the tiles that max_q allows hold no row."""
    _say("long prompt among single tokens", splits, sharing)
    rng = np.random.default_rng(53)
    qg.set_attn_splits(splits)
    qg.set_attn_sharing(sharing)
    new = [1, 0, 1, 150, 1, 1, 2, 1, 1]
    lens = [260 + 3 * i for i in range(9)]
    lens[3] = 430
    pg = SharedPaged(rng, lens, [(5, 16, 256), (2, 8, 128)], 2, 64, "f16", 16, DEV, before=1)
    _prefill(rng, pg, new, 8, "f16")


def test_rows_of_q_before_the_first_sequence():
    _say("offset rows")
    rng = np.random.default_rng(21)
    pg = SharedPaged(rng, [90, 80, 70], [(3, 4, 64)], 2, 64, "f16", 16, DEV)
    bits, q = _values(rng, (12, 4, 64), "f16")
    start = torch.tensor([3, 5, 5, 9], dtype=torch.int32, device=DEV)
    out = torch.full((12, 4, 64), 7.0, dtype=torch.float16, device=DEV)
    for splits in (1, 3):
        qg.set_attn_splits(splits)
        out.fill_(7.0)
        qg.attn_prefill_shared(to_torch(bits, "f16", DEV), pg.cache, pg.table_dev, start, pg.lens_dev, 4, 90, pg.group_start,
                               pg.shared_lens, 64, out=out)
        torch.cuda.synchronize()
        rows = [(0, 3, 88), (0, 4, 89)] + [(2, 5 + i, 66 + i) for i in range(4)]
        refs = [pg.attend(b, q[t], pos, 0.125) for b, t, pos in rows]
        check(oa.decode(to_bits(out), "f16")[[t for _, t, _ in rows]], refs, "f16", PREFILL_WEIGHTS["f16"], "offset")
        assert bool((out[:3] == 7.0).all()) and bool((out[9:] == 7.0).all())


def test_calls_on_two_streams_at_once():
    _say("two streams")
    rng = np.random.default_rng(22)
    pg = SharedPaged(rng, [700, 650, 660, 800], [(4, 32, 512)], 2, 128, "f16", 16, DEV)
    qs = [to_torch(_values(rng, (4, 8, 128), "f16")[0], "f16", DEV) for _ in range(2)]

    def call(q):
        return qg.attn_decode_shared(q, pg.cache, pg.table_dev, pg.lens_dev, 800, pg.group_start, pg.shared_lens, 512)

    want = [call(q) for q in qs]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], [[], []]
    for _ in range(20):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(call(qs[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(g, want[i]) for g in got[i])


@pytest.mark.parametrize("max_shared", [0, 15, 16, 40, 64, 1000])
def test_max_shared_bounds_what_is_shared(max_shared):
    _say("max_shared", max_shared)
    rng = np.random.default_rng(6)
    pg = SharedPaged(rng, [100, 90, 64], [(3, 4, 64)], 2, 64, "f16", 16, DEV)
    _decode(rng, pg, 4, "f16", max_shared=max_shared, max_len=100)
    _prefill(rng, pg, [4, 3, 2], 4, "f16", max_shared=max_shared)


def test_automatic_choices_agree():
    """Whatever the automatic rule takes, forced sharing and none give the same within the bounds."""
    rng = np.random.default_rng(7)
    for lens, groups in (([700] * 12, [(12, 32, 512)]), ([700, 90], [(1, 4, 64), (1, 2, 32)]), ([50] * 4, [])):
        for mode in (0, 1, 2):
            qg.set_attn_sharing(mode)
            pg = SharedPaged(rng, lens, groups, 4, 128, "bf16", 16, DEV)
            _decode(rng, pg, 8, "bf16", what=(groups, mode))
            _prefill(rng, pg, [2] * len(lens), 8, "bf16", what=(groups, mode))


def test_large_scores_move_the_maximum_between_the_parts():
    """The largest score among the own tokens, or among the shared ones, far above the others."""
    for at in (3, 100, 130, 180):
        _say("peak at", at)
        rng = np.random.default_rng(at)
        pg = SharedPaged(rng, [190, 185, 181], [(3, 8, 128)], 1, 64, "f16", 16, DEV)
        q = rng.standard_normal((3, 2, 64))
        q_bits = oa.encode(q, "f16")
        q = oa.decode(q_bits, "f16")
        # the key of token `at` is 12 times the first query
        peak = oa.encode(12 * q[0, 0], "f16")
        page, place = pg.table[0, at // 16], at % 16
        pg.k[page.item(), place, 0] = to_torch(peak, "f16", DEV)
        for b in range(3):
            if pg.table[b, at // 16] == page:
                pg.tokens[b][0][at, 0] = oa.decode(peak, "f16")
        for splits in (1, 4):
            qg.set_attn_splits(splits)
            out = qg.attn_decode_shared(to_torch(q_bits, "f16", DEV), pg.cache, pg.table_dev, pg.lens_dev, 190, pg.group_start,
                                        pg.shared_lens, 128)
            refs = [pg.attend(b, q[b], n - 1, 0.125) for b, n in enumerate(pg.lens)]
            check(oa.decode(to_bits(out), "f16"), refs, "f16", PREFILL_WEIGHTS["f16"], at)


def test_pages_out_of_range_are_masked():
    _say("lost pages")
    rng = np.random.default_rng(8)
    lost = [(b, col, entry) for b in range(3) for col, entry in ((1, -7), (5, 0))] + [(1, 9, 1000), (2, 8, -1)]
    pg = SharedPaged(rng, [190, 165, 150], [(3, 8, 128)], 2, 64, "f16", 16, DEV, missing=lost)
    for splits in (1, 3):
        qg.set_attn_splits(splits)
        _decode(rng, pg, 4, "f16", what="lost")
        _prefill(rng, pg, [3, 2, 5], 4, "f16", what="lost")
    # nothing at all is left
    pg = SharedPaged(rng, [64, 60], [(2, 4, 64)], 2, 64, "f16", 16, DEV, missing=[(b, c, -1) for b in range(2) for c in range(4)])
    out = qg.attn_decode_shared(to_torch(_values(rng, (2, 4, 64), "f16")[0], "f16", DEV), pg.cache, pg.table_dev, pg.lens_dev, 64,
                                pg.group_start, pg.shared_lens, 64)
    assert not to_bits(out).any()


def test_strided_rows_and_guards():
    _say("strides")
    rng = np.random.default_rng(9)
    pg = SharedPaged(rng, [100, 90, 70, 30], [(3, 4, 64)], 2, 64, "bf16", 16, DEV, layout="padded")
    H, D, new = 4, 64, [3, 0, 2, 4]
    T = 11   # two rows of no sequence
    start = torch.tensor([0, 3, 3, 5, 9], dtype=torch.int32, device=DEV)
    for prefill in (False, True):
        n = T if prefill else 4
        big = torch.zeros((n + 2, H, D + 16), dtype=torch.bfloat16, device=DEV)
        q = big[1:n + 1, :, 8:8 + D]
        bits, val = _values(rng, (n, H, D), "bf16")
        q.copy_(to_torch(bits, "bf16", DEV))
        hold = torch.full((n + 2, H, D + 8), 7.0, dtype=torch.bfloat16, device=DEV)
        out = hold[1:n + 1, :, :D]
        if prefill:
            got = qg.attn_prefill_shared(q, pg.cache, pg.table_dev, start, pg.lens_dev, 4, 100, pg.group_start, pg.shared_lens, 64,
                                         out=out)
            rows = [(b, int(start[b]) + i, pg.lens[b] - m + i) for b, m in enumerate(new) for i in range(m)]
        else:
            got = qg.attn_decode_shared(q, pg.cache, pg.table_dev, pg.lens_dev, 100, pg.group_start, pg.shared_lens, 64, out=out)
            rows = [(b, b, pg.lens[b] - 1) for b in range(4)]
        assert got is out
        torch.cuda.synchronize()
        refs = [pg.attend(b, val[t], pos, D ** -0.5) for b, t, pos in rows]
        values = oa.decode(to_bits(out), "bf16")
        check(values[[t for _, t, _ in rows]], refs, "bf16", PREFILL_WEIGHTS["bf16"], prefill)
        hold[1:n + 1, :, :D][:len(rows)] = 7.0
        assert bool((hold == 7.0).all())   # rows of no sequence, the space between


def test_rows_past_max_q_and_lengths_past_max_len():
    _say("bounds")
    rng = np.random.default_rng(10)
    pg = SharedPaged(rng, [100, 90], [(2, 4, 64)], 1, 64, "f16", 16, DEV)
    bits, q = _values(rng, (10, 2, 64), "f16")
    start = torch.tensor([0, 6, 10], dtype=torch.int32, device=DEV)
    out = torch.full((10, 2, 64), 7.0, dtype=torch.float16, device=DEV)
    # sequence 0 has 6 rows, of which 4 are computed, as the last 4 of at most 95 tokens
    qg.attn_prefill_shared(to_torch(bits, "f16", DEV), pg.cache, pg.table_dev, start, pg.lens_dev, 4, 95, pg.group_start,
                           pg.shared_lens, 64, out=out)
    torch.cuda.synchronize()
    assert bool((out[4:6] == 7.0).all())
    rows = [(0, i, 95 - 4 + i) for i in range(4)] + [(1, 6 + i, 86 + i) for i in range(4)]
    refs = [pg.attend(b, q[t], pos, 0.125) for b, t, pos in rows]
    check(oa.decode(to_bits(out), "f16")[[t for _, t, _ in rows]], refs, "f16", PREFILL_WEIGHTS["f16"], "bounds")


def test_groups_out_of_order_or_range_stay_in_bounds():
    """Entries of group_start that fall, or lie outside the batch, give some outputs and touch nothing else."""
    _say("bad groups")
    rng = np.random.default_rng(11)
    pg = SharedPaged(rng, [100, 90, 70, 30, 64], [(4, 1, 16)], 2, 64, "f16", 16, DEV)
    bits, _ = _values(rng, (9, 4, 64), "f16")
    q = to_torch(bits, "f16", DEV)
    start = torch.tensor([0, 3, 4, 5, 9, 9], dtype=torch.int32, device=DEV)
    for bad in ([3, 1, 4, 0], [-5, 2, 100, 1], [5, 5, 5, 5], [2 ** 31 - 1, -2 ** 31, 3, 2], [0, 4, 2, 5]):
        groups = torch.tensor(bad, dtype=torch.int32, device=DEV)
        for shared in ([16, 16, 16], [-1, 2 ** 31 - 1, -2 ** 31]):
            lens = torch.tensor(shared, dtype=torch.int32, device=DEV)
            for splits in (1, 2):
                qg.set_attn_splits(splits)
                hold = torch.full((11, 4, 64), 7.0, dtype=torch.float16, device=DEV)
                qg.attn_decode_shared(q[:5], pg.cache, pg.table_dev, pg.lens_dev, 100, groups, lens, 16, out=hold[1:6])
                qg.attn_prefill_shared(q, pg.cache, pg.table_dev, start, pg.lens_dev, 4, 100, groups, lens, 16, out=hold[1:10])
                torch.cuda.synchronize()
                assert bool((hold[0] == 7.0).all()) and bool((hold[10] == 7.0).all())


def test_repeats_streams_and_graphs():
    """The same bits on every call, on another stream, and in replays of a graph whose inputs change; the workspace serves
    other calls in between."""
    _say("repeats, streams, graphs")
    rng = np.random.default_rng(12)
    lens = [700, 650, 660, 800, 90]
    pg = SharedPaged(rng, lens, [(4, 32, 512)], 2, 128, "f16", 16, DEV)
    new = [2, 1, 3, 1, 4]
    start = torch.tensor(np.concatenate([[0], np.cumsum(new)]), dtype=torch.int32, device=DEV)
    q = to_torch(_values(rng, (11, 8, 128), "f16")[0], "f16", DEV)
    for splits in (0, 5):
        qg.set_attn_splits(splits)

        def calls(ws, outs=(None, None)):
            return (qg.attn_decode_shared(q[:5], pg.cache, pg.table_dev, pg.lens_dev, 800, pg.group_start, pg.shared_lens, 512,
                                          workspace=ws, out=outs[0]),
                    qg.attn_prefill_shared(q, pg.cache, pg.table_dev, start, pg.lens_dev, 4, 800, pg.group_start,
                                           pg.shared_lens, 512, workspace=ws, out=outs[1]),
                    qg.attn_decode(q[:5], pg.cache, pg.table_dev, pg.lens_dev, 800, workspace=ws))

        ws = qg.Workspace()
        first = calls(ws)
        for _ in range(3):
            assert all(torch.equal(a, b) for a, b in zip(calls(ws), first))
        torch.cuda.synchronize()
        side = torch.cuda.Stream()
        with torch.cuda.stream(side):
            other = calls(ws)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(other, first))
        outs = (torch.zeros_like(q[:5]), torch.zeros_like(q))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            calls(ws, outs)
        for i in range(3):
            q.copy_(to_torch(_values(rng, (11, 8, 128), "f16")[0], "f16", DEV))
            pg.shared_lens.fill_([512, 300, 0][i])
            want = calls(qg.Workspace())[:2]
            for o in outs:
                o.fill_(float("nan"))
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(outs, want)), (splits, i)
        pg.shared_lens.fill_(512)


def test_offsets_beyond_32_bits():
    """Shared and own pages at both ends of a cache of more than 2^32 elements."""
    _say("far pages")
    rng = np.random.default_rng(13)
    page, KV, D = 16, 1, 64
    pages = (1 << 32) // (page * D) + 8
    k, v = (torch.zeros((pages, page, KV, D), dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn) for _ in range(2))
    cache = qg.KVCache(k, v)
    where = [pages - 1, 0, pages - 3, 5, pages - 2, 7]
    tables = [[where[0], where[1], where[2], where[3]], [where[0], where[1], where[4], where[5]]]
    lens = [60, 64]
    got = {}
    for p in where:
        pair = []
        for t in (k, v):
            bits = oa.encode(rng.standard_normal((page, KV, D)), "fp8")
            t[p].view(torch.uint8).copy_(torch.from_numpy(bits).to(DEV))
            pair.append(oa.decode(bits, "fp8"))
        got[p] = pair
    bits, q = _values(rng, (2, 2, D), "f16")
    out = qg.attn_decode_shared(to_torch(bits, "f16", DEV), cache, torch.tensor(tables, dtype=torch.int32, device=DEV),
                                torch.tensor(lens, dtype=torch.int32, device=DEV), 64,
                                torch.tensor([0, 2], dtype=torch.int32, device=DEV),
                                torch.tensor([32], dtype=torch.int32, device=DEV), 32)
    refs = []
    for b in range(2):
        kk, vv = (np.concatenate([got[p][i] for p in tables[b]]) for i in range(2))
        see = np.arange(64) < lens[b]
        refs.append((*oa.attend(q[b], np.repeat(kk, 2, axis=1), np.repeat(vv, 2, axis=1), see, D ** -0.5), lens[b]))
    check(oa.decode(to_bits(out), "f16"), refs, "f16", PREFILL_WEIGHTS["f16"], "far")


def test_refusals():
    rng = np.random.default_rng(14)
    pg = SharedPaged(rng, [40, 40], [(2, 1, 16)], 1, 64, "f16", 16, DEV)
    q = torch.zeros((2, 2, 64), dtype=torch.float16, device=DEV)

    def call(group_start=pg.group_start, shared_lens=pg.shared_lens, max_shared=16, **kw):
        return qg.attn_decode_shared(q, pg.cache, pg.table_dev, pg.lens_dev, 40, group_start, shared_lens, max_shared, **kw)

    call()
    for bad in (dict(group_start=pg.group_start[:1]), dict(group_start=pg.group_start.long()), dict(group_start=pg.group_start.cpu()),
                dict(shared_lens=pg.shared_lens.float()), dict(shared_lens=pg.shared_lens[:, None])):
        with pytest.raises(ValueError):
            call(**bad)
    with pytest.raises(qg.QgemmError, match="SHAPE"):
        call(max_shared=-1)
    with pytest.raises(ValueError):
        call(max_shared=1 << 70)
    with pytest.raises(qg.QgemmError, match="ALIAS"):
        call(out=q)

"""Attention over tokens that sequences share: the accuracy of single tokens, which is the plain call's, and joins of more
rows than a launch has workgroups for at a time."""

import numpy as np
import pytest
import torch

import bit_weight_quantized_qgemm_amd as qg
from attn_problem import check, to_bits, to_torch
from oracle import attention as oa
from shared_problem import SharedPaged
from test_gpu_attn import DECODE_WEIGHTS, DEV, PREFILL_WEIGHTS, _say, _values, _weights
from test_gpu_attn_shared import DECODE

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _modes():
    qg.set_attn_splits(0)
    qg.set_attn_sharing(1)
    yield
    qg.set_attn_splits(0)
    qg.set_attn_sharing(0)


@pytest.mark.parametrize("splits", [0, 2])
@pytest.mark.parametrize("lens,groups,before,H,KV,D,act,cache,page,layout,window,sinks", DECODE)
def test_decode_weights_have_two_terms(lens, groups, before, H, KV, D, act, cache, page, layout, window, sinks, splits):
    """The bound of attn_decode, whose weights enter the second product as two 16-bit terms, holds for shared tokens too."""
    _say("decode weights", lens[:8], groups, before, H, KV, D, act, cache, page, layout, window, sinks, splits)
    rng = np.random.default_rng(len(lens) + D + window + 1000)
    scales = (2.0 ** -4, 2.0 ** -3) if cache == "fp8" else (1.0, 1.0)
    pg = SharedPaged(rng, lens, groups, KV, D, cache, page, DEV, layout, scales, before)
    qg.set_attn_splits(splits)
    bits, q = _values(rng, (len(lens), H, D), act)
    out = qg.attn_decode_shared(to_torch(bits, act, DEV), pg.cache, pg.table_dev, pg.lens_dev, max(lens), pg.group_start,
                                pg.shared_lens, pg.max_shared, window=window, sinks=sinks)
    refs = [pg.attend(b, q[b], n - 1, D ** -0.5, window, sinks) for b, n in enumerate(lens)]
    check(oa.decode(to_bits(out), act), refs, act, _weights(DECODE_WEIGHTS, act, pg.fmt), (lens[:8], splits))


@pytest.mark.parametrize("D,act,cache", [(80, "f16", "f16"), (128, "bf16", "fp8")])
def test_joins_of_many_full_tiles(D, act, cache):
    """From 1024 tiles of rows on a join's workgroups take several turns."""
    _say("joins", D, act, cache)
    rng = np.random.default_rng(D)
    B, KV, new = 16, 32, 140   # 140 rows of a head: a full tile of 128 and one of 12
    lens = [200 + 3 * i for i in range(B)]
    pg = SharedPaged(rng, lens, [(B, 3, 48)], KV, D, cache, 16, DEV, scales=(2.0 ** -4, 2.0 ** -3) if cache == "fp8" else (1.0, 1.0))
    T = B * new
    bits, q = _values(rng, (T, KV, D), act)
    start = torch.arange(0, T + 1, new, dtype=torch.int32, device=DEV)
    out = qg.attn_prefill_shared(to_torch(bits, act, DEV), pg.cache, pg.table_dev, start, pg.lens_dev, new, max(lens),
                                 pg.group_start, pg.shared_lens, pg.max_shared)
    torch.cuda.synchronize()
    refs = [pg.attend(t // new, q[t], lens[t // new] - new + t % new, D ** -0.5) for t in range(T)]
    check(oa.decode(to_bits(out), act), refs, act, _weights(PREFILL_WEIGHTS, act, pg.fmt), D)


@pytest.mark.parametrize("lowered", [None, 0, 600])
@pytest.mark.parametrize("act,cache,D,window,sinks", [("f16", "f16", 64, 0, 0), ("bf16", "fp8", 128, 0, 0), ("bf16", "bf16", 96, 500, 20),
                                                      ("f16", "f16", 256, 0, 0)])
def test_own_tokens_beyond_the_longest_context_less_the_shared_run(act, cache, D, window, sinks, lowered):
    """Sequences of no group, and of one whose shared run is shorter than max_shared, have more own tokens than the plan
    counts on, and more parts than the others."""
    _say("long own runs", act, cache, D, window, sinks, lowered)
    rng = np.random.default_rng(D + window)
    scales = (2.0 ** -4, 2.0 ** -3) if cache == "fp8" else (1.0, 1.0)
    lens = [1200, 1100, 1095, 1110, 1089, 1101, 700, 0, 1199, 300]
    pg = SharedPaged(rng, lens, [(5, 68, 1088), (2, 20, 320)], 2, D, cache, 16, DEV, scales=scales, before=1)
    if lowered is not None:
        pg.shared_lens[0] = lowered
    bits, q = _values(rng, (len(lens), 8, D), act)
    out = qg.attn_decode_shared(to_torch(bits, act, DEV), pg.cache, pg.table_dev, pg.lens_dev, 1200, pg.group_start,
                                pg.shared_lens, 1088, window=window, sinks=sinks)
    refs = [pg.attend(b, q[b], n - 1, D ** -0.5, window, sinks) for b, n in enumerate(lens)]
    check(oa.decode(to_bits(out), act), refs, act, _weights(DECODE_WEIGHTS, act, pg.fmt), (act, cache, D, lowered))


@pytest.mark.parametrize("act,cache,D,window,sinks", [("f16", "f16", 64, 0, 0), ("bf16", "fp8", 128, 0, 0), ("bf16", "bf16", 96, 500, 20),
                                                      ("f16", "f16", 256, 0, 0)])
def test_several_tokens_with_own_runs_beyond_the_plan(act, cache, D, window, sinks):
    """As above for several new tokens, a sequence of none and one of more than a tile of rows among them."""
    _say("long own runs, several tokens", act, cache, D, window, sinks)
    rng = np.random.default_rng(D + window + 1)
    scales = (2.0 ** -4, 2.0 ** -3) if cache == "fp8" else (1.0, 1.0)
    lens = [1200, 1100, 1095, 1110, 1089, 1101, 700, 5, 1199, 300]
    new = [3, 5, 2, 40, 1, 5, 5, 5, 2, 0]
    pg = SharedPaged(rng, lens, [(5, 68, 1088), (2, 20, 320)], 2, D, cache, 16, DEV, scales=scales, before=1)
    T, start = sum(new), np.concatenate([[0], np.cumsum(new)])
    bits, q = _values(rng, (T, 8, D), act)
    out = qg.attn_prefill_shared(to_torch(bits, act, DEV), pg.cache, pg.table_dev,
                                 torch.tensor(start, dtype=torch.int32, device=DEV), pg.lens_dev, 40, 1200, pg.group_start,
                                 pg.shared_lens, 1088, window=window, sinks=sinks)
    refs = [pg.attend(b, q[start[b] + i], n - m + i, D ** -0.5, window, sinks) for b, (m, n) in enumerate(zip(new, lens))
            for i in range(m)]
    check(oa.decode(to_bits(out), act), refs, act, _weights(PREFILL_WEIGHTS, act, pg.fmt), (act, cache, D))

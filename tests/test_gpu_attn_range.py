"""GPU parity of the attention operators at the ends of what their arguments may be, against the fp64 oracle as in
tests/test_gpu_attn.py: masks beyond the context, weights far below the largest."""

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

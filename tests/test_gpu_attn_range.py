"""GPU parity of the attention operators at the ends of what their arguments may be, against the fp64 oracle as in
tests/test_gpu_attn.py: masks beyond the context."""

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

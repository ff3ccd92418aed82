"""examples/serving_layer.py at small sizes: requests with adapters of their own behind one prompt, all together against
each alone.

Both ways round the same values to 16 bits at the same places: products, the sums with the adapters' products, rotated
queries and keys, attention outputs. They differ in the softmax weights (one 16-bit term or two, and another order of
sums), which moves an attention output by about its own rounding, and with it what is computed from it: a few times
2^-11 of the output. An e4m3 cache holds the same codes in both ways."""

import os
import sys

import pytest
import torch

import bit_weight_quantized_qgemm_amd as qg

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(autouse=True)
def _modes():
    yield
    qg.set_attn_sharing(0)


@pytest.mark.parametrize("sharing", [0, 1, 2], ids=["automatic", "shared", "unshared"])
@pytest.mark.parametrize("kw", [dict(), dict(cache="fp8", page=32), dict(heads=4, kv_heads=4, rank=40, adapters=1)],
                         ids=["f16", "fp8", "unshared heads"])
def test_requests_together_match_each_alone(kw, sharing):
    print("[case]", kw, sharing, flush=True)
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import serving_layer
    finally:
        sys.path.pop(0)
    qg.set_attn_sharing(sharing)
    args = dict(requests=5, prompt=150, question=9, steps=4, hidden=512, heads=8, kv_heads=2, dim=64, adapters=3)
    args.update(kw)
    diff, _, _ = serving_layer.run(**args)
    assert diff < 8 * 2.0 ** -11

"""examples/attention_layer.py at small sizes: tokens decoded one by one against the same tokens as one chunk.

Both ways round the same values to 16 bits at the same places except the softmax weights (one rounding to fp16 in the
chunk), the attention's output before the output product and that product's result: a few times 2^-11 of the output.
An e4m3 cache holds the same codes in both ways."""

import os
import sys

import pytest

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("kw", [dict(), dict(cache="fp8", page=32), dict(window=40, sinks=3), dict(heads=4, kv_heads=4)],
                         ids=["f16", "fp8", "window", "unshared heads"])
def test_decoded_tokens_match_a_prefilled_chunk(kw):
    print("[case]", kw, flush=True)
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import attention_layer
    finally:
        sys.path.pop(0)
    args = dict(batch=3, prompt=100, steps=9, hidden=512, heads=8, kv_heads=2, dim=64)
    args.update(kw)
    diff, _, _ = attention_layer.run(**args)
    assert diff < 8 * 2.0 ** -11

"""The low-rank adapters at the ends of their number formats: infinite second matrices. References are sums of products
in 64 bits, in which infinities and NaN go their own way."""

import numpy as np
import pytest
import torch

import bit_weight_quantized_qgemm_amd as qg
from attn_problem import to_bits, to_torch
from lora_problem import values
from oracle import attention as oa
from test_gpu_lora import DEV, _batch, _say

pytestmark = pytest.mark.gpu


def _formula(x, a, b, ids, scales):
    """base-less sums as the formula gives them (one slice); an infinity times zero is NaN."""
    out = np.zeros((x.shape[0], b.shape[1]))
    with np.errstate(all="ignore"):
        for t, i in enumerate(ids):
            y = (a[i, 0] * x[t]).sum(axis=1)
            out[t] = scales[i] * (b[i] * y).sum(axis=1)
    return out


@pytest.mark.parametrize("T", [5, 1100, 2600])
@pytest.mark.parametrize("rank", [8, 16, 24, 72, 256])
@pytest.mark.parametrize("fmt", ["f16", "bf16"])
def test_infinite_second_matrices(T, rank, fmt):
    """An infinite value of B gives an infinity of the product's sign, whatever the 16-bit terms of A x are: rests of
    either sign or zero (one-bit inputs), values far below their row's largest; NaN where A x is zero, where infinities of
    both signs meet, and where B has a NaN. Columns without one keep their bits."""
    _say("infinite B", T, rank, fmt)
    rng = np.random.default_rng(rank + T)
    n, K, N = 3, 16, 72
    x_bits, x = values(rng, (T, K), fmt)
    x_bits[1::7] = oa.encode(np.sign(x[1::7]), fmt)      # exact sums: no rest
    x_bits[2::11] = 0                                    # A x is zero
    x = oa.decode(x_bits, fmt)
    small, large = (2.0 ** -14, 2.0 ** 14) if fmt == "f16" else (2.0 ** -60, 2.0 ** 64)
    a = rng.choice([-1.0, -0.5, 0.5, 1.0], (n, 1, rank, K))
    a[:, :, 3::5] *= small                               # ranks far below the others
    a[:, :, ::5] *= large
    a_bits = oa.encode(a, fmt)
    a = oa.decode(a_bits, fmt)
    b_bits, plain = values(rng, (n, N, rank), fmt)
    inf, nan = {"f16": (0x7C00, 0x7E00), "bf16": (0x7F80, 0x7FC0)}[fmt]
    wild = b_bits.copy()
    for c, (r, sign) in enumerate([(0, 0), (3, 0), (rank - 1, 1), (1, 1), (3, 1), (2, 0), (4, 0)]):
        wild[:, 8 * c + 3, r] = inf | sign << 15
    wild[:, 60, 1], wild[:, 60, 4] = inf, inf            # two in a sum, of one sign or of both
    wild[:, 62, 2] = nan
    ids = np.arange(T) % n
    scales = np.array([1.0, -0.75, 2.0 ** -6], dtype=np.float32)
    pools = [qg.LoraAdapters(to_torch(a_bits, fmt, DEV), to_torch(w, fmt, DEV), scales=torch.from_numpy(scales).to(DEV))
             for w in (wild, b_bits)]
    xd, batch = to_torch(x_bits, fmt, DEV), _batch(ids, n)
    got, tame = (to_bits(qg.lora(xd, p, batch)) for p in pools)
    ref = _formula(x, a, oa.decode(wild, fmt), ids, scales)
    odd = (oa.decode(wild, fmt) - plain != 0).any(axis=2)[ids]   # NaN - x is not 0
    value = oa.decode(got, fmt)
    assert np.array_equal(np.isnan(value[odd]), np.isnan(ref[odd]))
    seen = odd & ~np.isnan(ref)
    assert np.isinf(ref[seen]).all() and np.array_equal(value[seen], ref[seen])
    assert np.array_equal(got[~odd], tame[~odd])

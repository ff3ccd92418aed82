"""The low-rank adapters at the ends of their number formats: infinite second matrices, products of very large and very
small values. References are sums of products in 64 bits, in which infinities and NaN go their own way."""

import numpy as np
import pytest
import torch

import bit_weight_quantized_qgemm_amd as qg
from attn_problem import to_bits, to_torch
from lora_problem import check, values
from oracle import attention as oa
from oracle import lora as lora_oracle
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


@pytest.mark.parametrize("T", [7, 1100, 2570])
@pytest.mark.parametrize("rank", [8, 16, 24, 72])
@pytest.mark.parametrize("fmt,x_dev,a_dev,b", [("bf16", 1.0, 1e-3, 2e38), ("bf16", 1.0, 1e-9, 2e38), ("bf16", 1e18, 1e18, 1e-36),
                                               ("bf16", 1e-18, 1e-18, 1e37), ("f16", 1.0, 1e-4, 4e4), ("f16", 1e3, 1e3, 1e-4)],
                         ids=str)
def test_values_at_the_ends_of_the_types(T, rank, fmt, x_dev, a_dev, b):
    """A x and B near the ends of their type, with results of ordinary size or at least finite."""
    _say("ends", T, rank, fmt, x_dev, a_dev, b)
    rng = np.random.default_rng(rank + T)
    n, K, N = 2, 40, 72
    x_bits, x = values(rng, (T, K), fmt, x_dev)
    a_bits, a = values(rng, (n, 1, rank, K), fmt, a_dev * K ** -0.5)
    b_bits = oa.encode(b * rng.choice([-1.5, -1.0, 1.0, 1.5], (n, N, rank)) * (1.0 + 0.05 * rng.random((n, N, rank))), fmt)
    ids = np.arange(T) % n
    out = qg.lora(to_torch(x_bits, fmt, DEV), qg.LoraAdapters(to_torch(a_bits, fmt, DEV), to_torch(b_bits, fmt, DEV)),
                  _batch(ids, n))
    ref, bound = lora_oracle.lora(x, a, oa.decode(b_bits, fmt), ids, fmt)
    assert np.abs(ref).max() < (60000 if fmt == "f16" else 1e38)
    check(out, ref, bound, fmt, (T, rank, fmt, b))


@pytest.mark.parametrize("T", [7, 1100, 2570])
@pytest.mark.parametrize("rank", [8, 24, 256])
def test_products_past_the_end_are_infinite(T, rank):
    """Finite values of one sign whose product with B passes bf16's end, with rests of either sign."""
    _say("past the end", T, rank)
    rng = np.random.default_rng(rank + T)
    n, K, N = 2, 24, 72
    x_bits, x = values(rng, (T, K), "bf16", 1e16)
    x_bits = oa.encode(np.abs(x) + 1e15, "bf16")
    a_bits = oa.encode(1e10 * (1 + rng.random((n, 1, rank, K))), "bf16")
    sign = rng.choice([-1.0, 1.0], (n, N, 1))
    b_bits = oa.encode(sign * 1e38 * (1 + rng.random((n, N, rank))), "bf16")
    ids = np.arange(T) % n
    out = qg.lora(to_torch(x_bits, "bf16", DEV), qg.LoraAdapters(to_torch(a_bits, "bf16", DEV), to_torch(b_bits, "bf16", DEV)),
                  _batch(ids, n))
    assert np.array_equal(oa.decode(to_bits(out), "bf16"), (sign[ids, :, 0] * np.inf))


@pytest.mark.parametrize("T", [7, 1100, 2570])
@pytest.mark.parametrize("rank", [8, 16, 24, 72])
def test_sums_near_the_end_of_fp32(T, rank):
    """A x of 1e36 to 1e38, a few powers of two below what fp32 holds, beside ranks of ordinary size; columns of B
    that are 0 stay 0."""
    _say("sums near the end", T, rank)
    rng = np.random.default_rng(rank + T)
    n, K, N = 2, 40, 72
    x_bits, x = values(rng, (T, K), "bf16", 5e18)
    a_bits, a = values(rng, (n, 1, rank, K), "bf16", 5e18 * K ** -0.5)
    small = oa.encode(a * np.where(np.arange(rank) % 4 == 1, 2.0 ** -120, 1.0)[:, None], "bf16")   # ranks 1, 5, ..
    small[:, :, 2::4] = oa.encode(a[:, :, 2::4] * 2.0 ** -24, "bf16")
    a = oa.decode(small, "bf16")
    b_bits, b = values(rng, (n, N, rank), "bf16", 1e-37)
    b_bits[:, ::8] = 0
    b = oa.decode(b_bits, "bf16")
    ids = np.arange(T) % n
    scales = torch.tensor([1.0, -300.0], device=DEV)
    out = qg.lora(to_torch(x_bits, "bf16", DEV), qg.LoraAdapters(to_torch(small, "bf16", DEV), to_torch(b_bits, "bf16", DEV),
                                                                scales=scales), _batch(ids, n))
    y = np.einsum("trk,tk->tr", a[ids, 0], x)
    assert 2.0 ** 124 < np.abs(y).max() < 3e38
    ref, bound = lora_oracle.lora(x, a, b, ids, "bf16", scales=scales.cpu().numpy())
    check(out, ref, bound, "bf16", (T, rank))
    assert not (to_bits(out)[:, ::8] & 0x7FFF).any()

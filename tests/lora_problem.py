"""Problems for the tests of the low-rank adapters: NumPy inputs as bit patterns, device tensors, oracle outputs."""

import numpy as np
import torch

import bit_weight_quantized_qgemm_amd as qg
from attn_problem import NAN, to_bits, to_torch
from oracle import attention as oa
from oracle import lora as ol


def values(rng, shape, fmt, dev_of=1.0):
    bits = oa.encode(rng.standard_normal(shape) * dev_of, fmt)
    return bits, oa.decode(bits, fmt)


class Pool:
    """Adapters of one projection; ranks that do not count, and the space between adapters, hold NaN."""

    def __init__(self, rng, n, K, widths, rank, fmt, dev, ranks=None, scaled=True, gap=0, a_dev=None, b_dev=None):
        S, N = len(widths), sum(widths)
        self.K, self.N, self.widths, self.rank, self.fmt, self.n = K, N, widths, rank, fmt, n
        a_bits, self.a = values(rng, (n, S, rank, K), fmt, K ** -0.5 if a_dev is None else a_dev)
        b_bits, self.b = values(rng, (n, N, rank), fmt, 0.5 * rank ** -0.5 if b_dev is None else b_dev)
        if ranks is not None:
            for i, r in enumerate(ranks):
                r = min(rank, (max(0, r) + 7) // 8 * 8)
                a_bits[i, :, r:] = NAN[fmt]
                b_bits[i, :, r:] = NAN[fmt]
        self.ranks = ranks
        self.scales = (0.5 + rng.random(n)).astype(np.float32) * np.where(np.arange(n) % 3 == 1, -1, 1).astype(np.float32) \
            if scaled else None
        dev_t = []
        for bits in (a_bits, b_bits):
            flat = np.full((n, bits[0].size + gap), NAN[fmt], dtype=np.uint16)
            flat[:, :bits[0].size] = bits.reshape(n, -1)
            dev_t.append(to_torch(flat, fmt, dev)[:, :bits[0].size].unflatten(1, bits.shape[1:]))
        self.adapters = qg.LoraAdapters(
            *dev_t, scales=None if self.scales is None else torch.from_numpy(self.scales).to(dev),
            ranks=None if ranks is None else torch.tensor(ranks, dtype=torch.int32, device=dev), widths=widths)

    def expected(self, x, ids, base=None):
        return ol.lora(x, self.a, self.b, ids, self.fmt, self.scales, self.ranks, self.widths, base)


def guarded(rows, cols, fmt, dev, gap=0, bits=None, fill=0x1234):
    """A [rows][cols] tensor of row stride cols + gap inside a larger buffer full of a pattern; (view, buffer)."""
    stride = cols + gap
    buf = np.full((rows + 2) * stride, fill, dtype=np.uint16)
    if bits is not None:
        buf[stride:stride + rows * stride].reshape(rows, stride)[:, :cols] = bits
    dev_buf = to_torch(buf, fmt, dev)
    return dev_buf[stride:stride + rows * stride].view(rows, stride)[:, :cols], dev_buf


def untouched(buf, rows, cols, gap=0, fill=0x1234):
    """Everything of a guarded buffer but its rows still holds the pattern."""
    bits, stride = to_bits(buf), cols + gap
    inner = bits[stride:stride + rows * stride].reshape(rows, stride)
    return (bits[:stride] == fill).all() and (bits[stride + rows * stride:] == fill).all() and (inner[:, cols:] == fill).all()


def check(out, ref, bound, fmt, what):
    got = oa.decode(to_bits(out), fmt)
    off = np.abs(got - ref)
    assert np.all(off <= bound), (what, int((~(off <= bound)).sum()), float(np.nanmax(off / bound)))

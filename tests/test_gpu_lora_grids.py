"""The low-rank adapters where the work is divided in other ways than small products reach: several runs of columns to a
wave, more tiles than the workspace has counters, more columns than one workgroup per tile of them allows, and both sides of
the row counts from which tiles are tall. Rows that are compared are the oracle's; all others must have been written."""

import numpy as np
import pytest
import torch

import bit_weight_quantized_qgemm_amd as qg
from attn_problem import NAN, to_torch
from lora_problem import Pool, check, guarded, untouched, values
from oracle import lora as lora_oracle
from test_gpu_lora import DEV, _batch, _say

pytestmark = pytest.mark.gpu


def _rows(rng, T, most=30):
    """Rows to compare: both ends and some between."""
    return np.unique(np.concatenate([np.arange(min(T, 3)), T - 1 - np.arange(min(T, 3)), rng.integers(0, T, most)]))


class Alike:
    """Many adapters as powers of two times one, made on the device: a pool that is quick to make."""

    def __init__(self, rng, n, K, widths, rank, fmt):
        self.N, self.widths, self.fmt = sum(widths), widths, fmt
        a_bits, self.a = values(rng, (len(widths), rank, K), fmt, K ** -0.5)
        b_bits, self.b = values(rng, (self.N, rank), fmt, 0.5 * rank ** -0.5)
        self.factor = 2.0 ** (np.arange(n) % 3) * np.where(np.arange(n) % 2, -1, 1)   # exact
        blocks = [to_torch(bits, fmt, DEV) for bits in (a_bits, b_bits)]
        made = [torch.empty((n, *block.shape), dtype=block.dtype, device=DEV) for block in blocks]
        for block, out in zip(blocks, made):
            for i in range(n):
                torch.mul(block, float(self.factor[i]), out=out[i])
        self.adapters = qg.LoraAdapters(*made, widths=widths)

    def expected(self, x, ids, base=None):
        """The oracle's, of few rows: each row with an adapter of its own."""
        f = self.factor[np.maximum(ids, 0)]
        own = np.where(ids >= 0, np.arange(len(ids)), -1)
        return lora_oracle.lora(x, f[:, None, None, None] * self.a, f[:, None, None] * self.b, own, self.fmt,
                                widths=self.widths, base=base)


def _compare(rng, T, K, widths, rank, n, fmt, ids, pool=Pool):
    _say(T, K, widths, rank, n, fmt)
    p = Pool(rng, n, K, widths, rank, fmt, DEV) if pool is Pool else pool(rng, n, K, widths, rank, fmt)
    x_bits, x = values(rng, (T, K), fmt)
    base_bits, base = values(rng, (1, p.N), fmt)
    turn = np.array([1.0, 2.0, -4.0])[np.arange(T) % 3][:, None]   # rows of the base: powers of two times one, exact
    one = to_torch(base_bits, fmt, DEV)
    bd = (one.float() * torch.from_numpy(turn).float().to(DEV)).to(one.dtype)
    xd = to_torch(x_bits, fmt, DEV)
    od, buf = guarded(T, p.N, fmt, DEV, 8, np.broadcast_to(np.uint16(NAN[fmt]), (T, p.N)))
    qg.lora(xd, p.adapters, _batch(ids, n), base=bd, out=od)
    same = bd.clone()
    qg.lora(xd, p.adapters, _batch(ids, n), base=same, out=same)   # in place
    torch.cuda.synchronize()
    assert torch.isfinite(od).all() and torch.equal(od, same)
    at = _rows(rng, T)
    check(od[torch.from_numpy(at).to(DEV)], *p.expected(x[at], ids[at], base * turn[at]), fmt, (T, K, widths, rank, n))
    assert untouched(buf, T, p.N, 8)


@pytest.mark.parametrize("T,rank,widths", [
    (512, 8, [16440]),                      # 65 workgroups of two runs each, the last part empty
    (520, 16, [8200, 264, 520, 7992]),      # slices that end inside a workgroup's and a wave's run
    (500, 24, [16968, 8]),
    (300, 72, [20000, 3000, 3000]),
    (2600, 16, [8000, 3608, 1032]),         # tall tiles
    (800, 40, [29256]),
    (1100, 136, [20000, 9000]),
], ids=str)
@pytest.mark.parametrize("fmt", ["f16", "bf16"])
def test_several_runs_of_columns_to_a_wave(T, rank, widths, fmt):
    rng = np.random.default_rng(T + rank)
    _compare(rng, T, 40, widths, rank, 5, fmt, rng.integers(-1, 5, T))


def test_more_tiles_than_counters():
    rng = np.random.default_rng(31)
    # 32 chunks of ranks for each of up to 600 tiles of 16 rows; 16 for each of 1100 of 64
    _compare(rng, 600, 1032, [8, 16, 8, 8, 24, 8, 8, 8], 256, 600, "f16", rng.permutation(600), Alike)
    _compare(rng, 1100, 520, [8] * 8, 128, 1100, "bf16", rng.permutation(1100), Alike)


@pytest.mark.parametrize("T,rank", [(767, 40), (768, 40), (1023, 16), (1024, 72), (2559, 32), (2560, 8)])
def test_the_last_row_counts_of_low_tiles(T, rank):
    rng = np.random.default_rng(T)
    _compare(rng, T, 72, [72, 136], rank, 5, "f16", np.sort(rng.integers(-1, 5, T)))
    _compare(rng, T, 72, [72, 136], rank, 2000, "bf16", rng.integers(0, 2000, T))


@pytest.mark.parametrize("tall", [False, True])
def test_a_million_columns(tall):
    """More column tiles than a grid of one workgroup for every four of them allows: four runs to a wave with 520 tiles of
    16 rows, and tall tiles of a pool of one."""
    T, n, N, R, K = (2600, 1, 1 << 20, 8, 16) if tall else (520, 520, 1 << 20, 8, 16)
    _say("a million columns", T, n)
    rng = np.random.default_rng(33)
    p = Alike(rng, n, K, [N], R, "f16")
    x_bits, x = values(rng, (T, K), "f16")
    ids = np.arange(T) % n
    ids[5] = -1
    out = torch.full((T, N), float("nan"), dtype=torch.float16, device=DEV)
    qg.lora(to_torch(x_bits, "f16", DEV), p.adapters, _batch(ids, n), out=out)
    torch.cuda.synchronize()
    for t in (0, 1, 5, T // 2, T - 1):
        check(out[t:t + 1], *p.expected(x[t:t + 1], ids[t:t + 1]), "f16", (tall, t))
    assert all(bool(torch.isfinite(rows).all()) for rows in out.split(64))

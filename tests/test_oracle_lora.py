"""The oracle of the low-rank adapters against the same formula written as dense matrices, and the sharpness of its bound:
what a wrong adapter, rank, slice or scale does to the outputs lies far outside it."""

import numpy as np
import pytest

from oracle import attention as oa
from oracle import lora as ol


def _problem(seed, T=7, K=24, widths=(16, 8), rank=16, n=3, fmt="f16"):
    rng = np.random.default_rng(seed)
    S, N = len(widths), sum(widths)

    def values(shape, dev_of):
        return oa.decode(oa.encode(rng.standard_normal(shape) * dev_of, fmt), fmt)

    return dict(x=values((T, K), 1.0), a=values((n, S, rank, K), K ** -0.5), b=values((n, N, rank), 0.3), fmt=fmt,
                ids=rng.integers(-1, n + 1, T), scales=0.5 + rng.random(n), ranks=np.array([16, 8, 3]), widths=list(widths),
                base=values((T, N), 1.0))


def _dense(p, t, ranks=True):
    i = int(p["ids"][t])
    out = p["base"][t].copy()
    if not 0 <= i < 3:
        return out
    keep = np.arange(16) < ((p["ranks"][i] + 7) // 8 * 8 if ranks else 16)
    at = 0
    for j, w in enumerate(p["widths"]):
        W = (p["b"][i, at:at + w] * keep) @ p["a"][i, j]
        out[at:at + w] += p["scales"][i] * (W @ p["x"][t])
        at += w
    return out


@pytest.mark.parametrize("fmt", ["f16", "bf16"])
@pytest.mark.parametrize("seed", range(4))
def test_matches_dense_matrices(seed, fmt):
    p = _problem(seed, fmt=fmt)
    out, bound = ol.lora(**p)
    for t in range(7):
        assert np.allclose(out[t], _dense(p, t), rtol=1e-12, atol=1e-12)
    # at least the output's rounding, and not many times it
    least = oa.ROUNDOFF[fmt] * np.abs(out)
    assert np.all(bound >= least) and np.all(bound <= least * 1.1 + 2e-3 * oa.ROUNDOFF[fmt] / oa.ROUNDOFF["f16"])


def test_defaults_and_missing_base():
    p = _problem(9, widths=(24,))
    full = ol.lora(p["x"], p["a"], p["b"], p["ids"], "f16", base=p["base"])[0]
    none = ol.lora(p["x"], p["a"], p["b"], p["ids"], "f16")[0]
    assert np.allclose(full - none, p["base"], atol=1e-12)
    assert not none[(p["ids"] < 0) | (p["ids"] >= 3)].any()


@pytest.mark.parametrize("change", [dict(ranks=np.array([16, 16, 16])), dict(ranks=np.array([8, 8, 3])),
                                    dict(scales=np.array([0.9, 0.8, 0.7])), dict(widths=[8, 16])])
def test_planted_mistakes_leave_the_bound(change):
    p = _problem(5)
    p["ids"] = np.array([0, 1, 2, 0, 1, 2, -1])
    out, bound = ol.lora(**p)
    wrong = ol.lora(**dict(p, **change))[0]
    assert np.any(np.abs(wrong - out) > 10 * bound)
    p2 = dict(p, ids=np.roll(p["ids"], 1))
    assert np.any(np.abs(ol.lora(**p2)[0] - out) > 10 * bound)

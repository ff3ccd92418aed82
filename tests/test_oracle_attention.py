"""The attention oracle against hand cases and brute force: number formats, rotation, visibility, attention."""

import numpy as np
import pytest

from oracle import attention as oa


def test_e4m3_values():
    assert oa.E4M3[0x38] == 1.0 and oa.E4M3[0x7E] == 448.0 and oa.E4M3[0x01] == 2.0 ** -9
    assert np.isnan(oa.E4M3[0x7F]) and np.isnan(oa.E4M3[0xFF]) and oa.E4M3[0xB8] == -1.0
    assert np.all(np.diff(oa.E4M3[:127]) > 0)


def test_e4m3_encode_round_trips_and_rounds_to_even():
    codes = np.array([c for c in range(256) if c % 128 != 127], dtype=np.uint8)
    assert np.array_equal(oa.encode(oa.decode(codes, "fp8"), "fp8"), codes)
    # halfway between 1 (mantissa 0) and 1.125 (mantissa 1), and between 1.125 and 1.25
    assert oa.encode(np.array([1.0625, 1.1875, 1e9, -1e9]), "fp8").tolist() == [0x38, 0x3A, 0x7E, 0xFE]
    assert oa.encode(np.array([np.nan]), "fp8")[0] == 0x7F


@pytest.mark.parametrize("fmt,x,bits", [("bf16", 1.0, 0x3F80), ("bf16", 1.00390625, 0x3F80), ("bf16", -2.5, 0xC020),
                                        ("f16", 1.0, 0x3C00), ("f16", 65504.0, 0x7BFF)])
def test_16_bit_patterns(fmt, x, bits):
    assert int(oa.encode(np.array([x]), fmt)[0]) == bits


def test_rotation_by_a_quarter_turn():
    x = np.arange(1.0, 9.0).reshape(1, 8)
    quarter = (np.zeros(2), np.ones(2))
    out, _ = oa.norm_rotate(x, None, 0.0, quarter, False)
    assert out.tolist() == [[-3, -4, 1, 2, 5, 6, 7, 8]]
    out, _ = oa.norm_rotate(x, None, 0.0, quarter, True)
    assert out.tolist() == [[-2, 1, -4, 3, 5, 6, 7, 8]]


def test_norm_has_unit_mean_square():
    x = np.random.default_rng(0).standard_normal((3, 32)) * 7
    out, _ = oa.norm_rotate(x, np.ones(32), 0.0, (np.ones(0), np.ones(0)), False)
    assert np.allclose((out ** 2).mean(axis=1), 1.0)


def test_visible_tokens():
    assert oa.visible(5, 8, 0, 0).tolist() == [True] * 6 + [False] * 2
    assert np.flatnonzero(oa.visible(9, 12, 3, 2)).tolist() == [0, 1, 7, 8, 9]
    assert np.flatnonzero(oa.visible(1, 12, 3, 2)).tolist() == [0, 1]
    assert not oa.visible(-1, 4, 0, 0).any()


def test_attention_brute_force():
    rng = np.random.default_rng(1)
    q, k, v = rng.standard_normal((2, 4)), rng.standard_normal((5, 2, 4)), rng.standard_normal((5, 2, 4))
    see = np.array([True, False, True, True, False])
    out, mag, _ = oa.attend(q, k, v, see, 0.7)
    for h in range(2):
        e = [np.exp(0.7 * sum(q[h, d] * k[j, h, d] for d in range(4))) if see[j] else 0.0 for j in range(5)]
        for d in range(4):
            assert out[h, d] == pytest.approx(sum(e[j] * v[j, h, d] for j in range(5)) / sum(e))
            assert mag[h, d] == pytest.approx(sum(e[j] * abs(v[j, h, d]) for j in range(5)) / sum(e))
    # equal keys give the mean, one visible token its own value, none zeros
    out, _, _ = oa.attend(q, np.ones((5, 2, 4)), v, see, 0.7)
    assert np.allclose(out, v[see].mean(axis=0))
    assert np.allclose(oa.attend(q, k, v, np.arange(5) == 3, 0.7)[0], v[3])
    assert not oa.attend(q, k, v, np.zeros(5, dtype=bool), 0.7)[0].any()

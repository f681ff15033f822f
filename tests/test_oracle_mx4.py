"""Pins of the MXFP4 oracle: the format's tables, the rounding rule, and the
formulas on cases with known answers."""
from fractions import Fraction

import numpy as np
import pytest

from oracle import mx4_oracle as M


def _pack(nibbles):
    n = np.asarray(nibbles, dtype=np.uint8).reshape(1, -1)
    return n[:, 0::2] | (n[:, 1::2] << 4)


def test_every_code_and_the_scale_bytes():
    codes = _pack(list(range(16)) * 2)
    want = [0, 0.5, 1, 1.5, 2, 3, 4, 6] + [-v for v in (0, 0.5, 1, 1.5, 2, 3, 4, 6)]
    for s in (0, 1, 126, 127, 128, 254):
        got = M.decode(codes, np.array([[s]], dtype=np.uint8))[0]
        assert [Fraction(v) for v in got] == [Fraction(v) * Fraction(2) ** (s - 127) for v in want * 2]
    assert np.isnan(M.decode(codes, np.array([[255]], dtype=np.uint8))).all()


def test_low_nibble_is_the_even_element():
    v = M.decode(np.array([[0x21] + [0] * 15], dtype=np.uint8), np.array([[127]], dtype=np.uint8))[0]
    assert v[0] == 0.5 and v[1] == 1.0 and not v[2:].any()


def test_values_of_the_grid_survive():
    rng = np.random.default_rng(3)
    for e in (-100, -3, 0, 9, 60):
        v = rng.choice(M.MAGNITUDES, (5, 64)) * rng.choice([-1, 1], (5, 64))
        v[:, ::32] = 6.0  # the block's scale is then 2^e
        x = np.ldexp(v, e)
        np.testing.assert_array_equal(M.decode(*M.quantize(x)), x)


@pytest.mark.parametrize("value,want", [(0.25, 0.0), (0.75, 1.0), (1.25, 1.0), (1.75, 2.0), (2.5, 2.0), (3.5, 4.0),
                                        (5.0, 4.0), (0.2500001, 0.5), (4.9999, 4.0), (5.0001, 6.0), (7.5, 6.0)])
def test_ties_go_to_the_even_code_and_six_saturates(value, want):
    x = np.zeros((1, 32))
    x[0, 0], x[0, 1], x[0, 2] = 4.0, value, -value
    got = M.decode(*M.quantize(x))[0]
    assert got[1] == want and got[2] == -want


def test_scale_rule_zero_subnormal_and_bad_blocks():
    x = np.zeros((1, 7 * 32), dtype=np.float32)
    x[0, 32] = 1.0                                # floor(log2) = 0 -> 2^-2
    x[0, 64] = np.float32(2.0 ** -149)            # below the lowest scale's half step
    x[0, 96] = np.float32(2.0 ** -127)
    x[0, 128] = np.nan
    x[0, 160] = np.inf
    x[0, 192] = np.finfo(np.float32).max
    codes, s = M.quantize(x)
    assert s[0].tolist() == [0, 125, 0, 0, 255, 255, 252]
    assert codes[0, 64:96].max() == 0 and codes[0, 32:48].max() == 0
    assert codes[0, 48] == 2                      # 2^-127 at scale byte 0 is 1.0
    assert codes[0, 96] == 7                      # saturates
    neg = np.full((1, 32), -0.0)
    assert (M.quantize(neg)[0] == 0x88).all()     # the sign stays


def test_rounding_is_nearest_by_brute_force():
    rng = np.random.default_rng(5)
    x = rng.standard_normal((40, 32))
    codes, s = M.quantize(x)
    got = M.decode(codes, s)
    grid = np.concatenate([M.MAGNITUDES, -M.MAGNITUDES])
    for r in range(40):
        unit = 2.0 ** (float(s[r, 0]) - 127)
        best = np.abs(x[r][:, None] - unit * grid).min(1)
        np.testing.assert_array_equal(np.abs(x[r] - got[r]), best)


def test_route_ties_nan_bias_and_renormalization():
    l = np.array([[1.0, 3.0, 3.0, np.nan, -np.inf]])
    with np.errstate(invalid="ignore"):
        ids, _ = M.route(l, 5, "sigmoid")
    assert ids.tolist() == [[1, 2, 0, 4, 3]]
    ids, w = M.route(np.array([[0.0, 0.0, 0.0, 0.0]]), 2)
    assert ids.tolist() == [[0, 1]] and np.allclose(w, 0.5)
    _, w = M.route(np.array([[0.0, 0.0, 0.0, 0.0]]), 2, renormalize=False, scale=3.0)
    assert np.allclose(w, 0.75)
    ids, w = M.route(np.array([[0.0, 1.0]]), 1, "sigmoid", bias=np.array([5.0, 0.0]), renormalize=False)
    assert ids.tolist() == [[0]] and np.allclose(w, 0.5)  # the bias chooses, it does not weigh


def test_moe_of_one_expert_is_its_mlp_and_the_shared_expert_adds():
    rng = np.random.default_rng(8)
    x = rng.standard_normal((3, 64))
    gu, dn = M.quantize(rng.standard_normal((2 * 32, 64))), M.quantize(rng.standard_normal((64, 32)))
    layer = {"router": np.zeros((1, 64)), "gate_up": (gu[0].reshape(1, 2, 32, 32), gu[1].reshape(1, 2, 32, 2)),
             "down": (dn[0].reshape(1, 1, 64, 16), dn[1].reshape(1, 1, 64, 1))}
    g, d = M.decode(*gu), M.decode(*dn)
    want = M.swiglu(x, g[:32], g[32:], d)
    y, ids, w = M.moe(x, layer, 1)
    np.testing.assert_allclose(y, want)
    layer["shared"] = (layer["gate_up"], layer["down"])
    layer["shared_gate"] = np.zeros(64)
    np.testing.assert_allclose(M.moe(x, layer, 1)[0], 1.5 * want)

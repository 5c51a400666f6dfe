"""Pins of the 4-bit cache's host oracle: hand-worked grids, the packing, the
rotation's invariances, and attention's masks."""

import numpy as np
import pytest

import kv4_cases
from oracle import kv4 as ok
from oracle import transform


def test_grid_hand_worked():
    # lo = -1, hi = 2: s = 3/15 = 0.2 to 20 bits, zero = 5
    c, s, z = ok.quantize(np.array([[-1.0, 2.0, 0.0, 0.31]]))
    assert abs(float(s[0]) / 0.2 - 1) <= 2.0 ** -20 and z[0] == 5
    assert c[0].tolist() == [0, 15, 5, 7]          # 0.31 / 0.2 = 1.55 -> 2
    # one-sided vectors keep 0 on the grid
    c, s, z = ok.quantize(np.array([[3.0, 1.0]]))
    assert z[0] == 0 and c[0].tolist() == [15, 5]
    # all zero
    c, s, z = ok.quantize(np.zeros((1, 4)))
    assert s[0] == 2.0 ** -100 and z[0] == 0 and not c.any()


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_grid_not_finite(bad):
    c, s, z = ok.quantize(np.array([[1.0, bad, -2.0]]))
    assert np.isnan(s[0]) and not c.any() and ok.words(s, z)[0] == 0x7FC00000


def test_values_within_half_a_step():
    r = np.random.default_rng(0)
    x = (r.standard_normal((50, 128)) * np.exp(r.uniform(-20, 20, (50, 1)))).astype(np.float32)
    c, s, z = ok.quantize(x)
    w = ok.words(s, z)
    # half a step of the code, and half a step of the zero point at the ends
    err = np.abs(ok.values(c, w) - x.astype(np.float64)).max(-1)
    assert (err <= 1.0001 * s.astype(np.float64)).all()
    assert (np.median(np.abs(ok.values(c, w) - x), -1) <= 0.5 * s).all()


def test_block_round_trip():
    r = np.random.default_rng(1)
    P, D = 16, 64
    block = np.zeros(P * (D + 8), dtype=np.uint8)
    c = r.integers(0, 16, (2, P, D)).astype(np.uint8)
    w = r.integers(0, 2 ** 32, (2, P), dtype=np.uint32)
    for i in (0, 1):
        for t in range(P):
            ok.put(block, P, D, t, c[i, t], w[i, t], i)
    kc, vc, kw, vw = ok.split_block(block, P, D)
    assert (kc == c[0]).all() and (vc == c[1]).all() and (kw == w[0]).all() and (vw == w[1]).all()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_keeps_scores(D, interleaved):
    """Scores depend on the distance of positions only, and the Hadamard
    transform (the library's, with its signs) does not change them."""
    r = np.random.default_rng(D)
    q, k = r.standard_normal((1, D)), r.standard_normal((1, D))
    f = 100.0 ** (-np.arange(0, D, 2) / D)
    row = lambda p: np.concatenate([np.cos(p * f), np.sin(p * f)])  # noqa: E731
    s = (1 - 2 * r.integers(0, 2, D)).astype(np.int8)
    a = float((ok.rotate(q, row(7), D, interleaved, None) @ ok.rotate(k, row(3), D, interleaved, None).T)[0, 0])
    b = float((ok.rotate(q, row(19), D, interleaved, s) @ ok.rotate(k, row(15), D, interleaved, s).T)[0, 0])
    assert abs(a - b) <= 1e-5 * D
    h = ok.rotate(q, row(0), 0, False, s)
    assert np.abs(h - q @ transform.dense(D, s).T).max() <= 1e-5


def test_masks():
    assert ok.visible(4, 8, True, 0, 0).tolist() == [1, 1, 1, 1, 1, 0, 0, 0]
    assert ok.visible(4, 8, True, 2, 0).tolist() == [0, 0, 0, 1, 1, 0, 0, 0]
    assert ok.visible(4, 8, True, 2, 1).tolist() == [1, 0, 0, 1, 1, 0, 0, 0]
    assert ok.visible(4, 8, False, 0, 0).all()
    assert not ok.visible(-1, 4, True, 0, 0).any()
    o, lse, p = ok.attend(np.ones(4), np.ones((3, 4)), np.ones((3, 4)), 1.0, np.zeros(3, bool))
    assert not o.any() and lse == -np.inf and not p.any()


@pytest.mark.parametrize("n,D", [(2, 64), (2, 128), (4, 256), (8, 128), (16, 64)])
def test_cancelling_pairs_catch_one_term(n, D):
    """The inputs of the GPU's test of fp16 weights in two terms: rounding them to one is beyond its bound
    (but where the few weights of a draw happen to lie next to fp16 numbers)."""
    caught = 0
    for seed in range(20):
        s, z, c = kv4_cases.pairs(np.random.default_rng(seed), n, D)
        o, v = kv4_cases.exact(s, z, c)
        tol = kv4_cases.bound(o, v, s, 2.0 ** -10)
        caught += (np.abs(kv4_cases.with_one_term(s, z, c) - o) > tol).any()
    assert caught >= 15

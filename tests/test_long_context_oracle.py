"""Pins of the float64 oracle of the long-context operators: closed forms,
central differences, and values worked by hand."""
import numpy as np
import pytest

from oracle import block_oracle as B
from oracle import long_context_oracle as L


def test_norm_has_unit_mean_square_and_turning_keeps_it():
    rng = np.random.default_rng(0)
    x, w = rng.standard_normal((5, 2, 12)), rng.standard_normal(12)
    ang = rng.uniform(-3, 3, (9, 4))
    table, pos = np.stack([np.cos(ang), np.sin(ang)], -1), rng.integers(0, 9, 5)
    y = L.qk_norm(x, None, pos, table, 0.0)
    np.testing.assert_allclose((y * y).mean(-1), 1, rtol=1e-12)
    np.testing.assert_allclose(L.qk_norm(3 * x, w, pos, table, 0.0), L.qk_norm(x, w, pos, table, 0.0), rtol=1e-12)
    np.testing.assert_allclose(L.qk_norm(x, w, pos, None, 0.5)[1, 1], x[1, 1] * w / np.sqrt((x[1, 1] ** 2).sum() / 12 + 0.5))


@pytest.mark.parametrize("pairs,turned", [(False, True), (True, True), (False, False)])
def test_norm_gradient_by_differences(pairs, turned):
    rng = np.random.default_rng(1)
    x, w, g = rng.standard_normal((3, 2, 8)), rng.standard_normal(8), rng.standard_normal((3, 2, 8))
    ang = rng.uniform(-3, 3, (9, 3))
    table, pos = np.stack([np.cos(ang), np.sin(ang)], -1) if turned else None, rng.integers(0, 9, 3)
    f = lambda x, w: (L.qk_norm(x, w, pos, table, 0.1, pairs) * g).sum()
    dx, dw, _, _ = L.qk_norm_grad(x, w, pos, table, 0.1, g, pairs)
    h = 1e-6
    for at in np.ndindex(x.shape):
        e = np.zeros_like(x)
        e[at] = h
        assert abs((f(x + e, w) - f(x - e, w)) / (2 * h) - dx[at]) < 1e-8
    for d in range(8):
        e = np.zeros(8)
        e[d] = h
        assert abs((f(x, w + e) - f(x, w - e)) / (2 * h) - dw[d]) < 1e-8


def test_window_mask_by_hand():
    seen, pos = L.window_mask(6, 6, [0, 6], [0, 6], 2, 1)
    want = ["100000", "110000", "111000", "101100", "100110", "100011"]
    assert ["".join(str(int(v)) for v in r) for r in seen] == want and list(pos) == list(range(6))
    seen, _ = L.window_mask(2, 5, [0, 2], [0, 5], 2, 0, causal=False)  # queries stand at 3 and 4
    assert ["".join(str(int(v)) for v in r) for r in seen] == ["00111", "00011"]
    a, _ = L.window_mask(7, 7, [0, 3, 7], [0, 3, 7], 100, 3)
    assert (a == B.mask(7, 7, [0, 3, 7], [0, 3, 7])[0]).all()


def test_ring_holds_the_sinks_and_the_newest():
    held = {}
    for p in range(23):
        held[L.ring_row(p, 3, 8)] = p
    assert sorted(held.values()) == [0, 1, 2, 18, 19, 20, 21, 22]
    rng = np.random.default_rng(2)
    k, v, q = rng.standard_normal((1, 23, 2, 4)), rng.standard_normal((1, 23, 2, 4)), rng.standard_normal((1, 4, 4))
    rk, rv = np.zeros((1, 8, 2, 4)), np.zeros((1, 8, 2, 4))
    for r, p in held.items():
        rk[0, r], rv[0, r] = k[0, p], v[0, p]
    s = np.array([0.5, 0.25, 0.0, 1.0])
    np.testing.assert_allclose(L.window_decode(q, rk, rv, [23], 5, 3, ring=True, cap=2.0, slopes=s),
                               L.window_decode(q, k, v, [23], 5, 3, cap=2.0, slopes=s), rtol=1e-12)


def test_four_bit_values_by_hand():
    x = np.zeros((1, 40))
    x[0, :6] = [6.9, -0.25, 0.75, 2.5, -5.0, 1.25]     # largest below 7: scale 1; ties to the even code
    x[0, 32:35] = [7.0, 1.0, -3.0]                      # 7: scale 2
    c, s = L.kv4_encode(x)
    assert s.tolist() == [[127, 128]]
    np.testing.assert_array_equal(L.kv4_decode(c, s, 40)[0, :6], [6.0, -0.0, 1.0, 2.0, -4.0, 1.0])
    np.testing.assert_array_equal(L.kv4_decode(c, s, 40)[0, 32:35], [8.0, 1.0, -3.0])
    assert c[0, 0] == (7 | 8 << 4) and c.shape == (1, 32)
    c, s = L.kv4_encode(np.array([[np.inf] + [0.0] * 31, [0.0] * 32, [3.0e38] + [0.0] * 31]))
    assert s.tolist() == [[255], [0], [252]] and np.isnan(L.kv4_decode(c, s, 32)[0]).all()
    assert L.kv4_decode(c, s, 32)[2, 0] == 6 * 2.0 ** 125
    assert not L.kv4_decode(c, s, 32)[1].any()


def test_four_bit_values_are_within_half_a_step():
    rng = np.random.default_rng(3)
    x = rng.standard_normal((20, 64)) * 10.0 ** rng.integers(-30, 30, (20, 1))
    c, s = L.kv4_encode(x)
    y = L.kv4_decode(c, s, 64)
    scale = np.repeat(2.0 ** (s.astype(float) - 127), 32, -1)
    a = np.abs(x) / scale
    half = np.where(a <= 2, 0.25, np.where(a <= 4, 0.5, 1.0))
    assert (np.abs(y - x) <= half * scale).all()
    c2, s2 = L.kv4_encode(y)
    np.testing.assert_array_equal(L.kv4_decode(c2, s2, 64), y)  # a held value stays what it is

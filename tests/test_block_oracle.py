"""The float64 oracle of the attention-block operators against what fixes it:
Philox 4x32-10's published test vectors, rotation by complex numbers, explicit
softmax, and central differences for every gradient.  CPU only."""
import numpy as np
import pytest

from oracle import block_oracle as B


@pytest.mark.parametrize("ctr,key,want", [
    ((0,) * 4, (0,) * 2, (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((B.M32,) * 4, (B.M32,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)),
])
def test_philox_vectors(ctr, key, want):
    assert tuple(B.philox(ctr, key)) == want


def test_dropout_mean_and_offset():
    n, p = 40000, 0.3
    k = B.keep(n, p, 77, 0)
    sd = (p * (1 - p) / n) ** 0.5
    assert abs(k.mean() - (1 - p)) < 5 * sd
    # an offset continues the same sequence
    np.testing.assert_array_equal(B.keep(100, p, 77, 24), k[24:124])
    x = np.array([1.0, np.nan, np.inf])
    assert np.array_equal(B.dropout(x, None, 1.0, 5, 0), np.zeros(3))
    assert np.array_equal(B.dropout(x[:1], [2.0], 0.0, 5, 0), [3.0])


@pytest.mark.parametrize("pairs", [False, True])
def test_rope_is_a_complex_product(pairs):
    rng = np.random.default_rng(0)
    x, ang = rng.standard_normal((5, 3, 12)), rng.standard_normal((9, 4))
    table, pos = np.stack([np.cos(ang), np.sin(ang)], -1), np.array([8, 0, 3, 3, 1])
    y = B.rope(x, pos, table, pairs)
    a, b = (np.s_[..., 0:8:2], np.s_[..., 1:8:2]) if pairs else (np.s_[..., 0:4], np.s_[..., 4:8])
    z = (x[a] + 1j * x[b]) * np.exp(1j * ang[pos])[:, None, :]
    np.testing.assert_allclose(y[a] + 1j * y[b], z, atol=1e-14)
    np.testing.assert_array_equal(y[..., 8:], x[..., 8:])
    np.testing.assert_allclose(B.rope(y, pos, table, pairs, inverse=True), x, atol=1e-14)


def test_mask_intervals():
    """Every mask leaves each query one interval of keys and each key one
    interval of queries, with bounds that grow inside a document."""
    for causal in (True, False):
        seen, pos = B.mask(14, 17, [0, 3, 3, 10, 12], [1, 4, 6, 12, 17], [2, 1, 5, 0], causal)
        for m in (seen, seen.T):
            for r in m:
                js = np.nonzero(r)[0]
                assert js.size == 0 or js[-1] - js[0] + 1 == js.size
        assert not seen[12:].any() and not seen[:, 0].any()


@pytest.mark.parametrize("cap,bias,causal", [(0.0, False, True), (2.0, True, True), (1.5, False, False)])
def test_attention_gradients_against_differences(cap, bias, causal):
    rng = np.random.default_rng(3)
    Tq, Tk, Hq, Hk, D = 7, 9, 4, 2, 8
    q, k, v = (rng.standard_normal(s) for s in ((Tq, Hq, D), (Tk, Hk, D), (Tk, Hk, D)))
    dout = rng.standard_normal(q.shape)
    seen, pos = B.mask(Tq, Tk, [0, 4, 6], [0, 3, 8], [0, 2], causal)
    slopes = [0.5, 0.25, 0.1, 0.0] if bias else None
    out = B.attention(q, k, v, seen, pos, None, cap, slopes, dout)
    f = lambda: float((B.attention(q, k, v, seen, pos, None, cap, slopes)["o"] * dout).sum())
    for name, x in (("dq", q), ("dk", k), ("dv", v)):
        for idx in [tuple(rng.integers(0, n) for n in x.shape) for _ in range(12)]:
            old, e = x[idx], 1e-5
            x[idx] = old + e
            hi = f()
            x[idx] = old - e
            lo = f()
            x[idx] = old
            # central differences: error e^2 plus rounding 1e-16 / e
            assert abs((hi - lo) / (2 * e) - out[name][idx]) < 1e-8


def test_attention_is_softmax_of_the_masked_matrix():
    rng = np.random.default_rng(4)
    q, k, v = rng.standard_normal((6, 1, 8)), rng.standard_normal((6, 1, 8)), rng.standard_normal((6, 1, 8))
    seen, pos = B.mask(6, 6, [0, 6], [0, 6], None, True)
    out = B.attention(q, k, v, seen, pos)
    s = np.where(seen, q[:, 0] @ k[:, 0].T / 8 ** 0.5, -np.inf)
    p = np.exp(s - s.max(1, keepdims=True))
    np.testing.assert_allclose(out["o"][:, 0], (p / p.sum(1, keepdims=True)) @ v[:, 0], atol=1e-14)
    np.testing.assert_allclose(B.decode(q[5:], k[None], v[None], None, [6])[0], out["o"][5], atol=1e-14)

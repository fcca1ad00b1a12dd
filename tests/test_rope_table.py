"""Rotary tables: frequencies and the scalings for long contexts.  CPU only."""
import math

import pytest
import torch

from orthogonal_reparameterized_02_amd.attention import rope_frequencies, rope_table


def test_plain_frequencies_and_table():
    f = rope_frequencies(8, base=10000.0)
    torch.testing.assert_close(f, torch.tensor([1.0, 0.1, 0.01, 0.001], dtype=torch.float64))
    t = rope_table(5, 8, magnitude=2.0, device="cpu")
    assert t.shape == (5, 4, 2) and t.dtype == torch.float32
    assert math.isclose(t[3, 1, 0], 2 * math.cos(0.3), rel_tol=1e-6)
    assert math.isclose(t[3, 1, 1], 2 * math.sin(0.3), rel_tol=1e-6)


def test_scalings():
    f = rope_frequencies(64)
    torch.testing.assert_close(rope_frequencies(64, scaling=("linear", 4.0)), f / 4)
    g = rope_frequencies(64, scaling=("base", 4.0))
    assert g[0] == f[0] and math.isclose(g[-1], f[-1] / 4, rel_tol=1e-12)
    n, low, high = 4096, 1, 32
    r = rope_frequencies(64, scaling=("ramp", 4.0, n, low, high)) / f
    turns = n * f / (2 * math.pi)
    assert (r[turns >= high] == 1).all() and torch.allclose(r[turns <= low], torch.tensor(0.25, dtype=torch.float64))
    mid = (turns > low) & (turns < high)
    assert mid.any() and ((r[mid] > 0.25) & (r[mid] < 1)).all() and (r[1:] <= r[:-1] + 1e-12).all()


@pytest.mark.parametrize("args", [dict(rot=3), dict(rot=0), dict(rot=8, scaling=("linear", 0.0)),
                                  dict(rot=2, scaling=("base", 2.0)), dict(rot=8, scaling=("ramp", 2.0, 128, 4, 2)),
                                  dict(rot=8, scaling=("other", 2.0))])
def test_refusals(args):
    with pytest.raises(ValueError):
        rope_frequencies(**args)

"""The long-context operators as a user has them, together: autograd of each
against the float64 oracle, the block with qk norms, a window and sinks trained
packed and served from rings, in its own type and in 4 bits.

Tolerances.  bf16 2-norm: three independent roundings of 2^-8 at most, spread
evenly, make 2^-8, and the bound is 1.5 of that, 3 * 2^-9, as for the block's
operators; float32 1e-5."""
import math
import os
import sys

import numpy as np
import pytest
import torch

from gpu_util import bits, to_f64
from orthogonal_reparameterized_02_amd import attention as A
from orthogonal_reparameterized_02_amd import poetx as P
from oracle import block_oracle as B
from oracle import long_context_oracle as L

pytestmark = pytest.mark.gpu

BF16 = 3 * 2.0 ** -9


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def rel(a, b):
    a = to_f64(a) if torch.is_tensor(a) else a
    return np.linalg.norm(a - b) / np.linalg.norm(b)


def randn(*shape, dtype=torch.bfloat16, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed + sum(shape))).to(dtype).cuda()


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def block_of(**kw):
    """A small block whose projections are not the identity."""
    kw = dict(positions=512, qk_norm=True, window=24, sinks=3) | kw
    block = A.POETXAttention(256, 4, 2, 32, 3, **kw)
    with torch.no_grad():
        for i, (n, p) in enumerate(block.named_parameters()):
            p.copy_((1.0 if "norm" in n else 0.0) + (0.2 if "norm" in n else 0.02) * randn(*p.shape, dtype=torch.float32, seed=i))
    return block


# ---- operators ---------------------------------------------------------------------------
@pytest.mark.parametrize("interleaved", [False, True])
def test_qk_norm_gradients(interleaved):
    table, pos = A.rope_table(64, 32), torch.arange(40, dtype=torch.int32, device="cuda") % 64
    f = dict(dtype=torch.float32)
    q, k = randn(40, 4, 64, **f).requires_grad_(), randn(40, 2, 64, **f).requires_grad_()
    wq, wk = (1 + 0.3 * randn(64, **f)).requires_grad_(), (1 + 0.3 * randn(64, seed=5, **f)).requires_grad_()
    gq, gk = randn(40, 4, 64, seed=1, **f), randn(40, 2, 64, seed=2, **f)
    qo, ko = A.qk_norm_rope(q, k, wq, wk, pos, table, 1e-5, interleaved)
    ((qo * gq).sum() + (ko * gk).sum()).backward()
    t, p = table.cpu().numpy(), pos.cpu().numpy()
    for x, w, y, g in ((q, wq, qo, gq), (k, wk, ko, gk)):
        dx, dw, _, _ = L.qk_norm_grad(to_f64(x), to_f64(w), p, t, 1e-5, to_f64(g), interleaved)
        assert rel(y, L.qk_norm(to_f64(x), to_f64(w), p, t, 1e-5, interleaved)) <= 1e-5
        assert rel(x.grad, dx) <= 1e-5 and rel(w.grad, dw) <= 1e-5
    # alone, without weights or positions, and with weights that want no gradient
    y = A.qk_norm_rope(q, None, None, None, None, None)
    assert rel(y, L.qk_norm(to_f64(q), None, None, None, 1e-6)) <= 1e-5
    A.qk_norm_rope(q, None, wq.detach(), None, pos, table).sum().backward()
    with pytest.raises(ValueError, match="without k"):
        A.qk_norm_rope(q, None, wq, wk, pos, table)


def test_window_attention_gradients_on_views_of_one_projection():
    T, Hq, Hkv, D = 150, 4, 2, 64
    fused = randn(T, (Hq + 2 * Hkv) * D).requires_grad_()
    q, k, v = (fused[:, a * D:b * D].unflatten(1, (b - a, D)) for a, b in ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, Hq + 2 * Hkv)))
    slopes, g = A.alibi_slopes(Hq), randn(T, Hq, D, seed=5)
    o = A.attention(q, k, v, A.AttentionPlan(i32(0, 90, 145), T, window=30, sinks=4), cap=20.0, slopes=slopes)
    o.backward(g)
    seen, pos = L.window_mask(T, T, [0, 90, 145], [0, 90, 145], 30, 4)
    ref = B.attention(to_f64(q), to_f64(k), to_f64(v), seen, pos, None, 20.0, slopes.cpu().numpy(), to_f64(g))
    assert rel(o, ref["o"]) <= BF16
    want = np.concatenate([ref[n].reshape(T, -1) for n in ("dq", "dk", "dv")], 1)
    assert rel(fused.grad, want) <= BF16


@pytest.mark.parametrize("op", ["norm", "window"])
def test_second_derivatives_are_refused(op):
    x = randn(8, 2, 64, dtype=torch.float32).requires_grad_()
    if op == "norm":
        y = A.qk_norm_rope(x, None, None, None, i32(*range(8)), A.rope_table(8, 64))
    else:
        y = A.attention(x, x, x, A.AttentionPlan(i32(0, 8), 8, window=3, sinks=1))
    g, = torch.autograd.grad(y.square().sum() + x.square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        g.sum().backward()


# ---- the caches ----------------------------------------------------------------------------
def test_cache_in_four_bits_holds_the_nearest_values():
    cache = A.KVCache4(3, 100, 2, 72)
    assert cache.rows == 128
    k, v = randn(90, 2, 72), randn(90, 2, 72, seed=1)
    cache.fill(1, k[:50], v[:50])
    cache.extend(1, k[50:], v[50:])
    nearest = lambda x: L.kv4_decode(*L.kv4_encode(to_f64(x)), 72)
    for got, want in zip(cache.held(1), (k, v)):
        np.testing.assert_array_equal(to_f64(got), nearest(want))
    k1, v1 = randn(3, 2, 72, seed=7), randn(3, 2, 72, seed=8)
    cache.append(k1, v1)
    assert cache.length.tolist() == [1, 91, 1] and cache.longest() == 91
    np.testing.assert_array_equal(to_f64(cache.held(0)[0]), nearest(k1[:1]))
    np.testing.assert_array_equal(to_f64(cache.held(1)[1][90:]), nearest(v1[1:2]))
    q = randn(3, 4, 72)
    o = A.attention_decode(q, cache, cap=9.0, slopes=A.alibi_slopes(4), start=i32(0, 5, 0))
    hk, hv = np.zeros((3, 128, 2, 72)), np.zeros((3, 128, 2, 72))
    for b in range(3):
        n = cache.tokens(b)
        hk[b, :n], hv[b, :n] = (to_f64(t) for t in cache.held(b))
    assert rel(o, B.decode(to_f64(q), hk, hv, [0, 5, 0], [1, 91, 1], None, 9.0, A.alibi_slopes(4).cpu().numpy())) <= BF16
    with pytest.raises(ValueError, match="fit"):
        cache.extend(1, k[:40], v[:40])


@pytest.mark.parametrize("form", [A.KVCache, A.KVCache4])
def test_decode_over_part_of_a_cache(form):
    """A window over a cache that holds everything, and over a ring."""
    full, ring = form(2, 320, 2, 64), form(2, 64, 2, 64, window=50, sinks=4)
    k, v, q, slopes = randn(300, 2, 64), randn(300, 2, 64, seed=1), randn(2, 4, 64), A.alibi_slopes(4)
    for c in (full, ring):
        c.fill(0, k, v)
        c.fill(1, k[:40], v[:40])
    a = A.attention_decode(q, full, slopes=slopes, window=50, sinks=4)
    b = A.attention_decode(q, ring, slopes=slopes)
    hk, hv = (np.stack([to_f64(t)] * 2) for t in full.held(0))
    ref = L.window_decode(to_f64(q), hk, hv, [300, 40], 50, 4, slopes=slopes.cpu().numpy())
    assert rel(a, ref) <= BF16 and rel(b, ref) <= BF16
    with pytest.raises(ValueError, match="ring"):
        A.attention_decode(q, ring, window=40, sinks=4)
    with pytest.raises(ValueError, match="start"):
        A.attention_decode(q, full, window=40, start=i32(0, 0))


# ---- the block --------------------------------------------------------------------------------
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("whole", [False, True])
def test_served_tokens_equal_packed_ones(whole, bias):
    """Prefill and decode of two sequences from rings (or from a cache that
    holds everything) against the packed forward pass: the same products, summed
    in another order: two roundings of attention and one of the output projection
    apart."""
    block = block_of(bias=bias, cap=30.0).eval()
    lens = (80, 97)
    x = randn(sum(lens), 256)
    pos = torch.cat([torch.arange(m, dtype=torch.int32) for m in lens]).cuda()
    with torch.no_grad():
        packed = block(x, block.plan(i32(0, 80, 177), 177), pos)
        cache = A.KVCache(2, 128, 2, block.D) if whole else block.cache(2, 128)
        assert whole or (cache.ring and cache.rows == 27)
        first = [block.prefill(x[:20], cache, 0), block.prefill(x[80:80 + 60], cache, 1)]
        steps = [block.decode(torch.stack([x[20 + i], x[140 + i]]), cache) for i in range(37)]
    seqs = [torch.cat([first[0]] + [s[:1] for s in steps]), torch.cat([first[1]] + [s[1:] for s in steps])]
    for got, want in zip(seqs, (packed[:57], packed[80:177])):
        assert rel(got, to_f64(want)) <= 2 * BF16


def test_prompt_in_parts():
    """A prompt prefilled in parts over a ring that drops tokens is the whole
    one; with a bias, whose distances the ring has lost, it is refused."""
    block = block_of(cap=30.0).eval()
    x = randn(200, 256)
    want = block.prefill(x, block.cache(1, 512))
    cache, got = block.cache(1, 512), []
    for a, b in ((0, 10), (10, 40), (40, 41), (41, 130), (130, 200)):
        got.append(block.prefill(x[a:b], cache, 0, follow=a > 0))
    assert rel(torch.cat(got), to_f64(want)) <= 2 * BF16 and cache.tokens(0) == 200
    full = A.KVCache(1, 220, 2, block.D)
    parts = torch.cat([block.prefill(x[:90], full, 0, follow=True), block.prefill(x[90:], full, 0, follow=True)])
    assert rel(parts, to_f64(want)) <= 2 * BF16
    with pytest.raises(ValueError, match="fit"):
        block.prefill(x[:30], full, 0, follow=True)
    assert full.tokens(0) == 200
    biased = block_of(bias=True).eval()
    cache = biased.cache(1, 512)
    biased.prefill(x[:20], cache)
    biased.prefill(x[20:60], cache, follow=True)
    with pytest.raises(ValueError, match="bias"):
        biased.prefill(x[60:], cache, follow=True)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_served_from_four_bits(dtype):
    """Each decoded token is the attention over what the cache holds then,
    value by value: the block's output recomputed from held()."""
    block = block_of(dtype=dtype).eval()
    cache = block.cache(2, 512, four_bits=True)
    assert cache.ring and cache.rows == 64
    x = randn(260, 256, dtype=dtype)
    block.prefill(x[:10], cache, 0)
    block.prefill(x[20:100], cache, 1)
    tol = 2 * BF16 if dtype == torch.bfloat16 else 2e-5
    for i in range(6):
        t = x[200 + 2 * i:202 + 2 * i]
        y = block.decode(t, cache)
        with torch.no_grad():
            q = block.q(t).view(2, 4, block.D)
            q = A.qk_norm_rope(q, None, block.q_norm, None, cache.length - 1, block.table, block.eps)
            o = torch.empty_like(q)
            for b in range(2):
                k, v = (to_f64(s) for s in cache.held(b))
                n = cache.tokens(b)
                at = list(range(n)) if n <= 64 else [0, 1, 2, *range(n - 61, n)]  # what the ring holds
                seen = [j for j, p in enumerate(at) if p < 3 or p >= n - 24]
                r = B.attention(to_f64(q[b:b + 1]), k[seen], v[seen], np.ones((1, len(seen)), bool), np.array([len(seen) - 1]))
                o[b] = torch.from_numpy(r["o"][0]).to(dtype).cuda()
            want = t + block.o(o.view(2, -1))
        assert rel(y, to_f64(want)) <= tol, i
    assert cache.length.tolist() == [16, 86]


def test_captured_steps_go_round_the_ring():
    """A step captured once and replayed past the ring's rows: the eager steps,
    replay by replay; past the rotary table it answers NaN."""
    block = block_of(positions=64).eval()
    x = randn(2, 256)
    for four in (False, True):
        fresh = lambda: block.cache(2, 512, four_bits=four)
        eager, cache = fresh(), fresh()
        block.decode(x, fresh())
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            y = block.decode(x, cache)
        for c in (eager, cache):
            block.prefill(randn(30, 256, seed=1), c, 0)
            block.prefill(randn(5, 256, seed=2), c, 1)
        for i in range(34):
            want = block.decode(x, eager)
            g.replay()
            torch.cuda.synchronize()
            np.testing.assert_array_equal(bits(y), bits(want))
            assert cache.length.tolist() == eager.length.tolist() == [31 + i, 6 + i]
        with pytest.raises(ValueError, match="64 positions"):
            block.decode(x, eager)
        g.replay()
        torch.cuda.synchronize()
        assert torch.isnan(y[0]).all() and torch.isfinite(y[1]).all()
        assert cache.tokens(0) == 65 and cache.longest() == 65


def test_captured_appends_to_a_full_cache_in_four_bits():
    block = block_of(window=0, sinks=0).eval()
    cache = block.cache(2, 64, four_bits=True)
    x = randn(2, 256)
    block.decode(x, block.cache(2, 64, four_bits=True))
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = block.decode(x, cache)
    block.prefill(randn(62, 256, seed=1), cache, 0)
    block.prefill(randn(5, 256, seed=2), cache, 1)
    for i in range(4):
        before = [t.clone() for t in cache._cache]
        g.replay()
        torch.cuda.synchronize()
        assert cache.length.tolist() == [min(63 + i, 64), 6 + i]
        assert torch.isnan(y[0]).all() == (i >= 2) and torch.isfinite(y[1]).all()
        if i >= 2:
            assert all(torch.equal(a[0], b[0]) for a, b in zip(before, cache._cache))
    with pytest.raises(ValueError, match="full"):
        block.decode(x, cache)


def test_mismatched_windows_are_refused():
    block = block_of().eval()
    x, pos = randn(8, 256), i32(*range(8))
    with pytest.raises(ValueError, match="plan of window=0"):
        block(x, A.AttentionPlan(i32(0, 8), 8), pos)
    with pytest.raises(ValueError, match="ring"):
        block.prefill(x, A.KVCache(1, 64, 2, block.D, window=30, sinks=3))
    with pytest.raises(ValueError, match="ring"):
        block.decode(x[:1], A.KVCache(1, 64, 2, block.D, window=24, sinks=2))


def test_float32_block_gradient_by_differences():
    """A directional derivative over input and all parameters against a central
    difference.  Its error: rounding 2^-22 |loss| / step, truncation step^2."""
    block = block_of(dtype=torch.float32, cap=20.0)
    T = 80
    f = dict(dtype=torch.float32)
    x, g = randn(T, 256, **f).requires_grad_(), randn(T, 256, seed=1, **f)
    plan, pos = block.plan(i32(0, 50, T), T), torch.cat([torch.arange(50), torch.arange(30)]).to(torch.int32).cuda()
    (block(x, plan, pos) * g).sum().backward()
    leaves = [x, *block.parameters()]
    dirs = [randn(*t.shape, seed=i, **f) * (1.0 if i == 0 else 0.1) for i, t in enumerate(leaves)]
    want = sum((t.grad.double() * d.double()).sum().item() for t, d in zip(leaves, dirs))
    scale = math.sqrt(sum(t.grad.double().square().sum().item() for t in leaves) * sum(d.double().square().sum().item() for d in dirs))
    assert all(torch.isfinite(t.grad).all() and t.grad.abs().max() > 0 for t in leaves)
    h, ends = 2.0 ** -9, []
    with torch.no_grad():
        for s in (1, -1):
            for t, d in zip(leaves, dirs):
                t.add_(d, alpha=s * h)
            ends.append((block(x, plan, pos).double() * g.double()).sum().item())
            for t, d in zip(leaves, dirs):
                t.sub_(d, alpha=s * h)
    assert abs((ends[0] - ends[1]) / (2 * h) - want) <= 1e-3 * scale


def test_example_runs():
    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import long_context_block
    grads, far, far4 = long_context_block.main(n=256, heads=4, kv_heads=2, b=32, lengths=(60, 25), window=16, sinks=2, steps=2)
    assert all(math.isfinite(x) and x > 0 for x in grads) and far <= 2 * BF16 and math.isfinite(far4)

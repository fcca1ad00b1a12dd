"""GPU parity of the norms of queries and keys with rotary positions against the
float64 oracle.

Tolerances, from the float32 arithmetic: a head's sum of squares passes through
at most 16 + 6 additions (22 roundings of 2^-24, halved by the root), the root
and its reciprocal add 2, the products and the turn at most 6: below 20
roundings, 2^-19, of the terms that an element is made of.  A sum for the
weights has in addition the depth of its additions: under 2^9 here, 2^-15 of the
sum of the terms' magnitudes.  Each output is then rounded once (bf16: 2^-8)."""
import sys

import numpy as np
import pytest
import torch

from gpu_util import bits, to_dev, to_f64
from orthogonal_reparameterized_02_amd import poetx as P
from oracle import long_context_oracle as L

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8}
EPS = 1e-6


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    P.lib()


def normal(rng, shape, dt, scale=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(DT[dt]).cuda()


def near(name, got, ref, size, dt, rel=2.0 ** -19):
    """|got - ref| <= rel * size + half a step of the result, element by element."""
    err = np.abs(to_f64(got) - ref)
    bound = rel * size + HALF[dt] * (np.abs(ref) + rel * size) + 1e-38
    worst = (err / bound).max() if err.size else 0.0
    print(f"  {name}: worst error / bound {worst:.2f}", file=sys.stderr, flush=True)
    assert worst <= 1, (name, worst)


def case(T, Hq, Hk, D, rot, pairs, dt, weights=True, seed=0):
    rng = np.random.default_rng(seed + T + D + rot)
    st = dict(pairs=pairs, rot=rot)
    for n, H in (("q", Hq), ("k", Hk)):
        st[n] = normal(rng, (T, H, D), dt, 2.0) if H else None
        st["g" + n] = normal(rng, (T, H, D), dt) if H else None
        st["w" + n] = to_dev((1 + 0.5 * rng.standard_normal(D)).astype(np.float32)) if weights and H else None
    ang = rng.uniform(-9, 9, (50, max(rot, 2) // 2))
    st["table"] = to_dev(np.stack([np.cos(ang), np.sin(ang)], -1).astype(np.float32)) if rot else None
    st["pos"] = to_dev(rng.integers(0, 50, T).astype(np.int32)) if rot else None
    return st


def empty(t):
    return None if t is None else torch.full(t.shape, 7.0, dtype=t.dtype, device="cuda")


def run(st, stream=None):
    out = {n + "o": empty(st[n]) for n in "qk"} | {"d" + n: empty(st[n]) for n in "qk"}
    D = st["q"].shape[2]
    out |= {"dw" + n: torch.full((D,), 7.0, device="cuda") if st[n] is not None else None for n in "qk"}
    ws = torch.empty(P.poetx_qk_norm_rope_workspace_bytes(P.qk_norm_shape(st["q"], st["k"], st["table"])),
                     dtype=torch.uint8, device="cuda")
    a = (st["wq"], st["wk"], st["pos"], st["table"])
    P.poetx_qk_norm_rope_fwd(st["q"], st["k"], *a, out["qo"], out["ko"], eps=EPS, interleaved=st["pairs"], stream=stream)
    P.poetx_qk_norm_rope_bwd(st["gq"], st["gk"], st["q"], st["k"], *a, out["dq"], out["dk"], out["dwq"], out["dwk"], ws,
                             eps=EPS, interleaved=st["pairs"], stream=stream)
    return out


def compare(st, out, dt):
    host = lambda t: None if t is None else t.cpu().numpy()
    pos, table = host(st["pos"]), host(st["table"])
    for n in "qk":
        if st[n] is None:
            continue
        x, w, g = to_f64(st[n]), host(st["w" + n]), to_f64(st["g" + n])
        y = L.qk_norm(x, w, pos, table, EPS, st["pairs"])
        size = np.abs(y)
        if table is not None:  # an element is made of both of its pair
            flat = L.qk_norm(x, w, pos, None, EPS)
            h, r = table.shape[1], 2 * table.shape[1]
            both = (np.abs(flat[..., 0:r:2]) + np.abs(flat[..., 1:r:2])) if st["pairs"] else \
                np.abs(flat[..., :h]) + np.abs(flat[..., h:r])
            for sl in ((slice(0, r, 2), slice(1, r, 2)) if st["pairs"] else (slice(0, h), slice(h, r))):
                size[..., sl] = both
        near(n, out[n + "o"], y, size, dt)
        dx, dw, dsize, dwsize = L.qk_norm_grad(x, w, pos, table, EPS, g, st["pairs"])
        # the turned gradient is made of both of its pair: as large as the row's
        near("d" + n, out["d" + n], dx, dsize + np.abs(dsize).max(-1, keepdims=True), dt)
        near("dw" + n, out["dw" + n], dw, dwsize + dwsize.max(), "f32", 2.0 ** -15)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("T,Hq,Hk,D,rot,pairs", [
    (1, 4, 1, 64, 64, False), (7, 3, 0, 128, 128, True), (65, 5, 5, 104, 40, True), (33, 2, 1, 40, 12, False),
    (130, 8, 2, 128, 64, False), (9, 1, 1, 8, 2, False), (5, 2, 2, 24, 6, True), (31, 4, 4, 256, 96, False),
    (3, 1, 2, 512, 512, False), (4, 2, 1, 512, 2, False), (6, 9, 3, 512, 34, True), (40, 7, 1, 72, 0, False),
    (700, 32, 8, 128, 128, False)])
def test_norms(dt, T, Hq, Hk, D, rot, pairs):
    st = case(T, Hq, Hk, D, rot, pairs, dt)
    compare(st, run(st), dt)
    st["wq"] = st["wk"] = None
    compare(st, run(st), dt)


def test_strides_in_place_and_weights_not_wanted():
    rng = np.random.default_rng(3)
    T, H, D = 37, 4, 64
    st = case(T, H, H, D, 32, False, "bf16")
    wide = normal(rng, (T, 3 * H * D), "bf16")
    st["q"], st["k"] = wide[:, :H * D].view(T, H, D), wide[:, H * D:2 * H * D].view(T, H, D)
    keep = wide.clone()
    want = run(st)
    compare(st, want, "bf16")
    a = (st["wq"], st["wk"], st["pos"], st["table"])
    ws = torch.empty(1 << 20, dtype=torch.uint8, device="cuda")
    gq, gk = st["gq"].clone(), st["gk"].clone()
    P.poetx_qk_norm_rope_bwd(gq, gk, st["q"], st["k"], *a, gq, gk, None, None, ws, eps=EPS)
    np.testing.assert_array_equal(bits(gq), bits(want["dq"]))
    np.testing.assert_array_equal(bits(gk), bits(want["dk"]))
    P.poetx_qk_norm_rope_fwd(st["q"], st["k"], *a, st["q"], st["k"], eps=EPS)
    np.testing.assert_array_equal(bits(st["q"].contiguous()), bits(want["qo"]))
    np.testing.assert_array_equal(bits(st["k"].contiguous()), bits(want["ko"]))
    np.testing.assert_array_equal(bits(wide[:, 2 * H * D:].contiguous()), bits(keep[:, 2 * H * D:].contiguous()))


def test_positions_outside_the_table_and_rows_that_are_not_finite():
    st = case(12, 2, 1, 64, 32, False, "f32")
    st["pos"][3], st["pos"][5] = -1, 50
    st["q"][7, 1, 9] = float("nan")
    out = run(st)
    y = to_f64(out["qo"])
    bad = np.isnan(y)
    assert bad[[3, 5], :, :32].all() and not bad[[3, 5], :, 32:].any()
    assert bad[7, 1].all() and not bad[7, 0].any() and not np.delete(bad, [3, 5, 7], 0).any()
    d = np.isnan(to_f64(out["dq"]))
    assert d[[3, 5]].all() and d[7, 1].all() and not d[7, 0].any() and not np.delete(d, [3, 5, 7], 0).any()
    assert np.isnan(to_f64(out["dwq"])).all() and np.isnan(to_f64(out["dwk"]))[:32].all()


def test_zero_rows_and_no_tokens():
    st = case(5, 2, 1, 64, 64, True, "f32")
    st["q"][2] = 0
    out = run(st)
    assert not to_f64(out["qo"])[2].any()
    compare(st, out, "f32")
    none = case(0, 2, 1, 64, 64, True, "f32")
    out = run(none)
    assert not to_f64(out["dwq"]).any() and not to_f64(out["dwk"]).any()


def test_same_bits_on_another_stream_and_in_a_graph():
    st = case(300, 8, 2, 128, 128, False, "bf16")
    want = {n: bits(t) for n, t in run(st).items()}
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = run(st)
    s.synchronize()
    for n, t in got.items():
        np.testing.assert_array_equal(bits(t), want[n])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = run(st)
    for i in range(3):
        st["q"].mul_(-1)  # an odd function: outputs and dw change sign, dx does not
        g.replay()
        torch.cuda.synchronize()
        flip = 1 if i % 2 else -1
        assert torch.equal(out["qo"] * flip, torch.from_numpy(want["qo"].view(np.int16)).view(torch.bfloat16).cuda())
        np.testing.assert_array_equal(bits(out["dq"]), want["dq"])
        np.testing.assert_array_equal(bits(out["dwq"] * flip), want["dwq"])


def test_rows_past_two_to_the_31():
    """Element offsets past 32 bits: the last rows of a tall tensor."""
    T, H, D = 2 ** 21 + 3, 8, 128
    q = torch.empty(T, H, D, dtype=torch.bfloat16, device="cuda")
    st = case(64, H, 0, D, 0, False, "bf16")
    q[-64:] = st["q"]
    y = torch.zeros_like(q)
    P.poetx_qk_norm_rope_fwd(q, None, st["wq"], None, None, None, y, None, eps=EPS)
    near("q", y[-64:], L.qk_norm(to_f64(st["q"]), st["wq"].cpu().numpy(), None, None, EPS),
         np.abs(L.qk_norm(to_f64(st["q"]), st["wq"].cpu().numpy(), None, None, EPS)), "bf16")
    g = torch.zeros_like(q)
    g[-64:] = st["gq"]
    ws = torch.empty(P.poetx_qk_norm_rope_workspace_bytes(P.qk_norm_shape(q, None, None)), dtype=torch.uint8, device="cuda")
    dw = torch.empty(D, device="cuda")
    q[:-64] = 1
    P.poetx_qk_norm_rope_bwd(g, None, q, None, st["wq"], None, None, None, y, None, dw, None, ws, eps=EPS)
    dx, dwr, size, dwsize = L.qk_norm_grad(to_f64(st["q"]), st["wq"].cpu().numpy(), None, None, EPS, to_f64(st["gq"]))
    near("dq", y[-64:], dx, size + size.max(-1, keepdims=True), "bf16")
    near("dwq", dw, dwr, dwsize + dwsize.max(), "f32", 2.0 ** -15)
    assert not y[:-64].any()

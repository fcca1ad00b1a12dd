"""GPU parity of attention with a window and sinks against the float64 oracle.

Tolerances.  float32: 1e-5 relative (2-norm) as for attention.  bf16: p and ds
are rounded to bf16 once as matrix operands, delta comes from the rounded o, and
each output is rounded once.  A rounding is off by at most 2^-8 of its value and
spread evenly within that, 2^-8 / sqrt(3) in the 2-norm; three independent ones
make 2^-8, and the bound is 1.5 of that: 3 * 2^-9.  The largest difference is
bounded by 2e-2 of the largest value, five half steps.  lse is a float32 sum of
float32 exponentials: 5e-5 absolute."""
import sys

import numpy as np
import pytest
import torch

from gpu_util import bits, to_dev, to_f64
from orthogonal_reparameterized_02_amd import poetx as P
from oracle import block_oracle as B
from oracle import long_context_oracle as L

pytestmark = pytest.mark.gpu

FRO = {"f32": 1e-5, "bf16": 3 * 2.0 ** -9}
MAX = {"f32": 1e-4, "bf16": 2e-2}
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    P.lib()


def normal(rng, shape, dt, scale=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * scale).astype(np.float32)).to(DT[dt]).cuda()


def close(name, got, ref, dt):
    """2-norm and largest difference, with equal NaN and infinity patterns."""
    got, ref = to_f64(got) if torch.is_tensor(got) else got, np.asarray(ref, np.float64)
    fin = np.isfinite(ref)
    np.testing.assert_array_equal(np.isfinite(got), fin, err_msg=name)
    np.testing.assert_array_equal(got[np.isinf(ref)], ref[np.isinf(ref)], err_msg=name)
    # a probability of exp(-distance slope) leaves float32 (2^-126): what is left of it is no number there
    g, r = got[fin], np.where(np.abs(ref) < 2.0 ** -126, 0.0, ref)[fin]
    if not r.size or not np.abs(r).max():
        assert not g.size or np.abs(g).max() <= FRO[dt], name
        return
    fro, mx = np.linalg.norm(g - r) / np.linalg.norm(r), np.abs(g - r).max() / np.abs(r).max()
    print(f"  {name}: fro={fro:.2e} max={mx:.2e}", file=sys.stderr, flush=True)
    assert fro <= FRO[dt] and mx <= MAX[dt], (name, fro, mx)


CASES = [  # q lengths, k lengths, rows before and after, Hq, Hkv, D, window, sinks, causal, cap, bias
    dict(q=[1], k=[1], Hq=1, Hkv=1, D=64, w=1, s=1),
    dict(q=[64], k=[64], Hq=4, Hkv=4, D=64, w=16, s=2),
    dict(q=[40], k=[40], Hq=2, Hkv=1, D=128, w=1, s=0),                     # each row itself alone
    dict(q=[300], k=[300], Hq=4, Hkv=2, D=128, w=50, s=4),
    dict(q=[300], k=[300], Hq=2, Hkv=2, D=128, w=1, s=1, cap=3.0),
    dict(q=[33, 1, 0, 95, 60], k=[33, 1, 0, 95, 60], pad=(3, 9), Hq=4, Hkv=2, D=128, w=8, s=3),   # many sinks in one tile
    dict(q=[20] * 14, k=[20] * 14, Hq=2, Hkv=1, D=64, w=4, s=2, bias=True),
    dict(q=[129, 200], k=[129, 200], Hq=3, Hkv=3, D=104, w=64, s=40, cap=5.0),                    # two blocks of sinks
    dict(q=[500], k=[500], Hq=4, Hkv=1, D=40, w=100, s=128),                # more sinks than window
    dict(q=[140, 130], k=[140, 130], Hq=2, Hkv=1, D=64, w=30, s=100, causal=False),
    dict(q=[129], k=[129], Hq=2, Hkv=1, D=128, w=20, s=5, causal=False, bias=True),
    dict(q=[40, 20], k=[300, 7], Hq=4, Hkv=2, D=128, w=33, s=4, cap=3.0, bias=True),   # a prompt's chunk; rows that see nothing
    dict(q=[50, 8], k=[10, 90], Hq=2, Hkv=2, D=8, w=6, s=3, causal=False),  # rows whose window is empty see the sinks
    dict(q=[5, 200, 3, 47], k=[64, 200, 0, 1], pad=(0, 70), Hq=5, Hkv=5, D=72, w=40, s=2),
    dict(q=[257], k=[257], Hq=8, Hkv=1, D=64, w=1000, s=4),                 # a window past the document
    dict(q=[257, 100], k=[257, 100], Hq=2, Hkv=1, D=64, w=0, s=4),          # none
    dict(q=[200, 90], k=[200, 90], Hq=4, Hkv=2, D=128, w=60, s=0, bias=True, cap=30.0),
    dict(q=[20, 30, 90], k=[400, 300, 350], Hq=2, Hkv=1, D=64, w=40, s=5),  # chunks of several prompts in one tile
    # the loops are cut into parts and joined
    dict(q=[64, 3], k=[1500, 1100], Hq=2, Hkv=1, D=64, w=900, s=4),
    dict(q=[33], k=[2049], pad=(1, 2), Hq=4, Hkv=1, D=128, w=1500, s=7, cap=6.0, bias=True),
    dict(q=[1100], k=[1100], Hq=8, Hkv=1, D=128, w=700, s=33),
    # enough tiles to be sorted by cost
    dict(q=[900, 5, 1300], k=[900, 5, 1300], Hq=1, Hkv=1, D=64, w=130, s=4),
]


def setup(c, dt, seed=0, scale=1.5):
    rng = np.random.default_rng(seed + sum(c["q"]) + c["D"])
    a, b = c.get("pad", (0, 0))
    cu_q, cu_k = (np.concatenate([[0], np.cumsum(c[n])]).astype(np.int32) + a for n in "qk")
    Tq, Tk = int(cu_q[-1]) + b, int(cu_k[-1]) + b
    Hq, Hkv, D = c["Hq"], c["Hkv"], c["D"]
    return dict(q=normal(rng, (Tq, Hq, D), dt, scale), k=normal(rng, (Tk, Hkv, D), dt), v=normal(rng, (Tk, Hkv, D), dt),
                dout=normal(rng, (Tq, Hq, D), dt), cu_q=cu_q, cu_k=cu_k, window=c["w"], sinks=c["s"],
                slopes=(2.0 ** -np.arange(1, Hq + 1)).astype(np.float32) if c.get("bias") else None,
                causal=c.get("causal", True), cap=c.get("cap", 0.0), ndoc=len(c["q"]))


def run(st, stream=None):
    sh, w = P.attn_shape(st["q"], st["k"], st["v"], st["ndoc"], st["causal"], 0.0, st["cap"]), P.window(st["window"], st["sinks"])
    e = lambda t: torch.full(t.shape, 7.0, dtype=t.dtype, device="cuda")
    # what nothing writes is NaN, and so is all that is made of it
    raw = lambda n: torch.full((max(16, n),), 255, dtype=torch.uint8, device="cuda")
    plan = raw(P.poetx_attn_window_plan_bytes(sh, w))
    ws = [raw(P.poetx_attn_window_workspace_bytes(sh, w, i)) for i in (0, 1)]
    slopes = None if st["slopes"] is None else to_dev(st["slopes"])
    out = {"o": e(st["q"]), "dq": e(st["q"]), "dk": e(st["k"]), "dv": e(st["v"]),
           "lse": torch.full((sh.Hq, sh.Tq), 7.0, device="cuda")}
    P.poetx_attn_window_plan(sh, w, to_dev(st["cu_q"]), to_dev(st["cu_k"]), plan)
    P.poetx_attn_window_fwd(sh, w, st["q"], st["k"], st["v"], plan, out["o"], out["lse"], ws[0], slopes)
    P.poetx_attn_window_bwd(sh, w, st["dout"], st["q"], st["k"], st["v"], out["o"], out["lse"], plan, out["dq"], out["dk"],
                            out["dv"], ws[1], slopes)
    torch.cuda.synchronize()
    return out


def reference(st):
    w = st["window"] or 10 ** 9
    seen, pos = L.window_mask(st["q"].shape[0], st["k"].shape[0], st["cu_q"], st["cu_k"], w, st["sinks"], st["causal"])
    with np.errstate(invalid="ignore"):
        return B.attention(to_f64(st["q"]), to_f64(st["k"]), to_f64(st["v"]), seen, pos, None, st["cap"], st["slopes"],
                           to_f64(st["dout"])), seen


def compare(st, out, dt):
    ref, _ = reference(st)
    np.testing.assert_array_equal(np.isinf(to_f64(out["lse"])), np.isinf(ref["lse"]))
    fin = np.isfinite(ref["lse"])
    assert np.abs(to_f64(out["lse"])[fin] - ref["lse"][fin]).max(initial=0) <= 5e-5
    for n in ("o", "dq", "dk", "dv"):
        close(n, out[n], ref[n], dt)
    # the first keys by themselves: they are summed apart.  All documents' together: dk of one key may be a
    # difference dp - delta that cancels (a query that sees little else), and its error is that of the terms
    at = np.concatenate([np.arange(a, min(a + st["sinks"], b)) for a, b in zip(st["cu_k"][:-1], st["cu_k"][1:])]).astype(np.int64)
    if at.size:
        for n in ("dk", "dv"):
            close(f"{n} of the sinks", to_f64(out[n])[at], ref[n][at], dt)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("i", range(len(CASES)))
def test_window_attention(i, dt):
    st = setup(CASES[i], dt)
    compare(st, run(st), dt)


@pytest.mark.parametrize("dt", ["f32", "bf16"])
@pytest.mark.parametrize("what", ["k", "v", "q", "dout"])
def test_what_is_hidden_has_no_influence(what, dt):
    """NaN and infinity in rows of another document, in rows between the sinks
    and the window, and in queries that do not see a key."""
    c = dict(q=[200, 100, 60], k=[200, 100, 60], Hq=4, Hkv=2, D=64, w=24, s=3)
    st = setup(c, dt)
    st[what][210:214] = float("nan")   # of the second document, past its sinks
    st[what][330] = float("inf")       # of the third
    out = run(st)
    ref, seen = reference(st)
    touched = np.isin(np.arange(360), [*range(210, 214), 330])
    rows = seen[:, touched].any(1) if what in "kv" else touched          # queries with a bad operand
    keys = seen[rows].any(0) | (touched if what in "kv" else False)      # keys that they see
    for n, bad in (("o", rows if what != "dout" else np.zeros(360, bool)), ("dq", rows), ("dk", keys), ("dv", keys)):
        got = to_f64(out[n])[~bad]
        assert np.isfinite(got).all(), n
        close(f"{n} of rows that see none", got, ref[n][~bad], dt)


def test_window_past_the_rows_is_plain_attention():
    """The same kernels' arithmetic: no window, and one that hides nothing."""
    c = dict(q=[70, 130], k=[70, 130], Hq=4, Hkv=2, D=64, w=0, s=0)
    st = setup(c, "bf16")
    plain = run(st)
    for w in (130, 2 ** 31 - 1):
        st["window"] = w
        wide = run(st)
        for n in plain:
            np.testing.assert_array_equal(bits(plain[n]), bits(wide[n]))


@pytest.mark.parametrize("dt", ["f32", "bf16"])
def test_same_bits_on_another_stream_and_in_a_graph(dt):
    st = setup(dict(q=[500, 300], k=[500, 300], Hq=4, Hkv=2, D=128, w=90, s=4), dt)
    want = {n: bits(t) for n, t in run(st).items()}
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = run(st)
    for n, t in got.items():
        np.testing.assert_array_equal(bits(t), want[n])
    sh, w = P.attn_shape(st["q"], st["k"], st["v"], 2), P.window(90, 4)
    raw = lambda n: torch.empty(max(16, n), dtype=torch.uint8, device="cuda")
    plan, ws = raw(P.poetx_attn_window_plan_bytes(sh, w)), raw(P.poetx_attn_window_workspace_bytes(sh, w, 1))
    cu, out = to_dev(st["cu_q"]), {n: torch.empty_like(t) for n, t in got.items()}
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        P.poetx_attn_window_plan(sh, w, cu, cu, plan)
        P.poetx_attn_window_fwd(sh, w, st["q"], st["k"], st["v"], plan, out["o"], out["lse"], ws)
        P.poetx_attn_window_bwd(sh, w, st["dout"], st["q"], st["k"], st["v"], out["o"], out["lse"], plan, out["dq"],
                                out["dk"], out["dv"], ws)
    for i in range(3):
        for t in out.values():
            t.fill_(float("nan"))
        ws.fill_(255)
        plan.fill_(255)
        g.replay()
        torch.cuda.synchronize()
        for n, t in out.items():
            np.testing.assert_array_equal(bits(t), want[n], err_msg=f"replay {i} {n}")


def test_columns_of_one_projection_and_rows_behind():
    """q, k and v as column ranges; rows before and after the documents get
    zeros, and what lies between the columns of an output stays as it was."""
    T, Hq, Hkv, D = 150, 4, 2, 64
    rng = np.random.default_rng(5)
    fused = normal(rng, (T, (Hq + 2 * Hkv) * D), "bf16")
    grads = torch.full((T, (Hq + 2 * Hkv) * D + 16), 7.0, dtype=torch.bfloat16, device="cuda")
    cut = lambda t: [t[:, a * D:b * D].unflatten(1, (b - a, D)) for a, b in ((0, Hq), (Hq, Hq + Hkv), (Hq + Hkv, Hq + 2 * Hkv))]
    q, k, v = cut(fused)
    dq, dk, dv = cut(grads)
    cu = np.array([3, 100, 140], np.int32)
    st = dict(q=q.contiguous(), k=k.contiguous(), v=v.contiguous(), dout=normal(rng, (T, Hq, D), "bf16"), cu_q=cu, cu_k=cu,
              window=20, sinks=2, slopes=None, causal=True, cap=0.0, ndoc=2)
    want = run(st)
    compare(st, want, "bf16")
    sh, w = P.attn_shape(q, k, v, 2), P.window(20, 2)
    raw = lambda n: torch.empty(max(16, n), dtype=torch.uint8, device="cuda")
    plan, ws = raw(P.poetx_attn_window_plan_bytes(sh, w)), raw(P.poetx_attn_window_workspace_bytes(sh, w, 1))
    o, lse = torch.empty_like(st["q"]), torch.empty(Hq, T, device="cuda")
    P.poetx_attn_window_plan(sh, w, to_dev(cu), to_dev(cu), plan)
    P.poetx_attn_window_fwd(sh, w, q, k, v, plan, o, lse, ws)
    P.poetx_attn_window_bwd(sh, w, st["dout"], q, k, v, o, lse, plan, dq, dk, dv, ws)
    for n, t in (("o", o), ("dq", dq), ("dk", dk), ("dv", dv)):
        np.testing.assert_array_equal(bits(t.contiguous()), bits(want[n]))
        assert not t[:3].any() and not t[140:].any()
    assert (grads[:, -16:] == 7).all()


def test_many_short_documents():
    """More documents than are searched in LDS, windows within them."""
    rng = np.random.default_rng(6)
    lens = rng.integers(0, 5, 1500)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    T = int(cu[-1])
    st = dict(q=normal(rng, (T, 1, 64), "f32"), k=normal(rng, (T, 1, 64), "f32"), v=normal(rng, (T, 1, 64), "f32"),
              dout=normal(rng, (T, 1, 64), "f32"), cu_q=cu, cu_k=cu, window=2, sinks=1, slopes=None, causal=True, cap=0.0, ndoc=1500)
    compare(st, run(st), "f32")


def test_few_documents_among_many_have_sinks_apart():
    """Partial sums are numbered by documents, or by windows where those are
    fewer: here 202 documents, of which two pass the window."""
    lens = [3] * 100 + [400] + [1] * 60 + [350] + [2] * 40
    compare_lens(lens, 300, 3)


def test_a_short_window_under_one_document():
    compare_lens([700], 1, 20)


def compare_lens(lens, window, sinks):
    rng = np.random.default_rng(window)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    T = int(cu[-1])
    st = dict(q=normal(rng, (T, 2, 64), "bf16"), k=normal(rng, (T, 1, 64), "bf16"), v=normal(rng, (T, 1, 64), "bf16"),
              dout=normal(rng, (T, 2, 64), "bf16"), cu_q=cu, cu_k=cu, window=window, sinks=sinks, slopes=None, causal=True,
              cap=0.0, ndoc=len(lens))
    compare(st, run(st), "bf16")

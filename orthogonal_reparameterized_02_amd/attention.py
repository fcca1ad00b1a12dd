"""An attention block around POET-X projections.

`rope_table`, `apply_rope`, `qk_norm_rope`, `dropout_add`, `AttentionPlan` /
`attention` and `KVCache`, `KVCache4` / `attention_decode` are the library's
attention-block operators (include/poetx.h) with autograd and their workspaces;
`POETXAttention` puts them between four `POETXLinear` projections: packed
documents for training, single tokens over a cache for serving.  PyTorch supplies device memory,
streams and autograd only.  The gradients have no gradients of their own:
differentiating them raises.  Capture a backward pass into a graph only where
no eager autograd graph of the same parameters is alive: PyTorch's accumulation
then waits across streams, which a capture does not survive.
"""
from __future__ import annotations

import math
import operator
from typing import Optional, Sequence

import torch
from torch.autograd.function import once_differentiable

from . import poetx as P
from .layer import POETXLinear


def _bytes(n: int, device) -> torch.Tensor:
    return torch.empty(max(int(n), 16), dtype=torch.uint8, device=device)


# ---- rotary positions -----------------------------------------------------------
def rope_frequencies(rot: int, base: float = 10000.0, scaling: Optional[Sequence] = None) -> torch.Tensor:
    """Angle per position of the rot/2 pairs, float64: base^(-2 i / rot).
    scaling, for contexts longer than the trained one:
      ("linear", s)            every frequency / s (positions interpolated);
      ("base", s)              base * s^(rot / (rot - 2)): the slowest pair is
                               slowed by s, the fastest keeps its frequency;
      ("ramp", s, n, low, high) by how often a pair turns in the trained
                               length n: from `high` turns on unchanged, up
                               to `low` turns / s, linear in the turns between."""
    if rot < 2 or rot % 2:
        raise ValueError(f"rot={rot} must be even and at least 2")
    i = torch.arange(rot // 2, dtype=torch.float64)
    if scaling is None:
        return base ** (-2.0 * i / rot)
    kind, s = scaling[0], float(scaling[1])
    if not s > 0:
        raise ValueError(f"scaling factor {s} must be positive")
    if kind == "linear":
        return base ** (-2.0 * i / rot) / s
    if kind == "base":
        if rot < 4:
            raise ValueError("scaling the base needs rot >= 4")
        return (base * s ** (rot / (rot - 2))) ** (-2.0 * i / rot)
    if kind == "ramp":
        n, low, high = (float(v) for v in scaling[2:])
        if not 0 < low < high or not n > 0:
            raise ValueError(f"ramp needs 0 < low < high and a trained length, got {scaling}")
        f = base ** (-2.0 * i / rot)
        keep = ((n * f / (2 * math.pi) - low) / (high - low)).clamp(0.0, 1.0)
        return f * (keep + (1.0 - keep) / s)
    raise ValueError(f"unknown scaling {kind!r}")


def rope_table(positions: int, rot: int, base: float = 10000.0, scaling: Optional[Sequence] = None,
               magnitude: float = 1.0, device="cuda") -> torch.Tensor:
    """[positions][rot/2][2] float32 table of magnitude * (cos, sin),
    computed in float64."""
    a = torch.arange(positions, dtype=torch.float64)[:, None] * rope_frequencies(rot, base, scaling)
    return (torch.stack([a.cos(), a.sin()], -1) * magnitude).to(torch.float32).to(device)


class _Rope(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, pos, table, interleaved):
        qo = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        ko = None if k is None else torch.empty(k.shape, dtype=k.dtype, device=k.device)
        P.poetx_rope(q, k, pos, table, qo, ko, interleaved)
        ctx.save_for_backward(pos, table)
        ctx.interleaved = interleaved
        return (qo,) if k is None else (qo, ko)

    @staticmethod
    @once_differentiable
    def backward(ctx, *grads):
        pos, table = ctx.saved_tensors
        g = [x.contiguous() for x in grads]
        out = [torch.empty_like(x) for x in g] + [None] * (2 - len(g))
        P.poetx_rope(g[0], g[1] if len(g) > 1 else None, pos, table, out[0], out[1], ctx.interleaved, True)
        return out[0], out[1], None, None, None


def apply_rope(q: torch.Tensor, k: Optional[torch.Tensor], pos: torch.Tensor, table: torch.Tensor,
               interleaved: bool = False):
    """q [T][Hq][D] (and k [T][Hk][D]) turned by the angles of their
    positions; returns the pair, or q alone without k."""
    out = _Rope.apply(q, k, pos, table, interleaved)
    return out[0] if k is None else out


class _QkNormRope(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, wq, wk, pos, table, eps, interleaved):
        qo = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        ko = None if k is None else torch.empty(k.shape, dtype=k.dtype, device=k.device)
        P.poetx_qk_norm_rope_fwd(q, k, wq, wk, pos, table, qo, ko, eps, interleaved)
        ctx.save_for_backward(q, k, wq, wk, pos, table)
        ctx.args = (eps, interleaved)
        return (qo,) if k is None else (qo, ko)

    @staticmethod
    @once_differentiable
    def backward(ctx, *grads):
        q, k, wq, wk, pos, table = ctx.saved_tensors
        eps, interleaved = ctx.args
        new = lambda t, want=True: torch.empty(t.shape, dtype=t.dtype, device=t.device) if t is not None and want else None
        dq, dk = new(q), new(k)
        dwq, dwk = new(wq, ctx.needs_input_grad[2]), new(wk, ctx.needs_input_grad[3])
        ws = _bytes(P.poetx_qk_norm_rope_workspace_bytes(P.qk_norm_shape(q, k, table, eps, interleaved)), q.device)
        P.poetx_qk_norm_rope_bwd(grads[0].contiguous(), None if k is None else grads[1].contiguous(), q, k, wq, wk, pos, table,
                                 dq, dk, dwq, dwk, ws, eps, interleaved)
        return dq, dk, dwq, dwk, None, None, None, None


def qk_norm_rope(q: torch.Tensor, k: Optional[torch.Tensor], wq: Optional[torch.Tensor], wk: Optional[torch.Tensor],
                 pos: Optional[torch.Tensor], table: Optional[torch.Tensor], eps: float = 1e-6, interleaved: bool = False):
    """Root mean square norms of the heads of q [T][Hq][D] (and k [T][Hk][D])
    times wq, wk [D] float32 (None: 1), then apply_rope (table None: norms
    alone), in one pass; returns the pair, or q alone without k."""
    if k is None and wk is not None:
        raise ValueError("wk without k")
    out = _QkNormRope.apply(q, k, wq, wk, pos, table, eps, interleaved)
    return out[0] if k is None else out


# ---- dropout ------------------------------------------------------------------------
class _DropoutAdd(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, residual, p, seed, offset, offset_dev):
        x = x.contiguous()
        y = torch.empty_like(x)
        P.poetx_dropout_fwd(x, None if residual is None else residual.contiguous(), y, p, seed, offset, offset_dev)
        ctx.args = (p, seed, offset)
        ctx.residual = residual is not None
        ctx.save_for_backward(offset_dev)
        return y

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        p, seed, offset = ctx.args
        dx = None
        if ctx.needs_input_grad[0]:
            dy = dy.contiguous()
            dx = torch.empty_like(dy)
            P.poetx_dropout_bwd(dy, dx, p, seed, offset, ctx.saved_tensors[0])
        return dx, dy if ctx.residual else None, None, None, None, None


def dropout_add(x: torch.Tensor, residual: Optional[torch.Tensor], p: float, seed: int, offset: int = 0,
                offset_dev: Optional[torch.Tensor] = None) -> torch.Tensor:
    """residual + dropout(x); the mask is made again in the backward pass.
    offset_dev (int64 [1] on the GPU) adds to offset and must keep its value
    until the backward pass."""
    if residual is not None and (residual.shape != x.shape or residual.dtype != x.dtype):
        raise ValueError(f"residual is {tuple(residual.shape)} {residual.dtype}, x {tuple(x.shape)} {x.dtype}")
    return _DropoutAdd.apply(x, residual, p, seed, offset, offset_dev)


# ---- attention ------------------------------------------------------------------------
def _window(window: int, sinks: int):
    """A window and its sinks; sinks alone would have no meaning."""
    if window < 0 or sinks < 0 or (sinks and not window):
        raise ValueError(f"window={window} and sinks={sinks}: both at least 0, sinks with a window only")
    return window, sinks


class AttentionPlan:
    """The mask of one packed batch, shared by every layer, head and
    direction: document offsets cu_q (and cu_k where the keys have other
    lengths) as int32 GPU tensors, prefix lengths, causal or not; or, without
    prefixes, a window: keys less than `window` away, and the first `sinks` of
    the document from wherever they lie behind."""

    def __init__(self, cu_q: torch.Tensor, Tq: int, cu_k: Optional[torch.Tensor] = None,
                 Tk: Optional[int] = None, prefix: Optional[torch.Tensor] = None, causal: bool = True,
                 window: int = 0, sinks: int = 0):
        if (cu_k is None) != (Tk is None):
            raise ValueError("cu_k and Tk go together")
        if window and prefix is not None:
            raise ValueError("a window has no prefixes")
        self.window, self.sinks = _window(window, sinks)
        self.win = P.window(window, sinks) if window else None
        self.Tq, self.Tk = Tq, Tq if Tk is None else Tk
        self.ndoc, self.causal = cu_q.numel() - 1, causal
        if self.ndoc < 0 or (cu_k is not None and cu_k.numel() != cu_q.numel()):
            raise ValueError("cu_q and cu_k hold one offset more than there are documents")
        sh = self.shape(1, 1, 8, P.F32)
        cu_k = cu_q if cu_k is None else cu_k
        if self.win is None:
            self.data = _bytes(P.poetx_attn_plan_bytes(sh), cu_q.device)
            P.poetx_attn_plan(sh, cu_q, cu_k, self.data, prefix)
        else:
            self.data = _bytes(P.poetx_attn_window_plan_bytes(sh, self.win), cu_q.device)
            P.poetx_attn_window_plan(sh, self.win, cu_q, cu_k, self.data)

    def shape(self, Hq: int, Hkv: int, D: int, act: int, scale: float = 0.0, cap: float = 0.0) -> P.AttnShape:
        wq, wk = Hq * D, Hkv * D
        return P.AttnShape(self.Tq, self.Tk, self.ndoc, Hq, Hkv, D, act, int(self.causal), scale, cap,
                           wq, wk, wk, wq, wq, wq, wk, wk)


class _Attention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, plan, scale, cap, slopes):
        Hq, D, Hkv = q.shape[1], q.shape[2], k.shape[1]
        sh = plan.shape(Hq, Hkv, D, P.act_of(q.dtype), scale, cap)
        o = torch.empty(q.shape, dtype=q.dtype, device=q.device)
        lse = torch.empty(Hq, plan.Tq, dtype=torch.float32, device=q.device)
        if plan.win is None:
            ws = _bytes(P.poetx_attn_workspace_bytes(sh, 0), q.device)
            P.poetx_attn_fwd(sh, q, k, v, plan.data, o, lse, ws, slopes)
        else:
            ws = _bytes(P.poetx_attn_window_workspace_bytes(sh, plan.win, 0), q.device)
            P.poetx_attn_window_fwd(sh, plan.win, q, k, v, plan.data, o, lse, ws, slopes)
        ctx.save_for_backward(q, k, v, o, lse, slopes)
        ctx.plan, ctx.sh = plan, sh
        return o

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        q, k, v, o, lse, slopes = ctx.saved_tensors
        dq, dk, dv = (torch.empty(t.shape, dtype=t.dtype, device=t.device) for t in (q, k, v))
        sh, plan, dout = ctx.sh, ctx.plan, dout.contiguous()
        if plan.win is None:
            ws = _bytes(P.poetx_attn_workspace_bytes(sh, 1), q.device)
            P.poetx_attn_bwd(sh, dout, q, k, v, o, lse, plan.data, dq, dk, dv, ws, slopes)
        else:
            ws = _bytes(P.poetx_attn_window_workspace_bytes(sh, plan.win, 1), q.device)
            P.poetx_attn_window_bwd(sh, plan.win, dout, q, k, v, o, lse, plan.data, dq, dk, dv, ws, slopes)
        return dq, dk, dv, None, None, None, None


def attention(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, plan: AttentionPlan, scale: float = 0.0,
              cap: float = 0.0, slopes: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Attention of q [Tq][Hq][D] over k, v [Tk][Hkv][D] of a packed batch.
    scale 0: 1 / sqrt(D); cap: scores cap * tanh(score / cap); slopes [Hq]
    float32: a bias of -slope * |distance|, constants without a gradient.
    q, k and v may be column ranges of one wider projection."""
    if slopes is not None and slopes.requires_grad:
        raise ValueError("slopes are constants: they get no gradient")
    return _Attention.apply(q, k, v, plan, scale, cap, slopes)


def alibi_slopes(heads: int, device="cuda") -> torch.Tensor:
    """Slopes 2^(-8 (h + 1) / heads): a geometric series over the heads."""
    h = torch.arange(1, heads + 1, dtype=torch.float64)
    return (2.0 ** (-8.0 * h / heads)).to(torch.float32).to(device)


# ---- single tokens over a cache -----------------------------------------------------------
class KVCache:
    """Keys and values of B sequences, up to `rows` tokens each.  An idle slot
    counts tokens like the others; fill it with none of them to empty it, before
    it is full or at the end of a block's rotary table.

    With a window the cache is a ring: it keeps the first `sinks` tokens of a
    sequence and the rows - sinks (at least `window`) newest ones, and is never
    full (a block's rotary table still ends); its queries see the last `window`
    tokens and the sinks.

    append refuses a full cache from a count on the host.  A replayed graph
    appends without the host: there a sequence without room keeps its rows and
    its length, and from the first captured call on the count is read from the
    GPU."""

    def __init__(self, B: int, rows: int, Hkv: int, D: int, dtype=torch.bfloat16, device="cuda", window: int = 0,
                 sinks: int = 0):
        self.B, self.rows, self.Hkv, self.D, self.dtype = B, rows, Hkv, D, dtype
        self.window, self.sinks = _window(window, sinks)
        self.ring = window > 0
        if self.ring and rows < window + sinks:
            raise ValueError(f"{rows} rows do not hold a window of {window} and {sinks} sinks")
        self._storage(device)
        self.length = torch.zeros(B, dtype=torch.int32, device=device)
        # the same on the host, so that no token waits for the GPU: each length less the tokens appended
        # to all, and the largest of them.  None: replays may have changed it
        self._filled: Optional[list] = [0] * B
        self._most, self._appended = 0, 0
        self._at = torch.arange(B, device=device)

    # -- where rows lie: what a cache of another form has of its own ------------------
    def _storage(self, device) -> None:
        self.k = torch.empty(self.B, self.rows, self.Hkv, self.D, dtype=self.dtype, device=device)
        self.v = torch.empty_like(self.k)

    def _row(self, pos: torch.Tensor) -> torch.Tensor:
        """Rows of positions."""
        pos = pos.long()
        if not self.ring:
            return pos
        return torch.where(pos < self.sinks, pos, self.sinks + (pos - self.sinks) % (self.rows - self.sinks))

    def _positions(self, spans) -> torch.Tensor:
        """Ranges of positions as one int32 tensor."""
        return torch.cat([torch.arange(a, b, dtype=torch.int32, device=self.length.device) for a, b in spans])

    def _write(self, b: int, spans, k: torch.Tensor, v: torch.Tensor) -> None:
        """k, v to the positions of spans, a list of ranges."""
        rows = self._row(self._positions(spans)) if self.ring else slice(*spans[0])
        self.k[b, rows], self.v[b, rows] = k, v

    def _read(self, b: int, spans):
        rows = self._row(self._positions(spans))
        return self.k[b, rows], self.v[b, rows]

    def _next(self, k: torch.Tensor, v: torch.Tensor) -> None:
        """Every sequence's token at its length."""
        at = self._row(self.length)
        self.k[self._at, at], self.v[self._at, at] = k, v

    def _next_where_room(self, k: torch.Tensor, v: torch.Tensor) -> None:
        """The same for a graph: what a replay finds full is written back as it
        was, so no replay writes outside the cache."""
        at, full = self.length.clamp(0, self.rows - 1).long(), (self.length >= self.rows)[:, None, None]
        for rows, new in ((self.k, k), (self.v, v)):
            rows[self._at, at] = torch.where(full, rows[self._at, at], new)

    def _decode(self, q, o, scale, cap, slopes, start, win) -> None:
        sh = P.decode_shape(q, self.k, self.v, scale, cap)
        if win is None:
            ws = _bytes(P.poetx_attn_decode_workspace_bytes(sh), q.device)
            P.poetx_attn_decode(sh, q, self.k, self.v, self.length, o, ws, start, slopes)
        else:
            ws = _bytes(P.poetx_attn_window_decode_workspace_bytes(sh, win), q.device)
            P.poetx_attn_window_decode(sh, win, q, self.k, self.v, self.length, o, ws, slopes, self.ring)

    # -- tokens ---------------------------------------------------------------------------
    def _captured(self) -> bool:
        return self.length.is_cuda and torch.cuda.is_current_stream_capturing()

    def longest(self) -> Optional[int]:
        """Tokens of the longest sequence; None while a graph is captured."""
        if self._captured():
            return None
        if self._filled is None or self.B == 0:
            return max(self.length.tolist(), default=0)
        return self._most + self._appended

    def _sequence(self, b: int) -> int:
        """b counted from the front: below 0 it counts from the end."""
        b = operator.index(b)
        if not -self.B <= b < self.B:
            raise IndexError(f"sequence {b} of a cache of {self.B}")
        return b % self.B

    def tokens(self, b: int) -> int:
        """Tokens of sequence b (also those that a ring no longer holds)."""
        b = self._sequence(b)
        if self._captured():  # a replay would take the count of now
            raise RuntimeError("the tokens of a sequence are not known while a graph is captured")
        return int(self.length[b]) if self._filled is None else self._filled[b] + self._appended

    def held(self, b: int):
        """k, v [n][Hkv][D] of sequence b: every token in order, or of a ring
        the sinks and the newest ones."""
        return self._read(self._sequence(b), self._held(self.tokens(b)))

    def _held(self, n: int, at: int = 0):
        """The positions from `at` on that n tokens leave in the cache, as
        ranges: all, or of a ring the sinks' and the newest."""
        if not self.ring or n <= self.rows:
            return [(at, n)]
        return [(min(at, self.sinks), self.sinks), (max(at, n - (self.rows - self.sinks)), n)]

    def fill(self, b: int, k: torch.Tensor, v: torch.Tensor) -> None:
        """Sequence b becomes k, v [n][Hkv][D] (a prompt's)."""
        self._put(b, 0, k, v)

    def extend(self, b: int, k: torch.Tensor, v: torch.Tensor) -> None:
        """n tokens k, v [n][Hkv][D] more for sequence b (a prompt's later part)."""
        self._put(b, self.tokens(b), k, v)

    def _put(self, b: int, at: int, k: torch.Tensor, v: torch.Tensor) -> None:
        b, n = self._sequence(b), at + k.shape[0]
        if not self.ring and n > self.rows:
            raise ValueError(f"{n} tokens do not fit a cache of {self.rows} rows")
        if k.shape[0]:
            spans = self._held(n, at)
            if len(spans) > 1:  # a ring that these tokens go round
                k, v = (torch.cat([t[x - at:y - at] for x, y in spans]) for t in (k, v))
            self._write(b, spans, k, v)
        self.length[b] = n
        if self._captured():
            self._filled = None
        elif self._filled is not None:
            self._filled[b] = n - self._appended
            self._most = max(self._filled)

    def append(self, k: torch.Tensor, v: torch.Tensor) -> None:
        """One token more for every sequence: k, v [B][Hkv][D]."""
        n = self.longest()
        if self.rows == 0 or (not self.ring and n is not None and n >= self.rows):
            raise ValueError(f"the cache is full ({self.rows} rows)")
        if n is None:
            self._filled = None
        if n is not None or self.ring:
            self._next(k, v)
            self.length += 1
            self._appended += n is not None
        else:
            self._next_where_room(k, v)
            self.length.add_(1).clamp_(max=self.rows)


class KVCache4(KVCache):
    """The same in 4 bits: keys and values are held in blocks of 32 elements of
    a head (include/poetx.h, poetx_kv4_write), 17 bytes a block.  rows is rounded
    up to a multiple of 64.  On a GPU only."""

    def __init__(self, B: int, rows: int, Hkv: int, D: int, dtype=torch.bfloat16, device="cuda", window: int = 0,
                 sinks: int = 0):
        super().__init__(B, (rows + 63) // 64 * 64, Hkv, D, dtype, device, window, sinks)

    def _storage(self, device) -> None:
        nb = P.kv4_blocks(self.D)
        new = lambda *s: torch.empty(*s, dtype=torch.uint8, device=device)
        self.kc, self.ks = new(self.B, self.Hkv, self.rows, nb * 16), new(self.B, self.Hkv, nb, self.rows)
        self.vc, self.vs = torch.empty_like(self.kc), torch.empty_like(self.ks)

    @property
    def _cache(self):
        return self.kc, self.ks, self.vc, self.vs

    def _write(self, b, spans, k, v) -> None:
        pos = self._positions(spans)
        P.poetx_kv4_write(k, v, torch.full_like(pos, b), pos, *self._cache, sinks=self.sinks, ring=self.ring)

    def _read(self, b, spans):
        pos = self._positions(spans)
        k = torch.empty(pos.numel(), self.Hkv, self.D, dtype=self.dtype, device=pos.device)
        v = torch.empty_like(k)
        P.poetx_kv4_read(torch.full_like(pos, b), pos, *self._cache, k, v, sinks=self.sinks, ring=self.ring)
        return k, v

    def append(self, k: torch.Tensor, v: torch.Tensor) -> None:
        # the kernel writes the tokens that there are: fewer would leave sequences without theirs
        if k.shape[0] != self.B or v.shape[0] != self.B:
            raise ValueError(f"tokens of {k.shape[0]} and {v.shape[0]} sequences for a cache of {self.B} sequences")
        super().append(k, v)

    def _next(self, k, v) -> None:
        P.poetx_kv4_write(k, v, None, self.length, *self._cache, sinks=self.sinks, ring=self.ring)

    _next_where_room = _next  # a position past the last row writes nothing

    def _decode(self, q, o, scale, cap, slopes, start, win) -> None:
        sh, win = P.kv4_decode_shape(q, self.kc, scale, cap), win or P.window(0)
        ws = _bytes(P.poetx_attn_kv4_decode_workspace_bytes(sh, win), q.device)
        P.poetx_attn_kv4_decode(sh, win, q, *self._cache, self.length, o, ws, start, slopes, self.ring)


def attention_decode(q: torch.Tensor, cache: KVCache, scale: float = 0.0, cap: float = 0.0,
                     slopes: Optional[torch.Tensor] = None, start: Optional[torch.Tensor] = None, window: int = 0,
                     sinks: int = 0) -> torch.Tensor:
    """One query per sequence, q [B][Hq][D], over the cache's rows
    [start[b], length[b]); or over the last `window` tokens and the first
    `sinks` (a ring's own, unless given)."""
    window, sinks = _window(window, sinks)
    if cache.ring:
        if (window or sinks) and (window, sinks) != (cache.window, cache.sinks):
            raise ValueError(f"a ring of window={cache.window} and sinks={cache.sinks}, called with {window} and {sinks}")
        window, sinks = cache.window, cache.sinks
    if window and start is not None:
        raise ValueError("start with a window")
    o = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    cache._decode(q, o, scale, cap, slopes, start, P.window(window, sinks) if window else None)
    return o


# ---- the block ---------------------------------------------------------------------------------
class POETXAttention(torch.nn.Module):
    """x + dropout(Wo attention(rope(Wq x), rope(Wk x), Wv x)) with POET-X
    projections of block size b and Neumann order k.
    qk_norm: the heads of Wq x and Wk x are normed before they turn, with
    weights of their own (q_norm, k_norm).  window, sinks: a token sees the last
    `window` ones and the first `sinks` of its document.

    forward(x, plan, pos, at): x [T][n] packed tokens, plan their AttentionPlan
    (self.plan makes one with the block's window), pos [T] int32 positions (of each token in its document; one outside the
    table gives NaN), at the place of the dropout mask (draw; by default the
    next one, which a recomputed pass could not find again).  prefill and
    decode serve: no dropout, no gradients, and no token past the table's
    `positions`, over a ring as over any cache."""

    def __init__(self, n: int, heads: int, kv_heads: int, b: int, k: int, head_dim: Optional[int] = None,
                 positions: int = 8192, rot: Optional[int] = None, base: float = 10000.0, scaling=None,
                 interleaved: bool = False, cap: float = 0.0, bias: bool = False, dropout: float = 0.0,
                 dtype=torch.bfloat16, seed: int = 0, device="cuda", qk_norm: bool = False, eps: float = 1e-6,
                 window: int = 0, sinks: int = 0):
        super().__init__()
        self.window, self.sinks = _window(window, sinks)
        self.eps = eps
        self.n, self.Hq, self.Hkv = n, heads, kv_heads
        self.D = head_dim or n // heads
        self.cap, self.p, self.interleaved, self.dtype = cap, dropout, interleaved, dtype
        lin = lambda i, o, s: POETXLinear(i, o, b, k, dtype=dtype, seed=seed * 8 + s, device=device)
        self.q, self.k = lin(n, heads * self.D, 0), lin(n, kv_heads * self.D, 1)
        self.v, self.o = lin(n, kv_heads * self.D, 2), lin(heads * self.D, n, 3)
        self.register_buffer("table", rope_table(positions, rot or self.D, base, scaling, device=device))
        self.register_buffer("slopes", alibi_slopes(heads, device) if bias else None)
        one = lambda: torch.nn.Parameter(torch.ones(self.D, device=device)) if qk_norm else None
        self.q_norm, self.k_norm = one(), one()
        # place in the mask's sequence, on the GPU: a captured step moves on too
        self.seed = seed
        self.register_buffer("drawn", torch.zeros(1, dtype=torch.int64, device=device))

    def _heads(self, x, pos):
        T = x.shape[0]
        q, k = self.q(x).view(T, self.Hq, self.D), self.k(x).view(T, self.Hkv, self.D)
        if self.q_norm is None:
            q, k = apply_rope(q, k, pos, self.table, self.interleaved)
        else:
            q, k = qk_norm_rope(q, k, self.q_norm, self.k_norm, pos, self.table, self.eps, self.interleaved)
        return q, k, self.v(x).view(T, self.Hkv, self.D)

    def plan(self, cu_q: torch.Tensor, Tq: int, cu_k: Optional[torch.Tensor] = None, Tk: Optional[int] = None) -> AttentionPlan:
        """The AttentionPlan of a packed batch under the block's window."""
        return AttentionPlan(cu_q, Tq, cu_k, Tk, window=self.window, sinks=self.sinks)

    def cache(self, B: int, rows: int, four_bits: bool = False) -> KVCache:
        """A cache for B sequences of up to `rows` tokens, in the block's type
        or held in 4 bits; a ring where the window and sinks are fewer."""
        form, need = KVCache4 if four_bits else KVCache, self.window + self.sinks
        if self.window and need < rows:
            return form(B, need, self.Hkv, self.D, self.dtype, self.table.device, self.window, self.sinks)
        return form(B, rows, self.Hkv, self.D, self.dtype, self.table.device)

    def _check_positions(self, n: int) -> None:
        if n > self.table.shape[0]:
            raise ValueError(f"{n} tokens, the rotary table has {self.table.shape[0]} positions")

    def draw(self, tokens: int) -> torch.Tensor:
        """The place of the next `tokens` tokens' mask in the seed's sequence
        ([1] int64 on the GPU), which moves on past it.  For a forward pass
        that will be recomputed:
            checkpoint(block, x, plan, pos, block.draw(x.shape[0]))"""
        at = self.drawn.clone()
        self.drawn += (tokens * self.n + 7) // 8 * 8
        return at

    def forward(self, x: torch.Tensor, plan: AttentionPlan, pos: torch.Tensor,
                at: Optional[torch.Tensor] = None) -> torch.Tensor:
        if (plan.window, plan.sinks) != (self.window, self.sinks):
            raise ValueError(f"a plan of window={plan.window} and sinks={plan.sinks} for a block of {self.window} and {self.sinks}")
        q, k, v = self._heads(x, pos)
        y = self.o(attention(q, k, v, plan, cap=self.cap, slopes=self.slopes).view(x.shape[0], -1))
        if not (self.training and self.p > 0):
            return x + y
        if at is None:
            # inside a backward pass: the sequence has moved on since the loss was formed
            if torch._C._current_graph_task_id() != -1:
                raise RuntimeError("a forward pass recomputed for the backward pass needs the place of its dropout "
                                   "mask: pass at=block.draw(tokens) (see POETXAttention.draw)")
            at = self.draw(x.shape[0])
        return dropout_add(y, x, self.p, self.seed, 0, at)

    @torch.no_grad()
    def prefill(self, x: torch.Tensor, cache: KVCache, b: int = 0, follow: bool = False) -> torch.Tensor:
        """A prompt x [n tokens][n] of sequence b from position 0; fills its
        cache rows.  follow: a later part of one, behind the tokens that the
        cache has of the sequence, all of which it reads from there."""
        T, at = x.shape[0], cache.tokens(b) if follow else 0
        self._check_cache(cache)
        self._check_positions(at + T)
        pos = torch.arange(at, at + T, dtype=torch.int32, device=x.device)
        q, k, v = self._heads(x, pos)
        cu = lambda n: torch.tensor([0, n], dtype=torch.int32, device=x.device)
        if at == 0:
            cache.fill(b, k, v)
            plan = self.plan(cu(T), T)
        else:
            # a ring's newest rows stand right behind its sinks here: the mask is
            # the same, for it counts from the ends, a bias is not
            if self.slopes is not None and cache.ring and at > cache.rows:
                raise ValueError("a later part of a prompt over a ring that has dropped tokens has no distances for a bias")
            if not cache.ring and at + T > cache.rows:
                raise ValueError(f"{at + T} tokens do not fit a cache of {cache.rows} rows")
            before = cache.held(b)
            cache.extend(b, k, v)
            k, v = torch.cat([before[0], k]), torch.cat([before[1], v])
            plan = self.plan(cu(T), T, cu(k.shape[0]), k.shape[0])
        return x + self.o(attention(q, k, v, plan, cap=self.cap, slopes=self.slopes).view(T, -1))

    def _check_cache(self, cache: KVCache) -> None:
        if cache.ring and (cache.window, cache.sinks) != (self.window, self.sinks):
            raise ValueError(f"a ring of window={cache.window} and sinks={cache.sinks} for a block of {self.window} and {self.sinks}")

    @torch.no_grad()
    def decode(self, x: torch.Tensor, cache: KVCache) -> torch.Tensor:
        """The next token of every sequence, x [B][n].  In a captured graph a
        sequence without room for it, or without a position in the rotary
        table, answers NaN (and so does a ring from then on: such a token's key
        is NaN in it until the sequence is filled again)."""
        self._check_cache(cache)
        n = cache.longest()
        full = cache.length >= cache.rows if n is None and not cache.ring else None
        if n is not None:
            self._check_positions(n + 1)
        q, k, v = self._heads(x, cache.length)
        cache.append(k, v)
        o = attention_decode(q, cache, cap=self.cap, slopes=self.slopes, window=self.window, sinks=self.sinks)
        if full is not None:
            o.masked_fill_(full[:, None, None], math.nan)
        return x + self.o(o.view(x.shape[0], -1))

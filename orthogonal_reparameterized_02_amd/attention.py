"""An attention block around POET-X projections.

`rope_table`, `apply_rope`, `dropout_add`, `AttentionPlan` / `attention` and
`KVCache` / `attention_decode` are the library's attention-block operators
(include/poetx.h) with autograd and their workspaces; `POETXAttention` puts
them between four `POETXLinear` projections: packed documents for training,
single tokens over a cache for serving.  PyTorch supplies device memory,
streams and autograd only.  The gradients have no gradients of their own:
differentiating them raises.
"""
from __future__ import annotations

import math
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
class AttentionPlan:
    """The mask of one packed batch, shared by every layer, head and
    direction: document offsets cu_q (and cu_k where the keys have other
    lengths) as int32 GPU tensors, prefix lengths, causal or not."""

    def __init__(self, cu_q: torch.Tensor, Tq: int, cu_k: Optional[torch.Tensor] = None,
                 Tk: Optional[int] = None, prefix: Optional[torch.Tensor] = None, causal: bool = True):
        if (cu_k is None) != (Tk is None):
            raise ValueError("cu_k and Tk go together")
        self.Tq, self.Tk = Tq, Tq if Tk is None else Tk
        self.ndoc, self.causal = cu_q.numel() - 1, causal
        if self.ndoc < 0 or (cu_k is not None and cu_k.numel() != cu_q.numel()):
            raise ValueError("cu_q and cu_k hold one offset more than there are documents")
        sh = self.shape(1, 1, 8, P.F32)
        self.data = _bytes(P.poetx_attn_plan_bytes(sh), cu_q.device)
        P.poetx_attn_plan(sh, cu_q, cu_q if cu_k is None else cu_k, self.data, prefix)

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
        ws = _bytes(P.poetx_attn_workspace_bytes(sh, 0), q.device)
        P.poetx_attn_fwd(sh, q, k, v, plan.data, o, lse, ws, slopes)
        ctx.save_for_backward(q, k, v, o, lse, slopes)
        ctx.plan, ctx.sh = plan, sh
        return o

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        q, k, v, o, lse, slopes = ctx.saved_tensors
        dq, dk, dv = (torch.empty(t.shape, dtype=t.dtype, device=t.device) for t in (q, k, v))
        ws = _bytes(P.poetx_attn_workspace_bytes(ctx.sh, 1), q.device)
        P.poetx_attn_bwd(ctx.sh, dout.contiguous(), q, k, v, o, lse, ctx.plan.data, dq, dk, dv, ws, slopes)
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
    counts tokens like the others; fill it with none of them to empty it.

    append refuses a full cache from a count on the host.  A replayed graph
    appends without the host: there a sequence without room keeps its rows and
    its length, and from the first captured call on the count is read from the
    GPU."""

    def __init__(self, B: int, rows: int, Hkv: int, D: int, dtype=torch.bfloat16, device="cuda"):
        self.k = torch.empty(B, rows, Hkv, D, dtype=dtype, device=device)
        self.v = torch.empty_like(self.k)
        self.length = torch.zeros(B, dtype=torch.int32, device=device)
        self.B, self.rows = B, rows
        # the same on the host, so that no token waits for the GPU: each length less the tokens appended
        # to all, and the largest of them.  None: replays may have changed it
        self._filled: Optional[list] = [0] * B
        self._most, self._appended = 0, 0
        self._at = torch.arange(B, device=device)

    def _captured(self) -> bool:
        return self.k.is_cuda and torch.cuda.is_current_stream_capturing()

    def longest(self) -> Optional[int]:
        """Tokens of the longest sequence; None while a graph is captured."""
        if self._captured():
            return None
        if self._filled is None or self.B == 0:
            return max(self.length.tolist(), default=0)
        return self._most + self._appended

    def fill(self, b: int, k: torch.Tensor, v: torch.Tensor) -> None:
        """Sequence b becomes k, v [n][Hkv][D] (a prompt's)."""
        n = k.shape[0]
        if n > self.rows:
            raise ValueError(f"{n} tokens do not fit a cache of {self.rows} rows")
        self.k[b, :n], self.v[b, :n] = k, v
        self.length[b] = n
        if self._captured():
            self._filled = None
        elif self._filled is not None:
            self._filled[b] = n - self._appended
            self._most = max(self._filled)

    def append(self, k: torch.Tensor, v: torch.Tensor) -> None:
        """One token more for every sequence: k, v [B][Hkv][D]."""
        n = self.longest()
        if self.rows == 0 or (n is not None and n >= self.rows):
            raise ValueError(f"the cache is full ({self.rows} rows)")
        if n is None:
            self._append_where_room(k, v)
            return
        at = self.length.long()
        self.k[self._at, at], self.v[self._at, at] = k, v
        self.length += 1
        self._appended += 1

    def _append_where_room(self, k: torch.Tensor, v: torch.Tensor) -> None:
        """append for a graph: what a replay finds full is written back as it
        was, so no replay writes outside the cache."""
        self._filled = None
        at, full = self.length.clamp(0, self.rows - 1).long(), (self.length >= self.rows)[:, None, None]
        for rows, new in ((self.k, k), (self.v, v)):
            rows[self._at, at] = torch.where(full, rows[self._at, at], new)
        self.length.add_(1).clamp_(max=self.rows)


def attention_decode(q: torch.Tensor, cache: KVCache, scale: float = 0.0, cap: float = 0.0,
                     slopes: Optional[torch.Tensor] = None, start: Optional[torch.Tensor] = None) -> torch.Tensor:
    """One query per sequence, q [B][Hq][D], over the cache's rows
    [start[b], length[b])."""
    sh = P.decode_shape(q, cache.k, cache.v, scale, cap)
    ws = _bytes(P.poetx_attn_decode_workspace_bytes(sh), q.device)
    o = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    P.poetx_attn_decode(sh, q, cache.k, cache.v, cache.length, o, ws, start, slopes)
    return o


# ---- the block ---------------------------------------------------------------------------------
class POETXAttention(torch.nn.Module):
    """x + dropout(Wo attention(rope(Wq x), rope(Wk x), Wv x)) with POET-X
    projections of block size b and Neumann order k.

    forward(x, plan, pos, at): x [T][n] packed tokens, plan their AttentionPlan,
    pos [T] int32 positions (of each token in its document; one outside the
    table gives NaN), at the place of the dropout mask (draw; by default the
    next one, which a recomputed pass could not find again).  prefill and
    decode serve: no dropout, no gradients, and no token past the table."""

    def __init__(self, n: int, heads: int, kv_heads: int, b: int, k: int, head_dim: Optional[int] = None,
                 positions: int = 8192, rot: Optional[int] = None, base: float = 10000.0, scaling=None,
                 interleaved: bool = False, cap: float = 0.0, bias: bool = False, dropout: float = 0.0,
                 dtype=torch.bfloat16, seed: int = 0, device="cuda"):
        super().__init__()
        self.n, self.Hq, self.Hkv = n, heads, kv_heads
        self.D = head_dim or n // heads
        self.cap, self.p, self.interleaved, self.dtype = cap, dropout, interleaved, dtype
        lin = lambda i, o, s: POETXLinear(i, o, b, k, dtype=dtype, seed=seed * 8 + s, device=device)
        self.q, self.k = lin(n, heads * self.D, 0), lin(n, kv_heads * self.D, 1)
        self.v, self.o = lin(n, kv_heads * self.D, 2), lin(heads * self.D, n, 3)
        self.register_buffer("table", rope_table(positions, rot or self.D, base, scaling, device=device))
        self.register_buffer("slopes", alibi_slopes(heads, device) if bias else None)
        # place in the mask's sequence, on the GPU: a captured step moves on too
        self.seed = seed
        self.register_buffer("drawn", torch.zeros(1, dtype=torch.int64, device=device))

    def _heads(self, x, pos):
        T = x.shape[0]
        q, k = self.q(x).view(T, self.Hq, self.D), self.k(x).view(T, self.Hkv, self.D)
        q, k = apply_rope(q, k, pos, self.table, self.interleaved)
        return q, k, self.v(x).view(T, self.Hkv, self.D)

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
    def prefill(self, x: torch.Tensor, cache: KVCache, b: int = 0) -> torch.Tensor:
        """A prompt x [n tokens][n] of sequence b from position 0; fills its
        cache rows."""
        T = x.shape[0]
        self._check_positions(T)
        pos = torch.arange(T, dtype=torch.int32, device=x.device)
        q, k, v = self._heads(x, pos)
        cache.fill(b, k, v)
        plan = AttentionPlan(torch.tensor([0, T], dtype=torch.int32, device=x.device), T)
        return x + self.o(attention(q, k, v, plan, cap=self.cap, slopes=self.slopes).view(T, -1))

    @torch.no_grad()
    def decode(self, x: torch.Tensor, cache: KVCache) -> torch.Tensor:
        """The next token of every sequence, x [B][n].  In a captured graph a
        sequence without room for it, or without a position in the rotary
        table, answers NaN."""
        n = cache.longest()
        full = cache.length >= cache.rows if n is None else None
        if n is not None:
            self._check_positions(n + 1)
        q, k, v = self._heads(x, cache.length)
        cache.append(k, v)
        o = attention_decode(q, cache, cap=self.cap, slopes=self.slopes)
        if full is not None:
            o.masked_fill_(full[:, None, None], math.nan)
        return x + self.o(o.view(x.shape[0], -1))

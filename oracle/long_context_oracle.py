"""Float64 oracle of the long-context operators of an attention block: norms of
queries and keys with rotary positions, attention with a window and sinks, a
cache in blocks of 4-bit numbers.  Plain NumPy from the formulas, test
infrastructure only; attention itself is block_oracle's, under these masks."""
import numpy as np

from . import block_oracle as B


# ---- norms of queries and keys, with rotary positions --------------------------
def qk_norm(x, w, pos, table, eps, interleaved=False):
    """x [T][H][D]; w [D] or None; table None: not turned."""
    x = np.asarray(x, np.float64)
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    if w is not None:
        y = y * np.asarray(w, np.float64)
    return y if table is None else B.rope(y, pos, table, interleaved)


def qk_norm_grad(x, w, pos, table, eps, dy, interleaved=False):
    """(dx, dw, and what rounding scales with: |terms| of dx, sum |terms| of dw)."""
    x, g = np.asarray(x, np.float64), np.asarray(dy, np.float64)
    if table is not None:
        g = B.rope(g, pos, table, interleaved, inverse=True)
    D = x.shape[-1]
    s = np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    u = g if w is None else g * np.asarray(w, np.float64)
    along = (u * x).sum(-1, keepdims=True) / (D * s ** 3)
    size = np.abs(u) / s + np.abs(x) * np.abs(u * x).sum(-1, keepdims=True) / (D * s ** 3)
    return u / s - x * along, (g * x / s).sum((0, 1)), size, np.abs(g * x / s).sum((0, 1))


# ---- a window and sinks --------------------------------------------------------------
def window_mask(Tq, Tk, cu_q, cu_k, window, sinks, causal=True):
    """(seen [Tq][Tk], position [Tq]): pair by pair from the definition."""
    seen, pos = B.mask(Tq, Tk, cu_q, cu_k, None, causal)
    for d in range(len(cu_q) - 1):
        for i in range(cu_q[d], cu_q[d + 1]):
            for j in range(cu_k[d], cu_k[d + 1]):
                if abs(pos[i] - j) >= window and j - cu_k[d] >= sinks:
                    seen[i, j] = False
    return seen, pos


def ring_row(p, sinks, rows):
    """Row of position p in a ring of `rows` rows."""
    return p if p < sinks else sinks + (p - sinks) % (rows - sinks)


def window_decode(q, k, v, length, window, sinks, ring=False, scale=None, cap=0.0, slopes=None):
    """q [B][Hq][D], caches [B][rows][Hkv][D]: the rows of the positions seen,
    in the order of the positions."""
    o = np.zeros(q.shape)
    rows = k.shape[1]
    for b in range(q.shape[0]):
        L = max(int(length[b]), 0) if ring else min(max(int(length[b]), 0), rows)
        ps = [p for p in range(L) if not window or p >= L - window or p < sinks]
        if not ps:
            continue
        at = [ring_row(p, sinks, rows) if ring else p for p in ps]
        kk, vv = np.zeros((L,) + k.shape[2:]), np.zeros((L,) + v.shape[2:])
        kk[ps], vv[ps] = k[b, at], v[b, at]
        seen = np.zeros((1, L), bool)
        seen[0, ps] = True
        o[b] = B.attention(q[b:b + 1], kk, vv, seen, np.array([L - 1]), scale, cap, slopes)["o"][0]
    return o


# ---- a cache in 4 bits -------------------------------------------------------------------
GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def kv4_encode(x):
    """x [..., D] -> codes [..., 16 blocks] (element 2i in the low half of byte
    i), scale bytes [..., blocks]; element by element."""
    x = np.asarray(x, np.float64)
    D, nb = x.shape[-1], (x.shape[-1] + 31) // 32
    flat = np.zeros((x.size // max(D, 1), nb * 32))
    flat[:, :D] = x.reshape(-1, D)
    codes, scales = np.zeros((flat.shape[0], nb * 16), np.uint8), np.zeros((flat.shape[0], nb), np.uint8)
    for r in range(flat.shape[0]):
        for b in range(nb):
            blk = flat[r, 32 * b:32 * b + 32]
            if not np.isfinite(blk).all():
                scales[r, b] = 255
                continue
            e = -127
            while e < 125 and np.abs(blk).max() >= 7 * 2.0 ** e:
                e += 1
            scales[r, b] = e + 127
            for i, val in enumerate(blk):
                a = min(abs(val) / 2.0 ** e, 6.0)
                # nearest; of two as near the even code
                c = min(range(8), key=lambda n: (abs(GRID[n] - a), n % 2))
                codes[r, 16 * b + i // 2] |= (c | (8 if np.signbit(val) else 0)) << (4 * (i % 2))
    return codes.reshape(x.shape[:-1] + (nb * 16,)), scales.reshape(x.shape[:-1] + (nb,))


def kv4_decode(codes, scales, D):
    """The values: sign, grid and 2^(scale - 127); a scale of 255 is NaN."""
    codes, scales = np.asarray(codes), np.asarray(scales).astype(np.float64)
    c = np.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[:-1] + (-1,))
    val = np.array(GRID + [-g for g in GRID])[c]
    s = np.where(scales == 255, np.nan, 2.0 ** (scales - 127))
    return (val * np.repeat(s, 32, -1))[..., :D]

"""Float64 oracle of the attention-block operators: rotary positions, dropout
from Philox 4x32-10, attention over packed documents and over a cache.  Plain
NumPy from the formulas, test infrastructure only."""
import numpy as np

M32 = 0xFFFFFFFF


# ---- rotary positions ---------------------------------------------------------
def rope(x, pos, table, interleaved=False, inverse=False):
    """x [T][H][D], table [P][rot/2][2]: each pair times its rotation matrix."""
    x, table = np.asarray(x, np.float64), np.asarray(table, np.float64)
    y = x.copy()
    n = table.shape[1]
    for i in range(n):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + n)
        c, s = table[pos, i, 0][:, None], table[pos, i, 1][:, None] * (-1.0 if inverse else 1.0)
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., a] * s + x[..., b] * c
    return y


# ---- dropout --------------------------------------------------------------------
def philox(ctr, key):
    """Philox 4x32-10 (Salmon et al., 2011) of one counter, Python integers."""
    c, k = list(ctr), list(key)
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
        c = [(b >> 32) ^ c[1] ^ k[0], b & M32, (a >> 32) ^ c[3] ^ k[1], a & M32]
        k = [(k[0] + 0x9E3779B9) & M32, (k[1] + 0xBB67AE85) & M32]
    return c


def keep(n, p, seed, offset):
    cut, out = round(p * 65536), np.zeros(n, bool)
    for blk in range(offset // 8, (offset + n + 7) // 8):
        w = philox((blk & M32, blk >> 32, 0, 0), (seed & M32, seed >> 32))
        for lane in range(8):
            i = blk * 8 + lane - offset
            if 0 <= i < n:
                out[i] = ((w[lane // 2] >> (16 * (lane % 2))) & 0xFFFF) >= cut
    return out


def dropout(x, residual, p, seed, offset):
    cut = round(p * 65536)
    g = 65536.0 / (65536 - cut) if cut < 65536 else 0.0
    x = np.asarray(x, np.float64).reshape(-1)
    y = np.where(keep(x.size, p, seed, offset), np.nan_to_num(x, nan=np.nan) * g, 0.0)
    return y if residual is None else y + np.asarray(residual, np.float64).reshape(-1)


# ---- attention --------------------------------------------------------------------
def mask(Tq, Tk, cu_q, cu_k, prefix=None, causal=True):
    """(seen [Tq][Tk], position [Tq])."""
    seen, pos = np.zeros((Tq, Tk), bool), np.zeros(Tq, np.int64)
    for d in range(len(cu_q) - 1):
        lq, lk = cu_q[d + 1] - cu_q[d], cu_k[d + 1] - cu_k[d]
        for i in range(lq):
            at = i + lk - lq
            pos[cu_q[d] + i] = cu_k[d] + at
            for j in range(lk):
                if not causal or j <= at or (prefix is not None and j < prefix[d]):
                    seen[cu_q[d] + i, cu_k[d] + j] = True
    return seen, pos


def _scores(q, k, scale, cap, slope, dist):
    x = scale * (q @ k.T)
    t = np.tanh(x / cap) if cap else None
    s = cap * t if cap else x
    return s - slope * dist, (1 - t * t if cap else np.ones_like(x))


def attention(q, k, v, seen, pos, scale=None, cap=0.0, slopes=None, dout=None):
    """q [Tq][Hq][D], k, v [Tk][Hkv][D] -> dict o, lse and, with dout, dq, dk,
    dv.  What a row does not see is never multiplied in: it is cut out first."""
    q, k, v = (np.asarray(a, np.float64) for a in (q, k, v))
    Tq, Hq, D = q.shape
    Tk, Hk, _ = k.shape
    g, scale = Hq // Hk, scale or D ** -0.5
    out = {"o": np.zeros((Tq, Hq, D)), "lse": np.full((Hq, Tq), -np.inf)}
    if dout is not None:
        dout = np.asarray(dout, np.float64)
        out |= {"dq": np.zeros_like(q), "dk": np.zeros_like(k), "dv": np.zeros_like(v)}
    for h in range(Hq):
        sl = 0.0 if slopes is None else float(slopes[h])
        for i in range(Tq):
            js = np.nonzero(seen[i])[0]
            if not js.size:
                continue
            kk, vv = k[js, h // g], v[js, h // g]
            s, dsdx = _scores(q[i:i + 1, h], kk, scale, cap, sl, np.abs(pos[i] - js)[None])
            s, dsdx = s[0], dsdx[0]
            top = s.max()
            e = np.exp(s - top)
            p = e / e.sum()
            o = p @ vv
            out["o"][i, h], out["lse"][h, i] = o, top + np.log(e.sum())
            if dout is not None:
                do = dout[i, h]
                ds = p * (vv @ do - do @ o) * dsdx * scale
                out["dq"][i, h] = ds @ kk
                out["dk"][js, h // g] += ds[:, None] * q[i, h]
                out["dv"][js, h // g] += p[:, None] * do
    return out


def decode(q, k, v, start, length, scale=None, cap=0.0, slopes=None):
    """q [B][Hq][D], caches [B][rows][Hkv][D]."""
    o = np.zeros(q.shape)
    for b in range(q.shape[0]):
        lo, hi = (0 if start is None else int(start[b])), int(length[b])
        if hi > lo:
            seen = np.zeros((1, k.shape[1]), bool)
            seen[0, lo:hi] = True
            o[b] = attention(q[b:b + 1], k[b], v[b], seen, np.array([hi - 1]), scale, cap, slopes)["o"][0]
    return o

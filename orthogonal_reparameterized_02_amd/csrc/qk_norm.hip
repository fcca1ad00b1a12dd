// Norms of queries and keys with the rotary positions in the same pass:
//   r = 1 / sqrt(mean x^2 + eps),  y = turn(x r w)
// over each head, and its gradient: with g = turn^-1(dy), u = g w, n = x r
//   dw = sum g n,  dx = r (u - n mean(u n)).
// Memory-bound: the forward pass reads x and writes y once, the backward pass
// reads x and dy and writes dx once (r is formed again from x, which has to be
// read anyway), and dw goes through one row of partial sums a workgroup.  These
// are float32 sums: dw is off by 1.7e-7 (2-norm, 16384 tokens).
//
// A head lies in a group of 2^n lanes, up to 16 elements a lane, in the units
// of the rotary kernel (W elements of the first half with their partners, W
// consecutive elements of pairs, or W elements that are not turned); its mean
// takes n exchanges.
//
// Measured, 16384 tokens, 32 + 8 heads of 128, bf16: forward 67 us (336 MB, 5.0
// TB/s, what a large copy reaches), backward 137 us (503 MB, 3.7 TB/s: three
// streams and 104 to 158 registers a lane for the sums of dw, three or four
// waves on a SIMD) and 8 us for the join of its rows; 211 us a training pass.
#include <algorithm>
#include <type_traits>

#include "attn.h"

namespace poetx {

namespace {

template <typename TS, int W> struct alignas(sizeof(TS) * W < 16 ? sizeof(TS) * W : 16) Pack { TS e[W]; };

constexpr int NTH = 256;
// Workgroups of the backward pass at most, each a row of partial sums.  16384
// tokens of 32 + 8 heads of 128, bf16, a training pass: 512 rows 251 us, 1024 230,
// 2048 211, 2304 206, 4096 219 (the join takes longer than the balance wins);
// 4099 of 40 heads of 104 in float32: 1536 86 us, 2048 81, 2304 85 (on the same
// inputs again and again, in turn; 90 where they change from pass to pass, for the
// last-level cache holds most of these 341 MB).
constexpr int MOST_ROWS = 2048;

// How a head's units lie in its lanes
struct Lanes {
  int turn, units;  // units that are turned, all units
  int lg;           // log2 of the lanes a head
};

__device__ __forceinline__ float group_sum(float x, int lg) {
  for (int i = 0; i < lg; ++i) x += __shfl_xor(x, 1 << i);
  return x;
}

// One head's elements in this lane: U units of W (two times W in the half
// layout), zero where there is none.
template <typename TS, int W, bool PAIRS> struct Head {
  static constexpr int U = 8 / W;              // units a lane at most: 64 lanes hold 512 elements
  static constexpr int P = PAIRS ? 1 : 2;      // packs a unit
  static constexpr int C = PAIRS ? W / 2 : W;  // angles a unit
  float v[U][P][W];

  // element of pack p of unit u
  static __device__ __forceinline__ int at(int u, int p, const Lanes& l, int rot) {
    return u < l.turn ? u * W + p * (rot / 2) : rot + (u - l.turn) * W;
  }
  static __device__ __forceinline__ bool has(int u, int p, const Lanes& l) { return u < (p ? l.turn : l.units); }

  // the elements as they are stored
  template <typename T> struct Raw {
    Pack<T, W> k[U][P];
    __device__ __forceinline__ void load(const T* x, int lane, const Lanes& l, int rot) {
#pragma unroll
      for (int i = 0; i < U; ++i)
#pragma unroll
        for (int p = 0; p < P; ++p) {
          const int u = lane + (i << l.lg);
          k[i][p] = {};
          if (has(u, p, l)) k[i][p] = *reinterpret_cast<const Pack<T, W>*>(x + at(u, p, l, rot));
        }
    }
  };
  template <typename T> __device__ __forceinline__ void set(const Raw<T>& r) {
#pragma unroll
    for (int i = 0; i < U; ++i)
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int e = 0; e < W; ++e) v[i][p][e] = St<T>::ld(&r.k[i][p].e[e]);
  }
  template <typename T> __device__ __forceinline__ void load(const T* x, int lane, const Lanes& l, int rot) {
    Raw<T> r;
    r.load(x, lane, l, rot);
    set(r);
  }
  __device__ __forceinline__ void store(TS* y, int lane, const Lanes& l, int rot) const {
#pragma unroll
    for (int i = 0; i < U; ++i)
#pragma unroll
      for (int p = 0; p < P; ++p) {
        const int u = lane + (i << l.lg);
        Pack<TS, W> k;
#pragma unroll
        for (int e = 0; e < W; ++e) St<TS>::st(&k.e[e], v[i][p][e]);
        if (has(u, p, l)) *reinterpret_cast<Pack<TS, W>*>(y + at(u, p, l, rot)) = k;
      }
  }
  // f(value index pack, element) over the lane's elements
  template <class F> static __device__ __forceinline__ void each(F f) {
#pragma unroll
    for (int i = 0; i < U; ++i)
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int e = 0; e < W; ++e) f(i, p, e);
  }
};

// cos and sin of this lane's pairs; a position outside the table turns by NaN
template <typename TS, int W, bool PAIRS> struct Angles {
  using H = Head<TS, W, PAIRS>;
  float2 cs[H::U][H::C];
  __device__ __forceinline__ void load(const QkNormArgs& a, long t, int lane, const Lanes& l) {
    if (l.turn == 0) return;
    const int p = a.pos[t];
    const bool in = (unsigned)p < (unsigned)a.P;
    const float2* row = reinterpret_cast<const float2*>(a.table) + (long)(in ? p : 0) * (a.rot / 2);
    const float nan = __uint_as_float(0x7fc00000u);
#pragma unroll
    for (int i = 0; i < H::U; ++i)
#pragma unroll
      for (int c = 0; c < H::C; ++c) {
        const int u = lane + (i << l.lg);
        cs[i][c] = make_float2(1.0f, 0.0f);
        if (u < l.turn) cs[i][c] = in ? row[u * H::C + c] : make_float2(nan, nan);
      }
  }
  template <bool INV> __device__ __forceinline__ void turn(H& h, int lane, const Lanes& l) const {
#pragma unroll
    for (int i = 0; i < H::U; ++i) {
      if (lane + (i << l.lg) >= l.turn) continue;
#pragma unroll
      for (int c = 0; c < H::C; ++c) {
        float& x = PAIRS ? h.v[i][0][2 * c] : h.v[i][0][c];
        float& y = PAIRS ? h.v[i][0][2 * c + 1] : h.v[i][H::P - 1][c];
        const float co = cs[i][c].x, s = INV ? -cs[i][c].y : cs[i][c].y, lo = x;
        x = lo * co - y * s;
        y = lo * s + y * co;
      }
    }
  }
};

// HPG heads of one token a group, so that weights and angles are loaded once
// for them.
template <typename TS, int W, bool PAIRS, int HPG>
__global__ __launch_bounds__(NTH) void k_qk_norm_fwd(QkNormArgs a, Lanes l, int cq, int per_token) {
  using H = Head<TS, W, PAIRS>;
  const int lane = threadIdx.x & ((1 << l.lg) - 1);
  const long id0 = (long)blockIdx.x * (NTH >> l.lg), t0 = id0 / per_token;
  const int n = (int)(id0 - t0 * per_token) + (threadIdx.x >> l.lg);
  const int dt = n / per_token, c = n - dt * per_token;
  const long t = t0 + dt;
  if (t >= a.T) return;
  const bool isq = c < cq;
  const int h0 = (isq ? c : c - cq) * HPG, heads = min(HPG, (isq ? a.Hq : a.Hk) - h0);
  const TS* x = (isq ? (const TS*)a.q + t * a.ldq : (const TS*)a.k + t * a.ldk) + (long)h0 * a.D;
  TS* y = (isq ? (TS*)a.qo + t * a.ldqo : (TS*)a.ko + t * a.ldko) + (long)h0 * a.D;
  const float* wp = isq ? a.wq : a.wk;
  H xs[HPG], w;
#pragma unroll
  for (int i = 0; i < HPG; ++i)
    if (i < heads) xs[i].load(x + (long)i * a.D, lane, l, a.rot);
  if (wp) w.load(wp, lane, l, a.rot);
  else H::each([&](int i, int p, int e) { w.v[i][p][e] = 1.0f; });
  Angles<TS, W, PAIRS> ang;
  ang.load(a, t, lane, l);
#pragma unroll
  for (int i = 0; i < HPG; ++i) {
    if (i >= heads) break;
    float ss = 0.0f;
    H::each([&](int j, int p, int e) { ss = fmaf(xs[i].v[j][p][e], xs[i].v[j][p][e], ss); });
    const float r = rsqrtf(fmaf(group_sum(ss, l.lg), a.inv_d, a.eps));
    H::each([&](int j, int p, int e) { xs[i].v[j][p][e] *= r * w.v[j][p][e]; });
    ang.template turn<false>(xs[i], lane, l);
    xs[i].store(y + (long)i * a.D, lane, l, a.rot);
  }
}

// A group takes `run` heads of one token, whose weights and angles it loads once,
// while the next head is on its way; then the next such run that is its own.
// The sum of dw stays in its registers.  The first rows_q workgroups take the
// queries.
template <typename TS, int W, bool PAIRS>
__global__ __launch_bounds__(NTH) void k_qk_norm_bwd(QkNormArgs a, Lanes l, int rows_q, int rows_k, int run, float* part) {
  using H = Head<TS, W, PAIRS>;
  __shared__ float red[NTH * 16];
  const int lane = threadIdx.x & ((1 << l.lg) - 1), group = threadIdx.x >> l.lg, groups = NTH >> l.lg;
  const bool isq = (int)blockIdx.x < rows_q;
  const int row = isq ? blockIdx.x : blockIdx.x - rows_q, rows = isq ? rows_q : rows_k;
  const int heads = isq ? a.Hq : a.Hk, chunks = (heads + run - 1) / run;
  const TS* x0 = isq ? (const TS*)a.q : (const TS*)a.k;
  const TS* g0 = isq ? (const TS*)a.gq : (const TS*)a.gk;
  TS* d0 = isq ? (TS*)a.dq : (TS*)a.dk;
  const long ldx = isq ? a.ldq : a.ldk, ldg = isq ? a.ldqo : a.ldko, ldd = isq ? a.lddq : a.lddk;
  const float* wp = isq ? a.wq : a.wk;
  H w, dw;
  if (wp) w.load(wp, lane, l, a.rot);
  else H::each([&](int i, int p, int e) { w.v[i][p][e] = 1.0f; });
  H::each([&](int i, int p, int e) { dw.v[i][p][e] = 0.0f; });
  const long step = (long)rows * groups, items = (long)a.T * chunks;
  for (long it = (long)row * groups + group; it < items; it += step) {
    const long t = it / chunks;
    const int h0 = (int)(it - t * chunks) * run, h1 = min(h0 + run, heads);
    const TS *xp = x0 + t * ldx, *gp = g0 + t * ldg;
    TS* dp = d0 + t * ldd;
    typename H::template Raw<TS> rx, rg;
    rx.load(xp + (long)h0 * a.D, lane, l, a.rot);
    rg.load(gp + (long)h0 * a.D, lane, l, a.rot);
    Angles<TS, W, PAIRS> ang;
    ang.load(a, t, lane, l);
    for (int h = h0; h < h1; ++h) {
      H x, g;
      x.set(rx);
      g.set(rg);
      if (h + 1 < h1) {
        rx.load(xp + (long)(h + 1) * a.D, lane, l, a.rot);
        rg.load(gp + (long)(h + 1) * a.D, lane, l, a.rot);
      }
      float ss = 0.0f, un = 0.0f;
      ang.template turn<true>(g, lane, l);
      H::each([&](int j, int p, int e) {
        ss = fmaf(x.v[j][p][e], x.v[j][p][e], ss);
        un = fmaf(g.v[j][p][e] * w.v[j][p][e], x.v[j][p][e], un);
      });
      const float r = rsqrtf(fmaf(group_sum(ss, l.lg), a.inv_d, a.eps));
      const float m = group_sum(un, l.lg) * r * a.inv_d;  // mean of u n
      H::each([&](int j, int p, int e) {
        const float nrm = x.v[j][p][e] * r, gv = g.v[j][p][e];
        dw.v[j][p][e] = fmaf(gv, nrm, dw.v[j][p][e]);
        x.v[j][p][e] = r * fmaf(-nrm, m, gv * w.v[j][p][e]);
      });
      x.store(dp + (long)h * a.D, lane, l, a.rot);
    }
  }
  if (!(isq ? a.dwq : a.dwk)) return;
  // the groups' sums in group order
#pragma unroll
  for (int i = 0; i < H::U; ++i)
#pragma unroll
    for (int p = 0; p < H::P; ++p) {
      const int u = lane + (i << l.lg);
      if (H::has(u, p, l))
#pragma unroll
        for (int e = 0; e < W; ++e) red[group * a.D + H::at(u, p, l, a.rot) + e] = dw.v[i][p][e];
    }
  __syncthreads();
  for (int d = threadIdx.x; d < a.D; d += NTH) {
    float s = 0.0f;
    for (int g = 0; g < groups; ++g) s += red[g * a.D + d];
    part[(long)blockIdx.x * a.D + d] = s;
  }
}

// dw[d] = sum of the rows: 64 columns a workgroup, four rows a wave's load, sixteen
// waves; a thread's rows, then four lanes, then the waves in order
constexpr int JW = 16;
__global__ __launch_bounds__(64 * JW) void k_qk_norm_join(int D, int rows_q, int rows_k, const float* part,
                                                          float* dwq, float* dwk) {
  __shared__ float4 red[JW][16];
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64, d = blockIdx.x * 64 + 4 * (lane & 15);
  float* out = blockIdx.y ? dwk : dwq;
  if (!out) return;
  const float* p = part + (blockIdx.y ? (long)rows_q * D : 0) + min(d, D - 4);
  const int rows = blockIdx.y ? rows_k : rows_q;
  float4 s = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
  for (int r = 4 * wave + (lane >> 4); r < rows; r += 4 * JW) {
    const float4 x = *reinterpret_cast<const float4*>(p + (long)r * D);
    s.x += x.x, s.y += x.y, s.z += x.z, s.w += x.w;
  }
#pragma unroll
  for (int m = 16; m < 64; m <<= 1) {
    s.x += __shfl_xor(s.x, m);
    s.y += __shfl_xor(s.y, m);
    s.z += __shfl_xor(s.z, m);
    s.w += __shfl_xor(s.w, m);
  }
  if (lane < 16) red[wave][lane] = s;
  __syncthreads();
  if (threadIdx.x < 64 && blockIdx.x * 64 + threadIdx.x < D) {
    float t = 0.0f;
#pragma unroll
    for (int w = 0; w < JW; ++w) t += reinterpret_cast<const float*>(red[w])[threadIdx.x];
    out[blockIdx.x * 64 + threadIdx.x] = t;
  }
}

struct Rows { int q, k; };
// Rows of partial sums for the queries and for the keys: as their work, at
// least one each, and 32 heads a row (as many as a workgroup holds at a time if
// they have 128 bf16; 1000 tokens of 40 heads: 2048 rows 31 us, 1024 27 us).
Rows rows_of(const QkNormArgs& a) {
  const long most = std::min((long)MOST_ROWS, ((long)a.T * (a.Hq + a.Hk) + 31) / 32);
  Rows r;
  r.q = (int)std::max(1L, most * a.Hq / (a.Hq + a.Hk));
  r.k = a.Hk ? (int)std::max(1L, most * a.Hk / (a.Hq + a.Hk)) : 0;
  return r;
}

// Heads of one token that a group of the forward kernel loads together: the
// weights and angles are loaded once for them.
constexpr int HPG_F = 4;

template <typename TS, int W, bool PAIRS> hipError_t norm_fwd(const QkNormArgs& a, const Lanes& l, hipStream_t s) {
  const int cq = (a.Hq + HPG_F - 1) / HPG_F, per_token = cq + (a.Hk + HPG_F - 1) / HPG_F;
  const int most = (int)std::max(1L, std::min((long)a.T, LAUNCH_THREADS / ((long)per_token << l.lg)));  // tokens a launch
  QkNormArgs b = a;
  constexpr long ES = sizeof(TS);
  for (long t = 0; t < a.T; t += most) {
    b.T = (int)std::min((long)most, a.T - t);
    b.pos = a.pos ? a.pos + t : nullptr;
    b.q = (const char*)a.q + t * a.ldq * ES, b.k = (const char*)a.k + t * a.ldk * ES;
    b.qo = (char*)a.qo + t * a.ldqo * ES, b.ko = (char*)a.ko + t * a.ldko * ES;
    const long threads = ((long)b.T * per_token) << l.lg;
    k_qk_norm_fwd<TS, W, PAIRS, HPG_F><<<dim3((unsigned)((threads + NTH - 1) / NTH)), NTH, 0, s>>>(b, l, cq, per_token);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

template <typename TS, int W, bool PAIRS> hipError_t norm_bwd(const QkNormArgs& a, const Lanes& l, float* ws, hipStream_t s) {
  const Rows r = rows_of(a);
  // as many heads as a group has to take anyway
  const long groups = (long)(r.q + r.k) * (NTH >> l.lg), all = (long)a.T * (a.Hq + a.Hk);
  const int run = (int)std::max(1L, std::min((all + groups - 1) / groups, (long)std::max(a.Hq, a.Hk)));
  k_qk_norm_bwd<TS, W, PAIRS><<<dim3(r.q + r.k), NTH, 0, s>>>(a, l, r.q, r.k, run, ws);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || (!a.dwq && !a.dwk)) return e;
  k_qk_norm_join<<<dim3((a.D + 63) / 64, 2), 64 * JW, 0, s>>>(a.D, r.q, r.k, ws, a.dwq, a.dwk);
  return hipGetLastError();
}

// W: the widest access (16 bytes at most) that divides the turned part (each
// half of it in the half layout) and the rest of the head
template <typename TS, class F> hipError_t by_width(const QkNormArgs& a, F f) {
  const int part = a.interleaved ? a.rot : a.rot / 2, parts = part | (a.D - a.rot);
  const auto go = [&](auto w) -> hipError_t {
    constexpr int W = decltype(w)::value;
    Lanes l;
    l.turn = part / W;
    l.units = l.turn + (a.D - a.rot) / W;
    l.lg = 0;
    while ((1 << l.lg) < l.units && l.lg < 6) ++l.lg;
    // an even rot leaves pairs at least two wide
    if constexpr (W >= 2)
      if (a.interleaved) return f(w, std::true_type{}, l);
    return f(w, std::false_type{}, l);
  };
  if (sizeof(TS) == 2 && parts % 8 == 0) return go(std::integral_constant<int, 16 / sizeof(TS)>{});
  if (parts % 4 == 0) return go(std::integral_constant<int, 4>{});
  if (parts % 2 == 0) return go(std::integral_constant<int, 2>{});
  return go(std::integral_constant<int, 1>{});
}

}  // namespace

size_t qk_norm_ws_bytes(const QkNormArgs& a) {
  const Rows r = rows_of(a);
  return (size_t)(r.q + r.k) * a.D * 4;
}

template <typename TS> hipError_t launch_qk_norm_fwd(const QkNormArgs& a, hipStream_t s) {
  return by_width<TS>(a, [&](auto w, auto pairs, const Lanes& l) {
    return norm_fwd<TS, decltype(w)::value, decltype(pairs)::value>(a, l, s);
  });
}
template <typename TS> hipError_t launch_qk_norm_bwd(const QkNormArgs& a, float* ws, hipStream_t s) {
  return by_width<TS>(a, [&](auto w, auto pairs, const Lanes& l) {
    return norm_bwd<TS, decltype(w)::value, decltype(pairs)::value>(a, l, ws, s);
  });
}

template hipError_t launch_qk_norm_fwd<bf16>(const QkNormArgs&, hipStream_t);
template hipError_t launch_qk_norm_fwd<float>(const QkNormArgs&, hipStream_t);
template hipError_t launch_qk_norm_bwd<bf16>(const QkNormArgs&, float*, hipStream_t);
template hipError_t launch_qk_norm_bwd<float>(const QkNormArgs&, float*, hipStream_t);

}  // namespace poetx

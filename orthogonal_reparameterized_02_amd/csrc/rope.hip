// Rotary positions: every pair of a head is turned by the angle of its
// token's position, (a, b) -> (a c - b s, a s + b c), with (c, s) from a
// table row; the rest of the head is copied.  Memory-bound: each element is
// read and written once, the table rows of nearby tokens come from cache.
#include "attn.h"

namespace poetx {

namespace {

// W values of one type as one access
template <typename TS, int W> struct alignas(sizeof(TS) * W) Pack { TS e[W]; };

constexpr int NTH = 256;

// One thread per unit of one head of one token.  A unit is, in the half
// layout, W elements of the first half with their partners (rot/2 further
// on); in the interleaved one W consecutive elements; past rot, W elements
// to copy.  W divides every part, so units never straddle.
template <typename TS, int W, bool PAIRS>
__global__ __launch_bounds__(NTH) void k_rope(RopeArgs a, const TS* q, const TS* k, TS* qo, TS* ko,
                                              int turn_units, int units, int per_token) {
  const long id = (long)blockIdx.x * NTH + threadIdx.x;
  const long t = id / per_token;
  if (t >= a.T) return;
  const int in = (int)(id - t * per_token);
  const int h = in / units, u = in - h * units;
  const bool isq = h < a.Hq;
  const TS* src = isq ? q + t * a.ldq + (long)h * a.D : k + t * a.ldk + (long)(h - a.Hq) * a.D;
  TS* dst = isq ? qo + t * a.ldqo + (long)h * a.D : ko + t * a.ldko + (long)(h - a.Hq) * a.D;
  using V = Pack<TS, W>;
  if (u >= turn_units) {
    const int e = a.rot + (u - turn_units) * W;
    *reinterpret_cast<V*>(dst + e) = *reinterpret_cast<const V*>(src + e);
    return;
  }
  const int p = a.pos[t];
  const bool in_table = (unsigned)p < (unsigned)a.P;
  const float2* cs = reinterpret_cast<const float2*>(a.table) + (long)(in_table ? p : 0) * (a.rot / 2);
  const float bad = in_table ? 0.0f : __uint_as_float(0x7fc00000u);
  if constexpr (PAIRS) {
    const int e = u * W;
    const V x = *reinterpret_cast<const V*>(src + e);
    V y;
#pragma unroll
    for (int i = 0; i < W; i += 2) {
      const float2 c = cs[(e + i) / 2];
      const float s = a.sgn * c.y, lo = St<TS>::ld(&x.e[i]), hi = St<TS>::ld(&x.e[i + 1]);
      St<TS>::st(&y.e[i], lo * c.x - hi * s + bad);
      St<TS>::st(&y.e[i + 1], lo * s + hi * c.x + bad);
    }
    *reinterpret_cast<V*>(dst + e) = y;
  } else {
    const int e = u * W, half = a.rot / 2;
    const V x0 = *reinterpret_cast<const V*>(src + e);
    const V x1 = *reinterpret_cast<const V*>(src + half + e);
    V y0, y1;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const float2 c = cs[e + i];
      const float s = a.sgn * c.y, lo = St<TS>::ld(&x0.e[i]), hi = St<TS>::ld(&x1.e[i]);
      St<TS>::st(&y0.e[i], lo * c.x - hi * s + bad);
      St<TS>::st(&y1.e[i], lo * s + hi * c.x + bad);
    }
    *reinterpret_cast<V*>(dst + e) = y0;
    *reinterpret_cast<V*>(dst + half + e) = y1;
  }
}

template <typename TS, int W>
hipError_t rope_w(const RopeArgs& a, const TS* q, const TS* k, TS* qo, TS* ko, hipStream_t s) {
  const int turn = (a.interleaved ? a.rot : a.rot / 2) / W, units = turn + (a.D - a.rot) / W;
  const int per_token = units * (a.Hq + a.Hk);
  const long total = (long)a.T * per_token;
  const dim3 grid((unsigned)((total + NTH - 1) / NTH));
  if constexpr (W >= 2) {
    if (a.interleaved) {
      k_rope<TS, W, true><<<grid, NTH, 0, s>>>(a, q, k, qo, ko, turn, units, per_token);
      return hipGetLastError();
    }
  }
  k_rope<TS, W, false><<<grid, NTH, 0, s>>>(a, q, k, qo, ko, turn, units, per_token);
  return hipGetLastError();
}

}  // namespace

// W: the widest access (16 bytes at most) that divides the turned part (each
// half of it in the half layout) and the rest of the head.
template <typename TS>
hipError_t launch_rope(const RopeArgs& a, const TS* q, const TS* k, TS* qo, TS* ko, hipStream_t s) {
  const int part = a.interleaved ? a.rot : a.rot / 2;
  const int parts = part | (a.D - a.rot);
  if (sizeof(TS) == 2 && parts % 8 == 0) return rope_w<TS, 16 / sizeof(TS)>(a, q, k, qo, ko, s);
  if (parts % 4 == 0) return rope_w<TS, 4>(a, q, k, qo, ko, s);
  if (parts % 2 == 0) return rope_w<TS, 2>(a, q, k, qo, ko, s);
  return rope_w<TS, 1>(a, q, k, qo, ko, s);
}

template hipError_t launch_rope<bf16>(const RopeArgs&, const bf16*, const bf16*, bf16*, bf16*, hipStream_t);
template hipError_t launch_rope<float>(const RopeArgs&, const float*, const float*, float*, float*, hipStream_t);

}  // namespace poetx

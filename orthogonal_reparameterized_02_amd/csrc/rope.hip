// Rotary positions: every pair of a head is turned by the angle of its
// token's position, (a, b) -> (a c - b s, a s + b c), with (c, s) from a
// table row; the rest of the head is copied.  Memory-bound: each element is
// read and written once, the table rows of nearby tokens come from cache.
// Measured: 16384 tokens of 32 + 8 heads of 128, bf16, 58.7 us = 5.7 TB/s;
// 4099 tokens of 40 heads of 104, 40 elements turned, float32, 27.3 us = 5.0
// TB/s (a copy of 1 GiB: 5.0).  Two or four units a thread were slower (65 and
// 72 us for the first).
#include <algorithm>
#include <type_traits>

#include "attn.h"

namespace poetx {

namespace {

// W values of one type as one access
template <typename TS, int W> struct alignas(sizeof(TS) * W) Pack { TS e[W]; };

constexpr int NTH = 256;

// One thread per unit of one head of one token.  A unit is, in the half
// layout, W elements of the first half with their partners (rot/2 further
// on); in the interleaved one W consecutive elements; past rot, W elements
// to copy.  W divides every part, so units never straddle.  The unit's own
// loads go out before the two dependent ones (position, then table row).
template <typename TS, int W, bool PAIRS>
__global__ __launch_bounds__(NTH) void k_rope(RopeArgs a, const TS* q, const TS* k, TS* qo, TS* ko,
                                              int turn_units, int units, int per_token,
                                              float inv_units, float inv_token) {
  using V = Pack<TS, W>;
  constexpr int C = PAIRS ? W / 2 : W;  // angles a unit
  // the block's first unit by one scalar division, the thread's by products
  // with reciprocals: (n + 1/2) / d truncates right for n below 2^21
  const long id0 = (long)blockIdx.x * NTH;
  const long t0 = id0 / per_token;
  const int n = (int)(id0 - t0 * per_token) + threadIdx.x;
  const int dt = (int)(((float)n + 0.5f) * inv_token);
  const long t = t0 + dt;
  if (t >= a.T) return;
  const int in = n - dt * per_token;
  const int h = (int)(((float)in + 0.5f) * inv_units), u = in - h * units;
  const bool isq = h < a.Hq;
  const int e = u < turn_units ? u * W : a.rot + (u - turn_units) * W;
  const TS* src = (isq ? q + t * a.ldq + (long)h * a.D : k + t * a.ldk + (long)(h - a.Hq) * a.D) + e;
  TS* dst = (isq ? qo + t * a.ldqo + (long)h * a.D : ko + t * a.ldko + (long)(h - a.Hq) * a.D) + e;
  V x0 = *reinterpret_cast<const V*>(src);
  if (u >= turn_units) {
    *reinterpret_cast<V*>(dst) = x0;
    return;
  }
  V x1;
  if constexpr (!PAIRS) x1 = *reinterpret_cast<const V*>(src + a.rot / 2);
  const int p = a.pos[t];
  const bool in_table = (unsigned)p < (unsigned)a.P;
  const float bad = in_table ? 0.0f : __uint_as_float(0x7fc00000u);
  const float2* cs = reinterpret_cast<const float2*>(a.table) + (long)(in_table ? p : 0) * (a.rot / 2) + u * C;
  V y0, y1;
#pragma unroll
  for (int i = 0; i < C; ++i) {
    const float c = cs[i].x, s = a.sgn * cs[i].y;
    const float lo = St<TS>::ld(PAIRS ? &x0.e[2 * i] : &x0.e[i]);
    const float hi = St<TS>::ld(PAIRS ? &x0.e[2 * i + 1] : &x1.e[i]);
    St<TS>::st(PAIRS ? &y0.e[2 * i] : &y0.e[i], lo * c - hi * s + bad);
    St<TS>::st(PAIRS ? &y0.e[2 * i + 1] : &y1.e[i], lo * s + hi * c + bad);
  }
  *reinterpret_cast<V*>(dst) = y0;
  if constexpr (!PAIRS) *reinterpret_cast<V*>(dst + a.rot / 2) = y1;
}

template <typename TS, int W>
hipError_t rope_w(const RopeArgs& a, const TS* q, const TS* k, TS* qo, TS* ko, hipStream_t s) {
  const int turn = (a.interleaved ? a.rot : a.rot / 2) / W, units = turn + (a.D - a.rot) / W;
  const int per_token = units * (a.Hq + a.Hk);
  const int most = (int)std::min((long)a.T, LAUNCH_THREADS / per_token);  // tokens a launch
  RopeArgs b = a;
  for (long t = 0; t < a.T; t += most) {
    b.T = (int)std::min((long)most, a.T - t);
    b.pos = a.pos + t;
    const TS *bq = q + t * a.ldq, *bk = k ? k + t * a.ldk : nullptr;
    TS *bqo = qo + t * a.ldqo, *bko = ko ? ko + t * a.ldko : nullptr;
    const dim3 grid((unsigned)(((long)b.T * per_token + NTH - 1) / NTH));
    const auto launch = [&](auto pairs) {
      k_rope<TS, W, decltype(pairs)::value><<<grid, NTH, 0, s>>>(b, bq, bk, bqo, bko, turn, units, per_token,
                                                                 1.0f / units, 1.0f / per_token);
    };
    // an even rot leaves pairs at least two wide
    if constexpr (W >= 2) a.interleaved ? launch(std::true_type{}) : launch(std::false_type{});
    else launch(std::false_type{});
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
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

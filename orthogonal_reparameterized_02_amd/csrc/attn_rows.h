// Attention one row at a time: a wave holds one query (or key) row, lane l
// its elements 2 l and 2 l + 1, and walks the rows that it sees.  Nothing
// outside the mask is read, so whatever stands there has no influence.
#pragma once

#include "attn.h"

namespace poetx {

__device__ __forceinline__ float wave_sum(float x) {
#pragma unroll
  for (int m = 32; m; m >>= 1) x += __shfl_xor(x, m);
  return x;
}

// elements 2 l, 2 l + 1 of a row of D <= 128 (0 past the end); rows are
// aligned to 16 bytes
__device__ __forceinline__ float2 ld2(const bf16* p, int lane, int D) {
  if (2 * lane >= D) return make_float2(0.0f, 0.0f);
  const uint32_t u = reinterpret_cast<const uint32_t*>(p)[lane];
  return make_float2(__uint_as_float(u << 16), __uint_as_float(u & 0xffff0000u));
}
__device__ __forceinline__ float2 ld2(const float* p, int lane, int D) {
  if (2 * lane >= D) return make_float2(0.0f, 0.0f);
  return reinterpret_cast<const float2*>(p)[lane];
}
__device__ __forceinline__ void st2(bf16* p, int lane, int D, float2 v) {
  if (2 * lane < D) reinterpret_cast<uint32_t*>(p)[lane] = pack2bf(v.x, v.y);
}
__device__ __forceinline__ void st2(float* p, int lane, int D, float2 v) {
  if (2 * lane < D) reinterpret_cast<float2*>(p)[lane] = v;
}

// the score of a pair from q.k; dsdx: its derivative by scale * q.k
__device__ __forceinline__ float pair_score(float qk, float scale, float cap, float slope, int dist,
                                            float& dsdx) {
  float s = qk * scale;
  dsdx = 1.0f;
  if (cap > 0.0f) {
    const float t = tanhf(s / cap);
    s = cap * t;
    dsdx = 1.0f - t * t;
  }
  return s - slope * (float)abs(dist);
}

// One query over keys [lo, hi): running maximum m, sum l = sum exp(s - m) and
// (returned) sum exp(s - m) v.  A maximum of -inf stands for 0, so scores that
// are all -inf give sums of 0.
template <typename TS>
__device__ __forceinline__ float2 attn_row(const TS* q, const TS* k, long ldk, const TS* v, long ldv,
                                           int lo, int hi, int pos, int D, float scale, float cap,
                                           float slope, int lane, float& m, float& l) {
  const float2 qv = ld2(q, lane, D);
  m = -INFINITY, l = 0.0f;
  float2 o = make_float2(0.0f, 0.0f);
  for (int j = lo; j < hi; ++j) {
    const float2 kv = ld2(k + (long)j * ldk, lane, D), vv = ld2(v + (long)j * ldv, lane, D);
    float unused;
    const float s = pair_score(wave_sum(qv.x * kv.x + qv.y * kv.y), scale, cap, slope, pos - j, unused);
    const float m2 = fmaxf(m, s), ref = m2 == -INFINITY ? 0.0f : m2;
    const float p = __expf(s - ref), f = __expf(m - ref);
    m = m2;
    l = l * f + p;
    o.x = o.x * f + p * vv.x;
    o.y = o.y * f + p * vv.y;
  }
  return o;
}

// dq / scale of one query over keys [lo, hi); delta = dout . o
template <typename TS>
__device__ __forceinline__ float2 attn_row_dq(const TS* q, const TS* dout, const TS* k, long ldk, const TS* v, long ldv, int lo, int hi,
                                              int pos, int D, float scale, float cap, float slope,
                                              float lse, float delta, int lane) {
  const float2 qv = ld2(q, lane, D), dv = ld2(dout, lane, D);
  float2 dq = make_float2(0.0f, 0.0f);
  for (int j = lo; j < hi; ++j) {
    const float2 kv = ld2(k + (long)j * ldk, lane, D), vv = ld2(v + (long)j * ldv, lane, D);
    float dsdx;
    const float s = pair_score(wave_sum(qv.x * kv.x + qv.y * kv.y), scale, cap, slope, pos - j, dsdx);
    const float dp = wave_sum(dv.x * vv.x + dv.y * vv.y);
    const float ds = lse == -INFINITY ? 0.0f : __expf(s - lse) * (dp - delta) * dsdx;
    dq.x += ds * kv.x;
    dq.y += ds * kv.y;
  }
  return dq;
}

// adds to dk and dv of one key row what query head h, rows [lo, hi), gives
template <typename TS>
__device__ __forceinline__ void attn_row_dkv(const AttnArgs& a, int h, int j, int lo, int hi, int lane,
                                             float2& dk, float2& dv) {
  const int hk = h / a.group;
  const float2 kv = ld2((const TS*)a.k + (long)j * a.ldk + (long)hk * a.D, lane, a.D);
  const float2 vv = ld2((const TS*)a.v + (long)j * a.ldv + (long)hk * a.D, lane, a.D);
  const float slope = a.slopes ? a.slopes[h] : 0.0f;
  for (int i = lo; i < hi; ++i) {
    const float2 qv = ld2((const TS*)a.q + (long)i * a.ldq + (long)h * a.D, lane, a.D);
    const float2 ov = ld2((const TS*)a.dout + (long)i * a.lddo + (long)h * a.D, lane, a.D);
    float dsdx;
    const float s = pair_score(wave_sum(qv.x * kv.x + qv.y * kv.y), a.scale, a.cap, slope,
                               a.pl.row_pos[i] - j, dsdx);
    const float dp = wave_sum(ov.x * vv.x + ov.y * vv.y);
    const float lse = a.lse[(long)h * a.Tq + i];
    const float p = lse == -INFINITY ? 0.0f : __expf(s - lse);
    const float ds = p * (dp - a.delta[(long)h * a.Tq + i]) * dsdx;
    dv.x += p * ov.x;
    dv.y += p * ov.y;
    dk.x += ds * qv.x;
    dk.y += ds * qv.y;
  }
}

}  // namespace poetx

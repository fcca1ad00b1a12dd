// Attention over packed documents and over a cache: one wave a row.
#include "attn_rows.h"

namespace poetx {

namespace {

constexpr int NTH = 256;

template <typename TS>
__global__ __launch_bounds__(NTH) void k_attn_dq_rows(AttnArgs a) {
  const int lane = threadIdx.x % 64, h = blockIdx.y;
  const int t = blockIdx.x * (NTH / 64) + threadIdx.x / 64;
  if (t >= a.Tq) return;
  const int hk = h / a.group;
  float delta;
  const float2 dq = attn_row_dq<TS>(
      (const TS*)a.q + (long)t * a.ldq + (long)h * a.D,
      (const TS*)a.dout + (long)t * a.lddo + (long)h * a.D,
      (const TS*)a.o + (long)t * a.ldo + (long)h * a.D, (const TS*)a.k + (long)hk * a.D, a.ldk,
      (const TS*)a.v + (long)hk * a.D, a.ldv, a.pl.row_lo[t], a.pl.row_hi[t], a.pl.row_pos[t], a.D,
      a.scale, a.cap, a.slopes ? a.slopes[h] : 0.0f, a.lse[(long)h * a.Tq + t], lane, delta);
  st2((TS*)a.dq + (long)t * a.lddq + (long)h * a.D, lane, a.D, dq);
  if (lane == 0) a.delta[(long)h * a.Tq + t] = delta;
}

template <typename TS>
__global__ __launch_bounds__(NTH) void k_attn_dkv_rows(AttnArgs a) {
  const int lane = threadIdx.x % 64, hk = blockIdx.y;
  const int j = blockIdx.x * (NTH / 64) + threadIdx.x / 64;
  if (j >= a.Tk) return;
  float2 dk, dv;
  attn_row_dkv<TS>(a, hk, j, lane, dk, dv);
  st2((TS*)a.dk + (long)j * a.lddk + (long)hk * a.D, lane, a.D, dk);
  st2((TS*)a.dv + (long)j * a.lddv + (long)hk * a.D, lane, a.D, dv);
}

template <typename TS>
__global__ __launch_bounds__(NTH) void k_attn_decode_rows(DecodeArgs a) {
  const int lane = threadIdx.x % 64, b = blockIdx.y;
  const int h = blockIdx.x * (NTH / 64) + threadIdx.x / 64;
  if (h >= a.Hq) return;
  const int hk = h / a.group;
  const int hi = min(max(a.len[b], 0), a.rows);
  const int lo = a.start ? max(a.start[b], 0) : 0;
  float lse;
  const float2 o = attn_row<TS>((const TS*)a.q + (long)b * a.ldq + (long)h * a.D,
                                (const TS*)a.k + (long)b * a.bsk + (long)hk * a.D, a.ldk,
                                (const TS*)a.v + (long)b * a.bsv + (long)hk * a.D, a.ldv, lo, hi,
                                hi - 1, a.D, a.scale, a.cap, a.slopes ? a.slopes[h] : 0.0f, lane, lse);
  st2((TS*)a.o + (long)b * a.ldo + (long)h * a.D, lane, a.D, o);
}

constexpr int ROWS = NTH / 64;

}  // namespace

template <typename TS> hipError_t launch_attn_bwd(const AttnArgs& a, hipStream_t s) {
  k_attn_dq_rows<TS><<<dim3((a.Tq + ROWS - 1) / ROWS, a.Hq), NTH, 0, s>>>(a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  k_attn_dkv_rows<TS><<<dim3((a.Tk + ROWS - 1) / ROWS, a.Hkv), NTH, 0, s>>>(a);
  return hipGetLastError();
}

template <typename TS> hipError_t launch_attn_decode(const DecodeArgs& a, hipStream_t s) {
  k_attn_decode_rows<TS><<<dim3((a.Hq + ROWS - 1) / ROWS, a.B), NTH, 0, s>>>(a);
  return hipGetLastError();
}

template hipError_t launch_attn_bwd<bf16>(const AttnArgs&, hipStream_t);
template hipError_t launch_attn_bwd<float>(const AttnArgs&, hipStream_t);
template hipError_t launch_attn_decode<bf16>(const DecodeArgs&, hipStream_t);
template hipError_t launch_attn_decode<float>(const DecodeArgs&, hipStream_t);

}  // namespace poetx

// Attention over a cache: one wave a row.
#include "attn_rows.h"

namespace poetx {

namespace {

constexpr int NTH = 256;

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

template <typename TS> hipError_t launch_attn_decode(const DecodeArgs& a, hipStream_t s) {
  k_attn_decode_rows<TS><<<dim3((a.Hq + ROWS - 1) / ROWS, a.B), NTH, 0, s>>>(a);
  return hipGetLastError();
}

template hipError_t launch_attn_decode<bf16>(const DecodeArgs&, hipStream_t);
template hipError_t launch_attn_decode<float>(const DecodeArgs&, hipStream_t);

}  // namespace poetx

// The second pass of attention over a cache: joins the pieces that a sequence's
// rows were cut into.
#pragma once

#include "attn_tile.h"

namespace poetx {

constexpr int JOIN_WAVES = 4;

// rows of a piece where `rows` rows are cut into at most `pieces`: a multiple
// of `grain`
__device__ __forceinline__ int piece_of(int rows, int pieces, int grain) {
  const int n = (rows + pieces - 1) / pieces;
  return (n + grain - 1) / grain * grain;
}

// One query head.  pieces.find gives the number of a sequence's pieces, at most
// 64, and the first one's place.  Lane l of every wave holds elements
// 2 l, 2 l + 1; wave w takes pieces w, w + NW, ...
template <typename T, class Pieces>
__global__ __launch_bounds__(64 * JOIN_WAVES) void k_attn_decode_join(DecodeArgs a, Pieces pieces, const float* part, const float* ml) {
  constexpr int NW = JOIN_WAVES;
  __shared__ float red[NW][130];
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
  const int h = blockIdx.x, b = blockIdx.y;
  long at;
  const int n = pieces.find(a, b, h, at);
  if (n <= 1) return;  // written by the first pass
  const float mine = lane < n ? ml[2 * (at + lane)] : -INFINITY;  // n <= 64
  float M = mine;
#pragma unroll
  for (int x = 32; x; x >>= 1) M = fmaxf(M, __shfl_xor(M, x));
  const float ref = M == -INFINITY ? 0.0f : M;
  const float f = exp2_hw(mine - ref);
  float L = lane < n ? f * ml[2 * (at + lane) + 1] : 0.0f;
#pragma unroll
  for (int x = 32; x; x >>= 1) L += __shfl_xor(L, x);
  float2 acc = make_float2(0.0f, 0.0f);
  const bool in = 2 * lane < a.D;
  for (int s = wave; s < n; s += NW) {
    const float w = __shfl(f, s);
    const float2 v = in ? *reinterpret_cast<const float2*>(part + (at + s) * a.D + 2 * lane) : make_float2(0.0f, 0.0f);
    acc.x = fmaf(w, v.x, acc.x);
    acc.y = fmaf(w, v.y, acc.y);
  }
  red[wave][2 * lane] = acc.x;
  red[wave][2 * lane + 1] = acc.y;
  __syncthreads();
  const int d = threadIdx.x;
  if (d < a.D) {
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < NW; ++w) sum += red[w][d];
    St<T>::st((T*)a.o + (long)b * a.ldo + (long)h * a.D + d, L == 0.0f ? 0.0f : sum / L);
  }
}

}  // namespace poetx

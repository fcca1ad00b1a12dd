// The mask of a packed batch as intervals (AttnPlan): documents, the causal
// bound and prefixes all leave every query one interval of keys, and every
// key one interval of queries.  Two launches of 3 to 5 us per batch, whatever
// the number of layers and heads.
#include <algorithm>

#include "attn_tile.h"

namespace poetx {

namespace {

constexpr int NTH = 256;
constexpr int STAGED = 1024;

// document of row t: the last d with cu[d] <= t, if it ends after t
// (offsets clamped to [0, T]); -1: none
__device__ __forceinline__ int doc_of(const int* cu, int ndoc, int t, int T) {
  int lo = 0, hi = ndoc + 1;  // cu[lo - 1] <= t < cu[hi] in sorted offsets
  while (lo < hi) {
    const int mid = lo + (hi - lo) / 2;
    if (min(max(cu[mid], 0), T) <= t) lo = mid + 1;
    else hi = mid;
  }
  return lo >= 1 && lo <= ndoc ? lo - 1 : -1;
}

// Blocks of query rows, then blocks of key rows; two waves are one tile.
__global__ __launch_bounds__(NTH) void k_attn_plan(int Tq, int Tk, int ndoc, int causal, int qblocks,
                                                   const int* cu_q, const int* cu_k,
                                                   const int* __restrict__ prefix, AttnPlan pl) {
  __shared__ int2 span[NTH / 64];
  // few offsets are searched in LDS: a search in memory waits for each step
  __shared__ int cu[2][STAGED];
  const bool staged = ndoc < STAGED;
  if (staged) {
    for (int i = threadIdx.x; i <= ndoc; i += NTH) {
      cu[0][i] = cu_q[i];
      cu[1][i] = cu_k[i];
    }
    __syncthreads();
    cu_q = cu[0];
    cu_k = cu[1];
  }
  const bool row = (int)blockIdx.x < qblocks;
  const int b = row ? blockIdx.x : blockIdx.x - qblocks, T = row ? Tq : Tk;
  const int t = b * NTH + threadIdx.x;
  const int d = t < T ? doc_of(row ? cu_q : cu_k, ndoc, t, T) : -1;
  int lo = 0, hi = 0, pos = 0;
  if (d >= 0) {
    const int q0 = min(max(cu_q[d], 0), Tq), q1 = min(max(cu_q[d + 1], q0), Tq);
    const int k0 = min(max(cu_k[d], 0), Tk), k1 = min(max(cu_k[d + 1], k0), Tk);
    const int pre = prefix ? min(max(prefix[d], 0), k1 - k0) : 0;
    if (row) {
      pos = k1 - (q1 - t);
      lo = k0;
      hi = causal ? max(min(pos + 1, k1), k0 + pre) : k1;
    } else {
      lo = causal && t >= k0 + pre ? max(q0, q1 - (k1 - t)) : q0;
      hi = q1;
    }
    if (hi <= lo) lo = hi = 0;
  }
  if (t < T) {
    if (row) {
      pl.row_lo[t] = lo;
      pl.row_hi[t] = hi;
      pl.row_pos[t] = pos;
    } else {
      pl.key_lo[t] = lo;
      pl.key_hi[t] = hi;
    }
  }
  const Span s = span_of(lo, hi);
  if (threadIdx.x % 64 == 0) span[threadIdx.x / 64] = make_int2(s.lo, s.hi);
  __syncthreads();
  constexpr int PER = NTH / ATTN_BM;  // tiles a block
  const int tile = b * PER + threadIdx.x, tiles = (T + ATTN_BM - 1) / ATTN_BM;
  if ((int)threadIdx.x < PER && tile < tiles) {
    const int2 x = span[2 * threadIdx.x], y = span[2 * threadIdx.x + 1];
    const int4 e = make_int4(tile, x.x < x.y ? x.x : y.x, y.x < y.y ? y.y : x.y, 0);
    // causal rows see more the later they come, causal keys are seen by fewer
    (row ? pl.qraw : pl.kraw)[row ? tiles - 1 - tile : tile] = e;
  }
}

// Tiles by falling cost: a tile goes where its rank among all puts it.  A
// wave a tile, the others counted 64 at a time.
__global__ __launch_bounds__(NTH) void k_attn_order(int tq, int tk, AttnPlan pl) {
  const int lane = threadIdx.x % 64, n = blockIdx.y ? tk : tq;
  const int4* raw = blockIdx.y ? pl.kraw : pl.qraw;
  const int i = blockIdx.x * (NTH / 64) + threadIdx.x / 64;
  if (i >= n) return;
  const int4 e = raw[i];
  const int mine = e.z - e.y;
  int rank = 0;
  for (int b = 0; b < n; b += 64) {
    const int j = b + lane;
    const int4 o = raw[min(j, n - 1)];
    const int c = o.z - o.y;
    rank += __popcll(__ballot(j < n && (c > mine || (c == mine && j < i))));
  }
  if (lane == 0) (blockIdx.y ? pl.ktab : pl.qtab)[rank] = e;
}

}  // namespace

hipError_t launch_attn_plan(int Tq, int Tk, int ndoc, int causal, const int* cu_q, const int* cu_k,
                            const int* prefix, const AttnPlan& pl, hipStream_t s) {
  const int qb = (Tq + NTH - 1) / NTH, kb = (Tk + NTH - 1) / NTH;
  k_attn_plan<<<dim3(qb + kb), NTH, 0, s>>>(Tq, Tk, ndoc, causal, qb, cu_q, cu_k, prefix, pl);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || pl.qtab == pl.qraw) return e;
  const int tq = attn_tiles(Tq), tk = attn_tiles(Tk);
  k_attn_order<<<dim3((std::max(tq, tk) + NTH / 64 - 1) / (NTH / 64), 2), NTH, 0, s>>>(tq, tk, pl);
  return hipGetLastError();
}

}  // namespace poetx

// The mask of a packed batch as intervals (AttnPlan): documents, the causal
// bound and prefixes all leave every query one interval of keys, and every
// key one interval of queries.
#include <algorithm>

#include "attn.h"

namespace poetx {

namespace {

constexpr int NTH = 256;

// document of row t: the last d with cu[d] <= t, if it ends after t
// (offsets clamped to [0, T]); -1: none
__device__ __forceinline__ int doc_of(const int* cu, int ndoc, int t, int T) {
  int lo = 0, hi = ndoc + 1;  // cu[lo - 1] <= t < cu[hi] in sorted offsets
  while (lo < hi) {
    const int mid = (lo + hi) / 2;
    if (min(max(cu[mid], 0), T) <= t) lo = mid + 1;
    else hi = mid;
  }
  return lo >= 1 && lo <= ndoc ? lo - 1 : -1;
}

__global__ __launch_bounds__(NTH) void k_attn_plan(int Tq, int Tk, int ndoc, int causal,
                                                   const int* __restrict__ cu_q,
                                                   const int* __restrict__ cu_k,
                                                   const int* __restrict__ prefix, AttnPlan pl) {
  const long id = (long)blockIdx.x * NTH + threadIdx.x;
  if (id >= (long)Tq + Tk) return;
  const bool row = id < Tq;
  const int t = (int)(row ? id : id - Tq);
  const int d = doc_of(row ? cu_q : cu_k, ndoc, t, row ? Tq : Tk);
  int lo = 0, hi = 0, pos = 0;
  if (d >= 0) {
    const int q0 = min(max(cu_q[d], 0), Tq), q1 = min(max(cu_q[d + 1], q0), Tq);
    const int k0 = min(max(cu_k[d], 0), Tk), k1 = min(max(cu_k[d + 1], k0), Tk);
    const int pre = prefix ? min(max(prefix[d], 0), k1 - k0) : 0;
    if (row) {
      pos = k1 - (q1 - t);
      lo = k0;
      hi = causal ? max(min(pos + 1, k1), k0 + pre) : k1;
      if (hi <= lo) lo = hi = 0;
    } else {
      lo = causal && t >= k0 + pre ? max(q0, q1 - (k1 - t)) : q0;
      hi = q1;
      if (hi <= lo) lo = hi = 0;
    }
  }
  if (row) {
    pl.row_lo[t] = lo;
    pl.row_hi[t] = hi;
    pl.row_pos[t] = pos;
  } else {
    pl.key_lo[t] = lo;
    pl.key_hi[t] = hi;
  }
}

}  // namespace

hipError_t launch_attn_plan(int Tq, int Tk, int ndoc, int causal, const int* cu_q, const int* cu_k,
                            const int* prefix, const AttnPlan& pl, hipStream_t s) {
  const long n = (long)Tq + Tk;
  k_attn_plan<<<dim3((unsigned)((n + NTH - 1) / NTH)), NTH, 0, s>>>(Tq, Tk, ndoc, causal, cu_q,
                                                                    cu_k, prefix, pl);
  return hipGetLastError();
}

}  // namespace poetx

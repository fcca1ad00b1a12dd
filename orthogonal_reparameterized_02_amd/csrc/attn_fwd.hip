// Attention forward on MFMA tiles: one pass over the keys with the running
// maximum and sum of the softmax.
//
// A wave owns 32 query rows (their operand fragments stay in registers), a
// workgroup four such waves; key and value tiles of BN rows stream through
// two LDS buffers by direct loads, one barrier a tile.  Scores are formed
// transposed (attn_tile.h), so a lane owns one query: the maximum of a tile
// is 16 or 32 register operations and one exchange with the lane that holds
// the other keys, and the probabilities are the next product's operand
// without leaving their lane.
#include "attn_rows.h"
#include "attn_tile.h"

namespace poetx {

namespace {

constexpr int NW = 4;         // waves
constexpr int BM = 32 * NW;   // query rows a workgroup
// The running maximum moves only when a score passes it by more than this
// (log2): until then probabilities may reach 2^8, which float32 sums and bf16
// operands hold with the same relative error, and the accumulators need not
// be scaled again.
constexpr float SLACK = 8.0f;

template <typename T, int DP> struct FwdCfg {
  static constexpr int BN = sizeof(T) == 2 ? 64 : 32;
  static constexpr int TILE = BN * Tile<T, DP>::RB;
  static constexpr int LDS = 4 * TILE;  // two buffers of keys and values
};

template <typename T, int DP, int MODE>
__global__ __launch_bounds__(64 * NW, sizeof(T) == 4 && DP == 128 ? 1 : 2) void k_attn_fwd(AttnArgs a, int tiles) {
  using L = Tile<T, DP>;
  using C = FwdCfg<T, DP>;
  constexpr int BN = C::BN, NS = BN / 32;
  extern __shared__ __align__(16) char smem[];
  const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int w = xcd_order(blockIdx.x, gridDim.x);
  const int h = w / tiles, q0 = (tiles - 1 - w % tiles) * BM;  // long rows (causal) first
  const int hk = h / a.group;
  const T* qp = (const T*)a.q + (long)h * a.D;
  const T* kp = (const T*)a.k + (long)hk * a.D;
  const T* vp = (const T*)a.v + (long)hk * a.D;

  // this lane's query, the wave's and the workgroup's keys
  const int t = q0 + 32 * wave + (lane & 31);
  const bool in = t < a.Tq;
  const int lo = in ? a.pl.row_lo[t] : 0, hi = in ? a.pl.row_hi[t] : 0;
  const float pos = MODE == 2 && in ? (float)a.pl.row_pos[t] : 0.0f;
  const Span sp = span_of(lo, hi);
  int klo, khi;
  span_rows(a.pl.row_lo, a.pl.row_hi, q0, BM, a.Tq, lane, klo, khi);

  uint4 qf[L::KS];
  rows_to_regs<T>(qf, qp, a.ldq, q0 + 32 * wave, a.Tq, a.D, lane);
  Loader<T, DP, BN, NW> lk, lv;
  lk.init(a.ldk, a.D, wave, lane);
  lv.init(a.ldv, a.D, wave, lane);
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)smem;

  const ScoreArgs sa = score_args(a, h);
  f32x16_t o[L::NT];
#pragma unroll
  for (int i = 0; i < L::NT; ++i) o[i] = (f32x16_t){};
  float m = -INFINITY, l = 0.0f;  // m: the reference of the exponentials, log2

  if (klo < khi) {
    lk.load(kp, a.ldk, klo, khi, lds0);
    lv.load(vp, a.ldv, klo, khi, lds0 + 2 * C::TILE);
  }
  int buf = 0;
  for (int j0 = klo; j0 < khi; j0 += BN, buf ^= 1) {
    // this tile has landed, and every wave has left the other buffer
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (j0 + BN < khi) {
      lk.load(kp, a.ldk, j0 + BN, khi, lds0 + (buf ^ 1) * C::TILE);
      lv.load(vp, a.ldv, j0 + BN, khi, lds0 + (2 + (buf ^ 1)) * C::TILE);
    }
    if (sp.lo >= j0 + BN || sp.hi <= j0) continue;  // nothing here for this wave
    const char* kt = smem + buf * C::TILE;
    const char* vt = smem + (2 + buf) * C::TILE;

    f32x16_t s[NS];
#pragma unroll
    for (int n = 0; n < NS; ++n) {
      s[n] = (f32x16_t){};
#pragma unroll
      for (int ks = 0; ks < L::KS; ++ks)
        s[n] = mma16((const T*)nullptr, L::row_frag(kt, 32 * n, ks, lane), qf[ks], s[n]);
    }
    const int jl = j0 + 4 * (lane >> 5);  // key of register 0
    float top = -INFINITY;
    if constexpr (MODE != 0) {
      float unused;
#pragma unroll
      for (int n = 0; n < NS; ++n)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          s[n][i] = score2<T, MODE>(s[n][i], sa, pos - (float)(jl + 32 * n + 8 * (i / 4) + i % 4), unused);
    }
    if (sp.all_lo > j0 || sp.all_hi < j0 + BN) {  // some pair is hidden
      const uint32_t width = (uint32_t)(hi - lo);
#pragma unroll
      for (int n = 0; n < NS; ++n)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          s[n][i] = (uint32_t)(jl - lo + 32 * n + 8 * (i / 4) + i % 4) < width ? s[n][i] : -INFINITY;
    }
#pragma unroll
    for (int n = 0; n < NS; ++n)
#pragma unroll
      for (int i = 0; i < 16; ++i) top = fmaxf(top, s[n][i]);
    top = fmaxf(top, other_half(top));
    if constexpr (MODE == 0) top *= sa.c;
    if (__any(top > m + SLACK)) {
      const float m2 = fmaxf(m, top);
      const float f = m2 == -INFINITY ? 1.0f : exp2_hw(m - m2);
      m = m2;
      l *= f;
#pragma unroll
      for (int i = 0; i < L::NT; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) o[i][r] *= f;
    }
    const float ref = m == -INFINITY ? 0.0f : m;
#pragma unroll
    for (int n = 0; n < NS; ++n) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        s[n][i] = exp2_hw(MODE == 0 ? fmaf(s[n][i], sa.c, -ref) : s[n][i] - ref);
        l += s[n][i];
      }
#pragma unroll
      for (int u = 0; u < L::CSTEP; ++u) {
        const uint4 p = L::score_frag(s[n], u);
#pragma unroll
        for (int ct = 0; ct < L::NT; ++ct)
          o[ct] = mma16((const T*)nullptr, L::col_frag(vt, 32 * n, u, ct, lane), p, o[ct]);
      }
    }
  }

  l += other_half(l);
  const bool empty = lo >= hi;
  // Hidden keys enter the products as 0 times their value.  Where that left
  // anything that is not finite, the rows are formed again one at a time, from
  // what each sees alone.
  const float probe = empty ? 0.0f : finite_probe<L::NT>(o) + l * 0.0f;
  if (__any(probe != 0.0f)) {
    for (int r = 0; r < 32; ++r) {
      const int tr = q0 + 32 * wave + r;
      if (tr >= a.Tq) break;
      float lse;
      const float2 ov = attn_row<T>(qp + (long)tr * a.ldq, kp, a.ldk, vp, a.ldv, a.pl.row_lo[tr],
                                    a.pl.row_hi[tr], a.pl.row_pos[tr], a.D, a.scale, a.cap,
                                    a.slopes ? a.slopes[h] : 0.0f, lane, lse);
      st2((T*)a.o + (long)tr * a.ldo + (long)h * a.D, lane, a.D, ov);
      if (lane == 0) a.lse[(long)h * a.Tq + tr] = lse;
    }
    return;
  }
  const bool none = empty || l == 0.0f;
  if (in && lane < 32) a.lse[(long)h * a.Tq + t] = none ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * LN2;
  // an empty row of a tile that was not masked has sums of its own: cleared
  if (empty) {
#pragma unroll
    for (int i = 0; i < L::NT; ++i) o[i] = (f32x16_t){};
  }
  store_rowsT<L::NT>((T*)a.o + (long)(in ? t : 0) * a.ldo + (long)h * a.D, o, none ? 0.0f : 1.0f / l, a.D, in, lane);
}

template <typename T, int DP, int MODE> hipError_t fwd(const AttnArgs& a, hipStream_t s) {
  constexpr int lds = FwdCfg<T, DP>::LDS;
  const hipError_t e = lds_opt_in((const void*)k_attn_fwd<T, DP, MODE>, lds);
  if (e != hipSuccess) return e;
  const int tiles = (a.Tq + BM - 1) / BM;
  k_attn_fwd<T, DP, MODE><<<dim3((unsigned)tiles * a.Hq), 64 * NW, lds, s>>>(a, tiles);
  return hipGetLastError();
}

template <typename T, int DP> hipError_t fwd_mode(const AttnArgs& a, hipStream_t s) {
  if (a.slopes) return fwd<T, DP, 2>(a, s);
  return a.cap > 0.0f ? fwd<T, DP, 1>(a, s) : fwd<T, DP, 0>(a, s);
}

}  // namespace

template <typename T> hipError_t launch_attn_fwd(const AttnArgs& a, hipStream_t s) {
  return a.D <= 64 ? fwd_mode<T, 64>(a, s) : fwd_mode<T, 128>(a, s);
}

template hipError_t launch_attn_fwd<bf16>(const AttnArgs&, hipStream_t);
template hipError_t launch_attn_fwd<float>(const AttnArgs&, hipStream_t);

}  // namespace poetx

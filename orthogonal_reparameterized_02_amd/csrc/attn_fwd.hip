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
//
// bf16 rounds the probabilities to bf16 as that operand: o is off by 2.1e-3
// (2-norm) where its own rounding makes 1.6e-3.  In two parts, as decoding has
// them, they would cost a third product beside two: 95 -> 118 us for the 9
// documents below, 517 -> 709 us for the one, 610 -> 774 us capped.
//
// Measured (bf16, D 128): 8192 causal tokens in one document, 32 heads on 8,
// 515 us = 1.07 PFLOP/s, where the library's 8192^3 product reaches 1.30; with
// counters 533 us, matrix pipes busy 0.55 of the cycles at a clock that the
// power limit holds at 1.8 GHz, 1.5 in later launches.  In 9 documents 94 us =
// 0.75 PFLOP/s: a fifth of the wave slots stands empty at the starts and ends
// of the short loops.  Capped, 2048 queries on 16384 keys, 611 us = 0.84
// PFLOP/s: bound by vector instructions, three transcendentals a score (16
// issue cycles each) beside four others.
// With a window, 8192 tokens in 3 documents, window 1024, 4 sinks: 142 us = 0.79
// PFLOP/s of the products that are seen, 0.9 of those formed (a tile at either
// edge of the window is half hidden, the sinks' tile nearly); capped, 2048
// queries on 16384 keys, window 4096: 177 us = 0.78 PFLOP/s (207 us under the
// profiler: vector instructions issue in 0.56 of the cycles, matrix pipes are busy
// in 0.31, and the two hardly overlap), o off by 2.3e-3.
#include <algorithm>

#include "attn_rows.h"
#include "attn_tile.h"

namespace poetx {

namespace {

constexpr int NW = 4;         // waves
constexpr int BM = ATTN_BM;   // query rows a workgroup
static_assert(BM == 32 * NW, "a wave owns 32 rows");
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

// SINK: rows see the first keys of their document besides an interval
// (KeyTiles); one key tile more a loop.
template <typename T, int DP, int MODE, bool SINK>
__global__ __launch_bounds__(64 * NW, 2) void k_attn_fwd(AttnArgs a, int parts) {
  using L = Tile<T, DP>;
  using C = FwdCfg<T, DP>;
  constexpr int BN = C::BN, NS = BN / 32;
  // scores capped by r, no bias: the maximum is taken of the products (the cap
  // is monotone), a probability is exp2(fma(-2 cap, r, cap - reference))
  constexpr bool LATE = cap_by_r<T, MODE> && !(MODE & 2);
  extern __shared__ __align__(16) char smem[];
  const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  int h, part, tile;
  work_of(blockIdx.x, a.Hq, parts, h, part, tile);
  int q0, klo, khi;
  tile_entry(a.pl.qtab, tile, BM, a.Tq, a.Tk, q0, klo, khi);
  const int hk = h / a.group;
  const T* qp = (const T*)a.q + (long)h * a.D;
  const T* kp = (const T*)a.k + (long)hk * a.D;
  const T* vp = (const T*)a.v + (long)hk * a.D;

  int jb, je;  // this part's keys; the first tiles are on their way before all else
  KeyTiles kt;
  if constexpr (SINK) {
    kt.init(a.pl.qfar, q0 / BM, klo, khi, a.Tk, BN, parts, part);
    jb = kt.row(kt.nb, BN);
    je = kt.nb < kt.ne ? kt.end(kt.nb) : jb;
  } else {
    part_of((khi - klo + BN - 1) / BN, parts, part, jb, je);
    jb = klo + jb * BN;
    je = min(klo + je * BN, khi);
  }
  Loader<T, DP, BN, NW> lk, lv;
  lk.init(a.ldk, a.D, wave, lane);
  lv.init(a.ldv, a.D, wave, lane);
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)smem;
  if (jb < je) {
    lk.load(kp, a.ldk, jb, je, lds0);
    lv.load(vp, a.ldv, jb, je, lds0 + 2 * C::TILE);
  }

  // this lane's query and the wave's keys
  const int t = q0 + 32 * wave + (lane & 31);
  const bool in = t < a.Tq;
  const int tc = min(t, a.Tq - 1);
  const int rlo = a.pl.row_lo[tc], rhi = a.pl.row_hi[tc], rpos = MODE & 2 ? a.pl.row_pos[tc] : 0;
  const int lo = in ? rlo : 0, hi = in ? rhi : 0;
  const Span sp = span_of(lo, hi);
  int2 sink = make_int2(0, 0);
  Span ssp = {};
  if constexpr (SINK) {
    const int2 rs = a.pl.row_sink[tc];
    sink = make_int2(in ? rs.x : 0, in ? rs.y : 0);
    ssp = span_of(sink.x, sink.y);
  }

  uint4 qf[L::KS];
  rows_to_regs<T>(qf, qp, a.ldq, q0 + 32 * wave, a.Tq, a.D, lane);

  const uint32_t rlane = L::row_lane(lane), clane = L::col_lane(lane);
  const ScoreArgs sa = score_args<T, MODE>(a, h);
  f32x16_t o[L::NT];
#pragma unroll
  for (int i = 0; i < L::NT; ++i) o[i] = (f32x16_t){};
  float m = -INFINITY, l = 0.0f;  // m: the reference of the exponentials, log2

  wait_loads();
  int buf = 0;
  for (int j0 = jb, n = SINK ? kt.nb : 0; SINK ? n < kt.ne : j0 < je; j0 = SINK ? kt.row(n + 1, BN) : j0 + BN, ++n, buf ^= 1) {
    // this tile has landed, and every wave has left the other buffer
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (SINK ? n + 1 < kt.ne : j0 + BN < je) {
      const int jn = SINK ? kt.row(n + 1, BN) : j0 + BN, jne = SINK ? kt.end(n + 1) : je;
      lk.load(kp, a.ldk, jn, jne, lds0 + (buf ^ 1) * C::TILE);
      lv.load(vp, a.ldv, jn, jne, lds0 + (2 + (buf ^ 1)) * C::TILE);
    }
    const bool far = SINK && n < kt.far;
    // nothing here for this wave
    if ((far || sp.lo >= j0 + BN || sp.hi <= j0) && (!SINK || ssp.lo >= j0 + BN || ssp.hi <= j0)) continue;
    const uint32_t kr = rlane + buf * C::TILE, vc = clane + (2 + buf) * C::TILE;

    f32x16_t s[NS];
#pragma unroll
    for (int n = 0; n < NS; ++n) s[n] = (f32x16_t){};
    {
      Pipe<NS * L::KS, 4> kp_;
      const auto ld = [&](int i) { return L::row_frag(smem, kr, 32 * (i / L::KS), i % L::KS); };
      kp_.start(ld);
      kp_.run(ld, [&](int i, uint4 f) { s[i / L::KS] = mma16((const T*)nullptr, f, qf[i % L::KS], s[i / L::KS]); });
    }
    // the first value fragments travel while the softmax is formed
    Pipe<NS * L::CSTEP * L::NT, 4> vp_;
    const auto ldv = [&](int i) {
      return L::col_frag(smem, vc, 32 * (i / (L::CSTEP * L::NT)), i / L::NT % L::CSTEP, i % L::NT);
    };
    vp_.start(ldv);
    const int jl = j0 + 4 * (lane >> 5);  // key of register 0
    float top = -INFINITY;
    if constexpr (MODE != 0 && !LATE) {
      const float d0 = (float)(rpos - jl);  // exact: rows past 2^24 are no float32 numbers
      float unused;
#pragma unroll
      for (int n = 0; n < NS; ++n)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          s[n][i] = score2<T, MODE>(s[n][i], sa, d0 - (float)(32 * n + 8 * (i / 4) + i % 4), unused);
    }
    const bool masked = far || sp.all_lo > j0 || sp.all_hi < j0 + BN;  // some pair is hidden
    Seen seen = {jl - lo, jl - sink.x, (uint32_t)(hi - lo), (uint32_t)(sink.y - sink.x)};
    if constexpr (SINK)
      if (far) seen = {jl - sink.x, 0, sink.x == kt.flo ? (uint32_t)(sink.y - sink.x) : 0, 0};
    const auto sees = [&](int j) { return SINK ? seen.either(j) : seen(j); };
    if (masked) {
#pragma unroll
      for (int n = 0; n < NS; ++n)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          s[n][i] = sees(32 * n + 8 * (i / 4) + i % 4) ? s[n][i] : -INFINITY;
    }
#pragma unroll
    for (int n = 0; n < NS; ++n)
#pragma unroll
      for (int i = 0; i < 16; ++i) top = fmaxf(top, s[n][i]);
    top = fmaxf(top, other_half(top));
    if constexpr (MODE == 0) top *= sa.c;
    // a product of -inf is -cap like any other; where every key is hidden, -cap
    // is no more than the scores to come
    if constexpr (LATE) top = fmaf(-2.0f * sa.capl, cap_r(top, sa), sa.capl);
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
    for (int n = 0; n < NS; ++n)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        if constexpr (LATE) s[n][i] = exp2_hw(fmaf(-2.0f * sa.capl, cap_r(s[n][i], sa), sa.capl - ref));
        else s[n][i] = exp2_hw(MODE == 0 ? fmaf(s[n][i], sa.c, -ref) : s[n][i] - ref);
      }
    if constexpr (LATE) {
      if (masked) {  // -inf is capped like any other product
#pragma unroll
        for (int n = 0; n < NS; ++n)
#pragma unroll
          for (int i = 0; i < 16; ++i) s[n][i] = sees(32 * n + 8 * (i / 4) + i % 4) ? s[n][i] : 0.0f;
      }
    }
#pragma unroll
    for (int n = 0; n < NS; ++n)
#pragma unroll
      for (int i = 0; i < 16; ++i) l += s[n][i];
    uint4 p;
    vp_.run(ldv, [&](int i, uint4 f) {
      if (i % L::NT == 0) p = L::score_frag(s[i / (L::CSTEP * L::NT)], i / L::NT % L::CSTEP);
      o[i % L::NT] = mma16((const T*)nullptr, f, p, o[i % L::NT]);
    });
  }

  l += other_half(l);
  const bool empty = lo >= hi;
  if (empty) {  // beside rows that see a whole tile it has sums of its own
    m = -INFINITY;
    l = 0.0f;
#pragma unroll
    for (int i = 0; i < L::NT; ++i) o[i] = (f32x16_t){};
  }
  float* po = a.part + ((long)part * a.Hq + h) * a.Tq * a.D;
  float* pm = a.part + (long)parts * a.Hq * a.Tq * a.D + ((long)part * a.Hq + h) * a.Tq * 2;
  // Hidden keys enter the products as 0 times their value.  Where that left
  // anything that is not finite, the rows are formed again one at a time, from
  // what each sees alone.
  if (__any(finite_probe<L::NT>(o) + l * 0.0f != 0.0f)) {
    for (int r = 0; r < 32; ++r) {
      const int tr = q0 + 32 * wave + r;
      if (tr >= a.Tq) break;
      float mr, lr;
      float2 ov;
      const float slope = a.slopes ? a.slopes[h] : 0.0f;
      if constexpr (SINK) {
        mr = -INFINITY, lr = 0.0f, ov = make_float2(0.0f, 0.0f);
        const int2 f = kt.far_keys(BN), w = kt.near_keys(BN), rs = a.pl.row_sink[tr];
        const auto more = [&](int x, int y) {
          attn_row_more<T>(qp + (long)tr * a.ldq, kp, a.ldk, vp, a.ldv, x, y, a.pl.row_pos[tr], a.D, a.scale, a.cap, slope,
                           lane, mr, lr, ov);
        };
        if (rs.x == kt.flo) more(max(rs.x, f.x), min(rs.y, f.y));
        more(max(rs.x, w.x), min(rs.y, w.y));
        more(max(a.pl.row_lo[tr], w.x), min(a.pl.row_hi[tr], w.y));
      } else {
        ov = attn_row<T>(qp + (long)tr * a.ldq, kp, a.ldk, vp, a.ldv, max(a.pl.row_lo[tr], jb),
                         min(a.pl.row_hi[tr], je), a.pl.row_pos[tr], a.D, a.scale, a.cap, slope, lane, mr, lr);
      }
      if (parts == 1) {
        const float inv = lr == 0.0f ? 0.0f : 1.0f / lr;
        st2((T*)a.o + (long)tr * a.ldo + (long)h * a.D, lane, a.D, make_float2(ov.x * inv, ov.y * inv));
        if (lane == 0) a.lse[(long)h * a.Tq + tr] = lr == 0.0f ? -INFINITY : mr + __logf(lr);
      } else {
        st2(po + (long)tr * a.D, lane, a.D, ov);
        if (lane == 0) {
          pm[2 * (long)tr] = mr * LOG2E;
          pm[2 * (long)tr + 1] = lr;
        }
      }
    }
    return;
  }
  const long tt = in ? t : 0;
  if (parts > 1) {
    if (in && lane < 32) {
      pm[2 * tt] = m;
      pm[2 * tt + 1] = l;
    }
    store_rowsT<L::NT>(po + tt * a.D, o, 1.0f, a.D, in, lane);
    return;
  }
  const bool none = l == 0.0f;
  if (in && lane < 32) a.lse[(long)h * a.Tq + t] = none ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * LN2;
  store_rowsT<L::NT>((T*)a.o + tt * a.ldo + (long)h * a.D, o, none ? 0.0f : 1.0f / l, a.D, in, lane);
}

// joins the parts of the query rows, in part order: eight elements a thread
template <typename T>
__global__ __launch_bounds__(256) void k_attn_fwd_join(AttnArgs a, int parts) {
  const int per = a.D / 8, r = threadIdx.x / per, e = (threadIdx.x - r * per) * 8;
  const int h = blockIdx.y, t = blockIdx.x * (256 / per) + r;
  if (r >= 256 / per || t >= a.Tq) return;
  const long row = (long)h * a.Tq + t, stride = (long)a.Hq * a.Tq;
  const float2* pm = reinterpret_cast<const float2*>(a.part + parts * stride * a.D) + row;
  float m = -INFINITY, l = 0.0f;
  for (int s = 0; s < parts; ++s) m = fmaxf(m, pm[s * stride].x);
  const float ref = m == -INFINITY ? 0.0f : m;
  float o[8] = {};
  for (int s = 0; s < parts; ++s) {
    const float2 ml = pm[s * stride];
    const float f = exp2_hw(ml.x - ref);
    const float4* p = reinterpret_cast<const float4*>(a.part + (s * stride + row) * a.D + e);
    const float4 x = p[0], y = p[1];
    l = fmaf(f, ml.y, l);
    const float v[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] = fmaf(f, v[i], o[i]);
  }
  const float inv = l == 0.0f ? 0.0f : 1.0f / l;
  T* out = (T*)a.o + (long)t * a.ldo + (long)h * a.D + e;
#pragma unroll
  for (int i = 0; i < 8; ++i) St<T>::st(out + i, o[i] * inv);
  if (e == 0) a.lse[row] = l == 0.0f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * LN2;
}

template <typename T> int fwd_parts(const AttnArgs& a) {
  return parts_for<T>((long)attn_tiles(a.Tq) * a.Hq, loop_rows(a.Tk, a.Tq, a.ndoc, a.reach()), 64);
}

template <typename T, int DP, int MODE, bool SINK> hipError_t fwd(const AttnArgs& a, hipStream_t s) {
  constexpr int lds = FwdCfg<T, DP>::LDS;
  const hipError_t e = lds_opt_in((const void*)k_attn_fwd<T, DP, MODE, SINK>, lds);
  if (e != hipSuccess) return e;
  const int tiles = attn_tiles(a.Tq), parts = fwd_parts<T>(a);
  k_attn_fwd<T, DP, MODE, SINK><<<dim3((unsigned)tiles * a.Hq * parts), 64 * NW, lds, s>>>(a, parts);
  const hipError_t e2 = hipGetLastError();
  if (e2 != hipSuccess || parts == 1) return e2;
  const int rows = 256 / (a.D / 8);
  k_attn_fwd_join<T><<<dim3((a.Tq + rows - 1) / rows, a.Hq), 256, 0, s>>>(a, parts);
  return hipGetLastError();
}

template <typename T, int DP> hipError_t fwd_mode(const AttnArgs& a, hipStream_t s) {
  return by_mode<T>(a.slopes, a.cap, [&](auto mode) {
    constexpr int MODE = decltype(mode)::value;
    return a.sinks ? fwd<T, DP, MODE, true>(a, s) : fwd<T, DP, MODE, false>(a, s);
  });
}

}  // namespace

template <typename T> size_t attn_fwd_part_bytes(const AttnArgs& a) {
  const int parts = fwd_parts<T>(a);
  return parts == 1 ? 0 : (size_t)parts * a.Hq * a.Tq * (a.D + 2) * 4;
}

template <typename T> hipError_t launch_attn_fwd(const AttnArgs& a, hipStream_t s) {
  return a.D <= 64 ? fwd_mode<T, 64>(a, s) : fwd_mode<T, 128>(a, s);
}

template size_t attn_fwd_part_bytes<bf16>(const AttnArgs&);
template size_t attn_fwd_part_bytes<float>(const AttnArgs&);
template hipError_t launch_attn_fwd<bf16>(const AttnArgs&, hipStream_t);
template hipError_t launch_attn_fwd<float>(const AttnArgs&, hipStream_t);

}  // namespace poetx

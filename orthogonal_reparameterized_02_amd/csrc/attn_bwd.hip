// Attention backward on MFMA tiles, in two passes without atomics: dq (a
// wave owns 32 queries and walks their keys), then dk and dv (a wave owns 32
// keys and walks the queries that see them, every query head of the group in
// turn).  Both form the scores again from q, k and lse.  The second forming
// costs two products in seven; adding dq tiles from the second pass into
// memory instead would need atomics, whose order changes the sums.
//   p = exp2(s2 - lse2),  ds = p (dp - delta) (1 - t^2),
//   dq = scale ds k,  dk = scale ds^T q,  dv = p^T dout
// -delta is the initial value of the dp accumulators; scale multiplies the
// finished sums.  In bf16, p and ds are rounded to bf16 as matrix operands
// (float32 operands would take eight times as long), and delta comes from the
// stored, rounded o: of a relative error of 2.6e-3 in dq and dk, the rounding
// of the result itself makes 1.7e-3, that of ds as much again, delta 1.1e-3.
// ds in two bf16 parts would leave 1.9e-3 (with a bias 2.3e-3), for two products
// more beside seven: a training pass of 9 documents 414 -> 462 us, of one 2235
// -> 2591 us.
//
// Measured (bf16, D 128, 32 heads on 8): 8192 causal tokens in one document
// 1.75 ms for both passes, dq at 1.19 and dk, dv at 1.06 PFLOP/s of the products
// they form, at the power limit; in 9 documents 320 us, a fifth of the wave
// slots empty as in the forward pass.  float32, D 64, two documents of 1024,
// 16 heads on 4, capped: 225 us, a third of the float32 matrix rate.
#include <algorithm>

#include "attn_rows.h"
#include "attn_tile.h"

namespace poetx {

namespace {

constexpr int NW = 4;         // waves
constexpr int BM = ATTN_BM;   // rows a workgroup owns
static_assert(BM == 32 * NW, "a wave owns 32 of them");

template <typename T, int DP> struct DqCfg {
  static constexpr int BN = sizeof(T) == 2 ? 64 : 32;  // rows of a streamed tile
  static constexpr int TILE = BN * Tile<T, DP>::RB;
  static constexpr int LDS = 4 * TILE;
  static constexpr int OCC = sizeof(T) == 2 || DP == 64 ? 2 : 1;  // waves a SIMD, by registers
};

// Second pass.  NQ = 2: two waves take the same 32 keys and every other 32
// queries, and add their sums at the end: eight waves, one workgroup a CU,
// whose loop, which decides when the last workgroup ends, is half as long.
// NQ = 1: four waves, two workgroups a CU, one's start and end beside the
// other's loop.  A wave holds two 32-row sums, keys and values; with 128 bf16
// columns that is a few registers more than two waves a SIMD have: the values
// stay in LDS, and three forms still spill one to three registers (NQ = 1
// plain; cap and bias together).
template <typename T, int DP, int NQ> struct DkvCfg {
  static constexpr bool VLDS = sizeof(T) == 2 && DP == 128;
  static constexpr int VS = 64;                        // a wave's load fills 64 values
  static constexpr int ROWV = 3 * VS * 4;              // lse2, delta, position of a tile's queries
  static constexpr int BQ = 32 * NQ;                   // queries of a streamed tile
  static constexpr int QTILE = BQ * Tile<T, DP>::RB;
  static constexpr int VTILE = VLDS ? BM * Tile<T, DP>::RB : 0;
  static constexpr int JOIN = NQ == 2 ? NW * 2 * 32 * DP * 4 : 0;
  static constexpr int LDS = std::max(4 * QTILE + 2 * ROWV + VTILE, JOIN);
  static constexpr int OCC = DqCfg<T, DP>::OCC;
};

__device__ __forceinline__ float dot8(const bf16*, uint4 a, uint4 b) {
  const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    s = fmaf(__uint_as_float(x[i] << 16), __uint_as_float(y[i] << 16), s);
    s = fmaf(__uint_as_float(x[i] & 0xffff0000u), __uint_as_float(y[i] & 0xffff0000u), s);
  }
  return s;
}
__device__ __forceinline__ float dot8(const float*, uint4 a, uint4 b) {
  float s = __uint_as_float(a.x) * __uint_as_float(b.x);
  s = fmaf(__uint_as_float(a.y), __uint_as_float(b.y), s);
  s = fmaf(__uint_as_float(a.z), __uint_as_float(b.z), s);
  return fmaf(__uint_as_float(a.w), __uint_as_float(b.w), s);
}

// dq, and for the second pass delta = dout . o and lse2 = lse log2e of every
// query (lse2 = +inf where lse = -inf: such a query's p is 0)
template <typename T, int DP, int MODE>
__global__ __launch_bounds__(64 * NW, (DqCfg<T, DP>::OCC)) void k_attn_dq(AttnArgs a, int parts) {
  using L = Tile<T, DP>;
  using C = DqCfg<T, DP>;
  constexpr float FACTOR = cap_factor<T, MODE>;
  constexpr int BN = C::BN, NS = BN / 32;
  extern __shared__ __align__(16) char smem[];
  const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  int h, part, tile;
  work_of(blockIdx.x, a.Hq, parts, h, part, tile);
  int q0, klo, khi;
  tile_entry(a.pl.qtab, tile, BM, a.Tq, a.Tk, q0, klo, khi);
  const int hk = h / a.group, r0 = q0 + 32 * wave;
  const T* qp = (const T*)a.q + (long)h * a.D;
  const T* kp = (const T*)a.k + (long)hk * a.D;
  const T* vp = (const T*)a.v + (long)hk * a.D;
  const T* dop = (const T*)a.dout + (long)h * a.D;
  const T* op = (const T*)a.o + (long)h * a.D;

  int jb, je;  // this part's keys; the first tiles are on their way before all else
  part_of((khi - klo + BN - 1) / BN, parts, part, jb, je);
  jb = klo + jb * BN;
  je = min(klo + je * BN, khi);
  Loader<T, DP, BN, NW> lk, lv;
  lk.init(a.ldk, a.D, wave, lane);
  lv.init(a.ldv, a.D, wave, lane);
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)smem;
  if (jb < je) {
    lk.load(kp, a.ldk, jb, je, lds0);
    lv.load(vp, a.ldv, jb, je, lds0 + 2 * C::TILE);
  }

  const int t = r0 + (lane & 31);
  const bool in = t < a.Tq;
  const int tc = min(t, a.Tq - 1);
  const int rlo = a.pl.row_lo[tc], rhi = a.pl.row_hi[tc], rpos = MODE & 2 ? a.pl.row_pos[tc] : 0;
  const int lo = in ? rlo : 0, hi = in ? rhi : 0;
  const Span sp = span_of(lo, hi);

  uint4 qf[L::KS], dof[L::KS];
  rows_to_regs<T>(dof, dop, a.lddo, r0, a.Tq, a.D, lane);
  float delta = 0.0f;
  {
    uint4 of[L::KS];
    rows_to_regs<T>(of, op, a.ldo, r0, a.Tq, a.D, lane);
#pragma unroll
    for (int ks = 0; ks < L::KS; ++ks) delta += dot8((const T*)nullptr, dof[ks], of[ks]);
  }
  delta += other_half(delta);
  const float lse = a.lse[(long)h * a.Tq + tc];
  const float lse2 = lse == -INFINITY ? INFINITY : lse * LOG2E;
  if (in && lane < 32 && part == 0) {
    a.delta[(long)h * a.Tq + t] = delta;
    a.lse2[(long)h * a.Tq + t] = lse2;
  }
  rows_to_regs<T>(qf, qp, a.ldq, r0, a.Tq, a.D, lane);

  const uint32_t rlane = L::row_lane(lane), clane = L::col_lane(lane);
  const ScoreArgs sa = score_args<T, MODE>(a, h);
  f32x16_t dq[L::NT];
#pragma unroll
  for (int i = 0; i < L::NT; ++i) dq[i] = (f32x16_t){};

  wait_loads();
  int buf = 0;
  for (int j0 = jb; j0 < je; j0 += BN, buf ^= 1) {
    // this tile has landed, and every wave has left the other buffer
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (j0 + BN < je) {
      lk.load(kp, a.ldk, j0 + BN, je, lds0 + (buf ^ 1) * C::TILE);
      lv.load(vp, a.ldv, j0 + BN, je, lds0 + (2 + (buf ^ 1)) * C::TILE);
    }
    const uint32_t kr = rlane + buf * C::TILE, vr = kr + 2 * C::TILE, kc = clane + buf * C::TILE;
#pragma unroll
    for (int n = 0; n < NS; ++n) {
      const int jn = j0 + 32 * n;
      if (sp.lo >= jn + 32 || sp.hi <= jn) continue;  // nothing here for this wave
      f32x16_t s = {}, dp;
#pragma unroll
      for (int i = 0; i < 16; ++i) dp[i] = -delta;
      {
        Pipe<2 * L::KS, 4> pp;
        const auto ld = [&](int i) {
          return L::row_frag(smem, i < L::KS ? kr : vr, 32 * n, i % L::KS);
        };
        pp.start(ld);
        pp.run(ld, [&](int i, uint4 f) {
          if (i < L::KS) s = mma16((const T*)nullptr, f, qf[i], s);
          else dp = mma16((const T*)nullptr, f, dof[i - L::KS], dp);
        });
      }
      Pipe<L::CSTEP * L::NT, 4> cp;
      const auto ldc = [&](int i) { return L::col_frag(smem, kc, 32 * n, i / L::NT, i % L::NT); };
      cp.start(ldc);
      const int jl = jn + 4 * (lane >> 5);  // key of register 0
      const float d0 = (float)(rpos - jl);  // exact: rows past 2^24 are no float32 numbers
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        float deriv;
        if constexpr (MODE == 0) s[i] = exp2_hw(fmaf(s[i], sa.c, -lse2)) * dp[i];
        else s[i] = exp2_hw(score2<T, MODE>(s[i], sa, d0 - (float)(8 * (i / 4) + i % 4), deriv) - lse2) * dp[i];
        if constexpr (MODE & 1) s[i] *= deriv;
      }
      if (sp.all_lo > jn || sp.all_hi < jn + 32) {  // some pair is hidden
        const uint32_t width = (uint32_t)(hi - lo);
#pragma unroll
        for (int i = 0; i < 16; ++i)
          s[i] = (uint32_t)(jl - lo + 8 * (i / 4) + i % 4) < width ? s[i] : 0.0f;
      }
      uint4 p;
      cp.run(ldc, [&](int i, uint4 f) {
        if (i % L::NT == 0) p = L::score_frag(s, i / L::NT);
        dq[i % L::NT] = mma16((const T*)nullptr, f, p, dq[i % L::NT]);
      });
    }
  }

  const bool empty = lo >= hi;
  if (empty) {  // beside rows that see a whole tile it has sums of its own
#pragma unroll
    for (int i = 0; i < L::NT; ++i) dq[i] = (f32x16_t){};
  }
  float* pq = a.part + (long)part * a.Tq * a.Hq * a.D + (long)h * a.D;
  const long ldp = (long)a.Hq * a.D;
  // as in the forward pass: what is not finite is formed again row by row
  if (__any(finite_probe<L::NT>(dq) != 0.0f)) {
    for (int r = 0; r < 32; ++r) {
      const int tr = r0 + r;
      if (tr >= a.Tq) break;
      const float2 x = ld2(dop + (long)tr * a.lddo, lane, a.D), y = ld2(op + (long)tr * a.ldo, lane, a.D);
      const float2 g = attn_row_dq<T>(qp + (long)tr * a.ldq, dop + (long)tr * a.lddo, kp, a.ldk, vp, a.ldv,
                                      max(a.pl.row_lo[tr], jb), min(a.pl.row_hi[tr], je), a.pl.row_pos[tr],
                                      a.D, a.scale, a.cap, a.slopes ? a.slopes[h] : 0.0f,
                                      a.lse[(long)h * a.Tq + tr], wave_sum(x.x * y.x + x.y * y.y), lane);
      if (parts > 1) st2(pq + tr * ldp, lane, a.D, g);
      else st2((T*)a.dq + (long)tr * a.lddq + (long)h * a.D, lane, a.D, make_float2(g.x * a.scale, g.y * a.scale));
    }
    return;
  }
  const long tt = in ? t : 0;
  if (parts > 1) store_rowsT<L::NT>(pq + tt * ldp, dq, FACTOR, a.D, in, lane);
  else store_rowsT<L::NT>((T*)a.dq + tt * a.lddq + (long)h * a.D, dq, a.scale * FACTOR, a.D, in, lane);
}

// dk and dv
template <typename T, int DP, int MODE, int NQ>
__global__ __launch_bounds__(64 * NW * NQ, (DkvCfg<T, DP, NQ>::OCC)) void k_attn_dkv(AttnArgs a, int parts) {
  using L = Tile<T, DP>;
  using C = DkvCfg<T, DP, NQ>;
  constexpr float FACTOR = cap_factor<T, MODE>;
  constexpr int BN = C::BQ, NWA = NW * NQ;
  extern __shared__ __align__(16) char smem[];
  const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  // 32 keys; 32 queries of a tile.  Wave w runs on SIMD w % 4: near the
  // diagonal, where the later keys have nothing to do, every SIMD then still
  // has a wave of the earlier ones.
  const int wk = wave / NQ, wq = wave % NQ;
  int hk, part, tile;
  work_of(blockIdx.x, a.Hkv, parts, hk, part, tile);
  int k0, qlo, qhi;
  tile_entry(a.pl.ktab, tile, BM, a.Tk, a.Tq, k0, qlo, qhi);
  const int r0 = k0 + 32 * wk;
  const T* kp = (const T*)a.k + (long)hk * a.D;
  const T* vp = (const T*)a.v + (long)hk * a.D;

  Loader<T, DP, BN, NWA> lq, lo_;
  lq.init(a.ldq, a.D, wave, lane);
  lo_.init(a.lddo, a.D, wave, lane);
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)smem;
  // tile n: query head n / per of the group, query rows from qlo + BN (n % per)
  const int per = (qhi - qlo + BN - 1) / BN;
  int nb, ne;  // this part's tiles
  part_of(per * a.group, parts, part, nb, ne);
  auto load = [&](int h, int i0, int buf) {
    lq.load((const T*)a.q + (long)h * a.D, a.ldq, i0, qhi, lds0 + buf * C::QTILE);
    lo_.load((const T*)a.dout + (long)h * a.D, a.lddo, i0, qhi, lds0 + (2 + buf) * C::QTILE);
    // one value a query: a dword a lane, wave by wave
    if (wave < (MODE & 2 ? 3 : 2)) {
      const float* src = wave == 0 ? a.lse2 + (long)h * a.Tq : wave == 1 ? a.delta + (long)h * a.Tq
                                                                         : (const float*)a.pl.row_pos;
      const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
          (void*)(src + i0), (short)0, min(qhi - i0, BN) * 4, 0x00020000);
      const uint32_t m0v = __builtin_amdgcn_readfirstlane(lds0 + 4 * C::QTILE + buf * C::ROWV + wave * C::VS * 4);
      asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds" ::"s"(m0v),
                   "v"(lane < BN ? lane * 4 : 0x60000000), "s"(rs)
                   : "memory");
    }
  };

  int h = hk * a.group, i0 = qlo;  // of the current tile
  if (nb < ne) {
    h += nb / per;
    i0 += nb % per * BN;
    load(h, i0, 0);
  }

  const int t = r0 + (lane & 31);
  const bool in = t < a.Tk;
  const int tc = min(t, a.Tk - 1);
  const int rlo = a.pl.key_lo[tc], rhi = a.pl.key_hi[tc];
  const int lo = in ? rlo : 0, hi = in ? rhi : 0;
  const Span sp = span_of(lo, hi);

  uint4 kf[L::KS], vf[C::VLDS ? 1 : L::KS];
  rows_to_regs<T>(kf, kp, a.ldk, r0, a.Tk, a.D, lane);
  // lane offsets into this wave's 32 queries of a tile, and its values
  const uint32_t rlane = L::row_lane(lane) + 32 * wq * L::RB, clane = L::col_lane(lane) + 32 * wq * L::RB;
  const uint32_t vr = L::row_lane(lane) + 4 * C::QTILE + 2 * C::ROWV + 32 * wk * L::RB;
  if constexpr (C::VLDS) {
    Loader<T, DP, BM, NWA> lv;
    lv.init(a.ldv, a.D, wave, lane);
    lv.load(vp, a.ldv, k0, a.Tk, lds0 + 4 * C::QTILE + 2 * C::ROWV);
  } else {
    rows_to_regs<T>(vf, vp, a.ldv, r0, a.Tk, a.D, lane);
  }
  f32x16_t dk[L::NT], dv[L::NT];
#pragma unroll
  for (int i = 0; i < L::NT; ++i) dk[i] = dv[i] = (f32x16_t){};

  wait_loads();  // also where there is no work: no load may outlive its workgroup
  int buf = 0;
  for (int n = nb; n < ne; ++n, buf ^= 1) {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    const int hc = h, in0 = i0 + 32 * wq;
    i0 += BN;
    if (i0 >= qhi) {
      i0 = qlo;
      ++h;
    }
    if (n + 1 < ne) load(h, i0, buf ^ 1);
    const ScoreArgs sa = score_args<T, MODE>(a, hc);
    const uint32_t qr = rlane + buf * C::QTILE, qc = clane + buf * C::QTILE;
    const uint32_t dr = qr + 2 * C::QTILE, dc = qc + 2 * C::QTILE;
    const float* rv = reinterpret_cast<const float*>(smem + 4 * C::QTILE + buf * C::ROWV);
    if (sp.lo >= in0 + 32 || sp.hi <= in0) continue;  // nothing here for this wave
    const float* row = rv + 32 * wq + 4 * (lane >> 5);  // quad g: row[8 g .. 8 g + 3]
    f32x16_t s = {}, dp, p;
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const float4 d = *reinterpret_cast<const float4*>(row + C::VS + 8 * g);
      dp[4 * g] = -d.x, dp[4 * g + 1] = -d.y, dp[4 * g + 2] = -d.z, dp[4 * g + 3] = -d.w;
    }
    {
      Pipe<L::KS, 4> sp_;
      const auto ld = [&](int i) { return L::row_frag(smem, qr, 0, i); };
      sp_.start(ld);
      sp_.run(ld, [&](int i, uint4 f) { s = mma16((const T*)nullptr, f, kf[i], s); });
    }
    if constexpr (C::VLDS) {
      Pipe<2 * L::KS, 8> dp_;  // dout and value fragments in turn
      const auto ld = [&](int i) {
        return L::row_frag(smem, i % 2 ? vr : dr, 0, i / 2);
      };
      uint4 of;
      dp_.start(ld);
      dp_.run(ld, [&](int i, uint4 f) {
        if (i % 2 == 0) of = f;
        else dp = mma16((const T*)nullptr, of, f, dp);
      });
    } else {
      Pipe<L::KS, 4> dp_;
      const auto ld = [&](int i) { return L::row_frag(smem, dr, 0, i); };
      dp_.start(ld);
      dp_.run(ld, [&](int i, uint4 f) { dp = mma16((const T*)nullptr, f, vf[i], dp); });
    }
    const int il = in0 + 4 * (lane >> 5);  // query of register 0
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const float4 e4 = *reinterpret_cast<const float4*>(row + 8 * g);
      const float e[4] = {e4.x, e4.y, e4.z, e4.w};
      int4 pq = make_int4(0, 0, 0, 0);
      if constexpr (MODE & 2) pq = *reinterpret_cast<const int4*>(row + 2 * C::VS + 8 * g);
      const int ps[4] = {pq.x, pq.y, pq.z, pq.w};
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int i = 4 * g + x;
        float deriv;
        if constexpr (MODE == 0) p[i] = exp2_hw(fmaf(s[i], sa.c, -e[x]));
        else p[i] = exp2_hw(score2<T, MODE>(s[i], sa, (float)(ps[x] - t), deriv) - e[x]);
        s[i] = p[i] * dp[i];
        if constexpr (MODE & 1) s[i] *= deriv;
      }
    }
    if (sp.all_lo > in0 || sp.all_hi < in0 + 32) {  // some pair is hidden
      const uint32_t width = (uint32_t)(hi - lo);
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const bool seen = (uint32_t)(il - lo + 8 * (i / 4) + i % 4) < width;
        p[i] = seen ? p[i] : 0.0f;
        s[i] = seen ? s[i] : 0.0f;
      }
    }
    {
      constexpr int H = L::NT;  // dv and dk products of one fragment of p and ds
      Pipe<2 * L::CSTEP * H, 4> cp;
      const auto ld = [&](int i) {
        return L::col_frag(smem, i % (2 * H) < H ? dc : qc, 0, i / (2 * H), i % H);
      };
      cp.start(ld);
      uint4 f2;
      cp.run(ld, [&](int i, uint4 f) {
        if (i % H == 0) f2 = L::score_frag(i % (2 * H) < H ? p : s, i / (2 * H));
        f32x16_t& acc = i % (2 * H) < H ? dv[i % H] : dk[i % H];
        acc = mma16((const T*)nullptr, f, f2, acc);
      });
    }
  }

  if constexpr (NQ == 2) {
    __syncthreads();
    float* red = reinterpret_cast<float*>(smem) + wk * (2 * 32 * DP) + lane;
    if (wq == 1) {
#pragma unroll
      for (int i = 0; i < L::NT; ++i)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          red[64 * (16 * i + r)] = dk[i][r];
          red[64 * (16 * (L::NT + i) + r)] = dv[i][r];
        }
    }
    __syncthreads();
    if (wq == 1) return;
#pragma unroll
    for (int i = 0; i < L::NT; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        dk[i][r] += red[64 * (16 * i + r)];
        dv[i][r] += red[64 * (16 * (L::NT + i) + r)];
      }
  }

  const bool empty = lo >= hi;
  if (empty) {  // beside rows that see a whole tile it has sums of its own
#pragma unroll
    for (int i = 0; i < L::NT; ++i) dk[i] = dv[i] = (f32x16_t){};
  }
  const long ldp = (long)a.Hkv * a.D;
  float* pk = a.part + (long)part * 2 * a.Tk * ldp + (long)hk * a.D;
  float* pv = pk + a.Tk * ldp;
  T* gk = (T*)a.dk + (long)hk * a.D;
  T* gv = (T*)a.dv + (long)hk * a.D;
  if (__any(finite_probe<L::NT>(dk) + finite_probe<L::NT>(dv) != 0.0f)) {
    for (int r = 0; r < 32; ++r) {
      const int tr = r0 + r;
      if (tr >= a.Tk) break;
      float2 xk = make_float2(0.0f, 0.0f), xv = xk;
      for (int n = nb; n < ne; ++n) {
        const int i0 = qlo + (n % per) * BN;
        attn_row_dkv<T>(a, hk * a.group + n / per, tr, max(a.pl.key_lo[tr], i0),
                        min(a.pl.key_hi[tr], min(i0 + BN, qhi)), lane, xk, xv);
      }
      if (parts > 1) {
        st2(pk + tr * ldp, lane, a.D, xk);
        st2(pv + tr * ldp, lane, a.D, xv);
      } else {
        st2(gk + tr * a.lddk, lane, a.D, make_float2(xk.x * a.scale, xk.y * a.scale));
        st2(gv + tr * a.lddv, lane, a.D, xv);
      }
    }
    return;
  }
  const long tt = in ? t : 0;
  if (parts > 1) {
    store_rowsT<L::NT>(pk + tt * ldp, dk, FACTOR, a.D, in, lane);
    store_rowsT<L::NT>(pv + tt * ldp, dv, 1.0f, a.D, in, lane);
  } else {
    store_rowsT<L::NT>(gk + tt * a.lddk, dk, a.scale * FACTOR, a.D, in, lane);
    store_rowsT<L::NT>(gv + tt * a.lddv, dv, 1.0f, a.D, in, lane);
  }
}

// out[t] = mul * sum over parts, in part order; eight elements a thread.
// blockIdx.y selects one of two tensors.
struct JoinArgs {
  const float* part[2];
  void* out[2];
  long ld[2];
  float mul[2];
};
template <typename T>
__global__ __launch_bounds__(256) void k_attn_sum_parts(JoinArgs j, int parts, long stride, int rows, int width) {
  const long e = ((long)blockIdx.x * 256 + threadIdx.x) * 8;
  if (e >= (long)rows * width) return;
  const long t = e / width, c = e - t * width;
  const float* p = j.part[blockIdx.y] + e;
  float v[8] = {};
  for (int s = 0; s < parts; ++s, p += stride) {
    const float4 x = *reinterpret_cast<const float4*>(p), y = *reinterpret_cast<const float4*>(p + 4);
    v[0] += x.x, v[1] += x.y, v[2] += x.z, v[3] += x.w;
    v[4] += y.x, v[5] += y.y, v[6] += y.z, v[7] += y.w;
  }
  T* o = (T*)j.out[blockIdx.y] + t * j.ld[blockIdx.y] + c;
#pragma unroll
  for (int i = 0; i < 8; ++i) St<T>::st(o + i, v[i] * j.mul[blockIdx.y]);
}

template <typename T> int dq_parts(const AttnArgs& a) {
  return parts_for<T>((long)attn_tiles(a.Tq) * a.Hq, loop_rows(a.Tk, a.Tq, a.ndoc), 64);
}
template <typename T> int dkv_parts(const AttnArgs& a) {
  // a bf16 workgroup has eight waves: it counts twice
  return parts_for<T>((long)attn_tiles(a.Tk) * a.Hkv * (sizeof(T) == 2 ? 2 : 1),
                      loop_rows(a.Tq, a.Tk, a.ndoc) * a.group, a.D > 64 ? 32 : 64);
}

// From 1024 workgroups on, two rounds of two a CU, the loops even out by
// themselves and NQ = 1 is faster (forward and backward of 8192 tokens in 8
// documents, 32 heads of 128 without groups: 513 against 552 us); below, NQ =
// 2 (the same tokens in one document, 32 heads on 8: 2382 against 2620 us).
// Parts count as workgroups: float32, two documents of 1024, 16 heads of 64
// in 16 parts: 302 against 330 us.
bool one_query_wave(const AttnArgs& a, int parts) { return (long)attn_tiles(a.Tk) * a.Hkv * parts >= 1024; }

template <typename T, int DP, int MODE, int NQ> hipError_t dkv(const AttnArgs& a, int parts, hipStream_t s) {
  constexpr int lds = DkvCfg<T, DP, NQ>::LDS;
  const hipError_t e = lds_opt_in((const void*)k_attn_dkv<T, DP, MODE, NQ>, lds);
  if (e != hipSuccess) return e;
  k_attn_dkv<T, DP, MODE, NQ><<<dim3((unsigned)attn_tiles(a.Tk) * a.Hkv * parts), 64 * NW * NQ, lds, s>>>(a, parts);
  return hipGetLastError();
}

template <typename T, int DP, int MODE> hipError_t bwd(const AttnArgs& a, hipStream_t s) {
  constexpr int lds = DqCfg<T, DP>::LDS;
  hipError_t e = lds_opt_in((const void*)k_attn_dq<T, DP, MODE>, lds);
  if (e != hipSuccess) return e;
  const int pq = dq_parts<T>(a), pk = dkv_parts<T>(a);
  const int wq = a.Hq * a.D, wk = a.Hkv * a.D;
  const auto blocks = [](long n) { return (unsigned)((n / 8 + 255) / 256); };
  if (a.Tq) {
    k_attn_dq<T, DP, MODE><<<dim3((unsigned)attn_tiles(a.Tq) * a.Hq * pq), 64 * NW, lds, s>>>(a, pq);
    e = hipGetLastError();
    if (e == hipSuccess && pq > 1) {
      const JoinArgs j = {{a.part}, {a.dq}, {a.lddq}, {a.scale}};
      k_attn_sum_parts<T><<<dim3(blocks((long)a.Tq * wq), 1), 256, 0, s>>>(j, pq, (long)a.Tq * wq, a.Tq, wq);
      e = hipGetLastError();
    }
    if (e != hipSuccess) return e;
  }
  if (a.Tk) {
    // float32 rows of 128 need all the registers of a SIMD: four waves
    if constexpr (sizeof(T) == 4 && DP == 128) e = dkv<T, DP, MODE, 1>(a, pk, s);
    else e = one_query_wave(a, pk) ? dkv<T, DP, MODE, 1>(a, pk, s) : dkv<T, DP, MODE, 2>(a, pk, s);
    if (e == hipSuccess && pk > 1) {
      const long n = (long)a.Tk * wk;
      const JoinArgs j = {{a.part, a.part + n}, {a.dk, a.dv}, {a.lddk, a.lddv}, {a.scale, 1.0f}};
      k_attn_sum_parts<T><<<dim3(blocks(n), 2), 256, 0, s>>>(j, pk, 2 * n, a.Tk, wk);
      e = hipGetLastError();
    }
  }
  return e;
}

template <typename T, int DP> hipError_t bwd_mode(const AttnArgs& a, hipStream_t s) {
  return by_mode<T>(a.slopes, a.cap, [&](auto mode) { return bwd<T, DP, decltype(mode)::value>(a, s); });
}

}  // namespace

// the two passes use the same bytes one after the other
template <typename T> size_t attn_bwd_part_bytes(const AttnArgs& a) {
  const int pq = dq_parts<T>(a), pk = dkv_parts<T>(a);
  const size_t q = pq > 1 ? (size_t)pq * a.Tq * a.Hq * a.D * 4 : 0;
  const size_t k = pk > 1 ? (size_t)pk * 2 * a.Tk * a.Hkv * a.D * 4 : 0;
  return std::max(q, k);
}

template <typename T> hipError_t launch_attn_bwd(const AttnArgs& a, hipStream_t s) {
  return a.D <= 64 ? bwd_mode<T, 64>(a, s) : bwd_mode<T, 128>(a, s);
}

template size_t attn_bwd_part_bytes<bf16>(const AttnArgs&);
template size_t attn_bwd_part_bytes<float>(const AttnArgs&);
template hipError_t launch_attn_bwd<bf16>(const AttnArgs&, hipStream_t);
template hipError_t launch_attn_bwd<float>(const AttnArgs&, hipStream_t);

}  // namespace poetx

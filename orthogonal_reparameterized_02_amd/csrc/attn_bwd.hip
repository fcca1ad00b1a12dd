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
// -> 2591 us.  With a window (below) dq is off by 2.5e-3 and dk by 2.4e-3; dq from
// two parts by 1.8e-3, for 644 -> 683 us, and dk, dv has no registers for them.
// Rows of a few keys, where dp and delta are alike, 3e-3, and 4e-3 where
// documents have four of them: delta's share, of o as it is stored.
//
// Measured (bf16, D 128, 32 heads on 8): 8192 causal tokens in one document
// 1.75 ms for both passes, dq at 1.19 and dk, dv at 1.06 PFLOP/s of the products
// they form, at the power limit; in 9 documents 320 us, a fifth of the wave
// slots empty as in the forward pass.  float32, D 64, two documents of 1024,
// 16 heads on 4, capped: 225 us, a third of the float32 matrix rate.
// With a window (8192 tokens in 3 documents, window 1024, 4 sinks) 477 us for both
// passes: 180 to 190 for dq, 268 to 290 for dk, dv, 33 for the sinks and 5 for
// their join, 0.59 PFLOP/s of the products that are seen.  A tenth more are formed
// at the edges of the window, the loops are short, and dk, dv's 512 workgroups of
// unequal loops are two rounds: matrix pipes busy in 0.42 (dq) and 0.35 (dk, dv) of
// the cycles.
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
//
// SINK: rows see the first keys of their document besides an interval.
template <typename T, int DP, int MODE, bool SINK>
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

  const int t = r0 + (lane & 31);
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
  for (int j0 = jb, n0 = SINK ? kt.nb : 0; SINK ? n0 < kt.ne : j0 < je; j0 = SINK ? kt.row(n0 + 1, BN) : j0 + BN, ++n0, buf ^= 1) {
    // this tile has landed, and every wave has left the other buffer
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    if (SINK ? n0 + 1 < kt.ne : j0 + BN < je) {
      const int jnx = SINK ? kt.row(n0 + 1, BN) : j0 + BN, jne = SINK ? kt.end(n0 + 1) : je;
      lk.load(kp, a.ldk, jnx, jne, lds0 + (buf ^ 1) * C::TILE);
      lv.load(vp, a.ldv, jnx, jne, lds0 + (2 + (buf ^ 1)) * C::TILE);
    }
    const bool far = SINK && n0 < kt.far;
    const uint32_t kr = rlane + buf * C::TILE, vr = kr + 2 * C::TILE, kc = clane + buf * C::TILE;
#pragma unroll
    for (int n = 0; n < NS; ++n) {
      const int jn = j0 + 32 * n;
      // nothing here for this wave
      if ((far || sp.lo >= jn + 32 || sp.hi <= jn) && (!SINK || ssp.lo >= jn + 32 || ssp.hi <= jn)) continue;
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
      if (far || sp.all_lo > jn || sp.all_hi < jn + 32) {  // some pair is hidden
        Seen seen = {jl - lo, jl - sink.x, (uint32_t)(hi - lo), (uint32_t)(sink.y - sink.x)};
        if constexpr (SINK)
          if (far) seen = {jl - sink.x, 0, sink.x == kt.flo ? (uint32_t)(sink.y - sink.x) : 0, 0};
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int j = 8 * (i / 4) + i % 4;
          s[i] = (SINK ? seen.either(j) : seen(j)) ? s[i] : 0.0f;
        }
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
      const float dl = wave_sum(x.x * y.x + x.y * y.y);
      const auto over = [&](int x0, int x1) {
        return attn_row_dq<T>(qp + (long)tr * a.ldq, dop + (long)tr * a.lddo, kp, a.ldk, vp, a.ldv, x0, x1, a.pl.row_pos[tr],
                              a.D, a.scale, a.cap, a.slopes ? a.slopes[h] : 0.0f, a.lse[(long)h * a.Tq + tr], dl, lane);
      };
      float2 g;
      if constexpr (SINK) {
        const int2 f = kt.far_keys(BN), w = kt.near_keys(BN), rs = a.pl.row_sink[tr];
        const float2 u = rs.x == kt.flo ? over(max(rs.x, f.x), min(rs.y, f.y)) : make_float2(0.0f, 0.0f);
        const float2 v = over(max(rs.x, w.x), min(rs.y, w.y)), z = over(max(a.pl.row_lo[tr], w.x), min(a.pl.row_hi[tr], w.y));
        g = make_float2(u.x + v.x + z.x, u.y + v.y + z.y);
      } else {
        g = over(max(a.pl.row_lo[tr], jb), min(a.pl.row_hi[tr], je));
      }
      if (parts > 1) st2(pq + tr * ldp, lane, a.D, g);
      else st2((T*)a.dq + (long)tr * a.lddq + (long)h * a.D, lane, a.D, make_float2(g.x * a.scale, g.y * a.scale));
    }
    return;
  }
  const long tt = in ? t : 0;
  if (parts > 1) store_rowsT<L::NT>(pq + tt * ldp, dq, FACTOR, a.D, in, lane);
  else store_rowsT<L::NT>((T*)a.dq + tt * a.lddq + (long)h * a.D, dq, a.scale * FACTOR, a.D, in, lane);
}

// dk and dv of the sinks that are seen past the window.  Such a key is seen by
// every later query, and would leave one workgroup of the second pass with a
// loop over the whole document; here a workgroup takes 128 queries and all query
// heads of one key head, a wave 32 of the queries, with blocks of 16 sinks of
// each document among them.  The sums, without those of other tiles, go to
// a.sink_part[tile + number][key head][dk, dv][sink][D].
//
// Bound by reading q and dout once more, from the last-level cache where they
// fit.  Measured (8192 tokens in 3 documents, window 1024, 4 sinks, 32 heads on
// 8, D 128, bf16): 33 us and 5 for the join; as a part of k_attn_dq, whose
// registers it fills, 52 us.  On 16 x 16 tiles: of 32 columns four sinks leave
// 28 idle, and the sums would take 128 registers (57 spilled, 50 us).
template <typename T, int DP> struct SinkCfg {
  using L = Tile<T, DP>;
  static constexpr int NS = 16;                      // sinks a block
  static constexpr int KS = L::RB / 64;              // row fragments: 64 bytes of a row over four lanes
  static constexpr int NT = DP / 16;                 // column tiles
  static constexpr int ROWS = 32 * L::RB;            // bytes of a wave's rows of q, of dout
  static constexpr int VAL = NW * 2 * ROWS;          // lse2 and delta of a wave's rows begin here
  static constexpr int LDS = VAL + NW * 256;
  static constexpr int OCC = sizeof(T) == 4 && DP == 128 ? 1 : 2;
  static_assert(VAL >= 2 * NW * NS * DP * 4, "room for the waves' sums");

  static __device__ __forceinline__ f32x4_t mma(uint4 x, uint4 y, f32x4_t c) {
    if constexpr (sizeof(T) == 2) return __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(x), as_bf16x8(y), c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(x.x), __uint_as_float(y.x), c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(x.y), __uint_as_float(y.y), c, 0, 0, 0);
    c = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(x.z), __uint_as_float(y.z), c, 0, 0, 0);
    return __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(x.w), __uint_as_float(y.w), c, 0, 0, 0);
  }
  // rows of a Tile as operands: lane l holds row l % 16, chunk 4 ks + l / 16
  static __device__ __forceinline__ uint32_t row_lane(int lane) {
    const int r = lane & 15;
    return r * L::RB + (((lane >> 4) ^ L::key(r)) << 4);
  }
  static __device__ __forceinline__ uint4 row_frag(const char* lds, uint32_t at, int m, int ks) {
    return *reinterpret_cast<const uint4*>(lds + ((at ^ (uint32_t)(ks << 6)) + 16 * m * L::RB));
  }
  // columns 16 ct + 0..15 as rows of the operand, K in the order that the
  // accumulators of 32 score rows have in a lane: 16 m + 4 (l / 16) + i
  static __device__ __forceinline__ uint32_t col_lane(int lane) {
    if constexpr (sizeof(T) == 2) {
      const int r = 4 * (lane >> 4) + ((lane & 15) >> 2);
      return r * L::RB + ((((lane & 3) >> 1) ^ L::key(r)) << 4) + (lane & 1) * 8;
    } else {
      const int r = 4 * (lane >> 4);
      return r * L::RB + ((((lane & 15) >> 2) ^ L::key(r)) << 4) + (lane & 3) * 4;
    }
  }
  // acc += columns^T x, x the scores' accumulators
  static __device__ __forceinline__ f32x4_t mma_cols(const char* lds, uint32_t at, int ct, const f32x4_t (&x)[2], uint4 frag, f32x4_t acc) {
    if constexpr (sizeof(T) == 2) {
      char* p = const_cast<char*>(lds) + (at ^ (uint32_t)(ct << 5));
      const s16x4_t h0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)p);
      const s16x4_t h1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)(p + 16 * L::RB));
      return mma(__builtin_bit_cast(uint4, __builtin_shufflevector(h0, h1, 0, 1, 2, 3, 4, 5, 6, 7)), frag, acc);
    } else {
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int i = 0; i < 4; ++i)  // i enters the key of row 4 (l / 16) + i as it stands
          acc = __builtin_amdgcn_mfma_f32_16x16x4f32(
              *reinterpret_cast<const float*>(lds + ((at ^ (uint32_t)(ct << 6 | i << 4)) + (16 * m + i) * L::RB)), x[m][i], acc, 0, 0, 0);
      return acc;
    }
  }
  static __device__ __forceinline__ uint4 pack(const f32x4_t (&x)[2]) {
    return make_uint4(pack2bf(x[0][0], x[0][1]), pack2bf(x[0][2], x[0][3]), pack2bf(x[1][0], x[1][1]), pack2bf(x[1][2], x[1][3]));
  }
};
template <typename T, int DP, int MODE>
__global__ __launch_bounds__(64 * NW, (SinkCfg<T, DP>::OCC)) void k_attn_sink(AttnArgs a) {
  using C = SinkCfg<T, DP>;
  constexpr int NS = C::NS;
  extern __shared__ __align__(16) char smem[];
  const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), g = lane >> 4;
  const int hk = blockIdx.x % a.Hkv, tile = blockIdx.x / a.Hkv, q0 = tile * BM, rows = min(a.Tq - q0, BM);
  const int r0 = q0 + 32 * wave, rend = min(r0 + 32, a.Tq);
  const T* kp = (const T*)a.k + (long)hk * a.D;
  const T* vp = (const T*)a.v + (long)hk * a.D;
  Loader<T, DP, 32, 1> lq, ld;
  lq.init(a.ldq, a.D, 0, lane);
  ld.init(a.lddo, a.D, 0, lane);
  const uint32_t at = wave * 2 * C::ROWS;
  const uint32_t ldsq = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)smem + at;
  float* vals = reinterpret_cast<float*>(smem + C::VAL + wave * 256);
  float* sums = reinterpret_cast<float*>(smem);  // [dk, dv][NW][NS][DP]
  for (int d = max(a.pl.tile_doc[tile], 0); d < a.ndoc; ++d) {
    const int4 e = a.pl.doc[d];
    const int dq0 = __builtin_amdgcn_readfirstlane(e.x), dq1 = __builtin_amdgcn_readfirstlane(e.y);
    const int dk0 = __builtin_amdgcn_readfirstlane(e.z), dk1 = __builtin_amdgcn_readfirstlane(e.w);
    if (dq0 >= q0 + rows) break;
    if (dq1 <= q0 || dq0 >= dq1 || !sinks_apart(dq1 - dq0, dk1 - dk0, a.causal, a.window)) continue;
    const int ns = min(a.sinks, dk1 - dk0), off = dq1 - dk1;
    float* out = a.sink_part + ((tile + sink_number(a, d, dq0, dk0)) * a.Hkv + hk) * 2 * a.sinks * a.D;
    for (int b = 0; b < ns; b += NS) {
      // queries that see this lane's key
      const int key = b + (lane & 15), t = dk0 + key;
      const int lo = key < ns ? max(a.causal ? t + off : dq0, dq0) : 0, hi = key < ns ? dq1 : 0;
      uint4 kf[C::KS], vf[C::KS];
      {
        const int r = dk0 + min(key, ns - 1);
        const T *pk = kp + (long)r * a.ldk, *pv = vp + (long)r * a.ldv;
#pragma unroll
        for (int i = 0; i < C::KS; ++i) {
          const int el = (64 * i + 16 * g) / (int)sizeof(T);
          kf[i] = *reinterpret_cast<const uint4*>(pk + (el < a.D ? el : 0));
          vf[i] = *reinterpret_cast<const uint4*>(pv + (el < a.D ? el : 0));
          if (el >= a.D) kf[i] = vf[i] = make_uint4(0, 0, 0, 0);
        }
      }
      f32x4_t dk[C::NT], dv[C::NT];
#pragma unroll
      for (int i = 0; i < C::NT; ++i) dk[i] = dv[i] = (f32x4_t){};
      // rows past the last one are zeros, and seen by none
      if (rend > r0 && r0 < dq1 && rend > dq0)
        for (int h = hk * a.group; h < (hk + 1) * a.group; ++h) {
          lq.load((const T*)a.q + (long)h * a.D, a.ldq, r0, rend, ldsq);
          ld.load((const T*)a.dout + (long)h * a.D, a.lddo, r0, rend, ldsq + C::ROWS);
          const long row = (long)h * a.Tq + min(r0 + (lane & 31), a.Tq - 1);
          const float own = lane < 32 ? a.lse2[row] : a.delta[row];
          wait_loads();
          vals[lane] = own;
          const ScoreArgs sa = score_args<T, MODE>(a, h);
          // a new value to the compiler: kept over the loop, the addresses of
          // the fragments would fill registers
          uint32_t rl = C::row_lane(lane), cl = C::col_lane(lane);
          asm volatile("" : "+v"(rl), "+v"(cl));
          const uint32_t qr = rl + at, dr = qr + C::ROWS, qc = cl + at, dc = qc + C::ROWS;
          f32x4_t s[2], dp[2], p[2];
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            s[m] = (f32x4_t){};
            dp[m] = -*reinterpret_cast<const f32x4_t*>(vals + 32 + 16 * m + 4 * g);
#pragma unroll
            for (int i = 0; i < C::KS; ++i) {
              s[m] = C::mma(C::row_frag(smem, qr, m, i), kf[i], s[m]);
              dp[m] = C::mma(C::row_frag(smem, dr, m, i), vf[i], dp[m]);
            }
          }
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            const f32x4_t l2 = *reinterpret_cast<const f32x4_t*>(vals + 16 * m + 4 * g);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int qrow = r0 + 16 * m + 4 * g + i;
              float deriv;
              if constexpr (MODE == 0) p[m][i] = exp2_hw(fmaf(s[m][i], sa.c, -l2[i]));
              else p[m][i] = exp2_hw(score2<T, MODE>(s[m][i], sa, (float)(qrow - off - t), deriv) - l2[i]);
              s[m][i] = p[m][i] * dp[m][i];
              if constexpr (MODE & 1) s[m][i] *= deriv;
              const bool seen = qrow >= lo && qrow < hi;
              p[m][i] = seen ? p[m][i] : 0.0f;
              s[m][i] = seen ? s[m][i] : 0.0f;
            }
          }
          const uint4 fp = C::pack(p), fs = C::pack(s);
#pragma unroll
          for (int ct = 0; ct < C::NT; ++ct) {
            dv[ct] = C::mma_cols(smem, dc, ct, p, fp, dv[ct]);
            dk[ct] = C::mma_cols(smem, qc, ct, s, fs, dk[ct]);
          }
          asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");  // the next rows may land
        }
      // rows of other documents enter as 0 times their value; where that left
      // what is not finite, the sums are formed again from what is seen
      float probe = 0.0f;
#pragma unroll
      for (int ct = 0; ct < C::NT; ++ct)
#pragma unroll
        for (int i = 0; i < 4; ++i) probe = fmaf(dk[ct][i], 0.0f, fmaf(dv[ct][i], 0.0f, probe));
      const int n = min(ns - b, NS);
      __syncthreads();  // the rows, or the sums before, have been read
      if (__any(probe != 0.0f)) {
        for (int j = 0; j < n; ++j) {
          const int tj = dk0 + b + j;
          float2 xk = make_float2(0.0f, 0.0f), xv = xk;
          for (int h = hk * a.group; h < (hk + 1) * a.group; ++h)
            attn_row_dkv<T>(a, h, tj, max(max(a.causal ? tj + off : dq0, dq0), r0), min(dq1, rend), lane, xk, xv);
          if (2 * lane < DP) {
            *reinterpret_cast<float2*>(sums + (wave * NS + j) * DP + 2 * lane) = xk;
            *reinterpret_cast<float2*>(sums + ((NW + wave) * NS + j) * DP + 2 * lane) = xv;
          }
        }
      } else if (key < ns) {
        float* mine = sums + (wave * NS + (lane & 15)) * DP + 4 * g;
#pragma unroll
        for (int ct = 0; ct < C::NT; ++ct) {
          *reinterpret_cast<f32x4_t*>(mine + 16 * ct) = dk[ct] * cap_factor<T, MODE>;
          *reinterpret_cast<f32x4_t*>(mine + NW * NS * DP + 16 * ct) = dv[ct];
        }
      }
      __syncthreads();
      for (int x = threadIdx.x; x < 2 * n * (DP / 2); x += 64 * NW) {
        const int which = x / (n * (DP / 2)), y = x - which * (n * (DP / 2)), j = y / (DP / 2), c = y % (DP / 2) * 2;
        float2 z = make_float2(0.0f, 0.0f);
#pragma unroll
        for (int w = 0; w < NW; ++w) {
          const float2 v = *reinterpret_cast<const float2*>(sums + ((which * NW + w) * NS + j) * DP + c);
          z.x += v.x, z.y += v.y;
        }
        if (c < a.D) *reinterpret_cast<float2*>(out + (long)(which * a.sinks + b + j) * a.D + c) = z;
      }
      __syncthreads();
    }
  }
}

// dk and dv of the sinks: what k_attn_sink left, over the tiles of a document.  A
// workgroup a sink and key head; sixteen waves take every sixteenth partial sum
// and join in wave order.  The second pass has left zeros in these rows.
constexpr int SW = 16;
template <typename T> __global__ __launch_bounds__(64 * SW) void k_attn_sink_join(AttnArgs a) {
  __shared__ float2 red[SW][2][64];
  const int lane = threadIdx.x % 64, wave = threadIdx.x / 64, d = blockIdx.x / a.sinks, s = blockIdx.x % a.sinks, hk = blockIdx.y;
  const int4 e = a.pl.doc[d];
  const int q0 = e.x, q1 = e.y, k0 = e.z, k1 = e.w;
  if (s >= k1 - k0 || !sinks_apart(q1 - q0, k1 - k0, a.causal, a.window)) return;
  const int t0 = q0 / BM, tiles = q1 > q0 ? (q1 - 1) / BM - t0 + 1 : 0;
  const long slot = t0 + sink_number(a, d, q0, k0), plane = (long)a.sinks * a.D;
  float2 x[2] = {make_float2(0.0f, 0.0f), make_float2(0.0f, 0.0f)};
  if (2 * lane < a.D) {
#pragma unroll 4
    for (int n = wave; n < tiles; n += SW) {
      const float* p = a.sink_part + (((slot + n) * a.Hkv + hk) * 2) * plane + (long)s * a.D + 2 * lane;
      const float2 u = *reinterpret_cast<const float2*>(p), v = *reinterpret_cast<const float2*>(p + plane);
      x[0].x += u.x, x[0].y += u.y, x[1].x += v.x, x[1].y += v.y;
    }
  }
  red[wave][0][lane] = x[0];
  red[wave][1][lane] = x[1];
  __syncthreads();
  if (wave > 1) return;
  float2 y = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int w = 0; w < SW; ++w) {
    const float2 u = red[w][wave][lane];
    y.x += u.x, y.y += u.y;
  }
  const float mul = wave ? 1.0f : a.scale;
  T* out = wave ? (T*)a.dv + (long)(k0 + s) * a.lddv : (T*)a.dk + (long)(k0 + s) * a.lddk;
  st2(out + (long)hk * a.D, lane, a.D, make_float2(y.x * mul, y.y * mul));
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
  return parts_for<T>((long)attn_tiles(a.Tq) * a.Hq, loop_rows(a.Tk, a.Tq, a.ndoc, a.reach()), 64);
}
template <typename T> int dkv_parts(const AttnArgs& a) {
  // a bf16 workgroup has eight waves: it counts twice
  return parts_for<T>((long)attn_tiles(a.Tk) * a.Hkv * (sizeof(T) == 2 ? 2 : 1),
                      loop_rows(a.Tq, a.Tk, a.ndoc, a.reach()) * a.group, a.D > 64 ? 32 : 64);
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

template <typename T, int DP, int MODE, bool SINK> hipError_t bwd(const AttnArgs& a, hipStream_t s) {
  constexpr int lds = DqCfg<T, DP>::LDS;
  hipError_t e = lds_opt_in((const void*)k_attn_dq<T, DP, MODE, SINK>, lds);
  if (e != hipSuccess) return e;
  const int pq = dq_parts<T>(a), pk = dkv_parts<T>(a);
  const int wq = a.Hq * a.D, wk = a.Hkv * a.D;
  const auto blocks = [](long n) { return (unsigned)((n / 8 + 255) / 256); };
  if (a.Tq) {
    k_attn_dq<T, DP, MODE, SINK><<<dim3((unsigned)attn_tiles(a.Tq) * a.Hq * pq), 64 * NW, lds, s>>>(a, pq);
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
    if (SINK && e == hipSuccess && a.ndoc && a.Tq) {
      constexpr int lds_s = SinkCfg<T, DP>::LDS;
      e = lds_opt_in((const void*)k_attn_sink<T, DP, MODE>, lds_s);
      if (e != hipSuccess) return e;
      k_attn_sink<T, DP, MODE><<<dim3((unsigned)attn_tiles(a.Tq) * a.Hkv), 64 * NW, lds_s, s>>>(a);
      e = hipGetLastError();
    }
    if (SINK && e == hipSuccess && a.ndoc) {
      k_attn_sink_join<T><<<dim3(a.ndoc * a.sinks, a.Hkv), 64 * SW, 0, s>>>(a);
      e = hipGetLastError();
    }
  }
  return e;
}

template <typename T, int DP> hipError_t bwd_mode(const AttnArgs& a, hipStream_t s) {
  return by_mode<T>(a.slopes, a.cap, [&](auto mode) {
    constexpr int MODE = decltype(mode)::value;
    return a.sinks ? bwd<T, DP, MODE, true>(a, s) : bwd<T, DP, MODE, false>(a, s);
  });
}

}  // namespace

// the two passes use the same bytes one after the other
template <typename T> size_t attn_bwd_part_bytes(const AttnArgs& a) {
  const int pq = dq_parts<T>(a), pk = dkv_parts<T>(a);
  const size_t q = pq > 1 ? (size_t)pq * a.Tq * a.Hq * a.D * 4 : 0;
  const size_t k = pk > 1 ? (size_t)pk * 2 * a.Tk * a.Hkv * a.D * 4 : 0;
  return std::max(q, k);
}

// a slot for every query tile of every document whose sinks are summed apart:
// tile + sink_number grows from one to the next
size_t attn_sink_part_bytes(const AttnArgs& a) {
  const size_t slots = attn_tiles(a.Tq) + std::min((long)a.ndoc, sink_place(a.Tq, a.Tk, a.window)) + 1;
  return a.sinks ? slots * a.Hkv * 2 * a.sinks * a.D * 4 : 0;
}

template <typename T> hipError_t launch_attn_bwd(const AttnArgs& a, hipStream_t s) {
  return a.D <= 64 ? bwd_mode<T, 64>(a, s) : bwd_mode<T, 128>(a, s);
}

template size_t attn_bwd_part_bytes<bf16>(const AttnArgs&);
template size_t attn_bwd_part_bytes<float>(const AttnArgs&);
template hipError_t launch_attn_bwd<bf16>(const AttnArgs&, hipStream_t);
template hipError_t launch_attn_bwd<float>(const AttnArgs&, hipStream_t);

}  // namespace poetx

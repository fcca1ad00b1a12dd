// Tiles, operand fragments and scores of the MFMA attention kernels.
//
// Products run on 32 x 32 MFMA tiles.  An operand fragment is 16 bytes a
// lane: lane l holds row l % 32, and of every 32-byte chunk of that row the
// half l / 32 (bf16: one v_mfma_f32_32x32x16_bf16 a chunk; float32: four
// v_mfma_f32_32x32x2_f32).  A and B are read alike, so the order of the
// elements within a chunk does not matter.  The accumulator holds
// D[8 (i/4) + 4 (l/32) + i % 4][l % 32] in register i: a lane owns one
// column, the four rows of a quad are consecutive.
// Scores are formed as D[key][query] where queries are what a wave owns (the
// forward pass, dq), or D[query][key] where keys are (dk, dv): the running
// maximum and sum, the mask and the next product's B operand then stay in the
// lane, for the quads of a 32-row score tile are exactly a B fragment whose
// K order is 8 g + 4 (l/32) + 0..3; the A fragment of the transposed tile
// (rows of V, K, Q or dO read down their columns) takes the same K order.
#pragma once

#include <float.h>

#include <type_traits>

#include "attn.h"

namespace poetx {

typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef short s16x8_t __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) s16x4_t lds_s16x4_t;

constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;

__device__ __forceinline__ float exp2_hw(float x) { return __builtin_amdgcn_exp2f(x); }

// ---- fragments ----------------------------------------------------------------
__device__ __forceinline__ f32x16_t mma16(const bf16*, uint4 a, uint4 b, f32x16_t c) {
  return mfma32x32x16(as_bf16x8(a), as_bf16x8(b), c);
}
__device__ __forceinline__ f32x16_t mma16(const float*, uint4 a, uint4 b, f32x16_t c) {
  c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a.x), __uint_as_float(b.x), c, 0, 0, 0);
  c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a.y), __uint_as_float(b.y), c, 0, 0, 0);
  c = __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a.z), __uint_as_float(b.z), c, 0, 0, 0);
  return __builtin_amdgcn_mfma_f32_32x32x2f32(__uint_as_float(a.w), __uint_as_float(b.w), c, 0, 0, 0);
}

// ---- tiles in LDS ---------------------------------------------------------------
// Rows of DP elements (DP = 64 or 128, the head width rounded up; elements
// past the head are zero), 16-byte chunk c of row r at position c ^ key(r).
// The keys keep two access patterns off each other's banks: a row fragment
// (16 rows, one chunk) and a column fragment (bf16: ds_read_b64_tr_b16, 4
// rows x 64 bytes; float32: two rows four apart, 128 bytes each).
template <typename T, int DP> struct Tile {
  static constexpr int ES = sizeof(T);
  static constexpr int RB = DP * ES;        // bytes a row
  static constexpr int LPR = RB / 16;       // lanes (chunks) a row
  static constexpr int RPL = 64 / LPR;      // rows one wave's load fills
  static constexpr int KS = RB / 32;        // row fragments a row
  static constexpr int NT = DP / 32;        // 32-wide column tiles

  static __device__ __forceinline__ int key(int r) {
    if constexpr (ES == 4) return (r & 3) | ((r & 8) >> 1) | ((r & 4) << 1);
    else if constexpr (RB == 256) return ((r & 3) << 2) | ((r >> 2) & 3);
    else return ((r & 2) << 1) | ((r >> 2) & 3);
  }
  // Fragment addresses: a tile's byte offset in LDS (a multiple of 512) plus
  // one of the two lane offsets below, then constants: the chunk numbers
  // enter by XOR, the rows by addition.  A fragment costs one XOR, and no
  // register is held for it.
  //
  // row fragment ks of rows r0 .. r0 + 31 (r0 a multiple of 32)
  static __device__ __forceinline__ uint32_t row_lane(int lane) {
    const int r = lane & 31;
    return r * RB + (((lane >> 5) ^ key(r)) << 4);
  }
  static __device__ __forceinline__ uint4 row_frag(const char* lds, uint32_t at, int r0, int ks) {
    return *reinterpret_cast<const uint4*>(lds + ((at ^ (uint32_t)(ks << 5)) + r0 * RB));
  }
  // column fragment: columns 32 ct + 0..31 as rows of the operand, K = the
  // tile rows of score quads: bf16 quads 2t, 2t+1 (16 rows), float32 quad t
  // (8 rows) of the 32 rows from r0
  static __device__ __forceinline__ uint32_t col_lane(int lane) {
    if constexpr (ES == 2) {
      const int r = 4 * (lane >> 5) + ((lane & 15) >> 2), c = 2 * ((lane >> 4) & 1) + ((lane & 3) >> 1);
      return r * RB + ((c ^ key(r)) << 4) + (lane & 1) * 8;
    } else {
      const int r = 4 * (lane >> 5), c = (lane & 31) >> 2;
      return r * RB + ((c ^ key(r)) << 4) + (lane & 3) * 4;
    }
  }
  static __device__ __forceinline__ uint4 col_frag(const char* lds, uint32_t at, int r0, int t, int ct) {
    if constexpr (ES == 2) {
      // 4 columns x 4 rows a lane; eight rows further the key differs in bit 1
      const uint32_t p = at ^ (uint32_t)(ct << 6), q = at ^ (uint32_t)((ct << 6) | 32);
      const int row = (r0 + 16 * t) * RB;
      const s16x4_t h0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)(const_cast<char*>(lds + (p + row))));
      const s16x4_t h1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)(const_cast<char*>(lds + (q + row + 8 * RB))));
      return __builtin_bit_cast(uint4, __builtin_shufflevector(h0, h1, 0, 1, 2, 3, 4, 5, 6, 7));
    } else {
      uint32_t u[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        u[e] = *reinterpret_cast<const uint32_t*>(
            lds + ((at ^ (uint32_t)((ct << 7) | (t & 1) << 6 | e << 4)) + (r0 + 8 * t + e) * RB));
      return make_uint4(u[0], u[1], u[2], u[3]);
    }
  }
  static constexpr int CSTEP = 32 * ES / 64 == 1 ? 2 : 4;  // column fragments per 32 tile rows

  // the B fragment of score quads (see col_frag) of one 32-row score tile
  static __device__ __forceinline__ uint4 score_frag(const f32x16_t& p, int t) {
    if constexpr (ES == 2)
      return make_uint4(pack2bf(p[8 * t], p[8 * t + 1]), pack2bf(p[8 * t + 2], p[8 * t + 3]),
                        pack2bf(p[8 * t + 4], p[8 * t + 5]), pack2bf(p[8 * t + 6], p[8 * t + 7]));
    else
      return make_uint4(__float_as_uint(p[4 * t]), __float_as_uint(p[4 * t + 1]),
                        __float_as_uint(p[4 * t + 2]), __float_as_uint(p[4 * t + 3]));
  }
  // The same in two parts that together hold 16 bits: f the next bf16 below
  // each score (>= 0), rest what that leaves, rounded.  Both are above 0 where
  // the score is: an infinite row of the other operand stays one, which 0 or
  // a negative rest would turn into NaN.
  static __device__ __forceinline__ void score_parts(const f32x16_t& p, int t, uint4& f, uint4& rest) {
    uint32_t h[4], r[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = p[8 * t + 2 * i], y = p[8 * t + 2 * i + 1];
      const uint32_t a = __builtin_elementwise_sub_sat(__float_as_uint(x), 1u) & 0xffff0000u;
      const uint32_t b = __builtin_elementwise_sub_sat(__float_as_uint(y), 1u) & 0xffff0000u;
      h[i] = a >> 16 | b;
      r[i] = pack2bf(x - __uint_as_float(a), y - __uint_as_float(b));
    }
    f = make_uint4(h[0], h[1], h[2], h[3]);
    rest = make_uint4(r[0], r[1], r[2], r[3]);
  }
};

// Loads of a tile straight into LDS (buffer_load_dwordx4 ... lds: a wave
// fills 1 KB).  Lane l lands at byte 16 l of the wave's part, so it fetches
// the chunk that belongs there.  The buffer range ends with the last row
// that counts: rows past it, and chunks past the head (whose offset is put
// out of range), arrive as zeros.  Completion is tracked by vmcnt.  A load needs
// a wait state after the write of m0, which the compiler does not add inside
// asm.
// NT: non-temporal, for rows that are read once (a cache of many gigabytes
// pushes everything else out of the last-level cache, and waits for it).
template <typename T, int DP, int ROWS, int NW, bool NT = false> struct Loader {
  using L = Tile<T, DP>;
  static constexpr int STEP = NW * L::RPL;        // rows one load of all waves fills
  static constexpr int N = ROWS / STEP;           // loads a wave
  static constexpr int VAR = STEP < 16 ? 16 / STEP : 1;  // lane offsets repeat every 16 rows
  static_assert(ROWS % STEP == 0 && STEP * VAR % 16 == 0, "tile split");
  int vo[VAR];
  int ldb;      // pitch in bytes
  int headb;    // head bytes
  int wave;

  __device__ __forceinline__ void init(long ld, int D, int wave_, int lane) {
    ldb = (int)ld * L::ES;
    headb = D * L::ES;
    wave = wave_;
#pragma unroll
    for (int u = 0; u < VAR; ++u) {
      const int r = (u * NW + wave) * L::RPL + lane / L::LPR;
      const int c = (lane % L::LPR) ^ L::key(r);
      vo[u] = c * 16 < headb ? r * ldb + c * 16 : 0x60000000;
    }
  }
  // rows [row0, row0 + ROWS) of base (a head's first element in row 0), of
  // which those below `end` count, into LDS at byte offset lds
  __device__ __forceinline__ void load(const T* base, long ld, int row0, int end, uint32_t lds) const {
    const int rows = min(max(end - row0, 0), ROWS);
    const __amdgpu_buffer_rsrc_t rs = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(base + (long)row0 * ld), (short)0, rows > 0 ? (rows - 1) * ldb + headb : 0, 0x00020000);
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const uint32_t m0v = __builtin_amdgcn_readfirstlane(lds + (j * NW + wave) * 1024);
      const int off = vo[j % VAR] + (j - j % VAR) * STEP * ldb;
      if constexpr (NT)
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen nt lds" ::"s"(m0v), "v"(off), "s"(rs)
                     : "memory");
      else
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(m0v), "v"(off), "s"(rs)
                     : "memory");
    }
  }
};

// A wave's 32 rows as row fragments in registers, straight from memory.
// Rows from `end` (> 0) on repeat the last one (nothing of theirs is
// stored), elements past the head are zero.  No branch: all loads are in
// flight together.
template <typename T, int KS>
__device__ __forceinline__ void rows_to_regs(uint4 (&f)[KS], const T* base, long ld,
                                             int row0, int end, int D, int lane) {
  const T* p = base + (long)min(row0 + (lane & 31), end - 1) * ld;
#pragma unroll
  for (int ks = 0; ks < KS; ++ks) {
    const int e = (32 * ks + 16 * (lane >> 5)) / (int)sizeof(T);
    f[ks] = *reinterpret_cast<const uint4*>(p + (e < D ? e : 0));
  }
#pragma unroll
  for (int ks = 0; ks < KS; ++ks) {
    const int e = (32 * ks + 16 * (lane >> 5)) / (int)sizeof(T);
    if (e >= D) f[ks] = make_uint4(0, 0, 0, 0);
  }
}

// acc (transposed: D[element][row], NT tiles of 32 elements) * mul to the
// wave's rows in memory: halves of lanes l and l + 32 are joined so that a
// lane stores eight consecutive elements.
template <int NT>
__device__ __forceinline__ void store_rowsT(bf16* p, const f32x16_t (&acc)[NT], float mul, int D,
                                            bool live, int lane) {
  const int h = lane >> 5;
#pragma unroll
  for (int ct = 0; ct < NT; ++ct)
#pragma unroll
    for (int g = 0; g < 4; g += 2) {
      uint32_t a0 = pack2bf(acc[ct][4 * g] * mul, acc[ct][4 * g + 1] * mul);
      uint32_t a1 = pack2bf(acc[ct][4 * g + 2] * mul, acc[ct][4 * g + 3] * mul);
      uint32_t b0 = pack2bf(acc[ct][4 * g + 4] * mul, acc[ct][4 * g + 5] * mul);
      uint32_t b1 = pack2bf(acc[ct][4 * g + 6] * mul, acc[ct][4 * g + 7] * mul);
      // upper half of a <-> lower half of b: lane half h then holds quad
      // g + h of both halves, elements 8 (g + h) + 0..7
      const auto s0 = __builtin_amdgcn_permlane32_swap(a0, b0, false, false);
      const auto s1 = __builtin_amdgcn_permlane32_swap(a1, b1, false, false);
      const int e = 32 * ct + 8 * (g + h);
      if (live && e < D) *reinterpret_cast<uint4*>(p + e) = make_uint4(s0[0], s1[0], s0[1], s1[1]);
    }
}
template <int NT>
__device__ __forceinline__ void store_rowsT(float* p, const f32x16_t (&acc)[NT], float mul, int D,
                                            bool live, int lane) {
  const int h = lane >> 5;
#pragma unroll
  for (int ct = 0; ct < NT; ++ct)
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int e = 32 * ct + 8 * g + 4 * h;
      if (live && e < D)
        *reinterpret_cast<float4*>(p + e) = make_float4(acc[ct][4 * g] * mul, acc[ct][4 * g + 1] * mul,
                                                        acc[ct][4 * g + 2] * mul, acc[ct][4 * g + 3] * mul);
    }
}

// 0 if every value is finite, NaN otherwise
template <int NT> __device__ __forceinline__ float finite_probe(const f32x16_t (&acc)[NT]) {
  float c = 0.0f;
#pragma unroll
  for (int ct = 0; ct < NT; ++ct)
#pragma unroll
    for (int i = 0; i < 16; ++i) c = fmaf(acc[ct][i], 0.0f, c);
  return c;
}

// sum or maximum over the two lanes that share a column
__device__ __forceinline__ float other_half(float x) {
  const uint32_t u = __float_as_uint(x);
  const auto s = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  return __uint_as_float((threadIdx.x & 32) ? s[0] : s[1]);
}

// Waits for every outstanding load in a form that the compiler counts: it
// then knows that registers loaded before a loop have arrived.  Left to wait
// at their first use, inside the loop, it would wait for the tile loads
// issued just before (it cannot see them) in every turn.
__device__ __forceinline__ void wait_loads() {
  __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0)
  asm volatile("" ::: "memory");
}

// N fragments read from LDS DEPTH ahead of the products that use them.  Left
// to the compiler's order, a read sits right before its product and each
// product waits for a whole LDS latency; here reads and products keep the
// order written (other arithmetic may move).
template <int N, int DEPTH> struct Pipe {
  uint4 f[DEPTH];
  template <class Ld> __device__ __forceinline__ void start(Ld ld) {
#pragma unroll
    for (int i = 0; i < DEPTH; ++i) f[i] = ld(i);
    __builtin_amdgcn_sched_barrier(0x6);
  }
  template <class Ld, class Use> __device__ __forceinline__ void run(Ld ld, Use use) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      use(i, f[i % DEPTH]);
      if (i + DEPTH < N) f[i % DEPTH] = ld(i + DEPTH);
      __builtin_amdgcn_sched_barrier(0x6);
    }
  }
};

// ---- scores ----------------------------------------------------------------------
// MODE bit 0: capped by a tanh; bit 1: distance bias; bit 2 (with bit 0): the
// tanh of bf16 scores formed as for float32.  Scores are in units of log2:
// s2 = log2(e) * score.  With
//   r = 1 / (1 + e^(2 x / cap)):  cap tanh(x / cap) = cap - 2 cap r,
//   1 - tanh^2 = 4 (r - r^2),
// bf16 takes caps up to CAP_R_MAX from one exponential and one reciprocal.
// The difference cancels where x is small: its absolute error is about cap
// 2^-23 (lse off by 1e-4 at a cap of 1024; at 1e6 o is off by 3%, at 1e8
// nothing is left of the scores), up to a cap of 128 below 2^-16, that of a
// float32 lse of a hundred.  Wider caps, and float32, take tanh itself: near
// 0 an odd polynomial (least squares on [0, 0.65], relative error 8e-8).  By r
// against tanh (caps of 128 and 200): 2048 queries on 16384 keys 614 and 739
// us, training on 9 documents 479 and 551, 16 long decoded sequences 234, 237.
constexpr float CAP_R_MAX = 128.0f;
template <typename T, int MODE> constexpr bool cap_by_r = (MODE & 1) && !(MODE & 4) && sizeof(T) == 2;

// launches f with the MODE of these scores as a constant
template <typename T, class F> auto by_mode(const float* slopes, float cap, F f) {
  if constexpr (sizeof(T) == 2)
    if (cap > CAP_R_MAX) return slopes ? f(std::integral_constant<int, 7>{}) : f(std::integral_constant<int, 5>{});
  if (slopes) return cap > 0.0f ? f(std::integral_constant<int, 3>{}) : f(std::integral_constant<int, 2>{});
  return cap > 0.0f ? f(std::integral_constant<int, 1>{}) : f(std::integral_constant<int, 0>{});
}

__device__ __forceinline__ float tanh_f32(float x) {
  const float big = 1.0f - 2.0f * __builtin_amdgcn_rcpf(1.0f + exp2_hw(x * (2.0f * LOG2E)));
  const float u = x * x;
  float p = -0.005514524877071381f;
  p = fmaf(p, u, 0.020468397065997124f);
  p = fmaf(p, u, -0.05368747189640999f);
  p = fmaf(p, u, 0.13330818712711334f);
  p = fmaf(p, u, -0.3333325982093811f);
  return fabsf(x) < 0.65f ? fmaf(x * u, p, x) : big;
}

struct ScoreArgs {
  float c;      // of q.k: scale log2e; capped: scale / cap, by r: 2 log2e scale / cap
  float capl;   // cap log2e
  float slope;  // slope log2e
};

template <typename T, int MODE>
__device__ __forceinline__ ScoreArgs score_args(float scale, float cap, float slope) {
  ScoreArgs s;
  // finite: a product of 0 stays 0 beside a large scale or a tiny cap
  s.c = fminf(!(MODE & 1) ? scale * LOG2E : cap_by_r<T, MODE> ? scale / cap * (2.0f * LOG2E) : scale / cap, FLT_MAX);
  s.capl = cap * LOG2E;
  s.slope = slope * LOG2E;
  return s;
}
template <typename T, int MODE> __device__ __forceinline__ ScoreArgs score_args(const AttnArgs& a, int h) {
  return score_args<T, MODE>(a.scale, a.cap, MODE & 2 ? a.slopes[h] : 0.0f);
}

__device__ __forceinline__ float cap_r(float qk, const ScoreArgs& s) {
  return __builtin_amdgcn_rcpf(1.0f + exp2_hw(qk * s.c));
}

// What the gradient of a capped score holds beside the derivative that
// score2 returns: 4 of 4 (r - r^2)
template <typename T, int MODE> constexpr float cap_factor = cap_by_r<T, MODE> ? 4.0f : 1.0f;

// s2 of q.k; deriv: its derivative by scale * q.k, less cap_factor (1 without
// a cap); dist: query position - key
template <typename T, int MODE>
__device__ __forceinline__ float score2(float qk, const ScoreArgs& s, float dist, float& deriv) {
  float x;
  if constexpr (!(MODE & 1)) {
    x = qk * s.c;
  } else if constexpr (cap_by_r<T, MODE>) {
    const float r = cap_r(qk, s);
    x = fmaf(-2.0f * s.capl, r, s.capl);
    deriv = fmaf(-r, r, r);
  } else {
    const float t = tanh_f32(qk * s.c);
    x = s.capl * t;
    deriv = fmaf(-t, t, 1.0f);
  }
  if constexpr (MODE & 2) x = fmaf(-s.slope, fabsf(dist), x);
  return x;
}

// ---- a wave's or workgroup's interval of visible rows ------------------------------
// Bounds of up to 64 rows per call, one a lane; intervals that are not empty
// grow with the row, so the first and the last of them give the bounds.
struct Span {
  int lo, hi;          // union of the intervals (lo >= hi: none)
  int all_lo, all_hi;  // intersection
};
__device__ __forceinline__ Span span_of(int lo, int hi) {
  const uint64_t some = __ballot(lo < hi);
  Span s = {0, 0, 0, 0};
  if (some) {
    const int first = __builtin_ctzll(some), last = 63 - __builtin_clzll(some);
    s.lo = __builtin_amdgcn_readlane(lo, first);
    s.hi = __builtin_amdgcn_readlane(hi, last);
    s.all_lo = __builtin_amdgcn_readlane(lo, last);
    s.all_hi = __builtin_amdgcn_readlane(hi, first);
  }
  return s;
}
// Work order: tile by tile (long ones first, AttnPlan), all heads of one
// before the next.  Head by head, a head's short tiles end beside another's
// long ones and the last round waits for the latter.
// Consecutive workgroups are dealt round-robin over the 8 XCDs; a head stays
// on one XCD, beside the heads that share its keys, where 8 divides the heads.
// The parts of a tile's loop (part_of) count as heads of their own here.
__device__ __forceinline__ void work_of(int id, int heads, int parts, int& head, int& part, int& tile) {
  const int n = heads * parts;
  int v;
  if (n % 8 == 0) {
    const int per = n / 8, y = id / 8;
    v = (id % 8) * per + y % per;
    tile = y / per;
  } else {
    v = id % n;
    tile = id / n;
  }
  head = v / parts;
  part = v - head * parts;
}

// Entry of a tile table (AttnPlan) in scalar registers: first row, and the
// range of the other side's rows.  Clamped, so that a plan that was never
// made gives wrong results and no access out of range.
__device__ __forceinline__ void tile_entry(const int4* tab, int tile, int bm, int rows, int others,
                                           int& row0, int& lo, int& hi) {
  const int4 e = tab[tile];
  row0 = min((unsigned)__builtin_amdgcn_readfirstlane(e.x), (unsigned)((rows - 1) / bm)) * bm;
  lo = min(max(__builtin_amdgcn_readfirstlane(e.y), 0), others);
  hi = min(max(__builtin_amdgcn_readfirstlane(e.z), 0), others);
}

// Where the tiles are too few to fill the card, a tile's loop is cut into
// parts whose float32 sums go to memory and are joined by a second kernel.
__device__ __forceinline__ void part_of(int n, int parts, int part, int& begin, int& end) {
  const int each = parts == 1 ? n : (n + parts - 1) / parts;
  begin = min(part * each, n);
  end = min(begin + each, n);
}

}  // namespace poetx

// Attention of one query row per sequence over a cache, on MFMA tiles.
//
// The query heads that share a key head are the columns of one 32-wide score
// tile, so the cache is read once for the whole group.  The pass is bound by
// that read: with a group of 4, seven of eight columns are idle, and the
// products still take a sixth of the time that the cache takes to arrive.
// A workgroup takes a piece of one sequence's range for one key head; each of
// its four waves streams 32-row key and value tiles of its own through LDS
// without any barrier (the next key tile is requested as soon as the scores
// are formed, the next value tile as soon as the sums are).  Waves join in
// LDS, pieces in a second small kernel, in a fixed order.
// bf16 operands hold a probability in two parts (score_parts): twice the value
// products, which the read hides but for 1% (16 long sequences 234.7 us, from
// one part 232.8), and o is off by its own rounding alone (2-norm 1.66e-3, from
// one part 1.80e-3).
//
// Measured (bf16, 32 heads on 8, D 128): 16 sequences of 8000 to 32768 rows
// 233 us = 6.1 TB/s (a copy of 1 GiB moves 5.0, reading alone 6.5); one
// sequence of up to 1024 rows 13 us, two launches.  float32 with a group of 4
// is bound by its products (one column in eight is used): 220 MB in 61 us.
// 64 sequences on rings, window 4096 with 4 sinks: 183 us = 5.8 TB/s.
#include <algorithm>

#include "attn_tile.h"
#include "decode_join.h"
#include "decode_view.h"

namespace poetx {

namespace {

constexpr int NW = 4;          // waves a workgroup
constexpr int BN = 32;         // keys a tile
constexpr int GRAIN = NW * BN; // a piece is a multiple of this
constexpr int MAX_PIECES = 64;

// Pieces that a sequence is cut into at most: 2048 workgroups, so that unequal
// lengths even out over the 512 resident ones, in pieces of 512 rows at least
// (a piece's start and join cost as much as a hundred rows: 8 sequences of up
// to 4096 rows 33.3 us in pieces of 128, 27.3 in 512); but one workgroup a CU
// from 128 rows on, where latency counts.
int pieces_of(const DecodeArgs& a) {
  const int per = a.B * a.Hkv * ((a.group + 31) / 32), rows = (int)std::min(view_rows(a, BN), (long)INT32_MAX - 65535);
  const auto cut = [&](int fill, int least) { return std::min((fill + per - 1) / per, (rows + least - 1) / least); };
  return std::max(1, std::min(std::max(cut(2048, 512), cut(256, GRAIN)), MAX_PIECES));
}

// the sequence's range and the piece length in effect
__device__ __forceinline__ void range_of(const DecodeArgs& a, int b, int pieces, int& lo, int& hi, int& piece) {
  hi = min(max(a.len[b], 0), a.rows);
  lo = a.start ? min(max(a.start[b], 0), hi) : 0;
  piece = piece_of(hi - lo, pieces, GRAIN);
}

// the same with a window: the padded rows of its view
__device__ __forceinline__ void range_of(const DecodeArgs& a, int b, int pieces, View& v, int& lo, int& hi, int& piece) {
  v.init<BN, false>(a, a.len[b], 0);
  lo = 0;
  hi = v.total;
  piece = piece_of(v.total, pieces, GRAIN);
}

template <bool WIN> struct Pieces {
  int pieces;
  __device__ __forceinline__ int find(const DecodeArgs& a, int b, int h, long& at) const {
    int lo, hi, piece;
    View v;
    if constexpr (WIN) range_of(a, b, pieces, v, lo, hi, piece);
    else range_of(a, b, pieces, lo, hi, piece);
    at = ((long)b * a.Hq + h) * pieces;
    return hi - lo <= piece ? 1 : (hi - lo + piece - 1) / piece;
  }
};

// WIN: the rows are those of a View, tile by tile
template <typename T, int DP, int MODE, bool WIN>
__global__ __launch_bounds__(64 * NW, sizeof(T) == 4 && DP == 128 ? 1 : 2) void k_attn_decode(DecodeArgs a, int pieces, float* part, float* ml) {
  using L = Tile<T, DP>;
  constexpr int TILE = BN * L::RB;
  constexpr int NL = TILE / 1024;  // loads of a tile
  extern __shared__ __align__(16) char smem[];
  const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int s = blockIdx.x, b = blockIdx.z;
  const int groups = (a.group + 31) / 32;
  const int hk = blockIdx.y / groups, g0 = 32 * (blockIdx.y % groups);
  const int heads = min(a.group - g0, 32), h0 = hk * a.group + g0;
  int lo, hi, piece;
  View view;
  if constexpr (WIN) range_of(a, b, pieces, view, lo, hi, piece);
  else range_of(a, b, pieces, lo, hi, piece);
  const int p0 = lo + s * piece, p1 = min(p0 + piece, hi);
  if (s > 0 && p0 >= hi) return;
  // rows [row, end) of the tile at j (past the piece: none), and the position
  // of its first row
  const auto rows_at = [&](int j, int& row, int& end, int& pos) {
    if constexpr (WIN) {
      row = end = pos = 0;
      if (j < p1) {
        int begin, shift;
        view.tile<BN, false>(j, row, begin, end, shift);
        pos = row + shift;
      }
    } else {
      row = pos = j;
      end = p1;
    }
  };

  const T* kp = (const T*)a.k + (long)b * a.bsk + (long)hk * a.D;
  const T* vp = (const T*)a.v + (long)b * a.bsv + (long)hk * a.D;
  uint4 qf[L::KS];
  rows_to_regs<T>(qf, (const T*)a.q + (long)b * a.ldq + (long)h0 * a.D, a.D, 0, heads, a.D, lane);
  const int head = lane & 31;
  const bool in = head < heads;
  const ScoreArgs sa = score_args<T, MODE>(a.scale, a.cap, MODE & 2 ? a.slopes[h0 + min(head, heads - 1)] : 0.0f);

  Loader<T, DP, BN, 1, true> lk, lv;
  lk.init(a.ldk, a.D, 0, lane);
  lv.init(a.ldv, a.D, 0, lane);
  const uint32_t kr = L::row_lane(lane) + wave * 2 * TILE, vc = L::col_lane(lane) + (wave * 2 + 1) * TILE;
  const uint32_t ldsk = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)smem + wave * 2 * TILE;
  const uint32_t ldsv = ldsk + TILE;

  f32x16_t o[L::NT];
#pragma unroll
  for (int i = 0; i < L::NT; ++i) o[i] = (f32x16_t){};
  float m = -INFINITY, l = 0.0f;
  int j0 = p0 + wave * BN;
  wait_loads();  // counts below are of tile loads only
  int row, end, pos;
  rows_at(j0, row, end, pos);
  if (j0 < p1) {
    lk.load(kp, a.ldk, row, end, ldsk);
    lv.load(vp, a.ldv, row, end, ldsv);
  }
  const int last = WIN ? view.last : hi - 1;
  for (; j0 < p1; j0 += GRAIN) {
    // the key tile has landed when only the value tile's loads are pending
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(NL) : "memory");
    f32x16_t sc = {};
#pragma unroll
    for (int ks = 0; ks < L::KS; ++ks) sc = mma16((const T*)nullptr, L::row_frag(smem, kr, 0, ks), qf[ks], sc);
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    const int jn = min(j0 + GRAIN, p1);  // a load past the piece has no rows: zeros
    // counted from the tile's first row: a position behind the query may pass 2^31
    const int jl = 4 * (lane >> 5), jend = end - row;
    const float d0 = (float)(last - pos - jl);
    rows_at(jn, row, end, pos);
    lk.load(kp, a.ldk, row, end, ldsk);
    float top = -INFINITY, unused;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int j = jl + 8 * (i / 4) + i % 4;
      sc[i] = score2<T, MODE>(sc[i], sa, d0 - (float)(8 * (i / 4) + i % 4), unused);
      sc[i] = j < jend ? sc[i] : -INFINITY;
      top = fmaxf(top, sc[i]);
    }
    top = fmaxf(top, other_half(top));
    const float m2 = fmaxf(m, top), ref = m2 == -INFINITY ? 0.0f : m2;
    const float f = exp2_hw(m - ref);
    m = m2;
    l *= f;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      sc[i] = exp2_hw(sc[i] - ref);
      l += sc[i];
    }
#pragma unroll
    for (int i = 0; i < L::NT; ++i)
#pragma unroll
      for (int r = 0; r < 16; ++r) o[i][r] *= f;
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(NL) : "memory");
#pragma unroll
    for (int u = 0; u < L::CSTEP; ++u) {
      uint4 p, rest;
      if constexpr (sizeof(T) == 2) L::score_parts(sc, u, p, rest);
      else p = L::score_frag(sc, u);
#pragma unroll
      for (int ct = 0; ct < L::NT; ++ct) {
        const uint4 f = L::col_frag(smem, vc, 0, u, ct);
        o[ct] = mma16((const T*)nullptr, f, p, o[ct]);
        if constexpr (sizeof(T) == 2) o[ct] = mma16((const T*)nullptr, f, rest, o[ct]);
      }
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    lv.load(vp, a.ldv, row, end, ldsv);
  }
  l += other_half(l);

  // the four waves join: a common maximum, then their sums in wave order
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  float* wm = reinterpret_cast<float*>(smem);      // [NW][32] maxima, then [NW][32] sums
  float* wo = wm + 2 * NW * 32;                    // [NW][32][DP]
  if (lane < 32) {
    wm[wave * 32 + head] = m;
    wm[(NW + wave) * 32 + head] = l;
  }
#pragma unroll
  for (int ct = 0; ct < L::NT; ++ct)
#pragma unroll
    for (int g = 0; g < 4; ++g)
      if (in)
        *reinterpret_cast<float4*>(wo + (wave * 32 + head) * DP + 32 * ct + 8 * g + 4 * (lane >> 5)) =
            make_float4(o[ct][4 * g], o[ct][4 * g + 1], o[ct][4 * g + 2], o[ct][4 * g + 3]);
  __syncthreads();
  const bool whole = hi - lo <= piece;  // one piece: this is the result
  for (int e = threadIdx.x; e < heads * DP; e += 64 * NW) {
    const int hh = e / DP, d = e % DP;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < NW; ++w) M = fmaxf(M, wm[w * 32 + hh]);
    const float ref = M == -INFINITY ? 0.0f : M;
    float sum = 0.0f, lsum = 0.0f;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
      const float f = exp2_hw(wm[w * 32 + hh] - ref);
      lsum += f * wm[(NW + w) * 32 + hh];
      sum += f * wo[(w * 32 + hh) * DP + d];
    }
    const int h = h0 + hh;
    if (whole) {
      if (d < a.D) St<T>::st((T*)a.o + (long)b * a.ldo + (long)h * a.D + d, lsum == 0.0f ? 0.0f : sum / lsum);
    } else {
      const long at = ((long)b * a.Hq + h) * pieces + s;
      if (d < a.D) part[at * a.D + d] = sum;
      if (d == 0) {
        ml[2 * at] = M;
        ml[2 * at + 1] = lsum;
      }
    }
  }
}

size_t part_floats(const DecodeArgs& a) { return (size_t)a.B * a.Hq * pieces_of(a) * a.D; }

template <typename T, int DP, int MODE, bool WIN> hipError_t decode(const DecodeArgs& a, float* ws, hipStream_t s) {
  constexpr int lds = std::max(NW * 2 * BN * Tile<T, DP>::RB, (2 * NW * 32 + NW * 32 * DP) * 4);
  const hipError_t e = lds_opt_in((const void*)k_attn_decode<T, DP, MODE, WIN>, lds);
  if (e != hipSuccess) return e;
  const int pieces = pieces_of(a);
  float* ml = ws + part_floats(a);
  k_attn_decode<T, DP, MODE, WIN><<<dim3(pieces, a.Hkv * ((a.group + 31) / 32), a.B), 64 * NW, lds, s>>>(a, pieces, ws, ml);
  const hipError_t e2 = hipGetLastError();
  if (e2 != hipSuccess || pieces == 1) return e2;
  k_attn_decode_join<T><<<dim3(a.Hq, a.B), 64 * NW, 0, s>>>(a, Pieces<WIN>{pieces}, ws, ml);
  return hipGetLastError();
}

template <typename T, int DP> hipError_t decode_mode(const DecodeArgs& a, float* ws, hipStream_t s) {
  return by_mode<T>(a.slopes, a.cap, [&](auto mode) {
    constexpr int MODE = decltype(mode)::value;
    return a.window ? decode<T, DP, MODE, true>(a, ws, s) : decode<T, DP, MODE, false>(a, ws, s);
  });
}

}  // namespace

size_t attn_decode_ws_bytes(const DecodeArgs& a) {
  return (part_floats(a) + (size_t)a.B * a.Hq * pieces_of(a) * 2) * 4;
}

template <typename T> hipError_t launch_attn_decode(const DecodeArgs& a, float* ws, hipStream_t s) {
  return a.D <= 64 ? decode_mode<T, 64>(a, ws, s) : decode_mode<T, 128>(a, ws, s);
}

template hipError_t launch_attn_decode<bf16>(const DecodeArgs&, float*, hipStream_t);
template hipError_t launch_attn_decode<float>(const DecodeArgs&, float*, hipStream_t);

}  // namespace poetx

// Attention of one query row per sequence over a cache in 4 bits (kv4.hip for
// the format), on MFMA tiles.
//
// The query heads that share a key head are the columns of 16-wide tiles: up to
// 16 of them, or copies of up to 8 or 4, so that every column works: a column of
// copy c keeps the scores of its part of the rows, and has a maximum and sums of
// its own until the end.  Softmax would else be formed in all 64 lanes for 4
// heads' worth of scores.  A workgroup takes a piece of one sequence's rows for one key
// head; each of its four waves goes through 64-row tiles of its own without any
// barrier, the next tile's codes on their way to registers.
//   Scores: lane (r, g) = (lane % 16, lane / 16) loads block g of row 16 t +
// 4 (r % 4) + r / 4, t = 0..3: sixteen bytes are 32 codes, which the conversion
// with a scale turns into exact bf16 numbers in the order of the A operand (K = 8
// elements of each of the four blocks; the queries are laid out alike).  Four
// neighbouring rows' scales of a block are one dword; this order of rows leaves
// every quad of lanes the same four dwords to take a byte of.  D[row][query]
// leaves lane (query, h) the rows 16 t + 4 i + h.
//   Each load takes a whole KB.  In rows 4 r + t, whose scales would need no
// exchange, two loads share every 128 bytes, and a cache that is read past the
// others (non-temporal) twice: 91 us for the 16 sequences below.
//   Values: sum over rows, so the operand is the transposed tile.  Converted
// values go through LDS, 32 rows of t and t + 1 at a time, and come back down their
// columns by ds_read_b64_tr_b16 in just that order of rows; 16-byte chunk c of
// row r lies at c ^ key(r), which spreads both accesses over the banks.
//
// Measured (bf16, 32 heads on 8, D 128): 16 sequences of 8000 to 32768 rows 82 us
// with the join, 4.6 TB/s, 5.8 to 6.3 where all are equally long (the bf16 cache
// 233 us); bound by the read, and by the longest sequences' pieces at the end.  One
// sequence of up to 1024 rows 13.5 us, two launches.
//
//   bf16 queries have probabilities in two bf16 parts, float32 ones both
// queries and probabilities in three: every product is exact, sums are float32.
#include <algorithm>

#include "attn_tile.h"
#include "decode_join.h"
#include "decode_view.h"

namespace poetx {

namespace {

constexpr int NW = 4;           // waves a workgroup
constexpr int BN = 64;          // rows a tile
constexpr int GRAIN = NW * BN;  // a piece is a multiple of this
constexpr int COLS = 16;        // columns of a tile: copies times heads
constexpr int MAX_PIECES = 64;
// The reference of the exponentials moves only when a score passes it by more
// than this (log2): float32 sums hold probabilities up to 2^8 as well, and
// without a move no lane has to hear of the others' maxima.
constexpr float SLACK = 8.0f;

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2_t __attribute__((ext_vector_type(2)));

__device__ __forceinline__ f32x4 mma(uint4 a, uint4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(a), as_bf16x8(b), c, 0, 0, 0);
}

// eight codes times a scale, as bf16
__device__ __forceinline__ uint4 expand(uint32_t c, float scale) {
  uint4 u;
  u.x = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 0));
  u.y = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 1));
  u.z = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 2));
  u.w = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 3));
  return u;
}
// scale of this lane's row of tile t: byte `shift` / 8 of lane 4 t + lane % 4 of
// these 16
template <int t> __device__ __forceinline__ float scale_of(uint32_t bytes, int shift) {
  const uint32_t d = (uint32_t)__builtin_amdgcn_ds_swizzle((int)bytes, t << 7 | 0x13);
  return __uint_as_float((d >> shift & 0xffu) << 23);
}

// x (>= 0, or any float for queries) as N bf16 parts: pack[n] gets part n of two
template <int N> __device__ __forceinline__ void parts2(float x, float y, uint32_t (&p)[N]) {
#pragma unroll
  for (int n = 0; n < N; ++n) {
    p[n] = pack2bf(x, y);
    x -= __uint_as_float(p[n] << 16);
    y -= __uint_as_float(p[n] & 0xffff0000u);
  }
}

// copies of the heads among the columns
int copies_of(const DecodeArgs& a) { return a.group <= 4 ? 4 : a.group <= 8 ? 2 : 1; }
int groups_of(const DecodeArgs& a) { return (a.group + COLS / copies_of(a) - 1) / (COLS / copies_of(a)); }

// Pieces that a sequence is cut into at most: two rounds of the workgroups that
// run at once, 2 to 4 a CU by their registers, in pieces of 1024 rows at least (16
// sequences of 8000 to 32768 rows: 82 us with two rounds, 84 to 98 with 1024, 2048
// or 4096 workgroups; 8 in float32 57, and 64 to 68); but one workgroup a CU from
// 256 rows on, where latency counts.  Pieces of one length over all sequences,
// found from the lengths by every wave, were slower: 100 us.
template <typename T> int pieces_of(const DecodeArgs& a) {
  const int per = a.B * a.Hkv * groups_of(a), rows = (int)std::min(view_rows(a, BN), (long)INT32_MAX - 65535);
  const int resident = 256 * (a.D <= 64 ? 4 : sizeof(T) == 2 ? 3 : 2);
  const auto cut = [&](int fill, int least) { return std::min((fill + per - 1) / per, (rows + least - 1) / least); };
  return std::max(1, std::min(std::max(cut(2 * resident, 1024), cut(256, GRAIN)), MAX_PIECES));
}

struct Pieces {
  int pieces;
  __device__ __forceinline__ int find(const DecodeArgs& a, int b, int h, long& at) const {
    View v;
    v.init<BN, true>(a, a.len[b], a.start ? a.start[b] : 0);
    const int piece = piece_of(v.total, pieces, GRAIN);
    at = ((long)b * a.Hq + h) * pieces;
    return v.total <= piece ? 1 : (v.total + piece - 1) / piece;
  }
};

// NBK: blocks a head, rounded up to 2 or 4; nb of them are there
template <typename T, int NBK, int MODE, int COPIES>
__global__ __launch_bounds__(64 * NW, 2) void k_attn_kv4(DecodeArgs a, int nb, int pieces, float* part, float* ml) {
  constexpr int DP = 32 * NBK, NT = DP / 16, RB = 2 * DP;
  constexpr int PQ = sizeof(T) == 2 ? 1 : 3, PP = sizeof(T) == 2 ? 2 : 3;
  constexpr int STAGE = 32 * RB;  // bytes of a wave's 32 rows of values
  constexpr int HEADS = COLS / COPIES, TPL = 4 / COPIES;  // heads a workgroup; tiles whose scores a lane keeps
  extern __shared__ __align__(16) char smem[];
  const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
  const int r = lane & 15, g = lane >> 4;
  const int copy = r / HEADS, head_r = r % HEADS;  // of column r
  const int s = blockIdx.x, b = blockIdx.z;
  const int groups = (a.group + HEADS - 1) / HEADS;
  const int hk = blockIdx.y / groups, g0 = HEADS * (blockIdx.y % groups);
  const int heads = min(a.group - g0, HEADS), h0 = hk * a.group + g0;
  View view;
  view.init<BN, true>(a, a.len[b], a.start ? a.start[b] : 0);
  const int piece = piece_of(view.total, pieces, GRAIN);
  const int p0 = s * piece, p1 = min(p0 + piece, view.total);
  if (s > 0 && p0 >= view.total) return;

  const int blk = NBK == 4 ? g : g >> 1;  // this lane's block of a row
  const bool there = blk < nb;
  const long plane = (long)b * a.Hkv + hk;
  const int rowb = nb * 16;
  const uint8_t* kc = (const uint8_t*)a.k + plane * a.rows * rowb;
  const uint8_t* vc = (const uint8_t*)a.v + plane * a.rows * rowb;
  const uint8_t* ks = a.ks + (plane * nb + (there ? blk : 0)) * a.rows + 4 * r;
  const uint8_t* vs = a.vs + (plane * nb + (there ? blk : 0)) * a.rows + 4 * r;
  const int off = (4 * (r & 3) + (r >> 2)) * rowb + (there ? g * (4 * NBK) : 0), byte = 8 * (r >> 2);

  const ScoreArgs sa = score_args<T, MODE>(a.scale, a.cap, MODE & 2 ? a.slopes[h0 + min(head_r, heads - 1)] : 0.0f);

  // The next tile's keys are asked for as soon as the scores are formed, its
  // values as soon as this tile's are in LDS: in the registers that these leave.
  struct Codes { uint32_t c[4][NBK], scales; };
  const auto fetch = [&](const uint8_t* codes, const uint8_t* scales, int row, Codes& o) {
    o.scales = *reinterpret_cast<const uint32_t*>(scales + row);
    const uint8_t* p = codes + (long)row * rowb + off;
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      if constexpr (NBK == 4) {
        const u32x4_t u = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t*>(p + 16 * t * rowb));
        o.c[t][0] = u[0], o.c[t][1] = u[1], o.c[t][2] = u[2], o.c[t][3] = u[3];
      } else {
        const u32x2_t u = __builtin_nontemporal_load(reinterpret_cast<const u32x2_t*>(p + 16 * t * rowb));
        o.c[t][0] = u[0], o.c[t][1] = u[1];
      }
    }
  };
  const auto blank = [&](Codes& o) {  // no such block: zero
    if (there) return;
    o.scales = 0x7f7f7f7fu;
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int i = 0; i < NBK; ++i) o.c[t][i] = 0;
  };

  // LDS of this wave: row n at n * RB, chunk c of it at c ^ key(n)
  // (eight rows that are read together lie in eight pairs of chunks)
  const auto key = [](int n) { return NBK == 4 ? (n & 7) << 1 | (n >> 3 & 1) : (n >> 1 & 3) << 1 | (n >> 3 & 1); };
  char* stage = smem + wave * STAGE;
  const int wr = r * RB + ((NBK * g ^ key(r)) << 4);  // first chunk written; + 16 rows: the same key
  // transposed read: lane i of 16 gives 4 columns of row 4 g + i / 4
  const int tr_row = 4 * g + (r >> 2);
  const int tr = tr_row * RB + ((((r & 3) >> 1) ^ key(tr_row)) << 4) + (r & 1) * 8;

  f32x4 o[NT];
#pragma unroll
  for (int i = 0; i < NT; ++i) o[i] = (f32x4){};
  float m = -INFINITY, l = 0.0f;
  int j0 = p0 + wave * BN;
  Codes k, v;
  int row = 0, begin = 0, end = 0, shift = 0;
  if (j0 < p1) {
    view.tile<BN, true>(j0, row, begin, end, shift);
    fetch(kc, ks, row, k);
    fetch(vc, vs, row, v);
  }
  // queries: column r, elements 8 NBK g + 8 c of step c
  uint4 qf[PQ][NBK];
  {
    const T* q = (const T*)a.q + (long)b * a.ldq + (long)(h0 + min(head_r, heads - 1)) * a.D;
    struct alignas(16) Eight { T e[8]; } x[NBK];
#pragma unroll
    for (int c = 0; c < NBK; ++c) {
      const int e = 8 * NBK * g + 8 * c;
      x[c] = *reinterpret_cast<const Eight*>(q + (e < a.D ? e : 0));
    }
#pragma unroll
    for (int c = 0; c < NBK; ++c) {
      const bool in = 8 * NBK * g + 8 * c < a.D && head_r < heads;
      uint32_t p[4][PQ];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        parts2<PQ>(in ? St<T>::ld(&x[c].e[2 * i]) : 0.0f, in ? St<T>::ld(&x[c].e[2 * i + 1]) : 0.0f, p[i]);
#pragma unroll
      for (int n = 0; n < PQ; ++n) qf[n][c] = make_uint4(p[0][n], p[1][n], p[2][n], p[3][n]);
    }
  }
  for (; j0 < p1; j0 += GRAIN) {
    blank(k);
    f32x4 all[4];
    const float kscale[4] = {scale_of<0>(k.scales, byte), scale_of<1>(k.scales, byte), scale_of<2>(k.scales, byte),
                             scale_of<3>(k.scales, byte)};
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      const float scale = kscale[t];
      all[t] = (f32x4){};
#pragma unroll
      for (int i = 0; i < NBK; ++i) {
        const uint4 f = expand(k.c[t][i], scale);
#pragma unroll
        for (int n = 0; n < PQ; ++n) all[t] = mma(f, qf[n][i], all[t]);
      }
    }
    const bool more = j0 + GRAIN < p1;
    int nrow = 0, nbegin = 0, nend = 0, nshift = 0;
    if (more) {
      view.tile<BN, true>(j0 + GRAIN, nrow, nbegin, nend, nshift);
      fetch(kc, ks, nrow, k);
    }
    // this lane's scores: rows row + 16 (TPL copy + x) + 4 i + g
    f32x4 sc[TPL];
#pragma unroll
    for (int x = 0; x < TPL; ++x) {
      sc[x] = all[x];
#pragma unroll
      for (int n = 1; n < COPIES; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i) sc[x][i] = copy == n ? all[n * TPL + x][i] : sc[x][i];
    }
    const int first = row + 16 * TPL * copy + g;
    const float d0 = (float)(view.last - shift - first);
    float top = -INFINITY, unused;
#pragma unroll
    for (int x = 0; x < TPL; ++x)
#pragma unroll
      for (int i = 0; i < 4; ++i) sc[x][i] = score2<T, MODE>(sc[x][i], sa, d0 - (float)(16 * x + 4 * i), unused);
    blank(v);
    if (begin > row || end < row + BN) {  // some row is not seen: no score, and a value of 0
#pragma unroll
      for (int x = 0; x < TPL; ++x)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int j = first + 16 * x + 4 * i;
          sc[x][i] = j >= begin && j < end ? sc[x][i] : -INFINITY;
        }
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const int jv = row + 4 * r + t;  // row of the scale
        if (jv < begin || jv >= end) v.scales &= ~(0xffu << (8 * t));
      }
    }
#pragma unroll
    for (int x = 0; x < TPL; ++x)
#pragma unroll
      for (int i = 0; i < 4; ++i) top = fmaxf(top, sc[x][i]);
    if (__any(top > m + SLACK)) {
      top = fmaxf(top, __shfl_xor(top, 16));
      top = fmaxf(top, __shfl_xor(top, 32));
      const float m2 = fmaxf(m, top);
      const float f = m2 == -INFINITY ? 1.0f : exp2_hw(m - m2);
      m = m2;
      l *= f;
#pragma unroll
      for (int i = 0; i < NT; ++i) o[i] *= f;
    }
    const float ref = m == -INFINITY ? 0.0f : m;
    uint32_t pk[TPL][2][PP];  // probabilities as operands
#pragma unroll
    for (int x = 0; x < TPL; ++x) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        sc[x][i] = exp2_hw(sc[x][i] - ref);
        l += sc[x][i];
      }
      parts2<PP>(sc[x][0], sc[x][1], pk[x][0]);
      parts2<PP>(sc[x][2], sc[x][3], pk[x][1]);
    }
    const float vscale[4] = {scale_of<0>(v.scales, byte), scale_of<1>(v.scales, byte), scale_of<2>(v.scales, byte),
                             scale_of<3>(v.scales, byte)};
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const float scale = vscale[2 * u + x];
#pragma unroll
        for (int i = 0; i < NBK; ++i)
          *reinterpret_cast<uint4*>(stage + (wr ^ (i << 4)) + x * 16 * RB) = expand(v.c[2 * u + x][i], scale);
      }
      if (u == 1 && more) fetch(vc, vs, nrow, v);
      // rows (2 u, 2 u + 1): a column has those of its copy, zeros elsewhere
      uint4 p[PP];
#pragma unroll
      for (int n = 0; n < PP; ++n) {
        if constexpr (COPIES == 1) {
          p[n] = make_uint4(pk[2 * u][0][n], pk[2 * u][1][n], pk[2 * u + 1][0][n], pk[2 * u + 1][1][n]);
        } else if constexpr (COPIES == 2) {
          const bool on = copy == u;
          p[n] = make_uint4(on ? pk[0][0][n] : 0, on ? pk[0][1][n] : 0, on ? pk[1][0][n] : 0, on ? pk[1][1][n] : 0);
        } else {
          const bool on0 = copy == 2 * u, on1 = copy == 2 * u + 1;
          p[n] = make_uint4(on0 ? pk[0][0][n] : 0, on0 ? pk[0][1][n] : 0, on1 ? pk[0][0][n] : 0, on1 ? pk[0][1][n] : 0);
        }
      }
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int ct = 0; ct < NT; ++ct) {
        char* at = stage + (tr ^ (ct << 5));
        const s16x4_t v0 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)at);
        const s16x4_t v1 = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4_t*)(at + 16 * RB));
        const uint4 f = __builtin_bit_cast(uint4, __builtin_shufflevector(v0, v1, 0, 1, 2, 3, 4, 5, 6, 7));
#pragma unroll
        for (int n = 0; n < PP; ++n) o[ct] = mma(f, p[n], o[ct]);
      }
      __builtin_amdgcn_wave_barrier();
    }
    row = nrow, begin = nbegin, end = nend, shift = nshift;
  }
  l += __shfl_xor(l, 16);
  l += __shfl_xor(l, 32);

  // the waves' columns join: a common maximum, then their sums in order
  __syncthreads();
  float* wm = reinterpret_cast<float*>(smem);     // [NW][COLS] maxima, then [NW][COLS] sums
  float* wo = wm + 2 * NW * COLS;                 // [NW][COLS][DP]
  if (lane < COLS) {
    wm[wave * COLS + r] = m;
    wm[(NW + wave) * COLS + r] = l;
  }
#pragma unroll
  for (int ct = 0; ct < NT; ++ct)
    *reinterpret_cast<f32x4*>(wo + (wave * COLS + r) * DP + 16 * ct + 4 * g) = o[ct];
  __syncthreads();
  const bool whole = view.total <= piece;  // one piece: this is the result
  if (threadIdx.x < COLS) {  // the factors of a head's columns, and its sum
    const int hh = threadIdx.x % HEADS;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < NW * COPIES; ++w) M = fmaxf(M, wm[w * HEADS + hh]);
    const float ref = M == -INFINITY ? 0.0f : M;
    float lsum = 0.0f, f[NW];
#pragma unroll
    for (int w = 0; w < NW * COPIES; ++w) {
      const float x = exp2_hw(wm[w * HEADS + hh] - ref);
      lsum += x * wm[NW * COLS + w * HEADS + hh];
      if (w % COPIES == threadIdx.x / HEADS) f[w / COPIES] = x;
    }
    float* wf = wo + NW * COLS * DP;  // [NW][COLS] factors, [COLS] maxima, [COLS] sums
#pragma unroll
    for (int w = 0; w < NW; ++w) wf[w * COLS + threadIdx.x] = f[w];
    wf[NW * COLS + threadIdx.x] = M;
    wf[(NW + 1) * COLS + threadIdx.x] = lsum;
  }
  __syncthreads();
  const float* wf = wo + NW * COLS * DP;
  for (int e = threadIdx.x; e < heads * DP; e += 64 * NW) {
    const int hh = e / DP, d = e % DP;
    float sum = 0.0f;
#pragma unroll
    for (int w = 0; w < NW * COPIES; ++w) sum = fmaf(wf[w * HEADS + hh], wo[(w * HEADS + hh) * DP + d], sum);
    const float M = wf[NW * COLS + hh], lsum = wf[(NW + 1) * COLS + hh];
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

template <typename T> size_t part_floats(const DecodeArgs& a) { return (size_t)a.B * a.Hq * pieces_of<T>(a) * a.D; }

template <typename T, int NBK, int MODE, int COPIES> hipError_t decode(const DecodeArgs& a, float* ws, hipStream_t s) {
  constexpr int DP = 32 * NBK, lds = std::max(NW * 32 * 2 * DP, (2 * NW * COLS + NW * COLS * DP + (NW + 2) * COLS) * 4);
  const hipError_t e = lds_opt_in((const void*)k_attn_kv4<T, NBK, MODE, COPIES>, lds);
  if (e != hipSuccess) return e;
  const int pieces = pieces_of<T>(a), nb = kv4_blocks(a.D);
  float* ml = ws + part_floats<T>(a);
  k_attn_kv4<T, NBK, MODE, COPIES><<<dim3(pieces, a.Hkv * groups_of(a), a.B), 64 * NW, lds, s>>>(a, nb, pieces, ws, ml);
  const hipError_t e2 = hipGetLastError();
  if (e2 != hipSuccess || pieces == 1) return e2;
  k_attn_decode_join<T><<<dim3(a.Hq, a.B), 64 * JOIN_WAVES, 0, s>>>(a, Pieces{pieces}, ws, ml);
  return hipGetLastError();
}

template <typename T, int NBK> hipError_t decode_mode(const DecodeArgs& a, float* ws, hipStream_t s) {
  return by_mode<T>(a.slopes, a.cap, [&](auto mode) {
    constexpr int MODE = decltype(mode)::value;
    const int n = copies_of(a);
    return n == 4 ? decode<T, NBK, MODE, 4>(a, ws, s) : n == 2 ? decode<T, NBK, MODE, 2>(a, ws, s) : decode<T, NBK, MODE, 1>(a, ws, s);
  });
}

}  // namespace

template <typename T> size_t attn_kv4_ws_bytes(const DecodeArgs& a) {
  return (part_floats<T>(a) + (size_t)a.B * a.Hq * pieces_of<T>(a) * 2) * 4;
}

template <typename T> hipError_t launch_attn_kv4(const DecodeArgs& a, float* ws, hipStream_t s) {
  return a.D <= 64 ? decode_mode<T, 2>(a, ws, s) : decode_mode<T, 4>(a, ws, s);
}

template size_t attn_kv4_ws_bytes<bf16>(const DecodeArgs&);
template size_t attn_kv4_ws_bytes<float>(const DecodeArgs&);
template hipError_t launch_attn_kv4<bf16>(const DecodeArgs&, float*, hipStream_t);
template hipError_t launch_attn_kv4<float>(const DecodeArgs&, float*, hipStream_t);

}  // namespace poetx

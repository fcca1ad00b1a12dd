// Host-side launchers and argument blocks of the attention-block operators
// (internal to libpoetx.so).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "common.h"

namespace poetx {

// A dispatch counts its threads in 32 bits, and what is past them is not run,
// without an error: larger work goes out in launches of at most this many.
constexpr long LAUNCH_THREADS = 1L << 31;

// ---- rotary positions (rope.hip) -------------------------------------------
struct RopeArgs {
  int T, Hq, Hk, D, rot, P, interleaved;
  float sgn;  // -1: inverse
  long ldq, ldk, ldqo, ldko;
  const int* pos;
  const float* table;
};
template <typename TS>
hipError_t launch_rope(const RopeArgs& a, const TS* q, const TS* k, TS* qo, TS* ko, hipStream_t s);

// ---- dropout (dropout.hip) --------------------------------------------------
// out[i] = (res ? res[i] : 0) + (keep(i) ? x[i] * gain : 0)
template <typename TS>
hipError_t launch_dropout(long n, const TS* x, const TS* res, TS* out, uint32_t cut, uint64_t seed,
                          uint64_t offset, const uint64_t* offset_dev, hipStream_t s);

// ---- attention (attn_*.hip) -------------------------------------------------
constexpr int ATTN_BM = 128;  // query (key) rows of a tile

// About the rows of the other side that a tile's loop goes through: a
// document's, and those of the documents that a tile spans.
inline long loop_rows(int others, int own, int ndoc) {
  const long r = others / (ndoc > 1 ? ndoc : 1) + (long)ATTN_BM * others / (own > 1 ? own : 1);
  return r < others ? r : others;
}

// Parts that a loop over about `rows` rows is cut into where `groups`
// workgroups run it; 16 at most.  bf16: up to one workgroup a CU, or two
// where a part still has 768 rows; cutting shorter loops costs more in
// partial sums than it evens out (1024 causal tokens, 32 heads on 8: one
// training pass 127 us with two a CU, 103 with one).  float32 products take
// eight times as long, so the traffic counts less and a loop that ends last
// is waited for longer: up to four a CU (two documents of 1024, 16 heads of
// 64: 330 us with four, 354 with eight), in parts of `least` rows, a
// tile of their kernels (765 tokens in 9 documents, 5 heads on 1: 173 us in
// parts of 256 rows, 70 of 64).  All tiles of a launch get the same number,
// from the mean loop: one long document beside many tiny ones is taken for
// short loops.
template <typename T> int parts_for(long groups, long rows, int least) {
  if (groups < 1) return 1;
  const auto cut = [&](long fill, long rows_a_part) {
    const long want = fill / groups, most = rows / rows_a_part;
    return want < most ? want : most;
  };
  const long a = sizeof(T) == 2 ? cut(256, 256) : cut(1024, least), b = sizeof(T) == 2 ? cut(512, 768) : 1;
  const long n = a > b ? a : b;
  return n < 1 ? 1 : n > 16 ? 16 : (int)n;
}

// The mask as intervals: query row t sees keys [row_lo, row_hi), stands at
// key position row_pos; key row j is seen by queries [key_lo, key_hi).
// Within a document both bounds grow with the row, so the rows of any tile
// see one interval's worth of keys.
struct AttnPlan {
  int *row_lo, *row_hi, *row_pos;  // [Tq]
  int *key_lo, *key_hi;            // [Tk]
  // tiles of ATTN_BM query (key) rows in the order they are worked on: {tile,
  // first, end of the keys (queries) that its rows see, 0}
  int4 *qtab, *ktab;
  int4 *qraw, *kraw;               // the same before sorting
};
inline int attn_tiles(int rows) { return (rows + ATTN_BM - 1) / ATTN_BM; }

struct AttnArgs {
  int Tq, Tk, Hq, Hkv, group, D;
  float scale, cap;
  const float* slopes;  // or null
  long ldq, ldk, ldv, ldo, lddo, lddq, lddk, lddv;
  const void *q, *k, *v;
  void* o;
  float* lse;
  // backward
  const void* dout;
  void *dq, *dk, *dv;
  float *delta, *lse2;  // [Hq][Tq] each
  float* part;          // partial sums (attn_ws_bytes)
  int ndoc;
  AttnPlan pl;
};

// (api.hip) LDS above 64 KB for a kernel on the current device
hipError_t lds_opt_in(const void* kern, int bytes);

hipError_t launch_attn_plan(int Tq, int Tk, int ndoc, int causal, const int* cu_q, const int* cu_k,
                            const int* prefix, const AttnPlan& pl, hipStream_t s);
// bytes of a.part for the forward and the backward pass
template <typename TS> size_t attn_fwd_part_bytes(const AttnArgs& a);
template <typename TS> size_t attn_bwd_part_bytes(const AttnArgs& a);
template <typename TS> hipError_t launch_attn_fwd(const AttnArgs& a, hipStream_t s);
template <typename TS> hipError_t launch_attn_bwd(const AttnArgs& a, hipStream_t s);

struct DecodeArgs {
  int B, Hq, Hkv, group, D, rows;
  float scale, cap;
  const float* slopes;
  long ldq, ldo, ldk, ldv, bsk, bsv;
  const void *q, *k, *v;
  void* o;
  const int *start, *len;
};
// ws: attn_decode_ws_bytes(a) bytes for the pieces' partial results
size_t attn_decode_ws_bytes(const DecodeArgs& a);
template <typename TS> hipError_t launch_attn_decode(const DecodeArgs& a, float* ws, hipStream_t s);

}  // namespace poetx

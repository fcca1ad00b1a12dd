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

// ---- norms of queries and keys with rotary positions (qk_norm.hip) -----------
struct QkNormArgs {
  int T, Hq, Hk, D, rot, P, interleaved;
  float eps, inv_d;
  long ldq, ldk, ldqo, ldko, lddq, lddk;  // backward: ldqo, ldko of gq, gk
  const void *q, *k;
  const float *wq, *wk;  // or null: 1
  const int* pos;
  const float* table;
  void *qo, *ko;
  // backward
  const void *gq, *gk;
  void *dq, *dk;
  float *dwq, *dwk;      // or null
};
// ws: qk_norm_ws_bytes(a) bytes for partial sums of dwq, dwk
size_t qk_norm_ws_bytes(const QkNormArgs& a);
template <typename TS> hipError_t launch_qk_norm_fwd(const QkNormArgs& a, hipStream_t s);
template <typename TS> hipError_t launch_qk_norm_bwd(const QkNormArgs& a, float* ws, hipStream_t s);

// ---- dropout (dropout.hip) --------------------------------------------------
// out[i] = (res ? res[i] : 0) + (keep(i) ? x[i] * gain : 0)
template <typename TS>
hipError_t launch_dropout(long n, const TS* x, const TS* res, TS* out, uint32_t cut, uint64_t seed,
                          uint64_t offset, const uint64_t* offset_dev, hipStream_t s);

// ---- attention (attn_*.hip) -------------------------------------------------
constexpr int ATTN_BM = 128;  // query (key) rows of a tile

// About the rows of the other side that a tile's loop goes through: a
// document's, and those of the documents that a tile spans; reach (0: none):
// no more than a window lets its rows see.
inline long loop_rows(int others, int own, int ndoc, long reach) {
  const long r = others / (ndoc > 1 ? ndoc : 1) + (long)ATTN_BM * others / (own > 1 ? own : 1);
  const long most = reach && reach + ATTN_BM < others ? reach + ATTN_BM : others;
  return r < most ? r : most;
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
  // With sinks a query row sees keys [row_sink.x, row_sink.y) besides, which
  // end at or before row_lo.  Those of a tile lie in its range of qtab, or, of
  // its first document, in [qfar.x, qfar.y) below it.
  int2* row_sink;                  // [Tq]
  int2* qfar;                      // [tiles]
  int* tile_doc;                   // [tiles] first document that ends after the tile's first row
  int4* doc;                       // [ndoc] {first query row, end, first key row, end}
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
  int causal, window, sinks;  // window 0: none; sinks 0: none
  float* sink_part;           // backward: partial dk and dv of the sinks
  AttnPlan pl;
  long reach() const { return causal ? window : 2L * window; }
};

// The sinks of a document are seen past the window where some query stands
// further than the window from some key.  Their gradients are then summed
// apart (attn_bwd.hip).  Each such document has a number that grows from one to
// the next: its index, or, where there are fewer of those, its place in windows: two
// of them begin more than a window apart, among the queries or the keys.
__host__ __device__ inline bool sinks_apart(int lq, int lk, int causal, int window) {
  return lk > window || (!causal && lq > window);
}
__host__ __device__ inline long sink_place(int q0, int k0, int window) {
  return q0 / ((long)window + 1) + k0 / ((long)window + 1);
}
__host__ __device__ inline long sink_number(const AttnArgs& a, int d, int q0, int k0) {
  return a.ndoc <= sink_place(a.Tq, a.Tk, a.window) ? d : sink_place(q0, k0, a.window);
}

// (api.hip) LDS above 64 KB for a kernel on the current device
hipError_t lds_opt_in(const void* kern, int bytes);

hipError_t launch_attn_window_plan(int Tq, int Tk, int ndoc, int causal, int window, int sinks,
                                   const int* cu_q, const int* cu_k, const AttnPlan& pl, hipStream_t s);
// bytes of a.sink_part
size_t attn_sink_part_bytes(const AttnArgs& a);
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
  int window, sinks, ring;  // window 0: every row
  const uint8_t *ks, *vs;   // scales of a cache in 4 bits
};
// ---- a cache in 4 bits (kv4.hip, attn_kv4.hip) ---------------------------------
// Blocks of 32 elements: codes [B][Hkv][rows][blocks * 16] bytes, element 2 i
// in the low half of byte i; scales [B][Hkv][blocks][rows].
inline __host__ __device__ int kv4_blocks(int D) { return (D + 31) / 32; }
struct Kv4Args {
  int T, B, rows, Hkv, D, sinks, ring;
  long ldk, ldv;
  const int *seq, *pos;  // seq null: token t is of sequence t
  void *k, *v;           // read from (write) or written (read)
  uint8_t *kc, *ks, *vc, *vs;
};
template <typename TS> hipError_t launch_kv4_write(const Kv4Args& a, hipStream_t s);
template <typename TS> hipError_t launch_kv4_read(const Kv4Args& a, hipStream_t s);
// a.k, a.v: codes
template <typename T> size_t attn_kv4_ws_bytes(const DecodeArgs& a);
template <typename T> hipError_t launch_attn_kv4(const DecodeArgs& a, float* ws, hipStream_t s);

// ws: attn_decode_ws_bytes(a) bytes for the pieces' partial results
size_t attn_decode_ws_bytes(const DecodeArgs& a);
template <typename TS> hipError_t launch_attn_decode(const DecodeArgs& a, float* ws, hipStream_t s);

}  // namespace poetx

// C ABI of the attention-block operators: validation, layouts and dispatch.
// Declarations and argument documentation: include/poetx.h.
#include <math.h>
#include <stdint.h>

#include <algorithm>

#include "../../include/poetx.h"
#include "api_util.h"
#include "attn.h"

using namespace poetx;

namespace {

constexpr int D_MAX = 128;       // attention head width
constexpr int ROPE_D_MAX = 512;
constexpr int H_MAX = 1024;      // heads
constexpr int B_MAX = 65535;     // sequences of a decode call
// packed rows, cache rows: a tile, or a piece of a cut loop, past the last one
// is still an int
constexpr int ROWS_MAX = INT32_MAX - 65535;

int32_t check_act(const char* fn, int32_t act) {
  if (act != POETX_F32 && act != POETX_BF16) return fail(POETX_ERR_ARG, "%s: act dtype %d", fn, act);
  return POETX_OK;
}

// a pitch holds its heads and keeps rows aligned
int32_t check_ld(const char* fn, const char* name, int64_t ld, int64_t width) {
  if (ld < width) return fail(POETX_ERR_ARG, "%s: %s=%lld < %lld", fn, name, (long long)ld, (long long)width);
  if (ld % 8) return fail(POETX_ERR_ARG, "%s: %s=%lld is not a multiple of 8", fn, name, (long long)ld);
  if (ld > (int64_t)1 << 20)
    return fail(POETX_ERR_ARG, "%s: %s=%lld above 2^20", fn, name, (long long)ld);
  return POETX_OK;
}

int32_t check_heads(const char* fn, int32_t Hq, int32_t Hkv, int32_t D) {
  if (Hkv < 1 || Hq < 1 || Hq > H_MAX || Hq % Hkv)
    return fail(POETX_ERR_ARG, "%s: Hq=%d must be a multiple of Hkv=%d, 1..%d", fn, Hq, Hkv, H_MAX);
  if (D < 8 || D % 8 || D > D_MAX)
    return fail(POETX_ERR_ARG, "%s: D=%d must be a multiple of 8, 8..%d", fn, D, D_MAX);
  return POETX_OK;
}

int32_t check_scores(const char* fn, float scale, float cap) {
  if (!isfinite(scale)) return fail(POETX_ERR_ARG, "%s: scale is not finite", fn);
  if (!(cap >= 0.0f) || !isfinite(cap)) return fail(POETX_ERR_ARG, "%s: cap=%g must be finite and >= 0", fn, cap);
  return POETX_OK;
}

// a cap in units of log2 stays finite: above 1e38 float32 scores feel none
float cap_of(float cap) { return fminf(cap, 1e38f); }

#define TRY(x)                          \
  do {                                  \
    const int32_t st_ = (x);            \
    if (st_ != POETX_OK) return st_;    \
  } while (0)

int32_t check_attn(const char* fn, const poetx_attn_shape* sh, bool back) {
  if (!sh) return fail(POETX_ERR_ARG, "%s: null shape", fn);
  if (sh->Tq < 0 || sh->Tk < 0 || sh->ndoc < 0 || sh->ndoc > (1 << 30))
    return fail(POETX_ERR_ARG, "%s: Tq=%d Tk=%d ndoc=%d must be >= 0", fn, sh->Tq, sh->Tk, sh->ndoc);
  if (sh->Tq > ROWS_MAX || sh->Tk > ROWS_MAX)
    return fail(POETX_ERR_ARG, "%s: Tq=%d Tk=%d above %d", fn, sh->Tq, sh->Tk, ROWS_MAX);
  TRY(check_heads(fn, sh->Hq, sh->Hkv, sh->D));
  // a tile of one head is 256 threads, a dispatch 2^32 - 1 of them at most
  if (std::max((int64_t)attn_tiles(sh->Tq) * sh->Hq, (int64_t)attn_tiles(sh->Tk) * sh->Hkv) >= 1 << 24)
    return fail(POETX_ERR_ARG, "%s: Tq=%d rows of Hq=%d heads, Tk=%d of Hkv=%d: 2^31 or more", fn, sh->Tq,
                sh->Hq, sh->Tk, sh->Hkv);
  TRY(check_act(fn, sh->act));
  TRY(check_scores(fn, sh->scale, sh->cap));
  const int64_t wq = (int64_t)sh->Hq * sh->D, wk = (int64_t)sh->Hkv * sh->D;
  TRY(check_ld(fn, "ldq", sh->ldq, wq));
  TRY(check_ld(fn, "ldk", sh->ldk, wk));
  TRY(check_ld(fn, "ldv", sh->ldv, wk));
  TRY(check_ld(fn, "ldo", sh->ldo, wq));
  if (back) {
    TRY(check_ld(fn, "lddo", sh->lddo, wq));
    TRY(check_ld(fn, "lddq", sh->lddq, wq));
    TRY(check_ld(fn, "lddk", sh->lddk, wk));
    TRY(check_ld(fn, "lddv", sh->lddv, wk));
  }
  return POETX_OK;
}

// From this many tiles on a side, tiles are sorted by cost: fewer run side by
// side in any order, and the sort is a launch of its own.
constexpr int SORT_TILES = 16;

bool sorts(const poetx_attn_shape* sh) { return attn_tiles(std::max(sh->Tq, sh->Tk)) >= SORT_TILES; }

// Five int32 arrays and the tile tables, each rounded up to 256 bytes.
struct PlanSizes { size_t q, k, tq, tk, total; };
PlanSizes plan_sizes(const poetx_attn_shape* sh) {
  PlanSizes z;
  z.q = align_up((size_t)sh->Tq * 4);
  z.k = align_up((size_t)sh->Tk * 4);
  z.tq = align_up((size_t)attn_tiles(sh->Tq) * 16);
  z.tk = align_up((size_t)attn_tiles(sh->Tk) * 16);
  z.total = 3 * z.q + 2 * z.k + (sorts(sh) ? 2 : 1) * (z.tq + z.tk) + 256;
  return z;
}
size_t plan_bytes_of(const poetx_attn_shape* sh) { return plan_sizes(sh).total; }

AttnPlan plan_at(const poetx_attn_shape* sh, const void* plan) {
  char* p = (char*)const_cast<void*>(plan);
  const PlanSizes z = plan_sizes(sh);
  AttnPlan pl;
  pl.row_lo = (int*)p;
  pl.row_hi = (int*)(p + z.q);
  pl.row_pos = (int*)(p + 2 * z.q);
  pl.key_lo = (int*)(p + 3 * z.q);
  pl.key_hi = (int*)(p + 3 * z.q + z.k);
  char* t = p + 3 * z.q + 2 * z.k;
  pl.qraw = pl.qtab = (int4*)t;
  pl.kraw = pl.ktab = (int4*)(t + z.tq);
  if (sorts(sh)) {
    pl.qtab = (int4*)(t + z.tq + z.tk);
    pl.ktab = (int4*)(t + 2 * z.tq + z.tk);
  }
  return pl;
}

AttnArgs args_of(const poetx_attn_shape* sh, const void* q, const void* k, const void* v,
                 const float* slopes, const void* plan) {
  AttnArgs a = {};
  a.Tq = sh->Tq, a.Tk = sh->Tk, a.Hq = sh->Hq, a.Hkv = sh->Hkv, a.D = sh->D;
  a.group = sh->Hq / sh->Hkv;
  a.scale = sh->scale > 0.0f ? sh->scale : 1.0f / sqrtf((float)sh->D);
  a.cap = cap_of(sh->cap);
  a.slopes = slopes;
  a.ldq = sh->ldq, a.ldk = sh->ldk, a.ldv = sh->ldv, a.ldo = sh->ldo;
  a.lddo = sh->lddo, a.lddq = sh->lddq, a.lddk = sh->lddk, a.lddv = sh->lddv;
  a.q = q, a.k = k, a.v = v;
  a.pl = plan_at(sh, plan);
  a.ndoc = sh->ndoc;
  return a;
}

// backward: delta and lse2, [Hq][Tq] float32 each; then partial sums (its
// workspace is large enough for the forward pass too)
size_t row_bytes(const poetx_attn_shape* sh) { return align_up((size_t)sh->Hq * sh->Tq * 4); }
size_t attn_ws(const poetx_attn_shape* sh, int which) {
  const AttnArgs a = args_of(sh, nullptr, nullptr, nullptr, nullptr, nullptr);
  const bool h = sh->act == POETX_BF16;
  const size_t fwd = align_up(h ? attn_fwd_part_bytes<bf16>(a) : attn_fwd_part_bytes<float>(a));
  if (which == 0) return fwd;
  const size_t bwd = 2 * row_bytes(sh) + align_up(h ? attn_bwd_part_bytes<bf16>(a) : attn_bwd_part_bytes<float>(a));
  return std::max(fwd, bwd);
}

int32_t check_decode(const char* fn, const poetx_decode_shape* sh) {
  if (!sh) return fail(POETX_ERR_ARG, "%s: null shape", fn);
  if (sh->B < 0 || sh->B > B_MAX || sh->rows < 0)
    return fail(POETX_ERR_ARG, "%s: B=%d (0..%d) rows=%d (>= 0)", fn, sh->B, B_MAX, sh->rows);
  if (sh->rows > ROWS_MAX) return fail(POETX_ERR_ARG, "%s: rows=%d above %d", fn, sh->rows, ROWS_MAX);
  TRY(check_heads(fn, sh->Hq, sh->Hkv, sh->D));
  TRY(check_act(fn, sh->act));
  TRY(check_scores(fn, sh->scale, sh->cap));
  const int64_t wq = (int64_t)sh->Hq * sh->D, wk = (int64_t)sh->Hkv * sh->D;
  TRY(check_ld(fn, "ldq", sh->ldq, wq));
  TRY(check_ld(fn, "ldo", sh->ldo, wq));
  TRY(check_ld(fn, "ldk", sh->ldk, wk));
  TRY(check_ld(fn, "ldv", sh->ldv, wk));
  if (sh->bsk < 0 || sh->bsv < 0 || sh->bsk % 8 || sh->bsv % 8)
    return fail(POETX_ERR_ARG, "%s: bsk=%lld bsv=%lld must be multiples of 8, >= 0", fn,
                (long long)sh->bsk, (long long)sh->bsv);
  return POETX_OK;
}

DecodeArgs decode_args(const poetx_decode_shape* sh) {
  DecodeArgs a = {};
  a.B = sh->B, a.Hq = sh->Hq, a.Hkv = sh->Hkv, a.group = sh->Hq / sh->Hkv, a.D = sh->D, a.rows = sh->rows;
  a.scale = sh->scale > 0.0f ? sh->scale : 1.0f / sqrtf((float)sh->D);
  a.cap = cap_of(sh->cap);
  a.ldq = sh->ldq, a.ldo = sh->ldo, a.ldk = sh->ldk, a.ldv = sh->ldv, a.bsk = sh->bsk, a.bsv = sh->bsv;
  return a;
}

size_t decode_ws(const poetx_decode_shape* sh) {
  return sh->B ? align_up(attn_decode_ws_bytes(decode_args(sh))) : 256;
}

int32_t check_dropout(const char* fn, int64_t n, int32_t act, double p, uint64_t offset,
                      const uint64_t* offset_dev) {
  if (n < 0) return fail(POETX_ERR_ARG, "%s: n=%lld < 0", fn, (long long)n);
  if (n >= (int64_t)1 << 40) return fail(POETX_ERR_ARG, "%s: n=%lld above 2^40", fn, (long long)n);
  TRY(check_act(fn, act));
  if (!(p >= 0.0 && p <= 1.0)) return fail(POETX_ERR_ARG, "%s: p=%g outside [0, 1]", fn, p);
  if (offset % 8) return fail(POETX_ERR_ARG, "%s: offset %llu is not a multiple of 8", fn, (unsigned long long)offset);
  if ((uintptr_t)offset_dev & 7) return fail(POETX_ERR_ARG, "%s: 'offset_dev' not 8-byte aligned", fn);
  return POETX_OK;
}

// p as a threshold for 16-bit draws
uint32_t cut_of(double p) { return (uint32_t)lrint(p * 65536.0); }

int32_t launched(hipError_t e, const char* fn) { return e == hipSuccess ? ok() : dev_fail(e, fn); }

}  // namespace

extern "C" {

int32_t poetx_rope(const poetx_rope_shape* sh, const void* q, const void* k, const int32_t* pos,
                   const float* table, void* qo, void* ko, poetx_stream_t stream) {
  const char* fn = "poetx_rope";
  if (!sh) return fail(POETX_ERR_ARG, "%s: null shape", fn);
  if (sh->T < 0 || sh->Hq < 1 || sh->Hk < 0 || sh->Hq > H_MAX || sh->Hk > H_MAX || sh->P < 1)
    return fail(POETX_ERR_ARG, "%s: T=%d Hq=%d Hk=%d P=%d", fn, sh->T, sh->Hq, sh->Hk, sh->P);
  if (sh->D < 8 || sh->D % 8 || sh->D > ROPE_D_MAX)
    return fail(POETX_ERR_ARG, "%s: D=%d must be a multiple of 8, 8..%d", fn, sh->D, ROPE_D_MAX);
  if (sh->rot < 2 || sh->rot % 2 || sh->rot > sh->D)
    return fail(POETX_ERR_ARG, "%s: rot=%d must be even, 2..D=%d", fn, sh->rot, sh->D);
  TRY(check_act(fn, sh->act));
  TRY(check_ld(fn, "ldq", sh->ldq, (int64_t)sh->Hq * sh->D));
  TRY(check_ld(fn, "ldqo", sh->ldqo, (int64_t)sh->Hq * sh->D));
  if (sh->Hk) {
    TRY(check_ld(fn, "ldk", sh->ldk, (int64_t)sh->Hk * sh->D));
    TRY(check_ld(fn, "ldko", sh->ldko, (int64_t)sh->Hk * sh->D));
  }
  if (sh->T == 0) return ok();
  NEED_PTR(q);
  NEED_PTR(qo);
  if (sh->Hk) {
    NEED_PTR(k);
    NEED_PTR(ko);
  }
  NEED_PTR(pos);
  NEED_PTR(table);
  if ((q == qo && sh->ldq != sh->ldqo) || (sh->Hk && k == ko && sh->ldk != sh->ldko))
    return fail(POETX_ERR_ARG, "%s: in place needs equal pitches", fn);
  const RopeArgs a = {sh->T, sh->Hq, sh->Hk, sh->D, sh->rot, sh->P, sh->interleaved,
                      sh->inverse ? -1.0f : 1.0f, sh->ldq, sh->ldk, sh->ldqo, sh->ldko, pos, table};
  const hipStream_t s = (hipStream_t)stream;
  return launched(sh->act == POETX_BF16
                      ? launch_rope<bf16>(a, (const bf16*)q, (const bf16*)k, (bf16*)qo, (bf16*)ko, s)
                      : launch_rope<float>(a, (const float*)q, (const float*)k, (float*)qo, (float*)ko, s),
                  fn);
}

int32_t poetx_dropout_fwd(int64_t n, int32_t act, const void* x, const void* residual, void* y,
                          double p, uint64_t seed, uint64_t offset, const uint64_t* offset_dev,
                          poetx_stream_t stream) {
  const char* fn = "poetx_dropout_fwd";
  TRY(check_dropout(fn, n, act, p, offset, offset_dev));
  if (n == 0) return ok();
  NEED_PTR(x);
  OPT_PTR(residual);
  NEED_PTR(y);
  const hipStream_t s = (hipStream_t)stream;
  return launched(act == POETX_BF16 ? launch_dropout<bf16>(n, (const bf16*)x, (const bf16*)residual, (bf16*)y,
                                                           cut_of(p), seed, offset, offset_dev, s)
                                    : launch_dropout<float>(n, (const float*)x, (const float*)residual, (float*)y,
                                                            cut_of(p), seed, offset, offset_dev, s),
                  fn);
}

int32_t poetx_dropout_bwd(int64_t n, int32_t act, const void* dy, void* dx, double p, uint64_t seed,
                          uint64_t offset, const uint64_t* offset_dev, poetx_stream_t stream) {
  const char* fn = "poetx_dropout_bwd";
  TRY(check_dropout(fn, n, act, p, offset, offset_dev));
  if (n == 0) return ok();
  NEED_PTR(dy);
  NEED_PTR(dx);
  const hipStream_t s = (hipStream_t)stream;
  return launched(act == POETX_BF16 ? launch_dropout<bf16>(n, (const bf16*)dy, nullptr, (bf16*)dx, cut_of(p),
                                                           seed, offset, offset_dev, s)
                                    : launch_dropout<float>(n, (const float*)dy, nullptr, (float*)dx, cut_of(p),
                                                            seed, offset, offset_dev, s),
                  fn);
}

size_t poetx_attn_plan_bytes(const poetx_attn_shape* sh) {
  return check_attn("poetx_attn_plan_bytes", sh, false) == POETX_OK ? plan_bytes_of(sh) : 0;
}

size_t poetx_attn_workspace_bytes(const poetx_attn_shape* sh, int32_t which) {
  if (which != 0 && which != 1) return 0;
  return check_attn("poetx_attn_workspace_bytes", sh, false) == POETX_OK ? attn_ws(sh, which) : 0;
}

int32_t poetx_attn_plan(const poetx_attn_shape* sh, const int32_t* cu_q, const int32_t* cu_k,
                        const int32_t* prefix, void* plan, size_t plan_bytes,
                        poetx_stream_t stream) {
  const char* fn = "poetx_attn_plan";
  TRY(check_attn(fn, sh, false));
  NEED_PTR(cu_q);
  NEED_PTR(cu_k);
  OPT_PTR(prefix);
  NEED_PTR(plan);
  const size_t need = plan_bytes_of(sh);
  if (plan_bytes < need) return fail(POETX_ERR_WORKSPACE, "%s: plan %zu < %zu bytes", fn, plan_bytes, need);
  if ((int64_t)sh->Tq + sh->Tk == 0) return ok();
  return launched(launch_attn_plan(sh->Tq, sh->Tk, sh->ndoc, sh->causal, cu_q, cu_k, prefix,
                                   plan_at(sh, plan), (hipStream_t)stream), fn);
}

int32_t poetx_attn_fwd(const poetx_attn_shape* sh, const void* q, const void* k, const void* v,
                       const float* slopes, const void* plan, void* o, float* lse, void* ws,
                       size_t ws_bytes, poetx_stream_t stream) {
  const char* fn = "poetx_attn_fwd";
  TRY(check_attn(fn, sh, false));
  if (sh->Tq == 0) return ok();
  NEED_PTR(q);
  if (sh->Tk) {
    NEED_PTR(k);
    NEED_PTR(v);
  }
  OPT_PTR(slopes);
  NEED_PTR(plan);
  NEED_PTR(o);
  NEED_PTR(lse);
  OPT_PTR(ws);
  const size_t need = attn_ws(sh, 0);
  if (ws_bytes < need || (need && !ws)) return fail(POETX_ERR_WORKSPACE, "%s: workspace %zu < %zu bytes", fn, ws_bytes, need);
  AttnArgs a = args_of(sh, q, k, v, slopes, plan);
  a.o = o;
  a.lse = lse;
  a.part = (float*)ws;
  const hipStream_t s = (hipStream_t)stream;
  return launched(sh->act == POETX_BF16 ? launch_attn_fwd<bf16>(a, s) : launch_attn_fwd<float>(a, s), fn);
}

int32_t poetx_attn_bwd(const poetx_attn_shape* sh, const void* dout, const void* q, const void* k,
                       const void* v, const void* o, const float* lse, const float* slopes,
                       const void* plan, void* dq, void* dk, void* dv, void* ws, size_t ws_bytes,
                       poetx_stream_t stream) {
  const char* fn = "poetx_attn_bwd";
  TRY(check_attn(fn, sh, true));
  if ((int64_t)sh->Tq + sh->Tk == 0) return ok();
  if (sh->Tq) {
    NEED_PTR(dout);
    NEED_PTR(q);
    NEED_PTR(o);
    NEED_PTR(lse);
    NEED_PTR(dq);
    NEED_PTR(ws);
  }
  if (sh->Tk) {
    NEED_PTR(k);
    NEED_PTR(v);
    NEED_PTR(dk);
    NEED_PTR(dv);
  }
  OPT_PTR(slopes);
  NEED_PTR(plan);
  const size_t need = attn_ws(sh, 1);
  if (ws_bytes < need) return fail(POETX_ERR_WORKSPACE, "%s: workspace %zu < %zu bytes", fn, ws_bytes, need);
  AttnArgs a = args_of(sh, q, k, v, slopes, plan);
  a.o = const_cast<void*>(o);
  a.lse = const_cast<float*>(lse);
  a.dout = dout;
  a.dq = dq, a.dk = dk, a.dv = dv;
  a.delta = (float*)ws;
  a.lse2 = (float*)((char*)ws + row_bytes(sh));
  a.part = (float*)((char*)ws + 2 * row_bytes(sh));
  const hipStream_t s = (hipStream_t)stream;
  return launched(sh->act == POETX_BF16 ? launch_attn_bwd<bf16>(a, s) : launch_attn_bwd<float>(a, s), fn);
}

size_t poetx_attn_decode_workspace_bytes(const poetx_decode_shape* sh) {
  return check_decode("poetx_attn_decode_workspace_bytes", sh) == POETX_OK ? decode_ws(sh) : 0;
}

int32_t poetx_attn_decode(const poetx_decode_shape* sh, const void* q, const void* k, const void* v,
                          const int32_t* start, const int32_t* len, const float* slopes, void* o,
                          void* ws, size_t ws_bytes, poetx_stream_t stream) {
  const char* fn = "poetx_attn_decode";
  TRY(check_decode(fn, sh));
  if (sh->B == 0) return ok();
  NEED_PTR(q);
  if (sh->rows) {
    NEED_PTR(k);
    NEED_PTR(v);
  }
  OPT_PTR(start);
  NEED_PTR(len);
  OPT_PTR(slopes);
  NEED_PTR(o);
  NEED_PTR(ws);
  const size_t need = decode_ws(sh);
  if (ws_bytes < need) return fail(POETX_ERR_WORKSPACE, "%s: workspace %zu < %zu bytes", fn, ws_bytes, need);
  DecodeArgs a = decode_args(sh);
  a.q = q, a.k = k, a.v = v, a.o = o;
  a.slopes = slopes;
  a.start = start, a.len = len;
  const hipStream_t s = (hipStream_t)stream;
  return launched(sh->act == POETX_BF16 ? launch_attn_decode<bf16>(a, (float*)ws, s)
                                               : launch_attn_decode<float>(a, (float*)ws, s), fn);
}

}  // extern "C"

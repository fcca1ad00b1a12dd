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
constexpr int SINKS_MAX = 128;   // first tokens that stay visible past a window
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

// A window that hides something, and its sinks; {0, 0}: none.
const poetx_window NO_WINDOW = {0, 0};
int32_t check_window(const char* fn, const poetx_window* w) {
  if (!w) return fail(POETX_ERR_ARG, "%s: null window", fn);
  if (w->window < 0) return fail(POETX_ERR_ARG, "%s: window=%d must be >= 0", fn, w->window);
  if (w->sinks < 0 || w->sinks > SINKS_MAX) return fail(POETX_ERR_ARG, "%s: sinks=%d outside 0..%d", fn, w->sinks, SINKS_MAX);
  return POETX_OK;
}
poetx_window window_of(const poetx_window* w) { return w->window ? *w : NO_WINDOW; }

int32_t check_attn_window(const char* fn, const poetx_attn_shape* sh, const poetx_window* w, bool back) {
  TRY(check_attn(fn, sh, back));
  TRY(check_window(fn, w));
  // a workgroup of 1024 threads a sink, a dispatch 2^32 - 1 of them at most
  if ((int64_t)sh->ndoc * window_of(w).sinks * sh->Hkv >= 1 << 22)
    return fail(POETX_ERR_ARG, "%s: ndoc=%d documents of sinks=%d and Hkv=%d heads: 2^22 or more", fn, sh->ndoc, w->sinks, sh->Hkv);
  return POETX_OK;
}

// Five int32 arrays and the tile tables, with sinks four arrays more, each
// rounded up to 256 bytes.
struct PlanSizes { size_t q, k, tq, tk, sink, far, first, doc, total; };
PlanSizes plan_sizes(const poetx_attn_shape* sh, const poetx_window& w) {
  PlanSizes z;
  z.q = align_up((size_t)sh->Tq * 4);
  z.k = align_up((size_t)sh->Tk * 4);
  z.tq = align_up((size_t)attn_tiles(sh->Tq) * 16);
  z.tk = align_up((size_t)attn_tiles(sh->Tk) * 16);
  z.sink = w.sinks ? align_up((size_t)sh->Tq * 8) : 0;
  z.far = w.sinks ? align_up((size_t)attn_tiles(sh->Tq) * 8) : 0;
  z.first = w.sinks ? align_up((size_t)attn_tiles(sh->Tq) * 4) : 0;
  z.doc = w.sinks ? align_up((size_t)sh->ndoc * 16) : 0;
  z.total = 3 * z.q + 2 * z.k + (sorts(sh) ? 2 : 1) * (z.tq + z.tk) + z.sink + z.far + z.first + z.doc + 256;
  return z;
}

AttnPlan plan_at(const poetx_attn_shape* sh, const poetx_window& w, const void* plan) {
  char* p = (char*)const_cast<void*>(plan);
  const PlanSizes z = plan_sizes(sh, w);
  AttnPlan pl = {};
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
  if (w.sinks) {
    char* u = p + z.total - 256 - z.sink - z.far - z.first - z.doc;
    pl.row_sink = (int2*)u;
    pl.qfar = (int2*)(u + z.sink);
    pl.tile_doc = (int*)(u + z.sink + z.far);
    pl.doc = (int4*)(u + z.sink + z.far + z.first);
  }
  return pl;
}

AttnArgs args_of(const poetx_attn_shape* sh, const poetx_window& w, const void* q, const void* k,
                 const void* v, const float* slopes, const void* plan) {
  AttnArgs a = {};
  a.Tq = sh->Tq, a.Tk = sh->Tk, a.Hq = sh->Hq, a.Hkv = sh->Hkv, a.D = sh->D;
  a.group = sh->Hq / sh->Hkv;
  a.scale = sh->scale > 0.0f ? sh->scale : 1.0f / sqrtf((float)sh->D);
  a.cap = cap_of(sh->cap);
  a.slopes = slopes;
  a.ldq = sh->ldq, a.ldk = sh->ldk, a.ldv = sh->ldv, a.ldo = sh->ldo;
  a.lddo = sh->lddo, a.lddq = sh->lddq, a.lddk = sh->lddk, a.lddv = sh->lddv;
  a.q = q, a.k = k, a.v = v;
  a.pl = plan_at(sh, w, plan);
  a.ndoc = sh->ndoc, a.causal = sh->causal;
  a.window = w.window, a.sinks = w.sinks;
  return a;
}

// backward: delta and lse2, [Hq][Tq] float32 each; then partial sums, those of
// the sinks last (its workspace is large enough for the forward pass too)
size_t row_bytes(const poetx_attn_shape* sh) { return align_up((size_t)sh->Hq * sh->Tq * 4); }
size_t sink_at(const poetx_attn_shape* sh, const AttnArgs& a) {
  return 2 * row_bytes(sh) + align_up(sh->act == POETX_BF16 ? attn_bwd_part_bytes<bf16>(a) : attn_bwd_part_bytes<float>(a));
}
size_t attn_ws(const poetx_attn_shape* sh, const poetx_window& w, int which) {
  const AttnArgs a = args_of(sh, w, nullptr, nullptr, nullptr, nullptr, nullptr);
  const size_t fwd = align_up(sh->act == POETX_BF16 ? attn_fwd_part_bytes<bf16>(a) : attn_fwd_part_bytes<float>(a));
  if (which == 0) return fwd;
  return std::max(fwd, sink_at(sh, a) + align_up(attn_sink_part_bytes(a)));
}

int32_t check_decode(const char* fn, const poetx_decode_shape* sh) {
  if (!sh) return fail(POETX_ERR_ARG, "%s: null shape", fn);
  if (sh->B < 0 || sh->B > B_MAX || sh->rows < 0)
    return fail(POETX_ERR_ARG, "%s: B=%d (0..%d) rows=%d (>= 0)", fn, sh->B, B_MAX, sh->rows);
  if (sh->rows > ROWS_MAX) return fail(POETX_ERR_ARG, "%s: rows=%d above %d", fn, sh->rows, ROWS_MAX);
  TRY(check_heads(fn, sh->Hq, sh->Hkv, sh->D));
  // a workgroup of 256 threads for 32 heads of a key head and sequence, a dispatch
  // 2^32 - 1 of them at most (pieces, and their join, are of far fewer workgroups)
  if ((int64_t)sh->B * sh->Hkv * ((sh->Hq / sh->Hkv + 31) / 32) >= 1 << 24)
    return fail(POETX_ERR_ARG, "%s: B=%d sequences of Hq=%d heads on Hkv=%d: 2^24 workgroups or more", fn, sh->B, sh->Hq, sh->Hkv);
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

int32_t check_qk_norm(const char* fn, const poetx_qk_norm_shape* sh, bool back) {
  if (!sh) return fail(POETX_ERR_ARG, "%s: null shape", fn);
  if (sh->T < 0 || sh->Hq < 1 || sh->Hk < 0 || sh->Hq > H_MAX || sh->Hk > H_MAX)
    return fail(POETX_ERR_ARG, "%s: T=%d Hq=%d Hk=%d", fn, sh->T, sh->Hq, sh->Hk);
  if (sh->D < 8 || sh->D % 8 || sh->D > ROPE_D_MAX)
    return fail(POETX_ERR_ARG, "%s: D=%d must be a multiple of 8, 8..%d", fn, sh->D, ROPE_D_MAX);
  if (sh->rot < 0 || sh->rot % 2 || sh->rot > sh->D)
    return fail(POETX_ERR_ARG, "%s: rot=%d must be even, 0..D=%d", fn, sh->rot, sh->D);
  if (sh->rot && sh->P < 1) return fail(POETX_ERR_ARG, "%s: P=%d positions", fn, sh->P);
  TRY(check_act(fn, sh->act));
  if (!(sh->eps >= 0.0f) || !isfinite(sh->eps)) return fail(POETX_ERR_ARG, "%s: eps=%g must be finite and >= 0", fn, sh->eps);
  const int64_t wq = (int64_t)sh->Hq * sh->D, wk = (int64_t)sh->Hk * sh->D;
  TRY(check_ld(fn, "ldq", sh->ldq, wq));
  TRY(check_ld(fn, "ldqo", sh->ldqo, wq));
  if (back) TRY(check_ld(fn, "lddq", sh->lddq, wq));
  if (sh->Hk) {
    TRY(check_ld(fn, "ldk", sh->ldk, wk));
    TRY(check_ld(fn, "ldko", sh->ldko, wk));
    if (back) TRY(check_ld(fn, "lddk", sh->lddk, wk));
  }
  return POETX_OK;
}

QkNormArgs qk_norm_args(const poetx_qk_norm_shape* sh) {
  QkNormArgs a = {};
  a.T = sh->T, a.Hq = sh->Hq, a.Hk = sh->Hk, a.D = sh->D, a.rot = sh->rot, a.P = sh->P;
  a.interleaved = sh->interleaved && sh->rot;
  a.eps = sh->eps, a.inv_d = 1.0f / (float)sh->D;
  a.ldq = sh->ldq, a.ldk = sh->ldk, a.ldqo = sh->ldqo, a.ldko = sh->ldko, a.lddq = sh->lddq, a.lddk = sh->lddk;
  return a;
}

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

int32_t poetx_qk_norm_rope_fwd(const poetx_qk_norm_shape* sh, const void* q, const void* k, const float* wq,
                               const float* wk, const int32_t* pos, const float* table, void* qo, void* ko,
                               poetx_stream_t stream) {
  const char* fn = "poetx_qk_norm_rope_fwd";
  TRY(check_qk_norm(fn, sh, false));
  if (sh->T == 0) return ok();
  NEED_PTR(q);
  NEED_PTR(qo);
  OPT_PTR(wq);
  if (sh->Hk) {
    NEED_PTR(k);
    NEED_PTR(ko);
    OPT_PTR(wk);
  }
  if (sh->rot) {
    NEED_PTR(pos);
    NEED_PTR(table);
  }
  if ((q == qo && sh->ldq != sh->ldqo) || (sh->Hk && k == ko && sh->ldk != sh->ldko))
    return fail(POETX_ERR_ARG, "%s: in place needs equal pitches", fn);
  QkNormArgs a = qk_norm_args(sh);
  a.q = q, a.k = k, a.wq = wq, a.wk = wk, a.pos = sh->rot ? pos : nullptr, a.table = table, a.qo = qo, a.ko = ko;
  const hipStream_t s = (hipStream_t)stream;
  return launched(sh->act == POETX_BF16 ? launch_qk_norm_fwd<bf16>(a, s) : launch_qk_norm_fwd<float>(a, s), fn);
}

size_t poetx_qk_norm_rope_workspace_bytes(const poetx_qk_norm_shape* sh) {
  return check_qk_norm("poetx_qk_norm_rope_workspace_bytes", sh, false) == POETX_OK
             ? align_up(qk_norm_ws_bytes(qk_norm_args(sh))) : 0;
}

int32_t poetx_qk_norm_rope_bwd(const poetx_qk_norm_shape* sh, const void* dqo, const void* dko, const void* q,
                               const void* k, const float* wq, const float* wk, const int32_t* pos,
                               const float* table, void* dq, void* dk, float* dwq, float* dwk, void* ws,
                               size_t ws_bytes, poetx_stream_t stream) {
  const char* fn = "poetx_qk_norm_rope_bwd";
  TRY(check_qk_norm(fn, sh, true));
  if (sh->T) {
    NEED_PTR(dqo);
    NEED_PTR(q);
    NEED_PTR(dq);
    if (sh->Hk) {
      NEED_PTR(dko);
      NEED_PTR(k);
      NEED_PTR(dk);
    }
    if (sh->rot) {
      NEED_PTR(pos);
      NEED_PTR(table);
    }
  }
  OPT_PTR(wq);
  OPT_PTR(dwq);
  if (sh->Hk) {
    OPT_PTR(wk);
    OPT_PTR(dwk);
  }
  if (!sh->T && !dwq && !(sh->Hk && dwk)) return ok();
  NEED_PTR(ws);
  if (sh->T && ((dqo == dq && sh->ldqo != sh->lddq) || (sh->Hk && dko == dk && sh->ldko != sh->lddk)))
    return fail(POETX_ERR_ARG, "%s: in place needs equal pitches", fn);
  QkNormArgs a = qk_norm_args(sh);
  const size_t need = align_up(qk_norm_ws_bytes(a));
  if (ws_bytes < need) return fail(POETX_ERR_WORKSPACE, "%s: workspace %zu < %zu bytes", fn, ws_bytes, need);
  a.q = q, a.k = k, a.wq = wq, a.wk = wk, a.pos = sh->rot ? pos : nullptr, a.table = table;
  a.gq = dqo, a.gk = dko, a.dq = dq, a.dk = dk, a.dwq = dwq, a.dwk = sh->Hk ? dwk : nullptr;
  const hipStream_t s = (hipStream_t)stream;
  return launched(sh->act == POETX_BF16 ? launch_qk_norm_bwd<bf16>(a, (float*)ws, s)
                                        : launch_qk_norm_bwd<float>(a, (float*)ws, s), fn);
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

}  // extern "C"

namespace {

// The entry points with and without a window: the same but for the window.
size_t plan_bytes_any(const char* fn, const poetx_attn_shape* sh, const poetx_window* w) {
  return check_attn_window(fn, sh, w, false) == POETX_OK ? plan_sizes(sh, window_of(w)).total : 0;
}

size_t workspace_any(const char* fn, const poetx_attn_shape* sh, const poetx_window* w, int32_t which) {
  if (which != 0 && which != 1) return 0;
  return check_attn_window(fn, sh, w, false) == POETX_OK ? attn_ws(sh, window_of(w), which) : 0;
}

int32_t plan_any(const char* fn, const poetx_attn_shape* sh, const poetx_window* win, const int32_t* cu_q,
                 const int32_t* cu_k, const int32_t* prefix, void* plan, size_t plan_bytes, poetx_stream_t stream) {
  TRY(check_attn_window(fn, sh, win, false));
  NEED_PTR(cu_q);
  NEED_PTR(cu_k);
  OPT_PTR(prefix);
  NEED_PTR(plan);
  const poetx_window w = window_of(win);
  const size_t need = plan_sizes(sh, w).total;
  if (plan_bytes < need) return fail(POETX_ERR_WORKSPACE, "%s: plan %zu < %zu bytes", fn, plan_bytes, need);
  if ((int64_t)sh->Tq + sh->Tk == 0) return ok();
  const AttnPlan pl = plan_at(sh, w, plan);
  const hipStream_t s = (hipStream_t)stream;
  return launched(w.window ? launch_attn_window_plan(sh->Tq, sh->Tk, sh->ndoc, sh->causal, w.window, w.sinks, cu_q, cu_k, pl, s)
                           : launch_attn_plan(sh->Tq, sh->Tk, sh->ndoc, sh->causal, cu_q, cu_k, prefix, pl, s), fn);
}

int32_t fwd_any(const char* fn, const poetx_attn_shape* sh, const poetx_window* win, const void* q, const void* k,
                const void* v, const float* slopes, const void* plan, void* o, float* lse, void* ws,
                size_t ws_bytes, poetx_stream_t stream) {
  TRY(check_attn_window(fn, sh, win, false));
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
  const poetx_window w = window_of(win);
  const size_t need = attn_ws(sh, w, 0);
  if (ws_bytes < need || (need && !ws)) return fail(POETX_ERR_WORKSPACE, "%s: workspace %zu < %zu bytes", fn, ws_bytes, need);
  AttnArgs a = args_of(sh, w, q, k, v, slopes, plan);
  a.o = o;
  a.lse = lse;
  a.part = (float*)ws;
  const hipStream_t s = (hipStream_t)stream;
  return launched(sh->act == POETX_BF16 ? launch_attn_fwd<bf16>(a, s) : launch_attn_fwd<float>(a, s), fn);
}

int32_t bwd_any(const char* fn, const poetx_attn_shape* sh, const poetx_window* win, const void* dout, const void* q,
                const void* k, const void* v, const void* o, const float* lse, const float* slopes,
                const void* plan, void* dq, void* dk, void* dv, void* ws, size_t ws_bytes, poetx_stream_t stream) {
  TRY(check_attn_window(fn, sh, win, true));
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
  const poetx_window w = window_of(win);
  const size_t need = attn_ws(sh, w, 1);
  if (ws_bytes < need) return fail(POETX_ERR_WORKSPACE, "%s: workspace %zu < %zu bytes", fn, ws_bytes, need);
  AttnArgs a = args_of(sh, w, q, k, v, slopes, plan);
  a.o = const_cast<void*>(o);
  a.lse = const_cast<float*>(lse);
  a.dout = dout;
  a.dq = dq, a.dk = dk, a.dv = dv;
  a.delta = (float*)ws;
  a.lse2 = (float*)((char*)ws + row_bytes(sh));
  a.part = (float*)((char*)ws + 2 * row_bytes(sh));
  a.sink_part = (float*)((char*)ws + sink_at(sh, a));
  const hipStream_t s = (hipStream_t)stream;
  return launched(sh->act == POETX_BF16 ? launch_attn_bwd<bf16>(a, s) : launch_attn_bwd<float>(a, s), fn);
}

}  // namespace

extern "C" {

size_t poetx_attn_plan_bytes(const poetx_attn_shape* sh) { return plan_bytes_any("poetx_attn_plan_bytes", sh, &NO_WINDOW); }
size_t poetx_attn_window_plan_bytes(const poetx_attn_shape* sh, const poetx_window* win) {
  return plan_bytes_any("poetx_attn_window_plan_bytes", sh, win);
}

size_t poetx_attn_workspace_bytes(const poetx_attn_shape* sh, int32_t which) {
  return workspace_any("poetx_attn_workspace_bytes", sh, &NO_WINDOW, which);
}
size_t poetx_attn_window_workspace_bytes(const poetx_attn_shape* sh, const poetx_window* win, int32_t which) {
  return workspace_any("poetx_attn_window_workspace_bytes", sh, win, which);
}

int32_t poetx_attn_plan(const poetx_attn_shape* sh, const int32_t* cu_q, const int32_t* cu_k,
                        const int32_t* prefix, void* plan, size_t plan_bytes,
                        poetx_stream_t stream) {
  return plan_any("poetx_attn_plan", sh, &NO_WINDOW, cu_q, cu_k, prefix, plan, plan_bytes, stream);
}
int32_t poetx_attn_window_plan(const poetx_attn_shape* sh, const poetx_window* win, const int32_t* cu_q,
                               const int32_t* cu_k, void* plan, size_t plan_bytes, poetx_stream_t stream) {
  return plan_any("poetx_attn_window_plan", sh, win, cu_q, cu_k, nullptr, plan, plan_bytes, stream);
}

int32_t poetx_attn_fwd(const poetx_attn_shape* sh, const void* q, const void* k, const void* v,
                       const float* slopes, const void* plan, void* o, float* lse, void* ws,
                       size_t ws_bytes, poetx_stream_t stream) {
  return fwd_any("poetx_attn_fwd", sh, &NO_WINDOW, q, k, v, slopes, plan, o, lse, ws, ws_bytes, stream);
}
int32_t poetx_attn_window_fwd(const poetx_attn_shape* sh, const poetx_window* win, const void* q, const void* k,
                              const void* v, const float* slopes, const void* plan, void* o, float* lse,
                              void* ws, size_t ws_bytes, poetx_stream_t stream) {
  return fwd_any("poetx_attn_window_fwd", sh, win, q, k, v, slopes, plan, o, lse, ws, ws_bytes, stream);
}

int32_t poetx_attn_bwd(const poetx_attn_shape* sh, const void* dout, const void* q, const void* k,
                       const void* v, const void* o, const float* lse, const float* slopes,
                       const void* plan, void* dq, void* dk, void* dv, void* ws, size_t ws_bytes,
                       poetx_stream_t stream) {
  return bwd_any("poetx_attn_bwd", sh, &NO_WINDOW, dout, q, k, v, o, lse, slopes, plan, dq, dk, dv, ws, ws_bytes, stream);
}
int32_t poetx_attn_window_bwd(const poetx_attn_shape* sh, const poetx_window* win, const void* dout, const void* q,
                              const void* k, const void* v, const void* o, const float* lse, const float* slopes,
                              const void* plan, void* dq, void* dk, void* dv, void* ws, size_t ws_bytes,
                              poetx_stream_t stream) {
  return bwd_any("poetx_attn_window_bwd", sh, win, dout, q, k, v, o, lse, slopes, plan, dq, dk, dv, ws, ws_bytes, stream);
}

}  // extern "C"

namespace {

// the window of a decoding call; a ring holds one.  These calls take fewer
// sequences and heads than the one without.
int32_t check_decode_window(const char* fn, const poetx_decode_shape* sh, const poetx_window* win, int32_t ring) {
  TRY(check_decode(fn, sh));
  if ((int64_t)sh->B * sh->Hq >= 1 << 24) return fail(POETX_ERR_ARG, "%s: B=%d sequences of Hq=%d heads: 2^24 or more", fn, sh->B, sh->Hq);
  TRY(check_window(fn, win));
  if (ring && win->window < 1) return fail(POETX_ERR_ARG, "%s: a ring needs a window", fn);
  if (ring && (int64_t)win->window + win->sinks > sh->rows)
    return fail(POETX_ERR_ARG, "%s: window=%d and sinks=%d in a ring of rows=%d", fn, win->window, win->sinks, sh->rows);
  return POETX_OK;
}

DecodeArgs decode_window_args(const poetx_decode_shape* sh, const poetx_window* win, int32_t ring) {
  DecodeArgs a = decode_args(sh);
  const poetx_window w = window_of(win);
  a.window = w.window, a.sinks = w.sinks, a.ring = ring != 0;
  return a;
}

size_t decode_ws(const DecodeArgs& a) { return a.B ? align_up(attn_decode_ws_bytes(a)) : 256; }

int32_t decode_any(const char* fn, const poetx_decode_shape* sh, const poetx_window* win, int32_t ring, const void* q,
                   const void* k, const void* v, const int32_t* start, const int32_t* len, const float* slopes,
                   void* o, void* ws, size_t ws_bytes, poetx_stream_t stream) {
  TRY(win == &NO_WINDOW ? check_decode(fn, sh) : check_decode_window(fn, sh, win, ring));
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
  DecodeArgs a = decode_window_args(sh, win, ring);
  const size_t need = decode_ws(a);
  if (ws_bytes < need) return fail(POETX_ERR_WORKSPACE, "%s: workspace %zu < %zu bytes", fn, ws_bytes, need);
  a.q = q, a.k = k, a.v = v, a.o = o;
  a.slopes = slopes;
  a.start = start, a.len = len;
  const hipStream_t s = (hipStream_t)stream;
  return launched(sh->act == POETX_BF16 ? launch_attn_decode<bf16>(a, (float*)ws, s)
                                               : launch_attn_decode<float>(a, (float*)ws, s), fn);
}

}  // namespace

extern "C" {

size_t poetx_attn_decode_workspace_bytes(const poetx_decode_shape* sh) {
  return check_decode("poetx_attn_decode_workspace_bytes", sh) == POETX_OK ? decode_ws(decode_args(sh)) : 0;
}
size_t poetx_attn_window_decode_workspace_bytes(const poetx_decode_shape* sh, const poetx_window* win) {
  return check_decode_window("poetx_attn_window_decode_workspace_bytes", sh, win, 0) == POETX_OK
             ? decode_ws(decode_window_args(sh, win, 0)) : 0;
}

int32_t poetx_attn_decode(const poetx_decode_shape* sh, const void* q, const void* k, const void* v,
                          const int32_t* start, const int32_t* len, const float* slopes, void* o,
                          void* ws, size_t ws_bytes, poetx_stream_t stream) {
  return decode_any("poetx_attn_decode", sh, &NO_WINDOW, 0, q, k, v, start, len, slopes, o, ws, ws_bytes, stream);
}
int32_t poetx_attn_window_decode(const poetx_decode_shape* sh, const poetx_window* win, int32_t ring, const void* q,
                                 const void* k, const void* v, const int32_t* len, const float* slopes, void* o,
                                 void* ws, size_t ws_bytes, poetx_stream_t stream) {
  return decode_any("poetx_attn_window_decode", sh, win, ring, q, k, v, nullptr, len, slopes, o, ws, ws_bytes, stream);
}

}  // extern "C"

namespace {

int32_t check_kv4(const char* fn, const poetx_kv4_shape* sh) {
  if (!sh) return fail(POETX_ERR_ARG, "%s: null shape", fn);
  if (sh->T < 0 || sh->T > ROWS_MAX || sh->B < 0 || sh->B > B_MAX)
    return fail(POETX_ERR_ARG, "%s: T=%d (0..%d) B=%d (0..%d)", fn, sh->T, ROWS_MAX, sh->B, B_MAX);
  if (sh->rows < 0 || sh->rows > ROWS_MAX || sh->rows % 64)
    return fail(POETX_ERR_ARG, "%s: rows=%d must be a multiple of 64, 0..%d", fn, sh->rows, ROWS_MAX);
  TRY(check_heads(fn, sh->Hkv, sh->Hkv, sh->D));
  TRY(check_act(fn, sh->act));
  if (sh->sinks < 0 || sh->sinks > SINKS_MAX) return fail(POETX_ERR_ARG, "%s: sinks=%d outside 0..%d", fn, sh->sinks, SINKS_MAX);
  if (sh->ring && sh->rows <= sh->sinks) return fail(POETX_ERR_ARG, "%s: rows=%d of a ring with sinks=%d", fn, sh->rows, sh->sinks);
  // a workgroup of 256 threads for 16 tokens of a head and more: 2^32 - 1 threads at most
  if (((int64_t)sh->T + 15) / 16 * 16 * sh->Hkv >= (int64_t)1 << 27)
    return fail(POETX_ERR_ARG, "%s: T=%d tokens of Hkv=%d heads: 2^27 or more", fn, sh->T, sh->Hkv);
  TRY(check_ld(fn, "ldk", sh->ldk, (int64_t)sh->Hkv * sh->D));
  TRY(check_ld(fn, "ldv", sh->ldv, (int64_t)sh->Hkv * sh->D));
  return POETX_OK;
}

Kv4Args kv4_args(const poetx_kv4_shape* sh) {
  Kv4Args a = {};
  a.T = sh->T, a.B = sh->B, a.rows = sh->rows, a.Hkv = sh->Hkv, a.D = sh->D, a.sinks = sh->sinks, a.ring = sh->ring != 0;
  a.ldk = sh->ldk, a.ldv = sh->ldv;
  return a;
}

size_t kv4_ws(const DecodeArgs& a, int32_t act) {
  return align_up(act == POETX_BF16 ? attn_kv4_ws_bytes<bf16>(a) : attn_kv4_ws_bytes<float>(a));
}

int32_t check_kv4_decode(const char* fn, const poetx_decode_shape* sh, const poetx_window* win, int32_t ring) {
  TRY(check_decode_window(fn, sh, win, ring));
  if (sh->rows % 64) return fail(POETX_ERR_ARG, "%s: rows=%d must be a multiple of 64", fn, sh->rows);
  return POETX_OK;
}

}  // namespace

extern "C" {

int32_t poetx_kv4_write(const poetx_kv4_shape* sh, const void* k, const void* v, const int32_t* seq, const int32_t* pos,
                        void* kc, void* ks, void* vc, void* vs, poetx_stream_t stream) {
  const char* fn = "poetx_kv4_write";
  TRY(check_kv4(fn, sh));
  if (sh->T == 0 || sh->B == 0 || sh->rows == 0) return ok();
  NEED_PTR(k);
  NEED_PTR(v);
  OPT_PTR(seq);
  NEED_PTR(pos);
  NEED_PTR(kc);
  NEED_PTR(ks);
  NEED_PTR(vc);
  NEED_PTR(vs);
  Kv4Args a = kv4_args(sh);
  a.k = const_cast<void*>(k), a.v = const_cast<void*>(v), a.seq = seq, a.pos = pos;
  a.kc = (uint8_t*)kc, a.ks = (uint8_t*)ks, a.vc = (uint8_t*)vc, a.vs = (uint8_t*)vs;
  const hipStream_t s = (hipStream_t)stream;
  return launched(sh->act == POETX_BF16 ? launch_kv4_write<bf16>(a, s) : launch_kv4_write<float>(a, s), fn);
}

int32_t poetx_kv4_read(const poetx_kv4_shape* sh, const int32_t* seq, const int32_t* pos, const void* kc, const void* ks,
                       const void* vc, const void* vs, void* k, void* v, poetx_stream_t stream) {
  const char* fn = "poetx_kv4_read";
  TRY(check_kv4(fn, sh));
  if (sh->T == 0) return ok();
  NEED_PTR(k);
  NEED_PTR(v);
  OPT_PTR(seq);
  NEED_PTR(pos);
  if (sh->B && sh->rows) {
    NEED_PTR(kc);
    NEED_PTR(ks);
    NEED_PTR(vc);
    NEED_PTR(vs);
  }
  Kv4Args a = kv4_args(sh);
  if (a.rows == 0) a.B = 0;  // every position is outside
  a.k = k, a.v = v, a.seq = seq, a.pos = pos;
  a.kc = (uint8_t*)const_cast<void*>(kc), a.ks = (uint8_t*)const_cast<void*>(ks);
  a.vc = (uint8_t*)const_cast<void*>(vc), a.vs = (uint8_t*)const_cast<void*>(vs);
  const hipStream_t s = (hipStream_t)stream;
  return launched(sh->act == POETX_BF16 ? launch_kv4_read<bf16>(a, s) : launch_kv4_read<float>(a, s), fn);
}

size_t poetx_attn_kv4_decode_workspace_bytes(const poetx_decode_shape* sh, const poetx_window* win) {
  if (check_kv4_decode("poetx_attn_kv4_decode_workspace_bytes", sh, win, 0) != POETX_OK) return 0;
  const DecodeArgs a = decode_window_args(sh, win, 0);
  return a.B ? kv4_ws(a, sh->act) : 256;
}

int32_t poetx_attn_kv4_decode(const poetx_decode_shape* sh, const poetx_window* win, int32_t ring, const void* q,
                              const void* kc, const void* ks, const void* vc, const void* vs, const int32_t* start,
                              const int32_t* len, const float* slopes, void* o, void* ws, size_t ws_bytes,
                              poetx_stream_t stream) {
  const char* fn = "poetx_attn_kv4_decode";
  TRY(check_kv4_decode(fn, sh, win, ring));
  if (sh->B == 0) return ok();
  NEED_PTR(q);
  if (sh->rows) {
    NEED_PTR(kc);
    NEED_PTR(ks);
    NEED_PTR(vc);
    NEED_PTR(vs);
  }
  OPT_PTR(start);
  if (start && win->window) return fail(POETX_ERR_ARG, "%s: 'start' with a window", fn);
  NEED_PTR(len);
  OPT_PTR(slopes);
  NEED_PTR(o);
  NEED_PTR(ws);
  DecodeArgs a = decode_window_args(sh, win, ring);
  const size_t need = kv4_ws(a, sh->act);
  if (ws_bytes < need) return fail(POETX_ERR_WORKSPACE, "%s: workspace %zu < %zu bytes", fn, ws_bytes, need);
  a.q = q, a.k = kc, a.v = vc, a.ks = (const uint8_t*)ks, a.vs = (const uint8_t*)vs, a.o = o;
  a.slopes = slopes;
  a.start = start, a.len = len;
  const hipStream_t s = (hipStream_t)stream;
  return launched(sh->act == POETX_BF16 ? launch_attn_kv4<bf16>(a, (float*)ws, s) : launch_attn_kv4<float>(a, (float*)ws, s), fn);
}

}  // extern "C"

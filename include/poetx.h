/*
 * poetx.h -- C ABI of libpoetx.so: forward and backward pass of one POET-X
 * reparameterized linear layer on AMD Instinct MI355X (gfx950), and of the
 * operators of an attention block around such layers (rotary positions,
 * attention, dropout; last part of this file).
 *
 * The layer ("Reparameterized LLM Training via Orthogonal Equivalence
 * Transformation", Abstract) computes y = x W^T with W = R W0 P, where W0 is
 * a fixed random [m, n] weight and R, P are learnable orthogonal matrices.
 * Following "POET-X: Memory-efficient LLM Training by Scaling Orthogonal
 * Transformation" (technical summary, sections 2.1-2.4):
 *   - R = Pi_R^T BD(G_R) Pi_R and P = Pi_P^T BD(G_P) Pi_P: block-diagonal
 *     orthogonal matrices with b x b blocks, conjugated by random
 *     permutations; permutation matrix of an index map: Pi[i, pi[i]] = 1;
 *   - each block is G = (I+Q)(I + Q + ... + Q^k), the Cayley transform with
 *     its inverse replaced by the Neumann series cut after Q^k, where Q is
 *     skew-symmetric and only its strict upper triangle is stored (b(b-1)/2
 *     parameters per block, row by row over i < j);
 *   - the evaluation is input-centric: W is never formed; the input passes
 *     through the P-side blocks, the fixed weight, then the R-side blocks;
 *   - permutations are index maps; the two next to W0 are folded into it
 *     once per inner loop: W0f[i, j] = W0[pi_R[i], pi_P[j]].
 * With that fold the forward pass is
 *   U = x[:, pi_P];  V_j = U_j G_Pj^T;  Z = V W0f^T;  S_i = Z_i G_Ri^T;
 *   y[:, pi_R[c]] = S[:, c]
 * (U_j: columns [j b, (j+1) b) of U), and the backward pass is
 *   dS = dy[:, pi_R];  dZ_i = dS_i G_Ri;  dG_Ri = sum_t dS_i^T Z_i;
 *   dV = dZ W0f;  dU_j = dV_j G_Pj;  dG_Pj = sum_t dV_j^T U_j;
 *   dx[:, pi_P[c]] = dU[:, c];  dtheta = CNP^T(theta, dG).
 * W0 is fixed and gets no gradient.
 *
 * Conventions for every entry point:
 *   - All tensor pointers are DEVICE pointers, row-major and contiguous, base
 *     aligned to 16 bytes.  The caller owns every buffer; the library never
 *     allocates or frees device memory.
 *   - Activation storage type `act` (POETX_F32 or POETX_BF16) applies to x,
 *     y, dy, dx, W0, W0f, W0fT, G and GT.  theta, dtheta and dG are float32.
 *     bf16 values are IEEE binary32 truncated to 16 bits; the library rounds
 *     to nearest-even whenever it narrows.  Arithmetic accumulates in fp32.
 *   - Work is enqueued asynchronously on `stream` (NULL = the null stream);
 *     no call synchronizes the host.  Device faults surface at the caller's
 *     next synchronization.
 *   - Arguments are validated on the host before anything is enqueued; on
 *     any error nothing is written.  Permutations being valid is a
 *     precondition that is not checked on the device.
 *   - Entry points are thread-safe and keep no state between calls, except
 *     poetx_cnp_fwd_noalloc, whose scratch array is shared by its calls.
 *   - poetx_last_error() returns a message for the calling thread's most
 *     recent failure.
 */
#ifndef POETX_H
#define POETX_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define POETX_ABI_VERSION 2

typedef enum {
  POETX_OK = 0,
  POETX_ERR_ARG = 1,          /* null pointer, bad size, misalignment      */
  POETX_ERR_UNSUPPORTED = 2,  /* valid but not built (dtype / b pair)       */
  POETX_ERR_WORKSPACE = 3,    /* workspace smaller than required            */
  POETX_ERR_DEVICE = 4        /* HIP launch or device query failed          */
} poetx_status;

typedef enum { POETX_F32 = 0, POETX_BF16 = 1, POETX_I8 = 2 } poetx_dtype;
/* POETX_I8 is a weight storage type only (poetx_fold_perm, poetx_dequant). */

/* Shape of one layer.  m: outputs, n: inputs, b: block size (m % b == 0 and
 * n % b == 0), k: Neumann order (>= 0), T: tokens (>= 1), act: poetx_dtype.
 * Supported b: 8, 16, 32, 64, 128, 256, 512; float32 activations need
 * b <= 64.  1 <= k <= 8 or k = 0. */
typedef struct {
  int32_t m, n, b, k, T;
  int32_t act;
} poetx_shape;

typedef void* poetx_stream_t; /* a hipStream_t */

/* ABI version of the loaded library (POETX_ABI_VERSION). */
int32_t poetx_abi_version(void);

/* Static string naming a status code. */
const char* poetx_status_str(int32_t status);

/* Message describing the calling thread's most recent error ("" if none). */
const char* poetx_last_error(void);

/*
 * poetx_cnp_fwd -- Cayley-Neumann parameterization, forward
 * ("POET-X ...", technical summary 2.4, "Efficient CNP"; the Italian page,
 * "Sommario tecnico" 2, CNP bullet).
 *   theta [nblk][b(b-1)/2] float32: packed strict upper triangle of each
 *         skew-symmetric Q (Q[i][j] = theta[t], Q[j][i] = -theta[t],
 *         t = i*b - i*(i+1)/2 + (j-i-1) for i < j).
 *   G     [nblk][b][b] in g_dtype: G = (I+Q)(I + Q + ... + Q^k).
 *   GT    [nblk][b][b] in g_dtype or NULL: G transposed (= CNP of -Q).
 *   ws    workspace of poetx_cnp_workspace_bytes(nblk, b, k, 0, g_dtype) bytes
 *         (may be NULL when that is 0).
 * Errors: ERR_ARG (nblk < 1, k outside 0..8, b unsupported, null theta/G),
 * ERR_UNSUPPORTED (float32 with b > 64), ERR_WORKSPACE, ERR_DEVICE.
 */
int32_t poetx_cnp_fwd(int32_t nblk, int32_t b, int32_t k, const float* theta,
                      void* G, void* GT, int32_t g_dtype, void* ws,
                      size_t ws_bytes, poetx_stream_t stream);

/*
 * poetx_cnp_fwd_noalloc -- poetx_cnp_fwd for callers that cannot allocate
 * device memory (code under HIP graph capture, tight serving loops,
 * harnesses that forbid hipMalloc): the same arguments without the
 * workspace, the same kernels, bitwise the same G and GT.  The unpacked Q
 * that poetx_cnp_fwd keeps in its workspace goes instead to a library-owned
 * device array of POETX_NOALLOC_SCRATCH_BYTES bytes, one per GPU, which
 * exists from the library's load on that GPU until the process ends; the
 * call itself allocates nothing.  It needs nblk*b*b*2 bytes for bf16 blocks
 * of 64..512 (e.g. up to 64 blocks of 512 or 256 of 256) and none
 * otherwise; more gives ERR_WORKSPACE with nothing enqueued.  Every call on
 * a GPU shares that GPU's array, and each call overwrites what it reads
 * before reading it (nothing needs clearing), so calls that overlap on one
 * GPU -- on different streams, or from different threads -- race and give
 * wrong G.  The array is the one of the calling thread's current device;
 * `stream` must belong to that device.
 * Errors as poetx_cnp_fwd (ERR_WORKSPACE: the blocks exceed the array).
 */
#define POETX_NOALLOC_SCRATCH_BYTES (32u << 20)
int32_t poetx_cnp_fwd_noalloc(int32_t nblk, int32_t b, int32_t k, const float* theta,
                              void* G, void* GT, int32_t g_dtype, poetx_stream_t stream);

/*
 * poetx_cnp_bwd -- gradient of the packed parameters (technical summary 2.4:
 * the backward pass reuses on-chip data and fuses, like the forward).
 * Given dG = dL/dG [nblk][b][b] float32, writes
 *   dtheta[t(i,j)] (=|+=) gQ[i][j] - gQ[j][i],  i < j,
 * where gQ = dL/dQ for G(Q) above.  accumulate != 0 adds into dtheta.
 *   prec: POETX_F32 (fp32 arithmetic, b <= 64) or POETX_BF16 (bf16 MFMA
 *         operands with fp32 accumulation), the class of the layer's G.
 *   ws: poetx_cnp_workspace_bytes(nblk, b, k, 1, prec) bytes.
 * Errors as poetx_cnp_fwd (null dG/dtheta -> ERR_ARG).
 */
int32_t poetx_cnp_bwd(int32_t nblk, int32_t b, int32_t k, const float* theta,
                      const float* dG, float* dtheta, int32_t accumulate,
                      int32_t prec, void* ws, size_t ws_bytes,
                      poetx_stream_t stream);

/*
 * poetx_cnp_bwd_after_fwd -- poetx_cnp_bwd for the step's own forward pass:
 * the same arguments and results (bitwise), but `ws` must be the workspace
 * that last served poetx_cnp_fwd with the same nblk, b, k, theta and
 * precision (g_dtype = prec), untouched since.  On the bf16 MFMA path the
 * forward leaves the unpacked Q at the start of its workspace and this call
 * reads it there instead of unpacking theta again (one kernel less); other
 * configurations do exactly what poetx_cnp_bwd does.  ws is sized for the
 * backward, poetx_cnp_workspace_bytes(nblk, b, k, 1, prec), which also
 * serves the forward.  Passing a workspace that does not hold that Q gives
 * wrong dtheta; it is not detected.
 * Errors as poetx_cnp_bwd.
 */
int32_t poetx_cnp_bwd_after_fwd(int32_t nblk, int32_t b, int32_t k, const float* theta,
                                const float* dG, float* dtheta, int32_t accumulate,
                                int32_t prec, void* ws, size_t ws_bytes,
                                poetx_stream_t stream);

/* Workspace bytes for poetx_cnp_fwd (which = 0) or poetx_cnp_bwd (1) with
 * float32 (act = POETX_F32) or bf16 (POETX_BF16) activations;
 * 0 on bad arguments. */
size_t poetx_cnp_workspace_bytes(int32_t nblk, int32_t b, int32_t k,
                                 int32_t which, int32_t act);

/*
 * poetx_fold_perm -- permutation reduction (technical summary 2.2: two of
 * the four forward permutations are merged into the weight before the inner
 * loop).  Pure data movement, bit-exact:
 *   W0f[i][j]  = W0[perm_R[i]][perm_P[j]]        [m][n]
 *   W0fT[j][i] = W0f[i][j]                       [n][m], or NULL
 *   perm_R_inv[perm_R[i]] = i  (m entries), perm_P_inv likewise (n), or NULL.
 * W0fT is the layout the backward dV = dZ W0f product reads.
 * Errors: ERR_ARG (m, n < 1, null W0/perm/W0f, dt not F32/BF16).
 */
int32_t poetx_fold_perm(int32_t m, int32_t n, int32_t dt, const void* W0,
                        const int32_t* perm_R, const int32_t* perm_P, void* W0f,
                        void* W0fT, int32_t* perm_R_inv, int32_t* perm_P_inv,
                        poetx_stream_t stream);

/*
 * POET-XQ ("POET-X ...", technical summary 2.6: training on a low-bit base
 * model, INT8, dequantized on the fly when needed; the high-precision weight
 * is never kept).  The base weight is held as int8 q with one fp32 scale per
 * output row: W0[i][j] = s[i] * q[i][j].  poetx_fold_perm folds q
 * (dt = POETX_I8) into q_f and q_fT; poetx_fold_scale folds the scales.
 * poetx_layer_fwd_q / poetx_layer_bwd_q run the layer on (q_f, q_fT, s_f)
 * directly: the dense kernel widens the int8 operand to bf16 as it reads it
 * (exact) and applies s_f to its fp32 sums, so no high-precision copy of the
 * weight exists at any point.  poetx_dequant (an explicit bf16 copy) remains
 * for callers that want one.
 *
 * poetx_fold_scale -- s_f[i] = s[perm_R[i]], i < m (fp32).
 * poetx_dequant -- out[r][c] = bf16(scale * q[r][c]) for q int8 [rows][cols]
 *   (cols % 16 == 0, 16-byte aligned); per_row = 1: scale[r] (q_f against
 *   s_f gives W0f), per_row = 0: scale[c] (q_fT against s_f gives W0fT).
 *   Rounds to nearest even.
 * Errors: ERR_ARG, ERR_DEVICE.
 */
int32_t poetx_fold_scale(int32_t m, const float* s, const int32_t* perm_R, float* s_f,
                         poetx_stream_t stream);
int32_t poetx_dequant(int32_t rows, int32_t cols, const void* q, const float* scale,
                      int32_t per_row, void* out, poetx_stream_t stream);

/*
 * poetx_layer_fwd_q / poetx_layer_bwd_q -- poetx_layer_fwd / _bwd (xmem = 0)
 * or their memory-saving variants (xmem != 0) on an int8 base weight
 * (technical summary 2.6), with W0f = diag(s_f) q_f in place of the bf16 W0f:
 *   q_f  [m][n] int8, q_fT [n][m] int8 (poetx_fold_perm with POETX_I8),
 *   s_f  [m] fp32 (poetx_fold_scale).
 * The forward forms Z = (V q_f^T) diag(s_f); the backward forms
 * dZ' = dZ diag(s_f) in the R-side block pass and dV = dZ' q_f.  Every
 * other argument, and the saved / workspace sizes (which 0..3 as for the
 * bf16 calls), are those of the bf16 calls.  bwd: G_P and q_f are read only
 * with xmem (may be NULL otherwise).  Needs bf16 activations, b >= 64 and
 * m, n multiples of 256 (ERR_UNSUPPORTED otherwise).
 * Errors: ERR_ARG, ERR_UNSUPPORTED, ERR_WORKSPACE, ERR_DEVICE.
 */
int32_t poetx_layer_fwd_q(const poetx_shape* sh, const void* x, const void* G_P, const void* G_R,
                          const int8_t* q_f, const float* s_f, const int32_t* perm_P,
                          const int32_t* perm_R_inv, void* y, void* saved, void* ws,
                          size_t ws_bytes, int32_t xmem, poetx_stream_t stream);
int32_t poetx_layer_bwd_q(const poetx_shape* sh, const void* dy, const void* G_P, const void* GT_P,
                          const void* GT_R, const int8_t* q_f, const int8_t* q_fT,
                          const float* s_f, const int32_t* perm_P_inv, const int32_t* perm_R,
                          const void* saved, void* dx, float* dG_P, float* dG_R, void* ws,
                          size_t ws_bytes, int32_t xmem, poetx_stream_t stream);

/*
 * poetx_layer_fwd -- input-centric forward pass (technical summary 2.1-2.3).
 *   x     [T][n]        input (act)
 *   G_P   [n/b][b][b]   P-side blocks (act), from poetx_cnp_fwd
 *   G_R   [m/b][b][b]   R-side blocks (act)
 *   W0f   [m][n]        folded weight (act), from poetx_fold_perm
 *   perm_P [n], perm_R_inv [m]  int32 index maps
 *   y     [T][m]        output (act)
 *   saved poetx_saved_bytes(sh) bytes: activations kept for the backward
 *         pass (U = x[:, pi_P] then Z, both [T][*] act); the caller keeps it
 *         alive and unmodified until poetx_layer_bwd.
 *   ws    poetx_workspace_bytes(sh, 0) bytes of scratch.
 * Errors: ERR_ARG, ERR_UNSUPPORTED, ERR_WORKSPACE, ERR_DEVICE.
 */
int32_t poetx_layer_fwd(const poetx_shape* sh, const void* x, const void* G_P,
                        const void* G_R, const void* W0f, const int32_t* perm_P,
                        const int32_t* perm_R_inv, void* y, void* saved,
                        void* ws, size_t ws_bytes, poetx_stream_t stream);

/*
 * poetx_layer_bwd -- backward pass ("POET-X ...", technical summary 2.1-2.3:
 * the same input-centric chain run in reverse, block products batched,
 * permutations as index maps; 2.5: the default, fast mode keeps the
 * forward's activations for it; "Reparameterized LLM Training ...",
 * Abstract: W0 stays fixed, only the orthogonal factors learn).
 *   dy    [T][m]        dL/dy (act)
 *   GT_P  [n/b][b][b]   P-side blocks transposed (act), from poetx_cnp_fwd
 *   GT_R  [m/b][b][b]   R-side blocks transposed (act)
 *   W0f   [m][n]        folded weight (act), the forward's own
 *   W0fT  [n][m]        its transpose (act) or NULL.  With NULL the dense
 *                       product dV = dZ W0f reads W0f itself (K-major), so
 *                       the fixed weight is held once; with a transposed
 *                       copy it reads that.  Both give bitwise the same
 *                       results.
 *   perm_P_inv [n], perm_R [m]  int32 index maps
 *   saved as written by poetx_layer_fwd for the same shape and inputs
 *   dx    [T][n]        dL/dx (act)
 *   dG_P  [n/b][b][b], dG_R [m/b][b][b]  float32 dL/dG (overwritten)
 *   ws    poetx_workspace_bytes(sh, 1) bytes of scratch.
 * The token reduction of dG is deterministic (no atomics): repeated calls
 * give bitwise-equal results.
 * Errors: ERR_ARG, ERR_UNSUPPORTED, ERR_WORKSPACE, ERR_DEVICE.
 */
int32_t poetx_layer_bwd(const poetx_shape* sh, const void* dy, const void* GT_P,
                        const void* GT_R, const void* W0f, const void* W0fT,
                        const int32_t* perm_P_inv, const int32_t* perm_R,
                        const void* saved, void* dx, float* dG_P, float* dG_R,
                        void* ws, size_t ws_bytes, poetx_stream_t stream);

/*
 * poetx_layer_fwd_xmem / poetx_layer_bwd_xmem -- the memory-saving mode
 * ("POET-X ...", technical summary 2.5: recompute in the backward pass
 * instead of keeping intermediates).  The forward keeps only U = x[:, pi_P]
 * in `saved` (poetx_saved_bytes_xmem(sh) bytes) and writes Z to its
 * workspace; the backward first recomputes V = U G_P^T and Z = V W0f^T with
 * the forward's own kernels, then runs as poetx_layer_bwd.  Outputs are
 * bitwise equal to those of poetx_layer_fwd / poetx_layer_bwd; the saved
 * buffer is T*m*sizeof(act) bytes smaller and the backward does one more
 * dense product (2 T m n flops) and one more block product (2 T n b flops).
 *   fwd: arguments as poetx_layer_fwd; ws poetx_workspace_bytes(sh, 2) bytes.
 *   bwd: arguments as poetx_layer_bwd plus G_P [n/b][b][b] (act) (W0fT
 *        may be NULL as there); ws poetx_workspace_bytes(sh, 3) bytes.
 * Errors: ERR_ARG, ERR_UNSUPPORTED, ERR_WORKSPACE, ERR_DEVICE.
 */
int32_t poetx_layer_fwd_xmem(const poetx_shape* sh, const void* x, const void* G_P,
                             const void* G_R, const void* W0f, const int32_t* perm_P,
                             const int32_t* perm_R_inv, void* y, void* saved,
                             void* ws, size_t ws_bytes, poetx_stream_t stream);
int32_t poetx_layer_bwd_xmem(const poetx_shape* sh, const void* dy, const void* G_P,
                             const void* GT_P, const void* GT_R, const void* W0f,
                             const void* W0fT, const int32_t* perm_P_inv,
                             const int32_t* perm_R, const void* saved, void* dx,
                             float* dG_P, float* dG_R, void* ws, size_t ws_bytes,
                             poetx_stream_t stream);

/* Bytes of the saved-activation buffer of the xmem mode; 0 on bad arguments. */
size_t poetx_saved_bytes_xmem(const poetx_shape* sh);

/*
 * poetx_merge -- end of an inner loop ("POET-X ...", technical summary 2.1:
 * the learned transforms are merged into the weight, W <- R W P, before new
 * ones start from the identity; 2.2: new permutations are then drawn and
 * folded).  Writes the current effective weight
 *   W0_out = R W0 P = Pi_R^T BD(G_R) W0f BD(G_P) Pi_P,
 *   W0_out[a][c] = M[pi_R^{-1}[a]][pi_P^{-1}[c]],  M = BD(G_R) W0f BD(G_P),
 * with two block products (4 m n b flops), two transposes and the
 * permutation.  The caller then resets theta to 0, draws new permutations
 * and calls poetx_fold_perm on W0_out.  T in `sh` is not used.
 *   W0f   [m][n]        folded weight (act)
 *   G_R   [m/b][b][b]   R-side blocks (act), GT_P [n/b][b][b] P-side blocks
 *                       transposed (act), both from poetx_cnp_fwd
 *   perm_R_inv [m], perm_P_inv [n]  from poetx_fold_perm
 *   W0_out [m][n] (act); must not alias W0f
 *   ws    poetx_workspace_bytes(sh, 4) bytes of scratch.
 * Errors: ERR_ARG, ERR_UNSUPPORTED, ERR_WORKSPACE, ERR_DEVICE.
 */
int32_t poetx_merge(const poetx_shape* sh, const void* W0f, const void* G_R,
                    const void* GT_P, const int32_t* perm_R_inv, const int32_t* perm_P_inv,
                    void* W0_out, void* ws, size_t ws_bytes, poetx_stream_t stream);

/*
 * poetx_set_stage_events -- timing hook for profilers and benchmarks.
 * While set, each poetx_layer_fwd / poetx_layer_bwd call on the calling
 * thread records events[i] (hipEvent_t handles owned by the caller) on its
 * stream at stage boundary i:
 *   forward  (count >= 6): 0 | gather x | 1 | P-side blocks | 2 | W0 product
 *            | 3 | R-side blocks | 4 | scatter y | 5
 *   backward (count >= 8): 0 | gather dy | 1 | R-side blocks | 2 | dG_R |
 *            3 | W0 product | 4 | P-side blocks | 5 | dG_P | 6 | scatter dx | 7
 * When two stages run in one kernel their shared boundary is recorded
 * twice, back to back.  With bf16 (b >= 64) the dG_R reduction runs in the
 * same launch as dG_P (for b = 64 and 128 only where that launch splits the
 * tokens): stage 2..3 is then empty and stage 5..6 holds both.
 * events = NULL clears the hook.
 * Errors: ERR_ARG (events non-NULL and count < 8).
 */
int32_t poetx_set_stage_events(void* const* events, int32_t count);

/*
 * poetx_set_fused_gather -- how the layer calls of this process run an
 * input-side gather and the block products that follow it ("POET-X ...",
 * technical summary 2.2: the index map reorders data as it is read; 2.3:
 * batched block products): the forward's U = x[:, pi_P], V = U G_P^T, the
 * backward's dS = dy[:, pi_R], dZ = dS G_R, and the memory-saving
 * backward's recompute of V.  on != 0: one pass that gathers straight into
 * the block products' operands, where the layer is bf16 with b = 256 and
 * the gathered width (n, or m for dy) is a multiple of 512 up to 4096;
 * 0 (the default): a gather pass, then a block pass.  Both forms are exact
 * on the gather and agree with each other to rounding (their block
 * products sum in different orders); on MI355X the one-pass form is the
 * slower of the two at the square 4096 workload.  Workspace sizes depend on
 * the setting: set it before sizing workspaces, and keep it between a
 * forward call and the backward call that uses its saved buffer.  Returns
 * the previous setting (0 or 1).
 */
int32_t poetx_set_fused_gather(int32_t on);

/* Scratch bytes for poetx_layer_fwd (which = 0), poetx_layer_bwd (1),
 * poetx_layer_fwd_xmem (2), poetx_layer_bwd_xmem (3) or poetx_merge (4);
 * 0 on bad arguments. */
size_t poetx_workspace_bytes(const poetx_shape* sh, int32_t which);

/* Bytes of the saved-activation buffer; 0 on bad arguments. */
size_t poetx_saved_bytes(const poetx_shape* sh);

/*
 * The operators of an attention block around POET-X projections: rotary
 * positions, attention, dropout with the residual sum.  They share the
 * conventions above.  Activations (q, k, v, o, x, y and their gradients) are
 * of type `act`; rows may have a pitch: a tensor of T rows of H heads of D
 * values has head h of row t at t * ld + h * D, so q, k and v may be column
 * ranges of one projection's output.  Pitches count elements, are at least
 * H * D, at most 2^20 and multiples of 8 (16 bytes for bf16, 32 for
 * float32); the rows of an output must not overlap each other or an input,
 * except where stated.
 */

/*
 * poetx_rope -- rotary positions for q and k in one launch (the gradient is
 * the same call with inverse = 1 on dq, dk).  For token t, row p = pos[t] of
 * the table holds (c_i, s_i), i < rot/2; of every head the pairs
 *   interleaved = 0: (x_i, x_{i + rot/2}),  1: (x_{2i}, x_{2i+1})
 * become (a c - b s, a s + b c) (s negated when inverse), and elements from
 * rot to D are copied.  Scaled or stretched frequencies, and a magnitude,
 * are properties of the table.
 *   q [T][Hq][D] -> qo, k [T][Hk][D] -> ko (Hk = 0: k, ko NULL); qo = q and
 *   ko = k (same pitch) turn in place.
 *   pos [T] int32; table [P][rot/2][2] float32.  A position outside [0, P)
 *   reads nothing and writes NaN to the turned part of its row.
 * D a multiple of 8 up to 512, rot even, 2 <= rot <= D; T = 0 does nothing.
 * Errors: ERR_ARG, ERR_DEVICE.
 */
typedef struct {
  int32_t T, Hq, Hk, D, rot, P, act, interleaved, inverse;
  int64_t ldq, ldk, ldqo, ldko;
} poetx_rope_shape;
int32_t poetx_rope(const poetx_rope_shape* sh, const void* q, const void* k, const int32_t* pos,
                   const float* table, void* qo, void* ko, poetx_stream_t stream);

/*
 * poetx_qk_norm_rope_fwd / poetx_qk_norm_rope_bwd -- root mean square norms of
 * the heads of q and k, and the rotary positions of poetx_rope, in one pass:
 *   r = 1 / sqrt(mean x^2 + eps) over the D elements of a head,
 *   y = turn(x r w),
 * with weights wq, wk [D] float32 that all heads of a tensor share (NULL: 1).
 * Sums are float32; each output is rounded once.  A head whose squares sum to
 * 2^128 or more (128 elements of 2^60.5) has r = 0: its outputs are zeros, and
 * its gradients too (NaN in dq, dk where the sum of dy w x passes 2^128 as well).
 * With eps = 0 a head's root mean square is to be above 2^-63.
 * rot = 0: norms alone, pos and table are not read.
 *   fwd: q [T][Hq][D] -> qo, k [T][Hk][D] -> ko (Hk = 0: k, ko NULL); qo = q
 *   and ko = k (same pitch) work in place.  A position outside the table
 *   reads nothing and writes NaN to the turned part of its row.
 *   bwd: dqo, dko gradients of the outputs (pitches ldqo, ldko), q and k the
 *   forward's inputs -> dq, dk (pitches lddq, lddk; dq = dqo and dk = dko work
 *   in place) and dwq, dwk [D] float32, overwritten (NULL: not wanted; T = 0:
 *   zero).  A position outside the table gives NaN in its rows and in dwq, dwk.
 *   The same call gives the same bits (no atomics).
 *   ws poetx_qk_norm_rope_workspace_bytes(sh) bytes.
 * D a multiple of 8 up to 512, rot even, 0 <= rot <= D, eps >= 0.
 * Errors: ERR_ARG, ERR_WORKSPACE, ERR_DEVICE.
 */
typedef struct {
  int32_t T, Hq, Hk, D, rot, P, act, interleaved;
  float eps;
  int64_t ldq, ldk, ldqo, ldko, lddq, lddk;
} poetx_qk_norm_shape;
size_t poetx_qk_norm_rope_workspace_bytes(const poetx_qk_norm_shape* sh);
int32_t poetx_qk_norm_rope_fwd(const poetx_qk_norm_shape* sh, const void* q, const void* k, const float* wq,
                               const float* wk, const int32_t* pos, const float* table, void* qo, void* ko,
                               poetx_stream_t stream);
int32_t poetx_qk_norm_rope_bwd(const poetx_qk_norm_shape* sh, const void* dqo, const void* dko, const void* q,
                               const void* k, const float* wq, const float* wk, const int32_t* pos,
                               const float* table, void* dq, void* dk, float* dwq, float* dwk, void* ws,
                               size_t ws_bytes, poetx_stream_t stream);

/*
 * poetx_dropout_fwd / poetx_dropout_bwd -- dropout whose mask is never
 * stored, with the residual sum:
 *   y[i] = residual[i] + (keep(i) ? x[i] * g : 0),   dx[i] = keep(i) ? dy[i] * g : 0
 * (residual NULL: 0; its gradient is dy itself).  keep(i): the 16-bit lane
 * (e mod 8) of Philox 4x32-10 (Salmon et al., "Parallel random numbers: as
 * easy as 1, 2, 3", 2011) with key `seed` and counter e / 8, e = offset + i,
 * is at least t = round(p * 65536); lane 2w is the low half of word w,
 * 2w + 1 its high half.  g = 65536 / (65536 - t), so E[y] = residual + x
 * for the probability t / 65536 in effect; t = 65536 drops everything.  A
 * dropped x is not read into the sum: NaN or infinity there leaves no trace.
 *   n >= 0 contiguous elements of type act; 0 <= p <= 1; offset a multiple
 *   of 8 (a caller advances it by n rounded up to 8 per call).
 *   offset_dev: NULL, or a device uint64 (a multiple of 8) added to offset,
 *   so that a captured graph draws a new mask each replay.
 * y may be x or residual, dx may be dy.
 * Errors: ERR_ARG, ERR_DEVICE.
 */
int32_t poetx_dropout_fwd(int64_t n, int32_t act, const void* x, const void* residual, void* y,
                          double p, uint64_t seed, uint64_t offset, const uint64_t* offset_dev,
                          poetx_stream_t stream);
int32_t poetx_dropout_bwd(int64_t n, int32_t act, const void* dy, void* dx, double p, uint64_t seed,
                          uint64_t offset, const uint64_t* offset_dev, poetx_stream_t stream);

/*
 * Attention over packed documents.  Tq query rows and Tk key rows hold ndoc
 * documents one after the other: document d has query rows [cu_q[d],
 * cu_q[d+1]) and key rows [cu_k[d], cu_k[d+1]) (lengths may differ and be
 * 0); rows before cu[0] and from cu[ndoc] on belong to none.  Query i (of Lq)
 * of a document stands at key position i + Lk - Lq (the ends are aligned);
 * it sees every key of its document, with causal != 0 only those at j <= its
 * position or j < prefix[d] (prefix NULL: 0).  Head h reads key head
 * h / (Hq / Hkv).  With x = scale * q.k,
 *   s = cap > 0 ? cap * tanh(x / cap) : x,   s -= slopes[h] * |position - j|,
 *   p = exp(s - lse),  lse = log sum_j exp(s),  o = sum_j p v_j
 * over the keys seen.  A query that sees none has o = 0, lse = -inf and
 * takes no part in any gradient.  Keys and values that a query does not see
 * have no influence on it, whatever they hold (NaN included); rows whose
 * result is not finite are formed once more, one at a time, which is slow.
 * Backward: delta = do.o;  dl = p (do.v - delta);  ds = dl (1 - tanh^2) scale;
 *   dq = sum ds k;  dk, dv sum over the query heads that share a key head.
 * slopes are constants (no gradient).  The bf16 path rounds p and ds to bf16
 * as matrix operands; sums, lse and delta are float32.  The same call gives
 * the same bits (no atomics); Tq, Tk, ndoc and the heads decide the order of
 * the sums, so a document's last bits may differ in another batch.
 *   scale <= 0 selects 1 / sqrt(D); cap = 0: no cap; slopes [Hq] or NULL.
 *   D a multiple of 8 up to 128; Hq a multiple of Hkv.  Tq and Tk are at most
 *   2^31 - 2^16, and tiles of 128 rows times heads fewer than 2^24 on a side.
 *   ldq, ldk, ldv, ldo: pitches of q, k, v, o; lddo, lddq, lddk, lddv of dout
 *   and the gradients.
 */
typedef struct {
  int32_t Tq, Tk, ndoc, Hq, Hkv, D, act, causal;
  float scale, cap;
  int64_t ldq, ldk, ldv, ldo, lddo, lddq, lddk, lddv;
} poetx_attn_shape;

/* Bytes of a plan (0 on bad arguments), and of the workspace of
 * poetx_attn_fwd (which = 0) or poetx_attn_bwd (1; also enough for the
 * forward pass of the same shape). */
size_t poetx_attn_plan_bytes(const poetx_attn_shape* sh);
size_t poetx_attn_workspace_bytes(const poetx_attn_shape* sh, int32_t which);

/*
 * poetx_attn_plan -- the mask of a packed batch as intervals: the keys each
 * query row sees and the queries that see each key row.  One plan serves
 * every layer, head and direction of that batch.  It depends on Tq, Tk, ndoc
 * and causal only.
 *   cu_q, cu_k [ndoc+1] int32, prefix [ndoc] int32 or NULL; plan
 *   poetx_attn_plan_bytes(sh) bytes.  Offsets that decrease or leave [0, T]
 *   are clamped: they give some mask, never an access out of range.
 * Errors: ERR_ARG, ERR_WORKSPACE (plan_bytes too small), ERR_DEVICE.
 */
int32_t poetx_attn_plan(const poetx_attn_shape* sh, const int32_t* cu_q, const int32_t* cu_k,
                        const int32_t* prefix, void* plan, size_t plan_bytes,
                        poetx_stream_t stream);

/*
 * poetx_attn_fwd / poetx_attn_bwd.
 *   q [Tq][Hq][D], k, v [Tk][Hkv][D], o, dout, dq like q, dk, dv like k (act);
 *   lse [Hq][Tq] float32 (written by fwd, read by bwd); plan from
 *   poetx_attn_plan; ws poetx_attn_workspace_bytes(sh, 0 | 1) bytes.
 * Errors: ERR_ARG, ERR_WORKSPACE, ERR_DEVICE.
 */
int32_t poetx_attn_fwd(const poetx_attn_shape* sh, const void* q, const void* k, const void* v,
                       const float* slopes, const void* plan, void* o, float* lse, void* ws,
                       size_t ws_bytes, poetx_stream_t stream);
int32_t poetx_attn_bwd(const poetx_attn_shape* sh, const void* dout, const void* q, const void* k,
                       const void* v, const void* o, const float* lse, const float* slopes,
                       const void* plan, void* dq, void* dk, void* dv, void* ws, size_t ws_bytes,
                       poetx_stream_t stream);

/*
 * Attention with a window and sinks: as above, but a query at position p sees
 * only keys closer than `window` (causal: p - window < j <= p, otherwise
 * |p - j| < window) and the first `sinks` keys of its document (causal: those
 * at j <= p).  There are no prefixes.  window = 0: no window (sinks is then
 * without meaning), the calls are those above.
 *   window >= 0; 0 <= sinks <= 128; ndoc sinks Hkv < 2^22.
 * plan, workspace and calls take the same window; everything else, errors
 * included, as in poetx_attn_plan, _fwd and _bwd.
 */
typedef struct { int32_t window, sinks; } poetx_window;
size_t poetx_attn_window_plan_bytes(const poetx_attn_shape* sh, const poetx_window* win);
size_t poetx_attn_window_workspace_bytes(const poetx_attn_shape* sh, const poetx_window* win, int32_t which);
int32_t poetx_attn_window_plan(const poetx_attn_shape* sh, const poetx_window* win, const int32_t* cu_q,
                               const int32_t* cu_k, void* plan, size_t plan_bytes, poetx_stream_t stream);
int32_t poetx_attn_window_fwd(const poetx_attn_shape* sh, const poetx_window* win, const void* q, const void* k,
                              const void* v, const float* slopes, const void* plan, void* o, float* lse,
                              void* ws, size_t ws_bytes, poetx_stream_t stream);
int32_t poetx_attn_window_bwd(const poetx_attn_shape* sh, const poetx_window* win, const void* dout, const void* q,
                              const void* k, const void* v, const void* o, const float* lse, const float* slopes,
                              const void* plan, void* dq, void* dk, void* dv, void* ws, size_t ws_bytes,
                              poetx_stream_t stream);

/*
 * poetx_attn_decode -- the single-token form: one query row per sequence over
 * a cache, same scores as above (bf16: p in two bf16 parts).  Sequence b sees cache rows [start[b],
 * len[b]) (start NULL: 0; both clamped to [0, rows]); its query stands at
 * position len[b] - 1.  An empty range gives o = 0.
 *   q, o [B][Hq][D] (pitches ldq, ldo); row j of sequence b of the caches
 *   at b * bsk + j * ldk, b * bsv + j * ldv (offsets are 64-bit), heads of
 *   D values side by side; rows: cache capacity per sequence, at most
 *   2^31 - 2^16; B Hkv ceil(Hq / Hkv / 32) below 2^24.
 *   ws poetx_attn_decode_workspace_bytes(sh) bytes.
 * Errors: ERR_ARG, ERR_WORKSPACE, ERR_DEVICE.
 */
typedef struct {
  int32_t B, Hq, Hkv, D, act, rows;
  float scale, cap;
  int64_t ldq, ldo, ldk, ldv, bsk, bsv;
} poetx_decode_shape;
size_t poetx_attn_decode_workspace_bytes(const poetx_decode_shape* sh);
int32_t poetx_attn_decode(const poetx_decode_shape* sh, const void* q, const void* k, const void* v,
                          const int32_t* start, const int32_t* len, const float* slopes, void* o,
                          void* ws, size_t ws_bytes, poetx_stream_t stream);

/*
 * poetx_attn_window_decode -- the same with a window and sinks: the query at
 * position len[b] - 1 sees the last `window` positions and the first `sinks`
 * ones (window = 0: all).
 *   ring = 0: position p lies in row p, len is clamped to [0, rows].
 *   ring != 0: the cache is a ring.  Positions below `sinks` lie in their rows,
 *   p >= sinks in row sinks + (p - sinks) mod (rows - sinks); len counts every
 *   token there has been and may pass rows.  1 <= window <= rows - sinks.
 *   B Hq below 2^24.
 *   ws poetx_attn_window_decode_workspace_bytes(sh, win) bytes, for either.
 * Everything else as in poetx_attn_decode.
 */
size_t poetx_attn_window_decode_workspace_bytes(const poetx_decode_shape* sh, const poetx_window* win);
int32_t poetx_attn_window_decode(const poetx_decode_shape* sh, const poetx_window* win, int32_t ring, const void* q,
                                 const void* k, const void* v, const int32_t* len, const float* slopes, void* o,
                                 void* ws, size_t ws_bytes, poetx_stream_t stream);

/*
 * A key/value cache held in 4 bits: blocks of 32 consecutive elements of a head
 * (the last one filled up with zeros), codes e2m1 (a sign and 0, .5, 1, 1.5, 2,
 * 3, 4 or 6: codes 0..7, 8 more when negative) and a scale 2^e, held as e + 127:
 * the microscaling format MXFP4 of the Open Compute Project, 4.25 bits an element.
 *   kc, vc  [B][Hkv][rows][blocks * 16] bytes, element 2 i of a row in the low
 *           half of byte i; blocks = (D + 31) / 32
 *   ks, vs  [B][Hkv][blocks][rows] bytes
 * rows is a multiple of 64.  A held value is exact in bf16.
 *
 * poetx_kv4_write puts token t, row t of k and v [T][Hkv][D] (act), at position
 * pos[t] of sequence seq[t] (seq NULL: t); nothing is written for a token whose
 * sequence or position the cache does not have.  e is the least from -127 on with
 * max |x| < 7 * 2^e, at most 125; a code is the nearest of x / 2^e, ties to the
 * even code, 6 above that.  A block with NaN or infinity reads as NaN.
 *   ring and sinks as in poetx_attn_window_decode: without a ring, position p
 *   lies in row p.  Tokens of one call must have rows of their own.
 * poetx_kv4_read gives back the values at such places (NaN where the cache has
 * none; in a ring, what the position's row holds now).
 *   T Hkv < 2^27, T rounded up to a multiple of 16; ldk, ldv: pitches of k and v.
 * Errors: ERR_ARG, ERR_DEVICE.
 */
typedef struct {
  int32_t T, B, rows, Hkv, D, act, sinks, ring;
  int64_t ldk, ldv;
} poetx_kv4_shape;
int32_t poetx_kv4_write(const poetx_kv4_shape* sh, const void* k, const void* v, const int32_t* seq, const int32_t* pos,
                        void* kc, void* ks, void* vc, void* vs, poetx_stream_t stream);
int32_t poetx_kv4_read(const poetx_kv4_shape* sh, const int32_t* seq, const int32_t* pos, const void* kc, const void* ks,
                       const void* vc, const void* vs, void* k, void* v, poetx_stream_t stream);

/*
 * poetx_attn_kv4_decode -- poetx_attn_decode (window = 0, with start) or
 * poetx_attn_window_decode (without) over such a cache, B Hq below 2^24.  The products of the
 * held values are exact, sums float32 (bf16: p in two bf16 parts; float32: q and
 * p in three).  Of the shape ldk, ldv, bsk and bsv have to be valid and are not
 * used.
 *   ws poetx_attn_kv4_decode_workspace_bytes(sh, win) bytes, for either kind of
 *   cache.
 * Errors: ERR_ARG, ERR_WORKSPACE, ERR_DEVICE.
 */
size_t poetx_attn_kv4_decode_workspace_bytes(const poetx_decode_shape* sh, const poetx_window* win);
int32_t poetx_attn_kv4_decode(const poetx_decode_shape* sh, const poetx_window* win, int32_t ring, const void* q,
                              const void* kc, const void* ks, const void* vc, const void* vs, const int32_t* start,
                              const int32_t* len, const float* slopes, void* o, void* ws, size_t ws_bytes,
                              poetx_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* POETX_H */

/*
 * dwconv_seq.h -- C ABI of the sequence operators of libdwconv.so (gfx950):
 * the parts of a recurrent token-mixing block around the depthwise filter.
 * Status codes, activations and the rules on ownership, execution and errors
 * are those of dwconv.h: device pointers owned by the caller, no allocation,
 * no state between calls, work enqueued on `stream`, every argument checked
 * before anything is enqueued.
 *
 * Tensors are token-major: a row per token, its channels contiguous, and
 * `ld*` elements from one row to the next (at least the row's width), so a
 * tensor may be a column range of a wider one.  Arrays without an `ld`
 * argument are dense.
 *
 * Sequences.  offsets = NULL: `seqs` sequences of `tokens` rows each, one
 * after the other.  Otherwise `tokens` is the number of rows in all and
 * offsets a DEVICE array of seqs + 1 int32: sequence s is the rows
 * [offsets[s], offsets[s+1]).  Offsets do not decrease, the first is 0 and
 * the last `tokens`; sequences of no row are allowed.  Offsets that break
 * this give unspecified rows, but no access outside the arrays: the kernels
 * clamp what they read.  tokens = 0 is allowed (pointers to arrays of no row
 * may then be NULL).
 *
 * Rows in all, sequences, and channels: at most DWCONV_SEQ_MAX_ROWS each (the
 * kernels count them in 32 bits and look some way ahead of the last one); outputs and
 * inputs of a linear map: fewer than 2^31.  Addresses are computed in 64 bits.
 * Pointers are aligned to their element.
 *
 * Arrays that are written must not overlap each other or an input, except
 * where an in-place update is named; two column ranges of one wider array
 * (equal row strides) do not overlap.
 *
 * Arithmetic is in float32 whatever the tensors' type, rounded once where a
 * result is stored, unless stated.  Sums over tokens are in a fixed order:
 * the same call gives the same bits.
 */
#ifndef DWCONV_SEQ_H
#define DWCONV_SEQ_H

#include "dwconv.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Element types (passed as int). */
#define DWCONV_T_F32  0
#define DWCONV_T_F16  1   /* IEEE binary16 */
#define DWCONV_T_BF16 2   /* bfloat16      */

#define DWCONV_SEQ_MAX_ROWS 2147418112   /* 2^31 - 2^16 */

#define DWCONV_CAUSAL_MAX_TAPS 8   /* taps of the causal filter: 1 .. 8 */

/* ---- causal depthwise convolution over tokens ----------------------------
 *
 *   z[t,c] = b[c] + sum_{j<K} w[c,j] * x[t - (K-1) + j, c],   y = act(z)
 *
 * within each sequence.  Rows before its start are the carried rows
 * init[s, 0..K-2] (oldest first), or zero where init is NULL.  final, if not
 * NULL, receives the K-1 rows that a continuation carries: the last K-1 rows
 * of (init, x).  x, y, init and final are of `type`; w is [C][K] of `wtype`;
 * b is [C] float32 or NULL; init and final are [seqs][K-1][C].
 */
int dwconv_causal_fwd(const void *x, long long ldx, int type, const void *w, int wtype,
                      const float *b, int act, const void *init, void *y, long long ldy,
                      void *final_state, int seqs, long long tokens, const int *offsets, int C,
                      int K, void *stream);

/* One token for each sequence: row s of x continues the carried rows
 * state[s] ([seqs][K-1][C]), which are updated in place. */
int dwconv_causal_step(const void *x, long long ldx, int type, const void *w, int wtype,
                       const float *b, int act, void *state, void *y, long long ldy, int seqs,
                       int C, int K, void *stream);

/* Gradients.  dy is the cotangent of y; dfinal ([seqs][K-1][C] of `type`)
 * that of final, or NULL for zero.  z is computed again from x, w, b, init.
 *
 *   dz = dy * act'(z)
 *   dx[t] = sum_j w[j] * dz[t + K-1-j]  (within the sequence)  + dfinal's share
 *   dw[c,j] = sum_t dz[t,c] * x[t - (K-1) + j, c],   db[c] = sum_t dz[t,c]
 *
 * act' is 0 at the corners of ReLU and ReLU6.  dx and dinit (NULL to skip)
 * are of `type`; dw [C][K] and db [C] (NULL to skip) float32.  workspace: at
 * least dwconv_causal_grad_workspace_size bytes, 16-byte aligned. */
int dwconv_causal_grad_workspace_size(int seqs, long long tokens, int packed, int C, int K,
                                      long long *bytes);
int dwconv_causal_grad(const void *dy, long long lddy, const void *x, long long ldx, int type,
                       const void *w, int wtype, const float *b, int act, const void *init,
                       const void *dfinal, void *dx, long long lddx, float *dw, float *db,
                       void *dinit, void *workspace, long long workspace_bytes, int seqs,
                       long long tokens, const int *offsets, int C, int K, void *stream);

/* ---- gated linear recurrence ----------------------------------------------
 *
 * With sigma the logistic function, per channel c and token t
 *
 *   log a[t,c] = -scale * softplus(lam[c]) * sigma(r[t,c])
 *   h[t,c] = a[t,c] * h[t-1,c] + sqrt(1 - a[t,c]^2) * sigma(i[t,c]) * x[t,c]
 *
 * within each sequence, h before its start being h0[s,c] (or zero where h0 is
 * NULL).  y = h in `type`, the type of x, r and i; lam is [C] float32; h0 and
 * hT, the state after the last token (h0 itself for a sequence of none; NULL
 * to skip), are [seqs][C] float32.  scale > 0 and finite.  Row strides are
 * below 2^21 elements.
 *
 * states (NULL to skip): dwconv_scan_states_size floats that the gradient
 * needs, the float32 state before each run of DWCONV_SCAN_RUN tokens of a
 * sequence.  workspace: at least dwconv_scan_workspace_size(grad = 0) bytes,
 * 16-byte aligned (NULL where that is 0). */
#define DWCONV_SCAN_RUN 8

int dwconv_scan_states_size(int seqs, long long tokens, int packed, int C, long long *floats);
int dwconv_scan_workspace_size(int grad, int seqs, long long tokens, int packed, int C,
                               long long *bytes);
int dwconv_scan_fwd(const void *x, long long ldx, const void *r, long long ldr, const void *i,
                    long long ldi, int type, const float *lam, float scale, const float *h0,
                    void *y, long long ldy, float *hT, float *states, void *workspace,
                    long long workspace_bytes, int seqs, long long tokens, const int *offsets,
                    int C, void *stream);

/* One token for each sequence; h [seqs][C] float32 is updated in place. */
int dwconv_scan_step(const void *x, long long ldx, const void *r, long long ldr, const void *i,
                     long long ldi, int type, const float *lam, float scale, float *h, void *y,
                     long long ldy, int seqs, int C, void *stream);

/* Gradients, from the states that the forward kept.  dy is the cotangent of
 * y, dhT [seqs][C] float32 that of hT (NULL for zero).
 *
 *   g[t] = dy[t] + a[t+1] * g[t+1]        (dhT added at the last token)
 *   dx = g * beta * sigma(i)              beta = sqrt(1 - a^2)
 *   di = g * beta * x * sigma(i) * (1 - sigma(i))
 *   dlog = g * (a * h[t-1] - sigma(i) * x * a^2 / beta)
 *   dr = -dlog * scale * softplus(lam) * sigma(r) * (1 - sigma(r))
 *   dlam = -sum_t dlog * sigma(r) * scale * sigma(lam),   dh0 = a[0] * g[0]
 *
 * Where beta is 0 (a gate that is fully shut) the second part of dr and dlam
 * is 0, its limit.  dx, dr, di are of `type`; dlam [C] and dh0 [seqs][C]
 * (NULL to skip) float32. */
int dwconv_scan_grad(const void *dy, long long lddy, const void *x, long long ldx, const void *r,
                     long long ldr, const void *i, long long ldi, int type, const float *lam,
                     float scale, const float *states, const float *dhT, void *dx,
                     long long lddx, void *dr, long long lddr, void *di, long long lddi,
                     float *dlam, float *dh0, void *workspace, long long workspace_bytes,
                     int seqs, long long tokens, const int *offsets, int C, void *stream);

/* ---- matrix product with bias, activation and residual ---------------------
 *
 *   z[m,n] = sum_k x[m,k] * w[n,k] + b[n],   y = act(z) + res
 *
 * x is M rows of K, w N rows of K, y, z and res M rows of N, all of `type`;
 * b [N] float32 or NULL; res NULL for none; z (NULL to skip) receives the
 * value before the activation, which the gradient needs.  Products of 16-bit
 * elements are exact and summed in float32; float32 elements are multiplied
 * to float32 accuracy.  workspace: at least dwconv_linear_workspace_size
 * (grad = 0) bytes, 16-byte aligned (NULL where that is 0).  M = 0 is
 * allowed.  Row strides are below 2^21 elements. */
int dwconv_linear_workspace_size(int grad, int type, int act, long long M, int N, int K,
                                 long long *bytes);
int dwconv_linear_fwd(const void *x, long long ldx, const void *w, long long ldw, int type,
                      const float *b, int act, const void *res, long long ldres, void *y,
                      long long ldy, void *z, long long ldz, void *workspace,
                      long long workspace_bytes, long long M, int N, int K, void *stream);

/* Gradients: dz = dy * act'(z), dx = dz w, dw = dz^T x, db = sum_m dz.  z is
 * what the forward kept (ignored, may be NULL, for DWCONV_ACT_NONE); the
 * residual's gradient is dy itself.  dx, dw, db: NULL to skip; dx and dw are
 * of `type`, db float32.  For 16-bit types dz enters the two products
 * rounded to `type`, as a stored gradient would; db sums it unrounded. */
int dwconv_linear_grad(const void *dy, long long lddy, const void *x, long long ldx,
                       const void *w, long long ldw, int type, int act, const void *z,
                       long long ldz, void *dx, long long lddx, void *dw, long long lddw,
                       float *db, void *workspace, long long workspace_bytes, long long M, int N,
                       int K, void *stream);

/* Describe, without touching the GPU, the kernel of one product of these calls:
 * y, dx or dw.  Writes its name (NUL-terminated, at most name_len bytes) and over
 * how many ranges of the summed index it is split, each where not NULL.
 * aligned: whether the addresses and row strides of both operands are multiples
 * of 16 bytes (dz, where there is an activation, is dense). */
#define DWCONV_LINEAR_Y  0
#define DWCONV_LINEAR_DX 1
#define DWCONV_LINEAR_DW 2
int dwconv_linear_describe(int product, int type, int aligned, long long M, int N, int K,
                           char *name, int name_len, int *splits);

#ifdef __cplusplus
}
#endif

#endif /* DWCONV_SEQ_H */

/*
 * dwconv_mix.h -- C ABI of the mixing operators of libdwconv.so (gfx950): what
 * a token-mixing block or a separable convolution net has around its filters
 * beside the operators of dwconv_seq.h, whose rules on tensors, sequences,
 * strides, aliasing and arithmetic hold here too (and with them those of
 * dwconv.h on ownership, execution and errors).
 */
#ifndef DWCONV_MIX_H
#define DWCONV_MIX_H

#include "dwconv_seq.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ---- linear attention with a decay for each head ---------------------------
 *
 * For each of H heads, with a = exp(log_decay[h]) and S a Dk x Dv matrix,
 *
 *   S[t] = a * S[t-1] + k[t] v[t]^T,     y[t] = scale * q[t] S[t]
 *
 * within each sequence, S before its start being h0[s] (or zero where h0 is
 * NULL).  A row of q is H heads of Dk elements, one after the other, of k KV
 * heads of Dk, of v KV heads of Dv, of y H heads of Dv, all of `type`; KV
 * divides H, and head h reads the keys and values of head h / (H / KV).
 * log_decay is [H] float32, a constant of the model (it has no gradient):
 * numbers above 0 count as 0, minus infinity forgets everything.  h0 and hT,
 * the state after the last token (h0 itself for a sequence of none; NULL to
 * skip), are [seqs][H][Dk][Dv] float32.  scale is finite.  Dk and Dv are at most
 * DWCONV_ATTENTION_MAX_DIM; row strides are below 2^21 elements.
 *
 * Tokens are taken in chunks.  For 16-bit types the scores q[i] . k[j] of a
 * chunk, times their decay, and the state that a chunk starts from enter a
 * product as the sum of two numbers of `type` (the state itself is kept and
 * passed on in float32); float32 tensors are multiplied to float32 accuracy.
 * What float16 has too few exponents for is scaled by a power of two, 16 columns of
 * the values or of the state and 16 rows of scores by one: besides the two numbers'
 * 2^-22 of itself, a number then loses at most 2^-25 while the largest of those beside
 * it is below 2^14, and 2^-38 of that one where it is above.
 * A token's infinities and NaN reach the tokens after it, never those before it; an
 * infinity of q or k may reach results of a 16-bit type as NaN.
 * workspace: at least dwconv_attention_workspace_size(grad = 0) bytes, 16-byte
 * aligned (NULL where that is 0). */
#define DWCONV_ATTENTION_MAX_DIM 256

int dwconv_attention_workspace_size(int grad, int type, int seqs, long long tokens, int packed,
                                    int H, int KV, int Dk, int Dv, long long *bytes);
int dwconv_attention_fwd(const void *q, long long ldq, const void *k, long long ldk,
                         const void *v, long long ldv, int type, const float *log_decay,
                         float scale, const float *h0, void *y, long long ldy, float *hT,
                         void *workspace, long long workspace_bytes, int seqs, long long tokens,
                         const int *offsets, int H, int KV, int Dk, int Dv, void *stream);

/* One token for each sequence; h [seqs][H][Dk][Dv] float32 is updated in place.
 * In float32 throughout. */
int dwconv_attention_step(const void *q, long long ldq, const void *k, long long ldk,
                          const void *v, long long ldv, int type, const float *log_decay,
                          float scale, float *h, void *y, long long ldy, int seqs, int H, int KV,
                          int Dk, int Dv, void *stream);

/* Gradients.  dy is the cotangent of y, dhT ([seqs][H][Dk][Dv] float32) that of
 * hT, or NULL for zero; the states are computed again from k, v and h0.
 *
 *   dq[t] = scale * S[t] dy[t]
 *   G[t] = a * G[t+1] + scale * q[t] dy[t]^T      (dhT added at the last token)
 *   dk[t] = G[t] v[t],   dv[t] = G[t]^T k[t],   dh0 = a * G[0]
 *
 * dk and dv are summed over the heads that share them.  dq, dk and dv (NULL to
 * skip) are of `type`, dh0 [seqs][H][Dk][Dv] (NULL to skip) float32; the dh0
 * of a sequence of no token is its dhT.  The remarks on precision above hold
 * here with dy, v and k, or v, dy and q, or k, q and dy in the places of q, k
 * and v. */
int dwconv_attention_grad(const void *dy, long long lddy, const void *q, long long ldq,
                          const void *k, long long ldk, const void *v, long long ldv, int type,
                          const float *log_decay, float scale, const float *h0, const float *dhT,
                          void *dq, long long lddq, void *dk, long long lddk, void *dv,
                          long long lddv, float *dh0, void *workspace, long long workspace_bytes,
                          int seqs, long long tokens, const int *offsets, int H, int KV, int Dk,
                          int Dv, void *stream);

/* ---- group normalisation with an activation, channels last ------------------
 *
 * x is N instances of P positions (at least one) of C channels: row n * P + p holds
 * position p of instance n.  A group is C / groups adjacent channels of one instance;
 *
 *   y = act((x - mean) * rstd * w[c] + b[c]),    rstd = 1 / sqrt(var + eps)
 *
 * with the mean and the variance (divided by the number of elements) over a
 * group's channels and positions.  x and y are of `type`, in place if y == x
 * with the same stride; w and b [C] float32 (NULL: 1 and 0); stats (NULL to
 * skip) [N][groups][2] float32 receives mean and rstd, which the gradient
 * needs.  eps >= 0 and finite.  N = 0 is allowed.  workspace: at least
 * dwconv_norm_workspace_size(grad = 0) bytes, 16-byte aligned (NULL where that is
 * 0). */
int dwconv_norm_workspace_size(int grad, int type, long long N, long long P, int C, int groups,
                               long long *bytes);
int dwconv_norm_fwd(const void *x, long long ldx, int type, const float *w, const float *b,
                    float eps, int act, void *y, long long ldy, float *stats, void *workspace,
                    long long workspace_bytes, long long N, long long P, int C, int groups,
                    void *stream);

/* Gradients, from the statistics that the forward kept.  With xhat = (x - mean)
 * * rstd, z = xhat * w + b, dz = dy * act'(z) and g = dz * w,
 *
 *   dx = rstd * (g - mean(g) - xhat * mean(g * xhat))      means over the group
 *   dw[c] = sum dz * xhat,   db[c] = sum dz                over N and P
 *
 * act' is 0 at the corners of ReLU and ReLU6.  dx (of `type`; in place if it is
 * dy with the same stride), dw and db [C] float32: NULL to skip. */
int dwconv_norm_grad(const void *dy, long long lddy, const void *x, long long ldx, int type,
                     const float *w, const float *b, int act, const float *stats, void *dx,
                     long long lddx, float *dw, float *db, void *workspace,
                     long long workspace_bytes, long long N, long long P, int C, int groups,
                     void *stream);

/* ---- matrix product in 8-bit integers ----------------------------------------
 *
 * Quantised rows: scale[m] = max_k |x[m,k]| * (1 / 127), the factor and the
 * product rounded to float32, and at least 2^-126; q[m,k] = x[m,k] / scale[m]
 * rounded to the nearest integer, halves to even, within -127 .. 127.  A row
 * that holds an infinity or a NaN has the scale NaN and numbers of 0, so that
 * its products are NaN.  x is M rows of K of a float `type`, q M rows of K int8
 * (ldq elements apart), scale [M] float32.  M = 0 is allowed. */
#define DWCONV_T_I8 3

int dwconv_quantize_rows(const void *x, long long ldx, int type, void *q, long long ldq,
                         float *scale, long long M, int K, void *stream);

/*   y[m,n] = act(x_scale[m] * w_scale[n] * sum_k x[m,k] * w[n,k] + b[n]) + res[m,n]
 *
 * w is N rows of K int8, w_scale [N] float32; b [N] float32 or NULL; y and res
 * (NULL for none) M rows of N of `type`.  x is M rows of K int8 with x_scale [M]
 * (xtype = DWCONV_T_I8), or of `type` (xtype = type, x_scale = NULL), and then
 * quantised as above in the same call.  Integer sums are exact: K is at most
 * DWCONV_I8_MAX_K.  workspace: at least dwconv_linear_i8_workspace_size bytes,
 * 16-byte aligned (NULL where that is 0).  M = 0 is allowed.  Row strides are
 * below 2^21 elements. */
#define DWCONV_I8_MAX_K 131071

int dwconv_linear_i8_workspace_size(int xtype, int type, long long M, int N, int K,
                                    long long *bytes);
int dwconv_linear_i8(const void *x, long long ldx, int xtype, const float *x_scale,
                     const void *w, long long ldw, const float *w_scale, int type, const float *b,
                     int act, const void *res, long long ldres, void *y, long long ldy,
                     void *workspace, long long workspace_bytes, long long M, int N, int K,
                     void *stream);

/* The kernel of such a product, as dwconv_linear_describe does: `quantized` is
 * whether x is given in int8, `aligned` whether the addresses and row strides of
 * w (and of x, if given in int8) are multiples of 16.  A kernel that quantises x
 * itself has "quantized" in its name. */
int dwconv_linear_i8_describe(int quantized, int type, int aligned, long long M, int N, int K,
                              char *name, int name_len, int *splits);

#ifdef __cplusplus
}
#endif

#endif /* DWCONV_MIX_H */

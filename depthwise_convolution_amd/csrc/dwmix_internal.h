// dwmix_internal.h -- what the host code and the kernel files of the mixing
// operators share (include/dwconv_mix.h): argument records, the planning rules
// that also size workspaces, and the launchers.  Plain C++.
#pragma once

#include "dwseq_internal.h"

namespace dwmix {

using dwseq::Batch;
using dwseq::cdiv;

// ---- linear attention with a decay for each head ----
struct AttentionArgs {
    const void *q, *k, *v, *dy;
    const float *log_decay, *h0, *dhT;
    void *y, *dq, *dk, *dv, *workspace;
    float *hT, *h, *dh0;
    long long ldq, ldk, ldv, ldy, lddy, lddq, lddk, lddv;
    float scale;
    int type, H, KV, Dk, Dv;
    Batch batch;
};
long long attention_workspace(bool grad, const Batch &b, bool packed, int H, int KV, int Dk,
                              int Dv);
int launch_attention_fwd(const AttentionArgs &a, void *stream);
int launch_attention_step(const AttentionArgs &a, void *stream);
int launch_attention_grad(const AttentionArgs &a, void *stream);

// ---- group normalisation ----
struct NormArgs {
    const void *x, *dy;
    const float *w, *b, *stats_in;
    void *y, *dx, *workspace;
    float *stats, *dw, *db;
    long long ldx, ldy, lddy, lddx;
    long long N, P;
    float eps;
    int type, act, C, groups;
};
long long norm_workspace(bool grad, int type, long long N, long long P, int C, int groups);
int launch_norm_fwd(const NormArgs &a, void *stream);
int launch_norm_grad(const NormArgs &a, void *stream);

// ---- matrix product in 8-bit integers ----
struct QuantizeArgs {
    const void *x;
    signed char *q;
    float *scale;
    long long ldx, ldq;
    int type, M, K;
};
int launch_quantize(const QuantizeArgs &a, void *stream);

struct LinearI8Args {
    const void *x, *w, *res;
    const float *x_scale, *w_scale, *b;     // x_scale nullptr: x is to be quantised
    void *y, *workspace;
    long long ldx, ldw, ldres, ldy;
    int type, act, M, N, K;
};
long long linear_i8_workspace(bool quantized, int M, int N, int K);
void linear_i8_describe(bool quantized, bool aligned, int M, int N, int K, const char **name,
                        int *splits);
// Few rows that are quantised by the product's own launch: 64 elements a thread of 512.
inline bool few_rows_fit(int M, int K) { return M <= 16 && (long long)M * K <= 32768; }
int launch_linear_few(const LinearI8Args &a, void *stream);
int launch_linear_i8(const LinearI8Args &a, void *stream);

}  // namespace dwmix

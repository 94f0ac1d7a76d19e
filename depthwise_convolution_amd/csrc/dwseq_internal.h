// dwseq_internal.h -- what the host code and the kernel files of the sequence
// operators share (include/dwconv_seq.h): argument records, the planning
// rules that also size workspaces, and the launchers.  Plain C++.
#pragma once

#include <cstdint>

namespace dwseq {

// The sequences of a batch.  off = nullptr: seqs sequences of `tokens` rows;
// else a device array of seqs + 1 offsets into `rows` rows.
struct Batch {
    int seqs;
    int tokens;         // rows per sequence (dense)
    int rows;           // rows in all
    const int *off;
};

// ---- causal depthwise convolution ----
struct CausalArgs {
    const void *x, *w, *init, *dy, *dfinal;
    const float *b;
    void *y, *final_state, *state, *dx, *dinit;
    float *dw, *db, *part;
    long long ldx, ldy, lddy, lddx;
    int type, wtype, act, C, K;
    Batch batch;
};

// Rows of partial sums of dw and db: the row chunks of the gradient kernel.
struct CausalGradPlan {
    int chunk;          // tokens that one thread walks
    int blocks;         // rows of partial sums
};
CausalGradPlan causal_grad_plan(int rows, int C);
long long causal_grad_workspace(int rows, int C, int K);

int launch_causal_fwd(const CausalArgs &a, void *stream);
int launch_causal_step(const CausalArgs &a, void *stream);
int launch_causal_grad(const CausalArgs &a, void *stream);

// ---- gated linear recurrence ----
struct ScanArgs {
    const void *x, *r, *i, *dy;
    const float *lam, *h0, *dhT, *states_in;
    void *y, *dx, *dr, *di;
    float *hT, *states, *dlam, *dh0, *h;
    void *workspace;
    float *part;                // within the workspace
    long long ldx, ldr, ldi, ldy, lddy, lddx, lddr, lddi;
    float scale;
    int type, C;
    Batch batch;
};

long long scan_states(const Batch &b, int C);
long long scan_workspace(bool grad, const Batch &b, int C, bool packed);

int launch_scan_fwd(const ScanArgs &a, void *stream);
int launch_scan_step(const ScanArgs &a, void *stream);
int launch_scan_grad(const ScanArgs &a, void *stream);

// ---- matrix product with epilogue ----
struct LinearArgs {
    const void *x, *w, *res, *dy, *z_in;
    const float *b;
    void *y, *z, *dx, *dw;
    float *db;
    void *workspace;
    long long ldx, ldw, ldres, ldy, ldz, lddy, lddx, lddw;
    int type, act;
    int M, N, K;
};
long long linear_workspace(bool grad, int type, int act, int M, int N, int K);
void linear_describe(int product, int type, bool aligned, int M, int N, int K, const char **name,
                     int *splits);
int launch_linear_fwd(const LinearArgs &a, void *stream);
int launch_linear_grad(const LinearArgs &a, void *stream);

inline int elem_size(int type) { return type == 0 ? 4 : 2; }
inline long long cdiv(long long a, long long b) { return (a + b - 1) / b; }

}  // namespace dwseq

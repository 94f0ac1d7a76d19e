// dwmix_api.cpp -- the extern "C" entry points of the mixing operators
// (include/dwconv_mix.h).  Every argument is checked before anything is
// enqueued, as in dwseq_api.cpp.
#include "../../include/dwconv_mix.h"
#include "dwmix_internal.h"
#include "dwseq_check.h"

#include <cmath>
#include <cstdio>

using namespace dwmix;
using namespace dwseq;

namespace {

int check_attention(int type, int H, int KV, int Dk, int Dv)
{
    if (!type_ok(type))
        return DWCONV_ERR_BAD_WTYPE;
    if (H < 1 || H > (1 << 16) || KV < 1 || H % KV != 0 || Dk < 1 ||
        Dk > DWCONV_ATTENTION_MAX_DIM || Dv < 1 || Dv > DWCONV_ATTENTION_MAX_DIM)
        return DWCONV_ERR_BAD_DIM;
    return DWCONV_OK;
}

// The arrays of q, k and v, and what of them the record holds.
void take_qkv(Check &c, AttentionArgs &a, const void *q, long long ldq, const void *k,
              long long ldk, const void *v, long long ldv, long long rows)
{
    const long long e = elem_size(a.type);
    c.in(q, region(q, rows, ldq * e, e * a.H * a.Dk), (int)e);
    c.in(k, region(k, rows, ldk * e, e * a.KV * a.Dk), (int)e);
    c.in(v, region(v, rows, ldv * e, e * a.KV * a.Dv), (int)e);
    c.in(a.log_decay, dense(a.log_decay, 4LL * a.H), 4);
    if (!short_ld_ok(ldq, (long long)a.H * a.Dk) || !short_ld_ok(ldk, (long long)a.KV * a.Dk) ||
        !short_ld_ok(ldv, (long long)a.KV * a.Dv))
        c.fail(DWCONV_ERR_ROW_STRIDE);
    a.q = q; a.k = k; a.v = v; a.ldq = ldq; a.ldk = ldk; a.ldv = ldv;
}

int check_norm(int type, long long N, long long P, int C, int groups)
{
    if (!type_ok(type))
        return DWCONV_ERR_BAD_WTYPE;
    if (N < 0 || N > DWCONV_SEQ_MAX_ROWS || P < 1 || P > DWCONV_SEQ_MAX_ROWS ||
        N * P > DWCONV_SEQ_MAX_ROWS || C < 1 || C > DWCONV_SEQ_MAX_ROWS || groups < 1 ||
        C % groups != 0)
        return DWCONV_ERR_BAD_DIM;
    return DWCONV_OK;
}

}  // namespace

extern "C" {

int dwconv_attention_workspace_size(int grad, int type, int seqs, long long tokens, int packed,
                                    int H, int KV, int Dk, int Dv, long long *bytes)
{
    if (!bytes)
        return DWCONV_ERR_NULL_PTR;
    Batch b;
    int st = check_attention(type, H, KV, Dk, Dv);
    if (st == DWCONV_OK)
        st = make_batch(seqs, tokens, nullptr, packed != 0, &b);
    if (st != DWCONV_OK)
        return st;
    *bytes = attention_workspace(grad != 0, b, packed != 0, H, KV, Dk, Dv);
    return DWCONV_OK;
}

int dwconv_attention_fwd(const void *q, long long ldq, const void *k, long long ldk,
                         const void *v, long long ldv, int type, const float *log_decay,
                         float scale, const float *h0, void *y, long long ldy, float *hT,
                         void *workspace, long long workspace_bytes, int seqs, long long tokens,
                         const int *offsets, int H, int KV, int Dk, int Dv, void *stream)
{
    AttentionArgs a{};
    int st = check_attention(type, H, KV, Dk, Dv);
    if (st == DWCONV_OK)
        st = make_batch(seqs, tokens, offsets, offsets != nullptr, &a.batch);
    if (st != DWCONV_OK)
        return st;
    if (!std::isfinite(scale))
        return DWCONV_ERR_BAD_EPILOGUE;
    a.log_decay = log_decay; a.scale = scale; a.type = type; a.H = H; a.KV = KV; a.Dk = Dk;
    a.Dv = Dv;
    const long long e = elem_size(type), rows = a.batch.rows, states = 4LL * seqs * H * Dk * Dv;
    const long long need = attention_workspace(false, a.batch, offsets != nullptr, H, KV, Dk, Dv);
    if (!short_ld_ok(ldy, (long long)H * Dv))
        return DWCONV_ERR_ROW_STRIDE;
    Check c;
    take_qkv(c, a, q, ldq, k, ldk, v, ldv, rows);
    c.in(h0, dense(h0, states), 4, false);
    c.in(offsets, dense(offsets, 4LL * (seqs + 1LL)), 4, false);
    c.out(y, region(y, rows, ldy * e, e * H * Dv), (int)e);
    c.out(hT, dense(hT, states), 4, false);
    c.out(workspace, dense(workspace, need), 1, false);
    if (c.done() != DWCONV_OK)
        return c.status;
    st = check_workspace(workspace, workspace_bytes, need);
    if (st != DWCONV_OK)
        return st;
    a.h0 = h0; a.y = y; a.ldy = ldy; a.hT = hT; a.workspace = workspace;
    return launch_attention_fwd(a, stream);
}

int dwconv_attention_step(const void *q, long long ldq, const void *k, long long ldk,
                          const void *v, long long ldv, int type, const float *log_decay,
                          float scale, float *h, void *y, long long ldy, int seqs, int H, int KV,
                          int Dk, int Dv, void *stream)
{
    AttentionArgs a{};
    int st = check_attention(type, H, KV, Dk, Dv);
    if (st == DWCONV_OK)
        st = make_batch(seqs, 1, nullptr, false, &a.batch);
    if (st != DWCONV_OK)
        return st;
    if (!std::isfinite(scale))
        return DWCONV_ERR_BAD_EPILOGUE;
    a.log_decay = log_decay; a.scale = scale; a.type = type; a.H = H; a.KV = KV; a.Dk = Dk;
    a.Dv = Dv;
    const long long e = elem_size(type);
    if (!short_ld_ok(ldy, (long long)H * Dv))
        return DWCONV_ERR_ROW_STRIDE;
    Check c;
    take_qkv(c, a, q, ldq, k, ldk, v, ldv, seqs);
    c.out(y, region(y, seqs, ldy * e, e * H * Dv), (int)e);
    c.out(h, dense(h, 4LL * seqs * H * Dk * Dv), 4);
    if (c.done() != DWCONV_OK)
        return c.status;
    a.y = y; a.ldy = ldy; a.h = h;
    return launch_attention_step(a, stream);
}

int dwconv_attention_grad(const void *dy, long long lddy, const void *q, long long ldq,
                          const void *k, long long ldk, const void *v, long long ldv, int type,
                          const float *log_decay, float scale, const float *h0, const float *dhT,
                          void *dq, long long lddq, void *dk, long long lddk, void *dv,
                          long long lddv, float *dh0, void *workspace, long long workspace_bytes,
                          int seqs, long long tokens, const int *offsets, int H, int KV, int Dk,
                          int Dv, void *stream)
{
    AttentionArgs a{};
    int st = check_attention(type, H, KV, Dk, Dv);
    if (st == DWCONV_OK)
        st = make_batch(seqs, tokens, offsets, offsets != nullptr, &a.batch);
    if (st != DWCONV_OK)
        return st;
    if (!std::isfinite(scale))
        return DWCONV_ERR_BAD_EPILOGUE;
    a.log_decay = log_decay; a.scale = scale; a.type = type; a.H = H; a.KV = KV; a.Dk = Dk;
    a.Dv = Dv;
    const long long e = elem_size(type), rows = a.batch.rows, states = 4LL * seqs * H * Dk * Dv;
    const long long need = attention_workspace(true, a.batch, offsets != nullptr, H, KV, Dk, Dv);
    if (!short_ld_ok(lddy, (long long)H * Dv) ||
        (dq && !short_ld_ok(lddq, (long long)H * Dk)) ||
        (dk && !short_ld_ok(lddk, (long long)KV * Dk)) ||
        (dv && !short_ld_ok(lddv, (long long)KV * Dv)))
        return DWCONV_ERR_ROW_STRIDE;
    Check c;
    take_qkv(c, a, q, ldq, k, ldk, v, ldv, rows);
    c.in(dy, region(dy, rows, lddy * e, e * H * Dv), (int)e);
    c.in(h0, dense(h0, states), 4, false);
    c.in(dhT, dense(dhT, states), 4, false);
    c.in(offsets, dense(offsets, 4LL * (seqs + 1LL)), 4, false);
    c.out(dq, region(dq, rows, lddq * e, e * H * Dk), (int)e, false);
    c.out(dk, region(dk, rows, lddk * e, e * KV * Dk), (int)e, false);
    c.out(dv, region(dv, rows, lddv * e, e * KV * Dv), (int)e, false);
    c.out(dh0, dense(dh0, states), 4, false);
    c.out(workspace, dense(workspace, need), 1, false);
    if (c.done() != DWCONV_OK)
        return c.status;
    st = check_workspace(workspace, workspace_bytes, need);
    if (st != DWCONV_OK)
        return st;
    a.dy = dy; a.lddy = lddy; a.h0 = h0; a.dhT = dhT; a.dq = dq; a.lddq = lddq; a.dk = dk;
    a.lddk = lddk; a.dv = dv; a.lddv = lddv; a.dh0 = dh0; a.workspace = workspace;
    return launch_attention_grad(a, stream);
}

int dwconv_norm_workspace_size(int grad, int type, long long N, long long P, int C, int groups,
                               long long *bytes)
{
    if (!bytes)
        return DWCONV_ERR_NULL_PTR;
    const int st = check_norm(type, N, P, C, groups);
    if (st != DWCONV_OK)
        return st;
    *bytes = norm_workspace(grad != 0, type, N, P, C, groups);
    return DWCONV_OK;
}

int dwconv_norm_fwd(const void *x, long long ldx, int type, const float *w, const float *b,
                    float eps, int act, void *y, long long ldy, float *stats, void *workspace,
                    long long workspace_bytes, long long N, long long P, int C, int groups,
                    void *stream)
{
    const int st = check_norm(type, N, P, C, groups);
    if (st != DWCONV_OK)
        return st;
    if (!act_ok(act) || !(eps >= 0.0f) || !std::isfinite(eps))
        return DWCONV_ERR_BAD_EPILOGUE;
    if (!ld_ok(ldx, C) || !ld_ok(ldy, C))
        return DWCONV_ERR_ROW_STRIDE;
    const long long e = elem_size(type), rows = N * P, wide = C * e;
    const long long need = norm_workspace(false, type, N, P, C, groups);
    const bool in_place = y == x && ldy == ldx;
    Check c;
    if (in_place)
        c.check(x, region(x, rows, ldx * e, wide), (int)e);
    else
        c.in(x, region(x, rows, ldx * e, wide), (int)e);
    c.in(w, dense(w, 4LL * C), 4, false);
    c.in(b, dense(b, 4LL * C), 4, false);
    c.out(y, region(y, rows, ldy * e, wide), (int)e);
    c.out(stats, dense(stats, 8LL * N * groups), 4, false);
    c.out(workspace, dense(workspace, need), 1, false);
    if (c.done() != DWCONV_OK)
        return c.status;
    if (check_workspace(workspace, workspace_bytes, need) != DWCONV_OK)
        return DWCONV_ERR_WORKSPACE;
    NormArgs a{};
    a.x = x; a.w = w; a.b = b; a.y = y; a.stats = stats; a.workspace = workspace; a.ldx = ldx;
    a.ldy = ldy; a.N = N; a.P = P; a.eps = eps; a.type = type; a.act = act; a.C = C;
    a.groups = groups;
    return launch_norm_fwd(a, stream);
}

int dwconv_norm_grad(const void *dy, long long lddy, const void *x, long long ldx, int type,
                     const float *w, const float *b, int act, const float *stats, void *dx,
                     long long lddx, float *dw, float *db, void *workspace,
                     long long workspace_bytes, long long N, long long P, int C, int groups,
                     void *stream)
{
    const int st = check_norm(type, N, P, C, groups);
    if (st != DWCONV_OK)
        return st;
    if (!act_ok(act))
        return DWCONV_ERR_BAD_EPILOGUE;
    if (!ld_ok(lddy, C) || !ld_ok(ldx, C) || (dx && !ld_ok(lddx, C)))
        return DWCONV_ERR_ROW_STRIDE;
    const long long e = elem_size(type), rows = N * P, wide = C * e;
    const long long need = norm_workspace(true, type, N, P, C, groups);
    Check c;
    if (dx == dy && lddx == lddy)
        c.check(dy, region(dy, rows, lddy * e, wide), (int)e);
    else
        c.in(dy, region(dy, rows, lddy * e, wide), (int)e);
    c.in(x, region(x, rows, ldx * e, wide), (int)e);
    c.in(w, dense(w, 4LL * C), 4, false);
    c.in(b, dense(b, 4LL * C), 4, false);
    c.in(stats, region(stats, N, 8LL * groups, 8LL * groups), 4);
    c.out(dx, region(dx, rows, lddx * e, wide), (int)e, false);
    c.out(dw, dense(dw, 4LL * C), 4, false);
    c.out(db, dense(db, 4LL * C), 4, false);
    c.out(workspace, dense(workspace, need), 1, false);
    if (c.done() != DWCONV_OK)
        return c.status;
    if (check_workspace(workspace, workspace_bytes, need) != DWCONV_OK)
        return DWCONV_ERR_WORKSPACE;
    NormArgs a{};
    a.dy = dy; a.x = x; a.w = w; a.b = b; a.stats_in = stats; a.dx = dx; a.dw = dw; a.db = db;
    a.workspace = workspace; a.lddy = lddy; a.ldx = ldx; a.lddx = lddx; a.N = N; a.P = P;
    a.type = type; a.act = act; a.C = C; a.groups = groups;
    return launch_norm_grad(a, stream);
}

int dwconv_quantize_rows(const void *x, long long ldx, int type, void *q, long long ldq,
                         float *scale, long long M, int K, void *stream)
{
    if (!type_ok(type))
        return DWCONV_ERR_BAD_WTYPE;
    if (M < 0 || M > DWCONV_SEQ_MAX_ROWS || K < 1)
        return DWCONV_ERR_BAD_DIM;
    if (!ld_ok(ldx, K) || !ld_ok(ldq, K))
        return DWCONV_ERR_ROW_STRIDE;
    const long long e = elem_size(type);
    Check c;
    c.in(x, region(x, M, ldx * e, K * e), (int)e);
    c.out(q, region(q, M, ldq, K), 1);
    c.out(scale, region(scale, M, 4, 4), 4);
    if (c.done() != DWCONV_OK)
        return c.status;
    return launch_quantize({x, static_cast<signed char *>(q), scale, ldx, ldq, type, (int)M, K},
                           stream);
}

int dwconv_linear_i8_workspace_size(int xtype, int type, long long M, int N, int K,
                                    long long *bytes)
{
    if (!bytes)
        return DWCONV_ERR_NULL_PTR;
    if (!type_ok(type) || (xtype != DWCONV_T_I8 && xtype != type))
        return DWCONV_ERR_BAD_WTYPE;
    if (M < 0 || M > DWCONV_SEQ_MAX_ROWS || N < 1 || K < 1 || K > DWCONV_I8_MAX_K)
        return DWCONV_ERR_BAD_DIM;
    *bytes = linear_i8_workspace(xtype == DWCONV_T_I8, (int)M, N, K);
    return DWCONV_OK;
}

int dwconv_linear_i8_describe(int quantized, int type, int aligned, long long M, int N, int K,
                              char *name, int name_len, int *splits)
{
    long long bytes = 0;
    const int st = dwconv_linear_i8_workspace_size(quantized ? DWCONV_T_I8 : type, type, M, N, K,
                                                   &bytes);
    if (st != DWCONV_OK)
        return st;
    const char *kernel = "";
    int ranges = 0;
    linear_i8_describe(quantized != 0, aligned != 0, (int)M, N, K, &kernel, &ranges);
    if (name && name_len > 0)
        std::snprintf(name, (size_t)name_len, "%s", kernel);
    if (splits)
        *splits = ranges;
    return DWCONV_OK;
}

int dwconv_linear_i8(const void *x, long long ldx, int xtype, const float *x_scale,
                     const void *w, long long ldw, const float *w_scale, int type, const float *b,
                     int act, const void *res, long long ldres, void *y, long long ldy,
                     void *workspace, long long workspace_bytes, long long M, int N, int K,
                     void *stream)
{
    long long need = 0;
    const int st = dwconv_linear_i8_workspace_size(xtype, type, M, N, K, &need);
    if (st != DWCONV_OK)
        return st;
    if (!act_ok(act))
        return DWCONV_ERR_BAD_EPILOGUE;
    if (!short_ld_ok(ldx, K) || !short_ld_ok(ldw, K) || !short_ld_ok(ldy, N) ||
        (res && !short_ld_ok(ldres, N)))
        return DWCONV_ERR_ROW_STRIDE;
    const bool quantized = xtype == DWCONV_T_I8;
    const long long e = elem_size(type), xe = quantized ? 1 : e;
    Check c;
    c.in(x, region(x, M, ldx * xe, K * xe), (int)xe);
    if (quantized)
        c.in(x_scale, region(x_scale, M, 4, 4), 4);
    else if (x_scale)
        c.fail(DWCONV_ERR_BAD_WTYPE);       // scales of an x that is not quantised
    c.in(w, region(w, N, ldw, K), 1);
    c.in(w_scale, dense(w_scale, 4LL * N), 4);
    c.in(b, dense(b, 4LL * N), 4, false);
    c.in(res, region(res, M, ldres * e, N * e), (int)e, false);
    c.out(y, region(y, M, ldy * e, N * e), (int)e);
    c.out(workspace, dense(workspace, need), 1, false);
    if (c.done() != DWCONV_OK)
        return c.status;
    if (check_workspace(workspace, workspace_bytes, need) != DWCONV_OK)
        return DWCONV_ERR_WORKSPACE;
    LinearI8Args a{};
    a.x = x; a.w = w; a.res = res; a.x_scale = x_scale; a.w_scale = w_scale; a.b = b; a.y = y;
    a.workspace = workspace; a.ldx = ldx; a.ldw = ldw; a.ldres = ldres; a.ldy = ldy;
    a.type = type; a.act = act; a.M = (int)M; a.N = N; a.K = K;
    return launch_linear_i8(a, stream);
}

}  // extern "C"

// dwseq_api.cpp -- the extern "C" entry points of the sequence operators
// (include/dwconv_seq.h).  Every argument is checked before anything is
// enqueued, as in dwconv_api.cpp.
#include "../../include/dwconv_seq.h"
#include "dwseq_internal.h"

#include <cmath>
#include <cstdint>
#include <cstdio>

using namespace dwseq;

namespace {

// An array of `rows` rows of `width` bytes, `ld` bytes from row to row.
struct Region {
    std::uintptr_t base;
    long long rows, ld, width;
    bool empty() const { return base == 0 || rows <= 0 || width <= 0; }
    std::uintptr_t end() const
    {
        return base + static_cast<std::uintptr_t>((rows - 1) * ld + width);
    }
};

Region region(const void *p, long long rows, long long ld, long long width)
{
    return Region{reinterpret_cast<std::uintptr_t>(p), rows, ld, width};
}

Region dense(const void *p, long long bytes) { return region(p, 1, bytes, bytes); }

// Whether two arrays share a byte.  Column ranges of one wider array (equal
// row strides) are told apart; other arrays by their extent alone.
bool overlap(const Region &a, const Region &b)
{
    if (a.empty() || b.empty() || a.base >= b.end() || b.base >= a.end())
        return false;
    if (a.ld != b.ld || (a.rows == 1 && b.rows == 1))
        return true;
    const Region &lo = a.base <= b.base ? a : b, &hi = a.base <= b.base ? b : a;
    const long long d = static_cast<long long>((hi.base - lo.base) % lo.ld);
    return !(d >= lo.width && d + hi.width <= lo.ld);
}

bool aligned(const void *p, int to) { return (reinterpret_cast<std::uintptr_t>(p) % to) == 0; }

// Collects the arrays of a call and what is wrong with them.
class Check {
  public:
    int status = DWCONV_OK;

    void fail(int code)
    {
        if (status == DWCONV_OK)
            status = code;
    }
    // must: the pointer may not be NULL (when the array has any row)
    void in(const void *p, const Region &r, int align, bool must = true)
    {
        array(p, r, align, must);
        if (!r.empty() && n_in < kMost)
            ins[n_in++] = r;
    }
    void out(const void *p, const Region &r, int align, bool must = true)
    {
        array(p, r, align, must);
        if (r.empty())
            return;
        for (int k = 0; k < n_out; ++k)
            if (overlap(outs[k], r))
                clash = true;
        if (n_out < kMost)
            outs[n_out++] = r;
    }
    int done()
    {
        for (int o = 0; o < n_out; ++o)
            for (int k = 0; k < n_in; ++k)
                if (overlap(outs[o], ins[k]))
                    clash = true;
        if (clash)
            fail(DWCONV_ERR_ALIAS);
        return status;
    }

  private:
    static constexpr int kMost = 16;
    Region ins[kMost], outs[kMost];
    int n_in = 0, n_out = 0;
    bool clash = false;

    void array(const void *p, const Region &r, int align, bool must)
    {
        if (!p && must && r.rows > 0)
            fail(DWCONV_ERR_NULL_PTR);
        if (p && !aligned(p, align))
            fail(DWCONV_ERR_MISALIGNED);
    }
};

bool type_ok(int type) { return type >= DWCONV_T_F32 && type <= DWCONV_T_BF16; }
bool act_ok(int act) { return act >= DWCONV_ACT_NONE && act <= DWCONV_ACT_SILU; }

// Rows of a batch: DWCONV_OK and *b, or what is wrong.
int make_batch(int seqs, long long tokens, const int *offsets, bool packed, Batch *b)
{
    if (seqs < 1 || seqs > DWCONV_SEQ_MAX_ROWS || tokens < 0 || tokens > DWCONV_SEQ_MAX_ROWS)
        return DWCONV_ERR_BAD_DIM;
    const long long rows = packed ? tokens : tokens * seqs;
    if (rows > DWCONV_SEQ_MAX_ROWS)
        return DWCONV_ERR_BAD_DIM;
    if (offsets && !aligned(offsets, 4))
        return DWCONV_ERR_MISALIGNED;
    b->seqs = seqs;
    b->rows = (int)rows;
    b->tokens = packed ? 0 : (int)tokens;
    b->off = offsets;
    return DWCONV_OK;
}

// Row strides may pass 2^31 elements, not the address space.
bool ld_ok(long long ld, long long width) { return ld >= width && ld < (1LL << 40); }

// The recurrence and the products address a tile's rows by 32-bit offsets.
bool short_ld_ok(long long ld, long long width) { return ld >= width && ld < (1LL << 21); }

int check_workspace(const void *ws, long long have, long long need)
{
    if (need > 0 && (!ws || !aligned(ws, 16) || have < need))
        return DWCONV_ERR_WORKSPACE;
    return DWCONV_OK;
}

int check_causal(int type, int wtype, int act, int C, int K)
{
    if (!type_ok(type) || !type_ok(wtype))
        return DWCONV_ERR_BAD_WTYPE;
    if (!act_ok(act))
        return DWCONV_ERR_BAD_EPILOGUE;
    if (C < 1 || C > DWCONV_SEQ_MAX_ROWS || K < 1 || K > DWCONV_CAUSAL_MAX_TAPS)
        return DWCONV_ERR_BAD_DIM;
    return DWCONV_OK;
}

}  // namespace

extern "C" {

int dwconv_causal_fwd(const void *x, long long ldx, int type, const void *w, int wtype,
                      const float *b, int act, const void *init, void *y, long long ldy,
                      void *final_state, int seqs, long long tokens, const int *offsets, int C,
                      int K, void *stream)
{
    CausalArgs a{};
    int st = check_causal(type, wtype, act, C, K);
    if (st == DWCONV_OK)
        st = make_batch(seqs, tokens, offsets, offsets != nullptr, &a.batch);
    if (st != DWCONV_OK)
        return st;
    if (!ld_ok(ldx, C) || !ld_ok(ldy, C))
        return DWCONV_ERR_ROW_STRIDE;
    const long long e = elem_size(type), we = elem_size(wtype), rows = a.batch.rows;
    const long long carried = e * seqs * (K - 1) * C;
    Check c;
    c.in(x, region(x, rows, ldx * e, C * e), (int)e);
    c.in(w, dense(w, we * C * K), (int)we);
    c.in(b, dense(b, 4LL * C), 4, false);
    c.in(init, dense(init, carried), (int)e, false);
    c.in(offsets, dense(offsets, 4LL * (seqs + 1LL)), 4, false);
    c.out(y, region(y, rows, ldy * e, C * e), (int)e);
    c.out(final_state, dense(final_state, carried), (int)e, false);
    if (c.done() != DWCONV_OK)
        return c.status;
    a.x = x; a.w = w; a.b = b; a.init = init; a.y = y; a.final_state = final_state;
    a.ldx = ldx; a.ldy = ldy; a.type = type; a.wtype = wtype; a.act = act; a.C = C; a.K = K;
    return launch_causal_fwd(a, stream);
}

int dwconv_causal_step(const void *x, long long ldx, int type, const void *w, int wtype,
                       const float *b, int act, void *state, void *y, long long ldy, int seqs,
                       int C, int K, void *stream)
{
    CausalArgs a{};
    int st = check_causal(type, wtype, act, C, K);
    if (st == DWCONV_OK)
        st = make_batch(seqs, 1, nullptr, false, &a.batch);
    if (st != DWCONV_OK)
        return st;
    if (!ld_ok(ldx, C) || !ld_ok(ldy, C))
        return DWCONV_ERR_ROW_STRIDE;
    const long long e = elem_size(type), we = elem_size(wtype);
    Check c;
    c.in(x, region(x, seqs, ldx * e, C * e), (int)e);
    c.in(w, dense(w, we * C * K), (int)we);
    c.in(b, dense(b, 4LL * C), 4, false);
    c.out(y, region(y, seqs, ldy * e, C * e), (int)e);
    c.out(state, dense(state, e * seqs * (K - 1) * C), (int)e, K > 1);
    if (c.done() != DWCONV_OK)
        return c.status;
    a.x = x; a.w = w; a.b = b; a.state = state; a.y = y;
    a.ldx = ldx; a.ldy = ldy; a.type = type; a.wtype = wtype; a.act = act; a.C = C; a.K = K;
    return launch_causal_step(a, stream);
}

int dwconv_causal_grad_workspace_size(int seqs, long long tokens, int packed, int C, int K,
                                      long long *bytes)
{
    if (!bytes)
        return DWCONV_ERR_NULL_PTR;
    Batch b;
    int st = check_causal(DWCONV_T_F32, DWCONV_T_F32, DWCONV_ACT_NONE, C, K);
    if (st == DWCONV_OK)
        st = make_batch(seqs, tokens, nullptr, packed != 0, &b);
    if (st != DWCONV_OK)
        return st;
    *bytes = causal_grad_workspace(b.rows, C, K);
    return DWCONV_OK;
}

int dwconv_causal_grad(const void *dy, long long lddy, const void *x, long long ldx, int type,
                       const void *w, int wtype, const float *b, int act, const void *init,
                       const void *dfinal, void *dx, long long lddx, float *dw, float *db,
                       void *dinit, void *workspace, long long workspace_bytes, int seqs,
                       long long tokens, const int *offsets, int C, int K, void *stream)
{
    CausalArgs a{};
    int st = check_causal(type, wtype, act, C, K);
    if (st == DWCONV_OK)
        st = make_batch(seqs, tokens, offsets, offsets != nullptr, &a.batch);
    if (st != DWCONV_OK)
        return st;
    if (!ld_ok(ldx, C) || !ld_ok(lddy, C) || !ld_ok(lddx, C))
        return DWCONV_ERR_ROW_STRIDE;
    const long long e = elem_size(type), we = elem_size(wtype), rows = a.batch.rows;
    const long long carried = e * seqs * (K - 1) * C;
    const long long need = causal_grad_workspace(a.batch.rows, C, K);
    Check c;
    c.in(dy, region(dy, rows, lddy * e, C * e), (int)e);
    c.in(x, region(x, rows, ldx * e, C * e), (int)e);
    c.in(w, dense(w, we * C * K), (int)we);
    c.in(b, dense(b, 4LL * C), 4, false);
    c.in(init, dense(init, carried), (int)e, false);
    c.in(dfinal, dense(dfinal, carried), (int)e, false);
    c.in(offsets, dense(offsets, 4LL * (seqs + 1LL)), 4, false);
    c.out(dx, region(dx, rows, lddx * e, C * e), (int)e);
    c.out(dw, dense(dw, 4LL * C * K), 4);
    c.out(db, dense(db, 4LL * C), 4, false);
    c.out(dinit, dense(dinit, carried), (int)e, false);
    c.out(workspace, dense(workspace, need), 1, false);
    if (c.done() != DWCONV_OK)
        return c.status;
    st = check_workspace(workspace, workspace_bytes, need);
    if (st != DWCONV_OK)
        return st;
    a.dy = dy; a.x = x; a.w = w; a.b = b; a.init = init; a.dfinal = dfinal; a.dx = dx;
    a.dw = dw; a.db = db; a.dinit = dinit; a.part = static_cast<float *>(workspace);
    a.lddy = lddy; a.ldx = ldx; a.lddx = lddx; a.type = type; a.wtype = wtype; a.act = act;
    a.C = C; a.K = K;
    return launch_causal_grad(a, stream);
}

int dwconv_scan_states_size(int seqs, long long tokens, int packed, int C, long long *floats)
{
    if (!floats)
        return DWCONV_ERR_NULL_PTR;
    Batch b;
    const int st = C < 1 ? DWCONV_ERR_BAD_DIM : make_batch(seqs, tokens, nullptr, packed != 0, &b);
    if (st != DWCONV_OK)
        return st;
    *floats = scan_states(b, C);
    return DWCONV_OK;
}

int dwconv_scan_workspace_size(int grad, int seqs, long long tokens, int packed, int C,
                               long long *bytes)
{
    if (!bytes)
        return DWCONV_ERR_NULL_PTR;
    Batch b;
    const int st = C < 1 ? DWCONV_ERR_BAD_DIM : make_batch(seqs, tokens, nullptr, packed != 0, &b);
    if (st != DWCONV_OK)
        return st;
    *bytes = scan_workspace(grad != 0, b, C, packed != 0);
    return DWCONV_OK;
}

int dwconv_scan_fwd(const void *x, long long ldx, const void *r, long long ldr, const void *i,
                    long long ldi, int type, const float *lam, float scale, const float *h0,
                    void *y, long long ldy, float *hT, float *states, void *workspace,
                    long long workspace_bytes, int seqs, long long tokens, const int *offsets,
                    int C, void *stream)
{
    ScanArgs a{};
    if (!type_ok(type))
        return DWCONV_ERR_BAD_WTYPE;
    if (C < 1)
        return DWCONV_ERR_BAD_DIM;
    int st = make_batch(seqs, tokens, offsets, offsets != nullptr, &a.batch);
    if (st != DWCONV_OK)
        return st;
    if (!(scale > 0.0f) || !std::isfinite(scale))
        return DWCONV_ERR_BAD_EPILOGUE;
    if (!short_ld_ok(ldx, C) || !short_ld_ok(ldr, C) || !short_ld_ok(ldi, C) ||
        !short_ld_ok(ldy, C))
        return DWCONV_ERR_ROW_STRIDE;
    const long long e = elem_size(type), rows = a.batch.rows, w = C * e;
    const long long need = scan_workspace(false, a.batch, C, offsets != nullptr);
    Check c;
    c.in(x, region(x, rows, ldx * e, w), (int)e);
    c.in(r, region(r, rows, ldr * e, w), (int)e);
    c.in(i, region(i, rows, ldi * e, w), (int)e);
    c.in(lam, dense(lam, 4LL * C), 4);
    c.in(h0, dense(h0, 4LL * seqs * C), 4, false);
    c.in(offsets, dense(offsets, 4LL * (seqs + 1LL)), 4, false);
    c.out(y, region(y, rows, ldy * e, w), (int)e);
    c.out(hT, dense(hT, 4LL * seqs * C), 4, false);
    c.out(states, dense(states, 4LL * scan_states(a.batch, C)), 4, false);
    c.out(workspace, dense(workspace, need), 1, false);
    if (c.done() != DWCONV_OK)
        return c.status;
    st = check_workspace(workspace, workspace_bytes, need);
    if (st != DWCONV_OK)
        return st;
    a.x = x; a.r = r; a.i = i; a.lam = lam; a.scale = scale; a.h0 = h0; a.y = y; a.hT = hT;
    a.states = states; a.workspace = workspace;
    a.ldx = ldx; a.ldr = ldr; a.ldi = ldi; a.ldy = ldy; a.type = type; a.C = C;
    return launch_scan_fwd(a, stream);
}

int dwconv_scan_step(const void *x, long long ldx, const void *r, long long ldr, const void *i,
                     long long ldi, int type, const float *lam, float scale, float *h, void *y,
                     long long ldy, int seqs, int C, void *stream)
{
    ScanArgs a{};
    if (!type_ok(type))
        return DWCONV_ERR_BAD_WTYPE;
    if (C < 1)
        return DWCONV_ERR_BAD_DIM;
    const int st = make_batch(seqs, 1, nullptr, false, &a.batch);
    if (st != DWCONV_OK)
        return st;
    if (!(scale > 0.0f) || !std::isfinite(scale))
        return DWCONV_ERR_BAD_EPILOGUE;
    if (!short_ld_ok(ldx, C) || !short_ld_ok(ldr, C) || !short_ld_ok(ldi, C) ||
        !short_ld_ok(ldy, C))
        return DWCONV_ERR_ROW_STRIDE;
    const long long e = elem_size(type), w = C * e;
    Check c;
    c.in(x, region(x, seqs, ldx * e, w), (int)e);
    c.in(r, region(r, seqs, ldr * e, w), (int)e);
    c.in(i, region(i, seqs, ldi * e, w), (int)e);
    c.in(lam, dense(lam, 4LL * C), 4);
    c.out(y, region(y, seqs, ldy * e, w), (int)e);
    c.out(h, dense(h, 4LL * seqs * C), 4);
    if (c.done() != DWCONV_OK)
        return c.status;
    a.x = x; a.r = r; a.i = i; a.lam = lam; a.scale = scale; a.h = h; a.y = y;
    a.ldx = ldx; a.ldr = ldr; a.ldi = ldi; a.ldy = ldy; a.type = type; a.C = C;
    return launch_scan_step(a, stream);
}

int dwconv_scan_grad(const void *dy, long long lddy, const void *x, long long ldx, const void *r,
                     long long ldr, const void *i, long long ldi, int type, const float *lam,
                     float scale, const float *states, const float *dhT, void *dx,
                     long long lddx, void *dr, long long lddr, void *di, long long lddi,
                     float *dlam, float *dh0, void *workspace, long long workspace_bytes,
                     int seqs, long long tokens, const int *offsets, int C, void *stream)
{
    ScanArgs a{};
    if (!type_ok(type))
        return DWCONV_ERR_BAD_WTYPE;
    if (C < 1)
        return DWCONV_ERR_BAD_DIM;
    int st = make_batch(seqs, tokens, offsets, offsets != nullptr, &a.batch);
    if (st != DWCONV_OK)
        return st;
    if (!(scale > 0.0f) || !std::isfinite(scale))
        return DWCONV_ERR_BAD_EPILOGUE;
    if (!short_ld_ok(lddy, C) || !short_ld_ok(ldx, C) || !short_ld_ok(ldr, C) ||
        !short_ld_ok(ldi, C) ||
        !short_ld_ok(lddx, C) || !short_ld_ok(lddr, C) || !short_ld_ok(lddi, C))
        return DWCONV_ERR_ROW_STRIDE;
    const long long e = elem_size(type), rows = a.batch.rows, w = C * e;
    const long long need = scan_workspace(true, a.batch, C, offsets != nullptr);
    Check c;
    c.in(dy, region(dy, rows, lddy * e, w), (int)e);
    c.in(x, region(x, rows, ldx * e, w), (int)e);
    c.in(r, region(r, rows, ldr * e, w), (int)e);
    c.in(i, region(i, rows, ldi * e, w), (int)e);
    c.in(lam, dense(lam, 4LL * C), 4);
    c.in(states, region(states, rows > 0, 4LL * scan_states(a.batch, C),
                        4LL * scan_states(a.batch, C)), 4);
    c.in(dhT, dense(dhT, 4LL * seqs * C), 4, false);
    c.in(offsets, dense(offsets, 4LL * (seqs + 1LL)), 4, false);
    c.out(dx, region(dx, rows, lddx * e, w), (int)e);
    c.out(dr, region(dr, rows, lddr * e, w), (int)e);
    c.out(di, region(di, rows, lddi * e, w), (int)e);
    c.out(dlam, dense(dlam, 4LL * C), 4);
    c.out(dh0, dense(dh0, 4LL * seqs * C), 4, false);
    c.out(workspace, dense(workspace, need), 1, false);
    if (c.done() != DWCONV_OK)
        return c.status;
    st = check_workspace(workspace, workspace_bytes, need);
    if (st != DWCONV_OK)
        return st;
    a.dy = dy; a.x = x; a.r = r; a.i = i; a.lam = lam; a.scale = scale; a.states_in = states;
    a.dhT = dhT; a.dx = dx; a.dr = dr; a.di = di; a.dlam = dlam; a.dh0 = dh0;
    a.workspace = workspace;
    a.lddy = lddy; a.ldx = ldx; a.ldr = ldr; a.ldi = ldi; a.lddx = lddx; a.lddr = lddr;
    a.lddi = lddi; a.type = type; a.C = C;
    return launch_scan_grad(a, stream);
}

int dwconv_linear_workspace_size(int grad, int type, int act, long long M, int N, int K,
                                 long long *bytes)
{
    if (!bytes)
        return DWCONV_ERR_NULL_PTR;
    if (!type_ok(type))
        return DWCONV_ERR_BAD_WTYPE;
    if (!act_ok(act))
        return DWCONV_ERR_BAD_EPILOGUE;
    if (M < 0 || M > DWCONV_SEQ_MAX_ROWS || N < 1 || K < 1)
        return DWCONV_ERR_BAD_DIM;
    *bytes = linear_workspace(grad != 0, type, act, (int)M, N, K);
    return DWCONV_OK;
}

int dwconv_linear_describe(int product, int type, int aligned, long long M, int N, int K,
                           char *name, int name_len, int *splits)
{
    if (product < DWCONV_LINEAR_Y || product > DWCONV_LINEAR_DW)
        return DWCONV_ERR_BAD_OP;
    long long bytes = 0;
    const int st = dwconv_linear_workspace_size(1, type, DWCONV_ACT_NONE, M, N, K, &bytes);
    if (st != DWCONV_OK)
        return st;
    const char *kernel = "";
    int ranges = 0;
    linear_describe(product, type, aligned != 0, (int)M, N, K, &kernel, &ranges);
    if (name && name_len > 0)
        std::snprintf(name, (size_t)name_len, "%s", kernel);
    if (splits)
        *splits = ranges;
    return DWCONV_OK;
}

int dwconv_linear_fwd(const void *x, long long ldx, const void *w, long long ldw, int type,
                      const float *b, int act, const void *res, long long ldres, void *y,
                      long long ldy, void *z, long long ldz, void *workspace,
                      long long workspace_bytes, long long M, int N, int K, void *stream)
{
    long long need = 0;
    const int st = dwconv_linear_workspace_size(0, type, act, M, N, K, &need);
    if (st != DWCONV_OK)
        return st;
    if (!short_ld_ok(ldx, K) || !short_ld_ok(ldw, K) || !short_ld_ok(ldy, N) ||
        (res && !short_ld_ok(ldres, N)) || (z && !short_ld_ok(ldz, N)))
        return DWCONV_ERR_ROW_STRIDE;
    const long long e = elem_size(type);
    Check c;
    c.in(x, region(x, M, ldx * e, K * e), (int)e);
    c.in(w, region(w, N, ldw * e, K * e), (int)e);
    c.in(b, dense(b, 4LL * N), 4, false);
    c.in(res, region(res, M, ldres * e, N * e), (int)e, false);
    c.out(y, region(y, M, ldy * e, N * e), (int)e);
    c.out(z, region(z, M, ldz * e, N * e), (int)e, false);
    c.out(workspace, dense(workspace, need), 1, false);
    if (c.done() != DWCONV_OK)
        return c.status;
    if (check_workspace(workspace, workspace_bytes, need) != DWCONV_OK)
        return DWCONV_ERR_WORKSPACE;
    if (M == 0)
        return DWCONV_OK;
    LinearArgs a{};
    a.x = x; a.w = w; a.b = b; a.res = res; a.y = y; a.z = z; a.workspace = workspace;
    a.ldx = ldx; a.ldw = ldw; a.ldres = ldres; a.ldy = ldy; a.ldz = ldz;
    a.type = type; a.act = act; a.M = (int)M; a.N = N; a.K = K;
    return launch_linear_fwd(a, stream);
}

int dwconv_linear_grad(const void *dy, long long lddy, const void *x, long long ldx,
                       const void *w, long long ldw, int type, int act, const void *z,
                       long long ldz, void *dx, long long lddx, void *dw, long long lddw,
                       float *db, void *workspace, long long workspace_bytes, long long M, int N,
                       int K, void *stream)
{
    long long need = 0;
    const int st = dwconv_linear_workspace_size(1, type, act, M, N, K, &need);
    if (st != DWCONV_OK)
        return st;
    const bool has_z = act != DWCONV_ACT_NONE;
    if (!short_ld_ok(lddy, N) || !short_ld_ok(ldx, K) || !short_ld_ok(ldw, K) ||
        (has_z && !short_ld_ok(ldz, N)) || (dx && !short_ld_ok(lddx, K)) ||
        (dw && !short_ld_ok(lddw, K)))
        return DWCONV_ERR_ROW_STRIDE;
    const long long e = elem_size(type);
    Check c;
    c.in(dy, region(dy, M, lddy * e, N * e), (int)e);
    c.in(x, region(x, M, ldx * e, K * e), (int)e, dw != nullptr);
    c.in(w, region(w, N, ldw * e, K * e), (int)e, dx != nullptr);
    if (has_z)
        c.in(z, region(z, M, ldz * e, N * e), (int)e);
    c.out(dx, region(dx, M, lddx * e, K * e), (int)e, false);
    c.out(dw, region(dw, N, lddw * e, K * e), (int)e, false);
    c.out(db, dense(db, 4LL * N), 4, false);
    c.out(workspace, dense(workspace, need), 1, false);
    if (c.done() != DWCONV_OK)
        return c.status;
    if (check_workspace(workspace, workspace_bytes, need) != DWCONV_OK)
        return DWCONV_ERR_WORKSPACE;
    LinearArgs a{};
    a.dy = dy; a.x = x; a.w = w; a.z_in = z; a.dx = dx; a.dw = dw; a.db = db;
    a.workspace = workspace;
    a.lddy = lddy; a.ldx = ldx; a.ldw = ldw; a.ldz = ldz; a.lddx = lddx; a.lddw = lddw;
    a.type = type; a.act = act; a.M = (int)M; a.N = N; a.K = K;
    return launch_linear_grad(a, stream);
}

}  // extern "C"

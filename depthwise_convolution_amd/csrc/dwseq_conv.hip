// dwseq_conv.hip -- causal depthwise convolution over tokens: forward, the
// single-token step and the gradients (include/dwconv_seq.h).
//
// One filter per channel and no sum over channels, so the work is a few
// multiply-adds per element read: bound by HBM.  A thread holds V adjacent
// channels (4; 2 in the gradient) and walks a chunk of tokens with the last
// K-1 rows in registers, so a row is read once per chunk, plus K-1
// rows before it that the neighbouring chunk has read too.  Rows of other
// sequences are never used in arithmetic (they may hold NaN): near the start
// of a sequence each tap is taken from the carried rows or as zero.
//
// Measured, with inputs from HBM (a large copy: 6.3 TB/s): forward, 8 x 4096 x 2048
// bfloat16, 4 taps and SiLU, 60 us (4.5 TB/s); 20011 x 1000 float32 in 37 sequences
// 38 us (4.2 TB/s); gradient, 16411 x 1536 float16 in 23 sequences, 43.5 us with its
// sums (3.5 TB/s); 8 x 4096 x 2048 96 us and 5 for the sums in bfloat16 (4.2 TB/s, the
// vector unit active 70% of the time), 175 in float32 (4.6 TB/s); single tokens, 64 x
// 2048, 3 us, a launch.  With the same tensors call after call, 4 channels a thread in the
// forward took 55 us where 8 took 67 (fewer waves); in the gradient 2 took 116 where 4
// took 145 (8 x 4096 x 2048; registers).
#include "dwseq_device.h"

namespace dwseq {
namespace {

constexpr int kThreads = 256;
constexpr int kAhead = 4;       // rows loaded before the first of them is used
constexpr int kGradAhead = 4;   // and in the gradient, which holds the next ones too

// w[c0 .. c0+V) of [C][K], as taps of a channel vector
template <int V, int K>
__device__ __forceinline__ void load_taps(const void *w, int wtype, int c0, float (&f)[K][V])
{
    auto take = [&](auto *p) {
        using T = std::remove_cv_t<std::remove_pointer_t<decltype(p)>>;
        float flat[V * K];
        load<T, V * K>(p + (long long)c0 * K, flat);
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int j = 0; j < K; ++j)
                f[j][v] = flat[v * K + j];
    };
    if (wtype == DWCONV_T_F32)
        take(static_cast<const float *>(w));
    else if (wtype == DWCONV_T_F16)
        take(static_cast<const f16 *>(w));
    else
        take(static_cast<const bf16 *>(w));
}

template <int V>
__device__ __forceinline__ void load_bias(const float *b, int c0, float (&f)[V])
{
#pragma unroll
    for (int v = 0; v < V; ++v)
        f[v] = 0.0f;
    if (b)
        load<float, V>(b + c0, f);
}

// The row `back` rows before the start-th + pos row of sequence s, whose
// start it may precede: a carried row, or zero.
template <typename T, int V>
__device__ __forceinline__ void carried_row(const T *init, int s, int row, int K, int C, int c0,
                                            float (&f)[V])
{
#pragma unroll
    for (int v = 0; v < V; ++v)
        f[v] = 0.0f;
    if (init)
        load<T, V>(init + ((long long)s * (K - 1) + row) * C + c0, f);
}

// A channel vector's first channel: the last vector of a row that V does not
// divide is moved back to end with it (both threads write the same values).
template <int V> __device__ __forceinline__ int first_channel(int group, int C)
{
    return min(group * V, C - V);
}

// Where a walk over rows is: the sequence of the row at hand.
struct Walk {
    int s, start, end;
    __device__ __forceinline__ Walk(const Batch &b, int t)
    {
        s = seq_of(b, t);
        start = min(seq_start(b, s), t);
        end = seq_start(b, s + 1);
    }
    __device__ __forceinline__ void to(const Batch &b, int t)
    {
        while (t >= end && s + 1 < b.seqs) {
            ++s;
            start = min(seq_start(b, s), t);
            end = seq_start(b, s + 1);
        }
    }
};

// ---------------------------------------------------------------------------
// Forward.  The first `main_blocks` workgroups compute y; the others copy the
// rows that a continuation carries.
// ---------------------------------------------------------------------------
template <typename T, int V, int K>
__global__ __launch_bounds__(kThreads) void k_causal_fwd(CausalArgs a, int groups, int chunk,
                                                         int chunks, int main_blocks)
{
    const T *x = static_cast<const T *>(a.x);
    const T *init = static_cast<const T *>(a.init);
    if (block_id() >= (unsigned)main_blocks) {
        long long id = (long long)(block_id() - main_blocks) * kThreads + threadIdx.x;
        const int c0 = first_channel<V>((int)(id % groups), a.C);
        id /= groups;
        if (K == 1 || !a.final_state || id >= (long long)a.batch.seqs * (K - 1))
            return;
        const int s = (int)(id / max(K - 1, 1)), j = (int)(id % max(K - 1, 1));
        const int start = seq_start(a.batch, s);
        const int at = max(seq_start(a.batch, s + 1) - start, 0) - (K - 1) + j;
        float f[V];
        if (at >= 0)
            load<T, V>(x + (long long)(start + at) * a.ldx + c0, f);
        else
            carried_row<T, V>(init, s, at + K - 1, K, a.C, c0, f);
        store<T, V>(static_cast<T *>(a.final_state) + id * a.C + c0, f);
        return;
    }
    const unsigned id = block_id() * kThreads + threadIdx.x;
    const unsigned ck = id / (unsigned)groups;
    if (ck >= (unsigned)chunks)
        return;
    const int c0 = first_channel<V>((int)(id - ck * (unsigned)groups), a.C);
    // (rows are at most 2^31 - 2^16, and chunks of 2^16 would take 2^47 elements;
    // t0 + min(chunk, rows - t0) took 64.4 us where this takes 60.0, 8 x 4096 x 2048
    // bfloat16)
    const int t0 = (int)ck * chunk, t1 = min((int)ck * chunk + chunk, a.batch.rows);
    float w[K][V], b[V], ext[K - 1 + kAhead][V];
    load_taps<V, K>(a.w, a.wtype, c0, w);
    load_bias<V>(a.b, c0, b);
    x += c0;
    T *y = static_cast<T *>(a.y) + c0;
#pragma unroll
    for (int j = 0; j < K - 1; ++j) {
#pragma unroll
        for (int v = 0; v < V; ++v)
            ext[j][v] = 0.0f;
        if (t0 - (K - 1) + j >= 0)
            load<T, V>(x + (long long)(t0 - (K - 1) + j) * a.ldx, ext[j]);
    }
    Walk at(a.batch, t0);
    for (int t = t0; t < t1; t += kAhead) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            load<T, V>(x + (long long)min(t + u, t1 - 1) * a.ldx, ext[K - 1 + u]);
        at.to(a.batch, t);
        const bool inside = t - at.start >= K - 1 && t + kAhead <= at.end;
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            float z[V];
#pragma unroll
            for (int v = 0; v < V; ++v)
                z[v] = b[v];
            if (inside) {
#pragma unroll
                for (int j = 0; j < K; ++j)
#pragma unroll
                    for (int v = 0; v < V; ++v)
                        z[v] = fmaf(w[j][v], ext[u + j][v], z[v]);
            } else if (t + u < t1) {
                at.to(a.batch, t + u);
                const int pos = t + u - at.start;
#pragma unroll
                for (int j = 0; j < K; ++j) {
                    float row[V];
                    if (pos >= K - 1 - j) {
#pragma unroll
                        for (int v = 0; v < V; ++v)
                            row[v] = ext[u + j][v];
                    } else {
                        carried_row<T, V>(init, at.s, pos + j, K, a.C, c0, row);
                    }
#pragma unroll
                    for (int v = 0; v < V; ++v)
                        z[v] = fmaf(w[j][v], row[v], z[v]);
                }
            }
            act_all(z, a.act);
            if (t + u < t1)
                store<T, V>(y + (long long)(t + u) * a.ldy, z);
        }
#pragma unroll
        for (int j = 0; j < K - 1; ++j)
#pragma unroll
            for (int v = 0; v < V; ++v)
                ext[j][v] = ext[j + kAhead][v];
    }
}

// ---------------------------------------------------------------------------
// One token per sequence: a thread reads a channel vector's K-1 carried rows
// and its new one, and writes the rows back one place on.  Vectors do not
// overlap here (the rows are updated in place): the channels that V does not
// divide are taken one by one.
// ---------------------------------------------------------------------------
template <typename T, int V, int K>
__device__ __forceinline__ void step_vector(const CausalArgs &a, int s, int c0)
{
    float w[K][V], z[V], row[V], next[V];
    load_taps<V, K>(a.w, a.wtype, c0, w);
    load_bias<V>(a.b, c0, z);
    T *state = static_cast<T *>(a.state) + (long long)s * (K - 1) * a.C + c0;
    load<T, V>(static_cast<const T *>(a.x) + s * a.ldx + c0, next);
    float rows[K > 1 ? K - 1 : 1][V];
#pragma unroll
    for (int j = 0; j < K - 1; ++j)
        load<T, V>(state + (long long)j * a.C, rows[j]);
#pragma unroll
    for (int j = 0; j < K; ++j) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            row[v] = j < K - 1 ? rows[j][v] : next[v];
            z[v] = fmaf(w[j][v], row[v], z[v]);
        }
        if (j > 0)
            store<T, V>(state + (long long)(j - 1) * a.C, row);
    }
    act_all(z, a.act);
    store<T, V>(static_cast<T *>(a.y) + s * a.ldy + c0, z);
}

template <typename T, int V, int K>
__global__ __launch_bounds__(kThreads) void k_causal_step(CausalArgs a, int groups)
{
    const long long id = (long long)block_id() * kThreads + threadIdx.x;
    if (id >= (long long)a.batch.seqs * groups)
        return;
    const int s = (int)(id / groups), c0 = (int)(id % groups) * V;
    if (c0 + V <= a.C)
        step_vector<T, V, K>(a, s, c0);
    else
        for (int c = c0; c < a.C; ++c)
            step_vector<T, 1, K>(a, s, c);
}

// ---------------------------------------------------------------------------
// Gradients.  A thread walks its chunk and K-1 tokens more: dz of a token adds
// w[j] * dz to the row K-1-j places earlier, held in accumulators that move on
// with the walk, so a row of dx is complete K-1 tokens later; tokens of the
// next sequence do not reach back over its start.  The sums of dw and db
// stay in registers over the chunk, are added over the workgroup's chunks in
// LDS and written as one row of partial sums; k_causal_grad_sum adds those.
// ---------------------------------------------------------------------------
template <typename T, int V, int K>
__global__ __launch_bounds__(kThreads) void k_causal_grad(CausalArgs a, int groups, int lanes,
                                                          int chunk)
{
    __shared__ float lds[kThreads * V];
    const int tid = threadIdx.x, lane = tid % lanes, slot = tid / lanes;
    const int group = blockIdx.x * lanes + lane;
    const bool valid = group < groups;
    const int c0 = first_channel<V>(min(group, groups - 1), a.C);
    const int rows = a.batch.rows;
    const long long first = ((long long)blockIdx.y * (kThreads / lanes) + slot) * chunk;
    const int t0 = (int)(first < rows ? first : rows);
    const int t1 = min(t0 + min(chunk, rows - t0), rows);
    const int t2 = min(t1 + min(K - 1, rows - t1), rows);
    const T *x = static_cast<const T *>(a.x) + c0;
    const T *dy = static_cast<const T *>(a.dy) + c0;
    const T *init = static_cast<const T *>(a.init);
    const T *dfinal = static_cast<const T *>(a.dfinal);
    T *dx = static_cast<T *>(a.dx) + c0;

    float w[K][V], b[V], ext[K - 1 + kGradAhead][V], acc[K - 1 + kGradAhead][V], dw[K][V], db[V];
    load_taps<V, K>(a.w, a.wtype, c0, w);
    load_bias<V>(a.b, c0, b);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        db[v] = 0.0f;
#pragma unroll
        for (int j = 0; j < K; ++j)
            dw[j][v] = 0.0f;
#pragma unroll
        for (int j = 0; j < K - 1 + kGradAhead; ++j)
            ext[j][v] = acc[j][v] = 0.0f;
    }
    if (valid && t0 < t1) {
#pragma unroll
        for (int j = 0; j < K - 1; ++j)
            if (t0 - (K - 1) + j >= 0)
                load<T, V>(x + (long long)(t0 - (K - 1) + j) * a.ldx, ext[j]);
        Walk at(a.batch, t0);
        Raw<T, V> xs[kGradAhead], dys[kGradAhead];
        // (a row's address is a 64-bit product, as dear as the row's arithmetic: one
        // for all rows where none of them needs to be held back)
        auto fetch = [&](int t) {
            const int row = min(t, t2 - 1);
            const T *px = x + row * a.ldx, *pd = dy + row * a.lddy;
            if (t + kGradAhead <= t2) {
#pragma unroll
                for (int u = 0; u < kGradAhead; ++u) {
                    xs[u].load(px + u * a.ldx);
                    dys[u].load(pd + u * a.lddy);
                }
            } else {
#pragma unroll
                for (int u = 0; u < kGradAhead; ++u) {
                    xs[u].load(px);
                    dys[u].load(pd);
                    if (t + u + 1 < t2) {
                        px += a.ldx;
                        pd += a.lddy;
                    }
                }
            }
        };
        fetch(t0);
        for (int t = t0; t < t1 + K - 1; t += kGradAhead) {
            float ds[kGradAhead][V];
#pragma unroll
            for (int u = 0; u < kGradAhead; ++u)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    ext[K - 1 + u][v] = xs[u].get(v);
                    ds[u][v] = dys[u].get(v);
                }
            // the next rows are on their way while these are worked on
            fetch(t + kGradAhead);
            at.to(a.batch, min(t, t2 - 1));
            // away from a sequence's ends and from the chunk's
            if (t - at.start >= K - 1 && t + kGradAhead + K - 1 <= at.end && t + kGradAhead <= t1) {
                float z[kGradAhead * V];
#pragma unroll
                for (int u = 0; u < kGradAhead; ++u)
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        z[u * V + v] = b[v];
#pragma unroll
                        for (int j = 0; j < K; ++j)
                            z[u * V + v] = fmaf(w[j][v], ext[u + j][v], z[u * V + v]);
                    }
                slope_all(z, a.act);
#pragma unroll
                for (int u = 0; u < kGradAhead; ++u)
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        const float dz = ds[u][v] * z[u * V + v];
                        db[v] += dz;
#pragma unroll
                        for (int j = 0; j < K; ++j) {
                            dw[j][v] = fmaf(dz, ext[u + j][v], dw[j][v]);
                            acc[u + j][v] = fmaf(w[j][v], dz, acc[u + j][v]);
                        }
                    }
            } else {
#pragma unroll
                for (int u = 0; u < kGradAhead; ++u) {
                    const int tt = t + u;
                    if (tt >= t2)
                        continue;
                    at.to(a.batch, tt);
                    const int pos = tt - at.start, left = at.end - 1 - tt;
                    float z[V], row[K][V];
#pragma unroll
                    for (int v = 0; v < V; ++v)
                        z[v] = b[v];
#pragma unroll
                    for (int j = 0; j < K; ++j) {
#pragma unroll
                        for (int v = 0; v < V; ++v)
                            row[j][v] = ext[u + j][v];
                        if (pos < K - 1 - j)
                            carried_row<T, V>(init, at.s, pos + j, K, a.C, c0, row[j]);
#pragma unroll
                        for (int v = 0; v < V; ++v)
                            z[v] = fmaf(w[j][v], row[j][v], z[v]);
                    }
                    slope_all(z, a.act);
#pragma unroll
                    for (int v = 0; v < V; ++v)
                        z[v] *= ds[u][v];
                    if (tt < t1) {
#pragma unroll
                        for (int v = 0; v < V; ++v)
                            db[v] += z[v];
#pragma unroll
                        for (int j = 0; j < K; ++j)
#pragma unroll
                            for (int v = 0; v < V; ++v)
                                dw[j][v] = fmaf(z[v], row[j][v], dw[j][v]);
                        if (dfinal && left < K - 1)
                            load<T, V>(dfinal + ((long long)at.s * (K - 1) + K - 2 - left) * a.C +
                                           c0, acc[u + K - 1]);
                    }
#pragma unroll
                    for (int j = 0; j < K; ++j)
                        if (pos >= K - 1 - j)
#pragma unroll
                            for (int v = 0; v < V; ++v)
                                acc[u + j][v] = fmaf(w[j][v], z[v], acc[u + j][v]);
                }
            }
            // rows K-1 places back are complete; the windows move on
            const int done = t - (K - 1);
            T *to = dx + done * a.lddx;
            if (done >= t0 && done + kGradAhead <= t1) {
#pragma unroll
                for (int u = 0; u < kGradAhead; ++u)
                    store<T, V>(to + u * a.lddx, acc[u]);
            } else {
#pragma unroll
                for (int u = 0; u < kGradAhead; ++u)
                    if (done + u >= t0 && done + u < t1)
                        store<T, V>(to + u * a.lddx, acc[u]);
            }
#pragma unroll
            for (int j = 0; j < K - 1 + kGradAhead; ++j)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    acc[j][v] = j < K - 1 ? acc[min(j, K - 2) + kGradAhead][v] : 0.0f;
                    if (j < K - 1)
                        ext[j][v] = ext[j + kGradAhead][v];
                }
        }
    }
    // the partial sums of the workgroup's chunks, one row after the other
    float *part = a.part + (long long)blockIdx.y * (K + 1) * a.C;
#pragma unroll
    for (int j = 0; j <= K; ++j) {
#pragma unroll
        for (int v = 0; v < V; ++v)
            lds[tid * V + v] = j < K ? dw[min(j, K - 1)][v] : db[v];
        __syncthreads();
        if (slot == 0 && valid) {
            float s[V];
#pragma unroll
            for (int v = 0; v < V; ++v)
                s[v] = 0.0f;
            for (int k = 0; k < kThreads / lanes; ++k)
#pragma unroll
                for (int v = 0; v < V; ++v)
                    s[v] += lds[(k * lanes + lane) * V + v];
            store<float, V>(part + (long long)j * a.C + c0, s);
        }
        __syncthreads();
    }
}

__global__ __launch_bounds__(1024) void k_causal_grad_sum(const float *part, int blocks, int C,
                                                          int K, float *dw, float *db)
{
    column_sums(part, blocks, (long long)(K + 1) * C, [=](long long col, float s) {
        const int j = (int)(col / C), c = (int)(col % C);
        if (j < K)
            dw[(long long)c * K + j] = s;
        else if (db)
            db[c] = s;
    });
}

// The gradient of the carried rows, a thread per element: row q collects
// w[j] * dz of the tokens t = q - j, and dfinal where the sequence is so short
// that the row is carried on.
template <typename T, int K>
__global__ __launch_bounds__(kThreads) void k_causal_grad_init(CausalArgs a)
{
    const long long id = (long long)block_id() * kThreads + threadIdx.x;
    const int c = (int)(id % a.C);
    const long long sq = id / a.C;
    if (sq >= (long long)a.batch.seqs * (K - 1))
        return;
    const int s = (int)(sq / (K - 1)), q = (int)(sq % (K - 1));
    const int start = seq_start(a.batch, s);
    const int len = max(seq_start(a.batch, s + 1) - start, 0);
    const T *x = static_cast<const T *>(a.x), *dy = static_cast<const T *>(a.dy);
    const T *init = static_cast<const T *>(a.init);
    float w[K][1], b[1];
    load_taps<1, K>(a.w, a.wtype, c, w);
    load_bias<1>(a.b, c, b);
    float g = 0.0f;
    if (a.dfinal && q >= len)
        g = (float)static_cast<const T *>(a.dfinal)[((long long)s * (K - 1) + q - len) * a.C + c];
    for (int j = 0; j <= q; ++j) {
        const int t = q - j;
        if (t >= len)
            continue;
        float z = b[0];
        float wj = 0.0f;
#pragma unroll
        for (int i = 0; i < K; ++i) {
            const int p = t - (K - 1) + i;
            float row[1];
            if (p >= 0)
                load<T, 1>(x + (long long)(start + p) * a.ldx + c, row);
            else
                carried_row<T, 1>(init, s, p + K - 1, K, a.C, c, row);
            z = fmaf(w[i][0], row[0], z);
            wj = i == j ? w[i][0] : wj;
        }
        const float d = (float)dy[(long long)(start + t) * a.lddy + c];
        g = fmaf(wj, d * act_slope(z, a.act), g);
    }
    static_cast<T *>(a.dinit)[id] = (T)g;
}

// f(taps) with the number of taps as a constant
template <typename F> int with_taps(int K, F f)
{
    switch (K) {
    case 1: return f(std::integral_constant<int, 1>());
    case 2: return f(std::integral_constant<int, 2>());
    case 3: return f(std::integral_constant<int, 3>());
    case 4: return f(std::integral_constant<int, 4>());
    case 5: return f(std::integral_constant<int, 5>());
    case 6: return f(std::integral_constant<int, 6>());
    case 7: return f(std::integral_constant<int, 7>());
    case 8: return f(std::integral_constant<int, 8>());
    }
    return DWCONV_ERR_BAD_DIM;
}

// f(element pointer type, channels per thread, taps): vectors of W channels, or
// single ones where a row is narrower than that
template <int W, typename F> int with_variant(const CausalArgs &a, F f)
{
    return with_type(a.type, [&](auto *t) {
        return with_taps(a.K, [&](auto k) {
            if (a.C >= W)
                return f(t, std::integral_constant<int, W>(), k);
            return f(t, std::integral_constant<int, 1>(), k);
        });
    });
}

}  // namespace

int launch_causal_fwd(const CausalArgs &a, void *stream)
{
    return with_variant<4>(a, [&](auto *t, auto v, auto k) {
        using T = std::remove_pointer_t<decltype(t)>;
        constexpr int V = decltype(v)::value, K = decltype(k)::value;
        const int groups = (int)cdiv(a.C, V);
        // Chunks as long as leaves 16 waves for each of the 256 CUs.  4 channels a
        // thread against 8 of 16 bits: 54.7 and 66.4 us on 8 x 4096 x 2048 bfloat16, 4
        // taps, SiLU, the same tensors each time: twice the waves, half the registers.
        int chunk = 32;
        while (chunk > kAhead && cdiv(a.batch.rows, chunk) * groups < 256 * 1024)
            chunk >>= 1;
        while (cdiv(a.batch.rows, chunk) * groups > 0x7fff0000LL)
            chunk <<= 1;
        const int chunks = (int)cdiv(a.batch.rows, chunk);
        const long long main_blocks = cdiv((long long)chunks * groups, kThreads);
        const long long rest = a.final_state && K > 1
                                   ? cdiv((long long)a.batch.seqs * (K - 1) * groups, kThreads)
                                   : 0;
        if (main_blocks + rest == 0)
            return DWCONV_OK;
        if (main_blocks + rest > 0x7fffffffLL)
            return DWCONV_ERR_BAD_DIM;
        return dwconv::launch_kernel(k_causal_fwd<T, V, K>, grid_of(main_blocks + rest),
                                     dim3(kThreads), 0, static_cast<hipStream_t>(stream), a,
                                     groups, chunk, chunks, (int)main_blocks);
    });
}

int launch_causal_step(const CausalArgs &a, void *stream)
{
    return with_variant<4>(a, [&](auto *t, auto v, auto k) {
        using T = std::remove_pointer_t<decltype(t)>;
        constexpr int V = decltype(v)::value, K = decltype(k)::value;
        const int groups = (int)cdiv(a.C, V);
        const long long blocks = cdiv((long long)a.batch.seqs * groups, kThreads);
        if (blocks > 0x7fffffffLL)
            return DWCONV_ERR_BAD_DIM;
        return dwconv::launch_kernel(k_causal_step<T, V, K>, grid_of(blocks), dim3(kThreads), 0,
                                     static_cast<hipStream_t>(stream), a, groups);
    });
}

// Chunks of 64 tokens, shorter where there would be too few workgroups, longer
// where there would be more than 512 rows of partial sums.  Measured on 8 x 4096 x
// 2048 bfloat16, 4 taps, before the last changes (the same tensors each time): 64 tokens
// and 2 channels a thread with the next rows in flight 115.7 us; 32 tokens 129.4; 4
// channels 130.6; 8 rows ahead 124.6; without the next rows in flight 152.
CausalGradPlan causal_grad_plan(int rows, int C)
{
    CausalGradPlan p;
    p.chunk = 64;
    while (p.chunk > 8 && cdiv(rows, 4LL * p.chunk) * cdiv(C, 128) < 512)
        p.chunk >>= 1;
    while (cdiv(rows, 4LL * p.chunk) > 512)
        p.chunk <<= 1;
    p.blocks = (int)cdiv(rows, 4LL * p.chunk);
    return p;
}

long long causal_grad_workspace(int rows, int C, int K)
{
    return 4LL * causal_grad_plan(rows, C).blocks * C * (K + 1);
}

int launch_causal_grad(const CausalArgs &a, void *stream)
{
    hipStream_t st = static_cast<hipStream_t>(stream);
    const CausalGradPlan p = causal_grad_plan(a.batch.rows, a.C);
    int rc = DWCONV_OK;
    if (p.blocks > 0)
        rc = with_variant<2>(a, [&](auto *t, auto v, auto k) {
            using T = std::remove_pointer_t<decltype(t)>;
            constexpr int V = decltype(v)::value, K = decltype(k)::value;
            const int groups = (int)cdiv(a.C, V);
            return dwconv::launch_kernel(k_causal_grad<T, V, K>,
                                         dim3((unsigned)cdiv(groups, 64), (unsigned)p.blocks),
                                         dim3(kThreads), 0, st, a, groups, 64, p.chunk);
        });
    if (rc == DWCONV_OK)
        rc = dwconv::launch_kernel(k_causal_grad_sum,
                                   grid_of(cdiv((long long)(a.K + 1) * a.C, 64)),
                                   dim3(1024), 0, st, (const float *)a.part, p.blocks, a.C, a.K,
                                   a.dw, a.db);
    if (rc == DWCONV_OK && a.dinit && a.K > 1)
        rc = with_type(a.type, [&](auto *t) {
            using T = std::remove_pointer_t<decltype(t)>;
            return with_taps(a.K, [&](auto k) {
                constexpr int K = decltype(k)::value;
                if constexpr (K == 1) {
                    return DWCONV_OK;
                } else {
                    const long long blocks =
                        cdiv((long long)a.batch.seqs * (K - 1) * a.C, kThreads);
                    if (blocks > 0x7fffffffLL)
                        return DWCONV_ERR_BAD_DIM;
                    return dwconv::launch_kernel(k_causal_grad_init<T, K>, grid_of(blocks),
                                                 dim3(kThreads), 0, st, a);
                }
            });
        });
    return rc;
}

}  // namespace dwseq

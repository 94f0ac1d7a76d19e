// dwmix_few.hip -- the product of 8-bit integers for few rows that are not quantised
// yet (the tokens of a decoding step), in one launch.
#define DWSEQ_GEMM_KERNELS
#include "dwmix_internal.h"
#include "dwmix_quantize.h"
#include "dwseq_gemm.h"

namespace dwmix {
namespace {

using namespace dwseq;

// Bound by reading w once, and below some MB by the latency of a launch.  A workgroup
// takes 16 NF columns; its 8 waves each take a range of k, as in the product of few rows
// that are numbers already.  Every workgroup quantises all of x for itself, into LDS,
// while its first rows of w are on their way: up to 64 elements a thread, about 2 us,
// where a launch of its own took 4 us and a pause (8 x 8192 x 2048: a call takes 12.5
// us for 17).
template <typename O, int NF> __global__ __launch_bounds__(512) void k_linear_few(LinearI8Args a)
{
    typedef I8<O> T;
    constexpr int V = 16 / (int)sizeof(O), kWaves = 8, step = 64, kAhead = 8 / NF;
    // [M][pitch]
    extern __shared__ __attribute__((aligned(16))) signed char numbers[];
    __shared__ f32x4 sums[kWaves][NF][64];
    __shared__ float scales[16];
    __shared__ unsigned tops[kWaves];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, i = lane & 15;
    const int n0 = blockIdx.x * 16 * NF, padded = (a.K + step - 1) / step * step, pitch = padded + 16;
    const signed char *w[NF];
#pragma unroll
    for (int n = 0; n < NF; ++n)
        w[n] = static_cast<const signed char *>(a.w) +
               (long long)min(n0 + n * 16 + i, a.N - 1) * a.ldw;
    const int per_wave = (padded / step + kWaves - 1) / kWaves * step;
    const int k0 = wave * per_wave, k1 = min(k0 + per_wave, padded);
    u32x4 fq[kAhead][NF];
    auto fetch = [&](int k) {
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
#pragma unroll
            for (int n = 0; n < NF; ++n)
                fq[u][n] = k + u * step < k1 ? chunk_of(w[n], k + u * step + g * 16, a.K)
                                             : u32x4{0, 0, 0, 0};
    };
    fetch(k0);
    // `team` waves a row
    const int team = a.M == 1 ? 8 : a.M == 2 ? 4 : a.M <= 4 ? 2 : 1, lanes = team * 64;
    const int at = wave % team * 64 + lane, whole = a.K / V;
    for (int m0 = 0; m0 < a.M; m0 += kWaves / team) {
        const int m = m0 + wave / team;
        const O *x = static_cast<const O *>(a.x) + (long long)min(m, a.M - 1) * a.ldx;
        constexpr int kKeep = 4;
        Raw<O, V> kept[kKeep];
        Largest<O> all;
#pragma unroll
        for (int j = 0; j < kKeep; ++j) {
            kept[j].clear();
            if (at + j * lanes < whole)
                kept[j].load(x + (at + j * lanes) * V);
        }
#pragma unroll
        for (int j = 0; j < kKeep; ++j)
            all.look(kept[j]);
        for (int c = at + kKeep * lanes; c < whole; c += lanes) {
            Raw<O, V> r;
            r.load(x + c * V);
            all.look(r);
        }
        unsigned top = all.get();
        const int tail = whole * V + at;        // fewer than V elements
        if (tail < a.K)
            top = max(top, magnitude(x[tail]));
        for (int d = 32; d; d >>= 1)
            top = max(top, (unsigned)__shfl_xor((int)top, d));
        if (lane == 0)
            tops[wave] = top;
        __syncthreads();
        for (int t = 0; t < team; ++t)
            top = max(top, tops[wave / team * team + t]);
        if (m < a.M) {
            const RowScale s(top);
            signed char *to = numbers + m * pitch;
            auto put = [&](const Raw<O, V> &r, int c) {
                *reinterpret_cast<Pack<signed char, V> *>(to + c * V) =
                    s.numbers<V>([&](int v) { return r.get(v); });
            };
#pragma unroll
            for (int j = 0; j < kKeep; ++j)
                if (at + j * lanes < whole)
                    put(kept[j], at + j * lanes);
            for (int c = at + kKeep * lanes; c < whole; c += lanes) {
                Raw<O, V> r;
                r.load(x + c * V);
                put(r, c);
            }
            if (tail < a.K)
                to[tail] = (signed char)s.exact((float)x[tail]);
            if (a.K + at < padded)      // up to 63
                to[a.K + at] = 0;
            if (at == 0)
                scales[m] = s.scale;
        }
        __syncthreads();
    }
    f32x4 acc[NF];
#pragma unroll
    for (int n = 0; n < NF; ++n)
        acc[n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    const signed char *p = numbers + min(i, a.M - 1) * pitch + g * 16;
    for (int k = k0; k < k1; k += kAhead * step) {
        u32x4 now[kAhead][NF];
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
#pragma unroll
            for (int n = 0; n < NF; ++n)
                now[u][n] = fq[u][n];
        fetch(k + kAhead * step);
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const u32x4 fp = *reinterpret_cast<const u32x4 *>(p + min(k + u * step, padded - step));
#pragma unroll
            for (int n = 0; n < NF; ++n)
                mma<T>(now[u][n], fp, acc[n]);
        }
    }
#pragma unroll
    for (int n = 0; n < NF; ++n)
        sums[wave][n][lane] = acc[n];
    __syncthreads();
    const int col = n0 + wave * 16 + g * 4;
    if (wave >= NF || i >= a.M || col >= a.N)
        return;
    float sum[4] = {}, b[4] = {}, cols[4];
#pragma unroll
    for (int v = 0; v < kWaves; ++v) {
        const f32x4 part = sums[v][wave][lane];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            sum[e] = add<T>(sum[e], part[e]);
    }
    get(a.w_scale + col, a.N - col, cols);
    widen<T>(sum, scales[i], cols);
    if (a.b)
        get(a.b + col, a.N - col, b);
    const Finish f{a.b, a.res, nullptr, a.y, a.ldres, 0, a.ldy, a.act, nullptr, nullptr, nullptr};
    Raw<O, 4> r;
    if (a.res)
        residual(f, i, col, a.N - col, r);
    finish<O>(f, i, col, a.N - col, b, r, sum);
}

}  // namespace

int launch_linear_few(const LinearI8Args &a, void *stream)
{
    const size_t lds = (size_t)a.M * (cdiv(a.K, 64) * 64 + 16);
    // 32 columns a workgroup, where that still is one for every CU: x is quantised half
    // as often
    const int nf = a.N >= 256 * 32 ? 2 : 1;
    return with_type(a.type, [&](auto *t) {
        using O = std::remove_pointer_t<decltype(t)>;
        return dwconv::launch_kernel(nf == 2 ? k_linear_few<O, 2> : k_linear_few<O, 1>,
                                     dim3((unsigned)cdiv(a.N, 16 * nf)), dim3(512), lds,
                                     static_cast<hipStream_t>(stream), a);
    });
}

}  // namespace dwmix

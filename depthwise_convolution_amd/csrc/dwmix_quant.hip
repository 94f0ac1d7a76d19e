// dwmix_quant.hip -- rows quantised to 8 bits, and the matrix product of 8-bit
// integers with a scale for each row and column (include/dwconv_mix.h).  The
// product's kernels are those of dwseq_gemm.h.
#include "dwmix_internal.h"
#include "dwseq_gemm.h"

namespace dwmix {
namespace {

using namespace dwseq;

// What a row's largest absolute value, as bits, gives: its scale, and the factors
// that its numbers are made with.  Rows of very small scales are computed 2^60
// times larger, so that a remainder next to a half never falls below the smallest
// float32.
struct RowScale {
    float scale, up, step, inv;

    __device__ __forceinline__ explicit RowScale(unsigned largest)
    {
        const bool finite = largest < 0x7f800000u;
        scale = fmaxf(__builtin_bit_cast(float, finite ? largest : 0u) * (1.0f / 127.0f),
                      0x1p-126f);
        up = scale < 0x1p-60f ? 0x1p60f : 1.0f;
        step = scale * up;
        inv = finite ? __builtin_amdgcn_rcpf(step) : 0.0f;
        if (!finite)
            scale = __builtin_nanf("");
    }
    // x / scale to the nearest integer, halves to even, 0 in a row that is not finite.
    // The estimate x * inv is off by a few units in its last place, so that its nearest
    // integer n is the quotient's unless the quotient lies that near to a half: where
    // |x - n scale|, which one multiply-add rounds once and so compares exactly with half
    // the scale, is not below it.
    //
    // Adding 3 * 2^22 rounds to an integer, which then is in the sum's low bits.
    __device__ __forceinline__ float shifted(float x) const
    {
        return __builtin_fmaf(x * up, inv, 0x1.8p23f);
    }
    __device__ __forceinline__ float rest(float x, float t) const
    {
        return fabsf(__builtin_fmaf(-(t - 0x1.8p23f), step, x * up));
    }
    __device__ __forceinline__ bool near_half(float rest) const { return !(rest < 0.5f * step); }
    // ... and what it is there
    __device__ int exact(float x) const
    {
        const float v = fabsf(x) * up;
        const float n = fminf(floorf(v * inv), 127.0f);
        const float above = __builtin_fmaf(-(n + 0.5f), step, v);
        int i = (int)n;
        i += above > 0.0f || (above == 0.0f && (i & 1));
        i = inv == 0.0f ? 0 : min(i, 127);
        return x < 0.0f ? -i : i;
    }
    // The numbers of V elements
    template <int V, typename F>
    __device__ __forceinline__ Pack<signed char, V> numbers(F get) const
    {
        float t[V], most = 0.0f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            t[v] = shifted(get(v));
            most = fmaxf(most, rest(get(v), t[v]));
        }
        Pack<signed char, V> n;
#pragma unroll
        for (int v = 0; v < V; ++v)
            n.v[v] = (signed char)__builtin_bit_cast(int, t[v]);
        if (near_half(most) || inv == 0.0f)
#pragma unroll
            for (int v = 0; v < V; ++v)
                n.v[v] = (signed char)exact(get(v));
        return n;
    }
};

template <int WAVES> __device__ __forceinline__ unsigned row_max(unsigned m)
{
    for (int d = 32; d; d >>= 1)
        m = max(m, (unsigned)__shfl_xor((int)m, d));
    if constexpr (WAVES > 1) {
        __shared__ unsigned lds[WAVES];
        if ((threadIdx.x & 63) == 0)
            lds[threadIdx.x >> 6] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < WAVES; ++w)
            m = max(m, lds[w]);
    }
    return m;
}

template <typename T> __device__ __forceinline__ unsigned magnitude(T v)
{
    return __builtin_bit_cast(unsigned, (float)v) & 0x7fffffffu;
}

// A row for each WAVES waves (a workgroup has 256 threads).  The largest magnitude
// is found on bit patterns, which order NaN above infinity above the rest.  A row
// of up to kKeep vectors a thread is read once and waits in registers; a longer
// one is read again, from the caches.
constexpr int kKeep = 4;

template <typename T, int WAVES>
__global__ __launch_bounds__(256) void k_quantize(QuantizeArgs a)
{
    constexpr int V = 16 / (int)sizeof(T), lanes = WAVES * 64, rows = 256 / lanes;
    const int m = (int)block_id() * rows + (int)threadIdx.x / lanes, at = threadIdx.x % lanes;
    if (m >= a.M)
        return;     // whole waves; with more than one wave a row, the whole workgroup
    const T *x = static_cast<const T *>(a.x) + (long long)m * a.ldx;
    signed char *q = a.q + (long long)m * a.ldq;
    const int whole = a.K / V;      // vectors
    Raw<T, V> kept[kKeep];
    unsigned largest = 0;
#pragma unroll
    for (int j = 0; j < kKeep; ++j)
        if (at + j * lanes < whole) {
            kept[j].load(x + (at + j * lanes) * V);
#pragma unroll
            for (int v = 0; v < V; ++v)
                largest = max(largest, magnitude(kept[j].get(v)));
        }
    for (int c = at + kKeep * lanes; c < whole; c += lanes) {
        Raw<T, V> r;
        r.load(x + (long long)c * V);
#pragma unroll
        for (int v = 0; v < V; ++v)
            largest = max(largest, magnitude(r.get(v)));
    }
    const int tail = whole * V + at;        // fewer than V elements
    if (tail < a.K)
        largest = max(largest, magnitude((float)x[tail]));
    const RowScale s(row_max<WAVES>(largest));
    auto put = [&](const Raw<T, V> &r, int c) {
        *reinterpret_cast<Pack<signed char, V> *>(q + (long long)c * V) =
            s.numbers<V>([&](int v) { return r.get(v); });
    };
#pragma unroll
    for (int j = 0; j < kKeep; ++j)
        if (at + j * lanes < whole)
            put(kept[j], at + j * lanes);
    for (int c = at + kKeep * lanes; c < whole; c += lanes) {
        Raw<T, V> r;
        r.load(x + (long long)c * V);
        put(r, c);
    }
    if (tail < a.K)
        q[tail] = (signed char)s.exact((float)x[tail]);
    if (at == 0)
        a.scale[m] = s.scale;
}

// The parts of a product's workspace: x's numbers (rows of a multiple of 16) and
// scales, and the partial sums.
struct Space {
    long long numbers, scales, sums, ld;
};

Space space_of(bool quantized, int M, int N, int K)
{
    Space s{};
    s.ld = cdiv(K, 16) * 16;
    if (!quantized) {
        s.numbers = s.ld * M;
        s.scales = cdiv(4LL * M, 16) * 16;
    }
    s.sums = gemm_workspace(1, 0, M, N, K);
    return s;
}

}  // namespace

int launch_quantize(const QuantizeArgs &a, void *stream)
{
    if (a.M == 0)
        return DWCONV_OK;
    hipStream_t st = static_cast<hipStream_t>(stream);
    return with_type(a.type, [&](auto *t) {
        using T = std::remove_pointer_t<decltype(t)>;
        // a wave for rows that it keeps whole (and where there are many), else four
        const bool narrow = a.K <= 64 * kKeep * 16 / (int)sizeof(T) && a.M >= 1024;
        return narrow ? dwconv::launch_kernel(k_quantize<T, 1>, grid_of(cdiv(a.M, 4)), dim3(256),
                                              0, st, a)
                      : dwconv::launch_kernel(k_quantize<T, 4>, grid_of(a.M), dim3(256), 0, st,
                                              a);
    });
}

long long linear_i8_workspace(bool quantized, int M, int N, int K)
{
    if (M == 0)
        return 0;
    const Space s = space_of(quantized, M, N, K);
    return s.numbers + s.scales + s.sums;
}

void linear_i8_describe(bool quantized, bool aligned, int M, int N, int K, const char **name,
                        int *splits)
{
    (void)quantized;
    const GemmPlan plan = gemm_plan(1, 0, M, N, K);
    const bool direct = aligned && direct_ok(nullptr, 0, false, K, 1);
    *splits = split_count(K, plan.splits, 1);
    *name = tile_name(tile_taken(plan.tile, direct, 1), direct);
}

int launch_linear_i8(const LinearI8Args &a, void *stream)
{
    if (a.M == 0)
        return DWCONV_OK;
    const bool quantized = a.x_scale != nullptr;
    const Space s = space_of(quantized, a.M, a.N, a.K);
    char *space = static_cast<char *>(a.workspace);
    const void *x = a.x;
    const float *rows = a.x_scale;
    long long ldx = a.ldx;
    if (!quantized) {
        float *scale = reinterpret_cast<float *>(space + s.numbers);
        const int rc = launch_quantize({a.x, reinterpret_cast<signed char *>(space), scale, a.ldx,
                                        s.ld, a.type, a.M, a.K},
                                       stream);
        if (rc != DWCONV_OK)
            return rc;
        x = space;
        rows = scale;
        ldx = s.ld;
    }
    return with_type(a.type, [&](auto *t) {
        using O = std::remove_pointer_t<decltype(t)>;
        const GemmPlan plan = gemm_plan(1, 0, a.M, a.N, a.K);
        Finish f{a.b, a.res, nullptr, a.y, a.ldres, 0, a.ldy, a.act, nullptr, rows, a.w_scale};
        f.part = reinterpret_cast<float *>(space + s.numbers + s.scales);
        return launch_gemm<I8<O>>(Product{x, a.w, ldx, a.ldw, false, false, a.M, a.N, a.K,
                                          plan.tile, plan.splits, f},
                                  static_cast<hipStream_t>(stream));
    });
}

}  // namespace dwmix

// dwmix_quant.hip -- rows quantised to 8 bits, and the matrix product of 8-bit
// integers with a scale for each row and column (include/dwconv_mix.h).  The
// product's kernels are those of dwseq_gemm.h.
#include "dwmix_internal.h"
#include "dwmix_quantize.h"
#include "dwseq_gemm.h"

namespace dwmix {
namespace {

using namespace dwseq;

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

// A row for each WAVES waves (a workgroup has 256 threads).  A row of up to kKeep
// vectors a thread is read once and waits in registers; a longer one is read again,
// from the caches.  Bound by HBM: 16384 x 2048 bfloat16 20 us, 5.0 TB/s (35 with
// every quotient's half decided exactly, 28 with the magnitudes one to a register).
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
    Largest<T> all;
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
        Raw<T, V> r;
        r.load(x + (long long)c * V);
        all.look(r);
    }
    unsigned largest = all.get();
    const int tail = whole * V;     // fewer than V elements from there on
    const bool ends = at < a.K - tail;
    if (ends)
        largest = max(largest, magnitude(x[tail + at]));
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
    if (ends)
        q[tail + at] = (signed char)s.exact((float)x[tail + at]);
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
    if (M == 0 || (!quantized && few_rows_fit(M, K)))
        return 0;
    const Space s = space_of(quantized, M, N, K);
    return s.numbers + s.scales + s.sums;
}

void linear_i8_describe(bool quantized, bool aligned, int M, int N, int K, const char **name,
                        int *splits)
{
    if (!quantized && few_rows_fit(M, K)) {
        *splits = 1;
        *name = "few_rows_quantized";
        return;
    }
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
    if (!quantized && few_rows_fit(a.M, a.K))
        return launch_linear_few(a, stream);
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

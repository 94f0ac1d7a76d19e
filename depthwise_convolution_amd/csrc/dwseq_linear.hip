// dwseq_linear.hip -- matrix product with bias, activation and residual, and
// its gradients (include/dwconv_seq.h).
#include "dwseq_gemm.h"

#include <cmath>

namespace dwseq {
namespace {

// dz = dy * act'(z), and its column sums over a strip of rows (db): a workgroup
// takes 32 vectors of V columns, its 8 rows of threads every 8th row of the
// strip each.  Bound by HBM: 8192 x 4096 bfloat16 with SiLU 42.6 us, 4.7 TB/s.
//
// dz is stored in the tensors' type, since the matrix instructions of the two
// products that read it take their operands in one type: a second part for what the
// rounding loses would double their work.  It is the only loss beside the results' own
// rounding: 8192 x 4096 x 2048 bfloat16 is 2.35e-3 from 64 bits (root mean
// square), where results rounded from an exact sum are 1.66e-3, and sqrt(2) of that
// is 2.35e-3.  db sums dz before the rounding.
constexpr int kDzLanes = 32, kDzSlots = 8;

struct DzPlan {
    int strip, strips;      // rows, and how many of them (1024 at most)
};

DzPlan dz_plan(int M, int N)
{
    int strip = 64;
    while (strip > kDzSlots && cdiv(M, strip) * cdiv(N, 256) < 512)
        strip /= 2;
    while (cdiv(M, strip) > 1024)
        strip *= 2;
    return {strip, (int)cdiv(M, strip)};
}

template <typename T, int V>
__global__ __launch_bounds__(kDzLanes *kDzSlots) void k_dz(LinearArgs a, T *dz, float *part,
                                                           int strip)
{
    __shared__ float lds[kDzSlots][kDzLanes * V];
    const int lane = threadIdx.x % kDzLanes, slot = threadIdx.x / kDzLanes;
    const int at = (blockIdx.x * kDzLanes + lane) * V;
    const bool mine = at < a.N;
    const int n = min(at, a.N - V);      // the last vector ends with the row
    const int m0 = (int)blockIdx.y * strip, m1 = m0 + min(strip, a.M - m0);
    float s[V] = {};
    if (mine)
#pragma unroll 4
        for (int m = m0 + slot; m < m1; m += kDzSlots) {
            float d[V], z[V];
            load<T, V>(static_cast<const T *>(a.dy) + m * a.lddy + n, d);
            if (a.act != DWCONV_ACT_NONE) {
                load<T, V>(static_cast<const T *>(a.z_in) + m * a.ldz + n, z);
                slope_all(z, a.act);
#pragma unroll
                for (int v = 0; v < V; ++v)
                    d[v] *= z[v];
                store<T, V>(dz + (long long)m * a.N + n, d);
            }
#pragma unroll
            for (int v = 0; v < V; ++v)
                s[v] += d[v];
        }
#pragma unroll
    for (int v = 0; v < V; ++v)
        lds[slot][lane * V + v] = s[v];
    __syncthreads();
    if (slot != 0 || !mine)
        return;
    for (int k = 1; k < kDzSlots; ++k)
#pragma unroll
        for (int v = 0; v < V; ++v)
            s[v] += lds[k][lane * V + v];
    store<float, V>(part + (long long)blockIdx.y * a.N + n, s);
}

__global__ __launch_bounds__(1024) void k_db(const float *part, int rows, int N, float *db)
{
    column_sums(part, rows, N, [=](long long n, float s) { db[n] = s; });
}

// Which kernel, and over how many ranges of k, by the time that a product
// should take (microseconds): rounds of the chip times (steps of k times a
// step's time, plus a tile's beginning and end).  A step's time grows from that
// of a workgroup alone on its CU to that of a full CU, and with the operands that
// are read across k.  All from measurements at 128 to 8192 rows and columns and K
// of 2048 to 8192, as is the time for the sum of the splits' results.
struct Shape {
    GemmTile tile;
    int rows, per_cu;
    double alone[3], full[3], ends;     // by the number of operands read across k
};
static const Shape kWide[] = {
    {TILE_256, 256, 1, {1.05, 1.40, 1.63}, {1.46, 1.70, 1.92}, 12.0},
    {TILE_128, 128, 2, {0.88, 0.95, 0.92}, {1.13, 1.18, 1.18}, 6.0},
    {TILE_64, 64, 5, {0.50, 0.52, 0.52}, {0.92, 0.99, 1.07}, 4.0},
    {TILE_64_DEEP, 64, 2, {0.34, 0.48, 0.50}, {0.41, 0.63, 0.71}, 4.0}};
static const Shape kNarrow[] = {
    {TILE_128, 128, 2, {2.30, 2.30, 2.30}, {4.10, 4.00, 4.00}, 6.0},
    {TILE_64, 64, 5, {0.75, 0.70, 0.70}, {2.65, 2.60, 2.60}, 4.0}};

}  // namespace

// Few rows of operands that are both read along k go to the kernel that reads Q
// once: measured against the 64 tile with 4 splits it is ahead while M / 16 * K is
// at most 4096 (at 32 x 4096 x 4096: 14.8 against 13.2 us; at 16 x 4096 x 2048: 6.7
// against 9.4); 8-bit operands are counted as half as many 16-bit ones.
GemmPlan gemm_plan(int size, int across, int M, int N, int K)
{
    if (across == 0 &&
        (M <= 16 || (M <= kFewRows && cdiv(M, 16) * K <= (size == 1 ? 8192 : 4096))))
        return {FEW_ROWS, 1};
    const Shape *shapes = size != 4 ? kWide : kNarrow;
    const int count = size != 4 ? 4 : 2, cus = 256;
    const long long steps = cdiv((long long)K * size, kStepBytes);
    GemmPlan best{TILE_64, 1};
    double least = 1e30;
    for (int t = 0; t < count; ++t)
        // up to 128 for the weight gradient of a narrow layer over many rows (100000 x
        // 48 x 64 float32: 160 us with 16, 36 with 128)
        for (int splits = 1; splits <= 128; splits *= 2) {
            const Shape &s = shapes[t];
            const double sums = 4.0 * M * N * splits;       // bytes of partial sums
            if (splits > 1 && (steps < 4 * splits || sums > 64e6))
                break;
            const double groups = (double)cdiv(M, s.rows) * cdiv(N, s.rows) * splits;
            // how far a CU is from one workgroup to as many as it holds; where it
            // holds one, how far the chip is from half full to full
            const double load = s.per_cu > 1 ? (groups / cus - 1.0) / (s.per_cu - 1.0)
                                             : 2.0 * groups / cus - 1.0;
            const double part = load < 0.0 ? 0.0 : load > 1.0 ? 1.0 : load;
            const double step = s.alone[across] + (s.full[across] - s.alone[across]) * part;
            // float32's small workgroups follow each other without rounds: their time is
            // the matrix instructions' (25088 x 256 x 128, kernels alone: 64 tile 25.9 us,
            // 128 tile 27.7; counted so, bfloat16 would lose: 12.3 against 11.4)
            const double fill = groups / (cus * s.per_cu);
            const double rounds = size == 4 && s.per_cu > 2 && fill > 1.0 ? fill : std::ceil(fill);
            double time = rounds * (cdiv(steps, splits) * step + s.ends);
            if (splits > 1)
                time += 3.0 + sums * 2.0 / 4e6;
            if (time < least) {
                least = time;
                best = {s.tile, splits};
            }
        }
    return best;
}

long long gemm_workspace(int size, int across, int M, int N, int K)
{
    const GemmPlan p = gemm_plan(size, across, M, N, K);
    return p.splits > 1 ? 4LL * M * N * p.splits : 0;
}

namespace {

template <typename T>
int product(const T *P, long long ldp, bool p_rows_k, const T *Q, long long ldq, bool q_rows_k,
            int M, int N, int K, Finish f, void *partials, hipStream_t st)
{
    if (M == 0 || N == 0)
        return DWCONV_OK;
    const GemmPlan plan = gemm_plan((int)sizeof(T), p_rows_k + q_rows_k, M, N, K);
    f.part = static_cast<float *>(partials);
    return launch_gemm<T>(Product{P, Q, ldp, ldq, p_rows_k, q_rows_k, M, N, K, plan.tile,
                                  plan.splits, f},
                          st);
}

}  // namespace

// The parts of a gradient's workspace: dz, the partial sums of db, and those of
// a product (dx's and dw's one after the other in the same place).
struct GradSpace {
    long long dz, db, sums;
};

static GradSpace grad_space(int type, int act, int M, int N, int K)
{
    const int size = elem_size(type);
    GradSpace g;
    g.dz = act == DWCONV_ACT_NONE ? 0 : cdiv((long long)M * N * size, 16) * 16;
    g.db = cdiv(4LL * dz_plan(M, N).strips * N, 16) * 16;
    const long long dx = gemm_workspace(size, 1, M, K, N), dw = gemm_workspace(size, 2, N, K, M);
    g.sums = dx > dw ? dx : dw;
    return g;
}

long long linear_workspace(bool grad, int type, int act, int M, int N, int K)
{
    if (M == 0)
        return 0;
    if (!grad)
        return gemm_workspace(elem_size(type), 0, M, N, K);
    const GradSpace g = grad_space(type, act, M, N, K);
    return g.dz + g.db + g.sums;
}

void linear_describe(int product, int type, bool aligned, int M, int N, int K, const char **name,
                     int *splits)
{
    // rows, columns and sum of the product, and the operands that are read across k
    const int size = elem_size(type), across = product;
    const int m = product == 2 ? N : M, n = product == 0 ? N : K;
    const int k = product == 0 ? K : product == 1 ? N : M;
    const GemmPlan plan = gemm_plan(size, across, m, n, k);
    const bool direct = aligned && (across == 2 || direct_ok(nullptr, 0, false, k, size));
    *splits = split_count(k, plan.splits, size);
    *name = tile_name(tile_taken(plan.tile, direct, size), direct);
}

int launch_linear_fwd(const LinearArgs &a, void *stream)
{
    return with_type(a.type, [&](auto *t) {
        using T = std::remove_pointer_t<decltype(t)>;
        const Finish f{a.b, a.res, a.z, a.y, a.ldres, a.ldz, a.ldy, a.act, nullptr};
        return product<T>(static_cast<const T *>(a.x), a.ldx, false, static_cast<const T *>(a.w),
                          a.ldw, false, a.M, a.N, a.K, f, a.workspace,
                          static_cast<hipStream_t>(stream));
    });
}

int launch_linear_grad(const LinearArgs &a, void *stream)
{
    hipStream_t st = static_cast<hipStream_t>(stream);
    return with_type(a.type, [&](auto *t) {
        using T = std::remove_pointer_t<decltype(t)>;
        const bool plain = a.act == DWCONV_ACT_NONE;
        const GradSpace g = grad_space(a.type, a.act, a.M, a.N, a.K);
        char *space = static_cast<char *>(a.workspace);
        T *dz = reinterpret_cast<T *>(space);
        float *part = reinterpret_cast<float *>(space + g.dz);
        void *sums = space + g.dz + g.db;
        int rc = DWCONV_OK;
        const DzPlan dp = dz_plan(a.M, a.N);
        auto make_dz = [&](auto v) {
            constexpr int V = decltype(v)::value;
            return dwconv::launch_kernel(
                k_dz<T, V>, dim3((unsigned)cdiv(a.N, kDzLanes * V), (unsigned)dp.strips),
                dim3(kDzLanes * kDzSlots), 0, st, a, dz, part, dp.strip);
        };
        if (dp.strips > 0 && (!plain || a.db))
            rc = a.N >= 16 / (int)sizeof(T)
                     ? make_dz(std::integral_constant<int, 16 / (int)sizeof(T)>())
                     : make_dz(std::integral_constant<int, 1>());
        if (rc == DWCONV_OK && a.db)
            rc = dwconv::launch_kernel(k_db, dim3((unsigned)cdiv(a.N, 64)), dim3(1024), 0, st,
                                       (const float *)part, dp.strips, a.N, a.db);
        const T *d = plain ? static_cast<const T *>(a.dy) : dz;
        const long long ldd = plain ? a.lddy : a.N;
        if (rc == DWCONV_OK && a.dx) {
            const Finish f{nullptr, nullptr, nullptr, a.dx, 0, 0, a.lddx, DWCONV_ACT_NONE, nullptr};
            rc = product<T>(d, ldd, false, static_cast<const T *>(a.w), a.ldw, true, a.M, a.K,
                            a.N, f, sums, st);
        }
        if (rc == DWCONV_OK && a.dw) {
            const Finish f{nullptr, nullptr, nullptr, a.dw, 0, 0, a.lddw, DWCONV_ACT_NONE, nullptr};
            rc = product<T>(d, ldd, true, static_cast<const T *>(a.x), a.ldx, true, a.N, a.K, a.M,
                            f, sums, st);
        }
        return rc;
    });
}

}  // namespace dwseq

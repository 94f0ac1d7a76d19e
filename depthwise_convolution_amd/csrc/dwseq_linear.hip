// dwseq_linear.hip -- matrix product with bias, activation and residual, and
// its gradients (include/dwconv_seq.h).
#include "dwseq_device.h"

namespace dwseq {
namespace {

// What happens to a sum on its way to memory.
struct Finish {
    const float *b;             // per column, or nullptr
    const void *res;            // nullptr: none
    void *z, *y;                // z nullptr: not kept
    long long ldres, ldz, ldy;
    int act;
};

template <typename T>
__device__ __forceinline__ void finish(const Finish &f, long long m, int n, float s)
{
    if (f.b)
        s += f.b[n];
    if (f.z)
        static_cast<T *>(f.z)[m * f.ldz + n] = (T)s;
    s = act_of(s, f.act);
    if (f.res)
        s += (float)static_cast<const T *>(f.res)[m * f.ldres + n];
    static_cast<T *>(f.y)[m * f.ldy + n] = (T)s;
}

// y[m,n] = sum_k A[m,k] B[n,k] by strides: a workgroup's 64 x 64 tile, 16 k at
// a time through LDS, 4 x 4 sums a thread.
template <typename T>
__global__ __launch_bounds__(256) void k_product(const T *A, long long am, long long ak,
                                                 const T *B, long long bn, long long bk, int M,
                                                 int N, int K, Finish f)
{
    __shared__ float sa[16][65], sb[16][65];
    const int tid = threadIdx.x, tx = tid % 16, ty = tid / 16;
    const long long tiles_n = (N + 63) / 64;
    const int m0 = (int)(blockIdx.x / tiles_n) * 64, n0 = (int)(blockIdx.x % tiles_n) * 64;
    float s[4][4] = {};
    for (int k0 = 0; k0 < K; k0 += 16) {
        for (int e = tid; e < 1024; e += 256) {
            const int row = ak == 1 ? e / 16 : e % 64, k = ak == 1 ? e % 16 : e / 64;
            sa[k][row] = m0 + row < M && k0 + k < K
                             ? (float)A[(m0 + row) * am + (long long)(k0 + k) * ak]
                             : 0.0f;
        }
        for (int e = tid; e < 1024; e += 256) {
            const int row = bk == 1 ? e / 16 : e % 64, k = bk == 1 ? e % 16 : e / 64;
            sb[k][row] = n0 + row < N && k0 + k < K
                             ? (float)B[(n0 + row) * bn + (long long)(k0 + k) * bk]
                             : 0.0f;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < 16; ++k)
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    s[i][j] = fmaf(sa[k][ty + 16 * i], sb[k][tx + 16 * j], s[i][j]);
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
            if (m < M && n < N)
                finish<T>(f, m, n, s[i][j]);
        }
}

// dz = dy * act'(z), and its column sums over a strip of rows (db).
constexpr int kStrip = 64;      // rows

template <typename T>
__global__ __launch_bounds__(256) void k_dz(LinearArgs a, T *dz, float *part)
{
    const int n = blockIdx.x * 256 + threadIdx.x;
    if (n >= a.N)
        return;
    const int m0 = (int)blockIdx.y * kStrip, m1 = min(m0 + kStrip, a.M);
    float s = 0.0f;
    for (int m = m0; m < m1; ++m) {
        float d = (float)static_cast<const T *>(a.dy)[m * a.lddy + n];
        if (a.act != DWCONV_ACT_NONE) {
            d *= act_slope((float)static_cast<const T *>(a.z_in)[m * a.ldz + n], a.act);
            dz[(long long)m * a.N + n] = (T)d;
        }
        s += d;
    }
    part[(long long)blockIdx.y * a.N + n] = s;
}

__global__ __launch_bounds__(1024) void k_db(const float *part, int rows, int N, float *db)
{
    column_sums(part, rows, N, [=](long long n, float s) { db[n] = s; });
}

template <typename T>
int product(const T *A, long long am, long long ak, const T *B, long long bn, long long bk, int M,
            int N, int K, const Finish &f, hipStream_t st)
{
    const long long blocks = cdiv(M, 64) * cdiv(N, 64);
    if (blocks == 0)
        return DWCONV_OK;
    if (blocks > 0x7fffffffLL)
        return DWCONV_ERR_BAD_DIM;
    return dwconv::launch_kernel(k_product<T>, dim3((unsigned)blocks), dim3(256), 0, st, A, am, ak,
                                 B, bn, bk, M, N, K, f);
}

}  // namespace

long long linear_workspace(bool grad, int type, int act, int M, int N, int)
{
    if (!grad)
        return 0;
    const long long dz = act == DWCONV_ACT_NONE ? 0 : (long long)M * N * elem_size(type);
    return (dz + 15) / 16 * 16 + 4LL * cdiv(M, kStrip) * N;
}

int launch_linear_fwd(const LinearArgs &a, void *stream)
{
    return with_type(a.type, [&](auto *t) {
        using T = std::remove_pointer_t<decltype(t)>;
        const Finish f{a.b, a.res, a.z, a.y, a.ldres, a.ldz, a.ldy, a.act};
        return product<T>(static_cast<const T *>(a.x), a.ldx, 1, static_cast<const T *>(a.w),
                          a.ldw, 1, a.M, a.N, a.K, f, static_cast<hipStream_t>(stream));
    });
}

int launch_linear_grad(const LinearArgs &a, void *stream)
{
    hipStream_t st = static_cast<hipStream_t>(stream);
    return with_type(a.type, [&](auto *t) {
        using T = std::remove_pointer_t<decltype(t)>;
        const bool plain = a.act == DWCONV_ACT_NONE;
        T *dz = static_cast<T *>(a.workspace);
        const long long dz_bytes =
            plain ? 0 : ((long long)a.M * a.N * (long long)sizeof(T) + 15) / 16 * 16;
        float *part = reinterpret_cast<float *>(static_cast<char *>(a.workspace) + dz_bytes);
        int rc = DWCONV_OK;
        const int strips = (int)cdiv(a.M, kStrip);
        if (strips > 0 && (!plain || a.db))
            rc = dwconv::launch_kernel(k_dz<T>, dim3((unsigned)cdiv(a.N, 256), (unsigned)strips),
                                       dim3(256), 0, st, a, dz, part);
        if (rc == DWCONV_OK && a.db)
            rc = dwconv::launch_kernel(k_db, dim3((unsigned)cdiv(a.N, 64)), dim3(1024), 0, st,
                                       (const float *)part, strips, a.N, a.db);
        const T *d = plain ? static_cast<const T *>(a.dy) : dz;
        const long long ldd = plain ? a.lddy : a.N;
        if (rc == DWCONV_OK && a.dx) {
            const Finish f{nullptr, nullptr, nullptr, a.dx, 0, 0, a.lddx, DWCONV_ACT_NONE};
            rc = product<T>(d, ldd, 1, static_cast<const T *>(a.w), 1, a.ldw, a.M, a.K, a.N, f,
                            st);
        }
        if (rc == DWCONV_OK && a.dw) {
            const Finish f{nullptr, nullptr, nullptr, a.dw, 0, 0, a.lddw, DWCONV_ACT_NONE};
            rc = product<T>(d, 1, ldd, static_cast<const T *>(a.x), 1, a.ldx, a.N, a.K, a.M, f,
                            st);
        }
        return rc;
    });
}

}  // namespace dwseq

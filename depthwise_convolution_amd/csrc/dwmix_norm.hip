// dwmix_norm.hip -- group normalisation with an activation, channels last, and
// its gradients (include/dwconv_mix.h).
//
// Bound by HBM.  Two ways, by the number of positions P of an instance:
//
// * P = 1 (tokens): a group is some adjacent channels of one row.  A team of lanes
//   holds it in registers, so that x is read once; mean, then the sum of squares
//   around it, both from registers.
// * P > 1 (images), and rows whose group no team holds: a pass over x takes, for
//   each range of rows, the mean and the sum of squares around it; the ranges' are
//   joined (counts, means, squares: no difference of large sums), and a second pass
//   normalises, over the ranges in the opposite order, so that it begins with what
//   the caches (256 MB before HBM) still hold.  It writes past them: results that
//   wait there to be written would drive x out, and slow down who reads next (1 x 512 x
//   512 x 256 float32: first pass 51 us for 77, second 81 for 84; with a kernel behind
//   it that reads the results, 280 us for 293, 8 x 56 x 56 x 128 24.5 for 24.9).
//
// Gradients need two sums over a group, sum(g) and sum(g * xhat), and per channel
// sum(dz) and sum(dz * xhat), whose w-weighted sums over a group's channels are the
// former.
#include "dwmix_internal.h"
#include "dwseq_device.h"

#include <algorithm>

namespace dwmix {
namespace {

using namespace dwseq;

// ------------------------------------------------------------------ P = 1
// L lanes a group (a power of two up to 64, or 256), each K vectors of V channels,
// L vectors apart.  A workgroup takes `gw` adjacent groups of `slots` rows.
struct RowsPlan {
    int L, V, K, gw, slots, windows, threads;
    int R;                      // rows that a team of the forward holds at once
    long long blocks;           // of rows, for the gradient (which walks the rows)
};

constexpr int kRowsKeep = 8;    // vectors of a lane at most

bool rows_plan(int size, long long N, long long P, int C, int groups, RowsPlan *p)
{
    const int cg = C / groups;
    int V = 16 / size;
    while (cg % V)
        V /= 2;
    const int vectors = cg / V;
    if (P != 1 || vectors > 256 * kRowsKeep)
        return false;
    int L = 1;
    while (L < 64 && L < vectors)
        L *= 2;
    if (vectors > 128)
        L = 256;
    p->L = L;
    p->V = V;
    p->K = 1;
    while (p->K * L < vectors)
        p->K *= 2;
    p->windows = (int)cdiv(groups, 256 / L);
    p->gw = (int)cdiv(groups, p->windows);
    p->slots = 256 / (L * p->gw);
    p->threads = (int)cdiv(L * p->gw * p->slots, 64) * 64;
    // Four vectors a lane in flight, which also share w and b, where that leaves two
    // workgroups for every CU (16384 rows of 2048 bfloat16, 16 groups: 31 us with 4
    // rows a team, 36.5 us with 1; 27.5 with x read through the caches).
    p->R = std::max(1, 4 / p->K);
    if (cdiv(N, (long long)p->slots * p->R) * p->windows < 512)
        p->R = 1;
    // the gradient's workgroups walk 8 rows at least; 512 rows of partial sums at most
    p->blocks = std::max(1LL, std::min(512LL, cdiv(N, 8LL * p->slots)));
    return true;
}

// Sum over a team, in every lane of it.
template <int NS>
__device__ __forceinline__ void team_sum(float (&s)[NS], int L)
{
    for (int d = 1; d < min(L, 64); d *= 2)
#pragma unroll
        for (int e = 0; e < NS; ++e)
            s[e] += __shfl_xor(s[e], d);
    if (L > 64) {
        __shared__ float lds[4][NS];
        __syncthreads();
        if ((threadIdx.x & 63) == 0)
#pragma unroll
            for (int e = 0; e < NS; ++e)
                lds[threadIdx.x >> 6][e] = s[e];
        __syncthreads();
#pragma unroll
        for (int e = 0; e < NS; ++e)
            s[e] = (lds[0][e] + lds[1][e]) + (lds[2][e] + lds[3][e]);
    }
}

template <int V>
__device__ __forceinline__ void get_all(const float *p, float (&v)[V], float none)
{
    if (p) {
        load<float, V>(p, v);
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e)
            v[e] = none;
    }
}

// Lanes of a team beyond its last vector, teams beyond the last group or row.
struct RowsAt {
    int lane, slot, g;
    bool team;
    __device__ __forceinline__ RowsAt(const RowsPlan &p, int groups)
    {
        const int t = (int)threadIdx.x / p.L;
        lane = threadIdx.x % p.L;
        slot = t / p.gw;
        g = (int)(block_id() % p.windows) * p.gw + t % p.gw;
        team = slot < p.slots && g < groups;
    }
};

template <typename T, int V, int K, int R>
__global__ __launch_bounds__(256) void k_norm_rows(NormArgs a, RowsPlan p)
{
    const RowsAt at(p, a.groups);
    const long long n0 = (long long)(block_id() / p.windows) * p.slots * R + at.slot;
    if (!at.team || n0 >= a.N)
        return;         // whole teams; a team of 256 is the workgroup
    const int cg = a.C / a.groups, c0 = at.g * cg;
    // row j; rows behind the last are read as the last one and not stored
    auto row = [&](int j) { return min(n0 + (long long)j * p.slots, a.N - 1); };
    Raw<T, V> r[R][K];
#pragma unroll
    for (int j = 0; j < R; ++j)
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (at.lane + k * p.L) * V;
            r[j][k].clear();
            if (c < cg)
                r[j][k].load(static_cast<const T *>(a.x) + row(j) * a.ldx + c0 + c);
            // (through the caches, where a residual finds x again: 16384 rows of 2048
            // bfloat16 27.5 us for 29.0, with a sum of x and y behind it 60.6 for 66.3)
        }
    constexpr bool kEarly = K <= 2;     // w and b wait in registers
    float w[kEarly ? K : 1][V], b[kEarly ? K : 1][V];
    auto params = [&](int k, int to) {
        const int c = min((at.lane + k * p.L) * V, cg - V);
        get_all<V>(a.w ? a.w + c0 + c : nullptr, w[to], 1.0f);
        get_all<V>(a.b ? a.b + c0 + c : nullptr, b[to], 0.0f);
    };
    if constexpr (kEarly)
#pragma unroll
        for (int k = 0; k < K; ++k)
            params(k, k);
    float mean[R] = {}, q[R] = {};
#pragma unroll
    for (int j = 0; j < R; ++j)
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int v = 0; v < V; ++v)
                mean[j] += r[j][k].get(v);
    team_sum(mean, p.L);
#pragma unroll
    for (int j = 0; j < R; ++j) {
        mean[j] /= (float)cg;
#pragma unroll
        for (int k = 0; k < K; ++k)
            if ((at.lane + k * p.L) * V < cg)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const float d = r[j][k].get(v) - mean[j];
                    q[j] += d * d;
                }
    }
    team_sum(q, p.L);
    float rstd[R];
#pragma unroll
    for (int j = 0; j < R; ++j)
        rstd[j] = 1.0f / sqrtf(q[j] / (float)cg + a.eps);
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int c = (at.lane + k * p.L) * V, of = kEarly ? k : 0;
        if constexpr (!kEarly)
            params(k, 0);
#pragma unroll
        for (int j = 0; j < R; ++j) {
            float z[V];
#pragma unroll
            for (int v = 0; v < V; ++v)
                z[v] = (r[j][k].get(v) - mean[j]) * rstd[j] * w[of][v] + b[of][v];
            act_all(z, a.act);
            if (c < cg && n0 + (long long)j * p.slots < a.N)
                Raw<T, V>(z).store_past(static_cast<T *>(a.y) + row(j) * a.ldy + c0 + c);
        }
    }
    if (a.stats && at.lane == 0)
#pragma unroll
        for (int j = 0; j < R; ++j)
            if (n0 + (long long)j * p.slots < a.N) {
                float *to = a.stats + (row(j) * a.groups + at.g) * 2;
                to[0] = mean[j];
                to[1] = rstd[j];
            }
}

// dz of V elements and their xhat
template <int V>
__device__ __forceinline__ void dz_of(const float (&x)[V], const float (&dy)[V],
                                      const float (&w)[V], const float (&b)[V], float mean,
                                      float rstd, int act, float (&xhat)[V], float (&dz)[V])
{
#pragma unroll
    for (int v = 0; v < V; ++v)
        xhat[v] = (x[v] - mean) * rstd;
    if (act == DWCONV_ACT_NONE) {
#pragma unroll
        for (int v = 0; v < V; ++v)
            dz[v] = dy[v];
        return;
    }
    float z[V];
#pragma unroll
    for (int v = 0; v < V; ++v)
        z[v] = xhat[v] * w[v] + b[v];
    slope_all(z, act);
#pragma unroll
    for (int v = 0; v < V; ++v)
        dz[v] = dy[v] * z[v];
}

template <typename T, int V, int K>
__global__ __launch_bounds__(256) void k_norm_rows_grad(NormArgs a, RowsPlan p, float *part)
{
    extern __shared__ float sums[];     // [slots][2][gw * cg]
    const RowsAt at(p, a.groups);
    const int cg = a.C / a.groups, c0 = at.g * cg, wide = p.gw * cg;
    const long long first = block_id() / p.windows;
    if (first >= p.blocks)
        return;
    float dw[K][V] = {}, db[K][V] = {}, w[K][V], b[K][V];
    if (at.team)
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = min((at.lane + k * p.L) * V, cg - V);
            get_all<V>(a.w ? a.w + c0 + c : nullptr, w[k], 1.0f);
            get_all<V>(a.b ? a.b + c0 + c : nullptr, b[k], 0.0f);
        }
    if (at.team)        // a team of 256 is the workgroup: its lanes meet at barriers
        for (long long n = first * p.slots + at.slot; n < a.N; n += p.blocks * p.slots) {
            const T *x = static_cast<const T *>(a.x) + n * a.ldx + c0;
            const T *dy = static_cast<const T *>(a.dy) + n * a.lddy + c0;
            const float *st = a.stats_in + (n * a.groups + at.g) * 2;
            const float mean = st[0], rstd = st[1];
            float xhat[K][V], g[K][V], s[2] = {};
            Raw<T, V> rx[K], rd[K];
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int c = (at.lane + k * p.L) * V;
                if (c < cg) {
                    rx[k].load(x + c);
                    rd[k].load(dy + c);
                }
            }
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int c = (at.lane + k * p.L) * V;
                if (c < cg) {
                    float xv[V], dv[V], dz[V];
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        xv[v] = rx[k].get(v);
                        dv[v] = rd[k].get(v);
                    }
                    dz_of(xv, dv, w[k], b[k], mean, rstd, a.act, xhat[k], dz);
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        db[k][v] += dz[v];
                        dw[k][v] += dz[v] * xhat[k][v];
                        g[k][v] = dz[v] * w[k][v];
                        s[0] += g[k][v];
                        s[1] += g[k][v] * xhat[k][v];
                    }
                }
            }
            if (!a.dx)
                continue;
            team_sum(s, p.L);
            const float m1 = s[0] / (float)cg, m2 = s[1] / (float)cg;
            T *dx = static_cast<T *>(a.dx) + n * a.lddx + c0;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int c = (at.lane + k * p.L) * V;
                if (c < cg) {
#pragma unroll
                    for (int v = 0; v < V; ++v)
                        g[k][v] = rstd * (g[k][v] - m1 - xhat[k][v] * m2);
                    store<T, V>(dx + c, g[k]);
                }
            }
        }
    if (!a.dw && !a.db)
        return;
    if (p.slots == 1) {
        if (at.team)
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int c = (at.lane + k * p.L) * V;
                if (c < cg) {
                    store<float, V>(part + first * 2 * a.C + c0 + c, dw[k]);
                    store<float, V>(part + (first * 2 + 1) * a.C + c0 + c, db[k]);
                }
            }
        return;
    }
    float *mine = sums + at.slot * 2 * wide + (at.g % p.gw) * cg;
    if (at.team)
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int c = (at.lane + k * p.L) * V;
            if (c < cg)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    mine[c + v] = dw[k][v];
                    mine[wide + c + v] = db[k][v];
                }
        }
    __syncthreads();
    const int c_first = (int)(block_id() % p.windows) * wide;
    for (int i = threadIdx.x; i < 2 * wide; i += blockDim.x) {
        const int c = c_first + i % wide;
        if (c >= a.C)
            continue;
        float s = 0.0f;
        for (int k = 0; k < p.slots; ++k)
            s += sums[k * 2 * wide + i];
        part[(first * 2 + i / wide) * a.C + c] = s;
    }
}

// dw and db from `rows` rows of (dw, db): all of them, or (to != nullptr) strips of
// them, to be summed once more.
__global__ __launch_bounds__(1024) void k_norm_columns(const float *part, int rows, int strip,
                                                       int C, float *to, float *dw, float *db)
{
    const int first = (int)blockIdx.z * strip;
    column_sums(part + first * 2LL * C, min(strip, rows - first), 2LL * C,
                [=](long long n, float s) {
                    float *out = to ? to + blockIdx.z * 2LL * C : n < C ? dw : db;
                    if (out)
                        out[to || n < C ? n : n - C] = s;
                });
}

// Rows of sums that are added up by one workgroup for each 64 columns; more are
// taken in strips first.
constexpr int kStrips = 128;

int strip_of(long long rows)
{
    return rows <= 512 ? (int)std::max(rows, 1LL) : (int)cdiv(rows, kStrips);
}

int launch_columns(const float *part, long long rows, int C, float *space, float *dw, float *db,
                   hipStream_t st)
{
    const dim3 g = grid_of(cdiv(2LL * C, 64));
    const int strip = strip_of(rows), strips = (int)cdiv(rows, strip);
    if (strips > 1) {
        const int rc = dwconv::launch_kernel(k_norm_columns, dim3(g.x, g.y, strips), dim3(1024), 0,
                                             st, part, (int)rows, strip, C, space, nullptr,
                                             nullptr);
        if (rc != DWCONV_OK)
            return rc;
        part = space;
        rows = strips;
    }
    return dwconv::launch_kernel(k_norm_columns, g, dim3(1024), 0, st, part, (int)rows, (int)rows,
                                 C, nullptr, dw, db);
}

// ------------------------------------------------------------- P > 1
// A workgroup takes a range of rows of one instance and up to 256 vectors of V
// channels (whatever the groups): tx vectors, ty rows at a time.
struct RangePlan {
    int V, tx, ty, cols, chunk, chunks; // column blocks; rows of a range, ranges
    int span;                           // column blocks that a group lies in, at most
    bool joined;                        // the second pass joins the ranges by itself
    bool means;                         // ... or (gradient) adds up a group's channels
    bool past;                          // it reads past the caches
    long long total;                    // workgroups
};

constexpr int kAtOnce = 8;      // rows that a thread loads at a time
constexpr int kJoin = 64;       // ranges that each workgroup of the second pass may join
constexpr int kJoinMost = 512;  // and parts of a group in all
constexpr int kMeansMost = 512; // channels of a group that it may add up

// Ranges are whole batches of all threads (32 KB of x in 16-byte vectors), as many as
// make 2048 workgroups at most.
RangePlan range_plan(int size, bool grad, long long N, long long P, int C, int groups)
{
    RangePlan p;
    p.V = 16 / size;
    while (C % p.V)
        p.V /= 2;
    const int vectors = C / p.V;
    p.tx = std::min(vectors, 256);
    p.ty = 256 / p.tx;
    p.cols = (int)cdiv(vectors, 256);
    const int cg = C / groups, block = 256 * p.V;
    p.span = block % cg == 0 ? 1 : std::min(p.cols, (cg - 1) / block + 2);
    const long long unit = (long long)kAtOnce * p.ty;
    long long chunks = std::max(1LL, cdiv(2048, std::max(1LL, N * p.cols)));
    chunks = std::min(chunks, cdiv(P, unit));
    p.joined = !grad && chunks <= 2 * kJoin;
    if (p.joined)
        chunks = std::min(chunks, (long long)kJoin);
    // Each of a group's workgroups reads all of its parts, or sums, again: as many reads as the
    // square of the group's width.  More parts than a wave has under way at once are left to
    // a launch of their own, and so are a gradient's sums of more than 512 channels, where
    // that costs nothing (4 x 64 x 64 bfloat16, gradient: 512 channels 27.4 us for 27.4, 1024
    // 39.6 for 43.1; 512 x 32768 151 for 1346).
    p.joined = p.joined && chunks * p.span <= kJoinMost;
    p.means = !grad || cg <= kMeansMost;
    p.chunk = (int)std::min(cdiv(cdiv(P, chunks), unit) * unit, P);
    p.chunks = (int)cdiv(P, p.chunk);
    p.total = N * p.chunks * p.cols;
    // An x that fills the caches by itself is read for the last time past them (268 MB:
    // 137 us for 141, 280 for 282 with a sum of x and y behind it); a smaller one is left
    // there for who reads it next, a residual or the gradient (op and sum: 201 MB 204 us for
    // 212, 67 MB 72 for 79, 13 MB 24.3 for 25.6; the op alone within 5 % either way).
    p.past = (long long)size * N * P >= (256LL << 20) / C;
    return p;
}

// A workgroup's instance, range and columns, and a thread's vector and first row.
struct RangeAt {
    int n, chunk, col, y, rows, c;      // c: first channel, or C and more
    long long row0;
    __device__ __forceinline__ RangeAt(const RangePlan &p, long long P, int C, bool back)
    {
        unsigned b = block_id();
        if (back)
            b = (unsigned)(p.total - 1) - b;
        col = (int)(b % p.cols);
        b /= p.cols;
        chunk = (int)(b % p.chunks);
        n = (int)(b / p.chunks);
        y = (int)threadIdx.x / p.tx;
        c = y < p.ty ? (col * 256 + (int)threadIdx.x % p.tx) * p.V : C;
        row0 = n * P + (long long)chunk * p.chunk;
        rows = (int)min((long long)p.chunk, P - (long long)chunk * p.chunk);
    }
    // the block's channels
    __device__ __forceinline__ int first(const RangePlan &p) const { return col * 256 * p.V; }
    __device__ __forceinline__ int last(const RangePlan &p, int C) const
    {
        return min(C, (col + 1) * 256 * p.V);
    }
};

// Lanes that join a group's parts: as many as leave every group of `count` a team.
__device__ __forceinline__ int join_lanes(int count)
{
    int l = 64;
    while (l > 4 && l * count > 256)
        l /= 2;
    return l;
}

// A batch of a thread's rows, from row r of its range on and ty rows apart.  Rows
// behind the range's last one are read as that one (so that all loads go out at once)
// and weigh nothing.
template <typename T, int V, int B> struct Rows {
    Raw<T, V> v[B];
    // LAST: for the last time
    template <bool LAST>
    __device__ __forceinline__ void load(const T *x, long long ld, int r, const RangePlan &p,
                                         int rows)
    {
        const auto from = [&](int k) { return x + min(r + k * p.ty, rows - 1) * ld; };
        if (LAST && p.past) {
            // (the compiler would make one load of the two, without the hint)
            asm volatile("" ::: "memory");
#pragma unroll
            for (int k = 0; k < B; ++k)
                v[k].load_past(from(k));
            asm volatile("" ::: "memory");
        } else {
#pragma unroll
            for (int k = 0; k < B; ++k)
                v[k].load(from(k));
        }
    }
};

// Count, mean and sum of squares around it of some numbers.
struct Moments {
    float n, mean, m2;
    __device__ __forceinline__ void add(float bn, float bmean, float bm2)
    {
        const float all = n + bn, part = all > 0.0f ? bn / all : 0.0f, d = bmean - mean;
        mean += d * part;
        m2 += bm2 + (d * n) * (d * part);      // 0 for n = 0, however large d
        n = all;
    }
    __device__ __forceinline__ void add_lanes(int lanes)
    {
        for (int d = 1; d < lanes; d *= 2)
            add(__shfl_xor(n, d), __shfl_xor(mean, d), __shfl_xor(m2, d));
    }
};

// The mean and the sum of squares around it, per channel of a thread, of rows taken 8
// at a time: those of the 8 are exact to rounding and are joined to the rest.

template <typename T, int V>
__global__ __launch_bounds__(256) void k_range_stats(NormArgs a, RangePlan p, float2 *part)
{
    __shared__ float means[256 * V], squares[256 * V];
    if (block_id() >= p.total)
        return;
    const RangeAt at(p, a.P, a.C, false);
    float mean[V] = {}, m2[V] = {}, count = 0.0f;
    if (at.c < a.C) {
        const T *x = static_cast<const T *>(a.x) + at.row0 * a.ldx + at.c;
        for (int r = at.y; r < at.rows; r += kAtOnce * p.ty) {
            Rows<T, V, kAtOnce> in;
            in.template load<false>(x, a.ldx, r, p, at.rows);
            const int left = (at.rows - 1 - r) / p.ty + 1;
            const float n = (float)min(left, kAtOnce), one = 1.0f / n;
            const float all = count + n, part_of = n / all;
#pragma unroll
            for (int e = 0; e < V; ++e) {
                float s = 0.0f, q = 0.0f;
#pragma unroll
                for (int k = 0; k < kAtOnce; ++k)
                    s += k < left ? in.v[k].get(e) : 0.0f;
                s *= one;
#pragma unroll
                for (int k = 0; k < kAtOnce; ++k) {
                    const float d = k < left ? in.v[k].get(e) - s : 0.0f;
                    q += d * d;
                }
                const float d = s - mean[e];
                mean[e] += d * part_of;
                m2[e] += q + (d * count) * (d * part_of);
            }
            count = all;
        }
    }
#pragma unroll
    for (int e = 0; e < V; ++e) {
        means[threadIdx.x * V + e] = mean[e];
        squares[threadIdx.x * V + e] = m2[e];
    }
    __syncthreads();
    // the groups that the block's channels touch
    const int cg = a.C / a.groups, c_first = at.first(p), c_last = at.last(p, a.C);
    const int g0 = c_first / cg, touched = (c_last - 1) / cg - g0 + 1;
    const int lanes = join_lanes(touched), lane = threadIdx.x % lanes;
    for (int g = g0 + (int)threadIdx.x / lanes; g < g0 + touched; g += 256 / lanes) {
        const int lo = max(g * cg, c_first) - c_first, hi = min((g + 1) * cg, c_last) - c_first;
        const int wide = hi - lo, items = wide * p.ty;
        auto of = [&](int i, auto f) {          // item i: row slot i / wide
            const int y = i / wide, n = (at.rows - y + p.ty - 1) / p.ty;
            const int k = y * p.tx * V + lo + i % wide;
            if (n > 0)
                f((float)n, means[k], squares[k]);
        };
        float s = 0.0f, q = 0.0f;
        for (int i = lane; i < items; i += lanes)
            of(i, [&](float n, float m, float) { s += n * m; });
        for (int d = 1; d < lanes; d *= 2)
            s += __shfl_xor(s, d);
        const float joint = s / ((float)at.rows * (float)wide);
        for (int i = lane; i < items; i += lanes)
            of(i, [&](float n, float m, float m2) { q += m2 + n * (m - joint) * (m - joint); });
        for (int d = 1; d < lanes; d *= 2)
            q += __shfl_xor(q, d);
        if (lane == 0)
            part[(((long long)at.n * a.groups + g) * p.chunks + at.chunk) * p.span + at.col -
                 g * cg / (256 * p.V)] = make_float2(joint, q);
    }
}

// A lane's share (of `lanes`) of the ranges of group g of instance n.
__device__ __forceinline__ Moments join(const NormArgs &a, const RangePlan &p,
                                        const float2 *part, int n, int g, int lane, int lanes)
{
    const int cg = a.C / a.groups, block = 256 * p.V;
    const int col0 = g * cg / block, cols = ((g + 1) * cg - 1) / block - col0 + 1;
    const float2 *from = part + ((long long)n * a.groups + g) * p.chunks * p.span;
    const int items = p.chunks * cols;
    Moments sum{};
    for (int i = lane; i < items; i += 8 * lanes) {
        float2 v[8];
        float count[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const int j = min(i + k * lanes, items - 1);
            const int chunk = cols == 1 ? j : j / cols, c = j - chunk * cols, col = col0 + c;
            const long long rows = min((long long)p.chunk, a.P - (long long)chunk * p.chunk);
            const int wide = min((g + 1) * cg, (col + 1) * block) - max(g * cg, col * block);
            count[k] = i + k * lanes < items ? (float)rows * (float)wide : 0.0f;
            v[k] = from[(long long)chunk * p.span + c];
        }
#pragma unroll
        for (int k = 0; k < 8; ++k)
            sum.add(count[k], v[k].x, count[k] > 0.0f ? v[k].y : 0.0f);
    }
    return sum;
}

__device__ __forceinline__ float2 stats_of(const Moments &m, float eps)
{
    return make_float2(m.mean, 1.0f / sqrtf(m.m2 / m.n + eps));
}

// A workgroup for each group of each instance.
__global__ __launch_bounds__(256) void k_norm_join(NormArgs a, RangePlan p, const float2 *part,
                                                   float2 *stats)
{
    __shared__ Moments of[4];
    const long long id = block_id();
    if (id >= a.N * a.groups)
        return;
    Moments m = join(a, p, part, (int)(id / a.groups), (int)(id % a.groups), threadIdx.x, 256);
    m.add_lanes(64);
    if ((threadIdx.x & 63) == 0)
        of[threadIdx.x >> 6] = m;
    __syncthreads();
    if (threadIdx.x == 0) {
#pragma unroll
        for (int k = 1; k < 4; ++k)
            m.add(of[k].n, of[k].mean, of[k].m2);
        stats[id] = stats_of(m, a.eps);
    }
}

// The second pass.  stats: all groups', or nullptr where they are joined here.
template <typename T, int V>
__global__ __launch_bounds__(256) void k_range_apply(NormArgs a, RangePlan p, const float2 *part,
                                                     const float2 *stats)
{
    __shared__ float2 of[256 * V];
    if (block_id() >= p.total)
        return;
    const RangeAt at(p, a.P, a.C, true);
    const int cg = a.C / a.groups, c_first = at.first(p), c_last = at.last(p, a.C);
    const int g0 = c_first / cg, touched = (c_last - 1) / cg - g0 + 1;
    // the first rows are on their way while the ranges are joined
    const T *x = static_cast<const T *>(a.x) + at.row0 * a.ldx + min(at.c, a.C - V);
    Rows<T, V, kAtOnce> in;
    in.template load<true>(x, a.ldx, at.y, p, at.rows);
    if (stats) {
        for (int g = threadIdx.x; g < touched; g += 256)
            of[g] = stats[(long long)at.n * a.groups + g0 + g];
    } else {
        const int lanes = join_lanes(touched), lane = threadIdx.x % lanes;
        for (int g = (int)threadIdx.x / lanes; g < touched; g += 256 / lanes) {
            Moments m = join(a, p, part, at.n, g0 + g, lane, lanes);
            m.add_lanes(lanes);
            if (lane == 0) {
                const float2 v = stats_of(m, a.eps);
                of[g] = v;
                // the block of the group's first channel keeps them
                if (a.stats && at.chunk == 0 && (g0 + g) * cg >= c_first)
                    reinterpret_cast<float2 *>(
                        a.stats)[(long long)at.n * a.groups + g0 + g] = v;
            }
        }
    }
    __syncthreads();
    if (at.c >= a.C)
        return;
    float mean[V], f[V], w[V], b[V];
    get_all<V>(a.w ? a.w + at.c : nullptr, w, 1.0f);
    get_all<V>(a.b ? a.b + at.c : nullptr, b, 0.0f);
#pragma unroll
    for (int e = 0; e < V; ++e) {
        const float2 v = of[(at.c + e) / cg - g0];
        mean[e] = v.x;
        f[e] = v.y * w[e];
    }
    T *y = static_cast<T *>(a.y) + at.row0 * a.ldy + at.c;
    for (int r = at.y;;) {
#pragma unroll
        for (int k = 0; k < kAtOnce; ++k) {
            float z[V];
#pragma unroll
            for (int e = 0; e < V; ++e)
                z[e] = (in.v[k].get(e) - mean[e]) * f[e] + b[e];
            act_all(z, a.act);
            if (r + k * p.ty < at.rows)
                Raw<T, V>(z).store_past(y + (r + k * p.ty) * a.ldy);
        }
        r += kAtOnce * p.ty;
        if (r >= at.rows)
            return;
        in.template load<true>(x, a.ldx, r, p, at.rows);
    }
}

// Gradient, first pass: per range and channel sum(dz * xhat) and sum(dz).  16 x 64 x 64 x
// 320 float16, 32 groups, SiLU: 22 us, the fold 5, the second pass 25 (84 MB read by each).
template <typename T, int V>
__global__ __launch_bounds__(256) void k_range_sums(NormArgs a, RangePlan p, float *part)
{
    __shared__ float lds[2][256 * V];
    if (block_id() >= p.total)
        return;
    const RangeAt at(p, a.P, a.C, false);
    const int cg = a.C / a.groups;
    float dw[V] = {}, db[V] = {};
    if (at.c < a.C) {
        float mean[V], rstd[V], w[V], b[V];
        get_all<V>(a.w ? a.w + at.c : nullptr, w, 1.0f);
        get_all<V>(a.b ? a.b + at.c : nullptr, b, 0.0f);
#pragma unroll
        for (int e = 0; e < V; ++e) {
            const float *st = a.stats_in + ((long long)at.n * a.groups + (at.c + e) / cg) * 2;
            mean[e] = st[0];
            rstd[e] = st[1];
        }
        const T *x = static_cast<const T *>(a.x) + at.row0 * a.ldx + at.c;
        const T *dy = static_cast<const T *>(a.dy) + at.row0 * a.lddy + at.c;
        constexpr int B = kAtOnce / 2;
        for (int r = at.y; r < at.rows; r += B * p.ty) {
            Rows<T, V, B> rx, rd;
            rx.template load<false>(x, a.ldx, r, p, at.rows);
            rd.template load<false>(dy, a.lddy, r, p, at.rows);
#pragma unroll
            for (int k = 0; k < B; ++k) {
                float z[V], xhat[V];
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    xhat[e] = (rx.v[k].get(e) - mean[e]) * rstd[e];
                    z[e] = xhat[e] * w[e] + b[e];
                }
                slope_all(z, a.act);
                const bool counts = r + k * p.ty < at.rows;
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    const float dz = counts ? rd.v[k].get(e) * z[e] : 0.0f;
                    db[e] += dz;
                    dw[e] += dz * xhat[e];
                }
            }
        }
    }
#pragma unroll
    for (int e = 0; e < V; ++e) {
        lds[0][threadIdx.x * V + e] = dw[e];
        lds[1][threadIdx.x * V + e] = db[e];
    }
    __syncthreads();
    if (at.y != 0 || at.c >= a.C)
        return;
    for (int y = 1; y < p.ty; ++y)
#pragma unroll
        for (int e = 0; e < V; ++e) {
            dw[e] += lds[0][(y * p.tx + threadIdx.x) * V + e];
            db[e] += lds[1][(y * p.tx + threadIdx.x) * V + e];
        }
    float *to = part + ((long long)at.n * p.chunks + at.chunk) * 2 * a.C + at.c;
    store<float, V>(to, dw);
    store<float, V>(to + a.C, db);
}

// The ranges' sums of each instance: grid.y instances, 64 of the 2 C columns a workgroup.
__global__ __launch_bounds__(1024) void k_range_fold(const float *part, int chunks, int C,
                                                     long long N, float *sums)
{
    __shared__ float lds[16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const long long wide = 2LL * C;
    const unsigned blocks = (unsigned)((wide + 63) / 64);
    const long long n = block_id() / blocks, col = (long long)(block_id() % blocks) * 64 + lane;
    if (n >= N)
        return;
    const float *from = part + n * chunks * wide + col;
    float s = 0.0f;
    if (col < wide)
#pragma unroll 4
        for (int k = wave; k < chunks; k += 16)
            s += from[k * wide];
    lds[wave][lane] = s;
    __syncthreads();
    if (wave == 0 && col < wide) {
#pragma unroll
        for (int k = 1; k < 16; ++k)
            s += lds[k][lane];
        sums[n * wide + col] = s;
    }
}

// The means of a gradient of each group of each instance, a workgroup each.  (In 64 bits, as
// a thread may add up a great many.)
__global__ __launch_bounds__(256) void k_range_means(NormArgs a, const float *sums, float2 *means)
{
    __shared__ double2 of[4];
    const long long id = block_id();
    if (id >= a.N * a.groups)
        return;
    const int cg = a.C / a.groups, g = (int)(id % a.groups);
    const float *dw = sums + id / a.groups * 2 * a.C + (long long)g * cg, *db = dw + a.C;
    const float *w = a.w ? a.w + (long long)g * cg : nullptr;
    double s1 = 0.0, s2 = 0.0;
#pragma unroll 4
    for (int c = threadIdx.x; c < cg; c += 256) {
        const double f = w ? w[c] : 1.0f;
        s1 += f * db[c];
        s2 += f * dw[c];
    }
    for (int d = 1; d < 64; d *= 2) {
        s1 += __shfl_xor(s1, d);
        s2 += __shfl_xor(s2, d);
    }
    if ((threadIdx.x & 63) == 0)
        of[threadIdx.x >> 6] = make_double2(s1, s2);
    __syncthreads();
    if (threadIdx.x == 0) {
        const double all = (double)a.P * cg;
        means[id] = make_float2((float)(((of[0].x + of[1].x) + (of[2].x + of[3].x)) / all),
                                (float)(((of[0].y + of[1].y) + (of[2].y + of[3].y)) / all));
    }
}

// dw and db of 64 of the 2 C columns from the instances' sums.
constexpr int kInstances = 64;

__device__ __forceinline__ void add_instances(const NormArgs &a, const float *sums, int block,
                                              float *lds)
{
    const long long col = block * 64LL + (threadIdx.x & 63), wide = 2LL * a.C;
    const int wave = threadIdx.x >> 6;
    float s = 0.0f;
    if (col < wide)
#pragma unroll 4
        for (int n = wave; n < a.N; n += 4)
            s += sums[n * wide + col];
    lds[threadIdx.x] = s;
    __syncthreads();
    float *to = col < a.C ? a.dw : a.db;
    if (wave == 0 && col < wide && to)
        to[col < a.C ? col : col - a.C] =
            ((lds[threadIdx.x] + lds[threadIdx.x + 64]) + lds[threadIdx.x + 128]) +
            lds[threadIdx.x + 192];
}

// Gradient, second pass: dx, with the groups' means from their channels' sums (means:
// all groups', or nullptr where they are added up here).
template <typename T, int V>
__global__ __launch_bounds__(256) void k_range_dx(NormArgs a, RangePlan p, const float *sums,
                                                  const float2 *means)
{
    __shared__ float2 of[256 * V];
    if (block_id() >= p.total) {
        // workgroups behind those of dx, if there are any, add up dw and db
        add_instances(a, sums, (int)(block_id() - p.total), reinterpret_cast<float *>(of));
        return;
    }
    const RangeAt at(p, a.P, a.C, true);
    const int cg = a.C / a.groups, c_first = at.first(p), c_last = at.last(p, a.C);
    const int g0 = c_first / cg, touched = (c_last - 1) / cg - g0 + 1;
    constexpr int B = kAtOnce / 2;
    const T *x = static_cast<const T *>(a.x) + at.row0 * a.ldx + min(at.c, a.C - V);
    const T *dy = static_cast<const T *>(a.dy) + at.row0 * a.lddy + min(at.c, a.C - V);
    Rows<T, V, B> rx, rd;
    rx.template load<true>(x, a.ldx, at.y, p, at.rows);
    rd.template load<true>(dy, a.lddy, at.y, p, at.rows);
    if (means) {
        for (int g = threadIdx.x; g < touched; g += 256)
            of[g] = means[(long long)at.n * a.groups + g0 + g];
    } else {
        const int lanes = join_lanes(touched), lane = threadIdx.x % lanes;
        const float *dw = sums + (long long)at.n * 2 * a.C, *db = dw + a.C;
        const float all = (float)a.P * (float)cg;
        for (int g = (int)threadIdx.x / lanes; g < touched; g += 256 / lanes) {
            float s1 = 0.0f, s2 = 0.0f;
            for (int c = (g0 + g) * cg + lane; c < (g0 + g + 1) * cg; c += lanes) {
                const float w = a.w ? a.w[c] : 1.0f;
                s1 += w * db[c];
                s2 += w * dw[c];
            }
            for (int d = 1; d < lanes; d *= 2) {
                s1 += __shfl_xor(s1, d);
                s2 += __shfl_xor(s2, d);
            }
            if (lane == 0)
                of[g] = make_float2(s1 / all, s2 / all);
        }
    }
    __syncthreads();
    if (at.c >= a.C)
        return;
    float mean[V], rstd[V], w[V], b[V], m1[V], m2[V];
    get_all<V>(a.w ? a.w + at.c : nullptr, w, 1.0f);
    get_all<V>(a.b ? a.b + at.c : nullptr, b, 0.0f);
#pragma unroll
    for (int e = 0; e < V; ++e) {
        const int g = (at.c + e) / cg;
        const float *st = a.stats_in + ((long long)at.n * a.groups + g) * 2;
        mean[e] = st[0];
        rstd[e] = st[1];
        m1[e] = of[g - g0].x;
        m2[e] = of[g - g0].y;
    }
    T *dx = static_cast<T *>(a.dx) + at.row0 * a.lddx + at.c;
    for (int r = at.y;;) {
#pragma unroll
        for (int k = 0; k < B; ++k) {
            float z[V], xhat[V];
#pragma unroll
            for (int e = 0; e < V; ++e) {
                xhat[e] = (rx.v[k].get(e) - mean[e]) * rstd[e];
                z[e] = xhat[e] * w[e] + b[e];
            }
            slope_all(z, a.act);
#pragma unroll
            for (int e = 0; e < V; ++e)
                z[e] = rstd[e] * (rd.v[k].get(e) * z[e] * w[e] - m1[e] - xhat[e] * m2[e]);
            if (r + k * p.ty < at.rows)
                Raw<T, V>(z).store_past(dx + (r + k * p.ty) * a.lddx);
        }
        r += B * p.ty;
        if (r >= at.rows)
            return;
        rx.template load<true>(x, a.ldx, r, p, at.rows);
        rd.template load<true>(dy, a.lddy, r, p, at.rows);
    }
}

// ---------------------------------------------------------------- launching
long long round16(long long bytes) { return cdiv(bytes, 16) * 16; }

// The parts of a workspace.
struct Space {
    long long part, sums, strips, means, total;
};

Space space_of(bool grad, int size, long long N, long long P, int C, int groups)
{
    Space s{};
    RowsPlan rows;
    if (rows_plan(size, N, P, C, groups, &rows)) {
        if (grad)
            s.part = round16(8LL * rows.blocks * C);
    } else {
        const RangePlan p = range_plan(size, grad, N, P, C, groups);
        if (!grad) {
            s.part = round16(8LL * N * p.chunks * p.span * groups);
            s.sums = p.joined ? 0 : round16(8LL * N * groups);
        } else {
            s.part = round16(8LL * N * p.chunks * C);
            s.sums = p.chunks > 1 ? round16(8LL * N * C) : 0;
            s.strips = N > strip_of(N) ? round16(8LL * kStrips * C) : 0;
            s.means = p.means ? 0 : round16(8LL * N * groups);
        }
    }
    s.total = s.part + s.sums + s.strips + s.means;
    return s;
}

// f(vector of V elements) for V = 16 / sizeof(T), .., 1
template <typename T, typename F> int with_width(int V, F f)
{
    if constexpr (sizeof(T) == 2)
        if (V == 8)
            return f(std::integral_constant<int, 8>());
    switch (V) {
    case 4: return f(std::integral_constant<int, 4>());
    case 2: return f(std::integral_constant<int, 2>());
    default: return f(std::integral_constant<int, 1>());
    }
}

template <typename F> int with_keep(int K, F f)
{
    switch (K) {
    case 1: return f(std::integral_constant<int, 1>());
    case 2: return f(std::integral_constant<int, 2>());
    case 4: return f(std::integral_constant<int, 4>());
    default: return f(std::integral_constant<int, kRowsKeep>());
    }
}

constexpr long long kMostBlocks = 0x7fffffffLL;

}  // namespace

long long norm_workspace(bool grad, int type, long long N, long long P, int C, int groups)
{
    return N == 0 ? 0 : space_of(grad, dwseq::elem_size(type), N, P, C, groups).total;
}

int launch_norm_fwd(const NormArgs &a, void *stream)
{
    if (a.N == 0)
        return DWCONV_OK;
    hipStream_t st = static_cast<hipStream_t>(stream);
    const int size = elem_size(a.type);
    RowsPlan rows;
    if (rows_plan(size, a.N, a.P, a.C, a.groups, &rows)) {
        const long long blocks = cdiv(a.N, (long long)rows.slots * rows.R) * rows.windows;
        if (blocks > kMostBlocks)
            return DWCONV_ERR_BAD_DIM;
        return with_type(a.type, [&](auto *t) {
            using T = std::remove_pointer_t<decltype(t)>;
            return with_width<T>(rows.V, [&](auto v) {
                return with_keep(rows.K, [&](auto k) {
                    constexpr int R = k.value < 4 ? 4 / k.value : 1;
                    return dwconv::launch_kernel(rows.R == 1 ? k_norm_rows<T, v.value, k.value, 1>
                                                             : k_norm_rows<T, v.value, k.value, R>,
                                                 grid_of(blocks), dim3(rows.threads), 0, st, a,
                                                 rows);
                });
            });
        });
    }
    const RangePlan p = range_plan(size, false, a.N, a.P, a.C, a.groups);
    if (p.total > kMostBlocks)
        return DWCONV_ERR_BAD_DIM;
    const Space s = space_of(false, size, a.N, a.P, a.C, a.groups);
    float2 *part = static_cast<float2 *>(a.workspace);
    float2 *joint = reinterpret_cast<float2 *>(static_cast<char *>(a.workspace) + s.part);
    if (a.stats)
        joint = reinterpret_cast<float2 *>(a.stats);
    return with_type(a.type, [&](auto *t) {
        using T = std::remove_pointer_t<decltype(t)>;
        return with_width<T>(p.V, [&](auto v) {
            int rc = dwconv::launch_kernel(k_range_stats<T, v.value>, grid_of(p.total), dim3(256),
                                           0, st, a, p, part);
            if (rc == DWCONV_OK && !p.joined)
                rc = dwconv::launch_kernel(k_norm_join, grid_of(a.N * a.groups),
                                           dim3(256), 0, st, a, p, (const float2 *)part, joint);
            if (rc == DWCONV_OK)
                rc = dwconv::launch_kernel(k_range_apply<T, v.value>, grid_of(p.total), dim3(256),
                                           0, st, a, p, (const float2 *)part,
                                           p.joined ? nullptr : (const float2 *)joint);
            return rc;
        });
    });
}

int launch_norm_grad(const NormArgs &a, void *stream)
{
    hipStream_t st = static_cast<hipStream_t>(stream);
    const int size = elem_size(a.type);
    if (a.N == 0)       // the sums of no row
        return a.dw || a.db ? launch_columns(nullptr, 0, a.C, nullptr, a.dw, a.db, st) : DWCONV_OK;
    const Space s = space_of(true, size, a.N, a.P, a.C, a.groups);
    char *space = static_cast<char *>(a.workspace);
    float *part = reinterpret_cast<float *>(space);
    float *strips = reinterpret_cast<float *>(space + s.part + s.sums);
    RowsPlan rows;
    if (rows_plan(size, a.N, a.P, a.C, a.groups, &rows)) {
        const long long blocks = rows.blocks * rows.windows;
        if (blocks > kMostBlocks)
            return DWCONV_ERR_BAD_DIM;
        const size_t lds =
            rows.slots > 1 ? sizeof(float) * 2 * rows.slots * rows.gw * (a.C / a.groups) : 0;
        const int rc = with_type(a.type, [&](auto *t) {
            using T = std::remove_pointer_t<decltype(t)>;
            return with_width<T>(rows.V, [&](auto v) {
                return with_keep(rows.K, [&](auto k) {
                    return dwconv::launch_kernel(k_norm_rows_grad<T, v.value, k.value>,
                                                 grid_of(blocks), dim3(rows.threads), lds, st, a,
                                                 rows, part);
                });
            });
        });
        if (rc != DWCONV_OK || (!a.dw && !a.db))
            return rc;
        return launch_columns(part, rows.blocks, a.C, strips, a.dw, a.db, st);
    }
    const RangePlan p = range_plan(size, true, a.N, a.P, a.C, a.groups);
    float *sums = p.chunks > 1 ? reinterpret_cast<float *>(space + s.part) : part;
    float2 *means = reinterpret_cast<float2 *>(space + s.part + s.sums + s.strips);
    // up to kInstances of them are added up beside dx, more by launches of their own
    const bool beside = a.dx && (a.dw || a.db) && a.N <= kInstances;
    const long long extra = beside ? cdiv(2LL * a.C, 64) : 0;
    if (p.total + extra > kMostBlocks)
        return DWCONV_ERR_BAD_DIM;
    int rc = with_type(a.type, [&](auto *t) {
        using T = std::remove_pointer_t<decltype(t)>;
        return with_width<T>(p.V, [&](auto v) {
            int rc = dwconv::launch_kernel(k_range_sums<T, v.value>, grid_of(p.total), dim3(256),
                                           0, st, a, p, part);
            if (rc == DWCONV_OK && p.chunks > 1)
                rc = dwconv::launch_kernel(k_range_fold, grid_of(a.N * cdiv(2LL * a.C, 64)),
                                           dim3(1024), 0, st, (const float *)part, p.chunks, a.C,
                                           a.N, sums);
            if (rc == DWCONV_OK && a.dx && !p.means)
                rc = dwconv::launch_kernel(k_range_means, grid_of(a.N * a.groups), dim3(256), 0,
                                           st, a, (const float *)sums, means);
            if (rc == DWCONV_OK && a.dx)
                rc = dwconv::launch_kernel(k_range_dx<T, v.value>, grid_of(p.total + extra),
                                           dim3(256), 0, st, a, p, (const float *)sums,
                                           p.means ? nullptr : (const float2 *)means);
            return rc;
        });
    });
    if (rc != DWCONV_OK || (!a.dw && !a.db) || beside)
        return rc;
    return launch_columns(sums, a.N, a.C, strips, a.dw, a.db, st);
}

}  // namespace dwmix

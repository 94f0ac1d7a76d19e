// dwseq_gemm.h -- the tiled matrix product behind dwconv_linear_*, one
// translation unit per element type (dwseq_gemm_*.hip).
//
//   out[m, n] = finish(sum_k P[m, k] * Q[n, k])
//
// with P and Q read either along k ("K": a row per m or n, k contiguous) or
// across it ("R": a row per k), so that the forward (x, w: K K), the input
// gradient (dz: K, w: R) and the weight gradient (dz, x: R R) are one kernel.
//
// A workgroup computes a BM x BN tile in steps of 128 bytes of k (64 16-bit or
// 32 float32 elements), both operands' steps double-buffered in LDS in 16-byte
// chunks.  Where addresses and strides are multiples of 16 bytes the chunks go
// from memory to LDS directly (buffer loads to LDS; what lies outside the
// matrices reads as zero by the descriptor's bounds); elsewhere through
// registers.  The chunks of an LDS row are
// permuted (XOR by the row) so that the lanes of one LDS read fall on
// different banks; since a direct load fills LDS in lane order, the
// permutation is applied to the global address.
//
// Matrix instructions: 16x16x32 for 16-bit elements, 16x16x4 for float32 (four
// of them per fragment; k is summed in the same permuted order on both sides).
// Q's fragment is the first operand, so a lane ends with 4 adjacent n of one m:
// bias, residual and results move as 4-element vectors.  An R operand's
// 16-bit fragments come through the LDS transpose read, its float32 ones as
// four single reads (the float32 instructions are 16 times slower, so LDS has
// the time).
#pragma once

#include "dwseq_device.h"

namespace dwseq {

constexpr int kStepBytes = 128;     // of k that a step multiplies

// What happens to a sum on its way to memory.
struct Finish {
    const float *b;             // per column, or nullptr
    const void *res;            // nullptr: none
    void *z, *y;                // z nullptr: not kept
    long long ldres, ldz, ldy;
    int act;
    float *part;                // not nullptr: float32 partial sums [split][M][N] instead
};

// Which kernel a product runs with: tiles of that many rows and columns (the
// DEEP one with more steps on their way), or the one for few rows.
enum GemmTile { TILE_256, TILE_128, TILE_64, TILE_64_DEEP, FEW_ROWS };
constexpr int kFewRows = 64;    // that the last one takes at most

struct Product {
    const void *p, *q;
    long long ldp, ldq;
    bool p_rows_k, q_rows_k;    // R: a row per k
    int M, N, K;
    GemmTile tile;
    int splits;                 // of k, each with a multiple of a step's length
    Finish f;
};

template <typename T> int launch_gemm(const Product &p, hipStream_t st);

// Whether an operand's chunks can go to LDS directly.
inline bool direct_ok(const void *p, long long ld, bool rows_k, int K, int size)
{
    return (reinterpret_cast<std::uintptr_t>(p) % 16) == 0 && (ld * size) % 16 == 0 &&
           (rows_k || ((long long)K * size) % 16 == 0);
}

// The kernel that runs for a plan's tile: the 256 tile is for 16-bit operands
// that go to LDS directly, and so is the deep ring.
inline GemmTile tile_taken(GemmTile tile, bool direct, int size)
{
    if (direct && size == 2)
        return tile;
    return tile == TILE_256 ? TILE_128 : tile == TILE_64_DEEP ? TILE_64 : tile;
}

// The length of k's ranges for a plan's number of them, and how many of these
// there are: a multiple of a step's length, none of them empty.
inline int split_length(int K, int splits, int size)
{
    const int step = kStepBytes / size;
    return (int)(cdiv(cdiv(K, step), splits) * step);
}
inline int split_count(int K, int splits, int size)
{
    return K ? (int)cdiv(K, split_length(K, splits, size)) : 1;
}

#ifdef DWSEQ_GEMM_KERNELS
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef f16 f16x8 __attribute__((ext_vector_type(8)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));

typedef __attribute__((address_space(3))) char *lds_ptr;
typedef __attribute__((address_space(3))) f32x4 *lds_f32x4;

constexpr int kFar = 0x7ffffff0;    // beyond every descriptor's bounds

template <typename T>
__device__ __forceinline__ void mma(const u32x4 &a, const u32x4 &b, f32x4 &c)
{
    if constexpr (std::is_same_v<T, bf16>) {
        c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a),
                                                    __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
    } else if constexpr (std::is_same_v<T, f16>) {
        c = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8, a),
                                                   __builtin_bit_cast(f16x8, b), c, 0, 0, 0);
    } else {
        const f32x4 fa = __builtin_bit_cast(f32x4, a), fb = __builtin_bit_cast(f32x4, b);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            c = __builtin_amdgcn_mfma_f32_16x16x4f32(fa[j], fb[j], c, 0, 0, 0);
    }
}

// One operand's step in LDS: ROWS rows of the tile (m or n) by kStepBytes of k.
// R = false: [row][8 chunks of k]; R = true: [k][chunks of rows].
template <typename T, int ROWS, bool R, int THREADS> struct Operand {
    static constexpr int size = (int)sizeof(T);
    static constexpr int elems = 16 / size;              // of a chunk
    static constexpr int step = kStepBytes / size;       // k per step
    static constexpr int bytes = ROWS * kStepBytes;
    static constexpr int count = bytes / 16 / THREADS;   // chunks a thread moves
    static constexpr int per_row = R ? ROWS / elems : 8;

    // where chunk c of LDS row `row` is kept
    static __device__ __forceinline__ int place(int row, int c)
    {
        if constexpr (!R)
            return c ^ ((row >> 1) & 7);
        else if constexpr (size == 2)
            return (c ^ (((row & 3) | (((row >> 3) & 1) << 2)) << 1)) & (per_row - 1);
        else
            return (c ^ (((row >> 2) & 3) << 2)) & (per_row - 1);
    }

    const char *base;       // of the tile's first row (R: first column), k = 0
    long long ld;           // bytes
    int rows, K;            // rows that the tile has (ROWS at most), k in all

    __device__ __forceinline__ Operand(const void *p, long long ld_elems, int row0, int all, int K_)
        : base(static_cast<const char *>(p) + (R ? (long long)row0 * size
                                                 : row0 * ld_elems * size)),
          ld(ld_elems * size), rows(min(all - row0, ROWS)), K(K_)
    {
    }

    // The step at k0 in memory: where it starts and how many bytes it has, none
    // past the last step or in a half with no row.  (Before the last step another
    // row of k follows an R operand's, so that its last element is in bounds by
    // whole words.)
    __device__ __forceinline__ const char *step_at(int k0) const
    {
        return base + (R ? (long long)k0 * ld : (long long)k0 * size);
    }
    __device__ __forceinline__ int bytes_at(int k0) const
    {
        const int left = K - k0;
        if (left <= 0 || rows <= 0)
            return 0;
        if (R)
            return left > step ? step * (int)ld + size : (left - 1) * (int)ld + rows * size;
        return (rows - 1) * (int)ld + left * size;
    }

    // Chunk number `idx` of a step is LDS row idx / per_row; its chunk of the
    // matrix is place() of it (an involution).
    __device__ __forceinline__ void stage_direct(char *lds, int k0, int wave, int lane) const
    {
        const int left = K - k0;
        // bounds are in whole words: round up to the word, which is aligned here,
        // that holds the last element
        const __amdgpu_buffer_rsrc_t rsrc =
            dwconv::make_rsrc(step_at(k0), (bytes_at(k0) + 3) & ~3);
#pragma unroll
        for (int j = 0; j < count; ++j) {
            const int first = (j * (THREADS / 64) + wave) * 64, idx = first + lane;
            const int row = idx / per_row, c = place(row, idx % per_row);
            int off = row * (int)ld + c * 16;
            if (!R && left < step)      // the last step alone
                off = c * elems >= left ? kFar : off;
            __builtin_amdgcn_raw_ptr_buffer_load_lds(
                rsrc, (__attribute__((address_space(3))) void *)(lds + first * 16), 16, off, 0, 0,
                0);
        }
    }

    // The same into registers, from any address, and with a last chunk that k
    // does not fill: what follows in its row is cut off in keep().
    __device__ __forceinline__ void fetch(u32x4 (&regs)[count], int k0, int tid) const
    {
        const int end = bytes_at(k0);
        const __amdgpu_buffer_rsrc_t rsrc = dwconv::make_rsrc(step_at(k0), end);
#pragma unroll
        for (int j = 0; j < count; ++j) {
            const int idx = j * THREADS + tid, row = idx / per_row, c = place(row, idx % per_row);
            const int off = row * (int)ld + c * 16;
            regs[j] = __builtin_bit_cast(
                u32x4, __builtin_amdgcn_raw_buffer_load_b128(rsrc, off, 0, 0));
            // a word that the array's last element fills by half is out of bounds:
            // that element by itself
            if (size == 2 && K - k0 <= step && ((end | (int)ld) & 2)) {
                const int last = end - 2 - off;
                const bool here = last >= 0 && last < 16 && (last & 3) == 0;
                const unsigned v =
                    __builtin_amdgcn_raw_buffer_load_b16(rsrc, here ? end - 2 : kFar, 0, 0);
#pragma unroll
                for (int w = 0; w < 4; ++w)
                    regs[j][w] |= here && last == w * 4 ? v & 0xffffu : 0u;
            }
        }
    }

    __device__ __forceinline__ void keep(char *lds, u32x4 (&regs)[count], int k0, int tid) const
    {
        const int left = K - k0;
        if (!R && left < step)
#pragma unroll
            for (int j = 0; j < count; ++j) {
                const int idx = j * THREADS + tid;
                const int in = left - place(idx / per_row, idx % per_row) * elems;  // of the chunk
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    constexpr int per_word = 4 / size;
                    const unsigned half = per_word == 2 && in == w * 2 + 1 ? 0xffffu : 0u;
                    regs[j][w] &= in >= (w + 1) * per_word ? ~0u : half;
                }
            }
#pragma unroll
        for (int j = 0; j < count; ++j)
            *reinterpret_cast<u32x4 *>(lds + (j * THREADS + tid) * 16) = regs[j];
    }
};

// The fragments that a lane reads of an operand's step: N of them, each 16
// rows, from row0 on.  What differs between them and between the two parts of
// the step's k is a constant offset where the permutation allows, so that it
// goes into the instruction: rows 16 apart (K) are permuted alike, and so are
// the two parts of k (R).
template <typename T, int ROWS, bool R, int N> struct Fragments {
    static constexpr int size = (int)sizeof(T), elems = 16 / size;
    static constexpr int line = R ? ROWS * size : kStepBytes;      // bytes of a row in LDS
    static constexpr int count = R ? N : 2;
    using Op = Operand<T, ROWS, R, 64>;
    lds_ptr at[count];

    __device__ __forceinline__ Fragments(char *lds, int row0, int lane)
    {
        const lds_ptr base = (lds_ptr)lds;
        const int g = lane >> 4, i = lane & 15;
#pragma unroll
        for (int c = 0; c < count; ++c) {
            if constexpr (!R) {
                at[c] = base + (row0 + i) * line + Op::place(row0 + i, c * 4 + g) * 16;
            } else if constexpr (size == 2) {
                const int k = g * 8 + (i >> 2);
                at[c] = base + k * line +
                        Op::place(k, row0 / elems + c * 2 + ((i & 3) >> 1)) * 16 + (i & 1) * 8;
            } else {
                const int k = g * 4;
                at[c] = base + k * line + Op::place(k, row0 / elems + c * 4 + (i >> 2)) * 16 +
                        (i & 3) * 4;
            }
        }
    }

    // the same fragments `bytes` further on in LDS, as addresses of their own
    __device__ __forceinline__ Fragments moved(int bytes) const
    {
        Fragments f = *this;
#pragma unroll
        for (int c = 0; c < count; ++c) {
            f.at[c] += bytes;
            asm("" : "+v"(f.at[c]));
        }
        return f;
    }

    // fragment f, part ks (of two) of the step's k, `offset` bytes further on
    __device__ __forceinline__ u32x4 read(int f, int ks, int offset) const
    {
        if constexpr (!R) {
            return *(__attribute__((address_space(3))) const u32x4 *)(at[ks] + f * 16 * line +
                                                                      offset);
        } else if constexpr (size == 2) {
            u32x4 v;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const s16x4 t = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (__attribute__((address_space(3))) s16x4 *)(at[f] + (ks * 32 + h * 4) * line +
                                                                offset));
                const uint2 w = __builtin_bit_cast(uint2, t);
                v[h * 2] = w.x;
                v[h * 2 + 1] = w.y;
            }
            return v;
        } else {
            u32x4 v;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                v[j] = *(__attribute__((address_space(3))) const unsigned *)(
                    at[f] + (ks * 16 + j) * line + offset);
            return v;
        }
    }
};

// Vectors of V columns, of which the first `width` exist.
template <typename E, int V>
__device__ __forceinline__ void get(const E *p, int width, float (&v)[V])
{
    if (width >= V) {
        load<E, V>(p, v);
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e)
            v[e] = e < width ? (float)p[e] : 0.0f;
    }
}

template <typename E, int V>
__device__ __forceinline__ void put(E *p, int width, const float (&v)[V])
{
    if (width >= V) {
        store<E, V>(p, v);
    } else {
#pragma unroll
        for (int e = 0; e < V; ++e)
            if (e < width)
                p[e] = (E)v[e];
    }
}

// The residuals of V adjacent sums of row m, from column n on.
template <typename T, int V>
__device__ __forceinline__ void residual(const Finish &f, long long m, int n, int width,
                                         Raw<T, V> &r)
{
    const T *p = static_cast<const T *>(f.res) + m * f.ldres + n;
    if (width >= V) {
        r.load(p);
    } else {
        float v[V];
        get(p, width, v);
        r = Raw<T, V>(v);
    }
}

// V adjacent sums of row m, from column n on; b: their biases, r: residuals
template <typename T, int V>
__device__ __forceinline__ void finish(const Finish &f, long long m, int n, int width,
                                       const float (&b)[V], const Raw<T, V> &r, float (&s)[V])
{
#pragma unroll
    for (int e = 0; e < V; ++e)
        s[e] += b[e];
    if (f.z)
        put(static_cast<T *>(f.z) + m * f.ldz + n, width, s);
    act_all(s, f.act);
    if (f.res)
#pragma unroll
        for (int e = 0; e < V; ++e)
            s[e] += r.get(e);
    put(static_cast<T *>(f.y) + m * f.ldy + n, width, s);
}

// The activation, and whether a tile has vectors of V columns that N cuts, as
// constants: one branch for a tile, and the code that runs lies in one piece
// (with the choices made row by row, the 256 tile's end was longer than the
// instruction cache).
template <typename F> __device__ __forceinline__ void with_act(int act, F f)
{
    switch (act) {
    case DWCONV_ACT_SILU: f(std::integral_constant<int, DWCONV_ACT_SILU>()); break;
    case DWCONV_ACT_RELU: f(std::integral_constant<int, DWCONV_ACT_RELU>()); break;
    case DWCONV_ACT_RELU6: f(std::integral_constant<int, DWCONV_ACT_RELU6>()); break;
    default: f(std::integral_constant<int, DWCONV_ACT_NONE>()); break;
    }
}

template <int V, typename F> __device__ __forceinline__ void with_cut(int left, int cols, F f)
{
    if (left < cols && left % V != 0)
        f(std::true_type());
    else
        f(std::false_type());
}

// The rows from m0 and columns from n0 on that a tile has in a matrix, of which a
// lane moves V adjacent columns from `col` on of row `line` + `row` (`line` the
// same in the wave).  The descriptor ends with the tile's last row, so that
// rows beyond M are neither read (as zero) nor written; lanes beyond N are sent out
// of bounds.  CUT: a vector that N cuts moves by element.
template <typename E, int V, bool CUT> struct Block {
    static constexpr int size = (int)sizeof(E);
    const char *base;
    int ld, bytes, left;        // bytes of a row's stride and in all; columns to N

    __device__ __forceinline__ Block(const void *p, long long ld_elems, int m0, int n0, int rows,
                                     int M, int N)
        : base(static_cast<const char *>(p) + (m0 * ld_elems + n0) * size),
          ld((int)ld_elems * size), bytes((min(M - m0, rows) - 1) * ld + (N - n0) * size),
          left(N - n0)
    {
    }
    __device__ __forceinline__ int at(int line, int col) const
    {
        return col + V <= left ? line * ld + col * size : kFar;
    }
    __device__ __forceinline__ int at(int line, int col, int e) const
    {
        return col + V > left && col + e < left ? line * ld + (col + e) * size : kFar;
    }
    __device__ __forceinline__ void load(Raw<E, V> &v, int line, int row, int col) const
    {
        const __amdgpu_buffer_rsrc_t rsrc = dwconv::make_rsrc(base, bytes);
        v.load(rsrc, at(line, col), row * ld);
        if constexpr (CUT)
#pragma unroll
            for (int e = 0; e < V - 1; ++e) {
                Raw<E, 1> one;
                one.load(rsrc, at(line, col, e), row * ld);
                v.w[e * size / 4] |= one.w[0] << (e * size % 4 * 8);
            }
    }
    __device__ __forceinline__ void store(const float (&s)[V], int line, int row, int col) const
    {
        const __amdgpu_buffer_rsrc_t rsrc = dwconv::make_rsrc(base, bytes);
        Raw<E, V>(s).store(rsrc, at(line, col), row * ld);
        if constexpr (CUT)
#pragma unroll
            for (int e = 0; e < V - 1; ++e) {
                const float one[1] = {s[e]};
                Raw<E, 1>(one).store(rsrc, at(line, col, e), row * ld);
            }
    }
};

// V adjacent sums of a tile on their way to memory; b: their biases, r: residuals
template <int ACT, typename T, int V, bool CUT>
__device__ __forceinline__ void finish(const Finish &f, const Block<T, V, CUT> &z,
                                       const Block<T, V, CUT> &y, const float (&b)[V],
                                       const Raw<T, V> &r, float (&s)[V], int line, int row,
                                       int col)
{
#pragma unroll
    for (int e = 0; e < V; ++e)
        s[e] += b[e];
    if (f.z)
        z.store(s, line, row, col);
#pragma unroll
    for (int e = 0; e < V; ++e)
        s[e] = act_of(s[e], ACT);
    if (f.res)
#pragma unroll
        for (int e = 0; e < V; ++e)
            s[e] += r.get(e);
    y.store(s, line, row, col);
}

// The tiles' grid: x, and past kGridRow tiles z too; y numbers the ranges of k.
// The number of this workgroup's tile may be one too many.
inline dim3 tile_grid(long long tiles, int splits)
{
    const dim3 g = grid_of(tiles);
    return dim3(g.x, (unsigned)splits, g.y);
}
__device__ __forceinline__ int tile_id() { return (int)(blockIdx.z * kGridRow + blockIdx.x); }

// Tile of workgroup b: each XCD (b % 8) takes a contiguous range of the tiles,
// which are numbered in bands of 8 tile rows, down the band first, so that the
// tiles at work in one XCD share rows of P and Q in its L2.
__device__ __forceinline__ void tile_of(int b, int tiles_m, int tiles_n, int &tm, int &tn)
{
    const int t = dwconv::xcd_tile(b, tiles_m * tiles_n);
    const int band = t / (8 * tiles_n), in = t - band * 8 * tiles_n;
    const int height = min(8, tiles_m - band * 8);
    tm = band * 8 + in % height;
    tn = in / height;
}

// vmcnt(n), lgkmcnt(0)
template <int N> __device__ __forceinline__ void wait_loads()
{
    __builtin_amdgcn_s_waitcnt((N & 15) | (7 << 4) | ((N >> 4) << 14));
}

// A workgroup barrier that nothing is moved across and that waits for no load.
__device__ __forceinline__ void bare_barrier()
{
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// ---------------------------------------------------------------------------
// The tiles of 128 and 64.  Direct: a ring of STAGES steps in LDS, STAGES - 1 of
// them on their way while one is multiplied; the one barrier of a step says both
// that every wave's share of the step has arrived and that the stage before it
// may be refilled.  Otherwise two stages, the steps after them
// in registers.
//
// Bound by LDS and latency: a 128 tile reads each fragment for 4 others
// (the 256 tile's hold 8).  Measured: 128 tile, weight gradient of 8192 x 4096 x
// 2048 bfloat16 155 us (887 TFLOP/s, matrix instructions busy 36% of the time), float32
// 4096 x 2048 x 2048 261 us (132 TFLOP/s, the matrix instructions' own 157); 64 tile,
// float32 25088 x 256 x 128 with bias and ReLU6 22.5 us among other calls (24.7 in a
// trace, from its own beginning to its end), of which 6 are its bytes: a tile has 4
// steps, so its beginning and end are not hidden; with 4 stages, bfloat16 1024^3 8.9
// us; through registers, 4001 x 4003 x 4005 204 us (628 TFLOP/s: one step in flight).
// ---------------------------------------------------------------------------
template <typename T, bool PR, bool QR, bool DIRECT, int BM, int BN, int WM, int WN, int STAGES>
__global__ __launch_bounds__(WM *WN * 64) void k_gemm(Product a, int tiles_m, int tiles_n,
                                                      int k_per_split)
{
    constexpr int kThr = WM * WN * 64;
    using P = Operand<T, BM, PR, kThr>;
    using Q = Operand<T, BN, QR, kThr>;
    constexpr int MF = BM / WM / 16, NF = BN / WN / 16, stage_bytes = P::bytes + Q::bytes;
    static_assert(DIRECT || STAGES == 2, "registers hold one step");
    __shared__ alignas(16) char lds[STAGES * stage_bytes];
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int split = blockIdx.y, k_first = split * k_per_split;
    const int k_last = min(k_first + k_per_split, a.K);
    if (tile_id() >= tiles_m * tiles_n)
        return;
    int tm, tn;
    tile_of(tile_id(), tiles_m, tiles_n, tm, tn);
    const P p(a.p, a.ldp, tm * BM, a.M, k_last);
    const Q q(a.q, a.ldq, tn * BN, a.N, k_last);
    const int wm = (wave / WN) * (BM / WM), wn = (wave % WN) * (BN / WN);

    // float32 sums are moved to a total every 4 steps: K / 4 roundings in a row
    // would cost a bit or two of the result
    constexpr bool kTotal = std::is_same_v<T, float>;
    f32x4 acc[NF][MF], total[kTotal ? NF : 1][kTotal ? MF : 1];
#pragma unroll
    for (int n = 0; n < NF; ++n)
#pragma unroll
        for (int m = 0; m < MF; ++m) {
            acc[n][m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
            if constexpr (kTotal)
                total[n][m] = acc[n][m];
        }
    auto to_total = [&] {
        if constexpr (kTotal) {
#pragma unroll
            for (int n = 0; n < NF; ++n)
#pragma unroll
                for (int m = 0; m < MF; ++m) {
                    total[n][m] += acc[n][m];
                    acc[n][m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
                }
        }
    };

    const Fragments<T, BM, PR, MF> at_p(lds, wm, lane);
    const Fragments<T, BN, QR, NF> at_q(lds + P::bytes, wn, lane);
    auto compute = [&](int offset) {
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
            u32x4 fp[MF], fq[NF];
#pragma unroll
            for (int m = 0; m < MF; ++m)
                fp[m] = at_p.read(m, ks, offset);
#pragma unroll
            for (int n = 0; n < NF; ++n)
                fq[n] = at_q.read(n, ks, offset);
#pragma unroll
            for (int n = 0; n < NF; ++n)
#pragma unroll
                for (int m = 0; m < MF; ++m)
                    mma<T>(fq[n], fp[m], acc[n][m]);
        }
    };
    const int steps = (k_last - k_first + P::step - 1) / P::step;
    if constexpr (DIRECT) {
        constexpr int loads = P::count + Q::count;     // of a wave, per step
        auto send = [&](int step, int slot) {
            char *to = lds + slot * stage_bytes;
            p.stage_direct(to, k_first + step * P::step, wave, lane);
            q.stage_direct(to + P::bytes, k_first + step * P::step, wave, lane);
        };
#pragma unroll
        for (int e = 0; e < STAGES - 1; ++e)
            send(e, e);
        int slot = 0;
        for (int s = 0; s < steps; ++s) {
            wait_loads<(STAGES - 2) * loads>();
            bare_barrier();
            send(s + STAGES - 1, slot == 0 ? STAGES - 1 : slot - 1);
            compute(slot * stage_bytes);
            if ((s & 3) == 3)
                to_total();
            slot = slot == STAGES - 1 ? 0 : slot + 1;
        }
        // a wave may not end with loads to its workgroup's LDS on their way
        wait_loads<0>();
    } else if (steps > 0) {
        // the next `ahead` steps wait in registers, or are on their way there
        constexpr int ahead = BM == 64 ? 3 : 1;
        u32x4 rp[ahead][P::count], rq[ahead][Q::count];
        auto fetch = [&](int step, auto d) {
            p.fetch(rp[d.value], k_first + step * P::step, tid);
            q.fetch(rq[d.value], k_first + step * P::step, tid);
        };
        auto settle = [&](int s, auto d) {
            char *to = lds + (s & 1) * stage_bytes;
            p.keep(to, rp[d.value], k_first + s * P::step, tid);
            q.keep(to + P::bytes, rq[d.value], k_first + s * P::step, tid);
            __syncthreads();
        };
        // step s, whose registers are number d
        auto one = [&](int s, auto d) {
            if (s >= steps)
                return;
            settle(s, d);
            fetch(s + ahead, d);
            compute((s & 1) * stage_bytes);
            if ((s & 3) == 3)
                to_total();
        };
        constexpr std::integral_constant<int, 0> d0;
        constexpr std::integral_constant<int, ahead == 3 ? 1 : 0> d1;
        constexpr std::integral_constant<int, ahead == 3 ? 2 : 0> d2;
        fetch(0, d0);
        if constexpr (ahead == 3) {
            fetch(1, d1);
            fetch(2, d2);
        }
        for (int s = 0; s < steps; s += ahead) {
            one(s, d0);
            if constexpr (ahead == 3) {
                one(s + 1, d1);
                one(s + 2, d2);
            }
        }
    }
    to_total();
    const int m0 = tm * BM, n0 = tn * BN, line = lane & 15, first = wn + (lane >> 4) * 4;
    auto sums_of = [&](int n, int m, float (&sum)[4]) {
        const f32x4 v = kTotal ? total[kTotal ? n : 0][kTotal ? m : 0] : acc[n][m];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            sum[e] = v[e];
    };
    with_cut<4>(a.N - n0, BN, [&](auto c) {
        constexpr bool CUT = decltype(c)::value;
        if (a.f.part) {
            const Block<float, 4, CUT> out(a.f.part + (long long)split * a.M * a.N, a.N, m0, n0,
                                           BM, a.M, a.N);
#pragma unroll
            for (int n = 0; n < NF; ++n)
#pragma unroll
                for (int m = 0; m < MF; ++m) {
                    float sum[4];
                    sums_of(n, m, sum);
                    out.store(sum, line, wm + m * 16, first + n * 16);
                }
            return;
        }
        const Block<T, 4, CUT> res(a.f.res, a.f.ldres, m0, n0, BM, a.M, a.N),
            z(a.f.z, a.f.ldz, m0, n0, BM, a.M, a.N), y(a.f.y, a.f.ldy, m0, n0, BM, a.M, a.N);
        const Block<float, 4, CUT> bias(a.f.b, 0, 0, n0, 1, 1, a.N);
        with_act(a.f.act, [&](auto act) {
#pragma unroll
            for (int n = 0; n < NF; ++n) {
                const int col = first + n * 16;
                Raw<T, 4> r[MF];
                Raw<float, 4> bn;
                bn.clear();
                if (a.f.b)
                    bias.load(bn, 0, 0, col);
                const float b[4] = {bn.get(0), bn.get(1), bn.get(2), bn.get(3)};
                if (a.f.res)
#pragma unroll
                    for (int m = 0; m < MF; ++m)
                        res.load(r[m], line, wm + m * 16, col);
#pragma unroll
                for (int m = 0; m < MF; ++m) {
                    float sum[4];
                    sums_of(n, m, sum);
                    finish<decltype(act)::value>(a.f, z, y, b, r[m], sum, line, wm + m * 16, col);
                }
            }
        });
    });
}

// ---------------------------------------------------------------------------
// The 256 x 256 tile, for operands that go to LDS directly.  8 waves, 4 along m
// and 2 along n, for 16-bit elements; each operand's step lies in LDS as two
// halves of 128 rows, and
// a wave computes one quadrant (half of its P, half of its Q) a phase:
//
//   phase 0: (P0, Q0)   1: (P0, Q1)   2: (P1, Q1)   3: (P1, Q0)
//
// so that a phase reads one half from LDS into registers and each half is read
// once.  Waves 0-3 and 4-7 (one of each on every SIMD) run half a phase apart: while
// one group's matrix instructions run, the other reads LDS and sends off loads.
// A half whose last reader is done is refilled at once, two steps ahead: every
// phase sends one half (2 loads a wave) and waits until at most 5 halves are on
// their way, which covers what the next phase reads.  Past the last step the
// loads' descriptors are empty, so the count stays the same.
//
// Measured: 8192^3 bfloat16 1505 TFLOP/s with both operands along k (1343 to 1368 on
// another card), 1220 with one and 1100 with both across it (two LDS reads a
// fragment); the matrix instructions are busy 76% of the time at the clock that the card's
// power allows.  16384 x 8192 x 2048 with bias, SiLU and residual 486 to 510 us:
// the product 418, and the residuals' 268 MB, which wait for the product's
// registers (touching their lines some steps earlier gained nothing).
// ---------------------------------------------------------------------------
constexpr int kPitch = 256 * 4 + 16;      // bytes of a row of sums in LDS

template <typename T, bool PR, bool QR>
__global__ __launch_bounds__(512) void k_gemm_256(Product a, int tiles_m, int tiles_n,
                                                  int k_per_split)
{
    using P = Operand<T, 128, PR, 512>;
    using Q = Operand<T, 128, QR, 512>;
    constexpr int half = P::bytes;
    __shared__ alignas(16) char lds[128 * kPitch];
    static_assert(8 * half <= sizeof(lds), "two steps of both operands");
    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int split = blockIdx.y, k_first = split * k_per_split;
    const int k_last = min(k_first + k_per_split, a.K);
    if (tile_id() >= tiles_m * tiles_n)
        return;
    int tm, tn;
    tile_of(tile_id(), tiles_m, tiles_n, tm, tn);
    const P p0(a.p, a.ldp, tm * 256, a.M, k_last), p1(a.p, a.ldp, tm * 256 + 128, a.M, k_last);
    const Q q0(a.q, a.ldq, tn * 256, a.N, k_last), q1(a.q, a.ldq, tn * 256 + 128, a.N, k_last);
    const int wm = (wave & 3) * 32, wn = (wave >> 2) * 64;
    // LDS: step parity, then P0, P1, Q0, Q1
    auto at = [&](int parity, int part) { return lds + (parity * 4 + part) * half; };

    f32x4 acc[2][2][4][2];      // half of Q, half of P, n, m
#pragma unroll
    for (int e = 0; e < 32; ++e)
        (&acc[0][0][0][0])[e] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    u32x4 fp[2][2], fq[2][2][4];    // part of k, row; Q: two of them

    auto send = [&](int part, int step, int parity) {
        const int k0 = k_first + step * P::step;
        char *to = at(parity, part);
        switch (part) {
        case 0: p0.stage_direct(to, k0, wave, lane); break;
        case 1: p1.stage_direct(to, k0, wave, lane); break;
        case 2: q0.stage_direct(to, k0, wave, lane); break;
        default: q1.stage_direct(to, k0, wave, lane); break;
        }
    };
    const Fragments<T, 128, PR, 2> even_p(lds, wm, lane), odd_p = even_p.moved(4 * half);
    const Fragments<T, 128, QR, 4> even_q(lds, wn, lane), odd_q = even_q.moved(4 * half);
    auto read_p = [&](int parity, int h) {
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
#pragma unroll
            for (int m = 0; m < 2; ++m)
                fp[ks][m] = (parity ? odd_p : even_p).read(m, ks, h * half);
    };
    auto read_q = [&](int parity, int h, auto into) {
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
#pragma unroll
            for (int n = 0; n < 4; ++n)
                fq[into.value][ks][n] = (parity ? odd_q : even_q).read(n, ks, (2 + h) * half);
    };
    auto multiply = [&](auto from, int hq, int hp) {
        wait_loads<10>();
        bare_barrier();
        __builtin_amdgcn_s_setprio(1);
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int m = 0; m < 2; ++m)
                    mma<T>(fq[from.value][ks][n], fp[ks][m], acc[hq][hp][n][m]);
        __builtin_amdgcn_s_setprio(0);
        bare_barrier();
    };
    // one step; its Q0 is already in registers `x`, Q1 goes to `y`, and the
    // next step's Q0 to `y` again as soon as Q1 has been used
    // (x is also the step's parity)
    auto step = [&](int s, auto x, auto y) {
        constexpr int b = decltype(x)::value;
        read_p(b, 0);
        send(1, s + 1, b ^ 1);
        multiply(x, 0, 0);
        read_q(b, 1, y);
        send(2, s + 2, b);
        multiply(y, 1, 0);
        read_p(b, 1);
        send(0, s + 2, b);
        multiply(y, 1, 1);
        read_q(b ^ 1, 0, y);
        send(3, s + 2, b);
        multiply(x, 0, 1);
    };
    constexpr std::integral_constant<int, 0> r0;
    constexpr std::integral_constant<int, 1> r1;
    const int steps = (k_last - k_first + P::step - 1) / P::step;
    for (int e = 0; e < 7; ++e) {       // Q0 P0 Q1 P1 of step 0, Q0 P0 Q1 of step 1
        const int part = (e & 3) == 0 ? 2 : (e & 3) == 1 ? 0 : (e & 3) == 2 ? 3 : 1;
        send(part, e >> 2, e >> 2);
    }
    wait_loads<10>();
    bare_barrier();
    read_q(0, 0, r0);
    if (wave >= 4)
        bare_barrier();
    for (int s = 0; s < steps; s += 2) {
        step(s, r0, r1);
        if (s + 1 < steps)
            step(s + 1, r1, r0);
    }
    if (wave < 4)
        bare_barrier();
    __builtin_amdgcn_s_waitcnt(0);
    __syncthreads();

    // The sums through LDS, 128 rows at a time, so that a wave's stores cover
    // whole rows of the tile; a thread takes 8 columns of every 16th row.  The
    // residuals are on their way before they are needed.
    constexpr int kRows = 128 / 16;
    const int m0 = tm * 256, n0 = tn * 256, line = tid >> 5, col = (tid & 31) * 8;
    auto spread = [&](int hp) {
#pragma unroll
        for (int hq = 0; hq < 2; ++hq)
#pragma unroll
            for (int n = 0; n < 4; ++n)
#pragma unroll
                for (int m = 0; m < 2; ++m)
                    *(lds_f32x4)((lds_ptr)lds + (wm + m * 16 + (lane & 15)) * kPitch +
                                 (hq * 128 + wn + n * 16 + (lane >> 4) * 4) * 4) =
                        acc[hq][hp][n][m];
        __syncthreads();
    };
    auto row_of = [&](int k, float (&s)[8]) {
        const lds_f32x4 from = (lds_f32x4)((lds_ptr)lds + (line + k * 16) * kPitch + col * 4);
        const f32x4 lo = from[0], hi = from[1];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            s[e] = lo[e];
            s[e + 4] = hi[e];
        }
    };
    if (a.f.part) {
        with_cut<4>(a.N - n0, 256, [&](auto c) {
            const Block<float, 4, decltype(c)::value> out(
                a.f.part + (long long)split * a.M * a.N, a.N, m0, n0, 256, a.M, a.N);
#pragma unroll
            for (int hp = 0; hp < 2; ++hp) {
                spread(hp);
#pragma unroll
                for (int k = 0; k < kRows; ++k) {
                    float s[8];
                    row_of(k, s);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const float half[4] = {s[h * 4], s[h * 4 + 1], s[h * 4 + 2], s[h * 4 + 3]};
                        out.store(half, line, hp * 128 + k * 16, col + h * 4);
                    }
                }
                __syncthreads();
            }
        });
        return;
    }
    with_cut<8>(a.N - n0, 256, [&](auto c) {
        constexpr bool CUT = decltype(c)::value;
        const Block<T, 8, CUT> from(a.f.res, a.f.ldres, m0, n0, 256, a.M, a.N),
            z(a.f.z, a.f.ldz, m0, n0, 256, a.M, a.N), y(a.f.y, a.f.ldy, m0, n0, 256, a.M, a.N);
        Raw<T, 8> res[kRows];
        auto fetch = [&](int hp) {
            if (a.f.res)
#pragma unroll
                for (int k = 0; k < kRows; ++k)
                    from.load(res[k], line, hp * 128 + k * 16, col);
        };
        fetch(0);
        float b[8] = {};
        if (a.f.b) {
            const Block<float, 4, CUT> bias(a.f.b, 0, 0, n0, 1, 1, a.N);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                Raw<float, 4> v;
                bias.load(v, 0, 0, col + h * 4);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    b[h * 4 + e] = v.get(e);
            }
        }
        with_act(a.f.act, [&](auto act) {
#pragma unroll
            for (int hp = 0; hp < 2; ++hp) {
                spread(hp);
#pragma unroll
                for (int k = 0; k < kRows; ++k) {
                    float s[8];
                    row_of(k, s);
                    finish<decltype(act)::value>(a.f, z, y, b, res[k], s, line, hp * 128 + k * 16,
                                                 col);
                }
                if (hp == 0)
                    fetch(1);
                __syncthreads();
            }
        });
    });
}

// ---------------------------------------------------------------------------
// Few rows m (single tokens of many sequences): bound by reading Q once.  A
// workgroup takes 16 columns n; its 8 waves each take a range of k straight from
// memory into fragments, and their sums are added in LDS in order.  P is read
// by every workgroup, from the caches.  8 x 8192 x 2048 bfloat16: 9 to 10 us, 3.5 TB/s
// (the weights alone at the rate of a large copy: 5.4); float32 18 us.
// ---------------------------------------------------------------------------
constexpr int kFewWaves = 8;

template <typename T>
__device__ __forceinline__ u32x4 chunk_of(const T *row, int k, int K)
{
    constexpr int elems = 16 / (int)sizeof(T);
    Pack<T, elems> v;
    if (k + elems <= K) {
        v = *reinterpret_cast<const Pack<T, elems> *>(row + k);
    } else {
#pragma unroll
        for (int e = 0; e < elems; ++e) {
            v.v[e] = (T)0.0f;
            if (k + e < K)
                v.v[e] = row[k + e];
        }
    }
    return __builtin_bit_cast(u32x4, v);
}

template <typename T, int MF>
__global__ __launch_bounds__(kFewWaves * 64) void k_few_rows(Product a, int k_per_wave)
{
    constexpr int elems = 16 / (int)sizeof(T), step = 4 * elems;    // k of a fragment
    __shared__ f32x4 lds[kFewWaves][MF][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int g = lane >> 4, i = lane & 15, n0 = blockIdx.x * 16;
    const T *q = static_cast<const T *>(a.q) + (long long)min(n0 + i, a.N - 1) * a.ldq;
    const T *p[MF];
#pragma unroll
    for (int m = 0; m < MF; ++m)
        p[m] = static_cast<const T *>(a.p) + (long long)min(m * 16 + i, a.M - 1) * a.ldp;
    f32x4 acc[MF];
#pragma unroll
    for (int m = 0; m < MF; ++m)
        acc[m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    const int k1 = min((wave + 1) * k_per_wave, a.K);
    int k = wave * k_per_wave;
    constexpr int kAhead = MF == 1 ? 8 : 4;     // fragments of Q on their way
    for (; k + kAhead * step <= k1; k += kAhead * step) {
        u32x4 fq[kAhead], fp[kAhead][MF];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            fq[u] = chunk_of(q, k + u * step + g * elems, a.K);
#pragma unroll
            for (int m = 0; m < MF; ++m)
                fp[u][m] = chunk_of(p[m], k + u * step + g * elems, a.K);
        }
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
#pragma unroll
            for (int m = 0; m < MF; ++m)
                mma<T>(fq[u], fp[u][m], acc[m]);
    }
    for (; k < k1; k += step) {
        const u32x4 fq = chunk_of(q, k + g * elems, a.K);
#pragma unroll
        for (int m = 0; m < MF; ++m)
            mma<T>(fq, chunk_of(p[m], k + g * elems, a.K), acc[m]);
    }
#pragma unroll
    for (int m = 0; m < MF; ++m)
        lds[wave][m][lane] = acc[m];
    __syncthreads();
    const int row = wave * 16 + i, col = n0 + g * 4;
    if (wave >= MF || row >= a.M || col >= a.N)
        return;
    float sum[4] = {}, b[4] = {};
#pragma unroll
    for (int w = 0; w < kFewWaves; ++w) {
        const f32x4 v = lds[w][wave][lane];
#pragma unroll
        for (int e = 0; e < 4; ++e)
            sum[e] += v[e];
    }
    if (a.f.b)
        get(a.f.b + col, a.N - col, b);
    Raw<T, 4> r;
    if (a.f.res)
        residual(a.f, row, col, a.N - col, r);
    finish<T>(a.f, row, col, a.N - col, b, r, sum);
}

// out = finish(the splits' partial sums, added in order): a thread per 4 columns.
template <typename T>
__global__ __launch_bounds__(256) void k_gemm_sum(Product a, int groups)
{
    const long long id = (long long)blockIdx.x * 256 + threadIdx.x;
    const int m = (int)(id / groups), n = (int)(id % groups) * 4, width = a.N - n;
    if (m >= a.M)
        return;
    float sum[4], b[4] = {};
    const float *part = a.f.part + (long long)m * a.N + n;
    get(part, width, sum);
    const long long next = (long long)a.M * a.N;
    int k = 1;
    constexpr int kAhead = 8;       // loads on their way
    for (; k + kAhead <= a.splits; k += kAhead) {
        float v[kAhead][4];
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            get(part + (k + u) * next, width, v[u]);
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
#pragma unroll
            for (int e = 0; e < 4; ++e)
                sum[e] += v[u][e];
    }
    for (; k < a.splits; ++k) {
        float v[4];
        get(part + k * next, width, v);
#pragma unroll
        for (int e = 0; e < 4; ++e)
            sum[e] += v[e];
    }
    if (a.f.b)
        get(a.f.b + n, width, b);
    Raw<T, 4> r;
    if (a.f.res)
        residual(a.f, m, n, width, r);
    finish<T>(a.f, m, n, width, b, r, sum);
}

}  // namespace

template <typename T> int launch_gemm(const Product &product, hipStream_t st)
{
    constexpr int size = (int)sizeof(T), step = kStepBytes / size;
    Product a = product;
    const int k_per_split = split_length(a.K, a.splits, size);
    a.splits = split_count(a.K, a.splits, size);
    if (a.splits == 1)
        a.f.part = nullptr;
    if (a.tile == FEW_ROWS) {
        const int k_per_wave = (int)(cdiv(a.K, kFewWaves * step) * step);
        auto few = [&](auto mf) {
            return dwconv::launch_kernel(k_few_rows<T, decltype(mf)::value>,
                                         dim3((unsigned)cdiv(a.N, 16)), dim3(kFewWaves * 64), 0,
                                         st, a, k_per_wave);
        };
        if (a.M <= 16)
            return few(std::integral_constant<int, 1>());
        if (a.M <= 32)
            return few(std::integral_constant<int, 2>());
        return few(std::integral_constant<int, 4>());
    }
    const bool direct = direct_ok(a.p, a.ldp, a.p_rows_k, a.K, size) &&
                        direct_ok(a.q, a.ldq, a.q_rows_k, a.K, size);
    const GemmTile tile = tile_taken(a.tile, direct, size);
    auto run = [&](auto pr, auto qr, auto dir, auto bm, auto bn, auto wm, auto wn, auto stages) {
        constexpr int BM = decltype(bm)::value, BN = decltype(bn)::value;
        constexpr int WM = decltype(wm)::value, WN = decltype(wn)::value;
        const long long tiles_m = cdiv(a.M, BM), tiles_n = cdiv(a.N, BN);
        if (tiles_m * tiles_n > 0x3fffffffLL)
            return (int)DWCONV_ERR_BAD_DIM;
        return dwconv::launch_kernel(
            k_gemm<T, decltype(pr)::value, decltype(qr)::value, decltype(dir)::value, BM, BN, WM,
                   WN, decltype(dir)::value ? decltype(stages)::value : 2>,
            tile_grid(tiles_m * tiles_n, a.splits), dim3(WM * WN * 64), 0, st, a, (int)tiles_m,
            (int)tiles_n, k_per_split);
    };
    auto sized = [&](auto pr, auto qr, auto dir) {
        using std::integral_constant;
        if constexpr (decltype(dir)::value && size == 2) {
            if (tile == TILE_256) {
                const long long tiles_m = cdiv(a.M, 256), tiles_n = cdiv(a.N, 256);
                if (tiles_m * tiles_n > 0x3fffffffLL)
                    return (int)DWCONV_ERR_BAD_DIM;
                return dwconv::launch_kernel(
                    k_gemm_256<T, decltype(pr)::value, decltype(qr)::value>,
                    tile_grid(tiles_m * tiles_n, a.splits), dim3(512), 0, st, a, (int)tiles_m,
                    (int)tiles_n, k_per_split);
            }
        }
        switch (tile) {
        case TILE_128:
            return run(pr, qr, dir, integral_constant<int, 128>(), integral_constant<int, 128>(),
                       integral_constant<int, 2>(), integral_constant<int, 2>(),
                       integral_constant<int, 2>());
        case TILE_64_DEEP:
            if constexpr (decltype(dir)::value && size == 2)
                return run(pr, qr, dir, integral_constant<int, 64>(), integral_constant<int, 64>(),
                           integral_constant<int, 2>(), integral_constant<int, 2>(),
                           integral_constant<int, 4>());
        default:
            return run(pr, qr, dir, integral_constant<int, 64>(), integral_constant<int, 64>(),
                       integral_constant<int, 2>(), integral_constant<int, 2>(),
                       integral_constant<int, 2>());
        }
    };
    auto ways = [&](auto dir) {
        if (!a.p_rows_k && !a.q_rows_k)
            return sized(std::false_type(), std::false_type(), dir);
        if (!a.p_rows_k)
            return sized(std::false_type(), std::true_type(), dir);
        return sized(std::true_type(), std::true_type(), dir);
    };
    const int rc = direct ? ways(std::true_type()) : ways(std::false_type());
    if (rc != DWCONV_OK || !a.f.part)
        return rc;
    const int groups = (int)cdiv(a.N, 4);
    const long long blocks = cdiv((long long)a.M * groups, 256);
    return dwconv::launch_kernel(k_gemm_sum<T>, dim3((unsigned)blocks), dim3(256), 0, st, a,
                                 groups);
}
#endif  // DWSEQ_GEMM_KERNELS

}  // namespace dwseq

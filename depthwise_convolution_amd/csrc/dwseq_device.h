// dwseq_device.h -- what the kernel files of the sequence operators share:
// element types and vectors, activations and their slopes, the lookup of a
// row's sequence, and the fixed-order sum of partial rows.
#pragma once

#include "dwconv_device.h"
#include "dwseq_internal.h"
#include "../../include/dwconv_seq.h"

namespace dwseq {
namespace {

typedef _Float16 f16;
typedef __bf16 bf16;

// V elements that need only their own type's alignment: the global loads and
// stores of gfx950 take a vector at any element's address (rows of odd width,
// column ranges), so one kernel serves every alignment.
template <typename T, int V> struct __attribute__((packed, aligned(sizeof(T)))) Pack { T v[V]; };

// V elements as float32 (one vector load), and back (rounded to nearest even)
template <typename T, int V>
__device__ __forceinline__ void load(const T *p, float (&f)[V])
{
    const Pack<T, V> t = *reinterpret_cast<const Pack<T, V> *>(p);
#pragma unroll
    for (int i = 0; i < V; ++i)
        f[i] = (float)t.v[i];
}

template <typename T, int V>
__device__ __forceinline__ void store(T *p, const float (&f)[V])
{
    Pack<T, V> t;
#pragma unroll
    for (int i = 0; i < V; ++i)
        t.v[i] = (T)f[i];
    *reinterpret_cast<Pack<T, V> *>(p) = t;
}

// V elements as they came from memory, two 16-bit ones to a register: what is
// kept for later (the compiler gives every element of a Pack a register).
template <typename T, int V> struct Raw {
    static constexpr int words = V * (int)sizeof(T) < 4 ? 1 : V * (int)sizeof(T) / 4;
    unsigned w[words];

    Raw() = default;
    __device__ __forceinline__ explicit Raw(const float (&f)[V])
    {
        static_assert(V == 1 || V % 2 == 0);
#pragma unroll
        for (int i = 0; i < words; ++i) {
            if constexpr (sizeof(T) == 4) {
                w[i] = __builtin_bit_cast(unsigned, f[i]);
            } else if constexpr (V == 1) {
                w[i] = __builtin_bit_cast(unsigned short, (T)f[0]);
            } else {
                typedef float f32x2 __attribute__((ext_vector_type(2)));
                typedef T t2 __attribute__((ext_vector_type(2)));
                const f32x2 pair = {f[2 * i], f[2 * i + 1]};
                w[i] = __builtin_bit_cast(unsigned, __builtin_convertvector(pair, t2));
            }
        }
    }

    __device__ __forceinline__ void load(const T *p)
    {
        if constexpr (V * sizeof(T) == 2) {
            w[0] = *reinterpret_cast<const unsigned short *>(p);
        } else {
            const Pack<T, V> t = *reinterpret_cast<const Pack<T, V> *>(p);
            static_assert(sizeof(w) == sizeof(t));
            __builtin_memcpy(w, &t, sizeof(t));
        }
    }
    // past the caches: what is not read again, or written and not read soon
    __device__ __forceinline__ void load_past(const T *p)
    {
        if constexpr (V * sizeof(T) == 2) {
            w[0] = __builtin_nontemporal_load(reinterpret_cast<const unsigned short *>(p));
        } else {
            typedef unsigned words_t
                __attribute__((ext_vector_type(words), aligned(sizeof(T))));
            const words_t t = __builtin_nontemporal_load(reinterpret_cast<const words_t *>(p));
            __builtin_memcpy(w, &t, sizeof(w));
        }
    }
    __device__ __forceinline__ void store_past(T *p) const
    {
        if constexpr (V * sizeof(T) == 2) {
            __builtin_nontemporal_store((unsigned short)w[0],
                                        reinterpret_cast<unsigned short *>(p));
        } else {
            typedef unsigned words_t
                __attribute__((ext_vector_type(words), aligned(sizeof(T))));
            words_t t;
            __builtin_memcpy(&t, w, sizeof(w));
            __builtin_nontemporal_store(t, reinterpret_cast<words_t *>(p));
        }
    }
    // through a buffer descriptor, `lane` plus `row` bytes from its start; HINT: the
    // instruction's cache bits
    template <int HINT = 0>
    __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t rsrc, int lane, int row)
    {
        if constexpr (V * sizeof(T) == 2) {
            w[0] = __builtin_amdgcn_raw_buffer_load_b16(rsrc, lane, row, HINT);
        } else if constexpr (words == 1) {
            w[0] = __builtin_amdgcn_raw_buffer_load_b32(rsrc, lane, row, HINT);
        } else if constexpr (words == 2) {
            *this = __builtin_bit_cast(Raw,
                                       __builtin_amdgcn_raw_buffer_load_b64(rsrc, lane, row, HINT));
        } else if constexpr (words == 4) {
            *this = __builtin_bit_cast(Raw,
                                       __builtin_amdgcn_raw_buffer_load_b128(rsrc, lane, row, HINT));
        } else {
            static_assert(words == 8);
            const auto lo = __builtin_amdgcn_raw_buffer_load_b128(rsrc, lane, row, HINT);
            const auto hi = __builtin_amdgcn_raw_buffer_load_b128(rsrc, lane + 16, row, HINT);
            __builtin_memcpy(w, &lo, 16);
            __builtin_memcpy(w + 4, &hi, 16);
        }
    }
    // Four words go without a scalar offset: the compiler takes such a store to
    // have read its registers at once and overwrites them in the next
    // instruction, which has been seen to change the last word of some lanes.
    // Without one it waits.
    template <int HINT = 0>
    __device__ __forceinline__ void store(__amdgpu_buffer_rsrc_t rsrc, int lane, int row) const
    {
        typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
        typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
        if constexpr (V * sizeof(T) == 2) {
            __builtin_amdgcn_raw_buffer_store_b16((unsigned short)w[0], rsrc, lane, row, HINT);
        } else if constexpr (words == 1) {
            __builtin_amdgcn_raw_buffer_store_b32(w[0], rsrc, lane, row, HINT);
        } else if constexpr (words == 2) {
            __builtin_amdgcn_raw_buffer_store_b64(__builtin_bit_cast(u32x2, *this), rsrc, lane, row,
                                                  HINT);
        } else if constexpr (words == 4) {
            __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(u32x4, *this), rsrc,
                                                   lane + row, 0, HINT);
        } else {
            static_assert(words == 8);
            __builtin_amdgcn_raw_buffer_store_b128(u32x4{w[0], w[1], w[2], w[3]}, rsrc, lane + row,
                                                   0, HINT);
            __builtin_amdgcn_raw_buffer_store_b128(u32x4{w[4], w[5], w[6], w[7]}, rsrc,
                                                   lane + row + 16, 0, HINT);
        }
    }
    __device__ __forceinline__ float get(int v) const
    {
        if constexpr (sizeof(T) == 4)
            return __builtin_bit_cast(float, w[v]);
        else if constexpr (std::is_same_v<T, bf16>)
            return __builtin_bit_cast(float, v & 1 ? w[v / 2] & 0xffff0000u : w[v / 2] << 16);
        else
            return (float)__builtin_bit_cast(f16, (unsigned short)(w[v / 2] >> (16 * (v & 1))));
    }
    __device__ __forceinline__ void clear()
    {
#pragma unroll
        for (int i = 0; i < words; ++i)
            w[i] = 0;
    }
};

// 1 / (1 + e^-v) with the hardware's exponential and reciprocal (one unit in
// the last place each, beside the rounding of the exponential's argument: for
// negative v a relative error of up to (1.25 |v| + 6) 2^-24); 0 and 1 at the infinities
__device__ __forceinline__ float logistic(float v)
{
    return __builtin_amdgcn_rcpf(1.0f + __expf(-v));
}

// NaN passes through every activation.
__device__ __forceinline__ float act_of(float z, int act)
{
    if (act == DWCONV_ACT_SILU)
        return z * logistic(z);
    if (act == DWCONV_ACT_RELU)
        return z < 0.0f ? 0.0f : z;
    if (act == DWCONV_ACT_RELU6)
        return z < 0.0f ? 0.0f : (z > 6.0f ? 6.0f : z);
    return z;
}

// the activation is the same for all: one branch
template <int V> __device__ __forceinline__ void act_all(float (&z)[V], int act)
{
    if (act == DWCONV_ACT_NONE)
        return;
    if (act == DWCONV_ACT_SILU) {
#pragma unroll
        for (int v = 0; v < V; ++v)
            z[v] = act_of(z[v], DWCONV_ACT_SILU);
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v)
            z[v] = act_of(z[v], act);
    }
}

__device__ __forceinline__ float act_slope(float z, int act)
{
    if (act == DWCONV_ACT_SILU) {
        const float p = logistic(z);
        return p * (1.0f + z * (1.0f - p));
    }
    if (act == DWCONV_ACT_RELU)
        return z > 0.0f ? 1.0f : 0.0f;
    if (act == DWCONV_ACT_RELU6)
        return z > 0.0f && z < 6.0f ? 1.0f : 0.0f;
    return 1.0f;
}

// z's slopes in its place, again with one branch for all: with one for each the
// exponentials and reciprocals wait for each other instead of overlapping
template <int V> __device__ __forceinline__ void slope_all(float (&z)[V], int act)
{
    if (act == DWCONV_ACT_SILU) {
#pragma unroll
        for (int v = 0; v < V; ++v)
            z[v] = act_slope(z[v], DWCONV_ACT_SILU);
    } else {
#pragma unroll
        for (int v = 0; v < V; ++v)
            z[v] = act == DWCONV_ACT_NONE ? 1.0f : act_slope(z[v], act);
    }
}

// First row of sequence s (s = seqs: the end).  Offsets are clamped to the
// rows there are, and the outer two are taken as given by the batch.
__device__ __forceinline__ int seq_start(const Batch &b, int s)
{
    if (s <= 0)
        return 0;
    if (s >= b.seqs)
        return b.rows;
    return b.off ? min(max(b.off[s], 0), b.rows) : s * b.tokens;
}

// The last sequence that starts at or before `row`.
__device__ __forceinline__ int seq_of(const Batch &b, int row)
{
    if (!b.off)
        return min(row / max(b.tokens, 1), b.seqs - 1);
    int lo = 0, hi = b.seqs - 1;
    while (lo < hi) {
        const int mid = lo + ((hi - lo + 1) >> 1);
        if (seq_start(b, mid) <= row)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

// A dimension of a grid holds fewer than 2^32 threads: past kGridRow workgroups
// (of 1024 threads at most) they go on in the second dimension, the last row of
// which may have some too many.  A multiple of the XCDs.
constexpr unsigned kGridRow = 1u << 21;

inline dim3 grid_of(long long blocks)
{
    return blocks <= kGridRow ? dim3((unsigned)blocks)
                              : dim3(kGridRow, (unsigned)cdiv(blocks, kGridRow));
}

__device__ __forceinline__ unsigned block_id() { return blockIdx.y * kGridRow + blockIdx.x; }

// Sum of the rows of part[rows][n] per column in a fixed order: a workgroup
// takes 64 columns, its 16 waves every 16th row each, added up in LDS.  The
// sums go to f(column, sum).
template <typename F>
__device__ __forceinline__ void column_sums(const float *part, int rows, long long n, F f)
{
    __shared__ float lds[16][64];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const long long col = (long long)block_id() * 64 + lane;
    float s = 0.0f;
    if (col < n)
#pragma unroll 4
        for (int k = wave; k < rows; k += 16)
            s += part[(long long)k * n + col];
    lds[wave][lane] = s;
    __syncthreads();
    if (wave == 0 && col < n) {
#pragma unroll
        for (int k = 1; k < 16; ++k)
            s += lds[k][lane];
        f(col, s);
    }
}

// f(std::integral_constant<type>) with the element type of `type`
template <typename F>
inline int with_type(int type, F f)
{
    switch (type) {
    case DWCONV_T_F32: return f((float *)nullptr);
    case DWCONV_T_F16: return f((f16 *)nullptr);
    case DWCONV_T_BF16: return f((bf16 *)nullptr);
    }
    return DWCONV_ERR_BAD_WTYPE;
}

}  // namespace
}  // namespace dwseq

// dwmix_quantize.h -- how rows become 8-bit integers, for the kernels that do it.
#pragma once

#include "dwseq_device.h"

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

template <typename T> __device__ __forceinline__ unsigned magnitude(T v)
{
    return __builtin_bit_cast(unsigned, (float)v) & 0x7fffffffu;
}

// The largest magnitude of many elements, on bit patterns, which order NaN above
// infinity above the rest: 16-bit ones as they are, two to a register.
template <typename T> struct Largest {
    typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
    unsigned most = 0;

    template <int V> __device__ __forceinline__ void look(const Raw<T, V> &r)
    {
#pragma unroll
        for (int i = 0; i < Raw<T, V>::words; ++i)
            if constexpr (sizeof(T) == 4)
                most = max(most, r.w[i] & 0x7fffffffu);
            else
                most = __builtin_bit_cast(
                    unsigned, __builtin_elementwise_max(
                                  __builtin_bit_cast(u16x2, most),
                                  __builtin_bit_cast(u16x2, r.w[i] & 0x7fff7fffu)));
    }
    // as float32's bits
    __device__ __forceinline__ unsigned get() const
    {
        if constexpr (sizeof(T) == 4)
            return most;
        else
            return magnitude(__builtin_bit_cast(T, (unsigned short)max(most & 0xffffu, most >> 16)));
    }
};

}  // namespace
}  // namespace dwmix

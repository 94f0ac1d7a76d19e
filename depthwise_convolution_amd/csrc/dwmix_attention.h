// dwmix_attention.h -- the walk along the tokens behind dwconv_attention_*, one
// translation unit per element type (dwmix_attention_*.hip).
//
//   out[i] = s0 * sum_{j <= i} a^(i-j) (q[i] . k[j]) v[j] + s1 * a^(i+1-late) q[i] S
//   S     <- a^n S + s2 * sum_j a^(n-1-j+late) k[j] v[j]^T          (n tokens)
//
// The forward is this walk over (q, k, v) with late = 0.  Each gradient is the
// same walk over other tensors: dq over (dy, v, k), with the transposed state; dk
// and dv from the last token to the first, with late = 1 (the cotangent of a state
// reaches the token that made it without a decay), over (v, dy, q) and (k, q, dy).
//
// A sequence is cut into segments, which run side by side: first the state that each
// adds by itself (k_states), then those linked one after the other (k_link), then
// the walk, each segment from its own start.  Where there are enough sequences
// and heads to fill the chip a sequence is one segment, and the walk is all.
//
// A workgroup walks one head of one segment, a tile of DVT of the state's columns
// with a wave for each 16 of them, in chunks of 128 bytes of tokens (64 16-bit, 32
// float32):
//
//   scores   P[i, j], some tiles of 16 x 16 a wave, times their decay, through LDS
//   output   a wave takes its 16 columns for all rows: its part of S is in registers
//            (float32, as the matrix instructions leave it), which is already the
//            layout of an operand that is summed over dk, so q S reads only q;
//            then P V on top
//   state    S = a^n S + K^T (V with its decays), the same columns
//
// so that LDS holds q, k, v and P (71 KB for widths of 128), a state never
// leaves its registers, and two workgroups share a CU.
//
// Roundings of 16-bit types.  P and the chunk's S become two numbers of the type each
// where they are operands, 16 bits and more of them, so that the output's own rounding
// is all that shows.  V with its decays, which the state is built from, is split into
// parts (three bfloat16, two float16) that hold 22 bits and more: what is lost
// there would add up in the float32 state.
//
// What bounds it (8 x 4096 tokens, 16 heads of 128 bfloat16: states 66 us, links 11,
// walk 155): HBM most, and nothing alone.  The walk reads 428 MB and writes 143, which take
// 91 us at 6.28 TB/s, 0.59 of its time; the vector units are active 0.54 of it, LDS 0.45, the
// matrix cores 0.31.  The three barriers of a chunk, and 16-bit types' loads that are sent
// for only after its results, keep these from overlapping more, at two workgroups a CU. The
// states' pass reads 3 of 4 segments, so that half of the CUs have two workgroups and half
// have one.
//
// float16 has too few exponents for scores and states: the values are scaled by a power
// of two, one for each wave, where their largest would be too large or too small.
//
// A number that is not finite: those of v are taken out of the products, which would spread
// them to other tokens by zero scores, and added one by one.  Those of q and k meet both
// numbers that a 16-bit operand was made, one of which may be zero: an infinity may then
// arrive as NaN.
#pragma once

#include "dwmix_internal.h"
#include "dwseq_device.h"
#include "../../include/dwconv_mix.h"

#include <algorithm>

namespace dwmix {

// One walk.
struct Walk {
    const void *q, *k, *v;
    void *out;                          // nullptr: only the state is wanted
    const float *log_decay, *state0;    // state0 nullptr: zero
    float *state1;                      // nullptr: not kept
    float *slots;                       // states that segments start from, [slot][H][Dk][Dv]
    bool ready;                         // slots are another walk's, and [slot][H][Dv][Dk]
    long long ldq, ldk, ldv, ldo;
    int gq, gk, gv;                     // heads that share one of the tensor's
    int H, Dk, Dv;
    float s0, s1, s2;
    int late, back;
    bool flip;                          // state0 and state1 are [..][Dv][Dk]
    bool out32;                         // out is float32
    Batch batch;
    int segment, per_seq, items;        // tokens; segments of a dense sequence; of all
};

// Up to kWalks walks of one batch that do not need each other's results, but that one
// may take another's slots.
constexpr int kWalks = 3;
template <typename T> int launch_walks(const Walk *w, int count, hipStream_t st);

// What one launch does of them: workgroups for each, a multiple of 8 (so that the
// order on the XCDs is the same for all).
struct Walks {
    Walk w[kWalks];
    int blocks[kWalks];
};
// columns of the state that a workgroup takes
inline int walk_tile(int Dk, int Dv) { return Dk > 128 || Dv <= 64 ? 64 : 128; }

#ifdef DWMIX_ATTENTION_KERNELS
namespace {

using namespace dwseq;

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));
typedef bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef f16 f16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) char *lds_ptr;
typedef __attribute__((address_space(3))) u32x4 *lds_u4;
typedef __attribute__((address_space(3))) u32x2 *lds_u2;
typedef __attribute__((address_space(3))) unsigned *lds_u1;

// c += a b of 16 x 16, over 32 16-bit or 16 float32 numbers
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

// Waits until the results of all matrix instructions may be read.  The compiler
// counts those waits itself, but not along every branch (seen: one that skipped
// further matrix instructions, and the last word of a result read too early), so
// no branch lies between a matrix instruction and this.
__device__ __forceinline__ void settle()
{
    __builtin_amdgcn_sched_barrier(0);
    asm volatile("s_nop 15\n\ts_nop 7" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
}

// V floats as elements of T, two 16-bit ones to a word
template <typename T, int V>
__device__ __forceinline__ void narrow(const float (&f)[V], unsigned *w)
{
    const Raw<T, V> r(f);
#pragma unroll
    for (int i = 0; i < Raw<T, V>::words; ++i)
        w[i] = r.w[i];
}

// Whether a word holds an infinity or a NaN (16-bit types: either of its two).
template <typename T> __device__ __forceinline__ unsigned odd_bits(unsigned w)
{
    if constexpr (std::is_same_v<T, bf16>)
        return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
    else if constexpr (std::is_same_v<T, f16>)
        return ((w & 0x7c007c00u) + 0x04000400u) & 0x80008000u;
    else
        return ((w & 0x7f800000u) + 0x00800000u) & 0x80000000u;
}

// The word with infinities and NaN replaced by zero.
template <typename T> __device__ __forceinline__ unsigned cleaned(unsigned w)
{
    const unsigned odd = odd_bits<T>(w);
    if constexpr (sizeof(T) == 4)
        return odd ? 0u : w;
    else
        return w & ~((odd >> 15) * 0xffffu);
}

// Sequence and segment of an item: sequence s has the items from
// start(s) / segment + s on (packed), which are at least as many as its segments.
struct Item {
    int seq, seg, row0, length;     // of the sequence
    __device__ __forceinline__ Item(const Walk &w, int item)
    {
        const Batch &b = w.batch;
        if (!b.off) {
            seq = item / w.per_seq;
            seg = item - seq * w.per_seq;
        } else {
            // a wave probes 64 places at once: a step for each 64-fold of sequences, not
            // for each doubling (a load's latency each).  lo is a place that does not lie
            // behind the item; the probes that do not are the first ones.
            int lo = 0, count = b.seqs;
            while (count > 1) {
                const int step = (count + 63) >> 6, at = (int)(threadIdx.x & 63) * step;
                const bool before = at < count &&
                                    seq_start(b, lo + at) / w.segment + lo + at <= item;
                const unsigned long long votes = ~__ballot(before);
                const int last = votes ? max((int)__builtin_ctzll(votes) - 1, 0) : 63;
                lo += last * step;
                count = min(step, count - last * step);
            }
            seq = __builtin_amdgcn_readfirstlane(lo);
            seg = item - (seq_start(b, seq) / w.segment + seq);
        }
        row0 = seq_start(b, seq);
        length = max(seq_start(b, seq + 1) - row0, 0);
    }
    __device__ __forceinline__ int segments(const Walk &w) const { return count(w, length); }
    static __device__ __forceinline__ int count(const Walk &w, int length)
    {
        return max(1, (int)(((long long)length + w.segment - 1) / w.segment));
    }
};

// log a of a head: 0 at most; finite, so that its product with 0 is 0
__device__ __forceinline__ float log_decay_of(const float *p, int h)
{
    const float g = p[h];
    return g != g ? g : fmaxf(fminf(g, 0.0f), -1e4f);
}

// The slot of segment `seg` of a sequence that begins with row0; segment 0 has none.  A
// sequence's last one is at most (row after it - 1) / segment - 1, before the next one's
// first: rows alone say how many there are.
__device__ __forceinline__ int slot_of(const Walk &w, int row0, int seg)
{
    return row0 / w.segment + seg - 1;
}

// Element [dk][dv] of a state array that is [Dk][Dv], or flipped.
__device__ __forceinline__ long long state_at(const Walk &w, bool flip, int dk, int dv)
{
    return flip ? (long long)dv * w.Dk + dk : (long long)dk * w.Dv + dv;
}

constexpr int kChunkBytes = 128;

// Kernels of their own, so that none pays registers for what it does not do: widths of
// whole chunks of 16 bytes with results of T, or (the parts of shared heads) of
// float32; and other widths.
enum Mode { ROWS, PARTS, ODD };

constexpr int kFar = 0x7ffffff0;        // beyond every descriptor's bounds

// A tile of C rows of D elements in LDS, 16 bytes between the rows: the reads below,
// of 16 rows at one chunk of 16 bytes, of 8 rows two apart at 32 bytes, or of 4 at 64,
// fall on different banks, and what differs between the reads of a lane is a constant.
template <typename T, int C, int D, int kThr> struct Tile {
    static constexpr int size = (int)sizeof(T), elems = 16 / size;
    static constexpr int per_row = D / elems, pitch = D * size + 16, bytes = C * pitch;
    static constexpr int count = C * per_row / kThr;    // chunks a thread stages
    static constexpr int apart = kThr / per_row;        // rows between them
    static_assert(count >= 1 && C * per_row % kThr == 0);

    // The chunk's rows from `from` on, columns up to `wide`; `lowest` is the row of lowest
    // address (which may lie before the array where `from` is not 0).
    // CUT: some width is no whole number of chunks.
    template <bool CUT>
    static __device__ __forceinline__ void fetch(u32x4 (&regs)[count], const T *lowest, int ld,
                                                 bool back, int from, int wide, int thread)
    {
        const __amdgpu_buffer_rsrc_t rsrc = dwconv::make_rsrc(lowest, kFar - 16);
        const int row = thread / per_row, col = thread % per_row * elems;
        const int first = (back ? C - 1 - row : row) * (ld * size) + col * size;
        const int step = (back ? -apart : apart) * (ld * size);
        if constexpr (!CUT) {
#pragma unroll
            for (int k = 0; k < count; ++k) {
                const bool in = row + k * apart >= from && col < wide;
                regs[k] = __builtin_bit_cast(
                    u32x4, __builtin_amdgcn_raw_buffer_load_b128(
                               rsrc, in ? first + k * step : kFar, 0, 0));
            }
        } else {        // rows that end within a chunk: element by element
#pragma unroll
            for (int k = 0; k < count; ++k) {
                unsigned v[elems];
#pragma unroll
                for (int e = 0; e < elems; ++e) {
                    const bool in = row + k * apart >= from && col + e < wide;
                    const int at = in ? first + k * step + e * size : kFar;
                    if constexpr (size == 2)
                        v[e] = __builtin_amdgcn_raw_buffer_load_b16(rsrc, at, 0, 0);
                    else
                        v[e] = __builtin_amdgcn_raw_buffer_load_b32(rsrc, at, 0, 0);
                }
                if constexpr (size == 2)
                    regs[k] = u32x4{v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16,
                                    v[6] | v[7] << 16};
                else
                    regs[k] = u32x4{v[0], v[1], v[2], v[3]};
            }
        }
    }
    // PAIRED: of each 32 16-bit columns, numbers 4g .. + 3 of both halves side by side,
    // which is the order that a matrix instruction leaves its results in.
    template <bool PAIRED = false>
    static __device__ __forceinline__ void keep(lds_ptr lds, const u32x4 (&regs)[count],
                                                int thread)
    {
        const int row = thread / per_row, c = thread % per_row;
#pragma unroll
        for (int k = 0; k < count; ++k) {
            const lds_ptr at = lds + (row + k * apart) * pitch;
            if constexpr (PAIRED && size == 2) {
                const lds_ptr to = at + paired(c);
                *(lds_u2)to = u32x2{regs[k][0], regs[k][1]};
                *(lds_u2)(to + 16) = u32x2{regs[k][2], regs[k][3]};
            } else {
                *(lds_u4)(at + c * 16) = regs[k];
            }
        }
    }
    // Where the first half of chunk c of a row is kept; the second half is 16 bytes on.
    static __device__ __forceinline__ int paired(int c)
    {
        return (c >> 2) * 64 + (c & 1) * 32 + (c >> 1 & 1) * 8;
    }

    // An operand that is summed along the row, the columns in their order: row `row`,
    // part u of it (32 16-bit or 16 float32 columns), the numbers of lane group g.
    template <bool PAIRED = false>
    static __device__ __forceinline__ u32x4 chunk(lds_ptr lds, int row, int u, int g)
    {
        if constexpr (PAIRED && size == 2) {
            const lds_ptr at = lds + row * pitch + u * 64 + (g & 1) * 32 + (g >> 1) * 8;
            const u32x2 lo = *(lds_u2)at, hi = *(lds_u2)(at + 16);
            return u32x4{lo.x, lo.y, hi.x, hi.y};
        } else {
            return *(lds_u4)(lds + row * pitch + u * 64 + g * 16);
        }
    }
    // The same of a PAIRED tile in the order that it is kept in.
    static __device__ __forceinline__ u32x4 along(lds_ptr lds, int row, int u, int g)
    {
        return *(lds_u4)(lds + row * pitch + u * 64 + g * 16);
    }
    // An operand that is summed across the rows: column col + (lane & 15), part
    // ks of the rows (32 or 16), the numbers of lane group g, in the order of row_of().
    static __device__ __forceinline__ u32x4 across(lds_ptr lds, int col, int ks, int lane)
    {
        const int g = lane >> 4, i = lane & 15;
        u32x4 v;
        if constexpr (size == 4) {
            const lds_ptr at = lds + g * 4 * pitch + i * 4;
#pragma unroll
            for (int j = 0; j < 4; ++j)
                v[j] = *(__attribute__((address_space(3))) const unsigned *)(
                    at + (ks * 16 + j) * pitch + col * 4);
        } else {
            // 4 rows, two apart, a read
            const lds_ptr at = lds + (g * 8 + (i >> 2) * 2) * pitch + (i & 3) * 8;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const s16x4 t = __builtin_amdgcn_ds_read_tr16_b64_v4i16(
                    (__attribute__((address_space(3))) s16x4 *)(at + (ks * 32 + h) * pitch +
                                                                col * 2));
                const uint2 w = __builtin_bit_cast(uint2, t);
                v[h * 2] = w.x;
                v[h * 2 + 1] = w.y;
            }
        }
        return v;
    }
    // The row of number e of such an operand.
    static __device__ __forceinline__ int row_of(int ks, int g, int e)
    {
        return size == 4 ? ks * 16 + g * 4 + e : ks * 32 + g * 8 + (e & 3) * 2 + (e >> 2);
    }
    static __device__ __forceinline__ float one(lds_ptr lds, int row, int col)
    {
        return (float)*(__attribute__((address_space(3))) const T *)(lds + row * pitch +
                                                                     col * size);
    }
};

// Element e of a fragment.  (The word is taken out first: a bit cast of a vector's
// element reads element 0 on this compiler.)
template <typename T> __device__ __forceinline__ float element(const u32x4 &v, int e)
{
    const unsigned word = v[sizeof(T) == 4 ? e : e / 2];
    if constexpr (sizeof(T) == 4)
        return __builtin_bit_cast(float, word);
    else if constexpr (std::is_same_v<T, bf16>)
        return __builtin_bit_cast(float, e & 1 ? word & 0xffff0000u : word << 16);
    else
        return (float)__builtin_bit_cast(f16, (unsigned short)(word >> (16 * (e & 1))));
}

__device__ __forceinline__ float wave_max(float m)
{
    for (int d = 1; d < 64; d *= 2)
        m = fmaxf(m, __shfl_xor(m, d));
    return m;
}

// The power of two that brings the largest finite size of a wave's numbers to [1, 2)
// where it is below lo, and to [2^13, 2^14) where it is above hi = 2^14 (which leaves the
// small ones beside it as many bits as float16 has); 1 between the two, which takes two
// votes.  `most`: a lane's largest size; finite(): its largest finite one; `up`: 2^up is
// the largest such power.
template <typename F>
__device__ __forceinline__ float range_scale(float most, float lo, float hi, F finite,
                                             int up = 120)
{
    if (!__any(most > hi) && __any(most >= lo))
        return 1.0f;
    const float m = wave_max(finite());
    if (!(m > 0.0f) || (m >= lo && m <= hi))
        return 1.0f;
    const int e = (int)((__builtin_bit_cast(unsigned, m) >> 23) & 255) - 127;
    return __builtin_bit_cast(float, (unsigned)(127 + min((m > hi ? 13 : 0) - e, up)) << 23);
}

// The largest power of two, 1 at least, that leaves a wave's numbers below 2^100 in size
// (`most`: a lane's largest finite one).
__device__ __forceinline__ float room_above(float most)
{
    const int e = (int)(__builtin_bit_cast(unsigned, wave_max(most)) >> 23) - 127;
    return __builtin_bit_cast(float, (unsigned)(127 + min(max(99 - e, 0), 120)) << 23);
}

// 1 / v of such a power of two
__device__ __forceinline__ float inverse(float v)
{
    return __builtin_bit_cast(float, 0x7f000000u - __builtin_bit_cast(unsigned, v));
}

__device__ __forceinline__ float finite_size(float v)
{
    return fabsf(v) <= 3.4e38f ? fabsf(v) : 0.0f;
}

template <typename T, int DK, int DVT, int MT> struct Body {
    static constexpr int size = (int)sizeof(T), elems = 16 / size;
    static constexpr int waves = DVT / (16 * MT), threads = waves * 64;
    static constexpr int C = kChunkBytes / size;        // tokens of a chunk
    static constexpr int CT = C / 16;                   // 16-row tiles of it
    static constexpr int span = 4 * elems;              // that a product sums over
    static constexpr int KS = C / span;                 // parts of a chunk's tokens
    static constexpr int NT = DK / 16, US = DK / span;  // tiles and parts of dk
    // score tiles of a wave, side by side in a row of tiles
    static constexpr int JT = CT * CT > waves ? CT * CT / waves : 1;
    static constexpr int parts = std::is_same_v<T, bf16> ? 3 : std::is_same_v<T, f16> ? 2 : 1;
    static constexpr bool is_f16 = std::is_same_v<T, f16>;
    // Numbers of T that a score and, where it meets q, an element of the state become:
    // two leave the results' error at their own rounding.  (With one, both roundings add
    // to it, 1.4 times as much and, where few numbers are summed, up to twice as much;
    // 8 x 4096 tokens, 16 heads of 128 bfloat16 136 us instead of 157.)
    static constexpr int score_parts = size == 4 ? 1 : 2, state_parts = score_parts;
    // Scores are scaled up by 2^48 at most, and the results that they are added to with
    // them: smaller scores, times values below 2^16, are nothing in a float16 result.
    static constexpr int kScoreUp = 48;
    using QK = Tile<T, C, DK, threads>;
    using VV = Tile<T, C, DVT, threads>;
    static constexpr int pitch = kChunkBytes + 16;      // of the scores' rows in LDS
    static constexpr int plane = C * pitch;             // of one of their parts
    // powers of the decay in LDS: number k is a^(C - k), and 0 from C + 1 on
    static constexpr int powers = 2 * C;
    typedef __attribute__((address_space(3))) const float *table;

    f32x4 S[NT][MT];    // rows 16 n + 4 g .. + 3 of column i of 16 of the wave's
    int thread, lane, wave, g, i;
    table pw;
    float near_pw[elems];       // a^(elems - 1 - m)

    __device__ __forceinline__ Body(table powers_, float ld)
        : thread(threadIdx.x), lane(thread & 63),
          wave(__builtin_amdgcn_readfirstlane(threadIdx.x >> 6)), g(lane >> 4), i(lane & 15),
          pw(powers_)
    {
#pragma unroll
        for (int m = 0; m < elems; ++m)
            near_pw[m] = __builtin_bit_cast(
                float, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(
                           int, expf(ld * (float)(elems - 1 - m)))));
    }
    static __device__ __forceinline__ void fill(float *to, float ld)
    {
        if ((int)threadIdx.x < powers)
            to[threadIdx.x] =
                (int)threadIdx.x <= C ? expf(ld * (float)(C - (int)threadIdx.x)) : 0.0f;
    }
    // At the start of a chunk and at the end: what follows from the lane is made anew, as
    // it would otherwise be kept over all chunks, in more registers than there are.
    __device__ __forceinline__ void next_chunk()
    {
        asm volatile("" : "+v"(thread));
        lane = thread & 63;
        g = lane >> 4;
        i = lane & 15;
    }

    // first of the wave's columns within the tile
    __device__ __forceinline__ int col0() const { return wave * 16 * MT; }

    // f(n, m, r, bytes) for the elements of a state array that is [Dk][Dv], or flipped:
    // bytes from its start, or (elements that it does not have) far away.
    template <typename F>
    __device__ __forceinline__ void places(const Walk &w, bool flip, int dv0, F f) const
    {
        const int dk_step = (flip ? 1 : w.Dv) * 4, dv_step = (flip ? w.Dk : 1) * 4;
#pragma unroll
        for (int m = 0; m < MT; ++m) {
            const int dv = dv0 + col0() + m * 16 + i;
            const int at = dv < w.Dv ? g * 4 * dk_step + dv * dv_step : kFar - DK * 1024;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int to = at + (n * 16 + r) * dk_step;
                    f(n, m, r, w.Dk == DK || n * 16 + g * 4 + r < w.Dk ? to : kFar);
                }
        }
    }
    // The state from memory (nullptr: zero) and to it.
    __device__ __forceinline__ void load_state(const Walk &w, const float *from, bool flip,
                                               int dv0)
    {
        // an empty descriptor reads as zero
        const __amdgpu_buffer_rsrc_t rsrc =
            dwconv::make_rsrc(from, from ? w.Dk * w.Dv * 4 : 0);
        places(w, flip, dv0, [&](int n, int m, int r, int at) {
            const unsigned v = __builtin_amdgcn_raw_buffer_load_b32(rsrc, at, 0, 0);
            S[n][m][r] = __builtin_bit_cast(float, v);
        });
    }
    __device__ __forceinline__ void store_state(const Walk &w, float *to, bool flip,
                                                int dv0) const
    {
        const __amdgpu_buffer_rsrc_t rsrc = dwconv::make_rsrc(to, w.Dk * w.Dv * 4);
        places(w, flip, dv0, [&](int n, int m, int r, int at) {
            const float v = S[n][m][r];
            __builtin_amdgcn_raw_buffer_store_b32(__builtin_bit_cast(unsigned, v), rsrc, at, 0,
                                                  0);
        });
    }

    // The wave's columns of V, as operands that are summed across the rows.
    __device__ __forceinline__ void columns(lds_ptr v, u32x4 (&f)[KS][MT]) const
    {
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
            for (int m = 0; m < MT; ++m)
                f[ks][m] = VV::across(v, col0() + m * 16, ks, lane);
    }

    // Whether they hold an infinity or a NaN, which are taken out.  (No matrix
    // instruction is at work here: see settle.)
    __device__ __forceinline__ bool strange(u32x4 (&f)[KS][MT]) const
    {
        unsigned odd = 0;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
#pragma unroll
            for (int m = 0; m < MT; ++m)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    odd |= odd_bits<T>(f[ks][m][e]);
        const bool any = __any(odd != 0);
        if (any)
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        f[ks][m][e] = cleaned<T>(f[ks][m][e]);
        return any;
    }

    // x as N numbers of T, pairs of them to a word.  bfloat16: the upper halves of x, of
    // what they leave, and of what that leaves, 8 bits each; the last of two is rounded.
    template <int N>
    static __device__ __forceinline__ void split(const float (&x)[elems], u32x4 (&p)[N])
    {
        if constexpr (std::is_same_v<T, bf16> && N > 1) {
            unsigned w[elems];
#pragma unroll
            for (int e = 0; e < elems; ++e)
                w[e] = __builtin_bit_cast(unsigned, x[e]);
#pragma unroll
            for (int q = 0; q < N; ++q) {
                if (N == 2 && q == 1) {
                    float rest[elems];
#pragma unroll
                    for (int e = 0; e < elems; ++e)
                        rest[e] = __builtin_bit_cast(float, w[e]);
                    unsigned word[4];
                    narrow<T, elems>(rest, word);
                    p[q] = u32x4{word[0], word[1], word[2], word[3]};
                    break;
                }
#pragma unroll
                for (int e = 0; e < elems; e += 2)      // the upper halves of two words
                    p[q][e / 2] = __builtin_amdgcn_perm(w[e + 1], w[e], 0x07060302u);
                if (q + 1 < N)
#pragma unroll
                    for (int e = 0; e < elems; ++e)
                        w[e] = __builtin_bit_cast(
                            unsigned, __builtin_bit_cast(float, w[e]) -
                                          __builtin_bit_cast(float, w[e] & 0xffff0000u));
            }
        } else {
            float rest[elems];
#pragma unroll
            for (int e = 0; e < elems; ++e)
                rest[e] = x[e];
#pragma unroll
            for (int q = 0; q < N; ++q) {
                unsigned word[4];
                narrow<T, elems>(rest, word);
                p[q] = u32x4{word[0], word[1], word[2], word[3]};
                if (q + 1 < N)
#pragma unroll
                    for (int e = 0; e < elems; ++e)
                        rest[e] -= element<T>(p[q], e);
            }
        }
    }

    // S = a^n S + s2 K^T (V with its decays).  vf: the wave's columns of V, without
    // infinities and NaN where there are `any`, which are added one by one: split in
    // parts they would leave NaN, and so would the zeros beside k's columns.
    __device__ __forceinline__ void update(const Walk &w, lds_ptr k, lds_ptr v,
                                           const u32x4 (&vf)[KS][MT], bool any, float a_n)
    {
        float up = 1.0f;
        if constexpr (is_f16) {     // small values would lose their last bits
            const auto largest = [&] {      // of columns without infinities
                float most = 0.0f;
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                    for (int m = 0; m < MT; ++m)
#pragma unroll
                        for (int e = 0; e < elems; ++e)
                            most = fmaxf(most, fabsf(element<T>(vf[ks][m], e)));
                return most * fabsf(w.s2);
            };
            up = range_scale(largest(), 0x1p-3f, 0x1p14f, largest);
            if (up > 1.0f) {    // the state is scaled with them
                float most = 0.0f;
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int m = 0; m < MT; ++m)
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            most = fmaxf(most, finite_size(S[t][m][r]));
                up = fminf(up, room_above(most));
            }
        }
        const float keep = a_n * up, s2 = w.s2 * up;
        const table late_pw = pw + (1 - w.late);        // a^(C - 1 - j + late) for row j
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int m = 0; m < MT; ++m)
                S[t][m] *= keep;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            // the lane's rows lie within `elems` adjacent ones: the last one's power,
            // times those of what the others are before it, which all lanes share
            const float last = late_pw[ks * span + g * elems + elems - 1] * s2;
            u32x4 p[MT][parts];
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                float x[elems];
#pragma unroll
                for (int e = 0; e < elems; ++e)
                    x[e] = element<T>(vf[ks][m], e) * (last * near_pw[VV::row_of(0, 0, e)]);
                split(x, p[m]);
            }
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                const u32x4 kf = QK::across(k, t * 16, ks, lane);
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int q = 0; q < parts; ++q)
                        mma<T>(kf, p[m][q], S[t][m]);
            }
        }
        settle();
        if constexpr (is_f16)
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int m = 0; m < MT; ++m)
                    S[t][m] *= inverse(up);
        if (any)
            for (int j = 0; j < C; ++j)
#pragma unroll
                for (int m = 0; m < MT; ++m) {
                    const float x = VV::one(v, j, col0() + m * 16 + i);
                    const float f = late_pw[j] * w.s2;
                    if (!(fabsf(x) <= 3.4e38f))
#pragma unroll
                        for (int t = 0; t < NT; ++t)
#pragma unroll
                            for (int r = 0; r < 4; ++r)
                                if (t * 16 + g * 4 + r < w.Dk)
                                    S[t][m][r] += f * QK::one(k, j, t * 16 + g * 4 + r) * x;
                }
    }

    // number h of the two in a word
    static __device__ __forceinline__ float part_of(unsigned word, int h)
    {
        return element<T>(u32x4{word, word, word, word}, h);
    }

    // Some tiles of a row of scores, times their decay, to LDS; the power of two that
    // they were divided by (float16) is returned.
    __device__ __forceinline__ float scores(lds_ptr q, lds_ptr k, lds_ptr p, float s0) const
    {
        const int row = wave % CT * 16 + i, col0 = wave / CT * JT * 16;
        if (wave / CT * JT >= CT)
            return 1.0f;
        f32x4 acc[JT];
#pragma unroll
        for (int t = 0; t < JT; ++t)
            acc[t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int u = 0; u < US; ++u) {
            const u32x4 qf = QK::template chunk<true>(q, row, u, g);
#pragma unroll
            for (int t = 0; t < JT; ++t)    // later tokens' too: no branch (see settle)
                mma<T>(QK::chunk(k, col0 + t * 16 + i, u, g), qf, acc[t]);
        }
        const int ahead = row - col0 - g * 4;       // of the first of the lane's columns
        const table gap_pw = pw + (C - ahead);
        float most = 0.0f, down = 1.0f, v[JT][4];
#pragma unroll
        for (int t = 0; t < JT; ++t)
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                // a score of a later token may be anything
                v[t][r] = ahead >= t * 16 + r ? acc[t][r] * (s0 * gap_pw[t * 16 + r]) : 0.0f;
                if constexpr (is_f16)
                    most = fmaxf(most, fabsf(v[t][r]));
            }
        if constexpr (is_f16)
            down = range_scale(most, 0x1p-2f, 0x1p14f, [&] {
                float m = 0.0f;
#pragma unroll
                for (int t = 0; t < JT; ++t)
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        m = fmaxf(m, finite_size(v[t][r]));
                return m;
            }, kScoreUp);
#pragma unroll
        for (int t = 0; t < JT; ++t) {
            if constexpr (is_f16)
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    v[t][r] *= down;
            // column 8a + 2m + h of a row is kept as number 4h + m of its chunk a: the
            // order in which across() reads the rows of V
            const lds_ptr to = p + row * pitch + (col0 + t * 16) * size;
            if constexpr (size == 4) {
                unsigned word[4];
                narrow<T, 4>(v[t], word);
                *(lds_u4)(to + g * 16) = u32x4{word[0], word[1], word[2], word[3]};
            } else {
                const lds_ptr at = to + (g >> 1) * 16 + (g & 1) * 4;
                float x[4] = {v[t][0], v[t][2], v[t][1], v[t][3]};
#pragma unroll
                for (int q = 0; q < score_parts; ++q) {
                    unsigned word[2];
                    narrow<T, 4>(x, word);
                    *(lds_u1)(at + q * plane) = word[0];
                    *(lds_u1)(at + q * plane + 8) = word[1];
#pragma unroll
                    for (int r = 0; r < 4; ++r) {       // nothing is left of an infinity
                        const float rest = x[r] - part_of(word[r / 2], r % 2);
                        x[r] = fabsf(rest) <= 3.4e38f ? rest : 0.0f;
                    }
                }
            }
        }
        return down;
    }

    // o[t][m]: columns 4 g .. + 3 of 16 of the wave's, row i of the 16 of tile t:
    // s1 a^(row - first + 1 - late) q S, `first` the chunk's first row
    __device__ __forceinline__ void from_state(lds_ptr q, f32x4 (&o)[CT][MT], float s1, int late,
                                               int first)
    {
#pragma unroll
        for (int t = 0; t < CT; ++t)
#pragma unroll
            for (int m = 0; m < MT; ++m)
                o[t][m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        float down = 1.0f;
        unsigned rest = ~0u;    // 0: infinities among the lane's elements, which leave NaN
        const auto largest = [&](auto size_of) {
                float most = 0.0f;
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int m = 0; m < MT; ++m)
#pragma unroll
                        for (int r = 0; r < 4; ++r)
                            most = fmaxf(most, size_of(S[n][m][r]));
                return most;
        };
        if constexpr (size == 2) {
            const float most = largest([](float v) { return fabsf(v); });
            if constexpr (is_f16)
                down = range_scale(most, 0x1p-2f, 0x1p14f, [&] { return largest(finite_size); });
            if constexpr (state_parts > 1)
                rest = most > 3.4e38f ? 0u : ~0u;
        }
#pragma unroll
        for (int u = 0; u < US; ++u) {
            u32x4 sf[MT][state_parts];
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                float f[elems];
#pragma unroll
                for (int e = 0; e < elems; ++e)
                    f[e] = S[u * (elems / 4) + e / 4][m][e % 4] * (is_f16 ? down : 1.0f);
                split(f, sf[m]);
                if constexpr (state_parts > 1)
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        sf[m][1][e] &= rest;
            }
#pragma unroll
            for (int t = 0; t < CT; ++t) {
                const u32x4 qf = QK::along(q, t * 16 + i, u, g);
#pragma unroll
                for (int m = 0; m < MT; ++m)
#pragma unroll
                    for (int z = 0; z < state_parts; ++z)
                        mma<T>(sf[m][z], qf, o[t][m]);
            }
        }
#pragma unroll
        for (int t = 0; t < CT; ++t) {
            const int n = max(t * 16 + i + 1 - late - first, 0);
            const float f = s1 * pw[C - n] * inverse(down);
#pragma unroll
            for (int m = 0; m < MT; ++m)
                o[t][m] *= f;
        }
    }

    // o += P V.  Infinities and NaN of V are added one by one: a zero score of a later
    // token times those would be NaN.
    __device__ __forceinline__ void from_scores(lds_ptr p, lds_ptr v, const float *downs,
                                                const u32x4 (&f)[KS][MT], bool any,
                                                f32x4 (&o)[CT][MT])
    {
        // what the scores of row tile t, part ks, were divided by
        auto down_of = [&](int t, int ks) {
            return is_f16 ? downs[t + ks * (span / 16) / JT * CT] : 1.0f;
        };
        auto product = [&](auto scaled) {
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                for (int t = 0; t < CT; ++t)
                    if (ks * span <= t * 16 + 15) {
                        u32x4 pf[score_parts];
#pragma unroll
                        for (int q = 0; q < score_parts; ++q)
                            pf[q] = *(lds_u4)(p + q * plane + (t * 16 + i) * pitch +
                                              (ks * 4 + g) * 16);
#pragma unroll
                        for (int m = 0; m < MT; ++m) {
                            if constexpr (scaled.value)
                                o[t][m] *= down_of(t, ks);
#pragma unroll
                            for (int q = 0; q < score_parts; ++q)
                                mma<T>(f[ks][m], pf[q], o[t][m]);
                            if constexpr (scaled.value)
                                o[t][m] *= inverse(down_of(t, ks));
                        }
                    }
        };
        if constexpr (is_f16) {
            const float mine = downs[lane % waves];
            if (__any(mine != 1.0f))
                product(std::true_type());
            else
                product(std::false_type());
        } else {
            product(std::false_type());
        }
        settle();
        if (any)
            for (int j = 0; j < C; ++j) {
                // where column j of the scores is kept
                const int slot = size == 4 ? j : (j & ~7) | (j & 1) << 2 | (j >> 1 & 3);
#pragma unroll
                for (int t = 0; t < CT; ++t) {
                    const float s =
                        (float)*(__attribute__((address_space(3))) const T *)(
                            p + (t * 16 + i) * pitch + slot * size) * inverse(down_of(t, j / span));
#pragma unroll
                    for (int m = 0; m < MT; ++m)
#pragma unroll
                        for (int r = 0; r < 4; ++r) {
                            const float x = VV::one(v, j, col0() + m * 16 + g * 4 + r);
                            if (j <= t * 16 + i && !(fabsf(x) <= 3.4e38f))
                                o[t][m][r] += s * x;
                        }
                }
            }
    }

    // Results of T go through the tile of V, whose columns a wave has read and writes
    // alone, so that whole rows are stored, 16 bytes a lane.
    static constexpr int words = 4 * size / 4;
    __device__ __forceinline__ void pack(const f32x4 (&o)[CT][MT],
                                         unsigned (&to)[CT][MT][words]) const
    {
#pragma unroll
        for (int c = 0; c < CT; ++c)
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const f32x4 v = o[c][m];
                const float s[4] = {v[0], v[1], v[2], v[3]};
                narrow<T, 4>(s, to[c][m]);
            }
    }
    __device__ __forceinline__ void spread(lds_ptr v, const unsigned (&w)[CT][MT][words]) const
    {
#pragma unroll
        for (int c = 0; c < CT; ++c)
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const lds_ptr at = v + (c * 16 + i) * VV::pitch + (col0() + m * 16 + g * 4) * size;
                if constexpr (size == 4)
                    *(lds_u4)at = u32x4{w[c][m][0], w[c][m][1], w[c][m][2], w[c][m][3]};
                else
                    *(lds_u2)at = u32x2{w[c][m][0], w[c][m][1]};
            }
    }
    // (A thread reads what it will write of the next V itself.)  The results are stored
    // past the caches, which keep the inputs that other passes read: 8 x 4096 tokens, 16
    // heads of 128 bfloat16 149 us for 160, gradients of 8 x 2048 78 for 84 a walk.  With a
    // kernel behind it that reads the results 275 us for 280, 2 x 4096 tokens 100 for 102, 1 x
    // 512 25.9 for 25.6 (it then waits for HBM by itself).
    static constexpr int kPast = 2;     // the "nt" bit of a store
    __device__ __forceinline__ void store_rows(lds_ptr v, const Walk &w, long long row0, int t,
                                               int first, int h, int dv0) const
    {
        const int wide = w.Dv - dv0, ldo = (int)w.ldo * size;
        const long long lowest = w.back ? row0 - t - (C - 1) : row0 + t;
        const __amdgpu_buffer_rsrc_t rsrc = dwconv::make_rsrc(
            static_cast<T *>(w.out) + lowest * w.ldo + h * w.Dv + dv0, kFar - 16);
        const int row = thread / VV::per_row, col = thread % VV::per_row * elems;
        typedef unsigned u4 __attribute__((ext_vector_type(4)));
#pragma unroll
        for (int k = 0; k < VV::count; ++k) {
            const int r = row + k * VV::apart;
            const u4 x = *(__attribute__((address_space(3))) u4 *)(v + r * VV::pitch + col * size);
            const int at = (w.back ? C - 1 - r : r) * ldo + col * size;
            __builtin_amdgcn_raw_buffer_store_b128(x, rsrc, r >= first && col < wide ? at : kFar,
                                                   0, kPast);
        }
    }

    // The chunk's rows from `first` on, 4 adjacent columns a lane; its row 0 is token t.
    template <bool CUT, typename E>
    __device__ __forceinline__ void store(E *out, const Walk &w, const f32x4 (&o)[CT][MT],
                                          long long row0, int t, int first, int h,
                                          int dv0) const
    {
        const int wide = w.Dv - dv0, ldo = (int)w.ldo * (int)sizeof(E);
        const long long lowest = w.back ? row0 - t - (C - 1) : row0 + t;
        const __amdgpu_buffer_rsrc_t rsrc =
            dwconv::make_rsrc(out + lowest * w.ldo + h * w.Dv + dv0, kFar - 16);
#pragma unroll
        for (int c = 0; c < CT; ++c)
#pragma unroll
            for (int m = 0; m < MT; ++m) {
                const int r = c * 16 + i, dv = col0() + m * 16 + g * 4;
                const int at = (w.back ? C - 1 - r : r) * ldo + dv * (int)sizeof(E);
                const f32x4 v = o[c][m];
                const float s[4] = {v[0], v[1], v[2], v[3]};
                if constexpr (!CUT) {
                    Raw<E, 4>(s).store(rsrc, r >= first && dv < wide ? at : kFar, 0);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const float one[1] = {s[e]};
                        Raw<E, 1>(one).store(
                            rsrc, r >= first && dv + e < wide ? at + e * (int)sizeof(E) : kFar,
                            0);
                    }
                }
            }
    }
};

// The rows of a walk's tensor: from token t on, the row of lowest address of a chunk.
template <typename T, int C> struct Rows {
    const T *base;          // token 0's row
    long long step;         // elements from a token to the next
    bool back;
    __device__ __forceinline__ Rows(const void *p, long long ld, bool turned, long long row,
                                    int column)
        : base(static_cast<const T *>(p) + row * ld + column), step(turned ? -ld : ld),
          back(turned)
    {
    }
    __device__ __forceinline__ const T *at(int t) const
    {
        return base + (back ? t + C - 1 : t) * step;
    }
};

// A chunk of a segment of n tokens: its row 0 is token t, and rows before `first` are
// zero.  The last chunk ends with the segment, so that a row is as far from the end
// of its chunk in all of them.
struct Chunk {
    int done, n, C, t, first;
    __device__ __forceinline__ Chunk(int n_, int C_, int done_ = 0) : done(done_), n(n_), C(C_)
    {
        first = C - max(min(C, n - done), 0);
        t = done - first;
    }
    __device__ __forceinline__ bool any() const { return done < n; }
    __device__ __forceinline__ Chunk next() const { return Chunk(n, C, done + C); }
};

// A workgroup's walk, and its number there.
struct Which {
    int i, block;
    __device__ __forceinline__ explicit Which(const Walks &all) : i(0), block((int)block_id())
    {
#pragma unroll
        for (int k = 0; k + 1 < kWalks; ++k)
            if (i == k && block >= all.blocks[k]) {
                block -= all.blocks[k];
                ++i;
            }
    }
};

// What a workgroup walks.
struct Part {
    int item, h, dv0;
    __device__ __forceinline__ Part(const Walk &w, int tile, int block)
    {
        const int tiles = (w.Dv + tile - 1) / tile;
        const int b = dwconv::xcd_tile(block, w.items * w.H * tiles);
        dv0 = b % tiles * tile;
        h = b / tiles % w.H;
        item = b / tiles / w.H;
    }
};

// Two workgroups a CU, with registers for them.
constexpr int waves_a_simd(int DK, int DVT, int MT)
{
    return DK > 128 || DVT < 32 * MT ? 1 : DVT / (16 * MT) * 2 / 4;
}

// The state that a segment adds by itself, to the slot of the next one.
template <typename T, int DK, int DVT, int MT, Mode MODE>
__global__ __launch_bounds__(DVT / MT * 4, waves_a_simd(DK, DVT, MT)) void k_states(Walks all)
{
    const Which which(all);
    const Walk &w = all.w[which.i];
    using B = Body<T, DK, DVT, MT>;
    __shared__ alignas(16) char lds[B::QK::bytes + B::VV::bytes];
    __shared__ float powers[B::powers];
    const lds_ptr lk = (lds_ptr)lds, lv = lk + B::QK::bytes;
    if (which.block >= w.items * w.H * (int)((w.Dv + DVT - 1) / DVT))
        return;
    const Part part(w, DVT, which.block);
    const Item at(w, part.item);
    if (at.seg + 1 >= at.segments(w))
        return;
    const float ld = log_decay_of(w.log_decay, part.h);
    B::fill(powers, ld);
    B b((typename B::table)powers, ld);
#pragma unroll
    for (int n = 0; n < B::NT; ++n)
#pragma unroll
        for (int m = 0; m < MT; ++m)
            b.S[n][m] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    const int t0 = at.seg * w.segment, n = w.segment;       // a whole one
    const long long row = w.back ? (long long)at.row0 + at.length - 1 - t0 : at.row0 + t0;
    const Rows<T, B::C> k(w.k, w.ldk, w.back, row, part.h / w.gk * w.Dk),
        v(w.v, w.ldv, w.back, row, part.h / w.gv * w.Dv + part.dv0);
    const int wide = w.Dv - part.dv0, ldk = (int)w.ldk, ldv = (int)w.ldv;
    const float whole = (float)exp((double)ld * B::C);
    // two chunks on their way: there are fewer workgroups than the chip holds, and
    // little to do but to wait for memory
    Chunk c(n, B::C);
    u32x4 rk[2][B::QK::count], rv[2][B::VV::count];
    auto fetch = [&](auto p, const Chunk &x) {
        B::QK::template fetch<MODE == ODD>(rk[p.value], k.at(x.t), ldk, w.back, x.first, w.Dk,
                                           b.thread);
        B::VV::template fetch<MODE == ODD>(rv[p.value], v.at(x.t), ldv, w.back, x.first, wide,
                                           b.thread);
    };
    auto step = [&](auto p) {
        b.next_chunk();
        B::QK::keep(lk, rk[p.value], b.thread);
        B::VV::keep(lv, rv[p.value], b.thread);
        __syncthreads();
        fetch(p, c.next().next());
        u32x4 vf[B::KS][MT];
        b.columns(lv, vf);
        const bool any = b.strange(vf);
        b.update(w, lk, lv, vf, any,
                 c.first == 0 ? whole : expf(ld * (float)(B::C - c.first)));
        __syncthreads();
        c = c.next();
    };
    constexpr std::integral_constant<int, 0> even;
    constexpr std::integral_constant<int, 1> odd;
    fetch(even, c);
    fetch(odd, c.next());
    while (c.any()) {
        step(even);
        if (c.any())
            step(odd);
    }
    b.next_chunk();
    const int slot = slot_of(w, at.row0, at.seg + 1);
    b.store_state(w, w.slots + ((long long)slot * w.H + part.h) * w.Dk * w.Dv, false, part.dv0);
}

// The segments' own states, each to be added to what it gets from those before it.  A
// thread takes 4 adjacent elements (or one, where a state is no whole number of 4); the
// segments of a sequence one after the other.  (Workgroups of one wave: 1 x 65537 tokens,
// 8 heads of 128, 18.3 us for 19.8, but gradients of 23 short sequences 15.9 for 13.8; 16
// slots on their way instead of 4: 13.2 for 11.0 with 4 segments.)
template <int V>
__global__ __launch_bounds__(256) void k_link(Walks all, int blocks)
{
    const Which which(all);
    const Walk &w = all.w[which.i];
    const int id = which.block, size = w.Dk * w.Dv;
    if (id >= w.batch.seqs * w.H * blocks)
        return;
    const int at = (id % blocks * 256 + (int)threadIdx.x) * V;
    const int h = id / blocks % w.H, seq = id / blocks / w.H;
    if (at >= size)
        return;
    // (from the sequence itself, which offsets that break the rules leave within the rows
    // and so within the slots)
    const int row0 = seq_start(w.batch, seq), end = seq_start(w.batch, seq + 1);
    const int count = Item::count(w, max(end - row0, 0));
    if (count == 1)
        return;
    const float ld = log_decay_of(w.log_decay, h);
    const float a = (float)exp((double)ld * w.segment);
    float run[V] = {};
    if (w.state0)
#pragma unroll
        for (int e = 0; e < V; ++e)
            run[e] = w.state0[((long long)seq * w.H + h) * size +
                              state_at(w, w.flip, (at + e) / w.Dv, (at + e) % w.Dv)];
    float *slot = w.slots + ((long long)slot_of(w, row0, 1) * w.H + h) * size + at;
    const long long next = (long long)w.H * size;
    constexpr int kAhead = 4;
    for (int j = 0; j < count - 1; j += kAhead) {
        float v[kAhead][V];
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            load<float, V>(slot + min(j + u, count - 2) * next, v[u]);
#pragma unroll
        for (int u = 0; u < kAhead; ++u)
            if (j + u < count - 1) {
#pragma unroll
                for (int e = 0; e < V; ++e)
                    run[e] = a * run[e] + v[u][e];
                store<float, V>(slot + (j + u) * next, run);
            }
    }
}

template <typename T, int DK, int DVT, int MT, Mode MODE>
__global__ __launch_bounds__(DVT / MT * 4, waves_a_simd(DK, DVT, MT)) void k_walk(Walks all)
{
    const Which which(all);
    const Walk &w = all.w[which.i];
    using B = Body<T, DK, DVT, MT>;
    __shared__ alignas(16) char lds[2 * B::QK::bytes + B::VV::bytes + B::score_parts * B::plane];
    __shared__ float downs[B::waves], powers[B::powers];
    const lds_ptr lq = (lds_ptr)lds, lk = lq + B::QK::bytes, lv = lk + B::QK::bytes,
                  lp = lv + B::VV::bytes;
    if (which.block >= w.items * w.H * (int)((w.Dv + DVT - 1) / DVT))
        return;
    const Part part(w, DVT, which.block);
    const Item at(w, part.item);
    const int count = at.segments(w);
    if (at.seg >= count)
        return;
    const float ld = log_decay_of(w.log_decay, part.h);
    B::fill(powers, ld);
    B b((typename B::table)powers, ld);
    const long long size = (long long)w.Dk * w.Dv;
    const long long own = ((long long)at.seq * w.H + part.h) * size;
    const long long slot = slot_of(w, at.row0, at.seg);
    const float *from = at.seg ? w.slots + (slot * w.H + part.h) * size
                               : w.state0 ? w.state0 + own : nullptr;
    b.load_state(w, from, at.seg ? w.ready : w.flip, part.dv0);
    const int t0 = at.seg * w.segment, n = min(w.segment, at.length - t0);
    const long long row = w.back ? (long long)at.row0 + at.length - 1 - t0 : at.row0 + t0;
    const Rows<T, B::C> q(w.q, w.ldq, w.back, row, part.h / w.gq * w.Dk),
        k(w.k, w.ldk, w.back, row, part.h / w.gk * w.Dk),
        v(w.v, w.ldv, w.back, row, part.h / w.gv * w.Dv + part.dv0);
    const int wide = w.Dv - part.dv0, ldq = (int)w.ldq, ldk = (int)w.ldk, ldv = (int)w.ldv;
    const float whole = (float)exp((double)ld * B::C);
    Chunk c(n, B::C);
    u32x4 rq[B::QK::count], rk[B::QK::count], rv[B::VV::count];
    auto fetch = [&](const Chunk &x) {
        B::QK::template fetch<MODE == ODD>(rq, q.at(x.t), ldq, w.back, x.first, w.Dk, b.thread);
        B::QK::template fetch<MODE == ODD>(rk, k.at(x.t), ldk, w.back, x.first, w.Dk, b.thread);
        B::VV::template fetch<MODE == ODD>(rv, v.at(x.t), ldv, w.back, x.first, wide, b.thread);
    };
    fetch(c);
    for (; c.any(); c = c.next()) {
        const Chunk next = c.next();
        b.next_chunk();
        B::QK::template keep<true>(lq, rq, b.thread);
        B::QK::keep(lk, rk, b.thread);
        B::VV::keep(lv, rv, b.thread);
        __syncthreads();
        // The next chunk's rows.  16-bit types send for them once scores and results are
        // done: next to the parts of S there are no registers for them, and spilled, they
        // are waited for at once (20011 tokens in 37 sequences, 12 heads of 96 and 80
        // float16 138 us, so 106; bfloat16 takes either as long).
        if constexpr (sizeof(T) == 4)
            fetch(next);
        __builtin_amdgcn_sched_barrier(0);
        const float down = b.scores(lq, lk, lp, w.s0);
        if (B::is_f16 && b.lane == 0)
            downs[b.wave] = down;
        __builtin_amdgcn_sched_barrier(0);
        f32x4 o[B::CT][MT];
        b.from_state(lq, o, w.s1, w.late, c.first);
        __syncthreads();
        __builtin_amdgcn_sched_barrier(0);
        u32x4 vf[B::KS][MT];
        b.columns(lv, vf);
        const bool any = b.strange(vf);
        b.from_scores(lp, lv, downs, vf, any, o);
        unsigned ow[B::CT][MT][B::words];
        if constexpr (MODE == ROWS) {
            b.pack(o, ow);
        } else {
            if (MODE == PARTS || w.out32)
                b.template store<MODE == ODD>(static_cast<float *>(w.out), w, o, row, c.t,
                                              c.first, part.h, part.dv0);
            else if (w.out)
                b.template store<MODE == ODD>(static_cast<T *>(w.out), w, o, row, c.t, c.first,
                                              part.h, part.dv0);
        }
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (sizeof(T) == 2)
            fetch(next);
        b.update(w, lk, lv, vf, any,
                 c.first == 0 ? whole : expf(ld * (float)(B::C - c.first)));
        if constexpr (MODE == ROWS)
            b.spread(lv, ow);
        __syncthreads();
        if (MODE == ROWS && w.out)
            b.store_rows(lv, w, row, c.t, c.first, part.h, part.dv0);
    }
    b.next_chunk();
    if (w.state1 && at.seg + 1 == count)
        b.store_state(w, w.state1 + own, w.flip, part.dv0);
}

}  // namespace

// The kernel that a walk takes.
struct Kind {
    int dk, dvt;
    Mode mode;
    bool operator==(const Kind &o) const
    {
        return dk == o.dk && dvt == o.dvt && mode == o.mode;
    }
};

template <typename T> Kind kind_of(const Walk &w)
{
    const int whole = 16 / (int)sizeof(T);
    const Mode mode = w.Dk % whole || w.Dv % whole ? ODD
                      : sizeof(T) == 2 && w.out32  ? PARTS
                                                   : ROWS;
    return {w.Dk > 128 ? 256 : w.Dk > 64 ? 128 : 64, walk_tile(w.Dk, w.Dv), mode};
}

template <typename T, typename F> int with_kind(const Kind &k, F f)
{
    using std::integral_constant;
    auto mode = [&](auto dk, auto dvt) {
        if (k.mode == ODD)
            return f(dk, dvt, integral_constant<Mode, ODD>());
        if constexpr (sizeof(T) == 2)
            if (k.mode == PARTS)
                return f(dk, dvt, integral_constant<Mode, PARTS>());
        return f(dk, dvt, integral_constant<Mode, ROWS>());
    };
    if (k.dk == 256)
        return mode(integral_constant<int, 256>(), integral_constant<int, 64>());
    if (k.dk == 128)
        return k.dvt > 64 ? mode(integral_constant<int, 128>(), integral_constant<int, 128>())
                          : mode(integral_constant<int, 128>(), integral_constant<int, 64>());
    return k.dvt > 64 ? mode(integral_constant<int, 64>(), integral_constant<int, 128>())
                      : mode(integral_constant<int, 64>(), integral_constant<int, 64>());
}

// Walks gathered for one launch.
struct Gather {
    Walks all{};
    int count = 0;
    long long total = 0;
    void add(const Walk &w, long long blocks)
    {
        blocks = cdiv(blocks, 8) * 8;
        total += blocks;
        all.w[count] = w;
        all.blocks[count++] = (int)std::min(blocks, 0x7fffffffLL);
    }
    // f(grid) launches; the last walk's number of workgroups is not looked at
    template <typename F> int launch(F f) const
    {
        return count == 0 ? (int)DWCONV_OK : f(grid_of(total));
    }
};

// For each kind among the walks that `wanted` names, one launch.
template <typename W, typename K, typename F>
int for_kinds(const Walk *w, int count, W wanted, K kind, F launch)
{
    bool done[kWalks] = {};
    int rc = DWCONV_OK;
    for (int i = 0; i < count && rc == DWCONV_OK; ++i) {
        if (done[i] || !wanted(w[i]))
            continue;
        const Kind k = kind(w[i]);
        Gather g;
        for (int j = i; j < count; ++j)
            if (!done[j] && wanted(w[j]) && kind(w[j]) == k) {
                g.add(w[j], (long long)w[j].items * w[j].H * cdiv(w[j].Dv, k.dvt));
                done[j] = true;
            }
        rc = launch(k, g);
    }
    return rc;
}

template <typename T> int launch_walks(const Walk *w, int count, hipStream_t st)
{
    auto cut = [](const Walk &x) { return x.slots && !x.ready; };
    long long most = 0;     // no launch before all are known to fit
    for (int i = 0; i < count; ++i) {
        const long long walk = (long long)w[i].items * w[i].H * cdiv(w[i].Dv, 64);
        const long long link = (long long)w[i].batch.seqs * w[i].H * cdiv(w[i].Dk * w[i].Dv, 256);
        most += std::max(walk, cut(w[i]) ? link : 0) + 8;
    }
    if (most > 0x7fffffffLL - kGridRow)
        return DWCONV_ERR_BAD_DIM;
    int rc = for_kinds(
        w, count, cut,
        [](const Walk &x) {         // states have no results
            Kind k = kind_of<T>(x);
            k.mode = k.mode == ODD ? ODD : ROWS;
            return k;
        },
        [&](const Kind &kind, const Gather &g) {
            return with_kind<T>(kind, [&](auto dk, auto dvt, auto mode) {
                constexpr int DK = decltype(dk)::value, DVT = decltype(dvt)::value;
                constexpr Mode MODE = decltype(mode)::value == ODD ? ODD : ROWS;
                return g.launch([&](dim3 grid) {
                    return dwconv::launch_kernel(k_states<T, DK, DVT, 1, MODE>, grid,
                                                 dim3(DVT * 4), 0, st, g.all);
                });
            });
        });
    if (rc != DWCONV_OK)
        return rc;
    Gather links;
    bool by4 = true;        // the same for all: Dk * Dv is
    int wide = 0;
    for (int i = 0; i < count; ++i)
        if (cut(w[i])) {
            by4 = w[i].Dk * w[i].Dv % 4 == 0;
            wide = (int)cdiv(w[i].Dk * w[i].Dv, by4 ? 1024 : 256);
            links.add(w[i], (long long)w[i].batch.seqs * w[i].H * wide);
        }
    rc = links.launch([&](dim3 grid) {
        return by4 ? dwconv::launch_kernel(k_link<4>, grid, dim3(256), 0, st, links.all, wide)
                   : dwconv::launch_kernel(k_link<1>, grid, dim3(256), 0, st, links.all, wide);
    });
    if (rc != DWCONV_OK)
        return rc;
    return for_kinds(
        w, count, [](const Walk &) { return true; }, [](const Walk &x) { return kind_of<T>(x); },
        [&](const Kind &kind, const Gather &g) {
            return with_kind<T>(kind, [&](auto dk, auto dvt, auto mode) {
                constexpr int DK = decltype(dk)::value, DVT = decltype(dvt)::value;
                return g.launch([&](dim3 grid) {
                    return dwconv::launch_kernel(k_walk<T, DK, DVT, 1, decltype(mode)::value>,
                                                 grid, dim3(DVT * 4), 0, st, g.all);
                });
            });
        });
}
#endif  // DWMIX_ATTENTION_KERNELS

}  // namespace dwmix

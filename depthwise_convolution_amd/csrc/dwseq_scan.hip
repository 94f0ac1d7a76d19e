// dwseq_scan.hip -- gated linear recurrence: forward, single-token step and
// gradients (include/dwconv_seq.h).
//
//   h[t] = a[t] h[t-1] + b[t],  a = e^L,  b = sqrt(1 - a^2) sigma(i) x,
//   L = -scale softplus(lam) sigma(r)
//
// Steps compose: applying (a1, b1) and then (a2, b2) is (a1 a2, a2 b1 + b2),
// which lets the tokens be scanned in parallel.  A workgroup takes 64 channels of
// one run of a sequence (128 tokens): a thread holds V channels of a few
// consecutive tokens in registers and folds them to one (a, b); the folds are
// scanned over the lanes of a wave that hold the same channels, then over the
// waves in LDS.  What is missing then is the state at the run's beginning, which
// comes from the runs before it: every workgroup publishes its run's (a, b) and,
// as soon as it knows it, the state after its run, and looks back over the
// last runs for the nearest known state, to which it applies the (a, b) between in
// order.  So each input is read once, h never leaves float32 registers on its
// way, and a sequence is spread over the whole chip.
//
// The waiting ends: runs are handed out by a counter in an order in which a run
// comes after those it waits for, so these have all started, on workgroups
// that keep their CU until they are done.  The order of arithmetic does not depend on
// timing: a state found further back is carried forward by the very operations
// that its own workgroups use.
//
// What bounds it: 4 arrays of 16 bits moved an element (forward) against 35
// instructions of the vector unit in the forward and 66 in the gradient, six and
// more of them at a quarter of the rate.  Neither is at its limit, as a run's loads, scan
// and stores follow one another in a workgroup and registers leave 3 (2) of them a
// CU: at 8 x 2048 x 2048 bfloat16 the forward takes 72 us (3.7 TB/s; a large copy
// 6.3) and the gradient 121 us (4.0 TB/s), at 1 x 65537 x 1280 the forward 176 us (3.8
// TB/s), of which the chain of 512 runs costs a tenth; the vector unit is active half
// of the time.  float32 takes 130 and 213 us, and 261: its rows of 4 words do not fit
// beside the gates (40 and 92 bytes of scratch a lane).  A run of 128 tokens is what 256
// threads hold in registers, 8 tokens of 4 channels each; a sequence's last run
// computes the gates of all 128, so that 64 sequences of 8 tokens, 2048 channels, take
// 20 us.
#include "dwseq_device.h"

namespace dwseq {
namespace {

constexpr int kRun = 128;                       // tokens that a workgroup scans
constexpr int kKept = DWCONV_SCAN_RUN;          // tokens from one kept state to the next
constexpr int kSlab = 64;       // channels of a workgroup
constexpr float kLog2e = 1.44269504088896341f;

// e^-|v| to 3 roundings for any v.  The hardware's exponential takes the product
// with log2(e), whose rounding alone would cost |v| / 2 of them; what the rounding
// and the constant lose is multiplied back.  (Past 200 the result is 0; a NaN stays.)
__device__ __forceinline__ float exp_neg(float v)
{
    constexpr float kRest = 1.925962989e-8f, kLn2 = 0.693147180559945f;  // log2(e) - kLog2e
    const float n = -__builtin_fabsf(v), x = n < -200.0f ? -200.0f : n;
    const float y = x * kLog2e;
    const float rest = fmaf(x, kRest, fmaf(x, kLog2e, -y));
    const float e = __builtin_amdgcn_exp2f(y);
    return fmaf(e, rest * kLn2, e);
}

// Decay constant of a channel: scale * softplus(lam), softplus(v) = max(v, 0) +
// log(1 + e), e = exp(-|v|).  Every thread of a run computes it for its
// channels, so the logarithm is short: for e up to 1/2 (very negative lam, the
// long memories, where log(1 + e) is about e) the polynomial of degree 6 for
// log(1 + e) / e with the least relative error (6.1e-8 with rounded
// coefficients, fitted on 4001 points), else the hardware's of 1 + e.  In all some
// 7 roundings of 2^-24.
__device__ __forceinline__ float decay_rate(float lam, float scale)
{
    const float e = exp_neg(lam);
    float q = fmaf(e, 3.867349773645401e-2f, -1.136968806385994e-1f);
    q = fmaf(e, q, 1.845046728849411e-1f);
    q = fmaf(e, q, -2.475198209285736e-1f);
    q = fmaf(e, q, 3.331380784511566e-1f);
    q = fmaf(e, q, -4.999941289424896e-1f);
    q = fmaf(e, q, 1.0f);
    const float near = e * q;
    const float far = __builtin_amdgcn_logf(1.0f + e) * 0.693147180559945f;
    return scale * (fmaxf(lam, 0.0f) + (e <= 0.5f ? near : far));
}

// One token's gate: a = e^-u and, without the cancellation of 1 - a,
// m = 1 - a = u (1 - u/2 + u^2/6 - ...), for u up to kSmall by the polynomial of
// degree 4 with the least relative error there (3.2e-8, its coefficients fitted
// on 4001 points).  a itself is then 1 - m, rounded once: over a long memory, an
// error of one sign in a would grow with 1 / (1 - a).  SMALL: every u of the
// workgroup is known to be small (u is at most the channel's rate), which saves
// the exponential and the choice: a quarter of a token's operations, and the
// scan is bound by those as much as by HBM.
constexpr float kSmall = 0.35f;

template <bool SMALL>
__device__ __forceinline__ void decay(float u, float &a, float &m)
{
    float q = fmaf(u, 7.204961031675339e-3f, -4.1327446699142456e-2f);
    q = fmaf(u, q, 1.6662432253360748e-1f);
    q = fmaf(u, q, -4.999981224536896e-1f);
    q = fmaf(u, q, 1.0f);
    m = u * q;
    a = 1.0f - m;
    if (!SMALL) {
        const float e = __builtin_amdgcn_exp2f(-u * kLog2e);
        const bool small = u <= kSmall;
        m = small ? m : 1.0f - e;
        a = small ? a : e;
    }
}

// A gate sigma(v) kept with its complement: the smaller of the two, t / (1 + t)
// with t = e^-|v|, with a minus sign where that is 1 - sigma(v).  The gradients
// need both; 1 - sigma(v) taken from a sigma(v) rounded near 1 would have an error
// of 2^-24 in a value of e^-v, and be 0 from v = 17 on.
__device__ __forceinline__ float two_sided(float v)
{
    const float x = v * -kLog2e;
    const float t = __builtin_amdgcn_exp2f(-__builtin_fabsf(x));
    return __builtin_copysignf(t * __builtin_amdgcn_rcpf(1.0f + t), x);
}
// sigma(v): q, or 1 + q where q is negative -- the smaller one of the two as unsigned
// words
__device__ __forceinline__ float gate_of(float q)
{
    const unsigned shut = __builtin_bit_cast(unsigned, q);
    const unsigned open = __builtin_bit_cast(unsigned, 1.0f + q);
    return __builtin_bit_cast(float, min(shut, open));
}
// sigma(v) (1 - sigma(v)), from the smaller one: at most half of it is taken off
__device__ __forceinline__ float gate_slope(float q)
{
    return fmaf(-q, q, __builtin_fabsf(q));
}

// Whether decay<true> serves this lane's channels and all others of its wave
// (every wave of a workgroup has the same channels).
template <int V> __device__ __forceinline__ bool all_small(const float (&rate)[V])
{
    bool small = true;
#pragma unroll
    for (int v = 0; v < V; ++v)
        small = small && rate[v] <= kSmall;
    return __all(small);
}

// sqrt(1 - a^2) = sqrt(2 m - m^2)
__device__ __forceinline__ float input_factor(float m)
{
    return __builtin_amdgcn_sqrtf(fmaf(-m, m, m + m));
}

// A run of a sequence: its q-th, tokens [t0, t1) of the batch's rows.  `item` is
// its number among all runs (ScanPlan); `any` is false for a number that no run
// has.  A sequence of no token has one run, of none.
struct Run {
    int s, q, count, t0, t1, item;
    long long state_row;
    bool any, first, last;
};

// The idx-th run in the order in which they are handed out: dense batches go
// through all sequences' first runs, then their second, so that a run's
// predecessors are long under way; packed ones sequence by sequence.  REV: each
// sequence from its end on.
template <bool REV>
__device__ __forceinline__ Run run_of(const Batch &b, int items, int idx)
{
    constexpr int run = kRun;
    Run g;
    int start, len;
    if (!b.off) {
        g.count = max((b.tokens + run - 1) / run, 1);
        const int round = idx / b.seqs;
        g.s = idx - round * b.seqs;
        g.q = REV ? g.count - 1 - round : round;
        g.item = g.s * g.count + g.q;
        start = g.s * b.tokens;
        len = b.tokens;
    } else {
        g.item = REV ? items - 1 - idx : idx;
        // the last sequence whose first run's number is at most `item`, 64
        // candidates at a time
        int lo = 0, width = b.seqs;
        while (width > 1) {
            const int stride = (width + 63) / 64;
            const int at = lo + (int)(threadIdx.x & 63) * stride;
            const bool before =
                at < lo + width && seq_start(b, min(at, b.seqs - 1)) / run + at <= g.item;
            const int found = max(__popcll(__ballot(before)) - 1, 0);
            width = min(stride, lo + width - (lo + found * stride));
            lo += found * stride;
        }
        g.s = __builtin_amdgcn_readfirstlane(lo);
        start = seq_start(b, g.s);
        len = max(seq_start(b, g.s + 1) - start, 0);
        g.count = max((int)(((long long)len + run - 1) / run), 1);
        g.q = g.item - (start / run + g.s);
    }
    g.any = g.q >= 0 && g.q < g.count;
    g.first = g.q == 0;
    g.last = g.q == g.count - 1;
    g.t0 = start + (g.any ? g.q * run : 0);
    g.t1 = g.t0 + (g.any ? min(run, len - g.q * run) : 0);
    g.state_row = (long long)(start / kKept) + g.s + (g.t0 - start) / kKept;
    return g;
}

// Thread layout of a workgroup: kSlab / V lanes cover the channels of a token,
// kRun / KT groups of lanes cover a run, each KT consecutive tokens.
template <int V> struct Layout {
    static constexpr int KT = kKept;
    static constexpr int lanes = kSlab / V;
    static constexpr int groups = kRun / KT;
    static constexpr int threads = lanes * groups;
    static constexpr int waves = threads / 64;
    static constexpr int per_wave = 64 / lanes;    // groups of one wave
};

// One array's rows of a run, for this lane's channels: a buffer descriptor that
// starts with the run and ends with the segment (reads past it give zero,
// writes are dropped), the lane's place in it, and the rows as scalar offsets.
// With 64-bit addresses the compiler keeps one for every row of every array,
// which takes more registers than the data.  Row strides are below 2^23 bytes.
template <typename T, int V> struct Rows {
    static constexpr int KT = kKept;
    char *base;         // the batch's first row
    long long ld;       // bytes
    int lane;           // of this lane's first row of a run, and channel
    int width;          // bytes of a row

    __device__ __forceinline__ Rows(const void *p, long long ld_elems, int C, int c0, int group)
        : base(const_cast<char *>(static_cast<const char *>(p))),
          ld(ld_elems * (int)sizeof(T)), lane(group * KT * (int)ld + c0 * (int)sizeof(T)),
          width(C * (int)sizeof(T))
    {
    }
    __device__ __forceinline__ __amdgpu_buffer_rsrc_t run(int row, int rows) const
    {
        return dwconv::make_rsrc(base + row * ld, (min(rows, kRun) - 1) * (int)ld + width);
    }
    __device__ __forceinline__ void fetch(Raw<T, V> (&v)[KT], int row, int rows) const
    {
        const __amdgpu_buffer_rsrc_t rsrc = run(row, rows);
#pragma unroll
        for (int k = 0; k < KT; ++k)
            v[k].load(rsrc, lane, k * (int)ld);
    }
};

// Exclusive scan of (A, B) over the groups of a wave in token order (REV: from
// the last group on), then over the waves through LDS.  On return (A, B) is the
// step from the run's beginning (REV: end) to this thread's first token, and
// `total` holds the whole run's per slot.
template <int V, bool REV>
__device__ __forceinline__ void scan_groups(float (&A)[V], float (&B)[V], float (*lds)[2][kSlab],
                                            float (*total)[kSlab])
{
    using L = Layout<V>;
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int col = (lane % L::lanes) * V;
    const int grp = lane / L::lanes;
    const int rank = REV ? L::per_wave - 1 - grp : grp;
    // inclusive over the wave
#pragma unroll
    for (int d = 1; d < L::per_wave; d <<= 1) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const int from = REV ? lane + d * L::lanes : lane - d * L::lanes;
            const float pa = __shfl(A[v], from & 63), pb = __shfl(B[v], from & 63);
            if (rank >= d) {
                B[v] = fmaf(A[v], pb, B[v]);
                A[v] *= pa;
            }
        }
    }
    if (rank == L::per_wave - 1) {
#pragma unroll
        for (int v = 0; v < V; ++v) {
            lds[wave][0][col + v] = A[v];
            lds[wave][1][col + v] = B[v];
        }
    }
    // exclusive over the wave
#pragma unroll
    for (int v = 0; v < V; ++v) {
        if constexpr (L::per_wave > 1) {
            const int from = REV ? lane + L::lanes : lane - L::lanes;
            const float pa = __shfl(A[v], from & 63), pb = __shfl(B[v], from & 63);
            A[v] = rank ? pa : 1.0f;
            B[v] = rank ? pb : 0.0f;
        } else {
            A[v] = 1.0f;
            B[v] = 0.0f;
        }
    }
    __syncthreads();
    // the waves before this one, in order; the first wave adds up all of them,
    // a slot a lane
    if (wave == 0) {
        float ta = 1.0f, tb = 0.0f;
#pragma unroll
        for (int k = 0; k < L::waves; ++k) {
            const int from = REV ? L::waves - 1 - k : k;
            tb = fmaf(lds[from][0][lane], tb, lds[from][1][lane]);
            ta *= lds[from][0][lane];
        }
        total[0][lane] = ta;
        total[1][lane] = tb;
    }
    float PA[V], PB[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        PA[v] = 1.0f;
        PB[v] = 0.0f;
    }
#pragma unroll
    for (int k = 0; k < L::waves - 1; ++k) {
        const int from = REV ? L::waves - 1 - k : k;
        if (REV ? from > wave : from < wave)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                const float wa = lds[from][0][col + v];
                PB[v] = fmaf(wa, PB[v], lds[from][1][col + v]);
                PA[v] *= wa;
            }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        B[v] = fmaf(A[v], PB[v], B[v]);
        A[v] *= PA[v];
    }
}

// What the runs tell each other, per run and channel of a slab, in 64-bit words
// that are written and read whole: the run's (a, b), and the state after it.  A word is
// not there yet while all its bits are set, which neither has: a is not negative
// (a NaN is given without a sign), and beside a state is 0.
struct Told {
    unsigned long long ab[kSlab], state[kSlab];
};
constexpr unsigned long long kUntold = ~0ull;

__global__ __launch_bounds__(256) void k_scan_clear(unsigned long long *words, long long count,
                                                    unsigned *counter)
{
    const long long id = (long long)block_id() * 256 + threadIdx.x;
    if (id < count)
        words[id] = kUntold;
    if (id == 0)
        *counter = 0;
}

// What the other XCDs see of a word needs no more order than the word itself.
__device__ __forceinline__ void tell(unsigned long long *word, float first, float second)
{
    const unsigned lo = __builtin_bit_cast(unsigned, first);
    const unsigned long long v =
        (unsigned long long)__builtin_bit_cast(unsigned, second) << 32 | lo;
    __hip_atomic_store(word, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

__device__ __forceinline__ unsigned long long hear(unsigned long long *word)
{
    return __hip_atomic_load(word, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// The state before a run, by one wave with a channel a lane.  `before`: how many
// runs of the sequence come before it (REV: after); `mine`: this run's words.
// Runs looked at in one go.  2, 4, 8 and 16 take 241, 184, 178 and 225 us in
// the forward at 1 x 65537 x 1280, where the chain is longest, and 72, 74, 77 and
// 96 at 8 x 2048 x 2048, where registers count.
constexpr int kLookBack = 4;

template <bool REV>
__device__ __forceinline__ float state_before(Told *mine, int slabs, int before)
{
    const int lane = threadIdx.x & 63;
    const int reach = min(before, kLookBack);
    for (;;) {
        unsigned long long ab[kLookBack], state[kLookBack];
#pragma unroll
        for (int j = 0; j < kLookBack; ++j) {
            // nearest first; past the reach, the furthest again
            Told *t = mine + (long long)(REV ? 1 : -1) * min(j + 1, reach) * slabs;
            ab[j] = hear(&t->ab[lane]);
            state[j] = hear(&t->state[lane]);
        }
        int found = -1;
        bool linked = true;     // every run nearer than j has told its (a, b)
#pragma unroll
        for (int j = 0; j < kLookBack; ++j) {
            if (found < 0 && j < reach && linked && __all(state[j] != kUntold))
                found = j;
            linked = linked && __all(ab[j] != kUntold);
        }
        if (found >= 0) {
            float h = 0.0f;
#pragma unroll
            for (int j = kLookBack - 1; j >= 0; --j) {
                const float a = __builtin_bit_cast(float, (unsigned)(ab[j] >> 32));
                const float b = __builtin_bit_cast(float, (unsigned)ab[j]);
                if (j == found)
                    h = __builtin_bit_cast(float, (unsigned)state[j]);
                else if (j < found)
                    h = fmaf(a, h, b);
            }
            return h;
        }
        __builtin_amdgcn_s_sleep(2);
    }
}

// How the runs are linked.  Every workgroup that takes a run tells its words, even
// where nobody should ask for them: the offsets of a packed batch are device
// data, and whatever they hold, a wait for a run with a smaller ticket ends.
struct Chain {
    Told *told;         // nullptr: every sequence has one run
    unsigned *counter;
    int slabs, items;
    unsigned runs;              // slabs * items
};

__device__ __forceinline__ void tell_nothing(const Chain &ch, const Run &g, int slab)
{
    if (ch.told && threadIdx.x < 64) {
        Told *mine = ch.told + (long long)g.item * ch.slabs + slab;
        tell(&mine->ab[threadIdx.x], 0.0f, 1.0f);
        tell(&mine->state[threadIdx.x], 0.0f, 0.0f);
    }
}

// Leaves in `carry` the state before the run, whose (a, b) the first wave has left
// in `total`; the first run (REV: the last) starts from h0, or zero where that is nullptr.  By
// the first wave, a slot of V channels' lanes each: slots are numbered as the
// scan's lanes are, so the last ones of a row may stand for channels again.
template <int V, bool REV>
__device__ __forceinline__ void link(const Chain &ch, const Run &g, int slab, int C,
                                     const float *h0, const float (*total)[kSlab], float *carry)
{
    const int slot = threadIdx.x;
    if (slot < 64) {
        const int before = REV ? g.count - 1 - g.q : g.q;
        Told *mine = ch.told + (long long)g.item * ch.slabs + slab;
        const float a = total[0][slot], b = total[1][slot];
        float h = 0.0f;
        if (ch.told)
            tell(&mine->ab[slot], b, __builtin_fabsf(a));
        if (before > 0) {
            h = state_before<REV>(mine, ch.slabs, before);
        } else if (h0) {
            const int c = min(slab * kSlab + slot / V * V, C - V) + slot % V;
            h = h0[(long long)g.s * C + c];
        }
        if (ch.told)
            tell(&mine->state[slot], fmaf(a, h, b), 0.0f);
        carry[slot] = h;
    }
    __syncthreads();
}

// The run that this workgroup takes; ch.runs or more: none is left for it.
__device__ __forceinline__ unsigned take(const Chain &ch)
{
    __shared__ unsigned ticket;
    if (!ch.told)
        return block_id();
    if (threadIdx.x == 0)
        ticket = __hip_atomic_fetch_add(ch.counter, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    __syncthreads();
    return __builtin_amdgcn_readfirstlane(ticket);
}

// ---------------------------------------------------------------------------
// Forward.  Registers for 3 workgroups a CU: with 4 the loads of a run
// no longer fit at once (8 x 2048 x 2048: 77 against 74 us).
// ---------------------------------------------------------------------------
template <typename T, int V>
__global__ __launch_bounds__(Layout<V>::threads, 3) void k_scan_fwd(ScanArgs a, Chain ch)
{
    using L = Layout<V>;
    constexpr int KT = L::KT;
    __shared__ float lds[L::waves][2][kSlab];
    __shared__ float total[2][kSlab], carry[kSlab];
    const unsigned ticket = take(ch);
    if (ticket >= ch.runs)
        return;
    const int idx = (int)ticket, slab = idx % ch.slabs;
    const Run g = run_of<false>(a.batch, ch.items, idx / ch.slabs);
    // Channels: a row that V does not divide ends with a vector moved back to its
    // end, and lanes past the row repeat it; equal values are written twice.
    const int lane = threadIdx.x % L::lanes, group = threadIdx.x / L::lanes;
    const int C = a.C, c0 = min(slab * kSlab + lane * V, C - V);
    if (g.t0 == g.t1) {         // no run, or a sequence of no token
        tell_nothing(ch, g, slab);
        if (g.any && a.hT && group == 0) {
            float h[V] = {};
            if (a.h0)
                load<float, V>(a.h0 + (long long)g.s * C + c0, h);
            store<float, V>(a.hT + (long long)g.s * C + c0, h);
        }
        return;
    }
    const Rows<T, V> x(a.x, a.ldx, C, c0, group), r(a.r, a.ldr, C, c0, group),
        in(a.i, a.ldi, C, c0, group), y(a.y, a.ldy, C, c0, group);
    const int rows = g.t1 - g.t0, mt = g.t0 + group * KT;
    Raw<T, V> px[KT], pr[KT], pi[KT];
    r.fetch(pr, g.t0, rows);
    in.fetch(pi, g.t0, rows);
    x.fetch(px, g.t0, rows);
    float rate[V];
    load<float, V>(a.lam + c0, rate);
#pragma unroll
    for (int v = 0; v < V; ++v)
        rate[v] = decay_rate(rate[v], a.scale);
    float av[KT][V], bv[KT][V], A[V], B[V];
    // Past the sequence's last token (in its last run alone) the reads are zero,
    // the stores dropped, and the run's (a, b) is not used.
    auto gates = [&](auto small) {
#pragma unroll
        for (int k = 0; k < KT; ++k)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float m;
                decay<decltype(small)::value>(rate[v] * logistic(pr[k].get(v)), av[k][v], m);
                bv[k][v] = input_factor(m) * logistic(pi[k].get(v)) * px[k].get(v);
            }
    };
    if (all_small(rate))
        gates(std::true_type());
    else
        gates(std::false_type());
#pragma unroll
    for (int v = 0; v < V; ++v) {
        A[v] = av[0][v];
        B[v] = bv[0][v];
#pragma unroll
        for (int k = 1; k < KT; ++k) {
            B[v] = fmaf(av[k][v], B[v], bv[k][v]);
            A[v] *= av[k][v];
        }
    }
    scan_groups<V, false>(A, B, lds, total);
    link<V, false>(ch, g, slab, C, a.h0, total, carry);
    float hk[V];
#pragma unroll
    for (int v = 0; v < V; ++v)
        hk[v] = fmaf(A[v], carry[lane * V + v], B[v]);
    if (a.states && mt < g.t1)
        store<float, V>(a.states + (g.state_row + group) * C + c0, hk);
    const __amdgpu_buffer_rsrc_t out = y.run(g.t0, rows);
#pragma unroll
    for (int k = 0; k < KT; ++k) {
#pragma unroll
        for (int v = 0; v < V; ++v)
            hk[v] = fmaf(av[k][v], hk[v], bv[k][v]);
        Raw<T, V>(hk).store(out, y.lane, k * (int)y.ld);
        if (mt + k == g.t1 - 1 && g.last && a.hT)
            store<float, V>(a.hT + (long long)g.s * C + c0, hk);
    }
}

// ---------------------------------------------------------------------------
// Gradients, from the last run to the first.  With p[t] = a[t] g[t] the reversed
// recurrence is p[t] = a[t] p[t+1] + a[t] dy[t], whose steps compose as the
// forward's do.  The state before each thread's tokens has been kept, so each
// input is read once: 7 arrays moved (dy, x, r, i; dx, dr, di) and an eighth of
// one in float32, the states.  66 instructions of the vector unit an element: 121 us
// at 8 x 2048 x 2048 bfloat16, 6 of which are what the gates' complements cost.
// ---------------------------------------------------------------------------
template <typename T, int V>
__global__ __launch_bounds__(Layout<V>::threads, V == 1 ? 4 : 2) void k_scan_grad(ScanArgs a,
                                                                                  Chain ch)
{
    using L = Layout<V>;
    constexpr int KT = L::KT;
    __shared__ float lds[L::waves][2][kSlab];
    __shared__ float total[2][kSlab], carry[kSlab];
    __shared__ float sums[L::groups][kSlab];
    const unsigned ticket = take(ch);
    if (ticket >= ch.runs)
        return;
    const int idx = (int)ticket, slab = idx % ch.slabs;
    const Run g = run_of<true>(a.batch, ch.items, idx / ch.slabs);
    const int lane = threadIdx.x % L::lanes, group = threadIdx.x / L::lanes;
    const int C = a.C, c0 = min(slab * kSlab + lane * V, C - V);
    float drate[V] = {};
    if (g.t0 == g.t1) {         // no token: nothing for dlam, dh0 = dhT
        tell_nothing(ch, g, slab);
        if (group == 0) {
            store<float, V>(a.part + (long long)g.item * C + c0, drate);
            if (g.any && a.dh0) {
                float p[V] = {};
                if (a.dhT)
                    load<float, V>(a.dhT + (long long)g.s * C + c0, p);
                store<float, V>(a.dh0 + (long long)g.s * C + c0, p);
            }
        }
        return;
    }
    const Rows<T, V> x(a.x, a.ldx, C, c0, group), r(a.r, a.ldr, C, c0, group),
        in(a.i, a.ldi, C, c0, group), dy(a.dy, a.lddy, C, c0, group),
        dx(a.dx, a.lddx, C, c0, group), dr(a.dr, a.lddr, C, c0, group),
        di(a.di, a.lddi, C, c0, group);
    const int rows = g.t1 - g.t0, mt = g.t0 + group * KT;
    Raw<T, V> px[KT], pr[KT], pi[KT], pd[KT];
    r.fetch(pr, g.t0, rows);
    dy.fetch(pd, g.t0, rows);
    in.fetch(pi, g.t0, rows);
    x.fetch(px, g.t0, rows);
    float rate[V], hk[V] = {};
    if (mt < g.t1)
        load<float, V>(a.states_in + (g.state_row + group) * C + c0, hk);
    load<float, V>(a.lam + c0, rate);
#pragma unroll
    for (int v = 0; v < V; ++v)
        rate[v] = decay_rate(rate[v], a.scale);
    float av[KT][V], gi[KT][V], bt[KT][V], gr[KT][V];
    auto gates = [&](auto small) {
#pragma unroll
        for (int k = 0; k < KT; ++k)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float m;
                gr[k][v] = two_sided(pr[k].get(v));
                decay<decltype(small)::value>(rate[v] * gate_of(gr[k][v]), av[k][v], m);
                bt[k][v] = input_factor(m);
                gi[k][v] = two_sided(pi[k].get(v));
            }
    };
    if (all_small(rate))
        gates(std::true_type());
    else
        gates(std::false_type());
    // tokens past the end change nothing (x and dy are zero there)
    if (rows < kRun)
#pragma unroll
        for (int k = 0; k < KT; ++k)
            if (mt + k >= g.t1)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    av[k][v] = 1.0f;
                    gr[k][v] = 0.0f;
                }
    float A[V], B[V], gt[KT][V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        A[v] = av[KT - 1][v];
        B[v] = A[v] * pd[KT - 1].get(v);
#pragma unroll
        for (int k = KT - 2; k >= 0; --k) {
            B[v] = av[k][v] * (B[v] + pd[k].get(v));
            A[v] *= av[k][v];
        }
    }
    scan_groups<V, true>(A, B, lds, total);
    link<V, true>(ch, g, slab, C, a.dhT, total, carry);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        float p = fmaf(A[v], carry[lane * V + v], B[v]);
#pragma unroll
        for (int k = KT - 1; k >= 0; --k) {
            gt[k][v] = p + pd[k].get(v);
            p = av[k][v] * gt[k][v];
        }
        A[v] = p;
    }
    if (g.first && a.dh0 && group == 0)
        store<float, V>(a.dh0 + (long long)g.s * C + c0, A);
    const __amdgpu_buffer_rsrc_t to_x = dx.run(g.t0, rows), to_r = dr.run(g.t0, rows),
                                 to_i = di.run(g.t0, rows);
#pragma unroll
    for (int k = 0; k < KT; ++k) {
        float ox[V], orr[V], oi[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float at = av[k][v], beta = bt[k][v], xv = px[k].get(v);
            const float si = gate_of(gi[k][v]), decayed = at * hk[v];
            const float in = gt[k][v] * beta, pull = gt[k][v] * xv * si;
            ox[v] = in * si;
            oi[v] = in * xv * gate_slope(gi[k][v]);
            // sigma(i) x a^2 / beta, nothing where beta is 0
            const float back =
                beta > 0.0f ? pull * at * at * __builtin_amdgcn_rcpf(beta) : 0.0f;
            const float dgate = back - gt[k][v] * decayed;
            drate[v] = fmaf(dgate, gate_of(gr[k][v]), drate[v]);
            orr[v] = dgate * rate[v] * gate_slope(gr[k][v]);
            hk[v] = fmaf(beta * si, xv, decayed);
        }
        Raw<T, V>(ox).store(to_x, dx.lane, k * (int)dx.ld);
        Raw<T, V>(orr).store(to_r, dr.lane, k * (int)dr.ld);
        Raw<T, V>(oi).store(to_i, di.lane, k * (int)di.ld);
    }
    // the run's share of dlam, the groups' sums added in order
#pragma unroll
    for (int v = 0; v < V; ++v)
        sums[group][lane * V + v] = drate[v];
    __syncthreads();
    if (group == 0) {
        for (int k = 1; k < L::groups; ++k)
#pragma unroll
            for (int v = 0; v < V; ++v)
                drate[v] += sums[k][lane * V + v];
        store<float, V>(a.part + (long long)g.item * C + c0, drate);
    }
}

// dlam = scale * sigma(lam) * (sum of the runs' shares)
__global__ __launch_bounds__(1024) void k_scan_grad_sum(const float *part, int runs, int C,
                                                        const float *lam, float scale,
                                                        float *dlam)
{
    column_sums(part, runs, C, [=](long long c, float s) {
        const float e = exp_neg(lam[c]), p = 1.0f / (1.0f + e);
        dlam[c] = s * scale * (lam[c] < 0.0f ? e * p : p);
    });
}

// One token per sequence, h in place: a thread per V channels, those that V
// does not divide one by one.
template <typename T, int V>
__device__ __forceinline__ void step_vector(const ScanArgs &a, int s, int c0)
{
    float x[V], r[V], in[V], rate[V], h[V];
    load<T, V>(static_cast<const T *>(a.x) + s * a.ldx + c0, x);
    load<T, V>(static_cast<const T *>(a.r) + s * a.ldr + c0, r);
    load<T, V>(static_cast<const T *>(a.i) + s * a.ldi + c0, in);
    load<float, V>(a.lam + c0, rate);
    float *hp = a.h + (long long)s * a.C + c0;
    load<float, V>(hp, h);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        float at, m;
        decay<false>(decay_rate(rate[v], a.scale) * logistic(r[v]), at, m);
        h[v] = fmaf(at, h[v], input_factor(m) * logistic(in[v]) * x[v]);
    }
    store<float, V>(hp, h);
    store<T, V>(static_cast<T *>(a.y) + s * a.ldy + c0, h);
}

template <typename T, int V>
__global__ __launch_bounds__(256) void k_scan_step(ScanArgs a, int groups)
{
    const long long id = (long long)block_id() * 256 + threadIdx.x;
    if (id >= (long long)a.batch.seqs * groups)
        return;
    const int s = (int)(id / groups), c0 = (int)(id % groups) * V;
    if (c0 + V <= a.C)
        step_vector<T, V>(a, s, c0);
    else
        for (int c = c0; c < a.C; ++c)
            step_vector<T, 1>(a, s, c);
}

// f(element pointer type, channels per thread): 4, or 1 where a row has fewer
template <typename F> int with_variant(const ScanArgs &a, F f)
{
    return with_type(a.type, [&](auto *t) {
        if (a.C >= 4)
            return f(t, std::integral_constant<int, 4>());
        return f(t, std::integral_constant<int, 1>());
    });
}

}  // namespace

// The runs: the q-th of sequence s has the number
// floor(start of s / kRun) + s + q (dense batches: s * runs + q), which no other
// has; `chained` where a sequence may have several.
struct ScanPlan {
    long long items, slabs, words;      // words: bytes of Told
    bool chained;
};

static ScanPlan scan_plan(const Batch &b, int C, bool packed)
{
    ScanPlan p;
    const long long runs = cdiv(b.tokens, kRun);
    p.items = packed ? (long long)b.rows / kRun + b.seqs : b.seqs * (runs > 1 ? runs : 1);
    p.slabs = cdiv(C, kSlab);
    p.chained = (packed ? b.rows : b.tokens) > kRun;
    p.words = p.chained ? p.items * p.slabs * (long long)sizeof(Told) : 0;
    return p;
}

long long scan_states(const Batch &b, int C)
{
    return ((long long)b.rows / kKept + b.seqs) * C;
}

// The words that the runs exchange, their counter (16 bytes), and for the
// gradient the runs' shares of dlam.
long long scan_workspace(bool grad, const Batch &b, int C, bool packed)
{
    const ScanPlan p = scan_plan(b, C, packed);
    return (p.chained ? p.words + 16 : 0) + (grad ? 4 * p.items * C : 0);
}

// Clears what the runs will exchange.
static int make_chain(const ScanPlan &p, void *space, hipStream_t st, Chain *ch)
{
    ch->slabs = (int)p.slabs;
    ch->items = (int)p.items;
    ch->told = nullptr;
    ch->counter = nullptr;
    if (p.items * p.slabs > 0x7fffffffLL)
        return DWCONV_ERR_BAD_DIM;
    ch->runs = (unsigned)(p.items * p.slabs);
    if (!p.chained)
        return DWCONV_OK;
    ch->counter = static_cast<unsigned *>(space);
    ch->told = reinterpret_cast<Told *>(static_cast<char *>(space) + 16);
    const long long words = p.words / 8;
    return dwconv::launch_kernel(k_scan_clear, grid_of(cdiv(words, 256)), dim3(256), 0, st,
                                 reinterpret_cast<unsigned long long *>(ch->told), words,
                                 ch->counter);
}

int launch_scan_fwd(const ScanArgs &a, void *stream)
{
    hipStream_t st = static_cast<hipStream_t>(stream);
    const ScanPlan p = scan_plan(a.batch, a.C, a.batch.off != nullptr);
    Chain ch;
    const int rc = make_chain(p, a.workspace, st, &ch);
    if (rc != DWCONV_OK)
        return rc;
    return with_variant(a, [&](auto *t, auto v) {
        using T = std::remove_pointer_t<decltype(t)>;
        constexpr int V = decltype(v)::value;
        return dwconv::launch_kernel(k_scan_fwd<T, V>, grid_of(p.items * p.slabs),
                                     dim3(Layout<V>::threads), 0, st, a, ch);
    });
}

int launch_scan_grad(const ScanArgs &args, void *stream)
{
    hipStream_t st = static_cast<hipStream_t>(stream);
    ScanArgs a = args;
    const ScanPlan p = scan_plan(a.batch, a.C, a.batch.off != nullptr);
    Chain ch;
    int rc = make_chain(p, a.workspace, st, &ch);
    if (rc != DWCONV_OK)
        return rc;
    a.part = reinterpret_cast<float *>(static_cast<char *>(a.workspace) +
                                       (p.chained ? p.words + 16 : 0));
    rc = with_variant(a, [&](auto *t, auto v) {
        using T = std::remove_pointer_t<decltype(t)>;
        constexpr int V = decltype(v)::value;
        return dwconv::launch_kernel(k_scan_grad<T, V>, grid_of(p.items * p.slabs),
                                     dim3(Layout<V>::threads), 0, st, a, ch);
    });
    if (rc == DWCONV_OK)
        rc = dwconv::launch_kernel(k_scan_grad_sum, dim3((unsigned)cdiv(a.C, 64)), dim3(1024), 0,
                                   st, (const float *)a.part, ch.items, a.C, a.lam, a.scale,
                                   a.dlam);
    return rc;
}

int launch_scan_step(const ScanArgs &a, void *stream)
{
    return with_variant(a, [&](auto *t, auto v) {
        using T = std::remove_pointer_t<decltype(t)>;
        constexpr int V = decltype(v)::value;
        const int groups = (int)cdiv(a.C, V);
        const long long blocks = cdiv((long long)a.batch.seqs * groups, 256);
        if (blocks > 0x7fffffffLL)
            return DWCONV_ERR_BAD_DIM;
        return dwconv::launch_kernel(k_scan_step<T, V>, grid_of(blocks), dim3(256), 0,
                                     static_cast<hipStream_t>(stream), a, groups);
    });
}

}  // namespace dwseq

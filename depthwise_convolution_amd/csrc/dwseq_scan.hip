// dwseq_scan.hip -- gated linear recurrence: forward, single-token step and
// gradients (include/dwconv_seq.h).
//
//   h[t] = a[t] h[t-1] + b[t],  a = e^L,  b = sqrt(1 - a^2) sigma(i) x,
//   L = -scale softplus(lam) sigma(r)
//
// Steps compose: applying (a1, b1) and then (a2, b2) is (a1 a2, a2 b1 + b2),
// which lets the tokens be scanned in parallel.  A workgroup owns 64 channels
// of one segment of a sequence and walks it in runs of 128 tokens: a thread
// holds V channels of a few consecutive tokens in registers and folds them to
// one (a, b); the folds are scanned over the lanes of a wave that hold the
// same channels, then over the waves in LDS, from the state that the run before
// left; then every thread walks its tokens from its own start and stores h.
// Each input is read once and h never leaves float32 registers on its way.
// Bound by HBM: 4 arrays (x, r, i, y) moved, some 40 operations an element.
//
// Where the sequences and channels give too few workgroups, sequences are cut
// into segments: a first pass folds each segment but the last of its sequence
// to one (a, b), which the second pass folds up to its own start, in order.
// No workgroup waits for another, and every order is fixed.
#include "dwseq_device.h"

namespace dwseq {
namespace {

constexpr int kRun = DWCONV_SCAN_RUN;
constexpr int kSlab = 64;       // channels of a workgroup
constexpr float kLog2e = 1.44269504088896341f;

// Decay constant of a channel: scale * softplus(lam)
__device__ __forceinline__ float decay_rate(float lam, float scale)
{
    return scale * softplus(lam);
}

// One token's gate: a = e^-u and, without the cancellation of 1 - a,
// m = 1 - a = u - u^2/2 + u^3/6 - ... for small u (remainder below 2^-24 m at
// u = 1/4).  a itself is then 1 - m, rounded once: over a long memory, an error
// of one sign in a would grow with 1 / (1 - a).
__device__ __forceinline__ void decay(float u, float &a, float &m)
{
    const float e = __builtin_amdgcn_exp2f(-u * kLog2e);
    float q = fmaf(u, -1.0f / 7.0f, 1.0f);
    q = fmaf(u * q, -1.0f / 6.0f, 1.0f);
    q = fmaf(u * q, -1.0f / 5.0f, 1.0f);
    q = fmaf(u * q, -1.0f / 4.0f, 1.0f);
    q = fmaf(u * q, -1.0f / 3.0f, 1.0f);
    q = fmaf(u * q, -1.0f / 2.0f, 1.0f);
    const bool small = u < 0.25f;
    m = small ? u * q : 1.0f - e;
    a = small ? 1.0f - m : e;
}

// sqrt(1 - a^2) = sqrt(m (2 - m))
__device__ __forceinline__ float input_factor(float m)
{
    return __builtin_amdgcn_sqrtf(m * (2.0f - m));
}

// A segment of a sequence: tokens [t0, t1) of the batch's rows; `index` is its
// number (ScanPlan), `q` its place in the sequence, `runs` the number of
// the state row of its first run.
struct Segment {
    int s, q, t0, t1, len, start, state_row;
    bool any, first, last;
};

__device__ __forceinline__ Segment segment_of(const Batch &b, int seg, int index)
{
    Segment g;
    // the last sequence whose first segment's number is at most `index`
    int lo = 0, hi = b.seqs - 1;
    while (lo < hi) {
        const int mid = lo + ((hi - lo + 1) >> 1);
        if (seq_start(b, mid) / seg + mid <= index)
            lo = mid;
        else
            hi = mid - 1;
    }
    g.s = lo;
    g.start = seq_start(b, lo);
    g.len = max(seq_start(b, lo + 1) - g.start, 0);
    g.q = index - (g.start / seg + lo);
    const long long from = (long long)g.q * seg;
    g.any = g.q == 0 || from < g.len;
    g.first = g.q == 0;
    g.last = from + seg >= g.len;
    g.t0 = g.start + (int)(from < g.len ? from : g.len);
    g.t1 = g.last ? g.start + g.len : g.t0 + seg;
    g.state_row = g.start / kRun + g.s + (int)(from / kRun);
    return g;
}

// Thread layout of a workgroup: kSlab / V lanes cover the channels of a token,
// kRun / KT groups of lanes cover a run, each KT consecutive tokens.
template <int V, int KT> struct Layout {
    static constexpr int lanes = kSlab / V;
    static constexpr int groups = kRun / KT;
    static constexpr int threads = lanes * groups;
    static constexpr int waves = threads / 64;
    static constexpr int per_wave = 64 / lanes;    // groups of one wave
};

// Exclusive scan of (A, B) over the groups of a wave in token order (reversed:
// from the last group on), then over the waves through LDS.  On return (A, B)
// is the step from the run's beginning to this thread's first token, and
// (TA, TB) the whole run's.
template <int V, int KT, bool REV>
__device__ __forceinline__ void scan_groups(float (&A)[V], float (&B)[V], float (&TA)[V],
                                            float (&TB)[V], float (*lds)[2][kSlab])
{
    using L = Layout<V, KT>;
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
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
    float PA[V], PB[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
        PA[v] = TA[v] = 1.0f;
        PB[v] = TB[v] = 0.0f;
    }
#pragma unroll
    for (int k = 0; k < L::waves; ++k) {
        const int from = REV ? L::waves - 1 - k : k;
        const bool before = REV ? from > wave : from < wave;
#pragma unroll
        for (int v = 0; v < V; ++v) {
            const float wa = lds[from][0][col + v], wb = lds[from][1][col + v];
            TB[v] = fmaf(wa, TB[v], wb);
            TA[v] *= wa;
            PA[v] = before ? TA[v] : PA[v];
            PB[v] = before ? TB[v] : PB[v];
        }
    }
#pragma unroll
    for (int v = 0; v < V; ++v) {
        B[v] = fmaf(A[v], PB[v], B[v]);
        A[v] *= PA[v];
    }
}

// The (a, b) of the segments before this one (REV: after it), folded in order
// onto h.
template <int V, bool REV>
__device__ __forceinline__ void fold_segments(const float *agg, int C, int c0, int index, int q,
                                              int count, float (&h)[V])
{
    for (int k = 0; k < (REV ? count - 1 - q : q); ++k) {
        const long long at = REV ? index - q + count - 1 - k : index - q + k;
        float A[V], B[V];
        load<float, V>(agg + at * 2 * C + c0, A);
        load<float, V>(agg + (at * 2 + 1) * C + c0, B);
#pragma unroll
        for (int v = 0; v < V; ++v)
            h[v] = fmaf(A[v], h[v], B[v]);
    }
}

// ---------------------------------------------------------------------------
// Forward.  FOLD: the first pass over cut sequences (no y; writes the
// segment's (a, b)).
// ---------------------------------------------------------------------------
template <typename T, int V, int KT, bool FOLD>
__global__ __launch_bounds__((Layout<V, KT>::threads)) void k_scan_fwd(ScanArgs a, int seg,
                                                                       int slabs)
{
    using L = Layout<V, KT>;
    __shared__ float lds[2][L::waves][2][kSlab];
    const int slab = blockIdx.x % slabs, index = blockIdx.x / slabs;
    const Segment g = segment_of(a.batch, seg, index);
    if (!g.any || (FOLD && g.last))
        return;
    const int lane = threadIdx.x % L::lanes, group = threadIdx.x / L::lanes;
    const int C = a.C, c0 = min(slab * kSlab + lane * V, C - V);
    const bool mine = slab * kSlab + lane * V < C;
    const T *x = static_cast<const T *>(a.x) + c0, *r = static_cast<const T *>(a.r) + c0,
            *in = static_cast<const T *>(a.i) + c0;
    T *y = static_cast<T *>(a.y) + c0;
    float rate[V], h[V], SA[V];
    load<float, V>(a.lam + c0, rate);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        rate[v] = decay_rate(rate[v], a.scale);
        h[v] = 0.0f;
        SA[v] = 1.0f;
    }
    if (!FOLD) {
        if (a.h0)
            load<float, V>(a.h0 + (long long)g.s * C + c0, h);
        fold_segments<V, false>(a.agg, C, c0, index, g.q, 0, h);
    }
    const bool lead = mine && group == 0;     // writes what there is one of per channel
    Pack<T, V> px[KT], pr[KT], pi[KT];
    auto fetch = [&](int t) {
#pragma unroll
        for (int k = 0; k < KT; ++k) {
            const long long row = min(t + k, g.t1 - 1);
            px[k] = *reinterpret_cast<const Pack<T, V> *>(x + row * a.ldx);
            pr[k] = *reinterpret_cast<const Pack<T, V> *>(r + row * a.ldr);
            pi[k] = *reinterpret_cast<const Pack<T, V> *>(in + row * a.ldi);
        }
    };
    if (g.t0 < g.t1)
        fetch(g.t0 + group * KT);
    int run = 0;
    for (int t = g.t0; t < g.t1; t += kRun, ++run) {
        const int mt = t + group * KT;
        float av[KT][V], bv[KT][V], A[V], B[V], TA[V], TB[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
            A[v] = 1.0f;
            B[v] = 0.0f;
        }
#pragma unroll
        for (int k = 0; k < KT; ++k)
#pragma unroll
            for (int v = 0; v < V; ++v) {
                float m;
                decay(rate[v] * logistic((float)pr[k].v[v]), av[k][v], m);
                bv[k][v] = input_factor(m) * logistic((float)pi[k].v[v]) * (float)px[k].v[v];
                if (mt + k >= g.t1) {
                    av[k][v] = 1.0f;
                    bv[k][v] = 0.0f;
                }
                B[v] = fmaf(av[k][v], B[v], bv[k][v]);
                A[v] *= av[k][v];
            }
        if (t + kRun < g.t1)
            fetch(mt + kRun);
        scan_groups<V, KT, false>(A, B, TA, TB, lds[run & 1]);
        if (!FOLD) {
            if (a.states && lead)
                store<float, V>(a.states + (long long)(g.state_row + run) * C + c0, h);
            float hk[V];
#pragma unroll
            for (int v = 0; v < V; ++v)
                hk[v] = fmaf(A[v], h[v], B[v]);
#pragma unroll
            for (int k = 0; k < KT; ++k) {
#pragma unroll
                for (int v = 0; v < V; ++v)
                    hk[v] = fmaf(av[k][v], hk[v], bv[k][v]);
                if (mine && mt + k < g.t1)
                    store<T, V>(y + (long long)(mt + k) * a.ldy, hk);
            }
        }
#pragma unroll
        for (int v = 0; v < V; ++v) {
            h[v] = fmaf(TA[v], h[v], TB[v]);
            SA[v] *= TA[v];
        }
    }
    if (!lead)
        return;
    if (FOLD) {
        store<float, V>(a.agg + (long long)index * 2 * C + c0, SA);
        store<float, V>(a.agg + ((long long)index * 2 + 1) * C + c0, h);
    } else if (g.last && a.hT) {
        store<float, V>(a.hT + (long long)g.s * C + c0, h);
    }
}

// ---------------------------------------------------------------------------
// Gradients, runs and segments from the last to the first.  With p[t] = a[t] g[t]
// the reversed recurrence is p[t] = a[t] p[t+1] + a[t] dy[t], whose steps compose
// as the forward's do.  A run's states are scanned again from the kept state
// before it, so each input is read once: 7 arrays moved (dy, x, r, i; dx, dr, di).
// ---------------------------------------------------------------------------
template <typename T, int V, int KT, bool FOLD>
__global__ __launch_bounds__((Layout<V, KT>::threads)) void k_scan_grad(ScanArgs a, int seg,
                                                                        int slabs)
{
    using L = Layout<V, KT>;
    __shared__ float lds[2][2][L::waves][2][kSlab];
    __shared__ float sums[L::groups][kSlab];
    const int slab = blockIdx.x % slabs, index = blockIdx.x / slabs;
    const Segment g = segment_of(a.batch, seg, index);
    const int lane = threadIdx.x % L::lanes, group = threadIdx.x / L::lanes;
    const int C = a.C, c0 = min(slab * kSlab + lane * V, C - V);
    const bool mine = slab * kSlab + lane * V < C;
    const bool lead = mine && group == 0;
    if (FOLD && (!g.any || g.first))
        return;
    const T *x = static_cast<const T *>(a.x) + c0, *r = static_cast<const T *>(a.r) + c0,
            *in = static_cast<const T *>(a.i) + c0, *dy = static_cast<const T *>(a.dy) + c0;
    T *dx = static_cast<T *>(a.dx) + c0, *dr = static_cast<T *>(a.dr) + c0,
      *di = static_cast<T *>(a.di) + c0;
    float rate[V], p[V], SA[V], drate[V];
    load<float, V>(a.lam + c0, rate);
#pragma unroll
    for (int v = 0; v < V; ++v) {
        rate[v] = decay_rate(rate[v], a.scale);
        p[v] = drate[v] = 0.0f;
        SA[v] = 1.0f;
    }
    if (g.any) {
        if (!FOLD) {
            if (a.dhT)
                load<float, V>(a.dhT + (long long)g.s * C + c0, p);
            const int count = max((int)(((long long)g.len + seg - 1) / seg), 1);
            fold_segments<V, true>(a.agg, C, c0, index, g.q, count, p);
        }
        const int runs = (g.t1 - g.t0 + kRun - 1) / kRun;
        for (int run = runs - 1; run >= 0; --run) {
            const int mt = g.t0 + run * kRun + group * KT;
            float av[KT][V], bv[KT][V], dv[KT][V], si[KT][V], bt[KT][V], sr[KT][V];
            float A[V], B[V], TA[V], TB[V], FA[V], FB[V];
            Pack<T, V> px[KT], pr[KT], pi[KT], pd[KT];
#pragma unroll
            for (int k = 0; k < KT; ++k) {
                const long long row = min(mt + k, g.t1 - 1);
                pr[k] = *reinterpret_cast<const Pack<T, V> *>(r + row * a.ldr);
                pd[k] = *reinterpret_cast<const Pack<T, V> *>(dy + row * a.lddy);
                if (!FOLD) {
                    px[k] = *reinterpret_cast<const Pack<T, V> *>(x + row * a.ldx);
                    pi[k] = *reinterpret_cast<const Pack<T, V> *>(in + row * a.ldi);
                }
            }
            float hk[V];
            if (!FOLD)
                load<float, V>(a.states_in + (long long)(g.state_row + run) * C + c0, hk);
#pragma unroll
            for (int v = 0; v < V; ++v) {
                FA[v] = 1.0f;
                FB[v] = 0.0f;
            }
#pragma unroll
            for (int k = 0; k < KT; ++k)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    float m;
                    sr[k][v] = logistic((float)pr[k].v[v]);
                    decay(rate[v] * sr[k][v], av[k][v], m);
                    dv[k][v] = (float)pd[k].v[v];
                    const bool out = mt + k >= g.t1;
                    if (!FOLD) {
                        bt[k][v] = input_factor(m);
                        si[k][v] = logistic((float)pi[k].v[v]);
                        bv[k][v] = bt[k][v] * si[k][v] * (float)px[k].v[v];
                    }
                    if (out) {
                        av[k][v] = 1.0f;
                        dv[k][v] = 0.0f;
                        bv[k][v] = 0.0f;
                    }
                    if (!FOLD) {
                        FB[v] = fmaf(av[k][v], FB[v], bv[k][v]);
                        FA[v] *= av[k][v];
                    }
                }
#pragma unroll
            for (int v = 0; v < V; ++v) {
                A[v] = 1.0f;
                B[v] = 0.0f;
            }
#pragma unroll
            for (int k = KT - 1; k >= 0; --k)
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    B[v] = av[k][v] * (B[v] + dv[k][v]);
                    A[v] *= av[k][v];
                }
            scan_groups<V, KT, true>(A, B, TA, TB, lds[run & 1][0]);
            if (!FOLD) {
                float UA[V], UB[V];
                scan_groups<V, KT, false>(FA, FB, UA, UB, lds[run & 1][1]);
                float before[KT][V], pk[V];
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    hk[v] = fmaf(FA[v], hk[v], FB[v]);
                    pk[v] = fmaf(A[v], p[v], B[v]);
                }
#pragma unroll
                for (int k = 0; k < KT; ++k)
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        before[k][v] = hk[v];
                        hk[v] = fmaf(av[k][v], hk[v], bv[k][v]);
                    }
#pragma unroll
                for (int k = KT - 1; k >= 0; --k) {
                    float ox[V], orr[V], oi[V];
                    const bool in_range = mt + k < g.t1;
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        const float gt = pk[v] + dv[k][v], at = av[k][v];
                        const float xv = (float)px[k].v[v];
                        const float gated = gt * si[k][v];
                        ox[v] = gated * bt[k][v];
                        oi[v] = ox[v] * xv * (1.0f - si[k][v]);
                        // sigma(i) x a^2 / beta, nothing where beta is 0
                        const float back = bt[k][v] > 0.0f
                                               ? gated * xv * at * at *
                                                     __builtin_amdgcn_rcpf(bt[k][v])
                                               : 0.0f;
                        const float dlog = gt * at * before[k][v] - back;
                        const float dgate = in_range ? -dlog * sr[k][v] : 0.0f;
                        drate[v] += dgate;
                        orr[v] = dgate * rate[v] * (1.0f - sr[k][v]);
                        pk[v] = at * gt;
                    }
                    if (mine && in_range) {
                        store<T, V>(dx + (long long)(mt + k) * a.lddx, ox);
                        store<T, V>(dr + (long long)(mt + k) * a.lddr, orr);
                        store<T, V>(di + (long long)(mt + k) * a.lddi, oi);
                    }
                }
            }
#pragma unroll
            for (int v = 0; v < V; ++v) {
                p[v] = fmaf(TA[v], p[v], TB[v]);
                SA[v] *= TA[v];
            }
        }
    }
    if (FOLD) {
        if (lead) {
            store<float, V>(a.agg + (long long)index * 2 * C + c0, SA);
            store<float, V>(a.agg + ((long long)index * 2 + 1) * C + c0, p);
        }
        return;
    }
    if (g.any && g.first && a.dh0 && lead)
        store<float, V>(a.dh0 + (long long)g.s * C + c0, p);
    // the segment's share of dlam, the groups' sums added in order
#pragma unroll
    for (int v = 0; v < V; ++v)
        sums[group][lane * V + v] = drate[v];
    __syncthreads();
    if (lead) {
        for (int k = 1; k < L::groups; ++k)
#pragma unroll
            for (int v = 0; v < V; ++v)
                drate[v] += sums[k][lane * V + v];
        store<float, V>(a.part + (long long)index * C + c0, drate);
    }
}

// dlam = scale * sigma(lam) * (sum of the segments' shares)
__global__ __launch_bounds__(1024) void k_scan_grad_sum(const float *part, int segs, int C,
                                                        const float *lam, float scale,
                                                        float *dlam)
{
    column_sums(part, segs, C, [=](long long c, float s) {
        dlam[c] = s * scale * logistic(lam[c]);
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
        decay(decay_rate(rate[v], a.scale) * logistic(r[v]), at, m);
        h[v] = fmaf(at, h[v], input_factor(m) * logistic(in[v]) * x[v]);
    }
    store<float, V>(hp, h);
    store<T, V>(static_cast<T *>(a.y) + s * a.ldy + c0, h);
}

template <typename T, int V>
__global__ __launch_bounds__(256) void k_scan_step(ScanArgs a, int groups)
{
    const long long id = (long long)blockIdx.x * 256 + threadIdx.x;
    const int s = (int)(id / groups), c0 = (int)(id % groups) * V;
    if (s >= a.batch.seqs)
        return;
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

// Workgroups are (slab of 64 channels) x (segment).  Uncut sequences are best
// where they give the chip enough of them: a cut sequence's inputs are read
// twice.
ScanPlan scan_plan(const Batch &b, int C, bool packed)
{
    const long long slabs = cdiv(C, kSlab), want = 512;
    ScanPlan p;
    // the segment length that gives `want` workgroups
    long long seg = cdiv(cdiv((long long)b.rows * slabs, want), kRun) * kRun;
    if (seg < 2 * kRun)
        seg = 2 * kRun;
    const long long longest = packed ? b.rows : b.tokens;
    if (seg >= longest)
        seg = cdiv(longest > 0 ? longest : 1, kRun) * kRun;
    p.seg = (int)(seg < 0x40000000 ? seg : 0x40000000);
    p.cut = p.seg < longest;
    p.segs = b.rows / p.seg + b.seqs;
    return p;
}

long long scan_states(const Batch &b, int C)
{
    return ((long long)b.rows / kRun + b.seqs) * C;
}

long long scan_workspace(bool grad, const Batch &b, int C, bool packed)
{
    const ScanPlan p = scan_plan(b, C, packed);
    long long floats = p.cut ? 2LL * p.segs * C : 0;
    if (grad)
        floats += (long long)p.segs * C;
    return 4 * floats;
}

int launch_scan_fwd(const ScanArgs &a, void *stream)
{
    hipStream_t st = static_cast<hipStream_t>(stream);
    const ScanPlan p = scan_plan(a.batch, a.C, a.batch.off != nullptr);
    const int slabs = (int)cdiv(a.C, kSlab);
    const long long blocks = (long long)slabs * p.segs;
    if (blocks > 0x7fffffffLL)
        return DWCONV_ERR_BAD_DIM;
    return with_variant(a, [&](auto *t, auto v) {
        using T = std::remove_pointer_t<decltype(t)>;
        constexpr int V = decltype(v)::value, KT = 8;
        int rc = DWCONV_OK;
        if (p.cut)
            rc = dwconv::launch_kernel(k_scan_fwd<T, V, KT, true>, dim3((unsigned)blocks),
                                       dim3(Layout<V, KT>::threads), 0, st, a, p.seg, slabs);
        if (rc == DWCONV_OK)
            rc = dwconv::launch_kernel(k_scan_fwd<T, V, KT, false>, dim3((unsigned)blocks),
                                       dim3(Layout<V, KT>::threads), 0, st, a, p.seg, slabs);
        return rc;
    });
}

int launch_scan_grad(const ScanArgs &args, void *stream)
{
    hipStream_t st = static_cast<hipStream_t>(stream);
    ScanArgs a = args;
    const ScanPlan p = scan_plan(a.batch, a.C, a.batch.off != nullptr);
    const int slabs = (int)cdiv(a.C, kSlab);
    const long long blocks = (long long)slabs * p.segs;
    if (blocks > 0x7fffffffLL)
        return DWCONV_ERR_BAD_DIM;
    a.part = p.cut ? a.agg + 2LL * p.segs * a.C : a.agg;
    return with_variant(a, [&](auto *t, auto v) {
        using T = std::remove_pointer_t<decltype(t)>;
        constexpr int V = decltype(v)::value, KT = V == 1 ? 8 : 4;
        int rc = DWCONV_OK;
        if (p.cut)
            rc = dwconv::launch_kernel(k_scan_grad<T, V, KT, true>, dim3((unsigned)blocks),
                                       dim3(Layout<V, KT>::threads), 0, st, a, p.seg, slabs);
        if (rc == DWCONV_OK)
            rc = dwconv::launch_kernel(k_scan_grad<T, V, KT, false>, dim3((unsigned)blocks),
                                       dim3(Layout<V, KT>::threads), 0, st, a, p.seg, slabs);
        if (rc == DWCONV_OK)
            rc = dwconv::launch_kernel(k_scan_grad_sum, dim3((unsigned)cdiv(a.C, 64)), dim3(1024),
                                       0, st, (const float *)a.part, p.segs, a.C, a.lam, a.scale,
                                       a.dlam);
        return rc;
    });
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
        return dwconv::launch_kernel(k_scan_step<T, V>, dim3((unsigned)blocks), dim3(256), 0,
                                     static_cast<hipStream_t>(stream), a, groups);
    });
}

}  // namespace dwseq

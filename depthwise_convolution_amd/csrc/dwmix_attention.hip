// dwmix_attention.hip -- linear attention with a decay for each head
// (include/dwconv_mix.h): the single-token step, and the walks that the forward
// and the gradients are made of (dwmix_attention.h).
#include "dwmix_attention.h"

#include <algorithm>

namespace dwmix {
namespace {

using namespace dwseq;

// ------------------------------------------------------------ one token
// S = a S + k v^T, y = scale q S, in float32.  Bound by reading and writing the states:
// a workgroup takes one head of one sequence; the lanes of a row of threads take V
// adjacent columns each, the rows of threads every `ty`-th row of S, and their parts
// of y are added in LDS in order.  64 sequences, 16 heads of 128: 22 us, 6.1 TB/s.
template <typename T, int V>
__global__ __launch_bounds__(256) void k_attention_step(AttentionArgs a, int tx, int ty)
{
    __shared__ float qk[2][DWCONV_ATTENTION_MAX_DIM], sums[256 * V];
    const long long id = block_id();
    if (id >= (long long)a.batch.seqs * a.H)
        return;
    const long long seq = id / a.H;
    const int h = (int)(id % a.H), kv = h / (a.H / a.KV);
    const T *q = static_cast<const T *>(a.q) + seq * a.ldq + h * a.Dk;
    const T *k = static_cast<const T *>(a.k) + seq * a.ldk + kv * a.Dk;
    const T *v = static_cast<const T *>(a.v) + seq * a.ldv + kv * a.Dv;
    if ((int)threadIdx.x < a.Dk) {
        qk[0][threadIdx.x] = (float)q[threadIdx.x] * a.scale;
        qk[1][threadIdx.x] = (float)k[threadIdx.x];
    }
    const int x = (int)threadIdx.x % tx, y = (int)threadIdx.x / tx, dv = x * V;
    const bool mine = y < ty && dv < a.Dv;
    const float g = a.log_decay[h];
    const float decay = g > 0.0f ? 1.0f : expf(g);
    float add[V] = {}, out[V] = {};
    if (mine)
        load<T, V>(v + dv, add);
    __syncthreads();
    float *s = a.h + (seq * a.H + h) * a.Dk * a.Dv + dv;
    if (mine) {
        constexpr int kAhead = 8;
        int d = y;
        for (; d + (kAhead - 1) * ty < a.Dk; d += kAhead * ty) {
            float r[kAhead][V];
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
                load<float, V>(s + (d + u * ty) * a.Dv, r[u]);
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                const float kd = qk[1][d + u * ty], qd = qk[0][d + u * ty];
#pragma unroll
                for (int e = 0; e < V; ++e) {
                    r[u][e] = decay * r[u][e] + kd * add[e];
                    out[e] += qd * r[u][e];
                }
                store<float, V>(s + (d + u * ty) * a.Dv, r[u]);
            }
        }
        for (; d < a.Dk; d += ty) {
            float r[V];
            load<float, V>(s + d * a.Dv, r);
#pragma unroll
            for (int e = 0; e < V; ++e) {
                r[e] = decay * r[e] + qk[1][d] * add[e];
                out[e] += qk[0][d] * r[e];
            }
            store<float, V>(s + d * a.Dv, r);
        }
    }
#pragma unroll
    for (int e = 0; e < V; ++e)
        sums[threadIdx.x * V + e] = out[e];
    __syncthreads();
    if (y != 0 || !mine)
        return;
    for (int r = 1; r < ty; ++r)
#pragma unroll
        for (int e = 0; e < V; ++e)
            out[e] += sums[(r * tx + x) * V + e];
    store<T, V>(static_cast<T *>(a.y) + seq * a.ldy + h * a.Dv + dv, out);
}

// ------------------------------------------------------- shared heads
// The gradients of a key or value head: the sum of its query heads', in order.
struct Shared {
    const float *part;
    void *out;
    long long ldo;
    int D, blocks;
};

template <typename T, int V>
__global__ __launch_bounds__(256) void k_shared(Shared k, Shared v, int rows, int H, int KV)
{
    const bool first = block_id() < (unsigned)k.blocks;
    const Shared &s = first ? k : v;
    if (!s.out)
        return;     // what the grid's last row has too many
    const unsigned wide = (unsigned)(KV * s.D / V);
    const long long id =
        (long long)(block_id() - (first ? 0u : (unsigned)k.blocks)) * 256 + threadIdx.x;
    const long long row = id / wide;
    if (row >= rows)
        return;
    const int at = (int)(id - row * wide) * V, group = H / KV;
    const float *from = s.part + row * H * s.D + (long long)(at / s.D) * group * s.D + at % s.D;
    float sum[V], more[V];
    load<float, V>(from, sum);
    for (int g = 1; g < group; ++g) {
        load<float, V>(from + (long long)g * s.D, more);
#pragma unroll
        for (int e = 0; e < V; ++e)
            sum[e] += more[e];
    }
    store<T, V>(static_cast<T *>(s.out) + row * s.ldo + at, sum);
}

// -------------------------------------------------------------- planning
// Segments: where sequences, heads and column tiles make fewer workgroups than the
// chip holds (two a CU), sequences are cut so that they fill it once; packed ones,
// whose lengths are not known here, into half as long parts, which are shared out more
// evenly (20011 tokens in 37 sequences, 12 heads of 96 and 80 float16: 163 us in all
// against 173; equal lengths lose by it: 8 x 4096, 16 heads of 128, 257 against 218).
// Two workgroups a CU is what the walk has room for with 128 x 128 tiles of 16-bit types, 71
// KB of LDS each.  Widths above 128 take 80 to 96 KB, one a CU (8 x 4096, 16 heads of 256
// bfloat16 867 us, 5.1 times the floor, where 128 has 2.7), tiles of 64 x 64 31 to 47 KB, three to
// five, and a gradient's walks share a launch: other numbers of segments have not been
// measured for these.
struct SegmentPlan {
    int segment, per_seq, items;
    bool cut;
    long long slots;            // bytes
};

constexpr int kChunk = 64, kFull = 512;

SegmentPlan segment_plan(const Batch &b, bool packed, int H, int Dk, int Dv)
{
    SegmentPlan p;
    const long long tiles = (long long)H * cdiv(Dv, walk_tile(Dk, Dv));
    const long long tokens = packed ? b.rows : b.tokens;
    long long segment = std::max(tokens, 1LL);
    if (tokens <= 2 * kChunk)
        ;           // two chunks: two more launches would cost more than they save
    else if (packed)
        segment = std::min(segment, cdiv(b.rows * tiles, 2 * kFull));
    else if (b.seqs * tiles < kFull)
        segment = cdiv(tokens, cdiv(kFull, b.seqs * tiles));
    segment = cdiv(std::max(segment, 1LL), kChunk) * kChunk;
    p.segment = (int)std::min(segment, 0x40000000LL);
    p.per_seq = (int)std::max(1LL, cdiv(b.tokens, p.segment));
    const long long items = packed ? b.rows / p.segment + (long long)b.seqs
                                   : (long long)b.seqs * p.per_seq;
    p.items = (int)std::min(items, 0x7fffffffLL);
    p.cut = tokens > p.segment;
    // one for each segment but the first that all rows would be cut into as one sequence
    p.slots = p.cut ? 4LL * (cdiv(b.rows, p.segment) - 1) * H * Dk * Dv : 0;
    return p;
}

long long round16(long long bytes) { return cdiv(bytes, 16) * 16; }

int walk(int type, const Walk *w, int count, hipStream_t st)
{
    return with_type(type, [&](auto *t) {
        return launch_walks<std::remove_pointer_t<decltype(t)>>(w, count, st);
    });
}

// The parts of the walk that a batch and its plan set.
void place(Walk &w, const SegmentPlan &p, const Batch &b, int H, int Dk, int Dv, void *slots)
{
    w.batch = b;
    w.H = H;
    w.Dk = Dk;
    w.Dv = Dv;
    w.segment = p.segment;
    w.per_seq = p.per_seq;
    w.items = p.items;
    w.slots = p.cut ? static_cast<float *>(slots) : nullptr;
}

// The gradients' segments and the parts of their workspace: the slots of dq and those
// of dk and dv, then shared heads' parts.
struct GradPlan {
    SegmentPlan q, k;
    long long slots, dk, dv, total;
};

GradPlan grad_plan(const Batch &b, bool packed, int H, int KV, int Dk, int Dv)
{
    GradPlan p;
    p.q = p.k = segment_plan(b, packed, H, Dv, Dk);
    p.slots = round16(p.q.slots);
    p.dk = KV == H ? 0 : round16(4LL * b.rows * H * Dk);
    p.dv = KV == H ? 0 : round16(4LL * b.rows * H * Dv);
    p.total = 2 * p.slots + p.dk + p.dv;
    return p;
}

}  // namespace

long long attention_workspace(bool grad, const Batch &b, bool packed, int H, int KV, int Dk,
                              int Dv)
{
    return grad ? grad_plan(b, packed, H, KV, Dk, Dv).total
                : round16(segment_plan(b, packed, H, Dk, Dv).slots);
}

int launch_attention_fwd(const AttentionArgs &a, void *stream)
{
    Walk w{};
    place(w, segment_plan(a.batch, a.batch.off != nullptr, a.H, a.Dk, a.Dv), a.batch, a.H, a.Dk,
          a.Dv, a.workspace);
    w.q = a.q; w.k = a.k; w.v = a.v; w.out = a.y;
    w.ldq = a.ldq; w.ldk = a.ldk; w.ldv = a.ldv; w.ldo = a.ldy;
    w.gq = 1;
    w.gk = w.gv = a.H / a.KV;
    w.log_decay = a.log_decay; w.state0 = a.h0; w.state1 = a.hT;
    w.s0 = w.s1 = a.scale;
    w.s2 = 1.0f;
    return walk(a.type, &w, 1, static_cast<hipStream_t>(stream));
}

// The walks of dq, of dk (and dh0) and of dv in the same launches.  The states of the
// last two, sums of q dy^T from the end, are each other's transposes: computed once.
int launch_attention_grad(const AttentionArgs &a, void *stream)
{
    hipStream_t st = static_cast<hipStream_t>(stream);
    const int group = a.H / a.KV;
    const GradPlan plan = grad_plan(a.batch, a.batch.off != nullptr, a.H, a.KV, a.Dk, a.Dv);
    char *space = static_cast<char *>(a.workspace), *parts = space + 2 * plan.slots;
    Walk walks[kWalks] = {};
    int count = 0;
    if (a.dq) {
        Walk &w = walks[count++];
        place(w, plan.q, a.batch, a.H, a.Dv, a.Dk, space);
        w.q = a.dy; w.k = a.v; w.v = a.k; w.out = a.dq;
        w.ldq = a.lddy; w.ldk = a.ldv; w.ldv = a.ldk; w.ldo = a.lddq;
        w.gq = 1;
        w.gk = w.gv = group;
        w.log_decay = a.log_decay; w.state0 = a.h0; w.flip = true;
        w.s0 = w.s1 = a.scale;
        w.s2 = 1.0f;
    }
    const bool with_k = a.dk || a.dh0;
    Shared dk{reinterpret_cast<float *>(parts), nullptr, a.lddk, a.Dk, 0};
    Shared dv{reinterpret_cast<float *>(parts + plan.dk), nullptr, a.lddv, a.Dv, 0};
    if (with_k) {
        Walk &w = walks[count++];
        place(w, plan.k, a.batch, a.H, a.Dv, a.Dk, space + plan.slots);
        w.q = a.v; w.k = a.dy; w.v = a.q;
        w.ldq = a.ldv; w.ldk = a.lddy; w.ldv = a.ldq;
        w.gq = group;
        w.gk = w.gv = 1;
        w.out = a.dk; w.ldo = a.lddk;
        if (group > 1 && a.dk) {
            w.out = parts;
            w.ldo = (long long)a.H * a.Dk;
            w.out32 = true;
            dk.out = a.dk;
        }
        w.log_decay = a.log_decay; w.state0 = a.dhT; w.state1 = a.dh0; w.flip = true;
        w.s0 = w.s2 = a.scale;
        w.s1 = 1.0f;
        w.late = w.back = 1;
    }
    if (a.dv) {
        Walk &w = walks[count++];
        place(w, plan.k, a.batch, a.H, a.Dk, a.Dv, space + plan.slots);
        w.ready = with_k;
        w.q = a.k; w.k = a.q; w.v = a.dy;
        w.ldq = a.ldk; w.ldk = a.ldq; w.ldv = a.lddy;
        w.gq = group;
        w.gk = w.gv = 1;
        w.out = a.dv; w.ldo = a.lddv;
        if (group > 1) {
            w.out = parts + plan.dk;
            w.ldo = (long long)a.H * a.Dv;
            w.out32 = true;
            dv.out = a.dv;
        }
        w.log_decay = a.log_decay; w.state0 = a.dhT;
        w.s0 = w.s2 = a.scale;
        w.s1 = 1.0f;
        w.late = w.back = 1;
    }
    const int rc = walk(a.type, walks, count, st);
    if (rc != DWCONV_OK || (!dk.out && !dv.out) || a.batch.rows == 0)
        return rc;
    const int vec = a.Dk % 4 == 0 && a.Dv % 4 == 0 ? 4 : 1;
    auto blocks_of = [&](const Shared &s) {
        return s.out ? cdiv((long long)a.batch.rows * a.KV * (s.D / vec), 256) : 0;
    };
    const long long total = blocks_of(dk) + blocks_of(dv);
    if (total > 0x7fffffffLL)
        return DWCONV_ERR_BAD_DIM;
    dk.blocks = (int)blocks_of(dk);
    dv.blocks = (int)blocks_of(dv);
    return with_type(a.type, [&](auto *t) {
        using T = std::remove_pointer_t<decltype(t)>;
        return dwconv::launch_kernel(vec == 4 ? k_shared<T, 4> : k_shared<T, 1>, grid_of(total),
                                     dim3(256), 0, st, dk, dv, a.batch.rows, a.H, a.KV);
    });
}

int launch_attention_step(const AttentionArgs &a, void *stream)
{
    hipStream_t st = static_cast<hipStream_t>(stream);
    const long long blocks = (long long)a.batch.seqs * a.H;
    if (blocks > 0x7fffffffLL)
        return DWCONV_ERR_BAD_DIM;
    return with_type(a.type, [&](auto *t) {
        using T = std::remove_pointer_t<decltype(t)>;
        auto run = [&](auto v) {
            constexpr int V = decltype(v)::value;
            const int tx = (int)cdiv(a.Dv, V), ty = 256 / tx;
            return dwconv::launch_kernel(k_attention_step<T, V>, grid_of(blocks), dim3(256), 0, st,
                                         a, tx, ty);
        };
        return a.Dv % 4 == 0 ? run(std::integral_constant<int, 4>())
                             : run(std::integral_constant<int, 1>());
    });
}

}  // namespace dwmix

// head_norm.cu -- norms of heads with rotary positions on several axes in the same pass: on packed
// rows, their gradient, and the append of queries, keys and values to the pages of a cache.
//
// cortiq-engine 0.8.49 src/gpu_wgpu/nemotron_audio.rs, kernel ae_qk, normalises each head of q and
// k (LayerNorm) and turns it by a table of cosines and sines.
//
//   y = w (x - mu) r + b, r = 1 / sqrt(mean((x - mu)^2) + eps), then pairs of y turned.
// Gradient, g = R^T dout, h = (x - mu) r, u = w g:
//   dx = r (u - h mean(u h) - mean(u)), the last term for LayerNorm only;
//   dw = sum g h, db = sum g over rows and heads.
//
// What bounds it: bytes, and for rows of several axes or types the instructions beside them.  A head
// is held by G lanes of a warp, eight values each in two runs of four (head_units.cuh), so its sums
// are log2 G shuffles and every value is read and written once; a group of lanes takes up to
// kHeadsPer heads of a row, whose loads are in flight together and share the row's angles.
// Measured: 4900 rows of 32 heads of 80 to bf16, LayerNorm, two axes 26 us (2.9 TB/s); gradient of 4096
// rows of 40 heads of 128 48 us (5.3 TB/s); append of 8002 tokens of 28/4 heads of 128, three axes
// 51 us (4.3 TB/s), of 256 tokens of 32/8 heads 5 us (the host's call).
#include <initializer_list>

#include "head_units.cuh"
#include "kv_internal.h"
#include "wq_device.cuh"

namespace wq {
namespace {

// Heads of a group of lanes: 1, 2 and 4 took 100, 63 and 60 us for an append of 8002 tokens.  Half the
// lanes and twice the values to a lane, with two heads: 72 in place of 52.
constexpr int kHeadsPer = 4;
constexpr int kGradHeads = 2;  // and of the gradient, which holds x and dout: 1, 2, 4 took 64, 48, 59
constexpr int kThreads = 128;

// A lane's units of a head.
template <int N, int U> struct Held {
    Vals<N> a[U], b[U];
};

// The lanes' common view of a head: G lanes, unit lane + G i for i < U.
template <int N, int G, int U> struct Lanes {
    int lane, units, head_dim;
    float inv_d;
    Place place[U];
    __device__ __forceinline__ Lanes(const AxesView &ax, int d) : head_dim(d) {
        lane = threadIdx.x & (G - 1);
        units = (d + 2 * N - 1) / (2 * N);
        inv_d = 1.f / d;
#pragma unroll
        for (int i = 0; i < U; ++i) place[i] = place_of<N>(lane + G * i, ax.rot, ax.flags);
    }
    __device__ __forceinline__ bool has(int i) const { return lane + G * i < units; }
    // An odd head_dim ends in a single value.
    __device__ __forceinline__ bool both(int i) const { return N > 1 || place[i].b < head_dim; }
    // A head at p + at (elements): 32-bit offsets from a row's address, which is worked out once.
    __device__ __forceinline__ void load(Held<N, U> &x, const float *p, unsigned at = 0) const {
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (has(i)) x.a[i] = load_vals<N>(p + (at + place[i].a));
            if (has(i) && both(i)) x.b[i] = load_vals<N>(p + (at + place[i].b));
        }
    }
    template <typename T>
    __device__ __forceinline__ void store(const Held<N, U> &x, T *p, unsigned at = 0) const {
#pragma unroll
        for (int i = 0; i < U; ++i) {
            if (has(i)) store_vals(p + (at + place[i].a), x.a[i]);
            if (has(i) && both(i)) store_vals(p + (at + place[i].b), x.b[i]);
        }
    }
    // Weights or biases: `fill` where there are none.
    __device__ __forceinline__ void load_or(Held<N, U> &x, const float *p, float fill) const {
#pragma unroll
        for (int i = 0; i < U; ++i)
#pragma unroll
            for (int j = 0; j < N; ++j) x.a[i].v[j] = x.b[i].v[j] = fill;
        if (p) load(x, p);
    }
    // f(i, j, b) over a lane's values of a head, and its sums over the G lanes of H heads together:
    // their shuffles are in flight at the same time.
    template <typename F> __device__ __forceinline__ static float part(F f) {
        float v = 0.f;
#pragma unroll
        for (int i = 0; i < U; ++i)
#pragma unroll
            for (int j = 0; j < N; ++j) v += f(i, j, false) + f(i, j, true);
        return v;
    }
    template <int H> __device__ __forceinline__ static void sum_groups(float (&v)[H]) {
#pragma unroll
        for (int o = G / 2; o > 0; o >>= 1)
#pragma unroll
            for (int h = 0; h < H; ++h) v[h] += __shfl_xor_sync(0xFFFFFFFFu, v[h], o);
    }
    // x become (x - mu) r by the group's kind of norm (none: as they were); their r.  Values beyond a
    // head are 0 and stay so.  `summed`: any lane of the launch takes a mean; a warp's lanes may
    // have different kinds and shuffle together.
    template <int H>
    __device__ __forceinline__ void hat(Held<N, U> (&x)[H], int kind, bool summed, float eps,
                                        float (&r)[H]) const {
        if (summed) {
            float mu[H];
#pragma unroll
            for (int h = 0; h < H; ++h)
                mu[h] = part([&](int i, int j, bool b) {
                    return b ? x[h].b[i].v[j] : x[h].a[i].v[j];
                });
            sum_groups(mu);
#pragma unroll
            for (int h = 0; h < H; ++h) {
                const float m = kind == WQ_HEAD_LAYER ? mu[h] * inv_d : 0.f;
#pragma unroll
                for (int i = 0; i < U; ++i)
#pragma unroll
                    for (int j = 0; j < N; ++j) {
                        x[h].a[i].v[j] -= has(i) ? m : 0.f;
                        x[h].b[i].v[j] -= has(i) && both(i) ? m : 0.f;
                    }
            }
        }
#pragma unroll
        for (int h = 0; h < H; ++h)
            r[h] = part([&](int i, int j, bool b) {
                const float v = b ? x[h].b[i].v[j] : x[h].a[i].v[j];
                return v * v;
            });
        sum_groups(r);
#pragma unroll
        for (int h = 0; h < H; ++h) {
            r[h] = kind == WQ_HEAD_NONE ? 1.f : rsqrtf(fmaf(r[h], inv_d, eps));
#pragma unroll
            for (int i = 0; i < U; ++i)
#pragma unroll
                for (int j = 0; j < N; ++j) x[h].a[i].v[j] *= r[h], x[h].b[i].v[j] *= r[h];
        }
    }
    // y of a head with its weights and biases.
    __device__ __forceinline__ void weigh(Held<N, U> &x, const Held<N, U> &w,
                                          const Held<N, U> &c) const {
#pragma unroll
        for (int i = 0; i < U; ++i)
#pragma unroll
            for (int j = 0; j < N; ++j) {
                x.a[i].v[j] = fmaf(x.a[i].v[j], w.a[i].v[j], c.a[i].v[j]);
                x.b[i].v[j] = fmaf(x.b[i].v[j], w.b[i].v[j], c.b[i].v[j]);
            }
    }
};

// A row's positions; false where one that turns something is out of range.
struct Where {
    int p[4];
    __device__ __forceinline__ bool load(const AxesView &ax, long long t) {
        bool ok = true;
#pragma unroll
        for (int a = 0; a < 4; ++a) {
            p[a] = a < ax.axes ? ax.pos[a * ax.pos_stride + t] : 0;
            if (a < ax.axes && (ax.used >> a & 1) && (unsigned)p[a] >= (unsigned)ax.table_rows)
                ok = false;
        }
        return ok;
    }
};

// The angles of the rows that a block works on, [rows][rot / 2] in shared memory, where pairs go by
// several axes: gathered once for all of a row's heads (each group of lanes for itself: an append
// of 8002 tokens took 60 us).  Positions out of range leave zeros, which no one uses.
__device__ __forceinline__ void stage_angles(const AxesView &ax, float2 *angles, long long t,
                                             int rows) {
    const int half = ax.rot >> 1;
    for (int i = threadIdx.x; i < rows * half; i += kThreads) {
        const int r = i / half, code = ax.code[i - r * half];
        const int pos = ax.pos[(code >> 8) * ax.pos_stride + t + r];
        angles[i] = (unsigned)pos < (unsigned)ax.table_rows
                        ? ax.table[(long long)pos * ax.table_pairs + (code & 255)]
                        : make_float2(0.f, 0.f);
    }
}
__device__ __forceinline__ bool stages(const AxesView &ax) { return ax.rot > 0 && !ax.straight; }

// A row's angles: `at` is its first.
template <int N, int G, int U> struct Turns {
    Angles<N> cs[U];
    __device__ __forceinline__ void load(const Lanes<N, G, U> &l, const float2 *at,
                                         unsigned flags) {
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (l.place[i].turn) cs[i] = load_angles<N>(at + (l.lane + G * i) * N, flags);
    }
    __device__ __forceinline__ void apply(const Lanes<N, G, U> &l, Held<N, U> &x,
                                          unsigned flags) const {
#pragma unroll
        for (int i = 0; i < U; ++i)
            if (l.place[i].turn) turn<N>(x.a[i], x.b[i], cs[i], flags);
    }
};

// Groups of lanes over rows and blocks of heads.
struct HeadDeal {
    FastDiv per_row;  // blocks of heads in a row
    unsigned count;
};

template <typename T, int N, int G, int U>
__global__ void __launch_bounds__(kThreads, N == 4 ? 6 : 1)
    norm_rope_kernel(const __grid_constant__ AxesView ax, NormView nv, HeadDeal deal, int head_dim,
                     const float *x, long long x_stride, int n_heads, T *out, long long out_stride,
                     long long t0) {
    extern __shared__ __align__(16) float2 s_angles[];
    pdl_enter();
    const unsigned first = blockIdx.x * (unsigned)(kThreads / G), at = first + threadIdx.x / G;
    // Every lane stays for the shuffles.
    const bool live = at < deal.count;
    const unsigned row0 = deal.per_row.div(first), row = live ? deal.per_row.div(at) : row0;
    const int h0 = live ? (int)(at - row * deal.per_row.d) * kHeadsPer : 0;
    const int n = live ? min(kHeadsPer, n_heads - h0) : 0;
    const long long t = t0 + row;
    const Lanes<N, G, U> l(ax, head_dim);
    const float *xi = x + t * x_stride + (long long)h0 * head_dim;
    T *o = out + t * out_stride + (long long)h0 * head_dim;
    Held<N, U> v[kHeadsPer] = {};
#pragma unroll
    for (int i = 0; i < kHeadsPer; ++i)
        if (i < n) l.load(v[i], xi, i * head_dim);
    Where w;
    const bool ok = w.load(ax, t);
    if (live && !ok && l.lane == 0) record_status(ax.status, kStBadIndex);
    if (stages(ax)) {
        const unsigned last = min(first + kThreads / G, deal.count) - 1;
        stage_angles(ax, s_angles, t0 + row0, (int)(deal.per_row.div(last) - row0) + 1);
        __syncthreads();
    }
    Turns<N, G, U> turns;
    if (ok && ax.rot > 0)
        turns.load(l, stages(ax) ? s_angles + (row - row0) * (ax.rot >> 1)
                                 : ax.table + (long long)w.p[0] * ax.table_pairs, ax.flags);
    Held<N, U> wt, bias;
    if (nv.kind != WQ_HEAD_NONE) {
        l.load_or(wt, nv.weight, 1.f);
        l.load_or(bias, nv.bias, 0.f);
    }
    if (nv.kind != WQ_HEAD_NONE) {
        float r[kHeadsPer];
        l.hat(v, nv.kind, nv.kind == WQ_HEAD_LAYER, nv.eps, r);
    }
#pragma unroll
    for (int i = 0; i < kHeadsPer; ++i)
        if (i < n && ok) {
            if (nv.kind != WQ_HEAD_NONE) l.weigh(v[i], wt, bias);
            turns.apply(l, v[i], ax.flags);
            l.store(v[i], o, i * head_dim);
        }
}

// Blocks of heads are of q, of k or of v alone: a group of lanes has one norm.
struct Roles {
    int q_blocks, kv_blocks;
};
// What a row's groups of lanes share, found by one thread: the row's offset in the pools (-1:
// nothing is written) and its position on axis 0.
struct Place1 {
    long long row;
    int pos;
};

template <int DT, typename Q, int N, int G, int U>
__global__ void __launch_bounds__(kThreads, N == 4 ? 8 : 1)
    append_norm_kernel(const __grid_constant__ AxesView ax, NormView q_norm, NormView k_norm,
                       AppendNormArgs a, KvView kv, HeadDeal deal, Roles roles, int t0) {
    extern __shared__ __align__(16) float2 s_angles[];
    __shared__ Place1 s_place[kThreads / G];
    pdl_enter();
    using T = typename KvType<DT>::T;
    const unsigned first = blockIdx.x * (unsigned)(kThreads / G), at = first + threadIdx.x / G;
    const bool live = at < deal.count;
    const unsigned row0 = deal.per_row.div(first), row_at = live ? deal.per_row.div(at) : row0;
    int block = live ? (int)(at - row_at * deal.per_row.d) : 0;
    const int role = block < roles.q_blocks                     ? 0
                     : block < roles.q_blocks + roles.kv_blocks ? 1
                                                                : 2;
    block -= role == 0 ? 0 : role == 1 ? roles.q_blocks : roles.q_blocks + roles.kv_blocks;
    const int d = kv.head_dim, heads = role == 0 ? a.h_q : kv.n_heads;
    const int h0 = block * kHeadsPer, n = live ? min(kHeadsPer, heads - h0) : 0;
    const int t = t0 + (int)row_at;
    const Lanes<N, G, U> l(ax, d);
    const float *const x = (role == 0   ? a.q + t * a.q_stride
                            : role == 1 ? a.k + t * a.k_stride
                                        : a.v + t * a.v_stride) +
                           (long long)h0 * d;
    // The values do not wait for the slot.
    Held<N, U> v[kHeadsPer] = {};
#pragma unroll
    for (int i = 0; i < kHeadsPer; ++i)
        if (i < n) l.load(v[i], x, i * d);
    {
        const int rows =
            (int)(deal.per_row.div(min(first + kThreads / G, deal.count) - 1) - row0) + 1;
        if ((int)threadIdx.x < rows) {
            const int tt = t0 + (int)row0 + threadIdx.x;
            const int slot = a.slot[tt], seq = a.seq ? a.seq[tt] : tt;
            Where w;
            bool ok = w.load(ax, tt);
            ok = ok && (unsigned)seq < (unsigned)a.n_seq && slot >= 0 && slot < a.n_slots;
            const long long at_row = ok ? kv.row(seq, 0, slot) : -1;
            if (at_row < 0 && slot >= 0) record_status(ax.status, kStBadIndex);
            s_place[threadIdx.x] = {at_row, w.p[0]};
        }
        if (stages(ax)) stage_angles(ax, s_angles, t0 + row0, rows);
        __syncthreads();
    }
    const Place1 place = s_place[row_at - row0];
    const long long row = place.row;
    const bool ok = row >= 0;
    Turns<N, G, U> turns;
    if (ok && role < 2 && ax.rot > 0)
        turns.load(l, stages(ax) ? s_angles + (row_at - row0) * (ax.rot >> 1)
                                 : ax.table + (long long)place.pos * ax.table_pairs, ax.flags);
    // The lanes of a warp may hold both roles: all of them run the sums that either norm has.
    const bool any = q_norm.kind != WQ_HEAD_NONE || k_norm.kind != WQ_HEAD_NONE;
    const bool layer = q_norm.kind == WQ_HEAD_LAYER || k_norm.kind == WQ_HEAD_LAYER;
    const int kind = role == 0 ? q_norm.kind : role == 1 ? k_norm.kind : WQ_HEAD_NONE;
    const float eps = role == 0 ? q_norm.eps : k_norm.eps;
    Held<N, U> wt, bias;
    if (kind != WQ_HEAD_NONE) {
        l.load_or(wt, role == 0 ? q_norm.weight : k_norm.weight, 1.f);
        l.load_or(bias, role == 0 ? q_norm.bias : k_norm.bias, 0.f);
    }
    if (any) {
        float r[kHeadsPer];
        l.hat(v, kind, layer, eps, r);
        if (kind != WQ_HEAD_NONE)
#pragma unroll
            for (int i = 0; i < kHeadsPer; ++i) l.weigh(v[i], wt, bias);
    }
    if (!ok) return;
    if (role == 0) {
        Q *const o = static_cast<Q *>(a.q_out) + t * a.q_out_stride + (long long)h0 * d;
#pragma unroll
        for (int i = 0; i < kHeadsPer; ++i)
            if (i < n) {
                turns.apply(l, v[i], ax.flags);
                l.store(v[i], o, i * d);
            }
        return;
    }
    char *o = (role == 1 ? kv.k : kv.v) + row + h0 * kv.head_stride;
#pragma unroll
    for (int i = 0; i < kHeadsPer; ++i, o += kv.head_stride)
        if (i < n) {
            if (role == 1) turns.apply(l, v[i], ax.flags);
            l.store(v[i], reinterpret_cast<T *>(o));
        }
    if (role == 1 && l.lane < n && (a.acc || a.slot_pos)) {
        const int slot = a.slot[t], seq = a.seq ? a.seq[t] : t;
        const long long to = ((long long)seq * kv.n_heads + h0 + l.lane) * a.acc_stride + slot;
        if (a.acc) a.acc[to] = 0.f;
        if (a.slot_pos) a.slot_pos[to] = place.pos;
    }
}

// Groups of lanes stride over the heads, so that a lane's dims, and with them its sums for dw and
// db, stay the same; the blocks' sums are added by grad_sums_kernel in a fixed order.
template <int N, int G, int U>
__global__ void __launch_bounds__(kThreads)
    norm_rope_grad_kernel(const __grid_constant__ AxesView ax, NormView nv, HeadDeal deal,
                          int head_dim, const float *x, long long x_stride, const float *grad,
                          long long grad_stride, int n_heads, float *grad_x,
                          long long grad_x_stride, float *parts) {
    // [groups][2][head_dim] at the end, and before it a step's angles
    extern __shared__ __align__(16) float s_sums[];
    float2 *const s_angles = reinterpret_cast<float2 *>(s_sums);
    pdl_enter();
    const Lanes<N, G, U> l(ax, head_dim);
    const unsigned flags = ax.flags | WQ_ROPE_TRANSPOSE;
    const unsigned groups = gridDim.x * (unsigned)(kThreads / G);
    const unsigned block0 = blockIdx.x * (unsigned)(kThreads / G), first = block0 + threadIdx.x / G;
    unsigned row0 = 0;
    Held<N, U> wt, sum_w = {}, sum_b = {};
    l.load_or(wt, nv.kind != WQ_HEAD_NONE ? nv.weight : nullptr, 1.f);
    const unsigned steps = (deal.count + groups - 1) / groups;
    for (unsigned step = 0; step < steps; ++step) {
        const unsigned long long where = (unsigned long long)step * groups + first;
        const bool live = where < deal.count;
        const unsigned at = live ? (unsigned)where : 0u;
        const unsigned t = deal.per_row.div(at);
        const int h0 = (int)(at - t * deal.per_row.d) * kGradHeads;
        const int n = live ? min(kGradHeads, n_heads - h0) : 0;
        Held<N, U> v[kGradHeads] = {}, g[kGradHeads] = {};
        const float *const xi = x + t * x_stride + (long long)h0 * head_dim;
        const float *const gi = grad + t * grad_stride + (long long)h0 * head_dim;
#pragma unroll
        for (int i = 0; i < kGradHeads; ++i)
            if (i < n) {
                l.load(v[i], xi, i * head_dim);
                l.load(g[i], gi, i * head_dim);
            }
        Where w;
        const bool ok = w.load(ax, t);
        if (live && !ok && l.lane == 0) record_status(ax.status, kStBadIndex);
        if (stages(ax)) {
            const unsigned long long from = (unsigned long long)step * groups + block0;
            __syncthreads();  // the step before has its angles
            if (from < deal.count) {
                const unsigned last = (unsigned)min(from + kThreads / G,
                                                    (unsigned long long)deal.count) - 1;
                row0 = deal.per_row.div((unsigned)from);
                stage_angles(ax, s_angles, row0, (int)(deal.per_row.div(last) - row0) + 1);
            }
            __syncthreads();
        }
        Turns<N, G, U> turns;
        if (ok && ax.rot > 0)
            turns.load(l, stages(ax) ? s_angles + (live ? t - row0 : 0u) * (ax.rot >> 1)
                                     : ax.table + (long long)w.p[0] * ax.table_pairs, flags);
#pragma unroll
        for (int i = 0; i < kGradHeads; ++i)
            if (i < n && ok) turns.apply(l, g[i], flags);
        if (nv.kind != WQ_HEAD_NONE) {
            float r[kGradHeads], uh[kGradHeads], mu[kGradHeads];
            l.hat(v, nv.kind, nv.kind == WQ_HEAD_LAYER, nv.eps, r);
#pragma unroll
            for (int i = 0; i < kGradHeads; ++i) {
                if (i < n && ok) {
#pragma unroll
                    for (int k = 0; k < U; ++k)
#pragma unroll
                        for (int j = 0; j < N; ++j) {
                            sum_w.a[k].v[j] = fmaf(g[i].a[k].v[j], v[i].a[k].v[j], sum_w.a[k].v[j]);
                            sum_w.b[k].v[j] = fmaf(g[i].b[k].v[j], v[i].b[k].v[j], sum_w.b[k].v[j]);
                            sum_b.a[k].v[j] += g[i].a[k].v[j];
                            sum_b.b[k].v[j] += g[i].b[k].v[j];
                        }
                }
#pragma unroll
                for (int k = 0; k < U; ++k)
#pragma unroll
                    for (int j = 0; j < N; ++j) {
                        g[i].a[k].v[j] *= wt.a[k].v[j];
                        g[i].b[k].v[j] *= wt.b[k].v[j];
                    }
                uh[i] = l.part([&](int k, int j, bool b) {
                    return b ? g[i].b[k].v[j] * v[i].b[k].v[j] : g[i].a[k].v[j] * v[i].a[k].v[j];
                });
                mu[i] = l.part([&](int k, int j, bool b) {
                    return b ? g[i].b[k].v[j] : g[i].a[k].v[j];
                });
            }
            l.sum_groups(uh);
            if (nv.kind == WQ_HEAD_LAYER) l.sum_groups(mu);
#pragma unroll
            for (int i = 0; i < kGradHeads; ++i) {
                const float h = uh[i] * l.inv_d;
                const float m = nv.kind == WQ_HEAD_LAYER ? mu[i] * l.inv_d : 0.f;
#pragma unroll
                for (int k = 0; k < U; ++k)
#pragma unroll
                    for (int j = 0; j < N; ++j) {
                        g[i].a[k].v[j] = r[i] * (g[i].a[k].v[j] - v[i].a[k].v[j] * h - m);
                        g[i].b[k].v[j] = r[i] * (g[i].b[k].v[j] - v[i].b[k].v[j] * h - m);
                    }
            }
        }
        float *const o = grad_x + t * grad_x_stride + (long long)h0 * head_dim;
#pragma unroll
        for (int i = 0; i < kGradHeads; ++i)
            if (i < n && ok) l.store(g[i], o, i * head_dim);
    }
    if (!parts) return;
    __syncthreads();
    float *mine = s_sums + (threadIdx.x / G) * 2 * head_dim;
    l.store(sum_w, mine);
    l.store(sum_b, mine + head_dim);
    __syncthreads();
    for (int c = threadIdx.x; c < 2 * head_dim; c += kThreads) {
        float s = 0.f;
        for (int gr = 0; gr < kThreads / G; ++gr) s += s_sums[gr * 2 * head_dim + c];
        parts[(long long)blockIdx.x * 2 * head_dim + c] = s;
    }
}

// dw and db from the blocks' sums: 32 columns of a block, 32 threads to a column.
__global__ void __launch_bounds__(1024) grad_sums_kernel(const float *parts, int blocks,
                                                         int head_dim, float *grad_weight,
                                                         float *grad_bias) {
    __shared__ float s[32][33];
    pdl_enter();
    const int c = blockIdx.x * 32 + threadIdx.x;
    float v = 0.f;
    if (c < 2 * head_dim)
        for (int b = threadIdx.y; b < blocks; b += 32) v += parts[(long long)b * 2 * head_dim + c];
    s[threadIdx.y][threadIdx.x] = v;
    __syncthreads();
    // Row y's warp adds column y of the block.
    const float total = warp_sum(s[threadIdx.x][threadIdx.y]);
    const int col = blockIdx.x * 32 + threadIdx.y;
    if (threadIdx.x == 0 && col < 2 * head_dim) {
        if (col < head_dim) {
            if (grad_weight) grad_weight[col] = total;
        } else if (grad_bias) {
            grad_bias[col - head_dim] = total;
        }
    }
}

bool all16(std::initializer_list<const void *> ps, std::initializer_list<long long> bytes) {
    for (const void *p : ps)
        if ((uintptr_t)p & 15u) return false;
    for (long long s : bytes)
        if (s % 16) return false;
    return true;
}

// Shared memory of the angles of the rows that `groups` groups of lanes span at most.
size_t angle_bytes(const AxesView &ax, const HeadDeal &deal, unsigned groups) {
    if (ax.rot == 0 || ax.straight) return 0;
    const unsigned per = deal.per_row.d, rows = per == 1 ? groups : (groups + per - 2) / per + 1;
    return (size_t)rows * (ax.rot / 2) * sizeof(float2);  // 16 groups, 32 pairs each: 4 KiB at most
}
HeadDeal deal_of(int blocks) { return {make_fast_div((uint32_t)blocks), 0u}; }
int blocks_of(int heads, int per) { return (heads + per - 1) / per; }

// F is called with the units' shape: pairs of a run, lanes of a head, units of a lane.
template <typename F> cudaError_t by_shape(bool wide, int head_dim, F f) {
    if (!wide) return f(std::integral_constant<int, 1>(), std::integral_constant<int, 32>(),
                        std::integral_constant<int, 4>());
    constexpr std::integral_constant<int, 4> four{};
    constexpr std::integral_constant<int, 1> one{};
    if (head_dim <= 64) return f(four, std::integral_constant<int, 8>(), one);
    if (head_dim <= 128) return f(four, std::integral_constant<int, 16>(), one);
    return f(four, std::integral_constant<int, 32>(), one);
}
int lanes_of(bool wide, int head_dim) {
    return !wide || head_dim > 128 ? 32 : head_dim > 64 ? 16 : 8;
}

template <typename F> cudaError_t by_type(int type, F f) {
    switch (type) {
    case kBF16: return f(static_cast<__nv_bfloat16 *>(nullptr));
    case kF16: return f(static_cast<__half *>(nullptr));
    default: return f(static_cast<float *>(nullptr));
    }
}

}  // namespace

cudaError_t launch_norm_rope(const AxesView &ax, const NormView &nv, int n, int n_heads,
                             int head_dim, const float *x, long long x_stride, int out_type,
                             void *out, long long out_stride, const DeviceInfo &dev,
                             cudaStream_t stream) {
    const int ob = out_type == kF32 ? 4 : 2;
    // A run of four 16-bit values is 8 bytes; the rows' 16-byte rule covers it.
    const bool wide = head_dim % 8 == 0 && ax.rot % 8 == 0 &&
                      all16({x, out, nv.weight, nv.bias}, {4 * x_stride, ob * out_stride});
    HeadDeal deal = deal_of(blocks_of(n_heads, kHeadsPer));
    // Launches of so many rows that their threads are counted in 31 bits.
    const long long step = (0x7FFFFF00ll / lanes_of(wide, head_dim)) / deal.per_row.d;
    for (long long t0 = 0; t0 < n; t0 += step) {
        deal.count = (unsigned)((n - t0 < step ? n - t0 : step) * deal.per_row.d);
        const cudaError_t err = by_type(out_type, [&](auto *type) {
            using T = std::remove_pointer_t<decltype(type)>;
            return by_shape(wide, head_dim, [&](auto N, auto G, auto U) {
                const unsigned per = kThreads / G.value;
                return launch_pdl(norm_rope_kernel<T, N.value, G.value, U.value>,
                                  dim3((deal.count + per - 1) / per), dim3(kThreads),
                                  angle_bytes(ax, deal, per), stream, ax, nv, deal, head_dim, x,
                                  x_stride, n_heads, static_cast<T *>(out), out_stride, t0);
            });
        });
        if (err != cudaSuccess) return err;
    }
    return cudaSuccess;
}

cudaError_t launch_append_norm(const AxesView &ax, const NormView &q_norm, const NormView &k_norm,
                               const AppendNormArgs &a, const KvView &kv, const DeviceInfo &dev,
                               cudaStream_t stream) {
    const int qb = a.q_type == kF32 ? 4 : 2;
    const bool q16 = a.h_q == 0 || all16({a.q, a.q_out}, {4 * a.q_stride, qb * a.q_out_stride});
    const bool wide = ax.rot % 8 == 0 && q16 &&
                      all16({a.k, a.v, q_norm.weight, q_norm.bias, k_norm.weight, k_norm.bias},
                            {4 * a.k_stride, 4 * a.v_stride});
    const int d = kv.head_dim;
    const Roles roles{blocks_of(a.h_q, kHeadsPer), blocks_of(kv.n_heads, kHeadsPer)};
    HeadDeal deal = deal_of(roles.q_blocks + 2 * roles.kv_blocks);
    const long long step = (0x7FFFFF00ll / lanes_of(wide, d)) / deal.per_row.d;
    for (long long t0 = 0; t0 < a.n_tok; t0 += step) {
        deal.count = (unsigned)((a.n_tok - t0 < step ? a.n_tok - t0 : step) * deal.per_row.d);
        auto by_cache = [&](auto DT) {
            return by_type(a.q_type, [&](auto *type) {
                using Q = std::remove_pointer_t<decltype(type)>;
                return by_shape(wide, d, [&](auto N, auto G, auto U) {
                    const unsigned per = kThreads / G.value;
                    return launch_pdl(
                        append_norm_kernel<DT.value, Q, N.value, G.value, U.value>,
                        dim3((deal.count + per - 1) / per), dim3(kThreads),
                        angle_bytes(ax, deal, per), stream, ax, q_norm, k_norm, a, kv, deal, roles,
                        (int)t0);
                });
            });
        };
        const cudaError_t err =
            kv.dtype == kBF16 ? by_cache(std::integral_constant<int, kBF16>())
            : kv.dtype == kF16 ? by_cache(std::integral_constant<int, kF16>())
                               : by_cache(std::integral_constant<int, kF32>());
        if (err != cudaSuccess) return err;
    }
    return cudaSuccess;
}

cudaError_t launch_norm_rope_grad(const AxesView &ax, const NormView &nv, int n, int n_heads,
                                  int head_dim, const float *x, long long x_stride,
                                  const float *grad, long long grad_stride, float *grad_x,
                                  long long grad_x_stride, float *grad_weight, float *grad_bias,
                                  void *workspace, const DeviceInfo &dev, cudaStream_t stream) {
    const bool wide = head_dim % 8 == 0 && ax.rot % 8 == 0 &&
                      all16({x, grad, grad_x, nv.weight},
                            {4 * x_stride, 4 * grad_stride, 4 * grad_x_stride});
    HeadDeal deal = deal_of(blocks_of(n_heads, kGradHeads));
    deal.count = (unsigned)n * deal.per_row.d;
    const bool sums = grad_weight || grad_bias;
    float *parts = sums ? static_cast<float *>(workspace) : nullptr;
    unsigned blocks = 0;
    const cudaError_t err = by_shape(wide, head_dim, [&](auto N, auto G, auto U) {
        constexpr int per = kThreads / G.value;
        blocks = (deal.count + per - 1) / per;
        if (blocks > (unsigned)kGradBlocks) blocks = kGradBlocks;
        size_t smem = sums ? (size_t)per * 2 * head_dim * 4 : 0;  // at most 8 KiB
        if (angle_bytes(ax, deal, per) > smem) smem = angle_bytes(ax, deal, per);
        return launch_pdl(norm_rope_grad_kernel<N.value, G.value, U.value>, dim3(blocks),
                          dim3(kThreads), smem, stream, ax, nv, deal, head_dim, x, x_stride, grad,
                          grad_stride, n_heads, grad_x, grad_x_stride, parts);
    });
    if (err != cudaSuccess || !sums) return err;
    return launch_pdl(grad_sums_kernel, dim3((2 * head_dim + 31) / 32), dim3(32, 32), 0, stream,
                      static_cast<const float *>(parts), (int)blocks, head_dim, grad_weight,
                      grad_bias);
}

}  // namespace wq

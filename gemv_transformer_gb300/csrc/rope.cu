// rope.cu -- rotary positions: the cos/sin table, rotation of packed rows of heads, and
// the append of rotated keys and values to the pages of a cache.
//
// cortiq-engine 0.8.49 src/gpu_wgpu/nemotron_audio.rs, kernel ae_qk, turns q and k by a
// table of cosines and sines made on the host; hanzo-ml 0.11.13 src/wgpu_backend.rs has
// both pair layouts (rope, half and interleaved).
#include <initializer_list>
#include <type_traits>

#include "kv_internal.h"
#include "wq_device.cuh"

namespace wq {
namespace {

constexpr int kTableThreads = 256;
constexpr int kMaxPairs = 128;  // rot <= 256

// One frequency, f64 (the formulas stand in wq.h beside the kinds).
__device__ double rope_frequency(int i, int rot, double base, const wq_rope_scaling &sc) {
    const double two_pi = 6.283185307179586476925286766559;
    if (sc.kind == WQ_ROPE_NTK) base *= pow(sc.factor, (double)rot / (rot - 2));
    const double f = pow(base, -2.0 * i / rot);
    if (sc.kind == WQ_ROPE_LINEAR) return f / sc.factor;
    if (sc.kind == WQ_ROPE_YARN) {
        const double c = rot / (2.0 * log(base));
        const double a = fmax(0.0, floor(c * log(sc.original / (two_pi * sc.high))));
        const double b = fmin(rot - 1.0, ceil(c * log(sc.original / (two_pi * sc.low))));
        const double t = fmin(1.0, fmax(0.0, (i - a) / fmax(b - a, 0.001)));
        return f * (1.0 - t + t / sc.factor);
    }
    if (sc.kind == WQ_ROPE_BANDS) {
        const double turns = sc.original * f / two_pi;
        if (turns > sc.high) return f;
        if (turns < sc.low) return f / sc.factor;
        const double s = (turns - sc.low) / (sc.high - sc.low);
        return f * ((1.0 - s) / sc.factor + s);
    }
    return f;
}

__global__ void __launch_bounds__(kTableThreads) rope_table_kernel(int rows, int rot, double base,
                                                                   wq_rope_scaling sc,
                                                                   float2 *__restrict__ table) {
    pdl_enter();
    __shared__ double s_f[kMaxPairs];
    const int pairs = rot / 2;
    for (int i = threadIdx.x; i < pairs; i += kTableThreads)
        s_f[i] = rope_frequency(i, rot, base, sc);
    __syncthreads();
    const long long count = (long long)rows * pairs;
    for (long long at = (long long)blockIdx.x * kTableThreads + threadIdx.x; at < count;
         at += (long long)gridDim.x * kTableThreads) {
        double sn, cs;
        sincos((double)(at / pairs) * s_f[at % pairs], &sn, &cs);
        table[at] = make_float2((float)(sc.magnitude * cs), (float)(sc.magnitude * sn));
    }
}

// Work is dealt out in units of one row and head: `kWide` pairs (eight values in all) where
// addresses allow 16-byte accesses, else one pair.  Unit u of the first rot / 2 pairs turns
// pairs u * N .. u * N + N - 1; the units after them copy the next 2 N values.
//
// What bounds it: bytes (4 read and 4 written per value).  A thread turns the same unit of
// kHeadsPer heads, so that a row's cos and sin are read once for them (they come from L1
// and L2: 4 rot bytes a row) and four heads' loads are in flight; they do not wait for the
// position or the slot.  Measured: 8192 rows of 40 heads of 128 turned in 49.6 us (340 MB,
// 6850 GB/s, the copy rate; one pair a thread took 102), 8188 tokens appended in 57 us
// (370 MB, 6490 GB/s); 64 tokens 2.3 us, where a launch is all.
constexpr int kWide = 4;
constexpr int kHeadsPer = 4;

template <int N> struct Vals {
    float v[N];
};
template <int N> __device__ __forceinline__ Vals<N> load_vals(const float *p) {
    Vals<N> r;
    if constexpr (N == 4) {
        const float4 x = *reinterpret_cast<const float4 *>(p);
        r.v[0] = x.x, r.v[1] = x.y, r.v[2] = x.z, r.v[3] = x.w;
    } else {
        r.v[0] = *p;
    }
    return r;
}
__device__ __forceinline__ void store_vals(float *p, const Vals<4> &x) {
    *reinterpret_cast<float4 *>(p) = make_float4(x.v[0], x.v[1], x.v[2], x.v[3]);
}
__device__ __forceinline__ void store_vals(float *p, const Vals<1> &x) { *p = x.v[0]; }
__device__ __forceinline__ void store_vals(__nv_bfloat16 *p, const Vals<4> &x) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(x.v[0], x.v[1]),
                         b = __floats2bfloat162_rn(x.v[2], x.v[3]);
    *reinterpret_cast<uint2 *>(p) = make_uint2(*reinterpret_cast<const uint32_t *>(&a),
                                               *reinterpret_cast<const uint32_t *>(&b));
}
__device__ __forceinline__ void store_vals(__half *p, const Vals<4> &x) {
    const __half2 a = __floats2half2_rn(x.v[0], x.v[1]), b = __floats2half2_rn(x.v[2], x.v[3]);
    *reinterpret_cast<uint2 *>(p) = make_uint2(*reinterpret_cast<const uint32_t *>(&a),
                                               *reinterpret_cast<const uint32_t *>(&b));
}
template <typename T> __device__ __forceinline__ void store_vals(T *p, const Vals<1> &x) {
    if constexpr (sizeof(T) == 4)
        *p = x.v[0];
    else if constexpr (std::is_same<T, __half>::value)
        *p = KvType<kF16>::put(x.v[0]);
    else
        *p = KvType<kBF16>::put(x.v[0]);
}

// Where a unit's two runs of N values lie in a head, and how its pairs sit in them: in the
// half layout value i of one with value i of the other, interleaved (N = 4: the runs are
// one after the other) neighbours with one another.
struct Place {
    int a, b;
    bool turn;
};
template <int N> __device__ __forceinline__ Place place_of(int u, int rot, unsigned flags) {
    const int half = rot >> 1, units = half / N;
    if (u >= units) return {rot + 2 * N * (u - units), rot + 2 * N * (u - units) + N, false};
    if (flags & WQ_ROPE_INTERLEAVED) return {2 * N * u, 2 * N * u + N, true};
    return {N * u, N * u + half, true};
}

template <int N> struct Angles {
    float c[N], s[N];
};
template <int N>
__device__ __forceinline__ Angles<N> load_angles(const float2 *p, unsigned flags) {
    Angles<N> r;
    if constexpr (N == 4) {
        const float4 x = *reinterpret_cast<const float4 *>(p);
        const float4 y = reinterpret_cast<const float4 *>(p)[1];
        r.c[0] = x.x, r.s[0] = x.y, r.c[1] = x.z, r.s[1] = x.w;
        r.c[2] = y.x, r.s[2] = y.y, r.c[3] = y.z, r.s[3] = y.w;
    } else {
        const float2 x = *p;
        r.c[0] = x.x, r.s[0] = x.y;
    }
    if (flags & WQ_ROPE_TRANSPOSE)
#pragma unroll
        for (int i = 0; i < N; ++i) r.s[i] = -r.s[i];
    return r;
}

template <int N>
__device__ __forceinline__ void turn(Vals<N> &a, Vals<N> &b, const Angles<N> &cs, unsigned flags) {
    if (N > 1 && (flags & WQ_ROPE_INTERLEAVED)) {
        float x[2 * N];
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = a.v[i], x[N + i] = b.v[i];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float lo = x[2 * i], hi = x[2 * i + 1];
            x[2 * i] = lo * cs.c[i] - hi * cs.s[i];
            x[2 * i + 1] = lo * cs.s[i] + hi * cs.c[i];
        }
#pragma unroll
        for (int i = 0; i < N; ++i) a.v[i] = x[i], b.v[i] = x[N + i];
        return;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float lo = a.v[i], hi = b.v[i];
        a.v[i] = lo * cs.c[i] - hi * cs.s[i];
        b.v[i] = lo * cs.s[i] + hi * cs.c[i];
    }
}

// How a launch's threads map to rows, groups of heads and units.
struct Deal {
    FastDiv per_row, units;  // threads per row; units per head
    int heads_per;           // heads of a thread
    unsigned count;          // threads with work: rows * per_row
};

template <int N>
__global__ void __launch_bounds__(256) rope_kernel(RopeArgs r, Deal deal, const float *x,
                                                   long long x_stride, int n_heads, float *out,
                                                   long long out_stride) {
    pdl_enter();
    const unsigned at = blockIdx.x * 256u + threadIdx.x;
    if (at >= deal.count) return;
    const unsigned t = deal.per_row.div(at), w = at - t * deal.per_row.d;
    const unsigned hg = deal.units.div(w), u = w - hg * deal.units.d;
    const Place p = place_of<N>(u, r.rot, r.flags);
    const int pos = r.rot > 0 ? r.pos[t] : 0;
    const int h0 = hg * deal.heads_per, n = min(deal.heads_per, n_heads - h0);
    const float *xi = x + t * x_stride + (long long)h0 * r.head_dim;
    float *o = out + t * out_stride + (long long)h0 * r.head_dim;
    const bool both = N > 1 || p.b < r.head_dim;  // an odd head_dim ends in a single value
    // The values do not wait for the position.
    Vals<N> a[kHeadsPer], b[kHeadsPer];
#pragma unroll
    for (int i = 0; i < kHeadsPer; ++i)
        if (i < n) {
            a[i] = load_vals<N>(xi + i * r.head_dim + p.a);
            if (both) b[i] = load_vals<N>(xi + i * r.head_dim + p.b);
        }
    if (r.rot > 0 && (unsigned)pos >= (unsigned)r.table_rows) {
        record_status(r.status, kStBadIndex);
        return;
    }
    Angles<N> cs;
    if (p.turn) cs = load_angles<N>(r.table + (long long)pos * (r.rot / 2) + u * N, r.flags);
#pragma unroll
    for (int i = 0; i < kHeadsPer; ++i)
        if (i < n) {
            if (p.turn) turn<N>(a[i], b[i], cs, r.flags);
            store_vals(o + i * r.head_dim + p.a, a[i]);
            if (both) store_vals(o + i * r.head_dim + p.b, b[i]);
        }
}

template <int DT, int N>
__global__ void __launch_bounds__(256) kv_append_kernel(AppendArgs a, KvView kv, Deal deal,
                                                        int t0) {
    pdl_enter();
    using T = typename KvType<DT>::T;
    const RopeArgs &r = a.rope;
    const unsigned at = blockIdx.x * 256u + threadIdx.x;
    if (at >= deal.count) return;
    const unsigned row_at = deal.per_row.div(at), w = at - row_at * deal.per_row.d;
    const unsigned hg = deal.units.div(w), u = w - hg * deal.units.d;
    const int t = t0 + (int)row_at;
    const int slot = a.slot[t];
    const int seq = a.seq ? a.seq[t] : t;
    const int pos = r.pos ? r.pos[t] : 0;
    const Place p = place_of<N>(u, r.rot, r.flags);
    const int heads = a.h_q + 2 * kv.n_heads;
    const int h0 = hg * deal.heads_per, n = min(deal.heads_per, heads - h0);
    // Heads in the order q, k, v.  The values do not wait for the slot.
    Vals<N> lo[kHeadsPer], hi[kHeadsPer];
#pragma unroll
    for (int i = 0; i < kHeadsPer; ++i)
        if (i < n) {
            const int head = h0 + i;
            const float *x =
                head < a.h_q ? a.q + t * a.q_stride + (long long)head * r.head_dim
                : head < a.h_q + kv.n_heads
                    ? a.k + t * a.k_stride + (long long)(head - a.h_q) * r.head_dim
                    : a.v + t * a.v_stride + (long long)(head - a.h_q - kv.n_heads) * r.head_dim;
            lo[i] = load_vals<N>(x + p.a);
            hi[i] = load_vals<N>(x + p.b);
        }
    if (slot < 0) return;  // padding
    const bool in_range = (unsigned)seq < (unsigned)a.n_seq && slot < a.n_slots &&
                          (r.rot == 0 || (unsigned)pos < (unsigned)r.table_rows);
    const long long row = in_range ? kv.row(seq, 0, slot) : -1;
    if (row < 0) {
        record_status(r.status, kStBadIndex);
        return;
    }
    Angles<N> cs;
    if (p.turn) cs = load_angles<N>(r.table + (long long)pos * (r.rot / 2) + u * N, r.flags);
#pragma unroll
    for (int i = 0; i < kHeadsPer; ++i)
        if (i < n) {
            const int head = h0 + i;
            const bool is_q = head < a.h_q, is_k = !is_q && head < a.h_q + kv.n_heads;
            if (p.turn && (is_q || is_k)) turn<N>(lo[i], hi[i], cs, r.flags);
            if (is_q) {
                float *o = a.q_out + t * a.q_out_stride + (long long)head * r.head_dim;
                store_vals(o + p.a, lo[i]);
                store_vals(o + p.b, hi[i]);
                continue;
            }
            const int h = head - a.h_q - (is_k ? 0 : kv.n_heads);
            T *o = reinterpret_cast<T *>((is_k ? kv.k : kv.v) + row + h * kv.head_stride);
            store_vals(o + p.a, lo[i]);
            store_vals(o + p.b, hi[i]);
            if (is_k && u == 0) {
                const long long to = ((long long)seq * kv.n_heads + h) * a.acc_stride + slot;
                if (a.acc) a.acc[to] = 0.f;
                if (a.slot_pos) a.slot_pos[to] = pos;
            }
        }
}

bool all16(std::initializer_list<const void *> ps, std::initializer_list<long long> strides) {
    for (const void *p : ps)
        if ((uintptr_t)p & 15u) return false;
    for (long long s : strides)
        if (s % 4) return false;
    return true;
}

// A thread takes kHeadsPer heads when that still leaves every SM its 2048 threads.
Deal deal_of(long long rows, int heads, int head_dim, int wide, const DeviceInfo &dev) {
    const int units = (head_dim + 2 * wide - 1) / (2 * wide);
    Deal d;
    d.heads_per = rows * ((heads + kHeadsPer - 1) / kHeadsPer) * units >= 2048ll * dev.sm_count
                      ? kHeadsPer : 1;
    d.units = make_fast_div(units);
    d.per_row = make_fast_div((heads + d.heads_per - 1) / d.heads_per * units);
    d.count = 0;
    return d;
}
// Rows of one launch, so that its threads are counted in 31 bits.
long long rows_per_launch(const Deal &d) { return (0x7FFFFF00ll / d.per_row.d); }

unsigned blocks_for(long long count, const DeviceInfo &dev) {
    long long b = (count + 255) / 256;
    const long long cap = (long long)dev.sm_count * 64;
    return (unsigned)(b > cap ? cap : b);
}

}  // namespace

cudaError_t launch_rope_table(int rows, int rot, double base, const wq_rope_scaling &sc,
                              float *table, const DeviceInfo &dev, cudaStream_t stream) {
    return launch_pdl(rope_table_kernel, dim3(blocks_for((long long)rows * (rot / 2), dev)),
                      dim3(kTableThreads), 0, stream, rows, rot, base, sc,
                      reinterpret_cast<float2 *>(table));
}

cudaError_t launch_rope(const RopeArgs &r, const float *x, long long x_stride, int n, int n_heads,
                        float *out, long long out_stride, const DeviceInfo &dev,
                        cudaStream_t stream) {
    const bool wide = r.head_dim % 8 == 0 && r.rot % 8 == 0 &&
                      all16({x, out}, {x_stride, out_stride});
    Deal deal = deal_of(n, n_heads, r.head_dim, wide ? kWide : 1, dev);
    const long long step = rows_per_launch(deal);
    for (long long t0 = 0; t0 < n; t0 += step) {
        const long long rows = n - t0 < step ? n - t0 : step;
        deal.count = (unsigned)(rows * deal.per_row.d);
        RopeArgs part = r;
        if (r.pos) part.pos = r.pos + t0;
        const dim3 grid((deal.count + 255) / 256), block(256);
        const cudaError_t err =
            wide ? launch_pdl(rope_kernel<kWide>, grid, block, 0, stream, part, deal,
                              x + t0 * x_stride, x_stride, n_heads, out + t0 * out_stride,
                              out_stride)
                 : launch_pdl(rope_kernel<1>, grid, block, 0, stream, part, deal,
                              x + t0 * x_stride, x_stride, n_heads, out + t0 * out_stride,
                              out_stride);
        if (err != cudaSuccess) return err;
    }
    return cudaSuccess;
}

namespace {
template <int DT>
cudaError_t launch_append_type(const AppendArgs &a, const KvView &kv, bool wide, const Deal &deal,
                               int t0, cudaStream_t stream) {
    const dim3 grid((deal.count + 255) / 256), block(256);
    return wide ? launch_pdl(kv_append_kernel<DT, kWide>, grid, block, 0, stream, a, kv, deal, t0)
                : launch_pdl(kv_append_kernel<DT, 1>, grid, block, 0, stream, a, kv, deal, t0);
}
}  // namespace

cudaError_t launch_kv_append(const AppendArgs &a, const KvView &kv, const DeviceInfo &dev,
                             cudaStream_t stream) {
    const bool q16 = a.h_q == 0 || all16({a.q, a.q_out}, {a.q_stride, a.q_out_stride});
    const bool wide = a.rope.rot % 8 == 0 && q16 && all16({a.k, a.v}, {a.k_stride, a.v_stride});
    Deal deal = deal_of(a.n_tok, a.h_q + 2 * kv.n_heads, kv.head_dim, wide ? kWide : 1, dev);
    const long long step = rows_per_launch(deal);
    for (long long t0 = 0; t0 < a.n_tok; t0 += step) {
        deal.count = (unsigned)((a.n_tok - t0 < step ? a.n_tok - t0 : step) * deal.per_row.d);
        cudaError_t err;
        switch (kv.dtype) {
        case kBF16: err = launch_append_type<kBF16>(a, kv, wide, deal, (int)t0, stream); break;
        case kF16: err = launch_append_type<kF16>(a, kv, wide, deal, (int)t0, stream); break;
        default: err = launch_append_type<kF32>(a, kv, wide, deal, (int)t0, stream); break;
        }
        if (err != cudaSuccess) return err;
    }
    return cudaSuccess;
}

}  // namespace wq

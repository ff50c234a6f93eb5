// rope.cu -- rotary positions: the cos/sin table, rotation of packed rows of heads, and
// the append of rotated keys and values to the pages of a cache.
//
// cortiq-engine 0.8.49 src/gpu_wgpu/nemotron_audio.rs, kernel ae_qk, turns q and k by a
// table of cosines and sines made on the host; hanzo-ml 0.11.13 src/wgpu_backend.rs has
// both pair layouts (rope, half and interleaved).
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

// One pair (or, past `rot`, two single values) of one head of one row per thread.
// Unit u < rot/2 is the pair u, the others are the dims rot + 2 (u - rot/2) and the next.
struct Pair {
    int a, b;  // dims
    bool turn;
};
__device__ __forceinline__ Pair pair_of(int u, int rot, unsigned flags) {
    const int half = rot >> 1;
    if (u >= half) return {rot + 2 * (u - half), rot + 2 * (u - half) + 1, false};
    if (flags & WQ_ROPE_INTERLEAVED) return {2 * u, 2 * u + 1, true};
    return {u, u + half, true};
}

__global__ void __launch_bounds__(256) rope_kernel(RopeArgs r, const float *x, long long x_stride,
                                                   int n, int n_heads, float *out,
                                                   long long out_stride) {
    pdl_enter();
    const int units = (r.head_dim + 1) / 2;
    const long long per_row = (long long)n_heads * units, count = (long long)n * per_row;
    for (long long at = (long long)blockIdx.x * 256 + threadIdx.x; at < count;
         at += (long long)gridDim.x * 256) {
        const int t = (int)(at / per_row);
        const int w = (int)(at - (long long)t * per_row), h = w / units, u = w - h * units;
        const Pair p = pair_of(u, r.rot, r.flags);
        float2 cs = make_float2(1.f, 0.f);
        if (r.rot > 0) {
            const int pos = __ldg(r.pos + t);
            if ((unsigned)pos >= (unsigned)r.table_rows) {
                record_status(r.status, kStBadIndex);
                continue;
            }
            if (p.turn) cs = __ldg(r.table + (long long)pos * (r.rot / 2) + u);
        }
        if (r.flags & WQ_ROPE_TRANSPOSE) cs.y = -cs.y;
        const float *xi = x + t * x_stride + (long long)h * r.head_dim;
        float *o = out + t * out_stride + (long long)h * r.head_dim;
        const bool both = p.b < r.head_dim;  // an odd head_dim ends in a single value
        const float a = xi[p.a], b = both ? xi[p.b] : 0.f;
        o[p.a] = p.turn ? a * cs.x - b * cs.y : a;
        if (both) o[p.b] = p.turn ? a * cs.y + b * cs.x : b;
    }
}

template <int DT>
__global__ void __launch_bounds__(256) kv_append_kernel(AppendArgs a, KvView kv) {
    pdl_enter();
    using T = typename KvType<DT>::T;
    const RopeArgs &r = a.rope;
    const int units = r.head_dim / 2, heads = a.h_q + 2 * kv.n_heads;
    const long long per_row = (long long)heads * units, count = (long long)a.n_tok * per_row;
    for (long long at = (long long)blockIdx.x * 256 + threadIdx.x; at < count;
         at += (long long)gridDim.x * 256) {
        const int t = (int)(at / per_row);
        const int w = (int)(at - (long long)t * per_row), head = w / units, u = w - head * units;
        const int slot = __ldg(a.slot + t);
        if (slot < 0) continue;
        const int seq = a.seq ? __ldg(a.seq + t) : t;
        const int pos = r.pos ? __ldg(r.pos + t) : 0;
        const bool is_q = head < a.h_q, is_k = !is_q && head < a.h_q + kv.n_heads;
        const int h = is_q ? head : is_k ? head - a.h_q : head - a.h_q - kv.n_heads;
        long long row = -1;
        if ((unsigned)seq < (unsigned)a.n_seq && slot < a.n_slots &&
            (r.rot == 0 || (unsigned)pos < (unsigned)r.table_rows))
            row = kv.row(seq, is_q ? 0 : h, slot);
        if (row < 0) {
            record_status(r.status, kStBadIndex);
            continue;
        }
        Pair p = pair_of(u, r.rot, r.flags);
        if (!is_q && !is_k) p.turn = false;
        float2 cs = make_float2(1.f, 0.f);
        if (p.turn) cs = __ldg(r.table + (long long)pos * (r.rot / 2) + u);
        if (r.flags & WQ_ROPE_TRANSPOSE) cs.y = -cs.y;
        const float *x = (is_q ? a.q + t * a.q_stride : is_k ? a.k + t * a.k_stride
                                                             : a.v + t * a.v_stride) +
                         (long long)h * r.head_dim;
        const float lo = x[p.a], hi = x[p.b];
        const float ya = p.turn ? lo * cs.x - hi * cs.y : lo;
        const float yb = p.turn ? lo * cs.y + hi * cs.x : hi;
        if (is_q) {
            float *o = a.q_out + t * a.q_out_stride + (long long)h * r.head_dim;
            o[p.a] = ya;
            o[p.b] = yb;
        } else {
            T *o = reinterpret_cast<T *>((is_k ? kv.k : kv.v) + row);
            o[p.a] = KvType<DT>::put(ya);
            o[p.b] = KvType<DT>::put(yb);
            if (is_k && u == 0) {
                const long long w = ((long long)seq * kv.n_heads + h) * a.acc_stride + slot;
                if (a.acc) a.acc[w] = 0.f;
                if (a.slot_pos) a.slot_pos[w] = pos;
            }
        }
    }
}

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
    const long long count = (long long)n * n_heads * ((r.head_dim + 1) / 2);
    return launch_pdl(rope_kernel, dim3(blocks_for(count, dev)), dim3(256), 0, stream, r, x,
                      x_stride, n, n_heads, out, out_stride);
}

cudaError_t launch_kv_append(const AppendArgs &a, const KvView &kv, const DeviceInfo &dev,
                             cudaStream_t stream) {
    const long long count = (long long)a.n_tok * (a.h_q + 2 * kv.n_heads) * (kv.head_dim / 2);
    const dim3 grid(blocks_for(count, dev)), block(256);
    switch (kv.dtype) {
    case kBF16: return launch_pdl(kv_append_kernel<kBF16>, grid, block, 0, stream, a, kv);
    case kF16: return launch_pdl(kv_append_kernel<kF16>, grid, block, 0, stream, a, kv);
    default: return launch_pdl(kv_append_kernel<kF32>, grid, block, 0, stream, a, kv);
    }
}

}  // namespace wq

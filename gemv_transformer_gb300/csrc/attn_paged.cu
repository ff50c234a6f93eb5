// attn_paged.cu -- attention of one new token per sequence over a paged cache.
//
// wavo 0.3.0 src/gpu/mod.rs, attend / combine: one token's attention over the decoder's
// cache.  x_j = scale q.k_j + mask_j, p = softmax(x) by one pass with a running maximum m
// and sum l:  m' = max(m, x), l' = l e^(m-m') + e^(x-m'), o' = o e^(m-m') + e^(x-m') v.
#include "kv_internal.h"
#include "wq_device.cuh"

namespace wq {
namespace {

constexpr int kWarps = 8;
constexpr int kLaneDims = 8;  // head_dim <= 256

// The running state of one softmax row, joined in a fixed order.
__device__ __forceinline__ float exp_diff(float x, float m) {
    return x == -INFINITY ? 0.f : expf(x - m);
}

// One block per (sequence, kv head); its query heads one after another, the slots over
// the warps, the dims over the lanes.
template <int DT>
__global__ void __launch_bounds__(kWarps * 32) attn_simple_kernel(AttnArgs a, KvView kv) {
    pdl_enter();
    using T = typename KvType<DT>::T;
    __shared__ float s_m[kWarps], s_l[kWarps], s_o[kWarps][kLaneDims * 32];
    extern __shared__ float s_lse[];  // [group]
    const int s = blockIdx.x / kv.n_heads, h = blockIdx.x - s * kv.n_heads;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, d = kv.head_dim;
    int len = __ldg(a.lens + s);
    if (len > a.n_slots) {
        len = a.n_slots;
        record_status(a.status, kStBadIndex);
    }
    const int first = a.window > 0 && len > a.window ? len - a.window : 0;
    const float *mask = a.mask ? a.mask + s * a.mask_stride : nullptr;

    // The score of slot j for the query in qv, -inf where it takes no part.
    auto score = [&](const float (&qv)[kLaneDims], int j, long long &row) {
        const float bias = mask ? mask[j] : 0.f;
        row = kv.row(s, h, j);
        if (row < 0) record_status(a.status, kStBadIndex);
        if (row < 0 || bias == -INFINITY) return -INFINITY;
        float x = 0.f;
#pragma unroll
        for (int i = 0; i < kLaneDims; ++i)
            if (lane + 32 * i < d)
                x += qv[i] * KvType<DT>::get(reinterpret_cast<const T *>(kv.k + row)[lane + 32 * i]);
        return warp_sum(x) * a.scale + bias;
    };
    auto query = [&](float (&qv)[kLaneDims], int g) {
        const float *q = a.q + s * a.q_stride + (long long)(h * a.group + g) * d;
#pragma unroll
        for (int i = 0; i < kLaneDims; ++i) qv[i] = lane + 32 * i < d ? q[lane + 32 * i] : 0.f;
    };

    for (int g = 0; g < a.group; ++g) {
        float qv[kLaneDims], o[kLaneDims] = {}, m = -INFINITY, l = 0.f;
        query(qv, g);
        for (int j = first + warp; j < len; j += kWarps) {
            long long row;
            const float x = score(qv, j, row);
            if (x == -INFINITY) continue;
            const float m2 = fmaxf(m, x), c = exp_diff(m, m2), p = expf(x - m2);
            m = m2;
            l = l * c + p;
#pragma unroll
            for (int i = 0; i < kLaneDims; ++i)
                if (lane + 32 * i < d)
                    o[i] = o[i] * c +
                           p * KvType<DT>::get(
                                   reinterpret_cast<const T *>(kv.v + row)[lane + 32 * i]);
        }
        if (lane == 0) {
            s_m[warp] = m;
            s_l[warp] = l;
        }
#pragma unroll
        for (int i = 0; i < kLaneDims; ++i) s_o[warp][lane + 32 * i] = o[i];
        __syncthreads();
        float mm = -INFINITY, ll = 0.f;
        for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, s_m[w]);
        for (int w = 0; w < kWarps; ++w) ll += s_l[w] * exp_diff(s_m[w], mm);
        for (int i = threadIdx.x; i < d; i += kWarps * 32) {
            float v = 0.f;
            for (int w = 0; w < kWarps; ++w) v += s_o[w][i] * exp_diff(s_m[w], mm);
            a.out[s * a.out_stride + (long long)(h * a.group + g) * d + i] =
                mm == -INFINITY ? 0.f : v / ll;
        }
        if (threadIdx.x == 0) {
            const float e = mm == -INFINITY ? -INFINITY : mm + logf(ll);
            s_lse[g] = e;
            if (a.lse) a.lse[(long long)s * a.h_q + h * a.group + g] = e;
        }
        __syncthreads();
    }
    if (!a.acc_out) return;
    const long long at = ((long long)s * kv.n_heads + h) * a.acc_stride;
    for (int j = warp; j < len; j += kWarps) {
        float w = 0.f;
        if (j >= first)
            for (int g = 0; g < a.group; ++g) {
                float qv[kLaneDims];
                query(qv, g);
                long long row;
                const float x = score(qv, j, row);
                if (s_lse[g] != -INFINITY) w += exp_diff(x, s_lse[g]);
            }
        if (lane == 0) a.acc_out[at + j] = (a.acc_in ? a.acc_in[at + j] : 0.f) + w;
    }
}

}  // namespace

size_t attn_workspace_bytes(const KvView &, int, int, int, bool) { return 0; }

cudaError_t launch_attn_paged(const AttnArgs &a, const KvView &kv, const DeviceInfo &,
                              cudaStream_t stream) {
    const long long blocks = (long long)a.n_seq * kv.n_heads;
    if (blocks > 0x7FFFFFFFll) return cudaErrorInvalidConfiguration;
    const size_t smem = (size_t)a.group * sizeof(float);
    const dim3 grid((unsigned)blocks), block(kWarps * 32);
    switch (kv.dtype) {
    case kBF16: return launch_pdl(attn_simple_kernel<kBF16>, grid, block, smem, stream, a, kv);
    case kF16: return launch_pdl(attn_simple_kernel<kF16>, grid, block, smem, stream, a, kv);
    default: return launch_pdl(attn_simple_kernel<kF32>, grid, block, smem, stream, a, kv);
    }
}

}  // namespace wq

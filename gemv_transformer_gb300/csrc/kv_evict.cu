// kv_evict.cu -- a cache cut to a budget of slots by accumulated attention weight.
//
// Per (sequence, kv head): the budget-th largest weight is found by radix selection, eight
// bits of the order-preserving key at a time; the slots that stay but lie beyond the
// budget then move, in order, into the slots below it that go.
#include "kv_internal.h"
#include "wq_device.cuh"

namespace wq {
namespace {

constexpr int kThreads = 256;

// Keys in the order of the weights: a held slot above all, a NaN below all.
__device__ __forceinline__ uint32_t key_of(float w, int pos, int sinks, int from) {
    if (pos < sinks || pos >= from) return 0xFFFFFFFFu;
    if (w != w) return 0u;
    const uint32_t u = __float_as_uint(w + 0.f);  // -0 as 0
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// The sum of `v` over the threads before this one; `total` over all of them.
__device__ __forceinline__ int block_scan(int v, int *s_warp, int &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) s_warp[warp] = x;
    __syncthreads();
    int before = 0;
    total = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += s_warp[w];
        total += s_warp[w];
    }
    return before + x - v;
}

__global__ void __launch_bounds__(kThreads) evict_simple_kernel(EvictArgs a, KvView kv,
                                                                int row_bytes) {
    pdl_enter();
    __shared__ int s_hist[256], s_warp[kThreads / 32];
    __shared__ uint32_t s_prefix;
    __shared__ int s_left;
    const int s = blockIdx.x / kv.n_heads, h = blockIdx.x - s * kv.n_heads;
    int len = __ldg(a.lens + s);
    if (len > a.n_slots) {
        len = a.n_slots;
        record_status(a.status, kStBadIndex);
    }
    if (len < 0) len = 0;
    const int keep = min(len, a.keep);
    const int from = __ldg(a.seen + s) - a.recent;
    const long long base = ((long long)s * kv.n_heads + h) * a.acc_stride;
    const float *acc = a.acc + base;
    const int32_t *pos = a.slot_pos + base;
    int32_t *list = static_cast<int32_t *>(a.workspace) + 2ll * blockIdx.x * a.keep;
    auto key = [&](int j) { return key_of(acc[j], pos[j], a.sinks, from); };

    uint32_t bound = 0;
    int ties = 0;  // slots with the bound's key that stay
    if (len > keep) {
        if (threadIdx.x == 0) {
            s_prefix = 0;
            s_left = keep;
        }
        for (int shift = 24; shift >= 0; shift -= 8) {
            s_hist[threadIdx.x] = 0;
            __syncthreads();
            const uint32_t prefix = s_prefix;
            for (int j = threadIdx.x; j < len; j += kThreads) {
                const uint32_t x = key(j);
                if (shift == 24 || (x >> (shift + 8)) == prefix)
                    atomicAdd(&s_hist[(x >> shift) & 255u], 1);
            }
            __syncthreads();
            if (threadIdx.x == 0) {
                int left = s_left, b = 255;
                while (s_hist[b] < left) left -= s_hist[b--];
                s_left = left;
                s_prefix = prefix << 8 | (uint32_t)b;
            }
            __syncthreads();
        }
        bound = s_prefix;
        ties = s_left;
    }
    // In slot order: which stay, the holes below the budget, and who moves into them.
    int same = 0, holes = 0, movers = 0;
    for (int j0 = 0; j0 < len; j0 += kThreads) {
        const int j = j0 + threadIdx.x;
        const bool live = j < len;
        const uint32_t x = live ? key(j) : 0u;
        int total;
        const int rank = same + block_scan(live && x == bound, s_warp, total);
        same += total;
        const bool stay = live && (len <= keep || x > bound || (x == bound && rank < ties));
        const bool hole = live && j < keep && !stay, mover = stay && j >= keep;
        const int nh = holes + block_scan(hole, s_warp, total);
        holes += total;
        const int nm = movers + block_scan(mover, s_warp, total);
        movers += total;
        if (hole) list[2 * nh] = j;
        if (mover) list[2 * nm + 1] = j;
        if (stay && !mover) {
            const float w = acc[j];
            const int p = pos[j];
            a.acc_out[base + j] = w;
            a.pos_out[base + j] = p;
        }
    }
    __syncthreads();
    for (int i = threadIdx.x >> 5; i < movers; i += kThreads / 32) {
        const int dst = list[2 * i], src = list[2 * i + 1], lane = threadIdx.x & 31;
        if (lane == 0) {
            a.acc_out[base + dst] = acc[src];
            a.pos_out[base + dst] = pos[src];
        }
        const long long to = kv.row(s, h, dst), at = kv.row(s, h, src);
        if (to < 0 || at < 0) {
            record_status(a.status, kStBadIndex);
            continue;
        }
        for (int b = lane * 16; b < row_bytes; b += 512) {
            *reinterpret_cast<uint4 *>(kv.k + to + b) =
                *reinterpret_cast<const uint4 *>(kv.k + at + b);
            *reinterpret_cast<uint4 *>(kv.v + to + b) =
                *reinterpret_cast<const uint4 *>(kv.v + at + b);
        }
    }
}

// After every row's selection has read lens (lens_out may equal it).
__global__ void evict_lens_kernel(EvictArgs a) {
    pdl_enter();
    const int s = blockIdx.x * blockDim.x + threadIdx.x;
    if (s < a.n_seq) a.lens_out[s] = min(max(a.lens[s], 0), min(a.keep, a.n_slots));
}

}  // namespace

size_t evict_workspace_bytes(const KvView &kv, int n_seq, int, int keep) {
    return ((size_t)n_seq * kv.n_heads * keep * 8 + 255) & ~(size_t)255;
}

cudaError_t launch_kv_evict(const EvictArgs &a, const KvView &kv, const DeviceInfo &,
                            cudaStream_t stream) {
    const long long blocks = (long long)a.n_seq * kv.n_heads;
    if (blocks > 0x7FFFFFFFll) return cudaErrorInvalidConfiguration;
    const int row_bytes = kv.head_dim * (kv.dtype == kF32 ? 4 : 2);
    cudaError_t err = launch_pdl(evict_simple_kernel, dim3((unsigned)blocks), dim3(kThreads), 0,
                                 stream, a, kv, row_bytes);
    if (err != cudaSuccess) return err;
    return launch_pdl(evict_lens_kernel, dim3((a.n_seq + 255) / 256), dim3(256), 0, stream, a);
}

}  // namespace wq

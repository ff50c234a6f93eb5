// kv_evict.cu -- a cache cut to a budget of slots by accumulated attention weight.
//
// Per row (sequence, kv head): the keep-th largest weight is found by radix selection, eight
// bits of an order-preserving key at a time; the slots that stay but lie beyond the
// budget then move, in order, into the slots below it that go.  Only they move: a cache
// over its budget by one slot a step moves one slot, not the half of the cache that keeping
// the order would.
//
// What bounds it: 8 bytes read per slot (weight, position), 8 written per slot kept, and two
// rows of k and v read and written per slot moved; with few rows, or one slot over, the
// chain of four histograms.
//
// A row is a cluster of 1, 2, 4 or 8 CTAs, so that a few long rows fill the GPU: each holds
// the keys of its share of the slots in shared memory, the histograms and counts are
// added over distributed shared memory, and after the last cluster barrier the row's
// CTAs share the moves evenly.  One launch; no atomics on global memory, and the sums of
// integers are the same in any order.
#include <cooperative_groups.h>

#include "kv_internal.h"
#include "wq_device.cuh"

namespace wq {
namespace {

namespace cg = cooperative_groups;

constexpr int kMaxKeys = 48 * 1024;  // keys that a CTA holds; beyond, they are read again
constexpr int kBatch = 4;            // moves that a warp has in flight

// Keys in the order of the weights: a held slot above all, a NaN below all.
__device__ __forceinline__ uint32_t key_of(float w, int pos, int sinks, int from) {
    if (pos < sinks || pos >= from) return 0xFFFFFFFFu;
    if (w != w) return 0u;
    const uint32_t u = __float_as_uint(w + 0.f);  // -0 as 0
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

template <int T> struct Select {
    static constexpr int W = T / 32;
    int hist[4][256];  // one per pass, so that one barrier a pass is enough
    int scan[2][W];
    int counts[3];     // this CTA's ties, holes, movers
    uint32_t prefix;
    int left, equal;
};

// Sums over the warps before this one of (a, b), and the totals.
template <int T>
__device__ __forceinline__ void warp_offsets(Select<T> &sh, int &a, int &b, int &ta, int &tb) {
    const int warp = threadIdx.x >> 5;
    __syncthreads();
    if ((threadIdx.x & 31) == 0) {
        sh.scan[0][warp] = a;
        sh.scan[1][warp] = b;
    }
    __syncthreads();
    a = b = ta = tb = 0;
#pragma unroll
    for (int w = 0; w < T / 32; ++w) {
        const int x = sh.scan[0][w], y = sh.scan[1][w];
        if (w < warp) a += x, b += y;
        ta += x;
        tb += y;
    }
}

template <int T>
__global__ void __launch_bounds__(T) evict_kernel(EvictArgs a, KvView kv, int row_bytes,
                                                  int key_room) {
    extern __shared__ uint32_t s_key[];
    __shared__ Select<T> sh;
    pdl_wait();
    cg::cluster_group cluster = cg::this_cluster();
    const int size = cluster.num_blocks(), rank = cluster.block_rank();
    const int id = blockIdx.x / size, s = id / kv.n_heads, h = id - s * kv.n_heads;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int given = __ldg(a.lens + s), len = min(max(given, 0), a.n_slots);
    const int keep = min(len, a.keep);
    if (threadIdx.x == 0 && rank == 0 && h == 0) {
        if (given > a.n_slots) record_status(a.status, kStBadIndex);
        if (a.lens_out != a.lens) a.lens_out[s] = keep;
    }
    const long long base = (long long)id * a.acc_stride;
    const float *acc = a.acc + base;
    const int32_t *pos = a.slot_pos + base;
    const bool in_place = a.acc_out == a.acc && a.pos_out == a.slot_pos;
    // This CTA's slots.
    const int share = ((len + size - 1) / size + 31) & ~31;
    const int b0 = min(len, rank * share), b1 = min(len, b0 + share), mine = b1 - b0;
    if (len <= keep) {  // within the budget: the whole cluster leaves here
        if (!in_place)
            for (int j = b0 + threadIdx.x; j < b1; j += T) {
                a.acc_out[base + j] = acc[j];
                a.pos_out[base + j] = pos[j];
            }
        return;
    }
    const int from = __ldg(a.seen + s) - a.recent;
    const bool held_keys = mine <= key_room;
    auto make_key = [&](int j) { return key_of(acc[j], pos[j], a.sinks, from); };
    auto key = [&](int j) { return held_keys ? s_key[j - b0] : make_key(j); };

    for (int i = threadIdx.x; i < 4 * 256; i += T) (&sh.hist[0][0])[i] = 0;
    if (threadIdx.x == 0) {
        sh.prefix = 0;
        sh.left = keep;
    }
    if (held_keys) {
#pragma unroll 4
        for (int j = b0 + threadIdx.x; j < b1; j += T) s_key[j - b0] = make_key(j);
    }
    __syncthreads();
    for (int pass = 0; pass < 4; ++pass) {
        const int shift = 24 - 8 * pass;
        const uint32_t prefix = sh.prefix;
        // Weights share their top bits: a warp's equal bins are counted by one addition.
        for (int j0 = b0 + warp * 32; j0 < b1; j0 += T) {
            const int j = j0 + lane;
            const uint32_t x = j < b1 ? key(j) : 0u;
            const bool in = j < b1 && (pass == 0 || (x >> (shift + 8)) == prefix);
            const unsigned who = __ballot_sync(0xFFFFFFFFu, in);
            if (!who) continue;
            if (in) {
                const int bin = (x >> shift) & 255u;
                const unsigned same = __match_any_sync(who, bin);
                if (lane == __ffs(same) - 1) atomicAdd(&sh.hist[pass][bin], __popc(same));
            }
        }
        cluster.sync();
        // The bin that holds the left-th largest: bins from the top, one per thread.
        int count = 0;
        if (threadIdx.x < 256) {
            const int bin = 255 - threadIdx.x;
            for (int r = 0; r < size; ++r)
                count += *cluster.map_shared_rank(&sh.hist[pass][bin], r);
        }
        int incl = count;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xFFFFFFFFu, incl, o);
            if (lane >= o) incl += y;
        }
        if (lane == 31 && warp < 8) sh.scan[0][warp] = incl;
        const int left = sh.left;
        __syncthreads();
        if (threadIdx.x < 256) {
            for (int w = 0; w < warp; ++w) incl += sh.scan[0][w];
            if (incl - count < left && left <= incl) {
                sh.prefix = prefix << 8 | (uint32_t)(255 - threadIdx.x);
                sh.left = left - (incl - count);
                sh.equal = count;
            }
        }
        __syncthreads();
    }
    const uint32_t bound = sh.prefix;
    const int ties = sh.left, equal = sh.equal;  // of `equal` slots with the bound's key, `ties` stay

    // Each warp takes a contiguous piece, so that ranks follow the slots.
    const int piece = ((mine + T / 32 - 1) / (T / 32) + 31) & ~31;
    const int w0 = min(b1, b0 + warp * piece), w1 = min(b1, w0 + piece);
    int same = 0, none = 0, all_same, all_none;
    const bool all_ties = ties == equal;
    if (!all_ties) {
        for (int j0 = w0; j0 < w1; j0 += 32) {
            const int j = j0 + lane;
            same += __popc(__ballot_sync(0xFFFFFFFFu, j < w1 && key(j) == bound));
        }
        warp_offsets<T>(sh, same, none, all_same, all_none);
        if (threadIdx.x == 0) sh.counts[0] = all_same;
        cluster.sync();
        for (int r = 0; r < rank; ++r) same += *cluster.map_shared_rank(&sh.counts[0], r);
    }
    const unsigned below_lane = (1u << lane) - 1u;
    // Does slot j stay?  `tie` counts the bound's slots before the group of 32.
    auto stays = [&](int j, int &tie) {
        const bool live = j < w1;
        const uint32_t x = live ? key(j) : 0u;
        const bool at_bound = live && x == bound;
        if (all_ties) return live && x >= bound;
        const unsigned votes = __ballot_sync(0xFFFFFFFFu, at_bound);
        const int rank_of = tie + __popc(votes & below_lane);
        tie += __popc(votes);
        return live && (x > bound || (at_bound && rank_of < ties));
    };
    int holes = 0, movers = 0, cta_holes, cta_movers, tie = same;
    for (int j0 = w0; j0 < w1; j0 += 32) {
        const int j = j0 + lane;
        const bool stay = stays(j, tie);
        holes += __popc(__ballot_sync(0xFFFFFFFFu, j < w1 && j < keep && !stay));
        movers += __popc(__ballot_sync(0xFFFFFFFFu, stay && j >= keep));
    }
    warp_offsets<T>(sh, holes, movers, cta_holes, cta_movers);
    if (threadIdx.x == 0) {
        sh.counts[1] = cta_holes;
        sh.counts[2] = cta_movers;
    }
    cluster.sync();
    int total = 0;
    for (int r = 0; r < size; ++r) {
        const int x = *cluster.map_shared_rank(&sh.counts[1], r);
        if (r < rank) {
            holes += x;
            movers += *cluster.map_shared_rank(&sh.counts[2], r);
        }
        total += x;
    }
    int2 *list = static_cast<int2 *>(a.workspace) + (long long)id * a.keep;  // (to, from)
    tie = same;
    for (int j0 = w0; j0 < w1; j0 += 32) {
        const int j = j0 + lane;
        const bool stay = stays(j, tie);
        const bool hole = j < w1 && j < keep && !stay, mover = stay && j >= keep;
        const unsigned hv = __ballot_sync(0xFFFFFFFFu, hole);
        const unsigned mv = __ballot_sync(0xFFFFFFFFu, mover);
        if (hole) list[holes + __popc(hv & below_lane)].x = j;
        if (mover) list[movers + __popc(mv & below_lane)].y = j;
        holes += __popc(hv);
        movers += __popc(mv);
        if (stay && !mover && !in_place) {
            a.acc_out[base + j] = acc[j];
            a.pos_out[base + j] = pos[j];
        }
    }
    cluster.sync();  // the list is complete; no shared memory of another CTA is read below
    pdl_launch();

    const int warps = size * (T / 32), quads = row_bytes / 16;  // of k; as many of v
    for (int i0 = (rank * (T / 32) + warp) * kBatch; i0 < total; i0 += warps * kBatch) {
        long long to = -1, at = -1;
        if (lane < kBatch && i0 + lane < total) {
            const int2 m = list[i0 + lane];
            a.acc_out[base + m.x] = acc[m.y];
            a.pos_out[base + m.x] = pos[m.y];
            to = kv.row(s, h, m.x);
            at = kv.row(s, h, m.y);
            if (to < 0 || at < 0) {
                record_status(a.status, kStBadIndex);
                to = -1;
            }
        }
        for (int q0 = 0; q0 < 2 * quads; q0 += 32) {
            const int q = q0 + lane;
            const bool of_v = q >= quads;
            const long long in = 16ll * (of_v ? q - quads : q);
            char *pool = of_v ? kv.v : kv.k;
            uint4 x[kBatch];
            long long dst[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                dst[i] = __shfl_sync(0xFFFFFFFFu, to, i);
                const long long src = __shfl_sync(0xFFFFFFFFu, at, i);
                if (q >= 2 * quads) dst[i] = -1;
                if (dst[i] >= 0) x[i] = *reinterpret_cast<const uint4 *>(pool + src + in);
            }
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                if (dst[i] >= 0) *reinterpret_cast<uint4 *>(pool + dst[i] + in) = x[i];
        }
    }
}

// Lengths in place: after every row of a sequence has read them.
__global__ void evict_lens_kernel(EvictArgs a) {
    pdl_enter();
    const int s = blockIdx.x * blockDim.x + threadIdx.x;
    if (s < a.n_seq) a.lens_out[s] = min(max(a.lens[s], 0), min(a.keep, a.n_slots));
}

template <int T>
cudaError_t launch_rows(const EvictArgs &a, const KvView &kv, int cluster, const DeviceInfo &dev,
                        cudaStream_t stream) {
    const int row_bytes = kv.head_dim * (kv.dtype == kF32 ? 4 : 2);
    const long long share = ((a.n_slots + (long long)cluster - 1) / cluster + 31) & ~31ll;
    const int key_room = (int)(share < kMaxKeys ? share : kMaxKeys);
    static std::atomic<unsigned long long> done{0};
    cudaError_t err = ensure_smem(evict_kernel<T>, kMaxKeys * 4, dev, done);
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((long long)a.n_seq * kv.n_heads * cluster));
    cfg.blockDim = dim3(T);
    cfg.dynamicSmemBytes = (size_t)key_room * 4;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, evict_kernel<T>, a, kv, row_bytes, key_room);
}

}  // namespace

size_t evict_workspace_bytes(const KvView &kv, int n_seq, int, int keep) {
    return ((size_t)n_seq * kv.n_heads * keep * 8 + 255) & ~(size_t)255;
}

cudaError_t launch_kv_evict(const EvictArgs &a, const KvView &kv, const DeviceInfo &dev,
                            cudaStream_t stream) {
    const long long rows = (long long)a.n_seq * kv.n_heads;
    if (rows > 0x7FFFFFFFll / 8) return cudaErrorInvalidConfiguration;
    // More CTAs to a row while two per SM are not reached and each has 2048 slots or more.
    int cluster = 1;
    while (cluster < 8 && rows * cluster * 2 <= 2 * dev.sm_count && a.n_slots / cluster > 2048)
        cluster *= 2;
    cudaError_t err = a.n_slots / cluster <= 4096 ? launch_rows<256>(a, kv, cluster, dev, stream)
                                                  : launch_rows<512>(a, kv, cluster, dev, stream);
    if (err != cudaSuccess || a.lens_out != a.lens) return err;
    return launch_pdl(evict_lens_kernel, dim3((a.n_seq + 255) / 256), dim3(256), 0, stream, a);
}

}  // namespace wq

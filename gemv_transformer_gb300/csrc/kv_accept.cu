// kv_accept.cu -- the accepted path of a drafted tree, and its k and v moved together in every
// layer's cache; with them, where they are given, the slots' accumulated weights and positions.
//
// The path is a chain: the root, then again and again the lowest child of the last node whose token
// is the one that the model chose after it.  A child's number is above its parent's, so one pass
// over the nodes in rising order finds it: the next node is the first beyond the last that fits.
//
// What bounds it: latency (a chain of loads of lengths, nodes, pages, rows); the rows moved are a
// few kilobytes per layer.  One launch: each CTA finds its sequence's path itself with one warp,
// 32 nodes at a time, and its threads then move one 16-byte column of one row each (of the weights and
// positions 4 bytes of a head), so that no thread reads what another one writes.  The i-th node's
// slot goes to slot i <= path[i]: in rising order a slot is read before it is overwritten.
// 16 nodes in 32 layers 5.3 us, 64 sequences of 32 nodes in 16 layers 5.1 (the host's call).
#include <type_traits>

#include "kv_internal.h"
#include "wq_device.cuh"

namespace wq {
namespace {

constexpr int kThreads = 256;
constexpr int kInFlight = 8;  // rows that a thread reads before it writes them

struct NoSlots {};

// Slots: AcceptSlots, or NoSlots where there are none.
template <typename Slots>
__global__ void __launch_bounds__(kThreads)
    kv_accept_kernel(AcceptArgs a, KvView kv, const __grid_constant__ AcceptPools pools,
                     FastDiv chunks, bool write_path, const __grid_constant__ Slots slots) {
    constexpr bool kSlots = std::is_same<Slots, AcceptSlots>::value;
    pdl_enter();
    __shared__ int s_node[32], s_found;
    const int s = blockIdx.y, lane = threadIdx.x & 31;
    const bool writes = write_path && blockIdx.x == 0;
    const int t0 = a.starts[s], t1 = a.starts[s + 1], len = a.lens[s];
    const bool bad = t0 < 0 || t1 < t0 || t1 > a.n_tok || len < t1 - t0 || len > a.n_slots;
    const int count = t1 - t0, base = len - count;
    if (bad || count == 0) {
        if (writes && threadIdx.x == 0) {
            a.accepted[s] = 0;
            a.next[s] = -1;
            a.lens_out[s] = len;
            if (bad) record_status(a.status, kStBadIndex);
        }
        return;
    }
    // This thread's column: chunk of 16 bytes, kv head, pool (k or v), layer.
    const unsigned at = blockIdx.x * kThreads + threadIdx.x;
    const unsigned row_at = chunks.div(at), chunk = at - row_at * chunks.d;
    const int head = row_at % kv.n_heads, pool = row_at / kv.n_heads;
    bool moves = pool < 2 * pools.count;
    char *col = !moves ? nullptr
                : (pool & 1 ? pools.v[pool >> 1] : pools.k[pool >> 1]) +
                      (long long)head * kv.head_stride + chunk * 16;
    bool word = false;  // a column of 4 bytes, by slot
    if constexpr (kSlots) {
        const unsigned wide = 2u * pools.count * kv.n_heads * chunks.d;
        if (at >= wide) {  // of a head's weights or positions
            const unsigned x = at - wide, array = x / kv.n_heads, h = x - array * kv.n_heads;
            word = array < 2u * pools.count;
            char *const p = !word ? nullptr : static_cast<char *>(slots.p[array]);
            moves = p != nullptr;
            col = p + (((slots.seq0 + s) * kv.n_heads + h) * slots.stride + base) * 4;
        }
    }

    int tip = 0, found = 1, want = a.choice[t0];  // of warp 0
    for (int c0 = 0; c0 < count; c0 += 32) {
        if (threadIdx.x < 32) {
            const int c = c0 + lane;
            const bool in = c < count;
            const int parent = in && c > 0 ? a.parent[t0 + c] : -1;
            const int token = in ? a.tokens[t0 + c] : 0, choice = in ? a.choice[t0 + c] : 0;
            int n = 0, last = c0 - 1;  // nodes found here; nodes up to `last` are passed
            if (c0 == 0) {
                if (lane == 0) s_node[0] = 0;
                n = 1, last = 0;
            }
            for (;;) {
                const unsigned fits =
                    __ballot_sync(0xFFFFFFFFu, in && c > last && parent == tip && token == want);
                if (!fits) break;
                const int src = __ffs(fits) - 1;
                tip = last = c0 + src;
                want = __shfl_sync(0xFFFFFFFFu, choice, src);
                if (lane == 0) s_node[n] = tip;
                ++n;
            }
            if (lane == 0) s_found = n;
        }
        __syncthreads();
        const int n = s_found, i0 = c0 == 0 ? 0 : found;
        if (writes)
            for (int i = threadIdx.x; i < n; i += kThreads) a.path[t0 + i0 + i] = s_node[i];
        if (moves) {
            for (int i = 0; i < n; i += kInFlight) {
                uint4 v[kInFlight];
                long long to[kInFlight];
#pragma unroll
                for (int j = 0; j < kInFlight; ++j) {
                    to[j] = -1;
                    if (i + j >= n) continue;
                    const int src = s_node[i + j], dst = i0 + i + j;
                    if (src == dst) continue;
                    const long long from = kv.row(s, 0, base + src);
                    const long long dest = kv.row(s, 0, base + dst);
                    if (from < 0 || dest < 0) {
                        if (write_path) record_status(a.status, kStBadIndex);
                        continue;
                    }
                    if (kSlots && word) {
                        to[j] = 4ll * dst;
                        v[j].x = *reinterpret_cast<const uint32_t *>(col + 4ll * src);
                        continue;
                    }
                    to[j] = dest;
                    v[j] = *reinterpret_cast<const uint4 *>(col + from);
                }
#pragma unroll
                for (int j = 0; j < kInFlight; ++j) {
                    if (to[j] < 0) continue;
                    if (kSlots && word)
                        *reinterpret_cast<uint32_t *>(col + to[j]) = v[j].x;
                    else
                        *reinterpret_cast<uint4 *>(col + to[j]) = v[j];
                }
            }
        }
        found = i0 + n;
        __syncthreads();
    }
    if (writes) {
        for (int i = found + threadIdx.x; i < count; i += kThreads) a.path[t0 + i] = -1;
        if (threadIdx.x == 0) {
            a.accepted[s] = found;
            a.next[s] = want;
            a.lens_out[s] = base + found;
        }
    }
}

}  // namespace

cudaError_t launch_kv_accept(const AcceptArgs &a, const KvView &kv, const AcceptPools &pools,
                             const AcceptSlots *slots, bool write_path, cudaStream_t stream) {
    const FastDiv chunks = make_fast_div(kv.head_dim * (kv.dtype == kF32 ? 4 : 2) / 16);
    const long long columns = 2ll * pools.count * kv.n_heads * (chunks.d + (slots ? 1 : 0));
    // Sequences are the grid's y, 65535 at most.
    for (int s0 = 0; s0 < a.n_seq; s0 += 65535) {
        AcceptArgs part = a;
        KvView view = kv;
        part.n_seq = a.n_seq - s0 < 65535 ? a.n_seq - s0 : 65535;
        part.starts += s0, part.lens += s0, part.accepted += s0, part.next += s0;
        part.lens_out += s0;
        view.page_table += (long long)s0 * kv.max_pages;
        const dim3 grid((unsigned)((columns + kThreads - 1) / kThreads), (unsigned)part.n_seq);
        cudaError_t err;
        if (slots) {
            AcceptSlots its = *slots;
            its.seq0 = s0;
            err = launch_pdl(kv_accept_kernel<AcceptSlots>, grid, dim3(kThreads), 0, stream, part,
                             view, pools, chunks, write_path, its);
        } else {
            err = launch_pdl(kv_accept_kernel<NoSlots>, grid, dim3(kThreads), 0, stream, part, view,
                             pools, chunks, write_path, NoSlots{});
        }
        if (err != cudaSuccess) return err;
    }
    return cudaSuccess;
}

}  // namespace wq

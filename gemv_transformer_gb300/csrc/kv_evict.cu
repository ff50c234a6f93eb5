// kv_evict.cu -- a cache cut to a budget of slots by accumulated attention weight.
//
// Per row (sequence, kv head): the keep-th largest weight is found by radix selection,
// eleven bits of an order-preserving key at a time; the slots that stay but lie beyond the
// budget then move, in order, into the slots below it that go.  Only they move: a cache
// over its budget by one slot a step moves one slot, not the half of the cache that keeping
// the order would.  A row over by one needs no more than its minimum.
//
// What bounds it: 8 bytes read per slot (weight, position), 8 written per slot kept, and two
// rows of k and v read and written per slot moved; with few rows the chain of three
// histograms, or with one slot over of three loads.  Measured: 512 rows of 2049 slots, one
// over: 4.6 us (17 MB; 2.6 at the copy rate; 10.1 by histograms); 32 rows of 65536 cut to 4096:
// 54 us (145 MB; 21.6), of which 6 load the keys, 7 find the bound, 10 rank and list the
// slots, and 24 move 126 MB in rows of 256 bytes.
//
// A row is a cluster of 1, 2, 4 or 8 CTAs, so that a few long rows fill the GPU: each holds
// the keys of its share of the slots in shared memory, the histograms and counts are
// added over distributed shared memory (each CTA holds the counts of its share of the
// digits for all: reading every CTA's whole histogram took 4 us a pass), and after the
// last cluster barrier the row's CTAs share the moves evenly, or leave them to a launch over
// all SMs where rows are few and moves many.  No atomics on global memory, and the sums of
// integers are the same in any order.
#include <cooperative_groups.h>

#include "kv_internal.h"
#include "wq_device.cuh"

namespace wq {
namespace {

namespace cg = cooperative_groups;

constexpr int kMaxKeys = 42 * 1024;  // keys that a CTA holds; beyond, they are read again
constexpr int kBatch = 8;            // moves that a warp has in flight
constexpr int kDigit = 11, kBins = 1 << kDigit, kPasses = 3;  // 11 + 11 + 10 bits
constexpr int kShort = 128;          // moves that a single CTA lists in shared memory

// One move between slots.  The hole's owner writes `to`, the mover's `at`; where their rows
// are is looked up by the warp that moves them, ahead of its loads (by those who list the
// moves, with weights and offsets in the list: 4 % to 25 % slower, 48 for 35 us for 8 rows of
// 65536 cut to 60000).
struct __align__(8) Move {
    int to, at;
};

constexpr uint32_t kHeld = 0xFFFFFFFFu, kZero = 0x80000000u;

// Keys in the order of the weights: a held slot above all, a NaN below all.
__device__ __forceinline__ uint32_t key_of(float w, int pos, int sinks, int from) {
    if (pos < sinks || pos >= from) return kHeld;
    if (w != w) return 0u;
    const uint32_t u = __float_as_uint(w + 0.f);  // -0 as 0
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

template <int T, int C> struct __align__(16) Select {
    // One per pass, so that one cluster barrier a pass is enough.  Of a row's C CTAs each
    // holds the counts of its kBins / C bins for all of them.
    int hist[kPasses][kBins];
    int own[C > 1 ? kBins : 4];  // the first digit's counts of this CTA's slots alone
    Move list[kShort];
    int scan[2][T / 32];
    int counts[3];             // this CTA's ties, holes, movers
    uint32_t bound;            // the key's digits so far, then the bound itself
    int left, equal;
};

// Sums over the warps before this one of (a, b), and the totals.
template <int T, int C>
__device__ __forceinline__ void warp_offsets(Select<T, C> &sh, int &a, int &b, int &ta, int &tb) {
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

// The moves of one row, dealt out to `warps` warps: each has kBatch loads in flight, of 32
// lanes' 16 bytes: one move's k and v, or (PER = 2) those of two moves of 128-byte rows.
// The next moves are looked up while these moves' rows are on their way.
template <int PER>
__device__ __forceinline__ void move_rows(const EvictArgs &a, const KvView &kv, int row_bytes,
                                          int id, const Move *list, int total, int warp,
                                          int warps) {
    const int s = id / kv.n_heads, h = id - s * kv.n_heads;
    const long long base = (long long)id * a.acc_stride;
    const int lane = threadIdx.x & 31, quads = row_bytes / 16;  // of k; as many of v
    constexpr int per = PER, batch = kBatch * PER;
    const int sub = PER == 1 ? 0 : lane / (32 / PER), first = PER == 1 ? lane : lane % (32 / PER);
    long long to, at;
    auto look_up = [&](int i0) {
        to = at = -1;
        if (lane < batch && i0 + lane < total) {
            const Move m = list[i0 + lane];
            at = kv.row(s, h, m.at);
            to = kv.row(s, h, m.to);
            const float w = a.acc[base + m.at];
            const int p = a.slot_pos[base + m.at];
            if (at < 0 || to < 0) {
                record_status(a.status, kStBadIndex);
                to = -1;
            }
            a.acc_out[base + m.to] = w;
            a.pos_out[base + m.to] = p;
        }
    };
    int i0 = warp * batch;
    look_up(i0);
    for (; i0 < total; i0 += warps * batch) {
        const long long to_now = to, at_now = at;
        for (int q0 = 0; q0 < 2 * quads; q0 += 32) {
            const int q = q0 + first;
            const bool of_v = q >= quads, in_row = q < 2 * quads;
            const long long in = 16ll * (of_v ? q - quads : q);
            char *pool = of_v ? kv.v : kv.k;
            uint4 x[kBatch];
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const bool live = __shfl_sync(0xFFFFFFFFu, to_now, i * per + sub) >= 0 && in_row;
                const long long src = __shfl_sync(0xFFFFFFFFu, at_now, i * per + sub);
                if (live) x[i] = *reinterpret_cast<const uint4 *>(pool + src + in);
            }
            if (q0 == 0) look_up(i0 + warps * batch);
#pragma unroll
            for (int i = 0; i < kBatch; ++i) {
                const long long dst = __shfl_sync(0xFFFFFFFFu, to_now, i * per + sub);
                if (dst >= 0 && in_row) *reinterpret_cast<uint4 *>(pool + dst + in) = x[i];
            }
        }
    }
}

__device__ __forceinline__ void move_all(const EvictArgs &a, const KvView &kv, int row_bytes,
                                         int id, const Move *list, int total, int warp,
                                         int warps) {
    if (row_bytes == 128)
        move_rows<2>(a, kv, row_bytes, id, list, total, warp, warps);
    else
        move_rows<1>(a, kv, row_bytes, id, list, total, warp, warps);
}

// One slot over the budget: the steady state of a cache that is cut after every token.  The
// slot of the least key goes (of equal ones the highest) and the last slot takes its place:
// a minimum in place of the histograms and ranks, and the last slot's rows, which move
// whichever slot goes, are read beside the weights.  8 rows of 2049 slots 2.7 us (by histograms
// 7.0), of 65536 4.6 (12.5); 1024 rows of 2049 8.1 (17.5).
template <int T, int C>
__device__ __forceinline__ void evict_one(const EvictArgs &a, const KvView &kv, Select<T, C> &sh,
                                          int row_bytes, long long base, int s, int h, int b0,
                                          int b1, int from) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, last = a.keep;
    const int rank = C == 1 ? 0 : cg::this_cluster().block_rank();
    const bool mover = rank == 0 && warp == 0, copies = a.acc_out != a.acc || a.pos_out != a.slot_pos;
    const int quads = row_bytes / 16;  // of k; as many of v
    long long at = -1;
    float w_last = 0.f;
    int p_last = 0;
    if (mover) {
        at = kv.row(s, h, last);
        w_last = a.acc[base + last];
        p_last = a.slot_pos[base + last];
    }
    constexpr int B = 8;  // slots of a thread in flight
    uint32_t key = kHeld;
    int slot = -1;
    for (int j0 = b0 + threadIdx.x; j0 < b1; j0 += B * T) {
        float w[B];
        int p[B];
#pragma unroll
        for (int i = 0; i < B; ++i)
            if (j0 + i * T < b1) w[i] = a.acc[base + j0 + i * T], p[i] = a.slot_pos[base + j0 + i * T];
#pragma unroll
        for (int i = 0; i < B; ++i) {
            const int j = j0 + i * T;
            if (j >= b1) continue;
            const uint32_t x = key_of(w[i], p[i], a.sinks, from);
            if (x <= key) key = x, slot = j;
            if (copies && j < last) {
                a.acc_out[base + j] = w[i];
                a.pos_out[base + j] = p[i];
            }
        }
    }
    // The last slot's k and v: four pieces of 512 bytes hold rows of 256 dims in f32.
    uint4 x[4];
    if (mover && at >= 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int q = lane + 32 * i;
            if (q < 2 * quads)
                x[i] = *reinterpret_cast<const uint4 *>(
                    (q < quads ? kv.k : kv.v) + at + 16ll * (q < quads ? q : q - quads));
        }
    }
    // The least key, then its highest slot.
    auto least = [&]() {
        const uint32_t k = __reduce_min_sync(0xFFFFFFFFu, key);
        slot = __reduce_max_sync(0xFFFFFFFFu, key == k ? slot : -1);
        key = k;
    };
    least();
    int *const keys = sh.scan[0], *const slots = sh.scan[1];
    if (lane == 0) keys[warp] = (int)key, slots[warp] = slot;
    __syncthreads();
    if (C > 1) {
        // Every CTA's goes to the first, beside the warps' own.
        if (warp == 0) {
            key = lane < T / 32 ? (uint32_t)keys[lane] : kHeld;
            slot = lane < T / 32 ? slots[lane] : -1;
            least();
            if (lane == 0) {
                cg::cluster_group cluster = cg::this_cluster();
                int *to = cluster.map_shared_rank(&sh.hist[0][0], 0);
                to[rank] = (int)key;
                to[C + rank] = slot;
            }
        }
        cg::this_cluster().sync();
    }
    pdl_launch();
    if (!mover) return;
    constexpr int kFrom = C > 1 ? C : T / 32;
    const int *const all_keys = C > 1 ? &sh.hist[0][0] : keys;
    const int *const all_slots = C > 1 ? &sh.hist[0][C] : slots;
    key = lane < kFrom ? (uint32_t)all_keys[lane] : kHeld;
    slot = lane < kFrom ? all_slots[lane] : -1;
    least();
    if (slot == last) return;
    const long long to = kv.row(s, h, slot);
    if (lane == 0) {
        a.acc_out[base + slot] = w_last;
        a.pos_out[base + slot] = p_last;
        if (to < 0 || at < 0) record_status(a.status, kStBadIndex);
    }
    if (to < 0 || at < 0) return;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int q = lane + 32 * i;
        if (q < 2 * quads)
            *reinterpret_cast<uint4 *>((q < quads ? kv.k : kv.v) + to +
                                       16ll * (q < quads ? q : q - quads)) = x[i];
    }
}

// C: the CTAs of a row; with one, its barriers are the CTA's.
template <int T, int C>
__global__ void __launch_bounds__(T, 1024 / T) evict_kernel(EvictArgs a, KvView kv, int row_bytes,
                                                                 int key_room, int *counts) {
    extern __shared__ __align__(16) uint8_t smem[];
    Select<T, C> &sh = *reinterpret_cast<Select<T, C> *>(smem);
    uint32_t *s_key = reinterpret_cast<uint32_t *>(smem + sizeof(Select<T, C>));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int i = threadIdx.x; i < kPasses * kBins / 4; i += T)
        reinterpret_cast<int4 *>(&sh.hist[0][0])[i] = make_int4(0, 0, 0, 0);
    constexpr bool ONE = C == 1;
    if (!ONE)
        for (int i = threadIdx.x; i < kBins; i += T) sh.own[i] = 0;
    cg::cluster_group cluster = cg::this_cluster();
    if (!ONE) cluster.sync();  // the counts are 0 before another CTA adds to them
    pdl_wait();
    const int rank = ONE ? 0 : cluster.block_rank();
    auto sync_row = [&]() {
        if (ONE)
            __syncthreads();
        else
            cluster.sync();
    };
    auto of = [&](auto *p, int r) { return ONE ? p : cluster.map_shared_rank(p, r); };
    auto counter = [&](int pass, int bin) {
        return of(&sh.hist[pass][bin], bin / (kBins / C));
    };
    const int id = blockIdx.x / C, s = id / kv.n_heads, h = id - s * kv.n_heads;
    const int given = a.lens[s], len = min(max(given, 0), a.n_slots);
    const int from = a.seen[s] - a.recent;
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
    const int share = ((len + C - 1) / C + 31) & ~31;
    const int b0 = min(len, rank * share), b1 = min(len, b0 + share), mine = b1 - b0;
    if (len <= keep) {  // within the budget: the whole cluster leaves here
        if (counts && threadIdx.x == 0 && rank == 0) counts[id] = 0;
        if (!in_place)
            for (int j = b0 + threadIdx.x; j < b1; j += T) {
                a.acc_out[base + j] = acc[j];
                a.pos_out[base + j] = pos[j];
            }
        return;
    }
    if (len == keep + 1) {
        evict_one<T, C>(a, kv, sh, row_bytes, base, s, h, b0, b1, from);
        if (counts && threadIdx.x == 0 && rank == 0) counts[id] = 0;
        return;
    }
    const bool held_keys = mine <= key_room;
    auto make_key = [&](int j) { return key_of(acc[j], pos[j], a.sinks, from); };
    // The keys of four slots from j on (j - b0 is a multiple of 4).  Those of slots at or beyond
    // b1 are whatever is there (key_room is a multiple of 32): every use checks the slot.
    auto keys4 = [&](int j, uint32_t (&x)[4]) {
        if (held_keys) {
            const uint4 v = *reinterpret_cast<const uint4 *>(s_key + (j - b0));
            x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = j + i < b1 ? make_key(j + i) : 0u;
        }
    };

    if (threadIdx.x == 0) {
        sh.bound = 0;
        sh.left = keep;
    }
    // Slots below the budget keep their places for now: the moves overwrite the holes' copies.
    for (int j0 = b0 + threadIdx.x; j0 < b1; j0 += 8 * T) {
        float w[8];
        int p[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (j0 + i * T < b1) w[i] = acc[j0 + i * T], p[i] = pos[j0 + i * T];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int j = j0 + i * T;
            if (j >= b1) continue;
            if (held_keys) s_key[j - b0] = key_of(w[i], p[i], a.sinks, from);
            if (!in_place && j < keep) {
                a.acc_out[base + j] = w[i];
                a.pos_out[base + j] = p[i];
            }
        }
    }
    __syncthreads();
    for (int pass = 0; pass < kPasses; ++pass) {
        const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : kDigit;
        const uint32_t above = sh.bound;  // the digits before this one, in place
        // Held slots and sums that are still 0 are many of one key: counted apart.  The first
        // digit's few bins are counted in this CTA and then added to the row's, later digits
        // straight away: few slots are left.
        auto add = [&](int bin, int n) {
            atomicAdd(!ONE && pass == 0 ? &sh.own[bin % (ONE ? 4 : kBins)] : counter(pass, bin), n);
        };
        int held = 0, zero = 0;
#pragma unroll 2
        for (int j = b0 + 4 * threadIdx.x; j < b1; j += 4 * T) {
            uint32_t x[4];
            keys4(j, x);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (j + i >= b1 || (pass > 0 && (x[i] ^ above) >> (shift + bits))) continue;
                if (x[i] == kHeld)
                    ++held;
                else if (x[i] == kZero)
                    ++zero;
                else
                    add((x[i] >> shift) & ((1 << bits) - 1), 1);
            }
        }
        held = __reduce_add_sync(0xFFFFFFFFu, held);
        zero = __reduce_add_sync(0xFFFFFFFFu, zero);
        if (lane == 0 && held) add((kHeld >> shift) & ((1 << bits) - 1), held);
        if (lane == 0 && zero) add((kZero >> shift) & ((1 << bits) - 1), zero);
        if (!ONE && pass == 0) {
            __syncthreads();
            for (int bin = threadIdx.x; bin < kBins; bin += T)
                if (const int n = sh.own[bin]) atomicAdd(counter(0, bin), n);
        }
        sync_row();
        // The bin that holds the left-th largest: each thread has kBins / T of them, from
        // the top.
        constexpr int kMine = kBins / T;
        const int top = kBins - kMine * (threadIdx.x + 1);  // this thread's lowest bin
        int count[kMine] = {}, sum = 0;
        const int2 *counts2 = reinterpret_cast<const int2 *>(counter(pass, top));
#pragma unroll
        for (int i = 0; i < kMine / 2; ++i) {
            const int2 v = counts2[i];
            count[2 * i] = v.x, count[2 * i + 1] = v.y;
        }
#pragma unroll
        for (int i = 0; i < kMine; ++i) sum += count[i];
        int incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xFFFFFFFFu, incl, o);
            if (lane >= o) incl += y;
        }
        if (lane == 31) sh.scan[0][warp] = incl;
        const int left = sh.left;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < T / 32; ++w)
            if (w < warp) incl += sh.scan[0][w];
        int before = incl - sum;
        if (before < left && left <= incl) {
#pragma unroll
            for (int i = kMine - 1; i >= 0; --i) {
                if (before < left && left <= before + count[i]) {
                    sh.bound = above | (uint32_t)(top + i) << shift;
                    sh.left = left - before;
                    sh.equal = count[i];
                }
                before += count[i];
            }
        }
        __syncthreads();
        if (sh.left == sh.equal) break;  // the whole bin stays: all keys >= bound do
    }
    const uint32_t bound = sh.bound;
    const int ties = sh.left;
    const bool all_ties = ties == sh.equal;  // else `ties` of the slots with the bound's key stay

    // Each warp takes a contiguous piece and each lane four slots of 128, so that ranks follow
    // the slots.
    const int piece = ((mine + T / 32 - 1) / (T / 32) + 127) & ~127;
    const int w0 = min(b1, b0 + warp * piece), w1 = min(b1, w0 + piece);
    int same = 0, none = 0, all_same, all_none;
    if (!all_ties) {
        for (int j = w0 + 4 * lane; j < w1; j += 128) {
            uint32_t x[4];
            keys4(j, x);
#pragma unroll
            for (int i = 0; i < 4; ++i) same += j + i < w1 && x[i] == bound;
        }
        same = __reduce_add_sync(0xFFFFFFFFu, same);
        warp_offsets<T, C>(sh, same, none, all_same, all_none);
        if (!ONE) {
            if (threadIdx.x == 0) sh.counts[0] = all_same;
            cluster.sync();
#pragma unroll
            for (int r = 0; r < C; ++r) {
                const int x = *cluster.map_shared_rank(&sh.counts[0], r);
                if (r < rank) same += x;
            }
        }
    }
    // The sums of x over the lanes before this one and over all.
    auto lane_offsets = [&](int x, int &all) {
        int incl = x;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xFFFFFFFFu, incl, o);
            if (lane >= o) incl += y;
        }
        all = __shfl_sync(0xFFFFFFFFu, incl, 31);
        return incl - x;
    };
    // Of this lane's four slots, those whose place changes hands (bits 0-3: holes below the
    // budget, 4-7: movers beyond it).  `tie` counts the bound's slots before the 128.
    auto vote = [&](int j, int &tie) {
        uint32_t x[4] = {};
        if (j < w1) keys4(j, x);
        int rank_of = 0;
        if (!all_ties) {
            int mine_at = 0, all;
#pragma unroll
            for (int i = 0; i < 4; ++i) mine_at += j + i < w1 && x[i] == bound;
            rank_of = tie + lane_offsets(mine_at, all);
            tie += all;
        }
        unsigned v = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (j + i >= w1) continue;
            bool stay = x[i] >= bound;
            if (!all_ties && x[i] == bound) stay = rank_of++ < ties;
            if (j + i < keep ? !stay : stay) v |= (j + i < keep ? 1u : 16u) << i;
        }
        return v;
    };
    int holes = 0, movers = 0, total, cta_movers, tie = same;
    for (int j0 = w0; j0 < w1; j0 += 128) {
        const unsigned v = vote(j0 + 4 * lane, tie);
        holes += __popc(v & 15u);
        movers += __popc(v >> 4);
    }
    holes = __reduce_add_sync(0xFFFFFFFFu, holes);
    movers = __reduce_add_sync(0xFFFFFFFFu, movers);
    warp_offsets<T, C>(sh, holes, movers, total, cta_movers);
    if (!ONE) {
        if (threadIdx.x == 0) {
            sh.counts[1] = total;
            sh.counts[2] = cta_movers;
        }
        cluster.sync();
        total = 0;
#pragma unroll
        for (int r = 0; r < C; ++r) {
            const int x = *cluster.map_shared_rank(&sh.counts[1], r);
            const int y = *cluster.map_shared_rank(&sh.counts[2], r);
            if (r < rank) holes += x, movers += y;
            total += x;
        }
    }
    // Every move, in slot order.
    Move *list = ONE && total <= kShort && !counts
                     ? sh.list
                     : static_cast<Move *>(a.workspace) + (long long)id * min(a.keep, a.n_slots);
    tie = same;
    for (int j0 = w0; j0 < w1; j0 += 128) {
        const int j = j0 + 4 * lane;
        const unsigned v = vote(j, tie);
        if (!__any_sync(0xFFFFFFFFu, v)) continue;
        int all;  // holes in the low half, movers in the high one
        const int at = lane_offsets(__popc(v & 15u) | __popc(v >> 4) << 16, all);
        Move *to_hole = list + holes + (at & 0xFFFF), *to_mover = list + movers + (at >> 16);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (v >> i & 1u) (to_hole++)->to = j + i;
            if (v >> i & 16u) (to_mover++)->at = j + i;
        }
        holes += all & 0xFFFF;
        movers += all >> 16;
    }
    sync_row();  // the list is complete; no shared memory of another CTA is read below
    pdl_launch();

    if (counts) {  // many moves of few rows: evict_move_kernel's
        if (threadIdx.x == 0 && rank == 0) counts[id] = total;
        return;
    }
    move_all(a, kv, row_bytes, id, list, total, rank * (T / 32) + warp, C * (T / 32));
}

// The moves of rows whose selection left them: blocks_per_row blocks to each.
__global__ void __launch_bounds__(256, 4) evict_move_kernel(EvictArgs a, KvView kv, int row_bytes,
                                                            const int *counts, int blocks_per_row) {
    pdl_enter();
    const int id = blockIdx.x / blocks_per_row, block = blockIdx.x - id * blocks_per_row;
    move_all(a, kv, row_bytes, id,
             static_cast<const Move *>(a.workspace) + (long long)id * min(a.keep, a.n_slots),
             counts[id], block * 8 + (threadIdx.x >> 5), blocks_per_row * 8);
}

// Lengths in place: after every row of a sequence has read them.
__global__ void evict_lens_kernel(EvictArgs a) {
    pdl_enter();
    const int s = blockIdx.x * blockDim.x + threadIdx.x;
    if (s < a.n_seq) a.lens_out[s] = min(max(a.lens[s], 0), min(a.keep, a.n_slots));
}

int row_bytes_of(const KvView &kv) { return kv.head_dim * (kv.dtype == kF32 ? 4 : 2); }

template <int T, int C>
cudaError_t launch_rows(const EvictArgs &a, const KvView &kv, int *counts, const DeviceInfo &dev,
                        cudaStream_t stream) {
    const int row_bytes = row_bytes_of(kv);
    const long long share = ((a.n_slots + (long long)C - 1) / C + 31) & ~31ll;
    const int key_room = (int)(share < kMaxKeys ? share : kMaxKeys);
    static std::atomic<unsigned long long> done{0};
    constexpr int kFixed = sizeof(Select<T, C>);
    static_assert(kFixed + kMaxKeys * 4 <= 227 * 1024, "shared memory");
    cudaError_t err = ensure_smem(evict_kernel<T, C>, kFixed + kMaxKeys * 4, dev, done);
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)((long long)a.n_seq * kv.n_heads * C));
    cfg.blockDim = dim3(T);
    cfg.dynamicSmemBytes = kFixed + (size_t)key_room * 4;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = C;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = C == 1 ? 1 : 2;
    return cudaLaunchKernelEx(&cfg, evict_kernel<T, C>, a, kv, row_bytes, key_room, counts);
}

}  // namespace

size_t evict_workspace_bytes(const KvView &kv, int n_seq, int n_slots, int keep) {
    if (keep > n_slots) keep = n_slots;
    // The moves, and how many each row has.
    return ((size_t)n_seq * kv.n_heads * (keep * sizeof(Move) + sizeof(int)) + 255) & ~(size_t)255;
}

cudaError_t launch_kv_evict(const EvictArgs &a, const KvView &kv, const DeviceInfo &dev,
                            cudaStream_t stream) {
    const long long rows = (long long)a.n_seq * kv.n_heads;
    if (rows > 0x7FFFFFFFll / 8) return cudaErrorInvalidConfiguration;
    // More CTAs to a row while two per SM are not reached and each has over 4096 slots or 128
    // moves (8 rows of 20000 slots, one over: 1 CTA 6.3 us, 8 take 3.5; of 2049: 2.7 and 3.2;
    // 8 rows of 4096 cut to 1024: 26.2 and 12.4).  512 threads while two such CTAs per SM hold
    // all rows or the rows are long, else 256 (512 rows of 2049, one over: 4.7 us, with 512
    // 5.8; of 8193 19.2 and 16.0).  1024 for few long rows, whose clusters of eight CTAs, of
    // an SM each, all find room at once (4 rows of 131072 cut to 16384 37 us, with 512 46; 14 rows
    // 97 and 108; 14 rows of 70000 cut to 60000 64 and 67, 16 rows 70 and 60).
    const long long moves = a.keep < a.n_slots - a.keep ? a.keep : a.n_slots - a.keep;
    int cluster = 1;
    while (cluster < 8 && rows * cluster * 2 <= 2 * dev.sm_count &&
           (a.n_slots / cluster > 4096 || moves / cluster > 128))
        cluster *= 2;
    // Where SMs have no row and a CTA may have 80 KB or more to move, the moves are a launch of
    // their own over all SMs (3 rows of 9293 cut to 3506, 214 KB: 12.8 us, by the rows' CTAs
    // 18.3; 105 KB: 13.4 and 14.9; 62 KB: 15.2 and 12.2).
    const int row_bytes = row_bytes_of(kv);
    int *counts = nullptr;
    if (rows * cluster <= dev.sm_count && moves * row_bytes * 2 >= cluster * (80ll << 10))
        counts = reinterpret_cast<int *>(static_cast<Move *>(a.workspace) +
                                         rows * (a.keep < a.n_slots ? a.keep : a.n_slots));
    cudaError_t err;
    switch (cluster) {
    case 1:
        err = rows <= 2 * dev.sm_count || a.n_slots > 6144 ? launch_rows<512, 1>(a, kv, counts, dev, stream)
                                                           : launch_rows<256, 1>(a, kv, counts, dev, stream);
        break;
    case 2: err = launch_rows<512, 2>(a, kv, counts, dev, stream); break;
    case 4: err = launch_rows<512, 4>(a, kv, counts, dev, stream); break;
    default:
        err = rows <= 14 && a.n_slots > 65536
                  ? launch_rows<1024, 8>(a, kv, counts, dev, stream)
                  : launch_rows<512, 8>(a, kv, counts, dev, stream);
    }
    if (err == cudaSuccess && counts) {
        const int blocks_per_row = (int)((4ll * dev.sm_count + rows - 1) / rows);
        err = launch_pdl(evict_move_kernel, dim3((unsigned)(rows * blocks_per_row)), dim3(256), 0,
                         stream, a, kv, row_bytes, (const int *)counts, blocks_per_row);
    }
    if (err != cudaSuccess || a.lens_out != a.lens) return err;
    return launch_pdl(evict_lens_kernel, dim3((a.n_seq + 255) / 256), dim3(256), 0, stream, a);
}

}  // namespace wq

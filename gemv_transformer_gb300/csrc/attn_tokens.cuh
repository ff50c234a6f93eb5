// attn_tokens.cuh -- what the kernels of wq_attn_tokens share: which slots a token sees, how the
// work is dealt out, and the parts of rows that several CTAs work on.
//
// A row is a (new token, query head) of one sequence and kv head, row = token * group + head in
// the group: the heads of a group share k and v.  A row tile is RT rows of a sequence, a key tile
// KT slots.  attn_plan_kernel lists the row tiles with the key tiles that any of their rows sees,
// sums their costs, and cuts the whole (all kv heads, one after another) into equal contiguous
// ranges, one for each CTA of a fixed grid, whatever the lengths.  A row tile within one CTA
// is written by it; the parts of the others are joined by the rule of the running softmax, in an
// order that the lengths fix: by whichever of their CTAs is the last to finish where a row tile
// has few parts (a 2048-token prompt: 57 us, with a launch for it 65), else by attn_parts_kernel
// (one CTA alone reads 20 parts in 28 us).
#pragma once

#include "kv_internal.h"
#include "wq_device.cuh"

namespace wq {
namespace tok {

constexpr int kMaxGrid = 304;  // two CTAs on each of 152 SMs

// A sequence's part in the call.
struct Seq {
    int t0, count, base, len;  // first token, new tokens, slots before them, live slots
};
// `bad`: what the header promises to record.
__device__ __forceinline__ Seq seq_of(const TokensArgs &a, int s, bool &bad) {
    const int t0 = a.starts[s], t1 = a.starts[s + 1], len = a.lens[s];
    Seq q{t0, t1 - t0, 0, min(max(len, 0), a.n_slots)};
    if (t0 < 0 || t1 < t0 || t1 > a.n_tok) {
        q.count = 0;
        bad = true;
    }
    q.base = q.len - q.count;
    if (q.len != len || q.base < 0) bad = true;
    return q;
}

// Positions are held where the differences of two, or of one and a slot, fit 32 bits.
__device__ __forceinline__ int near(int pos) { return min(max(pos, 1 - (1 << 30)), 1 << 30); }

// The slots that token j of a sequence sees: [lo, hi), and with a tree, of the new tokens' slots
// [own, own_end) those whose bit is set.
struct See {
    int lo, hi;
    int own, own_end, first, pos;  // tree only: own_end > own
    const uint32_t *bits;
    const int32_t *own_pos;        // positions of the new tokens where a window asks for them
};
__device__ __forceinline__ See see_of(const TokensArgs &a, const Seq &q, int s, int j) {
    See v{};
    const int t = q.t0 + j;
    v.first = a.first ? max(a.first[t], 0) : 0;
    v.pos = a.pos ? near(a.pos[t]) : q.base + j;
    v.lo = v.first;
    if (a.window > 0)
        v.lo = (int)max((long long)v.lo, min((long long)v.pos - a.window + 1, (long long)q.len));
    if (a.tree) {
        v.hi = max(q.base, 0);
        v.own = q.base;
        v.own_end = (int)min((long long)q.len, q.base + a.tree_stride * 32);
        v.bits = a.tree + (long long)t * a.tree_stride;
        v.own_pos = a.window > 0 && a.pos ? a.pos + q.t0 : nullptr;
        // Without positions of their own the new tokens' windows are by slot.
        if (a.window > 0 && !a.pos) v.first = v.lo;
    } else {
        v.hi = min(q.base + j + 1, q.len);
        if (a.prefix) v.hi = max(v.hi, min(a.prefix[s], q.len));
    }
    v.hi = max(v.hi, 0);
    return v;
}

__device__ __forceinline__ uint32_t below(int n) {  // the n lowest bits
    return n <= 0 ? 0u : n >= 32 ? 0xFFFFFFFFu : (1u << n) - 1u;
}
// Bit i: slot j0 + i is seen.
__device__ __forceinline__ uint32_t seen32(const TokensArgs &a, const See &v, int j0) {
    uint32_t m = below(v.hi - j0) & ~below(v.lo - j0);
    if (v.own_end > v.own && j0 + 32 > v.own && j0 < v.own_end) {
        // Bits b0 .. b0 + 31 of the token's row, those in [0, own_end - own).
        const int b0 = j0 - v.own, count = v.own_end - v.own;
        const int w = b0 >> 5;  // rounds down
        const uint32_t lo = w >= 0 && w * 32 < count ? v.bits[w] : 0u;
        const uint32_t hi = w + 1 >= 0 && (w + 1) * 32 < count ? v.bits[w + 1] : 0u;
        uint32_t own = __funnelshift_r(lo, hi, b0 & 31);
        own &= below(count - b0) & ~below(-b0) & ~below(v.first - j0);
        if (v.own_pos) {
            for (uint32_t left = own; left; left &= left - 1) {
                const int i = __ffs(left) - 1;
                if (v.pos - near(v.own_pos[b0 + i]) >= a.window) own &= ~(1u << i);
            }
        }
        m |= own;
    }
    return m;
}
// Position of slot j, for the distance bias.
__device__ __forceinline__ int slot_pos(const TokensArgs &a, const Seq &q, int j) {
    return a.pos && j >= q.base && j < q.len ? near(a.pos[q.t0 + j - q.base]) : j;
}

// --------------------------------------------------------------------- workspace --

struct Tile {
    int seq, row0;
    int k0, k1;        // key tiles
    int lo, hi;        // every row of the tile sees [lo, hi)
    Seq q;             // the sequence's
};
struct Begin {
    int head, tile, off;  // where a CTA's range starts: kv head, row tile, key tiles into it
    int tiles;            // row tiles of all sequences
    int lead, parts;      // off > 0: the first CTA that works on that row tile, and how many do
};
struct Room {
    Begin *plan;         // [grid + 1]
    unsigned *joined;    // [grid][2]: parts that are there of the row tile that a CTA leads, by
                         // warpgroup where those go by themselves; zeroed by the plan
    long long *before;   // [tiles + 1]: cost of the row tiles before each
    Tile *tiles;
    float2 *part_ml;     // [2 grid][RT]: running maximum (log2 units) and sum
    float4 *part_o;      // [2 grid][DP / 4][RT]
    size_t bytes;
};
__host__ __device__ inline size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }
__host__ __device__ inline long long most_tiles(int n_seq, int n_tok, int group, int rt) {
    return (long long)n_tok * group / rt + (n_seq < n_tok ? n_seq : n_tok) + 1;
}
__host__ __device__ inline Room room_of(void *p, int n_seq, int n_tok, int group, int rt, int dp,
                                        int grid) {
    char *c = static_cast<char *>(p);
    const size_t tiles = (size_t)most_tiles(n_seq, n_tok, group, rt);
    Room r;
    size_t at = 0;
    r.plan = reinterpret_cast<Begin *>(c + at);
    at += up256((kMaxGrid + 1) * sizeof(Begin));
    r.joined = reinterpret_cast<unsigned *>(c + at);
    at += up256(kMaxGrid * 2 * sizeof(unsigned));
    r.before = reinterpret_cast<long long *>(c + at);
    at += up256((tiles + 1) * sizeof(long long));
    r.tiles = reinterpret_cast<Tile *>(c + at);
    at += up256(tiles * sizeof(Tile));
    r.part_ml = reinterpret_cast<float2 *>(c + at);
    at += up256((size_t)2 * grid * rt * sizeof(float2));
    r.part_o = reinterpret_cast<float4 *>(c + at);
    at += up256((size_t)2 * grid * rt * dp * sizeof(float));
    r.bytes = at;
    return r;
}

// One stretch of a CTA's range: key tiles [k0, k1) of a row tile for a kv head.
struct Stretch {
    int tile, head, k0, k1;
    int part;         // -1: all of the row tile; else its place in this CTA's two parts
};
// Part i of a row tile: the second of the first CTA's, then the first of each other's.
__device__ __forceinline__ size_t part_place(int lead, int i) {
    return i == 0 ? 2 * lead + 1 : 2 * (lead + i);
}
// A part's CTA says that it is written; true for the one that is the last of them.  Called by one
// thread after a barrier behind the writers' fences; a fence and a barrier follow for the readers.
__device__ __forceinline__ bool part_last(const Room &room, const Stretch &st, int cta, int which,
                                          int &lead, int &parts) {
    const Begin *const b = room.plan + cta + st.part;  // (part 1: the next CTA begins in it)
    lead = b->lead, parts = b->parts;
    __threadfence();
    return atomicAdd(room.joined + 2 * lead + which, 1u) == (unsigned)parts - 1;
}
// The stretches of a CTA, one after another.  Little of it stays in registers: what it needs it
// reads again.
struct Walk {
    const Begin *plan;
    const Tile *tiles;
    int head, tile, off;
    __device__ __forceinline__ Walk(const Room &r, int cta) : plan(r.plan + cta), tiles(r.tiles) {
        head = plan->head, tile = plan->tile, off = plan->off;
    }
    __device__ __forceinline__ bool next(Stretch &s) {
        const int to_head = plan[1].head, to_tile = plan[1].tile, to_off = plan[1].off;
        if (head > to_head || (head == to_head && tile > to_tile)) return false;
        const bool last = head == to_head && tile == to_tile;
        if (last && off >= to_off) return false;
        const int k0 = tiles[tile].k0, k1 = tiles[tile].k1;
        s.tile = tile;
        s.head = head;
        s.k0 = k0 + off;
        s.k1 = last ? k0 + to_off : k1;
        s.part = off > 0 ? 0 : s.k1 < k1 ? 1 : -1;
        off = 0;
        if (++tile == plan->tiles) tile = 0, ++head;
        if (last) head = to_head + 1;
        return true;
    }
};

struct TypedOut {
    void *p;
    int type;
    __device__ __forceinline__ void put2(long long at, float2 v) const {
        if (type == kF32) {
            reinterpret_cast<float2 *>(p)[at >> 1] = v;
        } else if (type == kBF16) {
            reinterpret_cast<__nv_bfloat162 *>(p)[at >> 1] = __floats2bfloat162_rn(v.x, v.y);
        } else {
            reinterpret_cast<__half2 *>(p)[at >> 1] = __floats2half2_rn(v.x, v.y);
        }
    }
    __device__ __forceinline__ void put4(long long at, float4 v) const {
        if (type == kF32) {
            reinterpret_cast<float4 *>(p)[at >> 2] = v;
            return;
        }
        uint2 w;
        if (type == kBF16) {
            const __nv_bfloat162 x = __floats2bfloat162_rn(v.x, v.y),
                                 y = __floats2bfloat162_rn(v.z, v.w);
            w = make_uint2(*reinterpret_cast<const uint32_t *>(&x),
                           *reinterpret_cast<const uint32_t *>(&y));
        } else {
            const __half2 x = __floats2half2_rn(v.x, v.y), y = __floats2half2_rn(v.z, v.w);
            w = make_uint2(*reinterpret_cast<const uint32_t *>(&x),
                           *reinterpret_cast<const uint32_t *>(&y));
        }
        reinterpret_cast<uint2 *>(p)[at >> 2] = w;
    }
};

// 16 bytes to shared memory, zeros where the source is not live.
__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool live) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(live ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

constexpr float kLn2 = 0.693147180559945309f, kLog2e = 1.44269504088896341f;
__device__ __forceinline__ float lse_of(float m, float l) {
    return l == 0.f ? -INFINITY : fmaf(m, kLn2, logf(l));  // (scores that are not numbers: NaN)
}

// row_cost: a row tile's start and end count as so many key tiles.
// heads: kv heads, times the passes over a head's dims.
cudaError_t launch_attn_plan(const TokensArgs &a, int heads, int rt, int kt, int dp, int grid,
                             int row_cost, cudaStream_t stream);
// Does a row tile have few parts: are there as many row tiles as CTAs?  (That goes by the rows
// alone; lengths are known on the device only.)
inline bool joins_inside(const TokensArgs &a, int heads, int rt, int grid) {
    return (long long)a.n_tok * a.group.d / rt * heads >= grid;
}
cudaError_t launch_attn_parts(const TokensArgs &a, const KvView &kv, int passes, int rt, int dp,
                              int grid, cudaStream_t stream);

// The tensor-core kernels (attn_tokens_tc.cu).
bool tokens_tc_takes(const KvView &kv, int q_type);
void tokens_tc_shape(int n_seq, int n_tok, int group, int q_type, int head_dim, int &rt, int &dp,
                     int &grid);
cudaError_t launch_tokens_tc(const TokensArgs &a, const KvView &kv, const DeviceInfo &dev,
                             cudaStream_t stream);

}  // namespace tok
}  // namespace wq

// attn_paged.cu -- attention of one new token per sequence over a paged cache.
//
// wavo 0.3.0 src/gpu/mod.rs, attend / combine: one token's attention over the decoder's
// cache with the keys split into parts that are joined.  x_j = scale q.k_j + mask_j,
// p = softmax(x) by one pass with a running maximum m and sum l:
//   m' = max(m, x), l' = l e^(m-m') + e^(x-m'), o' = o e^(m-m') + e^(x-m') v,
// and parts (m, l, o) of a row are joined by the same rule, in an order that the lengths fix.
//
// What bounds it: every live slot's k and v are read once and used group times (4 group
// operations per 2 bytes of a bf16 cache), so the cache's bytes set the floor.  Measured (the
// whole call, back to back; 6704 GB/s is this GPU's copy rate): 64 sequences of 1 to 8192 slots, 8
// kv heads of 128 in bf16, 64 query heads, 1.08 GB: 167 us, 6430 GB/s; one sequence of
// 131072, 32 query heads: 90 us, 5960 GB/s, of which 7 us pass before the first tile is done
// (lengths, page numbers, the tile: three loads that wait for one another) and 4 after the
// last (the join).  Shorter calls are that chain: 391 slots 7.0 us.
//
// Products: the heads of a group are the rows of mma.sync operands, eight heads to a
// fragment, and an f32 value is split into terms of the operand's type, the first two in rows
// g and g + 8 of one product:
//   bf16 cache  q and p as three bf16 terms (24 bits): a second product has the third, or,
//               of four heads or fewer, rows 4 to 7 of the first;
//   f16 cache   tf32 products: k and v are exact in them, q and p two terms, each rounded
//               (within 2^-23; three, 24 bits, of four heads or fewer).  Two f16 terms are
//               faster (32 sequences to 4096: 64/8 heads of 128 56 us and 59, 128/8 77 and
//               106, 8/8 of 64 35 and 42) but lose small values: the rest of a p of e^-25 has
//               no f16 exponent (that p was off by 4 %).  Rests scaled up by 2^12 in rows of
//               their own reach 2^-39 of the largest value and end there, and a sum with
//               subnormal operands in it kept fewer bits (3e-6 of that p lost);
//   f32 cache   tf32 products: q and p two terms, each rounded (within 2^-23), k and v
//               three that cut them at 11 bits (exact), in three products.  Two are faster
//               (32 sequences to 4096, 32/8 heads of 128 102 us and 118) but lose up to
//               3 2^-23 of k and v, always toward zero; rounded ones would take the largest
//               finite values to infinity.
// 16-bit operands alone would leave 2^-9.  The tensor core truncates when it
// accumulates (measured: 1 + 0.92 ulp added 1000 times stays 1), so no accumulation is
// longer than head_dim / 16 steps of q.k, and every tile's p.v is added to o by an f32
// FMA that rescales it anyway.
//
// A k that is not finite has to show: a slot takes no part by its mask, length or page, never by
// its score.  A score of -inf would be that slot's weight 0, so every type has a product of an
// infinite k that is NaN, whatever q: the zero rows beside the third terms (0 inf), or for f32 k
// minus its high part.  Where f16 has two terms, a score of -inf has its k looked at.
//
// p's accumulator fragment is the next product's operand without a move.
//
// Loads: each warp keeps a ring of tiles of KT slots (k and v) in flight by cp.async and
// waits for no other warp: a CTA's warps meet only where a row (sequence, kv head, up to
// 16 query heads) ends.  64 KB per CTA and three CTAs per SM (two where registers or a row of
// 256 dims want it): 12 warps hide the chain of a tile better than 8 with a deeper ring
// (131072 slots: 91 and 110 us).  A slot that takes no part (beyond the length, masked by
// -inf, in a page out of range) is filled with zeros in shared memory and not read.
//
// Work: the rows' tiles, one row after another, are dealt out in equal contiguous ranges to
// a fixed grid, whatever the lengths; a CTA finds its range from the lengths.  A row within
// one CTA is written by it, the parts of the others are joined by attn_join_kernel.  Small
// calls give each row a cluster of CTAs that join their parts through shared memory.
#include <cooperative_groups.h>

#include <type_traits>

#include "kv_internal.h"
#include "wq_device.cuh"

namespace wq {
namespace {

namespace cg = cooperative_groups;

constexpr int kMaxCtas = 456;  // three on each of 152 SMs

// Q4 (16-bit types): groups of at most four heads, whose third terms take rows 4 to 7 of the one
// product.
template <int DT, int DP, int HT, bool Q4> struct Shape {
    static constexpr bool k16 = DT != kF32;            // elements of 16 bits
    static constexpr bool kTf = DT != kBF16;           // tf32 products
    static constexpr int kEb = k16 ? 2 : 4;            // bytes of an element
    static constexpr int kRow = DP * kEb;              // bytes of a slot's row in the ring
    static constexpr int kEpc = 16 / kEb;              // elements of a 16-byte chunk
    static constexpr int kChunks = kRow / 16;
    static constexpr int KT = k16 ? 16 : 8;            // slots of a warp's tile
    static constexpr int NT = KT / 8;
    static constexpr int W = DP == 256 ? 3 : 4;        // warps
    static constexpr int kCtas = HT * DP == 256 ? 2 : 3;  // per SM
    static constexpr int kTile = 2 * KT * kRow;        // bytes: k, then v
    static constexpr int kStages = DP == 64 ? 4 : HT * DP == 256 && DP == 128 && !kTf ? 3 : 2;
    static constexpr int BT = W * KT;                  // slots of a CTA's tile
    static constexpr int kHeads = HT * 8;              // query heads of a row
    static constexpr bool kQReg = !kTf && HT * DP <= 128;  // q's fragments in registers
    static constexpr int kStep = kTf ? 8 : 16;         // dims of a product step
    static constexpr int kSteps = DP / kStep;
    static constexpr bool k3 = !kTf && !Q4;            // a second product for the third term
    static constexpr int kQWords = k3 ? 6 : 4;         // registers of a step's fragment
    static constexpr int kQ = W * kStages * kTile;     // q fragments, unless in registers
    static constexpr int kQBytes = kQReg ? 0 : HT * kSteps * 32 * kQWords * 4;
    static constexpr int kBias = kQ + kQBytes;                     // [W][kStages][KT]
    static constexpr int kM = kBias + W * kStages * KT * 4;        // [W][kHeads], then factors
    static constexpr int kL = kM + W * kHeads * 4;                 // [W][kHeads]
    static constexpr int kTop = kL + W * kHeads * 4;               // [kHeads]
    static constexpr int kSum = kTop + kHeads * 4;                 // [kHeads]
    static constexpr int kSmem = kSum + kHeads * 4;
    static constexpr int kPart = kHeads * (DP + 2);    // floats of a part: m, l, o (16-byte rows)
    static_assert(kHeads * DP * 4 <= kTile, "a warp's o fits the tile just used");
    static_assert(kCtas * (kSmem + 1024) <= 228 * 1024, "CTAs per SM");
};

__device__ __forceinline__ long long div_any(long long a, long long b) {
    if (((a | b) >> 32) == 0) return (uint32_t)a / (uint32_t)b;
    return a / b;
}

// The schedule that every CTA derives from the lengths: a row of sequence s costs
// tiles(s) + kRowCost, a tile 1 and the end of a row (the warps meet, new queries) kRowCost;
// tiles(s) is never 0 (an empty row is written too).
// Measured on 64 sequences of 1 to 8192 slots: cost 0 207 us, 1 188 us, 2 183 us.
constexpr int kRowCost = 2;
struct Sched {
    long long total, q, r;  // cost of all rows; total / grid and the rest
    __device__ __forceinline__ Sched(long long t, int grid)
        : total(t), q(div_any(t, grid)), r(t - q * grid) {}
    __device__ __forceinline__ long long start(int b) const { return b * q + min((long long)b, r); }
    __device__ __forceinline__ int owner(long long t) const {
        const long long cut = r * (q + 1);
        return (int)(t < cut ? div_any(t, q + 1) : r + div_any(t - cut, q));
    }
};

struct Span { int len, first; };
__device__ __forceinline__ Span span_of(const AttnArgs &a, int s) {
    Span p;
    p.len = min(max(a.lens[s], 0), a.n_slots);
    p.first = a.window > 0 && p.len > a.window ? p.len - a.window : 0;
    return p;
}

__device__ __forceinline__ float exp_diff(float x, float m) {
    return x == -INFINITY ? 0.f : expf(x - m);
}

// ------------------------------------------------------------------- terms --

__device__ __forceinline__ uint32_t tf32(float x) {
    uint32_t r;
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}
// The terms of a pair, packed: t[0] + t[1] + t[2] = (x, y).
__device__ __forceinline__ void split2(float x, float y, uint32_t (&t)[3]) {
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        t[i] = bf16x2(x, y);
        x -= bf16_lo(t[i]);
        y -= bf16_hi(t[i]);
    }
}
// x's column of a tf32 fragment, (t0, t1): its terms in rows g and g + 8, or with THIRD, in
// the lanes of rows 4 to 7, what two terms leave and 0.
template <bool THIRD>
__device__ __forceinline__ void split_tf32(float x, bool third, uint32_t &t0, uint32_t &t1) {
    t0 = tf32(x);
    const float rest = x - __uint_as_float(t0);
    t1 = tf32(rest);
    if (THIRD && third) t0 = __float_as_uint(rest - __uint_as_float(t1)), t1 = 0u;
}

// ---------------------------------------------------------------- products --

// d = a * b + c; c = 0 costs no registers.
__device__ __forceinline__ void mma_tf32(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1, float c0, float c1, float c2, float c3) {
    asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c0), "f"(c1),
          "f"(c2), "f"(c3));
}
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1, float c0,
                                         float c1, float c2, float c3) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, "
        "{%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2),
          "f"(c3));
}
// A pair of f16 as tf32 operands.
__device__ __forceinline__ uint2 widen(uint32_t x) {
    const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&x));
    return make_uint2(__float_as_uint(v.x), __float_as_uint(v.y));
}
// An f32 value as three of 11, 11 and 2 bits.
struct Cut {
    uint32_t t[3];
};
__device__ __forceinline__ Cut cut3(uint32_t x) {
    Cut c;
    c.t[0] = x & 0xFFFFE000u;
    const float rest = __uint_as_float(x) - __uint_as_float(c.t[0]);
    c.t[1] = __float_as_uint(rest) & 0xFFFFE000u;
    c.t[2] = __float_as_uint(rest - __uint_as_float(c.t[1]));
    return c;
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr));
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
    return v;
}
// Four 8x8 matrices of 16-bit elements, their rows at the lanes' addresses.
template <bool TRANS> __device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr) {
    if (TRANS)
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                     : "r"(addr));
    else
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                     : "r"(addr));
}

// 16 bytes global -> shared, or 16 zero bytes.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool live) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(live ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N> __device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Chunk ch of slot r lies at chunk ch ^ swizzle of the slot's row.  16-bit types: the
// eight rows of a matrix at eight bank groups.  f32: a quarter warp reads two keys' four
// chunks, or four values' two.
template <int DT> __device__ __forceinline__ int swizzle_k(int r) {
    return DT == kF32 ? (r & 1) << 2 : r & 7;
}
template <int DT> __device__ __forceinline__ int swizzle_v(int r) {
    return DT == kF32 ? r & 6 : r & 7;
}

// A CTA's place in the rows' tiles.
struct Cursor {
    int s, row, tile, tiles;  // sequence, row within it, tile within the row
    Span span;
    __device__ __forceinline__ void load(const AttnArgs &a, int bt) {
        span = span_of(a, s);
        tiles = max(1, (span.len - span.first + bt - 1) / bt);
    }
    __device__ __forceinline__ void next(const AttnArgs &a, int rows, int bt) {
        if (++tile < tiles) return;
        tile = 0;
        if (++row < rows) return;
        row = 0;
        if (++s < a.n_seq) load(a, bt);
    }
};

// The workspace: the rows that are split, their parts, and for the weight sums where each row
// is, its heads' lse and every score.
struct Room {
    int4 *rows;         // [n_seq * rows], where there are no more rows than CTAs and for the
                        // weight sums: the row's first CTA, its CTAs, the first's part
    int4 *splits;       // [grid] the row that a CTA begins and others go on with: (sequence,
                        // row, CTAs, the first's part); no CTAs: none
    float *parts, *lse, *scores;
};
__host__ __device__ inline size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }
__host__ __device__ inline size_t rows_bytes(int n_seq, int h_q, bool with_acc) {
    return up256((with_acc ? (size_t)n_seq * h_q : 0) * 16 + kMaxCtas * 16);  // a row has a head
}
__host__ __device__ inline Room room_of(void *p, int n_seq, int h_q, size_t part_floats,
                                        bool with_acc) {
    char *c = static_cast<char *>(p);
    Room r;
    r.splits = reinterpret_cast<int4 *>(c);
    c += up256(kMaxCtas * 16);
    r.parts = reinterpret_cast<float *>(c);
    c += up256(2ull * kMaxCtas * part_floats * 4);
    r.rows = reinterpret_cast<int4 *>(c);
    c += rows_bytes(n_seq, h_q, with_acc);
    r.lse = reinterpret_cast<float *>(c);
    c += up256((size_t)n_seq * h_q * 4);
    r.scores = reinterpret_cast<float *>(c);
    return r;
}

// CL: a cluster of CTAs per row, no workspace parts and no second launch.
template <int DT, int DP, int HT, bool Q4, bool CL>
__global__ void __launch_bounds__(Shape<DT, DP, HT, Q4>::W * 32, Shape<DT, DP, HT, Q4>::kCtas)
    attn_kernel(AttnArgs a, KvView kv, int head_tiles) {
    using S = Shape<DT, DP, HT, Q4>;
    constexpr int NT = S::NT, KT = S::KT, W = S::W, kThreads = W * 32, kStages = S::kStages;
    extern __shared__ __align__(128) uint8_t smem[];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    pdl_wait();
    const Room room = room_of(a.workspace, a.n_seq, a.h_q, S::kPart, a.acc_out != nullptr);
    const int rows = kv.n_heads * head_tiles;
    __shared__ long long s_total;

    Cursor use;
    int left;           // cost that is left for this CTA; with clusters, tiles
    bool leads = true;  // is this the row at the start of the CTA's range
    if (CL) {
        const int size = cg::this_cluster().num_blocks(), rank = cg::this_cluster().block_rank();
        const int id = blockIdx.x / size;
        use.s = id / rows;
        use.row = id - use.s * rows;
        use.load(a, S::BT);
        use.tile = use.tiles * rank / size;
        left = use.tiles * (rank + 1) / size - use.tile;
        if (threadIdx.x == 0 && rank == 0 && use.row == 0 && a.lens[use.s] > a.n_slots)
            record_status(a.status, kStBadIndex);
    } else {
        // The costs before each thread's share of the sequences, and of all.
        __shared__ long long s_scan[W], s_before;
        __shared__ int s_seq;
        auto cost_of = [&](int s) {
            const Span p = span_of(a, s);
            return max(1, (p.len - p.first + S::BT - 1) / S::BT) + kRowCost;
        };
        const int share = (a.n_seq + kThreads - 1) / kThreads;
        const int s0 = min(a.n_seq, (int)threadIdx.x * share), s1 = min(a.n_seq, s0 + share);
        long long mine = 0;
        for (int s = s0; s < s1; ++s) {
            mine += cost_of(s);
            if (blockIdx.x == 0 && a.lens[s] > a.n_slots)
                record_status(a.status, kStBadIndex);
        }
        long long x = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xFFFFFFFFu, x, o);
            if (lane >= o) x += y;
        }
        if (lane == 31) s_scan[warp] = x;
        __syncthreads();
        long long before = x - mine, total = 0;
        for (int w = 0; w < W; ++w) {
            if (w < warp) before += s_scan[w];
            total += s_scan[w];
        }
        const Sched sched(total * rows, gridDim.x);
        const long long t0 = sched.start(blockIdx.x), t1 = sched.start(blockIdx.x + 1);
        if (threadIdx.x == 0) {
            room.splits[blockIdx.x] = make_int4(0, 0, 0, 0);
            s_total = sched.total;
        }
        if (t0 >= t1) return;
        if (t0 >= before * rows && t0 < (before + mine) * rows) {
            int s = s0;
            for (int n; t0 >= (before + (n = cost_of(s))) * rows; ++s) before += n;
            s_seq = s;
            s_before = before;
        }
        __syncthreads();
        use.s = s_seq;
        use.load(a, S::BT);
        const long long in = t0 - s_before * rows;
        use.row = (int)div_any(in, use.tiles + kRowCost);
        use.tile = (int)(in - (long long)use.row * (use.tiles + kRowCost));
        left = (int)(t1 - t0);
        if (use.tile >= use.tiles) {  // in the end of a row: the CTA before this one's
            leads = false;
            left -= use.tiles + kRowCost - use.tile;
            use.tile = use.tiles - 1;
            if (left > 0) use.next(a, rows, S::BT);
        }
    }
    Cursor fetch = use;  // the tile whose page numbers are asked for next
    int to_fetch = left;

    const uint32_t ring = smem_addr(smem) + warp * kStages * S::kTile;
    float *bias = reinterpret_cast<float *>(smem + S::kBias) + warp * kStages * KT;
    const int live_chunks = kv.head_dim / S::kEpc;

    const long long v_from_k = kv.v - kv.k;

    // Page numbers are asked for one tile ahead of the loads that need them.
    struct Ask {
        int page, in, head;
        float bias;
        bool live;
    };
    auto ask = [&]() {
        Ask k{-1, 0, -1, -INFINITY, false};  // head -1: no tile
        if (to_fetch <= 0) return k;
        to_fetch -= !CL && fetch.tile + 1 == fetch.tiles ? 1 + kRowCost : 1;
        const int j = fetch.span.first + fetch.tile * S::BT + warp * KT + lane;
        if (lane < KT && j < fetch.span.len) {
            const uint32_t p = kv.page_size.div((uint32_t)j);
            k.page = kv.page_table[(long long)fetch.s * kv.max_pages + p];
            k.in = j - (int)(p * kv.page_size.d);
            k.bias = a.mask ? a.mask[fetch.s * a.mask_stride + j] : 0.f;
            k.live = true;
        }
        k.head = head_tiles == 1 ? fetch.row : fetch.row / head_tiles;
        fetch.next(a, rows, S::BT);
        return k;
    };
    auto issue = [&](int stage, const Ask &k) {
        long long at = -1;
        float b = -INFINITY;
        if (k.live) {
            if ((unsigned)k.page >= (unsigned)kv.n_pages) {
                record_status(a.status, kStBadIndex);
            } else if (k.bias != -INFINITY) {
                b = k.bias;
                at = (long long)k.page * kv.page_stride + (long long)k.head * kv.head_stride +
                     (long long)k.in * kv.token_stride;
            }
        }
        // All of the tile's slots are there, and their rows fill the ring's: no checks.
        const bool full = __all_sync(0xFFFFFFFFu, lane >= KT || at >= 0) &&
                          live_chunks == S::kChunks;
        if (!__any_sync(0xFFFFFFFFu, k.live)) return;
        if (lane < KT) bias[stage * KT + lane] = b;
        // Eight lanes copy 128 bytes of a row at a time, four rows at once.
        const uint32_t to = ring + stage * S::kTile + (lane >> 3) * S::kRow;
        const char *const mine = kv.k + (lane & 7) * 16;
        auto copy = [&](auto checked) {
#pragma unroll
            for (int i = 0; i < KT / 4; ++i) {
                const int key = 4 * i + (lane >> 3);
                const long long from = __shfl_sync(0xFFFFFFFFu, at, key);
                const char *k = mine + (!checked || from >= 0 ? from : 0);
                const uint32_t dk = to + 4 * i * S::kRow + (((lane & 7) ^ swizzle_k<DT>(key)) << 4);
                const uint32_t dv = to + (KT + 4 * i) * S::kRow +
                                    (((lane & 7) ^ swizzle_v<DT>(key)) << 4);
                const char *v = k + v_from_k;
#pragma unroll
                for (int u = 0; u < S::kRow / 128; ++u) {
                    const bool live = !checked || (from >= 0 && (lane & 7) + 8 * u < live_chunks);
                    cp_async16(dk + 128 * u, checked && !live ? kv.k : k + 128 * u, live);
                    cp_async16(dv + 128 * u, checked && !live ? kv.k : v + 128 * u, live);
                }
            }
        };
        if (full)
            copy(std::false_type());
        else
            copy(std::true_type());
    };

    // The row's query heads, scaled, as the first product's operand: rows g and g + 8 of a
    // fragment are the first two terms of head g.  In registers where they fit: every warp
    // makes its own.  Else a bf16 head tile is made by one warp, tf32 ones by all.
    uint32_t qr[S::kQReg ? HT * S::kSteps : 1][S::kQWords];
    // Asked for first and turned into operands later, so that other loads go in between.
    constexpr int kRaw = S::kQReg ? HT * S::kSteps * 2
                         : !S::kTf ? S::kSteps * 2
                                   : (HT * S::kSteps * 32 + kThreads - 1) / kThreads;
    float2 raw[kRaw];
    auto fetch_q = [&](const Cursor &at) {
        const int h = at.row / head_tiles, ht0 = (at.row - h * head_tiles) * S::kHeads;
        const float *q0 = a.q + at.s * a.q_stride + ((long long)h * a.group + ht0) * kv.head_dim;
        auto q2 = [&](int head, int dim) {
            return ht0 + head < a.group && dim < kv.head_dim
                       ? *reinterpret_cast<const float2 *>(q0 + head * kv.head_dim + dim)
                       : make_float2(0.f, 0.f);
        };
#pragma unroll
        for (int i = 0; i < kRaw; ++i) {
            if (!S::kTf) {
                const int ht = S::kQReg ? i / (2 * S::kSteps) : warp;
                if (ht >= HT) break;
                raw[i] = q2(ht * 8 + (Q4 ? g & 3 : g), i % (2 * S::kSteps) * 8 + 2 * c);
            } else {  // a lane's dims are those of its registers of a key
                const int f = i * kThreads + threadIdx.x;
                const int l = f & 31, ks = (f >> 5) % S::kSteps, ht = (f >> 5) / S::kSteps;
                const int dim = S::k16 ? 8 * ks + 2 * (l & 3)
                                       : 16 * (ks >> 1) + 4 * (l & 3) + 2 * (ks & 1);
                if (ht < HT) raw[i] = q2(ht * 8 + (Q4 ? l >> 2 & 3 : l >> 2), dim);
            }
        }
    };
    auto make_q = [&]() {
        if (S::kTf) {
#pragma unroll
            for (int i = 0; i < kRaw; ++i) {
                const int f = i * kThreads + threadIdx.x;
                if (f >= HT * S::kSteps * 32) break;
                const bool third = f & 16;  // rows 4 to 7
                uint4 t;
                split_tf32<Q4>(raw[i].x * a.scale, third, t.x, t.y);
                split_tf32<Q4>(raw[i].y * a.scale, third, t.z, t.w);
                *reinterpret_cast<uint4 *>(smem + S::kQ + f * 16) = t;
            }
        }
#pragma unroll
        for (int u = 0; u < (S::kQReg ? HT : S::kTf ? 0 : 1); ++u) {
            const int ht = S::kQReg ? u : warp;
            if (ht >= HT) break;
            const float2 *r = raw + (S::kQReg ? u * S::kSteps * 2 : 0);
#pragma unroll
            for (int ks = 0; ks < S::kSteps; ++ks) {
                uint32_t t0[3], t1[3];
                const float2 x = r[2 * ks], y = r[2 * ks + 1];
                split2(x.x * a.scale, x.y * a.scale, t0);
                split2(y.x * a.scale, y.y * a.scale, t1);
                const int f = ht * S::kSteps + ks;
                if (Q4 && g >= 4) t0[0] = t0[2], t1[0] = t1[2], t0[1] = t1[1] = 0u;
                if (S::kQReg) {
                    uint32_t(&q)[S::kQWords] = qr[S::kQReg ? u * S::kSteps + ks : 0];
                    q[0] = t0[0], q[1] = t0[1], q[2] = t1[0], q[3] = t1[1];
                    if (S::k3) q[4 % S::kQWords] = t0[2], q[5 % S::kQWords] = t1[2];
                } else {
                    *reinterpret_cast<uint4 *>(smem + S::kQ + (f * 32 + lane) * 16) =
                        make_uint4(t0[0], t0[1], t1[0], t1[1]);
                    if (S::k3)
                        *reinterpret_cast<uint2 *>(smem + S::kQ + HT * S::kSteps * 512 +
                                                   (f * 32 + lane) * 8) = make_uint2(t0[2], t1[2]);
                }
            }
        }
    };
    // The first tiles' page numbers and the queries are on their way together, ahead of
    // the tiles, whose loads would hold them up.
    Ask asked[kStages];
#pragma unroll
    for (int st = 0; st < kStages; ++st) asked[st] = ask();
    fetch_q(use);
#pragma unroll
    for (int st = 0; st < kStages; ++st) {
        issue(st, asked[st]);
        cp_async_commit();
    }
    Ask next_ask = ask();
    make_q();
    __syncthreads();
    // The join's blocks wait beside the last of these CTAs.  They in turn let the next kernel
    // in only when they are done: with both early, CTAs of a next call wait beside these and
    // 131072 slots back to back take 130 us in place of 93.
    if (!CL) pdl_launch();

    constexpr int OI = DP / 8;  // 16-bit: o[i] = dims 8 i + 2 c, + 1; f32: see its loop
    float o[HT][OI][2], m[HT], l[HT];
    auto clear = [&]() {
#pragma unroll
        for (int h = 0; h < HT; ++h) {
            m[h] = -INFINITY;
            l[h] = 0.f;
#pragma unroll
            for (int i = 0; i < OI; ++i) o[h][i][0] = o[h][i][1] = 0.f;
        }
    };
    clear();
    bool whole = use.tile == 0;  // does this CTA have the row from its first tile
    int stage = 0;
    const int mat = lane >> 3, mrow = lane & 7;  // ldmatrix: this lane's matrix and row

    // One tile: x = q.k, the softmax step, o = o corr + p.v.
    auto step = [&]() {
        const uint32_t kb = ring + stage * S::kTile, vb = kb + KT * S::kRow;
        const float *bs = bias + stage * KT;
        float sc[HT][NT][2][4] = {};
        if (S::k16) {
            const int key = (mat >> 1) * 8 + mrow;
            const uint32_t at = kb + key * S::kRow;
#pragma unroll
            for (int ks = 0; ks < DP / 16; ++ks) {
                if (2 * ks >= live_chunks) break;
                uint32_t kf[4];
                ldmatrix4<false>(kf, at + (((2 * ks + (mat & 1)) ^ mrow) << 4));
#pragma unroll
                for (int h = 0; h < (S::kTf ? HT : 0); ++h)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {  // even and odd chunks' sums
                        const uint4 v = lds128(smem_addr(smem) + S::kQ +
                                               ((h * S::kSteps + 2 * ks + j) * 32 + lane) * 16);
                        const uint32_t q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                        for (int n = 0; n < NT; ++n) {
                            const uint2 b = widen(kf[2 * n + j]);
                            float(&x)[4] = sc[h][n][j];
                            mma_tf32(x, q, b.x, b.y, x[0], x[1], x[2], x[3]);
                        }
                    }
#pragma unroll
                for (int h = 0; h < (S::kTf ? 0 : HT); ++h) {
                    uint32_t q[6];
                    const int f = h * S::kSteps + ks;
                    if (S::kQReg) {
#pragma unroll
                        for (int i = 0; i < S::kQWords; ++i) q[i] = qr[S::kQReg ? f : 0][i];
                    } else {
                        const uint32_t qa = smem_addr(smem) + S::kQ;
                        const uint4 v = lds128(qa + (f * 32 + lane) * 16);
                        q[0] = v.x, q[1] = v.y, q[2] = v.z, q[3] = v.w;
                        if (S::k3) {
                            const uint2 u = lds64(qa + HT * S::kSteps * 512 + (f * 32 + lane) * 8);
                            q[4] = u.x, q[5] = u.y;
                        }
                    }
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        float(&x)[4] = sc[h][n][0], (&y)[4] = sc[h][n][1];
                        mma_bf16(x, q[0], q[1], q[2], q[3], kf[2 * n], kf[2 * n + 1], x[0], x[1],
                                 x[2], x[3]);
                        if (S::k3)
                            mma_bf16(y, q[4], 0u, q[5], 0u, kf[2 * n], kf[2 * n + 1], y[0], y[1],
                                     y[2], y[3]);
                    }
                }
            }
        } else {
            float lo[HT][2][4] = {};
#pragma unroll
            for (int i = 0; i < S::kChunks / 4; ++i) {
                if (4 * i >= live_chunks) break;
                const uint4 v = lds128(kb + g * S::kRow + (((4 * i + c) ^ swizzle_k<DT>(g)) << 4));
                const Cut k[4] = {cut3(v.x), cut3(v.y), cut3(v.z), cut3(v.w)};
#pragma unroll
                for (int h = 0; h < HT; ++h)
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const uint4 f = lds128(smem_addr(smem) + S::kQ +
                                               ((h * S::kSteps + 2 * i + j) * 32 + lane) * 16);
                        const uint32_t q[4] = {f.x, f.y, f.z, f.w};
                        // Four sums: high and low parts, even and odd steps.
                        float(&x)[4] = sc[h][0][j], (&y)[4] = lo[h][j];
                        const Cut &b0 = k[2 * j], &b1 = k[2 * j + 1];
                        mma_tf32(x, q, b0.t[0], b1.t[0], x[0], x[1], x[2], x[3]);
                        mma_tf32(y, q, b0.t[2], b1.t[2], y[0], y[1], y[2], y[3]);
                        mma_tf32(y, q, b0.t[1], b1.t[1], y[0], y[1], y[2], y[3]);
                    }
            }
#pragma unroll
            for (int h = 0; h < HT; ++h)
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) sc[h][0][j][i] += lo[h][j][i];
        }
        // Is there a k that is not finite in a slot of the tile (f16)?
        auto endless = [&](int slot) {
            bool any = false;
            for (int ch = 0; ch < live_chunks; ++ch) {
                const uint4 v = lds128(kb + slot * S::kRow + ((ch ^ swizzle_k<DT>(slot)) << 4));
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    any |= (w[i] & 0x7C00u) == 0x7C00u || (w[i] & 0x7C000000u) == 0x7C000000u;
            }
            return any;
        };
        uint32_t pt[HT][2][3];   // bf16: the terms of p at slots 2c, 2c + 1 (+ 8)
        uint32_t pf[HT][NT][4];  // tf32: p's fragments
        float corr[HT];
#pragma unroll
        for (int h = 0; h < HT; ++h) {
            float xs[NT][2], top = m[h];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float2 b = *reinterpret_cast<const float2 *>(bs + n * 8 + 2 * c);
                const float(&v)[2][4] = sc[h][n];
                float x0 = (v[0][0] + v[1][0]) + (v[0][2] + v[1][2]);
                float x1 = (v[0][1] + v[1][1]) + (v[0][3] + v[1][3]);
                if (DT == kF16 && !Q4) {
                    if (x0 == -INFINITY && endless(n * 8 + 2 * c)) x0 = NAN;
                    if (x1 == -INFINITY && endless(n * 8 + 2 * c + 1)) x1 = NAN;
                }
                if (Q4) {  // heads 0 to 3 now also in the lanes of rows 4 to 7
                    x0 += __shfl_xor_sync(0xFFFFFFFFu, x0, 16);
                    x1 += __shfl_xor_sync(0xFFFFFFFFu, x1, 16);
                }
                xs[n][0] = b.x == -INFINITY ? -INFINITY : x0 + b.x;
                xs[n][1] = b.y == -INFINITY ? -INFINITY : x1 + b.y;
                top = fmaxf(top, fmaxf(xs[n][0], xs[n][1]));
            }
            if (a.acc_out) {  // every score, for the weight sums
                const int hr = use.row / head_tiles;
                const int head = (use.row - hr * head_tiles) * S::kHeads + h * 8 + g;
                if (head < a.group) {
                    float *to = room.scores +
                                ((long long)use.s * a.h_q + hr * a.group + head) * a.n_slots;
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        const int j = use.span.first + use.tile * S::BT + warp * KT + n * 8 + 2 * c;
                        if (!((use.span.first | a.n_slots) & 1) && j + 1 < use.span.len) {
                            *reinterpret_cast<float2 *>(to + j) = make_float2(xs[n][0], xs[n][1]);
                        } else {
                            if (j < use.span.len) to[j] = xs[n][0];
                            if (j + 1 < use.span.len) to[j + 1] = xs[n][1];
                        }
                    }
                }
            }
            top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
            corr[h] = exp_diff(m[h], top);
            m[h] = top;
            float sum = 0.f;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float p0 = exp_diff(xs[n][0], top), p1 = exp_diff(xs[n][1], top);
                sum += p0 + p1;
                if (S::kTf) {
                    split_tf32<Q4>(p0, g >= 4, pf[h][n][0], pf[h][n][1]);
                    split_tf32<Q4>(p1, g >= 4, pf[h][n][2], pf[h][n][3]);
                } else {
                    split2(p0, p1, pt[h][n]);
                    if (Q4 && g >= 4) pt[h][n][0] = pt[h][n][2], pt[h][n][1] = 0u;
                }
            }
            l[h] = l[h] * corr[h] + sum;
        }
        if (S::k16) {
            const int key = (mat & 1) * 8 + mrow;
            const uint32_t at = vb + key * S::kRow;
            // Four independent products at a time.
#pragma unroll
            for (int i = 0; i < DP / 16; i += 2) {
                if (2 * i >= live_chunks) break;
                uint32_t vf[8];
#pragma unroll
                for (int u = 0; u < 2; ++u)
                    ldmatrix4<true>(reinterpret_cast<uint32_t(&)[4]>(vf[4 * u]),
                                    at + (((2 * (i + u) + (mat >> 1)) ^ mrow) << 4));
#pragma unroll
                for (int h = 0; h < HT; ++h) {
                    const uint32_t(&p0)[3] = pt[h][0], (&p1)[3] = pt[h][1];
                    float t[4][4];
                    if (S::kTf) {
#pragma unroll
                        for (int n = 0; n < NT; ++n)
#pragma unroll
                            for (int u = 0; u < 4; ++u) {
                                const uint2 b = widen(vf[2 * u + n]);
                                if (n == 0)
                                    mma_tf32(t[u], pf[h][n], b.x, b.y, 0.f, 0.f, 0.f, 0.f);
                                else
                                    mma_tf32(t[u], pf[h][n], b.x, b.y, t[u][0], t[u][1], t[u][2],
                                             t[u][3]);
                            }
                    } else {
#pragma unroll
                        for (int u = 0; u < 4; ++u)
                            mma_bf16(t[u], p0[0], p0[1], p1[0], p1[1], vf[2 * u], vf[2 * u + 1],
                                     0.f, 0.f, 0.f, 0.f);
                    }
                    if (S::k3)
#pragma unroll
                        for (int u = 0; u < 4; ++u)
                            mma_bf16(t[u], p0[2], 0u, p1[2], 0u, vf[2 * u], vf[2 * u + 1],
                                     t[u][0], t[u][1], t[u][2], t[u][3]);
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        float(&to)[2] = o[h][2 * i + u];
                        to[0] = to[0] * corr[h] + (t[u][0] + t[u][2]);
                        to[1] = to[1] * corr[h] + (t[u][1] + t[u][3]);
                    }
                }
            }
        } else {
            // Column g of product e is dim 4 (g + 8 i) + e.
#pragma unroll
            for (int i = 0; i < S::kChunks / 8; ++i) {
                if (8 * i >= live_chunks) break;
                const uint32_t at = vb + 2 * c * S::kRow + (((g + 8 * i) ^ (2 * c)) << 4);
                const uint4 v0 = lds128(at), v1 = lds128(at + S::kRow);
                const Cut c0[4] = {cut3(v0.x), cut3(v0.y), cut3(v0.z), cut3(v0.w)};
                const Cut c1[4] = {cut3(v1.x), cut3(v1.y), cut3(v1.z), cut3(v1.w)};
#pragma unroll
                for (int h = 0; h < HT; ++h) {
                    float t[4][4] = {};
#pragma unroll
                    for (int part = 2; part >= 0; --part)  // the small ones first
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            mma_tf32(t[e], pf[h][0], c0[e].t[part], c1[e].t[part], t[e][0],
                                     t[e][1], t[e][2], t[e][3]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float(&to)[2] = o[h][i * 4 + e];
                        to[0] = to[0] * corr[h] + (t[e][0] + t[e][2]);
                        to[1] = to[1] * corr[h] + (t[e][1] + t[e][3]);
                    }
                }
            }
        }
    };

    float *s_m = reinterpret_cast<float *>(smem + S::kM);
    float *s_l = reinterpret_cast<float *>(smem + S::kL);
    float *s_top = reinterpret_cast<float *>(smem + S::kTop);
    float *s_sum = reinterpret_cast<float *>(smem + S::kSum);
    auto slot_of = [&](int w) {  // a warp's tile just used, for its o
        return reinterpret_cast<float *>(smem + (w * kStages + stage) * S::kTile);
    };
    // The warps' parts through shared memory: afterwards s_m holds the warps' factors and
    // s_top, s_sum the joined m and l of each head.
    auto meet = [&]() {
        __syncwarp();  // every lane has read the tile
        float *mo = slot_of(warp);
#pragma unroll
        for (int h = 0; h < HT; ++h) {
            float sum = l[h];
            sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
            sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2);
            if (c == 0) {
                s_m[warp * S::kHeads + h * 8 + g] = m[h];
                s_l[warp * S::kHeads + h * 8 + g] = sum;
            }
            float *to = mo + (h * 8 + g) * DP;
            if (Q4) {
#pragma unroll
                for (int i = 0; i < OI; ++i)
#pragma unroll
                    for (int e = 0; e < 2; ++e)
                        o[h][i][e] += __shfl_xor_sync(0xFFFFFFFFu, o[h][i][e], 16);
            }
            if (S::k16) {
#pragma unroll
                for (int i = 0; i < OI; ++i)
                    *reinterpret_cast<float2 *>(to + 8 * i + 2 * c) =
                        make_float2(o[h][i][0], o[h][i][1]);
            } else {
#pragma unroll
                for (int i = 0; i < S::kChunks / 8; ++i)
#pragma unroll
                    for (int v = 0; v < 2; ++v)
                        *reinterpret_cast<float4 *>(to + 4 * (2 * c + v + 8 * i)) =
                            make_float4(o[h][i * 4][v], o[h][i * 4 + 1][v], o[h][i * 4 + 2][v],
                                        o[h][i * 4 + 3][v]);
            }
        }
        __syncthreads();
        if (threadIdx.x < S::kHeads) {
            float top = -INFINITY, sum = 0.f;
#pragma unroll
            for (int w = 0; w < W; ++w) top = fmaxf(top, s_m[w * S::kHeads + threadIdx.x]);
#pragma unroll
            for (int w = 0; w < W; ++w) {
                const float f = exp_diff(s_m[w * S::kHeads + threadIdx.x], top);
                sum += f * s_l[w * S::kHeads + threadIdx.x];
                s_m[w * S::kHeads + threadIdx.x] = f;
            }
            s_top[threadIdx.x] = top;
            s_sum[threadIdx.x] = sum;
        }
        __syncthreads();
    };
    // Four dims of the joined o.
    auto joined = [&](int head, int idx4) {
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const float f = s_m[w * S::kHeads + head];
            const float4 x = reinterpret_cast<const float4 *>(slot_of(w))[idx4];
            v.x += f * x.x;
            v.y += f * x.y;
            v.z += f * x.z;
            v.w += f * x.w;
        }
        return v;
    };
    auto is_none = [](float top, float sum) { return top == -INFINITY && sum == 0.f; };
    // out of four dims from dim `dim` of a head, and its lse at dim 0.
    auto finish = [&](const Cursor &at, int head, int dim, float4 v, float top, float sum) {
        const int hr = at.row / head_tiles;
        const int in_group = (at.row - hr * head_tiles) * S::kHeads + head;
        if (in_group >= a.group || dim >= kv.head_dim) return;
        const int qh = hr * a.group + in_group;
        const float inv = is_none(top, sum) ? 0.f : 1.f / sum;
        *reinterpret_cast<float4 *>(a.out + at.s * a.out_stride + (long long)qh * kv.head_dim +
                                    dim) =
            is_none(top, sum) ? make_float4(0.f, 0.f, 0.f, 0.f)
                              : make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
        if (dim == 0) {
            const float e = is_none(top, sum) ? -INFINITY : top + logf(sum);
            const long long to = (long long)at.s * a.h_q + qh;
            if (a.lse) a.lse[to] = e;
            if (!CL && a.acc_out) room.lse[to] = e;
        }
    };

    // The CTA of the last tile of the row that this CTA leaves unfinished.
    auto owner_of_end = [&]() {
        const Sched sched(s_total, gridDim.x);
        return sched.owner(sched.start(blockIdx.x + 1) - 1 + (use.tiles - 1 - use.tile));
    };

    const int first_tile = use.tile;
    while (left > 0) {
        cp_async_wait<kStages - 1>();
        __syncwarp();
        // A warp beyond the row's last slot has nothing in its tile, nor asked for it.
        if (use.span.first + use.tile * S::BT + warp * KT < use.span.len) step();
        const bool ends = use.tile + 1 == use.tiles;
        left -= !CL && ends ? 1 + kRowCost : 1;
        const bool last = left <= 0;
        if (!CL && (ends || last)) {
            meet();
            const bool begins = whole;  // the row's first tile is this CTA's
            whole = whole && ends;
            float *part = room.parts + (2ll * blockIdx.x + (leads ? 0 : 1)) * S::kPart;
            for (int i = threadIdx.x; i < S::kHeads * DP / 4; i += kThreads) {
                const int head = i / (DP / 4), dim = i % (DP / 4) * 4;
                const float4 v = joined(head, i);
                if (whole)
                    finish(use, head, dim, v, s_top[head], s_sum[head]);
                else
                    reinterpret_cast<float4 *>(part + 2 * S::kHeads)[i] = v;
            }
            if (!whole && threadIdx.x < S::kHeads) {
                part[threadIdx.x] = s_top[threadIdx.x];
                part[S::kHeads + threadIdx.x] = s_sum[threadIdx.x];
            }
            if (begins && threadIdx.x == 0) {
                const int n = ends ? 1 : owner_of_end() - (int)blockIdx.x + 1;
                if (n > 1) room.splits[blockIdx.x] = make_int4(use.s, use.row, n, leads ? 0 : 1);
                if (a.acc_out || (long long)a.n_seq * rows <= gridDim.x)
                    room.rows[(long long)use.s * rows + use.row] =
                        make_int4(blockIdx.x, n, leads ? 0 : 1, 0);
            }
            clear();
            leads = false;
            whole = true;
            if (!last) {
                Cursor nx = use;
                nx.next(a, rows, S::BT);
                fetch_q(nx);
                make_q();
            }
            __syncthreads();
        }
        if (!CL || !last) {
            use.next(a, rows, S::BT);
            __syncwarp();
            if (next_ask.head >= 0) issue(stage, next_ask);
            cp_async_commit();
            next_ask = ask();
            stage = stage + 1 == kStages ? 0 : stage + 1;
        }
    }
    if (CL) pdl_launch();
    cp_async_wait<0>();
    if (CL) {
        // Every CTA of the cluster, also one without tiles, shows its part; each then joins
        // and writes its share of the dims.
        cg::cluster_group cluster = cg::this_cluster();
        const int size = cluster.num_blocks(), rank = cluster.block_rank();
        __syncthreads();
        meet();
        float4 *mine = reinterpret_cast<float4 *>(slot_of(0));
        for (int i = threadIdx.x; i < S::kHeads * DP / 4; i += kThreads)
            mine[i] = joined(i / (DP / 4), i);  // reads the same elements that it replaces
        // The slot's place depends on the tiles that a CTA had: all go to one place.
        float4 *shown = reinterpret_cast<float4 *>(smem);
        if (stage != 0) {
            for (int i = threadIdx.x; i < S::kHeads * DP / 4; i += kThreads) shown[i] = mine[i];
        }
        cluster.sync();
        auto join_heads = [&](int head, float &top, float &sum) {
            top = -INFINITY;
            for (int r = 0; r < size; ++r)
                top = fmaxf(top, *cluster.map_shared_rank(s_top + head, r));
            sum = 0.f;
            for (int r = 0; r < size; ++r)
                sum += exp_diff(*cluster.map_shared_rank(s_top + head, r), top) *
                       *cluster.map_shared_rank(s_sum + head, r);
        };
        const int quads = S::kHeads * DP / 4;
        for (int i = rank * kThreads + threadIdx.x; i < quads; i += size * kThreads) {
            const int head = i / (DP / 4), dim = i % (DP / 4) * 4;
            float top, sum;
            join_heads(head, top, sum);
            float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int r = 0; r < size; ++r) {
                const float f = exp_diff(*cluster.map_shared_rank(s_top + head, r), top);
                const float4 x = *cluster.map_shared_rank(shown + i, r);
                v.x += f * x.x;
                v.y += f * x.y;
                v.z += f * x.z;
                v.w += f * x.w;
            }
            finish(use, head, dim, v, top, sum);
        }
        if (a.acc_out) {
            // The weights of this CTA's own slots (head_tiles is 1), from its own scores.
            float *s_lse = s_l;
            if (threadIdx.x < S::kHeads) {
                float top, sum;
                join_heads(threadIdx.x, top, sum);
                s_lse[threadIdx.x] = is_none(top, sum) ? -INFINITY : top + logf(sum);
            }
            __syncthreads();
            const long long at = ((long long)use.s * kv.n_heads + use.row) * a.acc_stride;
            const float *sc = room.scores + ((long long)use.s * a.h_q + use.row * a.group) * a.n_slots;
            const int tile1 = use.tiles * (rank + 1) / size;
            const int j0 = rank == 0 ? 0 : use.span.first + first_tile * S::BT;
            const int j1 = min(use.span.len, use.span.first + tile1 * S::BT);
            for (int j = j0 + threadIdx.x; j < j1; j += kThreads) {
                float w = 0.f;
                if (j >= use.span.first)
                    for (int i = 0; i < a.group; ++i)
                        if (s_lse[i] != -INFINITY)
                            w += exp_diff(sc[(long long)i * a.n_slots + j], s_lse[i]);
                a.acc_out[at + j] = (a.acc_in ? a.acc_in[at + j] : 0.f) + w;
            }
        }
        cluster.sync();  // no CTA's shared memory goes while another reads it
    }
}

constexpr int kJoinAtOnce = 64;  // parts whose m and l a warp asks for at once

// m and l of a row's head joined over n parts by one warp; the parts' factors go to f if given.
template <typename Part>
__device__ __forceinline__ void join_head(int n, int head, int heads, Part part, float *f,
                                          float &top, float &sum) {
    const int lane = threadIdx.x & 31;
    constexpr int kAtOnce = kJoinAtOnce / 32;
    float m[kAtOnce], l[kAtOnce];  // the first parts'
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
        const int i = lane + 32 * u;
        m[u] = i < n ? part(i)[head] : -INFINITY;
        l[u] = i < n ? part(i)[heads + head] : 0.f;
    }
    top = fmaxf(m[0], m[1]);
    for (int i = lane + kJoinAtOnce; i < n; i += 32) top = fmaxf(top, part(i)[head]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
    sum = 0.f;
#pragma unroll
    for (int u = 0; u < kAtOnce; ++u) {
        const float x = exp_diff(m[u], top);
        if (f && lane + 32 * u < n) f[lane + 32 * u] = x;
        sum += x * l[u];
    }
    for (int i = lane + kJoinAtOnce; i < n; i += 32) {
        const float x = exp_diff(part(i)[head], top);
        if (f) f[i] = x;
        sum += x * part(i)[heads + head];
    }
    sum = warp_sum(sum);
}

__device__ __forceinline__ float lse_of(float top, float sum) {
    return top == -INFINITY && sum == 0.f ? -INFINITY : top + logf(sum);
}

// After the split kernel.  The first `joins` blocks join the parts of the rows that several
// CTAs shared: each row where there are no more rows than CTAs, else the row that a CTA begins.
// With few rows a block is a head of a row and its warps share the parts;
// with more a block is a row, a warp joins a head of a few parts, and the block's warps meet
// for a head of many.
// The other blocks sum the weights, acc_out[s][h][j] = acc_in + sum over the group's heads of
// exp(x_j - lse): block (sequence and kv head, piece of the slots).  All are chains of loads
// that wait for one another, so whatever does not wait (the parts' o, the scores) is asked for
// before it is known what it is worth.  MANY: rows have over 64 parts on average.
// SLOTS: of a thread; sixteen scores of them are in flight (one after another of a slot's heads,
// four at a time, took 47 us for a group of 32 over 20000 slots, this 40).
constexpr int kJoinWarps = 8, kAhead = 4, kFewParts = 16;
constexpr int kLse = 1024;  // heads whose lse a block holds at a time, for the weight sums
constexpr int piece_of(int slots) { return slots * kJoinWarps * 32; }
template <bool MANY, int SLOTS>
__global__ void __launch_bounds__(kJoinWarps * 32, 4)
    attn_join_kernel(AttnArgs a, int n_heads, int head_dim, int head_tiles, int heads, int dp,
                     int grid, int joins, int blocks_per_row, int pieces) {
    __shared__ float s_f[kMaxCtas];
    __shared__ float4 s_o[kJoinWarps][64];
    __shared__ float s_red[2], s_top[MANY ? kJoinWarps : 1][16], s_sum[MANY ? kJoinWarps : 1][16];
    __shared__ float s_lse[kLse];
    pdl_wait();
    const int part_floats = heads * (dp + 2);
    const Room room =
        room_of(a.workspace, a.n_seq, a.h_q, part_floats, a.acc_out != nullptr);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rows = n_heads * head_tiles;
    if ((int)blockIdx.x < joins) {
        const bool by_rows = (long long)a.n_seq * rows <= grid;
        const int item = blockIdx.x / blocks_per_row;
        const int4 r = by_rows ? room.rows[item] : room.splits[item];
        const int s = by_rows ? item / rows : r.x, row = by_rows ? item - s * rows : r.y;
        const int first = by_rows ? r.x : item, n = by_rows ? r.y : r.z;
        const int skip = by_rows ? r.z : r.w;
        if (n <= 1) return;  // written by its CTA, or no row
        const int h = row / head_tiles, head0 = (row - h * head_tiles) * heads;
        const int quads = head_dim / 4;
        auto part = [&](int i) {
            return room.parts + (2ll * (first + i) + (i == 0 ? skip : 0)) * part_floats;
        };
        auto o_of = [&](int i, int head, int q) {
            return *reinterpret_cast<const float4 *>(part(i) + 2 * heads + head * dp + 4 * q);
        };
        auto add = [](float4 &v, const float4 &x, float f) {
            v.x += f * x.x;
            v.y += f * x.y;
            v.z += f * x.z;
            v.w += f * x.w;
        };
        auto store = [&](int head, int q, const float4 &v, float top, float sum) {
            const bool none = top == -INFINITY && sum == 0.f;
            const float inv = none ? 0.f : 1.f / sum;
            const int qh = h * a.group + head0 + head;
            *reinterpret_cast<float4 *>(a.out + s * a.out_stride + (long long)qh * head_dim +
                                        4 * q) =
                none ? make_float4(0.f, 0.f, 0.f, 0.f)
                     : make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
            if (q == 0 && a.lse) a.lse[(long long)s * a.h_q + qh] = lse_of(top, sum);
        };
        const bool by_head = blocks_per_row > 1;
        if (!by_head && n <= kFewParts) {
            for (int head = warp; head < heads && head0 + head < a.group; head += kJoinWarps) {
                float4 ahead[kAhead];
#pragma unroll
                for (int u = 0; u < kAhead; ++u)
                    if (u < n && lane < quads) ahead[u] = o_of(u, head, lane);
                float *f = s_f + warp * kFewParts, top, sum;
                join_head(n, head, heads, part, f, top, sum);
                __syncwarp();
                for (int q = lane; q < quads; q += 32) {
                    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                    const int from = q == lane ? kAhead : 0;
#pragma unroll
                    for (int u = 0; u < kAhead; ++u)
                        if (u < n && u < from) add(v, ahead[u], f[u]);
                    for (int i = from; i < n; ++i) add(v, o_of(i, head, q), f[i]);
                    store(head, q, v, top, sum);
                }
                __syncwarp();
            }
            return;
        }
        const int head1 = by_head ? blockIdx.x - item * blocks_per_row : 0;
        const int head2 = by_head ? head1 + 1 : heads;
        for (int head = head1; head < head2 && head0 + head < a.group; ++head) {
            float4 ahead[kAhead];  // this warp's first parts of dims 4 lane ..
#pragma unroll
            for (int u = 0; u < kAhead; ++u)
                if (warp + u * kJoinWarps < n && lane < quads)
                    ahead[u] = o_of(warp + u * kJoinWarps, head, lane);
            if (warp == 0) {
                float top, sum;
                join_head(n, head, heads, part, s_f, top, sum);
                if (lane == 0) {
                    s_red[0] = top;
                    s_red[1] = sum;
                }
            }
            __syncthreads();
            const float top = s_red[0], sum = s_red[1];
            for (int q = lane; q < quads; q += 32) {
                float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
                int i = warp;
                if (q == lane) {
#pragma unroll
                    for (int u = 0; u < kAhead; ++u, i += kJoinWarps)
                        if (i < n) add(v, ahead[u], s_f[i]);
                }
#pragma unroll 4
                for (; i < n; i += kJoinWarps) add(v, o_of(i, head, q), s_f[i]);
                s_o[warp][q] = v;
            }
            __syncthreads();
            for (int q = threadIdx.x; q < quads; q += kJoinWarps * 32) {
                float4 v = s_o[0][q];
#pragma unroll
                for (int w = 1; w < kJoinWarps; ++w) add(v, s_o[w][q], 1.f);
                store(head, q, v, top, sum);
            }
            __syncthreads();  // s_f, s_o and s_red are the next head's
        }
        return;
    }

    const int id = (blockIdx.x - joins) / pieces, piece = blockIdx.x - joins - id * pieces;
    const int s = id / n_heads, h = id - s * n_heads;
    const Span span = span_of(a, s);
    const int j0 = piece * piece_of(SLOTS) + threadIdx.x;
    if (piece * piece_of(SLOTS) >= span.len) return;
    const long long q0 = (long long)s * a.h_q + h * a.group;
    const long long at = (long long)id * a.acc_stride;
    constexpr int kHeadsAhead = 16 / SLOTS;
    float ahead[SLOTS][kHeadsAhead], w[SLOTS];
    auto ask = [&](int i0) {  // the scores of slots that take part; the others have none
#pragma unroll
        for (int u = 0; u < SLOTS; ++u) {
            const int j = j0 + u * kJoinWarps * 32;
            const bool live = j < span.len && j >= span.first;
#pragma unroll
            for (int i = 0; i < kHeadsAhead; ++i)
                ahead[u][i] = live && i0 + i < a.group
                                  ? room.scores[(q0 + i0 + i) * a.n_slots + j] : -INFINITY;
        }
    };
#pragma unroll
    for (int u = 0; u < SLOTS; ++u) {
        const int j = j0 + u * kJoinWarps * 32;
        w[u] = a.acc_in && j < span.len ? a.acc_in[at + j] : 0.f;
    }
    ask(0);
    // The group's lse: whole rows have theirs, and of a row of few parts a warp joins a head.
    // MANY: a lane joins a head of every (8 * 32 / heads)-th part: their m and l are short runs
    // of neighbours, of which a warp to a head reads a sector for each value (120000 slots, a
    // row of 8 heads in 456 parts: 27 us, 55 by warps; 57 parts: 58 and 57; 2 parts 16 and 14).
    float sum[SLOTS] = {};
    for (int g0 = 0; g0 < a.group; g0 += kLse) {
        const int g1 = min(a.group, g0 + kLse);
        if (g0 > 0) __syncthreads();  // the heads before have been read
        for (int ht = g0 / heads; ht * heads < g1; ++ht) {
            const int4 row = room.rows[(long long)id * head_tiles + ht];
            const int first = row.x, n = row.y, skip = row.z;
            const int in_tile = min(heads, a.group - ht * heads);
            float *lse = s_lse + ht * heads - g0;
            auto part = [&](int k) {
                return room.parts + (2ll * (first + k) + (k == 0 ? skip : 0)) * part_floats;
            };
            if (!MANY || n <= 1) {
                for (int head = warp; head < in_tile; head += kJoinWarps) {
                    const float whole = room.lse[q0 + ht * heads + head];  // unused if split
                    float top, sum;
                    if (n > 1) join_head(n, head, heads, part, (float *)nullptr, top, sum);
                    if (lane == 0) lse[head] = n > 1 ? lse_of(top, sum) : whole;
                }
                continue;
            }
            const int per = 32 / heads, head = lane & (heads - 1);
            float top = -INFINITY, sum = 0.f;
            auto join = [&](float m, float l) {
                const float t = fmaxf(top, m);
                sum = sum * exp_diff(top, t) + l * exp_diff(m, t);
                top = t;
            };
            for (int k0 = warp * per + lane / heads; k0 < n; k0 += kAhead * kJoinWarps * per) {
                float m[kAhead], l[kAhead];
#pragma unroll
                for (int u = 0; u < kAhead; ++u) {
                    const int k = k0 + u * kJoinWarps * per;
                    m[u] = k < n ? part(k)[head] : -INFINITY;
                    l[u] = k < n ? part(k)[heads + head] : 0.f;
                }
#pragma unroll
                for (int u = 0; u < kAhead; ++u) join(m[u], l[u]);
            }
            for (int o = heads; o < 32; o <<= 1) {
                const float m = __shfl_xor_sync(0xFFFFFFFFu, top, o);
                const float l = __shfl_xor_sync(0xFFFFFFFFu, sum, o);
                join(m, l);
            }
            __syncthreads();  // the tile before has been read
            if (lane < heads) s_top[warp][head] = top, s_sum[warp][head] = sum;
            __syncthreads();
            if (warp == 0 && lane < in_tile) {
                for (int w = 1; w < kJoinWarps; ++w) join(s_top[w][head], s_sum[w][head]);
                lse[head] = lse_of(top, sum);
            }
        }
        __syncthreads();
        for (int i0 = g0; i0 < g1; i0 += kHeadsAhead) {
#pragma unroll
            for (int i = 0; i < kHeadsAhead; ++i) {
                const float e = i0 + i < g1 ? s_lse[i0 + i - g0] : -INFINITY;
#pragma unroll
                for (int u = 0; u < SLOTS; ++u)
                    if (e != -INFINITY) sum[u] += exp_diff(ahead[u][i], e);
            }
            if (i0 + kHeadsAhead < a.group) ask(i0 + kHeadsAhead);
        }
    }
#pragma unroll
    for (int u = 0; u < SLOTS; ++u) {
        const int j = j0 + u * kJoinWarps * 32;
        if (j < span.len) a.acc_out[at + j] = w[u] + sum[u];
    }
}

// 16 query heads a row where a group has more than 8 (the cache is then read half as often),
// while o (registers) and q (shared memory) leave room for it; 8 otherwise.
int head_tile(int group, int dp, int dtype) {
    return group > 8 && dp <= (dtype == kF32 ? 64 : 128) ? 2 : 1;
}
int padded_dim(int d) { return d <= 64 ? 64 : d <= 128 ? 128 : 256; }

struct Plan {
    int head_tiles, cluster;  // cluster 0: the split kernel and the join
    int grid, tile;
};

template <int DT, int DP, int HT, bool Q4 = false>
cudaError_t launch_shape(const AttnArgs &a, const KvView &kv, const DeviceInfo &dev,
                         cudaStream_t stream) {
    using S = Shape<DT, DP, HT, Q4>;
    const int head_tiles = (a.group + S::kHeads - 1) / S::kHeads;
    const long long rows = (long long)a.n_seq * kv.n_heads * head_tiles;
    const int slots = min(kMaxCtas, S::kCtas * dev.sm_count);
    if (rows > 0x7FFFFFFFll / 8) return cudaErrorInvalidConfiguration;

    // A cluster per row, no parts and no second launch, while all rows' CTAs are resident and a
    // CTA has at most four tiles, or two where its cluster is of eight: there the split
    // kernel has SMs to spare.  More CTAs to a row while one per SM is not reached, or two
    // where one has over two tiles.  Cluster and split, us, by a CTA's tiles:
    //                                         1          2          3          4
    //   32/8 of 128 bf16,  8 rows (of 8)  7.3  8.7   8.8  9.3  10.1  9.5  11.5  9.9
    //                     32 rows (of 8)  7.5  9.6  10.8 12.0  12.4 12.7  14.1 13.8
    //                     96 rows (of 4)            10.6 12.9  12.1 14.0  13.9 15.8
    //                    256 rows (of 1)  8.5  9.0  10.3 12.1  11.8 13.5  13.6 14.9
    //                    800 rows (of 1) 15.7 14.2  19.3 19.0  22.4 22.5  27.8 27.8
    //   16/16 of 64 f16,  16 rows (of 8)  7.2  8.5   8.4  9.5   9.6  9.1  10.9 10.6
    //                    192 rows (of 2)  6.8  7.7   9.0 11.6  10.4 12.8  11.8 14.3
    //                    512 rows (of 1) 12.5 10.2  15.1 12.9  17.9 14.3  20.7 16.3
    //   16/4 of 256 bf16,  4 rows (of 8)  8.6 10.6  10.6 10.8  12.4 11.1  14.4 11.1
    //                    128 rows (of 2)            12.9 15.6  14.9 18.3  17.1 20.3
    //   32/2 of 256 f32,   4 rows (of 8)  9.3 11.2  12.1 11.5  14.8 11.9  17.6 12.2
    //                    128 rows (of 2)            15.6 19.7  19.1 22.9  22.4 26.2
    // The cache's size stands for the lengths, which are not known here.
    const long long span = a.window > 0 && a.window < a.n_slots ? a.window : a.n_slots;
    int cluster = 1;
    while (cluster < 8 && rows * cluster * 2 <= slots && span > cluster * S::BT &&
           (rows * cluster * 2 <= dev.sm_count || span > 2 * cluster * S::BT))
        cluster *= 2;
    const bool small = rows * cluster <= slots &&
                       span <= (cluster == 8 ? 2ll : 4ll) * cluster * S::BT &&
                       (!a.acc_out || head_tiles == 1);
    if (small) {
        static std::atomic<unsigned long long> done{0};
        cudaError_t err = ensure_smem(attn_kernel<DT, DP, HT, Q4, true>, S::kSmem, dev, done);
        if (err != cudaSuccess) return err;
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3((unsigned)(rows * cluster));
        cfg.blockDim = dim3(S::W * 32);
        cfg.dynamicSmemBytes = S::kSmem;
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
        return cudaLaunchKernelEx(&cfg, attn_kernel<DT, DP, HT, Q4, true>, a, kv, head_tiles);
    }
    static std::atomic<unsigned long long> done{0};
    cudaError_t err = ensure_smem(attn_kernel<DT, DP, HT, Q4, false>, S::kSmem, dev, done);
    if (err != cudaSuccess) return err;
    // A block of the join is a head of a row while two of them per SM are not reached (131072
    // slots, 8 rows of 4 heads 91 us, a row each 98; 4 sequences of 16384, 32 rows of 8 heads
    // 35 and 43; beyond, 16 of 4096 38 and 36, 32 of 4096 64 and 58).
    const int row_heads = min(a.group, S::kHeads);
    const int blocks_per_row = rows * row_heads <= 2 * dev.sm_count ? row_heads : 1;
    const int joins = (int)(rows <= slots ? rows : slots) * blocks_per_row;
    const int slots_per = a.n_slots <= piece_of(1) ? 1 : 4;
    const int pieces =
        a.acc_out ? (int)((a.n_slots + (long long)piece_of(slots_per) - 1) / piece_of(slots_per)) : 0;
    const long long blocks = joins + (long long)a.n_seq * kv.n_heads * pieces;
    if (blocks > 0x7FFFFFFFll) return cudaErrorInvalidConfiguration;
    err = launch_pdl(attn_kernel<DT, DP, HT, Q4, false>, dim3(slots), dim3(S::W * 32), S::kSmem, stream,
                     a, kv, head_tiles);
    if (err != cudaSuccess) return err;
    const bool many = rows * kJoinAtOnce < slots;
    return launch_pdl(slots_per == 1 ? attn_join_kernel<false, 1>
                      : many         ? attn_join_kernel<true, 4>
                                     : attn_join_kernel<false, 4>,
                      dim3((unsigned)blocks), dim3(kJoinWarps * 32), 0, stream, a, kv.n_heads,
                      kv.head_dim, head_tiles, S::kHeads, DP, slots, joins, blocks_per_row, pieces);
}

template <int DT>
cudaError_t launch_type(const AttnArgs &a, const KvView &kv, const DeviceInfo &dev,
                        cudaStream_t stream) {
    const int dp = padded_dim(kv.head_dim), ht = head_tile(a.group, dp, DT);
    if constexpr (DT != kF32)
        if (a.group <= 4)
            return dp == 64    ? launch_shape<DT, 64, 1, true>(a, kv, dev, stream)
                   : dp == 128 ? launch_shape<DT, 128, 1, true>(a, kv, dev, stream)
                               : launch_shape<DT, 256, 1, true>(a, kv, dev, stream);
    if (dp == 64)
        return ht == 2 ? launch_shape<DT, 64, 2>(a, kv, dev, stream)
                       : launch_shape<DT, 64, 1>(a, kv, dev, stream);
    if (dp == 128) {
        if constexpr (DT != kF32)
            if (ht == 2) return launch_shape<DT, 128, 2>(a, kv, dev, stream);
        return launch_shape<DT, 128, 1>(a, kv, dev, stream);
    }
    return launch_shape<DT, 256, 1>(a, kv, dev, stream);
}

}  // namespace

size_t attn_workspace_bytes(const KvView &kv, int n_seq, int h_q, int n_slots, bool with_acc) {
    const int dp = padded_dim(kv.head_dim), ht = head_tile(h_q / kv.n_heads, dp, kv.dtype);
    size_t bytes = up256(kMaxCtas * 16) + up256(2ull * kMaxCtas * ht * 8 * (dp + 2) * 4) +
                   rows_bytes(n_seq, h_q, with_acc);
    if (with_acc)
        bytes += up256((size_t)n_seq * h_q * 4) + up256((size_t)n_seq * h_q * n_slots * 4);
    return bytes;
}

cudaError_t launch_attn_paged(const AttnArgs &a, const KvView &kv, const DeviceInfo &dev,
                              cudaStream_t stream) {
    switch (kv.dtype) {
    case kBF16: return launch_type<kBF16>(a, kv, dev, stream);
    case kF16: return launch_type<kF16>(a, kv, dev, stream);
    default: return launch_type<kF32>(a, kv, dev, stream);
    }
}

}  // namespace wq

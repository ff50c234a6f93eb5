// attn_paged.cu -- attention of one new token per sequence over a paged cache.
//
// wavo 0.3.0 src/gpu/mod.rs, attend / combine: one token's attention over the decoder's
// cache with the keys split into parts that are joined.  x_j = scale q.k_j + mask_j,
// p = softmax(x) by one pass with a running maximum m and sum l:
//   m' = max(m, x), l' = l e^(m-m') + e^(x-m'), o' = o e^(m-m') + e^(x-m') v,
// and parts (m, l, o) of a row are joined by the same rule, always in slot order.
//
// What bounds it: every live slot's k and v are read once and used group times (4 group
// operations per 2 bytes of a bf16 cache), so the cache's bytes set the floor.
//
// Products: eight query heads of a kv head fill the 16 rows of mma.sync m16n8k8 (tf32) as
// q = hi + lo with 11 bits each in rows g and g + 8 of a fragment; bf16 and f16 keys and
// values are exact in tf32, f32 ones are split in the same way (two products).  The
// weights p enter the second product as hi + lo too.  So every product is within 2^-22 of
// exact, as everywhere in this library; 16-bit operands alone would leave 2^-9.  The
// tensor core truncates when it accumulates (measured: 1 + 0.92 ulp added 1000 times
// stays 1), so no accumulation is longer than head_dim / 16 steps of q.k, and every 16
// slots' p.v is added to o by an f32 FMA that rescales it anyway.  Rate needed at the
// memory floor: 2 x 300 TFLOP/s measured tf32 mma.sync is 2.9 times what eight heads of a
// bf16 cache take.
//
// Dims may be summed in any order, so a lane takes 16 bytes of a key's row (its own four or
// eight dims) as operands as they are, with q laid out to match; p's accumulator
// fragment is the next product's operand without a move.  No shuffles but the maxima.
//
// Loads: each warp keeps a ring of kStages tiles of KT slots (k and v) in flight by cp.async,
// 96 KB per CTA and two CTAs per SM, and waits for no other warp: a CTA's warps meet
// only where a row (sequence, kv head, up to 16 query heads) ends.  A slot that takes no
// part (beyond the length, masked by -inf, in a page out of range) is filled with zeros in
// shared memory and not read.
//
// Work: the rows' tiles, one row after another, are dealt out in equal contiguous ranges to
// a fixed grid, whatever the lengths; a CTA finds its range from the lengths.  A row within
// one CTA is written by it, the parts of the others are joined by attn_join_kernel.
#include "kv_internal.h"
#include "wq_device.cuh"

namespace wq {
namespace {

constexpr int kStages = 3;
constexpr int kMaxCtas = 304;  // two on each of 152 SMs

template <int DT, int DP, int HT> struct Shape {
    static constexpr int kEb = DT == kF32 ? 4 : 2;     // bytes of an element
    static constexpr int kRow = DP * kEb;              // bytes of a slot's row in the ring
    static constexpr int kEpc = 16 / kEb;              // elements of a 16-byte chunk
    static constexpr int kChunks = kRow / 16;
    static constexpr int KT = kRow <= 256 ? 16 : 8;    // slots of a warp's tile
    static constexpr int NT = KT / 8;
    static constexpr int W = kRow == 128 ? 8 : kRow == 1024 ? 2 : 4;  // warps
    static constexpr int kTile = 2 * KT * kRow;        // bytes: k, then v
    static constexpr int BT = W * KT;                  // slots of a CTA's tile
    static constexpr int kHeads = HT * 8;              // query heads of a row
    static constexpr int kQ = W * kStages * kTile;                 // q fragments
    static constexpr int kBias = kQ + HT * DP * 64;                // [W][kStages][KT]
    static constexpr int kL = kBias + W * kStages * KT * 4;        // [W][kHeads]
    static constexpr int kM = kL + W * kHeads * 4;                 // [W][kHeads], or in kBias
    static constexpr bool kMInBias = KT >= kHeads;
    static constexpr int kSmem = kM + (kMInBias ? 0 : W * kHeads * 4);
    static constexpr int kPart = kHeads * (DP + 2);    // floats of a part: m, l, o
    static_assert(kHeads * DP * 4 <= kTile, "a warp's o fits the tile just used");
};

// The schedule that every CTA derives from the lengths: rows of sequence s have
// tiles(s) tiles each, never 0 (an empty row is written too).
struct Sched {
    int rows;            // rows per sequence: kv heads x head tiles
    long long total;     // tiles of all rows
    __device__ __forceinline__ long long start(int b, int grid) const {
        const long long q = total / grid, r = total - q * grid;
        return b * q + min((long long)b, r);
    }
    __device__ __forceinline__ int owner(long long t, int grid) const {
        const long long q = total / grid, r = total - q * grid, cut = r * (q + 1);
        return (int)(t < cut ? t / (q + 1) : r + (t - cut) / q);
    }
};

struct Span { int len, first; };
__device__ __forceinline__ Span span_of(const AttnArgs &a, int s) {
    Span p;
    p.len = min(max(__ldg(a.lens + s), 0), a.n_slots);
    p.first = a.window > 0 && p.len > a.window ? p.len - a.window : 0;
    return p;
}

__device__ __forceinline__ float exp_diff(float x, float m) {
    return x == -INFINITY ? 0.f : expf(x - m);
}

__device__ __forceinline__ uint32_t tf32(float x) {
    uint32_t r;
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(r) : "f"(x));
    return r;
}
// x - hi, the part that hi leaves; an infinity is left to hi.
__device__ __forceinline__ uint32_t tf32_rest(float x, uint32_t hi) {
    const float h = __uint_as_float(hi);
    return __float_as_uint(fabsf(h) == INFINITY ? 0.f : x - h);
}

__device__ __forceinline__ void mma_tf32(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr));
    return v;
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

// Element pair j of a chunk as f32 bits (16-bit types: the two halves of word j).
template <int DT> __device__ __forceinline__ void pair_of(const uint4 &v, int j, uint32_t &a,
                                                          uint32_t &b) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if (DT == kBF16) {
        a = w[j] << 16;
        b = w[j] & 0xFFFF0000u;
    } else if (DT == kF16) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[j]));
        a = __float_as_uint(f.x);
        b = __float_as_uint(f.y);
    } else {
        a = w[2 * j];
        b = w[2 * j + 1];
    }
}
// Element e of a chunk.
template <int DT> __device__ __forceinline__ uint32_t element_of(const uint4 &v, int e) {
    if (DT == kF32) {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
        return w[e];
    }
    uint32_t a, b;
    pair_of<DT>(v, e >> 1, a, b);
    return e & 1 ? b : a;
}

// d += a * b with b exact in tf32, or in f32 (split: its high 11 bits and the rest).
template <int DT>
__device__ __forceinline__ void mma_kv(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                       uint32_t b1) {
    if (DT == kF32) {
        const uint32_t h0 = b0 & 0xFFFFE000u, h1 = b1 & 0xFFFFE000u;
        mma_tf32(c, a, h0, h1);
        mma_tf32(c, a, tf32_rest(__uint_as_float(b0), h0), tf32_rest(__uint_as_float(b1), h1));
    } else {
        mma_tf32(c, a, b0, b1);
    }
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

// The workspace: tiles before each sequence, the parts, and for the weight sums the rows'
// lse and every score.
struct Room {
    long long *before;  // [n_seq + 1], in rows' tiles (not times rows)
    float *parts, *lse, *scores;
};
__host__ __device__ inline size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }
__host__ __device__ inline Room room_of(void *p, int n_seq, int h_q, size_t part_floats) {
    char *c = static_cast<char *>(p);
    Room r;
    r.before = reinterpret_cast<long long *>(c);
    c += up256((size_t)(n_seq + 1) * 8);
    r.parts = reinterpret_cast<float *>(c);
    c += up256(2ull * kMaxCtas * part_floats * 4);
    r.lse = reinterpret_cast<float *>(c);
    c += up256((size_t)n_seq * h_q * 4);
    r.scores = reinterpret_cast<float *>(c);
    return r;
}

template <int DT, int DP, int HT>
__global__ void __launch_bounds__(Shape<DT, DP, HT>::W * 32, 2)
    attn_kernel(AttnArgs a, KvView kv, int head_tiles) {
    using S = Shape<DT, DP, HT>;
    constexpr int NT = S::NT, KT = S::KT, W = S::W, kThreads = W * 32;
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ long long s_scan[W], s_total;
    __shared__ int s_seq;
    __shared__ long long s_before;
    pdl_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c = lane & 3;
    pdl_wait();
    const Room room = room_of(a.workspace, a.n_seq, a.h_q, S::kPart);
    const int rows = kv.n_heads * head_tiles;

    // Tiles before each thread's share of the sequences, and in all.
    auto tiles_of = [&](int s) {
        const Span p = span_of(a, s);
        return max(1, (p.len - p.first + S::BT - 1) / S::BT);
    };
    const int share = (a.n_seq + kThreads - 1) / kThreads;
    const int s0 = min(a.n_seq, (int)threadIdx.x * share), s1 = min(a.n_seq, s0 + share);
    long long mine = 0;
    for (int s = s0; s < s1; ++s) {
        mine += tiles_of(s);
        if (blockIdx.x == 0 && __ldg(a.lens + s) > a.n_slots) record_status(a.status, kStBadIndex);
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
    Sched sched{rows, total * rows};
    const long long t0 = sched.start(blockIdx.x, gridDim.x),
                    t1 = sched.start(blockIdx.x + 1, gridDim.x);
    if (blockIdx.x == 0) {
        long long at = before;
        for (int s = s0; s < s1; ++s) {
            room.before[s] = at;
            at += tiles_of(s);
        }
        if (threadIdx.x == 0) room.before[a.n_seq] = total;
    }
    if (t0 >= t1) return;
    if (t0 >= before * rows && t0 < (before + mine) * rows) {
        int s = s0;
        for (int n; t0 >= (before + (n = tiles_of(s))) * rows; ++s) before += n;
        s_seq = s;
        s_before = before;
    }
    __syncthreads();
    Cursor use;
    use.s = s_seq;
    use.load(a, S::BT);
    {
        const long long in = t0 - s_before * rows;
        use.row = (int)(in / use.tiles);
        use.tile = (int)(in - (long long)use.row * use.tiles);
    }
    Cursor fetch = use;  // the tile whose page numbers are asked for next
    long long left = t1 - t0, to_fetch = left;

    const uint32_t ring = smem_addr(smem) + warp * kStages * S::kTile;
    const uint32_t qf = smem_addr(smem) + S::kQ;
    float *bias = reinterpret_cast<float *>(smem + S::kBias) + warp * kStages * KT;
    const int live_chunks = kv.head_dim / S::kEpc;

    // Page numbers are asked for one tile ahead of the loads that need them.
    int ask_page = -1, ask_in = 0, ask_head = 0;
    float ask_bias = -INFINITY;
    bool ask_live = false;
    auto ask = [&]() {
        ask_live = false;
        if (to_fetch <= 0) return;
        --to_fetch;
        const int j = fetch.span.first + fetch.tile * S::BT + warp * KT + lane;
        if (lane < KT && j < fetch.span.len) {
            const uint32_t p = kv.page_size.div((uint32_t)j);
            ask_page = __ldg(kv.page_table + (long long)fetch.s * kv.max_pages + p);
            ask_in = j - (int)(p * kv.page_size.d);
            ask_bias = a.mask ? __ldg(a.mask + fetch.s * a.mask_stride + j) : 0.f;
            ask_live = true;
        }
        ask_head = head_tiles == 1 ? fetch.row : fetch.row / head_tiles;
        fetch.next(a, rows, S::BT);
    };
    auto issue = [&](int stage) {
        long long at = -1;
        float b = -INFINITY;
        if (ask_live) {
            if ((unsigned)ask_page >= (unsigned)kv.n_pages) {
                record_status(a.status, kStBadIndex);
            } else if (ask_bias != -INFINITY) {
                b = ask_bias;
                at = (long long)ask_page * kv.page_stride + (long long)ask_head * kv.head_stride +
                     (long long)ask_in * kv.token_stride;
            }
        }
        if (lane < KT) bias[stage * KT + lane] = b;
        const uint32_t base = ring + stage * S::kTile;
#pragma unroll
        for (int i = 0; i < KT * S::kChunks / 32; ++i) {
            const int idx = i * 32 + lane, key = idx / S::kChunks, ch = idx % S::kChunks;
            const long long from = __shfl_sync(0xFFFFFFFFu, at, key);
            const bool live = from >= 0 && ch < live_chunks;
            const long long off = live ? from + ch * 16 : 0;
            cp_async16(base + key * S::kRow + ((ch ^ ((key & 1) << 2)) << 4), kv.k + off, live);
            cp_async16(base + KT * S::kRow + key * S::kRow + ((ch ^ (key & 6)) << 4), kv.v + off,
                       live);
        }
    };

    // The row's query heads, scaled, as the first product's operand.
    auto load_q = [&](const Cursor &at) {
        const int h = at.row / head_tiles, ht0 = (at.row - h * head_tiles) * S::kHeads;
        const float *q = a.q + at.s * a.q_stride + ((long long)h * a.group + ht0) * kv.head_dim;
        for (int i = threadIdx.x; i < HT * DP / 8 * 32; i += kThreads) {
            const int l = i & 31, ks = (i >> 5) % (DP / 8), ht = (i >> 5) / (DP / 8);
            const int head = ht * 8 + (l >> 2);
            const int dim = S::kEpc * (4 * (ks / (S::kEpc / 2)) + (l & 3)) +
                            2 * (ks % (S::kEpc / 2));
            float2 v = make_float2(0.f, 0.f);
            if (ht0 + head < a.group && dim < kv.head_dim)
                v = *reinterpret_cast<const float2 *>(q + head * kv.head_dim + dim);
            v.x *= a.scale;
            v.y *= a.scale;
            uint4 f;
            f.x = tf32(v.x);
            f.y = tf32(__uint_as_float(tf32_rest(v.x, f.x)));
            f.z = tf32(v.y);
            f.w = tf32(__uint_as_float(tf32_rest(v.y, f.z)));
            *reinterpret_cast<uint4 *>(smem + S::kQ + i * 16) = f;
        }
    };

    ask();
#pragma unroll
    for (int st = 0; st < kStages; ++st) {
        issue(st);
        cp_async_commit();
        ask();
    }
    load_q(use);
    __syncthreads();

    constexpr int OI = S::kChunks / 8;  // chunk groups of v per lane
    float o[HT][OI][S::kEpc][2], m[HT], l[HT];
    auto clear = [&]() {
#pragma unroll
        for (int h = 0; h < HT; ++h) {
            m[h] = -INFINITY;
            l[h] = 0.f;
#pragma unroll
            for (int i = 0; i < OI; ++i)
#pragma unroll
                for (int e = 0; e < S::kEpc; ++e) o[h][i][e][0] = o[h][i][e][1] = 0.f;
        }
    };
    clear();
    bool whole = use.tile == 0;  // does this CTA have the row from its first tile
    bool leads = true;           // is this the CTA's first row
    int stage = 0;
    for (; left > 0; --left) {
        cp_async_wait<kStages - 1>();
        __syncwarp();
        const uint32_t kb = ring + stage * S::kTile, vb = kb + KT * S::kRow;
        const float *bs = bias + stage * KT;

        // x = q.k: rows g and g + 8 hold the high and low parts of head g.
        float sc[HT][NT][2][4] = {};
#pragma unroll
        for (int i = 0; i < S::kChunks / 4; ++i) {
            uint4 kk[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n)
                kk[n] = lds128(kb + (n * 8 + g) * S::kRow + (((4 * i + c) ^ ((g & 1) << 2)) << 4));
#pragma unroll
            for (int j = 0; j < S::kEpc / 2; ++j) {
                const int ks = i * (S::kEpc / 2) + j;
#pragma unroll
                for (int h = 0; h < HT; ++h) {
                    const uint4 qv = lds128(qf + (((h * DP / 8 + ks) * 32 + lane) << 4));
                    const uint32_t qa[4] = {qv.x, qv.y, qv.z, qv.w};
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        uint32_t b0, b1;
                        pair_of<DT>(kk[n], j, b0, b1);
                        mma_kv<DT>(sc[h][n][ks & 1], qa, b0, b1);
                    }
                }
            }
        }
        uint32_t pa[HT][NT][4];
        float corr[HT];
#pragma unroll
        for (int h = 0; h < HT; ++h) {
            float xs[NT][2], top = m[h];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float2 b = *reinterpret_cast<const float2 *>(bs + n * 8 + 2 * c);
                const float(&v)[2][4] = sc[h][n];
                const float x0 = (v[0][0] + v[1][0]) + (v[0][2] + v[1][2]);
                const float x1 = (v[0][1] + v[1][1]) + (v[0][3] + v[1][3]);
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
                        if (j < use.span.len) to[j] = xs[n][0];
                        if (j + 1 < use.span.len) to[j + 1] = xs[n][1];
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
                pa[h][n][0] = tf32(p0);
                pa[h][n][1] = tf32(p0 - __uint_as_float(pa[h][n][0]));
                pa[h][n][2] = tf32(p1);
                pa[h][n][3] = tf32(p1 - __uint_as_float(pa[h][n][2]));
            }
            l[h] = l[h] * corr[h] + sum;
        }
        // o = o corr + p.v
#pragma unroll
        for (int i = 0; i < OI; ++i) {
            if (8 * i >= live_chunks) break;
            uint4 v0[NT], v1[NT];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const int r = n * 8 + 2 * c;  // r & 6 is the same for r + 1
                const uint32_t at = vb + r * S::kRow + (((g + 8 * i) ^ (2 * c)) << 4);
                v0[n] = lds128(at);
                v1[n] = lds128(at + S::kRow);
            }
#pragma unroll
            for (int e = 0; e < S::kEpc; ++e)
#pragma unroll
                for (int h = 0; h < HT; ++h) {
                    float t[4] = {};
#pragma unroll
                    for (int n = 0; n < NT; ++n)
                        mma_kv<DT>(t, pa[h][n], element_of<DT>(v0[n], e), element_of<DT>(v1[n], e));
                    o[h][i][e][0] = o[h][i][e][0] * corr[h] + (t[0] + t[2]);
                    o[h][i][e][1] = o[h][i][e][1] * corr[h] + (t[1] + t[3]);
                }
        }

        const bool ends = use.tile + 1 == use.tiles, last = left == 1;
        if (ends || last) {
            // The warps' parts, through the tiles just used.
            float *mo = reinterpret_cast<float *>(smem + (warp * kStages + stage) * S::kTile);
            float *s_l = reinterpret_cast<float *>(smem + S::kL);
            float *s_m = reinterpret_cast<float *>(smem + (S::kMInBias ? S::kBias : S::kM));
            const int m_step = S::kMInBias ? kStages * KT : S::kHeads;
            const int m_off = S::kMInBias ? stage * KT : 0;
            __syncwarp();  // every lane has read the tile and its biases
#pragma unroll
            for (int h = 0; h < HT; ++h) {
                float sum = l[h];
                sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 1);
                sum += __shfl_xor_sync(0xFFFFFFFFu, sum, 2);
                if (c == 0) {
                    s_l[warp * S::kHeads + h * 8 + g] = sum;
                    s_m[warp * m_step + m_off + h * 8 + g] = m[h];
                }
#pragma unroll
                for (int i = 0; i < OI; ++i)
#pragma unroll
                    for (int e = 0; e < S::kEpc; ++e) {
                        float *to = mo + (h * 8 + g) * DP + S::kEpc * (2 * c + 8 * i) + e;
                        to[0] = o[h][i][e][0];
                        to[S::kEpc] = o[h][i][e][1];
                    }
            }
            __syncthreads();
            whole = whole && ends;
            const int hr = use.row / head_tiles, head0 = (use.row - hr * head_tiles) * S::kHeads;
            float *part = room.parts + (2ll * blockIdx.x + (leads ? 0 : 1)) * S::kPart;
            for (int idx = threadIdx.x; idx < S::kHeads * DP; idx += kThreads) {
                const int head = idx / DP, dim = idx % DP;
                float top = -INFINITY, sum = 0.f, v = 0.f;
#pragma unroll
                for (int w = 0; w < W; ++w) top = fmaxf(top, s_m[w * m_step + m_off + head]);
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    const float f = exp_diff(s_m[w * m_step + m_off + head], top);
                    sum += f * s_l[w * S::kHeads + head];
                    v += f * reinterpret_cast<const float *>(
                                 smem + (w * kStages + stage) * S::kTile)[idx];
                }
                if (!whole) {
                    part[2 * S::kHeads + idx] = v;
                    if (dim == 0) {
                        part[head] = top;
                        part[S::kHeads + head] = sum;
                    }
                } else if (head0 + head < a.group && dim < kv.head_dim) {
                    const int qh = hr * a.group + head0 + head;
                    const bool none = top == -INFINITY && sum == 0.f;
                    a.out[use.s * a.out_stride + (long long)qh * kv.head_dim + dim] =
                        none ? 0.f : v / sum;
                    if (dim == 0) {
                        const float e = none ? -INFINITY : top + logf(sum);
                        const long long at = (long long)use.s * a.h_q + qh;
                        if (a.lse) a.lse[at] = e;
                        if (a.acc_out) room.lse[at] = e;
                    }
                }
            }
            clear();
            leads = false;
            whole = true;
            if (!last) {
                Cursor nx = use;
                nx.next(a, rows, S::BT);
                load_q(nx);
            }
            __syncthreads();
        }
        use.next(a, rows, S::BT);
        __syncwarp();
        if (left > kStages) issue(stage);
        cp_async_commit();
        ask();
        stage = stage + 1 == kStages ? 0 : stage + 1;
    }
    cp_async_wait<0>();
}

// Joins the parts of the rows that several CTAs shared.  One block per (row, query head).
__global__ void __launch_bounds__(128) attn_join_kernel(AttnArgs a, int n_heads, int head_dim,
                                                        int head_tiles, int heads, int dp,
                                                        int grid) {
    __shared__ float s_f[kMaxCtas];
    __shared__ float s_red[2];
    pdl_enter();
    const int part_floats = heads * (dp + 2);
    const Room room = room_of(a.workspace, a.n_seq, a.h_q, part_floats);
    const int rows = n_heads * head_tiles;
    const int s = blockIdx.x / rows, row = blockIdx.x - s * rows;
    const int hr = row / head_tiles, ht = row - hr * head_tiles;
    const int head = blockIdx.y, in_group = ht * heads + head;
    if (in_group >= a.group) return;
    Sched sched{rows, room.before[a.n_seq] * rows};
    const long long b0 = room.before[s], tiles = room.before[s + 1] - b0;
    const long long r0 = b0 * rows + row * tiles, r1 = r0 + tiles;
    const int c0 = sched.owner(r0, grid), c1 = sched.owner(r1 - 1, grid);
    if (c0 == c1) return;  // written by its CTA
    const int n = c1 - c0 + 1;
    const int at0 = r0 > sched.start(c0, grid) ? 1 : 0;
    auto part = [&](int i) {
        return room.parts + (2ll * (c0 + i) + (i == 0 ? at0 : 0)) * part_floats;
    };
    if (threadIdx.x < 32) {
        float top = -INFINITY;
        for (int i = threadIdx.x; i < n; i += 32) top = fmaxf(top, part(i)[head]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
        float sum = 0.f;
        for (int i = threadIdx.x; i < n; i += 32) {
            const float f = exp_diff(part(i)[head], top);
            s_f[i] = f;
            sum += f * part(i)[heads + head];
        }
        sum = warp_sum(sum);
        if (threadIdx.x == 0) {
            s_red[0] = top;
            s_red[1] = sum;
        }
    }
    __syncthreads();
    const float top = s_red[0], sum = s_red[1];
    const bool none = top == -INFINITY && sum == 0.f;
    const int qh = hr * a.group + in_group;
    for (int d = threadIdx.x; d < head_dim; d += 128) {
        float v = 0.f;
#pragma unroll 4
        for (int i = 0; i < n; ++i) v += s_f[i] * part(i)[2 * heads + head * dp + d];
        a.out[s * a.out_stride + (long long)qh * head_dim + d] = none ? 0.f : v / sum;
    }
    if (threadIdx.x == 0) {
        const float e = none ? -INFINITY : top + logf(sum);
        const long long at = (long long)s * a.h_q + qh;
        if (a.lse) a.lse[at] = e;
        if (a.acc_out) room.lse[at] = e;
    }
}

// acc_out[s][h][j] = acc_in + sum over the group's heads of exp(x - lse).
__global__ void __launch_bounds__(256) attn_weights_kernel(AttnArgs a, int n_heads,
                                                           size_t part_floats) {
    pdl_enter();
    const Room room = room_of(a.workspace, a.n_seq, a.h_q, part_floats);
    const int s = blockIdx.x / n_heads, h = blockIdx.x - s * n_heads;
    const Span span = span_of(a, s);
    const long long at = ((long long)s * n_heads + h) * a.acc_stride;
    const long long q0 = (long long)s * a.h_q + h * a.group;
    for (int j = blockIdx.y * 256 + threadIdx.x; j < span.len; j += gridDim.y * 256) {
        float w = 0.f;
        if (j >= span.first)
            for (int g = 0; g < a.group; ++g) {
                const float e = room.lse[q0 + g];
                if (e != -INFINITY) w += exp_diff(room.scores[(q0 + g) * a.n_slots + j], e);
            }
        a.acc_out[at + j] = (a.acc_in ? a.acc_in[at + j] : 0.f) + w;
    }
}

// 16 query heads a row where a group has more than 8 (the cache is then read half as often),
// while o and q leave room for it; 8 otherwise.
int head_tile(int group, int dp) { return group > 8 && dp <= 128 ? 2 : 1; }
int padded_dim(int d) { return d <= 64 ? 64 : d <= 128 ? 128 : 256; }

template <int DT, int DP, int HT>
cudaError_t launch_shape(const AttnArgs &a, const KvView &kv, int head_tiles, int grid,
                         const DeviceInfo &dev, cudaStream_t stream) {
    using S = Shape<DT, DP, HT>;
    static std::atomic<unsigned long long> done{0};
    cudaError_t err = ensure_smem(attn_kernel<DT, DP, HT>, S::kSmem, dev, done);
    if (err != cudaSuccess) return err;
    return launch_pdl(attn_kernel<DT, DP, HT>, dim3(grid), dim3(S::W * 32), S::kSmem, stream, a,
                      kv, head_tiles);
}

template <int DT>
cudaError_t launch_type(const AttnArgs &a, const KvView &kv, int dp, int ht, int head_tiles,
                        int grid, const DeviceInfo &dev, cudaStream_t stream) {
    if (dp == 64)
        return ht == 2 ? launch_shape<DT, 64, 2>(a, kv, head_tiles, grid, dev, stream)
                       : launch_shape<DT, 64, 1>(a, kv, head_tiles, grid, dev, stream);
    if (dp == 128)
        return ht == 2 ? launch_shape<DT, 128, 2>(a, kv, head_tiles, grid, dev, stream)
                       : launch_shape<DT, 128, 1>(a, kv, head_tiles, grid, dev, stream);
    return launch_shape<DT, 256, 1>(a, kv, head_tiles, grid, dev, stream);
}

}  // namespace

size_t attn_workspace_bytes(const KvView &kv, int n_seq, int h_q, int n_slots, bool with_acc) {
    const int dp = padded_dim(kv.head_dim), ht = head_tile(h_q / kv.n_heads, dp);
    size_t bytes = up256((size_t)(n_seq + 1) * 8) +
                   up256(2ull * kMaxCtas * ht * 8 * (dp + 2) * 4);
    if (with_acc)
        bytes += up256((size_t)n_seq * h_q * 4) + up256((size_t)n_seq * h_q * n_slots * 4);
    return bytes;
}

cudaError_t launch_attn_paged(const AttnArgs &a, const KvView &kv, const DeviceInfo &dev,
                              cudaStream_t stream) {
    const int dp = padded_dim(kv.head_dim), ht = head_tile(a.group, dp), heads = ht * 8;
    const int head_tiles = (a.group + heads - 1) / heads;
    const int grid = min(kMaxCtas, 2 * dev.sm_count);
    const long long rows = (long long)a.n_seq * kv.n_heads * head_tiles;
    if (rows > 0x7FFFFFFFll) return cudaErrorInvalidConfiguration;
    cudaError_t err;
    switch (kv.dtype) {
    case kBF16: err = launch_type<kBF16>(a, kv, dp, ht, head_tiles, grid, dev, stream); break;
    case kF16: err = launch_type<kF16>(a, kv, dp, ht, head_tiles, grid, dev, stream); break;
    default: err = launch_type<kF32>(a, kv, dp, ht, head_tiles, grid, dev, stream); break;
    }
    if (err != cudaSuccess) return err;
    err = launch_pdl(attn_join_kernel, dim3((unsigned)rows, heads < a.group ? heads : a.group),
                     dim3(128), 0, stream, a, kv.n_heads, kv.head_dim, head_tiles, heads, dp, grid);
    if (err != cudaSuccess || !a.acc_out) return err;
    const int chunks = (int)((a.n_slots + 1023ll) / 1024);
    return launch_pdl(attn_weights_kernel,
                      dim3((unsigned)(a.n_seq * kv.n_heads), chunks > 64 ? 64 : chunks), dim3(256),
                      0, stream, a, kv.n_heads, (size_t)heads * (dp + 2));
}

}  // namespace wq

// attn_tokens_tc.cu -- attention of several new tokens per sequence on the tcgen05 tensor cores.
//
// S = Q K^T and P V for 128 rows (new tokens x heads of a group) and a tile of KT slots, both in
// tensor memory; between them two warpgroups of 128 threads, a thread to a row, turn S into
// weights p = 2^(S - m).
//
//   16-bit q    one product each; p is rounded to the cache's type, its sum is not.  The output
//               stays in tensor memory: m is only raised, and the output scaled, when a row's
//               maximum has outgrown it by more than 2^8, which after the first tiles is rare (a
//               published step of others' work on attention for this generation).
//   f32 q       (bf16 caches) q and p as three bf16 terms, 24 bits, whose products are exact: three
//               products each, the smallest terms first.  The tensor core truncates when it
//               accumulates, so P V of a tile, T, is added to an output in registers: o = o 2^(m_old -
//               m) + T.
//
// PAIR: two row tiles, one to a warpgroup, share every k and v tile: prompts, where the products
// bound it (a prompt of 8192 tokens, 32/8 heads of 128: 443 us, 1240 TFLOP/s counting what is seen).
// A tile's period is 3000 to 3500 cycles, products 2048 of it; the exponentials of 256 x 128 weights are
// 1024 of their own unit (32 a cycle), and the rest is the chain from a warpgroup's scores to its
// weights, of which a second warpgroup's products hide a part.
// Otherwise one row tile, whose slot tiles the warpgroups take in turn and join at the end: drafted
// trees, where the cache's bytes bound it and a second tile in flight hides the chain of the
// first (32 trees to 8192 slots: 117 us, 4.75 TB/s).  f32 queries: the three products of a score,
// whose N is 64, are bound by shared memory (48 cycles in place of 32), the weights' chain comes
// close to them (12 trees to 6000 slots: 82 us, with a cap 102).
//
// Shared memory is rows of 128 bytes in the 128-byte swizzle; k is K-major, v MN-major (its
// dims are the contiguous ones), p is read from tensor memory over S.
//
// A v that is not finite under a weight of 0 would reach rows that do not see it: where not all
// rows see all of a tile each warpgroup looks through its v first, while the scores are under way,
// takes such slots out, and adds them to the rows that see them by FMA.
#include <cudaTypedefs.h>

#include <atomic>
#include <cstddef>

#include "attn_tokens.cuh"
#include "tc_ptx.cuh"

namespace wq {
namespace tok {
namespace {

using namespace tc;

constexpr int kGrid = 152;       // one CTA on each SM
constexpr int kTeam = 128;       // a warpgroup: a thread to a row of its tile
constexpr int kSoft = 2 * kTeam;
constexpr int kThreads = kSoft + 128;  // an MMA warp, two for k and v, one for q
constexpr int kLoaders = 64;      // of pages that are no boxes
constexpr int kMostV = 6;
constexpr int kSmemMost = 227 * 1024;
constexpr int kMisc = 3 * 1024;    // barriers and small arrays, before the 1024-byte aligned part

// Tensor memory columns of a warpgroup (256 each).
constexpr uint32_t kColS = 0, kColP0 = 0, kColP1 = 64, kColP2 = 96, kColT = 128;

template <int DQ_, int TERMS_, bool PAIR_, int ET_> struct TcShape {
    // Dims of q and k, and of v in a pass: heads of 256 take two passes over the slots, each for half
    // of the output (all of it and the scores of two warpgroups do not fit tensor memory).
    static constexpr int DQ = DQ_, DP = DQ > 128 ? 128 : DQ, kPasses = DQ / DP;
    static constexpr int TERMS = TERMS_, ET = ET_;
    static constexpr bool PAIR = PAIR_;
    static constexpr int KT = TERMS == 1 && DQ <= 128 ? 128 : 64;
    static constexpr int RT = PAIR ? 256 : 128;
    static constexpr int kHalf = 128 * 128;            // 128 rows of 64 dims
    static constexpr int kQTerm = RT * DQ * 2;
    static constexpr int kStage = TERMS * kQTerm;
    static constexpr int kSlotK = KT * DQ * 2, kSlotV = KT * DP * 2;  // a k and a v tile
    static constexpr int kAhead = PAIR ? 1 : 0;        // a step brings v of tile g, k of g + kAhead
    static constexpr int kFit =
        (kSmemMost - kMisc - kStage - kAhead * kSlotK) / (kSlotK + kSlotV);
    static constexpr int NV = kFit < kMostV ? kFit : kMostV;
    static constexpr int NK = NV + kAhead;             // places for v and k tiles
    static constexpr int kSmem = kMisc + kStage + NK * kSlotK + NV * kSlotV;
    static_assert(NV >= 2, "a tile for each warpgroup");
};

struct Shared {
    uint64_t first, full[kMostV], done[kMostV];
    uint64_t s_full[2], p_ready[2], t_full[2], q_ready, q_free, meet[3], drain;
    alignas(16) uint32_t none[kMostV][4];  // of a v tile: slots whose page is out of range
    uint32_t odd[2][2][2][4];       // of a warpgroup, by turns: slots whose v is not finite
    float2 ml[2][128];              // maxima and sums of the warpgroups' rows
    int last[2][2][3];              // of this CTA's two parts: part_last(), the first CTA, the parts
    uint32_t issued[2];             // steps of the loaders of k and of v
    uint32_t tmem, abort;
};
static_assert(sizeof(Shared) <= kMisc && offsetof(Shared, none) % 16 == 0, "read as 16 bytes");

// Shared-memory descriptors by their low words (the address, and for MN-major the bytes between
// 64-element chunks of the contiguous dimension); the high word, groups of eight rows 1024 bytes
// apart in the 128-byte swizzle, is the same for all.
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_low(uint32_t addr, uint32_t chunk) {
    return (addr >> 4) | (chunk >> 4) << 16;
}
// D += or = A B with A in shared memory, or (ts) in tensor memory.
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                       uint32_t accum) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tmov.b64 x, {%1, %5};\n\t"
        "mov.b64 y, {%2, %5};\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(accum), "n"(kDescHigh)
        : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                       uint32_t accum) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\tmov.b64 y, {%2, %5};\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n\t}" ::"r"(d),
        "r"(a), "r"(b), "r"(idesc), "r"(accum), "n"(kDescHigh)
        : "memory");
}
template <int ET> __host__ __device__ constexpr uint32_t idesc_of(int N, bool b_mn) {
    return (1u << 4) | (ET == kBF16 ? (1u << 7) | (1u << 10) : 0u) | (b_mn ? 1u << 16 : 0u) |
           ((uint32_t)(N >> 3) << 17) | ((uint32_t)(128 >> 4) << 24);
}

#define WQ_R32(r)                                                                              \
    "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),        \
        "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]),             \
        "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]),          \
        "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),          \
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
#define WQ_RW32(r)                                                                             \
    "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),        \
        "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]),             \
        "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]),          \
        "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),          \
        "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])
// 32 columns of this thread's row; the values are there after wait_ld of the same registers.
__device__ __forceinline__ void ld32(uint32_t (&r)[32], uint32_t at) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
        "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, "
        "%28, %29, %30, %31}, [%32];"
        : WQ_R32(r)
        : "r"(at)
        : "memory");
}
__device__ __forceinline__ void wait_ld(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" : WQ_RW32(r)::"memory");
}
__device__ __forceinline__ float ld1(uint32_t at) {
    uint32_t r;
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(r) : "r"(at) : "memory");
    asm volatile("tcgen05.wait::ld.sync.aligned;" : "+r"(r)::"memory");
    return __uint_as_float(r);
}
__device__ __forceinline__ void st32(uint32_t at, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
        "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, "
        "%28, %29, %30, %31, %32};" ::"r"(at),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
        "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]),
        "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
        "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}
template <int N> __device__ __forceinline__ void st16(uint32_t at, const uint32_t (&r)[N]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
        "%11, %12, %13, %14, %15, %16};" ::"r"(at),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
        "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
        "r"(r[15])
        : "memory");
}
__device__ __forceinline__ void wait_st() {
    asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
template <int ET> __device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t r;
    if (ET == kBF16)
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
template <int ET> __device__ __forceinline__ float widen(uint32_t w, int half) {
    if (ET == kBF16) return __uint_as_float(half ? w & 0xFFFF0000u : w << 16);
    return __half2float(__ushort_as_half((unsigned short)(half ? w >> 16 : w & 0xFFFFu)));
}
// The larger of |a| and |b| in each half, NaN where there is one; and is either half not finite?
template <int ET> __device__ __forceinline__ uint32_t most16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    if (ET == kBF16)
        asm("{\n\t.reg .b32 x;\n\tabs.bf16x2 x, %2;\n\tmax.NaN.bf16x2 %0, %1, x;\n\t}"
            : "=r"(r) : "r"(a), "r"(b));
    else
        asm("{\n\t.reg .b32 x;\n\tabs.f16x2 x, %2;\n\tmax.NaN.f16x2 %0, %1, x;\n\t}"
            : "=r"(r) : "r"(a), "r"(b));
    return r;
}
template <int ET> __device__ __forceinline__ bool odd16x2(uint32_t w) {
    constexpr uint32_t e = ET == kBF16 ? 0x7F80u : 0x7C00u;
    return (w & e) == e || (w & (e << 16)) == (e << 16);
}
// The fast tanh of 16-bit queries: within 2^-22 of 1 for any x, which a cap of kFastCap makes 2^-14 of
// a weight, far below its rounding; inf and NaN come out right.
constexpr float kFastCap = 256.f;
__device__ __forceinline__ float fast_tanh(float x) {
    return 1.f - __fdividef(2.f, ex2(x * (2.f * kLog2e)) + 1.f);
}

__device__ __forceinline__ uint4 lds16(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(at)
                 : "memory");
    return v;
}
__device__ __forceinline__ void sts16(uint32_t at, uint4 v) {
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z),
                 "r"(v.w)
                 : "memory");
}

struct Ctx {
    Shared *sh;
    uint32_t stage, k_ring, v_ring;  // shared-memory addresses of q and of the k and v tiles
    unsigned long long limit;
    unsigned *status;
    __device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity) const {
        return wait_or_abort(bar, parity, &sh->abort, limit, status);
    }
    // One arrival of a warp, after what its lanes did.
    __device__ __forceinline__ void warp_arrive(uint64_t *bar) const {
        __syncwarp();
        if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
    }
    // A warp gives up as one.
    __device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity) const {
        return __all_sync(0xFFFFFFFFu, wait(bar, parity));
    }
};

// -------------------------------------------------------------------- loader warps --
//
// The key tiles of a CTA's range are one stream, numbered g across its stretches.  Step g brings
// v of tile g and k of tile g + kAhead (where that is 1, k of tile 0 comes by itself, `first`) and
// has one barrier, full[g % NV]; done[g % NV] says that the products of tile g are over.  k of tile
// g + kAhead takes the place of tile g - NV's, whose scores came before its values.

// The page of slot j; -2 for one that is not live.
__device__ __forceinline__ int page_of(const KvView &kv, int seq, int j, int len) {
    if (j >= len) return -2;
    return kv.page_table[(long long)seq * kv.max_pages + kv.page_size.div((uint32_t)j)];
}

// The tiles of the stream, and what a stretch has for all of its tiles.
template <typename S> struct Stream {
    Walk walk;
    const Tile *tiles;
    Stretch st;
    int kt, seq, len;
    bool more;
    __device__ __forceinline__ Stream(const Room &room) : walk(room, blockIdx.x), tiles(room.tiles) {
        open();
    }
    __device__ __forceinline__ void open() {
        do more = walk.next(st);
        while (more && st.k0 == st.k1);
        if (!more) return;
        kt = st.k0, seq = tiles[st.tile].seq, len = tiles[st.tile].q.len;
    }
    __device__ __forceinline__ void next() {
        if (++kt == st.k1) open();
    }
};

// By TMA, one warp for k and one for v (a lane's copies are issued one after another, 65 cycles
// each): where the pages are whole groups of eight rows, boxes of the largest number of
// rows that divides a page and a tile.  What lies beyond the live slots of a page, or of a box that
// was not asked for, is whatever memory holds: no row sees it, and look() takes it out.
template <typename S>
__device__ void load_boxes(const TokensArgs &a, const KvView &kv, const CUtensorMap *map,
                           bool is_v, int box, const Room &room, const Ctx &c) {
    const int lane = threadIdx.x & 31, from = lane * box;
    const bool mine = lane < S::KT / box;
    // Boxes of 64 dims; known without is_v where there is one pass.
    const int chunks = (S::kPasses > 1 && is_v ? S::DP : S::DQ) / 64;
    struct Box {
        int page, row, head, dim;
        bool live;
        uint32_t lost;   // of all lanes
        uint32_t bytes;
    };
    Stream<S> in(room);
    auto ask = [&]() {
        Box x{-2, 0, 0, 0, false, 0u, 0u};
        if (!in.more) return x;
        const int j = in.kt * S::KT + from;
        x.head = in.st.head / S::kPasses;
        if (S::kPasses > 1 && is_v) x.dim = in.st.head % S::kPasses * S::DP;
        x.row = j - (int)(kv.page_size.div((uint32_t)j) * kv.page_size.d);
        if (mine) x.page = page_of(kv, in.seq, j, in.len);
        return x;
    };
    auto settle = [&](Box &x) {  // once the page is there
        x.live = (unsigned)x.page < (unsigned)kv.n_pages;
        x.lost = __ballot_sync(0xFFFFFFFFu, !x.live && x.page != -2);
        x.bytes = __popc(__ballot_sync(0xFFFFFFFFu, x.live)) * box * 128 * chunks;
    };
    auto copy = [&](const Box &x, uint32_t to, uint64_t *bar) {
        if (!x.live) return;
#pragma unroll
        for (int h = 0; h < S::DQ / 64; ++h) {
            if (S::kPasses > 1 && h == chunks) break;
            asm volatile(
                "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
                " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(to + from * 128 + h * (S::KT * 128)),
                "l"(reinterpret_cast<uint64_t>(map)), "r"((S::kPasses > 1 ? x.dim : 0) + 64 * h),
                "r"(x.row), "r"(x.head), "r"(x.page), "r"(smem_addr(bar))
                : "memory");
        }
    };
    const bool ahead = S::kAhead && !is_v;
    bool here = in.more;  // is there a step
    Box cur = ask();
    if (ahead && here) {
        settle(cur);
        if (lane == 0) mbar_arrive_expect_tx(&c.sh->first, cur.bytes);
        __syncwarp();
        copy(cur, c.k_ring, &c.sh->first);
        in.next();
        cur = ask();
    }
    uint32_t g = 0;
    for (; here; ++g) {
        Box x = cur;
        const bool some = in.more;  // of x
        if (some) {
            in.next();
            cur = ask();
        }
        const uint32_t slot = g % S::NV;
        if (g >= (uint32_t)S::NV && !c.warp_wait(&c.sh->done[slot], (g / S::NV & 1) ^ 1)) break;
        settle(x);
        if (lane == 0) {
            if (is_v) {
                for (int i = 0; i < S::KT / 32; ++i) {
                    uint32_t none = 0;
                    for (uint32_t left = x.lost; left; left &= left - 1) {
                        const int at = (__ffs(left) - 1) * box - 32 * i;
                        none |= below(at + box) & ~below(at);
                    }
                    c.sh->none[slot][i] = none;
                }
                if (x.lost) record_status(a.status, kStBadIndex);
            }
            mbar_arrive_expect_tx(&c.sh->full[slot], x.bytes);
        }
        __syncwarp();
        copy(x, is_v ? c.v_ring + slot * S::kSlotV
                     : c.k_ring + (g + S::kAhead) % S::NK * S::kSlotK,
             &c.sh->full[slot]);
        here = ahead ? some : in.more;
    }
    // The last copies have landed before shared memory is given up.  After an abort one warp may have
    // asked for steps that the other has not: it arrives for those, and both wait for all.
    if (lane == 0) c.sh->issued[is_v] = g;
    asm volatile("bar.sync 1, 64;" ::: "memory");  // the loaders: each gets here, its waits are bounded
    const uint32_t end = max(c.sh->issued[0], c.sh->issued[1]);
    if (lane == 0)
        for (uint32_t i = g; i < end; ++i) mbar_arrive(&c.sh->full[i % S::NV]);
    if (ahead && g > 0) mbar_wait(&c.sh->first, 0, kDrainPolls);
    for (uint32_t i = end < (uint32_t)S::NV ? 0 : end - S::NV; i < end; ++i)
        mbar_wait(&c.sh->full[i % S::NV], i / S::NV & 1, kDrainPolls);
}

// The same by cp.async and two warps for pages of any size; a step's barrier is arrived at when
// it has landed and NV - 1 others are under way, or the next one has to wait.  Slots beyond the
// live ones and in pages out of range are zeros.
template <typename S>
__device__ void load_rows(const TokensArgs &a, const KvView &kv, const Room &room, const Ctx &c) {
    static_assert(S::kPasses == 1, "all of a head's dims");
    constexpr int kLanes = S::DP / 8;         // 16-byte chunks, a lane each, of a row
    constexpr int kRows = 32 / kLanes;        // rows of a warp's copy
    constexpr int kGroups = S::KT / 32;
    const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) - kSoft / 32 - 1;
    const int chunk = lane % kLanes;
    const bool in_dim = chunk * 8 < kv.head_dim;
    struct Rows {
        int page[kGroups], j, head;  // of this lane's rows: lane + 32 i
    };
    Stream<S> in(room);
    auto ask = [&]() {
        Rows x;
        x.j = in.kt * S::KT + lane, x.head = in.st.head;
#pragma unroll
        for (int i = 0; i < kGroups; ++i)
            x.page[i] = in.more ? page_of(kv, in.seq, x.j + 32 * i, in.len) : -2;
        return x;
    };
    auto copy = [&](const Rows &x, const char *pool, uint32_t ring) {
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
            const int j = x.j + 32 * i;
            const int row_in = j - (int)(kv.page_size.div((uint32_t)j) * kv.page_size.d);
            const long long at = (unsigned)x.page[i] < (unsigned)kv.n_pages
                                     ? (long long)x.page[i] * kv.page_stride +
                                           (long long)x.head * kv.head_stride +
                                           (long long)row_in * kv.token_stride
                                     : -1;
            for (int k = warp; k < 32 / kRows; k += kLoaders / 32) {
                const int r = k * kRows + lane / kLanes, row = 32 * i + r;
                const long long from = __shfl_sync(0xFFFFFFFFu, at, r);
                const bool live = from >= 0 && in_dim;
                cp16(ring + (chunk >> 3) * (S::KT * 128) + row * 128 +
                         (((chunk & 7) ^ (row & 7)) << 4),
                     pool + (live ? from + chunk * 16 : 0), live);
            }
        }
    };
    if (!in.more) return;
    Rows cur = ask();
    if (S::kAhead) {
        copy(cur, kv.k, c.k_ring);
        cp_commit();
        cp_wait<0>();
        fence_proxy_async_smem();
        mbar_arrive(&c.sh->first);
    }
    uint32_t g = 0, landed = 0;
    auto land = [&]() {
        fence_proxy_async_smem();
        mbar_arrive(&c.sh->full[landed++ % S::NV]);
    };
    bool ok = true;
    for (bool some = true; some; ++g) {
        const Rows v = cur;
        in.next();
        some = in.more;
        cur = ask();
        const uint32_t slot = g % S::NV;
        if (g >= (uint32_t)S::NV) {
            uint64_t *const bar = &c.sh->done[slot];
            const uint32_t turn = (g / S::NV & 1) ^ 1;
            // What it waits for may wait for the step before.
            if (landed < g && !__all_sync(0xFFFFFFFFu, mbar_test_wait(bar, turn))) {
                cp_wait<0>();
                while (landed < g) land();
            }
            if (!c.warp_wait(bar, turn)) {
                ok = false;
                break;
            }
        }
#pragma unroll
        for (int i = 0; i < kGroups; ++i) {
            const uint32_t none = __ballot_sync(
                0xFFFFFFFFu, (unsigned)v.page[i] >= (unsigned)kv.n_pages && v.page[i] != -2);
            if (warp == 0 && lane == 0) {
                c.sh->none[slot][i] = none;
                if (none) record_status(a.status, kStBadIndex);
            }
        }
        if (!S::kAhead || some)
            copy(S::kAhead ? cur : v, kv.k, c.k_ring + (g + S::kAhead) % S::NK * S::kSlotK);
        copy(v, kv.v, c.v_ring + slot * S::kSlotV);
        cp_commit();
        if (g + 1 - landed >= (uint32_t)S::NV) {
            cp_wait<S::NV - 1>();
            land();
        }
    }
    cp_wait<0>();
    while (ok && landed < g) land();
}

// q of a stretch of 16-bit queries, by one warp, while the stretch before ends: its place is free
// when the last scores are done.  By TMA where whole tokens make up 128 rows (q_box tokens of group
// heads; the rows beyond the sequence's are another's, and written by no one), else by cp.async.
template <typename S>
__device__ void load_queries(const TokensArgs &a, const KvView &kv, const CUtensorMap *q_map,
                             int q_box, const Room &room, const Ctx &c) {
    constexpr int kChunks = S::DQ / 8;
    const int lane = threadIdx.x & 31, group = a.group.d;
    Walk walk(room, blockIdx.x);
    Stretch st;
    uint32_t n = 0;
    while (walk.next(st)) {
        if (st.k0 == st.k1) continue;
        const Tile *const tile = room.tiles + st.tile;
        const int row0 = tile->row0, t0 = tile->q.t0, rows = tile->q.count * group - row0;
        const int head0 = st.head / S::kPasses * group;
        if (n > 0 && !c.warp_wait(&c.sh->q_free, (n - 1) & 1)) break;
        if (q_box) {
            if (lane == 0) {
                mbar_arrive_expect_tx(&c.sh->q_ready, S::kQTerm);
#pragma unroll
                for (int x = 0; x < S::RT / 128 * (S::DQ / 64); ++x) {
                    const int r = x / (S::DQ / 64) * 128, h = x % (S::DQ / 64);
                    asm volatile(
                        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx"
                        "::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(
                            c.stage + r * (S::DQ * 2) + h * S::kHalf),
                        "l"(reinterpret_cast<uint64_t>(q_map)), "r"(64 * h),
                        "r"(head0), "r"(t0 + (int)a.group.div(row0 + r)),
                        "r"(smem_addr(&c.sh->q_ready))
                        : "memory");
                }
            }
            __syncwarp();
            ++n;
            continue;
        }
#pragma unroll 4
        for (int i = lane; i < S::RT * kChunks; i += 32) {
            const int r = i / kChunks, ch = i % kChunks;
            const bool live = r < rows && ch * 8 < kv.head_dim;
            const int rr = row0 + r, j = a.group.div(live ? rr : 0), h = rr - j * group;
            const long long at = (t0 + j) * a.q_stride +
                                 (long long)(head0 + h) * kv.head_dim + ch * 8;
            // Row r of its tile of 128 rows.
            cp16(c.stage + (r >> 7) * (128 * S::DQ * 2) + (ch >> 3) * S::kHalf + (r & 127) * 128 +
                     (((ch & 7) ^ (r & 7)) << 4),
                 static_cast<const uint16_t *>(a.q) + (live ? at : 0), live);
        }
        cp_commit();
        cp_wait<0>();
        fence_proxy_async_smem();
        c.warp_arrive(&c.sh->q_ready);
        ++n;
    }
    // The last copy has landed before shared memory is given up.
    if (q_box && n > 0) mbar_wait(&c.sh->q_ready, (n - 1) & 1, kDrainPolls);
}

// ------------------------------------------------------------------------ MMA warp --
//
// A wait that is over takes this thread 100 cycles, a commit 50 and the second in a row 360, in
// which no product is issued (64 cycles each): it has one wait for a step and one for each
// warpgroup's p.  That a tile's products are over, the second warpgroup sees by its next scores
// (pairs: it says done), or a commit of its own tells (one row tile, where loads bound it and
// should not wait for scores).

template <typename S>
__device__ void issue_products(const TokensArgs &a, const Room &room, const Ctx &c) {
    const uint32_t tmem = c.sh->tmem;
    Walk walk(room, blockIdx.x);
    Stretch st;
    uint32_t base = 0;                 // tiles before this stretch
    uint32_t stretches = 0, seen = 0;  // seen: steps that have been waited for
    uint32_t taken = 0;                // parity of each warpgroup's p
    constexpr uint32_t kId = idesc_of<S::ET>(S::KT, false), vId = idesc_of<S::ET>(S::DP, true);

    auto step = [&](uint32_t g) {
        if (g < seen) return true;
        if (!c.wait(&c.sh->full[g % S::NV], g / S::NV & 1)) return false;
        tc_fence_after();
        seen = g + 1;
        return true;
    };
    auto scores = [&](int wg, uint32_t tile) {  // S of a warpgroup from the tile's k
        const uint32_t k = desc_low(c.k_ring + tile % S::NK * S::kSlotK, 16);
        uint32_t accum = 0;
#pragma unroll
        for (int t = S::TERMS - 1; t >= 0; --t) {
            const uint32_t q =
                desc_low(c.stage + t * S::kQTerm + (S::PAIR ? wg * (128 * S::DQ * 2) : 0), 16);
#pragma unroll
            for (int h = 0; h < S::DQ / 64; ++h)
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    mma_ss(tmem + wg * 256 + kColS, q + (h * S::kHalf + 32 * s >> 4),
                           k + (h * (S::KT * 128) + 32 * s >> 4), kId, accum);
                    accum = 1;
                }
        }
        tc_commit(&c.sh->s_full[wg]);
    };
    // P V of a warpgroup from the tile's v.  That it is over shows by the next scores; `last` has
    // none.
    auto values = [&](int wg, uint32_t tile, bool last) {
        const uint32_t v = desc_low(c.v_ring + tile % S::NV * S::kSlotV, S::KT * 128);
        uint32_t accum = S::TERMS == 1;  // on top of the output, which began as zeros
        if (!c.wait(&c.sh->p_ready[wg], taken >> wg & 1)) return false;
        taken ^= 1u << wg;
        tc_fence_after();
#pragma unroll
        for (int t = S::TERMS - 1; t >= 0; --t) {
            const uint32_t p = tmem + wg * 256 + (t == 0 ? kColP0 : t == 1 ? kColP1 : kColP2);
#pragma unroll
            for (int s = 0; s < S::KT / 16; ++s) {
                mma_ts(tmem + wg * 256 + kColT, p + 8 * s, v + (2048 * s >> 4), vId, accum);
                accum = 1;
            }
        }
        if (S::TERMS > 1 || last) tc_commit(&c.sh->t_full[wg]);
        return true;
    };
    while (walk.next(st)) {
        const int n = st.k1 - st.k0;
        if (n == 0) continue;
        if (!c.wait(&c.sh->q_ready, stretches++ & 1)) return;
        tc_fence_after();
        if (S::PAIR) {
            // k of the stretch's first tile came with the step before.
            if (base == 0 && !c.wait(&c.sh->first, 0)) return;
            tc_fence_after();
            scores(0, base);
            scores(1, base);
            if (n == 1) tc_commit(&c.sh->q_free);
            for (int i = 0; i < n; ++i) {
                const uint32_t tile = base + i;
                const bool last = i + 1 == n;
                if (!step(tile)) return;
#pragma unroll
                for (int wg = 0; wg < 2; ++wg) {
                    if (!values(wg, tile, last)) return;
                    if (!last) scores(wg, tile + 1);
                }
                if (i + 2 == n) tc_commit(&c.sh->q_free);
            }
        } else {
            if (!step(base)) return;
            scores(0, base);
            if (n > 1) {
                if (!step(base + 1)) return;
                scores(1, base + 1);
            }
            if (n <= 2) tc_commit(&c.sh->q_free);
            for (int i = 0; i < n; ++i) {
                const uint32_t tile = base + i;
                const int wg = i & 1;
                const bool last = i + 2 >= n;
                if (!values(wg, tile, last)) return;
                tc_commit(&c.sh->done[tile % S::NV]);
                if (!last) {
                    if (!step(tile + 2)) return;
                    scores(wg, tile + 2);
                    if (i + 3 == n) tc_commit(&c.sh->q_free);
                }
            }
        }
        base += n;
    }
}

// -------------------------------------------------------------- softmax warpgroups --

// Two bf16 values held within bf16's largest, their signs kept.
__device__ __forceinline__ uint32_t held16x2(uint32_t w) {
    uint32_t r;
    asm("min.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(w), "r"(0x7F7F7F7Fu));
    return r;
}
// f32 queries of a row tile as three bf16 terms, by all softmax threads.  Only the last term may be
// infinite: a finite value that bf16 rounds to infinity has the rest of it in the next term, and an
// infinite one leaves an infinity, not inf - inf.  (A NaN does so too, as a NaN.)
template <typename S>
__device__ __forceinline__ void load_q(const TokensArgs &a, const KvView &kv, const Tile &tile,
                                       int head, const Ctx &c) {
    constexpr int kChunks = S::DP / 8, kItems = 128 * kChunks / kSoft, kBatch = 2;
    const int group = a.group.d, row0 = tile.row0, t0 = tile.q.t0, d = kv.head_dim;
    const int rows = tile.q.count * group - row0;
#pragma unroll 1
    for (int b = 0; b < kItems; b += kBatch) {
        uint4 x[kBatch][2];
        uint32_t to[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            const int i = threadIdx.x + (b + k) * kSoft;
            const int r = i / kChunks, ch = i % kChunks;
            const bool live = r < rows && ch * 8 < d;
            const int rr = row0 + r, j = a.group.div(live ? rr : 0);
            const int g = rr - j * group;
            const long long at =
                (t0 + j) * a.q_stride + (long long)(head * group + g) * d + ch * 8;
            to[k] = c.stage + (ch >> 3) * S::kHalf + r * 128 + (((ch & 7) ^ (r & 7)) << 4);
            const uint4 *const from =
                reinterpret_cast<const uint4 *>(static_cast<const float *>(a.q) + at);
#pragma unroll
            for (int h = 0; h < 2; ++h) x[k][h] = live ? from[h] : make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            float y[8];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                y[4 * h] = __uint_as_float(x[k][h].x), y[4 * h + 1] = __uint_as_float(x[k][h].y);
                y[4 * h + 2] = __uint_as_float(x[k][h].z), y[4 * h + 3] = __uint_as_float(x[k][h].w);
            }
#pragma unroll
            for (int t = 0; t < S::TERMS; ++t) {
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    w[e] = pack2<kBF16>(y[2 * e], y[2 * e + 1]);
                    if (t + 1 < S::TERMS) w[e] = held16x2(w[e]);
                    y[2 * e] -= bf16_lo(w[e]);
                    y[2 * e + 1] -= bf16_hi(w[e]);
                }
                sts16(to[k] + t * S::kQTerm, make_uint4(w[0], w[1], w[2], w[3]));
            }
        }
    }
}

// Two f32 operations of one instruction.
__device__ __forceinline__ void fma2(float &x, float &y, float a0, float a1, float b, float c) {
    asm("{\n\t.reg .b64 p, q, r, d;\n\tmov.b64 p, {%2, %3};\n\tmov.b64 q, {%4, %4};\n\t"
        "mov.b64 r, {%5, %5};\n\tfma.rn.f32x2 d, p, q, r;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(x), "=f"(y)
        : "f"(a0), "f"(a1), "f"(b), "f"(c));
}
__device__ __forceinline__ void add2(float &x, float &y, float a0, float a1) {
    asm("{\n\t.reg .b64 p, q, d;\n\tmov.b64 p, {%0, %1};\n\tmov.b64 q, {%2, %3};\n\t"
        "add.rn.f32x2 d, p, q;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "+f"(x), "+f"(y)
        : "f"(a0), "f"(a1));
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    float2 r;
    asm("{\n\t.reg .b64 p, q, r, d;\n\tmov.b64 p, {%2, %3};\n\tmov.b64 q, {%4, %5};\n\t"
        "mov.b64 r, {%6, %7};\n\tfma.rn.f32x2 d, p, q, r;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
    return r;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    float2 r;
    asm("{\n\t.reg .b64 p, q, d;\n\tmov.b64 p, {%2, %3};\n\tmov.b64 q, {%4, %5};\n\t"
        "mul.rn.f32x2 d, p, q;\n\tmov.b64 {%0, %1}, d;\n\t}"
        : "=f"(r.x), "=f"(r.y)
        : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    return r;
}
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// The smaller, NaN where x is.
__device__ __forceinline__ float held_below(float x, float top) {
    float y;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(x), "f"(top));
    return y;
}

// tanh of the cap for f32 queries, within a few 2^-24 of itself: Lambert's continued fraction cut to
// z (945 + 105 z^2 + z^4) / (945 + 420 z^2 + 15 z^4) up to 0.5 (off by 2e-9 there), beyond it
// (e - 1) / (e + 1) with e = exp(2 z), z held below 10 (tanh is 1 to 2^-27 there); one division, no
// branch, NaN stays NaN.  Two at a time.
__device__ __forceinline__ float2 fine_tanh(float2 x) {
    const float2 z = mul2(x, x);
    const float2 e2 = mul2(make_float2(held_below(x.x, 10.f), held_below(x.y, 10.f)),
                           both(2.f * kLog2e));
    const float2 e = make_float2(ex2(e2.x), ex2(e2.y));
    const float2 n0 = mul2(x, fma2(z, fma2(z, both(1.f), both(105.f)), both(945.f)));
    const float2 d0 = fma2(z, fma2(z, both(15.f), both(420.f)), both(945.f));
    const float2 n1 = fma2(e, both(1.f), both(-1.f)), d1 = fma2(e, both(1.f), both(1.f));
    const bool sx = z.x < 0.25f, sy = z.y < 0.25f;
    return mul2(make_float2(sx ? n0.x : n1.x, sy ? n0.y : n1.y),
                make_float2(rcp(sx ? d0.x : d1.x), rcp(sy ? d0.y : d1.y)));
}

// A softmax thread's row, and what the two kinds of softmax share.  What only border tiles and a
// stretch's end ask for is worked out there again: a tile's scores want the registers (spills go
// to L2: shared memory has taken L1).
template <typename S> struct Row {
    static constexpr int DP = S::DP, KT = S::KT, kChunks = KT / 32;
    static constexpr int kParts = DP / 64;             // rows of 128 bytes of a v
    // A warpgroup looks through a v by itself (both together: 60 us for pieces of prompts, where the
    // one waits for the other): rows of 128 bytes to a thread, or threads to a row.
    static constexpr int kEach = KT * kParts > kTeam ? KT * kParts / kTeam : 1;
    static constexpr int kPieces = KT * kParts > kTeam ? 1 : kTeam / (KT * kParts);
    const TokensArgs &a;
    const KvView &kv;
    const Ctx &c;
    const Tile *tile;    // of the stretch
    int head, pass;      // kv head, pass over its dims
    const uint32_t tm;   // the warpgroup's columns, this warp's lanes
    const float to_log2;
    uint32_t turns = 0;  // parities of the meetings of both and of this one, and of look()

    __device__ __forceinline__ Row(const TokensArgs &a_, const KvView &kv_, const Ctx &c_)
        : a(a_), kv(kv_), c(c_), tm(c_.sh->tmem + ((threadIdx.x & 96u) << 16) + wg() * 256),
          to_log2(formed() ? 1.f : a_.scale * kLog2e) {}

    __device__ __forceinline__ static int wg() { return threadIdx.x / kTeam; }
    __device__ __forceinline__ static int r() { return threadIdx.x & 127; }
    __device__ __forceinline__ static int row() { return S::PAIR ? wg() * 128 + r() : r(); }
    // More than a positive scale: worked out once, written back in log2 units.
    __device__ __forceinline__ bool formed() const {
        return a.softcap > 0.f || a.slopes || !(a.scale > 0.f);
    }
    // The row's place: token of the sequence and query head; false beyond the tile's rows.
    __device__ __forceinline__ bool place(int &j, int &h) const {
        const int group = a.group.d, rr = tile->row0 + row();
        const bool live = rr < tile->q.count * group;
        j = a.group.div(live ? rr : 0);
        h = head * group + (live ? rr : 0) - j * group;
        return live;
    }
    __device__ __forceinline__ See see() const {
        int j, h;
        return place(j, h) ? see_of(a, tile->q, tile->seq, j) : See{};
    }
    // The threads of this warpgroup, or of both.
    __device__ __forceinline__ bool meet(bool alone) {
        uint64_t *const bar = &c.sh->meet[alone ? 1 + wg() : 0];
        const int bit = alone;
        const uint32_t turn = turns >> bit & 1;
        turns ^= 1u << bit;
        c.warp_arrive(bar);
        return c.warp_wait(bar, turn);
    }
    // This thread's scores in tensor memory to log2 units after cap and bias, those that are not
    // seen to -inf; their maximum (where it is asked for: f32 queries).
    __device__ __forceinline__ float form(int j0, bool mixed, const uint32_t *none) {
        float top[2] = {-INFINITY, -INFINITY};
#pragma unroll 1
        for (int ch = 0; ch < kChunks; ++ch) {
            const int jc = j0 + 32 * ch;
            uint32_t v[32];
            ld32(v, tm + kColS + 32 * ch);
            wait_ld(v);
            if (formed()) {
                if (a.softcap > 0.f) {
                    const float in = a.scale / a.softcap, out = a.softcap * kLog2e;
                    if (S::TERMS == 1 && a.softcap <= kFastCap) {
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            v[e] = __float_as_uint(out * fast_tanh(__uint_as_float(v[e]) * in));
                    } else {
#pragma unroll
                        for (int e = 0; e < 32; e += 2) {
                            const float2 y = mul2(
                                fine_tanh(mul2(make_float2(__uint_as_float(v[e]),
                                                           __uint_as_float(v[e + 1])), both(in))),
                                both(out));
                            v[e] = __float_as_uint(y.x), v[e + 1] = __float_as_uint(y.y);
                        }
                    }
                } else {
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        v[e] = __float_as_uint(__uint_as_float(v[e]) * a.scale * kLog2e);
                }
                if (a.slopes) {
                    int j, h;
                    place(j, h);
                    const float slope = a.slopes[h] * kLog2e;
                    const Seq q = tile->q;
                    const bool own = a.pos && jc + 32 > q.base;
                    const int pos = a.pos ? near(a.pos[q.t0 + j]) : q.base + j;
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const int far = (own ? slot_pos(a, q, jc + e) : jc + e) - pos;
                        v[e] = __float_as_uint(fmaf(slope, (float)far, __uint_as_float(v[e])));
                    }
                }
            }
            if (mixed) {
                const uint32_t in = seen32(a, see(), jc) & ~none[ch];
                if (__any_sync(0xFFFFFFFFu, ~in)) {
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (!(in >> e & 1u)) v[e] = 0xFF800000u;
                }
            }
            st32(tm + kColS + 32 * ch, v);
            if (S::TERMS > 1) {
#pragma unroll
                for (int e = 0; e < 32; ++e) top[e & 1] = fmaxf(top[e & 1], __uint_as_float(v[e]));
            }
        }
        wait_st();
        return fmaxf(top[0], top[1]);
    }
    // Finds the slots of a v tile that are not finite; `any` is the same for all that look.
    struct Odd {
        uint32_t any, *words;
    };
    // The slot, and the first of its rows of 128 bytes or the piece of one, of a thread that looks.
    struct Line {
        int at, slot, part, piece;
    };
    __device__ __forceinline__ Line line() const {
        Line n;
        n.at = threadIdx.x % kTeam;
        n.slot = n.at % KT;
        const int rest = n.at / KT;
        n.part = kEach > 1 ? rest * kEach : rest % kParts;
        n.piece = kEach > 1 ? 0 : rest / kParts;
        return n;
    }
    __device__ __forceinline__ bool look(uint32_t v_at, Odd &o) {
        const Line n = line();
        uint32_t most[4] = {};
#pragma unroll 1
        for (int p = 0; p < kEach; ++p) {
            const uint32_t at = v_at + (n.part + p) * (KT * 128) + n.slot * 128;
#pragma unroll
            for (int ch = 0; ch < 8 / kPieces; ++ch) {
                const uint4 w = lds16(at + (((ch + n.piece * (8 / kPieces) + n.slot) & 7) << 4));
                most[0] = most16x2<S::ET>(most[0], w.x), most[1] = most16x2<S::ET>(most[1], w.y);
                most[2] = most16x2<S::ET>(most[2], w.z), most[3] = most16x2<S::ET>(most[3], w.w);
            }
        }
        const bool mine = odd16x2<S::ET>(most16x2<S::ET>(most16x2<S::ET>(most[0], most[1]),
                                                         most16x2<S::ET>(most[2], most[3])));
        const uint32_t found = __ballot_sync(0xFFFFFFFFu, mine);
        // By turns: the next scores, and with them the look after the next, come after all of the
        // warpgroup's weights.
        o.words = &c.sh->odd[wg()][turns >> 2 & 1][0][0];
        turns ^= 4u;
        if ((threadIdx.x & 31) == 0) o.words[n.at / KT * 4 + n.slot / 32] = found;
        tc_fence_before();
        if (!meet(true)) return false;
        tc_fence_after();
        o.any = 0;
#pragma unroll
        for (int ch = 0; ch < kChunks; ++ch) o.any |= word(o, ch);
        return true;
    }
    __device__ __forceinline__ static uint32_t word(const Odd &o, int ch) {
        uint32_t w = 0;
#pragma unroll
        for (int i = 0; i < kTeam / KT; ++i) w |= o.words[4 * i + ch];
        return w;
    }
    // f(slot, p) for each of them that the row sees, p its weight against the maximum `safe`; every
    // lane comes along.
    template <typename F>
    __device__ __forceinline__ void each_odd(const Odd &o, int j0, const uint32_t *none, float safe,
                                             F f) {
#pragma unroll 1
        for (int ch = 0; ch < kChunks; ++ch) {
            const uint32_t in = seen32(a, see(), j0 + 32 * ch) & ~none[ch];
#pragma unroll 1
            for (uint32_t left = word(o, ch); left; left &= left - 1) {
                const int b = __ffs(left) - 1;
                __syncwarp();
                const float x = ld1(tm + kColS + 32 * ch + b);
                f(32 * ch + b, (in >> b & 1u) != 0, ex2(fmaf(x, to_log2, -safe)));
            }
        }
    }
    __device__ __forceinline__ bool sees_odd(const Odd &o, int j0, const uint32_t *none) {
        uint32_t some = 0;
#pragma unroll 1
        for (int ch = 0; ch < kChunks; ++ch)
            some |= seen32(a, see(), j0 + 32 * ch) & ~none[ch] & word(o, ch);
        return some != 0;
    }
    // Eight dims of a slot's v.
    __device__ __forceinline__ static void v8(uint32_t v_at, int slot, int chunk, float (&x)[8]) {
        const uint4 u = lds16(v_at + (chunk >> 3) * (KT * 128) + slot * 128 +
                              (((chunk & 7) ^ (slot & 7)) << 4));
        const uint32_t z[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = widen<S::ET>(z[k >> 1], k & 1);
    }
    // Takes those slots out of the tile once every row has them: with pairs, those of both
    // warpgroups, which have found the same.
    __device__ __forceinline__ bool clear(uint32_t v_at, const Odd &o) {
        tc_fence_before();
        if (!meet(!S::PAIR)) return false;
        tc_fence_after();
        const Line n = line();
        if (word(o, n.slot >> 5) >> (n.slot & 31) & 1u) {
#pragma unroll 1
            for (int p = 0; p < kEach; ++p)
#pragma unroll
                for (int ch = 0; ch < 8 / kPieces; ++ch)
                    sts16(v_at + (n.part + p) * (KT * 128) + n.slot * 128 +
                              (ch + n.piece * (8 / kPieces)) * 16,
                          make_uint4(0u, 0u, 0u, 0u));
        }
        fence_proxy_async_smem();
        return true;
    }
    // The two warpgroups' halves of the slots, their outputs in tensor memory: each writes half of
    // the dims.
    __device__ __forceinline__ bool join(const Room &room, const Stretch &st, bool any, bool live,
                                         int j, int h, float m, float l) {
        c.sh->ml[wg()][r()] = make_float2(m, l);
        wait_st();
        tc_fence_before();
        if (!meet(false)) return false;
        tc_fence_after();
        const float2 x0 = c.sh->ml[0][r()], x1 = c.sh->ml[1][r()];
        const float both = fmaxf(x0.x, x1.x), safe = both == -INFINITY ? 0.f : both;
        const float f0 = ex2(x0.x - safe), f1 = ex2(x1.x - safe);
        const float sum = fmaf(x0.y, f0, x1.y * f1);
        const uint32_t t0 = tm - wg() * 256 + kColT, t1 = t0 + 256;
#pragma unroll 1
        for (int ch = wg() * (DP / 64); ch < (wg() + 1) * (DP / 64); ++ch) {
            uint32_t v[32] = {}, u[32] = {};
            if (any) {
                ld32(v, t0 + 32 * ch);
                ld32(u, t1 + 32 * ch);
                wait_ld(v);
                wait_ld(u);
            }
            float x[32];
#pragma unroll
            for (int e = 0; e < 32; ++e)
                x[e] = fmaf(__uint_as_float(v[e]), f0, __uint_as_float(u[e]) * f1);
            if (st.part >= 0)
                put_part(room, st, 32 * ch, x);
            else if (live)
                finish(j, h, both, sum, 32 * ch, x);
            __syncwarp();
        }
        if (st.part >= 0 && !join_parts(room, st, live, j, h, both, sum, wg() * (DP / 2),
                                        (wg() + 1) * (DP / 2)))
            return false;
        __syncwarp();
        tc_fence_before();
        if (!meet(false)) return false;  // both have read both
        tc_fence_after();
        return true;
    }
    // The part of a row tile that other CTAs work on too: written, and joined here if it is the last
    // of them, dims d0 .. d1 of this thread's row by this thread.
    __device__ __forceinline__ void put_part(const Room &room, const Stretch &st, int e,
                                             const float (&x)[32]) const {
        const size_t part = 2 * blockIdx.x + st.part;
#pragma unroll
        for (int k = 0; k < 32; k += 4)
            room.part_o[(part * (DP / 4) + (e + k) / 4) * S::RT + row()] =
                make_float4(x[k], x[k + 1], x[k + 2], x[k + 3]);
    }
    __device__ __forceinline__ bool join_parts(const Room &room, const Stretch &st, bool live, int j,
                                               int h, float m, float l, int d0, int d1) {
        if (d0 == 0)
            room.part_ml[(2 * blockIdx.x + st.part) * S::RT + row()] = make_float2(m, l);
        if (!a.join_inside) return true;
        __threadfence();
        const int which = S::PAIR ? wg() : 0;
        if (!meet(S::PAIR)) return false;
        if (threadIdx.x == which * kTeam) {
            int lead, parts;
            int *const to = c.sh->last[st.part][which];
            to[0] = part_last(room, st, blockIdx.x, which, lead, parts);
            to[1] = lead, to[2] = parts;
        }
        if (!meet(S::PAIR)) return false;
        if (!c.sh->last[st.part][which][0]) return true;
        __threadfence();
        if (!live) return true;
        const Joined to = joined(room, st, -1, 0.f, 0.f);
#pragma unroll 1
        for (int e = d0; e < d1; e += 32) {
            float x[32];
            join_dims(room, to, e, x);
            finish(j, h, to.m, to.l, e, x);
        }
        return true;
    }
    // Are all other parts of the row tile there?  Then this one joins them without being written: most
    // row tiles of prompts, whose first part is its CTA's last work and whose others began with theirs.
    // One thread looks, and a meeting later all know.
    __device__ __forceinline__ void peek(const Room &room, const Stretch &st) const {
        const int which = S::PAIR ? wg() : 0;
        if (threadIdx.x != which * kTeam) return;
        const Begin *const b = room.plan + blockIdx.x + st.part;
        int *const to = c.sh->last[st.part][which];
        const int lead = b->lead, parts = b->parts;
        to[0] = *(volatile unsigned *)(room.joined + 2 * lead + which) == (unsigned)parts - 1;
        to[1] = lead, to[2] = parts;
    }
    // The row's maximum and sum over all parts, of which this CTA's may be in its registers (own >= 0).
    struct Joined {
        int lead, parts, own;
        float m, l, mine;
    };
    __device__ __forceinline__ Joined joined(const Room &room, const Stretch &st, int own, float m,
                                             float l) const {
        const int *const last = c.sh->last[st.part][S::PAIR ? wg() : 0];
        Joined to{last[1], last[2], own, -INFINITY, 0.f, m};
        for (int i0 = 0; i0 < to.parts; i0 += 8) {
            float2 x[8];  // loads of several parts in flight: one SM reads them all
#pragma unroll
            for (int i = 0; i < 8; ++i)
                x[i] = __ldcg(room.part_ml +
                              part_place(to.lead, min(i0 + i, to.parts - 1)) * S::RT + row());
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (i0 + i >= to.parts) break;
                if (i0 + i == own) x[i] = make_float2(m, l);
                const float now = fmaxf(to.m, x[i].x), safe = now == -INFINITY ? 0.f : now;
                to.l = fmaf(to.l, ex2(to.m - safe), x[i].y * ex2(x[i].x - safe));
                to.m = now;
            }
        }
        return to;
    }
    // Dims e .. e + 31 of all parts, in their order whoever joins them; x holds this CTA's if to.own >= 0.
    __device__ __forceinline__ void join_dims(const Room &room, const Joined &to, int e,
                                              float (&x)[32]) const {
        const float safe = to.m == -INFINITY ? 0.f : to.m;
        float o[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) o[k] = 0.f;
#pragma unroll 1
        for (int i = 0; i < to.parts; ++i) {
            if (i == to.own) {
                const float g = ex2(to.mine - safe);
#pragma unroll
                for (int k = 0; k < 32; ++k) o[k] = fmaf(x[k], g, o[k]);
                continue;
            }
            const size_t part = part_place(to.lead, i);
            const float top = __ldcg(room.part_ml + part * S::RT + row()).x;
            float4 v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k)
                v[k] = __ldcg(room.part_o + (part * (DP / 4) + e / 4 + k) * S::RT + row());
            const float g = ex2(top - safe);
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                o[4 * k] = fmaf(v[k].x, g, o[4 * k]), o[4 * k + 1] = fmaf(v[k].y, g, o[4 * k + 1]);
                o[4 * k + 2] = fmaf(v[k].z, g, o[4 * k + 2]);
                o[4 * k + 3] = fmaf(v[k].w, g, o[4 * k + 3]);
            }
        }
#pragma unroll
        for (int k = 0; k < 32; ++k) x[k] = o[k];
    }
    // Dims e .. e + 31 of the row's result from its sums.
    __device__ __forceinline__ void finish(int j, int h, float m, float l, int e,
                                           float (&x)[32]) const {
        const int t = tile->q.t0 + j;
        const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
        for (int k = 0; k < 32; ++k) x[k] *= inv;
        const int dim0 = S::kPasses > 1 ? pass * DP : 0;
        const int left = kv.head_dim - dim0 - e;  // dims of the head from here on
        const long long to = t * a.out_stride + (long long)h * kv.head_dim + dim0 + e;
        if (a.out_type == kF32) {
            float *const p = static_cast<float *>(a.out) + to;
#pragma unroll
            for (int k = 0; k < 32; k += 8) {
                if (k >= left) break;
                reinterpret_cast<float4 *>(p + k)[0] =
                    make_float4(x[k], x[k + 1], x[k + 2], x[k + 3]);
                reinterpret_cast<float4 *>(p + k)[1] =
                    make_float4(x[k + 4], x[k + 5], x[k + 6], x[k + 7]);
            }
        } else {
            uint32_t w[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) w[k] = pack2<S::ET>(x[2 * k], x[2 * k + 1]);
            uint16_t *const p = static_cast<uint16_t *>(a.out) + to;
            if (a.wide_out) {  // 32 bytes at a time: whole sectors
#pragma unroll
                for (int k = 0; k < 16; k += 8) {
                    if (2 * k >= left) break;
                    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(
                                     p + 2 * k),
                                 "r"(w[k]), "r"(w[k + 1]), "r"(w[k + 2]), "r"(w[k + 3]),
                                 "r"(w[k + 4]), "r"(w[k + 5]), "r"(w[k + 6]), "r"(w[k + 7])
                                 : "memory");
                }
            } else {
#pragma unroll
                for (int k = 0; k < 16; k += 4) {
                    if (2 * k >= left) break;
                    *reinterpret_cast<uint4 *>(p + 2 * k) =
                        make_uint4(w[k], w[k + 1], w[k + 2], w[k + 3]);
                }
            }
        }
        if (dim0 + e == 0 && a.lse) a.lse[(long long)t * a.h_q + h] = lse_of(m, l);
    }
};

// 16-bit queries: the output in tensor memory.
template <typename S>
__device__ void softmax_16(const TokensArgs &a, const KvView &kv, const Room &room, const Ctx &c) {
    constexpr int DP = S::DP, KT = S::KT, kChunks = KT / 32;
    constexpr float kGrow = 8.f;  // p is at most 2^8: f16 holds it, and its sum
    using R = Row<S>;
    R w(a, kv, c);
    Shared *const sh = c.sh;
    Walk walk(room, blockIdx.x);
    Stretch st;
    // Tiles before this stretch, tiles of this warpgroup, stretches in which it had any.
    uint32_t base = 0, mine = 0, ended = 0;
    while (walk.next(st)) {
        __syncwarp();
        w.tile = room.tiles + st.tile;
        w.head = st.head / S::kPasses, w.pass = st.head % S::kPasses;
        const int n = st.k1 - st.k0;
        int j, h;
        // The row's maximum in use and its sum; rows beyond the tile's have weights of 0.
        float m = w.place(j, h) ? -INFINITY : INFINITY, l = 0.f;
        bool some = false;
        if (n > 0) {
            uint32_t zero[32] = {};
#pragma unroll
            for (int ch = 0; ch < DP / 32; ++ch) st32(w.tm + kColT + 32 * ch, zero);
        }
        const int lo = w.tile->lo, hi = w.tile->hi;  // every row of the tile sees [lo, hi)
        for (int i = S::PAIR ? 0 : w.wg(); i < n; i += S::PAIR ? 1 : 2) {
            const uint32_t g = base + i, vs = g % S::NV;
            const int j0 = (st.k0 + i) * KT;
            // What a border tile needs is found while its scores are under way.
            if (!c.warp_wait(&sh->full[vs], g / S::NV & 1)) return;
            uint32_t lost = 0;
            if constexpr (kChunks == 4) {
                const uint4 none = *reinterpret_cast<const uint4 *>(sh->none[vs]);
                lost = none.x | none.y | none.z | none.w;
            } else {
                lost = sh->none[vs][0] | sh->none[vs][1];
            }
            const bool mixed = j0 < lo || j0 + KT > hi || lost;
            const uint32_t v_at = c.v_ring + vs * S::kSlotV;
            uint32_t in[kChunks] = {};
            typename R::Odd odd{};
            if (mixed) {
                if (!w.formed()) {
                    const See see = w.see();
#pragma unroll 1  // little code: it is seldom in the instruction cache
                    for (int ch = 0; ch < kChunks; ++ch) {
                        const uint32_t x = seen32(a, see, j0 + 32 * ch) & ~sh->none[vs][ch];
#pragma unroll
                        for (int k = 0; k < kChunks; ++k) in[k] = k == ch ? x : in[k];
                    }
                }
                if (!w.look(v_at, odd)) return;
            }
            if (!c.warp_wait(&sh->s_full[w.wg()], mine & 1)) return;
            tc_fence_after();
            if (S::PAIR && threadIdx.x == kTeam && i > 0) mbar_arrive(&sh->done[(g - 1) % S::NV]);
            __syncwarp();
            uint32_t s[kChunks][32];
            if (w.formed()) w.form(j0, mixed, sh->none[vs]);
#pragma unroll
            for (int ch = 0; ch < kChunks; ++ch) ld32(s[ch], w.tm + kColS + 32 * ch);
            auto hide = [&](int ch) {  // the scores that are not seen
                if (__any_sync(0xFFFFFFFFu, ~in[ch])) {
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (!(in[ch] >> e & 1u)) s[ch][e] = 0xFF800000u;
                }
            };
            if (mixed && !w.formed()) {
#pragma unroll
                for (int ch = 0; ch < kChunks; ++ch) {
                    wait_ld(s[ch]);
                    hide(ch);
                }
            }
            float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int ch = 0; ch < kChunks; ++ch) {
                wait_ld(s[ch]);
#pragma unroll
                for (int e = 0; e < 32; e += 2)
                    top[(e >> 1) & 3] = fmaxf(top[(e >> 1) & 3],
                                              fmaxf(__uint_as_float(s[ch][e]),
                                                    __uint_as_float(s[ch][e + 1])));
            }
            float safe = m == -INFINITY ? 0.f : m, sums[4] = {0.f, 0.f, 0.f, 0.f};
            auto weigh = [&](int ch) {  // the chunk's weights take the place of its scores
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    float x, y;
                    fma2(x, y, __uint_as_float(s[ch][2 * e]), __uint_as_float(s[ch][2 * e + 1]),
                         w.to_log2, -safe);
                    x = ex2(x), y = ex2(y);
                    add2(sums[2 * (e & 1)], sums[2 * (e & 1) + 1], x, y);
                    s[ch][e] = pack2<S::ET>(x, y);
                }
            };
            // The first weights are worked out while the maximum is, which seldom changes.
            weigh(0);
            const float now =
                fmaxf(m, fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * w.to_log2);
            if (__any_sync(0xFFFFFFFFu, now > m + kGrow || m == -INFINITY)) {
                // Each row by itself, so that its bits do not depend on its neighbours.
                float f = 1.f;
                if (now > m + kGrow || m == -INFINITY) {
                    f = ex2(m - (now == -INFINITY ? 0.f : now));
                    m = now;
                }
                safe = m == -INFINITY ? 0.f : m;
                l *= f;
                if (some) {  // the last P V came before these scores
#pragma unroll 1
                    for (int ch = 0; ch < DP / 32; ++ch) {
                        uint32_t v[32];
                        ld32(v, w.tm + kColT + 32 * ch);
                        wait_ld(v);
#pragma unroll
                        for (int e = 0; e < 32; ++e)
                            v[e] = __float_as_uint(__uint_as_float(v[e]) * f);
                        st32(w.tm + kColT + 32 * ch, v);
                    }
                }
                ld32(s[0], w.tm + kColS);
                wait_ld(s[0]);
                if (mixed && !w.formed()) hide(0);
                sums[0] = sums[1] = sums[2] = sums[3] = 0.f;
                weigh(0);
            }
            if (odd.any) {
                wait_st();
#pragma unroll 1
                for (int ch = 0; ch < DP / 32; ++ch) {
                    uint32_t v[32];
                    ld32(v, w.tm + kColT + 32 * ch);
                    wait_ld(v);
                    w.each_odd(odd, j0, sh->none[vs], safe, [&](int slot, bool seen, float p) {
#pragma unroll
                        for (int e = 0; e < 32; e += 8) {
                            float x[8];
                            w.v8(v_at, slot, 4 * ch + e / 8, x);
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                if (seen)
                                    v[e + k] = __float_as_uint(
                                        fmaf(p, x[k], __uint_as_float(v[e + k])));
                        }
                    });
                    st32(w.tm + kColT + 32 * ch, v);
                }
                if (!w.clear(v_at, odd)) return;
            }
#pragma unroll
            for (int ch = 0; ch < kChunks; ++ch) {
                if (ch > 0) weigh(ch);
                st16(w.tm + kColP0 + 16 * ch, s[ch]);
            }
            wait_st();
            tc_fence_before();
            c.warp_arrive(&sh->p_ready[w.wg()]);
            l += (sums[0] + sums[1]) + (sums[2] + sums[3]);
            ++mine;
            some = true;
        }
        base += n;
        const bool peeks = S::PAIR && st.part >= 0 && a.join_inside;
        if (peeks) w.peek(room, st);
        if (some) {
            if (!c.warp_wait(&sh->t_full[w.wg()], ended & 1)) return;
            tc_fence_after();
            ++ended;
            if (S::PAIR && threadIdx.x == kTeam) mbar_arrive(&sh->done[(base - 1) % S::NV]);
        }
        const bool live = w.place(j, h);
        if (S::PAIR) {
            bool last = false;
            typename R::Joined to{};
            if (peeks) {
                if (!w.meet(true)) return;
                const int *const found = sh->last[st.part][w.wg()];
                last = found[0];
                if (last) {
                    __threadfence();
                    to = w.joined(room, st, st.part == 1 ? 0 : blockIdx.x - found[1], m, l);
                }
            }
#pragma unroll 1
            for (int ch = 0; ch < DP / 32; ++ch) {
                uint32_t v[32] = {};
                if (n > 0) {
                    ld32(v, w.tm + kColT + 32 * ch);
                    wait_ld(v);
                }
                float x[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) x[e] = __uint_as_float(v[e]);
                if (st.part >= 0 && !last) {
                    w.put_part(room, st, 32 * ch, x);
                } else if (live) {
                    if (last) w.join_dims(room, to, 32 * ch, x);
                    w.finish(j, h, last ? to.m : m, last ? to.l : l, 32 * ch, x);
                }
                __syncwarp();
            }
            if (st.part >= 0 && !last && !w.join_parts(room, st, live, j, h, m, l, 0, DP)) return;
        } else if (!w.join(room, st, n > 0, live, j, h, m, l)) {
            return;
        }
    }
}

// f32 queries: the output in registers.
template <typename S>
__device__ void softmax_32(const TokensArgs &a, const KvView &kv, const Room &room, const Ctx &c) {
    constexpr int DP = S::DP, KT = S::KT, kChunks = KT / 32;
    static_assert(!S::PAIR, "one row tile");
    Row<S> w(a, kv, c);
    Shared *const sh = c.sh;
    Walk walk(room, blockIdx.x);
    Stretch st;
    uint32_t base = 0, mine = 0;
    while (walk.next(st)) {
        __syncwarp();
        w.tile = room.tiles + st.tile;
        w.head = st.head / S::kPasses, w.pass = st.head % S::kPasses;
        const int n = st.k1 - st.k0;
        float o[DP];
#pragma unroll
        for (int e = 0; e < DP; ++e) o[e] = 0.f;
        float m = -INFINITY, l = 0.f, f = 0.f;
        bool pending = false;
        if (n > 0) {
            load_q<S>(a, kv, *w.tile, st.head, c);
            fence_proxy_async_smem();
            c.warp_arrive(&sh->q_ready);
        }
        const int lo = w.tile->lo, hi = w.tile->hi;  // every row of the tile sees [lo, hi)
        // o = o f + T of the tile before.
        auto take = [&]() {
            if (!c.warp_wait(&sh->t_full[w.wg()], (mine - 1) & 1)) return false;
            tc_fence_after();
#pragma unroll
            for (int ch = 0; ch < DP / 32; ++ch) {
                uint32_t v[32];
                ld32(v, w.tm + kColT + 32 * ch);
                wait_ld(v);
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    o[32 * ch + e] = fmaf(o[32 * ch + e], f, __uint_as_float(v[e]));
            }
            return true;
        };
        for (int i = w.wg(); i < n; i += 2) {
            if (pending && !take()) return;
            const uint32_t g = base + i, vs = g % S::NV;
            if (!c.warp_wait(&sh->full[vs], g / S::NV & 1)) return;
            const int j0 = (st.k0 + i) * KT;
            uint32_t lost = 0;
#pragma unroll
            for (int ch = 0; ch < kChunks; ++ch) lost |= sh->none[vs][ch];
            const bool mixed = j0 < lo || j0 + KT > hi || lost;
            const uint32_t v_at = c.v_ring + vs * S::kSlotV;
            typename Row<S>::Odd odd{};
            if (mixed && !w.look(v_at, odd)) return;
            if (!c.warp_wait(&sh->s_full[w.wg()], mine & 1)) return;
            tc_fence_after();
            float top = -INFINITY;
            if (w.formed() || mixed) {
                top = w.form(j0, mixed, sh->none[vs]);
            } else {
#pragma unroll
                for (int ch = 0; ch < kChunks; ++ch) {
                    uint32_t v[32];
                    ld32(v, w.tm + kColS + 32 * ch);
                    wait_ld(v);
#pragma unroll
                    for (int e = 0; e < 32; ++e) top = fmaxf(top, __uint_as_float(v[e]));
                }
            }
            const float now = fmaxf(m, top * w.to_log2);
            const float safe = now == -INFINITY ? 0.f : now;
            const float fl = ex2(m - safe);
            f = fl;
            m = now;
            if (odd.any) {
                // Only for rows that see one: what else the tile's place holds changes no bit.
                if (w.sees_odd(odd, j0, sh->none[vs])) {
#pragma unroll
                    for (int e = 0; e < DP; ++e) o[e] *= f;
                    f = 1.f;
                }
                w.each_odd(odd, j0, sh->none[vs], safe, [&](int slot, bool seen, float p) {
#pragma unroll
                    for (int e = 0; e < DP; e += 8) {
                        float x[8];
                        w.v8(v_at, slot, e / 8, x);
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            if (seen) o[e + k] = fmaf(p, x[k], o[e + k]);
                    }
                });
                if (!w.clear(v_at, odd)) return;
            }
            float sums[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int ch = 0; ch < kChunks; ++ch) {
                uint32_t v[32];
                ld32(v, w.tm + kColS + 32 * ch);
                wait_ld(v);
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    const float p = ex2(fmaf(__uint_as_float(v[e]), w.to_log2, -safe));
                    sums[e & 3] += p;
                    v[e] = __float_as_uint(p);
                }
#pragma unroll
                for (int t = 0; t < S::TERMS; ++t) {
                    uint32_t p[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        p[e] = pack2<S::ET>(__uint_as_float(v[2 * e]),
                                            __uint_as_float(v[2 * e + 1]));
                        v[2 * e] = __float_as_uint(__uint_as_float(v[2 * e]) - bf16_lo(p[e]));
                        v[2 * e + 1] =
                            __float_as_uint(__uint_as_float(v[2 * e + 1]) - bf16_hi(p[e]));
                    }
                    st16(w.tm + (t == 0 ? kColP0 : t == 1 ? kColP1 : kColP2) + 16 * ch, p);
                }
            }
            l = fmaf(l, fl, (sums[0] + sums[1]) + (sums[2] + sums[3]));
            wait_st();
            tc_fence_before();
            c.warp_arrive(&sh->p_ready[w.wg()]);
            ++mine;
            pending = true;
        }
        if (pending && !take()) return;
        base += n;
        if (n > 0) {
#pragma unroll
            for (int ch = 0; ch < DP / 32; ++ch) {
                uint32_t v[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(o[32 * ch + e]);
                st32(w.tm + kColT + 32 * ch, v);
            }
            wait_st();
        }
        int j, h;
        const bool live = w.place(j, h);
        if (!w.join(room, st, n > 0, live, j, h, m, l)) return;
    }
}

template <typename S>
__global__ void __launch_bounds__(kThreads, 1)
    attn_tokens_tc_kernel(TokensArgs a, KvView kv, const __grid_constant__ CUtensorMap k_map,
                          const __grid_constant__ CUtensorMap v_map,
                          const __grid_constant__ CUtensorMap q_map, int box, int q_box) {
    extern __shared__ __align__(1024) uint8_t smem[];
    Ctx c;
    c.sh = reinterpret_cast<Shared *>(smem);
    // Tiles lie on 1024-byte boundaries; the array is declared so, and nothing is done if it is not.
    c.stage = smem_addr(smem) + kMisc;
    if (c.stage & 1023u) {
        if (threadIdx.x == 0) record_status(a.status, kStTimeout);
        return;
    }
    c.k_ring = c.stage + S::kStage;
    c.v_ring = c.k_ring + S::NK * S::kSlotK;
    c.limit = a.wait_limit;
    c.status = a.status;
    const int warp = threadIdx.x >> 5;
    pdl_launch();
    if (threadIdx.x == 0) {
        if (box) prefetch_tmap(&k_map), prefetch_tmap(&v_map);
        if (q_box) prefetch_tmap(&q_map);
        mbar_init(&c.sh->first, box ? 1 : kLoaders);
        for (int i = 0; i < kMostV; ++i) {
            mbar_init(&c.sh->full[i], box ? 2 : kLoaders);
            mbar_init(&c.sh->done[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&c.sh->s_full[i], 1);
            mbar_init(&c.sh->p_ready[i], kTeam / 32);
            mbar_init(&c.sh->t_full[i], 1);
            mbar_init(&c.sh->meet[1 + i], kTeam / 32);
        }
        mbar_init(&c.sh->meet[0], kSoft / 32);
        mbar_init(&c.sh->q_ready, S::TERMS == 1 ? 1 : kSoft / 32);
        mbar_init(&c.sh->q_free, 1);
        mbar_init(&c.sh->drain, 1);
        c.sh->abort = 0u;
        fence_mbar_init();
    }
    constexpr int kMma = kSoft / 32;
    if (warp == kMma) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                         smem_addr(&c.sh->tmem)),
                     "r"(512u)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    pdl_wait();
    const Room room = room_of(a.workspace, a.n_seq, a.n_tok, a.group.d, S::RT, S::DP, kGrid);
    // What the softmax threads take over their share of the launch's registers the others give:
    // 384 x 168 = 256 x 216 + 128 x 72 = 256 x 224 + 128 x 56.
    if (warp < kMma) {
        if constexpr (S::TERMS == 1) {
            asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
            softmax_16<S>(a, kv, room, c);
        } else {
            asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
            softmax_32<S>(a, kv, room, c);
        }
    } else {
        if constexpr (S::TERMS == 1)
            asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        else
            asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        if (warp > kMma) {
            fence_proxy_async_global();  // q, k and v may be an earlier kernel's plain stores
            if (warp == kMma + 3) {
                if constexpr (S::TERMS == 1) load_queries<S>(a, kv, &q_map, q_box, room, c);
            } else if (!box) {
                if constexpr (S::kPasses == 1) load_rows<S>(a, kv, room, c);
            } else {
                const bool is_v = warp == kMma + 2;
                load_boxes<S>(a, kv, is_v ? &v_map : &k_map, is_v, box, room, c);
            }
        } else if ((threadIdx.x & 31) == 0) {
            issue_products<S>(a, room, c);
            // Every product is done before tensor memory and the tiles are given up.
            tc_commit(&c.sh->drain);
            mbar_wait(&c.sh->drain, 0, kDrainPolls);
        }
        __syncwarp();
    }
    if (warp < kMma) {  // a warp that gave up may have left a load or store of tensor memory under way
        wait_st();
        asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    if (warp == kMma) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(c.sh->tmem),
                     "r"(512u)
                     : "memory");
    }
}

// Two row tiles of 128 where the sequences have more rows than one on average, and fit.
bool pairs_rows(int n_seq, int n_tok, int group, int head_dim) {
    return head_dim <= 128 && (long long)n_tok * group > 128ll * n_seq;
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> known{nullptr};
    PFN_cuTensorMapEncodeTiled_v12000 fn = known.load(std::memory_order_acquire);
    if (!fn) {
        void *p = nullptr;
        cudaDriverEntryPointQueryResult st;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000,
                                             cudaEnableDefault, &st) == cudaSuccess &&
            st == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
        known.store(fn, std::memory_order_release);
    }
    return fn;
}
bool strides_fit(const KvView &kv) {  // a tensor map
    return (kv.token_stride | kv.head_stride | kv.page_stride) < (1ll << 40);
}
// A pool as [page][head][row][dim] in boxes of `box` rows of 64 dims, zeros beyond head_dim.
bool pool_map(CUtensorMap &map, const KvView &kv, char *pool, int box) {
    const PFN_cuTensorMapEncodeTiled_v12000 encode = encode_fn();
    const cuuint64_t dims[4] = {(cuuint64_t)kv.head_dim, kv.page_size.d, (cuuint64_t)kv.n_heads,
                                (cuuint64_t)kv.n_pages};
    const cuuint64_t strides[3] = {(cuuint64_t)kv.token_stride, (cuuint64_t)kv.head_stride,
                                   (cuuint64_t)kv.page_stride};
    if (!strides_fit(kv)) return false;
    const cuuint32_t boxes[4] = {64, (cuuint32_t)box, 1, 1}, steps[4] = {1, 1, 1, 1};
    return encode && encode(&map,
                            kv.dtype == kBF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                              : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                            4, pool, dims, strides, boxes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// q as [token][head][dim], in boxes of a group's heads of as many tokens as make up 128 rows; the
// number of tokens, or 0.
int query_map(CUtensorMap &map, const TokensArgs &a, const KvView &kv) {
    const PFN_cuTensorMapEncodeTiled_v12000 encode = encode_fn();
    const int group = a.group.d;
    if (!encode || a.q_type == kF32 || group > 128 || 128 % group) return 0;
    const cuuint64_t dims[3] = {(cuuint64_t)kv.head_dim, (cuuint64_t)a.h_q, (cuuint64_t)a.n_tok};
    const cuuint64_t strides[2] = {(cuuint64_t)kv.head_dim * 2, (cuuint64_t)a.q_stride * 2};
    if (strides[1] >= (1ull << 40)) return 0;
    const cuuint32_t boxes[3] = {64, (cuuint32_t)group, (cuuint32_t)(128 / group)};
    const cuuint32_t steps[3] = {1, 1, 1};
    return encode(&map,
                  a.q_type == kBF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                    : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                  3, const_cast<void *>(a.q), dims, strides, boxes, steps,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? 128 / group : 0;
}
// Rows of a box: the largest power of two, 8 at least, that divides a page and a tile; 0: none.
int box_of(const KvView &kv, int kt) {
    int box = kt;
    while (kv.page_size.d % box) box /= 2;
    return box >= 8 ? box : 0;
}

template <int DQ, int TERMS, bool PAIR, int ET>
cudaError_t launch_shape(const TokensArgs &a, const KvView &kv, const DeviceInfo &dev,
                         cudaStream_t stream) {
    using S = TcShape<DQ, TERMS, PAIR, ET>;
    static std::atomic<unsigned long long> raised{0};
    cudaError_t err = ensure_smem(attn_tokens_tc_kernel<S>, S::kSmem, dev, raised);
    if (err != cudaSuccess) return err;
    TokensArgs b = a;
    const int heads = kv.n_heads * S::kPasses;
    b.join_inside = joins_inside(a, heads, S::RT, kGrid);
    // What a row tile's start and end cost in key tiles (a prompt of 8192 tokens as 2, 3, 4: 438, 419,
    // 421 us; trees of f32 queries as 1, 2, 3: 123, 122, 117).
    err = launch_attn_plan(b, heads, S::RT, S::KT, S::DP, kGrid, PAIR || TERMS > 1 ? 3 : 2,
                           stream);
    if (err != cudaSuccess) return err;
    CUtensorMap k_map{}, v_map{}, q_map{};
    const int q_box = query_map(q_map, a, kv);
    int box = box_of(kv, S::KT);
    if (box && !(pool_map(k_map, kv, kv.k, box) && pool_map(v_map, kv, kv.v, box))) box = 0;
    if (S::kPasses > 1 && !box) return cudaErrorNotSupported;
    err = launch_pdl(attn_tokens_tc_kernel<S>, dim3(kGrid), dim3(kThreads), S::kSmem, stream, b, kv,
                     k_map, v_map, q_map, box, q_box);
    if (err != cudaSuccess || b.join_inside) return err;
    return launch_attn_parts(b, kv, S::kPasses, S::RT, S::DP, kGrid, stream);
}
template <int DQ, bool PAIR>
cudaError_t launch_16(const TokensArgs &a, const KvView &kv, const DeviceInfo &dev,
                      cudaStream_t stream) {
    return kv.dtype == kBF16 ? launch_shape<DQ, 1, PAIR, kBF16>(a, kv, dev, stream)
                             : launch_shape<DQ, 1, PAIR, kF16>(a, kv, dev, stream);
}
template <int DQ>
cudaError_t launch_dim(const TokensArgs &a, const KvView &kv, const DeviceInfo &dev,
                       cudaStream_t stream) {
    if (a.q_type == kF32) return launch_shape<DQ, 3, false, kBF16>(a, kv, dev, stream);
    return pairs_rows(a.n_seq, a.n_tok, a.group.d, kv.head_dim)
               ? launch_16<DQ, true>(a, kv, dev, stream)
               : launch_16<DQ, false>(a, kv, dev, stream);
}

}  // namespace

bool tokens_tc_takes(const KvView &kv, int q_type) {
    // Heads above 128 only where pages are boxes.
    if (q_type == kv.dtype)
        return q_type != kF32 && (kv.head_dim <= 128 || (kv.page_size.d % 8 == 0 && strides_fit(kv)));
    return kv.dtype == kBF16 && q_type == kF32 && kv.head_dim <= 128;
}

void tokens_tc_shape(int n_seq, int n_tok, int group, int q_type, int head_dim, int &rt, int &dp,
                     int &grid) {
    rt = q_type != kF32 && pairs_rows(n_seq, n_tok, group, head_dim) ? 256 : 128;
    dp = head_dim <= 64 ? 64 : 128;
    grid = kGrid;
}

cudaError_t launch_tokens_tc(const TokensArgs &a, const KvView &kv, const DeviceInfo &dev,
                             cudaStream_t stream) {
    if (kv.head_dim > 128) return launch_16<256, false>(a, kv, dev, stream);
    return kv.head_dim <= 64 ? launch_dim<64>(a, kv, dev, stream)
                             : launch_dim<128>(a, kv, dev, stream);
}

}  // namespace tok
}  // namespace wq

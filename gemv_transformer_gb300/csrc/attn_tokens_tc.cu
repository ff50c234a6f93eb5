// attn_tokens_tc.cu -- attention of several new tokens per sequence on the tcgen05 tensor cores.
//
// S = Q K^T and P V for 128 rows (new tokens x heads of a group) and a tile of KT slots, both in
// tensor memory; between them two warpgroups of 128 threads, a thread to a row, turn S into
// weights p = 2^(S - m).
//
//   16-bit q    one product each; p is rounded to the cache's type, its sum is not.  The output
//               stays in tensor memory: m is only raised, and the output scaled, when a row's
//               maximum has outgrown it by more than 2^8, which after the first tiles is rare.
//   f32 q       (bf16 caches) q and p as three bf16 terms, 24 bits, whose products are exact: three
//               products each, the smallest terms first.  The tensor core truncates when it
//               accumulates, so P V of a tile, T, is added to an output in registers: o = o 2^(m_old -
//               m) + T.
//
// PAIR: two row tiles, one to a warpgroup, share every k and v tile: prompts, where the products
// bound it.  Otherwise one row tile, whose slot tiles the warpgroups take in turn and join at
// the end: drafted trees, where the cache's bytes bound it and a second tile in flight hides the
// chain of the first.
//
// Shared memory is rows of 128 bytes in the 128-byte swizzle; k is K-major, v MN-major (its
// dims are the contiguous ones), p is read from tensor memory over S.
//
// A v that is not finite under a weight of 0 would reach rows that do not see it: where not all
// rows see all of a tile the warpgroups look through its v first, take such slots out, and add
// them to the rows that see them by FMA.
#include <cudaTypedefs.h>

#include <atomic>

#include "attn_tokens.cuh"
#include "tc_ptx.cuh"

namespace wq {
namespace tok {
namespace {

using namespace tc;

constexpr int kGrid = 152;       // one CTA on each SM
constexpr int kThreads = 384;    // two softmax warpgroups; an MMA warp and three loader warps
constexpr int kLoaders = 96;
constexpr int kMostSlots = 8;
constexpr int kSmemMost = 227 * 1024;
constexpr int kMisc = 2048;      // barriers and small arrays, before the 1024-byte aligned part

// Tensor memory columns of a warpgroup (256 each).
constexpr uint32_t kColS = 0, kColP0 = 0, kColP1 = 64, kColP2 = 96, kColT = 128;

template <int DP_, int TERMS_, bool PAIR_, int ET_> struct TcShape {
    static constexpr int DP = DP_, TERMS = TERMS_, ET = ET_;
    static constexpr bool PAIR = PAIR_;
    static constexpr int KT = TERMS == 1 ? 128 : 64;
    static constexpr int RT = PAIR ? 256 : 128;
    static constexpr int kHalf = 128 * 128;            // 128 rows of 64 dims
    static constexpr int kQTerm = RT * DP * 2;
    static constexpr int kJoin = PAIR ? 0 : 128 * DP * 4;
    static constexpr int kStage = TERMS * kQTerm > kJoin ? TERMS * kQTerm : kJoin;
    static constexpr int kSlot = KT * DP * 2;          // a k or a v tile
    static constexpr int kFit = (kSmemMost - kMisc - 1024 - kStage) / kSlot;
    static constexpr int kSlots = kFit < kMostSlots ? kFit : kMostSlots;
    static constexpr int kSmem = kMisc + 1024 + kStage + kSlots * kSlot;
    static_assert(kSlots >= 4, "a k and a v tile of each warpgroup");
};

struct Shared {
    uint64_t full[kMostSlots], empty[kMostSlots];
    uint64_t s_full[2], p_ready[2], t_full[2], q_ready, meet[3], drain;
    uint32_t none[kMostSlots][4];   // of a v tile: slots whose page is out of range
    uint32_t odd[2][2][4];          // slots whose v is not finite
    float2 ml[128];
    uint32_t tmem, abort;
};
static_assert(sizeof(Shared) <= kMisc, "the small arrays fit before the tiles");

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
__device__ __forceinline__ void st16(uint32_t at, const uint32_t (&r)[16]) {
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
// Has either half of w an exponent of all ones?
template <int ET> __device__ __forceinline__ bool odd16x2(uint32_t w) {
    constexpr uint32_t e = ET == kBF16 ? 0x7F80u : 0x7C00u;
    return (w & e) == e || (w & (e << 16)) == (e << 16);
}
// The fast tanh of 16-bit queries: within 2^-22 of 1 for any x; inf and NaN come out right.
__device__ __forceinline__ float fast_tanh(float x) {
    return 1.f - __fdividef(2.f, ex2(x * (2.f * kLog2e)) + 1.f);
}

__device__ __forceinline__ void cp16(uint32_t dst, const void *src, bool live) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
                 "r"(live ? 16 : 0)
                 : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N> __device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
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
    uint32_t stage, ring;  // shared-memory addresses of q and of the k and v tiles
    unsigned long long limit;
    unsigned *status;
    __device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity) const {
        return wait_or_abort(bar, parity, &sh->abort, limit, status);
    }
    // A warp gives up as one.
    __device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity) const {
        return __all_sync(0xFFFFFFFFu, wait(bar, parity));
    }
};

// -------------------------------------------------------------------- loader warps --

// The page of slot j, asked for a tile ahead of its use; -2 for one that is not live.
__device__ __forceinline__ int page_of(const KvView &kv, int seq, int j, int len) {
    if (j >= len) return -2;
    return kv.page_table[(long long)seq * kv.max_pages + kv.page_size.div((uint32_t)j)];
}

// The k and v tiles of the CTA's range, one after another, by TMA, one warp: where the pages are
// whole groups of eight rows, boxes of the largest number of rows that divides a page and a tile.
// What lies beyond the live slots of a page, or of a box that was not asked for, is whatever
// memory holds: no row sees it, and look() takes it out.
template <typename S>
__device__ void load_boxes(const TokensArgs &a, const KvView &kv, const CUtensorMap *k_map,
                           const CUtensorMap *v_map, int box, const Room &room, const Ctx &c) {
    const int lane = threadIdx.x & 31, boxes = S::KT / box, from = lane * box;
    const bool mine = lane < boxes;
    Walk walk(room, blockIdx.x);
    Stretch st;
    uint32_t n = 0;
    bool ok = true;
    while (ok && walk.next(st)) {
        const int len = mine ? st.tile.q.len : 0, seq = st.tile.seq;
        int j = st.k0 * S::KT + from, page = page_of(kv, seq, j, len);
        for (int kt = st.k0; kt < st.k1; ++kt, ++n, j += S::KT) {
            const int next = kt + 1 < st.k1 ? page_of(kv, seq, j + S::KT, len) : -2;
            const bool live = (unsigned)page < (unsigned)kv.n_pages;
            const uint32_t lost = __ballot_sync(0xFFFFFFFFu, !live && page != -2);
            const uint32_t bytes =
                __popc(__ballot_sync(0xFFFFFFFFu, live)) * box * 128 * (S::DP / 64);
            const int row = j - (int)(kv.page_size.div((uint32_t)j) * kv.page_size.d);
#pragma unroll
            for (int v = 0; v < 2; ++v) {
                const uint32_t i = 2 * n + v, slot = i % S::kSlots;
                if (!c.warp_wait(&c.sh->empty[slot], (i / S::kSlots & 1) ^ 1)) {
                    ok = false;
                    break;
                }
                if (lane == 0) {
                    if (v) {
                        for (int g = 0; g < S::KT / 32; ++g) {
                            uint32_t none = 0;
                            for (uint32_t left = lost; left; left &= left - 1) {
                                const int first = (__ffs(left) - 1) * box - 32 * g;
                                none |= below(first + box) & ~below(first);
                            }
                            c.sh->none[slot][g] = none;
                        }
                        if (lost) record_status(a.status, kStBadIndex);
                    }
                    mbar_arrive_expect_tx(&c.sh->full[slot], bytes);
                }
                __syncwarp();
                if (live) {
                    const uint32_t to = c.ring + slot * S::kSlot + from * 128;
#pragma unroll
                    for (int h = 0; h < S::DP / 64; ++h)
                        asm volatile(
                            "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx"
                            "::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
                                to + h * (S::KT * 128)),
                            "l"(reinterpret_cast<uint64_t>(v ? v_map : k_map)), "r"(64 * h),
                            "r"(row), "r"(st.head), "r"(page), "r"(smem_addr(&c.sh->full[slot]))
                            : "memory");
                }
                __syncwarp();
            }
            if (!ok) break;
            page = next;
        }
    }
    // The last copies have landed before shared memory is given up, after an abort too.
    const uint32_t asked = 2 * n, back = asked < (uint32_t)S::kSlots ? asked : S::kSlots;
    for (uint32_t i = asked - back; i < asked; ++i)
        mbar_wait(&c.sh->full[i % S::kSlots], i / S::kSlots & 1, kDrainPolls);
}

// The same by cp.async and three warps for pages of any size; a tile's barriers are arrived at
// when the next one is under way and it has landed.  Slots beyond the live ones and in pages out
// of range are zeros.
template <typename S>
__device__ void load_rows(const TokensArgs &a, const KvView &kv, const Room &room, const Ctx &c) {
    constexpr int kLanes = S::DP / 8;         // 16-byte chunks, a lane each, of a row
    constexpr int kRows = 32 / kLanes;        // rows of a warp's copy
    constexpr int kGroups = S::KT / 32;
    const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) - 9;
    Walk walk(room, blockIdx.x);
    Stretch st;
    uint32_t n = 0;         // tiles asked for
    uint32_t landed = 0;    // tiles whose barriers were arrived at
    bool ok = true;
    auto land = [&]() {
        fence_proxy_async_smem();
        mbar_arrive(&c.sh->full[2 * landed % S::kSlots]);
        mbar_arrive(&c.sh->full[(2 * landed + 1) % S::kSlots]);
        ++landed;
    };
    const int chunk = lane % kLanes;
    const bool in_dim = chunk * 8 < kv.head_dim;
    while (ok && walk.next(st)) {
        const int len = st.tile.q.len, seq = st.tile.seq;
        int page[kGroups];  // of this lane's rows: lane + 32 g
#pragma unroll
        for (int g = 0; g < kGroups; ++g)
            page[g] = page_of(kv, seq, st.k0 * S::KT + 32 * g + lane, len);
        for (int kt = st.k0; kt < st.k1; ++kt, ++n) {
            int next[kGroups];
#pragma unroll
            for (int g = 0; g < kGroups; ++g)
                next[g] = kt + 1 < st.k1
                              ? page_of(kv, seq, (kt + 1) * S::KT + 32 * g + lane, len) : -2;
            const uint32_t ks = 2 * n % S::kSlots, vs = (2 * n + 1) % S::kSlots;
            const uint32_t kp = (2 * n / S::kSlots & 1) ^ 1, vp = ((2 * n + 1) / S::kSlots & 1) ^ 1;
            if (!c.warp_wait(&c.sh->empty[ks], kp) || !c.warp_wait(&c.sh->empty[vs], vp)) {
                ok = false;
                break;
            }
            const uint32_t k_to = c.ring + ks * S::kSlot, v_to = c.ring + vs * S::kSlot;
#pragma unroll
            for (int g = 0; g < kGroups; ++g) {
                const int j = kt * S::KT + 32 * g + lane;
                const bool there = (unsigned)page[g] < (unsigned)kv.n_pages;
                const uint32_t none = __ballot_sync(0xFFFFFFFFu, !there && page[g] != -2);
                if (warp == 0 && lane == 0) {
                    c.sh->none[vs][g] = none;
                    if (none) record_status(a.status, kStBadIndex);
                }
                const int in = j - (int)(kv.page_size.div((uint32_t)j) * kv.page_size.d);
                const long long at = there ? (long long)page[g] * kv.page_stride +
                                                 (long long)st.head * kv.head_stride +
                                                 (long long)in * kv.token_stride
                                           : -1;
                for (int i = warp; i < 32 / kRows; i += 3) {
                    const int r = i * kRows + lane / kLanes, row = 32 * g + r;
                    const long long from = __shfl_sync(0xFFFFFFFFu, at, r);
                    const bool live = from >= 0 && in_dim;
                    const long long src = live ? from + chunk * 16 : 0;
                    const uint32_t to = (chunk >> 3) * (S::KT * 128) + row * 128 +
                                        (((chunk & 7) ^ (row & 7)) << 4);
                    cp16(k_to + to, kv.k + src, live);
                    cp16(v_to + to, kv.v + src, live);
                }
                page[g] = next[g];
            }
            cp_commit();
            if (n > landed) {
                cp_wait<1>();
                land();
            }
        }
    }
    cp_wait<0>();
    while (ok && landed < n) land();
}

// ------------------------------------------------------------------------ MMA warp --

template <typename S>
__device__ void issue_products(const TokensArgs &a, const Room &room, const Ctx &c) {
    const uint32_t tmem = c.sh->tmem;
    Walk walk(room, blockIdx.x);
    Stretch st;
    uint32_t base = 0;                 // tiles before this stretch
    uint32_t stretches = 0;
    uint32_t done[2] = {0, 0};         // tiles of each warpgroup whose P was taken
    constexpr uint32_t kId = idesc_of<S::ET>(S::KT, false), vId = idesc_of<S::ET>(S::DP, true);

    auto slot_full = [&](uint32_t i) {
        return c.wait(&c.sh->full[i % S::kSlots], i / S::kSlots & 1);
    };
    auto scores = [&](int wg, uint32_t tile) {  // S of a warpgroup from the tile's k
        const uint32_t k = desc_low(c.ring + 2 * tile % S::kSlots * S::kSlot, 16);
        uint32_t accum = 0;
#pragma unroll
        for (int t = S::TERMS - 1; t >= 0; --t) {
            const uint32_t q =
                desc_low(c.stage + t * S::kQTerm + (S::PAIR ? wg * (128 * S::DP * 2) : 0), 16);
#pragma unroll
            for (int h = 0; h < S::DP / 64; ++h)
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    mma_ss(tmem + wg * 256 + kColS, q + (h * S::kHalf + 32 * s >> 4),
                           k + (h * (S::KT * 128) + 32 * s >> 4), kId, accum);
                    accum = 1;
                }
        }
        tc_commit(&c.sh->s_full[wg]);
    };
    auto values = [&](int wg, uint32_t tile) {  // P V of a warpgroup from the tile's v
        const uint32_t v =
            desc_low(c.ring + (2 * tile + 1) % S::kSlots * S::kSlot, S::KT * 128);
        uint32_t accum = S::TERMS == 1;  // on top of the output, which began as zeros
#pragma unroll
        for (int t = S::TERMS - 1; t >= 0; --t) {
            const uint32_t p = tmem + wg * 256 + (t == 0 ? kColP0 : t == 1 ? kColP1 : kColP2);
#pragma unroll
            for (int s = 0; s < S::KT / 16; ++s) {
                mma_ts(tmem + wg * 256 + kColT, p + 8 * s, v + (2048 * s >> 4), vId, accum);
                accum = 1;
            }
        }
        tc_commit(&c.sh->t_full[wg]);
    };
    while (walk.next(st)) {
        const int n = st.k1 - st.k0;
        if (n == 0) continue;
        if (!c.wait(&c.sh->q_ready, stretches++ & 1)) return;
        tc_fence_after();
        if (S::PAIR) {
            if (!slot_full(2 * base)) return;
            tc_fence_after();
            scores(0, base);
            scores(1, base);
            tc_commit(&c.sh->empty[2 * base % S::kSlots]);
            for (int i = 0; i < n; ++i) {
                const uint32_t tile = base + i;
                if (!slot_full(2 * tile + 1)) return;
                if (i + 1 < n && !slot_full(2 * tile + 2)) return;
#pragma unroll
                for (int wg = 0; wg < 2; ++wg) {
                    if (!c.wait(&c.sh->p_ready[wg], done[wg]++ & 1)) return;
                    tc_fence_after();
                    values(wg, tile);
                    if (i + 1 < n) scores(wg, tile + 1);
                }
                tc_commit(&c.sh->empty[(2 * tile + 1) % S::kSlots]);
                if (i + 1 < n) tc_commit(&c.sh->empty[(2 * tile + 2) % S::kSlots]);
            }
        } else {
            for (int i = 0; i < 2 && i < n; ++i) {
                if (!slot_full(2 * (base + i))) return;
                tc_fence_after();
                scores(i, base + i);
                tc_commit(&c.sh->empty[2 * (base + i) % S::kSlots]);
            }
            for (int i = 0; i < n; ++i) {
                const uint32_t tile = base + i;
                const int wg = i & 1;
                if (!slot_full(2 * tile + 1)) return;
                if (!c.wait(&c.sh->p_ready[wg], done[wg]++ & 1)) return;
                tc_fence_after();
                values(wg, tile);
                tc_commit(&c.sh->empty[(2 * tile + 1) % S::kSlots]);
                if (i + 2 < n) {
                    if (!slot_full(2 * tile + 4)) return;
                    tc_fence_after();
                    scores(wg, tile + 2);
                    tc_commit(&c.sh->empty[(2 * tile + 4) % S::kSlots]);
                }
            }
        }
        base += n;
    }
}

// -------------------------------------------------------------- softmax warpgroups --

template <typename S>
__device__ __forceinline__ void load_q(const TokensArgs &a, const KvView &kv, const Seq &q,
                                       const Stretch &st, const Ctx &c, int first, int count,
                                       int thread, int threads) {
    constexpr int kChunks = S::DP / 8;
    const int group = a.group.d, rows = q.count * group - st.tile.row0, d = kv.head_dim;
    for (int i = thread; i < count * kChunks; i += threads) {
        const int r = first + i / kChunks, ch = i % kChunks;
        const bool live = r < rows && ch * 8 < d;
        const int rr = st.tile.row0 + r, j = a.group.div(live ? rr : 0), g = rr - j * group;
        const long long at =
            (q.t0 + j) * a.q_stride + (long long)(st.head * group + g) * d + ch * 8;
        // Row r of its tile of 128 rows.
        const uint32_t to = c.stage + (r >> 7) * (128 * S::DP * 2) + (ch >> 3) * S::kHalf +
                            (r & 127) * 128 + (((ch & 7) ^ (r & 7)) << 4);
        if (S::TERMS == 1) {
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (live) v = *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.q) + at);
            sts16(to, v);
        } else {
            float x[8] = {};
            if (live) {
                const float4 *p = reinterpret_cast<const float4 *>(static_cast<const float *>(a.q) + at);
                const float4 u = p[0], v = p[1];
                x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w;
                x[4] = v.x, x[5] = v.y, x[6] = v.z, x[7] = v.w;
            }
#pragma unroll
            for (int t = 0; t < S::TERMS; ++t) {
                uint32_t w[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    w[e] = pack2<kBF16>(x[2 * e], x[2 * e + 1]);
                    x[2 * e] -= bf16_lo(w[e]);
                    x[2 * e + 1] -= bf16_hi(w[e]);
                }
                sts16(to + t * S::kQTerm, make_uint4(w[0], w[1], w[2], w[3]));
            }
        }
    }
}

// tanh of the cap for f32 queries, within a few 2^-24 of itself: Lambert's continued fraction cut to
// z (945 + 105 z^2 + z^4) / (945 + 420 z^2 + 15 z^4) (off by 2e-9 at 0.5), beyond it by exponentials.
__device__ __forceinline__ float fine_tanh(float x) {
    const float z = x * x;
    const float small = x * fmaf(z, z + 105.f, 945.f) / fmaf(z, fmaf(z, 15.f, 420.f), 945.f);
    return z < 0.25f ? small : fast_tanh(x);
}

// A softmax thread's row of a stretch, and what the two kinds of softmax share.
template <typename S> struct Row {
    static constexpr int DP = S::DP, KT = S::KT, kChunks = KT / 32;
    static constexpr int kParts = DP / 64;             // rows of 128 bytes of a v
    static constexpr int kScan = S::PAIR ? 256 : 128;  // threads that look through a v tile
    static constexpr int kEach = KT * kParts > kScan ? KT * kParts / kScan : 1;
    const TokensArgs &a;
    const KvView &kv;
    const Ctx &c;
    Shared *const sh;
    const int wg, r, row;  // row of the row tile
    const uint32_t tm;     // the warpgroup's columns, this warp's lanes
    const bool formed;     // more than a positive scale: worked out once, written back in log2 units
    const float to_log2;
    uint32_t met[2] = {0, 0}, odd_turn = 0;
    // Of the stretch:
    Seq q;
    See see;
    float slope;
    bool live;
    int t, h;

    __device__ __forceinline__ Row(const TokensArgs &a_, const KvView &kv_, const Ctx &c_)
        : a(a_), kv(kv_), c(c_), sh(c_.sh), wg(threadIdx.x >> 7), r(threadIdx.x & 127),
          row(S::PAIR ? threadIdx.x : threadIdx.x & 127),
          tm(c_.sh->tmem + ((threadIdx.x & 96u) << 16) + (threadIdx.x >> 7) * 256),
          formed(a_.softcap > 0.f || a_.slopes || !(a_.scale > 0.f)),
          to_log2(formed ? 1.f : a_.scale * kLog2e) {}

    __device__ __forceinline__ void begin(const Stretch &st) {
        q = st.tile.q;
        const int group = a.group.d;
        live = row < min(S::RT, q.count * group - st.tile.row0);
        const int rr = st.tile.row0 + (live ? row : 0), j = a.group.div(rr), g = rr - j * group;
        see = See{};
        if (live) see = see_of(a, q, st.tile.seq, j);
        slope = a.slopes ? a.slopes[st.head * group + g] * kLog2e : 0.f;
        t = q.t0 + j, h = st.head * group + g;
    }
    // 0: both warpgroups; 1: those that look through a v tile together.
    __device__ __forceinline__ bool meet(int which) {
        uint64_t *const bar = &sh->meet[S::PAIR || which == 0 ? 0 : 1 + wg];
        const uint32_t turn = met[S::PAIR ? 0 : which]++;
        mbar_arrive(bar);
        return c.warp_wait(bar, turn & 1);
    }
    // Scores in tensor memory to log2 units after cap and bias, those that are not seen to -inf.
    __device__ __forceinline__ void form(int j0, bool mixed, const uint32_t *none) {
#pragma unroll 1
        for (int ch = 0; ch < kChunks; ++ch) {
            const int jc = j0 + 32 * ch;
            uint32_t v[32];
            ld32(v, tm + kColS + 32 * ch);
            wait_ld(v);
            if (formed) {
                const bool own = a.pos && jc + 32 > q.base;
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    float y = __uint_as_float(v[e]) * a.scale;
                    if (a.softcap > 0.f) {
                        const float z = __fdividef(y, a.softcap);
                        y = a.softcap * (S::TERMS == 1 ? fast_tanh(z) : fine_tanh(z));
                    }
                    v[e] = __float_as_uint(y * kLog2e);
                }
                if (a.slopes) {
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        const int far = (own ? slot_pos(a, q, jc + e) : jc + e) - see.pos;
                        v[e] = __float_as_uint(fmaf(slope, (float)far, __uint_as_float(v[e])));
                    }
                }
            }
            if (mixed) {
                const uint32_t in = seen32(a, see, jc) & ~none[ch];
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    if (!(in >> e & 1u)) v[e] = 0xFF800000u;
            }
            st32(tm + kColS + 32 * ch, v);
        }
        wait_st();
    }
    // Finds the slots of a v tile that are not finite; `any` is the same for all that look.
    struct Odd {
        uint32_t any, *words;
        bool mine;
    };
    __device__ __forceinline__ bool look(uint32_t v_at, Odd &o) {
        const int at = S::PAIR ? threadIdx.x : r;
        const int slot = at % KT, part0 = at / KT, scan_warp = at >> 5;
        o.mine = false;
        if (part0 < kParts) {
#pragma unroll 1
            for (int p = 0; p < kEach; ++p) {
                const uint32_t line = v_at + (part0 + p) * (KT * 128) + slot * 128;
#pragma unroll
                for (int ch = 0; ch < 8; ++ch) {
                    const uint4 w = lds16(line + (((ch + slot) & 7) << 4));
                    o.mine |= odd16x2<S::ET>(w.x) || odd16x2<S::ET>(w.y) ||
                              odd16x2<S::ET>(w.z) || odd16x2<S::ET>(w.w);
                }
            }
        }
        const uint32_t found = __ballot_sync(0xFFFFFFFFu, o.mine);
        // Two sets taken in turn: a warpgroup may be a tile ahead of the other's reading.
        o.words = &sh->odd[S::PAIR ? odd_turn++ & 1 : wg][0][0];
        if ((threadIdx.x & 31) == 0)
            o.words[scan_warp * 32 / KT * 4 + scan_warp * 32 % KT / 32] = found;
        if (!meet(1)) return false;
        o.any = 0;
#pragma unroll
        for (int ch = 0; ch < kChunks; ++ch) o.any |= word(o, ch);
        return true;
    }
    __device__ __forceinline__ static uint32_t word(const Odd &o, int ch) {
        uint32_t w = o.words[ch];
        if (kScan / KT > 1 && kParts > 1) w |= o.words[4 + ch];
        return w;
    }
    // f(slot, p) for each of them that the row sees, p its weight against the maximum `safe`; every
    // lane comes along.
    template <typename F>
    __device__ __forceinline__ void each_odd(const Odd &o, int j0, const uint32_t *none, float safe,
                                             F f) {
#pragma unroll 1
        for (int ch = 0; ch < kChunks; ++ch) {
            const uint32_t in = seen32(a, see, j0 + 32 * ch) & ~none[ch];
#pragma unroll 1
            for (uint32_t left = word(o, ch); left; left &= left - 1) {
                const int b = __ffs(left) - 1;
                __syncwarp();
                const float x = ld1(tm + kColS + 32 * ch + b);
                f(32 * ch + b, (in >> b & 1u) != 0, ex2(fmaf(x, to_log2, -safe)));
            }
        }
    }
    // Eight dims of a slot's v.
    __device__ __forceinline__ static void v8(uint32_t v_at, int slot, int chunk, float (&x)[8]) {
        const uint4 u = lds16(v_at + (chunk >> 3) * (KT * 128) + slot * 128 +
                              (((chunk & 7) ^ (slot & 7)) << 4));
        const uint32_t z[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = widen<S::ET>(z[k >> 1], k & 1);
    }
    // Takes those slots out of the tile once every row has them.
    __device__ __forceinline__ bool clear(uint32_t v_at, const Odd &o) {
        if (!meet(1)) return false;
        const int at = S::PAIR ? threadIdx.x : r;
        const int slot = at % KT, part0 = at / KT;
        if (word(o, slot >> 5) >> (slot & 31) & 1u) {
#pragma unroll 1
            for (int p = 0; p < kEach && part0 + p < kParts; ++p)
#pragma unroll
                for (int ch = 0; ch < 8; ++ch)
                    sts16(v_at + (part0 + p) * (KT * 128) + slot * 128 + ch * 16,
                          make_uint4(0u, 0u, 0u, 0u));
        }
        fence_proxy_async_smem();
        return true;
    }
    // Dims e .. e + 7 of the row's result.
    __device__ __forceinline__ void put8(int e, const float (&x)[8]) const {
        if (e >= kv.head_dim) return;
        const long long to = t * a.out_stride + (long long)h * kv.head_dim + e;
        if (a.out_type == kF32) {
            float4 *const p = reinterpret_cast<float4 *>(static_cast<float *>(a.out) + to);
            p[0] = make_float4(x[0], x[1], x[2], x[3]);
            p[1] = make_float4(x[4], x[5], x[6], x[7]);
        } else {
            *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out) + to) =
                make_uint4(pack2<S::ET>(x[0], x[1]), pack2<S::ET>(x[2], x[3]),
                           pack2<S::ET>(x[4], x[5]), pack2<S::ET>(x[6], x[7]));
        }
    }
    // Dims e .. e + 7 of the row's sums: its result, or its part.
    __device__ __forceinline__ void finish(const Room &room, const Stretch &st, float m, float l,
                                           int e, const float (&x)[8]) const {
        if (st.part >= 0) {
            const size_t part = 2 * blockIdx.x + st.part;
            room.part_o[(part * (DP / 4) + e / 4) * S::RT + row] =
                make_float4(x[0], x[1], x[2], x[3]);
            room.part_o[(part * (DP / 4) + e / 4 + 1) * S::RT + row] =
                make_float4(x[4], x[5], x[6], x[7]);
            if (e == 0) room.part_ml[part * S::RT + row] = make_float2(m, l);
            return;
        }
        const float inv = l == 0.f ? 0.f : 1.f / l;
        float y[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) y[k] = x[k] * inv;
        put8(e, y);
        if (e == 0 && a.lse) a.lse[(long long)t * a.h_q + h] = lse_of(m, l);
    }
};

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

// 16-bit queries: the output in tensor memory.
template <typename S>
__device__ void softmax_16(const TokensArgs &a, const KvView &kv, const Room &room, const Ctx &c) {
    constexpr int DP = S::DP, KT = S::KT, kChunks = KT / 32;
    constexpr float kGrow = 8.f;  // p is at most 2^8: f16 holds it, and its sum
    Row<S> w(a, kv, c);
    Shared *const sh = c.sh;
    Walk walk(room, blockIdx.x);
    Stretch st;
    uint32_t base = 0, mine = 0;  // tiles before this stretch; tiles of this warpgroup
    bool again = false;
    while (walk.next(st)) {
        __syncwarp();
        w.begin(st);
        const int n = st.k1 - st.k0;
        float m = -INFINITY, l = 0.f;
        bool some = false;
        if (n > 0) {
            if (!S::PAIR && again && !w.meet(0)) return;  // the last stretch's join was read
            again = true;
            uint32_t zero[32] = {};
#pragma unroll
            for (int ch = 0; ch < DP / 32; ++ch) st32(w.tm + kColT + 32 * ch, zero);
            if (S::PAIR)
                load_q<S>(a, kv, w.q, st, c, w.wg * 128, 128, w.r, 128);
            else
                load_q<S>(a, kv, w.q, st, c, 0, 128, threadIdx.x, 256);
            fence_proxy_async_smem();
            mbar_arrive(&sh->q_ready);
        }
        for (int i = S::PAIR ? 0 : w.wg; i < n; i += S::PAIR ? 1 : 2) {
            const uint32_t vi = 2 * (base + i) + 1, vs = vi % S::kSlots;
            if (!c.warp_wait(&sh->full[vs], vi / S::kSlots & 1)) return;
            if (!c.warp_wait(&sh->s_full[w.wg], mine & 1)) return;
            tc_fence_after();
            const int j0 = (st.k0 + i) * KT;
            uint32_t lost = 0;
#pragma unroll
            for (int ch = 0; ch < kChunks; ++ch) lost |= sh->none[vs][ch];
            const bool mixed = j0 < st.tile.lo || j0 + KT > st.tile.hi || lost;
            if (w.formed || mixed) w.form(j0, mixed, sh->none[vs]);
            uint32_t s[kChunks][32];
#pragma unroll
            for (int ch = 0; ch < kChunks; ++ch) ld32(s[ch], w.tm + kColS + 32 * ch);
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
            const float now =
                fmaxf(m, fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3])) * w.to_log2);
            if (__any_sync(0xFFFFFFFFu, now > m + kGrow || m == -INFINITY)) {
                const float f = ex2(m - (now == -INFINITY ? 0.f : now));
                m = now;
                l *= f;
                if (some) {
                    if (!c.warp_wait(&sh->t_full[w.wg], (mine - 1) & 1)) return;
                    tc_fence_after();
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
            }
            const float safe = m == -INFINITY ? 0.f : m;
            if (mixed) {
                const uint32_t v_at = c.ring + vs * S::kSlot;
                typename Row<S>::Odd odd;
                if (!w.look(v_at, odd)) return;
                if (odd.any) {
                    if (some && !c.warp_wait(&sh->t_full[w.wg], (mine - 1) & 1)) return;
                    tc_fence_after();
                    wait_st();
#pragma unroll 1
                    for (int ch = 0; ch < DP / 32; ++ch) {
                        uint32_t v[32];
                        ld32(v, w.tm + kColT + 32 * ch);
                        wait_ld(v);
                        w.each_odd(odd, j0, sh->none[vs], safe, [&](int slot, bool in, float p) {
#pragma unroll
                            for (int e = 0; e < 32; e += 8) {
                                float x[8];
                                w.v8(v_at, slot, 4 * ch + e / 8, x);
#pragma unroll
                                for (int k = 0; k < 8; ++k)
                                    if (in)
                                        v[e + k] = __float_as_uint(
                                            fmaf(p, x[k], __uint_as_float(v[e + k])));
                            }
                        });
                        st32(w.tm + kColT + 32 * ch, v);
                    }
                    if (!w.clear(v_at, odd)) return;
                }
            }
            float sums[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int ch = 0; ch < kChunks; ++ch) {
                uint32_t p[16];
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    float x, y;
                    fma2(x, y, __uint_as_float(s[ch][2 * e]), __uint_as_float(s[ch][2 * e + 1]),
                         w.to_log2, -safe);
                    x = ex2(x), y = ex2(y);
                    add2(sums[2 * (e & 1)], sums[2 * (e & 1) + 1], x, y);
                    p[e] = pack2<S::ET>(x, y);
                }
                st16(w.tm + kColP0 + 16 * ch, p);
            }
            l += (sums[0] + sums[1]) + (sums[2] + sums[3]);
            wait_st();
            tc_fence_before();
            mbar_arrive(&sh->p_ready[w.wg]);
            ++mine;
            some = true;
        }
        base += n;
        if (some && !c.warp_wait(&sh->t_full[w.wg], (mine - 1) & 1)) return;
        tc_fence_after();
        float fa = 1.f, fb = 0.f;
        if (!S::PAIR && n > 0) {
            // The two warpgroups' halves of the slots.
            if (!w.meet(0)) return;  // every product of q is done
            if (w.wg == 1) {
#pragma unroll 1
                for (int ch = 0; ch < DP / 32; ++ch) {
                    uint32_t v[32];
                    ld32(v, w.tm + kColT + 32 * ch);
                    wait_ld(v);
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        asm volatile("st.shared.u32 [%0], %1;" ::"r"(
                                         c.stage + ((32 * ch + e) * 128 + w.r) * 4),
                                     "r"(v[e])
                                     : "memory");
                }
                sh->ml[w.r] = make_float2(m, l);
            }
            if (!w.meet(0)) return;
            if (w.wg == 1) continue;
            const float2 other = sh->ml[w.r];
            const float both = fmaxf(m, other.x), safe = both == -INFINITY ? 0.f : both;
            fa = ex2(m - safe), fb = ex2(other.x - safe);
            m = both;
            l = fmaf(l, fa, other.y * fb);
        } else if (!S::PAIR && w.wg == 1) {
            continue;
        }
#pragma unroll 1
        for (int ch = 0; ch < DP / 32; ++ch) {
            uint32_t v[32] = {};
            if (n > 0) {
                ld32(v, w.tm + kColT + 32 * ch);
                wait_ld(v);
                if (!S::PAIR) {
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        float x;
                        asm volatile("ld.shared.f32 %0, [%1];"
                                     : "=f"(x)
                                     : "r"(c.stage + ((32 * ch + e) * 128 + w.r) * 4)
                                     : "memory");
                        v[e] = __float_as_uint(fmaf(__uint_as_float(v[e]), fa, x * fb));
                    }
                }
            }
            if (w.live) {
#pragma unroll
                for (int e = 0; e < 32; e += 8) {
                    float x[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) x[k] = __uint_as_float(v[e + k]);
                    w.finish(room, st, m, l, 32 * ch + e, x);
                }
            }
            __syncwarp();
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
    bool again = false;
    while (walk.next(st)) {
        __syncwarp();
        w.begin(st);
        const int n = st.k1 - st.k0;
        float o[DP];
#pragma unroll
        for (int e = 0; e < DP; ++e) o[e] = 0.f;
        float m = -INFINITY, l = 0.f, f = 0.f;
        bool pending = false;
        if (n > 0) {
            if (again && !w.meet(0)) return;  // the last stretch's join was read
            again = true;
            load_q<S>(a, kv, w.q, st, c, 0, 128, threadIdx.x, 256);
            fence_proxy_async_smem();
            mbar_arrive(&sh->q_ready);
        }
        // o = o f + T of the tile before.
        auto take = [&]() {
            if (!c.warp_wait(&sh->t_full[w.wg], (mine - 1) & 1)) return false;
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
        for (int i = w.wg; i < n; i += 2) {
            if (pending && !take()) return;
            const uint32_t vi = 2 * (base + i) + 1, vs = vi % S::kSlots;
            if (!c.warp_wait(&sh->full[vs], vi / S::kSlots & 1)) return;
            if (!c.warp_wait(&sh->s_full[w.wg], mine & 1)) return;
            tc_fence_after();
            const int j0 = (st.k0 + i) * KT;
            uint32_t lost = 0;
#pragma unroll
            for (int ch = 0; ch < kChunks; ++ch) lost |= sh->none[vs][ch];
            const bool mixed = j0 < st.tile.lo || j0 + KT > st.tile.hi || lost;
            if (w.formed || mixed) w.form(j0, mixed, sh->none[vs]);
            float top = -INFINITY;
#pragma unroll
            for (int ch = 0; ch < kChunks; ++ch) {
                uint32_t v[32];
                ld32(v, w.tm + kColS + 32 * ch);
                wait_ld(v);
#pragma unroll
                for (int e = 0; e < 32; ++e) top = fmaxf(top, __uint_as_float(v[e]));
            }
            const float now = fmaxf(m, top * w.to_log2);
            const float safe = now == -INFINITY ? 0.f : now;
            const float fl = ex2(m - safe);
            f = fl;
            m = now;
            if (mixed) {
                const uint32_t v_at = c.ring + vs * S::kSlot;
                typename Row<S>::Odd odd;
                if (!w.look(v_at, odd)) return;
                if (odd.any) {
#pragma unroll
                    for (int e = 0; e < DP; ++e) o[e] *= f;
                    f = 1.f;
                    w.each_odd(odd, j0, sh->none[vs], safe, [&](int slot, bool in, float p) {
#pragma unroll
                        for (int e = 0; e < DP; e += 8) {
                            float x[8];
                            w.v8(v_at, slot, e / 8, x);
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                if (in) o[e + k] = fmaf(p, x[k], o[e + k]);
                        }
                    });
                    if (!w.clear(v_at, odd)) return;
                }
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
            mbar_arrive(&sh->p_ready[w.wg]);
            ++mine;
            pending = true;
        }
        if (pending && !take()) return;
        base += n;
        if (n > 0) {
            // The two warpgroups' halves of the slots.
            if (!w.meet(0)) return;  // every product of q is done
            if (w.wg == 1) {
#pragma unroll
                for (int e = 0; e < DP; ++e)
                    asm volatile("st.shared.f32 [%0], %1;" ::"r"(c.stage + (e * 128 + w.r) * 4),
                                 "f"(o[e])
                                 : "memory");
                sh->ml[w.r] = make_float2(m, l);
            }
            if (!w.meet(0)) return;
            if (w.wg == 0) {
                const float2 other = sh->ml[w.r];
                const float both = fmaxf(m, other.x), safe = both == -INFINITY ? 0.f : both;
                const float fa = ex2(m - safe), fb = ex2(other.x - safe);
                m = both;
                l = fmaf(l, fa, other.y * fb);
#pragma unroll
                for (int e = 0; e < DP; ++e) {
                    float x;
                    asm volatile("ld.shared.f32 %0, [%1];"
                                 : "=f"(x)
                                 : "r"(c.stage + (e * 128 + w.r) * 4)
                                 : "memory");
                    o[e] = fmaf(o[e], fa, x * fb);
                }
            }
        }
        if (!w.live || w.wg == 1) continue;
#pragma unroll
        for (int e = 0; e < DP; e += 8) {
            float x[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) x[k] = o[e + k];
            w.finish(room, st, m, l, e, x);
        }
    }
}

template <typename S>
__global__ void __launch_bounds__(kThreads, 1)
    attn_tokens_tc_kernel(TokensArgs a, KvView kv, const __grid_constant__ CUtensorMap k_map,
                          const __grid_constant__ CUtensorMap v_map, int box) {
    extern __shared__ __align__(1024) uint8_t smem[];
    Ctx c;
    c.sh = reinterpret_cast<Shared *>(smem);
    c.stage = (smem_addr(smem) + kMisc + 1023) & ~1023u;
    c.ring = c.stage + S::kStage;
    c.limit = a.wait_limit;
    c.status = a.status;
    const int warp = threadIdx.x >> 5;
    pdl_launch();
    if (threadIdx.x == 0) {
        if (box) prefetch_tmap(&k_map), prefetch_tmap(&v_map);
        for (int i = 0; i < kMostSlots; ++i) {
            mbar_init(&c.sh->full[i], box ? 1 : kLoaders);
            mbar_init(&c.sh->empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&c.sh->s_full[i], 1);
            mbar_init(&c.sh->p_ready[i], 128);
            mbar_init(&c.sh->t_full[i], 1);
            mbar_init(&c.sh->meet[1 + i], 128);
        }
        mbar_init(&c.sh->meet[0], 256);
        mbar_init(&c.sh->q_ready, 256);
        mbar_init(&c.sh->drain, 1);
        c.sh->abort = 0u;
        fence_mbar_init();
    }
    if (warp == 8) {
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
    // 384 threads of 168 registers at the launch: 2 x 216 + 72 and 2 x 224 + 56 are 3 x 168.
    if (warp < 8) {
        if constexpr (S::TERMS == 1)
            asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
        else
            asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
        if constexpr (S::TERMS == 1)
            softmax_16<S>(a, kv, room, c);
        else
            softmax_32<S>(a, kv, room, c);
    } else {
        if constexpr (S::TERMS == 1)
            asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
        else
            asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        if (warp > 8) {
            fence_proxy_async_global();  // k and v may be an earlier kernel's plain stores
            if (!box)
                load_rows<S>(a, kv, room, c);
            else if (warp == 9)
                load_boxes<S>(a, kv, &k_map, &v_map, box, room, c);
        } else if ((threadIdx.x & 31) == 0) {
            issue_products<S>(a, room, c);
            // Every product is done before tensor memory and the tiles are given up.
            tc_commit(&c.sh->drain);
            mbar_wait(&c.sh->drain, 0, kDrainPolls);
        }
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 8) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(c.sh->tmem),
                     "r"(512u)
                     : "memory");
    }
}

// Two row tiles of 128 where the sequences have more rows than one on average.
bool pairs_rows(int n_seq, int n_tok, int group) {
    return (long long)n_tok * group > 128ll * n_seq;
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
// A pool as [page][head][row][dim] in boxes of `box` rows of 64 dims, zeros beyond head_dim.
bool pool_map(CUtensorMap &map, const KvView &kv, char *pool, int box) {
    const PFN_cuTensorMapEncodeTiled_v12000 encode = encode_fn();
    const cuuint64_t dims[4] = {(cuuint64_t)kv.head_dim, kv.page_size.d, (cuuint64_t)kv.n_heads,
                                (cuuint64_t)kv.n_pages};
    const cuuint64_t strides[3] = {(cuuint64_t)kv.token_stride, (cuuint64_t)kv.head_stride,
                                   (cuuint64_t)kv.page_stride};
    for (cuuint64_t st : strides)
        if (st >= (1ull << 40)) return false;
    const cuuint32_t boxes[4] = {64, (cuuint32_t)box, 1, 1}, steps[4] = {1, 1, 1, 1};
    return encode && encode(&map,
                            kv.dtype == kBF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                              : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
                            4, pool, dims, strides, boxes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// Rows of a box: the largest power of two, 8 at least, that divides a page and a tile; 0: none.
int box_of(const KvView &kv, int kt) {
    int box = kt;
    while (kv.page_size.d % box) box /= 2;
    return box >= 8 ? box : 0;
}

template <int DP, int TERMS, bool PAIR, int ET>
cudaError_t launch_shape(const TokensArgs &a, const KvView &kv, const DeviceInfo &dev,
                         cudaStream_t stream) {
    using S = TcShape<DP, TERMS, PAIR, ET>;
    static std::atomic<unsigned long long> raised{0};
    cudaError_t err = ensure_smem(attn_tokens_tc_kernel<S>, S::kSmem, dev, raised);
    if (err != cudaSuccess) return err;
    err = launch_attn_plan(a, kv, S::RT, S::KT, DP, kGrid, stream);
    if (err != cudaSuccess) return err;
    CUtensorMap k_map{}, v_map{};
    int box = box_of(kv, S::KT);
    if (box && !(pool_map(k_map, kv, kv.k, box) && pool_map(v_map, kv, kv.v, box))) box = 0;
    err = launch_pdl(attn_tokens_tc_kernel<S>, dim3(kGrid), dim3(kThreads), S::kSmem, stream, a, kv,
                     k_map, v_map, box);
    if (err != cudaSuccess) return err;
    return launch_attn_parts(a, kv, S::RT, DP, kGrid, stream);
}
template <int DP>
cudaError_t launch_dim(const TokensArgs &a, const KvView &kv, const DeviceInfo &dev,
                       cudaStream_t stream) {
    if (a.q_type == kF32) return launch_shape<DP, 3, false, kBF16>(a, kv, dev, stream);
    const bool pair = pairs_rows(a.n_seq, a.n_tok, a.group.d);
    if (kv.dtype == kBF16)
        return pair ? launch_shape<DP, 1, true, kBF16>(a, kv, dev, stream)
                    : launch_shape<DP, 1, false, kBF16>(a, kv, dev, stream);
    return pair ? launch_shape<DP, 1, true, kF16>(a, kv, dev, stream)
                : launch_shape<DP, 1, false, kF16>(a, kv, dev, stream);
}

}  // namespace

bool tokens_tc_takes(const KvView &kv, int q_type) {
    if (kv.head_dim > 128) return false;
    return kv.dtype == kBF16 ? q_type != kF16 : kv.dtype == kF16 && q_type == kF16;
}

void tokens_tc_shape(int n_seq, int n_tok, int group, int q_type, int head_dim, int &rt, int &dp,
                     int &grid) {
    rt = q_type != kF32 && pairs_rows(n_seq, n_tok, group) ? 256 : 128;
    dp = head_dim <= 64 ? 64 : 128;
    grid = kGrid;
}

cudaError_t launch_tokens_tc(const TokensArgs &a, const KvView &kv, const DeviceInfo &dev,
                             cudaStream_t stream) {
    return kv.head_dim <= 64 ? launch_dim<64>(a, kv, dev, stream)
                             : launch_dim<128>(a, kv, dev, stream);
}

}  // namespace tok
}  // namespace wq

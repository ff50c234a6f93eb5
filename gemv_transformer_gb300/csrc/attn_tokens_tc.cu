// attn_tokens_tc.cu -- attention of several new tokens per sequence on the tcgen05 tensor cores.
//
// S = Q K^T and T = P V for 128 rows (new tokens x heads of a group) and a tile of KT slots, both
// accumulated in tensor memory; between them two warpgroups of 128 threads, a thread to a row,
// turn S into weights against a running maximum, and add the previous tile's T to an output in
// registers: o = o 2^(m_old - m) + T.  So no sum on the tensor core is longer than one
// tile (it truncates when it accumulates), and a rescale is part of an FMA that is needed
// anyway.
//
//   16-bit q    one product each; p is rounded to the cache's type, its sum is not.
//   f32 q       (bf16 caches) q and p as three bf16 terms, 24 bits, whose products are exact: three
//               products each, the smallest terms first.
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

// A's rows in tensor memory.
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc,
                                          uint32_t accum) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(accum)
        : "memory");
}
// 64-column chunks of the contiguous dimension `chunk` bytes apart, groups of eight rows 1024.
__device__ __forceinline__ uint64_t smem_desc_mn(uint32_t addr, uint32_t chunk) {
    return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)(chunk >> 4) << 16) |
           ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
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

// The k and v tiles of the CTA's range, one after another, by cp.async; a tile's barriers are
// arrived at when the next one is under way and it has landed.  Slots beyond the live ones and
// in pages out of range are zeros.
template <typename S>
__device__ void load_tiles(const TokensArgs &a, const KvView &kv, const Room &room, const Ctx &c) {
    constexpr int kLanes = S::DP / 8;         // 16-byte chunks, a lane each, of a row
    constexpr int kRows = 32 / kLanes;        // rows of a warp's copy
    constexpr int kGroups = S::KT / 32;
    const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) - 9;
    Walk walk(room, blockIdx.x, room.plan[kGrid].pad);
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
        bool bad = false;
        const Seq q = seq_of(a, st.tile.seq, bad);
        for (int kt = st.k0; kt < st.k1; ++kt, ++n) {
            // This lane's rows of the tile: lane + 32 g.
            long long at[kGroups];
#pragma unroll
            for (int g = 0; g < kGroups; ++g) {
                const int j = kt * S::KT + 32 * g + lane;
                at[g] = -1;
                if (j < q.len) {
                    at[g] = kv.row(st.tile.seq, st.head, j);
                    if (at[g] < 0) at[g] = -2;
                }
            }
            const uint32_t ks = 2 * n % S::kSlots, vs = (2 * n + 1) % S::kSlots;
            const uint32_t kp = (2 * n / S::kSlots & 1) ^ 1, vp = ((2 * n + 1) / S::kSlots & 1) ^ 1;
            if (!c.warp_wait(&c.sh->empty[ks], kp) || !c.warp_wait(&c.sh->empty[vs], vp)) {
                ok = false;
                break;
            }
            if (warp == 0) {
#pragma unroll
                for (int g = 0; g < kGroups; ++g) {
                    const uint32_t none = __ballot_sync(0xFFFFFFFFu, at[g] == -2);
                    if (lane == 0) {
                        c.sh->none[vs][g] = none;
                        if (none) record_status(a.status, kStBadIndex);
                    }
                }
            }
            const uint32_t k_to = c.ring + ks * S::kSlot, v_to = c.ring + vs * S::kSlot;
#pragma unroll
            for (int g = 0; g < kGroups; ++g) {
                for (int i = warp; i < 32 / kRows; i += 3) {
                    const int r = i * kRows + lane / kLanes, row = 32 * g + r;
                    const long long from = __shfl_sync(0xFFFFFFFFu, at[g], r);
                    const bool live = from >= 0 && in_dim;
                    const long long src = live ? from + chunk * 16 : 0;
                    const uint32_t to = (chunk >> 3) * (S::KT * 128) + row * 128 +
                                        (((chunk & 7) ^ (row & 7)) << 4);
                    cp16(k_to + to, kv.k + src, live);
                    cp16(v_to + to, kv.v + src, live);
                }
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
    Walk walk(room, blockIdx.x, room.plan[kGrid].pad);
    Stretch st;
    uint32_t base = 0;                 // tiles before this stretch
    uint32_t stretches = 0;
    uint32_t done[2] = {0, 0};         // tiles of each warpgroup whose P was taken
    constexpr uint32_t kId = idesc_of<S::ET>(S::KT, false), vId = idesc_of<S::ET>(S::DP, true);

    auto slot_full = [&](uint32_t i) {
        return c.wait(&c.sh->full[i % S::kSlots], i / S::kSlots & 1);
    };
    auto scores = [&](int wg, uint32_t tile) {  // S of a warpgroup from the tile's k
        const uint32_t k = c.ring + 2 * tile % S::kSlots * S::kSlot;
        uint32_t accum = 0;
#pragma unroll
        for (int t = S::TERMS - 1; t >= 0; --t) {
            const uint32_t q = c.stage + t * S::kQTerm + (S::PAIR ? wg * (128 * S::DP * 2) : 0);
#pragma unroll
            for (int h = 0; h < S::DP / 64; ++h)
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    tc_mma(tmem + wg * 256 + kColS, smem_desc_sw128(q + h * S::kHalf + 32 * s),
                           smem_desc_sw128(k + h * (S::KT * 128) + 32 * s), kId, accum);
                    accum = 1;
                }
        }
        tc_commit(&c.sh->s_full[wg]);
    };
    auto values = [&](int wg, uint32_t tile) {  // T of a warpgroup from the tile's v
        const uint32_t v = c.ring + (2 * tile + 1) % S::kSlots * S::kSlot;
        uint32_t accum = 0;
#pragma unroll
        for (int t = S::TERMS - 1; t >= 0; --t) {
            const uint32_t p = tmem + wg * 256 + (t == 0 ? kColP0 : t == 1 ? kColP1 : kColP2);
#pragma unroll
            for (int s = 0; s < S::KT / 16; ++s) {
                tc_mma_ts(tmem + wg * 256 + kColT, p + 8 * s,
                          smem_desc_mn(v + 2048 * s, S::KT * 128), vId, accum);
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

template <typename S>
__device__ void softmax_rows(const TokensArgs &a, const KvView &kv, const Room &room,
                             const Ctx &c) {
    constexpr int DP = S::DP, KT = S::KT, kChunks = KT / 32;
    constexpr bool kFast = S::TERMS == 1;
    Shared *const sh = c.sh;
    const int wg = threadIdx.x >> 7, r = threadIdx.x & 127, warp = (threadIdx.x >> 5) & 3;
    const int row = S::PAIR ? threadIdx.x : r;  // of the row tile
    const uint32_t lanes = (uint32_t)(warp * 32) << 16;
    const uint32_t tm = sh->tmem + lanes + wg * 256;
    const int group = a.group.d;
    // A form beyond scale and mask is worked out once and written back in log2 units.
    const bool formed = a.softcap > 0.f || a.slopes || !(a.scale > 0.f);
    const float to_log2 = formed ? 1.f : a.scale * kLog2e;
    const TypedOut out{a.out, a.out_type};

    uint32_t met[2] = {0, 0}, odd_turn = 0;
    uint64_t *const scan_bar = S::PAIR ? &sh->meet[0] : &sh->meet[1 + wg];
    auto meet = [&](int which) {  // 0: both warpgroups, 1: those that look through a v tile
        uint64_t *const bar = which == 0 ? &sh->meet[0] : scan_bar;
        const uint32_t turn = S::PAIR ? met[0]++ : met[which]++;
        mbar_arrive(bar);
        return c.warp_wait(bar, turn & 1);
    };

    Walk walk(room, blockIdx.x, room.plan[kGrid].pad);
    Stretch st;
    uint32_t base = 0, mine = 0;  // tiles before this stretch; tiles of this warpgroup
    bool again = false;
    while (walk.next(st)) {
        __syncwarp();
        bool bad = false;
        const Seq q = seq_of(a, st.tile.seq, bad);
        const int rows = min(S::RT, q.count * group - st.tile.row0);
        const bool live = row < rows;
        const int rr = st.tile.row0 + (live ? row : 0), j = a.group.div(rr), g = rr - j * group;
        See see{};
        if (live) see = see_of(a, q, st.tile.seq, j);
        const float slope = a.slopes ? a.slopes[st.head * group + g] * kLog2e : 0.f;
        const int n = st.k1 - st.k0;

        float o[DP];
#pragma unroll
        for (int e = 0; e < DP; ++e) o[e] = 0.f;
        float m = -INFINITY, l = 0.f, f = 0.f;
        bool pending = false;
        if (n > 0) {
            if (!S::PAIR && again && !meet(0)) return;  // the last stretch's join was read
            if (S::PAIR)
                load_q<S>(a, kv, q, st, c, wg * 128, 128, r, 128);
            else
                load_q<S>(a, kv, q, st, c, 0, 128, threadIdx.x, 256);
            again = true;
            fence_proxy_async_smem();
            mbar_arrive(&sh->q_ready);
        }
        // o = o f + T of the tile before.
        auto take = [&]() {
            if (!c.warp_wait(&sh->t_full[wg], (mine - 1) & 1)) return false;
            tc_fence_after();
#pragma unroll
            for (int ch = 0; ch < DP / 32; ++ch) {
                uint32_t v[32];
                ld32(v, tm + kColT + 32 * ch);
                wait_ld(v);
#pragma unroll
                for (int e = 0; e < 32; ++e)
                    o[32 * ch + e] = fmaf(o[32 * ch + e], f, __uint_as_float(v[e]));
            }
            return true;
        };
        for (int i = S::PAIR ? 0 : wg; i < n; i += S::PAIR ? 1 : 2) {
            if (pending && !take()) return;
            const uint32_t vi = 2 * (base + i) + 1, vs = vi % S::kSlots;
            if (!c.warp_wait(&sh->full[vs], vi / S::kSlots & 1)) return;
            if (!c.warp_wait(&sh->s_full[wg], mine & 1)) return;
            tc_fence_after();
            const int j0 = (st.k0 + i) * KT;
            uint32_t none[kChunks], lost = 0;
#pragma unroll
            for (int ch = 0; ch < kChunks; ++ch) lost |= none[ch] = sh->none[vs][ch];
            const bool mixed = j0 < st.tile.lo || j0 + KT > st.tile.hi || lost;
            float top = -INFINITY;
#pragma unroll
            for (int ch = 0; ch < kChunks; ++ch) {
                uint32_t v[32];
                ld32(v, tm + kColS + 32 * ch);
                wait_ld(v);
                if (formed) {
                    const int from = j0 + 32 * ch - see.pos;
                    const bool own = a.pos && j0 + 32 * ch + 32 > q.base;
#pragma unroll
                    for (int e = 0; e < 32; ++e) {
                        float y = __uint_as_float(v[e]) * a.scale;
                        if (a.softcap > 0.f)
                            y = a.softcap * (kFast ? fast_tanh(__fdividef(y, a.softcap))
                                                   : tanhf(y / a.softcap));
                        y *= kLog2e;
                        if (a.slopes) {
                            const int far =
                                own ? slot_pos(a, q, j0 + 32 * ch + e) - see.pos : from + e;
                            y = fmaf(slope, (float)far, y);
                        }
                        v[e] = __float_as_uint(y);
                    }
                }
                if (mixed) {
                    const uint32_t in = seen32(a, see, j0 + 32 * ch) & ~none[ch];
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        if (!(in >> e & 1u)) v[e] = 0xFF800000u;
                }
                if (formed || mixed) st32(tm + kColS + 32 * ch, v);
                float t0 = -INFINITY, t1 = -INFINITY;
#pragma unroll
                for (int e = 0; e < 32; e += 2) {
                    t0 = fmaxf(t0, __uint_as_float(v[e]));
                    t1 = fmaxf(t1, __uint_as_float(v[e + 1]));
                }
                top = fmaxf(top, fmaxf(t0, t1));
            }
            if (formed || mixed) wait_st();
            const float now = fmaxf(m, top * to_log2);
            const float safe = now == -INFINITY ? 0.f : now;
            const float fl = ex2(m - safe);
            f = fl;
            m = now;
            if (mixed) {
                // Rows of 128 bytes of v: a thread looks through one, or through both of its slot's.
                const uint32_t v_at = c.ring + vs * S::kSlot;
                constexpr int kParts = DP / 64;                  // rows of 128 bytes to a slot
                constexpr int kScan = S::PAIR ? 256 : 128;       // threads
                constexpr int kEach = KT * kParts > kScan ? KT * kParts / kScan : 1;
                const int at = S::PAIR ? threadIdx.x : r;
                const int slot = at % KT, part0 = at / KT, scan_warp = at >> 5;
                bool mine_odd = false;
                if (part0 < kParts) {
#pragma unroll
                    for (int p = 0; p < kEach; ++p) {
                        const int part = part0 + p;
                        const uint32_t line = v_at + part * (KT * 128) + slot * 128;
#pragma unroll
                        for (int ch = 0; ch < 8; ++ch) {
                            const uint4 w = lds16(line + (((ch + slot) & 7) << 4));
                            mine_odd |= odd16x2<S::ET>(w.x) || odd16x2<S::ET>(w.y) ||
                                        odd16x2<S::ET>(w.z) || odd16x2<S::ET>(w.w);
                        }
                    }
                }
                const uint32_t found = __ballot_sync(0xFFFFFFFFu, mine_odd);
                // Words of this tile's slots, by the warp that looked: two sets taken in turn.
                uint32_t *const words = S::PAIR ? &sh->odd[odd_turn & 1][0][0]
                                                : &sh->odd[wg][0][0];
                if ((threadIdx.x & 31) == 0)
                    words[scan_warp * 32 / KT * 4 + scan_warp * 32 % KT / 32] = found;
                if (!meet(1)) return;
                uint32_t any = 0, w[kChunks];
#pragma unroll
                for (int ch = 0; ch < kChunks; ++ch) {
                    w[ch] = words[ch];
                    if (kScan / KT > 1 && kParts > 1) w[ch] |= words[4 + ch];
                    any |= w[ch];
                }
                ++odd_turn;
                if (any) {
#pragma unroll
                    for (int e = 0; e < DP; ++e) o[e] *= f;
                    f = 1.f;
#pragma unroll
                    for (int ch = 0; ch < kChunks; ++ch) {
                        const uint32_t in = seen32(a, see, j0 + 32 * ch) & ~none[ch];
                        for (uint32_t left = w[ch]; left; left &= left - 1) {
                            const int b = __ffs(left) - 1, s = 32 * ch + b;
                            __syncwarp();
                            const float x = ld1(tm + kColS + s);
                            if (!(in >> b & 1u)) continue;
                            const float p = ex2(fmaf(x, to_log2, -safe));
#pragma unroll
                            for (int e = 0; e < DP; e += 8) {
                                const int chunk = e / 8;
                                const uint4 u = lds16(v_at + (chunk >> 3) * (KT * 128) + s * 128 +
                                                      (((chunk & 7) ^ (s & 7)) << 4));
                                const uint32_t z[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                                for (int k = 0; k < 8; ++k)
                                    o[e + k] = fmaf(p, widen<S::ET>(z[k >> 1], k & 1), o[e + k]);
                            }
                        }
                    }
                    if (!meet(1)) return;
                    if (mine_odd || (w[slot >> 5] >> (slot & 31) & 1u)) {
#pragma unroll
                        for (int p = 0; p < kEach; ++p)
                            if (part0 + p < kParts)
#pragma unroll
                                for (int ch = 0; ch < 8; ++ch)
                                    sts16(v_at + (part0 + p) * (KT * 128) + slot * 128 + ch * 16,
                                          make_uint4(0u, 0u, 0u, 0u));
                    }
                    fence_proxy_async_smem();
                }
            }
            float sums[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int ch = 0; ch < kChunks; ++ch) {
                uint32_t v[32];
                ld32(v, tm + kColS + 32 * ch);
                wait_ld(v);
                float p[32];
#pragma unroll
                for (int e = 0; e < 32; ++e) {
                    p[e] = ex2(fmaf(__uint_as_float(v[e]), to_log2, -safe));
                    sums[e & 3] += p[e];
                }
#pragma unroll
                for (int t = 0; t < S::TERMS; ++t) {
                    uint32_t w[16];
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        w[e] = pack2<S::ET>(p[2 * e], p[2 * e + 1]);
                        if (t + 1 < S::TERMS) {
                            p[2 * e] -= bf16_lo(w[e]);
                            p[2 * e + 1] -= bf16_hi(w[e]);
                        }
                    }
                    st16(tm + (t == 0 ? kColP0 : t == 1 ? kColP1 : kColP2) + 16 * ch, w);
                }
            }
            l = fmaf(l, fl, (sums[0] + sums[1]) + (sums[2] + sums[3]));
            wait_st();
            tc_fence_before();
            mbar_arrive(&sh->p_ready[wg]);
            ++mine;
            pending = true;
        }
        if (pending && !take()) return;
        base += n;

        if (!S::PAIR && n > 0) {
            // The two warpgroups' halves of the slots.
            if (!meet(0)) return;  // every product of q is done
            if (wg == 1) {
#pragma unroll
                for (int e = 0; e < DP; ++e)
                    asm volatile("st.shared.f32 [%0], %1;" ::"r"(c.stage + (e * 128 + r) * 4),
                                 "f"(o[e])
                                 : "memory");
                sh->ml[r] = make_float2(m, l);
            }
            if (!meet(0)) return;
            if (wg == 0) {
                const float2 other = sh->ml[r];
                const float both = fmaxf(m, other.x), safe = both == -INFINITY ? 0.f : both;
                const float fa = ex2(m - safe), fb = ex2(other.x - safe);
                m = both;
                l = fmaf(l, fa, other.y * fb);
#pragma unroll
                for (int e = 0; e < DP; ++e) {
                    float x;
                    asm volatile("ld.shared.f32 %0, [%1];"
                                 : "=f"(x)
                                 : "r"(c.stage + (e * 128 + r) * 4)
                                 : "memory");
                    o[e] = fmaf(o[e], fa, x * fb);
                }
            }
        }
        if (!live || (!S::PAIR && wg == 1)) continue;
        if (st.part >= 0) {
            const size_t part = 2 * blockIdx.x + st.part;
#pragma unroll
            for (int e = 0; e < DP; e += 4)
                room.part_o[(part * (DP / 4) + e / 4) * S::RT + row] =
                    make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
            room.part_ml[part * S::RT + row] = make_float2(m, l);
            continue;
        }
        const int t = q.t0 + j, h = st.head * group + g;
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const long long to = t * a.out_stride + (long long)h * kv.head_dim;
#pragma unroll
        for (int e = 0; e < DP; e += 8) {
            if (e >= kv.head_dim) break;
            if (a.out_type == kF32) {
                out.put4(to + e, make_float4(o[e] * inv, o[e + 1] * inv, o[e + 2] * inv,
                                             o[e + 3] * inv));
                out.put4(to + e + 4, make_float4(o[e + 4] * inv, o[e + 5] * inv, o[e + 6] * inv,
                                                 o[e + 7] * inv));
            } else {
                uint4 w;
                w.x = pack2<S::ET>(o[e] * inv, o[e + 1] * inv);
                w.y = pack2<S::ET>(o[e + 2] * inv, o[e + 3] * inv);
                w.z = pack2<S::ET>(o[e + 4] * inv, o[e + 5] * inv);
                w.w = pack2<S::ET>(o[e + 6] * inv, o[e + 7] * inv);
                *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out) + to + e) = w;
            }
        }
        if (a.lse) a.lse[(long long)t * a.h_q + h] = lse_of(m, l);
    }
}

template <typename S>
__global__ void __launch_bounds__(kThreads, 1)
    attn_tokens_tc_kernel(TokensArgs a, KvView kv) {
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
        for (int i = 0; i < kMostSlots; ++i) {
            mbar_init(&c.sh->full[i], kLoaders);
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
    // 384 threads of 168 registers at the launch; 224 for each row's output and 56 for the others
    // add up to the same.
    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
        softmax_rows<S>(a, kv, room, c);
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        if (warp > 8) {
            load_tiles<S>(a, kv, room, c);
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

template <int DP, int TERMS, bool PAIR, int ET>
cudaError_t launch_shape(const TokensArgs &a, const KvView &kv, const DeviceInfo &dev,
                         cudaStream_t stream) {
    using S = TcShape<DP, TERMS, PAIR, ET>;
    static std::atomic<unsigned long long> raised{0};
    cudaError_t err = ensure_smem(attn_tokens_tc_kernel<S>, S::kSmem, dev, raised);
    if (err != cudaSuccess) return err;
    err = launch_attn_plan(a, kv, S::RT, S::KT, DP, kGrid, stream);
    if (err != cudaSuccess) return err;
    err = launch_pdl(attn_tokens_tc_kernel<S>, dim3(kGrid), dim3(kThreads), S::kSmem, stream, a, kv);
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

// attn_tokens.cu -- attention of several new tokens per sequence over a paged cache: the plan, the
// join of parts, and the kernel in f32 arithmetic that takes every type and head size.
//
// x = cap(scale q.k) + slope (pos_k - pos_q), p = softmax(x) with a running maximum and sum,
// in log2 units: y = x log2 e, p = 2^(y - m).
//
// attn_rows_kernel takes f32 caches, f32 queries over f16 caches, mixed 16-bit types, and of heads above
// 128 dims all but 16-bit ones in pages of a multiple of 8 slots: k and v are f32 in shared memory and
// every product is an f32 FMA, so it is exact to f32.
// What bounds it: the FMA pipe (4 head_dim operations per row and slot) and the shared memory that
// feeds it (48 wavefronts to 64 FMA cycles), and for short rows how evenly 304 ranges share few
// tiles.  A thread holds R rows by KT / 16 slots of the scores and R rows by DP / 16 dims of the
// output, two neighbouring dims to an instruction; the 16 lanes of a row join its maximum and sum
// by shuffles.  Three packed batches of documents, 12/6 heads of 96, f32: 67 us, a quarter of the FMA
// rate while a CTA works; 12 trees of f32 queries and an f32 cache to 6000 slots: 424 us.
#include "attn_tokens.cuh"

namespace wq {
namespace tok {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanTiles = 2048;
// A CTA's range is no shorter, or the parts cost more than they save: 2, 3 and 6 took 19.6, 20.8 and
// 28 us for 16 nodes behind 900 slots.
constexpr int kLeastCost = 2;

__device__ __forceinline__ long long warp_scan(long long x, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xFFFFFFFFu, x, o);
        if (lane >= o) x += y;
    }
    return x;
}
// Inclusive scan over the block; `total` of all.
__device__ __forceinline__ long long block_scan(long long x, long long *s_warp, long long &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    x = warp_scan(x, lane);
    if (lane == 31) s_warp[warp] = x;
    __syncthreads();
    if (warp == 0) s_warp[lane] = warp_scan(s_warp[lane], lane);
    __syncthreads();
    if (warp > 0) x += s_warp[warp - 1];
    total = s_warp[31];
    __syncthreads();
    return x;
}

__global__ void __launch_bounds__(kPlanThreads)
    attn_plan_kernel(TokensArgs a, int heads, int rt, int kt, int dp, int grid, int row_cost) {
    __shared__ long long s_warp[32];
    __shared__ int s_first[kPlanThreads + 1];
    __shared__ int s_keys[kPlanTiles];          // key tiles of the first row tiles,
    __shared__ long long s_before[kPlanTiles];  // and the costs before them
    pdl_enter();
    const int group = a.group.d, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const Room room = room_of(a.workspace, a.n_seq, a.n_tok, group, rt, dp, grid);
    if (threadIdx.x < 2 * grid) room.joined[threadIdx.x] = 0u;
    // Row tiles of the sequences, kPlanThreads sequences at a time.  Ranges of `starts` that overlap
    // may ask for more than there is room for: the rest is left out.
    const long long most = most_tiles(a.n_seq, a.n_tok, group, rt);
    int n_tiles = 0;
    for (int s0 = 0; s0 < a.n_seq; s0 += kPlanThreads) {
        int mine = 0;
        if (s0 + (int)threadIdx.x < a.n_seq) {
            bool bad = false;
            const Seq q = seq_of(a, s0 + threadIdx.x, bad);
            if (bad) record_status(a.status, kStBadIndex);
            mine = (int)(((long long)q.count * group + rt - 1) / rt);
        }
        long long all;
        const long long upto = block_scan(mine, s_warp, all);
        if (mine > 0 && n_tiles + upto > most) record_status(a.status, kStBadIndex);
        s_first[threadIdx.x + 1] = (int)min(n_tiles + upto, most);
        if (threadIdx.x == 0) s_first[0] = n_tiles;
        __syncthreads();
        // A warp lists a sequence's tiles, all warps those of few sequences.
        const int here = min(a.n_seq - s0, kPlanThreads);
        int share = 1;  // warps to a sequence
        while (2 * share * here <= kPlanThreads / 32) share *= 2;
        for (int i = warp / share; i < here; i += kPlanThreads / 32 / share) {
            const int first = s_first[i], count = s_first[i + 1] - first;
            if (count == 0) continue;
            bool bad = false;
            const int s = s0 + i;
            const Seq q = seq_of(a, s, bad);
            const bool each = a.first || (a.tree && a.window > 0);
            for (int r = warp % share * 32 + lane; r < count; r += 32 * share) {
                const int row0 = r * rt, row1 = min(row0 + rt, q.count * group);
                const int j0 = a.group.div(row0), j1 = a.group.div(row1 - 1);
                int lo = INT_MAX, hi = 0, lo_most = 0, hi_least = INT_MAX;
                // Without per-token arrays the bounds rise from token to token.
                for (int j = j0; j <= j1; j = each || j == j1 ? j + 1 : j1) {
                    const See v = see_of(a, q, s, j);
                    int l = v.lo, h = v.hi;
                    if (v.own_end > v.own) {  // its own slots may lie below its window
                        h = v.own_end;
                        l = min(l, max(v.own, 0));
                    }
                    lo = min(lo, l);
                    hi = max(hi, h);
                    lo_most = max(lo_most, v.lo);
                    hi_least = min(hi_least, v.hi);
                }
                Tile t{s, row0, 0, 0, lo_most, hi_least, q};
                if (hi > lo) t.k0 = lo / kt, t.k1 = (hi + kt - 1) / kt;
                room.tiles[first + r] = t;
                if (first + r < kPlanTiles) s_keys[first + r] = t.k1 - t.k0;
            }
        }
        n_tiles = (int)min(n_tiles + all, most);
        __syncthreads();
    }
    auto keys = [&](int i) {
        return i < kPlanTiles ? s_keys[i] : room.tiles[i].k1 - room.tiles[i].k0;
    };
    // Costs before each row tile.
    long long cost = 0;
    for (int i0 = 0; i0 < n_tiles; i0 += kPlanThreads) {
        const int i = i0 + threadIdx.x;
        long long mine = 0;
        if (i < n_tiles) mine = keys(i) + row_cost;
        long long all;
        const long long upto = block_scan(mine, s_warp, all);
        if (i < n_tiles) (i < kPlanTiles ? s_before[i] : room.before[i]) = cost + upto - mine;
        cost += all;
    }
    __syncthreads();
    auto before = [&](int i) { return i < kPlanTiles ? s_before[i] : room.before[i]; };
    for (int b = threadIdx.x; b <= grid; b += kPlanThreads) {
        Begin p{heads, 0, 0, n_tiles, 0, 0};
        if (cost > 0) {
            // CTA b begins at each b + min(b, rest).
            const long long total = cost * heads;
            const int ctas = (int)max(1ll, min((long long)grid, total / kLeastCost));
            const long long each = total / ctas, rest = total % ctas;
            auto owner = [&](long long t) {
                const long long cut = rest * (each + 1);
                return (int)(t < cut ? t / (each + 1) : rest + (t - cut) / each);
            };
            const long long at = min(total, each * b + min((long long)b, rest));
            const int head = (int)(at / cost);
            const long long in = at - head * cost;
            int x = 0, y = n_tiles;  // before(x) <= in < before(y)
            while (y - x > 1) {
                const int mid = (x + y) / 2;
                if (before(mid) <= in) x = mid; else y = mid;
            }
            p.head = head;
            p.tile = x;
            p.off = (int)(in - before(x));
            const int n = keys(x);
            if (p.off > 0 && p.off < n) {
                const long long begin = head * cost + before(x);
                p.lead = owner(begin);
                p.parts = owner(begin + n - 1) - p.lead + 1;
            } else if (p.off > 0) {  // in the end of a row tile
                p.off = 0;
                if (++p.tile == n_tiles) p.tile = 0, ++p.head;
            }
        }
        room.plan[b] = p;
    }
}

// Joins the parts of the row tile that CTA blockIdx.x leads and others go on with.  A thread takes
// four dims of a row at a time, with the loads of kAtOnce parts in flight.  (5 us of a call.)
constexpr int kAtOnce = 8;
__global__ void __launch_bounds__(256)
    attn_parts_kernel(TokensArgs a, KvView kv, int passes, int rt, int dp, int grid) {
    // What follows is let in when this is over: a next call's blocks, let in early, would take the
    // places of this one's (41 us instead of 24 for 4 sequences of 16 nodes, one call after another).
    pdl_wait();
    const int group = a.group.d;
    const Room room = room_of(a.workspace, a.n_seq, a.n_tok, group, rt, dp, grid);
    const Begin p = room.plan[blockIdx.x + 1];
    if (p.off == 0 || p.lead != (int)blockIdx.x) return;
    const Tile tile = room.tiles[p.tile];
    const Seq q = tile.q;
    const int rows = min(rt, q.count * group - tile.row0);
    const TypedOut out{a.out, a.out_type};
    const int head = p.head / passes, dim0 = p.head % passes * dp;
    const int dims = min(dp, kv.head_dim - dim0);
    for (int at = blockIdx.y * 256 + threadIdx.x; at < rt * (dims / 4); at += gridDim.y * 256) {
        const int row = at % rt, c = at / rt;  // rt is a power of two
        if (row >= rows) continue;
        float m = -INFINITY, l = 0.f;
        float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int i0 = 0; i0 < p.parts; i0 += kAtOnce) {
            float2 ml[kAtOnce];
            float4 v[kAtOnce];
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) {
                const size_t part = part_place(p.lead, min(i0 + i, p.parts - 1));
                ml[i] = room.part_ml[part * rt + row];
                v[i] = room.part_o[(part * (dp / 4) + c) * rt + row];
            }
#pragma unroll
            for (int i = 0; i < kAtOnce; ++i) {
                if (i0 + i >= p.parts) break;
                const float now = fmaxf(m, ml[i].x), safe = now == -INFINITY ? 0.f : now;
                const float f = exp2f(m - safe), g = exp2f(ml[i].x - safe);
                m = now;
                l = fmaf(l, f, ml[i].y * g);
                o.x = fmaf(o.x, f, v[i].x * g), o.y = fmaf(o.y, f, v[i].y * g);
                o.z = fmaf(o.z, f, v[i].z * g), o.w = fmaf(o.w, f, v[i].w * g);
            }
        }
        const float inv = l == 0.f ? 0.f : 1.f / l;
        const int rr = tile.row0 + row, j = a.group.div(rr), g = rr - j * group;
        const int t = q.t0 + j, h = head * group + g;
        out.put4(t * a.out_stride + (long long)h * kv.head_dim + dim0 + 4 * c,
                 make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv));
        if (a.lse && dim0 + c == 0) a.lse[(long long)t * a.h_q + h] = lse_of(m, l);
    }
}

// ------------------------------------------------------------------ f32 arithmetic --

template <typename T> __device__ __forceinline__ float to_f32(T x) {
    if constexpr (sizeof(T) == 4) return x;
    else if constexpr (std::is_same<T, __half>::value) return __half2float(x);
    else return __bfloat162float(x);
}
// Eight values of a row as f32.
template <typename T> __device__ __forceinline__ void load8(const void *p, float (&v)[8]) {
    if constexpr (sizeof(T) == 4) {
        const float4 x = reinterpret_cast<const float4 *>(p)[0],
                     y = reinterpret_cast<const float4 *>(p)[1];
        v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
        v[4] = y.x, v[5] = y.y, v[6] = y.z, v[7] = y.w;
    } else {
        const uint4 x = *reinterpret_cast<const uint4 *>(p);
        const T *t = reinterpret_cast<const T *>(&x);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = to_f32(t[i]);
    }
}

// Two f32 operations of one instruction, pairs of neighbouring dims.
using Pair = unsigned long long;
__device__ __forceinline__ void fma2(Pair &d, Pair a, Pair b) {
    asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(d) : "l"(a), "l"(b));
}
__device__ __forceinline__ Pair pair_of(float lo, float hi) {
    Pair r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ float2 floats_of(Pair x) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
    return r;
}

template <int DP, int R> struct RowsShape {
    static constexpr int KT = DP > 128 ? 32 : 64;
    static constexpr int RT = 16 * R;
    static constexpr int kPitch = DP + 4;       // floats of a row of q or k: rows four banks apart
    static constexpr int kQ = RT * kPitch, kK = KT * kPitch, kV = KT * DP, kP = RT * (KT + 4);
    static constexpr int kSmem = (kQ + kK + kV + kP) * 4 + RT * (int)sizeof(See);
    static constexpr int kCtas = 2 * (kSmem + 1200) <= 228 * 1024 ? 2 : 1;  // on an SM
    static constexpr int kGrid = 152 * kCtas;
};

template <typename T, int DP, int R>
__global__ void __launch_bounds__(256, RowsShape<DP, R>::kCtas)
    attn_rows_kernel(TokensArgs a, KvView kv) {
    using S = RowsShape<DP, R>;
    constexpr int KT = S::KT, RT = S::RT, NK = KT / 16, ND = DP / 32;
    constexpr bool kAsync = sizeof(T) == 4;
    constexpr int grid = S::kGrid;
    extern __shared__ __align__(16) float s_rows[];
    __shared__ int s_join[3];
    float *s_q = s_rows, *s_k = s_q + S::kQ, *s_v = s_k + S::kK, *s_p = s_v + S::kV;
    See *const s_see = reinterpret_cast<See *>(s_p + S::kP);
    pdl_enter();
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4, group = a.group.d;
    const Room room = room_of(a.workspace, a.n_seq, a.n_tok, group, RT, DP, grid);
    Walk walk(room, blockIdx.x);
    const TypedOut out{a.out, a.out_type};
    const int d = kv.head_dim;
    Stretch st;
    while (walk.next(st)) {
        const Tile tile = room.tiles[st.tile];
        const Seq q = tile.q;
        const int rows = min(RT, q.count * group - tile.row0);
        __syncthreads();
        for (int i = threadIdx.x; i < RT * (DP / 8); i += 256) {
            const int r = i / (DP / 8), c = i - r * (DP / 8);
            float v[8] = {};
            if (r < rows && c * 8 < d) {
                const int rr = tile.row0 + r, j = a.group.div(rr), g = rr - j * group;
                const long long at = (q.t0 + j) * a.q_stride +
                                     (long long)(st.head * group + g) * d + c * 8;
                if (a.q_type == kF32)
                    load8<float>(static_cast<const float *>(a.q) + at, v);
                else if (a.q_type == kBF16)
                    load8<__nv_bfloat16>(static_cast<const __nv_bfloat16 *>(a.q) + at, v);
                else
                    load8<__half>(static_cast<const __half *>(a.q) + at, v);
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) s_q[r * S::kPitch + c * 8 + e] = v[e];
        }
        if (threadIdx.x < RT) {
            const int rr = tile.row0 + min((int)threadIdx.x, rows - 1);
            s_see[threadIdx.x] = see_of(a, q, tile.seq, a.group.div(rr));
        }
        float slope[R];
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int rr = tile.row0 + min(ty * R + i, rows - 1);
            slope[i] = a.slopes ? a.slopes[st.head * group + rr - a.group.div(rr) * group] : 0.f;
        }
        float m[R], l[R];
        Pair o[R][ND];  // dims 32 e + 2 tx of the thread's rows
#pragma unroll
        for (int i = 0; i < R; ++i) {
            m[i] = -INFINITY, l[i] = 0.f;
#pragma unroll
            for (int e = 0; e < ND; ++e) o[i][e] = 0ull;
        }
        // k and v of a tile, zero beyond the live slots and where a page is out of range.  f32 caches:
        // k of the next tile is under way during the weights and products of this one, v during the
        // next one's scores.  16-bit caches are widened on their way, both together.
        uint32_t lost = 0;  // of the tile that is asked for: (bit 0) a slot without a page, (bit 1) a v
                            // that is not finite
        auto ask = [&](int kt, bool is_v) {
            if (kt >= st.k1 || (!kAsync && !is_v)) return;
            if (is_v) lost = 0;
            for (int i = threadIdx.x; i < KT * (DP / 8); i += 256) {
                const int r = i / (DP / 8), c = i - r * (DP / 8), j = kt * KT + r;
                long long at = -1;
                if (j < q.len) {
                    at = kv.row(tile.seq, st.head, j);
                    if (at < 0) lost |= 1u;
                }
                const bool live = at >= 0 && c * 8 < d;
                if constexpr (kAsync) {
                    const char *const from = (is_v ? kv.v : kv.k) + (live ? at + c * 32 : 0);
                    const uint32_t to = smem_addr((is_v ? s_v + r * DP : s_k + r * S::kPitch) + c * 8);
                    cp16(to, from, live);
                    cp16(to + 16, from + (live ? 16 : 0), live);
                } else {
                    float x[8] = {}, y[8] = {};
                    if (live) {
                        load8<T>(kv.k + at + c * 8 * sizeof(T), x);
                        load8<T>(kv.v + at + c * 8 * sizeof(T), y);
                    }
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        s_k[r * S::kPitch + c * 8 + e] = x[e];
                        s_v[r * DP + c * 8 + e] = y[e];
                        if (!isfinite(y[e])) lost |= 2u;
                    }
                }
            }
            if (kAsync) cp_commit();
        };
        ask(st.k0, false);
        ask(st.k0, true);
        for (int kt = st.k0; kt < st.k1; ++kt) {
            const int j0 = kt * KT;
            if (kAsync) cp_wait<1>();
            __syncthreads();
            Pair x2[R][NK];
#pragma unroll
            for (int i = 0; i < R; ++i)
#pragma unroll
                for (int n = 0; n < NK; ++n) x2[i][n] = 0ull;
#pragma unroll 4
            for (int c = 0; c < DP; c += 4) {
                ulonglong2 qa[R], ka[NK];
#pragma unroll
                for (int i = 0; i < R; ++i)
                    qa[i] = *reinterpret_cast<const ulonglong2 *>(s_q + (ty * R + i) * S::kPitch + c);
#pragma unroll
                for (int n = 0; n < NK; ++n)
                    ka[n] =
                        *reinterpret_cast<const ulonglong2 *>(s_k + (tx + 16 * n) * S::kPitch + c);
#pragma unroll
                for (int i = 0; i < R; ++i)
#pragma unroll
                    for (int n = 0; n < NK; ++n) {
                        fma2(x2[i][n], qa[i].x, ka[n].x);
                        fma2(x2[i][n], qa[i].y, ka[n].y);
                    }
            }
            float x[R][NK];
#pragma unroll
            for (int i = 0; i < R; ++i)
#pragma unroll
                for (int n = 0; n < NK; ++n) {
                    const float2 s = floats_of(x2[i][n]);
                    x[i][n] = s.x + s.y;
                }
            if constexpr (kAsync) {  // this thread's share of v
                cp_wait<0>();
                for (int i = threadIdx.x; i < KT * (DP / 8); i += 256) {
                    const float4 *const y = reinterpret_cast<const float4 *>(s_v + i * 8);
                    const float4 y0 = y[0], y1 = y[1];
                    if (!(isfinite(y0.x) && isfinite(y0.y) && isfinite(y0.z) && isfinite(y0.w) &&
                          isfinite(y1.x) && isfinite(y1.y) && isfinite(y1.z) && isfinite(y1.w)))
                        lost |= 2u;
                }
            }
            const int none = __syncthreads_or(lost & 1u), odd = __syncthreads_or(lost & 2u);
            if (none && threadIdx.x == 0) record_status(a.status, kStBadIndex);
            ask(kt + 1, false);
            const bool whole = j0 >= tile.lo && j0 + KT <= tile.hi && !none;
#pragma unroll
            for (int i = 0; i < R; ++i) {
                uint32_t seen[KT / 32];
#pragma unroll
                for (int w = 0; w < KT / 32; ++w)
                    seen[w] = whole ? 0xFFFFFFFFu : seen32(a, s_see[ty * R + i], j0 + 32 * w);
                const int pos = s_see[ty * R + i].pos;
                float top = -INFINITY;
#pragma unroll
                for (int n = 0; n < NK; ++n) {
                    const int r = tx + 16 * n, j = j0 + r;
                    float y = x[i][n] * a.scale;
                    if (a.softcap > 0.f) y = a.softcap * tanhf(y / a.softcap);
                    if (a.slopes) y = fmaf(slope[i], (float)(slot_pos(a, q, j) - pos), y);
                    bool in = seen[r >> 5] >> (r & 31) & 1u;
                    if (none && in) in = kv.row(tile.seq, st.head, j) >= 0;
                    // A score that is not a number stays one: only slots that are not seen are -inf.
                    x[i][n] = in ? y * kLog2e : -INFINITY;
                    if (!in) seen[r >> 5] &= ~(1u << (r & 31));
                    top = fmaxf(top, x[i][n]);
                }
#pragma unroll
                for (int s = 8; s > 0; s >>= 1)
                    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, s));
                const float now = fmaxf(m[i], top), safe = now == -INFINITY ? 0.f : now;
                const float f = exp2f(m[i] - safe);
                float sum = 0.f;
#pragma unroll
                for (int n = 0; n < NK; ++n) {
                    const int r = tx + 16 * n;
                    const float p = exp2f(x[i][n] - safe);
                    sum += p;
                    // -1 marks a slot that is not seen where 0 times v would not be 0.
                    const bool in = seen[r >> 5] >> (r & 31) & 1u;
                    s_p[(ty * R + i) * (KT + 4) + r] = odd && !in ? -1.f : p;
                }
#pragma unroll
                for (int s = 8; s > 0; s >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, s);
                l[i] = fmaf(l[i], f, sum);
                m[i] = now;
                const Pair f2 = pair_of(f, f);
#pragma unroll
                for (int e = 0; e < ND; ++e)
                    asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(o[i][e]) : "l"(f2));
            }
            __syncwarp();  // a row's 16 lanes are in one warp
            if (!odd) {
#pragma unroll 2
                for (int r = 0; r < KT; r += 4) {
                    float4 pa[R];
#pragma unroll
                    for (int i = 0; i < R; ++i)
                        pa[i] = *reinterpret_cast<const float4 *>(s_p + (ty * R + i) * (KT + 4) + r);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        Pair p[R];
#pragma unroll
                        for (int i = 0; i < R; ++i) {
                            const float w = k == 0   ? pa[i].x
                                            : k == 1 ? pa[i].y
                                            : k == 2 ? pa[i].z
                                                     : pa[i].w;
                            p[i] = pair_of(w, w);
                        }
#pragma unroll
                        for (int e = 0; e < ND; ++e) {
                            const Pair v =
                                *reinterpret_cast<const Pair *>(s_v + (r + k) * DP + 32 * e + 2 * tx);
#pragma unroll
                            for (int i = 0; i < R; ++i) fma2(o[i][e], p[i], v);
                        }
                    }
                }
            } else {
                for (int r = 0; r < KT; ++r)
#pragma unroll
                    for (int i = 0; i < R; ++i) {
                        const float p = s_p[(ty * R + i) * (KT + 4) + r];
                        if (p == -1.f) continue;
#pragma unroll
                        for (int e = 0; e < ND; ++e)
                            fma2(o[i][e], pair_of(p, p),
                                 *reinterpret_cast<const Pair *>(s_v + r * DP + 32 * e + 2 * tx));
                    }
            }
            __syncthreads();
            ask(kt + 1, true);
        }
        // Parts lie as [dims / 4][row][4].
        auto part_at = [&](size_t part, int r, int e) {
            const int c = 32 * e + 2 * tx;
            return reinterpret_cast<float *>(room.part_o) +
                   ((part * (DP / 4) + c / 4) * RT + r) * 4 + (c & 3);
        };
        if (st.part >= 0) {
            const size_t part = 2 * blockIdx.x + st.part;
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const int r = ty * R + i;
#pragma unroll
                for (int e = 0; e < ND; ++e)
                    *reinterpret_cast<float2 *>(part_at(part, r, e)) = floats_of(o[i][e]);
                if (tx == 0) room.part_ml[part * RT + r] = make_float2(m[i], l[i]);
            }
            if (!a.join_inside) continue;
            __threadfence();
            __syncthreads();
            if (threadIdx.x == 0) {
                int lead, parts;
                s_join[0] = part_last(room, st, blockIdx.x, 0, lead, parts);
                s_join[1] = lead, s_join[2] = parts;
            }
            __syncthreads();
            if (!s_join[0]) continue;
            __threadfence();
            const int lead = s_join[1], parts = s_join[2];
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const int r = ty * R + i;
                float2 sum[ND];
                m[i] = -INFINITY, l[i] = 0.f;
#pragma unroll
                for (int e = 0; e < ND; ++e) sum[e] = make_float2(0.f, 0.f);
                for (int k = 0; k < parts; ++k) {
                    const size_t from = part_place(lead, k);
                    const float2 ml = __ldcg(room.part_ml + from * RT + r);
                    const float now = fmaxf(m[i], ml.x), safe = now == -INFINITY ? 0.f : now;
                    const float f = exp2f(m[i] - safe), g = exp2f(ml.x - safe);
                    m[i] = now;
                    l[i] = fmaf(l[i], f, ml.y * g);
#pragma unroll
                    for (int e = 0; e < ND; ++e) {
                        const float2 v =
                            __ldcg(reinterpret_cast<const float2 *>(part_at(from, r, e)));
                        sum[e].x = fmaf(sum[e].x, f, v.x * g);
                        sum[e].y = fmaf(sum[e].y, f, v.y * g);
                    }
                }
#pragma unroll
                for (int e = 0; e < ND; ++e) o[i][e] = pair_of(sum[e].x, sum[e].y);
            }
        }
#pragma unroll
        for (int i = 0; i < R; ++i) {
            const int r = ty * R + i;
            if (r >= rows) continue;
            const int rr = tile.row0 + r, j = a.group.div(rr), g = rr - j * group;
            const int t = q.t0 + j, h = st.head * group + g;
            const float inv = l[i] == 0.f ? 0.f : 1.f / l[i];
#pragma unroll
            for (int e = 0; e < ND; ++e) {
                const int c = 32 * e + 2 * tx;
                const float2 v = floats_of(o[i][e]);
                if (c < d)
                    out.put2(t * a.out_stride + (long long)h * d + c,
                             make_float2(v.x * inv, v.y * inv));
            }
            if (a.lse && tx == 0) a.lse[(long long)t * a.h_q + h] = lse_of(m[i], l[i]);
        }
    }
}

// Rows of a thread: one where the sequences have few rows, else four.
int rows_per_thread(int n_seq, int n_tok, int group) {
    return (long long)n_tok * group <= 24ll * n_seq ? 1 : 4;
}
int padded_dim(int head_dim) {
    return head_dim <= 64 ? 64 : head_dim <= 96 ? 96 : head_dim <= 128 ? 128 : 256;
}

template <typename T, int DP, int R>
cudaError_t launch_rows(const TokensArgs &a, const KvView &kv, const DeviceInfo &dev,
                        cudaStream_t stream) {
    using S = RowsShape<DP, R>;
    static std::atomic<unsigned long long> raised{0};
    cudaError_t err = ensure_smem(attn_rows_kernel<T, DP, R>, S::kSmem, dev, raised);
    if (err != cudaSuccess) return err;
    const int grid = S::kGrid;
    TokensArgs b = a;
    b.join_inside = joins_inside(a, kv.n_heads, S::RT, grid);
    // A row tile's start and end as a key tile: as two, three and four packed documents took 76, 84
    // and 84 us instead of 69.
    err = launch_attn_plan(b, kv.n_heads, S::RT, S::KT, DP, grid, 1, stream);
    if (err != cudaSuccess) return err;
    err = launch_pdl(attn_rows_kernel<T, DP, R>, dim3(grid), dim3(256), S::kSmem, stream, b, kv);
    if (err != cudaSuccess || b.join_inside) return err;
    return launch_attn_parts(b, kv, 1, S::RT, DP, grid, stream);
}
template <typename T>
cudaError_t launch_rows_type(const TokensArgs &a, const KvView &kv, const DeviceInfo &dev,
                             cudaStream_t stream) {
    const bool one = rows_per_thread(a.n_seq, a.n_tok, a.group.d) == 1;
    switch (padded_dim(kv.head_dim)) {
    case 64: return one ? launch_rows<T, 64, 1>(a, kv, dev, stream)
                        : launch_rows<T, 64, 4>(a, kv, dev, stream);
    case 96: return one ? launch_rows<T, 96, 1>(a, kv, dev, stream)
                        : launch_rows<T, 96, 4>(a, kv, dev, stream);
    case 128: return one ? launch_rows<T, 128, 1>(a, kv, dev, stream)
                         : launch_rows<T, 128, 4>(a, kv, dev, stream);
    default: return one ? launch_rows<T, 256, 1>(a, kv, dev, stream)
                        : launch_rows<T, 256, 4>(a, kv, dev, stream);
    }
}

}  // namespace

cudaError_t launch_attn_plan(const TokensArgs &a, int heads, int rt, int kt, int dp, int grid,
                             int row_cost, cudaStream_t stream) {
    return launch_pdl(attn_plan_kernel, dim3(1), dim3(kPlanThreads), 0, stream, a, heads, rt, kt, dp,
                      grid, row_cost);
}

cudaError_t launch_attn_parts(const TokensArgs &a, const KvView &kv, int passes, int rt, int dp,
                              int grid, cudaStream_t stream) {
    const int blocks = (rt * (min(dp, kv.head_dim) / 4) + 255) / 256;
    return launch_pdl(attn_parts_kernel, dim3(grid - 1, blocks < 8 ? blocks : 8), dim3(256), 0,
                      stream, a, kv, passes, rt, dp, grid);
}

}  // namespace tok

size_t tokens_workspace_bytes(const KvView &kv, int n_seq, int n_tok, int h_q, int q_type) {
    const int group = h_q / kv.n_heads;
    int rt, dp, grid = tok::kMaxGrid;
    if (tok::tokens_tc_takes(kv, q_type)) {
        tok::tokens_tc_shape(n_seq, n_tok, group, q_type, kv.head_dim, rt, dp, grid);
    } else {
        rt = 16 * tok::rows_per_thread(n_seq, n_tok, group);
        dp = tok::padded_dim(kv.head_dim);
    }
    return tok::room_of(nullptr, n_seq, n_tok, group, rt, dp, grid).bytes;
}

cudaError_t launch_attn_tokens(const TokensArgs &a, const KvView &kv, const DeviceInfo &dev,
                               cudaStream_t stream) {
    if (tok::tokens_tc_takes(kv, a.q_type)) return tok::launch_tokens_tc(a, kv, dev, stream);
    switch (kv.dtype) {
    case kBF16: return tok::launch_rows_type<__nv_bfloat16>(a, kv, dev, stream);
    case kF16: return tok::launch_rows_type<__half>(a, kv, dev, stream);
    default: return tok::launch_rows_type<float>(a, kv, dev, stream);
    }
}

}  // namespace wq

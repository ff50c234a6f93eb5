// head_units.cuh -- a head's values in units of a thread: two runs of N (four where addresses
// allow 16-byte accesses, else one) that hold N pairs of a rotation or values that are copied.
#pragma once

#include <type_traits>

#include "kv_cache.cuh"
#include "wq.h"

namespace wq {

template <int N> struct Vals {
    float v[N];
};
template <int N> __device__ __forceinline__ Vals<N> load_vals(const float *p) {
    Vals<N> r;
    if constexpr (N == 4) {
        const float4 x = *reinterpret_cast<const float4 *>(p);
        r.v[0] = x.x, r.v[1] = x.y, r.v[2] = x.z, r.v[3] = x.w;
    } else {
        r.v[0] = *p;
    }
    return r;
}
__device__ __forceinline__ void store_vals(float *p, const Vals<4> &x) {
    *reinterpret_cast<float4 *>(p) = make_float4(x.v[0], x.v[1], x.v[2], x.v[3]);
}
__device__ __forceinline__ void store_vals(float *p, const Vals<1> &x) { *p = x.v[0]; }
__device__ __forceinline__ void store_vals(__nv_bfloat16 *p, const Vals<4> &x) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(x.v[0], x.v[1]),
                         b = __floats2bfloat162_rn(x.v[2], x.v[3]);
    *reinterpret_cast<uint2 *>(p) = make_uint2(*reinterpret_cast<const uint32_t *>(&a),
                                               *reinterpret_cast<const uint32_t *>(&b));
}
__device__ __forceinline__ void store_vals(__half *p, const Vals<4> &x) {
    const __half2 a = __floats2half2_rn(x.v[0], x.v[1]), b = __floats2half2_rn(x.v[2], x.v[3]);
    *reinterpret_cast<uint2 *>(p) = make_uint2(*reinterpret_cast<const uint32_t *>(&a),
                                               *reinterpret_cast<const uint32_t *>(&b));
}
template <typename T> __device__ __forceinline__ void store_vals(T *p, const Vals<1> &x) {
    if constexpr (sizeof(T) == 4)
        *p = x.v[0];
    else if constexpr (std::is_same<T, __half>::value)
        *p = KvType<kF16>::put(x.v[0]);
    else
        *p = KvType<kBF16>::put(x.v[0]);
}

// Where a unit's two runs of N values lie in a head, and how its pairs sit in them: in the
// half layout value i of one with value i of the other, interleaved (N = 4: the runs are
// one after the other) neighbours with one another.
struct Place {
    int a, b;
    bool turn;
};
template <int N> __device__ __forceinline__ Place place_of(int u, int rot, unsigned flags) {
    const int half = rot >> 1, units = half / N;
    if (u >= units) return {rot + 2 * N * (u - units), rot + 2 * N * (u - units) + N, false};
    if (flags & WQ_ROPE_INTERLEAVED) return {2 * N * u, 2 * N * u + N, true};
    return {N * u, N * u + half, true};
}

template <int N> struct Angles {
    float c[N], s[N];
};
template <int N>
__device__ __forceinline__ Angles<N> load_angles(const float2 *p, unsigned flags) {
    Angles<N> r;
    if constexpr (N == 4) {
        const float4 x = *reinterpret_cast<const float4 *>(p);
        const float4 y = reinterpret_cast<const float4 *>(p)[1];
        r.c[0] = x.x, r.s[0] = x.y, r.c[1] = x.z, r.s[1] = x.w;
        r.c[2] = y.x, r.s[2] = y.y, r.c[3] = y.z, r.s[3] = y.w;
    } else {
        const float2 x = *p;
        r.c[0] = x.x, r.s[0] = x.y;
    }
    if (flags & WQ_ROPE_TRANSPOSE)
#pragma unroll
        for (int i = 0; i < N; ++i) r.s[i] = -r.s[i];
    return r;
}

template <int N>
__device__ __forceinline__ void turn(Vals<N> &a, Vals<N> &b, const Angles<N> &cs, unsigned flags) {
    if (N > 1 && (flags & WQ_ROPE_INTERLEAVED)) {
        float x[2 * N];
#pragma unroll
        for (int i = 0; i < N; ++i) x[i] = a.v[i], x[N + i] = b.v[i];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float lo = x[2 * i], hi = x[2 * i + 1];
            x[2 * i] = lo * cs.c[i] - hi * cs.s[i];
            x[2 * i + 1] = lo * cs.s[i] + hi * cs.c[i];
        }
#pragma unroll
        for (int i = 0; i < N; ++i) a.v[i] = x[i], b.v[i] = x[N + i];
        return;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float lo = a.v[i], hi = b.v[i];
        a.v[i] = lo * cs.c[i] - hi * cs.s[i];
        b.v[i] = lo * cs.s[i] + hi * cs.c[i];
    }
}

}  // namespace wq

// moe_rows.cuh -- for the layer norm and the gradient kernels: arithmetic on pairs of binary32 values,
// and the sums of a row's values over the lanes of a warp and over a group of warps, in a fixed order.
#pragma once

#include "moe_internal.cuh"

namespace moe {

// Pairs of binary32 values.
typedef unsigned long long f2;
__device__ __forceinline__ f2 f2_make(float lo, float hi) {
    f2 r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void f2_split(f2 v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ f2 f2_fma(f2 a, f2 b, f2 c) {
    f2 r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ f2 f2_mul(f2 a, f2 b) {
    f2 r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ f2 f2_add(f2 a, f2 b) {
    f2 r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ float f2_sum(f2 v) {
    float lo, hi;
    f2_split(v, lo, hi);
    return lo + hi;
}
// Two bf16 values, the first in the lower half.
__device__ __forceinline__ f2 f2_bf16(uint32_t w) {
    return f2_make(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}

__device__ __forceinline__ void f2_unpack(const uint4& v, f2 f[4]) {
    f[0] = f2_bf16(v.x);
    f[1] = f2_bf16(v.y);
    f[2] = f2_bf16(v.z);
    f[3] = f2_bf16(v.w);
}
__device__ __forceinline__ uint4 f2_pack(const f2 f[4]) {
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) f2_split(f[i], v[2 * i], v[2 * i + 1]);
    return pack8(v);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// Sums of N values (a power of two) over 32 lanes, or (HALF) over lanes 0..15 and over 16..31:
// half of the values go to the other half of the lanes until one is left, so lane l ends with
// the sum of v[l / (lanes / N)].
template <int N, bool HALF>
__device__ __forceinline__ float lane_sums(float (&v)[N], int lane) {
    int off = HALF ? 8 : 16;
#pragma unroll
    for (int n = N / 2; n > 0; n /= 2, off /= 2) {
        const bool hi = lane & off;
#pragma unroll
        for (int i = 0; i < n; ++i) {
            const float give = hi ? v[i] : v[i + n], keep = hi ? v[i + n] : v[i];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, give, off);
        }
    }
#pragma unroll
    for (int o = (HALF ? 8 : 16) / N; o > 0; o /= 2) v[0] += __shfl_xor_sync(0xffffffffu, v[0], o);
    return v[0];
}

// The sums of N values over a group of gw <= 16 warps, the same in every thread; warp is the
// warp in its CTA and first the group's first one.  red: N floats a warp of the CTA, 16-byte
// aligned; sync: the group's barrier.  A caller alternates between two arrays.
//
// join(v, w, q), for gw > 1: makes the sums of the group's warp w, v, ready to be added to the
// others'; q: those of the group's first warp.
struct JoinNothing {
    template <int N>
    __device__ __forceinline__ void operator()(float (&)[N], int, const float*) const {}
};
template <int N, typename Sync, typename Join = JoinNothing>
__device__ __forceinline__ void group_sums(float (&v)[N], float* red, int gw, int first, int warp, int lane,
                                           const Sync& sync, const Join& join = Join()) {
    float mine = lane_sums<N, false>(v, lane);
    if (gw == 1) {
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] = __shfl_sync(0xffffffffu, mine, i * (32 / N));
        return;
    }
    if (lane % (32 / N) == 0) red[warp * N + lane / (32 / N)] = mine;
    sync();
    const int w = lane & 15;
    const float* q = red + (first + (w < gw ? w : 0)) * N;
    if (N == 4) {
        const float4 f = *reinterpret_cast<const float4*>(q);
        v[0] = f.x; v[1 % N] = f.y; v[2 % N] = f.z; v[3 % N] = f.w;
    } else if (N == 2) {
        const float2 f = *reinterpret_cast<const float2*>(q);
        v[0] = f.x; v[1 % N] = f.y;
    } else {
        v[0] = q[0];
    }
    join(v, w, red + first * N);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = w < gw ? v[i] : 0.f;
    mine = lane_sums<N, true>(v, lane);
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __shfl_sync(0xffffffffu, mine, i * (16 / N));
}

}  // namespace moe

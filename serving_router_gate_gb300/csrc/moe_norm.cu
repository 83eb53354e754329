// moe_norm.cu -- the norm in front of an MoE block: the residual's addition, the
// root-mean-square norm of the sum, and optionally the normalised rows in E4M3
// with one power-of-two scale per row.  Per row of H values
//
//   r = residual + x                        (binary32; stored in the stream's type)
//   y = (r * rstd) * w,  rstd = 1 / sqrt(sum(r^2) / H + eps)
//   y_bf16 = bf16(y)
//   e = the smallest integer >= -126 with max|y| <= 448 * 2^e
//   q = e4m3(y * 2^-e), scale = 2^e
//
// The norm is taken of the unrounded sum and both outputs round y once, so q is
// nearer to y than the E4M3 codes of the bf16 rows would be (those round twice).
// The scales have the form of the activation rows of the E4M3 experts.
//
// Bound: HBM.  A row is read once (x and residual) and written once (stream, y,
// q); the row's values stay in registers between the two reductions.
#include <cuda_fp8.h>

#include <algorithm>
#include <mutex>

#include "moe_internal.cuh"

namespace moe {
namespace {

constexpr int NM_THREADS = 256;
constexpr int NM_WARPS = NM_THREADS / 32;

__device__ __forceinline__ void nm_load8(const uint16_t* p, float f[8]) {
    unpack8(*reinterpret_cast<const uint4*>(p), f);
}

template <bool F32>
__device__ __forceinline__ void nm_load_res(const void* res, int64_t off, float f[8]) {
    if (F32) {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(res) + off);
        const float4 a = p[0], b = p[1];
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    } else {
        nm_load8(static_cast<const uint16_t*>(res) + off, f);
    }
}

__device__ __forceinline__ uint4 nm_pack8(const float f[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
}

// Smallest e >= -126 with amax <= 448 * 2^e (448 = 1.75 * 2^8), from the binary32 fields.
__device__ __forceinline__ int nm_exponent(float amax) {
    const uint32_t b = __float_as_uint(amax);
    const int e = (int)(b >> 23) - 135 + ((b & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return e < -126 ? -126 : e;
}

__device__ __forceinline__ uint32_t nm_e4m3x4(const float* f, float inv) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(f[0] * inv, f[1] * inv), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(f[2] * inv, f[3] * inv), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}

// One CTA per row at a time (grid-stride): each thread owns VPT vectors of 8 values.
template <int VPT, bool F32>
__global__ void __launch_bounds__(NM_THREADS) add_rmsnorm_kernel(const __grid_constant__ NormLaunch a) {
    __shared__ float red_sum[2][NM_WARPS];
    __shared__ uint32_t red_max[2][NM_WARPS];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int vec = a.H / 8;
    pdl_wait();
    pdl_trigger();
    int it = 0;
    for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x, it ^= 1) {
        const int64_t base = row * a.H;
        float f[VPT][8];
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = threadIdx.x + j * NM_THREADS;
            if (v >= vec) continue;
            nm_load8(a.x + base + 8 * v, f[j]);
            if (a.residual) {
                float r[8];
                nm_load_res<F32>(a.residual, base + 8 * v, r);
#pragma unroll
                for (int i = 0; i < 8; ++i) f[j][i] += r[i];
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) ss = fmaf(f[j][i], f[j][i], ss);
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, off);
        if (lane == 0) red_sum[it][warp] = ss;
        __syncthreads();
        float tot = 0.f;
#pragma unroll
        for (int w = 0; w < NM_WARPS; ++w) tot += red_sum[it][w];
        const float rstd = __frsqrt_rn(tot / (float)a.H + a.eps);
        uint32_t mx = 0u;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = threadIdx.x + j * NM_THREADS;
            if (v >= vec) continue;
            if (a.residual_out) {
                if (F32) {
                    float4* p = reinterpret_cast<float4*>(static_cast<float*>(a.residual_out) + base + 8 * v);
                    p[0] = make_float4(f[j][0], f[j][1], f[j][2], f[j][3]);
                    p[1] = make_float4(f[j][4], f[j][5], f[j][6], f[j][7]);
                } else {
                    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.residual_out) + base + 8 * v) = nm_pack8(f[j]);
                }
            }
            float w[8];
            nm_load8(a.weight + 8 * v, w);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                f[j][i] = (f[j][i] * rstd) * w[i];
                mx = max(mx, __float_as_uint(f[j][i]) & 0x7FFFFFFFu);
            }
            if (a.y) *reinterpret_cast<uint4*>(a.y + base + 8 * v) = nm_pack8(f[j]);
        }
        if (!a.q) continue;
        mx = __reduce_max_sync(0xffffffffu, mx);
        if (lane == 0) red_max[it][warp] = mx;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < NM_WARPS; ++w) mx = max(mx, red_max[it][w]);
        const int e = nm_exponent(__uint_as_float(mx));
        const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
        if (threadIdx.x == 0) a.scale[row] = __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = threadIdx.x + j * NM_THREADS;
            if (v < vec)
                *reinterpret_cast<uint2*>(a.q + base + 8 * v) =
                    make_uint2(nm_e4m3x4(f[j], inv), nm_e4m3x4(f[j] + 4, inv));
        }
    }
}

template <int VPT>
cudaError_t launch_norm_vpt(const NormLaunch& L, unsigned grid, cudaStream_t s) {
    if (L.f32) return launch_k("add_rmsnorm", add_rmsnorm_kernel<VPT, true>, dim3(grid), dim3(NM_THREADS), 0, s, L);
    return launch_k("add_rmsnorm", add_rmsnorm_kernel<VPT, false>, dim3(grid), dim3(NM_THREADS), 0, s, L);
}

}  // namespace

cudaError_t launch_add_rmsnorm(const NormLaunch& L, int num_sms, cudaStream_t s) {
    const int vpt = (L.H / 8 + NM_THREADS - 1) / NM_THREADS;
    const unsigned grid = (unsigned)std::max<int64_t>(1, std::min<int64_t>(L.T, (int64_t)num_sms * 8));
    if (vpt <= 1) return launch_norm_vpt<1>(L, grid, s);
    if (vpt <= 2) return launch_norm_vpt<2>(L, grid, s);
    if (vpt <= 4) return launch_norm_vpt<4>(L, grid, s);
    return launch_norm_vpt<8>(L, grid, s);
}

}  // namespace moe

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
// q); the row's values stay in registers between the two reductions.  16384 rows of
// 7168 with a bf16 stream, y and E4M3 rows: 164 us, 1.06 GB at 6.45 TB/s, 0.95 of this
// card's copy rate; with an fp32 stream 237 us, 1.53 GB at 6.43 TB/s.  Small batches are
// bound by latency: one row of 2048 1.9 us, 32 of 7168 with an fp32 stream 3.8 us, 777 of
// 1408 3.7 us, each call behind the last.
//
// The sum of squares, rstd, y before its rounding and the maximum are binary32.  The
// stream's bf16 form rounds r once, where the model's next layer would read it.
#include <cuda_fp8.h>

#include <algorithm>

#include "moe_internal.cuh"

namespace moe {
namespace {

constexpr int NM_WARPS = 8;      // rows of a CTA whose warps take one each
constexpr int NM_CTAS = 64;      // CTAs an SM before they loop over rows

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

// THREADS threads per row at a time, each with VPT vectors of 8 values (grid-stride over
// rows): a CTA, or (THREADS = 32) each of its NM_WARPS warps by itself.
template <int VPT, int THREADS, bool F32>
__global__ void __launch_bounds__(THREADS > 32 ? THREADS : NM_WARPS * 32) add_rmsnorm_kernel(const __grid_constant__ NormLaunch a) {
    constexpr int WARPS = THREADS / 32;
    __shared__ float red_sum[2][WARPS];
    __shared__ uint32_t red_max[2][WARPS];
    constexpr bool ALONE = THREADS == 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int first = ALONE ? lane : threadIdx.x;
    const int vec = a.H / 8;
    pdl_wait();
    pdl_trigger();
    int it = 0;
    const int64_t rows = (int64_t)gridDim.x * (ALONE ? NM_WARPS : 1);
    for (int64_t row = ALONE ? (int64_t)blockIdx.x * NM_WARPS + warp : blockIdx.x; row < a.T; row += rows, it ^= 1) {
        const int64_t base = row * a.H;
        float f[VPT][8];
        float ss = 0.f;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = first + j * THREADS;
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
        float tot = ss;
        if (!ALONE) {
            if (lane == 0) red_sum[it][warp] = ss;
            __syncthreads();
            tot = 0.f;
#pragma unroll
            for (int w = 0; w < WARPS; ++w) tot += red_sum[it][w];
        }
        // the root's reciprocal in two words: its own rounding, which would move a whole row of
        // y by up to 2^-24, is taken out.  ms stays one binary32 value: the roundings of the
        // sum, of the division and of eps move the row by half of theirs
        const float ms = tot / (float)a.H + a.eps;
        const float hi = __frsqrt_rn(ms);
        const float sq = ms * hi, err = fmaf(-sq, hi, 1.f) - fmaf(ms, hi, -sq) * hi;
        float lo = 0.5f * hi * err;
        if (!(fabsf(lo) < hi)) lo = 0.f;  // not finite: an infinite or zero mean square
        uint32_t mx = 0u;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = first + j * THREADS;
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
                f[j][i] = fmaf(f[j][i], hi, f[j][i] * lo) * w[i];
                mx = max(mx, __float_as_uint(f[j][i]) & 0x7FFFFFFFu);
            }
            if (a.y) *reinterpret_cast<uint4*>(a.y + base + 8 * v) = nm_pack8(f[j]);
        }
        if (!a.q) continue;
        mx = __reduce_max_sync(0xffffffffu, mx);
        if (!ALONE) {
            if (lane == 0) red_max[it][warp] = mx;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < WARPS; ++w) mx = max(mx, red_max[it][w]);
        }
        const int e = nm_exponent(__uint_as_float(mx));
        const float inv = __uint_as_float((uint32_t)(127 - e) << 23);
        if (first == 0) a.scale[row] = __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = first + j * THREADS;
            if (v < vec)
                *reinterpret_cast<uint2*>(a.q + base + 8 * v) =
                    make_uint2(nm_e4m3x4(f[j], inv), nm_e4m3x4(f[j] + 4, inv));
        }
    }
}

template <int VPT, int THREADS, bool F32>
cudaError_t launch_norm_size(const NormLaunch& L, int num_sms, cudaStream_t s) {
    constexpr int ROWS = THREADS == 32 ? NM_WARPS : 1;
    const unsigned grid = (unsigned)std::min<int64_t>((L.T + ROWS - 1) / ROWS, (int64_t)num_sms * NM_CTAS);
    return launch_k("add_rmsnorm", add_rmsnorm_kernel<VPT, THREADS, F32>, dim3(grid), dim3(THREADS * ROWS), 0, s, L);
}

template <bool F32>
cudaError_t launch_norm_type(const NormLaunch& L, int num_sms, cudaStream_t s) {
    // A warp to a row while its lanes hold it in two vectors each, then one vector a thread
    // to 2048 values, and a CTA of 224 or 256 threads with four: at 7168 values (16384 rows
    // with E4M3 rows) four of 224 threads take 164 us, two of 448 take 201, one of 896 197
    // and four of 256 (an eighth of them idle) 175.  That width alone was compared; the other
    // widths of these forms run at (16384 rows, of the copy rate): 4096 0.99, 5120 (a vector of
    // four idle) 0.90, 6144 0.90, and at 1.06 GB 8192 0.91, 16384 0.84.
    const int vec = L.H / 8;
    if (vec <= 32) return launch_norm_size<1, 32, F32>(L, num_sms, s);
    if (vec <= 64) return launch_norm_size<2, 32, F32>(L, num_sms, s);
    if (vec <= 128) return launch_norm_size<1, 128, F32>(L, num_sms, s);
    if (vec <= 256) return launch_norm_size<1, 256, F32>(L, num_sms, s);
    if (vec <= 512) return launch_norm_size<2, 256, F32>(L, num_sms, s);
    if (vec <= 896) return launch_norm_size<4, 224, F32>(L, num_sms, s);
    if (vec <= 1024) return launch_norm_size<4, 256, F32>(L, num_sms, s);
    return launch_norm_size<4, 512, F32>(L, num_sms, s);
}

}  // namespace

cudaError_t launch_add_rmsnorm(const NormLaunch& L, int num_sms, cudaStream_t s) {
    return L.f32 ? launch_norm_type<true>(L, num_sms, s) : launch_norm_type<false>(L, num_sms, s);
}

}  // namespace moe

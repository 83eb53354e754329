// moe_norm_bwd.cu -- the gradients of the two norms in front of an MoE block, and the
// column sums that weight gradients are.  Per row r of H values, with g = dy * weight,
// d = r - mean (layer norm) or r (RMS norm) and rstd = 1 / sqrt(sum(d^2) / H + eps):
//
//   dr = dstream + rstd * (g - [layer norm: sum(g) / H] - d * rstd^2 * sum(g d) / H)
//   dweight = sum over rows of dy * d * rstd,  dbias = sum over rows of dy
//
// The row's statistics are taken again from r: the row has to be read for d anyway.  All
// sums are binary32; dr is rounded once for each of its outputs.
#include <algorithm>

#include "moe_internal.cuh"

namespace moe {
namespace {

constexpr int NB_THREADS = 512;
constexpr int NB_VPT = 4;        // vectors of 8 values a thread owns: H <= 16384

template <bool F32>
__device__ __forceinline__ void nb_load(const void* p, int64_t off, float f[8]) {
    if (F32) {
        const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + off);
        const float4 a = q[0], b = q[1];
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    } else {
        unpack8(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + off), f);
    }
}

template <bool F32>
__device__ __forceinline__ void nb_store(void* p, int64_t off, const float f[8]) {
    if (F32) {
        float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + off);
        q[0] = make_float4(f[0], f[1], f[2], f[3]);
        q[1] = make_float4(f[4], f[5], f[6], f[7]);
    } else {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + off) = pack8(f);
    }
}

__device__ __forceinline__ float nb_block_sum(float v, float* red) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    float tot = 0.f;
    for (int w = 0; w < NB_THREADS / 32; ++w) tot += red[w];
    __syncthreads();
    return tot;
}

template <bool F32, bool LN>
__global__ void __launch_bounds__(NB_THREADS) norm_bwd_kernel(const __grid_constant__ NormBwdLaunch a) {
    __shared__ float red[NB_THREADS / 32];
    const int vec = a.H / 8;
    const float inv_h = 1.f / (float)a.H;
    float dw[NB_VPT][8] = {}, db[NB_VPT][8] = {};
    pdl_wait();
    pdl_trigger();
    for (int64_t row = blockIdx.x; row < a.T; row += gridDim.x) {
        const int64_t base = row * a.H;
        float mean = 0.f;
        if (LN) {
            float sum = 0.f;
            for (int v = threadIdx.x; v < vec; v += NB_THREADS) {
                float r[8];
                nb_load<F32>(a.r, base + 8 * v, r);
                for (int i = 0; i < 8; ++i) sum += r[i];
            }
            mean = nb_block_sum(sum, red) / (float)a.H;
        }
        float sd = 0.f, sg = 0.f, sgd = 0.f;
        for (int v = threadIdx.x; v < vec; v += NB_THREADS) {
            float r[8], g[8], w[8];
            nb_load<F32>(a.r, base + 8 * v, r);
            nb_load<false>(a.dy, base + 8 * v, g);
            nb_load<false>(a.weight, 8 * v, w);
            for (int i = 0; i < 8; ++i) {
                const float d = r[i] - mean, gw = g[i] * w[i];
                sd = fmaf(d, d, sd);
                sg += gw;
                sgd = fmaf(gw, d, sgd);
            }
        }
        sd = nb_block_sum(sd, red);
        if (LN) sg = nb_block_sum(sg, red);
        sgd = nb_block_sum(sgd, red);
        const float rstd = rsqrtf(sd / (float)a.H + a.eps);
        const float mg = LN ? sg * inv_h : 0.f, mgd = rstd * rstd * (sgd * inv_h);
#pragma unroll
        for (int j = 0; j < NB_VPT; ++j) {
            const int v = threadIdx.x + j * NB_THREADS;
            if (v >= vec) continue;
            float r[8], g[8], w[8], o[8] = {};
            nb_load<F32>(a.r, base + 8 * v, r);
            nb_load<false>(a.dy, base + 8 * v, g);
            nb_load<false>(a.weight, 8 * v, w);
            if (a.dstream) nb_load<F32>(a.dstream, base + 8 * v, o);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float d = r[i] - mean;
                dw[j][i] = fmaf(g[i], d * rstd, dw[j][i]);
                if (LN) db[j][i] += g[i];
                o[i] = fmaf(rstd, fmaf(g[i], w[i], -mg) - d * mgd, o[i]);
            }
            if (a.dr) nb_store<F32>(a.dr, base + 8 * v, o);
            if (a.dx) nb_store<false>(a.dx, base + 8 * v, o);
        }
    }
    float* part = a.part + (int64_t)blockIdx.x * 2 * a.H;
#pragma unroll
    for (int j = 0; j < NB_VPT; ++j) {
        const int v = threadIdx.x + j * NB_THREADS;
        if (v >= vec) continue;
        if (a.dweight) nb_store<true>(part, 8 * v, dw[j]);
        if (LN && a.dbias) nb_store<true>(part, a.H + 8 * v, db[j]);
    }
}

// A CTA adds 32 columns: warp w takes the partial rows w, w + 32, ..., then the warps' sums
// are added in order.
constexpr int SP_WARPS = 32;

__global__ void __launch_bounds__(SP_WARPS * 32) sum_partials_kernel(const float* part, int n, int64_t stride, int H,
                                                                   float* out0, float* out1) {
    __shared__ float red[SP_WARPS][33];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int col = blockIdx.x * 32 + lane;
    float* out = blockIdx.y ? out1 : out0;
    float s = 0.f;
    if (col < H && out)
        for (int i = warp; i < n; i += SP_WARPS) s += part[i * stride + (int64_t)blockIdx.y * H + col];
    red[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && col < H && out) {
        s = 0.f;
        for (int w = 0; w < SP_WARPS; ++w) s += red[w][lane];
        out[col] = s;
    }
}

}  // namespace

cudaError_t launch_sum_partials(const float* part, int n, int64_t stride, int H, float* out0, float* out1,
                                cudaStream_t s) {
    return launch_k("sum_partials", sum_partials_kernel, dim3((H + 31) / 32, out1 ? 2 : 1), dim3(SP_WARPS * 32), 0, s,
                    part, n, stride, H, out0, out1);
}

cudaError_t launch_norm_bwd(const NormBwdLaunch& L, int num_sms, cudaStream_t s) {
    const int grid = (int)std::min<int64_t>(L.T, std::min(num_sms, kBwdPartials));
    const auto kernel = L.f32 ? (L.ln ? norm_bwd_kernel<true, true> : norm_bwd_kernel<true, false>)
                              : (L.ln ? norm_bwd_kernel<false, true> : norm_bwd_kernel<false, false>);
    const cudaError_t e = launch_k(L.ln ? "layernorm_bwd" : "rmsnorm_bwd", kernel, dim3(grid), dim3(NB_THREADS), 0, s, L);
    if (e != cudaSuccess || (!L.dweight && !L.dbias)) return e;
    return launch_sum_partials(L.part, grid, 2 * (int64_t)L.H, L.H, L.dweight, L.dbias, s);
}

}  // namespace moe

// moe_finalize_bwd.cu -- the gradients of the rows sorted by slot and of the weighted
// combine: the way back of moe_permute and of moe_finalize.
//
// moe_finalize: out[t] = sum_j w[t,j] y[row(t,j)] + g_t y_sh[t], g_t = sigmoid(z_t), z_t = x[t] . gate_w:
//   dy[row(t,j)] = w[t,j] dout[t],  dw[t,j] = y[row(t,j)] . dout[t]
//   dy_sh[t] = g_t dout[t],  dz_t = g_t (1 - g_t) (dout[t] . y_sh[t]),  dgate_w = sum_t dz_t x[t]
// moe_permute: x_perm[row(t,j)] = w[t,j] x[t] (or x[t]):
//   dx[t] = add[t] + sum_j w[t,j] dx_perm[row(t,j)] + dz_t gate_w,  dw[t,j] = x[t] . dx_perm[row(t,j)]
//
// Every sum is binary32 in a fixed order and every bf16 output is rounded once.
#include <algorithm>

#include "moe_internal.cuh"

namespace moe {
namespace {

constexpr int FB_WARPS = 8;

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

__device__ __forceinline__ int32_t pair_row_of(const int32_t* pair_row, int64_t p, int64_t rows_cap, int32_t* status) {
    const int32_t r = pair_row[p];
    if (r >= -1 && r < rows_cap) return r;
    report(status, MOE_ERR_DEVICE_BOUNDS);
    return -1;
}

// A warp to a pair, or (the last T warps, with a gate) to a token's shared expert.
__global__ void __launch_bounds__(FB_WARPS * 32) finalize_bwd_kernel(const __grid_constant__ FinalizeBwdLaunch a) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, vec = a.H / 8;
    const int64_t pairs = a.T * a.k, units = pairs + (a.gate_w ? a.T : 0);
    for (int64_t u = (int64_t)blockIdx.x * FB_WARPS + warp; u < units; u += (int64_t)gridDim.x * FB_WARPS) {
        if (u < pairs) {
            const int64_t t = u / a.k;
            const int32_t r = pair_row_of(a.pair_row, u, a.rows_cap, lane == 0 ? &a.hdr->status : nullptr);
            float dot = 0.f;
            if (r >= 0) {
                const float w = a.w ? a.w[u] : 1.f;
                const uint4* dout = reinterpret_cast<const uint4*>(a.dout + t * a.H);
                const uint16_t* y = a.y + (int64_t)r * a.H;
                uint4* dy = reinterpret_cast<uint4*>(a.dy + (int64_t)r * a.H);
                for (int v = lane; v < vec; v += 32) {
                    float d[8], f[8];
                    unpack8(dout[v], d);
                    if (a.dw) {
                        unpack8(reinterpret_cast<const uint4*>(y)[v], f);
                        for (int i = 0; i < 8; ++i) dot = fmaf(d[i], f[i], dot);
                    }
                    for (int i = 0; i < 8; ++i) d[i] *= w;
                    dy[v] = pack8(d);
                }
            }
            if (a.dw) {
                dot = warp_sum(dot);
                if (lane == 0) a.dw[u] = dot;
            }
        } else {
            const int64_t t = u - pairs;
            const uint4* dout = reinterpret_cast<const uint4*>(a.dout + t * a.H);
            const uint4* ysh = reinterpret_cast<const uint4*>(a.y_sh + t * a.H);
            const uint4* x = reinterpret_cast<const uint4*>(a.x + t * a.H);
            const uint4* gw = reinterpret_cast<const uint4*>(a.gate_w);
            float z = 0.f, dot = 0.f;
            for (int v = lane; v < vec; v += 32) {
                float d[8], f[8];
                unpack8(x[v], d);
                unpack8(gw[v], f);
                for (int i = 0; i < 8; ++i) z = fmaf(d[i], f[i], z);
                unpack8(dout[v], d);
                unpack8(ysh[v], f);
                for (int i = 0; i < 8; ++i) dot = fmaf(d[i], f[i], dot);
            }
            z = warp_sum(z);
            dot = warp_sum(dot);
            const float g = 1.f / (1.f + expf(-z));
            if (lane == 0) a.dgate[t] = g * (1.f / (1.f + expf(z))) * dot;
            uint4* dysh = reinterpret_cast<uint4*>(a.dy_sh + t * a.H);
            for (int v = lane; v < vec; v += 32) {
                float d[8];
                unpack8(dout[v], d);
                for (int i = 0; i < 8; ++i) d[i] *= g;
                dysh[v] = pack8(d);
            }
        }
    }
}

// Partial column sums of dz_t x[t]: a CTA takes FB_WARPS * 32 vectors of 8 columns and every
// gridDim.y-th row.
__global__ void __launch_bounds__(FB_WARPS * 32) gate_weight_kernel(const float* dz, const uint16_t* x, int64_t T, int H,
                                                                  float* part) {
    pdl_wait();
    pdl_trigger();
    const int v = blockIdx.x * FB_WARPS * 32 + threadIdx.x;
    if (v >= H / 8) return;
    float acc[8] = {};
    for (int64_t t = blockIdx.y; t < T; t += gridDim.y) {
        float f[8];
        unpack8(reinterpret_cast<const uint4*>(x + t * H)[v], f);
        const float d = dz[t];
        for (int i = 0; i < 8; ++i) acc[i] = fmaf(d, f[i], acc[i]);
    }
    float4* o = reinterpret_cast<float4*>(part + (int64_t)blockIdx.y * H + 8 * v);
    o[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
    o[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
}

// A warp to a token; up to 8 pairs' dots at a time.
__global__ void __launch_bounds__(FB_WARPS * 32) permute_bwd_kernel(const __grid_constant__ PermuteBwdLaunch a) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, vec = a.H / 8;
    for (int64_t t = (int64_t)blockIdx.x * FB_WARPS + warp; t < a.T; t += (int64_t)gridDim.x * FB_WARPS) {
        int32_t my_row = -1;
        float my_w = 1.f, my_dot = 0.f;
        if (lane < a.k) {
            my_row = pair_row_of(a.pair_row, t * a.k + lane, a.rows_cap, &a.hdr->status);
            if (a.w) my_w = a.w[t * a.k + lane];
        }
        const float dz = a.dgate ? a.dgate[t] : 0.f;
        for (int v0 = 0; v0 < vec; v0 += 32) {
            const int v = v0 + lane;
            const bool in = v < vec;
            float x[8] = {}, acc[8] = {};
            if (in && a.dw) unpack8(reinterpret_cast<const uint4*>(a.x + t * a.H)[v], x);
            if (in && a.add) {
                if (a.add_f32) {
                    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(a.add) + t * a.H) + 2 * v;
                    const float4 lo = p[0], hi = p[1];
                    acc[0] = lo.x; acc[1] = lo.y; acc[2] = lo.z; acc[3] = lo.w;
                    acc[4] = hi.x; acc[5] = hi.y; acc[6] = hi.z; acc[7] = hi.w;
                } else {
                    unpack8(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.add) + t * a.H)[v], acc);
                }
            }
            for (int j = 0; j < a.k; ++j) {
                const int32_t r = __shfl_sync(0xffffffffu, my_row, j);
                const float w = __shfl_sync(0xffffffffu, my_w, j);
                if (r < 0) continue;
                float d[8] = {}, dot = 0.f;
                if (in) unpack8(reinterpret_cast<const uint4*>(a.dx_perm + (int64_t)r * a.H)[v], d);
                for (int i = 0; i < 8; ++i) {
                    acc[i] = fmaf(w, d[i], acc[i]);
                    dot = fmaf(x[i], d[i], dot);
                }
                if (a.dw) {
                    dot = warp_sum(dot);
                    if (lane == j) my_dot += dot;
                }
            }
            if (in && a.dgate) {
                float g[8];
                unpack8(reinterpret_cast<const uint4*>(a.gate_w)[v], g);
                for (int i = 0; i < 8; ++i) acc[i] = fmaf(dz, g[i], acc[i]);
            }
            if (in) reinterpret_cast<uint4*>(a.dx + t * a.H)[v] = pack8(acc);
        }
        if (a.dw && lane < a.k) a.dw[t * a.k + lane] = my_dot;
    }
}

}  // namespace

cudaError_t launch_finalize_bwd(const FinalizeBwdLaunch& L, int num_sms, cudaStream_t s) {
    const int64_t units = L.T * L.k + (L.gate_w ? L.T : 0);
    const unsigned grid = (unsigned)std::min<int64_t>((units + FB_WARPS - 1) / FB_WARPS, (int64_t)num_sms * 64);
    cudaError_t e = launch_k("finalize_bwd", finalize_bwd_kernel, dim3(grid), dim3(FB_WARPS * 32), 0, s, L);
    if (e != cudaSuccess || !L.dgate_w) return e;
    const int splits = (int)std::min<int64_t>(L.T, kBwdPartials);
    e = launch_k("gate_weight_bwd", gate_weight_kernel, dim3((L.H / 8 + FB_WARPS * 32 - 1) / (FB_WARPS * 32), splits),
                 dim3(FB_WARPS * 32), 0, s, L.dgate, L.x, L.T, L.H, L.part);
    if (e != cudaSuccess) return e;
    return launch_sum_partials(L.part, splits, L.H, L.H, L.dgate_w, nullptr, s);
}

cudaError_t launch_permute_bwd(const PermuteBwdLaunch& L, int num_sms, cudaStream_t s) {
    const unsigned grid = (unsigned)std::min<int64_t>((L.T + FB_WARPS - 1) / FB_WARPS, (int64_t)num_sms * 64);
    return launch_k("permute_bwd", permute_bwd_kernel, dim3(grid), dim3(FB_WARPS * 32), 0, s, L);
}

}  // namespace moe

// moe_w4.cu -- products of a few activation rows with 4-bit weights that carry one
// bf16 scale per group of consecutive elements of a row:
//
//   W[n][k] = s[n][k / group] * c[n][k],  c in -8 .. 7,   y[m][n] = sum_k x[m][k] W[n][k]
//
// as one matrix (moe_matvec_w4) and as the experts of an MoE layer at decode
// (moe_forward_w4: FC1 + SwiGLU, FC2, weighted combine, an optional shared expert).
//
// Packing: eight consecutive elements of a row share a 32-bit word (little-endian),
// element 2i in nibble i and element 2i + 1 in nibble i + 4, each as c + 8.  Masking
// a word shifted by 4i with 0x000F000F leaves elements 2i and 2i + 1 in the two
// 16-bit halves, and or-ing 0x4300 into each makes them the bf16 values 128 + (c + 8)
// (exact: bf16 has seven fraction bits), in the order in which the activations lie
// in memory.
#include <algorithm>

#include "moe_internal.cuh"

namespace moe {
namespace {

// ---------------------------------------------------------------------------
// Quantiser: one lane per word of eight elements, a group's lanes reduce together
// ---------------------------------------------------------------------------
constexpr int W4Q_THREADS = 256;

__global__ void __launch_bounds__(W4Q_THREADS) quantize_w4_rows_kernel(const uint16_t* __restrict__ w, int64_t words,
                                                                      int lanes, uint32_t* __restrict__ q,
                                                                      uint16_t* __restrict__ scale) {
    pdl_wait();
    pdl_trigger();
    const int64_t step = (int64_t)gridDim.x * W4Q_THREADS;
    // whole warps stay in the loop: a group never straddles two of them (lanes divides 32)
    const int64_t end = (words + 31) / 32 * 32;
    for (int64_t i = (int64_t)blockIdx.x * W4Q_THREADS + threadIdx.x; i < end; i += step) {
        const bool in = i < words;
        float f[8];
        unpack8(in ? __ldg(reinterpret_cast<const uint4*>(w) + i) : make_uint4(0, 0, 0, 0), f);
        float amax = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(f[j]));
        for (int off = 1; off < lanes; off <<= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
        const uint32_t sb = pack_bf16x2(__fdiv_rn(amax, 7.0f), 0.f) & 0xFFFFu;
        const float s = bf16_bits_to_float(sb);
        uint32_t word = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float c = s == 0.f ? 0.f : fminf(fmaxf(rintf(__fdiv_rn(f[j], s)), -8.f), 7.f);
            word |= (uint32_t)((int)c + 8) << (4 * (j / 2 + 4 * (j & 1)));
        }
        if (in) {
            q[i] = word;
            if (i % lanes == 0) scale[i / lanes] = (uint16_t)sb;
        }
    }
}

// ---------------------------------------------------------------------------
// Products, one warp per (row, output)
// ---------------------------------------------------------------------------
constexpr int W4_WARPS = 8;

// Lane-strided dot product of one weight row with one activation row; every lane
// gets the sum.
__device__ __forceinline__ float w4_dot(const uint8_t* wq, const uint16_t* ws, const uint16_t* x, int K, int group) {
    const int lane = threadIdx.x & 31;
    float acc = 0.f;
    for (int v = lane; v < K / 8; v += 32) {
        const uint32_t word = __ldg(reinterpret_cast<const uint32_t*>(wq) + v);
        float f[8];
        unpack8(*(reinterpret_cast<const uint4*>(x) + v), f);
        float p = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            p = fmaf((float)((int)((word >> (4 * (j / 2 + 4 * (j & 1)))) & 15u) - 8), f[j], p);
        acc = fmaf(bf16_bits_to_float(__ldg(ws + v * 8 / group)), p, acc);
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, off);
    return acc;
}

__device__ __forceinline__ void w4_output(const W4Problem& p, int64_t slot, const uint16_t* x, int64_t out_row, int n,
                                          bool swiglu, int group) {
    const int64_t rows = swiglu ? 2 * (int64_t)p.N_out : p.N_out;
    const uint8_t* wq = p.wq + slot * rows * (p.K / 2);
    const uint16_t* ws = p.ws + slot * rows * (p.K / group);
    float v = w4_dot(wq + (int64_t)n * (p.K / 2), ws + (int64_t)n * (p.K / group), x, p.K, group);
    if (swiglu) {
        const int64_t u = (int64_t)p.N_out + n;
        const float up = w4_dot(wq + u * (p.K / 2), ws + u * (p.K / group), x, p.K, group);
        v = v / (1.0f + expf(-v)) * up;
    }
    if ((threadIdx.x & 31) == 0) {
        if (p.out_f32)
            p.out_f32[out_row * p.N_out + n] = v;
        else
            p.out_bf16[out_row * p.N_out + n] = (uint16_t)(pack_bf16x2(v, 0.f) & 0xFFFFu);
    }
}

__global__ void __launch_bounds__(W4_WARPS * 32) w4_gemm_kernel(const __grid_constant__ W4Launch a) {
    pdl_wait();
    pdl_trigger();
    const int64_t step = (int64_t)gridDim.x * W4_WARPS;
    const int64_t first = (int64_t)blockIdx.x * W4_WARPS + (threadIdx.x >> 5);
    if (a.sh.wq)
        for (int64_t i = first; i < a.rows_sh * a.sh.N_out; i += step) {
            const int64_t r = i / a.sh.N_out;
            w4_output(a.sh, 0, a.sh.x + r * a.sh.K, r, (int)(i - r * a.sh.N_out), a.swiglu, a.group);
        }
    if (a.G == 0) return;
    const int64_t rows = min((int64_t)max(0, __ldg(a.offsets + a.G)), a.rows_cap);
    for (int64_t i = first; i < rows * a.rt.N_out; i += step) {
        const int64_t r = i / a.rt.N_out;
        int lo = 0, hi = a.G - 1;  // the last slot whose rows begin at or before r
        while (lo < hi) {
            const int mid = (lo + hi + 1) / 2;
            if (__ldg(a.offsets + mid) <= r)
                lo = mid;
            else
                hi = mid - 1;
        }
        int64_t xr = r;
        if (a.perm_src) {
            const int32_t p = a.perm_src[r];
            if (p < 0 || (int64_t)p >= a.T * a.k) {
                report(a.status, MOE_ERR_DEVICE_BOUNDS);
                continue;
            }
            xr = p / a.k;
        }
        w4_output(a.rt, lo, a.rt.x + xr * a.rt.K, r, (int)(i - r * a.rt.N_out), a.swiglu, a.group);
    }
}

// ---------------------------------------------------------------------------
// Combine: out[t] = bf16( sum_j w[t][j] y[row] + g_t shared[t] ), fixed j order
// ---------------------------------------------------------------------------
constexpr int W4C_THREADS = 256;
constexpr int W4C_MAXK = 32;

__global__ void __launch_bounds__(W4C_THREADS) w4_combine_kernel(const __grid_constant__ W4CombineLaunch a) {
    __shared__ int32_t s_row[W4C_MAXK];
    __shared__ float s_w[W4C_MAXK];
    __shared__ float s_dot[W4C_THREADS / 32];
    pdl_wait();
    pdl_trigger();
    const int64_t t = blockIdx.x;
    if (threadIdx.x < a.k) {
        int32_t r = a.pair_row[t * a.k + threadIdx.x];
        if (r < -1 || (int64_t)r >= a.rows_cap) {
            report(a.status, MOE_ERR_DEVICE_BOUNDS);
            r = -1;
        }
        s_row[threadIdx.x] = r;
        s_w[threadIdx.x] = a.w ? a.w[t * a.k + threadIdx.x] : 1.0f;
    }
    if (a.gate_w) {
        float d = 0.f;
        for (int v = threadIdx.x; v < a.H / 8; v += W4C_THREADS) {
            float f[8], g[8];
            unpack8(*(reinterpret_cast<const uint4*>(a.x + t * a.H) + v), f);
            unpack8(__ldg(reinterpret_cast<const uint4*>(a.gate_w) + v), g);
#pragma unroll
            for (int i = 0; i < 8; ++i) d = fmaf(f[i], g[i], d);
        }
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) d += __shfl_xor_sync(0xffffffffu, d, off);
        if ((threadIdx.x & 31) == 0) s_dot[threadIdx.x >> 5] = d;
    }
    __syncthreads();
    float g = 1.0f;
    if (a.gate_w) {
        float d = 0.f;
#pragma unroll
        for (int w = 0; w < W4C_THREADS / 32; ++w) d += s_dot[w];
        g = 1.0f / (1.0f + expf(-d));
    }
    // 4 outputs a thread, blockIdx.y a range of W4C_THREADS * 4 outputs
    const int n = (blockIdx.y * W4C_THREADS + threadIdx.x) * 4;
    if (n >= a.H) return;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int j = 0; j < a.k; ++j) {
        const int32_t r = s_row[j];
        if (r < 0) continue;
        const float4 v = *reinterpret_cast<const float4*>(a.y + (int64_t)r * a.H + n);
        const float w = s_w[j];
        acc.x = fmaf(w, v.x, acc.x);
        acc.y = fmaf(w, v.y, acc.y);
        acc.z = fmaf(w, v.z, acc.z);
        acc.w = fmaf(w, v.w, acc.w);
    }
    if (a.y_sh) {
        const float4 v = *reinterpret_cast<const float4*>(a.y_sh + t * a.H + n);
        acc.x = fmaf(g, v.x, acc.x);
        acc.y = fmaf(g, v.y, acc.y);
        acc.z = fmaf(g, v.z, acc.z);
        acc.w = fmaf(g, v.w, acc.w);
    }
    *reinterpret_cast<uint2*>(a.out + t * a.H + n) = make_uint2(pack_bf16x2(acc.x, acc.y), pack_bf16x2(acc.z, acc.w));
}

}  // namespace

cudaError_t launch_quantize_w4_rows(const uint16_t* w, int64_t rows, int K, int group, uint8_t* q, uint16_t* scale,
                                    int num_sms, cudaStream_t s) {
    const int64_t words = rows * (K / 8);
    const int64_t want = (words + W4Q_THREADS - 1) / W4Q_THREADS;
    const unsigned grid = (unsigned)std::max<int64_t>(1, std::min<int64_t>(want, (int64_t)num_sms * 8));
    return launch_k("quantize_w4_rows", quantize_w4_rows_kernel, dim3(grid), dim3(W4Q_THREADS), 0, s, w, words,
                    group / 8, reinterpret_cast<uint32_t*>(q), scale);
}

cudaError_t launch_w4_gemm(const W4Launch& L, int num_sms, cudaStream_t s) {
    const unsigned grid = (unsigned)num_sms * 8;
    return launch_k(L.name, w4_gemm_kernel, dim3(grid), dim3(W4_WARPS * 32), 0, s, L);
}

cudaError_t launch_w4_combine(const W4CombineLaunch& L, cudaStream_t s) {
    const dim3 grid((unsigned)L.T, (unsigned)((L.H + W4C_THREADS * 4 - 1) / (W4C_THREADS * 4)));
    return launch_k("w4_combine", w4_combine_kernel, grid, dim3(W4C_THREADS), 0, s, L);
}

}  // namespace moe

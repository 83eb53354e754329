// moe_route_bwd.cu -- the gradient of the routing weights with respect to the logits.
// Per token with chosen experts id_j, weights w_j and their gradients dw_j:
//
//   c = sum_j w_j dw_j
//   dlogits[e] = sum_j [e = id_j] w_j dw_j - c * p[e]
//
// where p is the softmax over all E logits, or with renormalised weights (a softmax over
// the chosen logits alone) p[e] = sum_j [e = id_j] w_j: 0 for every other expert, and
// sum_j [e = id_j] w_j (dw_j - c) for the chosen ones.
//
// Bound: HBM (4 bytes a logit written, 4 read without renormalisation), latency for small
// batches.  A warp to a token: its lanes write the whole row as if no expert were chosen, 16
// bytes each, and then the lanes of the pairs write their experts' values over it.
// Everything is binary32.
#include <algorithm>

#include "moe_rows.cuh"

namespace moe {
namespace {

constexpr int RB_WARPS = 8;

// A lane holds N logits: the float4s lane, lane + 32, ... of the row (VEC: E a multiple of 4),
// or its values lane, lane + 32, ....
template <int N, bool VEC>
__global__ void __launch_bounds__(RB_WARPS * 32) route_bwd_kernel(const __grid_constant__ RouteBwdLaunch a) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int64_t t = (int64_t)blockIdx.x * RB_WARPS + warp; t < a.T; t += (int64_t)gridDim.x * RB_WARPS) {
        const float* const logits = a.logits ? a.logits + t * a.E : nullptr;
        float* const out = a.dlogits + t * a.E;
        int32_t id = -1;
        float w = 0.f, dw = 0.f, own = 0.f;
        if (lane < a.k) {
            id = a.ids[t * a.k + lane];
            if (id >= 0 && id < a.E) {
                w = a.w[t * a.k + lane];
                dw = a.dw[t * a.k + lane];
            } else {
                report(&a.hdr->status, MOE_ERR_DEVICE_BOUNDS);
                id = -1;
            }
        }
        float l[N];
        if (logits) {
#pragma unroll
            for (int i = 0; i < N; ++i) l[i] = -INFINITY;
            if (VEC) {
#pragma unroll
                for (int i = 0; i < N / 4; ++i)
                    if (4 * (lane + 32 * i) < a.E) {
                        const float4 v = reinterpret_cast<const float4*>(logits)[lane + 32 * i];
                        l[4 * i] = v.x; l[4 * i + 1] = v.y; l[4 * i + 2] = v.z; l[4 * i + 3] = v.w;
                    }
            } else {
#pragma unroll
                for (int i = 0; i < N; ++i)
                    if (lane + 32 * i < a.E) l[i] = logits[lane + 32 * i];
            }
            if (id >= 0) own = logits[id];
        }
        const float c = warp_sum(w * dw);
        float value = logits ? w * dw : w * (dw - c);  // of this lane's pair
        // pairs of one expert (none of moe_route's): the first of them takes the sum of all
        const uint32_t mates = __match_any_sync(0xffffffffu, id);
        if (__any_sync(0xffffffffu, id >= 0 && (mates & (mates - 1))))
            for (int j = 1; j < a.k; ++j) {
                const float v = __shfl_sync(0xffffffffu, value, j);
                if (lane < j && (mates >> j & 1)) value += v;
            }
        const bool first = id >= 0 && lane == __ffs(mates) - 1;
        if (logits) {
            float m = -INFINITY, sum = 0.f;
#pragma unroll
            for (int i = 0; i < N; ++i) m = fmaxf(m, l[i]);
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
#pragma unroll
            for (int i = 0; i < N; ++i) {
                l[i] = expf(l[i] - m);
                sum += l[i];
            }
            const float scale = -c / warp_sum(sum);
#pragma unroll
            for (int i = 0; i < N; ++i) l[i] *= scale;
            value = fmaf(expf(own - m), scale, value);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) l[i] = 0.f;
        }
        __syncwarp();  // the pairs' logits are read: dlogits may be logits
        if (VEC) {
#pragma unroll
            for (int i = 0; i < N / 4; ++i)
                if (4 * (lane + 32 * i) < a.E)
                    reinterpret_cast<float4*>(out)[lane + 32 * i] =
                        make_float4(l[4 * i], l[4 * i + 1], l[4 * i + 2], l[4 * i + 3]);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i)
                if (lane + 32 * i < a.E) out[lane + 32 * i] = l[i];
        }
        __syncwarp();  // the row lies below the pairs' values
        if (first) out[id] = value;
    }
}

template <int N>
cudaError_t launch_route_size(const RouteBwdLaunch& L, int num_sms, cudaStream_t s) {
    const unsigned grid = (unsigned)std::min<int64_t>((L.T + RB_WARPS - 1) / RB_WARPS, (int64_t)num_sms * 64);
    const auto kernel = L.E % 4 == 0 ? route_bwd_kernel<N, true> : route_bwd_kernel<N, false>;
    return launch_k("route_bwd", kernel, dim3(grid), dim3(RB_WARPS * 32), 0, s, L);
}

}  // namespace

cudaError_t launch_route_bwd(const RouteBwdLaunch& L, int num_sms, cudaStream_t s) {
    if (L.E <= 128) return launch_route_size<4>(L, num_sms, s);
    if (L.E <= 256) return launch_route_size<8>(L, num_sms, s);
    return launch_route_size<16>(L, num_sms, s);
}

}  // namespace moe

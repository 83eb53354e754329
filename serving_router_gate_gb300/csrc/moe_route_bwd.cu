// moe_route_bwd.cu -- the gradient of the routing weights with respect to the logits.
// Per token with chosen experts id_j, weights w_j and their gradients dw_j:
//
//   c = sum_j w_j dw_j
//   dlogits[e] = sum_j [e = id_j] w_j dw_j - c * p[e]
//
// where p is the softmax over all E logits, or with renormalised weights (a softmax over
// the chosen logits alone) p[e] = sum_j [e = id_j] w_j: 0 for every other expert.
#include <algorithm>

#include "moe_internal.cuh"

namespace moe {
namespace {

constexpr int RB_WARPS = 8;

// A warp to a token, lane l holding the logits l, l + 32, ... (E <= 512).
template <int PL>
__global__ void __launch_bounds__(RB_WARPS * 32) route_bwd_kernel(const __grid_constant__ RouteBwdLaunch a) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int64_t t = (int64_t)blockIdx.x * RB_WARPS + warp; t < a.T; t += (int64_t)gridDim.x * RB_WARPS) {
        int32_t id = -1;
        float w = 0.f, dw = 0.f;
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
        float c = w * dw;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) c += __shfl_xor_sync(0xffffffffu, c, off);
        float l[PL], scale = 0.f;
        if (a.logits) {
            float m = -INFINITY, sum = 0.f;
#pragma unroll
            for (int i = 0; i < PL; ++i) {
                const int e = lane + 32 * i;
                l[i] = e < a.E ? a.logits[t * a.E + e] : -INFINITY;
                m = fmaxf(m, l[i]);
            }
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
#pragma unroll
            for (int i = 0; i < PL; ++i) {
                l[i] = expf(l[i] - m);
                sum += l[i];
            }
#pragma unroll
            for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
            scale = -c / sum;
        }
#pragma unroll
        for (int i = 0; i < PL; ++i) l[i] = a.logits ? l[i] * scale : 0.f;
        const float v = a.logits ? w * dw : w * (dw - c);
        for (int j = 0; j < a.k; ++j) {
            const int e = __shfl_sync(0xffffffffu, id, j);
            const float add = __shfl_sync(0xffffffffu, v, j);
#pragma unroll
            for (int i = 0; i < PL; ++i)
                if (e == lane + 32 * i) l[i] += add;
        }
#pragma unroll
        for (int i = 0; i < PL; ++i)
            if (lane + 32 * i < a.E) a.dlogits[t * a.E + lane + 32 * i] = l[i];
    }
}

template <int PL>
cudaError_t launch_route_size(const RouteBwdLaunch& L, int num_sms, cudaStream_t s) {
    const unsigned grid = (unsigned)std::min<int64_t>((L.T + RB_WARPS - 1) / RB_WARPS, (int64_t)num_sms * 64);
    return launch_k("route_bwd", route_bwd_kernel<PL>, dim3(grid), dim3(RB_WARPS * 32), 0, s, L);
}

}  // namespace

cudaError_t launch_route_bwd(const RouteBwdLaunch& L, int num_sms, cudaStream_t s) {
    if (L.E <= 64) return launch_route_size<2>(L, num_sms, s);
    if (L.E <= 128) return launch_route_size<4>(L, num_sms, s);
    if (L.E <= 256) return launch_route_size<8>(L, num_sms, s);
    return launch_route_size<16>(L, num_sms, s);
}

}  // namespace moe

// moe_norm_bwd.cu -- the gradients of the two norms in front of an MoE block, and the
// column sums that weight gradients are.  Per row r of H values, with g = dy * weight,
// d = r - mean (layer norm) or r (RMS norm) and rstd = 1 / sqrt(sum(d^2) / H + eps):
//
//   dr = dstream + rstd * (g - [layer norm: sum(g) / H] - d * rstd^2 * sum(g d) / H)
//   dweight = sum over rows of dy * d * rstd,  dbias = sum over rows of dy
//
// The row's statistics are taken again from r: the row has to be read for d anyway.  All
// sums are binary32; dr is rounded once for each of its outputs.
//
// Bound: HBM (8 bytes and about 20 operations an element with a bf16 stream).  A row
// belongs to a group of warps, each thread to the same columns of every row of its group,
// so the weight's sums stay in registers to the end of a persistent grid; a CTA's groups
// then add theirs in order, and a second kernel adds the CTAs'.  A thread copies its own
// columns of the rows to come into shared memory (cp.async): the copies need no barrier,
// and a row's one barrier (the layer norm's two: the mean comes first, so that a row far
// from zero keeps its variance) joins its warps' sums.
#include <algorithm>

#include "moe_internal.cuh"

namespace moe {
namespace {

constexpr int NB_WARPS = 16;           // warps of a CTA at most
constexpr int NB_THREADS = NB_WARPS * 32;
constexpr int NB_STAGES = 4;           // rows in flight per group at most
constexpr int NB_SMEM = 227 * 1024;    // of an SM, less 1 KB a CTA

struct NormBwdPlan {
    int gw, groups, stages;  // warps of a group, groups of a CTA, ring slots
    bool ds_ring;            // dstream goes through the ring
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void cp_async_wait_upto(int n) {  // n uniform, below NB_STAGES
    if (n == 0) cp_async_wait<0>();
    else if (n == 1) cp_async_wait<1>();
    else if (n == 2) cp_async_wait<2>();
    else cp_async_wait<3>();
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

// 8 values of slot[0], or (F32) of slot[0] and slot[n]: a thread's pieces lie n apart.
template <bool F32>
__device__ __forceinline__ void nb_slot(const uint4* slot, int n, float f[8]) {
    const uint4 a = slot[0];
    if (F32) {
        const uint4 b = slot[n];
        f[0] = __uint_as_float(a.x); f[1] = __uint_as_float(a.y); f[2] = __uint_as_float(a.z); f[3] = __uint_as_float(a.w);
        f[4] = __uint_as_float(b.x); f[5] = __uint_as_float(b.y); f[6] = __uint_as_float(b.z); f[7] = __uint_as_float(b.w);
    } else {
        unpack8(a, f);
    }
}

__device__ __forceinline__ float nb_xor_add(float v, int from) {
    for (int off = from; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

// The warp's sum of a in lanes 0..15 and of b in lanes 16..31.
__device__ __forceinline__ float nb_sum2(float a, float b, int lane) {
    const bool hi = lane & 16;
    const float got = __shfl_xor_sync(0xffffffffu, hi ? a : b, 16);
    return nb_xor_add((hi ? b : a) + got, 8);
}

// VPT vectors of 8 columns a thread.
template <int VPT, bool F32, bool LN>
__global__ void __launch_bounds__(NB_THREADS, VPT <= 2 ? 2 : 1)
    norm_bwd_kernel(const __grid_constant__ NormBwdLaunch a, const __grid_constant__ NormBwdPlan p) {
    extern __shared__ uint4 ring[];
    __shared__ float4 red[2][NB_WARPS];
    __shared__ float red_sum[2][NB_WARPS];
    constexpr int RP = F32 ? 2 : 1;  // 16-byte pieces of a vector of r
    const int nthr = blockDim.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int gthr = p.gw * 32, group = warp / p.gw, col = tid - group * gthr, vec = a.H / 8;
    const int pieces = VPT * (1 + RP + (p.ds_ring ? RP : 0));  // a stage's, of every thread
    const float inv_h = 1.f / (float)a.H;
    const int64_t stride = (int64_t)gridDim.x * p.groups;
    const int64_t first = (int64_t)group * gridDim.x + blockIdx.x;
    float dw[VPT][8] = {}, db[LN ? VPT : 1][8] = {};
    pdl_wait();
    pdl_trigger();
    const auto fetch = [&](int64_t row, int stage) {
        if (row < a.T) {
            const uint32_t s = smem_u32(ring + (size_t)stage * pieces * nthr + tid);
#pragma unroll
            for (int j = 0; j < VPT; ++j) {
                const int v = col + j * gthr;
                if (v >= vec) continue;
                const int64_t off = row * a.H + 8 * v;
                cp_async16(s + (j * nthr) * 16, a.dy + off);
#pragma unroll
                for (int i = 0; i < RP; ++i) {
                    cp_async16(s + ((VPT + RP * j + i) * nthr) * 16,
                               static_cast<const char*>(a.r) + off * (F32 ? 4 : 2) + 16 * i);
                    if (p.ds_ring)
                        cp_async16(s + ((VPT + RP * (VPT + j) + i) * nthr) * 16,
                                   static_cast<const char*>(a.dstream) + off * (F32 ? 4 : 2) + 16 * i);
                }
            }
        }
        cp_async_commit();
    };
    const auto group_sync = [&] {
        if (p.gw == 1) __syncwarp();
        else asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(gthr) : "memory");
    };
    for (int s = 0; s < p.stages; ++s) fetch(first + s * stride, s);
    int stage = 0, it = 0;
    for (int64_t row = first; row < a.T; row += stride, it ^= 1) {
        const uint4* slot = ring + (size_t)stage * pieces * nthr + tid;
        cp_async_wait_upto(p.stages - 1);
        float r[VPT][8];
        float mean = 0.f;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            if (col + j * gthr >= vec) continue;
            nb_slot<F32>(slot + (VPT + RP * j) * nthr, nthr, r[j]);
            if (LN)
#pragma unroll
                for (int i = 0; i < 8; ++i) mean += r[j][i];
        }
        if (LN) {
            mean = nb_xor_add(mean, 16);
            if (p.gw > 1) {
                if (lane == 0) red_sum[it][warp] = mean;
                group_sync();
                mean = 0.f;
                for (int w = 0; w < p.gw; ++w) mean += red_sum[it][group * p.gw + w];
            }
            mean *= inv_h;
        }
        float sd = 0.f, sg = 0.f, sgd = 0.f;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = col + j * gthr;
            if (v >= vec) continue;
            float g[8], w[8];
            unpack8(slot[j * nthr], g);
            unpack8(__ldg(reinterpret_cast<const uint4*>(a.weight) + v), w);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float d = LN ? r[j][i] - mean : r[j][i], gw = g[i] * w[i];
                sd = fmaf(d, d, sd);
                if (LN) sg += gw;
                sgd = fmaf(gw, d, sgd);
            }
        }
        // red[.][warp] = {sd, sgd, sg}
        const float two = nb_sum2(sd, sgd, lane);
        if (LN) sg = nb_xor_add(sg, 16);
        float* out = reinterpret_cast<float*>(&red[it][warp]);
        if (lane == 0) out[0] = two;
        if (lane == 16) out[1] = two;
        if (LN && lane == 1) out[2] = sg;
        group_sync();
        sd = sg = sgd = 0.f;
        for (int w = 0; w < p.gw; ++w) {
            const float4 q = red[it][group * p.gw + w];
            sd += q.x;
            sgd += q.y;
            if (LN) sg += q.z;
        }
        const float rstd = rsqrtf(sd / (float)a.H + a.eps);
        const float mg = LN ? sg * inv_h : 0.f, mgd = rstd * rstd * (sgd * inv_h);
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = col + j * gthr;
            if (v >= vec) continue;
            const int64_t off = row * a.H + 8 * v;
            float g[8], w[8], o[8] = {};
            unpack8(slot[j * nthr], g);
            nb_slot<F32>(slot + (VPT + RP * j) * nthr, nthr, r[j]);
            unpack8(__ldg(reinterpret_cast<const uint4*>(a.weight) + v), w);
            if (p.ds_ring) nb_slot<F32>(slot + (VPT + RP * (VPT + j)) * nthr, nthr, o);
            else if (a.dstream) nb_load<F32>(a.dstream, off, o);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float d = LN ? r[j][i] - mean : r[j][i];
                dw[j][i] = fmaf(g[i], d * rstd, dw[j][i]);
                if (LN) db[j][i] += g[i];
                o[i] = fmaf(rstd, fmaf(g[i], w[i], -mg) - d * mgd, o[i]);
            }
            if (a.dr) nb_store<F32>(a.dr, off, o);
            if (a.dx) nb_store<false>(a.dx, off, o);
        }
        fetch(row + p.stages * stride, stage);
        stage = stage + 1 == p.stages ? 0 : stage + 1;
    }
    cp_async_wait<0>();
    if (!a.dweight && !a.dbias) return;
    float* part = a.part + (int64_t)blockIdx.x * 2 * a.H;
    if (p.groups == 1) {
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = col + j * gthr;
            if (v >= vec) continue;
            nb_store<true>(part, 8 * v, dw[j]);
            if (LN) nb_store<true>(part, a.H + 8 * v, db[j]);
        }
        return;
    }
    // the groups' sums, one group behind the other, in the ring's memory
    float* acc = reinterpret_cast<float*>(ring);
    for (int g = 0; g < p.groups; ++g) {
        __syncthreads();
        if (g != group) continue;
#pragma unroll
        for (int j = 0; j < VPT; ++j) {
            const int v = col + j * gthr;
            if (v >= vec) continue;
#pragma unroll
            for (int b = 0; b < (LN ? 2 : 1); ++b) {
                float* q = acc + b * a.H + 8 * v;
                float s[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) s[i] = b ? db[LN ? j : 0][i] : dw[j][i];
                if (g > 0) {
                    float o[8];
                    nb_load<true>(q, 0, o);
#pragma unroll
                    for (int i = 0; i < 8; ++i) s[i] += o[i];
                }
                if (g + 1 < p.groups) nb_store<true>(q, 0, s);
                else nb_store<true>(part, b * a.H + 8 * v, s);
            }
        }
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

template <int VPT, bool F32, bool LN>
cudaError_t launch_norm_bwd_size(const NormBwdLaunch& L, int num_sms, cudaStream_t s) {
    NormBwdPlan p;
    const int vec = L.H / 8;
    p.gw = (vec + VPT * 32 - 1) / (VPT * 32);
    p.groups = NB_WARPS / p.gw;
    const int threads = p.gw * p.groups * 32;
    const size_t per = (size_t)threads * VPT * 16, rp = F32 ? 2 : 1;
    // two CTAs an SM where each then holds two stages, else one; dstream stays out of the ring
    // where it leaves no room for two
    p.ds_ring = L.dstream != nullptr;
    int ctas = VPT <= 2 ? 2 : 1;
    if (ctas == 2 && 2 * per * (1 + rp + (p.ds_ring ? rp : 0)) > NB_SMEM / 2 - 1024) ctas = 1;
    if (2 * per * (1 + rp + (p.ds_ring ? rp : 0)) > NB_SMEM - 1024) p.ds_ring = false;
    const size_t stage = per * (1 + rp + (p.ds_ring ? rp : 0)), room = NB_SMEM / ctas - 1024;
    p.stages = (int)std::min<size_t>(NB_STAGES, room / stage);
    const size_t smem = p.stages * stage;  // at least the 8 * H bytes that the groups' sums take
    const auto kernel = norm_bwd_kernel<VPT, F32, LN>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    const int grid = (int)std::min<int64_t>((L.T + p.groups - 1) / p.groups, std::min(ctas * num_sms, kBwdPartials));
    e = launch_k(LN ? "layernorm_bwd" : "rmsnorm_bwd", kernel, dim3(grid), dim3(threads), smem, s, L, p);
    if (e != cudaSuccess || (!L.dweight && !L.dbias)) return e;
    return launch_sum_partials(L.part, grid, 2 * (int64_t)L.H, L.H, L.dweight, L.dbias, s);
}

template <int VPT>
cudaError_t launch_norm_bwd_vpt(const NormBwdLaunch& L, int num_sms, cudaStream_t s) {
    if (L.f32)
        return L.ln ? launch_norm_bwd_size<VPT, true, true>(L, num_sms, s)
                    : launch_norm_bwd_size<VPT, true, false>(L, num_sms, s);
    return L.ln ? launch_norm_bwd_size<VPT, false, true>(L, num_sms, s)
                : launch_norm_bwd_size<VPT, false, false>(L, num_sms, s);
}

}  // namespace

cudaError_t launch_sum_partials(const float* part, int n, int64_t stride, int H, float* out0, float* out1,
                                cudaStream_t s) {
    return launch_k("sum_partials", sum_partials_kernel, dim3((H + 31) / 32, out1 ? 2 : 1), dim3(SP_WARPS * 32), 0, s,
                    part, n, stride, H, out0, out1);
}

cudaError_t launch_norm_bwd(const NormBwdLaunch& L, int num_sms, cudaStream_t s) {
    // a vector a thread up to 4096 values, two up to 8192, four beyond
    if (L.H <= 4096) return launch_norm_bwd_vpt<1>(L, num_sms, s);
    return L.H <= 8192 ? launch_norm_bwd_vpt<2>(L, num_sms, s) : launch_norm_bwd_vpt<4>(L, num_sms, s);
}

}  // namespace moe

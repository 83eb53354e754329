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
#include "moe_rows.cuh"

namespace moe {
namespace {

constexpr int FB_WARPS = 8;

__device__ __forceinline__ int32_t pair_row_of(const int32_t* pair_row, int64_t p, int64_t rows_cap, int32_t* status) {
    const int32_t r = pair_row[p];
    if (r >= -1 && r < rows_cap) return r;
    report(status, MOE_ERR_DEVICE_BOUNDS);
    return -1;
}

// A warp to a pair; FB_BATCH vectors of dout and of y a lane in flight before they are used.
//
// gate_first: launched behind gate_bwd_kernel, this kernel runs beside it.  It may start once
// every CTA of that one has passed its own wait, so all they both read is there; neither writes
// what the other touches; and the wait of one CTA at its end makes this kernel's end that of
// both, for whatever is launched behind it.
constexpr int FB_BATCH = 4;

// PP: pairs a warp takes at a time, for rows so short that one of them does not fill a batch (16384
// tokens of 256, 8 pairs: 36 us with four, 56 with one).
template <int PP>
__global__ void __launch_bounds__(FB_WARPS * 32) finalize_bwd_kernel(const __grid_constant__ FinalizeBwdLaunch a) {
    constexpr int V = FB_BATCH / PP;  // vectors of a pair in flight a lane
    if (!a.gate_first) pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5, vec = a.H / 8;
    const uint32_t pairs = (uint32_t)(a.T * a.k);  // below 2^31
    for (int64_t u0 = ((int64_t)blockIdx.x * warps + warp) * PP; u0 < pairs; u0 += (int64_t)gridDim.x * warps * PP) {
        int32_t r[PP];
        float w[PP], dot[PP] = {};
        const uint4 *dout[PP], *y[PP];
        uint4* dy[PP];
#pragma unroll
        for (int p = 0; p < PP; ++p) {
            const uint32_t u = (uint32_t)u0 + p;
            r[p] = PP == 1 || u < pairs ? pair_row_of(a.pair_row, u, a.rows_cap, lane == 0 ? &a.hdr->status : nullptr) : -1;
            w[p] = r[p] >= 0 && a.w ? a.w[u] : 1.f;
            const int64_t row = r[p] >= 0 ? r[p] : 0;
            dout[p] = reinterpret_cast<const uint4*>(a.dout + (int64_t)(u / (uint32_t)a.k) * a.H);
            y[p] = reinterpret_cast<const uint4*>(a.y + row * a.H);  // not __ldg: dy may be y
            dy[p] = reinterpret_cast<uint4*>(a.dy + row * a.H);
        }
        const int end = PP == 1 && r[0] < 0 ? 0 : vec;
        for (int v0 = lane; v0 < end; v0 += 32 * V) {
            uint4 d[PP][V], f[PP][V];
#pragma unroll
            for (int p = 0; p < PP; ++p)
#pragma unroll
                for (int b = 0; b < V; ++b) {
                    const bool ok = (PP == 1 || r[p] >= 0) && v0 + 32 * b < vec;
                    d[p][b] = ok ? dout[p][v0 + 32 * b] : make_uint4(0, 0, 0, 0);
                    f[p][b] = ok && a.dw ? y[p][v0 + 32 * b] : make_uint4(0, 0, 0, 0);
                }
#pragma unroll
            for (int p = 0; p < PP; ++p)
#pragma unroll
                for (int b = 0; b < V; ++b) {
                    float x[8], z[8];
                    unpack8(d[p][b], x);
                    unpack8(f[p][b], z);
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        dot[p] = fmaf(x[i], z[i], dot[p]);
                        x[i] *= w[p];
                    }
                    if ((PP == 1 || r[p] >= 0) && v0 + 32 * b < vec) dy[p][v0 + 32 * b] = pack8(x);
                }
        }
        if (a.dw)
#pragma unroll
            for (int p = 0; p < PP; ++p) {
                dot[p] = warp_sum(dot[p]);
                if (lane == 0 && (PP == 1 || (uint32_t)u0 + p < pairs)) a.dw[u0 + p] = dot[p];
            }
    }
    if (a.gate_first && blockIdx.x == 0) pdl_wait();
}

// The gated shared expert of rows of at most GB_MAX_H values: a group of gw warps to a token,
// 16 columns a thread (the same ones of every token, so that the gate weight's sums stay in
// registers over a persistent grid), the next token's rows in flight.  A CTA's groups add
// their sums in order, the CTAs' are added by another kernel.  A CTA an SM of GB_CTA_WARPS
// warps (more only for rows that need them) leaves room for the pairs' CTAs beside it: 4096
// tokens of 2048, 4 pairs, 35.5 us in all with 8 warps, 38 with 12, 39.6 with 16, 40.6 with 4;
// 39.1 one behind the other.
constexpr int GB_WARPS = 16, GB_MAX_H = GB_WARPS * 512, GB_CTA_WARPS = 8;

__device__ __forceinline__ float gate_of(float z) { return 1.f / (1.f + expf(-z)); }

__global__ void __launch_bounds__(GB_WARPS * 32, 1) gate_bwd_kernel(const __grid_constant__ FinalizeBwdLaunch a, int gw,
                                                                  int groups) {
    __shared__ alignas(16) float red[2][GB_WARPS * 2];
    extern __shared__ float4 acc[];  // with more than one group: H floats
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, vec = a.H / 8;
    const int group = warp / gw, col = (warp - group * gw) * 64 + lane;  // in vectors of 8: col and col + 32
    const bool in[2] = {col < vec, col + 32 < vec};
    const auto sync = [&] { asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(gw * 32) : "memory"); };
    const int64_t stride = (int64_t)gridDim.x * groups;
    float sum[2][8] = {};
    uint4 w[2] = {}, next[3][2] = {};
    pdl_wait();
    pdl_trigger();
    const uint16_t* const src[3] = {a.dout, a.y_sh, a.x};
    const auto fetch = [&](int64_t t) {
#pragma unroll
        for (int s = 0; s < 3; ++s)
#pragma unroll
            for (int j = 0; j < 2; ++j)
                if (t < a.T && in[j]) next[s][j] = __ldg(reinterpret_cast<const uint4*>(src[s] + t * a.H) + col + 32 * j);
    };
    int64_t t = (int64_t)group * gridDim.x + blockIdx.x;
    fetch(t);
#pragma unroll
    for (int j = 0; j < 2; ++j)
        if (in[j]) w[j] = __ldg(reinterpret_cast<const uint4*>(a.gate_w) + col + 32 * j);
    for (int it = 0; t < a.T; t += stride, it ^= 1) {
        uint4 cur[3][2];
#pragma unroll
        for (int s = 0; s < 3; ++s)
#pragma unroll
            for (int j = 0; j < 2; ++j) cur[s][j] = next[s][j];
        fetch(t + stride);
        float dots[2] = {0.f, 0.f};  // x . gate_w, dout . y_sh
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float p[8], q[8];
            unpack8(cur[2][j], p);
            unpack8(w[j], q);
#pragma unroll
            for (int i = 0; i < 8; ++i) dots[0] = fmaf(p[i], q[i], dots[0]);
            unpack8(cur[0][j], p);
            unpack8(cur[1][j], q);
#pragma unroll
            for (int i = 0; i < 8; ++i) dots[1] = fmaf(p[i], q[i], dots[1]);
        }
        group_sums<2>(dots, red[it], gw, group * gw, warp, lane, sync);
        const float g = gate_of(dots[0]), dz = g * gate_of(-dots[0]) * dots[1];
        if (col == 0) a.dgate[t] = dz;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            if (!in[j]) continue;
            float d[8], x[8];
            unpack8(cur[0][j], d);
            unpack8(cur[2][j], x);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                d[i] *= g;
                sum[j][i] = fmaf(dz, x[i], sum[j][i]);
            }
            reinterpret_cast<uint4*>(a.dy_sh + t * a.H)[col + 32 * j] = pack8(d);
        }
    }
    if (!a.dgate_w) return;
    float4* const part = reinterpret_cast<float4*>(gridDim.x > 1 ? a.part + (int64_t)blockIdx.x * a.H : a.dgate_w);
    for (int g = 0; g < groups; ++g) {
        if (groups > 1) __syncthreads();
        if (g != group) continue;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            if (!in[j]) continue;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int at = 2 * (col + 32 * j) + h;
                float4 s = make_float4(sum[j][4 * h], sum[j][4 * h + 1], sum[j][4 * h + 2], sum[j][4 * h + 3]);
                if (g > 0) {
                    const float4 o = acc[at];
                    s.x += o.x; s.y += o.y; s.z += o.z; s.w += o.w;
                }
                (g + 1 < groups ? acc : part)[at] = s;
            }
        }
    }
}

// The same for any H, without the gate weight's gradient: a warp to a token, its rows read twice.  With
// the pairs' kernel, this and the weight's one behind the other, 2 pairs: 4096 tokens of 12288 197 us of 120.6
// at the copy rate, 2048 of 16384 184 of 80.4 (4096 of 8192 in gate_bwd_kernel 94.3 of 80.4).
__global__ void __launch_bounds__(FB_WARPS * 32) gate_rows_kernel(const __grid_constant__ FinalizeBwdLaunch a) {
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, vec = a.H / 8;
    for (int64_t t = (int64_t)blockIdx.x * FB_WARPS + warp; t < a.T; t += (int64_t)gridDim.x * FB_WARPS) {
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
        const float g = gate_of(z);
        if (lane == 0) a.dgate[t] = g * gate_of(-z) * dot;
        uint4* dysh = reinterpret_cast<uint4*>(a.dy_sh + t * a.H);
        for (int v = lane; v < vec; v += 32) {
            float d[8];
            unpack8(dout[v], d);
            for (int i = 0; i < 8; ++i) d[i] *= g;
            dysh[v] = pack8(d);
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

// A token's row is spread over `split` of a CTA's warps (1, 2, 4 or 8).  A warp first lists
// its token's pairs that have a row, then takes U vectors of 8 values a lane at a time, with
// PB_LOADS of the pairs' vectors in flight before they are used.  MAXK: k at most; DW: with
// the weights' gradients, a lane's share of every pair's dot product stays in a register.
// U and the registers (through CTAS CTAs of WARPS warps an SM) are those that measured best: enough
// loads in flight against enough warps.  16384 tokens of 2048, us: 4 pairs with DW 62.9 (U 2, 28
// warps an SM; 24 warps 66.5; U 1, 40 warps 66.9), without 50.8 (U 2, 24; U 1, 36 52.9); 2 pairs
// with DW 43.0 (U 2, 28; 32 46.5; U 1, 36 44.4); 8 pairs with DW 104 (U 1, 32; 36 over 110; U 2, 24
// 106.6), without 88.2 (U 2, 24; U 1, 32 90.6, but 4096 tokens 25.5 against 27.5).  With DW the forms of up
// to 4 and of up to 8 pairs spill for that, 16 to 64 bytes a thread; 24 warps are what spills nothing.
// More than 8 pairs: 4096 tokens of 2048, 16 pairs 46.1 without DW (42.7 at the copy rate), 58.9 with (45.3);
// 32 pairs 86.9 (82.9), 102.4 (85.6); 16384 tokens, 9 pairs 97.9 (100.5), 158 (110.7: the dots of 32 are joined).
constexpr int PB_LOADS = 8;

template <int MAXK, bool DW, int U, int CTAS, int WARPS>
__global__ void __launch_bounds__(WARPS * 32, CTAS) permute_bwd_kernel(const __grid_constant__ PermuteBwdLaunch a,
                                                                  int split) {
    constexpr int BATCH = PB_LOADS / U < MAXK ? PB_LOADS / U : MAXK;
    __shared__ int32_t s_row[FB_WARPS][MAXK], s_pair[FB_WARPS][MAXK];
    __shared__ float s_w[FB_WARPS][MAXK], s_dot[FB_WARPS][DW ? MAXK : 1];
    pdl_wait();
    pdl_trigger();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, vec = a.H / 8;
    const int part = warp & (split - 1), tokens = (blockDim.x >> 5) / split;
    for (int64_t t0 = (int64_t)blockIdx.x * tokens; t0 < a.T; t0 += (int64_t)gridDim.x * tokens) {
        const int64_t t = t0 + warp / split;
        const bool live_t = t < a.T;
        int32_t row = -1;
        float w = 1.f;
        if (live_t && lane < a.k) {
            row = pair_row_of(a.pair_row, t * a.k + lane, a.rows_cap, part == 0 ? &a.hdr->status : nullptr);
            if (a.w) w = a.w[t * a.k + lane];
        }
        const uint32_t live = __ballot_sync(0xffffffffu, row >= 0);
        const int n = __popc(live);
        __syncwarp();
        if (row >= 0) {
            const int i = __popc(live & ((1u << lane) - 1));
            s_row[warp][i] = row;
            s_w[warp][i] = w;
            s_pair[warp][i] = lane;
        }
        __syncwarp();
        float dot[DW ? MAXK : 1] = {};
        const float dz = live_t && a.dgate ? a.dgate[t] : 0.f;
        const int last = live_t ? vec : 0;
        for (int v0 = part * 32 * U + lane; v0 < last; v0 += split * 32 * U) {
            const auto in = [&](int u) { return u == 0 || v0 + 32 * u < vec; };
            const int64_t at = t * a.H + 8 * v0;
            uint4 xp[U];
            float acc[U][8] = {};
            if (DW) {
#pragma unroll
                for (int u = 0; u < U; ++u)  // not __ldg: dx may be x
                    xp[u] = in(u) ? reinterpret_cast<const uint4*>(a.x + at)[32 * u] : make_uint4(0, 0, 0, 0);
            }
            if (a.add) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    if (!in(u)) continue;
                    if (a.add_f32) {
                        const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(a.add) + at + 256 * u);
                        const float4 lo = q[0], hi = q[1];
                        acc[u][0] = lo.x; acc[u][1] = lo.y; acc[u][2] = lo.z; acc[u][3] = lo.w;
                        acc[u][4] = hi.x; acc[u][5] = hi.y; acc[u][6] = hi.z; acc[u][7] = hi.w;
                    } else {
                        unpack8(*reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.add) + at + 256 * u), acc[u]);
                    }
                }
            }
#pragma unroll
            for (int j0 = 0; j0 < MAXK; j0 += BATCH) {
                if (j0 >= n) break;
                uint4 ld[BATCH][U];
#pragma unroll
                for (int b = 0; b < BATCH; ++b) {
                    const bool ok = j0 + b < n;
                    const uint4* q = reinterpret_cast<const uint4*>(a.dx_perm + (ok ? (int64_t)s_row[warp][j0 + b] * a.H : 0)) + v0;
#pragma unroll
                    for (int u = 0; u < U; ++u) ld[b][u] = ok && in(u) ? __ldg(q + 32 * u) : make_uint4(0, 0, 0, 0);
                }
#pragma unroll
                for (int b = 0; b < BATCH; ++b) {
                    if (j0 + b >= n) continue;
                    const float wj = s_w[warp][j0 + b];
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        float d[8], x[8];
                        unpack8(ld[b][u], d);
                        if (DW) unpack8(xp[u], x);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            acc[u][i] = fmaf(wj, d[i], acc[u][i]);
                            if (DW) dot[DW ? j0 + b : 0] = fmaf(x[i], d[i], dot[DW ? j0 + b : 0]);
                        }
                    }
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                if (!in(u)) continue;
                if (a.dgate) {
                    float g[8];
                    unpack8(__ldg(reinterpret_cast<const uint4*>(a.gate_w) + v0 + 32 * u), g);
#pragma unroll
                    for (int i = 0; i < 8; ++i) acc[u][i] = fmaf(dz, g[i], acc[u][i]);
                }
                reinterpret_cast<uint4*>(a.dx + at)[32 * u] = pack8(acc[u]);
            }
        }
        if (DW) {
            float mine = lane_sums<DW ? MAXK : 1, false>(dot, lane);  // to lane j: the sum of pair j
            mine = __shfl_sync(0xffffffffu, mine, lane * (32 / MAXK) & 31);
            if (split > 1) {
                if (lane < n) s_dot[warp][lane] = mine;
                __syncthreads();
                if (part == 0 && lane < n)
                    for (int q = 1; q < split; ++q) mine += s_dot[warp + q][lane];
            }
            if (part == 0 && live_t) {
                if (lane < n) a.dw[t * a.k + s_pair[warp][lane]] = mine;
                if (lane < a.k && row < 0) a.dw[t * a.k + lane] = 0.f;
            }
            if (split > 1) __syncthreads();  // the next token's dots
        }
    }
}

}  // namespace

cudaError_t launch_finalize_bwd(const FinalizeBwdLaunch& given, int num_sms, cudaStream_t s) {
    FinalizeBwdLaunch L = given;
    L.gate_first = L.gate_w && L.H <= GB_MAX_H;
    int parts = 0;
    cudaError_t e;
    if (L.gate_first) {
        const int gw = (L.H + 511) / 512, groups = std::max(1, GB_CTA_WARPS / gw);
        // as many tokens as a CTA has groups go to one CTA, whose sums need no other kernel
        parts = L.T <= groups ? 1 : (int)std::min<int64_t>((L.T + groups - 1) / groups, std::min(num_sms, kBwdPartials));
        e = launch_k("gate_bwd", gate_bwd_kernel, dim3(parts), dim3(gw * groups * 32),
                     groups > 1 ? (size_t)L.H * 4 : 0, s, L, gw, groups);
        if (e != cudaSuccess) return e;
    }
    // CTAs of few warps leave less of an SM idle at the end (16384 pairs of 2048: 24.9 us with four
    // warps, 25.2 with eight)
    constexpr int WARPS = 4;
    const int pp = L.H <= 256 ? 4 : L.H <= 512 ? 2 : 1;
    const unsigned grid = (unsigned)std::min<int64_t>((L.T * L.k + WARPS * pp - 1) / (WARPS * pp), (int64_t)num_sms * 128);
    const auto kernel = pp == 4 ? finalize_bwd_kernel<4> : pp == 2 ? finalize_bwd_kernel<2> : finalize_bwd_kernel<1>;
    e = launch_k("finalize_bwd", kernel, dim3(grid), dim3(WARPS * 32), 0, s, L);
    if (e != cudaSuccess || !L.gate_w) return e;
    if (!L.gate_first) {
        const unsigned rows = (unsigned)std::min<int64_t>((L.T + FB_WARPS - 1) / FB_WARPS, (int64_t)num_sms * 64);
        e = launch_k("gate_rows_bwd", gate_rows_kernel, dim3(rows), dim3(FB_WARPS * 32), 0, s, L);
        if (e != cudaSuccess || !L.dgate_w) return e;
        parts = (int)std::min<int64_t>(L.T, kBwdPartials);
        e = launch_k("gate_weight_bwd", gate_weight_kernel,
                     dim3((L.H / 8 + FB_WARPS * 32 - 1) / (FB_WARPS * 32), parts), dim3(FB_WARPS * 32), 0, s, L.dgate,
                     L.x, L.T, L.H, L.part);
    }
    if (e != cudaSuccess || !L.dgate_w || (L.gate_first && parts == 1)) return e;
    return launch_sum_partials(L.part, parts, L.H, L.H, L.dgate_w, nullptr, s);
}

cudaError_t launch_permute_bwd(const PermuteBwdLaunch& L, int num_sms, cudaStream_t s) {
    // A row over as many warps as give every SM a CTA, and where a warp keeps five vectors a lane
    // of it, as many as give every SM eight: shorter last waves (4096 tokens of 7168, 8 pairs: 106
    // us in four parts, 108 in one; without the weights' gradients 81 and 98).
    int split = 1;
    while (split < FB_WARPS && (L.T * split < (int64_t)num_sms * FB_WARPS ||
                                (L.T * split < 8LL * num_sms * FB_WARPS && L.H / 8 >= 2 * split * 5 * 32)))
        split *= 2;
    const int warps = std::max(split, 2), tokens = warps / split;  // few warps: less of an SM idle at the end
    const unsigned grid = (unsigned)std::min<int64_t>((L.T + tokens - 1) / tokens, (int64_t)num_sms * 128);
    const auto go = [&](auto kernel) {
        return launch_k("permute_bwd", kernel, dim3(grid), dim3(warps * 32), 0, s, L, split);
    };
    if (L.k > 8) return L.dw ? go(permute_bwd_kernel<32, true, 1, 2, 8>) : go(permute_bwd_kernel<32, false, 2, 3, 8>);
    if (warps > 2) {  // a token over four or eight warps
        if (L.k <= 2) return L.dw ? go(permute_bwd_kernel<2, true, 2, 4, 8>) : go(permute_bwd_kernel<2, false, 2, 4, 8>);
        if (L.k <= 4) return L.dw ? go(permute_bwd_kernel<4, true, 1, 5, 8>) : go(permute_bwd_kernel<4, false, 1, 5, 8>);
        return L.dw ? go(permute_bwd_kernel<8, true, 1, 4, 8>) : go(permute_bwd_kernel<8, false, 2, 3, 8>);
    }
    if (L.k <= 2) return L.dw ? go(permute_bwd_kernel<2, true, 2, 14, 2>) : go(permute_bwd_kernel<2, false, 2, 16, 2>);
    if (L.k <= 4) return L.dw ? go(permute_bwd_kernel<4, true, 2, 14, 2>) : go(permute_bwd_kernel<4, false, 2, 12, 2>);
    if (L.dw || L.T < 40LL * num_sms)
        return L.dw ? go(permute_bwd_kernel<8, true, 1, 16, 2>) : go(permute_bwd_kernel<8, false, 1, 16, 2>);
    return go(permute_bwd_kernel<8, false, 2, 12, 2>);
}

}  // namespace moe

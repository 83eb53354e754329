// moe_norm_bwd.cu -- the gradients of the two norms in front of an MoE block, and the
// column sums that weight gradients are.  Per row r of H values, with g = dy * weight,
// d = r - mean (layer norm) or r (RMS norm) and rstd = 1 / sqrt(sum(d^2) / H + eps):
//
//   dr = dstream + rstd * (g - [layer norm: sum(g) / H] - d * rstd^2 * sum(g d) / H)
//   dweight = sum over rows of dy * d * rstd,  dbias = sum over rows of dy
//
// The row's statistics are taken again from r: the row has to be read for d anyway.  (A bf16 stream
// holds r rounded: the gradient is taken there, where the forward normalised the unrounded sum.)
// All sums are binary32; dr is rounded once for each of its outputs.
//
// Bound: HBM (8 bytes an element with a bf16 stream and its gradient) and not far behind it
// the issue rate: 21 instructions an element in all (RMS, bf16), a third of them conversions, a
// third what a row costs beside its elements.  So the arithmetic is done on pairs (f32x2) and
// every address of a row is a base and a constant.  A row belongs to a group of warps, each
// thread to the same columns of every row of its group, so the weight's sums stay in registers
// to the end of a persistent grid; a CTA's groups then add theirs in order, and a second kernel
// adds the CTAs'.  A thread copies its own columns of the rows to come into shared memory
// (cp.async): the copies need no barrier, and a row's one barrier joins its warps' sums.
//
// The layer norm's row needs its mean before its squares, or a row far from zero loses its
// variance.  A warp takes the mean c of its own n columns and sums about that; with e = c - c0, c0
// the first warp's c, and sd the warp's sum of r - c, what the roundings of c left over, the row's
// sums are
//
//   m = sum(n e + sd) / H  (the row's mean is c0 + m),  sum(d^2) = sum(ss + e (n e + 2 sd)) - H m^2,
//   sum(g d) = sum(sgd + e sg) - m sum(sg)
//
// where H m^2 is at most H / n of the result, 16, whatever c0 is: one barrier instead of two
// (28672 rows of 2048, bf16, 85 -> 79 us).  1 / sqrt(eps) would carry sd into
// rows of little variance: an fp32 stream takes it along (without it an fp32 row of 100.3 had
// normalised values of 0.002 in place of 0).  A bf16 stream needs it not: where values of 8 bits lie
// close enough together for their rounding to matter, their binary32 sum is exact, and the quotient
// is rounded once.
//
// Narrow rows keep r, dy and the weight in registers from one pass to the next; rows of more
// columns a thread read them again (the weight from shared memory, in binary32).
//
// 16384 rows of 7168 with a stream's gradient: RMS, bf16 139 us, 6.8 TB/s, 1.01 of this card's
// copy rate, layer norm 156 us, 0.90; 8192 rows, fp32: 123 us, 1.0, and 124 us.  4096 of 2048,
// fp32, layer norm 26.5 us, 0.76; 777 of 1408, bf16 7.3 us, of which the second kernel 3.5.  The
// layer norm's bf16 rows issue 29 to 30 instructions an element in 50 to 57 % of their cycles: their
// 14 to 16 warps an SM wait for shared memory and for their own latency, no pipe is full.
#include <algorithm>
#include <atomic>

#include "moe_internal.cuh"
#include "moe_rows.cuh"

namespace moe {
namespace {

constexpr int NB_WARPS = 16;           // warps of a CTA at most, one CTA an SM
constexpr int NB_SMEM = 227 * 1024 - 1024;  // of a CTA, less the static arrays

// What a kernel keeps: the row's r, dy and the weight in registers from one pass to the next, or
// the weight in shared memory in binary32 (NB_SHARED_R: and r in registers; NB_SHARED_DS: the ring
// has no room for dstream), or nothing (and no room for dstream).
enum { NB_REGISTERS, NB_SHARED, NB_SHARED_R, NB_SHARED_DS, NB_NOTHING };
// Warps of a CTA that leave NB_SHARED_R its registers.  Layer norm, bf16, 9600 rows of 6144 80 us, 91
// with r read again; 5000 of 12288 87 / 100.
constexpr int NB_R_WARPS = 12;

struct NormBwdPlan {
    int gw, groups, slots;   // warps of a group, groups of a CTA, rows that a group's ring holds
    float* out;              // a CTA's column sums: CTA i's of dweight at i * out_stride, of dbias
    int64_t out_stride, out_bias;  // out_bias behind
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void cp_async_wait_upto(int n) {  // n uniform, at most 3
    if (n == 0) cp_async_wait<0>();
    else if (n == 1) cp_async_wait<1>();
    else if (n == 2) cp_async_wait<2>();
    else cp_async_wait<3>();
}

// C values: a piece of a bf16 row (C = 8: 16 bytes, C = 4: 8 bytes) or of an fp32 one (C = 4).
template <int C>
__device__ __forceinline__ void nb_bf16(const void* p, f2 f[C / 2]) {
    if (C == 8) {
        const uint4 v = *static_cast<const uint4*>(p);
        f[0] = f2_bf16(v.x); f[1] = f2_bf16(v.y); f[C / 2 - 2] = f2_bf16(v.z); f[C / 2 - 1] = f2_bf16(v.w);
    } else {
        const uint2 v = *static_cast<const uint2*>(p);
        f[0] = f2_bf16(v.x); f[1] = f2_bf16(v.y);
    }
}
__device__ __forceinline__ void nb_f32(const void* p, f2 f[2]) {
    const uint4 v = *static_cast<const uint4*>(p);
    f[0] = f2_make(__uint_as_float(v.x), __uint_as_float(v.y));
    f[1] = f2_make(__uint_as_float(v.z), __uint_as_float(v.w));
}
template <bool F32>
__device__ __forceinline__ void nb_stream(const void* p, f2 f[F32 ? 2 : 4]) {
    if (F32) nb_f32(p, f);
    else nb_bf16<8>(p, f);
}
template <int C>
__device__ __forceinline__ void nb_put_bf16(void* p, const f2 f[C / 2]) {
    uint32_t w[C / 2];
#pragma unroll
    for (int i = 0; i < C / 2; ++i) {
        float lo, hi;
        f2_split(f[i], lo, hi);
        w[i] = pack_bf16x2(lo, hi);
    }
    if (C == 8) *static_cast<uint4*>(p) = make_uint4(w[0], w[1], w[C / 2 - 2], w[C / 2 - 1]);
    else *static_cast<uint2*>(p) = make_uint2(w[0], w[1]);
}
__device__ __forceinline__ void nb_put_f32(void* p, const f2 f[2]) {
    float v[4];
    f2_split(f[0], v[0], v[1]);
    f2_split(f[1], v[2], v[3]);
    *static_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
}

// NP pieces a thread: 8 columns of a bf16 stream, or 4 of an fp32 one (16 bytes either way, so
// that a warp's copies and stores cover whole lines).  A warp's pieces lie side by side.
template <int NP, bool F32, bool LN, int KEEP>
__global__ void __launch_bounds__((KEEP == NB_SHARED_R ? NB_R_WARPS : NB_WARPS) * 32, 1)
    norm_bwd_kernel(const __grid_constant__ NormBwdLaunch a, const __grid_constant__ NormBwdPlan p) {
    extern __shared__ uint4 smem[];  // [NB_SHARED: gw * NP pieces of weight], [warp][slot] r, dy, dstream
    constexpr bool HOLD = KEEP == NB_REGISTERS, W_SMEM = !HOLD && KEEP != NB_NOTHING;
    constexpr bool HOLD_R = HOLD || KEEP == NB_SHARED_R, DS_RING = KEEP != NB_SHARED_DS && KEEP != NB_NOTHING;
    constexpr int DB = LN ? 2 : 4;                               // as many as leave the sums their registers
    constexpr int C = F32 ? 4 : 8, P = C / 2, SB = F32 ? 4 : 2;  // columns, pairs of a piece; bytes of a stream value
    constexpr int NS = LN ? 4 : 2;                               // a row's sums: d^2, g d (and g, d or c)
    constexpr int DY = NP * 512, DS = DY + NP * 64 * C;          // a slot's dy and dstream
    __shared__ alignas(16) float red[2][NB_WARPS * NS];
    constexpr bool SD = LN && F32;                               // the deviations' sum is one of the four
    __shared__ float near[2][SD ? NB_WARPS : 1];                 // and c stands here
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int group = warp / p.gw, gwarp = warp - group * p.gw;
    const int slot_bytes = DS + (DS_RING && a.dstream ? NP * 512 : 0);
    const int col = (gwarp * NP * 32 + lane) * C;                // of piece 0; piece k: + k * 32 * C
    uint32_t valid = 0;
#pragma unroll
    for (int k = 0; k < NP; ++k) valid |= (uint32_t)(col + k * 32 * C < a.H) << k;
    // dy is copied 8 columns a lane whatever a piece holds: with an fp32 stream a lane uses what
    // others copied, which the warp's barriers below are for
    constexpr int DYC = NP * C / 8;
    const int dy_col = gwarp * NP * 32 * C + lane * 8;
    uint32_t dy_valid = 0;
#pragma unroll
    for (int k = 0; k < DYC; ++k) dy_valid |= (uint32_t)(dy_col + k * 256 < a.H) << k;
    const float inv_h = 1.f / (float)a.H;
    const auto columns = [&](int w) { return (float)max(0, min(a.H - w * NP * 32 * C, NP * 32 * C)); };  // of warp w
    const float n = columns(gwarp), inv_n = 1.f / n;
    const int64_t stride = (int64_t)gridDim.x * p.groups;
    const int64_t first = (int64_t)group * gridDim.x + blockIdx.x;
    const auto group_sync = [&] { asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(p.gw * 32) : "memory"); };
    char* const weights = reinterpret_cast<char*>(smem) + (gwarp * NP * P * 16 + lane) * 16;
    char* const ring = reinterpret_cast<char*>(smem) + (W_SMEM ? p.gw * NP * 128 * C : 0) + warp * p.slots * slot_bytes;

    f2 dw[NP][P] = {}, db[LN ? NP : 1][P] = {};
    pdl_wait();
    pdl_trigger();
    const auto fetch = [&](int64_t row, int at) {
        if (row < a.T) {
            const uint32_t s = smem_u32(ring) + at;
            const char* r = static_cast<const char*>(a.r) + (row * a.H + col) * SB;
            const char* dy = reinterpret_cast<const char*>(a.dy + row * a.H + dy_col);
            const char* ds = static_cast<const char*>(a.dstream) + (row * a.H + col) * SB;
#pragma unroll
            for (int k = 0; k < NP; ++k) {
                if (!(valid >> k & 1)) continue;
                cp_async16(s + lane * 16 + k * 512, r + k * 512);
                if (DS_RING && a.dstream) cp_async16(s + lane * 16 + DS + k * 512, ds + k * 512);
                if (!DS_RING && a.dstream && lane % 8 == 0)  // 6000 rows of 9728, layer norm: 198 -> 154 us
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(ds + k * 512));
            }
#pragma unroll
            for (int k = 0; k < DYC; ++k)
                if (dy_valid >> k & 1) cp_async16(s + lane * 16 + DY + k * 512, dy + k * 512);
        }
        cp_async_commit();
    };
    for (int s = 0; s < p.slots; ++s) fetch(first + s * stride, s * slot_bytes);
    f2 held_w[HOLD ? NP : 1][P] = {};
    if (HOLD || (W_SMEM && group == 0)) {
#pragma unroll
        for (int k = 0; k < NP; ++k) {
            f2 w[P] = {};
            if (valid >> k & 1) nb_bf16<C>(a.weight + col + k * 32 * C, w);
#pragma unroll
            for (int i = 0; i < P; ++i)
                if (HOLD) held_w[HOLD ? k : 0][i] = w[i];
                else if (i % 2 == 0) nb_put_f32(weights + (k * (P / 2) + i / 2) * 512, w + i);
        }
    }
    if (W_SMEM) __syncthreads();
    const auto read_weight = [&](int k, f2 w[P]) {
        if (W_SMEM) {
#pragma unroll
            for (int i = 0; i < P / 2; ++i) nb_f32(weights + (k * (P / 2) + i) * 512, w + 2 * i);
        } else {
            nb_bf16<C>(a.weight + col + k * 32 * C, w);
        }
    };
    int at = 0, it = 0;
    for (int64_t row = first; row < a.T; row += stride, it ^= 1) {
        cp_async_wait_upto(p.slots - 1);
        if (F32) __syncwarp();
        const char* slot = ring + at;
        f2 r[NP][P], g[NP][P];  // NB_REGISTERS: kept from one pass to the next
        float mean = 0.f;       // c, of the warp's columns
        if (LN) {
            f2 sum = 0;
#pragma unroll
            for (int k = 0; k < NP; ++k) {
                if (!(valid >> k & 1)) continue;
                nb_stream<F32>(slot + lane * 16 + k * 512, r[k]);
#pragma unroll
                for (int i = 0; i < P; ++i) sum = f2_add(sum, r[k][i]);
            }
            const float total = warp_sum(f2_sum(sum));
            mean = total * inv_n;
            if (SD) {
                if (lane == 0) near[it][SD ? warp : 0] = mean;
            } else {
                mean = fmaf(fmaf(-mean, n, total), inv_n, mean);
            }
        }
        const f2 off = f2_make(-mean, -mean);
        f2 ss = 0, sg = 0, sgd = 0, sd = 0;
#pragma unroll
        for (int k = 0; k < NP; ++k) {
            if (!(valid >> k & 1)) continue;
            f2 w[P];
            if (!LN || !HOLD_R) nb_stream<F32>(slot + lane * 16 + k * 512, r[k]);
            nb_bf16<C>(slot + lane * 2 * C + DY + k * 64 * C, g[k]);
            if (!HOLD) read_weight(k, w);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                if (LN) r[k][i] = f2_add(r[k][i], off);
                const f2 gw = f2_mul(g[k][i], HOLD ? held_w[HOLD ? k : 0][i] : w[i]);
                ss = f2_fma(r[k][i], r[k][i], ss);
                sgd = f2_fma(gw, r[k][i], sgd);
                if (LN) {
                    sg = f2_add(sg, gw);
                    if (SD) sd = f2_add(sd, r[k][i]);
                }
            }
        }
        float sums[NS] = {};
        sums[0] = f2_sum(ss);
        sums[1] = f2_sum(sgd);
        float e = 0.f;  // the warp's c less the row's mean: d = r - c + e
        if constexpr (LN) {
            sums[NS - 2] = f2_sum(sg);
            sums[NS - 1] = SD ? f2_sum(sd) : lane == 0 && p.gw > 1 ? mean : 0.f;
            float first_c = mean;
            const auto join = [&](float (&v)[NS], int w, const float* q) {
                const float* const c = near[it] + (SD ? group * p.gw : 0);
                first_c = SD ? c[0] : q[NS - 1];
                const float n = columns(w), ew = (SD ? c[w < p.gw ? w : 0] : v[NS - 1]) - first_c;
                const float left = SD ? v[NS - 1] : 0.f;
                v[0] = fmaf(ew, fmaf(n, ew, 2.f * left), v[0]);
                v[1] = fmaf(ew, v[NS - 2], v[1]);
                v[NS - 1] = fmaf(n, ew, left);
            };
            group_sums<NS>(sums, red[it], p.gw, group * p.gw, warp, lane, group_sync, join);
            const float m = sums[NS - 1] * inv_h;  // the row's mean less the first warp's c
            e = (mean - first_c) - m;
            sums[0] = fmaf(-m, sums[NS - 1], sums[0]);
            if (sums[0] < 0.f) sums[0] = 0.f;  // NaN stays
            sums[1] = fmaf(-m, sums[NS - 2], sums[1]);
        } else {
            group_sums<NS>(sums, red[it], p.gw, group * p.gw, warp, lane, group_sync);
        }
        const float rstd = rsqrtf(fmaf(sums[0], inv_h, a.eps));
        const float mgd = -rstd * rstd * (sums[1] * inv_h), mg = LN ? fmaf(e, mgd, -sums[NS - 2] * inv_h) : 0.f;
        const f2 e_rstd2 = f2_make(e * rstd, e * rstd);
        const f2 rstd2 = f2_make(rstd, rstd), mg2 = f2_make(mg, mg), mgd2 = f2_make(mgd, mgd);
        const int64_t out = row * a.H + col;
        uint4 ds[DB];  // not DS_RING: so many pieces of dstream in flight
#pragma unroll
        for (int k = 0; k < NP; ++k) {
            if (!DS_RING && k % DB == 0 && a.dstream)
#pragma unroll
                for (int b = 0; b < DB; ++b)
                    if (valid >> (k + b) & 1)
                        ds[b] = *reinterpret_cast<const uint4*>(static_cast<const char*>(a.dstream) + out * SB +
                                                                (k + b) * 512);
            if (!(valid >> k & 1)) continue;
            f2 w[P], o[P] = {};
            if (!HOLD_R) nb_stream<F32>(slot + lane * 16 + k * 512, r[k]);
            if (!HOLD) {
                nb_bf16<C>(slot + lane * 2 * C + DY + k * 64 * C, g[k]);
                read_weight(k, w);
            }
            if (DS_RING && a.dstream) nb_stream<F32>(slot + lane * 16 + DS + k * 512, o);
            else if (!DS_RING && a.dstream) nb_stream<F32>(&ds[k % DB], o);
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const f2 wi = HOLD ? held_w[HOLD ? k : 0][i] : w[i];
                const f2 d = LN && !HOLD_R ? f2_add(r[k][i], off) : r[k][i];
                dw[k][i] = f2_fma(g[k][i], LN ? f2_fma(d, rstd2, e_rstd2) : f2_mul(d, rstd2), dw[k][i]);
                if (LN) db[LN ? k : 0][i] = f2_add(db[LN ? k : 0][i], g[k][i]);
                const f2 gw = LN ? f2_fma(g[k][i], wi, mg2) : f2_mul(g[k][i], wi);
                o[i] = f2_fma(rstd2, f2_fma(d, mgd2, gw), o[i]);
            }
            if (a.dr) {
                if (F32) nb_put_f32(static_cast<float*>(a.dr) + out + k * 32 * C, o);
                else nb_put_bf16<C>(static_cast<uint16_t*>(a.dr) + out + k * 32 * C, o);
            }
            if (a.dx) nb_put_bf16<C>(a.dx + out + k * 32 * C, o);
        }
        if (F32) __syncwarp();
        fetch(row + p.slots * stride, at);
        at += slot_bytes;
        if (at == p.slots * slot_bytes) at = 0;
    }
    cp_async_wait<0>();
    if (!a.dweight && !a.dbias) return;
    // the groups' sums, one group behind the other, in the ring's memory
    float* out = p.out + (int64_t)blockIdx.x * p.out_stride;
    float* acc = reinterpret_cast<float*>(smem);
    for (int g = 0; g < p.groups; ++g) {
        if (p.groups > 1) __syncthreads();
        if (g != group) continue;
        float* const to = g + 1 < p.groups ? acc : out;
        const int64_t to_bias = g + 1 < p.groups ? a.H : p.out_bias;
#pragma unroll
        for (int k = 0; k < NP; ++k) {
            if (!(valid >> k & 1)) continue;
#pragma unroll
            for (int b = 0; b < (LN ? 2 : 1); ++b) {
                f2* s = b ? db[LN ? k : 0] : dw[k];
                const int c = col + k * 32 * C;
#pragma unroll
                for (int i = 0; i < P; i += 2) {
                    if (g > 0) {
                        f2 o[2];
                        nb_f32(acc + b * a.H + c + 2 * i, o);
                        s[i] = f2_add(o[0], s[i]);
                        s[i + 1] = f2_add(o[1], s[i + 1]);
                    }
                    nb_put_f32(to + b * to_bias + c + 2 * i, s + i);
                }
            }
        }
    }
}

// A CTA adds 4 * SP_QUADS columns: a thread takes 4 columns of the partial rows l, l + SP_LANES,
// ..., SP_BATCH of them in flight (so that 152 rows are one round), then the lanes' sums are added
// in order.
constexpr int SP_QUADS = 16, SP_LANES = 16, SP_BATCH = 10;

__global__ void __launch_bounds__(SP_QUADS * SP_LANES) sum_partials_kernel(const float* part, int n, int64_t stride,
                                                                         int H, float* out0, float* out1) {
    __shared__ float red[SP_LANES][SP_QUADS * 4];
    const int quad = threadIdx.x % SP_QUADS, lane = threadIdx.x / SP_QUADS;
    const int first = blockIdx.x * SP_QUADS * 4, col = first + 4 * quad;
    float* out = blockIdx.y ? out1 : out0;
    pdl_wait();
    pdl_trigger();
    if (!out) return;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (col < H) {
        const float* p = part + (int64_t)blockIdx.y * H + col;
        for (int i0 = lane; i0 < n; i0 += SP_LANES * SP_BATCH) {
            float4 v[SP_BATCH];
#pragma unroll
            for (int b = 0; b < SP_BATCH; ++b) {
                const int i = i0 + SP_LANES * b;
                v[b] = i < n ? *reinterpret_cast<const float4*>(p + i * stride) : make_float4(0.f, 0.f, 0.f, 0.f);
            }
#pragma unroll
            for (int b = 0; b < SP_BATCH; ++b) {
                s.x += v[b].x; s.y += v[b].y; s.z += v[b].z; s.w += v[b].w;
            }
        }
    }
    *reinterpret_cast<float4*>(&red[lane][4 * quad]) = s;
    __syncthreads();
    if (threadIdx.x < SP_QUADS * 4 && first + threadIdx.x < H) {
        float t = 0.f;
#pragma unroll
        for (int l = 0; l < SP_LANES; ++l) t += red[l][threadIdx.x];
        out[first + threadIdx.x] = t;
    }
}

template <int NP, bool F32, bool LN, int KEEP>
cudaError_t launch_norm_bwd_kernel(const NormBwdLaunch& L, const NormBwdPlan& p, int grid, bool one, size_t smem,
                                   cudaStream_t s) {
    const auto kernel = norm_bwd_kernel<NP, F32, LN, KEEP>;
    static std::atomic<bool> granted[64];  // per device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64 || !granted[dev].load()) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)NB_SMEM);
        if (e != cudaSuccess) return e;
        if (dev >= 0 && dev < 64) granted[dev].store(true);
    }
    e = launch_k(LN ? "layernorm_bwd" : "rmsnorm_bwd", kernel, dim3(grid), dim3(p.gw * p.groups * 32), smem, s, L, p);
    if (e != cudaSuccess || one || (!L.dweight && !L.dbias)) return e;
    return launch_sum_partials(L.part, grid, 2 * (int64_t)L.H, L.H, L.dweight, L.dbias, s);
}

template <bool F32, bool LN>
cudaError_t launch_norm_bwd_type(const NormBwdLaunch& L, int num_sms, cudaStream_t s) {
    // 16 columns a thread, or 32: those share what a row costs beside its elements among more of
    // them and let more groups of warps work on a CTA's rows, where groups of 16 columns leave many
    // of the 16 warps idle.  The choice decides the order of a row's sums, so it does not depend on T.
    // us with 16 / 32, 58.7 M elements and dstream:
    // bf16, RMS: 4096 77 / 78, 5120 84 / 80 (10 warps / 15), 7168 76 / 78.
    // bf16, layer norm: 2560 82 / 86, 2816 96 / 82, 3584 89 / 84, 4096 81 / 83, 4608 114 / 83, 5632 97 / 85,
    // 6656 97 / 90, 7168 92 / 86, 8192 83 / 86; but 777 rows of 2816 10.4 / 13.9, 4608 14.2 / 16.1, 7168
    // 19.0 / 20.4.
    // fp32, layer norm, 29.4 M elements: with dstream 7 and 8 warps of 16 columns have room for one
    // group in the ring below, 32 columns for two of half the warps: 2560 70 / 94, 2816 68 / 87, 3136 94 /
    // 82, 3584 84 / 74, 4096 77 / 69, 4608 76 / 98, 5632 69 / 88, 7168 67 / 74, 8192 68 / 72; without it, by the
    // idle warps: 2560 55 / 57, 2816 61 / 56, 3584 57 / 58, 4096 54 / 55, 4608 72 / 60, 5632 63 / 56, 6144 59 /
    // 54, 6656 63 / 76, 7168 59 / 71.
    const int narrow = (L.H + 511) / 512;  // warps of a group, 16 columns a thread
    const int idle = narrow > NB_WARPS ? NB_WARPS : NB_WARPS % narrow;
    const bool wide = !LN ? (F32 ? L.H > 6144 : idle > 2)
                      : !F32 ? idle > 1
                             : narrow > NB_WARPS || (L.dstream ? narrow == 7 || narrow == 8 : idle > 3);
    const int columns = wide ? 32 : 16;
    NormBwdPlan p;
    p.gw = (L.H + columns * 32 - 1) / (columns * 32);
    const size_t stream = (size_t)p.gw * 32 * columns * (F32 ? 4 : 2), weight = wide ? (size_t)p.gw * 128 * columns : 0;
    const size_t slot = stream + (size_t)p.gw * 64 * columns;  // a row of a group, without dstream
    // dstream stays out of the ring where that leaves no room for two rows and the weight
    const bool ds_out = L.dstream && weight + 2 * (slot + stream) > NB_SMEM;
    const size_t row = slot + (L.dstream && !ds_out ? stream : 0);
    // Few rows an SM want fewer groups than a long run of them: a start of fewer copies and fewer
    // sums to add at the end, and no SM without rows.  12 warps instead of 16 (RMS: always), us:
    // bf16, RMS 4096 rows of 2048 16.6 / 18.1, 8192 of 1024 16.9 / 18.7; layer norm 4096 of 2048
    // 20.1 / 21.7, but 28672 99 / 86.
    const bool few = L.T * narrow < 160LL * num_sms;
    p.groups = (!wide && p.gw <= 4 && (!LN || few || (F32 && p.gw == 1)) ? 12 : NB_WARPS) / p.gw;
    const int64_t rows = (L.T + num_sms - 1) / num_sms;  // of an SM
    // bf16, layer norm, 32 columns: a group for every six rows.  us with 1 / 2 / 3 / 5 groups: 300 rows of
    // 4608 9.5 / 12.5, of 7168 12.8 / 14.7; 777 of 2816 13.9 / 11.9 / 12.9 / 14.8; 2048 of 2816 25.6 / 19.1 / 20.0 /
    // 20.0, of 3584 26.4 / 22.1 / 20.9 / 24.1; 6000 of 2816 63.2 / 40.8 / 36.6 / 33.3.
    if (LN && !F32 && wide) p.groups = (int)std::max<int64_t>(1, std::min<int64_t>(p.groups, (rows + 2) / 6));
    // An fp32 stream's rows on their way: with too many the memory slows down.  us of 123 at the
    // copy rate, groups x rows of each: RMS 28672 rows of 2048 3 x 2 122, 4 x 2 153; 22937 of 2560 1 x 2
    // 154, 2 x 3 129; layer norm 57344 of 1024 6 x 2 125, 4 x 3 129, 22937 of 2560 2 x 2 127, 2 x 3 122;
    // 9600 of 6144 1 x 2 124, 1 x 3 132.  Without dstream, of 88: RMS 2048 3 x 2 91, 3 x 3 103, 5120 1 x 2
    // 100, 1 x 3 89; layer norm 2048 4 x 2 93, 4 x 3 100, 8192 1 x 2 97, 1 x 3 93.
    int most = 3;
    if (F32) {
        const size_t ring = (LN ? 160 : L.dstream && p.gw > 1 ? 120 : 96) * 1024, start = LN && !wide ? 120 * 1024 : ring;
        p.groups = std::max(1, std::min(p.groups, (int)(start / (2 * row))));
        most = LN && p.groups > 3 ? 2 : (int)std::min<size_t>(3, std::max<size_t>(2, ring / (p.groups * row)));
    }
    // As many rows as one CTA has groups go to one CTA, whose sums need no second kernel (4 rows of
    // 512, layer norm 3.6 us against 4.4 on the GPU, and a launch less for the host).
    const bool one = L.T <= p.groups && L.dweight && (!LN || L.dbias);
    p.groups = (int)std::min<int64_t>(p.groups, one ? L.T : rows);
    const int grid = one ? 1 : (int)std::min<int64_t>((L.T + p.groups - 1) / p.groups, std::min(num_sms, kBwdPartials));
    p.out = one ? L.dweight : L.part;
    p.out_bias = one ? (int64_t)(reinterpret_cast<intptr_t>(L.dbias) - reinterpret_cast<intptr_t>(L.dweight)) / 4 : L.H;
    p.out_stride = 2 * (int64_t)L.H;
    const bool w_smem = wide && (!F32 || weight + 2 * row <= NB_SMEM);
    const size_t below = w_smem ? weight : 0;
    p.slots = (int)std::min<size_t>(most, (NB_SMEM - below) / (p.groups * row));
    const size_t smem = std::max(below + p.groups * p.slots * row, (size_t)8 * L.H);  // the groups' sums take 8 * H
    constexpr int NP = F32 ? 4 : 2;
    if (!wide) return launch_norm_bwd_kernel<NP, F32, LN, NB_REGISTERS>(L, p, grid, one, smem, s);
    if constexpr (F32)
        if (!w_smem) return launch_norm_bwd_kernel<2 * NP, F32, LN, NB_NOTHING>(L, p, grid, one, smem, s);
    if (ds_out) return launch_norm_bwd_kernel<2 * NP, F32, LN, NB_SHARED_DS>(L, p, grid, one, smem, s);
    if constexpr (LN && !F32)
        if (p.gw * p.groups <= NB_R_WARPS)
            return launch_norm_bwd_kernel<2 * NP, F32, LN, NB_SHARED_R>(L, p, grid, one, smem, s);
    return launch_norm_bwd_kernel<2 * NP, F32, LN, NB_SHARED>(L, p, grid, one, smem, s);
}

}  // namespace

cudaError_t launch_sum_partials(const float* part, int n, int64_t stride, int H, float* out0, float* out1,
                                cudaStream_t s) {
    return launch_k("sum_partials", sum_partials_kernel, dim3((H + 4 * SP_QUADS - 1) / (4 * SP_QUADS), out1 ? 2 : 1),
                    dim3(SP_QUADS * SP_LANES), 0, s,
                    part, n, stride, H, out0, out1);
}

cudaError_t launch_norm_bwd(const NormBwdLaunch& L, int num_sms, cudaStream_t s) {
    if (L.f32) return L.ln ? launch_norm_bwd_type<true, true>(L, num_sms, s) : launch_norm_bwd_type<true, false>(L, num_sms, s);
    return L.ln ? launch_norm_bwd_type<false, true>(L, num_sms, s) : launch_norm_bwd_type<false, false>(L, num_sms, s);
}

}  // namespace moe

// moe_w4.cu -- products of a few activation rows with 4-bit weights that carry one
// bf16 scale per group of consecutive elements of a row:
//
//   W[n][k] = s[n][k / group] * c[n][k],  c in -8 .. 7,   y[m][n] = sum_k x[m][k] W[n][k]
//
// as one matrix (moe_matvec_w4) and as the experts of an MoE layer at decode
// (moe_forward_w4: FC1 + SwiGLU, FC2, weighted combine, an optional shared expert).
//
// Packing: eight consecutive elements of a row share a 32-bit word (little-endian),
// element 2i in nibble i and element 2i + 1 in nibble i + 4, each as c + 8: a mask
// leaves elements 2i and 2i + 1 in the two 16-bit halves, in the order in which the
// activations lie in memory.
#include <algorithm>
#include <atomic>
#include <cmath>

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
// Products on mma.sync: a warp owns 32 weight rows (FC1: 16 gate and the matching
// 16 up rows) times up to 8 C activation rows
// ---------------------------------------------------------------------------
constexpr int W4_THREADS = 256;
constexpr int W4_WARPS = W4_THREADS / 32;
constexpr int W4_RING = 4;           // stages of 128 elements x 32 rows in each warp's ring
constexpr int W4_STAGE = 2048;       // bytes of a stage
constexpr int W4_MAXG = 1024;        // slots

__host__ __device__ constexpr size_t w4_smem_bytes(int C) {
    // ring of every warp, then two buffers of 32 x 8 C partial sums per warp
    return (size_t)W4_WARPS * (W4_RING * W4_STAGE + 2 * 32 * 8 * C * 4);
}

__device__ __forceinline__ void w4_cp16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void w4_cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void w4_cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// n consecutive words of shared memory
template <int n>
__device__ __forceinline__ void w4_lds(uint32_t (&v)[n], uint32_t addr) {
    if constexpr (n == 4)
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                     : "r"(addr)
                     : "memory");
    else if constexpr (n == 2)
        asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v[0]), "=r"(v[1]) : "r"(addr) : "memory");
    else
        asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v[0]) : "r"(addr) : "memory");
}

// D += A B (first: D = A B), A 16 x 16 (row), B 16 x 8 (column), bf16 inputs, fp32 sums
__device__ __forceinline__ void w4_mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void w4_mma_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}

// Elements 2j and 2j + 1 of a packed word as bf16 c / 64.  With a nibble n = c + 8 at
// bits 0-3 or 4-7 of a half, the half read as bf16 is n 2^-133 or n 2^-129: exponent
// fields 0 and 1 are one linear range (the lower one subnormal).  One fused
// multiply-add brings it to n / 64 - 8 / 64, exactly, on the FMA pipe; the ALU pipe,
// which the masks keep busiest, has five instructions a word.
__device__ __forceinline__ uint32_t w4_pair(uint32_t word, int j) {
    const uint32_t n = (j & 2 ? word >> 8 : word) & (j & 1 ? 0x00F000F0u : 0x000F000Fu);
    uint32_t v;
    asm("fma.rn.bf16x2 %0, %1, %2, %3;"
        : "=r"(v)
        : "r"(n), "r"(j & 1 ? 0x7D007D00u : 0x7F007F00u), "r"(0xBE00BE00u));  // 2^123 or 2^127, -1/8
    return v;
}

// The KS warps of a group (KS = 1: one warp) meet
__device__ __forceinline__ void w4_group_sync(int id, int KS) {
    if (KS == 1)
        __syncwarp();
    else
        asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(KS * 32) : "memory");
}

// One unit: 32 weight rows of one slot times m <= 8 C activation rows.
struct W4Unit {
    const W4Problem* p;
    const uint8_t* wq;      // the slot's packed weights
    const uint16_t* ws;     // and scales
    int n0;                 // first output
    int64_t row0;           // first output row
    int m;                  // rows
    bool routed;
};

template <bool SWIGLU, int GS, int C>
__device__ __forceinline__ void w4_run_unit(const W4Launch& a, const W4Unit& u, int KS, int ks, uint32_t ring,
                                            float* red, int group_warp0, int group_id, int buf) {
    constexpr int TN = SWIGLU ? 16 : 32;
    constexpr int NF = 4 / GS;  // groups in a stage
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    const int K = u.p->K, N = u.p->N_out;
    // this warp's stages: a contiguous range, so its rows' cache lines and scales follow each other
    const int nst_all = (K + 127) / 128;
    const int st0 = ks * nst_all / KS, nst = (ks + 1) * nst_all / KS - st0;
    // elements past the range's last whole stage (a row may end inside a stage, at a group's end)
    const int tail = min(K - (st0 + nst - 1) * 128, 128);

    // weight copies: row lane / 4 of each eight, 16-byte piece lane % 4
    const uint8_t* wsrc[4];
    const uint16_t* ssrc[4];  // scales of accumulator rows g, g + 8 of both 16-row tiles
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        int r = u.n0 + i * 8 + g;
        if (SWIGLU)
            r = i < 2 ? r : r - 16 + N;  // tile 1: the up rows
        else
            r = min(r, N - 1);
        wsrc[i] = u.wq + (int64_t)r * (K / 2) + st0 * 64 + t * 16;
        ssrc[i] = u.ws + (int64_t)r * (K / (32 * GS)) + st0 * NF;
    }
    // pieces rotate within a row so that the reads below meet every bank once
    const int sw = ((g >> 1) & 1) * 2 + (g >> 2);
    const uint32_t dst = ring + g * 64 + ((t ^ sw) << 4);
    const int lane_nst = t * 32 < tail ? nst : nst - 1;  // stages that hold this lane's piece
#define W4_ISSUE(i, off)                                                                                       \
    do {                                                                                                       \
        if ((i) < lane_nst) {                                                                                  \
            _Pragma("unroll") for (int q_ = 0; q_ < 4; ++q_)                                                   \
                w4_cp16(dst + ((off) % W4_RING) * W4_STAGE + q_ * 512, wsrc[q_] + (off) * 64);                 \
        }                                                                                                      \
        w4_cp_commit();                                                                                        \
    } while (0)
#pragma unroll
    for (int i = 0; i < W4_RING - 1; ++i) W4_ISSUE(i, i);

    // activation rows of this lane's B columns (column g of each tile of eight)
    const uint16_t* xsrc[C];
    int x_nst[C][NF];  // stages that hold the lane's elements of each group
#pragma unroll
    for (int c = 0; c < C; ++c) {
        const int col = c * 8 + g;
        bool ok = col < u.m;
        int64_t xr = u.row0 + (ok ? col : 0);
        if (u.routed && a.perm_src) {
            const int32_t p = a.perm_src[xr];
            if (p < 0 || (int64_t)p >= a.T * a.k) {
                report(a.status, MOE_ERR_DEVICE_BOUNDS);
                ok = false;
                xr = 0;
            } else {
                xr = p / a.k;
            }
        }
        xsrc[c] = u.p->x + xr * K + st0 * 128 + t * 8 * GS;
#pragma unroll
        for (int f = 0; f < NF; ++f) x_nst[c][f] = !ok ? 0 : f * 32 * GS < tail ? nst : nst - 1;
    }
    uint4 xb[C][4];
    uint32_t sb[NF][4];
#define W4_LOAD_X(i, off, f)                                                                                   \
    do {                                                                                                       \
        _Pragma("unroll") for (int c_ = 0; c_ < C; ++c_) {                                                     \
            if ((i) < x_nst[c_][f]) {                                                                          \
                _Pragma("unroll") for (int j_ = 0; j_ < GS; ++j_) xb[c_][(f) * GS + j_] =                      \
                    *reinterpret_cast<const uint4*>(xsrc[c_] + (off) * 128 + (f) * 32 * GS + j_ * 8);          \
            }                                                                                                  \
        }                                                                                                      \
    } while (0)
#define W4_LOAD_S(i, off, f)                                                                                   \
    do {                                                                                                       \
        if ((i) < (NF == 1 || (f) * 32 * GS < tail ? nst : nst - 1)) {                                         \
            _Pragma("unroll") for (int q_ = 0; q_ < 4; ++q_) sb[f][q_] = __ldg(ssrc[q_] + (off) * NF + (f));   \
        }                                                                                                      \
    } while (0)
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int j = 0; j < 4; ++j) xb[c][j] = make_uint4(0, 0, 0, 0);  // unused columns stay zero
#pragma unroll
    for (int f = 0; f < NF; ++f) {
        W4_LOAD_X(0, 0, f);
        W4_LOAD_S(0, 0, f);
    }

    float acc[2][C][4];
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[r][c][i] = 0.f;

    const uint32_t rd = ring + g * 64;
    // the stages, four at a time so that every address is a register and a constant
    for (int i0 = 0; i0 < nst; i0 += W4_RING) {
#pragma unroll
        for (int v = 0; v < W4_RING; ++v) {
            const int i = i0 + v;
            if (i < nst) {
                W4_ISSUE(i + W4_RING - 1, v + W4_RING - 1);
                w4_cp_wait<W4_RING - 1>();
                __syncwarp();
                const int left = i + 1 < nst ? 128 : tail;
#pragma unroll
                for (int f = 0; f < NF; ++f) {
                    if (NF == 1 || f * 32 * GS < left) {
                        // words 0 .. GS-1 of this lane in the group: elements t * 8 GS .. of the rows g + 8 q
                        uint32_t w[4][GS];
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const int byte = f * 16 * GS;  // of the group in the row; the lane's at + t * 4 GS
                            const uint32_t at = rd + v * W4_STAGE + q * 512 +
                                                ((((byte + t * 4 * GS) >> 4) ^ sw) << 4) + ((t * 4 * GS) & 15);
                            w4_lds<GS>(w[q], at);
                        }
                        float tmp[2][C][4];
#pragma unroll
                        for (int j = 0; j < GS; ++j)
#pragma unroll
                            for (int h = 0; h < 2; ++h) {
                                uint32_t A[2][4];
#pragma unroll
                                for (int r = 0; r < 2; ++r) {
                                    A[r][0] = w4_pair(w[2 * r][j], 2 * h);
                                    A[r][1] = w4_pair(w[2 * r + 1][j], 2 * h);
                                    A[r][2] = w4_pair(w[2 * r][j], 2 * h + 1);
                                    A[r][3] = w4_pair(w[2 * r + 1][j], 2 * h + 1);
                                }
#pragma unroll
                                for (int c = 0; c < C; ++c) {
                                    const uint4 b = xb[c][f * GS + j];
                                    const uint32_t b0 = h ? b.z : b.x, b1 = h ? b.w : b.y;
                                    if (j == 0 && h == 0) {
                                        w4_mma_first(tmp[0][c], A[0], b0, b1);
                                        w4_mma_first(tmp[1][c], A[1], b0, b1);
                                    } else {
                                        w4_mma(tmp[0][c], A[0], b0, b1);
                                        w4_mma(tmp[1][c], A[1], b0, b1);
                                    }
                                }
                            }
#pragma unroll
                        for (int r = 0; r < 2; ++r) {
                            const float s0 = bf16_bits_to_float(sb[f][2 * r]);
                            const float s1 = bf16_bits_to_float(sb[f][2 * r + 1]);
#pragma unroll
                            for (int c = 0; c < C; ++c) {
                                acc[r][c][0] = fmaf(s0, tmp[r][c][0], acc[r][c][0]);
                                acc[r][c][1] = fmaf(s0, tmp[r][c][1], acc[r][c][1]);
                                acc[r][c][2] = fmaf(s1, tmp[r][c][2], acc[r][c][2]);
                                acc[r][c][3] = fmaf(s1, tmp[r][c][3], acc[r][c][3]);
                            }
                        }
                    }
                    // the same registers take the next stage's values
                    W4_LOAD_X(i + 1, v + 1, f);
                    W4_LOAD_S(i + 1, v + 1, f);
                }
                __syncwarp();  // the ring slot just read is the next one written
            }
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            wsrc[q] += W4_RING * 64;
            ssrc[q] += W4_RING * NF;
        }
#pragma unroll
        for (int c = 0; c < C; ++c) xsrc[c] += W4_RING * 128;
    }
    w4_cp_wait<0>();
#undef W4_ISSUE
#undef W4_LOAD_X
#undef W4_LOAD_S

    // partial sums of the group's warps, added in order of their K ranges
    float* mine = red + (buf * W4_WARPS + warp) * (32 * 8 * C);
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int c = 0; c < C; ++c) {
            float* p = mine + (r * 16 + g) * (8 * C) + c * 8 + 2 * t;
            *reinterpret_cast<float2*>(p) = make_float2(64.f * acc[r][c][0], 64.f * acc[r][c][1]);
            *reinterpret_cast<float2*>(p + 8 * 8 * C) = make_float2(64.f * acc[r][c][2], 64.f * acc[r][c][3]);
        }
    w4_group_sync(group_id, KS);
    const float* all = red + (buf * W4_WARPS + group_warp0) * (32 * 8 * C);
    for (int o = ks * 32 + lane; o < TN * u.m; o += KS * 32) {
        const int f = o % TN, col = o / TN;
        float v = 0.f, up = 0.f;
        for (int q = 0; q < KS; ++q) {
            const float* p = all + q * (32 * 8 * C);
            v += p[f * (8 * C) + col];
            if (SWIGLU) up += p[(16 + f) * (8 * C) + col];
        }
        if (SWIGLU) v = v / (1.0f + expf(-v)) * up;
        const int n = u.n0 + f;
        if (n < N) {
            const int64_t at = (u.row0 + col) * N + n;
            if (u.p->out_f32)
                u.p->out_f32[at] = v;
            else
                u.p->out_bf16[at] = (uint16_t)(pack_bf16x2(v, 0.f) & 0xFFFFu);
        }
    }
}

template <bool SWIGLU, int GS, int C>
__global__ void __launch_bounds__(W4_THREADS, 2) w4_mma_kernel(const __grid_constant__ W4Launch a, int KS) {
    extern __shared__ __align__(128) uint8_t w4_smem[];
    __shared__ int32_t s_pre[W4_MAXG];  // units of the routed slots before each slot
    __shared__ int32_t s_part[W4_WARPS];
    constexpr int TN = SWIGLU ? 16 : 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t ring = smem_u32(w4_smem) + warp * (W4_RING * W4_STAGE);
    float* red = reinterpret_cast<float*>(w4_smem + W4_WARPS * W4_RING * W4_STAGE);
    pdl_wait();
    pdl_trigger();

    const int tiles_sh = a.sh.wq ? (a.sh.N_out + TN - 1) / TN : 0;
    const int ct_sh = (int)((a.rows_sh + 8 * C - 1) / (8 * C));
    const int units_sh = tiles_sh * ct_sh;
    const int tiles = a.G > 0 ? (a.rt.N_out + TN - 1) / TN : 0;
    int units = units_sh;
    if (a.G > 0) {
        // exclusive scan of the slots' units, four slots a thread
        const int s0 = threadIdx.x * (W4_MAXG / W4_THREADS);
        int n[W4_MAXG / W4_THREADS], sum = 0;
        int64_t lo = s0 <= a.G ? __ldg(a.offsets + s0) : 0;
#pragma unroll
        for (int i = 0; i < W4_MAXG / W4_THREADS; ++i) {
            n[i] = 0;
            if (s0 + i < a.G) {
                const int64_t hi = __ldg(a.offsets + s0 + i + 1);
                const int64_t m = max((int64_t)0, min(hi, a.rows_cap) - max(lo, (int64_t)0));
                n[i] = (int)((m + 8 * C - 1) / (8 * C)) * tiles;
                lo = hi;
            }
            sum += n[i];
        }
        int inc = sum;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, inc, off);
            if (lane >= off) inc += v;
        }
        if (lane == 31) s_part[warp] = inc;
        __syncthreads();
        int base = inc - sum, total = 0;
#pragma unroll
        for (int w = 0; w < W4_WARPS; ++w) {
            base += w < warp ? s_part[w] : 0;
            total += s_part[w];
        }
#pragma unroll
        for (int i = 0; i < W4_MAXG / W4_THREADS; ++i) {
            if (s0 + i < a.G) s_pre[s0 + i] = base;
            base += n[i];
        }
        units += total;
        __syncthreads();
    }

    const int groups = W4_WARPS / KS;
    const int grp = warp / KS, ks = warp - grp * KS;
    int buf = 0;
    for (int64_t v = (int64_t)grp * gridDim.x + blockIdx.x; v < units; v += (int64_t)groups * gridDim.x, buf ^= 1) {
        W4Unit u;
        if (v < units_sh) {
            const int c = (int)v % ct_sh;
            u.p = &a.sh;
            u.wq = a.sh.wq;
            u.ws = a.sh.ws;
            u.n0 = ((int)v / ct_sh) * TN;
            u.row0 = (int64_t)c * 8 * C;
            u.m = (int)min((int64_t)(8 * C), a.rows_sh - u.row0);
            u.routed = false;
        } else {
            const int w = (int)v - units_sh;
            int lo = 0, hi = a.G - 1;  // the last slot whose units begin at or before w
            while (lo < hi) {
                const int mid = (lo + hi + 1) / 2;
                if (s_pre[mid] <= w)
                    lo = mid;
                else
                    hi = mid - 1;
            }
            const int64_t first = max(0, __ldg(a.offsets + lo));
            const int64_t end = min((int64_t)__ldg(a.offsets + lo + 1), a.rows_cap);
            const int ct = (int)((end - first + 8 * C - 1) / (8 * C));
            const int q = w - s_pre[lo];
            const int64_t wrows = SWIGLU ? 2 * (int64_t)a.rt.N_out : a.rt.N_out;
            u.p = &a.rt;
            u.wq = a.rt.wq + lo * wrows * (a.rt.K / 2);
            u.ws = a.rt.ws + lo * wrows * (a.rt.K / (32 * GS));
            u.n0 = (q / ct) * TN;
            u.row0 = first + (int64_t)(q % ct) * 8 * C;
            u.m = (int)min((int64_t)(8 * C), end - u.row0);
            u.routed = true;
        }
        w4_run_unit<SWIGLU, GS, C>(a, u, KS, ks, ring, red, grp * KS, grp + 1, buf);
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

template <bool SWIGLU, int GS, int C>
static cudaError_t launch_w4_mma(const W4Launch& L, int num_sms, cudaStream_t s) {
    // the shared-memory limit is set once per device
    static std::atomic<bool> ready[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    const size_t smem = w4_smem_bytes(C);
    if (!ready[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(w4_mma_kernel<SWIGLU, GS, C>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        ready[dev].store(true, std::memory_order_release);
    }
    // Warps of a unit split its K among them: more of them shorten a unit, fewer waste
    // less on its ends.  KS minimises the list-scheduling bound over groups of KS warps,
    // sum of the units' stages / groups + the longest unit, a unit's ends counted as
    // three stages.  The routed units are bounded by one row tile per slot with pairs.
    constexpr int TN = SWIGLU ? 16 : 32;
    const double u_sh = L.sh.wq ? (double)((L.sh.N_out + TN - 1) / TN) * ((L.rows_sh + 8 * C - 1) / (8 * C)) : 0.0;
    const double u_rt = L.G > 0 ? (double)((L.rt.N_out + TN - 1) / TN) * std::min<int64_t>(L.rows_cap, L.G) : 0.0;
    const int n_sh = (L.sh.K + 127) / 128, n_rt = (L.rt.K + 127) / 128;
    int KS = 1;
    double best = 0.0;
    for (int ks = 1; ks <= W4_WARPS; ks *= 2) {
        const double groups = 2.0 * num_sms * W4_WARPS / ks;
        const double l_sh = (n_sh + ks - 1) / ks + 3, l_rt = (n_rt + ks - 1) / ks + 3;
        const double cost = (u_sh * l_sh + u_rt * l_rt) / groups + std::max(u_sh > 0 ? l_sh : 0.0, u_rt > 0 ? l_rt : 0.0);
        if (ks == 1 || cost < best) {
            best = cost;
            KS = ks;
        }
    }
    const double want = std::ceil((u_sh + u_rt) * KS / W4_WARPS);
    const unsigned grid = (unsigned)std::max(1.0, std::min(want, 2.0 * num_sms));
    return launch_k(L.name, w4_mma_kernel<SWIGLU, GS, C>, dim3(grid), dim3(W4_THREADS), smem, s, L, KS);
}

template <bool SWIGLU, int GS>
static cudaError_t launch_w4_rows(const W4Launch& L, int num_sms, cudaStream_t s) {
    // a slot has at most as many rows as there are tokens
    const int64_t most = std::max<int64_t>(L.sh.wq ? L.rows_sh : 0, L.G > 0 ? std::min(L.T, L.rows_cap) : 0);
    return most <= 8 ? launch_w4_mma<SWIGLU, GS, 1>(L, num_sms, s) : launch_w4_mma<SWIGLU, GS, 2>(L, num_sms, s);
}

template <bool SWIGLU>
static cudaError_t launch_w4_group(const W4Launch& L, int num_sms, cudaStream_t s) {
    if (L.group == 32) return launch_w4_rows<SWIGLU, 1>(L, num_sms, s);
    if (L.group == 64) return launch_w4_rows<SWIGLU, 2>(L, num_sms, s);
    return launch_w4_rows<SWIGLU, 4>(L, num_sms, s);
}

cudaError_t launch_w4_gemm(const W4Launch& L, int num_sms, cudaStream_t s) {
    return L.swiglu ? launch_w4_group<true>(L, num_sms, s) : launch_w4_group<false>(L, num_sms, s);
}

cudaError_t launch_w4_combine(const W4CombineLaunch& L, cudaStream_t s) {
    const dim3 grid((unsigned)L.T, (unsigned)((L.H + W4C_THREADS * 4 - 1) / (W4C_THREADS * 4)));
    return launch_k("w4_combine", w4_combine_kernel, grid, dim3(W4C_THREADS), 0, s, L);
}

}  // namespace moe

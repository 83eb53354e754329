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
// Products on mma.sync.  The work is a list of tiles, 32 weight rows of one slot
// (FC1: 16 gate rows and the matching 16 up rows) times up to 8 C activation rows;
// a tile's K is cut into stages of 128.  Every CTA takes a contiguous range of the
// list, about the same number of stages each, and its 8 warps take equal
// contiguous ranges of those stages, whatever tiles they fall into.  A warp streams
// its stages through a ring of its own without a break at a tile's end; it stores
// the tiles that are all its own, and leaves its part of the at most two that it
// shares with its neighbours in shared memory, where the warp that ends a tile adds
// the parts in stage order.
// ---------------------------------------------------------------------------
constexpr int W4_STAGE = 2048;  // bytes of a stage: 32 rows of 128 elements
constexpr int W4_MAXG = 1024;   // slots

// The narrow kernel (C = 1) runs two CTAs an SM: eight columns leave the tensor cores
// idle and the masks and the multiply-adds that widen the codes bound it, which more
// warps hide.  The wide one (C = 4) keeps four column tiles of sums and activations in
// the registers of one CTA.  Both have 128 KB of weights of an SM in their rings.
constexpr int W4_WARPS = 8;
__host__ __device__ constexpr int w4_ctas(int C) { return C == 1 ? 2 : 1; }  // on an SM
__host__ __device__ constexpr int w4_ring(int C) { return 8 / w4_ctas(C); }  // stages in each warp's ring

__host__ __device__ constexpr size_t w4_smem_bytes(int C) {
    // every warp's ring, then its parts of two shared tiles (16 C sums a lane)
    return (size_t)W4_WARPS * (w4_ring(C) * W4_STAGE + 2 * 32 * 8 * C * 4);
}

struct W4Tile {
    const uint8_t* wq;   // packed weights and scales of its first row
    const uint16_t* ws;
    int64_t row0;        // first output row
    int n0, m;           // first output, rows
    int ct;              // row tiles of its slot
    int x;               // where its activation rows stand
    bool routed;
};

__device__ __forceinline__ void w4_cp16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void w4_prefetch_l2(const void* p) {
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p) : "memory");
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

// One group of a stage: acc += scales * (codes x activations), C8 of the C column tiles
// of eight.  w: the lane's words of rows g + 8 q, xb: its activations, [column tile][4].
template <int GS, int C8, int C>
__device__ __forceinline__ void w4_group(float (&acc)[2][C][4], const uint32_t (&w)[4][GS], const uint4* xb,
                                         const uint32_t (&sb)[4]) {
    float tmp[2][C8][4];
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
            for (int c = 0; c < C8; ++c) {
                const uint4 b = xb[c * 4 + j];
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
        const float s0 = bf16_bits_to_float(sb[2 * r]), s1 = bf16_bits_to_float(sb[2 * r + 1]);
#pragma unroll
        for (int c = 0; c < C8; ++c) {
            acc[r][c][0] = fmaf(s0, tmp[r][c][0], acc[r][c][0]);
            acc[r][c][1] = fmaf(s0, tmp[r][c][1], acc[r][c][1]);
            acc[r][c][2] = fmaf(s1, tmp[r][c][2], acc[r][c][2]);
            acc[r][c][3] = fmaf(s1, tmp[r][c][3], acc[r][c][3]);
        }
    }
}

// The outputs of a tile from its accumulators: this lane has rows g, g + 8 of both
// 16-row halves and columns 2t, 2t + 1 of every eight.
template <bool SWIGLU, int C>
__device__ __forceinline__ void w4_store(const W4Problem& p, const W4Tile& d, const float (&acc)[2][C][4]) {
    const int g = (threadIdx.x & 31) >> 2, t = threadIdx.x & 3;
    const int64_t N = p.N_out;
    auto put = [&](int64_t at, float v) {
        if (p.out_f32)
            p.out_f32[at] = v;
        else
            p.out_bf16[at] = (uint16_t)(pack_bf16x2(v, 0.f) & 0xFFFFu);
    };
#pragma unroll
    for (int c = 0; c < C; ++c)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const int col = c * 8 + 2 * t + e;
            if (col >= d.m) continue;
            const int64_t at = (d.row0 + col) * N + d.n0 + g;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                // the codes were c / 64
                const float v0 = 64.f * acc[0][c][2 * h + e], v1 = 64.f * acc[1][c][2 * h + e];
                if (SWIGLU) {
                    put(at + 8 * h, v0 / (1.0f + expf(-v0)) * v1);
                } else {
                    if (d.n0 + 8 * h + g < N) put(at + 8 * h, v0);
                    if (d.n0 + 16 + 8 * h + g < N) put(at + 16 + 8 * h, v1);
                }
            }
        }
}

template <bool SWIGLU, int GS, int C>
__global__ void __launch_bounds__(W4_WARPS * 32, w4_ctas(C)) w4_kernel(const __grid_constant__ W4Launch a) {
    constexpr int WARPS = W4_WARPS, RING = w4_ring(C);
    constexpr int TILES = 2 * RING;  // tiles a warp has in hand: the copies run RING - 1 stages ahead
    extern __shared__ __align__(128) uint8_t w4_smem[];
    __shared__ int32_t s_pre[W4_MAXG];  // routed tiles before each slot
    __shared__ int32_t s_part[WARPS];
    __shared__ W4Tile s_tile[WARPS][TILES];
    __shared__ int32_t s_x[WARPS][TILES][8 * C];  // activation row of each column, -1: none
    constexpr int TN = SWIGLU ? 16 : 32;                // outputs of a tile
    constexpr int NF = 4 / GS;                          // groups in a stage
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int g = lane >> 2, t = lane & 3;
    // pieces rotate within a row of a stage so that the reads below meet every bank once
    const int sw = ((g >> 1) & 1) * 2 + (g >> 2);
    const uint32_t ring = smem_u32(w4_smem) + warp * (RING * W4_STAGE) + g * 64;
    // part [warp][0: of a tile begun by an earlier warp, 1: of one begun here][4 values][lane]
    float4* parts = reinterpret_cast<float4*>(w4_smem + WARPS * RING * W4_STAGE);
    // What a previous kernel may still be writing is waited for as late as the call allows:
    // the tables here, the weights before their first copy, the activations after it.
    if (!a.early && a.G > 0) {
        pdl_wait();
        pdl_trigger();
    }

    // the list: the dense problem's tiles, then the routed ones by slot; the row tiles of
    // one weight tile are neighbours
    const int ct_sh = (int)((a.rows_sh + 8 * C - 1) / (8 * C));
    const int n_sh = (a.sh.K + 127) / 128, n_rt = (a.rt.K + 127) / 128;  // stages of a tile
    const int tiles_rt = (a.rt.N_out + TN - 1) / TN;
    const int64_t list_sh = a.sh.wq ? (int64_t)((a.sh.N_out + TN - 1) / TN) * ct_sh : 0;
    int64_t list_rt = 0;
    if (a.G > 0) {
        constexpr int PER = W4_MAXG / (WARPS * 32);
        const int s0 = threadIdx.x * PER;
        int n[PER], sum = 0;
        int64_t lo = s0 <= a.G ? __ldg(a.offsets + s0) : 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            n[i] = 0;
            if (s0 + i < a.G) {
                const int64_t hi = __ldg(a.offsets + s0 + i + 1);
                const int64_t m = max((int64_t)0, min(hi, a.rows_cap) - max(lo, (int64_t)0));
                n[i] = (int)((m + 8 * C - 1) / (8 * C)) * tiles_rt;
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
        for (int w = 0; w < WARPS; ++w) {
            base += w < warp ? s_part[w] : 0;
            total += s_part[w];
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            if (s0 + i < a.G) s_pre[s0 + i] = base;
            base += n[i];
        }
        list_rt = total;
        __syncthreads();
    }
    // this CTA's tiles: from the first that starts at or after its share of the stages
    const int64_t stages_sh = list_sh * n_sh, stages = stages_sh + list_rt * n_rt;
    const bool small = stages * gridDim.x < (int64_t(1) << 31);  // divisions in 32 bits, a fifth of the 64-bit ones
    auto over = [small](int64_t x, int y) {
        return small ? (int64_t)((uint32_t)x / (uint32_t)y) : x / (int64_t)y;
    };
    auto first_tile = [&](int64_t cta) {
        const int64_t s = over(stages * cta, (int)gridDim.x);
        return s <= stages_sh ? (n_sh ? over(s + n_sh - 1, n_sh) : 0) : list_sh + over(s - stages_sh + n_rt - 1, n_rt);
    };
    auto start_of = [&](int64_t v) { return v <= list_sh ? v * n_sh : stages_sh + (v - list_sh) * n_rt; };
    const int64_t base = start_of(first_tile(blockIdx.x));
    const int64_t all = start_of(first_tile(blockIdx.x + 1)) - base;
    // this warp's stages: cnt from lo; the first one's tile
    const int64_t lo = base + all * warp / WARPS;
    const int cnt = (int)(base + all * (warp + 1) / WARPS - lo);
    const int64_t v0 = lo < stages_sh ? over(lo, n_sh) : list_sh + (n_rt ? over(lo - stages_sh, n_rt) : 0);

    // Three cursors run over the stages: the copies three ahead, the activations and
    // scales one ahead, the products.  Tile i from v0 is at s_tile[warp][i % TILES]
    // from when the copies reach it; ends count from lo.  (The loop is not unrolled over
    // the ring: four copies of what a tile's end takes overran the instruction cache,
    // 3 of 8 stalled cycles.)
    W4Tile* tiles = s_tile[warp];
    auto end_of = [&](int i) { return (int)(start_of(v0 + i + 1) - lo); };
    int xs = 0;  // activation row sets so far
    auto locate = [&](int i) {
        W4Tile d;
        const int64_t v = v0 + i;
        if (i > 0) {
            d = tiles[(i - 1) % TILES];
            const W4Problem& p = d.routed ? a.rt : a.sh;
            if (d.ct == 1 && d.n0 + TN < p.N_out) {  // the same rows, the next weights
                d.n0 += TN;
                d.wq += (int64_t)TN * (p.K / 2);
                d.ws += (int64_t)TN * (p.K / (32 * GS));
                __syncwarp();
                if (lane == 0) tiles[i % TILES] = d;
                __syncwarp();
                return;
            }
        }
        int64_t rows, at;  // the slot's end, its first weight row
        int q;             // tile of the slot
        if (v < list_sh) {
            q = (int)v;
            d.routed = false;
            d.ct = ct_sh;
            d.row0 = 0;
            rows = a.rows_sh;
            at = 0;
        } else {
            const int w = (int)(v - list_sh);
            int s_lo = 0, s_hi = a.G - 1;  // the last slot whose tiles begin at or before w
            while (s_lo < s_hi) {
                const int mid = (s_lo + s_hi + 1) / 2;
                if (s_pre[mid] <= w)
                    s_lo = mid;
                else
                    s_hi = mid - 1;
            }
            d.routed = true;
            d.row0 = max(0, __ldg(a.offsets + s_lo));
            rows = min((int64_t)__ldg(a.offsets + s_lo + 1), a.rows_cap);
            d.ct = (int)((rows - d.row0 + 8 * C - 1) / (8 * C));
            q = w - s_pre[s_lo];
            at = s_lo * (SWIGLU ? 2 * (int64_t)a.rt.N_out : a.rt.N_out);
        }
        const W4Problem& p = d.routed ? a.rt : a.sh;
        d.n0 = q / d.ct * TN;
        d.row0 += (int64_t)(q % d.ct) * 8 * C;
        d.m = (int)min((int64_t)(8 * C), rows - d.row0);
        d.wq = p.wq + (at + d.n0) * (p.K / 2);
        d.ws = p.ws + (at + d.n0) * (p.K / (32 * GS));
        d.x = xs++ % TILES;
        __syncwarp();
        if (lane == 0) tiles[i % TILES] = d;
        __syncwarp();
    };
    // the activation rows of tile i's columns (FC1 reads the routing table for them)
    int x_done = -1;
    auto rows_of = [&](int i) {
        const W4Tile& d = tiles[i % TILES];
        if (d.x == x_done) return;
        x_done = d.x;
        if (lane < 8 * C) {
            int32_t r = lane < d.m ? (int32_t)(d.row0 + lane) : -1;
            if (r >= 0 && d.routed && a.perm_src) {
                const int32_t p = a.perm_src[r];
                const bool ok = p >= 0 && (int64_t)p < a.T * a.k;
                if (!ok) report(a.status, MOE_ERR_DEVICE_BOUNDS);
                r = ok ? p / a.k : -1;
            }
            s_x[warp][d.x][lane] = r;
        }
        __syncwarp();
    };
    auto row_of = [&](const W4Problem& p, const W4Tile& d, int q) {  // weight row g + 8 q from the tile's first
        const int r = q * 8 + g;
        return SWIGLU ? (q < 2 ? r : r - 16 + p.N_out) : min(r, p.N_out - 1 - d.n0);
    };

    const uint8_t* wsrc[4];
    int w_tile = -1, w_end = 0, w_lane_end = 0;
    auto next_w = [&](int j) {  // the copies' next tile, from stage j
        locate(++w_tile);
        const W4Tile& d = tiles[w_tile % TILES];
        const W4Problem& p = d.routed ? a.rt : a.sh;
        const int n = d.routed ? n_rt : n_sh, end = end_of(w_tile);
#pragma unroll
        for (int q = 0; q < 4; ++q)
            wsrc[q] = d.wq + (int64_t)row_of(p, d, q) * (p.K / 2) + (j + n - end) * 64 + t * 16;
        w_end = min(end, cnt);
        // a row may end inside its last stage (at a group's end)
        const bool cut = GS < 4 && end <= cnt && t * 32 >= p.K - (n - 1) * 128;
        w_lane_end = w_end - (cut ? 1 : 0);
    };
    uint32_t w_slot = ring + ((t ^ sw) << 4), r_slot = ring;  // ring stages written and read next
    auto turn_slot = [&](uint32_t slot) {
        const uint32_t first = smem_u32(w4_smem) + warp * (RING * W4_STAGE);
        return first + ((slot - first + W4_STAGE) & (RING * W4_STAGE - 1));
    };
    auto issue = [&](int j) {
        if (j >= w_end && j < cnt) next_w(j);
        if (j < w_lane_end) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                w4_cp16(w_slot + q * 512, wsrc[q]);
                wsrc[q] += 64;
            }
        }
        w4_cp_commit();
        w_slot = turn_slot(w_slot);
    };
    if (!a.early && a.G == 0) {
        if (cnt > 0) {
            // the first stages' lines on their way to L2 meanwhile
            next_w(0);
            if (t == 0)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    w4_prefetch_l2(wsrc[q]);
                    if (w_end > 2) w4_prefetch_l2(wsrc[q] + 128);
                }
        }
        pdl_wait();
        pdl_trigger();
    }
#pragma unroll 1
    for (int j = 0; j < RING - 1; ++j) issue(j);

    if (a.early) {  // the tables and the weights do not depend on the previous kernel, the activations do
        pdl_wait();
        pdl_trigger();
    }

    const uint16_t* xsrc[C];
    const uint16_t* ssrc[4];  // scales of accumulator rows g, g + 8 of both 16-row halves
    bool x_ok[C];
    int p_tile = -1, p_end = 0;
    int p_last = 0, p_cut = 0;  // the stage that ends the tile's rows, and how many elements it holds
    auto next_p = [&](int j) {  // the activations' and scales' next tile, from stage j
        rows_of(++p_tile);
        const W4Tile& d = tiles[p_tile % TILES];
        const W4Problem& p = d.routed ? a.rt : a.sh;
        const int n = d.routed ? n_rt : n_sh;
        p_last = end_of(p_tile) - 1;
        p_cut = p.K - (n - 1) * 128;
        p_end = min(p_last + 1, cnt);
        const int stage = j + n - 1 - p_last;
#pragma unroll
        for (int q = 0; q < 4; ++q)
            ssrc[q] = d.ws + (int64_t)row_of(p, d, q) * (p.K / (32 * GS)) + stage * NF;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            const int32_t r = s_x[warp][d.x][c * 8 + g];
            x_ok[c] = r >= 0;
            xsrc[c] = p.x + (int64_t)max(r, 0) * p.K + stage * 128 + t * 8 * GS;
        }
    };
    uint4 xb[C][4];
    uint32_t sb[NF][4];
    auto load = [&](int f, int has) {  // group f of their stage, which holds `has` elements
        if (f * 32 * GS < has) {
#pragma unroll
            for (int c = 0; c < C; ++c)
                if (x_ok[c]) {
#pragma unroll
                    for (int j = 0; j < GS; ++j)
                        xb[c][f * GS + j] = *reinterpret_cast<const uint4*>(xsrc[c] + f * 32 * GS + j * 8);
                }
#pragma unroll
            for (int q = 0; q < 4; ++q) sb[f][q] = __ldg(ssrc[q] + f);
        }
    };
    auto step = [&] {
#pragma unroll
        for (int q = 0; q < 4; ++q) ssrc[q] += NF;
#pragma unroll
        for (int c = 0; c < C; ++c) xsrc[c] += 128;
    };
    float acc[2][C][4];
    auto clear = [&] {
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int c = 0; c < C; ++c)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[r][c][e] = 0.f;
    };
    clear();
    int left = 0;  // elements of the stage that is multiplied next
    int tile = 0, m = 0, end = 0;
    if (cnt > 0) {
        next_p(0);
        left = GS < 4 && p_last == 0 ? p_cut : 128;
#pragma unroll
        for (int c = 0; c < C; ++c)
#pragma unroll
            for (int j = 0; j < 4; ++j) xb[c][j] = make_uint4(0, 0, 0, 0);  // columns without a row stay zero
#pragma unroll
        for (int f = 0; f < NF; ++f) load(f, left);
        step();
        m = tiles[0].m;
        end = min(end_of(0), cnt);
    }
    bool begun = lo > start_of(v0);  // the tile in hand was begun by an earlier warp
    W4Tile head;                     // the tile that an earlier warp began and this one ended, or m = 0
    int64_t head_start = 0;
    head.m = 0;

#pragma unroll 1
    for (int i = 0; i < cnt; ++i) {
        issue(i + RING - 1);
        const bool turn = i + 1 == p_end && i + 1 < cnt;  // the next stage is another tile's
        if (turn) next_p(i + 1);
        const int next = i + 1 < cnt ? (GS < 4 && i + 1 == p_last ? p_cut : 128) : 0;
        w4_cp_wait<RING - 1>();
        __syncwarp();
#pragma unroll
        for (int f = 0; f < NF; ++f) {
            if (NF == 1 || f * 32 * GS < left) {
                // words 0 .. GS-1 of this lane in the group: elements t * 8 GS .. of the rows g + 8 q
                uint32_t w[4][GS];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const int byte = f * 16 * GS + t * 4 * GS;
                    w4_lds<GS>(w[q], r_slot + q * 512 + (((byte >> 4) ^ sw) << 4) + (byte & 15));
                }
                if (C == 1 || m <= 8)
                    w4_group<GS, 1, C>(acc, w, &xb[0][f * GS], sb[f]);
                else if (C == 2 || m <= 16)
                    w4_group<GS, C < 2 ? C : 2, C>(acc, w, &xb[0][f * GS], sb[f]);
                else
                    w4_group<GS, C, C>(acc, w, &xb[0][f * GS], sb[f]);
            }
            // the same registers take the next stage's values
            if (turn) {
#pragma unroll
                for (int c = 0; c < C; ++c)
                    if (!x_ok[c])
#pragma unroll
                        for (int j = 0; j < GS; ++j) xb[c][f * GS + j] = make_uint4(0, 0, 0, 0);
            }
            load(f, next);
        }
        __syncwarp();  // the ring slot just read is the next one written
        left = next;
        step();
        r_slot = turn_slot(r_slot);
        if (i + 1 == end) {  // the tile's last stage here
            const W4Tile& d = tiles[tile % TILES];
            const int tile_end = end_of(tile);
            if (!begun && tile_end <= cnt) {
                w4_store<SWIGLU, C>(d.routed ? a.rt : a.sh, d, acc);
            } else {
                float4* o = parts + ((warp * 2 + (begun ? 0 : 1)) * 2 * C) * 32 + lane;
#pragma unroll
                for (int r = 0; r < 2; ++r)
#pragma unroll
                    for (int c = 0; c < C; ++c)
                        o[(r * C + c) * 32] =
                            make_float4(acc[r][c][0], acc[r][c][1], acc[r][c][2], acc[r][c][3]);
                if (begun && tile_end <= cnt) {
                    head = d;
                    head_start = start_of(v0 + tile);
                }
            }
            clear();
            begun = false;
            if (i + 1 < cnt) {
                ++tile;
                m = tiles[tile % TILES].m;
                end = min(end_of(tile), cnt);
            }
        }
    }
    w4_cp_wait<0>();
    __syncthreads();

    // the parts of the tile that this warp ended, in stage order
    if (head.m > 0) {
        const int first = (int)((WARPS * (head_start - base + 1) - 1) / all);  // the warp that began it
        for (int w = first; w <= warp; ++w) {
            if (all * w / WARPS == all * (w + 1) / WARPS) continue;  // a warp without stages
            const float4* o = parts + ((w * 2 + (w == first ? 1 : 0)) * 2 * C) * 32 + lane;
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    const float4 f = o[(r * C + c) * 32];
                    acc[r][c][0] += f.x;
                    acc[r][c][1] += f.y;
                    acc[r][c][2] += f.z;
                    acc[r][c][3] += f.w;
                }
        }
        w4_store<SWIGLU, C>(head.routed ? a.rt : a.sh, head, acc);
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
    // the tables, x and the gate were written before FC2's predecessor began; only y waits
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
    pdl_wait();
    pdl_trigger();
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
static cudaError_t launch_w4_tiles(const W4Launch& L, int num_sms, cudaStream_t s) {
    // the shared-memory limit is set once per device
    static std::atomic<bool> ready[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    const size_t smem = w4_smem_bytes(C);
    if (!ready[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(w4_kernel<SWIGLU, GS, C>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        ready[dev].store(true, std::memory_order_release);
    }
    // No more CTAs than tiles, and no fewer stages to a CTA than its longest tile has
    // (between one CTA an SM and as many as fit).
    constexpr int TN = SWIGLU ? 16 : 32;
    const int n_sh = (L.sh.K + 127) / 128, n_rt = (L.rt.K + 127) / 128;
    const double sh = L.sh.wq ? (double)((L.sh.N_out + TN - 1) / TN) * ((L.rows_sh + 8 * C - 1) / (8 * C)) : 0.0;
    const double rt = L.G > 0 ? (double)((L.rt.N_out + TN - 1) / TN) * std::min<int64_t>(L.rows_cap, L.G) : 0.0;
    const double even = (sh * n_sh + rt * n_rt) / std::max(sh > 0 ? n_sh : 1, rt > 0 ? n_rt : 1);
    const double most = std::min(sh + rt, (double)w4_ctas(C) * num_sms);
    const unsigned grid = (unsigned)std::max(1.0, std::min(most, std::max(even, (double)num_sms)));
    return launch_k(L.name, w4_kernel<SWIGLU, GS, C>, dim3(grid), dim3(W4_WARPS * 32), smem, s, L);
}

template <bool SWIGLU, int GS>
static cudaError_t launch_w4_rows(const W4Launch& L, int num_sms, cudaStream_t s) {
    // Passes over the weights that the narrow kernel's 8 columns and the wide one's 32 take,
    // in weight rows; a slot holds rows_cap / G rows on average.
    const double sh = L.sh.wq ? (double)L.sh.N_out * L.sh.K : 0.0, rt = L.G > 0 ? (double)L.rt.N_out * L.rt.K : 0.0;
    const double slots = (double)std::min<int64_t>(L.G, L.rows_cap);
    const double mean = slots > 0 ? L.rows_cap / slots : 0.0;
    auto passes = [&](int rows) {
        return sh * std::ceil((double)L.rows_sh / rows) + rt * slots * std::max(1.0, mean / rows);
    };
#ifndef W4_WIDE
#define W4_WIDE 1.5
#endif
    return passes(8) < W4_WIDE * passes(32) ? launch_w4_tiles<SWIGLU, GS, 1>(L, num_sms, s)
                                            : launch_w4_tiles<SWIGLU, GS, 4>(L, num_sms, s);
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

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
#include <type_traits>

#include "moe_internal.cuh"

namespace moe {
namespace {

// ---------------------------------------------------------------------------
// Quantiser: one lane per word of eight elements, a group's lanes reduce together.
//
// A code is f / s to the nearest integer, ties to even.  f and s have eight significant
// bits, so f / s is a tie or at least 2^-12 (relative) away from one: f times the rounded
// 1 / s gives the integer except at a tie, and there the remainder f - c s, which is exact,
// tells.  Bound: instruction issue, above all the ALU (16384 x 7168: a scheduler issues in
// 0.83 of its cycles, the ALU is at 79 %, 251 instructions a warp of words).  65536 x 7168
// with groups of 32 (128): 426 .. 434 (457 .. 462) us, 2.8 (2.6) TB/s of weights read and
// codes written; eight IEEE divisions a lane instead 606 (628).  It runs once per weight.
// ---------------------------------------------------------------------------
constexpr int W4Q_THREADS = 256;
constexpr int W4Q_CTAS = 64;  // an SM before they loop; 8: 455 us at the size above

__global__ void __launch_bounds__(W4Q_THREADS) quantize_w4_rows_kernel(const uint16_t* __restrict__ w, int64_t words,
                                                                      int lane_bits, uint32_t* __restrict__ q,
                                                                      uint16_t* __restrict__ scale) {
    pdl_wait();
    pdl_trigger();
    const int64_t step = (int64_t)gridDim.x * W4Q_THREADS;
    // whole warps stay in the loop: a group, 2^lane_bits lanes, never straddles two of them
    const int64_t end = (words + 31) / 32 * 32;
    int64_t i = (int64_t)blockIdx.x * W4Q_THREADS + threadIdx.x;
    auto load = [&](int64_t at) {
        return at < words ? __ldg(reinterpret_cast<const uint4*>(w) + at) : make_uint4(0, 0, 0, 0);
    };
    uint4 next = load(i);
    for (; i < end; i += step) {
        float f[8];
        unpack8(next, f);
        next = load(i + step);
        float amax = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(f[j]));
        for (int b = 0; b < lane_bits; ++b) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1 << b));
        const uint32_t sb = pack_bf16x2(__fdiv_rn(amax, 7.0f), 0.f) & 0xFFFFu;
        float s = bf16_bits_to_float(sb);
        constexpr float ZERO = 0x1.8p23f + 8.f;  // its last four bits are those of code 0
        // (a scale below 2^-64 raised, and the elements with it, for a finite 1 / s)
        const float up = s < 0x1p-64f ? 0x1p64f : 1.f;
        s *= up;
        const float inv = s == 0.f ? 0.f : __frcp_rn(s), half = 0.5f * s;
        uint32_t word = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float v = f[j] * up;
            float c = fmaf(v, inv, ZERO);  // the nearest integer in the last bits
            const float d = fmaf(ZERO - c, s, v);
            if (fabsf(d) > half || (fabsf(d) == half && (__float_as_uint(c) & 1))) c += d < 0.f ? -1.f : 1.f;
            c = s == 0.f ? ZERO : fminf(fmaxf(c, ZERO - 8.f), ZERO + 7.f);
            word |= (__float_as_uint(c) & 15u) << (4 * (j / 2 + 4 * (j & 1)));
        }
        if (i < words) {
            q[i] = word;
            if ((i & ((1 << lane_bits) - 1)) == 0) scale[i >> lane_bits] = (uint16_t)sb;
        }
    }
}

// ---------------------------------------------------------------------------
// Products.  For one group of a weight row n and an activation row m
//
//   y[m][n] += s * sum_k c[n][k] x[m][k]
//
// the inner sum is an mma.sync chain in fp32 over the codes widened to bf16 (c / 64, exact)
// and the bf16 activations as they are (every product exact), the outer one an fp32 fused
// multiply-add per group; the matvec's y is rounded once, to bf16, the experts' y not at
// all.  FC1's h is rounded to bf16, the type that FC2's products take, as every other weight
// format of the layer rounds it: the workspace holds it at that width, and with the output's
// own rounding the experts are 2.3e-3 from 64 bits (2-norm; the output's alone 1.6e-3).
//
// The work is a list of tiles, 32 weight rows of one slot (FC1: 16 gate rows and the
// matching 16 up rows) times up to 8 C activation rows; a tile's K is cut into stages of
// 128.  Every CTA takes a contiguous range of the list, about the same number of stages
// each, and its 8 warps take equal contiguous ranges of those stages, whatever tiles they
// fall into.  A warp streams its stages through a ring of its own without a break at a
// tile's end; it stores the tiles that are all its own, and leaves its part of the at most
// two that it shares with its neighbours in shared memory, where the warp that ends a tile
// adds the parts in stage order.  (No atomics: a call repeats itself.  Where a sum over K is cut
// follows from the list: for a matrix from the sizes, and a row of up to 16 gives the same
// in any batch; for the experts also from the slots' rows, and a token's sums may be cut
// elsewhere in another batch.)
//
// Bound: HBM for the weights when they are many, else instruction issue.  A stage (2 KB of
// codes) takes a warp about 265 instructions (32768 x 7168 by one row with all else: 272), 144
// of them to widen (nine per word of eight codes),
// so the SMs together could take in 9 TB/s; at 16 warps an SM they issue in 0.6 of all
// cycles (the rest: the ALU's and the tensor pipe's turns, and latency).  Without the
// products, the loads alone, 65536 x 7168 takes 40 us.  tcgen05 would
// want the widened codes stored to shared memory and at least 128 rows a tile; registers
// feed mma.sync as they are, and a tile of 32 rows splits evenly at one row of activations.
// What else was measured for 65536 x 7168 by one row when it took 48 us: 24 warps an SM on
// 80 registers 59 us, 16 warps in one CTA no faster, the ring's loop unrolled by four
// slower (the instruction cache), codes as E4M3 pieces on m16n8k32 70 us, codes
// left as subnormals with activations scaled by a kernel in front 50 us.
//
// Measured (weights not in L2): 65536 x 7168, groups of 128, one row 42.8 .. 45.3 us (several
// boxes), 242 MB at 5.7 .. 5.3 TB/s; eight rows 46 .. 47 us, sixteen 67 .. 69 us; groups of 64
// 49, 53 and 105 us, of 32 77, 86 and 129 us.  Eight tokens, 8 of 256
// experts of 7168 x 2048: 217 .. 234 us for FC1, FC2 and the combine, 1.30 GB at 6.0 .. 5.6
// TB/s.  32 tokens, 6 of 64 experts of 2048 x 1408 and a shared one of 5632: 68 us (291 MB,
// 4.3 TB/s); one token of it 19.5 us (45 MB), most of it start-up: its 14080 and 7040 stages
// of FC1 and FC2 would take 6 and 4 us at that batch's rate, and the kernels alone and
// cold take 13.0, 12.2 and 6.3 us.
// ---------------------------------------------------------------------------
constexpr int W4_WARPS = 8;
constexpr int W4_THREADS = W4_WARPS * 32;
constexpr int W4_CTAS = 2;       // on an SM
constexpr int W4_RING = 4;       // stages in each warp's ring
constexpr int W4_STAGE = 2048;   // bytes of a stage: 32 rows of 128 elements
constexpr int W4_MAXG = 1024;    // slots
constexpr int W4_RUNS = 8;       // runs a warp has in hand: the copies are three stages ahead
// every warp's ring, then its parts of two shared tiles (8 C sums a lane)
constexpr size_t w4_smem_bytes(int C) { return (size_t)W4_WARPS * (W4_RING * W4_STAGE + 2 * 32 * 8 * C * 4); }

// Neighbouring tiles of the list with the same activation rows, from the first that a
// warp has a stage of.
struct W4Run {
    const uint8_t* wq;   // packed weights and scales of the first tile's first row
    const uint16_t* ws;
    int row0;            // first output row
    int n0, m;           // first output of the first tile, rows
    int tiles;
    bool routed;
};

// x / d for 0 <= x < 2^31 by the multiplier that the host made for d (w4_div: at most
// 2^(31 + shift) / d + 1, exact for 31-bit x by Granlund and Montgomery's bound): in 64 bits
// and as divisions, a warp's share of the work took it 1.0 us to find, so 0.5.
__device__ __forceinline__ int w4_over(int x, const W4Div& d) {
    return (int)(__umulhi(2 * (uint32_t)x, d.m) >> d.shift);
}

// a value that every lane of the warp has, said so
__device__ __forceinline__ int w4_uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }
__device__ __forceinline__ const uint8_t* w4_uniform(const uint8_t* p) {
    const uint64_t v = reinterpret_cast<uint64_t>(p);
    const uint32_t lo = w4_uniform((int)(uint32_t)v), hi = w4_uniform((int)(v >> 32));
    return reinterpret_cast<const uint8_t*>((uint64_t)hi << 32 | lo);
}

__device__ __forceinline__ void w4_cp16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void w4_prefetch_l2(const void* p) {
    asm volatile("prefetch.global.L2 [%0];" ::"l"(p) : "memory");
}
// 32 consecutive bytes; WIDE: p is a multiple of 32
template <bool WIDE>
__device__ __forceinline__ void w4_ld32(uint4& u, uint4& v, const void* p) {
    if (WIDE) {
        asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w), "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                     : "l"(p));
    } else {
        u = static_cast<const uint4*>(p)[0];
        v = static_cast<const uint4*>(p)[1];
    }
}
__device__ __forceinline__ void w4_cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void w4_cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint32_t w4_lds32(uint32_t addr) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void w4_lds64(uint32_t (&v)[2], uint32_t addr) {
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v[0]), "=r"(v[1]) : "r"(addr) : "memory");
}

// D = A B + C, A 16 x 16 (row), B 16 x 8 (column), bf16 inputs, fp32 sums
__device__ __forceinline__ void w4_mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1,
                                       const float (&c)[4]) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %11, %12, %13};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
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

// 32 elements of a stage: sum[column tile][half] += codes x activations.  u, v: the lane's
// words of rows g and g + 8 of both 16-row halves; x: its activations of each column tile.
template <int C8, int C>
__device__ __forceinline__ void w4_step(float (&sum)[C][2][4], const uint32_t (&u)[2], const uint32_t (&v)[2],
                                        const uint4 (&x)[C]) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const uint32_t A[4] = {w4_pair(u[r], 2 * h), w4_pair(v[r], 2 * h), w4_pair(u[r], 2 * h + 1),
                                   w4_pair(v[r], 2 * h + 1)};
#pragma unroll
            for (int c = 0; c < C8; ++c)
                w4_mma(sum[c][r], A, h ? x[c].z : x[c].x, h ? x[c].w : x[c].y, sum[c][r]);
        }
}

// The outputs of the tile at n0 from its accumulators [column tile][half][4], in units
// of 1/64: row g or g + 8 and column 2t or 2t + 1 as the product leaves them.  xrow: the activation row of each
// column, -1 for one that the tables got wrong (its outputs are zero).
template <bool SWIGLU, int C>
__device__ __forceinline__ void w4_store(const W4Problem& p, const W4Run& d, int n0, const int32_t* xrow,
                                         const float (&acc)[C][2][4]) {
    const int g = (threadIdx.x & 31) >> 2, t = threadIdx.x & 3;
    const int64_t N = p.N_out;
#pragma unroll
    for (int c = 0; c < 2 * C; ++c) {
        if (c == 2 && d.m <= 8) break;
        const int col = 8 * (c / 2) + 2 * t + c % 2;
        if (col >= d.m) continue;
        const bool ok = xrow[col] >= 0;  // (else the sums are of some other row, whose values may be NaN)
        const int64_t at = (int64_t)(d.row0 + col) * N + n0 + g;
        float v[2][2];
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int h = 0; h < 2; ++h) v[r][h] = ok ? acc[c / 2][r][2 * h + c % 2] * 64.f : 0.f;
        if (SWIGLU) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const float o = __fdividef(v[0][h], 1.0f + expf(-v[0][h])) * v[1][h];
                p.out_bf16[at + 8 * h] = (uint16_t)(pack_bf16x2(o, 0.f) & 0xFFFFu);
            }
        } else {
#pragma unroll
            for (int r = 0; r < 2; ++r)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (n0 + 16 * r + 8 * h + g >= N) continue;
                    if (p.out_f32)
                        p.out_f32[at + 16 * r + 8 * h] = v[r][h];
                    else
                        p.out_bf16[at + 16 * r + 8 * h] = (uint16_t)(pack_bf16x2(v[r][h], 0.f) & 0xFFFFu);
                }
        }
    }
}

// WIDE: an activation row's 32-byte pieces lie on 32 bytes and are fetched by one load each.
template <bool SWIGLU, int GS, int C, bool WIDE>
__global__ void __launch_bounds__(W4_THREADS, W4_CTAS) w4_kernel(const __grid_constant__ W4Launch a) {
    constexpr int ROWS = 8 * C;  // activation rows of a tile
    extern __shared__ __align__(128) uint8_t w4_smem[];
    __shared__ int32_t s_pre[W4_MAXG];  // routed tiles before each slot
    __shared__ int32_t s_off[W4_MAXG + 1];  // the slots' rows
    __shared__ int32_t s_part[W4_WARPS];
    __shared__ W4Run s_run[W4_WARPS][W4_RUNS + 1];            // in the last place, that of a tile
    __shared__ int32_t s_x[W4_WARPS][W4_RUNS + 1][ROWS];  // begun by an earlier warp; columns' activation rows
    constexpr int TN = SWIGLU ? 16 : 32;   // outputs of a tile
    constexpr int NF = 4 / GS;             // groups in a stage
    constexpr int WORDS = GS < 2 ? 1 : 2;  // consecutive words of a lane
    const int lane = threadIdx.x & 31, warp = w4_uniform(threadIdx.x >> 5);
    const int g = lane >> 2, t = lane & 3;
    // pieces rotate within a row of a stage so that the reads below meet every bank once
    const int sw = ((g >> 1) & 1) * 2 + (g >> 2);
    const uint32_t ring0 = smem_u32(w4_smem) + warp * (W4_RING * W4_STAGE);
    // part [warp][0: of a tile begun by an earlier warp, 1: of one begun here][2 C x 4 values][lane]
    float4* parts = reinterpret_cast<float4*>(w4_smem + W4_WARPS * W4_RING * W4_STAGE);
    // What a previous kernel may still be writing is waited for as late as the call allows:
    // the tables here, the weights before their first copy, the activations after it.
    if (!a.early && a.G > 0) {
        pdl_wait();
        pdl_trigger();
    }

    // the list: the dense problem's tiles, then the routed ones by slot; the row tiles of
    // one weight tile are neighbours
    const int rows_sh = (int)a.rows_sh, rows_cap = (int)a.rows_cap;
    const int ct_sh = (rows_sh + ROWS - 1) / ROWS;
    const int n_sh = (a.sh.K + 127) / 128, n_rt = (a.rt.K + 127) / 128;  // stages of a tile
    const int tiles_rt = (a.rt.N_out + TN - 1) / TN;
    const int list_sh = a.sh.wq ? (a.sh.N_out + TN - 1) / TN * ct_sh : 0;
    int list_rt = 0;
    if (a.G > 0) {
        constexpr int PER = W4_MAXG / W4_THREADS;
        const int s0 = threadIdx.x * PER;
        int n[PER], sum = 0;
        int lo = s0 <= a.G ? __ldg(a.offsets + s0) : 0;
        int ok = lo >= 0;  // ascending from 0 or more to rows_cap or less
        if (s0 <= a.G) s_off[s0] = lo;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            n[i] = 0;
            if (s0 + i < a.G) {
                const int hi = __ldg(a.offsets + s0 + i + 1);
                ok &= (hi >= lo) & (hi <= rows_cap);
                n[i] = (int)(((uint32_t)hi - (uint32_t)lo + ROWS - 1) / ROWS) * tiles_rt;
                lo = hi;
                if (i + 1 < PER || s0 + PER == a.G) s_off[s0 + i + 1] = hi;
            }
            sum += n[i];
        }
        int inc = sum;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, inc, off);
            if (lane >= off) inc += v;
        }
        // (offsets that descend or leave the rows would outgrow the list's count: no routed tile then)
        ok = __all_sync(0xffffffffu, ok);
        if (lane == 31) s_part[warp] = ok ? inc : -1;
        __syncthreads();
        int base = inc - sum, total = 0, bad = 0;
#pragma unroll
        for (int w = 0; w < W4_WARPS; ++w) {
            base += w < warp ? s_part[w] : 0;
            total += s_part[w];
            bad |= s_part[w];
        }
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            if (s0 + i < a.G) s_pre[s0 + i] = base;
            base += n[i];
        }
        list_rt = bad < 0 ? 0 : total;
        __syncthreads();
        if (bad < 0 && threadIdx.x == 0) report(a.status, MOE_ERR_DEVICE_BOUNDS);
    }
    // this CTA's tiles: from the first that starts at or after its share of the stages
    const int stages_sh = list_sh * n_sh, stages = stages_sh + list_rt * n_rt;
    const int share = w4_over(stages, a.by_grid), more = stages - share * (int)gridDim.x;  // (`more` CTAs: one more)
    auto first_tile = [&](int cta) {
        const int s = share * cta + min(cta, more);
        return s <= stages_sh ? w4_over(s + n_sh - 1, a.by_sh) : list_sh + w4_over(s - stages_sh + n_rt - 1, a.by_rt);
    };
    auto start_of = [&](int v) { return v <= list_sh ? v * n_sh : stages_sh + (v - list_sh) * n_rt; };
    const int base = start_of(first_tile(blockIdx.x));
    const int all = start_of(first_tile(blockIdx.x + 1)) - base;
    // this warp's stages: cnt from lo; the first one's tile
    const int lo = base + all * warp / W4_WARPS;
    const int cnt = base + all * (warp + 1) / W4_WARPS - lo;
    const int v0 = lo < stages_sh ? w4_over(lo, a.by_sh) : list_sh + w4_over(lo - stages_sh, a.by_rt);

    // Three cursors run over the stages: the copies three ahead, the activations and
    // scales one ahead, the products.  Each steps from tile to tile of a run by constants
    // and finds run i of the warp, when it gets there, at s_run[warp][i % W4_RUNS].  Stage
    // numbers count from lo.  (The loop is not unrolled over the ring: four copies of what
    // a tile's end takes overran the instruction cache, 3 of 8 stalled cycles.)
    W4Run* runs = s_run[warp];
    const int first = start_of(v0) - lo;  // where the first tile starts (<= 0)
    int next_v = v0;                      // the first tile past the runs so far
    int32_t xrow = 0;                     // the activation row (FC1: pair) of the run's column `lane`
    auto locate = [&](int i) {
        W4Run d;
        int64_t at = 0;  // the slot's first weight row
        int rows;        // its end
        int q, ct;       // tile of the slot, its row tiles
        if (next_v < list_sh) {
            q = next_v;
            d.routed = false;
            ct = ct_sh;
            d.row0 = 0;
            rows = rows_sh;
        } else {
            const int w = next_v - list_sh;
            // the last slot whose tiles begin at or before w: its 32, then itself
            int s_lo = 32 * lane;
            s_lo = 32 * (__popc(__ballot_sync(0xffffffffu, s_lo < a.G && s_pre[s_lo] <= w)) - 1);
            const int s_at = s_lo + lane;
            s_lo += __popc(__ballot_sync(0xffffffffu, s_at < a.G && s_pre[s_at] <= w)) - 1;
            d.routed = true;
            d.row0 = s_off[s_lo];
            rows = s_off[s_lo + 1];
            ct = (int)((uint32_t)(rows - d.row0 + ROWS - 1) / ROWS);
            q = w - s_pre[s_lo];
            at = s_lo * (SWIGLU ? 2 * (int64_t)a.rt.N_out : a.rt.N_out);
        }
        const W4Problem& p = d.routed ? a.rt : a.sh;
        const int tile = ct == 1 ? q : q / ct;
        d.n0 = tile * TN;
        d.row0 += (q - tile * ct) * ROWS;
        d.m = min(ROWS, rows - d.row0);
        d.wq = p.wq + (at + d.n0) * (p.K / 2);
        d.ws = p.ws + (at + d.n0) * (p.K / (32 * GS));
        // a last tile with fewer outputs stands alone: some of its rows repeat
        d.tiles = ct == 1 ? max(1, p.N_out / TN - tile) : 1;
        next_v += d.tiles;
        if (lane < ROWS) {  // (kept when the first copies are on their way)
            xrow = d.row0 + min(lane, d.m - 1);
            if (d.routed && a.perm_src) xrow = in_bounds(xrow, a.rows_cap, a.status) ? a.perm_src[xrow] : -1;
        }
        __syncwarp();
        if (lane == 0) runs[i % W4_RUNS] = d;
        __syncwarp();
    };
    auto row_of = [&](const W4Problem& p, const W4Run& d, int q) {  // weight row g + 8 q from the run's first
        const int r = q * 8 + g;
        return SWIGLU ? (q < 2 ? r : r - 16 + p.N_out) : min(r, p.N_out - 1 - d.n0);
    };

    // (bounds-checked library) the n bytes at p lie in the run's codes, scales or activations
    auto inside = [&](const void* p, const void* base, int64_t size, int n) {
        const int64_t at = static_cast<const uint8_t*>(p) - static_cast<const uint8_t*>(base);
        return in_bounds(at, size - n + 1, a.status);
    };
    auto codes_ok = [&](int run, const void* p) {
        const bool rt = runs[run % W4_RUNS].routed;
        const W4Problem& w = rt ? a.rt : a.sh;
        return inside(p, w.wq, (SWIGLU ? 2 : 1) * (int64_t)w.N_out * (rt ? a.G : 1) * (w.K / 2), 16);
    };
    auto scale_ok = [&](int run, const void* p) {
        const bool rt = runs[run % W4_RUNS].routed;
        const W4Problem& w = rt ? a.rt : a.sh;
        return inside(p, w.ws, (SWIGLU ? 2 : 1) * (int64_t)w.N_out * (rt ? a.G : 1) * (w.K / (32 * GS)) * 2, 2);
    };
    auto x_ok = [&](int run, const void* p, int n) {
        const bool rt = runs[run % W4_RUNS].routed;
        const W4Problem& w = rt ? a.rt : a.sh;
        return inside(p, w.x, (rt ? (a.perm_src ? a.T : a.rows_cap) : a.rows_sh) * w.K * 2, n);
    };
    auto tile_ok = [&](const W4Run& d, int n0) {
        const int64_t rows = d.routed ? a.rows_cap : a.rows_sh;
        const int N = d.routed ? a.rt.N_out : a.sh.N_out;
        return in_bounds(d.row0, rows, a.status) && in_bounds(d.row0 + d.m - 1, rows, a.status) &&
               in_bounds(SWIGLU ? n0 + TN - 1 : n0, N, a.status);
    };

    // rows g, g + 8 from the first base, g + 16, g + 24 (FC1: the up rows g, g + 8) from the second
    const uint8_t *w_base0 = nullptr, *w_base1 = nullptr;
    uint32_t woff[4];
    int w_run = -1, w_tiles = 1, w_end = first, w_n = 0, w_step = 0;
    bool w_cut = false;             // the lane's piece lies past the end of a row's last stage
    auto next_w = [&](int j) {  // the copies' next tile
        if (--w_tiles > 0) {
            w_base0 += w_step;
            if (SWIGLU) w_base1 += w_step;
        } else {
            locate(++w_run);
            const W4Run& d = runs[w_run % W4_RUNS];
            const W4Problem& p = d.routed ? a.rt : a.sh;
            w_n = w4_uniform(d.routed) ? n_rt : n_sh;
            w_tiles = w4_uniform(d.tiles);
            w_step = TN * (p.K / 2) - w_n * 64;
            w_cut = GS < 4 && t * 32 >= p.K - (w_n - 1) * 128;
            w_base0 = w4_uniform(d.wq) + (j - w_end) * 64;
            w_base1 = w_base0 + (SWIGLU ? (int64_t)p.N_out * (p.K / 2) : 0);
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int row = SWIGLU ? q % 2 * 8 + g : min(q * 8 + g, p.N_out - 1 - d.n0);
                woff[q] = row * (p.K / 2) + t * 16;
            }
        }
        w_end += w_n;
    };
    auto keep_rows = [&] {
        if (lane < ROWS) {
            int32_t r = xrow;
            if (runs[w_run % W4_RUNS].routed && a.perm_src) {  // FC1 reads the routing table for the rows
                const bool ok = r >= 0 && r < (int)(a.T * a.k);
                if (!ok) report(a.status, MOE_ERR_DEVICE_BOUNDS);
                r = ok ? w4_over(r, a.by_k) : -1;
            }
            s_x[warp][w_run % W4_RUNS][lane] = r;
        }
    };
    uint32_t w_off = 0, r_off = 0;  // ring stages written and read next
    const uint32_t w_slot = ring0 + g * 64 + ((t ^ sw) << 4), r_slot = ring0 + g * 64;
    bool w_open = false;  // the first tile's addresses stand
    auto issue = [&](int j) {
        if (j < cnt) {
            const int r = w_run;
            if (j == w_end || !w_open) next_w(j);
            w_open = true;
            if (GS == 4 || !(w_cut && j + 1 == w_end)) {
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint8_t* src = (SWIGLU && q >= 2 ? w_base1 : w_base0) + woff[q];
                    if (codes_ok(w_run, src)) w4_cp16(w_slot + w_off + q * 512, src);
                }
            }
            w_base0 += 64;
            if (SWIGLU) w_base1 += 64;
            if (r != w_run || j == 0) keep_rows();
        }
        w4_cp_commit();
        w_off = (w_off + W4_STAGE) & (W4_RING * W4_STAGE - 1);
    };
    if (!a.early && a.G == 0) {
        if (cnt > 0) {
            // the first stages' lines on their way to L2 meanwhile
            next_w(0);
            w_open = true;
            if (t == 0)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint8_t* p = (SWIGLU && q >= 2 ? w_base1 : w_base0) + woff[q];
                    w4_prefetch_l2(p);
                    if (w_end > 2) w4_prefetch_l2(p + 128);
                }
        }
        pdl_wait();
        pdl_trigger();
    }
#pragma unroll 1
    for (int j = 0; j < W4_RING - 1; ++j) issue(j);

    if (a.early) {  // the tables and the weights do not depend on the previous kernel, the activations do
        pdl_wait();
        pdl_trigger();
    }

    const uint16_t* xsrc[C] = {};    // the lane's activations, of column g of each eight (past the rows: the last)
    const uint16_t* ssrc = nullptr;  // the scales of weight row g + 8 t
    int p_run = -1, p_tiles = 1, p_end = first, p_n = 0, p_step = 0, p_m = 0;
    int p_cut = 0;  // elements of a row's last stage
    auto next_p = [&](int j) {  // the activations' and scales' next tile
        if (--p_tiles > 0) {  // (called with the pointers at the tile's last stage)
            ssrc += p_step;
#pragma unroll
            for (int c = 0; c < C; ++c) xsrc[c] -= (p_n - 1) * 128;
        } else {
            const W4Run& d = runs[++p_run % W4_RUNS];
            const W4Problem& p = d.routed ? a.rt : a.sh;
            __syncwarp();
            p_n = w4_uniform(d.routed) ? n_rt : n_sh;
            p_tiles = w4_uniform(d.tiles);
            p_m = w4_uniform(d.m);
            p_step = TN * (p.K / (32 * GS)) - (p_n - 1) * NF;
            p_cut = p.K - (p_n - 1) * 128;
            ssrc = d.ws + (int64_t)row_of(p, d, t) * (p.K / (32 * GS)) + (j - p_end) * NF;
#pragma unroll
            for (int c = 0; c < C; ++c)
                xsrc[c] = p.x + (int64_t)max(s_x[warp][p_run % W4_RUNS][8 * c + g], 0) * p.K + (j - p_end) * 128 +
                          t * 8 * WORDS;
        }
        p_end += p_n;
    };
    // A stage is two halves of two steps of 32 elements; the lane's word of a step is its word
    // of the half's t-th pair of words, or (groups of 32) the t-th word of the step.  Scales
    // are fetched a stage ahead, activations as far as registers allow: a stage, or with
    // sixteen columns half of one.
    constexpr int AHEAD = C == 1 ? 4 : 2;  // steps
    uint4 xb[AHEAD][C];
    uint32_t sb[NF];
    auto load_x = [&](int step, int has) {  // of the stage at xsrc, which holds `has` elements
        if (step / GS * 32 * GS < has) {  // (has = 0: there is no such stage, and xsrc may lie past x)
#pragma unroll
            for (int c = 0; c < C; ++c) {
                if (c && p_m <= 8) continue;
                if (GS < 2) {
                    if (x_ok(p_run, xsrc[c] + step * 32, 16))
                        xb[step % AHEAD][c] = *reinterpret_cast<const uint4*>(xsrc[c] + step * 32);
                } else if (step % 2) {  // both steps of a half: a lane's 32 consecutive bytes
                    if (x_ok(p_run, xsrc[c] + step / 2 * 64, 32))
                        w4_ld32<WIDE>(xb[step % AHEAD - 1][c], xb[step % AHEAD][c], xsrc[c] + step / 2 * 64);
                }
            }
        }
    };
    auto load_s = [&](int f, int has) {
        if (f * 32 * GS < has && scale_ok(p_run, ssrc + f)) sb[f] = __ldg(ssrc + f);
    };
    float acc[C][2][4] = {};
    int left = 0;  // elements of the stage that is multiplied next
    int run = 0, tiles = 0, n0 = 0, end = 0, n = 0, m = 0;
    if (cnt > 0) {
        next_p(0);
        left = GS < 4 && p_end == 1 ? p_cut : 128;
#pragma unroll
        for (int f = 0; f < NF; ++f) load_s(f, left);
#pragma unroll
        for (int j = 0; j < AHEAD; ++j) load_x(j, left);
        tiles = w4_uniform(runs[0].tiles);
        n0 = runs[0].n0;
        m = w4_uniform(runs[0].m);
        n = w4_uniform(runs[0].routed) ? n_rt : n_sh;
        end = first + n;
    }
    bool begun = first < 0;  // the tile in hand was begun by an earlier warp
    bool ended = false;      // and this one ended it

    // the products of stage i, in column tiles of a tile's rows
    auto multiply = [&](int i, auto columns) {
        constexpr int C8 = decltype(columns)::value;
        const uint32_t slot = r_slot + r_off;
        float sum[C][2][4];
        int next = 0;  // elements of the next stage
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            if (half == 2 - AHEAD / 2) {  // from here on the next stage's activations and scales are fetched
                if (i + 1 == p_end && i + 1 < cnt) {
                    next_p(i + 1);
                } else {
#pragma unroll
                    for (int c = 0; c < C; ++c) xsrc[c] += 128;
                    ssrc += NF;
                }
                next = i + 1 < cnt ? (GS < 4 && i + 2 == p_end ? p_cut : 128) : 0;
            }
            uint32_t w[4][2];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                if constexpr (GS < 2) {
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        w[q][j] = w4_lds32(slot + q * 512 + (((half * 2 + j) ^ sw) << 4) + t * 4);
                } else {
                    w4_lds64(w[q], slot + q * 512 + (((half * 2 + (t >> 1)) ^ sw) << 4) + (t & 1) * 8);
                }
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int step = 2 * half + j, f = step / GS;
                if (step % GS == 0) {
#pragma unroll
                    for (int e = 0; e < 8 * C8; ++e) sum[e >> 3][(e >> 2) & 1][e & 3] = 0.f;
                }
                if (GS == 4 || f * 32 * GS < left) {
                    const uint32_t u[2] = {w[0][j], w[2][j]}, v[2] = {w[1][j], w[3][j]};
                    w4_step<C8, C>(sum, u, v, xb[step % AHEAD]);
                    if (step % GS == GS - 1) {
                        const float mine = bf16_bits_to_float(sb[f]);
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const float sc = __shfl_sync(0xffffffffu, mine, (lane & 28) | q);
                            const int r = q >> 1, h = 2 * (q & 1);
#pragma unroll
                            for (int c = 0; c < C8; ++c) {
                                acc[c][r][h] = fmaf(sc, sum[c][r][h], acc[c][r][h]);
                                acc[c][r][h + 1] = fmaf(sc, sum[c][r][h + 1], acc[c][r][h + 1]);
                            }
                        }
                    }
                }
                // the registers take the values of AHEAD steps on
                if (step + AHEAD >= 4)
                    load_x((step + AHEAD) % 4, next);
                else
                    load_x(step + AHEAD, left);
            }
        }
#pragma unroll
        for (int f = 0; f < NF; ++f) load_s(f, next);
        left = next;
    };

#pragma unroll 1
    for (int i = 0; i < cnt; ++i) {
        issue(i + W4_RING - 1);
        w4_cp_wait<W4_RING - 1>();
        __syncwarp();
        if (C == 1 || m <= 8)
            multiply(i, std::integral_constant<int, 1>());
        else
            multiply(i, std::integral_constant<int, C>());
        __syncwarp();  // the ring slot just read is the next one written
        r_off = (r_off + W4_STAGE) & (W4_RING * W4_STAGE - 1);
        if (i + 1 == end || i + 1 == cnt) {  // the tile's last stage here
            const W4Run& d = runs[run % W4_RUNS];
            if (!begun && i + 1 == end) {
                if (tile_ok(d, n0))
                    w4_store<SWIGLU, C>(d.routed ? a.rt : a.sh, d, n0, s_x[warp][run % W4_RUNS], acc);
            } else {
                float4* o = parts + (warp * 2 + (begun ? 0 : 1)) * (64 * C) + lane;
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    if (c && d.m <= 8) break;
#pragma unroll
                    for (int r = 0; r < 2; ++r)
                        o[(2 * c + r) * 32] = make_float4(acc[c][r][0], acc[c][r][1], acc[c][r][2], acc[c][r][3]);
                }
                if (begun && i + 1 == end) {
                    ended = true;
                    if (lane == 0) runs[W4_RUNS] = d;
                    if (lane < ROWS) s_x[warp][W4_RUNS][lane] = s_x[warp][run % W4_RUNS][lane];
                }
            }
#pragma unroll
            for (int e = 0; e < 8 * C; ++e) acc[e >> 3][(e >> 2) & 1][e & 3] = 0.f;
            begun = false;
            if (--tiles > 0) {
                n0 += TN;
            } else if (i + 1 < cnt) {
                const W4Run& next_d = runs[++run % W4_RUNS];
                tiles = w4_uniform(next_d.tiles);
                n0 = next_d.n0;
                m = w4_uniform(next_d.m);
                n = w4_uniform(next_d.routed) ? n_rt : n_sh;
            }
            end += n;
        }
    }
    w4_cp_wait<0>();
    __syncthreads();

    // the parts of the tile that this warp ended, in stage order
    if (ended) {
        const int start = lo + first - base;                     // of the tile among the CTA's stages
        const int w0 = (W4_WARPS * (start + 1) - 1) / all;       // the warp that began it
        for (int w = w0; w <= warp; ++w) {
            if (all * w / W4_WARPS == all * (w + 1) / W4_WARPS) continue;  // a warp without stages
            const float4* o = parts + (w * 2 + (w == w0 ? 1 : 0)) * (64 * C) + lane;
#pragma unroll
            for (int c = 0; c < C; ++c) {
                if (c && runs[W4_RUNS].m <= 8) break;
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float4 f = o[(2 * c + r) * 32];
                    acc[c][r][0] += f.x;
                    acc[c][r][1] += f.y;
                    acc[c][r][2] += f.z;
                    acc[c][r][3] += f.w;
                }
            }
        }
        const W4Run& d = runs[W4_RUNS];
        if (tile_ok(d, d.n0)) w4_store<SWIGLU, C>(d.routed ? a.rt : a.sh, d, d.n0, s_x[warp][W4_RUNS], acc);
    }
}

// ---------------------------------------------------------------------------
// Combine: out[t] = bf16( sum_j w[t][j] y[row] + g_t shared[t] ), fixed j order,
// g_t = 1 / (1 + exp(-x[t] gate_w)) or 1.
//
// Bound: latency.  k + 1 fp32 rows are read per token, from L2 where FC2 has just left
// them; the tables and the gate are read and summed before FC2 is waited for.  From FC2's
// end to its own 2.8 us at one token, 3.2 us at 32 (H = 2048, k = 6: 1.8 MB), of which 1.5 us
// is the kernels' handover.  y is fp32: rounding it to bf16 here would add an error of the
// size of the output's own rounding for every expert.
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
    const unsigned grid = (unsigned)std::max<int64_t>(1, std::min<int64_t>(want, (int64_t)num_sms * W4Q_CTAS));
    return launch_k("quantize_w4_rows", quantize_w4_rows_kernel, dim3(grid), dim3(W4Q_THREADS), 0, s, w, words,
                    group == 32 ? 2 : group == 64 ? 3 : 4, reinterpret_cast<uint32_t*>(q), scale);
}

static W4Div w4_div(int d) {
    W4Div r = {d, 0, 0};
    if (d <= 0) return r;
    while ((int64_t(1) << r.shift) < d) ++r.shift;
    r.m = (uint32_t)((uint64_t(1) << (31 + r.shift)) / (uint64_t)d + 1);
    return r;
}

template <bool SWIGLU, int GS, int C, bool WIDE>
static cudaError_t launch_w4_tiles(const W4Launch& L, int num_sms, cudaStream_t s) {
    // the shared-memory limit is set once per device
    static std::atomic<bool> ready[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!ready[dev].load(std::memory_order_acquire)) {
        e = cudaFuncSetAttribute(w4_kernel<SWIGLU, GS, C, WIDE>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)w4_smem_bytes(C));
        if (e != cudaSuccess) return e;
        ready[dev].store(true, std::memory_order_release);
    }
    // No more CTAs than tiles, and no fewer stages to a CTA than its longest tile has
    // (between one CTA an SM and as many as fit).  The rows are on the GPU: a routed slot is
    // taken to have one row tile, so a few slots with more get fewer CTAs than tiles (one of
    // 2048 x 768 with 32 rows 13.3 us, 11.3 on a grid for all its tiles; but a grid for all that
    // T k pairs could make costs a rank with one of 64 slots, 32 tokens, 11.3 us for 10.1).
    constexpr int TN = SWIGLU ? 16 : 32;
    const int n_sh = (L.sh.K + 127) / 128, n_rt = (L.rt.K + 127) / 128;
    const double sh = L.sh.wq ? (double)((L.sh.N_out + TN - 1) / TN) * ((L.rows_sh + 8 * C - 1) / (8 * C)) : 0.0;
    const double rt = L.G > 0 ? (double)((L.rt.N_out + TN - 1) / TN) * std::min<int64_t>(L.rows_cap, L.G) : 0.0;
    const double even = (sh * n_sh + rt * n_rt) / std::max(sh > 0 ? n_sh : 1, rt > 0 ? n_rt : 1);
    const double most = std::min(sh + rt, (double)W4_CTAS * num_sms);
    const unsigned grid = (unsigned)std::max(1.0, std::min(most, std::max(even, (double)num_sms)));
    W4Launch K = L;
    K.by_grid = w4_div((int)grid);
    K.by_sh = w4_div(n_sh);
    K.by_rt = w4_div(n_rt);
    K.by_k = w4_div(L.k);
    return launch_k(L.name, w4_kernel<SWIGLU, GS, C, WIDE>, dim3(grid), dim3(W4_THREADS), w4_smem_bytes(C), s, K);
}

template <bool SWIGLU, int GS>
static cudaError_t launch_w4_rows(const W4Launch& L, int num_sms, cudaStream_t s) {
    // Passes over the weights in pieces of 8 and of 16 rows (a slot holds rows_cap / G rows on
    // average; fewer on a rank whose pairs are partly other ranks'): one of 16 takes 1.44 times
    // as long as one of 8 with groups of 128 (65536 x 7168: 67 and 47 us; 24 rows as two of 16
    // 117 us, as three of 8 133; 32 tokens over 64 experts, 3 rows to a slot and
    // 32 for the shared one, in pieces of 8 68 us, of 16 84).  Groups of 32: 1.49 (86 and 129 us).
    // Groups of 64: 2.0 (53 and 105 us); 9 to 16 rows stay one piece all the same, so that a
    // row of them gives the same in any batch.
    const double sh = L.sh.wq ? (double)L.sh.N_out * L.sh.K : 0.0;
    const double slots = (double)std::min<int64_t>(L.G, L.rows_cap);
    const double rt = slots * L.rt.N_out * L.rt.K, mean = slots > 0 ? L.rows_cap / slots : 0.0;
    auto passes = [&](double rows) { return sh * std::ceil(L.rows_sh / rows) + rt * std::max(1.0, mean / rows); };
    const bool narrow = passes(8) <= 1.44 * passes(16);
    // 32-byte loads of x where it allows them (half the requests: 65536 x 7168 by 16 rows 66 us,
    // by 16-byte loads 70); groups of 32 take 16 bytes of a row at a time
    if (GS > 1 && (((uintptr_t)L.sh.x | (uintptr_t)L.rt.x) & 31) == 0)
        return narrow ? launch_w4_tiles<SWIGLU, GS, 1, (GS > 1)>(L, num_sms, s)
                      : launch_w4_tiles<SWIGLU, GS, 2, (GS > 1)>(L, num_sms, s);
    return narrow ? launch_w4_tiles<SWIGLU, GS, 1, false>(L, num_sms, s)
                  : launch_w4_tiles<SWIGLU, GS, 2, false>(L, num_sms, s);
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

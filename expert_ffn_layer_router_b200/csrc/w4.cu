// w4.cu -- 4-bit weights with group scales: quantising, reading back, and the expert FFN over
// them (sm_100a).
//
// Format of a weight [E, N, K].  Columns are cut into groups of G = 32, 64 or 128 (the last may
// be short); group g of row n of expert e has a scale s and, optionally, an offset z, both
// bfloat16, stored [E, ceil(K / G), N].  A weight's value is s (q - 8) + z, q its nibble.  The
// nibbles are 32-bit words [E, N, 16 ceil(K / 128)]: word 4 t + j of 128-column chunk c holds
// columns 128 c + 32 j + 8 t + i, i = 0..7, column i in bits 4 (4 (i % 2) + i / 2) and up;
// columns past K hold 8.  The order is the one the products want: a lane's 16-byte load gives it
// 8 columns of each of the chunk's four 32-column groups, and a mask takes two neighbouring
// columns out of a word at once.
//
// The products, y_n = sum_k W_nk x_k for the few rows x an expert has in decoding, are bound by
// the bytes of W: each is read once, half a byte.  See w4_gemm_kernel.
#include <algorithm>
#include <cstdint>
#include <type_traits>

#include <cuda.h>

#include "common.cuh"
#include "kernels.h"
#include "tmap.h"

namespace moe {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kSm = 148;

__device__ __forceinline__ float bf16_bits(uint32_t v) { return __uint_as_float(v << 16); }
__device__ __forceinline__ uint16_t bf16_round(float v) {
    const __nv_bfloat16 b = __float2bfloat16_rn(v);
    return *reinterpret_cast<const uint16_t*>(&b);
}

// ------------------------------------------------------------------------------------------------
// Quantising: per group, without offsets s = bf16(max|w| * f32(1/7)); with offsets s = bf16((max -
// min) * f32(1/15)) and z = bf16(min + 8 s).  (Products with the float32 reciprocal, which is how
// float32 tensors are divided by a number elsewhere, so scales made there agree bit for bit.)  q - 8 =
// round-half-even((w - z) / s) clamped to [-8, 7], 0 where s = 0.  The rounding of s and z to
// bfloat16 (they are what is kept) comes before the division, so it costs at most half a step more.
//
// The quotients.  With i = 1 / s rounded once and t = w i, the corrected t + (w - t s) i (two fused
// steps) is the correctly rounded quotient (P. Markstein, "Computation of elementary functions on the
// IBM RISC System/6000 processor", 1990), so halves are met exactly; where s is so small that its
// reciprocal or the remainder leaves the normal range, a thread divides.  Adding 1.5 * 2^23 + 8
// rounds t half to even and leaves q in the low bits; the eight words of bits are joined as
// acc = 16 acc + bits modulo 2^32, and the constant's share is taken off at the end.
// (64 x 1024 x 2048 from bfloat16, 0.34 GB moved: 90 us, 52 at the copy bandwidth; issue-bound.  With a
// division near halves 143 us, half of the warps meeting one.)
// ------------------------------------------------------------------------------------------------
// A NaN reaches its group's extremes (and so the scale), and an infinity makes the scale infinite; both
// take the dividing path, whose nibbles stay in their places.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float min_nan(float a, float b) {
    float r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

constexpr float kRound = 12582920.0f;                  // 1.5 * 2^23 + 8 (even: halves stay halves)
constexpr uint32_t kRoundBits = 0x4b400008u - 8u;      // its bits, without the 8

template <class T>
__device__ __forceinline__ void unpack8(const uint4 (&raw)[sizeof(T) / 2], float (&f)[8]) {
#pragma unroll
    for (int q = 0; q < (int)sizeof(T) / 2; ++q) {
        const uint32_t u[4] = {raw[q].x, raw[q].y, raw[q].z, raw[q].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (sizeof(T) == 2) {
                f[2 * i] = __uint_as_float(u[i] << 16);
                f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
            } else {
                f[4 * q + i] = __uint_as_float(u[i]);
            }
        }
    }
}

// A block takes 32 rows x 4 chunks of one expert; 16 lanes hold a chunk of a row (8 columns each),
// so a group's extremes are log2(G / 8) shuffles.  Scales and offsets are staged to leave as
// 64-byte runs.
constexpr int kQRows = 32, kQChunks = 4;

// Bits of a nibble: column i of a word sits at 4 (4 (i % 2) + i / 2).
__device__ __forceinline__ constexpr int column_at(int nibble) {
    return nibble < 4 ? 2 * nibble : 2 * (nibble - 4) + 1;
}

template <class T, bool ZERO, int G>
__global__ void __launch_bounds__(256)
    w4_quantize_kernel(const T* __restrict__ W, int N, int K, int row_tiles,
                       uint32_t* __restrict__ q, uint16_t* __restrict__ scale,
                       uint16_t* __restrict__ zero) {
    pdl_begin();
    constexpr int kPer = 128 / G, kLanes = G / 8;
    __shared__ uint16_t s_scale[kQChunks * kPer][kQRows], s_zero[kQChunks * kPer][kQRows];
    const int e = blockIdx.y / row_tiles, n0 = (blockIdx.y - e * row_tiles) * kQRows;
    const int chunk0 = blockIdx.x * kQChunks, C = (K + 127) / 128;
    const int half = threadIdx.x >> 4, l = threadIdx.x & 15;
    const int c = chunk0 + half % kQChunks, k = c * 128 + l * 8;
    const float kInf = __int_as_float(0x7f800000);
    const T* src = W + ((long long)e * N + n0) * K + k;
    uint32_t* dst = q + ((long long)e * N + n0) * (16LL * C) + 16 * c + 4 * (l & 3) + (l >> 2);
    // (16 half-warps: 4 rows a step, 8 steps, the loads of kAhead of them in flight together)
    constexpr int kAhead = sizeof(T) == 2 ? 8 : 4;
#pragma unroll 1
    for (int step = 0; step < 8; step += kAhead) {
        uint4 raw[kAhead][sizeof(T) / 2];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int r = half / kQChunks + 4 * (step + i);
            const bool in = n0 + r < N && k < K;            // K is a multiple of 64
#pragma unroll
            for (int p = 0; p < (int)sizeof(T) / 2; ++p)
                raw[i][p] = in ? reinterpret_cast<const uint4*>(src + (long long)r * K)[p]
                               : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            const int r = half / kQChunks + 4 * (step + i);
            const bool in = n0 + r < N && k < K;
            float v[8];
            unpack8<T>(raw[i], v);
            // (A group past K or N gives scale 0 and is not stored.  The columns of a group of up to
            // 64 are all in or all out; in one of 128 the zeros past K could change only extremes
            // with offsets, which leave them out.)
            float s, z = 0.0f;
            if constexpr (ZERO) {
                float lo = in ? v[0] : kInf, hi = in ? v[0] : -kInf;
#pragma unroll
                for (int i = 1; i < 8; ++i) {
                    lo = min_nan(lo, in ? v[i] : kInf);
                    hi = max_nan(hi, in ? v[i] : -kInf);
                }
#pragma unroll
                for (int h = 1; h < kLanes; h *= 2) {
                    lo = min_nan(lo, __shfl_xor_sync(kFull, lo, h));
                    hi = max_nan(hi, __shfl_xor_sync(kFull, hi, h));
                }
                const bool any = !(hi < lo);
                s = any ? bf16_bits(bf16_round(__fmul_rn(__fsub_rn(hi, lo), 1.0f / 15.0f))) : 0.0f;
                z = any ? bf16_bits(bf16_round(__fadd_rn(lo, __fmul_rn(8.0f, s)))) : 0.0f;
            } else {
                float top = fabsf(v[0]);
#pragma unroll
                for (int i = 1; i < 8; ++i) top = max_nan(top, fabsf(v[i]));
#pragma unroll
                for (int h = 1; h < kLanes; h *= 2)
                    top = max_nan(top, __shfl_xor_sync(kFull, top, h));
                s = bf16_bits(bf16_round(__fmul_rn(top, 1.0f / 7.0f)));
            }
            const float inv = __frcp_rn(s);
            uint32_t acc = 0;
#pragma unroll
            for (int b = 7; b >= 0; --b) {                  // nibble b, from the highest
                const float w = ZERO ? __fsub_rn(v[column_at(b)], z) : v[column_at(b)];
                float t = __fmul_rn(w, inv);
                t = __fmaf_rn(__fmaf_rn(-t, s, w), inv, t);
                if constexpr (ZERO) t = fminf(fmaxf(t, -8.0f), 7.0f);
                acc = acc * 16u + __float_as_uint(__fadd_rn(t, kRound));
            }
            uint32_t word = acc - kRoundBits * 0x11111111u;
            // (without offsets |t| stays below 7.1 for such s, so nothing has to be clamped)
            if (!(s > 7.9e-31f && s < kInf)) {
                word = 0;
#pragma unroll
                for (int b = 0; b < 8; ++b) {
                    const float w = ZERO ? __fsub_rn(v[column_at(b)], z) : v[column_at(b)];
                    const float t = fminf(fmaxf(rintf(__fdiv_rn(w, s)), -8.0f), 7.0f);
                    word |= (uint32_t)((int)(s > 0.0f ? t : 0.0f) + 8) << (4 * b);
                }
            }
            if (!in) word = 0x88888888u;
            if (n0 + r < N && c < C) dst[(long long)r * 16 * C] = word;
            if (l % kLanes == 0) {
                s_scale[half % kQChunks * kPer + l / kLanes][r] =
                    (uint16_t)(__float_as_uint(s) >> 16);
                if (ZERO)
                    s_zero[half % kQChunks * kPer + l / kLanes][r] =
                        (uint16_t)(__float_as_uint(z) >> 16);
            }
        }
    }
    __syncthreads();
    const int groups = (K + G - 1) / G;
    for (int i = threadIdx.x; i < kQChunks * kPer * kQRows; i += 256) {
        const int g = chunk0 * kPer + i / kQRows, n = n0 + i % kQRows;
        if (g < groups && n < N) {
            const long long o = ((long long)e * groups + g) * N + n;
            scale[o] = s_scale[i / kQRows][i % kQRows];
            if (ZERO) zero[o] = s_zero[i / kQRows][i % kQRows];
        }
    }
}

// The two columns of pair i (columns 2 i, 2 i + 1) of a word, as exact bfloat16 integers q - 8:
// 0x4300 | q is 128 + q, and 136 is subtracted.  One lop3 needs both constants in registers;
// `Unpack` holds them where the compiler cannot see their values (it splits the lop3 otherwise).
struct Unpack {
    uint32_t mask, magic;
    __device__ __forceinline__ Unpack() {
        asm volatile("mov.b32 %0, 0x000f000f;" : "=r"(mask));
        asm volatile("mov.b32 %0, 0x43004300;" : "=r"(magic));
    }
    __device__ __forceinline__ uint32_t pair(uint32_t word, int i) const {
        uint32_t u;
        asm("lop3.b32 %0, %1, %2, %3, 0xea;"
            : "=r"(u)
            : "r"(word >> (4 * i)), "r"(mask), "r"(magic));
        const uint32_t k136 = 0x43084308u;
        const __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&u),
                                         *reinterpret_cast<const __nv_bfloat162*>(&k136));
        return *reinterpret_cast<const uint32_t*>(&r);
    }
};

// Values in bfloat16, [E, N, K], on the quantiser's tiles: a lane per word (8 columns, one 16-byte
// store; 16 lanes write 256 bytes in a row).  53 us for 64 x 1024 x 2048; its bytes take 52 at the copy
// bandwidth.  Without offsets the product s (q - 8) is exact in
// 12 bits, so the bfloat16 multiply rounds it once, like the float32 one.
template <bool ZERO, int G>
__global__ void __launch_bounds__(256)
    w4_dequantize_kernel(const uint32_t* __restrict__ q, const uint16_t* __restrict__ scale,
                         const uint16_t* __restrict__ zero, int N, int K, int row_tiles,
                         uint16_t* __restrict__ W) {
    pdl_begin();
    constexpr int kPer = 128 / G;
    __shared__ uint16_t s_scale[kQChunks * kPer][kQRows], s_zero[kQChunks * kPer][kQRows];
    const int e = blockIdx.y / row_tiles, n0 = (blockIdx.y - e * row_tiles) * kQRows;
    const int chunk0 = blockIdx.x * kQChunks, C = (K + 127) / 128, groups = (K + G - 1) / G;
    const Unpack unpack;
    const int half = threadIdx.x >> 4, l = threadIdx.x & 15, cc = half % kQChunks;
    const int c = chunk0 + cc;
    const uint32_t* src = q + ((long long)e * N + n0) * (16LL * C) + 16 * c + l;
    uint32_t word[kQRows / 4];
#pragma unroll
    for (int i = 0; i < kQRows / 4; ++i) {
        const int r = half / kQChunks + 4 * i;
        word[i] = n0 + r < N && c < C ? src[(long long)r * 16 * C] : 0;
    }
    for (int i = threadIdx.x; i < kQChunks * kPer * kQRows; i += 256) {
        const int g = chunk0 * kPer + i / kQRows, n = n0 + i % kQRows;
        const bool in = g < groups && n < N;
        const long long o = in ? ((long long)e * groups + g) * N + n : 0;
        s_scale[i / kQRows][i % kQRows] = in ? scale[o] : 0;
        if (ZERO) s_zero[i / kQRows][i % kQRows] = in ? zero[o] : 0;
    }
    __syncthreads();
    const int kk = (l & 3) * 32 + (l >> 2) * 8, k = c * 128 + kk;
    if (k >= K) return;
    uint16_t* dst = W + ((long long)e * N + n0) * K + k;
#pragma unroll
    for (int i = 0; i < kQRows / 4; ++i) {
        const int r = half / kQChunks + 4 * i;
        if (n0 + r >= N) break;
        const uint16_t sb = s_scale[cc * kPer + kk / G][r];
        uint32_t o[4];
        if constexpr (ZERO) {
            const float s = bf16_bits(sb), z = bf16_bits(s_zero[cc * kPer + kk / G][r]);
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                const uint32_t v = unpack.pair(word[i], p);
                o[p] = pack_bf16x2(fmaf(s, __uint_as_float(v << 16), z),
                                   fmaf(s, __uint_as_float(v & 0xffff0000u), z));
            }
        } else {
            const uint32_t s2 = sb * 0x10001u;
#pragma unroll
            for (int p = 0; p < 4; ++p) {
                const uint32_t v = unpack.pair(word[i], p);
                const __nv_bfloat162 r2 = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&v),
                                                  *reinterpret_cast<const __nv_bfloat162*>(&s2));
                o[p] = *reinterpret_cast<const uint32_t*>(&r2);
            }
        }
        *reinterpret_cast<uint4*>(dst + (long long)r * K) = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

// ------------------------------------------------------------------------------------------------
// The grouped products: D[r, n] = act(sum_k W[e]_nk A[row(r), k] + bias[e][n]) for the rows r of
// each expert e.
//
// A unit is (expert, 32 UG features, up to 32 / KS rows); persistent blocks (two per SM) of 8 product
// warps and two copying warps take equal runs of the list of units.  A step of a unit is KS chunks
// of 128 columns (KS = 2, 4 or 8, UG = 8 / KS): warp w works on 32 features (w / KS) and on
// chunk w % KS of the step; the KS sums are added through shared memory in a fixed order at the
// unit's end.  Many units: KS = 2; few (one token): KS = 8 spreads K over the warps.
//
// Features are the M side of mma.m16n8k16 (weights are the A operand: lane (g, t) owns features
// g + 8 r, r < 4, of the 32), rows the N side, so 8 rows cost one instruction per 16 x 16 weights.
// The integers q - 8 are exact in bfloat16, so a group's products are exact and their fp32 sum is
// scaled once per group; offsets multiply the sum of x over the group, which an all-ones operand
// gives.
//
// The copying warps fill a ring of stages that runs ahead across units: one the weights (tensor-map
// copies of 128-byte rows: 64-byte rows took twice as long, the copy engine moves a row in about 4
// cycles), one scales and rows (16-byte cp.async: bulk copies are issued lane by lane, and 20 of them
// took longer than a step's products).  Full / empty barriers hand the stages over.  Every wait is
// bounded; one that runs out records MOE_DEV_TIMEOUT and the block finishes without waiting any
// more.
//
// Measured, 64 experts of 2048 x 1024 (134 million weights, 72 MB with scales of 64 columns), 64
// tokens, 8 experts each: 28-31 us a product, 2.5 TB/s of weights.  What bounds it is the
// chain of a chunk (4096 weights: barrier, loads from shared memory, unpacking, products) with the 5
// warps per scheduler that 96 registers leave room for: its instructions, about 400, of which the
// unpacking takes 176 (7 of the integer unit, which starts one every second cycle, and 4 of the
// half-precision one a word), are issued in 45-50% of the cycles.  The copies alone take 16 us.  More
// than 16 rows of an expert are more units, each of which unpacks its weights again: the time grows
// with the rows (both products: 82 us at 16 rows, 136 at 32, 225 at 64).  On the way:
// K split over all 8 warps with rows from global memory 78 us; group sizes as template arguments (a
// runtime division is 30 instructions) 37; rows through the L1 cache 41; 16 product warps in one block
// per SM 33; KS as a template argument too: 4-6% less at every batch; a unit's offsets from shared
// memory: 1-3% less.  Unpacking into tensor memory for tcgen05 products was tried and took 42: at 16
// rows a product of 16 columns takes 40 cycles, and the barriers of a 16 KB stage half a microsecond.
// (At 32 rows an expert, where this kernel unpacks a weight twice, it was the faster one: 120 against
// 139 us for both products.)
// ------------------------------------------------------------------------------------------------
enum W4Epi { kW4SiLU = 0, kW4Bias = 1, kW4SwiGLU = 2 };

struct W4Args {
    const uint16_t* A;        // [*, K] bfloat16
    const int32_t* a_rows;    // nullable: A row of row r is a_rows[r]
    int a_row_limit;
    const int32_t* offsets;   // [E + 1]
    int E, K, N;              // N: rows of W per expert (2 F when gated)
    int max_rows;
    const uint16_t* scale;
    const uint16_t* zero;     // nullable
    const float* bias;        // [E, N], nullable
    uint16_t* D;
    int ldd;
    bool early;               // the launch before this one wrote A alone: all else may start first
    DeviceStatus* st;
};

constexpr int kWarps = 8;                          // product warps
constexpr int kThreads = (kWarps + 2) * 32;
constexpr int kStages = 3;
constexpr int kLines = 16;                         // row pieces of a stage (rows x boxes)
constexpr int kLineBytes = 512 + 64;               // 256 columns, padded: neighbours differ in bank
constexpr int kStageX = kLines * kLineBytes;
constexpr int kStageW = 128 * 128;                 // 32 UG features x KS chunks of 128 columns
constexpr int kRedStride = 36;                     // floats per row of the partial sums
constexpr int kRedBytes = kWarps * 8 * kRedStride * 4;

// A stage: weights (128-byte rows, 16-byte pieces swizzled by the row), rows, scales (and offsets).
template <int G>
constexpr int kSideBytes = 256 * (256 / G);
template <bool ZERO, int G>
constexpr int kStageBytes =
    kStageW + kStageX + ((ZERO ? 2 : 1) * kSideBytes<G> + 1023) / 1024 * 1024;
// (1024 bytes to align the ring; row pointers of the unit being copied; the list of units and the
// offsets; a flag)
template <bool ZERO, int G>
constexpr int w4_smem_bytes(int E) {
    return 1024 + kStages * kStageBytes<ZERO, G> + kRedBytes + 2 * kStages * 8 + kLines * 8 +
           (2 * E + 3) * 4;
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// d = a b (no accumulator to clear first).
__device__ __forceinline__ void mma_bf16_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                               uint32_t b1) {
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}

__device__ __forceinline__ float silu(float v) { return v / (1.0f + __expf(-v)); }

// A unit's place: expert, feature block, first row of the row tile, rows in it.
struct Unit { int e, fb, row0, rows; };

template <int EPI, bool ZERO, int G, int LKS>
struct W4Kernel {
    static constexpr int KS = 1 << LKS;           // warps that share a unit's K
    static constexpr int UG = kWarps / KS;        // groups of 32 features of a unit
    static constexpr int row_tile = 2 * kLines / KS;
    static constexpr int kTiles = LKS == 1 ? 2 : 1;          // 8-row tiles of a unit
    static constexpr int kPer = 256 / G;          // groups of a box
    const W4Args& a;
    const int* s_pre;         // units before each expert
    const int* s_off;         // the offsets
    int S, groups, nfb;       // 256-column boxes of K, groups of K, feature blocks

    __device__ __forceinline__ Unit unit_at(int u) const {
        int lo = 0, hi = a.E - 1;                 // largest e with s_pre[e] <= u
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (s_pre[mid] <= u) lo = mid; else hi = mid - 1;
        }
        const int r0 = s_off[lo], r1 = s_off[lo + 1];
        const int tiles = (r1 - r0 + row_tile - 1) / row_tile;
        const int i = u - s_pre[lo];
        Unit x;
        x.e = lo;
        x.fb = i / tiles;                         // row tiles of one feature block are neighbours:
        x.row0 = r0 + (i - x.fb * tiles) * row_tile;      // its weights are in the cache
        x.rows = min(row_tile, r1 - x.row0);
        return x;
    }
    // First rows of W of the two halves of a unit's features (gated: gate rows, up rows).
    __device__ __forceinline__ int first(const Unit& u, int h) const {
        constexpr int half = 16 * UG;
        if constexpr (EPI == kW4SwiGLU) return h ? a.N / 2 + u.fb * half : u.fb * half;
        return u.fb * 2 * half + h * half;
    }

    // ---- product warps ----
    // acc[n][m] += the products of this warp's chunk of a step for NT tiles of 8 rows; lane
    // (g, t) of group ug: sums of features g + 16 m (+ 8) for rows 2 t, 2 t + 1 of tile n.
    template <int NT>
    __device__ __forceinline__ void chunk(const uint8_t* wl,
                                          const uint8_t* sl, const uint8_t* xl,
                                          const Unpack& unpack, float (&acc)[kTiles][2][4]) const {
        // r-th feature of the lane: 8 rows on, and 16 UG rows on between gate and up.
        constexpr int up = EPI == kW4SwiGLU ? 16 * UG : 16;
        uint4 w[4];
#pragma unroll
        for (int r = 0; r < 4; ++r)
            w[r] = *reinterpret_cast<const uint4*>(wl + ((r & 1) * 8 + (r >> 1) * up) * 128);
        float part[NT][2][4], sum[NT][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const bool first = j * 32 % G == 0;
            uint32_t p[4][4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const uint32_t word = j == 0 ? w[r].x : j == 1 ? w[r].y : j == 2 ? w[r].z
                                                                                 : w[r].w;
#pragma unroll
                for (int i = 0; i < 4; ++i) p[r][i] = unpack.pair(word, i);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const uint4 v =
                    *reinterpret_cast<const uint4*>(xl + n * 8 * kLineBytes + j * 64);
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    const uint32_t a0[4] = {p[2 * m][0], p[2 * m + 1][0], p[2 * m][1],
                                            p[2 * m + 1][1]};
                    const uint32_t a1[4] = {p[2 * m][2], p[2 * m + 1][2], p[2 * m][3],
                                            p[2 * m + 1][3]};
                    if (first) mma_bf16_first(part[n][m], a0, v.x, v.y);
                    else mma_bf16(part[n][m], a0, v.x, v.y);
                    mma_bf16(part[n][m], a1, v.z, v.w);
                }
                if constexpr (ZERO) {
                    const uint32_t one[4] = {0x3f803f80u, 0x3f803f80u, 0x3f803f80u,
                                             0x3f803f80u};
                    if (first) mma_bf16_first(sum[n], one, v.x, v.y);
                    else mma_bf16(sum[n], one, v.x, v.y);
                    mma_bf16(sum[n], one, v.z, v.w);
                }
            }
            if ((j + 1) * 32 % G == 0) {
                const uint8_t* s = sl + j * 32 / G * (64 * UG);
                float sc[4], zo[4];
#pragma unroll
                for (int r = 0; r < 4; ++r) {
                    const int at = ((r & 1) * 8 + (r >> 1) * up) * 2;
                    sc[r] = bf16_bits(*reinterpret_cast<const uint16_t*>(s + at));
                    if constexpr (ZERO)
                        zo[r] = bf16_bits(*reinterpret_cast<const uint16_t*>(
                            s + kSideBytes<G> + at));
                }
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int m = 0; m < 2; ++m)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            acc[n][m][i] = fmaf(sc[2 * m + i / 2], part[n][m][i], acc[n][m][i]);
                            if constexpr (ZERO)
                                acc[n][m][i] = fmaf(zo[2 * m + i / 2], sum[n][i], acc[n][m][i]);
                        }
            }
        }
    }
    // Bias, activation and the store of one row's sums: v[r] of feature g + 8 r of 32-feature
    // block b (gated: gate g, gate g + 8, up g, up g + 8 of 16).
    __device__ __forceinline__ void store(const Unit& x, int b, int g, int row,
                                          const float (&sums)[4]) const {
        uint16_t* out = a.D + (long long)(x.row0 + row) * a.ldd;
        const float* bias = a.bias ? a.bias + (long long)x.e * a.N : nullptr;
        const int f = (EPI == kW4SwiGLU ? b * 16 : b * 32) + g;
        float v[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const int n = EPI == kW4SwiGLU ? f + 8 * (r & 1) + (r >> 1) * (a.N / 2) : f + 8 * r;
            v[r] = sums[r] + (bias ? bias[n] : 0.0f);
        }
        if constexpr (EPI == kW4SwiGLU) {
            out[f] = bf16_round(silu(v[0]) * v[2]);
            out[f + 8] = bf16_round(silu(v[1]) * v[3]);
        } else {
#pragma unroll
            for (int r = 0; r < 4; ++r)
                out[f + 8 * r] = bf16_round(EPI == kW4SiLU ? silu(v[r]) : v[r]);
        }
    }
};

template <int EPI, bool ZERO, int G, int LKS>
__global__ void __launch_bounds__(kThreads, 2)
    w4_gemm_kernel(const __grid_constant__ CUtensorMap tm, const W4Args args) {
    extern __shared__ __align__(16) uint8_t smem_raw[];
    constexpr int kStage = kStageBytes<ZERO, G>;
    uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
    float* red = reinterpret_cast<float*>(smem + kStages * kStage);
    const uint32_t bars = smem_u32(red) + kRedBytes;
    auto full_bar = [&](int s) { return bars + 8u * s; };
    auto empty_bar = [&](int s) { return bars + 8u * (kStages + s); };
    const uint16_t** s_row = reinterpret_cast<const uint16_t**>(
        reinterpret_cast<uint8_t*>(red) + kRedBytes + 2 * kStages * 8);
    int* s_pre = reinterpret_cast<int*>(s_row + kLines);
    int* s_off = s_pre + args.E + 1;
    int* s_bad = s_off + args.E + 1;
    using Kernel = W4Kernel<EPI, ZERO, G, LKS>;
    constexpr int KS = Kernel::KS, UG = Kernel::UG, row_tile = Kernel::row_tile;
    constexpr int kTiles = Kernel::kTiles, NB = KS / 2;      // (NB: 256-column boxes of a step)
    Kernel w{args, s_pre, s_off};
    w.S = (args.K + 255) / 256;
    w.groups = (args.K + G - 1) / G;
    w.nfb = (args.N / 32 + UG - 1) / UG;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int E = args.E;
    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            mbar_init(full_bar(s), 1 + 32);      // the weights' bytes; each lane's own copies
            mbar_init(empty_bar(s), kWarps);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("prefetch.tensormap [%0];" ::"l"(&tm) : "memory");
    }
    // Second product: offsets and weights were complete before the first one began (it waited for
    // its predecessors), so the list of units is made and weights are copied while the first one's
    // last blocks run; the warp that copies the rows waits for it.
    if (!args.early) pdl_begin();
    if (warp == 0) {
        // Units before each expert; offsets are checked as the grouped GEMM does: 0 first,
        // non-decreasing, at most max_rows.  Bad offsets: nothing is computed or stored.
        int total = 0;
        bool bad = false;
        if (lane == 0)
            bad = args.offsets[0] != 0 || args.offsets[E] > args.max_rows;
        for (int e0 = 0; e0 < E; e0 += 32) {
            const int e = e0 + lane;
            const int r0 = args.offsets[min(e, E)], r1 = args.offsets[min(e + 1, E)];
            if (e <= E) s_off[e] = r0;
            bad |= r1 < r0;                              // (their difference may wrap)
            const int n = max(r1 - r0, 0);
            const int units = (n + row_tile - 1) / row_tile * w.nfb;
            int inc = units;
#pragma unroll
            for (int h = 1; h < 32; h *= 2) {
                const int o = __shfl_up_sync(kFull, inc, h);
                if (lane >= h) inc += o;
            }
            if (e < E) s_pre[e] = total + inc - units;
            total += __shfl_sync(kFull, inc, 31);
        }
        bad = __any_sync(kFull, bad);
        if (lane == 0) {
            s_pre[E] = total;
            s_off[E] = args.offsets[E];
            *s_bad = bad;
            if (bad && blockIdx.x == 0) report(args.st, MOE_DEV_BAD_INDEX, 710);
        }
    }
    __syncthreads();
    if (*s_bad) {
        if (args.early) pdl_begin();
        return;
    }
    const int total = s_pre[E];
    // Equal runs of units.  Blocks i and i + 148 usually share an SM: they take neighbouring runs, so
    // that an SM's two shares add up to within one unit of the others'.
    const int run = (int)(blockIdx.x % kSm * 2 + blockIdx.x / kSm);
    const int u0 = (int)((long long)total * run / gridDim.x);
    const int u1 = (int)((long long)total * (run + 1) / gridDim.x);

    if (warp == kWarps) {
        // ---- copies the weights ----
        if (lane == 0) {
            int slot = 0;
            uint32_t phase = 0, issued = 0;
            constexpr int half = 16 * UG;
            bool ok = true;
            for (int u = u0; u < u1 && ok; ++u) {
                const Unit x = w.unit_at(u);
                const int r0 = x.e * args.N + w.first(x, 0), r1 = x.e * args.N + w.first(x, 1);
                for (int c = 0; c < w.S; c += NB) {
                    ok = mbar_wait(empty_bar(slot), phase ^ 1u, args.st, 71);
                    if (!ok) break;
                    // (features past the end: rows of the next expert, not used)
                    const int boxes = min(NB, w.S - c);
                    uint32_t dst = smem_u32(smem) + slot * kStage;
                    mbar_arrive_expect_tx(full_bar(slot), (uint32_t)(boxes * 2 * half * 128));
                    for (int q = 0; q < boxes; ++q, dst += 2 * half * 128) {
                        tma_load_2d(dst, &tm, full_bar(slot), (c + q) * 64, r0);
                        tma_load_2d(dst + half * 128, &tm, full_bar(slot), (c + q) * 64, r1);
                    }
                    ++issued;
                    if (++slot == kStages) {
                        slot = 0;
                        phase ^= 1u;
                    }
                }
            }
            // The last copies must land before the block's shared memory goes away, also when a
            // wait gave up and the product warps no longer wait for them (bounded again).
            for (uint32_t i = issued - min(issued, (uint32_t)kStages); i < issued; ++i) {
                const uint64_t t0 = global_ns();
                while (!mbar_try_wait(full_bar(i % kStages), (i / kStages) & 1u) &&
                       global_ns() - t0 < kWaitLimitNs) {}
            }
        }
        return;
    }
    if (warp == kWarps + 1) {
        // ---- copies scales and rows: lane l the 16-byte piece l of every line of rows ----
        if (args.early) pdl_begin();
        int slot = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int u = u0; u < u1 && ok; ++u) {
            const Unit x = w.unit_at(u);
            // Rows of the lines (box line / row_tile, row line % row_tile; null: no row).
            const bool two = LKS > 1 || x.rows > 8;           // (else lines 8 .. 15 are not read)
            __syncwarp();
            if (lane < kLines) {
                const int rr = lane % row_tile;
                const uint16_t* src = nullptr;
                if (rr < x.rows) {
                    int r = x.row0 + rr;
                    if (args.a_rows) {
                        r = args.a_rows[r];
                        if (r < 0 || r >= args.a_row_limit) {
                            report(args.st, MOE_DEV_BAD_INDEX, 720);
                            r = -1;
                        }
                    }
                    if (r >= 0)
                        src = args.A + (long long)r * args.K + lane / row_tile * 256;
                }
                s_row[lane] = src;
            }
            __syncwarp();
            // The lane's piece of each line; a line without a row is never copied (zeros).
            const uint16_t* line[kLines];
            uint32_t there = 0;
#pragma unroll
            for (int i = 0; i < kLines; ++i) {
                const uint16_t* src = s_row[i];
                there |= (src != nullptr ? 1u : 0u) << i;
                line[i] = src ? src + lane * 8 : args.A;
            }
            // Scales: piece i of the lane belongs to group i KS + lg of the step; 8 features from
            // f (past the end: none).
            const int lg = lane / (4 * UG), piece = lane % (4 * UG);
            const int f = w.first(x, piece >= 2 * UG) + piece % (2 * UG) * 8;
            const long long per_step = (long long)KS * args.N;
            long long side = ((long long)x.e * w.groups + lg) * args.N + f;
            int left = f < args.N ? w.groups - lg : 0;       // groups from this lane's first on
            int cols = args.K - lane * 8;                    // columns from this lane's piece on
            for (int c = 0; c < w.S; c += NB, cols -= NB * 256) {
                ok = __all_sync(kFull, mbar_wait(empty_bar(slot), phase ^ 1u, args.st, 73));
                if (!ok) break;
                const uint32_t dst = smem_u32(smem) + slot * kStage + kStageW + lane * 16;
#pragma unroll
                for (int i = 0; i < kLines; ++i) {
                    if (i == 8 && !two) break;
                    const bool in = ((there >> i) & 1u) && cols > i / row_tile * 256;
                    cp_async_16z(dst + i * kLineBytes, line[i], in ? 16 : 0);
                    if (cols > NB * 256) line[i] += NB * 256;    // (stays inside the row)
                }
#pragma unroll
                for (int i = 0; i < Kernel::kPer / 2; ++i) {
                    const bool in = left > 0;
                    const uint32_t d = dst + kStageX + 32 * i * 16;
                    cp_async_16z(d, args.scale + (in ? side : 0), in ? 16 : 0);
                    if constexpr (ZERO)
                        cp_async_16z(d + kSideBytes<G>, args.zero + (in ? side : 0), in ? 16 : 0);
                    side += per_step;
                    left -= KS;
                }
                cp_async_arrive_noinc(full_bar(slot));
                if (++slot == kStages) {
                    slot = 0;
                    phase ^= 1u;
                }
            }
        }
        cp_async_commit();
        cp_async_wait<0>();
        return;
    }

    const int g = lane >> 2, t = lane & 3, ug = warp / KS, ks = warp % KS;
    const Unpack unpack;
    // This lane's places in a stage: first feature's words, its scale, its row of the first tile.
    // (With KS > 4 a box has fewer than 8 rows; lanes of the columns past them read other lines, or
    // what lies behind the last one: their sums are not used.)
    const int box = ks >> 1, h = ks & 1;
    const int frow = EPI == kW4SwiGLU ? ug * 16 + g : ug * 32 + g;
    const int w_at = (box * 32 * UG + frow) * 128 + (((h * 4 + t) ^ g) << 4);
    const int x_at = kStageW + (box * row_tile + g) * kLineBytes + h * 256 + t * 16;
    const int s_at = kStageW + kStageX + (box * (256 / G) + h * (128 / G)) * 64 * UG + frow * 2;
    int slot = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int u = u0; u < u1; ++u) {
        const Unit x = w.unit_at(u);
        const int nt = kTiles == 1 ? 1 : (x.rows + 7) / 8;
        const int bl = x.fb * UG + ug;
        const bool feat = bl * 32 < args.N;
        float acc[kTiles][2][4];
#pragma unroll
        for (int n = 0; n < kTiles; ++n)
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[n][m][i] = 0.0f;
#pragma unroll 1
        for (int c = 0; c < w.S; c += NB) {
            if (ok) ok = __all_sync(kFull, mbar_wait(full_bar(slot), phase, args.st, 72));
            if (ok && feat && (c + box) * 256 + h * 128 < args.K) {
                const uint8_t* stage = smem + slot * kStage;
                if (nt == 1)
                    w.template chunk<1>(stage + w_at, stage + s_at, stage + x_at, unpack, acc);
                else if constexpr (kTiles == 2)
                    w.template chunk<2>(stage + w_at, stage + s_at, stage + x_at, unpack, acc);
            }
            // (A warp that gave up frees no stage: the copying warps then issue nothing over copies
            // that have not landed, and find the last of them by the barriers' parity.)
            __syncwarp();
            if (ok && lane == 0) mbar_arrive(empty_bar(slot));
            if (++slot == kStages) {
                slot = 0;
                phase ^= 1u;
            }
        }
        // acc[n][m][i]: row 2 t + i % 2 of tile n, feature g + 16 m + 8 (i / 2).
#pragma unroll
        for (int n = 0; n < kTiles; ++n) {
            if (n >= nt) break;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float* mine = red + (warp * 8 + 2 * t + i) * kRedStride + g;
#pragma unroll
                for (int q = 0; q < 4; ++q) mine[8 * q] = acc[n][q >> 1][i + 2 * (q & 1)];
            }
            asm volatile("bar.sync 1, 256;" ::: "memory");
            // Thread i < 64 UG joins 4 features of a row: (group, row, g).
            const int i = threadIdx.x, jg = i >> 6, row = (i >> 3) & 7, fg = i & 7;
            const int jb = x.fb * UG + jg;
            if (ok && jg < UG && n * 8 + row < x.rows && jb * 32 < args.N) {
                const float* s = red + (jg * KS * 8 + row) * kRedStride + fg;
                float v[4] = {s[0], s[8], s[16], s[24]};
                for (int q = 1; q < KS; ++q)
#pragma unroll
                    for (int r = 0; r < 4; ++r) v[r] += s[q * 8 * kRedStride + 8 * r];
                w.store(x, jb, fg, n * 8 + row, v);
            }
            asm volatile("bar.sync 1, 256;" ::: "memory");
        }
    }
}

template <int EPI, bool ZERO, int G, int LKS>
cudaError_t run_w4(const CUtensorMap& tm, const W4Args& a, cudaStream_t s) {
    auto kern = w4_gemm_kernel<EPI, ZERO, G, LKS>;
    const int smem = w4_smem_bytes<ZERO, G>(a.E);
    static std::atomic<int> allowed[64];
    const cudaError_t e = allow_smem(kern, allowed, smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3(2 * kSm), dim3(kThreads), smem, s, tm, a);
}

// Calls f(first expert, experts, grid) for the tiles of E experts: row tiles on y (at most 65535 a
// launch), chunks on x.
template <class F>
void w4_tiles(int E, int N, int K, F f) {
    const int row_tiles = (N + kQRows - 1) / kQRows, C = (K + 127) / 128;
    const int per = 65535 / row_tiles;
    for (int e0 = 0; e0 < E; e0 += per) {
        const int ne = std::min(per, E - e0);
        f(e0, row_tiles, dim3((C + kQChunks - 1) / kQChunks, ne * row_tiles));
    }
}

// f(bool constant, group constant)
template <class F>
void w4_format(bool zero, int G, F f) {
    auto with = [&](auto z) {
        if (G == 32) f(z, std::integral_constant<int, 32>());
        else if (G == 64) f(z, std::integral_constant<int, 64>());
        else f(z, std::integral_constant<int, 128>());
    };
    if (zero) with(std::true_type());
    else with(std::false_type());
}

}  // namespace

void launch_w4_quantize(int dtype, const void* W, int E, int N, int K, int G, uint32_t* q,
                        uint16_t* scale, uint16_t* zero, cudaStream_t s, int* launches) {
    const long long words = 16LL * ((K + 127) / 128), groups = (K + G - 1) / G;
    w4_tiles(E, N, K, [&](int e0, int row_tiles, dim3 grid) {
        const long long rows = (long long)e0 * N;
        w4_format(zero != nullptr, G, [&](auto z, auto g) {
            constexpr bool Z = decltype(z)::value;
            constexpr int kG = decltype(g)::value;
            uint16_t* zp = Z ? zero + rows * groups : nullptr;
            if (dtype == MOE_BF16)
                launch_pdl(w4_quantize_kernel<uint16_t, Z, kG>, grid, dim3(256), 0, s,
                           (const uint16_t*)W + rows * K, N, K, row_tiles, q + rows * words,
                           scale + rows * groups, zp);
            else
                launch_pdl(w4_quantize_kernel<float, Z, kG>, grid, dim3(256), 0, s,
                           (const float*)W + rows * K, N, K, row_tiles, q + rows * words,
                           scale + rows * groups, zp);
        });
        *launches += 1;
    });
}

void launch_w4_dequantize(const uint32_t* q, const uint16_t* scale, const uint16_t* zero, int E,
                          int N, int K, int G, void* W, cudaStream_t s, int* launches) {
    const long long words = 16LL * ((K + 127) / 128), groups = (K + G - 1) / G;
    w4_tiles(E, N, K, [&](int e0, int row_tiles, dim3 grid) {
        const long long rows = (long long)e0 * N;
        w4_format(zero != nullptr, G, [&](auto z, auto g) {
            constexpr bool Z = decltype(z)::value;
            launch_pdl(w4_dequantize_kernel<Z, decltype(g)::value>, grid, dim3(256), 0, s,
                       q + rows * words, scale + rows * groups,
                       Z ? zero + rows * groups : (const uint16_t*)nullptr, N, K, row_tiles,
                       (uint16_t*)W + rows * K);
        });
        *launches += 1;
    });
}

cudaError_t launch_w4_gemm(int which, const void* A, const int32_t* a_rows, int a_row_limit,
                           const int32_t* offsets, int E, int K, int N, int max_rows,
                           const uint32_t* q, const uint16_t* scale, const uint16_t* zero, int G,
                           const float* bias, void* D, int ldd, DeviceStatus* st, cudaStream_t s,
                           int* launches) {
    W4Args a{(const uint16_t*)A, a_rows, a_row_limit, offsets, E, K, N, max_rows, scale, zero,
             bias, (uint16_t*)D, ldd, a_rows == nullptr, st};
    // Warps that share a unit's K: the fewest that give every SM a unit, at most 8 and no more than
    // there are chunks.  (Both products, 64 experts of 2048 x 1024, KS = 2, 4, 8: 1 token 22, 17,
    // 16 us; 2 tokens 23, 20, 23; 4 tokens 29, 30, 33; 64 tokens 64, 77, 152.)
    int lks = 1;
    while (lks < 3 && (256 << lks) <= K &&
           (long long)std::min(E, max_rows) * (N / 32) < (long long)kSm * (kWarps >> lks))
        lks += 1;
    // Words as 16-bit pairs: boxes of 128 bytes (256 columns) x 16 UG rows.
    const int cols = 32 * ((K + 127) / 128);
    CUtensorMap tm;
    if (!make_tmap_2d(&tm, q, (long long)E * N, cols, cols, 64, 16 * (kWarps >> lks),
                      CU_TENSOR_MAP_SWIZZLE_128B))
        return note_launch(cudaErrorInvalidValue);
    cudaError_t e = cudaSuccess;
    w4_format(zero != nullptr, G, [&](auto z, auto g) {
        auto with = [&](auto epi) {
            constexpr int EPI = decltype(epi)::value, kG = decltype(g)::value;
            constexpr bool Z = decltype(z)::value;
            e = lks == 1   ? run_w4<EPI, Z, kG, 1>(tm, a, s)
                : lks == 2 ? run_w4<EPI, Z, kG, 2>(tm, a, s)
                           : run_w4<EPI, Z, kG, 3>(tm, a, s);
        };
        if (which == kW4SiLU) with(std::integral_constant<int, kW4SiLU>());
        else if (which == kW4Bias) with(std::integral_constant<int, kW4Bias>());
        else with(std::integral_constant<int, kW4SwiGLU>());
    });
    *launches += 1;
    return e;
}

}  // namespace moe

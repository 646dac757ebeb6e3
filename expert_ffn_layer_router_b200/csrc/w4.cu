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

#include "common.cuh"
#include "kernels.h"

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
// Quantising: per group, without offsets s = bf16(max|w| / 7); with offsets s = bf16((max - min) /
// 15) and z = bf16(min + 8 s).  q - 8 = round-half-even((w - z) / s) clamped to [-8, 7], 0 where
// s = 0.  The rounding of s and z to bfloat16 (they are what is kept) comes before the division,
// so it costs at most half a step more.
// ------------------------------------------------------------------------------------------------

// rint(a / s) as the IEEE quotient rounds, without a division unless the quotient is near a half:
// a * (1 / s) is within 2^-22 relative of it, and |quotient| < 16 where it matters.
__device__ __forceinline__ float quotient_rint(float a, float s, float inv) {
    float t = a * inv;
    const float f = t - truncf(t);
    if (fabsf(fabsf(f) - 0.5f) < 1e-4f || !(fabsf(t) < 64.0f)) t = __fdiv_rn(a, s);
    return rintf(t);
}

template <class T>
__device__ __forceinline__ void load8(const T* p, float (&f)[8]);
template <>
__device__ __forceinline__ void load8<float>(const float* p, float (&f)[8]) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}
template <>
__device__ __forceinline__ void load8<uint16_t>(const uint16_t* p, float (&f)[8]) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(u[i] << 16);
        f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
    }
}

// A block takes 32 rows x 4 chunks of one expert; 16 lanes hold a chunk of a row (8 columns each),
// so a group's extremes are log2(G / 8) shuffles.  Scales and offsets are staged to leave as
// 64-byte runs.
constexpr int kQRows = 32, kQChunks = 4;

template <class T>
__global__ void __launch_bounds__(256)
    w4_quantize_kernel(const T* __restrict__ W, int N, int K, int G, int row_tiles,
                       uint32_t* __restrict__ q, uint16_t* __restrict__ scale,
                       uint16_t* __restrict__ zero) {
    pdl_begin();
    __shared__ uint16_t s_scale[kQChunks * 4][kQRows], s_zero[kQChunks * 4][kQRows];
    const int e = blockIdx.y / row_tiles, n0 = (blockIdx.y % row_tiles) * kQRows;
    const int chunk0 = blockIdx.x * kQChunks, C = (K + 127) / 128;
    const int half = threadIdx.x >> 4, l = threadIdx.x & 15;
    const int lanes = G / 8, gpc = 128 / G;             // lanes per group, groups per chunk
    const float kInf = __int_as_float(0x7f800000);
#pragma unroll 2
    for (int it = half; it < kQRows * kQChunks; it += 16) {
        const int c = chunk0 + it % kQChunks, r = it / kQChunks, n = n0 + r;
        const int k = c * 128 + l * 8;
        const bool in = n < N && k < K;                 // K is a multiple of 64
        float v[8];
        if (in) {
            load8<T>(W + ((long long)e * N + n) * K + k, v);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = 0.0f;
        }
        float lo = kInf, hi = -kInf;
        if (in) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                lo = fminf(lo, v[i]);
                hi = fmaxf(hi, v[i]);
            }
        }
        for (int h = 1; h < lanes; h *= 2) {
            lo = fminf(lo, __shfl_xor_sync(kFull, lo, h));
            hi = fmaxf(hi, __shfl_xor_sync(kFull, hi, h));
        }
        uint16_t sb = 0, zb = 0;
        if (hi >= lo) {
            if (zero) {
                sb = bf16_round(__fdiv_rn(__fsub_rn(hi, lo), 15.0f));
                zb = bf16_round(__fadd_rn(lo, __fmul_rn(8.0f, bf16_bits(sb))));
            } else {
                sb = bf16_round(__fdiv_rn(fmaxf(hi, -lo), 7.0f));
            }
        }
        const float s = bf16_bits(sb), z = bf16_bits(zb), inv = 1.0f / s;
        uint32_t word = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            float t = 0.0f;
            if (in && s > 0.0f)
                t = fminf(fmaxf(quotient_rint(__fsub_rn(v[i], z), s, inv), -8.0f), 7.0f);
            word |= (uint32_t)((int)t + 8) << (4 * (4 * (i & 1) + i / 2));
        }
        if (n < N && c < C)
            q[((long long)e * N + n) * (16LL * C) + 16 * c + 4 * (l & 3) + (l >> 2)] = word;
        if (l % lanes == 0) {
            s_scale[(it % kQChunks) * gpc + l / lanes][r] = sb;
            s_zero[(it % kQChunks) * gpc + l / lanes][r] = zb;
        }
    }
    __syncthreads();
    const int groups = (K + G - 1) / G;
    for (int i = threadIdx.x; i < kQChunks * gpc * kQRows; i += 256) {
        const int g = chunk0 * gpc + i / kQRows, n = n0 + i % kQRows;
        if (g < groups && n < N) {
            const long long o = ((long long)e * groups + g) * N + n;
            scale[o] = s_scale[i / kQRows][i % kQRows];
            if (zero) zero[o] = s_zero[i / kQRows][i % kQRows];
        }
    }
}

// The two columns of pair i (columns 2 i, 2 i + 1) of a word, as exact bfloat16 integers q - 8:
// 0x4300 | q is 128 + q, and 136 is subtracted.
__device__ __forceinline__ uint32_t w4_pair(uint32_t word, int i) {
    const uint32_t u = ((word >> (4 * i)) & 0x000f000fu) | 0x43004300u;
    const uint32_t k136 = 0x43084308u;
    const __nv_bfloat162 r = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&u),
                                     *reinterpret_cast<const __nv_bfloat162*>(&k136));
    return *reinterpret_cast<const uint32_t*>(&r);
}

// Values in bfloat16, [E, N, K]: a thread per word (8 columns, one 16-byte store).
__global__ void __launch_bounds__(256)
    w4_dequantize_kernel(const uint32_t* __restrict__ q, const uint16_t* __restrict__ scale,
                         const uint16_t* __restrict__ zero, int N, int K, int G,
                         long long words, uint16_t* __restrict__ W) {
    pdl_begin();
    const int C = (K + 127) / 128, groups = (K + G - 1) / G;
    for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < words;
         i += (long long)gridDim.x * 256) {
        const long long row = i / (16 * C);
        const int w = (int)(i - row * (16 * C));
        const int k = (w >> 4) * 128 + (w & 3) * 32 + ((w >> 2) & 3) * 8;
        if (k >= K) continue;
        const uint32_t word = q[i];
        const long long e = row / N, at = (e * groups + k / G) * N + (row - e * N);
        const float s = bf16_bits(scale[at]), z = zero ? bf16_bits(zero[at]) : 0.0f;
        uint32_t o[4];
#pragma unroll
        for (int p = 0; p < 4; ++p) {
            const uint32_t v = w4_pair(word, p);
            o[p] = pack_bf16x2(fmaf(s, __uint_as_float(v << 16), z),
                               fmaf(s, __uint_as_float(v & 0xffff0000u), z));
        }
        *reinterpret_cast<uint4*>(W + row * K + k) = make_uint4(o[0], o[1], o[2], o[3]);
    }
}

// ------------------------------------------------------------------------------------------------
// The grouped products: D[r, n] = act(sum_k W[e]_nk A[row(r), k] + bias[e][n]) for the rows r of
// each expert e.
//
// A unit is (expert, 32 * UG features, up to 32 rows); persistent blocks of 8 warps take equal
// runs of the list of units.  Warp w works on 32 features (group w / KS) and every KS-th 128-column
// chunk of K; the KS partial sums are added through shared memory in a fixed order at the end of
// the unit.  Features are the M side of mma.m16n8k16 (weights as the A operand: lane (g, t) owns
// features 4 g .. 4 g + 3 of the 32), rows the N side, so 8 rows cost one instruction per 16 x 16
// weights.  The integers q - 8 are exact in bfloat16, so the products of a group are exact and
// their fp32 sum is scaled once per group; offsets multiply the sum of x over the group, which an
// all-ones operand gives.
//
// Weights and scales come through a ring of cp.async stages private to each warp (each lane copies
// the 16-byte pieces it uses itself), which runs ahead across units, so the stream of weights
// never waits for the ends of units.
// ------------------------------------------------------------------------------------------------
enum W4Epi { kW4SiLU = 0, kW4Bias = 1, kW4SwiGLU = 2 };

struct W4Args {
    const uint16_t* A;        // [*, K] bfloat16
    const int32_t* a_rows;    // nullable: A row of row r is a_rows[r]
    int a_row_limit;
    const int32_t* offsets;   // [E + 1]
    int E, K, N;              // N: rows of W per expert (2 F when gated)
    int max_rows;
    const uint32_t* q;
    const uint16_t* scale;
    const uint16_t* zero;     // nullable
    int G;
    const float* bias;        // [E, N], nullable
    uint16_t* D;
    int ldd;
    int ks;                   // warps that share a unit's K (1, 2, 4 or 8)
    DeviceStatus* st;
};

constexpr int kWarps = 8;
constexpr int kStages = 4;
constexpr int kRowTile = 32;                       // rows of a unit
constexpr int kStageW = 2048;                      // weights of a stage: 32 features x 128 columns
constexpr int kStageS = 256;                       // scales of a stage: 4 groups x 32 features
constexpr int kRedStride = 36;                     // floats per row of the partial sums
constexpr int kRedBytes = kWarps * 8 * kRedStride * 4;

template <bool ZERO>
constexpr int kStageBytes = kStageW + (ZERO ? 2 : 1) * kStageS;
template <bool ZERO>
constexpr int w4_smem_bytes(int E) {
    return kWarps * kStages * kStageBytes<ZERO> + 2 * kRedBytes + (E + 1) * 4;
}

__device__ __forceinline__ void cp_async_8(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void cp_async_4(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
    return v;
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A unit's place: expert, feature block, first row of the row tile, rows in it.
struct Unit { int e, fb, row0, rows; };

template <int EPI, bool ZERO>
struct W4Kernel {
    const W4Args& a;
    const int* s_pre;         // units before each expert
    int C, groups, UG, nfb;
    int warp, lane, g, t, ug, ks;

    __device__ __forceinline__ Unit unit_at(int u) const {
        int lo = 0, hi = a.E - 1;                 // largest e with s_pre[e] <= u
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (s_pre[mid] <= u) lo = mid; else hi = mid - 1;
        }
        const int r0 = a.offsets[lo], r1 = a.offsets[lo + 1];
        const int tiles = (r1 - r0 + kRowTile - 1) / kRowTile;
        const int i = u - s_pre[lo];
        Unit x;
        x.e = lo;
        x.fb = i / tiles;                         // row tiles of one feature block are neighbours:
        x.row0 = r0 + (i - x.fb * tiles) * kRowTile;      // its weights are in the cache
        x.rows = min(kRowTile, r1 - x.row0);
        return x;
    }
    // Row of W (within the expert) of this lane's first feature, and the step to the second pair:
    // gated units hold 16 gate rows and the 16 up rows that go with them.
    __device__ __forceinline__ int w_row(int fb) const {
        const int f32 = fb * UG + ug;             // 32-feature block
        return EPI == kW4SwiGLU ? f32 * 16 + 2 * g : f32 * 32 + 4 * g;
    }
    __device__ __forceinline__ bool has_features(int fb) const {
        return (fb * UG + ug) * 32 < a.N;
    }
    // Starts the copies of chunk c of unit x into the stage at `dst`.
    __device__ __forceinline__ void fetch(uint32_t dst, const Unit& x, int c) const {
        const int r = w_row(x.fb);
        const long long words = 16LL * C;
        const uint32_t* src = a.q + ((long long)x.e * a.N + r) * words + 16 * c + 4 * t;
        const long long up = EPI == kW4SwiGLU ? (long long)(a.N / 2) * words : 2 * words;
        cp_async_16(dst + lane * 16, src);
        cp_async_16(dst + 512 + lane * 16, src + words);
        cp_async_16(dst + 1024 + lane * 16, src + up);
        cp_async_16(dst + 1536 + lane * 16, src + up + words);
        const int gpc = 128 / a.G;
        if (t < gpc) {
            const int grp = c * gpc + t;
            const bool in = grp < groups;
            const long long at = ((long long)x.e * groups + (in ? grp : 0)) * a.N + r;
            const uint32_t d = dst + kStageW + t * 64 + g * 8;
            if constexpr (EPI == kW4SwiGLU) {
                cp_async_4(d, a.scale + at, in ? 4 : 0);
                cp_async_4(d + 4, a.scale + at + a.N / 2, in ? 4 : 0);
                if constexpr (ZERO) {
                    cp_async_4(d + kStageS, a.zero + at, in ? 4 : 0);
                    cp_async_4(d + kStageS + 4, a.zero + at + a.N / 2, in ? 4 : 0);
                }
            } else {
                cp_async_8(d, a.scale + at, in ? 8 : 0);
                if constexpr (ZERO) cp_async_8(d + kStageS, a.zero + at, in ? 8 : 0);
            }
        }
    }
    // acc[nt][m] += chunk c's products for NT tiles of 8 rows.
    template <int NT>
    __device__ __forceinline__ void chunk(uint32_t stage, int c, const uint16_t* const (&xr)[4],
                                          float (&acc)[4][2][4]) const {
        uint4 w[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) w[r] = lds128(stage + r * 512 + lane * 16);
        float part[NT][ZERO ? 3 : 2][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int m = 0; m < (ZERO ? 3 : 2); ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) part[n][m][i] = 0.0f;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint4 b[NT];
            const int k = c * 128 + j * 32 + t * 8;
#pragma unroll
            for (int n = 0; n < NT; ++n)
                b[n] = xr[n] && k < a.K ? *reinterpret_cast<const uint4*>(xr[n] + k)
                                        : make_uint4(0, 0, 0, 0);
            uint32_t p[4][4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const uint32_t word = j == 0 ? w[r].x : j == 1 ? w[r].y : j == 2 ? w[r].z : w[r].w;
#pragma unroll
                for (int i = 0; i < 4; ++i) p[r][i] = w4_pair(word, i);
            }
#pragma unroll
            for (int n = 0; n < NT; ++n) {
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    const uint32_t a0[4] = {p[2 * m][0], p[2 * m + 1][0], p[2 * m][1],
                                            p[2 * m + 1][1]};
                    const uint32_t a1[4] = {p[2 * m][2], p[2 * m + 1][2], p[2 * m][3],
                                            p[2 * m + 1][3]};
                    mma_bf16(part[n][m], a0, b[n].x, b[n].y);
                    mma_bf16(part[n][m], a1, b[n].z, b[n].w);
                }
                if constexpr (ZERO) {
                    const uint32_t one[4] = {0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u};
                    mma_bf16(part[n][2], one, b[n].x, b[n].y);
                    mma_bf16(part[n][2], one, b[n].z, b[n].w);
                }
            }
            if (((j + 1) * 32) % a.G == 0) {
                const int sg = j * 32 / a.G;
                const uint2 s = lds64(stage + kStageW + sg * 64 + g * 8);
                const float sc[4] = {bf16_bits(s.x & 0xffffu), bf16_bits(s.x >> 16),
                                     bf16_bits(s.y & 0xffffu), bf16_bits(s.y >> 16)};
#pragma unroll
                for (int n = 0; n < NT; ++n)
#pragma unroll
                    for (int m = 0; m < 2; ++m)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            acc[n][m][i] = fmaf(sc[2 * m + i / 2], part[n][m][i], acc[n][m][i]);
                            part[n][m][i] = 0.0f;
                        }
                if constexpr (ZERO) {
                    const uint2 zz = lds64(stage + kStageW + kStageS + sg * 64 + g * 8);
                    const float zo[4] = {bf16_bits(zz.x & 0xffffu), bf16_bits(zz.x >> 16),
                                         bf16_bits(zz.y & 0xffffu), bf16_bits(zz.y >> 16)};
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
#pragma unroll
                        for (int m = 0; m < 2; ++m)
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                acc[n][m][i] = fmaf(zo[2 * m + i / 2], part[n][2][i], acc[n][m][i]);
#pragma unroll
                        for (int i = 0; i < 4; ++i) part[n][2][i] = 0.0f;
                    }
                }
            }
        }
    }
};

__device__ __forceinline__ float silu(float v) { return v / (1.0f + __expf(-v)); }

template <int EPI, bool ZERO>
__global__ void __launch_bounds__(kWarps * 32, 2) w4_gemm_kernel(const W4Args args) {
    extern __shared__ __align__(16) uint8_t smem[];
    float* red = reinterpret_cast<float*>(smem + kWarps * kStages * kStageBytes<ZERO>);
    int* s_pre = reinterpret_cast<int*>(smem + kWarps * kStages * kStageBytes<ZERO> +
                                        2 * kRedBytes);
    W4Kernel<EPI, ZERO> w{args, s_pre};
    w.C = (args.K + 127) / 128;
    w.groups = (args.K + args.G - 1) / args.G;
    w.UG = kWarps / args.ks;
    w.nfb = (args.N / 32 + w.UG - 1) / w.UG;
    w.warp = threadIdx.x >> 5;
    w.lane = threadIdx.x & 31;
    w.g = w.lane >> 2;
    w.t = w.lane & 3;
    w.ug = w.warp / args.ks;
    w.ks = w.warp % args.ks;
    const int E = args.E, lane = w.lane;
    pdl_begin();
    __shared__ int s_bad;
    if (w.warp == 0) {
        // Units before each expert; offsets are checked as the grouped GEMM does: 0 first,
        // non-decreasing, at most max_rows.  Bad offsets: nothing is computed or stored.
        int total = 0;
        bool bad = false;
        if (lane == 0)
            bad = args.offsets[0] != 0 || args.offsets[E] > args.max_rows;
        for (int e0 = 0; e0 < E; e0 += 32) {
            const int e = e0 + lane;
            int n = e < E ? args.offsets[e + 1] - args.offsets[e] : 0;
            bad |= n < 0;
            n = max(n, 0);
            const int units = (n + kRowTile - 1) / kRowTile * w.nfb;
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
            s_bad = bad;
            if (bad && blockIdx.x == 0) report(args.st, MOE_DEV_BAD_INDEX, 710);
        }
    }
    __syncthreads();
    if (s_bad) return;
    const int total = s_pre[E];
    const int u0 = (int)((long long)total * blockIdx.x / gridDim.x);
    const int u1 = (int)((long long)total * (blockIdx.x + 1) / gridDim.x);
    if (u0 >= u1) return;

    const uint32_t ring = smem_u32(smem) + w.warp * kStages * kStageBytes<ZERO>;
    // The fetcher walks (unit, chunk) ahead of the products.
    int fu = u0, fc = w.ks, fslot = 0;
    Unit fx = w.unit_at(u0);
    auto fetch_next = [&]() {
        if (fu < u1) {
            // (no features, or no chunk of this warp: units of nothing to fetch are skipped)
            while (fu < u1 && (fc >= w.C || !w.has_features(fx.fb))) {
                fc = w.ks;
                if (++fu < u1) fx = w.unit_at(fu);
            }
            if (fu < u1) {
                w.fetch(ring + fslot * kStageBytes<ZERO>, fx, fc);
                fslot = fslot + 1 == kStages ? 0 : fslot + 1;
                fc += args.ks;
            }
        }
        cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) fetch_next();

    int slot = 0, buf = 0;
    for (int u = u0; u < u1; ++u) {
        const Unit x = w.unit_at(u);
        const int nt = (x.rows + 7) / 8;
        const uint16_t* xr[4];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const int r = n * 8 + w.g;
            xr[n] = nullptr;
            if (r < x.rows) {
                int src = x.row0 + r;
                if (args.a_rows) {
                    src = args.a_rows[src];
                    if (src < 0 || src >= args.a_row_limit) {
                        report(args.st, MOE_DEV_BAD_INDEX, 720);
                        src = -1;
                    }
                }
                if (src >= 0) xr[n] = args.A + (long long)src * args.K;
            }
        }
        float acc[4][2][4];
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[n][m][i] = 0.0f;
        if (w.has_features(x.fb)) {
            for (int c = w.ks; c < w.C; c += args.ks) {
                fetch_next();
                cp_async_wait<kStages - 1>();
                __syncwarp();          // scales were copied by other lanes of the warp
                const uint32_t stage = ring + slot * kStageBytes<ZERO>;
                if (nt == 1) w.template chunk<1>(stage, c, xr, acc);
                else if (nt == 2) w.template chunk<2>(stage, c, xr, acc);
                else w.template chunk<4>(stage, c, xr, acc);
                __syncwarp();          // before the stage is filled again
                slot = slot + 1 == kStages ? 0 : slot + 1;
            }
        }
        // Join the KS partial sums, 8 rows at a time, and store.
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            if (n < nt) {
                float* rb = red + buf * (kRedBytes / 4);
                float* mine = rb + (w.warp * 8 + 2 * w.t) * kRedStride + 4 * w.g;
                // rows 2t, 2t + 1; features 4g .. 4g + 3 = (m0 lo, m0 hi, m1 lo, m1 hi)
                *reinterpret_cast<float4*>(mine) = make_float4(acc[n][0][0], acc[n][0][2],
                                                               acc[n][1][0], acc[n][1][2]);
                *reinterpret_cast<float4*>(mine + kRedStride) =
                    make_float4(acc[n][0][1], acc[n][0][3], acc[n][1][1], acc[n][1][3]);
                __syncthreads();
                constexpr int kOut = EPI == kW4SwiGLU ? 16 : 32;      // features per 32 rows of W
                for (int i = threadIdx.x; i < w.UG * 8 * kOut; i += kWarps * 32) {
                    const int ug = i / (8 * kOut), row = i / kOut % 8, f = i % kOut;
                    const int f32 = x.fb * w.UG + ug;
                    if (n * 8 + row >= x.rows || f32 * 32 >= args.N) continue;
                    // Gated: features 2 g, 2 g + 1 of the 16 are columns 4 g, 4 g + 1 (gate) and
                    // 4 g + 2, 4 g + 3 (up) of the sums.
                    const int col = EPI == kW4SwiGLU ? 4 * (f >> 1) + (f & 1) : f;
                    const float* s = rb + (ug * args.ks * 8 + row) * kRedStride + col;
                    float v = 0.0f, up = 0.0f;
                    for (int q = 0; q < args.ks; ++q) {
                        v += s[q * 8 * kRedStride];
                        if (EPI == kW4SwiGLU) up += s[q * 8 * kRedStride + 2];
                    }
                    const int feat = f32 * kOut + f;
                    if (args.bias) {
                        const float* b = args.bias + (long long)x.e * args.N;
                        v += b[feat];
                        if (EPI == kW4SwiGLU) up += b[args.N / 2 + feat];
                    }
                    if (EPI == kW4SiLU) v = silu(v);
                    if (EPI == kW4SwiGLU) v = silu(v) * up;
                    args.D[(long long)(x.row0 + n * 8 + row) * args.ldd + feat] = bf16_round(v);
                }
                buf ^= 1;
            }
        }
    }
    cp_async_wait<0>();
}

template <int EPI, bool ZERO>
cudaError_t run_w4(const W4Args& a, cudaStream_t s) {
    auto kern = w4_gemm_kernel<EPI, ZERO>;
    const int smem = w4_smem_bytes<ZERO>(a.E);
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (note_launch(e) != cudaSuccess) return e;
    return launch_pdl(kern, dim3(2 * kSm), dim3(kWarps * 32), smem, s, a);
}

}  // namespace

void launch_w4_quantize(int dtype, const void* W, int E, int N, int K, int G, uint32_t* q,
                        uint16_t* scale, uint16_t* zero, cudaStream_t s, int* launches) {
    const int row_tiles = (N + kQRows - 1) / kQRows;
    const int C = (K + 127) / 128;
    // Row tiles of all experts on y (at most 65535 a launch), chunks on x.
    const int per = 65535 / row_tiles > 0 ? 65535 / row_tiles : 1;
    const int groups = (K + G - 1) / G;
    for (int e0 = 0; e0 < E; e0 += per) {
        const int ne = std::min(per, E - e0);
        const dim3 grid((C + kQChunks - 1) / kQChunks, ne * row_tiles);
        const long long rows = (long long)e0 * N;
        uint16_t* z = zero ? zero + rows * groups : nullptr;
        if (dtype == MOE_BF16)
            launch_pdl(w4_quantize_kernel<uint16_t>, grid, dim3(256), 0, s,
                       (const uint16_t*)W + rows * K, N, K, G, row_tiles, q + rows * 16 * C,
                       scale + rows * groups, z);
        else
            launch_pdl(w4_quantize_kernel<float>, grid, dim3(256), 0, s,
                       (const float*)W + rows * K, N, K, G, row_tiles, q + rows * 16 * C,
                       scale + rows * groups, z);
        *launches += 1;
    }
}

void launch_w4_dequantize(const uint32_t* q, const uint16_t* scale, const uint16_t* zero, int E,
                          int N, int K, int G, void* W, cudaStream_t s, int* launches) {
    const long long words = (long long)E * N * 16 * ((K + 127) / 128);
    const int blocks = (int)std::min<long long>((words + 255) / 256, kSm * 32);
    launch_pdl(w4_dequantize_kernel, dim3(blocks), dim3(256), 0, s, q, scale, zero, N, K, G, words,
               (uint16_t*)W);
    *launches += 1;
}

cudaError_t launch_w4_gemm(int which, const void* A, const int32_t* a_rows, int a_row_limit,
                           const int32_t* offsets, int E, int K, int N, int max_rows,
                           const uint32_t* q, const uint16_t* scale, const uint16_t* zero, int G,
                           const float* bias, void* D, int ldd, DeviceStatus* st, cudaStream_t s,
                           int* launches) {
    W4Args a{(const uint16_t*)A, a_rows, a_row_limit, offsets, E, K, N, max_rows, q, scale, zero,
             G, bias, (uint16_t*)D, ldd, 8, st};
    // Warps that share a unit's K: as many as there are chunks, at most 8.
    while (a.ks > 1 && a.ks > (K + 127) / 128) a.ks /= 2;
    cudaError_t e;
    if (which == kW4SiLU) e = zero ? run_w4<kW4SiLU, true>(a, s) : run_w4<kW4SiLU, false>(a, s);
    else if (which == kW4Bias) e = zero ? run_w4<kW4Bias, true>(a, s) : run_w4<kW4Bias, false>(a, s);
    else e = zero ? run_w4<kW4SwiGLU, true>(a, s) : run_w4<kW4SwiGLU, false>(a, s);
    *launches += 1;
    return e;
}

}  // namespace moe

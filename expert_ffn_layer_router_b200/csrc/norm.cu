// norm.cu -- the layer norm in front of the layer, forward and backward (sm_100a).
//
//   mean = sum_c x_c / d,  rstd = 1 / sqrt(sum_c (x_c - mean)^2 / d + eps),
//   xh = (x - mean) rstd,  y = gamma xh + beta
//   g = gamma dy,  dx = rstd (g - mean_c(g) - xh mean_c(g xh)) (+ dres),
//   dgamma = sum_t dy xh,  dbeta = sum_t dy.
//
// Both passes are bound by memory: a row is read once, kept on chip, and written once.
//
// Layout.  Persistent blocks walk the rows.  WPR warps share a row; lane l of warp w holds the
// vectors of VB elements at (v WPR 32 + w 32 + l) VB, 16 elements in all, so every load is
// contiguous over the warp, and gamma, beta (backward: the dgamma and dbeta sums) of a thread's
// columns stay in its registers.  VB is 16 bytes where rows and pointers allow: then rows come
// through a ring of cp.async stages, kRows rows ahead (a thread copies the pieces that it uses
// itself, so no barrier guards the ring); else VB is one element (odd widths), loaded directly.
// The variance is the two-pass one (the row is in registers, so the second pass costs no memory).
// Statistics and sums are fp32.  Of a row's statistics a lane adds at most 16 values before the tree
// over lanes and warps (d / 512 in the *_wide kernels); of dgamma and dbeta a thread adds its rows
// behind one another, rows / (296 row groups of a block) (rows / 16 in the wide kernel), before the
// partial rows are joined: 222 at 65536 x 4096.
// (65536 x 4096 bfloat16.  Forward 174 us, 164 at the copy bandwidth; with gamma and beta read for
// every row, which kept the load unit at 76%, 234.  Backward with the residual 346 us, 327 at the copy
// bandwidth; with rows loaded when they were needed, and the residual's after the sums, 566.)
//
// Backward.  Row groups of a block join their column sums in shared memory in order, blocks write
// one partial row each, and a second launch adds those in order.  No atomics: the result does not
// depend on scheduling.
//
// Rows wider than the register layout holds (kMaxCols) take the *_wide kernels: a block per row
// that reads the row again in each pass, and a column-wise pass for dgamma and dbeta.
#include <algorithm>
#include <cstdint>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kSm = 148;

constexpr int kElems = 16;                           // elements a lane holds of a row
constexpr int kMaxWarps = 16;
constexpr int kMaxCols = kElems * 32 * kMaxWarps;    // 8192

template <class T> struct Vec;
template <> struct Vec<float> {
    static constexpr int kWide = 4;
    __device__ static void load(const float* p, float (&f)[4]) {
        const float4 v = *reinterpret_cast<const float4*>(p);
        f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
    }
    __device__ static void store(float* p, const float (&f)[4]) {
        *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
    }
    __device__ static float to(float v) { return v; }
    __device__ static float from(float v) { return v; }
};
template <> struct Vec<__nv_bfloat16> {
    static constexpr int kWide = 8;
    __device__ static void load(const __nv_bfloat16* p, float (&f)[8]) {
        const uint4 v = *reinterpret_cast<const uint4*>(p);
        const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(u[i] << 16);
            f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    }
    __device__ static void store(__nv_bfloat16* p, const float (&f)[8]) {
        *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                                  pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
    }
    __device__ static float to(__nv_bfloat16 v) { return __bfloat162float(v); }
    __device__ static __nv_bfloat16 from(float v) { return __float2bfloat16_rn(v); }
};

// VB consecutive elements of a row at p (VB = 1 or the 16-byte width), zeros where !in.
template <class T, int VB>
__device__ __forceinline__ void load_elems(const T* p, bool in, float (&f)[VB]) {
    if constexpr (VB == 1) {
        f[0] = in ? Vec<T>::to(*p) : 0.0f;
    } else {
        if (in) {
            Vec<T>::load(p, f);
        } else {
#pragma unroll
            for (int i = 0; i < VB; ++i) f[i] = 0.0f;
        }
    }
}
template <class T, int VB>
__device__ __forceinline__ void store_elems(T* p, const float (&f)[VB]) {
    if constexpr (VB == 1) *p = Vec<T>::from(f[0]);
    else Vec<T>::store(p, f);
}
// VB consecutive fp32 parameters (16-byte aligned when VB > 1).
template <int VB>
__device__ __forceinline__ void load_params(const float* p, float (&f)[VB]) {
    if constexpr (VB == 1) {
        f[0] = *p;
    } else {
#pragma unroll
        for (int i = 0; i < VB; i += 4) {
            const float4 v = *reinterpret_cast<const float4*>(p + i);
            f[i] = v.x; f[i + 1] = v.y; f[i + 2] = v.z; f[i + 3] = v.w;
        }
    }
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int h = 16; h >= 1; h >>= 1) v += __shfl_xor_sync(kFull, v, h);
    return v;
}

// Sum of N floats in order (16-byte loads from 16-byte aligned shared memory when N allows).
template <int N>
__device__ __forceinline__ float sum_of(const float* p) {
    float v;
    if constexpr (N % 4 == 0) {
        v = 0.0f;
#pragma unroll
        for (int i = 0; i < N; i += 4) {
            const float4 f = *reinterpret_cast<const float4*>(p + i);
            v += f.x; v += f.y; v += f.z; v += f.w;
        }
    } else {
        v = p[0];
#pragma unroll
        for (int i = 1; i < N; ++i) v += p[i];
    }
    return v;
}

// Sum over the WPR warps of this thread's row (every thread of the block calls it together).
// buf: one float per warp of the block, not read any more by an earlier call.
template <int WPR>
__device__ __forceinline__ float row_sum(float v, float* buf) {
    v = warp_sum(v);
    if constexpr (WPR > 1) {
        const int warp = threadIdx.x >> 5;
        if ((threadIdx.x & 31) == 0) buf[warp] = v;
        __syncthreads();
        v = sum_of<WPR>(buf + warp / WPR * WPR);
    }
    return v;
}

// 1 / sqrt(a), a >= 0: the approximation and one step of Newton's iteration on y^-2 = a (not for 0
// and infinity, where the step would make a NaN of inf 0).
__device__ __forceinline__ float inv_sqrt(float a) {
    const float y = rsqrtf(a);
    return a > 0.0f && y > 0.0f ? y * fmaf(-0.5f * a * y, y, 1.5f) : y;
}

template <int WPR>
constexpr int kWarpsOf = WPR > 8 ? WPR : 8;

// Rows of STREAMS arrays on their way to this thread: a ring of kRows rows in shared memory, in
// pieces of 16 bytes that the thread copies and reads itself ([row][stream][piece][thread]).
template <class T, int VB, int STREAMS, int THREADS>
struct Ring {
    static constexpr bool kOn = VB > 1;
    static constexpr int kRows = 8 / sizeof(T);                       // 4 (bfloat16) or 2
    static constexpr int kRowBytes = STREAMS * THREADS * kElems * (int)sizeof(T);
    static constexpr int kBytes = kOn ? kRows * kRowBytes : 0;
    uint8_t* base;
    int put, get;

    __device__ __forceinline__ explicit Ring(uint8_t* smem) : base(smem + threadIdx.x * 16), put(0), get(0) {}
    __device__ __forceinline__ uint8_t* at(int slot, int stream, int v) const {
        return base + slot * kRowBytes + (stream * (kElems / VB) + v) * THREADS * 16;
    }
    __device__ __forceinline__ void copy(int stream, int v, const T* src) const {
        if constexpr (kOn) cp_async_16(smem_u32(at(put, stream, v)), src);
    }
    // One row's copies have been issued (also when there was none).
    __device__ __forceinline__ void issued() {
        if constexpr (kOn) {
            cp_async_commit();
            put = put + 1 == kRows ? 0 : put + 1;
        }
    }
    // The oldest row that was issued has landed.
    __device__ __forceinline__ void wait() const {
        if constexpr (kOn) cp_async_wait<kRows - 1>();
    }
    __device__ __forceinline__ void taken() {
        if constexpr (kOn) get = get + 1 == kRows ? 0 : get + 1;
    }
    // The thread's vector v of the oldest row; `src`: where it is in memory.
    __device__ __forceinline__ void take(int stream, int v, const T* src, bool in,
                                         float (&f)[VB]) const {
        if constexpr (kOn)
            load_elems<T, VB>(reinterpret_cast<const T*>(at(get, stream, v)), in, f);
        else
            load_elems<T, VB>(src, in, f);
    }
};

template <class T, int VB, int WPR>
__global__ void __launch_bounds__(kWarpsOf<WPR> * 32, WPR > 8 ? 1 : 3)
    layer_norm_kernel(const T* __restrict__ x, const float* __restrict__ gamma,
                      const float* __restrict__ beta, float eps, int rows, int d,
                      T* __restrict__ y, float* __restrict__ mean, float* __restrict__ rstd) {
    constexpr int NV = kElems / VB;
    constexpr int kWarps = kWarpsOf<WPR>;
    constexpr int RPC = kWarps / WPR;                 // rows in flight per block
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ __align__(16) float s_buf[2][2][kWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c0 = ((warp % WPR) * 32 + lane) * VB;
    constexpr int kStep = WPR * 32 * VB;              // columns from a lane's vector to its next
    const int all = gridDim.x * RPC;
    const int steps = (int)(((long long)rows + all - 1) / all);
    const long long row0 = blockIdx.x * RPC + warp / WPR;
    using R = Ring<T, VB, 1, kWarps * 32>;
    R ring(smem);
    pdl_begin();
    long long ahead = row0;                           // the next row to copy
    const T* xa = x + row0 * d + c0;
    auto fetch = [&]() {
        if (R::kOn && ahead < rows) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (c0 + i * kStep < d) ring.copy(0, i, xa + i * kStep);
        }
        ahead += all;
        xa += (long long)all * d;
        ring.issued();
    };
    for (int i = 0; i < R::kRows - 1; ++i) fetch();
    float ga[NV][VB], be[NV][VB];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
        for (int q = 0; q < VB; ++q) ga[i][q] = be[i][q] = 0.0f;
        if (c0 + i * kStep < d) {
            load_params<VB>(gamma + c0 + i * kStep, ga[i]);
            load_params<VB>(beta + c0 + i * kStep, be[i]);
        }
    }
    const float inv_d = 1.0f / (float)d;
    long long row = row0;
    const long long stride = (long long)all * d;
    const T* xr = x + row0 * d + c0;
    T* yr = y + row0 * d + c0;
    for (int it = 0; it < steps; ++it, row += all, xr += stride, yr += stride) {
        const bool live = row < rows;
        fetch();
        ring.wait();
        float v[NV][VB];
        float s = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            ring.take(0, i, xr + i * kStep, live && c0 + i * kStep < d, v[i]);
#pragma unroll
            for (int q = 0; q < VB; ++q) s += v[i][q];
        }
        ring.taken();
        const float mu = row_sum<WPR>(s, s_buf[it & 1][0]) * inv_d;
        float s2 = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const float m = c0 + i * kStep < d ? mu : 0.0f;      // (columns past d are zeros)
#pragma unroll
            for (int q = 0; q < VB; ++q) {
                v[i][q] -= m;
                s2 = fmaf(v[i][q], v[i][q], s2);
            }
        }
        const float rs = inv_sqrt(fmaf(row_sum<WPR>(s2, s_buf[it & 1][1]), inv_d, eps));
        if (live) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (c0 + i * kStep < d) {
#pragma unroll
                    for (int q = 0; q < VB; ++q)
                        v[i][q] = fmaf(v[i][q] * rs, ga[i][q], be[i][q]);
                    store_elems<T, VB>(yr + i * kStep, v[i]);
                }
            }
            if (warp % WPR == 0 && lane == 0) {
                mean[row] = mu;
                rstd[row] = rs;
            }
        }
    }
    if (R::kOn) cp_async_wait<0>();
}

// One block of 512 threads per row, the row read again in each pass.
template <class T>
__global__ void __launch_bounds__(512)
    layer_norm_wide_kernel(const T* __restrict__ x, const float* __restrict__ gamma,
                           const float* __restrict__ beta, float eps, int d, T* __restrict__ y,
                           float* __restrict__ mean, float* __restrict__ rstd) {
    pdl_begin();
    __shared__ __align__(16) float s_buf[2][16];
    const long long row = blockIdx.x;
    const T* xr = x + row * d;
    T* yr = y + row * d;
    float s = 0.0f;
    for (int c = threadIdx.x; c < d; c += 512) s += Vec<T>::to(xr[c]);
    const float mu = row_sum<16>(s, s_buf[0]) / (float)d;
    s = 0.0f;
    for (int c = threadIdx.x; c < d; c += 512) {
        const float v = Vec<T>::to(xr[c]) - mu;
        s = fmaf(v, v, s);
    }
    const float rs = 1.0f / sqrtf(row_sum<16>(s, s_buf[1]) / (float)d + eps);
    for (int c = threadIdx.x; c < d; c += 512)
        yr[c] = Vec<T>::from(fmaf((Vec<T>::to(xr[c]) - mu) * rs, gamma[c], beta[c]));
    if (threadIdx.x == 0) {
        mean[row] = mu;
        rstd[row] = rs;
    }
}

// part: [gridDim.x][2][d] fp32 (dgamma sums, dbeta sums of the block's rows).
template <class T, int VB, int WPR>
__global__ void __launch_bounds__(kWarpsOf<WPR> * 32, WPR > 8 ? 1 : 2)
    layer_norm_backward_kernel(const T* __restrict__ dy, const T* __restrict__ x,
                               const float* __restrict__ gamma, const float* __restrict__ mean,
                               const float* __restrict__ rstd, const T* __restrict__ dres,
                               int rows, int d, T* __restrict__ dx, float* __restrict__ part) {
    constexpr int NV = kElems / VB;
    constexpr int kWarps = kWarpsOf<WPR>;
    constexpr int RPC = kWarps / WPR;                 // rows in flight per block
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ __align__(16) float s_buf[2][2][kWarps];
    __shared__ float s_sum[RPC > 1 ? 2 : 1][RPC > 1 ? WPR * 32 * kElems : 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c0 = ((warp % WPR) * 32 + lane) * VB;
    constexpr int kStep = WPR * 32 * VB;
    const int all = gridDim.x * RPC;
    const int steps = (int)(((long long)rows + all - 1) / all);
    const long long row0 = blockIdx.x * RPC + warp / WPR;
    using R = Ring<T, VB, 3, kWarps * 32>;
    R ring(smem);
    pdl_begin();
    long long ahead = row0, ahead_at = row0 * d + c0;      // the next row to copy
    const long long stride = (long long)all * d;
    auto fetch = [&]() {
        if (R::kOn && ahead < rows) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (c0 + i * kStep < d) {
                    ring.copy(0, i, x + ahead_at + i * kStep);
                    ring.copy(1, i, dy + ahead_at + i * kStep);
                    if (dres) ring.copy(2, i, dres + ahead_at + i * kStep);
                }
            }
        }
        ahead += all;
        ahead_at += stride;
        ring.issued();
    };
    for (int i = 0; i < R::kRows - 1; ++i) fetch();
    float ga[NV][VB], dg[NV][VB], db[NV][VB];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
        for (int q = 0; q < VB; ++q) ga[i][q] = dg[i][q] = db[i][q] = 0.0f;
        if (c0 + i * kStep < d) load_params<VB>(gamma + c0 + i * kStep, ga[i]);
    }
    const float inv_d = 1.0f / (float)d;
    // The statistics of the next row are read a row ahead.
    float mu = row0 < rows ? mean[row0] : 0.0f, rs = row0 < rows ? rstd[row0] : 0.0f;
    long long row = row0, at0 = row0 * d + c0;
    for (int it = 0; it < steps; ++it, row += all, at0 += stride) {
        const bool live = row < rows, more = row + all < rows;
        fetch();
        const float mu_next = more ? mean[row + all] : 0.0f;
        const float rs_next = more ? rstd[row + all] : 0.0f;
        ring.wait();
        float xv[NV][VB], gv[NV][VB];
        float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const bool in = live && c0 + i * kStep < d;
            const long long at = at0 + i * kStep;
            ring.take(0, i, x + at, in, xv[i]);
            ring.take(1, i, dy + at, in, gv[i]);
#pragma unroll
            for (int q = 0; q < VB; ++q) {
                xv[i][q] = (xv[i][q] - mu) * rs;     // (past d: times a gradient of 0)
                dg[i][q] = fmaf(gv[i][q], xv[i][q], dg[i][q]);
                db[i][q] += gv[i][q];
                gv[i][q] *= ga[i][q];
                s1 += gv[i][q];
                s2 = fmaf(gv[i][q], xv[i][q], s2);
            }
        }
        s1 = warp_sum(s1);
        s2 = warp_sum(s2);
        if constexpr (WPR > 1) {
            float (*buf)[kWarps] = s_buf[it & 1];
            if (lane == 0) {
                buf[0][warp] = s1;
                buf[1][warp] = s2;
            }
            __syncthreads();
            s1 = sum_of<WPR>(buf[0] + warp / WPR * WPR);
            s2 = sum_of<WPR>(buf[1] + warp / WPR * WPR);
        }
        s1 *= inv_d;
        s2 *= inv_d;
        if (live) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (c0 + i * kStep < d) {
                    const long long at = at0 + i * kStep;
                    float res[VB];
                    ring.take(2, i, dres + at, dres != nullptr, res);
#pragma unroll
                    for (int q = 0; q < VB; ++q)
                        gv[i][q] = fmaf(gv[i][q] - s1 - xv[i][q] * s2, rs, res[q]);
                    store_elems<T, VB>(dx + at, gv[i]);
                }
            }
        }
        ring.taken();
        mu = mu_next;
        rs = rs_next;
    }
    if (R::kOn) cp_async_wait<0>();
    if constexpr (RPC > 1) {
        for (int g = 0; g < RPC; ++g) {
            if (warp / WPR == g) {
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int q = 0; q < VB; ++q) {
                        const int c = c0 + i * kStep + q;
                        if (g > 0) {
                            dg[i][q] += s_sum[0][c];
                            db[i][q] += s_sum[1][c];
                        }
                        s_sum[0][c] = dg[i][q];
                        s_sum[1][c] = db[i][q];
                    }
            }
            __syncthreads();
        }
    }
    if (warp / WPR == RPC - 1) {
        float* o = part + (long long)blockIdx.x * 2 * d;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = c0 + i * kStep;
            if (c < d) {
#pragma unroll
                for (int q = 0; q < VB; ++q) {
                    o[c + q] = dg[i][q];
                    o[d + c + q] = db[i][q];
                }
            }
        }
    }
}

// dgamma[c] and dbeta[c] = sums over nb partial rows, in a fixed order: 32 columns x 32 slices of
// rows a block.
__global__ void __launch_bounds__(1024)
    layer_norm_param_kernel(const float* __restrict__ part, int nb, int d,
                            float* __restrict__ dgamma, float* __restrict__ dbeta) {
    pdl_begin();
    __shared__ float s[32][33];
    const int cx = threadIdx.x & 31, sl = threadIdx.x >> 5;
    const long long c = (long long)blockIdx.x * 32 + cx;      // column of the 2 d sums
    float v = 0.0f;
    if (c < 2LL * d) {
#pragma unroll 5
        for (int b = sl; b < nb; b += 32) v += part[(long long)b * 2 * d + c];
    }
    s[sl][cx] = v;
    __syncthreads();
    // Warp w joins column w's 32 slices.
    v = warp_sum(s[cx][sl]);
    const long long cw = (long long)blockIdx.x * 32 + sl;
    if (cx == 0 && cw < 2LL * d) {
        if (cw < d) dgamma[cw] = v;
        else dbeta[cw - d] = v;
    }
}

template <class T>
__global__ void __launch_bounds__(512)
    layer_norm_backward_wide_kernel(const T* __restrict__ dy, const T* __restrict__ x,
                                    const float* __restrict__ gamma,
                                    const float* __restrict__ mean,
                                    const float* __restrict__ rstd, const T* __restrict__ dres,
                                    int d, T* __restrict__ dx) {
    pdl_begin();
    __shared__ __align__(16) float s_buf[2][16];
    const long long row = blockIdx.x;
    const float mu = mean[row], rs = rstd[row];
    float s1 = 0.0f, s2 = 0.0f;
    for (int c = threadIdx.x; c < d; c += 512) {
        const float g = Vec<T>::to(dy[row * d + c]) * gamma[c];
        s1 += g;
        s2 = fmaf(g, (Vec<T>::to(x[row * d + c]) - mu) * rs, s2);
    }
    s1 = row_sum<16>(s1, s_buf[0]) / (float)d;
    s2 = row_sum<16>(s2, s_buf[1]) / (float)d;
    for (int c = threadIdx.x; c < d; c += 512) {
        const float g = Vec<T>::to(dy[row * d + c]) * gamma[c];
        const float xh = (Vec<T>::to(x[row * d + c]) - mu) * rs;
        const float res = dres ? Vec<T>::to(dres[row * d + c]) : 0.0f;
        dx[row * d + c] = Vec<T>::from(fmaf(g - s1 - xh * s2, rs, res));
    }
}

// Partial column sums of rows [blockIdx.y * per, ...): a thread per column.
template <class T>
__global__ void __launch_bounds__(256)
    layer_norm_columns_kernel(const T* __restrict__ dy, const T* __restrict__ x,
                              const float* __restrict__ mean, const float* __restrict__ rstd,
                              int rows, int d, int per, float* __restrict__ part) {
    pdl_begin();
    const int c = blockIdx.x * 256 + threadIdx.x;
    if (c >= d) return;
    const int r0 = blockIdx.y * per, r1 = min(rows, r0 + per);
    float dg = 0.0f, db = 0.0f;
    for (int r = r0; r < r1; ++r) {
        const float g = Vec<T>::to(dy[(long long)r * d + c]);
        dg = fmaf(g, (Vec<T>::to(x[(long long)r * d + c]) - mean[r]) * rstd[r], dg);
        db += g;
    }
    float* o = part + (long long)blockIdx.y * 2 * d;
    o[c] = dg;
    o[d + c] = db;
}

// Warps per row: a power of two whose lanes hold the row.
int warps_per_row(int d) {
    int w = 1;
    while (w * 32 * kElems < d) w *= 2;
    return w;
}

// Persistent blocks: `per_sm` a SM (one where 16 warps share a row), but none without a row.
int norm_blocks(int rows, int d, int per_sm) {
    const int wpr = warps_per_row(d);
    const int rpc = wpr > 8 ? 1 : 8 / wpr;
    return (int)std::min<long long>(((long long)rows + rpc - 1) / rpc,
                                    kSm * (wpr > 8 ? 1 : per_sm));
}

// Blocks of the backward kernel, which are the partial rows.
int backward_blocks(int rows, int d) {
    return d > kMaxCols ? std::min(rows, 16) : norm_blocks(rows, d, 2);
}

bool wide_ok(int d, int elem_bytes, std::initializer_list<const void*> ptrs) {
    if ((long long)d * elem_bytes % 16 != 0) return false;
    for (const void* p : ptrs)
        if (reinterpret_cast<uintptr_t>(p) & 15) return false;
    return true;
}

template <class Kern, class... Args>
void launch_norm(Kern kern, std::atomic<int> (&allowed)[64], int blocks, int wpr, int smem,
                 cudaStream_t s, Args... args) {
    if (smem > 48 * 1024 && allow_smem(kern, allowed, smem) != cudaSuccess) return;
    launch_pdl(kern, dim3(blocks), dim3((wpr > 8 ? wpr : 8) * 32), smem, s, args...);
}

template <class T, int VB>
void forward_typed(const T* x, const float* gamma, const float* beta, float eps, int rows, int d,
                   T* y, float* mean, float* rstd, cudaStream_t s) {
    auto go = [&](auto kern, auto wpr) {
        constexpr int W = decltype(wpr)::value;
        static std::atomic<int> allowed[64];      // (one for each instance of this lambda)
        launch_norm(kern, allowed, norm_blocks(rows, d, 3), W, Ring<T, VB, 1, kWarpsOf<W> * 32>::kBytes, s,
                    x, gamma, beta, eps, rows, d, y, mean, rstd);
    };
    switch (warps_per_row(d)) {
        case 1: go(layer_norm_kernel<T, VB, 1>, std::integral_constant<int, 1>()); break;
        case 2: go(layer_norm_kernel<T, VB, 2>, std::integral_constant<int, 2>()); break;
        case 4: go(layer_norm_kernel<T, VB, 4>, std::integral_constant<int, 4>()); break;
        case 8: go(layer_norm_kernel<T, VB, 8>, std::integral_constant<int, 8>()); break;
        default: go(layer_norm_kernel<T, VB, 16>, std::integral_constant<int, 16>()); break;
    }
}

template <class T>
void forward_any(const T* x, const float* gamma, const float* beta, float eps, int rows, int d,
                 T* y, float* mean, float* rstd, cudaStream_t s) {
    if (d > kMaxCols)
        launch_pdl(layer_norm_wide_kernel<T>, dim3(rows), dim3(512), 0, s, x, gamma, beta, eps, d,
                   y, mean, rstd);
    else if (wide_ok(d, sizeof(T), {x, y, gamma, beta}))
        forward_typed<T, Vec<T>::kWide>(x, gamma, beta, eps, rows, d, y, mean, rstd, s);
    else
        forward_typed<T, 1>(x, gamma, beta, eps, rows, d, y, mean, rstd, s);
}

template <class T, int VB>
void backward_typed(const T* dy, const T* x, const float* gamma, const float* mean,
                    const float* rstd, const T* dres, int rows, int d, T* dx, float* part,
                    cudaStream_t s) {
    auto go = [&](auto kern, auto wpr) {
        constexpr int W = decltype(wpr)::value;
        static std::atomic<int> allowed[64];      // (one for each instance of this lambda)
        launch_norm(kern, allowed, backward_blocks(rows, d), W, Ring<T, VB, 3, kWarpsOf<W> * 32>::kBytes, s,
                    dy, x, gamma, mean, rstd, dres, rows, d, dx, part);
    };
    switch (warps_per_row(d)) {
        case 1: go(layer_norm_backward_kernel<T, VB, 1>, std::integral_constant<int, 1>()); break;
        case 2: go(layer_norm_backward_kernel<T, VB, 2>, std::integral_constant<int, 2>()); break;
        case 4: go(layer_norm_backward_kernel<T, VB, 4>, std::integral_constant<int, 4>()); break;
        case 8: go(layer_norm_backward_kernel<T, VB, 8>, std::integral_constant<int, 8>()); break;
        default: go(layer_norm_backward_kernel<T, VB, 16>, std::integral_constant<int, 16>()); break;
    }
}

template <class T>
void backward_any(const T* dy, const T* x, const float* gamma, const float* mean,
                  const float* rstd, const T* dres, int rows, int d, T* dx, float* dgamma,
                  float* dbeta, float* part, cudaStream_t s, int* launches) {
    const int nb = backward_blocks(rows, d);
    if (d > kMaxCols) {
        launch_pdl(layer_norm_backward_wide_kernel<T>, dim3(rows), dim3(512), 0, s, dy, x, gamma,
                   mean, rstd, dres, d, dx);
        launch_pdl(layer_norm_columns_kernel<T>, dim3((d + 255) / 256, nb), dim3(256), 0, s, dy, x,
                   mean, rstd, rows, d, (rows + nb - 1) / nb, part);
        *launches += 2;
    } else {
        if (wide_ok(d, sizeof(T), {dy, x, gamma, dres, dx}))
            backward_typed<T, Vec<T>::kWide>(dy, x, gamma, mean, rstd, dres, rows, d, dx, part, s);
        else
            backward_typed<T, 1>(dy, x, gamma, mean, rstd, dres, rows, d, dx, part, s);
        *launches += 1;
    }
    launch_pdl(layer_norm_param_kernel, dim3((unsigned)((2LL * d + 31) / 32)), dim3(1024), 0, s,
               (const float*)part, nb, d, dgamma, dbeta);
    *launches += 1;
}

}  // namespace

size_t layer_norm_scratch_bytes(int rows, int d) {
    return rows > 0 ? (size_t)backward_blocks(rows, d) * 2 * d * 4 : 0;
}

void launch_layer_norm(int dtype, const void* x, const float* gamma, const float* beta, float eps,
                       int rows, int d, void* y, float* mean, float* rstd, cudaStream_t s,
                       int* launches) {
    if (dtype == MOE_BF16)
        forward_any((const __nv_bfloat16*)x, gamma, beta, eps, rows, d, (__nv_bfloat16*)y, mean,
                    rstd, s);
    else
        forward_any((const float*)x, gamma, beta, eps, rows, d, (float*)y, mean, rstd, s);
    *launches += 1;
}

void launch_layer_norm_backward(int dtype, const void* dy, const void* x, const float* gamma,
                                const float* mean, const float* rstd, const void* dres, int rows,
                                int d, void* dx, float* dgamma, float* dbeta, float* part,
                                cudaStream_t s, int* launches) {
    if (dtype == MOE_BF16) {
        using B = __nv_bfloat16;
        backward_any((const B*)dy, (const B*)x, gamma, mean, rstd, (const B*)dres, rows, d, (B*)dx,
                     dgamma, dbeta, part, s, launches);
    } else {
        backward_any((const float*)dy, (const float*)x, gamma, mean, rstd, (const float*)dres,
                     rows, d, (float*)dx, dgamma, dbeta, part, s, launches);
    }
}

}  // namespace moe

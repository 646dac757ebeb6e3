// norm.cu -- the layer norm in front of the layer, forward and backward (sm_100a).
//
//   mean = sum_c x_c / d,  rstd = 1 / sqrt(sum_c (x_c - mean)^2 / d + eps),
//   xh = (x - mean) rstd,  y = gamma xh + beta
//   g = gamma dy,  dx = rstd (g - mean_c(g) - xh mean_c(g xh)) (+ dres),
//   dgamma = sum_t dy xh,  dbeta = sum_t dy.
//
// Both passes are bound by memory: a row is read once, kept in registers, and written once.
//
// Layout.  WPR warps share a row; lane l of warp w holds the vectors of VB elements at
// (v WPR 32 + w 32 + l) VB, v < NV, so every load is contiguous over the warp.  VB is 16 bytes
// where rows and pointers allow, else one element (odd widths).  The variance is the two-pass one
// (the row is in registers, so the second pass costs no memory).  Statistics and sums are fp32:
// a lane adds at most 32 values before the tree over lanes and warps.
//
// Backward.  Persistent blocks walk the rows; each thread owns fixed columns and keeps their
// dgamma and dbeta sums in registers; row groups of a block join theirs in shared memory in
// order, blocks write one partial row each, and a second launch adds those in order.  No atomics:
// the result does not depend on scheduling.
//
// Rows wider than the register layout holds (kMaxCols) take the *_wide kernels: a block per row
// that reads the row again in each pass, and a column-wise pass for dgamma and dbeta.
#include <algorithm>
#include <cstdint>

#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kSm = 148;

// Elements a lane holds of a row: forward 32 (x alone), backward 16 (x, dy and two sums each).
constexpr int kFwdElems = 32;
constexpr int kBwdElems = 16;
constexpr int kMaxWarps = 16;
constexpr int kFwdMaxCols = kFwdElems * 32 * kMaxWarps;   // 16384
constexpr int kBwdMaxCols = kBwdElems * 32 * kMaxWarps;   // 8192

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

// Sum over the WPR warps of this thread's row (every thread of the block calls it together).
// buf: one float per warp of the block, not read any more by an earlier call.
template <int WPR>
__device__ __forceinline__ float row_sum(float v, float* buf) {
    v = warp_sum(v);
    if constexpr (WPR > 1) {
        const int warp = threadIdx.x >> 5;
        if ((threadIdx.x & 31) == 0) buf[warp] = v;
        __syncthreads();
        const int w0 = warp / WPR * WPR;
        v = buf[w0];
#pragma unroll
        for (int w = 1; w < WPR; ++w) v += buf[w0 + w];
    }
    return v;
}

template <int WPR>
constexpr int kWarpsOf = WPR > 8 ? WPR : 8;

template <class T, int VB, int WPR>
__global__ void __launch_bounds__(kWarpsOf<WPR> * 32)
    layer_norm_kernel(const T* __restrict__ x, const float* __restrict__ gamma,
                      const float* __restrict__ beta, float eps, int rows, int d,
                      T* __restrict__ y, float* __restrict__ mean, float* __restrict__ rstd) {
    pdl_begin();
    constexpr int NV = kFwdElems / VB;
    constexpr int kWarps = kWarpsOf<WPR>;
    __shared__ float s_buf[2][kWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const long long row = (long long)blockIdx.x * (kWarps / WPR) + warp / WPR;
    const bool live = row < rows;
    const int c0 = ((warp % WPR) * 32 + lane) * VB;
    const T* xr = x + row * d;
    float v[NV][VB];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = c0 + i * WPR * 32 * VB;
        load_elems<T, VB>(xr + c, live && c < d, v[i]);
    }
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int q = 0; q < VB; ++q) s += v[i][q];
    const float mu = row_sum<WPR>(s, s_buf[0]) / (float)d;
    float s2 = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = c0 + i * WPR * 32 * VB;
        if (c < d) {
#pragma unroll
            for (int q = 0; q < VB; ++q) {
                v[i][q] -= mu;
                s2 = fmaf(v[i][q], v[i][q], s2);
            }
        }
    }
    const float rs = 1.0f / sqrtf(row_sum<WPR>(s2, s_buf[1]) / (float)d + eps);
    if (!live) return;
    T* yr = y + row * d;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = c0 + i * WPR * 32 * VB;
        if (c < d) {
            float ga[VB], be[VB];
            load_params<VB>(gamma + c, ga);
            load_params<VB>(beta + c, be);
#pragma unroll
            for (int q = 0; q < VB; ++q) v[i][q] = fmaf(v[i][q] * rs, ga[q], be[q]);
            store_elems<T, VB>(yr + c, v[i]);
        }
    }
    if (warp % WPR == 0 && lane == 0) {
        mean[row] = mu;
        rstd[row] = rs;
    }
}

// One block of 512 threads per row, the row read again in each pass.
template <class T>
__global__ void __launch_bounds__(512)
    layer_norm_wide_kernel(const T* __restrict__ x, const float* __restrict__ gamma,
                           const float* __restrict__ beta, float eps, int d, T* __restrict__ y,
                           float* __restrict__ mean, float* __restrict__ rstd) {
    pdl_begin();
    __shared__ float s_buf[2][16];
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
__global__ void __launch_bounds__(kWarpsOf<WPR> * 32)
    layer_norm_backward_kernel(const T* __restrict__ dy, const T* __restrict__ x,
                               const float* __restrict__ gamma, const float* __restrict__ mean,
                               const float* __restrict__ rstd, const T* __restrict__ dres,
                               int rows, int d, T* __restrict__ dx, float* __restrict__ part) {
    pdl_begin();
    constexpr int NV = kBwdElems / VB;
    constexpr int kWarps = kWarpsOf<WPR>;
    constexpr int RPC = kWarps / WPR;                 // rows in flight per block
    __shared__ float s_buf[2][2][kWarps];
    __shared__ float s_sum[RPC > 1 ? 2 : 1][RPC > 1 ? WPR * 32 * kBwdElems : 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c0 = ((warp % WPR) * 32 + lane) * VB;
    float ga[NV][VB], dg[NV][VB], db[NV][VB];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = c0 + i * WPR * 32 * VB;
#pragma unroll
        for (int q = 0; q < VB; ++q) ga[i][q] = dg[i][q] = db[i][q] = 0.0f;
        if (c < d) load_params<VB>(gamma + c, ga[i]);
    }
    const float inv_d = 1.0f / (float)d;
    const int all = gridDim.x * RPC;
    const int steps = (int)(((long long)rows + all - 1) / all);
    for (int it = 0; it < steps; ++it) {
        const long long row = (long long)it * all + blockIdx.x * RPC + warp / WPR;
        const bool live = row < rows;
        float xv[NV][VB], gv[NV][VB];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = c0 + i * WPR * 32 * VB;
            load_elems<T, VB>(x + row * d + c, live && c < d, xv[i]);
            load_elems<T, VB>(dy + row * d + c, live && c < d, gv[i]);
        }
        const float mu = live ? mean[row] : 0.0f, rs = live ? rstd[row] : 0.0f;
        float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int q = 0; q < VB; ++q) {
                xv[i][q] = (xv[i][q] - mu) * rs;
                dg[i][q] = fmaf(gv[i][q], xv[i][q], dg[i][q]);
                db[i][q] += gv[i][q];
                gv[i][q] *= ga[i][q];
                s1 += gv[i][q];
                s2 = fmaf(gv[i][q], xv[i][q], s2);
            }
        float (*buf)[kWarps] = s_buf[it & 1];
        s1 = row_sum<1>(s1, nullptr);
        s2 = row_sum<1>(s2, nullptr);
        if constexpr (WPR > 1) {
            if (lane == 0) {
                buf[0][warp] = s1;
                buf[1][warp] = s2;
            }
            __syncthreads();
            const int w0 = warp / WPR * WPR;
            s1 = buf[0][w0];
            s2 = buf[1][w0];
#pragma unroll
            for (int w = 1; w < WPR; ++w) {
                s1 += buf[0][w0 + w];
                s2 += buf[1][w0 + w];
            }
        }
        s1 *= inv_d;
        s2 *= inv_d;
        if (live) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = c0 + i * WPR * 32 * VB;
                if (c < d) {
                    float res[VB];
                    load_elems<T, VB>(dres + row * d + c, dres != nullptr, res);
#pragma unroll
                    for (int q = 0; q < VB; ++q)
                        gv[i][q] = fmaf(gv[i][q] - s1 - xv[i][q] * s2, rs, res[q]);
                    store_elems<T, VB>(dx + row * d + c, gv[i]);
                }
            }
        }
    }
    if constexpr (RPC > 1) {
        for (int g = 0; g < RPC; ++g) {
            if (warp / WPR == g) {
#pragma unroll
                for (int i = 0; i < NV; ++i)
#pragma unroll
                    for (int q = 0; q < VB; ++q) {
                        const int c = c0 + i * WPR * 32 * VB + q;
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
            const int c = c0 + i * WPR * 32 * VB;
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

// dgamma[c] and dbeta[c] = sums over nb partial rows, in order: 32 columns x 8 slices of rows a
// block.
__global__ void __launch_bounds__(256)
    layer_norm_param_kernel(const float* __restrict__ part, int nb, int d,
                            float* __restrict__ dgamma, float* __restrict__ dbeta) {
    pdl_begin();
    __shared__ float s[8][33];
    const int cx = threadIdx.x & 31, sl = threadIdx.x >> 5;
    const long long c = (long long)blockIdx.x * 32 + cx;      // column of the 2 d sums
    float v = 0.0f;
    if (c < 2LL * d) {
#pragma unroll 4
        for (int b = sl; b < nb; b += 8) v += part[(long long)b * 2 * d + c];
    }
    s[sl][cx] = v;
    __syncthreads();
    if (sl == 0 && c < 2LL * d) {
#pragma unroll
        for (int i = 1; i < 8; ++i) v += s[i][cx];
        if (c < d) dgamma[c] = v;
        else dbeta[c - d] = v;
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
    __shared__ float s_buf[2][16];
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
int warps_per_row(int d, int elems) {
    int w = 1;
    while (w * 32 * elems < d) w *= 2;
    return w;
}

// Blocks of the backward kernel (= partial rows): what the GPU holds of them, but no block
// without a row.
int backward_blocks(int rows, int d) {
    if (d > kBwdMaxCols) return std::min(rows, 16);
    const int wpr = warps_per_row(d, kBwdElems);
    const int rpc = wpr > 8 ? 1 : 8 / wpr;
    return std::min((int)(((long long)rows + rpc - 1) / rpc), kSm * (wpr > 8 ? 1 : 2));
}

bool wide_ok(int d, int elem_bytes, std::initializer_list<const void*> ptrs) {
    if ((long long)d * elem_bytes % 16 != 0) return false;
    for (const void* p : ptrs)
        if (reinterpret_cast<uintptr_t>(p) & 15) return false;
    return true;
}

template <class T, int VB>
void forward_typed(const T* x, const float* gamma, const float* beta, float eps, int rows, int d,
                   T* y, float* mean, float* rstd, cudaStream_t s) {
    auto go = [&](auto kern, int wpr) {
        const int warps = wpr > 8 ? wpr : 8, rpc = warps / wpr;
        launch_pdl(kern, dim3((unsigned)(((long long)rows + rpc - 1) / rpc)), dim3(warps * 32), 0, s, x, gamma, beta,
                   eps, rows, d, y, mean, rstd);
    };
    switch (warps_per_row(d, kFwdElems)) {
        case 1: go(layer_norm_kernel<T, VB, 1>, 1); break;
        case 2: go(layer_norm_kernel<T, VB, 2>, 2); break;
        case 4: go(layer_norm_kernel<T, VB, 4>, 4); break;
        case 8: go(layer_norm_kernel<T, VB, 8>, 8); break;
        default: go(layer_norm_kernel<T, VB, 16>, 16); break;
    }
}

template <class T>
void forward_any(const T* x, const float* gamma, const float* beta, float eps, int rows, int d,
                 T* y, float* mean, float* rstd, cudaStream_t s) {
    if (d > kFwdMaxCols)
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
    const int nb = backward_blocks(rows, d);
    auto go = [&](auto kern, int wpr) {
        launch_pdl(kern, dim3(nb), dim3((wpr > 8 ? wpr : 8) * 32), 0, s, dy, x, gamma, mean, rstd,
                   dres, rows, d, dx, part);
    };
    switch (warps_per_row(d, kBwdElems)) {
        case 1: go(layer_norm_backward_kernel<T, VB, 1>, 1); break;
        case 2: go(layer_norm_backward_kernel<T, VB, 2>, 2); break;
        case 4: go(layer_norm_backward_kernel<T, VB, 4>, 4); break;
        case 8: go(layer_norm_backward_kernel<T, VB, 8>, 8); break;
        default: go(layer_norm_backward_kernel<T, VB, 16>, 16); break;
    }
}

template <class T>
void backward_any(const T* dy, const T* x, const float* gamma, const float* mean,
                  const float* rstd, const T* dres, int rows, int d, T* dx, float* dgamma,
                  float* dbeta, float* part, cudaStream_t s, int* launches) {
    const int nb = backward_blocks(rows, d);
    if (d > kBwdMaxCols) {
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
    launch_pdl(layer_norm_param_kernel, dim3((unsigned)((2LL * d + 31) / 32)), dim3(256), 0, s,
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

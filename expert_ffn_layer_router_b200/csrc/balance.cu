// balance.cu -- the router's training losses and their gradient (sm_100a).
//
// For the n tokens that the mask leaves (all T without one), p = softmax(L_t) over the E experts:
//   counts_e = pairs (t, j) with ids[t, j] = e,   f_e = counts_e / (n k),   P_e = sum_t p_te / n,
//   losses[0] = E sum_e f_e P_e   (load balance; 1 when both are uniform),
//   losses[1] = sum_t lse_t^2 / n (router z-loss, lse_t = log sum_e exp L_te).
// Gradient, with g = grad_losses and dw = the gradient of the k routing weights:
//   dL_te = p_te (a_te - sum_c p_tc a_tc) + 2 g1 / n lse_t p_te,
//   a_te  = g0 E f_e / n + sum_{j: ids[t,j] = e} dw_tj.
// Weights renormalised over the k are a softmax of their own, w = softmax(L_tj over j): their part of
// dL_te is sum_{j: ids[t,j] = e} w_j (dw_j - sum_i dw_i w_i), added as it is.  (Through p it would be
// p_te (..) / sum_j p_j, which is 0 / 0 or overflows where the named experts lie some 90 below the
// row's maximum.  Its sum over a row is 0, so it has no share in the other sum.)
//
// Layout.  A group of G lanes holds one token's logits in registers, 4 NV per lane (16-byte loads
// when rows allow), so a row is read once and every sum over the experts is log2 G shuffles.
// Without atomics on floats: a lane keeps the running sums of its own experts over the group's
// tokens; they are joined over the warp by shuffles, over the block and a cluster of blocks
// through (distributed) shared memory, and over the clusters by a second launch, always in the
// same order, so results do not depend on scheduling.  All sums are fp32.  A lane adds one
// probability (and one lse^2) per token of its group before the tree over lanes, warps and blocks: one
// up to a few thousand tokens, then T / (256 groups of a block), which is 8 at 65536 x 128 and 512 at
// 2^20 x 1024.  Pair counts are integers.
//
// Measured, 65536 x 128: losses 17 us, gradient 13 us (22 with that of 8 renormalised weights); the bytes
// alone take 5 and 10.  16384 x 64, masked: 9 and 4 us.  The losses are bound by their steps behind one another
// (loads, cluster, second launch), the gradient by instructions.
#include <algorithm>

#include "common.cuh"
#include "kernels.h"

namespace moe {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr uint32_t kMaxCluster = 8;
// Clusters that run together: two blocks of 512 threads fit an SM, and a cluster's 8 have to lie in one
// part (GPC) of the GPU.  With 36 the last ones wait for a second turn (65536 x 128: 23.5 us against
// 17.1 with 32, 18.4 with 28, 21.9 with 18).
constexpr int kMaxClusters = 32;

// Block size: 4 NV values, as many sums and the loads in flight have to fit the registers.
template <int NV>
constexpr int kThreadsOf = NV >= 8 ? 256 : 512;

template <int G>
__device__ __forceinline__ float group_max(float v) {
#pragma unroll
    for (int h = G / 2; h >= 1; h >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, h));
    return v;
}
template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
    for (int h = G / 2; h >= 1; h >>= 1) v += __shfl_xor_sync(kFull, v, h);
    return v;
}

// Expert of element i (0 .. 4 NV - 1) of lane l of a group.
template <int G, bool VEC>
__device__ __forceinline__ int expert_of(int l, int i) {
    return VEC ? 4 * (l + G * (i >> 2)) + (i & 3) : l + G * i;
}

// The row's logits; -inf past E and in rows that are not `live`.
template <int G, int NV, bool VEC>
__device__ __forceinline__ void load_row(const float* __restrict__ row, int E, int l, bool live,
                                         float (&v)[4 * NV]) {
    const float kNone = __int_as_float(0xff800000);
    if constexpr (VEC) {
#pragma unroll
        for (int q = 0; q < NV; ++q) {
            const int e = 4 * (l + G * q);
            float4 f = make_float4(kNone, kNone, kNone, kNone);
            if (live && e < E) f = *reinterpret_cast<const float4*>(row + e);
            v[4 * q] = f.x; v[4 * q + 1] = f.y; v[4 * q + 2] = f.z; v[4 * q + 3] = f.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4 * NV; ++i) {
            const int e = l + G * i;
            v[i] = live && e < E ? row[e] : kNone;
        }
    }
}

// exp(x), x <= 0, through the hardware's 2^t: the product x log2(e) is off by |x| 2^-24 relative to the
// result, like the rounding of x = L - max itself, and 2^t by 2 ulp.
__device__ __forceinline__ float exp_of(float x) { return __expf(x); }

// v := exp(v - max); returns (max, sum).  A row that is not live gives max = 0, sum = 1 and zeros.
template <int G, int NV>
__device__ __forceinline__ float2 softmax_terms(float (&v)[4 * NV], bool live) {
    float m = v[0];
#pragma unroll
    for (int i = 1; i < 4 * NV; ++i) m = fmaxf(m, v[i]);
    m = group_max<G>(m);
    if (!live) m = 0.0f;
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < 4 * NV; ++i) {
        v[i] = exp_of(v[i] - m);
        s += v[i];
    }
    s = group_sum<G>(s);
    return make_float2(m, live ? s : 1.0f);
}

__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ int ld_cluster_s32(uint32_t addr) {
    int v;
    asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
                 "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// Sum over the block's threads in a fixed order; valid in every thread.  buf: 32 floats.
__device__ __forceinline__ float block_sum(float v, float* buf) {
    v = group_sum<32>(v);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, nw = blockDim.x >> 5;
    __syncthreads();
    if (lane == 0) buf[warp] = v;
    __syncthreads();
    return group_sum<32>(lane < nw ? buf[lane] : 0.0f);
}

// The losses from the totals (one block): cnt(e), psum(e) give expert e's pair count and sum of
// probabilities.
template <class Cnt, class Psum>
__device__ __forceinline__ void write_losses(int E, int k, int n, float zsum, Cnt cnt, Psum psum,
                                             float* losses, int32_t* counts, float* probs,
                                             float* buf) {
    const float n1 = (float)max(n, 1);
    float dot = 0.0f;
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
        const int c = cnt(e);
        const float P = psum(e) / n1;
        counts[e] = c;
        probs[e] = P;
        dot += (float)c / (n1 * (float)k) * P;
    }
    dot = block_sum(dot, buf);
    if (threadIdx.x == 0) {
        counts[E] = n;
        losses[0] = (float)E * dot;
        losses[1] = zsum / n1;
    }
}

// Partial totals of one cluster: float psum[E], z; int count[E], n (kept together, 2 (E + 1)
// words per cluster).
// part = null: the only cluster, which writes the results itself.
template <int G, int NV, bool VEC>
__global__ void __launch_bounds__(kThreadsOf<NV>, 2)
    balance_kernel(const float* __restrict__ logits, const int32_t* __restrict__ ids,
                   const uint8_t* __restrict__ mask, int T, int E, int k, int rows_per_block,
                   float* __restrict__ part, float* losses, int32_t* counts, float* probs,
                   DeviceStatus* st) {
    pdl_begin();
    constexpr int kThreads = kThreadsOf<NV>;
    constexpr int kWarps = kThreads / 32;
    constexpr int kGroups = kThreads / G;
    extern __shared__ float sm[];
    float* s_p = sm;                                          // [kWarps][E], then [0][E] the block's
    int* s_cnt = reinterpret_cast<int*>(sm + kWarps * E);     // [E]
    float* s_z = reinterpret_cast<float*>(s_cnt + E);         // z, then n (as int)
    int* s_n = reinterpret_cast<int*>(s_z + 1);
    __shared__ float s_buf[32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int l = lane & (G - 1);
    const long long t0 = min((long long)T, (long long)blockIdx.x * rows_per_block);
    const long long t1 = min((long long)T, t0 + rows_per_block);

    for (int e = threadIdx.x; e < E; e += kThreads) s_cnt[e] = 0;
    __syncthreads();
    // Pair counts of the block's tokens.
    for (long long t = t0 + threadIdx.x; t < t1; t += kThreads) {
        if (mask && !mask[t]) continue;
#pragma unroll 8
        for (int j = 0; j < k; ++j) {
            const int e = ids[t * k + j];
            if (e >= 0 && e < E) atomicAdd(&s_cnt[e], 1);
            else report(st, MOE_DEV_BAD_INDEX, 610);
        }
    }
    float acc[4 * NV];
#pragma unroll
    for (int i = 0; i < 4 * NV; ++i) acc[i] = 0.0f;
    float z = 0.0f;
    float n = 0.0f;
    // Every group of a warp makes the same number of steps (the shuffles name the whole warp).
    // The next row's logits are loaded before this one's sums.
    const int steps = (int)((t1 - t0 + kGroups - 1) / kGroups);
    long long t = t0 + threadIdx.x / G;
    bool coming = t < t1 && (!mask || mask[t]);
    float next[4 * NV];
    load_row<G, NV, VEC>(logits + t * E, E, l, coming, next);
    for (int i = 0; i < steps; ++i) {
        const bool live = coming;
        float v[4 * NV];
#pragma unroll
        for (int q = 0; q < 4 * NV; ++q) v[q] = next[q];
        t += kGroups;
        coming = t < t1 && (!mask || mask[t]);
        load_row<G, NV, VEC>(logits + t * E, E, l, coming, next);
        const float2 ms = softmax_terms<G, NV>(v, live);
        const float r = __frcp_rn(ms.y);
#pragma unroll
        for (int q = 0; q < 4 * NV; ++q) acc[q] = fmaf(v[q], r, acc[q]);
        if (live && l == 0) {
            const float lse = ms.x + logf(ms.y);
            z = fmaf(lse, lse, z);
            n += 1.0f;
        }
    }
#pragma unroll
    for (int q = 0; q < 4 * NV; ++q) {
#pragma unroll
        for (int h = 16; h >= G; h >>= 1) acc[q] += __shfl_xor_sync(kFull, acc[q], h);
        const int e = expert_of<G, VEC>(l, q);
        if (lane < G && e < E) s_p[warp * E + e] = acc[q];
    }
    z = block_sum(z, s_buf);      // (its barriers also complete s_p and s_cnt)
    n = block_sum(n, s_buf);      // at most T <= 2^24 tokens a block: exact
    for (int e = threadIdx.x; e < E; e += kThreads) {
        float p = s_p[e];
        for (int w = 1; w < kWarps; ++w) p += s_p[w * E + e];
        s_p[e] = p;
    }
    if (threadIdx.x == 0) {
        *s_z = z;
        *s_n = (int)n;
    }
    uint32_t rank, size;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(size));
    if (size > 1) cluster_sync(); else __syncthreads();
    if (rank == 0) {
        const uint32_t a_p = smem_u32(s_p), a_c = smem_u32(s_cnt), a_z = smem_u32(s_z);
        // (all ranks' words in flight together, added in rank order)
        auto psum_at = [&](uint32_t a) {
            float f[kMaxCluster], v = 0.0f;
#pragma unroll
            for (uint32_t r = 0; r < kMaxCluster; ++r)
                f[r] = r < size ? ld_cluster_f32(map_rank(a, r)) : 0.0f;
#pragma unroll
            for (uint32_t r = 0; r < kMaxCluster; ++r) v += f[r];
            return v;
        };
        auto cnt_at = [&](uint32_t a) {
            int f[kMaxCluster], v = 0;
#pragma unroll
            for (uint32_t r = 0; r < kMaxCluster; ++r)
                f[r] = r < size ? ld_cluster_s32(map_rank(a, r)) : 0;
#pragma unroll
            for (uint32_t r = 0; r < kMaxCluster; ++r) v += f[r];
            return v;
        };
        auto psum = [&](int e) { return psum_at(a_p + 4 * e); };
        auto cnt = [&](int e) { return cnt_at(a_c + 4 * e); };
        const float zs = psum_at(a_z);
        const int ns = cnt_at(a_z + 4);
        if (part) {
            float* o = part + (long long)(blockIdx.x / size) * 2 * (E + 1);
            int* oc = reinterpret_cast<int*>(o + E + 1);
            for (int e = threadIdx.x; e < E; e += kThreads) {
                o[e] = psum(e);
                oc[e] = cnt(e);
            }
            if (threadIdx.x == 0) {
                o[E] = zs;
                oc[E] = ns;
            }
        } else {
            write_losses(E, k, ns, zs, cnt, psum, losses, counts, probs, s_buf);
        }
    }
    if (size > 1) cluster_sync();      // the peers' shared memory stays until rank 0 has read it
}

// Joins the clusters' totals (one block): thread (g, c) adds column c of clusters g, g + groups, ...,
// whose loads are all in flight together, and the groups' sums are added in order.
__global__ void __launch_bounds__(1024)
    balance_final_kernel(const float* __restrict__ part, int nc, int E, int k, float* losses,
                         int32_t* counts, float* probs) {
    pdl_begin();
    __shared__ float s_buf[32];
    extern __shared__ float s_part[];                         // [groups][cols], then row 0 the totals
    const int cols = 2 * (E + 1);                             // floats, then ints from E + 1 on
    const int groups = cols > 1024 ? 1 : 1024 / cols;
    const int* ipart = reinterpret_cast<const int*>(part);
    int* s_ipart = reinterpret_cast<int*>(s_part);
    const int g = groups == 1 ? 0 : threadIdx.x / cols;
    for (int c = threadIdx.x - g * cols; c < cols && g < groups; c += 1024) {
        float f = 0.0f;
        int n = 0;
#pragma unroll 12
        for (int i = g; i < nc; i += groups) {
            if (c <= E) f += part[(long long)i * cols + c];
            else n += ipart[(long long)i * cols + c];
        }
        if (c <= E) s_part[g * cols + c] = f;
        else s_ipart[g * cols + c] = n;
    }
    __syncthreads();
    for (int c = threadIdx.x; c < cols; c += 1024) {
        for (int i = 1; i < groups; ++i) {
            if (c <= E) s_part[c] += s_part[i * cols + c];
            else s_ipart[c] += s_ipart[i * cols + c];
        }
    }
    __syncthreads();
    write_losses(E, k, s_ipart[E + 1 + E], s_part[E], [&](int e) { return s_ipart[E + 1 + e]; },
                 [&](int e) { return s_part[e]; }, losses, counts, probs, s_buf);
}

template <int G, int NV, bool VEC>
__global__ void __launch_bounds__(kThreadsOf<NV>)
    route_backward_kernel(const float* __restrict__ logits, const int32_t* __restrict__ ids,
                          const uint8_t* __restrict__ mask, const int32_t* __restrict__ counts,
                          const float* __restrict__ grad_losses,
                          const float* __restrict__ grad_w, int T, int E, int k, bool renorm,
                          float* __restrict__ dlogits, DeviceStatus* st) {
    pdl_begin();
    constexpr int kGroups = kThreadsOf<NV> / G;
    const int lane = threadIdx.x & 31;
    const int l = lane & (G - 1);
    // a_e without the routing weights' part, per lane; counts[E] = 0 only if no token is left.
    float base[4 * NV];
    float gz = 0.0f, scale = 0.0f;
    if (grad_losses) {
        const float n1 = (float)max(counts[E], 1);
        scale = grad_losses[0] * (float)E / (n1 * n1 * (float)k);
        gz = 2.0f * grad_losses[1] / n1;
    }
#pragma unroll
    for (int i = 0; i < 4 * NV; ++i) {
        const int e = expert_of<G, VEC>(l, i);
        base[i] = grad_losses && e < E ? scale * (float)counts[e] : 0.0f;
    }
    // grad_w: the group's row of dw (zeros between tokens) and of the lanes that own its entries.
    // Renormalised: of the finished terms of dL instead.
    extern __shared__ __align__(16) float s_rows[];
    float* row = s_rows + (threadIdx.x / G) * E;
    uint8_t* own = reinterpret_cast<uint8_t*>(s_rows + kGroups * E) + (threadIdx.x / G) * E;
    if (grad_w) {
        for (int e = l; e < E; e += G) row[e] = 0.0f;
        __syncwarp();
    }
    const bool added = renorm && grad_w;
    const long long all = (long long)gridDim.x * kGroups;
    const long long steps = (T + all - 1) / all;
    long long t = (long long)blockIdx.x * kGroups + threadIdx.x / G;
    // What a step reads of memory is loaded during the step before.
    float next[4 * NV];
    bool coming;
    int next_id = -1;
    float next_dw = 0.0f;
    auto fetch = [&]() {
        coming = t < T && (!mask || mask[t]);
        load_row<G, NV, VEC>(logits + t * E, E, l, coming, next);
        if (grad_w) {
            next_id = coming && l < k ? ids[t * k + l] : -1;
            next_dw = coming && l < k ? grad_w[t * k + l] : 0.0f;
        }
    };
    fetch();
    for (long long i = 0; i < steps; ++i) {
        const long long at = t;
        const bool in = at < T, live = coming;
        float v[4 * NV];
#pragma unroll
        for (int q = 0; q < 4 * NV; ++q) v[q] = next[q];
        int id = next_id;
        float dw = next_dw;
        t += all;
        fetch();
        const float2 ms = softmax_terms<G, NV>(v, live);
        const float r = __frcp_rn(ms.y);
        float a[4 * NV];
#pragma unroll
        for (int q = 0; q < 4 * NV; ++q) a[q] = base[q];
        if (grad_w) {
            // Lane j < k of the group holds pair j: its expert and dw.
            if (live && l < k && (id < 0 || id >= E)) {
                report(st, MOE_DEV_BAD_INDEX, 620);
                id = -1;
                dw = 0.0f;
            }
            if (renorm) {
                const float kNone = __int_as_float(0xff800000);
                const float lj = id >= 0 ? logits[at * E + id] : kNone;
                const float top = group_max<G>(lj);
                const float u = lj > kNone ? exp_of(lj - top) : 0.0f;
                const float sum = group_sum<G>(u);             // (at least 1, or no pair: 0)
                const float d = group_sum<G>(dw * u);
                const float rs = __frcp_rn(sum > 0.0f ? sum : 1.0f);
                dw = u * rs * (dw - d * rs);
            }
            // An expert named twice: the lane that did not win its entry sees another's number
            // there, and its pairs' dw are added up (in pair order) in every lane that names it.
            if (id >= 0) own[id] = (uint8_t)l;
            __syncwarp();
            if (__any_sync(kFull, id >= 0 && own[id] != l)) {
                float sum = 0.0f;
                for (int j = 0; j < G; ++j) {
                    const int oid = __shfl_sync(kFull, id, j, G);
                    const float o = __shfl_sync(kFull, dw, j, G);
                    if (oid == id) sum += o;
                }
                dw = sum;
            }
            if (id >= 0) row[id] = dw;
            __syncwarp();
            if (!renorm) {
#pragma unroll
                for (int q = 0; q < 4 * NV; ++q) {
                    const int e = expert_of<G, VEC>(l, q);
                    if (e < E) a[q] += row[e];
                }
            }
        }
        float dot = 0.0f;
#pragma unroll
        for (int q = 0; q < 4 * NV; ++q) {
            v[q] *= r;
            dot = fmaf(v[q], a[q], dot);
        }
        dot = group_sum<G>(dot);
        const float shift = live ? gz * (ms.x + logf(ms.y)) - dot : 0.0f;
        if (in) {
            float* out = dlogits + at * E;
            if constexpr (VEC) {
#pragma unroll
                for (int q = 0; q < NV; ++q) {
                    const int e = 4 * (l + G * q);
                    if (e < E) {
                        float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                        if (added) x = *reinterpret_cast<const float4*>(row + e);
                        *reinterpret_cast<float4*>(out + e) =
                            make_float4(fmaf(v[4 * q], a[4 * q] + shift, x.x),
                                        fmaf(v[4 * q + 1], a[4 * q + 1] + shift, x.y),
                                        fmaf(v[4 * q + 2], a[4 * q + 2] + shift, x.z),
                                        fmaf(v[4 * q + 3], a[4 * q + 3] + shift, x.w));
                    }
                }
            } else {
#pragma unroll
                for (int q = 0; q < 4 * NV; ++q) {
                    const int e = l + G * q;
                    if (e < E) out[e] = fmaf(v[q], a[q] + shift, added ? row[e] : 0.0f);
                }
            }
        }
        if (grad_w) {
            __syncwarp();
            if (id >= 0) row[id] = 0.0f;
        }
    }
}

struct Shape { int cfg, G, NV; };

// Lanes per token and 16-byte vectors per lane: the fewest lanes that hold E experts in 8
// registers each (few shuffles per token), at least `lanes`.
Shape shape_of(int E, int lanes) {
    static const Shape kShapes[] = {{0, 8, 1}, {1, 8, 2}, {2, 16, 2}, {3, 32, 2}, {4, 32, 4},
                                    {5, 32, 8}};
    for (const Shape& s : kShapes)
        if (s.G * s.NV * 4 >= E && s.G >= lanes) return s;
    return kShapes[5];
}

struct Grid { int threads, rows_per_block, blocks, cluster; };

// Blocks and clusters of the loss kernel: one step per group while one cluster can hold the
// batch, then as many clusters of 8 as the GPU holds blocks.
Grid grid_of(int T, const Shape& s) {
    Grid g;
    g.threads = s.NV >= 8 ? 256 : 512;
    const int groups = g.threads / s.G;
    const long long need = std::max<long long>(1, ((long long)T + groups - 1) / groups);
    if (need <= 2 * (int)kMaxCluster) {
        g.cluster = 1;
        while (g.cluster < (int)kMaxCluster && g.cluster < need) g.cluster *= 2;
        g.blocks = g.cluster;
    } else {
        g.cluster = kMaxCluster;
        const long long clusters = std::min<long long>((need + kMaxCluster - 1) / (int)kMaxCluster,
                                                       kMaxClusters);
        g.blocks = (int)clusters * kMaxCluster;
    }
    g.rows_per_block = (int)(((long long)T + g.blocks - 1) / g.blocks);
    return g;
}

bool vec_ok(const void* a, const void* b, int E) {
    return E % 4 == 0 && (reinterpret_cast<uintptr_t>(a) & 15) == 0 &&
           (reinterpret_cast<uintptr_t>(b) & 15) == 0;
}

template <int G, int NV, bool VEC>
void run_balance(const Grid& g, const float* logits, const int32_t* ids, const uint8_t* mask,
                 int T, int E, int k, float* part, float* losses, int32_t* counts, float* probs,
                 DeviceStatus* st, cudaStream_t s) {
    auto kern = balance_kernel<G, NV, VEC>;
    // At most 17 x 512 floats (E <= 512: 16 warps) or 9 x 1024: below 48 KB.
    const size_t smem = ((size_t)(g.threads / 32 + 1) * E + 2) * 4;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(g.blocks);
    cfg.blockDim = dim3(g.threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = g.cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    float* none = nullptr;
    note_launch(cudaLaunchKernelEx(&cfg, kern, logits, ids, mask, T, E, k, g.rows_per_block,
                                   g.blocks > g.cluster ? part : none, losses, counts, probs, st));
}

template <int G, int NV, bool VEC>
void run_backward(const float* logits, const int32_t* ids, const uint8_t* mask,
                  const int32_t* counts, const float* grad_losses, const float* grad_w, int T,
                  int E, int k, bool renorm, float* dlogits, DeviceStatus* st, cudaStream_t s) {
    constexpr int threads = kThreadsOf<NV>;
    const long long need = ((long long)T + threads / G - 1) / (threads / G);
    const int blocks = (int)std::min<long long>(need, 148LL * 4);
    // Rows of dw (float) and of their lanes (byte): at most 16 x 512 x 5 bytes, below 48 KB.
    const size_t smem = grad_w ? (size_t)(threads / G) * E * 5 : 0;
    launch_pdl(route_backward_kernel<G, NV, VEC>, dim3(blocks), dim3(threads), smem, s, logits, ids,
               mask, counts, grad_losses, grad_w, T, E, k, renorm, dlogits, st);
}

#define MOE_BALANCE_CASES(F, ...)                                   \
    switch (sh.cfg) {                                               \
        case 0: F<8, 1, VEC>(__VA_ARGS__); break;                   \
        case 1: F<8, 2, VEC>(__VA_ARGS__); break;                   \
        case 2: F<16, 2, VEC>(__VA_ARGS__); break;                  \
        case 3: F<32, 2, VEC>(__VA_ARGS__); break;                  \
        case 4: F<32, 4, VEC>(__VA_ARGS__); break;                  \
        default: F<32, 8, VEC>(__VA_ARGS__); break;                 \
    }

}  // namespace

size_t balance_scratch_bytes(int T, int E) {
    const Grid g = grid_of(T, shape_of(E, 1));
    return g.blocks > g.cluster ? (size_t)(g.blocks / g.cluster) * 2 * (E + 1) * 4 : 0;
}

void launch_balance(const float* logits, const int32_t* ids, const uint8_t* mask, int T, int E,
                    int k, float* part, float* losses, int32_t* counts, float* probs,
                    DeviceStatus* st, cudaStream_t s, int* launches) {
    const Shape sh = shape_of(E, 1);
    const Grid g = grid_of(T, sh);
    if (vec_ok(logits, logits, E)) {
        constexpr bool VEC = true;
        MOE_BALANCE_CASES(run_balance, g, logits, ids, mask, T, E, k, part, losses, counts, probs, st, s)
    } else {
        constexpr bool VEC = false;
        MOE_BALANCE_CASES(run_balance, g, logits, ids, mask, T, E, k, part, losses, counts, probs, st, s)
    }
    *launches += 1;
    if (g.blocks > g.cluster) {
        const size_t smem = (size_t)std::max(1024, 2 * (E + 1)) * 4;
        launch_pdl(balance_final_kernel, dim3(1), dim3(1024), smem, s, (const float*)part,
                   g.blocks / g.cluster, E, k, losses, counts, probs);
        *launches += 1;
    }
}

void launch_route_backward(const float* logits, const int32_t* ids, const uint8_t* mask,
                           const int32_t* counts, const float* grad_losses, const float* grad_w,
                           int T, int E, int k, bool renorm, float* dlogits, DeviceStatus* st,
                           cudaStream_t s, int* launches) {
    const Shape sh = shape_of(E, grad_w ? k : 1);
    if (vec_ok(logits, dlogits, E)) {
        constexpr bool VEC = true;
        MOE_BALANCE_CASES(run_backward, logits, ids, mask, counts, grad_losses, grad_w, T, E, k, renorm, dlogits, st, s)
    } else {
        constexpr bool VEC = false;
        MOE_BALANCE_CASES(run_backward, logits, ids, mask, counts, grad_losses, grad_w, T, E, k, renorm, dlogits, st, s)
    }
    *launches += 1;
}

}  // namespace moe

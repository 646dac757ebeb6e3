// common.cuh -- device helpers shared by the MoE kernels (sm_100a only).
#pragma once

#include <atomic>
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <mutex>

#include "../../include/moe_b200.h"

namespace moe {

// Workspace header: the first 256 bytes of every workspace.
struct DeviceStatus {
    int32_t code;      // MOE_DEV_*; first error wins, but a timeout replaces a bad index
    int32_t where;     // kernel-specific detail of that error
};

constexpr uint64_t kWaitLimitNs = 2000000000ull;   // a pipeline wait gives up after ~2 s

__device__ __forceinline__ uint64_t global_ns() {
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

__device__ __forceinline__ void report(DeviceStatus* st, int code, int where) {
    if (st && atomicCAS(&st->code, 0, code) == 0) st->where = where;
}

// A wait gave up: work is left out, which is more than a bad index costs, so it replaces one.
__device__ __forceinline__ void report_timeout(DeviceStatus* st, int where) {
    if (st && atomicExch(&st->code, MOE_DEV_TIMEOUT) != MOE_DEV_TIMEOUT) st->where = where;
}

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// ---------------------------------------------------------------------------------------------
// mbarrier
// ---------------------------------------------------------------------------------------------
__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void mbar_arrive_expect_tx(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
                 : "memory");
}

// kCluster: acquire at cluster scope (the phase was completed by arrivals from the other CTA of
// a pair); otherwise at CTA scope.
template <bool kCluster = false>
__device__ __forceinline__ bool mbar_try_wait(uint32_t bar, uint32_t parity) {
    uint32_t ok;
    if (kCluster)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar), "r"(parity)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(ok)
            : "r"(bar), "r"(parity)
            : "memory");
    return ok != 0;
}

// Waits for the phase of parity `parity` to complete.  Gives up after kWaitLimitNs, recording a
// timeout, or once another wait has recorded one, and then returns false.  (A bad index is an error
// of the data: it stops no thread, every phase still completes, and the rows beside it are valid.)
// The status word and the clock are read only every 32nd retry, so that a waiting thread is back in
// try_wait (not in a global load) when the phase completes.
template <bool kCluster = false>
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t parity, DeviceStatus* st,
                                          int where, uint64_t limit_ns = kWaitLimitNs) {
    if (mbar_try_wait<kCluster>(bar, parity)) return true;
    const uint64_t t0 = global_ns();
    for (uint32_t n = 1;; ++n) {
        if (mbar_try_wait<kCluster>(bar, parity)) return true;
        if ((n & 31u) == 0) {
            if (*reinterpret_cast<volatile int32_t*>(&st->code) == MOE_DEV_TIMEOUT) return false;
            if (global_ns() - t0 > limit_ns) {
                report_timeout(st, where);
                return false;
            }
        }
    }
}

// For a thread whose wait gave up: bulk copies and products that it has issued may still be on
// their way and must be done before the block's shared and tensor memory go away.  They take
// microseconds; what they would arrive on may never complete, so this waits a millisecond.
__device__ __forceinline__ void settle() {
    const uint64_t t0 = global_ns();
    while (global_ns() - t0 < 1000000ull) __nanosleep(1000);
}

// ---------------------------------------------------------------------------------------------
// Async copies
// ---------------------------------------------------------------------------------------------
__device__ __forceinline__ void cp_async_16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// 16 bytes to shared memory: copied (bytes = 16) or zeros (bytes = 0).
__device__ __forceinline__ void cp_async_16z(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes)
                 : "memory");
}
// Arrives on `bar` (asynchronously) once every cp.async issued so far by this thread has
// completed; the barrier's expected count includes this arrival (.noinc).
__device__ __forceinline__ void cp_async_arrive_noinc(uint32_t bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
    asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int N>
__device__ __forceinline__ void cp_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// Makes this thread's generic-proxy shared-memory writes visible to the async proxy
// (tensor-core operand reads).
__device__ __forceinline__ void fence_proxy_async_smem() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

__device__ __forceinline__ void tma_load_2d(uint32_t dst, const void* tmap, uint32_t bar, int c0,
                                            int c1) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
        "l"(tmap), "r"(bar), "r"(c0), "r"(c1)
        : "memory");
}

// ---------------------------------------------------------------------------------------------
// tcgen05 (5th-generation tensor cores, accumulators in tensor memory)
// ---------------------------------------------------------------------------------------------
__device__ __forceinline__ void tmem_alloc(uint32_t dst_smem, uint32_t ncols) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     dst_smem),
                 "r"(ncols)
                 : "memory");
}
__device__ __forceinline__ void tmem_relinquish() {
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t ncols) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols)
                 : "memory");
}
__device__ __forceinline__ void tc_fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// D[tmem] (+)= A[smem] * B[smem]^T, bf16 inputs, fp32 accumulate.
__device__ __forceinline__ void tc_mma_bf16(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc,
                                            uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
        "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}
// Arrives once on `bar` when every tcgen05.mma issued so far by this thread has completed.
__device__ __forceinline__ void tc_commit(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(bar)
        : "memory");
}
// Shared-memory matrix descriptor of a K-major operand tile stored with the 128-byte swizzle:
// rows of 64 bf16 (128 B), 8-row groups 1024 B apart, tile base 1024-byte aligned.
__device__ __forceinline__ uint64_t smem_desc_sw128(uint32_t saddr) {
    uint64_t d = 0;
    d |= (uint64_t)((saddr & 0x3FFFFu) >> 4);       // start address, 16-byte units
    d |= (uint64_t)1 << 16;                           // leading offset (unused when swizzled)
    d |= (uint64_t)(1024u >> 4) << 32;                // stride offset: next 8-row group
    d |= (uint64_t)1 << 46;                           // descriptor version (sm_100)
    d |= (uint64_t)2 << 61;                           // swizzle mode: 128 B
    return d;
}

// Instruction descriptor: bf16 x bf16 -> fp32, both operands K-major, M = m (128, or 256 for a
// CTA pair), N = n.
__host__ __device__ constexpr uint32_t idesc_bf16(int m, int n) {
    return (1u << 4)                       // D format fp32
           | (1u << 7)                     // A format bf16
           | (1u << 10)                    // B format bf16
           | ((uint32_t)(n >> 3) << 17)    // N / 8
           | ((uint32_t)(m >> 4) << 24);   // M / 16
}

// ---------------------------------------------------------------------------------------------
// Programmatic dependent launch.  Most kernels start with pdl_begin(): it waits until the
// preceding grid in the stream has completed and its memory is visible (a no-op without a
// programmatic dependency), then lets the next grid be scheduled, whose blocks in turn park in
// their own wait.  A dependent grid is scheduled only once every block of this grid has
// triggered, so all of them are resident by then and a waiting dependent cannot starve them.
// No kernel reads memory that a predecessor writes, or writes any memory, before its wait.
// Kernels whose set-up needs nothing from their predecessors split the two steps: the
// small-batch router and dispatch trigger first, so the expert GEMM can be scheduled early; a
// weight-streaming GEMM does its set-up (barriers, tensor memory, an L2 prefetch of its weights,
// which are read but never written by the call) before it waits.
// ---------------------------------------------------------------------------------------------
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void pdl_trigger() {
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void pdl_begin() {
    pdl_wait();
    pdl_trigger();
}

// The first failed launch (or stream operation) of the current API call on this host thread; the
// entry points clear it on entry and report it as MOE_ERR_CUDA.
inline thread_local cudaError_t g_launch_error = cudaSuccess;
inline cudaError_t note_launch(cudaError_t e) {
    if (e != cudaSuccess && g_launch_error == cudaSuccess) g_launch_error = e;
    return e;
}

// <<<grid, block, smem, s>>> with the programmatic-stream-serialization attribute.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                       cudaStream_t s, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return note_launch(cudaLaunchKernelEx(&cfg, kernel, args...));
}

// Lets `kernel` use `bytes` of dynamic shared memory on the current device (raised as needed; a
// kernel's limit is asked for once per device, as the driver call costs a microsecond).  Raised by
// one thread at a time: a smaller size set after a larger one would lower the limit again.
inline std::mutex g_smem_mutex;
template <typename... KArgs>
cudaError_t allow_smem(void (*kernel)(KArgs...), std::atomic<int> (&allowed)[64], int bytes) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return note_launch(e);
    auto enough = [&] { return dev < 64 && allowed[dev].load(std::memory_order_acquire) >= bytes; };
    if (enough()) return cudaSuccess;
    std::lock_guard<std::mutex> lock(g_smem_mutex);
    if (enough()) return cudaSuccess;
    e = note_launch(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         bytes));
    if (e == cudaSuccess && dev < 64) allowed[dev].store(bytes, std::memory_order_release);
    return e;
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&v);
}

}  // namespace moe

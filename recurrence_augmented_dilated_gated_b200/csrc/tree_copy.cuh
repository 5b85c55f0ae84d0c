// tree_copy.cuh -- mbarriers with bounded waits and TMA loads of cache rows, for
// the tensor-core forms of the tree step.
#pragma once

#include <cuda.h>

#include "rat_internal.cuh"

namespace rat {

// 3-D map (d, rows, blocks) of a [blocks, rows, d] tensor, box (128 bytes of
// channels, box_rows, 1), 128-byte swizzle (tree_maps.cu); false: the driver refused
bool encode_map_rows(CUtensorMap *map, const void *base, int dtype, long long rows, long long blocks, int d, int box_rows);

__device__ __forceinline__ uint32_t smem_u32(const void *p) {
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void mbar_init(uint64_t *bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(count) : "memory");
}
__device__ __forceinline__ void mbar_expect(uint64_t *bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap *map, uint64_t *bar, int x, int y, int z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void mbar_arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ bool mbar_try(uint64_t *bar, uint32_t parity) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}\n"
        : "=r"(ok) : "r"(smem_u32(bar)), "r"(parity) : "memory");
    return ok != 0;
}
// The waits of a CTA (shared memory): how long one may take, in ns, and whether a role
// gave up.  32 bits of the timer: a wait of more than two seconds is cut to that.
struct Waits {
    unsigned limit;
    volatile int abort;
};
__device__ __forceinline__ unsigned global_ns_lo() {
    unsigned t;
    asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t));
    return t;
}
// What the workspace's header says of them (as of the scan's): read where a kernel
// begins, used by the same thread once its first barrier is past, when the values have
// come (waiting for them before it took 2 us of a step of 423).  With failure injection the
// CTA's first tile, `bar`, awaits bytes that do not come.
struct WaitSettings {
    long long limit, stall;
};
__device__ __forceinline__ WaitSettings start_waits(Waits &w, const WsHeader *hdr) {
    w.limit = (unsigned)kDefaultSpinNs;
    w.abort = 0;
    return {hdr->spin_limit_ns, hdr->stall_ticket_plus1};
}
__device__ __forceinline__ void set_waits(Waits &w, const WaitSettings &s, uint64_t *bar) {
    if (s.limit > 0) w.limit = (unsigned)min(s.limit, 2000000000LL);
    if (s.stall == (long long)blockIdx.x + 1)
        asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], 16;" ::"r"(smem_u32(bar)) : "memory");
}
// False when the wait gave up or another role of the CTA has.
static __device__ __noinline__ bool mbar_wait_slow(uint64_t *bar, uint32_t parity, Waits *w) {
    const unsigned t0 = global_ns_lo();
    while (!mbar_try(bar, parity))
        if (w->abort || global_ns_lo() - t0 > w->limit) return false;
    return true;
}
__device__ __forceinline__ bool mbar_wait(uint64_t *bar, uint32_t parity, Waits *w) {
    return mbar_try(bar, parity) || mbar_wait_slow(bar, parity, w);
}
// For what is in flight when a CTA gives up: the default limit, and nothing ends it early.
static __device__ __noinline__ void mbar_drain(uint64_t *bar, uint32_t parity) {
    const unsigned long long t0 = global_ns();
    while (!mbar_try(bar, parity))
        if ((long long)(global_ns() - t0) > kDefaultSpinNs) return;
}
// orders this thread's ordinary accesses to shared memory before later TMA and
// tcgen05 accesses (with the barrier that follows)
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

}  // namespace rat

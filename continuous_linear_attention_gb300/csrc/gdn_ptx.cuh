// Thin inline-PTX wrappers for sm_103a: mbarriers, bulk (TMA) copies, and a
// wall-clock for bounded waits.  Every wait in this library gives up after a
// time limit and reports it through the layer's error word instead of
// spinning forever.
#pragma once

#include <stdint.h>

namespace gdn {

// A wait that has not completed after this many nanoseconds gives up.
constexpr uint64_t kWaitLimitNs = 2000000000ull;  // 2 s

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}

__device__ __forceinline__ uint64_t global_timer_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}

__device__ __forceinline__ void mbar_init(uint64_t* bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(count)
               : "memory");
}

// Makes initialised mbarriers visible to the async proxy (bulk copies).
__device__ __forceinline__ void fence_mbar_init() {
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

__device__ __forceinline__ void mbar_arrive_expect_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)),
               "r"(bytes)
               : "memory");
}

// One test of the phase; a thread whose phase is not complete may be
// suspended until it completes or for at most kSuspendNs, instead of
// spinning on the issue slots other warps could use.
constexpr uint32_t kSuspendNs = 200000;
__device__ __forceinline__ bool mbar_try_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity), "r"(kSuspendNs)
      : "memory");
  return ok != 0;
}

// Waits for the phase with the given parity to complete, for at most
// kWaitLimitNs.  Returns false on timeout.
__device__ __forceinline__ bool mbar_wait_bounded(uint64_t* bar, uint32_t parity) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity)) {
    if (global_timer_ns() - t0 > kWaitLimitNs) return false;
  }
  return true;
}

// Programmatic dependent launch: wait until the grid launched before this one
// on the stream has completed and its writes are visible (returns at once for
// a grid launched without the programmatic attribute), then allow the next
// grid to be scheduled while this one runs (its own wait keeps it ordered).
// The order of a stream's kernels rests on these rules:
//  - every kernel waits before it ends, so that its completion is also that of
//    all before it, and writes to global memory before its wait only what no
//    kernel before it touches;
//  - a kernel that is to read global memory before its wait reads what the
//    kernels before its predecessor have written, which is there if the
//    predecessor releases after its own wait, as here.
// Reading early are schedule_kernel (the call's lists; it also releases at
// once, so the kernel behind it may not) and the late kernels behind a prompt
// batch's last one, windowed attention's for few tokens behind its prompts' among
// them (the scheduler's lists, the inputs and states of other
// sequences; they release at once too, so that a scheduler may start beside
// them and the kernel before them, which write no lists).  The one writer of
// lists is plan_compact_kernel: move_blocks_kernel, always behind it, must not
// release before its wait.
__device__ __forceinline__ void pdl_wait_then_release() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Bulk global -> shared copy completing on `bar` (tx bytes).  Addresses
// 16-byte aligned, bytes a multiple of 16.
__device__ __forceinline__ void bulk_g2s(void* dst, const void* src, uint32_t bytes,
                                         uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

// Bulk shared -> global copy (async proxy), tracked in this thread's bulk
// group; addresses 16-byte aligned, bytes a multiple of 16.  The shared bytes
// must have been made visible to the async proxy (fence.proxy.async) by the
// threads that wrote them.
__device__ __forceinline__ void bulk_s2g(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst),
               "r"(smem_u32(src)), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void bulk_commit() {
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
// Wait until every committed bulk store of this thread has read its source
// (the shared bytes may be rewritten), or has completed entirely.
__device__ __forceinline__ void bulk_wait_read_all() {
  asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}
// The same for all but the most recently committed group.
__device__ __forceinline__ void bulk_wait_read_but_last() {
  asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
}
__device__ __forceinline__ void bulk_wait_all() {
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

}  // namespace gdn

namespace gdn {

// 2-D tiled TMA load (cp.async.bulk.tensor) of the box at coordinates
// (c0 = innermost, r0) of the tensor described by *tmap into shared memory,
// completing on `bar`.  c0 times the element size must be a multiple of 16
// bytes; r0 may be negative or past the end (those rows read as zero).
__device__ __forceinline__ void tma_load_2d(void* dst, const void* tmap, int c0, int r0,
                                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(c0), "r"(r0), "r"(smem_u32(bar))
      : "memory");
}

}  // namespace gdn

// cq_async.cuh -- shared-memory mbarriers, bulk (TMA) copies and the bounded
// wait used by every kernel of libcq that waits on its own copies.
#pragma once

#include <stdint.h>

namespace cq {
namespace async {

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
  return (uint32_t)__cvta_generic_to_shared(p);
}

__device__ __forceinline__ void mbar_init(uint64_t* bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(count)
               : "memory");
}

// Makes the initialised barriers visible to the bulk-copy (async) proxy.
__device__ __forceinline__ void mbar_fence_init() {
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// The producer's one arrival, announcing `bytes` of bulk copies.
__device__ __forceinline__ void mbar_arrive_expect_tx(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)),
               "r"(bytes)
               : "memory");
}

// Bulk copy global -> shared memory, completing `bytes` on `bar`. Both
// addresses 16-byte aligned, size a multiple of 16.
__device__ __forceinline__ void bulk_load(void* sdst, const void* gsrc, uint32_t bytes,
                                          uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(smem_u32(sdst)),
      "l"(gsrc), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ uint64_t globaltimer_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}

__device__ __forceinline__ bool mbar_try_wait(uint32_t bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}"
      : "=r"(done)
      : "r"(bar), "r"(parity)
      : "memory");
  return done != 0;
}

// Limits of every wait: about one second of the global timer, or this many
// polls, whichever comes first (the poll cap ends the wait even if the timer
// did not advance).
constexpr uint64_t kWaitLimitNs = 1000000000ull;
constexpr uint32_t kWaitMaxPolls = 1u << 24;

// Wait for the completion of phase `parity` of `bar`; false when a limit was
// reached first.
__device__ __forceinline__ bool mbar_wait(uint64_t* bar, uint32_t parity) {
  const uint32_t a = smem_u32(bar);
  if (mbar_try_wait(a, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t polls = 0; polls < kWaitMaxPolls; ++polls) {
    if (mbar_try_wait(a, parity)) return true;
    if (globaltimer_ns() - t0 > kWaitLimitNs) return false;
  }
  return false;
}

// Polls try_wait with the same limits by all lanes of a converged warp, with one
// verdict for the warp: lanes that poll and read the clock each for itself may
// differ. The votes make every branch uniform.
template <typename Try>
__device__ __forceinline__ bool wait_warp(Try try_wait) {
  constexpr uint32_t kAll = 0xffffffffu;
  if (__all_sync(kAll, try_wait())) return true;
  const uint64_t t0 = globaltimer_ns();
  for (uint32_t polls = 0; polls < kWaitMaxPolls; ++polls) {
    if (__all_sync(kAll, try_wait())) return true;
    if (__any_sync(kAll, globaltimer_ns() - t0 > kWaitLimitNs)) return false;
  }
  return false;
}

// mbar_wait by a converged warp.
__device__ __forceinline__ bool mbar_wait_warp(uint64_t* bar, uint32_t parity) {
  const uint32_t a = smem_u32(bar);
  return wait_warp([=] { return mbar_try_wait(a, parity); });
}

// Named barrier 1 of THREADS threads, and whether `ok` is true in all of them.
// Warps whose waits may have given up each for itself meet here before any other
// barrier, so that they go on, or leave, together.
template <int THREADS>
__device__ __forceinline__ bool meet(bool ok) {
  uint32_t all;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 q, %1, 0;\n bar.red.and.pred p, 1, %2, q;\n"
      " selp.u32 %0, 1, 0, p;\n}"
      : "=r"(all)
      : "r"((uint32_t)ok), "n"(THREADS)
      : "memory");
  return all != 0;
}
// The same at named barrier `id`.
template <int THREADS>
__device__ __forceinline__ bool meet(bool ok, int id) {
  uint32_t all;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 q, %1, 0;\n bar.red.and.pred p, %2, %3, q;\n"
      " selp.u32 %0, 1, 0, p;\n}"
      : "=r"(all)
      : "r"((uint32_t)ok), "r"(id), "n"(THREADS)
      : "memory");
  return all != 0;
}

// Hand a ring slot back to the producer after this warp has read it with
// ordinary (generic-proxy) shared-memory loads. The next write into the slot
// is a bulk copy (async proxy), which the release/acquire pair of the empty
// mbarrier alone does not order after loads still in flight: every lane
// first fences its reads against the async proxy, then the warp converges
// and one lane arrives. Without the fence a warp's last loads of a slot were
// seen returning bytes of the next row copied into it.
__device__ __forceinline__ void release_slot(uint64_t* empty_bar) {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(empty_bar);
}

__device__ __forceinline__ uint4 ld_shared_v4(const void* p) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(smem_u32(p))
               : "memory");
  return v;
}

}  // namespace async
}  // namespace cq

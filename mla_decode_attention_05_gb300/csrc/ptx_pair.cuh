// PTX helpers of the operators around the decode: waits with little code, and
// pairs of CTAs.
#pragma once

#include "ptx.cuh"

namespace mla {
namespace ptx {

// mbar_wait for kernels that are compiled for short limits (kPoll: below
// kShortWaitNs) and for others apart, as a choice at each wait costs one or two
// per cent of a call.  A short limit polls from the start (mbar_wait's first try
// may sleep past a microsecond).
template <bool kCluster, bool kPoll>
__device__ __forceinline__ bool mbar_wait_limited(uint32_t bar, uint32_t parity, volatile int *abort,
                                                  uint64_t limit_ns) {
  if constexpr (kPoll) {
    for (const uint64_t t0 = globaltimer();;) {
      if (kCluster ? mbar_test_wait_cluster(bar, parity) : mbar_test_wait(bar, parity)) return true;
      if (*abort || globaltimer() - t0 > limit_ns) return false;
    }
  } else {
    return mbar_wait<kCluster>(bar, parity, abort, limit_ns < kShortWaitNs ? kShortWaitNs : limit_ns);
  }
}

// mbar_wait with little code, for kernels whose roles share the instruction cache
// among many waits: true once the phase has completed; false, with *abort set,
// after limit_ns (at most 4e9) or when *abort is set already.
template <bool kCluster, bool kPoll>
__device__ __forceinline__ bool mbar_wait_small(uint32_t bar, uint32_t parity, volatile int *abort,
                                                uint32_t limit_ns) {
  uint32_t t0 = 0, it = 0;
  while (!(kPoll ? (kCluster ? mbar_test_wait_cluster(bar, parity) : mbar_test_wait(bar, parity))
                 : (kCluster ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity)))) {
    if (!kPoll && (++it & 15u)) continue;
    uint32_t t;
    asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t));
    if (t0 == 0) {
      t0 = t & ~1u;  // (0: the next look starts)
    } else if (*abort || t - t0 > limit_ns) {
      *abort = 1;
      return false;
    }
  }
  return true;
}

// ---- tcgen05, pairs of CTAs --------------------------------------------------------
//
// The two CTAs of a cluster of two as one MMA: M = 256 rows of D, 128 in the
// tensor memory of each; A's 128 rows and B's half of the N columns come from
// the shared memory of each, at the same offsets.  One thread of rank 0 issues.

__device__ __forceinline__ void tmem_alloc_pair(uint32_t dst_smem, uint32_t ncols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(dst_smem),
               "r"(ncols)
               : "memory");
}

__device__ __forceinline__ void tmem_relinquish_pair() {
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ void tmem_dealloc_pair(uint32_t taddr, uint32_t ncols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(ncols)
               : "memory");
}

__device__ __forceinline__ void mma_pair_ss(uint32_t d, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                            uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// Arrive on the barrier at this offset of both CTAs once all MMAs issued so far complete.
__device__ __forceinline__ void mma_commit_pair(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"((uint16_t)3)
      : "memory");
}

// A tile load into this CTA whose bytes are counted by a barrier of either
// CTA of the pair (cluster address).
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const void *map, uint32_t cluster_bar, int c0, int c1,
                                                 int c2, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(cluster_bar), "l"(policy)
      : "memory");
}

}  // namespace ptx
}  // namespace mla

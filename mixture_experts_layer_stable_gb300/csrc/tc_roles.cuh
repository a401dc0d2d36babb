// tc_roles.cuh -- what the warp-specialised product kernels of the operators (mxfp4.cu,
// product_tc.cuh) share: copies, commits and waits predicated on an elected lane, for
// loops that whole warps run without branches, and the clusters a kernel can have.
#pragma once

#include <atomic>

#include "ops_common.cuh"
#include "ptx.cuh"

namespace moe {

// High word of a shared-memory descriptor: 128-byte swizzle, 1024 bytes between groups
// of 8 rows.
constexpr uint32_t kDescSw128 = (1024 >> 4) | (1u << 14) | (2u << 29);

// The following do nothing in lanes where `on` is 0.
// One arrival on the barrier (of a pair: at this place in each CTA of mask) when what
// was issued so far has completed.
template <bool PAIR>
MOE_DEV void tc_commit_on(int on, uint32_t bar, uint16_t mask = 3) {
  if constexpr (PAIR)
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %2;\n\t}" ::
            "r"(bar),
        "r"(on), "h"(mask)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %1, 0;\n\t"
        "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(bar), "r"(on)
        : "memory");
}
MOE_DEV void expect_tx_on(int on, uint32_t bar, uint32_t bytes) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %2, 0;\n\t"
      "@q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(bar), "r"(bytes), "r"(on)
      : "memory");
}
// (Of a pair: `bar` may be the other CTA's, by its shared::cluster address.)
template <bool PAIR>
MOE_DEV void tma_load_2d_on(int on, uint32_t dst, const CUtensorMap* m, uint32_t bar, int c0, int c1) {
  if constexpr (PAIR) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];\n\t}" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(c0), "r"(c1), "r"(on)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %5, 0;\n\t"
        "@q cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4}], [%2];\n\t}" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(c0), "r"(c1), "r"(on)
        : "memory");
  }
}
template <bool PAIR>
MOE_DEV void tma_load_3d_on(int on, uint32_t dst, const CUtensorMap* m, uint32_t bar, int c0, int c1, int c2) {
  if constexpr (PAIR) {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %6, 0;\n\t"
        "@q cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];\n\t}" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(on)
        : "memory");
  } else {
    asm volatile(
        "{\n\t.reg .pred q;\n\t"
        "setp.ne.b32 q, %6, 0;\n\t"
        "@q cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];\n\t}" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(m)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(on)
        : "memory");
  }
}
MOE_DEV bool try_wait(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// The rest of a wait whose first try failed: gives up (false) on the abort flag
// or after kWaitLimitNs, which it reports.
static __device__ __noinline__ bool wait_on(uint32_t bar, uint32_t parity, volatile int* abort_flag, int* status, int where) {
  const uint64_t t0 = global_timer_ns();
  for (uint32_t it = 1;; ++it) {
    if (try_wait(bar, parity)) return true;
    if ((it & 63u) == 0) {
      if (*abort_flag) return false;
      if (global_timer_ns() - t0 > kWaitLimitNs) {
        *abort_flag = 1;
        report_status(status, kStatusTimeout, where);
        return false;
      }
    }
  }
}
// One lane of a converged warp.
MOE_DEV bool elect_one() {
  uint32_t p;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(p));
  return p != 0;
}
// A value that is the same in every lane, as one the compiler knows to be: a
// warp reduction's result is warp-uniform (a shuffle's is not).
MOE_DEV int uniform(int v) { return (int)__reduce_max_sync(0xffffffffu, (unsigned)v); }

// Clusters of two CTAs of kern that the GPU holds at once.  resident: the answer for
// each device (0: not asked yet), kept by the caller for its kernel; threads that ask
// at the same time store the same value.
template <typename K>
inline int pair_clusters(K kern, const cudaLaunchConfig_t& cfg, std::atomic<int> (&resident)[64]) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) dev = 0;
  int n = resident[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) != cudaSuccess || n < 1) n = num_sms() / 2;
    resident[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}


}  // namespace moe

// cluster.cuh -- data passed between the CTAs of a thread-block cluster:
// asynchronous stores into a peer's shared memory that count their bytes on an
// mbarrier of the peer.  A receiver waits for its own barrier alone, one way
// of the network, where plain remote stores and a cluster barrier take the
// stores' acknowledgements and a barrier round trip.
#pragma once

#include "pgd_device.cuh"

namespace pgd {

// The place in CTA r's shared memory that `local` is in ours.
__device__ __forceinline__ uint32_t peer_addr(const void *local, uint32_t r) {
  uint32_t remote;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
               : "=r"(remote)
               : "r"(smem_addr(local)), "r"(r));
  return remote;
}

// 16 or 8 bytes to CTA r's `local`, counted on CTA r's `bar`.
__device__ __forceinline__ void send16(const void *local, const uint64_t *bar, uint32_t r,
                                       uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile(
      "st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];"
      ::"r"(peer_addr(local, r)), "r"(a), "r"(b), "r"(c), "r"(d), "r"(peer_addr(bar, r))
      : "memory");
}
__device__ __forceinline__ void send8(const void *local, const uint64_t *bar, uint32_t r,
                                      uint32_t a, uint32_t b) {
  asm volatile(
      "st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.b32 [%0], {%1, %2}, [%3];"
      ::"r"(peer_addr(local, r)), "r"(a), "r"(b), "r"(peer_addr(bar, r))
      : "memory");
}

// Wait for a phase of a barrier that peers' stores complete, at most
// kWaitLimitNs (every CTA of the cluster sends before it waits, so the limit
// is never met); the stores are visible behind it.
__device__ __forceinline__ bool wait_for_peers(uint64_t *bar, uint32_t parity) {
  uint64_t t0 = 0;
  for (uint32_t i = 0;; ++i) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(smem_addr(bar)), "r"(parity)
        : "memory");
    if (done) return true;
    if ((i & 31u) == 0) {
      const uint64_t t = global_timer_ns();
      if (t0 == 0) t0 = t;
      if (t - t0 > kWaitLimitNs) return false;
    }
  }
}

// After a wait that gave up: until every thread of the cluster has come here or
// left, so that no peer stores into the memory of a CTA that has gone.
__device__ __forceinline__ void wait_to_leave() {
  asm volatile("barrier.cluster.arrive.relaxed;\n\tbarrier.cluster.wait;" ::: "memory");
}

}  // namespace pgd

// What the kernels of CTA pairs share: products and commits issued by a whole
// warp, barriers across the two CTAs, and waits that end.  The parameters P of
// a kernel have `timeout_ns` and the handle's error word `err`.
#pragma once

#include "common.cuh"
#include "op_common.cuh"

namespace muon {

// Pair products issued by a warp whose lanes stay together (see op_attn.cuh).
__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
  asm volatile(
      "{\n"
      " .reg .pred p, q;\n"
      " elect.sync _|q, 0xffffffff;\n"
      " setp.ne.b32 p, %4, 0;\n"
      " @q tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n"
      "}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void commit_pair(uint64_t* bar, uint16_t cta_mask) {
  asm volatile(
      "{\n"
      " .reg .pred q;\n"
      " elect.sync _|q, 0xffffffff;\n"
      " @q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n"
      "}\n" ::"r"(smem_u32(bar)),
      "h"(cta_mask)
      : "memory");
}

// The leader's product reads what the other CTA's warps wrote to their shared
// memory, so those writes have to be ordered before it across the CTAs.  Their
// fence hands them to the async proxy, a barrier of their own CTA collects
// them, and one warp then sends 16 bytes to the leader, an asynchronous copy
// that completes on the leader's barrier as a release at cluster scope.  (An
// arrival with that release by the writing warps held each for 1900 cycles and
// took 2.4 ms at 16384 x 4096 x 14336, one such arrival by the one warp 2.9;
// an arrival without it, which orders nothing between CTAs, 1.13.)
__device__ __forceinline__ void send_token(uint32_t dst, uint32_t src, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], 16, [%2];" ::"r"(dst),
               "r"(src), "r"(bar)
               : "memory");
}
__device__ __forceinline__ bool try_wait_cluster(uint32_t bar_addr, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n"
      " .reg .pred p;\n"
      " mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n"
      "}\n"
      : "=r"(ok)
      : "r"(bar_addr), "r"(parity)
      : "memory");
  return ok != 0;
}

__device__ __forceinline__ void gave_up(volatile int* abort, unsigned* err) {
  if (*abort == 0) atomicOr(err, ERRBIT_TIMEOUT);
  *abort = 1;
}
// A poll that fails has lasted 4 us, the hardware's own limit, so after each but
// the first the clock and the other warps' giving up are looked at: a wait ends
// within two polls of its limit.  (Looked at after every 32nd, 128 us, a limit below
// 256 us let no wait here end.  16384 x 4096 x 14336 from codes: 1.254 ms that way,
// 1.259 this way, 1.267 with the clock read before the second poll.)
struct WaitClock {
  uint64_t t0 = 0;
  __device__ __forceinline__ bool over(uint64_t limit) {
    const uint64_t now = globaltimer_ns();
    if (t0 == 0) t0 = now;
    return now - t0 > limit;
  }
};
// one thread
template <typename P>
__device__ __forceinline__ bool wait_one(uint64_t* bar, uint32_t parity, volatile int* abort, const P& p) {
  const uint32_t a = smem_u32(bar);
  if (mbar_try_wait(a, parity)) return true;
  WaitClock clock;
  for (;;) {
    if (mbar_try_wait(a, parity)) return true;
    if (*abort != 0 || clock.over(p.timeout_ns)) {
      gave_up(abort, p.err);
      return false;
    }
  }
}
// a warp; SLEEP: nanoseconds between polls where the wait is long and the
// issue slots are better left to the code warps; PAIR: for what the other CTA did
template <int SLEEP = 0, bool PAIR = false, typename P>
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort, const P& p) {
  const uint32_t a = smem_u32(bar);
  auto done = [&]() { return __all_sync(0xffffffffu, PAIR ? try_wait_cluster(a, parity) : mbar_try_wait(a, parity)) != 0; };
  if (done()) return true;
  WaitClock clock;
  for (;;) {
    if (SLEEP > 0) __nanosleep(SLEEP);
    if (done()) return true;
    const bool stop = *abort != 0 || clock.over(p.timeout_ns);
    if (__any_sync(0xffffffffu, stop)) {
      if ((threadIdx.x & 31) == 0) gave_up(abort, p.err);
      return false;
    }
  }
}

}  // namespace muon

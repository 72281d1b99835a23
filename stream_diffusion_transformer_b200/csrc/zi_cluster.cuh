// Waits of whole warps, and reading the shared memory of a cluster's other CTAs.
#pragma once
#include "zi_common.cuh"

namespace zi {

// mbar_wait by all 32 lanes with one answer: a lane that gives up takes its warp along, so that no
// other lane waits for it in a later warp-wide instruction.
ZI_DEV bool mbar_wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort, unsigned int code) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort, code));
}

// Loads from peers are predicated rather than branched around, so that those of all ranks are on
// their way together.

constexpr int kMaxCluster = 8;

// Address of this CTA's shared-memory offset `saddr` in CTA `rank` of the cluster.
ZI_DEV uint32_t peer_addr(uint32_t saddr, int rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(saddr), "r"(rank));
  return a;
}

// The value at a peer's address if `have`, else 0.
ZI_DEV float ld_peer(uint32_t addr, bool have) {
  float x;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.u32 p, %2, 0;\n\t"
      "mov.f32 %0, 0f00000000;\n\t"
      "@p ld.shared::cluster.f32 %0, [%1];\n\t}"
      : "=f"(x)
      : "r"(addr), "r"(uint32_t(have))
      : "memory");
  return x;
}
ZI_DEV float4 ld_peer4(uint32_t addr, bool have) {
  float4 x;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.u32 p, %5, 0;\n\t"
      "mov.f32 %0, 0f00000000;\n\tmov.f32 %1, 0f00000000;\n\tmov.f32 %2, 0f00000000;\n\tmov.f32 %3, 0f00000000;\n\t"
      "@p ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];\n\t}"
      : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w)
      : "r"(addr), "r"(uint32_t(have))
      : "memory");
  return x;
}

// Whether the 32-bit word at this CTA's offset is set in any of the cluster's first `ranks` CTAs.
ZI_DEV bool any_peer_set(const volatile int* word, int ranks) {
  const uint32_t saddr = smem_u32(const_cast<const int*>(word));
  int f = 0;
#pragma unroll
  for (int r = 0; r < kMaxCluster; ++r) f |= __float_as_int(ld_peer(peer_addr(saddr, r < ranks ? r : 0), r < ranks));
  return f != 0;
}

}  // namespace zi

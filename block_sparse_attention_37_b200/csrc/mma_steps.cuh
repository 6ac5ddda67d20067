// What the tcgen05 attention kernels share beyond common.cuh: the register
// split, named barriers, and the k-step loops of the two products.
#pragma once

#include <utility>

#include "common.cuh"

namespace bsa {

template <int N>
__device__ __forceinline__ void regs_release() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_claim() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

__device__ __forceinline__ void named_bar(int id, int n) {
  asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory");
}

// S = Q K^T over D/16 k-steps of 16 (K-major SW128 operands: k-step kk sits
// in 64-column chunk kk/4 (16 KB apart) at byte offset 32*(kk%4)).
template <int KK>
__device__ __forceinline__ void qk_step(uint32_t s_tmem, uint64_t qd, uint64_t kd, uint32_t idesc) {
  constexpr uint32_t off = ((KK >> 2) * 16384 + (KK & 3) * 32) >> 4;
  umma_ss_at_warp<off, off>(s_tmem, qd, kd, idesc, KK > 0 ? 1u : 0u);
}
template <int... KK>
__device__ __forceinline__ void qk_all(uint32_t s_tmem, uint64_t qd, uint64_t kd, uint32_t idesc,
                                       std::integer_sequence<int, KK...>) {
  (qk_step<KK>(s_tmem, qd, kd, idesc), ...);
}

// O (+)= P V over 8 k-steps of 16 keys: P from tensor memory (8 columns per
// step), V MN-major SW128 (16 rows = 2048 bytes per step).
template <int KK>
__device__ __forceinline__ void pv_step(uint32_t o_tmem, uint32_t p_tmem, uint64_t vd, uint32_t idesc, uint32_t first) {
  constexpr uint32_t voff = KK * 2048 / 16;
  umma_ts_at_warp<KK * 8, voff>(o_tmem, p_tmem, vd, idesc, (KK > 0 || !first) ? 1u : 0u);
}
template <int... KK>
__device__ __forceinline__ void pv_all(uint32_t o_tmem, uint32_t p_tmem, uint64_t vd, uint32_t idesc, uint32_t first,
                                       std::integer_sequence<int, KK...>) {
  (pv_step<KK>(o_tmem, p_tmem, vd, idesc, first), ...);
}

}  // namespace bsa

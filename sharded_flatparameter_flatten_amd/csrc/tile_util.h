// What the kernels of tiled products share: constants for unrolled loops, waits, tile order.
#pragma once

#include <type_traits>
#include <utility>

#include "device_util.h"

#pragma clang fp contract(off)

namespace fsdp {
namespace dev {

typedef float f32x16 __attribute__((ext_vector_type(16)));

// t / d for 0 <= t < 2^24, 0 < d and quotients below 2^20 (the estimate is then off by at most one): a few instructions, where a division takes 40 that wait for each other.
__device__ __forceinline__ int divide(int t, int d) {
  int q = int(float(t) * __builtin_amdgcn_rcpf(float(d)));
  q -= q * d > t;
  q += (q + 1) * d <= t;
  return __builtin_amdgcn_readfirstlane(q);
}
// Tile t of a ti x tj grid, walked in bands of 8 tile rows.
__device__ __forceinline__ void tile_of(int t, int ti, int tj, int& i, int& j) {
  const int r0 = divide(t, 8 * tj) * 8, h = ti - r0 < 8 ? ti - r0 : 8, in = t - r0 * tj;
  j = divide(in, h);
  i = r0 + in - j * h;
}

// At most N global loads of this wave are still under way, and no LDS read.
template <int N>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
}
__device__ __forceinline__ void meet() {
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// f(0), ..., f(N - 1) with constants, whatever the compiler's limits on unrolling.
template <int N, typename F, int... I>
__device__ __forceinline__ void static_for_each(F&& f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void static_for(F&& f) {
  static_for_each<N>(f, std::make_integer_sequence<int, N>{});
}

}  // namespace dev
}  // namespace fsdp

// Device and host helpers of the HIP files beside kernels.hip: element
// conversions, wide loads and stores, reductions, launch checks.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <vector>

#include "fsdp_internal.h"

#pragma clang fp contract(off)

namespace fsdp {
namespace dev {

typedef unsigned int u32x2 __attribute__((ext_vector_type(2)));
typedef unsigned int u32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4 __attribute__((ext_vector_type(4)));

// bf16 -> fp32 is exact: the bf16 bits are the high half of the fp32 bits.
__device__ __forceinline__ float lo_bf16(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_bf16(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ float widen(uint16_t h) { return __uint_as_float(uint32_t(h) << 16); }

// fp32 -> bf16, nearest, ties to even; NaN -> 0x7FC0 (the rounding of the step
// kernels: 0x7FFF plus the lowest kept bit carries exactly when it should).
__device__ __forceinline__ uint32_t to_bf16(float f) {
  const uint32_t x = __float_as_uint(f);
  if ((x & 0x7FFFFFFFu) > 0x7F800000u) return 0x7FC0u;
  return (x + 0x7FFFu + ((x >> 16) & 1u)) >> 16;
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return to_bf16(a) | (to_bf16(b) << 16);
}

// Wide accesses at element alignment: on gfx950 a global access of any width
// may start at any byte, so rows and windows that start off a 16-byte boundary
// take the same instructions (they only touch one more line).
template <typename V, int ALIGN>
struct __attribute__((packed, aligned(ALIGN))) Loose {
  V v;
};
template <typename V, int ALIGN>
__device__ __forceinline__ V ld_loose(const void* p) {
  return static_cast<const Loose<V, ALIGN>*>(p)->v;
}
template <typename V, int ALIGN>
__device__ __forceinline__ void st_loose(void* p, V x) {
  static_cast<Loose<V, ALIGN>*>(p)->v = x;
}

// Buffer descriptor over [base, base + bytes) (gfx9 raw-buffer format word);
// loads past it return zeros and stores past it are dropped.
constexpr int kRsrcWord3 = 0x00020000;
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rsrc(const void* base, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0,
                                           static_cast<int>(bytes), kRsrcWord3);
}
// A streaming store (device scope, not kept in L2: sc1 nt), for outputs far
// larger than L2: their write-back then ends within the kernel instead of
// slowing the next. Aligned to its size.
constexpr int kStoreStream = 18;
__device__ __forceinline__ void st_stream(__amdgpu_buffer_rsrc_t r, int off, u32x4 x) {
  __builtin_amdgcn_raw_buffer_store_b128(x, r, off, 0, kStoreStream);
}
__device__ __forceinline__ void st_stream(__amdgpu_buffer_rsrc_t r, int off, u32x2 x) {
  __builtin_amdgcn_raw_buffer_store_b64(x, r, off, 0, kStoreStream);
}
__device__ __forceinline__ void st_stream(__amdgpu_buffer_rsrc_t r, int off, uint32_t x) {
  __builtin_amdgcn_raw_buffer_store_b32(x, r, off, 0, kStoreStream);
}

template <typename T>
__device__ __forceinline__ T wave_sum(T x) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) x += __shfl_xor(x, d);
  return x;
}

}  // namespace dev

inline fsdp_status after_launch(const char* what) {
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess)
    return fail(FSDP_ERR_HIP, "%s: launch failed: %s", what, hipGetErrorString(e));
  return FSDP_OK;
}

// An error left pending by earlier work is left for its owner; nothing is enqueued.
inline fsdp_status check_no_pending_error(const char* what) {
  const hipError_t e = hipPeekAtLastError();
  if (e != hipSuccess)
    return fail(FSDP_ERR_HIP, "%s: a HIP error from earlier work is pending (%s); nothing was "
                "enqueued", what, hipGetErrorString(e));
  return FSDP_OK;
}

inline fsdp_status check_ptr(const void* p, const char* name, int align) {
  if (!p) return fail(FSDP_ERR_INVALID_ARG, "%s is NULL", name);
  if (reinterpret_cast<uintptr_t>(p) % static_cast<uintptr_t>(align))
    return fail(FSDP_ERR_INVALID_ARG, "%s is not %d-byte aligned", name, align);
  return FSDP_OK;
}

}  // namespace fsdp

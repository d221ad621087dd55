// Rows of bf16 or fp32 elements in groups of 8 columns, and the checks of row arguments:
// what the embedding, the dropout and the head's loss share.
#pragma once

#include <new>

#include "device_util.h"

#pragma clang fp contract(off)

namespace fsdp {
namespace dev {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// Two fp32 values to bf16 (nearest, ties to even) in one instruction: the bits of to_bf16
// for every value that is not NaN.
__device__ __forceinline__ uint32_t round_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
}

// Columns c to c + 7 of a row as they lie in memory, from element alignment; elements at or
// past `dim` are zeros.
template <typename T>
struct Group {
  u32x4 v[sizeof(T) / 2];
};
__device__ __forceinline__ Group<uint16_t> load_group(const uint16_t* p, int64_t c, int64_t dim) {
  if (c + 8 <= dim) return {{ld_loose<u32x4, 2>(p + c)}};
  Group<uint16_t> r{};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (c + e < dim) r.v[0][e / 2] |= uint32_t(p[c + e]) << (16 * (e & 1));
  return r;
}
__device__ __forceinline__ Group<float> load_group(const float* p, int64_t c, int64_t dim) {
  if (c + 8 <= dim) return {{ld_loose<u32x4, 4>(p + c), ld_loose<u32x4, 4>(p + c + 4)}};
  Group<float> r{};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (c + e < dim) r.v[e / 4][e % 4] = __float_as_uint(p[c + e]);
  return r;
}
__device__ __forceinline__ void unpack(const Group<uint16_t>& r, float (&x)[8]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) { x[2 * e] = lo_bf16(r.v[0][e]); x[2 * e + 1] = hi_bf16(r.v[0][e]); }
}
__device__ __forceinline__ void unpack(const Group<float>& r, float (&x)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) x[e] = __uint_as_float(r.v[e / 4][e % 4]);
}

// 8 values to columns c to c + 7, each rounded once; elements at or past `dim` are left alone.
// Every NaN of a bf16 row is 0x7FC0.
__device__ __forceinline__ void store_group(uint16_t* p, int64_t c, int64_t dim, const float (&x)[8]) {
  if (c + 8 <= dim) {
    bool nan = false;
    u32x4 q;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      nan |= __builtin_isunordered(x[2 * e], x[2 * e + 1]);
      q[e] = round_bf16(x[2 * e], x[2 * e + 1]);
    }
    if (__builtin_expect(__builtin_amdgcn_ballot_w64(nan) != 0, 0)) {
#pragma unroll
      for (int e = 0; e < 4; ++e) q[e] = pack_bf16(x[2 * e], x[2 * e + 1]);
    }
    st_loose<u32x4, 2>(p + c, q);
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (c + e < dim) p[c + e] = uint16_t(to_bf16(x[e]));
}
__device__ __forceinline__ void store_group(float* p, int64_t c, int64_t dim, const float (&x)[8]) {
  if (c + 8 <= dim) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
      st_loose<f32x4, 4>(p + c + 4 * h, f32x4{x[4 * h], x[4 * h + 1], x[4 * h + 2], x[4 * h + 3]});
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (c + e < dim) p[c + e] = x[e];
}

}  // namespace dev

// Lanes that share a row of `dim` elements in a workgroup of 256, a power of 2: as many as the
// row has groups of 8, so that short rows share a wave.
inline int lanes_of_row(int64_t dim) {
  int lanes = 1;
  while (lanes < 256 && int64_t(lanes) * 8 < dim) lanes *= 2;
  return lanes;
}

// A rows x dim argument with a row pitch: checked, its byte range recorded.
inline fsdp_status check_row_arg(const void* p, int64_t ld, int64_t rows, int64_t dim, int elem, bool write,
                                 const char* name, std::vector<ByteRange>* ranges) {
  if (fsdp_status st = check_ptr(p, name, elem)) return st;
  if (ld < dim || ld > (int64_t(1) << 32))
    return fail(FSDP_ERR_RANGE, "%s: row pitch %lld outside [dim, 2^32]", name, static_cast<long long>(ld));
  ranges->push_back(range_of(p, (rows - 1) * ld + dim, elem, write, name));
  return FSDP_OK;
}

inline fsdp_status check_row_sizes(int64_t rows, int64_t dim) {
  if (rows < 0 || rows >= (int64_t(1) << 22))
    return fail(FSDP_ERR_RANGE, "rows must be in [0, 2^22) (got %lld)", static_cast<long long>(rows));
  if (dim < 1 || dim > (int64_t(1) << 24))
    return fail(FSDP_ERR_RANGE, "dim must be in [1, 2^24] (got %lld)", static_cast<long long>(dim));
  return FSDP_OK;
}

inline fsdp_status check_row_type(fsdp_dtype dtype) {
  if (dtype != FSDP_F32 && dtype != FSDP_BF16)
    return fail(FSDP_ERR_UNSUPPORTED, "dtype %d not supported", static_cast<int>(dtype));
  return FSDP_OK;
}

inline fsdp_status check_workspace(const void* p, int64_t have, int64_t need, int align,
                                   std::vector<ByteRange>* ranges) {
  if (need == 0) return FSDP_OK;
  if (fsdp_status st = check_ptr(p, "workspace", align)) return st;
  if (have < need)
    return fail(FSDP_ERR_RANGE, "workspace has %lld bytes, needs %lld", static_cast<long long>(have),
                static_cast<long long>(need));
  ranges->push_back(range_of(p, need, 1, true, "workspace"));
  return FSDP_OK;
}

}  // namespace fsdp

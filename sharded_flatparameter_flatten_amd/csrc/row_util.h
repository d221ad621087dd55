// Rows of bf16 or fp32 elements in pieces of 16 bytes, and the checks of row arguments:
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

// 16 bytes of a row, kElems<T> consecutive elements: what a lane holds. (With 32 bytes of fp32 a
// lane the stores that stream past L2 would write half sectors.)
template <typename T>
constexpr int kElems = 16 / int(sizeof(T));

// From element alignment; elements at or past `dim` are zeros.
__device__ __forceinline__ u32x4 load_piece(const uint16_t* p, int64_t c, int64_t dim) {
  if (c + 8 <= dim) return ld_loose<u32x4, 2>(p + c);
  u32x4 r{};
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (c + e < dim) r[e / 2] |= uint32_t(p[c + e]) << (16 * (e & 1));
  return r;
}
__device__ __forceinline__ u32x4 load_piece(const float* p, int64_t c, int64_t dim) {
  if (c + 4 <= dim) return ld_loose<u32x4, 4>(p + c);
  u32x4 r{};
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (c + e < dim) r[e] = __float_as_uint(p[c + e]);
  return r;
}
__device__ __forceinline__ void unpack(u32x4 r, float (&x)[8]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) { x[2 * e] = lo_bf16(r[e]); x[2 * e + 1] = hi_bf16(r[e]); }
}
__device__ __forceinline__ void unpack(u32x4 r, float (&x)[4]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) x[e] = __uint_as_float(r[e]);
}

// STREAM: past L2, for a row that the whole wave is in, aligned to 16 bytes.
template <bool STREAM, typename T>
__device__ __forceinline__ void store_16(T* p, int64_t c, int64_t dim, u32x4 q) {
  if constexpr (STREAM) st_stream(rsrc(p, dim * int(sizeof(T))), int(c) * int(sizeof(T)), q);
  else st_loose<u32x4, sizeof(T)>(p + c, q);
}
// Values to the columns from c on, each rounded once; elements at or past `dim` are left alone.
// Every NaN of a bf16 row is 0x7FC0.
template <bool STREAM = false>
__device__ __forceinline__ void store_piece(uint16_t* p, int64_t c, int64_t dim, const float (&x)[8]) {
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
    store_16<STREAM>(p, c, dim, q);
    return;
  }
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (c + e < dim) p[c + e] = uint16_t(to_bf16(x[e]));
}
template <bool STREAM = false>
__device__ __forceinline__ void store_piece(float* p, int64_t c, int64_t dim, const float (&x)[4]) {
  if (c + 4 <= dim) {
    store_16<STREAM>(p, c, dim, u32x4{__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3])});
    return;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (c + e < dim) p[c + e] = x[e];
}

}  // namespace dev

// Lanes that share a row of `pieces` pieces in a workgroup of 256, a power of 2: as many as the
// row has pieces, so that short rows share a wave.
inline int lanes_of_row(int64_t pieces) {
  int lanes = 1;
  while (lanes < 256 && lanes < pieces) lanes *= 2;
  return lanes;
}

// Whether `rows` rows of output are streamed past L2: they are far larger than it, rows take
// whole waves, and every piece is aligned.
constexpr int64_t kStreamBytes = int64_t(32) << 20;
inline bool streams(const void* out, int64_t ld, int64_t rows, int64_t dim, int elem, int lanes) {
  return rows * dim * elem >= kStreamBytes && lanes >= 64 && reinterpret_cast<uintptr_t>(out) % 16 == 0 &&
         ld * elem % 16 == 0 && dim * elem < (int64_t(1) << 31);
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

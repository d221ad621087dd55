// Root-mean-square norm of rows on gfx950, its gradients, and their entry points.
//
// Forward, for a row h of `dim` elements (h = x, or x + residual rounded to
// x's type, which is also written):
//   rstd = 1 / sqrt(mean(h^2) + eps),  y = h * rstd * weight,
// and y in x's type, or in e4m3 as y / scale with scale = max|y| / 448.
// Backward, with xhat = x * rstd and g = dy * weight:
//   dx = rstd * (g - xhat * mean(g * xhat)) [+ dresidual],  dweight = sum over rows of dy * xhat.
// All arithmetic is fp32 (no fused multiply-add), each output rounded once.
//
// Both directions are bound by HBM: a row is read once into registers, its
// statistic is joined across the workgroup, and the outputs are written from
// the registers. Backward runs a fixed number of workgroups over the rows, so
// that each lane keeps the weight gradient of its columns in registers; the
// workgroups' sums are joined in a fixed order by a second kernel (no atomics:
// the same inputs give the same bits).

#include <algorithm>
#include <cmath>
#include <new>
#include <type_traits>

#include "device_util.h"

#pragma clang fp contract(off)

using fsdp::fail;
using namespace fsdp::dev;

namespace {

constexpr float kE4m3Max = 448.f;
constexpr float kMinScale = 1.1754943508222875e-38f;   // 2^-126: a row of zeros divides by this
constexpr int kMaxBlocks = 512;        // workgroups of a backward launch, at most
constexpr int64_t kRegDim = 32768;     // rows up to this length are held in registers

__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const uint16_t* p) { return widen(*p); }
__device__ __forceinline__ void store1(float* p, float x) { *p = x; }
__device__ __forceinline__ void store1(uint16_t* p, float x) { *p = uint16_t(to_bf16(x)); }

// 8 consecutive elements at column c of a row, from element alignment; the
// elements at or past `dim` are zeros (loads) or left alone (stores).
__device__ __forceinline__ void load8(const float* p, int64_t c, int64_t dim, float (&x)[8]) {
  if (c + 8 <= dim) {
    const f32x4 a = ld_loose<f32x4, 4>(p + c), b = ld_loose<f32x4, 4>(p + c + 4);
#pragma unroll
    for (int e = 0; e < 4; ++e) { x[e] = a[e]; x[4 + e] = b[e]; }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = c + e < dim ? p[c + e] : 0.f;
  }
}
__device__ __forceinline__ void load8(const uint16_t* p, int64_t c, int64_t dim, float (&x)[8]) {
  if (c + 8 <= dim) {
    const u32x4 q = ld_loose<u32x4, 2>(p + c);
#pragma unroll
    for (int e = 0; e < 4; ++e) { x[2 * e] = lo_bf16(q[e]); x[2 * e + 1] = hi_bf16(q[e]); }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = c + e < dim ? widen(p[c + e]) : 0.f;
  }
}
__device__ __forceinline__ void store8(float* p, int64_t c, int64_t dim, const float (&x)[8]) {
  if (c + 8 <= dim) {
    st_loose<f32x4, 4>(p + c, f32x4{x[0], x[1], x[2], x[3]});
    st_loose<f32x4, 4>(p + c + 4, f32x4{x[4], x[5], x[6], x[7]});
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c + e < dim) p[c + e] = x[e];
  }
}
__device__ __forceinline__ void store8(uint16_t* p, int64_t c, int64_t dim, const float (&x)[8]) {
  if (c + 8 <= dim) {
    st_loose<u32x4, 2>(p + c, u32x4{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]),
                                    pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7])});
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c + e < dim) store1(p + c + e, x[e]);
  }
}
// 8 values in e4m3 (nearest, ties to even; the caller clamped them).
__device__ __forceinline__ void store8_e4m3(uint8_t* p, int64_t c, int64_t dim, const float (&x)[8]) {
  int a = __builtin_amdgcn_cvt_pk_fp8_f32(x[0], x[1], 0, false);
  a = __builtin_amdgcn_cvt_pk_fp8_f32(x[2], x[3], a, true);
  int b = __builtin_amdgcn_cvt_pk_fp8_f32(x[4], x[5], 0, false);
  b = __builtin_amdgcn_cvt_pk_fp8_f32(x[6], x[7], b, true);
  if (c + 8 <= dim) {
    st_loose<u32x2, 1>(p + c, u32x2{uint32_t(a), uint32_t(b)});
  } else {
    const uint64_t q = uint32_t(a) | (uint64_t(uint32_t(b)) << 32);
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c + e < dim) p[c + e] = uint8_t(q >> (8 * e));
  }
}

__device__ __forceinline__ float round_to(float x, const float*) { return x; }
__device__ __forceinline__ float round_to(float x, const uint16_t*) { return __uint_as_float(to_bf16(x) << 16); }

// The sum (and the largest bit pattern) over a workgroup, the same in every lane.
template <int WAVES>
__device__ __forceinline__ float block_sum(float v, float* lds) {
  v = wave_sum(v);
  if constexpr (WAVES == 1) return v;
  __syncthreads();                      // lds may still be read by an earlier call
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = lds[0];
#pragma unroll
  for (int w = 1; w < WAVES; ++w) s += lds[w];
  return s;
}
template <int WAVES>
__device__ __forceinline__ uint32_t block_max(uint32_t v, float* lds) {
  v = wave_max(v);
  if constexpr (WAVES == 1) return v;
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = __uint_as_float(v);
  __syncthreads();
  uint32_t s = 0;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) s = max(s, __float_as_uint(lds[w]));
  return s;
}

template <typename T>
struct NormArgs {
  const T* x;
  const T* res;        // or null
  const T* w;
  T* sum;              // x + residual, or null
  void* out;           // T or e4m3
  float* rstd;         // or null
  float* scales;       // set when out is e4m3
  int64_t dim, x_ld, res_ld, sum_ld, out_ld;
  float eps;
};

__device__ __forceinline__ float rstd_of(float sum_sq, int64_t dim, float eps) {
  return 1.f / sqrtf(sum_sq / float(dim) + eps);
}
// The bits of |y| order like its value and put NaN above infinity, so a NaN
// anywhere in the row makes the scale NaN.
__device__ __forceinline__ uint32_t abs_bits(float y) { return __float_as_uint(y) & 0x7FFFFFFFu; }
__device__ __forceinline__ float scale_of(uint32_t top) {
  const float s = __uint_as_float(top) / kE4m3Max;
  return s < kMinScale ? kMinScale : s;         // NaN stays NaN
}
__device__ __forceinline__ float clamp_e4m3(float q) {
  return q > kE4m3Max ? kE4m3Max : q < -kE4m3Max ? -kE4m3Max : q;
}

// One row a workgroup, held in registers: lane t's chunk c is elements
// (c * threads + t) * 8 onward.
template <typename T, bool RES, bool BITS8, int WAVES, int CH>
__global__ __launch_bounds__(64 * WAVES) void k_norm(NormArgs<T> a) {
  __shared__ float lds[WAVES];
  const int64_t row = blockIdx.x, dim = a.dim;
  const T* x = a.x + row * a.x_ld;
  float h[CH][8];
  float sq = 0.f;
#pragma unroll
  for (int k = 0; k < CH; ++k) load8(x, (int64_t(k) * 64 * WAVES + threadIdx.x) * 8, dim, h[k]);
  if constexpr (RES) {
    const T* r = a.res + row * a.res_ld;
    T* s = a.sum + row * a.sum_ld;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int64_t c = (int64_t(k) * 64 * WAVES + threadIdx.x) * 8;
      float y[8];
      load8(r, c, dim, y);
#pragma unroll
      for (int e = 0; e < 8; ++e) h[k][e] = round_to(h[k][e] + y[e], s);
      store8(s, c, dim, h[k]);
    }
  }
#pragma unroll
  for (int k = 0; k < CH; ++k)
#pragma unroll
    for (int e = 0; e < 8; ++e) sq += h[k][e] * h[k][e];
  const float rstd = rstd_of(block_sum<WAVES>(sq, lds), dim, a.eps);
  if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
  uint32_t top = 0;
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    const int64_t c = (int64_t(k) * 64 * WAVES + threadIdx.x) * 8;
    float w[8];
    load8(a.w, c, dim, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      h[k][e] = h[k][e] * rstd * w[e];
      if (BITS8 && c + e < dim) top = max(top, abs_bits(h[k][e]));   // past dim: 0 * rstd may be NaN
    }
    if constexpr (!BITS8) store8(static_cast<T*>(a.out) + row * a.out_ld, c, dim, h[k]);
  }
  if constexpr (BITS8) {
    const float scale = scale_of(block_max<WAVES>(top, lds));
    if (threadIdx.x == 0) a.scales[row] = scale;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int64_t c = (int64_t(k) * 64 * WAVES + threadIdx.x) * 8;
#pragma unroll
      for (int e = 0; e < 8; ++e) h[k][e] = clamp_e4m3(h[k][e] / scale);
      store8_e4m3(static_cast<uint8_t*>(a.out) + row * a.out_ld, c, dim, h[k]);
    }
  }
}

// Rows too long for registers: the row is read again for each pass.
constexpr int kLongWaves = 16;
template <typename T, bool RES, bool BITS8>
__global__ __launch_bounds__(64 * kLongWaves) void k_norm_long(NormArgs<T> a) {
  __shared__ float lds[kLongWaves];
  const int64_t row = blockIdx.x, dim = a.dim, step = 64 * kLongWaves * 8;
  const T* x = a.x + row * a.x_ld;
  const T* r = RES ? a.res + row * a.res_ld : nullptr;
  auto get = [&](int64_t c, float (&h)[8]) {
    load8(x, c, dim, h);
    if constexpr (RES) {
      float y[8];
      load8(r, c, dim, y);
#pragma unroll
      for (int e = 0; e < 8; ++e) h[e] = round_to(h[e] + y[e], x);
    }
  };
  float sq = 0.f;
  for (int64_t c = int64_t(threadIdx.x) * 8; c < dim; c += step) {
    float h[8];
    get(c, h);
#pragma unroll
    for (int e = 0; e < 8; ++e) sq += h[e] * h[e];
    if constexpr (RES) store8(a.sum + row * a.sum_ld, c, dim, h);
  }
  const float rstd = rstd_of(block_sum<kLongWaves>(sq, lds), dim, a.eps);
  if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
  float scale = 1.f;
  if constexpr (BITS8) {
    uint32_t top = 0;
    for (int64_t c = int64_t(threadIdx.x) * 8; c < dim; c += step) {
      float h[8], w[8];
      get(c, h);
      load8(a.w, c, dim, w);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (c + e < dim) top = max(top, abs_bits(h[e] * rstd * w[e]));
    }
    scale = scale_of(block_max<kLongWaves>(top, lds));
    if (threadIdx.x == 0) a.scales[row] = scale;
  }
  for (int64_t c = int64_t(threadIdx.x) * 8; c < dim; c += step) {
    float h[8], w[8];
    get(c, h);
    load8(a.w, c, dim, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      h[e] = h[e] * rstd * w[e];
      if constexpr (BITS8) h[e] = clamp_e4m3(h[e] / scale);
    }
    if constexpr (BITS8) store8_e4m3(static_cast<uint8_t*>(a.out) + row * a.out_ld, c, dim, h);
    else store8(static_cast<T*>(a.out) + row * a.out_ld, c, dim, h);
  }
}

// ---------------------------------------------------------------------------
// backward
// ---------------------------------------------------------------------------

template <typename T>
struct NormBackArgs {
  const T* dy;
  const T* x;
  const T* w;
  const float* rstd;
  const T* dres;        // or null
  T* dx;
  float* partial;       // [gridDim.x][dim] sums for dweight, or null
  int64_t rows, dim, dy_ld, x_ld, dres_ld, dx_ld;
};

// Rows b, b + gridDim.x, ... of workgroup b; lane columns as in k_norm.
template <typename T, bool RES, int WAVES, int CH>
__global__ __launch_bounds__(64 * WAVES) void k_norm_back(NormBackArgs<T> a) {
  __shared__ float lds[WAVES];
  const int64_t dim = a.dim;
  float w[CH][8], dw[CH][8];
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    load8(a.w, (int64_t(k) * 64 * WAVES + threadIdx.x) * 8, dim, w[k]);
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[k][e] = 0.f;
  }
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* x = a.x + row * a.x_ld;
    const T* dy = a.dy + row * a.dy_ld;
    const float rstd = a.rstd[row];
    float h[CH][8], g[CH][8];
    float dot = 0.f;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int64_t c = (int64_t(k) * 64 * WAVES + threadIdx.x) * 8;
      load8(x, c, dim, h[k]);
      load8(dy, c, dim, g[k]);
    }
#pragma unroll
    for (int k = 0; k < CH; ++k)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        h[k][e] = h[k][e] * rstd;
        dw[k][e] += g[k][e] * h[k][e];
        g[k][e] = g[k][e] * w[k][e];
        if ((int64_t(k) * 64 * WAVES + threadIdx.x) * 8 + e < dim) dot += g[k][e] * h[k][e];
      }
    const float mean = block_sum<WAVES>(dot, lds) / float(dim);
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      const int64_t c = (int64_t(k) * 64 * WAVES + threadIdx.x) * 8;
#pragma unroll
      for (int e = 0; e < 8; ++e) h[k][e] = rstd * (g[k][e] - h[k][e] * mean);
      if constexpr (RES) {
        float y[8];
        load8(a.dres + row * a.dres_ld, c, dim, y);
#pragma unroll
        for (int e = 0; e < 8; ++e) h[k][e] += y[e];
      }
      store8(a.dx + row * a.dx_ld, c, dim, h[k]);
    }
  }
  if (a.partial) {
#pragma unroll
    for (int k = 0; k < CH; ++k)
      store8(a.partial + blockIdx.x * dim, (int64_t(k) * 64 * WAVES + threadIdx.x) * 8, dim, dw[k]);
  }
}

// Rows too long for registers: dx here, the weight's sums in k_norm_back_cols.
template <typename T, bool RES>
__global__ __launch_bounds__(64 * kLongWaves) void k_norm_back_long(NormBackArgs<T> a) {
  __shared__ float lds[kLongWaves];
  const int64_t dim = a.dim, step = 64 * kLongWaves * 8;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* x = a.x + row * a.x_ld;
    const T* dy = a.dy + row * a.dy_ld;
    const float rstd = a.rstd[row];
    float dot = 0.f;
    for (int64_t c = int64_t(threadIdx.x) * 8; c < dim; c += step) {
      float h[8], g[8], w[8];
      load8(x, c, dim, h);
      load8(dy, c, dim, g);
      load8(a.w, c, dim, w);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (c + e < dim) dot += g[e] * w[e] * (h[e] * rstd);
    }
    const float mean = block_sum<kLongWaves>(dot, lds) / float(dim);
    for (int64_t c = int64_t(threadIdx.x) * 8; c < dim; c += step) {
      float h[8], g[8], w[8];
      load8(x, c, dim, h);
      load8(dy, c, dim, g);
      load8(a.w, c, dim, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) h[e] = rstd * (g[e] * w[e] - h[e] * rstd * mean);
      if constexpr (RES) {
        float y[8];
        load8(a.dres + row * a.dres_ld, c, dim, y);
#pragma unroll
        for (int e = 0; e < 8; ++e) h[e] += y[e];
      }
      store8(a.dx + row * a.dx_ld, c, dim, h);
    }
  }
}
// The weight's sums of rows blockIdx.y, blockIdx.y + gridDim.y, ... for 2048 columns.
template <typename T>
__global__ __launch_bounds__(256) void k_norm_back_cols(NormBackArgs<T> a) {
  const int64_t c = (int64_t(blockIdx.x) * 256 + threadIdx.x) * 8;
  if (c >= a.dim) return;
  float dw[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
    float h[8], g[8];
    load8(a.x + row * a.x_ld, c, a.dim, h);
    load8(a.dy + row * a.dy_ld, c, a.dim, g);
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[e] += g[e] * (h[e] * a.rstd[row]);
  }
  store8(a.partial + int64_t(blockIdx.y) * a.dim, c, a.dim, dw);
}

// dweight[c] = the sum over the workgroups' partial rows, in a fixed order: 16
// waves take every 16th row each for 64 columns, then join in wave order.
template <typename T>
__global__ __launch_bounds__(1024) void k_norm_dweight(const float* partial, int32_t parts,
                                                       int64_t dim, T* dweight) {
  __shared__ float lds[16][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t c = int64_t(blockIdx.x) * 64 + lane;
  float s = 0.f;
  if (c < dim)
    for (int r = wave; r < parts; r += 16) s += partial[int64_t(r) * dim + c];
  lds[wave][lane] = s;
  __syncthreads();
  if (wave == 0 && c < dim) {
    for (int w = 1; w < 16; ++w) s += lds[w][lane];
    store1(dweight + c, s);
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

int32_t back_blocks(int64_t rows) { return int32_t(std::min<int64_t>(rows, kMaxBlocks)); }

// The row's shape: waves a workgroup and chunks of 8 elements a lane.
template <typename F>
void with_shape(int64_t dim, F&& f) {
  using std::integral_constant;
  if (dim <= 512) f(integral_constant<int, 1>{}, integral_constant<int, 1>{});
  else if (dim <= 1024) f(integral_constant<int, 1>{}, integral_constant<int, 2>{});
  else if (dim <= 2048) f(integral_constant<int, 4>{}, integral_constant<int, 1>{});
  else if (dim <= 4096) f(integral_constant<int, 4>{}, integral_constant<int, 2>{});
  else if (dim <= 8192) f(integral_constant<int, 16>{}, integral_constant<int, 1>{});
  else if (dim <= 16384) f(integral_constant<int, 16>{}, integral_constant<int, 2>{});
  else f(integral_constant<int, 16>{}, integral_constant<int, 4>{});
}

template <typename T, bool RES, bool BITS8>
void launch_norm(const NormArgs<T>& a, int64_t rows, hipStream_t stream) {
  if (a.dim > kRegDim) {
    k_norm_long<T, RES, BITS8><<<unsigned(rows), 64 * kLongWaves, 0, stream>>>(a);
    return;
  }
  with_shape(a.dim, [&](auto waves, auto ch) {
    k_norm<T, RES, BITS8, waves.value, ch.value><<<unsigned(rows), 64 * waves.value, 0, stream>>>(a);
  });
}

template <typename T, bool RES>
void launch_back(const NormBackArgs<T>& a, hipStream_t stream) {
  const int32_t blocks = back_blocks(a.rows);
  if (a.dim > kRegDim) {
    k_norm_back_long<T, RES><<<blocks, 64 * kLongWaves, 0, stream>>>(a);
    if (a.partial)
      k_norm_back_cols<T><<<dim3(unsigned((a.dim + 2047) / 2048), blocks), 256, 0, stream>>>(a);
    return;
  }
  with_shape(a.dim, [&](auto waves, auto ch) {
    k_norm_back<T, RES, waves.value, ch.value><<<blocks, 64 * waves.value, 0, stream>>>(a);
  });
}

fsdp_status check_sizes(int64_t rows, int64_t dim) {
  if (rows < 0 || rows >= (int64_t(1) << 22))
    return fail(FSDP_ERR_RANGE, "rows must be in [0, 2^22) (got %lld)", static_cast<long long>(rows));
  if (dim < 1 || dim > (int64_t(1) << 24))
    return fail(FSDP_ERR_RANGE, "dim must be in [1, 2^24] (got %lld)", static_cast<long long>(dim));
  return FSDP_OK;
}

// A rows x dim argument with a row pitch: checked, its byte range recorded.
fsdp_status check_rows(const void* p, int64_t ld, int64_t rows, int64_t dim, int elem, bool write,
                       const char* name, std::vector<fsdp::ByteRange>* ranges) {
  if (fsdp_status st = fsdp::check_ptr(p, name, elem)) return st;
  if (ld < dim || ld > (int64_t(1) << 32))
    return fail(FSDP_ERR_RANGE, "%s: row pitch %lld outside [dim, 2^32]", name,
                static_cast<long long>(ld));
  ranges->push_back(fsdp::range_of(p, (rows - 1) * ld + dim, elem, write, name));
  return FSDP_OK;
}

fsdp_status check_type(fsdp_dtype dtype) {
  if (dtype != FSDP_F32 && dtype != FSDP_BF16)
    return fail(FSDP_ERR_UNSUPPORTED, "dtype %d not supported", static_cast<int>(dtype));
  return FSDP_OK;
}

template <typename T>
fsdp_status launch_norm_as(const fsdp_rms_norm_args& n, hipStream_t stream) {
  NormArgs<T> a{};
  a.x = static_cast<const T*>(n.x);
  a.res = static_cast<const T*>(n.residual);
  a.w = static_cast<const T*>(n.weight);
  a.sum = static_cast<T*>(n.residual_out);
  a.out = n.out;
  a.rstd = n.rstd;
  a.scales = n.scales;
  a.dim = n.dim;
  a.x_ld = n.x_pitch;
  a.res_ld = n.residual_pitch;
  a.sum_ld = n.residual_out_pitch;
  a.out_ld = n.out_pitch;
  a.eps = static_cast<float>(n.eps);
  if (a.res && a.scales) launch_norm<T, true, true>(a, n.rows, stream);
  else if (a.res) launch_norm<T, true, false>(a, n.rows, stream);
  else if (a.scales) launch_norm<T, false, true>(a, n.rows, stream);
  else launch_norm<T, false, false>(a, n.rows, stream);
  return fsdp::after_launch("fsdp_rms_norm");
}

fsdp_status norm(const fsdp_rms_norm_args* n, hipStream_t stream) {
  if (!n) return fail(FSDP_ERR_INVALID_ARG, "arguments pointer is NULL");
  if (fsdp_status st = check_sizes(n->rows, n->dim)) return st;
  if (fsdp_status st = check_type(n->dtype)) return st;
  if (!std::isfinite(n->eps) || !(n->eps >= 0.0))
    return fail(FSDP_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if ((n->residual == nullptr) != (n->residual_out == nullptr))
    return fail(FSDP_ERR_INVALID_ARG, "residual and residual_out go together");
  if (n->rows == 0) return FSDP_OK;
  const int es = n->dtype == FSDP_F32 ? 4 : 2;
  std::vector<fsdp::ByteRange> ranges;
  if (fsdp_status st = check_rows(n->x, n->x_pitch, n->rows, n->dim, es, false, "x", &ranges)) return st;
  if (fsdp_status st = check_rows(n->weight, n->dim, 1, n->dim, es, false, "weight", &ranges)) return st;
  if (fsdp_status st = check_rows(n->out, n->out_pitch, n->rows, n->dim, n->scales ? 1 : es, true, "out", &ranges))
    return st;
  if (n->residual) {
    if (fsdp_status st = check_rows(n->residual, n->residual_pitch, n->rows, n->dim, es, false, "residual", &ranges))
      return st;
    if (fsdp_status st = check_rows(n->residual_out, n->residual_out_pitch, n->rows, n->dim, es, true,
                                    "residual_out", &ranges))
      return st;
  }
  if (n->rstd)
    if (fsdp_status st = check_rows(n->rstd, n->rows, 1, n->rows, 4, true, "rstd", &ranges)) return st;
  if (n->scales)
    if (fsdp_status st = check_rows(n->scales, n->rows, 1, n->rows, 4, true, "scales", &ranges)) return st;
  if (fsdp_status st = fsdp::check_alias(ranges)) return st;
  if (fsdp_status st = fsdp::check_no_pending_error("fsdp_rms_norm")) return st;
  return n->dtype == FSDP_F32 ? launch_norm_as<float>(*n, stream) : launch_norm_as<uint16_t>(*n, stream);
}

template <typename T>
fsdp_status launch_back_as(const fsdp_rms_norm_backward_args& n, hipStream_t stream) {
  NormBackArgs<T> a{};
  a.dy = static_cast<const T*>(n.dy);
  a.x = static_cast<const T*>(n.x);
  a.w = static_cast<const T*>(n.weight);
  a.rstd = n.rstd;
  a.dres = static_cast<const T*>(n.dresidual);
  a.dx = static_cast<T*>(n.dx);
  a.partial = n.dweight ? static_cast<float*>(n.workspace) : nullptr;
  a.rows = n.rows;
  a.dim = n.dim;
  a.dy_ld = n.dy_pitch;
  a.x_ld = n.x_pitch;
  a.dres_ld = n.dresidual_pitch;
  a.dx_ld = n.dx_pitch;
  if (n.rows > 0) {
    if (a.dres) launch_back<T, true>(a, stream);
    else launch_back<T, false>(a, stream);
    if (fsdp_status st = fsdp::after_launch("fsdp_rms_norm_backward")) return st;
  }
  if (!n.dweight) return FSDP_OK;
  k_norm_dweight<T><<<unsigned((n.dim + 63) / 64), 1024, 0, stream>>>(
      a.partial, back_blocks(n.rows), n.dim, static_cast<T*>(n.dweight));
  return fsdp::after_launch("fsdp_rms_norm_backward");
}

int64_t back_workspace(int64_t rows, int64_t dim) { return int64_t(back_blocks(rows)) * dim * 4; }

fsdp_status norm_backward(const fsdp_rms_norm_backward_args* n, hipStream_t stream) {
  if (!n) return fail(FSDP_ERR_INVALID_ARG, "arguments pointer is NULL");
  if (fsdp_status st = check_sizes(n->rows, n->dim)) return st;
  if (fsdp_status st = check_type(n->dtype)) return st;
  const int es = n->dtype == FSDP_F32 ? 4 : 2;
  std::vector<fsdp::ByteRange> ranges;
  if (n->rows > 0) {
    if (fsdp_status st = check_rows(n->dy, n->dy_pitch, n->rows, n->dim, es, false, "dy", &ranges)) return st;
    if (fsdp_status st = check_rows(n->x, n->x_pitch, n->rows, n->dim, es, false, "x", &ranges)) return st;
    if (fsdp_status st = check_rows(n->weight, n->dim, 1, n->dim, es, false, "weight", &ranges)) return st;
    if (fsdp_status st = check_rows(n->rstd, n->rows, 1, n->rows, 4, false, "rstd", &ranges)) return st;
    if (n->dresidual)
      if (fsdp_status st = check_rows(n->dresidual, n->dresidual_pitch, n->rows, n->dim, es, false, "dresidual",
                                      &ranges))
        return st;
    if (fsdp_status st = check_rows(n->dx, n->dx_pitch, n->rows, n->dim, es, true, "dx", &ranges)) return st;
  }
  if (n->dweight) {
    if (fsdp_status st = check_rows(n->dweight, n->dim, 1, n->dim, es, true, "dweight", &ranges)) return st;
    const int64_t need = back_workspace(n->rows, n->dim);
    if (need > 0) {
      if (fsdp_status st = fsdp::check_ptr(n->workspace, "workspace", 16)) return st;
      if (n->workspace_bytes < need)
        return fail(FSDP_ERR_RANGE, "workspace has %lld bytes, needs %lld",
                    static_cast<long long>(n->workspace_bytes), static_cast<long long>(need));
      ranges.push_back(fsdp::range_of(n->workspace, need, 1, true, "workspace"));
    }
  }
  if (fsdp_status st = fsdp::check_alias(ranges)) return st;
  if (n->rows == 0 && !n->dweight) return FSDP_OK;
  if (fsdp_status st = fsdp::check_no_pending_error("fsdp_rms_norm_backward")) return st;
  return n->dtype == FSDP_F32 ? launch_back_as<float>(*n, stream) : launch_back_as<uint16_t>(*n, stream);
}

}  // namespace

extern "C" {

fsdp_status fsdp_rms_norm(const fsdp_rms_norm_args* args, hipStream_t stream) {
  fsdp::clear_error();
  try {
    return norm(args, stream);
  } catch (const std::bad_alloc&) {
    return fail(FSDP_ERR_INVALID_ARG, "out of host memory");
  }
}

fsdp_status fsdp_rms_norm_backward_workspace(int64_t rows, int64_t dim, int64_t* bytes) {
  fsdp::clear_error();
  if (!bytes) return fail(FSDP_ERR_INVALID_ARG, "bytes pointer is NULL");
  if (fsdp_status st = check_sizes(rows, dim)) return st;
  *bytes = back_workspace(rows, dim);
  return FSDP_OK;
}

fsdp_status fsdp_rms_norm_backward(const fsdp_rms_norm_backward_args* args, hipStream_t stream) {
  fsdp::clear_error();
  try {
    return norm_backward(args, stream);
  } catch (const std::bad_alloc&) {
    return fail(FSDP_ERR_INVALID_ARG, "out of host memory");
  }
}

}  // extern "C"

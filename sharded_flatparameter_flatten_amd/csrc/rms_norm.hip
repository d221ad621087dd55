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
#include <limits>
#include <new>
#include <type_traits>

#include "device_util.h"

#pragma clang fp contract(off)

using fsdp::fail;
using namespace fsdp::dev;

namespace {

constexpr float kE4m3Max = 448.f;
constexpr float kMinScale = 1.1754943508222875e-38f;   // 2^-126: a row of zeros divides by this
constexpr int64_t kStreamBytes = int64_t(32) << 20;    // outputs from here on are streamed past L2

// Two fp32 values to bf16 (nearest, ties to even) in one instruction: the same bits as
// to_bf16 for every value that is not NaN. A NaN keeps bits of its own here.
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t round_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2{a, b}, bf16x2));
}

__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const uint16_t* p) { return widen(*p); }
__device__ __forceinline__ void store1(float* p, float x) { *p = x; }
__device__ __forceinline__ void store1(uint16_t* p, float x) { *p = uint16_t(to_bf16(x)); }

// 16 bytes of a row as they lie in memory, kElems<T> consecutive elements. A lane holds
// two of these of every array, each next to its neighbour lane's: with 32 bytes a lane in
// one piece the streamed stores of fp32 wrote half sectors (4096 rows of 4096: 79 us, 39 so).
template <typename T>
constexpr int kElems = 16 / int(sizeof(T));
constexpr int kChunks = 2;
template <typename T>
struct Raw {
  u32x4 v;
};
// From element alignment; elements at or past `dim` are zeros.
template <typename I>   // int within a row held in registers, int64_t in the long kernels
__device__ __forceinline__ Raw<uint16_t> load_raw(const uint16_t* p, I c, I dim) {
  if (c + 8 <= dim) return {ld_loose<u32x4, 2>(p + c)};
  Raw<uint16_t> r{};
  if (c >= dim) return r;             // most lanes of a row's last piece
#pragma unroll
  for (int e = 0; e < 8; ++e)
    if (c + e < dim) r.v[e / 2] |= uint32_t(p[c + e]) << (16 * (e & 1));
  return r;
}
template <typename I>
__device__ __forceinline__ Raw<float> load_raw(const float* p, I c, I dim) {
  if (c + 4 <= dim) return {ld_loose<u32x4, 4>(p + c)};
  Raw<float> r{};
  if (c >= dim) return r;             // most lanes of a row's last piece
#pragma unroll
  for (int e = 0; e < 4; ++e)
    if (c + e < dim) r.v[e] = __float_as_uint(p[c + e]);
  return r;
}
__device__ __forceinline__ void unpack(const Raw<uint16_t>& r, float (&x)[8]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) { x[2 * e] = lo_bf16(r.v[e]); x[2 * e + 1] = hi_bf16(r.v[e]); }
}
__device__ __forceinline__ void unpack(const Raw<float>& r, float (&x)[4]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) x[e] = __uint_as_float(r.v[e]);
}
template <typename T>
__device__ __forceinline__ void load_as(const T* p, int64_t c, int64_t dim, float (&x)[kElems<T>]) {
  unpack(load_raw(p, c, dim), x);
}

// How a store goes: to element alignment, or, aligned to its size, past L2: through a
// descriptor of the row, where a row has whole waves, or not kept (nt) where it has not.
enum Way { kPlain, kStream, kOnce };
template <Way WAY, typename V, typename T, typename I>
__device__ __forceinline__ void store_vector(T* p, I c, I dim, V x) {
  if constexpr (WAY == kStream) st_stream(rsrc(p, int64_t(dim) * sizeof(T)), int(c) * int(sizeof(T)), x);
  else if constexpr (WAY == kOnce) __builtin_nontemporal_store(x, reinterpret_cast<V*>(p + c));
  else st_loose<V, sizeof(T)>(p + c, x);
}
// N values to column c of a row; elements at or past `dim` are left alone.
template <int N>
__device__ __forceinline__ bool has_nan(const float (&x)[N]) {   // one comparison for two values
  bool nan = false;
#pragma unroll
  for (int e = 0; e < N; e += 2) nan |= __builtin_isunordered(x[e], x[e + 1]);
  return nan;
}
template <Way WAY, int N, typename I>
__device__ __forceinline__ void store_as(float* p, I c, I dim, const float (&x)[N]) {
#pragma unroll
  for (int q = 0; q < N; q += 4) {
    if (c + q + 4 <= dim) {
      store_vector<WAY>(p, I(c + q), dim, u32x4{__float_as_uint(x[q]), __float_as_uint(x[q + 1]),
                                                   __float_as_uint(x[q + 2]), __float_as_uint(x[q + 3])});
    } else if (c + q < dim) {
#pragma unroll
      for (int e = q; e < q + 4; ++e)
        if (c + e < dim) p[c + e] = x[e];
    }
  }
}
// Every NaN is to_bf16's, in a row's whole vectors as in its ragged end; `nan` says whether
// this lane may have one. The comparisons and the branch cost up to 1% (2% at 16384
// columns); a sum of squares that is at hand is one comparison for all of its values.
template <Way WAY, typename I>
__device__ __forceinline__ void store_as(uint16_t* p, I c, I dim, const float (&x)[8], bool nan) {
  if (c + 8 <= dim) {
    u32x4 q;
#pragma unroll
    for (int e = 0; e < 4; ++e) q[e] = round_bf16(x[2 * e], x[2 * e + 1]);
    if (__builtin_expect(__builtin_amdgcn_ballot_w64(nan) != 0, 0)) {
#pragma unroll
      for (int e = 0; e < 4; ++e) q[e] = pack_bf16(x[2 * e], x[2 * e + 1]);
    }
    store_vector<WAY>(p, c, dim, q);
  } else if (c < dim) {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (c + e < dim) store1(p + c + e, x[e]);
  }
}
template <Way WAY, typename I>
__device__ __forceinline__ void store_as(uint16_t* p, I c, I dim, const float (&x)[8]) {
  store_as<WAY>(p, c, dim, x, has_nan(x));
}
template <Way WAY, typename I>
__device__ __forceinline__ void store_as(float* p, I c, I dim, const float (&x)[4], bool) {
  store_as<WAY>(p, c, dim, x);
}
// N values in e4m3 (nearest, ties to even), whose magnitudes round to 448 at most.
template <Way WAY, int N, typename I>
__device__ __forceinline__ void store_e4m3(uint8_t* p, I c, I dim, const float (&x)[N]) {
  uint32_t q[N / 4];
#pragma unroll
  for (int e = 0; e < N; e += 4) {
    const int half = __builtin_amdgcn_cvt_pk_fp8_f32(x[e], x[e + 1], 0, false);
    q[e / 4] = uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(x[e + 2], x[e + 3], half, true));
  }
  if (c + N <= dim) {
    if constexpr (N == 8) store_vector<WAY>(p, c, dim, u32x2{q[0], q[1]});
    else store_vector<WAY>(p, c, dim, q[0]);
  } else if (c < dim) {
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (c + e < dim) p[c + e] = uint8_t(q[e / 4] >> (8 * (e & 3)));
  }
}

// h rounded to T's type, as values.
__device__ __forceinline__ void round_to(float (&)[4]) {}
__device__ __forceinline__ void round_to(float (&h)[8]) {
#pragma unroll
  for (int e = 0; e < 8; e += 2) {
    const uint32_t q = round_bf16(h[e], h[e + 1]);
    h[e] = lo_bf16(q);
    h[e + 1] = hi_bf16(q);
  }
}

// The sum (and the largest bit pattern) over a row's L lanes, the same in every lane;
// `lds` holds a value for each wave of the workgroup.
template <int L>
__device__ __forceinline__ float row_sum(float v, float* lds) {
#pragma unroll
  for (int d = (L < 64 ? L : 64) / 2; d > 0; d >>= 1) v += __shfl_xor(v, d);
  if constexpr (L <= 64) return v;
  constexpr int W = L / 64;
  const int wave = threadIdx.x >> 6;
  __syncthreads();                      // lds may still be read by an earlier call
  if ((threadIdx.x & 63) == 0) lds[wave] = v;
  __syncthreads();
  const float* mine = lds + wave / W * W;
  if constexpr (W < 16) {
    float s = mine[0];
#pragma unroll
    for (int w = 1; w < W; ++w) s += mine[w];
    return s;
  } else {                              // 16 values at once would spill in k_norm_back
    float s = mine[threadIdx.x % W];
#pragma unroll
    for (int d = W / 2; d > 0; d >>= 1) s += __shfl_xor(s, d);
    return s;
  }
}
template <int L>
__device__ __forceinline__ uint32_t row_max(uint32_t v, float* lds) {
#pragma unroll
  for (int d = (L < 64 ? L : 64) / 2; d > 0; d >>= 1) v = max(v, uint32_t(__shfl_xor(v, d)));
  if constexpr (L <= 64) return v;
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = __uint_as_float(v);
  __syncthreads();
  uint32_t s = 0;
#pragma unroll
  for (int w = 0; w < L / 64; ++w) s = max(s, __float_as_uint(lds[w]));
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
// y is multiplied by 1 / scale: |y| <= 448 scale, so the product is below 448 (1 + 2^-22),
// which still rounds to 448, and no clamp is needed. A division by scale for each value
// took a quarter of the kernel's time; this differs from it by at most an fp32 step.
// A row is held by L lanes in registers: lane t's piece k is elements (L k + t) * kElems<T>
// onward. Long rows take a workgroup each; rows that a part of a wave can hold share a
// workgroup of four waves (32768 bf16 rows of 64 with a residual: 21 us with a wave
// a row, 6.6 so; their gradients 31 and 15).
// All three arrays are loaded before the row's sum is waited for. 8192 bf16 rows of 4096
// with a residual take 35.4 us with an e4m3 output and 38.2 with a bf16 one on the same
// buffers again and again, 41.6 the former (5.6 TB/s) with inputs that were not read
// lately; a single row 3 us. Ordinary stores took 6 us more, workgroups that stay for
// many rows and load the next ahead 10.
template <int L>
constexpr int kNormRows = L < 64 ? 256 / L : 1;
template <typename T, bool RES, bool BITS8, int L, Way WAY>
__global__ __launch_bounds__(L * kNormRows<L>) void k_norm(NormArgs<T> a, int64_t rows) {
  constexpr int CH = kChunks, E = kElems<T>;
  __shared__ float lds[(L + 63) / 64];
  const int t = threadIdx.x % L;
  const int64_t row = int64_t(blockIdx.x) * kNormRows<L> + threadIdx.x / L;
  if (L < 64 && row >= rows) return;              // a whole row's lanes; nothing waits for them
  const int dim = int(a.dim);
  auto col = [&](int k) { return (k * L + t) * E; };
  Raw<T> x[CH], r[CH], w[CH];
#pragma unroll
  for (int k = 0; k < CH; ++k) x[k] = load_raw(a.x + row * a.x_ld, col(k), dim);
  if constexpr (RES) {
#pragma unroll
    for (int k = 0; k < CH; ++k) r[k] = load_raw(a.res + row * a.res_ld, col(k), dim);
  }
#pragma unroll
  for (int k = 0; k < CH; ++k) w[k] = load_raw(a.w, col(k), dim);
  float h[CH][E];
  float sq = 0.f;
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    unpack(x[k], h[k]);
    if constexpr (RES) {
      float y[E];
      unpack(r[k], y);
#pragma unroll
      for (int e = 0; e < E; ++e) h[k][e] += y[e];
      round_to(h[k]);
    }
#pragma unroll
    for (int e = 0; e < E; ++e) sq += h[k][e] * h[k][e];
    if constexpr (RES) store_as<WAY>(a.sum + row * a.sum_ld, col(k), dim, h[k], sq != sq);
  }
  const float rstd = rstd_of(row_sum<L>(sq, lds), dim, a.eps);
  if (a.rstd && t == 0) a.rstd[row] = rstd;
  uint32_t top = 0;
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    float wk[E];
    unpack(w[k], wk);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      h[k][e] = h[k][e] * rstd * wk[e];
      if (BITS8 && col(k) + e < dim) top = max(top, abs_bits(h[k][e]));   // past dim: 0 * rstd may be NaN
    }
    if constexpr (!BITS8) store_as<WAY>(static_cast<T*>(a.out) + row * a.out_ld, col(k), dim, h[k]);
  }
  if constexpr (BITS8) {
    const float scale = scale_of(row_max<L>(top, lds));
    const float inverse = 1.f / scale;
    if (t == 0) a.scales[row] = scale;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
#pragma unroll
      for (int e = 0; e < E; ++e) h[k][e] *= inverse;
      store_e4m3<WAY>(static_cast<uint8_t*>(a.out) + row * a.out_ld, col(k), dim, h[k]);
    }
  }
}

// Rows too long for registers: the row is read again for each pass.
constexpr int kLongWaves = 16;
template <typename T, bool RES, bool BITS8>
__global__ __launch_bounds__(64 * kLongWaves) void k_norm_long(NormArgs<T> a) {
  constexpr int E = kElems<T>;
  __shared__ float lds[kLongWaves];
  const int64_t row = blockIdx.x, dim = a.dim, step = 64 * kLongWaves * E;
  const T* x = a.x + row * a.x_ld;
  const T* r = RES ? a.res + row * a.res_ld : nullptr;
  auto get = [&](int64_t c, float (&h)[E]) {
    load_as(x, c, dim, h);
    if constexpr (RES) {
      float y[E];
      load_as(r, c, dim, y);
#pragma unroll
      for (int e = 0; e < E; ++e) h[e] += y[e];
      round_to(h);
    }
  };
  float sq = 0.f;
  for (int64_t c = int64_t(threadIdx.x) * E; c < dim; c += step) {
    float h[E];
    get(c, h);
#pragma unroll
    for (int e = 0; e < E; ++e) sq += h[e] * h[e];
    if constexpr (RES) store_as<kPlain>(a.sum + row * a.sum_ld, c, dim, h);
  }
  const float rstd = rstd_of(row_sum<64 * kLongWaves>(sq, lds), dim, a.eps);
  if (a.rstd && threadIdx.x == 0) a.rstd[row] = rstd;
  float inverse = 1.f;
  if constexpr (BITS8) {
    uint32_t top = 0;
    for (int64_t c = int64_t(threadIdx.x) * E; c < dim; c += step) {
      float h[E], w[E];
      get(c, h);
      load_as(a.w, c, dim, w);
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (c + e < dim) top = max(top, abs_bits(h[e] * rstd * w[e]));
    }
    const float scale = scale_of(row_max<64 * kLongWaves>(top, lds));
    inverse = 1.f / scale;
    if (threadIdx.x == 0) a.scales[row] = scale;
  }
  for (int64_t c = int64_t(threadIdx.x) * E; c < dim; c += step) {
    float h[E], w[E];
    get(c, h);
    load_as(a.w, c, dim, w);
#pragma unroll
    for (int e = 0; e < E; ++e) {
      h[e] = h[e] * rstd * w[e];
      if constexpr (BITS8) h[e] *= inverse;
    }
    if constexpr (BITS8) store_e4m3<kPlain>(static_cast<uint8_t*>(a.out) + row * a.out_ld, c, dim, h);
    else store_as<kPlain>(static_cast<T*>(a.out) + row * a.out_ld, c, dim, h);
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

// A workgroup of 16 waves holds kRows = 1024 / L rows at a time, L lanes each, lane
// columns as in k_norm. The arrays of the next rows are loaded before this row's
// sum is joined, so that memory is busy while the waves wait for each other
// (512 workgroups of one row at a time took 70 us where this takes 42, 6.4 TB/s,
// at 8192 bf16 rows of 4096 with dresidual). Each lane sums its columns of dweight over its rows; the rows
// of a workgroup are joined in LDS at the end.
constexpr int kBackWaves = 16;
template <typename T, bool RES, int L, Way WAY>
__global__ __launch_bounds__(64 * kBackWaves) void k_norm_back(NormBackArgs<T> a) {
  constexpr int CH = kChunks, E = kElems<T>, kRows = 64 * kBackWaves / L;
  // rows of dweight sums to be joined, after those within a wave
  constexpr int kJoin = L < 64 ? kBackWaves : kRows;
  constexpr bool kKeepW = L < 1024;                 // otherwise the kernel spills; L2 holds it
  __shared__ float lds[kBackWaves];
  __shared__ float join[kJoin > 1 ? (kJoin - 1) * L * CH * E : 1];
  const int dim = int(a.dim);
  const int t = threadIdx.x % L;
  int group = threadIdx.x / L;
  if constexpr (L >= 64) group = __builtin_amdgcn_readfirstlane(group);
  auto col = [&](int k) { return (k * L + t) * E; };
  Raw<T> w[CH], x[CH], y[CH], r[CH];
  float dw[CH][E];
#pragma unroll
  for (int k = 0; k < CH; ++k) {
    if (kKeepW) w[k] = load_raw(a.w, col(k), dim);
#pragma unroll
    for (int e = 0; e < E; ++e) dw[k][e] = 0.f;
  }
  const int64_t step = int64_t(gridDim.x) * kRows;
  float rstd = 0.f;
  auto load = [&](int64_t row) {
    if (row >= a.rows) return;
    rstd = a.rstd[row];
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      x[k] = load_raw(a.x + row * a.x_ld, col(k), dim);
      y[k] = load_raw(a.dy + row * a.dy_ld, col(k), dim);
      if constexpr (RES) r[k] = load_raw(a.dres + row * a.dres_ld, col(k), dim);
    }
  };
  int64_t row = int64_t(blockIdx.x) * kRows + group;
  load(row);
  // every wave of the workgroup runs the same number of rounds (they meet in row_sum)
  for (int64_t first = int64_t(blockIdx.x) * kRows; first < a.rows; first += step, row += step) {
    const bool live = row < a.rows;
    Raw<T> cx[CH], cy[CH], cr[CH];
    const float cs = rstd;
#pragma unroll
    for (int k = 0; k < CH; ++k) {
      cx[k] = x[k];
      cy[k] = y[k];
      if constexpr (RES) cr[k] = r[k];
    }
    load(row + step);
    float dot = 0.f;
    if (live) {
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        float h[E], g[E], wk[E];
        unpack(cx[k], h);
        unpack(cy[k], g);
        unpack(kKeepW ? w[k] : load_raw(a.w, col(k), dim), wk);
#pragma unroll
        for (int e = 0; e < E; ++e) {
          h[e] = h[e] * cs;
          dw[k][e] += g[e] * h[e];
          dot += g[e] * wk[e] * h[e];             // zeros past dim
        }
      }
    }
    const float mean = row_sum<L>(dot, lds) / float(dim);
    if (live) {
#pragma unroll
      for (int k = 0; k < CH; ++k) {
        float h[E], g[E], wk[E];
        unpack(cx[k], h);
        unpack(cy[k], g);
        unpack(kKeepW ? w[k] : load_raw(a.w, col(k), dim), wk);
#pragma unroll
        for (int e = 0; e < E; ++e) h[e] = cs * (g[e] * wk[e] - h[e] * cs * mean);
        if constexpr (RES) {
          unpack(cr[k], g);
#pragma unroll
          for (int e = 0; e < E; ++e) h[e] += g[e];
        }
        store_as<WAY>(a.dx + row * a.dx_ld, col(k), dim, h);
      }
    }
  }
  if (!a.partial) return;
  if constexpr (L < 64) {                           // the wave's rows, then wave by wave
#pragma unroll
    for (int d = L; d < 64; d <<= 1)
#pragma unroll
      for (int k = 0; k < CH; ++k)
#pragma unroll
        for (int e = 0; e < E; ++e) dw[k][e] += __shfl_xor(dw[k][e], d);
    group = threadIdx.x >> 6;
  }
  if constexpr (kJoin > 1) {
    const bool holds = L >= 64 || int(threadIdx.x & 63) < L;
    if (group > 0 && holds) {
#pragma unroll
      for (int k = 0; k < CH; ++k)
#pragma unroll
        for (int e = 0; e < E; ++e) join[((group - 1) * CH * E + k * E + e) * L + t] = dw[k][e];
    }
    __syncthreads();
    if (group > 0 || !holds) return;
    constexpr int kUnroll = kJoin <= 4 ? kJoin - 1 : 1;   // more spills
#pragma unroll kUnroll
    for (int q = 0; q < kJoin - 1; ++q)
#pragma unroll
      for (int k = 0; k < CH; ++k)
#pragma unroll
        for (int e = 0; e < E; ++e) dw[k][e] += join[(q * CH * E + k * E + e) * L + t];
  }
#pragma unroll
  for (int k = 0; k < CH; ++k) store_as<kPlain>(a.partial + int64_t(blockIdx.x) * dim, col(k), dim, dw[k]);
}

// Rows too long for registers: dx here, the weight's sums in k_norm_back_cols.
template <typename T, bool RES>
__global__ __launch_bounds__(64 * kLongWaves) void k_norm_back_long(NormBackArgs<T> a) {
  constexpr int E = kElems<T>;
  __shared__ float lds[kLongWaves];
  const int64_t dim = a.dim, step = 64 * kLongWaves * E;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const T* x = a.x + row * a.x_ld;
    const T* dy = a.dy + row * a.dy_ld;
    const float rstd = a.rstd[row];
    float dot = 0.f;
    for (int64_t c = int64_t(threadIdx.x) * E; c < dim; c += step) {
      float h[E], g[E], w[E];
      load_as(x, c, dim, h);
      load_as(dy, c, dim, g);
      load_as(a.w, c, dim, w);
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (c + e < dim) dot += g[e] * w[e] * (h[e] * rstd);
    }
    const float mean = row_sum<64 * kLongWaves>(dot, lds) / float(dim);
    for (int64_t c = int64_t(threadIdx.x) * E; c < dim; c += step) {
      float h[E], g[E], w[E];
      load_as(x, c, dim, h);
      load_as(dy, c, dim, g);
      load_as(a.w, c, dim, w);
#pragma unroll
      for (int e = 0; e < E; ++e) h[e] = rstd * (g[e] * w[e] - h[e] * rstd * mean);
      if constexpr (RES) {
        float y[E];
        load_as(a.dres + row * a.dres_ld, c, dim, y);
#pragma unroll
        for (int e = 0; e < E; ++e) h[e] += y[e];
      }
      store_as<kPlain>(a.dx + row * a.dx_ld, c, dim, h);
    }
  }
}
// The weight's sums of rows blockIdx.y, blockIdx.y + gridDim.y, ... for 256 lanes' columns.
template <typename T>
__global__ __launch_bounds__(256) void k_norm_back_cols(NormBackArgs<T> a) {
  constexpr int E = kElems<T>;
  const int64_t c = (int64_t(blockIdx.x) * 256 + threadIdx.x) * E;
  if (c >= a.dim) return;
  float dw[E] = {};
  for (int64_t row = blockIdx.y; row < a.rows; row += gridDim.y) {
    float h[E], g[E];
    load_as(a.x + row * a.x_ld, c, a.dim, h);
    load_as(a.dy + row * a.dy_ld, c, a.dim, g);
#pragma unroll
    for (int e = 0; e < E; ++e) dw[e] += g[e] * (h[e] * a.rstd[row]);
  }
  store_as<kPlain>(a.partial + int64_t(blockIdx.y) * a.dim, c, a.dim, dw);
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
  if (c < dim) {
    int r = wave;
    for (; r + 7 * 16 < parts; r += 8 * 16) {     // 8 loads under way
      float v[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) v[q] = partial[int64_t(r + 16 * q) * dim + c];
#pragma unroll
      for (int q = 0; q < 8; ++q) s += v[q];
    }
    for (; r < parts; r += 16) s += partial[int64_t(r) * dim + c];
  }
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

// Lanes that hold a row, 32 bytes each: 8 to 1024, a power of two. Longer rows go through
// the k_*_long kernels.
constexpr int kMaxLanes = 1024;
int row_lanes(int64_t dim, int elem) {
  int l = 8;
  while (l < kMaxLanes && l * int64_t(32 / elem) < dim) l *= 2;
  return l;
}
bool row_fits(int64_t dim, int elem) { return dim <= kMaxLanes * int64_t(32 / elem); }

// Workgroups (and partial rows) of a backward launch: one a CU, or fewer for
// few rows.
constexpr int64_t kBackBlocks = 256;
constexpr int64_t kLongBlocks = 512;
int32_t back_blocks(int64_t rows, int64_t dim, int elem) {
  if (!row_fits(dim, elem)) return int32_t(std::min(rows, kLongBlocks));
  const int64_t per = 64 * kBackWaves / row_lanes(dim, elem);
  return int32_t(std::min((rows + per - 1) / per, kBackBlocks));
}

template <int L = 8, typename F>
void with_lanes(int lanes, F&& f) {
  if constexpr (L < kMaxLanes) {
    if (lanes > L) return with_lanes<2 * L>(lanes, f);
  }
  f(std::integral_constant<int, L>{});
}

template <int L>
constexpr Way past_l2_way = L < 64 ? kOnce : kStream;

bool rows_aligned(const void* p, int64_t ld, int elem, int to) {
  return reinterpret_cast<uintptr_t>(p) % to == 0 && ld * elem % to == 0;
}

template <typename T, bool RES, bool BITS8>
void launch_norm(const NormArgs<T>& a, int64_t rows, hipStream_t stream) {
  if (!row_fits(a.dim, sizeof(T))) {
    k_norm_long<T, RES, BITS8><<<unsigned(rows), 64 * kLongWaves, 0, stream>>>(a);
    return;
  }
  const int64_t written = rows * a.dim * ((RES ? int(sizeof(T)) : 0) + (BITS8 ? 1 : int(sizeof(T))));
  const bool past_l2 = written >= kStreamBytes && rows_aligned(a.out, a.out_ld, BITS8 ? 1 : sizeof(T), BITS8 ? 8 : 16) &&
                      (!RES || rows_aligned(a.sum, a.sum_ld, sizeof(T), 16));
  with_lanes(row_lanes(a.dim, sizeof(T)), [&](auto l) {
    constexpr int L = l.value, per = kNormRows<L>;
    const unsigned blocks = unsigned((rows + per - 1) / per);
    if (past_l2) k_norm<T, RES, BITS8, L, past_l2_way<L>><<<blocks, L * per, 0, stream>>>(a, rows);
    else k_norm<T, RES, BITS8, L, kPlain><<<blocks, L * per, 0, stream>>>(a, rows);
  });
}

template <typename T, bool RES>
void launch_back(const NormBackArgs<T>& a, hipStream_t stream) {
  const int32_t blocks = back_blocks(a.rows, a.dim, sizeof(T));
  if (!row_fits(a.dim, sizeof(T))) {
    k_norm_back_long<T, RES><<<blocks, 64 * kLongWaves, 0, stream>>>(a);
    if (a.partial)
      k_norm_back_cols<T><<<dim3(unsigned((a.dim + 256 * kElems<T> - 1) / (256 * kElems<T>)), blocks), 256, 0, stream>>>(a);
    return;
  }
  const bool past_l2 = a.rows * a.dim * int64_t(sizeof(T)) >= kStreamBytes && rows_aligned(a.dx, a.dx_ld, sizeof(T), 16);
  with_lanes(row_lanes(a.dim, sizeof(T)), [&](auto l) {
    constexpr int L = l.value;
    if (past_l2) k_norm_back<T, RES, L, past_l2_way<L>><<<blocks, 64 * kBackWaves, 0, stream>>>(a);
    else k_norm_back<T, RES, L, kPlain><<<blocks, 64 * kBackWaves, 0, stream>>>(a);
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
  if (n.eps > 0.0 && a.eps == 0.f) a.eps = std::numeric_limits<float>::denorm_min();   // 0 / 0 otherwise
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
      a.partial, back_blocks(n.rows, n.dim, sizeof(T)), n.dim, static_cast<T*>(n.dweight));
  return fsdp::after_launch("fsdp_rms_norm_backward");
}

int64_t back_workspace(int64_t rows, int64_t dim) {
  return int64_t(std::max(back_blocks(rows, dim, 2), back_blocks(rows, dim, 4))) * dim * 4;
}

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

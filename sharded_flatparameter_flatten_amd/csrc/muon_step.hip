// The element-wise halves of the sharded Muon step on gfx950, and their entry
// points: the ranks' gradient rows folded into the momentum, and the
// orthogonalised matrices applied to this rank's window of the master weights.
//
// Both stream through HBM once and are bound by its bandwidth. Every
// floating-point step is one binary32 operation (no fused multiply-add).

#include <algorithm>
#include <cmath>
#include <new>

#include "device_util.h"

#pragma clang fp contract(off)

using fsdp::fail;
using namespace fsdp::dev;

namespace {

constexpr int kThreads = 64;      // one wave a workgroup
constexpr int kV = 4;             // consecutive elements a lane
constexpr int64_t kTile = int64_t(kThreads) * kV;
constexpr int64_t kFastElems = int64_t(1) << 22;   // windows from here on stream past L2
// Workgroups per CU of the streaming momentum kernel with 8 rows (the 7B block's
// window: 105 us without a limit, 100 with 14, 103 with 16 to 24, 117 with 10); with
// fewer rows more of them, for alike many bytes (a window of 26.2 M elements and one
// row: 65 us with 14, 48.5 so; 4 rows 79 and 72.7).
// The streaming apply is best without one (44 us; 47 with 16, 56 with 12).
constexpr int kMomentumPerCu = 14;

// ---------------------------------------------------------------------------
// gradient rows -> momentum and update
// ---------------------------------------------------------------------------

struct MomentumArgs {
  const uint16_t* g[FSDP_MAX_RANKS];   // rank-window start of each row
  float* m;
  uint16_t* u;
  int64_t n;
  int32_t n_grads;
  int32_t nesterov;
  float gs, mu;
};

__device__ __forceinline__ void momentum(const MomentumArgs& a, float g, float& m, float& u) {
  m = a.mu * m + g;
  u = a.nesterov ? g + a.mu * m : m;
}

// A lane's 4 elements of an array that a workgroup reads or writes at tile start
// t0. FAST: through a descriptor over the tile, the loads of data read once and
// the stores streamed; the addresses are aligned to the access. Otherwise at
// element alignment.
template <bool FAST, typename V, int CPOL, typename T>
__device__ __forceinline__ V load4(const T* p, int64_t t0, int64_t len) {
  const int off = int(threadIdx.x) * kV * int(sizeof(T));
  if constexpr (!FAST) return ld_loose<V, sizeof(T)>(reinterpret_cast<const char*>(p + t0) + off);
  else if constexpr (sizeof(V) == 8) return __builtin_amdgcn_raw_buffer_load_b64(rsrc(p + t0, len * sizeof(T)), off, 0, CPOL);
  else return __builtin_bit_cast(V, __builtin_amdgcn_raw_buffer_load_b128(rsrc(p + t0, len * sizeof(T)), off, 0, CPOL));
}
template <bool FAST, typename V, typename T>
__device__ __forceinline__ void store4(T* p, int64_t t0, int64_t len, V x) {
  const int off = int(threadIdx.x) * kV * int(sizeof(T));
  if constexpr (FAST) st_stream(rsrc(p + t0, len * sizeof(T)), off, x);
  else st_loose<V, sizeof(T)>(reinterpret_cast<char*>(p + t0) + off, x);
}
constexpr int kNt = 2;     // CPol nt

__device__ __forceinline__ u32x4 bits4(const float (&x)[kV]) {
  return u32x4{__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3])};
}

// The rows are folded in rank order from row 0 in fp32 and scaled, as the
// reduce of the other step calls does; 8 rows' loads are under way at a time.
// ROWS: the rows too are aligned (a rank's window of them often is not; then they are loaded
// at element alignment beside the streamed rest: 26.2 M elements of 8 rows off by one
// 115 us, 124 with nothing streamed, 104 with all of it).
template <bool FAST, bool ROWS>
__global__ __launch_bounds__(kThreads) void k_muon_momentum(MomentumArgs a) {
  const int64_t t0 = int64_t(blockIdx.x) * kTile, i = t0 + int64_t(threadIdx.x) * kV;
  const int64_t len = a.n - t0 < kTile ? a.n - t0 : kTile;
  if (i + kV <= a.n) {
    float acc[kV];
    for (int k = 0; k < a.n_grads; k += 8) {
      u32x2 q[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (k + j < a.n_grads) q[j] = load4<FAST && ROWS, u32x2, kNt>(a.g[k + j], t0, len);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (k + j < a.n_grads) {
          const float x[kV] = {lo_bf16(q[j].x), hi_bf16(q[j].x), lo_bf16(q[j].y), hi_bf16(q[j].y)};
#pragma unroll
          for (int e = 0; e < kV; ++e) acc[e] = k + j ? acc[e] + x[e] : x[e];
        }
    }
    const f32x4 old = load4<FAST, f32x4, 0>(a.m, t0, len);
    float m[kV], u[kV];
#pragma unroll
    for (int e = 0; e < kV; ++e) {
      m[e] = old[e];
      momentum(a, acc[e] * a.gs, m[e], u[e]);
    }
    store4<FAST>(a.m, t0, len, bits4(m));
    store4<FAST>(a.u, t0, len, u32x2{pack_bf16(u[0], u[1]), pack_bf16(u[2], u[3])});
  } else {
    for (int64_t j = i; j < a.n; ++j) {
      float acc = widen(a.g[0][j]);
      for (int k = 1; k < a.n_grads; ++k) acc = acc + widen(a.g[k][j]);
      float m = a.m[j], u;
      momentum(a, acc * a.gs, m, u);
      a.m[j] = m;
      a.u[j] = uint16_t(to_bf16(u));
    }
  }
}

// ---------------------------------------------------------------------------
// orthogonalised matrices -> master and bf16 parameter
// ---------------------------------------------------------------------------

// One tensor's part of the window.
struct Part {
  const uint16_t* u;     // its first element in the window
  int64_t at;            // where the part starts in the window
  int64_t len;
  int64_t tile_end;      // exclusive prefix of tiles over the launch
  float scale;
};
constexpr int kMaxParts = 64;
struct ApplyArgs {
  Part part[kMaxParts];
  float* p;
  uint16_t* w;           // bf16 parameter out, or null
  int64_t tiles;
  int32_t np;
  float lr, wd;
};

__device__ __forceinline__ float apply(const ApplyArgs& a, float scale, float u, float p) {
  return p - a.lr * (scale * u + a.wd * p);
}

// A part's tiles start at the window position at or below its start that is a
// multiple of 4, so the fp32 accesses keep the master's alignment whatever the
// tensors' lengths are; lanes that straddle an end go element by element.
template <bool FAST>
__global__ __launch_bounds__(kThreads) void k_muon_apply(ApplyArgs a) {
  const int64_t t = blockIdx.x;
  int lo = 0, hi = a.np - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (t < a.part[mid].tile_end) hi = mid;
    else lo = mid + 1;
  }
  const Part& d = a.part[lo];
  const int64_t tile0 = lo ? a.part[lo - 1].tile_end : 0;
  const int64_t t0 = d.at / kV * kV + (t - tile0) * kTile, i = t0 + int64_t(threadIdx.x) * kV;
  const int64_t end = d.at + d.len, len = end - t0 < kTile ? end - t0 : kTile;
  const uint16_t* u = d.u - d.at;      // only dereferenced within [at, end)
  if (i >= d.at && i + kV <= end) {
    const u32x2 q = ld_loose<u32x2, 2>(u + i);
    const f32x4 old = load4<FAST, f32x4, 0>(a.p, t0, len);
    const float x[kV] = {lo_bf16(q.x), hi_bf16(q.x), lo_bf16(q.y), hi_bf16(q.y)};
    float p[kV];
#pragma unroll
    for (int e = 0; e < kV; ++e) p[e] = apply(a, d.scale, x[e], old[e]);
    store4<FAST>(a.p, t0, len, bits4(p));
    if (a.w) store4<FAST>(a.w, t0, len, u32x2{pack_bf16(p[0], p[1]), pack_bf16(p[2], p[3])});
  } else {
    const int64_t from = i < d.at ? d.at : i, to = i + kV < end ? i + kV : end;
    for (int64_t j = from; j < to; ++j) {
      const float p = apply(a, d.scale, widen(u[j]), a.p[j]);
      a.p[j] = p;
      if (a.w) a.w[j] = uint16_t(to_bf16(p));
    }
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

fsdp_status check_hparams(const fsdp_muon_hparams* hp) {
  if (!hp) return fail(FSDP_ERR_INVALID_ARG, "hyper-parameters pointer is NULL");
  if (!std::isfinite(hp->lr) || hp->lr < 0.0)
    return fail(FSDP_ERR_INVALID_ARG, "lr must be finite and >= 0");
  if (!(hp->momentum >= 0.0 && hp->momentum < 1.0))
    return fail(FSDP_ERR_INVALID_ARG, "momentum must lie in [0, 1)");
  if (hp->nesterov != 0 && hp->nesterov != 1)
    return fail(FSDP_ERR_INVALID_ARG, "nesterov must be 0 or 1");
  if (!std::isfinite(hp->weight_decay))
    return fail(FSDP_ERR_INVALID_ARG, "weight_decay must be finite");
  if (!std::isfinite(hp->grad_scale))
    return fail(FSDP_ERR_INVALID_ARG, "grad_scale must be finite");
  return FSDP_OK;
}

bool aligned(const void* p, int to) { return reinterpret_cast<uintptr_t>(p) % to == 0; }

// Unused dynamic LDS that leaves room for n workgroups per CU (160 KiB of LDS).
size_t cap_lds(int n) { return size_t(163840 / n / 512 * 512); }

// A launch holds fewer than 2^32 threads.
fsdp_status check_grid(int64_t tiles, const char* what) {
  if (tiles > (int64_t(1) << 32) / kThreads - 1) return fail(FSDP_ERR_RANGE, "%s: the window needs too many workgroups", what);
  return FSDP_OK;
}

fsdp_status reduce_momentum(const fsdp_unit* u, int32_t n_grads, const void* const* grads,
                            float* momentum, void* update, const fsdp_muon_hparams* hp,
                            hipStream_t stream) {
  const char* what = "fsdp_reduce_momentum_shard";
  if (fsdp_status st = fsdp::check_unit(u)) return st;
  if (n_grads < 1 || n_grads > FSDP_MAX_RANKS)
    return fail(FSDP_ERR_INVALID_ARG, "n_grads must be in [1, %d] (got %d)", FSDP_MAX_RANKS, n_grads);
  if (fsdp_status st = check_hparams(hp)) return st;
  if (u->valid == 0) return FSDP_OK;            // a window of pad only: nothing to do
  if (!grads) return fail(FSDP_ERR_INVALID_ARG, "grads array is NULL");
  MomentumArgs a{};
  std::vector<fsdp::ByteRange> ranges;
  for (int32_t k = 0; k < n_grads; ++k) {
    if (!grads[k]) return fail(FSDP_ERR_INVALID_ARG, "grads[%d] is NULL", k);
    if (reinterpret_cast<uintptr_t>(grads[k]) & 1u)
      return fail(FSDP_ERR_INVALID_ARG, "grads[%d] is not 2-byte aligned", k);
    a.g[k] = static_cast<const uint16_t*>(grads[k]) + u->begin;
    ranges.push_back(fsdp::range_of(a.g[k], u->valid, 2, false, "grads", k));
  }
  if (fsdp_status st = fsdp::check_ptr(momentum, "momentum", 4)) return st;
  if (fsdp_status st = fsdp::check_ptr(update, "update_bf16_out", 2)) return st;
  ranges.push_back(fsdp::range_of(momentum, u->valid, 4, true, "momentum"));
  ranges.push_back(fsdp::range_of(update, u->valid, 2, true, "update_bf16_out"));
  if (fsdp_status st = fsdp::check_alias(ranges)) return st;
  const int64_t tiles = (u->valid + kTile - 1) / kTile;
  if (fsdp_status st = check_grid(tiles, what)) return st;
  a.m = momentum;
  a.u = static_cast<uint16_t*>(update);
  a.n = u->valid;
  a.n_grads = n_grads;
  a.nesterov = hp->nesterov;
  a.gs = static_cast<float>(hp->grad_scale);
  a.mu = static_cast<float>(hp->momentum);
  if (fsdp_status st = fsdp::check_no_pending_error(what)) return st;
  const bool fast = u->valid >= kFastElems && aligned(momentum, 16) && aligned(update, 8);
  bool rows = true;
  for (int32_t k = 0; k < n_grads; ++k) rows = rows && aligned(a.g[k], 8);
  const int per_cu = kMomentumPerCu * 80 / (8 * std::min(n_grads, 8) + 16);   // alike many bytes a CU
  const size_t lds = per_cu < 32 ? cap_lds(per_cu) : 0;
  if (fast && rows) k_muon_momentum<true, true><<<unsigned(tiles), kThreads, lds, stream>>>(a);
  else if (fast) k_muon_momentum<true, false><<<unsigned(tiles), kThreads, lds, stream>>>(a);
  else k_muon_momentum<false, false><<<unsigned(tiles), kThreads, 0, stream>>>(a);
  return fsdp::after_launch(what);
}

fsdp_status muon_apply(const fsdp_unit* u, const void* const* tensors, const double* scales,
                       float* master, void* param, const fsdp_muon_hparams* hp,
                       hipStream_t stream) {
  const char* what = "fsdp_muon_apply_shard";
  if (fsdp_status st = fsdp::check_unit(u)) return st;
  if (fsdp_status st = check_hparams(hp)) return st;
  if (u->valid == 0) return FSDP_OK;            // a window of pad only: nothing to do
  if (!tensors) return fail(FSDP_ERR_INVALID_ARG, "tensors array is NULL");
  if (!scales) return fail(FSDP_ERR_INVALID_ARG, "scales array is NULL");
  if (fsdp_status st = fsdp::check_ptr(master, "master", 4)) return st;
  if (reinterpret_cast<uintptr_t>(param) & 1u)
    return fail(FSDP_ERR_INVALID_ARG, "param_bf16_out is not 2-byte aligned");
  std::vector<fsdp::ByteRange> ranges;
  ranges.push_back(fsdp::range_of(master, u->valid, 4, true, "master"));
  if (param) ranges.push_back(fsdp::range_of(param, u->valid, 2, true, "param_bf16_out"));
  std::vector<ApplyArgs> launches;
  for (int32_t i = 0; i < u->T; ++i) {
    const int64_t lo = std::max(u->begin, u->offset[i]);
    const int64_t hi = std::min(u->begin + u->valid, u->offset[i + 1]);
    if (lo >= hi) continue;                     // outside the window: its pointer is not used
    if (fsdp_status st = fsdp::check_ptr(tensors[i], "a tensor in the window", 2)) return st;
    if (!std::isfinite(scales[i]))
      return fail(FSDP_ERR_INVALID_ARG, "scales[%d] must be finite", i);
    const uint16_t* src = static_cast<const uint16_t*>(tensors[i]) + (lo - u->offset[i]);
    ranges.push_back(fsdp::range_of(src, hi - lo, 2, false, "tensors", i));
    if (launches.empty() || launches.back().np == kMaxParts) {
      launches.emplace_back();
      launches.back() = ApplyArgs{};
      launches.back().p = master;
      launches.back().w = static_cast<uint16_t*>(param);
      launches.back().lr = static_cast<float>(hp->lr);
      launches.back().wd = static_cast<float>(hp->weight_decay);
    }
    ApplyArgs& a = launches.back();
    Part& d = a.part[a.np++];
    d.u = src;
    d.at = lo - u->begin;
    d.len = hi - lo;
    d.scale = static_cast<float>(scales[i]);
    a.tiles += (d.at + d.len - d.at / kV * kV + kTile - 1) / kTile;
    d.tile_end = a.tiles;
  }
  if (fsdp_status st = fsdp::check_alias(ranges)) return st;
  for (const ApplyArgs& a : launches)
    if (fsdp_status st = check_grid(a.tiles, what)) return st;
  if (fsdp_status st = fsdp::check_no_pending_error(what)) return st;
  const bool fast = u->valid >= kFastElems && aligned(master, 16) && aligned(param, 8);
  for (const ApplyArgs& a : launches) {
    if (fast) k_muon_apply<true><<<unsigned(a.tiles), kThreads, 0, stream>>>(a);
    else k_muon_apply<false><<<unsigned(a.tiles), kThreads, 0, stream>>>(a);
    if (fsdp_status st = fsdp::after_launch(what)) return st;
  }
  return FSDP_OK;
}

}  // namespace

extern "C" {

fsdp_status fsdp_reduce_momentum_shard(const fsdp_unit* u, int32_t n_grads,
                                       const void* const* grads, float* momentum,
                                       void* update_bf16_out, const fsdp_muon_hparams* hp,
                                       hipStream_t stream) {
  fsdp::clear_error();
  try {
    return reduce_momentum(u, n_grads, grads, momentum, update_bf16_out, hp, stream);
  } catch (const std::bad_alloc&) {
    return fail(FSDP_ERR_INVALID_ARG, "out of host memory");
  }
}

fsdp_status fsdp_muon_apply_shard(const fsdp_unit* u, const void* const* tensors_bf16,
                                  const double* scales, float* master, void* param_bf16_out,
                                  const fsdp_muon_hparams* hp, hipStream_t stream) {
  fsdp::clear_error();
  try {
    return muon_apply(u, tensors_bf16, scales, master, param_bf16_out, hp, stream);
  } catch (const std::bad_alloc&) {
    return fail(FSDP_ERR_INVALID_ARG, "out of host memory");
  }
}

}  // extern "C"

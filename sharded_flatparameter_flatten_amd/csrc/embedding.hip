// Embedding lookup with scaling on gfx950, its gradient by sorted tokens, and their entry points.
//
//   out[n] = scale * weight[t_n], a row of zeros where t_n is no row of weight;
//   dweight[v] = scale * sum over the n with t_n = v of dy[n]   [+ dweight[v]],
// in fp32, each output rounded once. A token outside [0, vocab), or equal to padding_idx, adds
// nothing to the gradient.
//
// The sums go in the order of n, whatever the launch, so the same inputs give the same bits: the
// positions are sorted by token first (one launch, no atomics on global memory), then each row of
// the vocabulary is summed from its list.

#include <cmath>

#include "row_util.h"

#pragma clang fp contract(off)

using fsdp::fail;
using namespace fsdp::dev;

namespace {

constexpr int kSortWaves = 16;
constexpr int kMaxRange = 512;       // rows of the vocabulary that a workgroup sorts, at most

template <typename T>
struct EmbedArgs {
  const int64_t* tokens;
  const T* w;
  T* out;
  int64_t rows, vocab, dim, w_ld, out_ld;
  float scale;
};

// `lanes` lanes a row, 256 / lanes rows a workgroup. Bound by HBM.
template <typename T>
__global__ __launch_bounds__(256) void k_embedding(EmbedArgs<T> a, int lanes) {
  const int64_t row = int64_t(blockIdx.x) * (256 / lanes) + threadIdx.x / lanes;
  if (row >= a.rows) return;
  const int64_t t = a.tokens[row];
  const bool inside = uint64_t(t) < uint64_t(a.vocab);
  const T* w = a.w + (inside ? t : 0) * a.w_ld;
  T* out = a.out + row * a.out_ld;
  for (int64_t c = threadIdx.x % lanes * 8; c < a.dim; c += lanes * 8) {
    float v[8];
    unpack(load_group(w, c, a.dim), v);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = inside ? v[e] * a.scale : 0.f;
    store_group(out, c, a.dim, v);
  }
}

// The positions of all tokens, sorted by token and, for equal ones, by position: `order`; the
// list of row v is order[start[v]] to order[start[v + 1] - 1].
//
// Workgroup g sorts what falls into its `range` rows of the vocabulary, on its own: every
// workgroup reads all tokens, so it also counts how many fall before its range, which is where
// its part of `order` begins. Each wave has a stretch of the tokens and counts, then places, its
// own; between the two the counts of the waves before it become its first places.
__global__ __launch_bounds__(64 * kSortWaves) void k_embed_sort(const int64_t* tokens, int64_t n, int64_t vocab,
                                                                int64_t padding, int range, int32_t* start,
                                                                int32_t* order) {
  __shared__ int32_t at[kSortWaves][kMaxRange];
  __shared__ int32_t total[kMaxRange], before[kSortWaves];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t lo = int64_t(blockIdx.x) * range;
  const int here = int(vocab - lo < range ? vocab - lo : range);
  const int64_t stretch = (n + 64 * kSortWaves - 1) / (64 * kSortWaves) * 64;
  const int64_t begin = wave * stretch, end = begin + stretch < n ? begin + stretch : n;
  for (int v = lane; v < here; v += 64) at[wave][v] = 0;
  int32_t less = 0;
  for (int64_t i = begin + lane; i < end; i += 64) {
    const int64_t t = tokens[i];
    if (t < 0 || t >= vocab || t == padding) continue;
    less += t < lo;
    if (t >= lo && t < lo + here) atomicAdd(&at[wave][t - lo], 1);
  }
  less = wave_sum(less);
  if (lane == 0) before[wave] = less;
  __syncthreads();
  int32_t base = 0;
#pragma unroll
  for (int w = 0; w < kSortWaves; ++w) base += before[w];
  const int v = threadIdx.x;
  if (v < here) {
    int32_t sum = 0;
    for (int w = 0; w < kSortWaves; ++w) sum += at[w][v];
    total[v] = sum;
  }
  __syncthreads();
  if (wave == 0) {                    // sums become places: an exclusive scan, 64 rows at a time
    int32_t carry = base;
    for (int v0 = 0; v0 < here; v0 += 64) {
      const int32_t own = v0 + lane < here ? total[v0 + lane] : 0;
      int32_t x = own;
#pragma unroll
      for (int d = 1; d < 64; d *= 2) {
        const int32_t y = __shfl_up(x, d);
        if (lane >= d) x += y;
      }
      if (v0 + lane < here) total[v0 + lane] = carry + x - own;
      carry += __shfl(x, 63);
    }
    if (lane == 0 && lo + here == vocab) start[vocab] = carry;
  }
  __syncthreads();
  if (v < here) {
    int32_t place = total[v];
    start[lo + v] = place;
    for (int w = 0; w < kSortWaves; ++w) {
      const int32_t own = at[w][v];
      at[w][v] = place;
      place += own;
    }
  }
  __syncthreads();
  for (int64_t i0 = begin; i0 < end; i0 += 64) {
    const int64_t i = i0 + lane;
    const int64_t t = i < end ? tokens[i] : -1;
    const bool mine = t >= lo && t < lo + here && t != padding;
    uint64_t left = __builtin_amdgcn_ballot_w64(mine);
    while (left) {                    // one token of the range at a time, all lanes that have it
      const int first = __builtin_ctzll(left);
      const int row = __builtin_amdgcn_readlane(int(t - lo), first);
      const uint64_t same = __builtin_amdgcn_ballot_w64(mine && t - lo == row);
      const int32_t place = at[wave][row];
      if (same >> lane & 1) order[place + __builtin_popcountll(same & ((uint64_t(1) << lane) - 1))] = int32_t(i);
      if (lane == first) at[wave][row] = place + __builtin_popcountll(same);
      left &= ~same;
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");   // the next round reads what one lane wrote
    }
  }
}

template <typename T>
struct EmbedBackArgs {
  const T* dy;
  T* dw;
  const int32_t* start;
  const int32_t* order;
  int64_t vocab, dim, dy_ld, dw_ld;
  float scale;
};

// `lanes` lanes a row of the vocabulary, 256 / lanes rows a workgroup. Bound by HBM: most rows
// are absent, and zeros are written.
template <typename T, bool ADD>
__global__ __launch_bounds__(256) void k_embed_back(EmbedBackArgs<T> a, int lanes) {
  const int64_t v = int64_t(blockIdx.x) * (256 / lanes) + threadIdx.x / lanes;
  if (v >= a.vocab) return;
  const int32_t begin = a.start[v], end = a.start[v + 1];
  if (ADD && begin == end) return;
  T* dw = a.dw + v * a.dw_ld;
  for (int64_t c = threadIdx.x % lanes * 8; c < a.dim; c += lanes * 8) {
    float sum[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int32_t i = begin; i < end; ++i) {
      float x[8];
      unpack(load_group(a.dy + int64_t(a.order[i]) * a.dy_ld, c, a.dim), x);
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[e] += x[e];
    }
    float old[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (ADD) unpack(load_group(dw, c, a.dim), old);
#pragma unroll
    for (int e = 0; e < 8; ++e) sum[e] = ADD ? old[e] + sum[e] * a.scale : sum[e] * a.scale;
    store_group(dw, c, a.dim, sum);
  }
}

int range_of_rows(int64_t vocab) {
  const int64_t range = (vocab + 255) / 256;
  return int(range < kMaxRange ? range : kMaxRange);
}

int64_t back_workspace(int64_t rows, int64_t vocab) { return ((vocab + 1 + rows) * 4 + 15) / 16 * 16; }

fsdp_status check_sizes(int64_t rows, int64_t vocab, int64_t dim) {
  if (fsdp_status st = fsdp::check_row_sizes(rows, dim)) return st;
  if (vocab < 1 || vocab >= (int64_t(1) << 22))
    return fail(FSDP_ERR_RANGE, "vocab must be in [1, 2^22) (got %lld)", static_cast<long long>(vocab));
  return FSDP_OK;
}

fsdp_status check_scale(double scale) {
  if (!std::isfinite(scale)) return fail(FSDP_ERR_INVALID_ARG, "scale must be finite");
  return FSDP_OK;
}

template <typename T>
fsdp_status launch(const fsdp_embedding_args& n, hipStream_t stream) {
  EmbedArgs<T> a{};
  a.tokens = n.tokens;
  a.w = static_cast<const T*>(n.weight);
  a.out = static_cast<T*>(n.out);
  a.rows = n.rows;
  a.vocab = n.vocab;
  a.dim = n.dim;
  a.w_ld = n.weight_pitch;
  a.out_ld = n.out_pitch;
  a.scale = static_cast<float>(n.scale);
  const int lanes = fsdp::lanes_of_row(n.dim), per = 256 / lanes;
  k_embedding<T><<<unsigned((n.rows + per - 1) / per), 256, 0, stream>>>(a, lanes);
  return fsdp::after_launch("fsdp_embedding");
}

fsdp_status embedding(const fsdp_embedding_args* n, hipStream_t stream) {
  if (!n) return fail(FSDP_ERR_INVALID_ARG, "arguments pointer is NULL");
  if (fsdp_status st = check_sizes(n->rows, n->vocab, n->dim)) return st;
  if (fsdp_status st = fsdp::check_row_type(n->dtype)) return st;
  if (fsdp_status st = check_scale(n->scale)) return st;
  if (n->rows == 0) return FSDP_OK;
  const int es = n->dtype == FSDP_F32 ? 4 : 2;
  std::vector<fsdp::ByteRange> ranges;
  if (fsdp_status st = fsdp::check_row_arg(n->tokens, n->rows, 1, n->rows, 8, false, "tokens", &ranges)) return st;
  if (fsdp_status st = fsdp::check_row_arg(n->weight, n->weight_pitch, n->vocab, n->dim, es, false, "weight", &ranges))
    return st;
  if (fsdp_status st = fsdp::check_row_arg(n->out, n->out_pitch, n->rows, n->dim, es, true, "out", &ranges)) return st;
  if (fsdp_status st = fsdp::check_alias(ranges)) return st;
  if (fsdp_status st = fsdp::check_no_pending_error("fsdp_embedding")) return st;
  return n->dtype == FSDP_F32 ? launch<float>(*n, stream) : launch<uint16_t>(*n, stream);
}

template <typename T>
fsdp_status launch_back(const fsdp_embedding_backward_args& n, hipStream_t stream) {
  int32_t* start = static_cast<int32_t*>(n.workspace);
  int32_t* order = start + n.vocab + 1;
  const int range = range_of_rows(n.vocab);
  k_embed_sort<<<unsigned((n.vocab + range - 1) / range), 64 * kSortWaves, 0, stream>>>(
      n.tokens, n.rows, n.vocab, n.padding_idx, range, start, order);
  if (fsdp_status st = fsdp::after_launch("fsdp_embedding_backward")) return st;
  EmbedBackArgs<T> a{};
  a.dy = static_cast<const T*>(n.dy);
  a.dw = static_cast<T*>(n.dweight);
  a.start = start;
  a.order = order;
  a.vocab = n.vocab;
  a.dim = n.dim;
  a.dy_ld = n.dy_pitch;
  a.dw_ld = n.dweight_pitch;
  a.scale = static_cast<float>(n.scale);
  const int lanes = fsdp::lanes_of_row(n.dim), per = 256 / lanes;
  const unsigned blocks = unsigned((n.vocab + per - 1) / per);
  if (n.accumulate) k_embed_back<T, true><<<blocks, 256, 0, stream>>>(a, lanes);
  else k_embed_back<T, false><<<blocks, 256, 0, stream>>>(a, lanes);
  return fsdp::after_launch("fsdp_embedding_backward");
}

fsdp_status backward(const fsdp_embedding_backward_args* n, hipStream_t stream) {
  if (!n) return fail(FSDP_ERR_INVALID_ARG, "arguments pointer is NULL");
  if (fsdp_status st = check_sizes(n->rows, n->vocab, n->dim)) return st;
  if (fsdp_status st = fsdp::check_row_type(n->dtype)) return st;
  if (fsdp_status st = check_scale(n->scale)) return st;
  if (n->accumulate != 0 && n->accumulate != 1) return fail(FSDP_ERR_INVALID_ARG, "accumulate must be 0 or 1");
  const int es = n->dtype == FSDP_F32 ? 4 : 2;
  std::vector<fsdp::ByteRange> ranges;
  if (n->rows > 0) {
    if (fsdp_status st = fsdp::check_row_arg(n->tokens, n->rows, 1, n->rows, 8, false, "tokens", &ranges)) return st;
    if (fsdp_status st = fsdp::check_row_arg(n->dy, n->dy_pitch, n->rows, n->dim, es, false, "dy", &ranges)) return st;
  } else if (n->accumulate) {
    return FSDP_OK;
  }
  if (fsdp_status st = fsdp::check_row_arg(n->dweight, n->dweight_pitch, n->vocab, n->dim, es, true, "dweight", &ranges))
    return st;
  if (fsdp_status st = fsdp::check_workspace(n->workspace, n->workspace_bytes, back_workspace(n->rows, n->vocab), 16,
                                             &ranges))
    return st;
  if (fsdp_status st = fsdp::check_alias(ranges)) return st;
  if (fsdp_status st = fsdp::check_no_pending_error("fsdp_embedding_backward")) return st;
  return n->dtype == FSDP_F32 ? launch_back<float>(*n, stream) : launch_back<uint16_t>(*n, stream);
}

}  // namespace

extern "C" {

fsdp_status fsdp_embedding(const fsdp_embedding_args* args, hipStream_t stream) {
  fsdp::clear_error();
  try {
    return embedding(args, stream);
  } catch (const std::bad_alloc&) {
    return fail(FSDP_ERR_INVALID_ARG, "out of host memory");
  }
}

fsdp_status fsdp_embedding_backward_workspace(int64_t rows, int64_t vocab, int64_t dim, int64_t* bytes) {
  fsdp::clear_error();
  if (!bytes) return fail(FSDP_ERR_INVALID_ARG, "bytes pointer is NULL");
  if (fsdp_status st = check_sizes(rows, vocab, dim)) return st;
  *bytes = back_workspace(rows, vocab);
  return FSDP_OK;
}

fsdp_status fsdp_embedding_backward(const fsdp_embedding_backward_args* args, hipStream_t stream) {
  fsdp::clear_error();
  try {
    return backward(args, stream);
  } catch (const std::bad_alloc&) {
    return fail(FSDP_ERR_INVALID_ARG, "out of host memory");
  }
}

}  // extern "C"

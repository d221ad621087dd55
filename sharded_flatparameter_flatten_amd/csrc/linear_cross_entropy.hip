// Softmax cross entropy of a head's logits, without keeping the logits, and its gradients, on
// gfx950, with its entry points.
//
// For the rows x_r of hidden whose target t_r is in [0, vocab), with z = x_r weight^T,
//   loss_r = log(1 + sum over v != t_r of exp(z_v - z_t)),
//   G = k (softmax(z) - onehot(t)),  dhidden = G weight,  dweight = G^T hidden.
//
// A call gathers the rows that count into the workspace, end to end (so the others cost nothing
// and what they hold reaches nothing), and works them off in pieces:
//   1. tiles of z: each leaves its rows' maximum m and sum S of exp(z - m), both without the
//      target's column, and P = exp(z - m) in fp16 (values in [0, 1], held to 2^-11);
//   2. a row's m and S joined over the tiles give its loss; P becomes
//      softmax(z) - onehot in bf16, in place;
//   3. the two products with it.
// So the logits' product is made once, 6 rows vocab dim operations in all, for a scratch of
// 2 bytes a logit of the piece. Keeping nothing would take the product twice.
//
// The target's column stays out of the sums because what matters of a sure row is
// sum exp(z_v - z_t), far below 1: as the difference of two logarithms it would be lost. Its
// entry of G is expm1(-loss), which does not cancel either.

#include <algorithm>
#include <cmath>

#include "row_util.h"

#pragma clang fp contract(off)

using fsdp::fail;
using namespace fsdp::dev;

namespace {

typedef _Float16 f16;
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

constexpr int kT = 64;                // tile
constexpr int kGatherRows = 32;       // rows a workgroup gathers
constexpr int64_t kScratch = int64_t(1) << 30;
constexpr int64_t kMaxProduct = int64_t(1) << 35;   // elements of an operand or a result: grids stay below 2^32 lanes

// What the kernels of one call share.
struct Loss {
  const uint16_t* x;                  // the caller's hidden
  const uint16_t* w;
  const int64_t* targets;
  int32_t* count;                     // rows that count
  int32_t* map;                       // their places among the caller's
  int32_t* target;                    // and targets
  uint16_t* xc;                       // and values, dim_pad + 64 apart, zeros past dim
  float* row_loss;
  float* loss;
  float* losses;                      // or NULL
  uint16_t* dx;
  uint16_t* dw;
  uint16_t* g;                        // P, then G: piece rows, g_ld apart
  f32x2* stats;                       // m and S of a piece's rows, tile by tile
  float* right;                       // the targets' logits of a piece's rows
  float* acc;                         // dweight's sums of the pieces before
  int64_t rows, vocab, dim, x_ld, xc_ld, w_ld, dx_ld, dw_ld, g_ld;
  int64_t piece;
  int32_t tiles;                      // of the vocabulary
  int32_t mean;
  int32_t grads;                      // dx or dw is wanted
  float scale;
};

__device__ __forceinline__ bool counts(const Loss& a, int64_t t) { return uint64_t(t) < uint64_t(a.vocab); }

// k of the gradients.
__device__ __forceinline__ float factor(const Loss& a) {
  return a.mean ? a.scale / float(*a.count > 1 ? *a.count : 1) : a.scale;
}

// Every workgroup counts the rows that count before its own, so it knows where they go.
__global__ __launch_bounds__(256) void k_loss_gather(Loss a) {
  __shared__ int32_t part[4];
  __shared__ int32_t to[kGatherRows];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t row0 = int64_t(blockIdx.x) * kGatherRows;
  int32_t before = 0;
  for (int64_t i = threadIdx.x; i < row0; i += 256) before += counts(a, a.targets[i]);
  before = wave_sum(before);
  if (lane == 0) part[wave] = before;
  __syncthreads();
  const int32_t base = part[0] + part[1] + part[2] + part[3];
  if (wave == 0) {
    const int64_t row = row0 + lane;
    const int64_t t = lane < kGatherRows && row < a.rows ? a.targets[row] : -1;
    const uint64_t have = __builtin_amdgcn_ballot_w64(counts(a, t));
    const int32_t c = base + __builtin_popcountll(have & ((uint64_t(1) << lane) - 1));
    if (lane < kGatherRows) to[lane] = counts(a, t) ? c : -1;
    if (counts(a, t)) {
      a.map[c] = int32_t(row);
      a.target[c] = int32_t(t);
    }
    if (lane == 0 && row0 + kGatherRows >= a.rows) *a.count = base + __builtin_popcountll(have);
  }
  __syncthreads();
  for (int r = wave; r < kGatherRows; r += 4) {
    const int64_t row = row0 + r;
    if (row >= a.rows) return;
    const int32_t c = to[r];
    if (c < 0) {
      if (a.losses && lane == 0) a.losses[row] = 0.f;
      if (!a.dx) continue;
      const float zero[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      for (int64_t k = lane * 8; k < a.dim; k += 512) store_group(a.dx + row * a.dx_ld, k, a.dim, zero);
      continue;
    }
    for (int64_t k = lane * 8; k < a.xc_ld - 64; k += 512)
      *reinterpret_cast<u32x4*>(a.xc + c * a.xc_ld + k) = load_group(a.x + row * a.x_ld, k, a.dim).v[0];
  }
}

enum Kind { kLogits, kHidden, kWeight };

// C[i][j] = sum over k of A[i][k] B[j][k], 64 x 64 by 4 waves:
//   kLogits  i: vocabulary, j: row, k: dim;
//   kHidden  i: dim, j: row, k: vocabulary;
//   kWeight  i: dim, j: vocabulary, k: row.
template <Kind KIND>
__global__ __launch_bounds__(256) void k_loss_product(Loss a, int64_t row0, int tiles_i) {
  constexpr int kPitch = 72;
  __shared__ __attribute__((aligned(16))) uint16_t la[kT * kPitch], lb[kT * kPitch];
  __shared__ float z[kT][kT + 1];
  const int64_t left = *a.count - row0;
  const int64_t n = left < 0 ? 0 : left < a.piece ? left : a.piece;
  const int64_t i0 = int64_t(blockIdx.x) % tiles_i * kT, j0 = int64_t(blockIdx.x) / tiles_i * kT;
  const int64_t side_i = KIND == kLogits ? a.vocab : a.dim;
  const int64_t side_j = KIND == kWeight ? a.vocab : n;
  const int64_t depth = KIND == kLogits ? a.dim : KIND == kHidden ? a.vocab : n;
  if (j0 >= side_j || (KIND == kWeight && row0 > 0 && n == 0)) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, wi = wave / 2 * 32, wj = wave % 2 * 32;
  const uint16_t* xc = a.xc + row0 * a.xc_ld;
  f32x16 acc;
#pragma unroll
  for (int e = 0; e < 16; ++e) acc[e] = 0.f;
  for (int64_t k0 = 0; k0 < depth; k0 += kT) {
    __syncthreads();
    for (int q = threadIdx.x; q < kT * kT; q += 256) {
      const int in = q % kT, out = q / kT;            // `in` runs along memory
      uint16_t u = 0, v = 0;
      if (KIND == kLogits) {
        if (i0 + out < side_i && k0 + in < depth) u = a.w[(i0 + out) * a.w_ld + k0 + in];
        la[out * kPitch + in] = u;
      } else if (KIND == kHidden) {
        if (k0 + out < depth && i0 + in < side_i) u = a.w[(k0 + out) * a.w_ld + i0 + in];
        la[in * kPitch + out] = u;
      } else {
        if (k0 + out < depth && i0 + in < side_i) u = xc[(k0 + out) * a.xc_ld + i0 + in];
        la[in * kPitch + out] = u;
      }
      if (KIND == kWeight) {
        if (k0 + out < depth && j0 + in < side_j) v = a.g[(k0 + out) * a.g_ld + j0 + in];
        lb[in * kPitch + out] = v;
      } else {
        const uint16_t* b = KIND == kLogits ? xc : a.g;
        const int64_t ld = KIND == kLogits ? a.xc_ld : a.g_ld;
        if (j0 + out < side_j && k0 + in < depth) v = b[(j0 + out) * ld + k0 + in];
        lb[out * kPitch + in] = v;
      }
    }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kT / 16; ++q) {
      const bf16x8 fa = *reinterpret_cast<const bf16x8*>(la + (wi + (lane & 31)) * kPitch + q * 16 + lane / 32 * 8);
      const bf16x8 fb = *reinterpret_cast<const bf16x8*>(lb + (wj + (lane & 31)) * kPitch + q * 16 + lane / 32 * 8);
      acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fa, fb, acc, 0, 0, 0);
    }
  }
  // a lane holds i = 8 g + 4 (lane / 32) + e, j = lane % 32 in element 4 g + e
#pragma unroll
  for (int e = 0; e < 16; ++e) z[wj + (lane & 31)][wi + e / 4 * 8 + lane / 32 * 4 + e % 4] = acc[e];
  __syncthreads();
  if (KIND == kLogits) {
    const int r = threadIdx.x / 4, c0 = threadIdx.x % 4 * 16;
    const int64_t row = j0 + r;
    const int64_t t = row < n ? a.target[row0 + row] - i0 : -1;
    float m = -INFINITY, s = 0.f;
    for (int c = c0; c < c0 + 16; ++c)
      if (i0 + c < side_i && c != t) m = fmaxf(m, z[r][c]);
    m = fmaxf(m, __shfl_xor(m, 1));
    m = fmaxf(m, __shfl_xor(m, 2));
    const float from = m == -INFINITY ? 0.f : m;
    for (int c = c0; c < c0 + 16; ++c) {
      const float p = i0 + c < side_i && c != t ? expf(z[r][c] - from) : 0.f;
      s += p;
      if (row < n && a.grads) reinterpret_cast<f16*>(a.g)[row * a.g_ld + i0 + c] = f16(p);
      if (c == t) a.right[row] = z[r][c];
    }
    s += __shfl_xor(s, 1);
    s += __shfl_xor(s, 2);
    if (row < n && c0 == 0) a.stats[row * a.tiles + i0 / kT] = f32x2{m, s};
    return;
  }
  const float k = factor(a);
  for (int q = threadIdx.x; q < kT * kT; q += 256) {
    const int in = q % kT, out = q / kT;
    if (i0 + in >= side_i || j0 + out >= side_j) continue;
    float v = z[out][in];
    if (KIND == kHidden) {
      a.dx[a.map[row0 + j0 + out] * a.dx_ld + i0 + in] = uint16_t(to_bf16(v * k));
      continue;
    }
    float* sum = a.acc ? a.acc + (j0 + out) * a.xc_ld + i0 + in : nullptr;
    if (row0 > 0) v += *sum;
    if (left <= a.piece) a.dw[(j0 + out) * a.dw_ld + i0 + in] = uint16_t(to_bf16(v * k));
    else *sum = v;
  }
}

// A row's loss from its tiles' m and S, and its row of G.
__global__ __launch_bounds__(256) void k_loss_rows(Loss a, int64_t row0) {
  __shared__ float part[8];
  const int64_t r = blockIdx.x;
  if (row0 + r >= *a.count) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const f32x2* stats = a.stats + r * a.tiles;
  float m = -INFINITY, s = 0.f;
  for (int t = threadIdx.x; t < a.tiles; t += 256) m = fmaxf(m, stats[t].x);
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor(m, d));
  if (lane == 0) part[wave] = m;
  __syncthreads();
  m = fmaxf(fmaxf(part[0], part[1]), fmaxf(part[2], part[3]));
  const float from = m == -INFINITY ? 0.f : m;
  for (int t = threadIdx.x; t < a.tiles; t += 256) s += stats[t].y * expf((stats[t].x == -INFINITY ? from : stats[t].x) - from);
  s = wave_sum(s);
  if (lane == 0) part[4 + wave] = s;
  __syncthreads();
  s = (part[4] + part[5]) + (part[6] + part[7]);
  const float right = a.right[r], ahead = m - right;
  const float loss = ahead > 0.f ? ahead + logf(s + expf(-ahead)) : log1pf(s * expf(ahead));
  if (threadIdx.x == 0) {
    a.row_loss[row0 + r] = loss;
    if (a.losses) a.losses[a.map[row0 + r]] = loss;
  }
  if (!a.grads) return;
  const int32_t target = a.target[row0 + r];
  uint16_t* g = a.g + r * a.g_ld;
  for (int64_t c = threadIdx.x; c < int64_t(a.tiles) * kT; c += 256) {
    const float mt = stats[c / kT].x;
    const float f = mt == -INFINITY ? 0.f : expf(mt - right - loss);
    const float p = float(reinterpret_cast<const f16*>(g)[c]) * f;
    g[c] = uint16_t(to_bf16(c == target ? expm1f(-loss) : p));
  }
}

__global__ __launch_bounds__(1024) void k_loss_mean(Loss a) {
  __shared__ double part[16];
  const int n = *a.count;
  double sum = 0.0;
  for (int i = threadIdx.x; i < n; i += 1024) sum += double(a.row_loss[i]);
  sum = wave_sum(sum);
  if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = sum;
  __syncthreads();
  if (threadIdx.x) return;
  sum = 0.0;
  for (int w = 0; w < 16; ++w) sum += part[w];
  *a.loss = float(a.mean ? sum / double(n > 1 ? n : 1) : sum);
}

int64_t round_up(int64_t x, int64_t to) { return (x + to - 1) / to * to; }

struct Plan {
  int64_t piece, pieces, tiles, g_ld, xc_ld;
  int64_t count, map, target, xc, row_loss, g, stats, right, acc, bytes;   // workspace offsets
};

Plan make_plan(const fsdp_linear_cross_entropy_args& n) {
  Plan p{};
  const bool grads = n.dhidden || n.dweight;
  p.tiles = (n.vocab + kT - 1) / kT;
  p.g_ld = p.tiles * kT + 64;
  p.xc_ld = round_up(n.dim, 64) + 64;
  p.piece = n.piece > 0 ? n.piece : std::max<int64_t>(256, kScratch / (2 * p.g_ld) / 256 * 256);
  p.piece = std::max<int64_t>(1, std::min(p.piece, n.rows));
  p.pieces = std::max<int64_t>(1, (n.rows + p.piece - 1) / p.piece);
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t here = at;
    at += round_up(bytes, 256);
    return here;
  };
  p.count = take(4);
  p.map = take(n.rows * 4);
  p.target = take(n.rows * 4);
  p.row_loss = take(n.rows * 4);
  p.right = take(p.piece * 4);
  p.stats = take(p.piece * p.tiles * 8);
  p.xc = take(n.rows * p.xc_ld * 2);
  p.g = take(grads ? p.piece * p.g_ld * 2 : 0);
  p.acc = take(n.dweight && p.pieces > 1 ? n.vocab * p.xc_ld * 4 : 0);
  p.bytes = at;
  return p;
}

fsdp_status check_sizes(const fsdp_linear_cross_entropy_args& n) {
  if (fsdp_status st = fsdp::check_row_sizes(n.rows, n.dim)) return st;
  if (n.dim > (int64_t(1) << 20))
    return fail(FSDP_ERR_RANGE, "dim must be in [1, 2^20] (got %lld)", static_cast<long long>(n.dim));
  if (n.vocab < 1 || n.vocab >= (int64_t(1) << 22))
    return fail(FSDP_ERR_RANGE, "vocab must be in [1, 2^22) (got %lld)", static_cast<long long>(n.vocab));
  if (n.piece < 0) return fail(FSDP_ERR_RANGE, "piece must be >= 0 (got %lld)", static_cast<long long>(n.piece));
  const int64_t rows = std::max<int64_t>(1, n.piece ? std::min(n.piece, n.rows) : n.rows);
  if (std::max({n.vocab * n.dim, rows * n.dim, n.piece ? rows * n.vocab : 1}) > kMaxProduct)
    return fail(FSDP_ERR_RANGE, "rows %lld (in a piece), vocab %lld, dim %lld: a product of two is over 2^35",
                static_cast<long long>(rows), static_cast<long long>(n.vocab), static_cast<long long>(n.dim));
  return FSDP_OK;
}

fsdp_status run(const fsdp_linear_cross_entropy_args* n, hipStream_t stream) {
  if (!n) return fail(FSDP_ERR_INVALID_ARG, "arguments pointer is NULL");
  if (fsdp_status st = check_sizes(*n)) return st;
  if (!std::isfinite(n->grad_scale)) return fail(FSDP_ERR_INVALID_ARG, "grad_scale must be finite");
  if (n->reduction != FSDP_MEAN && n->reduction != FSDP_SUM)
    return fail(FSDP_ERR_INVALID_ARG, "reduction %d is neither mean nor sum", static_cast<int>(n->reduction));
  std::vector<fsdp::ByteRange> ranges;
  auto rows_arg = [&](const void* p, int64_t ld, int64_t rows, bool write, const char* name) {
    return fsdp::check_row_arg(p, ld, rows, n->dim, 2, write, name, &ranges);
  };
  if (n->rows > 0) {
    if (fsdp_status st = rows_arg(n->hidden, n->hidden_pitch, n->rows, false, "hidden")) return st;
    if (fsdp_status st = rows_arg(n->weight, n->weight_pitch, n->vocab, false, "weight")) return st;
    if (fsdp_status st = fsdp::check_row_arg(n->targets, n->rows, 1, n->rows, 8, false, "targets", &ranges)) return st;
    if (n->losses)
      if (fsdp_status st = fsdp::check_row_arg(n->losses, n->rows, 1, n->rows, 4, true, "losses", &ranges)) return st;
    if (n->dhidden)
      if (fsdp_status st = rows_arg(n->dhidden, n->dhidden_pitch, n->rows, true, "dhidden")) return st;
  }
  if (n->dweight)
    if (fsdp_status st = rows_arg(n->dweight, n->dweight_pitch, n->vocab, true, "dweight")) return st;
  if (fsdp_status st = fsdp::check_row_arg(n->loss, 1, 1, 1, 4, true, "loss", &ranges)) return st;
  const Plan p = make_plan(*n);
  if (fsdp_status st = fsdp::check_workspace(n->workspace, n->workspace_bytes, p.bytes, 256, &ranges)) return st;
  if (fsdp_status st = fsdp::check_alias(ranges)) return st;
  if (fsdp_status st = fsdp::check_no_pending_error("fsdp_linear_cross_entropy")) return st;

  char* ws = static_cast<char*>(n->workspace);
  Loss a{};
  a.x = static_cast<const uint16_t*>(n->hidden);
  a.w = static_cast<const uint16_t*>(n->weight);
  a.targets = n->targets;
  a.count = reinterpret_cast<int32_t*>(ws + p.count);
  a.map = reinterpret_cast<int32_t*>(ws + p.map);
  a.target = reinterpret_cast<int32_t*>(ws + p.target);
  a.xc = reinterpret_cast<uint16_t*>(ws + p.xc);
  a.row_loss = reinterpret_cast<float*>(ws + p.row_loss);
  a.loss = n->loss;
  a.losses = n->losses;
  a.dx = static_cast<uint16_t*>(n->dhidden);
  a.dw = static_cast<uint16_t*>(n->dweight);
  a.g = reinterpret_cast<uint16_t*>(ws + p.g);
  a.stats = reinterpret_cast<f32x2*>(ws + p.stats);
  a.right = reinterpret_cast<float*>(ws + p.right);
  a.acc = n->dweight && p.pieces > 1 ? reinterpret_cast<float*>(ws + p.acc) : nullptr;
  a.rows = n->rows;
  a.vocab = n->vocab;
  a.dim = n->dim;
  a.x_ld = n->hidden_pitch;
  a.xc_ld = p.xc_ld;
  a.w_ld = n->weight_pitch;
  a.dx_ld = n->dhidden_pitch;
  a.dw_ld = n->dweight_pitch;
  a.g_ld = p.g_ld;
  a.piece = p.piece;
  a.tiles = int32_t(p.tiles);
  a.mean = n->reduction == FSDP_MEAN;
  a.grads = a.dx || a.dw;
  a.scale = static_cast<float>(n->grad_scale);

  auto tiles_of = [](int64_t side) { return int((side + kT - 1) / kT); };
  k_loss_gather<<<unsigned(std::max<int64_t>(1, (n->rows + kGatherRows - 1) / kGatherRows)), 256, 0, stream>>>(a);
  for (int64_t i = 0; i < p.pieces; ++i) {
    const int64_t row0 = i * p.piece;
    const int in_dim = tiles_of(n->dim), in_rows = tiles_of(std::min(p.piece, n->rows - row0)), in_vocab = tiles_of(n->vocab);
    if (in_rows > 0) {
      k_loss_product<kLogits><<<in_vocab * in_rows, 256, 0, stream>>>(a, row0, in_vocab);
      k_loss_rows<<<unsigned(std::min(p.piece, n->rows - row0)), 256, 0, stream>>>(a, row0);
      if (a.dx) k_loss_product<kHidden><<<in_dim * in_rows, 256, 0, stream>>>(a, row0, in_dim);
    }
    if (a.dw) k_loss_product<kWeight><<<in_dim * in_vocab, 256, 0, stream>>>(a, row0, in_dim);
    if (fsdp_status st = fsdp::after_launch("fsdp_linear_cross_entropy")) return st;
  }
  k_loss_mean<<<1, 1024, 0, stream>>>(a);
  return fsdp::after_launch("fsdp_linear_cross_entropy");
}

}  // namespace

extern "C" {

fsdp_status fsdp_linear_cross_entropy_workspace(const fsdp_linear_cross_entropy_args* args, int64_t* bytes) {
  fsdp::clear_error();
  if (!args) return fail(FSDP_ERR_INVALID_ARG, "arguments pointer is NULL");
  if (!bytes) return fail(FSDP_ERR_INVALID_ARG, "bytes pointer is NULL");
  if (fsdp_status st = check_sizes(*args)) return st;
  *bytes = make_plan(*args).bytes;
  return FSDP_OK;
}

fsdp_status fsdp_linear_cross_entropy(const fsdp_linear_cross_entropy_args* args, hipStream_t stream) {
  fsdp::clear_error();
  try {
    return run(args, stream);
  } catch (const std::bad_alloc&) {
    return fail(FSDP_ERR_INVALID_ARG, "out of host memory");
  }
}

}  // extern "C"

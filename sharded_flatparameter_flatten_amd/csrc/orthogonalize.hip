// Orthogonalisation of a list of matrices by Newton-Schulz products (the
// update of the Muon step) on gfx950, and its entry points.
//
// For a matrix G with m = min(rows, cols) and n = max(rows, cols), X is the
// m x n one of G and its transpose, and
//   X_0 = X / (|X|_F + eps)
//   S = X X^T,  P = a I + b S + c S S,  X <- P X          (`steps` times).
// All the work is in the three products, which are run as one kind of tiled
// product C = A B^T with both operands stored along the contracted axis:
//   S = X X^T                 rows of X with rows of X;
//   S S = S S^T               (S is symmetric);
//   (P X)^T = X^T P^T         rows of X^T with rows of P.
// X is therefore kept in both orientations; the epilogue of the third product
// writes both. S and P are symmetric: only the tiles on and below the diagonal
// are computed, and each is stored with its mirror image. The additions of
// a I and b S are in the second product's epilogue.
//
// Two steps at once: with S_2 = P_1 P_1 S_1 and P_2 its polynomial, X <- (P_2 P_1) X.
// Everything but the first S and the last product is then m x m and symmetric
// (polynomials of S commute), which is less work where n is well over m. The
// diagonal stays inside P: kept apart, as a I + P', the products cancel against
// it once S is near I. Pairs of steps and single ones alternate: two pairs in a
// row lose half as much again to rounding (3e-3 against 2.1e-3 after 5 steps),
// three steps at once up to six times as much.
//
// Numerics: the operands of the matrix instructions are fp16 and every sum is
// held in fp32. fp16 rather than bf16, at the same rate, because each rounding
// of X is amplified: the polynomial raises the small singular values (up to
// 3.4 times a step) over rounding errors that are relative to the large ones.
// With bf16 operands the result is about 1.1e-2 from the exact polynomial,
// with fp16 ones 1.4e-3 (2-norm, matrices with a few strong directions over
// noise). Both grow as the singular values fall faster: fp16 gives 3.6e-3 for
// 1/k and 2e-2 for 1/k^2 (384 x 1536), half to all of what a change of 2^-11 in
// each element of G makes, and a sixth of what G's own rounding to bf16 does. The
// values are scaled by powers of two to sit in fp16's normal range: X by
// 2^12, S and P by 2^10, so |X| < 16, |S| < 64 and |P| < 64 are representable;
// singular values start at 1 or less and stay below 1.3 with the usual
// coefficients. With others the host bounds what X, S and P can reach at each
// step and takes smaller powers (see Reach). A matrix whose norm is far below eps loses precision (its X
// has elements near fp16's subnormals once norm / eps < 1e-4).

#include <algorithm>
#include <cmath>
#include <initializer_list>
#include <new>

#include "tile_util.h"

#pragma clang fp contract(off)

using fsdp::fail;
using namespace fsdp::dev;

namespace {

typedef _Float16 f16;
typedef f16 f16x8 __attribute__((ext_vector_type(8)));
typedef f16 f16x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x16 __attribute__((ext_vector_type(16)));

constexpr double kScaleX = 4096;      // stored X is X * 2^12, at most
constexpr double kScaleS = 1024;      // stored S and P are times 2^10, at most
constexpr int kBK = 64;               // contracted elements per stage: one 128-byte line a row
constexpr int kPitchPad = 64;         // elements between rows: see pitch_of
constexpr int kMaxMats = 24;          // matrices per launch (kernel arguments < 4 KB)
constexpr int kSumBlocks = 256;       // partial sums of squares per matrix, at most
constexpr int kSumRow = 8192;         // a contiguous matrix is summed as rows of this length

// ---------------------------------------------------------------------------
// the tiled product
// ---------------------------------------------------------------------------

// One matrix's product in a launch: C[i][j] = sum_k A[i][k] B[j][k]. Every
// buffer is padded with zeros to whole tiles on both axes, so the kernel has
// no bounds to check except those of the final output.
enum Kind : int32_t {
  kSym,      // a symmetric result: alpha * sum
  kPoly,     // the same: alpha * sum + beta * A + delta * I
  kUpdate,   // any result: alpha * sum
  kFinal     // bf16 output: alpha * sum
};
struct Prod {
  const f16* a;
  const f16* b;
  f16* c;            // [i][j]
  f16* ct;           // [j][i]
  uint16_t* out;     // final bf16 output [j][i], bounded by out_j and out_i
  int64_t out_ld;
  int32_t lda, ldb, ldc, ldct;
  int32_t kt;        // stages
  int32_t kind;
  // A symmetric product of few tiles and a long contraction is split over the
  // stages: `splits` workgroups a tile store their sums, register by register,
  // in `part`, and a second launch (join) adds them in order and finishes.
  int32_t splits;
  int32_t join;      // 0, or the tile of the split launch
  float* part;
  float alpha, beta, delta;
  int32_t side_i, side_j;   // padded lengths
  int32_t ti, tj;    // tiles on each axis
  int32_t out_i, out_j;
  int32_t per_xcd;   // tiles on one XCD
};
// CAP: products a launch can hold. Arguments of few products are 6 us a call
// cheaper than those of 24 (19 launches; 95 against 100 us of GPU time), those of 8 3 us.
template <int CAP>
struct ProdArgs {
  Prod p[CAP];
  int32_t end[CAP];             // exclusive prefix of workgroups; past the last: the largest int
  int32_t run;                  // workgroups of one XCD's run over all products, or 0
  int32_t slots;                // workgroups on one XCD
};
constexpr int kFewMats = 4, kSomeMats = 8;

// Tile t of the lower triangle of n rows, in bands of 4 rows walked by columns:
// neighbours in this order share rows of both operands.
__device__ __forceinline__ void tri_of(int t, int n, int& i, int& j) {
  int r = __builtin_amdgcn_readfirstlane(int((__builtin_amdgcn_sqrtf(8.f * float(t) + 1.f) - 1.f) * 0.5f)) & ~3;
  while (r * (r + 1) / 2 > t) r -= 4;
  while (r + 4 < n && (r + 4) * (r + 5) / 2 <= t) r += 4;
  const int h = n - r < 4 ? n - r : 4;            // the band's rows
  int in = t - r * (r + 1) / 2;
  if (in < r * h) {
    j = divide(in, h);
    i = r + in - j * h;
    return;
  }
  in -= r * h;                                    // its own triangle
  int c = 0;
  while (in >= h - c) in -= h - c++;
  i = r + c + in;
  j = r + c;
}

// Row pitch of a buffer whose rows are `length` elements: one line more, so that
// the rows a stage reads, all at the same place of their row, do not fall on the
// same channels and sets of L2 when lengths are powers of two.
__host__ __device__ __forceinline__ int64_t pitch_of(int64_t length) { return length + kPitchPad; }

// The inverse of tri_of.
__device__ __forceinline__ int tri_index(int i, int j, int n) {
  const int r = i & ~3, h = n - r < 4 ? n - r : 4, c = j - r;
  if (c < 0) return r * (r + 1) / 2 + j * h + i - r;
  return r * (r + 1) / 2 + r * h + c * h - c * (c - 1) / 2 + i - j;
}

// T x T tile by WM x WN waves, on 32 x 32 x 16 matrix instructions.
//
// LDS holds S stages (a power of two) of both operands; a stage row is 128
// bytes, 8 chunks of 16. Global loads go straight to LDS, 8 rows each: lane l of
// a load fills chunk l % 8 of row l / 8. Chunk c of row r sits at c ^ (r / 2 % 8),
// so that the fragment reads (32 rows, one chunk each), which LDS serves 16
// lanes, 256 bytes, at a time, touch each of its 64 banks once.
//
// A stage is worked off in two halves, and the fragments of the next half are
// read while the matrix instructions of this one run. The stage's one barrier
// stands between the halves: by then every wave holds the second half's
// fragments in registers, so stage k + S may be loaded over stage k, and has
// S - 1 stages' time to arrive.
//
// What bounds it, in full launches of 256 tiles (the 7B block's matrices, 11.9 to 12.5 ms, 13.2
// TFLOP in whole tiles, 1.06 to 1.11 PFLOP/s): whole rounds of tiles on the CUs, which are busy
// for 85% of a launch (2064, 2608 and 952 tiles on 256 of them), and the card's power (with zeros
// for data 10.1 ms): a stage takes 2500 cycles at 1.65 GHz, 2048 of them matrix instructions, and
// reading its fragments keeps LDS as busy. The library's fp16 products of 4096 x 4096 x 4096 and
// x 11008 reach 1.42 and 1.50 PFLOP/s. With few tiles the latency of a launch: 5 us for a 64 tile
// of 4 stages, 0.2 us for each further one (16 KB at the 64 bytes a cycle that a CU loads).
//
// Why these tiles: 256 on 8 waves (two a SIMD) hides the stage's wait for loads better than 4
// waves of 128 x 128, which read a third less LDS (7B block 13.0 ms); half lines in twice as
// many stages took 13.0 ms too.
//
// run and end0 to end6 are args.run and args.end of up to 8 products, as arguments of
// their own because only such ones can be preloaded into registers.
template <int T, int WM, int WN, int S, int CAP>
__global__ __launch_bounds__(64 * WM * WN) void k_ortho_product(int32_t run, int32_t end0, int32_t end1,
                                                                int32_t end2, int32_t end3, int32_t end4,
                                                                int32_t end5, int32_t end6, ProdArgs<CAP> args) {
  const int32_t ends[kSomeMats - 1] = {end0, end1, end2, end3, end4, end5, end6};
  constexpr int kWaves = WM * WN;
  constexpr int kLoads = 2 * T / 8;               // 1 KB loads a stage
  static_assert(kWaves % 2 == 0 && kLoads % kWaves == 0, "whole loads per wave");
  constexpr int kPer = kLoads / kWaves;
  static_assert(kPer % 2 == 0, "a wave's first load is of an even q");
  static_assert(S >= 2 && (S & (S - 1)) == 0 && (S - 1) * kPer < 64, "stages");
  constexpr int MI = T / WM / 32, NI = T / WN / 32;
  constexpr int kStage = 2 * T * kBK * 2;
  constexpr int kLds = std::max(S * kStage, T * (2 * T + 64));   // the stages, or the result
  __shared__ __attribute__((aligned(1024))) char lds[kLds];

  // Workgroup b runs on XCD b % 8, and tiles that share rows should share its L2.
  // Where all products are equally long, an XCD takes one run of the tiles of all of
  // them (two 1024 x 8192 matrices: 359 us, 369 otherwise). Otherwise it takes an eighth
  // of each product, the longest first, so that no XCD gets more long tiles than the others.
  const int xcd = blockIdx.x % 8, slot = blockIdx.x / 8;
  const int key = run ? xcd * run + slot : slot;
  int s = 0, before = 0;
#pragma unroll
  for (int q = 0; q < CAP - 1; ++q) {             // past all products: an empty one, or the last
    const int end = CAP <= kSomeMats ? ends[q] : args.end[q];
    s += key >= end;
    before = key >= end ? end : before;
  }
  s = __builtin_amdgcn_readfirstlane(s);
  // The product's arguments in one round of scalar loads: as they are needed they would
  // be fetched in four, each waiting for the one before.
  u32x16 words[2];
  static_assert(sizeof(Prod) == sizeof(words), "two loads");
  __builtin_memcpy(words, &args.p[s], sizeof(words));
  asm volatile("" : "+s"(words[0]), "+s"(words[1]));
  const Prod p = __builtin_bit_cast(Prod, words);
  int local = key - __builtin_amdgcn_readfirstlane(before) + (run ? 0 : xcd * p.per_xcd);
  int ti, tj, k0 = 0, kt = p.kt;
  const int kind = p.kind, splits = p.splits;
  int64_t part = 0;                               // this workgroup's place in p.part, in tiles
  if (kind == kSym || kind == kPoly) {
    const int tiles = p.ti * (p.ti + 1) / 2;
    if (local >= (p.join ? tiles : tiles * splits)) return;
    part = local;
    if (splits > 1 && !p.join) {
      const int z = divide(local, tiles);
      local -= z * tiles;
      k0 = divide(kt * z, splits);
      kt = divide(kt * (z + 1), splits) - k0;
    }
    tri_of(local, p.ti, ti, tj);
  } else {
    if (local >= p.ti * p.tj) return;
    tile_of(local, p.ti, p.tj, ti, tj);
  }

  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN;
  // The first half of the waves load A's rows, the other half B's.
  const bool of_b = wave >= kWaves / 2;
  const int ld = of_b ? p.ldb : p.lda;
  const f16* base = (of_b ? p.b + int64_t(tj) * T * ld : p.a + int64_t(ti) * T * ld) + k0 * kBK;
  const __amdgpu_buffer_rsrc_t r = rsrc(base, (int64_t(T) * ld - k0 * kBK) * 2);
  const int first = (wave % (kWaves / 2)) * kPer;
  // row 8 q + lane / 8: its r / 2 % 8 is lane / 16, plus 4 for odd q
  const int v0 = (lane >> 3) * ld * 2 + ((lane & 7) ^ (lane >> 4)) * 16, v1 = v0 ^ 64;

  auto load_one = [&](int k, int q) {             // 8 rows of stage k
    char* to = lds + (k & (S - 1)) * kStage + (wave * kPer + q) * 1024;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        r, (__attribute__((address_space(3))) void*)to, 16, q & 1 ? v1 : v0,
        (first + q) * 8 * ld * 2 + k * (kBK * 2), 0, 0);
  };
  auto load = [&](int k) {
#pragma unroll
    for (int q = 0; q < kPer; ++q) load_one(k, q);
  };

  constexpr int kCols = T / 8, kStep = 64 * kWaves / kCols, kSteps = T / kStep;
  const int64_t i0 = int64_t(ti) * T, j0 = int64_t(tj) * T;
  const int il = wm * (T / WM) + (lane >> 5) * 4, jl = wn * (T / WN) + (lane & 31);
  const int row0 = threadIdx.x / kCols, col = threadIdx.x % kCols * 8;   // 16 bytes a lane, kStep rows a step
  // kPoly: A's tile, in the order of its mirror image. Small tiles load it ahead of the
  // products (0.5 us a launch); the largest have no registers left for it.
  u32x4 whole[kSteps];
  auto load_whole = [&] {
    const __amdgpu_buffer_rsrc_t from = rsrc(p.a + j0 * p.lda + i0, int64_t(T) * p.lda * 2);
#pragma unroll
    for (int q = 0; q < kSteps; ++q)
      whole[q] = __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(from, (row0 * p.lda + col) * 2,
                                                                                q * kStep * p.lda * 2, 0));
  };
  if (T < 256 && kind == kPoly) load_whole();

  f32x16 acc[MI][NI];
#pragma unroll
  for (int x = 0; x < MI; ++x)
#pragma unroll
    for (int y = 0; y < NI; ++y)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[x][y][e] = 0.f;

  // A lane's fragment: row lane % 32, 8 elements at chunk 2 q + lane / 32 of the stage row.
  const int frag = (lane & 31) * 128, c0 = ((lane >> 5) ^ ((lane >> 1) & 7)) * 16;
  const int oa = wm * (T / WM) * 128 + frag, ob = (T + wn * (T / WN)) * 128 + frag;
  constexpr int kReads = 2 * (MI + NI), kMuls = 2 * MI * NI;
  constexpr int kAhead = (kReads + kMuls - 1) / kMuls;   // reads before and after each multiply
  f16x8 fa[2][2][MI], fb[2][2][NI];               // [half][q][fragment]
  auto read_one = [&](int k, int h, int n) {      // the n-th fragment of a half
    const int q = n / (MI + NI), w = n % (MI + NI);
    const char* st = lds + (k & (S - 1)) * kStage + (c0 ^ (h * 64 + q * 32));
    if (w < NI) fb[h][q][w] = *reinterpret_cast<const f16x8*>(st + ob + w * 4096);
    else fa[h][q][w - NI] = *reinterpret_cast<const f16x8*>(st + oa + (w - NI) * 4096);
  };
  // The multiplies of half h of stage k, each followed by a share of the next
  // half's fragment reads and, in the second half, of the loads of stage k + S
  // (reads and loads in this order: both are LDS accesses to the compiler).
  auto half = [&](int k, auto of, auto load_next, auto read_next) {
    static_for<kMuls>([&](auto at) {
      constexpr int h = of.value, i = at.value;
      constexpr int r0 = i ? std::min(kReads, i * kAhead + 1) : 0, r1 = std::min(kReads, (i + 1) * kAhead + 1);
      constexpr int l0 = std::min(kPer, (i * kPer * 2 + kMuls - 1) / kMuls);
      constexpr int l1 = std::min(kPer, ((i + 1) * kPer * 2 + kMuls - 1) / kMuls);
      if constexpr (read_next.value)
        static_for<r1 - r0>([&](auto z) {
          read_one(h ? k + 1 : k, 1 - h, r0 + z.value);
          __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        });
      constexpr int q = i / (MI * NI), x = i % (MI * NI) / NI, y = i % NI;
      acc[x][y] = __builtin_amdgcn_mfma_f32_32x32x16_f16(fa[h][q][x], fb[h][q][y], acc[x][y], 0, 0, 0);
      __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
      if constexpr (load_next.value)
        static_for<l1 - l0>([&](auto z) {
          load_one(k + S, l0 + z.value);
          __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);
        });
    });
    __builtin_amdgcn_sched_barrier(0);
  };
  const std::integral_constant<int, 0> lower;
  const std::integral_constant<int, 1> upper;
  using std::false_type;
  using std::true_type;

  if (!p.join) {
    if (kt >= S) {
#pragma unroll
      for (int k = 0; k < S; ++k) load(k);
      wait_loads<(S - 1) * kPer>();
    } else {
      for (int k = 0; k < kt; ++k) load(k);
      wait_loads<0>();
    }
    meet();
#pragma unroll
    for (int n = 0; n < kReads; ++n) read_one(0, 0, n);
    int k = 0;
    for (; k + S < kt; ++k) {                       // stages k + 2 to k + S - 1 may be under way
      half(k, lower, false_type{}, true_type{});
      wait_loads<(S - 2) * kPer>();
      meet();
      half(k, upper, true_type{}, true_type{});
    }
    for (; k + 1 < kt; ++k) {
      half(k, lower, false_type{}, true_type{});
      wait_loads<0>();
      meet();
      half(k, upper, false_type{}, true_type{});
    }
    half(k, lower, false_type{}, true_type{});
    wait_loads<0>();
    meet();
    half(k, upper, false_type{}, false_type{});
    if constexpr (T < 256) {
      if (splits > 1) {
        f32x4* to = reinterpret_cast<f32x4*>(p.part + part * (T * T)) + threadIdx.x;
#pragma unroll
        for (int x = 0; x < MI; ++x)
#pragma unroll
          for (int y = 0; y < NI; ++y)
#pragma unroll
            for (int g = 0; g < 4; ++g)
              to[((x * NI + y) * 4 + g) * 64 * kWaves] = f32x4{acc[x][y][4 * g], acc[x][y][4 * g + 1],
                                                               acc[x][y][4 * g + 2], acc[x][y][4 * g + 3]};
        return;
      }
    }
  } else if constexpr (T == 64) {
    // A 64 tile of the sums of a launch on 64 or 128 tiles. In the latter it is one
    // wave's share, and this workgroup's waves are that wave's four fragments.
    int64_t tile = part, tiles = int64_t(p.ti) * (p.ti + 1) / 2;
    int at = threadIdx.x;
    if (p.join == 128) {
      const int n = p.ti / 2;
      tile = tri_index(ti / 2, tj / 2, n);
      tiles = int64_t(n) * (n + 1) / 2;
      at = wave * 1024 + ((ti & 1) * 2 + (tj & 1)) * 64 + lane;
    }
    const int area = p.join * p.join;
    for (int z = 0; z < splits; ++z) {
      const f32x4* from = reinterpret_cast<const f32x4*>(p.part + (z * tiles + tile) * area) + at;
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const f32x4 q = from[g * 256];
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[0][0][4 * g + e] += q[e];
      }
    }
  }

  // The result goes through LDS, so that global memory is written in whole
  // lines, first as it lies (rows j), then turned (rows i). A lane holds 4
  // consecutive i of one j = lane % 32 at a time. LDS rows are T values and a pad
  // that spreads the 8-byte writes of a wave over all banks.
  constexpr int kRowJ = 2 * T + 16, kRowI = 2 * T + 64;
  // where there is room the turned form has a place of its own, which saves two of three barriers
  constexpr bool kApart = T * (kRowJ + kRowI) <= kLds;
  char* const lds_i = lds + (kApart ? T * kRowJ : 0);
  auto each_four = [&](auto f) {
#pragma unroll
    for (int x = 0; x < MI; ++x)
#pragma unroll
      for (int y = 0; y < NI; ++y)
#pragma unroll
        for (int g = 0; g < 4; ++g) f(x, y, g, il + x * 32 + g * 8, jl + y * 32);
  };
  const float alpha = p.alpha;
  auto scaled = [&](int x, int y, int g) {
    f32x4 v;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = acc[x][y][4 * g + e] * alpha;
    return v;
  };
  auto place = [&](int i, int j) { return reinterpret_cast<u32x2*>(lds + j * kRowJ + i * 2); };

  if (kind == kFinal) {
    each_four([&](int x, int y, int g, int i, int j) {
      const f32x4 v = scaled(x, y, g);
      *place(i, j) = u32x2{pack_bf16(v.x, v.y), pack_bf16(v.z, v.w)};
    });
    __syncthreads();
#pragma unroll
    for (int q = 0; q < kSteps; ++q) {
      const int row = row0 + q * kStep;
      if (j0 + row >= p.out_j || i0 + col >= p.out_i) continue;
      const u32x4 v = *reinterpret_cast<const u32x4*>(lds + row * kRowJ + col * 2);
      uint16_t* o = p.out + (j0 + row) * p.out_ld + i0 + col;
      if (i0 + col + 8 <= p.out_i) {
        st_loose<u32x4, 2>(o, v);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (i0 + col + e < p.out_i) o[e] = uint16_t(v[e / 2] >> (16 * (e & 1)));
      }
    }
    return;
  }

  // The step's offset is added to the lane's: with a scalar offset in the store the
  // compiler lets the next instruction overwrite the registers being stored, and
  // now and then one of them went out with its new value.
  auto store = [&](u32x4 v, __amdgpu_buffer_rsrc_t to, int ld, int q) {
    __builtin_amdgcn_raw_buffer_store_b128(v, to, ((row0 + q * kStep) * ld + col) * 2, 0, 0);
  };
  f16x4 result[MI][NI][4];
  auto keep = [&](int x, int y, int g, int i, int j, f32x4 v) {
    result[x][y][g] = f16x4{f16(v.x), f16(v.y), f16(v.z), f16(v.w)};
    *place(i, j) = __builtin_bit_cast(u32x2, result[x][y][g]);
  };
  if (kind == kPoly) {
    if (T == 256) load_whole();
#pragma unroll
    for (int q = 0; q < kSteps; ++q)
      *reinterpret_cast<u32x4*>(lds + (row0 + q * kStep) * kRowJ + col * 2) = whole[q];
    __syncthreads();
    const float beta = p.beta, delta = p.delta;
    const int diagonal = ti == tj ? 0 : T;        // i - j of the diagonal's elements in this tile
    each_four([&](int x, int y, int g, int i, int j) {
      f32x4 r = scaled(x, y, g);
      const f16x4 d = __builtin_bit_cast(f16x4, *place(i, j));
#pragma unroll
      for (int e = 0; e < 4; ++e) r[e] = r[e] + beta * float(d[e]) + (i + e - j == diagonal ? delta : 0.f);
      keep(x, y, g, i, j, r);
    });
  } else {
    each_four([&](int x, int y, int g, int i, int j) { keep(x, y, g, i, j, scaled(x, y, g)); });
  }
  // A tile on the diagonal is made exactly symmetric, like the mirrored ones: a
  // product of two matrices that commute only up to rounding is not, and later
  // products would amplify the difference (four times the error after 5 steps).
  const bool diagonal = kind != kUpdate && ti == tj;
  // Turned in registers: four lanes of consecutive j exchange their 4 x 4 values
  // (first with the neighbour, then with the lane two further), after which lane
  // l of the four holds row i + l of the four j and writes 8 bytes.
  const bool odd = lane & 1, high = lane & 2;
  const uint32_t select = odd ? 0x03020706u : 0x05040100u;
  auto turn = [&] {
    each_four([&](int x, int y, int g, int i, int j) {
      const u32x2 d = __builtin_bit_cast(u32x2, result[x][y][g]);
      const uint32_t r0 = __builtin_amdgcn_perm(__builtin_amdgcn_mov_dpp(d.x, 0xB1, 0xF, 0xF, true), d.x, select);
      const uint32_t r1 = __builtin_amdgcn_perm(__builtin_amdgcn_mov_dpp(d.y, 0xB1, 0xF, 0xF, true), d.y, select);
      const uint32_t other = __builtin_amdgcn_mov_dpp(high ? r0 : r1, 0x4E, 0xF, 0xF, true);
      *reinterpret_cast<u32x2*>(lds_i + (i + (lane & 3)) * kRowI + (j & ~3) * 2) =
          high ? u32x2{other, r1} : u32x2{r0, other};
    });
  };
  if (kApart && !diagonal) turn();
  __syncthreads();
  const __amdgpu_buffer_rsrc_t to_j = rsrc(p.ct + j0 * p.ldct + i0, int64_t(T) * p.ldct * 2);
#pragma unroll
  for (int q = 0; q < kSteps; ++q) {
    const int row = row0 + q * kStep;
    u32x4 v = *reinterpret_cast<const u32x4*>(lds + row * kRowJ + col * 2);
    if (diagonal && col < row) {
      f16x8 w = __builtin_bit_cast(f16x8, v);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (col + e < row) w[e] = *reinterpret_cast<const f16*>(lds + (col + e) * kRowJ + row * 2);
      v = __builtin_bit_cast(u32x4, w);
    }
    store(v, to_j, p.ldct, q);
  }
  if (diagonal) return;
  if (!kApart) {
    __syncthreads();
    turn();
    __syncthreads();
  }
  const __amdgpu_buffer_rsrc_t to_i = rsrc(p.c + i0 * p.ldc + j0, int64_t(T) * p.ldc * 2);
#pragma unroll
  for (int q = 0; q < kSteps; ++q)
    store(*reinterpret_cast<const u32x4*>(lds_i + (row0 + q * kStep) * kRowI + col * 2), to_i, p.ldc, q);
}

// ---------------------------------------------------------------------------
// the norm, and X_0 in both orientations
// ---------------------------------------------------------------------------

struct Source {
  const void* g;      // the caller's matrix: rows x cols, `ld` elements a row
  int64_t ld;
  int32_t rows, cols;
  f16* x;             // m x n, padded to mp x np
  f16* xt;            // n x m, padded to np x mp
  double* partial;    // sums of squares
  int32_t mp, np;
  int32_t parts;      // partial sums
  int32_t end;        // exclusive prefix of workgroups over the launch
};
struct SourceArgs {
  Source s[kMaxMats];
  int32_t ns;
  double eps;
};

// 8 consecutive elements as fp32, from element alignment.
__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const f32x4 a = ld_loose<f32x4, 4>(p), b = ld_loose<f32x4, 4>(p + 4);
#pragma unroll
  for (int e = 0; e < 4; ++e) { x[e] = a[e]; x[4 + e] = b[e]; }
}
__device__ __forceinline__ void load8(const uint16_t* p, float (&x)[8]) {
  const u32x4 q = ld_loose<u32x4, 2>(p);
#pragma unroll
  for (int e = 0; e < 4; ++e) { x[2 * e] = lo_bf16(q[e]); x[2 * e + 1] = hi_bf16(q[e]); }
}
__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const uint16_t* p) { return widen(*p); }

__device__ __forceinline__ double block_sum_256(double v, double* lds4) {
  v = wave_sum(v);
  if ((threadIdx.x & 63) == 0) lds4[threadIdx.x >> 6] = v;
  __syncthreads();
  return (lds4[0] + lds4[1]) + (lds4[2] + lds4[3]);
}

// Sums of squares in fp64 (an fp32 element's square can leave fp32's range),
// one partial a workgroup, joined in a fixed order by k_ortho_start. Bound by HBM:
// 405 MB in 84 us (4.8 TB/s).
template <typename T>
__global__ __launch_bounds__(256) void k_ortho_sumsq(SourceArgs args) {
  int s = 0;
  while (int(blockIdx.x) >= args.s[s].end) ++s;
  const Source& src = args.s[s];
  const int part = int(blockIdx.x) - (s ? args.s[s - 1].end : 0);
  const T* g = static_cast<const T*>(src.g);
  const bool flat = src.ld == src.cols;
  const int64_t total = int64_t(src.rows) * src.cols;
  const int64_t len = flat ? kSumRow : src.cols, ld = flat ? kSumRow : src.ld;
  const int64_t rows = flat ? (total + kSumRow - 1) / kSumRow : src.rows;
  double sum = 0.0;
  for (int64_t r = part; r < rows; r += src.parts) {
    const T* row = g + r * ld;
    const int64_t n = flat && total - r * len < len ? total - r * len : len;
    int64_t c = int64_t(threadIdx.x) * 8;
    for (; c + 3 * 2048 + 8 <= n; c += 4 * 2048) {          // four loads under way
      float x[4][8];
#pragma unroll
      for (int u = 0; u < 4; ++u) load8(row + c + u * 2048, x[u]);
#pragma unroll
      for (int u = 0; u < 4; ++u)
#pragma unroll
        for (int e = 0; e < 8; ++e) sum += double(x[u][e]) * double(x[u][e]);
    }
    for (; c < n; c += 2048) {
      if (c + 8 <= n) {
        float x[8];
        load8(row + c, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum += double(x[e]) * double(x[e]);
      } else {
        for (int64_t e = c; e < n; ++e) sum += double(load1(row + e)) * double(load1(row + e));
      }
    }
  }
  __shared__ double lds4[4];
  sum = block_sum_256(sum, lds4);
  if (threadIdx.x == 0) src.partial[part] = sum;
}

// X_0 from a 64 x 64 block of G: scaled, rounded to fp16, written as it lies
// and transposed; what lies past G's edge is zero. Bound by HBM: 405 MB of bf16 into
// 810 MB in 216 us (5.6 TB/s).
template <typename T>
__global__ __launch_bounds__(256) void k_ortho_start(SourceArgs args) {
  int s = 0;
  while (int(blockIdx.x) >= args.s[s].end) ++s;
  const Source& src = args.s[s];
  const int local = int(blockIdx.x) - (s ? args.s[s - 1].end : 0);
  __shared__ double lds4[4];
  __shared__ f16 tile[64][64 + 8];
  const double sq = block_sum_256(int(threadIdx.x) < src.parts ? src.partial[threadIdx.x] : 0.0, lds4);
  // The scale as mantissa and exponent: it passes fp32's range where norm + eps is below
  // 2^-116, and is subnormal far above 2^127. Where both are 0 it is infinite and X NaN.
  const double norm = sqrt(sq) + args.eps;
  double scale = kScaleX / norm;
  if (norm > 0.0 && scale > 0x1p1000) scale = 0x1p1000;      // zeros only, and an eps below 2^-988
  const float mantissa = float(__builtin_amdgcn_frexp_mant(scale));
  const int exponent = __builtin_amdgcn_frexp_exp(scale);

  const bool tall = src.rows > src.cols;
  const int pr = tall ? src.np : src.mp, pc = tall ? src.mp : src.np;   // G's padded sides
  f16* as_is = tall ? src.xt : src.x;
  f16* turned = tall ? src.x : src.xt;
  const int bc = pc / 64, r0 = local / bc * 64, c0 = local % bc * 64;
  const T* g = static_cast<const T*>(src.g);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int r = (threadIdx.x >> 3) + 32 * k, c = (threadIdx.x & 7) * 8;
    float x[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (r0 + r < src.rows) {
      const T* p = g + int64_t(r0 + r) * src.ld + c0 + c;
      if (c0 + c + 8 <= src.cols) {
        load8(p, x);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (c0 + c + e < src.cols) x[e] = load1(p + e);
      }
    }
    f16x8 q;
#pragma unroll
    for (int e = 0; e < 8; ++e) q[e] = f16(__builtin_amdgcn_ldexpf(x[e], exponent) * mantissa);
    *reinterpret_cast<f16x8*>(as_is + int64_t(r0 + r) * pitch_of(pc) + c0 + c) = q;
    *reinterpret_cast<f16x8*>(&tile[r][c]) = q;
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int r = (threadIdx.x >> 3) + 32 * k, c = (threadIdx.x & 7) * 8;
    f16x8 q;
#pragma unroll
    for (int e = 0; e < 8; ++e) q[e] = tile[c + e][r];
    *reinterpret_cast<f16x8*>(turned + int64_t(c0 + r) * pitch_of(pr) + r0 + c) = q;
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------

struct Plan {
  int32_t rows, cols, m, n;   // m <= n
  int64_t mp, np;             // padded
  int64_t x, xt0, xt1, sym0, sym1, sym2, partial;   // workspace offsets
  int32_t parts;
  bool pairs;
};

int64_t round_up(int64_t x, int64_t to) { return (x + to - 1) / to * to; }

// What a call's matrices are padded to: the largest tile that grows no side's
// share of the work much. Every launch then takes that tile or a smaller one.
int choose_pad(int32_t count, const int64_t* rows, const int64_t* cols) {
  double least = 0;
  int best = 64;
  for (int t : {64, 128, 256}) {
    double work = 0;
    for (int32_t i = 0; i < count; ++i) {
      const double m = double(round_up(std::min(rows[i], cols[i]), t)), n = double(round_up(std::max(rows[i], cols[i]), t));
      work += 3 * m * m * n + m * m * m;
    }
    work *= t == 256 ? 1.0 : t == 128 ? 1.2 : 1.6;       // measured at full size
    if (t == 64 || work <= least) {
      best = t;
      least = work;
    }
  }
  return best;
}

// Whether a matrix takes its steps in pairs (see the head of this file): the
// products of a pair cost 3 m^2 n + 5 m^3 multiply-adds against 6 m^2 n + 2 m^3
// and one launch more, so they pay from some n / m above 1 on. Nearly square
// matrices, whose least singular values are tiny, also lose more that way
// (2.9e-3 against 2.3e-3 after 5 steps at n = m; alike from n = 1.25 m on).
bool may_pair(int64_t m, int64_t n, int64_t mp, int64_t np) { return 4 * n >= 5 * m && 4 * np >= 5 * mp; }
// For short matrices the launch weighs more. Measured in us, pairs and single steps:
// 128 x 512 80 and 73, 256 x 1024 twice 90 and 87, 512 x 1536 alike, 512 x 2048 116 and
// 120, 1024 x 2048 155 and 152, 1024 x 3000 175 and 181, 2048 x 4096 475 and 496. The
// matrices of a call do alike, since their n-th products share a launch: pairs where one
// of them gains (of 515 x 1373, 2049 x 771 and a square the first in single steps 204, both in pairs 195).
bool gains_by_pairs(int64_t mp, int64_t np) { return np >= mp + 1152; }

constexpr int64_t kMaxSide = int64_t(1) << 20;

fsdp_status check_shapes(int32_t count, const int64_t* rows, const int64_t* cols) {
  if (count < 0 || count > FSDP_MAX_TENSORS)
    return fail(FSDP_ERR_INVALID_ARG, "n_mats must be in [0, %d] (got %d)", FSDP_MAX_TENSORS, count);
  if (count > 0 && (!rows || !cols)) return fail(FSDP_ERR_INVALID_ARG, "rows or cols is NULL");
  for (int32_t i = 0; i < count; ++i) {
    if (rows[i] < 0 || cols[i] < 0)
      return fail(FSDP_ERR_INVALID_ARG, "matrix %d: negative size", i);
    if (rows[i] > kMaxSide || cols[i] > kMaxSide)
      return fail(FSDP_ERR_RANGE, "matrix %d: %lld x %lld is over %lld a side", i,
                  static_cast<long long>(rows[i]), static_cast<long long>(cols[i]),
                  static_cast<long long>(kMaxSide));
  }
  return FSDP_OK;
}

constexpr int kSplitSlots = 256;          // workgroups of a split launch, at most
constexpr int kSplitStages = 8;           // stages of a split, at least

// Lays the buffers of every matrix that has elements out in the workspace; *part
// is where the sums of split launches go, or -1 if the call's S = X X^T have
// enough tiles, or stages too few, to be split.
int64_t make_plan(int32_t count, const int64_t* rows, const int64_t* cols, int pad,
                  std::vector<Plan>* plans, int64_t* part) {
  int64_t at = 0, tiles = 0, longest = 0;
  const int tile = std::min(pad, 128);
  bool gain = false;
  for (int32_t i = 0; i < count; ++i) {
    const int64_t m = std::min(rows[i], cols[i]), n = std::max(rows[i], cols[i]);
    const int64_t mp = round_up(m, pad), np = round_up(n, pad);
    gain = gain || (m > 0 && may_pair(m, n, mp, np) && gains_by_pairs(mp, np));
  }
  auto take = [&](int64_t bytes) {
    const int64_t here = at;
    at += round_up(bytes, 1024);
    return here;
  };
  for (int32_t i = 0; i < count; ++i) {
    Plan q{};
    q.rows = int32_t(rows[i]);
    q.cols = int32_t(cols[i]);
    q.m = std::min(q.rows, q.cols);
    q.n = std::max(q.rows, q.cols);
    if (q.m > 0) {
      q.mp = round_up(q.m, pad);
      q.np = round_up(q.n, pad);
      q.x = take(q.mp * pitch_of(q.np) * 2);
      q.xt0 = take(q.np * pitch_of(q.mp) * 2);
      q.xt1 = take(q.np * pitch_of(q.mp) * 2);
      q.sym0 = take(q.mp * pitch_of(q.mp) * 2);
      q.sym1 = take(q.mp * pitch_of(q.mp) * 2);
      q.pairs = gain && may_pair(q.m, q.n, q.mp, q.np);
      q.sym2 = q.pairs ? take(q.mp * pitch_of(q.mp) * 2) : 0;
      q.parts = int32_t(std::min<int64_t>(kSumBlocks, (int64_t(q.m) * q.n + kSumRow - 1) / kSumRow));
      q.partial = take(q.parts * 8);
      const int64_t side = q.mp / tile;
      tiles += side * (side + 1) / 2;
      longest = std::max(longest, q.np / kBK);
    }
    if (plans) plans->push_back(q);
  }
  const bool split = tiles > 0 && 2 * tiles <= kSplitSlots && longest >= 2 * kSplitStages;
  *part = split ? take(int64_t(kSplitSlots) * tile * tile * 4) : -1;
  return at;
}

// Workgroups of a product on tiles of t.
int64_t tiles_of(const Prod& p, int t) {
  const int64_t i = p.side_i / t, j = p.side_j / t;
  return p.kind == kSym || p.kind == kPoly ? i * (i + 1) / 2 : i * j;
}

// How a launch is run: its tile, and whether its products' stages are split over
// several workgroups a tile (joined by a second launch): what takes the least
// estimated time. A launch takes at least the time of its longest tile, and at
// least the work of all tiles over the 256 CUs, in whole rounds. Measured, in
// units of 1.1 us: a tile of kt stages on a CU of its own takes 16 + 0.9 kt, 6 +
// 0.5 kt or 2 + 0.2 kt (tiles of 256, 128, 64; 5 + 0.42 kt with the deeper
// pipeline of launches of at most one 128 tile a CU), and a CU among many busy ones gets through one in
// 14 + 1.4 kt, 3 + 0.45 kt or 0.9 + 0.18 kt. A join takes 5.
struct Shape {
  int tile;
  bool split;
};
int splits_of(const Prod& p, int64_t all_tiles) {
  return int(std::max<int64_t>(1, std::min<int64_t>(kSplitSlots / all_tiles, p.kt / kSplitStages)));
}
Shape launch_shape(const std::vector<const Prod*>& now, int pad, bool may_split) {
  Shape best{pad, false};
  double least = 0;
  for (int t = pad; t >= 64; t /= 2) {
    int64_t tiles = 0;
    bool sym = true;
    for (const Prod* p : now) {
      tiles += tiles_of(*p, t);
      sym = sym && p->kind == kSym;
    }
    for (int split = 0; split <= (may_split && sym && t < 256 && 2 * tiles <= kSplitSlots); ++split) {
      double work = 0, longest = 0;
      int64_t groups = 0;
      for (const Prod* p : now) {
        const int z = split ? splits_of(*p, tiles) : 1;
        const double kt = double(p->kt) / z, n = double(tiles_of(*p, t)) * z;
        work += n * (t == 256 ? 14 + 1.4 * kt : t == 128 ? 3 + 0.45 * kt : 0.9 + 0.18 * kt);
        longest = std::max(longest, t == 256              ? 16 + 0.9 * kt
                                    : t == 128 && tiles <= 256 ? 5 + 0.42 * kt
                                    : t == 128            ? 6 + 0.5 * kt
                                                          : 2 + 0.2 * kt);
        groups += tiles_of(*p, t) * z;
      }
      const double time = std::max(longest, work / groups * double((groups + 255) / 256)) + (split ? 5 : 0);
      if ((t == pad && !split) || time < least) {
        best = Shape{t, split != 0};
        least = time;
      }
    }
  }
  return best;
}

// One launch of a shape's: the products, or (join) the sums of a split one.
template <int CAP>
void launch_products(const std::vector<const Prod*>& now, Shape shape, bool join, float* part,
                     hipStream_t stream) {
  ProdArgs<CAP> a{};
  std::fill(a.end, a.end + CAP, INT32_MAX);
  int64_t all_tiles = 0;
  for (const Prod* p : now) all_tiles += tiles_of(*p, shape.tile);
  const int tile = join ? 64 : shape.tile;
  // 256 tiles keep a share of each product an XCD (the 7B block, both in turn: 12.05 ms, 12.42 in runs)
  bool even = tile < 256;
  for (const Prod* p : now) even = even && p->kt == now[0]->kt;
  int n = 0, groups = 0;
  for (const Prod* p : now) {
    Prod& to = a.p[n] = *p;
    to.ti = p->side_i / tile;
    to.tj = p->side_j / tile;
    to.splits = shape.split ? splits_of(*p, all_tiles) : 1;
    to.join = join ? shape.tile : 0;
    to.part = part;
    part += tiles_of(*p, shape.tile) * to.splits * shape.tile * shape.tile;
    if (join && to.splits == 1) {                 // too short to be split: the first launch finished it
      to = Prod{};
      continue;
    }
    const int count = int(tiles_of(*p, tile) * (join ? 1 : to.splits));
    groups += count;
    to.per_xcd = (count + 7) / 8;
    a.slots += to.per_xcd;
    a.end[n++] = even ? groups : a.slots;
  }
  if (even) a.run = a.slots = (groups + 7) / 8;
  const int blocks = 8 * a.slots;
  int32_t e[kSomeMats - 1];
  std::fill(e, e + kSomeMats - 1, INT32_MAX);
  std::copy(a.end, a.end + std::min(CAP, kSomeMats - 1), e);
  auto go = [&](auto kernel, int threads) {
    kernel<<<blocks, threads, 0, stream>>>(a.run, e[0], e[1], e[2], e[3], e[4], e[5], e[6], a);
  };
  if (tile == 256) go(k_ortho_product<256, 2, 4, 2, CAP>, 512);
  else if (tile == 128 && groups <= 256) go(k_ortho_product<128, 2, 2, 4, CAP>, 256);
  else if (tile == 128) go(k_ortho_product<128, 2, 2, 2, CAP>, 256);
  else go(k_ortho_product<64, 2, 2, 4, CAP>, 256);
}

fsdp_status launch(const std::vector<const Prod*>& now, int pad, float* part, hipStream_t stream) {
  const Shape shape = launch_shape(now, pad, part != nullptr);
  for (int join = 0; join <= int(shape.split); ++join) {
    if (now.size() <= kFewMats) launch_products<kFewMats>(now, shape, join != 0, part, stream);
    else if (now.size() <= kSomeMats) launch_products<kSomeMats>(now, shape, join != 0, part, stream);
    else launch_products<kMaxMats>(now, shape, join != 0, part, stream);
    if (fsdp_status st = fsdp::after_launch("fsdp_orthogonalize")) return st;
  }
  return FSDP_OK;
}

// What the coefficients let a step's matrices reach. A singular value x of X becomes
// x p(x^2), p(s) = a + b s + c s^2, and starts at 1 or less; with S's eigenvalues
// s = x^2 in [0, top^2] nothing in S, p(S) or X passes the largest value of s, |p(s)| or
// |x p(x^2)| there, which lie at an end or where a derivative is zero. Past kMostX and
// kMostS the bounds end: the scales would push ordinary values below fp16's range.
constexpr double kMostX = 1024, kMostS = 1 << 20;
struct Reach {
  const double* k;
  double p(double s) const { return std::fabs(k[0] + s * (k[1] + s * k[2])); }
  template <typename F>
  static double most(std::initializer_list<double> at, double end, double cap, F&& f) {
    double m = f(end);
    for (double s : at)
      if (s >= 0 && s < end) m = std::max(m, f(s));
    return m < cap ? m : cap;         // the cap for NaN too
  }
  double poly(double top) const {
    return most({0.0, -k[1] / (2 * k[2])}, top * top, kMostS, [&](double s) { return p(s); });
  }
  // and 1% for the roundings of X and S
  double step(double top) const {
    const double b = 3 * k[1], c = 5 * k[2];        // a + b s + c s^2 = 0
    const double q = -0.5 * (b + std::copysign(std::sqrt(b * b - 4 * k[0] * c), b));
    return most({q / c, k[0] / q}, top * top, kMostX, [&](double s) { return 1.01 * std::sqrt(s) * p(s); });
  }
};
// The power of two for values up to `most`: the usual one where it leaves an eighth of fp16's range.
double scale_for(double most, double usual) {
  while (most * usual > 57344) usual /= 2;
  return usual;
}

// The products of one matrix, in order; the n-th of every matrix go into one launch.
void list_products(const Plan& q, char* ws, int steps, const double* coeffs,
                   void* out, int64_t out_ld, std::vector<Prod>* list) {
  struct Sym {                                  // a symmetric matrix and its scale
    f16* at;
    double scale;
  };
  auto at = [&](int64_t offset) { return reinterpret_cast<f16*>(ws + offset); };
  f16 *x = at(q.x), *xt = at(q.xt0), *xt_next = at(q.xt1);
  f16 *s0 = at(q.sym0), *s1 = at(q.sym1), *s2 = at(q.sym2);
  auto add = [&](Kind kind, const f16* a, const f16* b, int64_t length, double alpha) -> Prod& {
    list->emplace_back();
    Prod& p = list->back();
    p = Prod{};
    p.kind = kind;
    p.a = a;
    p.b = b;
    p.lda = p.ldb = int32_t(pitch_of(length));
    p.kt = int32_t(length / kBK);
    p.alpha = float(alpha);
    p.side_i = p.side_j = int32_t(q.mp);
    return p;
  };
  auto symmetric = [&](Kind kind, const f16* a, const f16* b, f16* to, int64_t length, double alpha) -> Prod& {
    Prod& p = add(kind, a, b, length, alpha);
    p.c = p.ct = to;
    p.ldc = p.ldct = int32_t(pitch_of(q.mp));
    return p;
  };
  auto poly = [&](Sym s, f16* to, double most) {
    const double scale = scale_for(most, kScaleS);
    Prod& p = symmetric(kPoly, s.at, s.at, to, q.mp, coeffs[2] * scale / (s.scale * s.scale));
    p.beta = float(coeffs[1] * scale / s.scale);
    p.delta = float(coeffs[0] * scale);
    return Sym{to, scale};
  };
  auto multiply = [&](Sym a, Sym b, f16* to, double most) {
    const double scale = scale_for(most, kScaleS);
    symmetric(kSym, a.at, b.at, to, q.mp, scale / (a.scale * b.scale));
    return Sym{to, scale};
  };
  const Reach reach{coeffs};
  double top = 1, scale = kScaleX;              // of X
  for (int step = 0, group = 0; step < steps; ++group) {
    const int n = q.pairs && group % 2 == 0 && step + 2 <= steps ? 2 : 1;
    step += n;
    const Sym s = {s0, scale_for(top * top, kScaleS)};
    symmetric(kSym, x, x, s0, q.np, s.scale / (scale * scale));
    double most = reach.poly(top), next = reach.step(top);
    Sym p = poly(s, s1, most);                  // P_1
    if (n == 2) {
      const Sym ps = multiply(p, s, s2, top * next);        // P_1 S_1
      const Sym second = multiply(p, ps, s0, next * next);  // S_2 = P_1 P_1 S_1
      const double most2 = reach.poly(next);
      const Sym p2 = poly(second, s2, most2);               // P_2
      p = multiply(p2, p, s0, std::min(most * most2, kMostS));   // P_2 P_1
      next = reach.step(next);
    }
    top = next;
    const bool last = step == steps;
    const double next_scale = last ? 1.0 : scale_for(top, kScaleX);
    Prod& u = add(last ? kFinal : kUpdate, xt, p.at, q.mp, next_scale / (p.scale * scale));
    scale = next_scale;
    u.side_i = int32_t(q.np);
    u.out_i = q.n;
    u.out_j = q.m;
    if (!last) {
      u.c = xt_next;
      u.ldc = int32_t(pitch_of(q.mp));
      u.ct = x;
      u.ldct = int32_t(pitch_of(q.np));
      std::swap(xt, xt_next);
    } else {
      u.out = static_cast<uint16_t*>(out);
      u.out_ld = out_ld;
      if (q.rows > q.cols) {                    // the output's rows are X^T's
        std::swap(u.a, u.b);
        std::swap(u.side_i, u.side_j);
        std::swap(u.out_i, u.out_j);
      }
    }
  }
}

template <typename T>
fsdp_status run(const std::vector<Plan>& plans, const void* const* mats, const int64_t* mat_ld,
                void* const* outs, const int64_t* out_ld, char* ws, float* part, int pad,
                int steps, const double* coeffs, double eps, hipStream_t stream) {
  const char* what = "fsdp_orthogonalize";
  std::vector<int> live;
  for (size_t i = 0; i < plans.size(); ++i)
    if (plans[i].m > 0) live.push_back(int(i));
  for (size_t b = 0; b < live.size(); b += kMaxMats) {
    const int nb = int(std::min<size_t>(kMaxMats, live.size() - b));
    SourceArgs src{};
    src.ns = nb;
    src.eps = eps;
    int blocks = 0;
    for (int k = 0; k < nb; ++k) {
      const int i = live[b + k];
      const Plan& q = plans[i];
      Source& d = src.s[k];
      d.g = mats[i];
      d.ld = mat_ld[i];
      d.rows = q.rows;
      d.cols = q.cols;
      d.x = reinterpret_cast<f16*>(ws + q.x);
      d.xt = reinterpret_cast<f16*>(ws + q.xt0);
      d.partial = reinterpret_cast<double*>(ws + q.partial);
      d.mp = int32_t(q.mp);
      d.np = int32_t(q.np);
      d.parts = q.parts;
      blocks += q.parts;
      d.end = blocks;
    }
    k_ortho_sumsq<T><<<blocks, 256, 0, stream>>>(src);
    if (fsdp_status st = fsdp::after_launch(what)) return st;
    blocks = 0;
    for (int k = 0; k < nb; ++k) {
      blocks += int(plans[live[b + k]].mp / 64 * (plans[live[b + k]].np / 64));
      src.s[k].end = blocks;
    }
    k_ortho_start<T><<<blocks, 256, 0, stream>>>(src);
    if (fsdp_status st = fsdp::after_launch(what)) return st;

    std::vector<std::vector<Prod>> lists(nb);
    size_t longest = 0;
    for (int k = 0; k < nb; ++k) {
      const int i = live[b + k];
      list_products(plans[i], ws, steps, coeffs, outs[i], out_ld[i], &lists[k]);
      longest = std::max(longest, lists[k].size());
    }
    for (size_t n = 0; n < longest; ++n) {
      std::vector<const Prod*> now;
      for (const std::vector<Prod>& list : lists)
        if (n < list.size()) now.push_back(&list[n]);
      std::stable_sort(now.begin(), now.end(), [](const Prod* a, const Prod* b) { return a->kt > b->kt; });
      if (fsdp_status st = launch(now, pad, part, stream)) return st;
    }
  }
  return FSDP_OK;
}

fsdp_status orthogonalize(int32_t count, fsdp_dtype dtype, const void* const* mats,
                          const int64_t* rows, const int64_t* cols, const int64_t* mat_ld,
                          void* const* outs, const int64_t* out_ld, void* workspace,
                          int64_t workspace_bytes, int32_t steps, const double* coeffs, double eps,
                          hipStream_t stream) {
  const char* what = "fsdp_orthogonalize";
  if (fsdp_status st = check_shapes(count, rows, cols)) return st;
  if (dtype != FSDP_F32 && dtype != FSDP_BF16)
    return fail(FSDP_ERR_UNSUPPORTED, "dtype %d not supported", static_cast<int>(dtype));
  if (steps < 1 || steps > 64)
    return fail(FSDP_ERR_INVALID_ARG, "steps must be in [1, 64] (got %d)", steps);
  if (!coeffs) return fail(FSDP_ERR_INVALID_ARG, "coeffs is NULL");
  for (int k = 0; k < 3; ++k)
    if (!std::isfinite(coeffs[k])) return fail(FSDP_ERR_INVALID_ARG, "coeffs must be finite");
  if (!std::isfinite(eps) || !(eps >= 0.0))
    return fail(FSDP_ERR_INVALID_ARG, "eps must be finite and >= 0");
  if (count == 0) return FSDP_OK;
  const int64_t es = dtype == FSDP_F32 ? 4 : 2;
  const int pad = choose_pad(count, rows, cols);
  std::vector<Plan> plans;
  int64_t part_at = -1;
  const int64_t need = make_plan(count, rows, cols, pad, &plans, &part_at);
  if (need == 0) return FSDP_OK;               // only empty matrices
  if (!mats || !mat_ld || !outs || !out_ld)
    return fail(FSDP_ERR_INVALID_ARG, "a matrix array is NULL");
  std::vector<fsdp::ByteRange> ranges;
  for (int32_t i = 0; i < count; ++i) {
    if (plans[i].m == 0) continue;
    if (!mats[i] || !outs[i]) return fail(FSDP_ERR_INVALID_ARG, "%s[%d] is NULL", mats[i] ? "outs" : "mats", i);
    if (reinterpret_cast<uintptr_t>(mats[i]) % es)
      return fail(FSDP_ERR_INVALID_ARG, "mats[%d] is not element aligned", i);
    if (reinterpret_cast<uintptr_t>(outs[i]) % 2)
      return fail(FSDP_ERR_INVALID_ARG, "outs[%d] is not 2-byte aligned", i);
    if (mat_ld[i] < cols[i] || out_ld[i] < cols[i])
      return fail(FSDP_ERR_RANGE, "matrix %d: a row pitch is below its %lld columns", i,
                  static_cast<long long>(cols[i]));
    if (mat_ld[i] > (int64_t(1) << 40) || out_ld[i] > (int64_t(1) << 40))
      return fail(FSDP_ERR_RANGE, "matrix %d: row pitch too large", i);
    ranges.push_back(fsdp::range_of(mats[i], (rows[i] - 1) * mat_ld[i] + cols[i], es, false, "mats", i));
    ranges.push_back(fsdp::range_of(outs[i], (rows[i] - 1) * out_ld[i] + cols[i], 2, true, "outs", i));
  }
  if (fsdp_status st = fsdp::check_ptr(workspace, "workspace", 256)) return st;
  if (workspace_bytes < need)
    return fail(FSDP_ERR_RANGE, "workspace has %lld bytes, needs %lld",
                static_cast<long long>(workspace_bytes), static_cast<long long>(need));
  ranges.push_back(fsdp::range_of(workspace, need, 1, true, "workspace"));
  if (fsdp_status st = fsdp::check_alias(ranges)) return st;
  if (fsdp_status st = fsdp::check_no_pending_error(what)) return st;
  char* ws = static_cast<char*>(workspace);
  float* part = part_at >= 0 ? reinterpret_cast<float*>(ws + part_at) : nullptr;
  if (dtype == FSDP_F32)
    return run<float>(plans, mats, mat_ld, outs, out_ld, ws, part, pad, steps, coeffs, eps, stream);
  return run<uint16_t>(plans, mats, mat_ld, outs, out_ld, ws, part, pad, steps, coeffs, eps, stream);
}

}  // namespace

extern "C" {

fsdp_status fsdp_orthogonalize_workspace(int32_t n_mats, const int64_t* rows, const int64_t* cols,
                                         int64_t* bytes) {
  fsdp::clear_error();
  if (!bytes) return fail(FSDP_ERR_INVALID_ARG, "bytes pointer is NULL");
  if (fsdp_status st = check_shapes(n_mats, rows, cols)) return st;
  int64_t part_at = -1;
  *bytes = make_plan(n_mats, rows, cols, choose_pad(n_mats, rows, cols), nullptr, &part_at);
  return FSDP_OK;
}

fsdp_status fsdp_orthogonalize(int32_t n_mats, fsdp_dtype dtype, const void* const* mats,
                               const int64_t* rows, const int64_t* cols, const int64_t* mat_ld,
                               void* const* outs, const int64_t* out_ld, void* workspace,
                               int64_t workspace_bytes, int32_t steps, const double* coeffs,
                               double eps, hipStream_t stream) {
  fsdp::clear_error();
  try {
    return orthogonalize(n_mats, dtype, mats, rows, cols, mat_ld, outs, out_ld, workspace,
                         workspace_bytes, steps, coeffs, eps, stream);
  } catch (const std::bad_alloc&) {
    return fail(FSDP_ERR_INVALID_ARG, "out of host memory");
  }
}

}  // extern "C"

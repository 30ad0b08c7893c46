// loss_kernels.hip -- softmax cross entropy over a large vocabulary from the
// hidden states x (T x H) and the projection's weights w (V x H), both bf16:
//   logits = x w^T (fp32, never stored);  lse = log sum exp logits;
//   loss = lse - logits[target]  (0 where the target is negative)
// and its gradients, with g = (exp(logits - lse) - onehot(target)) dloss:
//   dx = g w,   dw = g^T x.
//
// Forward: tiles of logits are formed in registers; each wave reduces its
// columns of a row (128 of them in a 256 x 256 tile) to a maximum and a sum of
// exponentials, and a second kernel joins those of a row.  V / 128 pairs a row
// are 1/32 of what bf16 logits would take.
//
// Backward: rows that do not count are left out first (x's other rows are
// copied together), so they cost nothing and whatever they hold (a NaN in
// padding) reaches no sum.  Then, for a piece of the vocabulary at a time, the
// logits are formed again, g of the piece is stored as bf16, and two products
// read it: dw of the piece, complete, and the piece's share of dx, added up
// in fp32.  g is the one quantity rounded to bf16 in between: the matrix
// instructions take bf16 pairs, and g in two bf16 parts would take both
// products twice.  That adds one rounding, independent from entry to entry, to
// the outputs' own: the gradients' error against 64 bits is 0.0022 to 0.0023 of
// their norm, the outputs' rounding alone 0.0017 (1001 tokens x 32001 entries x
// 2000).  g is divided by the significand of the largest |dloss|, and the
// products are multiplied by it in fp32: where dloss is the same in every row,
// as for a mean, the one-hot part is then a power of two, and what is rounded is
// the sum of it and the target's probability: 0.0017 where that is small (random
// targets), 0.0018 with targets drawn from the model's own probabilities, 0.0020
// where those are 0.13 on average.
//
// The tiles are 256 x 256 with the GEMM's K loop, or 128 or 64 rows and columns
// (midtile.hpp) where those are too few or too large; in the backward pass
// the small tiles' two products share a launch and K is split.  Very few
// logits with much K take 16 x 32 tiles whose waves split K.
//
// Bound: the matrix instructions (one product forward, three backward), or
// for small ones launches and latency, or with few tokens reading the weights.
// Measured: 4096 tokens x 131072 entries x 4096 forward 3.46 ms (1.27
// PFLOP/s), 8192 tokens forward and backward 26 ms (four products, a tenth of
// the backward pass's rows left out: 1.25 PFLOP/s); 100 x 50000 x 1000 forward
// 37 us, of which the tiles take 24 (4.2 TB/s of weights), the join 6.
#include <hip/hip_runtime.h>

#include <math.h>

#include <type_traits>

#include "../kernel/epilogue.hpp"
#include "../kernel/gfx950.hpp"
#include "../kernel/mainloop.hpp"
#include "../kernel/params.hpp"
#include "../kernel/scheduler.hpp"
#include "midtile.hpp"
#include "operators.h"
#include "tile_store.hpp"

namespace migemm {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

// exp(v - m) for v <= m.  The difference is formed first: the product's
// rounding is then relative to it, not to v.
__device__ __forceinline__ float exp_diff(float v, float m) {
  return __builtin_amdgcn_exp2f((v - m) * kLog2e);
}
// What exponents are taken against: the maximum where it is finite, else 0
// (an infinite maximum then gives a sum of 0 or infinity, not a NaN).
__device__ __forceinline__ float reference_of(float m) { return fabsf(m) == INFINITY ? 0.0f : m; }

// The lane and wave as values the compiler cannot see through: per-lane
// offsets are formed per tile instead of being held across the tile loop.
struct Ids {
  int lane, wave;
  __device__ __forceinline__ Ids(int l, int w) : lane(l), wave(w) {
    asm volatile("" : "+v"(lane));
    asm volatile("" : "+s"(wave));
  }
};

// ------------------------------------------------------------------- forward

// The wave's 32 BM x 32 BN logits of rows m0.., columns n0..: per row the
// largest and the sum of exponentials against it, over the columns below V;
// and the target's logit where it is among them.
template <int BM, int BN>
__device__ __forceinline__ void reduce_logits(f32x16 (&v)[BM][BN], const LossArgs& s, int64_t m0, int64_t n0,
                                              int lane) {
  constexpr int kCols = 32 * BN;
  const int64_t T = s.gemm.M, V = s.gemm.N;
  const int lr = lane & 31, half = lane >> 5;
  if (n0 >= V) return;
  const int left = V - n0 < kCols ? (int)(V - n0) : kCols;
  float2* part = s.parts + (n0 / kCols) * s.part_rows;
  int want[BM];  // the target's column here, or -1
#pragma unroll
  for (int bi = 0; bi < BM; ++bi) {
    const int64_t row = m0 + 32 * bi + lr;
    const int64_t at = row < T ? s.target[row] - n0 : -1;
    want[bi] = at >= 0 && at < left ? (int)at : -1;
  }
#pragma unroll
  for (int bi = 0; bi < BM; ++bi) {
    const int64_t row = m0 + 32 * bi + lr;
    // (Block after block, and nothing shared between them: the accumulators
    // leave few registers.)
    sched_fence();
    int first = 4 * half;  // the lane's columns are first + 32 bj + 8 q + c
    asm volatile("" : "+v"(first));
    if (left < kCols) {
#pragma unroll
      for (int bj = 0; bj < BN; ++bj)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          v[bi][bj][i] = first + 32 * bj + 8 * (i >> 2) + (i & 3) < left ? v[bi][bj][i] : -INFINITY;
    }
    float m = v[bi][0][0];
#pragma unroll
    for (int bj = 0; bj < BN; ++bj)
#pragma unroll
      for (int i = 0; i < 16; ++i) m = fmaxf(m, v[bi][bj][i]);
    m = fmaxf(m, __shfl_xor(m, 32, 64));
    const float ref = reference_of(m);
    float sum = 0.0f;
#pragma unroll
    for (int bj = 0; bj < BN; ++bj)
#pragma unroll
      for (int i = 0; i < 16; ++i) sum += exp_diff(v[bi][bj][i], ref);
    sum += __shfl_xor(sum, 32, 64);
    if (row < T && half == 0) part[row] = {m, sum};
    // (A row's target lies in one window of the vocabulary: the search is rare.)
    if (__ballot(want[bi] >= 0) != 0) {
      const int at = want[bi] - 4 * half;  // of the lane's columns, 32 bj + 8 q + c
      float found = 0.0f;
#pragma unroll
      for (int bj = 0; bj < BN; ++bj)
#pragma unroll
        for (int i = 0; i < 16; ++i) found = 32 * bj + 8 * (i >> 2) + (i & 3) == at ? v[bi][bj][i] : found;
      if (want[bi] >= 0 && (want[bi] & 4) == 4 * half) s.target_logit[row] = found;
    }
  }
}

__global__ __launch_bounds__(kThreads, 1) void loss_forward_tiles(LossArgs s) {
  const int lane = threadIdx.x & 63, wave = wave_id();
  const KernelArgs& a = s.gemm;
  Accum acc;
  NoSideWork none;
  for (int L = persistent_slot(blockIdx.x, gridDim.x); L < a.num_tiles; L += gridDim.x) {
    const TileCoord t = tile_of(L, a);
    const Ids id(lane, wave);
    mainloop<2, true, true>(acc, a, t.tm, t.tn, id.wave, id.lane, none);
    const Ids ie(lane, wave);
    reduce_logits(acc.v, s, (int64_t)t.tm * kTileM + (ie.wave >> 1) * kWaveTile,
                  (int64_t)t.tn * kTileN + (ie.wave & 1) * kWaveTile, ie.lane);
  }
}

// Waves a SIMD: what the ring leaves room for, or the accumulators.
constexpr int mid_waves(int tm, int tn, int slots) {
  return tm * tn <= 64 * 64 ? 4 : ((tm + tn) * 128 * slots <= 80 * 1024 ? 2 : 1);
}

template <int TM, int TN, int SLOTS>
__global__ __launch_bounds__(256, mid_waves(TM, TN, SLOTS)) void loss_forward_mid(LossArgs s) {
  typedef MidGeom<TM, TN, SLOTS> G;
  const int lane = threadIdx.x & 63, wave = wave_id();
  const KernelArgs& a = s.gemm;
  const MidTile t = mid_tile(persistent_slot(blockIdx.x, gridDim.x), (int)((a.M + TM - 1) / TM),
                             (int)((a.N + TN - 1) / TN));
  MidAccum<G::kBM, G::kBN> acc;
  mid_loop<2, true, true, TM, TN, SLOTS>(acc, a, (int64_t)t.tm * TM, (int64_t)t.tn * TN, wave, lane, 0,
                                         (int)((a.K + 63) / 64), a.K);
  reduce_logits(acc.v, s, (int64_t)t.tm * TM + (wave >> 1) * 32 * G::kBM,
                (int64_t)t.tn * TN + (wave & 1) * 32 * G::kBN, lane);
}

// Few tiles and much K: 16 x 32 tiles whose 16 waves split K (rowblock.hpp).
constexpr int kRowsNB = 2, kRowsWaves = 16;
template <class Done>
__device__ __forceinline__ void rows_tile(const KernelArgs& a, int64_t m0, int64_t n0, f32x4* part, int wave,
                                          int lane, Done&& done) {
  RowBlock<1> ra;
  RowBlock<kRowsNB> rb;
  ra.init(a.A, a.lda * 2, a.M, m0, a.K * 2, lane);
  rb.init(a.B, a.ldb * 2, a.N, n0, a.K * 2, lane);
  f32x4 acc[1][kRowsNB] = {};
  rowblock_loop<2, 1, kRowsNB, kRowsWaves, 1>(acc, ra, rb, a.K * 2, wave, lane);
  rowblock_join<1, kRowsNB, kRowsWaves>(acc, part, wave, lane, [&](int, int nb, f32x4 v) {
    done(m0 + (lane & 15), n0 + 16 * nb + 4 * (lane >> 4), v);
  });
}
__global__ __launch_bounds__(64 * kRowsWaves) void loss_forward_rows(LossArgs s) {
  __shared__ f32x4 part[kRowsWaves * kRowsNB * 64];
  const int lane = threadIdx.x & 63, wave = wave_id();
  const KernelArgs& a = s.gemm;
  const int tiles_m = (int)((a.M + 15) / 16), t = persistent_slot(blockIdx.x, gridDim.x);
  rows_tile(a, (int64_t)(t % tiles_m) * 16, (int64_t)(t / tiles_m) * 32, part, wave, lane,
            [&](int64_t m, int64_t n, f32x4 v) {
              const int64_t left = a.N - n;
#pragma unroll
              for (int c = 0; c < 4; ++c) v[c] = c < left ? v[c] : -INFINITY;
              float top = fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3]));
              top = fmaxf(top, __shfl_xor(top, 16, 64));
              top = fmaxf(top, __shfl_xor(top, 32, 64));
              const float ref = reference_of(top);
              float sum = (exp_diff(v[0], ref) + exp_diff(v[1], ref)) + (exp_diff(v[2], ref) + exp_diff(v[3], ref));
              sum += __shfl_xor(sum, 16, 64);
              sum += __shfl_xor(sum, 32, 64);
              if (m >= a.M || (n & ~(int64_t)15) >= a.N) return;
              if (lane < 16) s.parts[(n >> 4) * s.part_rows + m] = {top, sum};
              const int64_t at = s.target[m] - n;
              if (at >= 0 && at < 4 && at < left) s.target_logit[m] = v[at];
            });
}

// A largest logit and the sum of exponentials against it (of them all).
struct Pair {
  float m, sum;
};
__device__ __forceinline__ Pair join(Pair a, Pair b) {
  const float top = fmaxf(a.m, b.m), ref = reference_of(top);
  // (The factors are chosen, not the terms: a NaN sum stays one.)
  return {top, a.sum * (a.m == -INFINITY ? 0.0f : exp_diff(reference_of(a.m), ref)) +
                   b.sum * (b.m == -INFINITY ? 0.0f : exp_diff(reference_of(b.m), ref))};
}

// A row's pairs joined: ROWS rows a workgroup, 1024 / ROWS threads a row (few
// rows: more threads each, and more workgroups).
template <int ROWS>
__global__ __launch_bounds__(1024) void loss_join(LossArgs s) {
  constexpr int kGroups = 1024 / ROWS;
  __shared__ Pair pairs[16][ROWS];
  const int r = threadIdx.x % ROWS, group = threadIdx.x / ROWS;
  const int64_t row = (int64_t)blockIdx.x * ROWS + r;
  const bool in = row < s.gemm.M;
  const int64_t parts = (s.gemm.N + s.part_cols - 1) / s.part_cols;
  Pair p = {-INFINITY, 0.0f};
  for (int64_t first = group; first < parts; first += 4 * kGroups) {
    float2 x[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t at = first + i * kGroups;
      x[i] = in && at < parts ? s.parts[at * s.part_rows + row] : float2{-INFINITY, 0.0f};
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) p = join(p, Pair{x[i].x, x[i].y});
  }
#pragma unroll
  for (int d = ROWS; d < 64; d <<= 1) p = join(p, Pair{__shfl_xor(p.m, d, 64), __shfl_xor(p.sum, d, 64)});
  if ((threadIdx.x & 63) < ROWS) pairs[threadIdx.x >> 6][r] = p;
  __syncthreads();
  if (threadIdx.x < ROWS && in) {
#pragma unroll
    for (int i = 1; i < 16; ++i) p = join(p, pairs[i][r]);
    const float lse = reference_of(p.m) + logf(p.sum);
    s.lse[row] = lse;
    const int64_t t = s.target[row];
    s.loss[row] = t < 0 ? 0.0f : (t < s.gemm.N ? lse - s.target_logit[row] : NAN);
  }
}

// ------------------------------------------------------------------ backward

// The rows that count (0 <= target < V), numbered in order and copied
// together: x, with what their gradient needs; zeros in dx for the others.
// from[number] is the row.  The first workgroup counts them all and finds the
// largest |dloss|, whose significand (1 .. 2) is the gradients' factor; each
// other one takes `rows` consecutive rows, and counts the targets before them
// itself.  A wave copies a row.
__global__ __launch_bounds__(1024) void loss_gather_rows(LossArgs s, int64_t rows) {
  __shared__ int totals[16];
  __shared__ float tops[16];
  __shared__ int places[1024];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  // (The last workgroups may have no rows: nothing past T is read either.)
  const int64_t from_row = ((int64_t)blockIdx.x - 1) * rows;
  const int64_t begin = from_row < s.T ? from_row : s.T;
  const int64_t end = begin + rows < s.T ? begin + rows : s.T;
  auto counts = [&](int64_t t) { return t >= 0 && t < s.V; };
  auto add_up = [&](int n) {
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) n += __shfl_xor(n, d, 64);
    if (lane == 0) totals[wave] = n;
    __syncthreads();
    n = 0;
#pragma unroll
    for (int w = 0; w < 16; ++w) n += totals[w];
    __syncthreads();
    return n;
  };
  if (blockIdx.x == 0) {
    int n = 0;
    float top = 0.0f;
#pragma unroll 4
    for (int64_t i = threadIdx.x; i < s.T; i += 1024) {
      const float d = fabsf(s.dloss[i]);
      if (counts(s.target[i])) {
        ++n;
        if (d < INFINITY) top = fmaxf(top, d);  // (neither infinity nor NaN)
      }
    }
    n = add_up(n);
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor(top, d, 64));
    if (lane == 0) tops[wave] = top;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int w = 1; w < 16; ++w) top = fmaxf(top, tops[w]);
      int exponent;
      s.head->count = n;
      s.head->factor = top > 0.0f ? 2.0f * frexpf(top, &exponent) : 1.0f;
    }
    return;
  }
  int base = 0;
#pragma unroll 4
  for (int64_t i = threadIdx.x; i < begin; i += 1024) base += counts(s.target[i]);
  base = add_up(base);
  for (int64_t first = begin; first < end; first += 1024) {
    const int64_t own = first + threadIdx.x;
    const int64_t t = own < end ? s.target[own] : -1;
    const uint64_t mask = __ballot(counts(t));
    if (lane == 0) totals[wave] = __popcll(mask);
    __syncthreads();
    int at = base + __popcll(mask & (((uint64_t)1 << lane) - 1));
    for (int w = 0; w < 16; ++w) {
      if (w < wave) at += totals[w];
      base += totals[w];
    }
    places[threadIdx.x] = counts(t) ? at : -1;
    if (counts(t)) {
      s.from[at] = (int)own;
      s.rows_lse[at] = s.lse[own];
      s.rows_dloss[at] = s.dloss[own];
      s.rows_target[at] = (int)t;
    }
    __syncthreads();
    for (int i = wave; i < 1024 && first + i < end; i += 16) {
      const int64_t row = first + i;
      const int place = places[i];
      if (place >= 0) {
        // (Whole 16-byte blocks: the last one's bytes past H are never used.)
        const u32x4* from = reinterpret_cast<const u32x4*>(static_cast<const unsigned short*>(s.x) + row * s.x_rs);
        u32x4* to = reinterpret_cast<u32x4*>(s.rows_x + (int64_t)place * s.rows_ld);
#pragma unroll 4
        for (int64_t c = lane; c * 8 < s.H; c += 64) to[c] = from[c];
      } else {
        unsigned short* d = static_cast<unsigned short*>(s.dx) + row * s.dx_rs;
        for (int64_t c = (int64_t)lane * 8; c < s.H; c += 512) {
          if (c + 8 <= s.H) {
            *reinterpret_cast<u32x4*>(d + c) = u32x4{0, 0, 0, 0};
          } else {
            for (int e = 0; c + e < s.H; ++e) d[c + e] = 0;
          }
        }
      }
    }
    __syncthreads();  // places and totals are read before the next rows' are written
  }
}

// The arguments of a product whose rows (M) are the rows that count.
__device__ __forceinline__ KernelArgs with_rows(const LossArgs& s, KernelArgs a) {
  const int count = s.head->count;
  a.M = count;
  a.a_bytes = count > 0 ? ((int64_t)(count - 1) * a.lda + a.K) * 2 : 0;
  a.tiles_m = (count + kTileM - 1) / kTileM;
  a.num_tiles = a.tiles_per_batch = a.tiles_m * a.tiles_n;
  a.group_m = a.tiles_m < 8 ? (a.tiles_m > 0 ? a.tiles_m : 1) : 8;
  return a;
}

// The wave's logits of rows m0.., columns n0.. of the piece (first_col ..) made
// g over the factor.
template <int BM, int BN>
__device__ __forceinline__ void logits_to_gradient(f32x16 (&v)[BM][BN], const LossArgs& s, int64_t rows,
                                                   int64_t m0, int64_t n0, int lane) {
  const int lr = lane & 31, half = lane >> 5;
  const float factor = s.head->factor;
  float lse[BM], scale[BM];
  int want[BM];  // the target's column here, or -1
#pragma unroll
  for (int bi = 0; bi < BM; ++bi) {
    const int64_t row = m0 + 32 * bi + lr;
    const bool in = row < rows;
    lse[bi] = in ? s.rows_lse[row] : 0.0f;
    scale[bi] = in ? s.rows_dloss[row] / factor : 0.0f;
    const int64_t at = in ? (int64_t)s.rows_target[row] - s.first_col - n0 : -1;
    want[bi] = at >= 0 && at < 32 * BN ? (int)at : -1;
  }
#pragma unroll
  for (int bi = 0; bi < BM; ++bi) {
    sched_fence();
#pragma unroll
    for (int bj = 0; bj < BN; ++bj)
#pragma unroll
      for (int i = 0; i < 16; ++i) v[bi][bj][i] = exp_diff(v[bi][bj][i], lse[bi]);
    // (A row's target lies in one window of the vocabulary: the search is rare.)
    if (__ballot(want[bi] >= 0) != 0) {
      const int at = want[bi] - 4 * half;  // of the lane's columns, 32 bj + 8 q + c
#pragma unroll
      for (int bj = 0; bj < BN; ++bj)
#pragma unroll
        for (int i = 0; i < 16; ++i) v[bi][bj][i] -= 32 * bj + 8 * (i >> 2) + (i & 3) == at ? 1.0f : 0.0f;
    }
#pragma unroll
    for (int bj = 0; bj < BN; ++bj)
#pragma unroll
      for (int i = 0; i < 16; ++i) v[bi][bj][i] *= scale[bi];
  }
}
__device__ __forceinline__ f32x4 quarter_of(const f32x16& v, int q) {
  return f32x4{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
}

// g of one piece of the vocabulary.
__global__ __launch_bounds__(kThreads, 1) void loss_gradient_tiles(LossArgs s) {
  const int lane = threadIdx.x & 63, wave = wave_id();
  const KernelArgs a = with_rows(s, s.gemm);
  Accum acc;
  NoSideWork none;
  for (int L = persistent_slot(blockIdx.x, gridDim.x); L < a.num_tiles; L += gridDim.x) {
    const TileCoord t = tile_of(L, a);
    const Ids id(lane, wave);
    mainloop<2, true, true>(acc, a, t.tm, t.tn, id.wave, id.lane, none);
    const Ids ie(lane, wave);
    const int64_t m0 = (int64_t)t.tm * kTileM + (ie.wave >> 1) * kWaveTile;
    const int64_t n0 = (int64_t)t.tn * kTileN + (ie.wave & 1) * kWaveTile;
    logits_to_gradient(acc.v, s, a.M, m0, n0, ie.lane);
    tile_store<false>(a.D, a.ldd, a.M, a.N, m0, n0, ie.wave, ie.lane,
                      [&](int bi, int bj, int q) { return quarter_of(acc.v[bi][bj], q); });
    wait_lgkmcnt<0>();  // staging reads done ...
    barrier();          // ... in every wave before the ring is refilled
  }
}

template <int TM, int TN, int SLOTS>
__global__ __launch_bounds__(256, mid_waves(TM, TN, SLOTS)) void loss_gradient_mid(LossArgs s) {
  typedef MidGeom<TM, TN, SLOTS> G;
  const int lane = threadIdx.x & 63, wave = wave_id();
  const MidTile t = mid_tile(persistent_slot(blockIdx.x, gridDim.x), (int)((s.gemm.M + TM - 1) / TM),
                             (int)((s.gemm.N + TN - 1) / TN));
  const KernelArgs a = with_rows(s, s.gemm);
  if ((int64_t)t.tm * TM >= a.M) return;
  MidAccum<G::kBM, G::kBN> acc;
  mid_loop<2, true, true, TM, TN, SLOTS>(acc, a, (int64_t)t.tm * TM, (int64_t)t.tn * TN, wave, lane, 0,
                                         (int)((a.K + 63) / 64), a.K);
  const int64_t m0 = (int64_t)t.tm * TM + (wave >> 1) * 32 * G::kBM;
  const int64_t n0 = (int64_t)t.tn * TN + (wave & 1) * 32 * G::kBN;
  logits_to_gradient(acc.v, s, a.M, m0, n0, lane);
  mid_store<G::kBM, G::kBN>(
      a.D, a.ldd, a.M, a.N, m0, n0, wave, lane,
      [&](int bi, int bj, int q) { return quarter_of(acc.v[bi][bj], q); }, [](int64_t r) { return r; });
}

__global__ __launch_bounds__(64 * kRowsWaves) void loss_gradient_rows(LossArgs s) {
  __shared__ f32x4 part[kRowsWaves * kRowsNB * 64];
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int tiles_m = (int)((s.gemm.M + 15) / 16), t = persistent_slot(blockIdx.x, gridDim.x);
  const KernelArgs a = with_rows(s, s.gemm);
  const float factor = s.head->factor;
  const int64_t m0 = (int64_t)(t % tiles_m) * 16;
  if (m0 >= a.M) return;
  rows_tile(a, m0, (int64_t)(t / tiles_m) * 32, part, wave, lane, [&](int64_t m, int64_t n, f32x4 v) {
    if (m >= a.M || n >= a.N) return;
    const float lse = s.rows_lse[m], scale = s.rows_dloss[m] / factor;
    const int64_t at = (int64_t)s.rows_target[m] - s.first_col - n;
#pragma unroll
    for (int c = 0; c < 4; ++c) v[c] = (exp_diff(v[c], lse) - (c == at ? 1.0f : 0.0f)) * scale;
    store4(static_cast<unsigned short*>(a.D) + m * a.ldd + n, a.N - n, v);
  });
}

// dw of the piece = g^T x: rows are the piece's vocabulary, K the rows that
// count.
__global__ __launch_bounds__(kThreads, 1) void loss_dw_tiles(LossArgs s) {
  const int lane = threadIdx.x & 63, wave = wave_id();
  KernelArgs a = s.gemm;
  const int count = s.head->count;
  const float factor = s.head->factor;
  a.K = count;
  a.a_bytes = count > 0 ? ((int64_t)(count - 1) * a.lda + a.M) * 2 : 0;
  a.b_bytes = count > 0 ? ((int64_t)(count - 1) * a.ldb + a.N) * 2 : 0;
  Accum acc;
  NoSideWork none;
  for (int L = persistent_slot(blockIdx.x, gridDim.x); L < a.num_tiles; L += gridDim.x) {
    const TileCoord t = tile_of(L, a);
    const Ids id(lane, wave);
    mainloop<2, false, false>(acc, a, t.tm, t.tn, id.wave, id.lane, none);
    const Ids ie(lane, wave);
    tile_store<true>(a.D, a.ldd, a.M, a.N, (int64_t)t.tm * kTileM + (ie.wave >> 1) * kWaveTile,
                     (int64_t)t.tn * kTileN + (ie.wave & 1) * kWaveTile, ie.wave, ie.lane,
                     [&](int bi, int bj, int q) { return quarter_of(acc.v[bi][bj], q) * factor; });
    wait_lgkmcnt<0>();
    barrier();
  }
}

// A wave's share of a 256 x 256 tile's fp32 sums in register order: piece
// (block b, quarter q) of lane l at ((4 b + q) * 64 + l) * 16.
__device__ __forceinline__ f32x4* dx_pieces(const LossArgs& s, int split, int64_t tile, int wave) {
  return s.dx_sums + ((split * s.dx_tiles + tile) * kWaves + wave) * (kWaveTile * kWaveTile / 4);
}

// The piece's share of dx = g w, K split `splits` ways; each split adds to
// its own sums (the first piece of the vocabulary sets them).
__global__ __launch_bounds__(kThreads, 1) void loss_dx_tiles(LossArgs s) {
  const int lane = threadIdx.x & 63, wave = wave_id();
  const KernelArgs a = with_rows(s, s.gemm_dx);
  const int stages = (int)((a.K + 63) / 64);
  const int items = a.num_tiles * s.splits;
  Accum acc;
  NoSideWork none;
  for (int L = persistent_slot(blockIdx.x, gridDim.x); L < items; L += gridDim.x) {
    const int split = L / a.num_tiles;
    const TileCoord t = tile_of(L - split * a.num_tiles, a);
    int k0 = (int)((int64_t)stages * split / s.splits);
    int nk = (int)((int64_t)stages * (split + 1) / s.splits) - k0;
    const int64_t kend = (int64_t)(k0 + nk) * 64 < a.K ? (int64_t)(k0 + nk) * 64 : a.K;
    asm volatile("" : "+s"(k0), "+s"(nk));
    const Ids id(lane, wave);
    mainloop_range<2, true, false>(acc, a, t.tm, t.tn, id.wave, id.lane, none, k0, nk, kend);
    const Ids ie(lane, wave);
    f32x4* p = dx_pieces(s, split, (int64_t)t.tm * a.tiles_n + t.tn, ie.wave);
#pragma unroll
    for (int b = 0; b < 16; ++b)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const f32x16& v = acc.v[b >> 2][b & 3];
        f32x4 x = {v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
        f32x4* at = p + (4 * b + q) * 64 + ie.lane;
        if (!s.first_piece) x += *at;
        *at = x;
      }
  }
}

// The small tiles' products, in one launch if both take the same: the first
// dx_items workgroups are the parts of dx (K split `splits` ways), those after
// them the parts of dw.  A product
// that one workgroup finishes is stored at once; else the sums go to memory in
// register order (those of dx are added to from piece to piece) and
// loss_finish adds them up.
template <int TM, int TN, int SLOTS>
__global__ __launch_bounds__(256, mid_waves(TM, TN, SLOTS)) void loss_products_mid(LossArgs s) {
  typedef MidGeom<TM, TN, SLOTS> G;
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int count = s.head->count;
  const float factor = s.head->factor;
  const int dx_tiles_m = (int)((s.T + TM - 1) / TM), tiles_n = (int)((s.H + TN - 1) / TN);
  const int dx_tiles = dx_tiles_m * tiles_n, dx_items = s.dx_items;
  // (Each product's parts are dealt over the XCDs by themselves: dx's are the
  // longer ones, and few.)
  const bool is_dx = (int)blockIdx.x < dx_items;
  const int slot = is_dx ? persistent_slot(blockIdx.x, dx_items)
                         : persistent_slot(blockIdx.x - dx_items, gridDim.x - dx_items);
  MidAccum<G::kBM, G::kBN> acc;
  if (is_dx) {
    const KernelArgs a = with_rows(s, s.gemm_dx);
    const int split = slot / dx_tiles;
    const MidTile t = mid_tile(slot - split * dx_tiles, dx_tiles_m, tiles_n);
    if ((int64_t)t.tm * TM >= a.M) return;
    const int stages = (int)((a.K + 63) / 64);
    const int k0 = (int)((int64_t)stages * split / s.splits), k1 = (int)((int64_t)stages * (split + 1) / s.splits);
    const int64_t kend = (int64_t)k1 * 64 < a.K ? (int64_t)k1 * 64 : a.K;
    mid_loop<2, true, false, TM, TN, SLOTS>(acc, a, (int64_t)t.tm * TM, (int64_t)t.tn * TN, wave, lane, k0, k1 - k0,
                                            kend);
    if (s.dx_summed) {
      if (!s.first_piece) mid_add_all(s.dx_sums, slot, acc, wave, lane);
      mid_put(s.dx_sums, slot, acc, wave, lane);
    } else {
      mid_store<G::kBM, G::kBN>(
          a.D, a.ldd, a.M, a.N, (int64_t)t.tm * TM + (wave >> 1) * 32 * G::kBM,
          (int64_t)t.tn * TN + (wave & 1) * 32 * G::kBN, wave, lane,
          [&](int bi, int bj, int q) { return quarter_of(acc.v[bi][bj], q) * factor; },
          [&](int64_t r) { return (int64_t)s.from[r]; });
    }
  } else {
    KernelArgs a = s.gemm;
    a.K = count;
    a.a_bytes = count > 0 ? ((int64_t)(count - 1) * a.lda + a.M) * 2 : 0;
    a.b_bytes = count > 0 ? ((int64_t)(count - 1) * a.ldb + a.N) * 2 : 0;
    const int tiles_m = (int)((a.M + TM - 1) / TM), tiles = tiles_m * tiles_n;
    const int split = slot / tiles;
    const MidTile t = mid_tile(slot - split * tiles, tiles_m, tiles_n);
    const int stages = (count + 63) / 64;
    const int k0 = (int)((int64_t)stages * split / s.dw_splits);
    const int k1 = (int)((int64_t)stages * (split + 1) / s.dw_splits);
    mid_loop<2, false, false, TM, TN, SLOTS>(acc, a, (int64_t)t.tm * TM, (int64_t)t.tn * TN, wave, lane, k0,
                                             k1 - k0, k1 * 64 < count ? k1 * 64 : count);
    if (s.dw_splits > 1) {
      mid_put(s.dw_sums, slot, acc, wave, lane);
    } else {
      mid_store<G::kBM, G::kBN>(
          a.D, a.ldd, a.M, a.N, (int64_t)t.tm * TM + (wave >> 1) * 32 * G::kBM,
          (int64_t)t.tn * TN + (wave & 1) * 32 * G::kBN, wave, lane,
          [&](int bi, int bj, int q) { return quarter_of(acc.v[bi][bj], q) * factor; }, [](int64_t r) { return r; });
    }
  }
}

// The sums of one 32 x 32 block of dx (the first dx_blocks workgroups) or dw,
// added up, scaled and stored.  WAVES waves share the splits: each adds its
// own in order, then the first adds the others' (with 48 splits 4 waves take 6
// us where one takes 12).
template <int TM, int TN, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void loss_finish(LossArgs s, int dx_blocks) {
  constexpr int BM = TM / 64, BN = TN / 64;
  const int lane = threadIdx.x & 63, share = threadIdx.x >> 6;
  const bool dx = (int)blockIdx.x < dx_blocks;
  const int at = dx ? blockIdx.x : blockIdx.x - dx_blocks;
  const int64_t M = dx ? s.head->count : s.gemm.M;
  const int tiles_m = (int)(((dx ? s.T : M) + TM - 1) / TM), tiles_n = (int)((s.H + TN - 1) / TN);
  const int part = at % (4 * BM * BN), tile = at / (4 * BM * BN);
  const int wave = part / (BM * BN), block = part % (BM * BN);
  // (loss_dx_tiles numbers its sums row by row of tiles.)
  const MidTile t = TM == kTileM ? MidTile{tile / tiles_n, tile % tiles_n} : mid_tile(tile, tiles_m, tiles_n);
  const int64_t m = (int64_t)t.tm * TM + (wave >> 1) * 32 * BM + 32 * (block / BN) + (lane & 31);
  const int64_t n0 = (int64_t)t.tn * TN + (wave & 1) * 32 * BN + 32 * (block % BN);
  if (m - (lane & 31) >= M || n0 >= s.H) return;  // (the whole workgroup)
  const float factor = s.head->factor;
  MidAccum<1, 1> acc = {};
  const int splits = dx ? s.splits : s.dw_splits;
  const mid_piece* sums = dx ? s.dx_sums : s.dw_sums;
#pragma unroll 8
  for (int i = splits * share / WAVES; i < splits * (share + 1) / WAVES; ++i)
    mid_add<BM, BN>(sums, (int64_t)i * tiles_m * tiles_n + tile, acc, wave, block, lane);
  if constexpr (WAVES > 1) {
    __shared__ f32x4 shares[WAVES][4][64];
#pragma unroll
    for (int q = 0; q < 4; ++q) shares[share][q][lane] = quarter_of(acc.v[0][0], q);
    __syncthreads();
    if (share != 0) return;
#pragma unroll
    for (int w = 1; w < WAVES; ++w)
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int c = 0; c < 4; ++c) acc.v[0][0][4 * q + c] += shares[w][q][lane][c];
  }
  if (m >= M) return;
  unsigned short* d = dx ? static_cast<unsigned short*>(s.dx) + (int64_t)s.from[m] * s.dx_rs
                         : static_cast<unsigned short*>(s.gemm.D) + m * s.gemm.ldd;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int64_t n = n0 + 8 * q + 4 * (lane >> 5);
    store4(d + n, s.H - n, quarter_of(acc.v[0][0], q) * factor);
  }
}

typedef void (*loss_fn)(LossArgs);
struct MidKernels {
  int lds;
  loss_fn forward, gradient, products;
};
template <int TM, int TN, int SLOTS>
constexpr MidKernels mid_kernels() {
  return {(int)MidGeom<TM, TN, SLOTS>::kLds, loss_forward_mid<TM, TN, SLOTS>, loss_gradient_mid<TM, TN, SLOTS>,
          loss_products_mid<TM, TN, SLOTS>};
}
// From kLoss128 on.
const MidKernels kMid[] = {mid_kernels<128, 128, 2>(), mid_kernels<64, 128, 3>(), mid_kernels<64, 64, 4>()};
typedef void (*finish_fn)(LossArgs, int);
const finish_fn kFinish[][2] = {{loss_finish<256, 256, 1>, loss_finish<256, 256, 4>},
                                {loss_finish<128, 128, 1>, loss_finish<128, 128, 4>},
                                {loss_finish<64, 128, 1>, loss_finish<64, 128, 4>},
                                {loss_finish<64, 64, 1>, loss_finish<64, 64, 4>}};

// What the tiles cost, in microseconds: a K stage of 64 with one tile a
// compute unit and with two, and a tile besides, by what it makes.
enum LossProduct { kForward, kGradient, kDw, kDx };
struct LossCost {
  int per_cu;
  double stage1, stage2, tile[4];
};
const LossCost kCost[kLossTiles] = {{1, 1.26, 1.26, {14.6, 14.6, 10.7, 7.2}},
                                    {2, 0.66, 1.00, {3.1, 4.6, 2.8, 3.2}},
                                    {2, 0.42, 0.69, {2.5, 4.1, 2.5, 2.7}},
                                    {2, 0.35, 0.50, {2.3, 3.2, 1.7, 2.1}}};
// Microseconds for a rows x cols product of `bytes` in all, its K of `stages`
// stages split; and the workgroups that takes.
struct ProductCost {
  double us, items;
};
ProductCost cost_of(int tile, LossProduct what, int64_t rows, int64_t cols, int64_t stages, int splits, double bytes,
                    int cu_count) {
  const LossCost& c = kCost[tile];
  const double items = (double)loss_tiles(tile, rows, cols) * splits, st = ceil((double)stages / splits);
  const double at_once = (double)c.per_cu * cu_count, full = floor(items / at_once), rest = items - full * at_once;
  double t = full * (st * c.stage2 + c.tile[what]);
  if (rest > 0) t += st * (rest <= cu_count ? c.stage1 : c.stage2) + c.tile[what];
  const double memory = bytes / 5.1e6;
  return {2.5 + (t > memory ? t : memory), items};
}

}  // namespace

// The tiles and splits that cost least.  The figures are a fit to 140 losses
// of 1 to 8192 rows, 100 to 131072 entries and hidden sizes of 64 to 4096, each
// product timed in every tile and with up to five splits; what it picks is 2 to
// 4% slower than the fastest of them on average.
LossChoice choose_loss(int64_t T, int64_t V, int64_t H, int64_t piece, int cu_count) {
  LossChoice c = {};
  const int64_t W = piece < V ? piece : V, sh = (H + 63) / 64, sw = (W + 63) / 64, st = (T + 63) / 64;
  const double t = (double)T, v = (double)V, h = (double)H, w = (double)W;
  // A launch holds fewer than 2^32 threads (256 x 256 tiles are taken one after
  // another).
  auto fits = [](int tile, int64_t rows, int64_t cols, int splits) {
    return tile == kLoss256 || (double)loss_tiles(tile, rows, cols) * splits < (1 << 21);
  };
  double least_f = 1e301, least_g = 1e301;
  for (int i = 0; i <= kLossRows; ++i) {
    auto logits = [&](LossProduct what, int64_t cols, double bytes) {
      if (!fits(i, T, cols, 1)) return 1e300;
      if (i < kLossTiles) return cost_of(i, what, T, cols, sh, 1, bytes, cu_count).us;
      // What a compute unit takes in, and the memory.
      const double tiles = (double)loss_tiles(i, T, cols), rounds = tiles > cu_count ? tiles / cu_count : 1.0;
      const double cu = rounds * (kLossTileM[i] + kLossTileN[i]) * 2 * h / 52e3, memory = bytes / 5.1e6;
      return 3.0 + (cu > memory ? cu : memory) + 0.6 * ceil(tiles / (2 * cu_count));
    };
    // (A row's pairs, one for half a tile's columns, are written and joined.)
    const double f = logits(kForward, V, 2 * h * (t + v)) + 16 * t * (v / (kLossTileN[i] / 2)) / 4e6;
    if (f < least_f) least_f = f, c.forward = i;
    const double g = logits(kGradient, W, 2 * (h * (t + w) + t * w));
    if (g < least_g) least_g = g, c.gradient = i;
  }
  // Both products' tiles and splits together: alike, they share the launches.
  double least = 1e300;
  constexpr int kSplits[] = {1, 2, 3, 4, 6, 8, 12, 16, 24, 32, 48, 64};
  const double launch = 3.5;
  auto finish = [&](int splits, double elements) {
    return launch + 0.05 * splits + (4.0 * splits + 2) * elements / 4.5e6;
  };
  // Every way that each product can take (a tile, splits; +infinity: none),
  // and what its sums' end costs.
  constexpr int kWays = sizeof(kSplits) / sizeof(int);
  struct Way {
    double us, items, end;
  } dx[kLossTiles][kWays], dw[kLossTiles][kWays];
  for (int i = 0; i < kLossTiles; ++i)
    for (int k = 0; k < kWays; ++k) {
      const int n = kSplits[k];
      const bool summed = i == kLoss256 || n > 1 || W < V;
      const double sums = 4 * t * h * n, dw_sums = 4 * w * h * n;
      dx[i][k] = dw[i][k] = {1e300, 0, 0};
      if (fits(i, T, H, n) && (n == 1 || (sw >= 3 * n && sums <= (512 << 20)))) {
        const ProductCost p =
            cost_of(i, kDx, T, H, sw, n, 2 * (t * w + w * h) + (summed ? sums : 2 * t * h), cu_count);
        dx[i][k] = {p.us, p.items, summed ? finish(n, t * h) : 0};
      }
      if (fits(i, W, H, n) && (n == 1 || (i != kLoss256 && st >= 3 * n && dw_sums <= (512 << 20)))) {
        const ProductCost p =
            cost_of(i, kDw, W, H, st, n, 2 * (t * w + t * h) + (n > 1 ? dw_sums : 2 * w * h), cu_count);
        dw[i][k] = {p.us, p.items, n > 1 ? finish(n, w * h) : 0};
      }
    }
  for (int x = 0; x < kLossTiles; ++x)
    for (int i = 0; i < kWays; ++i) {
      const Way& p = dx[x][i];
      if (p.us >= least) continue;
      for (int y = 0; y < kLossTiles; ++y)
        for (int j = 0; j < kWays; ++j) {
          const Way& q = dw[y][j];
          double both = p.us + q.us + launch + p.end + q.end;
          if (x == y && x != kLoss256) {
            // Side by side where both fit the chip.
            both = p.items + q.items <= kCost[x].per_cu * (double)cu_count ? (p.us > q.us ? p.us : q.us) + 1
                                                                           : p.us + q.us - 2.5;
            both += p.end + q.end - (p.end > 0 && q.end > 0 ? launch : 0);
          }
          if (both < least) {
            least = both;
            c.dx = x, c.dx_splits = kSplits[i], c.dw = y, c.dw_splits = kSplits[j];
          }
        }
    }
  return c;
}

hipError_t prepare_loss() {
  struct {
    loss_fn f;
    int lds;
  } all[16] = {{loss_forward_tiles, kPlainLdsBytes}, {loss_gradient_tiles, kPlainLdsBytes},
               {loss_dw_tiles, kPlainLdsBytes}, {loss_dx_tiles, kPlainLdsBytes}};
  int n = 4;
  for (const MidKernels& m : kMid)
    for (loss_fn f : {m.forward, m.gradient, m.products}) all[n++] = {f, m.lds};
  for (int i = 0; i < n; ++i) {
    const auto& k = all[i];
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(k.f),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, k.lds);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

#define MIGEMM_LAUNCH(kernel, grid, threads, lds, ...)                                          \
  do {                                                                                       \
    hipLaunchKernelGGL(kernel, dim3((uint32_t)(grid)), dim3(threads), lds, stream, __VA_ARGS__); \
    const hipError_t e = hipGetLastError();                                                  \
    if (e != hipSuccess) return e;                                                           \
  } while (0)

hipError_t launch_loss_forward(const LossArgs& s, int tile, int cu_count, hipStream_t stream) {
  const int64_t tiles = loss_tiles(tile, s.gemm.M, s.gemm.N);
  if (tile == kLoss256) {
    MIGEMM_LAUNCH(loss_forward_tiles, tiles < cu_count ? tiles : cu_count, kThreads, kPlainLdsBytes, s);
  } else if (tile == kLossRows) {
    MIGEMM_LAUNCH(loss_forward_rows, tiles, 64 * kRowsWaves, 0, s);
  } else {
    MIGEMM_LAUNCH(kMid[tile - 1].forward, tiles, 256, kMid[tile - 1].lds, s);
  }
  // Few rows: 4 a workgroup.
  if (s.gemm.M <= 2048) MIGEMM_LAUNCH(loss_join<4>, (s.gemm.M + 3) / 4, 1024, 0, s);
  else MIGEMM_LAUNCH(loss_join<16>, (s.gemm.M + 15) / 16, 1024, 0, s);
  return hipSuccess;
}

hipError_t launch_loss_rows(const LossArgs& s, hipStream_t stream) {
  int64_t grid = (s.T + 3) / 4;
  grid = grid < 1 ? 1 : (grid > 255 ? 255 : grid);
  MIGEMM_LAUNCH(loss_gather_rows, grid + 1, 1024, 0, s, (s.T + grid - 1) / grid);
  return hipSuccess;
}
hipError_t launch_loss_gradient(const LossArgs& s, int tile, int cu_count, hipStream_t stream) {
  const int64_t tiles = loss_tiles(tile, s.gemm.M, s.gemm.N);
  if (tile == kLoss256) {
    MIGEMM_LAUNCH(loss_gradient_tiles, tiles < cu_count ? tiles : cu_count, kThreads, kPlainLdsBytes, s);
  } else if (tile == kLossRows) {
    MIGEMM_LAUNCH(loss_gradient_rows, tiles, 64 * kRowsWaves, 0, s);
  } else {
    MIGEMM_LAUNCH(kMid[tile - 1].gradient, tiles, 256, kMid[tile - 1].lds, s);
  }
  return hipSuccess;
}
hipError_t launch_loss_products(const LossArgs& args, const LossChoice& c, bool last_piece, int cu_count,
                                hipStream_t stream) {
  LossArgs s = args;
  const int64_t dx_items = s.dx_tiles * s.splits;
  const int64_t dw_tiles = loss_tiles(c.dw, s.gemm.M, s.H), dw_items = dw_tiles * s.dw_splits;
  auto blocks = [](int tile) { return (kLossTileM[tile] / 32) * (kLossTileN[tile] / 32); };
  const int64_t dx_blocks = s.dx_summed && last_piece ? s.dx_tiles * blocks(c.dx) : 0;
  const int64_t dw_blocks = s.dw_splits > 1 ? dw_tiles * blocks(c.dw) : 0;
  const bool together = c.dx == c.dw && c.dx != kLoss256;
  if (together) {
    s.dx_items = (int)dx_items;
    MIGEMM_LAUNCH(kMid[c.dx - 1].products, dx_items + dw_items, 256, kMid[c.dx - 1].lds, s);
  } else {
    if (c.dw == kLoss256) {
      MIGEMM_LAUNCH(loss_dw_tiles, dw_items < cu_count ? dw_items : cu_count, kThreads, kPlainLdsBytes, s);
    } else {
      s.dx_items = 0;
      MIGEMM_LAUNCH(kMid[c.dw - 1].products, dw_items, 256, kMid[c.dw - 1].lds, s);
    }
    if (dx_items > 0) {
      if (c.dx == kLoss256) {
        MIGEMM_LAUNCH(loss_dx_tiles, dx_items < cu_count ? dx_items : cu_count, kThreads, kPlainLdsBytes, s);
      } else {
        s.dx_items = (int)dx_items;
        MIGEMM_LAUNCH(kMid[c.dx - 1].products, dx_items, 256, kMid[c.dx - 1].lds, s);
      }
    }
  }
  auto finish = [&](int tile, int64_t of_dx, int64_t of_dw, int splits) {
    if (of_dx + of_dw == 0) return hipSuccess;
    const bool shared = splits >= 8;
    MIGEMM_LAUNCH(kFinish[tile][shared], of_dx + of_dw, shared ? 256 : 64, 0, s, (int)of_dx);
    return hipSuccess;
  };
  if (together) return finish(c.dx, dx_blocks, dw_blocks, s.splits > s.dw_splits ? s.splits : s.dw_splits);
  const hipError_t e = finish(c.dw, 0, dw_blocks, s.dw_splits);
  return e != hipSuccess ? e : finish(c.dx, dx_blocks, 0, s.splits);
}

}  // namespace migemm

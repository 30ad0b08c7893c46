// loss_kernels.hip -- softmax cross entropy over a large vocabulary from the
// hidden states x (T x H) and the projection's weights w (V x H), both bf16:
//   logits = x w^T (fp32, never stored);  lse = log sum exp logits;
//   loss = lse - logits[target]  (0 where the target is negative)
// and its gradients, with g = (exp(logits - lse) - onehot(target)) dloss:
//   dx = g w,   dw = g^T x.
//
// Forward: the GEMM's K loop makes 256 x 256 tiles of logits in registers;
// each wave reduces its 128 columns of a row to a maximum and a sum of
// exponentials, and a second kernel joins those of a row.  V / 128 pairs a
// row are 1/32 of what bf16 logits would take.
//
// Backward: rows that do not count are left out first (x's other rows are
// copied together), so they cost nothing and whatever they hold (a NaN in
// padding) reaches no sum.  Then, for a piece of the vocabulary at a time, the
// logits are formed again, g of the piece is stored as bf16, and two products
// read it: dw of the piece, complete, and the piece's share of dx, added up
// in fp32.  g is the one quantity rounded to bf16 in between: the matrix
// instructions take bf16 pairs; its rounding, half a step of 2^-8 a term and
// independent from term to term, is of the size of the rounding of the
// outputs themselves.
//
// Bound: the matrix instructions (one product forward, three backward).
#include <hip/hip_runtime.h>

#include <type_traits>

#include "../kernel/epilogue.hpp"
#include "../kernel/gfx950.hpp"
#include "../kernel/mainloop.hpp"
#include "../kernel/params.hpp"
#include "../kernel/scheduler.hpp"
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

// The wave's 128 x 128 logits of rows m0.., columns n0..: per row the largest
// and the sum of exponentials against it, over the columns below V; and the
// target's logit where it is among them.
__device__ __forceinline__ void reduce_logits(Accum& acc, const LossArgs& s, int64_t m0, int64_t n0,
                                              int lane) {
  const int64_t T = s.gemm.M, V = s.gemm.N;
  const int lr = lane & 31, half = lane >> 5;
  if (n0 >= V) return;
  const int left = V - n0 < kWaveTile ? (int)(V - n0) : kWaveTile;
  float2* part = s.parts + (n0 / kWaveTile) * s.part_rows;
#pragma unroll
  for (int bi = 0; bi < 4; ++bi) {
    const int64_t row = m0 + 32 * bi + lr;
    if (left < kWaveTile) {
#pragma unroll
      for (int bj = 0; bj < 4; ++bj)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (32 * bj + 8 * (i >> 2) + 4 * half + (i & 3) >= left) acc.v[bi][bj][i] = -INFINITY;
    }
    float m = acc.v[bi][0][0];
#pragma unroll
    for (int bj = 0; bj < 4; ++bj)
#pragma unroll
      for (int i = 0; i < 16; ++i) m = fmaxf(m, acc.v[bi][bj][i]);
    m = fmaxf(m, __shfl_xor(m, 32, 64));
    const float ref = reference_of(m);
    float sum = 0.0f;
#pragma unroll
    for (int bj = 0; bj < 4; ++bj)
#pragma unroll
      for (int i = 0; i < 16; ++i) sum += exp_diff(acc.v[bi][bj][i], ref);
    sum += __shfl_xor(sum, 32, 64);
    if (row < T && half == 0) part[row] = {m, sum};
    // (A row's target lies in one window of V / 128: the search is rare.)
    const int64_t at = row < T ? s.target[row] - n0 : -1;
    const bool here = at >= 0 && at < left;
    if (__ballot(here) != 0) {
      const int want = here ? (int)at : -1;
#pragma unroll
      for (int bj = 0; bj < 4; ++bj)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (32 * bj + 8 * (i >> 2) + 4 * half + (i & 3) == want) s.target_logit[row] = acc.v[bi][bj][i];
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
    reduce_logits(acc, s, (int64_t)t.tm * kTileM + (ie.wave >> 1) * kWaveTile,
                  (int64_t)t.tn * kTileN + (ie.wave & 1) * kWaveTile, ie.lane);
  }
}

// A row's pairs joined: 16 rows a workgroup, 64 threads a row.
__global__ __launch_bounds__(1024) void loss_join(LossArgs s) {
  __shared__ float ms[64][17], ss[64][17];
  const int r = threadIdx.x & 15, group = threadIdx.x >> 4;
  const int64_t row = (int64_t)blockIdx.x * 16 + r;
  const int64_t parts = (s.gemm.N + kWaveTile - 1) / kWaveTile;
  float m = -INFINITY, sum = 0.0f;
  if (row < s.gemm.M) {
    for (int64_t p = group; p < parts; p += 64) {
      const float2 x = s.parts[p * s.part_rows + row];
      const float top = fmaxf(m, x.x), ref = reference_of(top);
      // (The factors are chosen, not the terms: a NaN sum stays one.)
      sum = sum * (m == -INFINITY ? 0.0f : exp_diff(reference_of(m), ref)) +
            x.y * (x.x == -INFINITY ? 0.0f : exp_diff(reference_of(x.x), ref));
      m = top;
    }
  }
  ms[group][r] = m;
  ss[group][r] = sum;
  __syncthreads();
  if (group == 0 && row < s.gemm.M) {
    for (int i = 1; i < 64; ++i) m = fmaxf(m, ms[i][r]);
    const float ref = reference_of(m);
    sum = 0.0f;
    for (int i = 0; i < 64; ++i)
      if (ms[i][r] != -INFINITY || ss[i][r] != 0.0f) sum += ss[i][r] * exp_diff(reference_of(ms[i][r]), ref);
    const float lse = ref + logf(sum);
    s.lse[row] = lse;
    const int64_t t = s.target[row];
    s.loss[row] = t < 0 ? 0.0f : (t < s.gemm.N ? lse - s.target_logit[row] : NAN);
  }
}

// ------------------------------------------------------------------ backward

// The rows that count (0 <= target < V), numbered in order: place[row] is the
// row's number or -1, from[number] the row.  One workgroup.
__global__ __launch_bounds__(1024) void loss_number_rows(LossArgs s) {
  __shared__ int totals[16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int base = 0;
  for (int64_t first = 0; first < s.T; first += 1024) {
    const int64_t row = first + threadIdx.x;
    const int64_t t = row < s.T ? s.target[row] : -1;
    const bool counts = t >= 0 && t < s.V;
    const uint64_t mask = __ballot(counts);
    if (lane == 0) totals[wave] = __popcll(mask);
    __syncthreads();
    int at = base + __popcll(mask & (((uint64_t)1 << lane) - 1));
    for (int w = 0; w < 16; ++w) {
      if (w < wave) at += totals[w];
      base += totals[w];
    }
    if (row < s.T) s.place[row] = counts ? at : -1;
    if (counts) s.from[at] = (int)row;
    __syncthreads();
  }
  if (threadIdx.x == 0) *s.count = base;
}

// Row by row: x of the rows that count copied together, with what their
// gradient needs; zeros in dx for the others.  A wave takes a row.
__global__ __launch_bounds__(256) void loss_gather_rows(LossArgs s) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int64_t row = (int64_t)blockIdx.x * 4 + wave; row < s.T; row += (int64_t)gridDim.x * 4) {
    const int at = s.place[row];
    if (at >= 0) {
      // (Whole 16-byte blocks: the last one's bytes past H are never used.)
      const u32x4* from = reinterpret_cast<const u32x4*>(static_cast<const unsigned short*>(s.x) + row * s.x_rs);
      u32x4* to = reinterpret_cast<u32x4*>(s.rows_x + (int64_t)at * s.rows_ld);
      for (int64_t c = lane; c * 8 < s.H; c += 64) to[c] = from[c];
      if (lane == 0) {
        s.rows_lse[at] = s.lse[row];
        s.rows_dloss[at] = s.dloss[row];
        s.rows_target[at] = (int)s.target[row];
      }
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
}

// The arguments of a product whose rows (M) are the rows that count.
__device__ __forceinline__ KernelArgs with_rows(const LossArgs& s) {
  KernelArgs a = s.gemm;
  const int count = *s.count;
  a.M = count;
  a.a_bytes = count > 0 ? ((int64_t)(count - 1) * a.lda + a.K) * 2 : 0;
  a.tiles_m = (count + kTileM - 1) / kTileM;
  a.num_tiles = a.tiles_per_batch = a.tiles_m * a.tiles_n;
  a.group_m = a.tiles_m < 8 ? (a.tiles_m > 0 ? a.tiles_m : 1) : 8;
  return a;
}

// g of one piece of the vocabulary: columns first_col .. + N.
__global__ __launch_bounds__(kThreads, 1) void loss_gradient_tiles(LossArgs s) {
  const int lane = threadIdx.x & 63, wave = wave_id();
  const KernelArgs a = with_rows(s);
  Accum acc;
  NoSideWork none;
  for (int L = persistent_slot(blockIdx.x, gridDim.x); L < a.num_tiles; L += gridDim.x) {
    const TileCoord t = tile_of(L, a);
    const Ids id(lane, wave);
    mainloop<2, true, true>(acc, a, t.tm, t.tn, id.wave, id.lane, none);
    const Ids ie(lane, wave);
    const int64_t m0 = (int64_t)t.tm * kTileM + (ie.wave >> 1) * kWaveTile;
    const int64_t n0 = (int64_t)t.tn * kTileN + (ie.wave & 1) * kWaveTile;
    const int lr = ie.lane & 31, half = ie.lane >> 5;
#pragma unroll
    for (int bi = 0; bi < 4; ++bi) {
      const int64_t row = m0 + 32 * bi + lr;
      const bool in = row < a.M;
      const float lse = in ? s.rows_lse[row] : 0.0f, dl = in ? s.rows_dloss[row] : 0.0f;
      const int64_t at = in ? (int64_t)s.rows_target[row] - s.first_col - n0 : -1;
      const bool here = at >= 0 && at < kWaveTile;
      const int want = here ? (int)at : -1;
      const bool search = __ballot(here) != 0;
#pragma unroll
      for (int bj = 0; bj < 4; ++bj)
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          float p = exp_diff(acc.v[bi][bj][i], lse);
          if (search && 32 * bj + 8 * (i >> 2) + 4 * half + (i & 3) == want) p -= 1.0f;
          acc.v[bi][bj][i] = p * dl;
        }
    }
    tile_store<false>(a.D, a.ldd, a.M, a.N, m0, n0, ie.wave, ie.lane, [&](int bi, int bj, int q) {
      const f32x16& v = acc.v[bi][bj];
      return f32x4{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
    });
    wait_lgkmcnt<0>();  // staging reads done ...
    barrier();          // ... in every wave before the ring is refilled
  }
}

// dw of the piece = g^T x: rows are the piece's vocabulary, K the rows that
// count.
__global__ __launch_bounds__(kThreads, 1) void loss_dw_tiles(LossArgs s) {
  const int lane = threadIdx.x & 63, wave = wave_id();
  KernelArgs a = s.gemm;
  const int count = *s.count;
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
                     [&](int bi, int bj, int q) {
                       const f32x16& v = acc.v[bi][bj];
                       return f32x4{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
                     });
    wait_lgkmcnt<0>();
    barrier();
  }
}

// A wave's 16 KiB-per-row-block share of a tile's fp32 sums in register
// order: piece (block b, quarter q) of lane l at ((4 b + q) * 64 + l) * 16.
__device__ __forceinline__ f32x4* dx_pieces(const LossArgs& s, int split, int64_t tile, int wave) {
  return s.dx_sums + ((split * s.dx_tiles + tile) * kWaves + wave) * (kWaveTile * kWaveTile / 4);
}

// The piece's share of dx = g w, K split `splits` ways; each split adds to
// its own sums (the first piece of the vocabulary sets them).
__global__ __launch_bounds__(kThreads, 1) void loss_dx_tiles(LossArgs s) {
  const int lane = threadIdx.x & 63, wave = wave_id();
  const KernelArgs a = with_rows(s);
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

// dx of the rows that count: the splits' sums added in order, rounded once.
// A workgroup takes 1/16 of a tile.
__global__ __launch_bounds__(256) void loss_dx_finish(LossArgs s) {
  const int64_t tile = blockIdx.x >> 4;
  const int part = blockIdx.x & 15, wave = part >> 2, bi = part & 3;
  const int tiles_n = s.gemm.tiles_n;
  const int64_t tm = tile / tiles_n, tn = tile % tiles_n;
  const int lane = threadIdx.x & 63, bj = threadIdx.x >> 6;
  const int64_t row = tm * kTileM + (wave >> 1) * kWaveTile + 32 * bi + (lane & 31);
  if (row >= *s.count) return;
  unsigned short* d = static_cast<unsigned short*>(s.dx) + (int64_t)s.from[row] * s.dx_rs;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int64_t c = tn * kTileN + (wave & 1) * kWaveTile + 32 * bj + 8 * q + 4 * (lane >> 5);
    if (c >= s.H) continue;
    f32x4 x = {0, 0, 0, 0};
    for (int i = 0; i < s.splits; ++i) x += dx_pieces(s, i, tile, wave)[(4 * (4 * bi + bj) + q) * 64 + lane];
    const u32x2 w = {pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3])};
    if (c + 4 <= s.H) {
      *reinterpret_cast<u32x2*>(d + c) = w;
    } else {
      for (int e = 0; e < (int)(s.H - c); ++e) d[c + e] = (unsigned short)(w[e >> 1] >> (16 * (e & 1)));
    }
  }
}

}  // namespace

hipError_t prepare_loss() {
  const void* f[] = {reinterpret_cast<const void*>(loss_forward_tiles),
                     reinterpret_cast<const void*>(loss_gradient_tiles),
                     reinterpret_cast<const void*>(loss_dw_tiles),
                     reinterpret_cast<const void*>(loss_dx_tiles)};
  for (const void* k : f) {
    const hipError_t e = hipFuncSetAttribute(k, hipFuncAttributeMaxDynamicSharedMemorySize, kPlainLdsBytes);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

#define MIGEMM_LAUNCH(kernel, grid, threads, lds)                                            \
  do {                                                                                       \
    hipLaunchKernelGGL(kernel, dim3((uint32_t)(grid)), dim3(threads), lds, stream, s);       \
    const hipError_t e = hipGetLastError();                                                  \
    if (e != hipSuccess) return e;                                                           \
  } while (0)

hipError_t launch_loss_forward(const LossArgs& s, int grid, hipStream_t stream) {
  MIGEMM_LAUNCH(loss_forward_tiles, grid, kThreads, kPlainLdsBytes);
  MIGEMM_LAUNCH(loss_join, (s.gemm.M + 15) / 16, 1024, 0);
  return hipSuccess;
}

hipError_t launch_loss_rows(const LossArgs& s, hipStream_t stream) {
  MIGEMM_LAUNCH(loss_number_rows, 1, 1024, 0);
  if (s.T > 0) {
    const int64_t grid = (s.T + 3) / 4;
    MIGEMM_LAUNCH(loss_gather_rows, grid < 65536 ? grid : 65536, 256, 0);
  }
  return hipSuccess;
}
hipError_t launch_loss_gradient(const LossArgs& s, int grid, hipStream_t stream) {
  MIGEMM_LAUNCH(loss_gradient_tiles, grid, kThreads, kPlainLdsBytes);
  return hipSuccess;
}
hipError_t launch_loss_dw(const LossArgs& s, int grid, hipStream_t stream) {
  MIGEMM_LAUNCH(loss_dw_tiles, grid, kThreads, kPlainLdsBytes);
  return hipSuccess;
}
hipError_t launch_loss_dx(const LossArgs& s, int grid, hipStream_t stream) {
  MIGEMM_LAUNCH(loss_dx_tiles, grid, kThreads, kPlainLdsBytes);
  return hipSuccess;
}
hipError_t launch_loss_dx_finish(const LossArgs& s, hipStream_t stream) {
  MIGEMM_LAUNCH(loss_dx_finish, s.dx_tiles * 16, 256, 0);
  return hipSuccess;
}

}  // namespace migemm

// scaled_tiles.hpp -- kernels of the product of 8-bit rows with a scale per row
// and per output channel, of e4m3 codes (scaled_kernels.hip) and of int8
// (int8_kernels.hip):
//   d[m][n] = bf16(a_scale[m] b_scale[n] sum_k a[m][k] b[n][k] [+ bias[n]])
// MUL says how the bytes are multiplied.  int8's sums are int32, exact; they
// travel as the bits of the fp32 accumulators until a scale is applied, which
// rounds them to fp32 first (2^-24 of the sum).
#pragma once

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
#include "rowblock.hpp"
#include "tile_store.hpp"

namespace migemm {
namespace {

// Row scales and column scales of a wave's 32 BM x 32 BN part at (m0, n0).
// Scales past the matrix read as zero; what they scale is not stored.
template <int BM, int BN, bool INT8 = false>
struct Scales {
  float rows[BM];
  f32x4 cols[BN][4];
  f32x4 bias[INT8 ? BN : 1][4];
  __device__ __forceinline__ void load(const ScaledArgs& s, int64_t m0, int64_t n0, int lane) {
    auto vec = [](const float* p, int64_t from, int64_t n) {
      int64_t left = (n - from) * 4;
      left = left < 0 ? 0 : (left > 512 ? 512 : left);
      return make_rsrc(p + from, (uint32_t)left);
    };
    const __amdgpu_buffer_rsrc_t ra = vec(s.a_scale, m0, s.gemm.M), rb = vec(s.b_scale, n0, s.gemm.N);
#pragma unroll
    for (int i = 0; i < BM; ++i)
      rows[i] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(ra, (32 * i + (lane & 31)) * 4, 0, 0));
#pragma unroll
    for (int j = 0; j < BN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        cols[j][q] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                   rb, (32 * j + 8 * q + 4 * (lane >> 5)) * 4, 0, 0));
    if constexpr (INT8) {  // (no bias: zeros)
      const __amdgpu_buffer_rsrc_t rz = vec(s.bias, n0, s.bias ? s.gemm.N : 0);
#pragma unroll
      for (int j = 0; j < BN; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          bias[j][q] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                     rz, (32 * j + 8 * q + 4 * (lane >> 5)) * 4, 0, 0));
    }
  }
  __device__ __forceinline__ f32x4 apply(f32x4 v, int bi, int bj, int q) const {
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if constexpr (INT8) v[c] = (float)__float_as_int(v[c]) * rows[bi] * cols[bj][q][c] + bias[bj][q][c];
      else v[c] = v[c] * rows[bi] * cols[bj][q][c];
    }
    return v;
  }
};

// 64 BM x 256 tiles, one after another.
template <MidMul MUL, int BM>
__global__ __launch_bounds__(kThreads, 1) void scaled_tile(ScaledArgs s) {
  const int lane0 = threadIdx.x & 63, wave0 = wave_id();
  const KernelArgs& a = s.gemm;
  Accum acc;
  NoSideWork none;
  for (int L = persistent_slot(blockIdx.x, gridDim.x); L < a.num_tiles; L += gridDim.x) {
    const TileCoord t = tile_of(L, a);
    int lane = lane0, wave = wave0;
    asm volatile("" : "+v"(lane));  // per-lane offsets are formed per tile, not held across tiles
    asm volatile("" : "+s"(wave));
    mainloop<1, true, true, BM, MUL == kMulInt8>(acc, a, t.tm, t.tn, wave, lane, none);
    const int64_t m0 = (int64_t)t.tm * (64 * BM) + (wave >> 1) * (32 * BM);
    const int64_t n0 = (int64_t)t.tn * kTileN + (wave & 1) * kWaveTile;
    Scales<BM, 4, MUL == kMulInt8> scales;
    scales.load(s, m0, n0, lane);
    tile_store<true, BM>(a.D, a.ldd, a.M, a.N, m0, n0, wave, lane, [&](int bi, int bj, int q) {
      const f32x16& v = acc.v[bi][bj];
      return scales.apply(f32x4{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]}, bi, bj, q);
    });
    wait_lgkmcnt<0>();  // staging reads done ...
    barrier();          // ... in every wave before the ring is refilled
  }
}

// One tile of 16 MB x 16 NB a workgroup.  Tiles are numbered down the rows
// first and dealt so that one XCD takes consecutive ones: those share a panel
// of b, which then comes from that XCD's L2.
template <int ES, int MB, int NB, int W, int U>
__global__ __launch_bounds__(64 * W) void scaled_rows(ScaledArgs s) {
  constexpr bool kInt = ES == kInt8;
  typedef std::conditional_t<kInt, i32x4, f32x4> V;
  __shared__ V part[W * MB * NB * 64];
  const int lane = threadIdx.x & 63, wave = wave_id();
  const KernelArgs& a = s.gemm;
  const int tiles_m = (int)((a.M + 16 * MB - 1) / (16 * MB));
  const int t = persistent_slot(blockIdx.x, gridDim.x);
  const int64_t m0 = (int64_t)(t % tiles_m) * 16 * MB, n0 = (int64_t)(t / tiles_m) * 16 * NB;
  RowBlock<MB> ra;
  RowBlock<NB> rb;
  ra.init(a.A, a.lda, a.M, m0, a.K, lane);
  rb.init(a.B, a.ldb, a.N, n0, a.K, lane);
  f32x4 acc[MB][NB] = {};
  rowblock_loop<ES, MB, NB, W, U>(acc, ra, rb, a.K, wave, lane);
  rowblock_join<MB, NB, W>(acc, part, wave, lane, [&](int mb, int nb, V sum) {
    const int64_t m = m0 + 16 * mb + (lane & 15), n = n0 + 16 * nb + 4 * (lane >> 4);
    if (m >= a.M || n >= a.N) return;
    const float sa = s.a_scale[m];
    f32x4 v;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      v[c] = n + c < a.N ? (float)sum[c] * sa * s.b_scale[n + c] : 0.0f;
      if constexpr (kInt) v[c] += s.bias && n + c < a.N ? s.bias[n + c] : 0.0f;
    }
    store4(static_cast<unsigned short*>(a.D) + m * a.ldd + n, a.N - n, v);
  });
}

// TM x TN tiles (midtile.hpp), a workgroup for each of a tile's `splits`
// ranges of K stages.  With one it stores the result; with more each stores
// its fp32 sums in register order, and scaled_join adds them up.
template <MidMul MUL, int TM, int TN, int SLOTS>
__global__ __launch_bounds__(256, TM * TN <= 64 * 64 ? 4 : (TM * TN <= 64 * 128 || SLOTS == 2 ? 2 : 1)) void scaled_mid(ScaledArgs s) {
  typedef MidGeom<TM, TN, SLOTS> G;
  const int lane = threadIdx.x & 63, wave = wave_id();
  const KernelArgs& a = s.gemm;
  const int tiles_m = (int)((a.M + TM - 1) / TM), tiles_n = (int)((a.N + TN - 1) / TN);
  const int slot = persistent_slot(blockIdx.x, gridDim.x), tiles = tiles_m * tiles_n;
  const int split = slot / tiles, tile = slot - split * tiles;
  const MidTile t = mid_tile(tile, tiles_m, tiles_n);
  const int stages = (int)((a.K + kStageKBytes - 1) / kStageKBytes);
  const int k0 = (int)((int64_t)stages * split / s.splits), k1 = (int)((int64_t)stages * (split + 1) / s.splits);
  const int64_t kend = (int64_t)k1 * kStageKBytes < a.K ? (int64_t)k1 * kStageKBytes : a.K;
  MidAccum<G::kBM, G::kBN> acc;
  mid_loop<1, true, true, TM, TN, SLOTS, MUL>(acc, a, (int64_t)t.tm * TM, (int64_t)t.tn * TN, wave, lane, k0,
                                                k1 - k0, kend);
  const int64_t m0 = (int64_t)t.tm * TM + (wave >> 1) * 32 * G::kBM;
  const int64_t n0 = (int64_t)t.tn * TN + (wave & 1) * 32 * G::kBN;
  if (s.splits > 1) {
    mid_put(s.partials, slot, acc, wave, lane);
    return;
  }
  Scales<G::kBM, G::kBN, MUL == kMulInt8> scales;
  scales.load(s, m0, n0, lane);
  mid_store<G::kBM, G::kBN>(
      a.D, a.ldd, a.M, a.N, m0, n0, wave, lane,
      [&](int bi, int bj, int q) {
        const f32x16& v = acc.v[bi][bj];
        return scales.apply(f32x4{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]}, bi, bj, q);
      },
      [](int64_t r) { return r; });
}

// The splits' sums of one 32 x 32 block, added in order, scaled and stored: a
// wave a block.
template <bool INT8, int TM, int TN>
__global__ __launch_bounds__(64) void scaled_join(ScaledArgs s) {
  constexpr int BM = TM / 64, BN = TN / 64;
  const int lane = threadIdx.x;
  const KernelArgs& a = s.gemm;
  const int tiles_m = (int)((a.M + TM - 1) / TM), tiles_n = (int)((a.N + TN - 1) / TN);
  const int part = blockIdx.x % (4 * BM * BN), tile = blockIdx.x / (4 * BM * BN);
  const int wave = part / (BM * BN), block = part % (BM * BN);
  const MidTile t = mid_tile(tile, tiles_m, tiles_n);
  const int64_t m0 = (int64_t)t.tm * TM + (wave >> 1) * 32 * BM + 32 * (block / BN);
  const int64_t n0 = (int64_t)t.tn * TN + (wave & 1) * 32 * BN + 32 * (block % BN);
  if (m0 >= a.M || n0 >= a.N) return;
  Scales<1, 1, INT8> scales;
  scales.load(s, m0, n0, lane);
  MidAccum<1, 1> acc = {};
  for (int i = 0; i < s.splits; ++i) mid_add<BM, BN, INT8>(s.partials, i * tiles_m * tiles_n + tile, acc, wave, block, lane);
  const int64_t m = m0 + (lane & 31);
  if (m >= a.M) return;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int64_t n = n0 + 8 * q + 4 * (lane >> 5);
    const f32x16& v = acc.v[0][0];
    const f32x4 x = scales.apply(f32x4{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]}, 0, 0, q);
    store4(static_cast<unsigned short*>(a.D) + m * a.ldd + n, a.N - n, x);
  }
}

// The kernels a product can take: TM x TN tiles, one a workgroup (256 x 256 and
// 192 x 256: one after another).  join: the tile's K may be split.
struct Variant {
  int tm, tn, threads, lds;
  void (*kernel)(ScaledArgs);
  void (*join)(ScaledArgs);
  int per_cu;  // tiles a compute unit takes at once, for the cost
  // What its tiles cost (cost_of), in microseconds: a K stage of 128 with one
  // tile a compute unit and with two, and a tile besides; of a rows variant the
  // bytes that a compute unit takes in in one, and the launch besides.
  double stage1, stage2, tile;
};
template <MidMul MUL, int BM>
constexpr Variant tile_variant(double stage, double tile) {
  return {64 * BM, kTileN, kThreads, kPlainLdsBytes, scaled_tile<MUL, BM>, nullptr, 1, stage, stage, tile};
}
template <int ES, int MB, int NB, int W, int U>
constexpr Variant rows_variant(int per_cu, double bytes = 52e3, double launch = 0) {
  return {16 * MB, 16 * NB, 64 * W, 0, scaled_rows<ES, MB, NB, W, U>, nullptr, per_cu, bytes, bytes, launch};
}
template <MidMul MUL, int TM, int TN, int SLOTS>
constexpr Variant mid_variant(int per_cu, double stage1, double stage2, double tile) {
  return {TM, TN, 256, (int)MidGeom<TM, TN, SLOTS>::kLds, scaled_mid<MUL, TM, TN, SLOTS>,
          MUL == kMulExact ? nullptr : scaled_join<MUL == kMulInt8, TM, TN>, per_cu, stage1, stage2, tile};
}
// A table of variants starts with these, then has its mid variants.
enum { kTile256, kTile192, kRowsFirst, kRowsLast = 5, kMidFirst };

inline int64_t tiles_of(const Variant& v, int64_t M, int64_t N) {
  return ((M + v.tm - 1) / v.tm) * ((N + v.tn - 1) / v.tn);
}
// What the costs of a table's variants share.
struct CostModel {
  int last;          // the last variant that is chosen by its cost
  double memory;     // bytes a microsecond
  // Rows variants: the part of the lesser of memory's and the compute unit's
  // time that the greater does not hide; a round of two tiles a unit, besides.
  // (existing: of a tile's rows only those that the matrix has are read.)
  double overlap, round;
  bool existing;
  double join, put;  // a split's: microseconds, and bytes of the sums a microsecond
};
// Microseconds that a kernel takes, after what the launch takes.
inline double cost_of(const CostModel& m, const Variant* variants, int variant, int64_t M, int64_t N, int64_t K,
                      int splits, int cu_count) {
  const Variant& v = variants[variant];
  const double tiles = (double)tiles_of(v, M, N), cus = cu_count;
  const double memory = ((double)M * K + (double)N * K + 2.0 * M * N) / m.memory;
  if (variant >= kRowsFirst && variant <= kRowsLast) {
    // What a compute unit takes in, and the memory; they overlap in part.
    const double rounds = tiles <= cus ? 1.0 : (v.per_cu == 1 ? ceil(tiles / cus) : tiles / cus);
    const double rows = m.existing && M < v.tm ? M : v.tm;
    const double cu = rounds * (rows + v.tn) * K / v.stage1;
    return (cu > memory ? cu + m.overlap * memory : memory + m.overlap * cu) + m.round * ceil(tiles / (2 * cus)) +
           v.tile;
  }
  const double stages = ceil(ceil(K / 128.0) / splits), items = tiles * splits;
  const double at_once = v.per_cu * cus, full = floor(items / at_once), rest = items - full * at_once;
  double t = full * (stages * v.stage2 + v.tile);
  if (rest > 0) t += stages * (rest <= cus ? v.stage1 : v.stage2) + v.tile;
  t = t > memory ? t : memory;
  if (splits > 1) t += m.join + 2 * items * v.tm * v.tn * 4 / m.put;  // scaled_join, and its sums to memory and back
  return t;
}

// The variant that costs least.
inline ScaledChoice cheapest_variant(const CostModel& model, const Variant* variants, int64_t M, int64_t N, int64_t K,
                                     int cu_count) {
  ScaledChoice best = {kTile256, 1, kTileM, 0};
  double least = 1e300;
  // (Past 2^30 results only the large tiles, whose count stays within 31 bits.)
  const int last = (double)M * N > 1e9 ? kTile192 : model.last;
  for (int i = kTile256; i <= last; ++i)
    for (int splits : {1, 2, 3, 4, 6, 8, 12, 16}) {
      if (splits > 1 && (i < kMidFirst || K < 128 * 3 * splits)) break;
      const double cost = cost_of(model, variants, i, M, N, K, splits, cu_count);
      if (cost >= least) continue;
      least = cost;
      best = {i, splits, kTileM, 0};
    }
  const Variant& v = variants[best.variant];
  best.tile_m = v.tm;
  if (best.splits > 1) best.workspace_bytes = tiles_of(v, M, N) * best.splits * v.tm * v.tn * 4;
  return best;
}

// A variant's stages of K in LDS (0: none).
inline int lds_stages(const Variant* variants, int variant) {
  const Variant& v = variants[variant];
  return variant <= kTile192 ? kStages : v.lds / ((v.tm + v.tn) * (int)kStageKBytes);
}

template <int COUNT>
hipError_t prepare_variants(const Variant (&variants)[COUNT]) {
  for (const Variant& v : variants) {
    if (v.lds == 0) continue;
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(v.kernel),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, v.lds);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

inline hipError_t launch_variant(const Variant& v, bool persistent, const ScaledArgs& all, int cu_count,
                                 hipStream_t stream) {
  ScaledArgs s = all;
  // A launch holds fewer than 2^32 threads: columns in slabs (of whole tiles)
  // where one tile a workgroup would take more.
  const int64_t tiles_m = tiles_of(v, all.gemm.M, 1), tiles_n = tiles_of(v, 1, all.gemm.N);
  int64_t slab = tiles_n;
  if (!persistent && tiles_m * tiles_n * s.splits > ((int64_t)1 << 31) / v.threads) {
    slab = ((int64_t)1 << 31) / v.threads / (tiles_m * s.splits);
    slab = slab < 1 ? 1 : slab;
  }
  for (int64_t first = 0; first < tiles_n; first += slab) {
    const int64_t col = first * v.tn, left = all.gemm.N - col;
    s.gemm.N = left < slab * v.tn ? left : slab * v.tn;
    s.gemm.B = static_cast<const unsigned char*>(all.gemm.B) + col * all.gemm.ldb;
    s.gemm.b_bytes = (s.gemm.N - 1) * s.gemm.ldb + s.gemm.K;
    s.gemm.D = static_cast<unsigned short*>(all.gemm.D) + col;
    s.b_scale = all.b_scale + col;
    if (all.bias) s.bias = all.bias + col;
    const int64_t tiles = tiles_of(v, s.gemm.M, s.gemm.N);
    const int64_t grid = persistent ? (tiles < cu_count ? tiles : cu_count) : tiles * s.splits;
    hipLaunchKernelGGL(v.kernel, dim3((uint32_t)grid), dim3(v.threads), v.lds, stream, s);
    hipError_t e = hipGetLastError();
    if (e == hipSuccess && s.splits > 1) {
      hipLaunchKernelGGL(v.join, dim3((uint32_t)(tiles * (v.tm / 32) * (v.tn / 32))), dim3(64), 0, stream, s);
      e = hipGetLastError();
    }
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace
}  // namespace migemm

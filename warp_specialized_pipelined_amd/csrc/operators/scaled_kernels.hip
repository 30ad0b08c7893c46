// scaled_kernels.hip -- the product of 8-bit rows with a scale per row and
// per output channel:
//   d[m][n] = bf16(a_scale[m] b_scale[n] sum_k a[m][k] b[n][k])
// a and b are e4m3 codes, K-contiguous; the sum is fp32.
//
// scaled_tile: 256 x 256 or 192 x 256 tiles with the GEMM's K loop, where the
// product fills the chip with them (bound by the matrix instructions and the
// power they take: 8192 x 8192 x 16384 in 786 us, 2.80 PFLOP/s; 4000 x 3000 x
// 5000 in 62 us with 192 rows a tile, 252 tiles for 256 compute units, against
// 66 with 256 rows, 192 tiles).  scaled_mid: smaller tiles, their K split
// where there are few (bound by loads into LDS; 40 x 16384 x 8192 in 33 us,
// 4.1 TB/s of weights).  scaled_rows: tiles of 16 to 64 rows whose waves split
// K (bound by reading the weights, or by latency; 1 x 8192 x 8192 in 12.6 us,
// 5.3 TB/s).
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
template <int BM, int BN>
struct Scales {
  float rows[BM];
  f32x4 cols[BN][4];
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
  }
  __device__ __forceinline__ f32x4 apply(f32x4 v, int bi, int bj, int q) const {
#pragma unroll
    for (int c = 0; c < 4; ++c) v[c] = v[c] * rows[bi] * cols[bj][q][c];
    return v;
  }
};

// 64 BM x 256 tiles, one after another.
template <int BM>
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
    mainloop<1, true, true, BM>(acc, a, t.tm, t.tn, wave, lane, none);
    const int64_t m0 = (int64_t)t.tm * (64 * BM) + (wave >> 1) * (32 * BM);
    const int64_t n0 = (int64_t)t.tn * kTileN + (wave & 1) * kWaveTile;
    Scales<BM, 4> scales;
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
  __shared__ f32x4 part[W * MB * NB * 64];
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
  rowblock_join<MB, NB, W>(acc, part, wave, lane, [&](int mb, int nb, f32x4 v) {
    const int64_t m = m0 + 16 * mb + (lane & 15), n = n0 + 16 * nb + 4 * (lane >> 4);
    if (m >= a.M || n >= a.N) return;
    const float sa = s.a_scale[m];
#pragma unroll
    for (int c = 0; c < 4; ++c) v[c] = n + c < a.N ? v[c] * sa * s.b_scale[n + c] : 0.0f;
    store4(static_cast<unsigned short*>(a.D) + m * a.ldd + n, a.N - n, v);
  });
}

// TM x TN tiles (midtile.hpp), a workgroup for each of a tile's `splits`
// ranges of K stages.  With one it stores the result; with more each stores
// its fp32 sums in register order, and scaled_join adds them up.
template <bool EXACT, int TM, int TN, int SLOTS>
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
  mid_loop<1, true, true, TM, TN, SLOTS, EXACT>(acc, a, (int64_t)t.tm * TM, (int64_t)t.tn * TN, wave, lane, k0,
                                                k1 - k0, kend);
  const int64_t m0 = (int64_t)t.tm * TM + (wave >> 1) * 32 * G::kBM;
  const int64_t n0 = (int64_t)t.tn * TN + (wave & 1) * 32 * G::kBN;
  if (s.splits > 1) {
    mid_put(s.partials, slot, acc, wave, lane);
    return;
  }
  Scales<G::kBM, G::kBN> scales;
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
template <int TM, int TN>
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
  Scales<1, 1> scales;
  scales.load(s, m0, n0, lane);
  MidAccum<1, 1> acc = {};
  for (int i = 0; i < s.splits; ++i) mid_add<BM, BN>(s.partials, i * tiles_m * tiles_n + tile, acc, wave, block, lane);
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

// The kernels a product can take: TM x TN tiles, one a workgroup (256 x 256:
// one after another).  join: the tile's K may be split.  128 x 128 comes
// twice: a ring of four slots, one workgroup a compute unit, hides the loads'
// latency where there is one tile a unit (424 x 6578 x 7971: 51 us, 58 with
// two slots); two slots, two workgroups a unit, each loading while the other
// multiplies, where there are more (1600 x 4000 x 16000: 125 us, 149 with 192
// rows a tile, 165 with 64 x 128; 2773 x 2191 x 552: 15.0, 25.6 and 18.4).
struct Variant {
  int tm, tn, threads, lds;
  void (*kernel)(ScaledArgs);
  void (*join)(ScaledArgs);
  int per_cu;  // tiles a compute unit takes at once, for the cost
  // What its tiles cost (choose_scaled), in microseconds: a K stage of 128
  // with one tile a compute unit and with two, and a tile besides.
  double stage1, stage2, tile;
};
template <int ES, int MB, int NB, int W, int U>
constexpr Variant rows_variant(int per_cu) {
  return {16 * MB, 16 * NB, 64 * W, 0, scaled_rows<ES, MB, NB, W, U>, nullptr, per_cu, 0, 0, 0};
}
template <bool EXACT, int TM, int TN, int SLOTS>
constexpr Variant mid_variant(int per_cu, double stage1, double stage2, double tile) {
  return {TM, TN, 256, (int)MidGeom<TM, TN, SLOTS>::kLds, scaled_mid<EXACT, TM, TN, SLOTS>,
          EXACT ? nullptr : scaled_join<TM, TN>, per_cu, stage1, stage2, tile};
}
enum { kTile256, kTile192, kRowsFirst, kRowsLast = 5, kMidFirst, kMidLast = 9, kExactRows, kExactMid };
const Variant kVariants[] = {
    {kTileM, kTileN, kThreads, kPlainLdsBytes, scaled_tile<4>, nullptr, 1, 1.1, 1.1, 7.0},
    {kTileMShort, kTileN, kThreads, kPlainLdsBytes, scaled_tile<3>, nullptr, 1, 0.95, 0.95, 6.0},
    rows_variant<1, 1, 1, 16, 2>(1),
    rows_variant<1, 1, 2, 16, 1>(2),
    rows_variant<1, 2, 2, 8, 1>(2),
    rows_variant<1, 4, 2, 8, 1>(2),
    mid_variant<false, 64, 64, 4>(2, 0.30, 0.48, 1.7),
    mid_variant<false, 64, 128, 3>(2, 0.43, 0.64, 1.3),
    mid_variant<false, 128, 128, 4>(1, 0.52, 0.52, 2.4),
    mid_variant<false, 128, 128, 2>(2, 0.60, 0.80, 2.0),
    rows_variant<kExactE4M3, 1, 4, 2, 1>(2),
    mid_variant<true, 64, 64, 2>(2, 0, 0, 0),
};

int64_t tiles_of(const Variant& v, int64_t M, int64_t N) {
  return ((M + v.tm - 1) / v.tm) * ((N + v.tn - 1) / v.tn);
}
// Microseconds that v's kernel takes, after what the launch takes.
double cost_of(const Variant& v, bool rows, int64_t M, int64_t N, int64_t K, int splits, int cu_count) {
  const double tiles = (double)tiles_of(v, M, N), cus = cu_count;
  const double memory = ((double)M * K + (double)N * K + 2.0 * M * N) / 5.5e6;
  if (rows) {
    // What a compute unit takes in, and the memory; they overlap in part.
    const double rounds = tiles <= cus ? 1.0 : (v.per_cu == 1 ? ceil(tiles / cus) : tiles / cus);
    const double cu = rounds * (v.tm + v.tn) * K / 52e3;
    return (cu > memory ? cu + 0.26 * memory : memory + 0.26 * cu) + 0.6 * ceil(tiles / (2 * cus));
  }
  const double stages = ceil(ceil(K / 128.0) / splits), items = tiles * splits;
  const double at_once = v.per_cu * cus, full = floor(items / at_once), rest = items - full * at_once;
  double t = full * (stages * v.stage2 + v.tile);
  if (rest > 0) t += stages * (rest <= cus ? v.stage1 : v.stage2) + v.tile;
  t = t > memory ? t : memory;
  if (splits > 1) t += 4.0 + 2 * items * v.tm * v.tn * 4 / 5.2e6;  // scaled_join, and its sums to memory and back
  return t;
}

}  // namespace

// The kernel that costs least: the figures are a fit to 690 products of 1 to
// 8192 rows, 64 to 8192 columns and K of 257 to 16384, each timed with every
// kernel and up to 16 splits; what it picks is 2.5% slower than the fastest
// of them on average.
ScaledChoice choose_scaled(int64_t M, int64_t N, int64_t K, int cu_count) {
  // Short sums in exact products (rowblock.hpp): up to here fp32's own bound, K
  // 2^-23 of the sum of magnitudes, is about what the e4m3 instructions lose of
  // normal values, 1e-5 and at most 3e-5 of it.  Few results pay nothing for it
  // (300 x 2000 x 128: 4.9 us, 4.8 in e4m3; 16 x 8192 x 256: 4.5 and 4.7), many
  // up to twice the time (2000 x 4096 x 256: 15.6 and 8.3; 8192 x 8192 x 256: 85
  // and 44).  Further up it would be two to three times (16 x 8192 x 4096: 15.8
  // and 9.4; 2000 x 4096 x 1024: 31.5 and 13.5), where longer sums average the
  // loss out.
  if (K <= 256) return {M <= 16 ? kExactRows : kExactMid, 1, kTileM, 0};
  ScaledChoice best = {kTile256, 1, kTileM, 0};
  double least = 1e300;
  // (Past 2^30 results only the large tiles, whose count stays within 31 bits.)
  const int last = (double)M * N > 1e9 ? kTile192 : kMidLast;
  for (int i = kTile256; i <= last; ++i)
    for (int splits : {1, 2, 3, 4, 6, 8, 12, 16}) {
      if (splits > 1 && (i < kMidFirst || K < 128 * 3 * splits)) break;
      const double cost =
          cost_of(kVariants[i], i >= kRowsFirst && i <= kRowsLast, M, N, K, splits, cu_count);
      if (cost >= least) continue;
      least = cost;
      best = {i, splits, kTileM, 0};
    }
  const Variant& v = kVariants[best.variant];
  best.tile_m = v.tm;
  if (best.splits > 1) best.workspace_bytes = tiles_of(v, M, N) * best.splits * v.tm * v.tn * 4;
  return best;
}

ScaledKernel scaled_kernel(int variant) {
  const Variant& v = kVariants[variant];
  const int stages = variant <= kTile192 ? kStages : v.lds / ((v.tm + v.tn) * (int)kStageKBytes);
  return {v.tm, v.tn, stages, variant >= kExactRows};
}

hipError_t prepare_scaled() {
  for (const Variant& v : kVariants) {
    if (v.lds == 0) continue;
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(v.kernel),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, v.lds);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_scaled(const ScaledArgs& all, int variant, int cu_count, hipStream_t stream) {
  const Variant& v = kVariants[variant];
  ScaledArgs s = all;
  // A launch holds fewer than 2^32 threads: columns in slabs (of whole tiles)
  // where one tile a workgroup would take more.
  const int64_t tiles_m = tiles_of(v, all.gemm.M, 1), tiles_n = tiles_of(v, 1, all.gemm.N);
  int64_t slab = tiles_n;
  if (variant > kTile192 && tiles_m * tiles_n * s.splits > ((int64_t)1 << 31) / v.threads) {
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
    const int64_t tiles = tiles_of(v, s.gemm.M, s.gemm.N);
    const int64_t grid = variant <= kTile192 ? (tiles < cu_count ? tiles : cu_count) : tiles * s.splits;
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

}  // namespace migemm

// checkpoint_kernels.hip -- activations kept in 8 bits for the backward pass,
// and the weights' gradient from them.
//
// The kept form: e4m3 codes with a power of two for each 32 tokens of a column,
//   x ~ code 2^(e - 127),   e the least with max |x| <= 448 2^(e - 127)
// (18 <= e <= 246, so that code and power multiply exactly in bf16).  The
// groups run along the tokens because that is what the weights' gradient sums
// over, and because a model's large activations stand in a few columns.  A
// column's 16 tokens lie together (16 bytes): what a lane of a matrix
// instruction takes.
//
//   dw[n][k] = sum over tokens of dy[t][n] code[t][k] 2^(e[t / 32][k] - 127)
// on the bf16 instructions: the products are exact, the sums fp32.
//
// Packing is bound by memory (3 bytes an element: 8192 x 8192 42 us, 4.8 TB/s;
// 48 with 16-byte stores of each lane's own columns, which leave lines half
// written), unpacking too (40 us).  The gradient: kepttile.hpp; 8192^3 to fp32
// 810 us, 1.36 PFLOP/s, and 880 added to what is there (2048 x 4096 x 11008: 169
// and 228), which each tile reads behind its products.
#include <hip/hip_runtime.h>

#include <math.h>

#include "../kernel/gfx950.hpp"
#include "../kernel/scheduler.hpp"
#include "kepttile.hpp"
#include "operators.h"
#include "rows.hpp"

namespace migemm {
namespace {

typedef short i16x2 __attribute__((ext_vector_type(2)));

// A group's exponent from its largest magnitude (a bf16 pattern of at most
// 0x7F60, 1.75 2^127).
__device__ __forceinline__ uint32_t exponent_of(uint32_t top) {
  const int e = (int)(top >> 7) - 8 + ((top & 0x7F) > 0x60 ? 1 : 0);
  return (uint32_t)(e < 18 ? 18 : (e > 246 ? 246 : e));
}
__device__ __forceinline__ float power_of(uint32_t e) { return __uint_as_float(e << 23); }

// A wave's item: tokens of a group x 64 COLS columns, numbered along the columns
// first; lane l holds columns COLS l .. + COLS - 1 of them.
template <int COLS>
struct PackItem {
  int64_t group, col;
  __device__ __forceinline__ PackItem(int64_t item, int64_t ld, int lane) {
    const int64_t across = (ld + 64 * COLS - 1) / (64 * COLS);
    group = item / across;
    col = ((item - group * across) * 64 + lane) * COLS;
  }
};

// 32 tokens x 256 columns, four a lane.
constexpr int kPackCols = 4;
typedef uint32_t pack_words __attribute__((ext_vector_type(kPackCols / 2)));
typedef uint32_t pack_bytes __attribute__((ext_vector_type(kPackCols / 4)));
__device__ __forceinline__ void pack_item(const CheckpointArgs& a, int64_t item, int lane) {
  constexpr int W = kPackCols / 2;
  const PackItem<kPackCols> at(item, a.ld, lane);
  const int64_t c = at.col, t0 = at.group * 32;
  const unsigned short* x = static_cast<const unsigned short*>(a.x) + t0 * a.x_rs + c;
  pack_words v[32];
#pragma unroll
  for (int t = 0; t < 32; ++t) {
    v[t] = pack_words{};
    if (t0 + t < a.tokens && c < a.cols) v[t] = *reinterpret_cast<const pack_words*>(x + t * a.x_rs);
  }
  // (Columns past the last: their bytes may hold anything.)
  if (a.cols - c < kPackCols) {
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const int64_t left = a.cols - c - 2 * w;
      const uint32_t keep = left >= 2 ? 0xFFFFFFFFu : (left == 1 ? 0xFFFFu : 0u);
#pragma unroll
      for (int t = 0; t < 32; ++t) v[t][w] &= keep;
    }
  }
  uint32_t exponents[kPackCols];
#pragma unroll
  for (int w = 0; w < W; ++w) {
    uint32_t top = 0;
#pragma unroll
    for (int t = 0; t < 32; ++t) top = max_u16x2(top, v[t][w] & 0x7FFF7FFFu);
    if ((top & 0xFFFFu) > 0x7F60u || (top >> 16) > 0x7F60u) {
      // Infinities and NaN become NaN and leave the group's power to the rest;
      // what is past 1.75 2^127 becomes that.
      top = 0;
#pragma unroll
      for (int t = 0; t < 32; ++t) {
        const uint32_t m = v[t][w] & 0x7FFF7FFFu;
        uint32_t o = 0, f = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t b = (m >> (16 * h)) & 0xFFFFu;
          b = b >= 0x7F80u ? 0x7FC0u : (b > 0x7F60u ? 0x7F60u : b);
          o |= b << (16 * h);
          f |= (b >= 0x7F80u ? 0u : b) << (16 * h);
        }
        v[t][w] = o | (v[t][w] & 0x80008000u);
        top = max_u16x2(top, f);
      }
    }
    exponents[2 * w] = exponent_of(top & 0xFFFFu);
    exponents[2 * w + 1] = exponent_of(top >> 16);
  }
  // A lane's chunks (16 tokens of a column) go through LDS, so that the stores of
  // a wave are whole lines: chunk h of lane l is at C l + (h + l / (16 / C)) % C,
  // which spreads 16 lanes over all banks both when it is written and when lane
  // i reads column 64 s + i.
  constexpr int C = kPackCols;
  __shared__ u32x4 chunks[64 * C];
  auto place = [](int l, int h) { return C * l + ((h + l / (16 / C)) & (C - 1)); };
  const int64_t first = c - C * lane;
#pragma unroll
  for (int g = 0; g < 2; ++g) {
    if (g > 0) __syncthreads();
#pragma unroll
    for (int h = 0; h < C; ++h) {
      const float scale = power_of(exponents[h]);
      const uint32_t sel = h & 1 ? 0x07060302u : 0x05040100u;
      u32x4 o;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int t = 16 * g + 4 * q;
        const uint32_t p0 = __builtin_amdgcn_perm(v[t + 1][h / 2], v[t][h / 2], sel);
        const uint32_t p1 = __builtin_amdgcn_perm(v[t + 3][h / 2], v[t + 2][h / 2], sel);
        i16x2 d = {0, 0};
        d = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(d, __builtin_bit_cast(bf16x2, p0), scale, false);
        d = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(d, __builtin_bit_cast(bf16x2, p1), scale, true);
        o[q] = __builtin_bit_cast(uint32_t, d);
      }
      chunks[place(lane, h)] = o;
    }
    __syncthreads();
    u32x4* codes = reinterpret_cast<u32x4*>(a.codes) + (t0 / 16 + g) * a.ld + first;
#pragma unroll
    for (int s = 0; s < C; ++s)
      if (first + 64 * s + lane < a.ld) codes[64 * s + lane] = chunks[place((64 * s + lane) / C, lane & (C - 1))];
  }
  __syncthreads();
  if (c < a.ld) {
    pack_bytes e;
#pragma unroll
    for (int w = 0; w < C / 4; ++w)
      e[w] = exponents[4 * w] | exponents[4 * w + 1] << 8 | exponents[4 * w + 2] << 16 | exponents[4 * w + 3] << 24;
    *reinterpret_cast<pack_bytes*>(a.scales + at.group * a.ld + c) = e;
  }
}
__global__ __launch_bounds__(64) void checkpoint_pack(CheckpointArgs a, int64_t items) {
  for (int64_t i = blockIdx.x; i < items; i += gridDim.x) pack_item(a, i, threadIdx.x);
}

__device__ __forceinline__ uint32_t two_bf16(uint32_t codes, float scale, bool upper) {
  return __builtin_bit_cast(uint32_t, upper ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, scale, true)
                                            : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, scale, false));
}

// 16 tokens x 256 columns, four a lane.
constexpr int kUnpackCols = 4;
__device__ __forceinline__ void unpack_item(const CheckpointArgs& a, int64_t item, int lane) {
  const PackItem<kUnpackCols> at(item, a.ld, lane);
  const int64_t c = at.col, t0 = at.group * 16;
  if (c >= a.cols) return;
  const u32x4* codes = reinterpret_cast<const u32x4*>(a.codes) + at.group * a.ld + c;
  const uint32_t exponents = *reinterpret_cast<const uint32_t*>(a.scales + (at.group / 2) * a.ld + c);
  u32x4 v[kUnpackCols];
#pragma unroll
  for (int i = 0; i < kUnpackCols; ++i) v[i] = codes[i];
  unsigned short* x = static_cast<unsigned short*>(a.x_out) + t0 * a.x_rs + c;
  const int64_t left = a.cols - c;
#pragma unroll
  for (int t = 0; t < 16; t += 2) {
    uint32_t p[kUnpackCols];  // tokens t and t + 1 of a column
#pragma unroll
    for (int i = 0; i < kUnpackCols; ++i)
      p[i] = two_bf16(v[i][t >> 2], power_of((exponents >> (8 * i)) & 0xFFu), t & 2);
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      if (t0 + t + s >= a.tokens) continue;
      const uint32_t sel = s ? 0x07060302u : 0x05040100u;
      const u32x2 o = {__builtin_amdgcn_perm(p[1], p[0], sel), __builtin_amdgcn_perm(p[3], p[2], sel)};
      unsigned short* d = x + (t + s) * a.x_rs;
      if (left >= 4) {
        *reinterpret_cast<u32x2*>(d) = o;
      } else {
        for (int e = 0; e < (int)left; ++e) d[e] = (unsigned short)(o[e >> 1] >> (16 * (e & 1)));
      }
    }
  }
}

__global__ __launch_bounds__(64) void checkpoint_unpack(CheckpointArgs a, int64_t items) {
  for (int64_t i = blockIdx.x; i < items; i += gridDim.x) unpack_item(a, i, threadIdx.x);
}

// TM x TN tiles of dw (kepttile.hpp), a workgroup for each of a tile's `splits`
// ranges of the tokens.  With one it stores the result; with more each stores
// its fp32 sums in register order, and kept_join adds them up.
template <int TM, int TN, int SLOTS, int WM, int WN, int PER_SIMD>
__global__ __launch_bounds__(64 * WM * WN, PER_SIMD) void kept_gradient(CheckpointArgs a) {
  typedef KeptGeom<TM, TN, SLOTS, WM, WN> T;
  constexpr int BM = T::kBM, BN = T::kBN;
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int tiles_m = (int)((a.out_cols + TM - 1) / TM), tiles_n = (int)((a.cols + TN - 1) / TN);
  const int slot = persistent_slot(blockIdx.x, gridDim.x), tiles = tiles_m * tiles_n;
  const int split = slot / tiles, tile = slot - split * tiles;
  const MidTile t = mid_tile(tile, tiles_m, tiles_n);
  const int stages = (int)((a.tokens + kKeptTokens - 1) / kKeptTokens);
  const int k0 = (int)((int64_t)stages * split / a.splits), k1 = (int)((int64_t)stages * (split + 1) / a.splits);
  MidAccum<BM, BN> acc;
  kept_loop<TM, TN, SLOTS, WM, WN>(acc, a, (int64_t)t.tm * TM, (int64_t)t.tn * TN, wave, lane, k0, k1 - k0);
  if (a.splits > 1) {
    mid_put(a.partials, slot * (T::kWaves / 4) + wave / 4, acc, wave % 4, lane);
    return;
  }
  const int64_t m0 = (int64_t)t.tm * TM + wave / WN * 32 * BM;
  const int64_t n0 = (int64_t)t.tn * TN + wave % WN * 32 * BN;
  if (!a.fp32) {
    mid_store<BM, BN>(
        a.dw, a.dw_rs, a.out_cols, a.cols, m0, n0, wave, lane,
        [&](int bi, int bj, int q) {
          const f32x16& v = acc.v[bi][bj];
          return f32x4{v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
        },
        [](int64_t r) { return r; });
  } else if (a.accumulate) {
    kept_store32<BM, BN, true>(a, acc, m0, n0, wave, lane);
  } else {
    kept_store32<BM, BN, false>(a, acc, m0, n0, wave, lane);
  }
}

// The ranges' sums of one 32 x 32 block, added in order and stored: a wave a
// block.
template <int TM, int TN, int WM, int WN>
__global__ __launch_bounds__(64) void kept_join(CheckpointArgs a) {
  constexpr int BM = TM / (32 * WM), BN = TN / (32 * WN);
  const int lane = threadIdx.x;
  const int tiles_m = (int)((a.out_cols + TM - 1) / TM), tiles_n = (int)((a.cols + TN - 1) / TN);
  const int part = blockIdx.x % (WM * WN * BM * BN), tile = blockIdx.x / (WM * WN * BM * BN);
  const int wave = part / (BM * BN), block = part % (BM * BN);
  const MidTile t = mid_tile(tile, tiles_m, tiles_n);
  const int64_t m = (int64_t)t.tm * TM + wave / WN * 32 * BM + 32 * (block / BN) + (lane & 31);
  const int64_t n0 = (int64_t)t.tn * TN + wave % WN * 32 * BN + 32 * (block % BN);
  if (m - (lane & 31) >= a.out_cols || n0 >= a.cols) return;
  MidAccum<1, 1> acc = {};
#pragma unroll 4
  for (int i = 0; i < a.splits; ++i)
    mid_add<BM, BN>(a.partials, (int64_t)(i * tiles_m * tiles_n + tile) * (WM * WN / 4) + wave / 4, acc, wave % 4, block, lane);
  if (m >= a.out_cols) return;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int64_t n = n0 + 8 * q + 4 * (lane >> 5), left = a.cols - n;
    const f32x16& v = acc.v[0][0];
    const f32x4 x = {v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]};
    if (!a.fp32) {
      store4(static_cast<unsigned short*>(a.dw) + m * a.dw_rs + n, left, x);
    } else {
      float* d = static_cast<float*>(a.dw) + m * a.dw_rs + n;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (e < left) d[e] = a.accumulate ? d[e] + x[e] : x[e];
    }
  }
}

struct KeptVariant {
  int tm, tn, slots, threads, lds;
  void (*kernel)(CheckpointArgs);
  void (*join)(CheckpointArgs);
  // What its tiles cost (choose_checkpoint), in microseconds: a stage with one
  // tile a compute unit and with as many as fit, and a tile besides.
  int per_cu;
  double stage1, stage2, tile;
};
template <int TM, int TN, int SLOTS, int WM, int WN, int PER_SIMD>
constexpr KeptVariant kept_variant(int per_cu, double stage1, double stage2, double tile) {
  return {TM, TN, SLOTS, 64 * WM * WN, (int)KeptGeom<TM, TN, SLOTS, WM, WN>::kLds,
          kept_gradient<TM, TN, SLOTS, WM, WN, PER_SIMD>, kept_join<TM, TN, WM, WN>, per_cu, stage1, stage2, tile};
}
const KeptVariant kVariants[] = {
    kept_variant<256, 256, 3, 2, 4, 2>(1, 1.15, 1.10, 5.5),
    kept_variant<192, 256, 3, 2, 4, 2>(1, 0.83, 0.80, 5.0),
    kept_variant<128, 128, 3, 2, 2, 2>(2, 0.50, 0.70, 2.1),
    kept_variant<64, 64, 4, 2, 2, 3>(3, 0.27, 0.52, 1.3),
};
int64_t tiles_of(const KeptVariant& v, int64_t out_cols, int64_t cols) {
  return ((out_cols + v.tm - 1) / v.tm) * ((cols + v.tn - 1) / v.tn);
}

}  // namespace

// A launch holds fewer than 2^32 threads.
static uint32_t wave_grid(int64_t items) { return (uint32_t)(items < (1 << 25) ? items : 1 << 25); }

hipError_t launch_checkpoint_pack(const CheckpointArgs& a, hipStream_t stream) {
  const int64_t items = (a.tokens + 31) / 32 * ((a.ld + 64 * kPackCols - 1) / (64 * kPackCols));
  hipLaunchKernelGGL(checkpoint_pack, dim3(wave_grid(items)), dim3(64), 0, stream, a, items);
  return hipGetLastError();
}

hipError_t launch_checkpoint_unpack(const CheckpointArgs& a, hipStream_t stream) {
  const int64_t items = (a.tokens + 15) / 16 * ((a.ld + 64 * kUnpackCols - 1) / (64 * kUnpackCols));
  hipLaunchKernelGGL(checkpoint_unpack, dim3(wave_grid(items)), dim3(64), 0, stream, a, items);
  return hipGetLastError();
}

// The tiles and splits that cost least.  The figures are a fit to 1848 gradients
// of 1 to 8192 tokens and 64 to 8192 columns on either side, each timed with
// every kernel and up to 32 splits; what it picks is 0.7% slower than the fastest
// of them on average.
CheckpointChoice choose_checkpoint(int64_t tokens, int64_t cols, int64_t out_cols, int es, int cu_count) {
  CheckpointChoice best = {0, 1, 0};
  double least = 1e300;
  const double all = (double)((tokens + kKeptTokens - 1) / kKeptTokens), results = (double)cols * out_cols;
  for (int i = 0; i < (int)(sizeof(kVariants) / sizeof(kVariants[0])); ++i)
    for (int splits : {1, 2, 3, 4, 6, 8, 12, 16, 24, 32}) {
      const KeptVariant& v = kVariants[i];
      const double tiles = (double)tiles_of(v, out_cols, cols), items = tiles * splits;
      if (splits > 1 && (all < 3 * splits || items * v.tm * v.tn * 4 > (512 << 20))) break;
      // (A launch holds fewer than 2^32 threads; the largest tiles always fit.)
      if (items * v.threads > 4e9 && i > 0) break;
      const double stages = ceil(all / splits), at_once = (double)v.per_cu * cu_count;
      const double full = floor(items / at_once), rest = items - full * at_once;
      double t = full * (stages * v.stage2 + v.tile);
      if (rest > 0) t += stages * (rest <= cu_count ? v.stage1 : v.stage2) + v.tile;
      const double memory = ((double)tokens * cols + 2.0 * tokens * out_cols + es * results) / 5.4e6;
      t = t > memory ? t + 0.64 * memory : memory + 0.64 * t;  // they overlap in part
      if (splits > 1) t += 3.0 + 0.05 * splits + (2 * items * v.tm * v.tn * 4 + es * results) / 5.1e6;  // kept_join
      if (t >= least) continue;
      least = t;
      best = {i, splits, splits > 1 ? (int64_t)items * v.tm * v.tn * 4 : 0};
    }
  return best;
}

CheckpointKernel checkpoint_kernel(int variant) {
  const KeptVariant& v = kVariants[variant];
  return {v.tm, v.tn, v.slots};
}

hipError_t prepare_checkpoint() {
  for (const KeptVariant& v : kVariants) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(v.kernel),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, v.lds);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_checkpoint_gradient(const CheckpointArgs& a, int variant, hipStream_t stream) {
  const KeptVariant& v = kVariants[variant];
  const int64_t tiles = tiles_of(v, a.out_cols, a.cols);
  hipLaunchKernelGGL(v.kernel, dim3((uint32_t)(tiles * a.splits)), dim3(v.threads), v.lds, stream, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.splits == 1) return e;
  hipLaunchKernelGGL(v.join, dim3((uint32_t)(tiles * (v.tm / 32) * (v.tn / 32))), dim3(64), 0, stream, a);
  return hipGetLastError();
}

}  // namespace migemm

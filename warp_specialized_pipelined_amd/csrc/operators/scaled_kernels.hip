// scaled_kernels.hip -- the product of 8-bit rows with a scale per row and
// per output channel:
//   d[m][n] = bf16(a_scale[m] b_scale[n] sum_k a[m][k] b[n][k])
// a and b are e4m3 codes, K-contiguous; the sum is fp32.
//
// Two kernels.  scaled_tile: 256 x 256 tiles with the GEMM's K loop, where
// the product is large enough to fill the chip with them (bound by the matrix
// instructions).  scaled_rows: small tiles whose waves split K, for few rows
// or columns (bound by reading the weights, or by latency).
#include <hip/hip_runtime.h>

#include <type_traits>

#include "../kernel/epilogue.hpp"
#include "../kernel/gfx950.hpp"
#include "../kernel/mainloop.hpp"
#include "../kernel/params.hpp"
#include "../kernel/scheduler.hpp"
#include "operators.h"
#include "rowblock.hpp"
#include "tile_store.hpp"

namespace migemm {
namespace {

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
    mainloop<1, true, true>(acc, a, t.tm, t.tn, wave, lane, none);
    const int64_t m0 = (int64_t)t.tm * kTileM + (wave >> 1) * kWaveTile;
    const int64_t n0 = (int64_t)t.tn * kTileN + (wave & 1) * kWaveTile;
    // Scales past the matrix read as zero; what they scale is not stored.
    auto vec = [](const float* p, int64_t from, int64_t n) {
      int64_t left = (n - from) * 4;
      left = left < 0 ? 0 : (left > 512 ? 512 : left);
      return make_rsrc(p + from, (uint32_t)left);
    };
    const __amdgpu_buffer_rsrc_t ra = vec(s.a_scale, m0, a.M), rb = vec(s.b_scale, n0, a.N);
    float rows[4];
    f32x4 cols[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      rows[i] = __uint_as_float(
          __builtin_amdgcn_raw_buffer_load_b32(ra, (32 * i + (lane & 31)) * 4, 0, 0));
#pragma unroll
      for (int q = 0; q < 4; ++q)
        cols[i][q] = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                                   rb, (32 * i + 8 * q + 4 * (lane >> 5)) * 4, 0, 0));
    }
    tile_store<true>(a.D, a.ldd, a.M, a.N, m0, n0, wave, lane, [&](int bi, int bj, int q) {
      f32x4 v;
#pragma unroll
      for (int c = 0; c < 4; ++c) v[c] = acc.v[bi][bj][4 * q + c] * rows[bi] * cols[bj][q][c];
      return v;
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
    unsigned short* d = static_cast<unsigned short*>(a.D) + m * a.ldd + n;
    const float sa = s.a_scale[m];
    float o[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) o[c] = n + c < a.N ? v[c] * sa * s.b_scale[n + c] : 0.0f;
    const u32x2 w = {pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3])};
    if (n + 4 <= a.N) {
      *reinterpret_cast<u32x2*>(d) = w;
    } else {
      for (int c = 0; c < (int)(a.N - n); ++c) d[c] = (unsigned short)(w[c >> 1] >> (16 * (c & 1)));
    }
  });
}

// The variants of scaled_rows: 16-row blocks, 16-column blocks, waves.
struct RowsVariant {
  int mb, nb, waves;
  void (*kernel)(ScaledArgs);
};
const RowsVariant kRows[] = {
    {1, 1, 16, scaled_rows<1, 1, 1, 16, 2>},
    {2, 2, 8, scaled_rows<1, 2, 2, 8, 1>},
    {3, 2, 8, scaled_rows<1, 3, 2, 8, 1>},
    {4, 2, 8, scaled_rows<1, 4, 2, 8, 1>},
    {4, 4, 4, scaled_rows<1, 4, 4, 4, 1>},
    {1, 4, 2, scaled_rows<kExactE4M3, 1, 4, 2, 1>},
    {4, 4, 2, scaled_rows<kExactE4M3, 4, 4, 2, 1>},
};

}  // namespace

int scaled_variant(int64_t M, int64_t N, int64_t K, int cu_count) {
  // Short sums in exact products: with two K steps at most the time goes into
  // launch and output, whichever instruction multiplies.
  if (K <= 256) return M <= 16 ? 6 : 7;
  const int64_t tiles = ((M + kTileM - 1) / kTileM) * ((N + kTileN - 1) / kTileN);
  if (M > 64 && tiles * 2 >= cu_count) return 0;
  return M <= 16 ? 1 : (M <= 32 ? 2 : (M <= 48 ? 3 : (M <= 64 ? 4 : 5)));
}

hipError_t prepare_scaled() {
  return hipFuncSetAttribute(reinterpret_cast<const void*>(scaled_tile),
                             hipFuncAttributeMaxDynamicSharedMemorySize, kPlainLdsBytes);
}

hipError_t launch_scaled(const ScaledArgs& s, int variant, int grid, hipStream_t stream) {
  if (variant == 0) {
    hipLaunchKernelGGL(scaled_tile, dim3(grid), dim3(kThreads), kPlainLdsBytes, stream, s);
  } else {
    const RowsVariant& v = kRows[variant - 1];
    const int64_t tiles = ((s.gemm.M + 16 * v.mb - 1) / (16 * v.mb)) *
                          ((s.gemm.N + 16 * v.nb - 1) / (16 * v.nb));
    hipLaunchKernelGGL(v.kernel, dim3((uint32_t)tiles), dim3(64 * v.waves), 0, stream, s);
  }
  return hipGetLastError();
}

}  // namespace migemm

// tile_store.hpp -- a wave's 128 x 128 quarter of a 256 x 256 tile (BM = 3: 96
// x 128 of a 192 x 256 tile), each value transformed, rounded to bf16, staged through LDS and stored to a
// row-major matrix with 16-byte stores (the layout and the order of accesses
// are those of the GEMM's epilogue).
#pragma once

#include "../kernel/epilogue.hpp"

namespace migemm {

// value(bi, bj, q) gives the four results of row 32 bi + l % 32, columns
// 32 bj + 8 q + 4 (l / 32) .. + 3 of the wave's quarter.  NT: stores carry the
// non-temporal hint (for results not read again soon).
template <bool NT, int BM = 4, class Value>
__device__ __forceinline__ void tile_store(void* D, int64_t ldd, int64_t M, int64_t N, int64_t m0,
                                           int64_t n0, int wave, int lane, Value&& value) {
  const int lr = lane & 31, half = lane >> 5;
  const uint32_t st_base = wave * kStagingWaveBytes + lr * kStagingRowBytes + 8 * half;
#pragma unroll
  for (int bi = 0; bi < BM; ++bi)
#pragma unroll
    for (int bj = 0; bj < 4; ++bj)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const f32x4 v = value(bi, bj, q);
        const u32x2 w = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
        *(MIGEMM_LDS u32x2*)lds_at(st_base + 32 * bi * kStagingRowBytes + (4 * bj + q) * 16) = w;
      }
  // The wave reads back only what it wrote itself; its LDS accesses complete
  // in order.
  const __amdgpu_buffer_rsrc_t rd = matrix_rsrc(D, ldd, M, N, m0, n0, false);
  const int rsub = lane >> 4, chunk = lane & 15;
  const int64_t rows_left = M - m0, cols_left = N - n0 - 8 * chunk;
  const uint32_t rd_base = wave * kStagingWaveBytes + rsub * kStagingRowBytes + chunk * 16;
  const uint32_t d_lane = (uint32_t)((rsub * ldd + 8 * chunk) * 2);
#pragma unroll 8
  for (int i = 0; i < 8 * BM; ++i) {
    const u32x4 v = *(const MIGEMM_LDS u32x4*)lds_at(rd_base + 4 * i * kStagingRowBytes);
    const int row = 4 * i + rsub;
    if (row < rows_left && cols_left > 0) {
      const uint32_t off = d_lane + (uint32_t)(4 * i * ldd * 2);
      if (cols_left >= 8) {
        __builtin_amdgcn_raw_buffer_store_b128(v, rd, off, 0, NT ? kCpolNt : 0);
      } else {
        for (int e = 0; e < cols_left; ++e)
          __builtin_amdgcn_raw_buffer_store_b16((unsigned short)(v[e >> 1] >> (16 * (e & 1))), rd,
                                                off + 2 * e, 0, 0);
      }
    }
  }
}

}  // namespace migemm

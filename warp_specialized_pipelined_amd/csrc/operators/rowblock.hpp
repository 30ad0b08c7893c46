// rowblock.hpp -- small output tiles of a product of two K-contiguous
// operands, for few rows or few columns.
//
// A workgroup of W waves computes a tile of 16 MB rows by 16 NB columns.  The
// waves split K: wave w takes the 128-byte K steps w, w + W, ...  Each loads
// its fragments straight from global memory into registers -- no LDS, no
// barrier in the loop, so with many waves per compute unit enough loads are
// in flight to reach the memory's rate -- and at the end the W partial tiles
// are added through LDS, in the order of the waves.
//
// MFMA 16x16x128 (e4m3) or twice 16x16x32 (bf16) a step: lane l holds the
// 16-byte chunks l / 16 and 4 + l / 16 of its row's 128 bytes.  Which K the
// hardware takes a chunk for does not matter, as both operands use the same
// order.  As in the large tiles the product is formed as (B A^T), so a lane
// ends up with four consecutive columns of one row:
//   acc[mb][nb][c] = D[m0 + 16 mb + l % 16][n0 + 16 nb + 4 (l / 16) + c].
#pragma once

#include "../kernel/gfx950.hpp"

namespace migemm {

__device__ __forceinline__ f32x4 mfma_16(i32x4 b0, i32x4 b1, i32x4 a0, i32x4 a1, f32x4 c,
                                         std::integral_constant<int, 1>) {
  const i32x8 a = {a0[0], a0[1], a0[2], a0[3], a1[0], a1[1], a1[2], a1[3]};
  const i32x8 b = {b0[0], b0[1], b0[2], b0[3], b1[0], b1[1], b1[2], b1[3]};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(b, a, c, 0, 0, 0, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma_16(i32x4 b0, i32x4 b1, i32x4 a0, i32x4 a1, f32x4 c,
                                         std::integral_constant<int, 2>) {
  c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, b0),
                                              __builtin_bit_cast(bf16x8, a0), c, 0, 0, 0);
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, b1),
                                                 __builtin_bit_cast(bf16x8, a1), c, 0, 0, 0);
}

// e4m3 through bf16: every e4m3 value and every product of two is exact in
// the bf16 instructions, whose sums keep 24 bits.  The e4m3 instructions, both
// shapes, add the products of eight consecutive K first, each cut toward zero
// to a multiple of 2^(E - 13), where E is the largest sum of two exponents of
// the eight (measured: with two products of 448 x 448 that cancel, or of 256 x
// 256, what is beside them comes out as a multiple of 8; with 16 x 16 of 2^-5);
// the rest of the sum is fp32's.  Normal values lose up to 1e-5 of the sum of
// magnitudes by that at any K, values with a 448 in one octet of eight 1e-4.
__device__ __forceinline__ void widen(i32x4 x, i32x4& lo, i32x4& hi) {
  typedef float f32x2 __attribute__((ext_vector_type(2)));
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    const f32x2 p = __builtin_amdgcn_cvt_pk_f32_fp8(x[w], false);
    const f32x2 q = __builtin_amdgcn_cvt_pk_f32_fp8(x[w], true);
    // the upper halves: exact, an e4m3 value has 4 significant bits
    const int a = (int)__builtin_amdgcn_perm(__float_as_uint(p[1]), __float_as_uint(p[0]), 0x07060302u);
    const int b = (int)__builtin_amdgcn_perm(__float_as_uint(q[1]), __float_as_uint(q[0]), 0x07060302u);
    (w < 2 ? lo : hi)[2 * (w & 1)] = a;
    (w < 2 ? lo : hi)[2 * (w & 1) + 1] = b;
  }
}
constexpr int kExactE4M3 = 3;  // in place of an element size: e4m3 through bf16
constexpr int kInt8 = 4;       // and int8, whose int32 sums travel as fp32 bits
__device__ __forceinline__ f32x4 mfma_16(i32x4 b0, i32x4 b1, i32x4 a0, i32x4 a1, f32x4 c,
                                         std::integral_constant<int, kInt8>) {
  const i32x4 s = __builtin_amdgcn_mfma_i32_16x16x64_i8(b0, a0, __builtin_bit_cast(i32x4, c), 0, 0, 0);
  return __builtin_bit_cast(f32x4, __builtin_amdgcn_mfma_i32_16x16x64_i8(b1, a1, s, 0, 0, 0));
}
__device__ __forceinline__ f32x4 mfma_16(i32x4 b0, i32x4 b1, i32x4 a0, i32x4 a1, f32x4 c,
                                         std::integral_constant<int, kExactE4M3>) {
  const std::integral_constant<int, 2> bf16;
  i32x4 al, ah, bl, bh;
  widen(a0, al, ah);
  widen(b0, bl, bh);
  c = mfma_16(bl, bh, al, ah, c, bf16);
  widen(a1, al, ah);
  widen(b1, bl, bh);
  return mfma_16(bl, bh, al, ah, c, bf16);
}

// An operand's 16 NBLK rows from `row0` on: rows past the operand's last are
// read as the last one (their results are never stored).
template <int NBLK>
struct RowBlock {
  __amdgpu_buffer_rsrc_t rsrc;
  uint32_t off[NBLK];  // byte offset of the lane's row, and chunk l / 16
  __device__ __forceinline__ void init(const void* base, int64_t row_bytes, int64_t rows,
                                       int64_t row0, int64_t k_bytes, int lane) {
    const int64_t left = rows - 1 - row0;  // >= 0: the tile's first row exists
    int64_t bytes = left * row_bytes + ((k_bytes + 15) & ~(int64_t)15);
    bytes = bytes > 0x7FFFFFF0 ? 0x7FFFFFF0 : bytes;
    rsrc = make_rsrc(static_cast<const unsigned char*>(base) + row0 * row_bytes, (uint32_t)bytes);
#pragma unroll
    for (int i = 0; i < NBLK; ++i) {
      int64_t r = 16 * i + (lane & 15);
      r = r > left ? left : r;
      off[i] = (uint32_t)(r * row_bytes) + 16 * (lane >> 4);
    }
  }
  // Both chunks of K step `step`, or zeros where it is past the last whole one.
  __device__ __forceinline__ void load(int i, int step, bool valid, i32x4 (&v)[2]) const {
    const uint32_t o = valid ? off[i] : kOobOffset;
    v[0] = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(rsrc, o, step * 128, 0));
    v[1] = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(rsrc, o + 64, step * 128, 0));
  }
  // The last, partial step: `left` (1 .. 127) of its bytes are the operand's.
  // What a row's storage holds past them must not reach the MFMAs (a NaN
  // there times the other operand's zero is a NaN).
  __device__ __forceinline__ void load_tail(int i, int step, int left, int lane, i32x4 (&v)[2]) const {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int nb = left - 64 * h - 16 * (lane >> 4);  // valid bytes of this chunk
      i32x4 x = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(
                                              rsrc, nb > 0 ? off[i] + 64 * h : kOobOffset, step * 128, 0));
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const int vb = nb - 4 * w;
        x[w] &= vb >= 4 ? -1 : (vb <= 0 ? 0 : (int)((1u << (8 * vb)) - 1u));
      }
      v[h] = x;
    }
  }
};

// This wave's share of the tile: every W-th K step from `wave` on.  U steps
// are loaded while the U before them are multiplied.
template <int ES, int MB, int NB, int W, int U>
__device__ __forceinline__ void rowblock_loop(f32x4 (&acc)[MB][NB], const RowBlock<MB>& ra,
                                              const RowBlock<NB>& rb, int64_t k_bytes, int wave,
                                              int lane) {
  struct Step {
    i32x4 a[MB][2], b[NB][2];
  };
  const int whole = (int)(k_bytes >> 7);
  const std::integral_constant<int, ES> es;
  auto load = [&](Step (&s)[U], int first) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int step = first + u * W;
#pragma unroll
      for (int i = 0; i < NB; ++i) rb.load(i, step, step < whole, s[u].b[i]);
#pragma unroll
      for (int i = 0; i < MB; ++i) ra.load(i, step, step < whole, s[u].a[i]);
    }
  };
  auto multiply = [&](const Step& s) {
#pragma unroll
    for (int m = 0; m < MB; ++m)
#pragma unroll
      for (int n = 0; n < NB; ++n)
        acc[m][n] = mfma_16(s.b[n][0], s.b[n][1], s.a[m][0], s.a[m][1], acc[m][n], es);
  };
  Step x[U], y[U];
  load(x, wave);
  for (int s = wave; s < whole; s += 2 * U * W) {
    load(y, s + U * W);
#pragma unroll
    for (int u = 0; u < U; ++u) multiply(x[u]);
    load(x, s + 2 * U * W);
#pragma unroll
    for (int u = 0; u < U; ++u) multiply(y[u]);
  }
  const int left = (int)(k_bytes & 127);
  if (left != 0 && wave == whole % W) {
#pragma unroll
    for (int i = 0; i < NB; ++i) rb.load_tail(i, whole, left, lane, x[0].b[i]);
#pragma unroll
    for (int i = 0; i < MB; ++i) ra.load_tail(i, whole, left, lane, x[0].a[i]);
    multiply(x[0]);
  }
}

// The waves' partial tiles are added in the order of the waves: block
// mb * NB + nb is summed by wave (mb * NB + nb) % W, which then calls
// done(mb, nb, sum).  `part` holds W MB NB * 64 pieces of 16 bytes, of type V
// (i32x4 for int8: the bits that acc holds).
template <int MB, int NB, int W, class V, class Done>
__device__ __forceinline__ void rowblock_join(const f32x4 (&acc)[MB][NB], V* part, int wave,
                                              int lane, Done&& done) {
#pragma unroll
  for (int m = 0; m < MB; ++m)
#pragma unroll
    for (int n = 0; n < NB; ++n) part[(wave * MB * NB + m * NB + n) * 64 + lane] = __builtin_bit_cast(V, acc[m][n]);
  __syncthreads();
  for (int b = wave; b < MB * NB; b += W) {
    V sum = part[b * 64 + lane];
#pragma unroll
    for (int w = 1; w < W; ++w) sum += part[(w * MB * NB + b) * 64 + lane];
    done(b / NB, b % NB, sum);
  }
}

}  // namespace migemm

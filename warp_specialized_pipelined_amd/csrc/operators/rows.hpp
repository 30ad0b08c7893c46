// rows.hpp -- a row of a bf16 matrix held by one wave or by the waves of a
// workgroup: reductions, 16-byte accesses that end with the columns, e4m3 codes.
#pragma once

#include "../kernel/gfx950.hpp"

namespace migemm {

constexpr float kE4M3Max = 448.0f;

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d, 64);
  return v;
}
// Maximum of non-negative floats (and NaN) as unsigned bit patterns: a NaN's
// pattern is above infinity's, so it wins.
__device__ __forceinline__ uint32_t wave_max_bits(uint32_t v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) {
    const uint32_t o = __shfl_xor(v, d, 64);
    v = o > v ? o : v;
  }
  return v;
}

// Eight consecutive bf16 of a row at column c.  The row starts on a 16-byte
// boundary, so a vector that holds the last columns may be read whole (the
// bytes past them share its 16-byte block); what lies past the columns is
// replaced by zeros.
__device__ __forceinline__ u32x4 load8(const unsigned short* row, int64_t c, int64_t cols) {
  u32x4 v = {0, 0, 0, 0};
  if (c < cols) {
    v = *reinterpret_cast<const u32x4*>(row + c);
    const int left = cols - c < 8 ? (int)(cols - c) : 8;
    if (left < 8) {
#pragma unroll
      for (int w = 0; w < 4; ++w)
        v[w] = 2 * w + 2 <= left ? v[w] : (2 * w + 1 == left ? v[w] & 0xFFFFu : 0u);
    }
  }
  return v;
}
__device__ __forceinline__ void store8(unsigned short* row, int64_t c, int64_t cols, u32x4 v) {
  if (c + 8 <= cols) {
    *reinterpret_cast<u32x4*>(row + c) = v;
  } else if (c < cols) {
    for (int e = 0; e < (int)(cols - c); ++e)
      row[c + e] = (unsigned short)(v[e >> 1] >> (16 * (e & 1)));
  }
}
// Eight bytes of a row at column c.
__device__ __forceinline__ void store8_bytes(unsigned char* row, int64_t c, int64_t cols, u32x2 v) {
  if (c + 8 <= cols) {
    *reinterpret_cast<u32x2*>(row + c) = v;
  } else if (c < cols) {
    for (int e = 0; e < (int)(cols - c); ++e) row[c + e] = (unsigned char)(v[e >> 2] >> (8 * (e & 3)));
  }
}
// A row through a buffer resource over its columns: what a lane has past them
// reads as zeros and is not written, without branches (range checks work on
// dwords; the element or bytes in a last, partial one are seen to apart: ODD,
// with an odd number of columns).  Wave-uniform.
template <bool ODD>
struct RowView {
  __amdgpu_buffer_rsrc_t rsrc;
  int cols;
  // bf16 to be read: the range ends with the last dword.
  static __device__ __forceinline__ RowView in(const void* m, int64_t elements, int64_t cols) {
    return {make_rsrc(static_cast<const unsigned short*>(m) + elements, (uint32_t)((cols * 2 + 3) & ~(int64_t)3)), (int)cols};
  }
  // To be written: the range ends with the last element (of ES bytes).
  template <int ES>
  static __device__ __forceinline__ RowView out(void* m, int64_t elements, int64_t cols) {
    return {make_rsrc(static_cast<unsigned char*>(m) + elements * ES, (uint32_t)(cols * ES)), (int)cols};
  }
  // Eight bf16 at column c; with ODD the one past the last column holds anything
  // until it is cleared, which waits for the load.
  __device__ __forceinline__ u32x4 load(int c) const {
    return __builtin_bit_cast(u32x4, __builtin_amdgcn_raw_buffer_load_b128(rsrc, 2 * c, 0, 0));
  }
  static __device__ __forceinline__ void clear_past(u32x4& v, int c, int64_t cols) {
    if constexpr (ODD) {
      const int last = ((int)cols - c) >> 1;  // the dword that holds the last column
#pragma unroll
      for (int w = 0; w < 4; ++w) v[w] = w == last ? v[w] & 0xFFFFu : v[w];
    }
  }
  __device__ __forceinline__ u32x4 load_cleared(int c) const {
    u32x4 v = load(c);
    clear_past(v, c, cols);
    return v;
  }
  __device__ __forceinline__ void store(int c, u32x4 v) const {
    __builtin_amdgcn_raw_buffer_store_b128(v, rsrc, 2 * c, 0, 0);
    if constexpr (ODD) {
#pragma unroll
      for (int w = 0; w < 4; ++w)
        if (w == (cols - c) >> 1) __builtin_amdgcn_raw_buffer_store_b16((unsigned short)v[w], rsrc, 2 * (c + 2 * w), 0, 0);
    }
  }
  // Eight bytes at column c.
  __device__ __forceinline__ void store_bytes(int c, u32x2 v) const {
    __builtin_amdgcn_raw_buffer_store_b64(v, rsrc, c, 0, 0);
    if (cols & 3) {
#pragma unroll
      for (int w = 0; w < 2; ++w)
        if (w == (cols - c) >> 2)
          for (int b = 0; b < (cols & 3); ++b)
            __builtin_amdgcn_raw_buffer_store_b8((unsigned char)(v[w] >> (8 * b)), rsrc, c + 4 * w + b, 0, 0);
    }
  }
};
// The larger of each half's unsigned 16 bits.
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(u16x2, a), __builtin_bit_cast(u16x2, b)));
}
__device__ __forceinline__ float lo(uint32_t w) { return bf16_lo(w); }
__device__ __forceinline__ float hi(uint32_t w) { return bf16_hi(w); }

// Past +-448 (by rounding only: |v| <= 448 (1 + 2^-23)) the value is 448;
// a NaN stays one.
__device__ __forceinline__ float clamp448(float v) {
  return fabsf(v) > kE4M3Max ? copysignf(kE4M3Max, v) : v;
}
__device__ __forceinline__ uint32_t pack_e4m3x4(float a, float b, float c, float d) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(clamp448(a), clamp448(b), 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(clamp448(c), clamp448(d), w, true);
}

// Four values of at most 127 in magnitude to int8, ties to even: adding 1.5 *
// 2^23 rounds to a whole number, whose low byte is then the sum's.
__device__ __forceinline__ uint32_t pack_i8x4(float a, float b, float c, float d) {
  constexpr float kRound = 12582912.0f;
  const uint32_t ab = __builtin_amdgcn_perm(__float_as_uint(b + kRound), __float_as_uint(a + kRound), 0x0C0C0400u);
  const uint32_t cd = __builtin_amdgcn_perm(__float_as_uint(d + kRound), __float_as_uint(c + kRound), 0x04000C0Cu);
  return ab | cd;
}

constexpr int threads_of(int waves) { return waves == 1 ? 256 : 64 * waves; }
constexpr int rows_of(int waves) { return waves == 1 ? 4 : 1; }

}  // namespace migemm

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
#include <hip/hip_runtime.h>

#include "../kernel/gfx950.hpp"
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

// Columns a lane packs or unpacks.
constexpr int kPackCols = 4;

// A wave's item: tokens of a group x 256 columns, numbered along the columns
// first; lane l holds columns 4 l .. 4 l + 3 of them.
struct PackItem {
  int64_t group, col;
  __device__ __forceinline__ PackItem(int64_t item, int64_t ld, int lane) {
    const int64_t across = (ld + 64 * kPackCols - 1) / (64 * kPackCols);
    group = item / across;
    col = ((item - group * across) * 64 + lane) * kPackCols;
  }
};

// 32 tokens x 256 columns.
__device__ __forceinline__ void pack_item(const CheckpointArgs& a, int64_t item, int lane) {
  const PackItem at(item, a.ld, lane);
  const int64_t c = at.col, t0 = at.group * 32;
  if (c >= a.ld) return;
  const unsigned short* x = static_cast<const unsigned short*>(a.x) + t0 * a.x_rs + c;
  u32x2 v[32];
#pragma unroll
  for (int t = 0; t < 32; ++t) {
    v[t] = u32x2{0, 0};
    if (t0 + t < a.tokens && c < a.cols) v[t] = *reinterpret_cast<const u32x2*>(x + t * a.x_rs);
  }
  // (Columns past the last: their bytes may hold anything.)
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    const int64_t left = a.cols - c - 2 * w;
    const uint32_t keep = left >= 2 ? 0xFFFFFFFFu : (left == 1 ? 0xFFFFu : 0u);
#pragma unroll
    for (int t = 0; t < 32; ++t) v[t][w] &= keep;
  }
  unsigned char* codes = a.codes + (t0 / 16) * a.ld * 16 + c * 16;
  uint32_t exponents = 0;
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    uint32_t top = 0;
#pragma unroll
    for (int t = 0; t < 32; ++t) top = max_u16x2(top, v[t][w] & 0x7FFF7FFFu);
    if ((top & 0xFFFFu) > 0x7F60u || (top >> 16) > 0x7F60u) {
      // Infinities and NaN become NaN and leave the group's power to the rest;
      // what is past 1.75 2^127 becomes that.
      top = 0;
#pragma unroll
      for (int t = 0; t < 32; ++t) {
        uint32_t m = v[t][w] & 0x7FFF7FFFu, s = v[t][w] & 0x80008000u, o = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t b = (m >> (16 * h)) & 0xFFFFu;
          if (b >= 0x7F80u) b = 0x7FC0u;
          else if (b > 0x7F60u) b = 0x7F60u;
          o |= b << (16 * h);
        }
        v[t][w] = o | s;
        const uint32_t f = ((o & 0xFFFFu) >= 0x7F80u ? 0 : o & 0xFFFFu) | ((o >> 16) >= 0x7F80u ? 0 : o & 0xFFFF0000u);
        top = max_u16x2(top, f);
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t e = exponent_of(h ? top >> 16 : top & 0xFFFFu);
      exponents |= e << (8 * (2 * w + h));
      const float scale = power_of(e);
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        u32x4 o;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          i16x2 d = {0, 0};
          const int t = 16 * g + 4 * q;
          const uint32_t p0 = __builtin_amdgcn_perm(v[t + 1][w], v[t][w], h ? 0x07060302u : 0x05040100u);
          const uint32_t p1 = __builtin_amdgcn_perm(v[t + 3][w], v[t + 2][w], h ? 0x07060302u : 0x05040100u);
          d = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(d, __builtin_bit_cast(bf16x2, p0), scale, false);
          d = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(d, __builtin_bit_cast(bf16x2, p1), scale, true);
          o[q] = __builtin_bit_cast(uint32_t, d);
        }
        *reinterpret_cast<u32x4*>(codes + g * a.ld * 16 + (2 * w + h) * 16) = o;
      }
    }
  }
  *reinterpret_cast<uint32_t*>(a.scales + at.group * a.ld + c) = exponents;
}
__global__ __launch_bounds__(64) void checkpoint_pack(CheckpointArgs a, int64_t items) {
  for (int64_t i = blockIdx.x; i < items; i += gridDim.x) pack_item(a, i, threadIdx.x);
}

__device__ __forceinline__ uint32_t two_bf16(uint32_t codes, float scale, bool upper) {
  return __builtin_bit_cast(uint32_t, upper ? __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, scale, true)
                                            : __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(codes, scale, false));
}

// 16 tokens x 256 columns.
__device__ __forceinline__ void unpack_item(const CheckpointArgs& a, int64_t item, int lane) {
  const PackItem at(item, a.ld, lane);
  const int64_t c = at.col, t0 = at.group * 16;
  if (c >= a.cols) return;
  const u32x4* codes = reinterpret_cast<const u32x4*>(a.codes) + at.group * a.ld + c;
  const uint32_t exponents = *reinterpret_cast<const uint32_t*>(a.scales + (at.group / 2) * a.ld + c);
  u32x4 v[kPackCols];
#pragma unroll
  for (int i = 0; i < kPackCols; ++i) v[i] = codes[i];
  unsigned short* x = static_cast<unsigned short*>(a.x_out) + t0 * a.x_rs + c;
  const int64_t left = a.cols - c;
#pragma unroll
  for (int t = 0; t < 16; t += 2) {
    uint32_t p[kPackCols];  // tokens t and t + 1 of a column
#pragma unroll
    for (int i = 0; i < kPackCols; ++i)
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

// A 32 x 32 tile of dw a wave, its operands straight from memory.  Lane l holds
// column l % 32 of dy (and of the kept activations) and, of a group of 32
// tokens, 16 (l / 32) .. + 15: eight for each of two instructions.
__global__ __launch_bounds__(64) void checkpoint_gradient_simple(CheckpointArgs a) {
  const int lane = threadIdx.x, l = lane & 31, half = lane >> 5;
  const int64_t across = (a.cols + 31) / 32;
  const int64_t n0 = blockIdx.x / across * 32, k0 = blockIdx.x % across * 32;
  const int64_t n = n0 + l, k = k0 + l;
  const unsigned short* dy = static_cast<const unsigned short*>(a.dy);
  f32x16 acc = {};
  for (int64_t t0 = 0; t0 < a.tokens; t0 += 32) {
    u32x4 code = {0, 0, 0, 0};
    float scale = 1.0f;
    if (k < a.ld) {
      code = *reinterpret_cast<const u32x4*>(a.codes + ((t0 / 16 + half) * a.ld + k) * 16);
      scale = power_of(a.scales[(t0 / 32) * a.ld + k]);
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      u32x4 av, bv;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int64_t t = t0 + 16 * half + 8 * s + 2 * q;
        const uint32_t d0 = n < a.out_cols && t < a.tokens ? dy[t * a.dy_rs + n] : 0;
        const uint32_t d1 = n < a.out_cols && t + 1 < a.tokens ? dy[(t + 1) * a.dy_rs + n] : 0;
        av[q] = d0 | d1 << 16;
        bv[q] = two_bf16(code[2 * s + (q >> 1)], scale, q & 1);
      }
      acc = mfma_bf16_32x32x16(__builtin_bit_cast(bf16x8, bv), __builtin_bit_cast(bf16x8, av), acc);
    }
  }
  if (n >= a.out_cols) return;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int64_t col = k0 + 8 * (i >> 2) + 4 * half + (i & 3);
    if (col >= a.cols) continue;
    const int64_t at = n * a.dw_rs + col;
    if (a.fp32) {
      float* d = static_cast<float*>(a.dw) + at;
      *d = a.accumulate ? *d + acc[i] : acc[i];
    } else {
      static_cast<unsigned short*>(a.dw)[at] = (unsigned short)pack_bf16x2(acc[i], 0.0f);
    }
  }
}

}  // namespace

// A launch holds fewer than 2^32 threads.
static uint32_t wave_grid(int64_t items) { return (uint32_t)(items < (1 << 25) ? items : 1 << 25); }

hipError_t launch_checkpoint_pack(const CheckpointArgs& a, hipStream_t stream) {
  const int64_t items = (a.tokens + 31) / 32 * ((a.ld + 255) / 256);
  hipLaunchKernelGGL(checkpoint_pack, dim3(wave_grid(items)), dim3(64), 0, stream, a, items);
  return hipGetLastError();
}

hipError_t launch_checkpoint_unpack(const CheckpointArgs& a, hipStream_t stream) {
  const int64_t items = (a.tokens + 15) / 16 * ((a.ld + 255) / 256);
  hipLaunchKernelGGL(checkpoint_unpack, dim3(wave_grid(items)), dim3(64), 0, stream, a, items);
  return hipGetLastError();
}

hipError_t launch_checkpoint_gradient(const CheckpointArgs& a, hipStream_t stream) {
  hipLaunchKernelGGL(checkpoint_gradient_simple, dim3((uint32_t)((a.cols + 31) / 32 * ((a.out_cols + 31) / 32))), dim3(64), 0,
                     stream, a);
  return hipGetLastError();
}

}  // namespace migemm

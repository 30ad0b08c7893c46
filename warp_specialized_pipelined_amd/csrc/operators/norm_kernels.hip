// norm_kernels.hip -- the residual's addition and the root-mean-square norm
// of each row, with bf16 or e4m3 output, and its gradient.
//
// Forward, per row of n columns:
//   h = bf16(x + r)                       (h = x without a residual)
//   rstd = 1 / sqrt(sum h^2 / n + eps)    (fp32 sum)
//   bf16:  y = bf16(h rstd w)
//   e4m3:  top = max |h w|;  scale = top rstd / 448;  y = e4m3(h w 448 / top)
// The e4m3 codes do not need rstd (it cancels: y / scale = h w 448 / top), so
// the sum and the maximum come out of one pass over registers and one
// reduction.
//
// Backward, with n = h rstd and g = dy:
//   dx = rstd (g w - n mean(g w n)) + dh,   dweight = sum over rows of g n
//
// Bound: memory (4 to 14 bytes an element).  A row is read once, 16 bytes a
// lane, and stays in registers between the reduction and the output.  Measured:
// 8192 x 8192 to e4m3 rows 82 us (5.7 TB/s); 4000 x 5000 without a residual 15
// us where its 80 MB are still in the last-level cache, 20 from memory (4.1
// TB/s); 8192 x 4096 forward 46 us and backward 47 us (5.8 and 5.7 TB/s) and 5
// us for the column sums; one row of 8192 3.2 us (with 4 waves instead of 16:
// 3.9; a row of 1000 to bf16: 2.4).
#include <hip/hip_runtime.h>

#include "../kernel/gfx950.hpp"
#include "operators.h"

namespace migemm {
namespace {

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

constexpr int threads_of(int waves) { return waves == 1 ? 256 : 64 * waves; }
constexpr int rows_of(int waves) { return waves == 1 ? 4 : 1; }

// WAVES waves share a row (with one, a workgroup takes 4 rows), NV vectors
// of 8 columns each lane.
template <int WAVES, int NV, bool RES, bool E4M3>
__device__ __forceinline__ void norm_row(const NormArgs& a, int64_t row, int t, int wave, int lane,
                                         int phase) {
  constexpr int kLanes = 64 * WAVES;
  const unsigned short* x = static_cast<const unsigned short*>(a.x) + row * a.x_rs;
  const unsigned short* w = static_cast<const unsigned short*>(a.weight);

  u32x4 hv[NV], wv[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) hv[i] = load8(x, (int64_t)(i * kLanes + t) * 8, a.cols);
  if constexpr (RES) {
    const unsigned short* r = static_cast<const unsigned short*>(a.r) + row * a.r_rs;
    u32x4 rv[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) rv[i] = load8(r, (int64_t)(i * kLanes + t) * 8, a.cols);
#pragma unroll
    for (int i = 0; i < NV; ++i) wv[i] = load8(w, (int64_t)(i * kLanes + t) * 8, a.cols);
    unsigned short* h = static_cast<unsigned short*>(a.h) + row * a.h_rs;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        hv[i][q] = pack_bf16x2(lo(hv[i][q]) + lo(rv[i][q]), hi(hv[i][q]) + hi(rv[i][q]));
      store8(h, (int64_t)(i * kLanes + t) * 8, a.cols, hv[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) wv[i] = load8(w, (int64_t)(i * kLanes + t) * 8, a.cols);
  }

  float sum = 0.0f;
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float h0 = lo(hv[i][q]), h1 = hi(hv[i][q]);
      sum += h0 * h0;
      sum += h1 * h1;
      if constexpr (E4M3) {
        const uint32_t b0 = __float_as_uint(h0 * lo(wv[i][q])) & 0x7FFFFFFFu;
        const uint32_t b1 = __float_as_uint(h1 * hi(wv[i][q])) & 0x7FFFFFFFu;
        top = b0 > top ? b0 : top;
        top = b1 > top ? b1 : top;
      }
    }
  sum = wave_sum(sum);
  if constexpr (E4M3) top = wave_max_bits(top);
  if constexpr (WAVES > 1) {
    // Two buffers: a wave that is already at its next row writes the other
    // one, and cannot come round to this one before the barrier between.
    __shared__ float sums[2][WAVES];
    __shared__ uint32_t tops[2][WAVES];
    if (lane == 0) {
      sums[phase][wave] = sum;
      tops[phase][wave] = top;
    }
    __syncthreads();
    sum = 0.0f;
    top = 0;
#pragma unroll
    for (int i = 0; i < WAVES; ++i) {
      sum += sums[phase][i];
      top = tops[phase][i] > top ? tops[phase][i] : top;
    }
  }
  const float rstd = rsqrtf(sum / (float)a.cols + a.eps);
  if (t == 0) a.rstd[row] = rstd;

  if constexpr (E4M3) {
    const float largest = __uint_as_float(top);
    if (t == 0) a.scale[row] = largest * rstd / kE4M3Max;
    // Rows of values so small that 448 / largest would overflow are lifted.
    const float lift = largest < 0x1p-96f ? 0x1p96f : 1.0f;
    const float inv = largest == 0.0f ? 0.0f : kE4M3Max / (largest * lift);
    unsigned char* y = static_cast<unsigned char*>(a.y) + row * a.y_rs;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t c = (int64_t)(i * kLanes + t) * 8;
      float v[8];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        v[2 * q] = lo(hv[i][q]) * lo(wv[i][q]) * lift * inv;
        v[2 * q + 1] = hi(hv[i][q]) * hi(wv[i][q]) * lift * inv;
      }
      const u32x2 o = {pack_e4m3x4(v[0], v[1], v[2], v[3]), pack_e4m3x4(v[4], v[5], v[6], v[7])};
      if (c + 8 <= a.cols) {
        *reinterpret_cast<u32x2*>(y + c) = o;
      } else if (c < a.cols) {
        for (int e = 0; e < (int)(a.cols - c); ++e) y[c + e] = (unsigned char)(o[e >> 2] >> (8 * (e & 3)));
      }
    }
  } else {
    unsigned short* y = static_cast<unsigned short*>(a.y) + row * a.y_rs;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      u32x4 o;
#pragma unroll
      for (int q = 0; q < 4; ++q)
        o[q] = pack_bf16x2(lo(hv[i][q]) * rstd * lo(wv[i][q]), hi(hv[i][q]) * rstd * hi(wv[i][q]));
      store8(y, (int64_t)(i * kLanes + t) * 8, a.cols, o);
    }
  }
}

template <int WAVES, int NV, bool RES, bool E4M3>
__global__ __launch_bounds__(threads_of(WAVES)) void norm_forward(NormArgs a) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int t = WAVES == 1 ? lane : (int)threadIdx.x;
  // One row, unless the grid is at its cap (launch_norm_forward).
  int phase = 0;
  const int64_t step = (int64_t)gridDim.x * rows_of(WAVES);
  for (int64_t row = (int64_t)blockIdx.x * rows_of(WAVES) + (WAVES == 1 ? wave : 0); row < a.rows;
       row += step, phase ^= 1)
    norm_row<WAVES, NV, RES, E4M3>(a, row, t, wave, lane, phase);
}

// Each walker (a workgroup, or with WAVES = 1 a wave) takes rows walker,
// walker + walkers, ... and keeps its columns' sums of g n in registers; the
// workgroup's sums (with WAVES = 1 its four waves', added through LDS) go to
// its row of the workspace, and norm_sum_partials adds those rows in a fixed
// order: no atomics, the same result on every run.  One workgroup alone writes
// dweight itself.
template <int WAVES, int NV, bool RES>
__global__ __launch_bounds__(threads_of(WAVES)) void norm_backward(NormArgs a) {
  constexpr int kLanes = 64 * WAVES;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t walker = (int64_t)blockIdx.x * rows_of(WAVES) + (WAVES == 1 ? wave : 0);
  const int64_t walkers = (int64_t)gridDim.x * rows_of(WAVES);
  const int t = WAVES == 1 ? lane : (int)threadIdx.x;
  const unsigned short* w = static_cast<const unsigned short*>(a.weight);
  const float cols = (float)a.cols;

  u32x4 wv[NV];
  float dw[NV][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    wv[i] = load8(w, (int64_t)(i * kLanes + t) * 8, a.cols);
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[i][e] = 0.0f;
  }
  __shared__ float sums[2][WAVES];
  int phase = 0;
  for (int64_t row = walker; row < a.rows; row += walkers) {
    const unsigned short* g = static_cast<const unsigned short*>(a.dy) + row * a.dy_rs;
    const unsigned short* h = static_cast<const unsigned short*>(a.x) + row * a.x_rs;
    u32x4 gv[NV], hv[NV], dhv[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) gv[i] = load8(g, (int64_t)(i * kLanes + t) * 8, a.cols);
#pragma unroll
    for (int i = 0; i < NV; ++i) hv[i] = load8(h, (int64_t)(i * kLanes + t) * 8, a.cols);
    if constexpr (RES) {
      const unsigned short* dh = static_cast<const unsigned short*>(a.dh) + row * a.dh_rs;
#pragma unroll
      for (int i = 0; i < NV; ++i) dhv[i] = load8(dh, (int64_t)(i * kLanes + t) * 8, a.cols);
    }
    const float rstd = a.rstd[row];
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float n0 = lo(hv[i][q]) * rstd, n1 = hi(hv[i][q]) * rstd;
        const float g0 = lo(gv[i][q]), g1 = hi(gv[i][q]);
        dw[i][2 * q] += g0 * n0;
        dw[i][2 * q + 1] += g1 * n1;
        s += g0 * lo(wv[i][q]) * n0;
        s += g1 * hi(wv[i][q]) * n1;
      }
    s = wave_sum(s);
    if constexpr (WAVES > 1) {
      // (Two buffers, as in the forward pass.)
      if (lane == 0) sums[phase][wave] = s;
      __syncthreads();
      s = 0.0f;
#pragma unroll
      for (int i = 0; i < WAVES; ++i) s += sums[phase][i];
      phase ^= 1;
    }
    const float mean = s / cols;
    unsigned short* dx = static_cast<unsigned short*>(a.dx) + row * a.dx_rs;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      u32x4 o;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float n0 = lo(hv[i][q]) * rstd, n1 = hi(hv[i][q]) * rstd;
        float d0 = rstd * (lo(gv[i][q]) * lo(wv[i][q]) - n0 * mean);
        float d1 = rstd * (hi(gv[i][q]) * hi(wv[i][q]) - n1 * mean);
        if constexpr (RES) {
          d0 += lo(dhv[i][q]);
          d1 += hi(dhv[i][q]);
        }
        o[q] = pack_bf16x2(d0, d1);
      }
      store8(dx, (int64_t)(i * kLanes + t) * 8, a.cols, o);
    }
  }
  float* p = a.partial_rows == 1 ? a.dweight : a.partials + (int64_t)blockIdx.x * a.cols;
  if constexpr (WAVES == 1) {
    __shared__ float all[4][NV * 512];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) all[wave][(i * 64 + lane) * 8 + e] = dw[i][e];
    __syncthreads();
    for (int64_t c = threadIdx.x; c < a.cols; c += 256) p[c] = ((all[0][c] + all[1][c]) + all[2][c]) + all[3][c];
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t c = (int64_t)(i * kLanes + t) * 8;
      if (c + 8 <= a.cols) {
        // (16-byte stores, which need an address that is a multiple of 4.)
        typedef float f32x4_4 __attribute__((ext_vector_type(4), aligned(4)));
        *reinterpret_cast<f32x4_4*>(p + c) = f32x4_4{dw[i][0], dw[i][1], dw[i][2], dw[i][3]};
        *reinterpret_cast<f32x4_4*>(p + c + 4) = f32x4_4{dw[i][4], dw[i][5], dw[i][6], dw[i][7]};
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (c + e < a.cols) p[c + e] = dw[i][e];
      }
    }
  }
}

// dweight[c] = sum over partial rows: GROUPS threads a column add every
// GROUPS-th row, then one adds their sums in order.
template <int GROUPS, int COLS>
__global__ __launch_bounds__(GROUPS * COLS) void norm_sum_partials(NormArgs a) {
  const int col = threadIdx.x % COLS, group = threadIdx.x / COLS;
  const int64_t c = (int64_t)blockIdx.x * COLS + col;
  float s = 0.0f;
  if (c < a.cols)
#pragma unroll 8
    for (int64_t p = group; p < a.partial_rows; p += GROUPS) s += a.partials[p * a.cols + c];
  if constexpr (GROUPS > 1) {
    __shared__ float part[GROUPS][COLS + 1];
    part[group][col] = s;
    __syncthreads();
    if (group != 0) return;
#pragma unroll
    for (int i = 1; i < GROUPS; ++i) s += part[i][col];
  }
  if (c < a.cols) a.dweight[c] = s;
}

typedef void (*norm_fn)(NormArgs);

template <int WAVES, int NV>
norm_fn forward_of(bool res, bool e4m3) {
  if (res) return e4m3 ? norm_forward<WAVES, NV, true, true> : norm_forward<WAVES, NV, true, false>;
  return e4m3 ? norm_forward<WAVES, NV, false, true> : norm_forward<WAVES, NV, false, false>;
}
template <int WAVES>
norm_fn forward_pick(int nv, bool res, bool e4m3) {
  return nv == 1 ? forward_of<WAVES, 1>(res, e4m3)
                 : (nv == 2 ? forward_of<WAVES, 2>(res, e4m3) : forward_of<WAVES, 4>(res, e4m3));
}
template <int WAVES>
norm_fn backward_pick(int nv, bool res) {
  if (res) return nv == 1 ? norm_backward<WAVES, 1, true>
                          : (nv == 2 ? norm_backward<WAVES, 2, true> : norm_backward<WAVES, 4, true>);
  return nv == 1 ? norm_backward<WAVES, 1, false>
                 : (nv == 2 ? norm_backward<WAVES, 2, false> : norm_backward<WAVES, 4, false>);
}

}  // namespace

// The fewest waves (1, 4, 16) whose lanes hold the row in `most` vectors, and
// the vectors that takes.  Few rows: one vector a lane where 16 waves allow, for
// a row's latency counts (one wave up to 512 columns, four up to 2048).  Many:
// up to four (one wave up to 2048 columns, four up to 8192), which leaves more
// rows in flight: 8192 x 1100 forward and backward 45 us with one wave a row, 66
// with four, 4096 x 1100 29 and 38 (8192 x 2048 53 and 56; at 1000 x 2048 four
// waves are 2 us faster, 14 and 16).
NormShape norm_shape(int64_t rows, int64_t cols) {
  const int most = rows <= 256 ? 1 : 4;
  int waves = 1;
  while (waves < 16 && (int64_t)waves * 512 * most < cols) waves *= 4;
  const int64_t v = (cols + waves * 512 - 1) / (waves * 512);
  return {waves, v <= 1 ? 1 : (v <= 2 ? 2 : 4)};
}

// A second kernel costs about as much as three rows one after another.
int64_t norm_partial_rows(int64_t rows, int64_t cols, int cu_count) {
  const int at_once = rows_of(norm_shape(rows, cols).waves);
  if (rows <= 3 * at_once) return rows > 0 ? 1 : 0;
  const int64_t groups = (rows + at_once - 1) / at_once, most = (int64_t)cu_count * 2;
  return groups < most ? groups : most;
}

hipError_t launch_norm_forward(const NormArgs& a, bool e4m3, hipStream_t stream) {
  const NormShape s = norm_shape(a.rows, a.cols);
  const bool res = a.r != nullptr;
  const norm_fn f = s.waves == 1 ? forward_pick<1>(s.vectors, res, e4m3)
                                 : (s.waves == 4 ? forward_pick<4>(s.vectors, res, e4m3)
                                                 : forward_pick<16>(s.vectors, res, e4m3));
  int64_t grid = (a.rows + rows_of(s.waves) - 1) / rows_of(s.waves);
  if (grid > (1 << 20)) grid = 1 << 20;  // a launch holds fewer than 2^32 threads
  hipLaunchKernelGGL(f, dim3((uint32_t)grid), dim3(threads_of(s.waves)), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_norm_backward(const NormArgs& a, hipStream_t stream) {
  const NormShape s = norm_shape(a.rows, a.cols);
  const bool res = a.dh != nullptr;
  if (a.partial_rows > 0) {
    const norm_fn f = s.waves == 1 ? backward_pick<1>(s.vectors, res)
                                   : (s.waves == 4 ? backward_pick<4>(s.vectors, res)
                                                   : backward_pick<16>(s.vectors, res));
    hipLaunchKernelGGL(f, dim3((uint32_t)a.partial_rows), dim3(threads_of(s.waves)), 0, stream, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.partial_rows == 1) return e;
  }
  // Few rows of sums: a thread a column.
  if (a.partial_rows <= 16)
    hipLaunchKernelGGL((norm_sum_partials<1, 64>), dim3((uint32_t)((a.cols + 63) / 64)), dim3(64), 0, stream, a);
  else
    hipLaunchKernelGGL((norm_sum_partials<32, 32>), dim3((uint32_t)((a.cols + 31) / 32)), dim3(1024), 0, stream, a);
  return hipGetLastError();
}

}  // namespace migemm

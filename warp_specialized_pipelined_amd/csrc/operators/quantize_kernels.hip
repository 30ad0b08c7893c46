// quantize_kernels.hip -- bf16 rows to 8 bits with a scale each:
//   scale = max |x| / top,   q = round(x top / max |x|)     (top: 127 or 448)
// rounded to the nearest code, ties to even.
//
// The quotient is formed exactly enough that every code is the definition's.
// x and max |x| have 8 significant bits, so x top is exact in fp32, and a
// quotient that is not on the border of two codes is 2^-17 of itself or more
// away from it; one that is on it is a multiple of a half of a code, which fp32
// holds, and there the quotient has to come out exactly: q0 = x (top / max |x|)
// is off by a few units in its last place, the remainder x top - q0 max |x| is
// exact in one fma, and q0 plus remainder / max |x| is rounded once.
//
// Bound: memory (3 bytes an element); a row is read once and stays in registers
// between its maximum and its codes.  8192 x 16384: 74 us, 5.4 TB/s; 33 x 8192:
// 3.5 us, what a launch of any kernel takes.
#include <hip/hip_runtime.h>

#include "../kernel/gfx950.hpp"
#include "operators.h"
#include "rows.hpp"

namespace migemm {
namespace {

template <int WAVES, int NV, bool E4M3>
__device__ __forceinline__ void quantize_row(const QuantizeArgs& a, int64_t row, int t, int wave, int lane,
                                             int phase) {
  constexpr int kLanes = 64 * WAVES;
  constexpr float kTop = E4M3 ? kE4M3Max : 127.0f;
  const unsigned short* x = static_cast<const unsigned short*>(a.x) + row * a.x_rs;
  u32x4 v[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) v[i] = load8(x, (int64_t)(i * kLanes + t) * 8, a.cols);
  uint32_t top = 0;  // the largest magnitude as a bf16 pattern (NaN above infinity)
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int q = 0; q < 4; ++q) top = max_u16x2(top, v[i][q] & 0x7FFF7FFFu);
  top = (top & 0xFFFFu) > (top >> 16) ? top & 0xFFFFu : top >> 16;
  top = wave_max_bits(top);
  if constexpr (WAVES > 1) {
    __shared__ uint32_t tops[2][WAVES];  // two buffers, as in norm_kernels.hip
    if (lane == 0) tops[phase][wave] = top;
    __syncthreads();
    top = 0;
#pragma unroll
    for (int i = 0; i < WAVES; ++i) top = tops[phase][i] > top ? tops[phase][i] : top;
  }
  // A row that holds an infinity or a NaN has no scale: NaN, and codes of 0.
  const bool finite = top < 0x7F80u;
  const float largest = __uint_as_float(top << 16);
  if (t == 0) a.scale[row] = finite ? largest / kTop : NAN;
  // (Rows of very large or small values are moved to where nothing overflows;
  // values that a move makes subnormal are far below half a code.)
  const float move = largest >= 0x1p64f ? 0x1p-64f : (largest < 0x1p-62f ? 0x1p64f : 1.0f);
  const float m = largest * move, inv = top == 0 ? 0.0f : 1.0f / m, factor = kTop * inv;
  auto code = [&](float e) {
    const float q0 = e * move * factor;
    return fmaf(fmaf(-q0, m, e * move * kTop), inv, q0);
  };
  unsigned char* q = static_cast<unsigned char*>(a.q) + row * a.q_rs;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t c = (int64_t)(i * kLanes + t) * 8;
    float f[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[2 * j] = code(lo(v[i][j]));
      f[2 * j + 1] = code(hi(v[i][j]));
    }
    u32x2 o;
    if constexpr (E4M3) o = {pack_e4m3x4(f[0], f[1], f[2], f[3]), pack_e4m3x4(f[4], f[5], f[6], f[7])};
    else o = {pack_i8x4(f[0], f[1], f[2], f[3]), pack_i8x4(f[4], f[5], f[6], f[7])};
    if (!finite) o = u32x2{0, 0};
    store8_bytes(q, c, a.cols, o);
  }
}

template <int WAVES, int NV, bool E4M3>
__global__ __launch_bounds__(threads_of(WAVES)) void quantize_rows(QuantizeArgs a) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int t = WAVES == 1 ? lane : (int)threadIdx.x;
  int phase = 0;
  const int64_t step = (int64_t)gridDim.x * rows_of(WAVES);
  for (int64_t row = (int64_t)blockIdx.x * rows_of(WAVES) + (WAVES == 1 ? wave : 0); row < a.rows;
       row += step, phase ^= 1)
    quantize_row<WAVES, NV, E4M3>(a, row, t, wave, lane, phase);
}

typedef void (*quantize_fn)(QuantizeArgs);
template <int WAVES, bool E4M3>
quantize_fn pick(int nv) {
  return nv == 1 ? quantize_rows<WAVES, 1, E4M3>
                 : (nv == 2 ? quantize_rows<WAVES, 2, E4M3> : quantize_rows<WAVES, 4, E4M3>);
}
template <bool E4M3>
quantize_fn pick_shape(NormShape s) {
  if (s.vectors == 8) return quantize_rows<4, 8, E4M3>;
  return s.waves == 1 ? pick<1, E4M3>(s.vectors) : (s.waves == 4 ? pick<4, E4M3>(s.vectors) : pick<16, E4M3>(s.vectors));
}

}  // namespace

// The norm's shapes, but many rows of 8193 to 16384 columns are shared by four
// waves with eight vectors a lane: a wave has more bytes on their way before
// the first wait (8192 x 16384: 74 us, 90 with sixteen waves and two vectors).
// Few rows are better off with more waves.
NormShape quantize_shape(int64_t rows, int64_t cols) {
  const NormShape s = norm_shape(rows, cols);
  return rows > 256 && s.waves == 16 && s.vectors <= 2 ? NormShape{4, 8} : s;
}

hipError_t launch_quantize(const QuantizeArgs& a, bool e4m3, hipStream_t stream) {
  const NormShape s = quantize_shape(a.rows, a.cols);
  const quantize_fn f = e4m3 ? pick_shape<true>(s) : pick_shape<false>(s);
  int64_t grid = (a.rows + rows_of(s.waves) - 1) / rows_of(s.waves);
  if (grid > (1 << 20)) grid = 1 << 20;  // a launch holds fewer than 2^32 threads
  hipLaunchKernelGGL(f, dim3((uint32_t)grid), dim3(threads_of(s.waves)), 0, stream, a);
  return hipGetLastError();
}

}  // namespace migemm

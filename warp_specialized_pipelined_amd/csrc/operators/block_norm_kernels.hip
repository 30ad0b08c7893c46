// block_norm_kernels.hip -- what stands between two blocks: the norm of a
// block's output x, its gate and scale, the residual's addition and the next
// block's norm, and the gradients.
//
// Forward, per row of n columns:
//   p = x post_rstd,  post_rstd = 1 / sqrt(sum x^2 / n + eps),  u = p w_post
//   (without the norm behind the block, u = x)
//   h = residual r + branch sigmoid(z) u          (without a gate, sigmoid: 1)
//   rstd = 1 / sqrt(sum h^2 / n + eps)
//   y = h rstd w in bf16; or with top = max |h w| codes h w (448 or 127) / top
// h is rounded once, where it is stored; the second norm reads it before that.
//
// Backward, with n2 = h rstd (h as stored), g = dy, s = sigmoid(z):
//   d = dh + rstd (g w - n2 mean(g w n2)),     dw = sum over rows of g n2
//   dr = residual d,   v = branch d,   dz = v u s (1 - s),   v = v s
//   dx = post_rstd (v w_post - p mean(v w_post p)),  dw_post = sum of v p
//   (without the norm behind the block, dx = v)
//
// Bound: memory (9 to 16 bytes an element).  A row is read once, 16 bytes a
// lane, and stays in registers through both reductions.
#include <hip/hip_runtime.h>

#include "../kernel/gfx950.hpp"
#include "operators.h"
#include "rows.hpp"

namespace migemm {
namespace {

enum RowType { kRowBf16, kRowE4M3, kRowInt8 };

__device__ __forceinline__ float element(const u32x4& v, int e) { return e & 1 ? hi(v[e >> 1]) : lo(v[e >> 1]); }

// s = 1 / (1 + exp(-z)) and its derivative s (1 - s), both from exp(-|z|): no
// overflow, and nothing lost where s is next to 1.
struct Gate {
  float s, ds;
  __device__ __forceinline__ explicit Gate(float z) {
    const float e = __builtin_amdgcn_exp2f(-fabsf(z) * 1.4426950408889634f), r = 1.0f / (1.0f + e);
    s = z < 0.0f ? e * r : r;
    ds = e * r * r;
  }
};

// The sum over the row of every lane's v, given to all of them: WAVES waves
// share the row, `buffer` holds a sum of each.
template <int WAVES>
__device__ __forceinline__ float row_sum(float v, float* buffer, int wave, int lane) {
  v = wave_sum(v);
  if constexpr (WAVES > 1) {
    if (lane == 0) buffer[wave] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < WAVES; ++i) v += buffer[i];
  }
  return v;
}

template <int WAVES, int NV, bool GATE, RowType Y>
__device__ __forceinline__ void block_norm_row(const BlockNormArgs& a, int64_t row, int t, int wave, int lane,
                                               int phase) {
  constexpr int kLanes = 64 * WAVES;
  // Two buffers each: a wave that is already at its next row writes the other
  // ones, and cannot come round to these before a barrier between.
  __shared__ float posts[2][WAVES], sums[2][WAVES];
  __shared__ uint32_t tops[2][WAVES];
  const auto row_of = [&](const void* m, int64_t rs) { return static_cast<const unsigned short*>(m) + row * rs; };
  const auto at = [&](int i) { return (int64_t)(i * kLanes + t) * 8; };
  const unsigned short* x = row_of(a.x, a.x_rs);
  const unsigned short* r = row_of(a.r, a.r_rs);
  const unsigned short* w = static_cast<const unsigned short*>(a.weight);
  const unsigned short* pw = static_cast<const unsigned short*>(a.post_weight);
  u32x4 xv[NV], rv[NV], zv[NV], wv[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) xv[i] = load8(x, at(i), a.cols);
  if constexpr (GATE) {
    const unsigned short* z = row_of(a.z, a.z_rs);
#pragma unroll
    for (int i = 0; i < NV; ++i) zv[i] = load8(z, at(i), a.cols);
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) rv[i] = load8(r, at(i), a.cols);
#pragma unroll
  for (int i = 0; i < NV; ++i) wv[i] = load8(w, at(i), a.cols);
  // With one vector a lane, where a row's latency counts, w_post is on its way
  // before the first sum, too; else it is read behind it, from the caches.
  u32x4 early = {0, 0, 0, 0};
  if (NV == 1 && a.post_weight) early = load8(pw, at(0), a.cols);

  float post = 1.0f;
  if (a.post_weight) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) s += element(xv[i], e) * element(xv[i], e);
    post = rsqrtf(row_sum<WAVES>(s, posts[phase], wave, lane) / (float)a.cols + a.eps);
    if (t == 0) a.post_rstd[row] = post;
  }
  float h[NV][8], sum = 0.0f;
  uint32_t top = 0;
  unsigned short* ho = static_cast<unsigned short*>(a.h) + row * a.h_rs;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    u32x4 pv = early;
    if (NV > 1 && a.post_weight) pv = load8(pw, at(i), a.cols);
    u32x4 o;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float u = element(xv[i], e);
      if (a.post_weight) u = u * post * element(pv, e);
      if constexpr (GATE) u *= Gate(element(zv[i], e)).s;
      const float v = a.residual * element(rv[i], e) + a.branch * u;
      h[i][e] = v;
      sum += v * v;
      if constexpr (Y != kRowBf16) {
        const uint32_t b = __float_as_uint(v * element(wv[i], e)) & 0x7FFFFFFFu;
        top = b > top ? b : top;
      }
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) o[q] = pack_bf16x2(h[i][2 * q], h[i][2 * q + 1]);
    store8(ho, at(i), a.cols, o);
  }
  if constexpr (Y != kRowBf16) {
    top = wave_max_bits(top);
    if (WAVES > 1 && lane == 0) tops[phase][wave] = top;
  }
  const float rstd = rsqrtf(row_sum<WAVES>(sum, sums[phase], wave, lane) / (float)a.cols + a.eps);
  if (t == 0) a.rstd[row] = rstd;
  if constexpr (Y == kRowBf16) {
    unsigned short* y = static_cast<unsigned short*>(a.y) + row * a.y_rs;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      u32x4 o;
#pragma unroll
      for (int q = 0; q < 4; ++q)
        o[q] = pack_bf16x2(h[i][2 * q] * rstd * lo(wv[i][q]), h[i][2 * q + 1] * rstd * hi(wv[i][q]));
      store8(y, at(i), a.cols, o);
    }
  } else {
    if constexpr (WAVES > 1) {
#pragma unroll
      for (int i = 0; i < WAVES; ++i) top = tops[phase][i] > top ? tops[phase][i] : top;
    }
    constexpr float kTop = Y == kRowE4M3 ? kE4M3Max : 127.0f;
    const float largest = __uint_as_float(top);
    // Not a finite row: an e4m3 row keeps its NaN codes, an int8 one is zeros
    // with a NaN for its scale.
    const bool finite = top < 0x7F800000u;
    if (t == 0) a.scale[row] = finite || Y == kRowE4M3 ? largest * rstd / kTop : NAN;
    // Rows of values so small that kTop / largest would overflow are lifted.
    const float lift = largest < 0x1p-96f ? 0x1p96f : 1.0f;
    const float inv = largest == 0.0f ? 0.0f : kTop / (largest * lift);
    unsigned char* y = static_cast<unsigned char*>(a.y) + row * a.y_rs;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float v[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = h[i][e] * element(wv[i], e) * lift * inv;
      u32x2 o;
      if constexpr (Y == kRowE4M3) {
        o = {pack_e4m3x4(v[0], v[1], v[2], v[3]), pack_e4m3x4(v[4], v[5], v[6], v[7])};
      } else {
        o = {pack_i8x4(v[0], v[1], v[2], v[3]), pack_i8x4(v[4], v[5], v[6], v[7])};
        if (!finite) o = u32x2{0, 0};
      }
      store8_bytes(y, at(i), a.cols, o);
    }
  }
}

template <int WAVES, int NV, bool GATE, RowType Y>
__global__ __launch_bounds__(threads_of(WAVES)) void block_norm_forward(BlockNormArgs a) {
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int t = WAVES == 1 ? lane : (int)threadIdx.x;
  int phase = 0;
  const int64_t step = (int64_t)gridDim.x * rows_of(WAVES);
  for (int64_t row = (int64_t)blockIdx.x * rows_of(WAVES) + (WAVES == 1 ? wave : 0); row < a.rows;
       row += step, phase ^= 1)
    block_norm_row<WAVES, NV, GATE, Y>(a, row, t, wave, lane, phase);
}

// The workgroup's sums of its columns go to its row of the workspace (dw's,
// then dw_post's); block_norm_sum_partials adds those rows in a fixed order.
// One workgroup alone writes the gradients itself.
template <int WAVES, int NV>
__device__ __forceinline__ void put_sums(const BlockNormArgs& a, const float (&dw)[NV][8], float* p, int t, int wave,
                                         int lane) {
  constexpr int kLanes = 64 * WAVES;
  if constexpr (WAVES == 1) {
    __shared__ float all[4][NV * 512];
    __syncthreads();
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

// Each walker (a workgroup, or with WAVES = 1 a wave) takes rows walker,
// walker + walkers, ... and keeps its columns' sums in registers.
template <int WAVES, int NV, bool GATE, bool POST>
__global__ __launch_bounds__(threads_of(WAVES), WAVES == 16 ? 4 : 2) void block_norm_backward(BlockNormArgs a) {
  constexpr int kLanes = 64 * WAVES;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  const int64_t walker = (int64_t)blockIdx.x * rows_of(WAVES) + (WAVES == 1 ? wave : 0);
  const int64_t walkers = (int64_t)gridDim.x * rows_of(WAVES);
  const int t = WAVES == 1 ? lane : (int)threadIdx.x;
  const unsigned short* w = static_cast<const unsigned short*>(a.weight);
  const unsigned short* pw = static_cast<const unsigned short*>(a.post_weight);
  const float cols = (float)a.cols;
  const auto at = [&](int i) { return (int64_t)(i * kLanes + t) * 8; };
  __shared__ float sums[2][WAVES], posts[2][WAVES];

  u32x4 wv[NV], pv[POST ? NV : 1];
  float dw[NV][8], dpw[POST ? NV : 1][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    wv[i] = load8(w, at(i), a.cols);
    if constexpr (POST) pv[i] = load8(pw, at(i), a.cols);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      dw[i][e] = 0.0f;
      if constexpr (POST) dpw[i][e] = 0.0f;
    }
  }
  int phase = 0;
  for (int64_t row = walker; row < a.rows; row += walkers, phase ^= 1) {
    const auto row_of = [&](const void* m, int64_t rs) { return static_cast<const unsigned short*>(m) + row * rs; };
    const auto load = [&](u32x4 (&v)[NV], const void* m, int64_t rs) {
      const unsigned short* p = row_of(m, rs);
#pragma unroll
      for (int i = 0; i < NV; ++i) v[i] = load8(p, at(i), a.cols);
    };
    u32x4 gv[NV], hv[NV], dv[NV], xv[NV], zv[NV];
    load(gv, a.dy, a.dy_rs);
    load(hv, a.h, a.h_rs);
    if (a.dh) {
      load(dv, a.dh, a.dh_rs);
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i) dv[i] = u32x4{0, 0, 0, 0};
    }
    if constexpr (GATE || POST) load(xv, a.x, a.x_rs);
    if constexpr (GATE) load(zv, a.z, a.z_rs);
    const float rstd = a.rstd[row], post = POST ? a.post_rstd[row] : 1.0f;
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float n = element(hv[i], e) * rstd, g = element(gv[i], e);
        dw[i][e] += g * n;
        s += g * element(wv[i], e) * n;
      }
    const float mean = row_sum<WAVES>(s, sums[phase], wave, lane) / cols;
    unsigned short* dr = static_cast<unsigned short*>(a.dr) + row * a.dr_rs;
    unsigned short* dz = static_cast<unsigned short*>(a.dz) + row * a.dz_rs;
    unsigned short* dx = static_cast<unsigned short*>(a.dx) + row * a.dx_rs;
    // v of the row, in fp32, over what is needed of it no more.
    float v[NV][8];
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      u32x4 o, oz;
      float f[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float n = element(hv[i], e) * rstd;
        const float d = element(dv[i], e) + rstd * (element(gv[i], e) * element(wv[i], e) - n * mean);
        f[e] = a.residual * d;
        v[i][e] = a.branch * d;
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) o[q] = pack_bf16x2(f[2 * q], f[2 * q + 1]);
      store8(dr, at(i), a.cols, o);
      if constexpr (GATE) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const Gate gate(element(zv[i], e));
          float u = element(xv[i], e);
          if constexpr (POST) u = u * post * element(pv[i], e);
          f[e] = v[i][e] * u * gate.ds;
          v[i][e] *= gate.s;
        }
#pragma unroll
        for (int q = 0; q < 4; ++q) oz[q] = pack_bf16x2(f[2 * q], f[2 * q + 1]);
        store8(dz, at(i), a.cols, oz);
      }
      if constexpr (POST) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float p = element(xv[i], e) * post;
          dpw[i][e] += v[i][e] * p;
          v[i][e] *= element(pv[i], e);
          s += v[i][e] * p;
        }
      }
    }
    float post_mean = 0.0f;
    if constexpr (POST) post_mean = row_sum<WAVES>(s, posts[phase], wave, lane) / cols;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      u32x4 o;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if constexpr (POST) v[i][e] = post * (v[i][e] - element(xv[i], e) * post * post_mean);
#pragma unroll
      for (int q = 0; q < 4; ++q) o[q] = pack_bf16x2(v[i][2 * q], v[i][2 * q + 1]);
      store8(dx, at(i), a.cols, o);
    }
  }
  const bool alone = a.partial_rows == 1;
  float* p = a.partials + (int64_t)blockIdx.x * a.cols * (POST ? 2 : 1);
  put_sums<WAVES>(a, dw, alone ? a.dweight : p, t, wave, lane);
  if constexpr (POST) put_sums<WAVES>(a, dpw, alone ? a.dpost_weight : p + a.cols, t, wave, lane);
}

// The sum over partial rows of column c of `width` (cols, twice with a norm
// behind the block): GROUPS threads a column add every GROUPS-th row, then
// one adds their sums in order.
template <int GROUPS, int COLS>
__global__ __launch_bounds__(GROUPS * COLS) void block_norm_sum_partials(BlockNormArgs a, int64_t width) {
  const int col = threadIdx.x % COLS, group = threadIdx.x / COLS;
  const int64_t c = (int64_t)blockIdx.x * COLS + col;
  float s = 0.0f;
  if (c < width)
#pragma unroll 8
    for (int64_t p = group; p < a.partial_rows; p += GROUPS) s += a.partials[p * width + c];
  if constexpr (GROUPS > 1) {
    __shared__ float part[GROUPS][COLS + 1];
    part[group][col] = s;
    __syncthreads();
    if (group != 0) return;
#pragma unroll
    for (int i = 1; i < GROUPS; ++i) s += part[i][col];
  }
  if (c < a.cols) a.dweight[c] = s;
  else if (c < width) a.dpost_weight[c - a.cols] = s;
}

typedef void (*block_norm_fn)(BlockNormArgs);
template <int WAVES, int NV>
block_norm_fn forward_of(bool gate, int y) {
  if (gate)
    return y == kRowBf16 ? block_norm_forward<WAVES, NV, true, kRowBf16>
                         : (y == kRowE4M3 ? block_norm_forward<WAVES, NV, true, kRowE4M3>
                                          : block_norm_forward<WAVES, NV, true, kRowInt8>);
  return y == kRowBf16 ? block_norm_forward<WAVES, NV, false, kRowBf16>
                       : (y == kRowE4M3 ? block_norm_forward<WAVES, NV, false, kRowE4M3>
                                        : block_norm_forward<WAVES, NV, false, kRowInt8>);
}
template <int WAVES, int NV>
block_norm_fn backward_of(bool gate, bool post) {
  if (gate) return post ? block_norm_backward<WAVES, NV, true, true> : block_norm_backward<WAVES, NV, true, false>;
  return post ? block_norm_backward<WAVES, NV, false, true> : block_norm_backward<WAVES, NV, false, false>;
}
// (16 waves: rows of up to kBlockNormMaxCols take two vectors a lane.)
block_norm_fn forward_pick(NormShape s, bool gate, int y) {
  if (s.waves == 16) return s.vectors == 1 ? forward_of<16, 1>(gate, y) : forward_of<16, 2>(gate, y);
  if (s.waves == 4)
    return s.vectors == 1 ? forward_of<4, 1>(gate, y)
                          : (s.vectors == 2 ? forward_of<4, 2>(gate, y) : forward_of<4, 4>(gate, y));
  return s.vectors == 1 ? forward_of<1, 1>(gate, y)
                        : (s.vectors == 2 ? forward_of<1, 2>(gate, y) : forward_of<1, 4>(gate, y));
}
block_norm_fn backward_pick(NormShape s, bool gate, bool post) {
  if (s.waves == 16) return s.vectors == 1 ? backward_of<16, 1>(gate, post) : backward_of<16, 2>(gate, post);
  if (s.waves == 4)
    return s.vectors == 1 ? backward_of<4, 1>(gate, post)
                          : (s.vectors == 2 ? backward_of<4, 2>(gate, post) : backward_of<4, 4>(gate, post));
  return s.vectors == 1 ? backward_of<1, 1>(gate, post)
                        : (s.vectors == 2 ? backward_of<1, 2>(gate, post) : backward_of<1, 4>(gate, post));
}

}  // namespace

hipError_t launch_block_norm_forward(const BlockNormArgs& a, int y_type, hipStream_t stream) {
  const NormShape s = norm_shape(a.rows, a.cols);
  const block_norm_fn f = forward_pick(s, a.z != nullptr, y_type);
  int64_t grid = (a.rows + rows_of(s.waves) - 1) / rows_of(s.waves);
  if (grid > (1 << 20)) grid = 1 << 20;  // a launch holds fewer than 2^32 threads
  hipLaunchKernelGGL(f, dim3((uint32_t)grid), dim3(threads_of(s.waves)), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_block_norm_backward(const BlockNormArgs& a, hipStream_t stream) {
  const NormShape s = norm_shape(a.rows, a.cols);
  const bool post = a.dpost_weight != nullptr;
  if (a.partial_rows > 0) {
    const block_norm_fn f = backward_pick(s, a.dz != nullptr, post);
    hipLaunchKernelGGL(f, dim3((uint32_t)a.partial_rows), dim3(threads_of(s.waves)), 0, stream, a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || a.partial_rows == 1) return e;
  }
  const int64_t width = a.cols * (post ? 2 : 1);
  // Few rows of sums: a thread a column.
  if (a.partial_rows <= 16)
    hipLaunchKernelGGL((block_norm_sum_partials<1, 64>), dim3((uint32_t)((width + 63) / 64)), dim3(64), 0, stream, a,
                       width);
  else
    hipLaunchKernelGGL((block_norm_sum_partials<32, 32>), dim3((uint32_t)((width + 31) / 32)), dim3(1024), 0, stream,
                       a, width);
  return hipGetLastError();
}

}  // namespace migemm

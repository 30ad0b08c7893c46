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
// Bound: memory (forward 7 bytes an element to codes, with a gate 9; backward
// with everything 16).  A row is read once, 16 bytes a lane, and stays in
// registers through both reductions.  8192 x 8192 to e4m3 with a gate: 115 us,
// 5.3 TB/s; one row of 8192: 4.2 us, two reductions and three waits for memory;
// backward 8192 x 4096 with everything: 109 us and 5 for the columns' sums, 4.9
// TB/s.  Rows of an odd number of columns have kernels of their own (RowView),
// which clear the value past the last once all of a row's loads are on their
// way: 8192 x 3001 96 us backward and 56 forward; 173 and 72 with a branch and
// a wait at each load, and 104 and 57 with a branch for the row in all kernels.
#include <hip/hip_runtime.h>

#include "../kernel/gfx950.hpp"
#include "operators.h"
#include "rows.hpp"

namespace migemm {
namespace {

enum RowType { kRowBf16, kRowE4M3, kRowInt8 };

__device__ __forceinline__ float element(const u32x4& v, int e) { return e & 1 ? hi(v[e >> 1]) : lo(v[e >> 1]); }

// s = 1 / (1 + exp(-z)) and its derivative s (1 - s), both from exp(-|z|): no
// overflow, and nothing lost where s is next to 1.  What the product with log2 e
// rounds off is put back (or exp would be off by |z| 2^-24), and the reciprocal
// is refined: a code of y changes where its value crosses a border of two, which
// it does as often as h is off.
struct Gate {
  float s, ds;
  __device__ __forceinline__ explicit Gate(float z) {
    constexpr float kLog2e = 1.44269502f, kRest = 1.92596302e-8f, kLn2 = 0.693147182f;  // log2 e in two parts
    const float m = fminf(fabsf(z), 128.0f);  // (exp is 0 in fp32 from 104 on)
    const float t = -m * kLog2e, rest = -m * kRest - fmaf(m, kLog2e, t);
    const float x = __builtin_amdgcn_exp2f(t), e = fmaf(x, rest * kLn2, x);
    const float d = 1.0f + e, q = __builtin_amdgcn_rcpf(d), r = fmaf(q, fmaf(-d, q, 1.0f), q);
    s = z < 0.0f ? e * r : r;
    ds = e * r * r;
    if (z != z) s = ds = z;
  }
};

// Values the compiler cannot see through: what was unpacked from them before
// is unpacked again where it is needed, instead of being held in registers
// twice as wide across a reduction (which did not fit: 8192 x 8192 backward
// took 998 us with spilled registers).
template <int N>
__device__ __forceinline__ void hide(u32x4 (&v)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) asm volatile("" : "+v"(v[i]));
}

__device__ __forceinline__ void apart() { __builtin_amdgcn_sched_barrier(0); }

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

template <int WAVES, int NV, bool GATE, RowType Y, bool ODD>
__device__ __forceinline__ void block_norm_row(const BlockNormArgs& a, int64_t row, int t, int wave, int lane,
                                               int phase) {
  typedef RowView<ODD> Row;
  constexpr int kLanes = 64 * WAVES;
  // Two buffers each: a wave that is already at its next row writes the other
  // ones, and cannot come round to these before a barrier between.
  __shared__ float posts[2][WAVES], sums[2][WAVES];
  __shared__ uint32_t tops[2][WAVES];
  const auto at = [&](int i) { return (i * kLanes + t) * 8; };
  const auto load = [&](u32x4 (&v)[NV], const void* m, int64_t rs) {
    const Row from = Row::in(m, row * rs, a.cols);
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = from.load(at(i));
  };
  const Row pw = Row::in(a.post_weight, 0, a.post_weight ? a.cols : 0);
  u32x4 xv[NV], rv[NV], zv[NV], wv[NV];
  load(xv, a.x, a.x_rs);
  if constexpr (GATE) load(zv, a.z, a.z_rs);
  load(rv, a.r, a.r_rs);
  load(wv, a.weight, 0);
  // With one vector a lane, where a row's latency counts, w_post is on its way
  // before the first sum, too; else it is read behind it, from the caches.
  u32x4 early = {0, 0, 0, 0};
  if (NV == 1 && a.post_weight) early = pw.load(at(0));
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    Row::clear_past(xv[i], at(i), a.cols);
    if constexpr (GATE) Row::clear_past(zv[i], at(i), a.cols);
    Row::clear_past(rv[i], at(i), a.cols);
    Row::clear_past(wv[i], at(i), a.cols);
  }
  Row::clear_past(early, at(0), a.cols);

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
  const Row ho = Row::template out<2>(a.h, row * a.h_rs, a.cols);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    u32x4 pv = early;
    if (NV > 1 && a.post_weight) pv = pw.load_cleared(at(i));
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
    ho.store(at(i), o);
  }
  if constexpr (Y != kRowBf16) {
    top = wave_max_bits(top);
    if (WAVES > 1 && lane == 0) tops[phase][wave] = top;
  }
  const float rstd = rsqrtf(row_sum<WAVES>(sum, sums[phase], wave, lane) / (float)a.cols + a.eps);
  if (t == 0) a.rstd[row] = rstd;
  if constexpr (Y == kRowBf16) {
    const Row y = Row::template out<2>(a.y, row * a.y_rs, a.cols);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      u32x4 o;
#pragma unroll
      for (int q = 0; q < 4; ++q)
        o[q] = pack_bf16x2(h[i][2 * q] * rstd * lo(wv[i][q]), h[i][2 * q + 1] * rstd * hi(wv[i][q]));
      y.store(at(i), o);
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
    const Row y = Row::template out<1>(a.y, row * a.y_rs, a.cols);
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
      y.store_bytes(at(i), o);
    }
  }
}

template <int WAVES, int NV, bool GATE, RowType Y, bool ODD>
__global__ __launch_bounds__(threads_of(WAVES)) void block_norm_forward(BlockNormArgs a) {
  const int wave = wave_id(), lane = threadIdx.x & 63;
  const int t = WAVES == 1 ? lane : (int)threadIdx.x;
  int phase = 0;
  const int64_t step = (int64_t)gridDim.x * rows_of(WAVES);
  for (int64_t row = (int64_t)blockIdx.x * rows_of(WAVES) + (WAVES == 1 ? wave : 0); row < a.rows;
       row += step, phase ^= 1)
    block_norm_row<WAVES, NV, GATE, Y, ODD>(a, row, t, wave, lane, phase);
}

// What a lane holds of a row: the gradients that come in, h as it was stored,
// and the block's output and its gate.
template <int NV, bool GATE, bool POST, bool ODD>
struct BackwardRow {
  typedef RowView<ODD> Row;
  u32x4 g[NV], h[NV], d[NV], x[GATE || POST ? NV : 1], z[GATE ? NV : 1];
  float rstd, post;
  // (A row past the last: zeros, and nothing is read.)
  template <class At>
  __device__ __forceinline__ void load(const BlockNormArgs& a, int64_t row, At&& at) {
    const bool in = row < a.rows;
    const auto all = [&](u32x4* v, const void* m, int64_t rs) {
      const Row from = Row::in(m, row * rs, in && m ? a.cols : 0);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        v[i] = from.load(at(i));
        apart();  // (in this order: 8192 x 5000 178 us without, 160 with this and the stores kept in theirs)
      }
    };
    all(g, a.dy, a.dy_rs);
    all(h, a.h, a.h_rs);
    all(d, a.dh, a.dh_rs);
    if constexpr (GATE || POST) all(x, a.x, a.x_rs);
    if constexpr (GATE) all(z, a.z, a.z_rs);
    rstd = in ? a.rstd[row] : 0.0f;
    post = POST && in ? a.post_rstd[row] : 1.0f;
  }
  template <class At>
  __device__ __forceinline__ void clear_past(int64_t cols, At&& at) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      Row::clear_past(g[i], at(i), cols);
      Row::clear_past(h[i], at(i), cols);
      Row::clear_past(d[i], at(i), cols);
      if constexpr (GATE || POST) Row::clear_past(x[i], at(i), cols);
      if constexpr (GATE) Row::clear_past(z[i], at(i), cols);
    }
  }
};

// Each walker (a workgroup, or with WAVES = 1 a wave) takes rows walker,
// walker + walkers, ..., the next one on its way while a row is worked on (not
// with 16 waves, which come with few rows and half the registers), and adds up
// its columns' sums: in registers, or, with WIDE, where those would not
// hold them beside four vectors of a row, in LDS (each lane its own columns).
// The workgroup's sums go to its row of the workspace (dw's, then dw_post's);
// block_norm_sum_partials adds those rows in a fixed order.  One workgroup alone
// writes the gradients itself.
template <int WAVES, int NV, bool GATE, bool POST, bool WIDE, bool ODD>
__global__ __launch_bounds__(threads_of(WAVES), WAVES == 16 ? 4 : 2) void block_norm_backward(BlockNormArgs a) {
  typedef RowView<ODD> Row;
  constexpr int kLanes = 64 * WAVES;
  static_assert(!WIDE || WAVES > 1, "a wave's own sums stay in registers");
  // (WIDE: the weights are read again for each row, from the caches.)
  constexpr bool kReload = WIDE, kAhead = WAVES < 16;
  const int wave = wave_id(), lane = threadIdx.x & 63;
  const int64_t walker = (int64_t)blockIdx.x * rows_of(WAVES) + (WAVES == 1 ? wave : 0);
  const int64_t walkers = (int64_t)gridDim.x * rows_of(WAVES);
  const int t = WAVES == 1 ? lane : (int)threadIdx.x;
  const float cols = (float)a.cols;
  const auto at = [&](int i) { return (i * kLanes + t) * 8; };
  __shared__ float sums[2][WAVES], posts[2][WAVES];
  // WIDE: [dw, dw_post][vector][half][lane], 16 bytes each.
  f32x4* lds = WIDE ? (f32x4*)lds_at(0) : nullptr;
  const auto slot = [&](int which, int i, int half) { return ((which * NV + i) * 2 + half) * kLanes + t; };

  const Row w = Row::in(a.weight, 0, a.cols), pw = Row::in(a.post_weight, 0, POST ? a.cols : 0);
  u32x4 wv[NV], pv[POST ? NV : 1];
  float dw[WIDE ? 1 : NV][8], dpw[POST && !WIDE ? NV : 1][8];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if constexpr (WIDE) {
#pragma unroll
      for (int k = 0; k < (POST ? 4 : 2); ++k) lds[slot(k / 2, i, k % 2)] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    } else {
      if constexpr (!kReload) wv[i] = w.load_cleared(at(i));
      if constexpr (POST && !kReload) pv[i] = pw.load_cleared(at(i));
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        dw[i][e] = 0.0f;
        if constexpr (POST) dpw[i][e] = 0.0f;
      }
    }
  }
  BackwardRow<NV, GATE, POST, ODD> c, next;
  if constexpr (kAhead) next.load(a, walker, at);
  int phase = 0;
  for (int64_t row = walker; row < a.rows; row += walkers, phase ^= 1) {
    if constexpr (kAhead) c = next;
    else c.load(a, row, at);
    if constexpr (kAhead && !WIDE) next.load(a, row + walkers, at);
    c.clear_past(a.cols, at);
    // (Pairs of elements are kept apart: all of a row's at once would not fit the
    // registers.)
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if constexpr (kReload) wv[i] = w.load_cleared(at(i));
      float f[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (e % 2 == 0) apart();
        const float n = element(c.h[i], e) * c.rstd, g = element(c.g[i], e);
        f[e] = g * n;
        s += g * element(wv[i], e) * n;
        if constexpr (!WIDE) dw[i][e] += f[e];
      }
      if constexpr (WIDE) {
        lds[slot(0, i, 0)] += f32x4{f[0], f[1], f[2], f[3]};
        lds[slot(0, i, 1)] += f32x4{f[4], f[5], f[6], f[7]};
      }
    }
    const float mean = row_sum<WAVES>(s, sums[phase], wave, lane) / cols;
    hide(c.g);
    hide(c.h);
    hide(wv);
    if constexpr (POST && !kReload) hide(pv);
    const Row dr = Row::template out<2>(a.dr, row * a.dr_rs, a.cols);
    const Row dz = Row::template out<2>(a.dz, row * a.dz_rs, a.cols);
    const Row dx = Row::template out<2>(a.dx, row * a.dx_rs, a.cols);
    float v[NV][8];
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if constexpr (POST && kReload) pv[i] = pw.load_cleared(at(i));
      u32x4 o, oz;
      float f[8];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        apart();
        float r[2], z[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int e = 2 * q + k;
          const float n = element(c.h[i], e) * c.rstd;
          const float d = element(c.d[i], e) + c.rstd * (element(c.g[i], e) * element(wv[i], e) - n * mean);
          r[k] = a.residual * d;
          float g = a.branch * d;
          const float p = GATE || POST ? element(c.x[i], e) * c.post : 0.0f;
          const float pw_e = POST ? element(pv[i], e) : 1.0f;
          if constexpr (GATE) {
            const Gate gate(element(c.z[i], e));
            z[k] = g * (p * pw_e) * gate.ds;
            g *= gate.s;
          }
          if constexpr (POST) {
            f[e] = g * p;
            if constexpr (!WIDE) dpw[i][e] += f[e];
            g *= pw_e;
            s += g * p;
          }
          v[i][e] = g;
        }
        o[q] = pack_bf16x2(r[0], r[1]);
        if constexpr (GATE) oz[q] = pack_bf16x2(z[0], z[1]);
      }
      dr.store(at(i), o);
      if constexpr (GATE) dz.store(at(i), oz);
      apart();
      if constexpr (POST && WIDE) {
        lds[slot(1, i, 0)] += f32x4{f[0], f[1], f[2], f[3]};
        lds[slot(1, i, 1)] += f32x4{f[4], f[5], f[6], f[7]};
      }
    }
    if constexpr (WIDE) next.load(a, row + walkers, at);  // (over the registers that are free now)
    float post_mean = 0.0f;
    if constexpr (POST) {
      post_mean = row_sum<WAVES>(s, posts[phase], wave, lane) / cols;
      hide(c.x);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      u32x4 o;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        apart();
        float x[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int e = 2 * q + k;
          x[k] = POST ? c.post * (v[i][e] - element(c.x[i], e) * c.post * post_mean) : v[i][e];
        }
        o[q] = pack_bf16x2(x[0], x[1]);
      }
      dx.store(at(i), o);
    }
  }
  const bool alone = a.partial_rows == 1;
  float* p = a.partials + (int64_t)blockIdx.x * a.cols * (POST ? 2 : 1);
#pragma unroll
  for (int which = 0; which < (POST ? 2 : 1); ++which) {
    float* to = which == 0 ? (alone ? a.dweight : p) : (alone ? a.dpost_weight : p + a.cols);
    if constexpr (WAVES == 1) {
      // The four waves' sums, added in order.
      __shared__ float all[4][NV * 512];
      __syncthreads();
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) all[wave][at(i) + e] = which == 0 ? dw[i][e] : dpw[POST ? i : 0][e];
      __syncthreads();
      for (int64_t k = threadIdx.x; k < a.cols; k += 256) to[k] = ((all[0][k] + all[1][k]) + all[2][k]) + all[3][k];
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          f32x4 v;
          if constexpr (WIDE) v = lds[slot(which, i, half)];
          else
#pragma unroll
            for (int e = 0; e < 4; ++e) v[e] = which == 0 ? dw[i][4 * half + e] : dpw[POST ? i : 0][4 * half + e];
          const int64_t k = at(i) + 4 * half;
          if (k + 4 <= a.cols) {
            // (16-byte stores, which need an address that is a multiple of 4.)
            typedef float f32x4_4 __attribute__((ext_vector_type(4), aligned(4)));
            *reinterpret_cast<f32x4_4*>(to + k) = v;
          } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (k + e < a.cols) to[k + e] = v[e];
          }
        }
    }
  }
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
template <int WAVES, int NV, bool ODD>
block_norm_fn forward_of(bool gate, int y) {
  if (gate)
    return y == kRowBf16 ? block_norm_forward<WAVES, NV, true, kRowBf16, ODD>
                         : (y == kRowE4M3 ? block_norm_forward<WAVES, NV, true, kRowE4M3, ODD>
                                          : block_norm_forward<WAVES, NV, true, kRowInt8, ODD>);
  return y == kRowBf16 ? block_norm_forward<WAVES, NV, false, kRowBf16, ODD>
                       : (y == kRowE4M3 ? block_norm_forward<WAVES, NV, false, kRowE4M3, ODD>
                                        : block_norm_forward<WAVES, NV, false, kRowInt8, ODD>);
}
template <int WAVES, int NV, bool WIDE, bool ODD>
block_norm_fn backward_of(bool gate, bool post) {
  if (gate)
    return post ? block_norm_backward<WAVES, NV, true, true, WIDE, ODD>
                : block_norm_backward<WAVES, NV, true, false, WIDE, ODD>;
  return post ? block_norm_backward<WAVES, NV, false, true, WIDE, ODD>
              : block_norm_backward<WAVES, NV, false, false, WIDE, ODD>;
}
template <bool ODD>
block_norm_fn forward_pick(NormShape s, bool gate, int y) {
  if (s.waves == 16) return forward_of<16, 1, ODD>(gate, y);
  if (s.waves == 8) return forward_of<8, 4, ODD>(gate, y);
  if (s.waves == 4)
    return s.vectors == 1 ? forward_of<4, 1, ODD>(gate, y)
                          : (s.vectors == 2 ? forward_of<4, 2, ODD>(gate, y) : forward_of<4, 4, ODD>(gate, y));
  return s.vectors == 1 ? forward_of<1, 1, ODD>(gate, y)
                        : (s.vectors == 2 ? forward_of<1, 2, ODD>(gate, y) : forward_of<1, 4, ODD>(gate, y));
}
template <bool ODD>
block_norm_fn backward_pick(NormShape s, bool gate, bool post) {
  if (s.waves == 16) return backward_of<16, 1, false, ODD>(gate, post);
  if (s.waves == 8)
    return s.vectors == 2 ? backward_of<8, 2, false, ODD>(gate, post) : backward_of<8, 4, true, ODD>(gate, post);
  if (s.waves == 4)
    return s.vectors == 1 ? backward_of<4, 1, false, ODD>(gate, post) : backward_of<4, 2, false, ODD>(gate, post);
  return s.vectors == 1 ? backward_of<1, 1, false, ODD>(gate, post) : backward_of<1, 2, false, ODD>(gate, post);
}
// LDS of the wide backward kernel: both weights' sums of 16384 columns.
constexpr int kWideLds = 2 * 4 * (int)kBlockNormMaxCols;

}  // namespace

// Forward, the norm's shapes, but rows of more than 8192 columns are shared by
// eight waves with four vectors a lane (4096 x 16384: 129 us, 5.2 TB/s).
NormShape block_norm_forward_shape(int64_t rows, int64_t cols) {
  if (cols > 8192) return {8, 4};
  return norm_shape(rows, cols);
}

// Backward a lane holds up to two vectors of a row (of five matrices, their
// sums and the next row's), or four with the sums in LDS (4096 x 16384: 255 us;
// 867 with two vectors and sixteen waves, whose registers did not hold the next
// row).  Few rows, whose latency counts: one vector.
NormShape block_norm_backward_shape(int64_t rows, int64_t cols) {
  if (cols > 8192) return {8, 4};
  if (rows <= 256) return cols <= 512 ? NormShape{1, 1} : (cols <= 2048 ? NormShape{4, 1} : NormShape{16, 1});
  if (cols <= 1024) return {1, cols <= 512 ? 1 : 2};
  if (cols <= 4096) return {4, cols <= 2048 ? 1 : 2};
  return {8, 2};
}

// A second kernel costs about as much as three rows one after another.  As many
// workgroups as the chip holds at once.
int64_t block_norm_partial_rows(int64_t rows, int64_t cols, int cu_count) {
  const int waves = block_norm_backward_shape(rows, cols).waves, at_once = rows_of(waves);
  if (rows <= 3 * at_once) return rows > 0 ? 1 : 0;
  const int64_t groups = (rows + at_once - 1) / at_once, most = (int64_t)cu_count * (waves <= 4 ? 2 : 1);
  return groups < most ? groups : most;
}

hipError_t prepare_block_norm() {
  for (bool gate : {false, true})
    for (bool post : {false, true}) {
      for (block_norm_fn f : {backward_of<8, 4, true, false>(gate, post), backward_of<8, 4, true, true>(gate, post)}) {
        const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(f),
                                                 hipFuncAttributeMaxDynamicSharedMemorySize, kWideLds);
        if (e != hipSuccess) return e;
      }
    }
  return hipSuccess;
}

hipError_t launch_block_norm_forward(const BlockNormArgs& a, int y_type, hipStream_t stream) {
  const NormShape s = block_norm_forward_shape(a.rows, a.cols);
  const bool gate = a.z != nullptr;
  const block_norm_fn f = a.cols & 1 ? forward_pick<true>(s, gate, y_type) : forward_pick<false>(s, gate, y_type);
  int64_t grid = (a.rows + rows_of(s.waves) - 1) / rows_of(s.waves);
  if (grid > (1 << 20)) grid = 1 << 20;  // a launch holds fewer than 2^32 threads
  hipLaunchKernelGGL(f, dim3((uint32_t)grid), dim3(threads_of(s.waves)), 0, stream, a);
  return hipGetLastError();
}

hipError_t launch_block_norm_backward(const BlockNormArgs& a, hipStream_t stream) {
  const NormShape s = block_norm_backward_shape(a.rows, a.cols);
  const bool post = a.dpost_weight != nullptr;
  if (a.partial_rows > 0) {
    const bool gate = a.dz != nullptr;
    const block_norm_fn f = a.cols & 1 ? backward_pick<true>(s, gate, post) : backward_pick<false>(s, gate, post);
    hipLaunchKernelGGL(f, dim3((uint32_t)a.partial_rows), dim3(threads_of(s.waves)), s.vectors == 4 ? kWideLds : 0, stream,
                       a);
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

// operators.h -- internal interface between the operators' plan layer
// (operators_api.cpp) and their kernels: argument blocks and launches.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../kernel/params.hpp"

namespace migemm {

// ------------------------------------------------------------------- norm

struct NormArgs {
  const void* x;        // forward: bf16 input; backward: h, the normed input
  const void* r;        // forward: residual in (NULL: none)
  const void* dy;       // backward
  const void* dh;       // backward: the residual's gradient (NULL: none)
  const void* weight;   // bf16 [cols]
  void* h;              // forward: residual out
  void* y;              // forward: bf16 or e4m3
  void* dx;             // backward
  float* scale;         // forward, e4m3
  float* rstd;          // forward: out; backward: in
  float* dweight;       // backward
  float* partials;      // backward: workspace, one row of cols sums per row walker
  int64_t rows, cols;
  int64_t x_rs, r_rs, h_rs, y_rs, dy_rs, dh_rs, dx_rs;  // elements
  int64_t partial_rows;
  float eps;
};

// Widest row the kernels hold in registers.
constexpr int64_t kNormMaxCols = 16 * 64 * 4 * 8;

// How a row is shared out: waves per row (1, 4 or 16) and 16-byte vectors
// per lane (1, 2 or 4).
struct NormShape {
  int waves, vectors;
};
NormShape norm_shape(int64_t rows, int64_t cols);
// Rows of partial column sums the backward pass leaves in its workspace.
int64_t norm_partial_rows(int64_t rows, int64_t cols, int cu_count);

hipError_t launch_norm_forward(const NormArgs& a, bool e4m3, hipStream_t stream);
hipError_t launch_norm_backward(const NormArgs& a, hipStream_t stream);

// ----------------------------------------------------------------- scaled

// Four fp32 sums.
typedef float mid_piece __attribute__((ext_vector_type(4)));

struct ScaledArgs {
  KernelArgs gemm;       // A, B: e4m3, K-contiguous; strides in elements
  const float* a_scale;  // [M]
  const float* b_scale;  // [N], 16-byte aligned
  mid_piece* partials;   // workspace: the splits' sums
  int32_t splits;
};

// Which kernel takes a product, into how many ranges K is split, the height
// of its tiles where it takes them one after another, and the workspace.
struct ScaledChoice {
  int variant, splits, tile_m;
  int64_t workspace_bytes;
};
ScaledChoice choose_scaled(int64_t M, int64_t N, int64_t K, int cu_count);
// What a variant's kernel is: its tile, its stages of K in LDS (0: none), and
// whether it multiplies the codes as bf16.
struct ScaledKernel {
  int tile_m, tile_n, lds_stages;
  bool exact;
};
ScaledKernel scaled_kernel(int variant);
hipError_t prepare_scaled();
hipError_t launch_scaled(const ScaledArgs& a, int variant, int cu_count, hipStream_t stream);

// ------------------------------------------------------------------- loss

// What the backward pass finds out about its rows.
struct LossHead {
  int count;     // rows that count
  float factor;  // the significand (1 .. 2) of the largest |dloss| of theirs, or 1
};

struct LossArgs {
  KernelArgs gemm;        // the product a kernel forms
  KernelArgs gemm_dx;     // loss_products_mid: dx's, beside dw's
  int64_t T, V, H;
  const void* x;          // the caller's, T x H
  int64_t x_rs, dx_rs;
  const int64_t* target;
  // Forward.  (target, loss, lse and target_logit start at the first of the
  // gemm.M rows that a launch takes.)
  float* loss;
  float* lse;             // backward: in
  float2* parts;          // [V / part_cols][part_rows]: largest logit, sum of exponentials
  int64_t part_rows, part_cols;
  float* target_logit;
  // Backward.
  const float* dloss;
  void* dx;
  LossHead* head;
  int* from;              // [count]: the row's number among T
  unsigned short* rows_x; // [count][rows_ld]
  int64_t rows_ld;
  float* rows_lse;
  float* rows_dloss;
  int* rows_target;
  int64_t first_col;      // the piece's first vocabulary entry
  mid_piece* dx_sums;     // [splits][dx_tiles] tiles of fp32 sums in register order
  mid_piece* dw_sums;     // [dw_splits][tiles of dw]
  int64_t dx_tiles;
  int32_t splits, dw_splits;
  int32_t dx_items;       // loss_products_mid: its workgroups that form dx
  int32_t first_piece, dx_summed;
};

// Tiles of the loss's products: 256 x 256 (the GEMM's K loop), smaller
// (midtile.hpp), and for the logits alone 16 x 32 (rowblock.hpp).
enum LossTile { kLoss256, kLoss128, kLoss64x128, kLoss64, kLossTiles, kLossRows = kLossTiles };
constexpr int kLossTileM[] = {256, 128, 64, 64, 16};
constexpr int kLossTileN[] = {256, 128, 128, 64, 32};
inline int64_t loss_tiles(int tile, int64_t rows, int64_t cols) {
  return ((rows + kLossTileM[tile] - 1) / kLossTileM[tile]) * ((cols + kLossTileN[tile] - 1) / kLossTileN[tile]);
}

// The tiles of the logits forward and backward and of the backward pass's
// products, and the ways K of those is split.  `piece`: vocabulary entries
// that the backward pass takes at a time.
struct LossChoice {
  int forward, gradient, dx, dw, dx_splits, dw_splits;
};
LossChoice choose_loss(int64_t T, int64_t V, int64_t H, int64_t piece, int cu_count);

hipError_t prepare_loss();
hipError_t launch_loss_forward(const LossArgs& s, int tile, int cu_count, hipStream_t stream);
hipError_t launch_loss_rows(const LossArgs& s, hipStream_t stream);
hipError_t launch_loss_gradient(const LossArgs& s, int tile, int cu_count, hipStream_t stream);
// dw of a piece (s.gemm) and its share of dx (s.gemm_dx; after the last piece
// dx itself).
hipError_t launch_loss_products(const LossArgs& s, const LossChoice& c, bool last_piece, int cu_count,
                                hipStream_t stream);

}  // namespace migemm

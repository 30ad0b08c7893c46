// operators.h -- internal interface between the operators' plan layer
// (operators_api.cpp, block_api.cpp) and their kernels: argument blocks and launches.
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

// --------------------------------------------------------------- quantize

struct QuantizeArgs {
  const void* x;  // bf16
  void* q;        // e4m3 or int8
  float* scale;
  int64_t rows, cols;
  int64_t x_rs, q_rs;  // elements
};
NormShape quantize_shape(int64_t rows, int64_t cols);
hipError_t launch_quantize(const QuantizeArgs& a, bool e4m3, hipStream_t stream);

// ------------------------------------------------------------- block norm

struct BlockNormArgs {
  const void* x;            // bf16, like every matrix but y
  const void* z;            // the gate (NULL: none)
  const void* r;            // forward
  const void* dy;           // backward
  const void* dh;           // backward (NULL: none)
  const void* post_weight;  // bf16 [cols] (NULL: no norm behind the block)
  const void* weight;
  void* h;                  // forward: out; backward: in
  void* y;                  // forward: bf16, e4m3 or int8
  void* dx;                 // backward
  void* dz;
  void* dr;
  float* scale;             // forward, e4m3 and int8
  float* post_rstd;         // forward: out; backward: in
  float* rstd;
  float* dpost_weight;      // backward
  float* dweight;
  float* partials;          // backward: workspace, one row of sums per row walker
  int64_t rows, cols;
  int64_t x_rs, z_rs, r_rs, h_rs, y_rs, dy_rs, dh_rs, dx_rs, dz_rs, dr_rs;  // elements
  int64_t partial_rows;
  float eps, branch, residual;
};

// Widest row the kernels hold in registers.
constexpr int64_t kBlockNormMaxCols = 8 * 64 * 4 * 8;
NormShape block_norm_forward_shape(int64_t rows, int64_t cols);
NormShape block_norm_backward_shape(int64_t rows, int64_t cols);
// Rows of partial column sums the backward pass leaves in its workspace.
int64_t block_norm_partial_rows(int64_t rows, int64_t cols, int cu_count);
hipError_t prepare_block_norm();

// y_type: 0 bf16, 1 e4m3, 2 int8.
hipError_t launch_block_norm_forward(const BlockNormArgs& a, int y_type, hipStream_t stream);
hipError_t launch_block_norm_backward(const BlockNormArgs& a, hipStream_t stream);

// ----------------------------------------------------------------- scaled

// Four fp32 sums.
typedef float mid_piece __attribute__((ext_vector_type(4)));

struct ScaledArgs {
  KernelArgs gemm;       // A, B: e4m3, K-contiguous; strides in elements
  const float* a_scale;  // [M]
  const float* b_scale;  // [N], 16-byte aligned
  const float* bias;     // int8: [N], 16-byte aligned (NULL: none)
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

// The same of int8 (A, B: int8).
ScaledChoice choose_int8(int64_t M, int64_t N, int64_t K, int cu_count);
ScaledKernel int8_kernel(int variant);
hipError_t prepare_int8();
hipError_t launch_int8(const ScaledArgs& a, int variant, int cu_count, hipStream_t stream);

// ------------------------------------------------------------- checkpoint

// The kept activations of T tokens x `cols`: e4m3 codes [tokens / 16][ld][16
// tokens] for T rounded up to 32 tokens and ld = cols rounded up to 16, then
// a byte for each 32 tokens and column, [tokens / 32][ld]: the exponent of a
// power of two, plus 127.
struct CheckpointArgs {
  const void* x;          // pack: in (bf16)
  void* x_out;            // unpack: out
  unsigned char* codes;
  unsigned char* scales;
  int64_t tokens, cols, ld;
  int64_t x_rs;           // elements
  // The weights' gradient dw (out_cols x cols) = dy^T (kept activations).
  const void* dy;         // tokens x out_cols, bf16
  void* dw;               // bf16 or fp32
  int64_t out_cols, dy_rs, dw_rs;
  bool fp32, accumulate;  // accumulate: dw += (fp32)
  int32_t splits;
  mid_piece* partials;    // workspace: the splits' sums
};
hipError_t launch_checkpoint_pack(const CheckpointArgs& a, hipStream_t stream);
hipError_t launch_checkpoint_unpack(const CheckpointArgs& a, hipStream_t stream);
// The gradient's kernel, the ranges its tokens are split into, and the
// workspace.  es: bytes of an element of dw.
struct CheckpointChoice {
  int variant, splits;
  int64_t workspace_bytes;
};
CheckpointChoice choose_checkpoint(int64_t tokens, int64_t cols, int64_t out_cols, int es, int cu_count);
struct CheckpointKernel {
  int tile_m, tile_n, lds_stages;
};
CheckpointKernel checkpoint_kernel(int variant);
hipError_t prepare_checkpoint();
hipError_t launch_checkpoint_gradient(const CheckpointArgs& a, int variant, hipStream_t stream);

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

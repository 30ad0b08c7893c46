// block_api.cpp -- the C ABI of the operators between and inside a block's
// 8-bit products (include/migemm.h): the int8 product, rows to 8 bits, the
// block norm and the 8-bit checkpoints; description checks, plans and runs.
#include <hip/hip_runtime.h>

#include <atomic>
#include <cmath>
#include <new>

#include "plan_layer.hpp"

struct migemm_int8_plan {
  migemm_int8_desc desc;
  migemm::ScaledArgs base;  // the shape's part of the kernel arguments
  int variant, cus;
  size_t workspace_bytes;
};

struct migemm_quantize_plan {
  migemm_quantize_desc desc;
  int cus;
};

struct migemm_block_norm_plan {
  migemm_block_norm_desc desc;
  int cus;
  int64_t partial_rows;
  size_t workspace_bytes;
};

struct migemm_checkpoint_plan {
  migemm_checkpoint_desc desc;
  int cus;
  int64_t ld, code_bytes, scale_bytes;
  int variant, splits;
  size_t workspace_bytes;
};

namespace {

using namespace migemm;

// Nothing to prepare.
hipError_t nothing() { return hipSuccess; }

// --------------------------------------------------------------------- int8

// The largest K whose sums stay within int32 for every code, -128 among them.
constexpr int64_t kInt8MaxK = 131071;

int validate_int8(const migemm_int8_desc* d) {
  if (!d || d->M < 0 || d->N < 0 || d->K < 0 || d->reserved != 0) return MIGEMM_ERR_INVALID_ARG;
  int st = check_matrix(d->M, d->K, d->a_rs, 1);
  if (st == MIGEMM_OK) st = check_matrix(d->N, d->K, d->b_cs, 1);
  if (st == MIGEMM_OK) st = check_matrix(d->M, d->N, d->d_rs, 2);
  if (st != MIGEMM_OK) return st;
  if (!band_fits(d->a_rs, 1) || !band_fits(d->b_cs, 1) || !band_fits(d->d_rs, 2) ||
      !tiles_fit(d->M, d->N) || d->K > kInt8MaxK)
    return MIGEMM_ERR_UNSUPPORTED;
  return MIGEMM_OK;
}

// ----------------------------------------------------------------- quantize

int validate_quantize(const migemm_quantize_desc* d) {
  if (!d || d->rows < 0 || d->cols < 1 || d->reserved != 0) return MIGEMM_ERR_INVALID_ARG;
  if (d->q_type != MIGEMM_INT8 && d->q_type != MIGEMM_FP8_E4M3) return MIGEMM_ERR_INVALID_ARG;
  int st = check_matrix(d->rows, d->cols, d->x_rs, 2);
  if (st == MIGEMM_OK) st = check_matrix(d->rows, d->cols, d->q_rs, 1);
  if (st != MIGEMM_OK) return st;
  return d->cols > kNormMaxCols ? MIGEMM_ERR_UNSUPPORTED : MIGEMM_OK;
}

// --------------------------------------------------------------- block norm

bool with_gate(const migemm_block_norm_desc& d) { return d.z_rs != 0; }
bool with_backward(const migemm_block_norm_desc& d) { return d.dx_rs != 0; }

int validate_block_norm(const migemm_block_norm_desc* d) {
  if (!d || d->rows < 0 || d->cols < 1 || (d->post_norm != 0 && d->post_norm != 1)) return MIGEMM_ERR_INVALID_ARG;
  if (!(d->eps > 0.0f) || !std::isfinite(d->eps)) return MIGEMM_ERR_INVALID_ARG;
  if (!std::isfinite(d->branch_scale) || !std::isfinite(d->residual_scale)) return MIGEMM_ERR_INVALID_ARG;
  if (d->y_type != MIGEMM_BF16 && d->y_type != MIGEMM_FP8_E4M3 && d->y_type != MIGEMM_INT8)
    return MIGEMM_ERR_INVALID_ARG;
  // The backward pass's operands come together: the gate's gradient with a
  // gate, the residual's incoming gradient or none.
  const bool back = d->dx_rs != 0;
  if ((d->dy_rs != 0) != back || (d->dr_rs != 0) != back || (d->dz_rs != 0) != (back && d->z_rs != 0) ||
      (d->dh_rs != 0 && !back))
    return MIGEMM_ERR_INVALID_ARG;
  const struct { int64_t rs; int es; bool used; } m[] = {
      {d->x_rs, 2, true}, {d->r_rs, 2, true}, {d->h_rs, 2, true},
      {d->y_rs, d->y_type == MIGEMM_BF16 ? 2 : 1, true},
      {d->z_rs, 2, d->z_rs != 0}, {d->dy_rs, 2, back}, {d->dx_rs, 2, back}, {d->dr_rs, 2, back},
      {d->dz_rs, 2, d->dz_rs != 0}, {d->dh_rs, 2, d->dh_rs != 0}};
  for (const auto& e : m) {
    if (!e.used) continue;
    const int st = check_matrix(d->rows, d->cols, e.rs, e.es);
    if (st != MIGEMM_OK) return st;
  }
  return d->cols > kBlockNormMaxCols ? MIGEMM_ERR_UNSUPPORTED : MIGEMM_OK;
}

// --------------------------------------------------------------- checkpoint

bool with_gradient(const migemm_checkpoint_desc& d) { return d.dw_rs != 0; }

int validate_checkpoint(const migemm_checkpoint_desc* d) {
  if (!d || d->tokens < 0 || d->cols < 1 || d->out_cols < 0 || d->reserved != 0) return MIGEMM_ERR_INVALID_ARG;
  if (d->accumulate != 0 && d->accumulate != 1) return MIGEMM_ERR_INVALID_ARG;
  const bool grad = d->dw_rs != 0;
  if ((d->dy_rs != 0) != grad || (d->out_cols != 0) != grad) return MIGEMM_ERR_INVALID_ARG;
  // Sums are added to in fp32 only: a bf16 gradient would lose what it adds.
  if (d->dw_type != MIGEMM_BF16 && d->dw_type != MIGEMM_FP32) return MIGEMM_ERR_INVALID_ARG;
  if (d->accumulate && (!grad || d->dw_type != MIGEMM_FP32)) return MIGEMM_ERR_INVALID_ARG;
  int st = check_matrix(d->tokens, d->cols, d->x_rs, 2);
  if (st == MIGEMM_OK && grad) st = check_matrix(d->tokens, d->out_cols, d->dy_rs, 2);
  if (st == MIGEMM_OK && grad) st = check_matrix(d->out_cols, d->cols, d->dw_rs, d->dw_type == MIGEMM_FP32 ? 4 : 2);
  if (st != MIGEMM_OK) return st;
  // 64 tokens of dy and of the codes, and 256 rows of dw, are reached with
  // 32-bit offsets; tokens are counted in 32 bits, and a launch of a workgroup
  // of 512 for each 256 x 256 tile holds fewer than 2^32 threads.
  if (!band_fits(d->cols, 1) || d->tokens >= ((int64_t)1 << 31) - 64) return MIGEMM_ERR_UNSUPPORTED;
  if (grad && (!band_fits(d->dy_rs, 2) || !band_fits(d->dw_rs, d->dw_type == MIGEMM_FP32 ? 4 : 2) ||
               d->out_cols >= ((int64_t)1 << 38) / d->cols))
    return MIGEMM_ERR_UNSUPPORTED;
  return MIGEMM_OK;
}

CheckpointArgs checkpoint_args(const migemm_checkpoint_plan* p, const void* kept) {
  const migemm_checkpoint_desc& d = p->desc;
  CheckpointArgs a = {};
  a.codes = static_cast<unsigned char*>(const_cast<void*>(kept));
  a.scales = a.codes + p->code_bytes;
  a.tokens = d.tokens, a.cols = d.cols, a.ld = p->ld, a.x_rs = d.x_rs;
  return a;
}

}  // namespace

extern "C" {

int gemm_int8_desc_validate(const migemm_int8_desc* desc) { return validate_int8(desc); }

int gemm_int8_plan_create(const migemm_int8_desc* desc, migemm_int8_plan** out) {
  if (!out) return MIGEMM_ERR_INVALID_ARG;
  *out = nullptr;
  int st = validate_int8(desc);
  if (st != MIGEMM_OK) return st;
  int cus = 0;
  static std::atomic<bool> prepared[kMaxDevices];
  st = check_device(desc->device, &cus, prepared, prepare_int8);
  if (st != MIGEMM_OK) return st;
  migemm_int8_plan* p = new (std::nothrow) migemm_int8_plan();
  if (!p) return MIGEMM_ERR_INVALID_ARG;
  p->desc = *desc;
  KernelArgs& a = p->base.gemm;
  a.M = desc->M, a.N = desc->N, a.K = desc->K;
  a.lda = desc->a_rs, a.ldb = desc->b_cs, a.ldd = desc->d_rs;
  a.a_bytes = a.M > 0 ? (a.M - 1) * a.lda + a.K : 0;
  a.b_bytes = a.N > 0 ? (a.N - 1) * a.ldb + a.K : 0;
  const ScaledChoice c = choose_int8(a.M, a.N, a.K, cus);
  set_tiles(a, c.tile_m);
  p->variant = c.variant;
  p->base.splits = c.splits;
  p->workspace_bytes = (size_t)c.workspace_bytes;
  p->cus = cus;
  return add_live(p, kInt8, out);
}

int gemm_int8_plan_destroy(migemm_int8_plan* plan) { return destroy(plan, kInt8); }

size_t gemm_int8_workspace_size(const migemm_int8_plan* plan) {
  return is_live(plan, kInt8) ? plan->workspace_bytes : 0;
}

int gemm_int8_plan_get_info(const migemm_int8_plan* p, migemm_int8_info* out) {
  if (!is_live(p, kInt8) || !out) return MIGEMM_ERR_INVALID_ARG;
  const ScaledKernel k = int8_kernel(p->variant);
  *out = {k.tile_m, k.tile_n, k.lds_stages, p->base.splits, p->cus};
  return MIGEMM_OK;
}

int gemm_int8_run(const migemm_int8_plan* p, const void* a, const float* a_scale, const void* b,
                  const float* b_scale, const float* bias, void* d, void* workspace, void* stream) {
  if (!is_live(p, kInt8)) return MIGEMM_ERR_INVALID_ARG;
  const migemm_int8_desc& e = p->desc;
  if (e.M == 0 || e.N == 0) return MIGEMM_OK;
  if (!a_scale || !b_scale || !d || (e.K > 0 && (!a || !b))) return MIGEMM_ERR_INVALID_ARG;
  if (!aligned(a, 16) || !aligned(b, 16) || !aligned(d, 16) || !aligned(a_scale, 16) ||
      !aligned(b_scale, 16) || !aligned(bias, 16))
    return MIGEMM_ERR_MISALIGNED;
  const int st = check_workspace(p->workspace_bytes, workspace);
  if (st != MIGEMM_OK) return st;
  if (!current_device_is(e.device)) return MIGEMM_ERR_DEVICE;
  ScaledArgs s = p->base;
  s.gemm.A = a, s.gemm.B = b, s.gemm.D = d;
  s.a_scale = a_scale, s.b_scale = b_scale, s.bias = bias;
  s.partials = static_cast<mid_piece*>(workspace);
  return launched(launch_int8(s, p->variant, p->cus, static_cast<hipStream_t>(stream)));
}

int gemm_quantize_desc_validate(const migemm_quantize_desc* desc) { return validate_quantize(desc); }

int gemm_quantize_plan_create(const migemm_quantize_desc* desc, migemm_quantize_plan** out) {
  if (!out) return MIGEMM_ERR_INVALID_ARG;
  *out = nullptr;
  int st = validate_quantize(desc);
  if (st != MIGEMM_OK) return st;
  int cus = 0;
  static std::atomic<bool> prepared[kMaxDevices];
  st = check_device(desc->device, &cus, prepared, nothing);
  if (st != MIGEMM_OK) return st;
  migemm_quantize_plan* p = new (std::nothrow) migemm_quantize_plan();
  if (!p) return MIGEMM_ERR_INVALID_ARG;
  p->desc = *desc;
  p->cus = cus;
  return add_live(p, kQuantize, out);
}

int gemm_quantize_plan_destroy(migemm_quantize_plan* plan) { return destroy(plan, kQuantize); }

size_t gemm_quantize_workspace_size(const migemm_quantize_plan*) { return 0; }

int gemm_quantize_plan_get_info(const migemm_quantize_plan* p, migemm_quantize_info* out) {
  if (!is_live(p, kQuantize) || !out) return MIGEMM_ERR_INVALID_ARG;
  const NormShape s = quantize_shape(p->desc.rows, p->desc.cols);
  *out = {s.waves, s.vectors, p->cus};
  return MIGEMM_OK;
}

int gemm_quantize_run(const migemm_quantize_plan* p, const void* x, void* q, float* scale, void* stream) {
  if (!is_live(p, kQuantize)) return MIGEMM_ERR_INVALID_ARG;
  const migemm_quantize_desc& d = p->desc;
  if (d.rows == 0) return MIGEMM_OK;
  if (!x || !q || !scale) return MIGEMM_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(q, 16) || !aligned(scale, 4)) return MIGEMM_ERR_MISALIGNED;
  if (!current_device_is(d.device)) return MIGEMM_ERR_DEVICE;
  QuantizeArgs a = {};
  a.x = x, a.q = q, a.scale = scale;
  a.rows = d.rows, a.cols = d.cols, a.x_rs = d.x_rs, a.q_rs = d.q_rs;
  return launched(launch_quantize(a, d.q_type == MIGEMM_FP8_E4M3, static_cast<hipStream_t>(stream)));
}

int gemm_block_norm_desc_validate(const migemm_block_norm_desc* desc) { return validate_block_norm(desc); }

int gemm_block_norm_plan_create(const migemm_block_norm_desc* desc, migemm_block_norm_plan** out) {
  if (!out) return MIGEMM_ERR_INVALID_ARG;
  *out = nullptr;
  int st = validate_block_norm(desc);
  if (st != MIGEMM_OK) return st;
  int cus = 0;
  static std::atomic<bool> prepared[kMaxDevices];
  st = check_device(desc->device, &cus, prepared, prepare_block_norm);
  if (st != MIGEMM_OK) return st;
  migemm_block_norm_plan* p = new (std::nothrow) migemm_block_norm_plan();
  if (!p) return MIGEMM_ERR_INVALID_ARG;
  p->desc = *desc;
  p->cus = cus;
  if (with_backward(*desc)) {
    p->partial_rows = block_norm_partial_rows(desc->rows, desc->cols, cus);
    p->workspace_bytes = (size_t)(p->partial_rows * desc->cols * (desc->post_norm ? 2 : 1) * 4);
  }
  return add_live(p, kBlockNorm, out);
}

int gemm_block_norm_plan_destroy(migemm_block_norm_plan* plan) { return destroy(plan, kBlockNorm); }

size_t gemm_block_norm_workspace_size(const migemm_block_norm_plan* plan) {
  return is_live(plan, kBlockNorm) ? plan->workspace_bytes : 0;
}

int gemm_block_norm_plan_get_info(const migemm_block_norm_plan* p, migemm_block_norm_info* out) {
  if (!is_live(p, kBlockNorm) || !out) return MIGEMM_ERR_INVALID_ARG;
  const NormShape f = block_norm_forward_shape(p->desc.rows, p->desc.cols);
  const NormShape b = block_norm_backward_shape(p->desc.rows, p->desc.cols);
  const bool back = with_backward(p->desc);
  *out = {f.waves, f.vectors, back ? b.waves : 0, back ? b.vectors : 0, (int32_t)p->partial_rows, p->cus};
  return MIGEMM_OK;
}

int gemm_block_norm_run(const migemm_block_norm_plan* p, const void* x, const void* z, const void* r,
                        const void* post_weight, const void* weight, void* h, void* y, float* scale,
                        float* post_rstd, float* rstd, void* stream) {
  if (!is_live(p, kBlockNorm)) return MIGEMM_ERR_INVALID_ARG;
  const migemm_block_norm_desc& d = p->desc;
  if (d.rows == 0) return MIGEMM_OK;
  const bool post = d.post_norm != 0, codes = d.y_type != MIGEMM_BF16;
  if ((z != nullptr) != with_gate(d) || (post_weight != nullptr) != post || (post_rstd != nullptr) != post ||
      (scale != nullptr) != codes)
    return MIGEMM_ERR_INVALID_ARG;
  if (!x || !r || !weight || !h || !y || !rstd) return MIGEMM_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(z, 16) || !aligned(r, 16) || !aligned(post_weight, 16) || !aligned(weight, 16) ||
      !aligned(h, 16) || !aligned(y, 16) || !aligned(scale, 4) || !aligned(post_rstd, 4) || !aligned(rstd, 4))
    return MIGEMM_ERR_MISALIGNED;
  if (!current_device_is(d.device)) return MIGEMM_ERR_DEVICE;
  BlockNormArgs a = {};
  a.x = x, a.z = z, a.r = r, a.post_weight = post_weight, a.weight = weight, a.h = h, a.y = y;
  a.scale = scale, a.post_rstd = post_rstd, a.rstd = rstd;
  a.rows = d.rows, a.cols = d.cols, a.eps = d.eps, a.branch = d.branch_scale, a.residual = d.residual_scale;
  a.x_rs = d.x_rs, a.z_rs = d.z_rs, a.r_rs = d.r_rs, a.h_rs = d.h_rs, a.y_rs = d.y_rs;
  const int y_type = d.y_type == MIGEMM_BF16 ? 0 : (d.y_type == MIGEMM_FP8_E4M3 ? 1 : 2);
  return launched(launch_block_norm_forward(a, y_type, static_cast<hipStream_t>(stream)));
}

int gemm_block_norm_run_backward(const migemm_block_norm_plan* p, const void* dy, const void* dh, const void* x,
                                 const void* z, const void* h, const void* post_weight, const void* weight,
                                 const float* post_rstd, const float* rstd, void* dx, void* dz, void* dr,
                                 float* dpost_weight, float* dweight, void* workspace, void* stream) {
  if (!is_live(p, kBlockNorm) || !with_backward(p->desc)) return MIGEMM_ERR_INVALID_ARG;
  const migemm_block_norm_desc& d = p->desc;
  const bool post = d.post_norm != 0, gate = with_gate(d);
  if (!dweight || (dpost_weight != nullptr) != post) return MIGEMM_ERR_INVALID_ARG;
  if (d.rows > 0) {
    if (!dy || !h || !weight || !rstd || !dx || !dr || (dh != nullptr) != (d.dh_rs != 0)) return MIGEMM_ERR_INVALID_ARG;
    if ((z != nullptr) != gate || (dz != nullptr) != gate || (post_weight != nullptr) != post ||
        (post_rstd != nullptr) != post || ((gate || post) && !x))
      return MIGEMM_ERR_INVALID_ARG;
  }
  if (!aligned(dy, 16) || !aligned(dh, 16) || !aligned(x, 16) || !aligned(z, 16) || !aligned(h, 16) ||
      !aligned(post_weight, 16) || !aligned(weight, 16) || !aligned(post_rstd, 4) || !aligned(rstd, 4) ||
      !aligned(dx, 16) || !aligned(dz, 16) || !aligned(dr, 16) || !aligned(dpost_weight, 4) || !aligned(dweight, 4))
    return MIGEMM_ERR_MISALIGNED;
  const int st = check_workspace(p->workspace_bytes, workspace);
  if (st != MIGEMM_OK) return st;
  if (!current_device_is(d.device)) return MIGEMM_ERR_DEVICE;
  BlockNormArgs a = {};
  a.dy = dy, a.dh = dh, a.x = x, a.z = z, a.h = const_cast<void*>(h), a.post_weight = post_weight, a.weight = weight;
  a.post_rstd = const_cast<float*>(post_rstd), a.rstd = const_cast<float*>(rstd);
  a.dx = dx, a.dz = dz, a.dr = dr, a.dpost_weight = dpost_weight, a.dweight = dweight;
  a.partials = static_cast<float*>(workspace);
  a.rows = d.rows, a.cols = d.cols, a.partial_rows = p->partial_rows;
  a.branch = d.branch_scale, a.residual = d.residual_scale;
  a.x_rs = d.x_rs, a.z_rs = d.z_rs, a.h_rs = d.h_rs, a.dy_rs = d.dy_rs, a.dh_rs = d.dh_rs, a.dx_rs = d.dx_rs;
  a.dz_rs = d.dz_rs, a.dr_rs = d.dr_rs;
  return launched(launch_block_norm_backward(a, static_cast<hipStream_t>(stream)));
}

int gemm_checkpoint_desc_validate(const migemm_checkpoint_desc* desc) { return validate_checkpoint(desc); }

int gemm_checkpoint_plan_create(const migemm_checkpoint_desc* desc, migemm_checkpoint_plan** out) {
  if (!out) return MIGEMM_ERR_INVALID_ARG;
  *out = nullptr;
  int st = validate_checkpoint(desc);
  if (st != MIGEMM_OK) return st;
  int cus = 0;
  static std::atomic<bool> prepared[kMaxDevices];
  st = check_device(desc->device, &cus, prepared, prepare_checkpoint);
  if (st != MIGEMM_OK) return st;
  migemm_checkpoint_plan* p = new (std::nothrow) migemm_checkpoint_plan();
  if (!p) return MIGEMM_ERR_INVALID_ARG;
  p->desc = *desc;
  p->cus = cus;
  p->ld = up(desc->cols, 16);
  p->code_bytes = up(desc->tokens, 32) * p->ld;
  p->scale_bytes = p->code_bytes / 32;
  if (with_gradient(*desc)) {
    const CheckpointChoice c =
        choose_checkpoint(desc->tokens, desc->cols, desc->out_cols, desc->dw_type == MIGEMM_FP32 ? 4 : 2, cus);
    p->variant = c.variant, p->splits = c.splits;
    p->workspace_bytes = (size_t)c.workspace_bytes;
  }
  return add_live(p, kCheckpoint, out);
}

int gemm_checkpoint_plan_destroy(migemm_checkpoint_plan* plan) { return destroy(plan, kCheckpoint); }

size_t gemm_checkpoint_workspace_size(const migemm_checkpoint_plan* plan) {
  return is_live(plan, kCheckpoint) ? plan->workspace_bytes : 0;
}

size_t gemm_checkpoint_size(const migemm_checkpoint_plan* plan) {
  return is_live(plan, kCheckpoint) ? (size_t)(plan->code_bytes + plan->scale_bytes) : 0;
}

int gemm_checkpoint_plan_get_info(const migemm_checkpoint_plan* p, migemm_checkpoint_info* out) {
  if (!is_live(p, kCheckpoint) || !out) return MIGEMM_ERR_INVALID_ARG;
  *out = {};
  out->code_bytes = p->code_bytes, out->scale_bytes = p->scale_bytes;
  out->cu_count = p->cus;
  if (!with_gradient(p->desc)) return MIGEMM_OK;
  const CheckpointKernel k = checkpoint_kernel(p->variant);
  out->tile_m = k.tile_m, out->tile_n = k.tile_n, out->lds_stages = k.lds_stages;
  out->splits = p->splits;
  return MIGEMM_OK;
}

int gemm_checkpoint_pack(const migemm_checkpoint_plan* p, const void* x, void* kept, void* stream) {
  if (!is_live(p, kCheckpoint)) return MIGEMM_ERR_INVALID_ARG;
  if (p->desc.tokens == 0) return MIGEMM_OK;
  if (!x || !kept) return MIGEMM_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(kept, 16)) return MIGEMM_ERR_MISALIGNED;
  if (!current_device_is(p->desc.device)) return MIGEMM_ERR_DEVICE;
  CheckpointArgs a = checkpoint_args(p, kept);
  a.x = x;
  return launched(launch_checkpoint_pack(a, static_cast<hipStream_t>(stream)));
}

int gemm_checkpoint_unpack(const migemm_checkpoint_plan* p, const void* kept, void* x, void* stream) {
  if (!is_live(p, kCheckpoint)) return MIGEMM_ERR_INVALID_ARG;
  if (p->desc.tokens == 0) return MIGEMM_OK;
  if (!x || !kept) return MIGEMM_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(kept, 16)) return MIGEMM_ERR_MISALIGNED;
  if (!current_device_is(p->desc.device)) return MIGEMM_ERR_DEVICE;
  CheckpointArgs a = checkpoint_args(p, kept);
  a.x_out = x;
  return launched(launch_checkpoint_unpack(a, static_cast<hipStream_t>(stream)));
}

int gemm_checkpoint_weight_gradient(const migemm_checkpoint_plan* p, const void* dy, const void* kept, void* dw,
                                    void* workspace, void* stream) {
  if (!is_live(p, kCheckpoint) || !with_gradient(p->desc)) return MIGEMM_ERR_INVALID_ARG;
  const migemm_checkpoint_desc& d = p->desc;
  if (!dw || (d.tokens > 0 && (!dy || !kept))) return MIGEMM_ERR_INVALID_ARG;
  if (!aligned(dy, 16) || !aligned(kept, 16) || !aligned(dw, 16)) return MIGEMM_ERR_MISALIGNED;
  const int st = check_workspace(p->workspace_bytes, workspace);
  if (st != MIGEMM_OK) return st;
  if (!current_device_is(d.device)) return MIGEMM_ERR_DEVICE;
  CheckpointArgs a = checkpoint_args(p, kept);
  a.dy = dy, a.dw = dw, a.out_cols = d.out_cols, a.dy_rs = d.dy_rs, a.dw_rs = d.dw_rs;
  a.fp32 = d.dw_type == MIGEMM_FP32, a.accumulate = d.accumulate != 0;
  a.splits = p->splits, a.partials = static_cast<mid_piece*>(workspace);
  return launched(launch_checkpoint_gradient(a, p->variant, static_cast<hipStream_t>(stream)));
}

}  // extern "C"

// operators_api.cpp -- the C ABI of the operators around the product
// (include/migemm.h): description checks, plans and run entry points.
#include <hip/hip_runtime.h>

#include <atomic>
#include <cmath>
#include <new>

#include "plan_layer.hpp"

struct migemm_scaled_plan {
  migemm_scaled_desc desc;
  migemm::ScaledArgs base;  // the shape's part of the kernel arguments
  int variant, cus;
  size_t workspace_bytes;
};

struct migemm_vocab_loss_plan {
  migemm_vocab_loss_desc desc;
  int cus;
  // Forward: rows a launch takes (the workspace holds one launch's pairs).
  int64_t chunk;
  // Backward: vocabulary entries a piece, g's row stride, and where things
  // lie in the workspace.
  int64_t piece, g_rs, rows_rs, dx_tiles;
  migemm::LossChoice choice;
  bool dx_summed;
  size_t at_from, at_lse, at_dloss, at_target, at_rows, at_g, at_dx, at_dw;
  size_t workspace_bytes;
};

struct migemm_norm_plan {
  migemm_norm_desc desc;
  int cus;
  int64_t partial_rows;
  size_t workspace_bytes;
};

namespace {

using namespace migemm;

// --------------------------------------------------------------------- norm

bool norm_residual(const migemm_norm_desc& d) { return d.r_rs != 0; }
bool norm_backward(const migemm_norm_desc& d) { return d.dx_rs != 0; }

int validate_norm(const migemm_norm_desc* d) {
  if (!d || d->rows < 0 || d->cols < 1 || d->reserved != 0) return MIGEMM_ERR_INVALID_ARG;
  if (!(d->eps > 0.0f) || !std::isfinite(d->eps)) return MIGEMM_ERR_INVALID_ARG;
  if (d->y_type != MIGEMM_BF16 && d->y_type != MIGEMM_FP8_E4M3) return MIGEMM_ERR_INVALID_ARG;
  // The residual comes in and goes out, or neither; likewise the backward
  // pass's operands; the residual's gradient needs a backward pass.
  if ((d->r_rs != 0) != (d->h_rs != 0) || (d->dy_rs != 0) != (d->dx_rs != 0) ||
      (d->dh_rs != 0 && d->dx_rs == 0))
    return MIGEMM_ERR_INVALID_ARG;
  const struct { int64_t rs; int es; bool used; } m[] = {
      {d->x_rs, 2, true},
      {d->y_rs, d->y_type == MIGEMM_BF16 ? 2 : 1, true},
      {d->r_rs, 2, d->r_rs != 0}, {d->h_rs, 2, d->h_rs != 0}, {d->dy_rs, 2, d->dy_rs != 0},
      {d->dh_rs, 2, d->dh_rs != 0}, {d->dx_rs, 2, d->dx_rs != 0}};
  for (const auto& e : m) {
    if (!e.used) continue;
    const int st = check_matrix(d->rows, d->cols, e.rs, e.es);
    if (st != MIGEMM_OK) return st;
  }
  return d->cols > migemm::kNormMaxCols ? MIGEMM_ERR_UNSUPPORTED : MIGEMM_OK;
}

// ------------------------------------------------------------------- scaled

int validate_scaled(const migemm_scaled_desc* d) {
  if (!d || d->M < 0 || d->N < 0 || d->K < 0 || d->reserved != 0) return MIGEMM_ERR_INVALID_ARG;
  int st = check_matrix(d->M, d->K, d->a_rs, 1);
  if (st == MIGEMM_OK) st = check_matrix(d->N, d->K, d->b_cs, 1);
  if (st == MIGEMM_OK) st = check_matrix(d->M, d->N, d->d_rs, 2);
  if (st != MIGEMM_OK) return st;
  if (!band_fits(d->a_rs, 1) || !band_fits(d->b_cs, 1) || !band_fits(d->d_rs, 2) ||
      !tiles_fit(d->M, d->N))
    return MIGEMM_ERR_UNSUPPORTED;
  return MIGEMM_OK;
}

// --------------------------------------------------------------------- loss

int validate_loss(const migemm_vocab_loss_desc* d) {
  if (!d || d->rows < 0 || d->vocab < 1 || d->hidden < 1 || d->reserved != 0)
    return MIGEMM_ERR_INVALID_ARG;
  if ((d->dx_rs != 0) != (d->dw_rs != 0)) return MIGEMM_ERR_INVALID_ARG;
  const bool back = d->dx_rs != 0;
  int st = check_matrix(d->rows, d->hidden, d->x_rs, 2);
  if (st == MIGEMM_OK) st = check_matrix(d->vocab, d->hidden, d->w_rs, 2);
  if (st == MIGEMM_OK && back) st = check_matrix(d->rows, d->hidden, d->dx_rs, 2);
  if (st == MIGEMM_OK && back) st = check_matrix(d->vocab, d->hidden, d->dw_rs, 2);
  if (st != MIGEMM_OK) return st;
  if (!band_fits(d->x_rs, 2) || !band_fits(d->w_rs, 2) ||
      (back && (!band_fits(d->dx_rs, 2) || !band_fits(d->dw_rs, 2))))
    return MIGEMM_ERR_UNSUPPORTED;
  // Row numbers and vocabulary entries are 32-bit in the kernels.
  if (d->rows >= ((int64_t)1 << 28) || d->vocab >= ((int64_t)1 << 28)) return MIGEMM_ERR_UNSUPPORTED;
  if (!tiles_fit(d->rows, 16 * 256) || !tiles_fit(d->vocab, 16384)) return MIGEMM_ERR_UNSUPPORTED;
  return MIGEMM_OK;
}

// Rows of the forward pass a launch takes: their pairs of the whole
// vocabulary are the workspace (at 131072 entries 128 MiB).
constexpr int64_t kLossChunk = 16384;
// The most a piece of g takes, the padding of its rows aside -- unless that is
// less than kPieceLeast entries: adding a piece's dx to the fp32 sums moves 8
// bytes a row and hidden unit, which takes the time of a product of about that
// many entries, and smaller pieces would spend more on it than on the product.
constexpr int64_t kPieceBytes = (int64_t)512 << 20;
constexpr int64_t kPieceLeast = 1024;

void lay_out_loss(migemm_vocab_loss_plan* p) {
  const migemm_vocab_loss_desc& d = p->desc;
  const int64_t T = d.rows, V = d.vocab, H = d.hidden;
  p->chunk = T < kLossChunk ? T : kLossChunk;
  // Pieces of equal width.
  int64_t most = kPieceBytes / 2 / up(T > 0 ? T : 1, 256) / 256 * 256;
  most = most < kPieceLeast ? kPieceLeast : (most > (1 << 20) ? 1 << 20 : most);
  const int64_t pieces = (V + most - 1) / most;
  p->piece = up((V + pieces - 1) / pieces, 256);
  p->choice = migemm::choose_loss(T, V, H, p->piece, p->cus);
  const migemm::LossChoice& c = p->choice;
  const int64_t part_cols = migemm::kLossTileN[c.forward] / 2;
  p->workspace_bytes = (size_t)((V + part_cols - 1) / part_cols * p->chunk * 8 + p->chunk * 4);
  if (d.dx_rs == 0) return;
  const int64_t width = p->piece < V ? p->piece : V;
  p->g_rs = up(width, 64) + 64;  // rows not a power of two apart
  p->rows_rs = up(H, 64);
  auto tile_bytes = [](int tile) { return (int64_t)4 * migemm::kLossTileM[tile] * migemm::kLossTileN[tile]; };
  p->dx_tiles = migemm::loss_tiles(c.dx, T, H);
  p->dx_summed = c.dx == migemm::kLoss256 || c.dx_splits > 1 || p->piece < V;
  size_t at = 256;  // the head
  auto take = [&](int64_t bytes) {
    const size_t from = at;
    at += (size_t)up(bytes, 256);
    return from;
  };
  p->at_from = take(T * 4);
  p->at_lse = take(T * 4);
  p->at_dloss = take(T * 4);
  p->at_target = take(T * 4);
  p->at_rows = take(T * p->rows_rs * 2);
  p->at_g = take(T * p->g_rs * 2);
  p->at_dx = take(p->dx_summed ? c.dx_splits * p->dx_tiles * tile_bytes(c.dx) : 0);
  p->at_dw = take(c.dw_splits > 1 ? c.dw_splits * migemm::loss_tiles(c.dw, width, H) * tile_bytes(c.dw) : 0);
  if (at > p->workspace_bytes) p->workspace_bytes = at;
}

// M x N x K of bf16 operands with the given strides, in 256 x 256 tiles.
migemm::KernelArgs product(int64_t M, int64_t N, int64_t K, const void* A, int64_t lda, bool a_kmajor,
                           const void* B, int64_t ldb, bool b_kmajor, void* D, int64_t ldd) {
  migemm::KernelArgs a = {};
  a.M = M, a.N = N, a.K = K, a.A = A, a.B = B, a.D = D, a.lda = lda, a.ldb = ldb, a.ldd = ldd;
  a.a_bytes = a_kmajor ? (M > 0 ? ((M - 1) * lda + K) * 2 : 0) : (K > 0 ? ((K - 1) * lda + M) * 2 : 0);
  a.b_bytes = b_kmajor ? (N > 0 ? ((N - 1) * ldb + K) * 2 : 0) : (K > 0 ? ((K - 1) * ldb + N) * 2 : 0);
  set_tiles(a);
  return a;
}

}  // namespace

extern "C" {

int gemm_vocab_loss_desc_validate(const migemm_vocab_loss_desc* desc) { return validate_loss(desc); }

int gemm_vocab_loss_plan_create(const migemm_vocab_loss_desc* desc, migemm_vocab_loss_plan** out) {
  if (!out) return MIGEMM_ERR_INVALID_ARG;
  *out = nullptr;
  int st = validate_loss(desc);
  if (st != MIGEMM_OK) return st;
  int cus = 0;
  static std::atomic<bool> prepared[kMaxDevices];
  st = check_device(desc->device, &cus, prepared, migemm::prepare_loss);
  if (st != MIGEMM_OK) return st;
  migemm_vocab_loss_plan* p = new (std::nothrow) migemm_vocab_loss_plan();
  if (!p) return MIGEMM_ERR_INVALID_ARG;
  p->desc = *desc;
  p->cus = cus;
  lay_out_loss(p);
  return add_live(p, kVocabLoss, out);
}

int gemm_vocab_loss_plan_destroy(migemm_vocab_loss_plan* plan) { return destroy(plan, kVocabLoss); }

size_t gemm_vocab_loss_workspace_size(const migemm_vocab_loss_plan* plan) {
  return is_live(plan, kVocabLoss) ? plan->workspace_bytes : 0;
}

int gemm_vocab_loss_plan_get_info(const migemm_vocab_loss_plan* p, migemm_vocab_loss_info* out) {
  if (!is_live(p, kVocabLoss) || !out) return MIGEMM_ERR_INVALID_ARG;
  const migemm::LossChoice& c = p->choice;
  const auto m = [](int tile) { return (int32_t)migemm::kLossTileM[tile]; };
  const auto n = [](int tile) { return (int32_t)migemm::kLossTileN[tile]; };
  *out = {m(c.forward), n(c.forward)};
  out->cu_count = p->cus;
  if (p->desc.dx_rs == 0) return MIGEMM_OK;
  out->gradient_tile_m = m(c.gradient), out->gradient_tile_n = n(c.gradient);
  out->dx_tile_m = m(c.dx), out->dx_tile_n = n(c.dx), out->dx_splits = c.dx_splits;
  out->dw_tile_m = m(c.dw), out->dw_tile_n = n(c.dw), out->dw_splits = c.dw_splits;
  out->pieces = (int32_t)((p->desc.vocab + p->piece - 1) / p->piece);
  out->piece = p->piece;
  return MIGEMM_OK;
}

int gemm_vocab_loss_run(const migemm_vocab_loss_plan* p, const void* x, const void* w,
                        const int64_t* target, float* loss, float* lse, void* workspace,
                        void* stream) {
  if (!is_live(p, kVocabLoss)) return MIGEMM_ERR_INVALID_ARG;
  const migemm_vocab_loss_desc& d = p->desc;
  if (d.rows == 0) return MIGEMM_OK;
  if (!x || !w || !target || !loss || !lse) return MIGEMM_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(target, 8) || !aligned(loss, 4) || !aligned(lse, 4))
    return MIGEMM_ERR_MISALIGNED;
  const int st = check_workspace(p->workspace_bytes, workspace);
  if (st != MIGEMM_OK) return st;
  if (!current_device_is(d.device)) return MIGEMM_ERR_DEVICE;
  migemm::LossArgs s = {};
  s.V = d.vocab, s.H = d.hidden;
  s.parts = static_cast<float2*>(workspace);
  s.part_rows = p->chunk;
  s.part_cols = migemm::kLossTileN[p->choice.forward] / 2;
  s.target_logit = reinterpret_cast<float*>(s.parts + (d.vocab + s.part_cols - 1) / s.part_cols * p->chunk);
  for (int64_t r = 0; r < d.rows; r += p->chunk) {
    const int64_t rows = d.rows - r < p->chunk ? d.rows - r : p->chunk;
    s.gemm = product(rows, d.vocab, d.hidden, static_cast<const char*>(x) + r * d.x_rs * 2, d.x_rs,
                     true, w, d.w_rs, true, nullptr, 0);
    s.target = target + r, s.loss = loss + r, s.lse = lse + r;
    const hipError_t e =
        migemm::launch_loss_forward(s, p->choice.forward, p->cus, static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return MIGEMM_ERR_LAUNCH;
  }
  return MIGEMM_OK;
}

int gemm_vocab_loss_run_backward(const migemm_vocab_loss_plan* p, const void* x, const void* w,
                                 const int64_t* target, const float* lse, const float* dloss, void* dx,
                                 void* dw, void* workspace, void* stream) {
  if (!is_live(p, kVocabLoss) || p->desc.dx_rs == 0) return MIGEMM_ERR_INVALID_ARG;
  const migemm_vocab_loss_desc& d = p->desc;
  if (!w || !dw || (d.rows > 0 && (!x || !target || !lse || !dloss || !dx)))
    return MIGEMM_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(w, 16) || !aligned(target, 8) || !aligned(lse, 4) ||
      !aligned(dloss, 4) || !aligned(dx, 16) || !aligned(dw, 16))
    return MIGEMM_ERR_MISALIGNED;
  const int st = check_workspace(p->workspace_bytes, workspace);
  if (st != MIGEMM_OK) return st;
  if (!current_device_is(d.device)) return MIGEMM_ERR_DEVICE;
  hipStream_t hs = static_cast<hipStream_t>(stream);
  char* ws = static_cast<char*>(workspace);
  migemm::LossArgs s = {};
  s.T = d.rows, s.V = d.vocab, s.H = d.hidden;
  s.x = x, s.x_rs = d.x_rs, s.dx = dx, s.dx_rs = d.dx_rs;
  s.target = target, s.lse = const_cast<float*>(lse), s.dloss = dloss;
  s.head = reinterpret_cast<migemm::LossHead*>(ws);
  s.from = reinterpret_cast<int*>(ws + p->at_from);
  s.rows_lse = reinterpret_cast<float*>(ws + p->at_lse);
  s.rows_dloss = reinterpret_cast<float*>(ws + p->at_dloss);
  s.rows_target = reinterpret_cast<int*>(ws + p->at_target);
  s.rows_x = reinterpret_cast<unsigned short*>(ws + p->at_rows);
  s.rows_ld = p->rows_rs;
  s.dx_sums = reinterpret_cast<migemm::mid_piece*>(ws + p->at_dx);
  s.dw_sums = reinterpret_cast<migemm::mid_piece*>(ws + p->at_dw);
  s.dx_tiles = p->dx_tiles;
  s.splits = p->choice.dx_splits;
  s.dw_splits = p->choice.dw_splits;
  s.dx_summed = p->dx_summed;
  void* g = ws + p->at_g;
  hipError_t e = migemm::launch_loss_rows(s, hs);
  for (int64_t c = 0; c < d.vocab && e == hipSuccess; c += p->piece) {
    const int64_t cols = d.vocab - c < p->piece ? d.vocab - c : p->piece;
    const char* wc = static_cast<const char*>(w) + c * d.w_rs * 2;
    const bool last = c + cols == d.vocab;
    s.first_col = c;
    s.first_piece = c == 0;
    if (d.rows > 0) {
      s.gemm = product(d.rows, cols, d.hidden, s.rows_x, s.rows_ld, true, wc, d.w_rs, true, g, p->g_rs);
      e = migemm::launch_loss_gradient(s, p->choice.gradient, p->cus, hs);
      if (e != hipSuccess) break;
    }
    s.gemm = product(cols, d.hidden, d.rows, g, p->g_rs, false, s.rows_x, s.rows_ld, false,
                     static_cast<char*>(dw) + c * d.dw_rs * 2, d.dw_rs);
    s.gemm_dx = product(d.rows, d.hidden, cols, g, p->g_rs, true, wc, d.w_rs, false, dx, d.dx_rs);
    e = migemm::launch_loss_products(s, p->choice, last, p->cus, hs);
  }
  return launched(e);
}

int gemm_scaled_desc_validate(const migemm_scaled_desc* desc) { return validate_scaled(desc); }

int gemm_scaled_plan_create(const migemm_scaled_desc* desc, migemm_scaled_plan** out) {
  if (!out) return MIGEMM_ERR_INVALID_ARG;
  *out = nullptr;
  int st = validate_scaled(desc);
  if (st != MIGEMM_OK) return st;
  int cus = 0;
  static std::atomic<bool> prepared[kMaxDevices];
  st = check_device(desc->device, &cus, prepared, migemm::prepare_scaled);
  if (st != MIGEMM_OK) return st;
  migemm_scaled_plan* p = new (std::nothrow) migemm_scaled_plan();
  if (!p) return MIGEMM_ERR_INVALID_ARG;
  p->desc = *desc;
  migemm::KernelArgs& a = p->base.gemm;
  a.M = desc->M, a.N = desc->N, a.K = desc->K;
  a.lda = desc->a_rs, a.ldb = desc->b_cs, a.ldd = desc->d_rs;
  a.a_bytes = a.M > 0 ? (a.M - 1) * a.lda + a.K : 0;
  a.b_bytes = a.N > 0 ? (a.N - 1) * a.ldb + a.K : 0;
  const migemm::ScaledChoice c = migemm::choose_scaled(a.M, a.N, a.K, cus);
  set_tiles(a, c.tile_m);
  p->variant = c.variant;
  p->base.splits = c.splits;
  p->workspace_bytes = (size_t)c.workspace_bytes;
  p->cus = cus;
  return add_live(p, kScaled, out);
}

int gemm_scaled_plan_destroy(migemm_scaled_plan* plan) { return destroy(plan, kScaled); }

size_t gemm_scaled_workspace_size(const migemm_scaled_plan* plan) {
  return is_live(plan, kScaled) ? plan->workspace_bytes : 0;
}

int gemm_scaled_plan_get_info(const migemm_scaled_plan* p, migemm_scaled_info* out) {
  if (!is_live(p, kScaled) || !out) return MIGEMM_ERR_INVALID_ARG;
  const migemm::ScaledKernel k = migemm::scaled_kernel(p->variant);
  *out = {k.tile_m, k.tile_n, k.lds_stages, p->base.splits, k.exact ? 1 : 0, p->cus};
  return MIGEMM_OK;
}

int gemm_scaled_run(const migemm_scaled_plan* p, const void* a, const float* a_scale, const void* b,
                    const float* b_scale, void* d, void* workspace, void* stream) {
  if (!is_live(p, kScaled)) return MIGEMM_ERR_INVALID_ARG;
  const migemm_scaled_desc& e = p->desc;
  if (e.M == 0 || e.N == 0) return MIGEMM_OK;
  if (!a_scale || !b_scale || !d || (e.K > 0 && (!a || !b))) return MIGEMM_ERR_INVALID_ARG;
  if (!aligned(a, 16) || !aligned(b, 16) || !aligned(d, 16) || !aligned(a_scale, 16) ||
      !aligned(b_scale, 16))
    return MIGEMM_ERR_MISALIGNED;
  const int st = check_workspace(p->workspace_bytes, workspace);
  if (st != MIGEMM_OK) return st;
  if (!current_device_is(e.device)) return MIGEMM_ERR_DEVICE;
  migemm::ScaledArgs s = p->base;
  s.gemm.A = a, s.gemm.B = b, s.gemm.D = d;
  s.a_scale = a_scale, s.b_scale = b_scale;
  s.partials = static_cast<migemm::mid_piece*>(workspace);
  return launched(migemm::launch_scaled(s, p->variant, p->cus, static_cast<hipStream_t>(stream)));
}

int gemm_norm_desc_validate(const migemm_norm_desc* desc) { return validate_norm(desc); }

int gemm_norm_plan_create(const migemm_norm_desc* desc, migemm_norm_plan** out) {
  if (!out) return MIGEMM_ERR_INVALID_ARG;
  *out = nullptr;
  int st = validate_norm(desc);
  if (st != MIGEMM_OK) return st;
  int cus = 0;
  static std::atomic<bool> prepared[kMaxDevices];
  st = check_device(desc->device, &cus, prepared, [] { return hipSuccess; });
  if (st != MIGEMM_OK) return st;
  migemm_norm_plan* p = new (std::nothrow) migemm_norm_plan();
  if (!p) return MIGEMM_ERR_INVALID_ARG;
  p->desc = *desc;
  p->cus = cus;
  if (norm_backward(*desc)) {
    p->partial_rows = migemm::norm_partial_rows(desc->rows, desc->cols, cus);
    p->workspace_bytes = (size_t)(p->partial_rows * desc->cols * 4);
  }
  return add_live(p, kNorm, out);
}

int gemm_norm_plan_destroy(migemm_norm_plan* plan) { return destroy(plan, kNorm); }

size_t gemm_norm_workspace_size(const migemm_norm_plan* plan) {
  return is_live(plan, kNorm) ? plan->workspace_bytes : 0;
}

int gemm_norm_plan_get_info(const migemm_norm_plan* p, migemm_norm_info* out) {
  if (!is_live(p, kNorm) || !out) return MIGEMM_ERR_INVALID_ARG;
  const migemm::NormShape f = migemm::norm_shape(p->desc.rows, p->desc.cols);
  const bool back = norm_backward(p->desc);
  *out = {f.waves, f.vectors, back ? f.waves : 0, back ? f.vectors : 0, (int32_t)p->partial_rows, p->cus};
  return MIGEMM_OK;
}

int gemm_norm_run(const migemm_norm_plan* p, const void* x, const void* r, const void* weight,
                  void* h, void* y, float* scale, float* rstd, void* stream) {
  if (!is_live(p, kNorm)) return MIGEMM_ERR_INVALID_ARG;
  const migemm_norm_desc& d = p->desc;
  if (d.rows == 0) return MIGEMM_OK;
  const bool res = norm_residual(d), e4m3 = d.y_type == MIGEMM_FP8_E4M3;
  if ((r != nullptr) != res || (h != nullptr) != res || (scale != nullptr) != e4m3)
    return MIGEMM_ERR_INVALID_ARG;
  if (!x || !weight || !y || !rstd) return MIGEMM_ERR_INVALID_ARG;
  if (!aligned(x, 16) || !aligned(r, 16) || !aligned(weight, 16) || !aligned(h, 16) ||
      !aligned(y, 16) || !aligned(scale, 4) || !aligned(rstd, 4))
    return MIGEMM_ERR_MISALIGNED;
  if (!current_device_is(d.device)) return MIGEMM_ERR_DEVICE;
  migemm::NormArgs a = {};
  a.x = x, a.r = r, a.weight = weight, a.h = h, a.y = y, a.scale = scale, a.rstd = rstd;
  a.rows = d.rows, a.cols = d.cols, a.eps = d.eps;
  a.x_rs = d.x_rs, a.r_rs = d.r_rs, a.h_rs = d.h_rs, a.y_rs = d.y_rs;
  return launched(migemm::launch_norm_forward(a, e4m3, static_cast<hipStream_t>(stream)));
}

int gemm_norm_run_backward(const migemm_norm_plan* p, const void* dy, const void* h,
                           const void* weight, const float* rstd, const void* dh, void* dx,
                           float* dweight, void* workspace, void* stream) {
  if (!is_live(p, kNorm) || !norm_backward(p->desc)) return MIGEMM_ERR_INVALID_ARG;
  const migemm_norm_desc& d = p->desc;
  if (!dweight) return MIGEMM_ERR_INVALID_ARG;
  if (d.rows > 0 && (!dy || !h || !weight || !rstd || !dx || (dh != nullptr) != (d.dh_rs != 0)))
    return MIGEMM_ERR_INVALID_ARG;
  if (!aligned(dy, 16) || !aligned(h, 16) || !aligned(weight, 16) || !aligned(rstd, 4) ||
      !aligned(dh, 16) || !aligned(dx, 16) || !aligned(dweight, 4))
    return MIGEMM_ERR_MISALIGNED;
  const int st = check_workspace(p->workspace_bytes, workspace);
  if (st != MIGEMM_OK) return st;
  if (!current_device_is(d.device)) return MIGEMM_ERR_DEVICE;
  migemm::NormArgs a = {};
  a.x = h, a.dy = dy, a.dh = dh, a.weight = weight, a.dx = dx, a.dweight = dweight;
  a.rstd = const_cast<float*>(rstd), a.partials = static_cast<float*>(workspace);
  a.rows = d.rows, a.cols = d.cols, a.partial_rows = p->partial_rows;
  a.x_rs = norm_residual(d) ? d.h_rs : d.x_rs;
  a.dy_rs = d.dy_rs, a.dh_rs = d.dh_rs, a.dx_rs = d.dx_rs;
  return launched(migemm::launch_norm_backward(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"

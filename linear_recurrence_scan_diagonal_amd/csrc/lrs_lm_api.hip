// lrs_lm_api.hip -- the C ABI declared in include/lrs_lm.h: argument validation,
// workspace carving and launch-plan choice.  All device work is enqueued on
// the caller's stream; nothing here allocates device memory.
#include <math.h>
#include <string.h>

#include "../../include/lrs_lm.h"
#include "lrs_host.hpp"
#include "lrs_internal.hpp"

namespace lrs {
hipError_t launch_copy_or_zero(float* dst, const float* src, int64_t n, hipStream_t s);
}

namespace {

struct Span {
  const void* p;
  size_t n;
};

bool any_overlap(const Span* outs, int no, const Span* ins, int ni) {
  for (int o = 0; o < no; ++o) {
    for (int i = 0; i < ni; ++i)
      if (overlap(outs[o].p, outs[o].n, ins[i].p, ins[i].n)) return true;
    for (int o2 = o + 1; o2 < no; ++o2)
      if (overlap(outs[o].p, outs[o].n, outs[o2].p, outs[o2].n)) return true;
  }
  return false;
}

// Bytes from the first to past the last element of `rows` rows of D elements,
// ld apart.
size_t strided_bytes(int64_t rows, int64_t ld, int64_t D, size_t es) {
  return rows <= 0 ? 0 : ((size_t)(rows - 1) * (size_t)ld + (size_t)D) * es;
}

// Whether two sets of `rows` rows of D elements, each ld apart, share an
// element: their extents may interleave (slices of one wider array).
bool rows_overlap(const void* p, const void* q, int64_t rows, int64_t ld, int64_t D, size_t es) {
  const size_t n = strided_bytes(rows, ld, D, es);
  if (!overlap(p, n, q, n)) return false;
  const uintptr_t a = (uintptr_t)p, b = (uintptr_t)q;
  const size_t off = (size_t)(a < b ? b - a : a - b) % ((size_t)ld * es);
  return !(off >= (size_t)D * es && off <= (size_t)(ld - D) * es);
}

bool io_ok(int io) { return io == LRS_F32 || io == LRS_BF16; }
size_t io_size(int io) { return io == LRS_BF16 ? 2 : 4; }

// Sizes of a gated linear recurrence: no overflow, and 32-bit offsets inside
// one time step.
bool glr_shape(int64_t T, int64_t B, int64_t D, int64_t* C, int64_t* N) {
  return shape_ok(B, D, T, C, N);
}
bool glr_step_fits(int64_t B, int64_t C, int64_t ld) {
  int64_t row;  // 32-bit byte offsets inside a time step
  return C < ((int64_t)1 << 31) && mul_ok(B, ld, &row) && row < ((int64_t)1 << 30);
}

// Workspace of a plan with look-back: the rates of every feature, the status
// words and the tickets.
size_t glr_lookback_bytes(const lrs::ColPlan& p, int64_t D) {
  const int64_t nst = lrs::col_status_words(p);
  return nst > 0 ? lookback_bytes(nst, p.ncb) + align_up((size_t)(2 * D) * 4) : 0;
}

// Pitched extents inside int64 bytes.
bool pitch_ok(int64_t T, int64_t B, int64_t ld) {
  int64_t rows, n;
  return mul_ok(T, B, &rows) && mul_ok(rows, ld, &n) && n <= ((int64_t)1 << 60);
}

}  // namespace

extern "C" {

// ------------------------------------------------- gated linear recurrence

int64_t lrs_glr_checkpoint_rows(int64_t T) {
  return T <= 0 ? 0 : (T - 1) / lrs::kGlrRows + 1;
}

size_t lrs_glr_workspace_bytes(int64_t T, int64_t B, int64_t D) {
  int64_t C, N;
  if (!glr_shape(T, B, D, &C, &N) || N == 0) return 0;
  // the fp32 tiles are the shorter ones
  const size_t a = glr_lookback_bytes(lrs::plan_glr(C, T, LRS_F32, 1, false), D);
  const size_t b = glr_lookback_bytes(lrs::plan_glr(C, T, LRS_F32, 2, false), D);
  return a > b ? a : b;
}

int lrs_glr_fwd(const void* z_r, const void* z_i, const void* x, int64_t ld, const float* bias_r,
                const float* bias_i, const float* decay, const uint8_t* reset, const float* h0,
                void* h, float* h_last, float* checkpoints, int64_t T, int64_t B, int64_t D,
                float c, int io_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  int64_t C, N;
  if (!glr_shape(T, B, D, &C, &N) || !io_ok(io_dtype) || !(c > 0.0f && isfinite(c)))
    return LRS_ERR_INVALID_ARG;
  hipStream_t s = (hipStream_t)stream;
  if (N == 0) {
    if (T == 0 && C > 0 && h_last) return hip_status(lrs::launch_copy_or_zero(h_last, h0, C, s));
    return LRS_OK;
  }
  if (!z_r || !z_i || !x || !bias_r || !bias_i || !decay || !h || ld < D || !pitch_ok(T, B, ld))
    return LRS_ERR_INVALID_ARG;
  const size_t es = io_size(io_dtype);
  if (!aligned(z_r, es) || !aligned(z_i, es) || !aligned(x, es) || !aligned(h, es) ||
      !aligned(bias_r, 4) || !aligned(bias_i, 4) || !aligned(decay, 4) || !aligned(h0, 4) ||
      !aligned(h_last, 4) || !aligned(checkpoints, 4))
    return LRS_ERR_INVALID_ARG;
  const size_t zb = strided_bytes(T * B, ld, D, es), cb = (size_t)C * 4, db = (size_t)D * 4;
  const Span ins[] = {{z_r, zb}, {z_i, zb}, {x, zb}, {bias_r, db}, {bias_i, db}, {decay, db},
                      {reset, (size_t)(T * B)}, {h0, cb}};
  const Span outs[] = {{h, (size_t)N * es}, {h_last, cb},
                       {checkpoints, (size_t)lrs_glr_checkpoint_rows(T) * cb}};
  if (any_overlap(outs, 3, ins, 8)) return LRS_ERR_INVALID_ARG;
  const size_t pair = 2 * es;
  const bool pairs = D % 2 == 0 && ld % 2 == 0 && aligned(z_r, pair) && aligned(z_i, pair) &&
                     aligned(x, pair) && aligned(h, pair) && aligned(checkpoints, 8);
  const lrs::ColPlan p = lrs::plan_glr(C, T, io_dtype, pairs ? 2 : 1);
  if (!glr_step_fits(B, C, ld) || !grid_ok(p.persist ? p.ncb : p.ncb * p.ntb, p.nw * 64))
    return LRS_ERR_UNSUPPORTED;
  const size_t need = glr_lookback_bytes(p, D);
  if (need && (!workspace || workspace_bytes < need)) return LRS_ERR_WORKSPACE;
  uint64_t* status = nullptr;
  unsigned* tickets = nullptr;
  float* rates = nullptr;
  if (need) {
    Carve cv(align_ptr(workspace));
    status = cv.take<uint64_t>(lrs::col_status_words(p));
    tickets = cv.take<unsigned>(p.ncb);
    rates = cv.take<float>(2 * D);
  }
  lrs::GlrArgs g = {};
  g.z_r = z_r;
  g.z_i = z_i;
  g.x = x;
  g.bias_r = bias_r;
  g.bias_i = bias_i;
  g.decay = decay;
  g.reset = reset;
  g.h0 = h0;
  g.h = h;
  g.h_last = h_last;
  g.checkpoints = checkpoints;
  g.T = T;
  g.B = B;
  g.D = D;
  g.ld = ld;
  g.c = c;
  return hip_status(lrs::launch_glr_fwd(g, io_dtype, p, rates, status, tickets, s));
}

static size_t glr_bwd_ws(const lrs::ColPlan& p, int64_t B, int64_t D) {
  return kAlign + lookback_bytes(lrs::col_status_words(p), p.ncb) +
         align_up((size_t)(3 * p.ntb * B * D) * 4) + align_up((size_t)(2 * D) * 4) +
         align_up((size_t)(2 * lrs::col_sum_blocks(p.ntb * B) * D) * 8);
}

size_t lrs_glr_bwd_workspace_bytes(int64_t T, int64_t B, int64_t D) {
  int64_t C, N;
  if (!glr_shape(T, B, D, &C, &N) || N == 0) return 0;
  const size_t a = glr_bwd_ws(lrs::plan_glr_bwd(C, T, LRS_F32, 1, false), B, D);
  const size_t b = glr_bwd_ws(lrs::plan_glr_bwd(C, T, LRS_F32, 2, false), B, D);
  return a > b ? a : b;
}

int lrs_glr_bwd(const void* z_r, const void* z_i, const void* x, int64_t ld, const float* bias_r,
                const float* bias_i, const float* decay, const uint8_t* reset,
                const float* checkpoints, const void* grad_h, const float* grad_h_last,
                void* grad_zr, void* grad_zi, void* grad_x, int64_t ld_grad, float* grad_bias_r,
                float* grad_bias_i, float* grad_decay, float* grad_h0, int64_t T, int64_t B,
                int64_t D, float c, int io_dtype, void* workspace, size_t workspace_bytes,
                void* stream) {
  int64_t C, N;
  if (!glr_shape(T, B, D, &C, &N) || !io_ok(io_dtype) || !(c > 0.0f && isfinite(c)))
    return LRS_ERR_INVALID_ARG;
  hipStream_t s = (hipStream_t)stream;
  if (N == 0) {
    // no steps: the parameters' gradients are empty sums; dL/dh0 = dL/dh_T
    float* sums[3] = {grad_bias_r, grad_bias_i, grad_decay};
    int rc = LRS_OK;
    for (int i = 0; i < 3 && rc == LRS_OK; ++i)
      if (D > 0 && sums[i]) rc = hip_status(lrs::launch_copy_or_zero(sums[i], nullptr, D, s));
    if (rc == LRS_OK && T == 0 && C > 0 && grad_h0)
      rc = hip_status(lrs::launch_copy_or_zero(grad_h0, grad_h_last, C, s));
    return rc;
  }
  if (!z_r || !z_i || !x || !bias_r || !bias_i || !decay || !checkpoints || !grad_h || !grad_zr ||
      !grad_zi || !grad_x || !grad_bias_r || !grad_bias_i || !grad_decay || ld < D ||
      ld_grad < D || !pitch_ok(T, B, ld) || !pitch_ok(T, B, ld_grad))
    return LRS_ERR_INVALID_ARG;
  const size_t es = io_size(io_dtype);
  const void* io[7] = {z_r, z_i, x, grad_h, grad_zr, grad_zi, grad_x};
  for (const void* p : io)
    if (!aligned(p, es)) return LRS_ERR_INVALID_ARG;
  const void* f32[9] = {bias_r, bias_i, decay, checkpoints, grad_h_last,
                        grad_bias_r, grad_bias_i, grad_decay, grad_h0};
  for (const void* p : f32)
    if (!aligned(p, 4)) return LRS_ERR_INVALID_ARG;
  const size_t zb = strided_bytes(T * B, ld, D, es), gb = strided_bytes(T * B, ld_grad, D, es);
  const size_t cb = (size_t)C * 4, db = (size_t)D * 4;
  const Span ins[] = {{z_r, zb}, {z_i, zb}, {x, zb}, {bias_r, db}, {bias_i, db}, {decay, db},
                      {reset, (size_t)(T * B)},
                      {checkpoints, (size_t)lrs_glr_checkpoint_rows(T) * cb},
                      {grad_h, (size_t)N * es}, {grad_h_last, cb}};
  const Span sums[] = {{grad_bias_r, db}, {grad_bias_i, db}, {grad_decay, db}, {grad_h0, cb}};
  if (any_overlap(sums, 4, ins, 10)) return LRS_ERR_INVALID_ARG;
  const void* gz[3] = {grad_zr, grad_zi, grad_x};
  for (int i = 0; i < 3; ++i) {
    const Span one[] = {{gz[i], gb}};
    if (any_overlap(one, 1, ins, 10) || any_overlap(one, 1, sums, 4)) return LRS_ERR_INVALID_ARG;
    if (rows_overlap(gz[i], gz[(i + 1) % 3], T * B, ld_grad, D, es)) return LRS_ERR_INVALID_ARG;
  }
  bool pairs = D % 2 == 0 && ld % 2 == 0 && ld_grad % 2 == 0;
  for (const void* q : io) pairs = pairs && aligned(q, 2 * es);
  const lrs::ColPlan p = lrs::plan_glr_bwd(C, T, io_dtype, pairs ? 2 : 1);
  if (!glr_step_fits(B, C, ld) || !glr_step_fits(B, C, ld_grad) ||
      !grid_ok(p.persist ? p.ncb : p.ncb * p.ntb, p.nw * 64))
    return LRS_ERR_UNSUPPORTED;
  if (!workspace || workspace_bytes < lrs_glr_bwd_workspace_bytes(T, B, D))
    return LRS_ERR_WORKSPACE;
  Carve cv(align_ptr(workspace));
  lrs::GlrArgs g = {};
  g.part = cv.take<float>(3 * p.ntb * C);
  double* acc = cv.take<double>(2 * lrs::col_sum_blocks(p.ntb * B) * D);
  uint64_t* status = nullptr;
  unsigned* tickets = nullptr;
  const int64_t nst = lrs::col_status_words(p);
  if (nst > 0) {
    status = cv.take<uint64_t>(nst);
    tickets = cv.take<unsigned>(p.ncb);
  }
  float* rates = cv.take<float>(2 * D);
  g.z_r = z_r;
  g.z_i = z_i;
  g.x = x;
  g.bias_r = bias_r;
  g.bias_i = bias_i;
  g.decay = decay;
  g.reset = reset;
  g.checkpoints = const_cast<float*>(checkpoints);
  g.T = T;
  g.B = B;
  g.D = D;
  g.ld = ld;
  g.c = c;
  g.grad_h = grad_h;
  g.grad_h_last = grad_h_last;
  g.grad_zr = grad_zr;
  g.grad_zi = grad_zi;
  g.grad_x = grad_x;
  g.ld_grad = ld_grad;
  g.grad_h0 = grad_h0;
  return hip_status(lrs::launch_glr_bwd(g, io_dtype, p, rates, status, tickets, acc,
                                        grad_bias_r, grad_bias_i, grad_decay, s));
}

int lrs_glr_step(const void* z_r, const void* z_i, const void* x, int64_t ld, const float* bias_r,
                 const float* bias_i, const float* decay, const int32_t* slots, float* state,
                 void* h, int64_t B, int64_t D, int64_t S, float c, int io_dtype, void* stream) {
  int64_t C, N, sn;
  if (!glr_shape(1, B, D, &C, &N) || S < 0 || !mul_ok(S, D, &sn) || sn > ((int64_t)1 << 60) ||
      !io_ok(io_dtype) || !(c > 0.0f && isfinite(c)))
    return LRS_ERR_INVALID_ARG;
  if (N == 0) return LRS_OK;
  if (!z_r || !z_i || !x || !bias_r || !bias_i || !decay || !h || (!state && S > 0) || ld < D ||
      !pitch_ok(1, B, ld) || (!slots && S < B))
    return LRS_ERR_INVALID_ARG;
  const size_t es = io_size(io_dtype);
  if (!aligned(z_r, es) || !aligned(z_i, es) || !aligned(x, es) || !aligned(h, es) ||
      !aligned(bias_r, 4) || !aligned(bias_i, 4) || !aligned(decay, 4) || !aligned(slots, 4) ||
      !aligned(state, 4))
    return LRS_ERR_INVALID_ARG;
  const size_t zb = strided_bytes(B, ld, D, es), db = (size_t)D * 4;
  const Span ins[] = {{z_r, zb}, {z_i, zb}, {x, zb}, {bias_r, db}, {bias_i, db}, {decay, db},
                      {slots, (size_t)B * 4}};
  const Span outs[] = {{h, (size_t)C * es}, {state, (size_t)sn * 4}};
  if (any_overlap(outs, 2, ins, 7)) return LRS_ERR_INVALID_ARG;
  if (!glr_step_fits(B, C, ld)) return LRS_ERR_UNSUPPORTED;
  lrs::GlrArgs g = {};
  g.z_r = z_r;
  g.z_i = z_i;
  g.x = x;
  g.bias_r = bias_r;
  g.bias_i = bias_i;
  g.decay = decay;
  g.h = h;
  g.T = 1;
  g.B = B;
  g.D = D;
  g.ld = ld;
  g.c = c;
  return hip_status(lrs::launch_glr_step(g, io_dtype, slots, state, S, (hipStream_t)stream));
}

// -------------------------------------------------------------- layer norm

// A row has 64 threads up to 1024 features (four rows a workgroup), at most 1024
// beyond.
static bool ln_grid_ok(int64_t R, int64_t D) {
  return D <= 1024 ? grid_ok((R + 3) / 4, 256) : grid_ok(R, 1024);
}

int lrs_layernorm_fwd(const void* x, const void* residual, const float* gamma, const float* beta,
                      void* y, void* sum, float* mean, float* rstd, int64_t R, int64_t D,
                      float eps, int io_dtype, void* stream) {
  int64_t n, n2;
  if (!shape_ok(R, D, 1, &n, &n2) || !io_ok(io_dtype) || !(eps >= 0.0f && isfinite(eps)))
    return LRS_ERR_INVALID_ARG;
  if (n == 0) return LRS_OK;
  if (!x || !gamma || !y || !residual != !sum || !mean != !rstd) return LRS_ERR_INVALID_ARG;
  const size_t es = io_size(io_dtype);
  if (!aligned(x, es) || !aligned(residual, es) || !aligned(y, es) || !aligned(sum, es) ||
      !aligned(gamma, 4) || !aligned(beta, 4) || !aligned(mean, 4) || !aligned(rstd, 4))
    return LRS_ERR_INVALID_ARG;
  const size_t nb = (size_t)n * es, db = (size_t)D * 4, rb = (size_t)R * 4;
  // sum may be x or residual themselves: each element is read before it is written
  const bool sx = sum == x, sr = sum == residual;
  const Span ins[] = {{x, nb}, {residual, nb}, {gamma, db}, {beta, db}};
  const Span outs[] = {{y, nb}, {mean, rb}, {rstd, rb}};
  const Span sums[] = {{sum, nb}};
  const Span others[] = {{gamma, db}, {beta, db}, {y, nb}, {mean, rb}, {rstd, rb},
                         {sx ? nullptr : x, nb}, {sr ? nullptr : residual, nb}};
  if (any_overlap(outs, 3, ins, 4) || any_overlap(sums, 1, others, 7)) return LRS_ERR_INVALID_ARG;
  if (!ln_grid_ok(R, D)) return LRS_ERR_UNSUPPORTED;
  return hip_status(lrs::launch_layernorm_fwd(x, residual, gamma, beta, y, sum, mean, rstd, R, D,
                                              eps, io_dtype, (hipStream_t)stream));
}

size_t lrs_layernorm_bwd_workspace_bytes(int64_t R, int64_t D) {
  int64_t n, n2;
  if (!shape_ok(R, D, 1, &n, &n2) || n == 0) return 0;
  const int64_t nb = lrs::ln_bwd_blocks(R, D);
  return kAlign + align_up((size_t)(2 * nb * D) * 4) +
         align_up((size_t)(2 * lrs::col_sum_blocks(nb) * D) * 8);
}

int lrs_layernorm_bwd(const void* s, const float* gamma, const float* mean, const float* rstd,
                      const void* grad_y, const void* grad_sum, void* grad_x, float* grad_gamma,
                      float* grad_beta, int64_t R, int64_t D, int io_dtype, void* workspace,
                      size_t workspace_bytes, void* stream) {
  int64_t n, n2;
  if (!shape_ok(R, D, 1, &n, &n2) || !io_ok(io_dtype)) return LRS_ERR_INVALID_ARG;
  hipStream_t st = (hipStream_t)stream;
  if (n == 0) {  // no rows: empty sums
    int rc = LRS_OK;
    if (D > 0 && grad_gamma) rc = hip_status(lrs::launch_copy_or_zero(grad_gamma, nullptr, D, st));
    if (rc == LRS_OK && D > 0 && grad_beta)
      rc = hip_status(lrs::launch_copy_or_zero(grad_beta, nullptr, D, st));
    return rc;
  }
  if (!s || !gamma || !mean || !rstd || !grad_y || !grad_x || !grad_gamma)
    return LRS_ERR_INVALID_ARG;
  const size_t es = io_size(io_dtype);
  if (!aligned(s, es) || !aligned(grad_y, es) || !aligned(grad_sum, es) || !aligned(grad_x, es) ||
      !aligned(gamma, 4) || !aligned(mean, 4) || !aligned(rstd, 4) || !aligned(grad_gamma, 4) ||
      !aligned(grad_beta, 4))
    return LRS_ERR_INVALID_ARG;
  const size_t nb = (size_t)n * es, db = (size_t)D * 4, rb = (size_t)R * 4;
  const Span ins[] = {{s, nb}, {gamma, db}, {mean, rb}, {rstd, rb},
                      {grad_x == grad_y ? nullptr : grad_y, nb},
                      {grad_x == grad_sum ? nullptr : grad_sum, nb}};
  const Span outs[] = {{grad_x, nb}, {grad_gamma, db}, {grad_beta, db}};
  if (any_overlap(outs, 3, ins, 6)) return LRS_ERR_INVALID_ARG;
  const int64_t blocks = lrs::ln_bwd_blocks(R, D);
  if (!ln_grid_ok(R, D) || D > ((int64_t)1 << 31)) return LRS_ERR_UNSUPPORTED;
  if (!workspace || workspace_bytes < lrs_layernorm_bwd_workspace_bytes(R, D))
    return LRS_ERR_WORKSPACE;
  Carve cv(align_ptr(workspace));
  float* part = cv.take<float>(2 * blocks * D);
  double* acc = cv.take<double>(2 * lrs::col_sum_blocks(blocks) * D);
  return hip_status(lrs::launch_layernorm_bwd(s, gamma, mean, rstd, grad_y, grad_sum, grad_x,
                                              grad_gamma, grad_beta, R, D, io_dtype, part, acc,
                                              st));
}

// ------------------------------------------- cross entropy of a linear head

}  // extern "C"

namespace {

constexpr int64_t kCeMost = (int64_t)1 << 21;

// Carves the workspace of one call; with a null base it only counts.  A call
// without the gradient uses the first part only.
size_t ce_carve(const lrs::CePlan& p, int64_t N, int64_t V, int64_t D, bool backward, void* ws,
                lrs::CeArgs* a) {
  Carve cv(ws);
  const bool f32 = p.parts > 1;
  a->part = (float2*)cv.take<uint64_t>(backward ? p.piece * p.tiles_l : p.piece_f * p.tiles_f);
  a->tlogit = cv.take<float>(backward ? p.piece : p.piece_f);
  a->x_rows = cv.take<uint16_t>(N * p.parts * p.Dp);
  a->w_rows = cv.take<uint16_t>(V * p.parts * p.Dp);
  a->x_unscale = cv.take<float>(f32 ? N : 0);
  a->w_unscale = cv.take<float>(f32 ? p.Vp : 0);
  a->x_top = cv.take<float>(f32 ? N : 0);
  a->w_top = cv.take<float>(f32 ? V : 0);
  a->x_scale = cv.take<float>(f32 ? 2 : 0);
  a->w_scale = cv.take<float>(f32 ? 2 : 0);
  if (!backward) return cv.used;
  a->ratio = cv.take<float>(N);
  a->row_scale = cv.take<float>(N);
  a->top = cv.take<float>(1);
  a->x_cols = cv.take<uint16_t>(D * p.ldx);
  a->w_cols = cv.take<uint16_t>(D * p.ldw);
  a->g = cv.take<uint16_t>(p.piece * p.ldg);
  a->e = f32 ? (void*)cv.take<float>(p.piece * (p.Vp + 32)) : (void*)a->g;
  a->lde = f32 ? p.Vp + 32 : p.ldg;
  a->slots_x = cv.take<float>(p.slots_x ? p.split_x * p.piece * D : 0);
  a->slots_w = cv.take<float>(p.slots_w ? p.split_w * V * D : 0);
  return cv.used;
}

bool ce_sizes(int64_t N, int64_t V, int64_t D, int io) {
  return N >= 0 && V >= 1 && D >= 1 && io_ok(io);
}
bool ce_fits(int64_t N, int64_t V, int64_t D) { return N < kCeMost && V < kCeMost && D < kCeMost; }

int ce_call(const void* x, const void* w, const int64_t* target, const float* grad_loss,
            float* loss, float* lse, void* grad_x, void* grad_w, int64_t N, int64_t V, int64_t D,
            int io, bool forward, bool backward, void* workspace, size_t workspace_bytes,
            void* stream) {
  if (!ce_sizes(N, V, D, io)) return LRS_ERR_INVALID_ARG;
  if (!ce_fits(N, V, D)) return LRS_ERR_UNSUPPORTED;
  hipStream_t s = (hipStream_t)stream;
  const size_t es = io_size(io);
  const size_t wb = (size_t)(V * D) * es;
  if (N == 0) {  // no rows: the gradient of w is an empty sum
    if (!backward) return LRS_OK;
    if (!grad_w || !aligned(grad_w, es)) return LRS_ERR_INVALID_ARG;
    return hip_status(lrs::launch_zero(grad_w, (int64_t)wb, s));
  }
  if (!x || !w || !target || !lse || (forward && !loss) ||
      (backward && (!grad_loss || !grad_x || !grad_w)))
    return LRS_ERR_INVALID_ARG;
  if (!aligned(x, es) || !aligned(w, es) || !aligned(target, 8) || !aligned(lse, 4) ||
      !aligned(loss, 4) || !aligned(grad_loss, 4) || !aligned(grad_x, es) || !aligned(grad_w, es))
    return LRS_ERR_INVALID_ARG;
  const size_t xb = (size_t)(N * D) * es, nb = (size_t)N * 4;
  Span ins[5] = {{x, xb}, {w, wb}, {target, (size_t)N * 8}, {grad_loss, nb}, {nullptr, 0}};
  Span outs[4] = {{loss, nb}, {grad_x, xb}, {grad_w, wb}, {nullptr, 0}};
  (forward ? outs[3] : ins[4]) = {lse, nb};
  if (any_overlap(outs, 4, ins, 5)) return LRS_ERR_INVALID_ARG;
  const lrs::CePlan p = lrs::plan_ce(N, V, D, io);
  lrs::CeArgs a = {};
  const size_t need = kAlign + ce_carve(p, N, V, D, backward, nullptr, &a);
  if (!workspace || workspace_bytes < need) return LRS_ERR_WORKSPACE;
  ce_carve(p, N, V, D, backward, align_ptr(workspace), &a);
  a.x = x;
  a.w = w;
  a.target = target;
  a.grad_loss = grad_loss;
  a.loss = loss;
  a.lse = lse;
  a.grad_x = grad_x;
  a.grad_w = grad_w;
  a.N = N;
  a.V = V;
  a.D = D;
  a.forward = forward;
  a.backward = backward;
  return hip_status(lrs::launch_linear_ce(p, a, io, s));
}

}  // namespace

extern "C" {

size_t lrs_linear_ce_workspace_bytes(int64_t N, int64_t V, int64_t D, int io_dtype, int backward) {
  if (!ce_sizes(N, V, D, io_dtype) || !ce_fits(N, V, D) || N == 0) return 0;
  lrs::CeArgs a = {};
  return kAlign +
         ce_carve(lrs::plan_ce(N, V, D, io_dtype), N, V, D, backward != 0, nullptr, &a);
}

int lrs_linear_ce_fwd(const void* x, const void* w, const int64_t* target, float* loss, float* lse,
                      int64_t N, int64_t V, int64_t D, int io_dtype, void* workspace,
                      size_t workspace_bytes, void* stream) {
  return ce_call(x, w, target, nullptr, loss, lse, nullptr, nullptr, N, V, D, io_dtype, true,
                 false, workspace, workspace_bytes, stream);
}

int lrs_linear_ce_bwd(const void* x, const void* w, const int64_t* target, const float* lse,
                      const float* grad_loss, void* grad_x, void* grad_w, int64_t N, int64_t V,
                      int64_t D, int io_dtype, void* workspace, size_t workspace_bytes,
                      void* stream) {
  return ce_call(x, w, target, grad_loss, nullptr, const_cast<float*>(lse), grad_x, grad_w, N, V, D,
                 io_dtype, false, true, workspace, workspace_bytes, stream);
}

int lrs_linear_ce_fwd_bwd(const void* x, const void* w, const int64_t* target,
                          const float* grad_loss, float* loss, float* lse, void* grad_x,
                          void* grad_w, int64_t N, int64_t V, int64_t D, int io_dtype,
                          void* workspace, size_t workspace_bytes, void* stream) {
  return ce_call(x, w, target, grad_loss, loss, lse, grad_x, grad_w, N, V, D, io_dtype, true, true,
                 workspace, workspace_bytes, stream);
}

}  // extern "C"

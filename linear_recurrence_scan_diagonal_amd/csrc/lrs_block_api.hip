// lrs_block_api.hip -- the C ABI declared in include/lrs_block.h: argument validation
// and workspace carving.  All device work is enqueued on the caller's stream; nothing
// here allocates device memory.
#include <math.h>

#include "../../include/lrs_block.h"
#include "lrs_host.hpp"
#include "lrs_internal.hpp"

namespace lrs {
hipError_t launch_copy_or_zero(float* dst, const float* src, int64_t n, hipStream_t s);
}

namespace {

// What the sizes of a gated delta rule give; no overflow anywhere.
struct GdrSizes {
  int64_t chunks, rows, states, kw, vw;  // T B, B H K V, Hk K, H V
  size_t es, saved;                    // bytes of an element, and of the checkpoints
};
bool gdr_sizes(int64_t T, int64_t B, int64_t H, int64_t Hk, int64_t K, int64_t V, int io,
               GdrSizes* s) {
  if (T < 0 || B < 0 || H < 1 || Hk < 1 || K < 1 || V < 1 || H % Hk != 0 || !io_ok(io))
    return false;
  int64_t n, m;
  if (!mul_ok(Hk, K, &s->kw) || !mul_ok(H, V, &s->vw) || !mul_ok(s->vw, K, &n) ||
      !mul_ok(n, B, &s->states) || !mul_ok(T, B, &s->rows) || !mul_ok(s->rows, s->vw, &n) ||
      !mul_ok(s->rows, s->kw, &m) || n > ((int64_t)1 << 56) || m > ((int64_t)1 << 56) ||
      s->states > ((int64_t)1 << 56))
    return false;
  s->chunks = T / lrs::kGdrRows + (T % lrs::kGdrRows != 0);
  if (!mul_ok(s->chunks, s->states, &n) || n > ((int64_t)1 << 58)) return false;
  if (!mul_ok(n, 4 * (lrs::kGdrRows + 1), &m) || m > ((int64_t)1 << 60)) return false;
  s->es = io_size(io);
  s->saved = (size_t)(s->chunks * B * H * (K + lrs::kGdrRows) * lrs::gdr_saved_pitch(V)) * 4;
  return true;
}
// The kernels' grids and 32-bit sizes: 256 threads a chunk and head, 512 in the backward.
bool gdr_fits(int64_t chunks, int64_t B, int64_t H, int64_t K, int64_t V, bool backward) {
  const int64_t most = (int64_t)1 << 26, columns = (V + 15) / 16;
  int64_t n;
  return K <= lrs::kGdrMostK && V < ((int64_t)1 << 24) && H < ((int64_t)1 << 24) &&
         mul_ok(B, H, &n) && mul_ok(n, chunks > 0 ? chunks : 1, &n) && n < most / (backward ? 8 : 4) &&
         mul_ok(n, columns, &n) && n < most;
}

// 31-bit byte offsets inside a chunk's rows of an array and inside what is kept of a chunk.
bool gdr_rows_fit(int64_t B, int64_t ld, int64_t K, int64_t V) {
  int64_t n;
  return mul_ok(B, ld, &n) && n < ((int64_t)1 << 23) &&
         (K + lrs::kGdrRows) * lrs::gdr_saved_pitch(V) < ((int64_t)1 << 29);
}

// Carves the workspace of a call; with a null base it only counts.
size_t gdr_carve(int64_t chunks, int64_t B, int64_t H, int64_t Hk, int64_t K, int64_t V, int io,
                 bool backward, void* ws, lrs::GdrArgs* a) {
  Carve cv(ws);
  constexpr int64_t C = lrs::kGdrRows;
  const int64_t nv = chunks * B * H, nk = chunks * B * Hk;
  // q and k as fragments of 64 steps, in one or two 16-bit parts
  const int64_t set = (io == LRS_F32 ? 2 : 1) * C * (K <= 64 ? 64 : 128);
  a->cuts = cv.take<uint64_t>(chunks * B);
  a->keeps = cv.take<float>(nv);
  a->mats = cv.take<uint16_t>(nv * lrs::kGdrMats);
  a->kq_rows = cv.take<uint16_t>(nk * 2 * set);
  if (!backward) return cv.used;
  a->decay_sums = cv.take<double>(nv * C);
  a->w = cv.take<float>(nv * C * lrs::gdr_saved_pitch(V));
  a->grad_states = cv.take<float>(nv * K * lrs::gdr_saved_pitch(V));
  a->shared = cv.take<float>(H > Hk ? nv * 2 * C * K : 0);
  return cv.used;
}

size_t gdr_workspace(int64_t T, int64_t B, int64_t H, int64_t Hk, int64_t K, int64_t V, int io,
                     bool backward) {
  GdrSizes z;
  if (!gdr_sizes(T, B, H, Hk, K, V, io, &z) || z.rows == 0 || !gdr_fits(z.chunks, B, H, K, V, backward))
    return 0;
  lrs::GdrArgs a = {};
  return kAlign + gdr_carve(z.chunks, B, H, Hk, K, V, io, backward, nullptr, &a);
}

lrs::GdrArgs gdr_args(const void* q, int64_t ld_q, const void* k, int64_t ld_k, const void* v,
                      int64_t ld_v, const float* log_decay, const float* beta, int64_t T,
                      int64_t B, int64_t H, int64_t Hk, int64_t K, int64_t V, float scale) {
  lrs::GdrArgs a = {};
  a.q = q;
  a.k = k;
  a.v = v;
  a.ld_q = ld_q;
  a.ld_k = ld_k;
  a.ld_v = ld_v;
  a.log_decay = log_decay;
  a.beta = beta;
  a.T = T;
  a.B = B;
  a.H = (int)H;
  a.Hk = (int)Hk;
  a.K = (int)K;
  a.V = (int)V;
  a.scale = scale;
  return a;
}

// 64 threads a row up to 1024 features, at most 1024 beyond.
bool rms_grid_ok(int64_t R, int64_t D) {
  return D <= 1024 ? grid_ok((R + 3) / 4, 256) : grid_ok(R, 1024);
}

// The norm's forward in both forms: y in the I/O type, or bytes with scales.
int rms_call(const void* x, const void* residual, const float* gamma, void* y, float* scales,
             void* sum, float* rstd, int64_t R, int64_t D, int64_t group, float eps, int io,
             void* stream) {
  int64_t n, n2;
  if (!shape_ok(R, D, 1, &n, &n2) || !io_ok(io) || !(eps >= 0.0f && isfinite(eps)))
    return LRS_ERR_INVALID_ARG;
  if (group != 0 && group != 128) return LRS_ERR_INVALID_ARG;
  if (n == 0) return LRS_OK;
  const size_t es = io_size(io);
  const bool bytes = scales != nullptr;
  if (!x || !gamma || !y || !residual != !sum) return LRS_ERR_INVALID_ARG;
  if (!aligned(x, es) || !aligned(residual, es) || (!bytes && !aligned(y, es)) ||
      !aligned(sum, es) || !aligned(gamma, 4) || !aligned(scales, 4) || !aligned(rstd, 4))
    return LRS_ERR_INVALID_ARG;
  const size_t nb = (size_t)n * es, yb = (size_t)n * (bytes ? 1 : es), db = (size_t)D * 4;
  const size_t sb = (size_t)R * (size_t)(group ? (D + group - 1) / group : 1) * 4;
  // sum may be x or residual themselves: each element is read before it is written
  const bool sx = sum == x, sr = sum == residual;
  const Span ins[] = {{x, nb}, {residual, nb}, {gamma, db}};
  const Span outs[] = {{y, yb}, {scales, sb}, {rstd, (size_t)R * 4}};
  const Span sums[] = {{sum, nb}};
  const Span others[] = {{gamma, db}, {y, yb}, {scales, sb}, {rstd, (size_t)R * 4},
                         {sx ? nullptr : x, nb}, {sr ? nullptr : residual, nb}};
  if (any_overlap(outs, 3, ins, 3) || any_overlap(sums, 1, others, 6)) return LRS_ERR_INVALID_ARG;
  if (!rms_grid_ok(R, D)) return LRS_ERR_UNSUPPORTED;
  hipStream_t s = (hipStream_t)stream;
  return hip_status(bytes ? lrs::launch_rmsnorm_fp8(x, residual, gamma, y, scales, sum, R, D,
                                                    group, eps, io, s)
                          : lrs::launch_rmsnorm_fwd(x, residual, gamma, y, sum, rstd, R, D, eps, io,
                                                    s));
}

// An index below 2^24 in the kernels, and 256 threads a row (more only for few rows).
constexpr int64_t kLpMost = (int64_t)1 << 24;

}  // namespace

extern "C" {

// -------------------------------------------------------- gated delta rule

int64_t lrs_gdr_checkpoint_rows(int64_t T) {
  return T <= 0 ? 0 : (T - 1) / lrs::kGdrRows + 1;
}

size_t lrs_gdr_workspace_bytes(int64_t T, int64_t B, int64_t H, int64_t Hk, int64_t K, int64_t V,
                               int io_dtype) {
  return gdr_workspace(T, B, H, Hk, K, V, io_dtype, false);
}

int lrs_gdr_fwd(const void* q, int64_t ld_q, const void* k, int64_t ld_k, const void* v,
                int64_t ld_v, const float* log_decay, const float* beta, const uint8_t* reset,
                const float* state0, void* o, float* state, float* checkpoints, int64_t T,
                int64_t B, int64_t H, int64_t Hk, int64_t K, int64_t V, float scale, int io_dtype,
                void* workspace, size_t workspace_bytes, void* stream) {
  GdrSizes z;
  if (!gdr_sizes(T, B, H, Hk, K, V, io_dtype, &z) || !isfinite(scale)) return LRS_ERR_INVALID_ARG;
  hipStream_t s = (hipStream_t)stream;
  const size_t sb = (size_t)z.states * 4;
  if (!aligned(state0, 4) || !aligned(state, 4)) return LRS_ERR_INVALID_ARG;
  if (z.rows == 0) {
    if (B == 0 || !state) return LRS_OK;
    if (state != state0 && overlap(state, sb, state0, sb)) return LRS_ERR_INVALID_ARG;
    return hip_status(lrs::launch_copy_or_zero(state, state0, z.states, s));
  }
  if (!q || !k || !v || !log_decay || !beta || !o || ld_q < z.kw || ld_k < z.kw || ld_v < z.vw ||
      !pitch_ok(T, B, ld_q) || !pitch_ok(T, B, ld_k) || !pitch_ok(T, B, ld_v))
    return LRS_ERR_INVALID_ARG;
  const size_t es = z.es;
  if (!aligned(q, es) || !aligned(k, es) || !aligned(v, es) || !aligned(o, es) ||
      !aligned(log_decay, 4) || !aligned(beta, 4) || !aligned(checkpoints, 4))
    return LRS_ERR_INVALID_ARG;
  const size_t gb = (size_t)z.rows * (size_t)H * 4;
  const Span ins[] = {{q, strided_bytes(z.rows, ld_q, z.kw, es)},
                      {k, strided_bytes(z.rows, ld_k, z.kw, es)},
                      {v, strided_bytes(z.rows, ld_v, z.vw, es)},
                      {log_decay, gb}, {beta, gb}, {reset, (size_t)z.rows},
                      {state == state0 ? nullptr : state0, sb}};
  const Span outs[] = {{o, (size_t)(z.rows * z.vw) * es}, {state, sb},
                       {checkpoints, z.saved}};
  if (any_overlap(outs, 3, ins, 7)) return LRS_ERR_INVALID_ARG;
  if (!gdr_fits(z.chunks, B, H, K, V, false) || !gdr_rows_fit(B, ld_q, K, V) ||
      !gdr_rows_fit(B, ld_k, K, V) || !gdr_rows_fit(B, ld_v, K, V) || !gdr_rows_fit(B, z.vw, K, V))
    return LRS_ERR_UNSUPPORTED;
  if (!workspace || workspace_bytes < gdr_workspace(T, B, H, Hk, K, V, io_dtype, false))
    return LRS_ERR_WORKSPACE;
  lrs::GdrArgs a = gdr_args(q, ld_q, k, ld_k, v, ld_v, log_decay, beta, T, B, H, Hk, K, V, scale);
  gdr_carve(z.chunks, B, H, Hk, K, V, io_dtype, false, align_ptr(workspace), &a);
  a.reset = reset;
  a.state0 = state0;
  a.o = o;
  a.state = state;
  a.checkpoints = checkpoints;
  return hip_status(lrs::launch_gdr_fwd(a, io_dtype, s));
}

size_t lrs_gdr_bwd_workspace_bytes(int64_t T, int64_t B, int64_t H, int64_t Hk, int64_t K,
                                   int64_t V, int io_dtype) {
  return gdr_workspace(T, B, H, Hk, K, V, io_dtype, true);
}

int lrs_gdr_bwd(const void* q, int64_t ld_q, const void* k, int64_t ld_k, const void* v,
                int64_t ld_v, const float* log_decay, const float* beta, const uint8_t* reset,
                const float* checkpoints, const void* grad_o, const float* grad_state,
                void* grad_q, int64_t ld_gq, void* grad_k, int64_t ld_gk, void* grad_v,
                int64_t ld_gv, float* grad_log_decay, float* grad_beta, float* grad_state0,
                int64_t T, int64_t B, int64_t H, int64_t Hk, int64_t K, int64_t V, float scale,
                int io_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  GdrSizes z;
  if (!gdr_sizes(T, B, H, Hk, K, V, io_dtype, &z) || !isfinite(scale)) return LRS_ERR_INVALID_ARG;
  hipStream_t s = (hipStream_t)stream;
  const size_t sb = (size_t)z.states * 4;
  if (!aligned(grad_state, 4) || !aligned(grad_state0, 4)) return LRS_ERR_INVALID_ARG;
  if (z.rows == 0) {
    if (B == 0 || !grad_state0) return LRS_OK;
    if (grad_state0 != grad_state && overlap(grad_state0, sb, grad_state, sb))
      return LRS_ERR_INVALID_ARG;
    return hip_status(lrs::launch_copy_or_zero(grad_state0, grad_state, z.states, s));
  }
  if (!q || !k || !v || !log_decay || !beta || !checkpoints || !grad_o || !grad_q || !grad_k ||
      !grad_v || !grad_log_decay || !grad_beta || ld_q < z.kw || ld_k < z.kw || ld_v < z.vw ||
      ld_gq < z.kw || ld_gk < z.kw || ld_gv < z.vw)
    return LRS_ERR_INVALID_ARG;
  const int64_t lds[6] = {ld_q, ld_k, ld_v, ld_gq, ld_gk, ld_gv};
  for (int64_t ld : lds)
    if (!pitch_ok(T, B, ld)) return LRS_ERR_INVALID_ARG;
  const size_t es = z.es;
  const void* io[7] = {q, k, v, grad_o, grad_q, grad_k, grad_v};
  for (const void* p : io)
    if (!aligned(p, es)) return LRS_ERR_INVALID_ARG;
  const void* f32[5] = {log_decay, beta, checkpoints, grad_log_decay, grad_beta};
  for (const void* p : f32)
    if (!aligned(p, 4)) return LRS_ERR_INVALID_ARG;
  const size_t gb = (size_t)z.rows * (size_t)H * 4;
  const Span ins[] = {{q, strided_bytes(z.rows, ld_q, z.kw, es)},
                      {k, strided_bytes(z.rows, ld_k, z.kw, es)},
                      {v, strided_bytes(z.rows, ld_v, z.vw, es)},
                      {log_decay, gb}, {beta, gb}, {reset, (size_t)z.rows},
                      {checkpoints, z.saved},
                      {grad_o, (size_t)(z.rows * z.vw) * es},
                      {grad_state == grad_state0 ? nullptr : grad_state, sb}};
  const Span outs[] = {{grad_log_decay, gb}, {grad_beta, gb}, {grad_state0, sb}};
  if (any_overlap(outs, 3, ins, 9)) return LRS_ERR_INVALID_ARG;
  struct Slice {
    const void* p;
    int64_t ld, w;
  } gz[3] = {{grad_q, ld_gq, z.kw}, {grad_k, ld_gk, z.kw}, {grad_v, ld_gv, z.vw}};
  for (int i = 0; i < 3; ++i) {
    const Span one[] = {{gz[i].p, strided_bytes(z.rows, gz[i].ld, gz[i].w, es)}};
    if (any_overlap(one, 1, ins, 9) || any_overlap(one, 1, outs, 3)) return LRS_ERR_INVALID_ARG;
    const Slice& o = gz[(i + 1) % 3];
    if (slices_overlap(gz[i].p, gz[i].ld, gz[i].w, o.p, o.ld, o.w, z.rows, es))
      return LRS_ERR_INVALID_ARG;
  }
  if (!gdr_fits(z.chunks, B, H, K, V, true) || !gdr_rows_fit(B, z.vw, K, V))
    return LRS_ERR_UNSUPPORTED;
  for (int64_t ld : lds)
    if (!gdr_rows_fit(B, ld, K, V)) return LRS_ERR_UNSUPPORTED;
  if (!workspace || workspace_bytes < gdr_workspace(T, B, H, Hk, K, V, io_dtype, true))
    return LRS_ERR_WORKSPACE;
  lrs::GdrArgs a = gdr_args(q, ld_q, k, ld_k, v, ld_v, log_decay, beta, T, B, H, Hk, K, V, scale);
  gdr_carve(z.chunks, B, H, Hk, K, V, io_dtype, true, align_ptr(workspace), &a);
  a.reset = reset;
  a.checkpoints = const_cast<float*>(checkpoints);
  a.grad_o = grad_o;
  a.grad_state = grad_state;
  a.grad_q = grad_q;
  a.grad_k = grad_k;
  a.grad_v = grad_v;
  a.ld_gq = ld_gq;
  a.ld_gk = ld_gk;
  a.ld_gv = ld_gv;
  a.grad_log_decay = grad_log_decay;
  a.grad_beta = grad_beta;
  a.grad_state0 = grad_state0;
  return hip_status(lrs::launch_gdr_bwd(a, io_dtype, s));
}

int lrs_gdr_step(const void* q, int64_t ld_q, const void* k, int64_t ld_k, const void* v,
                 int64_t ld_v, const float* log_decay, const float* beta, const int32_t* slots,
                 float* state, void* o, int64_t B, int64_t H, int64_t Hk, int64_t K, int64_t V,
                 int64_t S, float scale, int io_dtype, void* stream) {
  GdrSizes z, pool;
  if (!gdr_sizes(1, B, H, Hk, K, V, io_dtype, &z) || !isfinite(scale) || S < 0 ||
      !gdr_sizes(1, S, H, Hk, K, V, io_dtype, &pool))
    return LRS_ERR_INVALID_ARG;
  if (B == 0) return LRS_OK;
  if (!q || !k || !v || !log_decay || !beta || !o || (!state && S > 0) || (!slots && S < B) ||
      ld_q < z.kw || ld_k < z.kw || ld_v < z.vw || !pitch_ok(1, B, ld_q) || !pitch_ok(1, B, ld_k) ||
      !pitch_ok(1, B, ld_v))
    return LRS_ERR_INVALID_ARG;
  const size_t es = z.es;
  if (!aligned(q, es) || !aligned(k, es) || !aligned(v, es) || !aligned(o, es) ||
      !aligned(log_decay, 4) || !aligned(beta, 4) || !aligned(slots, 4) || !aligned(state, 4))
    return LRS_ERR_INVALID_ARG;
  const size_t gb = (size_t)B * (size_t)H * 4;
  const Span ins[] = {{q, strided_bytes(B, ld_q, z.kw, es)}, {k, strided_bytes(B, ld_k, z.kw, es)},
                      {v, strided_bytes(B, ld_v, z.vw, es)}, {log_decay, gb}, {beta, gb},
                      {slots, (size_t)B * 4}};
  const Span outs[] = {{o, (size_t)(B * z.vw) * es}, {state, (size_t)pool.states * 4}};
  if (any_overlap(outs, 2, ins, 6)) return LRS_ERR_INVALID_ARG;
  int64_t blocks;
  if (K > lrs::kGdrMostK || V >= ((int64_t)1 << 24) || H >= ((int64_t)1 << 24) ||
      !mul_ok(B * H, (V + 127) / 128, &blocks) || !grid_ok(blocks, 256))
    return LRS_ERR_UNSUPPORTED;
  lrs::GdrArgs a = gdr_args(q, ld_q, k, ld_k, v, ld_v, log_decay, beta, 1, B, H, Hk, K, V, scale);
  a.o = o;
  return hip_status(lrs::launch_gdr_step(a, io_dtype, slots, state, S, (hipStream_t)stream));
}

// ---------------------------------------------------------------- RMS norm

int lrs_rmsnorm_fwd(const void* x, const void* residual, const float* gamma, void* y, void* sum,
                    float* rstd, int64_t R, int64_t D, float eps, int io_dtype, void* stream) {
  return rms_call(x, residual, gamma, y, nullptr, sum, rstd, R, D, 0, eps, io_dtype, stream);
}

int lrs_rmsnorm_fwd_fp8(const void* x, const void* residual, const float* gamma, void* q,
                        float* scales, void* sum, int64_t R, int64_t D, int64_t group, float eps,
                        int io_dtype, void* stream) {
  int64_t n, n2;
  if (shape_ok(R, D, 1, &n, &n2) && n > 0 && !scales) return LRS_ERR_INVALID_ARG;
  return rms_call(x, residual, gamma, q, scales, sum, nullptr, R, D, group, eps, io_dtype, stream);
}

size_t lrs_rmsnorm_bwd_workspace_bytes(int64_t R, int64_t D) {
  int64_t n, n2;
  if (!shape_ok(R, D, 1, &n, &n2) || n == 0) return 0;
  const int64_t nb = lrs::rms_bwd_blocks(R, D);
  return kAlign + align_up((size_t)(nb * D) * 4) +
         align_up((size_t)(lrs::col_sum_blocks(nb) * D) * 8);
}

int lrs_rmsnorm_bwd(const void* s, const float* gamma, const float* rstd, const void* grad_y,
                    const void* grad_sum, void* grad_x, float* grad_gamma, int64_t R, int64_t D,
                    int io_dtype, void* workspace, size_t workspace_bytes, void* stream) {
  int64_t n, n2;
  if (!shape_ok(R, D, 1, &n, &n2) || !io_ok(io_dtype)) return LRS_ERR_INVALID_ARG;
  hipStream_t st = (hipStream_t)stream;
  if (n == 0) {  // no rows: an empty sum
    if (D == 0 || !grad_gamma) return LRS_OK;
    if (!aligned(grad_gamma, 4)) return LRS_ERR_INVALID_ARG;
    return hip_status(lrs::launch_copy_or_zero(grad_gamma, nullptr, D, st));
  }
  if (!s || !gamma || !rstd || !grad_y || !grad_x || !grad_gamma) return LRS_ERR_INVALID_ARG;
  const size_t es = io_size(io_dtype);
  if (!aligned(s, es) || !aligned(grad_y, es) || !aligned(grad_sum, es) || !aligned(grad_x, es) ||
      !aligned(gamma, 4) || !aligned(rstd, 4) || !aligned(grad_gamma, 4))
    return LRS_ERR_INVALID_ARG;
  const size_t nb = (size_t)n * es, db = (size_t)D * 4;
  const Span ins[] = {{s, nb}, {gamma, db}, {rstd, (size_t)R * 4},
                      {grad_x == grad_y ? nullptr : grad_y, nb},
                      {grad_x == grad_sum ? nullptr : grad_sum, nb}};
  const Span outs[] = {{grad_x, nb}, {grad_gamma, db}};
  const Span grads[] = {{grad_y, nb}, {grad_sum, nb}};
  const Span gg[] = {{grad_gamma, db}};
  if (any_overlap(outs, 2, ins, 5) || any_overlap(gg, 1, grads, 2)) return LRS_ERR_INVALID_ARG;
  const int64_t blocks = lrs::rms_bwd_blocks(R, D);
  if (!rms_grid_ok(R, D) || D > ((int64_t)1 << 31)) return LRS_ERR_UNSUPPORTED;
  if (!workspace || workspace_bytes < lrs_rmsnorm_bwd_workspace_bytes(R, D))
    return LRS_ERR_WORKSPACE;
  Carve cv(align_ptr(workspace));
  float* part = cv.take<float>(blocks * D);
  double* acc = cv.take<double>(lrs::col_sum_blocks(blocks) * D);
  return hip_status(lrs::launch_rmsnorm_bwd(s, gamma, rstd, grad_y, grad_sum, grad_x, grad_gamma, R,
                                            D, io_dtype, part, acc, st));
}

// ------------------------------------- log probabilities of given tokens

int lrs_logprobs_fwd(const void* logits, int64_t ld, const int64_t* target, float* logprob,
                     float* entropy, float* lse, int64_t* top_ids, float* top_logprobs, int64_t N,
                     int64_t V, int64_t top, int io_dtype, void* stream) {
  if (N < 0 || V < 1 || top < 0 || top > 64 || top > V || !io_ok(io_dtype))
    return LRS_ERR_INVALID_ARG;
  if (N == 0) return LRS_OK;
  if (!logits || !target || !logprob || !entropy || !lse || ld < V || !pitch_ok(1, N, ld) ||
      (top > 0 && (!top_ids || !top_logprobs)))
    return LRS_ERR_INVALID_ARG;
  const size_t es = io_size(io_dtype);
  if (!aligned(logits, es) || !aligned(target, 8) || !aligned(logprob, 4) ||
      !aligned(entropy, 4) || !aligned(lse, 4) || !aligned(top_ids, 8) || !aligned(top_logprobs, 4))
    return LRS_ERR_INVALID_ARG;
  if (N >= kLpMost || V >= kLpMost) return LRS_ERR_UNSUPPORTED;
  const size_t nb = (size_t)N * 4, tn = (size_t)(N * top);
  const Span ins[] = {{logits, strided_bytes(N, ld, V, es)}, {target, (size_t)N * 8}};
  const Span outs[] = {{logprob, nb}, {entropy, nb}, {lse, nb}, {top_ids, tn * 8},
                       {top_logprobs, tn * 4}};
  if (any_overlap(outs, 5, ins, 2)) return LRS_ERR_INVALID_ARG;
  lrs::LogprobArgs a = {};
  a.logits = logits;
  a.ld = ld;
  a.target = target;
  a.logprob = logprob;
  a.entropy = entropy;
  a.lse = lse;
  a.top_ids = top_ids;
  a.top_logprobs = top_logprobs;
  a.N = N;
  a.V = V;
  a.top = (int)top;
  return hip_status(lrs::launch_logprobs_fwd(a, io_dtype, (hipStream_t)stream));
}

int lrs_logprobs_bwd(const void* logits, int64_t ld, const int64_t* target, const float* lse,
                     const float* entropy, const float* grad_logprob, const float* grad_entropy,
                     void* grad_logits, int64_t ld_grad, int64_t N, int64_t V, int io_dtype,
                     void* stream) {
  if (N < 0 || V < 1 || !io_ok(io_dtype)) return LRS_ERR_INVALID_ARG;
  if (N == 0) return LRS_OK;
  if (!logits || !target || !lse || !grad_logprob || !grad_logits || (grad_entropy && !entropy) ||
      ld < V || ld_grad < V || !pitch_ok(1, N, ld) || !pitch_ok(1, N, ld_grad))
    return LRS_ERR_INVALID_ARG;
  const size_t es = io_size(io_dtype);
  if (!aligned(logits, es) || !aligned(grad_logits, es) || !aligned(target, 8) || !aligned(lse, 4) ||
      !aligned(entropy, 4) || !aligned(grad_logprob, 4) || !aligned(grad_entropy, 4))
    return LRS_ERR_INVALID_ARG;
  if (N >= kLpMost || V >= kLpMost) return LRS_ERR_UNSUPPORTED;
  const size_t nb = (size_t)N * 4;
  const bool own = grad_logits == logits && ld == ld_grad;
  const Span ins[] = {{own ? nullptr : logits, strided_bytes(N, ld, V, es)},
                      {target, (size_t)N * 8}, {lse, nb}, {grad_entropy ? entropy : nullptr, nb},
                      {grad_logprob, nb}, {grad_entropy, nb}};
  const Span outs[] = {{grad_logits, strided_bytes(N, ld_grad, V, es)}};
  if (any_overlap(outs, 1, ins, 6)) return LRS_ERR_INVALID_ARG;
  lrs::LogprobArgs a = {};
  a.logits = logits;
  a.ld = ld;
  a.target = target;
  a.lse = const_cast<float*>(lse);
  a.entropy = const_cast<float*>(entropy);
  a.N = N;
  a.V = V;
  a.grad_logprob = grad_logprob;
  a.grad_entropy = grad_entropy;
  a.grad_logits = grad_logits;
  a.ld_grad = ld_grad;
  return hip_status(lrs::launch_logprobs_bwd(a, io_dtype, (hipStream_t)stream));
}

}  // extern "C"

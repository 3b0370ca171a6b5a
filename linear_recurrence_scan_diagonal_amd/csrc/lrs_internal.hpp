// lrs_internal.hpp -- host-side plumbing shared by the kernel files and the
// C ABI implementation (launch plans and launchers).  Not installed.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace lrs {

// A call whose arrays (all it reads and writes) total at least this many bytes,
// twice the memory-side cache, streams them with nontemporal loads and stores:
// none of its data can still be cached for the next call, and keeping it out of
// the caches measured 8-12% faster.  Smaller calls keep the default policy, so
// that e.g. a backward pass finds part of the forward pass's data in cache.
constexpr int64_t kStreamFootprint = (int64_t)512 << 20;

// Plan overrides of one call (the C ABI's lrs_options); a negative field
// keeps the measured default.
struct Opts {
  int64_t serial_fwd_max_t = -1;    // one lane per channel for T <= this ([B,D,T] forward)
  int64_t serial_bwd_max_t = -1;    // the same for the backward
  int64_t packed_max_t = -1;        // whole channels packed per workgroup for T <= this
  int64_t persist_min_blocks = -1;  // [T,B,D] layers: persistent walk from this many blocks
  int deer_fuse = -1;               // 0: one launch per Newton iteration
};

// Time-contiguous kernels: chunks of nw waves x r rows x 256 steps, nchunk
// chunks per channel.
struct RowPlan {
  int nw = 8;
  int r = 2;
  int64_t nchunk = 1;
  bool stream = false;  // nontemporal loads and stores (arrays far larger than the caches)
  int sub = 1;          // sequential sub-chunks per workgroup (single-workgroup channels)
  bool serial = false;  // short channels: one lane walks each channel (scan_serial.hip)
  int packed = 0;       // short channels: k whole channels per 8-wave, 2048-step workgroup
  int threads() const { return nw * 64; }
  int64_t chunk() const { return (int64_t)nw * r * 256; }
};
// Element type of the scan arrays (the C ABI's LRS_F32 / LRS_BF16); state and
// arithmetic are fp32 either way.
constexpr int kIoF32 = 0, kIoBf16 = 1;
constexpr int64_t io_bytes(int io) { return io == kIoBf16 ? 2 : 4; }
RowPlan plan_scan_fwd_rows(int64_t C, int64_t T, const Opts& o = Opts(), int io = kIoF32);
RowPlan plan_scan_bwd_rows(int64_t C, int64_t T, const Opts& o = Opts(), int io = kIoF32);
RowPlan plan_deer_rows(int64_t C, int64_t T);
RowPlan plan_scan_fused_rows(int64_t C, int64_t T, int io = kIoF32);
RowPlan plan_deer_bwd_rows(int64_t C, int64_t T);

// Feature-contiguous kernels: blocks of 64*cpt channels x nw*l steps.
struct ColPlan {
  int nw = 8, l = 8, cpt = 4;
  int64_t ncb = 1, ntb = 1;
  bool stream = false;   // nontemporal loads and stores (see kStreamFootprint)
  bool persist = false;  // one workgroup per channel block walks all time tiles (no look-back)
};
// Compute units of the current device (cached per device).
int device_cus();
// Channel blocks from which the [T,B,D] layer kernels run persistent
// (device_cus(), or the caller's override).
int64_t persist_min_blocks(const Opts& o = Opts());
ColPlan plan_cols(int64_t C, int64_t T, int nw, int l, int cpt);
ColPlan plan_scan_fwd_tbd(int64_t C, int64_t T, int io = kIoF32);
ColPlan plan_scan_bwd_tbd(int64_t C, int64_t T, int io = kIoF32);
// allow_persist = false: the look-back tile plan (workspace queries size for it).
ColPlan plan_sru(int64_t C, int64_t T, int io_dtype, bool allow_persist = true,
                 const Opts& o = Opts());
int64_t col_status_words(const ColPlan& p);

// Resets look-back state: status words to "not ready", tickets and the
// optional 32-bit words `zero` to 0.  Plain stores from a kernel, so the call
// is safe inside captured graphs.
hipError_t launch_reset(uint64_t* status, int64_t nstatus, unsigned* tickets, int64_t ntickets,
                        uint32_t* zero, int64_t nzero, hipStream_t stream);

// Scan launchers: a, b, h, g, da, db are arrays of element type `io` (kIoF32
// or kIoBf16); h0 and dh0 are fp32.  `vec`: rows and base pointers allow
// 4-element accesses (T % 4 == 0, pointers aligned to 4 elements).
hipError_t launch_scan_fwd_bdt(const void* a, const void* b, const float* h0, void* h, int io,
                               int64_t C, int64_t T, const RowPlan& p, int vec, uint64_t* status,
                               unsigned* tickets, hipStream_t stream);
hipError_t launch_scan_bwd_bdt(const void* a, const void* h, const float* h0, const void* g,
                               void* da, void* db, float* dh0, int io, int64_t C, int64_t T,
                               const RowPlan& p, int vec, uint64_t* status, unsigned* tickets,
                               hipStream_t stream);
// Sequential per-channel scans (one lane per channel) for short channels.
hipError_t launch_scan_fwd_serial(const void* a, const void* b, const float* h0, void* h, int io,
                                  int64_t C, int64_t T, int vec, hipStream_t stream);
hipError_t launch_scan_bwd_serial(const void* a, const void* h, const float* h0, const void* g,
                                  void* da, void* db, float* dh0, int io, int64_t C, int64_t T,
                                  int vec, hipStream_t stream);
// Packed short channels (plan.packed = channels per workgroup).
hipError_t launch_scan_fwd_packed(const void* a, const void* b, const float* h0, void* h, int io,
                                  int64_t C, int64_t T, int k, int vec, hipStream_t stream);
hipError_t launch_scan_bwd_packed(const void* a, const void* h, const float* h0, const void* g,
                                  void* da, void* db, float* dh0, int io, int64_t C, int64_t T,
                                  int k, int vec, hipStream_t stream);
// Forward and backward scan in one pass; the plan must be single-chunk.
hipError_t launch_scan_fused_bdt(const void* a, const void* b, const float* h0, const void* g,
                                 void* h, void* da, void* db, float* dh0, int io, int64_t C,
                                 int64_t T, const RowPlan& p, int vec, hipStream_t stream);
// DEER update norms: three rotating sets of kDeltaSlots words, kDeltaStride
// words apart (one cache line per slot).
constexpr int kDeltaSlots = 64;
constexpr int kDeltaStride = 32;
constexpr int64_t kDeltaSetWords = 3 * kDeltaSlots * kDeltaStride;
// Solve record written by the finish kernel: iterations, converged, non-finite.
constexpr int kDeerRecordWords = 4;
hipError_t launch_deer_finish(const uint32_t* delta_bits, uint32_t* delta_out, int* rec,
                              int k_max, float eps, hipStream_t stream);
hipError_t launch_deer_select(const float* p0, const float* p1, float* h, int64_t n,
                              const int* rec, hipStream_t stream);
// Adjoint of the nonlinear RNN at its solution: the reverse scan kernel, then
// dL/dw from `part` (nchunk * B * D floats) via launch_col_sums.
hipError_t launch_deer_bwd(const float* w, const float* h, const float* h0, const float* g,
                           float* du, float* dw, float* dh0, float* part, double* acc, int64_t B,
                           int64_t D, int64_t T, const RowPlan& p, int vec, uint64_t* status,
                           unsigned* tickets, hipStream_t stream);
// Sequential tanh RNN (one lane per channel, ceil(C / 64) one-wave workgroups;
// vec: T % 4 == 0 and u, h 16-byte aligned).
hipError_t launch_rnn_seq(const float* w, const float* u, const float* h0, float* h, int64_t C,
                          int64_t D, int64_t T, int vec, hipStream_t stream);
// One Newton iteration.  seq_slots != nullptr: per-sequence stopping (norm
// slots kSeqSlots per sequence per set, three sets; seq_delta[seq * k_max + i]
// holds sequence seq's norm of iteration i once k_deer_seq_book folded it).
constexpr int kSeqSlots = 4;
hipError_t launch_deer_iter(const float* w, const float* u, const float* y, const float* h0,
                            float* yn, int64_t C, int64_t D, int64_t T, const RowPlan& p, int vec,
                            uint64_t* status, unsigned* tickets, uint32_t* delta_bits,
                            uint32_t* delta_out, int iter, float eps, hipStream_t stream,
                            uint32_t* seq_slots = nullptr, const uint32_t* seq_delta = nullptr,
                            int k_max = 0);
// DEER with the Newton iterations fused into one walk over each channel
// (single-workgroup channels, k_max <= kDeerFuseMax): the pass over all k_max
// iterations into `out` (h, or a buffer when h holds the starting iterate),
// the finish kernel writing the record and norms, the redo launch when the stop
// rule fired earlier, and the copy into h.  `sets` holds k_max slot sets of
// kDeltaSlots * kDeltaStride words, cleared beforehand.  Per-sequence
// stopping: seq_delta (B * k_max norms, cleared) and seq_rec (4 words per
// sequence) replace sets, delta_out and rec.
constexpr int kDeerFuseMax = 8;
hipError_t launch_deer_fused(const float* w, const float* u, const float* y0, const float* h0,
                             float* out, float* h, int64_t C, int64_t D, int64_t T,
                             const RowPlan& p, int vec, int k_max, float eps, uint32_t* sets,
                             uint32_t* delta_out, int* rec, hipStream_t stream,
                             uint32_t* seq_delta = nullptr, int* seq_rec = nullptr);
// Pieces shared by the fused solves: the record from the norm sets, and the
// copy of the pass's result into h unless a redo wrote h.
hipError_t launch_deer_fused_finish(const uint32_t* sets, uint32_t* delta_out, int* rec,
                                    int k_max, float eps, hipStream_t stream);
hipError_t launch_deer_fused_select(const float* src, float* h, int64_t n, const int* rec,
                                    int k_max, hipStream_t stream);
hipError_t launch_deer_seq_book(uint32_t* seq_slots, uint32_t* seq_delta, int64_t nseq, int k_max,
                                int iter, hipStream_t stream);
hipError_t launch_deer_seq_finish(const uint32_t* seq_delta, int* seq_rec, int64_t nseq,
                                  int k_max, float eps, hipStream_t stream);
hipError_t launch_deer_seq_select(const float* p0, const float* p1, float* h, int64_t nseq,
                                  int64_t n, const int* seq_rec, hipStream_t stream);

hipError_t launch_scan_fwd_tbd(const void* a, const void* b, const float* h0, void* h, int io,
                               int64_t C, int64_t T, const ColPlan& p, int vec, uint64_t* status,
                               unsigned* tickets, hipStream_t stream);
hipError_t launch_scan_bwd_tbd(const void* a, const void* h, const float* h0, const void* g,
                               void* da, void* db, float* dh0, int io, int64_t C, int64_t T,
                               const ColPlan& p, int vec, uint64_t* status, unsigned* tickets,
                               hipStream_t stream);
hipError_t launch_sru_fwd(const void* zf, const void* zr, const void* zx, const float* bias_f,
                          const float* bias_r, const float* c0, void* h, float* c_last,
                          float* c_states, int64_t T, int64_t B, int64_t D, int io_dtype,
                          const ColPlan& p, int vec, uint64_t* status, unsigned* tickets,
                          hipStream_t stream);
ColPlan plan_sru_bwd(int64_t C, int64_t T, int io_dtype);
// Per-feature parameter gradients: column sums of nmat consecutive [R, D]
// matrices of partial sums (R = partials per feature), accumulated in fp64 in a
// fixed order into out0 (and out1 for nmat = 2).  `acc` holds
// nmat * col_sum_blocks(R) * D doubles.
int64_t col_sum_blocks(int64_t R);
hipError_t launch_col_sums(const float* part, int nmat, int64_t R, int64_t D, double* acc,
                           float* out0, float* out1, hipStream_t stream);

// The same for up to three matrices and as many outputs, for the operators of
// lrs_lm.h: one launch while R is small (any D at the same speed), the two
// stages above otherwise.  `acc` as above for nmat matrices.
hipError_t launch_param_sums(const float* part, int nmat, int64_t R, int64_t D, double* acc,
                             float* const* outs, hipStream_t stream);

// Launches the SRU backward kernel and the bias-gradient reduction; `part`
// holds 2 * ntb * B * D floats of per-tile partial sums.
hipError_t launch_sru_bwd(const void* zf, const void* zr, const void* zx, const float* bias_f,
                          const float* bias_r, const float* c0, const float* cs, const void* gh,
                          const float* gcl, void* dzf, void* dzr, void* dzx, float* dbf,
                          float* dbr, float* dc0, float* part, double* acc, int64_t T, int64_t B,
                          int64_t D, int io_dtype, const ColPlan& p, int vec, uint64_t* status,
                          unsigned* tickets, hipStream_t stream);

// LSTM cell-state layer with input-only gates (gated_cell.hip).  `save`: the
// forward also writes the cell states.
// allow_persist = false: the look-back tile plan (workspace queries size for it).
ColPlan plan_lstm(int64_t C, int64_t T, int io_dtype, bool save, bool allow_persist = true,
                  const Opts& o = Opts());
ColPlan plan_lstm_bwd(int64_t C, int64_t T, int io_dtype);
hipError_t launch_lstm_fwd(const void* zf, const void* zi, const void* zc, const void* zo,
                           const float* c0, void* h, float* c_last, float* c_states, int64_t T,
                           int64_t C, int io_dtype, const ColPlan& p, int vec, uint64_t* status,
                           unsigned* tickets, hipStream_t stream);
hipError_t launch_lstm_bwd(const void* zf, const void* zi, const void* zc, const void* zo,
                           const float* c0, const float* cs, const void* gh, const float* gcl,
                           void* dzf, void* dzi, void* dzc, void* dzo, float* dc0, int64_t T,
                           int64_t C, int io_dtype, const ColPlan& p, int vec, uint64_t* status,
                           unsigned* tickets, hipStream_t stream);

// SRU with v_f * c_{t-1} in the forget gate, by DEER (sru_deer.hip).
ColPlan plan_sru_deer(int64_t C, int64_t T, int io_dtype, bool allow_persist = true,
                      const Opts& o = Opts());
hipError_t launch_sru_deer_iter(const void* zf, const void* zx, const float* bias_f,
                                const float* v_f, const float* c0, const float* y, float* yn,
                                int64_t T, int64_t C, int64_t D, int io_dtype, const ColPlan& p,
                                int vec, uint64_t* status, unsigned* tickets,
                                uint32_t* delta_bits, uint32_t* delta_out, int iter, float eps,
                                hipStream_t stream);
// SRU-by-DEER with the iterations fused into the persistent walk (plan.persist,
// k_max <= kDeerFuseMax): pass into `out`, finish, redo into c_states, select.
hipError_t launch_sru_deer_fused(const void* zf, const void* zx, const float* bias_f,
                                 const float* v_f, const float* c0, const float* c_init,
                                 float* out, float* c_states, int64_t T, int64_t C, int64_t D,
                                 int io_dtype, const ColPlan& p, int vec, int k_max, float eps,
                                 uint32_t* sets, uint32_t* delta_out, int* rec,
                                 hipStream_t stream);
hipError_t launch_sru_deer_out(const void* zr, const void* zx, const float* bias_r,
                               const float* c, void* h, float* c_last, int64_t N, int64_t C,
                               int64_t D, int io_dtype, int vec, hipStream_t stream);

// Gated linear recurrence (glr.hip).  Arrays as in lrs_lm.h; the forward reads
// and writes the first group, the backward also the second.
constexpr int kGlrRows = 64;  // time steps a tile, and between two checkpoints
struct GlrArgs {
  const void *z_r, *z_i, *x;
  const float *bias_r, *bias_i, *decay;
  const uint8_t* reset;
  const float* h0;
  void* h;
  float *h_last, *checkpoints;
  int64_t T, B, D, ld;
  float c;
  const void* grad_h;
  const float* grad_h_last;
  void *grad_zr, *grad_zi, *grad_x;
  int64_t ld_grad;
  float* grad_h0;
  float* part;  // [3][ntb * B][D]: the tiles' sums for bias_r, bias_i and decay
  const float* rates;  // [2][D]: k and dk of every feature (glr_rates), or null
};
// allow_persist = false: the look-back tile plan (workspace queries size for it).
// cpt: channels a lane, 2 where every row of every array can be read in aligned
// pairs, else 1.
ColPlan plan_glr(int64_t C, int64_t T, int io, int cpt, bool allow_persist = true);
ColPlan plan_glr_bwd(int64_t C, int64_t T, int io, int cpt, bool allow_persist = true);
// rates: [2][D] fp32 of workspace; status and tickets (reset here) null where the
// plan needs no look-back.
hipError_t launch_glr_fwd(GlrArgs& g, int io, const ColPlan& p, float* rates,
                          uint64_t* status, unsigned* tickets, hipStream_t stream);
hipError_t launch_glr_bwd(GlrArgs& g, int io, const ColPlan& p, float* rates,
                          uint64_t* status, unsigned* tickets, double* acc, float* grad_bias_r,
                          float* grad_bias_i, float* grad_decay, hipStream_t stream);
hipError_t launch_glr_step(const GlrArgs& g, int io, const int32_t* slots, float* state, int64_t S,
                           hipStream_t stream);

// Layer norm (layernorm.hip).  ln_bwd_blocks: row blocks of the backward, each
// leaving one partial sum a feature in part ([2][blocks][D]).
hipError_t launch_layernorm_fwd(const void* x, const void* residual, const float* gamma,
                                const float* beta, void* y, void* sum, float* mean, float* rstd,
                                int64_t R, int64_t D, float eps, int io, hipStream_t stream);
int64_t ln_bwd_blocks(int64_t R, int64_t D);
hipError_t launch_layernorm_bwd(const void* s, const float* gamma, const float* mean,
                                const float* rstd, const void* grad_y, const void* grad_sum,
                                void* grad_x, float* grad_gamma, float* grad_beta, int64_t R,
                                int64_t D, int io, float* part, double* acc, hipStream_t stream);

// Cross entropy of a linear head (linear_ce.hip).  The plan of a shape, and the
// arrays of a call; the workspace's own are bf16 or fp16 (uint16_t) or fp32.
struct CePlan {
  int parts = 1;        // 16-bit parts of an operand's element
  int64_t Dp = 0, Vp = 0;           // features and classes, rounded up
  int64_t piece = 0, pieces = 0;    // rows of a piece of the gradient, and how many
  int64_t piece_f = 0;              // rows of a piece of the forward alone
  int64_t ldg = 0, ldw = 0, ldx = 0;  // row pitch of G, of w^T and of x^T
  int64_t tiles_f = 0, tiles_l = 0; // class tiles, forward alone and a piece's
  int tm_l = 0;                     // classes of a piece's tile
  int shape_f = 0, shape_l = 0, shape_x = 0, shape_w = 0;  // tile shapes of the products
  int64_t split_x = 1, split_w = 1;        // shares of the gradients' k loops
  bool slots_x = false, slots_w = false;   // fp32 partial results are kept
};
struct CeArgs {
  const void *x, *w;
  const int64_t* target;
  const float* grad_loss;
  float *loss, *lse;
  void *grad_x, *grad_w;
  int64_t N, V, D;
  bool forward, backward;
  uint16_t *x_rows, *w_rows;  // [N][parts Dp], [V][parts Dp]
  float *x_unscale, *w_unscale, *x_top, *w_top;  // [N], [Vp], [N], [V] (fp32 inputs)
  float *x_scale, *w_scale;   // 2 each (fp32 inputs)
  float2* part;               // [piece][class tiles]
  float* tlogit;              // [piece]
  // the gradient's
  uint16_t *x_cols, *w_cols;  // [D][ldx], [D][ldw]
  void* e;                    // [piece][lde]; bf16 inputs: G's own memory
  int64_t lde;
  uint16_t* g;                // [piece][ldg]
  float *ratio, *row_scale, *top;  // [N], [N], 1
  float *slots_x, *slots_w;   // [split_x][piece][D], [split_w][V][D]
};
CePlan plan_ce(int64_t N, int64_t V, int64_t D, int io);
hipError_t launch_linear_ce(const CePlan& p, const CeArgs& a, int io, hipStream_t stream);
// Fill with zero bytes (p aligned to 2, an even number of bytes).
hipError_t launch_zero(void* p, int64_t bytes, hipStream_t stream);


// Gated delta rule (gdr.hip).  Arrays as in lrs_block.h, then the workspace's own, by
// chunk of kGdrRows steps, sequence and head (of v, or of q and k where marked *); the
// backward also has the last group.
constexpr int kGdrRows = 64;   // steps a chunk, and between two checkpoints
constexpr int kGdrMostK = 128;
// Elements from row to row of the states and vectors kept in fp32: V in fours.
__host__ __device__ __forceinline__ int64_t gdr_saved_pitch(int64_t V) { return (V + 3) & ~(int64_t)3; }
constexpr int kGdrMats = 13312;  // 16-bit values of a chunk's matrices and coefficients
struct GdrArgs {
  const void *q, *k, *v;
  int64_t ld_q, ld_k, ld_v;
  const float *log_decay, *beta;
  const uint8_t* reset;
  const float* state0;
  void* o;
  float *state, *checkpoints;
  int64_t T, B;
  int H, Hk, K, V;
  float scale;
  uint64_t* cuts;                             // a bit a step that begins a document, by chunk and sequence
  float* keeps;                               // 1: the whole chunk's decay
  uint16_t* mats;                             // [kGdrMats]
  uint16_t* kq_rows;                          // * fragments of k, then of q
  const void* grad_o;
  const float* grad_state;
  void *grad_q, *grad_k, *grad_v;
  int64_t ld_gq, ld_gk, ld_gv;
  float *grad_log_decay, *grad_beta, *grad_state0;
  double* decay_sums;                         // [64]
  float* w;                                   // [64][V], rows gdr_saved_pitch apart
  float* grad_states;                         // [K][V], the same
  float* shared;                              // [2][64][K]: dq and dk of heads that share q and k
};
hipError_t launch_gdr_fwd(const GdrArgs& a, int io, hipStream_t stream);
hipError_t launch_gdr_bwd(const GdrArgs& a, int io, hipStream_t stream);
hipError_t launch_gdr_step(const GdrArgs& a, int io, const int32_t* slots, float* state,
                           int64_t nslots, hipStream_t stream);

// RMS norm (rmsnorm.hip).  rms_bwd_blocks as ln_bwd_blocks, one sum a feature.
hipError_t launch_rmsnorm_fwd(const void* x, const void* residual, const float* gamma, void* y,
                              void* sum, float* rstd, int64_t R, int64_t D, float eps, int io,
                              hipStream_t stream);
// group: features that share a scale, 128 or D.
hipError_t launch_rmsnorm_fp8(const void* x, const void* residual, const float* gamma, void* y,
                              float* scales, void* sum, int64_t R, int64_t D, int64_t group,
                              float eps, int io, hipStream_t stream);
int64_t rms_bwd_blocks(int64_t R, int64_t D);
hipError_t launch_rmsnorm_bwd(const void* s, const float* gamma, const float* rstd,
                              const void* grad_y, const void* grad_sum, void* grad_x,
                              float* grad_gamma, int64_t R, int64_t D, int io, float* part,
                              double* acc, hipStream_t stream);

// Log probabilities of given logits (logprobs.hip).
struct LogprobArgs {
  const void* logits;
  int64_t ld;
  const int64_t* target;
  float *logprob, *entropy, *lse;
  int64_t* top_ids;
  float* top_logprobs;
  int64_t N, V;
  int top;
  const float *grad_logprob, *grad_entropy;
  void* grad_logits;
  int64_t ld_grad;
};
hipError_t launch_logprobs_fwd(const LogprobArgs& a, int io, hipStream_t stream);
hipError_t launch_logprobs_bwd(const LogprobArgs& a, int io, hipStream_t stream);

}  // namespace lrs

// gdr.hip -- the gated delta rule: forward, backward and single tokens.
//
// A head's state S is a [K,V] matrix; with a_t = exp(log_decay_t) (0 at a restart)
//   S <- a_t S,  delta_t = v_t - S^T k_t,  S <- S + k_t (beta_t delta_t)^T,
//   o_t = scale S^T q_t.
//
// Chunks of 64 steps.  With S0 the state entering a chunk, G_i the sum of the chunk's
// log decays up to step i, D_ij = exp(G_i - G_j) and (j < i) L_ij = D_ij k_i.k_j:
//   R = V - diag(exp G) K S0,  (I + L diag(beta)) delta = R,  u = beta delta,
//   o_i = scale (exp(G_i) S0^T q_i + sum_{j<=i} D_ij (q_i.k_j) u_j),
//   S  <- exp(G_C) S0 + sum_i exp(G_C - G_i) k_i u_i^T.
// The columns of S (and of V, R, delta, u, o) do not depend on each other, so a wave
// walks the chunks of 16 columns by itself, its [K,16] piece of S in registers.
//   k_gdr_prep   every chunk at once: the [64,64] matrices D q k^T (P) and
//                T2 = (I + L diag(beta))^-1, and q, k and these as operands of the
//                matrix cores;
//   k_gdr_chain  the chain over the chunks (and, for the backward, delta of every
//                chunk from its checkpoint, all chunks at once);
//   k_gdr_back   the same chain in reverse, for dS: with do' = scale do
//                du = P^T do' + exp(G_C - G) K dS,  w = T^T du (T = (I + diag(beta) L)^-1),
//                dv = dR = beta w,  dS0 = exp(G_C) dS + (exp G q)^T do' - (exp G k)^T dR;
//   k_gdr_grads  every chunk at once, from S0, dS, delta and w: dbeta = w.delta,
//                dP = do' u^T, dL = -dR u^T and through them and the states dq, dk and
//                the decay's gradient.
//
// Restarts.  A chunk is taken apart into its documents' segments: the matrices are made
// and used a segment at a time, rows outside count as 0 by selection, never by a
// product, so that nothing of a document reaches another, NaN and infinities included.
//
// Numbers.  Sums, states and decays are fp32 or more.  What a product of the matrix
// cores takes is split into two fp16 parts, hi + lo = x to 2^-22, scaled by a power of
// two that brings its row's (or, for the states and what is like V, its column's)
// largest value near fp16's largest: 2^-22 of an element or 2^-39 of that largest is
// lost.  bf16 q, k and do need one part.  So a product takes two or three products of
// parts, at the matrix cores' fp16 rate, where their fp32 rate is a sixteenth of it.
//
// An operand that is multiplied from the left is kept as fragments, the 1 KiB that the
// 64 lanes read of 16 rows x 32 columns: lane l = 16 g + r has row r, and for e < 8 the
// column kappa(g, e) = 16 (e / 4) + 4 g + e % 4.  In that order the accumulators of two
// products on top of each other (lane l: column r, rows 4 g + 0..3) are the right
// operand of the next product as they are.
#include "lrs_device.hpp"
#include "lrs_internal.hpp"

namespace lrs {

namespace {

typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x2_any __attribute__((ext_vector_type(2), aligned(2)));

constexpr int kC = kGdrRows;   // steps a chunk
constexpr int kPad = 4;        // floats between the rows of a [64,64] matrix in LDS
constexpr int kFrag = 512;     // values of a fragment
constexpr float kLeastDecay = -16384.0f;  // below it a factor is 0 in fp32 either way

template <typename IO>
constexpr int kParts = sizeof(IO) == 4 ? 2 : 1;

struct Split {
  f16x8_t hi, lo;
};

// A power of two that brings a largest absolute value to [2^14, 2^15), and its inverse.
// An infinity or NaN counts as the largest finite binade: it stays what it is.
struct Scale {
  float up, down;
};
__device__ __forceinline__ Scale scale_of(uint32_t top) {  // bits of the absolute value
  uint32_t e = top >> 23;
  e = e < 15u ? 15u : e > 254u ? 254u : e;
  return {as_f32((268u - e) << 23), as_f32((e - 14u) << 23)};
}
__device__ __forceinline__ uint32_t abs_bits(float v) { return as_u32(v) & 0x7FFFFFFFu; }
__device__ __forceinline__ uint32_t max_u(uint32_t a, uint32_t b) { return a > b ? a : b; }

// The largest over the four lanes that share a row or column (r = lane % 16).
__device__ __forceinline__ uint32_t quad_max(uint32_t m) {
  m = max_u(m, (uint32_t)__shfl_xor((int)m, 16));
  return max_u(m, (uint32_t)__shfl_xor((int)m, 32));
}
template <int N>
__device__ __forceinline__ uint32_t top_of(const float (&v)[N]) {
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < N; ++i) m = max_u(m, abs_bits(v[i]));
  return m;
}

// Two fp16 parts of eight values times a power of two.
template <bool LOW = true>
__device__ __forceinline__ Split split8(const float* v, float up) {
  Split s;
#pragma unroll
  for (int i = 0; i < 8; i += 2) {
    const f32x2_t x = {v[i] * up, v[i + 1] * up};
    const f16x2_t h = __builtin_convertvector(x, f16x2_t);
    s.hi[i] = h[0];
    s.hi[i + 1] = h[1];
    if constexpr (LOW) {
      const f32x2_t y = {x[0] - (float)h[0], x[1] - (float)h[1]};
      const f16x2_t l = __builtin_convertvector(y, f16x2_t);
      s.lo[i] = l[0];
      s.lo[i + 1] = l[1];
    }
  }
  return s;
}

__device__ __forceinline__ f32x4_t mma(f16x8_t a, f16x8_t b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}
// a b for operands of one or two parts; the product of two low parts, 2^-22 of it, is left out.
template <int PA, int PB>
__device__ __forceinline__ f32x4_t mma_parts(const f16x8_t (&a)[PA], const f16x8_t (&b)[PB],
                                             f32x4_t c) {
  if constexpr (PA == 2) c = mma(a[1], b[0], c);
  if constexpr (PB == 2) c = mma(a[0], b[1], c);
  return mma(a[0], b[0], c);
}

constexpr f32x4_t kZero4 = {0.0f, 0.0f, 0.0f, 0.0f};

// Four elements from column c on of a row of n; 0 past the end.
__device__ __forceinline__ void ld4(const float* row, int c, int n, float* v) {
  if (c + 4 <= n) {
    const f32x4_any q = *reinterpret_cast<const f32x4_any*>(row + c);
    v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = c + j < n ? row[c + j] : 0.0f;
}
__device__ __forceinline__ void ld4(const uint16_t* row, int c, int n, float* v) {
  if (c + 4 <= n) {
    const u32x2_any q = *reinterpret_cast<const u32x2_any*>(row + c);
    v[0] = bf16_lo(q.x); v[1] = bf16_hi(q.x); v[2] = bf16_lo(q.y); v[3] = bf16_hi(q.y);
    return;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = c + j < n ? io_ld(row, c + j) : 0.0f;
}

// The segment that step i belongs to: its first step, given the chunk's restarts.
__device__ __forceinline__ int seg_start(uint64_t cuts, int i) {
  const uint64_t m = cuts & (~0ull >> (63 - i));
  return m ? 63 - __builtin_clzll(m) : 0;
}
// The step after the last one of the segment that begins at i.
__device__ __forceinline__ int seg_end(uint64_t cuts, int i) {
  const uint64_t m = i >= 63 ? 0ull : cuts & (~0ull << (i + 1));
  return m ? __builtin_ctzll(m) : kC;
}

// Bytes 0xFFFF for the columns (steps) of [s, e) in a fragment's k step ks.
__device__ __forceinline__ f16x8_t keep_steps(f16x8_t f, int ks, int s, int e) {
  const int g = (threadIdx.x & 63) >> 4;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int step = 32 * ks + 16 * (i >> 2) + 4 * g + (i & 3);
    f[i] = step >= s && step < e ? f[i] : (_Float16)0.0f;
  }
  return f;
}

// ---------------------------------------------------------------------------
// Workspace of a call, in arrays of chunk-heads: index (c B + b) Hk + hk, or with H, h.
// ---------------------------------------------------------------------------
// fp32 values a step that k_gdr_prep leaves, [chunk-head][kCoef][64]
enum { kEnterK, kEnterQ, kLeaveK, kBeta, kRowT, kRowP, kRowT2, kRowKq, kRowKk, kCoef };

template <int KP>
__device__ __forceinline__ f16x8_t frag(const uint16_t* base, int index) {
  return *reinterpret_cast<const f16x8_t*>(base + (int64_t)index * kFrag + (threadIdx.x & 63) * 8);
}

// ---------------------------------------------------------------------------
// k_gdr_prep
// ---------------------------------------------------------------------------
typedef float Mat[kC][kC + kPad];

// tm = (I + am)^-1 for a strictly lower triangular am; 256 threads.  The diagonal
// blocks of 16 by substitution, a wave each; then block (i, j) = -inv_i sum_m am_im tm_mj
// by fp32 products, a diagonal of blocks at a time.
__device__ void invert(const Mat& am, Mat& tm) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, g = lane >> 4, r = lane & 15;
  float x[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float s = i == r ? 1.0f : 0.0f;
#pragma unroll
    for (int j = 0; j < i; ++j) s = __builtin_fmaf(-am[16 * w + i][16 * w + j], x[j], s);
    x[i] = s;
  }
#pragma unroll
  for (int i = 0; i < 16; ++i)
    if (g == 0) tm[16 * w + i][16 * w + r] = x[i];
  __syncthreads();
#pragma unroll
  for (int d = 1; d < 4; ++d) {
    if (w >= d) {
      const int j = w - d;
      f32x4_t acc = kZero4;
      for (int m = j; m < w; ++m)
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          acc = __builtin_amdgcn_mfma_f32_16x16x4f32(am[16 * w + r][16 * m + 4 * kk + g],
                                                     tm[16 * m + 4 * kk + g][16 * j + r], acc, 0, 0, 0);
      f32x4_t out = kZero4;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        out = __builtin_amdgcn_mfma_f32_16x16x4f32(tm[16 * w + r][16 * w + 4 * g + i], acc[i], out,
                                                   0, 0, 0);
#pragma unroll
      for (int i = 0; i < 4; ++i) tm[16 * w + 4 * g + i][16 * j + r] = -out[i];
    }
    __syncthreads();
  }
}

// Rows [s, e) of m (or of its transpose) as fragments in two parts, each row scaled by
// its largest; 4 waves, 16 rows each.  dst: [part][row tile][k step][512].
template <bool TRANSPOSED>
__device__ __forceinline__ void emit(const Mat& m, uint16_t* dst, float* row_scale, int s, int e) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, g = lane >> 4, r = lane & 15;
  const int row = 16 * w + r;
  float v[16];
#pragma unroll
  for (int ks = 0; ks < 2; ++ks)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int col = 32 * ks + 16 * (j >> 2) + 4 * g + (j & 3);
      v[8 * ks + j] = TRANSPOSED ? m[col][row] : m[row][col];
    }
  const Scale sc = scale_of(quad_max(top_of(v)));
  if (row < s || row >= e) return;
#pragma unroll
  for (int ks = 0; ks < 2; ++ks) {
    const Split p = split8(v + 8 * ks, sc.up);
    uint16_t* to = dst + (w * 2 + ks) * kFrag + lane * 8;
    *reinterpret_cast<f16x8_t*>(to) = p.hi;
    *reinterpret_cast<f16x8_t*>(to + 8 * kFrag) = p.lo;
  }
  if (g == 0) row_scale[row] = sc.down;
}

template <typename IO, int KP, bool BWD>
__global__ __launch_bounds__(256) void k_gdr_prep(GdrArgs a) {
  constexpr int NP = kParts<IO>, KS = KP / 32;
  __shared__ __align__(16) uint16_t kf[NP][4 * KS * kFrag];
  __shared__ __align__(16) uint16_t qf[NP][4 * KS * kFrag];
  __shared__ Mat am, tm;
  __shared__ float rk[kC], rq[kC], bt[kC];
  __shared__ double gs[kC];
  __shared__ uint64_t cuts_s;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, g = lane >> 4, r = lane & 15;
  const int64_t ch = blockIdx.x;
  const int h = (int)(ch % a.H), share = a.H / a.Hk, hk = h / share;
  const int64_t cb = ch / a.H;
  const int64_t b = cb % a.B, c = cb / a.B;
  const int64_t kh = cb * a.Hk + hk;

  if (w == 0) {
    const int64_t t = c * kC + lane;
    const bool in = t < a.T;
    double G = 0.0;
    bool cut = false;
    float beta = 0.0f;
    if (in) {
      const float l = a.log_decay[(t * a.B + b) * a.H + h];
      G = (double)(l < kLeastDecay ? kLeastDecay : l);
      beta = a.beta[(t * a.B + b) * a.H + h];
      cut = a.reset && a.reset[t * a.B + b];
    }
    const uint64_t cuts = __ballot(cut);
    if (cut) G = 0.0;  // the sum starts again behind a restart
    const int first = seg_start(cuts, lane);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const double before = __shfl_up(G, d);
      if (lane - d >= first) G += before;
    }
    gs[lane] = G;
    bt[lane] = beta;
    if (lane == 0) {
      cuts_s = cuts;
      if (h == 0) a.cuts[cb] = cuts;
    }
    if constexpr (BWD) a.decay_sums[ch * kC + lane] = G;
  }

  // 16 rows of k and q a wave
  const int row = 16 * w + r;
  const int64_t t = c * kC + row;
  auto load = [&](const IO* base, int64_t ld, float (&v)[KP / 4]) __attribute__((always_inline)) {
    const IO* p = base + ((t * a.B + b) * ld + (int64_t)hk * a.K);
#pragma unroll
    for (int j = 0; j < 2 * KS; ++j) {
      if (t < a.T) ld4(p, 16 * j + 4 * g, a.K, v + 4 * j);
      else v[4 * j] = v[4 * j + 1] = v[4 * j + 2] = v[4 * j + 3] = 0.0f;
    }
  };
  float kv[KP / 4], qv[KP / 4];
  load((const IO*)a.k, a.ld_k, kv);
  load((const IO*)a.q, a.ld_q, qv);
  const Scale sk = scale_of(quad_max(top_of(kv))), sq = scale_of(quad_max(top_of(qv)));
  f16x8_t qa[KS][NP];
#pragma unroll
  for (int ks = 0; ks < KS; ++ks) {
    const Split k2 = split8<NP == 2>(kv + 8 * ks, sk.up), q2 = split8<NP == 2>(qv + 8 * ks, sq.up);
    const int at = (w * KS + ks) * kFrag + lane * 8;
    *reinterpret_cast<f16x8_t*>(&kf[0][at]) = k2.hi;
    *reinterpret_cast<f16x8_t*>(&qf[0][at]) = q2.hi;
    qa[ks][0] = q2.hi;
    if constexpr (NP == 2) {
      *reinterpret_cast<f16x8_t*>(&kf[1][at]) = k2.lo;
      *reinterpret_cast<f16x8_t*>(&qf[1][at]) = q2.lo;
      qa[ks][1] = q2.lo;
    }
  }
  if (g == 0) {
    rk[row] = sk.down;
    rq[row] = sq.down;
  }
  __syncthreads();

  // the heads that share k and q leave them once, and as columns over the steps too
  if (h % share == 0) {
    constexpr int kSet = NP * 4 * KS * kFrag;
    for (int i = threadIdx.x; i < kSet / 8; i += 256) {
      *reinterpret_cast<f16x8_t*>(a.k_rows + kh * kSet + i * 8) =
          *reinterpret_cast<const f16x8_t*>(&kf[0][0] + i * 8);
      *reinterpret_cast<f16x8_t*>(a.q_rows + kh * kSet + i * 8) =
          *reinterpret_cast<const f16x8_t*>(&qf[0][0] + i * 8);
    }
    // fragment (part, row tile of K, k step of 32 steps)
    for (int i = threadIdx.x; i < kSet / 8; i += 256) {
      const int l = i & 63, f = i >> 6, ks = f & 1, kt = (f >> 1) % (KP / 16), p = f / (KP / 8);
      const int col = 16 * kt + (l & 15);  // of K: its place in a row's fragments
      const int in = (col >> 5) * kFrag + ((col >> 2) & 3) * 128 + ((col >> 4) & 1) * 4 + (col & 3);
      f16x8_t kc, qc;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int step = 32 * ks + 16 * (e >> 2) + 4 * (l >> 4) + (e & 3);
        const int at = (step >> 4) * KS * kFrag + in + (step & 15) * 8;
        kc[e] = __builtin_bit_cast(_Float16, kf[p][at]);
        if constexpr (BWD) qc[e] = __builtin_bit_cast(_Float16, qf[p][at]);
      }
      *reinterpret_cast<f16x8_t*>(a.k_cols + kh * kSet + i * 8) = kc;
      if constexpr (BWD) *reinterpret_cast<f16x8_t*>(a.q_cols + kh * kSet + i * 8) = qc;
    }
  }

  // rows 16 w..: k k^T and q k^T (the blocks up to the diagonal)
  f32x4_t kk[4], qk[4];
#pragma unroll
  for (int ct = 0; ct < 4; ++ct) {
    kk[ct] = qk[ct] = kZero4;
    if (ct > w) continue;
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) {
      f16x8_t ka[NP], kb[NP];
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        ka[p] = *reinterpret_cast<const f16x8_t*>(&kf[p][(w * KS + ks) * kFrag + lane * 8]);
        kb[p] = *reinterpret_cast<const f16x8_t*>(&kf[p][(ct * KS + ks) * kFrag + lane * 8]);
      }
      kk[ct] = mma_parts<NP, NP>(ka, kb, kk[ct]);
      qk[ct] = mma_parts<NP, NP>(qa[ks], kb, qk[ct]);
    }
  }

  const uint64_t cuts = cuts_s;
  float* coef = a.coef + ch * (kCoef * kC);
  if (threadIdx.x < kC) {
    const int i = threadIdx.x;
    const float enter = expf((float)gs[i]), leave = expf((float)(gs[kC - 1] - gs[i]));
    coef[kEnterK * kC + i] = enter * rk[i];
    coef[kEnterQ * kC + i] = enter * rq[i] * a.scale;
    coef[kLeaveK * kC + i] = leave * rk[i];
    coef[kBeta * kC + i] = bt[i];
    coef[kRowKk * kC + i] = rk[i];
    coef[kRowKq * kC + i] = rq[i];
    if (i == 0) a.keeps[ch] = expf((float)gs[kC - 1]);
  }
  uint16_t* t2 = a.t2_rows + ch * (2 * 8 * kFrag);
  uint16_t* pf = a.p_rows + ch * (2 * 8 * kFrag);
  uint16_t* tt = BWD ? a.tt_rows + ch * (2 * 8 * kFrag) : nullptr;
  for (int s = 0; s < kC;) {
    const int e = seg_end(cuts, s);
    // P, then L diag(beta) (and diag(beta) L for the backward)
#pragma unroll
    for (int ct = 0; ct < 4; ++ct)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int ri = 16 * w + 4 * g + i, cj = 16 * ct + r;
        const bool in = cj <= ri && cj >= s && ri < e;
        const float d = in ? expf((float)(gs[ri] - gs[cj])) * rk[cj] : 0.0f;
        tm[ri][cj] = in ? qk[ct][i] * rq[ri] * d : 0.0f;
        am[ri][cj] = in && cj < ri ? kk[ct][i] * rk[ri] * d * bt[cj] : 0.0f;
      }
    __syncthreads();
    emit<BWD>(tm, pf, coef + kRowP * kC, s, e);
    __syncthreads();
#pragma unroll
    for (int ct = 0; ct < 4; ++ct)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (ct != w) tm[16 * w + 4 * g + i][16 * ct + r] = 0.0f;  // each wave its rows
    __syncthreads();
    invert(am, tm);
    emit<false>(tm, t2, coef + kRowT2 * kC, s, e);
    __syncthreads();
    if constexpr (BWD) {
#pragma unroll
      for (int ct = 0; ct < 4; ++ct)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int ri = 16 * w + 4 * g + i, cj = 16 * ct + r;
          const bool in = cj < ri && cj >= s && ri < e;
          am[ri][cj] =
              in ? kk[ct][i] * rk[ri] * rk[cj] * expf((float)(gs[ri] - gs[cj])) * bt[ri] : 0.0f;
        }
      __syncthreads();
      invert(am, tm);
      emit<true>(tm, tt, coef + kRowT * kC, s, e);
      __syncthreads();
    }
    s = e;
  }
}

// ---------------------------------------------------------------------------
// The chains.  A wave has 16 columns; the four lanes of a column hold its rows.
// ---------------------------------------------------------------------------

// A column's largest value over the four lanes that hold it, as its scale.
template <int N>
__device__ __forceinline__ Scale col_scale(const f32x4_t (&v)[N]) {
  uint32_t m = 0u;
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) m = max_u(m, abs_bits(v[i][j]));
  return scale_of(quad_max(m));
}
// Accumulators of 16-row tiles as right operands of k steps of 32.
template <int PARTS, int N>
__device__ __forceinline__ void to_operand(const f32x4_t (&v)[N], float up,
                                           f16x8_t (&out)[N / 2][PARTS]) {
#pragma unroll
  for (int ks = 0; ks < N / 2; ++ks) {
    float x[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[j] = v[2 * ks][j];
      x[4 + j] = v[2 * ks + 1][j];
    }
    const Split s = split8<PARTS == 2>(x, up);
    out[ks][0] = s.hi;
    if constexpr (PARTS == 2) out[ks][1] = s.lo;
  }
}
// Four coefficients of the steps that the lane's accumulators of row tile rt hold.
__device__ __forceinline__ f32x4_t coef4(const float* coef, int which, int rt) {
  const int g = (threadIdx.x & 63) >> 4;
  return *reinterpret_cast<const f32x4_t*>(coef + which * kC + 16 * rt + 4 * g);
}

// DELTA: one chunk a wave; leaves its delta, from its checkpoint.
// Otherwise: the chain over all chunks.
template <typename IO, int KP, bool DELTA>
__global__ __launch_bounds__(256) void k_gdr_chain(GdrArgs a) {
  constexpr int NP = kParts<IO>, KS = KP / 32, KT = KP / 16;
  constexpr int kSet = NP * 4 * KS * kFrag;
  const int lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
  const int vblocks = (a.V + 15) / 16;
  const int64_t nc = (a.T + kC - 1) / kC, chains = a.B * a.H * vblocks;
  int64_t id = (int64_t)blockIdx.x * (blockDim.x / 64) + (threadIdx.x >> 6);
  if (id >= (DELTA ? nc : 1) * chains) return;  // whole waves
  const int64_t c0 = DELTA ? id / chains : 0, c1 = DELTA ? c0 + 1 : nc;
  if constexpr (DELTA) id -= c0 * chains;
  const int vb = (int)(id % vblocks);
  const int64_t bh = id / vblocks, b = bh / a.H;
  const int h = (int)(bh % a.H), hk = h / (a.H / a.Hk);
  const int col = 16 * vb + r;
  const bool colin = col < a.V;
  const int64_t sn = (int64_t)a.K * a.V;  // of one state

  f32x4_t S[KT];
  auto load_state = [&](const float* p) __attribute__((always_inline)) {
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int k = 16 * kt + 4 * g + i;
        S[kt][i] = colin && k < a.K ? p[(int64_t)k * a.V + col] : 0.0f;
      }
  };
  auto store_state = [&](float* p) __attribute__((always_inline)) {
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int k = 16 * kt + 4 * g + i;
        if (colin && k < a.K) p[(int64_t)k * a.V + col] = S[kt][i];
      }
  };
  if constexpr (DELTA) {
    load_state(a.checkpoints + (c0 * a.B * a.H + bh) * sn);
  } else if (a.state0) {
    load_state(a.state0 + bh * sn);
  } else {
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) S[kt] = kZero4;
  }

  for (int64_t c = c0; c < c1; ++c) {
    const int64_t ch = (c * a.B + b) * a.H + h, kh = (c * a.B + b) * a.Hk + hk;
    if (!DELTA && a.checkpoints) store_state(a.checkpoints + ch * sn);
    const uint64_t cuts = a.cuts[c * a.B + b];
    const float* coef = a.coef + ch * (kCoef * kC);
    const uint16_t* kf = a.k_rows + kh * kSet;
    const uint16_t* qf = a.q_rows + kh * kSet;
    const uint16_t* kc = a.k_cols + kh * kSet;
    const uint16_t* t2 = a.t2_rows + ch * (16 * kFrag);
    const uint16_t* pf = a.p_rows + ch * (16 * kFrag);
    float vv[4][4];
#pragma unroll
    for (int rt = 0; rt < 4; ++rt)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t t = c * kC + 16 * rt + 4 * g + i;
        vv[rt][i] = colin && t < a.T
                        ? io_ld((const IO*)a.v, (t * a.B + b) * a.ld_v + (int64_t)h * a.V + col)
                        : 0.0f;
      }
    for (int s = 0; s < kC;) {
      const int e = seg_end(cuts, s);
      const bool fresh = (cuts >> s) & 1, whole = s == 0 && e == kC;
      f32x4_t R[4], O[4];
      if (fresh) {
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) S[kt] = kZero4;
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) {
          O[rt] = kZero4;
#pragma unroll
          for (int i = 0; i < 4; ++i) R[rt][i] = vv[rt][i];
        }
      } else {
        const Scale sc = col_scale(S);
        f16x8_t sb[KS][2];
        to_operand<2>(S, sc.up, sb);
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) {
          f32x4_t x = kZero4, y = kZero4;
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            f16x8_t ka[NP], qa[NP];
#pragma unroll
            for (int p = 0; p < NP; ++p) {
              ka[p] = frag<KP>(kf, (p * 4 + rt) * KS + ks);
              if (!DELTA) qa[p] = frag<KP>(qf, (p * 4 + rt) * KS + ks);
            }
            x = mma_parts<NP, 2>(ka, sb[ks], x);
            if (!DELTA) y = mma_parts<NP, 2>(qa, sb[ks], y);
          }
          const f32x4_t ek = coef4(coef, kEnterK, rt), eq = coef4(coef, kEnterQ, rt);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            R[rt][i] = __builtin_fmaf(-ek[i], x[i] * sc.down, vv[rt][i]);
            O[rt][i] = DELTA ? 0.0f : eq[i] * (y[i] * sc.down);
          }
        }
      }
      if (!whole) {
#pragma unroll
        for (int rt = 0; rt < 4; ++rt)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int step = 16 * rt + 4 * g + i;
            R[rt][i] = step >= s && step < e ? R[rt][i] : 0.0f;
          }
      }
      // delta = T2 R, u = beta delta
      f32x4_t U[4];
      {
        const Scale sc = col_scale(R);
        f16x8_t rb[2][2];
        to_operand<2>(R, sc.up, rb);
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) {
          f32x4_t x = kZero4;
#pragma unroll
          for (int ks = 0; ks <= rt / 2; ++ks) {
            const f16x8_t ta[2] = {frag<KP>(t2, rt * 2 + ks), frag<KP>(t2, 8 + rt * 2 + ks)};
            x = mma_parts<2, 2>(ta, rb[ks], x);
          }
          const f32x4_t rs = coef4(coef, kRowT2, rt), be = coef4(coef, kBeta, rt);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int step = 16 * rt + 4 * g + i;
            const bool in = whole || (step >= s && step < e);
            const float d = x[i] * sc.down * rs[i];
            if constexpr (DELTA) {
              if (in) a.delta[(ch * kC + step) * a.Vp + col] = colin ? d : 0.0f;
            }
            U[rt][i] = in ? d * be[i] : 0.0f;
          }
        }
      }
      if constexpr (!DELTA) {
        const Scale sc = col_scale(U);
        f16x8_t ub[2][2];
        to_operand<2>(U, sc.up, ub);
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) {
          f32x4_t x = kZero4;
#pragma unroll
          for (int ks = 0; ks <= rt / 2; ++ks) {
            const f16x8_t pa[2] = {frag<KP>(pf, rt * 2 + ks), frag<KP>(pf, 8 + rt * 2 + ks)};
            x = mma_parts<2, 2>(pa, ub[ks], x);
          }
          const f32x4_t rs = coef4(coef, kRowP, rt);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int step = 16 * rt + 4 * g + i;
            const int64_t t = c * kC + step;
            if (colin && t < a.T && step >= s && step < e)
              io_st((IO*)a.o, ((t * a.B + b) * a.H + h) * a.V + col,
                    __builtin_fmaf(x[i] * sc.down, rs[i] * a.scale, O[rt][i]));
          }
        }
        if (e == kC) {  // the segment that leaves the chunk
          f32x4_t L[4];
#pragma unroll
          for (int rt = 0; rt < 4; ++rt) {
            const f32x4_t lv = coef4(coef, kLeaveK, rt);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int step = 16 * rt + 4 * g + i;
              L[rt][i] = whole || step >= s ? U[rt][i] * lv[i] : 0.0f;
            }
          }
          const Scale sl = col_scale(L);
          f16x8_t lb[2][2];
          to_operand<2>(L, sl.up, lb);
          const float keep = a.keeps[ch];
#pragma unroll
          for (int kt = 0; kt < KT; ++kt) {
            f32x4_t x = kZero4;
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
              f16x8_t ka[NP];
#pragma unroll
              for (int p = 0; p < NP; ++p) {
                ka[p] = frag<KP>(kc, (p * KT + kt) * 2 + ks);
                if (!whole) ka[p] = keep_steps(ka[p], ks, s, e);
              }
              x = mma_parts<NP, 2>(ka, lb[ks], x);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float add = x[i] * sl.down;
              S[kt][i] = fresh ? add : __builtin_fmaf(keep, S[kt][i], add);
            }
          }
        }
      }
      s = e;
    }
  }
  if constexpr (!DELTA) {
    if (a.state) store_state(a.state + bh * sn);
  }
}

// The chain in reverse: dS, and w, dv and every chunk's dS on the way.
template <typename IO, int KP>
__global__ __launch_bounds__(256) void k_gdr_back(GdrArgs a) {
  constexpr int NP = kParts<IO>, KS = KP / 32, KT = KP / 16;
  constexpr int kSet = NP * 4 * KS * kFrag;
  const int lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
  const int vblocks = (a.V + 15) / 16;
  const int64_t id = (int64_t)blockIdx.x * (blockDim.x / 64) + (threadIdx.x >> 6);
  if (id >= a.B * a.H * vblocks) return;  // whole waves
  const int vb = (int)(id % vblocks);
  const int64_t bh = id / vblocks, b = bh / a.H;
  const int h = (int)(bh % a.H), hk = h / (a.H / a.Hk);
  const int col = 16 * vb + r;
  const bool colin = col < a.V;
  const int64_t nc = (a.T + kC - 1) / kC;
  const int64_t sn = (int64_t)a.K * a.V;

  f32x4_t S[KT];  // dS
#pragma unroll
  for (int kt = 0; kt < KT; ++kt)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int k = 16 * kt + 4 * g + i;
      S[kt][i] = a.grad_state && colin && k < a.K ? a.grad_state[bh * sn + (int64_t)k * a.V + col]
                                                  : 0.0f;
    }
  auto store_state = [&](float* p) __attribute__((always_inline)) {
#pragma unroll
    for (int kt = 0; kt < KT; ++kt)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int k = 16 * kt + 4 * g + i;
        if (colin && k < a.K) p[(int64_t)k * a.V + col] = S[kt][i];
      }
  };

  for (int64_t c = nc - 1; c >= 0; --c) {
    const int64_t ch = (c * a.B + b) * a.H + h, kh = (c * a.B + b) * a.Hk + hk;
    store_state(a.grad_states + ch * sn);
    const uint64_t cuts = a.cuts[c * a.B + b];
    const float* coef = a.coef + ch * (kCoef * kC);
    const uint16_t* kf = a.k_rows + kh * kSet;
    const uint16_t* kc = a.k_cols + kh * kSet;
    const uint16_t* qc = a.q_cols + kh * kSet;
    const uint16_t* tt = a.tt_rows + ch * (16 * kFrag);
    const uint16_t* pt = a.p_rows + ch * (16 * kFrag);
    f32x4_t go[4];
#pragma unroll
    for (int rt = 0; rt < 4; ++rt)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t t = c * kC + 16 * rt + 4 * g + i;
        go[rt][i] = colin && t < a.T
                        ? io_ld((const IO*)a.grad_o, ((t * a.B + b) * a.H + h) * a.V + col)
                        : 0.0f;
      }
    for (int e = kC; e > 0;) {
      const int s = seg_start(cuts, e - 1);
      const bool fresh = (cuts >> s) & 1, whole = s == 0 && e == kC;
      f32x4_t dO[4], U[4];
#pragma unroll
      for (int rt = 0; rt < 4; ++rt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int step = 16 * rt + 4 * g + i;
          dO[rt][i] = whole || (step >= s && step < e) ? go[rt][i] : 0.0f;
        }
      // du = scale P^T do + exp(G_C - G) K dS
      {
        const Scale sc = col_scale(dO);
        f16x8_t ob[2][NP];
        to_operand<NP>(dO, sc.up, ob);
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) {
          f32x4_t x = kZero4;
#pragma unroll
          for (int ks = rt / 2; ks < 2; ++ks) {
            const f16x8_t pa[2] = {frag<KP>(pt, rt * 2 + ks), frag<KP>(pt, 8 + rt * 2 + ks)};
            x = mma_parts<2, NP>(pa, ob[ks], x);
          }
          const f32x4_t rs = coef4(coef, kRowP, rt);
#pragma unroll
          for (int i = 0; i < 4; ++i) U[rt][i] = x[i] * sc.down * (rs[i] * a.scale);
        }
      }
      if (e == kC) {
        const Scale sc = col_scale(S);
        f16x8_t sb[KS][2];
        to_operand<2>(S, sc.up, sb);
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) {
          f32x4_t x = kZero4;
#pragma unroll
          for (int ks = 0; ks < KS; ++ks) {
            f16x8_t ka[NP];
#pragma unroll
            for (int p = 0; p < NP; ++p) ka[p] = frag<KP>(kf, (p * 4 + rt) * KS + ks);
            x = mma_parts<NP, 2>(ka, sb[ks], x);
          }
          const f32x4_t lv = coef4(coef, kLeaveK, rt);
#pragma unroll
          for (int i = 0; i < 4; ++i) U[rt][i] = __builtin_fmaf(x[i] * sc.down, lv[i], U[rt][i]);
        }
      }
      if (!whole) {
#pragma unroll
        for (int rt = 0; rt < 4; ++rt)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int step = 16 * rt + 4 * g + i;
            U[rt][i] = step >= s && step < e ? U[rt][i] : 0.0f;
          }
      }
      // w = T^T du, dv = beta w
      f32x4_t W[4];
      {
        const Scale sc = col_scale(U);
        f16x8_t ub[2][2];
        to_operand<2>(U, sc.up, ub);
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) {
          f32x4_t x = kZero4;
#pragma unroll
          for (int ks = rt / 2; ks < 2; ++ks) {
            const f16x8_t ta[2] = {frag<KP>(tt, rt * 2 + ks), frag<KP>(tt, 8 + rt * 2 + ks)};
            x = mma_parts<2, 2>(ta, ub[ks], x);
          }
          const f32x4_t rs = coef4(coef, kRowT, rt), be = coef4(coef, kBeta, rt);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int step = 16 * rt + 4 * g + i;
            const int64_t t = c * kC + step;
            const bool in = step >= s && step < e;
            const float d = in ? x[i] * sc.down * rs[i] : 0.0f;
            const float dv = d * be[i];
            if (in) a.w[(ch * kC + step) * a.Vp + col] = colin ? d : 0.0f;
            if (in && colin && t < a.T)
              io_st((IO*)a.grad_v, (t * a.B + b) * a.ld_gv + (int64_t)h * a.V + col, dv);
            W[rt][i] = dv;
          }
        }
      }
      if (fresh) {
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) S[kt] = kZero4;
      } else {
        // dS0 = exp(G_C) dS (of the last segment) + (exp G q)^T do' - (exp G k)^T dv
        f32x4_t X[4], Y[4];
#pragma unroll
        for (int rt = 0; rt < 4; ++rt) {
          const f32x4_t eq = coef4(coef, kEnterQ, rt), ek = coef4(coef, kEnterK, rt);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int step = 16 * rt + 4 * g + i;
            const bool in = whole || (step >= s && step < e);
            X[rt][i] = in ? dO[rt][i] * eq[i] : 0.0f;
            Y[rt][i] = in ? W[rt][i] * ek[i] : 0.0f;
          }
        }
        const Scale sx = col_scale(X), sy = col_scale(Y);
        f16x8_t xb[2][2], yb[2][2];
        to_operand<2>(X, sx.up, xb);
        to_operand<2>(Y, sy.up, yb);
        const float keep = a.keeps[ch];
#pragma unroll
        for (int kt = 0; kt < KT; ++kt) {
          f32x4_t x = kZero4, y = kZero4;
#pragma unroll
          for (int ks = 0; ks < 2; ++ks) {
            f16x8_t qa[NP], ka[NP];
#pragma unroll
            for (int p = 0; p < NP; ++p) {
              qa[p] = frag<KP>(qc, (p * KT + kt) * 2 + ks);
              ka[p] = frag<KP>(kc, (p * KT + kt) * 2 + ks);
              if (!whole) {
                qa[p] = keep_steps(qa[p], ks, s, e);
                ka[p] = keep_steps(ka[p], ks, s, e);
              }
            }
            x = mma_parts<NP, 2>(qa, xb[ks], x);
            y = mma_parts<NP, 2>(ka, yb[ks], y);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float add = x[i] * sx.down - y[i] * sy.down;
            S[kt][i] = e == kC ? __builtin_fmaf(keep, S[kt][i], add) : add;
          }
        }
      }
      e = s;
    }
  }
  if (a.grad_state0) store_state(a.grad_state0 + bh * sn);
}

// ---------------------------------------------------------------------------
// k_gdr_grads: one chunk of one head of q and k a workgroup, the heads that share them
// one after the other, so that their sums need no atomics.  Wave w has the steps 16 w...
// ---------------------------------------------------------------------------
// Sum over the 16 lanes of a row of an accumulator.
__device__ __forceinline__ float row16_sum(float v) {
#pragma unroll
  for (int d = 1; d < 16; d <<= 1) v += __shfl_xor(v, d);
  return v;
}

constexpr int kVB = 64;  // columns of V at a time

template <typename IO, int KP>
__global__ __launch_bounds__(256) void k_gdr_grads(GdrArgs a) {
  constexpr int NP = kParts<IO>, KS = KP / 32, KT = KP / 16;
  constexpr int kSet = NP * 4 * KS * kFrag;
  constexpr int kStates = 2 * KT * 4 * kFrag * 2, kMats = 2 * (int)sizeof(Mat);
  // fragments of S0 and dS, [row tile][32 columns][part]; then the matrices X and Z
  __shared__ __align__(16) char big[kStates > kMats ? kStates : kMats];
  __shared__ __align__(16) uint16_t df[16 * kFrag];  // of delta
  __shared__ float ro[kC], rw[kC], rd[kC], rs[KP], rg[KP], bt[kC], gam[kC], tail[kC], rkk[kC], rkq[kC];
  __shared__ float row_e[kC], col_e[4][kC], rx[kC], rz[kC], rt_s[kC], dots[4], tails[4], bsum[kC];
  __shared__ double gs[kC];
  uint16_t* sf = (uint16_t*)big;
  uint16_t* gf = sf + KT * 4 * kFrag;
  Mat& xm = *(Mat*)big;
  Mat& zm = *(Mat*)(big + sizeof(Mat));
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, g = lane >> 4, r = lane & 15;
  const int64_t kh = blockIdx.x;
  const int hk = (int)(kh % a.Hk), share = a.H / a.Hk;
  const int64_t cb = kh / a.Hk, b = cb % a.B, c = cb / a.B;
  const int64_t sn = (int64_t)a.K * a.V;
  const uint64_t cuts = a.cuts[cb];
  const bool enters = !(cuts & 1), whole = cuts == 0;
  const int first_end = seg_end(cuts, 0), last_start = seg_start(cuts, kC - 1);
  const uint16_t* kf = a.k_rows + kh * kSet;
  const uint16_t* qf = a.q_rows + kh * kSet;
  const uint16_t* kc = a.k_cols + kh * kSet;
  const uint16_t* qc = a.q_cols + kh * kSet;

  f32x4_t tq[KT], tk[KT];
#pragma unroll
  for (int kt = 0; kt < KT; ++kt) tq[kt] = tk[kt] = kZero4;

  for (int hh = 0; hh < share; ++hh) {
    const int h = hk * share + hh;
    const int64_t ch = cb * a.H + h;
    if (threadIdx.x < kC) {
      const int i = threadIdx.x;
      const float* coef = a.coef + ch * (kCoef * kC);
      gs[i] = a.decay_sums[ch * kC + i];
      bt[i] = coef[kBeta * kC + i];
      rkk[i] = coef[kRowKk * kC + i];
      rkq[i] = coef[kRowKq * kC + i];
      gam[i] = expf((float)gs[i]);
      tail[i] = expf((float)(a.decay_sums[ch * kC + kC - 1] - gs[i]));
    }
    f32x4_t dP[4], dL[4], Q1[KT], K1[KT], K2[KT];
#pragma unroll
    for (int i = 0; i < 4; ++i) dP[i] = dL[i] = kZero4;
#pragma unroll
    for (int i = 0; i < KT; ++i) Q1[i] = K1[i] = K2[i] = kZero4;
    float dbeta = 0.0f, dot = 0.0f;

    for (int v0 = 0; v0 < a.V; v0 += kVB) {
      f16x8_t oa[2][NP], wa[2][2], da[2][2];
      {
        const int row = 16 * w + r;
        const int64_t t = c * kC + row;
        float ov[16], wv[16], dv[16];
        const float* wr = a.w + (ch * kC + row) * a.Vp;
        const float* dr = a.delta + (ch * kC + row) * a.Vp;
        const IO* orow = (const IO*)a.grad_o + ((t * a.B + b) * a.H + h) * a.V;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int col = v0 + 32 * (j >> 1) + 8 * g + 4 * (j & 1);
          ld4(wr, col, a.V, wv + 4 * j);
          ld4(dr, col, a.V, dv + 4 * j);
          if (t < a.T) ld4(orow, col, a.V, ov + 4 * j);
          else ov[4 * j] = ov[4 * j + 1] = ov[4 * j + 2] = ov[4 * j + 3] = 0.0f;
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) dbeta = __builtin_fmaf(wv[j], dv[j], dbeta);
        const Scale so = scale_of(quad_max(top_of(ov))), sw = scale_of(quad_max(top_of(wv))),
                    sd = scale_of(quad_max(top_of(dv)));
#pragma unroll
        for (int vs = 0; vs < 2; ++vs) {
          const Split o2 = split8<NP == 2>(ov + 8 * vs, so.up), w2 = split8(wv + 8 * vs, sw.up),
                      d2 = split8(dv + 8 * vs, sd.up);
          oa[vs][0] = o2.hi;
          if constexpr (NP == 2) oa[vs][1] = o2.lo;
          wa[vs][0] = w2.hi;
          wa[vs][1] = w2.lo;
          da[vs][0] = d2.hi;
          da[vs][1] = d2.lo;
#pragma unroll
          for (int p = 0; p < 2; ++p)
            *reinterpret_cast<f16x8_t*>(df + ((w * 2 + vs) * 2 + p) * kFrag + lane * 8) = da[vs][p];
        }
        if (g == 0) {
          ro[row] = so.down;
          rw[row] = sw.down;
          rd[row] = sd.down;
        }
      }
      for (int kt = w; kt < KT; kt += 4) {
        const int k = 16 * kt + r;
        float s0[16], ds[16];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int col = v0 + 32 * (j >> 1) + 8 * g + 4 * (j & 1);
          const int n = k < a.K ? a.V : 0;
          ld4(a.checkpoints + ch * sn + (int64_t)k * a.V, col, enters ? n : 0, s0 + 4 * j);
          ld4(a.grad_states + ch * sn + (int64_t)k * a.V, col, n, ds + 4 * j);
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) dot = __builtin_fmaf(s0[j], ds[j], dot);
        const Scale ss = scale_of(quad_max(top_of(s0))), sg = scale_of(quad_max(top_of(ds)));
#pragma unroll
        for (int vs = 0; vs < 2; ++vs) {
          const Split s2 = split8(s0 + 8 * vs, ss.up), g2 = split8(ds + 8 * vs, sg.up);
          const int at = (kt * 2 + vs) * 2 * kFrag + lane * 8;
          *reinterpret_cast<f16x8_t*>(sf + at) = s2.hi;
          *reinterpret_cast<f16x8_t*>(sf + at + kFrag) = s2.lo;
          *reinterpret_cast<f16x8_t*>(gf + at) = g2.hi;
          *reinterpret_cast<f16x8_t*>(gf + at + kFrag) = g2.lo;
        }
        if (g == 0) {
          rs[k] = ss.down;
          rg[k] = sg.down;
        }
      }
      __syncthreads();
      const f32x4_t fo = *reinterpret_cast<const f32x4_t*>(ro + 16 * w + 4 * g);
      const f32x4_t fw = *reinterpret_cast<const f32x4_t*>(rw + 16 * w + 4 * g);
      const f32x4_t fd = *reinterpret_cast<const f32x4_t*>(rd + 16 * w + 4 * g);
#pragma unroll
      for (int ct = 0; ct < 4; ++ct) {
        if (ct > w) continue;
        f32x4_t x = kZero4, y = kZero4;
#pragma unroll
        for (int vs = 0; vs < 2; ++vs) {
          const f16x8_t db[2] = {frag<KP>(df, (ct * 2 + vs) * 2), frag<KP>(df, (ct * 2 + vs) * 2 + 1)};
          x = mma_parts<NP, 2>(oa[vs], db, x);
          y = mma_parts<2, 2>(wa[vs], db, y);
        }
        const float f = rd[16 * ct + r];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          dP[ct][i] = __builtin_fmaf(x[i], fo[i] * f, dP[ct][i]);
          dL[ct][i] = __builtin_fmaf(y[i], fw[i] * f, dL[ct][i]);
        }
      }
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) {
        f32x4_t x = kZero4, y = kZero4, z = kZero4;
#pragma unroll
        for (int vs = 0; vs < 2; ++vs) {
          const int at = (kt * 2 + vs) * 2;
          if (enters) {
            const f16x8_t sb[2] = {frag<KP>(sf, at), frag<KP>(sf, at + 1)};
            x = mma_parts<NP, 2>(oa[vs], sb, x);
            y = mma_parts<2, 2>(wa[vs], sb, y);
          }
          const f16x8_t gb[2] = {frag<KP>(gf, at), frag<KP>(gf, at + 1)};
          z = mma_parts<2, 2>(da[vs], gb, z);
        }
        const float f = rs[16 * kt + r], fz = rg[16 * kt + r];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          Q1[kt][i] = __builtin_fmaf(x[i], fo[i] * f, Q1[kt][i]);
          K1[kt][i] = __builtin_fmaf(y[i], fw[i] * f, K1[kt][i]);
          K2[kt][i] = __builtin_fmaf(z[i], fd[i] * fz, K2[kt][i]);
        }
      }
      __syncthreads();
    }

    // the rows' factors; what their segment does not reach is 0, whatever it holds
    float dq_q[4], dk_k[4], dk_t[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = 16 * w + 4 * g + i;
      const int64_t t = c * kC + row;
      const bool first = enters && row < first_end, last = row >= last_start;
      const float fq = gam[row] * a.scale, fk = -gam[row] * bt[row], ft = tail[row] * bt[row];
      float s1 = 0.0f, s2 = 0.0f, s3 = 0.0f;
      const IO* qp = (const IO*)a.q + (t * a.B + b) * a.ld_q + (int64_t)hk * a.K;
      const IO* kp = (const IO*)a.k + (t * a.B + b) * a.ld_k + (int64_t)hk * a.K;
#pragma unroll
      for (int kt = 0; kt < KT; ++kt) {
        Q1[kt][i] = first ? Q1[kt][i] * fq : 0.0f;
        K1[kt][i] = first ? K1[kt][i] * fk : 0.0f;
        K2[kt][i] = last ? K2[kt][i] * ft : 0.0f;
        const int k = 16 * kt + r;
        if (t < a.T && k < a.K) {
          const float qv = io_ld(qp, k), kv = io_ld(kp, k);
          s1 = __builtin_fmaf(qv, Q1[kt][i], s1);
          s2 = __builtin_fmaf(kv, K1[kt][i], s2);
          s3 = last ? __builtin_fmaf(kv, K2[kt][i], s3) : 0.0f;
        }
      }
      dq_q[i] = row16_sum(s1);
      dk_k[i] = row16_sum(s2);
      dk_t[i] = row16_sum(s3);
    }

    // X = dP D, Z = dL D and its transpose, and what the decay sums take from both
    float re[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int ct = 0; ct < 4; ++ct) {
      f32x4_t kk = kZero4, qk = kZero4;
      if (ct <= w) {
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          f16x8_t ka[NP], qa[NP], kb[NP];
#pragma unroll
          for (int p = 0; p < NP; ++p) {
            ka[p] = frag<KP>(kf, (p * 4 + w) * KS + ks);
            qa[p] = frag<KP>(qf, (p * 4 + w) * KS + ks);
            kb[p] = frag<KP>(kf, (p * 4 + ct) * KS + ks);
          }
          kk = mma_parts<NP, NP>(ka, kb, kk);
          qk = mma_parts<NP, NP>(qa, kb, qk);
        }
      }
      const int cj = 16 * ct + r;
      float ce = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int ri = 16 * w + 4 * g + i;
        float x = 0.0f, z = 0.0f;
        if (cj <= ri && cj >= seg_start(cuts, ri)) {
          const float d = expf((float)(gs[ri] - gs[cj]));
          x = dP[ct][i] * (a.scale * bt[cj]) * d;
          float en = x * qk[i] * (rkq[ri] * rkk[cj]);
          if (cj < ri) {
            z = -dL[ct][i] * (bt[ri] * bt[cj]) * d;
            en = __builtin_fmaf(z, kk[i] * (rkk[ri] * rkk[cj]), en);
          }
          re[i] += en;
          ce += en;
        }
        xm[ri][cj] = x;
        if (cj < ri) zm[ri][cj] = zm[cj][ri] = z;
        if (cj == ri) zm[ri][ri] = 0.0f;
      }
      ce += __shfl_xor(ce, 16);
      ce += __shfl_xor(ce, 32);
      if (g == 0) col_e[w][cj] = ce;
    }
    float tsum = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float e = row16_sum(re[i]);
      if (r == 0) row_e[16 * w + 4 * g + i] = e + dq_q[i] + dk_k[i] - dk_t[i];
      tsum += dk_t[i];
    }
    tsum += __shfl_xor(tsum, 16);
    tsum += __shfl_xor(tsum, 32);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) dot += __shfl_xor(dot, d);
    dbeta += __shfl_xor(dbeta, 16);
    dbeta += __shfl_xor(dbeta, 32);
    if (g == 0) bsum[16 * w + r] = dbeta;
    if (lane == 0) {
      tails[w] = tsum;
      dots[w] = dot;
    }
    __syncthreads();

    if (w == 0) {
      // dlog_decay_t = sum of dG_i over the steps i >= t of its segment
      double G = (double)row_e[lane] -
                 ((((double)col_e[0][lane] + col_e[1][lane]) + col_e[2][lane]) + col_e[3][lane]);
      const int end = seg_end(cuts, lane);
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const double after = __shfl_down(G, d);
        if (lane + d < end) G += after;
      }
      if (end == kC) {
        G += (((double)tails[0] + tails[1]) + tails[2]) + tails[3];
        if (whole)
          G += (double)gam[kC - 1] * ((((double)dots[0] + dots[1]) + dots[2]) + dots[3]);
      }
      const int64_t t = c * kC + lane;
      if (t < a.T) {
        const bool cut = (cuts >> lane) & 1;
        a.grad_log_decay[(t * a.B + b) * a.H + h] = cut ? 0.0f : (float)G;
        a.grad_beta[(t * a.B + b) * a.H + h] = bsum[lane];
      }
    }

    // dq += X k, dk += Z k + X^T q
    {
      const int row = 16 * w + r;
      float xv[16], zv[16], tv[16];
#pragma unroll
      for (int ks = 0; ks < 2; ++ks)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int col = 32 * ks + 16 * (j >> 2) + 4 * g + (j & 3);
          xv[8 * ks + j] = xm[row][col] * rkk[col];
          zv[8 * ks + j] = zm[row][col] * rkk[col];
          tv[8 * ks + j] = xm[col][row] * rkq[col];
        }
      if (!whole) {  // a factor that is not finite belongs to its own segment
        const int s = seg_start(cuts, row), e = seg_end(cuts, row);
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int col = 32 * ks + 16 * (j >> 2) + 4 * g + (j & 3);
            if (col < s || col >= e) xv[8 * ks + j] = zv[8 * ks + j] = tv[8 * ks + j] = 0.0f;
          }
      }
      const Scale sx = scale_of(quad_max(top_of(xv))), sz = scale_of(quad_max(top_of(zv))),
                  st = scale_of(quad_max(top_of(tv)));
      if (g == 0) {
        rx[row] = sx.down;
        rz[row] = sz.down;
        rt_s[row] = st.down;
      }
      f16x8_t xa[2][2], za[2][2], ta[2][2];
#pragma unroll
      for (int ks = 0; ks < 2; ++ks) {
        const Split x2 = split8(xv + 8 * ks, sx.up), z2 = split8(zv + 8 * ks, sz.up),
                    t2 = split8(tv + 8 * ks, st.up);
        xa[ks][0] = x2.hi; xa[ks][1] = x2.lo;
        za[ks][0] = z2.hi; za[ks][1] = z2.lo;
        ta[ks][0] = t2.hi; ta[ks][1] = t2.lo;
      }
      __syncthreads();
      const f32x4_t fx = *reinterpret_cast<const f32x4_t*>(rx + 16 * w + 4 * g);
      const f32x4_t fz = *reinterpret_cast<const f32x4_t*>(rz + 16 * w + 4 * g);
      const f32x4_t ft = *reinterpret_cast<const f32x4_t*>(rt_s + 16 * w + 4 * g);
      for (int s = 0; s < kC;) {
        const int e = seg_end(cuts, s);
        if (e > 16 * w && s < 16 * w + 16) {
#pragma unroll
          for (int kt = 0; kt < KT; ++kt) {
            f32x4_t x = kZero4, y = kZero4, z = kZero4;
#pragma unroll
            for (int ks = 0; ks < 2; ++ks) {
              f16x8_t kb[NP], qb[NP];
#pragma unroll
              for (int p = 0; p < NP; ++p) {
                kb[p] = frag<KP>(kc, (p * KT + kt) * 2 + ks);
                qb[p] = frag<KP>(qc, (p * KT + kt) * 2 + ks);
                if (!whole) {
                  kb[p] = keep_steps(kb[p], ks, s, e);
                  qb[p] = keep_steps(qb[p], ks, s, e);
                }
              }
              x = mma_parts<2, NP>(xa[ks], kb, x);
              y = mma_parts<2, NP>(za[ks], kb, y);
              z = mma_parts<2, NP>(ta[ks], qb, z);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int ri = 16 * w + 4 * g + i;
              if (ri >= s && ri < e) {
                tq[kt][i] += __builtin_fmaf(x[i], fx[i], Q1[kt][i]);
                tk[kt][i] += (K1[kt][i] + K2[kt][i]) + __builtin_fmaf(z[i], ft[i], y[i] * fz[i]);
              }
            }
          }
        }
        s = e;
      }
      __syncthreads();
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int64_t t = c * kC + 16 * w + 4 * g + i;
    if (t >= a.T) continue;
    IO* qo = (IO*)a.grad_q + (t * a.B + b) * a.ld_gq + (int64_t)hk * a.K;
    IO* ko = (IO*)a.grad_k + (t * a.B + b) * a.ld_gk + (int64_t)hk * a.K;
#pragma unroll
    for (int kt = 0; kt < KT; ++kt) {
      const int k = 16 * kt + r;
      if (k < a.K) {
        io_st(qo, k, tq[kt][i]);
        io_st(ko, k, tk[kt][i]);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// Single tokens: a workgroup has 128 columns of one head's state, a thread four columns of
// every eighth row, read once, kept in registers and written once.
// ---------------------------------------------------------------------------
template <typename IO, bool VEC>
__global__ __launch_bounds__(256) void k_gdr_step(GdrArgs a, const int32_t* __restrict__ slots,
                                                  float* state, int64_t nslots) {
  constexpr int kRows = 16;  // a thread: 128 rows
  __shared__ float ks[128], qs[128], red[8][128];
  const int vtiles = (a.V + 127) / 128;
  const int64_t id = blockIdx.x;
  const int vt = (int)(id % vtiles);
  const int64_t bh = id / vtiles, b = bh / a.H;
  const int h = (int)(bh % a.H), hk = h / (a.H / a.Hk);
  const int c4 = 4 * (threadIdx.x & 31), sub = threadIdx.x >> 5, col = 128 * vt + c4;
  const int64_t slot = slots ? slots[b] : b;
  IO* out = (IO*)a.o + (b * a.H + h) * (int64_t)a.V;
  if (slot < 0 || slot >= nslots) {  // idle
    if (sub == 0)
      for (int j = 0; j < 4; ++j)
        if (col + j < a.V) io_st(out, col + j, 0.0f);
    return;
  }
  float* S = state + (slot * a.H + h) * (int64_t)a.K * a.V;
  float s[kRows][4];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int k = 8 * i + sub;
    if (VEC && k < a.K && col < a.V) {
      const f32x4_t x = *reinterpret_cast<const f32x4_t*>(S + (int64_t)k * a.V + col);
      s[i][0] = x.x; s[i][1] = x.y; s[i][2] = x.z; s[i][3] = x.w;
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        s[i][j] = !VEC && k < a.K && col + j < a.V ? S[(int64_t)k * a.V + col + j] : 0.0f;
    }
  }
  {
    const int k = threadIdx.x & 127;
    const IO* p = threadIdx.x < 128 ? (const IO*)a.k + b * a.ld_k : (const IO*)a.q + b * a.ld_q;
    (threadIdx.x < 128 ? ks : qs)[k] = k < a.K ? io_ld(p, (int64_t)hk * a.K + k) : 0.0f;
  }
  const float decay = expf(a.log_decay[b * a.H + h]), beta = a.beta[b * a.H + h];
  __syncthreads();
  float m[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const float k = ks[8 * i + sub];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      s[i][j] *= decay;
      m[j] = __builtin_fmaf(k, s[i][j], m[j]);
    }
  }
  *reinterpret_cast<f32x4_t*>(&red[sub][c4]) = f32x4_t{m[0], m[1], m[2], m[3]};
  __syncthreads();
  float u[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float x = red[0][c4 + j];
#pragma unroll
    for (int i = 1; i < 8; ++i) x += red[i][c4 + j];
    const float v = col + j < a.V ? io_ld((const IO*)a.v, b * a.ld_v + (int64_t)h * a.V + col + j) : 0.0f;
    u[j] = beta * (v - x);
    m[j] = 0.0f;
  }
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int k = 8 * i + sub;
    const float kv = ks[k], qv = qs[k];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      s[i][j] = __builtin_fmaf(kv, u[j], s[i][j]);
      m[j] = __builtin_fmaf(qv, s[i][j], m[j]);
    }
    if (VEC && k < a.K && col < a.V) {
      *reinterpret_cast<f32x4_t*>(S + (int64_t)k * a.V + col) =
          f32x4_t{s[i][0], s[i][1], s[i][2], s[i][3]};
    } else if (!VEC && k < a.K) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (col + j < a.V) S[(int64_t)k * a.V + col + j] = s[i][j];
    }
  }
  __syncthreads();
  *reinterpret_cast<f32x4_t*>(&red[sub][c4]) = f32x4_t{m[0], m[1], m[2], m[3]};
  __syncthreads();
  if (threadIdx.x < 128 && 128 * vt + (int)threadIdx.x < a.V) {
    const int n = threadIdx.x;
    float x = red[0][n];
#pragma unroll
    for (int i = 1; i < 8; ++i) x += red[i][n];
    io_st(out, 128 * vt + n, x * a.scale);
  }
}

template <typename IO, int KP>
hipError_t gdr_fwd(const GdrArgs& a, hipStream_t stream) {
  const int64_t nc = (a.T + kC - 1) / kC, waves = a.B * a.H * ((a.V + 15) / 16);
  hipLaunchKernelGGL((k_gdr_prep<IO, KP, false>), dim3((unsigned)(nc * a.B * a.H)), dim3(256), 0,
                     stream, a);
  hipLaunchKernelGGL((k_gdr_chain<IO, KP, false>), dim3((unsigned)((waves + 3) / 4)), dim3(256), 0,
                     stream, a);
  return hipGetLastError();
}
template <typename IO, int KP>
hipError_t gdr_bwd(const GdrArgs& a, hipStream_t stream) {
  const int64_t nc = (a.T + kC - 1) / kC, waves = a.B * a.H * ((a.V + 15) / 16);
  hipLaunchKernelGGL((k_gdr_prep<IO, KP, true>), dim3((unsigned)(nc * a.B * a.H)), dim3(256), 0,
                     stream, a);
  hipLaunchKernelGGL((k_gdr_chain<IO, KP, true>), dim3((unsigned)((nc * waves + 3) / 4)), dim3(256),
                     0, stream, a);
  hipLaunchKernelGGL((k_gdr_back<IO, KP>), dim3((unsigned)((waves + 3) / 4)), dim3(256), 0, stream,
                     a);
  hipLaunchKernelGGL((k_gdr_grads<IO, KP>), dim3((unsigned)(nc * a.B * a.Hk)), dim3(256), 0, stream,
                     a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_gdr_fwd(const GdrArgs& a, int io, hipStream_t stream) {
  if (io == kIoBf16) return a.K <= 64 ? gdr_fwd<uint16_t, 64>(a, stream) : gdr_fwd<uint16_t, 128>(a, stream);
  return a.K <= 64 ? gdr_fwd<float, 64>(a, stream) : gdr_fwd<float, 128>(a, stream);
}
hipError_t launch_gdr_bwd(const GdrArgs& a, int io, hipStream_t stream) {
  if (io == kIoBf16) return a.K <= 64 ? gdr_bwd<uint16_t, 64>(a, stream) : gdr_bwd<uint16_t, 128>(a, stream);
  return a.K <= 64 ? gdr_bwd<float, 64>(a, stream) : gdr_bwd<float, 128>(a, stream);
}

hipError_t launch_gdr_step(const GdrArgs& a, int io, const int32_t* slots, float* state,
                           int64_t nslots, hipStream_t stream) {
  const dim3 grid((unsigned)(a.B * a.H * ((a.V + 127) / 128)));
  const bool vec = a.V % 4 == 0 && ((uintptr_t)state & 15) == 0;
#define LRS_GDR_STEP(IO, VEC) \
  hipLaunchKernelGGL((k_gdr_step<IO, VEC>), grid, dim3(256), 0, stream, a, slots, state, nslots)
  if (io == kIoBf16) {
    if (vec) LRS_GDR_STEP(uint16_t, true);
    else LRS_GDR_STEP(uint16_t, false);
  } else {
    if (vec) LRS_GDR_STEP(float, true);
    else LRS_GDR_STEP(float, false);
  }
#undef LRS_GDR_STEP
  return hipGetLastError();
}

}  // namespace lrs

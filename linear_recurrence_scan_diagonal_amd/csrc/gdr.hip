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
// The columns of S (and of V, R, delta, u, o) do not depend on each other: four waves walk
// the chunks of 16 or 32 columns, each with 32 rows of that piece of S in registers.
//   k_gdr_prep   every chunk at once: the [64,64] matrices D q k^T (P) and
//                T2 = (I + L diag(beta))^-1, and q, k and these as operands of the
//                matrix cores;
//   k_gdr_chain  the chain over the chunks, which leaves for the backward the state that
//                enters each of them and its delta;
//   k_gdr_back   the same chain in reverse, for dS: with do' = scale do
//                du = P^T do' + exp(G_C - G) K dS,  w = T^T du (T = (I + diag(beta) L)^-1),
//                dv = dR = beta w,  dS0 = exp(G_C) dS + (exp G q)^T do' - (exp G k)^T dR;
//   k_gdr_grads  every chunk at once, from S0, dS, delta and w: dbeta = w.delta,
//                dP = do' u^T, dL = -dR u^T and through them and the states dq, dk and
//                the decay's gradient.
// What bounds it.  The bytes of a long prompt take 40 us at 16384 steps of 16 heads (K = V =
// 128, bf16); it takes 103 us (prep) and 621 us (chain: 2.42 us a chunk, of which a wave
// issues for 0.7 us and waits for the others' barriers, LDS and the matrix cores else).
// Training at 2048 x 8 x 16 heads, 151 us of inputs and outputs, and 1.3 GB more of kept
// states and operands: prep 124 us in the forward and 126 in the backward, at two waves a SIMD
// for its LDS; chain 275 us and back 297, where a wave issues for 29 % of its time, is held up by
// the others' instructions for 32 and waits for 38; grads 477 us at two waves a SIMD (201
// registers), which issue for 28 % of their time and wait, for memory and the two barriers of
// every 32 columns, for 58.
// Two column blocks a wave and two waves a SIMD want more than 256 registers: of the chain
// 3 (bf16, K > 64) and 28 (fp32, K > 64) go to scratch, of back 15 (bf16, K > 64), 3 (bf16) and
// 21 (fp32, K <= 64).
//
// Restarts.  A chunk is taken apart into its documents' segments: the matrices are made
// and used a segment at a time, rows outside count as 0 by selection, never by a
// product, so that nothing of a document reaches another, NaN and infinities included.
// So each segment costs the work of a chunk, in prep and in both chains: 2048 x 8 x 16 heads
// bf16, forward / backward in us: without restarts 375 / 850, documents of 128 steps 425 / 950,
// of 32 589 / 1142, of 10 1042 / 1633, of 4 2038 / 2692, of one 6841 / 7758.
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
// An infinity counts as the largest finite binade: it stays what it is.
struct Scale {
  float up, down;
};
__device__ __forceinline__ Scale scale_of(float top) {
  uint32_t e = as_u32(top) >> 23;
  e = e < 15u ? 15u : e > 254u ? 254u : e;
  return {as_f32((268u - e) << 23), as_f32((e - 14u) << 23)};
}

// The largest absolute value over the four lanes that share a row or column (r = lane %
// 16).  A NaN does not count; it stays NaN at any scale.
__device__ __forceinline__ float quad_max(float m) {
  // not negative: whole numbers in the same order, without the instructions that make
  // signalling NaNs quiet
  const uint32_t u = as_u32(m);
  const u32x2_t a = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_permlane16_swap(u, u, false, false));
  const uint32_t v = a.x > a.y ? a.x : a.y;
  const u32x2_t b = __builtin_bit_cast(u32x2_t, __builtin_amdgcn_permlane32_swap(v, v, false, false));
  return as_f32(b.x > b.y ? b.x : b.y);
}
template <int N>
__device__ __forceinline__ float top_of(const float (&v)[N]) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i) m = fmaxf(m, fabsf(v[i]));
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

// Keeps the compiler from beginning the reads of what follows: it would begin them all and
// run out of registers.
__device__ __forceinline__ void fence() { __builtin_amdgcn_sched_barrier(0); }

constexpr f32x4_t kZero4 = {0.0f, 0.0f, 0.0f, 0.0f};

// `bytes` (below 2^31) of memory from a base that is the same for all lanes, at 32-bit
// offsets of the lanes' own: a load past the end gives 0 and a store there is dropped.
// The second offset is the same for all lanes, and inside the array.
struct Buffer {
  __amdgpu_buffer_rsrc_t r;
  __device__ __forceinline__ Buffer(const void* p, int64_t bytes)
      : r(__builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)(uint32_t)bytes, 0x00027000)) {}
  __device__ __forceinline__ u32x4_t load16(uint32_t at, int uniform) const {
    return __builtin_bit_cast(u32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, (int)at, uniform, 0));
  }
  __device__ __forceinline__ u32x2_t load8(uint32_t at) const {
    return __builtin_bit_cast(u32x2_t, __builtin_amdgcn_raw_buffer_load_b64(r, (int)at, 0, 0));
  }
  __device__ __forceinline__ void load(uint32_t at, float& v) const {
    v = as_f32((uint32_t)__builtin_amdgcn_raw_buffer_load_b32(r, (int)at, 0, 0));
  }
  __device__ __forceinline__ void load(uint32_t at, uint16_t& v) const {
    v = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(r, (int)at, 0, 0);
  }
  __device__ __forceinline__ void store(uint32_t at, float v, const float*) const {
    __builtin_amdgcn_raw_buffer_store_b32(as_u32(v), r, (int)at, 0, 0);
  }
  __device__ __forceinline__ void store(uint32_t at, float v, const uint16_t*) const {
    __builtin_amdgcn_raw_buffer_store_b16((short)(pack_bf16x2(v, 0.0f) & 0xFFFFu), r, (int)at, 0, 0);
  }
};

constexpr uint32_t kNowhere = 0x80000000u;  // past the end of any array here

// Four neighbouring elements as they are in memory: a conversion would wait for them.
template <typename IO>
struct Quad;
template <>
struct Quad<float> {
  u32x4_t q;
  __device__ __forceinline__ void get(float* v) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = as_f32(q[j]);
  }
};
template <>
struct Quad<uint16_t> {
  u32x2_t q;
  __device__ __forceinline__ void get(float* v) const {
    v[0] = bf16_lo(q.x); v[1] = bf16_hi(q.x); v[2] = bf16_lo(q.y); v[3] = bf16_hi(q.y);
  }
};
// Elements c..c+3 of a row of n that begins at byte `row` of the buffer; 0 from n on and
// in rows that are not there.  VEC: n is a multiple of four and the rows are aligned to it.
template <bool VEC>
__device__ __forceinline__ void ld_quad(const Buffer& b, uint32_t row, bool there, int c, int n,
                                        Quad<float>& q) {
  if constexpr (VEC) {
    q.q = b.load16(there && c < n ? row + (uint32_t)c * 4u : kNowhere, 0);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float v;
      b.load(there && c + j < n ? row + (uint32_t)(c + j) * 4u : kNowhere, v);
      q.q[j] = as_u32(v);
    }
  }
}
template <bool VEC>
__device__ __forceinline__ void ld_quad(const Buffer& b, uint32_t row, bool there, int c, int n,
                                        Quad<uint16_t>& q) {
  if constexpr (VEC) {
    q.q = b.load8(there && c < n ? row + (uint32_t)c * 2u : kNowhere);
  } else {
    uint16_t v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) b.load(there && c + j < n ? row + (uint32_t)(c + j) * 2u : kNowhere, v[j]);
    q.q = u32x2_t{(uint32_t)v[0] | (uint32_t)v[1] << 16, (uint32_t)v[2] | (uint32_t)v[3] << 16};
  }
}
// Whether rows of n elements, ld apart from p on, can be read in fours.
template <typename IO>
__host__ __device__ __forceinline__ bool quads(const void* p, int64_t ld, int n) {
  return ((ld | n) & 3) == 0 && ((uintptr_t)p & (4 * sizeof(IO) - 1)) == 0;
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

// Elements from row to row of the states and vectors that are kept in fp32: V in fours.
__host__ __device__ __forceinline__ int64_t saved_pitch(int64_t V) { return gdr_saved_pitch(V); }

// ---------------------------------------------------------------------------
// Workspace of a call, in arrays of chunk-heads: index (c B + b) Hk + hk, or with H, h.
// ---------------------------------------------------------------------------
// fp32 values a step that k_gdr_prep leaves, [chunk-head][kCoef][64]
enum { kEnterK, kEnterQ, kLeaveK, kBeta, kRowP, kRowT, kRowKq, kRowKk, kCoef };
constexpr int kStagedCoefs = kRowT + 1;


__device__ __forceinline__ f16x8_t frag(const uint16_t* base, int index) {
  return *reinterpret_cast<const f16x8_t*>(base + index * kFrag + (threadIdx.x & 63) * 8);
}
// Of a triangular [64,64] matrix six fragments are not all zeros: row tile rt has the
// k steps 0..rt/2, and where the matrix is transposed rt/2..1.
constexpr int kTri = 6;
constexpr int kTriSet = 2 * kTri * kFrag;  // in two parts
static_assert(kGdrMats == 2 * kTriSet + kCoef * kC * 2, "the workspace's");
template <bool TRANSPOSED>
__device__ __forceinline__ constexpr int tri(int rt, int ks) {
  return TRANSPOSED ? (rt < 2 ? 2 * rt + ks : rt + 2) : (rt < 2 ? rt : 2 * rt - 2 + ks);
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
// its largest; 4 waves, 16 rows each.  dst: [part][kTri][512].
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
    if (TRANSPOSED ? ks < w / 2 : ks > w / 2) continue;
    const Split p = split8(v + 8 * ks, sc.up);
    uint16_t* to = dst + tri<TRANSPOSED>(w, ks) * kFrag + lane * 8;
    *reinterpret_cast<f16x8_t*>(to) = p.hi;
    *reinterpret_cast<f16x8_t*>(to + kTri * kFrag) = p.lo;
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

  // 16 rows of k and q a wave
  const int row = 16 * w + r;
  const int64_t left = a.T - c * kC;
  auto load = [&](const IO* base, int64_t ld, Quad<IO> (&v)[2 * KS]) __attribute__((always_inline)) {
    const IO* p = base + ((c * kC * a.B + b) * ld + (int64_t)hk * a.K);
    const int64_t pitch = a.B * ld, n = left < kC ? left : kC;
    const Buffer buf(p, ((n - 1) * pitch + a.K) * (int64_t)sizeof(IO));
    const bool vec = quads<IO>(base, ld, a.K);
    const uint32_t at = (uint32_t)row * (uint32_t)pitch * (uint32_t)sizeof(IO);
    if (vec) {
#pragma unroll
      for (int j = 0; j < 2 * KS; ++j) ld_quad<true>(buf, at, row < n, 16 * j + 4 * g, a.K, v[j]);
    } else {
#pragma unroll
      for (int j = 0; j < 2 * KS; ++j) ld_quad<false>(buf, at, row < n, 16 * j + 4 * g, a.K, v[j]);
    }
  };
  Quad<IO> kraw[2 * KS], qraw[2 * KS];
  load((const IO*)a.k, a.ld_k, kraw);
  load((const IO*)a.q, a.ld_q, qraw);
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
  float kv[KP / 4], qv[KP / 4];
#pragma unroll
  for (int j = 0; j < 2 * KS; ++j) {
    kraw[j].get(kv + 4 * j);
    qraw[j].get(qv + 4 * j);
  }
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

  // the heads that share k and q leave them once
  if (h % share == 0) {
    constexpr int kSet = NP * 4 * KS * kFrag;
    uint16_t* to = a.kq_rows + kh * (2 * kSet);
    for (int i = threadIdx.x; i < kSet / 8; i += 256) {
      *reinterpret_cast<f16x8_t*>(to + i * 8) = *reinterpret_cast<const f16x8_t*>(&kf[0][0] + i * 8);
      *reinterpret_cast<f16x8_t*>(to + kSet + i * 8) =
          *reinterpret_cast<const f16x8_t*>(&qf[0][0] + i * 8);
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
  float* coef = (float*)(a.mats + ch * kGdrMats + 2 * kTriSet);
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
  uint16_t* tf = a.mats + ch * kGdrMats;
  uint16_t* pf = tf + kTriSet;
  for (int s = 0; s < kC;) {
    const int e = seg_end(cuts, s);
    // P, and L diag(beta), for the backward diag(beta) L
#pragma unroll
    for (int ct = 0; ct < 4; ++ct)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int ri = 16 * w + 4 * g + i, cj = 16 * ct + r;
        const bool in = cj <= ri && cj >= s && ri < e;
        const float d = in ? expf((float)(gs[ri] - gs[cj])) * rk[cj] : 0.0f;
        tm[ri][cj] = in ? qk[ct][i] * rq[ri] * d : 0.0f;
        am[ri][cj] = in && cj < ri ? kk[ct][i] * rk[ri] * d * bt[BWD ? ri : cj] : 0.0f;
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
    emit<BWD>(tm, tf, coef + kRowT * kC, s, e);
    __syncthreads();
    s = e;
  }
}

// ---------------------------------------------------------------------------
// The chains.  A wave has 16 columns; the four lanes of a column hold its rows.
// ---------------------------------------------------------------------------

// A column's largest value over the four lanes that hold it, as its scale.
template <int N>
__device__ __forceinline__ Scale col_scale(const f32x4_t (&v)[N]) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < N; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) m = fmaxf(m, fabsf(v[i][j]));
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

// One chunk's operands: in registers on their way from memory, then in LDS for all waves
// of the workgroup: k, q, T2 (or, transposed, T), P and the steps' coefficients.
template <int NP, int KS, int NT>
struct Stage {
  static constexpr int kSet = NP * 4 * KS * kFrag;  // values of k or of q
  static constexpr int kMats = 2 * kTriSet + kStagedCoefs * kC * 2;
  static constexpr int kBytes = (2 * kSet + kMats) * 2;
  static constexpr int NQ = 2 * kSet / 8 / NT, NM = (kMats / 8 + NT - 1) / NT;
  static_assert(NQ * NT * 8 == 2 * kSet, "whole loads");
  u32x4_t kq[NQ], m[NM];
  __device__ __forceinline__ void fetch(const GdrArgs& a, int64_t cb, int h, int hk) {
    const int64_t ch = cb * a.H + h, kh = cb * a.Hk + hk;
    const uint32_t at = (threadIdx.x % NT) * 16u;
    const Buffer fq(a.kq_rows + kh * (2 * kSet), 4 * kSet), fm(a.mats + ch * kGdrMats, 2 * kMats);
#pragma unroll
    for (int i = 0; i < NQ; ++i) kq[i] = fq.load16(at, i * NT * 16);
#pragma unroll
    for (int i = 0; i < NM; ++i) m[i] = fm.load16(at + (uint32_t)(i * NT * 16), 0);
  }
  __device__ __forceinline__ void put(char* lds) const {
    u32x4_t* to = reinterpret_cast<u32x4_t*>(lds) + threadIdx.x % NT;
#pragma unroll
    for (int i = 0; i < NQ; ++i) to[i * NT] = kq[i];
    to += NQ * NT;
#pragma unroll
    for (int i = 0; i < NM; ++i)
      if ((i + 1) * NT <= kMats / 8 || (int)(threadIdx.x % NT) + i * NT < kMats / 8) to[i * NT] = m[i];
  }
};
// What a chunk's steps have in common.
struct Marks {
  u32x2_t cuts_v;  // the same for all lanes; read where they are used, so that the loads are
  float keep_v;    // not waited for here
  __device__ __forceinline__ void fetch(const GdrArgs& a, int64_t cb, int h) {
    cuts_v = Buffer(a.cuts + cb, 8).load8(0);
    Buffer(a.keeps + cb * a.H + h, 4).load(0, keep_v);
  }
  __device__ __forceinline__ float keep() const {
    return as_f32((uint32_t)__builtin_amdgcn_readfirstlane((int)as_u32(keep_v)));
  }
  __device__ __forceinline__ uint64_t cuts() const {
    return (uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane(cuts_v.y) << 32 |
           (uint32_t)__builtin_amdgcn_readfirstlane(cuts_v.x);
  }
};
// A fragment of k^T or q^T (row tile kt of K, steps 32 ks...) from their rows in LDS: the
// transposing read gives each of 16 lanes one column of the four rows that they address
// together, eight bytes a lane.
template <int KS>
__device__ __forceinline__ f16x8_t cols(const uint16_t* rows, int part, int kt, int ks) {
  typedef short s16x4_t __attribute__((ext_vector_type(4)));
  typedef short s16x8_t __attribute__((ext_vector_type(8)));
  typedef __attribute__((address_space(3))) s16x4_t lds_t;
  const int lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
  const uint16_t* at = rows + ((part * 4 + 2 * ks) * KS + (kt >> 1)) * kFrag +
                       ((r & 3) * 16 + 4 * g + (r >> 2)) * 8 + 4 * (kt & 1);
  const s16x4_t lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_t*)at);
  const s16x4_t hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_t*)(at + KS * kFrag));
  return __builtin_bit_cast(f16x8_t, (s16x8_t)__builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7));
}

struct Yes {
  __device__ constexpr operator bool() const { return true; }
};
struct No {
  __device__ constexpr operator bool() const { return false; }
};

// What a chain's wave has.  A workgroup has NW * CB blocks of 16 columns of a head, and four
// waves for every CB of them; lane l has column r = l % 16 of each.  Wave j of the four has the
// steps 16 j... of a chunk, and the rows 32 j... of the state (where K <= 64: waves 0 and 1 alone).
// With two times four waves and one block a wave, the workgroup has one block in all: the
// first four walk the chain, and the others compute what the chain does not wait for.
template <int NW, int CB>
constexpr bool kHelped = NW == 2 && CB == 1;
// Then the helpers alone bring in the operands, into the other of two buffers, where LDS has
// room for two.
template <typename IO, int KP, int NW, int CB>
constexpr bool kTwo = kHelped<NW, CB> && (sizeof(IO) == 2 || KP == 64);
struct Wave {
  int64_t bh, b;
  int h, hk, j, block;  // block: the first one, in the workgroup
  int col;              // the lane's column of it
  bool walks;           // not a helper
  template <int NW, int CB>
  static __device__ __forceinline__ Wave make(const GdrArgs& a) {
    constexpr bool HELPED = kHelped<NW, CB>;
    constexpr int kCols = 16 * (HELPED ? 1 : NW) * CB;
    const uint32_t vblocks = (uint32_t)(a.V + kCols - 1) / kCols;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    Wave w;
    // workgroups go to the eight XCDs in turn: those of one head to the same, for its L2 cache
    const uint32_t x = blockIdx.x % 8, some = gridDim.x / 8, more = gridDim.x % 8;
    const uint32_t n = x * some + (x < more ? x : more) + blockIdx.x / 8;
    const uint32_t bh = n / vblocks;
    w.bh = bh;
    w.b = bh / (uint32_t)a.H;
    w.h = (int)(bh % (uint32_t)a.H);
    w.hk = w.h / (a.H / a.Hk);
    w.j = wave & 3;
    w.block = HELPED ? 0 : (wave >> 2) * CB;
    w.walks = !HELPED || wave < 4;
    w.col = (int)(n % vblocks) * kCols + w.block * 16 + (threadIdx.x & 15);
    return w;
  }
};

// 16 N rows of an array from row 16 t0 on, `pitch` elements apart: of rows 16 t + 4 g + 0..3
// the lane's column.  Rows from `rows` on read as 0 and are not written, nor are columns
// from `width` on.
template <typename IO>
struct Rows {
  Buffer buf;
  uint32_t pitch, lane;
  int t0;
  __device__ __forceinline__ Rows(const IO* p, int64_t pitch_, int64_t rows, int width, int col,
                                  int t0_)
      : buf(p, rows <= 0 ? 0 : ((rows - 1) * pitch_ + width) * (int64_t)sizeof(IO)), t0(t0_) {
    pitch = (uint32_t)pitch_ * (uint32_t)sizeof(IO);
    const uint32_t g = (threadIdx.x & 63) >> 4;
    lane = col < width ? 4u * g * pitch + (uint32_t)col * (uint32_t)sizeof(IO) : kNowhere;
  }
  __device__ __forceinline__ uint32_t at(int t, int i) const {
    return lane + (uint32_t)(16 * (t0 + t) + i) * pitch;
  }
  template <int N>
  __device__ __forceinline__ void load(IO (&v)[N][4]) const {
#pragma unroll
    for (int t = 0; t < N; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) buf.load(at(t, i), v[t][i]);
  }
  template <int N>
  __device__ __forceinline__ void store(const f32x4_t (&v)[N]) const {
#pragma unroll
    for (int t = 0; t < N; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) buf.store(at(t, i), v[t][i], (const IO*)nullptr);
  }
  // of one tile the rows [s, e) only
  __device__ __forceinline__ void store(const f32x4_t (&v)[1], int s, int e) const {
    const int g = (threadIdx.x & 63) >> 4;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = 16 * t0 + 4 * g + i;
      buf.store(row >= s && row < e ? at(0, i) : kNowhere, v[0][i], (const IO*)nullptr);
    }
  }
};
__device__ __forceinline__ float widen(float v) { return v; }
__device__ __forceinline__ float widen(uint16_t v) { return as_f32((uint32_t)v << 16); }
template <typename IO, int N>
__device__ __forceinline__ void widen(const IO (&v)[N][4], f32x4_t (&out)[N]) {
#pragma unroll
  for (int t = 0; t < N; ++t)
#pragma unroll
    for (int i = 0; i < 4; ++i) out[t][i] = widen(v[t][i]);
}

// What the four waves of a column block hand each other: the state as a right operand with
// a scale for every 32 rows, and the 64 steps of VECS vectors in fp32, 16 bytes a lane and
// wave.
template <int KS, int VECS>
struct Exchange {
  static constexpr int kState = KS * 2 * kFrag * 2, kVec = 4 * 64 * 16;
  static constexpr int kBytes = kState + kVec * VECS + KS * 16 * 4;
  char* base;
  __device__ __forceinline__ uint16_t* state(int ks, int part) const {
    return (uint16_t*)base + (ks * 2 + part) * kFrag + (threadIdx.x & 63) * 8;
  }
  __device__ __forceinline__ f32x4_t* vec(int which, int j) const {
    return (f32x4_t*)(base + kState + which * kVec) + j * 64 + (threadIdx.x & 63);
  }
  __device__ __forceinline__ float* down(int ks) const {
    return (float*)(base + kState + kVec * VECS) + ks * 16 + (threadIdx.x & 15);
  }
  // the wave's 32 rows of the state
  __device__ __forceinline__ void put_state(const f32x4_t (&S)[2], int j) const {
    const Scale sc = col_scale(S);
    f16x8_t b[1][2];
    to_operand<2>(S, sc.up, b);
    *reinterpret_cast<f16x8_t*>(state(j, 0)) = b[0][0];
    *reinterpret_cast<f16x8_t*>(state(j, 1)) = b[0][1];
    if ((threadIdx.x & 63) < 16) *down(j) = sc.down;
  }
  __device__ __forceinline__ void get_vec(int which, f32x4_t (&v)[4]) const {
#pragma unroll
    for (int t = 0; t < 4; ++t) v[t] = *vec(which, t);
  }
};

// 16 rows of k S, and of q S, for CB column blocks: a product for every 32 rows of the state,
// which have scales of their own.
template <int NP, int KS, int CB, bool BOTH, typename X>
__device__ __forceinline__ void times_state(const uint16_t* k_rows, const uint16_t* q_rows, int rt,
                                            const X (&x)[CB], f32x4_t (&k_out)[CB],
                                            f32x4_t (&q_out)[CB]) {
#pragma unroll
  for (int ks = 0; ks < KS; ++ks) {
    f16x8_t ka[NP], qa[NP];
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      ka[p] = frag(k_rows, (p * 4 + rt) * KS + ks);
      if (BOTH) qa[p] = frag(q_rows, (p * 4 + rt) * KS + ks);
    }
#pragma unroll
    for (int c = 0; c < CB; ++c) {
      const f16x8_t sb[2] = {*reinterpret_cast<const f16x8_t*>(x[c].state(ks, 0)),
                             *reinterpret_cast<const f16x8_t*>(x[c].state(ks, 1))};
      const float down = *x[c].down(ks);
      const f32x4_t y = mma_parts<NP, 2>(ka, sb, kZero4);
      f32x4_t z = kZero4;
      if (BOTH) z = mma_parts<NP, 2>(qa, sb, kZero4);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        k_out[c][i] = ks == 0 ? y[i] * down : __builtin_fmaf(y[i], down, k_out[c][i]);
        if (BOTH) q_out[c][i] = ks == 0 ? z[i] * down : __builtin_fmaf(z[i], down, q_out[c][i]);
      }
    }
    if (CB > 1) fence();
  }
}
// 16 rows of a triangular matrix times vectors' right operands.
template <bool TRANSPOSED, int CB, int PB>
__device__ __forceinline__ void times_tri(const uint16_t* m, int rt, const f16x8_t (&b)[CB][2][PB],
                                          f32x4_t (&x)[CB]) {
#pragma unroll
  for (int c = 0; c < CB; ++c) x[c] = kZero4;
#pragma unroll
  for (int ks = 0; ks < 2; ++ks) {
    if (TRANSPOSED ? ks < rt / 2 : ks > rt / 2) continue;
    const int f = tri<TRANSPOSED>(rt, ks);
    const f16x8_t ma[2] = {frag(m, f), frag(m, kTri + f)};
#pragma unroll
    for (int c = 0; c < CB; ++c) x[c] = mma_parts<2, PB>(ma, b[c][ks], x[c]);
  }
}
// 16 rows of k^T (or q^T) times vectors' right operands.
template <int NP, int KS, int CB, bool FULL>
__device__ __forceinline__ void times_cols(const uint16_t* rows, int kt, const f16x8_t (&b)[CB][2][2],
                                           int s, int e, f32x4_t (&x)[CB]) {
#pragma unroll
  for (int c = 0; c < CB; ++c) x[c] = kZero4;
#pragma unroll
  for (int ks = 0; ks < 2; ++ks) {
    f16x8_t ka[NP];
#pragma unroll
    for (int p = 0; p < NP; ++p) {
      ka[p] = cols<KS>(rows, p, kt, ks);
      if (!FULL) ka[p] = keep_steps(ka[p], ks, s, e);
    }
#pragma unroll
    for (int c = 0; c < CB; ++c) x[c] = mma_parts<NP, 2>(ka, b[c][ks], x[c]);
  }
}
template <int PARTS>
__device__ __forceinline__ float vec_operand(const f32x4_t (&v)[4], f16x8_t (&b)[2][PARTS]) {
  const Scale sc = col_scale(v);
  to_operand<PARTS>(v, sc.up, b);
  return sc.down;
}

// The chain over the chunks.  Between two barriers a wave makes 16 of a vector's 64 steps
// from the whole of the one before: R from the state, delta and u from R, the state's next
// value (32 rows) and o from u.
template <typename IO, int KP, int NW, int CB>
__global__ __launch_bounds__(256 * NW) void k_gdr_chain(GdrArgs a) {
  constexpr int NP = kParts<IO>, KS = KP / 32;
  constexpr bool HELPED = kHelped<NW, CB>, TWO = kTwo<IO, KP, NW, CB>;
  typedef Stage<NP, KS, TWO ? 256 : 256 * NW> St;
  typedef Exchange<KS, 2> X;
  constexpr int kOperands = St::kBytes * (TWO ? 2 : 1);
  __shared__ __align__(16) char lds[kOperands + (HELPED ? 1 : NW) * CB * X::kBytes];
  const int g = (threadIdx.x & 63) >> 4;
  const Wave w = Wave::make<NW, CB>(a);
  X x[CB];
#pragma unroll
  for (int c = 0; c < CB; ++c) x[c].base = lds + kOperands + (w.block + c) * X::kBytes;
  const int64_t nc = (a.T + kC - 1) / kC;
  const int64_t sn = (int64_t)a.K * a.V, vrow = (int64_t)a.H * a.V;
  const int vp = (int)saved_pitch(a.V);
  const int64_t cn = (int64_t)(a.K + kC) * vp;  // of a checkpoint

  auto run = [&](auto walks, auto helps) __attribute__((always_inline)) {
    constexpr bool WALKS = decltype(walks)(), HELPS = decltype(helps)();
    const bool owner = WALKS && w.j < KS;
    f32x4_t S[CB][2];
#pragma unroll
    for (int c = 0; c < CB; ++c) {
      float s0[2][4];
      Rows<float>(a.state0 + w.bh * sn, a.V, a.state0 && owner ? a.K : 0, a.V, w.col + 16 * c, 2 * w.j)
          .load(s0);
      widen(s0, S[c]);
      if (owner) x[c].put_state(S[c], w.j);
    }
    St st;
    IO nv[CB][1][4];  // the next chunk's v
    // (the address of a chunk behind the last is not read: a length of 0)
    auto fetch_v = [&](int64_t t) __attribute__((always_inline)) {
      const int64_t left = a.T - t * kC;
#pragma unroll
      for (int c = 0; c < CB; ++c)
        Rows<IO>((const IO*)a.v + (t * kC * a.B + w.b) * a.ld_v + (int64_t)w.h * a.V, a.B * a.ld_v,
                 left < kC ? left : kC, a.V, w.col + 16 * c, w.j)
            .load(nv[c]);
    };
    if (WALKS) fetch_v(0);
    Marks marks;
    auto fetch = [&](int64_t t) __attribute__((always_inline)) {
      st.fetch(a, (t < nc ? t : nc - 1) * a.B + w.b, w.h, w.hk);
    };
    marks.fetch(a, w.b, w.h);
    if (!TWO || !WALKS) fetch(0);
    if constexpr (TWO) {
      if (!WALKS) {
        st.put(lds);
        fetch(1);
      }
      __syncthreads();
    }
    for (int64_t t = 0; t < nc; ++t) {
      const int here = TWO && (t & 1) ? St::kBytes : 0;
      const uint16_t* kf = (const uint16_t*)(lds + here);
      const uint16_t* qf = kf + St::kSet;
      const uint16_t* tf = qf + St::kSet;
      const uint16_t* pf = tf + kTriSet;
      const float* coef = (const float*)(pf + kTriSet);
      if constexpr (!TWO) {
        st.put(lds);
        fetch(t + 1);
      }
      const uint64_t cuts = marks.cuts();
      const float keep = marks.keep();
      marks.fetch(a, (t + 1 < nc ? t + 1 : t) * a.B + w.b, w.h);
      const int64_t ch = (t * a.B + w.b) * a.H + w.h, left = a.T - t * kC;
      float* ck = a.checkpoints ? a.checkpoints + ch * cn : nullptr;
      if (ck && owner) {
#pragma unroll
        for (int c = 0; c < CB; ++c) Rows<float>(ck, vp, a.K, vp, w.col + 16 * c, 2 * w.j).store(S[c]);
      }
      if constexpr (!TWO) __syncthreads();
      f32x4_t R[CB][1];
      // The next chunk's v.  Two blocks have no registers for it before the first product.
      auto take_v = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int c = 0; c < CB; ++c) widen(nv[c], R[c]);
        fetch_v(t + 1);
      };
      if (WALKS && CB == 1) take_v();

      // The next chunk's operands, into the buffer that the chunk before has left; where o is
      // not yet written, as the loads are waited for in order with the stores.
      auto bring = [&]() __attribute__((always_inline)) {
        if constexpr (TWO && !WALKS) {
          st.put(lds + (St::kBytes - here));
          fetch(t + 2);
        }
      };

      // steps [s, e) of the chunk, v in R; FULL: all of them, of a document that goes on
      auto segment = [&](auto full, int s, int e, bool fresh) __attribute__((always_inline)) {
        constexpr bool FULL = decltype(full)();
        auto in = [&](int rt, int i) __attribute__((always_inline)) {
          const int step = 16 * rt + 4 * g + i;
          return FULL || (step >= s && step < e);
        };
        f32x4_t Q[CB][1], D[CB][1], V[4], y[CB], z[CB];
        // helpers have q S in y
        if (FULL || !fresh) times_state<NP, KS, CB, !HELPED>(WALKS ? kf : qf, qf, w.j, x, y, z);
        if (WALKS && CB > 1 && s == 0) take_v();
        {
          const f32x4_t ek = coef4(coef, kEnterK, w.j), eq = coef4(coef, kEnterQ, w.j);
#pragma unroll
          for (int c = 0; c < CB; ++c) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float d = R[c][0][i], q = 0.0f;
              if (FULL || !fresh) {
                d = __builtin_fmaf(-ek[i], y[c][i], d);
                q = eq[i] * (HELPED ? y : z)[c][i];
              }
              D[c][0][i] = in(w.j, i) ? d : 0.0f;
              Q[c][0][i] = q;
            }
            if (WALKS) *x[c].vec(0, w.j) = D[c][0];
          }
        }
        __syncthreads();
        if constexpr (FULL) bring();
        if (WALKS) {  // delta = T2 R, u = beta delta
          f16x8_t b[CB][2][2];
          float down[CB];
#pragma unroll
          for (int c = 0; c < CB; ++c) {
            x[c].get_vec(0, V);
            down[c] = vec_operand<2>(V, b[c]);
            if (CB > 1) fence();
          }
          times_tri<false, CB, 2>(tf, w.j, b, y);
          const f32x4_t rs = coef4(coef, kRowT, w.j), be = coef4(coef, kBeta, w.j);
#pragma unroll
          for (int c = 0; c < CB; ++c) {
#pragma unroll
            for (int i = 0; i < 4; ++i) D[c][0][i] = y[c][i] * (down[c] * rs[i]);
            if (ck) {
              const Rows<float> delta(ck + (int64_t)a.K * vp, vp, kC, vp, w.col + 16 * c, w.j);
              if (FULL) delta.store(D[c]);
              else delta.store(D[c], s, e);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) D[c][0][i] = in(w.j, i) ? D[c][0][i] * be[i] : 0.0f;
            *x[c].vec(1, w.j) = D[c][0];
          }
        }
        __syncthreads();
        // u for o, and for the state; two blocks read it twice, one at a time, to have the registers
        f16x8_t b[CB][2][2];
        float down[CB];
        if (CB == 1) {
          x[0].get_vec(1, V);
          if (HELPS) down[0] = vec_operand<2>(V, b[0]);
        }
        if (e == kC && owner) {  // the segment that leaves the chunk
          f16x8_t bl[CB][2][2];
          float downl[CB];
#pragma unroll
          for (int c = 0; c < CB; ++c) {
            if (CB > 1) x[c].get_vec(1, V);
#pragma unroll
            for (int rt = 0; rt < 4; ++rt) {
              const f32x4_t lv = coef4(coef, kLeaveK, rt);
#pragma unroll
              for (int i = 0; i < 4; ++i) V[rt][i] = in(rt, i) ? V[rt][i] * lv[i] : 0.0f;
            }
            downl[c] = vec_operand<2>(V, bl[c]);
            if (CB > 1) fence();
          }
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            times_cols<NP, KS, CB, FULL>(kf, 2 * w.j + k, bl, s, e, y);
#pragma unroll
            for (int c = 0; c < CB; ++c)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                S[c][k][i] = __builtin_fmaf(y[c][i], downl[c], !FULL && fresh ? 0.0f : keep * S[c][k][i]);
            if (CB > 1) fence();
          }
#pragma unroll
          for (int c = 0; c < CB; ++c) x[c].put_state(S[c], w.j);
          if (CB > 1) fence();
        }
        if (CB > 1) {
#pragma unroll
          for (int c = 0; c < CB; ++c) {
            x[c].get_vec(1, V);
            down[c] = vec_operand<2>(V, b[c]);
            fence();
          }
        }
        if (!HELPS) return;
        times_tri<false, CB, 2>(pf, w.j, b, y);
        const f32x4_t rs = coef4(coef, kRowP, w.j);
#pragma unroll
        for (int c = 0; c < CB; ++c) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            Q[c][0][i] = __builtin_fmaf(y[c][i], down[c] * (rs[i] * a.scale), Q[c][0][i]);
          const Rows<IO> out((const IO*)a.o + (t * kC * a.B + w.b) * vrow + (int64_t)w.h * a.V, a.B * vrow,
                             left < kC ? left : kC, a.V, w.col + 16 * c, w.j);
          if (FULL) out.store(Q[c]);
          else out.store(Q[c], s, e);
        }
      };
      if (cuts == 0) {
        segment(Yes(), 0, kC, false);
      } else {
#pragma unroll 1
        for (int s = 0; s < kC;) {
          const int e = seg_end(cuts, s);
          segment(No(), s, e, (cuts >> s) & 1);
          s = e;
        }
        bring();
      }
      __syncthreads();  // the next state and operands are there, and these may be written over
    }
    if (a.state && owner) {
#pragma unroll
      for (int c = 0; c < CB; ++c)
        Rows<float>(a.state + w.bh * sn, a.V, a.K, a.V, w.col + 16 * c, 2 * w.j).store(S[c]);
    }
  };
  // code of their own, with as many barriers
  if constexpr (!HELPED) run(Yes(), Yes());
  else if (w.walks) run(Yes(), No());
  else run(No(), Yes());
}

// The chain in reverse: dS, and w, dv and every chunk's dS on the way.
template <typename IO, int KP, int NW, int CB>
__global__ __launch_bounds__(256 * NW) void k_gdr_back(GdrArgs a) {
  constexpr int NP = kParts<IO>, KS = KP / 32;
  constexpr bool HELPED = kHelped<NW, CB>, TWO = kTwo<IO, KP, NW, CB>;
  typedef Stage<NP, KS, TWO ? 256 : 256 * NW> St;
  // with helpers also their part of du, and of dS: two vectors' room
  typedef Exchange<KS, HELPED ? 6 : 3> X;
  constexpr int kOperands = St::kBytes * (TWO ? 2 : 1);
  __shared__ __align__(16) char lds[kOperands + (HELPED ? 1 : NW) * CB * X::kBytes];
  const int g = (threadIdx.x & 63) >> 4;
  const Wave w = Wave::make<NW, CB>(a);
  X x[CB];
#pragma unroll
  for (int c = 0; c < CB; ++c) x[c].base = lds + kOperands + (w.block + c) * X::kBytes;
  const int64_t nc = (a.T + kC - 1) / kC;
  const int64_t sn = (int64_t)a.K * a.V, vrow = (int64_t)a.H * a.V;
  const int vp = (int)saved_pitch(a.V);

  auto run = [&](auto walks, auto helps) __attribute__((always_inline)) {
    constexpr bool WALKS = decltype(walks)(), HELPS = decltype(helps)();
    const bool owner = WALKS && w.j < KS;
    f32x4_t S[CB][2];  // dS
    IO ng[CB][1][4];   // the next chunk's grad_o
    auto fetch_o = [&](int64_t t) __attribute__((always_inline)) {
      const int64_t left = a.T - t * kC;
#pragma unroll
      for (int c = 0; c < CB; ++c)
        Rows<IO>((const IO*)a.grad_o + (t * kC * a.B + w.b) * vrow + (int64_t)w.h * a.V, a.B * vrow,
                 left < kC ? left : kC, a.V, w.col + 16 * c, w.j)
            .load(ng[c]);
    };
    auto put_o = [&]() __attribute__((always_inline)) {
#pragma unroll
      for (int c = 0; c < CB; ++c) {
        f32x4_t go[1];
        widen(ng[c], go);
        *x[c].vec(2, w.j) = go[0];
      }
    };
    St st;
    if (WALKS) fetch_o(nc - 1);
    Marks marks;
    auto fetch = [&](int64_t t) __attribute__((always_inline)) {
      st.fetch(a, (t > 0 ? t : 0) * a.B + w.b, w.h, w.hk);
    };
    marks.fetch(a, (nc - 1) * a.B + w.b, w.h);
    if (!TWO || !WALKS) fetch(nc - 1);
#pragma unroll
    for (int c = 0; c < CB; ++c) {
      float s0[2][4];
      Rows<float>(a.grad_state + w.bh * sn, a.V, a.grad_state && owner ? a.K : 0, a.V, w.col + 16 * c,
                  2 * w.j)
          .load(s0);
      widen(s0, S[c]);
      if (owner) x[c].put_state(S[c], w.j);
    }
    if (WALKS) put_o();
    if constexpr (TWO) {
      if (!WALKS) {
        st.put(lds + ((nc - 1) & 1) * St::kBytes);
        fetch(nc - 2);
      }
      __syncthreads();
    }
    for (int64_t t = nc - 1; t >= 0; --t) {
      const int here = TWO && (t & 1) ? St::kBytes : 0;
      const uint16_t* kf = (const uint16_t*)(lds + here);
      const uint16_t* qf = kf + St::kSet;
      const uint16_t* tf = qf + St::kSet;
      const uint16_t* pf = tf + kTriSet;
      const float* coef = (const float*)(pf + kTriSet);
      if constexpr (!TWO) st.put(lds);
      const uint64_t cuts = marks.cuts();
      const float keep = marks.keep();
      const int64_t next = t > 0 ? t - 1 : 0;
      if (WALKS) fetch_o(next);
      if constexpr (!TWO) fetch(next);
      marks.fetch(a, next * a.B + w.b, w.h);
      const int64_t ch = (t * a.B + w.b) * a.H + w.h, left = a.T - t * kC;
      if (owner) {
#pragma unroll
        for (int c = 0; c < CB; ++c)
          Rows<float>(a.grad_states + ch * a.K * vp, vp, a.K, vp, w.col + 16 * c, 2 * w.j).store(S[c]);
      }
      if constexpr (!TWO) __syncthreads();

      auto segment = [&](auto full, int s, int e, bool fresh) __attribute__((always_inline)) {
        constexpr bool FULL = decltype(full)();
        auto in = [&](int rt, int i) __attribute__((always_inline)) {
          const int step = 16 * rt + 4 * g + i;
          return FULL || (step >= s && step < e);
        };
        f32x4_t D[CB][1], dO[CB][4], V[4], y[CB], z[CB];
        if (HELPS) {  // du = scale P^T do + exp(G_C - G) K dS
          f16x8_t b[CB][2][NP];
          float down[CB];
#pragma unroll
          for (int c = 0; c < CB; ++c) {
            x[c].get_vec(2, dO[c]);
#pragma unroll
            for (int rt = 0; rt < 4; ++rt)
#pragma unroll
              for (int i = 0; i < 4; ++i) dO[c][rt][i] = in(rt, i) ? dO[c][rt][i] : 0.0f;
            down[c] = vec_operand<NP>(dO[c], b[c]);
            if (CB > 1) fence();
          }
          times_tri<true, CB, NP>(pf, w.j, b, y);
          const f32x4_t rs = coef4(coef, kRowP, w.j);
#pragma unroll
          for (int c = 0; c < CB; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i) D[c][0][i] = y[c][i] * (down[c] * (rs[i] * a.scale));
          if constexpr (HELPED) {
#pragma unroll
            for (int i = 0; i < 4; ++i) D[0][0][i] = in(w.j, i) ? D[0][0][i] : 0.0f;
            *x[0].vec(3, w.j) = D[0][0];
          }
        } else {
#pragma unroll
          for (int c = 0; c < CB; ++c) D[c][0] = kZero4;
        }
        if (WALKS && e == kC) {
          times_state<NP, KS, CB, false>(kf, nullptr, w.j, x, y, z);
          const f32x4_t lv = coef4(coef, kLeaveK, w.j);
#pragma unroll
          for (int c = 0; c < CB; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i) D[c][0][i] = __builtin_fmaf(y[c][i], lv[i], D[c][0][i]);
        }
#pragma unroll
        for (int c = 0; c < CB; ++c) {
#pragma unroll
          for (int i = 0; i < 4; ++i) D[c][0][i] = in(w.j, i) ? D[c][0][i] : 0.0f;
          if (WALKS) *x[c].vec(0, w.j) = D[c][0];
        }
        __syncthreads();
        if constexpr (HELPED) {
          if (!WALKS && w.j < KS && !(!FULL && fresh)) {  // (exp G q)^T do', 32 rows
            f16x8_t b[1][2][2];
#pragma unroll
            for (int rt = 0; rt < 4; ++rt) {
              const f32x4_t eq = coef4(coef, kEnterQ, rt);
#pragma unroll
              for (int i = 0; i < 4; ++i) dO[0][rt][i] = in(rt, i) ? dO[0][rt][i] * eq[i] : 0.0f;
            }
            const float down = vec_operand<2>(dO[0], b[0]);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              times_cols<NP, KS, 1, FULL>(qf, 2 * w.j + k, b, s, e, y);
              *x[0].vec(4 + k, w.j) = y[0] * down;
            }
          }
        }
        if (WALKS) {  // w = T^T du, dv = beta w
          f16x8_t b[CB][2][2];
          float down[CB];
#pragma unroll
          for (int c = 0; c < CB; ++c) {
            x[c].get_vec(0, V);
            if constexpr (HELPED) {
#pragma unroll
              for (int rt = 0; rt < 4; ++rt) V[rt] += *x[c].vec(3, rt);
            }
            down[c] = vec_operand<2>(V, b[c]);
            if (CB > 1) fence();
          }
          times_tri<true, CB, 2>(tf, w.j, b, y);
          const f32x4_t rs = coef4(coef, kRowT, w.j), be = coef4(coef, kBeta, w.j);
#pragma unroll
          for (int c = 0; c < CB; ++c) {
#pragma unroll
            for (int i = 0; i < 4; ++i) D[c][0][i] = y[c][i] * (down[c] * rs[i]);
            const Rows<float> wout(a.w + ch * kC * vp, vp, kC, vp, w.col + 16 * c, w.j);
            if (FULL) wout.store(D[c]);
            else wout.store(D[c], s, e);
#pragma unroll
            for (int i = 0; i < 4; ++i) D[c][0][i] = in(w.j, i) ? D[c][0][i] * be[i] : 0.0f;
            *x[c].vec(1, w.j) = D[c][0];
            const Rows<IO> vout((const IO*)a.grad_v + (t * kC * a.B + w.b) * a.ld_gv + (int64_t)w.h * a.V,
                                a.B * a.ld_gv, left < kC ? left : kC, a.V, w.col + 16 * c, w.j);
            if (FULL) vout.store(D[c]);
            else vout.store(D[c], s, e);
          }
        }
        __syncthreads();
        if (!owner) return;
        if (!FULL && fresh) {
#pragma unroll
          for (int c = 0; c < CB; ++c) S[c][0] = S[c][1] = kZero4;
          return;
        }
        // dS0 = exp(G_C) dS (of the last segment) + (exp G q)^T do' - (exp G k)^T dv
        f16x8_t xb[CB][2][2], yb[CB][2][2];
        float dx[CB], dy[CB];
#pragma unroll
        for (int c = 0; c < CB; ++c) {
          x[c].get_vec(1, V);
#pragma unroll
          for (int rt = 0; rt < 4; ++rt) {
            const f32x4_t eq = coef4(coef, kEnterQ, rt), ek = coef4(coef, kEnterK, rt);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              if (!HELPED) dO[c][rt][i] = in(rt, i) ? dO[c][rt][i] * eq[i] : 0.0f;
              V[rt][i] = in(rt, i) ? V[rt][i] * ek[i] : 0.0f;
            }
          }
          dx[c] = HELPED ? 1.0f : vec_operand<2>(dO[c], xb[c]);
          dy[c] = vec_operand<2>(V, yb[c]);
          if (CB > 1) fence();
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          if constexpr (HELPED) y[0] = *x[0].vec(4 + k, w.j);
          else times_cols<NP, KS, CB, FULL>(qf, 2 * w.j + k, xb, s, e, y);
          times_cols<NP, KS, CB, FULL>(kf, 2 * w.j + k, yb, s, e, z);
#pragma unroll
          for (int c = 0; c < CB; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              S[c][k][i] = __builtin_fmaf(y[c][i], dx[c],
                                          __builtin_fmaf(-z[c][i], dy[c],
                                                         FULL || e == kC ? keep * S[c][k][i] : 0.0f));
          if (CB > 1) fence();
        }
      };
      if (cuts == 0) {
        segment(Yes(), 0, kC, false);
      } else {
#pragma unroll 1
        for (int e = kC; e > 0;) {
          const int s = seg_start(cuts, e - 1);
          segment(No(), s, e, (cuts >> s) & 1);
          e = s;
        }
      }
      // the state was read before the chunk's first barrier, grad_o before its last segment's
      if (owner) {
#pragma unroll
        for (int c = 0; c < CB; ++c) x[c].put_state(S[c], w.j);
      }
      if (WALKS) put_o();
      if constexpr (TWO && !WALKS) {  // the chunk behind has left the other buffer
        st.put(lds + (St::kBytes - here));
        fetch(t - 2);
      }
      __syncthreads();  // the next state and operands are there, and these may be written over
    }
    if (a.grad_state0 && owner) {
#pragma unroll
      for (int c = 0; c < CB; ++c)
        Rows<float>(a.grad_state0 + w.bh * sn, a.V, a.K, a.V, w.col + 16 * c, 2 * w.j).store(S[c]);
    }
  };
  // code of their own, with as many barriers
  if constexpr (!HELPED) run(Yes(), Yes());
  else if (w.walks) run(Yes(), No());
  else run(No(), Yes());
}

// ---------------------------------------------------------------------------
// k_gdr_grads: one chunk of a head a workgroup.  Heads that share q and k leave their parts
// of dq and dk in fp32, and k_gdr_shared adds them up, in the heads' order.
// ---------------------------------------------------------------------------
// Sum over the 16 lanes of a row of an accumulator.
__device__ __forceinline__ float row16_sum(float v) {
#define LRS_ROR(N) \
  v += as_f32((uint32_t)__builtin_amdgcn_update_dpp(0, (int)as_u32(v), 0x120 + N, 0xf, 0xf, false))
  LRS_ROR(8);
  LRS_ROR(4);
  LRS_ROR(2);
  LRS_ROR(1);
#undef LRS_ROR
  return v;
}
__device__ __forceinline__ double row16_sum(double v) {
#define LRS_ROR(N)                                                                              \
  {                                                                                             \
    const u32x2_t u = __builtin_bit_cast(u32x2_t, v);                                           \
    const u32x2_t x = {(uint32_t)__builtin_amdgcn_update_dpp(0, (int)u.x, 0x120 + N, 0xf, 0xf, false), \
                       (uint32_t)__builtin_amdgcn_update_dpp(0, (int)u.y, 0x120 + N, 0xf, 0xf, false)}; \
    v += __builtin_bit_cast(double, x);                                                         \
  }
  LRS_ROR(8)
  LRS_ROR(4)
  LRS_ROR(2)
  LRS_ROR(1)
#undef LRS_ROR
  return v;
}

constexpr int kVB = 32;  // columns of V at a time

// Wave 4 x + j of the eight has the steps 16 j... and half x of the columns of its products.
// VEC: the rows of grad_o can be read in fours.
template <typename IO, int KP, bool VEC>
__global__ __launch_bounds__(512) void k_gdr_grads(GdrArgs a) {
  constexpr int NP = kParts<IO>, KS = KP / 32, KT = KP / 16, KH = KT / 2;
  constexpr int kSet = NP * 4 * KS * kFrag;
  // fragments of 32 columns of do, w, delta, S0 and dS; then the matrices X and Z, k and q
  constexpr int kBlock = (4 * NP + 16 + 4 * KT) * kFrag * 2, kMats = 2 * (int)sizeof(Mat) + 2 * kSet * 2;
  __shared__ __align__(16) char big[kBlock > kMats ? kBlock : kMats];
  __shared__ float ro[kC], rw[kC], rd[kC], rs[KP], rg[KP], bt[kC], gam[kC], tail[kC], rkk[kC], rkq[kC];
  __shared__ float row_t[2][kC], rx[kC], rz[kC], rt_s[kC], dots[8], bsum[kC];
  __shared__ double gs[kC], row_e[2][kC], col_e[4][kC];
  uint16_t* of = (uint16_t*)big;
  uint16_t* wf = of + 4 * NP * kFrag;
  uint16_t* df = wf + 8 * kFrag;
  uint16_t* sf = df + 8 * kFrag;
  uint16_t* gf = sf + 2 * KT * kFrag;
  Mat& xm = *(Mat*)big;
  Mat& zm = *(Mat*)(big + sizeof(Mat));
  uint16_t* kl = (uint16_t*)(big + 2 * sizeof(Mat));
  uint16_t* ql = kl + kSet;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int w = wv & 3, half = wv >> 2;
  const int lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
  const int64_t ch = blockIdx.x;
  const int h = (int)((uint32_t)ch % (uint32_t)a.H), hk = h / (a.H / a.Hk);
  const int64_t cb = (uint32_t)ch / (uint32_t)a.H, b = (uint32_t)cb % (uint32_t)a.B,
                c = (uint32_t)cb / (uint32_t)a.B, kh = cb * a.Hk + hk;
  const int vp = (int)saved_pitch(a.V);
  const int64_t sn = (int64_t)a.K * vp, cn = (int64_t)(a.K + kC) * vp;
  const int64_t left = a.T - c * kC, n = left < kC ? left : kC;
  const uint64_t cuts = a.cuts[cb];
  const bool enters = !(cuts & 1), whole = cuts == 0;
  const int first_end = seg_end(cuts, 0), last_start = seg_start(cuts, kC - 1);
  const uint16_t* kq = a.kq_rows + kh * (2 * kSet);

  if (threadIdx.x < kC) {
    const int i = threadIdx.x;
    const float* coef = (const float*)(a.mats + ch * kGdrMats + 2 * kTriSet);
    const double G = a.decay_sums[ch * kC + i], last = a.decay_sums[ch * kC + kC - 1];
    gs[i] = G;
    bt[i] = coef[kBeta * kC + i];
    rkk[i] = coef[kRowKk * kC + i];
    rkq[i] = coef[kRowKq * kC + i];
    gam[i] = expf((float)G);
    tail[i] = expf((float)(last - G));
  }
  f32x4_t dP[2], dL[2], Q1[KH], K1[KH], K2[KH];
  dP[0] = dP[1] = dL[0] = dL[1] = kZero4;
#pragma unroll
  for (int t = 0; t < KH; ++t) Q1[t] = K1[t] = K2[t] = kZero4;
  float dbeta = 0.0f, dot = 0.0f;

  const Buffer bs(a.checkpoints + ch * cn, cn * 4), bg(a.grad_states + ch * sn, sn * 4);
  const Buffer bw(a.w + ch * kC * vp, (int64_t)kC * vp * 4);
  const int64_t po = a.B * a.H * a.V;
  const Buffer bo((const IO*)a.grad_o + (c * kC * a.B + b) * a.H * a.V + (int64_t)h * a.V,
                  ((n - 1) * po + a.V) * (int64_t)sizeof(IO));
  // 16 rows x 32 columns as a fragment in two parts (column 8 g + e), scaled by row
  auto put = [&](const float (&v)[8], uint16_t* to, int parts, float* down, int row)
      __attribute__((always_inline)) {
    const Scale sc = scale_of(quad_max(top_of(v)));
    const Split p = split8(v, sc.up);
    *reinterpret_cast<f16x8_t*>(to + lane * 8) = p.hi;
    if (parts == 2) *reinterpret_cast<f16x8_t*>(to + kFrag + lane * 8) = p.lo;
    if (g == 0) down[row] = sc.down;
  };
  // the next 32 columns are in flight, as they are in memory
  Quad<float> s0[2], ds[2], wq[2], dq[2];
  Quad<IO> oq[2];
  const int row = 16 * w + r, k = 16 * wv + r;
  auto fetch = [&](int v0) __attribute__((always_inline)) {
    const int col = v0 + 8 * g;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if (wv < KT) {
        const uint32_t at = (uint32_t)k * (uint32_t)vp * 4u;
        ld_quad<true>(bs, at, enters && k < a.K, col + 4 * j, vp, s0[j]);
        ld_quad<true>(bg, at, k < a.K, col + 4 * j, vp, ds[j]);
      }
      if (half == 0) {
        ld_quad<VEC>(bo, (uint32_t)row * (uint32_t)po * (uint32_t)sizeof(IO), row < n, col + 4 * j,
                     a.V, oq[j]);
      } else {
        ld_quad<true>(bw, (uint32_t)row * (uint32_t)vp * 4u, true, col + 4 * j, vp, wq[j]);
        ld_quad<true>(bs, (uint32_t)(a.K + row) * (uint32_t)vp * 4u, true, col + 4 * j, vp, dq[j]);
      }
    }
  };
  fetch(0);
  for (int v0 = 0; v0 < a.V; v0 += kVB) {
    if (half == 0) {
      float v[8];
      oq[0].get(v);
      oq[1].get(v + 4);
      put(v, of + w * NP * kFrag, NP, ro, row);
    } else {
      float v[8], u[8];
      wq[0].get(v);
      wq[1].get(v + 4);
      dq[0].get(u);
      dq[1].get(u + 4);
#pragma unroll
      for (int j = 0; j < 8; ++j) dbeta = __builtin_fmaf(v[j], u[j], dbeta);
      put(v, wf + w * 2 * kFrag, 2, rw, row);
      put(u, df + w * 2 * kFrag, 2, rd, row);
    }
    if (wv < KT) {
      float v[8], u[8];
      s0[0].get(v);
      s0[1].get(v + 4);
      ds[0].get(u);
      ds[1].get(u + 4);
#pragma unroll
      for (int j = 0; j < 8; ++j) dot = __builtin_fmaf(v[j], u[j], dot);
      put(v, sf + wv * 2 * kFrag, 2, rs, k);
      put(u, gf + wv * 2 * kFrag, 2, rg, k);
    }
    if (v0 + kVB < a.V) fetch(v0 + kVB);
    __syncthreads();
    f16x8_t oa[NP], wa[2], da[2];
#pragma unroll
    for (int p = 0; p < NP; ++p) oa[p] = frag(of, w * NP + p);
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      wa[p] = frag(wf, w * 2 + p);
      da[p] = frag(df, w * 2 + p);
    }
    const f32x4_t fo = *reinterpret_cast<const f32x4_t*>(ro + 16 * w + 4 * g);
    const f32x4_t fw = *reinterpret_cast<const f32x4_t*>(rw + 16 * w + 4 * g);
    const f32x4_t fd = *reinterpret_cast<const f32x4_t*>(rd + 16 * w + 4 * g);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const int ct = 2 * half + t;
      if (ct > w) continue;
      const f16x8_t db[2] = {frag(df, ct * 2), frag(df, ct * 2 + 1)};
      const f32x4_t x = mma_parts<NP, 2>(oa, db, kZero4), y = mma_parts<2, 2>(wa, db, kZero4);
      const float f = rd[16 * ct + r];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        dP[t][i] = __builtin_fmaf(x[i], fo[i] * f, dP[t][i]);
        dL[t][i] = __builtin_fmaf(y[i], fw[i] * f, dL[t][i]);
      }
    }
    fence();
#pragma unroll
    for (int t = 0; t < KH; ++t) {
      const int kt = half * KH + t;
      const f16x8_t sb[2] = {frag(sf, kt * 2), frag(sf, kt * 2 + 1)};
      const f16x8_t gb[2] = {frag(gf, kt * 2), frag(gf, kt * 2 + 1)};
      const f32x4_t x = mma_parts<NP, 2>(oa, sb, kZero4), y = mma_parts<2, 2>(wa, sb, kZero4),
                    z = mma_parts<2, 2>(da, gb, kZero4);
      const float f = rs[16 * kt + r], fz = rg[16 * kt + r];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        Q1[t][i] = __builtin_fmaf(x[i], fo[i] * f, Q1[t][i]);
        K1[t][i] = __builtin_fmaf(y[i], fw[i] * f, K1[t][i]);
        K2[t][i] = __builtin_fmaf(z[i], fd[i] * fz, K2[t][i]);
      }
      fence();
    }
    __syncthreads();
  }
  for (int i = threadIdx.x; i < 2 * kSet / 8; i += 512)
    *reinterpret_cast<u32x4_t*>(kl + i * 8) = *reinterpret_cast<const u32x4_t*>(kq + i * 8);
  __syncthreads();

  // the rows' factors; what their segment does not reach is 0, whatever it holds
  double e_row[4];
  float e_tail[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int row = 16 * w + 4 * g + i;
    const bool first = enters && row < first_end, last = row >= last_start;
    const float fq = gam[row] * a.scale, fk = -gam[row] * bt[row], ft = tail[row] * bt[row];
    float s1 = 0.0f, s2 = 0.0f, s3 = 0.0f;
#pragma unroll
    for (int t = 0; t < KH; ++t) {
      Q1[t][i] = first ? Q1[t][i] * fq : 0.0f;
      K1[t][i] = first ? K1[t][i] * fk : 0.0f;
      K2[t][i] = last ? K2[t][i] * ft : 0.0f;
      const int kt = half * KH + t;
      float qv = 0.0f, kv = 0.0f;
#pragma unroll
      for (int p = 0; p < NP; ++p) {
        const int at = ((p * 4 + w) * KS + (kt >> 1)) * kFrag + ((r >> 2) * 16 + 4 * g + i) * 8 +
                       4 * (kt & 1) + (r & 3);
        qv += (float)__builtin_bit_cast(_Float16, ql[at]);
        kv += (float)__builtin_bit_cast(_Float16, kl[at]);
      }
      s1 = __builtin_fmaf(qv, Q1[t][i], s1);
      s2 = __builtin_fmaf(kv, K1[t][i], s2);
      s3 = __builtin_fmaf(kv, K2[t][i], s3);
    }
    // of this lane's columns; summed over the lanes below
    e_row[i] = s1 * rkq[row] + s2 * rkk[row];
    e_tail[i] = last ? s3 * rkk[row] : 0.0f;
    fence();
  }

  // X = dP D, Z = dL D and its transpose, and what the decay sums take from both: E_ij with the
  // factor exp(G_i - G_j).  Step t's gradient has the E_ij of j < t <= i, as the sum of the
  // rows minus the columns from t on; the others cancel, and may be larger by any power of e.
  // So both sums are in fp64, and the diagonal, which has no such factor, is in neither.
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const int ct = 2 * half + t;
    f32x4_t kk = kZero4, qk = kZero4;
    if (ct <= w) {
#pragma unroll
      for (int ks = 0; ks < KS; ++ks) {
        f16x8_t ka[NP], qa[NP], kb[NP];
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          ka[p] = frag(kl, (p * 4 + w) * KS + ks);
          qa[p] = frag(ql, (p * 4 + w) * KS + ks);
          kb[p] = frag(kl, (p * 4 + ct) * KS + ks);
        }
        kk = mma_parts<NP, NP>(ka, kb, kk);
        qk = mma_parts<NP, NP>(qa, kb, qk);
        if (ks & 1) fence();
      }
    }
    const int cj = 16 * ct + r;
    double ce = 0.0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int ri = 16 * w + 4 * g + i;
      // selected, not branched over: the exponential may be anything outside the segment
      const bool low = cj < ri && cj >= seg_start(cuts, ri);
      const float d = expf((float)(gs[ri] - gs[cj]));
      const float x = low || cj == ri ? dP[t][i] * (a.scale * bt[cj]) * (cj == ri ? 1.0f : d) : 0.0f;
      const float z = low ? -dL[t][i] * (bt[ri] * bt[cj]) * d : 0.0f;
      const float en = low ? __builtin_fmaf(z, kk[i] * (rkk[ri] * rkk[cj]),
                                            x * qk[i] * (rkq[ri] * rkk[cj])) : 0.0f;
      e_row[i] += (double)en;
      ce += (double)en;
      xm[ri][cj] = x;
      if (cj < ri) zm[ri][cj] = zm[cj][ri] = z;
      if (cj == ri) zm[ri][ri] = 0.0f;
    }
    ce += __shfl_xor(ce, 16);
    ce += __shfl_xor(ce, 32);
    if (g == 0) col_e[w][cj] = ce;
    fence();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    e_row[i] = row16_sum(e_row[i]);
    e_tail[i] = row16_sum(e_tail[i]);
    if (r == 0) {
      row_e[half][16 * w + 4 * g + i] = e_row[i];
      row_t[half][16 * w + 4 * g + i] = e_tail[i];
    }
  }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) dot += __shfl_xor(dot, d);
  if (half == 1) {
    dbeta += __shfl_xor(dbeta, 16);
    dbeta += __shfl_xor(dbeta, 32);
    if (g == 0) bsum[16 * w + r] = dbeta;
  }
  if (lane == 0) dots[wv] = dot;
  __syncthreads();

  if (wv == 0) {
    // dlog_decay_t = sum of dG_i over the steps i >= t of its segment, and of what its steps
    // before t leave for the chunks behind
    double G = (row_e[0][lane] + row_e[1][lane]) -
               (((col_e[0][lane] + col_e[1][lane]) + col_e[2][lane]) + col_e[3][lane]);
    double t = (double)row_t[0][lane] + row_t[1][lane];
    const int end = seg_end(cuts, lane);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const double after = __shfl_down(G, d), before = __shfl_up(t, d);
      if (lane + d < end) G += after;
      if (lane >= d) t += before;
    }
    const double left_behind = __shfl_up(t, 1);
    if (end == kC) {
      if (lane > 0) G += left_behind;
      if (whole) {
        double s = 0.0;
#pragma unroll
        for (int i = 0; i < 8; ++i) s += dots[i];
        G += (double)gam[kC - 1] * s;
      }
    }
    if (lane < n) {
      const bool cut = (cuts >> lane) & 1;
      const int64_t at = ((c * kC + lane) * a.B + b) * a.H + h;
      a.grad_log_decay[at] = cut ? 0.0f : (float)G;
      a.grad_beta[at] = bsum[lane];
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
    if (g == 0 && half == 0) {
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
    // rows of segment [s, e); FULL: all
    auto products = [&](auto full, int s, int e) __attribute__((always_inline)) {
      constexpr bool FULL = decltype(full)();
#pragma unroll
      for (int t = 0; t < KH; ++t) {
        const int kt = half * KH + t;
        f32x4_t x = kZero4, y = kZero4, z = kZero4;
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
          f16x8_t kb[NP], qb[NP];
#pragma unroll
          for (int p = 0; p < NP; ++p) {
            kb[p] = cols<KS>(kl, p, kt, ks);
            qb[p] = cols<KS>(ql, p, kt, ks);
            if (!FULL) {
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
          if (FULL || (ri >= s && ri < e)) {
            Q1[t][i] = __builtin_fmaf(x[i], fx[i], Q1[t][i]);
            K1[t][i] = (K1[t][i] + K2[t][i]) + __builtin_fmaf(z[i], ft[i], y[i] * fz[i]);
          }
        }
        fence();
      }
    };
    if (whole) {
      products(Yes(), 0, kC);
    } else {
#pragma unroll 1
      for (int s = 0; s < kC;) {
        const int e = seg_end(cuts, s);
        if (e > 16 * w && s < 16 * w + 16) products(No(), s, e);
        s = e;
      }
    }
  }

  // dq and dk: rows 16 w + 4 g + i, columns 16 (half KH + t) + r
  auto write = [&](const auto* to, int64_t pitch, const f32x4_t (&v)[KH]) __attribute__((always_inline)) {
    typedef decltype(to) P;
    constexpr uint32_t es = sizeof(*to);
    const Buffer buf(to, ((n - 1) * pitch + a.K) * (int64_t)es);
#pragma unroll
    for (int t = 0; t < KH; ++t) {
      const int col = 16 * (half * KH + t) + r;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int at = 16 * w + 4 * g + i;
        buf.store(at < n && col < a.K ? ((uint32_t)at * (uint32_t)pitch + (uint32_t)col) * es : kNowhere,
                  v[t][i], (P)nullptr);
      }
    }
  };
  if (a.shared) {
    const float* to = a.shared + ch * 2 * kC * a.K;
    write(to, a.K, Q1);
    write(to + kC * a.K, a.K, K1);
  } else {
    write((const IO*)a.grad_q + (c * kC * a.B + b) * a.ld_gq + (int64_t)hk * a.K, a.B * a.ld_gq, Q1);
    write((const IO*)a.grad_k + (c * kC * a.B + b) * a.ld_gk + (int64_t)hk * a.K, a.B * a.ld_gk, K1);
  }
}

// blockIdx.x: chunk, sequence and head of q and k; the sums over the heads that share them.
template <typename IO>
__global__ __launch_bounds__(256) void k_gdr_shared(GdrArgs a) {
  const uint32_t kh = blockIdx.x, hk = kh % (uint32_t)a.Hk, cb = kh / (uint32_t)a.Hk;
  const int64_t b = cb % (uint32_t)a.B, c = cb / (uint32_t)a.B;
  const int share = a.H / a.Hk;
  const int64_t left = a.T - c * kC;
  const int size = kC * a.K, rows = (int)(left < kC ? left : kC);
  const float* from = a.shared + ((int64_t)cb * a.H + (int64_t)hk * share) * 2 * size;
  for (int i = threadIdx.x; i < rows * a.K; i += 256) {
    float q = from[i], k = from[size + i];
    for (int s = 1; s < share; ++s) {
      q += from[(int64_t)s * 2 * size + i];
      k += from[(int64_t)s * 2 * size + size + i];
    }
    const int row = i / a.K, col = i - row * a.K;
    const int64_t at = (c * kC + row) * a.B + b;
    io_st((IO*)a.grad_q, at * a.ld_gq + (int64_t)hk * a.K + col, q);
    io_st((IO*)a.grad_k, at * a.ld_gk + (int64_t)hk * a.K + col, k);
  }
}

// ---------------------------------------------------------------------------
// Single tokens: a workgroup has 128 columns of one head's state, a thread four columns of
// every eighth row, read once, kept in registers and written once: 19.7 us for 128 MB of
// state read and written (6.9 TB/s; what the last call wrote is in part still in the
// memory-side cache).
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

// Column blocks of a chain's workgroup: one with helpers, for the shortest chunk, while every
// workgroup has a compute unit of its own, then two, then four (two a wave), which read a
// chunk's operands together and hide each other's waits.  Forward / backward of 1024 steps with K
// = V = 128, bf16, in us a call:
//   heads      one        two        four
//   32       64 / 126   95 / 165  108 / 189
//   64      110 / 238  107 / 250  119 / 268
//   96      160 / 356  191 / 412  133 / 353
//   128     212 / 483  206 / 493  150 / 433
//
// The backward follows the forward's rule; at 64 heads it would rather have one, by 5 %.
template <typename F>
void chain_shape(const GdrArgs& a, bool most_four, F launch) {
  const int64_t heads = a.B * a.H, cus = device_cus();
  const int n = heads * ((a.V + 15) / 16) <= cus ? 1 : heads * ((a.V + 31) / 32) <= cus || !most_four ? 2 : 4;
  launch(n, dim3((unsigned)(heads * ((a.V + 16 * n - 1) / (16 * n)))));
}

template <typename IO, int KP>
hipError_t gdr_fwd(const GdrArgs& a, hipStream_t stream) {
  const int64_t nc = (a.T + kC - 1) / kC;
  hipLaunchKernelGGL((k_gdr_prep<IO, KP, false>), dim3((unsigned)(nc * a.B * a.H)), dim3(256), 0,
                     stream, a);
  chain_shape(a, true, [&](int n, dim3 grid) {
    if (n == 4) hipLaunchKernelGGL((k_gdr_chain<IO, KP, 2, 2>), grid, dim3(512), 0, stream, a);
    else if (n == 2) hipLaunchKernelGGL((k_gdr_chain<IO, KP, 1, 2>), grid, dim3(256), 0, stream, a);
    else hipLaunchKernelGGL((k_gdr_chain<IO, KP, 2, 1>), grid, dim3(512), 0, stream, a);
  });
  return hipGetLastError();
}
template <typename IO, int KP>
hipError_t gdr_bwd(const GdrArgs& a, hipStream_t stream) {
  const int64_t nc = (a.T + kC - 1) / kC;
  // four blocks of fp32 with K > 64 do not fit into LDS
  constexpr bool kFour = sizeof(IO) == 2 || KP == 64;
  hipLaunchKernelGGL((k_gdr_prep<IO, KP, true>), dim3((unsigned)(nc * a.B * a.H)), dim3(256), 0,
                     stream, a);
  chain_shape(a, kFour, [&](int n, dim3 grid) {
    if (kFour && n == 4)
      hipLaunchKernelGGL((k_gdr_back<IO, KP, kFour ? 2 : 1, 2>), grid, dim3(512), 0, stream, a);
    else if (n == 2)
      hipLaunchKernelGGL((k_gdr_back<IO, KP, 1, 2>), grid, dim3(256), 0, stream, a);
    else
      hipLaunchKernelGGL((k_gdr_back<IO, KP, 2, 1>), grid, dim3(512), 0, stream, a);
  });
  const dim3 groups((unsigned)(nc * a.B * a.H));
  if (quads<IO>(a.grad_o, 0, a.V))
    hipLaunchKernelGGL((k_gdr_grads<IO, KP, true>), groups, dim3(512), 0, stream, a);
  else
    hipLaunchKernelGGL((k_gdr_grads<IO, KP, false>), groups, dim3(512), 0, stream, a);
  if (a.shared)
    hipLaunchKernelGGL((k_gdr_shared<IO>), dim3((unsigned)(nc * a.B * a.Hk)), dim3(256), 0, stream, a);
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

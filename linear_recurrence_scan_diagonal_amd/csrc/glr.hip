// glr.hip -- gated linear recurrence with a learned decay, [T, B, D] layout:
// forward, backward with recomputed states, and single tokens over a pool of
// states.
//
//   r = sigmoid(z_r + bias_r),  i = sigmoid(z_i + bias_i),
//   la = -c softplus(decay) r,  a = exp(la),  m = sqrt(1 - a^2) = sqrt(-expm1(2 la)),
//   h_t = a h_{t-1} + m i x;    a reset sets a = 0, m = 1.
//
// The recurrence is an affine map a step, so the tiles, the look-back and the
// persistent walk are those of the other [T, B, D] layers (lrs_tbd.hpp); the
// gates are evaluated once an element next to their loads.  With resets the
// maps compose through affine<true> and factor<true>, which let a factor of 0 replace
// the state rather than multiply it, next to any other factor, and keep the factors of a
// document from rounding to 0: a NaN or an infinity of one document stays there, a gate
// that is NaN included, and stays to its end.
//
// Inputs are rows of a wider projection (pitch ld): a lane's channels are at
// b * ld + d of a row, computed once a thread.  A lane has two channels, read as
// one pair (the caller has seen to it that pairs are aligned and do not cross
// two sequences), or one.
//
// The backward pass reads no h: the forward leaves the states that enter each
// tile of kGlrRows steps (one fp32 state in 64 elements), and the tile runs its
// own forward maps again from there, which is exact in fp32 where a saved bf16 h
// would add its rounding to dL/dz_r.
//
// What bounds it.  The forward moves 4 values an element and issues about 55
// instructions (two sigmoids, an exponential, a root), the backward 7 and about 95.
// At 2048 x 32 x 1024 bf16 the forward takes 115 us and the backward 191 (4.7 and 4.9
// TB/s), with restarts 124 to 141 and 202 to 228: loads and issue overlap, and neither
// alone would take that long.  A prompt of 16384 x 1 x 1024 takes 44 us (3.1 TB/s): 128
// workgroups a time, joined by the look-back.
#include "lrs_tbd.hpp"

namespace lrs {

namespace {

// Time tiles of a look-back group.  The end states of the groups form a chain: with
// 16 tiles a group a prompt of 16384 steps (bf16: tiles of 128) has 8 links.  Groups
// of 8, as in the other layers, take the same 40 to 45 us there; half the links
// leave room for the longer prompts.
constexpr int kGlrGroup = 16;

// One row of a strided array: the lane's channels at byte offsets zo from a
// wave-uniform pointer (32 bits: no address arithmetic a row); FULL: all in one
// aligned group at zo[0].
template <typename IO>
__device__ __forceinline__ const IO* at(const IO* p, uint32_t bytes) {
  return reinterpret_cast<const IO*>(reinterpret_cast<const char*>(p) + bytes);
}
template <typename IO>
__device__ __forceinline__ IO* at(IO* p, uint32_t bytes) {
  return reinterpret_cast<IO*>(reinterpret_cast<char*>(p) + bytes);
}
template <int CPT, bool FULL, bool NT>
__device__ __forceinline__ void glr_ld(const uint16_t* p, const uint32_t (&zo)[CPT], int nv,
                                       IoRow<uint16_t, CPT>& r) {
  if constexpr (FULL) {
    r.template load<true, NT>(at(p, zo[0]), 0, CPT);
  } else if constexpr (CPT == 1) {
    r.w = nv > 0 ? *at(p, zo[0]) : 0u;
  } else {
#pragma unroll
    for (int k = 0; k < CPT / 2; ++k) {
      const uint32_t lo = 2 * k < nv ? *at(p, zo[2 * k]) : 0u;
      const uint32_t hi = 2 * k + 1 < nv ? *at(p, zo[2 * k + 1]) : 0u;
      r.w[k] = lo | (hi << 16);
    }
  }
}
template <int CPT, bool FULL, bool NT>
__device__ __forceinline__ void glr_ld(const float* p, const uint32_t (&zo)[CPT], int nv,
                                       IoRow<float, CPT>& r) {
  if constexpr (FULL) {
    r.template load<true, NT>(at(p, zo[0]), 0, CPT);
  } else {
#pragma unroll
    for (int k = 0; k < CPT; ++k) r.v[k] = k < nv ? *at(p, zo[k]) : 0.0f;
  }
}
template <int CPT, bool FULL, bool NT, typename IO>
__device__ __forceinline__ void glr_st(IO* p, const uint32_t (&zo)[CPT], int nv,
                                       const float (&v)[CPT]) {
  if constexpr (FULL) {
    IoRow<IO, CPT>::template store<true, NT>(at(p, zo[0]), 0, CPT, v);
  } else {
#pragma unroll
    for (int k = 0; k < CPT; ++k)
      if (k < nv) io_st(at(p, zo[k]), 0, v[k]);
  }
}

// softplus(v) = max(v, 0) + log(1 + exp(-|v|)).
__device__ __forceinline__ float softplus(float v) { return fmaxf(v, 0.0f) + log1pf(expf(-fabsf(v))); }

// The exponent of a fully open gate, k = c softplus(decay), and -c times the
// derivative of softplus: computed once a call (k_glr_prep) where a tile is one
// of many, because with its 16 elements a thread the library functions and the
// division below would be a seventh of the backward's instructions.
__device__ __forceinline__ void glr_rates(const GlrArgs& g, uint32_t d, float& k, float& dk) {
  const float v = g.decay[d];
  k = g.c * softplus(v);
  dk = -g.c * fast_sigmoid(v, 0.0f);
}

// What a channel's parameters become: biases in the sigmoid's log2 units, and k.
template <int CPT>
struct GlrChan {
  float br[CPT], bi[CPT], k[CPT];
  uint32_t zo[CPT];  // byte offsets in a row of the inputs
  uint32_t b[CPT], d[CPT];
  bool near;  // k < 1/8 in every channel of the wave
  // off: the lane's first channel in its block, which begins at cbase
  __device__ __forceinline__ void set(const GlrArgs& g, int64_t cbase, uint32_t off, int nvc,
                                      uint32_t es) {
    const uint32_t D = (uint32_t)g.D;
    const uint32_t b0 = __builtin_amdgcn_readfirstlane((uint32_t)cbase / D);
    const uint32_t d0 = (uint32_t)cbase - b0 * D;
    bool low = true;
#pragma unroll
    for (int j = 0; j < CPT; ++j) {
      const uint32_t e = j < nvc ? d0 + off + j : d0;
      if (D >= kWave * CPT) {  // a block meets at most one border of two sequences
        b[j] = e >= D ? b0 + 1 : b0;
        d[j] = e >= D ? e - D : e;
      } else {
        const uint32_t q = e / D;
        b[j] = b0 + q;
        d[j] = e - q * D;
      }
      zo[j] = (b[j] * (uint32_t)g.ld + d[j]) * es;
      br[j] = -kLog2e * g.bias_r[d[j]];
      bi[j] = -kLog2e * g.bias_i[d[j]];
      if (g.rates) {
        k[j] = g.rates[d[j]];
      } else {
        float dk;
        glr_rates(g, d[j], k[j], dk);
      }
      low = low && k[j] < 0.125f;
    }
    near = __all(low);
  }
};

// a = exp(-t) and m^2 = 1 - a^2 for t = c softplus(decay) r >= 0.  For a long
// memory (t < 1/8) 1 - a comes from the series of -expm1(-t), cut after the
// fifth term (t^5 / 720 = 4e-8 of it there), and a and 1 - a^2 = (1 - a)(1 + a)
// from that: subtracting a^2 from 1 would lose the digits of 1 - a, and the
// exponential instruction's last bit, which does not round to nearest, would
// add up over the steps that the state survives (2e-5 of h over 640 of them).
// NEAR: every t is below 1/8 (k is, and r is at most 1), and the rest is left out: 115
// and 191 us (forward, backward, 2048 x 32 x 1024 bf16) against 118 and 199 with the
// general form, 44 against 47 for a prompt of 16384 x 1 x 1024.
template <bool NEAR>
__device__ __forceinline__ void glr_decay(float t, float& a, float& m2) {
  float p = __builtin_fmaf(t, 1.0f / 120.0f, -1.0f / 24.0f);
  p = __builtin_fmaf(t, p, 1.0f / 6.0f);
  p = __builtin_fmaf(t, p, -0.5f);
  p = __builtin_fmaf(t, p, 1.0f);
  const float e = t * p;
  if constexpr (NEAR) {
    a = 1.0f - e;
    m2 = e * (2.0f - e);
    return;
  }
  const float far = __builtin_amdgcn_exp2f(-kLog2e * t);
  const bool near = t < 0.125f;
  a = near ? 1.0f - e : far + kLeastFactor;  // not 0, which is a restart
  m2 = near ? e * (2.0f - e) : __builtin_fmaf(-far, far, 1.0f);
}

struct GlrGate {
  float r, i, a, m;
};
template <bool NEAR>
__device__ __forceinline__ GlrGate glr_gate(float zr, float zi, float br, float bi, float k,
                                            bool cut) {
  GlrGate g;
  g.r = fast_sigmoid(zr, br);
  g.i = fast_sigmoid(zi, bi);
  float m2;
  glr_decay<NEAR>(k * g.r, g.a, m2);
  g.m = __builtin_amdgcn_sqrtf(m2);
  if (cut) {
    g.a = 0.0f;
    g.m = 1.0f;
  }
  return g;
}

// The reset bytes of a row for the lane's channels (FULL: one sequence a lane).
template <int CPT, bool FULL, bool RST>
__device__ __forceinline__ void glr_cut(const uint8_t* reset, int64_t row, const GlrArgs& g,
                                        const GlrChan<CPT>& ch, int nv, uint32_t (&cut)[CPT]) {
#pragma unroll
  for (int k = 0; k < CPT; ++k) cut[k] = 0;
  if constexpr (RST) {
    if constexpr (FULL) {
      cut[0] = reset[row * g.B + ch.b[0]];
#pragma unroll
      for (int k = 1; k < CPT; ++k) cut[k] = cut[0];
    } else {
#pragma unroll
      for (int k = 0; k < CPT; ++k)
        if (k < nv) cut[k] = reset[row * g.B + ch.b[k]];
    }
  }
}

// One step a * x + b, where with SEL a factor of 0 gives b whatever x is (the legacy
// product: two instructions a step, where affine's compare and select make three).
template <bool SEL>
__device__ __forceinline__ float step(float a, float x, float b) {
  return SEL ? scale<SEL>(a, x) + b : __builtin_fmaf(a, x, b);
}

template <typename IO, int L, int CPT>
struct GlrRows {
  IoRow<IO, CPT> zr[L], zi[L], x[L];
  uint32_t cut[L][CPT];
};

template <typename IO, int L, int CPT, bool FULL, bool NT, bool RST>
__device__ __forceinline__ void glr_load(const GlrArgs& g, const GlrChan<CPT>& ch, int64_t row0,
                                         int nvc, GlrRows<IO, L, CPT>& rows) {
  const int64_t pitch = g.B * g.ld;
  const IO* rp = (const IO*)g.z_r + row0 * pitch;
  const IO* ip = (const IO*)g.z_i + row0 * pitch;
  const IO* xp = (const IO*)g.x + row0 * pitch;
#pragma unroll
  for (int i = 0; i < L; ++i) {
    const int nv = (FULL || row0 + i < g.T) ? nvc : 0;
    glr_ld<CPT, FULL, NT>(rp, ch.zo, nv, rows.zr[i]);
    glr_ld<CPT, FULL, NT>(ip, ch.zo, nv, rows.zi[i]);
    glr_ld<CPT, FULL, NT>(xp, ch.zo, nv, rows.x[i]);
    glr_cut<CPT, FULL, RST>(g.reset, row0 + i, g, ch, nv, rows.cut[i]);
    rp += pitch;
    ip += pitch;
    xp += pitch;
  }
}

// The step maps (a, m i x) of the loaded rows; identity past the end.
template <bool NEAR, typename IO, int L, int CPT, bool FULL>
__device__ __forceinline__ void glr_maps(const GlrArgs& g, const GlrChan<CPT>& ch, int64_t row0,
                                         int nvc, const GlrRows<IO, L, CPT>& rows,
                                         float (&av)[L][CPT], float (&bv)[L][CPT]) {
#pragma unroll
  for (int i = 0; i < L; ++i) {
    const bool row_ok = FULL || row0 + i < g.T;
#pragma unroll
    for (int k = 0; k < CPT; ++k) {
      if (FULL || (row_ok && k < nvc)) {
        const GlrGate q = glr_gate<NEAR>(rows.zr[i].get(k), rows.zi[i].get(k), ch.br[k],
                                         ch.bi[k], ch.k[k], rows.cut[i][k] != 0);
        av[i][k] = q.a;
        bv[i][k] = q.m * q.i * rows.x[i].get(k);
      } else {
        av[i][k] = 1.0f;
        bv[i][k] = 0.0f;
      }
    }
  }
}

// Both forms, chosen once a wave: an open gate keeps more than 0.88 of the state
// (k < 1/8) in all of its channels, or not.
template <typename IO, int L, int CPT, bool FULL>
__device__ __forceinline__ void glr_maps(const GlrArgs& g, const GlrChan<CPT>& ch, int64_t row0,
                                         int nvc, const GlrRows<IO, L, CPT>& rows,
                                         float (&av)[L][CPT], float (&bv)[L][CPT]) {
  if (ch.near) glr_maps<true, IO, L, CPT, FULL>(g, ch, row0, nvc, rows, av, bv);
  else glr_maps<false, IO, L, CPT, FULL>(g, ch, row0, nvc, rows, av, bv);
}

template <int L, int CPT, bool SEL>
__device__ __forceinline__ void glr_fold(const float (&av)[L][CPT], const float (&bv)[L][CPT],
                                         float (&A)[CPT], float (&B)[CPT]) {
#pragma unroll
  for (int k = 0; k < CPT; ++k) {
    A[k] = av[0][k];
    B[k] = bv[0][k];
    float least = av[0][k];
#pragma unroll
    for (int i = 1; i < L; ++i) {
      B[k] = step<SEL>(av[i][k], B[k], bv[i][k]);
      A[k] = A[k] * av[i][k];
      least = fminf(least, av[i][k]);
    }
    A[k] = factor<SEL>(A[k], least);
  }
}

// The wave's steps from its entering state x, h written on the way; x ends as
// the state after the wave's last row.
template <typename IO, int L, int CPT, bool FULL, bool NT, bool SEL>
__device__ __forceinline__ void glr_walk(const GlrArgs& g, int64_t row0, int64_t cbase,
                                         uint32_t off, int nvc, const float (&av)[L][CPT],
                                         const float (&bv)[L][CPT], float (&x)[CPT]) {
  const int64_t C = g.B * g.D;
  IO* hp = (IO*)g.h + row0 * C + cbase;
#pragma unroll
  for (int i = 0; i < L; ++i) {
#pragma unroll
    for (int k = 0; k < CPT; ++k) x[k] = step<SEL>(av[i][k], x[k], bv[i][k]);
    const int nv = (FULL || row0 + i < g.T) ? nvc : 0;
    IoRow<IO, CPT>::template store<FULL, NT>(at(hp, off * (uint32_t)sizeof(IO)), 0, nv, x);
    hp += C;
  }
}

// The state entering row0, where a checkpoint's stretch begins there.
template <int CPT, bool FULL>
__device__ __forceinline__ void glr_checkpoint(const GlrArgs& g, int64_t row0, int64_t cbase,
                                               uint32_t off, int nvc, const float (&x)[CPT]) {
  if (g.checkpoints && row0 % kGlrRows == 0 && row0 < g.T)
    store_row<CPT, FULL, false>(g.checkpoints + row0 / kGlrRows * (g.B * g.D) + cbase, off, nvc, x);
}

// ---------------------------------------------------------------------------
// forward, look-back tiles: where the channel blocks alone leave compute units idle
// (1531 x 5 x 517 fp32: 23 us, 2.7 TB/s)
// ---------------------------------------------------------------------------
template <typename IO, int NW, int L, int CPT, bool FULL, bool NT, bool RST>
__device__ __forceinline__ void glr_tile(const GlrArgs& g, int tb, int cb, bool multi,
                                         uint64_t* st, ColShared<NW, CPT>& s) {
  const int64_t C = g.B * g.D;
  const ColPos q = col_pos<NW, L, CPT>(tb, cb, C);
  const int64_t cbase = (int64_t)cb * (kWave * CPT);
  GlrChan<CPT> ch;
  ch.set(g, cbase, q.off, q.nvc, sizeof(IO));
  GlrRows<IO, L, CPT> rows;
  glr_load<IO, L, CPT, FULL, NT, RST>(g, ch, q.row0, q.nvc, rows);
  float av[L][CPT], bv[L][CPT], A[CPT], B[CPT], x0[CPT], x[CPT];
  glr_maps<IO, L, CPT, FULL>(g, ch, q.row0, q.nvc, rows, av, bv);
  glr_fold<L, CPT, RST>(av, bv, A, B);
#pragma unroll
  for (int k = 0; k < CPT; ++k) x0[k] = (g.h0 && k < q.nvc) ? g.h0[q.c0 + k] : 0.0f;
  col_enter_state<NW, CPT, RST, kGlrGroup>(A, B, multi, tb, x0, g.h0, cbase,
                                           clamp_valid(C - cbase, kWave * CPT), st, s, x);
  glr_checkpoint<CPT, FULL>(g, q.row0, cbase, q.off, q.nvc, x);
  glr_walk<IO, L, CPT, FULL, NT, RST>(g, q.row0, cbase, q.off, q.nvc, av, bv, x);
  // rows past the end keep the state, so the wave that holds row T-1 ends with h_T
  if (g.h_last && q.row0 < g.T && q.row0 + L >= g.T) {
#pragma unroll
    for (int k = 0; k < CPT; ++k)
      if (k < q.nvc) g.h_last[q.c0 + k] = x[k];
  }
}

template <typename IO, int NW, int L, int CPT, bool NT, bool RST>
__global__ __launch_bounds__(NW* kWave) void k_glr_fwd(GlrArgs g, int ncb, int ntb,
                                                       uint64_t* __restrict__ status,
                                                       unsigned* __restrict__ tickets) {
  constexpr int CW = kWave * CPT, TW = NW * L;
  static_assert(TW % kGlrRows == 0 && kGlrRows % L == 0, "stretches begin with a wave's rows");
  __shared__ ColShared<NW, CPT> s;
  const bool multi = ntb > 1;
  const int cb = (int)(blockIdx.x % (unsigned)ncb);
  const int tb = col_ticket<NW, CPT>(multi, tickets, cb, s);
  uint64_t* st = status + (int64_t)cb * ntb * CW;
  const bool full = (int64_t)(tb + 1) * TW <= g.T && (int64_t)(cb + 1) * CW <= g.B * g.D;
  if (full)
    glr_tile<IO, NW, L, CPT, true, NT, RST>(g, tb, cb, multi, st, s);
  else
    glr_tile<IO, NW, L, CPT, false, NT, RST>(g, tb, cb, multi, st, s);
}

// ---------------------------------------------------------------------------
// persistent forward: one workgroup per channel block visits every time tile in
// order, the state entering the tile carried in LDS, the next tile's rows loaded
// into registers while the current one is processed; no look-back state and no
// kernel that resets it.  Used when the channel blocks alone fill the GPU (2048 x 32
// x 1024 bf16, 256 blocks: 4.1 TB/s).
// ---------------------------------------------------------------------------
template <typename IO, int NW, int L, int CPT, bool FULL, int PF, bool NT, bool RST>
__device__ __forceinline__ void glr_persist_tile(const GlrArgs& g, const GlrChan<CPT>& ch,
                                                 int64_t row0, int64_t cbase, uint32_t off, int nvc,
                                                 GlrRows<IO, L, CPT>& rows,
                                                 PersistShared<NW, CPT>& s, int wid, int par) {
  float av[L][CPT], bv[L][CPT], A[CPT], B[CPT], x[CPT];
  glr_maps<IO, L, CPT, FULL>(g, ch, row0, nvc, rows, av, bv);
  if (PF == 1) glr_load<IO, L, CPT, true, NT, RST>(g, ch, row0 + NW * L, nvc, rows);
  else if (PF == 2) glr_load<IO, L, CPT, false, NT, RST>(g, ch, row0 + NW * L, nvc, rows);
  glr_fold<L, CPT, RST>(av, bv, A, B);
  persist_enter<NW, CPT, RST>(A, B, s, wid, off, x, par);
  glr_checkpoint<CPT, FULL>(g, row0, cbase, off, nvc, x);
  glr_walk<IO, L, CPT, FULL, NT, RST>(g, row0, cbase, off, nvc, av, bv, x);
  persist_advance<NW, CPT>(x, s, wid, off, par);
}

template <typename IO, int NW, int L, int CPT, bool NT, bool RST>
__global__ __launch_bounds__(NW* kWave) void k_glr_fwd_persist(GlrArgs g) {
  constexpr int CW = kWave * CPT, TW = NW * L;
  __shared__ PersistShared<NW, CPT> s;
  const int64_t C = g.B * g.D;
  const int lane = threadIdx.x & (kWave - 1);
  const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int64_t cbase = (int64_t)blockIdx.x * CW;
  const uint32_t off = (uint32_t)(lane * CPT);
  const int nvc = clamp_valid(C - (cbase + off), CPT);
  const bool cfull = cbase + CW <= C;
  for (int j = threadIdx.x; j < CW; j += NW * kWave)
    s.carry[0][j] = (g.h0 && cbase + j < C) ? g.h0[cbase + j] : 0.0f;
  GlrChan<CPT> ch;
  ch.set(g, cbase, off, nvc, sizeof(IO));
  const int64_t ntb = (g.T + TW - 1) / TW, nfull = g.T / TW;
  const int64_t w0 = (int64_t)wid * L;
  GlrRows<IO, L, CPT> rows;
#define LRS_TILE(FULLT, PFT, TB)                                                                \
  glr_persist_tile<IO, NW, L, CPT, FULLT, PFT, NT, RST>(g, ch, (TB) * TW + w0, cbase, off, nvc, \
                                                        rows, s, wid, (int)((TB) & 1))
  if (cfull && nfull > 0) {
    glr_load<IO, L, CPT, true, NT, RST>(g, ch, w0, nvc, rows);
    for (int64_t tb = 0; tb + 1 < nfull; ++tb) LRS_TILE(true, 1, tb);
    if (ntb > nfull) {
      LRS_TILE(true, 2, nfull - 1);
      LRS_TILE(false, 0, nfull);
    } else {
      LRS_TILE(true, 0, nfull - 1);
    }
  } else {
    glr_load<IO, L, CPT, false, NT, RST>(g, ch, w0, nvc, rows);
    for (int64_t tb = 0; tb < ntb; ++tb) {
      if (tb + 1 < ntb) LRS_TILE(false, 2, tb);
      else LRS_TILE(false, 0, tb);
    }
  }
#undef LRS_TILE
  if (g.h_last) {  // rows past the end keep the state
    __syncthreads();
    for (int j = threadIdx.x; j < CW; j += NW * kWave)
      if (cbase + j < C) g.h_last[cbase + j] = s.carry[ntb & 1][j];
  }
}

// ---------------------------------------------------------------------------
// backward: logical time block 0 is the last physical one, wave 0 takes its
// latest steps (as the other layers' backward passes).  Two chains run through
// a tile: forward, the states from the tile's checkpoint (within the tile
// only), and in reverse time the gradient y_t = a_t lam_t, tiles joined by the
// look-back.
// ---------------------------------------------------------------------------
template <int NW, int CPT>
struct GlrBwdShared {
  float fA[NW][kWave * CPT], fB[NW][kWave * CPT];  // forward maps of the waves
  float red[3][NW][kWave * CPT];                   // parameter gradients of the waves
};

template <bool NEAR, typename IO, int L, int CPT, bool FULL>
__device__ __forceinline__ void glr_gates(const GlrArgs& g, const GlrChan<CPT>& ch, int64_t row0,
                                          int nvc, const GlrRows<IO, L, CPT>& rows,
                                          float (&r)[L][CPT], float (&gi)[L][CPT],
                                          float (&av)[L][CPT], float (&m)[L][CPT]) {
#pragma unroll
  for (int i = 0; i < L; ++i) {
    const bool row_ok = FULL || row0 + i < g.T;
#pragma unroll
    for (int k = 0; k < CPT; ++k) {
      GlrGate q;
      if (FULL || (row_ok && k < nvc)) {
        q = glr_gate<NEAR>(rows.zr[i].get(k), rows.zi[i].get(k), ch.br[k], ch.bi[k], ch.k[k],
                           rows.cut[i][k] != 0);
      } else {
        q.r = q.i = q.m = 0.0f;
        q.a = 1.0f;
      }
      r[i][k] = q.r;
      gi[i][k] = q.i;
      av[i][k] = q.a;
      m[i][k] = q.m;
    }
  }
}

// A wave's rows of one tile: the packed inputs and what the gates make of them.
template <typename IO, int L, int CPT>
struct GlrBwdRows {
  GlrRows<IO, L, CPT> in;
  IoRow<IO, CPT> gh[L];
};

template <typename IO, int L, int CPT, bool FULL, bool NT, bool RST>
__device__ __forceinline__ void glr_bwd_load(const GlrArgs& g, const GlrChan<CPT>& ch, int64_t row0,
                                             int64_t cbase, uint32_t off, int nvc,
                                             GlrBwdRows<IO, L, CPT>& w) {
  const int64_t C = g.B * g.D;
  glr_load<IO, L, CPT, FULL, NT, RST>(g, ch, row0, nvc, w.in);
  const IO* gp = (const IO*)g.grad_h + row0 * C + cbase;
#pragma unroll
  for (int i = 0; i < L; ++i) {
    w.gh[i].template load<FULL, NT>(at(gp, off * (uint32_t)sizeof(IO)), 0,
                                    (FULL || row0 + i < g.T) ? nvc : 0);
    gp += C;
  }
}

// The wave's maps of both chains: forward (FA, FB) for the states, reverse (A, B)
// for y.
template <int L, int CPT, bool RST, typename IO>
__device__ __forceinline__ void glr_bwd_fold(const IoRow<IO, CPT> (&x)[L],
                                             const IoRow<IO, CPT> (&gh)[L],
                                             const float (&gi)[L][CPT], const float (&av)[L][CPT],
                                             const float (&m)[L][CPT], float (&FA)[CPT],
                                             float (&FB)[CPT], float (&A)[CPT], float (&B)[CPT]) {
#pragma unroll
  for (int k = 0; k < CPT; ++k) {
    float least = av[0][k];
#pragma unroll
    for (int i = 0; i < L; ++i) {
      const float b = m[i][k] * gi[i][k] * x[i].get(k);  // 0 past the end (x reads as 0 there)
      FB[k] = i == 0 ? b : step<RST>(av[i][k], FB[k], b);
      FA[k] = i == 0 ? av[i][k] : FA[k] * av[i][k];
      least = fminf(least, av[i][k]);
    }
    FA[k] = factor<RST>(FA[k], least);
    // y passed on: lam_{L-1} = gh_{L-1} + y_in, lam_i = gh_i + a_{i+1} lam_{i+1},
    // y_out = a_0 lam_0 (gh and a are 0 and 1 past the end): the same factor
    A[k] = FA[k];
    B[k] = gh[L - 1].get(k);
#pragma unroll
    for (int i = L - 2; i >= 0; --i) B[k] = step<RST>(av[i + 1][k], B[k], gh[i].get(k));
    B[k] = scale<RST>(av[0][k], B[k]);
  }
}

// x and grad_h stay packed across the barriers: unpacked copies kept by the
// compiler would cost registers that the waves of a compute unit do not have.
template <int L, int CPT>
__device__ __forceinline__ void keep_packed(IoRow<uint16_t, CPT> (&x)[L],
                                            IoRow<uint16_t, CPT> (&gh)[L]) {
#pragma unroll
  for (int i = 0; i < L; ++i)
#pragma unroll
    for (int k = 0; k < CPT / 2; ++k) asm("" : "+v"(x[i].w[k]), "+v"(gh[i].w[k]));
}
template <int L>
__device__ __forceinline__ void keep_packed(IoRow<uint16_t, 1> (&x)[L], IoRow<uint16_t, 1> (&gh)[L]) {
#pragma unroll
  for (int i = 0; i < L; ++i) asm("" : "+v"(x[i].w), "+v"(gh[i].w));
}
template <int L, int CPT>
__device__ __forceinline__ void keep_packed(IoRow<float, CPT> (&)[L], IoRow<float, CPT> (&)[L]) {}

// Sums for bias_r, bias_i and k: S = float over a wave's rows of a tile, and S = double
// over the tiles of a persistent walk, whose number has no bound (fp32 would lose 7e-5
// of 40000 equal terms).
template <int CPT, typename S = float>
struct GlrSums {
  S r[CPT], i[CPT], d[CPT];
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int k = 0; k < CPT; ++k) r[k] = i[k] = d[k] = 0;
  }
  template <typename T>
  __device__ __forceinline__ void add(const GlrSums<CPT, T>& s) {
#pragma unroll
    for (int k = 0; k < CPT; ++k) {
      r[k] += (S)s.r[k];
      i[k] += (S)s.i[k];
      d[k] += (S)s.d[k];
    }
  }
};

// The wave's rows from the state hs before them and y after them: the gradients,
// and y before them.
template <typename IO, int L, int CPT, bool FULL, bool NT, bool RST>
__device__ __forceinline__ void glr_bwd_walk(const GlrArgs& g, const GlrChan<CPT>& ch,
                                             const uint32_t (&go)[CPT], int64_t row0, int nvc,
                                             const IoRow<IO, CPT> (&x)[L],
                                             const IoRow<IO, CPT> (&gh)[L],
                                             const float (&r)[L][CPT], const float (&gi)[L][CPT],
                                             const float (&av)[L][CPT], const float (&m)[L][CPT],
                                             float (&hs)[CPT], float (&y)[CPT],
                                             GlrSums<CPT>& sum) {
  float hp[L][CPT];
#pragma unroll
  for (int i = 0; i < L; ++i) {
#pragma unroll
    for (int k = 0; k < CPT; ++k) {
      hp[i][k] = hs[k];
      hs[k] = step<RST>(av[i][k], hs[k], m[i][k] * gi[i][k] * x[i].get(k));
    }
  }
  const int64_t gpitch = g.B * g.ld_grad;
  IO* qr = (IO*)g.grad_zr + (row0 + L - 1) * gpitch;
  IO* qi = (IO*)g.grad_zi + (row0 + L - 1) * gpitch;
  IO* qx = (IO*)g.grad_x + (row0 + L - 1) * gpitch;
#pragma unroll
  for (int i = L - 1; i >= 0; --i) {
    float dr[CPT], di[CPT], dx[CPT];
#pragma unroll
    for (int k = 0; k < CPT; ++k) {
      y[k] = i == L - 1 ? y[k] + gh[i].get(k) : step<RST>(av[i + 1][k], y[k], gh[i].get(k));  // lam_t
      const float u = gi[i][k] * x[i].get(k), a = av[i][k], mm = m[i][k], lam = y[k];
      const float dgx = lam * mm;
      dx[k] = dgx * gi[i][k];
      di[k] = dgx * u * (1.0f - gi[i][k]);
      const float rm = mm == 0.0f ? 0.0f : __builtin_amdgcn_rcpf(mm);
      const float dla = scale<RST>(a, lam * __builtin_fmaf(-a * rm, u, hp[i][k]));
      // at a restart 0 whatever the gate would have been
      const float dlr = scale<RST>(dla, r[i][k]);
      dr[k] = scale<RST>(-dlr * ch.k[k], 1.0f - r[i][k]);  // la = -k r
      sum.r[k] += dr[k];
      sum.i[k] += di[k];
      sum.d[k] += dlr;
    }
    const int nv = (FULL || row0 + i < g.T) ? nvc : 0;
    glr_st<CPT, FULL, NT>(qr, go, nv, dr);
    glr_st<CPT, FULL, NT>(qi, go, nv, di);
    glr_st<CPT, FULL, NT>(qx, go, nv, dx);
    qr -= gpitch;
    qi -= gpitch;
    qx -= gpitch;
  }
#pragma unroll
  for (int k = 0; k < CPT; ++k) y[k] = scale<RST>(av[0][k], y[k]);
}

// The waves' sums of a workgroup, added in wave order, to row `slot` of the
// partial sums' `slots` rows.
template <int NW, int CPT, typename S>
__device__ __forceinline__ void glr_bwd_sums(const GlrArgs& g, const GlrChan<CPT>& ch,
                                             const GlrSums<CPT, S>& sum,
                                             float (&red)[3][NW][kWave * CPT], int wid, uint32_t off,
                                             int64_t cbase, int64_t slot, int64_t slots) {
  constexpr int CW = kWave * CPT;
  const int64_t C = g.B * g.D;
#pragma unroll
  for (int k = 0; k < CPT; ++k) {
    red[0][wid][off + k] = (float)sum.r[k];
    red[1][wid][off + k] = (float)sum.i[k];
    red[2][wid][off + k] = (float)(sum.d[k] * g.rates[g.D + ch.d[k]]);  // with d k / d decay
  }
  __syncthreads();
  for (int j = threadIdx.x; j < 3 * CW; j += NW * kWave) {
    const int which = j / CW, c = j % CW;
    float t = 0.0f;
#pragma unroll
    for (int w = 0; w < NW; ++w) t += red[which][w][c];
    if (cbase + c < C) g.part[((int64_t)which * slots + slot) * C + cbase + c] = t;
  }
}

template <typename IO, int NW, int L, int CPT, bool FULL, bool NT, bool RST>
__device__ __forceinline__ void glr_bwd_tile(const GlrArgs& g, int tb, int ntb, int cb, bool multi,
                                             uint64_t* st, ColShared<NW, CPT>& s,
                                             GlrBwdShared<NW, CPT>& f) {
  constexpr int CW = kWave * CPT;
  const int64_t C = g.B * g.D;
  const int lane = threadIdx.x & (kWave - 1);
  const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int ptb = ntb - 1 - tb;
  const uint32_t off = (uint32_t)(lane * CPT);
  const int64_t cbase = (int64_t)cb * CW;
  const int64_t c0 = cbase + off;
  const int nvc = FULL ? CPT : clamp_valid(C - c0, CPT);
  const int64_t row0 = (int64_t)ptb * (NW * L) + (int64_t)(NW - 1 - wid) * L;
  GlrChan<CPT> ch;
  ch.set(g, cbase, off, nvc, sizeof(IO));
  GlrBwdRows<IO, L, CPT> w;
  glr_bwd_load<IO, L, CPT, FULL, NT, RST>(g, ch, row0, cbase, off, nvc, w);
  float r[L][CPT], gi[L][CPT], av[L][CPT], m[L][CPT];
  float FA[CPT], FB[CPT], A[CPT], B[CPT];
  if (ch.near) glr_gates<true, IO, L, CPT, FULL>(g, ch, row0, nvc, w.in, r, gi, av, m);
  else glr_gates<false, IO, L, CPT, FULL>(g, ch, row0, nvc, w.in, r, gi, av, m);
  glr_bwd_fold<L, CPT, RST>(w.in.x, w.gh, gi, av, m, FA, FB, A, B);
  float x0[CPT], y[CPT], hs[CPT];
#pragma unroll
  for (int k = 0; k < CPT; ++k) {
    f.fA[wid][off + k] = FA[k];
    f.fB[wid][off + k] = FB[k];
    x0[k] = (g.grad_h_last && k < nvc) ? g.grad_h_last[c0 + k] : 0.0f;
    hs[k] = k < nvc ? g.checkpoints[(int64_t)ptb * C + c0 + k] : 0.0f;
  }
  col_enter_state<NW, CPT, RST>(A, B, multi, tb, x0, g.grad_h_last, cbase,
                                clamp_valid(C - cbase, CW), st, s, y);
  keep_packed(w.in.x, w.gh);
  // past a barrier: the states before each of the wave's rows
  for (int v = NW - 1; v > wid; --v) {
#pragma unroll
    for (int k = 0; k < CPT; ++k) hs[k] = affine<RST>(f.fA[v][off + k], hs[k], f.fB[v][off + k]);
  }
  uint32_t go[CPT];
#pragma unroll
  for (int k = 0; k < CPT; ++k)
    go[k] = (ch.b[k] * (uint32_t)g.ld_grad + ch.d[k]) * (uint32_t)sizeof(IO);
  GlrSums<CPT> sum;
  sum.clear();
  glr_bwd_walk<IO, L, CPT, FULL, NT, RST>(g, ch, go, row0, nvc, w.in.x, w.gh, r, gi, av, m, hs, y,
                                          sum);
  if (g.grad_h0 && row0 == 0) {
#pragma unroll
    for (int k = 0; k < CPT; ++k)
      if (k < nvc) g.grad_h0[c0 + k] = y[k];
  }
  glr_bwd_sums<NW>(g, ch, sum, f.red, wid, off, cbase, ptb, ntb);
}

template <typename IO, int NW, int L, int CPT, bool NT, bool RST>
__global__ __launch_bounds__(NW* kWave) void k_glr_bwd(GlrArgs g, int ncb, int ntb,
                                                       uint64_t* __restrict__ status,
                                                       unsigned* __restrict__ tickets) {
  constexpr int CW = kWave * CPT, TW = NW * L;
  static_assert(TW == kGlrRows, "a tile is a checkpoint's stretch");
  __shared__ ColShared<NW, CPT> s;
  __shared__ GlrBwdShared<NW, CPT> f;
  const bool multi = ntb > 1;
  const int cb = (int)(blockIdx.x % (unsigned)ncb);
  const int tb = col_ticket<NW, CPT>(multi, tickets, cb, s);
  uint64_t* st = status + (int64_t)cb * ntb * CW;
  const int ptb = ntb - 1 - tb;
  const bool full = (int64_t)(ptb + 1) * TW <= g.T && (int64_t)(cb + 1) * CW <= g.B * g.D;
  if (full)
    glr_bwd_tile<IO, NW, L, CPT, true, NT, RST>(g, tb, ntb, cb, multi, st, s, f);
  else
    glr_bwd_tile<IO, NW, L, CPT, false, NT, RST>(g, tb, ntb, cb, multi, st, s, f);
}

// ---------------------------------------------------------------------------
// persistent backward: one workgroup per channel block walks the tiles from the
// last to the first, y in LDS, the next tile's rows and checkpoint in flight
// while the current one is processed, the parameters' sums in registers until
// the end.  As the forward, where the channel blocks alone fill the GPU: a tile's
// rows and gates take 170 registers, so that a compute unit holds one workgroup
// either way, and without the prefetch its loads and its arithmetic take turns (308
// us as look-back tiles against 204 to 218 at 2048 x 32 x 1024 bf16).
// ---------------------------------------------------------------------------
template <int NW, int CPT>
struct GlrWalkShared {
  PersistShared<NW, CPT> y;
  float fA[2][NW][kWave * CPT], fB[2][NW][kWave * CPT];
};

template <typename IO, int NW, int L, int CPT, bool FULL, int PF, bool NT, bool RST>
__device__ __forceinline__ void glr_bwd_persist_tile(
    const GlrArgs& g, const GlrChan<CPT>& ch, const uint32_t (&go)[CPT], int64_t row0, int64_t cbase,
    uint32_t off, int nvc, GlrBwdRows<IO, L, CPT>& w, float (&ck)[CPT],
    GlrSums<CPT, double>& sum, GlrWalkShared<NW, CPT>& s, int wid, int par) {
  float r[L][CPT], gi[L][CPT], av[L][CPT], m[L][CPT];
  float FA[CPT], FB[CPT], A[CPT], B[CPT], y[CPT], hs[CPT];
  if (ch.near) glr_gates<true, IO, L, CPT, FULL>(g, ch, row0, nvc, w.in, r, gi, av, m);
  else glr_gates<false, IO, L, CPT, FULL>(g, ch, row0, nvc, w.in, r, gi, av, m);
  IoRow<IO, CPT> x[L], gh[L];
#pragma unroll
  for (int i = 0; i < L; ++i) {
    x[i] = w.in.x[i];
    gh[i] = w.gh[i];
  }
#pragma unroll
  for (int k = 0; k < CPT; ++k) hs[k] = ck[k];
  if (PF != 0) {  // the tile before this one: whole rows
    glr_bwd_load<IO, L, CPT, PF == 1, NT, RST>(g, ch, row0 - NW * L, cbase, off, nvc, w);
    const float* p = g.checkpoints + (row0 / kGlrRows - 1) * (g.B * g.D) + cbase + off;
#pragma unroll
    for (int k = 0; k < CPT; ++k) ck[k] = k < nvc ? p[k] : 0.0f;
  }
  glr_bwd_fold<L, CPT, RST>(x, gh, gi, av, m, FA, FB, A, B);
#pragma unroll
  for (int k = 0; k < CPT; ++k) {
    s.fA[par][wid][off + k] = FA[k];
    s.fB[par][wid][off + k] = FB[k];
  }
  persist_enter<NW, CPT, RST>(A, B, s.y, wid, off, y, par);  // its barrier covers fA and fB
  keep_packed(x, gh);
  for (int v = NW - 1; v > wid; --v) {
#pragma unroll
    for (int k = 0; k < CPT; ++k)
      hs[k] = affine<RST>(s.fA[par][v][off + k], hs[k], s.fB[par][v][off + k]);
  }
  GlrSums<CPT> tile;
  tile.clear();
  glr_bwd_walk<IO, L, CPT, FULL, NT, RST>(g, ch, go, row0, nvc, x, gh, r, gi, av, m, hs, y, tile);
  sum.add(tile);
  persist_advance<NW, CPT>(y, s.y, wid, off, par);
}

template <typename IO, int NW, int L, int CPT, bool NT, bool RST>
__global__ __launch_bounds__(NW* kWave) void k_glr_bwd_persist(GlrArgs g) {
  constexpr int CW = kWave * CPT, TW = NW * L;
  static_assert(TW == kGlrRows, "a tile is a checkpoint's stretch");
  __shared__ GlrWalkShared<NW, CPT> s;
  __shared__ float red[3][NW][CW];
  const int64_t C = g.B * g.D;
  const int lane = threadIdx.x & (kWave - 1);
  const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int64_t cbase = (int64_t)blockIdx.x * CW;
  const uint32_t off = (uint32_t)(lane * CPT);
  const int nvc = clamp_valid(C - (cbase + off), CPT);
  const bool cfull = cbase + CW <= C;
  for (int j = threadIdx.x; j < CW; j += NW * kWave)
    s.y.carry[0][j] = (g.grad_h_last && cbase + j < C) ? g.grad_h_last[cbase + j] : 0.0f;
  GlrChan<CPT> ch;
  ch.set(g, cbase, off, nvc, sizeof(IO));
  uint32_t go[CPT];
#pragma unroll
  for (int k = 0; k < CPT; ++k)
    go[k] = (ch.b[k] * (uint32_t)g.ld_grad + ch.d[k]) * (uint32_t)sizeof(IO);
  const int64_t ntb = (g.T + TW - 1) / TW;
  const int64_t w0 = (int64_t)(NW - 1 - wid) * L;
  GlrSums<CPT, double> sum;
  sum.clear();
  GlrBwdRows<IO, L, CPT> w;
  float ck[CPT];
#pragma unroll
  for (int k = 0; k < CPT; ++k)
    ck[k] = k < nvc ? g.checkpoints[(ntb - 1) * C + cbase + off + k] : 0.0f;
  // tile tb of the walk is the physical one ntb - 1 - tb; the first may be ragged
#define LRS_TILE(FULLT, PFT, TB)                                                               \
  glr_bwd_persist_tile<IO, NW, L, CPT, FULLT, PFT, NT, RST>(g, ch, go, (ntb - 1 - (TB)) * TW + w0, \
                                                            cbase, off, nvc, w, ck, sum, s, wid, \
                                                            (int)((TB) & 1))
  int64_t tb = 0;
  if (cfull) {
    if (g.T % TW) {
      glr_bwd_load<IO, L, CPT, false, NT, RST>(g, ch, (ntb - 1) * TW + w0, cbase, off, nvc, w);
      if (ntb > 1) LRS_TILE(false, 1, 0);
      else LRS_TILE(false, 0, 0);
      tb = 1;
    } else {
      glr_bwd_load<IO, L, CPT, true, NT, RST>(g, ch, (ntb - 1) * TW + w0, cbase, off, nvc, w);
    }
    for (; tb + 1 < ntb; ++tb) LRS_TILE(true, 1, tb);
    if (tb < ntb) LRS_TILE(true, 0, tb);
  } else {
    glr_bwd_load<IO, L, CPT, false, NT, RST>(g, ch, (ntb - 1) * TW + w0, cbase, off, nvc, w);
    for (; tb + 1 < ntb; ++tb) LRS_TILE(false, 2, tb);
    LRS_TILE(false, 0, tb);
  }
#undef LRS_TILE
  glr_bwd_sums<NW>(g, ch, sum, red, wid, off, cbase, 0, 1);
  if (g.grad_h0)  // past a barrier
    for (int j = threadIdx.x; j < CW; j += NW * kWave)
      if (cbase + j < C) g.grad_h0[cbase + j] = s.y.carry[ntb & 1][j];
}

// Before the tiles of a call: k and dk of every feature, and the look-back state
// reset (one launch for both).
__global__ __launch_bounds__(256) void k_glr_prep(GlrArgs g, float* __restrict__ rates,
                                                  uint4* __restrict__ status, int64_t npairs,
                                                  unsigned* __restrict__ tickets,
                                                  int64_t ntickets) {
  const int64_t stride = (int64_t)gridDim.x * 256;
  const int64_t i0 = (int64_t)blockIdx.x * 256 + threadIdx.x;
  for (int64_t d = i0; d < g.D; d += stride) glr_rates(g, (uint32_t)d, rates[d], rates[g.D + d]);
  const uint4 empty = make_uint4(~0u, ~0u, ~0u, ~0u);  // two status words, not ready
  for (int64_t i = i0; i < npairs; i += stride) status[i] = empty;
  for (int64_t i = i0; i < ntickets; i += stride) tickets[i] = 0u;
}

// ---------------------------------------------------------------------------
// single tokens: element-wise over [B, D], the state's row by its slot.  One thread
// an element: at 64 x 1024 the 256 workgroups take 3.2 us, which is a launch and two
// dependent loads; the caller's side of a call costs four times that.
// ---------------------------------------------------------------------------
template <typename IO>
__global__ __launch_bounds__(256) void k_glr_step(GlrArgs g, const int32_t* __restrict__ slots,
                                                  float* __restrict__ state, int64_t S) {
  const int64_t n = g.B * g.D;
  const int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (e >= n) return;
  const uint32_t b = (uint32_t)e / (uint32_t)g.D, d = (uint32_t)e - b * (uint32_t)g.D;
  const int64_t slot = slots ? slots[b] : (int64_t)b;
  const int64_t z = (int64_t)b * g.ld + d;
  float h = 0.0f;
  if (slot >= 0 && slot < S) {
    const GlrGate q = glr_gate<false>(io_ld((const IO*)g.z_r, z), io_ld((const IO*)g.z_i, z),
                               -kLog2e * g.bias_r[d], -kLog2e * g.bias_i[d],
                               g.c * softplus(g.decay[d]), false);
    float* p = state + slot * g.D + d;
    h = __builtin_fmaf(q.a, *p, q.m * q.i * io_ld((const IO*)g.x, z));
    *p = h;
  }
  io_st((IO*)g.h, e, h);
}

}  // namespace

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
// Two channels a lane where rows and pointers allow pairs; one otherwise (odd
// widths, odd pitches, views that begin at an odd element), which keeps full
// rows of 64 elements: predicated pairs took 26 and 42 us (forward, backward) at
// 1531 x 5 x 517 fp32 against 23 and 35.
// The rows a wave takes, and whether the walk is persistent, do not depend on it:
// a result has the same bits whatever its arrays' alignment.
static bool glr_persist(int64_t C, bool allow) {
  return allow && (C + 2 * kWave - 1) / (2 * kWave) >= persist_min_blocks();
}

ColPlan plan_glr(int64_t C, int64_t T, int io, int cpt, bool allow_persist) {
  const bool persist = glr_persist(C, allow_persist);
  ColPlan p = plan_cols(C, T, 8, io == kIoBf16 && !persist ? 16 : 8, cpt);
  p.persist = persist;
  p.stream = C * T * 4 * io_bytes(io) >= kStreamFootprint;
  return p;
}

ColPlan plan_glr_bwd(int64_t C, int64_t T, int io, int cpt, bool allow_persist) {
  ColPlan p = plan_cols(C, T, 8, 8, cpt);
  p.persist = glr_persist(C, allow_persist);
  p.stream = C * T * 7 * io_bytes(io) >= kStreamFootprint;
  return p;
}

#define LRS_GLR_PICK(LAUNCH)                        \
  if (io == kIoBf16) {                              \
    if (p.stream) {                                 \
      if (g.reset) LAUNCH(uint16_t, true, true)     \
      else LAUNCH(uint16_t, true, false)            \
    } else {                                        \
      if (g.reset) LAUNCH(uint16_t, false, true)    \
      else LAUNCH(uint16_t, false, false)           \
    }                                               \
  } else {                                          \
    if (p.stream) {                                 \
      if (g.reset) LAUNCH(float, true, true)        \
      else LAUNCH(float, true, false)               \
    } else {                                        \
      if (g.reset) LAUNCH(float, false, true)       \
      else LAUNCH(float, false, false)              \
    }                                               \
  }

// status: whole pairs of words, 16-byte aligned.
static hipError_t glr_prep(const GlrArgs& g, const ColPlan& p, float* rates, uint64_t* status,
                           unsigned* tickets, hipStream_t stream) {
  const int64_t npairs = col_status_words(p) / 2;
  int64_t n = npairs > g.D ? npairs : g.D;
  if (p.ncb > n) n = p.ncb;
  int64_t blocks = (n + 255) / 256;
  if (blocks > 2048) blocks = 2048;
  hipLaunchKernelGGL(k_glr_prep, dim3((unsigned)blocks), dim3(256), 0, stream, g, rates,
                     (uint4*)status, npairs, tickets, npairs > 0 ? p.ncb : 0);
  return hipGetLastError();
}

hipError_t launch_glr_fwd(GlrArgs& g, int io, const ColPlan& p, float* rates,
                          uint64_t* status, unsigned* tickets, hipStream_t stream) {
  if (status) {
    const hipError_t e = glr_prep(g, p, rates, status, tickets, stream);
    if (e != hipSuccess) return e;
    g.rates = rates;
  }
  if (p.persist) {
#define LRS_GLR_P(IO, NTF, RSTF)                                                              \
  {                                                                                           \
    if (p.cpt == 2)                                                                           \
      hipLaunchKernelGGL((k_glr_fwd_persist<IO, 8, 8, 2, NTF, RSTF>), dim3((unsigned)p.ncb),  \
                         dim3(512), 0, stream, g);                                            \
    else                                                                                      \
      hipLaunchKernelGGL((k_glr_fwd_persist<IO, 8, 8, 1, NTF, RSTF>), dim3((unsigned)p.ncb),  \
                         dim3(512), 0, stream, g);                                            \
  }
    LRS_GLR_PICK(LRS_GLR_P)
#undef LRS_GLR_P
    return hipGetLastError();
  }
  const dim3 grid((unsigned)(p.ncb * p.ntb));
#define LRS_GLR_F(IO, NTF, RSTF)                                                            \
  {                                                                                         \
    constexpr int L = sizeof(IO) == 2 ? 16 : 8;                                             \
    if (p.cpt == 2)                                                                         \
      hipLaunchKernelGGL((k_glr_fwd<IO, 8, L, 2, NTF, RSTF>), grid, dim3(512), 0, stream,   \
                         g, (int)p.ncb, (int)p.ntb, status, tickets);                       \
    else                                                                                    \
      hipLaunchKernelGGL((k_glr_fwd<IO, 8, L, 1, NTF, RSTF>), grid, dim3(512), 0, stream,   \
                         g, (int)p.ncb, (int)p.ntb, status, tickets);                       \
  }
  LRS_GLR_PICK(LRS_GLR_F)
#undef LRS_GLR_F
  return hipGetLastError();
}

hipError_t launch_glr_bwd(GlrArgs& g, int io, const ColPlan& p, float* rates,
                          uint64_t* status, unsigned* tickets, double* acc, float* grad_bias_r,
                          float* grad_bias_i, float* grad_decay, hipStream_t stream) {
  const hipError_t e0 = glr_prep(g, p, rates, status, tickets, stream);
  if (e0 != hipSuccess) return e0;
  g.rates = rates;
  if (p.persist) {
#define LRS_GLR_Q(IO, NTF, RSTF)                                                              \
  {                                                                                           \
    if (p.cpt == 2)                                                                           \
      hipLaunchKernelGGL((k_glr_bwd_persist<IO, 8, 8, 2, NTF, RSTF>), dim3((unsigned)p.ncb),  \
                         dim3(512), 0, stream, g);                                            \
    else                                                                                      \
      hipLaunchKernelGGL((k_glr_bwd_persist<IO, 8, 8, 1, NTF, RSTF>), dim3((unsigned)p.ncb),  \
                         dim3(512), 0, stream, g);                                            \
  }
    LRS_GLR_PICK(LRS_GLR_Q)
#undef LRS_GLR_Q
  } else {
    const dim3 grid((unsigned)(p.ncb * p.ntb));
#define LRS_GLR_B(IO, NTF, RSTF)                                                             \
  {                                                                                          \
    if (p.cpt == 2)                                                                          \
      hipLaunchKernelGGL((k_glr_bwd<IO, 8, 8, 2, NTF, RSTF>), grid, dim3(512), 0, stream, g, \
                         (int)p.ncb, (int)p.ntb, status, tickets);                           \
    else                                                                                     \
      hipLaunchKernelGGL((k_glr_bwd<IO, 8, 8, 1, NTF, RSTF>), grid, dim3(512), 0, stream, g, \
                         (int)p.ncb, (int)p.ntb, status, tickets);                           \
  }
    LRS_GLR_PICK(LRS_GLR_B)
#undef LRS_GLR_B
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  float* const outs[3] = {grad_bias_r, grad_bias_i, grad_decay};
  return launch_param_sums(g.part, 3, (p.persist ? 1 : p.ntb) * g.B, g.D, acc, outs, stream);
}

hipError_t launch_glr_step(const GlrArgs& g, int io, const int32_t* slots, float* state, int64_t S,
                           hipStream_t stream) {
  const dim3 grid((unsigned)((g.B * g.D + 255) / 256));
  if (io == kIoBf16)
    hipLaunchKernelGGL(k_glr_step<uint16_t>, grid, dim3(256), 0, stream, g, slots, state, S);
  else
    hipLaunchKernelGGL(k_glr_step<float>, grid, dim3(256), 0, stream, g, slots, state, S);
  return hipGetLastError();
}

}  // namespace lrs

// linear_ce.hip -- softmax cross entropy of the logits l = x w^T against one
// class a row, and its gradient, without storing all logits.
//
//   lse_n = log sum_v exp l_nv,  loss_n = lse_n - l_{n,target},
//   G = exp(l - lse) - onehot (0 in ignored rows),
//   grad_x = diag(grad_loss) G w,  grad_w = G^T diag(grad_loss) x.
//
// Three products carry the work, all of the form C[m][n] = sum_k A[m][k] B[n][k]
// (one matrix-core kernel, k_gemm, with two epilogues):
//   logits  m = class, n = row, k = feature, A = w, B = x.  A lane holds one n and
//           32 values of m, so most of the softmax's maximum and sum over classes
//           runs inside a lane.  Each wave leaves the (maximum, sum) of its classes
//           a row, joined afterwards;
//   grad_w  m = class, n = feature, k = row, A = G read by columns, B = x^T;
//   grad_x  m = row, n = feature, k = class, A = G, B = w^T.
// For the gradient the rows are taken in pieces, whose e = exp(l - tile maximum)
// is kept (fp16 for bf16 inputs, fp32 for fp32) until lse is known, turned into G
// by one pass (for bf16 in place), and used up by the two gradient products; the
// piece is chosen so that this stays within a fixed number of bytes.
// What bounds it: the matrix cores' power.  At 16384 x 32768 x 1024 bf16 the
// products run at 1440 (grad_x), 1340 to 1400 (grad_w) and 1000 TFLOP/s (logits, with
// the exponentials) where a large library product reaches 1360 to 1650; the rest, 0.45
// of 3.1 ms, is k_ce_g and the transposed copies at 5.4 to 6 TB/s.
// Operands that are not laid out like that (x^T, w^T, rows that are not a whole
// number of k steps or not 16-byte aligned) are copied once into the workspace.
//
// fp32 operands are two fp16 parts, hi + lo = x to 2^-22, scaled by a power of
// two that brings the row's (x and w as rows) or the array's (transposed) largest
// value near fp16's largest, so that the parts' range is no limit: what is lost
// is 2^-22 of an element or 2^-39 of the largest (for G 2^-50, see kLowLift).  A
// product is the three part products hi hi + hi lo + lo hi (a loop of the same
// kernel over pairs of parts), about as exact as fp32 and, at the matrix cores' fp16
// rate, five times as fast as their fp32 rate.  An infinity has no such parts: it makes
// NaN of its row's or class's logits.
//
// Rounding.  G is rounded to bf16 (two fp16 parts for fp32 inputs) before the
// second and third product: an error of 2^-9 an element with random sign, which
// adds to that of the rounded gradient.  The sum of grad_w runs over rows, so each
// row's grad_loss has to be in one of its factors.  For bf16 G carries the row's
// share grad_loss / max |grad_loss|, and the maximum is applied in fp32 at the end:
// the share of a mean is exactly 1, and the entries that dominate, p - 1 at the
// target, lie next to -1, where they are rounded finely; scaled by a common
// grad_loss, they would all be rounded the same way.  x stays as it is: rounding it
// a second time would cost more than it saves.  For fp32 the two parts of x^T carry
// the share (2^-22 of an element is lost either way) and G none, so that a row with
// a small grad_loss keeps all digits of its grad_x, which is scaled by grad_loss at
// the end.  Keeping e in fp16 (2^-12, see kLift) adds 1% to the error of G in bf16.
#include "lrs_device.hpp"
#include "lrs_internal.hpp"

namespace lrs {

namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x8_t __attribute__((ext_vector_type(8)));
typedef _Float16 f16x2_t __attribute__((ext_vector_type(2)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef short s16x8_t __attribute__((ext_vector_type(8)));

constexpr float kLog2eF = 1.4426950408889634f;
constexpr int kMaxPairs = 3;
// fp32 inputs: G's parts are of G * 2^14, the low one times 2^11 besides, where fp16 has
// digits for it (it is at most 2^-11 of the high one); its partner in the products is the
// other operand's high part over 2^11, a third part of x^T and w^T.  So G, whose elements
// are as small as the classes are rare, is known to 2^-22 or 2^-50, whichever is more,
// where unlifted parts end at 2^-39.
constexpr float kGScale = 16384.0f, kLowLift = 2048.0f;

// What a logits tile leaves besides its maximum and sum.
enum { kKeepNone = 0, kKeepF16 = 1, kKeepF32 = 2 };
// e = 2^kLift exp(l - tile maximum).  fp16 (bf16 inputs) has all of its digits down to
// 2^-14: lifted by 15, a class keeps them to 2^-29 of its tile's largest (20 nats) and
// is 0 from 2^-40 on (27.7 nats).  The largest is a power of two, so that p - 1 of a
// target that is nearly certain loses nothing to fp16.
template <int KEEP>
constexpr float kLift = KEEP == kKeepF16 ? 15.0f : 0.0f;
// Maxima from here on are subtracted from the logits before the exponential's product
// (one instruction a logit): in 2^(l log2 e - mx log2 e) the second product's rounding
// would be an error of 2e-6 of e and grow with mx.
constexpr float kLargeLogit = 32.0f;
enum { kEpiLogits = 0, kEpiOut = 1 };
// How A is stored: [m][k], or [k][m].
enum { kRowsM = 0, kRowsK = 1 };

struct GemmArgs {
  const uint16_t *a, *b;  // [M][lda] (kRowsK: [k][lda]), [N][ldb], bf16 or fp16
  int64_t lda, ldb;
  int64_t M, N;
  int64_t k;                         // of one part, a multiple of 64
  int npair;                         // part products: 1, or 3 for fp32
  int64_t pa[kMaxPairs], pb[kMaxPairs];  // where the pair's parts begin along k
  int tm, tn, splits;                // tiles, and contiguous shares of the k loop
  // logits (m = class, n = row)
  const int64_t* target;
  float2* part;     // [N][tm WM]: maximum and sum of each wave's classes
  float* tlogit;    // [N]: the target's logit
  const float *a_unscale, *b_unscale;  // [M to a whole tile], [N]: powers of two (fp32 operands)
  void* e;          // [N][lde]: 2^kLift exp(l - tile maximum), fp16 or fp32
  int64_t lde;
  // products
  float* slots;        // [splits][M][N] fp32, or null
  int add;             // the slots hold what earlier pieces left: add to it
  int last;            // write out (from the slots too, if add)
  void* out;           // [M][N], I/O type
  int out_bf16;
  const float* row_scale;  // [M] or null
  const float *scale, *unscale;  // one value each, or null
};

// One 16-byte piece a lane from global memory straight to LDS (lane l's piece
// lands at dst + 16 l).  The instruction has no output register; the wait is
// the caller's, by count.  m0 is reserved: the compiler keeps nothing in it from one
// statement to the next (and takes no clobber of it).
__device__ __forceinline__ void dma16(uint32_t dst, uint32_t off, const uint16_t* base) {
  const uint64_t b = (uint64_t)base;
  const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)b);
  const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(b >> 32));
  const uint64_t ub = (uint64_t)hi << 32 | lo;  // wave-uniform, in scalar registers
  asm volatile(
      "s_mov_b32 m0, %0\n\t"
      "s_nop 0\n\t"
      "global_load_lds_dwordx4 %1, %2"
      :
      : "s"(__builtin_amdgcn_readfirstlane(dst)), "v"(off), "s"(ub)
      : "memory");
}

template <int N>
__device__ __forceinline__ void wait_vm() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
}

// Workgroup -> tile.  Workgroups go to the eight dies in turn; each die is
// given a contiguous share of the order, in which groups of eight tiles of m
// are walked across n, so that what runs together on a die shares its rows in
// that die's L2.
__device__ __forceinline__ void tile_of(const GemmArgs& g, int& tm, int& tn, int& split) {
  const unsigned n = gridDim.x;
  unsigned id = blockIdx.x;
  const unsigned q = n / 8, r = n % 8, x = id % 8;
  id = x * q + (x < r ? x : r) + id / 8;
  const unsigned tiles = (unsigned)g.tm * (unsigned)g.tn;
  split = 0;
  if (g.splits > 1) {
    split = (int)(id / tiles);
    id -= (unsigned)split * tiles;
  }
  const unsigned per = 8u * (unsigned)g.tn;
  const unsigned grp = id / per, in = id - grp * per;
  const unsigned left = (unsigned)g.tm - grp * 8u;
  const unsigned gm = left < 8u ? left : 8u;
  tn = (int)(gm == 8u ? in / 8u : in / gm);
  tm = (int)(grp * 8u + in - (unsigned)tn * gm);
}

// The piece of 16 bytes at which piece p of row r is kept in LDS is p ^ swizzle(r):
// the rows that a fragment read touches at once then fall on different banks (rows
// of 128 bytes).  Counted: no conflict; with bit 3 of the row in it as well, four
// of a read's eight cycles (the products take the same time: power bounds them).
__device__ __forceinline__ int swizzle(int r) { return r & 7; }

// A stored as [k][m]: a stage is 64 rows of TM values, in LDS as rows of TM / 16
// blocks of 32 bytes, block c of row r at c ^ swizzle_k(r).  The transposing read
// gives each of 16 lanes one column of four rows that the lanes address together
// (32 bytes of each); two such groups go through the banks at once, rows 0..3 and
// 8..11 or the like, which the swizzle puts on eight different blocks (counted: no conflict).
__device__ __forceinline__ int swizzle_k(int r) {
  return (r & 3) | ((r >> 3) & 1) << 2;
}
__device__ __forceinline__ s16x4_t read_columns(const char* p) {
  typedef __attribute__((address_space(3))) s16x4_t lds_t;
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_t*)p);
}

// The 16x16x32 product: lane l gives 8 values along k of row l % 16, from k =
// 8 (l / 16) on, and holds n = l % 16, m = 4 (l / 16) + 0..3 of the result.
// Written as an instruction that adds in place: through the builtin the register
// allocator rotates hundreds of accumulators by copies in the loop.  Volatile,
// so that products and the loads to LDS keep the order they are written in.
// The wait states between the last product and the first use of a result, which
// the compiler would count for the builtin, are part of mma_last.
template <bool F16>
struct Frag;
template <>
struct Frag<false> {
  typedef bf16x8_t V;
  static __device__ __forceinline__ void mma(V a, V b, f32x4_t& c) {
    asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
  }
  static __device__ __forceinline__ void mma_last(V a, V b, f32x4_t& c) {
    asm volatile("v_mfma_f32_16x16x32_bf16 %0, %1, %2, %0\n\ts_nop 15\n\ts_nop 15"
                 : "+a"(c)
                 : "v"(a), "v"(b));
  }
};
template <>
struct Frag<true> {
  typedef f16x8_t V;
  static __device__ __forceinline__ void mma(V a, V b, f32x4_t& c) {
    asm volatile("v_mfma_f32_16x16x32_f16 %0, %1, %2, %0" : "+a"(c) : "v"(a), "v"(b));
  }
  static __device__ __forceinline__ void mma_last(V a, V b, f32x4_t& c) {
    asm volatile("v_mfma_f32_16x16x32_f16 %0, %1, %2, %0\n\ts_nop 15\n\ts_nop 15"
                 : "+a"(c)
                 : "v"(a), "v"(b));
  }
};

// Tile TM x TN by WM x WN waves, k in stages of 64 (rows of 128 bytes: whole
// cache lines), NA buffers of A's part of a stage and NB of B's.
template <int TM_, int TN_, int WM_, int WN_, int NA_, int NB_, int MINW_>
struct Shape {
  static constexpr int TM = TM_, TN = TN_, WM = WM_, WN = WN_, NA = NA_, NB = NB_, MINW = MINW_;
  static constexpr int kThreads = WM * WN * kWave;
  static constexpr int kStageA = TM * 128, kStageB = TN * 128;
  static constexpr int kLoadsA = TM / 8 / (WM * WN), kLoadsB = TN / 8 / (WM * WN);
  static constexpr int MT = TM / WM / 16, NT = TN / WN / 16;
  static constexpr int kKeep = WM * TN * (TM / WM + 8) * 2;  // an fp16 tile, by wave
  static constexpr int kBuffers = NA * kStageA + NB * kStageB;
  static constexpr int kLds = kBuffers > kKeep ? kBuffers : kKeep;
  static_assert(TM % (8 * WM * WN) == 0 && TN % (8 * WM * WN) == 0 && NB >= 2 && NA == NB + 1,
                "whole loads, and the order of the waits");
};

template <class S, int EPI, int KEEP, bool F16, int ROWS>
__global__ __launch_bounds__(S::kThreads, S::MINW) void k_gemm(GemmArgs g) {
  constexpr int TM = S::TM, TN = S::TN, WM = S::WM, WN = S::WN, NA = S::NA, NB = S::NB;
  constexpr int MT = S::MT, NT = S::NT, LA = S::kLoadsA, LB = S::kLoadsB;
  typedef typename Frag<F16>::V frag_t;
  __shared__ __align__(128) char lds[S::kLds];
  const int lane = threadIdx.x & (kWave - 1);
  const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int wm = wid / WN, wn = wid % WN;
  int tm, tn, split;
  tile_of(g, tm, tn, split);
  const int64_t m0 = (int64_t)tm * TM, n0 = (int64_t)tn * TN;
  const uint16_t* abase = ROWS == kRowsM ? g.a + m0 * g.lda : g.a + m0;
  const int64_t astep = ROWS == kRowsM ? 64 : 64 * g.lda;  // to the next stage
  const uint16_t* bbase = g.b + n0 * g.ldb;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)lds;

  // This lane's global piece of each of the wave's loads (a load fills 1024 bytes,
  // eight rows of 128).  Rows past the end read the last row (their results are
  // not used); rows of m in [k][m] are padded to whole tiles.
  uint32_t offa[LA], offb[LB];
  {
    const int r = lane >> 3, p = lane & 7;
    const int lasta = (int)(g.M - m0) - 1, lastb = (int)(g.N - n0) - 1;
    const uint32_t pitcha = (uint32_t)g.lda * 2u, pitchb = (uint32_t)g.ldb * 2u;
#pragma unroll
    for (int j = 0; j < LA; ++j) {
      if constexpr (ROWS == kRowsK) {
        constexpr int P = TM / 8;  // pieces of 16 bytes in a row
        const int row = (wid * LA + j) * (kWave / P) + lane / P;
        offa[j] = (uint32_t)row * pitcha +
                  (uint32_t)((lane & (P - 1)) ^ swizzle_k(row) << 1) * 16u;
        continue;
      }
      const int row = (wid * LA + j) * 8 + r;
      offa[j] = (uint32_t)(row < lasta ? row : lasta) * pitcha + (uint32_t)(p ^ swizzle(row & 15)) * 16u;
    }
#pragma unroll
    for (int j = 0; j < LB; ++j) {
      const int row = (wid * LB + j) * 8 + r;
      offb[j] = (uint32_t)(row < lastb ? row : lastb) * pitchb + (uint32_t)(p ^ swizzle(row & 15)) * 16u;
    }
  }
  // at most 3 * 2^15 stages, in at most 16 shares
  const unsigned kt = (unsigned)g.k / 64u, total = kt * (unsigned)g.npair;
  int it0 = 0, nk = (int)total, pair0 = 0, k0 = 0;
  if (g.splits > 1) {
    it0 = (int)(total * (unsigned)split / (unsigned)g.splits);
    nk = (int)(total * (unsigned)(split + 1) / (unsigned)g.splits) - it0;
    pair0 = (int)((unsigned)it0 / kt);
    k0 = it0 - pair0 * (int)kt;
  }

  // One operand's walk along k: the address of the next stage to load.
  struct Walk {
    const uint16_t *base, *p;
    int pair, k;
  };
  Walk wa = {abase, abase + g.pa[pair0] + k0 * astep, pair0, k0};
  Walk wb = {bbase, bbase + g.pb[pair0] + k0 * 64, pair0, k0};
  auto advance = [&](Walk& w, const int64_t* parts, int64_t step) __attribute__((always_inline)) {
    w.p += step;
    if (++w.k == (int)kt && ++w.pair < g.npair) {
      w.k = 0;
      w.p = w.base + parts[w.pair];
    }
  };
  auto load_a = [&](int buf, int j) __attribute__((always_inline)) {
    dma16(lds0 + (uint32_t)(buf * S::kStageA + (wid * LA + j) * 1024), offa[j], wa.p);
  };
  auto load_b = [&](int buf, int j) __attribute__((always_inline)) {
    dma16(lds0 + (uint32_t)(NA * S::kStageA + buf * S::kStageB + (wid * LB + j) * 1024), offb[j],
          wb.p);
  };

  f32x4_t acc[MT][NT];

  // Pipeline.  A stage is two steps of 32 along k.  The fragments of a step are
  // read while the step before it is multiplied, also across the border of two
  // stages: before a stage's second step its own reads are complete and the next
  // stage has landed; one barrier makes both true for all waves, its buffers are
  // filled again and the products go on from registers.  B's loads are begun
  // right after the barrier, A's in the first step of the stage after it: A has
  // one buffer more, because it is the operand that streams from memory (B's
  // rows are shared by all tiles of m and come from the caches).
  // A step is MT chunks of NT products, each with its share of the fragment
  // reads and of the loads; the compiler is kept from moving anything between
  // chunks (it would put the reads next to their use, and the loads in front of
  // all products, where their addresses queue up).
  frag_t af[2][MT], bf[2][NT];
  // fragment addresses: row lane % 16 of a block of 16, piece 4 kk + lane / 16
  const int fr = lane & 15, fsw = swizzle(fr);
  const int fa = (wm * (TM / WM) + fr) * 128;
  // A as [k][m]: row 8 (lane / 16) + (lane % 16) / 4 of a step, 8 bytes a lane
  const int fk = (lane >> 4) * 8 + (fr >> 2);
  const int fb = NA * S::kStageA + (wn * (TN / WN) + fr) * 128;
  // Fragment reads of a chunk: all of B come first, since the first chunk of the
  // next step needs every one of them; A's are needed one a chunk.
  auto read_share = [&](int bufa, int bufb, int kk, int set, int j) __attribute__((always_inline)) {
    constexpr int R = MT + NT;
    const int pc = ((kk * 4 + (lane >> 4)) ^ fsw) * 16;
    const char* sa = lds + bufa * S::kStageA + fa + pc;
    const char* sb = lds + bufb * S::kStageB + fb + pc;
#pragma unroll
    for (int r = R * j / MT; r < R * (j + 1) / MT; ++r) {
      if (r < NT) {
        bf[set][r] = *reinterpret_cast<const frag_t*>(sb + r * 2048);
      } else if constexpr (ROWS == kRowsM) {
        af[set][r - NT] = *reinterpret_cast<const frag_t*>(sa + (r - NT) * 2048);
      } else {
        // four rows (of k) a read; the swizzle of a row and of the row 4 on are the same
        const char* sk = lds + bufa * S::kStageA + (kk * 32 + fk) * (TM * 2) + (fr & 3) * 8 +
                         ((wm * (TM / WM / 16) + r - NT) ^ swizzle_k(fk)) * 32;
        const s16x4_t lo = read_columns(sk), hi = read_columns(sk + 4 * TM * 2);
        const s16x8_t both = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        af[set][r - NT] = __builtin_bit_cast(frag_t, both);
      }
    }
  };
  auto multiply = [&](int set, int j, bool last) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < NT; ++q) {
      if (last && q == NT - 1) Frag<F16>::mma_last(af[set][j], bf[set][q], acc[j][q]);
      else Frag<F16>::mma(af[set][j], bf[set][q], acc[j][q]);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  // B's loads go into the first chunks of their step
  constexpr int CB = MT > 2 ? MT / 2 : MT;
  // buffers of the current stage, and A's of the one before it
  int ca = 0, cb = 0, oa = NA - 1;
  // one stage; `fill`: the buffers that are freed are filled again (A's with the
  // stage NA after the one before, B's with the stage NB after this one: the
  // same stage, since NA = NB + 1)
  auto body = [&](auto fill) __attribute__((always_inline)) {
    const int na = ca == NA - 1 ? 0 : ca + 1, nb = cb == NB - 1 ? 0 : cb + 1;
#pragma unroll
    for (int j = 0; j < MT; ++j) {
      read_share(ca, cb, 1, 1, j);
      if (fill) {
#pragma unroll
        for (int l = LA * j / MT; l < LA * (j + 1) / MT; ++l) load_a(oa, l);
      }
      multiply(0, j, false);
    }
    // the next stage has landed; begun after its last load: an A, and NB - 2 stages
    if (fill) wait_vm<LA + (NB - 2) * (LA + LB)>();
    else wait_vm<0>();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
#pragma unroll
    for (int j = 0; j < MT; ++j) {
      read_share(na, nb, 0, 0, j);  // past the last stage: read and not used
      if (fill && j < CB) {
#pragma unroll
        for (int l = LB * j / CB; l < LB * (j + 1) / CB; ++l) load_b(cb, l);
      }
      multiply(1, j, !fill && j == MT - 1);  // a stage without loads may be the last
    }
    if (fill) {
      advance(wa, g.pa, astep);
      advance(wb, g.pb, 64);
    }
    oa = ca;
    ca = na;
    cb = nb;
  };
  // Before the first stage, in the order in which the stages before it would
  // have begun them: A 0; B 0, A 1; B 1, A 2; ...; B NB-1 (A NB follows in the
  // first step).
#pragma unroll
  for (int s = 0; s < NB; ++s) {
    if (s < nk) {
#pragma unroll
      for (int j = 0; j < LA; ++j) load_a(s, j);
      advance(wa, g.pa, astep);
#pragma unroll
      for (int j = 0; j < LB; ++j) load_b(s, j);
      advance(wb, g.pb, 64);
    }
  }
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[i][j] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
  // stage 0 has landed: begun after it, NB - 1 stages
  if (nk >= NB) wait_vm<(NB - 1) * (LA + LB)>();
  else wait_vm<0>();
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
#pragma unroll
  for (int j = 0; j < MT; ++j) read_share(0, 0, 0, 0, j);
  struct Yes { __device__ constexpr operator bool() const { return true; } };
  struct No { __device__ constexpr operator bool() const { return false; } };
  int i = 0;
  for (; i + NB < nk; ++i) body(Yes());
  for (; i < nk; ++i) body(No());
  __syncthreads();  // the epilogues reuse the buffers

  // The lane's values: n = nb + 16 q, m = mb + 16 j + e.
  const int ln = wn * (TN / WN) + (lane & 15);
  const int lm = wm * (TM / WM) + 4 * (lane >> 4);
  const int64_t nb = n0 + ln, mb = m0 + lm;
  const int mleft = (int)(g.M - mb < 16 * MT ? g.M - mb : 16 * MT);  // <= 0: none

  if constexpr (EPI == kEpiLogits) {
    // A wave's classes are a tile of the softmax of their own: no wave waits for
    // another, and every logit is taken from its accumulator once.
    constexpr int PG = TM / WM + 8;   // a padded row of e in LDS, the wave's own
    constexpr int RP = TM / WM / 8;   // pieces of 16 bytes in such a row
    uint16_t* keep = reinterpret_cast<uint16_t*>(lds) + wid * NT * 16 * PG;
    const bool whole = m0 + TM <= g.M;
    const int64_t wave = (int64_t)tm * WM + wm, waves = (int64_t)g.tm * WM;
    f32x4_t au[F16 ? MT : 1];
    if constexpr (F16) {
      // past the last class: room of the workspace, masked below
#pragma unroll
      for (int j = 0; j < MT; ++j) au[j] = *reinterpret_cast<const f32x4_t*>(g.a_unscale + mb + 16 * j);
    }
#pragma unroll
    for (int q = 0; q < NT; ++q) {
      const int64_t n = nb + 16 * q;
      f32x4_t v[MT];
      const float bu = F16 && n < g.N ? g.b_unscale[n] : 0.0f;
#pragma unroll
      for (int j = 0; j < MT; ++j) {
        asm volatile("" : "+a"(acc[j][q]));  // not read earlier: 128 values would not fit
        v[j] = acc[j][q];
        if constexpr (F16) v[j] = v[j] * bu * au[j];
      }
      // the target's place among the lane's classes (it has those with bits 2 and 3 clear)
      const int64_t d = (n < g.N ? g.target[n] : -1) - mb;
      const int at = d >= 0 && d < mleft && (d & 12) == 0 ? (int)d : -1;
      if (__ballot(at >= 0)) {  // few tiles hold the target of one of 16 rows
        float tl = 0.0f;
#pragma unroll
        for (int j = 0; j < MT; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (16 * j + e == at) tl = v[j][e];
        if (at >= 0) g.tlogit[n] = tl;
      }
      if (!whole) {
        int left = mleft;
        asm volatile("" : "+v"(left));  // 32 masks kept for all q would not fit
#pragma unroll
        for (int j = 0; j < MT; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (16 * j + e >= left) v[j][e] = -__builtin_inff();
      }
      float mx = -__builtin_inff();
#pragma unroll
      for (int j = 0; j < MT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) mx = fmaxf(mx, v[j][e]);
      mx = fmaxf(mx, __shfl_xor(mx, 16));
      mx = fmaxf(mx, __shfl_xor(mx, 32));
      // no class, or every logit -inf: all e are 0
      float ref = mx == -__builtin_inff() ? 0.0f : mx;
      if (__ballot(fabsf(ref) >= kLargeLogit)) {  // for those rows of the 16 alone
        const float take = fabsf(ref) >= kLargeLogit ? ref : 0.0f;
#pragma unroll
        for (int j = 0; j < MT; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) v[j][e] -= take;
        ref -= take;
      }
      const float lift = __builtin_fmaf(-ref, kLog2eF, kLift<KEEP>);
      float sum = 0.0f;
#pragma unroll
      for (int j = 0; j < MT; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[j][e] = __builtin_amdgcn_exp2f(__builtin_fmaf(v[j][e], kLog2eF, lift));
          sum += v[j][e];
        }
      sum += __shfl_xor(sum, 16);
      sum += __shfl_xor(sum, 32);
      // the sum to mx itself: without the lift as the exponents had it, rounding and all
      sum *= __builtin_amdgcn_exp2f(-__builtin_fmaf(ref, kLog2eF, lift));
      if (lane < 16 && n < g.N) g.part[n * waves + wave] = make_float2(mx, sum);
      if constexpr (KEEP == kKeepF16) {
        uint16_t* mine = keep + q * 16 * PG;
#pragma unroll
        for (int j = 0; j < MT; ++j) {
          const f16x2_t lo = {(_Float16)v[j][0], (_Float16)v[j][1]};
          const f16x2_t hi = {(_Float16)v[j][2], (_Float16)v[j][3]};
          *reinterpret_cast<u32x2_t*>(mine + (lane & 15) * PG + 4 * (lane >> 4) + 16 * j) =
              u32x2_t{__builtin_bit_cast(uint32_t, lo), __builtin_bit_cast(uint32_t, hi)};
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        // whole rows of the wave's classes, so that full cache lines are written
#pragma unroll
        for (int c = lane; c < 16 * RP; c += kWave) {
          const int r = c / RP, k = c % RP * 8;
          const int64_t row = n0 + wn * (TN / WN) + 16 * q + r;
          if (row < g.N)
            *reinterpret_cast<u32x4_t*>((uint16_t*)g.e + row * g.lde + m0 + wm * (TM / WM) + k) =
                *reinterpret_cast<const u32x4_t*>(mine + r * PG + k);
        }
      }
      if constexpr (KEEP == kKeepF32) {
        if (n < g.N) {
          float* o = (float*)g.e + n * g.lde + mb;
#pragma unroll
          for (int j = 0; j < MT; ++j) *reinterpret_cast<f32x4_t*>(o + 16 * j) = v[j];
        }
      }
      __builtin_amdgcn_sched_barrier(0);  // one q's values at a time
    }
  }

  if constexpr (EPI == kEpiOut) {
    const float sc = (g.scale ? *g.scale : 1.0f), un = g.unscale ? *g.unscale : 1.0f;
    const bool slot = g.slots != nullptr;
#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int dm = 16 * j + e;
        if (dm >= mleft) continue;
        const int64_t m = mb + dm;
        const float rs = g.row_scale ? g.row_scale[m] : sc;
#pragma unroll
        for (int q = 0; q < NT; ++q) {
          const int64_t n = nb + 16 * q;
          if (n >= g.N) continue;
          float v = acc[j][q][e] * un;
          float* p = g.slots + ((int64_t)split * g.M + m) * g.N + n;
          if (slot && g.add) v += *p;
          if (g.last) {
            // a scale of 0 (an ignored row) is a gradient of 0 whatever v is
            v = rs == 0.0f ? 0.0f : v * rs;
            if (g.out_bf16) io_st((uint16_t*)g.out, m * g.N + n, v);
            else ((float*)g.out)[m * g.N + n] = v;
          } else {
            *p = v;
          }
        }
      }
  }
}

// ---- small kernels -----------------------------------------------------------

__device__ __forceinline__ bool row_counts(int64_t t, int64_t V) { return t >= 0 && t < V; }

// A value as the products take it: bf16 unchanged, fp32 as two fp16 parts.
__device__ __forceinline__ uint16_t f16_bits(float v) {
  return __builtin_bit_cast(uint16_t, (_Float16)v);
}
template <int P>
__device__ __forceinline__ void split_parts(float v, uint16_t (&p)[P], float low_lift = 1.0f) {
  if constexpr (P == 1) {
    p[0] = (uint16_t)(pack_bf16x2(v, 0.0f) & 0xFFFFu);
  } else {
    p[0] = f16_bits(v);
    p[1] = f16_bits((v - (float)__builtin_bit_cast(_Float16, p[0])) * low_lift);
  }
}

// The power of two that brings values up to `top` to at most 2^14, and its
// inverse (1 for 0, infinities and NaN).
__device__ __forceinline__ float scale_for(float top, float& inverse) {
  int e = (int)((as_u32(top) >> 23) & 255) - 127;  // top = 1.x * 2^e
  const bool ok = top > 0.0f && e < 128;
  e = ok ? 13 - e : 0;
  e = e < -126 ? -126 : e > 126 ? 126 : e;
  inverse = as_f32((uint32_t)(127 - e) << 23);
  return as_f32((uint32_t)(127 + e) << 23);
}

__device__ __forceinline__ float wave_top(float v) {
#pragma unroll
  for (int o = kWave / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o));
  return v;
}

// bf16 [rows][D] -> [rows][Dp], zero past D; one wave a row, two values a lane and
// four such pairs in flight (rows of an odd D are aligned to one value).
__global__ __launch_bounds__(256) void k_ce_rows_bf16(const uint16_t* __restrict__ src,
                                                      uint16_t* __restrict__ dst, int64_t rows,
                                                      int64_t D, int64_t Dp) {
  const int lane = threadIdx.x & (kWave - 1);
  for (int64_t row = (int64_t)blockIdx.x * 4 + threadIdx.x / kWave; row < rows;
       row += (int64_t)gridDim.x * 4) {
    const uint16_t* s = src + row * D;
    for (int64_t d0 = 2 * lane; d0 < Dp; d0 += 8 * kWave) {
      uint32_t v[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t d = d0 + i * 2 * kWave;
        v[i] = (d < D ? (uint32_t)s[d] : 0u) | (d + 1 < D ? (uint32_t)s[d + 1] << 16 : 0u);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t d = d0 + i * 2 * kWave;
        if (d < Dp) *reinterpret_cast<uint32_t*>(dst + row * Dp + d) = v[i];
      }
    }
  }
}

// fp32 [rows][D] -> two fp16 parts [rows][2][Dp] scaled by the row's power of
// two; unscale[row] undoes it and top[row] is the row's largest finite value, times its
// `share` of the gradient if there are shares: what the transposed copy will hold of the
// row (0 where the share is 0, whatever the row holds).  One wave a row.
__global__ __launch_bounds__(256) void k_ce_rows_f32(const float* __restrict__ src,
                                                     const float* __restrict__ shares,
                                                     uint16_t* __restrict__ dst,
                                                     float* __restrict__ unscale,
                                                     float* __restrict__ top_out, int64_t rows,
                                                     int64_t D, int64_t Dp) {
  const int lane = threadIdx.x & (kWave - 1);
  for (int64_t row = (int64_t)blockIdx.x * 4 + threadIdx.x / kWave; row < rows;
       row += (int64_t)gridDim.x * 4) {
    float top = 0.0f, finite = 0.0f;
    for (int64_t d = lane; d < D; d += kWave) {
      const float v = fabsf(src[row * D + d]);
      top = fmaxf(top, v);
      finite = fmaxf(finite, v < __builtin_inff() ? v : 0.0f);
    }
    top = wave_top(top);
    finite = wave_top(finite);
    float inv;
    const float sc = scale_for(top, inv);
    for (int64_t d = lane; d < Dp; d += kWave) {
      uint16_t p[2];
      split_parts<2>(d < D ? src[row * D + d] * sc : 0.0f, p);
      dst[row * 2 * Dp + d] = p[0];
      dst[(row * 2 + 1) * Dp + d] = p[1];
    }
    if (lane == 0) {
      unscale[row] = inv;
      const float share = shares ? fabsf(shares[row]) : 1.0f;
      top_out[row] = share > 0.0f && share < __builtin_inff() ? finite * share : 0.0f;
    }
  }
}

// The largest of top[0 .. n), as a scale for a whole array: scale[0] and
// scale[1] / kGScale, which undoes it and G's.  One workgroup.
__global__ __launch_bounds__(1024) void k_ce_top(const float* __restrict__ top, int64_t n,
                                                 float* __restrict__ scale) {
  __shared__ float red[16];
  float v = 0.0f;
  for (int64_t i = threadIdx.x; i < n; i += 1024) v = fmaxf(v, top[i]);
  v = wave_top(v);
  if ((threadIdx.x & (kWave - 1)) == 0) red[threadIdx.x / kWave] = v;
  __syncthreads();
  if (threadIdx.x == 0) {
    v = red[0];
    for (int w = 1; w < 16; ++w) v = fmaxf(v, red[w]);
    float inv;
    scale[0] = scale_for(v, inv);
    scale[1] = inv / kGScale;
  }
}

// [rows][D] -> [D][P][Rp] (row pitch ld), zero past `rows`; two-part rows have the high
// part over kLowLift as a third.  With `ratio`, rows whose share of the gradient is 0 are
// zero too, whatever they hold, and two-part rows are multiplied by their share.
template <typename IO, int P>
__global__ __launch_bounds__(256) void k_ce_cols(const IO* __restrict__ src,
                                                 const float* __restrict__ ratio,
                                                 const float* __restrict__ scale,
                                                 uint16_t* __restrict__ dst, int64_t rows,
                                                 int64_t D, int64_t Rp, int64_t ld) {
  __shared__ float tile[64][65];
  const int64_t r0 = (int64_t)blockIdx.x * 64, d0 = (int64_t)blockIdx.y * 64;
  const int tx = threadIdx.x & 63, ty = threadIdx.x >> 6;
  const float sc = P == 1 ? 1.0f : *scale;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int64_t r = r0 + ty + 4 * i, d = d0 + tx;
    bool ok = r < rows && d < D;
    float share = 1.0f;
    if (ok && ratio) {
      share = ratio[r];
      ok = share != 0.0f;
    }
    tile[ty + 4 * i][tx] = ok ? io_ld(src, r * D + d) * (P == 1 ? 1.0f : sc * share) : 0.0f;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int64_t d = d0 + ty + 4 * i, r = r0 + tx;
    if (d < D && r < Rp) {
      uint16_t p[P];
      split_parts<P>(tile[tx][ty + 4 * i], p);
#pragma unroll
      for (int k = 0; k < P; ++k) dst[d * ld + k * Rp + r] = p[k];
      if constexpr (P == 2)
        dst[d * ld + 2 * Rp + r] =
            f16_bits((float)__builtin_bit_cast(_Float16, p[0]) * (1.0f / kLowLift));
    }
  }
}

// One wave a row: the tiles' maxima and sums become lse, and the loss.  One pass,
// four loads in flight a lane (two passes of single loads: 8.2 us against 3.9 for
// 32 rows of 1000 tiles).
__global__ __launch_bounds__(256) void k_ce_join(const float2* __restrict__ part,
                                                 const float* __restrict__ tlogit,
                                                 const int64_t* __restrict__ target,
                                                 float* __restrict__ loss, float* __restrict__ lse,
                                                 int64_t N, int64_t V, int64_t tiles) {
  const int lane = threadIdx.x & (kWave - 1);
  const int64_t n = (int64_t)blockIdx.x * 4 + threadIdx.x / kWave;
  if (n >= N) return;
  const float2* p = part + n * tiles;
  const float low = -__builtin_inff();
  // (maximum, sum) of what was seen; a maximum of -inf means a sum of 0
  auto base = [&](float t) { return t == low ? 0.0f : t; };
  float top = low, sum = 0.0f;
  for (int64_t t0 = lane; t0 < tiles; t0 += 4 * kWave) {
    float2 v[4];
    float next = top;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = t0 + i * kWave < tiles ? p[t0 + i * kWave] : make_float2(low, 0.0f);
      next = fmaxf(next, v[i].x);
    }
    sum *= __builtin_amdgcn_exp2f((top - base(next)) * kLog2eF);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      sum += v[i].y * __builtin_amdgcn_exp2f((v[i].x - base(next)) * kLog2eF);
    top = next;
  }
  const float mine = top;
  top = wave_top(top);
  sum *= __builtin_amdgcn_exp2f((mine - base(top)) * kLog2eF);
#pragma unroll
  for (int o = kWave / 2; o > 0; o >>= 1) sum += __shfl_xor(sum, o);
  if (lane == 0) {
    const float l = top + logf(sum);
    lse[n] = l;
    loss[n] = row_counts(target[n], V) ? l - tlogit[n] : 0.0f;
  }
}

// top = the largest finite |grad_loss| of the rows that count (1 if that is 0), each
// row's share grad_loss / top, and what its grad_x is multiplied by in the end: top
// where G carries the share, else grad_loss; 0 in rows without a gradient.  One
// workgroup.
__global__ __launch_bounds__(1024) void k_ce_scale(const float* __restrict__ grad_loss,
                                                   const int64_t* __restrict__ target, int64_t N,
                                                   int64_t V, int shared,
                                                   float* __restrict__ ratio,
                                                   float* __restrict__ row_scale,
                                                   float* __restrict__ top_out) {
  __shared__ float red[16];
  float top = 0.0f;
#pragma unroll 8
  for (int64_t n = threadIdx.x; n < N; n += 1024) {
    const int64_t t = target[n];
    const float g = grad_loss[n], v = row_counts(t, V) ? fabsf(g) : 0.0f;
    top = fmaxf(top, v < __builtin_inff() ? v : 0.0f);
  }
  top = wave_top(top);
  if ((threadIdx.x & (kWave - 1)) == 0) red[threadIdx.x / kWave] = top;
  __syncthreads();
  top = red[0];
#pragma unroll
  for (int w = 1; w < 16; ++w) top = fmaxf(top, red[w]);
  if (top == 0.0f) top = 1.0f;
#pragma unroll 8
  for (int64_t n = threadIdx.x; n < N; n += 1024) {
    const int64_t t = target[n];
    const float g = grad_loss[n], v = row_counts(t, V) ? g : 0.0f;
    row_scale[n] = v == 0.0f ? 0.0f : shared ? top : v;
    ratio[n] = v == 0.0f ? 0.0f : v / top;
  }
  if (threadIdx.x == 0) *top_out = top;
}

// Memory bound: 355 us for 1 GiB of e in bf16's case, 6.0 TB/s.
// e -> G [rows][P][Vp] (row pitch ldg), per_row workgroups a row; rows up to the next
// multiple of 64 are written as 0, as are rows whose `share` is 0, whatever their e
// holds.  bf16 (P 1): over e's own fp16 values, G multiplied by the row's share.
// fp32 (P 2): two parts of G itself, share only tells the rows without a gradient.
// Classes of padding hold e = 0.
template <typename E, int P>
__global__ __launch_bounds__(256) void k_ce_g(const E* e, int64_t lde, const float2* __restrict__ part,
                                              int64_t tiles, int tile_m,
                                              const float* __restrict__ lse,
                                              const int64_t* __restrict__ target,
                                              const float* __restrict__ shares, uint16_t* g,
                                              int64_t ldg, int64_t rows, int64_t Vp,
                                              unsigned per_row) {
  const int64_t n = blockIdx.x / per_row;
  const int64_t t = n < rows ? target[n] : -1;
  const float share = n < rows ? shares[n] : 0.0f;
  const float own = share == 0.0f ? 0.0f : lse[n];
  const float gs = P == 1 ? share : kGScale;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t v = ((int64_t)(blockIdx.x % per_row) * 512 + i * 256 + threadIdx.x) * 8;
    if (v >= Vp) return;
    uint32_t q[P][4] = {};
    if (share != 0.0f && v < tiles * tile_m) {
      // eight classes lie inside one tile of the logits
      const float f = __builtin_amdgcn_exp2f(
          __builtin_fmaf(part[n * tiles + v / tile_m].x - own, kLog2eF, -kLift<P == 1 ? kKeepF16 : kKeepF32>));
      float ev[8];
      if constexpr (sizeof(E) == 2) {
        const u32x4_t w = *reinterpret_cast<const u32x4_t*>(e + n * lde + v);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint32_t wk = w[k];  // a bit cast of an element takes the vector's first
          const f16x2_t h = __builtin_bit_cast(f16x2_t, wk);
          ev[2 * k] = (float)h.x;
          ev[2 * k + 1] = (float)h.y;
        }
      } else {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const f32x4_t w = *reinterpret_cast<const f32x4_t*>(e + n * lde + v + 4 * k);
#pragma unroll
          for (int j = 0; j < 4; ++j) ev[4 * k + j] = w[j];
        }
      }
      const int64_t at = t - v;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint16_t lo[P], hi[P];
        split_parts<P>(__builtin_fmaf(ev[2 * k], f, at == 2 * k ? -1.0f : 0.0f) * gs, lo, kLowLift);
        split_parts<P>(__builtin_fmaf(ev[2 * k + 1], f, at == 2 * k + 1 ? -1.0f : 0.0f) * gs, hi,
                       kLowLift);
#pragma unroll
        for (int m = 0; m < P; ++m) q[m][k] = (uint32_t)lo[m] | (uint32_t)hi[m] << 16;
      }
    }
#pragma unroll
    for (int m = 0; m < P; ++m)
      *reinterpret_cast<u32x4_t*>(g + n * ldg + m * Vp + v) =
          u32x4_t{q[m][0], q[m][1], q[m][2], q[m][3]};
  }
}

// out[m][n] = scale of the row (or of all) times the sum of the slots, in order.
__global__ __launch_bounds__(256) void k_ce_join_slots(const float* __restrict__ slots, int splits,
                                                       int64_t M, int64_t N,
                                                       const float* __restrict__ row_scale,
                                                       const float* __restrict__ scale,
                                                       void* __restrict__ out, int out_bf16) {
  const int64_t n = M * N;
  const int64_t stride = (int64_t)gridDim.x * 256;
  for (int64_t e = (int64_t)blockIdx.x * 256 + threadIdx.x; e < n; e += stride) {
    float v = slots[e];
    for (int s = 1; s < splits; ++s) v += slots[(int64_t)s * n + e];
    const float sc = row_scale ? row_scale[e / N] : *scale;
    v = sc == 0.0f ? 0.0f : v * sc;
    if (out_bf16) io_st((uint16_t*)out, e, v);
    else ((float*)out)[e] = v;
  }
}

// Zero bytes, an even number of them from an even address: whole words, and what lies
// before and behind them.
__global__ __launch_bounds__(256) void k_ce_zero(uint16_t* __restrict__ p, int64_t bytes) {
  const int64_t n = bytes / 2, head = ((uintptr_t)p & 2) ? 1 : 0, words = (n - head) / 2;
  const int64_t stride = (int64_t)gridDim.x * 256;
  const int64_t i0 = (int64_t)blockIdx.x * 256 + threadIdx.x;
  uint32_t* w = reinterpret_cast<uint32_t*>(p + head);
  for (int64_t i = i0; i < words; i += stride) w[i] = 0u;
  if (i0 == 0 && head) p[0] = 0;
  if (i0 == 0 && head + 2 * words < n) p[n - 1] = 0;
}

int64_t up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

unsigned blocks_for(int64_t n, int64_t per) {
  const int64_t b = (n + per - 1) / per;
  return (unsigned)(b < 1 ? 1 : b > 65536 ? 65536 : b);
}

// The tile shapes, with what a product of many tiles of it reaches (TFLOP/s, by
// which they are compared, measured at 8192 x 1024 x 32768) and the workgroups a compute unit holds: 256
// x 256 by eight waves of 128 x 64 fills the LDS alone; the others are for
// products with few tiles, where the largest would leave compute units idle.
typedef Shape<256, 256, 2, 4, 3, 2, 2> Large;
typedef Shape<128, 128, 2, 2, 3, 2, 2> Medium;
typedef Shape<128, 64, 4, 1, 3, 2, 2> Small;
struct ShapeInfo {
  int tm, tn, wm, wgs;
  double tflops;
};
constexpr ShapeInfo kShapes[3] = {{Large::TM, Large::TN, Large::WM, 1, 1150.0},
                                  {Medium::TM, Medium::TN, Medium::WM, 2, 880.0},
                                  {Small::TM, Small::TN, Small::WM, 2, 600.0}};

int64_t tiles_of(int64_t M, int64_t N, const ShapeInfo& s) {
  return up(M, s.tm) / s.tm * (up(N, s.tn) / s.tn);
}

// The shape, and for the gradients the number of shares of the k loop, with the
// least estimated time: rounds of workgroups at the shape's rate, and 8 bytes of
// every fp32 partial result at the memory's.
void choose(int64_t M, int64_t N, int64_t K, int most_splits, int* shape, int64_t* splits) {
  double best = 0.0;
  for (int i = 0; i < 3; ++i) {
    const ShapeInfo& s = kShapes[i];
    const int64_t tiles = tiles_of(M, N, s), slots = 256 * s.wgs;
    for (int64_t n = 1; n <= most_splits && (n == 1 || K / n >= 512); n *= 2) {
      const int64_t rounds = (tiles * n + slots - 1) / slots;
      const double k = (double)((K + n - 1) / n + 192);  // and the pipeline's start
      double t = rounds * s.wgs * 2.0 * s.tm * s.tn * k / (s.tflops * 1e12 / 256);
      if (n > 1) t += 8.0 * n * M * N / 4e12 + 3e-6;
      if (best == 0.0 || t < best) {
        best = t;
        *shape = i;
        *splits = n;
      }
    }
  }
}

template <class S, int EPI, int KEEP, int ROWS, bool F16>
hipError_t run_gemm(GemmArgs& g, hipStream_t stream) {
  g.tm = (int)(up(g.M, S::TM) / S::TM);
  g.tn = (int)(up(g.N, S::TN) / S::TN);
  hipLaunchKernelGGL((k_gemm<S, EPI, KEEP, F16, ROWS>),
                     dim3((unsigned)((int64_t)g.tm * g.tn * g.splits)), dim3(S::kThreads), 0, stream,
                     g);
  return hipGetLastError();
}

// What e is kept as goes with the operands' type.
template <class S, int EPI, int KEEP, int ROWS>
hipError_t run_shape(GemmArgs& g, bool f16, hipStream_t stream) {
  if constexpr (KEEP == kKeepF16) return run_gemm<S, EPI, KEEP, ROWS, false>(g, stream);
  else if constexpr (KEEP == kKeepF32) return run_gemm<S, EPI, KEEP, ROWS, true>(g, stream);
  else
    return f16 ? run_gemm<S, EPI, KEEP, ROWS, true>(g, stream)
               : run_gemm<S, EPI, KEEP, ROWS, false>(g, stream);
}

template <int EPI, int KEEP, int ROWS = kRowsM>
hipError_t run(GemmArgs& g, int shape, bool f16, hipStream_t stream) {
  switch (shape) {
    case 0: return run_shape<Large, EPI, KEEP, ROWS>(g, f16, stream);
    case 1: return run_shape<Medium, EPI, KEEP, ROWS>(g, f16, stream);
    default: return run_shape<Small, EPI, KEEP, ROWS>(g, f16, stream);
  }
}

}  // namespace

// Pieces of the rows whose G takes at most this many bytes.  Every piece adds its
// part to an fp32 grad_w, so fewer are faster, and each takes its bytes of workspace.
// Training in ms with 256 MiB, 512 MiB, 1, 2 and 4 GiB: 16384 x 32768 x 1024 bf16 3.66,
// 3.29, 3.12 (one piece from here on); 32768 x 50021 x 512 bf16 8.65, 7.91, 6.57, 6.46,
// 6.49; 16384 x 50021 x 512 fp32 11.3, 10.2, 8.74, 8.42, 8.50; 65536 x 131072 x 1024
// bf16 88.7, 66.8, 56.2, 51.6, 50.5.  1 GiB is where most of it is gained; the last, of 16
// pieces, is 8% from its best.
constexpr int64_t kCePieceBytes = (int64_t)1 << 30;

CePlan plan_ce(int64_t N, int64_t V, int64_t D, int io) {
  CePlan p;
  p.parts = io == kIoBf16 ? 1 : 2;
  p.Dp = up(D, 64);
  p.Vp = up(V, 256);
  const int64_t most = kCePieceBytes / (p.Vp * 2 * p.parts) / 256 * 256;
  const int64_t cap = most < 256 ? 256 : most;
  const int64_t pieces = (N + cap - 1) / cap;
  p.piece = up((N + pieces - 1) / pieces, 256);
  p.pieces = (N + p.piece - 1) / p.piece;
  // 128 bytes past a power of two: rows a power of two apart would meet in few
  // of the cache's channels
  const int64_t parts_b = p.parts == 1 ? 1 : 3;
  p.ldg = p.parts * p.Vp + 64;
  p.ldw = parts_b * p.Vp + 64;
  p.ldx = parts_b * p.piece + 64;
  // the forward's only growing array is (maximum, sum) of each tile and row: pieces
  // of rows for it too (128 MiB at 128 classes a tile, and the shapes with smaller
  // tiles are only chosen for so few rows that they stay below; each still fills the GPU)
  const int64_t most_f = (kCePieceBytes / 8) / (p.Vp / 128 * 8) / 256 * 256;
  p.piece_f = most_f < 256 ? 256 : most_f > N ? N : most_f;
  int64_t one;
  const int64_t K = p.Dp * (p.parts == 1 ? 1 : 3);
  choose(V, p.piece_f < N ? p.piece_f : N, K, 1, &p.shape_f, &one);
  choose(V, p.piece < N ? p.piece : N, K, 1, &p.shape_l, &one);
  // a tile of the softmax is a wave's classes
  const ShapeInfo &sf = kShapes[p.shape_f], &sl = kShapes[p.shape_l];
  p.tm_l = sl.tm / sl.wm;
  p.tiles_f = up(V, sf.tm) / sf.tm * sf.wm;
  p.tiles_l = up(V, sl.tm) / p.tm_l;
  const int64_t n = p.piece < N ? p.piece : N, f = p.parts == 1 ? 1 : 3;
  choose(n, D, up(V, 64) * f, 16, &p.shape_x, &p.split_x);
  choose(V, D, up(n, 64) * f, 16, &p.shape_w, &p.split_w);
  p.slots_x = p.split_x > 1;
  p.slots_w = p.split_w > 1 || p.pieces > 1;
  return p;
}

hipError_t launch_linear_ce(const CePlan& p, const CeArgs& a, int io, hipStream_t stream) {
  const bool bf = io == kIoBf16;
  const int64_t es = bf ? 2 : 4;
  hipError_t e = hipSuccess;
#define LRS_CE(call)               \
  do {                             \
    e = (call);                    \
    if (e != hipSuccess) return e; \
  } while (0)
  GemmArgs base = {};
  base.npair = bf ? 1 : 3;
  // smallest products first: lo hi, hi lo, hi hi; lifted: A's low part is lifted, and
  // multiplied by B's third part
  auto pairs = [&](GemmArgs& g, int64_t ka, int64_t kb, int64_t k, bool lifted) {
    if (!bf) {
      g.pa[0] = ka;
      g.pb[0] = lifted ? 2 * kb : 0;
      g.pb[1] = kb;
    }
    g.k = k;
  };
  base.splits = 1;
  // rows of x and w as the logits' product takes them
  const uint16_t *xr = (const uint16_t*)a.x, *wr = (const uint16_t*)a.w;
  auto rows = [&](const void* src, uint16_t* dst, int64_t n, const float* shares, float* unscale,
                  float* top, const uint16_t** out) -> hipError_t {
    if (bf && p.Dp == a.D && ((uintptr_t)src & 15) == 0) return hipSuccess;
    *out = dst;
    if (bf)
      hipLaunchKernelGGL(k_ce_rows_bf16, dim3(blocks_for(n, 4)), dim3(256), 0, stream,
                         (const uint16_t*)src, dst, n, a.D, p.Dp);
    else
      hipLaunchKernelGGL(k_ce_rows_f32, dim3(blocks_for(n, 4)), dim3(256), 0, stream,
                         (const float*)src, shares, dst, unscale, top, n, a.D, p.Dp);
    return hipGetLastError();
  };
  if (a.backward) {  // first: the shares enter the scale of x^T
    hipLaunchKernelGGL(k_ce_scale, dim3(1), dim3(1024), 0, stream, a.grad_loss, a.target, a.N, a.V,
                       bf ? 1 : 0, a.ratio, a.row_scale, a.top);
    LRS_CE(hipGetLastError());
  }
  LRS_CE(rows(a.x, a.x_rows, a.N, a.backward ? a.ratio : nullptr, a.x_unscale, a.x_top, &xr));
  LRS_CE(rows(a.w, a.w_rows, a.V, nullptr, a.w_unscale, a.w_top, &wr));
  auto logits = [&](int64_t n0, int64_t n) {
    GemmArgs g = base;
    g.a = wr;
    g.b = xr + n0 * p.parts * p.Dp;
    g.lda = g.ldb = p.parts * p.Dp;
    g.M = a.V;
    g.N = n;
    g.target = a.target + n0;
    g.part = a.part;
    g.tlogit = a.tlogit;  // of this piece's rows
    g.a_unscale = a.w_unscale;
    g.b_unscale = a.x_unscale + n0;
    g.e = a.e;
    g.lde = a.lde;
    pairs(g, p.Dp, p.Dp, p.Dp, false);
    return g;
  };
  auto join = [&](int64_t n0, int64_t n, int64_t tiles) {
    hipLaunchKernelGGL(k_ce_join, dim3((unsigned)((n + 3) / 4)), dim3(256), 0, stream, a.part,
                       a.tlogit, a.target + n0, a.loss + n0, a.lse + n0, n, a.V, tiles);
    return hipGetLastError();
  };
  if (!a.backward) {
    for (int64_t n0 = 0; n0 < a.N; n0 += p.piece_f) {
      const int64_t n = a.N - n0 < p.piece_f ? a.N - n0 : p.piece_f;
      GemmArgs g = logits(n0, n);
      LRS_CE((run<kEpiLogits, kKeepNone>(g, p.shape_f, !bf, stream)));
      LRS_CE(join(n0, n, p.tiles_f));
    }
    return hipSuccess;
  }
  if (!bf) {
    hipLaunchKernelGGL(k_ce_top, dim3(1), dim3(1024), 0, stream, a.x_top, a.N, a.x_scale);
    LRS_CE(hipGetLastError());
    hipLaunchKernelGGL(k_ce_top, dim3(1), dim3(1024), 0, stream, a.w_top, a.V, a.w_scale);
    LRS_CE(hipGetLastError());
  }
  auto cols = [&](const void* src, const float* ratio, const float* scale, uint16_t* dst,
                  int64_t n, int64_t np, int64_t ld) -> hipError_t {
    const dim3 grid((unsigned)(up(np, 64) / 64), (unsigned)(up(a.D, 64) / 64));
    if (bf)
      hipLaunchKernelGGL((k_ce_cols<uint16_t, 1>), grid, dim3(256), 0, stream, (const uint16_t*)src,
                         ratio, scale, dst, n, a.D, np, ld);
    else
      hipLaunchKernelGGL((k_ce_cols<float, 2>), grid, dim3(256), 0, stream, (const float*)src,
                         ratio, scale, dst, n, a.D, np, ld);
    return hipGetLastError();
  };
  LRS_CE(cols(a.w, nullptr, a.w_scale, a.w_cols, a.V, p.Vp, p.ldw));
  for (int64_t n0 = 0; n0 < a.N; n0 += p.piece) {
    const int64_t n = a.N - n0 < p.piece ? a.N - n0 : p.piece;
    const bool last = n0 + n == a.N;
    GemmArgs l = logits(n0, n);
    LRS_CE(bf ? (run<kEpiLogits, kKeepF16>(l, p.shape_l, false, stream))
              : (run<kEpiLogits, kKeepF32>(l, p.shape_l, true, stream)));
    if (a.forward) LRS_CE(join(n0, n, p.tiles_l));
    const int tile_m = p.tm_l;
    const unsigned per_row = (unsigned)(up(p.Vp, 4096) / 4096);
    const dim3 gg(per_row * (unsigned)up(n, 64));
    if (bf)
      hipLaunchKernelGGL((k_ce_g<uint16_t, 1>), gg, dim3(256), 0, stream, (const uint16_t*)a.e,
                         a.lde, a.part, p.tiles_l, tile_m, a.lse + n0, a.target + n0, a.ratio + n0,
                         a.g, p.ldg, n, p.Vp, per_row);
    else
      hipLaunchKernelGGL((k_ce_g<float, 2>), gg, dim3(256), 0, stream, (const float*)a.e, a.lde,
                         a.part, p.tiles_l, tile_m, a.lse + n0, a.target + n0, a.row_scale + n0,
                         a.g, p.ldg, n, p.Vp, per_row);
    LRS_CE(hipGetLastError());
    LRS_CE(cols((const char*)a.x + n0 * a.D * es, a.ratio + n0, a.x_scale, a.x_cols, n, p.piece,
                p.ldx));
    {
      GemmArgs g = base;
      g.a = a.g;
      g.b = a.x_cols;
      g.lda = p.ldg;
      g.ldb = p.ldx;
      g.M = a.V;
      g.N = a.D;
      pairs(g, p.Vp, p.piece, up(n, 64), true);
      g.splits = (int)p.split_w;
      g.slots = p.slots_w ? a.slots_w : nullptr;
      g.add = n0 > 0;
      g.last = last && p.split_w == 1;
      g.out = a.grad_w;
      g.out_bf16 = bf;
      g.scale = a.top;
      g.unscale = bf ? nullptr : a.x_scale + 1;
      LRS_CE((run<kEpiOut, kKeepNone, kRowsK>(g, p.shape_w, !bf, stream)));
    }
    {
      GemmArgs g = base;
      g.a = a.g;
      g.b = a.w_cols;
      g.lda = p.ldg;
      g.ldb = p.ldw;
      g.M = n;
      g.N = a.D;
      pairs(g, p.Vp, p.Vp, up(a.V, 64), true);
      g.splits = (int)p.split_x;
      g.slots = p.slots_x ? a.slots_x : nullptr;
      g.last = p.split_x == 1;
      g.out = (char*)a.grad_x + n0 * a.D * es;
      g.out_bf16 = bf;
      g.row_scale = a.row_scale + n0;
      g.unscale = bf ? nullptr : a.w_scale + 1;
      LRS_CE((run<kEpiOut, kKeepNone>(g, p.shape_x, !bf, stream)));
      if (p.split_x > 1) {
        hipLaunchKernelGGL(k_ce_join_slots, dim3(blocks_for(n * a.D, 1024)), dim3(256), 0, stream,
                           a.slots_x, (int)p.split_x, n, a.D, a.row_scale + n0, nullptr, g.out,
                           bf ? 1 : 0);
        LRS_CE(hipGetLastError());
      }
    }
  }
  if (p.split_w > 1) {
    hipLaunchKernelGGL(k_ce_join_slots, dim3(blocks_for(a.V * a.D, 1024)), dim3(256), 0, stream,
                       a.slots_w, (int)p.split_w, a.V, a.D, nullptr, a.top, a.grad_w, bf ? 1 : 0);
    LRS_CE(hipGetLastError());
  }
#undef LRS_CE
  return hipSuccess;
}

hipError_t launch_zero(void* p, int64_t bytes, hipStream_t stream) {
  if (bytes <= 0) return hipSuccess;
  hipLaunchKernelGGL(k_ce_zero, dim3(blocks_for(bytes, 4096)), dim3(256), 0, stream, (uint16_t*)p,
                     bytes);
  return hipGetLastError();
}

}  // namespace lrs

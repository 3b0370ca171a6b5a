// linear_ce.hip -- softmax cross entropy of the logits l = x w^T against one
// class a row, and its gradient, without storing the logits.
//
//   lse_n = log sum_v exp l_nv,  loss_n = lse_n - l_{n,target},
//   G = exp(l - lse) - onehot (0 in ignored rows),
//   grad_x = diag(grad_loss) G w,  grad_w = G^T diag(grad_loss) x.
//
// Three products carry the work, all of the form C[m][n] = sum_k A[m][k] B[n][k]
// with both operands contiguous along k (one matrix-core kernel, k_gemm, with
// three epilogues):
//   logits  m = class, n = row, k = feature, A = w, B = x.  A lane of the
//           32x32 product holds one n and 16 values of m, so the softmax's
//           maximum and sum over classes run inside a lane.  The forward leaves
//           (maximum, sum) of each 256-class tile and row, joined afterwards;
//           the backward makes the logits again and writes G and G^T of one
//           piece of the vocabulary, rounded to bf16, through LDS;
//   grad_w  m = class, n = feature, k = row, A = G^T, B = x^T;
//   grad_x  m = row, n = feature, k = class, A = G, B = w^T.
// Operands that are not laid out like that (x^T, w^T, rows that are not a whole
// number of 32-wide steps or not 16-byte aligned) are copied once into the
// workspace.
//
// fp32 operands are three bf16 parts, hi + mid + lo = x to 2^-24, side by side
// along k, and a product is the six part products of order up to 2^-16 (a loop
// of the same kernel over pairs of parts): the vector fp32 rate of the matrix
// cores is 1/16 of the bf16 rate, so six bf16 products cost less than half.
//
// Rounding.  G is rounded to bf16 before the second and third product (its
// error, 2^-9 an element with random sign, adds to that of the rounded
// gradient).  It is rounded unscaled, where the entries that dominate, p - 1 at
// the target, lie next to -1: scaled by a common grad_loss, they would all be
// rounded the same way.  grad_x is scaled by row in fp32 afterwards.  grad_w's
// sum runs over rows, so G^T carries grad_loss / max |grad_loss| (exactly 1 for
// a mean) and the maximum is applied in fp32 at the end.
#include "lrs_device.hpp"
#include "lrs_internal.hpp"

namespace lrs {

namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));

constexpr float kLog2eF = 1.4426950408889634f;
constexpr int kBK = 32;  // k a step: rows of 64 bytes in LDS
constexpr int kMaxPairs = 6;

enum { kEpiLse = 0, kEpiGrad = 1, kEpiOut = 2 };

struct GemmArgs {
  const uint16_t *a, *b;  // [M][lda], [N][ldb], bf16
  int64_t lda, ldb;
  int64_t M, N;
  int kt;                         // steps of 32 along k, of one part
  int npair;                      // part products: 1, or 6 for fp32
  int pa[kMaxPairs], pb[kMaxPairs];  // where the pair's parts begin along k
  int tm, tn, splits;             // tiles, and contiguous shares of the k loop
  // logits (m = class v0 + m, n = row)
  const int64_t* target;
  int64_t v0, V;
  float2* part;     // [N][part_ld]: maximum and sum of each class tile
  int64_t part_ld, part0;
  float* tlogit;    // [N]: the target's logit
  const float* lse;
  const float* ratio;  // [N]: grad_loss / max |grad_loss|, 0 where ignored
  uint16_t *g, *gt;    // G [N][ldg], G^T [M][ldgt], parts side by side
  int64_t ldg, ldgt;
  int nparts;
  int64_t part_k, part_kt;  // a part's length along k in g and gt
  // products
  float* slots;        // [splits][M][N] fp32, or null: straight to out
  int accumulate;      // add to the slots
  void* out;           // [M][N], I/O type
  int out_bf16;
  const float* row_scale;  // [M] or null
  const float* scale;      // one value, or null
};

// One 16-byte piece a lane from global memory straight to LDS (lane l's piece
// lands at dst + 16 l).  The instruction has no output register; the wait is
// the caller's, by count.
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

// Where a row's target lies from the lane's first class on (m = class v0 + m);
// out of the lane's reach: -1.  An ignored target never matches.
__device__ __forceinline__ int class_at(int64_t t, const GemmArgs& g, int64_t mb) {
  const int64_t d = t - g.v0 - mb;
  return t >= 0 && t < g.V && d >= 0 && d < 1024 ? (int)d : -1;
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
  split = (int)(id / tiles);
  id %= tiles;
  const unsigned per = 8u * (unsigned)g.tn;
  const unsigned grp = id / per, in = id % per;
  const unsigned left = (unsigned)g.tm - grp * 8u;
  const unsigned gm = left < 8u ? left : 8u;
  tm = (int)(grp * 8u + in % gm);
  tn = (int)(in / gm);
}

template <int TM, int TN, int WM, int WN, int NST, int EPI>
struct GemmCfg {
  static constexpr int kThreads = WM * WN * kWave;
  static constexpr int kRows = TM + TN;
  static constexpr int kStage = kRows * kBK * 2;  // bytes
  static constexpr int kIssue = kRows / 16 / (WM * WN);
  static constexpr int MT = TM / WM / 32, NT = TN / WN / 32;
  static constexpr int kStageG = TN * (TM + 8) * 2, kStageGt = TM * (TN + 8) * 2;
  static constexpr int kLds =
      NST * kStage > (kStageG > kStageGt ? kStageG : kStageGt)
          ? NST * kStage
          : (kStageG > kStageGt ? kStageG : kStageGt);
  static_assert(kRows % (16 * WM * WN) == 0, "whole loads");
};

template <int TM, int TN, int WM, int WN, int NST, int EPI>
__global__ __launch_bounds__(WM* WN* kWave, 2) void k_gemm(GemmArgs g) {
  using Cfg = GemmCfg<TM, TN, WM, WN, NST, EPI>;
  constexpr int MT = Cfg::MT, NT = Cfg::NT, NI = Cfg::kIssue;
  __shared__ __align__(128) char lds[Cfg::kLds];
  const int lane = threadIdx.x & (kWave - 1);
  const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int wm = wid / WN, wn = wid % WN;
  int tm, tn, split;
  tile_of(g, tm, tn, split);
  const int64_t m0 = (int64_t)tm * TM, n0 = (int64_t)tn * TN;
  const uint16_t* abase = g.a + m0 * g.lda;
  const uint16_t* bbase = g.b + n0 * g.ldb;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)lds;

  // This lane's global piece of each of the wave's loads.  A load fills 16 rows
  // of 64 bytes; the four 16-byte pieces of row r are stored in the order
  // piece ^ f(r), f(r) = ((r >> 1) & 3) ^ ((r >> 3) & 1), so that the 8 (or 16)
  // rows that a fragment read touches at once fall on different banks.  Rows
  // past the end read the last row (their results are not used).
  uint32_t voff[NI];
  {
    const int r = lane >> 2;
    const uint32_t piece = (uint32_t)((lane & 3) ^ ((r >> 1) & 3) ^ ((r >> 3) & 1));
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      const int row = (wid * NI + j) * 16 + r;
      const bool isb = (wid * NI + j) * 16 >= TM;
      const int64_t last = (isb ? g.N - n0 : g.M - m0) - 1;
      int64_t rr = isb ? row - TM : row;
      rr = rr < last ? rr : last;
      voff[j] = (uint32_t)(rr * (isb ? g.ldb : g.lda) * 2) + piece * 16u;
    }
  }
  const int total = g.kt * g.npair;
  const int it0 = (int)((int64_t)total * split / g.splits);
  const int nk = (int)((int64_t)total * (split + 1) / g.splits) - it0;

  int ipair = it0 / g.kt, ik = it0 % g.kt;  // the next step to load
  auto issue = [&](int stage) {
    const uint16_t* ap = abase + g.pa[ipair] + ik * kBK;
    const uint16_t* bp = bbase + g.pb[ipair] + ik * kBK;
    const uint32_t dst = lds0 + (uint32_t)(stage * Cfg::kStage);
#pragma unroll
    for (int j = 0; j < NI; ++j) {
      const int idx = wid * NI + j;
      dma16(dst + (uint32_t)idx * 1024u, voff[j], idx * 16 >= TM ? bp : ap);
    }
    if (++ik == g.kt) {
      ik = 0;
      ++ipair;
    }
  };

  f32x16_t acc[MT][NT];
#pragma unroll
  for (int i = 0; i < MT; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;

  // fragment addresses: row lane % 32 of a 32-row block, piece 2 kk + lane / 32
  const int fr = lane & 31;
  const int fsw = ((fr >> 1) & 3) ^ ((fr >> 3) & 1);
  const int fa = (wm * (TM / WM) + fr) * 64, fb = (TM + wn * (TN / WN) + fr) * 64;

#pragma unroll
  for (int s = 0; s < NST - 1; ++s)
    if (s < nk) issue(s);
  int stage = 0;
  for (int i = 0; i < nk; ++i) {
    // this step's loads have landed (the later steps' may be in flight), and
    // every wave has finished reading the buffer that is filled next
    if (i + NST - 2 < nk) wait_vm<NI*(NST - 2)>();
    else wait_vm<0>();
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    if (i + NST - 1 < nk) issue(stage == 0 ? NST - 1 : stage - 1);
    const char* st = lds + stage * Cfg::kStage;
#pragma unroll
    for (int kk = 0; kk < 2; ++kk) {
      const int pc = ((kk * 2 + (lane >> 5)) ^ fsw) * 16;
      bf16x8_t af[MT], bf[NT];
#pragma unroll
      for (int j = 0; j < NT; ++j)
        bf[j] = *reinterpret_cast<const bf16x8_t*>(st + fb + j * 32 * 64 + pc);
#pragma unroll
      for (int j = 0; j < MT; ++j)
        af[j] = *reinterpret_cast<const bf16x8_t*>(st + fa + j * 32 * 64 + pc);
#pragma unroll
      for (int j = 0; j < MT; ++j)
#pragma unroll
        for (int q = 0; q < NT; ++q)
          acc[j][q] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(af[j], bf[q], acc[j][q], 0, 0, 0);
    }
    stage = stage == NST - 1 ? 0 : stage + 1;
  }
  __syncthreads();  // the epilogues reuse the buffers

  // The lane's values: n = nb + 32 q, m = mb + 32 j + 8 (e / 4) + e % 4.
  const int ln = wn * (TN / WN) + (lane & 31);
  const int lm = wm * (TM / WM) + 4 * (lane >> 5);
  const int64_t nb = n0 + ln, mb = m0 + lm;
  const int mleft = (int)(g.M - mb < 32 * MT ? g.M - mb : 32 * MT);  // classes left (<= 0: none)

  if constexpr (EPI == kEpiLse) {
    float2* red = reinterpret_cast<float2*>(lds);  // [WM][TN]
#pragma unroll
    for (int q = 0; q < NT; ++q) {
      const int64_t n = nb + 32 * q;
      const int at = class_at(n < g.N ? g.target[n] : -1, g, mb);
      float mx = -__builtin_inff(), tl = 0.0f;
#pragma unroll
      for (int j = 0; j < MT; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int m = 32 * j + 8 * (e / 4) + e % 4;
          if (m >= mleft) acc[j][q][e] = -__builtin_inff();
          mx = fmaxf(mx, acc[j][q][e]);
          if (m == at) tl = acc[j][q][e];
        }
      if (at >= 0 && at < 32 * MT && (at & 4) == 0) g.tlogit[n] = tl;
      float sum = 0.0f;
      if (mx > -__builtin_inff()) {
#pragma unroll
        for (int j = 0; j < MT; ++j)
#pragma unroll
          for (int e = 0; e < 16; ++e)
            sum += __builtin_amdgcn_exp2f((acc[j][q][e] - mx) * kLog2eF);
      }
      const float mx2 = __shfl_xor(mx, 32), sum2 = __shfl_xor(sum, 32);
      const float top = fmaxf(mx, mx2);
      float all = 0.0f;
      if (sum > 0.0f || sum != sum) all += sum * __builtin_amdgcn_exp2f((mx - top) * kLog2eF);
      if (sum2 > 0.0f || sum2 != sum2) all += sum2 * __builtin_amdgcn_exp2f((mx2 - top) * kLog2eF);
      if (lane < 32) red[wm * TN + ln + 32 * q] = make_float2(top, all);
    }
    __syncthreads();
    for (int c = threadIdx.x; c < TN; c += Cfg::kThreads) {
      if (n0 + c >= g.N) continue;
      float top = -__builtin_inff(), all = 0.0f;
#pragma unroll
      for (int w = 0; w < WM; ++w) top = fmaxf(top, red[w * TN + c].x);
#pragma unroll
      for (int w = 0; w < WM; ++w) {
        const float2 v = red[w * TN + c];
        if (v.y > 0.0f || v.y != v.y) all += v.y * __builtin_amdgcn_exp2f((v.x - top) * kLog2eF);
      }
      g.part[(n0 + c) * g.part_ld + g.part0 + tm] = make_float2(top, all);
    }
  }

  if constexpr (EPI == kEpiGrad) {
    constexpr int PG = TM + 8, PT = TN + 8;  // padded rows in LDS
    uint16_t* sg = reinterpret_cast<uint16_t*>(lds);
    float ratio[NT];
#pragma unroll
    for (int q = 0; q < NT; ++q) {
      const int64_t n = nb + 32 * q;
      const bool in = n < g.N;
      const int64_t t = in ? g.target[n] : -1;
      const bool counts = t >= 0 && t < g.V;
      const float l2 = counts ? g.lse[n] * kLog2eF : 0.0f;
      const int at = class_at(t, g, mb), mend = counts ? mleft : 0;
      ratio[q] = in ? g.ratio[n] : 0.0f;
#pragma unroll
      for (int j = 0; j < MT; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          const int m = 32 * j + 8 * (e / 4) + e % 4;
          float p = __builtin_amdgcn_exp2f(__builtin_fmaf(acc[j][q][e], kLog2eF, -l2));
          if (m == at) p -= 1.0f;
          acc[j][q][e] = m < mend ? p : 0.0f;
        }
    }
    for (int part = 0; part < g.nparts; ++part) {
      // G: rows of n, TM classes each.  The residue of this part stays in acc.
#pragma unroll
      for (int q = 0; q < NT; ++q)
#pragma unroll
        for (int j = 0; j < MT; ++j)
#pragma unroll
          for (int e4 = 0; e4 < 4; ++e4) {
            const u32x2_t w = {pack_bf16x2(acc[j][q][4 * e4], acc[j][q][4 * e4 + 1]),
                               pack_bf16x2(acc[j][q][4 * e4 + 2], acc[j][q][4 * e4 + 3])};
            *reinterpret_cast<u32x2_t*>(sg + (ln + 32 * q) * PG + lm + 32 * j + 8 * e4) = w;
          }
      __syncthreads();
      for (int c = threadIdx.x; c < TN * (TM / 8); c += Cfg::kThreads) {
        const int r = c / (TM / 8), k = c % (TM / 8) * 8;
        if (n0 + r < g.N)
          *reinterpret_cast<u32x4_t*>(g.g + (n0 + r) * g.ldg + part * g.part_k + m0 + k) =
              *reinterpret_cast<const u32x4_t*>(sg + r * PG + k);
      }
      if (g.nparts > 1) {
#pragma unroll
        for (int q = 0; q < NT; ++q)
#pragma unroll
          for (int j = 0; j < MT; ++j)
#pragma unroll
            for (int e = 0; e < 16; ++e)
              acc[j][q][e] -= bf16_lo(pack_bf16x2(acc[j][q][e], 0.0f));
      }
      __syncthreads();
    }
    if (g.nparts > 1) {
      // the residue is spent: p once more from what was written would round
      // twice, so the parts of G^T are split from the sum of G's three
      // parts (exact in fp32)
      for (int c = threadIdx.x; c < TM * TN; c += Cfg::kThreads) {
        const int n = c / TM, m = c % TM;
        if (n0 + n < g.N && m0 + m < g.M) {
          const uint16_t* p = g.g + (n0 + n) * g.ldg + m0 + m;
          float v = io_ld(p, 0) + io_ld(p, g.part_k) + io_ld(p, 2 * g.part_k);
          v *= g.ratio[n0 + n];
          uint16_t* o = g.gt + (m0 + m) * g.ldgt + n0 + n;
          for (int part = 0; part < 3; ++part) {
            io_st(o, part * g.part_kt, v);
            v -= bf16_lo(pack_bf16x2(v, 0.0f));
          }
        } else if (m0 + m < g.M) {
          uint16_t* o = g.gt + (m0 + m) * g.ldgt + n0 + n;
          for (int part = 0; part < 3; ++part) o[part * g.part_kt] = 0;
        }
      }
    } else {
      // G^T: rows of m, TN rows of x each
#pragma unroll
      for (int q = 0; q < NT; ++q)
#pragma unroll
        for (int j = 0; j < MT; ++j)
#pragma unroll
          for (int e = 0; e < 16; ++e)
            io_st(sg, (lm + 32 * j + 8 * (e / 4) + e % 4) * PT + ln + 32 * q,
                  acc[j][q][e] * ratio[q]);
      __syncthreads();
      for (int c = threadIdx.x; c < TM * (TN / 8); c += Cfg::kThreads) {
        const int r = c / (TN / 8), k = c % (TN / 8) * 8;
        if (m0 + r < g.M)
          *reinterpret_cast<u32x4_t*>(g.gt + (m0 + r) * g.ldgt + n0 + k) =
              *reinterpret_cast<const u32x4_t*>(sg + r * PT + k);
      }
    }
  }

  if constexpr (EPI == kEpiOut) {
    const float sc = g.scale ? *g.scale : 1.0f;
#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int64_t m = mb + 32 * j + 8 * (e / 4) + e % 4;
        if (m >= g.M) continue;
        const float rs = g.slots ? 1.0f : g.row_scale ? g.row_scale[m] : sc;
#pragma unroll
        for (int q = 0; q < NT; ++q) {
          const int64_t n = nb + 32 * q;
          if (n >= g.N) continue;
          float v = acc[j][q][e];
          if (g.slots) {
            float* p = g.slots + ((int64_t)split * g.M + m) * g.N + n;
            *p = g.accumulate ? *p + v : v;
          } else {
            // a scale of 0 (an ignored row) is a gradient of 0 whatever v is
            v = rs == 0.0f ? 0.0f : v * rs;
            if (g.out_bf16) io_st((uint16_t*)g.out, m * g.N + n, v);
            else ((float*)g.out)[m * g.N + n] = v;
          }
        }
      }
  }
}

// ---- small kernels -----------------------------------------------------------

// bf16 parts of v, most significant first.
template <int P>
__device__ __forceinline__ void split_parts(float v, uint16_t (&p)[P]) {
#pragma unroll
  for (int i = 0; i < P; ++i) {
    p[i] = (uint16_t)(pack_bf16x2(v, 0.0f) & 0xFFFFu);
    v -= as_f32((uint32_t)p[i] << 16);
  }
}

// [rows][D] -> bf16 [rows][P * Dp], zero past D.
template <typename IO, int P>
__global__ __launch_bounds__(256) void k_ce_pack(const IO* __restrict__ src,
                                                 uint16_t* __restrict__ dst, int64_t rows,
                                                 int64_t D, int64_t Dp) {
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x)
    for (int64_t d = threadIdx.x; d < Dp; d += 256) {
      uint16_t p[P];
      split_parts<P>(d < D ? io_ld(src, row * D + d) : 0.0f, p);
#pragma unroll
      for (int i = 0; i < P; ++i) dst[(row * P + i) * Dp + d] = p[i];
    }
}

// [rows][D] -> bf16 [D][P * Rp], zero past `rows` and in ignored rows (whatever
// they hold).
template <typename IO, int P>
__global__ __launch_bounds__(256) void k_ce_pack_t(const IO* __restrict__ src,
                                                   const int64_t* __restrict__ target, int64_t V,
                                                   uint16_t* __restrict__ dst, int64_t rows,
                                                   int64_t D, int64_t Rp) {
  __shared__ float tile[64][65];
  const int64_t r0 = (int64_t)blockIdx.x * 64, d0 = (int64_t)blockIdx.y * 64;
  const int tx = threadIdx.x & 63, ty = threadIdx.x >> 6;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int64_t r = r0 + ty + 4 * i, d = d0 + tx;
    bool ok = r < rows && d < D;
    if (ok && target) ok = target[r] >= 0 && target[r] < V;
    tile[ty + 4 * i][tx] = ok ? io_ld(src, r * D + d) : 0.0f;
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const int64_t d = d0 + ty + 4 * i, r = r0 + tx;
    if (d < D && r < Rp) {
      uint16_t p[P];
      split_parts<P>(tile[tx][ty + 4 * i], p);
#pragma unroll
      for (int k = 0; k < P; ++k) dst[(d * P + k) * Rp + r] = p[k];
    }
  }
}

// One wave a row: the tiles' maxima and sums become lse, and the loss.
__global__ __launch_bounds__(256) void k_ce_join(const float2* __restrict__ part,
                                                 const float* __restrict__ tlogit,
                                                 const int64_t* __restrict__ target,
                                                 float* __restrict__ loss, float* __restrict__ lse,
                                                 int64_t N, int64_t V, int64_t tiles) {
  const int lane = threadIdx.x & (kWave - 1);
  const int64_t n = (int64_t)blockIdx.x * 4 + threadIdx.x / kWave;
  if (n >= N) return;
  const float2* p = part + n * tiles;
  float top = -__builtin_inff(), sum = 0.0f;
  for (int64_t t = lane; t < tiles; t += kWave) top = fmaxf(top, p[t].x);
#pragma unroll
  for (int o = kWave / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
  for (int64_t t = lane; t < tiles; t += kWave)
    sum += p[t].y * __builtin_amdgcn_exp2f((p[t].x - top) * kLog2eF);
#pragma unroll
  for (int o = kWave / 2; o > 0; o >>= 1) sum += __shfl_xor(sum, o);
  if (lane == 0) {
    const float l = top + logf(sum);
    lse[n] = l;
    const int64_t t = target[n];
    loss[n] = t >= 0 && t < V ? l - tlogit[n] : 0.0f;
  }
}

// max |grad_loss| over the rows that count, and each row's share of it.  One
// workgroup.
__global__ __launch_bounds__(1024) void k_ce_scale(const float* __restrict__ grad_loss,
                                                   const int64_t* __restrict__ target, int64_t N,
                                                   int64_t V, float* __restrict__ ratio,
                                                   float* __restrict__ row_scale,
                                                   float* __restrict__ top_out) {
  __shared__ float red[16];
  float top = 0.0f;
  for (int64_t n = threadIdx.x; n < N; n += 1024) {
    const bool ok = target[n] >= 0 && target[n] < V;
    if (ok) top = fmaxf(top, fabsf(grad_loss[n]));
  }
#pragma unroll
  for (int o = kWave / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor(top, o));
  if ((threadIdx.x & (kWave - 1)) == 0) red[threadIdx.x / kWave] = top;
  __syncthreads();
  top = red[0];
#pragma unroll
  for (int w = 1; w < 16; ++w) top = fmaxf(top, red[w]);
  for (int64_t n = threadIdx.x; n < N; n += 1024) {
    const bool ok = target[n] >= 0 && target[n] < V;
    const float v = ok ? grad_loss[n] : 0.0f;
    row_scale[n] = v;
    ratio[n] = v == 0.0f ? 0.0f : v / top;
  }
  if (threadIdx.x == 0) *top_out = top;
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

__global__ __launch_bounds__(256) void k_ce_zero(uint32_t* __restrict__ p, int64_t bytes) {
  const int64_t stride = (int64_t)gridDim.x * 256;
  const int64_t i0 = (int64_t)blockIdx.x * 256 + threadIdx.x;
  for (int64_t i = i0; i < bytes / 4; i += stride) p[i] = 0u;
  if (i0 == 0 && (bytes & 2)) reinterpret_cast<uint16_t*>(p)[bytes / 2 - 1] = 0;
}

int64_t up(int64_t v, int64_t to) { return (v + to - 1) / to * to; }

unsigned blocks_for(int64_t n, int64_t per) {
  const int64_t b = (n + per - 1) / per;
  return (unsigned)(b < 1 ? 1 : b > 65536 ? 65536 : b);
}

// The two tile shapes: 256 x 128 with four waves of 128 x 64, three buffers,
// two workgroups a compute unit; and 128 x 64 for products with few tiles.
constexpr int kBigM = 256, kBigN = 128, kSmallM = 128, kSmallN = 64;

int64_t tiles_of(int64_t M, int64_t N, bool big) {
  return big ? up(M, kBigM) / kBigM * (up(N, kBigN) / kBigN)
             : up(M, kSmallM) / kSmallM * (up(N, kSmallN) / kSmallN);
}
bool use_big(int64_t M, int64_t N) { return tiles_of(M, N, true) >= 256; }

template <int EPI>
hipError_t run_gemm(GemmArgs& g, bool big, hipStream_t stream) {
  g.tm = (int)(up(g.M, big ? kBigM : kSmallM) / (big ? kBigM : kSmallM));
  g.tn = (int)(up(g.N, big ? kBigN : kSmallN) / (big ? kBigN : kSmallN));
  const dim3 grid((unsigned)((int64_t)g.tm * g.tn * g.splits));
  if (big)
    hipLaunchKernelGGL((k_gemm<kBigM, kBigN, 2, 2, 3, EPI>), grid, dim3(256), 0, stream, g);
  else
    hipLaunchKernelGGL((k_gemm<kSmallM, kSmallN, 4, 1, 6, EPI>), grid, dim3(256), 0, stream, g);
  return hipGetLastError();
}

template <typename IO, int P>
hipError_t pack(const void* src, uint16_t* dst, int64_t rows, int64_t D, int64_t Dp,
                hipStream_t stream) {
  hipLaunchKernelGGL((k_ce_pack<IO, P>), dim3(blocks_for(rows, 1)), dim3(256), 0, stream,
                     (const IO*)src, dst, rows, D, Dp);
  return hipGetLastError();
}
template <typename IO, int P>
hipError_t pack_t(const void* src, const int64_t* target, int64_t V, uint16_t* dst, int64_t rows,
                  int64_t D, int64_t Rp, hipStream_t stream) {
  hipLaunchKernelGGL((k_ce_pack_t<IO, P>),
                     dim3((unsigned)(up(Rp, 64) / 64), (unsigned)(up(D, 64) / 64)), dim3(256), 0,
                     stream, (const IO*)src, target, V, dst, rows, D, Rp);
  return hipGetLastError();
}

}  // namespace

// Pieces of the vocabulary whose G takes at most this many bytes.
constexpr int64_t kCePieceBytes = (int64_t)512 << 20;

CePlan plan_ce(int64_t N, int64_t V, int64_t D, int io) {
  CePlan p;
  p.parts = io == kIoBf16 ? 1 : 3;
  p.Dp = up(D, kBK);
  p.Np = up(N, kBigN);
  const int64_t most = kCePieceBytes / (p.Np * 2 * p.parts) / kBigM * kBigM;
  const int64_t pieces = (V + (most < kBigM ? kBigM : most) - 1) / (most < kBigM ? kBigM : most);
  p.piece = up((V + pieces - 1) / pieces, kBigM);
  p.pieces = (V + p.piece - 1) / p.piece;
  p.big_l = use_big(p.piece, N);
  p.tiles = p.big_l ? up(V, kBigM) / kBigM : up(V, kSmallM) / kSmallM;
  auto splits = [](int64_t M, int64_t N_, int64_t K, bool big) -> int64_t {
    // enough workgroups for two a compute unit, each with 16 steps at least
    int64_t s = 512 / tiles_of(M, N_, big);
    const int64_t most_s = K / (16 * kBK);
    s = s > most_s ? most_s : s;
    return s < 1 ? 1 : s > 16 ? 16 : s;
  };
  p.big_x = use_big(N, D) || tiles_of(N, D, true) * 8 >= 256;
  p.big_w = use_big(p.piece, D) || tiles_of(p.piece, D, true) * 8 >= 256;
  p.split_x = splits(N, D, p.piece, p.big_x);
  p.split_w = splits(p.piece, D, p.Np, p.big_w);
  p.slots_x = p.split_x > 1 || p.pieces > 1;
  p.slots_w = p.split_w > 1;
  return p;
}

hipError_t launch_linear_ce(const CePlan& p, const CeArgs& a, int io, hipStream_t stream) {
  const bool bf = io == kIoBf16;
  const int64_t es = bf ? 2 : 4;
  hipError_t e = hipSuccess;
#define LRS_CE(call)                 \
  do {                               \
    e = (call);                      \
    if (e != hipSuccess) return e;   \
  } while (0)
  GemmArgs base = {};
  base.npair = p.parts == 1 ? 1 : 6;
  // smallest products first: lo hi, hi lo, mid mid, mid hi, hi mid, hi hi
  const int ia[6] = {2, 0, 1, 1, 0, 0}, ib[6] = {0, 2, 1, 0, 1, 0};
  auto pairs = [&](GemmArgs& g, int64_t ka, int64_t kb, int64_t k) {
    for (int i = 0; i < base.npair; ++i) {
      g.pa[i] = p.parts == 1 ? 0 : (int)(ia[i] * ka);
      g.pb[i] = p.parts == 1 ? 0 : (int)(ib[i] * kb);
    }
    g.kt = (int)(k / kBK);
  };
  base.splits = 1;
  base.target = a.target;
  base.V = a.V;
  base.lse = a.lse;
  // rows of x and w as the logits' product takes them
  const bool raw_x = bf && p.Dp == a.D && ((uintptr_t)a.x & 15) == 0;
  const bool raw_w = bf && p.Dp == a.D && ((uintptr_t)a.w & 15) == 0;
  const uint16_t* xr = raw_x ? (const uint16_t*)a.x : a.x_rows;
  if (!raw_x)
    LRS_CE(bf ? (pack<uint16_t, 1>(a.x, a.x_rows, a.N, a.D, p.Dp, stream))
              : (pack<float, 3>(a.x, a.x_rows, a.N, a.D, p.Dp, stream)));
  auto w_rows = [&](int64_t v0, int64_t n, const uint16_t** out) -> hipError_t {
    const char* src = (const char*)a.w + v0 * a.D * es;
    if (raw_w) {
      *out = (const uint16_t*)src;
      return hipSuccess;
    }
    *out = a.w_rows;
    return bf ? pack<uint16_t, 1>(src, a.w_rows, n, a.D, p.Dp, stream)
              : pack<float, 3>(src, a.w_rows, n, a.D, p.Dp, stream);
  };
  auto logits = [&](GemmArgs& g, const uint16_t* wr, int64_t v0, int64_t n) {
    g.a = wr;
    g.b = xr;
    g.lda = g.ldb = p.parts * p.Dp;
    g.M = n;
    g.N = a.N;
    g.v0 = v0;
    pairs(g, p.Dp, p.Dp, p.Dp);
  };
  bool packed_whole = false;  // a.w_rows holds the only piece
  if (a.forward) {
    for (int64_t v0 = 0; v0 < a.V; v0 += p.piece) {
      const int64_t n = a.V - v0 < p.piece ? a.V - v0 : p.piece;
      const uint16_t* wr;
      LRS_CE(w_rows(v0, n, &wr));
      GemmArgs g = base;
      logits(g, wr, v0, n);
      g.part = a.part;
      g.part0 = v0 / (p.big_l ? kBigM : kSmallM);
      g.part_ld = p.tiles;
      g.tlogit = a.tlogit;
      LRS_CE(run_gemm<kEpiLse>(g, p.big_l, stream));
      if (v0 + p.piece >= a.V) {
        hipLaunchKernelGGL(k_ce_join, dim3((unsigned)((a.N + 3) / 4)), dim3(256), 0, stream, a.part,
                           a.tlogit, a.target, a.loss, a.lse, a.N, a.V, p.tiles);
        LRS_CE(hipGetLastError());
      }
    }
    packed_whole = p.pieces == 1;
  }
  if (!a.backward) return hipSuccess;
  hipLaunchKernelGGL(k_ce_scale, dim3(1), dim3(1024), 0, stream, a.grad_loss, a.target, a.N, a.V,
                     a.ratio, a.row_scale, a.top);
  LRS_CE(hipGetLastError());
  LRS_CE(bf ? (pack_t<uint16_t, 1>(a.x, a.target, a.V, a.x_cols, a.N, a.D, p.Np, stream))
            : (pack_t<float, 3>(a.x, a.target, a.V, a.x_cols, a.N, a.D, p.Np, stream)));
  for (int64_t v0 = 0; v0 < a.V; v0 += p.piece) {
    const int64_t n = a.V - v0 < p.piece ? a.V - v0 : p.piece;
    const char* src = (const char*)a.w + v0 * a.D * es;
    const uint16_t* wr = a.w_rows;
    if (!packed_whole || raw_w) LRS_CE(w_rows(v0, n, &wr));
    LRS_CE(bf ? (pack_t<uint16_t, 1>(src, nullptr, 0, a.w_cols, n, a.D, p.piece, stream))
              : (pack_t<float, 3>(src, nullptr, 0, a.w_cols, n, a.D, p.piece, stream)));
    {
      GemmArgs g = base;
      logits(g, wr, v0, n);
      g.ratio = a.ratio;
      g.g = a.g;
      g.gt = a.gt;
      g.nparts = p.parts;
      g.part_k = p.piece;
      g.part_kt = p.Np;
      g.ldg = p.parts * p.piece;
      g.ldgt = p.parts * p.Np;
      // a whole number of tiles writes all of G's padded columns: the last
      // piece's k loop below stops at its own whole number of tiles
      LRS_CE(run_gemm<kEpiGrad>(g, p.big_l, stream));
    }
    {
      GemmArgs g = base;
      g.a = a.gt;
      g.b = a.x_cols;
      g.lda = g.ldb = p.parts * p.Np;
      g.M = n;
      g.N = a.D;
      pairs(g, p.Np, p.Np, up(a.N, kSmallN));
      g.splits = (int)p.split_w;
      g.slots = p.slots_w ? a.slots_w : nullptr;
      g.out = (char*)a.grad_w + v0 * a.D * es;
      g.out_bf16 = bf;
      g.scale = a.top;
      LRS_CE(run_gemm<kEpiOut>(g, p.big_w, stream));
      if (p.slots_w) {
        hipLaunchKernelGGL(k_ce_join_slots, dim3(blocks_for(n * a.D, 1024)), dim3(256), 0, stream,
                           a.slots_w, (int)p.split_w, n, a.D, nullptr, a.top, g.out, bf ? 1 : 0);
        LRS_CE(hipGetLastError());
      }
    }
    {
      GemmArgs g = base;
      g.a = a.g;
      g.b = a.w_cols;
      g.lda = g.ldb = p.parts * p.piece;
      g.M = a.N;
      g.N = a.D;
      pairs(g, p.piece, p.piece, up(n, kSmallM));
      g.splits = (int)p.split_x;
      g.slots = p.slots_x ? a.slots_x : nullptr;
      g.accumulate = v0 > 0;
      g.out = a.grad_x;
      g.out_bf16 = bf;
      g.row_scale = a.row_scale;
      LRS_CE(run_gemm<kEpiOut>(g, p.big_x, stream));
    }
  }
  if (p.slots_x) {
    hipLaunchKernelGGL(k_ce_join_slots, dim3(blocks_for(a.N * a.D, 1024)), dim3(256), 0, stream,
                       a.slots_x, (int)p.split_x, a.N, a.D, a.row_scale, nullptr, a.grad_x,
                       bf ? 1 : 0);
    LRS_CE(hipGetLastError());
  }
#undef LRS_CE
  return hipSuccess;
}

hipError_t launch_zero(void* p, int64_t bytes, hipStream_t stream) {
  if (bytes <= 0) return hipSuccess;
  hipLaunchKernelGGL(k_ce_zero, dim3(blocks_for(bytes, 4096)), dim3(256), 0, stream, (uint32_t*)p,
                     bytes);
  return hipGetLastError();
}

}  // namespace lrs

// logprobs.hip -- log probabilities of given tokens from given logits, with the entropy
// and the likeliest alternatives, and their gradient.
//
//   m = max l,  s = sum exp(l - m),  t = sum exp(l - m) (l - m),
//   lse = m + log s,  logprob = (l_target - m) - log s,  entropy = log s - t / s;
//   grad_l = grad_logprob (onehot - p) - grad_entropy p (log p + entropy).
//
// Memory bound: the logits are read once.  A row streams through the 256 (or, where rows
// are few, 1024) threads of a workgroup, each with a maximum of its own so far and sums
// relative to it, which a larger value rescales.  A thread finds one in its i-th group once in
// about i rows, so that in nearly every group some of a wave's 64 do (32768 bf16 logits are 16
// groups a thread): the wave pays for the rescaling, one exponential beside the group's eight,
// each time.
//
// The `top` largest.  Every thread also keeps the place of the first of its largest values;
// the largest of 64 (or 128) groups of threads are ranked, and the top-th of them is a
// bound: there are `top` values at or above it, and hardly more (25 for the 20 largest of
// random logits).  Only threads whose own largest reaches it read their part again, leave
// the values in LDS, and those are ranked by counting.  A value and its index make one
// whole number, so that nothing is equal and the order does not depend on who came first.
// Where the bound is -infinity (few tokens are allowed), the values above it are
// candidates, and the first 128 places, among which are enough of the others.  Rows with
// more candidates than the LDS holds (many equal values over 1024 threads, or a NaN) are
// read `top` times again, each time for the largest below the one before.
//
// Measured: 8192 x 32768 bf16 with 20 alternatives 148 to 160 us (3.4 to 3.6 TB/s), in which
// vector instructions take some 80 % of the SIMDs' cycles; 4099 x 50021 fp32 forward 142 us
// (5.8 TB/s), backward 308 us (5.3 TB/s); 64 x 32000 bf16 with 8 alternatives 13.7 us: a row's
// 16 waves' loads, sums, ranks and a second reading one behind the other (12.2 with the row kept
// in registers, which took up to 193 us at 8192 rows).
#include "lrs_device.hpp"
#include "lrs_internal.hpp"
#include "lrs_rows.hpp"

namespace lrs {

namespace {

constexpr float kLog2eF = 1.4426950408889634f;
constexpr float kFarBelow = -200.0f;  // exp of it is 0: a logit of -infinity adds 0, not 0 * infinity
constexpr int kCandidates = 2048;  // a row of equal values has 32 a rank (256 threads)
constexpr uint64_t kNoKey = 0;
constexpr uint32_t kFirst = 0x80000000u;  // the low half of index 0; an index is below 2^24

// The order of the values (NaN above all), then of the indices from behind.
__device__ __forceinline__ uint64_t key_of(float v, int index) {
  const uint32_t b = as_u32(v + 0.0f);  // -0 is 0
  const uint32_t o = v != v ? ~0u : (b >> 31) ? ~b : b | 0x80000000u;
  return (uint64_t)o << 32 | (kFirst - (uint32_t)index);
}
__device__ __forceinline__ float key_value(uint64_t k) {
  const uint32_t o = (uint32_t)(k >> 32);
  return o == ~0u ? __builtin_nanf("") : as_f32((o >> 31) ? o ^ 0x80000000u : ~o);
}
__device__ __forceinline__ int64_t key_index(uint64_t k) { return (int64_t)(kFirst - (uint32_t)k); }
__device__ __forceinline__ uint64_t max_key(uint64_t a, uint64_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint64_t shfl_xor_key(uint64_t k, int o) {
  const uint32_t lo = (uint32_t)__shfl_xor((int)(uint32_t)k, o);
  const uint32_t hi = (uint32_t)__shfl_xor((int)(uint32_t)(k >> 32), o);
  return (uint64_t)hi << 32 | lo;
}

struct RowOut {
  float m, log_s, entropy;
};

// What a row's sums say.  m is the largest value that is not a NaN.
__device__ __forceinline__ RowOut row_out(float m, float s, float t) {
  RowOut o;
  o.m = m;
  o.log_s = logf(s);
  o.entropy = o.log_s - t / s;
  return o;
}
// s is NaN with a NaN or an infinite maximum in the row: then lse is NaN or that maximum.
__device__ __forceinline__ float row_lse(const RowOut& o, bool has_nan) {
  if (o.log_s == o.log_s) return o.m + o.log_s;
  return has_nan ? __builtin_nanf("") : o.m;
}

constexpr float kInf = __builtin_inff();
constexpr float kLowest = -3.402823466e38f;  // the lowest finite value, a mask to some
// The backward takes |lse| up to here as it was rounded, to 2^-17; beyond, where rounding
// would show in p, it sums the row again.
constexpr float kExactLse = 256.0f;

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int o = kWave / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o));
  return v;
}

// exp(l - m) and its product with l - m, added up over a group, and then to the thread's sums:
// a sum of n additions is known to n 2^-25 of itself where all of them round one way, as in rows of
// many equal logits.  While there is nothing but -infinity, m is that, and the lowest finite
// value stands for it.
template <int G>
__device__ __forceinline__ void add_group(const float (&v)[G], float m, float& s, float& t) {
  m = fmaxf(m, kLowest);
  float gs = 0.0f, gt = 0.0f;
#pragma unroll
  for (int j = 0; j < G; ++j) {
    const float c = v[j] - m;
    const float x = __builtin_amdgcn_exp2f(c * kLog2eF);
    gs = j == 0 ? x : gs + x;
    gt = j == 0 ? x * fmaxf(c, kFarBelow) : __builtin_fmaf(x, fmaxf(c, kFarBelow), gt);
  }
  s += gs;
  t += gt;
}
// A larger maximum: the sums become relative to it.
__device__ __forceinline__ void raise(float x, float& m, float& s, float& t) {
  const float d = m - x, f = __builtin_amdgcn_exp2f(d * kLog2eF);
  t = __builtin_fmaf(s * f, d, t * f);
  s *= f;
  m = x;
  if (!(s > 0.0f)) t = s = s == s ? 0.0f : s;  // nothing yet: d was not finite
}
// A thread's sums, relative to the row's maximum.
__device__ __forceinline__ void lower(float top, float m, float& s, float& t) {
  const float d = fmaxf(m - top, kFarBelow), f = __builtin_amdgcn_exp2f(d * kLog2eF);
  t = __builtin_fmaf(s * f, d, t * f);
  s *= f;
}

// A row's groups of 16 bytes, every BT-th a thread's.  An index is below 2^24.
template <typename IO, int BT>
struct Row {
  static constexpr int G = kGroup<IO>;
  const IO* row;
  int V;
  __device__ __forceinline__ int at(int i) const { return (i * BT + (int)threadIdx.x) * G; }
  // the values of the group that begins at e, `fill` behind the row's end
  __device__ __forceinline__ void group(int e, float fill, float (&v)[G]) const {
    unpack(ld_raw<false>(row, e, V), v);
#pragma unroll
    for (int j = 0; j < G; ++j) v[j] = e + j < V ? v[j] : fill;
  }
  // f(values, first index), every group of this thread in rising order, four in flight
  template <typename F>
  __device__ __forceinline__ void each(float fill, F f) const {
    constexpr int kStep = BT * G;
    int i = 0;
    for (; (i + 4) * kStep <= V; i += 4) {
      u32x4_t q[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) q[k] = *reinterpret_cast<const u32x4_any*>(row + at(i + k));
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        float v[G];
        unpack(q[k], v);
        f(v, at(i + k));
      }
    }
    for (; at(i) < V; ++i) {
      float v[G];
      group(at(i), fill, v);
      f(v, at(i));
    }
  }
};
template <int G>
__device__ __forceinline__ float group_max(const float (&v)[G]) {
  float x = v[0];
#pragma unroll
  for (int j = 1; j < G; ++j) x = fmaxf(x, v[j]);
  return x;
}

// Whether the row has a NaN, for all threads of the workgroup.
template <typename R>
__device__ __forceinline__ bool row_has_nan(const R& row, int* bad) {
  if (threadIdx.x == 0) *bad = 0;
  __syncthreads();
  bool nan = false;
  row.each(0.0f, [&](const auto& v, int e) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < R::G; ++j) nan |= v[j] != v[j];
  });
  if (nan) *bad = 1;
  __syncthreads();
  return *bad != 0;
}

__device__ __forceinline__ void write_row(const LogprobArgs& a, int64_t n, const RowOut& o,
                                          float target_logit, bool counted, bool nan) {
  a.logprob[n] = counted ? (target_logit - o.m) - o.log_s : 0.0f;
  a.entropy[n] = o.entropy;
  a.lse[n] = row_lse(o, nan);
}

template <typename IO, int BT, bool TOP>
__global__ __launch_bounds__(BT) void k_logprobs(LogprobArgs a) {
  constexpr int G = kGroup<IO>, NW = BT / kWave;
  __shared__ float red[NW][3];
  __shared__ uint64_t cand[TOP ? kCandidates : 1], best_of[TOP ? NW : 1];
  __shared__ int count, bad;
  const int64_t n = blockIdx.x;
  const Row<IO, BT> row = {(const IO*)a.logits + n * a.ld, (int)a.V};
  const int64_t target = a.target[n];
  const bool counted = target >= 0 && target < a.V;
  float tl = 0.0f;
  if (threadIdx.x == 0) {
    if (TOP) count = 0;
    if (counted) tl = io_ld(row.row, target);
  }

  float m = -kInf, s = 0.0f, t = 0.0f;
  int where = row.at(0);  // the first group that holds the thread's largest
  row.each(-kInf, [&](const float (&v)[G], int e) __attribute__((always_inline)) {
    const float x = group_max(v);
    if (x > m) {
      where = e;
      raise(x, m, s, t);
    }
    add_group(v, m, s, t);
  });
  const int w = threadIdx.x / kWave;
  {
    const float wm = wave_max(m);
    if ((threadIdx.x & (kWave - 1)) == 0) red[w][0] = wm;
  }
  uint64_t mine = kNoKey;
  const int groups = a.top > 32 ? 128 : 64;
  if constexpr (TOP) {
    if (row.at(0) < row.V) {
      float v[G];
      row.group(where, -kInf, v);
#pragma unroll
      for (int j = G - 1; j >= 0; --j)
        if (v[j] == m && where + j < row.V) mine = key_of(m, where + j);
    }
    const int per = BT / groups;
    uint64_t key = mine;
    for (int o = per / 2; o > 0; o >>= 1) key = max_key(key, shfl_xor_key(key, o));
    if (threadIdx.x % per == 0) cand[threadIdx.x / per] = key;
  }
  __syncthreads();
  // the threads' sums, brought to the row's maximum
  float top_value = red[0][0];
#pragma unroll
  for (int i = 1; i < NW; ++i) top_value = fmaxf(top_value, red[i][0]);
  lower(top_value, m, s, t);
#pragma unroll
  for (int o = kWave / 2; o > 0; o >>= 1) {
    s += __shfl_xor(s, o);
    t += __shfl_xor(t, o);
  }
  if ((threadIdx.x & (kWave - 1)) == 0) {
    red[w][1] = s;
    red[w][2] = t;
  }
  if constexpr (TOP) {
    if ((int)threadIdx.x < groups) {
      const uint64_t k = cand[threadIdx.x];
      int rank = 0;
#pragma unroll 16
      for (int i = 0; i < groups; ++i) {
        const uint64_t o = cand[i];
        rank += o > k || (o == k && i < (int)threadIdx.x);
      }
      if (rank == a.top - 1) best_of[0] = k;
    }
  }
  __syncthreads();
  s = t = 0.0f;
#pragma unroll
  for (int i = 0; i < NW; ++i) {
    s += red[i][1];
    t += red[i][2];
  }
  // the same for all threads: nothing but -infinity, an infinity or a NaN
  const bool odd = !(s > 0.0f) || !(fabsf(top_value) < kInf);
  bool nan = false;
  if (odd) {
    nan = row_has_nan(row, &bad);
    s = __builtin_nanf("");
  }
  const RowOut out = row_out(top_value, s, t);
  if (threadIdx.x == 0) write_row(a, n, out, tl, counted, nan);
  if constexpr (TOP) {
    const int top = a.top;
    int64_t* ids = a.top_ids + n * top;
    float* lps = a.top_logprobs + n * top;
    auto emit = [&](int rank, uint64_t key) __attribute__((always_inline)) {
      ids[rank] = key_index(key);
      lps[rank] = (key_value(key) - out.m) - out.log_s;
    };
    const uint64_t bound = best_of[0];
    bool many = odd;
    if (!odd) {
      __syncthreads();  // cand is written again
      const float least = bound == kNoKey ? -kInf : key_value(bound);  // no key: groups without values
      if (mine >= bound || least == -kInf) {
        row.each(-kInf, [&](const float (&v)[G], int e) __attribute__((always_inline)) {
          const float x = group_max(v);
          if (!(least == -kInf ? x > least || e < 128 : x >= least)) return;
#pragma unroll
          for (int j = 0; j < G; ++j) {
            const uint64_t k = key_of(v[j], e + j);
            if (e + j < row.V && (least == -kInf ? v[j] > least || e + j < 128 : k >= bound)) {
              const int i = atomicAdd(&count, 1);
              if (i < kCandidates) cand[i] = k;
            }
          }
        });
      }
      __syncthreads();
      const int found = count;
      many = found > kCandidates;
      if (!many) {
        for (int i = threadIdx.x; i < found; i += BT) {
          const uint64_t k = cand[i];
          int rank = 0;
#pragma unroll 8
          for (int j = 0; j < found; ++j) rank += cand[j] > k;
          if (rank < top) emit(rank, k);
        }
      }
    }
    if (many) {
      uint64_t last = ~0ull;  // above every key
      for (int r = 0; r < top; ++r) {
        uint64_t key = kNoKey;
        row.each(-kInf, [&](const float (&v)[G], int e) __attribute__((always_inline)) {
#pragma unroll
          for (int j = 0; j < G; ++j) {
            const uint64_t k = key_of(v[j], e + j);
            if (k < last && e + j < row.V) key = max_key(key, k);
          }
        });
#pragma unroll
        for (int o = kWave / 2; o > 0; o >>= 1) key = max_key(key, shfl_xor_key(key, o));
        __syncthreads();
        if ((threadIdx.x & (kWave - 1)) == 0) best_of[threadIdx.x / kWave] = key;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NW; ++i) key = max_key(key, best_of[i]);
        if (threadIdx.x == 0) emit(r, key);
        last = key;
      }
    }
  }
}

// A row's maximum and the logarithm of its sum.
template <typename IO>
__device__ __forceinline__ float2 row_sum_of(const IO* row, int V) {
  constexpr int G = kGroup<IO>;
  __shared__ float red[2][256 / kWave];
  const Row<IO, 256> all = {row, V};
  float s = 0.0f, t = 0.0f;
  float m = -kInf;
  all.each(-kInf, [&](const float (&v)[G], int) __attribute__((always_inline)) {
    const float x = group_max(v);
    if (x > m) raise(x, m, s, t);
    add_group(v, m, s, t);
  });
  const float wm = wave_max(m);
  if ((threadIdx.x & (kWave - 1)) == 0) red[0][threadIdx.x / kWave] = wm;
  __syncthreads();
  float top = red[0][0];
#pragma unroll
  for (int i = 1; i < 256 / kWave; ++i) top = fmaxf(top, red[0][i]);
  lower(top, m, s, t);
  s = wave_sum(s);
  if ((threadIdx.x & (kWave - 1)) == 0) red[1][threadIdx.x / kWave] = s;
  __syncthreads();
  s = red[1][0];
#pragma unroll
  for (int i = 1; i < 256 / kWave; ++i) s += red[1][i];
  return make_float2(top, logf(s));
}

// One group of 16 bytes a thread and step; blockIdx.x = row, blockIdx.y = piece of it, and of
// a row that is summed again, by each workgroup that has a part of it, a larger piece.
template <typename IO, bool NT>
__global__ __launch_bounds__(256) void k_logprobs_bwd(LogprobArgs a, int64_t piece, int64_t far_piece) {
  constexpr int G = kGroup<IO>;
  const int64_t n = blockIdx.x;
  const IO* row = (const IO*)a.logits + n * a.ld;
  IO* out = (IO*)a.grad_logits + n * a.ld_grad;
  const int64_t target = a.target[n];
  const float lse = a.lse[n], ge = a.grad_entropy ? a.grad_entropy[n] : 0.0f;
  const float h = a.grad_entropy ? a.entropy[n] : 0.0f;
  const float gl = target >= 0 && target < a.V ? a.grad_logprob[n] : 0.0f;
  const float base = __builtin_fmaf(ge, h, gl);  // grad = -p (gl + ge (c + h))
  // a row that asks for nothing gets 0, whatever its logits are (padding)
  const bool none = !(target >= 0 && target < a.V) && ge == 0.0f;
  // log p = (l - m) - log_s
  float m = lse, log_s = 0.0f;
  if (fabsf(lse) > kExactLse && fabsf(lse) < kInf) {  // the same for all threads
    piece = far_piece;
    if (blockIdx.y * piece >= a.V) return;
    const float2 all = row_sum_of<IO>(row, (int)a.V);
    m = all.x;
    log_s = all.y;
  }
  const int64_t e1 = (int64_t)(blockIdx.y + 1) * piece;
  const int64_t end = e1 < a.V ? e1 : a.V;
#pragma unroll 4
  for (int64_t e = blockIdx.y * piece + (int64_t)threadIdx.x * G; e < end; e += 256 * G) {
    float v[G];
    ld_group<NT>(row, e, a.V, v);
#pragma unroll
    for (int j = 0; j < G; ++j) {
      const float c = (v[j] - m) - log_s;
      const float p = __builtin_amdgcn_exp2f(c * kLog2eF);
      const float g = p * -__builtin_fmaf(ge, fmaxf(c, kFarBelow), base);
      v[j] = none ? 0.0f : e + j == target ? g + gl : g;
    }
    st_group<NT>(out, e, a.V, v);
  }
}

template <typename IO>
void logprobs(const LogprobArgs& a, hipStream_t stream) {
  const int64_t groups = (a.V + kGroup<IO> - 1) / kGroup<IO>;
  const dim3 grid((unsigned)a.N);
  // Several rows a compute unit while there are rows enough, else the most threads a row:
  // 64 x 32000 takes 13.9 us with 1024 threads, 14.7 with 512.
  const bool few = a.N < 2 * device_cus() && groups > 512;
#define LRS_LP(BT, TOP) hipLaunchKernelGGL((k_logprobs<IO, BT, TOP>), grid, dim3(BT), 0, stream, a)
  if (a.top > 0) {
    if (few) LRS_LP(1024, true);
    else LRS_LP(256, true);
  } else {
    if (few) LRS_LP(1024, false);
    else LRS_LP(256, false);
  }
#undef LRS_LP
}

}  // namespace

hipError_t launch_logprobs_fwd(const LogprobArgs& a, int io, hipStream_t stream) {
  if (io == kIoBf16) logprobs<uint16_t>(a, stream);
  else logprobs<float>(a, stream);
  return hipGetLastError();
}

hipError_t launch_logprobs_bwd(const LogprobArgs& a, int io, hipStream_t stream) {
  const int group = io == kIoBf16 ? 8 : 4;
  const bool nt = 2 * a.N * a.V * (io == kIoBf16 ? 2 : 4) >= kStreamFootprint;
  // pieces of eight groups a thread; in place one, as a workgroup may read the whole row
  const int64_t step = 256 * 8 * group, steps = (a.V + step - 1) / step;
  const int64_t pieces = a.grad_logits == a.logits ? 1 : steps, piece = step * (steps / pieces);
  // Summing a row again reads all of it, so a piece each would read it V / 8192 times (fp32):
  // then as many as fill the compute units with four workgroups each.  Logits 1000 away from 0,
  // fp32, in us, by every piece and so: 1000 x 150000 2428 and 334 (239 near 0), 256 x 150000 411
  // and 103 (112 by one workgroup a row), 16 x 150000 31 both (77 by one).
  const int64_t most = 4 * (int64_t)device_cus() / a.N, far = most < 1 ? 1 : most < pieces ? most : pieces;
  const int64_t far_piece = piece * ((pieces + far - 1) / far);
  const dim3 grid((unsigned)a.N, (unsigned)pieces);
#define LRS_LPB(IO, NT) \
  hipLaunchKernelGGL((k_logprobs_bwd<IO, NT>), grid, dim3(256), 0, stream, a, piece, far_piece)
  if (io == kIoBf16) {
    if (nt) LRS_LPB(uint16_t, true);
    else LRS_LPB(uint16_t, false);
  } else {
    if (nt) LRS_LPB(float, true);
    else LRS_LPB(float, false);
  }
#undef LRS_LPB
  return hipGetLastError();
}

}  // namespace lrs

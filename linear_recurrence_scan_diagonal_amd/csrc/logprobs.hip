// logprobs.hip -- log probabilities of given tokens from given logits, with the entropy
// and the likeliest alternatives, and their gradient.
//
//   m = max l,  s = sum exp(l - m),  t = sum exp(l - m) (l - m),
//   lse = m + log s,  logprob = (l_target - m) - log s,  entropy = log s - t / s;
//   grad_l = grad_logprob (onehot - p) - grad_entropy p (log p + entropy).
//
// Memory bound: the logits are read once.  Without alternatives a row streams through its
// threads, each with a maximum of its own so far and sums relative to it (a larger value
// rescales them, which is rare after the first few).  With alternatives a row is held in
// the registers of 256 to 1024 threads (up to 16 groups of 16 bytes a thread), where it is
// looked at three times; rows too wide for that are read again (and found in the caches).
//
// The `top` largest.  Every thread has the first of its largest values from the pass over
// the maximum; the largest of 64 (or 128) groups of threads are ranked, and the top-th of
// them is a bound: there are `top` values at or above it, and hardly more (25 for the 20
// largest of random logits).  Those are collected in LDS, which few threads have to take
// part in, and ranked by counting.  A value and its index make one whole number, so that
// nothing is equal and the order does not depend on who came first.  Where the bound is
// -infinity (few tokens are allowed), those that are not are candidates, and the first 128
// places, among which are enough of the others.  Rows with more candidates than the LDS
// holds (large values side by side, or a NaN) are read `top` times again, each time for
// the largest below the one before.
#include "lrs_device.hpp"
#include "lrs_internal.hpp"
#include "lrs_rows.hpp"

namespace lrs {

namespace {

constexpr float kLog2eF = 1.4426950408889634f;
constexpr float kFarBelow = -200.0f;  // exp of it is 0: a logit of -infinity adds 0, not 0 * infinity
constexpr int kCandidates = 2048;  // a row of equal values has 64 to 2048
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
constexpr float kLowest = -3.4e38f;  // behind a row's end, where sums are made: adds 0

__device__ __forceinline__ float wave_max(float v) {
#pragma unroll
  for (int o = kWave / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o));
  return v;
}

// exp(l - m) and its product with l - m, added up over a group.  CLAMP: -infinity among
// the values adds 0 instead of NaN to the second sum.
template <bool CLAMP, int G>
__device__ __forceinline__ void add_group(const float (&v)[G], float m, float& s, float& t) {
#pragma unroll
  for (int j = 0; j < G; ++j) {
    const float c = v[j] - m;
    const float x = __builtin_amdgcn_exp2f(c * kLog2eF);
    s += x;
    t = __builtin_fmaf(x, CLAMP ? fmaxf(c, kFarBelow) : c, t);
  }
}

// The groups of 16 bytes of a row, held in registers (NV > 0) or read again (NV = 0).  An
// index is below 2^24.
template <typename IO, int BT, int NV>
struct Row {
  static constexpr int G = kGroup<IO>;
  u32x4_t q[NV > 0 ? NV : 1];
  const IO* row;
  int V;
  // whether every thread's group i is inside the row; the same for all threads
  __device__ __forceinline__ bool full(int i) const { return (i + 1) * (BT * G) <= V; }
  __device__ __forceinline__ int at(int i) const { return (i * BT + (int)threadIdx.x) * G; }
  __device__ __forceinline__ u32x4_t load(int i) const {
    if (full(i)) return *reinterpret_cast<const u32x4_any*>(row + at(i));
    return ld_raw<false>(row, at(i), V);
  }
  __device__ __forceinline__ void open(const IO* p, int64_t n) {
    row = p;
    V = (int)n;
#pragma unroll
    for (int i = 0; i < NV; ++i) q[i] = load(i);
  }
  // the values of a group that begins at e, `fill` behind the row's end
  __device__ __forceinline__ void get(u32x4_t raw, int e, float fill, float (&v)[G]) const {
    unpack(raw, v);
#pragma unroll
    for (int j = 0; j < G; ++j) v[j] = e + j < V ? v[j] : fill;
  }
  // f(values, first index), every group of this thread in rising order
  template <typename F>
  __device__ __forceinline__ void each(float fill, F f) {
    if constexpr (NV > 0) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float v[G];
        // opaque, or a pass's unpacked values would be kept for the next one
        asm volatile("" : "+v"(q[i]));
        if (full(i)) unpack(q[i], v);
        else get(q[i], at(i), fill, v);
        f(v, at(i));
        __builtin_amdgcn_sched_barrier(0);  // one group after the other: registers
      }
    } else {
      int i = 0;
#pragma unroll 4
      for (; full(i); ++i) {
        float v[G];
        unpack(*reinterpret_cast<const u32x4_any*>(row + at(i)), v);
        f(v, at(i));
      }
      if (at(i) < V) {
        float v[G];
        get(ld_raw<false>(row, at(i), V), at(i), fill, v);
        f(v, at(i));
      }
    }
  }
  __device__ __forceinline__ void group(int e, float fill, float (&v)[G]) const {
    u32x4_t raw = {0u, 0u, 0u, 0u};
    if constexpr (NV > 0) {
#pragma unroll
      for (int i = 0; i < NV; ++i) raw = at(i) == e ? q[i] : raw;
    } else {
      raw = ld_raw<false>(row, e, V);
    }
    get(raw, e, fill, v);
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
__device__ __forceinline__ bool row_has_nan(R& row, int* bad) {
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

// No alternatives: the row streams past.
template <typename IO, int BT>
__global__ __launch_bounds__(BT) void k_logprobs(LogprobArgs a) {
  constexpr int G = kGroup<IO>, NW = BT / kWave;
  __shared__ float red[NW][3];
  __shared__ int bad;
  const int64_t n = blockIdx.x;
  Row<IO, BT, 0> row;
  row.open((const IO*)a.logits + n * a.ld, a.V);
  const int64_t target = a.target[n];
  const bool counted = target >= 0 && target < a.V;
  float tl = 0.0f;
  if (threadIdx.x == 0 && counted) tl = io_ld(row.row, target);

  float m = kLowest, s = 0.0f, t = 0.0f;
  row.each(kLowest, [&](const float (&v)[G], int e) __attribute__((always_inline)) {
    const float x = group_max(v);
    if (x > m) {  // exp(m - x), and t is relative to the new maximum
      const float d = m - x, f = __builtin_amdgcn_exp2f(d * kLog2eF);
      t = __builtin_fmaf(s * f, d, t * f);
      s *= f;
      m = x;
      if (!(s > 0.0f)) t = s = s == s ? 0.0f : s;  // nothing yet: d was not finite
    }
    add_group<true>(v, m, s, t);
  });
  // the threads' sums, brought to the row's maximum
  const float wm = wave_max(m);
  const int w = threadIdx.x / kWave;
  if ((threadIdx.x & (kWave - 1)) == 0) red[w][0] = wm;
  __syncthreads();
  float top = red[0][0];
#pragma unroll
  for (int i = 1; i < NW; ++i) top = fmaxf(top, red[i][0]);
  {
    const float d = fmaxf(m - top, kFarBelow), f = __builtin_amdgcn_exp2f(d * kLog2eF);
    t = __builtin_fmaf(s * f, d, t * f);
    s *= f;
  }
#pragma unroll
  for (int o = kWave / 2; o > 0; o >>= 1) {
    s += __shfl_xor(s, o);
    t += __shfl_xor(t, o);
  }
  if ((threadIdx.x & (kWave - 1)) == 0) {
    red[w][1] = s;
    red[w][2] = t;
  }
  __syncthreads();
  s = t = 0.0f;
#pragma unroll
  for (int i = 0; i < NW; ++i) {
    s += red[i][1];
    t += red[i][2];
  }
  // the same for all threads: nothing but -infinity, an infinity or a NaN
  const bool odd = !(s > 0.0f) || !(fabsf(top) < -kLowest);
  bool nan = false;
  if (odd) {
    nan = row_has_nan(row, &bad);
    if (!(top > kLowest)) top = -kInf;
    if (!(fabsf(top) < kInf) || nan) s = __builtin_nanf("");
  }
  if (threadIdx.x == 0) write_row(a, n, row_out(top, s, t), tl, counted, nan);
}

// With alternatives.
template <typename IO, int BT, int NV>
__global__ __launch_bounds__(BT) void k_logprobs_top(LogprobArgs a) {
  constexpr int G = kGroup<IO>, NW = BT / kWave;
  __shared__ float red[NW][3];
  __shared__ uint64_t cand[kCandidates], best_of[NW];
  __shared__ int count, bad;
  const int64_t n = blockIdx.x;
  Row<IO, BT, NV> row;
  row.open((const IO*)a.logits + n * a.ld, a.V);
  const int64_t target = a.target[n];
  const bool counted = target >= 0 && target < a.V;
  float tl = 0.0f;
  if (threadIdx.x == 0) {
    count = 0;
    if (counted) tl = io_ld(row.row, target);
  }

  // the maximum, and the thread's first group that holds its own
  float m = -kInf;
  int where = row.at(0);
  row.each(-kInf, [&](const float (&v)[G], int e) __attribute__((always_inline)) {
    const float x = group_max(v);
    where = x > m ? e : where;
    m = fmaxf(m, x);
  });
  const float own = m;
  const int w = threadIdx.x / kWave;
  m = wave_max(m);
  if ((threadIdx.x & (kWave - 1)) == 0) red[w][0] = m;
  // the thread's largest value and its first place, and the largest of each group of threads:
  // 64 groups, 128 for more than 32 alternatives
  uint64_t mine = kNoKey;
  if (row.at(0) < a.V) {
    float v[G];
    row.group(where, -kInf, v);
    int j0 = G;
#pragma unroll
    for (int j = G - 1; j >= 0; --j) j0 = v[j] == own && where + j < a.V ? j : j0;
    if (j0 < G) mine = key_of(own, where + j0);
  }
  const int groups = a.top > 32 ? 128 : 64, per = BT / groups;
  {
    uint64_t key = mine;
    for (int o = per / 2; o > 0; o >>= 1) key = max_key(key, shfl_xor_key(key, o));
    if (threadIdx.x % per == 0) cand[threadIdx.x / per] = key;
  }
  __syncthreads();
  m = red[0][0];
#pragma unroll
  for (int i = 1; i < NW; ++i) m = fmaxf(m, red[i][0]);
  // the top-th largest of the groups, found by the first wave (or two) while the others go on
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
  float s = 0.0f, t = 0.0f;
  row.each(kLowest, [&](const float (&v)[G], int e) __attribute__((always_inline)) {
    add_group<false>(v, m, s, t);
  });
  if (t != t && s == s) {  // -infinity among the values
    s = t = 0.0f;
    Row<IO, BT, 0> again;
    again.open(row.row, row.V);
    again.each(kLowest, [&](const float (&v)[G], int e) __attribute__((always_inline)) {
      add_group<true>(v, m, s, t);
    });
  }
#pragma unroll
  for (int o = kWave / 2; o > 0; o >>= 1) {
    s += __shfl_xor(s, o);
    t += __shfl_xor(t, o);
  }
  if ((threadIdx.x & (kWave - 1)) == 0) {
    red[w][1] = s;
    red[w][2] = t;
  }
  __syncthreads();
  const uint64_t found_bound = best_of[0];
  s = t = 0.0f;
#pragma unroll
  for (int i = 0; i < NW; ++i) {
    s += red[i][1];
    t += red[i][2];
  }
  const bool odd = !(fabsf(m) < kInf) || s != s;  // the same for all threads
  bool nan = false;
  if (odd) {
    Row<IO, BT, 0> again;
    again.open(row.row, row.V);
    nan = row_has_nan(again, &bad);
  }
  const RowOut out = row_out(m, odd ? __builtin_nanf("") : s, t);
  if (threadIdx.x == 0) write_row(a, n, out, tl, counted, nan);

  const int top = a.top;
  int64_t* ids = a.top_ids + n * top;
  float* lps = a.top_logprobs + n * top;
  auto emit = [&](int rank, uint64_t key) __attribute__((always_inline)) {
    ids[rank] = key_index(key);
    lps[rank] = (key_value(key) - m) - out.log_s;
  };
  bool many = odd;
  if (!odd) {
    const uint64_t bound = found_bound;
    const float least = bound == kNoKey ? -kInf : key_value(bound);  // no key: groups without values
    if (mine >= bound || least == -kInf) {
      // the groups that hold candidates, by number, and then those one at a time, read again
      auto take = [&](int e) __attribute__((always_inline)) {
        float v[G];
        row.get(ld_raw<false>(row.row, e, row.V), e, -kInf, v);
#pragma unroll
        for (int j = 0; j < G; ++j) {
          const uint64_t k = key_of(v[j], e + j);
          if (e + j < row.V && (least == -kInf ? v[j] > least || e + j < 128 : k >= bound)) {
            const int i = atomicAdd(&count, 1);
            if (i < kCandidates) cand[i] = k;
          }
        }
      };
      auto holds = [&](const float (&v)[G], int e) __attribute__((always_inline)) {
        const float x = group_max(v);
        return least == -kInf ? x > least || e < 128 : x >= least;
      };
      if constexpr (NV > 0) {
        uint32_t some = 0u;
        int i = 0;
        row.each(-kInf, [&](const float (&v)[G], int e) __attribute__((always_inline)) {
          some |= holds(v, e) ? 1u << i : 0u;
          ++i;
        });
        while (some) {
          const int n = __builtin_ctz(some);
          some &= some - 1u;
          take(row.at(n));
        }
      } else {
        row.each(-kInf, [&](const float (&v)[G], int e) __attribute__((always_inline)) {
          if (holds(v, e)) take(e);
        });
      }
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
    Row<IO, BT, 0> again;
    again.open(row.row, row.V);
    uint64_t last = ~0ull;  // above every key
    for (int r = 0; r < top; ++r) {
      uint64_t key = kNoKey;
      again.each(-kInf, [&](const float (&v)[G], int e) __attribute__((always_inline)) {
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

// One group of 16 bytes a thread and step; blockIdx.x = row, blockIdx.y = piece of it.
template <typename IO, bool NT>
__global__ __launch_bounds__(256) void k_logprobs_bwd(LogprobArgs a, int64_t piece) {
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
  const int64_t e1 = (int64_t)(blockIdx.y + 1) * piece;
  const int64_t end = e1 < a.V ? e1 : a.V;
#pragma unroll 4
  for (int64_t e = blockIdx.y * piece + (int64_t)threadIdx.x * G; e < end; e += 256 * G) {
    float v[G];
    ld_group<NT>(row, e, a.V, v);
#pragma unroll
    for (int j = 0; j < G; ++j) {
      const float c = v[j] - lse;
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
  if (a.top == 0) {
    // several rows a compute unit while there are rows enough, else the most threads a row
    if (a.N >= 2 * device_cus() || groups <= 512)
      hipLaunchKernelGGL((k_logprobs<IO, 256>), grid, dim3(256), 0, stream, a);
    else
      hipLaunchKernelGGL((k_logprobs<IO, 1024>), grid, dim3(1024), 0, stream, a);
    return;
  }
#define LRS_LP(BT, NV) hipLaunchKernelGGL((k_logprobs_top<IO, BT, NV>), grid, dim3(BT), 0, stream, a)
  if (groups <= 256 * 4) LRS_LP(256, 4);
  else if (groups <= 512 * 4) LRS_LP(512, 4);
  else if (groups <= 512 * 8) LRS_LP(512, 8);
  else if (groups <= 1024 * 8) LRS_LP(1024, 8);
  else if (groups <= 1024 * 16) LRS_LP(1024, 16);
  else LRS_LP(1024, 0);
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
  // pieces of four to eight groups a thread
  const int64_t piece = 256 * 8 * group, pieces = (a.V + piece - 1) / piece;
  const dim3 grid((unsigned)a.N, (unsigned)pieces);
#define LRS_LPB(IO, NT) \
  hipLaunchKernelGGL((k_logprobs_bwd<IO, NT>), grid, dim3(256), 0, stream, a, piece)
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

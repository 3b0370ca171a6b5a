// logprobs.hip -- log probabilities of given tokens from given logits, with the entropy
// and the likeliest alternatives, and their gradient.
//
//   m = max l,  s = sum exp(l - m),  t = sum exp(l - m) (l - m),
//   lse = m + log s,  logprob = (l_target - m) - log s,  entropy = log s - t / s;
//   grad_l = grad_logprob (onehot - p) - grad_entropy p (log p + entropy).
//
// Memory bound: the logits are read once.  A row is held in the registers of 256, 512 or
// 1024 threads (up to 16 groups of 16 bytes a thread), so that the maximum is known before
// the first exponential and the sums need no rescaling; rows too wide for that are walked
// again (and found in the caches).
//
// The `top` largest.  Every thread has the first of its largest values from the pass over
// the maximum; the largest of 64 (or 128) groups of threads are put in order, and the
// top-th of them is a bound: there are `top` values at or above it, and hardly more (25
// for the 20 largest of random logits).  Those are collected in LDS, which few threads
// have to take part in, and ranked by counting.  A value and its index make one whole
// number, so that nothing is equal and the order does not depend on who came first.  Rows
// with more candidates than the LDS holds (order along the row, or a NaN) take `top`
// passes over the registers instead, each for the largest below the one before.
#include "lrs_device.hpp"
#include "lrs_internal.hpp"
#include "lrs_rows.hpp"

namespace lrs {

namespace {

constexpr float kLog2eF = 1.4426950408889634f;
constexpr float kFarBelow = -200.0f;  // exp of it is 0: a logit of -infinity adds 0, not 0 * infinity
constexpr int kCandidates = 512;
constexpr uint64_t kNoKey = 0;
constexpr uint32_t kFirst = 0x80000000u;  // the low half of index 0; an index is below 2^24

// The order of the values (NaN above all), then of the indices from behind.
__device__ __forceinline__ uint64_t key_of(float v, int64_t index) {
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

template <int BT>
__device__ __forceinline__ float block_max(float v, float* red) {
#pragma unroll
  for (int o = kWave / 2; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor(v, o));
  if ((threadIdx.x & (kWave - 1)) == 0) red[threadIdx.x / kWave] = v;
  __syncthreads();
  v = red[0];
#pragma unroll
  for (int w = 1; w < BT / kWave; ++w) v = fmaxf(v, red[w]);
  return v;
}

// The groups of 16 bytes of a row, held in registers (NV > 0) or read again (NV = 0).
// Past the end of the row a value is -infinity.
template <typename IO, int BT, int NV>
struct Row {
  static constexpr int G = kGroup<IO>;
  u32x4_t q[NV > 0 ? NV : 1];
  const IO* row;
  int64_t V;
  __device__ __forceinline__ void open(const IO* p, int64_t n) {
    row = p;
    V = n;
#pragma unroll
    for (int i = 0; i < NV; ++i) q[i] = ld_raw<false>(row, at(i), V);
  }
  __device__ __forceinline__ int64_t at(int64_t i) const {
    return (i * BT + (int64_t)threadIdx.x) * G;
  }
  __device__ __forceinline__ void get(u32x4_t raw, int64_t e, float (&v)[G]) const {
    unpack(raw, v);
    if (e + G > V) {
#pragma unroll
      for (int j = 0; j < G; ++j) v[j] = e + j < V ? v[j] : -__builtin_inff();
    }
  }
  // f(values, first index), every group of this thread in rising order
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    if constexpr (NV > 0) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float v[G];
        if (at(i) < V) {
          get(q[i], at(i), v);
          f(v, at(i));
        }
      }
    } else {
      for (int64_t i = 0; at(i) < V; ++i) {
        float v[G];
        get(ld_raw<false>(row, at(i), V), at(i), v);
        f(v, at(i));
      }
    }
  }
};

template <typename IO, int BT, int NV, bool TOP>
__global__ __launch_bounds__(BT) void k_logprobs(LogprobArgs a) {
  constexpr int G = kGroup<IO>, NW = BT / kWave;
  __shared__ float red[2 * NW];
  __shared__ float reds[NW][2];
  __shared__ uint64_t cand[TOP ? kCandidates : 1], best_of[TOP ? NW : 1];
  __shared__ int count, bad;
  const int64_t n = blockIdx.x;
  Row<IO, BT, NV> row;
  row.open((const IO*)a.logits + n * a.ld, a.V);
  if (TOP && threadIdx.x == 0) count = 0;
  if (threadIdx.x == 0) bad = 0;

  // the maximum; with alternatives, the thread's first group that holds its own
  float m = -__builtin_inff();
  int64_t where = row.at(0);
  row.each([&](const float (&v)[G], int64_t e) __attribute__((always_inline)) {
    float x = v[0];
#pragma unroll
    for (int j = 1; j < G; ++j) x = fmaxf(x, v[j]);
    if (TOP && x > m) where = e;
    m = fmaxf(m, x);
  });
  const float own = m;
  m = block_max<BT>(m, red);
  const bool infinite = !(fabsf(m) < __builtin_inff());
  float s = 0.0f, t = 0.0f;
  row.each([&](const float (&v)[G], int64_t e) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < G; ++j) {
      const float c = v[j] - m;
      const float x = __builtin_amdgcn_exp2f(c * kLog2eF);
      s += x;
      t = __builtin_fmaf(x, fmaxf(c, kFarBelow), t);
    }
  });
#pragma unroll
  for (int o = kWave / 2; o > 0; o >>= 1) {
    s += __shfl_xor(s, o);
    t += __shfl_xor(t, o);
  }
  if ((threadIdx.x & (kWave - 1)) == 0) {
    reds[threadIdx.x / kWave][0] = s;
    reds[threadIdx.x / kWave][1] = t;
  }
  __syncthreads();
  s = t = 0.0f;
#pragma unroll
  for (int w = 0; w < NW; ++w) {
    s += reds[w][0];
    t += reds[w][1];
  }
  const bool odd = infinite || s != s;  // the same for all threads
  if (odd) {
    // -infinity past the end of a row of nothing else is not one of its values
    bool nan = false;
    row.each([&](const float (&v)[G], int64_t e) __attribute__((always_inline)) {
#pragma unroll
      for (int j = 0; j < G; ++j) nan |= v[j] != v[j];
    });
    if (nan) bad = 1;
    __syncthreads();
  }
  const RowOut out = row_out(m, odd ? __builtin_nanf("") : s, t);
  if (threadIdx.x == 0) {
    const int64_t target = a.target[n];
    float lp = 0.0f;
    if (target >= 0 && target < a.V) lp = (io_ld(row.row, target) - m) - out.log_s;
    a.logprob[n] = lp;
    a.entropy[n] = out.entropy;
    a.lse[n] = row_lse(out, odd && bad);
  }
  if constexpr (!TOP) return;

  const int top = a.top;
  int64_t* ids = a.top_ids + n * top;
  float* lps = a.top_logprobs + n * top;
  auto emit = [&](int rank, uint64_t key) __attribute__((always_inline)) {
    ids[rank] = key_index(key);
    lps[rank] = (key_value(key) - m) - out.log_s;
  };
  bool many = odd;
  if (!odd) {
    // this thread's largest, and its first place
    uint64_t key = kNoKey;
    if (row.at(0) < a.V) {
      if constexpr (NV > 0) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          if (row.at(i) == where) {
            float v[G];
            row.get(row.q[i], where, v);
#pragma unroll
            for (int j = G - 1; j >= 0; --j)
              if (v[j] == own && where + j < a.V) key = key_of(v[j], where + j);
          }
        }
      } else {
        float v[G];
        row.get(ld_raw<false>(row.row, where, a.V), where, v);
#pragma unroll
        for (int j = G - 1; j >= 0; --j)
          if (v[j] == own && where + j < a.V) key = key_of(v[j], where + j);
      }
    }
    const uint64_t mine = key;
    // the largest of 64 groups of threads, 128 for more than 32 alternatives, in order
    const int groups = top > 32 ? 128 : 64, per = BT / groups;
    for (int o = per / 2; o > 0; o >>= 1) key = max_key(key, shfl_xor_key(key, o));
    if (threadIdx.x % per == 0) cand[threadIdx.x / per] = key;
    __syncthreads();
    uint64_t bound = kNoKey;
    if ((int)threadIdx.x < groups) {
      const uint64_t k = cand[threadIdx.x];
      int rank = 0;
      for (int i = 0; i < groups; ++i) rank += cand[i] > k || (cand[i] == k && i < (int)threadIdx.x);
      if (rank == top - 1) best_of[0] = k;
    }
    __syncthreads();
    bound = best_of[0];
    // fewer groups with values than alternatives: everything is a candidate
    if (bound == kNoKey) bound = 1;
    if (mine >= bound) {
      row.each([&](const float (&v)[G], int64_t e) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < G; ++j) {
          const uint64_t k = key_of(v[j], e + j);
          if (k >= bound && e + j < a.V) {
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
        for (int j = 0; j < found; ++j) rank += cand[j] > k;
        if (rank < top) emit(rank, k);
      }
    }
  }
  if (many) {
    uint64_t last = ~0ull;  // above every key
    for (int r = 0; r < top; ++r) {
      uint64_t key = kNoKey;
      row.each([&](const float (&v)[G], int64_t e) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < G; ++j) {
          const uint64_t k = key_of(v[j], e + j);
          if (k < last && e + j < a.V) key = max_key(key, k);
        }
      });
#pragma unroll
      for (int o = kWave / 2; o > 0; o >>= 1) key = max_key(key, shfl_xor_key(key, o));
      __syncthreads();
      if ((threadIdx.x & (kWave - 1)) == 0) best_of[threadIdx.x / kWave] = key;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < NW; ++w) key = max_key(key, best_of[w]);
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

template <typename IO, bool TOP>
void logprobs(const LogprobArgs& a, hipStream_t stream) {
  const int64_t groups = (a.V + kGroup<IO> - 1) / kGroup<IO>;
  const dim3 grid((unsigned)a.N);
#define LRS_LP(BT, NV) hipLaunchKernelGGL((k_logprobs<IO, BT, NV, TOP>), grid, dim3(BT), 0, stream, a)
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
  if (io == kIoBf16) a.top > 0 ? logprobs<uint16_t, true>(a, stream) : logprobs<uint16_t, false>(a, stream);
  else a.top > 0 ? logprobs<float, true>(a, stream) : logprobs<float, false>(a, stream);
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

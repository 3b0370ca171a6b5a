// layernorm.hip -- layer norm over the last axis with the residual added in,
// forward and backward.
//
//   s = x + residual,  mean = sum s / D,  var = sum (s - mean)^2 / D,
//   xh = (s - mean) rstd,  y = xh gamma + beta;
//   q = grad_y gamma,  dx = rstd (q - mean(q) - xh mean(q xh)) + grad_sum,
//   dgamma = sum_rows grad_y xh,  dbeta = sum_rows grad_y.
//
// Memory bound: a row is read once into registers, where the mean and then the
// variance about it are summed in fp32 (no sum of squares minus a square, which
// cancels for rows with a large mean).  A row belongs to TPR threads of a
// workgroup of 256 (64 = one wave, four rows a workgroup; 256) or to 1024
// threads, each holding NV groups of 16 bytes; rows too wide for that are
// walked in three passes (the later ones find the row in the caches).
//
// Measured: 65536 x 1024 bf16 with a residual 91 us forward (5.9 TB/s) and 92 us
// backward (5.8 TB/s; a copy of that size reaches 5.2); 5003 x 1711 fp32 16 and 25 us
// (4.2 TB/s); 8192 x 8192 bf16 without a residual 62 us (4.3 TB/s; 45 where part of the
// input or output is still in the memory-side cache); 64 rows, 4.6 us, are a launch and
// one pass of latency.  Wide rows are read once more for dx and once more for the sums
// over rows: 8192 x 8192 fp32 backward 315 us, 2.6 TB/s of what it has to move.
//
// Groups are read at element alignment (the hardware allows it for global
// memory), so that odd widths take the same path; only the last, incomplete
// group of a row is read element by element.
#include "lrs_device.hpp"
#include "lrs_internal.hpp"

namespace lrs {

namespace {

// Elements of one 16-byte group.
template <typename IO>
constexpr int kGroup = 16 / (int)sizeof(IO);

typedef f32x4_t f32x4_any __attribute__((aligned(4)));
typedef u32x4_t u32x4_any __attribute__((aligned(2)));

// The group at element e of a row of D elements, as it is in memory; 0 past the
// end.  NT: nontemporal (see kStreamFootprint).
template <bool NT, typename IO>
__device__ __forceinline__ u32x4_t ld_raw(const IO* row, int64_t e, int64_t D) {
  u32x4_t q = {0u, 0u, 0u, 0u};
  if (e + kGroup<IO> <= D) {
    const u32x4_any* p = reinterpret_cast<const u32x4_any*>(row + e);
    if constexpr (NT) return __builtin_nontemporal_load(p);
    else return *p;
  }
#pragma unroll
  for (int j = 0; j < kGroup<IO>; ++j) {
    if constexpr (sizeof(IO) == 4) {
      if (e + j < D) q[j] = as_u32(row[e + j]);
    } else {
      if (e + j < D) q[j / 2] |= (uint32_t)row[e + j] << (16 * (j % 2));
    }
  }
  return q;
}
__device__ __forceinline__ void unpack(u32x4_t q, float (&v)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = as_f32(q[j]);
}
__device__ __forceinline__ void unpack(u32x4_t q, float (&v)[8]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v[2 * j] = bf16_lo(q[j]);
    v[2 * j + 1] = bf16_hi(q[j]);
  }
}
template <bool NT, typename IO>
__device__ __forceinline__ void ld_group(const IO* row, int64_t e, int64_t D,
                                         float (&v)[kGroup<IO>]) {
  unpack(ld_raw<NT>(row, e, D), v);
}
template <bool NT>
__device__ __forceinline__ void st_group(float* row, int64_t e, int64_t D, const float (&v)[4]) {
  if (e + 4 <= D) {
    f32x4_any* p = reinterpret_cast<f32x4_any*>(row + e);
    const f32x4_t q = {v[0], v[1], v[2], v[3]};
    if constexpr (NT) __builtin_nontemporal_store(q, p);
    else *p = q;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (e + j < D) row[e + j] = v[j];
  }
}
template <bool NT>
__device__ __forceinline__ void st_group(uint16_t* row, int64_t e, int64_t D, const float (&v)[8]) {
  if (e + 8 <= D) {
    u32x4_t q;
#pragma unroll
    for (int j = 0; j < 4; ++j) q[j] = pack_bf16x2(v[2 * j], v[2 * j + 1]);
    u32x4_any* p = reinterpret_cast<u32x4_any*>(row + e);
    if constexpr (NT) __builtin_nontemporal_store(q, p);
    else *p = q;
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (e + j < D) io_st(row, e + j, v[j]);
  }
}
// Per-feature parameters of a group of G features.
template <int G>
__device__ __forceinline__ void ld_param(const float* p, int64_t e, int64_t D, float (&v)[G]) {
#pragma unroll
  for (int j = 0; j < G; j += 4) {
    if (e + j + 4 <= D) {
      const f32x4_t q = *reinterpret_cast<const f32x4_any*>(p + e + j);
      v[j] = q.x; v[j + 1] = q.y; v[j + 2] = q.z; v[j + 3] = q.w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[j + i] = e + j + i < D ? p[e + j + i] : 0.0f;
    }
  }
}

__device__ __forceinline__ float round_io(float v, const float*) { return v; }
__device__ __forceinline__ float round_io(float v, const uint16_t*) {
  return bf16_lo(pack_bf16x2(v, 0.0f));
}

// Sum over the TPR threads of a row, in a fixed order, returned to all of them.
// TPR > 64: all threads of the workgroup call it; `red` holds TPR/64 floats a
// call, and calls alternate between two of them.
__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int o = kWave / 2; o > 0; o >>= 1) v += __shfl_xor(v, o);
  return v;
}
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* red) {
  v = wave_sum(v);
  if constexpr (TPR > kWave) {
    constexpr int NWR = TPR / kWave;
    if ((threadIdx.x & (kWave - 1)) == 0) red[threadIdx.x / kWave] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int w = 0; w < NWR; ++w) v += red[w];
  }
  return v;
}
// Two sums behind one barrier.
template <int TPR>
__device__ __forceinline__ void row_sums(float& a, float& b, float (*red)[2]) {
  a = wave_sum(a);
  b = wave_sum(b);
  if constexpr (TPR > kWave) {
    constexpr int NWR = TPR / kWave;
    if ((threadIdx.x & (kWave - 1)) == 0) {
      red[threadIdx.x / kWave][0] = a;
      red[threadIdx.x / kWave][1] = b;
    }
    __syncthreads();
    a = b = 0.0f;
#pragma unroll
    for (int w = 0; w < NWR; ++w) {
      a += red[w][0];
      b += red[w][1];
    }
  }
}

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------
template <typename IO, int TPR, int NV, bool NT>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void k_ln_fwd(
    const IO* x, const IO* residual, const float* __restrict__ gamma,
    const float* __restrict__ beta, IO* __restrict__ y, IO* sum, float* __restrict__ mean_out,
    float* __restrict__ rstd_out, int64_t R, int64_t D, float eps) {
  constexpr int G = kGroup<IO>, BT = TPR < 256 ? 256 : TPR;
  __shared__ float red[2][BT / kWave];
  const int t = threadIdx.x % TPR;
  const int64_t row = (int64_t)blockIdx.x * (BT / TPR) + threadIdx.x / TPR;
  if (row >= R) return;  // a whole wave (TPR = 64), or the whole workgroup
  const IO* xr = x + row * D;
  float v[NV][G];
#pragma unroll
  for (int i = 0; i < NV; ++i) ld_group<NT>(xr, ((int64_t)i * TPR + t) * G, D, v[i]);
  if (residual) {
    const IO* rr = residual + row * D;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t e = ((int64_t)i * TPR + t) * G;
      float a[G];
      ld_group<NT>(rr, e, D, a);
#pragma unroll
      for (int j = 0; j < G; ++j) v[i][j] = round_io(v[i][j] + a[j], x);
      st_group<NT>(sum + row * D, e, D, v[i]);
    }
  }
  float part = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < G; ++j) part += v[i][j];
  // divided, not multiplied by 1 / D: a row of one value has exactly that mean,
  // and rstd (up to 1 / sqrt(eps)) would magnify the last bit's error
  const float n = (float)D;
  const float mean = row_sum<TPR>(part, red[0]) / n;
  part = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t e = ((int64_t)i * TPR + t) * G;
#pragma unroll
    for (int j = 0; j < G; ++j) {
      const float c = e + j < D ? v[i][j] - mean : 0.0f;
      v[i][j] = c;
      part = __builtin_fmaf(c, c, part);
    }
  }
  const float var = row_sum<TPR>(part, red[1]) / n;
  const float rstd = 1.0f / sqrtf(var + eps);
  IO* yr = y + row * D;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t e = ((int64_t)i * TPR + t) * G;
    if (e < D) {
      float ga[G], be[G], o[G];
      ld_param<G>(gamma, e, D, ga);
      if (beta) ld_param<G>(beta, e, D, be);
#pragma unroll
      for (int j = 0; j < G; ++j)
        o[j] = __builtin_fmaf(v[i][j] * rstd, ga[j], beta ? be[j] : 0.0f);
      st_group<NT>(yr, e, D, o);
    }
  }
  if (mean_out && t == 0) {
    mean_out[row] = mean;
    rstd_out[row] = rstd;
  }
}

// Rows of any width: 1024 threads walk the row for the mean, the variance and
// the result.
template <typename IO>
__global__ __launch_bounds__(1024) void k_ln_fwd_wide(
    const IO* x, const IO* residual, const float* __restrict__ gamma,
    const float* __restrict__ beta, IO* __restrict__ y, IO* sum, float* __restrict__ mean_out,
    float* __restrict__ rstd_out, int64_t D, float eps) {
  constexpr int G = kGroup<IO>;
  __shared__ float red[2][16];
  const int64_t row = blockIdx.x;
  const IO* xr = x + row * D;
  float part = 0.0f;
  for (int64_t e = (int64_t)threadIdx.x * G; e < D; e += 1024 * G) {
    float v[G];
    ld_group<false>(xr, e, D, v);
    if (residual) {
      float a[G];
      ld_group<false>(residual + row * D, e, D, a);
#pragma unroll
      for (int j = 0; j < G; ++j) v[j] = round_io(v[j] + a[j], x);
      st_group<false>(sum + row * D, e, D, v);
    }
#pragma unroll
    for (int j = 0; j < G; ++j) part += v[j];
  }
  // the later passes read what this thread itself stored
  const IO* sr = residual ? sum + row * D : xr;
  const float n = (float)D;
  const float mean = row_sum<1024>(part, red[0]) / n;
  part = 0.0f;
  for (int64_t e = (int64_t)threadIdx.x * G; e < D; e += 1024 * G) {
    float v[G];
    ld_group<false>(sr, e, D, v);
#pragma unroll
    for (int j = 0; j < G; ++j) {
      const float c = e + j < D ? v[j] - mean : 0.0f;
      part = __builtin_fmaf(c, c, part);
    }
  }
  const float rstd = 1.0f / sqrtf(row_sum<1024>(part, red[1]) / n + eps);
  for (int64_t e = (int64_t)threadIdx.x * G; e < D; e += 1024 * G) {
    float v[G], ga[G], be[G];
    ld_group<false>(sr, e, D, v);
    ld_param<G>(gamma, e, D, ga);
    if (beta) ld_param<G>(beta, e, D, be);
#pragma unroll
    for (int j = 0; j < G; ++j)
      v[j] = __builtin_fmaf((v[j] - mean) * rstd, ga[j], beta ? be[j] : 0.0f);
    st_group<false>(y + row * D, e, D, v);
  }
  if (mean_out && threadIdx.x == 0) {
    mean_out[row] = mean;
    rstd_out[row] = rstd;
  }
}

// ---------------------------------------------------------------------------
// backward: a workgroup walks rows gridDim.x * (rows a workgroup) apart with
// its features' gamma and gradient sums in registers; the sums of its rows go
// to part[0][block][d] (dgamma) and part[1][block][d] (dbeta), which the column
// sums (common.hip) add up in a fixed order.
// ---------------------------------------------------------------------------
template <typename IO, int TPR, int NV, bool NT>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void k_ln_bwd(
    const IO* s, const float* __restrict__ gamma, const float* __restrict__ mean_in,
    const float* __restrict__ rstd_in, const IO* grad_y, const IO* grad_sum, IO* grad_x,
    float* __restrict__ part, int64_t R, int64_t D) {
  constexpr int G = kGroup<IO>, BT = TPR < 256 ? 256 : TPR, RPB = BT / TPR;
  __shared__ float red[2][BT / kWave][2];
  __shared__ float comb[RPB > 1 ? RPB * TPR * G : 1];
  const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  const float inv = 1.0f / (float)D;
  float ga[NV][G], dg[NV][G], db[NV][G];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    ld_param<G>(gamma, ((int64_t)i * TPR + t) * G, D, ga[i]);
#pragma unroll
    for (int j = 0; j < G; ++j) dg[i][j] = db[i][j] = 0.0f;
  }
  // the next row is in flight, packed, while the current one is summed and written
  u32x4_t ns[NV], ng[NV], na[NV];
  float nmean = 0.0f, nrstd = 0.0f;
  auto fetch = [&](int64_t row) __attribute__((always_inline)) {
    nmean = mean_in[row];
    nrstd = rstd_in[row];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t e = ((int64_t)i * TPR + t) * G;
      ns[i] = ld_raw<NT>(s + row * D, e, D);
      ng[i] = ld_raw<NT>(grad_y + row * D, e, D);
      if (grad_sum) na[i] = ld_raw<NT>(grad_sum + row * D, e, D);
    }
  };
  const int64_t stride = (int64_t)gridDim.x * RPB;
  int64_t row = (int64_t)blockIdx.x * RPB + sub;
  if (row < R) fetch(row);
  for (int par = 0; row < R; row += stride, par ^= 1) {
    const float mean = nmean, rstd = nrstd;
    float xh[NV][G], q[NV][G];
    u32x4_t add[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      unpack(ns[i], xh[i]);
      unpack(ng[i], q[i]);
      add[i] = na[i];
    }
    if (row + stride < R) fetch(row + stride);
    float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int j = 0; j < G; ++j) {
        const float h = (xh[i][j] - mean) * rstd, g = q[i][j];  // g and gamma are 0 past the end
        dg[i][j] = __builtin_fmaf(g, h, dg[i][j]);
        db[i][j] += g;
        q[i][j] = g * ga[i][j];
        xh[i][j] = h;
        s1 += q[i][j];
        s2 = __builtin_fmaf(q[i][j], h, s2);
      }
    }
    row_sums<TPR>(s1, s2, red[par]);
    s1 *= inv;
    s2 *= inv;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t e = ((int64_t)i * TPR + t) * G;
      if (e < D) {
        float o[G];
        if (grad_sum) unpack(add[i], o);
#pragma unroll
        for (int j = 0; j < G; ++j) {
          const float d = rstd * (q[i][j] - __builtin_fmaf(xh[i][j], s2, s1));
          o[j] = grad_sum ? d + o[j] : d;
        }
        st_group<NT>(grad_x + row * D, e, D, o);
      }
    }
  }
  // the workgroup's sums: its RPB groups of threads in order
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    float* out = part + ((int64_t)which * gridDim.x + blockIdx.x) * D;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t e = ((int64_t)i * TPR + t) * G;
      float v[G];
#pragma unroll
      for (int j = 0; j < G; ++j) v[j] = which == 0 ? dg[i][j] : db[i][j];
      if constexpr (RPB > 1) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < G; ++j) comb[(sub * G + j) * TPR + t] = v[j];
        __syncthreads();
        if (sub == 0) {
#pragma unroll
          for (int j = 0; j < G; ++j)
            for (int w = 1; w < RPB; ++w) v[j] += comb[(w * G + j) * TPR + t];
        }
      }
      if (sub == 0) {
#pragma unroll
        for (int j = 0; j < G; ++j)
          if (e + j < D) out[e + j] = v[j];
      }
    }
  }
}

// Rows of any width: the row's two sums and dx by 1024 threads.
template <typename IO>
__global__ __launch_bounds__(1024) void k_ln_bwd_wide(
    const IO* s, const float* __restrict__ gamma, const float* __restrict__ mean_in,
    const float* __restrict__ rstd_in, const IO* grad_y, const IO* grad_sum, IO* grad_x,
    int64_t D) {
  constexpr int G = kGroup<IO>;
  __shared__ float red[2][16];
  const int64_t row = blockIdx.x;
  const float mean = mean_in[row], rstd = rstd_in[row], inv = 1.0f / (float)D;
  float s1 = 0.0f, s2 = 0.0f;
  for (int64_t e = (int64_t)threadIdx.x * G; e < D; e += 1024 * G) {
    float x[G], g[G], ga[G];
    ld_group<false>(s + row * D, e, D, x);
    ld_group<false>(grad_y + row * D, e, D, g);
    ld_param<G>(gamma, e, D, ga);
#pragma unroll
    for (int j = 0; j < G; ++j) {
      const float q = g[j] * ga[j];
      s1 += q;
      s2 = __builtin_fmaf(q, (x[j] - mean) * rstd, s2);
    }
  }
  s1 = row_sum<1024>(s1, red[0]) * inv;
  s2 = row_sum<1024>(s2, red[1]) * inv;
  for (int64_t e = (int64_t)threadIdx.x * G; e < D; e += 1024 * G) {
    float x[G], g[G], ga[G], o[G];
    ld_group<false>(s + row * D, e, D, x);
    ld_group<false>(grad_y + row * D, e, D, g);
    ld_param<G>(gamma, e, D, ga);
    if (grad_sum) ld_group<false>(grad_sum + row * D, e, D, o);
#pragma unroll
    for (int j = 0; j < G; ++j) {
      const float d = rstd * (g[j] * ga[j] - __builtin_fmaf((x[j] - mean) * rstd, s2, s1));
      o[j] = grad_sum ? d + o[j] : d;
    }
    st_group<false>(grad_x + row * D, e, D, o);
  }
}

// The weight's gradients of wide rows: block (x, y) sums rows y, y + gridDim.y,
// ... for 256 features.  It runs before k_ln_bwd_wide, which may overwrite
// grad_y.
template <typename IO>
__global__ __launch_bounds__(256) void k_ln_bwd_cols(const IO* s, const float* __restrict__ mean_in,
                                                     const float* __restrict__ rstd_in,
                                                     const IO* grad_y, float* __restrict__ part,
                                                     int64_t R, int64_t D) {
  const int64_t d = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (d >= D) return;
  float dg = 0.0f, db = 0.0f;
  for (int64_t row = blockIdx.y; row < R; row += gridDim.y) {
    const float g = io_ld(grad_y, row * D + d);
    dg = __builtin_fmaf(g, (io_ld(s, row * D + d) - mean_in[row]) * rstd_in[row], dg);
    db += g;
  }
  part[(int64_t)blockIdx.y * D + d] = dg;
  part[((int64_t)gridDim.y + blockIdx.y) * D + d] = db;
}

// Threads a row and groups a thread, from the number of 16-byte groups in a
// row: one wave up to 4 groups a lane, so that no barrier is needed; then 256
// threads; the widest rows 1024, so that they still fit in registers.
struct LnShape {
  int tpr = 0, nv = 0;  // 0: wide rows
};
// most_tpr: the forward goes to 1024 threads a row; the backward, which holds
// four values an element, would spill there and stops at 256.
LnShape ln_shape(int64_t D, int group, int most_tpr) {
  const int64_t n = (D + group - 1) / group;
  LnShape s;
  s.tpr = n <= 256 ? 64 : n <= 1024 ? 256 : 1024;
  const int64_t nv = (n + s.tpr - 1) / s.tpr;
  if (nv > 4 || s.tpr > most_tpr) return LnShape();
  s.nv = nv <= 1 ? 1 : nv <= 2 ? 2 : 4;
  return s;
}

}  // namespace

#define LRS_LN_PICK(LAUNCH, IO)                     \
  if (sh.tpr == 64) {                               \
    if (sh.nv == 1) LAUNCH(IO, 64, 1);              \
    else if (sh.nv == 2) LAUNCH(IO, 64, 2);         \
    else LAUNCH(IO, 64, 4);                         \
  } else if (sh.tpr == 256) {                       \
    if (sh.nv <= 2) LAUNCH(IO, 256, 2);             \
    else LAUNCH(IO, 256, 4);                        \
  }

template <typename IO>
static hipError_t ln_fwd(const IO* x, const IO* residual, const float* gamma, const float* beta,
                         IO* y, IO* sum, float* mean, float* rstd, int64_t R, int64_t D, float eps,
                         hipStream_t stream) {
  const LnShape sh = ln_shape(D, kGroup<IO>, 1024);
  if (sh.tpr == 0) {
    hipLaunchKernelGGL(k_ln_fwd_wide<IO>, dim3((unsigned)R), dim3(1024), 0, stream, x, residual,
                       gamma, beta, y, sum, mean, rstd, D, eps);
    return hipGetLastError();
  }
  const int rpb = sh.tpr < 256 ? 256 / sh.tpr : 1;
  const dim3 grid((unsigned)((R + rpb - 1) / rpb));
  const bool nt = R * D * (residual ? 4 : 2) * (int64_t)sizeof(IO) >= kStreamFootprint;
#define LRS_LN_F(IO_, TPR, NV)                                                                \
  do {                                                                                        \
    const dim3 wg(TPR < 256 ? 256 : TPR);                                                     \
    if (nt)                                                                                   \
      hipLaunchKernelGGL((k_ln_fwd<IO_, TPR, NV, true>), grid, wg, 0, stream, x, residual,    \
                         gamma, beta, y, sum, mean, rstd, R, D, eps);                         \
    else                                                                                      \
      hipLaunchKernelGGL((k_ln_fwd<IO_, TPR, NV, false>), grid, wg, 0, stream, x, residual,   \
                         gamma, beta, y, sum, mean, rstd, R, D, eps);                         \
  } while (0)
  LRS_LN_PICK(LRS_LN_F, IO)
  else if (sh.nv <= 2) LRS_LN_F(IO, 1024, 2);
  else LRS_LN_F(IO, 1024, 4);
#undef LRS_LN_F
  return hipGetLastError();
}

hipError_t launch_layernorm_fwd(const void* x, const void* residual, const float* gamma,
                                const float* beta, void* y, void* sum, float* mean, float* rstd,
                                int64_t R, int64_t D, float eps, int io, hipStream_t stream) {
  if (io == kIoBf16)
    return ln_fwd((const uint16_t*)x, (const uint16_t*)residual, gamma, beta, (uint16_t*)y,
                  (uint16_t*)sum, mean, rstd, R, D, eps, stream);
  return ln_fwd((const float*)x, (const float*)residual, gamma, beta, (float*)y, (float*)sum, mean,
                rstd, R, D, eps, stream);
}

// Four workgroups for each of 256 compute units, as far as there are rows (four
// rows a workgroup where a row is one wave's); more where each would add up more than
// 256 rows in fp32 (a sum of 4000 equal terms is off by 5e-5).
int64_t ln_bwd_blocks(int64_t R, int64_t D) {
  const int64_t need = D <= 1024 ? (R + 3) / 4 : R;
  const int64_t few = (need + 255) / 256;
  return need < 1024 ? need : few < 1024 ? 1024 : few;
}

template <typename IO>
static hipError_t ln_bwd(const IO* s, const float* gamma, const float* mean, const float* rstd,
                         const IO* grad_y, const IO* grad_sum, IO* grad_x, float* grad_gamma,
                         float* grad_beta, int64_t R, int64_t D, float* part, double* acc,
                         hipStream_t stream) {
  const LnShape sh = ln_shape(D, kGroup<IO>, 256);
  const int64_t nb = ln_bwd_blocks(R, D);
  const dim3 grid((unsigned)nb);
  if (sh.tpr == 0) {
    hipLaunchKernelGGL(k_ln_bwd_cols<IO>, dim3((unsigned)((D + 255) / 256), (unsigned)nb), dim3(256),
                       0, stream, s, mean, rstd, grad_y, part, R, D);
    hipLaunchKernelGGL(k_ln_bwd_wide<IO>, dim3((unsigned)R), dim3(1024), 0, stream, s, gamma, mean,
                       rstd, grad_y, grad_sum, grad_x, D);
  } else {
    const bool nt = R * D * (grad_sum ? 4 : 3) * (int64_t)sizeof(IO) >= kStreamFootprint;
#define LRS_LN_B(IO_, TPR, NV)                                                                \
  do {                                                                                        \
    const dim3 wg(TPR < 256 ? 256 : TPR);                                                     \
    if (nt)                                                                                   \
      hipLaunchKernelGGL((k_ln_bwd<IO_, TPR, NV, true>), grid, wg, 0, stream, s, gamma, mean, \
                         rstd, grad_y, grad_sum, grad_x, part, R, D);                         \
    else                                                                                      \
      hipLaunchKernelGGL((k_ln_bwd<IO_, TPR, NV, false>), grid, wg, 0, stream, s, gamma,      \
                         mean, rstd, grad_y, grad_sum, grad_x, part, R, D);                   \
  } while (0)
    LRS_LN_PICK(LRS_LN_B, IO)
#undef LRS_LN_B
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  float* const outs[2] = {grad_gamma, grad_beta};
  return launch_param_sums(part, grad_beta ? 2 : 1, nb, D, acc, outs, stream);
}

hipError_t launch_layernorm_bwd(const void* s, const float* gamma, const float* mean,
                                const float* rstd, const void* grad_y, const void* grad_sum,
                                void* grad_x, float* grad_gamma, float* grad_beta, int64_t R,
                                int64_t D, int io, float* part, double* acc, hipStream_t stream) {
  if (io == kIoBf16)
    return ln_bwd((const uint16_t*)s, gamma, mean, rstd, (const uint16_t*)grad_y,
                  (const uint16_t*)grad_sum, (uint16_t*)grad_x, grad_gamma, grad_beta, R, D, part,
                  acc, stream);
  return ln_bwd((const float*)s, gamma, mean, rstd, (const float*)grad_y, (const float*)grad_sum,
                (float*)grad_x, grad_gamma, grad_beta, R, D, part, acc, stream);
}

}  // namespace lrs

// rmsnorm.hip -- root-mean-square norm over the last axis with the residual added in,
// forward (also to 8 bits with scales) and backward.
//
//   s = x + residual,  rstd = 1 / sqrt(sum s^2 / D + eps),  y = s rstd gamma;
//   8 bits: scale = max |y| / 448 over a group, q = y / scale in e4m3;
//   xh = s rstd,  g = grad_y gamma,  dx = rstd (g - xh mean(g xh)) + grad_sum,
//   dgamma = sum_rows grad_y xh.
//
// Memory bound: a row is read once into the registers of 64 threads (one wave, four rows
// a workgroup), 256 or 1024, each holding NV groups of 16 bytes; rows too wide for that
// are walked in two or three passes (the later ones find the row in the caches).  The 8-bit
// form needs y's largest value before the first byte is written: with the row in registers
// that is a maximum over 16 (bf16) or 32 (fp32) lanes for groups of 128, and one more sum
// over the row's threads for a scale a row.
//
// Measured: 16384 x 4096 bf16 with residual to 8 bits 84 to 89 us (5.3 to 5.6 TB/s); 32768 x
// 2048 bf16 with residual forward 88 us (6.1 TB/s), backward 97 us and 5 us for the column
// sums, with nontemporal accesses (a copy of 1 GiB reaches 5.1 TB/s); 5003 x 1711 fp32, whose
// rows do not begin on 16 bytes, 14, 22 and 5.5 us; 64 x 1024 4.2 us.
#include "lrs_device.hpp"
#include "lrs_internal.hpp"
#include "lrs_rows.hpp"

namespace lrs {

namespace {

constexpr float kMostE4m3 = 448.0f;
constexpr float kLeastScale = 0x1p-120f;

// What the forward writes: y in the I/O type, or 8 bits with a scale for 128 features
// or for the row.
enum { kOutIo = 0, kOutGroup = 1, kOutRow = 2 };

// v / by in fp32, by inv = 1 / by: their product, less what it is off by.  The product alone
// rounds twice, and now and then takes the neighbour at a border between two bytes; a division
// for every value takes 88.0 us where this takes 86.0 (16384 x 4096 bf16 with residual).  The
// quotient is the division's at every border, and for 448 at every v, as long as what is left
// of v does not fall below fp32's range.
__device__ __forceinline__ float quotient(float v, float by, float inv) {
  const float q = v * inv;
  return __builtin_fmaf(__builtin_fmaf(q, by, -v), -inv, q);  // signs that keep a -0
}
constexpr float kLeastExact = 0x1p-90f;  // of `by`: 24 bits of it times 24 of 2^-10 stay above 2^-149

// A group's scale and what y is divided by, from the bits of its largest |y|.
__device__ __forceinline__ float group_scale(uint32_t top, float& by) {
  const float m = as_f32(top);
  if (top >= 0x7F800000u) {  // NaN and infinities: every value of the group is NaN
    by = __builtin_nanf("");
    return m;
  }
  by = m == 0.0f ? 1.0f : fmaxf(quotient(m, kMostE4m3, 1.0f / kMostE4m3), kLeastScale);
  return by;
}
__device__ __forceinline__ uint32_t max_bits(uint32_t a, uint32_t b) { return a > b ? a : b; }
template <int G>
__device__ __forceinline__ uint32_t top_bits(const float (&v)[G]) {
  uint32_t m = 0u;
#pragma unroll
  for (int j = 0; j < G; ++j) m = max_bits(m, as_u32(v[j]) & 0x7FFFFFFFu);
  return m;
}
// The largest over N neighbouring lanes.
template <int N>
__device__ __forceinline__ uint32_t lanes_max(uint32_t m) {
#pragma unroll
  for (int o = N / 2; o > 0; o >>= 1) m = max_bits(m, (uint32_t)__shfl_xor((int)m, o));
  return m;
}
// The largest over the TPR threads of a row; as row_sum.
template <int TPR>
__device__ __forceinline__ uint32_t row_max(uint32_t m, uint32_t* red) {
  m = lanes_max<kWave>(m);
  if constexpr (TPR > kWave) {
    if ((threadIdx.x & (kWave - 1)) == 0) red[threadIdx.x / kWave] = m;
    __syncthreads();
    m = 0u;
#pragma unroll
    for (int w = 0; w < TPR / kWave; ++w) m = max_bits(m, red[w]);
  }
  return m;
}

typedef uint32_t u32_any __attribute__((aligned(1)));
typedef uint32_t u32x2_bytes __attribute__((ext_vector_type(2), aligned(1)));


// G values divided by `by`, rounded to e4m3, at element e of a row of D bytes.
template <int G>
__device__ __forceinline__ void st_e4m3(uint8_t* row, int64_t e, int64_t D, const float (&v)[G],
                                        float by) {
  float r[G];
  if (by < kLeastExact) {
#pragma unroll
    for (int j = 0; j < G; ++j) r[j] = v[j] / by;
  } else {
    const float inv = 1.0f / by;
#pragma unroll
    for (int j = 0; j < G; ++j) r[j] = quotient(v[j], by, inv);
  }
  uint32_t q[G / 4];
#pragma unroll
  for (int j = 0; j < G; j += 4) {
    int p = __builtin_amdgcn_cvt_pk_fp8_f32(r[j], r[j + 1], 0, false);
    p = __builtin_amdgcn_cvt_pk_fp8_f32(r[j + 2], r[j + 3], p, true);
    q[j / 4] = (uint32_t)p;
  }
  if (e + G <= D) {
    if constexpr (G == 8) *reinterpret_cast<u32x2_bytes*>(row + e) = u32x2_t{q[0], q[1]};
    else *reinterpret_cast<u32_any*>(row + e) = q[0];
    return;
  }
#pragma unroll
  for (int j = 0; j < G; ++j)
    if (e + j < D) row[e + j] = (uint8_t)(q[j / 4] >> (8 * (j % 4)));
}

// ---------------------------------------------------------------------------
// forward
// ---------------------------------------------------------------------------
template <typename IO, int TPR, int NV, bool NT, int OUT>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void k_rms_fwd(
    const IO* x, const IO* residual, const float* __restrict__ gamma, void* __restrict__ y,
    float* __restrict__ scales, IO* sum, float* __restrict__ rstd_out, int64_t R, int64_t D,
    float eps) {
  constexpr int G = kGroup<IO>, BT = TPR < 256 ? 256 : TPR;
  __shared__ float red[BT / kWave];
  __shared__ uint32_t redm[BT / kWave];
  const int t = threadIdx.x % TPR;
  const int64_t row = (int64_t)blockIdx.x * (BT / TPR) + threadIdx.x / TPR;
  if (row >= R) return;  // a whole wave (TPR = 64), or the whole workgroup
  const IO* xr = x + row * D;
  float v[NV][G];
#pragma unroll
  for (int i = 0; i < NV; ++i) ld_group<NT>(xr, ((int64_t)i * TPR + t) * G, D, v[i]);
  if (residual) {
    const IO* rr = residual + row * D;
    float a[NV][G];
#pragma unroll
    for (int i = 0; i < NV; ++i) ld_group<NT>(rr, ((int64_t)i * TPR + t) * G, D, a[i]);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t e = ((int64_t)i * TPR + t) * G;
#pragma unroll
      for (int j = 0; j < G; ++j) v[i][j] = round_io(v[i][j] + a[i][j], x);
      st_group<NT>(sum + row * D, e, D, v[i]);
    }
  }
  float part = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int j = 0; j < G; ++j) part = __builtin_fmaf(v[i][j], v[i][j], part);
  const float rstd = 1.0f / sqrtf(row_sum<TPR>(part, red) / (float)D + eps);
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t e = ((int64_t)i * TPR + t) * G;
    float ga[G];
    ld_param<G>(gamma, e, D, ga);  // 0 past the end
#pragma unroll
    for (int j = 0; j < G; ++j) v[i][j] = v[i][j] * rstd * ga[j];
  }
  if constexpr (OUT == kOutIo) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t e = ((int64_t)i * TPR + t) * G;
      if (e < D) st_group<NT>((IO*)y + row * D, e, D, v[i]);
    }
    if (rstd_out && t == 0) rstd_out[row] = rstd;
    return;
  }
  uint32_t top = 0u;
  float by = 1.0f;
  if constexpr (OUT == kOutRow) {
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < G; ++j)
        if (((int64_t)i * TPR + t) * G + j < D) top = max_bits(top, as_u32(v[i][j]) & 0x7FFFFFFFu);
    const float s = group_scale(row_max<TPR>(top, redm), by);
    if (t == 0) scales[row] = s;
  }
  const int64_t groups = (D + 127) / 128;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t e = ((int64_t)i * TPR + t) * G;
    if constexpr (OUT == kOutGroup) {
      float in[G];  // an infinite rstd makes NaN of the zeros past the end
#pragma unroll
      for (int j = 0; j < G; ++j) in[j] = e + j < D ? v[i][j] : 0.0f;
      const float s = group_scale(lanes_max<128 / G>(top_bits(in)), by);
      if (e % 128 == 0 && e < D) scales[row * groups + e / 128] = s;
    }
    if (e < D) st_e4m3<G>((uint8_t*)y + row * D, e, D, v[i], by);
  }
}

// Rows of any width: 1024 threads walk the row for the sum, the largest value of a row's
// scale, and the result.
template <typename IO, int OUT>
__global__ __launch_bounds__(1024) void k_rms_fwd_wide(
    const IO* x, const IO* residual, const float* __restrict__ gamma, void* __restrict__ y,
    float* __restrict__ scales, IO* sum, float* __restrict__ rstd_out, int64_t D, float eps) {
  constexpr int G = kGroup<IO>;
  __shared__ float red[16];
  __shared__ uint32_t redm[16];
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
    for (int j = 0; j < G; ++j) part = __builtin_fmaf(v[j], v[j], part);
  }
  // the later passes read what this thread itself stored
  const IO* sr = residual ? sum + row * D : xr;
  const float rstd = 1.0f / sqrtf(row_sum<1024>(part, red) / (float)D + eps);
  if (rstd_out && threadIdx.x == 0) rstd_out[row] = rstd;
  auto value = [&](int64_t e, float (&v)[G]) __attribute__((always_inline)) {
    float ga[G];
    ld_group<false>(sr, e, D, v);
    ld_param<G>(gamma, e, D, ga);
#pragma unroll
    for (int j = 0; j < G; ++j) v[j] = e + j < D ? v[j] * rstd * ga[j] : 0.0f;
  };
  float by = 1.0f;
  if constexpr (OUT == kOutRow) {
    uint32_t top = 0u;
    for (int64_t e = (int64_t)threadIdx.x * G; e < D; e += 1024 * G) {
      float v[G];
      value(e, v);
      top = max_bits(top, top_bits(v));
    }
    const float s = group_scale(row_max<1024>(top, redm), by);
    if (threadIdx.x == 0) scales[row] = s;
  }
  const int64_t groups = (D + 127) / 128;
  for (int64_t e0 = 0; e0 < D; e0 += 1024 * G) {  // whole waves, for the groups' largest
    const int64_t e = e0 + (int64_t)threadIdx.x * G;
    float v[G];
    value(e, v);
    if constexpr (OUT == kOutGroup) {
      const float s = group_scale(lanes_max<128 / G>(top_bits(v)), by);
      if (e % 128 == 0 && e < D) scales[row * groups + e / 128] = s;
    }
    if (e >= D) continue;
    if constexpr (OUT == kOutIo) st_group<false>((IO*)y + row * D, e, D, v);
    else st_e4m3<G>((uint8_t*)y + row * D, e, D, v, by);
  }
}

// ---------------------------------------------------------------------------
// backward: a workgroup walks rows gridDim.x * (rows a workgroup) apart with its
// features' gamma and gradient sums in registers, the next row in flight; the sums of its
// rows go to part[block][d], which the column sums (common.hip) add up in a fixed order.
// ---------------------------------------------------------------------------
template <typename IO, int TPR, int NV, bool NT>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void k_rms_bwd(
    const IO* s, const float* __restrict__ gamma, const float* __restrict__ rstd_in,
    const IO* grad_y, const IO* grad_sum, IO* grad_x, float* __restrict__ part, int64_t R,
    int64_t D) {
  constexpr int G = kGroup<IO>, BT = TPR < 256 ? 256 : TPR, RPB = BT / TPR;
  __shared__ float red[2][BT / kWave];
  __shared__ float comb[RPB > 1 ? RPB * TPR * G : 1];
  const int t = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  const float inv = 1.0f / (float)D;
  float ga[NV][G], dg[NV][G];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    ld_param<G>(gamma, ((int64_t)i * TPR + t) * G, D, ga[i]);
#pragma unroll
    for (int j = 0; j < G; ++j) dg[i][j] = 0.0f;
  }
  u32x4_t ns[NV], ng[NV], na[NV];
  float nrstd = 0.0f;
  auto fetch = [&](int64_t row) __attribute__((always_inline)) {
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
    const float rstd = nrstd;
    float xh[NV][G], q[NV][G];
    u32x4_t add[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      unpack(ns[i], xh[i]);
      unpack(ng[i], q[i]);
      add[i] = na[i];
    }
    if (row + stride < R) fetch(row + stride);
    float s2 = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
#pragma unroll
      for (int j = 0; j < G; ++j) {
        const float h = xh[i][j] * rstd, g = q[i][j];  // g and gamma are 0 past the end
        dg[i][j] = __builtin_fmaf(g, h, dg[i][j]);
        q[i][j] = g * ga[i][j];
        xh[i][j] = h;
        s2 = __builtin_fmaf(q[i][j], h, s2);
      }
    }
    s2 = row_sum<TPR>(s2, red[par]) * inv;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int64_t e = ((int64_t)i * TPR + t) * G;
      if (e < D) {
        float o[G];
        if (grad_sum) unpack(add[i], o);
#pragma unroll
        for (int j = 0; j < G; ++j) {
          const float d = rstd * __builtin_fmaf(-xh[i][j], s2, q[i][j]);
          o[j] = grad_sum ? d + o[j] : d;
        }
        st_group<NT>(grad_x + row * D, e, D, o);
      }
    }
  }
  // the workgroup's sums: its RPB groups of threads in order
  float* out = part + (int64_t)blockIdx.x * D;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int64_t e = ((int64_t)i * TPR + t) * G;
    float v[G];
#pragma unroll
    for (int j = 0; j < G; ++j) v[j] = dg[i][j];
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

// Rows of any width: the row's sum and dx by 1024 threads.
template <typename IO>
__global__ __launch_bounds__(1024) void k_rms_bwd_wide(
    const IO* s, const float* __restrict__ gamma, const float* __restrict__ rstd_in,
    const IO* grad_y, const IO* grad_sum, IO* grad_x, int64_t D) {
  constexpr int G = kGroup<IO>;
  __shared__ float red[16];
  const int64_t row = blockIdx.x;
  const float rstd = rstd_in[row], inv = 1.0f / (float)D;
  float s2 = 0.0f;
  for (int64_t e = (int64_t)threadIdx.x * G; e < D; e += 1024 * G) {
    float x[G], g[G], ga[G];
    ld_group<false>(s + row * D, e, D, x);
    ld_group<false>(grad_y + row * D, e, D, g);
    ld_param<G>(gamma, e, D, ga);
#pragma unroll
    for (int j = 0; j < G; ++j) s2 = __builtin_fmaf(g[j] * ga[j], x[j] * rstd, s2);
  }
  s2 = row_sum<1024>(s2, red) * inv;
  for (int64_t e = (int64_t)threadIdx.x * G; e < D; e += 1024 * G) {
    float x[G], g[G], ga[G], o[G];
    ld_group<false>(s + row * D, e, D, x);
    ld_group<false>(grad_y + row * D, e, D, g);
    ld_param<G>(gamma, e, D, ga);
    if (grad_sum) ld_group<false>(grad_sum + row * D, e, D, o);
#pragma unroll
    for (int j = 0; j < G; ++j) {
      const float d = rstd * __builtin_fmaf(-(x[j] * rstd), s2, g[j] * ga[j]);
      o[j] = grad_sum ? d + o[j] : d;
    }
    st_group<false>(grad_x + row * D, e, D, o);
  }
}

// The weight's gradient of wide rows: block (x, y) sums rows y, y + gridDim.y, ... for 256
// features.  It runs before k_rms_bwd_wide, which may overwrite grad_y.
template <typename IO>
__global__ __launch_bounds__(256) void k_rms_bwd_cols(const IO* s, const float* __restrict__ rstd_in,
                                                      const IO* grad_y, float* __restrict__ part,
                                                      int64_t R, int64_t D) {
  const int64_t d = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (d >= D) return;
  float dg = 0.0f;
  for (int64_t row = blockIdx.y; row < R; row += gridDim.y)
    dg = __builtin_fmaf(io_ld(grad_y, row * D + d), io_ld(s, row * D + d) * rstd_in[row], dg);
  part[(int64_t)blockIdx.y * D + d] = dg;
}

template <typename IO, int OUT>
hipError_t rms_fwd(const void* x_, const void* residual_, const float* gamma, void* y,
                   float* scales, void* sum_, float* rstd, int64_t R, int64_t D, float eps,
                   hipStream_t stream) {
  const IO *x = (const IO*)x_, *residual = (const IO*)residual_;
  IO* sum = (IO*)sum_;
  const LnShape sh = ln_shape(D, kGroup<IO>, 1024);
  if (sh.tpr == 0) {
    hipLaunchKernelGGL((k_rms_fwd_wide<IO, OUT>), dim3((unsigned)R), dim3(1024), 0, stream, x,
                       residual, gamma, y, scales, sum, rstd, D, eps);
    return hipGetLastError();
  }
  const int rpb = sh.tpr < 256 ? 256 / sh.tpr : 1;
  const dim3 grid((unsigned)((R + rpb - 1) / rpb));
  const bool nt = R * D * ((residual ? 3 : 1) * (int64_t)sizeof(IO) + (OUT == kOutIo ? sizeof(IO) : 1)) >=
                  kStreamFootprint;
#define LRS_RMS_F(IO_, TPR, NV)                                                                   \
  do {                                                                                            \
    const dim3 wg(TPR < 256 ? 256 : TPR);                                                         \
    if (nt)                                                                                       \
      hipLaunchKernelGGL((k_rms_fwd<IO_, TPR, NV, true, OUT>), grid, wg, 0, stream, x, residual,  \
                         gamma, y, scales, sum, rstd, R, D, eps);                                 \
    else                                                                                          \
      hipLaunchKernelGGL((k_rms_fwd<IO_, TPR, NV, false, OUT>), grid, wg, 0, stream, x, residual, \
                         gamma, y, scales, sum, rstd, R, D, eps);                                 \
  } while (0)
  LRS_LN_PICK(LRS_RMS_F, IO)
  else if (sh.nv <= 2) LRS_RMS_F(IO, 1024, 2);
  else LRS_RMS_F(IO, 1024, 4);
#undef LRS_RMS_F
  return hipGetLastError();
}

template <typename IO>
hipError_t rms_bwd(const void* s_, const float* gamma, const float* rstd, const void* gy_,
                   const void* gsum_, void* gx_, float* grad_gamma, int64_t R, int64_t D,
                   float* part, double* acc, hipStream_t stream) {
  const IO *s = (const IO*)s_, *grad_y = (const IO*)gy_, *grad_sum = (const IO*)gsum_;
  IO* grad_x = (IO*)gx_;
  const LnShape sh = ln_shape(D, kGroup<IO>, 256);
  const int64_t nb = rms_bwd_blocks(R, D);
  const dim3 grid((unsigned)nb);
  if (sh.tpr == 0) {
    hipLaunchKernelGGL(k_rms_bwd_cols<IO>, dim3((unsigned)((D + 255) / 256), (unsigned)nb),
                       dim3(256), 0, stream, s, rstd, grad_y, part, R, D);
    hipLaunchKernelGGL(k_rms_bwd_wide<IO>, dim3((unsigned)R), dim3(1024), 0, stream, s, gamma, rstd,
                       grad_y, grad_sum, grad_x, D);
  } else {
    const bool nt = R * D * (grad_sum ? 4 : 3) * (int64_t)sizeof(IO) >= kStreamFootprint;
#define LRS_RMS_B(IO_, TPR, NV)                                                                \
  do {                                                                                         \
    const dim3 wg(TPR < 256 ? 256 : TPR);                                                      \
    if (nt)                                                                                    \
      hipLaunchKernelGGL((k_rms_bwd<IO_, TPR, NV, true>), grid, wg, 0, stream, s, gamma, rstd, \
                         grad_y, grad_sum, grad_x, part, R, D);                                \
    else                                                                                       \
      hipLaunchKernelGGL((k_rms_bwd<IO_, TPR, NV, false>), grid, wg, 0, stream, s, gamma,      \
                         rstd, grad_y, grad_sum, grad_x, part, R, D);                          \
  } while (0)
    LRS_LN_PICK(LRS_RMS_B, IO)
#undef LRS_RMS_B
  }
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  float* const outs[1] = {grad_gamma};
  return launch_param_sums(part, 1, nb, D, acc, outs, stream);
}

}  // namespace

hipError_t launch_rmsnorm_fwd(const void* x, const void* residual, const float* gamma, void* y,
                              void* sum, float* rstd, int64_t R, int64_t D, float eps, int io,
                              hipStream_t stream) {
  return io == kIoBf16 ? rms_fwd<uint16_t, kOutIo>(x, residual, gamma, y, nullptr, sum, rstd, R, D,
                                                   eps, stream)
                       : rms_fwd<float, kOutIo>(x, residual, gamma, y, nullptr, sum, rstd, R, D, eps,
                                                stream);
}

hipError_t launch_rmsnorm_fp8(const void* x, const void* residual, const float* gamma, void* y,
                              float* scales, void* sum, int64_t R, int64_t D, int64_t group,
                              float eps, int io, hipStream_t stream) {
#define LRS_RMS_Q(IO, OUT) \
  return rms_fwd<IO, OUT>(x, residual, gamma, y, scales, sum, nullptr, R, D, eps, stream)
  if (io == kIoBf16) {
    if (group == 128) LRS_RMS_Q(uint16_t, kOutGroup);
    LRS_RMS_Q(uint16_t, kOutRow);
  }
  if (group == 128) LRS_RMS_Q(float, kOutGroup);
  LRS_RMS_Q(float, kOutRow);
#undef LRS_RMS_Q
}

// As for the layer norm's backward: four workgroups a compute unit as far as there are
// rows, and at most 256 rows a workgroup, which it adds up in fp32.
int64_t rms_bwd_blocks(int64_t R, int64_t D) { return ln_bwd_blocks(R, D); }

hipError_t launch_rmsnorm_bwd(const void* s, const float* gamma, const float* rstd,
                              const void* grad_y, const void* grad_sum, void* grad_x,
                              float* grad_gamma, int64_t R, int64_t D, int io, float* part,
                              double* acc, hipStream_t stream) {
  return io == kIoBf16 ? rms_bwd<uint16_t>(s, gamma, rstd, grad_y, grad_sum, grad_x, grad_gamma, R,
                                           D, part, acc, stream)
                       : rms_bwd<float>(s, gamma, rstd, grad_y, grad_sum, grad_x, grad_gamma, R, D,
                                        part, acc, stream);
}

}  // namespace lrs

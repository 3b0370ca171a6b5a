// lrs_rows.hpp -- reading, summing and writing the rows of an [R,D] array, for the
// kernels that hold a row in the registers of 64, 256 or 1024 threads.
//
// Groups are read at element alignment (the hardware allows it for global
// memory), so that odd widths take the same path; only the last, incomplete
// group of a row is read element by element.
#pragma once

#include "lrs_device.hpp"

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

}  // namespace lrs

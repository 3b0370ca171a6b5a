// lrs_host.hpp -- host-side helpers of the C ABI files: size checks, overlap
// and alignment tests, workspace carving.  Not installed.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/lrs.h"

namespace {

constexpr size_t kAlign = 256;

size_t align_up(size_t x) { return (x + kAlign - 1) & ~(kAlign - 1); }

bool mul_ok(int64_t a, int64_t b, int64_t* out) {
  return !__builtin_mul_overflow(a, b, out);
}

// B*D*T without overflow, and small enough that byte offsets fit in int64.
bool shape_ok(int64_t B, int64_t D, int64_t T, int64_t* C, int64_t* N) {
  if (B < 0 || D < 0 || T < 0) return false;
  if (!mul_ok(B, D, C) || !mul_ok(*C, T, N)) return false;
  return *N <= ((int64_t)1 << 60);
}

bool aligned(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

bool overlap(const void* p, size_t pn, const void* q, size_t qn) {
  if (!p || !q || pn == 0 || qn == 0) return false;
  const uintptr_t a = (uintptr_t)p, b = (uintptr_t)q;
  return a < b + qn && b < a + pn;
}

struct Carve {
  char* base;
  size_t used = 0;
  explicit Carve(void* ws) : base((char*)ws) {}
  template <typename T>
  T* take(int64_t n) {
    if (n <= 0) return nullptr;
    T* p = (T*)(base + used);
    used = align_up(used + (size_t)n * sizeof(T));
    return p;
  }
};

// Bytes to carve `nstatus` 64-bit words + `ntickets` counters (+ slack so the
// caller's pointer need not be aligned).
size_t lookback_bytes(int64_t nstatus, int64_t ntickets) {
  if (nstatus <= 0) return 0;
  return kAlign + align_up((size_t)nstatus * 8) + align_up((size_t)ntickets * 4);
}

void* align_ptr(void* p) { return (void*)(((uintptr_t)p + kAlign - 1) & ~(uintptr_t)(kAlign - 1)); }

int hip_status(hipError_t e) { return e == hipSuccess ? LRS_OK : LRS_ERR_HIP; }

// Launch-size guard: HIP grids are limited to 2^32-1 work-items per dimension.
bool grid_ok(int64_t blocks, int threads) { return blocks > 0 && blocks * threads < (1ll << 32); }

}  // namespace

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

struct Span {
  const void* p;
  size_t n;
};

bool any_overlap(const Span* outs, int no, const Span* ins, int ni) {
  for (int o = 0; o < no; ++o) {
    for (int i = 0; i < ni; ++i)
      if (overlap(outs[o].p, outs[o].n, ins[i].p, ins[i].n)) return true;
    for (int o2 = o + 1; o2 < no; ++o2)
      if (overlap(outs[o].p, outs[o].n, outs[o2].p, outs[o2].n)) return true;
  }
  return false;
}

// Bytes from the first to past the last element of `rows` rows of D elements,
// ld apart.
size_t strided_bytes(int64_t rows, int64_t ld, int64_t D, size_t es) {
  return rows <= 0 ? 0 : ((size_t)(rows - 1) * (size_t)ld + (size_t)D) * es;
}

// Whether two sets of `rows` rows of D elements, each ld apart, share an
// element: their extents may interleave (slices of one wider array).
bool rows_overlap(const void* p, const void* q, int64_t rows, int64_t ld, int64_t D, size_t es) {
  const size_t n = strided_bytes(rows, ld, D, es);
  if (!overlap(p, n, q, n)) return false;
  const uintptr_t a = (uintptr_t)p, b = (uintptr_t)q;
  const size_t off = (size_t)(a < b ? b - a : a - b) % ((size_t)ld * es);
  return !(off >= (size_t)D * es && off <= (size_t)(ld - D) * es);
}

bool io_ok(int io) { return io == LRS_F32 || io == LRS_BF16; }
size_t io_size(int io) { return io == LRS_BF16 ? 2 : 4; }

// Pitched extents inside int64 bytes.
bool pitch_ok(int64_t T, int64_t B, int64_t ld) {
  int64_t rows, n;
  return mul_ok(T, B, &rows) && mul_ok(rows, ld, &n) && n <= ((int64_t)1 << 60);
}

// Whether two sets of `rows` rows share an element: rows of dp and dq elements, ldp and
// ldq apart, which may interleave where the pitch is the same (slices of one wider array).
bool slices_overlap(const void* p, int64_t ldp, int64_t dp, const void* q, int64_t ldq, int64_t dq,
                    int64_t rows, size_t es) {
  if (!overlap(p, strided_bytes(rows, ldp, dp, es), q, strided_bytes(rows, ldq, dq, es)))
    return false;
  if (ldp != ldq) return true;
  const uintptr_t a = (uintptr_t)p, b = (uintptr_t)q;
  const size_t da = (size_t)(a <= b ? dp : dq) * es, db = (size_t)(a <= b ? dq : dp) * es;
  const size_t off = (size_t)(a <= b ? b - a : a - b) % ((size_t)ldp * es);
  return !(off >= da && off + db <= (size_t)ldp * es);
}

}  // namespace

// Rows of a paged cache, for the kernels that write them and read them back
// (paged_cache.cu, paged_rope.cu): where they lie, and their codes.
#pragma once

#include <cuda_fp8.h>

#include "paged_util.cuh"

namespace dfl {

// Two values over s, y = 1 / s correctly rounded, as float32 quotients.  The
// quotient's rounding matters, since values that lie exactly half way between
// two codes are common (0.75 of the largest value is one).  q = x y is a unit or
// two in the last place off, r = x - q s is exact in a fused operation, and
// q + r y rounded once is the quotient (P. Markstein, "Computation of elementary
// functions on the IBM RISC System/6000 processor", 1990), three operations
// where a division takes ten or more.  A scale so small that y or r could leave
// float32's range takes the division (quotients_small).
__device__ __forceinline__ float2 quotients(float2 x, float s, float y) {
  const float2 y2 = make_float2(y, y), ms = make_float2(-s, -s);
  const float2 q = mul2(x, y2);
  return fma2(fma2(q, ms, x), y2, q);
}
__device__ __forceinline__ bool quotients_small(float s) { return s < 0x1p-100f; }
__device__ __forceinline__ float2 quotients_slow(float2 x, float s) {
  return make_float2(__fdiv_rn(x.x, s), __fdiv_rn(x.y, s));
}

struct Place {
  bool owned;  // some request owns the row
  bool there;  // and its position has a row of the cache
  long long page;
  int at;
  int pos;     // of an owned row
};

// What a block learns from the requests that fit the call.
struct Found {
  int b0;    // the first one that ends after the block's first row
  int end;   // the row behind the last that any of them owns: none from there on is touched
  int odd;   // some request does not fit: row_start need not rise
};
template <int THREADS>
__device__ __forceinline__ void look_through(const PagedBatch& p, int n0, int* status, Found* found) {
  if (threadIdx.x == 0) *found = {p.B, 0, 0};
  __syncthreads();
  int b0 = p.B, end = 0, odd = 0;
  for (int b = threadIdx.x; b < p.B; b += THREADS) {
    RequestSpan r;
    if (!request_span(p, b, &r)) {
      odd = 1;
      if (blockIdx.x == 0) report_status(status, DFLASH_ERR_SHAPE);
    } else if (r.n > 0) {
      if (r.s0 + r.n > n0) b0 = min(b0, b);
      end = max(end, r.s0 + r.n);
    }
  }
  if (b0 < p.B) atomicMin(&found->b0, b0);
  if (end) atomicMax(&found->end, end);
  if (odd) found->odd = 1;
  __syncthreads();
}

__device__ __forceinline__ Place find_row(const PagedBatch& p, const Found& found, int n, int* status) {
  Place r = {false, false, 0, 0, 0};
  RequestSpan sp;
  int b = found.b0;
  for (;; ++b) {
    if (b >= p.B) return r;
    if (__ldg(p.row_start + b + 1) <= n || !request_span(p, b, &sp)) continue;
    if (n >= sp.s0) break;
    if (!found.odd) return r;  // rows before the first request's
  }
  r.owned = true;
  const int pos = sp.len - sp.n + (n - sp.s0);
  r.pos = pos;
  if (pos < 0) {
    report_status(status, DFLASH_ERR_SHAPE);
    return r;
  }
  const int page = __ldg(p.table + b * p.table_stride + (pos >> p.page_shift));
  if (page < 0 || page >= p.n_pages) {
    report_status(status, DFLASH_ERR_ARG);
    return r;
  }
  r.there = true;
  r.page = page;
  r.at = pos & ((1 << p.page_shift) - 1);
  return r;
}

// E2M1: two codes (the first in the lower half of the byte) of two values,
// rounded to nearest, ties to even, at most 6; and two codes as fp16, exactly.
__device__ __forceinline__ uint32_t e2m1x2(float2 x) {
  uint32_t r;
  asm("{\n\t.reg .b8 c;\n\tcvt.rn.satfinite.e2m1x2.f32 c, %2, %1;\n\tcvt.u32.u8 %0, c;\n\t}"
      : "=r"(r)
      : "f"(x.x), "f"(x.y));
  return r;
}

}  // namespace dfl

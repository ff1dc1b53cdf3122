// Small device helpers of the attention kernels over an E2M1 cache
// (paged_attention_e2m1.cu, paged_attention_e2m1_rows.cu).
#pragma once

#include "paged_line.cuh"

namespace dfl {
namespace line {

// What either kernel wants of a call beside the line of work.
struct E2m1Args : LineArgs {
  const uint8_t *k_pages, *v_pages;
  long long k_stride, v_stride;
  int bf16;   // type of queries and outputs
  int slots;  // tiles of codes on their way
};

__device__ __forceinline__ void bulk_load(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_u32(dst)),
      "l"(src), "r"(bytes), "r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ bool any_of(int id, int threads, bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 p, %3, 0;\n\tbar.red.or.pred q, %1, %2, p;\n\tselp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(threads), "r"((uint32_t)p)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ void st_shared_x4(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
template <int N>
__device__ __forceinline__ void reg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}

// The largest scale of a record (its magnitude's bits), of the blocks that hold values:
// append gives a block of zeros a scale of 1, and a power of two taken from that would pull
// the references up, or leave the other blocks' products without places.  Such scales
// become 0.  Only where 1 is the largest can they matter (beside larger ones they are below
// the row's power of two), and codes are read only there: blocks of 8 139 -> 142 us, prompt
// chunk 923 -> 937.  (A vote before the branch, or a look at one such block before all:
// 172 and 160 us for blocks of 8.)
template <int HD>
__device__ __forceinline__ uint32_t largest_scale(uint32_t (&scale)[HD / 32], const uint8_t* rec) {
  auto largest = [&] {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < HD / 32; ++i) m = __vmaxu2(m, scale[i] & 0x7FFF7FFFu);
    return max(m & 0xFFFFu, m >> 16);
  };
  uint32_t m = largest();
  if (m == 0x3F80u) {
#pragma unroll
    for (int i = 0; i < HD / 32; ++i) {
      const uint2 c0 = *reinterpret_cast<const uint2*>(rec + 16 * i), c1 = *reinterpret_cast<const uint2*>(rec + 16 * i + 8);
      if (!((c0.x | c0.y) & 0x77777777u)) scale[i] &= 0xFFFF0000u;
      if (!((c1.x | c1.y) & 0x77777777u)) scale[i] &= 0x0000FFFFu;
    }
    m = largest();
  }
  return m;
}
// Rows of zeros in V still weigh in l.  Their power of two is 2^-32 of the largest among the
// 32 neighbours that a warp holds, so that they pull no reference up and their weights stay
// far from float32's end; 2^-32 where all of those are zeros (a biased exponent).
constexpr int kZeroBelow = 32, kZeroV = 127 - 32;

// Queries as fp16: 8 values of a row by each of kCh lanes (powers of two), times the power
// of two that brings the row's largest to [2^14, 2^15); *e gets the biased exponent of
// that largest (15 at least, 255 for a row that is not finite: it becomes NaN).
template <int kCh>
__device__ __forceinline__ uint4 widen_q(uint4 w, int bf16, int* e) {
  uint32_t v[4] = {w.x, w.y, w.z, w.w};
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = __vmaxu2(m, v[i] & 0x7FFF7FFFu);
#pragma unroll
  for (int o = kCh / 2; o > 0; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
  m = max(m & 0xFFFFu, m >> 16);
  const float top = bf16 ? unpack16<true>(m).x : unpack16<false>(m).x;
  *e = max((int)(__float_as_uint(top) >> 23), 15);
  const float f = *e < 255 ? __uint_as_float((uint32_t)(268 - *e) << 23) : __uint_as_float(0x7FC00000u);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 y = bf16 ? unpack16<true>(v[i]) : unpack16<false>(v[i]);
    v[i] = pack16<false>(y.x * f, y.y * f);
  }
  return make_uint4(v[0], v[1], v[2], v[3]);
}
// What a score of such a row is multiplied by.
__device__ __forceinline__ float q_factor(int e, float scale_log2) {
  return scale_log2 * __uint_as_float((uint32_t)(min(e, 254) - 14) << 23);
}

}  // namespace line

// paged_attention_e2m1_rows.cu: calls with more than 128 packed rows to a request.
int launch_paged_attention_e2m1_rows(line::E2m1Args& k, int head_dim, cudaStream_t s);

}  // namespace dfl

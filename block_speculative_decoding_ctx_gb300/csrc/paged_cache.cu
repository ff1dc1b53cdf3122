// Writing rows of keys and values into a paged cache, quantised to E4M3 on the
// way if the cache is, and reading them back (dflash_paged_append and
// dflash_paged_gather; the rules are in include/dflash.h).
//
// Both move every byte once and compute next to nothing, so memory (or, for a
// step's few rows, the latency of the dependent loads row_start -> kv_len ->
// page_table) bounds them.  A thread moves 16 values of one (row, KV head,
// K or V): 32 bytes on the 16-bit side and 32 or 16 on the cache's, so 8 or 4
// neighbouring threads hold a whole row of head_dim values and find its
// largest magnitude with shuffles.
#include <cuda_fp8.h>

#include "paged_util.cuh"

namespace dfl {
namespace {

constexpr int kMoveThreads = 256;
constexpr float kE4M3Max = 448.0f;

struct Place {
  bool owned;  // some request owns the row
  bool there;  // and its position has a row of the cache
  long long page;
  int at;
};

// First request that ends after row n0, found by the whole block.
__device__ __forceinline__ int first_request(const PagedBatch& p, int n0, int* status) {
  __shared__ int b0;
  if (threadIdx.x == 0) b0 = p.B;
  __syncthreads();
  int mine = p.B;
  for (int b = threadIdx.x; b < p.B; b += kMoveThreads) {
    if (__ldg(p.row_start + b + 1) > n0) mine = min(mine, b);
    RequestSpan r;
    if (blockIdx.x == 0 && !request_span(p, b, &r)) report_status(status, DFLASH_ERR_SHAPE);
  }
  if (mine < p.B) atomicMin(&b0, mine);
  __syncthreads();
  return b0;
}

__device__ __forceinline__ Place find_row(const PagedBatch& p, int b, int n, int* status) {
  Place r = {false, false, 0, 0};
  while (b < p.B && __ldg(p.row_start + b + 1) <= n) ++b;
  RequestSpan sp;
  if (b >= p.B || !request_span(p, b, &sp) || n < sp.s0) return r;
  r.owned = true;
  const int pos = sp.len - sp.n + (n - sp.s0);
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

template <int HD, bool E4M3, bool BF16, bool APPEND>
__global__ void __launch_bounds__(kMoveThreads) paged_move_kernel(const PagedMoveArgs a) {
  pdl_enter();
  constexpr int kLanes = HD / 16;                   // threads per (row, head, side)
  constexpr int kUnits = kMoveThreads / kLanes;     // (row, head, side) per block
  constexpr int kCell = E4M3 ? 1 : 2;               // bytes of a cached value
  const long long u0 = (long long)blockIdx.x * kUnits;
  const int per_row = 2 * a.n_kv;
  const int b0 = first_request(a.batch, (int)(u0 / per_row), a.status);

  const long long u = u0 + threadIdx.x / kLanes;
  const int lane = threadIdx.x % kLanes;
  const long long n = u / per_row;
  const int hs = (int)(u - n * per_row), side = hs >= a.n_kv, head = side ? hs - a.n_kv : hs;
  Place pl = {false, false, 0, 0};
  if (n < a.batch.rows) pl = find_row(a.batch, b0, (int)n, a.status);

  uint8_t* x = a.x[side] + ((size_t)n * a.row_stride[side] + (size_t)head * a.head_stride[side] + lane * 16) * 2;
  const size_t row = ((size_t)head << a.batch.page_shift) + pl.at;   // row of the page
  uint8_t* cell = a.pages[side] + ((size_t)pl.page * a.page_stride[side] + row * HD + lane * 16) * kCell;
  float* scale = E4M3 ? a.scale[side] + ((((size_t)pl.page * a.n_kv) << a.batch.page_shift) + row) : nullptr;

  if (APPEND) {
    uint4 w[2] = {};
    if (pl.there) {
      w[0] = __ldg(reinterpret_cast<const uint4*>(x));
      w[1] = __ldg(reinterpret_cast<const uint4*>(x) + 1);
    }
    if (!E4M3) {
      if (pl.there) {
        reinterpret_cast<uint4*>(cell)[0] = w[0];
        reinterpret_cast<uint4*>(cell)[1] = w[1];
      }
      return;
    }
    // magnitudes of both types order like their bits, NaN above infinity
    const uint32_t v[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = __vmaxu2(m, v[i] & 0x7FFF7FFFu);
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
    m = max(m & 0xFFFFu, m >> 16);
    const bool finite = m < (BF16 ? 0x7F80u : 0x7C00u);
    const float amax = unpack16<BF16>(m).x;
    const float s = !finite ? __uint_as_float(0x7FC00000u) : m ? __fdiv_rn(amax, kE4M3Max) : 1.0f;
    if (!pl.there) return;
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = unpack16<BF16>(v[2 * i]), g = unpack16<BF16>(v[2 * i + 1]);
      const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(f.x, s), __fdiv_rn(f.y, s)),
                                                   __NV_SATFINITE, __NV_E4M3);
      const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(__fdiv_rn(g.x, s), __fdiv_rn(g.y, s)),
                                                   __NV_SATFINITE, __NV_E4M3);
      c[i] = lo | (hi << 16);
    }
    *reinterpret_cast<uint4*>(cell) = make_uint4(c[0], c[1], c[2], c[3]);
    if (lane == 0) *scale = s;
  } else {
    if (!pl.owned) return;
    uint4 w[2] = {};
    if (pl.there) {
      if (E4M3) {
        const uint4 c = __ldg(reinterpret_cast<const uint4*>(cell));
        const float s = __ldg(scale);
        const uint32_t v[4] = {c.x, c.y, c.z, c.w};
        uint32_t o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t h = e4m3x2_to_f16x2((uint16_t)(v[i / 2] >> (16 * (i & 1))));
          const float2 f = unpack16<false>(h);
          o[i] = pack16<BF16>(f.x * s, f.y * s);
        }
        w[0] = make_uint4(o[0], o[1], o[2], o[3]);
        w[1] = make_uint4(o[4], o[5], o[6], o[7]);
      } else {
        w[0] = __ldg(reinterpret_cast<const uint4*>(cell));
        w[1] = __ldg(reinterpret_cast<const uint4*>(cell) + 1);
      }
    }
    reinterpret_cast<uint4*>(x)[0] = w[0];
    reinterpret_cast<uint4*>(x)[1] = w[1];
  }
}

template <int HD, bool E4M3, bool BF16, bool APPEND>
int launch_move(const PagedMoveArgs& a, cudaStream_t s) {
  const long long units = (long long)a.batch.rows * 2 * a.n_kv;
  const long long per = kMoveThreads / (HD / 16);
  const long long grid = units > 0 ? (units + per - 1) / per : 1;
  if (grid > 0x7FFFFFFFll) return DFLASH_ERR_SHAPE;
  return launch_pdl(paged_move_kernel<HD, E4M3, BF16, APPEND>, dim3((unsigned)grid), dim3(kMoveThreads), 0, s, a);
}

template <bool APPEND>
int dispatch(const PagedMoveArgs& a, int head_dim, int format, int type, cudaStream_t s) {
  const bool bf = type == DFLASH_TYPE_BF16, e = format == DFLASH_CACHE_E4M3;
  if (head_dim == 128) {
    if (!e) return launch_move<128, false, false, APPEND>(a, s);
    return bf ? launch_move<128, true, true, APPEND>(a, s) : launch_move<128, true, false, APPEND>(a, s);
  }
  if (!e) return launch_move<64, false, false, APPEND>(a, s);
  return bf ? launch_move<64, true, true, APPEND>(a, s) : launch_move<64, true, false, APPEND>(a, s);
}

}  // namespace

int launch_paged_append(const PagedMoveArgs& a, int head_dim, int format, int type, cudaStream_t s) {
  return dispatch<true>(a, head_dim, format, type, s);
}
int launch_paged_gather(const PagedMoveArgs& a, int head_dim, int format, int type, cudaStream_t s) {
  return dispatch<false>(a, head_dim, format, type, s);
}

}  // namespace dfl

// Attention of new rows over a paged cache (dflash_paged_attention; the rules
// are in include/dflash.h): one warp per (row, query head), the keys one after
// another with a running maximum and sum.
#include "paged_util.cuh"

namespace dfl {
namespace {

template <int HD, bool E4M3, bool BF16>
__global__ void __launch_bounds__(256) paged_attention_kernel(const PagedAttnArgs a) {
  pdl_enter();
  const PagedBatch& p = a.batch;
  const int lane = threadIdx.x & 31, head = blockIdx.y, b = blockIdx.z;
  const int j = blockIdx.x * 8 + (threadIdx.x >> 5);
  RequestSpan r;
  if (!request_span(p, b, &r) || r.n > a.max_rows) {
    if (threadIdx.x == 0) report_status(a.status, DFLASH_ERR_SHAPE);
    return;
  }
  if (j >= r.n) return;
  constexpr int kE = HD / 32;  // values per lane
  const size_t row = r.s0 + j;
  const int kv = head / a.group;
  float q[kE], o[kE], m = -INFINITY, l = 0.0f;
  auto load = [&](const uint8_t* x, float (&f)[kE]) {  // kE 16-bit values
    const uint32_t* w = reinterpret_cast<const uint32_t*>(x);
#pragma unroll
    for (int i = 0; i < kE / 2; ++i) {
      const float2 t = unpack16<BF16>(__ldg(w + i));
      f[2 * i] = t.x;
      f[2 * i + 1] = t.y;
    }
  };
  load(a.q + (row * a.q_row + (size_t)head * a.q_head + lane * kE) * 2, q);
#pragma unroll
  for (int i = 0; i < kE; ++i) o[i] = 0.0f;
  const int pos = r.len - r.n + j;
  const int hi = a.causal ? min(r.len, pos + 1) : r.len;
  const int lo = a.window ? max(0, pos - a.window + 1) : 0;
  for (int s = lo; s < hi; ++s) {
    const int page = __ldg(p.table + b * p.table_stride + (s >> p.page_shift));
    const bool there = page >= 0 && page < p.n_pages;
    if (!there) report_status(a.status, DFLASH_ERR_ARG);
    const size_t at = ((size_t)kv << p.page_shift) + (s & ((1 << p.page_shift) - 1));
    float k[kE] = {}, v[kE] = {};
    if (there) {
      const size_t ko = (size_t)page * a.k_page_stride + at * HD + lane * kE;
      const size_t vo = (size_t)page * a.v_page_stride + at * HD + lane * kE;
      if (E4M3) {
        const size_t so = (((size_t)page * a.n_kv) << p.page_shift) + at;
        const float ks = __ldg(a.k_scale + so), vs = __ldg(a.v_scale + so);
#pragma unroll
        for (int i = 0; i < kE; i += 2) {
          const float2 kf = unpack16<false>(e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(a.k_pages + ko + i)));
          const float2 vf = unpack16<false>(e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t*>(a.v_pages + vo + i)));
          k[i] = kf.x * ks;
          k[i + 1] = kf.y * ks;
          v[i] = vf.x * vs;
          v[i + 1] = vf.y * vs;
        }
      } else {
        load(a.k_pages + ko * 2, k);
        load(a.v_pages + vo * 2, v);
      }
    }
    float z = 0.0f;
#pragma unroll
    for (int i = 0; i < kE; ++i) z = fmaf(q[i], k[i], z);
    z = warp_sum(z) * a.scale_log2;
    const float mn = fmaxf(m, z);
    const float f = m == -INFINITY ? 0.0f : exp2f(m - mn), w = exp2f(z - mn);
    m = mn;
    l = l * f + w;
#pragma unroll
    for (int i = 0; i < kE; ++i) o[i] = fmaf(o[i], f, w * v[i]);
  }
  const float inv = l > 0.0f ? 1.0f / l : (l == l ? 0.0f : l);
  uint32_t* out = reinterpret_cast<uint32_t*>(a.out + (row * a.o_row + (size_t)head * a.o_head + lane * kE) * 2);
#pragma unroll
  for (int i = 0; i < kE / 2; ++i) out[i] = pack16<BF16>(o[2 * i] * inv, o[2 * i + 1] * inv);
  if (a.lse && lane == 0) a.lse[row * a.n_q + head] = (m + log2f(l)) * 0.693147180559945309f;
}

template <int HD, bool E4M3, bool BF16>
int launch(const PagedAttnArgs& a, cudaStream_t s) {
  return launch_pdl(paged_attention_kernel<HD, E4M3, BF16>, dim3(ceil_div(a.max_rows, 8), a.n_q, a.batch.B), dim3(256), 0, s, a);
}

}  // namespace

size_t paged_attention_workspace(int, int, int, int) { return kWsHeader; }

int launch_paged_attention(const PagedAttnArgs& a, int head_dim, int format, int type, void*, cudaStream_t s) {
  const bool bf = type == DFLASH_TYPE_BF16, e = format == DFLASH_CACHE_E4M3;
  if (head_dim == 128) {
    if (e) return bf ? launch<128, true, true>(a, s) : launch<128, true, false>(a, s);
    return bf ? launch<128, false, true>(a, s) : launch<128, false, false>(a, s);
  }
  if (e) return bf ? launch<64, true, true>(a, s) : launch<64, true, false>(a, s);
  return bf ? launch<64, false, true>(a, s) : launch<64, false, false>(a, s);
}

}  // namespace dfl

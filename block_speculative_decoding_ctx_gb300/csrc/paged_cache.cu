// Writing rows of keys and values into a paged cache, quantised to E4M3 on the
// way if the cache is, and reading them back (dflash_paged_append and
// dflash_paged_gather; the rules are in include/dflash.h).  paged_rope.cu writes
// E2M1 caches; they are read back here.
//
// Both move every byte once and compute next to nothing, so memory (or, for a
// step's few rows, the latency of the dependent loads row_start -> kv_len ->
// page_table) bounds them.  A block has a few rows; one thread each finds
// their places in the cache, once for all heads, K and V.  Then a thread moves
// 16 values of one (row, KV head, K or V) at a time, two such pieces on their
// way: 32 bytes each on the 16-bit side and 32 or 16 on the cache's, so that 8
// or 4 neighbouring threads hold a whole row of head_dim values and find its
// largest magnitude with shuffles.
//
// Measured on GB300 (8 KV heads of 128), bytes at the measured copy's rate in
// brackets: E4M3 prefixes read back (776 MB) 119 us [0.96]; 16-bit prompts
// written 57 us [0.92]; the same quantised on the way (274 MB) 58 us [0.70],
// which instructions bound (66% of the issue slots; 250 a warp for 16 values a
// thread, some 80 of them quotients, conversions, maxima and packing, most others
// addresses); a step's 256 rows 8 us, latency.  E2M1 prompts read back (237 MB) 46 us
// [0.77].
#include "paged_rows.cuh"

namespace dfl {
namespace {

constexpr int kMoveThreads = 256;
constexpr float kE4M3Max = 448.0f;
// Pieces of a thread on their way: 1 / 2 / 4 take 65 / 59 / 73 us to quantise
// prompts and 123 / 119 / 124 to read prefixes back.
constexpr int kPieces = 2;
// Pieces of one block (128 / 256 / 512: prompts 60.4 / 58.6 / 60.5 us, prefixes
// 120.6 / 119.3 / 123.0), and the number of blocks (4 for each of 152 SMs) that
// comes first: a step's few rows are spread over as many.
constexpr int kMostUnits = 256, kBlocks = 608;

// E4M3 codes of 16 values over s: x / s rounded to float32, then to E4M3.
template <bool BF16>
__device__ __forceinline__ uint4 quantize16(const uint32_t (&v)[8], float s) {
  const float y = __fdiv_rn(1.0f, s);
  uint32_t c[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    c[i] = __nv_cvt_float2_to_fp8x2(quotients(unpack16<BF16>(v[i]), s, y), __NV_SATFINITE, __NV_E4M3);
  if (quotients_small(s)) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      c[i] = __nv_cvt_float2_to_fp8x2(quotients_slow(unpack16<BF16>(v[i]), s), __NV_SATFINITE, __NV_E4M3);
  }
  return make_uint4(c[0] | (c[1] << 16), c[2] | (c[3] << 16), c[4] | (c[5] << 16), c[6] | (c[7] << 16));
}

// rows: of a block, at most kMoveThreads.
template <int HD, int FORMAT, bool BF16, bool APPEND>
__global__ void __launch_bounds__(kMoveThreads) paged_move_kernel(const PagedMoveArgs a, int rows) {
  pdl_enter();
  constexpr bool E4M3 = FORMAT == DFLASH_CACHE_E4M3, E2M1 = FORMAT == DFLASH_CACHE_E2M1;
  static_assert(!(E2M1 && APPEND), "paged_rope.cu writes those");
  constexpr int kLanes = HD / 16;                   // threads per (row, head, side)
  constexpr int kUnits = kMoveThreads / kLanes;     // (row, head, side) at once
  constexpr int kCell = E4M3 ? 1 : 2;               // bytes of a cached value
  __shared__ Place places[kMoveThreads];
  __shared__ Found found;
  const int n0 = blockIdx.x * rows, lane = threadIdx.x % kLanes;
  const uint32_t per_row = 2u * a.n_kv;
  look_through<kMoveThreads>(a.batch, n0, a.status, &found);
  const int mine = max(0, min(rows, found.end - n0));
  const uint32_t units = mine * per_row;

  struct Piece {
    int row, head, side;  // row of the block
    uint8_t* x;
  };
  auto piece = [&](uint32_t u) {
    Piece p;
    p.row = (int)(u / per_row);
    const int hs = (int)(u - p.row * per_row);
    p.side = hs >= a.n_kv;
    p.head = p.side ? hs - a.n_kv : hs;
    p.x = a.x[p.side] +
          ((size_t)(n0 + p.row) * a.row_stride[p.side] + (size_t)p.head * a.head_stride[p.side] + lane * 16) * 2;
    return p;
  };
  uint4 w[kPieces][2] = {};
  auto load_rows = [&](uint32_t u0) {
#pragma unroll
    for (int q = 0; q < kPieces; ++q) {
      const uint32_t u = u0 + q * kUnits;
      if (u < units) {
        const uint4* x = reinterpret_cast<const uint4*>(piece(u).x);
        w[q][0] = __ldg(x);
        w[q][1] = __ldg(x + 1);
      }
    }
  };
  // the first rows are on their way while the places are looked up
  if (APPEND) load_rows(threadIdx.x / kLanes);
  if ((int)threadIdx.x < mine) places[threadIdx.x] = find_row(a.batch, found, n0 + threadIdx.x, a.status);
  __syncthreads();

  // whole warps stay together: pieces past the last take part in the shuffles
  const uint32_t turns = (units + kUnits * kPieces - 1) / (kUnits * kPieces);
  for (uint32_t turn = 0; turn < turns; ++turn) {
    const uint32_t u0 = turn * (kUnits * kPieces) + threadIdx.x / kLanes;
    uint8_t *x[kPieces], *cell[kPieces];
    float* scale[kPieces];
    bool owned[kPieces], there[kPieces];
#pragma unroll
    for (int q = 0; q < kPieces; ++q) {
      const uint32_t u = u0 + q * kUnits;
      const Piece p = piece(min(u, units - 1));
      const Place pl = places[p.row];
      x[q] = p.x;
      owned[q] = pl.owned && u < units;
      there[q] = pl.there && u < units;
      const size_t row = ((size_t)p.head << a.batch.page_shift) + pl.at;
      cell[q] = E2M1 ? a.pages[p.side] + (size_t)pl.page * a.page_stride[p.side] + row * e2m1_record(HD) + lane * 8
                     : a.pages[p.side] + ((size_t)pl.page * a.page_stride[p.side] + row * HD + lane * 16) * kCell;
      scale[q] = a.scale[p.side] + (((size_t)pl.page * a.n_kv) << a.batch.page_shift) + row;
    }
    if (APPEND) {
#pragma unroll
      for (int q = 0; q < kPieces; ++q) {
        if (!E4M3) {
          if (there[q]) {
            reinterpret_cast<uint4*>(cell[q])[0] = w[q][0];
            reinterpret_cast<uint4*>(cell[q])[1] = w[q][1];
          }
          continue;
        }
        // magnitudes of both types order like their bits, NaN above infinity
        const uint32_t v[8] = {w[q][0].x, w[q][0].y, w[q][0].z, w[q][0].w, w[q][1].x, w[q][1].y, w[q][1].z, w[q][1].w};
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) m = __vmaxu2(m, v[i] & 0x7FFF7FFFu);
#pragma unroll
        for (int o = kLanes / 2; o > 0; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
        m = max(m & 0xFFFFu, m >> 16);
        const bool finite = m < (BF16 ? 0x7F80u : 0x7C00u);
        const float amax = unpack16<BF16>(m).x;
        const float s = !finite ? __uint_as_float(0x7FC00000u) : m ? __fdiv_rn(amax, kE4M3Max) : 1.0f;
        if (!there[q]) continue;
        *reinterpret_cast<uint4*>(cell[q]) = quantize16<BF16>(v, s);
        if (lane == 0) *scale[q] = s;
      }
      if (turn + 1 < turns) load_rows(u0 + kUnits * kPieces);
    } else {
      uint4 c[kPieces];
      float s[kPieces];
#pragma unroll
      for (int q = 0; q < kPieces; ++q) {
        w[q][0] = w[q][1] = make_uint4(0u, 0u, 0u, 0u);
        if (!there[q]) continue;
        if (E2M1) {
          const uint2 w8 = __ldg(reinterpret_cast<const uint2*>(cell[q]));
          c[q] = make_uint4(w8.x, w8.y, 0u, 0u);
          s[q] = __uint_as_float((uint32_t)__ldg(reinterpret_cast<const uint16_t*>(cell[q] + HD / 2 - lane * 6)) << 16);
        } else if (E4M3) {
          c[q] = __ldg(reinterpret_cast<const uint4*>(cell[q]));
          s[q] = __ldg(scale[q]);
        } else {
          w[q][0] = __ldg(reinterpret_cast<const uint4*>(cell[q]));
          w[q][1] = __ldg(reinterpret_cast<const uint4*>(cell[q]) + 1);
        }
      }
#pragma unroll
      for (int q = 0; q < kPieces; ++q) {
        if (!owned[q]) continue;
        if (E2M1 && there[q]) {
          uint32_t f[8], o[8];
          e2m1x8_to_f16x2(c[q].x, reinterpret_cast<uint32_t(&)[4]>(f[0]));
          e2m1x8_to_f16x2(c[q].y, reinterpret_cast<uint32_t(&)[4]>(f[4]));
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float2 x2 = unpack16<false>(f[i]);
            o[i] = pack16<BF16>(x2.x * s[q], x2.y * s[q]);
          }
          w[q][0] = make_uint4(o[0], o[1], o[2], o[3]);
          w[q][1] = make_uint4(o[4], o[5], o[6], o[7]);
        }
        if (E4M3 && there[q]) {
          const uint32_t v[4] = {c[q].x, c[q].y, c[q].z, c[q].w};
          uint32_t o[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float2 f = unpack16<false>(e4m3x2_to_f16x2((uint16_t)(v[i / 2] >> (16 * (i & 1)))));
            o[i] = pack16<BF16>(f.x * s[q], f.y * s[q]);
          }
          w[q][0] = make_uint4(o[0], o[1], o[2], o[3]);
          w[q][1] = make_uint4(o[4], o[5], o[6], o[7]);
        }
        reinterpret_cast<uint4*>(x[q])[0] = w[q][0];
        reinterpret_cast<uint4*>(x[q])[1] = w[q][1];
      }
    }
  }
}

template <int HD, int FORMAT, bool BF16, bool APPEND>
int launch_move(const PagedMoveArgs& a, cudaStream_t s) {
  const int per_row = 2 * a.n_kv, at_once = kMoveThreads / (HD / 16);
  const long long units = (long long)a.batch.rows * per_row;
  const long long each = min((long long)kMostUnits, max((long long)at_once, units / kBlocks));
  const int rows = min(kMoveThreads, max(1, (int)(each / per_row)));
  const int grid = max(1, ceil_div(a.batch.rows, rows));
  return launch_pdl(paged_move_kernel<HD, FORMAT, BF16, APPEND>, dim3(grid), dim3(kMoveThreads), 0, s, a, rows);
}

// The 16-bit formats move alike.
template <int HD, bool APPEND>
int dispatch(const PagedMoveArgs& a, int format, int type, cudaStream_t s) {
  const bool bf = type == DFLASH_TYPE_BF16;
  if (format == DFLASH_CACHE_E4M3)
    return bf ? launch_move<HD, DFLASH_CACHE_E4M3, true, APPEND>(a, s)
              : launch_move<HD, DFLASH_CACHE_E4M3, false, APPEND>(a, s);
  if constexpr (!APPEND) {
    if (format == DFLASH_CACHE_E2M1)
      return bf ? launch_move<HD, DFLASH_CACHE_E2M1, true, APPEND>(a, s)
                : launch_move<HD, DFLASH_CACHE_E2M1, false, APPEND>(a, s);
  }
  return launch_move<HD, DFLASH_CACHE_F16, false, APPEND>(a, s);
}

}  // namespace

int launch_paged_append(const PagedMoveArgs& a, int head_dim, int format, int type, cudaStream_t s) {
  return head_dim == 128 ? dispatch<128, true>(a, format, type, s) : dispatch<64, true>(a, format, type, s);
}
int launch_paged_gather(const PagedMoveArgs& a, int head_dim, int format, int type, cudaStream_t s) {
  return head_dim == 128 ? dispatch<128, false>(a, format, type, s) : dispatch<64, false>(a, format, type, s);
}

}  // namespace dfl

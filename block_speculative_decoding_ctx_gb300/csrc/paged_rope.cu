// Writing rows of keys and values into a paged cache with positions rotated into
// the keys, and into queries beside them (dflash_paged_append_rope), and writing
// E2M1 caches with or without (dflash_paged_append); the rules are in
// include/dflash.h.
//
//   a' = f (a cos t - b sin t),  b' = f (b cos t + a sin t),  t = P w_j
//
// Every byte is moved once and a value takes a handful of operations, so memory
// bounds it (or, for a step's few rows, the latency of row_start -> kv_len ->
// page_table).  A block has a few rows.  It finds their places and makes their
// sines and cosines once for all heads: P times w_j / (2 pi) in 2^-64ths of a
// turn is a product of integers modulo 2^64, exact for any position; what is left
// of it beside the nearest quarter turn is at most an eighth of a turn and becomes
// two float32s.
//   Then a thread moves 16 values of one (row, head of q, k or v) at a time, two
// such pieces on their way: two runs of 8 values, for a rotated row of layout
// HALF the two whose values are each other's pairs (values 8 l and rotary_dim / 2
// + 8 l on), else neighbours.  rotary_dim is a multiple of 32, so that a block of
// 16 values (E2M1) is two lanes' lower runs, two lanes' upper runs or one lane's
// both, and one shuffle finds its largest magnitude.
//
// Measured on GB300 (40 query and 8 KV heads of 128), calls back to back, bytes at the
// measured copy's rate in brackets: prompts rotated into a 16-bit cache, queries beside
// them (782 MB) 125 us [0.93], into E4M3 (728 MB) 151 us [0.72], into 4 bits (705 MB) 134
// us [0.79]; prompts into 4 bits as they come (237 MB) 50 us [0.70], 57 with L2 flushed
// [0.62].  The last one's loads are asked for only after the turn before has stored all
// (54 % of the issue slots, 194 instructions a warp for 16 values a thread).  The rotated,
// quantised ones have more alive than the 64 registers that four blocks an SM leave a
// thread: 8 bytes stored and 48 loaded again into E4M3, 28 and 60 into 4 bits (the fp16
// append into 4 bits without rotation 28 and 40, the others none).  A step's 256 rows 11 to
// 13 us, the host's launch.  The sweeps below are of this code, in the same four cases.
#include "paged_rows.cuh"

namespace dfl {
namespace {

constexpr int kThreads = 256;  // (128: 133 / 160 / 133 / 56 us)
// Pieces of a thread on their way (with rotation, 1 / 2 / 3: 130 / 125 / 132 us, into E4M3
// 148 / 151 / 193, into 4 bits 123 / 134 / 159: one count for all).
constexpr int kPieces = 2;
constexpr int kMaxRows = 32;   // of a block
// (row, head) of a block, as far as that is no single row (256 / 512 / 1,024: rotated prompts
// 129 / 125 / 132 us, into E4M3 156 / 151 / 151, into 4 bits 139 / 134 / 135, prompts into 4
// bits as they come 54 / 50 / 50).
constexpr int kMostUnits = 512;

// Cosine and sine of `turns` 2^-64ths of a turn, times f, each rounded about once: what
// they turn is rounded into 4 bits next, and a value that falls on the other side of a
// code's border is a whole step off (with sincospif, 1.8e-5 of the 16-bit results differ for
// 1.4e-5, as fast).  Beside the nearest quarter turn, the
// angle is p + e, p a float32 of at most pi / 4 and e its rest; Taylor's series of sine to
// p^11 and of cosine to p^10 (2^-36 and 2^-33 are left out), added to their first terms last.
__device__ __forceinline__ float2 cos_sin(unsigned long long turns, float f) {
  const uint32_t quarter = (uint32_t)((turns + (1ull << 61)) >> 62);
  const long long rest = (long long)(turns - ((unsigned long long)quarter << 62));
  const float h = (float)(int)(rest >> 32);
  const float low = (float)(rest - ((long long)(int)h << 32));
  constexpr double kTurn = 6.283185307179586 / 4294967296.0;  // 2^-32 of a turn
  constexpr float kHi = (float)kTurn, kLo = (float)(kTurn - (double)kHi), kLow = (float)(kTurn / 4294967296.0);
  const float p = h * kHi, e = fmaf(h, kHi, -p) + fmaf(h, kLo, low * kLow);
  const float t = p * p, t_rest = fmaf(p, p, -t);
  float s3 = fmaf(t, -1.0f / 39916800.0f, 1.0f / 362880.0f);  // (sine / p - 1) / t
  s3 = fmaf(t, fmaf(t, fmaf(t, s3, -1.0f / 5040.0f), 1.0f / 120.0f), -1.0f / 6.0f);
  float c4 = fmaf(t, -1.0f / 3628800.0f, 1.0f / 40320.0f);  // (cosine - 1 + t / 2) / t^2
  c4 = fmaf(t, fmaf(t, c4, -1.0f / 720.0f), 1.0f / 24.0f);
  const float w = fmaf(t, -0.5f, 1.0f), w_rest = fmaf(t, -0.5f, 1.0f - w);  // 1 - t / 2
  const float s_rest = fmaf(p * t, s3, e * fmaf(t * t, c4, w));
  const float c_rest = w_rest + fmaf(t * t, c4, fmaf(-0.5f, t_rest, -e * fmaf(p * t, s3, p)));
  const float s = fmaf(p, f, s_rest * f), c = fmaf(w, f, c_rest * f);
  const float x = quarter & 1 ? s : c, y = quarter & 1 ? c : s;
  // quarter 0: (c, s)  1: (-s, c)  2: (-c, -s)  3: (s, -c)
  return make_float2(quarter == 1 || quarter == 2 ? -x : x, quarter >= 2 ? -y : y);
}
// x c - y s and y c + x s.  (Adding the rounded product's rounding back, Kahan's difference
// of products, makes 1.2e-5 of the 16-bit results other than the exact ones' rounding for
// 1.4e-5, and rotated prompts take 132 us for 125, into 4 bits 146 for 134.)
__device__ __forceinline__ void turn2(float2& x, float2& y, float2 c, float2 s) {
  const float2 ns = make_float2(-s.x, -s.y);
  const float2 a = fma2(x, c, mul2(y, ns)), b = fma2(y, c, mul2(x, s));
  x = a;
  y = b;
}

// Where a row goes.
struct Spot {
  uint8_t* page[2];  // of K and of V, or null: nowhere
  int id, at;        // the page's, and row of a head there
  int pos;           // below 0: none, or no row of a request's
};

// The larger magnitudes of two pairs, under signs of no meaning; NaN where either is.
template <bool BF16>
__device__ __forceinline__ uint32_t max_abs(uint32_t a, uint32_t b) {
  uint32_t r;
  if (BF16)
    asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else
    asm("max.NaN.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Scales for which quotients() is not made come to a size where it is, and their values
// along: the quotient stays.
__device__ __forceinline__ void raise(float2* x, float& s) {
  if (!quotients_small(s)) return;
#pragma unroll
  for (int e = 0; e < 4; ++e) x[e] = mul2(x[e], make_float2(0x1p100f, 0x1p100f));
  s *= 0x1p100f;
}

struct Piece {
  int row, slot;        // of the block; head of q, then k, then v
  int c0, c1;           // first columns of its two runs
  bool turned;
  const uint8_t* x;
};

// ROPE: else a plain append (an E2M1 cache's).
template <int HD, int FORMAT, bool BF16, bool ROPE>
__global__ void __launch_bounds__(kThreads, 4) paged_rope_kernel(const PagedRopeArgs a, int rows, uint32_t magic) {
  pdl_enter();
  constexpr bool E4M3 = FORMAT == DFLASH_CACHE_E4M3, E2M1 = FORMAT == DFLASH_CACHE_E2M1;
  constexpr int kLanes = HD / 16;              // threads per (row, head)
  constexpr int kUnits = kThreads / kLanes;    // (row, head) at once
  // A thread's pieces: without rotation the same row and head of k and of v, so that one
  // place serves both, else any.
  constexpr uint32_t kStep = ROPE ? kUnits : 0, kTurn = ROPE ? kUnits * kPieces : kUnits;
  static_assert(ROPE || kPieces == 2, "of k and of v");
  __shared__ Spot spots[kMaxRows];
  __shared__ Found found;
  __shared__ float2 turn_s[ROPE ? kMaxRows : 1][64];  // cosine and sine
  const PagedMoveArgs& m = a.m;
  const int n0 = blockIdx.x * rows, lane = threadIdx.x % kLanes;
  const int half = a.rope.rotary_dim / 2;      // pairs
  const int n_q = ROPE ? a.n_q : 0;
  const uint32_t per_row = ROPE ? n_q + 2u * m.n_kv : m.n_kv;
  look_through<kThreads>(m.batch, n0, m.status, &found);
  const int mine = max(0, min(rows, found.end - n0));
  const uint32_t units = mine * per_row;

  auto piece = [&](uint32_t u, int i) {
    Piece p;
    p.row = (int)__umulhi(ROPE ? u : 2 * u, magic);  // u / per_row (launch_rope)
    p.slot = (int)(u - p.row * per_row) + (ROPE ? 0 : i * m.n_kv);
    const size_t n = n0 + p.row;
    p.turned = ROPE && p.slot < n_q + m.n_kv && lane * 8 < half;
    p.c0 = p.turned ? lane * 8 : lane * 16;
    p.c1 = p.turned ? half + lane * 8 : lane * 16 + 8;
    if (p.slot < n_q) {
      p.x = a.q + (n * a.q_row + (size_t)p.slot * a.q_head) * 2;
    } else {
      const int side = ROPE ? p.slot >= n_q + m.n_kv : i, head = p.slot - n_q - side * m.n_kv;
      p.x = m.x[side] + (n * m.row_stride[side] + (size_t)head * m.head_stride[side]) * 2;
    }
    return p;
  };
  uint4 w[kPieces][2] = {};
  auto load_row = [&](uint32_t u0, int i) {
    const uint32_t u = u0 + i * kStep;
    if (u < units) {
      const Piece p = piece(u, i);
      w[i][0] = *reinterpret_cast<const uint4*>(p.x + p.c0 * 2);
      w[i][1] = *reinterpret_cast<const uint4*>(p.x + p.c1 * 2);
    }
  };
  // the first rows are on their way while places and angles are made
#pragma unroll
  for (int i = 0; i < kPieces; ++i) load_row(threadIdx.x / kLanes, i);
  if ((int)threadIdx.x < mine) {
    const Place pl = find_row(m.batch, found, n0 + threadIdx.x, m.status);
    Spot spot;
#pragma unroll
    for (int side = 0; side < 2; ++side)
      spot.page[side] = pl.there ? m.pages[side] + (size_t)pl.page * m.page_stride[side] * (E4M3 || E2M1 ? 1 : 2) : nullptr;
    spot.id = (int)pl.page;
    spot.at = pl.at;
    spot.pos = pl.owned ? pl.pos : -1;
    spots[threadIdx.x] = spot;
  }
  __syncthreads();
  if (ROPE) {
    for (int i = threadIdx.x; i < mine * half; i += kThreads) {
      const int row = i / half, j = i - row * half;
      const long long pos = a.positions ? (long long)__ldg(a.positions + n0 + row) : spots[row].pos;
      turn_s[row][j] = cos_sin((unsigned long long)pos * a.rope.turns[j], a.rope.factor);
    }
    __syncthreads();
  }

  // whole warps stay together: pieces past the last take part in the shuffles
  const uint32_t turns = (units + kTurn - 1) / kTurn;
  for (uint32_t turn = 0; turn < turns; ++turn) {
    const uint32_t u0 = turn * kTurn + threadIdx.x / kLanes;
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const uint32_t u = u0 + i * kStep;
      const Piece p = piece(min(u, units - 1), i);
      const uint32_t v[8] = {w[i][0].x, w[i][0].y, w[i][0].z, w[i][0].w, w[i][1].x, w[i][1].y, w[i][1].z, w[i][1].w};
      float2 f[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = unpack16<BF16>(v[e]);
      // the next turn's rows, as early as their registers are free (rotated prompts 125 us for
      // 130, into E4M3 151 for 170; without rotation, where more is live here, 57 for 50)
      if (ROPE) load_row(u0 + kTurn, i);
      if (p.turned) {
        const float2* t = turn_s[p.row];
        if (a.rope.layout == DFLASH_ROPE_HALF) {
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float4 cs = *reinterpret_cast<const float4*>(t + p.c0 + 2 * e);
            turn2(f[e], f[4 + e], make_float2(cs.x, cs.z), make_float2(cs.y, cs.w));
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; e += 2) {
            const float4 cs = *reinterpret_cast<const float4*>(t + (e < 4 ? p.c0 : p.c1) / 2 + (e & 3));
            float2 x = make_float2(f[e].x, f[e + 1].x), y = make_float2(f[e].y, f[e + 1].y);
            turn2(x, y, make_float2(cs.x, cs.z), make_float2(cs.y, cs.w));
            f[e] = make_float2(x.x, y.x);
            f[e + 1] = make_float2(x.y, y.y);
          }
        }
      }
      uint32_t o[8];
      if (p.slot < n_q || (!E4M3 && !E2M1)) {
#pragma unroll
        for (int e = 0; e < 8; ++e) o[e] = pack16<BF16>(f[e].x, f[e].y);
      }
      // magnitudes order like their bits, NaN above infinity
      uint32_t m0 = 0, m1 = 0;
      if (!ROPE) {  // as they came, two at a time
#pragma unroll
        for (int e = 0; e < 8; ++e) m0 = max_abs<BF16>(m0, v[e]);
        const float2 top = unpack16<BF16>(m0 & 0x7FFF7FFFu);
        m0 = m1 = max(__float_as_uint(top.x), __float_as_uint(top.y));
      } else if ((E4M3 || E2M1) && __any_sync(0xffffffffu, p.slot >= n_q)) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          m0 = max(m0, max(__float_as_uint(f[e].x) & 0x7FFFFFFFu, __float_as_uint(f[e].y) & 0x7FFFFFFFu));
          m1 = max(m1, max(__float_as_uint(f[4 + e].x) & 0x7FFFFFFFu, __float_as_uint(f[4 + e].y) & 0x7FFFFFFFu));
        }
        const uint32_t both = max(m0, m1);
        if (E4M3) {
          m0 = both;
#pragma unroll
          for (int s = kLanes / 2; s > 0; s >>= 1) m0 = max(m0, __shfl_xor_sync(0xffffffffu, m0, s));
        } else {
          const uint32_t o0 = __shfl_xor_sync(0xffffffffu, m0, 1), o1 = __shfl_xor_sync(0xffffffffu, m1, 1);
          m0 = p.turned ? max(m0, o0) : both;
          m1 = p.turned ? max(m1, o1) : both;
        }
      }
      if (u >= units) continue;
      if (p.slot < n_q) {
        if (spots[p.row].pos < 0) continue;
        uint8_t* q = a.q_out + ((size_t)(n0 + p.row) * a.o_row + (size_t)p.slot * a.o_head) * 2;
        *reinterpret_cast<uint4*>(q + p.c0 * 2) = make_uint4(o[0], o[1], o[2], o[3]);
        *reinterpret_cast<uint4*>(q + p.c1 * 2) = make_uint4(o[4], o[5], o[6], o[7]);
        continue;
      }
      const int side = ROPE ? p.slot >= n_q + m.n_kv : i, head = p.slot - n_q - side * m.n_kv;
      uint8_t* const page = spots[p.row].page[side];
      if (!page) continue;
      const uint32_t row = ((uint32_t)head << m.batch.page_shift) + spots[p.row].at;  // below 2^19
      if (E2M1) {
        uint8_t* rec = page + row * e2m1_record(HD);
        auto scale = [](uint32_t top) {
          // top / 6 as quotients() makes it
          const float x = __uint_as_float(top), y = 1.0f / 6.0f, q = x * y;
          const float by6 = x < 0x1p-100f ? __fdiv_rn(x, 6.0f) : fmaf(fmaf(q, -6.0f, x), y, q);
          const float s = __bfloat162float(__float2bfloat16_rn(by6));
          return top >= 0x7F800000u ? __uint_as_float(0x7FC00000u) : s == 0.0f ? 1.0f : s;
        };
        auto codes = [&](float2* x, float s) {
          if (ROPE) raise(x, s);
          const float y = __frcp_rn(s), y_rest = fmaf(-s, y, 1.0f) * y;
          uint32_t c = 0;
          if (!ROPE && (quotients_small(s) || s > 0x1p100f)) {  // (there y_rest has few bits)
#pragma unroll 1
            for (int e = 0; e < 4; ++e) {
              const float2 q = quotients_slow(e == 0 ? x[0] : e == 1 ? x[1] : e == 2 ? x[2] : x[3], s);
              c |= e2m1x2(make_float2(q.x + 0.0f, q.y + 0.0f)) << (8 * e);  // -0 becomes 0, as below
            }
            return c;
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            // 16-bit values lie on a border between codes or 2^-14 of themselves from it, and
            // x times the reciprocal to 48 bits is the border where x / s is (-0 becomes 0)
            const float2 q = ROPE ? quotients(x[e], s, y)
                                  : fma2(x[e], make_float2(y, y), fma2(x[e], make_float2(y_rest, y_rest), make_float2(0.0f, 0.0f)));
            c |= e2m1x2(q) << (8 * e);
          }
          return c;
        };
        const float s0 = scale(m0), s1 = ROPE ? scale(m1) : s0;
        const uint32_t c0 = codes(f, s0), c1 = codes(f + 4, s1);
        if (ROPE) {
          *reinterpret_cast<uint32_t*>(rec + p.c0 / 2) = c0;
          *reinterpret_cast<uint32_t*>(rec + p.c1 / 2) = c1;
        } else {
          *reinterpret_cast<uint2*>(rec + p.c0 / 2) = make_uint2(c0, c1);
        }
        // a block's scale by the lane with its first run
        uint16_t* scales = reinterpret_cast<uint16_t*>(rec + HD / 2);
        if (p.c0 % 16 == 0) scales[p.c0 / 16] = (uint16_t)(__float_as_uint(s0) >> 16);
        if (p.c1 % 16 == 0) scales[p.c1 / 16] = (uint16_t)(__float_as_uint(s1) >> 16);
      } else if (E4M3) {
        const bool finite = m0 < 0x7F800000u;
        const float by448 = __fdiv_rn(__uint_as_float(m0), 448.0f);  // 0 of rotated values below 2^-141, too
        const float s = !finite ? __uint_as_float(0x7FC00000u) : by448 == 0.0f ? 1.0f : by448;
        float up = s;  // of the lower values; the upper ones' is the same
        raise(f + 4, up);
        raise(f, up = s);
        const float y = __fdiv_rn(1.0f, up);
        uint32_t c[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) c[e] = __nv_cvt_float2_to_fp8x2(quotients(f[e], up, y), __NV_SATFINITE, __NV_E4M3);
        *reinterpret_cast<uint2*>(page + row * HD + p.c0) = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
        *reinterpret_cast<uint2*>(page + row * HD + p.c1) = make_uint2(c[4] | (c[5] << 16), c[6] | (c[7] << 16));
        if (lane == 0) m.scale[side][(((size_t)spots[p.row].id * m.n_kv) << m.batch.page_shift) + row] = s;
      } else {
        *reinterpret_cast<uint4*>(page + (row * HD + p.c0) * 2) = make_uint4(o[0], o[1], o[2], o[3]);
        *reinterpret_cast<uint4*>(page + (row * HD + p.c1) * 2) = make_uint4(o[4], o[5], o[6], o[7]);
      }
    }
    if (!ROPE) {
#pragma unroll
      for (int i = 0; i < kPieces; ++i) load_row(u0 + kTurn, i);
    }
  }
}

template <int HD, int FORMAT, bool BF16, bool ROPE>
int launch_rope(const PagedRopeArgs& a, cudaStream_t s) {
  const long long each = ceil_div(a.m.batch.rows, 608);  // 4 blocks for each of 152 SMs come first
  const int per_row = a.n_q + 2 * a.m.n_kv;
  const int most = min(kMaxRows, max(1, kMostUnits / per_row));
  // ... and what is more comes in equal shares (prompts into 4 bits 50 us, 52 with blocks of `most`)
  const long long waves = max(1ll, (each + most - 1) / most);
  const int rows = (int)max(1ll, (each + waves - 1) / waves);
  const int grid = max(1, ceil_div(a.m.batch.rows, rows));
  // u / per_row = u * magic / 2^32 for u < rows * per_row (without rotation twice a pair's
  // number): 0 for a single row, else u and
  // per_row are at most kMostUnits
  const uint32_t magic = rows == 1 ? 0u : (uint32_t)(((1ull << 32) + per_row - 1) / per_row);
  return launch_pdl(paged_rope_kernel<HD, FORMAT, BF16, ROPE>, dim3(grid), dim3(kThreads), 0, s, a, rows, magic);
}

template <int HD, bool BF16>
int dispatch(const PagedRopeArgs& a, int format, cudaStream_t s) {
  if (!a.rope.rotary_dim) return launch_rope<HD, DFLASH_CACHE_E2M1, BF16, false>(a, s);
  if (format == DFLASH_CACHE_E2M1) return launch_rope<HD, DFLASH_CACHE_E2M1, BF16, true>(a, s);
  if (format == DFLASH_CACHE_E4M3) return launch_rope<HD, DFLASH_CACHE_E4M3, BF16, true>(a, s);
  return launch_rope<HD, BF16 ? DFLASH_CACHE_BF16 : DFLASH_CACHE_F16, BF16, true>(a, s);
}

}  // namespace

int launch_paged_append_rope(const PagedRopeArgs& a, int head_dim, int format, int type, cudaStream_t s) {
  const bool bf = type == DFLASH_TYPE_BF16;
  if (head_dim == 128) return bf ? dispatch<128, true>(a, format, s) : dispatch<128, false>(a, format, s);
  return bf ? dispatch<64, true>(a, format, s) : dispatch<64, false>(a, format, s);
}

}  // namespace dfl

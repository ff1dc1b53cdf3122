// Attention of new rows over a paged cache held in 4 bits (dflash_paged_attention
// with DFLASH_CACHE_E2M1; the rules are in include/dflash.h), on the 5th-generation
// tensor cores.
//
//   z_s = scale q . k_s over the visible s;  out = sum 2^(z' - m) v_s / l,
//   m a running reference of z' = z log2(e), l = sum 2^(z' - m), one pass.
//
// Everything is transposed: keys lie on the lanes of tensor memory and query rows
// on its columns,
//   S^T [128 keys, N rows] = K Q^T,   O^T [128 values, N rows] += V^T P^T,
// N the item's rows up to a multiple of 16 (above 64: 96 or 128).  So a block of 8
// positions or a single token costs the softmax what its rows are, not 128, and all
// its threads have keys; and the widened K goes from the codes straight to tensor
// memory as an operand, a row to a lane, without a trip through shared memory, which
// is the busiest part here.  Calls with more than 128 packed rows to a request go to
// paged_attention_e2m1_rows.cu (launch_paged_attention_e2m1 below).
//
// Values.  A code times its scale has 10 significant bits.  A row's scales are
// brought to [2^12, 2^13) by a power of two of the row's largest, so that the
// products are fp16 values, exact but for 2^-34 of the largest scale; the power comes
// back in float32, for K as a factor of the scores, for V added to the exponent of
// the weights.  Queries become fp16 times a power of two per row.
//   What a row's reference follows is the largest of weight times the power of its
// value row, so that the tail behind a dominant key with small values keeps its
// places: weights are fp16 up to 2^15, 2^4 at least for the largest when a reference
// is set, and end at 2^-24, so their last place is 2^-28 of the largest.  (References
// at 2^11 / 2^8 / 2^4 / 2^0: blocks of 8 155 / 150 / 145 / 141 us, ragged blocks 158 /
// 152 / 145 / 139; the lower, the rarer they grow, and the more of a long tail is
// rounded away: 2^-28 of 131,072 keys is 2^-11 of the largest, 2^-24 would be 2^-7.)
//
// Roles (640 threads, a persistent CTA on its part of the line, see paged_line.cuh;
// items of at most 128 rows):
//   warps 0, 3   page table and bulk copies of K and of V: a page's records are one
//                run of bytes
//   warp 1       issues the products, whatever is ready
//   warp 2       describes the CTA's segments of items, ahead of the others
//   warps 4-11   softmax: a thread has two columns of every group of 8, of four keys
//   warps 12-15  widen the codes of K into tensor memory, a key per thread
//   warps 16-19  widen those of V into shared memory (M-major operand)
// Modes.  An item of more than 64 rows: the warpgroups share each tile's columns, S
// has two buffers of 128 columns.  A smaller one: they take every other tile, all
// its columns, each with an O of its own, joined at the end, and S has four buffers
// of 64 columns, so that a warpgroup's next scores are made while it weighs.
// Tensor memory: S, 256 columns; O, 128; K0 | K1, head_dim / 2 each.
//
// What bounds it, measured on GB300 (8 KV heads of 128, groups of 5, bf16):
//   32 requests, blocks of 8, context 8,192: 143 us for 341 MB, 2.4 TB/s, 0.36 of the
//     measured copy (with L2 flushed 149; a bf16 cache 193, E4M3 182).  The products'
//     operands: in a timeline of a CTA the issuer is never without a product to issue, and a
//     tile's take 1,850 clocks, 750 for the scores and 1,100 for the values.  Alone a
//     product (16 deep, of up to 64 columns) takes 49 clocks where K comes from tensor
//     memory and 72 where V comes from shared memory, 970 a tile; beside them the widening
//     and the weights keep shared memory busy, 0.6 of its cycles in all.  Tensor cores
//     16 % of their rate, issue slots 52 %;
//   16 blocks of 16, context 512 to 131,072: 140 us (flushed 147, bf16 150, E4M3 158).
//     74 key tiles an SM take some 3,400 clocks each, where the products alone take
//     1,528: above 64 rows both warpgroups share a tile and S has two buffers, so that
//     tiles go through the chain scores, weights, values nearly one after another, and
//     80 rows take 96 columns;
//   without references that grow these two took 131 and 127 where they took 138 and 137:
//     each time one does its stream is held up for about 2,000 clocks;
//   one token, context 1,000: latency, 12 us.
//
// All waits are bounded.  When one gives up, the softmax warps run on to the end of
// their segment without waiting (their barriers stay matched, results are void,
// the status word says so) and the CTA ends as usual.
#include "paged_e2m1.cuh"

namespace dfl {
namespace {

using namespace line;

constexpr int kThreads = 640;
// Registers: of the softmax warpgroups, of the others, and what a thread is launched with
// (softmax 144 / 152 / 160: ragged blocks 145 / 143 / 147 us, blocks of 8 alike).
constexpr int kRegsSoftmax = 152, kRegsOthers = 56, kRegsLaunch = 96;
static_assert(256 * kRegsSoftmax + (kThreads - 256) * kRegsOthers <= kThreads * kRegsLaunch, "the block's registers");
constexpr int kRows = 128;     // of an item at most
constexpr int kMaxSlots = 8;
constexpr int kSegs = 4;       // descriptions ahead
constexpr int kAltRows = 64;   // items of so many rows at most: see Modes
constexpr uint32_t kColO = 256, kColK = 384;
constexpr int kScaleExp = 12;  // of a row's largest scale
constexpr float kUnscale = 0x1p-12f;
constexpr float kUnseen = 0x1p100f;  // minus the reference of a column that has seen no key
// Weights, log2: the largest there may be, and what a reference that grows makes of its
// tile's largest.
constexpr float kMaxWeight = 15.0f, kFreshWeight = 4.0f;
// A weight that makes its column's reference grow once some other column's has to: all
// that are about to do so at once (when prompt chunks ran here, 1,487 us for the 1,567
// with 15; blocks alike).
constexpr float kRenewWeight = 6.0f;
// Exponents (biased) that rows of K and V are scaled by: so that the factors stay
// normal numbers.  Of V 2^-64 at least: the sums l, in which that power is taken
// off the weights again, stay finite.
constexpr int kLeastK = 13, kLeastV = 127 - 64, kMost = 253;

struct KernelArgs : E2m1Args {
  int spans;  // of 64 rows (columns of P, rows of Q)
};

struct Seg : line::Seg {
  int more;
};

struct Ctrl {
  uint64_t full[kMaxSlots], empty[2][kMaxSlots];  // slots of a tile's K and V, given back one by one
  uint64_t k_full[2], k_empty[2], v_full[2];
  uint64_t s_full[4], p_full[2], pv_done[2];
  uint64_t q_full, o_full, fin;
  uint64_t seg_full[kSegs], seg_empty[kSegs];
  Start start;
  Walk<kRows> walk;
  Seg seg[kSegs];
  int abort_flag;
  uint32_t tmem;
  uint32_t bad[2][kMaxSlots];   // pages of the tile whose id is none
  uint32_t exponent[8][kKT];    // of the rows of K and (upper half) V, by tile: K may be six ahead of the softmax
  alignas(16) float4 col[2][kRows / 4];  // of two columns of a warpgroup: score factors, minus their references
  int2 range[kRows];            // positions that a column's row sees
  long long out_at[kRows];      // where its output row lies, or -1
  alignas(16) float red[2][4][kRows / 2];   // of a warpgroup: by warp and column
  alignas(16) float fac[2][kRows / 2];  // likewise, by column: what l and O shrink by,
  int high[2][kRows / 2];              // scores above what the references allow, as ordered(),
  uint32_t shrink[2][2];               // and which columns shrink
  float2 sum[2][kRows / 2];            // m and l of a warpgroup's columns
  float2 out_fac[2][kRows / 2];
  unsigned long long scan[33];
};
constexpr int kCtrlBytes = (int)((sizeof(Ctrl) + 1023) / 1024 * 1024);

template <int HD>
struct Cfg {
  static constexpr int kRec = e2m1_record(HD);
  static constexpr int kSlot = 2 * kKT * kRec;          // a tile's records of K, then of V
  static constexpr int kSpan = kKT * 128;               // bytes of 128 rows x 64 columns of fp16
  static constexpr int kWide = kSpan * (HD / 64);       // widened V of a tile
  // For head_dim 64 the upper 64 rows of V^T are a span of zeros.
  static constexpr int kWideAll = 2 * kWide + (HD == 64 ? kSpan : 0);
};

// ------------------------------------------------------------------ helpers

// Columns of an item of so many rows, and its mode.
__device__ __forceinline__ int columns(int rows) { return rows <= kAltRows ? (rows + 15) / 16 * 16 : rows <= 96 ? 96 : kRows; }
// Columns of a tile's scores.
__device__ __forceinline__ uint32_t s_col(bool alt, uint32_t tile) {
  return alt ? (tile & 3u) * kAltRows : (tile & 1u) * kRows;
}

// Eight columns, waited for.
__device__ __forceinline__ void tmem_ld_x8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
      : "r"(taddr)
      : "memory");
}
// *at = max(*at, v) by the threads where p holds, without a branch.
__device__ __forceinline__ void max_shared_if(bool p, int* at, int v) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %0, 0;\n\t@p red.shared.max.s32 [%1], %2;\n\t}" ::"r"((uint32_t)p),
               "r"(smem_u32(at)), "r"(v)
               : "memory");
}
// A float's bits as an integer of the same order, and back; what no score has.
__device__ __forceinline__ int ordered(int bits) { return bits ^ ((bits >> 31) & 0x7FFFFFFF); }
constexpr int kNone = (int)0x80000000;
__device__ __forceinline__ void st_shared(uint32_t at, uint32_t a) {
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(at), "r"(a) : "memory");
}
// A record: codes and scales as words.
template <int HD>
struct Record {
  uint32_t code[HD / 8];
  uint32_t scale[HD / 32];  // two each
};
template <int HD>
__device__ __forceinline__ void read_record(Record<HD>& r, const uint8_t* p, bool there) {
  if (HD == 128) {
#pragma unroll
    for (int i = 0; i < 5; ++i) {
      const uint4 w = there ? *reinterpret_cast<const uint4*>(p + 16 * i) : make_uint4(0u, 0u, 0u, 0u);
      uint32_t* d = i < 4 ? r.code + 4 * i : r.scale;
      d[0] = w.x;
      d[1] = w.y;
      d[2] = w.z;
      d[3] = w.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 5; ++i) {
      const uint2 w = there ? *reinterpret_cast<const uint2*>(p + 8 * i) : make_uint2(0u, 0u);
      uint32_t* d = i < 4 ? r.code + 2 * i : r.scale;
      d[0] = w.x;
      d[1] = w.y;
    }
  }
}
template <int HD>
__device__ __forceinline__ void read_scales(uint32_t (&scale)[HD / 32], const uint8_t* p) {
  if (HD == 128) {
    const uint4 w = *reinterpret_cast<const uint4*>(p + HD / 2);
    scale[0] = w.x;
    scale[1] = w.y;
    scale[HD / 64] = w.z;
    scale[HD / 32 - 1] = w.w;
  } else {
    const uint2 w = *reinterpret_cast<const uint2*>(p + HD / 2);
    scale[0] = w.x;
    scale[HD / 32 - 1] = w.y;
  }
}
// The biased exponent of a record's largest scale, within limits.
template <int HD>
__device__ __forceinline__ int largest_exponent(Record<HD>& r, const uint8_t* p, int least) {
  return min(max((int)(largest_scale<HD>(r.scale, p) >> 7), least), kMost);
}
// Scale i of the record, brought to the row's power of two, as a pair of fp16.
template <int HD>
__device__ __forceinline__ uint32_t scale_pair(const Record<HD>& r, int i, float f) {
  const uint32_t w = r.scale[i / 2];
  const uint32_t both = pack16<false>(__uint_as_float(w << 16) * f, __uint_as_float(w & 0xFFFF0000u) * f);
  return __byte_perm(both, 0u, i & 1 ? 0x3232 : 0x1010);
}

// ------------------------------------------------------------------ softmax

// Who a thread of the softmax is, and its warpgroup's columns of the segment.
struct Stream {
  int wg, w4, t, lane;
  bool alt;
  int col0;        // first column of the item
  uint32_t lanes;  // tensor memory at the warp's lanes
  int all_lo, all_hi;  // positions that every row of the item sees
};

// 16 lanes of two groups of 8 columns, as a matrix product's fragments: a thread has
// of either group (v[0 .. 3] and v[4 .. 7]) columns 2 (lane % 4) and the next of the
// rows lane / 4 (the first two) and 8 + lane / 4.
__device__ __forceinline__ void load_fragments(uint32_t taddr, float (&v)[2][4]) {
  asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=f"(v[0][0]), "=f"(v[0][1]), "=f"(v[0][2]), "=f"(v[0][3]), "=f"(v[1][0]), "=f"(v[1][1]), "=f"(v[1][2]),
                 "=f"(v[1][3])
               : "r"(taddr));
}
__device__ __forceinline__ void wait_fragments(float (&v)[2][4]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+f"(v[0][0]), "+f"(v[0][1]), "+f"(v[0][2]), "+f"(v[0][3]), "+f"(v[1][0]), "+f"(v[1][1]), "+f"(v[1][2]),
                 "+f"(v[1][3]));
}

// Some column's weight would pass 2^15, or it sees its first key (its reference was
// kUnseen): its reference becomes the tile's largest, what l and O shrink by is in fac,
// and O shrinks.  top: of the thread's columns, their largest over its keys.  By all
// threads of a warpgroup.  Only those that hold such a weight tell it, by a maximum
// under a predicate: exchanging the columns' largest values between lanes takes 2,000
// clocks beside everything else that wants shared memory, a branch for each column 800.
// (Without the second barrier, every warp working references and factors out from the
// maxima for itself: prompt chunk 1,714 us for 1,667.)
template <int NCH>
__device__ __forceinline__ void grow_references(const KernelArgs& k, Ctrl* c, const Stream& st, const float2 (&top)[NCH],
                                                const float2 (&nb)[NCH], uint32_t tO, uint32_t T, bool held) {
  const int wg = st.wg, t = st.t;
  int* const high = c->high[wg] + 2 * (st.lane & 3);
#pragma unroll
  for (int g = 0; g < NCH; ++g) {
    max_shared_if(top[g].x + nb[g].x > kRenewWeight, high + g * 8, ordered(__float_as_int(top[g].x)));
    max_shared_if(top[g].y + nb[g].y > kRenewWeight, high + g * 8 + 1, ordered(__float_as_int(top[g].y)));
  }
  named_sync(1 + wg, 128);
  if (st.w4 < 2) {
    bool shrinks = false;
    if (t < 8 * NCH) {
      const int m = c->high[wg][t];
      float* const at = reinterpret_cast<float*>(&c->col[wg][t >> 1]) + 2 + (t & 1);
      float fo = 1.0f;
      if (m != kNone) {
        c->high[wg][t] = kNone;
        const float old = *at, fresh = kFreshWeight - __int_as_float(ordered(m));
        *at = fresh;
        shrinks = old != kUnseen;
        if (shrinks) fo = ex2_approx(fresh - old);
      }
      c->fac[wg][t] = fo;
    }
    const uint32_t b = __ballot_sync(0xffffffffu, shrinks);
    if (st.lane == 0) c->shrink[wg][st.w4] = b;
  }
  named_sync(1 + wg, 128);
  if (!held) return;
  // O holds the tiles before: wait for the last one's product; the next waits for this
  // tile's weights
  const uint32_t b0 = c->shrink[wg][0], b1 = c->shrink[wg][1];
  if (!(b0 | b1)) return;
  const uint32_t last = T - (st.alt ? 2u : 1u);
  (void)warp_wait_on(&c->pv_done[last & 1u], (last >> 1) & 1u, &c->abort_flag, k.a.status);
  tc_fence_after();
  // (bit g: one of group g's eight columns does)
  auto groups = [](uint32_t b) {
    b |= b >> 4;
    b |= b >> 2;
    b |= b >> 1;
    return (b & 1u) | ((b >> 7) & 2u) | ((b >> 14) & 4u) | ((b >> 21) & 8u);
  };
#pragma unroll 1
  for (uint32_t todo = groups(b0) | (groups(b1) << 4); todo; todo &= todo - 1) {
    const int g = __ffs(todo) - 1;
    uint32_t o[8];
    tmem_ld_x8(tO + g * 8, o);
    const float4 f0 = *reinterpret_cast<const float4*>(&c->fac[wg][g * 8]), f1 = *reinterpret_cast<const float4*>(&c->fac[wg][g * 8 + 4]);
    const float f[8] = {f0.x, f0.y, f0.z, f0.w, f1.x, f1.y, f1.z, f1.w};
#pragma unroll
    for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f[e]);
    tmem_st(tO + g * 8, o);
  }
  tc_wait_st();
}

// The weights of a warpgroup's NCH groups of 8 columns over the tiles of a segment, and
// the sums of its l in red.  A thread has, of every group, two columns of four keys
// (load_fragments), so that the columns' factors and references stay in its registers:
// with a key to a thread and all columns, each of them read from shared memory for each
// tile, blocks of 8 took 246 us and 219 so.  Unrolled over the groups without a branch,
// so that their chains overlap (369 us with one for each group, 252 without).  Weights
// go out word by word: as fragments (stmatrix) prompt chunk 1,542 us for 1,513.
template <int HD, int NCH>
__device__ __forceinline__ void softmax_tiles(const KernelArgs& k, Ctrl* c, const Seg& s, const Stream& st, uint8_t* p_s,
                                              uint32_t& T) {
  const PagedAttnArgs& a = k.a;
  volatile int* stop = &c->abort_flag;
  const int wg = st.wg, row = st.w4 * 32 + (st.lane >> 2), pair = st.lane & 3;
  const bool alt = st.alt;
  const uint32_t tO = st.lanes + kColO + (alt ? wg * kAltRows : st.col0);
  float2 cs[NCH], nb[NCH], l[NCH];
#pragma unroll
  for (int g = 0; g < NCH; ++g) {
    const float4 cn = c->col[wg][g * 4 + pair];
    cs[g] = make_float2(cn.x, cn.y);
    nb[g] = make_float2(cn.z, cn.w);
    l[g] = make_float2(0.0f, 0.0f);
  }
  int done = 0;  // tiles of this stream
#pragma unroll 1
  for (int j = 0; j < s.nt; ++j, ++T) {
    const uint32_t i2 = T & 1u;
    if (alt && (int)i2 != wg) continue;
    const int key0 = (s.t0 + j) * kKT;
    const bool edge = key0 < st.all_lo || key0 + kKT > st.all_hi;
    const uint32_t tS = st.lanes + s_col(alt, T) + st.col0;
    (void)warp_wait_on(&c->s_full[T & 3u], (T >> 2) & 1u, stop, a.status);
    tc_fence_after();
    float z[2][NCH][4];  // [half of the warp's keys][group]
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int g = 0; g < NCH; g += 2) load_fragments(tS + ((uint32_t)(h * 16) << 16) + g * 8, reinterpret_cast<float(&)[2][4]>(z[h][g]));
    // of the thread's keys 16 h + 8 u: score factor; power of the value row, and its inverse
    float kf[4], vb[4], inv[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint32_t ex = c->exponent[T & 7u][row + 8 * u];
      kf[u] = __uint_as_float(((ex & 0xFFFFu) - kScaleExp) << 23);
      vb[u] = (float)((int)(ex >> 16) - 127);
      inv[u] = __uint_as_float((254 - (ex >> 16)) << 23);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int g = 0; g < NCH; g += 2) wait_fragments(reinterpret_cast<float(&)[2][4]>(z[h][g]));
    // ---- exponents of weight times the value row's power
#pragma unroll
    for (int g = 0; g < NCH; ++g)
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        float* const y = &z[u >> 1][g][(u & 1) * 2];
        const float2 x = fma2(make_float2(y[0], y[1]), mul2(make_float2(kf[u], kf[u]), cs[g]), make_float2(vb[u], vb[u]));
        y[0] = x.x;
        y[1] = x.y;
      }
    if (edge) {
#pragma unroll
      for (int g = 0; g < NCH; ++g)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int2 sees = c->range[st.col0 + g * 8 + pair * 2 + e];
#pragma unroll
          for (int u = 0; u < 4; ++u)
            if ((uint32_t)(key0 + row + 8 * u - sees.x) >= (uint32_t)(sees.y - sees.x)) z[u >> 1][g][(u & 1) * 2 + e] = -INFINITY;
        }
    }
    float2 top[NCH];
    float most = -INFINITY;
#pragma unroll
    for (int g = 0; g < NCH; ++g) {
      top[g].x = fmaxf(fmaxf(z[0][g][0], z[0][g][2]), fmaxf(z[1][g][0], z[1][g][2]));
      top[g].y = fmaxf(fmaxf(z[0][g][1], z[0][g][3]), fmaxf(z[1][g][1], z[1][g][3]));
      const float2 x = add2(top[g], nb[g]);
      most = fmaxf(most, fmaxf(x.x, x.y));
    }
    if (any_of(1 + wg, 128, most > kMaxWeight)) {
      grow_references<NCH>(k, c, st, top, nb, tO, T, done > 0);
#pragma unroll
      for (int g = 0; g < NCH; ++g) {
        const float4 cn = c->col[wg][g * 4 + pair];
        nb[g] = make_float2(cn.z, cn.w);
        l[g] = mul2(l[g], *reinterpret_cast<const float2*>(&c->fac[wg][g * 8 + 2 * pair]));
      }
    }
    // ---- weights; l without the value rows' powers.  (Where the warpgroups share a
    // tile its scores came after the last reader of this buffer.)
    if (alt && T >= 2) (void)warp_wait_on(&c->pv_done[i2], ((T - 2) >> 1) & 1u, stop, a.status);
    ++done;
    const uint32_t p_at = smem_u32(p_s) + i2 * k.spans * Cfg<HD>::kSpan + row * 128 + pair * 4;
#pragma unroll
    for (int g = 0; g < NCH; ++g) {
      const int ch = st.col0 / 8 + g;
      const uint32_t to = p_at + (ch >> 3) * Cfg<HD>::kSpan + (((ch ^ row) & 7) << 4);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float* const y = &z[u >> 1][g][(u & 1) * 2];
        const float2 x = add2(make_float2(y[0], y[1]), nb[g]);
        const float2 p = make_float2(ex2_approx(x.x), ex2_approx(x.y));
        l[g] = fma2(p, make_float2(inv[u], inv[u]), l[g]);
        st_shared(to + u * 1024, pack16<false>(p.x, p.y));
      }
    }
    fence_proxy_async_smem();
    tc_fence_before();
    __syncwarp();
    if (st.lane == 0) {
      mbar_arrive(&c->p_full[i2]);
      if (alt) mbar_arrive(&c->p_full[i2]);
    }
  }
#pragma unroll
  for (int g = 0; g < NCH; ++g) {
#pragma unroll
    for (int o = 4; o <= 16; o <<= 1) {
      l[g].x += __shfl_xor_sync(0xffffffffu, l[g].x, o);
      l[g].y += __shfl_xor_sync(0xffffffffu, l[g].y, o);
    }
    if (st.lane < 4) *reinterpret_cast<float2*>(&c->red[wg][st.w4][g * 8 + 2 * st.lane]) = l[g];
  }
}

// ------------------------------------------------------------------ kernel

template <int HD>
__global__ void __launch_bounds__(kThreads, 1) paged_attention_e2m1_kernel(const __grid_constant__ KernelArgs k) {
  using C = Cfg<HD>;
  grid_dependents_launch();
  extern __shared__ __align__(1024) uint8_t smem[];
  const PagedAttnArgs& a = k.a;
  uint8_t* const wide_s = smem;                                    // widened V, two tiles
  uint8_t* const p_s = wide_s + C::kWideAll;                       // weights, two tiles
  uint8_t* const q_s = p_s + 2 * k.spans * C::kSpan;               // queries
  const int q_span = k.spans * 64 * 128;                           // bytes of 64 of their columns
  uint8_t* const ring_s = q_s + q_span * (HD / 64);
  auto* c = reinterpret_cast<Ctrl*>(smem + kSmem - kCtrlBytes);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = blockIdx.x;
  if (smem_u32(smem) & 1023) {  // the swizzled tiles want 1024-byte atoms
    grid_dependency_wait();
    if (tid == 0) {
      report_status(a.status, DFLASH_ERR_UNSUPPORTED);
      k.rec[cta].pair = -1;
    }
    return;
  }

  // ---- what waits for nobody: barriers and tensor memory
  if (tid == 0) {
    for (int s = 0; s < k.slots; ++s) {
      mbar_init(&c->full[s], 2);
      mbar_init(&c->empty[0][s], 4);
      mbar_init(&c->empty[1][s], 8);  // (of V's scales, too)
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&c->k_full[i], 4);
      mbar_init(&c->k_empty[i], 1);
      mbar_init(&c->v_full[i], 4);
      mbar_init(&c->p_full[i], 8);
      mbar_init(&c->pv_done[i], 1);
    }
    for (int i = 0; i < 4; ++i) mbar_init(&c->s_full[i], 2);
    for (int i = 0; i < kSegs; ++i) {
      mbar_init(&c->seg_full[i], 1);
      mbar_init(&c->seg_empty[i], 19);  // 2 producers, issuer, 8 widening and 8 softmax warps
    }
    mbar_init(&c->q_full, 1);
    mbar_init(&c->o_full, 1);
    mbar_init(&c->fin, 1);
    c->abort_flag = 0;
    for (int i = 0; i < kRows; ++i) c->high[i / (kRows / 2)][i % (kRows / 2)] = kNone;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(&c->tmem, 512);
    tmem_relinquish();
  }
  if (HD == 64)
    for (int i = tid; i < C::kSpan / 16; i += kThreads)
      reinterpret_cast<uint4*>(wide_s + 2 * C::kWide)[i] = make_uint4(0u, 0u, 0u, 0u);
  grid_dependency_wait();

  const Part part = find_part<kRows, kThreads>(k, c->scan, &c->start);
  if (cta >= part.ctas) {
    if (tid == 0) k.rec[cta].pair = -1;
    if (warp == 1) tmem_dealloc(c->tmem, 512);  // the scan's barriers came after its allocation
    return;
  }
  fence_proxy_async_smem();  // the zeros
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = c->tmem;
  volatile int* stop = &c->abort_flag;

  if (warp < 4) {
    reg_dec<kRegsOthers>();
    if (warp == 0 || warp == 3) {
      // ------------------------------------------------ producers of K (0) and V (3)
      const int side = warp ? 1 : 0;
      const bool lead = elect_one();
      uint64_t* const empty = c->empty[side];
      const uint8_t* const pages = side ? k.v_pages : k.k_pages;
      const long long stride = side ? k.v_stride : k.k_stride;
      const int shift = a.batch.page_shift, per_tile = kKT >> shift;
      const uint32_t run = (uint32_t)C::kRec << shift;  // bytes of a page's rows of a head
      uint32_t used = 0, parity = 0;  // per slot: in use, phase of its last load
      int slot = 0;
      uint32_t ph = 0;
      bool ok = true;
      for (uint32_t seg = 0; ok; ++seg) {
        const int sg = seg % kSegs;
        ok = warp_wait_on(&c->seg_full[sg], (seg / kSegs) & 1u, stop, a.status);
        if (!ok || !c->seg[sg].more) break;
        const Seg s = c->seg[sg];
        __syncwarp();
        if (lead) mbar_arrive(&c->seg_empty[sg]);
        const int32_t* table = a.batch.table + s.it.b * a.batch.table_stride;
        const int g_lo = s.it.lo >> shift, g_hi = (s.it.hi - 1) >> shift;  // pages in sight
        // ids of 32 pages, one per lane, and of the next 32
        auto look_up = [&](int from) {
          const int g = from + lane;
          return g >= g_lo && g <= g_hi ? __ldg(table + g) : 0;
        };
        int ids_at = s.t0 * per_tile, ids = 0, ids_next = 0;
        if (s.nt > 0) {
          ids = look_up(ids_at);
          ids_next = look_up(ids_at + 32);
        }
        for (int t = s.t0; ok && t < s.t0 + s.nt; ++t) {
          const int first = t * per_tile;
          if (first + per_tile > ids_at + 32) {
            ids_at += 32;
            ids = ids_next;
            ids_next = look_up(ids_at + 32);
          }
          ok = warp_wait_on(&empty[slot], ph ^ 1u, stop, a.status);
          if (!ok) break;
          const int g = first + lane;
          const int id = __shfl_sync(0xffffffffu, ids, (g - ids_at) & 31);
          const bool in = lane < per_tile && g >= g_lo && g <= g_hi;
          const bool good = in && id >= 0 && id < a.batch.n_pages;
          const uint32_t bad = __ballot_sync(0xffffffffu, in && !good);
          const uint32_t n = __popc(__ballot_sync(0xffffffffu, good));
          if (lead) {
            if (bad) report_status(a.status, DFLASH_ERR_ARG);
            c->bad[side][slot] = bad;
            mbar_arrive_expect_tx(&c->full[slot], n * run);
          }
          __syncwarp();
          if (good)
            bulk_load(ring_s + (slot * 2 + side) * (kKT * C::kRec) + lane * run,
                      pages + (size_t)id * stride + (size_t)s.head * run, run, &c->full[slot]);
          __syncwarp();
          used |= 1u << slot;
          parity = (parity & ~(1u << slot)) | (ph << slot);
          if (++slot == k.slots) {
            slot = 0;
            ph ^= 1u;
          }
        }
      }
      if (!ok && lead) {
        // a wait gave up: let the copies in flight land before the CTA leaves
        int dummy = 0;
        for (int j = 0; j < k.slots; ++j)
          if ((used >> j) & 1u) (void)mbar_wait_bounded(&c->full[j], (parity >> j) & 1u, &dummy, nullptr, 100000000ull);
      }
      __syncwarp();
    } else if (warp == 1) {
      // ------------------------------------------------ issuer
      const bool lead = elect_one();
      constexpr uint32_t kHi = (uint32_t)((8 * 128) >> 4) | (1u << 14) | (2u << 29);  // 128-byte swizzle
      const uint32_t q_d = (smem_u32(q_s) >> 4) + (1u << 16);
      uint32_t T = 0;  // tiles so far
      bool ok = true;
      for (uint32_t seg = 0; ok; ++seg) {
        const int sg = seg % kSegs;
        ok = warp_wait_on(&c->seg_full[sg], (seg / kSegs) & 1u, stop, a.status);
        if (!ok || !c->seg[sg].more) break;
        const int nt = c->seg[sg].nt;
        const uint32_t n = columns(c->seg[sg].it.rows);
        const bool alt = n <= kAltRows;
        __syncwarp();
        if (lead) mbar_arrive(&c->seg_empty[sg]);
        const uint32_t id_qk = idesc_f32acc(kKT, 0, false) | ((n >> 3) << 17);
        const uint32_t id_pv = id_qk | (1u << 15) | (1u << 16);  // both operands M- and N-major
        ok = warp_wait_on(&c->q_full, seg & 1u, stop, a.status);
        tc_fence_after();
        auto scores = [&](uint32_t u) {
          const uint32_t i = u & 1u;
          tc_fence_after();
          if (lead) {
#pragma unroll
            for (int kk = 0; kk < HD / 16; ++kk)
              tc_mma_f16_ta(tmem + s_col(alt, u), tmem + kColK + i * (HD / 2) + kk * 8,
                            desc64(q_d + (kk >> 2) * (q_span >> 4) + (kk & 3) * 2, kHi), id_qk, kk > 0);
            tc_commit(&c->s_full[u & 3u]);
            mbar_arrive(&c->s_full[u & 3u]);  // hands on what was written before k_full: the exponents
            tc_commit(&c->k_empty[i]);
          }
          __syncwarp();
        };
        auto values = [&](uint32_t u, bool keep) {
          const uint32_t i = u & 1u;
          tc_fence_after();
          if (lead) {
            const uint32_t v_at = smem_u32(wide_s + i * C::kWide) >> 4, p_at = smem_u32(p_s + i * k.spans * C::kSpan) >> 4;
            // next span along M: the row's upper 64 values, or the zeros
            const uint32_t v_d = v_at + ((uint32_t)((HD == 128 ? 1 : 2 - (int)i) * C::kSpan >> 4) << 16);
            const uint32_t p_d = p_at + ((uint32_t)(C::kSpan >> 4) << 16);
#pragma unroll
            for (int kk = 0; kk < kKT / 16; ++kk)
              tc_mma_f16(tmem + kColO + (alt ? i * kAltRows : 0u), desc64(v_d + kk * 128, kHi), desc64(p_d + kk * 128, kHi), id_pv,
                         kk > 0 ? 1u : (uint32_t)keep);
            tc_commit(&c->pv_done[i]);
          }
          __syncwarp();
        };
        // Whatever is ready goes next: in a fixed order either waits for what the other's
        // operands wait for (ragged blocks 156 us for 147, when that was tried).
        const int buffers = alt ? 4 : 2;  // of S
        int ns = 0, nv = 0;               // scores and values issued
        unsigned long long since = 0;
#pragma unroll 1
        for (uint32_t polls = 1; ok && nv < nt; ++polls) {
          const uint32_t us = T + ns, uv = T + nv;
          if (ns < nt && ns - nv < buffers && __all_sync(0xffffffffu, mbar_test(&c->k_full[us & 1u], (us >> 1) & 1u))) {
            scores(us);
            ++ns;
            polls = since = 0;
          } else if (nv < ns && __all_sync(0xffffffffu, mbar_test(&c->p_full[uv & 1u], (uv >> 1) & 1u)) &&
                     __all_sync(0xffffffffu, mbar_test(&c->v_full[uv & 1u], (uv >> 1) & 1u))) {
            values(uv, nv >= (alt ? 2 : 1));  // O holds tiles before this one
            ++nv;
            polls = since = 0;
          } else if ((polls & 63u) == 0) {
            const unsigned long long now = globaltimer_ns();
            if (!since) since = now;
            const bool late = now - since > kWaitLimitNs;
            if (__any_sync(0xffffffffu, *stop || late)) {
              ok = false;
              if (lead) {
                *stop = 1;
                report_status(a.status, DFLASH_ERR_DEVICE_TIMEOUT);
              }
            }
          }
        }
        T += nt;
        if (!ok) break;
        if (lead) tc_commit(&c->o_full);
        __syncwarp();
      }
      if (lead) tc_commit(&c->fin);  // every MMA this thread issued
      __syncwarp();
    } else if (warp == 2) {
      // ------------------------------------------------ the segments
      if (lane == 0) {
        c->walk.begin(c->start, part.w1 - part.w0);
        k.rec[cta].pair = -1;
        for (uint32_t seg = 0;; ++seg) {
          const int sg = seg % kSegs;
          if (!wait_on(&c->seg_empty[sg], ((seg / kSegs) & 1u) ^ 1u, stop, a.status)) break;
          Seg* n = &c->seg[sg];
          const bool more = c->walk.next(k, n);
          n->more = more;
          mbar_arrive(&c->seg_full[sg]);
          if (!more) break;
          if (n->first && !n->last)
            k.rec[cta] = Rec{n->pair, n->head, n->slot, part.owner(part.w0 + n->end - 1), n->it.s0, n->it.row0, n->it.rows};
        }
      }
      __syncwarp();
    }
  } else if (warp >= 12) {
    // ------------------------------------------------ widening of K and of V
    reg_dec<kRegsOthers>();
    const bool of_v = warp >= 16;
    const int r = tid & 127;
    const uint32_t t_k = tmem + kColK + ((uint32_t)((warp & 3) * 32) << 16);
    const int shift = a.batch.page_shift;
    int slot = 0;
    uint32_t ph = 0, T = 0;
    bool ok = true;
    for (uint32_t seg = 0; ok; ++seg) {
      const int sg = seg % kSegs;
      ok = warp_wait_on(&c->seg_full[sg], (seg / kSegs) & 1u, stop, a.status);
      if (!ok || !c->seg[sg].more) break;
      const int nt = c->seg[sg].nt, t0 = c->seg[sg].t0, lo = c->seg[sg].it.lo, hi = c->seg[sg].it.hi;
      __syncwarp();
      if (lane == 0) mbar_arrive(&c->seg_empty[sg]);
#pragma unroll 1
      for (int t = t0; t < t0 + nt; ++t, ++T) {
        const uint32_t i = T & 1u, before = ((T >> 1) & 1u) ^ 1u;
        ok = warp_wait_on(&c->full[slot], ph, stop, a.status);
        if (!ok) break;
        // rows that no row of the item sees, and those of no page, count as zeros
        const int key = t * kKT + r;
        const bool in = key >= lo && key < hi;
        const bool in_v = in && !((c->bad[1][slot] >> (r >> shift)) & 1u);
        const uint8_t* const from = ring_s + slot * C::kSlot + r * C::kRec;
        Record<HD> x;
        if (of_v) {
          read_record<HD>(x, from + kKT * C::kRec, in_v);
          const float f = __uint_as_float((uint32_t)(254 + kScaleExp - largest_exponent<HD>(x, from + kKT * C::kRec, kLeastV)) << 23);
          ok = warp_wait_on(&c->pv_done[i], before, stop, a.status);
          if (!ok) break;
          // (128-byte swizzle: chunk c of row r lies at c ^ r % 8)
          const uint32_t to = smem_u32(wide_s + i * C::kWide) + r * 128 + ((r & 7) << 4);
#pragma unroll
          for (int b = 0; b < HD / 16; ++b) {
            const uint32_t s = scale_pair<HD>(x, b, f);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              uint32_t w[4];
              e2m1x8_to_f16x2(x.code[2 * b + h], w);
              const int ch = 2 * b + h;
              st_shared_x4((to ^ ((ch & 7) << 4)) + (ch >> 3) * C::kSpan, hmul2(w[0], s), hmul2(w[1], s), hmul2(w[2], s),
                           hmul2(w[3], s));
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&c->v_full[i]);
            mbar_arrive(&c->empty[1][slot]);
          }
        } else {
          // V's exponents are wanted with the scores
          int ev = 0;
          if (in_v) {
            uint32_t scale[HD / 32];
            read_scales<HD>(scale, from + kKT * C::kRec);
            ev = (int)(largest_scale<HD>(scale, from + kKT * C::kRec) >> 7);
          }
          if (__any_sync(0xffffffffu, ev == 0)) {
            const int top = (int)__reduce_max_sync(0xffffffffu, (unsigned)ev);
            if (ev == 0) ev = top ? top - kZeroBelow : kZeroV;
          }
          ev = min(max(ev, kLeastV), kMost);
          read_record<HD>(x, from, in && !((c->bad[0][slot] >> (r >> shift)) & 1u));
          const int ek = largest_exponent<HD>(x, from, kLeastK);
          const float f = __uint_as_float((uint32_t)(254 + kScaleExp - ek) << 23);
          c->exponent[T & 7u][r] = (uint32_t)ek | ((uint32_t)ev << 16);
          ok = warp_wait_on(&c->k_empty[i], before, stop, a.status);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int b = 0; b < HD / 32; ++b) {  // two blocks of 16
            uint32_t w[16];
#pragma unroll
            for (int q = 0; q < 4; ++q) e2m1x8_to_f16x2(x.code[4 * b + q], reinterpret_cast<uint32_t(&)[4]>(w[4 * q]));
            const uint32_t s0 = scale_pair<HD>(x, 2 * b, f), s1 = scale_pair<HD>(x, 2 * b + 1, f);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              w[e] = hmul2(w[e], s0);
              w[8 + e] = hmul2(w[8 + e], s1);
            }
            tmem_st(t_k + i * (HD / 2) + b * 16, w);
          }
          tc_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&c->k_full[i]);
            mbar_arrive(&c->empty[0][slot]);
            mbar_arrive(&c->empty[1][slot]);
          }
        }
        if (++slot == k.slots) {
          slot = 0;
          ph ^= 1u;
        }
      }
    }
  } else {
    // ------------------------------------------------ softmax
    reg_inc<kRegsSoftmax>();
    const int wg = (warp >> 2) - 1, w4 = warp & 3, t = tid & 127, t2 = tid - 128;
    const uint32_t lanes = (uint32_t)(w4 * 32) << 16;
    uint32_t T = 0;
    for (uint32_t seg = 0;; ++seg) {
      const int sg = seg % kSegs;
      const bool have = warp_wait_on(&c->seg_full[sg], (seg / kSegs) & 1u, stop, a.status);
      // also: everybody is past the last segment
      if (any_of(3, 256, !have) || !c->seg[sg].more) break;
      const Seg& s = c->seg[sg];
      const Item& it = s.it;
      const int n = columns(it.rows);
      const bool alt = n <= kAltRows;
      const int mine = alt ? n : n / 2, nch = mine / 8, col0 = alt ? 0 : wg * mine;  // this warpgroup's columns

      // ---- queries: fp16 times a power of two per row; the columns' tables
      constexpr int kCh = HD / 8;
#pragma unroll 1
      for (int idx = t2; idx < n * kCh; idx += 256) {
        const int r = idx / kCh, ch = idx % kCh;
        uint4 w = make_uint4(0u, 0u, 0u, 0u);
        if (r < it.rows) {
          const int packed = it.row0 + r, tok = packed / a.group, g = packed - tok * a.group;
          w = __ldg(reinterpret_cast<const uint4*>(
              a.q + ((size_t)(it.s0 + tok) * a.q_row + (size_t)(s.head * a.group + g) * a.q_head + ch * 8) * 2));
        }
        int e;
        w = widen_q<kCh>(w, k.bf16, &e);
        *reinterpret_cast<uint4*>(q_s + (ch >> 3) * q_span + swz(r, (ch & 7) * 8)) = w;
        if (ch == 0) {
          // columns without a row: weights of zero
          const bool real = r < it.rows;
          for (int w = 0; w < 2; ++w) {
            const int own = alt ? r : r - w * mine;
            if (own < 0 || own >= mine) continue;
            float* cs = reinterpret_cast<float*>(&c->col[w][own >> 1]) + (own & 1);
            cs[0] = real ? q_factor(e, a.scale_log2) : 0.0f;
            cs[2] = real ? kUnseen : -1000.0f;
          }
          const int packed = it.row0 + (real ? r : 0), tok = packed / a.group, g = packed - tok * a.group;
          const int pos = it.len - it.n + tok, head = s.head * a.group + g;
          const int from = a.window ? max(0, pos - a.window + 1) : 0;
          c->range[r] = make_int2(from, max(from, a.causal ? min(it.len, pos + 1) : it.len));
          c->out_at[r] = real ? (long long)(it.s0 + tok) * a.o_row + (long long)head * a.o_head : -1;
        }
      }
      fence_proxy_async_smem();
      named_sync(3, 256);
      if (t2 == 0) mbar_arrive(&c->q_full);
      // positions that every row sees
      const int p0 = it.len - it.n + it.row0 / a.group, p1 = it.len - it.n + (it.row0 + it.rows - 1) / a.group;
      const int all_lo = a.window ? p1 - a.window + 1 : 0, all_hi = a.causal ? min(it.len, p0 + 1) : it.len;

      const uint32_t first_tile = T;
      const Stream st = {wg, w4, t, lane, alt, col0, tmem + lanes, all_lo, all_hi};
      if (nch == 8) softmax_tiles<HD, 8>(k, c, s, st, p_s, T);
      else if (nch == 6) softmax_tiles<HD, 6>(k, c, s, st, p_s, T);
      else if (nch == 4) softmax_tiles<HD, 4>(k, c, s, st, p_s, T);
      else softmax_tiles<HD, 2>(k, c, s, st, p_s, T);

      // ---- end of the segment: O is final
      (void)warp_wait_on(&c->o_full, seg & 1u, stop, a.status);
      tc_fence_after();
      const bool whole = s.first && s.last;
      const size_t part_at = (size_t)(cta * 2 + s.slot) * k.part_rows;
      named_sync(1 + wg, 128);
      if (t < mine) {
        const float L = (c->red[wg][0][t] + c->red[wg][1][t]) + (c->red[wg][2][t] + c->red[wg][3][t]);
        // (nothing seen: no reference)
        c->sum[wg][t] = make_float2(L == 0.0f ? -INFINITY : -(reinterpret_cast<const float*>(&c->col[wg][t >> 1])[2 + (t & 1)]), L);
      }
      if (alt)
        named_sync(3, 256);
      else
        named_sync(1 + wg, 128);
      const bool have0 = s.nt > (alt && (first_tile & 1u)), have1 = alt && s.nt > !(first_tile & 1u);  // tiles of the streams
      if (t < mine) {
        const int r = col0 + t;
        float M, L, f0 = 1.0f, f1 = 0.0f;
        if (alt) {
          const float2 x = c->sum[0][t], y = c->sum[1][t];
          M = fmaxf(x.x, y.x);
          f0 = x.x == -INFINITY ? 0.0f : ex2_approx(x.x - M);
          f1 = y.x == -INFINITY ? 0.0f : ex2_approx(y.x - M);
          L = x.y * f0 + y.y * f1;
        } else {
          M = c->sum[wg][t].x;
          L = c->sum[wg][t].y;
        }
        const float inv = (whole ? (L > 0.0f || L != L ? 1.0f / L : 0.0f) : 1.0f) * kUnscale;
        c->out_fac[wg][t] = make_float2(f0 * inv, f1 * inv);
        if (r < it.rows && (!alt || wg == 0)) {
          if (!whole) {
            k.ml[part_at + r] = make_float2(M, L);
          } else if (a.lse) {
            const int packed = it.row0 + r, tok = packed / a.group, g = packed - tok * a.group;
            a.lse[(size_t)(it.s0 + tok) * a.n_q + s.head * a.group + g] = (M + log2f(L)) * kLn2;
          }
        }
      }
      named_sync(1 + wg, 128);
      const int d = w4 * 32 + lane;
      // either warpgroup its columns, or every other group of 8
#pragma unroll 1
      for (int q = alt ? wg : 0; q < nch; q += alt ? 2 : 1) {
        const uint32_t tO = tmem + lanes + kColO + col0 + q * 8;
        uint32_t o[8] = {}, o1[8] = {};
        if (have0) tmem_ld_x8(tO, o);
        if (have1) tmem_ld_x8(tO + kAltRows, o1);
        if (d >= HD) continue;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int r = col0 + q * 8 + e;
          if (r >= it.rows) break;
          const float2 f = c->out_fac[wg][q * 8 + e];
          float x = __uint_as_float(o[e]) * f.x;
          if (have1) x = fmaf(__uint_as_float(o1[e]), f.y, x);
          if (whole) {
            const uint32_t h = k.bf16 ? pack16<true>(x, x) : pack16<false>(x, x);
            reinterpret_cast<uint16_t*>(a.out)[c->out_at[r] + d] = (uint16_t)h;
          } else {
            k.part[(part_at + r) * HD + d] = x;
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&c->seg_empty[sg]);
    }
  }

  // tensor memory is no longer read: free it once every MMA has completed
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    int dummy = 0;
    if (lane == 0) (void)mbar_wait_bounded(&c->fin, 0, &dummy, nullptr, 100000000ull);
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// -------------------------------------------------------------------- host

template <int HD>
int launch(KernelArgs& k, cudaStream_t s) {
  using C = Cfg<HD>;
  auto kern = paged_attention_e2m1_kernel<HD>;
  int dev = 0, sms = 0;
  DFL_CUDA_TRY(cudaGetDevice(&dev));
  static std::atomic<int> known[64];  // SMs of the devices the attribute is set on
  if (dev < 64 && (sms = known[dev].load())) {
  } else {
    DFL_CUDA_TRY(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
    DFL_CUDA_TRY(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem));
    cudaFuncAttributes attr;
    DFL_CUDA_TRY(cudaFuncGetAttributes(&attr, kern));
    if (attr.numRegs != kRegsLaunch) return DFLASH_ERR_UNSUPPORTED;  // the softmax's share would never come free
    if (dev < 64) known[dev].store(sms);
  }
  const int most = k.a.max_rows * k.a.group;  // at most kRows
  k.rts = 1;
  // What an item costs beside its tiles, for the cut of the line (queries, their factors,
  // the first references, the end): of 4 / 8 tiles ragged blocks take 170 / 145 us,
  // with 1 / 16, when that was tried, 223 / 149; blocks of 8 with 16 154 for 147.
  k.seg_cost = 8;
  k.spans = most > 64 ? 2 : 1;
  const int fixed = C::kWideAll + 2 * k.spans * C::kSpan + k.spans * 64 * 128 * (HD / 64) + kCtrlBytes;
  k.slots = min(kMaxSlots, (kSmem - fixed) / C::kSlot);
  const int grid = sms < kMaxCtas ? sms : kMaxCtas;
  int rc;
  if ((rc = launch_pdl(kern, dim3(grid), dim3(kThreads), kSmem, s, k))) return rc;
  const int y = min(kJoinBlocks, most);
  const LineArgs& line = k;
  return k.bf16 ? launch_pdl(paged_join_kernel<HD, true>, dim3(grid, y), dim3(256), 0, s, line)
                : launch_pdl(paged_join_kernel<HD, false>, dim3(grid, y), dim3(256), 0, s, line);
}

}  // namespace

int launch_paged_attention_e2m1(const dflash_paged_cache& c, const PagedAttnArgs& a, int type, void* ws,
                                cudaStream_t s) {
  KernelArgs k;
  k.a = a;
  const Layout l = layout(ws, a.group, c.head_dim, a.max_rows);
  k.part = l.part;
  k.ml = l.ml;
  k.rec = l.rec;
  k.part_rows = part_rows(a.group, a.max_rows);
  k.k_pages = static_cast<const uint8_t*>(c.k_pages);
  k.v_pages = static_cast<const uint8_t*>(c.v_pages);
  k.k_stride = c.k_page_stride;
  k.v_stride = c.v_page_stride;
  k.bf16 = type == DFLASH_TYPE_BF16;
  // By the bound max_rows, for what a request really has is on the device.  With 5 query
  // heads to a KV head over 8,192 keys: 16 requests of 25 rows (125 packed) take 141 us here
  // and 140 there, of 20 137 and 133; ragged blocks of 16 (80) 140 and 160, blocks of 8 (40)
  // 143 and 213, 32 single tokens 108 and 198.  So a max_rows above 128 packed rows costs a
  // call of few rows up to that much.  (A max_rows above 64 of them, 121 for the tokens: the
  // room for weights is taken from the slots.)  31 tokens beside a chunk of 2,048 rows
  // take 624 us in one call, 105 and 384 in two.
  if ((long long)a.max_rows * a.group > kRows) return launch_paged_attention_e2m1_rows(k, c.head_dim, s);
  return c.head_dim == 128 ? launch<128>(k, s) : launch<64>(k, s);
}

}  // namespace dfl

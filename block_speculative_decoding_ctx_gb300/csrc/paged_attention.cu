// Attention of new rows over a paged cache (dflash_paged_attention; the rules
// are in include/dflash.h), on the 5th-generation tensor cores.
//
//   z_s = scale q . k_s over the visible s;  out = sum 2^(z' - m) v_s / l,
//   m a running reference of z' = z log2(e), l = sum 2^(z' - m), one pass.
//
// Work.  The rows of one request that read one KV head, n_b x group of them
// (packed row = new row x group + query head of the group), are cut into items
// of at most 256; an item runs over the key tiles (128 positions) that any of
// its rows sees.  All key tiles of all items, in order, are one line that is
// cut into equal parts, one for each CTA (one CTA per SM): unequal lengths,
// causal triangles and single long requests all balance.  A CTA that holds a
// whole item writes its result; an item cut between CTAs leaves partial (O, m,
// l) in the workspace, which a second kernel joins in CTA order.  The cut
// depends on the lengths alone, so results are the same on every run.
//
// Inside a CTA two streams of jobs (Q tile of 128 rows x half a key tile, 64
// keys) run side by side, each with its own S and O in tensor memory and its
// own softmax warpgroup, so that one's softmax runs under the other's products,
// and a stream's scores of one half are made while the other half is weighed
// (prompt chunk: 992 us with whole tiles of 128 keys, 925 so, when that was tried):
//   an item of more than 128 rows: its two Q tiles, both over every key tile
//     (each K/V byte feeds 256 rows);
//   a smaller one: even and odd key tiles of its one Q tile, joined at the end.
// Roles (384 threads):
//   warps 0, 3  page table and TMA: K and V tiles into two rings of slots, for an
//               item of two Q tiles one of K and one of V tiles, for a smaller
//               one a ring per stream: whoever reads a ring waits for every
//               phase of its barriers in turn.  (One ring for both streams of a
//               smaller item would not do: loads may land out of order, and a
//               wait whose previous phase is still open returns at once.)
//   warps 1, 2  issue their stream's S = Q K^T (both from shared memory; a warp
//               for both streams made each wait for the other's: blocks of 8
//               203 us against 178, when that was tried) and
//               O += P V (P from tensor memory, V MN-major as TMA left it), and
//               (16-bit caches) zero the V rows that no row of the item sees (a
//               weight of 0 times whatever lies there must not become NaN)
//   warps 4-7   softmax of stream 0, one query row per thread; warps 8-11
//               stream 1.  P overwrites S in place.  O is rescaled only when a
//               row's reference grows by more than a headroom, a few times a
//               row.
// Tensor memory: S0 | S1 | O0 | O1, 128 columns each (S two halves of 64), all
// 512 of it; the shared memory of a CTA keeps any other off its SM.
//
// E4M3 caches.  The scores' products take the codes as they lie in the cache
// (kind::f8f6f4, twice the rate of 16 bits); Q, times a power of two per row
// that brings its largest value to [128, 256), is a sum of an E4M3 term of 4
// bits and E5M2 ones of 3 bits, 1 for bf16 and 2 for fp16, each rounded to
// nearest.  That is exact for values of at least 2^-6.  Of a smaller one the
// first term leaves up to 2^-10 and each further one an eighth of what it finds,
// down to 2^-17: all in all 2^-13 for bf16 and 2^-16 for fp16, 2^-20 and 2^-23 of
// the row's largest.  (E4M3 terms throughout leave 2^-17 of it.)  The key scale
// multiplies the score in float32.
//   The weights, times the value scales in float32, and V are fp16: the softmax
// warpgroup of a stream, its weights made, widens the codes of the half tile that
// they weigh into a buffer of its own, exactly (widen_v).  A first position that
// takes nine tenths of a row over 131,072 keys leaves the others 2^-20 of its
// weight, and they are the output if its values are small, as such positions'
// are.  So what a row's reference follows is weight times value scale: the
// largest score of four neighbouring keys and the largest of their value scales
// (a key's own: 201 us for the ragged blocks where four take 196), and the last
// place of a weight is 2^-35 of that.  (Weights as three E5M2 terms for
// kind::f8f6f4 end at 2^-24; outputs behind a dominant key came out a tenth too
// small and worse.  bf16 weights and values need no such care, but the weights'
// rounding is as large as the output's: errors of 2.3e-3 to 2.5e-3 where these
// have 1.6e-3.)
//   If a small item has no more than 64 rows, its two softmax warps without rows
// widen all of V, for the two with rows set the pace (32 x 8 rows with bf16
// weights: 182 us, where all four widen 219).
//
// All waits are bounded.  When one gives up, the softmax warps run on without
// waiting (their barriers stay matched, results are void, the status word says
// so) and the CTA ends as usual.
//
// What bounds it, measured on GB300 (8 KV heads of 128, groups of 5, bf16):
//   32 requests, blocks of 8, context 8,192: HBM.  171 us for 1.08 GB, 6.3 TB/s,
//     0.93 of the measured copy;
//   the same over an E4M3 cache: 177 us for 0.56 GB.  Softmax warps (scales and
//     their barriers, two products more per weight); prompt chunks 1,622 us, where
//     each stream widens V for itself, 1.8 times the bf16 cache's;
//   prompt chunk, 2 x 2,048 rows, context up to 16,384: the tensor cores under
//     the power limit, 911 us, 1.32 PFLOP/s at 1.75 GHz and 1,390 W, 0.77 of
//     what a library product sustains;
//   one token, context 1,000: latency.  12 us, of them 6 in this kernel (setting up
//     0.7, finding its part 1.2, queries to the last weights 2.6, the end 1.8), 2
//     to 4 in the join.
//   Where most items are cut the join is a share: 15 of 113 us for prompt chunks
//     of 200 to 700 rows, 8 of 24 for short windowed ones.
#include <atomic>
#include <cstddef>
#include <mutex>

#include <cuda_fp8.h>
#include <cudaTypedefs.h>

#include "attention_util.cuh"
#include "paged_util.cuh"

namespace dfl {
namespace {

using namespace attn;

constexpr int kKT = 128;           // keys per tile: what TMA loads
constexpr int kHK = 64;            // keys per job: half a tile
constexpr int kMT = 128;           // rows of a Q tile
constexpr int kThreads = 384;
constexpr int kMaxCtas = 160;      // the workspace has room for so many
constexpr int kMaxSlots = 12;
constexpr int kJoinBlocks = 32;    // see paged_join_kernel
constexpr int kSmem = 227 * 1024;  // all that a CTA may have
constexpr uint32_t kColO = 256;    // O of stream 0; S of stream s at 128 s
constexpr float kLn2 = 0.693147180559945309f;

// Where an item that this CTA starts but does not finish continues.
struct Rec {
  int pair, head, slot, last_cta;  // pair < 0: none
  int s0, row0, rows;              // its rows (Item)
};

struct KernelArgs {
  PagedAttnArgs a;
  float* part;    // [CTA][2][part_rows][HD]
  float2* ml;     // [CTA][2][part_rows]
  Rec* rec;       // [CTA]
  int rts;        // items per request at most
  int part_rows;  // 128 or 256
  int half;       // slots of each of the two rings
  int seg_cost;   // what beginning an item costs, in key tiles (launch)
  int q_tiles;    // Q tiles in shared memory
};

// ------------------------------------------------------------------- items

struct Item {
  int b, s0, n, len;     // request
  int row0, rows;        // packed rows
  int lo, hi;            // positions that some row sees
  int t_lo, tiles;       // key tiles
  int units;             // length on the line: the tiles and seg_cost for the rest, 1 for an empty item
};

__device__ __forceinline__ bool item_rows(const PagedAttnArgs& a, int b, RequestSpan* r) {
  return request_span(a.batch, b, r) && r->n <= a.max_rows;
}

__device__ __forceinline__ Item make_item(const KernelArgs& k, const RequestSpan& r, int b, int rt) {
  const PagedAttnArgs& a = k.a;
  Item it;
  it.b = b;
  it.s0 = r.s0;
  it.n = r.n;
  it.len = r.len;
  it.row0 = rt * (2 * kMT);
  it.rows = min(2 * kMT, r.n * a.group - it.row0);
  const int p0 = r.len - r.n + it.row0 / a.group;
  const int p1 = r.len - r.n + (it.row0 + it.rows - 1) / a.group;
  it.hi = a.causal ? min(r.len, p1 + 1) : r.len;
  it.lo = a.window ? max(0, p0 - a.window + 1) : 0;
  it.t_lo = it.lo / kKT;
  it.tiles = it.hi > it.lo ? (it.hi + kKT - 1) / kKT - it.t_lo : 0;
  it.units = it.tiles ? it.tiles + k.seg_cost : 1;
  return it;
}

// First item at or after pair (request x rts + item) on the line; pair moves
// to it.  False past the last request.
__device__ __forceinline__ bool find_item(const KernelArgs& k, int* pair, int end, Item* it) {
  while (*pair < end) {
    const int b = *pair / k.rts, rt = *pair - b * k.rts;
    RequestSpan r;
    if (item_rows(k.a, b, &r) && rt * (2 * kMT) < r.n * k.a.group) {
      *it = make_item(k, r, b, rt);
      return true;
    }
    *pair = (b + 1) * k.rts;
  }
  return false;
}

// Where a reader stands in the two rings of slots: the first slot of the
// segment in either, and the phase it waits for there.
struct Rings {
  int at[2];
  uint32_t phase[2];

  static __device__ __forceinline__ void advance(int half, int& at, uint32_t& phase, int n) {
    at += n;
    if (at >= half) {
      at -= half;
      phase ^= 1u;
    }
  }
  // past a segment of nt tiles: of K in one ring and V in the other, or (split)
  // of both in the ring of the stream that has every other tile
  __device__ __forceinline__ void leave(int half, bool split, int nt) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int n = at[i] + (split ? 2 * ((nt + 1 - i) / 2) : nt);
      at[i] = n % half;
      phase[i] ^= (uint32_t)(n / half) & 1u;
    }
  }
};

// The CTA's part of the line as segments of items.
struct Seg {
  Item it;
  int head;        // KV head
  int t0, nt;      // key tiles
  bool split;      // one Q tile, streams take every other key tile
  bool first, last;
  int slot;        // partial slot
  int pair;
  int v_at;        // E4M3: the stream's first V slot in its ring, and its phase
  uint32_t v_phase;
  long long end;   // where the item ends on the line, from the CTA's first unit on
};

// Where a CTA's part of the line begins.
struct Start {
  Item it;
  int pair, head, off;  // off: units of (pair, head) before it
};

struct Walk {
  long long left, total;
  int pair, head, off;
  bool loaded;
  Item it;
  __device__ void begin(const Start& st, long long n) {
    left = total = n;
    it = st.it;
    pair = st.pair;
    head = st.head;
    off = st.off;
    loaded = true;
  }
  __device__ bool next(const KernelArgs& k, Seg* s) {
    while (left > 0) {
      if (!loaded) {
        if (!find_item(k, &pair, k.a.batch.B * k.rts, &it)) return false;
        loaded = true;
      }
      // the item's first seg_cost units stand for its beginning and end; the
      // CTA that holds its first tile does that work
      const int skip = it.tiles ? k.seg_cost : 0;
      const int take = (int)min(left, (long long)(it.units - off));
      const int a0 = max(off - skip, 0), a1 = max(off + take - skip, 0);
      const bool any = a1 > 0;
      s->it = it;
      s->head = head;
      s->t0 = it.t_lo + a0;
      s->nt = it.tiles ? a1 - a0 : 0;
      s->split = it.rows <= kMT;
      s->first = a0 == 0;
      s->last = off + take == it.units;
      s->slot = left == total ? 0 : 1;
      s->pair = pair;
      s->end = total - left - off + it.units;
      left -= take;
      off = 0;
      if (++head == k.a.n_kv) {
        head = 0;
        ++pair;
        loaded = false;
      }
      if (any) return true;
    }
    return false;
  }
};

// E4M3 scales of a tile: this one's, the next one's, and the last one's that a
// slower warp may still be reading.
constexpr int kScaleTurns = 3;
constexpr int kScales = 2 * kKT + kKT / 4;  // key scales, value scales, log2 of the largest of every four of these

template <bool E4M3>
struct Ctrl {
  uint64_t full[kMaxSlots], empty[kMaxSlots];
  uint64_t s_full[2][2], p_full[2][2], pv_done[2][2];  // [stream][half of the key tile]
  uint64_t q_full[2], o_full, fin;
  Start start;
  Walk walk[2];  // of the softmax warpgroups: kept here, not in every thread's registers
  Rings rings[2];  // theirs too (E4M3)
  Seg seg[2][2];  // [warpgroup][turn]
  int more[2][2];
  int abort_flag;
  uint32_t tmem;
  // per warpgroup: scales; (m, l) of the join; row scales of Q.
  // Before the roles start: scratch of the scan
  alignas(16) float x[2][E4M3 ? kScaleTurns * kScales : 256];
};
template <bool E4M3>
constexpr int kCtrlBytes = (int)((sizeof(Ctrl<E4M3>) + 1023) / 1024 * 1024);
static_assert(kCtrlBytes<false> <= 3 * 1024, "control block: six 32 KiB slots beside one Q tile");

// -------------------------------------------------------------- PTX helpers

// Bounded wait on an mbarrier phase, like mbar_wait_bounded; the clock and the
// abort flag are looked at after every 64 polls only (a poll already suspends
// the thread for a while).
__device__ __forceinline__ bool wait_on(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* status) {
  if (mbar_try_wait(bar, parity)) return true;
  unsigned long long t0 = 0;
  for (int i = 0;; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((i & 63) != 63) continue;
    if (*abort_flag) return false;
    const unsigned long long t = globaltimer_ns();
    if (!t0) t0 = t;
    if (t - t0 > kWaitLimitNs) {
      *abort_flag = 1;
      report_status(status, DFLASH_ERR_DEVICE_TIMEOUT);
      return false;
    }
  }
}
// Whether the phase is complete, without waiting.
__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ bool warp_wait_on(uint64_t* bar, uint32_t parity, volatile int* abort_flag, int* status) {
  const bool ok = wait_on(bar, parity, abort_flag, status);
  return __all_sync(0xffffffffu, ok);
}

__device__ __forceinline__ void tma_load_3d(void* dst, const void* tmap, uint64_t* bar, int c0, int c1, int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(tmap)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}

// Tensor-memory accesses of the softmax.  They touch no C++ memory, so none
// clobbers it (shared-memory loads may move across them); being volatile they
// keep their order, and the wait passes the loaded values through, so that no
// use of them moves above it.
__device__ __forceinline__ void tmem_ld_x32(uint32_t taddr, float (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]),
        "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]),
        "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]),
        "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
      : "r"(taddr));
}
__device__ __forceinline__ void wait_ld(float (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
      : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
        "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]),
        "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]),
        "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]), "+f"(v[30]), "+f"(v[31]));
}
template <int N>
__device__ __forceinline__ void tmem_st(uint32_t taddr, const uint32_t (&r)[N]) {
  static_assert(N == 8 || N == 16, "columns");
  if (N == 8)
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]));
  else
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[N - 8]),
        "r"(r[N - 7]), "r"(r[N - 6]), "r"(r[N - 5]), "r"(r[N - 4]), "r"(r[N - 3]), "r"(r[N - 2]), "r"(r[N - 1]));
}

// Instruction descriptor of kind::f8f6f4: float32 accumulator, A E4M3 (0) or
// E5M2 (1), B E4M3.
__host__ __device__ constexpr uint32_t idesc_f8(int M, int N, uint32_t a_format) {
  return (1u << 4) | (a_format << 7) | ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// The warp's MMA instructions are executed by one elected lane while the whole
// warp runs the same control flow, so that descriptors stay in uniform
// registers.
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r != 0;
}

__device__ __forceinline__ uint64_t desc64(uint32_t lo, uint32_t hi) { return ((uint64_t)hi << 32) | lo; }

template <bool E4M3>
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  if (!E4M3) {
    tc_mma_f16(d, a, b, idesc, accumulate);
  } else {
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
  }
}
// Half a tile's V, kHK rows of codes as TMA left them, as fp16 in the layout of
// a 16-bit tile (spans of 64 columns, 128-byte swizzle), by the threads t = 0 ..
// N - 1; rows outside [lo, hi) as zeros: no row of the item sees them, and a
// weight of 0 times whatever lies there must not become NaN.  Eight threads read
// 4 chunks of 16 codes from either of two rows whose chunks lie in different
// banks, as they come and as they go: r and r ^ 5 for rows of 128 codes, r and
// r ^ 1 for rows of 64.
template <int HD, int N>
__device__ __forceinline__ void widen_v(const uint8_t* codes, uint8_t* wide, int lo, int hi, int t) {
  constexpr int kRows = N * 16 / HD;  // at once
  const int other = (t >> 2) & 1;
  const int r0 = HD == 128 ? (t >> 6) * 8 + (((t >> 3) & 3) ^ (other * 5)) : (t >> 3) * 2 + other;
  const int ch = HD == 128 ? ((t >> 5) & 1) * 4 + (t & 3) : t & 3;
  // all that the rows' swizzle depends on repeats with kRows
  const uint8_t* from = codes + r0 * HD + (HD == 128 ? ch ^ (r0 & 7) : ch ^ ((r0 >> 1) & 3)) * 16;
  uint8_t* to = wide + (ch >> 2) * (kHK * 128) + r0 * 128;
  const int at = (2 * ch) & 7;
  uint8_t *const to0 = to + ((at ^ (r0 & 7)) << 4), *const to1 = to + (((at + 1) ^ (r0 & 7)) << 4);
#pragma unroll
  for (int r = 0; r < kHK; r += kRows) {
    uint4 c = make_uint4(0u, 0u, 0u, 0u), w;
    if (r0 + r >= lo && r0 + r < hi) c = *reinterpret_cast<const uint4*>(from + r * HD);
    w = make_uint4(e4m3x2_to_f16x2((uint16_t)c.x), e4m3x2_to_f16x2((uint16_t)(c.x >> 16)),
                   e4m3x2_to_f16x2((uint16_t)c.y), e4m3x2_to_f16x2((uint16_t)(c.y >> 16)));
    *reinterpret_cast<uint4*>(to0 + r * 128) = w;
    w = make_uint4(e4m3x2_to_f16x2((uint16_t)c.z), e4m3x2_to_f16x2((uint16_t)(c.z >> 16)),
                   e4m3x2_to_f16x2((uint16_t)c.w), e4m3x2_to_f16x2((uint16_t)(c.w >> 16)));
    *reinterpret_cast<uint4*>(to1 + r * 128) = w;
  }
}

template <int HD, bool E4M3, bool BF16>
struct Cfg {
  static constexpr int kRow = E4M3 ? HD : HD * 2;          // bytes of a cached row
  static constexpr int kTile = kKT * kRow;                 // of a K or V tile
  static constexpr int kQTerms = E4M3 ? (BF16 ? 2 : 3) : 1;
  static constexpr bool kPBf16 = !E4M3 && BF16;            // type of the weights and of V
  static constexpr int kQTile = kMT * kRow * kQTerms;
  static constexpr int kWide = E4M3 ? kHK * HD * 2 : 0;    // V of half a tile, widened to fp16
  // Growth of a row's reference (log2) before O is rescaled: as much as the
  // weights' type holds beside the factor on them (fp16 to 2^15).  A bf16 has
  // float32's exponents (mid-size prompt chunk: 112.7 us with 2^60, 112.9 with
  // 2^30, 115.4 with 2^15).
  static constexpr float kHeadroom = kPBf16 ? 30.0f : 4.0f;
  // log2 of the factor on the weights.  A bf16 weight is at most 1, whatever its
  // reference has grown by since, so that the sums of weights and values stay
  // finite as far as the formula's do (2^30 let values above 2^80 overflow); what
  // is lost for it lies 2^96 below the largest.  An fp16 ends at 2^-24: the weights
  // of a long tail behind one dominant key need the range more than rescaling
  // needs headroom.  Their last place is 2^-35 of the reference; without the factor
  // it is 2^-24, no less than each of 131,072 keys weighs that share a hundredth of
  // a row.  2^0 / 2^7 / 2^9 / 2^11 / 2^13, the headroom what they leave of 2^15:
  // mid-size fp16 prompt chunk 137.8 / 142.2 / 143.5 / 144.8 / 146.4 us, long one
  // 860 / 878 / 880 / 890 / 899, blocks alike.  Over codes 2^7 / 2^9 / 2^11: ragged
  // blocks 192.5 / 193.9 / 195.9 us, long prompt chunk 1,611 / 1,615 / 1,622.
  static constexpr float kShift = kPBf16 ? -kHeadroom : 15.0f - kHeadroom;
  // log2 of the smallest value scale that a reference follows: weights without
  // their scales, at most 2^15 over it, stay far from float32's end.
  static constexpr float kLeastScale = -64.0f;
  // Operand layouts.  A row of K or Q is kRow bytes cut into spans of at most
  // 128; a span of all rows is one swizzled tile (128-byte swizzle, or 64 for
  // 64-byte rows), spans kKT x span bytes apart.
  static constexpr int kSpan = kRow < 128 ? kRow : 128;
  static constexpr int kStepsPerSpan = kSpan / 32;         // an MMA takes 32 bytes of K and Q
  static constexpr int kQkSteps = kRow / 32;
  static constexpr int kPvSteps = kHK / 16;  // keys per MMA
  static constexpr int kVStep = 16 * 128;    // bytes of V to the next MMA's keys
  // Column of the weights of MMA kk in S: the weights of 32 keys lie in the first
  // of the 32 columns that held those keys' scores.
  static __host__ __device__ constexpr uint32_t p_col(int kk) { return (kk >> 1) * 32 + (kk & 1) * 8; }
  static constexpr uint32_t kDescHi = (uint32_t)((8 * kSpan) >> 4) | (1u << 14) | ((kSpan == 64 ? 4u : 2u) << 29);
  // V, 16-bit spans of 128 bytes: next span along N in the lower word
  static constexpr uint32_t kVDescHi = (uint32_t)((8 * 128) >> 4) | (1u << 14) | (2u << 29);
  static constexpr uint32_t kVDescLo = (uint32_t)(((E4M3 ? kHK : kKT) * 128) >> 4) << 16;
  static __host__ __device__ constexpr uint32_t id_qk(int term) {
    return E4M3 ? idesc_f8(kMT, kHK, term > 0) : idesc_f32acc(kMT, kHK, BF16);
  }
  static constexpr uint32_t kIdPv = idesc_f32acc(kMT, HD, kPBf16) | (1u << 16);  // V MN-major
};

// ------------------------------------------------------------------ Q tile

// Rows [row0, row0 + 128) of the item's packed rows, those of them in
// [r_begin, r_end), into a swizzled tile by the 128 threads of a warpgroup;
// rows past the item's keep what was there: it only reaches lanes that nobody
// reads.  E4M3: as terms, the inverse of the row's factor in row_scale.
template <int HD, bool E4M3, bool BF16>
__device__ __forceinline__ void load_q(const PagedAttnArgs& a, const Item& it, int head, int row0, uint8_t* q_s,
                                       float* row_scale, int t, int r_begin, int r_end) {
  constexpr int kCh = HD / 8;  // 16-byte chunks of a row
  r_end = min(r_end, it.rows - row0);
  auto source = [&](int idx, bool* ok) {
    const int pr = row0 + idx / kCh;
    *ok = pr < it.rows;
    const int packed = it.row0 + (*ok ? pr : 0);
    const int tok = packed / a.group, g = packed - tok * a.group;
    return a.q + ((size_t)(it.s0 + tok) * a.q_row + (size_t)(head * a.group + g) * a.q_head + (idx % kCh) * 8) * 2;
  };
  if (!E4M3) {
    for (int idx = r_begin * kCh + t; idx < r_end * kCh; idx += 128) {
      bool ok;
      const uint8_t* src = source(idx, &ok);
      const int r = idx / kCh, ch = idx % kCh;
      cp_async16(q_s + (ch >> 3) * (kMT * 128) + swz(r, (ch & 7) * 8), src, true);
    }
    return;
  }
  constexpr int kBatch = 4;  // loads in flight per thread
  for (int i0 = r_begin * kCh; i0 < r_end * kCh; i0 += 128 * kBatch) {
    uint4 w[kBatch];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      bool ok;
      const uint8_t* src = source(i0 + u * 128 + t, &ok);
      w[u] = ok ? __ldg(reinterpret_cast<const uint4*>(src)) : make_uint4(0u, 0u, 0u, 0u);
    }
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      const int idx = i0 + u * 128 + t, r = idx / kCh, ch = idx % kCh;
      const uint32_t v[4] = {w[u].x, w[u].y, w[u].z, w[u].w};
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) m = __vmaxu2(m, v[i] & 0x7FFF7FFFu);
#pragma unroll
      for (int o = kCh / 2; o > 0; o >>= 1) m = __vmaxu2(m, __shfl_xor_sync(0xffffffffu, m, o));
      m = max(m & 0xFFFFu, m >> 16);
      // exponent field of the row's largest magnitude; a row that is not
      // finite becomes NaN
      const int e = max((int)(__float_as_uint(unpack16<BF16>(m).x) >> 23), 8);
      const float f = e < 255 ? __uint_as_float((uint32_t)(261 - e) << 23) : __uint_as_float(0x7FC00000u);
      float x[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 y = unpack16<BF16>(v[i]);
        x[2 * i] = y.x * f;
        x[2 * i + 1] = y.y * f;
      }
      const int chunk = HD == 128 ? (ch >> 1) ^ (r & 7) : (ch >> 1) ^ ((r >> 1) & 3);
      uint8_t* dst = q_s + r * HD + chunk * 16 + (ch & 1) * 8;
#pragma unroll
      for (int term = 0; term < Cfg<HD, E4M3, BF16>::kQTerms; ++term) {
        uint32_t c[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          c[i] = __nv_cvt_float2_to_fp8x2(make_float2(x[2 * i], x[2 * i + 1]), __NV_SATFINITE,
                                          term ? __NV_E5M2 : __NV_E4M3);
          // an E5M2 is the upper byte of an fp16
          const float2 y = unpack16<false>(term ? __byte_perm(c[i], 0u, 0x1404) : e4m3x2_to_f16x2((uint16_t)c[i]));
          x[2 * i] -= y.x;
          x[2 * i + 1] -= y.y;
        }
        *reinterpret_cast<uint2*>(dst + term * (kMT * HD)) = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
      }
      if (ch == 0) row_scale[r] = e < 255 ? __uint_as_float((uint32_t)(e - 7) << 23) : 1.0f;
    }
  }
}

// ------------------------------------------------------------------ kernel

// WIDES: E4M3, buffers of widened V that a stream has: one for either half of a
// tile, or one for both.
template <int HD, bool E4M3, bool BF16, int WIDES>
__global__ void __launch_bounds__(kThreads, 1)
    paged_attention_kernel(const __grid_constant__ CUtensorMap tmK, const __grid_constant__ CUtensorMap tmV,
                           const KernelArgs k) {
  using C = Cfg<HD, E4M3, BF16>;
  grid_dependents_launch();
  extern __shared__ __align__(1024) uint8_t smem[];
  const PagedAttnArgs& a = k.a;
  uint8_t* ring_s = smem;
  uint8_t* q_s = ring_s + 2 * k.half * C::kTile;
  uint8_t* wide_s = q_s + k.q_tiles * C::kQTile;  // E4M3: widened V, [stream][buffer]
  auto* c = reinterpret_cast<Ctrl<E4M3>*>(smem + kSmem - kCtrlBytes<E4M3>);
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
    for (int s = 0; s < 2 * k.half; ++s) {
      mbar_init(&c->full[s], 1);
      mbar_init(&c->empty[s], 2);
    }
    for (int i = 0; i < 2; ++i) {
      for (int h = 0; h < 2; ++h) {
        mbar_init(&c->s_full[i][h], 1);
        mbar_init(&c->p_full[i][h], 4);
        mbar_init(&c->pv_done[i][h], 1);
      }
      mbar_init(&c->q_full[i], 1);
    }
    mbar_init(&c->o_full, 2);
    mbar_init(&c->fin, 2);
    c->abort_flag = 0;
    fence_barrier_init();
    tma_prefetch_desc(&tmK);
    tma_prefetch_desc(&tmV);
  }
  if (warp == 1) {
    tmem_alloc(&c->tmem, 512);
    tmem_relinquish();
  }
  grid_dependency_wait();

  // ---- the line's length and this CTA's part of it
  const int pairs = a.batch.B * k.rts;
  const int per = (pairs + kThreads - 1) / kThreads;
  const int p0 = min(pairs, tid * per), p1 = min(pairs, p0 + per);
  unsigned long long mine = 0;
  for (int p = p0; p < p1;) {
    const int b = p / k.rts;
    int rt = p - b * k.rts;
    RequestSpan r;
    if (!item_rows(a, b, &r)) {
      if (blockIdx.x == 0) report_status(a.status, DFLASH_ERR_SHAPE);
      p = (b + 1) * k.rts;
      continue;
    }
    const int items = (r.n * a.group + 2 * kMT - 1) / (2 * kMT);
    for (; rt < items && p < p1; ++rt, ++p) mine += make_item(k, r, b, rt).units;
    if (rt >= items) p = (b + 1) * k.rts;
  }
  unsigned long long total;
  const unsigned long long excl = block_exclusive_scan(mine, reinterpret_cast<unsigned long long*>(c->x), &total);
  const long long W = (long long)total * a.n_kv;
  const int ctas = (int)min((long long)gridDim.x, W);
  if (cta >= ctas) {
    if (tid == 0) k.rec[cta].pair = -1;
    if (warp == 1) tmem_dealloc(c->tmem, 512);  // the scan's barriers came after its allocation
    return;
  }
  // short divisions where they do
  const bool few = W < 1 << 23;
  const long long w0 = few ? (int)W * cta / ctas : W * cta / ctas;
  const long long w1 = few ? (int)W * (cta + 1) / ctas : W * (cta + 1) / ctas;
  if ((long long)excl * a.n_kv <= w0 && w0 < (long long)(excl + mine) * a.n_kv) {
    long long at = (long long)excl * a.n_kv;
    int p = p0;
    Item it;
    while (find_item(k, &p, pairs, &it)) {
      const long long n = (long long)it.units * a.n_kv;
      if (w0 < at + n) break;
      at += n;
      ++p;
    }
    const int off = (int)(w0 - at);  // fewer than n_kv x units of an item
    c->start.it = it;
    c->start.pair = p;
    c->start.head = off / it.units;
    c->start.off = off - c->start.head * it.units;
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = c->tmem;
  volatile int* stop = &c->abort_flag;
  if (warp < 4) {
    if (warp == 0 || warp == 3) {
      // -------------------------------------- producers: K (0) and V (3)
      const int side = warp ? 1 : 0;
      const bool lead = elect_one();
      const void* map = side ? &tmV : &tmK;
      Walk walk;
      Seg s;
      walk.begin(c->start, w1 - w0);
      const int shift = a.batch.page_shift, page_rows = 1 << shift, per_tile = kKT >> shift;
      auto advance = [&](int& at, uint32_t& phase, int n) { Rings::advance(k.half, at, phase, n); };
      Rings rings = {};
      uint32_t used = 0, parity = 0;  // per slot: in use, phase of its last load
      bool ok = true;
      while (ok && walk.next(k, &s)) {
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
        int s0 = rings.at[0], s1 = rings.at[1];
        uint32_t q0 = rings.phase[0], q1 = rings.phase[1];
        if (s.split) {
          advance(s0, q0, side);
          advance(s1, q1, side);
        }
        for (int t = s.t0; ok && t < s.t0 + s.nt; ++t) {
          const int first = t * per_tile;
          // pages of the tile that hold a visible position
          const int g0 = max(first, g_lo), g1 = min(first + per_tile, g_hi + 1);
          if (first + per_tile > ids_at + 32) {
            ids_at += 32;
            ids = ids_next;
            ids_next = look_up(ids_at + 32);
          }
          const int r = s.split ? (t - s.t0) & 1 : side;
          const int slot = r ? k.half + s1 : s0;
          const uint32_t ph = r ? q1 : q0;
          ok = warp_wait_on(&c->empty[slot], ph ^ 1u, stop, a.status);
          if (!ok) break;
          uint8_t* dst = ring_s + slot * C::kTile;
          if (lead) mbar_arrive_expect_tx(&c->full[slot], (uint32_t)((g1 - g0) << shift) * C::kRow);
          for (int g = g0; g < g1; ++g) {
            int id = __shfl_sync(0xffffffffu, ids, g - ids_at);
            if (id < 0 || id >= a.batch.n_pages) {
              if (lead) report_status(a.status, DFLASH_ERR_ARG);
              id = a.batch.n_pages;  // outside the tensor: TMA fills zeros
            }
            if (lead) {
              const int row = (g - first) << shift;
#pragma unroll
              for (int h = 0; h < C::kRow / C::kSpan; ++h)
                tma_load_3d(dst + (h * kKT + row) * C::kSpan, map, &c->full[slot], h * 64, s.head * page_rows, id);
            }
          }
          __syncwarp();
          used |= 1u << slot;
          parity = (parity & ~(1u << slot)) | (ph << slot);
          if (r)
            advance(s1, q1, s.split ? 2 : 1);
          else
            advance(s0, q0, s.split ? 2 : 1);
        }
        rings.leave(k.half, s.split, s.nt);
      }
      if (!ok && lead) {
        // a wait gave up: let the copies in flight land before the CTA leaves
        int dummy = 0;
        for (int j = 0; j < 2 * k.half; ++j)
          if ((used >> j) & 1u) (void)mbar_wait_bounded(&c->full[j], (parity >> j) & 1u, &dummy, nullptr, 100000000ull);
      }
      __syncwarp();
    } else {
      // ------------------------------------------ MMA issuer of one stream
      // A wait costs hundreds of clocks even when its phase is long complete
      // (the operand reads of the tensor cores keep shared memory busy), so
      // each stream has a warp of its own, and K and V are waited for before
      // P: after it the products follow one another without a wait.
      const int st = warp - 1;
      const bool lead = elect_one();
      const uint32_t q_d = smem_u32(q_s) >> 4;
      constexpr uint32_t kTileD = C::kTile >> 4;
      const uint32_t tS = tmem + st * kKT, tO = tmem + kColO + st * 128;
      constexpr uint32_t kHalfD = (kHK * C::kSpan) >> 4;  // a tile's second half of K rows
      constexpr uint32_t kHalfV = E4M3 ? (WIDES - 1) * (C::kWide >> 4) : kHalfD;  // of V
      uint32_t seg = 0, p_phase = 0;
      Rings rings = {};
      bool ok = true;
      while (true) {
        ok = warp_wait_on(&c->q_full[0], seg & 1u, stop, a.status) &&
             warp_wait_on(&c->q_full[1], seg & 1u, stop, a.status);
        // the segment as this stream's warpgroup described it (it stays until o_full)
        const Seg& s = c->seg[st][seg & 1u];
        if (!ok || !c->more[st][seg & 1u]) break;
        ++seg;
        const bool split = s.split;
        const int nt = s.nt, lo = s.it.lo, hi = s.it.hi;
        const int stride = split ? 2 : 1, first = split ? st : 0;
        int k0 = (s.t0 + first) * kKT;  // first key of the job
        auto advance = [&](int& at, uint32_t& phase, int n) { Rings::advance(k.half, at, phase, n); };
        // K and V slots: of the stream's own ring in turn, or of the K and the V ring
        const bool kr = split && st, vr = !split || st;
        uint8_t* const k_s = ring_s + (kr ? k.half * C::kTile : 0);
        uint8_t* const v_s = ring_s + (vr ? k.half * C::kTile : 0);
        uint64_t *const k_full = c->full + (kr ? k.half : 0), *const k_empty = c->empty + (kr ? k.half : 0);
        uint64_t *const v_full = c->full + (vr ? k.half : 0), *const v_empty = c->empty + (vr ? k.half : 0);
        const uint32_t k_d = smem_u32(k_s) >> 4;
        const uint32_t v_d = smem_u32(E4M3 ? wide_s + st * WIDES * C::kWide : v_s) >> 4;
        int ks = rings.at[kr], vs = rings.at[vr];
        uint32_t kp = rings.phase[kr], vp = rings.phase[vr];
        if (split) advance(vs, vp, 1);
        const uint32_t qd = q_d + (split ? 0u : (uint32_t)st * (C::kQTile >> 4)) + (1u << 16);
        // every slot is given back twice: by both streams, or twice by one
        auto give_back = [&](uint64_t* bar) {
          tc_commit(bar);
          if (split) mbar_arrive(bar);
        };
        auto qk = [&](int h) {
          const uint32_t kd = k_d + ks * kTileD + h * kHalfD + (1u << 16);
          if (lead) {
#pragma unroll
            for (int term = 0; term < C::kQTerms; ++term)
#pragma unroll
              for (int kk = 0; kk < C::kQkSteps; ++kk) {
                const uint32_t off = (kk / C::kStepsPerSpan) * ((kKT * C::kSpan) >> 4) + (kk % C::kStepsPerSpan) * 2;
                mma_ss<E4M3>(tS + h * kHK, desc64(qd + term * ((kMT * C::kRow) >> 4) + off, C::kDescHi),
                             desc64(kd + off, C::kDescHi), C::id_qk(term), term > 0 || kk > 0);
              }
            tc_commit(&c->s_full[st][h]);
            if (h) give_back(&k_empty[ks]);
          }
          __syncwarp();
          if (h) advance(ks, kp, stride);
        };
        tc_fence_after();
        if (first < nt) {
          ok = warp_wait_on(&k_full[ks], kp, stop, a.status);
          tc_fence_after();
          if (ok) {
            qk(0);
            qk(1);
          }
        }
        for (int t = first; ok && t < nt; t += stride, k0 += stride * kKT) {
          if (!E4M3) ok = warp_wait_on(&v_full[vs], vp, stop, a.status);
          if (!E4M3 && (k0 < lo || k0 + kKT > hi)) {
            // V rows that no row of the item sees
            uint4* v = reinterpret_cast<uint4*>(v_s + vs * C::kTile);
            for (int idx = lane; idx < kKT * (C::kRow / 16); idx += 32) {
              const int key = k0 + (idx / (C::kSpan / 16)) % kKT;  // a row of a span: all its chunks, whatever the swizzle
              if (key < lo || key >= hi) v[idx] = make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();
            __syncwarp();
          }
          const bool more = t + stride < nt;
          bool early = false;  // the next tile's first scores are on their way
          const uint32_t vd = v_d + (E4M3 ? 0u : vs * kTileD) + C::kVDescLo;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            ok = ok && warp_wait_on(&c->p_full[st][h], p_phase, stop, a.status);
            if (!ok) break;
            tc_fence_after();
            if (lead) {
              const uint32_t keep = t > first || h > 0;  // O holds earlier jobs
#pragma unroll
              for (int kk = 0; kk < C::kPvSteps; ++kk)
                tc_mma_f16_ta(tO, tS + h * kHK + C::p_col(kk),
                              desc64(vd + h * kHalfV + kk * (C::kVStep >> 4), C::kVDescHi), C::kIdPv,
                              kk > 0 ? 1u : keep);
              tc_commit(&c->pv_done[st][h]);
              if (h && !E4M3) give_back(&v_empty[vs]);
              if (h && E4M3) {  // its codes have been read: P came after them
                mbar_arrive(&v_empty[vs]);
                if (split) mbar_arrive(&v_empty[vs]);
              }
            }
            __syncwarp();
            // P of a job overwrites its S: the half's next scores follow its
            // P V in the tensor pipe's order.  If the next K tile is not there
            // yet, this tile's second half goes first, so that V is given back
            // (decoding, where the loads set the pace).
            if (more && h == 0) early = __all_sync(0xffffffffu, mbar_test(&k_full[ks], kp));
            if (more && h == 1 && !early) {
              ok = warp_wait_on(&k_full[ks], kp, stop, a.status);
              if (!ok) break;
            }
            if (more && (h == 1 || early)) tc_fence_after();
            if (more && ((h == 0) == early)) qk(0);
            if (more && h == 1) qk(1);
          }
          if (!ok) break;
          p_phase ^= 1u;
          advance(vs, vp, stride);
        }
        if (!ok) break;
        if (lead) tc_commit(&c->o_full);
        __syncwarp();
        rings.leave(k.half, split, nt);
      }
      if (lead) tc_commit(&c->fin);  // every MMA this thread issued
      __syncwarp();
    }
  } else {
    // ------------------------------------------------------------ softmax
    const int wg = (warp >> 2) - 1, t = tid & 127;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lane_off + wg * kKT, tO = tmem + lane_off + kColO;
    float* const x0 = c->x[wg];
    uint32_t tiles = 0, seg = 0;
    // the next segment's description, a segment ahead
    auto describe = [&](uint32_t turn) {
      Seg* n = &c->seg[wg][turn & 1u];
      const bool more = c->walk[wg].next(k, n);
      c->more[wg][turn & 1u] = more;
      if (E4M3 && more) {
        Rings& rings = c->rings[wg];
        const int vr = !n->split || wg;
        n->v_at = rings.at[vr];
        n->v_phase = rings.phase[vr];
        if (n->split) Rings::advance(k.half, n->v_at, n->v_phase, 1);
        rings.leave(k.half, n->split, n->nt);
      }
      if (wg == 0 && more && n->first && !n->last) {
        const long long u = w0 + n->end - 1;  // the item's last unit
        const int last = few ? ((int)(u + 1) * ctas - 1) / (int)W : (int)(((u + 1) * ctas - 1) / W);
        k.rec[cta] = Rec{n->pair, n->head, n->slot, last, n->it.s0, n->it.row0, n->it.rows};
      }
    };
    if (t == 0) {
      c->walk[wg].begin(c->start, w1 - w0);
      c->rings[wg] = {};
      if (wg == 0) k.rec[cta].pair = -1;
      describe(0);
    }
    for (;; ++seg) {
      named_sync(1 + wg, 128);
      if (!c->more[wg][seg & 1u]) {
        if (t == 0) mbar_arrive(&c->q_full[wg]);  // wakes the MMA warp, which sees the end too
        break;
      }
      const Seg& s = c->seg[wg][seg & 1u];
      const Item& it = s.it;
      // ---- queries of this stream (a split item's one tile: half by each
      // warpgroup, or all by both where the row scales are needed by both)
      if (s.split) {
        load_q<HD, E4M3, BF16>(a, it, s.head, 0, q_s, x0, t, E4M3 ? 0 : 64 * wg, E4M3 ? kMT : 64 * wg + 64);
      } else {
        load_q<HD, E4M3, BF16>(a, it, s.head, kMT * wg, q_s + wg * C::kQTile, x0, t, 0, kMT);
      }
      if (!E4M3) cp_async_wait_all();
      fence_proxy_async_smem();
      named_sync(1 + wg, 128);
      if (t == 0) {
        mbar_arrive(&c->q_full[wg]);
        describe(seg + 1);
      }
      const int pr = (s.split ? 0 : kMT * wg) + t;   // row of the item
      const bool real = pr < it.rows;
      const bool live = __any_sync(0xffffffffu, real);
      const int packed = it.row0 + (real ? pr : 0);
      const int tok = packed / a.group, g = packed - tok * a.group;
      const int pos = it.len - it.n + tok;
      // rows past the item's do not ask for masking
      const int hi = !real ? 1 << 30 : a.causal ? min(it.len, pos + 1) : it.len;
      const int lo = real && a.window ? pos - a.window + 1 : -(1 << 30);
      // (a row of tiny queries and a tiny scale: not 0, which a masked score,
      // -infinity, would turn into NaN)
      const float cs = !real ? 0.0f : E4M3 ? fmaxf(a.scale_log2 * x0[t], 0x1p-126f) : a.scale_log2;

      float m_ref = -INFINITY, l = 0.0f;
      const int step = s.split ? 2 : 1, j0 = s.split ? wg : 0, nt = s.nt, t0 = s.t0;
      // E4M3: scales of key t of the next tile, and the page of the one after
      // it, so that neither load is waited for in its own tile
      float nks = 0.0f, nvs = 0.0f;
      int page = -1;
      auto look_up = [&](int tile) {
        const int key = tile * kKT + t;
        page = -1;
        if (key >= it.lo && key < it.hi)
          page = __ldg(a.batch.table + it.b * a.batch.table_stride + (key >> a.batch.page_shift));
      };
      auto fetch = [&](int tile) {
        const int at = (tile * kKT + t) & ((1 << a.batch.page_shift) - 1);
        nks = nvs = 0.0f;
        if (page >= 0 && page < a.batch.n_pages) {
          const size_t o = (((size_t)page * a.n_kv + s.head) << a.batch.page_shift) + at;
          nks = __ldg(a.k_scale + o);
          nvs = __ldg(a.v_scale + o);
        }
      };
      // what was fetched into one of the buffers
      auto put = [&](int turn) {
        x0[turn * kScales + t] = nks;
        x0[turn * kScales + kKT + t] = nvs;
        float top = fabsf(nvs);
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        if ((t & 3) == 0) x0[turn * kScales + 2 * kKT + t / 4] = fmaxf(__log2f(top), C::kLeastScale);
      };
      // no more than 64 rows: the two warps without any widen all of V
      const bool idle = s.split && it.rows <= 64;
      // E4M3: this stream's V slots, as its MMA warp would follow them
      int vs = s.v_at;
      uint32_t vp = s.v_phase;
      int turn = 0;
      if (E4M3) {
        look_up(t0 + j0);
        fetch(t0 + j0);
        look_up(t0 + j0 + step);
        named_sync(1 + wg, 128);  // the row scales of Q have been read from there
        put(0);
        fetch(t0 + j0 + step);
        look_up(t0 + j0 + 2 * step);
      }
      for (int j = j0; j < nt; j += step) {
        const float* x = x0 + turn * kScales;
        if (E4M3) {
          // the next tile's scales go where the last but one's were; after the
          // barrier this tile's are there and nobody reads the last one's
          const int next = turn == 2 ? 0 : turn + 1;
          put(next);
          fetch(t0 + j + 2 * step);
          look_up(t0 + j + 3 * step);
          named_sync(1 + wg, 128);
          turn = next;
        }
        const uint32_t phase = tiles++ & 1u;
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          (void)warp_wait_on(&c->s_full[wg][h], phase, stop, a.status);
          tc_fence_after();
          // E4M3: this half of V for the tensor cores.  Its buffer's last reader
          // was the P V before these scores (two jobs ago) or, with one buffer,
          // the last one.
          auto widen = [&] {
            if (!E4M3) return;
            const int slot = (s.split && !wg ? 0 : k.half) + vs, at = (t0 + j) * kKT + h * kHK;
            if (h) Rings::advance(k.half, vs, vp, step);
            if (idle && t < 64) return;
            if (h == 0) (void)warp_wait_on(&c->full[slot], vp, stop, a.status);
            if (WIDES == 1 && (j > j0 || h))
              (void)warp_wait_on(&c->pv_done[wg][h ^ 1], h ? phase : phase ^ 1u, stop, a.status);
            const uint8_t* codes = ring_s + slot * C::kTile + h * (kHK * C::kRow);
            uint8_t* wide = wide_s + (wg * WIDES + h * (WIDES - 1)) * C::kWide;
            if (idle)
              widen_v<HD, 64>(codes, wide, it.lo - at, it.hi - at, t - 64);
            else
              widen_v<HD, 128>(codes, wide, it.lo - at, it.hi - at, t);
            fence_proxy_async_smem();
          };
          if (!live) {
            // no query row in this warp's lanes: whatever their P holds only
            // reaches lanes of O that nobody reads
            widen();
            __syncwarp();
            if (lane == 0) mbar_arrive(&c->p_full[wg][h]);
            continue;
          }
          const uint32_t ta = tS + h * kHK;
          float v0[32], v1[32];
          tmem_ld_x32(ta, v0);
          tmem_ld_x32(ta + 32, v1);
          const int k0 = (t0 + j) * kKT + h * kHK;
          const bool edge = !__all_sync(0xffffffffu, k0 >= lo && k0 + kHK <= hi);
          const int e0 = lo - k0, e1 = hi - k0;  // visible: e0 <= e < e1
          // the scores of 32 keys, scaled and masked
          auto ready = [&](int q, float (&v)[32]) {
            if (E4M3) {
#pragma unroll
              for (int e = 0; e < 32; e += 4) {
                const float4 f = *reinterpret_cast<const float4*>(x + h * kHK + q * 32 + e);
                const float2 a0 = mul2(make_float2(v[e], v[e + 1]), make_float2(f.x, f.y));
                const float2 a1 = mul2(make_float2(v[e + 2], v[e + 3]), make_float2(f.z, f.w));
                v[e] = a0.x;
                v[e + 1] = a0.y;
                v[e + 2] = a1.x;
                v[e + 3] = a1.y;
              }
            }
            if (edge) {
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (q * 32 + e < e0 || q * 32 + e >= e1) v[e] = -INFINITY;
            }
          };
          wait_ld(v0);
          wait_ld(v1);
          ready(0, v0);
          ready(1, v1);
          // ---- the row's largest score; E4M3: of score and value scale
          float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            if (E4M3) {
              // a score times its scale is at most the largest of four times theirs
              const float* l4 = x + 2 * kKT + (h * kHK + e) / 4;
              mx[0] = fmaxf(mx[0], fmaf(fmaxf(fmaxf(v0[e], v0[e + 1]), fmaxf(v0[e + 2], v0[e + 3])), cs, l4[0]));
              mx[1] = fmaxf(mx[1], fmaf(fmaxf(fmaxf(v1[e], v1[e + 1]), fmaxf(v1[e + 2], v1[e + 3])), cs, l4[8]));
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i) mx[i] = fmaxf(mx[i], fmaxf(v0[e + i], v1[e + i]));
            }
          }
          const float m_tile = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * (E4M3 ? 1.0f : cs);
          const bool grow = m_tile > m_ref + C::kHeadroom || (m_ref == -INFINITY && m_tile > -INFINITY);
          if (__any_sync(0xffffffffu, grow)) {
            const float m_new = grow ? m_tile : m_ref;
            const float fo = grow ? ex2_approx(m_ref - m_new) : 1.0f;  // 0 while nothing was seen
            if (j > j0 || h) {
              // O holds the stream's earlier jobs: wait for the last one's
              // P V; the next one waits for this P
              (void)warp_wait_on(&c->pv_done[wg][h ^ 1], h ? phase : phase ^ 1u, stop, a.status);
              tc_fence_after();
#pragma unroll 1
              for (int i = 0; i < HD / 32; ++i) {
                const uint32_t oa = tO + wg * 128 + i * 32;
                float o[32];
                uint32_t r[16];
                tmem_ld_x32(oa, o);
                wait_ld(o);
#pragma unroll
                for (int q = 0; q < 2; ++q) {
#pragma unroll
                  for (int e = 0; e < 16; ++e) r[e] = __float_as_uint(o[q * 16 + e] * fo);
                  tmem_st(oa + q * 16, r);
                }
              }
            }
            l *= fo;
            m_ref = m_new;
          }
          // ---- weights 2^(z - m_ref + kShift); l and O carry the factor, too
          const float nb = m_ref == -INFINITY ? 0.0f : C::kShift - m_ref;
          const float2 cs2 = make_float2(cs, cs), nb2 = make_float2(nb, nb);
          float2 ls0 = make_float2(0.0f, 0.0f), ls1 = ls0;
          auto weigh = [&](int q, const float (&v)[32]) {
            uint32_t pw[16];  // 16-bit weights of 32 keys
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              float2 p0 = fma2(make_float2(v[e], v[e + 1]), cs2, nb2), p1 = fma2(make_float2(v[e + 2], v[e + 3]), cs2, nb2);
              p0 = make_float2(ex2_approx(p0.x), ex2_approx(p0.y));
              p1 = make_float2(ex2_approx(p1.x), ex2_approx(p1.y));
              ls0 = add2(ls0, p0);
              ls1 = add2(ls1, p1);
              if (E4M3) {
                const float4 f = *reinterpret_cast<const float4*>(x + kKT + h * kHK + q * 32 + e);
                p0 = mul2(p0, make_float2(f.x, f.y));
                p1 = mul2(p1, make_float2(f.z, f.w));
              }
              pw[e / 2] = pack16<C::kPBf16>(p0.x, p0.y);
              pw[e / 2 + 1] = pack16<C::kPBf16>(p1.x, p1.y);
            }
            tmem_st(ta + q * 32, pw);
          };
          weigh(0, v0);
          weigh(1, v1);
          l += (ls0.x + ls0.y) + (ls1.x + ls1.y);
          widen();
          tc_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&c->p_full[wg][h]);
        }
      }

      // ---- end of the segment: O is final
      (void)warp_wait_on(&c->o_full, seg & 1u, stop, a.status);
      tc_fence_after();
      const bool whole = s.first && s.last;
      // factors of O0 and O1 (a row-split item: of its own O)
      float f0 = 1.0f, f1 = 0.0f, M = m_ref - C::kShift, L = l;
      if (s.split) {
        named_sync(1 + wg, 128);  // scales are no longer read
        x0[t] = M;
        x0[128 + t] = l;
        named_sync(3, 256);
        const float m0 = c->x[0][t], m1 = c->x[1][t];
        M = fmaxf(m0, m1);
        f0 = m0 == -INFINITY ? 0.0f : ex2_approx(m0 - M);
        f1 = m1 == -INFINITY ? 0.0f : ex2_approx(m1 - M);
        L = c->x[0][128 + t] * f0 + c->x[1][128 + t] * f1;
        named_sync(3, 256);  // read by all before the next segment's scales
      }
      const float inv = whole ? (L > 0.0f || L != L ? 1.0f / L : 0.0f) : 1.0f;
      f0 *= inv;
      f1 *= inv;
      // columns: a split item's are shared out between the warpgroups
      const int col0 = s.split ? wg * (HD / 2) : 0, cols = s.split ? HD / 2 : HD;
      const bool have0 = s.nt > 0, have1 = s.split && s.nt > 1;
      if (live) {
        const size_t pi = (size_t)(cta * 2 + s.slot) * k.part_rows + pr;
        uint8_t* out = a.out + ((size_t)(it.s0 + tok) * a.o_row + (size_t)(s.head * a.group + g) * a.o_head) * 2;
#pragma unroll 1
        for (int i = 0; i < cols / 32; ++i) {
          const int col = col0 + i * 32;
          float o[32] = {}, o1[32] = {};
          if (have0) tmem_ld_x32(tO + (s.split ? 0 : wg * 128) + col, o);
          if (have1) tmem_ld_x32(tO + 128 + col, o1);
          wait_ld(o);
          wait_ld(o1);
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            o[e] *= f0;
            if (have1) o[e] = fmaf(o1[e], f1, o[e]);
          }
          if (!real) continue;
          if (whole) {
            uint4* dst = reinterpret_cast<uint4*>(out + col * 2);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              dst[e] = make_uint4(pack16<BF16>(o[8 * e], o[8 * e + 1]), pack16<BF16>(o[8 * e + 2], o[8 * e + 3]),
                                  pack16<BF16>(o[8 * e + 4], o[8 * e + 5]), pack16<BF16>(o[8 * e + 6], o[8 * e + 7]));
          } else {
            float4* dst = reinterpret_cast<float4*>(k.part + pi * HD + col);
#pragma unroll
            for (int e = 0; e < 8; ++e) dst[e] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          }
        }
        if (real && (!s.split || wg == 0)) {
          if (!whole)
            k.ml[pi] = make_float2(M, L);
          else if (a.lse)
            a.lse[(size_t)(it.s0 + tok) * a.n_q + s.head * a.group + g] = (M + log2f(L)) * kLn2;
        }
      }
      tc_fence_before();
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

// Joins the partial results of the item that CTA blockIdx.x of the kernel
// above started and did not finish.  What bounds it is the latency of a row's
// loads, one part after another, so a row's n parts are read by 1 to 8 warps,
// every per-th part each, whose sums are added in order; and a row of the grid
// has up to kJoinBlocks blocks.  One request of 60,000 keys and one KV head, cut
// into 152 parts, 8 rows: 56.1 us with one warp to a row, 18.7 so, of which 10.8
// are the kernel above; 64 rows: 59.7 -> 32.4 (78.9 / 50.7 / 32.4 / 29.9 us with
// 8 / 16 / 32 / 64 blocks, but a short chunk of a prompt, whose blocks mostly find
// nothing to do, takes 111.6 / 111.8 / 112.3 / 114.5).
template <int HD, bool BF16>
__global__ void __launch_bounds__(256) paged_join_kernel(const KernelArgs k) {
  __shared__ float red_o[8][HD];
  __shared__ float red_l[8];
  pdl_enter();
  const int cta = blockIdx.x;
  const Rec rec = k.rec[cta];
  if (rec.pair < 0) return;
  const PagedAttnArgs& a = k.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int n = rec.last_cta - cta + 1;
  const int per = n > 16 ? 8 : n > 8 ? 4 : n > 4 ? 2 : 1;
  static_assert(kMaxCtas <= 8 * 32 && kMaxCtas % 32 == 0, "a lane for each of a warp's parts");
  const int sub = warp & (per - 1), rows = 8 / per;
  const int mine = (n - sub + per - 1) / per;
  constexpr int kLoads = 4;
  constexpr int kE = HD / 32;
  for (int base = blockIdx.y * rows; base < rec.rows; base += gridDim.y * rows) {
    const int row = base + warp / per;
    const bool have = row < rec.rows;
    auto place = [&](int i) { return (size_t)((cta + i) * 2 + (i ? 0 : rec.slot)) * k.part_rows + row; };
    float M = -INFINITY, L = 0.0f, o[kE] = {};
    if (have) {
      // all that does not depend on M is asked for before it
      float2 v[kLoads][kE / 2];
      auto load = [&](int i0) {
#pragma unroll
        for (int u = 0; u < kLoads; ++u) {
          const float* p = k.part + place(sub + min(i0 + u, mine - 1) * per) * HD + lane * kE;
#pragma unroll
          for (int e = 0; e < kE; e += 2) v[u][e / 2] = *reinterpret_cast<const float2*>(p + e);
        }
      };
      float m[kMaxCtas / 32];
#pragma unroll
      for (int i = 0; i < kMaxCtas / 32; ++i) m[i] = i * 32 + lane < n ? k.ml[place(i * 32 + lane)].x : -INFINITY;
      const float2 ml = lane < mine ? k.ml[place(sub + lane * per)] : make_float2(-INFINITY, 0.0f);
      load(0);
#pragma unroll
      for (int i = 0; i < kMaxCtas / 32; ++i) M = fmaxf(M, m[i]);
      M = warp_max_f(M);
      const float f = ml.x == -INFINITY ? 0.0f : exp2f(ml.x - M);
      L = warp_sum(f * ml.y);
      for (int i0 = 0;;) {
#pragma unroll
        for (int u = 0; u < kLoads; ++u) {
          const float fi = __shfl_sync(0xffffffffu, f, (i0 + u) & 31);
          if (i0 + u >= mine) break;
#pragma unroll
          for (int e = 0; e < kE; e += 2) {
            o[e] = fmaf(fi, v[u][e / 2].x, o[e]);
            o[e + 1] = fmaf(fi, v[u][e / 2].y, o[e + 1]);
          }
        }
        if ((i0 += kLoads) >= mine) break;
        load(i0);
      }
    }
    if (per > 1) {
#pragma unroll
      for (int e = 0; e < kE; ++e) red_o[warp][lane * kE + e] = o[e];
      if (lane == 0) red_l[warp] = L;
      __syncthreads();
      if (sub == 0)
        for (int i = 1; i < per; ++i) {
          L += red_l[warp + i];
#pragma unroll
          for (int e = 0; e < kE; ++e) o[e] += red_o[warp + i][lane * kE + e];
        }
      __syncthreads();
    }
    if (!have || sub) continue;
    const float inv = L > 0.0f || L != L ? 1.0f / L : 0.0f;
    const int packed = rec.row0 + row, tok = packed / a.group, g = packed - tok * a.group;
    uint32_t* out = reinterpret_cast<uint32_t*>(
        a.out + ((size_t)(rec.s0 + tok) * a.o_row + (size_t)(rec.head * a.group + g) * a.o_head + lane * kE) * 2);
#pragma unroll
    for (int e = 0; e < kE; e += 2) out[e / 2] = pack16<BF16>(o[e] * inv, o[e + 1] * inv);
    if (a.lse && lane == 0)
      a.lse[(size_t)(rec.s0 + tok) * a.n_q + rec.head * a.group + g] = (M + log2f(L)) * kLn2;
  }
}

// -------------------------------------------------------------------- host

PFN_cuTensorMapEncodeTiled_v12000 g_encode = nullptr;
std::once_flag g_encode_once;

// Tensor map of one side of the cache: [pages][heads x page rows][head_dim].
int encode_pages(CUtensorMap* map, const dflash_paged_cache& c, const void* ptr, long long page_stride) {
  std::call_once(g_encode_once, [] {
    cudaDriverEntryPointQueryResult q;
    void* fn = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      g_encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  });
  if (!g_encode) return DFLASH_ERR_CUDA;
  const bool e4m3 = c.format == DFLASH_CACHE_E4M3;
  const int cell = e4m3 ? 1 : 2;
  cuuint64_t dims[3] = {(cuuint64_t)c.head_dim, (cuuint64_t)c.n_kv_heads * c.page_size, (cuuint64_t)c.n_pages};
  cuuint64_t strides[2] = {(cuuint64_t)c.head_dim * cell, (cuuint64_t)page_stride * cell};
  cuuint32_t box[3] = {(cuuint32_t)(e4m3 ? c.head_dim : 64), (cuuint32_t)c.page_size, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  const CUtensorMapDataType dt = e4m3                               ? CU_TENSOR_MAP_DATA_TYPE_UINT8
                                 : c.format == DFLASH_CACHE_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                                                 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const CUresult r = g_encode(map, dt, 3, const_cast<void*>(ptr), dims, strides, box, estr,
                              CU_TENSOR_MAP_INTERLEAVE_NONE,
                              e4m3 && c.head_dim == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? DFLASH_OK : DFLASH_ERR_CUDA;
}

struct Layout {
  float* part;
  float2* ml;
  Rec* rec;
  size_t bytes;
};

int part_rows(int group, int max_rows) { return (long long)group * max_rows > kMT ? 2 * kMT : kMT; }

Layout layout(void* ws, int group, int hd, int max_rows) {
  Carve cv(ws, kWsHeader);
  const size_t rows = (size_t)kMaxCtas * 2 * part_rows(group, max_rows);
  Layout l;
  l.rec = cv.take<Rec>(kMaxCtas);
  l.ml = cv.take<float2>(rows);
  l.part = cv.take<float>(rows * hd);
  l.bytes = cv.off;
  return l;
}

template <int HD, bool E4M3, bool BF16, int WIDES>
int launch(const CUtensorMap& tk, const CUtensorMap& tv, const PagedAttnArgs& a, void* ws, cudaStream_t s) {
  using C = Cfg<HD, E4M3, BF16>;
  auto kern = paged_attention_kernel<HD, E4M3, BF16, WIDES>;
  int dev = 0, sms = 0;
  DFL_CUDA_TRY(cudaGetDevice(&dev));
  static std::atomic<int> known[64];  // SMs of the devices the attribute is set on
  if (dev < 64 && (sms = known[dev].load())) {
  } else {
    DFL_CUDA_TRY(cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev));
    DFL_CUDA_TRY(cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem));
    if (dev < 64) known[dev].store(sms);
  }
  KernelArgs k;
  k.a = a;
  const Layout l = layout(ws, a.group, HD, a.max_rows);
  k.part = l.part;
  k.ml = l.ml;
  k.rec = l.rec;
  const long long rts = ((long long)a.max_rows * a.group + 2 * kMT - 1) / (2 * kMT);
  if (rts * a.batch.B > 1 << 30) return DFLASH_ERR_SHAPE;
  k.rts = (int)rts;
  k.part_rows = part_rows(a.group, a.max_rows);
  k.q_tiles = k.part_rows / kMT;
  k.half = min(kMaxSlots, (kSmem - kCtrlBytes<E4M3> - k.q_tiles * C::kQTile - 2 * WIDES * C::kWide) / C::kTile) / 2;
  // Cost of an item beside its tiles, for the cut of the line: setting out, the
  // queries (terms of them for E4M3), the end.  Of 0 / 1 / 2 / 4 / 8 tiles: ragged
  // E4M3 blocks 294 / 267 / 253 / 217 / 196 us; bf16 prompt chunks of 200 to 700
  // 126 / 124 / 116 / 113 / 112; 64 single tokens over 500 keys 41.3 / 39.7 / 40.0 /
  // 40.5 / 41.5.
  k.seg_cost = E4M3 ? 8 : 4;
  const int grid = sms < kMaxCtas ? sms : kMaxCtas;
  int rc;
  if ((rc = launch_pdl(kern, dim3(grid), dim3(kThreads), kSmem, s, tk, tv, k))) return rc;
  const int y = (int)min((long long)kJoinBlocks, (long long)a.max_rows * a.group);
  return launch_pdl(paged_join_kernel<HD, BF16>, dim3(grid, y), dim3(256), 0, s, k);
}

}  // namespace

size_t paged_attention_workspace(int n_q, int n_kv, int head_dim, int max_rows) {
  return layout(nullptr, n_q / n_kv, head_dim, max_rows).bytes;
}

int encode_paged_maps(const dflash_paged_cache& c, CUtensorMap* k, CUtensorMap* v) {
  const int rc = encode_pages(k, c, c.k_pages, c.k_page_stride);
  return rc ? rc : encode_pages(v, c, c.v_pages, c.v_page_stride);
}

int launch_paged_attention(const CUtensorMap& k, const CUtensorMap& v, const PagedAttnArgs& a, int head_dim,
                           int format, int type, void* ws, cudaStream_t s) {
  const bool bf = type == DFLASH_TYPE_BF16, e = format == DFLASH_CACHE_E4M3;
  // Three terms of two Q tiles leave the rings one slot each beside four widened
  // halves of V: two then.  (Elsewhere four: with two, when that was tried, ragged
  // blocks took 235 us against 216, a prompt chunk 1,696 against 1,709.)
  const bool two = part_rows(a.group, a.max_rows) > kMT;
  if (head_dim == 128) {
    if (e && bf) return launch<128, true, true, 2>(k, v, a, ws, s);
    if (e) return two ? launch<128, true, false, 1>(k, v, a, ws, s) : launch<128, true, false, 2>(k, v, a, ws, s);
    return bf ? launch<128, false, true, 2>(k, v, a, ws, s) : launch<128, false, false, 2>(k, v, a, ws, s);
  }
  if (e) return bf ? launch<64, true, true, 2>(k, v, a, ws, s) : launch<64, true, false, 2>(k, v, a, ws, s);
  return bf ? launch<64, false, true, 2>(k, v, a, ws, s) : launch<64, false, false, 2>(k, v, a, ws, s);
}

}  // namespace dfl

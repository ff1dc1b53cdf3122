// What the attention kernels over a paged cache share (paged_attention.cu,
// paged_attention_e2m1.cu): the line of work and its cut, waits, tensor-memory
// accesses, and the join of partial results.
//
// The rows of one request that read one KV head, n_b x group of them (packed row
// = new row x group + query head of the group), are cut into items of at most
// ROWS; an item runs over the key tiles (128 positions) that any of its rows
// sees.  All key tiles of all items, in order, are one line that is cut into
// equal parts, one for each CTA (one CTA per SM): unequal lengths, causal
// triangles and single long requests all balance.  A CTA that holds a whole item
// writes its result; an item cut between CTAs leaves partial (O, m, l) in the
// workspace, which a second kernel joins in CTA order.  The cut depends on the
// lengths alone, so results are the same on every run.
#pragma once

#include <atomic>
#include <cstddef>

#include "attention_util.cuh"
#include "paged_util.cuh"

namespace dfl {
namespace line {

using namespace attn;

constexpr int kKT = 128;           // keys per tile
constexpr int kMaxCtas = 160;      // the workspace has room for so many
constexpr int kJoinBlocks = 32;    // see paged_join_kernel
constexpr int kSmem = 227 * 1024;  // all that a CTA may have
constexpr float kLn2 = 0.693147180559945309f;

// Where an item that this CTA starts but does not finish continues.
struct Rec {
  int pair, head, slot, last_cta;  // pair < 0: none
  int s0, row0, rows;              // its rows (Item)
};

struct LineArgs {
  PagedAttnArgs a;
  float* part;    // [CTA][2][part_rows][HD]
  float2* ml;     // [CTA][2][part_rows]
  Rec* rec;       // [CTA]
  int rts;        // items per request at most
  int part_rows;  // 128 or 256
  int seg_cost;   // what beginning an item costs, in key tiles (launch)
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

template <int ROWS>
__device__ __forceinline__ Item make_item(const LineArgs& k, const RequestSpan& r, int b, int rt) {
  const PagedAttnArgs& a = k.a;
  Item it;
  it.b = b;
  it.s0 = r.s0;
  it.n = r.n;
  it.len = r.len;
  it.row0 = rt * ROWS;
  it.rows = min(ROWS, r.n * a.group - it.row0);
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
template <int ROWS>
__device__ __forceinline__ bool find_item(const LineArgs& k, int* pair, int end, Item* it) {
  while (*pair < end) {
    const int b = *pair / k.rts, rt = *pair - b * k.rts;
    RequestSpan r;
    if (item_rows(k.a, b, &r) && rt * ROWS < r.n * k.a.group) {
      *it = make_item<ROWS>(k, r, b, rt);
      return true;
    }
    *pair = (b + 1) * k.rts;
  }
  return false;
}

// The CTA's part of the line as segments of items.
struct Seg {
  Item it;
  int head;        // KV head
  int t0, nt;      // key tiles
  bool first, last;
  int slot;        // partial slot
  int pair;
  long long end;   // where the item ends on the line, from the CTA's first unit on
};

// Where a CTA's part of the line begins.
struct Start {
  Item it;
  int pair, head, off;  // off: units of (pair, head) before it
};

template <int ROWS>
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
  __device__ bool next(const LineArgs& k, Seg* s) {
    while (left > 0) {
      if (!loaded) {
        if (!find_item<ROWS>(k, &pair, k.a.batch.B * k.rts, &it)) return false;
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

// The line's length and this CTA's part [w0, w1) of it, by all threads; one of
// them writes *start.
struct Part {
  long long W, w0, w1;
  int ctas;  // that have a part
  bool few;  // short divisions do
  __device__ int owner(long long unit) const {  // CTA of a unit
    return few ? ((int)(unit + 1) * ctas - 1) / (int)W : (int)(((unit + 1) * ctas - 1) / W);
  }
};
template <int ROWS, int THREADS>
__device__ __forceinline__ Part find_part(const LineArgs& k, unsigned long long* scratch, Start* start) {
  const PagedAttnArgs& a = k.a;
  const int pairs = a.batch.B * k.rts;
  const int per = (pairs + THREADS - 1) / THREADS;
  const int p0 = min(pairs, (int)threadIdx.x * per), p1 = min(pairs, p0 + per);
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
    const int items = (r.n * a.group + ROWS - 1) / ROWS;
    for (; rt < items && p < p1; ++rt, ++p) mine += make_item<ROWS>(k, r, b, rt).units;
    if (rt >= items) p = (b + 1) * k.rts;
  }
  unsigned long long total;
  const unsigned long long excl = block_exclusive_scan(mine, scratch, &total);
  Part part;
  const long long W = part.W = (long long)total * a.n_kv;
  const int cta = blockIdx.x, ctas = part.ctas = (int)min((long long)gridDim.x, W);
  part.w0 = part.w1 = 0;
  const bool few = part.few = W < 1 << 23;
  if (cta >= ctas) return part;
  const long long w0 = part.w0 = few ? (int)W * cta / ctas : W * cta / ctas;
  part.w1 = few ? (int)W * (cta + 1) / ctas : W * (cta + 1) / ctas;
  if ((long long)excl * a.n_kv <= w0 && w0 < (long long)(excl + mine) * a.n_kv) {
    long long at = (long long)excl * a.n_kv;
    int p = p0;
    Item it;
    while (find_item<ROWS>(k, &p, pairs, &it)) {
      const long long n = (long long)it.units * a.n_kv;
      if (w0 < at + n) break;
      at += n;
      ++p;
    }
    const int off = (int)(w0 - at);  // fewer than n_kv x units of an item
    start->it = it;
    start->pair = p;
    start->head = off / it.units;
    start->off = off - start->head * it.units;
  }
  return part;
}

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
__global__ void __launch_bounds__(256) paged_join_kernel(const LineArgs k) {
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

struct Layout {
  float* part;
  float2* ml;
  Rec* rec;
  size_t bytes;
};

inline int part_rows(int group, int max_rows) { return (long long)group * max_rows > 128 ? 256 : 128; }

inline Layout layout(void* ws, int group, int hd, int max_rows) {
  Carve cv(ws, kWsHeader);
  const size_t rows = (size_t)kMaxCtas * 2 * part_rows(group, max_rows);
  Layout l;
  l.rec = cv.take<Rec>(kMaxCtas);
  l.ml = cv.take<float2>(rows);
  l.part = cv.take<float>(rows * hd);
  l.bytes = cv.off;
  return l;
}

}  // namespace line
}  // namespace dfl

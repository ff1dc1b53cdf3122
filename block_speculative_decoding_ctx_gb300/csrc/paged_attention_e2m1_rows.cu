// Attention of new rows over a paged cache held in 4 bits, for requests with more than
// 128 packed rows (prompt chunks); paged_attention_e2m1.cu has the others, the format
// and the formulas.
//
// Query rows lie on the lanes of tensor memory and keys on its columns, so that 256
// rows share a widened tile and weights go from the softmax to the values' product
// through tensor memory, not shared memory:
//   S [128 rows, 64 keys] = Q K^T,   O [128 rows, head_dim] += P V,
// for two Q tiles (streams) side by side, in jobs of half a key tile, two S to a stream.
// (Transposed, 128 rows to a tile and weights in shared memory, the prompt chunk below
// takes 1,489 us.)  An item of up to 128 rows leaves a stream idle; streams that take every
// other tile of such a one instead cost a mixed batch 557 us for 540 and prompt chunks
// 956 for 922.
//
// Values.  Widened rows are fp16 times a power of two of 32 neighbouring keys, that of the
// largest of their scales (brought to [2^12, 2^13), so 2^-34 of it may be lost): one for a
// warp that widens, and for the softmax, whose thread has a row of all 32, a factor of
// the scores and a term of the weights' exponents that it uses 32 times.
//
// Roles (640 threads):
//   warp 0        page table and bulk copies of K and V
//   warps 1, 2    issue their stream's products
//   warp 3        describes the CTA's segments of items, ahead of the others
//   warps 4-11    softmax, a warpgroup to a stream, a row to a thread; weights replace
//                 their scores in place
//   warps 12-15   widen K, half a tile at a time, half a row to a thread
//   warps 16-19   widen V
// Tensor memory: S of stream 0 | 1, 2 x 64 columns each, O of stream 0 | 1, 128 each.
//
// What bounds it, measured on GB300 (8 KV heads of 128, groups of 5, bf16): prompt chunk, 2 x
// 2,048 rows, context 8,192 to 16,384, 948 us, 1.10 PFLOP/s, 0.56 of the measured burst
// (a bf16 cache 746, E4M3 1,253).  The products as they are issued: a score product of 64
// keys with both operands in shared memory takes 80 clocks, for half the work of one of 128
// keys in 112; a job's 8 of them and 4 of the values (79 each) 956, a tile of both streams
// 3,824.  62,272 tiles of items are 410 an SM, 1.57 M of the kernel's 1.75 M cycles.  The
// tensor cores count 48 % of their rate, since the operands' reads are no work; issue slots
// 59 % (643 M instructions), shared memory 0.73 of its cycles.  Scores of 128 keys at once
// would take 3,056 clocks a tile, queries in tensor memory 2,848; neither is built.
//
// All waits are bounded, as in paged_attention_e2m1.cu.
#include "paged_e2m1.cuh"

namespace dfl {
namespace {

using namespace line;

constexpr int kThreads = 640;
// Registers: of the softmax warpgroups, of the others, and what a thread is launched with
// (softmax 144 / 152 / 160: prompt chunk 928 / 920 / 926 us).
constexpr int kRegsSoftmax = 152, kRegsOthers = 56, kRegsLaunch = 96;
static_assert(256 * kRegsSoftmax + (kThreads - 256) * kRegsOthers <= kThreads * kRegsLaunch, "the block's registers");
constexpr int kMT = 128, kItemRows = 2 * kMT;
constexpr int kHK = 64;        // keys of a job
constexpr int kMaxSlots = 4;
constexpr int kSegs = 4;       // descriptions ahead
constexpr int kWides = 3;      // widened halves of K, and of V
constexpr uint32_t kColO = 256;
constexpr int kScaleExp = 12;  // of 32 keys' largest scale
constexpr float kUnscale = 0x1p-12f;
// Weights, log2: the largest there may be, and what a reference that grows makes of its
// job's largest, so that the last place of a weight is 2^-32 of that (2^4 / 2^8 / 2^11:
// prompt chunk 920 / 936 / 952 us).
constexpr float kMaxWeight = 15.0f, kFreshWeight = 8.0f;
constexpr int kLeastK = 13, kLeastV = 127 - 64, kMost = 253;

struct Seg : line::Seg {
  int more;
};

struct Ctrl {
  uint64_t full[kMaxSlots], empty[kMaxSlots];
  uint64_t k_full[kWides], k_empty[kWides], v_full[kWides], v_empty[kWides];
  uint64_t s_full[2][2], p_full[2][2], pv_done[2][2];  // [stream][half]
  uint64_t q_full, o_full[2], fin;
  uint64_t seg_full[kSegs], seg_empty[kSegs];
  Start start;
  Walk<kItemRows> walk;
  Seg seg[kSegs];
  int abort_flag;
  uint32_t tmem;
  uint32_t bad[kMaxSlots];      // pages of the tile whose id is none
  // Exponents of K (lower half) and V of either 32 keys of a job; K may be six jobs ahead
  // of a softmax.
  alignas(8) uint32_t power[8][2];
  float factor[kItemRows];      // of a row's scores
  unsigned long long scan[33];
};
constexpr int kCtrlBytes = (int)((sizeof(Ctrl) + 1023) / 1024 * 1024);

template <int HD>
struct Cfg {
  static constexpr int kRec = e2m1_record(HD);
  static constexpr int kSlot = 2 * kKT * kRec;           // a tile's records of K, then of V
  static constexpr int kSpan = kHK * 128;                // 64 rows x 64 columns of fp16
  static constexpr int kWide = kSpan * (HD / 64);        // widened half of a tile
  static constexpr int kQTile = kMT * HD * 2;
  static constexpr int kFixed = 2 * kQTile + 2 * kWides * kWide + kCtrlBytes;
  static constexpr int kSlots = (kSmem - kFixed) / kSlot < kMaxSlots ? (kSmem - kFixed) / kSlot : kMaxSlots;
  static_assert(kSlots >= 2, "shared memory");
};

// The exponent (biased) of a record's largest scale, and its scales.
template <int HD>
__device__ __forceinline__ int row_exponent(const uint8_t* rec, bool there, uint32_t (&scale)[HD / 32]) {
  const uint8_t* const p = rec + HD / 2;
  if (HD == 128) {
    const uint4 w = *reinterpret_cast<const uint4*>(p);
    scale[0] = w.x;
    scale[1] = w.y;
    scale[HD / 64] = w.z;
    scale[HD / 32 - 1] = w.w;
  } else {
    const uint2 w = *reinterpret_cast<const uint2*>(p);
    scale[0] = w.x;
    scale[HD / 32 - 1] = w.y;
  }
#pragma unroll
  for (int i = 0; i < HD / 32; ++i) scale[i] = there ? scale[i] : 0u;  // zeros make any codes zeros
  return (int)(largest_scale<HD>(scale, rec) >> 7);
}
// Half of a record's codes as fp16 over 2^(e - kScaleExp), into a row of a widened half (`to`: the
// address of its first chunk under the 128-byte swizzle).
template <int HD>
__device__ __forceinline__ void widen_half_row(const uint8_t* rec, const uint32_t (&scale)[HD / 32], int part, int e, uint32_t to) {
  const float f = __uint_as_float((uint32_t)(254 + kScaleExp - e) << 23);
  const uint8_t* const from = rec + part * (HD / 4);
  uint32_t code[HD / 16];
  if (HD == 128) {
#pragma unroll
    for (int i = 0; i < HD / 64; ++i) {
      const uint4 w = *reinterpret_cast<const uint4*>(from + 16 * i);
      code[4 * i] = w.x;
      code[4 * i + 1] = w.y;
      code[4 * i + 2] = w.z;
      code[4 * i + 3] = w.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint2 w = *reinterpret_cast<const uint2*>(from + 8 * i);
      code[2 * i] = w.x;
      code[2 * i + 1] = w.y;
    }
  }
#pragma unroll
  for (int i = 0; i < HD / 64; ++i) {  // two blocks of 16
    const uint32_t w = part ? scale[HD / 64 + i] : scale[i];
    const uint32_t both = pack16<false>(__uint_as_float(w << 16) * f, __uint_as_float(w & 0xFFFF0000u) * f);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const uint32_t s = __byte_perm(both, 0u, c & 2 ? 0x3232 : 0x1010);
      uint32_t x[4];
      e2m1x8_to_f16x2(code[4 * i + c], x);
      const int ch = 4 * i + c;  // of this half of the row
      st_shared_x4(to ^ (ch << 4), hmul2(x[0], s), hmul2(x[1], s), hmul2(x[2], s), hmul2(x[3], s));
    }
  }
}

template <int HD>
__global__ void __launch_bounds__(kThreads, 1) paged_attention_e2m1_rows_kernel(const __grid_constant__ E2m1Args k) {
  using C = Cfg<HD>;
  grid_dependents_launch();
  extern __shared__ __align__(1024) uint8_t smem[];
  const PagedAttnArgs& a = k.a;
  uint8_t* const q_s = smem;                               // two Q tiles
  uint8_t* const k_s = q_s + 2 * C::kQTile;                // widened halves of K
  uint8_t* const v_s = k_s + kWides * C::kWide;            // and of V
  uint8_t* const ring_s = v_s + kWides * C::kWide;
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
    for (int s = 0; s < C::kSlots; ++s) {
      mbar_init(&c->full[s], 1);
      mbar_init(&c->empty[s], 8);
    }
    for (int i = 0; i < kWides; ++i) {
      mbar_init(&c->k_full[i], 4);
      mbar_init(&c->v_full[i], 4);
      mbar_init(&c->k_empty[i], 2);
      mbar_init(&c->v_empty[i], 2);
    }
    for (int i = 0; i < 2; ++i) {
      for (int h = 0; h < 2; ++h) {
        mbar_init(&c->s_full[i][h], 2);
        mbar_init(&c->p_full[i][h], 4);
        mbar_init(&c->pv_done[i][h], 1);
      }
      mbar_init(&c->o_full[i], 1);
    }
    for (int i = 0; i < kSegs; ++i) {
      mbar_init(&c->seg_full[i], 1);
      mbar_init(&c->seg_empty[i], 19);  // producer, 2 issuers, 8 widening and 8 softmax warps
    }
    mbar_init(&c->q_full, 1);
    mbar_init(&c->fin, 2);
    c->abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc(&c->tmem, 512);
    tmem_relinquish();
  }
  grid_dependency_wait();

  const Part part = find_part<kItemRows, kThreads>(k, c->scan, &c->start);
  if (cta >= part.ctas) {
    if (tid == 0) k.rec[cta].pair = -1;
    if (warp == 1) tmem_dealloc(c->tmem, 512);  // the scan's barriers came after its allocation
    return;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = c->tmem;
  volatile int* stop = &c->abort_flag;

  if (warp < 4) {
    reg_dec<kRegsOthers>();
    if (warp == 0) {
      // ------------------------------------------------ producer
      const bool lead = elect_one();
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
          ok = warp_wait_on(&c->empty[slot], ph ^ 1u, stop, a.status);
          if (!ok) break;
          const int g = first + lane;
          const int id = __shfl_sync(0xffffffffu, ids, (g - ids_at) & 31);
          const bool in = lane < per_tile && g >= g_lo && g <= g_hi;
          const bool good = in && id >= 0 && id < a.batch.n_pages;
          const uint32_t bad = __ballot_sync(0xffffffffu, in && !good);
          const uint32_t n = __popc(__ballot_sync(0xffffffffu, good));
          if (lead) {
            if (bad) report_status(a.status, DFLASH_ERR_ARG);
            c->bad[slot] = bad;
            mbar_arrive_expect_tx(&c->full[slot], n * run * 2);
          }
          __syncwarp();
          if (good) {
            uint8_t* const dst = ring_s + slot * C::kSlot + lane * run;
            const size_t head = (size_t)s.head * run;
            bulk_load(dst, k.k_pages + (size_t)id * k.k_stride + head, run, &c->full[slot]);
            bulk_load(dst + kKT * C::kRec, k.v_pages + (size_t)id * k.v_stride + head, run, &c->full[slot]);
          }
          __syncwarp();
          used |= 1u << slot;
          parity = (parity & ~(1u << slot)) | (ph << slot);
          if (++slot == C::kSlots) {
            slot = 0;
            ph ^= 1u;
          }
        }
      }
      if (!ok && lead) {
        // a wait gave up: let the copies in flight land before the CTA leaves
        int dummy = 0;
        for (int j = 0; j < C::kSlots; ++j)
          if ((used >> j) & 1u) (void)mbar_wait_bounded(&c->full[j], (parity >> j) & 1u, &dummy, nullptr, 100000000ull);
      }
      __syncwarp();
    } else if (warp < 3) {
      // ------------------------------------------------ issuer of one stream
      const int st = warp - 1;
      const bool lead = elect_one();
      constexpr uint32_t kHi = (uint32_t)((8 * 128) >> 4) | (1u << 14) | (2u << 29);  // 128-byte swizzle
      constexpr uint32_t id_qk = idesc_f32acc(kMT, kHK, false);
      constexpr uint32_t id_pv = idesc_f32acc(kMT, HD, false) | (1u << 16);  // V N-major
      const uint32_t q_d = (smem_u32(q_s + st * C::kQTile) >> 4) + (1u << 16);
      const uint32_t k_d = (smem_u32(k_s) >> 4) + (1u << 16), v_d = (smem_u32(v_s) >> 4) + ((uint32_t)(C::kSpan >> 4) << 16);
      const uint32_t tS = tmem + st * kMT, tO = tmem + kColO + st * 128;
      int wk = 0, wv = 0;              // widened halves of the next scores, of the next values
      uint32_t phk = 0, phv = 0, J = 0;  // their phases; jobs so far
      bool ok = true;
      for (uint32_t seg = 0; ok; ++seg) {
        const int sg = seg % kSegs;
        ok = warp_wait_on(&c->seg_full[sg], (seg / kSegs) & 1u, stop, a.status);
        if (!ok || !c->seg[sg].more) break;
        const int jobs = 2 * c->seg[sg].nt;
        const bool live = c->seg[sg].it.rows > st * kMT;
        __syncwarp();
        if (lead) mbar_arrive(&c->seg_empty[sg]);
        ok = warp_wait_on(&c->q_full, seg & 1u, stop, a.status);
        tc_fence_after();
        auto scores = [&](int h) {
          ok = ok && warp_wait_on(&c->k_full[wk], phk, stop, a.status);
          if (!ok) return;
          tc_fence_after();
          if (lead) {
            if (live) {
#pragma unroll
              for (int kk = 0; kk < HD / 16; ++kk)
                tc_mma_f16(tS + h * kHK, desc64(q_d + (kk >> 2) * ((kMT * 128) >> 4) + (kk & 3) * 2, kHi),
                           desc64(k_d + wk * (C::kWide >> 4) + (kk >> 2) * (C::kSpan >> 4) + (kk & 3) * 2, kHi), id_qk, kk > 0);
              tc_commit(&c->s_full[st][h]);
              mbar_arrive(&c->s_full[st][h]);  // hands on what was written before k_full: the powers
              tc_commit(&c->k_empty[wk]);
            } else {
              mbar_arrive(&c->k_empty[wk]);
            }
          }
          __syncwarp();
          if (++wk == kWides) {
            wk = 0;
            phk ^= 1u;
          }
        };
        auto values = [&](int h, bool keep) {
          ok = ok && warp_wait_on(&c->v_full[wv], phv, stop, a.status);
          if (ok && live) ok = warp_wait_on(&c->p_full[st][h], (J >> 1) & 1u, stop, a.status);
          if (!ok) return;
          tc_fence_after();
          if (lead) {
            if (live) {
#pragma unroll
              for (int kk = 0; kk < kHK / 16; ++kk)
                // the weights of 32 keys lie in the first of the 32 columns that held their scores
                tc_mma_f16_ta(tO, tS + h * kHK + (kk >> 1) * 32 + (kk & 1) * 8,
                              desc64(v_d + wv * (C::kWide >> 4) + kk * 128, kHi), id_pv, kk > 0 ? 1u : (uint32_t)keep);
              tc_commit(&c->pv_done[st][h]);
              tc_commit(&c->v_empty[wv]);
            } else {
              mbar_arrive(&c->v_empty[wv]);
            }
          }
          __syncwarp();
          if (++wv == kWides) {
            wv = 0;
            phv ^= 1u;
          }
        };
        // Weights replace their scores: a half's next scores follow its values' product
        // in the tensor pipe's order.
#pragma unroll 1
        for (int j = -2; ok && j < jobs; ++j) {
          if (j >= 0) {
            values(j & 1, j > 0);
            if (live) ++J;
          }
          if (j + 2 < jobs) scores(j & 1);
        }
        if (!ok) break;
        if (lead) tc_commit(&c->o_full[st]);
        __syncwarp();
      }
      if (lead) tc_commit(&c->fin);  // every MMA this thread issued
      __syncwarp();
    } else {
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
    const int t = tid & 127, r = t & 63, half_row = t >> 6;  // row of the job; which half of it
    const int shift = a.batch.page_shift;
    uint64_t *const w_full = of_v ? c->v_full : c->k_full, *const w_empty = of_v ? c->v_empty : c->k_empty;
    const uint32_t wide = smem_u32(of_v ? v_s : k_s) + (HD == 128 ? half_row * C::kSpan : half_row * 64) + r * 128;
    int slot = 0, w = 0;
    uint32_t ph = 0, phw = 0, J = 0;
    bool ok = true;
    for (uint32_t seg = 0; ok; ++seg) {
      const int sg = seg % kSegs;
      ok = warp_wait_on(&c->seg_full[sg], (seg / kSegs) & 1u, stop, a.status);
      if (!ok || !c->seg[sg].more) break;
      const int nt = c->seg[sg].nt, t0 = c->seg[sg].t0, lo = c->seg[sg].it.lo, hi = c->seg[sg].it.hi;
      __syncwarp();
      if (lane == 0) mbar_arrive(&c->seg_empty[sg]);
#pragma unroll 1
      for (int j = 0; j < 2 * nt; ++j, ++J) {
        const int h = j & 1;
        if (h == 0) {
          ok = warp_wait_on(&c->full[slot], ph, stop, a.status);
          if (!ok) break;
        }
        // rows that no row of the item sees, and those of no page, count as zeros
        const int at = h * kHK + r, key = (t0 + (j >> 1)) * kKT + at;
        const bool there = key >= lo && key < hi && !((c->bad[slot] >> (at >> shift)) & 1u);
        const uint8_t* const rec = ring_s + slot * C::kSlot + at * C::kRec;
        uint32_t scale[HD / 32];
        int ev = row_exponent<HD>(rec + kKT * C::kRec, there, scale);
        ev = (int)__reduce_max_sync(0xffffffffu, (unsigned)ev);
        ev = ev ? min(max(ev, kLeastV), kMost) : kZeroV;
        int e = ev;
        if (!of_v) {
          e = row_exponent<HD>(rec, there, scale);
          e = min(max((int)__reduce_max_sync(0xffffffffu, (unsigned)e), kLeastK), kMost);
          // (by the warps of the rows' first halves)
          if (lane == 0 && half_row == 0) c->power[J & 7u][r >> 5] = (uint32_t)e | ((uint32_t)ev << 16);
        }
        ok = warp_wait_on(&w_empty[w], phw ^ 1u, stop, a.status);
        if (!ok) break;
        // (128-byte swizzle: chunk c of row r lies at c ^ r % 8)
        widen_half_row<HD>(of_v ? rec + kKT * C::kRec : rec, scale, half_row, e, (wide + w * C::kWide) ^ ((r & 7) << 4));
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&w_full[w]);
          if (h) mbar_arrive(&c->empty[slot]);
        }
        if (++w == kWides) {
          w = 0;
          phw ^= 1u;
        }
        if (h && ++slot == C::kSlots) {
          slot = 0;
          ph ^= 1u;
        }
      }
    }
  } else {
    // ------------------------------------------------ softmax
    reg_inc<kRegsSoftmax>();
    const int wg = (warp >> 2) - 1, t = tid & 127;
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lanes + wg * kMT, tO = tmem + lanes + kColO + wg * 128;
    uint32_t J = 0, before = 0;  // jobs of this stream; of all earlier segments, whose or not
    for (uint32_t seg = 0;; ++seg) {
      const int sg = seg % kSegs;
      const bool have = warp_wait_on(&c->seg_full[sg], (seg / kSegs) & 1u, stop, a.status);
      // also: everybody is past the last segment
      if (any_of(3, 256, !have) || !c->seg[sg].more) break;
      const Seg& s = c->seg[sg];
      const Item& it = s.it;
      // ---- queries of this stream; rows past the item's keep what was there: it only
      // reaches lanes that nobody reads
      constexpr int kCh = HD / 8;
#pragma unroll 1
      for (int idx = t; idx < kMT * kCh; idx += 128) {
        const int r = idx / kCh, ch = idx % kCh, pr = wg * kMT + r;
        const bool real = pr < it.rows;
        if (!__any_sync(0xffffffffu, real)) break;
        const int packed = it.row0 + (real ? pr : 0), tok = packed / a.group, g = packed - tok * a.group;
        int e;
        const uint4 w = widen_q<kCh>(
            __ldg(reinterpret_cast<const uint4*>(
                a.q + ((size_t)(it.s0 + tok) * a.q_row + (size_t)(s.head * a.group + g) * a.q_head + ch * 8) * 2)),
            k.bf16, &e);
        *reinterpret_cast<uint4*>(q_s + wg * C::kQTile + (ch >> 3) * (kMT * 128) + swz(r, (ch & 7) * 8)) = w;
        if (ch == 0) c->factor[pr] = q_factor(e, a.scale_log2);
      }
      fence_proxy_async_smem();
      named_sync(3, 256);
      if (tid == 128) mbar_arrive(&c->q_full);
      const int pr = wg * kMT + t;  // row of the item
      const bool real = pr < it.rows, live = it.rows > wg * kMT;
      const int packed = it.row0 + (real ? pr : 0);
      const int tok = packed / a.group, g = packed - tok * a.group;
      const int pos = it.len - it.n + tok;
      // rows past the item's do not ask for masking
      const int hi = !real ? 1 << 30 : a.causal ? min(it.len, pos + 1) : it.len;
      const int lo = real && a.window ? pos - a.window + 1 : -(1 << 30);
      const float cs = real ? c->factor[pr] : 0.0f;
      float m_ref = -INFINITY, l = 0.0f;
      const int jobs = live ? 2 * s.nt : 0;
#pragma unroll 1
      for (int j = 0; j < jobs; ++j, ++J) {
        const int h = j & 1;
        const uint32_t phase = (J >> 1) & 1u, ta = tS + h * kHK;
        (void)warp_wait_on(&c->s_full[wg][h], phase, stop, a.status);
        tc_fence_after();
        float v0[32], v1[32];
        tmem_ld_x32(ta, v0);
        tmem_ld_x32(ta + 32, v1);
        const uint2 pw = *reinterpret_cast<const uint2*>(c->power[(before + j) & 7u]);
        float cq[2], bq[2], iq[2];
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          const uint32_t w = q ? pw.y : pw.x;
          // (tiny queries and keys: not 0, which a masked score, -infinity, would turn into NaN)
          cq[q] = fmaxf(cs * __uint_as_float(((w & 0xFFFFu) - kScaleExp) << 23), 0x1p-126f);
          bq[q] = (float)((int)(w >> 16) - 127);
          iq[q] = __uint_as_float((254u - (w >> 16)) << 23);
        }
        const int k0 = s.t0 * kKT + j * kHK;
        const bool edge = !__all_sync(0xffffffffu, k0 >= lo && k0 + kHK <= hi);
        wait_ld(v0);
        wait_ld(v1);
        if (edge) {
          const int e0 = lo - k0, e1 = hi - k0;  // visible: e0 <= e < e1
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            if (e < e0 || e >= e1) v0[e] = -INFINITY;
            if (32 + e < e0 || 32 + e >= e1) v1[e] = -INFINITY;
          }
        }
        // ---- the row's largest score, times the factor of its 32 keys
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          mx[0] = fmaxf(mx[0], v0[e]);
          mx[1] = fmaxf(mx[1], v0[e + 1]);
          mx[2] = fmaxf(mx[2], v1[e]);
          mx[3] = fmaxf(mx[3], v1[e + 1]);
        }
        const float m_tile = fmaxf(fmaf(fmaxf(mx[0], mx[1]), cq[0], bq[0]), fmaf(fmaxf(mx[2], mx[3]), cq[1], bq[1]));
        const bool grow = m_tile > m_ref + (kMaxWeight - kFreshWeight) || (m_ref == -INFINITY && m_tile > -INFINITY);
        if (__any_sync(0xffffffffu, grow)) {
          const float m_new = grow ? m_tile : m_ref;
          const float fo = grow ? ex2_approx(m_ref - m_new) : 1.0f;  // 0 while nothing was seen
          if (j > 0) {
            // O holds the stream's earlier jobs: wait for the last one's product; the next
            // waits for this P
            const uint32_t last = J - 1;
            (void)warp_wait_on(&c->pv_done[wg][last & 1u], (last >> 1) & 1u, stop, a.status);
            tc_fence_after();
#pragma unroll 1
            for (int i = 0; i < HD / 32; ++i) {
              float o[32];
              uint32_t w[16];
              tmem_ld_x32(tO + i * 32, o);
              wait_ld(o);
#pragma unroll
              for (int q = 0; q < 2; ++q) {
#pragma unroll
                for (int e = 0; e < 16; ++e) w[e] = __float_as_uint(o[q * 16 + e] * fo);
                tmem_st(tO + i * 32 + q * 16, w);
              }
            }
          }
          l *= fo;
          m_ref = m_new;
        }
        // ---- weights; l without the values' powers
        const float nb = m_ref == -INFINITY ? 0.0f : kFreshWeight - m_ref;
        auto weigh = [&](int q, const float (&v)[32]) {
          const float2 c2 = make_float2(cq[q], cq[q]), b2 = make_float2(bq[q] + nb, bq[q] + nb);
          float2 ls0 = make_float2(0.0f, 0.0f), ls1 = ls0;
          uint32_t w[16];  // 16-bit weights of 32 keys
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            float2 p0 = fma2(make_float2(v[e], v[e + 1]), c2, b2), p1 = fma2(make_float2(v[e + 2], v[e + 3]), c2, b2);
            p0 = make_float2(ex2_approx(p0.x), ex2_approx(p0.y));
            p1 = make_float2(ex2_approx(p1.x), ex2_approx(p1.y));
            ls0 = add2(ls0, p0);
            ls1 = add2(ls1, p1);
            w[e / 2] = pack16<false>(p0.x, p0.y);
            w[e / 2 + 1] = pack16<false>(p1.x, p1.y);
          }
          tmem_st(ta + q * 32, w);
          l = fmaf((ls0.x + ls0.y) + (ls1.x + ls1.y), iq[q], l);
        };
        weigh(0, v0);
        weigh(1, v1);
        tc_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&c->p_full[wg][h]);
      }

      // ---- end of the segment: O is final
      (void)warp_wait_on(&c->o_full[wg], seg & 1u, stop, a.status);
      before += 2 * s.nt;
      tc_fence_after();
      if (live) {
        const bool whole = s.first && s.last;
        const float M = m_ref == -INFINITY ? -INFINITY : m_ref - kFreshWeight;
        const float f = (whole ? (l > 0.0f || l != l ? 1.0f / l : 0.0f) : 1.0f) * kUnscale;
        const size_t pi = (size_t)(cta * 2 + s.slot) * k.part_rows + pr;
        uint8_t* const out = a.out + ((size_t)(it.s0 + tok) * a.o_row + (size_t)(s.head * a.group + g) * a.o_head) * 2;
#pragma unroll 1
        for (int i = 0; i < HD / 32; ++i) {
          float o[32] = {};
          if (s.nt > 0) tmem_ld_x32(tO + i * 32, o);
          wait_ld(o);
          if (!real) continue;
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] *= f;
          if (whole) {
            uint4* const dst = reinterpret_cast<uint4*>(out + i * 64);
            auto pack = [&](int e) { return k.bf16 ? pack16<true>(o[e], o[e + 1]) : pack16<false>(o[e], o[e + 1]); };
#pragma unroll
            for (int e = 0; e < 4; ++e) dst[e] = make_uint4(pack(8 * e), pack(8 * e + 2), pack(8 * e + 4), pack(8 * e + 6));
          } else {
            float4* const dst = reinterpret_cast<float4*>(k.part + pi * HD + i * 32);
#pragma unroll
            for (int e = 0; e < 8; ++e) dst[e] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
          }
        }
        if (real) {
          if (!whole)
            k.ml[pi] = make_float2(M, l);
          else if (a.lse)
            a.lse[(size_t)(it.s0 + tok) * a.n_q + s.head * a.group + g] = (M + log2f(l)) * kLn2;
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
int launch(E2m1Args& k, cudaStream_t s) {
  using C = Cfg<HD>;
  auto kern = paged_attention_e2m1_rows_kernel<HD>;
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
  const long long most = (long long)k.a.max_rows * k.a.group;
  k.rts = (int)((most + kItemRows - 1) / kItemRows);
  // What an item costs beside its tiles, for the cut of the line: of 2 / 4 / 8 tiles
  // prompt chunks take 922 / 920 / 907 us.
  k.seg_cost = 8;
  k.slots = C::kSlots;
  const int grid = sms < kMaxCtas ? sms : kMaxCtas;
  int rc;
  if ((rc = launch_pdl(kern, dim3(grid), dim3(kThreads), kSmem, s, k))) return rc;
  const int y = (int)min((long long)kJoinBlocks, most);
  const LineArgs& line = k;
  return k.bf16 ? launch_pdl(paged_join_kernel<HD, true>, dim3(grid, y), dim3(256), 0, s, line)
                : launch_pdl(paged_join_kernel<HD, false>, dim3(grid, y), dim3(256), 0, s, line);
}

}  // namespace

int launch_paged_attention_e2m1_rows(line::E2m1Args& k, int head_dim, cudaStream_t s) {
  return head_dim == 128 ? launch<128>(k, s) : launch<64>(k, s);
}

}  // namespace dfl

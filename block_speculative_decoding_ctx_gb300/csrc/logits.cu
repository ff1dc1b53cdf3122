// Penalties, biases and token masks on the logits of a block
// (dflash_logits_adjust; the rules are in include/dflash.h).
//
// Memory bounds it: a logit is read once (4 or 2 bytes) and written once (4);
// the arithmetic is a product, a sum and a few selects.  A block of 256
// threads takes a chunk of 2,048 ids of one request, 8 a thread, for one
// position or for several in turn: counts, prompt bits and what a rule names
// by id (drafts, biases) are then read once for all of them, and a position's
// logits are on their way (16-byte loads where the rows allow it) while the
// one before is written.  The few named ids of the chunk are gathered in list
// order; at every position one thread each computes them whole, and they are
// written over the chunk's after a barrier (an id that is named twice is
// computed twice, to the same bits).
//
// Measured on GB300, vocabulary 151,936, every rule in use: 32 requests x 16
// positions 121 us (5.4 TB/s of the bytes it cannot do without, 0.80 of the
// measured copy); ids per block x blocks an SM: 4,096 x 3 129 us, 4,096 x 2
// 125, 2,048 x 4 121, 2,048 x 5 (fewer registers, loads waited for in turn)
// 162.  16 x 8 positions of a vocabulary that is not a multiple of 4, one
// logit a load: 44 us (0.56); 69 where every id looked its mask's word up.
#include <type_traits>

#include "paged_util.cuh"

namespace dfl {
namespace {

constexpr int kLT = 256;           // threads
constexpr int kLC = 2048;          // ids per block
constexpr int kPer = kLC / kLT;    // per thread
constexpr int kWin = 4 * kLT;      // bias entries looked through at a time
// Blocks (16 for each of 152 SMs) beyond which a block takes several positions:
// one position a block leaves counts and rules to be read again by each (279 us
// where several take 121, measured below); fewer and longer blocks leave a
// single request's block of 8 on too few SMs.
constexpr int kBlocks = 2432;

template <typename T>
__device__ __forceinline__ float to_f32(T x);
template <>
__device__ __forceinline__ float to_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <>
__device__ __forceinline__ float to_f32<__half>(__half x) { return __half2float(x); }

// Logits as they are loaded: four neighbours (VEC) or one.
template <typename T, bool VEC>
struct Raw {
  using type = T;
};
template <>
struct Raw<float, true> {
  using type = float4;
};
template <>
struct Raw<__nv_bfloat16, true> {
  using type = uint2;
};
template <>
struct Raw<__half, true> {
  using type = uint2;
};
template <typename T>
__device__ __forceinline__ void widen(const float4& u, float* x) {
  x[0] = u.x;
  x[1] = u.y;
  x[2] = u.z;
  x[3] = u.w;
}
template <typename T>
__device__ __forceinline__ void widen(const uint2& u, float* x) {
  constexpr bool kBF = sizeof(T) == 2 && std::is_same_v<T, __nv_bfloat16>;
  const float2 a = unpack16<kBF>(u.x), b = unpack16<kBF>(u.y);
  x[0] = a.x;
  x[1] = a.y;
  x[2] = b.x;
  x[3] = b.y;
}
template <typename T>
__device__ __forceinline__ void widen(const T& u, float* x) {
  x[0] = to_f32(u);
}

struct Penalty {
  float r, inv_r, f, p;
};

// The quotient by r as a product with 1 / r: two roundings, a unit in the last
// place at most.
__device__ __forceinline__ float penalise(float l, int c, bool prompt, const Penalty& w) {
  if (c > 0 || prompt) l = l > 0.0f ? l * w.inv_r : l * w.r;
  return l - (w.f * (float)c + (c > 0 ? w.p : 0.0f));
}

// VEC: rows of logits, counts and outputs all lie on 16 bytes (8 for 16-bit
// logits) and V is a multiple of 4.  per: positions of a block.
template <typename T, bool VEC>
__global__ void __launch_bounds__(kLT, 4) logits_adjust_kernel(const LogitsArgs a, int per) {
  pdl_enter();
  __shared__ int d_ids[64], d_pos[64], d_n, b_ids[kWin], warp_n[kLT / 32];
  __shared__ float b_vals[kWin], more_vals[63 + kWin - kLT];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int groups = (a.G + per - 1) / per;
  const int b = blockIdx.y / groups, i0 = (blockIdx.y - b * groups) * per, i1 = min(a.G, i0 + per);
  const int v0 = blockIdx.x * kLC, v1 = min(a.V, v0 + kLC);
  const int words = (a.V + 31) / 32;

  int slot = a.r.req_slot ? __ldg(a.r.req_slot + b) : b;
  const bool slot_ok = slot >= 0 && slot < a.r.slots;
  if (!slot_ok && (a.r.counts || a.r.prompt_mask) && tid == 0) report_status(a.status, DFLASH_ERR_ARG);
  if (!slot_ok) slot = 0;
  const int32_t* counts = a.r.counts && slot_ok ? a.r.counts + (size_t)slot * a.V : nullptr;
  const uint32_t* prompt = a.r.prompt_mask && slot_ok
                               ? reinterpret_cast<const uint32_t*>(a.r.prompt_mask) + (size_t)slot * words
                               : nullptr;
  const int32_t* draft = a.r.draft ? a.r.draft + (size_t)b * (a.G - 1) : nullptr;
  auto logits = [&](int i) { return static_cast<const T*>(a.logits) + b * a.l_b + i * a.l_i; };
  auto allowed = [&](int i) {
    return a.r.allow ? reinterpret_cast<const uint32_t*>(a.r.allow) + ((size_t)b * a.G + i) * words : nullptr;
  };
  auto bit = [&](const uint32_t* m, int v) { return (__ldg(m + (v >> 5)) >> (v & 31)) & 1u; };

  // ---- this thread's ids: VEC 2 groups of 4 neighbours; otherwise one of each
  // of the warp's 8 words of a mask, which lane k < 8 holds for all of it
  auto place = [&](int k) {
    return v0 + (VEC ? ((k >> 2) * kLT + tid) * 4 + (k & 3) : (warp * kPer + k) * 32 + lane);
  };
  auto words_of = [&](const uint32_t* m) {
    const int word = (v0 >> 5) + warp * kPer + lane;
    return lane < kPer && word < words ? __ldg(m + word) : 0u;
  };
  // logits of a position and their mask words, as they come: nothing here may
  // wait for them
  constexpr int kStep = VEC ? 4 : 1, kLoads = kPer / kStep, kMasks = VEC ? kLoads : 1;
  using RawT = typename Raw<T, VEC>::type;
  auto load = [&](int i, RawT (&x)[kLoads], uint32_t (&ok)[kMasks]) {
    const T* l = logits(i);
    const uint32_t* m = allowed(i);
#pragma unroll
    for (int k = 0; k < kLoads; ++k) {
      const int v = place(k * kStep);
      if (VEC) ok[k] = ~0u;
      if (v < v1) {
        x[k] = *reinterpret_cast<const RawT*>(l + v);
        if (VEC && m) ok[k] = __ldg(m + (v >> 5));
      }
    }
    if (!VEC) ok[0] = m ? words_of(m) : ~0u;
  };
  RawT x[kLoads] = {};
  uint32_t ok[kMasks];
  load(i0, x, ok);

  Penalty w;
  w.r = a.r.repetition ? __ldg(a.r.repetition + b) : 1.0f;
  w.inv_r = __fdiv_rn(1.0f, w.r);
  w.f = a.r.frequency ? __ldg(a.r.frequency + b) : 0.0f;
  w.p = a.r.presence ? __ldg(a.r.presence + b) : 0.0f;
  // what is taken off each id's logit before the block's own drafts count, and
  // which of them were seen (bit k)
  float off[kPer];
  uint32_t seen = 0;
  const uint32_t prompts = !VEC && prompt ? words_of(prompt) : 0u;
#pragma unroll
  for (int k = 0; k < kPer; k += kStep) {
    const int v = place(k);
    int c[4] = {0, 0, 0, 0};
    if (v < v1) {
      if constexpr (VEC) {
        if (counts) {
          const int4 n = __ldg(reinterpret_cast<const int4*>(counts + v));
          c[0] = n.x;
          c[1] = n.y;
          c[2] = n.z;
          c[3] = n.w;
        }
        if (prompt) seen |= ((__ldg(prompt + (v >> 5)) >> (v & 31)) & 15u) << k;
      } else {
        if (counts) c[0] = __ldg(counts + v);
      }
    }
    if (!VEC) seen |= ((__shfl_sync(0xffffffffu, prompts, k) >> lane) & 1u) << k;
#pragma unroll
    for (int e = 0; e < kStep; ++e) {
      off[k + e] = w.f * (float)c[e] + (c[e] > 0 ? w.p : 0.0f);
      if (c[e] > 0) seen |= 1u << (k + e);
    }
  }

  int bias0 = 0, bias1 = 0;
  if (a.r.bias_start) {
    bias0 = __ldg(a.r.bias_start + b);
    bias1 = __ldg(a.r.bias_start + b + 1);
    if (bias0 < 0 || bias1 < bias0 || bias1 > a.r.n_bias) {
      if (tid == 0) report_status(a.status, DFLASH_ERR_ARG);
      bias0 = bias1 = 0;
    }
  }

  // ---- ids named by a rule.  The first kWin biases come with the drafts; any
  // further ones are added to what has been written.
  if (tid == 0) d_n = 0;
  __syncthreads();
  if (draft && tid < i1 - 1) {
    const int d = __ldg(draft + tid);
    if (d >= v0 && d < v1) {
      const int at = atomicAdd(&d_n, 1);  // their order does not matter
      d_ids[at] = d;
      d_pos[at] = tid;
    }
  }
  // entries [e0, e1) of the list that lie in the chunk, in list order; all
  // threads see the count
  auto gather = [&](int e0, int e1) {
    int total = 0;
    for (int u = e0; u < e1; u += kLT) {
      const int e = u + tid;
      int id = -1;
      if (e < e1) {
        id = __ldg(a.r.bias_ids + e);
        if ((id < 0 || id >= a.V) && blockIdx.x == 0) report_status(a.status, DFLASH_ERR_ARG);
      }
      const bool here = id >= v0 && id < v1;
      const unsigned ball = __ballot_sync(0xffffffffu, here);
      if (lane == 0) warp_n[warp] = __popc(ball);
      __syncthreads();
      int at = total;
#pragma unroll
      for (int k = 0; k < kLT / 32; ++k) {
        at += k < warp ? warp_n[k] : 0;
        total += warp_n[k];
      }
      if (here) {
        at += __popc(ball & ((1u << lane) - 1));
        b_ids[at] = id;
        b_vals[at] = __ldg(a.r.bias_vals + e);
      }
      __syncthreads();
    }
    return total;
  };
  int nb = gather(bias0, min(bias1, bias0 + kWin));
  __syncthreads();
  const int nd = d_n, named = nd + nb;
  const bool further = bias1 - bias0 > kWin;

  // thread e < named has named id e (the further ones of more than 256 are
  // taken in turn, out of line): what stays the same over the positions, and
  // its logit, loaded a position ahead
  auto named_id = [&](int e) { return e < nd ? d_ids[e] : b_ids[e - nd]; };
  auto bias_of = [&](int id) {
    float y = 0.0f;
    for (int j = 0; j < nb; ++j)
      if (b_ids[j] == id) y += b_vals[j];
    return y;
  };
  auto drafts_of = [&](int id, int i) {
    int n = 0;
    for (int j = 0; j < nd; ++j) n += d_ids[j] == id && d_pos[j] < i;
    return n;
  };
  const bool mine = tid < named;
  const int id = mine ? named_id(tid) : 0;
  int n0 = 0;
  bool seen0 = false;
  float bias = 0.0f;
  T l0 = {};
  uint32_t word0 = ~0u;
  auto load_named = [&](int i) {
    if (!mine) return;
    const uint32_t* m = allowed(i);
    l0 = logits(i)[id];
    if (m) word0 = __ldg(m + (id >> 5));
  };
  if (mine) {
    if (counts) n0 = __ldg(counts + id);
    if (prompt) seen0 = bit(prompt, id);
    bias = bias_of(id);
  }
  load_named(i0);

  for (int i = i0; i < i1; ++i) {
    float* out = a.out + b * a.o_b + i * a.o_i;
    const uint32_t* m = allowed(i);
    float value = -INFINITY;
    if (mine && ((word0 >> (id & 31)) & 1u)) value = penalise(to_f32(l0), n0 + drafts_of(id, i), seen0, w) + bias;
    for (int e = tid + kLT; e < named; e += kLT) {
      const int v = named_id(e);
      float y = penalise(to_f32(logits(i)[v]), (counts ? __ldg(counts + v) : 0) + drafts_of(v, i),
                         prompt && bit(prompt, v), w) + bias_of(v);
      more_vals[e - kLT] = !m || bit(m, v) ? y : -INFINITY;
    }
    RawT next[kLoads] = {};
    uint32_t next_ok[kMasks] = {};
    if (i + 1 < i1) {
      load(i + 1, next, next_ok);
      load_named(i + 1);
    }
    // out may be logits: every read of a named one comes before the writes
    if (named) __syncthreads();
    // ---- all of the chunk
#pragma unroll
    for (int k = 0; k < kLoads; ++k) {
      const int v = place(k * kStep);
      float y[kStep];
      widen<T>(x[k], y);
      const uint32_t may = VEC ? ok[k] >> (v & 31) : __shfl_sync(0xffffffffu, ok[0], k) >> lane;
#pragma unroll
      for (int e = 0; e < kStep; ++e) {
        const int n = k * kStep + e;
        if ((seen >> n) & 1u) y[e] = y[e] > 0.0f ? y[e] * w.inv_r : y[e] * w.r;
        y[e] = (may >> e) & 1u ? y[e] - off[n] : -INFINITY;
      }
      if (v >= v1) continue;
      if constexpr (VEC)
        *reinterpret_cast<float4*>(out + v) = make_float4(y[0], y[1], y[2], y[3]);
      else
        out[v] = y[0];
    }
    // ---- the named ones over it
    if (named) {
      __syncthreads();
      if (mine) out[id] = value;
      for (int e = tid + kLT; e < named; e += kLT) out[named_id(e)] = more_vals[e - kLT];
    }
#pragma unroll
    for (int k = 0; k < kLoads; ++k) x[k] = next[k];
#pragma unroll
    for (int k = 0; k < kMasks; ++k) ok[k] = next_ok[k];
  }

  if (!further) return;
  for (int e0 = bias0 + kWin; e0 < bias1; e0 += kWin) {
    __syncthreads();
    nb = gather(e0, min(bias1, e0 + kWin));
    for (int e = tid; e < nb; e += kLT) {
      // the first entry of an id adds all of them
      bool first = true;
      for (int j = 0; j < e; ++j) first = first && b_ids[j] != b_ids[e];
      if (!first) continue;
      for (int i = i0; i < i1; ++i) {
        // what is not allowed stays -infinity, whatever would be added
        const uint32_t* m = allowed(i);
        if (m && !bit(m, b_ids[e])) continue;
        float* out = a.out + b * a.o_b + i * a.o_i;
        float y = out[b_ids[e]];
        for (int j = e; j < nb; ++j)
          if (b_ids[j] == b_ids[e]) y += b_vals[j];
        out[b_ids[e]] = y;
      }
    }
  }
}

template <typename T, bool VEC>
int launch(const LogitsArgs& a, cudaStream_t s) {
  // several positions a block once there are blocks enough for every SM
  const int chunks = ceil_div(a.V, kLC);
  const int per = min(a.G, max(1, ceil_div(chunks * a.B * a.G, kBlocks)));
  return launch_pdl(logits_adjust_kernel<T, VEC>, dim3(chunks, a.B * ceil_div(a.G, per)), dim3(kLT), 0, s, a, per);
}

template <typename T>
int launch_type(const LogitsArgs& a, cudaStream_t s) {
  auto on = [](const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; };
  const bool vec = a.V % 4 == 0 && a.l_b % 4 == 0 && a.l_i % 4 == 0 && a.o_b % 4 == 0 && a.o_i % 4 == 0 &&
                   on(a.logits, 4 * sizeof(T)) && on(a.out, 16) && on(a.r.counts, 16);
  return vec ? launch<T, true>(a, s) : launch<T, false>(a, s);
}

}  // namespace

int launch_logits_adjust(const LogitsArgs& a, int type, cudaStream_t s) {
  if (type == DFLASH_TYPE_F32) return launch_type<float>(a, s);
  if (type == DFLASH_TYPE_BF16) return launch_type<__nv_bfloat16>(a, s);
  return launch_type<__half>(a, s);
}

}  // namespace dfl

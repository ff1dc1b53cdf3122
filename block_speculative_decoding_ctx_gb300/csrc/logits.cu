// Penalties, biases and token masks on the logits of a block
// (dflash_logits_adjust; the rules are in include/dflash.h).
//
// One block of 256 threads adjusts a chunk of 4,096 logits of one (request,
// position).  Every logit is read and written once; counts and prompt bits are
// shared by the positions of a request and come from L2 after the first.  The
// few tokens that a rule names by id (drafts before the position, biases) are
// collected per chunk, in list order, and applied to the chunk in shared
// memory; a chunk that holds none, most of them, goes from registers to the
// output.
#include "paged_util.cuh"

namespace dfl {
namespace {

constexpr int kLT = 256;       // threads
constexpr int kLC = 4096;      // logits per block
constexpr int kLI = kLC / kLT / 4;

template <typename T>
__device__ __forceinline__ float to_f32(T x);
template <>
__device__ __forceinline__ float to_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 x) { return __bfloat162float(x); }
template <>
__device__ __forceinline__ float to_f32<__half>(__half x) { return __half2float(x); }

struct Penalty {
  float r, f, p;
};

__device__ __forceinline__ float penalise(float l, int c, bool prompt, const Penalty& w) {
  if (c > 0 || prompt) l = l > 0.0f ? __fdiv_rn(l, w.r) : l * w.r;
  return l - (w.f * (float)c + (c > 0 ? w.p : 0.0f));
}

template <typename T>
__global__ void __launch_bounds__(kLT) logits_adjust_kernel(const LogitsArgs a) {
  pdl_enter();
  __shared__ float buf[kLC];
  __shared__ int ids[kLT], warp_n[kLT / 32];
  __shared__ float vals[kLT];
  const int tid = threadIdx.x, lane = tid & 31;
  const int row = blockIdx.y, b = row / a.G, i = row - b * a.G;
  const int v0 = blockIdx.x * kLC, v1 = min(a.V, v0 + kLC);
  const int words = (a.V + 31) / 32;
  const T* l = static_cast<const T*>(a.logits) + b * a.l_b + i * a.l_i;
  float* out = a.out + b * a.o_b + i * a.o_i;

  int slot = a.r.req_slot ? __ldg(a.r.req_slot + b) : b;
  const bool slot_ok = slot >= 0 && slot < a.r.slots;
  if (!slot_ok && (a.r.counts || a.r.prompt_mask) && tid == 0) report_status(a.status, DFLASH_ERR_ARG);
  if (!slot_ok) slot = 0;
  const int32_t* counts = a.r.counts && slot_ok ? a.r.counts + (size_t)slot * a.V : nullptr;
  const int32_t* prompt = a.r.prompt_mask && slot_ok ? a.r.prompt_mask + (size_t)slot * words : nullptr;
  const int32_t* allow = a.r.allow ? a.r.allow + (size_t)row * words : nullptr;
  const int32_t* draft = a.r.draft ? a.r.draft + (size_t)b * (a.G - 1) : nullptr;
  const Penalty w = {a.r.repetition ? __ldg(a.r.repetition + b) : 1.0f, a.r.frequency ? __ldg(a.r.frequency + b) : 0.0f,
                     a.r.presence ? __ldg(a.r.presence + b) : 0.0f};
  int bias0 = 0, bias1 = 0;
  if (a.r.bias_start) {
    bias0 = __ldg(a.r.bias_start + b);
    bias1 = __ldg(a.r.bias_start + b + 1);
    if (bias0 < 0 || bias1 < bias0 || bias1 > a.r.n_bias) {
      if (tid == 0) report_status(a.status, DFLASH_ERR_ARG);
      bias0 = bias1 = 0;
    }
  }
  auto bit = [&](const int32_t* m, int v) { return ((__ldg(m + (v >> 5)) >> (v & 31)) & 1) != 0; };

  for (int v = v0 + tid; v < v1; v += kLT)
    buf[v - v0] = penalise(to_f32(l[v]), counts ? __ldg(counts + v) : 0, prompt && bit(prompt, v), w);
  __syncthreads();

  // drafts before this position: their tokens again, with the larger count
  if (draft && tid < i) {
    const int d = __ldg(draft + tid);
    if (d >= v0 && d < v1) {
      int c = counts ? __ldg(counts + d) : 0;
      bool first = true;
      for (int j = 0; j < i; ++j) {
        const bool same = __ldg(draft + j) == d;
        c += same;
        if (same && j < tid) first = false;
      }
      if (first) buf[d - v0] = penalise(to_f32(l[d]), c, true, w);
    }
  }
  __syncthreads();

  // biases, 256 list entries at a time: those of this chunk in list order
  for (int e0 = bias0; e0 < bias1; e0 += kLT) {
    const int e = e0 + tid;
    int id = -1;
    if (e < bias1) {
      id = __ldg(a.r.bias_ids + e);
      if ((id < 0 || id >= a.V) && blockIdx.x == 0) report_status(a.status, DFLASH_ERR_ARG);
    }
    const bool here = id >= v0 && id < v1;
    const unsigned ball = __ballot_sync(0xffffffffu, here);
    if (lane == 0) warp_n[tid >> 5] = __popc(ball);
    __syncthreads();
    int at = 0, n = 0;
#pragma unroll
    for (int k = 0; k < kLT / 32; ++k) {
      at += k < (tid >> 5) ? warp_n[k] : 0;
      n += warp_n[k];
    }
    if (here) {
      at += __popc(ball & ((1u << lane) - 1));
      ids[at] = id;
      vals[at] = __ldg(a.r.bias_vals + e);
    }
    __syncthreads();
    if (tid < n) {
      // the first entry of an id adds all of them
      bool first = true;
      for (int j = 0; j < tid; ++j) first = first && ids[j] != ids[tid];
      if (first) {
        float x = buf[ids[tid] - v0];
        for (int j = tid; j < n; ++j)
          if (ids[j] == ids[tid]) x += vals[j];
        buf[ids[tid] - v0] = x;
      }
    }
    __syncthreads();
  }

  for (int v = v0 + tid; v < v1; v += kLT) out[v] = !allow || bit(allow, v) ? buf[v - v0] : -INFINITY;
}

template <typename T>
int launch(const LogitsArgs& a, cudaStream_t s) {
  return launch_pdl(logits_adjust_kernel<T>, dim3(ceil_div(a.V, kLC), a.B * a.G), dim3(kLT), 0, s, a);
}

}  // namespace

int launch_logits_adjust(const LogitsArgs& a, int type, cudaStream_t s) {
  if (type == DFLASH_TYPE_F32) return launch<float>(a, s);
  if (type == DFLASH_TYPE_BF16) return launch<__nv_bfloat16>(a, s);
  return launch<__half>(a, s);
}

}  // namespace dfl

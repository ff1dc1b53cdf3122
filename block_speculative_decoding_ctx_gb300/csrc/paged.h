// Internal interface of the paged-cache operators (paged_cache.cu,
// paged_attention.cu) and of the logit adjustment (logits.cu).
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "dflash.h"

namespace dfl {

// Requests of a call as the kernels see them (see dflash_paged_batch).
struct PagedBatch {
  const int32_t* row_start;
  const int64_t* kv_len;
  const int32_t* table;
  long long table_stride;
  int B, max_pages, rows;
  int n_pages, page_shift;  // page_size = 1 << page_shift
};

struct PagedMoveArgs {
  PagedBatch batch;
  uint8_t* pages[2];     // K, V
  float* scale[2];
  long long page_stride[2];
  uint8_t* x[2];         // the row tensors
  long long row_stride[2], head_stride[2];
  int n_kv;
  int* status;
};

int launch_paged_append(const PagedMoveArgs& a, int head_dim, int format, int type, cudaStream_t s);
int launch_paged_gather(const PagedMoveArgs& a, int head_dim, int format, int type, cudaStream_t s);

// What dflash_paged_maps holds.
struct PagedMaps {
  dflash_paged_cache cache;  // with maps = nullptr
  CUtensorMap k, v;
};
static_assert(sizeof(PagedMaps) <= sizeof(dflash_paged_maps), "opaque size");

int encode_paged_maps(const dflash_paged_cache& c, CUtensorMap* k, CUtensorMap* v);

struct PagedAttnArgs {
  PagedBatch batch;
  const float* k_scale;
  const float* v_scale;
  const uint8_t* q;
  uint8_t* out;
  long long q_row, q_head, o_row, o_head;
  float* lse;
  int n_q, n_kv, group, max_rows;
  int causal, window;
  float scale_log2;  // scale * log2(e)
  int* status;
};

size_t paged_attention_workspace(int n_q, int n_kv, int head_dim, int max_rows);
int launch_paged_attention(const CUtensorMap& k, const CUtensorMap& v, const PagedAttnArgs& a, int head_dim,
                           int format, int type, void* workspace, cudaStream_t s);

struct LogitsArgs {
  const void* logits;
  float* out;
  long long l_b, l_i, o_b, o_i;
  int B, G, V;
  dflash_logit_rules r;
  int* status;
};

int launch_logits_adjust(const LogitsArgs& a, int type, cudaStream_t s);

}  // namespace dfl

// Host-side interface of the paged key-value cache: tables, rotary append, decode attention.
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "../../include/tpx.h"

namespace tpx {

struct TablesArgs {
  const int32_t *lens, *add, *free_pages, *head;
  int32_t *table, *lens_out, *cu_rows, *positions, *slots, *counts;
  int32_t M, n_free, rows;
  int32_t page_shift, n_pages, max_pages, table_stride;
};
cudaError_t launch_paged_tables(const TablesArgs& a, cudaStream_t st);

struct RopeArgs {
  tp_rope rope;  // rot_dim 0: nothing is turned
  const __nv_bfloat16* qkv;
  const int32_t *positions, *slots;
  const float *k_scale, *v_scale;
  __nv_bfloat16* q_out;  // heads in order; for launch_rope: the whole qkv, in the order it came
  void *k_pages, *v_pages;
  int32_t M, t, n_q, n_kv, hd;
  int32_t page_shift, n_pages;
  unsigned* counters;  // launch_rope_append: the attention workspace's, to be zeroed, or nullptr
};
cudaError_t launch_rope(const RopeArgs& a, cudaStream_t st);
cudaError_t launch_rope_append(const RopeArgs& a, int kv_dtype, cudaStream_t st);

struct PagedAttnArgs {
  const __nv_bfloat16* q;
  const float *k_scale, *v_scale;  // e4m3 pages: [n_kv], or nullptr
  const int32_t *table, *lens;
  __nv_bfloat16* o;
  float* lse;    // or nullptr
  unsigned* ws;  // counters, then the pieces
  unsigned* err;
  int32_t M, t, n_q, n_kv, window;
  int32_t page_shift, n_pages, max_pages, table_stride;
  float scale;
};
// the largest grid
constexpr int kPagedMaxCtas = 256;
// counter words at the front of the workspace, zero between calls
constexpr int kPagedCounters = 4 * kPagedMaxCtas;
size_t paged_attn_workspace_bytes(int G, int hd);
cudaError_t launch_paged_attn(const PagedAttnArgs& a, int kv_dtype, int hd, const void* k_pages, const void* v_pages,
                              cudaStream_t st);

struct LogprobsArgs {
  const float* logits;
  int64_t ldl;
  const int32_t* ids;
  float *logprob, *entropy, *top_logprob;
  int32_t *rank, *top_id;
  int32_t M, vocab, k;
};
cudaError_t launch_token_logprobs(const LogprobsArgs& a, cudaStream_t st);

// Launch with programmatic dependent launch allowed: the kernel must wait for the work before it
// (griddepcontrol.wait) before it reads or writes anything that work may touch.
template <class K, class... A>
cudaError_t launch_dependent(K kernel, dim3 grid, dim3 block, size_t smem, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace tpx

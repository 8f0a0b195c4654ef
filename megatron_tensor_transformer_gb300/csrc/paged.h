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

// Requests that share prefixes.  What a request attends to is split between its group and itself; the parts are sum p v,
// their reference and sum p (0: nothing counted, and the other two may hold anything).
struct GroupedAttnArgs : PagedAttnArgs {
  const int32_t *cu_groups, *prefix_lens;
  int32_t n_groups;
  const uint8_t *k_pages, *v_pages;
  float *part_o, *part_ref, *part_l;  // the requests' own, where not split: [M, n_q, hd], [M, n_q] twice
  long long* own_plan;                // units of all requests, CTAs, each request's first unit: for the join
  float* own_pieces;                  // [2 kTailMaxCtas][own_piece]: [G][hd], [G] twice
  int32_t own_piece;
};
constexpr int kTailMaxCtas = 480;
constexpr int kTailEnds = 2;  // a run's beginning and end, in stages
// positions of a stage: 16 KB of k, and of v
constexpr int tail_positions(int hd, bool fp8) {
  const int n = 16384 / (hd * (fp8 ? 1 : 2));
  return n < 128 ? n : 128;
}
// launched behind launch_prefix_attn's first kernel, for whose end it does not wait before its own; that one has to begin
// after all work that this one reads or overwrites
cudaError_t launch_tail_attn(const GroupedAttnArgs& a, int kv_dtype, int hd, cudaStream_t st);
// What groups share, the requests' own positions, and the two joined: three launches.  a: with groups and pages set; ws:
// prefix_attn_workspace_bytes.
size_t prefix_attn_workspace_bytes(int n_q, int n_kv, int hd, int M);
cudaError_t launch_prefix_attn(const GroupedAttnArgs& a, int kv_dtype, int hd, cudaStream_t st);

struct LogprobsArgs {
  const float* logits;
  int64_t ldl;
  const int32_t* ids;
  float *logprob, *entropy, *top_logprob;
  int32_t *rank, *top_id;
  int32_t M, vocab, k;
};
cudaError_t launch_token_logprobs(const LogprobsArgs& a, cudaStream_t st);

struct SampleArgs {
  const float* logits;
  int64_t ldl;
  const float *u, *temperature, *top_p, *min_p;  // all but u may be nullptr
  const int32_t* top_k;
  int32_t* ids;
  float* logprob;  // or nullptr
  int32_t M, vocab;
};
constexpr int kSampleMaxVocab = 1 << 19;  // 2^19 weights of at most 2^44 sum below 2^64
cudaError_t launch_sample_tokens(const SampleArgs& a, cudaStream_t st);

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

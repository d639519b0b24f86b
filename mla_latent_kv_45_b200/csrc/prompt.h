// Internal launch interfaces of the prompt operators: cache append of packed
// rows, cache gather and causal attention over packed sequences.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "common.cuh"

namespace mla {

// Element (t, h, i) of a packed [tokens][heads][width] tensor at
// ptr + t * token + h * head + i (strides in elements).
struct HeadsView {
  const void *ptr;
  int64_t token, head;
};

struct PromptAppendArgs {
  const void *x;  // [n_tokens][d_c + d_rope], rows x_stride elements apart
  int64_t x_stride;
  const void *gamma;
  const int32_t *cu, *ctx;  // ctx == nullptr: all zero
  int batch, n_tokens, n_heads, d_c;
  HeadsView q, q_out;  // q.ptr == nullptr: no queries
  void *pool;
  const int32_t *block_table;
  int num_pages, page_size, max_pages;
  double eps;
  int *err;
};

cudaError_t launch_prompt_append_f32(const PromptAppendArgs &a, const RopeParams &rp,
                                     cudaStream_t s);
// bf16, d_c = 512, d_rope = 64; native or 656-byte int8 rows
cudaError_t launch_prompt_append_bf16(const PromptAppendArgs &a, const RopeParams &rp,
                                      bool int8_rows, cudaStream_t s);

struct GatherArgs {
  const void *pool;
  const int32_t *block_table, *cu, *first;  // first == nullptr: all zero
  int batch, n_rows, num_pages, page_size, max_pages;
  void *rows;
  int *err;
};

cudaError_t launch_gather_f32(const GatherArgs &a, int row, cudaStream_t s);
cudaError_t launch_gather_bf16(const GatherArgs &a, bool int8_rows, cudaStream_t s);

// One block of query rows of one sequence (every head of it is computed).
struct PromptItem {
  int q0;    // first token in the packed queries
  int rows;  // tokens of the block
  int k0;    // first key of the sequence in the packed keys
  int lk;    // keys of the sequence
  int see;   // keys that the block's first token sees (may be <= 0); row r sees see + r
  int pad[3];
};

struct PromptPlanHeader {
  int items;
  int next;  // work counter of the attention kernel
};

struct PromptPlanArgs {
  const int32_t *cu_q, *cu_k;
  int batch, n_q, n_k, tile;
  PromptPlanHeader *hdr;
  PromptItem *items;  // [prompt_max_items(n_q, batch, tile)]
  int *err;
};

// Blocks of at most `tile` rows that sequences of n_q tokens in all can have.
inline long prompt_max_items(long n_q, long batch, int tile) { return n_q / tile + batch; }

cudaError_t launch_prompt_plan(const PromptPlanArgs &a, cudaStream_t s);

struct PromptAttnArgs {
  HeadsView q_nope, q_rope, k_nope, v;
  const void *k_rope;
  int64_t k_rope_stride;
  int n_q, n_k, n_heads, n_kv_heads, d_nope, d_rope, d_v;
  long max_items;
  float scale;
  PromptPlanHeader *hdr;
  const PromptItem *items;
  void *out;   // [n_q][n_heads][d_v]
  float *lse;  // [n_q][n_heads] or nullptr
  int *err;
};

constexpr int kPromptTileSimt = 16;
constexpr int kPromptTileSm100 = 256;

template <class T>
cudaError_t launch_prompt_attn_simt(const PromptAttnArgs &a, cudaStream_t s);

namespace sm100 {
// bf16, d_nope = d_v = 128, d_rope = 64, items of at most kPromptTileSm100 rows
cudaError_t launch_prompt_attn(const PromptAttnArgs &a, cudaStream_t s);
}  // namespace sm100

}  // namespace mla

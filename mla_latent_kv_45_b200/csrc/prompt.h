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
  bool x_f32;     // x is fp32 (always with fp32 dims)
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
  int part;  // -1, or the partial result that this range of the block's keys fills
};

// A block whose keys were cut into pieces: partial results first .. first + pieces - 1
// (of every pack of heads) make up its rows.
struct PromptJoin {
  int q0, tokens, first, pieces;   // pieces == 0: nothing to join
  int see;   // keys that the block's first token sees (may be <= 0); row r sees see + r
};

// The attention kernel's work counter, and the CTAs that are through with it: the
// last one sets both back to zero, which mla_workspace_init has them start at.
struct PromptPlanHeader {
  int items;
  int next;
  unsigned done;
};

// Multiprocessors of a B200, where a rule counts them.
constexpr int kPromptSms = 148;
// Partial results of a call, one for each CTA at most.
constexpr int kPromptParts = kPromptSms;

struct PromptPlanArgs {
  const int32_t *cu_q, *cu_k;
  int batch, n_q, n_k, tile;
  int few_tokens;     // sequences of so many tokens at most have no items (0: all have)
  int max_items;      // prompt_max_items(n_q, batch, tile); offsets that overlap could ask for more
  PromptPlanHeader *hdr;
  PromptItem *items;  // [max_items]
  int *err;
};

// Blocks of at most `tile` rows that sequences of n_q tokens in all can have.
inline long prompt_max_items(long n_q, long batch, int tile) { return n_q / tile + batch; }

cudaError_t launch_prompt_plan(const PromptPlanArgs &a, cudaStream_t s);

// The rows of sequence b; false when its offsets do not ascend or leave the tensors.
__device__ __forceinline__ bool prompt_seq(const int32_t *cu_q, const int32_t *cu_k, int n_q,
                                           int n_k, int b, int &q0, int &lq, int &k0, int &lk) {
  q0 = cu_q[b];
  const int q1 = cu_q[b + 1];
  k0 = cu_k[b];
  const int k1 = cu_k[b + 1];
  lq = q1 - q0;
  lk = k1 - k0;
  return q0 >= 0 && q1 >= q0 && q1 <= n_q && k0 >= 0 && k1 >= k0 && k1 <= n_k;
}

// The block of at most `tile` rows that starts at row r of a sequence.
__device__ __forceinline__ PromptItem prompt_item(int q0, int lq, int k0, int lk, int r, int tile) {
  PromptItem it{};
  it.q0 = q0 + r;
  it.rows = min(tile, lq - r);
  it.k0 = k0;
  it.lk = lk;
  it.see = r + lk - lq + 1;
  it.part = -1;
  return it;
}

// Keys that the block's last row sees.
__device__ __forceinline__ int prompt_keys(const PromptItem &it) {
  return max(0, min(it.lk, it.see + it.rows - 1));
}

struct PromptAttnArgs {
  HeadsView q_nope, q_rope, k_nope, v;
  const void *k_rope;
  int64_t k_rope_stride;
  int n_q, n_k, n_heads, n_kv_heads, d_nope, d_rope, d_v;
  int pack_log2;   // sm_100a: heads of a group that share a tile (log2)
  long max_items;
  float scale;
  PromptPlanHeader *hdr;
  const PromptItem *items;
  const int32_t *cu_q, *cu_k;
  int batch;
  int few_tokens;  // sequences of so many tokens at most are left to prompt_few_kernel (0: none)
  // Keys of few blocks cut into pieces: [kPromptParts][256 rows][128], and the rows'
  // m (log2 units) and l.
  float *part_O, *part_m, *part_l;
  PromptJoin *join;  // [max_items]
  void *out;   // [n_q][n_heads][d_v]
  float *lse;  // [n_q][n_heads] or nullptr
  int *err;
  uint64_t wait_ns;  // sm_100a: limit of a wait between the kernel's warps
};

// A row that sees keys, all of them with a score of -inf, gets 0 / 0 = NaN and lse = -inf as
// the formula has it, unlike a row that sees none: each kernel asks what a row sees, not
// whether its sum is zero.
constexpr int kPromptTileSimt = 16;
constexpr int kPromptTileSm100 = 256;   // rows of an item: (token, head) pairs
constexpr int kPromptFewRows = 16;      // rows of a sequence and key head that prompt_few_kernel takes
constexpr int kPromptSplitKeys = 1024;  // fewest keys of a call whose blocks are cut into pieces
// Up to this many items the sm_100a kernel plans for itself and needs no plan kernel.
constexpr int kPromptOwnItems = 512;

// fp32
cudaError_t launch_prompt_attn_simt(const PromptAttnArgs &a, cudaStream_t s);

// bf16, d_nope = d_v = 128, d_rope = 64: the sequences of at most few_tokens tokens
cudaError_t launch_prompt_few(const PromptAttnArgs &a, cudaStream_t s);

namespace sm100 {
// bf16, d_nope = d_v = 128, d_rope = 64, items of at most kPromptTileSm100 rows
cudaError_t launch_prompt_attn(const PromptAttnArgs &a, cudaStream_t s);
}  // namespace sm100

}  // namespace mla

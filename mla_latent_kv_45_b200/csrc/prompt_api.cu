// Host side of the prompt calls declared in include/mla.h: argument checks,
// workspace layout and dispatch.  Nothing here allocates or synchronises.
#include <atomic>

#include <cuda_runtime.h>

#include "api_checks.h"
#include "common.cuh"
#include "mla.h"
#include "prompt.h"

namespace {

using namespace mla;
using api::aligned16;
using api::aligned4;

#define MLA_TRY(x)                 \
  do {                             \
    mla_status st_ = (x);          \
    if (st_ != MLA_OK) return st_; \
  } while (0)

mla_status cuda_ok(cudaError_t e) { return e == cudaSuccess ? MLA_OK : MLA_ERR_CUDA; }

// log2 of the heads that share a tile: the largest power of two that divides a
// group of `rep` query heads, 128 at most.
int pack_log2(int rep) {
  int lg = 0;
  while (lg < 7 && rep % (2 << lg) == 0) ++lg;
  return lg;
}

// Tokens of an item with groups of `rep` heads.
int tile_tokens(const mla_dims &d, int rep) {
  return d.dtype == MLA_BF16 ? kPromptTileSm100 >> pack_log2(rep) : kPromptTileSimt;
}

// ... the fewest that any grouping of the heads has.
int least_tile_tokens(const mla_dims &d) {
  int least = tile_tokens(d, 1);
  for (int rep = 2; rep <= d.n_heads; ++rep)
    if (d.n_heads % rep == 0 && tile_tokens(d, rep) < least) least = tile_tokens(d, rep);
  return least;
}

// Tokens up to which a sequence goes to the kernel for few rows (bf16; 0: that kernel is not
// launched).  The lengths are on the device only, so the average decides whether it
// is worth a launch (100 sequences of 0-8 tokens, 128 heads: 79 us, 223 without it).  Few
// blocks whose keys may be long are cut into pieces instead, from twice the keys on that
// cutting starts at.  The more heads, the later that pays (a block has fewer pieces): one
// token over 1200, 1600, 2000, 2600 and 3200 rows takes with 16 heads 14.3, 17.6, 20.8, 25.5 and
// 30.1 us here and 15.5, 15.4, 16.2, 17.8 and 18.4 cut, with 32 heads 14.6, 17.7, 21.0, 25.9 and
// 30.3 here and 15.8, 16.1, 18.0, 20.4 and 21.3 cut, with 64 heads 14.5, 17.7, 21.0, 25.9 and
// 30.6 here and 19.0, 21.1, 23.9, 28.1 and 31.3 cut.
int few_tokens(const mla_dims &d, int rep, int batch, int n_q, int n_k, long max_items) {
  if (d.dtype != MLA_BF16 || rep > kPromptFewRows) return 0;
  const int most = kPromptFewRows / rep;
  const long work = max_items * (d.n_heads >> pack_log2(rep));
  if ((long)batch * (d.n_heads / rep) > 0x7fffffffL) return 0;     // a grid's blocks
  if (n_q > (long)most * batch || (2 * work <= kPromptParts && n_k >= 2 * kPromptSplitKeys))
    return 0;
  return most;
}

// The error word and the plan header share the first 256 bytes (the part that
// mla_workspace_init clears); the plan's items follow.  The header holds counters that
// outlive a call, so it lies where no other call of the library writes: a workspace
// may serve decode and prompt calls in turn.
constexpr size_t kItemsAt = 256, kHeaderAt = 192;

constexpr size_t kPartBytes = sizeof(float) * 256 * (128 + 2);   // O, m and l of a partial result

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// bf16: bytes up to the partial results (20 MB), which small calls over long keys use.
// They are always part of the size, so that a workspace for many tokens does for few.
size_t plan_bytes(const mla_dims &d, int batch, int n_tokens) {
  return align256(kItemsAt +
                  sizeof(PromptItem) * (size_t)prompt_max_items(n_tokens, batch,
                                                                least_tile_tokens(d)));
}

size_t prompt_ws_bytes(const mla_dims &d, int batch, int n_tokens) {
  return d.dtype == MLA_BF16 ? plan_bytes(d, batch, n_tokens) + kPromptParts * kPartBytes : kItemsAt;
}

mla_status check_ws(const void *ws, size_t ws_bytes, size_t need) {
  if (!ws) return MLA_ERR_INVALID_ARG;
  if (!aligned16(ws)) return MLA_ERR_ALIGNMENT;
  return ws_bytes < need ? MLA_ERR_WORKSPACE : MLA_OK;
}

// Limit of a wait between the attention kernel's warps.  The longest one is for an item
// by the warps that write its output: a step of 80 keys takes 1.2 us, so 100 ns a key beside
// the 2 s leave a factor of six.  (0: no test hook, see mla_debug_prompt_timeout.)
std::atomic<unsigned long long> g_debug_wait_ns{0};

uint64_t wait_limit_ns(int n_k) {
  const unsigned long long d = g_debug_wait_ns.load(std::memory_order_relaxed);
  return d ? d : 2000000000ull + 100ull * (unsigned)n_k;
}

int *err_of(void *ws) { return static_cast<int *>(ws); }

mla_status check_heads(const mla_dims &d, const mla_heads *h, int tokens, int heads, int width) {
  if (!h || !h->ptr) return MLA_ERR_INVALID_ARG;
  if (!aligned16(h->ptr)) return MLA_ERR_ALIGNMENT;
  if (heads > 1 && h->head_stride < width) return MLA_ERR_INVALID_ARG;
  if (tokens > 1 && h->token_stride < width) return MLA_ERR_INVALID_ARG;
  if (d.dtype == MLA_BF16 &&
      ((heads > 1 && h->head_stride % 8) || (tokens > 1 && h->token_stride % 8)))
    return MLA_ERR_ALIGNMENT;
  return MLA_OK;
}

// Strides of an extent of one are not used; the kernels get a harmless value.
HeadsView view(const mla_heads *h, int tokens, int heads, int width) {
  HeadsView v{};
  if (!h) return v;
  v.ptr = h->ptr;
  v.token = tokens > 1 ? h->token_stride : width;
  v.head = heads > 1 ? h->head_stride : width;
  return v;
}

}  // namespace

extern "C" {

size_t mla_prompt_workspace_size(const mla_dims *dims, int batch, int n_tokens) {
  if (api::check_prompt_dims(dims) != MLA_OK || batch < 1 || n_tokens < 0) return 0;
  return prompt_ws_bytes(*dims, batch, n_tokens);
}

mla_status mla_prompt_append(const mla_dims *dims, const mla_paged_cache *cache, int batch,
                             int n_tokens, const void *x, int x_dtype, int64_t x_stride,
                             const void *gamma,
                             const int32_t *cu_tokens, const int32_t *ctx_lens,
                             const mla_heads *q_rope, const mla_heads *q_out, void *ws,
                             size_t ws_bytes, mla_stream_t stream) {
  MLA_TRY(api::check_prompt_dims(dims));
  MLA_TRY(api::check_cache(cache));
  const mla_dims &d = *dims;
  if (batch < 1 || n_tokens < 0 || !gamma || !cu_tokens || !q_rope != !q_out)
    return MLA_ERR_INVALID_ARG;
  if (x_dtype != MLA_FP32 && x_dtype != d.dtype) return MLA_ERR_INVALID_ARG;
  MLA_TRY(check_ws(ws, ws_bytes, kItemsAt));
  if (!aligned16(gamma) || !aligned4(cu_tokens) || !aligned4(ctx_lens)) return MLA_ERR_ALIGNMENT;
  if (n_tokens == 0) return MLA_OK;
  if (!x || (n_tokens > 1 && x_stride < d.d_c + d.d_rope)) return MLA_ERR_INVALID_ARG;
  if (!aligned16(x) || (d.dtype == MLA_BF16 && n_tokens > 1 && x_stride % 8))
    return MLA_ERR_ALIGNMENT;
  if (q_rope) {
    MLA_TRY(check_heads(d, q_rope, n_tokens, d.n_heads, d.d_rope));
    MLA_TRY(check_heads(d, q_out, n_tokens, d.n_heads, d.d_rope));
  }
  PromptAppendArgs a{};
  a.x = x;
  a.x_stride = x_stride;
  a.x_f32 = x_dtype == MLA_FP32;
  a.gamma = gamma;
  a.cu = cu_tokens;
  a.ctx = ctx_lens;
  a.batch = batch;
  a.n_tokens = n_tokens;
  a.n_heads = d.n_heads;
  a.d_c = d.d_c;
  a.q = view(q_rope, n_tokens, d.n_heads, d.d_rope);
  a.q_out = view(q_out, n_tokens, d.n_heads, d.d_rope);
  a.pool = cache->pool;
  a.block_table = cache->block_table;
  a.num_pages = cache->num_pages;
  a.page_size = d.page_size;
  a.max_pages = cache->max_pages_per_seq;
  a.eps = d.rms_eps;
  a.err = err_of(ws);
  const RopeParams rp = api::rope_params(d);
  cudaStream_t s = (cudaStream_t)stream;
  if (d.dtype == MLA_FP32) return cuda_ok(launch_prompt_append_f32(a, rp, s));
  return cuda_ok(launch_prompt_append_bf16(a, rp, d.cache_format == MLA_CACHE_INT8, s));
}

mla_status mla_cache_gather(const mla_dims *dims, const mla_paged_cache *cache, int batch,
                            int n_rows, const int32_t *cu_rows, const int32_t *first_rows,
                            void *rows, void *ws, size_t ws_bytes, mla_stream_t stream) {
  MLA_TRY(api::check_prompt_dims(dims));
  MLA_TRY(api::check_cache(cache));
  const mla_dims &d = *dims;
  if (batch < 1 || n_rows < 0 || !cu_rows) return MLA_ERR_INVALID_ARG;
  MLA_TRY(check_ws(ws, ws_bytes, kItemsAt));
  if (!aligned4(cu_rows) || !aligned4(first_rows)) return MLA_ERR_ALIGNMENT;
  if (n_rows == 0) return MLA_OK;
  if (!rows) return MLA_ERR_INVALID_ARG;
  if (!aligned16(rows)) return MLA_ERR_ALIGNMENT;
  GatherArgs a{};
  a.pool = cache->pool;
  a.block_table = cache->block_table;
  a.cu = cu_rows;
  a.first = first_rows;
  a.batch = batch;
  a.n_rows = n_rows;
  a.num_pages = cache->num_pages;
  a.page_size = d.page_size;
  a.max_pages = cache->max_pages_per_seq;
  a.rows = rows;
  a.err = err_of(ws);
  cudaStream_t s = (cudaStream_t)stream;
  if (d.dtype == MLA_FP32) return cuda_ok(launch_gather_f32(a, d.d_c + d.d_rope, s));
  return cuda_ok(launch_gather_bf16(a, d.cache_format == MLA_CACHE_INT8, s));
}

mla_status mla_prompt_attn(const mla_dims *dims, int batch, int n_q, int n_k, int n_kv_heads,
                           const mla_heads *q_nope, const mla_heads *q_rope,
                           const mla_heads *k_nope, const void *k_rope, int64_t k_rope_stride,
                           const mla_heads *v, const int32_t *cu_q, const int32_t *cu_k, void *out,
                           float *lse, void *ws, size_t ws_bytes, mla_stream_t stream) {
  MLA_TRY(api::check_prompt_dims(dims));
  const mla_dims &d = *dims;
  if (batch < 1 || n_q < 0 || n_k < 0 || n_kv_heads < 1 || n_kv_heads > d.n_heads || !cu_q || !cu_k)
    return MLA_ERR_INVALID_ARG;
  if (d.n_heads % n_kv_heads) return MLA_ERR_INVALID_ARG;
  if (!aligned4(cu_q) || !aligned4(cu_k) || !aligned4(lse)) return MLA_ERR_ALIGNMENT;
  MLA_TRY(check_ws(ws, ws_bytes, prompt_ws_bytes(d, batch, n_q)));
  if (n_q == 0) return MLA_OK;
  if (!out) return MLA_ERR_INVALID_ARG;
  if (!aligned16(out)) return MLA_ERR_ALIGNMENT;
  MLA_TRY(check_heads(d, q_nope, n_q, d.n_heads, d.d_nope));
  MLA_TRY(check_heads(d, q_rope, n_q, d.n_heads, d.d_rope));
  if (n_k > 0) {
    MLA_TRY(check_heads(d, k_nope, n_k, n_kv_heads, d.d_nope));
    MLA_TRY(check_heads(d, v, n_k, n_kv_heads, d.d_v));
    const mla_heads kr{const_cast<void *>(k_rope), k_rope_stride, 0};
    MLA_TRY(check_heads(d, &kr, n_k, 1, d.d_rope));
  }
  cudaStream_t s = (cudaStream_t)stream;
  PromptPlanArgs pa{};
  pa.cu_q = cu_q;
  pa.cu_k = cu_k;
  pa.batch = batch;
  pa.n_q = n_q;
  pa.n_k = n_k;
  const int rep = d.n_heads / n_kv_heads;
  pa.tile = tile_tokens(d, rep);
  pa.hdr = reinterpret_cast<PromptPlanHeader *>(static_cast<char *>(ws) + kHeaderAt);
  pa.items = reinterpret_cast<PromptItem *>(static_cast<char *>(ws) + kItemsAt);
  pa.err = err_of(ws);
  const long max_items = prompt_max_items(n_q, batch, pa.tile);
  pa.max_items = (int)max_items;
  pa.few_tokens = few_tokens(d, rep, batch, n_q, n_k, max_items);
  // (where no sequence can have more tokens, there is nothing to plan)
  const bool only_few = n_q <= pa.few_tokens;
  if (d.dtype == MLA_BF16 && max_items > kPromptOwnItems && !only_few)
    MLA_TRY(cuda_ok(launch_prompt_plan(pa, s)));
  PromptAttnArgs a{};
  a.q_nope = view(q_nope, n_q, d.n_heads, d.d_nope);
  a.q_rope = view(q_rope, n_q, d.n_heads, d.d_rope);
  if (n_k > 0) {
    a.k_nope = view(k_nope, n_k, n_kv_heads, d.d_nope);
    a.v = view(v, n_k, n_kv_heads, d.d_v);
    a.k_rope = k_rope;
    a.k_rope_stride = n_k > 1 ? k_rope_stride : d.d_rope;
  }
  a.n_q = n_q;
  a.n_k = n_k;
  a.n_heads = d.n_heads;
  a.n_kv_heads = n_kv_heads;
  a.pack_log2 = pack_log2(rep);
  a.d_nope = d.d_nope;
  a.d_rope = d.d_rope;
  a.d_v = d.d_v;
  a.max_items = max_items;
  a.cu_q = cu_q;
  a.cu_k = cu_k;
  a.batch = batch;
  a.few_tokens = pa.few_tokens;
  a.scale = api::softmax_scale(d);
  a.hdr = pa.hdr;
  a.items = pa.items;
  if (d.dtype == MLA_BF16) {
    a.part_O = reinterpret_cast<float *>(static_cast<char *>(ws) + plan_bytes(d, batch, n_q));
    a.part_m = a.part_O + (size_t)kPromptParts * 256 * 128;
    a.part_l = a.part_m + (size_t)kPromptParts * 256;
    a.join = reinterpret_cast<PromptJoin *>(pa.items);   // the plan's place, which it does not use
  }
  a.out = out;
  a.lse = lse;
  a.err = pa.err;
  a.wait_ns = wait_limit_ns(n_k);
  if (d.dtype == MLA_FP32) return cuda_ok(launch_prompt_attn_simt(a, s));
  if (a.few_tokens > 0) MLA_TRY(cuda_ok(launch_prompt_few(a, s)));
  return only_few ? MLA_OK : cuda_ok(sm100::launch_prompt_attn(a, s));
}

mla_status mla_debug_prompt_timeout(int enable, unsigned wait_limit_us) {
  if (enable && wait_limit_us == 0) return MLA_ERR_INVALID_ARG;
  g_debug_wait_ns.store(enable ? 1000ull * wait_limit_us : 0);
  return MLA_OK;
}

}  // extern "C"

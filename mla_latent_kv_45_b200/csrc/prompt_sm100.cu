// Causal attention over packed sequences on sm_100a tensor cores (bf16, scores
// over 128 + 64 values, 128-wide values).
//
// out_i = sum_j softmax_j(scale (q_nope_i . k_nope_j + q_rope_i . k_rope_j)) v_j in
// one pass over the keys with a running maximum m and sum l per row
// ("从零理解 MLA", 解耦 RoPE MLADecoupledRoPE.forward).
//
// One work item is 256 query rows: two 128-row tiles that share every key and value
// in shared memory.  A row is a (token, head) pair.  With one key head per query head
// they are 256 tokens of one head; grouped heads are packed, 2^lg heads of the group
// (the largest power of two that divides it, 128 at most) of 256 / 2^lg tokens, so a
// key head is read once for all of them and short chunks still fill a tile (4 chunks
// of 64 tokens over 2000 rows, 128 heads in 8 groups: 45 us, 113 us a head at a time).
// Per step of 80 keys a tile costs S = Q K^T (K = 192, the two score terms are one
// product) and O += P V.
//  * 80 keys a step, because TMEM then holds S (80 columns) beside P (bf16, 40
//    columns) and O (128) of both tiles: 496 of 512 columns.  A step's scores are
//    computed as soon as the previous step's have been read into registers, and
//    the products P V run while the next softmax does.  (128 keys with P in the
//    place of S: 2446 us for 8192 tokens and 128 heads, this 2253 us in the same run.)
//  * Warps 0-3 and 4-7 are the softmax of tile 0 and 1, one thread a row: no
//    reduction crosses threads.  (Two threads a row: 10 % slower.)
//  * m moves only when the maximum grows by more than 2^8 (p stays below
//    256); only then does the thread rescale O.
//  * Warps 8-11 write the output of an item through shared memory (whole rows
//    of 128 bytes) while the others are at the next one; warp 12 loads Q, K and V
//    by TMA (two stages of keys and values); warp 13 zeroes values behind a
//    sequence's last key; warps 14 and 15 issue the MMAs, one thread a tile (one
//    thread for both was the bottleneck: every wait of one tile held up the other).
//  * Work comes from a counter: the CTAs are persistent and fetch (block, head)
//    pairs, blocks with most keys first.
//  * Sequences of few rows may be left to prompt_few.cu: they have no items.
//  * Every wait is bounded (PromptAttnArgs::wait_ns); on expiry the error word is set, the
//    warps stop, and the loading warp and the MMA threads wait for what they have in flight.
//
// What bounds it: a step takes about 2180 cycles.  The MMAs read 196 KB of operands
// from shared memory in it and TMA writes 50 KB there, which at 128 bytes a cycle is
// 1920 cycles; the softmax of a tile is a chain of about 1830.  An item costs about
// 6000 cycles beside its steps (the tile with the earlier rows waits for the other).
// 8192 tokens, 128 heads: 2.03 ms by itself (1350 TFLOP/s, 83 % of the measured
// matrix rate), 2.36 ms back to back, where the power limit lowers the clock.
#include <cuda.h>

#include "api_checks.h"
#include "prompt.h"
#include "prompt_ptx.cuh"

namespace mla {
namespace sm100 {
namespace {

using namespace ptx;
using bf16 = __nv_bfloat16;

constexpr int kRows = 128;              // query rows of a tile
constexpr int kKeys = 80;               // keys of a step
constexpr int kMinSteps = 4;            // of a piece of a block's keys
constexpr int kSched = 3;               // work items in flight between the warps
constexpr int kWarpOut = 8;             // warps 8-11
constexpr int kWarpLoad = 12, kWarpFix = 13, kWarpMma = 14, kWarps = 16;   // MMA: 14, 15
constexpr int kThreads = 32 * kWarps;
constexpr uint64_t kDrainNs = 2000000000ull;   // for copies and products in flight at the end
constexpr uint32_t kSleepNs = 20000;

// Shared memory: boxes of 64 columns (128 bytes, 128-byte swizzle)
constexpr int kQBox = kRows * 128, kKBox = kKeys * 128;
constexpr int kQTile = 3 * kQBox, kKStage = 3 * kKBox, kVStage = 2 * kKBox;
constexpr int kOffQ = 0;
constexpr int kOffK = kOffQ + 2 * kQTile;
constexpr int kOffV = kOffK + 2 * kKStage;
constexpr int kOffOut = kOffV + 2 * kVStage;      // [4 output warps][32 rows][128 bytes]
constexpr int kOffInv = kOffOut + 4 * 4096;       // [2 tiles][128] 1 / row sum, then lse
constexpr int kOffBar = kOffInv + 2048;
constexpr int kOffItems = kOffBar + 1024;         // the CTA's own plan
constexpr int kSmemBytes = kOffItems + kPromptOwnItems * (int)sizeof(PromptItem);
static_assert(kKBox % 1024 == 0 && kOffOut % 1024 == 0, "swizzled boxes start on 1024 bytes");
static_assert(kSmemBytes <= 232448, "shared memory per CTA");

// TMEM columns of tile t
constexpr uint32_t kTmemO = 0, kTmemS = 256, kTmemP = 256 + 2 * kKeys, kTmemCols = 512;
static_assert(kTmemP + kKeys <= kTmemCols, "TMEM columns");
constexpr uint32_t kIdescS = idesc_bf16(kRows, kKeys, 0, 0);
constexpr uint32_t kIdescPV = idesc_bf16(kRows, 128, 0, 1);     // V is [key][column]

// One (block of rows, head) pair on its way from the loading warp to the others.
struct Work {
  PromptItem it;
  int head;   // -1: no more work
};

// Steps are counted through (g) over all items of a CTA; step g uses stage g % 2.
struct Bars {
  uint64_t k_full[2], k_free[2], v_full[2], v_free[2];
  uint64_t v_raw[2];      // values that end inside the step landed; the fixing warp fills v_full
  uint64_t q_full[2], q_empty[2];
  uint64_t s_full[2];     // scores of the tile complete
  uint64_t s_free[2];     // ... and read by its four warps
  uint64_t p_full[2];     // P written (and O rescaled) by the tile's four warps
  uint64_t pv_done[2];    // O += P V complete
  uint64_t o_full[2];     // ... for the item's last step
  uint64_t l_full[2];     // the reciprocal row sums are in shared memory
  uint64_t o_free[2];     // O and the row sums have been read
  uint64_t w_full[kSched], w_empty[kSched];
  uint64_t drain[2];
  Work work[kSched];
  uint32_t tmem_base;
  volatile int abort;
};
static_assert(sizeof(Bars) <= 1024, "barrier region");

struct Ctx {
  Bars *bars;
  int *err;
  uint64_t limit;   // of a wait, ns
};

__device__ __forceinline__ bool wait_bar(const Ctx &c, uint64_t *bar, uint32_t parity) {
  const uint32_t a = smem_u32(bar);
  if (mbar_try_wait(a, parity)) return true;
  const uint64_t t0 = globaltimer();
  while (true) {
    if (mbar_try_wait(a, parity)) return true;
    if (c.bars->abort) return false;
    if (globaltimer() - t0 > c.limit) {
      set_error(c.err, kErrTimeout);
      c.bars->abort = 1;
      return false;
    }
  }
}

// Waits (bounded, ignoring the abort flag) for asynchronous work this CTA issued.
__device__ __forceinline__ void drain_bar(uint64_t *bar, uint32_t parity) {
  const uint32_t a = smem_u32(bar);
  const uint64_t t0 = globaltimer();
  while (!mbar_try_wait_sleep(a, parity, kSleepNs))
    if (globaltimer() - t0 > kDrainNs) return;
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}

// 8 words of P: the weights 2^(scale v - m) of 16 columns, added to the row sum
// unrounded.  They are rounded to bf16 because both operands of the product with V have one
// type and V is bf16: each is off by 2^-8 of itself at most, which leaves the result
// 1.2-1.4x as far from 64 bits as weights in 32 bits do (2.0e-3 against 1.5e-3 for 8192 tokens,
// most of both the rounding of the result).  A second bf16 term for the remainder would
// double the product, 40 % of a step's MMAs.  (Part of the exponentials on the FMA pipe
// instead of the special-function unit made the kernel slower at every share: it is short
// of issue slots, not of that unit.)
__device__ __forceinline__ void weights16(const float *v, uint64_t scale2, uint64_t base2,
                                          uint64_t (&sum)[2], uint32_t *p) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint64_t x = f2_fma(f2_pack(v[2 * i], v[2 * i + 1]), scale2, base2);
    float a, b;
    f2_unpack(x, a, b);
    a = ex2(a);
    b = ex2(b);
    sum[i & 1] = f2_add(sum[i & 1], f2_pack(a, b));
    p[i] = pack2(a, b);
  }
}

// Tokens of tile t of an item (a tile has 128 >> lg of them, each with 1 << lg heads),
// and the steps that its last token's keys take.
__device__ __forceinline__ int tile_tokens(const PromptItem &it, int t, int lg) {
  const int tt = kRows >> lg;
  return max(0, min(tt, it.rows - t * tt));
}
__device__ __forceinline__ int tile_steps(const PromptItem &it, int t, int lg) {
  const int toks = tile_tokens(it, t, lg);
  if (toks == 0) return 0;
  const int keys = max(0, min(it.lk, it.see + t * (kRows >> lg) + toks - 1));
  return (keys + kKeys - 1) / kKeys;
}

// Plan of the whole call by one CTA for itself, the same in every CTA: item i of the
// list is the block with the i-th most keys (ties by sequence and block), so the
// blocks that take longest start first.  A thread a sequence, then a thread an item;
// the rank is counted (items^2 / 512 comparisons a thread).  A launch of its own
// would cost about 6 us, this takes about 1.  Returns the number of items.
//
// split: there are fewer blocks than half the CTAs, so their keys are cut into as many
// pieces as there are CTAs for, by their number of steps (at least kMinSteps a
// piece).  A piece is an item of its own whose keys are a range of the block's; it
// leaves an unnormalised result that the join kernel merges.
// `scratch`: 12.4 KB of shared memory.
__device__ __forceinline__ int own_plan(const PromptAttnArgs &a, PromptItem *list, int *scratch,
                                        bool split) {
  static_assert(kThreads == kPromptOwnItems, "a thread an item");
  int *first = scratch;          // [512] items before the sequence
  int *keys = first + 512;       // [512] of item i, before sorting
  int *warp_tot = keys + 512;    // [16]
  int4 *seq = reinterpret_cast<int4 *>(warp_tot + 16);   // [512] q0, lq, k0, lk
  const int tid = threadIdx.x, lane = tid & 31, tile = kPromptTileSm100 >> a.pack_log2;
  int q0, lq, k0, lk, n = 0;
  if (tid < a.batch) {
    if (prompt_seq(a.cu_q, a.cu_k, a.n_q, a.n_k, tid, q0, lq, k0, lk))
      n = lq > a.few_tokens ? (lq + tile - 1) / tile : 0;
    else if (blockIdx.x == 0)
      set_error(a.err, kErrRange);
    seq[tid] = make_int4(q0, lq, k0, lk);
  }
  int v = n;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += x;
  }
  if (lane == 31) warp_tot[tid >> 5] = v;
  __syncthreads();
  int before = 0, items = 0;
#pragma unroll
  for (int i = 0; i < kWarps; ++i) {
    before += i < (tid >> 5) ? warp_tot[i] : 0;
    items += warp_tot[i];
  }
  items = min(items, (int)a.max_items);   // offsets that overlap could ask for more
  first[tid] = before + v - n;
  __syncthreads();
  PromptItem it{};
  int mine = -1;
  if (tid < items) {
    int b = 0;      // the last sequence that starts at item tid or before and is not empty
#pragma unroll
    for (int step = kPromptOwnItems / 2; step > 0; step >>= 1)
      if (b + step < a.batch && first[b + step] <= tid) b += step;
    const int4 x = seq[b];
    it = prompt_item(x.x, x.y, x.z, x.w, (tid - first[b]) * tile, tile);
    mine = prompt_keys(it);
  }
  keys[tid] = mine;
  __syncthreads();
  if (split) {
    // (items <= max_items <= 74 and 148 pieces at most beside them fit the list)
    const int steps = (max(mine, 0) + kKeys - 1) / kKeys, packs = a.n_heads >> a.pack_log2;
    int all = 0;
    for (int i = 0; i < items; ++i) all += (keys[i] + kKeys - 1) / kKeys;
    auto pieces = [&](int st) {
      const int most = min(st / kMinSteps, (int)((long)st * kPromptParts / (max(all, 1) * packs)));
      return max(1, most);
    };
    int at = 0, part = 0, n = 0;
    for (int i = 0; i < items; ++i) {
      const int c = pieces((keys[i] + kKeys - 1) / kKeys);
      at += i < tid ? c : 0;
      part += i < tid && c > 1 ? c : 0;
      n += c;
    }
    if (tid < items) {
      const int c = pieces(steps);
      for (int i = 0; i < c; ++i) {
        const int s0 = (int)((long)steps * i / c), s1 = (int)((long)steps * (i + 1) / c);
        PromptItem x = it;
        if (c > 1) {
          x.k0 += s0 * kKeys;
          x.lk = min(it.lk - s0 * kKeys, (s1 - s0) * kKeys);
          x.see -= s0 * kKeys;
          x.part = part + i;
        }
        list[at + i] = x;
      }
      // (a block that is cut has keys: what a row sees is bounded by `see` alone)
      if (blockIdx.x == 0)
        a.join[tid] = PromptJoin{it.q0, it.rows, part, c > 1 ? c : 0, it.see};
    }
    if (blockIdx.x == 0 && tid >= items && tid < a.max_items) a.join[tid] = PromptJoin{};
    __syncthreads();
    return n;
  }
  if (tid < items) {
    int rank = 0;
    for (int i = 0; i < items; ++i) rank += keys[i] > mine || (keys[i] == mine && i < tid);
    list[rank] = it;
  }
  __syncthreads();
  return items;
}

__global__ void __launch_bounds__(kThreads, 1)
    prompt_attn_kernel(const __grid_constant__ CUtensorMap tm_qn,
                       const __grid_constant__ CUtensorMap tm_qr,
                       const __grid_constant__ CUtensorMap tm_kn,
                       const __grid_constant__ CUtensorMap tm_kr,
                       const __grid_constant__ CUtensorMap tm_v, const PromptAttnArgs a,
                       const float scale_log2, const int heads_per_group,
                       const bool split) {
  extern __shared__ __align__(1024) uint8_t smem[];
  Bars *bars = reinterpret_cast<Bars *>(smem + kOffBar);
  const Ctx ctx{bars, a.err, a.wait_ns};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int lg = a.pack_log2, tt = kRows >> lg;   // heads a token has in a tile, tokens of a tile

  const bool own = a.max_items <= kPromptOwnItems;    // (a.batch is not above a.max_items)
  if (a.few_tokens > 0) {
    // The other kernel may have taken every sequence: nothing is set up then.
    grid_dep_wait();
    const int b = threadIdx.x;
    const bool some = own ? b < a.batch && a.cu_q[b + 1] - a.cu_q[b] > a.few_tokens
                          : a.hdr->items > 0;
    if (!__syncthreads_or(some)) {
      grid_dep_launch();
      if (split && blockIdx.x == 0 && b < a.max_items) a.join[b] = PromptJoin{};
      return;
    }
  }

  // The swizzled boxes need a 1024-byte boundary, which the dynamic shared memory
  // starts on (there is no static part in front of it).
  if (smem_u32(smem) & 1023) {
    if (threadIdx.x == 0) set_error(a.err, kErrTimeout);
    return;
  }
  if (threadIdx.x == 0) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(&bars->k_full[t], 1);
      mbar_init(&bars->k_free[t], 2);   // both tiles
      mbar_init(&bars->v_full[t], 1);
      mbar_init(&bars->v_free[t], 2);
      mbar_init(&bars->v_raw[t], 1);
      mbar_init(&bars->q_full[t], 1);
      mbar_init(&bars->q_empty[t], 1);
      mbar_init(&bars->s_full[t], 1);
      mbar_init(&bars->s_free[t], 4);
      mbar_init(&bars->p_full[t], 4);
      mbar_init(&bars->pv_done[t], 1);
      mbar_init(&bars->o_full[t], 1);
      mbar_init(&bars->l_full[t], 4);
      mbar_init(&bars->o_free[t], 4);
    }
    for (int i = 0; i < kSched; ++i) {
      mbar_init(&bars->w_full[i], 1);
      mbar_init(&bars->w_empty[i], 15);   // eight softmax, four output warps, two MMA, fixing
    }
    mbar_init(&bars->drain[0], 1);
    mbar_init(&bars->drain[1], 1);
    bars->abort = 0;
    fence_mbar_init();
  }
  if (warp == kWarpLoad && lane == 0) {
    prefetch_tmap(&tm_qn);
    prefetch_tmap(&tm_qr);
    prefetch_tmap(&tm_kn);
    prefetch_tmap(&tm_kr);
    prefetch_tmap(&tm_v);
  }
  if (warp == kWarpMma) {
    tmem_alloc(&bars->tmem_base, kTmemCols);
    tc_fence_before();
  }
  __syncwarp();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem_base;
  grid_dep_wait();     // nothing of the call is read before this
  grid_dep_launch();
  PromptItem *const own_items = reinterpret_cast<PromptItem *>(smem + kOffItems);
  const int items = own ? own_plan(a, own_items, reinterpret_cast<int *>(smem + kOffOut), split)
                        : a.hdr->items;

  // the k-th work item of this CTA, as a whole warp reads it
  auto take = [&](int k, Work &w) -> bool {
    const int slot = k % kSched;
    bool ok = wait_bar(ctx, &bars->w_full[slot], (k / kSched) & 1);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) return false;
    w = bars->work[slot];
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars->w_empty[slot]);
    return w.head >= 0;
  };
  auto wait_all = [&](uint64_t *bar, uint32_t parity) -> bool {   // by a whole warp
    return __all_sync(0xffffffffu, wait_bar(ctx, bar, parity));
  };

  if (warp < 8) {
    // ------------------------------------------------ softmax, one thread a row
    const int t = warp >> 2;
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_addr = tmem + lane_off + kTmemS + kKeys * t;
    const uint32_t p_addr = tmem + lane_off + kTmemP + kKeys / 2 * t;
    const uint32_t o_addr = tmem + lane_off + kTmemO + 128 * t;
    float *inv_s = reinterpret_cast<float *>(smem + kOffInv) + 128 * t;
    const uint64_t scale2 = f2_pack(scale_log2, scale_log2);
    int ns = 0, ni = 0;      // steps and items (with keys) of this tile so far
    bool ok = true;
    Work w;
    for (int k = 0; ok && take(k, w); ++k) {
      const int steps = tile_steps(w.it, t, lg);
      if (steps == 0) continue;
      const int see = max(0, min(w.it.lk, w.it.see + t * tt + (row >> lg)));   // keys this row sees
      const int see_warp = __shfl_sync(0xffffffffu, see, 0);              // ... the warp's fewest
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < steps; ++j, ++ns) {
        ok = wait_all(&bars->s_full[t], ns & 1);
        if (!ok) break;
        tc_fence_after();
        if ((j + 1) * kKeys > see_warp) {
          // A step that some row of the warp does not see in full: the scores behind a
          // row's last key are overwritten in TMEM.  (A loop of 16 columns: unrolled
          // over all of them in registers the code, run once or twice an item, took
          // longer to fetch than to execute.)
          const int lim = see - j * kKeys;
#pragma unroll 1
          for (int c = max(0, see_warp - j * kKeys) & ~15; c < kKeys; c += 16) {
            uint32_t r[16];
            tmem_ld16(s_addr + c, r);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) r[i] = c + i < lim ? r[i] : 0xff800000u;
            tmem_st16(s_addr + c, r);
          }
          tmem_wait_st();
        }
        float v[kKeys];
        tmem_ld32f(s_addr, v);
        tmem_ld32f(s_addr + 32, v + 32);
        tmem_ld16f(s_addr + 64, v + 64);
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->s_free[t]);
        float mx[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
        for (int c = 4; c < 76; c += 8) {
#pragma unroll
          for (int i = 0; i < 4; ++i) mx[i] = max3_nan(mx[i], v[c + i], v[c + 4 + i]);
        }
        mx[0] = max3_nan(mx[0], v[76], v[77]);
        mx[1] = max3_nan(mx[1], v[78], v[79]);
        const float top = max3_nan(max3_nan(mx[0], mx[1], mx[2]), mx[3], mx[3]) * scale_log2;
        // NaN (a NaN score that the row sees) takes over m, and with it l and O
        const float m_new = top <= m + 8.0f && m != -INFINITY ? m : top;
        const bool moved = m_new != m;
        const float base = m_new == -INFINITY ? 0.f : m_new;   // a row that sees nothing so far
        // P is free and O complete once the previous step's product is; the product read P
        // from TMEM asynchronously, so the stores below need the fence whether m moved or not
        if (ns > 0) ok = wait_all(&bars->pv_done[t], (ns - 1) & 1);
        if (!ok) break;
        tc_fence_after();
        if (j > 0 && __any_sync(0xffffffffu, moved)) {
          const float f = moved ? ex2(m - base) : 1.f;
          l *= f;
#pragma unroll 1
          for (int c = 0; c < 128; c += 16) {
            uint32_t r[16];
            tmem_ld16(o_addr + c, r);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * f);
            tmem_st16(o_addr + c, r);
          }
        }
        m = m_new;
        uint64_t sum[2] = {0, 0};
        const uint64_t base2 = f2_pack(-base, -base);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t p[16];
          weights16(v + 32 * q, scale2, base2, sum, p);
          weights16(v + 32 * q + 16, scale2, base2, sum, p + 8);
          tmem_st16(p_addr + 16 * q, p);
        }
        uint32_t p[8];
        weights16(v + 64, scale2, base2, sum, p);
        tmem_st8(p_addr + 32, p);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->p_full[t]);
        float s0, s1;
        f2_unpack(f2_add(sum[0], sum[1]), s0, s1);
        l += s0 + s1;
      }
      if (!ok) break;
      // ---- the item's row sums, for the output warps
      if (ni > 0) ok = wait_all(&bars->o_free[t], (ni - 1) & 1);
      if (!ok) break;
      ++ni;
      if (w.it.part >= 0) {      // a piece of the row's keys: as they are
        inv_s[row] = l;
        inv_s[256 + row] = m;
      } else {
        inv_s[row] = see > 0 ? 1.f / l : 0.f;
        inv_s[256 + row] = see > 0 ? (m + __log2f(l)) * 0.6931471805599453f : -INFINITY;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->l_full[t]);
    }
  } else if (warp < kWarpOut + 4) {
    // ---------- output: O / row sum, while the softmax warps go on with the next item
    const int warp_row = (warp & 3) * 32, row = warp_row + lane;
    const uint32_t lane_off = static_cast<uint32_t>(warp_row) << 16;
    const float *inv_s = reinterpret_cast<const float *>(smem + kOffInv);
    uint8_t *stage = smem + kOffOut + (warp & 3) * 4096;   // [32 rows][8 units of 16 bytes]
    int no[2] = {0, 0};
    // The tile's O, l and m for a piece of its keys, not normalised (32 columns at a
    // time through the staging rows).
    auto store_part = [&](const Work &w, int t, int steps, int toks, float l) {
      const long slot = (long)w.it.part * (a.n_heads >> lg) + (w.head >> lg);
      const long r0 = slot * 256 + 128 * t + warp_row;
      if ((row >> lg) < toks) {
        a.part_l[r0 + lane] = steps > 0 ? l : 0.f;
        a.part_m[r0 + lane] = steps > 0 ? inv_s[256 + 128 * t + row] : -INFINITY;
      }
      if (steps == 0) return;
#pragma unroll 1
      for (int q = 0; q < 4; ++q) {
        float o[32];
        tmem_ld32f(tmem + lane_off + kTmemO + 128 * t + 32 * q, o);
        tmem_wait_ld();
        if (q == 3) tc_fence_before();
#pragma unroll
        for (int i = 0; i < 8; ++i)
          *reinterpret_cast<float4 *>(stage + lane * 128 + ((i ^ (lane & 7)) << 4)) =
              make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
        __syncwarp();
        if (q == 3 && lane == 0) mbar_arrive(&bars->o_free[t]);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = 4 * i + (lane >> 3), u = lane & 7;
          const float4 x =
              *reinterpret_cast<const float4 *>(stage + r * 128 + ((u ^ (r & 7)) << 4));
          if (((warp_row + r) >> lg) < toks)
            *reinterpret_cast<float4 *>(a.part_O + (r0 + r) * 128 + 32 * q + 4 * u) = x;
        }
        __syncwarp();
      }
    };
    bool ok = true;
    Work w;
    for (int k = 0; ok && take(k, w); ++k) {
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int toks = tile_tokens(w.it, t, lg), steps = tile_steps(w.it, t, lg);
        if (toks == 0) continue;
        const bool sees = min(w.it.lk, w.it.see + t * tt + (row >> lg)) > 0;
        // (token, head) number of the tile's row r, from that of its first
        const long at0 = (long)(w.it.q0 + t * tt) * a.n_heads + w.head;
        auto at = [&](int r) { return at0 + (long)(r >> lg) * a.n_heads + (r & ((1 << lg) - 1)); };
        float inv = 0.f;
        if (steps > 0) {
          ok = wait_all(&bars->l_full[t], no[t] & 1) && wait_all(&bars->o_full[t], no[t] & 1);
          if (!ok) break;
          ++no[t];
          tc_fence_after();
          inv = inv_s[128 * t + row];
        }
        if (w.it.part >= 0) {
          store_part(w, t, steps, toks, inv);
          continue;
        }
        if ((row >> lg) < toks && a.lse)
          a.lse[at(row)] = steps > 0 ? inv_s[256 + 128 * t + row] : -INFINITY;
        const uint32_t o_addr = tmem + lane_off + kTmemO + 128 * t;
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
#pragma unroll 1
          for (int q = 0; q < 2; ++q) {
            float o[32];
            if (steps > 0) {
              tmem_ld32f(o_addr + 64 * h + 32 * q, o);
              tmem_wait_ld();
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t x[4];
#pragma unroll
              for (int e = 0; e < 4; ++e)
                x[e] = steps > 0 && sees
                           ? pack2(o[8 * i + 2 * e] * inv, o[8 * i + 2 * e + 1] * inv) : 0u;
              *reinterpret_cast<uint4 *>(stage + lane * 128 + (((4 * q + i) ^ (lane & 7)) << 4)) =
                  make_uint4(x[0], x[1], x[2], x[3]);
            }
          }
          if (h == 1 && steps > 0) tc_fence_before();
          __syncwarp();
          if (h == 1 && steps > 0 && lane == 0) mbar_arrive(&bars->o_free[t]);
          bf16 *dst = static_cast<bf16 *>(a.out) + 64 * h;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int r = 4 * i + (lane >> 3), u = lane & 7;
            const uint4 x =
                *reinterpret_cast<const uint4 *>(stage + r * 128 + ((u ^ (r & 7)) << 4));
            if (((warp_row + r) >> lg) < toks)
              *reinterpret_cast<uint4 *>(dst + at(warp_row + r) * 128 + 8 * u) = x;
          }
          __syncwarp();
        }
      }
    }
  } else if (warp == kWarpLoad) {
    if (elect_one()) {
      const int rep = a.n_heads / a.n_kv_heads;
      const int total = items * (a.n_heads >> lg);
      const int group_work = items * heads_per_group;
      int gk = 0, gv = 0, nq[2] = {0, 0}, raw[2] = {0, 0};
      bool tail[2] = {false, false};
      int v_tok = 0, v_kv = 0, v_left = 0;     // the step whose values are still to be loaded
      // The values of a step are asked for after the keys of the next one, which
      // are needed first.
      auto load_v = [&]() -> bool {
        const int g = gv, u = g & 1;
        if (g >= 2 && !wait_bar(ctx, &bars->v_free[u], ((g >> 1) - 1) & 1)) return false;
        ++gv;
        tail[u] = v_left < kKeys;
        raw[u] += tail[u];
        uint64_t *bar = tail[u] ? &bars->v_raw[u] : &bars->v_full[u];
        mbar_expect_tx(bar, kVStage);
        uint8_t *dst = smem + kOffV + u * kVStage;
        tma_load_3d(dst, &tm_v, 0, v_kv, v_tok, bar);
        tma_load_3d(dst + kKBox, &tm_v, 64, v_kv, v_tok, bar);
        return true;
      };
      bool ok = true;
      int idx = blockIdx.x;
      for (int k = 0; ok; ++k) {
        Work w;
        w.head = -1;
        if (idx < total) {
          const int g = idx / group_work, r = idx % group_work;
          w.it = own ? own_items[r / heads_per_group] : a.items[r / heads_per_group];
          w.head = (g * heads_per_group + r % heads_per_group) << lg;
        }
        const int slot = k % kSched;
        if (k >= kSched && !wait_bar(ctx, &bars->w_empty[slot], ((k / kSched) - 1) & 1)) break;
        bars->work[slot] = w;
        mbar_arrive(&bars->w_full[slot]);
        if (w.head < 0) break;
        idx = (int)gridDim.x + atomicAdd(&a.hdr->next, 1);
        const int kv = w.head / rep;
        const int n_t[2] = {tile_steps(w.it, 0, lg), tile_steps(w.it, 1, lg)};
        const int n = max(n_t[0], n_t[1]);
        // no keys follow soon: the values of the step before may not wait for them
        if (n == 0 && gv < gk) ok = load_v();
        // Q of tile t, once the item before has its last scores
        auto load_q = [&](int t) -> bool {
          if (n_t[t] == 0) return true;
          if (nq[t] > 0 && !wait_bar(ctx, &bars->q_empty[t], (nq[t] - 1) & 1)) return false;
          ++nq[t];
          uint8_t *q = smem + kOffQ + t * kQTile;
          const int row = w.it.q0 + t * tt;
          mbar_expect_tx(&bars->q_full[t], kQTile);
          tma_load_3d(q, &tm_qn, 0, w.head, row, &bars->q_full[t]);
          tma_load_3d(q + kQBox, &tm_qn, 64, w.head, row, &bars->q_full[t]);
          tma_load_3d(q + 2 * kQBox, &tm_qr, 0, w.head, row, &bars->q_full[t]);
          return true;
        };
        // tile 0 is through with its Q first: it sees fewer keys
        if (n > 0) ok = load_q(0);
        for (int j = 0; j < n && ok; ++j) {
          const int g = gk, u = g & 1, tok = w.it.k0 + j * kKeys;
          if (g >= 2 && !wait_bar(ctx, &bars->k_free[u], ((g >> 1) - 1) & 1)) {
            ok = false;
            break;
          }
          ++gk;
          uint8_t *dst = smem + kOffK + u * kKStage;
          mbar_expect_tx(&bars->k_full[u], kKStage);
          tma_load_3d(dst, &tm_kn, 0, kv, tok, &bars->k_full[u]);
          tma_load_3d(dst + kKBox, &tm_kn, 64, kv, tok, &bars->k_full[u]);
          tma_load_2d(dst + 2 * kKBox, &tm_kr, 0, tok, &bars->k_full[u]);
          if (gv < g) ok = load_v();      // (of the step before, if not already on its way)
          v_tok = tok;
          v_kv = kv;
          v_left = w.it.lk - j * kKeys;
          if (j == 0 && ok) ok = load_q(1);
        }
      }
      if (ok && !bars->abort && gv < gk) load_v();
      // no CTA asks for work any more once all have been here
      if (atomicInc(&a.hdr->done, gridDim.x - 1) == gridDim.x - 1) a.hdr->next = 0;
      // What is in flight must land before the CTA ends, and another warp's wait may run out
      // after this one is through, so these are waited for whether one has or not.
      for (int g = max(0, gk - 2); g < gk; ++g) drain_bar(&bars->k_full[g & 1], (g >> 1) & 1);
      for (int g = max(0, gv - 2); g < gv; ++g)
        if (tail[g & 1])
          drain_bar(&bars->v_raw[g & 1], (raw[g & 1] - 1) & 1);
        else
          drain_bar(&bars->v_full[g & 1], (g >> 1) & 1);
      for (int t = 0; t < 2; ++t)
        if (nq[t] > 0) drain_bar(&bars->q_full[t], (nq[t] - 1) & 1);
    }
  } else if (warp == kWarpFix) {
    // Rows behind a sequence's last key belong to another sequence and may hold
    // anything: 0 * NaN must not reach O, so the values there are zeroed.
    int g0 = 0;
    uint32_t ph[2] = {0, 0};
    Work w;
    for (int k = 0; take(k, w); ++k) {
      const int n = max(tile_steps(w.it, 0, lg), tile_steps(w.it, 1, lg));
      const int left = w.it.lk - (n - 1) * kKeys;   // keys of the item's last step
      if (n > 0 && left < kKeys) {
        const int u = (g0 + n - 1) & 1;
        if (!wait_all(&bars->v_raw[u], u ? ph[1] : ph[0])) break;
        ph[0] ^= u ^ 1;
        ph[1] ^= u;
        for (int i = left * 16 + lane; i < kKeys * 16; i += 32)
          *reinterpret_cast<uint4 *>(smem + kOffV + u * kVStage + ((i >> 3) & 1) * kKBox +
                                     (i >> 4) * 128 + (i & 7) * 16) = make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->v_full[u]);
      }
      g0 += n;
    }
  } else {
    // ------------------------------------------------ MMAs, a thread for each tile
    if (elect_one()) {
      const int t = warp - kWarpMma;
      const uint64_t qd0 = sdesc(smem_u32(smem + kOffQ + t * kQTile), 16, 1024, 2);
      const uint64_t kd0 = sdesc(smem_u32(smem + kOffK), 16, 1024, 2);
      const uint64_t vd0 = sdesc(smem_u32(smem + kOffV), kKBox, 1024, 2);
      const uint32_t s_tmem = tmem + kTmemS + kKeys * t, p_tmem = tmem + kTmemP + kKeys / 2 * t;
      const uint32_t o_tmem = tmem + kTmemO + 128 * t;
      int nw = 0;                           // items read
      int no = 0, ni = 0, ns = 0, np = 0;   // of the tile: Q tiles, items, scores, products
      int n_t = 0, n = 0;                   // the item's steps: of this tile, in all
      // The next item.  One at a time: an item without keys may not hold up the product
      // of the item before, which the output warps need before they take more items.
      auto next_work = [&]() -> bool {
        const int slot = nw % kSched;
        if (!wait_bar(ctx, &bars->w_full[slot], (nw / kSched) & 1)) return false;
        ++nw;
        const Work w = bars->work[slot];
        mbar_arrive(&bars->w_empty[slot]);
        if (w.head < 0) return false;
        n_t = tile_steps(w.it, t, lg);
        n = max(n_t, tile_steps(w.it, t ^ 1, lg));
        return true;
      };
      // S = Q K^T with the keys of step g, once the scores before have been read
      auto scores = [&](int g, bool first, bool last) -> bool {
        const int u = g & 1;
        if (!wait_bar(ctx, &bars->k_full[u], (g >> 1) & 1)) return false;
        if (first && !wait_bar(ctx, &bars->q_full[t], no & 1)) return false;
        no += first;
        if (ns > 0 && !wait_bar(ctx, &bars->s_free[t], (ns - 1) & 1)) return false;
        ++ns;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < 3; ++c) {
          const uint64_t qd = qd0 + (uint64_t)((c * kQBox) >> 4);
          const uint64_t kd = kd0 + (uint64_t)((u * kKStage + c * kKBox) >> 4);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            umma_bf16(s_tmem, qd + (uint64_t)((32 * k) >> 4), kd + (uint64_t)((32 * k) >> 4),
                      kIdescS, (c | k) ? 1u : 0u);
        }
        umma_commit(&bars->s_full[t]);
        umma_commit(&bars->k_free[u]);
        if (last) umma_commit(&bars->q_empty[t]);
        return true;
      };
      // O += P V with the values of step g
      auto values = [&](int g, bool first, bool last) -> bool {
        const int u = g & 1;
        if (!wait_bar(ctx, &bars->v_full[u], (g >> 1) & 1)) return false;
        // the first product of an item overwrites the O of the one before (items are
        // counted by their first scores, and those of the next one may be out already)
        if (first && ++ni > 1 && !wait_bar(ctx, &bars->o_free[t], (ni - 2) & 1)) return false;
        if (!wait_bar(ctx, &bars->p_full[t], np & 1)) return false;
        ++np;
        tc_fence_after();
        const uint64_t vd = vd0 + (uint64_t)((u * kVStage) >> 4);
#pragma unroll
        for (int k = 0; k < kKeys / 16; ++k)
          umma_bf16_ts(o_tmem, p_tmem + 8 * k, vd + (uint64_t)((2048 * k) >> 4), kIdescPV,
                       (first && k == 0) ? 0u : 1u);
        umma_commit(&bars->pv_done[t]);
        umma_commit(&bars->v_free[u]);
        if (last) umma_commit(&bars->o_full[t]);
        return true;
      };
      bool more = next_work(), ok = true, ahead = false;   // ahead: the item's first S is out
      for (int g0 = 0; more && ok;) {
        const int steps = n_t, all = n;
        if (all == 0) {
          more = next_work();
          continue;
        }
        if (steps > 0 && !ahead) ok = scores(g0, true, steps == 1);
        ahead = false;
        for (int j = 0; j < steps && ok; ++j) {
          const bool last = j + 1 == steps;
          if (!last) {
            ok = scores(g0 + j + 1, false, j + 2 == steps);
          } else if (steps == all) {
            more = next_work();
            ahead = more && n_t > 0;
            if (ahead) ok = scores(g0 + all, true, n_t == 1);
          }
          ok = ok && values(g0 + j, j == 0, last);
        }
        // Steps of the other tile alone.  (A release counts for the phase that is
        // running, so it waits until the step's load is in.)
        for (int g = g0 + steps; g < g0 + all && ok; ++g) {
          ok = wait_bar(ctx, &bars->k_full[g & 1], (g >> 1) & 1);
          if (ok) mbar_arrive(&bars->k_free[g & 1]);
          ok = ok && wait_bar(ctx, &bars->v_full[g & 1], (g >> 1) & 1);
          if (ok) mbar_arrive(&bars->v_free[g & 1]);
        }
        g0 += all;
        if (steps < all && ok) more = next_work();
      }
      umma_commit(&bars->drain[t]);
      drain_bar(&bars->drain[t], 0);
    }
  }

  __syncwarp();
  __syncthreads();
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Rows whose keys were cut into pieces: M = max_j m_j, w_j = 2^(m_j - M),
// out = sum_j w_j O_j / sum_j w_j l_j, lse = ln 2 (M + log2 sum_j w_j l_j), pieces in
// order.  One warp a row: a lane a piece for m and l, then a lane four columns of O.  A
// piece that the row sees nothing of has l = 0 and is not read.
__global__ void __launch_bounds__(256) prompt_join_kernel(const PromptAttnArgs a) {
  const int lane = threadIdx.x & 31, lg = a.pack_log2;
  const int packs = a.n_heads >> lg, item = blockIdx.x / packs, pack = blockIdx.x % packs;
  const int row = blockIdx.y * 8 + (threadIdx.x >> 5);
  grid_dep_wait();
  grid_dep_launch();
  const PromptJoin jn = a.join[item];
  if (jn.pieces == 0 || row >= jn.tokens << lg) return;
  const long at0 = ((long)jn.first * packs + pack) * 256 + row, step = (long)packs * 256;
  constexpr int kRounds = (kPromptParts + 31) / 32;
  float lj[kRounds], mj[kRounds], top = -INFINITY;
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    const int j = 32 * r + lane;
    lj[r] = j < jn.pieces ? a.part_l[at0 + j * step] : 0.f;
    mj[r] = j < jn.pieces ? a.part_m[at0 + j * step] : 0.f;
  }
#pragma unroll
  for (int r = 0; r < kRounds; ++r)
    if (lj[r] != 0.f) top = max3_nan(top, mj[r], top);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = max3_nan(top, __shfl_xor_sync(0xffffffffu, top, o), top);
  float l = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int r = 0; r < kRounds; ++r) {
    const float w = lj[r] != 0.f ? ex2(mj[r] - top) : 0.f;
    l += w * lj[r];
    const int n = min(32, jn.pieces - 32 * r);
#pragma unroll 8
    for (int j = 0; j < n; ++j) {
      const float wj = __shfl_sync(0xffffffffu, w, j);
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
      if (wj != 0.f)
        x = *reinterpret_cast<const float4 *>(a.part_O + (at0 + (32 * r + j) * step) * 128 +
                                              4 * lane);
      acc[0] = fmaf(wj, x.x, acc[0]);
      acc[1] = fmaf(wj, x.y, acc[1]);
      acc[2] = fmaf(wj, x.z, acc[2]);
      acc[3] = fmaf(wj, x.w, acc[3]);
    }
  }
  l = warp_sum(l);
  const bool some = jn.see + (row >> lg) > 0;      // the row sees a key
  const float inv = some ? 1.f / l : 0.f;
  const long dst = (long)(jn.q0 + (row >> lg)) * a.n_heads + (pack << lg) + (row & ((1 << lg) - 1));
  *reinterpret_cast<uint2 *>(static_cast<bf16 *>(a.out) + dst * 128 + 4 * lane) =
      make_uint2(pack2(acc[0] * inv, acc[1] * inv), pack2(acc[2] * inv, acc[3] * inv));
  if (a.lse && lane == 0) a.lse[dst] = some ? (top + __log2f(l)) * 0.6931471805599453f : -INFINITY;
}

// ------------------------------------------------------------------ host side

typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                  const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                  const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) !=
            cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeTiledFn>(p);
  }();
  return fn;
}

// Map of a packed [tokens][heads][width] bf16 view; box = 64 columns of box_heads
// heads of box_tokens tokens, heads running faster.  Tokens past the end read as zeros.
bool map_heads(CUtensorMap *m, const HeadsView &v, int tokens, int heads, int width,
               int box_heads, int box_tokens) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)width, (cuuint64_t)heads, (cuuint64_t)tokens};
  const cuuint64_t strides[2] = {(cuuint64_t)v.head * 2, (cuuint64_t)v.token * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_tokens}, estr[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(v.ptr), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool map_rows(CUtensorMap *m, const void *ptr, int64_t stride, int tokens) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[2] = {64, (cuuint64_t)tokens};
  const cuuint64_t strides[1] = {(cuuint64_t)stride * 2};
  const cuuint32_t box[2] = {64, kKeys}, estr[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(ptr), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

cudaError_t launch_prompt_attn(const PromptAttnArgs &a, cudaStream_t s) {
  static api::PerDeviceOnce smem_attr;
  cudaError_t e = smem_attr.run([] {
    return cudaFuncSetAttribute(prompt_attn_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                kSmemBytes);
  });
  if (e != cudaSuccess) return e;
  CUtensorMap qn, qr, kn, kr, v;
  const int pack = 1 << a.pack_log2;
  if (!map_heads(&qn, a.q_nope, a.n_q, a.n_heads, 128, pack, kRows / pack) ||
      !map_heads(&qr, a.q_rope, a.n_q, a.n_heads, 64, pack, kRows / pack))
    return cudaErrorInvalidValue;
  if (a.n_k > 0) {
    if (!map_heads(&kn, a.k_nope, a.n_k, a.n_kv_heads, 128, 1, kKeys) ||
        !map_rows(&kr, a.k_rope, a.k_rope_stride, a.n_k) ||
        !map_heads(&v, a.v, a.n_k, a.n_kv_heads, 128, 1, kKeys))
      return cudaErrorInvalidValue;
  } else {
    kn = kr = v = qn;   // no key exists, so nothing is loaded through them
  }
  int dev = 0, sms = 148;
  e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  // Heads are taken in groups whose keys and values stay in L2 together while
  // their blocks are worked off, most keys first within the group.
  const int packs = a.n_heads / pack;
  const long kv_bytes = 512L * a.n_k * a.n_kv_heads / packs + 1;   // of the heads of one pack
  int group = packs;
  while (group > 1 && (packs % group || kv_bytes * group > (60L << 20))) --group;
  const long work = a.max_items * packs;
  // Few blocks with long keys: see own_plan.  (The bounds that the host knows decide;
  // what the lengths then allow is decided on the device.)
  const bool split = 2 * work <= sms && 2 * work <= kPromptParts && a.n_k >= kPromptSplitKeys;
  const float scale_log2 = a.scale * 1.4426950408889634f;
  const long ctas = split ? (sms < kPromptParts ? sms : kPromptParts) : work < sms ? work : sms;
  e = launch_pdl(prompt_attn_kernel, dim3((unsigned)ctas), dim3(kThreads), kSmemBytes, s, qn, qr, kn,
                 kr, v, a, scale_log2, split ? packs : group, split);
  if (e != cudaSuccess || !split) return e;
  return launch_pdl(prompt_join_kernel, dim3((unsigned)work, kPromptTileSm100 / 8), dim3(256), 0, s, a);
}

}  // namespace sm100
}  // namespace mla

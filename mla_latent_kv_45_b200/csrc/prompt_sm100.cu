// Causal attention over packed sequences on sm_100a tensor cores (bf16, scores
// over 128 + 64 values, 128-wide values).
//
// out_i = sum_j softmax_j(scale (q_nope_i . k_nope_j + q_rope_i . k_rope_j)) v_j in
// one pass over the keys with a running maximum m and sum l per row
// ("从零理解 MLA", 解耦 RoPE MLADecoupledRoPE.forward).
//
// One work item is 256 query rows of one head: two 128-row tiles that share
// every key and value tile in shared memory.  Per 128 keys a tile costs
// S = Q K^T (K = 192, the two score terms are one product) and O += P V.
//  * TMEM holds S of both tiles (2 x 128 columns) and O of both (2 x 128): all
//    512.  P (bf16) overwrites its S in place and is the A operand of P V.
//  * Warps 0-3 and 4-7 are the softmax of tile 0 and 1, one thread a row: no
//    reduction crosses threads.  While one tile is in its softmax the other has
//    the tensor pipe.
//  * m moves only when the maximum grows by more than 2^8 (p stays below
//    256); only then does the thread rescale O, so the P V products wait for
//    nothing else.
//  * Warp 8 streams keys and values through a ring of eight 16 KB chunks (64
//    score columns of 128 keys, or 64 keys of 128 value columns), warp 9 issues
//    the MMAs.
//  * Work comes from a counter: the CTAs are persistent and fetch (block, head)
//    pairs, blocks with most keys first.
//  * Every wait is bounded as in the decode kernel; on expiry the error word is set.
#include <cuda.h>

#include "api_checks.h"
#include "prompt.h"
#include "ptx.cuh"

namespace mla {
namespace sm100 {
namespace {

using namespace ptx;
using bf16 = __nv_bfloat16;

constexpr int kTile = 128;              // rows of a tile, keys of a step
constexpr int kChunk = 16384;           // bytes of a ring slot and of a 64-column box of Q
constexpr int kSlots = 8;
constexpr int kSched = 3;               // work items in flight between the warps
constexpr int kWarpOut = 8;             // warps 8-11 write the output
constexpr int kWarpLoad = 12, kWarpMma = 13, kWarpFix = 14, kWarps = 16;
constexpr int kThreads = 32 * kWarps;
// Registers a thread: a softmax row keeps its 128 scores, the other two
// warpgroups (one warp idle) need few.  Launched with 65536 / 512 = 128.
constexpr int kRegsSoftmax = 176, kRegsOther = 80;
static_assert(256 * kRegsSoftmax + 256 * kRegsOther <= kThreads * 128, "register split");
constexpr uint64_t kTimeoutNs = 2000000000ull;
constexpr uint32_t kSleepNs = 20000;

constexpr int kOffQ = 0;                          // [2 tiles][3 boxes]
constexpr int kOffRing = kOffQ + 6 * kChunk;
constexpr int kOffBar = kOffRing + kSlots * kChunk;
constexpr int kOffInv = kOffBar + 1024;           // [2 tiles][128] 1 / row sum
constexpr int kSmemBytes = kOffInv + 1024;
static_assert(kSmemBytes <= 232448, "shared memory per CTA");

constexpr uint32_t kTmemS = 0, kTmemO = 256, kTmemCols = 512;   // tile t at + 128 t
constexpr uint32_t kIdescS = idesc_bf16(128, 128, 0, 0);
constexpr uint32_t kIdescPV = idesc_bf16(128, 128, 0, 1);       // V is [key][column]

// One (block of rows, head) pair on its way from the loading warp to the others.
struct Work {
  PromptItem it;
  int head;   // -1: no more work
};

// Steps are counted through (g) over all items of a CTA.  Step g's keys are ring
// chunks 5 g .. 5 g + 2 (mod 8), its values 5 g + 3 and 5 g + 4, so the keys of g take the
// place of the last key chunk and the values of g - 2, the values of g that of the
// first two key chunks of g - 1.
struct Bars {
  uint64_t k_full[2], k_free[2], v_full[2], v_free[2];   // of step g at g % 2
  uint64_t v_raw[2];      // values that end inside the step landed; the fixing warp fills v_full
  uint64_t q_full[2], q_empty[2];
  uint64_t s_full[2];     // scores of the tile complete (and its P V products so far)
  uint64_t p_full[2][2];  // half of P written (and O rescaled) by the tile's four warps
  uint64_t o_full[2];     // the item's last O += P V complete
  uint64_t l_full[2];     // the reciprocal row sums are in shared memory
  uint64_t o_free[2];     // O and the row sums have been read
  uint64_t w_full[kSched], w_empty[kSched];
  uint64_t drain;
  Work work[kSched];
  uint32_t tmem_base;
  volatile int abort;
};
static_assert(sizeof(Bars) <= 1024, "barrier region");

struct Ctx {
  Bars *bars;
  int *err;
};

__device__ __forceinline__ bool wait_bar(const Ctx &c, uint64_t *bar, uint32_t parity) {
  const uint32_t a = smem_u32(bar);
  if (mbar_try_wait(a, parity)) return true;
  const uint64_t t0 = globaltimer();
  while (true) {
    if (mbar_try_wait(a, parity)) return true;
    if (c.bars->abort) return false;
    if (globaltimer() - t0 > kTimeoutNs) {
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
    if (globaltimer() - t0 > kTimeoutNs) return;
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}

__device__ __forceinline__ uint64_t exp2_sfu(uint64_t x) {
  float a, b;
  f2_unpack(x, a, b);
  return f2_pack(ex2(a), ex2(b));
}

// 32 bytes (a whole sector of L2) to a 32-byte aligned address.
__device__ __forceinline__ void st_global_32(void *p, uint32_t a, uint32_t b, uint32_t c,
                                             uint32_t d, uint32_t e, uint32_t f, uint32_t g,
                                             uint32_t h) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(a), "r"(b),
               "r"(c), "r"(d), "r"(e), "r"(f), "r"(g), "r"(h)
               : "memory");
}

// Rows of tile t of an item, and the steps of 128 keys that its last row sees.
__device__ __forceinline__ int tile_rows(const PromptItem &it, int t) {
  return max(0, min(kTile, it.rows - t * kTile));
}
__device__ __forceinline__ int tile_steps(const PromptItem &it, int t) {
  const int rows = tile_rows(it, t);
  if (rows == 0) return 0;
  const int keys = max(0, min(it.lk, it.see + t * kTile + rows - 1));
  return (keys + kTile - 1) / kTile;
}

__global__ void __launch_bounds__(kThreads, 1)
    prompt_attn_kernel(const __grid_constant__ CUtensorMap tm_qn,
                       const __grid_constant__ CUtensorMap tm_qr,
                       const __grid_constant__ CUtensorMap tm_kn,
                       const __grid_constant__ CUtensorMap tm_kr,
                       const __grid_constant__ CUtensorMap tm_v, const PromptAttnArgs a,
                       const float scale_log2, const int heads_per_group) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t *smem = smem_raw;
  Bars *bars = reinterpret_cast<Bars *>(smem + kOffBar);
  const Ctx ctx{bars, a.err};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // The swizzled boxes need a 1024-byte boundary, which the dynamic shared memory
  // starts on (there is no static part in front of it).
  if (smem_u32(smem) & 1023) {
    if (threadIdx.x == 0) set_error(a.err, kErrTimeout);
    return;
  }
  if (threadIdx.x == 0) {
    for (int t = 0; t < 2; ++t) {
      mbar_init(&bars->k_full[t], 1);
      mbar_init(&bars->k_free[t], 1);
      mbar_init(&bars->v_full[t], 1);
      mbar_init(&bars->v_free[t], 1);
      mbar_init(&bars->v_raw[t], 1);
      mbar_init(&bars->q_full[t], 1);
      mbar_init(&bars->q_empty[t], 1);
      mbar_init(&bars->s_full[t], 1);
      mbar_init(&bars->p_full[t][0], 4);
      mbar_init(&bars->p_full[t][1], 4);
      mbar_init(&bars->o_full[t], 1);
      mbar_init(&bars->l_full[t], 4);
      mbar_init(&bars->o_free[t], 4);
    }
    for (int i = 0; i < kSched; ++i) {
      mbar_init(&bars->w_full[i], 1);
      mbar_init(&bars->w_empty[i], 14);   // eight softmax, four output warps, MMA, fixing
    }
    mbar_init(&bars->drain, 1);
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
  grid_dep_wait();     // the plan is read from here on
  grid_dep_launch();

  // the k-th work item of this CTA, as every warp but the loading one reads it
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

  // the register moves stand inside the roles: what follows a point that all warps
  // reach would be compiled for the smaller share
  if (warp < 8) {
    regs_raise<kRegsSoftmax>();
    // ------------------------------------------------ softmax and output, one thread a row
    const int t = warp >> 2;
    const int row = (warp & 3) * 32 + lane;
    const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_addr = tmem + lane_off + kTmemS + 128 * t;
    const uint32_t o_addr = tmem + lane_off + kTmemO + 128 * t;
    float *inv_s = reinterpret_cast<float *>(smem + kOffInv) + 128 * t;
    int ns = 0, ni = 0;      // steps and items (with keys) of this tile so far
    bool ok = true;
    Work w;
    for (int k = 0; ok && take(k, w); ++k) {
      const int rows = tile_rows(w.it, t);
      const int steps = tile_steps(w.it, t);
      if (steps == 0) continue;
      const int see = max(0, min(w.it.lk, w.it.see + t * kTile + row));   // keys this row sees
      const int see_warp = __shfl_sync(0xffffffffu, see, 0);              // ... the warp's fewest
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < steps; ++j, ++ns) {
        ok = __all_sync(0xffffffffu, wait_bar(ctx, &bars->s_full[t], ns & 1));
        if (!ok) break;
        tc_fence_after();
        float v[128];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32f(s_addr + 32 * c, v + 32 * c);
        tmem_wait_ld();
        if ((j + 1) * kTile > see_warp) {
          const int lim = see - j * kTile;
#pragma unroll
          for (int c = 0; c < 128; ++c) v[c] = c < lim ? v[c] : -INFINITY;
        }
        float mx[4] = {v[0], v[1], v[2], v[3]};
#pragma unroll
        for (int c = 4; c < 124; c += 8) {
#pragma unroll
          for (int i = 0; i < 4; ++i) mx[i] = max3_nan(mx[i], v[c + i], v[c + 4 + i]);
        }
        mx[0] = max3_nan(mx[0], v[124], v[125]);
        mx[1] = max3_nan(mx[1], v[126], v[127]);
        const float top = max3_nan(max3_nan(mx[0], mx[1], mx[2]), mx[3], mx[3]) * scale_log2;
        // NaN (a NaN score that the row sees) takes over m, and with it l and O
        const float m_new = top <= m + 8.0f && m != -INFINITY ? m : top;
        const bool moved = m_new != m;
        const float base = m_new == -INFINITY ? 0.f : m_new;   // a row that sees nothing so far
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
        const uint64_t scale2 = f2_pack(scale_log2, scale_log2), base2 = f2_pack(-base, -base);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            uint32_t p[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const int c = 64 * h + 32 * q + 2 * i;
              const uint64_t e = exp2_sfu(f2_fma(f2_pack(v[c], v[c + 1]), scale2, base2));
              sum[i & 1] = f2_add(sum[i & 1], e);
              float e0, e1;
              f2_unpack(e, e0, e1);
              p[i] = pack2(e0, e1);
            }
            tmem_st16(s_addr + 32 * h + 16 * q, p);
          }
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->p_full[t][h]);
        }
        float s0, s1;
        f2_unpack(f2_add(sum[0], sum[1]), s0, s1);
        l += s0 + s1;
      }
      if (!ok) break;
      // ---- the item's row sums, for the output warps
      if (ni > 0)
        ok = __all_sync(0xffffffffu, wait_bar(ctx, &bars->o_free[t], (ni - 1) & 1));
      if (!ok) break;
      ++ni;
      inv_s[row] = 1.f / l;
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars->l_full[t]);
      if (row < rows && a.lse)
        a.lse[(long)(w.it.q0 + t * kTile + row) * a.n_heads + w.head] =
            see > 0 ? (m + __log2f(l)) * 0.6931471805599453f : -INFINITY;
    }
  } else {
    regs_lower<kRegsOther>();
    if (warp < kWarpOut + 4) {
      // ---------- output: O / row sum of the tile's rows, one thread a row, while the
      // softmax warps go on with the next item
      const int row = (warp & 3) * 32 + lane;
      const uint32_t lane_off = static_cast<uint32_t>((warp & 3) * 32) << 16;
      const float *inv_s = reinterpret_cast<const float *>(smem + kOffInv);
      int no[2] = {0, 0};
      bool ok = true;
      Work w;
      for (int k = 0; ok && take(k, w); ++k) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const int rows = tile_rows(w.it, t), steps = tile_steps(w.it, t);
          if (rows == 0) continue;
          const int see = min(w.it.lk, w.it.see + t * kTile + row);
          const long at = (long)(w.it.q0 + t * kTile + row) * a.n_heads + w.head;
          bf16 *dst = static_cast<bf16 *>(a.out) + at * 128;
          if (steps == 0) {      // no row of the tile sees a key
            if (row < rows) {
              for (int c = 0; c < 128; c += 16) st_global_32(dst + c, 0, 0, 0, 0, 0, 0, 0, 0);
              if (a.lse) a.lse[at] = -INFINITY;
            }
            continue;
          }
          ok = wait_bar(ctx, &bars->l_full[t], no[t] & 1) &&
               wait_bar(ctx, &bars->o_full[t], no[t] & 1);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          ++no[t];
          tc_fence_after();
          const float inv = inv_s[128 * t + row];
          const uint32_t o_addr = tmem + lane_off + kTmemO + 128 * t;
#pragma unroll 1
          for (int c = 0; c < 128; c += 32) {
            float o[32];
            tmem_ld32f(o_addr + c, o);
            tmem_wait_ld();
            if (c == 96) {
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(&bars->o_free[t]);
            }
            uint32_t x[16];
#pragma unroll
            for (int i = 0; i < 16; ++i)
              x[i] = see > 0 ? pack2(o[2 * i] * inv, o[2 * i + 1] * inv) : 0u;
            if (row < rows) {
              st_global_32(dst + c, x[0], x[1], x[2], x[3], x[4], x[5], x[6], x[7]);
              st_global_32(dst + c + 16, x[8], x[9], x[10], x[11], x[12], x[13], x[14], x[15]);
            }
          }
        }
      }
    } else if (warp == kWarpLoad) {
      if (lane == 0) {
        const int rep = a.n_heads / a.n_kv_heads;
        const int items = a.hdr->items, total = items * a.n_heads;
        const int group_work = items * heads_per_group;
        int gk = 0, gv = 0, nq[2] = {0, 0}, raw[2] = {0, 0};
        bool tail[2] = {false, false};
        bool ok = true;
        int idx = blockIdx.x;
        for (int k = 0; ok; ++k) {
          Work w;
          w.head = -1;
          if (idx < total) {
            const int g = idx / group_work, r = idx % group_work;
            w.it = a.items[r / heads_per_group];
            w.head = g * heads_per_group + r % heads_per_group;
          }
          const int slot = k % kSched;
          if (k >= kSched && !wait_bar(ctx, &bars->w_empty[slot], ((k / kSched) - 1) & 1)) break;
          bars->work[slot] = w;
          mbar_arrive(&bars->w_full[slot]);
          if (w.head < 0) break;
          const int next = (int)gridDim.x + atomicAdd(&a.hdr->next, 1);
          const int kv = w.head / rep;
          int n_t[2], n = 0;
          for (int t = 0; t < 2; ++t) {
            n_t[t] = tile_steps(w.it, t);
            n = max(n, n_t[t]);
          }
          auto ring = [&](int c) { return smem + kOffRing + (c & (kSlots - 1)) * kChunk; };
          auto load_k = [&](int j) -> bool {
            const int g = gk, u = g & 1;
            if (g >= 2 && (!wait_bar(ctx, &bars->k_free[u], ((g >> 1) - 1) & 1) ||
                           !wait_bar(ctx, &bars->v_free[u], ((g >> 1) - 1) & 1)))
              return false;
            ++gk;
            const int tok = w.it.k0 + j * kTile;
            mbar_expect_tx(&bars->k_full[u], 3 * kChunk);
            tma_load_3d(ring(5 * g), &tm_kn, 0, kv, tok, &bars->k_full[u]);
            tma_load_3d(ring(5 * g + 1), &tm_kn, 64, kv, tok, &bars->k_full[u]);
            tma_load_2d(ring(5 * g + 2), &tm_kr, 0, tok, &bars->k_full[u]);
            return true;
          };
          auto load_v = [&](int j) -> bool {
            const int g = gv, u = g & 1;
            if (g >= 1 && !wait_bar(ctx, &bars->k_free[u ^ 1], ((g - 1) >> 1) & 1)) return false;
            ++gv;
            tail[u] = w.it.lk - j * kTile < kTile;
            raw[u] += tail[u];
            uint64_t *bar = tail[u] ? &bars->v_raw[u] : &bars->v_full[u];
            mbar_expect_tx(bar, 2 * kChunk);
            for (int c = 0; c < 2; ++c) {
              uint8_t *dst = ring(5 * g + 3 + c);
              const int tok = w.it.k0 + j * kTile + 64 * c;
              tma_load_3d(dst, &tm_v, 0, kv, tok, bar);
              tma_load_3d(dst + kChunk / 2, &tm_v, 64, kv, tok, bar);
            }
            return true;
          };
          for (int t = 0; t < 2 && ok; ++t) {
            if (n_t[t] == 0) continue;
            if (nq[t] > 0 && !wait_bar(ctx, &bars->q_empty[t], (nq[t] - 1) & 1)) {
              ok = false;
              break;
            }
            ++nq[t];
            uint8_t *dst = smem + kOffQ + 3 * t * kChunk;
            const int tok = w.it.q0 + t * kTile;
            mbar_expect_tx(&bars->q_full[t], 3 * kChunk);
            tma_load_3d(dst, &tm_qn, 0, w.head, tok, &bars->q_full[t]);
            tma_load_3d(dst + kChunk, &tm_qn, 64, w.head, tok, &bars->q_full[t]);
            tma_load_3d(dst + 2 * kChunk, &tm_qr, 0, w.head, tok, &bars->q_full[t]);
          }
          if (ok && n > 0) ok = load_k(0);
          for (int j = 0; j < n && ok; ++j) {
            ok = load_v(j);
            if (ok && j + 1 < n) ok = load_k(j + 1);
          }
          idx = next;
        }
        if (bars->abort) {
          // what is in flight must land before the CTA ends
          for (int g = max(0, gk - 2); g < gk; ++g) drain_bar(&bars->k_full[g & 1], (g >> 1) & 1);
          for (int g = max(0, gv - 2); g < gv; ++g)
            if (tail[g & 1])
              drain_bar(&bars->v_raw[g & 1], (raw[g & 1] - 1) & 1);
            else
              drain_bar(&bars->v_full[g & 1], (g >> 1) & 1);
          for (int t = 0; t < 2; ++t)
            if (nq[t] > 0) drain_bar(&bars->q_full[t], (nq[t] - 1) & 1);
        }
      }
    } else if (warp == kWarpFix) {
      // Rows behind a sequence's last key belong to another sequence and may hold
      // anything: 0 * NaN must not reach O, so the values there are zeroed.
      int g0 = 0;
      uint32_t ph[2] = {0, 0};
      Work w;
      for (int k = 0; take(k, w); ++k) {
        const int n = max(tile_steps(w.it, 0), tile_steps(w.it, 1));
        const int left = w.it.lk - (n - 1) * kTile;   // keys of the item's last step
        if (n > 0 && left < kTile) {
          const int g = g0 + n - 1, u = g & 1;
          if (!__all_sync(0xffffffffu, wait_bar(ctx, &bars->v_raw[u], u ? ph[1] : ph[0]))) break;
          ph[0] ^= u ^ 1;
          ph[1] ^= u;
          for (int i = left * 16 + lane; i < kTile * 16; i += 32) {
            const int row = i >> 4, c = 5 * g + 3 + (row >> 6);
            *reinterpret_cast<uint4 *>(smem + kOffRing + (c & (kSlots - 1)) * kChunk +
                                       ((i >> 3) & 1) * (kChunk / 2) + (row & 63) * 128 +
                                       (i & 7) * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->v_full[u]);
        }
        g0 += n;
      }
    } else if (warp == kWarpMma) {
      if (elect_one()) {
        const uint64_t qd0 = sdesc(smem_u32(smem + kOffQ), 16, 1024, 2);
        const uint64_t kd0 = sdesc(smem_u32(smem + kOffRing), 16, 1024, 2);
        const uint64_t vd0 = sdesc(smem_u32(smem + kOffRing), kChunk / 2, 1024, 2);
        int g = 0, ni = 0;   // steps and items so far
        int no[2] = {0, 0};          // items with keys, per tile
        uint32_t p_ph[2] = {0, 0}, q_ph[2] = {0, 0};
        Work w;
        int n_t[2] = {0, 0}, n = 0;
        // the next item that has any keys
        auto next_work = [&]() -> bool {
          while (true) {
            const int slot = ni % kSched;
            if (!wait_bar(ctx, &bars->w_full[slot], (ni / kSched) & 1)) return false;
            ++ni;
            w = bars->work[slot];
            mbar_arrive(&bars->w_empty[slot]);
            if (w.head < 0) return false;
            n_t[0] = tile_steps(w.it, 0);
            n_t[1] = tile_steps(w.it, 1);
            n = max(n_t[0], n_t[1]);
            if (n > 0) return true;
          }
        };
        // S of tile t = Q K^T with the keys of step gk
        auto scores = [&](int t, int gk) {
#pragma unroll
          for (int c = 0; c < 3; ++c) {
            const uint64_t qd = qd0 + (uint64_t)(((3 * t + c) * kChunk) >> 4);
            const uint64_t kd = kd0 + (uint64_t)((((5 * gk + c) & (kSlots - 1)) * kChunk) >> 4);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              umma_bf16(tmem + kTmemS + 128 * t, qd + (uint64_t)((32 * k) >> 4),
                        kd + (uint64_t)((32 * k) >> 4), kIdescS, (c | k) ? 1u : 0u);
          }
          umma_commit(&bars->s_full[t]);
        };
        auto k_ready = [&](int gk) {
          const bool r = wait_bar(ctx, &bars->k_full[gk & 1], (gk >> 1) & 1);
          tc_fence_after();
          return r;
        };
        // S of step 0 of the current item's tile t
        auto first_scores = [&](int t, int gk) -> bool {
          if (!wait_bar(ctx, &bars->q_full[t], q_ph[t])) return false;
          q_ph[t] ^= 1;
          tc_fence_after();
          scores(t, gk);
          if (n_t[t] == 1) umma_commit(&bars->q_empty[t]);
          return true;
        };
        bool more = next_work(), ok = true;
        if (more) {
          ok = k_ready(0);
          for (int t = 0; t < 2 && ok; ++t)
            if (n_t[t] > 0) ok = first_scores(t, 0);
          if (ok) umma_commit(&bars->k_free[0]);
        }
        while (more && ok) {
          const int steps = n, nt[2] = {n_t[0], n_t[1]};
          for (int j = 0; j < steps && ok; ++j, ++g) {
            const bool last = j + 1 == steps;
            if (last) more = next_work();
            const bool keys = !last || more;    // step g + 1 exists
            ok = wait_bar(ctx, &bars->v_full[g & 1], (g >> 1) & 1);
            bool keys_in = false;
#pragma unroll
            for (int t = 0; t < 2; ++t) {
              if (ok && j < nt[t]) {
                // the first product of an item overwrites the O of the one before
                if (j == 0 && no[t]++ > 0) ok = wait_bar(ctx, &bars->o_free[t], (no[t] - 2) & 1);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  ok = ok && wait_bar(ctx, &bars->p_full[t][h], p_ph[t]);
                  if (!ok) break;
                  tc_fence_after();
                  const uint64_t vd =
                      vd0 + (uint64_t)((((5 * g + 3 + h) & (kSlots - 1)) * kChunk) >> 4);
#pragma unroll
                  for (int k = 0; k < 4; ++k)
                    umma_bf16_ts(tmem + kTmemO + 128 * t, tmem + kTmemS + 128 * t + 32 * h + 8 * k,
                                 vd + (uint64_t)((2048 * k) >> 4), kIdescPV,
                                 (j == 0 && h == 0 && k == 0) ? 0u : 1u);
                }
                p_ph[t] ^= 1;
                if (j + 1 == nt[t]) umma_commit(&bars->o_full[t]);
              }
              if (!ok) break;
              if (t == 1) umma_commit(&bars->v_free[g & 1]);
              if (last ? more && n_t[t] > 0 : j + 1 < nt[t]) {
                if (!keys_in) ok = k_ready(g + 1);
                keys_in = true;
                if (!ok) break;
                if (last) {
                  ok = first_scores(t, g + 1);
                } else {
                  scores(t, g + 1);
                  if (j + 2 == nt[t]) umma_commit(&bars->q_empty[t]);
                }
              }
              if (!ok) break;
            }
            if (ok && keys) umma_commit(&bars->k_free[(g + 1) & 1]);
          }
        }
        umma_commit(&bars->drain);
        drain_bar(&bars->drain, 0);
      }
    }
  }

  __syncwarp();
  __syncthreads();
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
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

// Map of a packed [tokens][heads][width] bf16 view; box = 64 columns of one head
// of `box_tokens` tokens.  Tokens past the end read as zeros.
bool map_heads(CUtensorMap *m, const HeadsView &v, int tokens, int heads, int width,
               int box_tokens) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)width, (cuuint64_t)heads, (cuuint64_t)tokens};
  const cuuint64_t strides[2] = {(cuuint64_t)v.head * 2, (cuuint64_t)v.token * 2};
  const cuuint32_t box[3] = {64, 1, (cuuint32_t)box_tokens}, estr[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(v.ptr), dims, strides, box,
             estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool map_rows(CUtensorMap *m, const void *ptr, int64_t stride, int tokens) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t dims[2] = {64, (cuuint64_t)tokens};
  const cuuint64_t strides[1] = {(cuuint64_t)stride * 2};
  const cuuint32_t box[2] = {64, kTile}, estr[2] = {1, 1};
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
  if (!map_heads(&qn, a.q_nope, a.n_q, a.n_heads, 128, kTile) ||
      !map_heads(&qr, a.q_rope, a.n_q, a.n_heads, 64, kTile))
    return cudaErrorInvalidValue;
  if (a.n_k > 0) {
    if (!map_heads(&kn, a.k_nope, a.n_k, a.n_kv_heads, 128, kTile) ||
        !map_rows(&kr, a.k_rope, a.k_rope_stride, a.n_k) ||
        !map_heads(&v, a.v, a.n_k, a.n_kv_heads, 128, 64))
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
  const long kv_bytes = 512L * a.n_k * a.n_kv_heads / a.n_heads + 1;   // of one query head
  int group = a.n_heads;
  while (group > 1 && (a.n_heads % group || kv_bytes * group > (60L << 20))) --group;
  const long work = a.max_items * a.n_heads;
  const float scale_log2 = a.scale * 1.4426950408889634f;
  return launch_pdl(prompt_attn_kernel, dim3((unsigned)(work < sms ? work : sms)), dim3(kThreads),
                    kSmemBytes, s, qn, qr, kn, kr, v, a, scale_log2, group);
}

}  // namespace sm100
}  // namespace mla

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
constexpr int kWarpLoad = 8, kWarpMma = 9, kWarps = 12;
constexpr int kThreads = 32 * kWarps;
// Registers a thread: a softmax row keeps its 128 scores, the third warpgroup (two
// of its warps idle) needs few.  Launched with 65536 / 384 = 168 (a multiple of 8).
constexpr int kRegsSoftmax = 200, kRegsOther = 104;
static_assert(256 * kRegsSoftmax + 128 * kRegsOther <= kThreads * 168, "register split");
constexpr uint64_t kTimeoutNs = 2000000000ull;
constexpr uint32_t kSleepNs = 20000;

constexpr int kOffQ = 0;                          // [2 tiles][3 boxes]
constexpr int kOffRing = kOffQ + 6 * kChunk;
constexpr int kOffBar = kOffRing + kSlots * kChunk;
constexpr int kSmemBytes = kOffBar + 1024 + 1024;
static_assert(kSmemBytes <= 232448, "shared memory per CTA");

constexpr uint32_t kTmemS = 0, kTmemO = 256, kTmemCols = 512;   // tile t at + 128 t
constexpr uint32_t kIdescS = idesc_bf16(128, 128, 0, 0);
constexpr uint32_t kIdescPV = idesc_bf16(128, 128, 0, 1);       // V is [key][column]

// One (block of rows, head) pair on its way from the loading warp to the others.
struct Work {
  PromptItem it;
  int head;   // -1: no more work
};

struct Bars {
  uint64_t full[kSlots], empty[kSlots];
  uint64_t q_full[2], q_empty[2];
  uint64_t s_full[2];     // scores of the tile complete
  uint64_t p_full[2];     // P written (and O rescaled) by the tile's four warps
  uint64_t pv_done[2];    // O += P V complete
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
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  Bars *bars = reinterpret_cast<Bars *>(smem + kOffBar);
  const Ctx ctx{bars, a.err};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&bars->full[i], 1);
      mbar_init(&bars->empty[i], 1);
    }
    for (int t = 0; t < 2; ++t) {
      mbar_init(&bars->q_full[t], 1);
      mbar_init(&bars->q_empty[t], 1);
      mbar_init(&bars->s_full[t], 1);
      mbar_init(&bars->p_full[t], 4);
      mbar_init(&bars->pv_done[t], 1);
    }
    for (int i = 0; i < kSched; ++i) {
      mbar_init(&bars->w_full[i], 1);
      mbar_init(&bars->w_empty[i], 9);   // the MMA warp and the eight softmax warps
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
    int ns = 0;      // steps of this tile so far
    bool ok = true;
    Work w;
    for (int k = 0; ok && take(k, w); ++k) {
      const int rows = tile_rows(w.it, t);
      if (rows == 0) continue;
      const int steps = tile_steps(w.it, t);
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
        for (int c = 4; c < 128; c += 8) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            mx[i] = fmaxf(mx[i], c + 4 + i < 128 ? fmaxf(v[c + i], v[c + 4 + i]) : v[c + i]);
        }
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * scale_log2;
        const float m_new = top > m + 8.0f || m == -INFINITY ? top : m;
        const bool moved = m_new != m;
        const float base = m_new == -INFINITY ? 0.f : m_new;   // a row that sees nothing so far
        if (j > 0 && __any_sync(0xffffffffu, moved)) {
          const float f = moved ? ex2(m - base) : 1.f;
          l *= f;
          ok = __all_sync(0xffffffffu, wait_bar(ctx, &bars->pv_done[t], (ns - 1) & 1));
          if (!ok) break;
          tc_fence_after();
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
        float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t p[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const float a0 = ex2(fmaf(v[64 * h + 2 * i], scale_log2, -base));
            const float a1 = ex2(fmaf(v[64 * h + 2 * i + 1], scale_log2, -base));
            sum[(2 * i) & 3] += a0;
            sum[(2 * i + 1) & 3] += a1;
            p[i] = pack2(a0, a1);
          }
          tmem_st32(s_addr + 32 * h, p);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->p_full[t]);
        l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
      }
      if (!ok) break;
      // ---- the item's rows
      if (steps > 0) {
        ok = __all_sync(0xffffffffu, wait_bar(ctx, &bars->pv_done[t], (ns - 1) & 1));
        if (!ok) break;
        tc_fence_after();
      }
      const float inv = see > 0 ? 1.f / l : 0.f;
      const long at = (long)(w.it.q0 + t * kTile + row) * a.n_heads + w.head;
      if (row < rows && a.lse)
        a.lse[at] = see > 0 ? (m + __log2f(l)) * 0.6931471805599453f : -INFINITY;
      uint4 *dst = reinterpret_cast<uint4 *>(static_cast<bf16 *>(a.out) + at * 128);
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        float o[32];
        if (steps > 0) {
          tmem_ld32f(o_addr + 32 * c, o);
          tmem_wait_ld();
        }
        if (row < rows) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              x[e] = see > 0 ? pack2(o[8 * i + 2 * e] * inv, o[8 * i + 2 * e + 1] * inv) : 0u;
            dst[4 * c + i] = make_uint4(x[0], x[1], x[2], x[3]);
          }
        }
      }
      tc_fence_before();   // O is free: the next P of this tile says so to the MMA warp
    }
  } else {
    regs_lower<kRegsOther>();
    if (warp == kWarpLoad) {
      if (lane == 0) {
        const int rep = a.n_heads / a.n_kv_heads;
        const int items = a.hdr->items, total = items * a.n_heads;
        const int group_work = items * heads_per_group;
        int nl = 0, nq[2] = {0, 0};
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
          auto slot_for = [&]() -> int {
            const int s = nl % kSlots;
            if (nl >= kSlots && !wait_bar(ctx, &bars->empty[s], ((nl / kSlots) - 1) & 1)) return -1;
            ++nl;
            mbar_expect_tx(&bars->full[s], kChunk);
            return s;
          };
          auto load_k = [&](int j) -> bool {
            const int tok = w.it.k0 + j * kTile;
            for (int c = 0; c < 3; ++c) {
              const int s = slot_for();
              if (s < 0) return false;
              uint8_t *dst = smem + kOffRing + s * kChunk;
              if (c < 2)
                tma_load_3d(dst, &tm_kn, 64 * c, kv, tok, &bars->full[s]);
              else
                tma_load_2d(dst, &tm_kr, 0, tok, &bars->full[s]);
            }
            return true;
          };
          auto load_v = [&](int j) -> bool {
            for (int c = 0; c < 2; ++c) {
              const int s = slot_for();
              if (s < 0) return false;
              uint8_t *dst = smem + kOffRing + s * kChunk;
              const int tok = w.it.k0 + j * kTile + 64 * c;
              tma_load_3d(dst, &tm_v, 0, kv, tok, &bars->full[s]);
              tma_load_3d(dst + kChunk / 2, &tm_v, 64, kv, tok, &bars->full[s]);
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
          for (int i = max(0, nl - kSlots); i < nl; ++i)
            drain_bar(&bars->full[i % kSlots], (i / kSlots) & 1);
          for (int t = 0; t < 2; ++t)
            if (nq[t] > 0) drain_bar(&bars->q_full[t], (nq[t] - 1) & 1);
        }
      }
    } else if (warp == kWarpMma) {
      const uint64_t qd0 = sdesc(smem_u32(smem + kOffQ), 16, 1024, 2);
      const uint64_t kd0 = sdesc(smem_u32(smem + kOffRing), 16, 1024, 2);
      const uint64_t vd0 = sdesc(smem_u32(smem + kOffRing), kChunk / 2, 1024, 2);
      int nl = 0;               // ring chunks consumed (and released)
      int np[2] = {0, 0};       // P tiles consumed
      int nq[2] = {0, 0};       // Q tiles consumed
      auto wait = [&](uint64_t *bar, uint32_t parity) -> bool {
        const bool ok = wait_bar(ctx, bar, parity);
        return __all_sync(0xffffffffu, ok);
      };
      // S of tile t from the three ring chunks that start at chunk c0
      auto scores = [&](int t, int c0) -> bool {
        for (int c = 0; c < 3; ++c) {
          const int s = (c0 + c) % kSlots;
          if (!wait(&bars->full[s], ((c0 + c) / kSlots) & 1)) return false;
          tc_fence_after();
          if (elect_one()) {
            const uint64_t qd = qd0 + (uint64_t)(((3 * t + c) * kChunk) >> 4);
            const uint64_t kd = kd0 + (uint64_t)((s * kChunk) >> 4);
  #pragma unroll
            for (int k = 0; k < 4; ++k)
              umma_bf16(tmem + kTmemS + 128 * t, qd + (uint64_t)((32 * k) >> 4),
                        kd + (uint64_t)((32 * k) >> 4), kIdescS, (c | k) ? 1u : 0u);
          }
        }
        if (elect_one()) umma_commit(&bars->s_full[t]);
        __syncwarp();
        return true;
      };
      auto release = [&](int c0, int n) {
        if (elect_one())
          for (int c = 0; c < n; ++c) umma_commit(&bars->empty[(c0 + c) % kSlots]);
        __syncwarp();
      };
      // O of tile t += P V, V in the two chunks that start at c0; `left` keys of the step exist
      auto values = [&](int t, int c0, int left, bool zero, bool first) -> bool {
        for (int c = 0; c < 2; ++c) {
          const int s = (c0 + c) % kSlots;
          if (!wait(&bars->full[s], ((c0 + c) / kSlots) & 1)) return false;
          if (zero && left < 64 * (c + 1)) {
            // rows behind the sequence's last key belong to another sequence and
            // may hold anything: 0 * NaN must not reach O
            uint8_t *v = smem + kOffRing + s * kChunk;
            const int from = max(0, left - 64 * c);
            for (int i = lane; i < (64 - from) * 16; i += 32) {
              const int row = from + (i >> 4);
              *reinterpret_cast<uint4 *>(v + ((i >> 3) & 1) * (kChunk / 2) + row * 128 +
                                         (i & 7) * 16) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
            __syncwarp();
          }
        }
        if (!wait(&bars->p_full[t], np[t] & 1)) return false;
        ++np[t];
        tc_fence_after();
        if (elect_one()) {
  #pragma unroll
          for (int c = 0; c < 2; ++c) {
            const uint64_t vd = vd0 + (uint64_t)((((c0 + c) % kSlots) * kChunk) >> 4);
  #pragma unroll
            for (int k = 0; k < 4; ++k)
              umma_bf16_ts(tmem + kTmemO + 128 * t, tmem + kTmemS + 128 * t + 32 * c + 8 * k,
                           vd + (uint64_t)((2048 * k) >> 4), kIdescPV,
                           (first && c == 0 && k == 0) ? 0u : 1u);
          }
          umma_commit(&bars->pv_done[t]);
        }
        __syncwarp();
        return true;
      };
      int k = 0;
      int n_t[2] = {0, 0}, n = 0;
      Work w;
      // the next item that has any keys
      auto next_work = [&]() -> bool {
        while (take(k, w)) {
          ++k;
          n_t[0] = tile_steps(w.it, 0);
          n_t[1] = tile_steps(w.it, 1);
          n = max(n_t[0], n_t[1]);
          if (n > 0) return true;
        }
        return false;
      };
      // S of step 0 of the item's tile t
      auto first_scores = [&](int t) -> bool {
        if (n_t[t] == 0) return true;
        if (!wait(&bars->q_full[t], nq[t] & 1)) return false;
        ++nq[t];
        if (!scores(t, nl)) return false;
        if (n_t[t] == 1 && elect_one()) umma_commit(&bars->q_empty[t]);
        __syncwarp();
        return true;
      };
      bool more = next_work();
      bool ok = true;
      if (more) {
        ok = first_scores(0) && first_scores(1);
        if (ok) release(nl, 3);
        nl += 3;
      }
      while (more && ok) {
        const Work cur = w;
        const int steps = n, nt[2] = {n_t[0], n_t[1]};
        for (int j = 0; j < steps && ok; ++j) {
          const int v0 = nl, k0 = nl + 2;
          const bool last = j + 1 == steps;
          const int left = cur.it.lk - j * kTile;
          if (last) more = next_work();
          bool zero = left < kTile;
          if (last) nl = k0;      // first_scores reads the next item's keys there
          for (int t = 0; t < 2 && ok; ++t) {
            if (j < nt[t]) {
              ok = values(t, v0, left, zero, j == 0);
              zero = false;
            }
            if (!ok) break;
            if (!last && j + 1 < nt[t]) {
              ok = scores(t, k0);
              if (ok && j + 2 == nt[t] && elect_one()) umma_commit(&bars->q_empty[t]);
              __syncwarp();
            } else if (last && more) {
              ok = first_scores(t);
            }
          }
          if (!ok) break;
          release(v0, 2);
          if (!last || more) release(k0, 3);
          nl = last && !more ? k0 : k0 + 3;
        }
      }
      if (elect_one()) {
        umma_commit(&bars->drain);
        drain_bar(&bars->drain, 0);
      }
      __syncwarp();
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

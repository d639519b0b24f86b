// Causal attention of sequences with few queries (bf16; scores over 128 + 64 values,
// 128-wide values): the sequences of a packed call whose (token, head) pairs of a key
// head are 16 rows at most.  The formula is that of prompt_sm100.cu.
//
// Bound by the keys and values, which 16 rows at most share, so what counts is how many
// bytes are on their way.  A 128-row tcgen05 tile spent 3.7 us on each such block, step
// after step of a few hundred instructions that wait for one another (52 sequences of
// 1-2 tokens over 95 rows, 128 heads: 165 us, here 88; one token alone 7.6, here 3.7).  A
// CTA takes a (sequence, key head); each of its warps loads every second or eighth 16 keys
// by itself, two loads ahead (172 KB of a multiprocessor on their way), and keeps m, l and
// O of its keys in registers (mma.sync, one 16-row tile).  The warps are merged at the end
// in a fixed order.
#include "api_checks.h"
#include "prompt.h"

namespace mla {
namespace {

using bf16 = __nv_bfloat16;

constexpr int kChunk = 16;                   // keys of a warp's step
// Rows in shared memory, padded to an odd number of 16-byte units: eight rows of a
// matrix load lie in different banks.
constexpr int kLdK = (192 + 8) * 2, kLdV = (128 + 8) * 2;
constexpr int kStageBytes = kChunk * (kLdK + kLdV);
constexpr int kOffStage = kPromptFewRows * kLdK;
constexpr int kLdO = 132;                    // floats of a merged row
static_assert(kPromptFewRows * kLdO * 4 <= kStageBytes, "a warp's O takes the place of a stage");
static_assert(kPromptFewRows == 16 && kChunk == 16, "one m16n8k16 tile of rows, one k16 of keys");

__device__ __forceinline__ uint32_t smem_addr(const void *p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// 16 bytes, or zeros.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(real ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void load4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void load4t(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float pow2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}

template <int kWarps, int kStages, int kCtas>
__global__ void __launch_bounds__(32 * kWarps, kCtas)
    prompt_few_kernel(const PromptAttnArgs a, const float scale_log2) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float m_s[kWarps][kPromptFewRows], l_s[kWarps][kPromptFewRows];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rep = a.n_heads / a.n_kv_heads;
  const int b = blockIdx.x / a.n_kv_heads, kv = blockIdx.x % a.n_kv_heads;
  grid_dep_wait();
  grid_dep_launch();
  int q0, lq, k0, lk;
  if (!prompt_seq(a.cu_q, a.cu_k, a.n_q, a.n_k, b, q0, lq, k0, lk)) {
    if (kv == 0 && tid == 0) set_error(a.err, kErrRange);
    return;
  }
  if (lq == 0 || lq > a.few_tokens) return;
  const int rows = lq * rep, base = lk - lq + 1;   // token i sees the keys j < base + i
  const int chunks = (lk + kChunk - 1) / kChunk;

  // ---- a warp's chunk: 16 keys of 24 units and 16 values of 16 units of 16 bytes; keys
  // behind the sequence's last one are zeros
  const bf16 *kn = static_cast<const bf16 *>(a.k_nope.ptr) + kv * a.k_nope.head;
  const bf16 *kr = static_cast<const bf16 *>(a.k_rope);
  const bf16 *vp = static_cast<const bf16 *>(a.v.ptr) + kv * a.v.head;
  const uint32_t stage0 = smem_addr(smem + kOffStage) + warp * kStages * kStageBytes;
  auto fetch = [&](int c, int stage) {
    if (c < chunks) {
      const uint32_t ks = stage0 + stage * kStageBytes, vs = ks + kChunk * kLdK;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = 2 * i + (lane >> 4), u = lane & 15, j = c * kChunk + r;
        const bool real = j < lk;
        const long t = k0 + (real ? j : 0);
        copy16(ks + r * kLdK + 16 * u, kn + t * a.k_nope.token + 8 * u, real);
        copy16(vs + r * kLdV + 16 * u, vp + t * a.v.token + 8 * u, real);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = 4 * i + (lane >> 3), u = lane & 7, j = c * kChunk + r;
        const bool real = j < lk;
        copy16(ks + r * kLdK + 256 + 16 * u, kr + (k0 + (real ? j : 0)) * a.k_rope_stride + 8 * u,
               real);
      }
    }
    copies_commit();
  };
  // ---- the queries: row r is token r / rep, head kv rep + r % rep
  for (int i = tid; i < kPromptFewRows * 24; i += 32 * kWarps) {
    const int r = i / 24, u = i % 24, h = kv * rep + r % rep;
    const bool real = r < rows;
    const long t = q0 + (real ? r / rep : 0);
    const bf16 *src =
        u < 16 ? static_cast<const bf16 *>(a.q_nope.ptr) + t * a.q_nope.token +
                     h * a.q_nope.head + 8 * u
               : static_cast<const bf16 *>(a.q_rope.ptr) + t * a.q_rope.token +
                     h * a.q_rope.head + 8 * (u - 16);
    copy16(smem_addr(smem) + r * kLdK + 16 * u, src, real);
  }
  copies_commit();
  for (int s = 0; s < kStages; ++s) fetch(warp + s * kWarps, s);
  copies_wait<kStages>();
  __syncthreads();
  uint32_t q[12][4];
#pragma unroll
  for (int i = 0; i < 12; ++i)
    load4(q[i], smem_addr(smem) + (lane & 15) * kLdK + 32 * i + 16 * (lane >> 4));

  // A thread has rows g and g + 8, two neighbouring columns of every eight.
  const int g = lane >> 2, t2 = 2 * (lane & 3);
  const int see[2] = {base + g / rep, base + (g + 8) / rep};
  float o[16][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 16; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  int stage = 0;
  for (int c = warp; c < chunks; c += kWarps) {
    copies_wait<kStages - 1>();
    __syncwarp();
    const uint32_t ks = stage0 + stage * kStageBytes, vs = ks + kChunk * kLdK;
    float s[2][4] = {};
    const uint32_t kat = ks + ((lane >> 4) * 8 + (lane & 7)) * kLdK + 16 * ((lane >> 3) & 1);
#pragma unroll
    for (int i = 0; i < 12; ++i) {
      uint32_t k[4];
      load4(k, kat + 32 * i);
      mma16816(s[0], q[i], k[0], k[1]);
      mma16816(s[1], q[i], k[2], k[3]);
    }
    float p[2][4];
#pragma unroll
    for (int h = 0; h < 2; ++h) {      // row g, row g + 8
      float x[4];
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        const int j = c * kChunk + 8 * (n >> 1) + t2 + (n & 1);
        x[n] = j < min(see[h], lk) ? s[n >> 1][2 * h + (n & 1)] * scale_log2 : -INFINITY;
      }
      float top = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
      const float m_new = fmaxf(m[h], top);
      const float at = m_new == -INFINITY ? 0.f : m_new;    // a row that sees nothing so far
      const float f = pow2(m[h] - at);
      m[h] = m_new;
#pragma unroll
      for (int n = 0; n < 4; ++n) p[n >> 1][2 * h + (n & 1)] = pow2(x[n] - at);
      l[h] = l[h] * f + ((p[0][2 * h] + p[0][2 * h + 1]) + (p[1][2 * h] + p[1][2 * h + 1]));
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        o[i][2 * h] *= f;
        o[i][2 * h + 1] *= f;
      }
    }
    // the weights rounded to bf16 for the product (their sum is not), as in the tile kernel
    const uint32_t w[4] = {pack(p[0][0], p[0][1]), pack(p[0][2], p[0][3]), pack(p[1][0], p[1][1]),
                           pack(p[1][2], p[1][3])};
    const uint32_t vat = vs + (((lane >> 3) & 1) * 8 + (lane & 7)) * kLdV + 16 * (lane >> 4);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint32_t v[4];
      load4t(v, vat + 32 * i);
      mma16816(o[2 * i], w, v[0], v[1]);
      mma16816(o[2 * i + 1], w, v[2], v[3]);
    }
    __syncwarp();
    fetch(c + kStages * kWarps, stage);
    stage = stage + 1 == kStages ? 0 : stage + 1;
  }
  copies_wait<0>();
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
  }
  __syncthreads();       // every warp is through with its stages, which O takes the place of
  float *om = reinterpret_cast<float *>(smem + kOffStage) + warp * kPromptFewRows * kLdO;
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    *reinterpret_cast<float2 *>(om + g * kLdO + 8 * i + t2) = make_float2(o[i][0], o[i][1]);
    *reinterpret_cast<float2 *>(om + (g + 8) * kLdO + 8 * i + t2) = make_float2(o[i][2], o[i][3]);
  }
  if ((lane & 3) == 0) {
    m_s[warp][g] = m[0];
    m_s[warp][g + 8] = m[1];
    l_s[warp][g] = l[0];
    l_s[warp][g + 8] = l[1];
  }
  __syncthreads();

  // ---- merge: M = max m_w, out = sum_w 2^(m_w - M) O_w / sum_w 2^(m_w - M) l_w; a thread
  // has kCols columns of a row
  constexpr int kCols = kPromptFewRows * 128 / (32 * kWarps);
  const int r = tid / (128 / kCols), col = kCols * (tid % (128 / kCols));
  if (r >= rows) return;
  float top = -INFINITY, sum = 0.f, acc[kCols];
#pragma unroll
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, m_s[w][r]);
  const float at = top == -INFINITY ? 0.f : top;
#pragma unroll
  for (int i = 0; i < kCols; ++i) acc[i] = 0.f;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const float f = pow2(m_s[w][r] - at);
    sum = fmaf(f, l_s[w][r], sum);
    const float *src = reinterpret_cast<const float *>(smem + kOffStage) +
                       (w * kPromptFewRows + r) * kLdO + col;
#pragma unroll
    for (int i = 0; i < kCols; i += 4) {
      const float4 x = *reinterpret_cast<const float4 *>(src + i);
      acc[i] = fmaf(f, x.x, acc[i]);
      acc[i + 1] = fmaf(f, x.y, acc[i + 1]);
      acc[i + 2] = fmaf(f, x.z, acc[i + 2]);
      acc[i + 3] = fmaf(f, x.w, acc[i + 3]);
    }
  }
  const bool some = lk > 0 && base + r / rep > 0;      // the row sees a key
  const float inv = some ? 1.f / sum : 0.f;
  const long row = (long)(q0 + r / rep) * a.n_heads + kv * rep + r % rep;
  uint4 *out = reinterpret_cast<uint4 *>(static_cast<bf16 *>(a.out) + row * 128 + col);
#pragma unroll
  for (int i = 0; i < kCols / 8; ++i)
    out[i] = some ? make_uint4(pack(acc[8 * i] * inv, acc[8 * i + 1] * inv),
                               pack(acc[8 * i + 2] * inv, acc[8 * i + 3] * inv),
                               pack(acc[8 * i + 4] * inv, acc[8 * i + 5] * inv),
                               pack(acc[8 * i + 6] * inv, acc[8 * i + 7] * inv))
                  : make_uint4(0, 0, 0, 0);
  if (a.lse && col == 0)
    a.lse[row] = some ? (top + __log2f(sum)) * 0.6931471805599453f : -INFINITY;
}

template <int kWarps, int kStages, int kCtas>
cudaError_t launch(const PromptAttnArgs &a, cudaStream_t s) {
  constexpr int smem = kOffStage + kWarps * kStages * kStageBytes;
  static api::PerDeviceOnce once;
  const cudaError_t e = once.run([] {
    return cudaFuncSetAttribute(prompt_few_kernel<kWarps, kStages, kCtas>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  });
  if (e != cudaSuccess) return e;
  return launch_pdl(prompt_few_kernel<kWarps, kStages, kCtas>,
                    dim3((unsigned)a.batch * (unsigned)a.n_kv_heads), dim3(32 * kWarps), smem, s, a,
                    a.scale * 1.4426950408889634f);
}

}  // namespace

cudaError_t launch_prompt_few(const PromptAttnArgs &a, cudaStream_t s) {
  // A CTA on a multiprocessor, eight warps on its keys, where there are no more CTAs than
  // that or their keys are many; else four CTAs of two warps, so that one computes while
  // another's first loads are on their way.  (1 token over 4001 rows, 128 heads: 50 us
  // and 83; 64 x 1 token over 100-2000 rows, 8 key heads: 64 and 73; 52 x 1-2 tokens over 95
  // rows, 128 heads: 172 and 88; 64 x 1-16 tokens over 100-200 rows: 270 and 153.)
  // The host knows the keys' average alone, and the border lies where lengths differ: 64 x 1
  // token over 20 to twice the average, 16 heads, takes 47.9 us and 40.0 at an average of
  // 300, 62.2 and 57.5 at 512, 67.6 and 71.7 at 600, 84 and 92 at 830; in 4 key heads 21.8 and
  // 32.8 at 512; 61 over 60 rows beside 3 over 11581 127 and 274.  Equal lengths would go on with
  // two warps: 61.6 and 49.4 at 512 each, 98 and 88 at 1024.
  const long ctas = (long)a.batch * a.n_kv_heads;
  return ctas <= kPromptSms || a.n_k >= 512L * a.batch ? launch<8, 2, 1>(a, s) : launch<2, 2, 4>(a, s);
}

}  // namespace mla

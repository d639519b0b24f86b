// Prompt operators on CUDA cores: cache append of packed rows (RMSNorm, RoPE,
// paged write, query rotation), cache gather, the plan of the packed
// attention, and the fp32 validation attention.
#include "api_checks.h"
#include "common.cuh"
#include "prompt.h"

namespace mla {
namespace {

using bf16 = __nv_bfloat16;

// The sequence b with cu[b] <= t < cu[b + 1], by one warp (every lane gets the
// result): the number of cu[1 .. batch] that are <= t, found 32 probes at a
// time.  -1 when no sequence holds t; offsets that do not ascend end up there
// or at a sequence that does hold t.
__device__ __forceinline__ int warp_find_seq(const int32_t *cu, int batch, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = batch;  // the count is in [lo, lo + n]
  while (n > 0) {
    const int step = (n + 31) / 32;
    const int at = lo + min(n, (lane + 1) * step);
    const unsigned below = __ballot_sync(0xffffffffu, cu[at] <= t);
    const int k = __popc(below);  // lanes whose probe is <= t
    if (step == 1) {
      lo += min(n, k);
      break;
    }
    const int skip = min(n, k * step);
    lo += skip;
    n = min(n - skip, step - 1);
  }
  if (lo >= batch || t < cu[lo] || t >= cu[lo + 1]) return -1;
  return lo;
}

// Records offsets that do not ascend or that leave the n packed rows (rows that some sequence
// holds are handled all the same).  The work of a block of its own, the launch's first: in
// the warps that have rows to move it cost a small call 0.1-0.2 us, here 0.02-0.1.
__device__ __forceinline__ void check_offsets(const int32_t *cu, int batch, int n, int *err) {
  for (long b = threadIdx.x; b < batch; b += blockDim.x)
    if (cu[b] < 0 || cu[b + 1] < cu[b] || cu[b + 1] > n) set_error(err, kErrRange);
}

// The page and slot of row `pos` of sequence b; page -1 when out of range.
__device__ __forceinline__ int page_of(const int32_t *table, int max_pages, int num_pages,
                                       int page_size, int b, long pos) {
  if (pos < 0 || pos >= (long)max_pages * page_size) return -1;
  const int page = table[(long)b * max_pages + pos / page_size];
  return page >= 0 && page < num_pages ? page : -1;
}

__device__ __forceinline__ void unpack8(const uint4 &u, float *f) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float *f) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t *>(&v);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// 8 values as loaded, turned into floats where they are needed.
template <class X>
struct Raw8;
template <>
struct Raw8<bf16> {
  uint4 v;
  __device__ __forceinline__ void load(const bf16 *p) { v = *reinterpret_cast<const uint4 *>(p); }
  __device__ __forceinline__ void get(float *f) const { unpack8(v, f); }
};
template <>
struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float *p) {
    a = reinterpret_cast<const float4 *>(p)[0];
    b = reinterpret_cast<const float4 *>(p)[1];
  }
  __device__ __forceinline__ void get(float *f) const {
    reinterpret_cast<float4 *>(f)[0] = a;
    reinterpret_cast<float4 *>(f)[1] = b;
  }
};

// ---------------------------------------------------------------------------
// Cache append of packed rows
// ---------------------------------------------------------------------------

__global__ void prompt_append_f32(PromptAppendArgs a, RopeParams rp) {
  __shared__ float cs[64], sn[64], red[32];
  __shared__ float inv_rms;
  grid_dep_wait();
  if (blockIdx.x == 0) return check_offsets(a.cu, a.batch, a.n_tokens, a.err);
  const int t = blockIdx.x - 1, half = rp.d_rope / 2, row = a.d_c + rp.d_rope;
  const int b = warp_find_seq(a.cu, a.batch, t);
  if (b < 0) {
    // tokens outside [cu[0], cu[batch]) are not there; one inside that no
    // sequence holds means offsets that do not ascend
    if (threadIdx.x == 0 && t >= a.cu[0] && t < a.cu[a.batch]) set_error(a.err, kErrRange);
    return;
  }
  const long pos = (long)(a.ctx ? a.ctx[b] : 0) + (t - a.cu[b]);
  const int page = page_of(a.block_table, a.max_pages, a.num_pages, a.page_size, b, pos);
  if (pos < 0 || pos > 0x7fffffffL) {
    if (threadIdx.x == 0) set_error(a.err, kErrRange);
    return;
  }
  for (int i = threadIdx.x; i < half; i += blockDim.x)
    rope_cos_sin((int)pos, rp.theta[i], cs[i], sn[i]);
  const float *x = static_cast<const float *>(a.x) + t * a.x_stride;
  float ss = 0.f;
  for (int i = threadIdx.x; i < a.d_c; i += blockDim.x) ss += x[i] * x[i];
  ss = warp_sum(ss);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = ss;
  __syncthreads();
  if (threadIdx.x < 32) {
    const float v = warp_sum(threadIdx.x < (blockDim.x >> 5) ? red[threadIdx.x] : 0.f);
    if (threadIdx.x == 0) inv_rms = 1.0f / sqrtf(v / (float)a.d_c + (float)a.eps);
  }
  __syncthreads();
  if (page < 0) {
    if (threadIdx.x == 0) set_error(a.err, kErrRange);
  } else {
    float *dst = static_cast<float *>(a.pool) + ((long)page * a.page_size + pos % a.page_size) * row;
    const float *gamma = static_cast<const float *>(a.gamma);
    for (int i = threadIdx.x; i < a.d_c; i += blockDim.x) dst[i] = gamma[i] * (x[i] * inv_rms);
    for (int i = threadIdx.x; i < half; i += blockDim.x) {
      int j0, j1;
      rope_idx(rp, i, j0, j1);
      float x0 = x[a.d_c + j0], x1 = x[a.d_c + j1];
      rope_rotate(cs[i], sn[i], x0, x1);
      dst[a.d_c + j0] = x0;
      dst[a.d_c + j1] = x1;
    }
  }
  if (!a.q.ptr) return;
  const float *q = static_cast<const float *>(a.q.ptr) + t * a.q.token;
  float *qo = static_cast<float *>(const_cast<void *>(a.q_out.ptr)) + t * a.q_out.token;
  for (int k = threadIdx.x; k < a.n_heads * half; k += blockDim.x) {
    const int h = k / half, i = k % half;
    int j0, j1;
    rope_idx(rp, i, j0, j1);
    float x0 = q[h * a.q.head + j0], x1 = q[h * a.q.head + j1];
    rope_rotate(cs[i], sn[i], x0, x1);
    qo[h * a.q_out.head + j0] = x0;
    qo[h * a.q_out.head + j1] = x1;
  }
}

constexpr int kSlab = 32;  // heads a warp rotates per round: 4 units of 8 pairs a lane

// A token is the work of `group` warps: the last one normalises, rotates and
// writes the cache row, the others rotate the heads.  Every warp finds its
// token's sequence and evaluates the 32 angles (one a lane) by itself, so
// nothing is shared between warps and nothing waits.  Bound by the bytes (a token
// of 128 heads moves 34.5 KB), so a warp asks for its first 4 KB before it looks
// for the sequence.
//
// A unit is 8 rotation pairs = two 16-byte vectors of a 64-wide head:
// interleaved pairs (vectors 2u, 2u + 1) or split halves (vectors u, u + 4).  Lane l
// handles unit l % 4, so its 8 cosines and sines stay in registers for all heads.
template <bool kI8, class X>
__global__ void prompt_append_bf16(PromptAppendArgs a, const __grid_constant__ RopeParams rp,
                                   int group) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = ((int)blockIdx.x - 1) * (int)(blockDim.x / 32 / group) + warp / group;
  const int role = warp % group;
  const int u = lane & 3;
  const int v0 = rp.half ? u : 2 * u, v1 = rp.half ? u + 4 : 2 * u + 1;
  grid_dep_wait();
  if (blockIdx.x == 0) return check_offsets(a.cu, a.batch, a.n_tokens, a.err);
  if (t >= a.n_tokens) return;
  uint4 p[4], r[4];
  const bf16 *q = static_cast<const bf16 *>(a.q.ptr) + t * a.q.token;
  auto load = [&](int h0) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int h = h0 + 8 * k + (lane >> 2);
      if (h < a.n_heads) {
        const uint4 *src = reinterpret_cast<const uint4 *>(q + h * a.q.head);
        p[k] = src[v0];
        r[k] = src[v1];
      }
    }
  };
  Raw8<X> rc[2], rr[2];
  if (role < group - 1) {
    load(role * kSlab);
  } else {
    const X *x = static_cast<const X *>(a.x) + t * a.x_stride;
    rc[0].load(x + 8 * lane);
    rc[1].load(x + 256 + 8 * lane);
    rr[0].load(x + 512 + 8 * v0);
    rr[1].load(x + 512 + 8 * v1);
  }
  const int b = warp_find_seq(a.cu, a.batch, t);
  if (b < 0) {
    if (lane == 0 && t >= a.cu[0] && t < a.cu[a.batch]) set_error(a.err, kErrRange);
    return;
  }
  const long pos = (long)(a.ctx ? a.ctx[b] : 0) + (t - a.cu[b]);
  if (pos < 0 || pos > 0x7fffffffL) {
    if (lane == 0) set_error(a.err, kErrRange);
    return;
  }
  float cf, sf;
  rope_cos_sin((int)pos, rp.theta[lane], cf, sf);
  float cs[8], sn[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    cs[i] = __shfl_sync(0xffffffffu, cf, 8 * u + i);
    sn[i] = __shfl_sync(0xffffffffu, sf, 8 * u + i);
  }
  auto turn = [&](float (&f)[16]) {     // the unit's two vectors
    if (rp.half) {
#pragma unroll
      for (int i = 0; i < 8; ++i) rope_rotate(cs[i], sn[i], f[i], f[8 + i]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) rope_rotate(cs[i], sn[i], f[2 * i], f[2 * i + 1]);
    }
  };

  if (role < group - 1) {
    bf16 *qo = static_cast<bf16 *>(const_cast<void *>(a.q_out.ptr)) + t * a.q_out.token;
    for (int h0 = role * kSlab; h0 < a.n_heads;) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int h = h0 + 8 * k + (lane >> 2);
        if (h < a.n_heads) {
          float f[16];
          unpack8(p[k], f);
          unpack8(r[k], f + 8);
          turn(f);
          uint4 *dst = reinterpret_cast<uint4 *>(qo + h * a.q_out.head);
          dst[v0] = pack8(f);
          dst[v1] = pack8(f + 8);
        }
      }
      h0 += (group - 1) * kSlab;
      load(h0);
    }
    return;
  }

  // the cache row: lane l holds latent values [8 l, 8 l + 8) and [256 + 8 l, 256 + 8 l + 8),
  // lanes 0..3 also one unit of k_R
  const int page = page_of(a.block_table, a.max_pages, a.num_pages, a.page_size, b, pos);
  if (page < 0) {
    if (lane == 0) set_error(a.err, kErrRange);
    return;
  }
  const uint4 *g = static_cast<const uint4 *>(a.gamma);
  float c[16], gm[16], xr[16];
  rc[0].get(c);
  rc[1].get(c + 8);
  rr[0].get(xr);
  rr[1].get(xr + 8);
  unpack8(g[lane], gm);
  unpack8(g[32 + lane], gm + 8);
  turn(xr);
  const uint4 kp = pack8(xr), kr = pack8(xr + 8);
  const long slot = (long)page * a.page_size + pos % a.page_size;
  if (!kI8) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) ss += c[i] * c[i];
    const float inv = 1.0f / sqrtf(warp_sum(ss) / 512.f + (float)a.eps);
#pragma unroll
    for (int i = 0; i < 16; ++i) c[i] = gm[i] * (c[i] * inv);
    uint4 *dst = reinterpret_cast<uint4 *>(static_cast<bf16 *>(a.pool) + slot * 576);
    dst[lane] = pack8(c);
    dst[32 + lane] = pack8(c + 8);
    if (lane < 4) {
      dst[64 + v0] = kp;
      dst[64 + v1] = kr;
    }
  } else {
    // In 64 bits: a code is a rounding of c / 2^e, and a 32-bit c next to a
    // border between two codes would fall on the wrong side of it.  Some 50 such
    // operations a lane, which cost more than the row's bytes: 8,192 rows take 14.9 us
    // without queries and 53.8 with those of 128 heads, bf16 rows 10.0 and 46.1; 65,536 rows
    // 104 us, bf16 rows 66.
    double ss = 0.0;
#pragma unroll
    for (int i = 0; i < 16; ++i) ss += (double)c[i] * (double)c[i];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
    const double inv = 1.0 / sqrt(ss / 512.0 + a.eps);
    double d[16], am = 0.0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      d[i] = (double)gm[i] * (double)c[i] * inv;
      am = fmax(am, isfinite(d[i]) ? fabs(d[i]) : HUGE_VAL);     // (fmax alone drops NaN)
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) am = fmax(am, __shfl_xor_sync(0xffffffffu, am, o));
    // am in [2^k, 2^(k+1)): 127 * 2^(k-6) = 1.98 * 2^k, so e is k - 6 or k - 5
    const bool finite = am < HUGE_VAL;      // else the row's scale is NaN, and every c read from it
    int e = 0;
    if (finite && am > 0.0) {
      e = ilogb(am) - 6;
      if (am > ldexp(127.0, e)) ++e;
    }
    const double inv_s = ldexp(1.0, -e);
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int q = finite ? max(-127, min(127, __double2int_rn(d[i] * inv_s))) : 0;
      w[i >> 2] |= (uint32_t)(q & 255) << (8 * (i & 3));
    }
    uint4 *dst = reinterpret_cast<uint4 *>(static_cast<uint8_t *>(a.pool) + slot * 656);
    reinterpret_cast<uint2 *>(dst)[lane] = make_uint2(w[0], w[1]);
    reinterpret_cast<uint2 *>(dst)[32 + lane] = make_uint2(w[2], w[3]);
    if (lane < 4) {
      dst[32 + v0] = kp;
      dst[32 + v1] = kr;
    }
    if (lane == 4)
      dst[40] = make_uint4(finite ? __float_as_uint(ldexpf(1.f, e)) : 0x7fc00000u, 0, 0, 0);
  }
}

// ---------------------------------------------------------------------------
// Cache gather: packed rows out of the pages
// ---------------------------------------------------------------------------

// One warp a row.  A row without a place in the cache is zeroed.
__global__ void gather_f32(GatherArgs a, int row) {
  const int t = ((int)blockIdx.x - 1) * (int)(blockDim.x >> 5) + (int)(threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  grid_dep_wait();
  if (blockIdx.x == 0) return check_offsets(a.cu, a.batch, a.n_rows, a.err);
  if (t >= a.n_rows) return;
  const int b = warp_find_seq(a.cu, a.batch, t);
  long src = -2;
  if (b >= 0) {
    const long pos = (long)(a.first ? a.first[b] : 0) + (t - a.cu[b]);
    const int page = page_of(a.block_table, a.max_pages, a.num_pages, a.page_size, b, pos);
    if (page >= 0) src = (long)page * a.page_size + pos % a.page_size;
  } else if (t < a.cu[0] || t >= a.cu[a.batch]) {
    return;
  }
  if (src < 0 && lane == 0) set_error(a.err, kErrRange);
  const float *p = static_cast<const float *>(a.pool) + (src < 0 ? 0 : src) * row;
  float *o = static_cast<float *>(a.rows) + (long)t * row;
  for (int i = lane; i < row; i += 32) o[i] = src < 0 ? 0.f : p[i];
}

// 8 int8 codes times the power-of-two scale s, as 8 bf16 values.  The byte q + 128
// in the low mantissa bits of 2^23 makes the float 2^23 + q + 128, so one fma gives
// q s, which has 8 significant bits at most: exact in fp32 and in bf16.
__device__ __forceinline__ uint4 codes8(const uint2 &in, float s) {
  const float bias = -8388736.0f * s;
  const uint32_t w[2] = {in.x ^ 0x80808080u, in.y ^ 0x80808080u};
  float f[8];
#pragma unroll
  for (int i = 0; i < 8; ++i)
    f[i] = fmaf(__uint_as_float(__byte_perm(w[i >> 2], 0x4B000000u, 0x7540u + (i & 3))), s, bias);
  return pack8(f);
}

constexpr int kGatherRows = 2;  // rows of a warp, all asked for before the first is written

// One warp two rows (one or four: 5 % slower for bf16 or for int8 rows): a pass of reads and
// writes, bound by the bytes.
template <bool kI8>
__global__ void gather_bf16(GatherArgs a) {
  const int lane = threadIdx.x & 31;
  const int t0 = (((int)blockIdx.x - 1) * (int)(blockDim.x >> 5) + (int)(threadIdx.x >> 5)) *
                 kGatherRows;
  grid_dep_wait();
  if (blockIdx.x == 0) return check_offsets(a.cu, a.batch, a.n_rows, a.err);
  if (t0 >= a.n_rows) return;
  // the first row's sequence by the whole warp, then lane i looks for row i's place
  const int b0 = warp_find_seq(a.cu, a.batch, t0);
  long mine = -1;
  const int t = t0 + lane;
  if (lane < kGatherRows && t < a.n_rows) {
    int b = max(b0, 0);
    while (b + 1 < a.batch && t >= a.cu[b + 1]) ++b;
    if (t >= a.cu[b] && t < a.cu[b + 1]) {
      const long pos = (long)(a.first ? a.first[b] : 0) + (t - a.cu[b]);
      const int page = page_of(a.block_table, a.max_pages, a.num_pages, a.page_size, b, pos);
      mine = page < 0 ? -2 : (long)page * a.page_size + pos % a.page_size;
    } else if (t >= a.cu[0] && t < a.cu[a.batch]) {
      mine = -2;
    }
    if (mine == -2) set_error(a.err, kErrRange);
  }
  long src[kGatherRows];
#pragma unroll
  for (int i = 0; i < kGatherRows; ++i) src[i] = __shfl_sync(0xffffffffu, mine, i);
  // lane l writes vectors l, 32 + l and (l < 8) 64 + l of a row, whole lines at a time
  uint4 x[kGatherRows][3];
  uint2 y[kGatherRows][2];
  float s[kGatherRows];
#pragma unroll
  for (int i = 0; i < kGatherRows; ++i) {
#pragma unroll
    for (int k = 0; k < 3; ++k) x[i][k] = make_uint4(0, 0, 0, 0);
    y[i][0] = y[i][1] = make_uint2(0x80808080u, 0x80808080u);
    s[i] = 0.f;
    if (src[i] < 0) continue;
    const uint8_t *p = static_cast<const uint8_t *>(a.pool) + src[i] * (kI8 ? 656 : 1152);
    const uint4 *v = reinterpret_cast<const uint4 *>(p);
    if (kI8) {
      const uint2 *c = reinterpret_cast<const uint2 *>(p);
      y[i][0] = c[lane];
      y[i][1] = c[32 + lane];
      if (lane < 8) x[i][2] = v[32 + lane];
      s[i] = *reinterpret_cast<const float *>(p + 640);
    } else {
      x[i][0] = v[lane];
      x[i][1] = v[32 + lane];
      if (lane < 8) x[i][2] = v[64 + lane];
    }
  }
#pragma unroll
  for (int i = 0; i < kGatherRows; ++i) {
    if (src[i] == -1) continue;      // a row that no sequence has; one without a page is zeroed
    uint4 *o = reinterpret_cast<uint4 *>(static_cast<bf16 *>(a.rows) + (long)(t0 + i) * 576);
    o[lane] = kI8 ? codes8(y[i][0], s[i]) : x[i][0];
    o[32 + lane] = kI8 ? codes8(y[i][1], s[i]) : x[i][1];
    if (lane < 8) o[64 + lane] = x[i][2];
  }
}

// ---------------------------------------------------------------------------
// Plan of the packed attention: the query blocks, most keys first
// ---------------------------------------------------------------------------
//
// Blocks are laid out by a counting sort on the keys that their last row sees,
// in kBins equal steps, so that the blocks which take longest start first and
// the short ones fill the end.
constexpr int kBins = 1024;

__global__ void __launch_bounds__(1024) prompt_plan_kernel(PromptPlanArgs a) {
  __shared__ int bins[kBins], warp_tot[32], top_s;
  const int tid = threadIdx.x, lane = tid & 31;
  grid_dep_wait();
  grid_dep_launch();
  for (int i = tid; i < kBins; i += blockDim.x) bins[i] = 0;
  if (tid == 0) top_s = 1;
  __syncthreads();
  // a sequence is walked by one warp, a block by one lane
  auto each = [&](auto &&f) {
    for (int b = tid >> 5; b < a.batch; b += blockDim.x >> 5) {
      int q0, lq, k0, lk;
      if (!prompt_seq(a.cu_q, a.cu_k, a.n_q, a.n_k, b, q0, lq, k0, lk)) {
        if (lane == 0) set_error(a.err, kErrRange);
        continue;
      }
      if (lq <= a.few_tokens) continue;
      for (int r = lane * a.tile; r < lq; r += 32 * a.tile) {
        const PromptItem it = prompt_item(q0, lq, k0, lk, r, a.tile);
        f(it, prompt_keys(it));
      }
    }
  };
  int top = 1;
  for (int b = tid; b < a.batch; b += blockDim.x) {
    int q0, lq, k0, lk;
    if (prompt_seq(a.cu_q, a.cu_k, a.n_q, a.n_k, b, q0, lq, k0, lk) && lq > a.few_tokens)
      top = max(top, lk);
  }
  atomicMax(&top_s, top);
  __syncthreads();
  top = top_s;
  auto bin_of = [&](int keys) { return kBins - 1 - (int)((long)keys * (kBins - 1) / top); };
  each([&](const PromptItem &, int keys) { atomicAdd(&bins[bin_of(keys)], 1); });
  __syncthreads();
  // exclusive scan of the bins (one a thread)
  const int n = bins[tid];
  int v = n;
  for (int o = 1; o < 32; o <<= 1) {
    const int w = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += w;
  }
  if (lane == 31) warp_tot[tid >> 5] = v;
  __syncthreads();
  if (tid < 32) {
    int w = warp_tot[tid];
    for (int o = 1; o < 32; o <<= 1) {
      const int z = __shfl_up_sync(0xffffffffu, w, o);
      if (tid >= o) w += z;
    }
    warp_tot[tid] = w;
  }
  __syncthreads();
  const int incl = v + ((tid >> 5) ? warp_tot[(tid >> 5) - 1] : 0);
  bins[tid] = incl - n;
  if (tid == kBins - 1) {
    a.hdr->items = min(incl, a.max_items);
  }
  __syncthreads();
  each([&](const PromptItem &it, int keys) {
    const int at = atomicAdd(&bins[bin_of(keys)], 1);
    if (at < a.max_items) a.items[at] = it;
  });
}

// ---------------------------------------------------------------------------
// fp32 attention over packed sequences (validation path)
// ---------------------------------------------------------------------------

constexpr int kSimtKeys = 32;

// Block `at` of the call's blocks in the order of the sequences (false: there are fewer),
// found by the CTA's 128 threads, a thread a sequence: its blocks are counted and summed
// up.  (A plan of all blocks by a launch of its own cost 5 us more than this.)
__device__ __forceinline__ bool simt_block(const PromptAttnArgs &a, int at, PromptItem &it) {
  __shared__ PromptItem found;
  __shared__ int warp_tot[4];
  const int tid = threadIdx.x, lane = tid & 31;
  int before = 0;      // blocks of the sequences before
  for (int b0 = 0; b0 < a.batch; b0 += 128) {
    const int b = b0 + tid;
    int q0, lq, k0, lk, n = 0;
    if (b < a.batch) {
      if (prompt_seq(a.cu_q, a.cu_k, a.n_q, a.n_k, b, q0, lq, k0, lk))
        n = (lq + kPromptTileSimt - 1) / kPromptTileSimt;
      else if (at == 0)
        set_error(a.err, kErrRange);
    }
    int v = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += x;
    }
    if (lane == 31) warp_tot[tid >> 5] = v;
    __syncthreads();
    int first = before + v - n, all = before;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      first += i < (tid >> 5) ? warp_tot[i] : 0;
      all += warp_tot[i];
    }
    if (at >= first && at < first + n)
      found = prompt_item(q0, lq, k0, lk, (at - first) * kPromptTileSimt, kPromptTileSimt);
    __syncthreads();
    // block 0 looks at every sequence's offsets
    if (at < all && (at > 0 || b0 + 128 >= a.batch)) {
      it = found;
      return true;
    }
    before = all;
  }
  return false;
}

// One block of 16 rows of one head per CTA (128 threads), 32 keys at a time
// through shared memory, one pass with the running maximum and sum.  Small sizes are
// bound by the chain of a step: loads, scores (a warp's four rows side by side), two
// reductions, O (4 x 64 tokens behind 64 rows, 8 heads: 13.1 us, 20.9 a row at a time and
// with a division per loaded value).
__global__ void __launch_bounds__(128) prompt_attn_simt(PromptAttnArgs a) {
  extern __shared__ float sm[];
  const int dq = a.d_nope + a.d_rope, ldk = dq + 1;
  float *qs = sm;                           // [16][dq]
  float *ks = qs + kPromptTileSimt * dq;    // [32][dq + 1]
  float *vs = ks + kSimtKeys * ldk;         // [32][d_v]
  float *ps = vs + kSimtKeys * a.d_v;       // [16][33]
  __shared__ float m_s[kPromptTileSimt], l_s[kPromptTileSimt], f_s[kPromptTileSimt];
  grid_dep_wait();
  grid_dep_launch();
  PromptItem it;
  if (!simt_block(a, blockIdx.x, it)) return;
  const int h = blockIdx.y, kv = h / (a.n_heads / a.n_kv_heads), tid = threadIdx.x;
  const float *qn = static_cast<const float *>(a.q_nope.ptr) + h * a.q_nope.head;
  const float *qr = static_cast<const float *>(a.q_rope.ptr) + h * a.q_rope.head;
  const float *kn = static_cast<const float *>(a.k_nope.ptr) + kv * a.k_nope.head;
  const float *kr = static_cast<const float *>(a.k_rope);
  const float *vp = static_cast<const float *>(a.v.ptr) + kv * a.v.head;
  // rows x width values into shared memory, four of a thread asked for at a time; the
  // next one's place by addition (a division each took longer than the loads)
  auto fill = [&](float *dst, int rows, int width, int ld, auto &&get) {
    const int dr = 128 / width, dc = 128 % width;
    int r = tid / width, c = tid % width;
    while (r < rows) {
      float x[4];
      int at[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        at[u] = r < rows ? r * ld + c : -1;
        if (r < rows) x[u] = get(r, c);
        r += dr;
        c += dc;
        if (c >= width) {
          c -= width;
          ++r;
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (at[u] >= 0) dst[at[u]] = x[u];
    }
  };
  fill(qs, kPromptTileSimt, dq, dq, [&](int r, int c) {     // (rows that are not there: zeros)
    const long t = it.q0 + r;
    return r >= it.rows ? 0.f
           : c < a.d_nope ? qn[t * a.q_nope.token + c]
                          : qr[t * a.q_rope.token + c - a.d_nope];
  });
  if (tid < kPromptTileSimt) {
    m_s[tid] = -INFINITY;
    l_s[tid] = 0.f;
  }
  const int cols = (a.d_v + 7) / 8;  // a thread: row tid / 8, values tid % 8 + 8 j
  float acc[32];
#pragma unroll
  for (int j = 0; j < 32; ++j) acc[j] = 0.f;
  const int r_o = tid >> 3, c_o = tid & 7;
  const int keys = prompt_keys(it);
  for (int j0 = 0; j0 < keys; j0 += kSimtKeys) {
    const int nk = min(kSimtKeys, keys - j0);
    __syncthreads();
    fill(ks, nk, dq, ldk, [&](int j, int c) {
      const long t = it.k0 + j0 + j;
      return c < a.d_nope ? kn[t * a.k_nope.token + c] : kr[t * a.k_rope_stride + c - a.d_nope];
    });
    fill(vs, nk, a.d_v, a.d_v, [&](int j, int c) { return vp[(it.k0 + j0 + j) * a.v.token + c]; });
    __syncthreads();
    // scores: warp w has rows w, w + 4, w + 8 and w + 12, side by side; lane = key
    constexpr int kMine = kPromptTileSimt / 4;
    const int j = tid & 31, w = tid >> 5;
    float x[kMine] = {}, top[kMine], p[kMine], sum[kMine];
    bool seen[kMine];
    if (j < nk)
      for (int c = 0; c < dq; ++c) {
        const float k = ks[j * ldk + c];
#pragma unroll
        for (int i = 0; i < kMine; ++i) x[i] = fmaf(qs[(w + 4 * i) * dq + c], k, x[i]);
      }
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      const int r = w + 4 * i;
      seen[i] = r < it.rows && j < nk && j0 + j < it.see + r;
      x[i] = seen[i] ? x[i] * a.scale : -INFINITY;
      top[i] = x[i];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
#pragma unroll
      for (int i = 0; i < kMine; ++i)
        top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], o));
    }
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      top[i] = fmaxf(m_s[w + 4 * i], top[i]);
      const float base = top[i] == -INFINITY ? 0.f : top[i];
      p[i] = seen[i] ? expf(x[i] - base) : 0.f;
      sum[i] = p[i];
      ps[(w + 4 * i) * 33 + j] = p[i];
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
#pragma unroll
      for (int i = 0; i < kMine; ++i) sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], o);
    }
    if (j < kMine) {      // lane i keeps row w + 4 i's numbers
      float t = top[0], s = sum[0];
#pragma unroll
      for (int i = 1; i < kMine; ++i) {
        t = j == i ? top[i] : t;
        s = j == i ? sum[i] : s;
      }
      const int r = w + 4 * j;
      const float f = expf(m_s[r] - (t == -INFINITY ? 0.f : t));
      f_s[r] = f;
      l_s[r] = l_s[r] * f + s;
      m_s[r] = t;
    }
    __syncthreads();
    // a row adds up only the keys it sees: a masked value is never multiplied
    const float f = f_s[r_o];
    const int mine = max(0, min(nk, it.see + r_o - j0));
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      if (j >= cols) break;
      const int c = c_o + 8 * j;
      if (c >= a.d_v) continue;
      float o = acc[j] * f;
#pragma unroll 4
      for (int k = 0; k < mine; ++k) o = fmaf(ps[r_o * 33 + k], vs[k * a.d_v + c], o);
      acc[j] = o;
    }
  }
  __syncthreads();
  if (r_o >= it.rows) return;
  const bool some = min(it.lk, it.see + r_o) > 0;      // the row sees a key
  const float l = l_s[r_o], inv = some ? 1.f / l : 0.f;
  const long at = (long)(it.q0 + r_o) * a.n_heads + h;
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    const int c = c_o + 8 * j;
    if (j < cols && c < a.d_v) static_cast<float *>(a.out)[at * a.d_v + c] = acc[j] * inv;
  }
  if (a.lse && c_o == 0) a.lse[at] = some ? m_s[r_o] + logf(l) : -INFINITY;
}

}  // namespace

cudaError_t launch_prompt_append_f32(const PromptAppendArgs &a, const RopeParams &rp,
                                     cudaStream_t s) {
  return launch_pdl(prompt_append_f32, dim3(1u + a.n_tokens), dim3(128), 0, s, a, rp);
}

cudaError_t launch_prompt_append_bf16(const PromptAppendArgs &a, const RopeParams &rp,
                                      bool int8_rows, cudaStream_t s) {
  int group = 1;  // warps a token
  if (a.q.ptr) {
    const int slabs = (a.n_heads + kSlab - 1) / kSlab;
    group += slabs < 8 ? slabs : 8;
  }
  const int per = group >= 8 ? 1 : 8 / group;
  const dim3 grid(1u + (a.n_tokens + per - 1) / per), block(32 * per * group);   // (1: check_offsets)
  if (a.x_f32)
    return int8_rows
               ? launch_pdl(prompt_append_bf16<true, float>, grid, block, 0, s, a, rp, group)
               : launch_pdl(prompt_append_bf16<false, float>, grid, block, 0, s, a, rp, group);
  return int8_rows ? launch_pdl(prompt_append_bf16<true, bf16>, grid, block, 0, s, a, rp, group)
                   : launch_pdl(prompt_append_bf16<false, bf16>, grid, block, 0, s, a, rp, group);
}

cudaError_t launch_gather_f32(const GatherArgs &a, int row, cudaStream_t s) {
  return launch_pdl(gather_f32, dim3(1u + (a.n_rows + 7) / 8), dim3(256), 0, s, a, row);
}

cudaError_t launch_gather_bf16(const GatherArgs &a, bool int8_rows, cudaStream_t s) {
  const dim3 grid(1u + (a.n_rows + 8 * kGatherRows - 1) / (8 * kGatherRows));
  return int8_rows ? launch_pdl(gather_bf16<true>, grid, dim3(256), 0, s, a)
                   : launch_pdl(gather_bf16<false>, grid, dim3(256), 0, s, a);
}

cudaError_t launch_prompt_plan(const PromptPlanArgs &a, cudaStream_t s) {
  static_assert(kBins == 1024, "the scan takes one bin a thread");
  return launch_pdl(prompt_plan_kernel, dim3(1), dim3(kBins), 0, s, a);
}

cudaError_t launch_prompt_attn_simt(const PromptAttnArgs &a, cudaStream_t s) {
  const int dq = a.d_nope + a.d_rope;
  const size_t smem = sizeof(float) * (kPromptTileSimt * dq + kSimtKeys * (dq + 1) +
                                       kSimtKeys * a.d_v + kPromptTileSimt * 33);
  static api::PerDeviceOnce once;
  const cudaError_t e = once.run([] {
    return cudaFuncSetAttribute(prompt_attn_simt, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                120 * 1024);
  });
  if (e != cudaSuccess) return e;
  return launch_pdl(prompt_attn_simt, dim3((unsigned)a.max_items, a.n_heads), dim3(128), smem, s,
                    a);
}

}  // namespace mla

// qk_norm_rope_store_fp8.cu -- RMSNorm and rotary embedding of the query and key heads of new
// tokens on their way into the 8-bit cache (the format is in fp8_cache.cuh).
//
// «nano-vLLM 最小化vLLM重新实现», 架构 6 模型: QK 归一化, then RoPE from a precomputed cos/sin
// cache; 架构 5: K and V written into the paged cache. A projection row holds Hq query heads, Hkv
// key heads and Hkv value heads of 128 values. For a query or key head x with weight w, in fp32:
//     n = x * rsqrt(mean(x^2) + eps) * w       (without weights: n = x)
//     y_i = n_i c_i - n_{i+64} s_i,  y_{i+64} = n_{i+64} c_i + n_i s_i,  i < 64
// Nothing is rounded before y, which is rounded once: queries to bf16, keys to e4m3 at the scale
// of their group. (pkv_qk_norm_rope_store rounds n and a key's y to bf16, as the model's layers do
// between them; here a key has 4 significant bits left, and a second rounding before those
// would only add to the error of the first.)
//
// As in kv_store_fp8 one CTA owns a run (the new rows of one sequence that lie in one group of 64
// positions) of some of the K or V heads, so that nothing else touches their scales; other CTAs
// take the run's query heads. A thread holds the 8 + 8 values of a row that turn into one another.
// A step of one token per sequence takes half a warp per head row. Bound by HBM: a row is read
// once, 2 bytes a value, and written once.
#include <math.h>

#include <algorithm>

#include "device_common.cuh"
#include "fp8_cache.cuh"
#include "launch.h"
#include "pkv.h"

namespace pkv {
namespace {

constexpr int kD = 128;
constexpr unsigned kFull = 0xffffffffu;

struct AppendParams {
  const uint8_t *qkv;
  int64_t tok_stride;  // bytes
  int64_t num_tokens;
  const int64_t *positions;
  const uint8_t *q_weight, *k_weight;  // nullptr: no norm
  float eps;
  const float *cos_sin;
  int64_t max_position;
  const int32_t *cu;  // nullptr: one token per sequence
  const int32_t *context_lens;
  const int32_t *block_tables;
  int32_t table_width, num_seqs;
  uint8_t *q_out;
  uint8_t *k_cache, *v_cache;
  float *k_scale, *v_scale;
  int32_t hq, hkv, block_size;
  int64_t num_blocks;
  unsigned int *err;
};

__device__ __forceinline__ void widen8(const uint4 w, float (&f)[8]) {
  f[0] = bf16_lo(w.x), f[1] = bf16_hi(w.x), f[2] = bf16_lo(w.y), f[3] = bf16_hi(w.y);
  f[4] = bf16_lo(w.z), f[5] = bf16_hi(w.z), f[6] = bf16_lo(w.w), f[7] = bf16_hi(w.w);
}
__device__ __forceinline__ uint4 round8(const float (&f)[8]) {
  return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                    pack_bf16x2(f[6], f[7]));
}
__device__ __forceinline__ uint2 quantize8(const float (&f)[8], float inv) {
  return make_uint2(cvt_e4m3x2(f[0] * inv, f[1] * inv) | cvt_e4m3x2(f[2] * inv, f[3] * inv) << 16,
                    cvt_e4m3x2(f[4] * inv, f[5] * inv) | cvt_e4m3x2(f[6] * inv, f[7] * inv) << 16);
}
// largest finite |f| of eight values, as fp32 bits, or above
__device__ __forceinline__ uint32_t finite_max8(uint32_t m, const float (&f)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t a = __float_as_uint(f[i]) & 0x7fffffffu;
    m = max(m, a < 0x7f800000u ? a : 0u);
  }
  return m;
}
// The scale for a group whose largest finite |x| has the fp32 bits `amax`: fp8_scale_exp's rule
// with fp32's mantissa.
__device__ __forceinline__ float scale_of(uint32_t amax) {
  const int e = (int)(amax >> 23) - 135 + ((amax & 0x7fffffu) > 0x600000u ? 1 : 0);
  return pow2f(max(e, kFp8MinExp));
}

// n of the values [8 i, +8) and [64 + 8 i, +8) of a row, given its sum of squares
__device__ __forceinline__ void normalise(const AppendParams &p, const uint8_t *weight, float ss,
                                          int i, float (&a)[8], float (&b)[8]) {
  const float rs = rsqrtf(ss * (1.f / kD) + p.eps);
  float wa[8], wb[8];
  widen8(*reinterpret_cast<const uint4 *>(weight + 16 * i), wa);
  widen8(*reinterpret_cast<const uint4 *>(weight + kD + 16 * i), wb);
#pragma unroll
  for (int d = 0; d < 8; ++d) {
    a[d] = a[d] * rs * wa[d];
    b[d] = b[d] * rs * wb[d];
  }
}
// y of them, the position's row of the cos/sin cache being `cs`
__device__ __forceinline__ void rotate(const float *cs, int i, float (&a)[8], float (&b)[8]) {
#pragma unroll
  for (int d = 0; d < 8; d += 4) {
    const float4 c = *reinterpret_cast<const float4 *>(cs + 8 * i + d);
    const float4 s = *reinterpret_cast<const float4 *>(cs + kD / 2 + 8 * i + d);
    const float cc[4] = {c.x, c.y, c.z, c.w}, sc[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float x = a[d + k], y = b[d + k];
      a[d + k] = x * cc[k] - y * sc[k];
      b[d + k] = y * cc[k] + x * sc[k];
    }
  }
}

constexpr int kRunThreads = 128;
constexpr int kRunWarps = kRunThreads / 32;
constexpr int kRowsPerPass = kRunThreads / 8;
constexpr int kPasses = kFp8Group / kRowsPerPass;

// The CTAs of a run: parts of its query, key and value heads.
__global__ void __launch_bounds__(kRunThreads)
    append_run_kernel(const AppendParams p, int heads_per_cta) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ uint32_t warp_max[2][kRunWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int qparts = (p.hq + heads_per_cta - 1) / heads_per_cta;
  const int kparts = (p.hkv + heads_per_cta - 1) / heads_per_cta;
  const int parts = qparts + 2 * kparts;
  const int64_t r = blockIdx.x / parts;
  int part = (int)(blockIdx.x % parts);
  const int kind = part < qparts ? 0 : part < qparts + kparts ? 1 : 2;  // query, key, value
  part -= kind == 0 ? 0 : kind == 1 ? qparts : qparts + kparts;
  const int h0 = part * heads_per_cta, h1 = min(kind ? p.hkv : p.hq, h0 + heads_per_cta);
  const int n = find_sequence(p.cu, p.num_seqs, r, lane);
  const int64_t c0 = *(p.cu + n), c1 = *(p.cu + n + 1), ctx = *(p.context_lens + n);
  const int64_t j = r - run_base((int32_t)c0, n);
  const int64_t capacity = (int64_t)p.table_width * p.block_size;
  if (blockIdx.x == 0) {  // the batch's lengths, looked over once
    for (int i = tid; i < p.num_seqs; i += kRunThreads) {
      const int64_t a = *(p.cu + i), e = *(p.cu + i + 1), len = *(p.context_lens + i);
      if (a < 0 || e < a || e > p.num_tokens || len < e - a) record_error(p.err, PKV_DEVERR_SEQLEN_RANGE);
      else if (len > capacity) record_error(p.err, PKV_DEVERR_CONTEXT_RANGE);
    }
  }
  if (c0 < 0 || c1 < c0 || c1 > p.num_tokens || ctx < c1 - c0 || ctx > capacity) return;
  const int64_t start = ctx - (c1 - c0);                // first new position
  const int64_t group = start / kFp8Group + j;          // group index in the sequence
  const int64_t begin = max(start, group * kFp8Group);
  const int64_t end = min(ctx, (group + 1) * kFp8Group);
  if (j < 0 || begin >= end) return;
  const int rows = (int)(end - begin);
  const int i8 = tid & 7, row0 = tid >> 3;
  const int64_t tok0 = c0 + begin - start + row0;
  // an earlier wait gave up somewhere: write nothing (decided by the CTA together)
  if (__syncthreads_or(tid == 0 && aborted(p.err))) return;
  const float *cs[kPasses];  // of this thread's rows; nullptr: past the run, or a bad position
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    cs[i] = nullptr;
    if (kind < 2 && row0 + i * kRowsPerPass < rows) {
      const int64_t pos = *(p.positions + tok0 + i * kRowsPerPass);
      if (pos >= 0 && pos < p.max_position) cs[i] = p.cos_sin + pos * kD;
      else if (i8 == 0) record_error(p.err, PKV_DEVERR_POSITION_RANGE);
    }
  }
  int64_t blk = 0;
  if (kind) {
    blk = *(p.block_tables + (int64_t)n * p.table_width + begin / p.block_size);
    if (blk < 0 || blk >= p.num_blocks) {
      if (tid == 0) record_error(p.err, PKV_DEVERR_BLOCK_RANGE);
      return;
    }
  }
  const int in_block = (int)(begin % p.block_size);
  const int before = in_block % kFp8Group;  // rows of the group from before the call
  const int64_t rstride = (int64_t)p.hkv * kD;
  float *const scales = kind == 2 ? p.v_scale : p.k_scale;
  uint8_t *const dst0 =
      (kind == 2 ? p.v_cache : p.k_cache) + (blk * p.block_size + in_block) * rstride;
  const uint8_t *weight = kind == 0 ? p.q_weight : p.k_weight;
  const uint8_t *const src = p.qkv + tok0 * p.tok_stride + 16 * i8 +
                             (kind == 0 ? 0 : kind == 1 ? p.hq : p.hq + p.hkv) * (2 * kD);
  int buf = 0;
  for (int h = h0; h < h1; ++h) {
    float a[kPasses][8], b[kPasses][8];
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      uint4 lo = make_uint4(0, 0, 0, 0), hi = lo;
      if (row0 + i * kRowsPerPass < rows) {
        const uint8_t *x = src + i * kRowsPerPass * p.tok_stride + h * (2 * kD);
        lo = ld_once_u4(reinterpret_cast<const uint4 *>(x));
        hi = ld_once_u4(reinterpret_cast<const uint4 *>(x + kD));
      }
      widen8(lo, a[i]);
      widen8(hi, b[i]);
    }
    if (kind < 2) {
#pragma unroll
      for (int i = 0; i < kPasses; ++i) {
        if (weight) {
          float ss = 0.f;
#pragma unroll
          for (int d = 0; d < 8; ++d) ss = fmaf(a[i][d], a[i][d], fmaf(b[i][d], b[i][d], ss));
#pragma unroll
          for (int o = 1; o < 8; o <<= 1) ss += __shfl_xor_sync(kFull, ss, o);
          normalise(p, weight, ss, i8, a[i], b[i]);
        }
        if (cs[i]) rotate(cs[i], i8, a[i], b[i]);
      }
    }
    if (kind == 0) {
#pragma unroll
      for (int i = 0; i < kPasses; ++i)
        if (cs[i]) {
          uint4 *q = reinterpret_cast<uint4 *>(
              p.q_out + ((tok0 + i * kRowsPerPass) * p.hq + h) * (2 * kD) + 16 * i8);
          q[0] = round8(a[i]);
          q[kD / 16] = round8(b[i]);
        }
      continue;
    }
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kPasses; ++i)
      if (kind == 2 ? row0 + i * kRowsPerPass < rows : cs[i] != nullptr)
        m = finite_max8(finite_max8(m, a[i]), b[i]);
    m = __reduce_max_sync(kFull, m);
    if (lane == 0) warp_max[buf][warp] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kRunWarps; ++w) m = max(m, warp_max[buf][w]);
    buf ^= 1;  // (the next use of this half is a barrier away)
    const int64_t sc = (blk * p.hkv + h) * (p.block_size / kFp8Group) + in_block / kFp8Group;
    float scale = scale_of(m);
    uint8_t *dst = dst0 + h * kD;
    if (before) {
      const float old = scales[sc];
      scale = fmaxf(scale, old);
      if (scale > old) {  // the rows from before, at the scale that grew
        const float ratio = old / scale;
        for (int i = tid; i < before * 8; i += kRunThreads) {
          uint4 *q = reinterpret_cast<uint4 *>(dst - (int64_t)(before - i / 8) * rstride + (i % 8) * 16);
          uint4 w = *q;
          w.x = rescale4(w.x, ratio);
          w.y = rescale4(w.y, ratio);
          w.z = rescale4(w.z, ratio);
          w.w = rescale4(w.w, ratio);
          *q = w;
        }
      }
      __syncthreads();  // every thread has read the old scale
    }
    if (tid == 0) scales[sc] = scale;
    const float inv = 1.f / scale;
#pragma unroll
    for (int i = 0; i < kPasses; ++i)
      if (kind == 2 ? row0 + i * kRowsPerPass < rows : cs[i] != nullptr) {
        uint8_t *d = dst + (row0 + i * kRowsPerPass) * rstride + 8 * i8;
        *reinterpret_cast<uint2 *>(d) = quantize8(a[i], inv);
        *reinterpret_cast<uint2 *>(d + kD / 2) = quantize8(b[i], inv);
      }
  }
}

// Half a warp: one head row of a sequence's new token. Lane i of it holds the values [8 i, +8).
constexpr int kTokenWarps = 4;
__global__ void __launch_bounds__(kTokenWarps * 32) append_token_kernel(const AppendParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31, i = lane & 15;
  const int heads = p.hq + 2 * p.hkv;
  const int64_t unit = ((int64_t)blockIdx.x * kTokenWarps * 32 + threadIdx.x) >> 4;
  const bool any = unit < (int64_t)p.num_seqs * heads;
  const int n = any ? (int)(unit / heads) : 0, row = any ? (int)(unit % heads) : 0;
  const int kind = row < p.hq ? 0 : row < p.hq + p.hkv ? 1 : 2;
  const int h = row - (kind == 0 ? 0 : kind == 1 ? p.hq : p.hq + p.hkv);
  float x[8];
  widen8(ld_once_u4(reinterpret_cast<const uint4 *>(p.qkv + n * p.tok_stride + row * (2 * kD) + 16 * i)), x);
  const int64_t pos = *(p.positions + n), ctx = *(p.context_lens + n);
  const bool pos_ok = pos >= 0 && pos < p.max_position;
  const bool stop = __any_sync(kFull, aborted(p.err));
  if (any && i == 0 && row == 0 && !pos_ok) record_error(p.err, PKV_DEVERR_POSITION_RANGE);
  if (kind < 2) {
    const uint8_t *weight = kind == 0 ? p.q_weight : p.k_weight;
    float ss = 0.f;
#pragma unroll
    for (int d = 0; d < 8; ++d) ss = fmaf(x[d], x[d], ss);
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) ss += __shfl_xor_sync(0xffffu << (lane & 16), ss, o);
    if (weight) {
      const float rs = rsqrtf(ss * (1.f / kD) + p.eps);
      float w[8];
      widen8(*reinterpret_cast<const uint4 *>(weight + 16 * i), w);
#pragma unroll
      for (int d = 0; d < 8; ++d) x[d] = x[d] * rs * w[d];
    }
    float y[8];
#pragma unroll
    for (int d = 0; d < 8; ++d) y[d] = __shfl_xor_sync(0xffffu << (lane & 16), x[d], 8);
    if (pos_ok) {
      const float *cs = p.cos_sin + pos * kD + 8 * (i & 7);
#pragma unroll
      for (int d = 0; d < 8; ++d)
        x[d] = i < 8 ? x[d] * cs[d] - y[d] * cs[kD / 2 + d] : x[d] * cs[d] + y[d] * cs[kD / 2 + d];
    }
  }
  if (!any || stop || (kind < 2 && !pos_ok)) return;
  if (kind == 0) {
    *reinterpret_cast<uint4 *>(p.q_out + ((int64_t)n * p.hq + h) * (2 * kD) + 16 * i) = round8(x);
    return;
  }
  if (ctx == 0) return;  // a padding row
  const bool tell = i == 0 && row == p.hq;
  if (ctx < 0 || ctx > (int64_t)p.table_width * p.block_size) {
    if (tell) record_error(p.err, PKV_DEVERR_CONTEXT_RANGE);
    return;
  }
  const int64_t blk = *(p.block_tables + (int64_t)n * p.table_width + (ctx - 1) / p.block_size);
  if (blk < 0 || blk >= p.num_blocks) {
    if (tell) record_error(p.err, PKV_DEVERR_BLOCK_RANGE);
    return;
  }
  const int in_block = (int)((ctx - 1) % p.block_size);
  const int before = in_block % kFp8Group;
  const int64_t sc = (blk * p.hkv + h) * (p.block_size / kFp8Group) + in_block / kFp8Group;
  float *scales = kind == 2 ? p.v_scale : p.k_scale;
  const float old = before ? scales[sc] : 0.f;
  uint32_t m = finite_max8(0, x);
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) m = max(m, __shfl_xor_sync(0xffffu << (lane & 16), m, o));
  const float scale = fmaxf(scale_of(m), old);
  const int64_t rstride = (int64_t)p.hkv * kD;
  uint8_t *dst = (kind == 2 ? p.v_cache : p.k_cache) + (blk * p.block_size + in_block) * rstride +
                 h * kD + i * 8;
  if (before && scale > old) {
    const float ratio = old / scale;
#pragma unroll 4
    for (int t = 1; t <= before; ++t) {
      uint2 *q = reinterpret_cast<uint2 *>(dst - t * rstride);
      const uint2 w = *q;
      *q = make_uint2(rescale4(w.x, ratio), rescale4(w.y, ratio));
    }
  }
  *reinterpret_cast<uint2 *>(dst) = quantize8(x, 1.f / scale);
  if (i == 0) scales[sc] = scale;
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace
}  // namespace pkv

extern "C" pkv_status pkv_qk_norm_rope_store_fp8(
    const void *qkv, int64_t qkv_tok_stride, int64_t num_tokens, const int64_t *positions,
    const void *q_norm_weight, const void *k_norm_weight, float eps, const float *cos_sin_cache,
    int64_t max_position, const int32_t *cu_seqlens, const int32_t *context_lens,
    const int32_t *block_tables, int32_t block_table_width, int32_t num_seqs, void *q_out,
    void *k_cache, void *v_cache, float *k_scale, float *v_scale, int32_t num_q_heads,
    int32_t num_kv_heads, int32_t head_dim, int32_t block_size, int64_t num_blocks, void *stream) {
  using namespace pkv;
  if (num_seqs < 0 || num_tokens < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 ||
      block_size <= 0 || num_blocks <= 0 || block_table_width <= 0 || max_position <= 0 ||
      !(eps >= 0.f) || !isfinite(eps))
    return PKV_ERR_INVALID_ARG;
  const int64_t heads = (int64_t)num_q_heads + 2 * (int64_t)num_kv_heads;
  if (qkv_tok_stride < heads * head_dim) return PKV_ERR_INVALID_ARG;
  if (!cu_seqlens && num_tokens != num_seqs) return PKV_ERR_INVALID_ARG;
  if (!q_norm_weight != !k_norm_weight) return PKV_ERR_INVALID_ARG;
  if (num_seqs == 0 || num_tokens == 0) return PKV_OK;
  if (!qkv || !positions || !cos_sin_cache || !context_lens || !block_tables || !q_out ||
      !k_cache || !v_cache || !k_scale || !v_scale)
    return PKV_ERR_INVALID_ARG;
  if (head_dim != kD || block_size % 256 != 0 || num_tokens > INT32_MAX || heads > (1 << 20))
    return PKV_ERR_UNSUPPORTED;
  if (qkv_tok_stride % 8 != 0 || !aligned16(qkv) || !aligned16(q_norm_weight) ||
      !aligned16(k_norm_weight) || !aligned16(cos_sin_cache) || !aligned16(q_out) ||
      !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(k_scale) || !aligned16(v_scale))
    return PKV_ERR_UNSUPPORTED;
  const int num_sms = current_sm_count();
  unsigned int *err = current_error_word();
  if (num_sms <= 0 || !err) return PKV_ERR_CUDA;
  AppendParams prm{};
  prm.qkv = static_cast<const uint8_t *>(qkv);
  prm.tok_stride = qkv_tok_stride * 2;
  prm.num_tokens = num_tokens;
  prm.positions = positions;
  prm.q_weight = static_cast<const uint8_t *>(q_norm_weight);
  prm.k_weight = static_cast<const uint8_t *>(k_norm_weight);
  prm.eps = eps;
  prm.cos_sin = cos_sin_cache;
  prm.max_position = max_position;
  prm.cu = cu_seqlens;
  prm.context_lens = context_lens;
  prm.block_tables = block_tables;
  prm.table_width = block_table_width;
  prm.num_seqs = num_seqs;
  prm.q_out = static_cast<uint8_t *>(q_out);
  prm.k_cache = static_cast<uint8_t *>(k_cache);
  prm.v_cache = static_cast<uint8_t *>(v_cache);
  prm.k_scale = k_scale;
  prm.v_scale = v_scale;
  prm.hq = num_q_heads;
  prm.hkv = num_kv_heads;
  prm.block_size = block_size;
  prm.num_blocks = num_blocks;
  prm.err = err;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (!cu_seqlens) {
    const int64_t grid = (num_seqs * heads + 2 * kTokenWarps - 1) / (2 * kTokenWarps);
    if (grid > INT32_MAX) return PKV_ERR_UNSUPPORTED;
    return launch_after(append_token_kernel, (unsigned)grid, kTokenWarps * 32, st, prm) ==
                   cudaSuccess
               ? PKV_OK
               : PKV_ERR_CUDA;
  }
  // as many heads to a CTA as still leave every SM about ten CTAs
  const int64_t runs = num_tokens / kFp8Group + 2 * (int64_t)num_seqs;
  const int64_t per = std::max<int64_t>(
      1, std::min<int64_t>(num_kv_heads, runs * heads / (10 * (int64_t)num_sms)));
  const int64_t grid =
      runs * ((num_q_heads + per - 1) / per + 2 * ((num_kv_heads + per - 1) / per));
  if (grid > INT32_MAX) return PKV_ERR_UNSUPPORTED;
  return launch_after(append_run_kernel, (unsigned)grid, kRunThreads, st, prm, (int)per) ==
                 cudaSuccess
             ? PKV_OK
             : PKV_ERR_CUDA;
}

// fp8_cache.cu -- writing the 8-bit cache (kv_store_fp8) and reading it back as bf16
// (kv_gather_fp8). The format is in fp8_cache.cuh.
//
// Store: the new tokens are each sequence's last positions. One CTA owns one run (the new rows
// of one sequence that lie in one group of 64 positions) of K or of V and goes through the KV
// heads, so nothing else touches a group's scale: it holds a head's rows in registers, reduces
// max |x| over them, takes the larger of the scale that asks for and the scale of the rows the
// group already held, and writes the codes. Each row is read once and written once:
// 512 + 256 bytes per token and head, nothing else of that order. When the scale grows, the
// rows from before the call are re-rounded to it in place (at most 63 rows of 128 bytes).
// A step of one token per sequence takes a warp per (sequence, head) instead of a CTA.
//
// Gather: whole rows of all heads, K or V; 128 bytes in and 256 bytes out per token and head.
//
// Both are bound by HBM.
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
constexpr unsigned int kErrBlock = 2u, kErrContext = 4u, kErrSeqlen = 8u;  // PKV_DEVERR_*

struct StoreParams {
  const uint8_t *k, *v;           // bf16 rows
  int64_t k_stride, v_stride;     // bytes per token
  const int32_t *cu;              // nullptr: one token per sequence
  const int32_t *context_lens;
  const int32_t *block_tables;
  int32_t table_width, num_seqs;
  int64_t num_tokens;
  uint8_t *k_cache, *v_cache;
  float *k_scale, *v_scale;
  int32_t hkv, block_size;
  int64_t num_blocks;
  bool wide;  // rows and strides of k and v are 32-byte aligned
  unsigned int *err;
};

// 32 bytes of a bf16 row
struct Row32 {
  uint4 lo, hi;
};
__device__ __forceinline__ uint32_t absmax8(const uint4 &x) {
  return __vmaxu2(bf16x2_absmax(x.x, x.y), bf16x2_absmax(x.z, x.w));
}
__device__ __forceinline__ uint4 finite8(const uint4 &x) {
  return make_uint4(bf16x2_finite(x.x), bf16x2_finite(x.y), bf16x2_finite(x.z),
                    bf16x2_finite(x.w));
}
// (one load where the address allows it)
__device__ __forceinline__ void ld_once_32b(const uint8_t *p, bool wide, uint4 &lo, uint4 &hi) {
  if (wide) {
    asm volatile(
        "ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
        : "=r"(lo.x), "=r"(lo.y), "=r"(lo.z), "=r"(lo.w), "=r"(hi.x), "=r"(hi.y), "=r"(hi.z),
          "=r"(hi.w)
        : "l"(p)
        : "memory");
  } else {
    lo = ld_once_u4(reinterpret_cast<const uint4 *>(p));
    hi = ld_once_u4(reinterpret_cast<const uint4 *>(p + 16));
  }
}

// Block of position pos of a sequence's table row, or -1 (recorded) for a bad id.
__device__ __forceinline__ int64_t block_of(const int32_t *table, int64_t pos, int32_t block_size,
                                            int64_t num_blocks, unsigned int *err, bool record) {
  const int32_t b = *(table + pos / block_size);
  if (b >= 0 && b < num_blocks) return b;
  if (record) record_error(err, kErrBlock);
  return -1;
}

// The batch's lengths, looked over once (by the first CTA): every sequence whose cu or context
// length is bad, which the runs' own checks leave out.
template <bool kStore>
__device__ __forceinline__ void check_lengths(const int32_t *cu, const int32_t *context_lens,
                                              int32_t num_seqs, int64_t total, int64_t capacity,
                                              unsigned int *err) {
  for (int i = threadIdx.x; i < num_seqs; i += blockDim.x) {
    const int32_t c0 = *(cu + i), c1 = *(cu + i + 1);
    const int64_t ctx = kStore ? (int64_t)*(context_lens + i) : (int64_t)c1 - c0;
    if (c0 < 0 || c1 < c0 || c1 > total || ctx < (int64_t)c1 - c0) record_error(err, kErrSeqlen);
    else if (ctx > capacity) record_error(err, kErrContext);
  }
}

// One CTA: K or V of a run (up to 64 rows of one group) for `heads_per_cta` consecutive heads, one
// head at a time while the next one's rows are on their way: thread t holds bytes
// [32 (t % 8), +32) of rows t / 8 + 16 i. A CTA has 32 KiB in flight and five fit on an SM; going
// through the heads in one CTA pays the dependent loads of its start (cu_seqlens, the table,
// 2-3 us) once. 145k tokens of 8 heads take 127 us (6.6 TB/s): 255 us with a CTA of 256 threads
// for each head, K and V together; 139 us with 16-byte loads and plain 8-byte stores; 130 us with
// those stores marked as not read again.
constexpr int kRunThreads = 128;
constexpr int kRunWarps = kRunThreads / 32;
constexpr int kRowsPerPass = kRunThreads / 8;
constexpr int kPasses = kFp8Group / kRowsPerPass;

__global__ void __launch_bounds__(kRunThreads, 5)
    kv_store_fp8_run_kernel(const StoreParams p, int heads_per_cta) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ uint32_t warp_max[2][kRunWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int parts = (p.hkv + heads_per_cta - 1) / heads_per_cta;
  const bool is_v = blockIdx.x & 1;
  const int64_t r = (blockIdx.x >> 1) / parts;
  const int h0 = (int)((blockIdx.x >> 1) % parts) * heads_per_cta;
  const int h1 = min(p.hkv, h0 + heads_per_cta);
  const int n = find_sequence(p.cu, p.num_seqs, r, lane);
  const int32_t c0 = p.cu[n], c1 = p.cu[n + 1], ctx = p.context_lens[n];
  const int64_t j = r - run_base(c0, n);
  const int64_t capacity = (int64_t)p.table_width * p.block_size;
  if (blockIdx.x == 0)
    check_lengths<true>(p.cu, p.context_lens, p.num_seqs, p.num_tokens, capacity, p.err);
  if (c0 < 0 || c1 < c0 || c1 > p.num_tokens || ctx < (int64_t)c1 - c0 || ctx > capacity) return;
  const int start = ctx - (c1 - c0);                        // first new position
  const int64_t group = (int64_t)(start / kFp8Group) + j;   // group index in the sequence
  const int64_t begin = max((int64_t)start, group * kFp8Group);
  const int64_t end = min((int64_t)ctx, (group + 1) * kFp8Group);
  if (j < 0 || begin >= end) return;
  const int rows = (int)(end - begin);
  const int part = threadIdx.x & 7, row0 = threadIdx.x >> 3;
  const int64_t stride = is_v ? p.v_stride : p.k_stride;
  const uint8_t *src = (is_v ? p.v : p.k) + (c0 + begin - start + row0) * stride + part * 32;
  Row32 x[2][kPasses];
  auto load = [&](Row32(&y)[kPasses], int h) {
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      y[i].lo = y[i].hi = make_uint4(0, 0, 0, 0);
      if (row0 + i * kRowsPerPass < rows)
        ld_once_32b(src + i * kRowsPerPass * stride + h * (kD * 2), p.wide, y[i].lo, y[i].hi);
    }
  };
  load(x[0], h0);
  const int64_t blk = block_of(p.block_tables + (int64_t)n * p.table_width, begin, p.block_size,
                               p.num_blocks, p.err, threadIdx.x == 0 && h0 == 0);
  // an earlier wait gave up somewhere: write nothing (decided by the CTA together)
  if (__syncthreads_or(threadIdx.x == 0 && aborted(p.err)) || blk < 0) return;
  const int in_block = (int)(begin % p.block_size);
  const int before = in_block % kFp8Group;  // rows of the group from before the call
  const int64_t rstride = (int64_t)p.hkv * kD;
  float *const scales = is_v ? p.v_scale : p.k_scale;
  uint8_t *const dst0 =
      (is_v ? p.v_cache : p.k_cache) + (blk * p.block_size + in_block) * rstride;

  // max |x| over the CTA, as bf16 bits
  int buf = 0;
  auto cta_max = [&](uint32_t m) {
    m = __reduce_max_sync(kFull, max(m & 0xffffu, m >> 16));
    if (lane == 0) warp_max[buf][warp] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kRunWarps; ++w) m = max(m, warp_max[buf][w]);
    buf ^= 1;  // (the next use of this half is two barriers away)
    return m;
  };
  auto store = [&](const Row32(&y)[kPasses], int h) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < kPasses; ++i)
      m = __vmaxu2(m, __vmaxu2(absmax8(y[i].lo), absmax8(y[i].hi)));
    m = cta_max(m);
    if (m >= 0x7f80u) {  // infinities or NaNs: the largest finite value counts
      m = 0;
#pragma unroll
      for (int i = 0; i < kPasses; ++i)
        m = __vmaxu2(m, __vmaxu2(absmax8(finite8(y[i].lo)), absmax8(finite8(y[i].hi))));
      m = cta_max(m);
    }
    const int64_t sc = (blk * p.hkv + h) * (p.block_size / kFp8Group) + in_block / kFp8Group;
    float scale = pow2f(fp8_scale_exp(m));
    uint8_t *dst = dst0 + h * kD;
    if (before) {
      const float old = scales[sc];
      scale = fmaxf(scale, old);
      if (scale > old) {  // the rows from before, at the scale that grew
        const float ratio = old / scale;
        for (int i = threadIdx.x; i < before * 8; i += kRunThreads) {
          uint4 *q =
              reinterpret_cast<uint4 *>(dst - (int64_t)(before - i / 8) * rstride + (i % 8) * 16);
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
    if (threadIdx.x == 0) scales[sc] = scale;
    const float inv = 1.f / scale;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int row = row0 + i * kRowsPerPass;
      if (row < rows)
        __stcs(reinterpret_cast<uint4 *>(dst + row * rstride + part * 16),
               make_uint4(quantize4(y[i].lo.x, y[i].lo.y, inv), quantize4(y[i].lo.z, y[i].lo.w, inv),
                          quantize4(y[i].hi.x, y[i].hi.y, inv),
                          quantize4(y[i].hi.z, y[i].hi.w, inv)));
    }
  };
  for (int h = h0; h < h1; h += 2) {
    if (h + 1 < h1) load(x[1], h + 1);
    store(x[0], h);
    if (h + 1 >= h1) break;
    if (h + 2 < h1) load(x[0], h + 2);
    store(x[1], h + 1);
  }
}

// One warp: the new token of one sequence, one head. Lanes 0-15 hold K, lanes 16-31 V, eight
// values each.
constexpr int kTokenWarps = 4;
__global__ void __launch_bounds__(kTokenWarps * 32)
    kv_store_fp8_token_kernel(const StoreParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31, part = lane & 15;
  const bool is_v = lane >= 16;
  const int64_t unit = (int64_t)blockIdx.x * kTokenWarps + (threadIdx.x >> 5);
  if (unit >= (int64_t)p.num_seqs * p.hkv) return;
  const int n = (int)(unit / p.hkv), h = (int)(unit % p.hkv);
  const uint8_t *src = is_v ? p.v + n * p.v_stride : p.k + n * p.k_stride;
  const uint4 x = ld_once_u4(reinterpret_cast<const uint4 *>(src + h * (kD * 2) + part * 16));
  const int32_t ctx = *(p.context_lens + n);
  if (ctx == 0) return;  // a padding row
  if (ctx < 0 || (int64_t)ctx > (int64_t)p.table_width * p.block_size) {
    if (lane == 0 && h == 0) record_error(p.err, kErrContext);
    return;
  }
  if (__any_sync(kFull, aborted(p.err))) return;  // (warp-uniform)
  const int64_t blk = block_of(p.block_tables + (int64_t)n * p.table_width, ctx - 1, p.block_size,
                               p.num_blocks, p.err, lane == 0 && h == 0);
  if (blk < 0) return;
  const int in_block = (ctx - 1) % p.block_size;
  const int before = in_block % kFp8Group;
  const int64_t sc = (blk * p.hkv + h) * (p.block_size / kFp8Group) + in_block / kFp8Group;
  float *scales = is_v ? p.v_scale : p.k_scale;
  const float old = before ? scales[sc] : 0.f;
  uint32_t m = absmax8(x);
  m = max(m & 0xffffu, m >> 16);
  if (m >= 0x7f80u) {
    m = absmax8(finite8(x));
    m = max(m & 0xffffu, m >> 16);
  }
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(kFull, m, o));
  const float scale = fmaxf(pow2f(fp8_scale_exp(m)), old);
  const int64_t rstride = (int64_t)p.hkv * kD;
  uint8_t *dst = (is_v ? p.v_cache : p.k_cache) + (blk * p.block_size + in_block) * rstride +
                 h * kD + part * 8;
  if (before && scale > old) {
    const float ratio = old / scale;
#pragma unroll 4
    for (int i = 1; i <= before; ++i) {
      uint2 *q = reinterpret_cast<uint2 *>(dst - i * rstride);
      const uint2 w = *q;
      *q = make_uint2(rescale4(w.x, ratio), rescale4(w.y, ratio));
    }
  }
  const float inv = 1.f / scale;
  *reinterpret_cast<uint2 *>(dst) = make_uint2(quantize4(x.x, x.y, inv), quantize4(x.z, x.w, inv));
  if (part == 0) scales[sc] = scale;
}

struct GatherParams {
  const uint8_t *k_cache, *v_cache;
  const float *k_scale, *v_scale;
  const int32_t *block_table;
  int32_t table_width;
  const int32_t *cu;
  int32_t num_seqs;
  int64_t total;
  uint8_t *k_out, *v_out;
  int32_t hkv, block_size;
  int64_t num_blocks;
  unsigned int *err;
};

// One CTA: K or V of `rows_per_cta` rows of a run (up to 64 positions of one group), all heads: the
// rows are read and written whole (hkv x 128 bytes in, twice that out), 16 codes to a lane, eight
// loads of a thread in flight. A lane's 32 bytes go out as one store: 164k tokens of 8 heads take
// 151 us (6.7 TB/s), 174 us with two 16-byte stores.
constexpr int kGatherThreads = 256;
constexpr int kGatherLoads = 8;
__global__ void __launch_bounds__(kGatherThreads)
    kv_gather_fp8_kernel(const GatherParams p, int rows_per_cta) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int parts = kFp8Group / rows_per_cta;
  const bool is_v = blockIdx.x & 1;
  const int64_t r = (blockIdx.x >> 1) / parts;
  const int row_from = (int)((blockIdx.x >> 1) % parts) * rows_per_cta;
  const int n = find_sequence(p.cu, p.num_seqs, r, lane);
  const int32_t c0 = p.cu[n], c1 = p.cu[n + 1];
  const int64_t j = r - run_base(c0, n);
  const int64_t capacity = (int64_t)p.table_width * p.block_size;
  if (blockIdx.x == 0)
    check_lengths<false>(p.cu, nullptr, p.num_seqs, p.total, capacity, p.err);
  const int64_t len = (int64_t)c1 - c0;
  if (c0 < 0 || len < 0 || c1 > p.total || len > capacity) return;
  const int64_t begin = j * kFp8Group + row_from;
  if (j < 0 || begin >= len || aborted(p.err)) return;
  const int rows = (int)min(len - begin, (int64_t)rows_per_cta);
  const int64_t blk = block_of(p.block_table + (int64_t)n * p.table_width, begin, p.block_size,
                               p.num_blocks, p.err, threadIdx.x == 0);
  const int in_block = (int)(begin % p.block_size), groups = p.block_size / kFp8Group;
  const int64_t rstride = (int64_t)p.hkv * kD;
  const uint4 *const src = reinterpret_cast<const uint4 *>(
      (is_v ? p.v_cache : p.k_cache) + (blk * p.block_size + in_block) * rstride);
  const float *const scales =
      (is_v ? p.v_scale : p.k_scale) + blk * p.hkv * groups + in_block / kFp8Group;
  uint4 *const dst =
      reinterpret_cast<uint4 *>((is_v ? p.v_out : p.k_out) + (c0 + begin) * rstride * 2);
  const uint32_t cols = (uint32_t)p.hkv * 8u;  // 16-byte pieces of a row, 8 to a head
  const uint32_t all = (uint32_t)rows * cols;
  const bool whole = (reinterpret_cast<uintptr_t>(dst) & 31u) == 0;  // (row lengths are)
  for (uint32_t u0 = threadIdx.x; u0 < all; u0 += kGatherThreads * kGatherLoads) {
    uint4 x[kGatherLoads];
    float scale[kGatherLoads];
#pragma unroll
    for (int i = 0; i < kGatherLoads; ++i) {
      const uint32_t u = u0 + i * kGatherThreads;
      x[i] = make_uint4(0, 0, 0, 0);  // the rows of a bad block id are zeros, as in attention
      scale[i] = 0.f;
      if (u < all && blk >= 0) {
        x[i] = ld_once_u4(src + u);
        scale[i] = scales[(int64_t)((u % cols) >> 3) * groups];
      }
    }
#pragma unroll
    for (int i = 0; i < kGatherLoads; ++i) {
      const uint32_t u = u0 + i * kGatherThreads;
      if (u < all) {
        const uint2 a = dequantize4(x[i].x, scale[i]), b = dequantize4(x[i].y, scale[i]);
        const uint2 c = dequantize4(x[i].z, scale[i]), d = dequantize4(x[i].w, scale[i]);
        const uint32_t w[8] = {a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
        if (whole) {
          st_global_32b(dst + 2 * (int64_t)u, w);
        } else {
          dst[2 * (int64_t)u] = make_uint4(w[0], w[1], w[2], w[3]);
          dst[2 * (int64_t)u + 1] = make_uint4(w[4], w[5], w[6], w[7]);
        }
      }
    }
  }
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace
}  // namespace pkv

extern "C" pkv_status pkv_kv_store_fp8(const void *k, int64_t k_tok_stride, const void *v,
                                       int64_t v_tok_stride, const int32_t *cu_seqlens,
                                       const int32_t *context_lens, const int32_t *block_tables,
                                       int32_t block_table_width, int32_t num_seqs,
                                       int64_t num_tokens, void *k_cache, void *v_cache,
                                       float *k_scale, float *v_scale, int32_t num_kv_heads,
                                       int32_t head_dim, int32_t block_size, int64_t num_blocks,
                                       void *stream) {
  using namespace pkv;
  if (num_seqs < 0 || num_tokens < 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 ||
      num_blocks <= 0 || block_table_width <= 0)
    return PKV_ERR_INVALID_ARG;
  const int64_t row = (int64_t)num_kv_heads * head_dim;
  if (k_tok_stride < row || v_tok_stride < row) return PKV_ERR_INVALID_ARG;
  if (!cu_seqlens && num_tokens != num_seqs) return PKV_ERR_INVALID_ARG;
  if (num_seqs == 0 || num_tokens == 0) return PKV_OK;
  if (!k || !v || !context_lens || !block_tables || !k_cache || !v_cache || !k_scale || !v_scale)
    return PKV_ERR_INVALID_ARG;
  if (head_dim != kD || block_size % 256 != 0 || num_tokens > INT32_MAX)
    return PKV_ERR_UNSUPPORTED;
  if (k_tok_stride % 8 != 0 || v_tok_stride % 8 != 0 || !aligned16(k) || !aligned16(v) ||
      !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(k_scale) || !aligned16(v_scale))
    return PKV_ERR_UNSUPPORTED;
  const int num_sms = current_sm_count();
  unsigned int *err = current_error_word();
  if (num_sms <= 0 || !err) return PKV_ERR_CUDA;
  StoreParams prm{};
  prm.k = static_cast<const uint8_t *>(k);
  prm.v = static_cast<const uint8_t *>(v);
  prm.k_stride = k_tok_stride * 2;
  prm.v_stride = v_tok_stride * 2;
  prm.cu = cu_seqlens;
  prm.context_lens = context_lens;
  prm.block_tables = block_tables;
  prm.table_width = block_table_width;
  prm.num_seqs = num_seqs;
  prm.num_tokens = num_tokens;
  prm.k_cache = static_cast<uint8_t *>(k_cache);
  prm.v_cache = static_cast<uint8_t *>(v_cache);
  prm.k_scale = k_scale;
  prm.v_scale = v_scale;
  prm.hkv = num_kv_heads;
  prm.block_size = block_size;
  prm.num_blocks = num_blocks;
  prm.wide = ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & 31u) == 0 &&
             k_tok_stride % 16 == 0 && v_tok_stride % 16 == 0;
  prm.err = err;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (!cu_seqlens) {
    const int64_t units = (int64_t)num_seqs * num_kv_heads;
    const int64_t grid = (units + kTokenWarps - 1) / kTokenWarps;
    if (grid > INT32_MAX) return PKV_ERR_UNSUPPORTED;
    return launch_after(kv_store_fp8_token_kernel, grid, kTokenWarps * 32, st, prm) == cudaSuccess
               ? PKV_OK
               : PKV_ERR_CUDA;
  }
  // as many heads to a CTA as still leave every SM about ten CTAs
  const int64_t runs = num_tokens / kFp8Group + 2 * (int64_t)num_seqs;
  const int64_t heads_per_cta =
      std::max<int64_t>(1, std::min<int64_t>(num_kv_heads, 2 * runs * num_kv_heads /
                                                               (10 * (int64_t)num_sms)));
  const int64_t grid = 2 * runs * ((num_kv_heads + heads_per_cta - 1) / heads_per_cta);
  if (grid > INT32_MAX) return PKV_ERR_UNSUPPORTED;
  return launch_after(kv_store_fp8_run_kernel, grid, kRunThreads, st, prm, (int)heads_per_cta) ==
                 cudaSuccess
             ? PKV_OK
             : PKV_ERR_CUDA;
}

extern "C" pkv_status pkv_kv_gather_fp8(const void *k_cache, const void *v_cache,
                                        const float *k_scale, const float *v_scale,
                                        const int32_t *block_table, int32_t block_table_width,
                                        const int32_t *cu_seqlens_k, int32_t num_seqs,
                                        int64_t total_k, void *k_out, void *v_out,
                                        int32_t num_kv_heads, int32_t head_dim,
                                        int32_t block_size, int64_t num_blocks, void *stream) {
  using namespace pkv;
  if (num_seqs < 0 || total_k < 0 || num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 ||
      num_blocks <= 0 || block_table_width <= 0)
    return PKV_ERR_INVALID_ARG;
  if (num_seqs == 0 || total_k == 0) return PKV_OK;
  if (!k_cache || !v_cache || !k_scale || !v_scale || !block_table || !cu_seqlens_k || !k_out ||
      !v_out)
    return PKV_ERR_INVALID_ARG;
  if (head_dim != kD || block_size % 256 != 0 || total_k > INT32_MAX) return PKV_ERR_UNSUPPORTED;
  if (!aligned16(k_cache) || !aligned16(v_cache) || !aligned16(k_scale) || !aligned16(v_scale) ||
      !aligned16(k_out) || !aligned16(v_out))
    return PKV_ERR_UNSUPPORTED;
  const int num_sms = current_sm_count();
  unsigned int *err = current_error_word();
  if (num_sms <= 0 || !err) return PKV_ERR_CUDA;
  GatherParams prm{};
  prm.k_cache = static_cast<const uint8_t *>(k_cache);
  prm.v_cache = static_cast<const uint8_t *>(v_cache);
  prm.k_scale = k_scale;
  prm.v_scale = v_scale;
  prm.block_table = block_table;
  prm.table_width = block_table_width;
  prm.cu = cu_seqlens_k;
  prm.num_seqs = num_seqs;
  prm.total = total_k;
  prm.k_out = static_cast<uint8_t *>(k_out);
  prm.v_out = static_cast<uint8_t *>(v_out);
  prm.hkv = num_kv_heads;
  prm.block_size = block_size;
  prm.num_blocks = num_blocks;
  prm.err = err;
  // runs in parts of fewer rows while there are less than about ten CTAs for an SM
  const int64_t runs = total_k / kFp8Group + 2 * (int64_t)num_seqs;
  int rows_per_cta = kFp8Group;
  while (rows_per_cta > 8 && 2 * runs * (kFp8Group / rows_per_cta) < 10 * (int64_t)num_sms)
    rows_per_cta /= 2;
  const int64_t grid = 2 * runs * (kFp8Group / rows_per_cta);
  if (grid > INT32_MAX || num_kv_heads > (1 << 20)) return PKV_ERR_UNSUPPORTED;
  return launch_after(kv_gather_fp8_kernel, grid, kGatherThreads, static_cast<cudaStream_t>(stream),
                      prm, rows_per_cta) == cudaSuccess
             ? PKV_OK
             : PKV_ERR_CUDA;
}

// evict.cu -- eviction from the cache by accumulated attention weight (kv_evict).
//
// Of a sequence of L > budget tokens each KV head keeps `budget`: the `recent` last ones, and of
// the earlier ones those with the largest weights (ties: the lower position; a NaN weight counts
// as smaller than every number). Their rows are compacted, in order, into the blocks of a
// second table: row kept[j] becomes row j. The source blocks are only read, so blocks shared
// with other sequences, or registered in the prefix cache, keep their contents.
//
// Two kernels. evict_select_kernel, one CTA per (sequence, head): a radix select over the
// weights' ordered bits (11 + 11 + 10, histograms in shared memory) finds the smallest kept key
// and how many of its equals are kept, then one ordered pass with prefix sums writes the kept
// positions.
// evict_copy_kernel, one CTA per (sequence, 64 or 128 kept rows, head), moves the K and V rows and the
// kept weights; it is bound by HBM: each kept row is read once and written once (16 x 32768
// tokens to 8192, 1.07 GB: 160 us). In an 8-bit cache 64 rows are one group of the
// destination, whose scale is the largest of its rows' scales (powers of two: rows of a smaller
// one lose only what falls below e4m3's normal range).
#include <algorithm>

#include "device_common.cuh"
#include "fp8_cache.cuh"
#include "launch.h"
#include "pkv.h"

namespace pkv {
namespace {

constexpr int kD = 128;
constexpr unsigned kFull = 0xffffffffu;
constexpr unsigned int kErrBlock = 2u, kErrContext = 4u;  // PKV_DEVERR_*
constexpr int kGroup = kFp8Group;

struct EvictParams {
  const float *weights;
  int64_t weights_stride;
  const int32_t *context_lens;
  int32_t batch, max_context_len, budget, recent;
  const int32_t *src_tables, *dst_tables;
  int32_t src_width, dst_width;
  uint8_t *k_cache, *v_cache;
  float *k_scale, *v_scale;
  int32_t hkv, block_size;
  int64_t num_blocks;
  int32_t *kept;
  float *weights_out;
  int64_t weights_out_stride;
  int32_t *new_lens;
  unsigned int *err;
};

// Bits that order like the numbers (NaN first, -0 equal to +0: x + 0 is +0 for both).
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t b = __float_as_uint(x + 0.f);
  const uint32_t key = b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
  return isnan(x) ? 0u : key;
}

constexpr int kBins = 2048;
// A warp's part of a row, up to kHeld chunks of 128 elements, stays in its lanes' registers as
// ordered keys, so a row of up to 32768 weights is loaded once, all loads in flight together; a
// longer row is taken in pieces of 32768 that each pass loads again. What bounds the kernel is its
// instructions: 32 rows of 18168 to 32660 weights took 17.1 us (both kernels) when every key was
// compared and branched on in every pass, 12.9 us with a vote for each 128 keys first.
//
// Three instances (WARPS warps, kHeld chunks): 32 x 8 holds 32768, 8 x 8 holds 8192, 8 x 2 holds
// 2048. Smaller CTAs cost less to launch and to synchronise, and more of them run on an SM: 172 rows
// of up to 3899 weights 15.7 -> 8.8 us, 512 rows of up to 2048 54 -> 35 us (both kernels).
constexpr uint32_t kTopKey = 0xffffffffu;  // a recent position's: above every number's

// Inclusive sum over the warp's lanes up to this one.
__device__ __forceinline__ uint32_t warp_scan(uint32_t x, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t y = __shfl_up_sync(kFull, x, o);
    if (lane >= o) x += y;
  }
  return x;
}

// The thread's kOwn bins (a power of two of them), the highest first; its share of clearing.
template <int kOwn>
__device__ __forceinline__ void load_own(const uint32_t *hist, uint32_t (&own)[kOwn]) {
  if constexpr (kOwn % 4 == 0) {
    const uint4 *h = reinterpret_cast<const uint4 *>(hist + kBins - kOwn * (threadIdx.x + 1));
#pragma unroll
    for (int i = 0; i < kOwn / 4; ++i) {
      const uint4 x = h[kOwn / 4 - 1 - i];
      own[4 * i] = x.w;
      own[4 * i + 1] = x.z;
      own[4 * i + 2] = x.y;
      own[4 * i + 3] = x.x;
    }
  } else {
#pragma unroll
    for (int i = 0; i < kOwn; ++i) own[i] = hist[kBins - 1 - kOwn * threadIdx.x - i];
  }
}
template <int kOwn>
__device__ __forceinline__ void clear_own(uint32_t *hist) {
  if constexpr (kOwn % 4 == 0) {
#pragma unroll
    for (int i = 0; i < kOwn / 4; ++i)
      reinterpret_cast<uint4 *>(hist)[threadIdx.x + i * (kBins / kOwn)] = make_uint4(0, 0, 0, 0);
  } else {
#pragma unroll
    for (int i = 0; i < kOwn; ++i) hist[threadIdx.x + i * (kBins / kOwn)] = 0u;
  }
}

// Exclusive sum over the CTA's threads up to this one. `sums` (a word for each warp) may be used
// again after the next __syncthreads.
template <int WARPS>
__device__ __forceinline__ uint32_t block_scan(uint32_t x, uint32_t *sums) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const uint32_t inc = warp_scan(x, lane);
  if (lane == 31) sums[warp] = inc;
  __syncthreads();
  const uint32_t w = warp_scan(lane < WARPS ? sums[lane] : 0u, lane);
  const uint32_t before = __shfl_sync(kFull, w, max(warp - 1, 0));
  return inc - x + (warp ? before : 0u);
}

template <int WARPS, int kHeld>
__global__ void __launch_bounds__(WARPS * 32) evict_select_kernel(const EvictParams p) {
  constexpr int kThreads = WARPS * 32;
  constexpr int kPiece = kHeld * 128 * WARPS;
  constexpr int kOwn = kBins / kThreads;  // bins of a thread
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ alignas(16) uint32_t hist[kBins];
  __shared__ uint32_t sums[2][WARPS];
  __shared__ uint32_t found_bin, found_above;
  const int64_t bh = blockIdx.x;
  const int b = (int)(bh / p.hkv), h = (int)(bh % p.hkv);
  const int32_t L = ld_global_s32(p.context_lens + b);
  const bool stop = threadIdx.x == 0 && aborted(p.err);  // (both loads in flight together)
  if (__syncthreads_or(stop)) return;
  const bool bad = L < 0 || L > p.max_context_len ||
                   (int64_t)L > (int64_t)p.src_width * p.block_size ||
                   (int64_t)min(L, p.budget) > (int64_t)p.dst_width * p.block_size;
  const int32_t n = bad ? 0 : min(L, p.budget);
  if (threadIdx.x == 0 && h == 0) {
    p.new_lens[b] = n;
    if (bad) record_error(p.err, kErrContext);
  }
  const float *w = p.weights + bh * p.weights_stride;
  int32_t *kept = p.kept + bh * p.budget;
  float *w_out = p.weights_out ? p.weights_out + bh * p.weights_out_stride : nullptr;

  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (L > p.budget && !bad) {
    const uint32_t len = (uint32_t)L, older = (uint32_t)(L - p.recent);
    const bool vec = (reinterpret_cast<uintptr_t>(w) & 15u) == 0;
    const uint32_t pieces = (len + kPiece - 1) / kPiece;
    uint32_t key[kHeld][4];
    uint32_t want = (uint32_t)p.budget;  // still to be kept, of the keys that share `prefix`
    uint32_t prefix = 0u;
    uint32_t above0 = 0u, equal0 = 0u;   // last pass: kept in the pieces before
    // Passes 0-2 count the keys' digits and find the smallest kept key, `prefix` in the end, and
    // how many of its equals are kept, `want`. Pass 3 writes, in order: a larger key is kept, an
    // equal one if it is among the first `want`. (One loop: the code of a pass per pass did not
    // fit the instruction cache.)
#pragma unroll 1
    for (int pass = 0; pass < 4; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const uint32_t digit = pass == 2 ? 1023u : 2047u;
      const uint32_t mask = pass == 0 ? 0u : pass == 1 ? 0xffe00000u : 0xfffffc00u;
      if (pass < 3) {
        clear_own<kOwn>(hist);
        __syncthreads();
      }
#pragma unroll 1
      for (uint32_t piece = 0; piece < pieces; ++piece) {
        const uint32_t base = piece * kPiece;
        const uint32_t in_piece = min(len - base, (uint32_t)kPiece);
        const int chunks = (int)((in_piece + 128 * WARPS - 1) / (128 * WARPS));
        const uint32_t at0 = base + (uint32_t)(warp * chunks * 128 + lane * 4);
        if (pass == 0 || pieces > 1) {
          // The keys: recent positions get the top one, what lies past the row the lowest (0, a
          // NaN's: it is never kept, the row has `budget` elements at lower positions).
#pragma unroll
          for (int c = 0; c < kHeld; ++c) {
            const uint32_t i = at0 + c * 128;
            if (vec && c < chunks && i + 4 <= len) {
              const uint4 x = *reinterpret_cast<const uint4 *>(w + i);
              key[c][0] = x.x;
              key[c][1] = x.y;
              key[c][2] = x.z;
              key[c][3] = x.w;
            } else {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                key[c][e] = c < chunks && i + e < len ? __float_as_uint(w[i + e]) : 0x7fffffffu;
            }
          }
#pragma unroll
          for (int c = 0; c < kHeld; ++c) {
            if (c >= chunks) break;
            const uint32_t i = at0 + c * 128;
#pragma unroll
            for (int e = 0; e < 4; ++e) key[c][e] = ordered(__uint_as_float(key[c][e]));
            if (i + 4 > older)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (i + e >= older && i + e < len) key[c][e] = kTopKey;
          }
        }
        if (pass < 3) {
#pragma unroll
          for (int c = 0; c < kHeld; ++c) {
            if (c >= chunks) break;
            if (pass > 0) {  // (few keys still share the prefix: mostly no lane's)
              uint32_t off = kTopKey;
#pragma unroll
              for (int e = 0; e < 4; ++e) off = min(off, (key[c][e] ^ prefix) & mask);
              if (!__any_sync(kFull, off == 0u)) continue;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (((key[c][e] ^ prefix) & mask) == 0u)
                atomicAdd(&hist[(key[c][e] >> shift) & digit], 1u);
          }
          continue;
        }
        // each warp counts its keys, the block sums the counts up, then each warp walks its chunks
        uint32_t cnt[kHeld], mine = 0u;  // larger in the upper half, equal in the lower
#pragma unroll
        for (int c = 0; c < kHeld; ++c) {
          cnt[c] = 0u;
          if (c >= chunks) continue;
#pragma unroll
          for (int e = 0; e < 4; ++e)
            cnt[c] += key[c][e] > prefix ? 0x10000u : key[c][e] == prefix ? 1u : 0u;
          mine += cnt[c];
        }
        mine = __reduce_add_sync(kFull, mine);  // (at most 1024 of each)
        __syncthreads();  // the sums of the step before have been read
        if (lane == 0) {
          sums[0][warp] = mine >> 16;
          sums[1][warp] = mine & 0xffffu;
        }
        __syncthreads();
        const uint32_t sa = warp_scan(lane < WARPS ? sums[0][lane] : 0u, lane);
        const uint32_t se = warp_scan(lane < WARPS ? sums[1][lane] : 0u, lane);
        const uint32_t pa = __shfl_sync(kFull, sa, max(warp - 1, 0));
        const uint32_t pe = __shfl_sync(kFull, se, max(warp - 1, 0));
        uint32_t a = above0 + (warp ? pa : 0u), q = equal0 + (warp ? pe : 0u);
        above0 += __shfl_sync(kFull, sa, 31);
        equal0 += __shfl_sync(kFull, se, 31);
#pragma unroll
        for (int c = 0; c < kHeld; ++c) {
          if (c >= chunks) break;
          if (!__any_sync(kFull, cnt[c] != 0u)) continue;  // nothing to keep among these 128
          const uint32_t inc = warp_scan(cnt[c], lane);
          const uint32_t all = __shfl_sync(kFull, inc, 31);
          const uint32_t before = inc - cnt[c], i = at0 + c * 128;
          uint32_t at = a + (before >> 16);
          if ((all & 0xffffu) == 0u) {  // no equals here
            at += min(q, want);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              if (key[c][e] > prefix) kept[at++] = (int32_t)(i + e);
          } else {
            uint32_t le = q + (before & 0xffffu);
            at += min(le, want);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const bool equal = key[c][e] == prefix;
              if (key[c][e] > prefix || (equal && le < want)) kept[at++] = (int32_t)(i + e);
              le += equal;
            }
          }
          a += all >> 16;
          q += all & 0xffffu;
        }
      }
      if (pass == 3) break;
      __syncthreads();
      // thread t owns the bins kOwn t .. counted from the top
      const int hi = kBins - 1 - kOwn * threadIdx.x;
      uint32_t own[kOwn], mine = 0u;  // (the highest first)
      load_own<kOwn>(hist, own);
#pragma unroll
      for (int i = 0; i < kOwn; ++i) mine += own[i];
      uint32_t above = block_scan<WARPS>(mine, sums[0]);
      if (above < want && want <= above + mine) {
#pragma unroll
        for (int i = 0; i < kOwn; ++i) {
          if (above < want && want <= above + own[i]) {
            found_bin = (uint32_t)(hi - i);
            found_above = above;
          }
          above += own[i];
        }
      }
      __syncthreads();
      want -= found_above;
      prefix |= found_bin << shift;
    }
  } else {
    for (int64_t j = threadIdx.x; j < n; j += kThreads) kept[j] = (int32_t)j;
  }
  for (int64_t j = n + (int64_t)threadIdx.x; j < p.budget; j += kThreads) {
    kept[j] = -1;
    if (w_out) w_out[j] = 0.f;
  }
}

// One CTA: 64 kept rows of one head, of an 8-bit cache 128 (two groups of the destination). 16 (bf16)
// or 8 (8-bit) lanes move a row, 16 bytes each; all the loads of the CTA's K and V rows, 32 KiB, are
// in flight at once (64 contexts of 4000 to 8192 tokens cut to 2048: 112 us, of which the selection
// takes 15-16 and the copy 95; 124 with 64 rows of an 8-bit cache, 16 KiB, to a CTA).
constexpr int kCopyThreads = 256;
template <bool FP8>
constexpr int kCopyRows = FP8 ? 2 * kGroup : kGroup;

template <bool FP8>
__global__ void __launch_bounds__(kCopyThreads) evict_copy_kernel(const EvictParams p, int chunks) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  constexpr int kRowBytes = FP8 ? kD : 2 * kD;
  constexpr int kLanes = kRowBytes / 16, kRowsPerPass = kCopyThreads / kLanes;
  constexpr int kRows = kCopyRows<FP8>, kPasses = kRows / kRowsPerPass;
  __shared__ int64_t src_slot[kRows];        // pool row of a kept row, -1: none
  __shared__ float src_scale[2][kRows];      // 8-bit: its scales, K's and V's
  __shared__ float new_scale[2][kRows / kGroup];
  const int h = (int)(blockIdx.x % p.hkv);
  const int64_t bc = blockIdx.x / p.hkv;
  const int c = (int)(bc % chunks), b = (int)(bc / chunks);
  const int j0 = c * kRows, t = threadIdx.x;
  const int64_t bh = (int64_t)b * p.hkv + h;
  // what nothing else is needed for, all in flight together (the kept list has `budget` entries)
  const int dst_at = min(j0 / p.block_size, p.dst_width - 1);
  const int32_t n = ld_global_s32(p.new_lens + b);
  const int32_t dst_blk = ld_global_s32(p.dst_tables + (int64_t)b * p.dst_width + dst_at);
  const bool stop = t == 0 && aborted(p.err);  // an earlier wait gave up somewhere
  const int32_t kept = t < kRows && j0 + t < p.budget
                           ? ld_global_s32(p.kept + bh * p.budget + j0 + t) : -1;
  // (decided by the CTA together; after an abort the kept list may hold anything)
  if (__syncthreads_or(stop) || j0 >= n) return;
  const int rows = min(kRows, n - j0);
  const bool dst_ok = dst_blk >= 0 && dst_blk < p.num_blocks;
  if (!dst_ok && threadIdx.x == 0 && h == 0) record_error(p.err, kErrBlock);
  const int dst_in = j0 % p.block_size;
  float s[2] = {0.f, 0.f};
  if (t < kRows) {
    int64_t slot = -1;
    if (t < rows) {
      const int32_t blk =
          ld_global_s32(p.src_tables + (int64_t)b * p.src_width + kept / p.block_size);
      if (p.weights_out)
        p.weights_out[bh * p.weights_out_stride + j0 + t] = p.weights[bh * p.weights_stride + kept];
      if (blk >= 0 && blk < p.num_blocks) {
        const int in = kept % p.block_size;
        slot = (int64_t)blk * p.block_size + in;
        if constexpr (FP8) {  // (in flight while the rows are asked for)
          const int64_t at = ((int64_t)blk * p.hkv + h) * (p.block_size / kGroup) + in / kGroup;
          s[0] = p.k_scale[at];
          s[1] = p.v_scale[at];
        }
      } else {
        record_error(p.err, kErrBlock);  // its row becomes zeros
      }
    }
    src_slot[t] = slot;
  }
  if (!dst_ok) return;  // (the rows that would go there are dropped, their weights are not)
  __syncthreads();
  const int part = t % kLanes, row0 = t / kLanes;
  const int64_t rstride = (int64_t)p.hkv * kRowBytes;
  const int64_t col = (int64_t)h * kRowBytes + part * 16;
  uint4 x[2][kPasses];
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int row = row0 + i * kRowsPerPass;
    const int64_t slot = src_slot[row];
    x[0][i] = x[1][i] = make_uint4(0, 0, 0, 0);
    if (slot >= 0) {
      x[0][i] = ld_once_u4(reinterpret_cast<const uint4 *>(p.k_cache + slot * rstride + col));
      x[1][i] = ld_once_u4(reinterpret_cast<const uint4 *>(p.v_cache + slot * rstride + col));
    }
  }
  if constexpr (FP8) {
    if (t < kRows) {
      src_scale[0][t] = s[0];
      src_scale[1][t] = s[1];
    }
    __syncthreads();
    if (t < 32 * 2 * (kRows / kGroup)) {  // a warp for each group of K and of V: its largest scale
      const int kv = (t >> 5) & 1, grp = t >> 6, l = t & 31;
      float m = fmaxf(src_scale[kv][grp * kGroup + l], src_scale[kv][grp * kGroup + l + 32]);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
      if (l == 0 && grp * kGroup < rows) {
        m = m > 0.f ? m : pow2f(kFp8MinExp);
        new_scale[kv][grp] = m;
        const int64_t at =
            ((int64_t)dst_blk * p.hkv + h) * (p.block_size / kGroup) + dst_in / kGroup + grp;
        (kv ? p.v_scale : p.k_scale)[at] = m;
      }
    }
    __syncthreads();
  }
  const int64_t dst0 = ((int64_t)dst_blk * p.block_size + dst_in) * rstride + col;
#pragma unroll
  for (int kv = 0; kv < 2; ++kv)
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const int row = row0 + i * kRowsPerPass;
      if (row >= rows) continue;
      uint4 v = x[kv][i];
      if constexpr (FP8) {
        const float f = src_scale[kv][row] / new_scale[kv][row / kGroup];
        if (f != 1.f) {
          v.x = rescale4(v.x, f);
          v.y = rescale4(v.y, f);
          v.z = rescale4(v.z, f);
          v.w = rescale4(v.w, f);
        }
      }
      *reinterpret_cast<uint4 *>((kv ? p.v_cache : p.k_cache) + dst0 + row * rstride) = v;
    }
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace
}  // namespace pkv

extern "C" pkv_status pkv_kv_evict(const float *weights, int64_t weights_stride,
                                   const int32_t *context_lens, int32_t batch,
                                   int32_t max_context_len, int32_t budget, int32_t recent,
                                   const int32_t *block_tables, int32_t block_table_width,
                                   const int32_t *dst_block_tables, int32_t dst_block_table_width,
                                   void *k_cache, void *v_cache, float *k_scale, float *v_scale,
                                   int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                                   int64_t num_blocks, int32_t *kept, float *weights_out,
                                   int64_t weights_out_stride, int32_t *new_context_lens,
                                   void *stream) {
  using namespace pkv;
  if (batch < 0 || max_context_len < 0 || budget <= 0 || recent < 0 || recent > budget ||
      num_kv_heads <= 0 || head_dim <= 0 || block_size <= 0 || num_blocks <= 0 ||
      block_table_width <= 0 || dst_block_table_width <= 0 || weights_stride < max_context_len ||
      (weights_out && weights_out_stride < budget))
    return PKV_ERR_INVALID_ARG;
  if (batch == 0) return PKV_OK;
  if (!weights || !context_lens || !block_tables || !dst_block_tables || !k_cache || !v_cache ||
      !kept || !new_context_lens || !k_scale != !v_scale)
    return PKV_ERR_INVALID_ARG;
  // the call reads these while it writes those
  if (dst_block_tables == block_tables || new_context_lens == context_lens ||
      weights_out == weights)
    return PKV_ERR_INVALID_ARG;
  const bool fp8 = k_scale != nullptr;
  if (head_dim != kD || block_size % (fp8 ? 256 : kGroup) != 0) return PKV_ERR_UNSUPPORTED;
  if (!aligned16(k_cache) || !aligned16(v_cache)) return PKV_ERR_UNSUPPORTED;
  const int64_t rows = (int64_t)batch * num_kv_heads;
  const int copy_rows = fp8 ? kCopyRows<true> : kCopyRows<false>;
  const int64_t chunks =
      ((int64_t)std::min(budget, std::max(max_context_len, 1)) + copy_rows - 1) / copy_rows;
  if (rows * chunks > INT32_MAX) return PKV_ERR_UNSUPPORTED;
  EvictParams prm{};
  prm.err = current_error_word();
  if (!prm.err) return PKV_ERR_CUDA;
  prm.weights = weights;
  prm.weights_stride = weights_stride;
  prm.context_lens = context_lens;
  prm.batch = batch;
  prm.max_context_len = max_context_len;
  prm.budget = budget;
  prm.recent = recent;
  prm.src_tables = block_tables;
  prm.dst_tables = dst_block_tables;
  prm.src_width = block_table_width;
  prm.dst_width = dst_block_table_width;
  prm.k_cache = static_cast<uint8_t *>(k_cache);
  prm.v_cache = static_cast<uint8_t *>(v_cache);
  prm.k_scale = k_scale;
  prm.v_scale = v_scale;
  prm.hkv = num_kv_heads;
  prm.block_size = block_size;
  prm.num_blocks = num_blocks;
  prm.kept = kept;
  prm.weights_out = weights_out;
  prm.weights_out_stride = weights_out_stride;
  prm.new_lens = new_context_lens;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  // (the longest rows that one CTA of 256 threads holds take it longer than one of 1024: that is
  // made up for where there are more rows than SMs)
  const int small = rows > current_sm_count() ? 8192 : 4096;
  cudaError_t e =
      max_context_len <= 2048    ? launch_after(evict_select_kernel<8, 2>, rows, 256, s, prm)
      : max_context_len <= small ? launch_after(evict_select_kernel<8, 8>, rows, 256, s, prm)
                                 : launch_after(evict_select_kernel<32, 8>, rows, 1024, s, prm);
  if (e == cudaSuccess)
    e = launch_after(fp8 ? evict_copy_kernel<true> : evict_copy_kernel<false>, rows * chunks,
                     kCopyThreads, s, prm, (int)chunks);
  return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

// decode_common.cuh -- what the decode kernels of the two caches share: the work units and their
// order, the kernels' parameters, and the merge of the splits that did not meet in a cluster.
#pragma once

#include <math.h>

#include <algorithm>
#include <type_traits>

#include "device_common.cuh"
#include "launch.h"

namespace pkv {
namespace {

constexpr int kD = 128;
constexpr int kMaxCluster = 8;  // largest portable thread-block cluster
constexpr unsigned int kErrWorkspace = 64u;  // PKV_DEVERR_WORKSPACE
constexpr float kLog2e = 1.4426950408889634f;
constexpr unsigned kFull = 0xffffffffu;

struct DecodeParams {
  const uint16_t *q;
  const int32_t *block_tables;
  const int32_t *context_lens;
  float *part_o;
  float *part_lse;
  uint16_t *out;
  int32_t *queue;  // next unit to hand out (the workspace's first word); nullptr: CTA i takes
                   // unit i only
  // > 0: the splits of one (sequence, head group) form a cluster of this many CTAs (CTA i
  // takes unit i, ordered split-minor); rank 0 merges them through distributed shared memory
  int32_t cluster;
  unsigned int *err;
  int64_t num_blocks;
  int64_t cap;  // longest context the table rows and the split grid can address
  int32_t table_width;
  int32_t batch;
  int32_t num_q_heads;
  int32_t group;
  int32_t head_groups;
  int32_t xgroups;  // num_kv_heads * head_groups
  int32_t block_size;
  int32_t chunk;
  int32_t splits;
  int32_t units;    // splits * batch * xgroups
  float qscale;
  // the step's new tokens (k_new == nullptr: nothing to store)
  const uint16_t *k_new;
  const uint16_t *v_new;
  int64_t k_new_stride, v_new_stride;  // elements per token
  const int64_t *slots;
  int64_t num_slots;
  uint16_t *k_cache_w;
  uint16_t *v_cache_w;
  int32_t num_kv_heads;
  // 8-bit cache: [num_blocks, num_kv_heads, block_size / 64]
  const float *k_scale;
  const float *v_scale;
  // for the weights kernel: scores [batch, num_q_heads, score_stride] (log2 domain) and the
  // log2-sum-exp of each query head
  float *scores;
  int64_t score_stride;
  float *lse;
  // where the decode kernel forms the weights itself (w_out != nullptr)
  const float *w_in;
  int64_t w_in_stride;
  float *w_out;
  int64_t w_out_stride;
};

// The attention weights of positions [begin, end) of sequence b and KV head h, from the scores that
// this CTA left (a barrier has made them visible to its threads) and the query heads'
// log2-sum-exps: decode_weights_kernel's sums, in its order. Thread `tid` of `threads` takes every
// threads-th position; the first ones' loads are under way once the object is made, before the
// log2-sum-exps have to be known.
template <int GC>
struct WeightsPass {
  static constexpr int kAhead = GC <= 2 ? 4 : GC == 4 ? 2 : 1;  // positions loaded together
  const float *s, *in;
  float *out;
  int64_t stride;
  int i0, end, step, group;
  float x[kAhead][GC], w[kAhead];
  uint32_t err;

  __device__ __forceinline__ WeightsPass(const DecodeParams &p, int b, int h, int begin, int last,
                                         int tid, int threads) {
    const int64_t bh = (int64_t)b * p.num_kv_heads + h;
    group = p.group;
    stride = p.score_stride;
    s = p.scores + bh * group * stride;
    in = p.w_in ? p.w_in + bh * p.w_in_stride : nullptr;
    out = p.w_out + bh * p.w_out_stride;
    i0 = begin + tid;
    end = last;
    step = threads;
    err = (uint32_t)ld_global_s32(reinterpret_cast<const int32_t *>(p.err));
    load();
  }
  __device__ __forceinline__ void load() {
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const int i = i0 + k * step;
      w[k] = in && i < end ? in[i] : 0.f;
#pragma unroll
      for (int g = 0; g < GC; ++g) x[k][g] = g < group && i < end ? s[g * stride + i] : -INFINITY;
    }
  }
  __device__ __forceinline__ void finish(const float *lse) {
    if (err & kErrTimeout) return;  // a wait gave up somewhere: the scores may not be complete
    while (i0 < end) {
#pragma unroll
      for (int k = 0; k < kAhead; ++k) {
        const int i = i0 + k * step;
        float sum = 0.f;
#pragma unroll
        for (int g = 0; g < GC; ++g)
          if (g < group) sum += fast_exp2(x[k][g] - lse[g]);
        if (i < end) out[i] = w[k] + sum;
      }
      i0 += kAhead * step;
      if (i0 < end) load();
    }
  }
};

struct NoWeights {
  __device__ __forceinline__ NoWeights(const DecodeParams &, int, int, int, int, int, int) {}
};

// Unit u -> (split s, sequence b, head group xg). A cluster launch orders the units
// split-minor (the splits of one sequence and head group adjacent), otherwise split-major.
__device__ __forceinline__ void unit_coords(const DecodeParams &p, int u, int &s, int &b,
                                            int &xg) {
  if (p.cluster) {
    s = u % p.splits;
    b = (u / p.splits) / p.xgroups;
    xg = (u / p.splits) % p.xgroups;
  } else {
    s = u / (p.batch * p.xgroups);
    const int r = u % (p.batch * p.xgroups);
    b = r / p.xgroups;
    xg = r % p.xgroups;
  }
}

// One warp per (sequence, query head): out = sum_s 2^(lse_s - lse) o_s over the sequence's
// splits, lse = log2 sum_s 2^lse_s. A sequence with no token gets zeros; one whose context
// fits one split was written by the split kernel.
// kNan: a split with a NaN makes the result NaN also where no other split has a key (the bf16
// kernel without weights gives zeros there).
template <bool kNan>
__global__ void __launch_bounds__(128)
    decode_combine_kernel(const float *__restrict__ part_o, const float *__restrict__ part_lse,
                          const int32_t *__restrict__ context_lens, int32_t batch,
                          int32_t num_q_heads, int32_t chunk, int32_t splits, int64_t cap,
                          uint16_t *__restrict__ out, float *__restrict__ lse_out,
                          const unsigned int *err) {
  // the stream's next kernel (the next call's split kernel) may be scheduled now: it waits
  // for this grid's completion before it touches global memory
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // launched as a programmatic dependent of the split kernel: wait until that grid has
  // completed and its partial results are visible
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (aborted(err)) return;  // an earlier wait gave up: the partials are not complete
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (row >= (int64_t)batch * num_q_heads) return;
  const int lane = threadIdx.x & 31;
  const int b = (int)(row / num_q_heads);
  int64_t L = context_lens[b];
  L = L < 0 ? 0 : (L > cap ? cap : L);
  const int ns = (int)((L + chunk - 1) / chunk);
  if (ns == 1) return;  // one split: the split kernel wrote this row itself
  const float *lse = part_lse + row * splits;
  float M = -INFINITY;
  for (int s = lane; s < ns; s += 32) M = fmaxf(M, lse[s]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(kFull, M, o));
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float wsum = 0.f;
  if (kNan && M == -INFINITY) M = 0.f;
  if (kNan || M != -INFINITY) {
    for (int s = 0; s < ns; ++s) {
      const float wgt = fast_exp2(lse[s] - M);
      const float4 o4 = *reinterpret_cast<const float4 *>(part_o + (row * splits + s) * kD + 4 * lane);
      wsum += wgt;
      acc.x = fmaf(wgt, o4.x, acc.x);
      acc.y = fmaf(wgt, o4.y, acc.y);
      acc.z = fmaf(wgt, o4.z, acc.z);
      acc.w = fmaf(wgt, o4.w, acc.w);
    }
  }
  if (lse_out && lane == 0) lse_out[row] = M + __log2f(wsum);  // ns == 0: -inf, not read
  const float inv = (kNan ? wsum != 0.f : wsum > 0.f) ? 1.f / wsum : 0.f;
  const uint32_t lo = (uint32_t)bf16_bits_rn(acc.x * inv) | ((uint32_t)bf16_bits_rn(acc.y * inv) << 16);
  const uint32_t hi = (uint32_t)bf16_bits_rn(acc.z * inv) | ((uint32_t)bf16_bits_rn(acc.w * inv) << 16);
  *reinterpret_cast<uint2 *>(out + row * kD + 4 * lane) = make_uint2(lo, hi);
}

// The parameters both kernels take from a call and its plan.
inline DecodeParams decode_params(const DecodeArgs &a, const DecodePlan &p) {
  uint8_t *ws = static_cast<uint8_t *>(a.workspace);
  float *const part_base = reinterpret_cast<float *>(ws + kDecodeQueueBytes);  // after the counter
  DecodeParams prm{};
  prm.q = static_cast<const uint16_t *>(a.q);
  prm.block_tables = a.block_tables;
  prm.context_lens = a.context_lens;
  prm.part_o = p.splits > 1 ? part_base : nullptr;
  prm.part_lse = p.splits > 1 ? prm.part_o + (size_t)a.batch * a.num_q_heads * p.splits * kD
                              : nullptr;
  prm.out = static_cast<uint16_t *>(a.out);
  prm.queue = reinterpret_cast<int32_t *>(ws);
  prm.err = a.err;
  prm.num_blocks = a.num_blocks;
  prm.cap = std::min({(int64_t)a.table_width * a.block_size, (int64_t)p.splits * p.chunk,
                      (int64_t)a.max_context_len});
  prm.table_width = a.table_width;
  prm.batch = a.batch;
  prm.num_q_heads = a.num_q_heads;
  prm.group = a.num_q_heads / a.num_kv_heads;
  prm.head_groups = p.head_groups;
  prm.xgroups = a.num_kv_heads * p.head_groups;
  prm.block_size = a.block_size;
  prm.chunk = p.chunk;
  prm.splits = p.splits;
  prm.qscale = a.scale * kLog2e;
  prm.num_kv_heads = a.num_kv_heads;
  prm.k_scale = a.k_scale;
  prm.v_scale = a.v_scale;
  if (p.scores_at) {
    prm.scores = reinterpret_cast<float *>(ws + p.scores_at);
    prm.score_stride = p.score_stride;
    prm.lse = reinterpret_cast<float *>(ws + p.lse_at);
    if (decode_forms_weights(a, p)) {
      prm.w_in = a.weights_in;
      prm.w_in_stride = a.weights_in_stride;
      prm.w_out = a.weights_out;
      prm.w_out_stride = a.weights_out_stride;
    }
  }
  return prm;
}

// The merge kernel of a call whose splits left their partials in the workspace.
template <bool kNan>
inline cudaError_t launch_combine(const DecodeArgs &a, const DecodePlan &p, const DecodeParams &prm,
                                  cudaStream_t stream) {
  const int64_t rows_out = (int64_t)a.batch * a.num_q_heads;
  // programmatic dependent launch: the merge grid is set up while the split kernel runs
  return launch_after(decode_combine_kernel<kNan>, dim3((unsigned)((rows_out + 3) / 4)), 128, stream,
                      (const float *)prm.part_o, (const float *)prm.part_lse, a.context_lens,
                      a.batch, a.num_q_heads, p.chunk, p.splits, prm.cap,
                      static_cast<uint16_t *>(a.out), prm.lse, (const unsigned int *)a.err);
}

}  // namespace
}  // namespace pkv

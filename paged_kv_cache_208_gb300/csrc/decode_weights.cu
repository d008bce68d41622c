// decode_weights.cu -- the attention weights of a decode step whose split kernel does not form them
// itself (decode_forms_weights: several units share a KV head, the splits meet in the merge kernel,
// or eight heads a unit come with the work queue or splits of more than 1280 tokens), and the entry
// points of decode attention over the 8-bit cache and of decode attention
// with weights.
//
// The split kernel has left every key's scaled score s (log2 domain) and every query head's
// log2-sum-exp; the weight that KV head h's query heads give to position i is
//
//     w[b, h, i] = sum_g 2^(s[b, hG + g, i] - lse[b, hG + g]),     w_out = w_in + w
//
// Keeping the scores costs 4 bytes written and read per (query head, token) -- for two heads to
// a KV head 3% of the K and V bytes of a bf16 cache, 6% of an 8-bit one -- where a second pass
// over K would cost a half; up to 126 MB of them stay in L2. The sum over g runs in a fixed
// order and every weight has one writer.
#include <math.h>

#include <algorithm>

#include "device_common.cuh"
#include "launch.h"
#include "pkv.h"

namespace pkv {
namespace {

constexpr int kThreads = 256;
constexpr int kSpan = kThreads * 4;  // positions of a CTA: four consecutive ones to a thread
constexpr int kFirst = 2;            // heads whose loads are issued together

struct WeightsParams {
  const float *scores;
  int64_t score_stride;
  const float *lse;
  const int32_t *context_lens;
  int64_t cap;  // longest context the decode call took
  const float *in;
  int64_t in_stride;
  float *out;
  int64_t out_stride;
  int32_t hkv, group;
  bool vec;  // the rows of in and out are 16-byte aligned
  const unsigned int *err;
};

__global__ void __launch_bounds__(kThreads) decode_weights_kernel(const WeightsParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  // what the loads below need, all in flight together: the length, the error word and the first
  // heads' log-sum-exps
  const int64_t bh = blockIdx.x;
  const int64_t b = bh / p.hkv;
  const float *const lse = p.lse + bh * p.group;
  const int32_t length = ld_global_s32(p.context_lens + b);
  const uint32_t err = (uint32_t)ld_global_s32(reinterpret_cast<const int32_t *>(p.err));
  float lse0[kFirst];
#pragma unroll
  for (int g = 0; g < kFirst; ++g)
    lse0[g] = __int_as_float(ld_global_s32(reinterpret_cast<const int32_t *>(lse) +
                                           min(g, p.group - 1)));
  if (err & kErrTimeout) return;  // an earlier wait gave up: the scores are not complete
  const int64_t L = length < 0 ? 0 : min((int64_t)length, p.cap);
  const float *const in = p.in ? p.in + bh * p.in_stride : nullptr;
  float *const out = p.out + bh * p.out_stride;
  for (int64_t i = (int64_t)blockIdx.y * kSpan + 4 * threadIdx.x; i < L;
       i += (int64_t)gridDim.y * kSpan) {
    const float *s = p.scores + bh * p.group * p.score_stride + i;  // 16-byte aligned
    float4 w = make_float4(0.f, 0.f, 0.f, 0.f), before = w;
    const bool whole = p.vec && i + 4 <= L;
    if (in && whole) {
      before = *reinterpret_cast<const float4 *>(in + i);
    } else if (in) {
      before.x = in[i];
      if (i + 1 < L) before.y = in[i + 1];
      if (i + 2 < L) before.z = in[i + 2];
      if (i + 3 < L) before.w = in[i + 3];
    }
    float4 x[kFirst];
#pragma unroll
    for (int g = 0; g < kFirst; ++g)  // (entries past L: not used)
      if (g < p.group) x[g] = *reinterpret_cast<const float4 *>(s + g * p.score_stride);
    auto add = [&](const float4 &y, float z) {
      w.x += fast_exp2(y.x - z);
      w.y += fast_exp2(y.y - z);
      w.z += fast_exp2(y.z - z);
      w.w += fast_exp2(y.w - z);
    };
#pragma unroll
    for (int g = 0; g < kFirst; ++g)
      if (g < p.group) add(x[g], lse0[g]);
#pragma unroll 4
    for (int g = kFirst; g < p.group; ++g)
      add(*reinterpret_cast<const float4 *>(s + g * p.score_stride), lse[g]);
    w = make_float4(before.x + w.x, before.y + w.y, before.z + w.z, before.w + w.w);
    if (whole) {
      *reinterpret_cast<float4 *>(out + i) = w;
    } else {
      out[i] = w.x;
      if (i + 1 < L) out[i + 1] = w.y;
      if (i + 2 < L) out[i + 2] = w.z;
      if (i + 3 < L) out[i + 3] = w.w;
    }
  }
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct Call {
  DecodeArgs a;
  int32_t max_context_len, head_dim, num_splits;
  size_t workspace_bytes;
  bool fp8;
  bool weights;
  const float *weights_in;
  int64_t weights_in_stride;
  float *weights_out;
  int64_t weights_out_stride;
};

pkv_status decode_with_weights(Call c, cudaStream_t stream) {
  DecodeArgs &a = c.a;
  if (a.batch < 0 || c.max_context_len < 0 || c.num_splits < 0 || a.num_q_heads <= 0 ||
      a.num_kv_heads <= 0 || a.num_q_heads % a.num_kv_heads != 0 || c.head_dim <= 0 ||
      a.block_size <= 0 || a.num_blocks <= 0 || a.table_width <= 0 || !isfinite(a.scale))
    return PKV_ERR_INVALID_ARG;
  if (c.weights_in && !c.weights) return PKV_ERR_INVALID_ARG;
  if (c.weights && (c.weights_out_stride < c.max_context_len ||
                    (c.weights_in && c.weights_in_stride < c.max_context_len)))
    return PKV_ERR_INVALID_ARG;
  if (a.batch == 0) return PKV_OK;
  if (!a.q || !a.k_cache || !a.v_cache || !a.block_tables || !a.context_lens || !a.out ||
      (c.fp8 && (!a.k_scale || !a.v_scale)) || (c.weights && !c.weights_out))
    return PKV_ERR_INVALID_ARG;
  if (c.head_dim != 128 || a.block_size % 256 != 0) return PKV_ERR_UNSUPPORTED;
  if (a.num_blocks * (int64_t)a.block_size > INT32_MAX) return PKV_ERR_UNSUPPORTED;
  if (!aligned16(a.q) || !aligned16(a.k_cache) || !aligned16(a.v_cache) || !aligned16(a.out) ||
      (c.fp8 && (!aligned16(a.k_scale) || !aligned16(a.v_scale))))
    return PKV_ERR_UNSUPPORTED;
  const int64_t rows = (int64_t)a.batch * a.num_kv_heads;
  if (c.weights && rows > INT32_MAX) return PKV_ERR_UNSUPPORTED;
  a.num_sms = current_sm_count();
  a.err = current_error_word();
  if (a.num_sms <= 0 || !a.err) return PKV_ERR_CUDA;
  if (c.weights) {
    a.weights_in = c.weights_in;
    a.weights_in_stride = c.weights_in_stride;
    a.weights_out = c.weights_out;
    a.weights_out_stride = c.weights_out_stride;
  }
  a.max_context_len = c.max_context_len;
  const DecodePlan plan = plan_decode(a.batch, a.num_q_heads, a.num_kv_heads, c.max_context_len,
                                      c.num_splits, a.num_sms, c.fp8, c.weights);
  if (!a.workspace || c.workspace_bytes < plan.workspace_bytes || !aligned16(a.workspace))
    return PKV_ERR_WORKSPACE;
  cudaError_t e = c.fp8 ? launch_paged_decode_fp8(a, plan, stream)
                        : launch_paged_decode(a, plan, stream);
  if (e != cudaSuccess || !c.weights || c.max_context_len == 0 || decode_forms_weights(a, plan))
    return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
  uint8_t *ws = static_cast<uint8_t *>(a.workspace);
  WeightsParams w{};
  w.scores = reinterpret_cast<const float *>(ws + plan.scores_at);
  w.score_stride = plan.score_stride;
  w.lse = reinterpret_cast<const float *>(ws + plan.lse_at);
  w.context_lens = a.context_lens;
  // what the decode kernels clamp a context to, and no more than the rows of weights hold
  w.cap = std::min({(int64_t)a.table_width * a.block_size, (int64_t)plan.splits * plan.chunk,
                    (int64_t)c.max_context_len});
  w.in = c.weights_in;
  w.in_stride = c.weights_in_stride;
  w.out = c.weights_out;
  w.out_stride = c.weights_out_stride;
  w.hkv = a.num_kv_heads;
  w.group = a.num_q_heads / a.num_kv_heads;
  w.vec = (!w.in || (aligned16(w.in) && w.in_stride % 4 == 0)) && aligned16(w.out) &&
          w.out_stride % 4 == 0;
  w.err = a.err;
  const int64_t spans = ((int64_t)c.max_context_len + kSpan - 1) / kSpan;
  e = launch_after(decode_weights_kernel,
                   dim3((unsigned)rows, (unsigned)std::min<int64_t>(spans, 65535)), kThreads,
                   stream, w);
  return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

size_t workspace_bytes(int32_t batch, int32_t num_q_heads, int32_t num_kv_heads,
                       int32_t head_dim, int32_t max_context_len, int32_t num_splits, bool fp8,
                       bool weights) {
  if (batch <= 0 || num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads != 0 ||
      head_dim != 128 || max_context_len < 0 || num_splits < 0)
    return 0;
  const int num_sms = current_sm_count();
  if (num_sms <= 0) return 0;
  return plan_decode(batch, num_q_heads, num_kv_heads, max_context_len, num_splits, num_sms, fp8,
                     weights)
      .workspace_bytes;
}

}  // namespace
}  // namespace pkv

extern "C" size_t pkv_decode_weights_workspace_bytes(int32_t batch, int32_t num_q_heads,
                                                     int32_t num_kv_heads, int32_t head_dim,
                                                     int32_t max_context_len,
                                                     int32_t num_splits) {
  return pkv::workspace_bytes(batch, num_q_heads, num_kv_heads, head_dim, max_context_len,
                              num_splits, false, true);
}

extern "C" size_t pkv_decode_fp8_workspace_bytes(int32_t batch, int32_t num_q_heads,
                                                 int32_t num_kv_heads, int32_t head_dim,
                                                 int32_t max_context_len, int32_t num_splits,
                                                 int32_t weights) {
  return pkv::workspace_bytes(batch, num_q_heads, num_kv_heads, head_dim, max_context_len,
                              num_splits, true, weights != 0);
}

extern "C" pkv_status pkv_paged_decode_attn_weights(
    const void *q, const void *k_cache, const void *v_cache, const int32_t *block_tables,
    int32_t block_table_width, const int32_t *context_lens, int32_t batch,
    int32_t max_context_len, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
    int32_t block_size, int64_t num_blocks, float scale, int32_t num_splits,
    const float *weights_in, int64_t weights_in_stride, float *weights_out,
    int64_t weights_out_stride, void *workspace, size_t workspace_bytes, void *out,
    void *stream) {
  pkv::Call c{};
  c.a = pkv::DecodeArgs{q,          k_cache,      v_cache,     block_tables, block_table_width,
                        context_lens, batch,      num_q_heads, num_kv_heads, block_size,
                        num_blocks, scale,        workspace,   out,          nullptr,
                        0};
  c.max_context_len = max_context_len;
  c.head_dim = head_dim;
  c.num_splits = num_splits;
  c.workspace_bytes = workspace_bytes;
  c.weights = true;
  c.weights_in = weights_in;
  c.weights_in_stride = weights_in_stride;
  c.weights_out = weights_out;
  c.weights_out_stride = weights_out_stride;
  return pkv::decode_with_weights(c, static_cast<cudaStream_t>(stream));
}

extern "C" pkv_status pkv_paged_decode_attn_fp8(
    const void *q, const void *k_cache, const void *v_cache, const float *k_scale,
    const float *v_scale, const int32_t *block_tables, int32_t block_table_width,
    const int32_t *context_lens, int32_t batch, int32_t max_context_len, int32_t num_q_heads,
    int32_t num_kv_heads, int32_t head_dim, int32_t block_size, int64_t num_blocks, float scale,
    int32_t num_splits, const float *weights_in, int64_t weights_in_stride, float *weights_out,
    int64_t weights_out_stride, void *workspace, size_t workspace_bytes, void *out,
    void *stream) {
  pkv::Call c{};
  c.a = pkv::DecodeArgs{q,          k_cache,      v_cache,     block_tables, block_table_width,
                        context_lens, batch,      num_q_heads, num_kv_heads, block_size,
                        num_blocks, scale,        workspace,   out,          nullptr,
                        0};
  c.a.k_scale = k_scale;
  c.a.v_scale = v_scale;
  c.max_context_len = max_context_len;
  c.head_dim = head_dim;
  c.num_splits = num_splits;
  c.workspace_bytes = workspace_bytes;
  c.fp8 = true;
  c.weights = weights_out != nullptr;
  c.weights_in = weights_in;
  c.weights_in_stride = weights_in_stride;
  c.weights_out = weights_out;
  c.weights_out_stride = weights_out_stride;
  return pkv::decode_with_weights(c, static_cast<cudaStream_t>(stream));
}

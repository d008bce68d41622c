// tree_attn.cu -- attention of drafted tokens over the paged cache (paged_tree_attn): the last n
// positions of a context are the nodes of a tree, and each attends to the context before them and
// to the nodes that its mask names.
//
// One warp per node and query head: a lane holds four dims of q and of the output, the running
// maximum and sum of the softmax are the warp's.
#include <math.h>

#include "device_common.cuh"
#include "fp8_cache.cuh"
#include "launch.h"
#include "pkv.h"

namespace pkv {
namespace {

constexpr int kD = 128;
constexpr unsigned kFull = 0xffffffffu;
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kWarps = 4;

struct TreeParams {
  const uint16_t *q;
  int64_t q_stride;
  int64_t total_q;
  const uint8_t *k_cache, *v_cache;
  const float *k_scale, *v_scale;  // of an 8-bit cache
  const int32_t *block_tables;
  int32_t table_width;
  const int32_t *context_lens;
  const int32_t *cu;
  int32_t max_nodes, max_context;
  const uint64_t *mask;
  int32_t mask_words;
  int32_t hq, hkv, block_size;
  int64_t num_blocks;
  float scale_log2;
  uint16_t *out;
  unsigned int *err;
};

template <bool F8>
__global__ void __launch_bounds__(kWarps * 32) tree_attn_kernel(const TreeParams p) {
  const int lane = threadIdx.x & 31;
  const int b = blockIdx.y;
  const int unit = blockIdx.x * kWarps + (threadIdx.x >> 5);
  const int node = unit / p.hq, hq = unit % p.hq, h = hq / (p.hq / p.hkv);
  const int64_t c0 = p.cu[b], n = p.cu[b + 1] - c0;
  if (c0 < 0 || n < 0 || c0 + n > p.total_q || n > p.max_nodes) {
    if (unit == 0 && lane == 0) record_error(p.err, PKV_DEVERR_SEQLEN_RANGE);
    return;
  }
  if (node >= n) return;
  int64_t L = p.context_lens[b];
  if (L < n || L > p.max_context || L > (int64_t)p.table_width * p.block_size) {
    if (unit == 0 && lane == 0) record_error(p.err, PKV_DEVERR_CONTEXT_RANGE);
    L = 0;
  }
  const uint2 qw = *reinterpret_cast<const uint2 *>(p.q + (c0 + node) * p.q_stride + hq * kD + 4 * lane);
  const float q[4] = {bf16_lo(qw.x), bf16_hi(qw.x), bf16_lo(qw.y), bf16_hi(qw.y)};
  const uint64_t *mask = p.mask ? p.mask + (c0 + node) * p.mask_words : nullptr;
  float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  for (int64_t i = 0; i < L; ++i) {
    const int64_t j = i - (L - n);
    if (j >= 0 && !(mask ? mask[j >> 6] >> (j & 63) & 1 : j <= node)) continue;
    const int64_t blk = p.block_tables[(int64_t)b * p.table_width + i / p.block_size];
    const bool ok = blk >= 0 && blk < p.num_blocks;
    if (!ok && lane == 0) record_error(p.err, PKV_DEVERR_BLOCK_RANGE);
    const int64_t at = ((blk * p.block_size + i % p.block_size) * p.hkv + h) * kD + 4 * lane;
    float k[4] = {0.f, 0.f, 0.f, 0.f}, v[4] = {0.f, 0.f, 0.f, 0.f};
    if (ok && !F8) {
      const uint2 kw = *reinterpret_cast<const uint2 *>(p.k_cache + 2 * at);
      const uint2 vw = *reinterpret_cast<const uint2 *>(p.v_cache + 2 * at);
      k[0] = bf16_lo(kw.x), k[1] = bf16_hi(kw.x), k[2] = bf16_lo(kw.y), k[3] = bf16_hi(kw.y);
      v[0] = bf16_lo(vw.x), v[1] = bf16_hi(vw.x), v[2] = bf16_lo(vw.y), v[3] = bf16_hi(vw.y);
    } else if (ok) {
      const int groups = p.block_size / kFp8Group;
      const int64_t sc = (blk * p.hkv + h) * groups + i % p.block_size / kFp8Group;
      const uint32_t kw = *reinterpret_cast<const uint32_t *>(p.k_cache + at);
      const uint32_t vw = *reinterpret_cast<const uint32_t *>(p.v_cache + at);
      const float ks = p.k_scale[sc], vs = p.v_scale[sc];
      const float2 k0 = f16x2_to_f32(cvt_f16x2_e4m3x2(kw)), k1 = f16x2_to_f32(cvt_f16x2_e4m3x2_hi(kw));
      const float2 v0 = f16x2_to_f32(cvt_f16x2_e4m3x2(vw)), v1 = f16x2_to_f32(cvt_f16x2_e4m3x2_hi(vw));
      k[0] = k0.x * ks, k[1] = k0.y * ks, k[2] = k1.x * ks, k[3] = k1.y * ks;
      v[0] = v0.x * vs, v[1] = v0.y * vs, v[2] = v1.x * vs, v[3] = v1.y * vs;
    }
    float s = q[0] * k[0] + q[1] * k[1] + q[2] * k[2] + q[3] * k[3];
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(kFull, s, d);
    s *= p.scale_log2;
    const float top = fmaxf(m, s);
    const float old = m == -INFINITY ? 0.f : exp2f(m - top), w = exp2f(s - top);
    m = top;
    l = l * old + w;
#pragma unroll
    for (int d = 0; d < 4; ++d) o[d] = o[d] * old + w * v[d];
  }
  const float inv = l > 0.f ? 1.f / l : 0.f;
  *reinterpret_cast<uint2 *>(p.out + ((c0 + node) * p.hq + hq) * kD + 4 * lane) =
      make_uint2(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv));
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

pkv_status tree_attn(const void *q, int64_t q_tok_stride, int64_t total_q, const void *k_cache,
                     const void *v_cache, const float *k_scale, const float *v_scale, bool fp8,
                     const int32_t *block_tables, int32_t block_table_width,
                     const int32_t *context_lens, const int32_t *cu_seqlens_q, int32_t num_seqs,
                     int32_t max_seqlen_q, int32_t max_context_len, const int64_t *tree_mask,
                     int32_t mask_words, int32_t num_q_heads, int32_t num_kv_heads,
                     int32_t head_dim, int32_t block_size, int64_t num_blocks, float scale,
                     void *workspace, size_t workspace_bytes, void *out, void *stream) {
  if (num_seqs < 0 || total_q < 0 || max_seqlen_q < 0 || max_context_len < 0 ||
      num_q_heads <= 0 || num_kv_heads <= 0 || num_q_heads % num_kv_heads != 0 || head_dim <= 0 ||
      block_size <= 0 || num_blocks <= 0 || block_table_width <= 0 || !isfinite(scale))
    return PKV_ERR_INVALID_ARG;
  if (q_tok_stride < (int64_t)num_q_heads * head_dim) return PKV_ERR_INVALID_ARG;
  if (tree_mask && (mask_words < 0 || 64 * (int64_t)mask_words < max_seqlen_q))
    return PKV_ERR_INVALID_ARG;
  if (num_seqs == 0 || total_q == 0 || max_seqlen_q == 0) return PKV_OK;
  if (!q || !k_cache || !v_cache || !block_tables || !context_lens || !cu_seqlens_q || !out ||
      (fp8 && (!k_scale || !v_scale)))
    return PKV_ERR_INVALID_ARG;
  if (head_dim != kD || block_size % 256 != 0 || total_q > INT32_MAX ||
      num_blocks * (int64_t)block_size > INT32_MAX)
    return PKV_ERR_UNSUPPORTED;
  if (q_tok_stride % 8 != 0 || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) ||
      !aligned16(out) || (fp8 && (!aligned16(k_scale) || !aligned16(v_scale))))
    return PKV_ERR_UNSUPPORTED;
  if (!workspace || !aligned16(workspace) ||
      workspace_bytes < pkv_tree_workspace_bytes(num_seqs, max_seqlen_q, num_q_heads, num_kv_heads,
                                                 head_dim, max_context_len))
    return PKV_ERR_WORKSPACE;
  unsigned int *err = current_error_word();
  if (!err) return PKV_ERR_CUDA;
  const int64_t units = ((int64_t)max_seqlen_q * num_q_heads + kWarps - 1) / kWarps;
  if (units > INT32_MAX || num_seqs > 65535) return PKV_ERR_UNSUPPORTED;
  TreeParams prm{};
  prm.q = static_cast<const uint16_t *>(q);
  prm.q_stride = q_tok_stride;
  prm.total_q = total_q;
  prm.k_cache = static_cast<const uint8_t *>(k_cache);
  prm.v_cache = static_cast<const uint8_t *>(v_cache);
  prm.k_scale = k_scale;
  prm.v_scale = v_scale;
  prm.block_tables = block_tables;
  prm.table_width = block_table_width;
  prm.context_lens = context_lens;
  prm.cu = cu_seqlens_q;
  prm.max_nodes = max_seqlen_q;
  prm.max_context = max_context_len;
  prm.mask = reinterpret_cast<const uint64_t *>(tree_mask);
  prm.mask_words = mask_words;
  prm.hq = num_q_heads;
  prm.hkv = num_kv_heads;
  prm.block_size = block_size;
  prm.num_blocks = num_blocks;
  prm.scale_log2 = scale * kLog2e;
  prm.out = static_cast<uint16_t *>(out);
  prm.err = err;
  const dim3 grid((unsigned)units, (unsigned)num_seqs);
  if (fp8) tree_attn_kernel<true><<<grid, kWarps * 32, 0, static_cast<cudaStream_t>(stream)>>>(prm);
  else tree_attn_kernel<false><<<grid, kWarps * 32, 0, static_cast<cudaStream_t>(stream)>>>(prm);
  return cudaGetLastError() == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // namespace
}  // namespace pkv

extern "C" size_t pkv_tree_workspace_bytes(int32_t num_seqs, int32_t max_seqlen_q,
                                           int32_t num_q_heads, int32_t num_kv_heads,
                                           int32_t head_dim, int32_t max_context_len) {
  if (num_seqs < 0 || max_seqlen_q < 0 || num_q_heads <= 0 || num_kv_heads <= 0 ||
      num_q_heads % num_kv_heads != 0 || head_dim != pkv::kD || max_context_len < 0)
    return 0;
  return 16;
}

extern "C" pkv_status pkv_paged_tree_attn(
    const void *q, int64_t q_tok_stride, int64_t total_q, const void *k_cache, const void *v_cache,
    const int32_t *block_tables, int32_t block_table_width, const int32_t *context_lens,
    const int32_t *cu_seqlens_q, int32_t num_seqs, int32_t max_seqlen_q, int32_t max_context_len,
    const int64_t *tree_mask, int32_t mask_words, int32_t num_q_heads, int32_t num_kv_heads,
    int32_t head_dim, int32_t block_size, int64_t num_blocks, float scale, void *workspace,
    size_t workspace_bytes, void *out, void *stream) {
  return pkv::tree_attn(q, q_tok_stride, total_q, k_cache, v_cache, nullptr, nullptr, false,
                        block_tables, block_table_width, context_lens, cu_seqlens_q, num_seqs,
                        max_seqlen_q, max_context_len, tree_mask, mask_words, num_q_heads,
                        num_kv_heads, head_dim, block_size, num_blocks, scale, workspace,
                        workspace_bytes, out, stream);
}

extern "C" pkv_status pkv_paged_tree_attn_fp8(
    const void *q, int64_t q_tok_stride, int64_t total_q, const void *k_cache, const void *v_cache,
    const float *k_scale, const float *v_scale, const int32_t *block_tables,
    int32_t block_table_width, const int32_t *context_lens, const int32_t *cu_seqlens_q,
    int32_t num_seqs, int32_t max_seqlen_q, int32_t max_context_len, const int64_t *tree_mask,
    int32_t mask_words, int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim,
    int32_t block_size, int64_t num_blocks, float scale, void *workspace, size_t workspace_bytes,
    void *out, void *stream) {
  return pkv::tree_attn(q, q_tok_stride, total_q, k_cache, v_cache, k_scale, v_scale, true,
                        block_tables, block_table_width, context_lens, cu_seqlens_q, num_seqs,
                        max_seqlen_q, max_context_len, tree_mask, mask_words, num_q_heads,
                        num_kv_heads, head_dim, block_size, num_blocks, scale, workspace,
                        workspace_bytes, out, stream);
}

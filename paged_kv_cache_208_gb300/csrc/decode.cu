// decode.cu -- paged decode attention over the bf16 cache: the split plan of every decode call
// and the launches. The kernel is in decode_kernel.cuh.
#include "decode_kernel.cuh"

namespace pkv {

DecodePlan plan_decode(int32_t batch, int32_t num_q_heads, int32_t num_kv_heads,
                       int32_t max_context_len, int32_t num_splits, int num_sms, bool fp8,
                       bool weights) {
  DecodePlan p{};
  const int group = num_q_heads / num_kv_heads;
  const int kTile = fp8 ? 128 : 64;
  // bf16: one or two heads a unit. 8-bit: as many of a group as its 8 MMA columns hold (the
  // heads of a unit read each code once), rounded up to a kernel instance.
  p.heads_per_cta = fp8 ? (group > 4 ? 8 : group > 2 ? 4 : group) : (group % 2 == 0) ? 2 : 1;
  p.head_groups = (group + p.heads_per_cta - 1) / p.heads_per_cta;
  const int64_t max_ctx = max_context_len > 0 ? max_context_len : 1;
  const int64_t max_tiles = (max_ctx + kTile - 1) / kTile;
  if (num_splits > 0) {
    const int64_t S = num_splits < max_tiles ? num_splits : max_tiles;
    const int64_t per = (max_ctx + S - 1) / S;
    p.chunk = (int32_t)((per + kTile - 1) / kTile * kTile);
  } else {
    // At most 16 tiles per unit (a CTA streams its unit through a 3-tile ring, so long
    // units cap the bandwidth of a skewed batch; the work queue balances short ones), or 32
    // once there are at least 8 units per SM: then the queue hides the long units' tail, and
    // one split fewer saves the partial results and the merge (Qwen3 batch, 256 contexts up
    // to 2048 tokens: 1 split 178.5 us per call against 179.9 us with 2). Below that, more
    // splits give more CTAs for a small batch, but every CTA past one per SM shares an SM,
    // and a unit's fixed costs (its first tile's latency, the merges) do not shrink.
    // Measured on batches 1..64 at 1024 tokens, the best split count is the largest that
    // keeps its splits within one cluster and the grid within about 1.7 CTAs per SM, or
    // within one CTA per SM for clusters of more than 4 (larger clusters do not all fit at
    // once when SMs hold two CTAs).
    const int64_t units = (int64_t)batch * num_kv_heads * p.head_groups;
    const int64_t max_unit_tiles = units >= 8LL * num_sms ? 32 : 16;
    int64_t S = (max_tiles + max_unit_tiles - 1) / max_unit_tiles;
    while (S < max_tiles && S < kMaxCluster &&
           units * (S + 1) <= (S + 1 > 4 ? (int64_t)num_sms : (int64_t)num_sms * 17 / 10))
      ++S;
    const int64_t per = (max_ctx + S - 1) / S;
    p.chunk = (int32_t)((per + kTile - 1) / kTile * kTile);
  }
  p.splits = (int32_t)((max_ctx + p.chunk - 1) / p.chunk);
  const size_t partials =
      p.splits > 1 ? (size_t)batch * num_q_heads * p.splits * (kD + 1) * sizeof(float) : 0;
  p.workspace_bytes = kDecodeQueueBytes + (partials + 15) / 16 * 16;  // the counters first
  if (weights) {
    p.lse_at = p.workspace_bytes;
    p.scores_at = p.lse_at + align16((size_t)batch * num_q_heads * sizeof(float));
    p.score_stride = (int64_t)p.splits * p.chunk;
    p.workspace_bytes =
        p.scores_at + (size_t)batch * num_q_heads * p.score_stride * sizeof(float);
  }
  return p;
}

cudaError_t launch_paged_decode(const DecodeArgs &a, const DecodePlan &plan,
                                cudaStream_t stream) {
  return plan.scores_at ? launch_decode<false, true>(a, plan, stream)
                        : launch_decode<false, false>(a, plan, stream);
}

}  // namespace pkv

// launch.h -- host-side launchers behind the C ABI (internal to libpkv).
//
// The extern "C" entry points in pkv_api.cu validate arguments and then call these; each
// launcher only enqueues kernels on `stream` and returns the launch status.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace pkv {

inline size_t align16(size_t x) { return (x + 15) & ~size_t(15); }

// Do the `rows` rows of `bytes` bytes at a, `stride` bytes apart, reach into the `size` bytes at b?
// (A gap between rows counts as theirs.)
inline bool overlap(const void *a, int64_t rows, __int128 stride, int64_t bytes, const void *b,
                    int64_t size) {
  if (rows <= 0 || bytes <= 0 || size <= 0) return false;
  const __int128 x = (__int128)reinterpret_cast<uintptr_t>(a);
  const __int128 y = (__int128)reinterpret_cast<uintptr_t>(b);
  return x < y + size && y < x + (__int128)(rows - 1) * stride + bytes;
}

// kv_store.cu
cudaError_t launch_kv_store(const void *k, int64_t k_tok_stride, const void *v,
                            int64_t v_tok_stride, const int64_t *slot_mapping, int64_t num_tokens,
                            void *k_cache, void *v_cache, int64_t num_slots, int64_t row_elems,
                            unsigned int *err, int num_sms, cudaStream_t stream);

// decode.cu
struct DecodePlan {
  int32_t chunk;       // logical tokens per split (a multiple of the tile: 64, of an 8-bit cache 128)
  int32_t splits;      // splits of the longest context
  int32_t head_groups; // units per KV head and split
  int32_t heads_per_cta;  // query heads of a unit: at most 2, with weights 4, of an 8-bit cache 8
  int32_t max_cluster; // splits that may meet in a cluster
  size_t workspace_bytes;
  // with weights: where the log2-sum-exps and the scores [batch, num_q_heads, score_stride]
  // lie in the workspace (0: no weights)
  size_t lse_at;
  size_t scores_at;
  int64_t score_stride;
};
DecodePlan plan_decode(int32_t batch, int32_t num_q_heads, int32_t num_kv_heads,
                       int32_t max_context_len, int32_t num_splits, int num_sms,
                       bool fp8 = false, bool weights = false);

struct DecodeArgs {
  const void *q;
  const void *k_cache;
  const void *v_cache;
  const int32_t *block_tables;
  int32_t table_width;
  const int32_t *context_lens;
  int32_t batch;
  int32_t num_q_heads;
  int32_t num_kv_heads;
  int32_t block_size;
  int64_t num_blocks;
  float scale;
  void *workspace;
  void *out;
  unsigned int *err;
  int num_sms;
  // optional: the step's new tokens, stored into the pools before they are read (one per
  // sequence, [batch, num_kv_heads, 128] with these token strides, at slot_mapping[b])
  const void *k_new = nullptr;
  const void *v_new = nullptr;
  int64_t k_new_stride = 0;
  int64_t v_new_stride = 0;
  const int64_t *slot_mapping = nullptr;
  int64_t num_slots = 0;
  // 8-bit cache: [num_blocks, num_kv_heads, block_size / 64]
  const float *k_scale = nullptr;
  const float *v_scale = nullptr;
  // attention weights [batch, num_kv_heads, >= max_context_len], rows these strides apart
  const float *weights_in = nullptr;
  int64_t weights_in_stride = 0;
  float *weights_out = nullptr;
  int64_t weights_out_stride = 0;
  // a longer context is an error and counts as this long (without it: what the splits hold)
  int32_t max_context_len = INT32_MAX;
};
constexpr size_t kDecodeQueueBytes = 16;  // the workspace's header: the work counters
cudaError_t launch_paged_decode(const DecodeArgs &a, const DecodePlan &plan,
                                cudaStream_t stream);
// the units of a call go through the work queue (else each CTA has one, and splits meet in clusters)
bool decode_queued(const DecodeArgs &a, const DecodePlan &plan);
// the decode kernel itself forms the attention weights: no kernel after it does
bool decode_forms_weights(const DecodeArgs &a, const DecodePlan &plan);

// decode_fp8.cu
cudaError_t launch_paged_decode_fp8(const DecodeArgs &a, const DecodePlan &plan,
                                    cudaStream_t stream);

// prefill.cu
struct PrefillArgs {
  const void *q;
  int64_t q_tok_stride;
  int64_t total_q;   // rows of q (and of out)
  const void *k;
  const void *v;
  int64_t kv_tok_stride;
  int64_t kv_rows;   // rows addressable through k/v (Tk, or num_blocks * block_size)
  const int32_t *cu_seqlens_q;
  const int32_t *cu_seqlens_k;
  int32_t num_seqs;
  int32_t max_seqlen_q;
  int32_t max_seqlen_k;
  const int32_t *block_table;
  int32_t table_width;
  int32_t block_size;
  int64_t num_blocks;
  int32_t num_q_heads;
  int32_t num_kv_heads;
  float scale;
  int32_t causal;
  void *out;
  void *workspace;   // prefill_workspace_layout(...).bytes: the work list and its counter
  unsigned int *err;
};

// The prefill workspace: a 16-byte header (work counter, number of work units), the
// per-sequence query-block counts, the sequences ranked by that count, the first unit of each
// ranked sequence, two histograms over the counts, and the unit list itself -- one
// (sequence, query block) pair per unit, at most num_seqs * ceil(max_seqlen_q / 128).
struct PrefillWorkspace {
  size_t counts, ranked, unit_start, hist, fill, units, bytes;
  int64_t max_units;
  int32_t levels;  // ceil(max_seqlen_q / 128): the query blocks of the longest sequence
};
inline PrefillWorkspace prefill_workspace_layout(int32_t num_seqs, int32_t max_seqlen_q) {
  PrefillWorkspace w{};
  w.levels = (int32_t)(((int64_t)max_seqlen_q + 127) / 128);
  w.max_units = (int64_t)num_seqs * w.levels;
  const size_t n = (size_t)num_seqs, l = (size_t)w.levels + 1;
  w.counts = 16;
  w.ranked = align16(w.counts + 4 * n);
  w.unit_start = align16(w.ranked + 4 * n);
  w.hist = align16(w.unit_start + 4 * (n + 1));
  w.fill = align16(w.hist + 4 * l);
  w.units = align16(w.fill + 4 * l);
  w.bytes = align16(w.units + 8 * (size_t)w.max_units);
  return w;
}
cudaError_t launch_varlen_prefill(const PrefillArgs &a, int num_sms, cudaStream_t stream);
bool prefill_group_supported(int group);  // num_q_heads / num_kv_heads

// Launch as a programmatic dependent of the stream's previous kernel: the launch overlaps that
// kernel's tail. The kernel has to wait for it (griddepcontrol.wait) before it reads or writes
// anything another kernel touches.
template <class... Formal, class... Args>
inline cudaError_t launch_after(void (*kernel)(Formal...), dim3 grid, int threads,
                                cudaStream_t stream, Args... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// the current device's SM count and the address of the device error word (pkv_api.cu);
// 0 / nullptr when the CUDA runtime cannot answer
int current_sm_count();
unsigned int *current_error_word();

// tensor maps (pkv_api.cu): the driver's cuTensorMapEncodeTiled, fetched at run time
CUresult encode_tensor_map(CUtensorMap *map, CUtensorMapDataType dtype, uint32_t rank,
                           void *base, const uint64_t *dims, const uint64_t *strides_bytes,
                           const uint32_t *box, CUtensorMapSwizzle swizzle,
                           CUtensorMapL2promotion promotion);

}  // namespace pkv

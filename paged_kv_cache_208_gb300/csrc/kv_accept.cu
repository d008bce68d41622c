// kv_accept.cu -- after the drafted tokens of a step have been judged: the rows of the accepted
// path of each sequence's tree move up behind the context, in place.
//
// The nodes of sequence b are positions P .. L - 1, P = L - n. Row P + j becomes row P + a_j for
// the accepted nodes a_0 < a_1 < .. of the path. Ascending nodes have a_j >= j, so no row is
// written that a later one still reads: rows are moved in passes of ascending j, each pass read
// whole before it is written. In an 8-bit cache the rows that come into a group of 64 positions
// may bring larger scales: the group then takes the largest, and what it holds is re-rounded.
//
// One CTA owns K or V of a sequence for some of its heads. The bytes are few (the moved rows, read
// and written once), so what counts is the chain of dependent loads: list and lengths, table, rows
// (and their scales beside them). Each step of it is taken for all rows at once. 8 small trees take
// 2.8 us, which is that chain; the paths of 256 trees of 64 nodes (37 MB) 8.9 us, 9.6 us in the 8-bit
// cache (18 MB, the scales, the re-rounding of groups whose scale grew): 14.4 and 18.8 us with CTAs of
// 256 threads, of which four fit on an SM, divisions in place of shifts, and the rows asked for after
// the scales; 12.1 us in 8 bits with 80 registers a thread, so that a wave held 912 of the 1024 CTAs
// (four loads at once for the re-rounding: 11.0, by its registers).
#include <math.h>

#include <algorithm>

#include "device_common.cuh"
#include "fp8_cache.cuh"
#include "launch.h"
#include "pkv.h"

namespace pkv {
namespace {

constexpr int kD = 128;
constexpr int kThreads = 128;
constexpr int kRows = 64;       // rows of a round: in an 8-bit cache those of one group
constexpr int kMaxHeads = 8;    // heads of a CTA
constexpr int kLoads = 8;       // 16-byte pieces of a thread in flight

struct AcceptParams {
  const int32_t *accepted;
  int32_t accepted_width;
  const int32_t *num_accepted;
  const int32_t *cu;
  const int32_t *context_lens;
  const int32_t *block_tables;
  int32_t table_width;
  uint8_t *k_cache, *v_cache;
  float *k_scale, *v_scale;
  int32_t hkv, block_size;
  int32_t heads_shift;  // a CTA's heads, as a power of two
  int64_t num_blocks;
  int32_t *new_context_lens;
  unsigned int *err;
};

__device__ __forceinline__ uint4 rescale16(uint4 w, float ratio) {
  return make_uint4(rescale4(w.x, ratio), rescale4(w.y, ratio), rescale4(w.z, ratio),
                    rescale4(w.w, ratio));
}

template <bool F8>
__global__ void __launch_bounds__(kThreads, 7) kv_accept_kernel(const AcceptParams p) {
  constexpr int kShift = F8 ? 3 : 4;  // a head's row has 2^kShift pieces of 16 bytes
  __shared__ int64_t src_row[kRows], dst_row[kRows];  // pool rows; -1: a bad block
  __shared__ float src_scale[F8 ? kRows : 1][kMaxHeads];
  __shared__ float old_scale[kMaxHeads];
  __shared__ uint32_t new_scale[kMaxHeads];  // bits: of positive numbers in the same order
  __shared__ int32_t path[kThreads];  // the list's first entries
  __shared__ int32_t count;
  const int tid = threadIdx.x;
  const int per = 1 << p.heads_shift, parts = (p.hkv + per - 1) >> p.heads_shift;
  const int part = blockIdx.x % parts;
  const bool is_v = (blockIdx.x / parts) & 1;
  const int b = blockIdx.x / parts / 2;
  const int h0 = part * per, heads = min(per, p.hkv - h0);
  const bool first = part == 0 && !is_v;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int32_t *list = p.accepted + (int64_t)b * p.accepted_width;
  path[tid] = tid < p.accepted_width ? *(list + tid) : -1;
  const int64_t c0 = *(p.cu + b), c1 = *(p.cu + b + 1), L = *(p.context_lens + b);
  int many = *(p.num_accepted + b);
  const int64_t n = c1 - c0, start = L - n;
  // an earlier wait gave up somewhere: write nothing (decided by the CTA together)
  if (__syncthreads_or(tid == 0 && aborted(p.err))) return;
  if (n < 0 || start < 0 || L > (int64_t)p.table_width * p.block_size) {
    if (first && tid == 0) {
      record_error(p.err, n < 0 ? PKV_DEVERR_SEQLEN_RANGE : PKV_DEVERR_CONTEXT_RANGE);
      p.new_context_lens[b] = 0;
    }
    return;
  }
  if (many < 0 || many > n || many > p.accepted_width) {
    if (first && tid == 0) record_error(p.err, PKV_DEVERR_NODE_RANGE);
    many = 0;
  }
  auto entry = [&](int j) { return j < kThreads ? path[j] : *(list + j); };
  // the path ends before the first entry that is no later node of the tree
  if (tid == 0) count = many;
  __syncthreads();
  for (int j = tid; j < many; j += kThreads) {
    const int32_t a = entry(j), before = j ? entry(j - 1) : -1;
    if (a <= before || a >= n) {
      atomicMin(&count, j);
      if (first) record_error(p.err, PKV_DEVERR_NODE_RANGE);
    }
  }
  __syncthreads();
  many = count;
  if (first && tid == 0) p.new_context_lens[b] = (int32_t)start + many;
  if (many == 0) return;
  const int32_t *table = p.block_tables + (int64_t)b * p.table_width;
  auto pool_row = [&](int64_t pos) -> int64_t {
    const int64_t blk = *(table + pos / p.block_size);
    if (blk < 0 || blk >= p.num_blocks) {
      record_error(p.err, PKV_DEVERR_BLOCK_RANGE);
      return -1;
    }
    return blk * p.block_size + pos % p.block_size;
  };
  uint8_t *const pool = is_v ? p.v_cache : p.k_cache;
  float *const scales = is_v ? p.v_scale : p.k_scale;
  const int groups = p.block_size / kFp8Group;
  auto scale_at = [&](int64_t row, int h) -> int64_t {
    return (row / p.block_size * p.hkv + h) * groups + row % p.block_size / kFp8Group;
  };
  const int64_t row_pieces = (int64_t)p.hkv << kShift;
  // A thread always has the same piece of a row (kThreads is a multiple of a row's pieces): it
  // counts those of absent heads too, so that a row's number is a shift.
  const int shift = p.heads_shift + kShift, piece = tid & ((1 << shift) - 1), h = piece >> kShift;
  const int row_step = kThreads >> shift, r0 = tid >> shift;
  const bool any = h < heads;
  uint4 *const base = reinterpret_cast<uint4 *>(pool) + (h0 << kShift) + piece;
  auto piece_of = [&](int64_t row) { return base + row * row_pieces; };
  for (int j0 = 0, rows; j0 < many; j0 += rows) {
    rows = min(kRows, many - j0);
    // (of an 8-bit cache: the rows that go to one group)
    if (F8) rows = min(rows, kFp8Group - (int)((start + j0) % kFp8Group));
    if (tid < rows) {
      src_row[tid] = pool_row(start + entry(j0 + tid));
      dst_row[tid] = pool_row(start + j0 + tid);
    }
    if (F8 && tid < kMaxHeads) new_scale[tid] = 0;
    __syncthreads();
    for (int i0 = 0; i0 < rows; i0 += row_step * kLoads) {
      uint4 x[kLoads];
#pragma unroll
      for (int u = 0; u < kLoads; ++u) {
        const int r = i0 + u * row_step + r0;
        x[u] = make_uint4(0, 0, 0, 0);
        if (any && r < rows && src_row[r] >= 0) x[u] = *piece_of(src_row[r]);
      }
      const int64_t d0 = dst_row[0];
      if (F8 && i0 == 0 && d0 >= 0) {  // (while the rows are on their way)
        auto raise = [&](int k, float s) {
          if (s > 0.f) atomicMax(&new_scale[k], __float_as_uint(s));
        };
        if (tid < heads) {
          old_scale[tid] = scales[scale_at(d0, h0 + tid)];
          raise(tid, old_scale[tid]);
        }
        for (int i = tid; i < rows << p.heads_shift; i += kThreads) {
          const int r = i >> p.heads_shift, k = i & (per - 1);
          const float s =
              k < heads && src_row[r] >= 0 ? scales[scale_at(src_row[r], h0 + k)] : 0.f;
          src_scale[r][k] = s;
          raise(k, s);
        }
        __syncthreads();
        if (tid < heads && __uint_as_float(new_scale[tid]) > old_scale[tid])
          scales[scale_at(d0, h0 + tid)] = __uint_as_float(new_scale[tid]);
        // the rows of the group from before the tree, at the scale that grew
        const int before = j0 == 0 ? (int)(start % kFp8Group) : 0;
        const float scale = __uint_as_float(new_scale[h]);
        if (any && scale > old_scale[h])
          for (int r = r0; r < before; r += row_step) {
            uint4 *w = piece_of(d0 - before + r);
            *w = rescale16(*w, old_scale[h] / scale);
          }
      }
      __syncthreads();  // (each pass is read before it is written)
#pragma unroll
      for (int u = 0; u < kLoads; ++u) {
        const int r = i0 + u * row_step + r0;
        if (!any || r >= rows || dst_row[r] < 0) continue;
        bool same = src_row[r] == dst_row[r];
        if (F8) {
          const float ratio = src_scale[r][h] / __uint_as_float(new_scale[h]);
          if (ratio < 1.f) {
            x[u] = rescale16(x[u], ratio);
            same = false;
          }
        }
        if (!same) *piece_of(dst_row[r]) = x[u];
      }
      __syncthreads();
    }
  }
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace
}  // namespace pkv

extern "C" pkv_status pkv_kv_accept(const int32_t *accepted, int32_t accepted_width,
                                    const int32_t *num_accepted, const int32_t *cu_seqlens_q,
                                    const int32_t *context_lens, const int32_t *block_tables,
                                    int32_t block_table_width, int32_t num_seqs, void *k_cache,
                                    void *v_cache, float *k_scale, float *v_scale,
                                    int32_t num_kv_heads, int32_t head_dim, int32_t block_size,
                                    int64_t num_blocks, int32_t *new_context_lens, void *stream) {
  using namespace pkv;
  if (num_seqs < 0 || accepted_width < 0 || num_kv_heads <= 0 || head_dim <= 0 ||
      block_size <= 0 || num_blocks <= 0 || block_table_width <= 0)
    return PKV_ERR_INVALID_ARG;
  if (num_seqs == 0) return PKV_OK;
  if (!num_accepted || !cu_seqlens_q || !context_lens || !block_tables || !k_cache || !v_cache ||
      !new_context_lens || (accepted_width > 0 && !accepted) || !k_scale != !v_scale)
    return PKV_ERR_INVALID_ARG;
  // (the calls of a step's other layers read the old lengths, and the CTAs of a sequence its numbers)
  const int64_t ints = 4 * (int64_t)num_seqs;
  if (overlap(new_context_lens, 1, 0, ints, context_lens, ints) ||
      overlap(new_context_lens, 1, 0, ints, num_accepted, ints) ||
      overlap(new_context_lens, 1, 0, ints, cu_seqlens_q, ints + 4) ||
      overlap(new_context_lens, 1, 0, ints, accepted, ints * accepted_width) ||
      overlap(new_context_lens, 1, 0, ints, block_tables, ints * block_table_width))
    return PKV_ERR_INVALID_ARG;
  if (head_dim != kD || block_size % (k_scale ? 256 : kFp8Group) != 0) return PKV_ERR_UNSUPPORTED;
  if (!aligned16(k_cache) || !aligned16(v_cache)) return PKV_ERR_UNSUPPORTED;
  const int num_sms = current_sm_count();
  unsigned int *err = current_error_word();
  if (num_sms <= 0 || !err) return PKV_ERR_CUDA;
  AcceptParams prm{};
  prm.accepted = accepted;
  prm.accepted_width = accepted_width;
  prm.num_accepted = num_accepted;
  prm.cu = cu_seqlens_q;
  prm.context_lens = context_lens;
  prm.block_tables = block_tables;
  prm.table_width = block_table_width;
  prm.k_cache = static_cast<uint8_t *>(k_cache);
  prm.v_cache = static_cast<uint8_t *>(v_cache);
  prm.k_scale = k_scale;
  prm.v_scale = v_scale;
  prm.hkv = num_kv_heads;
  prm.block_size = block_size;
  prm.num_blocks = num_blocks;
  prm.new_context_lens = new_context_lens;
  prm.err = err;
  // as many heads to a CTA as still leave every SM about six CTAs
  while ((2 << prm.heads_shift) <= kMaxHeads && (1 << prm.heads_shift) < num_kv_heads &&
         2 * (int64_t)num_seqs * num_kv_heads >> (prm.heads_shift + 1) >= 6 * (int64_t)num_sms)
    ++prm.heads_shift;
  const int64_t grid = 2 * (int64_t)num_seqs *
                       ((num_kv_heads + (1 << prm.heads_shift) - 1) >> prm.heads_shift);
  if (grid > INT32_MAX) return PKV_ERR_UNSUPPORTED;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e =
      k_scale ? launch_after(kv_accept_kernel<true>, (unsigned)grid, kThreads, st, prm)
              : launch_after(kv_accept_kernel<false>, (unsigned)grid, kThreads, st, prm);
  return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

// tree_attn.cu -- attention of drafted tokens over the paged cache (paged_tree_attn): the last n
// positions of a context are the nodes of a tree, and each attends to the context before them and
// to the nodes that its mask names.
//
// The rows that share a KV head -- (node, query head of the group) pairs -- attend over the same
// keys, so all of them together are the M of a matrix product: K and V are read once for up to
// 128 rows (64 nodes of two heads, 16 of eight). With some tens of rows a key of 512 bytes
// costs 512 * rows multiplications, far below what the tensor cores do in the time of its load:
// the kernel is bound by HBM, and its work is cut so that every SM reads the same number of keys.
//
// Work. A unit is (sequence, KV head, tile of 128 rows); its length is its context in granules
// of 64 keys. All units in a row make one axis of granules, which the workers share out
// evenly: worker w takes [w T / W, (w + 1) T / W), whatever the units' lengths. The lengths are
// device data, so every CTA sums them up at its start (one scan over the sequences) and walks its
// own part. A unit that lies within a worker's part is written out directly; what a cut leaves is
// normalised, goes to the workspace with its log2-sum-exp, and tree_combine_kernel merges it.
// Which parts there are depends on the lengths alone, so the same call gives the same bits.
// Where trees have more rows than a tile, `group` neighbouring CTAs are one worker and take the
// row tiles of the same keys at the same time: K and V then come from L2 for all but one of them.
//
// Per tile of 128 keys (M = 128 rows, one CTA):
//   S = Q K^T    Q in tensor memory (the A operand), K rows in shared memory
//   softmax      8 warps, two threads to a row: running maximum and sum in fp32, P = 2^(s - m)
//                written back over S as two bf16 parts (P = hi + lo within 2^-17 of itself): the
//                second product's cost is hidden behind the loads, and the output differs from
//                one with fp32 weights in its last rounding only
//   O += P V     P from tensor memory, V rows in shared memory
// S has two buffers, Q two (the next unit's is loaded while this one's tiles are in work).
// O is rescaled only when a row's maximum grows by more than 2^8, as in prefill.cu.
//
// Rows. 16 rows make a chunk: nb = 16 / G nodes with their G query heads (with more than 16 heads
// one node and 16 of them). Chunk c of a tile lies in 16 of the 128 TMEM lanes that warp c reads,
// lane quadrant c % 4: with few rows the softmax is spread over all four SM sub-partitions.
//
// Warps (512 threads): 0-7 softmax and epilogue (warp c: chunk c), 8 work walk and K loads, 9 S
// products, 10 V loads, 11 PV products, 12-15 Q into tensor memory. Loads are TMA with 128-byte
// swizzle, 64 keys to a box (a granule never straddles a block).
// TMEM (512 columns): Q [0, 64) [64, 128), S [128, 256) [256, 384), O [384, 512).
//
// Masked places. A key that a row does not see is left out of its maximum and gets P = 0; V rows
// past the context are zeroed in shared memory. A node that others do not see may hold
// infinities or NaNs, and 0 x NaN would reach them: the V warp looks through the nodes' rows, puts
// zeros in the place of what is not finite, and the rows that do see such a node are put right
// in memory (not_finite_fix).
#include <math.h>

#include <algorithm>

#include "device_common.cuh"
#include "fp8_cache.cuh"
#include "launch.h"
#include "pkv.h"
#include "tcgen05.cuh"

namespace pkv {
namespace {

constexpr int kD = 128;
constexpr unsigned kFull = 0xffffffffu;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kRescaleLog2 = 8.0f;
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
  int32_t num_seqs;
  float scale_log2;  // of the scale's magnitude
  uint32_t q_sign;   // flips the signs of two bf16 where the scale is negative
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

constexpr int kTile = 128;    // keys
constexpr int kGranule = 64;  // keys of a TMA box, and what the work is measured in
constexpr int kChunkRows = 16;
constexpr int kChunks = 8;    // of a row tile
constexpr int kSoftmaxWarps = 8;
constexpr int kKWarp = 8, kSWarp = 9, kVWarp = 10, kPvWarp = 11, kQWarp0 = 12;
constexpr int kThreads = 16 * 32;
constexpr int kKSlots = 4, kVSlots = 3;
constexpr uint32_t kTileBytes = kTile * kD * 2;
constexpr uint32_t kPlane = kTileBytes / 2;         // 64 dims of the tile's keys, 128-byte rows
constexpr uint32_t kGranuleBytes = kGranule * 128;  // of a plane
constexpr int kRing = 4;
constexpr uint32_t kQCol = 0, kSCol = 128, kOCol = 384, kTmemCols = 512;
constexpr int kItemConsumers = kSoftmaxWarps + 3 + 4;  // S, V, PV and Q warps
constexpr int kMaxGroup = 4;

// A worker's share of a unit.
struct Item {
  int32_t last;        // 1: no more work
  int32_t b, h;
  int32_t q0, n, L;    // the sequence's rows of q, its nodes and its context (0: an empty one)
  int32_t c0, chunks;  // the row tile's first chunk, and its chunks
  int32_t key0, key1;  // positions
  int32_t tiles;
  int32_t to;          // 0, 1: a partial result, into this slot of the CTA's; 2: the output
  int32_t pad[4];
};
static_assert(sizeof(Item) == 64, "");

// What tree_combine_kernel has to know of a CTA's first item.
struct CutInfo {
  int32_t parts;       // 0: this CTA's part starts with a unit, or is not the unit's first cut
  int32_t b, h, q0, n, L, c0, chunks;
  int32_t dirty[2];    // the slots' items met values that are not finite
  int32_t pad[6];
};
static_assert(sizeof(CutInfo) == 64, "");

struct TreeSmem {
  uint8_t k[kKSlots][kTileBytes];  // 1024-byte aligned (128-byte swizzle atoms)
  uint8_t v[kVSlots][kTileBytes];
  Item items[kRing];
  int32_t dirty[kRing];            // of the item in this ring slot
  uint64_t k_full[kKSlots], k_empty[kKSlots], v_full[kVSlots], v_empty[kVSlots];
  uint64_t v_fixed[kVSlots];       // rows past the context zeroed, nodes looked through
  uint64_t q_full[2], q_empty[2];
  uint64_t s_full[2], p_full[2], o_full[2], o_free, drain[2];
  uint64_t item_full[kRing], item_empty[kRing], scanned[kRing];
  uint32_t tmem_base;
  int32_t stop;
  int64_t warp_sums[16];
  int32_t start_b;                 // the sequence that the CTA's part starts in
  int64_t start_at, total;         // where that sequence starts on the axis; the axis' length
};

static_assert(sizeof(TreeSmem) + 1024 <= 232448, "fits the SM");

struct FlashParams {
  TreeParams t;
  int32_t group, workers;  // CTAs of a worker; workers
  int32_t hb, nb, parts;   // heads and nodes of a chunk; chunks that share its nodes
  bool out_32b;
  CutInfo *cuts;           // one per CTA
  float *part_o, *part_lse;  // [CTA][2][rows][kD], [CTA][2][rows]
  int32_t part_rows;
};

// Rows of a sequence as the work is counted: its nodes (0: none, or a bad cu_seqlens) and its
// context (0 also for a bad length, whose rows become zeros).
struct Seq {
  int32_t q0, n, L;
  int64_t units, length;  // row tiles (of `group` CTAs) x KV heads, granules of one
  __device__ __forceinline__ int64_t cost() const { return units * length; }
};
__device__ __forceinline__ Seq sequence(const FlashParams &f, int b, bool record) {
  const TreeParams &p = f.t;
  Seq s{};
  const int64_t c0 = ld_global_s32(p.cu + b), c1 = ld_global_s32(p.cu + b + 1);
  const int64_t L = ld_global_s32(p.context_lens + b);
  const int64_t n = c1 - c0;
  if (c0 < 0 || n < 0 || c1 > p.total_q || n > p.max_nodes) {
    if (record) record_error(p.err, PKV_DEVERR_SEQLEN_RANGE);
    return s;
  }
  if (n == 0) return s;
  const bool ok = L >= n && L <= p.max_context && L <= (int64_t)p.table_width * p.block_size;
  if (!ok && record) record_error(p.err, PKV_DEVERR_CONTEXT_RANGE);
  s.q0 = (int32_t)c0;
  s.n = (int32_t)n;
  s.L = ok ? (int32_t)L : 0;
  const int chunks = (s.n + f.nb - 1) / f.nb * f.parts;
  const int per = kChunks * f.group;
  s.units = (int64_t)p.hkv * ((chunks + per - 1) / per);
  s.length = max(1, (s.L + kGranule - 1) / kGranule);
  return s;
}

// Bit j - 64 w of the result: node `node` (row `row` of q) sees node j, for 64 w <= j < 64 (w + 1).
__device__ __forceinline__ uint64_t mask_word(const TreeParams &p, int64_t row, int node, int w) {
  if (p.mask) return w < p.mask_words ? p.mask[row * p.mask_words + w] : 0;
  const int top = node - 64 * w;
  return top < 0 ? 0 : top >= 63 ? ~0ull : (2ull << top) - 1;
}

// V rows of the nodes that a row sees may hold values that are not finite, which the products left
// out: what they add up to replaces the row's result. dims [d0, d0 + count), count a multiple of 4.
__device__ __forceinline__ void not_finite_fix(const TreeParams &p, int b, int h, int n, int L,
                                            int64_t row, int node, uint16_t *out, int d0,
                                            int count) {
#pragma unroll 1
  for (int d = d0; d < d0 + count; d += 4) {
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
    for (int j = 0; j < n; ++j) {
      if (!(mask_word(p, row, node, j >> 6) >> (j & 63) & 1)) continue;
      const int64_t pos = (int64_t)L - n + j;
      const int64_t blk = p.block_tables[(int64_t)b * p.table_width + pos / p.block_size];
      if (blk < 0 || blk >= p.num_blocks) continue;
      const int64_t at = ((blk * p.block_size + pos % p.block_size) * p.hkv + h) * kD + d;
      const uint2 w = *reinterpret_cast<const uint2 *>(p.v_cache + 2 * at);
      const float x[4] = {bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y)};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (!isfinite(x[i])) sum[i] += x[i];
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (!(sum[i] == 0.f)) out[d + i] = bf16_bits_rn(sum[i]);
  }
}

// Walks a worker's part of the axis, one item at a time (one thread).
struct Walk {
  int64_t x, x1, at;  // where the walk is, where the part ends, where sequence b starts
  int b;
  Seq s;
  __device__ __forceinline__ bool next(const FlashParams &f, int rank, Item &it, int64_t &unit,
                                       int64_t &off) {
    while (x < x1) {
      while (x >= at + s.cost()) {
        at += s.cost();
        s = sequence(f, ++b, false);
      }
      const int64_t rel = x - at;
      const int64_t u = rel / s.length;
      off = rel - u * s.length;
      const int64_t take = min(s.length - off, x1 - x);
      unit = x - off;
      x += take;
      const int chunks = (s.n + f.nb - 1) / f.nb * f.parts;
      it.last = 0;
      it.b = b;
      it.h = (int32_t)(u % f.t.hkv);
      it.q0 = s.q0;
      it.n = s.n;
      it.L = s.L;
      it.c0 = ((int32_t)(u / f.t.hkv) * f.group + rank) * kChunks;
      it.chunks = min(kChunks, chunks - it.c0);
      it.key0 = (int32_t)min((int64_t)s.L, off * kGranule);
      it.key1 = (int32_t)min((int64_t)s.L, (off + take) * kGranule);
      it.tiles = (it.key1 - it.key0 + kTile - 1) / kTile;
      it.to = off > 0 ? 0 : take < s.length ? 1 : 2;
      if (it.chunks > 0) return true;  // (this CTA's row tile of a smaller tree is empty)
    }
    return false;
  }
};

// First pool row of the granule at position pos; a bad block id is flagged and gives a row wholly
// outside the pool (TMA fills zeros). The block id is read once per block.
struct RowOf {
  int32_t at = -1;
  int64_t blk = -1;
  __device__ __forceinline__ int32_t operator()(const TreeParams &p, int b, int32_t pos) {
    const int32_t i = pos / p.block_size;
    if (i != at) {
      at = i;
      blk = ld_global_s32(p.block_tables + (int64_t)b * p.table_width + i);
      if (blk < 0 || blk >= p.num_blocks) {
        record_error(p.err, PKV_DEVERR_BLOCK_RANGE);
        blk = -1;
      }
    }
    return blk < 0 ? -2 * kTile : (int32_t)(blk * p.block_size + pos % p.block_size);
  }
};

__device__ __forceinline__ const Item *wait_item(TreeSmem &sm, uint32_t taken, unsigned int *err) {
  const int slot = taken % kRing;
  return __all_sync(kFull, wait_parity(&sm.item_full[slot], (taken / kRing) & 1, err))
             ? &sm.items[slot]
             : nullptr;
}
__device__ __forceinline__ void release_item(TreeSmem &sm, uint32_t taken, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(&sm.item_empty[taken % kRing]);
}

__global__ void __launch_bounds__(kThreads, 1)
    tree_flash_kernel(const __grid_constant__ CUtensorMap kmap,
                      const __grid_constant__ CUtensorMap vmap,
                      const __grid_constant__ FlashParams f) {
  const TreeParams &p = f.t;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  extern __shared__ uint8_t smem_raw[];
  TreeSmem &sm = *reinterpret_cast<TreeSmem *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  if (tid == 0) {
    for (int i = 0; i < kKSlots; ++i) {
      mbar_init(&sm.k_full[i], 1);
      mbar_init(&sm.k_empty[i], 1);
    }
    for (int i = 0; i < kVSlots; ++i) {
      mbar_init(&sm.v_full[i], 1);
      mbar_init(&sm.v_empty[i], 1);
      mbar_init(&sm.v_fixed[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.q_full[i], 4);
      mbar_init(&sm.q_empty[i], 1);
      mbar_init(&sm.s_full[i], 1);
      mbar_init(&sm.p_full[i], kSoftmaxWarps);
      mbar_init(&sm.o_full[i], 1);
      mbar_init(&sm.drain[i], 1);
    }
    mbar_init(&sm.o_free, kSoftmaxWarps);
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&sm.item_full[i], 1);
      mbar_init(&sm.item_empty[i], kItemConsumers);
      mbar_init(&sm.scanned[i], 1);
    }
    sm.start_b = 0;
    sm.start_at = 0;
    fence_mbar_init();
    prefetch_tensormap(&kmap);
    prefetch_tensormap(&vmap);
  }
  if (warp == kSWarp) {
    tmem_alloc(&sm.tmem_base, kTmemCols);
    tmem_relinquish();
  }
  // everything above may overlap the stream's previous kernel
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // The axis: every sequence's granules, summed over the batch. Thread t adds up one sequence of
  // every kThreads; the sequence that the worker's part starts in is found on the way when the
  // batch fits the block, else by a second pass.
  const int worker = blockIdx.x / f.group, rank = blockIdx.x % f.group;
  auto scan = [&](int base, int64_t &mine) -> int64_t {  // exclusive prefix; sm.total: the sum
    const int b = base + tid;
    mine = b < p.num_seqs ? sequence(f, b, blockIdx.x == 0).cost() : 0;
    int64_t x = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(kFull, x, o);
      if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) sm.warp_sums[warp] = x;
    __syncthreads();
    int64_t before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) before += sm.warp_sums[w];
      all += sm.warp_sums[w];
    }
    if (tid == 0) sm.total = all;
    return before + x - mine;
  };
  int64_t total = 0, mine = 0, prefix = 0;
  for (int base = 0; base < p.num_seqs; base += kThreads) {
    prefix = scan(base, mine);
    __syncthreads();
    total += sm.total;
  }
  const int64_t workers = min((int64_t)f.workers, total);
  const bool works = worker < workers;
  const int64_t x0 = works ? worker * total / workers : 0;
  const int64_t x1 = works ? (worker + 1) * total / workers : 0;
  if (p.num_seqs <= kThreads) {
    if (mine > 0 && prefix <= x0 && x0 < prefix + mine) {
      sm.start_b = tid;
      sm.start_at = prefix;
    }
  } else {
    int64_t carry = 0;
    for (int base = 0; base < p.num_seqs; base += kThreads) {
      prefix = carry + scan(base, mine);
      if (mine > 0 && prefix <= x0 && x0 < prefix + mine) {
        sm.start_b = base + tid;
        sm.start_at = prefix;
      }
      __syncthreads();
      carry += sm.total;
    }
  }
  if (tid == 0) sm.stop = aborted(p.err) ? 1 : 0;
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = sm.tmem_base;
  // the kernel that follows may be set up (not before this CTA has its tensor memory)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (!sm.stop) {
    // (the branches below do not meet before the end: what follows setmaxnreg has its registers)
    if (warp >= kSoftmaxWarps) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == kKWarp) {
      // ------------------------------------------------------------ work walk and K loads
      if (lane == 0) {
        const uint64_t policy = f.group == 1 ? policy_evict_first() : policy_evict_last();
        Walk w{x0, x1, sm.start_at, sm.start_b, {}};
        if (works) w.s = sequence(f, w.b, false);
        uint32_t pushed = 0, g = 0;
        bool ok = true;
        CutInfo cut{};
        // the next item is handed out before this one's tiles are loaded
        Item it, nx;
        int64_t unit, off;
        auto push = [&](Item &d) -> bool {
          const bool more = w.next(f, rank, d, unit, off);
          if (!more) {
            d = Item{};
            d.last = 1;
          }
          const int slot = pushed % kRing;
          if (pushed >= kRing && !wait_parity(&sm.item_empty[slot], ((pushed / kRing) - 1) & 1, p.err))
            return false;
          sm.items[slot] = d;
          sm.dirty[slot] = 0;
          mbar_arrive(&sm.item_full[slot]);
          ++pushed;
          return true;
        };
        ok = push(it);
        // the first unit's cut, if it is that unit's first one: worker - 1 has the part before
        if (ok && !it.last && it.to == 0 && unit + off == x0 &&
            unit >= (worker - 1) * total / workers) {
          const int64_t end = unit + w.s.length - 1;
          cut.parts = (int32_t)(((end + 1) * workers - 1) / total) - worker + 2;
          cut.b = it.b;
          cut.h = it.h;
          cut.q0 = it.q0;
          cut.n = it.n;
          cut.L = it.L;
          cut.c0 = it.c0;
          cut.chunks = it.chunks;
        }
        {
          int4 *dst = reinterpret_cast<int4 *>(f.cuts + blockIdx.x);
          dst[0] = make_int4(cut.parts, cut.b, cut.h, cut.q0);
          dst[1] = make_int4(cut.n, cut.L, cut.c0, cut.chunks);
        }
        RowOf row_of;
        int last_b = -1;
        while (ok && !it.last) {
          ok = push(nx);
          if (!ok) break;
          if (it.b != last_b) row_of.at = -1;
          last_b = it.b;
          for (int j = 0; j < it.tiles; ++j, ++g) {
            const int slot = g % kKSlots;
            if (g >= kKSlots && !wait_parity(&sm.k_empty[slot], ((g / kKSlots) - 1) & 1, p.err)) {
              ok = false;
              break;
            }
            const int32_t pos = it.key0 + j * kTile;
            const int granules = it.key1 - pos > kGranule ? 2 : 1;
            mbar_arrive_expect_tx(&sm.k_full[slot], granules * 2 * kGranuleBytes);
            for (int r = 0; r < granules; ++r) {
              const int32_t row = row_of(p, it.b, pos + r * kGranule);
#pragma unroll
              for (int hf = 0; hf < 2; ++hf)
                tma_load_3d(sm.k[slot] + hf * kPlane + r * kGranuleBytes, &kmap, &sm.k_full[slot], 0,
                            row, 2 * it.h + hf, policy);
            }
          }
          it = nx;
        }
        // keep the CTA alive until every copy it issued has landed
        bool drained = true;
        for (uint32_t t = g > kKSlots ? g - kKSlots : 0; drained && t < g; ++t)
          drained = wait_own(&sm.k_full[t % kKSlots], (t / kKSlots) & 1, p.err);
      }
      __syncwarp();
    } else if (warp == kVWarp) {
      // ------------------------------------------------------------ V loads
      uint64_t policy = 0;
      if (lane == 0) policy = f.group == 1 ? policy_evict_first() : policy_evict_last();
      uint32_t taken = 0, g = 0;
      bool ok = true;
      RowOf row_of;
      int last_b = -1;
      while (ok) {
        const Item *ip = wait_item(sm, taken, p.err);
        if (!ip) break;
        const Item it = *ip;
        if (it.b != last_b) row_of.at = -1;
        last_b = it.b;
        const int root = it.L - it.n;
        bool dirty = false;
        for (int j = 0; j < it.tiles && ok && !it.last; ++j, ++g) {
          const int slot = g % kVSlots;
          const int32_t pos = it.key0 + j * kTile;
          const int keys = min(kTile, it.key1 - pos);
          if (lane == 0) {
            if (g >= kVSlots) ok = wait_parity(&sm.v_empty[slot], ((g / kVSlots) - 1) & 1, p.err);
            if (ok) {
              const int granules = keys > kGranule ? 2 : 1;
              mbar_arrive_expect_tx(&sm.v_full[slot], granules * 2 * kGranuleBytes);
              for (int r = 0; r < granules; ++r) {
                const int32_t row = row_of(p, it.b, pos + r * kGranule);
#pragma unroll
                for (int hf = 0; hf < 2; ++hf)
                  tma_load_3d(sm.v[slot] + hf * kPlane + r * kGranuleBytes, &vmap,
                              &sm.v_full[slot], 0, row, 2 * it.h + hf, policy);
              }
            }
          }
          ok = __shfl_sync(kFull, ok ? 1 : 0, 0) != 0;
          if (!ok) break;  // (g counts the copies that were issued)
          if (pos + kTile > root) {
            ok = __all_sync(kFull, wait_parity(&sm.v_full[slot], (g / kVSlots) & 1, p.err));
            if (!ok) {
              ++g;  // (its copies have been issued)
              break;
            }
            // 16-byte pieces: those of nodes looked through, those past the keys zeroed
            const int from = max(0, root - pos), up = (keys + 15) & ~15;
            bool here = false;
            for (int i = lane + from * 16; i < up * 16; i += 32) {
              uint4 *w = reinterpret_cast<uint4 *>(sm.v[slot] + ((i & 15) >> 3) * kPlane +
                                                   (i >> 4) * 128 + (i & 7) * 16);
              if ((i >> 4) >= keys) {
                *w = make_uint4(0, 0, 0, 0);
              } else {
                const uint4 x = *w;
                const uint4 y = make_uint4(bf16x2_finite(x.x), bf16x2_finite(x.y),
                                           bf16x2_finite(x.z), bf16x2_finite(x.w));
                if (x.x != y.x || x.y != y.y || x.z != y.z || x.w != y.w) {
                  *w = y;
                  here = true;
                }
              }
            }
            dirty |= __any_sync(kFull, here);
            fence_async_shared();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sm.v_fixed[slot]);
          }
        }
        const bool last = it.last;
        if (lane == 0) {
          if (dirty) sm.dirty[taken % kRing] = 1;
          mbar_arrive(&sm.scanned[taken % kRing]);
        }
        release_item(sm, taken, lane);
        ++taken;
        if (last) break;
      }
      if (lane == 0) {
        bool drained = true;
        for (uint32_t t = g > kVSlots ? g - kVSlots : 0; drained && t < g; ++t)
          drained = wait_own(&sm.v_full[t % kVSlots], (t / kVSlots) & 1, p.err);
      }
      __syncwarp();
    } else if (warp >= kQWarp0) {
      // ------------------------------------------------------------ Q into tensor memory
      // thread = TMEM lane: row (lane & 15) of chunk quad + 4 (lane / 16). A negative scale is
      // taken out of the scores here, by the sign of q.
      const int quad = warp & 3, c = quad + 4 * (lane >> 4), r = lane & 15;
      const int i = r / f.hb, group = p.hq / p.hkv;
      uint32_t taken = 0, used = 0;
      while (true) {
        const Item *ip = wait_item(sm, taken, p.err);
        if (!ip) break;
        const int last = ip->last, tiles = ip->tiles, chunk = ip->c0 + c;
        const bool store = quad < ip->chunks;  // (warp-uniform)
        const int node = chunk / f.parts * f.nb + i;
        const int head = (chunk % f.parts) * kChunkRows + r % f.hb;
        const bool row = c < ip->chunks && i < f.nb && node < ip->n && head < group;
        const uint4 *src = reinterpret_cast<const uint4 *>(
            p.q + (int64_t)(ip->q0 + node) * p.q_stride + (ip->h * group + head) * kD);
        release_item(sm, taken, lane);
        ++taken;
        if (last) break;
        if (tiles == 0) continue;
        const int buf = used & 1;
        if (used >= 2 &&
            !__all_sync(kFull, wait_parity(&sm.q_empty[buf], ((used >> 1) - 1) & 1, p.err)))
          break;
        ++used;
        tc_fence_after_sync();
        if (store) {
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            uint32_t w[32];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const uint4 x = row ? ld_once_u4(src + 8 * hf + k) : make_uint4(0, 0, 0, 0);
              w[4 * k] = x.x ^ p.q_sign;
              w[4 * k + 1] = x.y ^ p.q_sign;
              w[4 * k + 2] = x.z ^ p.q_sign;
              w[4 * k + 3] = x.w ^ p.q_sign;
            }
            tmem_st32(tmem + ((uint32_t)(quad * 32) << 16) + kQCol + 64 * buf + 32 * hf, w);
          }
          tmem_st_wait();
        }
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.q_full[buf]);
      }
    } else if (warp == kSWarp || warp == kPvWarp) {
      // ------------------------------------------------------------ UMMA issuers
      // The warp runs its loop converged and one elected lane issues (commits track the issuing
      // thread's UMMAs).
      auto wait_all = [&](uint64_t *bar, uint32_t parity) -> bool {
        return __all_sync(kFull, wait_parity(bar, parity, p.err));
      };
      const bool s_role = warp == kSWarp;
      const uint64_t dk0 = smem_desc_sw128(smem_addr(sm.k[0]), 16, 1024);
      const uint64_t dv0 = smem_desc_sw128(smem_addr(sm.v[0]), kPlane, 1024);
      uint32_t taken = 0, g = 0, used = 0, fix_parity = 0;
      bool ok = true;
      while (ok) {
        const Item *ip = wait_item(sm, taken, p.err);
        if (!ip) break;
        const int last = ip->last, tiles = ip->tiles, key0 = ip->key0, key1 = ip->key1;
        const int root = ip->L - ip->n;
        release_item(sm, taken, lane);
        ++taken;
        if (last) break;
        if (tiles == 0) continue;
        for (int j = 0; j < tiles && ok; ++j, ++g) {
          const uint32_t sb = g & 1;
          const int pos = key0 + j * kTile;
          const int steps = (min(kTile, key1 - pos) + 15) / 16;
          if (s_role) {  // S over as many columns as there are keys, in steps of 16
            const uint32_t ks = g % kKSlots, qb = used & 1;
            ok = wait_all(&sm.k_full[ks], (g / kKSlots) & 1);
            if (ok && j == 0) ok = wait_all(&sm.q_full[qb], (used >> 1) & 1);
            // the buffer's previous P has been read by its PV
            if (ok && g >= 2) ok = wait_all(&sm.o_full[sb], ((g >> 1) - 1) & 1);
            if (!ok) break;
            tc_fence_after_sync();
            if (elect_one()) {
              const uint32_t idesc = idesc_bf16_f32(128, 16 * steps, 0, 0);
              const uint64_t dk = dk0 + ks * (kTileBytes >> 4);
#pragma unroll
              for (int kk = 0; kk < kD / 16; ++kk)
                umma_f16_ts(tmem + kSCol + 128 * sb, tmem + kQCol + 64 * qb + 8 * kk,
                            dk + (((kk >> 2) * kPlane + (kk & 3) * 32) >> 4), idesc, kk > 0);
              umma_commit(&sm.s_full[sb]);
              umma_commit(&sm.k_empty[ks]);
              if (j == tiles - 1) umma_commit(&sm.q_empty[qb]);
            }
          } else {
            const uint32_t vs = g % kVSlots;
            const bool fix = pos + kTile > root;
            ok = wait_all(&sm.p_full[sb], (g >> 1) & 1);
            // the item's first PV overwrites O: the previous item's O must have been read
            if (ok && j == 0 && used > 0) ok = wait_all(&sm.o_free, (used - 1) & 1);
            if (ok) ok = wait_all(&sm.v_full[vs], (g / kVSlots) & 1);
            if (ok && fix) {
              ok = wait_all(&sm.v_fixed[vs], (fix_parity >> vs) & 1);
              fix_parity ^= 1u << vs;
            }
            if (!ok) break;
            tc_fence_after_sync();
            if (elect_one()) {
              constexpr uint32_t kIdesc = idesc_bf16_f32(128, kD, 0, 1);  // V: MN-major
              const uint64_t dv = dv0 + vs * (kTileBytes >> 4);
              const uint32_t pc = tmem + kSCol + 128 * sb;
              for (int kk = 0; kk < steps; ++kk) {
                umma_f16_ts(tmem + kOCol, pc + 8 * kk, dv + ((kk * 16 * 128) >> 4), kIdesc,
                            j > 0 || kk > 0);
                umma_f16_ts(tmem + kOCol, pc + 64 + 8 * kk, dv + ((kk * 16 * 128) >> 4), kIdesc,
                            true);
              }
              umma_commit(&sm.o_full[sb]);
              umma_commit(&sm.v_empty[vs]);
            }
          }
          __syncwarp();
        }
        ++used;
      }
      // every UMMA must be complete before the tensor memory is released, also after an abort
      uint64_t *bar = &sm.drain[s_role ? 0 : 1];
      if (elect_one()) umma_commit(bar);
      __syncwarp();
      __all_sync(kFull, wait_own(bar, 0, p.err));
    } else {
      // ------------------------------------------------------------ softmax warps
      asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
      const int c = warp, ch = lane >> 4, r = lane & 15;  // chunk, column half, row
      const uint32_t lane_addr = tmem + ((uint32_t)((c & 3) * 32 + (c >> 2) * 16) << 16);
      const float2 sl2 = make_float2(p.scale_log2, p.scale_log2);
      const int i = r / f.hb, group = p.hq / p.hkv;
      uint32_t taken = 0, g = 0;
      bool ok = true;
      while (ok) {
        const Item *ip = wait_item(sm, taken, p.err);
        if (!ip) break;
        if (ip->last) {
          release_item(sm, taken, lane);
          break;
        }
        const int tiles = ip->tiles, key0 = ip->key0, key1 = ip->key1, root = ip->L - ip->n;
        const bool mine = c < ip->chunks;  // (warp-uniform)
        const int chunk = ip->c0 + c, node = chunk / f.parts * f.nb + i;
        const int64_t q_row = (int64_t)ip->q0 + node;
        const int head = (chunk % f.parts) * kChunkRows + r % f.hb;
        const bool row = mine && i < f.nb && node < ip->n && head < group;
        if (tiles == 0) {  // nothing to see: zeros
          if (row) {
            uint4 *dst = reinterpret_cast<uint4 *>(
                p.out + (q_row * p.hq + ip->h * group + head) * kD + 64 * ch);
            for (int k = 0; k < 8; ++k) dst[k] = make_uint4(0, 0, 0, 0);
          }
          release_item(sm, taken, lane);
          ++taken;
          continue;
        }
        float m_run = -INFINITY, l_run = 0.f;
        for (int j = 0; j < tiles; ++j, ++g) {
          const uint32_t sb = g & 1, s_col = kSCol + 128 * sb;
          // warp-uniform results: the TMEM loads and stores below are .sync.aligned
          ok = __all_sync(kFull, wait_parity(&sm.s_full[sb], (g >> 1) & 1, p.err));
          if (!ok) break;
          if (mine) {
            tc_fence_after_sync();
            // the keys of this thread's half that the row sees
            const int pos = key0 + j * kTile + 64 * ch;
            uint64_t sees = ~0ull;
            if (pos + 64 > key1) sees = pos >= key1 ? 0 : ~0ull >> (64 - (key1 - pos));
            if (pos + 64 > root && sees != 0) {
              const int base = pos - root, w = base >> 6, sh = base & 63;  // (w = -1 before the root)
              uint64_t bits = w < 0 ? ~0ull : row ? mask_word(p, q_row, node, w) : 0;
              if (sh) {
                const uint64_t up = row ? mask_word(p, q_row, node, w + 1) : 0;
                bits = bits >> sh | up << (64 - sh);
              }
              sees &= bits;
            }
            uint32_t x[2][32];  // keys 64 ch + 32 k + e
#pragma unroll
            for (int k = 0; k < 2; ++k) tmem_ld16x2_32<64>(lane_addr + s_col + 32 * k, x[k]);
#pragma unroll
            for (int k = 0; k < 2; ++k) tmem_ld_wait(x[k]);
            if (sees != ~0ull) {
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const uint32_t bits = (uint32_t)(sees >> 32 * k);
#pragma unroll
                for (int e = 0; e < 32; ++e)
                  if (!(bits >> e & 1)) x[k][e] = __float_as_uint(-INFINITY);
              }
            }
            float mx[2];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              mx[k] = -INFINITY;
#pragma unroll
              for (int e = 0; e < 32; e += 2)
                mx[k] = fmax3(mx[k], __uint_as_float(x[k][e]), __uint_as_float(x[k][e + 1]));
            }
            float m_tile = fmaxf(mx[0], mx[1]);
            m_tile = fmaxf(m_tile, __shfl_xor_sync(kFull, m_tile, 16)) * p.scale_log2;
            const float m_new = fmaxf(m_run, m_tile);
            const bool rescale = m_new > m_run + kRescaleLog2;
            float alpha = 1.f;
            if (rescale) {
              alpha = fast_exp2(m_run - m_new);
              m_run = m_new;
              l_run *= alpha;
            }
            const float neg_m = m_run == -INFINITY ? 0.f : -m_run;
            // O holds the item's tiles before this one: rescale it (never on the first tile)
            if (j > 0 && __any_sync(kFull, rescale)) {
              ok = __all_sync(kFull, wait_parity(&sm.o_full[(g - 1) & 1], ((g - 1) >> 1) & 1, p.err));
              if (!ok) break;
              tc_fence_after_sync();
#pragma unroll 1
              for (int k = 0; k < 2; ++k) {
                uint32_t o[32];
                tmem_ld16x2_32<64>(lane_addr + kOCol + 32 * k, o);
                tmem_ld_wait(o);
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                tmem_st16x2_32<64>(lane_addr + kOCol + 32 * k, o);
              }
            }
            // P = hi + lo, two keys to a column: hi over the first 64 columns of S, lo over the
            // rest (this warp has read all of its rows' S)
            const float2 nm2 = make_float2(neg_m, neg_m);
            float2 rs0 = make_float2(0.f, 0.f), rs1 = make_float2(0.f, 0.f);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t hi[8], lo[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const int at = 16 * (k & 1) + 2 * e;
                const float2 t = ffma2(make_float2(__uint_as_float(x[k >> 1][at]),
                                                   __uint_as_float(x[k >> 1][at + 1])), sl2, nm2);
                const float2 pe = make_float2(fast_exp2(t.x), fast_exp2(t.y));
                if (e & 1) rs1 = fadd2(rs1, pe);
                else rs0 = fadd2(rs0, pe);
                hi[e] = pack_bf16x2(pe.x, pe.y);
                lo[e] = pack_bf16x2(pe.x - bf16_lo(hi[e]), pe.y - bf16_hi(hi[e]));
              }
              tmem_st16x2_8<32>(lane_addr + s_col + 8 * k, hi);
              tmem_st16x2_8<32>(lane_addr + s_col + 64 + 8 * k, lo);
            }
            tmem_st_wait();
            l_run += (rs0.x + rs0.y) + (rs1.x + rs1.y);
            tc_fence_before_sync();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.p_full[sb]);
        }
        if (!ok) break;
        // O, once the last PV is done
        const Item &it = *ip;
        const float l = l_run + __shfl_xor_sync(kFull, l_run, 16);
        if (!__all_sync(kFull, wait_parity(&sm.o_full[(g - 1) & 1], ((g - 1) >> 1) & 1, p.err)))
          break;
        tc_fence_after_sync();
        uint32_t o[2][32];
        if (mine) {
#pragma unroll
          for (int k = 0; k < 2; ++k) tmem_ld16x2_32<64>(lane_addr + kOCol + 32 * k, o[k]);
#pragma unroll
          for (int k = 0; k < 2; ++k) tmem_ld_wait(o[k]);
        }
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.o_free);
        if (!__all_sync(kFull, wait_parity(&sm.scanned[taken % kRing],
                                           (taken / kRing) & 1, p.err)))
          break;
        const bool dirty = sm.dirty[taken % kRing] != 0;
        const float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;  // (NaN stays)
        if (it.to == 2) {
          if (row) {
            uint16_t *dst = p.out + ((int64_t)(it.q0 + node) * p.hq + it.h * group + head) * kD;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint32_t w[8];
#pragma unroll
              for (int e = 0; e < 8; ++e)
                w[e] = pack_bf16x2(__uint_as_float(o[k >> 1][16 * (k & 1) + 2 * e]) * inv,
                                   __uint_as_float(o[k >> 1][16 * (k & 1) + 2 * e + 1]) * inv);
              uint4 *d = reinterpret_cast<uint4 *>(dst + 64 * ch + 16 * k);
              if (f.out_32b) {
                st_global_32b(d, w);
              } else {
                d[0] = make_uint4(w[0], w[1], w[2], w[3]);
                d[1] = make_uint4(w[4], w[5], w[6], w[7]);
              }
            }
            if (dirty)
              not_finite_fix(p, it.b, it.h, it.n, it.L, it.q0 + node, node, dst, 64 * ch, 64);
          }
        } else {
          const int64_t slot = 2 * (int64_t)blockIdx.x + it.to;
          if (row) {
            const int64_t at = slot * f.part_rows + c * kChunkRows + r;
            float *dst = f.part_o + at * kD + 64 * ch;
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              uint32_t w[8];
#pragma unroll
              for (int e = 0; e < 8; ++e)
                w[e] = __float_as_uint(__uint_as_float(o[k >> 2][8 * (k & 3) + e]) * inv);
              st_global_32b(dst + 8 * k, w);
            }
            if (ch == 0) f.part_lse[at] = l > 0.f ? m_run + log2_approx(l) : l == 0.f ? -INFINITY : l;
          }
          if (warp == 0 && lane == 0) f.cuts[blockIdx.x].dirty[it.to] = dirty;
        }
        release_item(sm, taken, lane);
        ++taken;
      }
    }
  }
  // every role is done with its own copies and UMMAs
  __syncwarp();
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  if (warp == kSWarp) tmem_dealloc(tmem, kTmemCols);
}

// Merges the parts of the units that a cut between two workers went through. Block (x, y): the
// unit whose first cut is where CTA x starts, rows [8 y, +8) of its tile, a warp each.
constexpr int kCombineRows = 8;
__global__ void __launch_bounds__(kCombineRows * 32) tree_combine_kernel(const __grid_constant__ FlashParams f) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const TreeParams &p = f.t;
  const CutInfo cut = f.cuts[blockIdx.x];
  if (aborted(p.err) || cut.parts == 0) return;
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.y * kCombineRows + (threadIdx.x >> 5);  // row of the tile
  const int c = t / kChunkRows, r = t % kChunkRows, i = r / f.hb, group = p.hq / p.hkv;
  const int chunk = cut.c0 + c, node = chunk / f.parts * f.nb + i;
  const int head = (chunk % f.parts) * kChunkRows + r % f.hb;
  if (c >= cut.chunks || i >= f.nb || node >= cut.n || head >= group) return;
  // part 0 is the last item of the worker before, the others are their workers' first items
  auto slot = [&](int k) -> int64_t {
    return 2 * ((int64_t)blockIdx.x + (int64_t)(k - 1) * f.group) + (k == 0 ? 1 : 0);
  };
  float m = -INFINITY;
  bool dirty = false;
  for (int k = lane; k < cut.parts; k += 32) {
    m = fmaxf(m, f.part_lse[slot(k) * f.part_rows + t]);
    dirty |= f.cuts[slot(k) >> 1].dirty[slot(k) & 1] != 0;
  }
  dirty = __any_sync(kFull, dirty);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
  const float base = m == -INFINITY ? 0.f : m;
  float sum = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
  for (int k = 0; k < cut.parts; ++k) {
    const int64_t at = slot(k) * f.part_rows + t;
    const float w = fast_exp2(f.part_lse[at] - base);
    const float4 x = *reinterpret_cast<const float4 *>(f.part_o + at * kD + 4 * lane);
    sum += w;
    o[0] += w * x.x;
    o[1] += w * x.y;
    o[2] += w * x.z;
    o[3] += w * x.w;
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  uint16_t *dst = p.out + ((int64_t)(cut.q0 + node) * p.hq + cut.h * group + head) * kD;
  *reinterpret_cast<uint2 *>(dst + 4 * lane) =
      make_uint2(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv));
  if (dirty)
    not_finite_fix(p, cut.b, cut.h, cut.n, cut.L, cut.q0 + node, node, dst, 4 * lane, 4);
}

// How a call's work is cut, from what the host knows.
struct TreePlan {
  int32_t hb, nb, parts;  // heads and nodes of a chunk, chunks that share its nodes
  int32_t group, workers, part_rows;
  size_t part_o, part_lse, bytes;  // of the workspace
};
TreePlan plan_tree(int32_t num_seqs, int32_t max_nodes, int32_t hq, int32_t hkv,
                   int32_t max_context, int num_sms) {
  TreePlan t{};
  const int g = hq / hkv;
  t.hb = std::min(g, kChunkRows);
  t.nb = kChunkRows / t.hb;
  t.parts = (g + kChunkRows - 1) / kChunkRows;
  const int64_t chunks = ((int64_t)max_nodes + t.nb - 1) / t.nb * t.parts;
  const int64_t tiles = std::max<int64_t>(1, (chunks + kChunks - 1) / kChunks);
  t.group = (int32_t)std::min<int64_t>(kMaxGroup, tiles);
  const int64_t units = (int64_t)num_seqs * hkv * ((tiles + t.group - 1) / t.group);
  const int64_t most = units * std::max(1, (int)(((int64_t)max_context + kGranule - 1) / kGranule));
  t.workers = (int32_t)std::max<int64_t>(1, std::min<int64_t>(num_sms / t.group, most));
  t.part_rows = (int32_t)(std::min<int64_t>(kChunks, std::max<int64_t>(1, chunks)) * kChunkRows);
  const size_t ctas = (size_t)t.workers * t.group;
  t.part_o = ctas * sizeof(CutInfo);
  t.part_lse = t.part_o + ctas * 2 * t.part_rows * kD * sizeof(float);
  t.bytes = align16(t.part_lse + ctas * 2 * t.part_rows * sizeof(float));
  return t;
}

cudaError_t launch_flash(const TreeParams &p, const TreePlan &t, void *workspace,
                         cudaStream_t stream) {
  CUtensorMap km, vm;
  const uint64_t dims[3] = {64, (uint64_t)p.num_blocks * p.block_size, (uint64_t)p.hkv * 2};
  const uint64_t strides[2] = {(uint64_t)p.hkv * kD * 2, 128};
  const uint32_t box[3] = {64, kGranule, 1};
  auto encode = [&](CUtensorMap *map, const uint8_t *pool) {
    return encode_tensor_map(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<uint8_t *>(pool),
                             dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B,
                             CU_TENSOR_MAP_L2_PROMOTION_L2_256B) == CUDA_SUCCESS;
  };
  if (!encode(&km, p.k_cache) || !encode(&vm, p.v_cache)) return cudaErrorInvalidValue;
  FlashParams f{};
  f.t = p;
  f.group = t.group;
  f.workers = t.workers;
  f.hb = t.hb;
  f.nb = t.nb;
  f.parts = t.parts;
  f.out_32b = (reinterpret_cast<uintptr_t>(p.out) & 31u) == 0;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  f.cuts = reinterpret_cast<CutInfo *>(ws);
  f.part_o = reinterpret_cast<float *>(ws + t.part_o);
  f.part_lse = reinterpret_cast<float *>(ws + t.part_lse);
  f.part_rows = t.part_rows;
  const size_t smem = sizeof(TreeSmem) + 1024;
  static bool ready[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !ready[dev]) {
    e = cudaFuncSetAttribute(tree_flash_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)smem);
    if (e != cudaSuccess) return e;
    if (dev < 64) ready[dev] = true;
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(t.workers * t.group));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, tree_flash_kernel, km, vm, f);
  if (e != cudaSuccess || t.workers == 1) return e;
  return launch_after(tree_combine_kernel,
                      dim3(cfg.gridDim.x, (unsigned)(t.part_rows / kCombineRows)),
                      kCombineRows * 32, stream, f);
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
  unsigned int *err = current_error_word();
  const int num_sms = current_sm_count();
  if (!err || num_sms <= 0) return PKV_ERR_CUDA;
  const TreePlan plan =
      plan_tree(num_seqs, max_seqlen_q, num_q_heads, num_kv_heads, max_context_len, num_sms);
  if (!workspace || !aligned16(workspace) || workspace_bytes < plan.bytes) return PKV_ERR_WORKSPACE;
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
  prm.num_seqs = num_seqs;
  // (a scale of 0 would turn the -inf of a masked score into NaN)
  prm.scale_log2 = std::min(std::max(fabsf(scale) * kLog2e, 1e-37f), 1e37f);
  prm.q_sign = scale < 0.f ? 0x80008000u : 0u;
  prm.out = static_cast<uint16_t *>(out);
  prm.err = err;
  const dim3 grid((unsigned)units, (unsigned)num_seqs);
  if (fp8) tree_attn_kernel<true><<<grid, kWarps * 32, 0, static_cast<cudaStream_t>(stream)>>>(prm);
  else return launch_flash(prm, plan, workspace, static_cast<cudaStream_t>(stream)) == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
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
  const int num_sms = pkv::current_sm_count();
  if (num_sms <= 0) return 0;
  return pkv::plan_tree(num_seqs, max_seqlen_q, num_q_heads, num_kv_heads, max_context_len, num_sms)
      .bytes;
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

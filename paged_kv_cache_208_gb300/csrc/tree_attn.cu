// tree_attn.cu -- attention of drafted tokens over the paged cache (paged_tree_attn): the last n
// positions of a context are the nodes of a tree, and each attends to the context before them and
// to the nodes that its mask names.
//
// The rows that share a KV head -- (node, query head of the group) pairs -- attend over the same
// keys, so all of them together are the M of a matrix product: K and V are read once for up to
// 128 rows (64 nodes of two heads, 16 of eight). With some tens of rows the tensor cores are through
// with a key long before the next one has been loaded: the kernel is bound by HBM, and its work
// is cut so that every SM reads the same number of keys.
//
// Work. A unit is a sequence's row tile (128 rows of each of `heads` neighbouring KV heads), its
// length the context in granules of 64 keys. All units in a row make one axis of granules, which the
// workers share out evenly, whatever the units' lengths; a worker is a group of CTAs that take the
// heads of a unit (whose values lie in the same DRAM pages) and, where trees have more rows than a
// tile, up to four row tiles of the same keys at the same time (K and V then come from L2 for all
// but one of them). The lengths are device data, so every CTA sums them up at its start (one scan
// over the sequences) and walks its own part. A cut costs an item more, its part of the rows in fp32 and
// the merge: a part's start that lies within 8 granules of a unit's end moves there, and where there
// are no more units than workers and none is much longer than an equal part, a worker takes a whole
// one (us, with and without: 33 x 1250, 31 nodes of 16 / 2 heads 26 and 32, 16 x 1024, 4 nodes of
// 16 / 8 18.4 and 21.5, 8-bit 33 x 100 to 4999 46 and 50; the other way 10 x 4096 37.1 and 35.1, which
// moved starts make uneven). A unit within a worker's part is written out
// directly; what a cut leaves is normalised and goes to the workspace with its log2-sum-exp, and
// tree_combine_kernel merges it. Which parts there are depends on the lengths alone, so the same
// call gives the same bits.
//
// Per tile of 128 keys (M = 128 rows, one CTA):
//   S = Q K^T    Q in tensor memory (the A operand), K rows in shared memory
//   softmax      8 warps, two threads to a row: running maximum and sum in fp32, P = 2^(s - m)
//                written back over S
//   O += P V     P from tensor memory, V rows in shared memory
// S has two buffers, Q two (the next item's is loaded while this one's tiles are in work). O is
// rescaled only when a row's maximum grows by more than 2^8, as in prefill.cu.
//
// What P is rounded to:
//   bf16 cache, a sequence whose rows fit one tile: two bf16 parts, P = hi + lo within 2^-16 of itself.
//                The second product's time is hidden behind the loads (a tile's 64 KiB take an SM about
//                2700 cycles, its products 1536), and the output is that of fp32 weights.
//   bf16 cache, more rows: bf16 (2^-8). The tensor cores are the limit there (the same keys once per
//                tile), and two parts would cost half as much again. This goes by the sequence's own
//                nodes: that others of the call have larger trees costs a small one no precision.
//   8-bit cache: fp16 (2^-11), see below. Two parts would make a long call a quarter longer (16 x 32768,
//                4 nodes 220 -> 267 us, 256 ragged 168 -> 223), for values that e4m3 rounds by 2^-4.
//
// The 8-bit cache. S is a product of e4m3 operands, K as it lies: a row of Q, multiplied by a power of
// two (its largest |q| becomes 128 to 256), enters as two e4m3 parts, which hold a bf16 value
// exactly down to 2^-9 of that largest one and are off by 2^-17 of it at most below. V is widened to
// fp16 in shared memory (an e4m3 code is an fp16 value) and multiplied by P in fp16. (Widening K too
// is bound by shared memory: 192 KiB through it per tile, 1536 cycles, where a tile's loads take
// 1350; this way 144.) The K scale of a key's group and the row's power multiply the scores. The V scale
// is part of P: with v = log2 of it, m runs over s + v, P' = 2^(s + v - m + 6), and l sums
// P' / 2^(v + 6), before it is rounded. A row's largest P' lies between 2^6 and 2^14 (m may lag behind by
// 2^8). fp16 has normal numbers from 2^-14 and steps of 2^-24 below: a P' is off by 2^-11 of itself
// or 2^-25, which is 2^-31 of the largest.
//
// Rows. 16 rows make a chunk: nb = 16 / G nodes with their G query heads (with more than 16 heads
// one node and 16 of them). Chunk c of a tile lies in 16 of the 128 TMEM lanes, in quadrant c % 4, that
// softmax warps c and c + 4 reach: with few rows the softmax is spread over all four SM
// sub-partitions, and the warps take turns, an item each.
//
// Warps (512 threads): 0-7 softmax and epilogue (a chunk each), 8 work walk and K loads, 9 S
// products, 10 V loads, 11 PV products, 12-15 Q into tensor memory, a look through the nodes' V rows,
// and the widening of an 8-bit cache's V. Loads are TMA with 128-byte swizzle, 64 keys to a box (a granule
// never straddles a block). K and V have two slots each: more (3 + 3, 4 + 3) made every bf16 case slower,
// K tiles far ahead taking their turn before V tiles that are needed sooner. K's codes of an 8-bit cache
// have four (16 x 32768, 4 nodes 237 -> 221 us; four of V's codes change nothing).
// TMEM (512 columns): Q [0, 64) [64, 128), S [128, 256) [256, 384), O [384, 512).
//
// Measured (us; the bytes of K, V, q and out at 6.8 TB/s in brackets):
//   bf16, 2 heads to a KV head, 8 KV heads: 8 x 1024, chains of 4    15.7 (5.0)
//         256 sequences of 100 to 2048, trees of 5 to 8 nodes       193 (178)
//   bf16, 3 to a KV head, 4 of them: 1 x 17188, 13 nodes             17.6 (5.2)
//   bf16, 4 to a KV head, 8 of them: 16 x 32768, 4 nodes 308 (316), 32 nodes 333 (317); 16 x 30000 to
//         32768, 48 to 64 nodes, two row tiles, 428, 475 where calls follow one another for long and the
//         power limit lowers the clock (303; their exponentials 232, their products 232)
//   8-bit, 2 to a KV head, 8 of them: 8 x 1024, 16 nodes             15.7 (2.5)
//         256 sequences of 100 to 2048, trees of 5 to 8 nodes       168 (89)
//   8-bit, 8 to a KV head, 2 of them: 33 x 100 to 4999               46.6 (7.5)
//   8-bit, 4 to a KV head, 8 of them: 16 x 32768, 4 nodes 220 (158), 32 nodes 267, 64 nodes 510
// The CTAs of a worker are as many as the call's largest tree asks for (max_seqlen_q): those that a
// smaller one has no rows for wait. The same 256 sequences, 8 to 64 nodes allowed / up to 128 / 192 / more:
// bf16 193 / 301 / 435 / 567, 8-bit 168 / 325 / 475 / 619; with one tree of two tiles among them (32 / 8
// heads, 64 nodes) 198 -> 305 and 173 -> 328.
// A call of a few keys takes 7 us (the launch, the scan, the chain of loads). Long bf16 contexts
// go at the memory's rate. What bounds the rest is the chain of a tile's steps (S, softmax, P V, the
// hand-over of a buffer between two warps four times): about 1 us a tile and two of them under
// way; leaving out the widening, the exponentials or three quarters of the products one at a
// time takes 3 % off a long 8-bit call, all of them together 15 %. An item more costs 3 to 5 us where
// it has one tile (152 x 64 keys: a row of q takes a trip to memory; with more than four chunks the
// softmax warps wait for the last product before they write). And code: the warps run some twelve
// different loops side by side, and each KiB more in them has cost about 2 % of a call, in whichever
// warp it was; that is why waits are a function, loops are not unrolled and nothing is written twice.
//
// Masked places. A key that a row does not see is left out of its maximum and gets P = 0; V rows
// past the context are zeroed in shared memory. A node that others do not see may hold
// infinities or NaNs, and 0 x NaN would reach them: the nodes' V rows are looked through, what is
// not finite becomes zero there, and the rows that do see such a node are put right in memory. So are
// rows of which infinities of the context have made NaN (not_finite_fix, parts_fix).
#include <math.h>

#include <algorithm>
#include <type_traits>

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

constexpr int kTile = 128;    // keys
constexpr int kGranule = 64;  // keys of a TMA box, and what the work is measured in
static_assert(kGranule == kFp8Group, "a granule has one scale");
constexpr int kChunkRows = 16;
constexpr int kChunks = 8;    // of a row tile
constexpr int kSoftmaxWarps = 8;
constexpr int kKWarp = 8, kSWarp = 9, kVWarp = 10, kPvWarp = 11, kQWarp0 = 12;
constexpr int kThreads = 16 * 32;
constexpr int kSlots = 2;     // of K and of V
constexpr int kRawSlots = 2;  // of V's codes, 8-bit cache
constexpr int kKSlots8 = 4;   // of K's codes
constexpr uint32_t kTileBytes = kTile * kD * 2;
constexpr uint32_t kPlane = kTileBytes / 2;         // 64 dims of the tile's keys, 128-byte rows
constexpr uint32_t kGranuleBytes = kGranule * 128;  // of a plane, or of an 8-bit pool
constexpr uint32_t kRawBytes = kTile * kD;
constexpr int kScaleTiles = 8;  // a tile's scales stay until its softmax: six tiles at most
constexpr int kRing = 4;
constexpr uint32_t kQCol = 0, kSCol = 128, kOCol = 384, kTmemCols = 512;
constexpr int kItemConsumers = kSoftmaxWarps + 3 + 4;  // S, V, PV and Q warps
constexpr int kMaxGroup = 8, kMaxTiles = 4;  // CTAs, and row tiles, of a worker
constexpr int kNear = 8;        // granules that a part may grow or shrink by at an end
constexpr int kOffset8 = 6;     // log2 of what P' is larger by, 8-bit cache

enum Mode { kBf16, kFp8 };

// A worker's share of a unit.
struct Item {
  int32_t last;        // 1: no more work
  int32_t b, h;
  int32_t q0, n, L;    // the sequence's rows of q, its nodes and its context (0: an empty one)
  int32_t c0, chunks;  // the row tile's first chunk, and its chunks
  int32_t key0, key1;  // positions
  int32_t tiles;
  int32_t to;          // 0, 1: a partial result, into this slot of the CTA's; 2: the output
  int32_t two;         // bf16 cache: P in two parts
  int32_t pad[3];
};
static_assert(sizeof(Item) == 64, "");

// What tree_combine_kernel has to know of a unit's row tile that is cut.
struct CutInfo {
  int32_t parts;       // 0: not cut
  int32_t worker;      // that has the unit's start
  int32_t b, h, q0, n, L, c0, chunks;
  int32_t pad[7];
};
static_assert(sizeof(CutInfo) == 64, "");

struct RawSmem {  // 8-bit cache
  uint8_t v[kRawSlots][kRawBytes];
  alignas(16) float scale[kScaleTiles][2][2][4];  // [tile][granule][K, V]: four groups' around it
  float q_power[kRing][kChunks * kChunkRows];     // log2 of what the rows of q were divided by
  uint64_t v_full[kRawSlots], v_empty[kRawSlots];
};
struct NoRaw {};

template <Mode M>
struct TreeSmem {
  static constexpr int kKSlots = M == kFp8 ? kKSlots8 : kSlots;
  static constexpr uint32_t kKBytes = M == kFp8 ? kRawBytes : kTileBytes;
  uint8_t k[kKSlots][kKBytes];  // 1024-byte aligned (128-byte swizzle atoms)
  uint8_t v[kSlots][kTileBytes];
  std::conditional_t<M == kFp8, RawSmem, NoRaw> raw;
  Item items[kRing];
  int32_t dirty[kRing];            // of the item in this ring slot
  uint64_t k_full[kKSlots], k_empty[kKSlots], v_full[kSlots], v_empty[kSlots];
  // bf16: a V tile that holds nodes has landed; they have been looked through, rows past the
  // context zeroed
  uint64_t v_ready[kSlots], v_fixed[kSlots];
  uint64_t q_full[2], q_empty[2];
  uint64_t s_full[2], p_full[2], o_full[2], o_free, drain[2];
  uint64_t item_full[kRing], item_empty[kRing];
  uint64_t scanned[kRing];         // `dirty` is known
  uint64_t past[kRing];            // the item's last S has been waited for
  uint32_t tmem_base;
  int32_t stop;
  int3 warp_sums[kThreads / 32];  // granules, units, the longest unit
  // the sequence that the CTA's part starts in, and where that starts on the axis
  int32_t start_b, start_at, start_units, start_q0, start_n, start_L;
  int32_t x0, x1;  // the part
};
static_assert(sizeof(TreeSmem<kFp8>) + 1024 <= 232448, "fits the SM");

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
  int32_t hq, hkv, group_heads, block_size;  // group_heads: query heads of a KV head
  int64_t num_blocks;
  int32_t num_seqs;
  float scale_log2;  // of the scale's magnitude
  uint32_t q_sign;   // flips the signs of two bf16 where the scale is negative
  uint16_t *out;
  bool out_32b;
  unsigned int *err;
  // how the work is cut
  int32_t workers, group;        // workers, and the CTAs of one: `heads` KV heads of `at_once` tiles
  int32_t heads, at_once;
  int32_t per_tile;              // hkv / heads: units that share a row tile
  int32_t hb, nb, parts;         // heads and nodes of a chunk; chunks that share its nodes
  uint32_t nb_magic, hb_magic;   // x / nb is the high word of x * nb_magic, for x < 2^24
  // cuts: one for each unit and CTA of a worker (by_unit: there are no more units than workers), or
  // one for each CTA, the unit that its part ends in.
  bool by_unit;
  int32_t max_units;
  CutInfo *cuts;
  float *part_o, *part_lse;      // [CTA][2][part_rows][kD], [CTA][2][part_rows]
  int32_t part_rows, row_warps, block_warps;  // of tree_combine_kernel: warps for a row, of a block
  int32_t whole;  // granules that a unit may be longer than a part without being cut

  __device__ __forceinline__ int chunks_of(int n) const {
    return nb == 1 ? n * parts : (int)__umulhi(n + nb - 1, nb_magic);  // (nb > 1: one part)
  }
  // the first node and head (of the group) of a chunk
  __device__ __forceinline__ int first_node(int chunk) const {
    return nb > 1 ? chunk * nb : parts == 1 ? chunk : chunk / parts;
  }
  __device__ __forceinline__ int first_head(int chunk) const {
    return parts == 1 ? 0 : chunk % parts * kChunkRows;
  }
  // row r of a chunk: its node, from the chunk's first one
  __device__ __forceinline__ int node_of(int r) const {
    return hb == 1 ? r : (int)__umulhi(r, hb_magic);
  }
  // The axis in `workers` parts, the first `rest` of them one granule longer.
  __device__ __forceinline__ static int32_t part_start(int w, int32_t each, int32_t rest) {
    return w * each + min(w, rest);
  }
  __device__ __forceinline__ static int32_t part_of(int32_t x, int32_t each, int32_t rest) {
    const int32_t longer = rest * (each + 1);
    return x < longer ? x / (each + 1) : rest + (x - longer) / each;
  }
  // A part's start at x in the unit [start, end) moves to an end of the unit that is near.
  __device__ __forceinline__ static int32_t nearness(int32_t each) {
    return min(kNear, max(0, (each - 1) / 2));
  }
  __device__ __forceinline__ static int32_t moved(int32_t x, int32_t start, int32_t end,
                                                  int32_t near) {
    return x - start <= near ? start : end - x <= near ? end : x;
  }
};

// Rows of a sequence as the work is counted: its nodes (0: none, or a bad cu_seqlens) and its
// context (0 also for a bad length, whose rows become zeros).
struct Seq {
  int32_t q0, n, L;
  int32_t units, length;  // what its workers have to do, and the granules of each
  __device__ __forceinline__ int32_t cost() const { return units * length; }
  __device__ __forceinline__ void set(const TreeParams &p, int32_t first, int32_t nodes,
                                      int32_t context) {
    q0 = first;
    n = nodes;
    L = context;
    const int tiles = (p.chunks_of(n) + kChunks - 1) / kChunks;
    units = p.per_tile * (p.at_once == 1 ? tiles : (tiles + p.at_once - 1) / p.at_once);
    length = max(1, (L + kGranule - 1) / kGranule);
  }
};
__device__ __forceinline__ Seq sequence(const TreeParams &p, int b, bool record) {
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
  s.set(p, (int32_t)c0, (int32_t)n, ok ? (int32_t)L : 0);
  return s;
}

// Bit j - 64 w of the result: node `node` (row `row` of q) sees node j, for 64 w <= j < 64 (w + 1).
__device__ __forceinline__ uint64_t mask_word(const TreeParams &p, int64_t row, int node, int w) {
  if (p.mask) return w < p.mask_words ? p.mask[row * p.mask_words + w] : 0;
  const int top = node - 64 * w;
  return top < 0 ? 0 : top >= 63 ? ~0ull : (2ull << top) - 1;
}

// Values of V that are not finite. Those of nodes were left out of the products: what a row sees of
// them is added to its result. Infinities of the context were not, but the products may have made NaN
// of them (a weight enters as a sum whose second term is often zero or negative, and one below fp32's
// range as zero), where an infinity is right as long as there is no NaN and none of the other sign:
// with `again` a NaN is replaced by what the context's values that are not finite add up to.
// A warp for a chunk of an item, lane r has row r's `to` (bf16, or fp32 of a part) and whether it is to be
// put right (`sound`: a row whose normaliser is not is NaN already). Four dims to a lane, eight rows of V in
// flight: a granule takes 5 us, or 80 with 64 infinite nodes, and the CTA's other warps wait for 2 s.
template <Mode M>
__device__ __noinline__ void not_finite_fix(const TreeParams &p, int b, int h, int32_t root, int32_t key0,
                                            int32_t key1, bool again, bool sound, int64_t q_row,
                                            int node, void *to, bool part) {
  const int lane = threadIdx.x & 31;
  const int32_t *const table = p.block_tables + (int64_t)b * p.table_width;
  constexpr int kBytes = M == kFp8 ? 1 : 2, kLoads = 8;
  using Word = std::conditional_t<M == kFp8, uint32_t, uint2>;  // four values
  auto odd = [](Word x, float (&f)[4]) {  // zeros for finite ones
    if constexpr (M == kFp8) {
      const float2 lo = f16x2_to_f32(cvt_f16x2_e4m3x2(x)), hi = f16x2_to_f32(cvt_f16x2_e4m3x2_hi(x));
      f[0] = lo.x, f[1] = lo.y, f[2] = hi.x, f[3] = hi.y;
    } else {
      f[0] = bf16_lo(x.x), f[1] = bf16_hi(x.x), f[2] = bf16_lo(x.y), f[3] = bf16_hi(x.y);
    }
#pragma unroll
    for (int d = 0; d < 4; ++d)
      if (isfinite(f[d])) f[d] = 0.f;
  };
  auto add = [&](int r, const float (&sum)[4], bool replace) {  // to row r's results
    const uint64_t at = __shfl_sync(kFull, reinterpret_cast<uint64_t>(to), r);
    if (!__shfl_sync(kFull, sound, r)) return;
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      if (sum[d] == 0.f) continue;
      float *const x32 = reinterpret_cast<float *>(at) + 4 * lane + d;
      uint16_t *const x16 = reinterpret_cast<uint16_t *>(at) + 4 * lane + d;
      const float x = part ? *x32 : __uint_as_float((uint32_t)*x16 << 16);
      const float y = replace && isnan(x) ? sum[d] : x + sum[d];
      if (part) *x32 = y;
      else *x16 = bf16_bits_rn(y);
    }
  };
  __syncwarp();  // the results have been written
  float all[4] = {0.f, 0.f, 0.f, 0.f};  // of the context
#pragma unroll 1
  for (int32_t pos = again ? key0 : max(key0, root & ~(kGranule - 1)); pos < key1; pos += kGranule) {
    const int count = min(kGranule, key1 - pos), nodes_at = root - pos;
    const int32_t i = pos / p.block_size, blk = table[i];
    const bool any = blk >= 0 && blk < p.num_blocks;
    const int64_t row = (int64_t)blk * p.block_size + (pos - i * p.block_size);
    const int64_t stride = (int64_t)p.hkv * (kD * kBytes);
    const uint8_t *const src = p.v_cache + row * stride + (h * kD + 4 * lane) * kBytes;
    uint64_t bad = 0;
#pragma unroll 1
    for (int j = 0; any && j < count; j += kLoads) {
      Word x[kLoads];
#pragma unroll
      for (int u = 0; u < kLoads; ++u)
        x[u] = j + u < count ? *reinterpret_cast<const Word *>(src + (j + u) * stride) : Word{};
#pragma unroll
      for (int u = 0; u < kLoads; ++u) {
        float f[4];
        odd(x[u], f);
        if (j + u < nodes_at) {
#pragma unroll
          for (int d = 0; d < 4; ++d) all[d] += f[d];
        } else if (!(f[0] == 0.f && f[1] == 0.f && f[2] == 0.f && f[3] == 0.f)) {
          bad |= 1ull << (j + u);
        }
      }
    }
    // (the granule that the item's part of the context ends in)
    if (again && pos < root && pos + kGranule >= min(root, key1))
#pragma unroll 1
      for (int r = 0; r < kChunkRows; ++r) add(r, all, true);
    bad = (uint64_t)__reduce_or_sync(kFull, (uint32_t)(bad >> 32)) << 32 |
          __reduce_or_sync(kFull, (uint32_t)bad);
    if (bad == 0) continue;
    const int w = -nodes_at >> 6, sh = -nodes_at & 63;  // (w = -1: positions before the tree)
#pragma unroll 1
    for (int r = 0; r < kChunkRows; ++r) {
      const int64_t at = __shfl_sync(kFull, q_row, r);
      const int i_node = __shfl_sync(kFull, node, r);
      if (!__shfl_sync(kFull, sound, r)) continue;
      uint64_t bits = w < 0 ? 0 : mask_word(p, at, i_node, w);
      if (sh) bits = bits >> sh | mask_word(p, at, i_node, w + 1) << (64 - sh);
      bits &= bad;
      float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
      while (bits) {
        Word x[kLoads];
#pragma unroll
        for (int u = 0; u < kLoads; ++u) {
          x[u] = bits ? *reinterpret_cast<const Word *>(src + (__ffsll(bits) - 1) * stride) : Word{};
          bits &= bits - 1;
        }
#pragma unroll
        for (int u = 0; u < kLoads; ++u) {
          float f[4];
          odd(x[u], f);
#pragma unroll
          for (int d = 0; d < 4; ++d) sum[d] += f[d];
        }
      }
      add(r, sum, false);
    }
  }
  __syncwarp();
}

// Walks a worker's part of the axis, one item at a time (one thread).
struct Walk {
  int32_t x, x1, at;  // where the walk is, where the part ends, where sequence b starts
  int32_t units_at;   // units before sequence b
  int b;
  Seq s;
  // unit: the item's unit, start: where that starts
  __device__ __forceinline__ bool next(const TreeParams &p, int head, int row_tile, Item &it,
                                       int32_t &unit, int32_t &start) {
    if (x < x1) {
      while (x >= at + s.cost()) {
        at += s.cost();
        units_at += s.units;
        s = sequence(p, ++b, false);
      }
      const int32_t rel = x - at;
      const int32_t u = s.units == 1 ? 0 : rel / s.length;
      const int32_t off = rel - u * s.length;
      const int32_t take = min(s.length - off, x1 - x);
      unit = units_at + u;
      start = x - off;
      x += take;
      const int tile = u < p.per_tile ? 0 : u / p.per_tile;
      it.last = 0;
      it.b = b;
      it.h = (u - tile * p.per_tile) * p.heads + head;
      it.q0 = s.q0;
      it.n = s.n;
      it.L = s.L;
      it.c0 = (tile * p.at_once + row_tile) * kChunks;
      it.chunks = min(kChunks, p.chunks_of(s.n) - it.c0);
      it.two = p.chunks_of(s.n) <= kChunks;
      it.key0 = min(s.L, off * kGranule);
      it.key1 = (int32_t)min((int64_t)s.L, (int64_t)(off + take) * kGranule);
      it.tiles = (it.key1 - it.key0 + kTile - 1) / kTile;
      it.to = off > 0 ? 0 : take < s.length ? 1 : 2;
      return true;
    }
    return false;
  }
};

// First pool rows of an item's granules, one after the other; a bad block id is flagged and gives a
// row wholly outside the pool (TMA fills zeros). A block's id is read once.
struct Rows {
  const int32_t *next_id;
  int32_t blk, in_block;
  __device__ __forceinline__ void read(const TreeParams &p) {
    blk = ld_global_s32(next_id++);
    if (blk < 0 || blk >= p.num_blocks) {
      record_error(p.err, PKV_DEVERR_BLOCK_RANGE);
      blk = -1;
    }
  }
  __device__ __forceinline__ void start(const TreeParams &p, int b, int32_t pos) {
    const int32_t i = pos / p.block_size;
    next_id = p.block_tables + (int64_t)b * p.table_width + i;
    in_block = pos - i * p.block_size;
    read(p);
  }
  __device__ __forceinline__ int32_t next(const TreeParams &p) {
    if (in_block == p.block_size) {
      in_block = 0;
      read(p);
    }
    const int32_t row = blk < 0 ? -2 * kTile : blk * p.block_size + in_block;
    in_block += kGranule;
    return row;
  }
};

// Raise the phase's expected transaction bytes without arriving.
__device__ __forceinline__ void mbar_expect_tx(uint64_t *bar, uint32_t bytes) {
  asm volatile("mbarrier.expect_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_addr(bar)),
               "r"(bytes)
               : "memory");
}

// mbar_arrive for `count` arrivals at once.
__device__ __forceinline__ void mbar_arrive_count(uint64_t *bar, uint32_t count) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(smem_addr(bar)), "r"(count)
               : "memory");
}

// ld_once_u4 for data that are read again.
__device__ __forceinline__ uint4 ld_u4(const uint4 *p) {
  uint4 r;
  asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p)
               : "memory");
  return r;
}

// wait_parity in fewer instructions (this kernel has some thirty waits, and its warps run code of their
// own side by side: what does not fit the instruction caches costs more than the waits): the clock
// and the abort bit are looked at once in 256 polls, each of which waits for some time itself.
__device__ __noinline__ bool wait_longer(uint32_t bar, uint32_t parity, unsigned int *err) {
  uint64_t since = 0;
  for (uint32_t n = 1;; ++n) {
    uint32_t done;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done)
        : "r"(bar), "r"(parity)
        : "memory");
    if (done) return true;
    if (n & 255) continue;
    if (aborted(err)) return false;
    const uint64_t now = global_timer_ns();
    if (since == 0) since = now;
    if (now - since > kWaitLimitNs) {
      record_error(err, kErrTimeout);
      return false;
    }
  }
}
__device__ __forceinline__ bool wait_bar(uint64_t *bar, uint32_t parity, unsigned int *err) {
  return mbar_try_wait(bar, parity) || wait_longer(smem_addr(bar), parity, err);
}

template <class Smem>
__device__ __forceinline__ const Item *wait_item(Smem &sm, uint32_t taken, unsigned int *err) {
  const int slot = taken % kRing;
  return __all_sync(kFull, wait_bar(&sm.item_full[slot], (taken / kRing) & 1, err))
             ? &sm.items[slot]
             : nullptr;
}
template <class Smem>
__device__ __forceinline__ void release_item(Smem &sm, uint32_t taken, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(&sm.item_empty[taken % kRing]);
}

// Sixteen e4m3 codes as fp16, in two 16-byte pieces.
__device__ __forceinline__ void widen16(const uint4 x, uint4 &lo, uint4 &hi) {
  lo = make_uint4(cvt_f16x2_e4m3x2(x.x), cvt_f16x2_e4m3x2_hi(x.x), cvt_f16x2_e4m3x2(x.y),
                  cvt_f16x2_e4m3x2_hi(x.y));
  hi = make_uint4(cvt_f16x2_e4m3x2(x.z), cvt_f16x2_e4m3x2_hi(x.z), cvt_f16x2_e4m3x2(x.w),
                  cvt_f16x2_e4m3x2_hi(x.w));
}
// four codes with NaNs replaced by zero
__device__ __forceinline__ uint32_t no_nan4(uint32_t w) {
  return w & ~__vcmpeq4(w & 0x7f7f7f7fu, 0x7f7f7f7fu);
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

template <Mode M>
__global__ void __launch_bounds__(kThreads, 1)
    tree_flash_kernel(const __grid_constant__ CUtensorMap kmap,
                      const __grid_constant__ CUtensorMap vmap,
                      const __grid_constant__ TreeParams p) {
  constexpr bool F8 = M == kFp8;
  constexpr int kKSlots = TreeSmem<M>::kKSlots;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  extern __shared__ uint8_t smem_raw[];
  TreeSmem<M> &sm = *reinterpret_cast<TreeSmem<M> *>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  if (tid == 0) {
    for (int i = 0; i < kKSlots; ++i) {
      mbar_init(&sm.k_full[i], 1);
      mbar_init(&sm.k_empty[i], 1);
    }
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&sm.v_full[i], F8 ? 4 : 1);  // (8-bit: four warps widen a tile)
      mbar_init(&sm.v_empty[i], 1);
      mbar_init(&sm.v_ready[i], 1);
      mbar_init(&sm.v_fixed[i], 4);
    }
    if constexpr (F8)
      for (int i = 0; i < kRawSlots; ++i) {
        mbar_init(&sm.raw.v_full[i], 1);
        mbar_init(&sm.raw.v_empty[i], 4);
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
      mbar_init(&sm.scanned[i], 4);
      mbar_init(&sm.past[i], 1);
    }
    fence_mbar_init();
    prefetch_tensormap(&kmap);
    prefetch_tensormap(&vmap);
  }
  if (warp == kSWarp) {
    tmem_alloc(&sm.tmem_base, kTmemCols);
    tmem_relinquish();
  }
  const int worker = blockIdx.x / p.group, rank = blockIdx.x - worker * p.group;
  const int rank_tile = p.at_once == 1 ? 0 : rank / p.heads;
  const int rank_head = rank - rank_tile * p.heads;
  // everything above may overlap the stream's previous kernel
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // The axis: every sequence's granules, summed over the batch. Up to 32 sequences are one to a
  // lane, and each warp scans them by itself; else one to a thread, kThreads at a time. The
  // sequence that the worker's part starts in is found on the way when the batch is scanned at
  // once, else by a second pass.
  const bool stop = tid == 0 && aborted(p.err);
  const bool one_warp = p.num_seqs <= 32, at_once = p.num_seqs <= kThreads;
  bool works = false;
  bool whole = false;  // there are no more units than workers, and a worker takes one
  int32_t total = 0, each = 0, rest = 0, x0 = 0, x1 = 0, all_units = 0, longest = 0;
  for (int pass = 0; pass < 2; ++pass) {
    int32_t carry = 0, units_carry = 0;
    for (int base = 0; base < p.num_seqs; base += kThreads) {
      const int b = base + (one_warp ? lane : tid);
      Seq own{};
      if (b < p.num_seqs) own = sequence(p, b, blockIdx.x == 0 && (!one_warp || warp == 0));
      const int32_t mine = own.cost();
      // (what has no unit has no cost)
      int32_t x = mine, units = own.units;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int32_t y = __shfl_up_sync(kFull, x, o), z = __shfl_up_sync(kFull, units, o);
        if (lane >= o) {
          x += y;
          units += z;
        }
      }
      int32_t sum = __shfl_sync(kFull, x, 31), units_sum = __shfl_sync(kFull, units, 31);
      int32_t most = __reduce_max_sync(kFull, own.length);
      if (!one_warp) {
        __syncthreads();
        if (lane == 31) sm.warp_sums[warp] = make_int3(x, units, most);
        __syncthreads();
        const int3 v = lane < kThreads / 32 ? sm.warp_sums[lane] : make_int3(0, 0, 0);
        x += __reduce_add_sync(kFull, lane < warp ? v.x : 0);
        units += __reduce_add_sync(kFull, lane < warp ? v.y : 0);
        sum = __reduce_add_sync(kFull, v.x);
        units_sum = __reduce_add_sync(kFull, v.y);
        most = __reduce_max_sync(kFull, v.z);
      }
      const int32_t prefix = carry + x - mine, units_at = units_carry + units - own.units;
      carry += sum;
      units_carry += units_sum;
      longest = max(longest, most);
      if (pass == 0 && base + kThreads >= p.num_seqs) {  // the axis' length is known
        total = carry;
        all_units = units_carry;
        const int32_t workers = min(p.workers, total);
        each = total > 0 ? total / workers : 0;
        rest = total - each * workers;
        whole = all_units <= workers && longest <= each + p.whole;
        works = worker < (whole ? all_units : workers);
        x0 = works && !whole ? TreeParams::part_start(worker, each, rest) : 0;
        x1 = works && !whole ? TreeParams::part_start(worker + 1, each, rest) : 0;
      }
      // (batches scanned at once: by the warp that needs it, or by all)
      if ((pass == 0 && !at_once) || (one_warp && warp != kKWarp)) continue;
      const auto within = [&](int32_t y) {
        return whole ? units_at <= worker && worker < units_at + own.units
                     : mine > 0 && prefix <= y && y < prefix + mine;
      };
      const auto move = [&](int32_t y) {
        if (whole) return prefix + (worker - units_at) * own.length;
        const int32_t start = prefix + (y - prefix) / own.length * own.length;
        return TreeParams::moved(y, start, start + own.length, TreeParams::nearness(each));
      };
      if (works && within(x1)) sm.x1 = move(x1) + (whole ? own.length : 0);
      if (within(x0)) {
        sm.x0 = move(x0);
        sm.start_b = b;
        sm.start_at = prefix;
        sm.start_units = units_at;
        sm.start_q0 = own.q0;
        sm.start_n = own.n;
        sm.start_L = own.L;
      }
    }
    if (at_once) break;
  }
  if (tid == 0) sm.stop = stop;
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = sm.tmem_base;
  // the kernel that follows may be set up (not before this CTA has its tensor memory)
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (!sm.stop) {
    if (warp == kKWarp) {
      // ------------------------------------------------------------ work walk and K loads
      if (lane == 0) {
        const uint64_t policy = policy_evict_first();
        if (works) {
          x0 = sm.x0;
          if (x1 < total) x1 = sm.x1;
        }
        Walk w{x0, x1, sm.start_at, sm.start_units, sm.start_b, {}};
        if (works) w.s.set(p, sm.start_q0, sm.start_n, sm.start_L);
        uint32_t pushed = 0, g = 0;
        bool ok = true;
        bool told = false;
        if (p.by_unit)  // no unit there
          for (int u = all_units * p.group + blockIdx.x; u < p.max_units * p.group; u += gridDim.x)
            p.cuts[u].parts = 0;
        // An item is handed out while the one before it is loaded, after that one's second tile
        // (the walk starts with an item of no tiles in hand).
        Item it{}, nx{};
        Rows rows;
        while (ok && !it.last) {
          if (it.tiles > 0) rows.start(p, it.b, it.key0);
          const int steps = max(1, it.tiles), push_at = min(1, steps - 1);
          for (int j = 0; j < steps && ok; ++j) {
            if (j < it.tiles) {
              const int slot = g % kKSlots;
              uint64_t *const full = &sm.k_full[slot];
              ok = g < kKSlots ||
                   wait_bar(&sm.k_empty[slot], ((g / kKSlots) - 1) & 1, p.err);
              if (!ok) break;  // (g counts the copies that were issued)
              const int32_t pos = it.key0 + j * kTile;
              const int granules = it.key1 - pos > kGranule ? 2 : 1;
              if constexpr (!F8) mbar_arrive_expect_tx(full, granules * 2 * kGranuleBytes);
              for (int r = 0; r < granules; ++r) {
                const int32_t row = rows.next(p);
                if constexpr (F8) {
                  // with the granule's scales of K and V and those of three groups beside it (16
                  // bytes); the zeros of a bad block have a scale of 1
                  float(*dst)[4] = sm.raw.scale[g % kScaleTiles][r];
                  const uint32_t bytes = row < 0 ? kGranuleBytes : kGranuleBytes + 32;
                  if (row < 0)
                    for (int e = 0; e < 8; ++e) dst[e >> 2][e & 3] = 1.f;
                  if (r + 1 < granules) mbar_expect_tx(full, bytes);
                  else mbar_arrive_expect_tx(full, bytes);
                  tma_load_3d(sm.k[slot] + r * kGranuleBytes, &kmap, full, 0, row, it.h, policy);
                  if (row >= 0) {
                    const int64_t at =
                        ((int64_t)rows.blk * p.hkv + it.h) * (p.block_size / kFp8Group) +
                        ((rows.in_block - kGranule) / kGranule & ~3);
                    bulk_copy_g2s(dst[0], p.k_scale + at, 16, full);
                    bulk_copy_g2s(dst[1], p.v_scale + at, 16, full);
                  }
                } else {
#pragma unroll
                  for (int hf = 0; hf < 2; ++hf)
                    tma_load_3d(sm.k[slot] + hf * kPlane + r * kGranuleBytes, &kmap, full, 0, row,
                                2 * it.h + hf, policy);
                }
              }
              ++g;
            }
            if (j == push_at) {
              bool more;
              do {
                int32_t unit, start;
                more = w.next(p, rank_head, rank_tile, nx, unit, start);
                // the CTA with a unit's start says whether it is cut (one without rows: not)
                const bool cut = more && nx.to == 1 && nx.chunks > 0;
                if (more ? cut || (p.by_unit && nx.to != 0) : !p.by_unit && !told) {
                  int4 *dst = reinterpret_cast<int4 *>(
                      p.cuts + (p.by_unit ? unit * p.group + rank : (int)blockIdx.x));
                  int parts = 0;
                  if (cut) {  // up to the last worker with a start in the unit, unless that has moved out
                    const int32_t end = start + w.s.length;
                    const int past = TreeParams::part_of(end - 1, each, rest);
                    parts = past - worker + 1;
                    if (TreeParams::moved(TreeParams::part_start(past, each, rest), start, end,
                                          TreeParams::nearness(each)) == end)
                      --parts;
                  }
                  dst[0] = make_int4(parts, worker, nx.b, nx.h);
                  dst[1] = make_int4(nx.q0, nx.n, nx.L, nx.c0);
                  dst[2] = make_int4(nx.chunks, 0, 0, 0);
                  told = true;
                }
              } while (more && nx.chunks <= 0);  // (this CTA's row tile of a smaller tree is empty)
              if (!more) {
                nx = Item{};
                nx.last = 1;
              }
              const int slot = pushed % kRing;
              ok = pushed < kRing ||
                   wait_bar(&sm.item_empty[slot], ((pushed / kRing) - 1) & 1, p.err);
              if (!ok) break;
              sm.items[slot] = nx;
              sm.dirty[slot] = 0;
              mbar_arrive(&sm.item_full[slot]);
              ++pushed;
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
      if (lane == 0) {
        const uint64_t policy = policy_evict_first();
        constexpr uint32_t kN = F8 ? kRawSlots : kSlots;
        uint32_t taken = 0, g = 0;
        bool ok = true;
        Rows rows;
        while (ok) {
          const int ring = taken % kRing;
          if (!wait_bar(&sm.item_full[ring], (taken / kRing) & 1, p.err)) break;
          const Item it = sm.items[ring];
          mbar_arrive(&sm.item_empty[ring]);
          ++taken;
          if (it.last) break;
          if (it.tiles > 0) rows.start(p, it.b, it.key0);
          for (int j = 0; j < it.tiles; ++j, ++g) {
            const int slot = g % kN;
            uint64_t *full, *empty;
            if constexpr (F8) full = &sm.raw.v_full[slot], empty = &sm.raw.v_empty[slot];
            else full = &sm.v_full[slot], empty = &sm.v_empty[slot];
            ok = g < kN || wait_bar(empty, ((g / kN) - 1) & 1, p.err);
            if (!ok) break;
            const int32_t pos = it.key0 + j * kTile;
            const int granules = it.key1 - pos > kGranule ? 2 : 1;
            mbar_arrive_expect_tx(full, granules * (F8 ? kGranuleBytes : 2 * kGranuleBytes));
            for (int r = 0; r < granules; ++r) {
              const int32_t row = rows.next(p);
              if constexpr (F8) {
                tma_load_3d(sm.raw.v[slot] + r * kGranuleBytes, &vmap, full, 0, row, it.h, policy);
              } else {
#pragma unroll
                for (int hf = 0; hf < 2; ++hf)
                  tma_load_3d(sm.v[slot] + hf * kPlane + r * kGranuleBytes, &vmap, full, 0, row,
                              2 * it.h + hf, policy);
              }
            }
          }
        }
        bool drained = true;
        for (uint32_t t = g > kN ? g - kN : 0; drained && t < g; ++t) {
          if constexpr (F8) drained = wait_own(&sm.raw.v_full[t % kN], (t / kN) & 1, p.err);
          else drained = wait_own(&sm.v_full[t % kN], (t / kN) & 1, p.err);
        }
      }
      __syncwarp();
    } else if (warp >= kQWarp0) {
      // ------------------------------------------------------------ Q; V looked through; codes
      // For Q thread = TMEM lane: row (lane & 15) of chunk quad + 4 (lane / 16). A negative scale is
      // taken out of the scores by the sign of q.
      const int quad = warp & 3, c = quad + 4 * (lane >> 4), r = lane & 15;
      const int i = p.node_of(r), head_r = r - i * p.hb;
      const uint32_t lane_addr = tmem + ((uint32_t)(quad * 32) << 16);
      uint32_t used = 0, g = 0, fix_parity = 0;
      // Q of item k. `last`: there is none.
      auto load_q = [&](int k, bool &last) -> bool {
        const Item *ip = wait_item(sm, k, p.err);
        if (!ip) return false;
        last = ip->last;
        if (last || ip->tiles == 0) return true;
        const int chunk = ip->c0 + c;
        const int node = p.first_node(chunk) + i, head = p.first_head(chunk) + head_r;
        const bool row = c < ip->chunks && i < p.nb && node < ip->n && head < p.group_heads;
        const uint4 *src = reinterpret_cast<const uint4 *>(
            p.q + (int64_t)(ip->q0 + node) * p.q_stride + (ip->h * p.group_heads + head) * kD);
        const int buf = used & 1;
        if (used >= 2 &&
            !__all_sync(kFull, wait_bar(&sm.q_empty[buf], ((used >> 1) - 1) & 1, p.err)))
          return false;
        ++used;
        tc_fence_after_sync();
        if (quad < ip->chunks) {  // (warp-uniform)
          if constexpr (F8) {
            uint32_t top = 0;  // (the row's loads all at once; the second time they come from L1)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const uint4 x = row ? ld_u4(src + e) : make_uint4(0, 0, 0, 0);
              top = __vmaxu2(top, __vmaxu2(bf16x2_absmax(x.x, x.y), bf16x2_absmax(x.z, x.w)));
            }
            top = max(top & 0xffffu, top >> 16);
            // what takes the largest |q| to 2^7; a row with infinities or NaNs becomes NaN
            const int e7 = min(max((int)(top >> 7) - 134, -120), 120);
            const float mul = pow2f(-e7);
            const uint32_t bad = top >= 0x7f80u ? 0x7f7f7f7fu : 0u;
            sm.raw.q_power[k % kRing][c * kChunkRows + r] = (float)e7;
#pragma unroll 1
            for (int q4 = 0; q4 < 4; ++q4) {  // 32 dims: 8 columns of each part
              uint32_t hi[8], lo[8];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const uint4 x = row ? ld_u4(src + 4 * q4 + e) : make_uint4(0, 0, 0, 0);
                const uint32_t w[4] = {x.x ^ p.q_sign, x.y ^ p.q_sign, x.z ^ p.q_sign, x.w ^ p.q_sign};
#pragma unroll
                for (int z = 0; z < 2; ++z) {
                  const float f[4] = {bf16_lo(w[2 * z]) * mul, bf16_hi(w[2 * z]) * mul,
                                      bf16_lo(w[2 * z + 1]) * mul, bf16_hi(w[2 * z + 1]) * mul};
                  const uint32_t a = cvt_e4m3x2(f[0], f[1]), b = cvt_e4m3x2(f[2], f[3]);
                  const float2 fa = f16x2_to_f32(cvt_f16x2_e4m3x2(a)), fb = f16x2_to_f32(cvt_f16x2_e4m3x2(b));
                  hi[2 * e + z] = a | b << 16 | bad;
                  lo[2 * e + z] = cvt_e4m3x2(f[0] - fa.x, f[1] - fa.y) |
                                  cvt_e4m3x2(f[2] - fb.x, f[3] - fb.y) << 16;
                }
              }
              tmem_st_cols(lane_addr + kQCol + 64 * buf + 8 * q4, hi);
              tmem_st_cols(lane_addr + kQCol + 64 * buf + 32 + 8 * q4, lo);
            }
          } else {
#pragma unroll 1
            for (int hf = 0; hf < 2; ++hf) {
              uint32_t w[32];
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const uint4 x = row ? ld_once_u4(src + 8 * hf + e) : make_uint4(0, 0, 0, 0);
                w[4 * e] = x.x ^ p.q_sign;
                w[4 * e + 1] = x.y ^ p.q_sign;
                w[4 * e + 2] = x.z ^ p.q_sign;
                w[4 * e + 3] = x.w ^ p.q_sign;
              }
              tmem_st32(lane_addr + kQCol + 64 * buf + 32 * hf, w);
            }
          }
          tmem_st_wait();
        }
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.q_full[buf]);
        return true;
      };
      // (Item -1 has no tiles, it only brings the first Q.)
      bool last = false, ok = true;
      for (int k = -1; ok && !last; ++k) {
        const Item &it = sm.items[(k + kRing) % kRing];
        const int tiles = k < 0 ? 0 : it.tiles, key0 = it.key0, key1 = it.key1, root = it.L - it.n;
        bool found = false;
        // 8-bit cache: each warp widens 32 rows of every V tile; the next item's Q before the last
        // one, it is needed right after. Else the next item's Q, then the tiles that hold nodes
        // (one that ends inside a step of 16 keys among them) are looked through: the PV warp says
        // when such a tile has landed, it waits for all of them in turn.
        const int from = F8 || tiles == 0 ? 0 : max(0, (root - key0) / kTile);
        const int q_at = F8 ? max(0, tiles - 1) : from;
        for (int j = from; j < max(from + 1, tiles) && ok; ++j) {
          if (j == q_at) ok = load_q(k + 1, last);
          if (j >= tiles || !ok) break;
          const int pos = key0 + j * kTile, keys = min(kTile, key1 - pos);
          const bool nodes = pos + kTile > root;
          if (!F8 && !nodes) continue;
          const uint32_t at = g + j, slot = at % kSlots;
          uint8_t *tile;  // this warp's 32 rows of it
          if constexpr (F8) {
            tile = sm.raw.v[at % kRawSlots] + 32 * quad * 128;
            ok = __all_sync(kFull, wait_bar(&sm.raw.v_full[at % kRawSlots], (at / kRawSlots) & 1, p.err));
            if (ok && at >= kSlots)
              ok = __all_sync(kFull, wait_bar(&sm.v_empty[slot], ((at / kSlots) - 1) & 1, p.err));
          } else {
            tile = sm.v[slot] + 32 * quad * 128;
            ok = __all_sync(kFull, wait_bar(&sm.v_ready[slot], (fix_parity >> slot) & 1, p.err));
            fix_parity ^= 1u << slot;
          }
          if (!ok) break;
          const int up = min(32, ((keys + 15) & ~15) - 32 * quad);  // rows that are multiplied
          if (nodes) {
            // 16 bytes at a time: rows past the keys zeroed, what is not finite in nodes' rows too
            const int first = max(0, root - pos - 32 * quad);  // the first node's row
#pragma unroll 1
            for (int h = 0; h < (F8 ? 1 : 2); ++h) {
#pragma unroll 1
              for (int e = lane + first * 8; e < up * 8; e += 32) {
                uint4 *w = reinterpret_cast<uint4 *>(tile + h * kPlane + e * 16);
                uint4 x = make_uint4(0, 0, 0, 0);
                if (32 * quad + (e >> 3) < keys) {
                  x = *w;
                  const uint4 y = F8 ? make_uint4(no_nan4(x.x), no_nan4(x.y), no_nan4(x.z), no_nan4(x.w))
                                     : make_uint4(bf16x2_finite(x.x), bf16x2_finite(x.y),
                                                  bf16x2_finite(x.z), bf16x2_finite(x.w));
                  if (((x.x ^ y.x) | (x.y ^ y.y) | (x.z ^ y.z) | (x.w ^ y.w)) == 0) continue;
                  x = y;
                  found = true;
                }
                *w = x;
              }
            }
            __syncwarp();
          }
          if constexpr (F8) {
            // 16 rows x 8 pieces of 16 codes, four pieces of a lane in flight; rows next to one
            // another in a quarter warp, so that neither side has bank conflicts
            uint8_t *const dst = sm.v[slot] + 32 * quad * 128;
            const int low = lane & 7, a0 = lane >> 3;
#pragma unroll 1
            for (int e = 0; e < up; e += 16) {
              uint4 x[4];  // rows e + low and e + 8 + low, pieces a0 and a0 + 4
#pragma unroll
              for (int u = 0; u < 4; ++u)
                x[u] = *reinterpret_cast<const uint4 *>(tile + (e + 8 * (u >> 1) + low) * 128 +
                                                        (((a0 + 4 * (u & 1)) ^ low) << 4));
#pragma unroll
              for (int u = 0; u < 4; ++u) {
                uint4 lo, hi;
                widen16(x[u], lo, hi);
                uint8_t *const to = dst + (u & 1) * kPlane + (e + 8 * (u >> 1) + low) * 128;
                *reinterpret_cast<uint4 *>(to + (((2 * a0) ^ low) << 4)) = lo;
                *reinterpret_cast<uint4 *>(to + (((2 * a0 + 1) ^ low) << 4)) = hi;
              }
            }
          }
          fence_async_shared();
          __syncwarp();
          if (lane == 0) {
            if constexpr (F8) {
              mbar_arrive(&sm.v_full[slot]);
              mbar_arrive(&sm.raw.v_empty[at % kRawSlots]);
            } else {
              mbar_arrive(&sm.v_fixed[slot]);
            }
          }
        }
        if (k < 0 || !ok) continue;
        g += tiles;
        if (__any_sync(kFull, found) && lane == 0) sm.dirty[k % kRing] = 1;
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.scanned[k % kRing]);
        release_item(sm, k, lane);
      }
    } else if (warp == kSWarp || warp == kPvWarp) {
      // ------------------------------------------------------------ UMMA issuers
      // The warp runs its loop converged and one elected lane issues (commits track the issuing
      // thread's UMMAs).
      auto wait_all = [&](uint64_t *bar, uint32_t parity) -> bool {
        return __all_sync(kFull, wait_bar(bar, parity, p.err));
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
        [[maybe_unused]] const bool two = ip->two;
        release_item(sm, taken, lane);
        ++taken;
        if (last) break;
        if (tiles == 0) continue;
        for (int j = 0; j < tiles && ok; ++j, ++g) {
          const uint32_t sb = g & 1, slot = g % (s_role ? kKSlots : kSlots);
          const int pos = key0 + j * kTile;
          const int steps = (min(kTile, key1 - pos) + 15) / 16;
          if (s_role) {  // S over as many columns as there are keys, in steps of 16
            const uint32_t qb = used & 1;
            ok = wait_all(&sm.k_full[slot], (g / kKSlots) & 1);
            if (ok && j == 0) ok = wait_all(&sm.q_full[qb], (used >> 1) & 1);
            // the buffer's previous P has been read by its PV
            if (ok && g >= 2) ok = wait_all(&sm.o_full[sb], ((g >> 1) - 1) & 1);
            if (!ok) break;
            tc_fence_after_sync();
            if (elect_one()) {
              const uint64_t dk = dk0 + slot * (TreeSmem<M>::kKBytes >> 4);
              const uint32_t sc = tmem + kSCol + 128 * sb, qc = tmem + kQCol + 64 * qb;
              if constexpr (F8) {
                const uint32_t idesc = idesc_e4m3_f32(128, 16 * steps, 0, 0);
#pragma unroll
                for (int kk = 0; kk < 2 * (kD / 32); ++kk)  // 32 dims of a part of Q
                  umma_e4m3_ts(sc, qc + 8 * kk, dk + ((kk & 3) * 32 >> 4), idesc, kk > 0);
              } else {
                const uint32_t idesc = idesc_bf16_f32(128, 16 * steps, 0, 0);
#pragma unroll
                for (int kk = 0; kk < kD / 16; ++kk)
                  umma_f16_ts(sc, qc + 8 * kk, dk + (((kk >> 2) * kPlane + (kk & 3) * 32) >> 4),
                              idesc, kk > 0);
              }
              umma_commit(&sm.s_full[sb]);
              umma_commit(&sm.k_empty[slot]);
              if (j == tiles - 1) umma_commit(&sm.q_empty[qb]);
            }
          } else {
            const bool nodes = !F8 && pos + kTile > root;
            ok = wait_all(&sm.v_full[slot], (g / kSlots) & 1);
            if (ok && nodes && lane == 0) mbar_arrive(&sm.v_ready[slot]);
            if (ok) ok = wait_all(&sm.p_full[sb], (g >> 1) & 1);
            // the item's first PV overwrites O: the previous item's O must have been read
            if (ok && j == 0 && used > 0) ok = wait_all(&sm.o_free, (used - 1) & 1);
            if (ok && nodes) {
              ok = wait_all(&sm.v_fixed[slot], (fix_parity >> slot) & 1);
              fix_parity ^= 1u << slot;
            }
            if (!ok) break;
            tc_fence_after_sync();
            if (elect_one()) {
              constexpr uint32_t kIdesc =  // V: MN-major
                  F8 ? idesc_f16_f32(128, kD, 0, 1) : idesc_bf16_f32(128, kD, 0, 1);
              const uint64_t dv = dv0 + slot * (kTileBytes >> 4);
              const uint32_t p0 = tmem + kSCol + 128 * sb;  // a granule's P over its own S columns
              auto step = [&](int kk) {
                const uint32_t pc = p0 + 64 * (kk >> 2) + 8 * (kk & 3);
                umma_f16_ts(tmem + kOCol, pc, dv + ((kk * 16 * 128) >> 4), kIdesc,
                            j > 0 || kk > 0);
                if constexpr (!F8)
                  if (two) umma_f16_ts(tmem + kOCol, pc + 32, dv + ((kk * 16 * 128) >> 4), kIdesc, true);
              };
              // (in a loop an issue takes 67 cycles, about as long as the product)
              if (steps == kTile / 16) {
#pragma unroll
                for (int kk = 0; kk < kTile / 16; ++kk) step(kk);
              } else {
#pragma unroll 1
                for (int kk = 0; kk < steps; ++kk) step(kk);
              }
              umma_commit(&sm.o_full[sb]);
              umma_commit(&sm.v_empty[slot]);
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
      // ------------------------------------------------------------ softmax and epilogue
      // A warp goes through a tile a granule at a time, 32 of its keys to a thread. The loops over
      // granules stay loops: unrolled, a tile's code does not fit the instruction caches beside the
      // other warps'. (Two warps to a chunk where there are few, a granule or a tile each in turn:
      // slower for the same reason, and by what they have to agree on.)
      const int ch = lane >> 4, r = lane & 15;  // half of the granule's keys, row
      const int i = p.node_of(r), head_r = r - i * p.hb;
      uint32_t taken = 0, g = 0;
      bool ok = true;
      while (ok) {
        const Item *ip = wait_item(sm, taken, p.err);
        if (!ip || ip->last) break;
        const int ring = taken % kRing;
        const int tiles = ip->tiles, key0 = ip->key0, key1 = ip->key1, n = ip->n, root = ip->L - n;
        // The chunk: warps c and c + 4 reach the lanes of chunks c and c + 4. They change places from item
        // to item, so that with up to four chunks one half writes an item out while the other is at
        // the next one.
        const int c = (warp + 4 * (taken & 1)) & 7;
        const uint32_t lane_addr = tmem + ((uint32_t)((c & 3) * 32 + (c >> 2) * 16) << 16);
        const bool mine = c < ip->chunks;  // (warp-uniform)
        [[maybe_unused]] const bool two = ip->two;
        const int chunk = ip->c0 + c, node = p.first_node(chunk) + i;
        const int head = p.first_head(chunk) + head_r;
        const int64_t q_row = (int64_t)ip->q0 + node;
        const bool row = mine && i < p.nb && node < n && head < p.group_heads;
        uint16_t *const dst = p.out + (q_row * p.hq + ip->h * p.group_heads + head) * kD;
        if (tiles == 0) {  // nothing to see: zeros
          if (row)
            for (int e = 0; e < 8; ++e)
              reinterpret_cast<uint4 *>(dst + 64 * ch)[e] = make_uint4(0, 0, 0, 0);
        } else if (!mine) {
          // The first chunk's warp arrives for it. (Its next wait for an S is not before the one
          // before that is over: a wait knows two phases of a barrier.)
          g += tiles;
          ok = __all_sync(kFull, wait_bar(&sm.past[ring], (taken / kRing) & 1, p.err));
          if (!ok) break;
        }
        if (tiles == 0 || !mine) {
          if (tiles == 0 && c == 0 && lane == 0) mbar_arrive(&sm.past[ring]);
          release_item(sm, taken, lane);
          ++taken;
          continue;
        }
        const uint32_t arrivals = c == 0 ? kSoftmaxWarps + 1 - ip->chunks : 1;
        // what the row sees of its tree's first 64 nodes, loaded ahead of the tiles that need it
        const uint64_t first_word = row && key1 > root ? mask_word(p, q_row, node, 0) : 0;
        auto word = [&](int w) -> uint64_t {
          return w == 0 ? first_word : row && 64 * w < n ? mask_word(p, q_row, node, w) : 0;
        };
        float m_run = -INFINITY, l_run = 0.f, row_scale = p.scale_log2;
        for (int j = 0; j < tiles; ++j, ++g) {
          const uint32_t sb = g & 1, s_addr = lane_addr + kSCol + 128 * sb;
          // warp-uniform results: the TMEM loads and stores below are .sync.aligned
          ok = __all_sync(kFull, wait_bar(&sm.s_full[sb], (g >> 1) & 1, p.err));
          if (!ok) break;
          if (j == tiles - 1 && c == 0 && lane == 0) mbar_arrive(&sm.past[ring]);
          tc_fence_after_sync();
          if constexpr (F8)
            if (j == 0)
              row_scale = p.scale_log2 * pow2f((int)sm.raw.q_power[ring][c * kChunkRows + r]);
          // 8-bit cache: what multiplies the scores of granule k, log2 of its V scale (a granule past
          // the keys has no scales)
          auto factors = [&](int k, float &factor, float &v_scale) {
            factor = row_scale;
            v_scale = 1.f;
            if constexpr (F8) {
              const int pos = key0 + j * kTile + 64 * k;
              if (pos < key1) {
                const float(*sc)[4] = sm.raw.scale[g % kScaleTiles][k];
                factor *= sc[0][pos / kGranule & 3];
                v_scale = sc[1][pos / kGranule & 3];
              }
              // (a row of zeros has a power of 2^-120; see scale_log2)
              factor = fmaxf(factor, 1e-38f);
            }
          };
          float m_tile = -INFINITY;
#pragma unroll 1
          for (int k = 0; k < 2; ++k) {
            uint32_t x[32];  // keys 64 k + 32 ch + e
            tmem_ld16x2_32<32>(s_addr + 64 * k, x);
            const int pos = key0 + j * kTile + 64 * k + 32 * ch;
            float factor, v_scale;
            factors(k, factor, v_scale);
            tmem_ld_wait(x);
            if (key0 + j * kTile + 64 * (k + 1) > min(key1, root)) {
              // the keys of this thread's that the row sees; the others' scores become -inf
              uint32_t sees = pos >= key1 ? 0 : pos + 32 > key1 ? ~0u >> (32 - (key1 - pos)) : ~0u;
              if (pos + 32 > root && sees != 0) {
                const int base = pos - root, w = base >> 6, sh = base & 63;  // (w = -1: before it)
                uint64_t bits = w < 0 ? ~0ull : word(w);
                if (sh) bits = bits >> sh | word(w + 1) << (64 - sh);
                sees &= (uint32_t)bits;
              }
#pragma unroll
              for (int e = 0; e < 32; ++e)
                if (!(sees >> e & 1)) x[e] = __float_as_uint(-INFINITY);
              tmem_st16x2_32<32>(s_addr + 64 * k, x);
              tmem_st_wait();
            }
            float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              mx[0] = fmax3(mx[0], __uint_as_float(x[e]), __uint_as_float(x[e + 1]));
              mx[1] = fmax3(mx[1], __uint_as_float(x[e + 2]), __uint_as_float(x[e + 3]));
            }
            float m = fmaxf(mx[0], mx[1]) * factor;
            if constexpr (F8) m += log2_approx(v_scale);
            m_tile = fmaxf(m_tile, m);
          }
          m_tile = fmaxf(m_tile, __shfl_xor_sync(kFull, m_tile, 16));
          const bool grows = m_tile > m_run + kRescaleLog2;
          if (__any_sync(kFull, grows)) {
            const float alpha = grows ? fast_exp2(m_run - m_tile) : 1.f;
            if (grows) m_run = m_tile;
            l_run *= alpha;
            // O holds the item's tiles before this one: rescale it (never on the first tile)
            if (j > 0) {
              ok = __all_sync(kFull, wait_bar(&sm.o_full[(g - 1) & 1], ((g - 1) >> 1) & 1, p.err));
              if (!ok) break;
              tc_fence_after_sync();
#pragma unroll 1
              for (int k = 0; k < 2; ++k) {
                uint32_t o[32];
                tmem_ld16x2_32<32>(lane_addr + kOCol + 64 * k, o);
                tmem_ld_wait(o);
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
                tmem_st16x2_32<32>(lane_addr + kOCol + 64 * k, o);
              }
            }
          }
          // P, two keys to a column, over the first half of the granule's S columns; a second part
          // over the other half
          const float base = m_run == -INFINITY ? 0.f : m_run;
#pragma unroll 1
          for (int k = 0; k < 2; ++k) {
            uint32_t x[32];
            tmem_ld16x2_32<32>(s_addr + 64 * k, x);
            float factor, v_scale;
            factors(k, factor, v_scale);
            float offset = -base, per_v = 1.f;
            if constexpr (F8) {
              offset += log2_approx(v_scale) + kOffset8;
              per_v = rcp_approx(v_scale * (1 << kOffset8));
            }
            const float2 mul2 = make_float2(factor, factor), add2 = make_float2(offset, offset);
            float2 rs0 = make_float2(0.f, 0.f), rs1 = make_float2(0.f, 0.f);
            tmem_ld_wait(x);
            uint32_t hi[16];
            [[maybe_unused]] uint32_t lo[16];  // (bf16 cache: the second part, used or not)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float2 t = ffma2(
                  make_float2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])), mul2, add2);
              const float2 pe = make_float2(fast_exp2(t.x), fast_exp2(t.y));
              if (e & 1) rs1 = fadd2(rs1, pe);
              else rs0 = fadd2(rs0, pe);
              if constexpr (F8) {
                hi[e] = pack_f16x2(pe.x, pe.y);
              } else {
                hi[e] = pack_bf16x2(pe.x, pe.y);
                x[2 * e] = __float_as_uint(pe.x);
                x[2 * e + 1] = __float_as_uint(pe.y);
              }
            }
            tmem_st16x2_16<16>(s_addr + 64 * k, hi);
            if constexpr (!F8)
              if (two) {
#pragma unroll
                for (int e = 0; e < 16; ++e)
                  lo[e] = pack_bf16x2(__uint_as_float(x[2 * e]) - bf16_lo(hi[e]),
                                      __uint_as_float(x[2 * e + 1]) - bf16_hi(hi[e]));
                tmem_st16x2_16<16>(s_addr + 64 * k + 32, lo);
              }
            l_run += ((rs0.x + rs0.y) + (rs1.x + rs1.y)) * per_v;
          }
          tmem_st_wait();
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive_count(&sm.p_full[sb], arrivals);
        }
        if (!ok) break;
        // O, once the last PV is done
        const float l = l_run + __shfl_xor_sync(kFull, l_run, 16);
        ok = __all_sync(kFull, wait_bar(&sm.o_full[(g - 1) & 1], ((g - 1) >> 1) & 1, p.err) &&
                                   wait_bar(&sm.scanned[ring], (taken / kRing) & 1, p.err));
        if (!ok) break;
        const Item &it = *ip;
        const bool dirty = sm.dirty[ring] != 0;
        // (NaN stays; a row that sees nothing gets zeros)
        float inv = l > 0.f ? 1.f / l : l == 0.f ? 0.f : l;
        if constexpr (F8) inv *= 1.f / (1 << kOffset8);
        const int64_t slot = 2 * (int64_t)blockIdx.x + it.to;
        const int64_t at = slot * p.part_rows + c * kChunkRows + r;
        [[maybe_unused]] float2 odd = make_float2(0.f, 0.f);  // NaN: O is not finite somewhere
        tc_fence_after_sync();
#pragma unroll 1
        for (int k = 0; k < 2; ++k) {
          uint32_t o[32];  // dims 64 k + 32 ch + e
          tmem_ld16x2_32<32>(lane_addr + kOCol + 64 * k, o);
          tmem_ld_wait(o);
          if (k == 1) {
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive_count(&sm.o_free, arrivals);
          }
          if (!row) continue;
          if constexpr (!F8) {
            const float2 zero = make_float2(0.f, 0.f);
#pragma unroll
            for (int e = 0; e < 32; e += 2)
              odd = ffma2(make_float2(__uint_as_float(o[e]), __uint_as_float(o[e + 1])), zero, odd);
          }
          if (it.to == 2) {
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              uint32_t w[8];
#pragma unroll
              for (int e = 0; e < 8; ++e)
                w[e] = pack_bf16x2(__uint_as_float(o[16 * z + 2 * e]) * inv,
                                   __uint_as_float(o[16 * z + 2 * e + 1]) * inv);
              uint4 *d = reinterpret_cast<uint4 *>(dst + 64 * k + 32 * ch + 16 * z);
              if (p.out_32b) {
                st_global_32b(d, w);
              } else {
                d[0] = make_uint4(w[0], w[1], w[2], w[3]);
                d[1] = make_uint4(w[4], w[5], w[6], w[7]);
              }
            }
          } else {
#pragma unroll
            for (int z = 0; z < 4; ++z) {
              uint32_t w[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) w[e] = __float_as_uint(__uint_as_float(o[8 * z + e]) * inv);
              st_global_32b(p.part_o + at * kD + 64 * k + 32 * ch + 8 * z, w);
            }
          }
        }
        const bool sound = l > 0.f && l < INFINITY;  // (the same in both lanes of a row)
        // (an 8-bit cache has NaNs only, which the context's products spread themselves)
        const bool again = !F8 && __any_sync(kFull, sound && !(odd.x + odd.y == 0.f));
        if (dirty || again)
          not_finite_fix<M>(p, it.b, it.h, root, key0, key1, again, row && sound, q_row, node,
                            it.to == 2 ? static_cast<void *>(dst) : p.part_o + at * kD, it.to != 2);
        if (it.to < 2) {
          if (row && ch == 0)
            p.part_lse[at] = l > 0.f ? m_run + log2_approx(l) : l == 0.f ? -INFINITY : l;
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

// Merges the parts of the units that a cut between two workers went through. Block (x, y): cut x, from
// the y-th on every gridDim.y-th p.block_warps / p.row_warps rows of its tile. A row's warps take its
// parts in turn, four in flight, each with a running maximum; what they have is merged in shared
// memory. The time is that of dependent loads (the cut, then all parts at once) and of blocks that
// find no cut: there are as many cuts as units, or workers where that is fewer. It takes 2 to 4 us of
// a call; where no unit can be cut (no more units than workers, contexts up to 512 to 1536) it is not
// launched (33 x 512, 31 nodes of 16 / 2 heads: 19.5 -> 14.5 us).
constexpr int kCombineWarps = 8, kInFlight = 4;  // warps of a block: at most
// Where a part holds an infinity and its weight is below fp32's range, the product is NaN: the dims of
// `odd` (a bit each) become what the parts' values that are not finite add up to. slots: of part 0, and
// of part k, k step further.
__device__ __noinline__ void parts_fix(const TreeParams &p, int parts, int64_t slot0, int64_t slot1,
                                       int step, int t, uint32_t odd, uint16_t *out) {
#pragma unroll 1
  for (int d = 0; d < 4; ++d) {
    if (!(odd >> d & 1)) continue;
    float sum = 0.f;
#pragma unroll 1
    for (int k = 0; k < parts; ++k) {
      const int64_t slot = k == 0 ? slot0 : slot1 + (int64_t)(k - 1) * step;
      const float x = p.part_o[(slot * p.part_rows + t) * kD + d + 4 * (threadIdx.x & 31)];
      if (!isfinite(x)) sum += x;
    }
    out[d] = bf16_bits_rn(sum);
  }
}
template <Mode M>
__global__ void __launch_bounds__(kCombineWarps * 32)
    tree_combine_kernel(const __grid_constant__ TreeParams p) {
  __shared__ float4 outs[kCombineWarps][32];
  __shared__ float2 stats[kCombineWarps];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const CutInfo cut = p.cuts[blockIdx.x];
  if (aborted(p.err) || cut.parts == 0) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row_in = warp / p.row_warps, sub = warp - row_in * p.row_warps;
  // part 0 is its worker's last item, the others are their workers' first ones
  const int rank = blockIdx.x % p.group;
  auto slot = [&](int k) -> int64_t {
    return 2 * ((int64_t)(cut.worker + k) * p.group + rank) + (k == 0 ? 1 : 0);
  };
  // (with several warps to a row there are as many blocks as it takes)
  for (int y = blockIdx.y; y < p.part_rows * p.row_warps / p.block_warps; y += gridDim.y) {
    const int t = y * (p.block_warps / p.row_warps) + row_in;  // row of the tile
    const int c = t / kChunkRows, r = t % kChunkRows, i = p.node_of(r);
    const int chunk = cut.c0 + c, node = p.first_node(chunk) + i;
    const int head = p.first_head(chunk) + r - i * p.hb;
    const bool row = c < cut.chunks && i < p.nb && node < cut.n && head < p.group_heads;
    float m = -INFINITY, sum = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
    if (row) {
#pragma unroll 1
      for (int k0 = sub; k0 < cut.parts; k0 += kInFlight * p.row_warps) {
        float lse[kInFlight];
        float4 x[kInFlight];
#pragma unroll
        for (int u = 0; u < kInFlight; ++u) {
          const int k = k0 + u * p.row_warps;
          lse[u] = -INFINITY;
          x[u] = make_float4(0.f, 0.f, 0.f, 0.f);
          if (k < cut.parts) {
            const int64_t at = slot(k) * p.part_rows + t;
            lse[u] = p.part_lse[at];
            x[u] = *reinterpret_cast<const float4 *>(p.part_o + at * kD + 4 * lane);
          }
        }
        float top = m;
#pragma unroll
        for (int u = 0; u < kInFlight; ++u) top = fmaxf(top, lse[u]);
        const float base = top == -INFINITY ? 0.f : top, old = fast_exp2(m - base);
        m = top;
        sum *= old;
#pragma unroll
        for (int d = 0; d < 4; ++d) o[d] *= old;
#pragma unroll
        for (int u = 0; u < kInFlight; ++u) {
          const float w = fast_exp2(lse[u] - base);  // (NaN stays)
          sum += w;
          o[0] += w * x[u].x;
          o[1] += w * x[u].y;
          o[2] += w * x[u].z;
          o[3] += w * x[u].w;
        }
      }
    }
    if (p.row_warps > 1) {
      outs[warp][lane] = make_float4(o[0], o[1], o[2], o[3]);
      if (lane == 0) stats[warp] = make_float2(m, sum);
      __syncthreads();
      if (sub != 0) continue;
      float top = m;
      for (int k = 1; k < p.row_warps; ++k) top = fmaxf(top, stats[warp + k].x);
      const float base = top == -INFINITY ? 0.f : top;
      sum = 0.f;
      o[0] = o[1] = o[2] = o[3] = 0.f;
      for (int k = 0; k < p.row_warps; ++k) {
        const float2 st = stats[warp + k];
        const float4 x = outs[warp + k][lane];
        const float w = fast_exp2(st.x - base);
        sum += w * st.y;
        o[0] += w * x.x;
        o[1] += w * x.y;
        o[2] += w * x.z;
        o[3] += w * x.w;
      }
    }
    if (!row) continue;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    uint16_t *dst = p.out + ((int64_t)(cut.q0 + node) * p.hq + cut.h * p.group_heads + head) * kD;
    *reinterpret_cast<uint2 *>(dst + 4 * lane) =
        make_uint2(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv));
    uint32_t odd = 0;
#pragma unroll
    for (int d = 0; d < 4; ++d) odd |= (uint32_t)isnan(o[d]) << d;
    if (odd && !isnan(sum))
      parts_fix(p, cut.parts, slot(0), slot(1), 2 * p.group, t, odd, dst + 4 * lane);
  }
}

// How a call's work is cut, from what the host knows.
struct TreePlan {
  int32_t hb, nb, parts;  // heads and nodes of a chunk, chunks that share its nodes
  int32_t workers, group, heads, at_once, part_rows, row_warps, block_warps;
  int64_t longest, units;  // bounds of the axis and of the units
  bool by_unit, uncut;     // uncut: whatever the lengths are, no unit is cut
  int32_t whole;             // see TreeParams
  int32_t cuts, cut_blocks;  // and blocks to merge one
  size_t part_o, part_lse, bytes;  // of the workspace
};
// x * y, or 2^40 where that is less (no product of sizes overflows)
int64_t times(int64_t x, int64_t y) {
  return (int64_t)std::min<__int128>((__int128)x * y, (__int128)1 << 40);
}
TreePlan plan_tree(int32_t num_seqs, int32_t max_nodes, int32_t hq, int32_t hkv,
                   int32_t max_context, int num_sms) {
  TreePlan t{};
  const int g = hq / hkv;
  t.hb = std::min(g, kChunkRows);
  t.nb = kChunkRows / t.hb;
  t.parts = (g + kChunkRows - 1) / kChunkRows;
  const int64_t chunks = ((int64_t)max_nodes + t.nb - 1) / t.nb * t.parts;
  const int64_t tiles = std::max<int64_t>(1, (chunks + kChunks - 1) / kChunks);
  t.at_once = (int)std::min<int64_t>(kMaxTiles, tiles);
  t.heads = 1;
  while (t.heads * 2 * t.at_once <= kMaxGroup && hkv % (t.heads * 2) == 0) t.heads *= 2;
  t.group = t.heads * t.at_once;
  const int64_t rounds = (tiles + t.at_once - 1) / t.at_once;
  const int64_t units = t.units = times(times(num_seqs, hkv / t.heads), rounds);
  const int64_t granules = std::max<int64_t>(1, ((int64_t)max_context + kGranule - 1) / kGranule);
  t.longest = times(units, granules);
  t.workers = (int32_t)std::max<int64_t>(1, std::min<int64_t>(num_sms / t.group, t.longest));
  t.part_rows = (int32_t)(std::min<int64_t>(kChunks, std::max<int64_t>(1, chunks)) * kChunkRows);
  // as many warps to a row as leave each about four of its parts (of units of equal length)
  t.row_warps = 1;
  while (units > 0 && t.row_warps < kCombineWarps && t.workers / units >= 4 * t.row_warps)
    t.row_warps *= 2;
  const int32_t ctas = t.workers * t.group;
  t.by_unit = units <= t.workers;
  // Contexts short enough (by max_context_len: 8 x 1024 takes 17.3 us where that is 32768, 15.5 where it
  // is 1024) are not cut and the merge is not launched, which pays the longer, the fewer workers are left
  // without a unit. The limits were read off these shapes of 16 / 8 heads, 19 workers, and go for all (us,
  // whole and cut): 1 x 832 12.6 and 10.7; 5 x 1024 14.5 and 16.3, 5 x 1152 15.9 and 15.1; 8 x 1024 15.7
  // and 17.2, 8 x 1536 20.0 and 20.3; 16 x 1536 23.6 and 25.2. Where the merge has to be launched for
  // longer ones, a whole unit pays up to 12 granules (8 x 1536: 21.5 and 20.3), with many workers to
  // spare up to 7.
  const int64_t spare = units > 0 ? t.workers / units : 0;
  const int32_t limit = spare >= 8 ? 8 : spare >= 3 ? 16 : spare >= 2 ? 20 : 24;
  t.uncut = t.by_unit && max_context <= limit * kGranule;
  t.whole = t.uncut ? limit : spare >= 4 ? 7 : 12;
  t.cuts = t.by_unit ? (int32_t)std::max<int64_t>(1, units) * t.group : ctas;
  // Blocks of two warps fit beside the main kernel's CTA over the 8-bit cache (118 of 128 registers a
  // thread) and are there when it ends (256 ragged 170 us, 172 with four warps, 176 with eight; the bf16
  // kernel's CTA has all registers); with many rows more blocks cost more (8 x 1024, 64 nodes of 16 / 8
  // heads: 23.8, 23.0, 22.6). As many as all rows take, but no more than run at once unless a row takes
  // several warps.
  t.block_warps = std::max(t.part_rows <= 32 ? 2 : 4, t.row_warps);
  t.cut_blocks = t.part_rows * t.row_warps / t.block_warps;
  if (t.row_warps == 1)
    t.cut_blocks = std::max(1, std::min(t.cut_blocks, 32 / t.block_warps * num_sms / t.cuts));
  // The workspace has room for as many CTAs and cuts as a call of these bounds or smaller ones can have:
  // a workspace for a program's largest call is large enough for all others, although one more row
  // tile may leave fewer CTAs (two groups of 76 make 152, three of 50 make 150).
  const size_t most =
      (size_t)std::max<int64_t>(ctas, std::min<int64_t>(num_sms, times(t.longest, t.group)));
  t.part_o = most * sizeof(CutInfo);
  t.part_lse = t.part_o + most * 2 * t.part_rows * kD * sizeof(float);
  t.bytes = align16(t.part_lse + most * 2 * t.part_rows * sizeof(float)) + 16;  // (see launch_tree)
  return t;
}

template <Mode M>
cudaError_t launch_tree(TreeParams p, const TreePlan &t, void *workspace, cudaStream_t stream) {
  CUtensorMap km, vm;
  const uint64_t rows = (uint64_t)p.num_blocks * p.block_size;
  const uint64_t wide[3] = {64, rows, (uint64_t)p.hkv * 2}, narrow[3] = {kD, rows, (uint64_t)p.hkv};
  const uint64_t wide_strides[2] = {(uint64_t)p.hkv * kD * 2, 128};
  const uint64_t narrow_strides[2] = {(uint64_t)p.hkv * kD, kD};
  const uint32_t wide_box[3] = {64, kGranule, 1}, narrow_box[3] = {kD, kGranule, 1};
  auto encode = [&](CUtensorMap *map, const uint8_t *pool) {
    return encode_tensor_map(
               map, M == kFp8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
               const_cast<uint8_t *>(pool), M == kFp8 ? narrow : wide,
               M == kFp8 ? narrow_strides : wide_strides, M == kFp8 ? narrow_box : wide_box,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B) == CUDA_SUCCESS;
  };
  if (!encode(&km, p.k_cache) || !encode(&vm, p.v_cache)) return cudaErrorInvalidValue;
  p.group = t.group;
  p.heads = t.heads;
  p.at_once = t.at_once;
  p.per_tile = p.hkv / t.heads;
  p.nb_magic = t.nb > 1 ? (uint32_t)((1ull << 32) / t.nb + 1) : 0;
  p.hb_magic = t.hb > 1 ? (uint32_t)((1ull << 32) / t.hb + 1) : 0;
  p.workers = t.workers;
  p.whole = t.whole;
  p.hb = t.hb;
  p.nb = t.nb;
  p.parts = t.parts;
  // (the caller's 16 bytes of alignment made the 32 that the partial results are stored with)
  uint8_t *ws =
      reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(workspace) + 31) & ~uintptr_t(31));
  p.cuts = reinterpret_cast<CutInfo *>(ws);
  p.by_unit = t.by_unit;
  p.max_units = (int32_t)t.units;
  p.part_o = reinterpret_cast<float *>(ws + t.part_o);
  p.part_lse = reinterpret_cast<float *>(ws + t.part_lse);
  p.part_rows = t.part_rows;
  p.row_warps = t.row_warps;
  p.block_warps = t.block_warps;
  const size_t smem = sizeof(TreeSmem<M>) + 1024;
  static bool ready[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev >= 64 || !ready[dev]) {
    e = cudaFuncSetAttribute(tree_flash_kernel<M>, cudaFuncAttributeMaxDynamicSharedMemorySize,
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
  e = cudaLaunchKernelEx(&cfg, tree_flash_kernel<M>, km, vm, p);
  if (e != cudaSuccess || t.workers == 1 || t.uncut) return e;
  return launch_after(tree_combine_kernel<M>, dim3((unsigned)t.cuts, (unsigned)t.cut_blocks),
                      t.block_warps * 32, stream, p);
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
      max_seqlen_q > (1 << 20) || num_blocks > INT32_MAX / block_size)
    return PKV_ERR_UNSUPPORTED;
  if (q_tok_stride % 8 != 0 || !aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) ||
      !aligned16(out) || (fp8 && (!aligned16(k_scale) || !aligned16(v_scale))))
    return PKV_ERR_UNSUPPORTED;
  // (a CTA reads rows of q whose outputs another one has written)
  if (overlap(q, total_q, 2 * (__int128)q_tok_stride, 2 * (int64_t)num_q_heads * head_dim, out,
              2 * total_q * num_q_heads * head_dim))
    return PKV_ERR_INVALID_ARG;
  unsigned int *err = current_error_word();
  const int num_sms = current_sm_count();
  if (!err || num_sms <= 0) return PKV_ERR_CUDA;
  // (positions up to a tile past the context are 32 bits)
  const int32_t longest = (int32_t)std::min<int64_t>(
      std::min(max_context_len, INT32_MAX - 1024), (int64_t)block_table_width * block_size);
  const TreePlan plan =
      plan_tree(num_seqs, max_seqlen_q, num_q_heads, num_kv_heads, longest, num_sms);
  if (plan.longest > (1 << 30)) return PKV_ERR_UNSUPPORTED;
  if (!workspace || !aligned16(workspace) || workspace_bytes < plan.bytes) return PKV_ERR_WORKSPACE;
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
  prm.max_context = longest;
  prm.mask = reinterpret_cast<const uint64_t *>(tree_mask);
  prm.mask_words = mask_words;
  prm.hq = num_q_heads;
  prm.hkv = num_kv_heads;
  prm.group_heads = num_q_heads / num_kv_heads;
  prm.block_size = block_size;
  prm.num_blocks = num_blocks;
  prm.num_seqs = num_seqs;
  // (a scale of 0 would turn the -inf of a masked score into NaN)
  prm.scale_log2 = std::min(std::max(fabsf(scale) * kLog2e, 1e-37f), 1e37f);
  prm.q_sign = scale < 0.f ? 0x80008000u : 0u;
  prm.out = static_cast<uint16_t *>(out);
  prm.out_32b = (reinterpret_cast<uintptr_t>(out) & 31u) == 0;
  prm.err = err;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = fp8 ? launch_tree<kFp8>(prm, plan, workspace, st)
                            : launch_tree<kBf16>(prm, plan, workspace, st);
  return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
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

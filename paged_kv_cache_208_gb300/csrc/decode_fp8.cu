// decode_fp8.cu -- paged decode attention over the 8-bit cache on the 5th-generation tensor cores
// (sm_103a). The format is in fp8_cache.cuh.
//
// Work units, their queue, the clusters of splits and the merges are the bf16 decode kernel's
// (decode.cu): a unit is one sequence, one KV head, up to eight of its query heads and one split
// of the context. What differs is that half the bytes leave half the time for each token. With
// warp MMAs every code has to be converted (K and V to fp16: 64 conversions and 24 MMAs per warp
// and 16 tokens kept the SM's ALUs 45% busy, 97 us for 256 ragged contexts where the bytes take
// 77); tcgen05 reads the e4m3 tiles from shared memory as TMA left them. Per 128-token tile, M =
// 128 both times:
//
//   S^T (128 tokens x 16)   = K (128 x 128 dims) Q^T      A = the K tile, K-major
//   O^T (128 dims x N)     += V^T (128 x 128 tokens) P^T  A = the V tile, M-major
//
// q and P enter as sums of e4m3 numbers, in columns of their own (N is at least 16 anyway):
//   q:  q' = q times the power of two that brings the head's maximum into [128, 256);
//       hi = e4m3(q'), lo = e4m3(32 (q' - hi)). 4 + 4 bits hold bf16's 8: exact down to 2^-14 of
//       the maximum, within 2^-22 of it below.
//   P:  w = 2^(s + ev - R + 5) with ev = log2 of V's scale of the group and R a reference that
//       no s + ev exceeds by more than 3, so w <= 256; w = t1 + t2 / 32 + t3 / 32^2 + t4 / 32^3,
//       each t the e4m3 of 32 times what the ones before left: within 2^-19 of w (2^-4 and three
//       times 2^-5) or, where t4 is below e4m3's normal range, 2^-25 (2^-30 of the reference's own
//       weight). Three parts hold 2^-14 and 2^-20: 131071 equal weights of 2^-24.6 beside a token
//       with nearly all of the weight gave an output of 3.48 for 2.36 in one split, and 0.9% of
//       the outputs of 256 ragged contexts rounded to another neighbour than with fp32 weights
//       (0.05% with four). The columns are there anyway; the fourth conversion costs 0.1 us of 7.2
//       (8 x 1024), 0.2 of 16.8 (33 x 4999 with 16 / 2 heads), 0.8 of 64.3 (256 up to 1024, 64 / 8).
// K's scale multiplies the scores. V's scale is in the exponent, so that one accumulator serves
// groups of any scales: it holds sum w code = 2^(5 - R) sum 2^s v, and l sums w 2^-ev =
// 2^(5 - R) 2^s in fp32 from the unrounded w; their quotient is the output.
//
// R is the maximum over the unit's first tile; later tiles raise it (and rescale O in tensor
// memory and l) only when a token exceeds it by more than 3, which the softmax threads agree on
// with one barrier reduction per tile.
//
// Warps (352 threads, two CTAs per SM): 0-7 softmax (two threads per token of the tile, each for
// half of the heads; in the epilogue two per dimension of O), 8 issues S (and turns each unit's q
// into its two parts), 9 issues PV, 10 loads: TMA tiles of K and of V in rings of 16 KiB slots, the scales of the
// tile's 256-token page (16 bytes each of K and V) with V's tile. S and P have two buffers, so
// S(t + 1) is computed while the softmax works on tile t; O has two, so a unit's first PV does
// not wait for the last unit's epilogue.
//
// Of a context's last tile only the boxes (of 32 and 16 rows) with its tokens are loaded; V's rows
// past them are zeroed in shared memory, as 0 x NaN from a stale row would poison O.
#include "decode_common.cuh"
#include "fp8_cache.cuh"
#include "tcgen05.cuh"

namespace pkv {
namespace {

constexpr int kTile = 128;
constexpr int kTileBytes = kTile * kD;  // one head's K or V codes of a tile: 16 KiB
// Slots of the K ring and of the V ring. (Six, for grids of one CTA per SM, were no faster -- one
// CTA's loads arrive at a tile per 0.65 us either way -- and clusters of 5 and more then do not
// all fit at once.)
constexpr int kSlots = 3;
// Boxes of a context's last tile: as many of 32 rows as fit, the rest in one more of 32 or of 16
// rows. One thread issues every load, and each costs it about 250 cycles: in boxes of 8 rows a tile
// of 60 rows took 16 of them (300 contexts of 1 to 500 tokens, 32 / 8 heads: 53.1 us, so 49.8).
constexpr int kBoxRows = 32, kSmallBoxRows = 16;
constexpr int kSoftmaxWarps = 8;  // two for each quadrant of tensor memory's lanes
constexpr int kSoftmaxThreads = kSoftmaxWarps * 32;
constexpr int kSWarp = 8, kPvWarp = 9, kLoadWarp = 10;
constexpr int kThreads = 11 * 32;
constexpr int kUnitConsumers = kSoftmaxWarps + 2;
constexpr float kTop = 5.f;       // log2 of the reference's own w
constexpr float kHeadroom = 3.f;  // log2 of how far a w may exceed it
constexpr float kMinScale = 7.8886090522101181e-31f;  // 2^-100

template <int GC>
struct Kind {
  // Heads of a softmax thread: the first or the second half of the unit's. Rows of Q (columns of
  // S) are hi then lo of the first half's heads, then of the second's; columns of P (and of O)
  // likewise t1 to t4, the second half's from column kHalf on.
  static constexpr int kGH = GC / 2;
  static constexpr int kRing = GC <= 4 ? 4 : 2;  // units in flight
  static constexpr int kQRows = GC <= 4 ? 8 : 16;   // 2 GC rows used
  static constexpr int kNO = GC <= 4 ? 16 : 32;     // N of the second product, P's columns
  static constexpr int kHalf = kNO / 2;             // a half's columns, 4 GH of them used
  static constexpr uint32_t kOBase = 32;            // TMEM: S buffers at 0 and 16, then O's
  static constexpr uint32_t kTmemCols = GC <= 4 ? 64 : 128;
  // Where a cluster's rank 0 receives its peers' results: with up to this many splits in an
  // area past the fixed layout (two CTAs still fit on an SM), else in its K slots, lent once it
  // needs them no more. (splits - 1) x GC x kD outputs, then (splits - 1) x GC log2-sum-exps.
  static constexpr int kLandSplits = GC <= 2 ? 4 : 1;
};

// Q tiles have rows of 128 bytes, 128-byte swizzle. N = 16 rows are multiplied; those past the
// allocated ones run into what follows in shared memory (the next buffer; from the last Q tile the
// queued q rows), and give columns that nothing reads.
// P tiles are stored by token (MN-major: 16 bytes of a token's columns, 8 tokens to a 128-byte
// block), so that a softmax thread writes its heads' codes as one word, not byte by byte into the
// rows of a K-major tile: with eight heads 16 byte stores and their shifts fewer per thread, 33 x
// 4999 with 16 / 2 heads 20.5 -> 17.5 us, 8 x 1024 7.7 -> 7.3 us. With two heads a unit a half's
// columns from the fifth on hold anything; nothing reads theirs of O.
// A unit as the loader hands it out: everything about it that the others need.
struct Unit8 {
  int32_t b, s, xg, ntiles;  // ntiles < 0: no more work
  int32_t tokens;            // of the split
  int32_t whole;             // the split is the whole context: its result is the output
  int32_t skip;              // the ring's next tile is a speculative load to be dropped
  int32_t h, head0;          // KV head; first query head of the unit in its group
};

template <int GC>
struct DecodeFp8Smem {
  using K = Kind<GC>;
  uint8_t k[kSlots][kTileBytes];  // 1024-byte aligned, as the layout (128-byte swizzle atoms)
  uint8_t v[kSlots][kTileBytes];
  uint8_t p[2][K::kNO * kTile];
  uint8_t q[2][K::kQRows * 128];
  uint16_t qs[K::kRing][GC][kD];  // q rows of the queued units, as they came
  alignas(16) float tile_scale[kSlots][2][4];  // scales of the tile's page: K's, V's
  float qscale[2][GC];                         // softmax scale log2(e) over q's power of two
  float warp_max[kSoftmaxWarps][GC / 2];
  float warp_l[2][kSoftmaxWarps][GC / 2];
  Unit8 unit[K::kRing];
  int32_t stop;  // set by the producer: an earlier wait gave up, this CTA does no work
  uint32_t tmem_base;
  uint64_t k_full[kSlots], k_empty[kSlots], v_full[kSlots], v_empty[kSlots];
  uint64_t q_ready[2], s_full[2], p_full[2], pv_done[2], o_full[2], o_free[2];
  uint64_t unit_full[K::kRing], unit_empty[K::kRing];
  uint64_t drain[2];
  // cluster merge: the peers' results have landed; the area is lent; in a peer: the merged
  // log2-sum-exps have landed in `lse`
  uint64_t cl_bar, cl_ready, cl_lse;
  float lse[GC];  // of the whole context, for the weights
};

template <int GC>
__host__ __device__ constexpr size_t land_offset() {
  return (sizeof(DecodeFp8Smem<GC>) + 15) / 16 * 16;
}
template <int GC>
__host__ __device__ constexpr size_t fp8_smem_bytes(int cluster) {
  return (cluster >= 2 && cluster <= Kind<GC>::kLandSplits
              ? land_offset<GC>() + (size_t)(cluster - 1) * GC * (kD + 1) * sizeof(float)
              : sizeof(DecodeFp8Smem<GC>));
}
// two CTAs per SM: 228 KiB less 1 KiB each that the system keeps
static_assert(fp8_smem_bytes<2>(4) <= 113 * 1024 && fp8_smem_bytes<4>(1) <= 113 * 1024 &&
                  fp8_smem_bytes<8>(1) <= 113 * 1024,
              "two CTAs fit on an SM");
static_assert((kMaxCluster - 1) * 8 * (kD + 1) * sizeof(float) <= kSlots * kTileBytes,
              "the peers' results fit in rank 0's K slots");

// A position in a ring of tiles: the slot, and the parity of the phase a use of it completes.
struct Ring {
  int slot = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void next() {
    if (++slot == kSlots) {
      slot = 0;
      parity ^= 1u;
    }
  }
};

__device__ __forceinline__ float redux_max(float x) {
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(x));
  return r;
}

constexpr int kParts = 4;  // e4m3 numbers to a softmax weight

// The e4m3 parts of a pair of weights (0 <= w <= 256), each pair's codes in 16 bits; every
// difference is exact.
__device__ __forceinline__ void split_weights(float a, float b, uint32_t (&t)[kParts]) {
  const float2 up = make_float2(32.f, 32.f), down = make_float2(-32.f, -32.f);
  const float2 zero = make_float2(0.f, 0.f);
  float2 r = make_float2(a, b);
  t[0] = cvt_e4m3x2(a, b);
#pragma unroll
  for (int i = 1; i < kParts; ++i) {
    r = ffma2(f16x2_to_f32(cvt_f16x2_e4m3x2(t[i - 1])), down, ffma2(r, up, zero));
    t[i] = cvt_e4m3x2(r.x, r.y);
  }
}

template <int GC, bool W>
__global__ void __launch_bounds__(kThreads, 2)
    decode_fp8_kernel(const __grid_constant__ CUtensorMap kmap,
                      const __grid_constant__ CUtensorMap vmap,
                      const __grid_constant__ CUtensorMap kmap32,
                      const __grid_constant__ CUtensorMap vmap32,
                      const __grid_constant__ CUtensorMap kmap16,
                      const __grid_constant__ CUtensorMap vmap16, const DecodeParams p) {
  using K = Kind<GC>;
  constexpr int kRing = K::kRing, GH = K::kGH;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  DecodeFp8Smem<GC> &sm = *reinterpret_cast<DecodeFp8Smem<GC> *>(smem_raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    sm.stop = 0;
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(&sm.k_full[i], 1);
      mbar_init(&sm.k_empty[i], 1);
      mbar_init(&sm.v_full[i], 1);
      mbar_init(&sm.v_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.q_ready[i], 1);
      mbar_init(&sm.s_full[i], 2);
      mbar_init(&sm.p_full[i], kSoftmaxWarps);
      mbar_init(&sm.pv_done[i], 1);
      mbar_init(&sm.o_full[i], 1);
      mbar_init(&sm.o_free[i], kSoftmaxWarps);
      mbar_init(&sm.drain[i], 1);
    }
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&sm.unit_full[i], 1);
      mbar_init(&sm.unit_empty[i], kUnitConsumers);
    }
    if (p.cluster) {
      mbar_init(&sm.cl_bar, p.cluster - 1);  // one arrival per peer
      mbar_init(&sm.cl_ready, 1);
      mbar_init(&sm.cl_lse, 1);
    }
    fence_mbar_init();
  }
  if (warp == kSWarp) {
    tmem_alloc(&sm.tmem_base, K::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = sm.tmem_base;
  // in a cluster: this CTA's barriers are set up (waited for before the first remote access)
  if (p.cluster) cluster_arrive_relaxed();
  // cluster merge: this CTA's normalised outputs of dimension threadIdx.x % 128 (the thread's
  // heads) and their log2-sum-exps
  float cl_o[GH], cl_lse[GH];
  [[maybe_unused]] int cl_end = 0;  // where its positions end
#pragma unroll
  for (int g = 0; g < GH; ++g) {
    cl_o[g] = 0.f;
    cl_lse[g] = -INFINITY;
  }

  // Launched as a programmatic dependent of the stream's previous kernel: everything above may
  // overlap its tail; wait for that grid's completion and memory before touching global memory.
  // While it finishes, the loader of a static grid warms L2 with its context length, and with
  // its first tiles through a block id read ahead of the wait (only a hint: every value used
  // below is read again).
  int32_t spec_blk = -1, spec_row = -1, spec_h = 0;
  if (threadIdx.x == kLoadWarp * 32) {
    prefetch_tensormap(&kmap);
    prefetch_tensormap(&vmap);
    prefetch_tensormap(&kmap32);
    prefetch_tensormap(&vmap32);
    prefetch_tensormap(&kmap16);
    prefetch_tensormap(&vmap16);
    if (!p.queue) {
      int s, b, xg;
      unit_coords(p, blockIdx.x, s, b, xg);
      prefetch_l2(p.context_lens + b);
      const int64_t begin = (int64_t)s * p.chunk;
      if (begin < p.cap) {
        const int32_t blk =
            ld_global_cg_s32(p.block_tables + (int64_t)b * p.table_width + begin / p.block_size);
        if (blk >= 0 && blk < p.num_blocks) {
          const int in_block = (int)(begin % p.block_size);
          const int n = min(2 * kSlots, min(p.chunk, p.block_size - in_block) / kTile);
          spec_h = xg / p.head_groups;
          spec_blk = blk;
          spec_row = (int32_t)((int64_t)blk * p.block_size + in_block);
          for (int t = 0; t < n; ++t) {
            tma_prefetch_3d(&kmap, 0, spec_row + t * kTile, spec_h);
            tma_prefetch_3d(&vmap, 0, spec_row + t * kTile, spec_h);
          }
        }
      }
    }
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
  // the kernel that follows may be scheduled now: it waits for this grid's completion (and its
  // memory) before reading anything
  if (threadIdx.x == 0) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (warp == kLoadWarp) {
    // ------------------------------------------------------------------------ loads
    if (lane == 0) {
      const uint64_t policy = policy_evict_first();
      uint32_t pushed = 0;
      Ring kr, vr;                     // the next slot of K and of V
      int k_issued = 0, v_issued = 0;  // capped at the rings' length
      bool ok = true, first_unit = true;
      int static_next = blockIdx.x;  // without a queue: unit blockIdx.x, then nothing
      // The work counter (queued grid): as in decode.cu, every CTA draws until it draws past the
      // last unit, once, and the CTA with the last of those draws sets it back to zero.
      bool first_draw = true, past_end = false;
      auto draw = [&]() -> int {
        const int u = atomicAdd(p.queue, 1);
        if (first_draw) {
          first_draw = false;
          if (u < 0 || u >= p.units + (int)gridDim.x) record_error(p.err, kErrWorkspace);
        }
        if (u < 0 || u >= p.units) {
          past_end = true;
          if (u == p.units + (int)gridDim.x - 1) atomicExch(p.queue, 0);
        }
        return u;
      };
      // the scales of the 256-token page around row in_block of a block, 16 bytes each
      auto load_scales = [&](int slot, int64_t blk, int in_block, int h) {
        const int64_t at = (blk * p.num_kv_heads + h) * (p.block_size / kFp8Group) +
                           (in_block & ~255) / kFp8Group;
        bulk_copy_g2s(sm.tile_scale[slot][0], p.k_scale + at, 16, &sm.v_full[slot]);
        bulk_copy_g2s(sm.tile_scale[slot][1], p.v_scale + at, 16, &sm.v_full[slot]);
      };
      constexpr uint32_t kScaleBytes = 32;
      // The first tile, at once, with the block id read ahead of the wait; kept if the id still
      // holds when the table is read again, else dropped (Unit::skip) and loaded again.
      bool spec_pending = false;
      if (spec_row >= 0) {
        mbar_arrive_expect_tx(&sm.k_full[0], kTileBytes);
        tma_load_3d(sm.k[0], &kmap, &sm.k_full[0], 0, spec_row, spec_h, policy);
        mbar_arrive_expect_tx(&sm.v_full[0], kTileBytes + kScaleBytes);
        tma_load_3d(sm.v[0], &vmap, &sm.v_full[0], 0, spec_row, spec_h, policy);
        load_scales(0, spec_blk, (int)(spec_row - (int64_t)spec_blk * p.block_size), spec_h);
        kr.next();
        vr.next();
        k_issued = v_issued = 1;
        spec_pending = true;
      }
      while (ok) {
        // next unit with work (or one that must write zeros); ntiles < 0 ends the walk
        Unit8 un{0, 0, 0, -1, 0, 0, 0};
        int32_t first_blk = -1;   // block id of the unit's first tile
        int first_it = 0;         // tiles of the unit already loaded
        while (true) {
          int u;
          if (p.queue) {
            u = draw();
          } else {
            u = static_next;
            static_next = p.units;
          }
          if (u < 0 || u >= p.units) break;
          int s, b, xg;
          unit_coords(p, u, s, b, xg);
          // the first tile's block id does not depend on the context length: both loads are in
          // flight together (a unit that starts past the table's end reads no entry)
          const int64_t begin = (int64_t)s * p.chunk;
          const uint32_t err_now =
              first_unit ? (uint32_t)ld_global_s32(reinterpret_cast<const int32_t *>(p.err)) : 0u;
          int64_t L = ld_global_s32(p.context_lens + b);
          if (begin < p.cap)
            first_blk = ld_global_s32(p.block_tables + (int64_t)b * p.table_width +
                                      begin / p.block_size);
          if (first_unit) {
            first_unit = false;
            if (err_now & kErrTimeout) {  // an earlier wait gave up somewhere: end the walk
              sm.stop = 1;
              break;
            }
          }
          if (L < 0 || L > p.cap) {
            if (s == 0 && xg == 0) record_error(p.err, 4u /* CONTEXT_RANGE */);
            L = L < 0 ? 0 : p.cap;
          }
          if (begin < L) {
            const int64_t end = min(L, begin + p.chunk);
            un = Unit8{b, s, xg, (int)((end - begin + kTile - 1) / kTile), (int)(end - begin),
                       p.splits == 1 || (s == 0 && end == L) ? 1 : 0, 0};
            if (spec_pending) {
              if (first_blk == spec_blk) first_it = 1;
              else un.skip = 1;
              spec_pending = false;
            }
            break;
          }
          if (p.cluster || (L == 0 && s == 0 && p.splits == 1)) {
            // nothing to read: zeros (empty context), or in a cluster no result (the unit
            // still leaves its -inf log2-sum-exp for the merge)
            un = Unit8{b, s, xg, 0, 0, p.splits == 1 ? 1 : 0, spec_pending ? 1 : 0};
            spec_pending = false;
            break;
          }
        }
        const int slot = pushed % kRing;
        if (pushed >= kRing &&
            !wait_parity(&sm.unit_empty[slot], ((pushed / kRing) - 1) & 1, p.err)) {
          ok = false;
          break;
        }
        const int h = un.xg / p.head_groups;
        un.h = h;
        un.head0 = (un.xg - h * p.head_groups) * GC;
        sm.unit[slot] = un;
        ++pushed;
        if (un.ntiles < 0) {
          mbar_arrive(&sm.unit_full[slot]);
          break;
        }
        const uint32_t q_bytes = min(GC, p.group - un.head0) * kD * 2;
        mbar_arrive_expect_tx(&sm.unit_full[slot], q_bytes);
        bulk_copy_g2s(sm.qs[slot],
                      p.q + ((int64_t)un.b * p.num_q_heads + h * p.group + un.head0) * kD, q_bytes,
                      &sm.unit_full[slot]);
        // The table is read a block ahead (an entry's latency is longer than a tile's share of the
        // bandwidth: with a read per tile the loads ran at one tile per 0.68 us and CTA).
        const int32_t *entry =
            p.block_tables + (int64_t)un.b * p.table_width + un.s * p.chunk / p.block_size;
        int in_block = un.s * p.chunk % p.block_size;
        int left = un.tokens;  // from the current tile on
        int32_t blk = first_blk, next_blk = -1;
        if (left > p.block_size - in_block) next_blk = ld_global_s32(++entry);
        for (int it = 0; it < un.ntiles; ++it) {
          if (it > 0) {
            left -= kTile;
            in_block += kTile;
            if (in_block == p.block_size) {
              in_block = 0;
              blk = next_blk;
              if (left > p.block_size) next_blk = ld_global_s32(++entry);
            }
          }
          if (it < first_it) continue;
          const bool blk_ok = blk >= 0 && blk < p.num_blocks;
          if (!blk_ok) record_error(p.err, 2u /* BLOCK_RANGE */);
          // (a row wholly outside the pool: TMA fills zeros, nothing is read)
          const int32_t row = blk_ok ? blk * p.block_size + in_block : -2 * kTile;
          const int rows_here = min(left, kTile);
          // (blocks are whole tiles: a box that runs past the context stays inside the block)
          const bool whole = rows_here > kTile - kSmallBoxRows || !blk_ok;
          const int boxes = (rows_here + kBoxRows - kSmallBoxRows - 1) / kBoxRows;
          const int boxed = boxes * kBoxRows;
          const bool rest = boxed < rows_here;
          const uint32_t bytes =
              whole ? kTileBytes : (uint32_t)(boxed + (rest ? kSmallBoxRows : 0)) * kD;
          auto load = [&](uint8_t *dst, const CUtensorMap *map, const CUtensorMap *map32,
                          const CUtensorMap *map16, uint64_t *bar) {
            if (whole) return tma_load_3d(dst, map, bar, 0, row, h, policy);
            for (int r = 0; r < boxed; r += kBoxRows)
              tma_load_3d(dst + r * kD, map32, bar, 0, row + r, h, policy);
            if (rest) tma_load_3d(dst + boxed * kD, map16, bar, 0, row + boxed, h, policy);
          };
          // (a slot's first use finds it empty; later ones wait for the use before, whose phase has
          // the other parity)
          if (k_issued == kSlots && !wait_parity(&sm.k_empty[kr.slot], kr.parity ^ 1u, p.err)) {
            ok = false;
            break;
          }
          uint8_t *kd = sm.k[kr.slot], *vd = sm.v[vr.slot];
          uint64_t *kbar = &sm.k_full[kr.slot], *vbar = &sm.v_full[vr.slot];
          mbar_arrive_expect_tx(kbar, bytes);
          load(kd, &kmap, &kmap32, &kmap16, kbar);
          kr.next();
          k_issued = min(k_issued + 1, kSlots);
          if (v_issued == kSlots && !wait_parity(&sm.v_empty[vr.slot], vr.parity ^ 1u, p.err)) {
            ok = false;
            break;
          }
          if (blk_ok) {
            mbar_arrive_expect_tx(vbar, bytes + kScaleBytes);
            load_scales(vr.slot, blk, in_block, h);
          } else {
            // the zero rows of a bad block id: a scale of 1 (no block's scales are theirs, and
            // any block's may be unwritten)
            float4 *const scales = reinterpret_cast<float4 *>(sm.tile_scale[vr.slot]);
            scales[0] = scales[1] = make_float4(1.f, 1.f, 1.f, 1.f);
            fence_async_shared();  // (the slot's next scales come by a bulk copy)
            mbar_arrive_expect_tx(vbar, bytes);
          }
          load(vd, &vmap, &vmap32, &vmap16, vbar);
          vr.next();
          v_issued = min(v_issued + 1, kSlots);
        }
      }
      // a CTA that stopped early still draws past the last unit once, so that the counter goes
      // back to zero
      if (p.queue)
        while (!past_end) draw();
      // keep the CTA alive until every copy it issued has landed (these waits ignore the abort
      // bit; the counts are of issued copies)
      bool drained = true;
      // (slot i's last use was in this turn of the ring if the position is past it, else in the
      // turn before)
      for (int i = 0; drained && i < k_issued; ++i)
        drained = wait_own(&sm.k_full[i], i < kr.slot ? kr.parity : kr.parity ^ 1u, p.err);
      for (int i = 0; drained && i < v_issued; ++i)
        drained = wait_own(&sm.v_full[i], i < vr.slot ? vr.parity : vr.parity ^ 1u, p.err);
      for (uint32_t t = pushed > kRing ? pushed - kRing : 0; drained && t < pushed; ++t)
        drained = wait_own(&sm.unit_full[t % kRing], (t / kRing) & 1, p.err);
    }
    __syncwarp();
  } else if (warp == kSWarp) {
    // ------------------------------------------------------------------------ S = K Q^T
    constexpr uint32_t kId = idesc_e4m3_f32(128, 16, 0, 0);
    const uint64_t dk = smem_desc_sw128(smem_addr(sm.k[0]), 16, 1024);
    const uint64_t dq = smem_desc_sw128(smem_addr(sm.q[0]), 16, 1024);
    auto wait_all = [&](uint64_t *bar, uint32_t parity) -> bool {
      return __all_sync(kFull, wait_parity(bar, parity, p.err));
    };
    uint32_t taken = 0, units = 0, t = 0;  // t: tiles computed
    Ring kr, vr;
    bool ok = true;
    while (ok) {
      const int slot = taken % kRing;
      if (!(ok = wait_all(&sm.unit_full[slot], (taken / kRing) & 1))) break;
      const Unit8 un = sm.unit[slot];
      ++taken;
      if (un.ntiles < 0) break;
      if (un.skip) {  // a speculative load that did not hold: let it land, drop it
        if (!(ok = wait_all(&sm.k_full[kr.slot], kr.parity))) break;
        if (lane == 0) mbar_arrive(&sm.k_empty[kr.slot]);
        kr.next();
        vr.next();
      }
      if (un.ntiles > 0) {
        // This unit's Q tile was last read by the unit before the last one, all of whose tiles
        // precede tile t - 1: their S is complete once the softmax has answered tile t - 2.
        if (t >= 2 && !(ok = wait_all(&sm.p_full[t & 1], ((t - 2) >> 1) & 1))) break;
        const int qb = units & 1;
        const int heads = min(GC, p.group - un.head0);
        uint8_t *qt = sm.q[qb];
        // row r, lane's four dimensions: byte 4 lane of the 128, swizzled by 16-byte chunks
        auto at = [&](int r) {
          return reinterpret_cast<uint32_t *>(qt + r * 128 + (((lane >> 2) ^ (r & 7)) << 4) +
                                              (lane & 3) * 4);
        };
#pragma unroll
        for (int g = 0; g < GC; ++g) {
          uint32_t hi = 0u, lo = 0u;
          if (g < heads) {
            const uint2 w = *reinterpret_cast<const uint2 *>(&sm.qs[slot][g][4 * lane]);
            const float a[4] = {bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y)};
            // the head's largest |q| as bits (a NaN is larger than everything, and its own code
            // makes the scores NaN)
            const uint32_t top = __reduce_max_sync(
                kFull, max(max(__float_as_uint(a[0]) & 0x7fffffffu, __float_as_uint(a[1]) & 0x7fffffffu),
                           max(__float_as_uint(a[2]) & 0x7fffffffu, __float_as_uint(a[3]) & 0x7fffffffu)));
            const int e = min(max((int)(top >> 23), 8), 254);             // 2^(e - 127) <= max |q|
            const float up = __uint_as_float((uint32_t)(261 - e) << 23);  // 2^(134 - e)
            hi = cvt_e4m3x2(a[0] * up, a[1] * up) | (cvt_e4m3x2(a[2] * up, a[3] * up) << 16);
            const float2 r0 = f16x2_to_f32(cvt_f16x2_e4m3x2(hi));
            const float2 r1 = f16x2_to_f32(cvt_f16x2_e4m3x2_hi(hi));
            lo = cvt_e4m3x2(fmaf(a[0], up, -r0.x) * 32.f, fmaf(a[1], up, -r0.y) * 32.f) |
                 (cvt_e4m3x2(fmaf(a[2], up, -r1.x) * 32.f, fmaf(a[3], up, -r1.y) * 32.f) << 16);
            // softmax scale / up; an infinite q makes its head's scores NaN
            if (lane == 0)
              sm.qscale[qb][g] = top == 0x7f800000u
                                     ? __uint_as_float(0x7fffffffu)
                                     : p.qscale * __uint_as_float((uint32_t)(e - 7) << 23);
          } else if (lane == 0) {
            sm.qscale[qb][g] = 0.f;
          }
          *at((g / GH) * 2 * GH + g % GH) = hi;
          *at((g / GH) * 2 * GH + GH + g % GH) = lo;
        }
        fence_async_shared();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&sm.q_ready[qb]);
          mbar_arrive(&sm.unit_empty[slot]);
        }
        ++units;
        for (int it = 0; it < un.ntiles; ++it, ++t, kr.next(), vr.next()) {
          // S(t)'s buffer was tile t - 2's, which the softmax has read; P(t)'s was tile t - 2's
          // too, which its PV has read. With V's tile (and the scales) here as well, s_full tells
          // the softmax threads all they would else wait for one by one, 100 cycles each.
          if (t >= 2 && !(ok = wait_all(&sm.pv_done[t & 1], ((t - 2) >> 1) & 1))) break;
          if (!(ok = wait_all(&sm.k_full[kr.slot], kr.parity))) break;
          if (!(ok = wait_all(&sm.v_full[vr.slot], vr.parity))) break;
          tc_fence_after_sync();
          if (elect_one()) {
            const uint64_t a = dk + kr.slot * (kTileBytes >> 4);
            const uint64_t b = dq + qb * (K::kQRows * 128 >> 4);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)  // 32 dims: 32 bytes along the swizzled rows
              umma_e4m3_ss(tmem + 16 * (t & 1), a + 2 * kk, b + 2 * kk, kId, kk > 0);
            mbar_arrive(&sm.s_full[t & 1]);  // (releases what this thread has seen)
            umma_commit(&sm.s_full[t & 1]);
            umma_commit(&sm.k_empty[kr.slot]);
          }
          __syncwarp();
        }
      } else if (lane == 0) {
        mbar_arrive(&sm.unit_empty[slot]);
      }
    }
    // every UMMA must be complete before the CTA exits, also after an abort
    if (elect_one()) umma_commit(&sm.drain[0]);
    __syncwarp();
    wait_own(&sm.drain[0], 0, p.err);
    __syncwarp();
  } else if (warp == kPvWarp) {
    // ------------------------------------------------------------------------ O += V^T P^T
    constexpr uint32_t kId = idesc_e4m3_f32(128, K::kNO, 1, 1);
    const uint64_t dv = smem_desc_sw128(smem_addr(sm.v[0]), kTileBytes, 1024);
    const uint64_t dp = smem_desc_mn(smem_addr(sm.p[0]), 128, 16 * kTile);
    auto wait_all = [&](uint64_t *bar, uint32_t parity) -> bool {
      return __all_sync(kFull, wait_parity(bar, parity, p.err));
    };
    uint32_t taken = 0, units = 0, t = 0;
    Ring vr;
    bool ok = true;
    while (ok) {
      const int slot = taken % kRing;
      if (!(ok = wait_all(&sm.unit_full[slot], (taken / kRing) & 1))) break;
      const int ntiles = sm.unit[slot].ntiles, skip = sm.unit[slot].skip;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.unit_empty[slot]);
      ++taken;
      if (ntiles < 0) break;
      if (skip) {
        if (!(ok = wait_all(&sm.v_full[vr.slot], vr.parity))) break;
        if (lane == 0) mbar_arrive(&sm.v_empty[vr.slot]);
        vr.next();
      }
      if (ntiles == 0) continue;
      const int ob = units & 1;
      // the unit before the last one's epilogue has read this accumulator
      if (units >= 2 && !(ok = wait_all(&sm.o_free[ob], ((units >> 1) - 1) & 1))) break;
      ++units;
      for (int it = 0; it < ntiles; ++it, ++t, vr.next()) {
        if (!(ok = wait_all(&sm.v_full[vr.slot], vr.parity))) break;
        if (!(ok = wait_all(&sm.p_full[t & 1], (t >> 1) & 1))) break;
        tc_fence_after_sync();
        if (elect_one()) {
          const uint64_t a = dv + vr.slot * (kTileBytes >> 4);
          const uint64_t b = dp + (t & 1) * (K::kNO * kTile >> 4);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk)  // 32 tokens: 32 rows of V, 32 bytes of P's rows
            umma_e4m3_ss(tmem + K::kOBase + ob * K::kNO, a + kk * (32 * 128 >> 4), b + 32 * kk, kId,
                         it > 0 || kk > 0);
          umma_commit(&sm.pv_done[t & 1]);
          umma_commit(&sm.v_empty[vr.slot]);
          if (it == ntiles - 1) umma_commit(&sm.o_full[ob]);
        }
        __syncwarp();
      }
    }
    if (elect_one()) umma_commit(&sm.drain[1]);
    __syncwarp();
    wait_own(&sm.drain[1], 0, p.err);
    __syncwarp();
  } else {
    // ------------------------------------------------------------------------ softmax
    // Threads i and i + 128: token i of every tile, lane i of tensor memory; in the epilogue
    // dimension i. Each has half of the heads, g0 .. g0 + GH - 1. Every decision to leave the loops
    // is taken by the softmax threads together, and a thread whose wait gave up (ok = false) still
    // takes part in the barriers of its unit.
    const int i = threadIdx.x & 127, half = warp >> 2, quad = warp & 3;
    const int g0 = half * GH;
    const uint32_t lanes = tmem + ((uint32_t)(quad * 32) << 16);
    uint32_t taken = 0, units = 0, t = 0;
    Ring vr;
    while (true) {
      const int slot = taken % kRing;
      const bool got = wait_parity(&sm.unit_full[slot], (taken / kRing) & 1, p.err);
      if (barrier_or(1, kSoftmaxThreads, !got)) break;
      const Unit8 un = sm.unit[slot];
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.unit_empty[slot]);
      ++taken;
      if (un.ntiles < 0) break;
      if (un.skip) vr.next();
      [[maybe_unused]] const int h = un.h;
      const int heads = min(GC, p.group - un.head0) - g0;  // of this thread (may be <= 0)
      const int tok_begin = un.s * p.chunk;
      const int64_t row0 = (int64_t)un.b * p.num_q_heads + h * p.group + un.head0 + g0;
      const int ub = units & 1;
      const uint32_t o_addr = lanes + K::kOBase + ub * K::kNO + half * K::kHalf;

      float nref[GH], l[GH], qsc[GH];  // nref: kTop - R
#pragma unroll
      for (int g = 0; g < GH; ++g) {
        nref[g] = INFINITY;
        l[g] = qsc[g] = 0.f;
      }
      bool ok = true;
      if (un.ntiles > 0) {
        ok = wait_parity(&sm.q_ready[ub], (units >> 1) & 1, p.err);
#pragma unroll
        for (int g = 0; g < GH; ++g) qsc[g] = sm.qscale[ub][g0 + g];
      }
      for (int it = 0; it < un.ntiles; ++it, ++t, vr.next()) {
        const int vs = vr.slot, buf = t & 1;
        const int n_valid = un.tokens - it * kTile;  // >= 1; < 128 only in a last tile
        const bool valid = i < n_valid;
        // (all lanes of a warp together: the loads of tensor memory are the warp's)
        ok = __all_sync(kFull, ok && wait_parity(&sm.s_full[buf], (t >> 1) & 1, p.err));
        float x[GH], inv_vs = 1.f;
        bool over = false;
        if (ok) {
          tc_fence_after_sync();
          uint32_t c[2 * GH];
          tmem_ld_cols(lanes + 16 * buf + 2 * g0, c);
          const int grp = (((tok_begin + it * kTile) & 255) >> 6) + (quad >> 1);
          const float ks = sm.tile_scale[vs][0][grp];
          // (a group past the context has no scale: whatever is there must not enter R or l)
          float ev = 0.f;
          if ((quad >> 1) * 64 < n_valid) {
            const float v_scale = fmaxf(sm.tile_scale[vs][1][grp], kMinScale);
            ev = log2_approx(v_scale);
            inv_vs = rcp_approx(v_scale);
          }
          float *const scores = p.scores + row0 * p.score_stride + tok_begin + it * kTile + i;
#pragma unroll
          for (int g = 0; g < GH; ++g) {
            if constexpr (GH == 1) {
              const float s = fmaf(__uint_as_float(c[1]), 1.f / 32.f, __uint_as_float(c[0])) *
                              (ks * qsc[0]);
              if (W && heads > 0) scores[0] = s;
              x[0] = valid ? s + ev : -INFINITY;
            } else if (g % 2 == 0) {
              const float2 sum = ffma2(
                  make_float2(__uint_as_float(c[GH + g]), __uint_as_float(c[GH + g + 1])),
                  make_float2(1.f / 32.f, 1.f / 32.f),
                  make_float2(__uint_as_float(c[g]), __uint_as_float(c[g + 1])));
              const float2 zero = make_float2(0.f, 0.f);
              const float2 sc = ffma2(make_float2(qsc[g], qsc[g + 1]), make_float2(ks, ks), zero);
              float2 y;
              if constexpr (W) {
                y = ffma2(sum, sc, zero);
                if (g < heads) scores[g * p.score_stride] = y.x;
                if (g + 1 < heads) scores[(g + 1) * p.score_stride] = y.y;
                y = fadd2(y, make_float2(ev, ev));
              } else {
                y = ffma2(sum, sc, make_float2(ev, ev));
              }
              x[g] = valid ? y.x : -INFINITY;
              x[g + 1] = valid ? y.y : -INFINITY;
            }
          }
#pragma unroll
          for (int g = 0; g < GH; ++g) over = over || x[g] + nref[g] > kTop + kHeadroom;
        }
        // a token above the reference (in the unit's first tile there is one): raise it
        if (it == 0 || barrier_or(2, kSoftmaxThreads, over)) {
#pragma unroll
          for (int g = 0; g < GH; ++g) {
            const float m = redux_max(ok ? x[g] : -INFINITY);
            if (lane == 0) sm.warp_max[warp][g] = m;
          }
          named_barrier_sync(3, kSoftmaxThreads);
          float alpha[GH];
#pragma unroll
          for (int g = 0; g < GH; ++g) {
            float m = -INFINITY;
#pragma unroll
            for (int w = 0; w < 4; ++w) m = fmaxf(m, sm.warp_max[4 * half + w][g]);
            m = fminf(nref[g], kTop - m);
            alpha[g] = m == INFINITY ? 1.f : fast_exp2(m - nref[g]);
            nref[g] = m;
            l[g] *= alpha[g];
          }
          if (it > 0) {  // O's columns t1 .. t4 of head g: wait for the PVs so far, scale
            ok = __all_sync(kFull, ok && wait_parity(&sm.pv_done[buf ^ 1], ((t - 1) >> 1) & 1, p.err));
            if (ok) {
              tc_fence_after_sync();
#pragma unroll
              for (int pair = 0; pair < kParts; pair += 2) {
                uint32_t o[2 * GH];
                tmem_ld_cols(o_addr + pair * GH, o);
#pragma unroll
                for (int c = 0; c < 2 * GH; ++c)
                  o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha[c % GH]);
                tmem_st_cols(o_addr + pair * GH, o);
              }
              tmem_st_wait();
            }
          }
        }
        if (ok) {
          float w[GH + 1];
          uint32_t code[kParts];
#pragma unroll
          for (int g = 0; g < GH; ++g) {
            if constexpr (GH == 1) {
              w[0] = fast_exp2(x[0] + nref[0]);  // (0 for a token past the context)
              l[0] = fmaf(w[0], inv_vs, l[0]);
            } else if (g % 2 == 0) {
              const float2 y = fadd2(make_float2(x[g], x[g + 1]), make_float2(nref[g], nref[g + 1]));
              w[g] = fast_exp2(y.x);
              w[g + 1] = fast_exp2(y.y);
              const float2 z = ffma2(make_float2(w[g], w[g + 1]), make_float2(inv_vs, inv_vs),
                                     make_float2(l[g], l[g + 1]));
              l[g] = z.x;
              l[g + 1] = z.y;
            }
          }
#pragma unroll
          for (int g = 0; g < GH; g += 2) {
            uint32_t part[kParts];
            split_weights(w[g], w[g + 1 < GH ? g + 1 : g], part);
#pragma unroll
            for (int j = 0; j < kParts; ++j)
              code[j] = g == 0 ? part[j] : __byte_perm(code[j], part[j], 0x5410);
          }
          // the token's row of P: 16 bytes of each group of 16 columns
          if constexpr (GH == 4)
            *reinterpret_cast<uint4 *>(sm.p[buf] + half * (16 * kTile) + i * 16) =
                make_uint4(code[0], code[1], code[2], code[3]);
          else if constexpr (GH == 2)
            *reinterpret_cast<uint2 *>(sm.p[buf] + i * 16 + half * 8) =
                make_uint2(__byte_perm(code[0], code[1], 0x5410), __byte_perm(code[2], code[3], 0x5410));
          else
            *reinterpret_cast<uint32_t *>(sm.p[buf] + i * 16 + half * 8) =
                __byte_perm(__byte_perm(code[0], code[1], 0x0040),
                            __byte_perm(code[2], code[3], 0x0040), 0x5410);
          if (!valid) {  // this token's V row is whatever the slot held: zero it (0 x NaN)
            uint4 *v = reinterpret_cast<uint4 *>(sm.v[vs] + i * 128 + half * 64);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = make_uint4(0, 0, 0, 0);
          }
          fence_async_shared();
          tc_fence_before_sync();
          __syncwarp();
          if (lane == 0) mbar_arrive(&sm.p_full[buf]);
        }
      }

      // ---- the unit's output: l over the 128 tokens, O from tensor memory
      if (un.ntiles > 0) {
#pragma unroll
        for (int g = 0; g < GH; ++g) {
#pragma unroll
          for (int o = 16; o > 0; o >>= 1) l[g] += __shfl_xor_sync(kFull, l[g], o);
          if (lane == 0) sm.warp_l[ub][warp][g] = l[g];
        }
        ok = __all_sync(kFull, ok && wait_parity(&sm.o_full[ub], (units >> 1) & 1, p.err));
        ++units;
      }
      if (barrier_or(1, kSoftmaxThreads, !ok)) break;  // a wait gave up: stop together
      float acc[GH];  // t1 + (t2 + (t3 + t4 / 32) / 32) / 32
      if (un.ntiles > 0) {
        tc_fence_after_sync();
        uint32_t o[2 * GH];
        tmem_ld_cols(o_addr + 2 * GH, o);
#pragma unroll
        for (int g = 0; g < GH; ++g)
          acc[g] = fmaf(__uint_as_float(o[GH + g]), 1.f / 32.f, __uint_as_float(o[g]));
        tmem_ld_cols(o_addr, o);
#pragma unroll
        for (int g = 0; g < GH; ++g)
          acc[g] = fmaf(fmaf(acc[g], 1.f / 32.f, __uint_as_float(o[GH + g])), 1.f / 32.f,
                        __uint_as_float(o[g]));
        tc_fence_before_sync();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.o_free[ub]);
      }
#pragma unroll
      for (int g = 0; g < GH; ++g) {
        float out = 0.f, lse = -INFINITY;
        if (un.ntiles > 0) {
          float sum = 0.f;
#pragma unroll
          for (int w = 0; w < 4; ++w) sum += sm.warp_l[ub][4 * half + w][g];
          // sum lies far inside the normal range (2^5 over a scale in [2^-100, 2^120], times the
          // tokens); the approximate division and log2 err far below one bf16 rounding
          out = __fdividef(acc[g], sum);
          lse = __log2f(sum) - nref[g];
        }
        if (W && i == 0 && !p.cluster) sm.lse[g0 + g] = lse;
        if (p.cluster) {  // merged by the cluster's rank 0 at the end
          cl_end = tok_begin + un.tokens;
          cl_o[g] = out;
          cl_lse[g] = lse;
        } else if (g < heads) {
          const int64_t row = row0 + g;
          if (un.whole) {
            // the unit holds the whole context: the output itself (the merge kernel skips it)
            p.out[row * kD + i] = bf16_bits_rn(out);
            if (W && i == 0 && !p.w_out) p.lse[row] = lse;
          } else {
            p.part_o[(row * p.splits + un.s) * kD + i] = out;
            if (i == 0) p.part_lse[row * p.splits + un.s] = lse;
          }
        }
      }
      if constexpr (W) {
        if (p.w_out && !p.cluster) {
          // (the scores are visible since the barrier above, the log2-sum-exps after this one)
          WeightsPass<GC> pass(p, un.b, h, tok_begin, tok_begin + un.tokens, threadIdx.x,
                               kSoftmaxThreads);
          named_barrier_sync(3, kSoftmaxThreads);
          pass.finish(sm.lse);
        }
      }
      if (!p.queue) break;  // a static grid gives each CTA one unit: nothing follows
    }
  }
  tc_fence_before_sync();
  __syncthreads();  // every load has landed, every UMMA is complete
  if (warp == kSWarp) tmem_dealloc(tmem, K::kTmemCols);
  if (!p.cluster) return;
  // ---------------------------------------------------------------- cluster merge
  // As in decode.cu: each peer sends its result into rank 0's landing area with asynchronous
  // stores counted on rank 0's barrier and leaves; rank 0 merges. (With more than kLandSplits
  // splits the area is rank 0's K slots, lent now that nothing uses them.) The waits ignore the
  // abort bit: every CTA reaches this point, rank 0 always lends and every peer always sends.
  cluster_wait();  // every CTA's barriers are set up
  if (threadIdx.x >= kSoftmaxThreads) return;
  const uint32_t rank = cluster_ctarank();
  const bool lend = p.cluster > K::kLandSplits;
  float *land_o = lend ? reinterpret_cast<float *>(sm.k[0])  // peer r + 1's outputs at [r][g][d]
                       : reinterpret_cast<float *>(reinterpret_cast<uint8_t *>(&sm) +
                                                   land_offset<GC>());
  float *land_lse = land_o + (size_t)(p.cluster - 1) * GC * kD;
  const int d = threadIdx.x & 127, g0 = (threadIdx.x >> 7) * GH;
  // With weights: this CTA's share of them (its scores are visible to all its threads since the
  // barrier above).
  std::conditional_t<W, WeightsPass<GC>, NoWeights> pass(
      p, (blockIdx.x / p.splits) / p.xgroups, (blockIdx.x / p.splits) % p.xgroups,
      (int)rank * p.chunk, p.w_out ? cl_end : 0, threadIdx.x, kSoftmaxThreads);
  if (rank != 0) {
    if (lend && !wait_own(&sm.cl_ready, 0, p.err)) return;
    const uint32_t bar = cluster_addr(smem_addr(&sm.cl_bar), 0);
    if (threadIdx.x == 0) mbar_arrive_expect_tx_remote(bar, GC * (kD + 1) * sizeof(float));
    const int r = (int)rank - 1;
#pragma unroll
    for (int g = 0; g < GH; ++g) {
      const int at = r * GC + g0 + g;
      st_async_f32(cluster_addr(smem_addr(land_o + (size_t)at * kD + d), 0), cl_o[g], bar);
      if (d == 0) st_async_f32(cluster_addr(smem_addr(land_lse + at), 0), cl_lse[g], bar);
    }
    if constexpr (W) {
      if (p.w_out) {  // the weights of this split, once rank 0 has merged the log2-sum-exps
        if (threadIdx.x == 0) mbar_arrive_expect_tx(&sm.cl_lse, GC * sizeof(float));
        if (wait_own(&sm.cl_lse, 0, p.err)) {
          pass.finish(sm.lse);
        } else {  // no answer: stay until no other CTA can write here any more
          cluster_arrive_relaxed();
          cluster_wait();
        }
      }
    }
    return;
  }
  if (lend && threadIdx.x == 0)
    for (int r = 1; r < p.cluster; ++r)
      mbar_arrive_remote(cluster_addr(smem_addr(&sm.cl_ready), r));
  if (!wait_own(&sm.cl_bar, 0, p.err)) return;
  const int unit0 = blockIdx.x;  // rank 0 holds split 0
  const int b = (unit0 / p.splits) / p.xgroups, xg = (unit0 / p.splits) % p.xgroups;
  const int h = xg / p.head_groups, hg = xg % p.head_groups;
#pragma unroll
  for (int g = 0; g < GH; ++g) {
    float M = cl_lse[g];
    for (int r = 0; r < p.cluster - 1; ++r) M = fmaxf(M, land_lse[r * GC + g0 + g]);
    if (M == -INFINITY) M = 0.f;  // no keys, or NaN scores only
    float wsum = fast_exp2(cl_lse[g] - M);  // 0 for a split with no keys, NaN for one with a NaN
    float acc = wsum * cl_o[g];
    for (int r = 0; r < p.cluster - 1; ++r) {
      const float wgt = fast_exp2(land_lse[r * GC + g0 + g] - M);
      wsum += wgt;
      acc = fmaf(wgt, land_o[((size_t)r * GC + g0 + g) * kD + d], acc);
    }
    const int in_group = hg * GC + g0 + g;
    const int64_t row = (int64_t)b * p.num_q_heads + h * p.group + in_group;
    if (!sm.stop && in_group < p.group) {
      p.out[row * kD + d] = bf16_bits_rn(wsum == 0.f ? 0.f : acc / wsum);
      if (W && d == 0 && !p.w_out) p.lse[row] = M + __log2f(wsum);
    }
    if (W && d == 0 && p.w_out) {
      const float lse = M + __log2f(wsum);
      sm.lse[g0 + g] = lse;
      for (int r = 1; r < p.cluster; ++r)
        st_async_f32(cluster_addr(smem_addr(&sm.lse[g0 + g]), r), lse,
                     cluster_addr(smem_addr(&sm.cl_lse), r));
    }
  }
  if constexpr (W) {
    if (p.w_out) {
      named_barrier_sync(3, kSoftmaxThreads);
      pass.finish(sm.lse);
    }
  }
}

template <int GC, bool W>
cudaError_t launch_split_fp8(const CUtensorMap (&km)[3], const CUtensorMap (&vm)[3],
                             const DecodeParams &prm, int num_sms, cudaStream_t stream) {
  static bool configured[64] = {};
  int dev = 0;
  cudaGetDevice(&dev);
  if (dev >= 64 || !configured[dev]) {
    cudaError_t e = cudaFuncSetAttribute(decode_fp8_kernel<GC, W>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)fp8_smem_bytes<GC>(Kind<GC>::kLandSplits));
    if (e != cudaSuccess) return e;
    // all of the unified L1/shared storage as shared memory, so two CTAs fit on an SM
    e = cudaFuncSetAttribute(decode_fp8_kernel<GC, W>,
                             cudaFuncAttributePreferredSharedMemoryCarveout,
                             cudaSharedmemCarveoutMaxShared);
    if (e != cudaSuccess) return e;
    if (dev < 64) configured[dev] = true;
  }
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)std::min<int64_t>((int64_t)num_sms * 2, prm.units));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = fp8_smem_bytes<GC>(prm.cluster);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (prm.cluster) {  // one CTA per unit, the splits of a (sequence, head group) in a cluster
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)prm.cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
  }
  return cudaLaunchKernelEx(&cfg, decode_fp8_kernel<GC, W>, km[0], vm[0], km[1], vm[1], km[2], vm[2],
                            prm);
}

}  // namespace

cudaError_t launch_paged_decode_fp8(const DecodeArgs &a, const DecodePlan &p,
                                    cudaStream_t stream) {
  // TMA views of the two pools: {128 dims, num_blocks * block_size rows, Hkv heads} of bytes, a
  // box per tile, and smaller boxes for a context's last tile
  CUtensorMap km[3], vm[3];
  const uint64_t rows = (uint64_t)a.num_blocks * a.block_size;
  const uint64_t dims[3] = {kD, rows, (uint64_t)a.num_kv_heads};
  const uint64_t strides[2] = {(uint64_t)a.num_kv_heads * kD, kD};
  const uint32_t box_rows[3] = {kTile, kBoxRows, kSmallBoxRows};
  auto encode = [&](CUtensorMap *map, const void *pool, uint32_t rows_in_box) {
    const uint32_t box[3] = {kD, rows_in_box, 1};
    return encode_tensor_map(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(pool), dims,
                             strides, box, CU_TENSOR_MAP_SWIZZLE_128B,
                             CU_TENSOR_MAP_L2_PROMOTION_L2_256B) == CUDA_SUCCESS;
  };
  for (int i = 0; i < 3; ++i)
    if (!encode(&km[i], a.k_cache, box_rows[i]) || !encode(&vm[i], a.v_cache, box_rows[i]))
      return cudaErrorInvalidValue;
  DecodeParams prm = decode_params(a, p);
  const int64_t units = (int64_t)p.splits * a.batch * prm.xgroups;
  // the work counter runs to units + grid size - 1 (an int): keep that in range
  if (units + 2 * (int64_t)a.num_sms > INT32_MAX) return cudaErrorInvalidValue;
  prm.units = (int32_t)units;
  // as for the bf16 cache: with no more units than CTAs each CTA takes one and the splits of a
  // (sequence, head group) meet in a cluster; else the queue, and a merge kernel
  const bool queued = decode_queued(a, p);
  if (!queued) prm.queue = nullptr;
  prm.cluster = !queued && p.splits >= 2 && p.splits <= p.max_cluster ? p.splits : 0;
  const bool w = p.scores_at != 0;
  auto split = [&](auto launch) { return launch(km, vm, prm, a.num_sms, stream); };
  const cudaError_t e =
      p.heads_per_cta == 8   ? split(w ? launch_split_fp8<8, true> : launch_split_fp8<8, false>)
      : p.heads_per_cta == 4 ? split(w ? launch_split_fp8<4, true> : launch_split_fp8<4, false>)
                             : split(w ? launch_split_fp8<2, true> : launch_split_fp8<2, false>);
  if (e != cudaSuccess || p.splits == 1 || prm.cluster) return e;
  return launch_combine<true>(a, p, prm, stream);
}

}  // namespace pkv

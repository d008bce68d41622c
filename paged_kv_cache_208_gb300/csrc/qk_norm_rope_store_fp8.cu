// qk_norm_rope_store_fp8.cu -- RMSNorm and rotary embedding of the query and key heads of new
// tokens on their way into the 8-bit cache (the format is in fp8_cache.cuh).
//
// «nano-vLLM 最小化vLLM重新实现», 架构 6 模型: QK 归一化, then RoPE from a precomputed cos/sin
// cache; 架构 5: K and V written into the paged cache. A projection row holds Hq query heads, Hkv
// key heads and Hkv value heads of 128 values. For a query or key head x with weight w, in fp32:
//     n = x * rsqrt(mean(x^2) + eps) * w       (without weights: n = x)
//     y_i = n_i c_i - n_{i+64} s_i,  y_{i+64} = n_{i+64} c_i + n_i s_i,  i < 64
// Nothing is rounded before y, which is rounded once: queries to bf16, keys to e4m3 at the scale
// of their group. (pkv_qk_norm_rope_store rounds n and a key's y to bf16, as the model's layers do
// between them; here a key has 4 significant bits left, and a second rounding before those
// would only add to the error of the first.)
//
// Bound by HBM: a row is read once, 2 bytes a value, and written once. As in kv_store_fp8 a CTA
// owns the K or V heads it takes of a run (the new rows of one sequence that lie in one group of 64
// positions), so that nothing else touches their scales; it goes through them a head at a time, the
// next one's rows on their way. Four lanes hold a head's row, each the 16 + 16 values that turn
// into one another, in 32-byte loads. Another CTA takes the run's query heads, a warp to a token,
// eight heads at a time: what it reads and writes is contiguous, and the lanes of different heads
// read the same cosines and weights at once.
// 132k tokens of 16 + 2 x 8 heads take 329 us (6.0 TB/s): 460 us with eight lanes to a row and a
// quarter of a head's 64 rows in each thread, 357 us with half of them and the next head loaded
// ahead, 350 us with two values to an instruction, 344 us with the queries by tokens. Three CTAs of
// 80 registers (12 bytes of them spilled) fit an SM; two of 128 take 348 us, four of 64 spill more and take
// 378 us. A few drafted tokens behind a context are where it is far from its bytes: 256 sequences of 5 to 8 take
// 26 us (4.3 us of bytes), 45 us where every scale grows, since a CTA's heads follow one another, each with a
// barrier and an old scale to load.
//
// A step of one token per sequence takes half a warp per head row: 8 tokens 2.6 us, the latency
// of a launch and of three loads that depend on one another; 14 us where a group's scale grows (256 tokens:
// 4.1 and 19 us), since the half warp then re-rounds the up to 63 rows from before one after the other.
#include <math.h>

#include <algorithm>

#include "device_common.cuh"
#include "fp8_cache.cuh"
#include "launch.h"
#include "pkv.h"

namespace pkv {
namespace {

constexpr int kD = 128;
constexpr unsigned kFull = 0xffffffffu;

struct AppendParams {
  const uint8_t *qkv;
  int64_t tok_stride;  // bytes
  int64_t num_tokens;
  const int64_t *positions;
  const uint8_t *q_weight, *k_weight;  // nullptr: no norm
  float eps;
  const float *cos_sin;
  int64_t max_position;
  const int32_t *cu;  // nullptr: one token per sequence
  const int32_t *context_lens;
  const int32_t *block_tables;
  int32_t table_width, num_seqs;
  uint8_t *q_out;
  uint8_t *k_cache, *v_cache;
  float *k_scale, *v_scale;
  int32_t hq, hkv, block_size;
  int64_t num_blocks;
  bool wide;  // rows and q_out lie at multiples of 32 bytes
  unsigned int *err;
};

// Two fp32 values in a 64-bit register: one instruction then works on both.
__device__ __forceinline__ uint64_t pair_of(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 unpair(uint64_t x) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(x));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t x, uint64_t y) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(x), "l"(y));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t x, uint64_t y, uint64_t z) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(x), "l"(y), "l"(z));
  return r;
}
// 32 bytes that are read once; `wide`: the address is a multiple of 32, not only of 16
__device__ __forceinline__ void ld_once_32b(const uint8_t *p, uint32_t (&w)[8], bool wide) {
  if (wide) {
    asm volatile(
        "ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
        : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]),
          "=r"(w[7])
        : "l"(p)
        : "memory");
  } else {
    const uint4 x = ld_once_u4(reinterpret_cast<const uint4 *>(p));
    const uint4 y = ld_once_u4(reinterpret_cast<const uint4 *>(p) + 1);
    w[0] = x.x, w[1] = x.y, w[2] = x.z, w[3] = x.w, w[4] = y.x, w[5] = y.y, w[6] = y.z, w[7] = y.w;
  }
}

// 2 N values, a pair to a register pair
template <int N>
struct Pairs {
  uint64_t v[N];
};
template <int N>
__device__ __forceinline__ Pairs<N> widen(const uint32_t (&w)[N]) {
  Pairs<N> r;
#pragma unroll
  for (int k = 0; k < N; ++k) r.v[k] = pair_of(bf16_lo(w[k]), bf16_hi(w[k]));
  return r;
}
template <int N>
__device__ __forceinline__ void round_to_bf16(const Pairs<N> &x, uint32_t (&w)[N]) {
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const float2 f = unpair(x.v[k]);
    w[k] = pack_bf16x2(f.x, f.y);
  }
}
// codes of four values
__device__ __forceinline__ uint32_t quantize4(uint64_t x, uint64_t y, uint64_t inv) {
  const float2 f = unpair(mul2(x, inv)), g = unpair(mul2(y, inv));
  return cvt_e4m3x2(f.x, f.y) | cvt_e4m3x2(g.x, g.y) << 16;
}
// Largest finite |x|, as fp32 bits. fmaxf passes over NaN; an infinity is rare and sends the values
// through again.
template <int N>
__device__ __noinline__ float finite_max_again(const Pairs<N> x) {
  float m = 0.f;
  for (int k = 0; k < N; ++k) {
    const float2 f = unpair(x.v[k]);
    if (fabsf(f.x) < INFINITY) m = fmaxf(m, fabsf(f.x));
    if (fabsf(f.y) < INFINITY) m = fmaxf(m, fabsf(f.y));
  }
  return m;
}
template <int N>
__device__ __forceinline__ float finite_max(const Pairs<N> &x) {
  float m = 0.f;
#pragma unroll
  for (int k = 0; k < N; ++k) {
    const float2 f = unpair(x.v[k]);
    m = fmaxf(m, fmaxf(fabsf(f.x), fabsf(f.y)));
  }
  return m < INFINITY ? m : finite_max_again(x);
}
// The scale for a group whose largest finite |x| has the fp32 bits `amax`: fp8_scale_exp's rule
// with fp32's mantissa.
__device__ __forceinline__ float scale_of(uint32_t amax) {
  const int e = (int)(amax >> 23) - 135 + ((amax & 0x7fffffu) > 0x600000u ? 1 : 0);
  return pow2f(max(e, kFp8MinExp));
}
template <int N>
__device__ __forceinline__ float square_sum(const Pairs<N> &x, uint64_t s = 0) {  // (0.f, 0.f)
#pragma unroll
  for (int k = 0; k < N; ++k) s = fma2(x.v[k], x.v[k], s);
  const float2 f = unpair(s);
  return f.x + f.y;
}

// A quarter of a head's row: the values [16 i, +16) and [64 + 16 i, +16).
struct Quarter {
  Pairs<8> a, b;
};
// n of them, the four lanes of a row together
__device__ __forceinline__ void normalise(const uint8_t *weight, float eps, int i, Quarter &x) {
  float ss = square_sum(x.a) + square_sum(x.b);
  ss += __shfl_xor_sync(kFull, ss, 1);
  ss += __shfl_xor_sync(kFull, ss, 2);
  const float rs = rsqrtf(ss * (1.f / kD) + eps);
  const uint64_t rs2 = pair_of(rs, rs);
#pragma unroll
  for (int k = 0; k < 8; k += 4) {
    const uint4 u = *reinterpret_cast<const uint4 *>(weight + 32 * i + 4 * k);
    const uint4 v = *reinterpret_cast<const uint4 *>(weight + kD + 32 * i + 4 * k);
    const Pairs<4> wa = widen<4>({u.x, u.y, u.z, u.w}), wb = widen<4>({v.x, v.y, v.z, v.w});
#pragma unroll
    for (int d = 0; d < 4; ++d) {
      x.a.v[k + d] = mul2(mul2(x.a.v[k + d], rs2), wa.v[d]);
      x.b.v[k + d] = mul2(mul2(x.b.v[k + d], rs2), wb.v[d]);
    }
  }
}
// y of them, the position's row of the cos/sin cache being `cs`
__device__ __forceinline__ void rotate(const float *cs, int i, Quarter &x) {
#pragma unroll
  for (int k = 0; k < 8; k += 2) {
    const float4 c = *reinterpret_cast<const float4 *>(cs + 16 * i + 2 * k);
    const float4 s = *reinterpret_cast<const float4 *>(cs + kD / 2 + 16 * i + 2 * k);
    const uint64_t cc[2] = {pair_of(c.x, c.y), pair_of(c.z, c.w)};
    const uint64_t sn[2] = {pair_of(s.x, s.y), pair_of(s.z, s.w)};
    const uint64_t minus[2] = {pair_of(-s.x, -s.y), pair_of(-s.z, -s.w)};
#pragma unroll
    for (int d = 0; d < 2; ++d) {
      const uint64_t a = x.a.v[k + d], b = x.b.v[k + d];
      x.a.v[k + d] = fma2(a, cc[d], mul2(b, minus[d]));
      x.b.v[k + d] = fma2(b, cc[d], mul2(a, sn[d]));
    }
  }
}

constexpr int kRunThreads = 256;
constexpr int kRunWarps = kRunThreads / 32;
static_assert(kRunThreads == 4 * kFp8Group);

// The query heads of rows t0 .. t0 + rows - 1, a warp to a row at a time, which lies contiguous in
// memory, and four lanes to a head.
__device__ __forceinline__ void append_queries(const AppendParams &p, int64_t t0, int rows, int warp,
                                               int lane) {
  const int i4 = lane & 3;
  for (int r = warp; r < rows; r += kRunWarps) {
    const int64_t t = t0 + r, pos = *(p.positions + t);
    const uint8_t *const src = p.qkv + t * p.tok_stride + 32 * i4;
    uint8_t *const dst = p.q_out + t * p.hq * (2 * kD) + 32 * i4;
    if (pos < 0 || pos >= p.max_position) {
      if (lane == 0) record_error(p.err, PKV_DEVERR_POSITION_RANGE);
      continue;
    }
#pragma unroll 1
    for (int g = 0; g < p.hq; g += 8) {
      const int h = g + (lane >> 2);
      uint32_t w[2][8];
      const uint8_t *const from = src + min(h, p.hq - 1) * (2 * kD);
      ld_once_32b(from, w[0], p.wide);
      ld_once_32b(from + kD, w[1], p.wide);
      Quarter x{widen(w[0]), widen(w[1])};
      if (p.q_weight) normalise(p.q_weight, p.eps, i4, x);
      rotate(p.cos_sin + pos * kD, i4, x);
      if (h >= p.hq) continue;
      round_to_bf16(x.a, w[0]);
      round_to_bf16(x.b, w[1]);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        uint8_t *const d = dst + h * (2 * kD) + e * kD;
        if (p.wide) {
          st_global_32b(d, w[e]);
        } else {
          reinterpret_cast<uint4 *>(d)[0] = make_uint4(w[e][0], w[e][1], w[e][2], w[e][3]);
          reinterpret_cast<uint4 *>(d)[1] = make_uint4(w[e][4], w[e][5], w[e][6], w[e][7]);
        }
      }
    }
  }
}

// The CTAs of a run: one for its query heads, the others for parts of its key and value heads.
__global__ void __launch_bounds__(kRunThreads, 3)
    append_run_kernel(const AppendParams p, int heads_per_cta) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ uint32_t warp_max[2][kRunWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int heads = p.hq + 2 * p.hkv;  // of a projection row: queries, keys, values
  const int parts = 1 + (2 * p.hkv + heads_per_cta - 1) / heads_per_cta;
  const int64_t r = blockIdx.x / parts;
  const int part = (int)(blockIdx.x % parts);
  const int h0 = p.hq + (part - 1) * heads_per_cta, h1 = min(heads, h0 + heads_per_cta);
  const bool turned = h0 < p.hq + p.hkv;  // it has key heads
  const int n = find_sequence(p.cu, p.num_seqs, r, lane);
  const int64_t c0 = *(p.cu + n), c1 = *(p.cu + n + 1), ctx = *(p.context_lens + n);
  const int64_t j = r - run_base((int32_t)c0, n);
  const int64_t capacity = (int64_t)p.table_width * p.block_size;
  if (blockIdx.x == 0) {  // the batch's lengths, looked over once
    for (int i = tid; i < p.num_seqs; i += kRunThreads) {
      const int64_t a = *(p.cu + i), e = *(p.cu + i + 1), len = *(p.context_lens + i);
      if (a < 0 || e < a || e > p.num_tokens || len < e - a) record_error(p.err, PKV_DEVERR_SEQLEN_RANGE);
      else if (len > capacity) record_error(p.err, PKV_DEVERR_CONTEXT_RANGE);
    }
  }
  if (c0 < 0 || c1 < c0 || c1 > p.num_tokens || ctx < c1 - c0 || ctx > capacity) return;
  const int64_t start = ctx - (c1 - c0);                // first new position
  const int64_t group = start / kFp8Group + j;          // group index in the sequence
  const int64_t begin = max(start, group * kFp8Group);
  const int64_t end = min(ctx, (group + 1) * kFp8Group);
  if (j < 0 || begin >= end) return;
  const int rows = (int)(end - begin);
  if (part == 0) {
    if (!aborted(p.err)) append_queries(p, c0 + begin - start, rows, warp, lane);
    return;
  }
  const int i4 = tid & 3, row0 = tid >> 2;
  const bool here = row0 < rows;
  const int64_t tok = c0 + begin - start + row0;
  const uint8_t *const src = p.qkv + tok * p.tok_stride + 32 * i4;
  uint32_t next[2][8] = {};
  if (here) {
    ld_once_32b(src + h0 * (2 * kD), next[0], p.wide);
    ld_once_32b(src + h0 * (2 * kD) + kD, next[1], p.wide);
  }
  const float *cs = nullptr;  // of this thread's row; nullptr: past the run, or a bad position
  if (turned && here) {
    const int64_t pos = *(p.positions + tok);
    if (pos >= 0 && pos < p.max_position) cs = p.cos_sin + pos * kD;
    else if (i4 == 0) record_error(p.err, PKV_DEVERR_POSITION_RANGE);
  }
  const int64_t blk = *(p.block_tables + (int64_t)n * p.table_width + begin / p.block_size);
  const bool blk_ok = blk >= 0 && blk < p.num_blocks;
  if (!blk_ok && tid == 0) record_error(p.err, PKV_DEVERR_BLOCK_RANGE);
  // an earlier wait gave up somewhere: write nothing (decided by the CTA together)
  if (__syncthreads_or(tid == 0 && aborted(p.err)) || !blk_ok) return;
  const int in_block = (int)(begin % p.block_size);
  const int before = in_block % kFp8Group;  // rows of the group from before the call
  const int64_t rstride = (int64_t)p.hkv * kD;
  const int64_t dst0 = (blk * p.block_size + in_block) * rstride;
  int buf = 0;
#pragma unroll 1
  for (int row = h0; row < h1; ++row) {
    const bool is_v = row >= p.hq + p.hkv;
    const int h = row - p.hq - (is_v ? p.hkv : 0);
    Quarter x{widen(next[0]), widen(next[1])};
    if (here && row + 1 < h1) {  // in flight while this head is worked on
      ld_once_32b(src + (row + 1) * (2 * kD), next[0], p.wide);
      ld_once_32b(src + (row + 1) * (2 * kD) + kD, next[1], p.wide);
    }
    if (!is_v) {
      if (p.k_weight) normalise(p.k_weight, p.eps, i4, x);
      if (cs) rotate(cs, i4, x);
    }
    const bool good = is_v ? here : cs != nullptr;
    float *const scales = is_v ? p.v_scale : p.k_scale;
    uint32_t m = __reduce_max_sync(
        kFull, good ? __float_as_uint(fmaxf(finite_max(x.a), finite_max(x.b))) : 0u);
    if (lane == 0) warp_max[buf][warp] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kRunWarps; ++w) m = max(m, warp_max[buf][w]);
    buf ^= 1;  // (the next use of this half is a barrier away)
    const int64_t sc = (blk * p.hkv + h) * (p.block_size / kFp8Group) + in_block / kFp8Group;
    float scale = scale_of(m);
    uint8_t *dst = (is_v ? p.v_cache : p.k_cache) + dst0 + h * kD;
    if (before) {
      const float old = scales[sc];
      scale = fmaxf(scale, old);
      if (scale > old) {  // the rows from before, at the scale that grew
        const float ratio = old / scale;
        for (int i = tid; i < before * 8; i += kRunThreads) {
          uint4 *q = reinterpret_cast<uint4 *>(dst - (int64_t)(before - i / 8) * rstride + (i % 8) * 16);
          uint4 w = *q;
          w.x = rescale4(w.x, ratio);
          w.y = rescale4(w.y, ratio);
          w.z = rescale4(w.z, ratio);
          w.w = rescale4(w.w, ratio);
          *q = w;
        }
      }
      __syncthreads();  // every thread has read the old scale
    }
    if (tid == 0) scales[sc] = scale;
    const uint64_t inv = pair_of(1.f / scale, 1.f / scale);
    if (good) {
      uint4 *const d = reinterpret_cast<uint4 *>(dst + row0 * rstride + 16 * i4);
      uint32_t q[2][4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        q[0][k] = quantize4(x.a.v[2 * k], x.a.v[2 * k + 1], inv);
        q[1][k] = quantize4(x.b.v[2 * k], x.b.v[2 * k + 1], inv);
      }
      d[0] = make_uint4(q[0][0], q[0][1], q[0][2], q[0][3]);
      d[kD / 32] = make_uint4(q[1][0], q[1][1], q[1][2], q[1][3]);
    }
  }
}

// Half a warp: one head row of a sequence's new token. Lane i of it holds the values [8 i, +8).
constexpr int kTokenWarps = 4;
__global__ void __launch_bounds__(kTokenWarps * 32) append_token_kernel(const AppendParams p) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int lane = threadIdx.x & 31, i = lane & 15;
  const int heads = p.hq + 2 * p.hkv;
  const int64_t unit = ((int64_t)blockIdx.x * kTokenWarps * 32 + threadIdx.x) >> 4;
  const bool any = unit < (int64_t)p.num_seqs * heads;
  const int n = any ? (int)(unit / heads) : 0, row = any ? (int)(unit % heads) : 0;
  const int kind = row < p.hq ? 0 : row < p.hq + p.hkv ? 1 : 2;
  const int h = row - (kind == 0 ? 0 : kind == 1 ? p.hq : p.hq + p.hkv);
  auto eight = [](const uint4 w) { return widen<4>({w.x, w.y, w.z, w.w}); };
  Pairs<4> x = eight(
      ld_once_u4(reinterpret_cast<const uint4 *>(p.qkv + n * p.tok_stride + row * (2 * kD) + 16 * i)));
  const int64_t pos = *(p.positions + n), ctx = *(p.context_lens + n);
  const bool pos_ok = pos >= 0 && pos < p.max_position;
  const bool stop = __any_sync(kFull, aborted(p.err));
  if (any && i == 0 && row == 0 && !pos_ok) record_error(p.err, PKV_DEVERR_POSITION_RANGE);
  if (kind < 2) {
    const uint8_t *weight = kind == 0 ? p.q_weight : p.k_weight;
    float ss = square_sum(x);
#pragma unroll
    for (int o = 1; o < 16; o <<= 1) ss += __shfl_xor_sync(0xffffu << (lane & 16), ss, o);
    if (weight) {
      const float rs = rsqrtf(ss * (1.f / kD) + p.eps);
      const Pairs<4> w = eight(*reinterpret_cast<const uint4 *>(weight + 16 * i));
#pragma unroll
      for (int k = 0; k < 4; ++k) x.v[k] = mul2(mul2(x.v[k], pair_of(rs, rs)), w.v[k]);
    }
    Pairs<4> y;
#pragma unroll
    for (int k = 0; k < 4; ++k) y.v[k] = __shfl_xor_sync(0xffffu << (lane & 16), x.v[k], 8);
    if (pos_ok) {
      const float *cs = p.cos_sin + pos * kD + 8 * (i & 7);
      const float sign = i < 8 ? -1.f : 1.f;
#pragma unroll
      for (int k = 0; k < 4; k += 2) {
        const float4 c = *reinterpret_cast<const float4 *>(cs + 2 * k);
        const float4 s = *reinterpret_cast<const float4 *>(cs + kD / 2 + 2 * k);
        x.v[k] = fma2(x.v[k], pair_of(c.x, c.y), mul2(y.v[k], pair_of(sign * s.x, sign * s.y)));
        x.v[k + 1] =
            fma2(x.v[k + 1], pair_of(c.z, c.w), mul2(y.v[k + 1], pair_of(sign * s.z, sign * s.w)));
      }
    }
  }
  if (!any || stop || (kind < 2 && !pos_ok)) return;
  if (kind == 0) {
    uint32_t w[4];
    round_to_bf16(x, w);
    *reinterpret_cast<uint4 *>(p.q_out + ((int64_t)n * p.hq + h) * (2 * kD) + 16 * i) =
        make_uint4(w[0], w[1], w[2], w[3]);
    return;
  }
  if (ctx == 0) return;  // a padding row
  const bool tell = i == 0 && row == p.hq;
  if (ctx < 0 || ctx > (int64_t)p.table_width * p.block_size) {
    if (tell) record_error(p.err, PKV_DEVERR_CONTEXT_RANGE);
    return;
  }
  const int64_t blk = *(p.block_tables + (int64_t)n * p.table_width + (ctx - 1) / p.block_size);
  if (blk < 0 || blk >= p.num_blocks) {
    if (tell) record_error(p.err, PKV_DEVERR_BLOCK_RANGE);
    return;
  }
  const int in_block = (int)((ctx - 1) % p.block_size);
  const int before = in_block % kFp8Group;
  const int64_t sc = (blk * p.hkv + h) * (p.block_size / kFp8Group) + in_block / kFp8Group;
  float *scales = kind == 2 ? p.v_scale : p.k_scale;
  const float old = before ? scales[sc] : 0.f;
  uint32_t m = __float_as_uint(finite_max(x));
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) m = max(m, __shfl_xor_sync(0xffffu << (lane & 16), m, o));
  const float scale = fmaxf(scale_of(m), old);
  const int64_t rstride = (int64_t)p.hkv * kD;
  uint8_t *dst = (kind == 2 ? p.v_cache : p.k_cache) + (blk * p.block_size + in_block) * rstride +
                 h * kD + i * 8;
  if (before && scale > old) {
    const float ratio = old / scale;
#pragma unroll 4
    for (int t = 1; t <= before; ++t) {
      uint2 *q = reinterpret_cast<uint2 *>(dst - t * rstride);
      const uint2 w = *q;
      *q = make_uint2(rescale4(w.x, ratio), rescale4(w.y, ratio));
    }
  }
  const uint64_t inv = pair_of(1.f / scale, 1.f / scale);
  *reinterpret_cast<uint2 *>(dst) =
      make_uint2(quantize4(x.v[0], x.v[1], inv), quantize4(x.v[2], x.v[3], inv));
  if (i == 0) scales[sc] = scale;
}

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace
}  // namespace pkv

extern "C" pkv_status pkv_qk_norm_rope_store_fp8(
    const void *qkv, int64_t qkv_tok_stride, int64_t num_tokens, const int64_t *positions,
    const void *q_norm_weight, const void *k_norm_weight, float eps, const float *cos_sin_cache,
    int64_t max_position, const int32_t *cu_seqlens, const int32_t *context_lens,
    const int32_t *block_tables, int32_t block_table_width, int32_t num_seqs, void *q_out,
    void *k_cache, void *v_cache, float *k_scale, float *v_scale, int32_t num_q_heads,
    int32_t num_kv_heads, int32_t head_dim, int32_t block_size, int64_t num_blocks, void *stream) {
  using namespace pkv;
  if (num_seqs < 0 || num_tokens < 0 || num_q_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 ||
      block_size <= 0 || num_blocks <= 0 || block_table_width <= 0 || max_position <= 0 ||
      !(eps >= 0.f) || !isfinite(eps))
    return PKV_ERR_INVALID_ARG;
  const int64_t heads = (int64_t)num_q_heads + 2 * (int64_t)num_kv_heads;
  if (qkv_tok_stride < heads * head_dim) return PKV_ERR_INVALID_ARG;
  if (!cu_seqlens && num_tokens != num_seqs) return PKV_ERR_INVALID_ARG;
  if (!q_norm_weight != !k_norm_weight) return PKV_ERR_INVALID_ARG;
  if (num_seqs == 0 || num_tokens == 0) return PKV_OK;
  if (!qkv || !positions || !cos_sin_cache || !context_lens || !block_tables || !q_out ||
      !k_cache || !v_cache || !k_scale || !v_scale)
    return PKV_ERR_INVALID_ARG;
  if (head_dim != kD || block_size % 256 != 0 || num_tokens > INT32_MAX || heads > (1 << 20))
    return PKV_ERR_UNSUPPORTED;
  if (qkv_tok_stride % 8 != 0 || !aligned16(qkv) || !aligned16(q_norm_weight) ||
      !aligned16(k_norm_weight) || !aligned16(cos_sin_cache) || !aligned16(q_out) ||
      !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(k_scale) || !aligned16(v_scale))
    return PKV_ERR_UNSUPPORTED;
  if (overlap(qkv, num_tokens, 2 * (__int128)qkv_tok_stride, 2 * heads * head_dim, q_out,
              2 * num_tokens * num_q_heads * head_dim))
    return PKV_ERR_INVALID_ARG;
  const int num_sms = current_sm_count();
  unsigned int *err = current_error_word();
  if (num_sms <= 0 || !err) return PKV_ERR_CUDA;
  AppendParams prm{};
  prm.qkv = static_cast<const uint8_t *>(qkv);
  prm.tok_stride = qkv_tok_stride * 2;
  prm.num_tokens = num_tokens;
  prm.positions = positions;
  prm.q_weight = static_cast<const uint8_t *>(q_norm_weight);
  prm.k_weight = static_cast<const uint8_t *>(k_norm_weight);
  prm.eps = eps;
  prm.cos_sin = cos_sin_cache;
  prm.max_position = max_position;
  prm.cu = cu_seqlens;
  prm.context_lens = context_lens;
  prm.block_tables = block_tables;
  prm.table_width = block_table_width;
  prm.num_seqs = num_seqs;
  prm.q_out = static_cast<uint8_t *>(q_out);
  prm.k_cache = static_cast<uint8_t *>(k_cache);
  prm.v_cache = static_cast<uint8_t *>(v_cache);
  prm.k_scale = k_scale;
  prm.v_scale = v_scale;
  prm.hq = num_q_heads;
  prm.hkv = num_kv_heads;
  prm.block_size = block_size;
  prm.num_blocks = num_blocks;
  prm.wide = qkv_tok_stride % 16 == 0 &&
             ((reinterpret_cast<uintptr_t>(qkv) | reinterpret_cast<uintptr_t>(q_out)) & 31u) == 0;
  prm.err = err;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (!cu_seqlens) {
    const int64_t grid = (num_seqs * heads + 2 * kTokenWarps - 1) / (2 * kTokenWarps);
    if (grid > INT32_MAX) return PKV_ERR_UNSUPPORTED;
    return launch_after(append_token_kernel, (unsigned)grid, kTokenWarps * 32, st, prm) ==
                   cudaSuccess
               ? PKV_OK
               : PKV_ERR_CUDA;
  }
  // As many K and V heads to a CTA as still leave every SM about ten CTAs: a CTA's first loads wait
  // for three others (2-3 us). At 132k tokens all 16 take 329 us, 8 take 335, 4 take 349.
  const int64_t runs = num_tokens / kFp8Group + 2 * (int64_t)num_seqs;
  const int64_t per = std::max<int64_t>(
      1, std::min<int64_t>(2 * num_kv_heads, runs * heads / (10 * (int64_t)num_sms)));
  const int64_t grid = runs * (1 + (2 * num_kv_heads + per - 1) / per);
  if (grid > INT32_MAX) return PKV_ERR_UNSUPPORTED;
  return launch_after(append_run_kernel, (unsigned)grid, kRunThreads, st, prm, (int)per) ==
                 cudaSuccess
             ? PKV_OK
             : PKV_ERR_CUDA;
}

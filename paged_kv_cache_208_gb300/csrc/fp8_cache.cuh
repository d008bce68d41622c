// fp8_cache.cuh -- the 8-bit cache format, shared by the kernels that write and read it.
//
// A pool is [num_blocks, block_size, num_kv_heads, 128] e4m3 codes with one scale for every
// 64 consecutive tokens of a block ("group") and head: scale[block, head, token / 64], fp32.
// A cached value is code * scale. The store writes powers of two:
//
//     scale = 2^e,  e = max(-90, the smallest integer with  max |x| <= 448 * 2^e)
//
// over the finite values of the group's head. A power of two costs no precision (e4m3 is a
// floating-point format: a finer scale would move its grid, not refine it), the division by
// it is exact, so a value is rounded once, its product with a code is exact in bf16 (4
// significant bits; e >= -90 keeps it far from bf16's subnormals), and a scale that has to
// grow re-rounds only the codes that fall below the normal range.
#pragma once

#include <cuda_fp16.h>

#include "device_common.cuh"

namespace pkv {

constexpr int kFp8Group = 64;    // tokens that share a scale
constexpr int kFp8MinExp = -90;  // smallest scale exponent

// 2^e as fp32, e in the normal range
__device__ __forceinline__ float pow2f(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// Scale exponent for a group whose largest finite |x| has the bf16 bits `amax` (sign clear):
// x = (1 + M / 128) 2^(E - 127) and 448 = 1.75 * 2^8, so e = E - 127 - 8, one more when the
// mantissa exceeds 1.75.
__device__ __forceinline__ int fp8_scale_exp(uint32_t amax) {
  const int e = (int)(amax >> 7) - 135 + ((amax & 127u) > 96u ? 1 : 0);
  return max(e, kFp8MinExp);
}

// Largest |x| of a pair of bf16 words, as bf16 bits in both halves of the word.
__device__ __forceinline__ uint32_t bf16x2_absmax(uint32_t a, uint32_t b) {
  return __vmaxu2(a & 0x7fff7fffu, b & 0x7fff7fffu);
}
// a word with its infinities and NaNs replaced by zero
__device__ __forceinline__ uint32_t bf16x2_finite(uint32_t a) {
  if ((a & 0x7f80u) == 0x7f80u) a &= 0xffff0000u;
  if ((a & 0x7f800000u) == 0x7f800000u) a &= 0x0000ffffu;
  return a;
}

// Two fp32 values rounded to e4m3 (nearest even, saturated to +-448, NaN stays NaN); lo in the
// low byte.
__device__ __forceinline__ uint32_t cvt_e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
// Two e4m3 codes (low 16 bits) widened to an fp16 pair, exactly.
__device__ __forceinline__ uint32_t cvt_f16x2_e4m3x2(uint32_t codes) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, lo;\n\t}"
      : "=r"(r)
      : "r"(codes));
  return r;
}
__device__ __forceinline__ uint32_t cvt_f16x2_e4m3x2_hi(uint32_t codes) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, hi;\n\t}"
      : "=r"(r)
      : "r"(codes));
  return r;
}
__device__ __forceinline__ float2 f16x2_to_f32(uint32_t h) {
  return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

// Four bf16 (two words) times `inv`, as four e4m3 codes.
__device__ __forceinline__ uint32_t quantize4(uint32_t w0, uint32_t w1, float inv) {
  const uint32_t lo = cvt_e4m3x2(bf16_lo(w0) * inv, bf16_hi(w0) * inv);
  const uint32_t hi = cvt_e4m3x2(bf16_lo(w1) * inv, bf16_hi(w1) * inv);
  return lo | (hi << 16);
}
// Four codes at a scale that grew by 1 / ratio.
__device__ __forceinline__ uint32_t rescale4(uint32_t codes, float ratio) {
  const float2 a = f16x2_to_f32(cvt_f16x2_e4m3x2(codes));
  const float2 b = f16x2_to_f32(cvt_f16x2_e4m3x2_hi(codes));
  return cvt_e4m3x2(a.x * ratio, a.y * ratio) | (cvt_e4m3x2(b.x * ratio, b.y * ratio) << 16);
}
// Four codes times scale as four bf16 (exact for a power-of-two scale).
__device__ __forceinline__ uint2 dequantize4(uint32_t codes, float scale) {
  const float2 a = f16x2_to_f32(cvt_f16x2_e4m3x2(codes));
  const float2 b = f16x2_to_f32(cvt_f16x2_e4m3x2_hi(codes));
  return make_uint2(pack_bf16x2(a.x * scale, a.y * scale), pack_bf16x2(b.x * scale, b.y * scale));
}

// ------------------------------------------------------------------------ runs of a batch
// Packed sequences (cu[0 .. n]) cut into runs: the positions of one sequence that lie in one
// group. Sequence i is given the run slots [base(i), base(i + 1)) with
// base(i) = cu[i] / 64 + 2 i, which is never fewer than the groups its cu[i + 1] - cu[i]
// consecutive positions can touch (at most (len - 1) / 64 + 2), wherever they start; a slot
// past its runs has no work. Any cu gives a slot at most one (sequence, run), and every
// (sequence, run) at most one slot.
//
// The sequence of slot r: the largest i in [0, n) with base(i) <= r, by a 32-way search (every
// lane of the warp calls this; n >= 1).
__device__ __forceinline__ int find_sequence(const int32_t *cu, int n, int64_t r, int lane) {
  int lo = 0, len = n;
  while (len > 1) {
    const int stride = (len + 31) >> 5;
    const int i = lane * stride;
    const bool le = i < len && (int64_t)(*(cu + lo + i) >> 6) + 2 * (int64_t)(lo + i) <= r;
    const int c = __popc(__ballot_sync(0xffffffffu, le));
    const int step = (c > 0 ? c - 1 : 0) * stride;
    lo += step;
    len = min(stride, len - step);
  }
  return lo;
}
__device__ __forceinline__ int64_t run_base(int32_t cu_i, int i) {
  return (int64_t)(cu_i >> 6) + 2 * (int64_t)i;
}

}  // namespace pkv

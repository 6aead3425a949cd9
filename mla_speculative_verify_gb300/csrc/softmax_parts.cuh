// softmax_parts.cuh -- pieces of the decode kernels' softmax: how far a reference lags, and how Q and P
// are held in two 8-bit parts for an e4m3 cache.
#pragma once
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <stdint.h>

namespace mla {

constexpr float kRefSlack = 8.0f;    // octaves a score may exceed the row reference before it moves
// e4m3 path: a smaller slack (p <= 16) so that P can be stored times 2^4 (<= 256 < 448,
// the largest e4m3); probabilities down to 2^-10 of the reference stay in e4m3's normal
// range (split_p has the smaller ones). The 2^4 is applied by keeping the stored reference
// kPShiftFp8 octaves below the row's reference, so exp2(s - ref) is already P times 2^4; l
// carries the same factor, which cancels in O / l and in the LSE.
constexpr float kRefSlackFp8 = 4.0f;
constexpr float kPShiftFp8 = 4.0f;

// An fp32 rounded to the precision of e4m3 (4 significant bits, round to nearest even),
// still as fp32; exact for magnitudes in e4m3's normal range.
__device__ __forceinline__ float round_to_e4m3_precision(float x) {
  const uint32_t u = __float_as_uint(x);
  return __uint_as_float((u + 0x7FFFFu + ((u >> 20) & 1u)) & 0xFFF00000u);
}
// Two fp32 -> two e4m3 codes (round to nearest even, saturating), first in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
// Two P of one key (<= 256; P times 2^kPShiftFp8) -> an e4m3 part (hi) and the remainder in
// e5m2 (lo), through f16x2 (11 significant bits, and exact down to 2^-25). Each result holds
// the first value in its low byte.
//
// From 2^-6 on, where e4m3 is normal, lo is rounded to nearest and hi + lo is within 2^-8 of P.
// Below that hi ends on its grid of 2^-9 and lo has only its own 3 bits left, and what counts is
// the sum over many keys: a few strong keys beside a long, nearly flat rest, each of it 2^-15 of
// the largest, the rest as heavy as they are. Rounded to nearest, equal small P would all be off
// by the same up to 1/8 (with both parts in e4m3 everything below 2^-10 was lost: half of the
// output over 64k keys). So there lo is rounded up or down by comparing what is cut with a
// number that the key's position gives: f16's upper byte is an e5m2, so adding d in [0, 256) to
// the f16's bits and taking that byte rounds up with d's odds. d runs through a sequence that is
// evenly spread over any stretch of keys (multiples of the golden ratio, modulo 1), so the errors
// of a sum's keys cancel (64k flat keys beside a strong one: output off by 1.8e-3, its own bf16
// rounding), and equal calls give equal bits. It costs 1 to 2 % (2^20 keys, q = 8: block scales
// 220 -> 223 us, one scale 220 -> 225).
constexpr uint32_t kDitherStep = 0x9E3779B1u;  // 2^32 times the golden ratio's fraction, odd
__device__ __forceinline__ uint32_t dither_of(uint32_t at) { return __byte_perm(at, 0u, 0x4343u); }  // at's top byte, in both halves
__device__ __forceinline__ void split_p(float a, float b, uint32_t dither, uint32_t& hi, uint32_t& lo) {
  const __half2 w = __floats2half2_rn(a, b);
  const __nv_fp8x2_storage_t h = __nv_cvt_halfraw2_to_fp8x2(*reinterpret_cast<const __half2_raw*>(&w), __NV_SATFINITE,
                                                           __NV_E4M3);
  const __half2_raw hb = __nv_cvt_fp8x2_to_halfraw2(h, __NV_E4M3);
  const __half2 r = __hsub2(w, *reinterpret_cast<const __half2*>(&hb));
  const uint32_t normal = __hge2_mask(w, __half2half2(__ushort_as_half(0x2400)));  // >= 2^-6
  const uint32_t bits = *reinterpret_cast<const uint32_t*>(&r) + ((normal & 0x00800080u) | (~normal & dither));
  hi = (uint32_t)h;
  lo = __byte_perm(bits, 0u, 0x4431u);  // the upper bytes
}
// Byte offset of (row, column) in a 64-byte-swizzled e4m3 region with 64-byte rows.
__device__ __forceinline__ int sw64_offset(int row, int col) {
  return row * 64 + ((((col >> 4) ^ (row >> 1)) & 3) << 4) + (col & 15);
}

}  // namespace mla

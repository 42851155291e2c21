// 4-bit latent cache rows (416 bytes): 512 E2M1 codes in words of eight, 32 scales of 8 bits, 64 bf16 rope values.
//
// A scale is an unsigned float of 5 exponent and 3 mantissa bits: the sign bit that an E4M3 scale never uses goes to the exponent,
// so blocks from 1e-4 to 3e5 keep their precision without a second scale per row, and a float32 is made from the code by a
// shift.  Code times scale has 6 significant bits, so a value is exact in bf16.  In a word, values 2j and 2j + 1 lie 16 bits
// apart: one shift and one mask bring both to the same place of a bf16 pair.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp4.h>
#include <stdint.h>

namespace mtpsd {
namespace lat4 {

constexpr int ROW = 416;          // bytes
constexpr int OFF_SCALE = 256;
constexpr int OFF_ROPE = 288;
constexpr int BIAS = 8 * 111;     // scale code + BIAS = the float32 bits of its value >> 20

// Scale code of a block whose largest magnitude has the float32 bits m (as integers: a NaN is larger than any number).
__device__ __forceinline__ uint32_t scale_code(uint32_t m) {
  if (m >= 0x7f800000u) return 255u;
  const uint32_t b = __float_as_uint(__fdiv_rn(__uint_as_float(m), 6.0f));
  const int c = (int)((b + 0x7ffffu + ((b >> 20) & 1u)) >> 20) - BIAS;   // to 3 mantissa bits, ties to even
  if (c > 0) return (uint32_t)min(c, 254);
  return __uint_as_float(b) > 4.5f * 0x1p-19f ? 1u : 0u;                 // nearer to code 1 (9 * 2^-19) than to 0
}
__device__ __forceinline__ float scale_value(uint32_t c) {
  return c == 0 ? 0.f : __uint_as_float(c == 255 ? 0x7fffffffu : (c + BIAS) << 20);
}

// The word of eight values under a scale (value 2j in bits 4j .., value 2j + 1 in bits 16 + 4j ..).
__device__ __forceinline__ uint32_t encode8(const float* v, uint32_t code) {
  if (code == 255) return 0u;
  const float s = code == 0 ? 1.f : scale_value(code);
  float q[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) q[i] = __fdiv_rn(v[i], s);
  // .x is the low nibble
  const uint32_t b0 = __nv_cvt_float2_to_fp4x2(make_float2(q[0], q[2]), __NV_E2M1, cudaRoundNearest);
  const uint32_t b1 = __nv_cvt_float2_to_fp4x2(make_float2(q[4], q[6]), __NV_E2M1, cudaRoundNearest);
  const uint32_t b2 = __nv_cvt_float2_to_fp4x2(make_float2(q[1], q[3]), __NV_E2M1, cudaRoundNearest);
  const uint32_t b3 = __nv_cvt_float2_to_fp4x2(make_float2(q[5], q[7]), __NV_E2M1, cudaRoundNearest);
  return b0 | (b1 << 8) | (b2 << 16) | (b3 << 24);
}

// A warp's row: lane l brings values 8 l .. 8 l + 7 (v[0]) and 256 + 8 l .. (v[1]).
__device__ __forceinline__ void store_values(const float (*v)[8], uint8_t* row, int lane) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[h][i]) & 0x7fffffffu);
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    const uint32_t code = scale_code(m);
    *(uint32_t*)(row + h * 128 + 4 * lane) = encode8(v[h], code);
    // four lanes pairs' scales as one word
    uint32_t sc = code << (8 * ((lane >> 1) & 3));
    sc |= __shfl_xor_sync(0xffffffffu, sc, 2);
    sc |= __shfl_xor_sync(0xffffffffu, sc, 4);
    if ((lane & 7) == 0) *(uint32_t*)(row + OFF_SCALE + h * 16 + lane / 2) = sc;
  }
}
// Rope values 8 l .. 8 l + 7 of lane l < 8.
__device__ __forceinline__ void store_rope(const float* r, uint8_t* row, int lane) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(r[2 * i], r[2 * i + 1]);
    w[i] = *(const uint32_t*)&b;
  }
  *(uint4*)(row + OFF_ROPE + 16 * lane) = make_uint4(w[0], w[1], w[2], w[3]);
}

// Values 2j and 2j + 1 of a word as bf16 bits (low half: 2j) times 2^-126: the code's exponent and mantissa bits become the lowest
// exponent bits and the highest mantissa bit (code 1, 0.5, becomes a subnormal).
template <int J>
__device__ __forceinline__ uint32_t pair_bits(uint32_t w) {
  const uint32_t mag = J < 2 ? w << (6 - 4 * (J < 2 ? J : 0)) : w >> (4 * (J < 2 ? 2 : J) - 6);
  return (mag & 0x01c001c0u) | ((w << (12 - 4 * J)) & 0x80008000u);
}

// Eight values as four bf16 pairs, exact.
__device__ __forceinline__ void decode8(uint32_t w, float scale, uint32_t* out) {
  const uint32_t t[4] = {pair_bits<0>(w), pair_bits<1>(w), pair_bits<2>(w), pair_bits<3>(w)};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float lo = __uint_as_float(t[j] << 16) * 0x1p126f * scale, hi = __uint_as_float(t[j] & 0xffff0000u) * 0x1p126f * scale;
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    out[j] = *(const uint32_t*)&b;
  }
}

}  // namespace lat4
}  // namespace mtpsd

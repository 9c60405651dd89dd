// MXFP4 device helpers: blocks of 32 E2M1 codes with one E8M0 scale, stored
// in panels of 256 elements (include/nvfp4ns.h describes the layout).
//
// Encoding of a block: byte = max(E(amax) - 2, 0) with E the biased FP32
// exponent of the block's largest magnitude, which is
// floor(log2 amax) - 2 + 127 clamped to the E8M0 range (amax < 2^-124 and
// all-zero blocks take byte 0).  Codes are RNE_E2M1(x / 2^(byte - 127)) by
// v_cvt_scalef32_pk_fp4: the division by a power of two is exact, ties go to
// the even code, magnitudes of 5 and above become 6 (checked against
// comparisons at every midpoint and its neighbours, and for scales down to
// 2^-127).  A block with a NaN or an infinity gets byte 0xFF and codes 0.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace nvfp4 {
namespace mx {

constexpr int kPanel = 256;        // elements per panel row
constexpr int kPanelBytes = 128;   // code bytes per panel row
constexpr int kPanelScales = 8;    // scale bytes per panel row

typedef float floatx2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
// neighbours in memory that are aligned to one element only
typedef float float4u __attribute__((ext_vector_type(4), aligned(4)));
typedef uint16_t bf16x8u __attribute__((ext_vector_type(8), aligned(2)));

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// E8M0 byte of a block whose largest magnitude has the FP32 bits `amax`.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
  const uint32_t e = amax >> 23;
  return e >= 255u ? 255u : (e > 2u ? e - 2u : 0u);
}

// The FP32 value 2^(byte - 127); byte 0 is a subnormal, byte 255 gives inf.
__device__ __forceinline__ float scale_value(uint32_t byte) {
  return __uint_as_float(byte ? byte << 23 : 0x00400000u);
}

// Two codes in byte SEL of `old`.
template <int SEL>
__device__ __forceinline__ uint32_t encode2(uint32_t old, float lo, float hi, float scale) {
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(old, lo, hi, scale, SEL);
}

// Eight codes (one word) of eight values under one scale byte.
__device__ __forceinline__ uint32_t encode8(const float (&v)[8], uint32_t byte) {
  const float s = scale_value(byte);
  uint32_t w = 0;
  w = encode2<0>(w, v[0], v[1], s);
  w = encode2<1>(w, v[2], v[3], s);
  w = encode2<2>(w, v[4], v[5], s);
  w = encode2<3>(w, v[6], v[7], s);
  return byte == 255u ? 0u : w;
}

// The value of one E2M1 code times 2^(byte - 127), exact in FP32; NaN for
// byte 255.
template <int SEL>
__device__ __forceinline__ floatx2 decode2(uint32_t w, float scale) {
  return __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, SEL);
}
__device__ __forceinline__ void decode8(uint32_t w, uint32_t byte, float (&v)[8]) {
  const float s = scale_value(byte);
  const floatx2 a = decode2<0>(w, s), b = decode2<1>(w, s), c = decode2<2>(w, s), d = decode2<3>(w, s);
  v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
  v[4] = c.x; v[5] = c.y; v[6] = d.x; v[7] = d.y;
  if (byte == 255u) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __uint_as_float(0x7FC00000u);
  }
}

__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }
__device__ __forceinline__ uint32_t mag_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// Two FP32 values to packed BF16, round to nearest even (NaN stays NaN).
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  union { bf16x2 v; uint32_t u; } r;
  r.v[0] = (__bf16)lo;
  r.v[1] = (__bf16)hi;
  return r.u;
}

// BF16 in pairs, as they lie in memory: maxima by 16-bit integers, codes
// without widening.
typedef unsigned short ushortx2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  union { uint32_t u; ushortx2 v; } x{a}, y{b};
  x.v = __builtin_elementwise_max(x.v, y.v);
  return x.u;
}
// Two codes in byte SEL of `old`, from a pair of BF16 values.
template <int SEL>
__device__ __forceinline__ uint32_t encode2_bf16(uint32_t old, uint32_t pair, float scale) {
  union { uint32_t u; bf16x2 v; } x{pair};
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(old, x.v, scale, SEL);
}
__device__ __forceinline__ uint32_t encode8_bf16(const uint32_t (&p)[4], uint32_t byte) {
  const float s = scale_value(byte);
  uint32_t w = 0;
  w = encode2_bf16<0>(w, p[0], s);
  w = encode2_bf16<1>(w, p[1], s);
  w = encode2_bf16<2>(w, p[2], s);
  w = encode2_bf16<3>(w, p[3], s);
  return byte == 255u ? 0u : w;
}

}  // namespace mx
}  // namespace nvfp4

// MXFP8 device helpers: blocks of 32 E4M3 codes with one E8M0 scale, in panels
// of 256 elements (include/nvfp4ns.h describes the layout), and eight
// neighbours of a row at any alignment of the element type.
//
// Encoding of a block: byte = max(E(amax) - 8, 0) with E the biased FP32
// exponent of the block's largest magnitude, which is floor(log2 amax) - 8 + 127
// clamped to the E8M0 range.  Codes are RNE_E4M3(x / 2^(byte - 127)) by
// v_cvt_scalef32_pk_fp8, which divides by a power of two exactly and ties to
// even but turns what rounds beyond 448 into NaN: magnitudes are cut at 448
// units first.
#pragma once
#include "mxfp4_device.hpp"

namespace nvfp4 {
namespace mx {

constexpr int kPanelBytes8 = 256;  // code bytes per panel row

__device__ __forceinline__ uint32_t scale_byte8(uint32_t amax) {
  const uint32_t e = amax >> 23;
  return e >= 255u ? 255u : (e > 8u ? e - 8u : 0u);
}

// Eight codes of eight values under one scale byte.
__device__ __forceinline__ uint2 encode8_e4m3(const float (&v)[8], uint32_t byte) {
  typedef short shortx2 __attribute__((ext_vector_type(2)));
  const float s = scale_value(byte), top = 448.0f * s;
  union { shortx2 h[4]; uint2 u; } r;
  r.u = make_uint2(0, 0);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float a = __builtin_amdgcn_fmed3f(v[2 * i], -top, top), b = __builtin_amdgcn_fmed3f(v[2 * i + 1], -top, top);
    if (i & 1) r.h[i >> 1] = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r.h[i >> 1], a, b, s, true);
    else r.h[i >> 1] = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(r.h[i >> 1], a, b, s, false);
  }
  return byte == 255u ? make_uint2(0, 0) : r.u;
}

// The values of eight codes, exact in FP32; NaN for byte 255.
__device__ __forceinline__ void decode8_e4m3(uint2 c, uint32_t byte, float (&v)[8]) {
  const float s = byte == 255u ? __uint_as_float(0x7FC00000u) : scale_value(byte);
  const floatx2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)c.x, false), b = __builtin_amdgcn_cvt_pk_f32_fp8((int)c.x, true);
  const floatx2 d = __builtin_amdgcn_cvt_pk_f32_fp8((int)c.y, false), e = __builtin_amdgcn_cvt_pk_f32_fp8((int)c.y, true);
  v[0] = a.x * s; v[1] = a.y * s; v[2] = b.x * s; v[3] = b.y * s;
  v[4] = d.x * s; v[5] = d.y * s; v[6] = e.x * s; v[7] = e.y * s;
}

// Largest magnitude of the four lanes of a block.
__device__ __forceinline__ uint32_t quad_amax(uint32_t a) {
  a = umax(a, (uint32_t)__builtin_amdgcn_mov_dpp((int)a, 0xB1, 0xF, 0xF, true));   // lane ^ 1
  return umax(a, (uint32_t)__builtin_amdgcn_mov_dpp((int)a, 0x4E, 0xF, 0xF, true)); // lane ^ 2
}

// Eight neighbours as they lie in memory; the last n of a row, zeros behind
// them.  Global memory takes any alignment of the element type.
template <class T> struct Raw8;
inline bool turns(int C) { return C > 8 && C % 8 != 0; }
template <> struct Raw8<float> {
  float4u a, b;
  __device__ __forceinline__ void load(const float* p, int n) {
    if (n >= 8) {
      a = *reinterpret_cast<const float4u*>(p);
      b = *reinterpret_cast<const float4u*>(p + 4);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[i] = i < n ? p[i] : 0.0f;
        b[i] = 4 + i < n ? p[4 + i] : 0.0f;
      }
    }
  }
  __device__ __forceinline__ float get(int i) const { return i < 4 ? a[i & 3] : b[i & 3]; }
  // Elements c to c + 7 of a row of C, zeros behind its end.  TURNS (turns(C)):
  // its last eight, in one access without a branch on the lane, and, once they
  // are used, moved to their places (10 rows of 3687 normed: 8.0 us with the last
  // elements loaded one by one, 7.1 so; where rows end with an eight, the test
  // alone costs 1%).
  template <bool TURNS> __device__ __forceinline__ void load_row(const float* row, int c, int C) {
    if constexpr (TURNS) load(row + (c + 8 <= C ? c : C - 8), 8);
    else load(row + c, C - c);
  }
  template <bool TURNS> __device__ __forceinline__ void turn(int c, int C) {
    if (!TURNS || c + 8 <= C) return;
    const int d = c + 8 - C;
#pragma unroll
    for (int bit = 1; bit < 8; bit *= 2)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float moved = i + bit < 8 ? get((i + bit) & 7) : 0.0f, v = d & bit ? moved : get(i);
        if (i < 4) a[i & 3] = v;
        else b[i & 3] = v;
      }
    if (d >= 8) a = b = float4u{0, 0, 0, 0};
  }
};
template <> struct Raw8<uint16_t> {   // BF16 bits
  typedef uint32_t word4u __attribute__((ext_vector_type(4), aligned(2)));
  word4u w;
  __device__ __forceinline__ void load(const uint16_t* p, int n) {
    if (n >= 8) {
      w = *reinterpret_cast<const word4u*>(p);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = (2 * i < n ? (uint32_t)p[2 * i] : 0u) | (2 * i + 1 < n ? (uint32_t)p[2 * i + 1] << 16 : 0u);
    }
  }
  __device__ __forceinline__ float get(int i) const { return i & 1 ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1]); }
  template <bool TURNS> __device__ __forceinline__ void load_row(const uint16_t* row, int c, int C) {
    if constexpr (TURNS) load(row + (c + 8 <= C ? c : C - 8), 8);
    else load(row + c, C - c);
  }
  template <bool TURNS> __device__ __forceinline__ void turn(int c, int C) {
    if (!TURNS || c + 8 <= C) return;
    const int d = c + 8 - C;
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = d & 1 ? (w[i] >> 16) | (i < 3 ? w[(i + 1) & 3] << 16 : 0u) : w[i];
#pragma unroll
    for (int bit = 1; bit < 4; bit *= 2)
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = d & (2 * bit) ? (i + bit < 4 ? w[(i + bit) & 3] : 0u) : w[i];
    if (d >= 8) w = word4u{0, 0, 0, 0};
  }
};
__device__ __forceinline__ void store8u(float* p, int n, const float (&v)[8]) {
  if (n >= 8) {
    *reinterpret_cast<float4u*>(p) = float4u{v[0], v[1], v[2], v[3]};
    *reinterpret_cast<float4u*>(p + 4) = float4u{v[4], v[5], v[6], v[7]};
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = v[i];
  }
}
__device__ __forceinline__ void store8u(uint16_t* p, int n, const float (&v)[8]) {
  typedef uint32_t word4u __attribute__((ext_vector_type(4), aligned(2)));
  if (n >= 8) {
    *reinterpret_cast<word4u*>(p) =
        word4u{pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) p[i] = (uint16_t)pack_bf16(v[i], 0.0f);
  }
}
// What a value becomes when it is stored as T.
__device__ __forceinline__ float as_stored(float v, const float*) { return v; }
__device__ __forceinline__ float as_stored(float v, const uint16_t*) { return bf16_lo(pack_bf16(v, 0.0f)); }

}  // namespace mx
}  // namespace nvfp4

// y = x W^T with W in NVFP4 (16-element blocks with E4M3 scales, one FP32 scale
// s_g) and x as it is: the linear layer of few tokens, whose time is the
// weights' way from memory.
//
// A weight's value without s_g, E2M1 times E4M3, has at most six significant
// bits and is exact in BF16, so BF16 rows of x multiply it on
// v_mfma_f32_16x16x32_bf16 without a rounding before the FP32 sum; FP32 rows do
// so in three BF16 parts of eight bits each, which hold all 24.
//
// A workgroup takes 16 rows of W, its waves divide K; of 128 elements a lane
// has 32 of one row (16 bytes of codes, two scales), eight a matrix
// instruction.  The waves' sums meet in LDS, in wave order.
#include "layer.hpp"
#include "mx8_device.hpp"

namespace nvfp4 {
namespace {
using namespace mx;

typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef uint16_t u16_any __attribute__((aligned(1)));   // two neighbouring scales, K / 16 of any parity
typedef uint32_t wordx4 __attribute__((ext_vector_type(4)));
typedef uint32_t word4_8 __attribute__((ext_vector_type(4), aligned(8)));

struct Nv {
  const void* x;
  const uint8_t *codes, *scales;
  const float* sg;
  void* y;
  int T, N, groups;      // groups: of 16 rows of W
  int64_t K;
};

// Eight weights: codes times their block's scale.
__device__ __forceinline__ bf16x8 weights8(uint32_t w, float s) {
  const floatx2 a = decode2<0>(w, 1.0f), b = decode2<1>(w, 1.0f), c = decode2<2>(w, 1.0f), d = decode2<3>(w, 1.0f);
  union { uint32_t u[4]; bf16x8 v; } r;
  r.u[0] = pack_bf16(a.x * s, a.y * s);
  r.u[1] = pack_bf16(b.x * s, b.y * s);
  r.u[2] = pack_bf16(c.x * s, c.y * s);
  r.u[3] = pack_bf16(d.x * s, d.y * s);
  return r.v;
}

// Eight values of x as BF16 operands that sum to them: one, or three for FP32.
template <class X> struct Parts;
template <> struct Parts<uint16_t> {
  static constexpr int kParts = 1;
  wordx4 w;
  __device__ __forceinline__ void load(const uint16_t* p, bool in) {
    w = in ? *reinterpret_cast<const wordx4*>(p) : wordx4{0, 0, 0, 0};
  }
  __device__ __forceinline__ bf16x8 part(int) const {
    union { wordx4 u; bf16x8 v; } r{w};
    return r.v;
  }
};
template <> struct Parts<float> {
  static constexpr int kParts = 3;
  floatx4 a, b;
  __device__ __forceinline__ void load(const float* p, bool in) {
    a = in ? *reinterpret_cast<const floatx4*>(p) : floatx4{0, 0, 0, 0};
    b = in ? *reinterpret_cast<const floatx4*>(p + 4) : floatx4{0, 0, 0, 0};
  }
  // The next part: the leading bits, cut off; what is left stays.  Infinities
  // and NaN go whole into the first.
  static __device__ __forceinline__ uint32_t take(float& v) {
    const uint32_t bits = __float_as_uint(v);
    if (!(fabsf(v) < __builtin_inff())) {
      const uint32_t top = v != v ? 0x7FC00000u : bits;
      v = 0.0f;
      return top;
    }
    const uint32_t top = bits & 0xFFFF0000u;
    v -= __uint_as_float(top);
    return top;
  }
  __device__ __forceinline__ bf16x8 part(int) {
    union { uint32_t u[4]; bf16x8 v; } r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float lo = i < 2 ? a[2 * i] : b[2 * i - 4], hi = i < 2 ? a[2 * i + 1] : b[2 * i - 3];
      const uint32_t l = take(lo), h = take(hi);
      r.u[i] = l >> 16 | h;
      if (i < 2) {
        a[2 * i] = lo;
        a[2 * i + 1] = hi;
      } else {
        b[2 * i - 4] = lo;
        b[2 * i - 3] = hi;
      }
    }
    return r.v;
  }
};

template <class X, int TG, Dt OT, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void nv_kernel(const Nv a) {
  constexpr int kDeep = 4;                                  // steps of 128 in flight
  __shared__ floatx4 sums[WAVES][TG][64];
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = (int)(blockIdx.x % (unsigned)a.groups) * 16, t0 = (int)(blockIdx.x / (unsigned)a.groups) * 16 * TG;
  // rows behind an operand's end: its last row, into values that are not written
  const int64_t row = n0 + r < a.N ? n0 + r : a.N - 1;
  const uint8_t* codes = a.codes + row * (a.K / 2);
  const uint8_t* scales = a.scales + row * (a.K / 16);
  const X* x[TG];
#pragma unroll
  for (int g = 0; g < TG; ++g) {
    const int t = t0 + 16 * g + r;
    x[g] = static_cast<const X*>(a.x) + (int64_t)(t < a.T ? t : a.T - 1) * a.K;
  }
  const int64_t steps = (a.K + 127) / 128;
  const int64_t s0 = steps * wave / WAVES, s1 = steps * (wave + 1) / WAVES;
  floatx4 acc[TG];
#pragma unroll
  for (int g = 0; g < TG; ++g) acc[g] = floatx4{0, 0, 0, 0};
  for (int64_t s = s0; s < s1; s += kDeep) {
    wordx4 c[kDeep];
    uint32_t sc[kDeep];
#pragma unroll
    for (int i = 0; i < kDeep; ++i) {
      // K is a multiple of 16: of a lane's 32 elements all, the first half or none
      const int64_t k = 128 * (s + i) + 32 * q;
      c[i] = wordx4{0, 0, 0, 0};
      sc[i] = 0;
      if (s + i < s1) {
        if (k + 32 <= a.K) {
          c[i] = *reinterpret_cast<const word4_8*>(codes + k / 2);
          sc[i] = *reinterpret_cast<const u16_any*>(scales + k / 16);
        } else if (k < a.K) {
          const uint2 h = *reinterpret_cast<const uint2*>(codes + k / 2);
          c[i] = wordx4{h.x, h.y, 0, 0};
          sc[i] = scales[k / 16];
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kDeep; ++i) {
      if (s + i >= s1) break;
      const int64_t k = 128 * (s + i) + 32 * q;
      const float f[2] = {__builtin_amdgcn_cvt_f32_fp8((int)sc[i], 0), __builtin_amdgcn_cvt_f32_fp8((int)sc[i], 1)};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bf16x8 w = weights8(c[i][j], f[j >> 1]);
#pragma unroll
        for (int g = 0; g < TG; ++g) {
          Parts<X> v;
          v.load(x[g] + k + 8 * j, k + 8 * j < a.K);
#pragma unroll
          for (int p = 0; p < Parts<X>::kParts; ++p)
            acc[g] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w, v.part(p), acc[g], 0, 0, 0);
        }
      }
    }
  }
#pragma unroll
  for (int g = 0; g < TG; ++g) sums[wave][g][lane] = acc[g];
  __syncthreads();
  // lane: rows n0 + 4 q .. + 3 of W, row r of x's group `wave`
  if (wave >= TG) return;
  const int t = t0 + 16 * wave + r, n = n0 + 4 * q;
  if (t >= a.T || n >= a.N) return;
  floatx4 v = sums[0][wave][lane];
  for (int w = 1; w < WAVES; ++w) v += sums[w][wave][lane];
  v *= *a.sg;
  const int64_t at = (int64_t)t * a.N + n;
  if (a.N % 4 == 0) {
    if constexpr (OT == Dt::F32) *reinterpret_cast<floatx4*>(static_cast<float*>(a.y) + at) = v;
    else *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.y) + at) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (n + e < a.N) {
        if constexpr (OT == Dt::F32) static_cast<float*>(a.y)[at + e] = v[e];
        else static_cast<uint16_t*>(a.y)[at + e] = (uint16_t)pack_bf16(v[e], 0.0f);
      }
  }
}

template <class X, int TG, Dt OT>
hipError_t launch(const Nv& a, hipStream_t s) {
  const unsigned grid = (unsigned)a.groups * (unsigned)((a.T + 16 * TG - 1) / (16 * TG));
  // enough waves to cover the chip several times, none without a step
  if (grid < 512 && a.K >= 2048) nv_kernel<X, TG, OT, 16><<<grid, 1024, 0, s>>>(a);
  else nv_kernel<X, TG, OT, 4><<<grid, 256, 0, s>>>(a);
  return hipGetLastError();
}
template <class X>
hipError_t by_shape(const Nv& a, Dt ot, hipStream_t s) {
  if (a.T <= 16) return ot == Dt::F32 ? launch<X, 1, Dt::F32>(a, s) : launch<X, 1, Dt::BF16>(a, s);
  return ot == Dt::F32 ? launch<X, 2, Dt::F32>(a, s) : launch<X, 2, Dt::BF16>(a, s);
}

}  // namespace

hipError_t launch_nv_linear(const void* x, Dt xt, int64_t T, int64_t K, const uint8_t* codes, const uint8_t* scales,
                            const float* sg, int64_t N, void* y, Dt yt, hipStream_t s) {
  const Nv a{x, codes, scales, sg, y, (int)T, (int)N, (int)((N + 15) / 16), K};
  return xt == Dt::F32 ? by_shape<float>(a, yt, s) : by_shape<uint16_t>(a, yt, s);
}

}  // namespace nvfp4

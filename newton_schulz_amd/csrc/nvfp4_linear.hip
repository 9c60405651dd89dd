// y = x W^T with W in NVFP4 (16-element blocks with E4M3 scales, one FP32 scale
// s_g) and x as it is: the linear layer of few tokens, whose time is the
// weights' way from memory as long as decoding them (two or three vector
// instructions a pair) stays below it.
//
// x enters as BF16 operands that sum to it: BF16 rows as they are, FP32 rows in
// three parts of eight bits each, which hold all 24.  E2M1 codes, and codes
// times their E4M3 scale (at most six significant bits), are exact in BF16 too,
// so every product is exact and sums are FP32.  What lies below 2^-133, BF16's
// last bit, of an FP32 x is cut off.
//
// Codes times block scales reach 2688, and s_g brings them back: a sum without
// s_g would leave FP32 where y does not (from |x| = 2^128 / 2688 on).  So the
// power of two of s_g is in the blocks' scales (products stay exact), and what is
// left of s_g, 1 to 2, follows the sum (Global).
//
// One or two tokens (gemv_kernel): a wave takes rows of W whole, 32 codes a
// lane, x in LDS; v_dot2_f32_bf16 adds a block's sixteen products without its
// scale, which one fused multiply-add a block applies.  1 x 11008 x 4096 BF16: 25 MB
// in 7.5 to 8.0 us, 3.2 of them a launch; vector instructions fill 72% of the CUs'
// busy cycles.
// More (nv_kernel): a workgroup takes 16 or 32 rows of W, its waves divide K; codes
// times scales feed v_mfma_f32_16x16x32_bf16.  16 x 4096 x 11008 BF16: 11.3 us, each
// CU drawing all of x (352 KB, from L2) beside its 100 KB of codes; LDS is busy a
// quarter of the time, the matrix units 6%.
#include <type_traits>

#include "dma.hpp"
#include "layer.hpp"
#include "mx8_device.hpp"

namespace nvfp4 {
namespace {
using namespace mx;

typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t wordx4 __attribute__((ext_vector_type(4)));
// as rows of W lie where K is an odd multiple of 16
typedef uint32_t wordx4u __attribute__((ext_vector_type(4), aligned(8)));
typedef uint16_t half_u __attribute__((aligned(1)));

struct Nv {
  const void* x;
  const uint8_t *codes, *scales;
  const float* sg;
  void* y;
  int T, N, groups;      // groups: workgroups along N
  int64_t K;
};

// Eight neighbours of a row of x, and the BF16 operands that sum to them.
template <class X> struct Parts;
template <> struct Parts<uint16_t> {
  static constexpr int kParts = 1, kWords = 1;     // sixteen bytes each, as in memory
  wordx4 w;
  __device__ __forceinline__ wordx4 word(int) const { return w; }
  __device__ __forceinline__ void set(int, wordx4 v) { w = v; }
  __device__ __forceinline__ void load(const uint16_t* p) { w = *reinterpret_cast<const wordx4*>(p); }
  __device__ __forceinline__ void clear() { w = wordx4{0, 0, 0, 0}; }
  __device__ __forceinline__ void split(wordx4 (&parts)[1]) const { parts[0] = w; }
};
template <> struct Parts<float> {
  static constexpr int kParts = 3, kWords = 2;
  floatx4 a, b;
  __device__ __forceinline__ wordx4 word(int i) const {
    union { floatx4 f; wordx4 u; } r{i ? b : a};
    return r.u;
  }
  __device__ __forceinline__ void set(int i, wordx4 v) {
    union { wordx4 u; floatx4 f; } r{v};
    (i ? b : a) = r.f;
  }
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const floatx4*>(p);
    b = *reinterpret_cast<const floatx4*>(p + 4);
  }
  __device__ __forceinline__ void clear() { a = b = floatx4{0, 0, 0, 0}; }
  // The leading bits, cut off, the leading bits of what is left, and the rest.
  // Infinities and NaN go whole into the first (their lanes are looked for, not
  // waited for: the whole wave takes the short way where there are none).
  __device__ __forceinline__ void split(wordx4 (&parts)[3]) const {
    float v[8];
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = i < 4 ? a[i & 3] : b[i & 3];
      most = umax(most, mag_bits(v[i]));
    }
    const bool odd = __any(most >= 0x7F800000u);
#pragma unroll
    for (int p = 0; p < 3; ++p) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        parts[p][i] = __builtin_amdgcn_perm(__float_as_uint(v[2 * i + 1]), __float_as_uint(v[2 * i]), 0x07060302u);
      if (p == 2) break;
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] -= __uint_as_float(__float_as_uint(v[i]) & 0xFFFF0000u);
      if (p == 0 && odd) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float f = i < 4 ? a[i & 3] : b[i & 3];
          if (fabsf(f) < __builtin_inff()) continue;
          v[i] = 0.0f;
          if (f != f) parts[0][i >> 1] |= i & 1 ? 0x7FC00000u : 0x7FC0u;
        }
      }
    }
  }
};

// s_g = unit * rest: unit a power of two, as large as s_g's but for scales that
// would take a block's factor out of FP32 or its weights below BF16's normal
// numbers; rest carries the sign, NaN, infinities and zero.
struct Global {
  float sg;
  __device__ __forceinline__ explicit Global(const float* p)
      : sg(*(const __attribute__((address_space(4))) float*)(uintptr_t)p) {}
  // To be used from here on: taken before the loads of x and W go out, a wave
  // would wait for it first (1 x 11008 x 4096 FP32 9.8 us, so 9.4).
  __device__ __forceinline__ void landed() { asm volatile("" : "+s"(sg)); }
  __device__ __forceinline__ int bits() const {
    const int e = (int)(__float_as_uint(sg) >> 23 & 255u) - 127;
    return e < -116 ? -116 : e > 111 ? 111 : e;
  }
  // 2^more unit
  __device__ __forceinline__ float unit(int more) const { return __uint_as_float((uint32_t)(127 + bits() + more) << 23); }
  __device__ __forceinline__ float rest() const { return sg * __uint_as_float((uint32_t)(127 - bits()) << 23); }
};

// Two blocks' scales in the low bytes of b, times a power of two.
__device__ __forceinline__ floatx2 scales2(uint32_t b, float unit) {
  return __builtin_amdgcn_cvt_scalef32_pk_f32_fp8(b, unit, false);
}

template <Dt OT>
__device__ __forceinline__ void put1(void* y, int64_t at, float v) {
  if constexpr (OT == Dt::F32) static_cast<float*>(y)[at] = v;
  else static_cast<uint16_t*>(y)[at] = (uint16_t)pack_bf16(v, 0.0f);
}

// ---- one or two tokens --------------------------------------------------------
constexpr int kStep = 64 * 32;            // elements of a row that a wave takes at a time
constexpr int kGemvWaves = 8;
// Rows of W a wave: of BF16 x one (11008 x 4096 7.9 us, two 8.1, four 8.25; 4096 x
// 11008 7.6, 7.8, 9.9), of FP32 x two, which share the reads of its three parts.
template <class X> constexpr int kGemvRows = Parts<X>::kParts == 1 ? 1 : 2;
constexpr int kGemvLds = 65536;           // bytes of x a workgroup holds at most

// The sum over a wave's lanes, in every lane.
__device__ __forceinline__ float lane_sum(float v) {
  v += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0xB1, 0xF, 0xF, true));    // lane ^ 1
  v += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x4E, 0xF, 0xF, true));    // lane ^ 2
  v += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x141, 0xF, 0xF, true));   // mirrored in eight
  v += __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(v), 0x140, 0xF, 0xF, true));   // mirrored in sixteen
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}

// Two codes in byte SEL of w, as BF16, over 2^7: a block's sum of sixteen times x,
// at most 96 |x|, stays in FP32.
constexpr int kCodeBits = 7;
template <int SEL>
__device__ __forceinline__ bf16x2 pair_of(uint32_t w) {
  return __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, 1.0f / (1 << kCodeBits), SEL);
}
__device__ __forceinline__ float dot8(uint32_t c, wordx4 x, float sum) {
  union { uint32_t u; bf16x2 v; } x0{x[0]}, x1{x[1]}, x2{x[2]}, x3{x[3]};
  sum = __builtin_amdgcn_fdot2_f32_bf16(pair_of<0>(c), x0.v, sum, false);
  sum = __builtin_amdgcn_fdot2_f32_bf16(pair_of<1>(c), x1.v, sum, false);
  sum = __builtin_amdgcn_fdot2_f32_bf16(pair_of<2>(c), x2.v, sum, false);
  return __builtin_amdgcn_fdot2_f32_bf16(pair_of<3>(c), x3.v, sum, false);
}

// span: elements of K in LDS at a time, a multiple of kStep.  K is at least 32.
// A part of a row of x lies in LDS in chunks of eight elements; chunk
// 4 l + j, which lane l reads as its j-th, at 4 l + (j ^ l / 4 % 4), so that eight
// lanes reading their j-th hit distinct banks.
// K32: K is a multiple of 32 (the other case costs 11008 x 4096 0.4 us).
template <class X, int T, Dt OT, bool K32>
__global__ __launch_bounds__(64 * kGemvWaves) void gemv_kernel(const Nv a, int span) {
  constexpr int P = Parts<X>::kParts, R = kGemvRows<X>;
  extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
  wordx4* xs = reinterpret_cast<wordx4*>(lds);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = ((int)blockIdx.x * kGemvWaves + wave) * R;
  const uint8_t *codes[R], *scales[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int64_t n = n0 + r < a.N ? n0 + r : a.N - 1;      // rows behind W's end: not written
    codes[r] = a.codes + n * (a.K / 2);
    scales[r] = a.scales + n * (a.K / 16);
  }
  float acc[R][T];
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int t = 0; t < T; ++t) acc[r][t] = 0.0f;
  const int chunks = span / 8;            // of a part in LDS
  Global sg(a.sg);
  typedef std::conditional_t<K32, wordx4, wordx4u> Codes;
  typedef std::conditional_t<K32, uint16_t, half_u> Scales;
  Codes c[R];
  uint32_t sc[R];
  // the lane's codes of the step at k; behind a row's end its last 32
  auto fetch = [&](int64_t k) {
    const int64_t kl = k + 32 * lane, kc = kl + 32 <= a.K ? kl : a.K - 32;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      c[r] = *reinterpret_cast<const Codes*>(codes[r] + kc / 2);
      sc[r] = *reinterpret_cast<const Scales*>(scales[r] + kc / 16);
    }
  };
  fetch(0);
  for (int64_t k0 = 0; k0 < a.K; k0 += span) {
    if (k0) __syncthreads();              // all waves are through with the span before
    const int64_t left = a.K - k0;
    for (int i = threadIdx.x; i < T * chunks; i += 64 * kGemvWaves) {
      const int t = T == 1 ? 0 : i >= chunks, ch = i - t * chunks;
      Parts<X> v;
      v.clear();
      if (8 * (int64_t)ch < left) v.load(static_cast<const X*>(a.x) + t * a.K + k0 + 8 * ch);
      const int l = ch >> 2, at = 4 * l + ((ch ^ (l >> 2)) & 3);
      wordx4 parts[P];
      v.split(parts);
#pragma unroll
      for (int p = 0; p < P; ++p) xs[(t * P + p) * chunks + at] = parts[p];
    }
    __syncthreads();
    sg.landed();
    const float unit = sg.unit(kCodeBits);
    const int64_t k1 = k0 + span < a.K ? k0 + span : a.K;
    for (int64_t k = k0; k < k1; k += kStep) {
      wordx4 u[R];
      float s[R][2];
      // where K ends in a lane's middle, its sixteen are the second half of the
      // row's last 32; what lies behind K has scales of zero
      const int64_t here = a.K - (k + 32 * lane);
      const bool half = !K32 && here == 16;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        u[r] = half ? wordx4{c[r][2], c[r][3], 0, 0} : wordx4{c[r][0], c[r][1], c[r][2], c[r][3]};
        const uint32_t b = here <= 0 ? 0u : half ? sc[r] >> 8 : sc[r];
        const floatx2 f = scales2(b, unit);
        s[r][0] = f.x;
        s[r][1] = f.y;
      }
      fetch(k + kStep < a.K ? k + kStep : k);
#pragma unroll
      for (int t = 0; t < T; ++t)
#pragma unroll
        for (int p = 0; p < P; ++p) {
          const wordx4* x = xs + (t * P + p) * chunks + (int)(k - k0) / 8 + 4 * lane;
          wordx4 v[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] = x[j ^ ((lane >> 2) & 3)];
#pragma unroll
          for (int r = 0; r < R; ++r) {
            acc[r][t] = fmaf(s[r][0], dot8(u[r][1], v[1], dot8(u[r][0], v[0], 0.0f)), acc[r][t]);
            acc[r][t] = fmaf(s[r][1], dot8(u[r][3], v[3], dot8(u[r][2], v[2], 0.0f)), acc[r][t]);
          }
        }
    }
  }
#pragma unroll
  for (int r = 0; r < R; ++r)
#pragma unroll
    for (int t = 0; t < T; ++t) {
      const float v = lane_sum(acc[r][t]) * sg.rest();
      if (lane == r * T + t && n0 + r < a.N) put1<OT>(a.y, (int64_t)t * a.N + n0 + r, v);
    }
}

// ---- more tokens ------------------------------------------------------------------
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

// Of a step of 128 elements lane (q, r) = (l / 16, l % 16) multiplies row r's
// elements 32 q .. + 31, eight an instruction.  Its codes are 16 bytes of W's row;
// x comes in whole lines (four rows an instruction) and turns in LDS of the
// wave's own, as it lies in memory: chunk c (eight elements) of row r at position
// c ^ r, FP32's halves apart.
// Everything that DEEP steps read goes out before the first is used, from
// clamped places instead of behind branches, which would wait for each other;
// the places are 32-bit offsets from scalar bases.
// K32: K is a multiple of 32, a lane's 32 elements all in or all behind the end.
template <class X, int TG, int NG, Dt OT, int WAVES, int DEEP, bool K32>
__global__ __launch_bounds__(64 * WAVES) void nv_kernel(const Nv a) {
  constexpr int P = Parts<X>::kParts, W = Parts<X>::kWords;
  __shared__ wordx4 turn[WAVES][W * TG][16][16];
  __shared__ floatx4 sums[WAVES][NG * TG][64];
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = (int)(blockIdx.x % (unsigned)a.groups) * 16 * NG, t0 = (int)(blockIdx.x / (unsigned)a.groups) * 16 * TG;
  const int64_t K = a.K;
  const int steps = (int)((K + 127) / 128), last = (int)(K - 128 * (int64_t)(steps - 1));   // elements of the last step
  const int s0 = (int)((int64_t)steps * wave / WAVES), s1 = (int)((int64_t)steps * (wave + 1) / WAVES);
  // rows behind an operand's end: its last row, into values that are not written
  const uint8_t* codes = a.codes + (int64_t)n0 * (K / 2);
  const uint8_t* scales = a.scales + (int64_t)n0 * (K / 16);
  const X* x = static_cast<const X*>(a.x) + (int64_t)t0 * K;
  uint32_t crow[NG], srow[NG];
#pragma unroll
  for (int n = 0; n < NG; ++n) {
    const uint32_t row = (uint32_t)(n0 + 16 * n + r < a.N ? 16 * n + r : a.N - 1 - n0);
    crow[n] = row * (uint32_t)(K / 2);
    srow[n] = row * (uint32_t)(K / 16);
  }
  uint32_t xrow[TG][4];
#pragma unroll
  for (int g = 0; g < TG; ++g)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int t = 16 * g + 4 * i + q;
      xrow[g][i] = (uint32_t)(t0 + t < a.T ? t : a.T - 1 - t0) * (uint32_t)K;
    }
  floatx4 acc[NG][TG];
#pragma unroll
  for (int n = 0; n < NG; ++n)
#pragma unroll
    for (int g = 0; g < TG; ++g) acc[n][g] = floatx4{0, 0, 0, 0};
  Global sg(a.sg);
  for (int s = s0; s < s1; s += DEEP) {
    wordx4 c[DEEP][NG];
    uint32_t sc[DEEP][NG];
    Parts<X> v[DEEP][TG][4];
#pragma unroll
    for (int i = 0; i < DEEP; ++i) {
      const int at = s + i < s1 ? s + i : s1 - 1;             // the last again: not multiplied
      const int end = at == steps - 1 ? last : 128;           // elements of this step
      const uint8_t* cs = codes + (int64_t)at * 64;
      const uint8_t* ss = scales + (int64_t)at * 8;
#pragma unroll
      for (int n = 0; n < NG; ++n)
        if constexpr (K32) {
          const uint32_t e = 32 * q < end ? 32u * q : 0u;
          c[i][n] = *reinterpret_cast<const wordx4*>(cs + (crow[n] + e / 2));
          sc[i][n] = *reinterpret_cast<const uint16_t*>(ss + (srow[n] + e / 16));
        } else {
          const uint32_t e0 = 32 * q < end ? 32u * q : 0u, e1 = 32 * q + 16 < end ? 32u * q + 16 : 0u;
          const uint2 lo = *reinterpret_cast<const uint2*>(cs + (crow[n] + e0 / 2)), hi = *reinterpret_cast<const uint2*>(cs + (crow[n] + e1 / 2));
          c[i][n] = wordx4{lo.x, lo.y, hi.x, hi.y};
          sc[i][n] = ss[srow[n] + e0 / 16] | (uint32_t)ss[srow[n] + e1 / 16] << 8;
        }
      const X* xc = x + (int64_t)at * 128;
      const uint32_t e = 8 * r < end ? 8u * r : 0u;
#pragma unroll
      for (int g = 0; g < TG; ++g)
#pragma unroll
        for (int j = 0; j < 4; ++j) v[i][g][j].load(xc + (xrow[g][j] + e));
    }
    __builtin_amdgcn_sched_barrier(0);
    sg.landed();
    const float unit = sg.unit(0);
#pragma unroll
    for (int i = 0; i < DEEP; ++i) {
      if (s + i >= s1) break;
      if (s + i == steps - 1 && last < 128) {                 // nothing behind K
#pragma unroll
        for (int n = 0; n < NG; ++n) sc[i][n] = 32 * q + 32 <= last ? sc[i][n] : 32 * q < last ? sc[i][n] & 0xFFu : 0u;
        if (8 * r >= last) {
#pragma unroll
          for (int g = 0; g < TG; ++g)
#pragma unroll
            for (int j = 0; j < 4; ++j) v[i][g][j].clear();
        }
      }
      // row 4 j + q, chunk r
#pragma unroll
      for (int g = 0; g < TG; ++g)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int p = 0; p < W; ++p) turn[wave][g * W + p][4 * j + q][r ^ (4 * j + q)] = v[i][g][j].word(p);
      wave_sync();
      float f[NG][2];
#pragma unroll
      for (int n = 0; n < NG; ++n) {
        const floatx2 t = scales2(sc[i][n], unit);
        f[n][0] = t.x;
        f[n][1] = t.y;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        bf16x8 w[NG];
#pragma unroll
        for (int n = 0; n < NG; ++n) w[n] = weights8(c[i][n][j], f[n][j >> 1]);
#pragma unroll
        for (int g = 0; g < TG; ++g) {
          Parts<X> e;
#pragma unroll
          for (int p = 0; p < W; ++p) e.set(p, turn[wave][g * W + p][r][(4 * q + j) ^ r]);
          wordx4 parts[P];
          e.split(parts);
#pragma unroll
          for (int p = 0; p < P; ++p) {
            union { wordx4 u; bf16x8 v; } b{parts[p]};
#pragma unroll
            for (int n = 0; n < NG; ++n) acc[n][g] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w[n], b.v, acc[n][g], 0, 0, 0);
          }
        }
      }
      wave_sync();
    }
  }
#pragma unroll
  for (int n = 0; n < NG; ++n)
#pragma unroll
    for (int g = 0; g < TG; ++g) sums[wave][n * TG + g][lane] = acc[n][g];
  __syncthreads();
  // wave: rows of W and tokens number `wave`; lane: four rows of W, a token
  if (wave >= NG * TG) return;
  const int t = t0 + 16 * (wave % TG) + r, n = n0 + 16 * (wave / TG) + 4 * q;
  if (t >= a.T || n >= a.N) return;
  floatx4 v = sums[0][wave][lane];
  for (int w = 1; w < WAVES; ++w) v += sums[w][wave][lane];
  v *= sg.rest();
  const int64_t at = (int64_t)t * a.N + n;
  if (a.N % 4 == 0) {
    if constexpr (OT == Dt::F32) *reinterpret_cast<floatx4*>(static_cast<float*>(a.y) + at) = v;
    else *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.y) + at) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (n + e < a.N) put1<OT>(a.y, at + e, v[e]);
  }
}

template <class X, int T, Dt OT>
hipError_t gemv(Nv a, hipStream_t s) {
  constexpr int kBytes = 2 * T * Parts<X>::kParts;           // of LDS an element of K
  const int64_t most = kGemvLds / kBytes / kStep * kStep, all = (a.K + kStep - 1) / kStep * kStep;
  const int span = (int)(all < most ? all : most);
  a.groups = (a.N + kGemvWaves * kGemvRows<X> - 1) / (kGemvWaves * kGemvRows<X>);
  const dim3 grid((unsigned)a.groups), block(64 * kGemvWaves);
  if (a.K % 32 == 0) gemv_kernel<X, T, OT, true><<<grid, block, (size_t)span * kBytes, s>>>(a, span);
  else gemv_kernel<X, T, OT, false><<<grid, block, (size_t)span * kBytes, s>>>(a, span);
  return hipGetLastError();
}

template <class X, int TG, Dt OT, bool K32>
hipError_t launch(Nv a, hipStream_t s) {
  const unsigned tokens = (unsigned)((a.T + 16 * TG - 1) / (16 * TG)), grid = (unsigned)a.groups * tokens;
  constexpr int kDeep = sizeof(X) == 2 && TG == 1 ? 2 : 1;
  // FP32 rows cost a wave three times the instructions: while each workgroup has a
  // CU to itself sixteen waves share K (10 tokens, 938 x 3664: 8.3 us, with eight
  // 9.2; 16 tokens, 4000 x 4096: 8.7, 9.3; BF16 there 6.3, 5.8)
  if constexpr (sizeof(X) == 4)
    if (grid <= 256) {
      nv_kernel<X, TG, 1, OT, 16, kDeep, K32><<<grid, 1024, 0, s>>>(a);
      return hipGetLastError();
    }
  // Pairs of row groups share x's way through LDS (and its split): a workgroup of
  // two takes 1.6 times as long as one (FP32 1.4), which pays unless the CUs are
  // then loaded unevenly (us, there / one by one; BF16: 5 x 6000 x 4096 7.7 / 8.3,
  // 16 x 8192 x 2048 5.3 / 5.6, 100 x 4096 x 4096 16.4 / 18.5, but 16 x 11008 x 4096
  // 13.7 / 11.9; FP32: 5 x 6000 x 4096 11.9 / 12.7, 32 x 11008 x 4096 24.8 / 32.4)
  const unsigned pairs = (unsigned)(a.groups + 1) / 2 * tokens;
  if (grid > 256 && (pairs + 255) / 256 * (sizeof(X) == 4 ? 7 : 8) < (grid + 255) / 256 * 5) {
    a.groups = (a.groups + 1) / 2;
    nv_kernel<X, TG, 2, OT, 8, 1, K32><<<pairs, 512, 0, s>>>(a);
    return hipGetLastError();
  }
  nv_kernel<X, TG, 1, OT, 8, kDeep, K32><<<grid, 512, 0, s>>>(a);
  return hipGetLastError();
}
template <class X, int TG, Dt OT>
hipError_t by_width(const Nv& a, hipStream_t s) {
  return a.K % 32 == 0 ? launch<X, TG, OT, true>(a, s) : launch<X, TG, OT, false>(a, s);
}
template <class X, Dt OT>
hipError_t by_tokens(const Nv& a, hipStream_t s) {
  if (a.K >= 32 && a.T == 1) return gemv<X, 1, OT>(a, s);
  if (a.K >= 32 && a.T == 2) return gemv<X, 2, OT>(a, s);
  if constexpr (sizeof(X) == 2)
    if (a.T > 16) return by_width<X, 2, OT>(a, s);
  return by_width<X, 1, OT>(a, s);
}

}  // namespace

hipError_t launch_nv_linear(const void* x, Dt xt, int64_t T, int64_t K, const uint8_t* codes, const uint8_t* scales,
                            const float* sg, int64_t N, void* y, Dt yt, hipStream_t s) {
  const Nv a{x, codes, scales, sg, y, (int)T, (int)N, (int)((N + 15) / 16), K};
  if (xt == Dt::F32) return yt == Dt::F32 ? by_tokens<float, Dt::F32>(a, s) : by_tokens<float, Dt::BF16>(a, s);
  return yt == Dt::F32 ? by_tokens<uint16_t, Dt::F32>(a, s) : by_tokens<uint16_t, Dt::BF16>(a, s);
}

}  // namespace nvfp4

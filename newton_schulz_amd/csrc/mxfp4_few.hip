// MXFP4 products with few rows on one side: out[t][n] = beta addend + alpha
// sum_k x[t][k] w[n][k] for up to 32 rows of x, quantized on the way in (the
// linear layer's decode) or held in MXFP4 already.
//
// What counts is reading w once.  A workgroup takes 16 rows of w, its waves
// divide the panels of K and have their loads of w -- up to four panels, 8 KB
// a wave -- in flight before anything waits; meanwhile a wave quantizes its
// panels of x, a lane one 32-element block at a time, into LDS of its own.  In
// v_mfma_scale_f32_16x16x128 lane l holds one block of row l % 16 of either
// operand.  The waves' sums meet in LDS, in wave order.
//
// Measured in a graph, x in BF16: 1 x 11008 x 4096 6.2 us (24 MB of weights and
// scales, 3.9 TB/s with the launch in it), 16 x 4096 x 4096 6.2 us.
#include "mxfp4_device.hpp"
#include "panel.hpp"

namespace nvfp4 {
namespace {
using namespace mx;

typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef int intx4 __attribute__((ext_vector_type(4)));
typedef int intx8 __attribute__((ext_vector_type(8)));

struct Few {
  const void* x;                  // [T][K], or codes in panels of T rows
  const uint8_t* x_scales;        // with codes
  const uint8_t* w;
  const uint8_t* w_scales;
  const float* addend;
  void* out;
  int T, N, panels;
  int64_t K;
  float alpha, beta;
};

struct Block {
  intx4 codes;
  uint32_t byte;
};

// Block `b` (32 elements) of row t of x, zero behind the row's end.
template <bool VEC>
__device__ __forceinline__ Block block_of(const float* x, int64_t K, int64_t t, int64_t k) {
  const float* p = x + t * K + k;
  float v[32];
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    if constexpr (VEC) {
      const float4 f = k + 4 * q < K ? *reinterpret_cast<const float4*>(p + 4 * q) : make_float4(0, 0, 0, 0);
      v[4 * q] = f.x; v[4 * q + 1] = f.y; v[4 * q + 2] = f.z; v[4 * q + 3] = f.w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[4 * q + i] = k + 4 * q + i < K ? p[4 * q + i] : 0.0f;
    }
  }
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < 32; ++i) a = umax(a, mag_bits(v[i]));
  Block r;
  r.byte = scale_byte(a);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    float e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = v[8 * q + i];
    r.codes[q] = (int)encode8(e, r.byte);
  }
  return r;
}
template <bool VEC>
__device__ __forceinline__ Block block_of(const uint16_t* x, int64_t K, int64_t t, int64_t k) {
  const uint16_t* p = x + t * K + k;
  uint32_t v[4][4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if constexpr (VEC) {
      const uint4 f = k + 8 * q < K ? *reinterpret_cast<const uint4*>(p + 8 * q) : make_uint4(0, 0, 0, 0);
      v[q][0] = f.x; v[q][1] = f.y; v[q][2] = f.z; v[q][3] = f.w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t e = k + 8 * q + 2 * i;
        v[q][i] = (e < K ? (uint32_t)p[8 * q + 2 * i] : 0u) | (e + 1 < K ? (uint32_t)p[8 * q + 2 * i + 1] << 16 : 0u);
      }
    }
  }
  uint32_t a = 0;
#pragma unroll
  for (int q = 0; q < 4; ++q)
#pragma unroll
    for (int i = 0; i < 4; ++i) a = max_u16x2(a, v[q][i] & 0x7FFF7FFFu);
  Block r;
  r.byte = scale_byte(umax(a << 16, a & 0xFFFF0000u));
#pragma unroll
  for (int q = 0; q < 4; ++q) r.codes[q] = (int)encode8_bf16(v[q], r.byte);
  return r;
}

__device__ __forceinline__ floatx4 mfma(intx4 a, uint32_t sa, intx4 b, uint32_t sb, floatx4 c) {
  // 4-bit operands are four registers; the rest of the builtin's eight is not read
  const intx8 x = __builtin_shufflevector(a, a, 0, 1, 2, 3, -1, -1, -1, -1);
  const intx8 y = __builtin_shufflevector(b, b, 0, 1, 2, 3, -1, -1, -1, -1);
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(x, y, c, 4, 4, 0, (int)sa, 0, (int)sb);
}

// Orders a wave's own LDS writes before its reads of other lanes' values.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// X: float, uint16_t (BF16 bits) or uint8_t (codes).  TG: groups of 16 rows of
// x.  DEEP: panels a wave has in flight.
template <class X, int TG, Dt OT, bool VEC, int WAVES, int DEEP>
__global__ __launch_bounds__(64 * WAVES) void few_kernel(const Few f) {
  constexpr bool kHeld = sizeof(X) == 1;
  constexpr int kBlocks = 8 * DEEP;                         // blocks of a row in flight
  __shared__ floatx4 sums[WAVES][TG][64];
  __shared__ intx4 xc[kHeld ? 1 : WAVES][kHeld ? 1 : 16 * TG * kBlocks];
  __shared__ uint8_t xb[kHeld ? 1 : WAVES][kHeld ? 1 : 16 * TG * kBlocks];
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = (int)blockIdx.x * 16;
  const int64_t row = n0 + r < f.N ? n0 + r : f.N - 1;      // rows behind w's end: not written
  const int p0 = f.panels * wave / WAVES, p1 = f.panels * (wave + 1) / WAVES;
  floatx4 acc[TG];
#pragma unroll
  for (int g = 0; g < TG; ++g) acc[g] = floatx4{0, 0, 0, 0};
  for (int p = p0; p < p1; p += DEEP) {
    intx4 wc[DEEP][2];
    uint2 ws[DEEP];
    Block held[kHeld ? DEEP : 1][2][TG];
#pragma unroll
    for (int i = 0; i < DEEP; ++i) {
      const int64_t pi = p + i < p1 ? p + i : p1 - 1;       // the last again: not multiplied
      const uint8_t* c = f.w + (pi * f.N + row) * kPanelBytes + 16 * q;
      wc[i][0] = *reinterpret_cast<const intx4*>(c);
      wc[i][1] = *reinterpret_cast<const intx4*>(c + 64);
      ws[i] = *reinterpret_cast<const uint2*>(f.w_scales + (pi * f.N + row) * kPanelScales);
      if constexpr (kHeld) {
        // rows behind x's end: its last row, into columns that are not written
#pragma unroll
        for (int g = 0; g < TG; ++g) {
          const int64_t at = pi * f.T + (16 * g + r < f.T ? 16 * g + r : f.T - 1);
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            held[i][u][g].codes = *reinterpret_cast<const intx4*>(static_cast<const uint8_t*>(f.x) + at * kPanelBytes + 64 * u + 16 * q);
            held[i][u][g].byte = f.x_scales[at * kPanelScales + 4 * u + q];
          }
        }
      }
    }
    if constexpr (!kHeld) {
      // block b of row t at slot t kBlocks + (b ^ t % 8): sixteen rows' reads
      // of one block spread over the banks
      const int live = (p1 - p < DEEP ? p1 - p : DEEP) * 8;
      for (int k = lane; k < f.T * kBlocks; k += 64) {
        const int t = k / kBlocks, b = k % kBlocks;
        if (b >= live) continue;
        const Block e = block_of<VEC>(static_cast<const X*>(f.x), f.K, t, (int64_t)p * kPanel + 32 * b);
        xc[wave][t * kBlocks + (b ^ (t & 7))] = e.codes;
        xb[wave][t * kBlocks + b] = (uint8_t)e.byte;
      }
      wave_sync();
    }
#pragma unroll
    for (int i = 0; i < DEEP; ++i) {
      if (p + i >= p1) break;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const uint32_t sw = (u ? ws[i].y : ws[i].x) >> (8 * q);
#pragma unroll
        for (int g = 0; g < TG; ++g) {
          Block b;
          if constexpr (kHeld) {
            b = held[i][u][g];
          } else {
            const int t = 16 * g + r < f.T ? 16 * g + r : 0, k = 8 * i + 4 * u + q;
            b.codes = xc[wave][t * kBlocks + (k ^ (t & 7))];
            b.byte = xb[wave][t * kBlocks + k];
          }
          acc[g] = mfma(wc[i][u], sw, b.codes, b.byte, acc[g]);
        }
      }
    }
    if constexpr (!kHeld) wave_sync();
  }
#pragma unroll
  for (int g = 0; g < TG; ++g) sums[wave][g][lane] = acc[g];
  __syncthreads();
  // lane: rows n0 + 4 q .. + 3 of w, row r of x; group g by wave g
  if (wave >= TG) return;
  const int t = 16 * wave + r, n = n0 + 4 * q;
  if (t >= f.T || n >= f.N) return;
  floatx4 v = sums[0][wave][lane];
  for (int w = 1; w < WAVES; ++w) v += sums[w][wave][lane];
  const int64_t at = (int64_t)t * f.N + n;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v[e] *= f.alpha;
    if (f.addend && n + e < f.N) v[e] = fmaf(f.beta, f.addend[at + e], v[e]);
  }
  if (f.N % 4 == 0) {
    if constexpr (OT == Dt::F32)
      *reinterpret_cast<floatx4*>(static_cast<float*>(f.out) + at) = v;
    else
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(f.out) + at) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (n + e < f.N) {
        if constexpr (OT == Dt::F32) static_cast<float*>(f.out)[at + e] = v[e];
        else static_cast<uint16_t*>(f.out)[at + e] = (uint16_t)pack_bf16(v[e], 0.0f);
      }
  }
}

template <class X, int TG, Dt OT, bool VEC>
hipError_t launch(const Few& f, hipStream_t s) {
  const int groups = (f.N + 15) / 16;
  // enough waves to cover the chip several times, none without a panel
  if (groups < 512 && f.panels >= 16)
    few_kernel<X, TG, OT, VEC, 16, 1><<<groups, 1024, 0, s>>>(f);
  else
    few_kernel<X, TG, OT, VEC, 4, 4><<<groups, 256, 0, s>>>(f);
  return hipGetLastError();
}
template <class X, Dt OT, bool VEC>
hipError_t by_rows_of_x(const Few& f, hipStream_t s) {
  return f.T <= 16 ? launch<X, 1, OT, VEC>(f, s) : launch<X, 2, OT, VEC>(f, s);
}
template <class X, bool VEC>
hipError_t by_out(const Few& f, Dt ot, hipStream_t s) {
  return ot == Dt::F32 ? by_rows_of_x<X, Dt::F32, VEC>(f, s) : by_rows_of_x<X, Dt::BF16, VEC>(f, s);
}

}  // namespace

hipError_t launch_mx_few(const void* x, Dt xt, const uint8_t* x_scales, int64_t T, int64_t K, const uint8_t* w,
                         const uint8_t* w_scales, int64_t N, float alpha, float beta, const float* addend, void* out,
                         Dt ot, hipStream_t s) {
  if (T < 1 || T > kMxFewRows) return hipErrorInvalidValue;
  Few f{x, x_scales, w, w_scales, addend, out, (int)T, (int)N, (int)((K + kPanel - 1) / kPanel), K, alpha, beta};
  if (x_scales) return by_out<uint8_t, true>(f, ot, s);
  if (xt == Dt::F32) return K % 4 == 0 ? by_out<float, true>(f, ot, s) : by_out<float, false>(f, ot, s);
  return K % 8 == 0 ? by_out<uint16_t, true>(f, ot, s) : by_out<uint16_t, false>(f, ot, s);
}

}  // namespace nvfp4

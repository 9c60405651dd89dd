// out = beta addend + alpha P Q^T with P in MXFP8 and Q in MXFP4 (activations
// in 8 bits, weights in 4): the block-scaled matrix instructions take the two
// formats together, at FP8's rate, with FP32 accumulation.
//
// Which elements meet: in v_mfma_scale_f32_32x32x64 lane l holds row l % 32.
// Its 4-bit operand is slot h = l / 32, 32 neighbours with the lane's own scale;
// its 8-bit operand's first 16 bytes are elements 16 h .. of slot 0, the last 16
// the same of slot 1, with the lane's scale for slot h (in 16x16x128 there are
// four slots: q = l / 16 holds half q % 2 of slots q / 2 and 2 + q / 2).  Any
// blocks of K serve as slots as long as both operands take the same.
//
// What the instruction rounds: it adds the products of eight neighbours of K
// in a window that ends 13 bits below the largest one's leading bit (2^(Ea + Eb)),
// each product cut off there, and everything else in FP32 (measured; a test
// holds it).  A product of codes has its last bit at most 4 + 13 bits below the
// largest code's product of one pair of 4-bit values, so that smaller
// neighbours lose up to 7 * 2^-13 of the largest product.  For BF16 outputs
// that is less than their own rounding; FP32 outputs, and the product of few
// rows, which waits for memory anyway, take P in two parts, codes from 2 on and
// below: each spans 8 exponents, and 7 + 4 + 2 bits fit the window exactly.
#include "layer.hpp"
#include "mx8_device.hpp"

namespace nvfp4 {
namespace {
using namespace mx;

typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef float floatx16 __attribute__((ext_vector_type(16)));
typedef int intx4 __attribute__((ext_vector_type(4)));
typedef int intx8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ intx8 four_bits(intx4 a) {
  // 4-bit operands are four registers; the rest of the builtin's eight is not read
  return __builtin_shufflevector(a, a, 0, 1, 2, 3, -1, -1, -1, -1);
}

// The two parts of 8-bit codes: exponent field 8 and above (bit 6), or below.
// What is not in a part leaves a zero with its sign.
__device__ __forceinline__ void two_parts(intx8 x, intx8& high, intx8& low) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t w = (uint32_t)x[i], t = w & 0x40404040u, m = (t << 1) - (t >> 6);
    high[i] = (int)(w & (m | 0x80808080u));
    low[i] = (int)(w & ~m);
  }
}

// beta addend + alpha v of `n` neighbours (n <= 4), rounded once.
template <Dt OT>
__device__ __forceinline__ void put4(const Product8& g, int64_t at, int n, bool vec, floatx4 v) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    v[e] *= g.alpha;
    if (g.addend && e < n) v[e] = fmaf(g.beta, g.addend[at + e], v[e]);
  }
  if (vec) {
    if constexpr (OT == Dt::F32) *reinterpret_cast<floatx4*>(static_cast<float*>(g.out) + at) = v;
    else *reinterpret_cast<uint2*>(static_cast<uint16_t*>(g.out) + at) = make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < n) {
        if constexpr (OT == Dt::F32) static_cast<float*>(g.out)[at + e] = v[e];
        else static_cast<uint16_t*>(g.out)[at + e] = (uint16_t)pack_bf16(v[e], 0.0f);
      }
  }
}

// Sixteen rows of Q a workgroup, 16 TG rows of P; the waves divide the panels
// of K and have DEEP of them in flight; their sums meet in LDS, in wave order.
template <int TG, Dt OT, int WAVES, int DEEP>
__global__ __launch_bounds__(64 * WAVES) void few8_kernel(const Product8 g, int panels) {
  __shared__ floatx4 sums[WAVES][TG][64];
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = (int)blockIdx.x * 16, t0 = (int)blockIdx.y * 16 * TG;
  const int M = (int)g.M, N = (int)g.N;
  // rows behind an operand's end read its last row: not written
  const int64_t row = n0 + r < N ? n0 + r : N - 1;
  int64_t prow[TG];
#pragma unroll
  for (int i = 0; i < TG; ++i) prow[i] = t0 + 16 * i + r < M ? t0 + 16 * i + r : M - 1;
  const int p0 = panels * wave / WAVES, p1 = panels * (wave + 1) / WAVES;
  floatx4 acc[TG];
#pragma unroll
  for (int i = 0; i < TG; ++i) acc[i] = floatx4{0, 0, 0, 0};
  for (int p = p0; p < p1; p += DEEP) {
    intx4 wc[DEEP][2];
    uint2 ws[DEEP];
    intx8 xc[DEEP][2][TG];
    uint2 xs[DEEP][TG];
#pragma unroll
    for (int i = 0; i < DEEP; ++i) {
      const int64_t pi = p + i < p1 ? p + i : p1 - 1;       // the last again: not multiplied
      const uint8_t* c = g.q + (pi * N + row) * kPanelBytes + 16 * q;
      wc[i][0] = *reinterpret_cast<const intx4*>(c);
      wc[i][1] = *reinterpret_cast<const intx4*>(c + 64);
      ws[i] = *reinterpret_cast<const uint2*>(g.q_scales + (pi * N + row) * kPanelScales);
#pragma unroll
      for (int k = 0; k < TG; ++k) {
        const uint8_t* x = g.p + (pi * M + prow[k]) * kPanelBytes8 + 16 * q;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const intx4 lo = *reinterpret_cast<const intx4*>(x + 128 * u), hi = *reinterpret_cast<const intx4*>(x + 128 * u + 64);
          xc[i][u][k] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        }
        xs[i][k] = *reinterpret_cast<const uint2*>(g.p_scales + (pi * M + prow[k]) * kPanelScales);
      }
    }
#pragma unroll
    for (int i = 0; i < DEEP; ++i) {
      if (p + i >= p1) break;
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int k = 0; k < TG; ++k) {
          intx8 high, low;
          two_parts(xc[i][u][k], high, low);
          const int sw = (int)((u ? ws[i].y : ws[i].x) >> (8 * q)), sx = (int)((u ? xs[i][k].y : xs[i][k].x) >> (8 * q));
          acc[k] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(four_bits(wc[i][u]), high, acc[k], 4, 0, 0, sw, 0, sx);
          acc[k] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(four_bits(wc[i][u]), low, acc[k], 4, 0, 0, sw, 0, sx);
        }
    }
  }
#pragma unroll
  for (int i = 0; i < TG; ++i) sums[wave][i][lane] = acc[i];
  __syncthreads();
  // lane: rows n0 + 4 q .. + 3 of Q, row r of P's group `wave`
  if (wave >= TG) return;
  const int t = t0 + 16 * wave + r, n = n0 + 4 * q;
  if (t >= M || n >= N) return;
  floatx4 v = sums[0][wave][lane];
  for (int w = 1; w < WAVES; ++w) v += sums[w][wave][lane];
  put4<OT>(g, (int64_t)t * N + n, N - n, N % 4 == 0, v);
}

template <int TG, Dt OT>
hipError_t few(const Product8& g, hipStream_t s) {
  const int panels = (int)((g.K + kPanel - 1) / kPanel);
  const dim3 grid((unsigned)((g.N + 15) / 16), (unsigned)((g.M + 16 * TG - 1) / (16 * TG)));
  // enough waves to cover the chip several times, none without a panel
  if (grid.x * grid.y < 512 && panels >= 16) few8_kernel<TG, OT, 16, 1><<<grid, 1024, 0, s>>>(g, panels);
  else few8_kernel<TG, OT, 4, TG == 1 ? 4 : 2><<<grid, 256, 0, s>>>(g, panels);
  return hipGetLastError();
}

}  // namespace

size_t mx8_workspace(int64_t, int64_t, int64_t) { return 0; }

hipError_t launch_mx8_product(const Product8& g, void*, hipStream_t s) {
  if (g.M <= 16) return g.ot == Dt::F32 ? few<1, Dt::F32>(g, s) : few<1, Dt::BF16>(g, s);
  return g.ot == Dt::F32 ? few<2, Dt::F32>(g, s) : few<2, Dt::BF16>(g, s);
}

}  // namespace nvfp4

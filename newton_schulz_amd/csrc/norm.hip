// Root-mean-square norm with the residual's addition and dropout in front, and
// its output in 16 or 32 bits, MXFP8 or MXFP4; its gradients; dropout by
// itself.
//
//   h = residual + k x / (1 - p)       rounded to h's type (k: dropout's mask)
//   r = 1 / sqrt(mean(h^2) + eps)      sum and root in FP64, r in FP32
//   y = (h r) w                        two FP32 products in this order
//
// A code changes where its value crosses a border, so y must not depend on how
// the sum is split over lanes: with FP64 sums r is the same FP32 number (but
// for one split in 1e8) whichever variant, pass or oracle computes it, and y is
// then the same to the bit.
//
// All of it is bound by memory: every tensor is read once and written once, a
// row staying in registers between its sum and its outputs.
#include <type_traits>

#include "layer.hpp"
#include "mx8_device.hpp"
#include "philox.hpp"

namespace nvfp4 {
namespace {
using namespace mx;

// w[c .. c + 7] of either type, zeros behind its C.
template <bool TURNS>
__device__ __forceinline__ void load_weights(const void* w, Dt t, int c, int C, float (&v)[8]) {
  if (t == Dt::F32) {
    Raw8<float> r;
    r.template load_row<TURNS>(static_cast<const float*>(w), c, C);
    r.template turn<TURNS>(c, C);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = r.get(i);
  } else {
    Raw8<uint16_t> r;
    r.template load_row<TURNS>(static_cast<const uint16_t*>(w), c, C);
    r.template turn<TURNS>(c, C);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = r.get(i);
  }
}
__device__ __forceinline__ void store_as(void* p, Dt t, int64_t at, int n, const float (&v)[8]) {
  if (t == Dt::F32) store8u(static_cast<float*>(p) + at, n, v);
  else store8u(static_cast<uint16_t*>(p) + at, n, v);
}

// The sum over groups of N lanes, in every lane.
template <int N = 64, class V>
__device__ __forceinline__ V wave_sum(V v) {
#pragma unroll
  for (int d = N / 2; d > 0; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

// LPR lanes a row, NV vectors of eight neighbours a lane: vector k of a lane
// holds columns 8 (k LPR + lane) on, so that 32 lanes hold a panel's 256
// columns of the row and four of them a block.
// 8192 x 4096: BF16 x on an FP32 residual to h and MXFP8 370 MB in 73 us (5.1 TB/s,
// 98% of a large copy); BF16 with dropout to h and MXFP4 220 MB in 46 us.  One row
// of 4096: 3.6 us, a launch and two trips to memory behind each other.
template <class X, class H, int LPR, int NV, bool TURNS>
__global__ __launch_bounds__(LPR < 256 ? 256 : LPR) void norm_kernel(const NormForward a) {
  constexpr int kThreads = LPR < 256 ? 256 : LPR, kRows = kThreads / LPR, kWaves = LPR / 64;
  static_assert(kRows == 1 || kWaves <= 1, "rows that share a workgroup take a wave each at most");
  __shared__ double sums[kWaves > 0 ? kWaves : 1];
  const int lane = threadIdx.x % LPR;
  const int64_t t = (int64_t)blockIdx.x * kRows + threadIdx.x / LPR;
  if (kRows > 1 && t >= a.T) return;
  const int C = a.C, padded = (C + kPanel - 1) / kPanel * kPanel;
  const int64_t at = t * C;
  float v[NV][8];
  {
    Raw8<X> x[NV];
    Raw8<H> r[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = 8 * (k * LPR + lane);
      x[k].template load_row<TURNS>(static_cast<const X*>(a.x) + at, c, C);
      if (a.residual) r[k].template load_row<TURNS>(static_cast<const H*>(a.residual) + at, c, C);
    }
    uint64_t seed = 0, offset = 0;
    if (a.drop.rng) {
      seed = a.drop.rng[0];
      offset = a.drop.rng[1];
    }
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = 8 * (k * LPR + lane);
      x[k].template turn<TURNS>(c, C);
      if (a.residual) r[k].template turn<TURNS>(c, C);
      if (a.drop.rng) {
        const Mask8 m((uint32_t)(c >> 3), (uint32_t)t, seed, offset);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float base = a.residual ? r[k].get(i) : 0.0f;
          v[k][i] = m.keeps(i, a.drop.cut) ? fmaf(x[k].get(i), a.drop.scale, base) : base;
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) v[k][i] = a.residual ? x[k].get(i) + r[k].get(i) : x[k].get(i);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) v[k][i] = as_stored(v[k][i], static_cast<const H*>(nullptr));
      if (a.h && c < C) store8u(static_cast<H*>(a.h) + at + c, C - c, v[k]);
    }
  }
  double s0 = 0.0, s1 = 0.0;
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      s0 = fma((double)v[k][i], (double)v[k][i], s0);
      s1 = fma((double)v[k][i + 1], (double)v[k][i + 1], s1);
    }
  double sum = wave_sum<(LPR < 64 ? LPR : 64)>(s0 + s1);
  if constexpr (kWaves > 1) {
    if ((lane & 63) == 0) sums[lane >> 6] = sum;
    __syncthreads();
    sum = 0.0;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) sum += sums[i];
  }
  const float rstd = (float)(1.0 / sqrt(sum / (double)C + a.eps));
  if (a.rstd && lane == 0) a.rstd[t] = rstd;
  if (!a.y && !a.codes8 && !a.codes4) return;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = 8 * (k * LPR + lane);
    if (c >= padded) break;                  // whole 32-lane groups leave together
    float w[8];
    load_weights<TURNS>(a.w, a.wt, c, C, w);
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[k][i] = v[k][i] * rstd * w[i];
      // behind the row's end 0, also beside a rstd of NaN
      if (c + i >= C) v[k][i] = 0.0f;
      top = umax(top, mag_bits(v[k][i]));
    }
    if (a.y && c < C) store_as(a.y, a.yt, at + c, C - c, v[k]);
    if (a.codes8 || a.codes4) {
      top = quad_amax(top);
      const int64_t line = (int64_t)(c / kPanel) * a.T + t;
      const int l = (c >> 3) & 31;
      if (a.codes8) {
        const uint32_t byte = scale_byte8(top);
        *reinterpret_cast<uint2*>(a.codes8 + line * kPanelBytes8 + 8 * l) = encode8_e4m3(v[k], byte);
        if ((l & 3) == 0) a.scales8[line * kPanelScales + (l >> 2)] = (uint8_t)byte;
      }
      if (a.codes4) {
        const uint32_t byte = scale_byte(top);
        *reinterpret_cast<uint32_t*>(a.codes4 + line * kPanelBytes + 4 * l) = encode8(v[k], byte);
        if ((l & 3) == 0) a.scales4[line * kPanelScales + (l >> 2)] = (uint8_t)byte;
      }
    }
  }
  if constexpr (LPR < 32) {
    // the rest of the row's one panel
    for (int l = LPR + lane; l < 32; l += LPR) {
      if (a.codes8) {
        *reinterpret_cast<uint2*>(a.codes8 + t * kPanelBytes8 + 8 * l) = make_uint2(0, 0);
        if ((l & 3) == 0) a.scales8[t * kPanelScales + (l >> 2)] = 0;
      }
      if (a.codes4) {
        *reinterpret_cast<uint32_t*>(a.codes4 + t * kPanelBytes + 4 * l) = 0;
        if ((l & 3) == 0) a.scales4[t * kPanelScales + (l >> 2)] = 0;
      }
    }
  }
}

// The normed rows in MXFP4 along the tokens.  A workgroup takes 256 tokens (one
// panel of y^T) x 128 columns: a wave a block of 32 tokens, a lane two
// neighbouring columns of it, whose codes and scales pass through LDS so that
// each column's 128-byte line leaves whole.  8192 x 4096 BF16: 87 MB in 15.7 us.
constexpr int kTileCols = 128;

// Two neighbouring columns of a row, as they lie in memory.
template <class H> struct Two;
template <> struct Two<float> {
  float2 v;
  template <bool VEC> __device__ __forceinline__ void load(const float* p, int n) {
    if constexpr (VEC) v = *reinterpret_cast<const float2*>(p);
    else v = make_float2(p[0], n > 1 ? p[1] : 0.0f);
  }
  __device__ __forceinline__ void clear() { v = make_float2(0.0f, 0.0f); }
  __device__ __forceinline__ float get(int j) const { return j ? v.y : v.x; }
};
template <> struct Two<uint16_t> {
  uint32_t v;
  template <bool VEC> __device__ __forceinline__ void load(const uint16_t* p, int n) {
    if constexpr (VEC) v = *reinterpret_cast<const uint32_t*>(p);
    else v = (uint32_t)p[0] | (n > 1 ? (uint32_t)p[1] << 16 : 0u);
  }
  __device__ __forceinline__ void clear() { v = 0; }
  __device__ __forceinline__ float get(int j) const { return j ? bf16_hi(v) : bf16_lo(v); }
};

template <class H, bool VEC>
__global__ __launch_bounds__(512) void norm_cols_kernel(const H* h, const float* rstd, const void* weight, Dt wt, int64_t T,
                                                        int64_t C, uint32_t tiles, uint8_t* codes, uint8_t* scales) {
  __shared__ __attribute__((aligned(16))) uint8_t lc[kTileCols * 128];
  __shared__ __attribute__((aligned(16))) uint8_t ls[kTileCols * 8];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t c0 = (int64_t)(blockIdx.x % tiles) * kTileCols, g = blockIdx.x / tiles;
  const int64_t t0 = g * kPanel + 32 * wave;
  const int64_t c = c0 + 2 * lane;
  const int n = c < C ? (C - c < 2 ? 1 : 2) : 0;
  // blocks behind the last token are zero whatever the weight is (in one with a
  // token an infinite or NaN weight makes the block NaN anyway)
  float w[2] = {0.0f, 0.0f};
  if (n && t0 < T) {
    if (wt == Dt::F32) {
      Two<float> t;
      t.template load<false>(static_cast<const float*>(weight) + c, n);
      w[0] = t.get(0);
      w[1] = t.get(1);
    } else {
      Two<uint16_t> t;
      t.template load<false>(static_cast<const uint16_t*>(weight) + c, n);
      w[0] = t.get(0);
      w[1] = t.get(1);
    }
  }
  Two<H> u[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    if (t0 + i < T && n) u[i].template load<VEC>(h + (t0 + i) * C + c, n);
    else u[i].clear();
  }
  float r[32];                                   // the tokens' rstd, 0 behind the last
#pragma unroll
  for (int i = 0; i < 32; ++i) r[i] = t0 + i < T ? rstd[t0 + i] : 0.0f;
  // codes of tokens behind the last are 0, where 0 * 0 * w is -0 beside w < 0
  uint32_t mask[4];
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const int64_t left = T - t0 - 8 * s;
    mask[s] = left >= 8 ? 0xFFFFFFFFu : left > 0 ? (1u << (4 * (int)left)) - 1u : 0u;
  }
  // y is computed for its maximum and again for its codes: kept in between, its
  // 64 values a lane cost more than 128 products do (8192 x 4096 BF16: 28.7 us
  // kept, 15.7 so)
  uint4 k[2];
  uint32_t b[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 32; ++i) top = umax(top, mag_bits(u[i].get(j) * r[i] * w[j]));
    b[j] = scale_byte(top);
    uint32_t q[4];
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      float e[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) e[i] = u[8 * s + i].get(j) * r[8 * s + i] * w[j];
      q[s] = encode8(e, b[j]) & mask[s];
    }
    k[j] = make_uint4(q[0], q[1], q[2], q[3]);
    __builtin_amdgcn_sched_barrier(0);
  }
  // column j's line: chunk `wave` at position wave ^ (j / 2 % 8), so that the
  // 64 lanes' 16-byte writes spread over the banks
  const int pos = 16 * (wave ^ (lane & 7));
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    *reinterpret_cast<uint4*>(lc + (2 * lane + j) * 128 + pos) = k[j];
    ls[(2 * lane + j) * 8 + wave] = (uint8_t)b[j];
  }
  __syncthreads();
  for (int i = tid; i < kTileCols * 8; i += 512) {
    const int j = i >> 3, p = i & 7;             // column, 16-byte position
    if (c0 + j < C)
      *reinterpret_cast<uint4*>(codes + (g * C + c0 + j) * kPanelBytes + 16 * (p ^ ((j >> 1) & 7))) =
          *reinterpret_cast<const uint4*>(lc + j * 128 + 16 * p);
  }
  if (tid < kTileCols && c0 + tid < C)
    *reinterpret_cast<uint2*>(scales + (g * C + c0 + tid) * kPanelScales) = *reinterpret_cast<const uint2*>(ls + tid * 8);
}

// ---- gradients ------------------------------------------------------------------
//   xhat = h r, g = w dy, m = mean(g xhat)
//   dh = dh_in + r (g - xhat m);  dx = k dh / (1 - p);  dw = sum over tokens of dy xhat
// A workgroup takes every gridDim-th group of rows and keeps its columns' share
// of dw in registers; the shares are summed by norm_weight_kernel in a fixed
// order, so that the result is the same every time.  8192 x 4096 BF16 with dh in and
// dropout: 347 MB in 72 us (4.8 TB/s) and 4.6 us for the shares of 768 workgroups,
// three a CU; 333 x 1111 FP32 5.2 and 3.6 us, each a launch and its trips to memory.
// dh and, through the dropout, dx of eight columns of row t.
template <class H>
__device__ __forceinline__ void put_gradients(const NormBackward& a, int64_t t, int c, uint64_t seed, uint64_t offset,
                                              float (&d)[8]) {
  const int64_t at = t * a.C + c;
  store8u(static_cast<H*>(a.dh) + at, a.C - c, d);
  if (!a.dx) return;
  if (a.drop.rng) {
    const Mask8 mask((uint32_t)(c >> 3), (uint32_t)t, seed, offset);
#pragma unroll
    for (int i = 0; i < 8; ++i) d[i] = mask.keeps(i, a.drop.cut) ? d[i] * a.drop.scale : 0.0f;
  }
  store_as(a.dx, a.xt, at, a.C - c, d);
}

template <class D, class H, int LPR, int NV, bool TURNS>
__global__ __launch_bounds__(LPR < 256 ? 256 : LPR) void norm_backward_kernel(const NormBackward a) {
  constexpr int kThreads = LPR < 256 ? 256 : LPR, kRows = kThreads / LPR, kWaves = LPR / 64;
  __shared__ float sums[2][kWaves > 0 ? kWaves : 1];
  const int lane = threadIdx.x % LPR, sub = threadIdx.x / LPR;
  const int C = a.C;
  const float inv = 1.0f / (float)C;
  float dw[NV][8];
#pragma unroll
  for (int k = 0; k < NV; ++k)
#pragma unroll
    for (int i = 0; i < 8; ++i) dw[k][i] = 0.0f;
  uint64_t seed = 0, offset = 0;
  if (a.drop.rng) {
    seed = a.drop.rng[0];
    offset = a.drop.rng[1];
  }
  const int64_t step = (int64_t)gridDim.x * kRows;
  int buf = 0;
  for (int64_t t = (int64_t)blockIdx.x * kRows + sub; t < a.T; t += step) {
    const int64_t at = t * C;
    Raw8<D> dy[NV];
    Raw8<H> h[NV], in[NV];
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = 8 * (k * LPR + lane);
      dy[k].template load_row<TURNS>(static_cast<const D*>(a.dy) + at, c, C);
      h[k].template load_row<TURNS>(static_cast<const H*>(a.h) + at, c, C);
      if (a.dh_in) in[k].template load_row<TURNS>(static_cast<const H*>(a.dh_in) + at, c, C);
    }
    const float r = a.rstd[t];
    float m = 0.0f;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = 8 * (k * LPR + lane);
      float w[8];
      load_weights<TURNS>(a.w, a.wt, c, C, w);
      dy[k].template turn<TURNS>(c, C);
      h[k].template turn<TURNS>(c, C);
      if (a.dh_in) in[k].template turn<TURNS>(c, C);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float xhat = h[k].get(i) * r, p = dy[k].get(i) * xhat;
        // behind the row's end nothing, also beside an r that is not finite
        if (c + i < C) {
          m = fmaf(p, w[i], m);
          dw[k][i] += p;
        }
      }
    }
    m = wave_sum<(LPR < 64 ? LPR : 64)>(m);
    if constexpr (kWaves > 1) {
      // two buffers: a wave writes one again only behind the barrier of the
      // row between, when all have read it
      if ((lane & 63) == 0) sums[buf][lane >> 6] = m;
      __syncthreads();
      m = 0.0f;
#pragma unroll
      for (int i = 0; i < kWaves; ++i) m += sums[buf][i];
      buf ^= 1;
    }
    m *= inv;
#pragma unroll
    for (int k = 0; k < NV; ++k) {
      const int c = 8 * (k * LPR + lane);
      if (c >= C) break;
      float w[8], d[8];
      load_weights<TURNS>(a.w, a.wt, c, C, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float v = r * (dy[k].get(i) * w[i] - h[k].get(i) * r * m);
        d[i] = a.dh_in ? in[k].get(i) + v : v;
      }
      put_gradients<H>(a, t, c, seed, offset, d);
    }
  }
  if (!a.dw) return;
  if constexpr (kRows > 1) {
    // the rows' shares meet first
    __shared__ float shares[kRows][8][NV * LPR];
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i) shares[sub][i][k * LPR + lane] = dw[k][i];
    __syncthreads();
    if (sub) return;
#pragma unroll
    for (int k = 0; k < NV; ++k)
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int y = 1; y < kRows; ++y) dw[k][i] += shares[y][i][k * LPR + lane];
  }
  float* part = a.partials + (int64_t)blockIdx.x * C;
#pragma unroll
  for (int k = 0; k < NV; ++k) {
    const int c = 8 * (k * LPR + lane);
    if (c < C) store8u(part + c, C - c, dw[k]);
  }
}

// The same for rows of more than 8192 columns, for which a lane's registers
// would not do: 1024 lanes walk a row twice, the second time from the caches, and
// hold its columns' share of dw in LDS.  2048 x 16384 with dh in, both launches: BF16
// 67.5 us for 268 MB, FP32 131 us for 537 MB (4.0 and 4.1 TB/s); 2048 x 10240 BF16 51.
template <class D, class H, int V>
__global__ __launch_bounds__(1024) void norm_backward_wide_kernel(const NormBackward a) {
  __shared__ float share[V * 8 * 1024];
  __shared__ float sums[2][16];
  const int lane = threadIdx.x, C = a.C;
  const float inv = 1.0f / (float)C;
  for (int k = 0; k < 8 * V; ++k) share[k * 1024 + lane] = 0.0f;
  uint64_t seed = 0, offset = 0;
  if (a.drop.rng) {
    seed = a.drop.rng[0];
    offset = a.drop.rng[1];
  }
  int buf = 0;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    const int64_t at = t * C;
    const float r = a.rstd[t];
    float m = 0.0f;
#pragma unroll 1
    for (int k = 0; k < V; ++k) {
      const int c = 8 * (k * 1024 + lane);
      if (c >= C) break;
      Raw8<D> dy;
      Raw8<H> h;
      dy.load(static_cast<const D*>(a.dy) + at + c, C - c);
      h.load(static_cast<const H*>(a.h) + at + c, C - c);
      float w[8];
      load_weights<false>(a.w, a.wt, c, C, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (c + i >= C) break;
        const float p = dy.get(i) * (h.get(i) * r);
        m = fmaf(p, w[i], m);
        share[(8 * k + i) * 1024 + lane] += p;
      }
    }
    m = wave_sum(m);
    if ((lane & 63) == 0) sums[buf][lane >> 6] = m;
    __syncthreads();
    m = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) m += sums[buf][i];
    buf ^= 1;
    m *= inv;
#pragma unroll 1
    for (int k = 0; k < V; ++k) {
      const int c = 8 * (k * 1024 + lane);
      if (c >= C) break;
      Raw8<D> dy;
      Raw8<H> h, in;
      dy.load(static_cast<const D*>(a.dy) + at + c, C - c);
      h.load(static_cast<const H*>(a.h) + at + c, C - c);
      if (a.dh_in) in.load(static_cast<const H*>(a.dh_in) + at + c, C - c);
      float w[8], d[8];
      load_weights<false>(a.w, a.wt, c, C, w);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float v = r * (dy.get(i) * w[i] - h.get(i) * r * m);
        d[i] = a.dh_in ? in.get(i) + v : v;
      }
      put_gradients<H>(a, t, c, seed, offset, d);
    }
  }
  if (!a.dw) return;
  float* part = a.partials + (int64_t)blockIdx.x * C;
  for (int k = 0; k < V; ++k) {
    const int c = 8 * (k * 1024 + lane);
    if (c >= C) break;
    float d[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) d[i] = share[(8 * k + i) * 1024 + lane];
    store8u(part + c, C - c, d);
  }
}

// dw = beta dw + the partial rows: 32 columns a workgroup, 32 groups of rows.
__global__ __launch_bounds__(1024) void norm_weight_kernel(const float* part, int rows, int C, float beta, float* dw) {
  __shared__ float sums[32][33];
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5, c = (int)blockIdx.x * 32 + x;
  float s = 0.0f;
  if (c < C) {
#pragma unroll 8
    for (int p = y; p < rows; p += 32) s += part[(int64_t)p * C + c];
  }
  sums[y][x] = s;
  __syncthreads();
  if (y != 0 || c >= C) return;
  s = 0.0f;
#pragma unroll
  for (int i = 0; i < 32; ++i) s += sums[i][x];
  dw[c] = beta != 0.0f ? fmaf(beta, dw[c], s) : s;
}

// ---- dropout --------------------------------------------------------------------
// A lane's vectors are eight neighbours of a row, `nv` to a row; a workgroup
// takes a run of kDropVectors of them.  inv: 2^32 / nv rounded up, exact for
// quotients below 2 kDropVectors / nv where nv < kDropVectors.
// 8192 x 11008 BF16: 361 MB in 69 us, 5.2 TB/s as a copy; vector instructions, most
// of them the generator's (one call for eight elements), fill 63% of the cycles
// behind it.  777 x 1501 FP32 5.4 us.
constexpr int kDropUnroll = 4, kDropVectors = 256 * kDropUnroll;

template <class X>
__global__ __launch_bounds__(256) void dropout_kernel(const X* x, int64_t rows, int64_t cols, uint32_t nv, uint32_t inv,
                                                      Drop d, X* out) {
  const uint64_t seed = d.rng[0], offset = d.rng[1];
  const uint64_t v0 = (uint64_t)blockIdx.x * kDropVectors;
  const uint64_t row0 = v0 / nv;
  const uint32_t first = (uint32_t)(v0 - row0 * nv);
  Raw8<X> raw[kDropUnroll];
  int64_t at[kDropUnroll];
  uint32_t row[kDropUnroll], vec[kDropUnroll];
  int n[kDropUnroll];
#pragma unroll
  for (int k = 0; k < kDropUnroll; ++k) {
    const uint32_t v = first + (uint32_t)(k * 256 + threadIdx.x);
    // v < nv + kDropVectors: one subtraction where a row is longer than that
    const uint32_t q = nv >= (uint32_t)kDropVectors ? (v >= nv ? 1u : 0u) : (nv == 1 ? v : __umulhi(v, inv));
    vec[k] = v - q * nv;
    const int64_t t = (int64_t)row0 + q;
    row[k] = (uint32_t)t;
    at[k] = t * cols + 8 * (int64_t)vec[k];
    const int64_t left = cols - 8 * (int64_t)vec[k];
    n[k] = t < rows ? (left < 8 ? (int)left : 8) : 0;
    raw[k].load(x + at[k], n[k]);
  }
#pragma unroll
  for (int k = 0; k < kDropUnroll; ++k) {
    const Mask8 m(vec[k], row[k], seed, offset);
    float v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = m.keeps(i, d.cut) ? raw[k].get(i) * d.scale : 0.0f;
    if (n[k]) store8u(out + at[k], n[k], v);
  }
}

template <class X>
hipError_t dropout(const X* x, int64_t rows, int64_t cols, const Drop& d, X* out, hipStream_t s) {
  const uint32_t nv = (uint32_t)((cols + 7) / 8);
  const uint64_t blocks = ((uint64_t)rows * nv + kDropVectors - 1) / kDropVectors;
  const uint32_t inv = nv > 1 ? (uint32_t)((((uint64_t)1 << 32) + nv - 1) / nv) : 0;
  dropout_kernel<X><<<dim3((unsigned)blocks), 256, 0, s>>>(x, rows, cols, nv, inv, d, out);
  return hipGetLastError();
}

// ---- launches -------------------------------------------------------------------
template <class X, class H, int LPR, int NV>
hipError_t forward(const NormForward& a, hipStream_t s) {
  constexpr int kThreads = LPR < 256 ? 256 : LPR, kRows = kThreads / LPR;
  const dim3 grid((unsigned)((a.T + kRows - 1) / kRows));
  if (turns(a.C)) norm_kernel<X, H, LPR, NV, true><<<grid, kThreads, 0, s>>>(a);
  else norm_kernel<X, H, LPR, NV, false><<<grid, kThreads, 0, s>>>(a);
  return hipGetLastError();
}
// Lanes and vectors that hold a row: an eighth, a quarter or half of a wave up to a
// panel (262144 x 128 BF16: a wave 95 us, half 53, a quarter 31, of 134 MB), a wave
// up to 1024 columns, then a workgroup, which needs a barrier but leaves registers
// for other workgroups.
template <class X, class H>
hipError_t forward_by_width(const NormForward& a, hipStream_t s) {
  if (a.C <= 64) return forward<X, H, 8, 1>(a, s);
  if (a.C <= 128) return forward<X, H, 16, 1>(a, s);
  if (a.C <= kPanel) return forward<X, H, 32, 1>(a, s);
  if (a.C <= 512) return forward<X, H, 64, 1>(a, s);
  if (a.C <= 1024) return forward<X, H, 64, 2>(a, s);
  if (a.C <= 2048) return forward<X, H, 256, 1>(a, s);
  if (a.C <= 4096) return forward<X, H, 256, 2>(a, s);
  if (a.C <= 8192) return forward<X, H, 256, 4>(a, s);
  if (a.C <= 16384) return forward<X, H, 1024, 2>(a, s);
  return forward<X, H, 1024, 4>(a, s);
}

constexpr int64_t kBackwardGroups = 768;     // workgroups at most, three a CU
int64_t backward_groups(int64_t T, int64_t C) {
  if (C > 8192) return T < 256 ? T : 256;    // of 1024 lanes, one a CU
  const int rows = C <= 64 ? 32 : C <= 128 ? 16 : C <= kPanel ? 8 : C <= 1024 ? 4 : 1;
  const int64_t n = (T + rows - 1) / rows;
  return n < kBackwardGroups ? n : kBackwardGroups;
}

template <class D, class H, int LPR, int NV>
hipError_t backward(const NormBackward& a, hipStream_t s) {
  const dim3 grid((unsigned)backward_groups(a.T, a.C)), block(LPR < 256 ? 256 : LPR);
  if (turns(a.C)) norm_backward_kernel<D, H, LPR, NV, true><<<grid, block, 0, s>>>(a);
  else norm_backward_kernel<D, H, LPR, NV, false><<<grid, block, 0, s>>>(a);
  return hipGetLastError();
}
template <class D, class H>
hipError_t backward_by_width(const NormBackward& a, hipStream_t s) {
  if (a.C <= 64) return backward<D, H, 8, 1>(a, s);
  if (a.C <= 128) return backward<D, H, 16, 1>(a, s);
  if (a.C <= kPanel) return backward<D, H, 32, 1>(a, s);
  if (a.C <= 512) return backward<D, H, 64, 1>(a, s);
  if (a.C <= 1024) return backward<D, H, 64, 2>(a, s);
  if (a.C <= 2048) return backward<D, H, 256, 1>(a, s);
  if (a.C <= 4096) return backward<D, H, 256, 2>(a, s);
  if (a.C <= 8192) return backward<D, H, 256, 4>(a, s);
  const dim3 grid((unsigned)backward_groups(a.T, a.C));
  if (a.C <= 16384) norm_backward_wide_kernel<D, H, 2><<<grid, 1024, 0, s>>>(a);
  else norm_backward_wide_kernel<D, H, 4><<<grid, 1024, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_dropout(const void* x, Dt t, int64_t rows, int64_t cols, const Drop& d, void* out, hipStream_t s) {
  return t == Dt::F32 ? dropout(static_cast<const float*>(x), rows, cols, d, static_cast<float*>(out), s)
                      : dropout(static_cast<const uint16_t*>(x), rows, cols, d, static_cast<uint16_t*>(out), s);
}

hipError_t launch_norm(const NormForward& n, hipStream_t s) {
  if (n.C < 1 || n.C > kNormMaxCols) return hipErrorInvalidValue;
  if (n.xt == Dt::F32)
    return n.ht == Dt::F32 ? forward_by_width<float, float>(n, s) : forward_by_width<float, uint16_t>(n, s);
  return n.ht == Dt::F32 ? forward_by_width<uint16_t, float>(n, s) : forward_by_width<uint16_t, uint16_t>(n, s);
}

hipError_t launch_norm_cols(const void* h, Dt ht, const float* rstd, const void* w, Dt wt, int64_t T, int64_t C,
                            uint8_t* codes, uint8_t* scales, hipStream_t s) {
  const uint32_t tiles = (uint32_t)((C + kTileCols - 1) / kTileCols);
  const dim3 grid(tiles * (uint32_t)((T + kPanel - 1) / kPanel));
  auto go = [&](auto* p) {
    if (C % 2 == 0) norm_cols_kernel<std::remove_cv_t<std::remove_pointer_t<decltype(p)>>, true><<<grid, 512, 0, s>>>(p, rstd, w, wt, T, C, tiles, codes, scales);
    else norm_cols_kernel<std::remove_cv_t<std::remove_pointer_t<decltype(p)>>, false><<<grid, 512, 0, s>>>(p, rstd, w, wt, T, C, tiles, codes, scales);
  };
  if (ht == Dt::F32) go(static_cast<const float*>(h));
  else go(static_cast<const uint16_t*>(h));
  return hipGetLastError();
}

int64_t norm_partials(int64_t T, int64_t C) { return backward_groups(T, C); }

hipError_t launch_norm_backward(const NormBackward& n, hipStream_t s) {
  if (n.C < 1 || n.C > kNormMaxCols) return hipErrorInvalidValue;
  hipError_t e;
  if (n.dyt == Dt::F32)
    e = n.ht == Dt::F32 ? backward_by_width<float, float>(n, s) : backward_by_width<float, uint16_t>(n, s);
  else
    e = n.ht == Dt::F32 ? backward_by_width<uint16_t, float>(n, s) : backward_by_width<uint16_t, uint16_t>(n, s);
  if (e != hipSuccess || !n.dw) return e;
  norm_weight_kernel<<<dim3((unsigned)((n.C + 31) / 32)), 1024, 0, s>>>(n.partials, (int)norm_partials(n.T, n.C), n.C, n.beta, n.dw);
  return hipGetLastError();
}

}  // namespace nvfp4

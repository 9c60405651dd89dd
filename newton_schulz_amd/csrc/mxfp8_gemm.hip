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
// holds it): the seven smaller ones of a group lose at most 7 * 2^-13 of the
// largest.  BF16 outputs, off by up to 2^-8 themselves, take that: 1.2% of those of
// 8192 x 11008 x 4096 are not the exact sum's nearest, and the relative error
// against 64 bits is 0.0016615 in place of 0.0016608.  FP32 outputs, and the
// product of few rows, which waits for memory anyway, take P in two parts, codes
// from 2 on and below: each spans 8 exponents, and 7 + 4 + 2 bits fit the window
// exactly.
#include <algorithm>

#include "dma.hpp"
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

// Sixteen rows of Q a workgroup, up to 16 rows of P; the waves divide the
// panels of K and have DEEP of them in flight; their sums meet in LDS, in wave
// order.  1 x 11008 x 4096: 24 MB in 8.0 us, a launch and one round of 688 workgroups
// that all wait for their first lines; the matrix units are busy a tenth of it.
template <Dt OT, int WAVES, int DEEP>
__global__ __launch_bounds__(64 * WAVES) void few8_kernel(const Product8 g, int panels) {
  __shared__ floatx4 sums[WAVES][64];
  const int lane = threadIdx.x & 63, r = lane & 15, q = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int n0 = (int)blockIdx.x * 16;
  const int M = (int)g.M, N = (int)g.N;
  // rows behind an operand's end read its last row: not written
  const int64_t row = n0 + r < N ? n0 + r : N - 1, prow = r < M ? r : M - 1;
  const int p0 = panels * wave / WAVES, p1 = panels * (wave + 1) / WAVES;
  floatx4 acc = floatx4{0, 0, 0, 0};
  for (int p = p0; p < p1; p += DEEP) {
    intx4 wc[DEEP][2];
    uint2 ws[DEEP], xs[DEEP];
    intx8 xc[DEEP][2];
#pragma unroll
    for (int i = 0; i < DEEP; ++i) {
      const int64_t pi = p + i < p1 ? p + i : p1 - 1;       // the last again: not multiplied
      const uint8_t* c = g.q + (pi * N + row) * kPanelBytes + 16 * q;
      wc[i][0] = *reinterpret_cast<const intx4*>(c);
      wc[i][1] = *reinterpret_cast<const intx4*>(c + 64);
      ws[i] = *reinterpret_cast<const uint2*>(g.q_scales + (pi * N + row) * kPanelScales);
      const uint8_t* x = g.p + (pi * M + prow) * kPanelBytes8 + 16 * q;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const intx4 lo = *reinterpret_cast<const intx4*>(x + 128 * u), hi = *reinterpret_cast<const intx4*>(x + 128 * u + 64);
        xc[i][u] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
      }
      xs[i] = *reinterpret_cast<const uint2*>(g.p_scales + (pi * M + prow) * kPanelScales);
    }
#pragma unroll
    for (int i = 0; i < DEEP; ++i) {
      if (p + i >= p1) break;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        intx8 high, low;
        two_parts(xc[i][u], high, low);
        const int sw = (int)((u ? ws[i].y : ws[i].x) >> (8 * q)), sx = (int)((u ? xs[i].y : xs[i].x) >> (8 * q));
        acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(four_bits(wc[i][u]), high, acc, 4, 0, 0, sw, 0, sx);
        acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(four_bits(wc[i][u]), low, acc, 4, 0, 0, sw, 0, sx);
      }
    }
  }
  sums[wave][lane] = acc;
  __syncthreads();
  // lane: rows n0 + 4 q .. + 3 of Q, row r of P
  if (wave) return;
  const int n = n0 + 4 * q;
  if (r >= M || n >= N) return;
  floatx4 v = sums[0][lane];
  for (int w = 1; w < WAVES; ++w) v += sums[w][lane];
  put4<OT>(g, (int64_t)r * N + n, N - n, N % 4 == 0, v);
}

template <Dt OT>
hipError_t few(const Product8& g, hipStream_t s) {
  const int panels = (int)((g.K + kPanel - 1) / kPanel);
  const dim3 grid((unsigned)((g.N + 15) / 16));
  // enough waves to cover the chip several times, none without a panel
  if (grid.x < 512 && panels >= 16) few8_kernel<OT, 16, 1><<<grid, 1024, 0, s>>>(g, panels);
  else few8_kernel<OT, 4, 4><<<grid, 256, 0, s>>>(g, panels);
  return hipGetLastError();
}

// ---- tiles ----------------------------------------------------------------------
// A stage is one panel (256 of K) of the tile's rows in lines of 128 bytes: the
// first halves of P's rows, their second halves, Q's rows; behind them the
// scales, eight bytes a row.  Chunk c of row r lies at position c ^ swizzle(r) of
// its line, so that 32 lanes reading one chunk of 32 rows hit distinct banks.
// Step s of four multiplies blocks s and 4 + s of every row: of a row of Q a
// lane of half h takes block 4 h + s (chunk 4 h + s), of a row of P sixteen bytes
// of either block (chunk 2 s + h of both lines), and the scales are byte s of
// word h.
//
// Workgroups stay for as many tiles as there are per slot, and the stages of
// their tiles form one stream through the buffers, so that a tile's first panel
// loads while the tile before leaves.  8192 x 11008 x 4096 on 128 x 256 tiles took
// 310 us with the matrix units busy 63% of the cycles; 1000 x 777 x 1501 in FP32
// takes 10 us on 64 x 64, six panels of 1 us behind a launch and the first trip to
// memory.
template <int BM_, int BN_, int WM_, int WN_, int NST_>
struct Tile {
  static constexpr int BM = BM_, BN = BN_, WM = WM_, WN = WN_, NST = NST_;
  static constexpr int kWaves = WM * WN, kThreads = 64 * kWaves;
  static constexpr int FM = BM / (32 * WM), FN = BN / (32 * WN);
  static constexpr int kLines = 2 * BM + BN, kCodeBytes = kLines * 128;
  static constexpr int kCodeLoads = kLines / 8 / kWaves;           // DMA instructions a wave and stage
  static constexpr int kScaleGroups = (BM + BN) / 32;              // 256 bytes each
  static constexpr int kScaleLoads = (kScaleGroups + kWaves - 1) / kWaves;
  static constexpr int kStage = kCodeBytes + kScaleGroups * 256;
  static constexpr int kScratch = 2304;                            // of a wave's epilogue: 576 floats
  static constexpr int kLds = NST * kStage + kWaves * kScratch;
  static_assert(kCodeLoads * 8 * kWaves == kLines && BM % 8 == 0, "uneven loads");
};

// A unit is K-part `u / tiles` of tile u % tiles, `per` panels of it.
struct Args {
  Product8 g;
  int panels, per, TM, TN, tiles, units, slots;       // slots: workgroups per XCD
  float* partials;                                    // [parts][M][N], with more than one part
};

constexpr int kXcds = 8, kCusPerXcd = 32, kStrip = 4;

// The kernel's arguments read again: what the epilogue needs of them would
// otherwise wait in scalar registers through the whole product, and spill.
__device__ __forceinline__ const Product8& product_again() {
  uint64_t at = (uint64_t)(uintptr_t)__builtin_amdgcn_kernarg_segment_ptr();
  asm volatile("" : "+s"(at));
  return *(const Product8*)(const __attribute__((address_space(4))) Product8*)at;
}

// Strips of kStrip tile rows, column by column within a strip.
__device__ __forceinline__ void place_of(const Args& a, int u, int& I, int& J, int& part) {
  part = __builtin_amdgcn_readfirstlane(u / a.tiles);
  int t = u - part * a.tiles;
  const int s = t / (kStrip * a.TN) * kStrip, w = a.TM - s < kStrip ? a.TM - s : kStrip;
  t -= s * a.TN;
  I = __builtin_amdgcn_readfirstlane(s + t % w);
  J = __builtin_amdgcn_readfirstlane(t / w);
}

// Where a workgroup's loads stand: tile and next panel, and the byte offsets of
// a lane's loads from the tile's first row.  Rows past an operand's end read its
// last row: they feed only values that are not written.
template <class C>
struct Loads {
  static constexpr int kLoads = C::kCodeLoads + C::kScaleLoads;
  // whether every wave's loads are of one operand: then `p` and `ps` stand for it
  static constexpr bool kOne = C::BM % (8 * C::kCodeLoads) == 0 && C::BM / 32 % C::kScaleLoads == 0;
  int u, g, end;                          // unit, next panel and the unit's last + 1
  const uint8_t *p, *q, *ps, *qs;         // the tile's first rows in panel g
  uint32_t code[C::kCodeLoads], scale[C::kScaleLoads];

  static __device__ __forceinline__ int scale_group(int wave, int k) {
    const int n = wave * C::kScaleLoads + k;              // the last groups twice where they do not divide
    return n < C::kScaleGroups ? n : C::kScaleGroups - 1;
  }
  __device__ __forceinline__ void start(const Args& a, int unit, int wave, int lane) {
    int I, J, part;
    place_of(a, unit, I, J, part);
    u = unit;
    g = part * a.per;
    end = g + a.per < a.panels ? g + a.per : a.panels;
    const int64_t m0 = (int64_t)I * C::BM, n0 = (int64_t)J * C::BN;
    p = a.g.p + (g * a.g.M + m0) * kPanelBytes8;
    q = a.g.q + (g * a.g.N + n0) * kPanelBytes;
    ps = a.g.p_scales + (g * a.g.M + m0) * kPanelScales;
    qs = a.g.q_scales + (g * a.g.N + n0) * kPanelScales;
    if constexpr (kOne) {
      if (8 * wave * C::kCodeLoads >= 2 * C::BM) p = q;
      if (32 * wave * C::kScaleLoads >= C::BM) ps = qs;
    }
    const int pm = (int)(a.g.M - m0 < C::BM ? a.g.M - m0 : C::BM) - 1, qm = (int)(a.g.N - n0 < C::BN ? a.g.N - n0 : C::BN) - 1;
    auto place = [&](int k, bool isP, int first, int half) {
      const int r = first + (lane >> 3), last = isP ? pm : qm;
      const uint32_t row = (uint32_t)(r < last ? r : last);
      code[k] = (isP ? row * kPanelBytes8 + 128u * half : row * kPanelBytes) + 16u * (uint32_t)((lane & 7) ^ swizzle(r));
    };
    const int line0 = 8 * wave * C::kCodeLoads;
    if constexpr (kOne) {
      // one operand, and of P one half of its rows
      const bool isP = line0 < 2 * C::BM;
      const int half = isP && line0 >= C::BM, first = isP ? line0 - half * C::BM : line0 - 2 * C::BM;
#pragma unroll
      for (int k = 0; k < C::kCodeLoads; ++k) place(k, isP, first + 8 * k, half);
    } else {
#pragma unroll
      for (int k = 0; k < C::kCodeLoads; ++k) {
        const int line = line0 + 8 * k;
        const bool isP = line < 2 * C::BM;
        place(k, isP, isP ? line % C::BM : line - 2 * C::BM, line >= C::BM);
      }
    }
#pragma unroll
    for (int k = 0; k < C::kScaleLoads; ++k) {
      const int n = 32 * scale_group(wave, k), r = (n < C::BM ? n : n - C::BM) + (lane >> 1), last = n < C::BM ? pm : qm;
      scale[k] = (uint32_t)(r < last ? r : last) * kPanelScales + 4u * (uint32_t)(lane & 1);
    }
  }
  // Load number k of the wave's share into the stage at LDS address `stage`.
  __device__ __forceinline__ void load(uint32_t stage, int wave, int k) const {
    if (k < C::kCodeLoads) {
      const int n = wave * C::kCodeLoads + k;
      dma16(kOne || 8 * n < 2 * C::BM ? p : q, code[k], stage + (uint32_t)n * 1024u);
    } else {
      const int n = scale_group(wave, k - C::kCodeLoads);
      dma4(kOne || 32 * n < C::BM ? ps : qs, scale[k - C::kCodeLoads], stage + (uint32_t)(C::kCodeBytes + 256 * n));
    }
  }
  // To the next panel: of this unit, of the workgroup's next one, or, behind
  // the last, the same again (into a buffer that nothing reads).
  __device__ __forceinline__ void advance(const Args& a, int units, int wave, int lane) {
    if (g + 1 < end) {
      ++g;
      if constexpr (kOne) {
        p += 8 * wave * C::kCodeLoads < 2 * C::BM ? a.g.M * kPanelBytes8 : a.g.N * kPanelBytes;
        ps += (32 * wave * C::kScaleLoads < C::BM ? a.g.M : a.g.N) * kPanelScales;
      } else {
        p += a.g.M * kPanelBytes8;
        q += a.g.N * kPanelBytes;
        ps += a.g.M * kPanelScales;
        qs += a.g.N * kPanelScales;
      }
    } else if (u + a.slots < units) {
      start(a, u + a.slots, wave, renewed(lane));
    }
  }
};

template <class C>
struct Frags {
  intx4 q[C::FN];
  intx4 p[C::FM][2];
};
template <class C>
struct Scales {
  uint32_t q[C::FN], p[C::FM];
};

// Read number k of a step: Q's fragments, then the halves of P's.
template <class C>
__device__ __forceinline__ void read_frag(const uint8_t* st, uint32_t qo, uint32_t po, int wm, int wn, int k, Frags<C>& f) {
  if (k < C::FN) {
    f.q[k] = *reinterpret_cast<const intx4*>(st + qo + (2 * C::BM + (wn * C::FN + k) * 32) * 128);
  } else {
    const int i = (k - C::FN) >> 1, half = (k - C::FN) & 1;
    f.p[i][half] = *reinterpret_cast<const intx4*>(st + po + (half * C::BM + (wm * C::FM + i) * 32) * 128);
  }
}
template <class C>
__device__ __forceinline__ void read_scale(const uint8_t* st, uint32_t off, int wm, int wn, int k, Scales<C>& f) {
  st += C::kCodeBytes;
  if (k < C::FN) f.q[k] = *reinterpret_cast<const uint32_t*>(st + off + (C::BM + (wn * C::FN + k) * 32) * 8);
  else if (k < C::FN + C::FM) f.p[k - C::FN] = *reinterpret_cast<const uint32_t*>(st + off + (wm * C::FM + k - C::FN) * 32 * 8);
}

__device__ __forceinline__ constexpr int share(int total, int k, int n) { return total * k / n; }

// One step's matrix instructions; `between(k)` puts memory operations behind
// the k-th block's, and the compiler keeps this order.
template <class C, bool EXACT, int S, class F>
__device__ __forceinline__ void step(const Frags<C>& f, const Scales<C>& sc, floatx16 (&acc)[C::FM][C::FN], F&& between) {
#pragma unroll
  for (int i = 0; i < C::FM; ++i) {
    const intx8 x = __builtin_shufflevector(f.p[i][0], f.p[i][1], 0, 1, 2, 3, 4, 5, 6, 7);
    intx8 high, low;
    if constexpr (EXACT) two_parts(x, high, low);
#pragma unroll
    for (int j = 0; j < C::FN; ++j) {
      if constexpr (EXACT) {
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(high, four_bits(f.q[j]), acc[i][j], 0, 4, S, (int)sc.p[i], S, (int)sc.q[j]);
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(low, four_bits(f.q[j]), acc[i][j], 0, 4, S, (int)sc.p[i], S, (int)sc.q[j]);
      } else {
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, four_bits(f.q[j]), acc[i][j], 0, 4, S, (int)sc.p[i], S, (int)sc.q[j]);
      }
      __builtin_amdgcn_sched_barrier(0);
      between(i * C::FN + j);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
}

// beta addend + alpha v of eight neighbours, or the first n, rounded once.
template <Dt OT>
__device__ __forceinline__ void put8(const Product8& g, int64_t at, int n, float (&v)[8]) {
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] *= g.alpha;
  if (g.addend) {
    Raw8<float> o;
    o.load(g.addend + at, n);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = fmaf(g.beta, o.get(e), v[e]);
  }
  if constexpr (OT == Dt::F32) store8u(static_cast<float*>(g.out) + at, n, v);
  else store8u(static_cast<uint16_t*>(g.out) + at, n, v);
}

// acc[i][j][4 q + t] of a lane is row (wm FM + i) 32 + 8 q + 4 (lane / 32) + t,
// column (wn FN + j) 32 + lane % 32 of the tile.  Eight rows of two blocks, or
// sixteen of one, at a time pass through the wave's own LDS, from where a lane
// takes eight neighbours of a row.
// Two blocks' rows end inside fewer lines than one's: 5366 x 10987 x 60 with an
// addend 151 us, one by one 201.
// PART: as they are, to a part's own [M][N].
template <class C, Dt OT, bool PART>
__device__ __forceinline__ void epilogue(const Product8& g, float* part, const floatx16 (&acc)[C::FM][C::FN], int64_t m0, int64_t n0, int wm,
                                         int wn, int lane, uint8_t* lds) {
  constexpr int kPair = C::FN % 2 == 0 ? 2 : 1, kPitch = kPair == 2 ? 72 : 36, kQs = 2 / kPair, kLanes = 4 * kPair;
  float* t = reinterpret_cast<float*>(lds);
#pragma unroll
  for (int i = 0; i < C::FM; ++i)
#pragma unroll
    for (int q0 = 0; q0 < 4; q0 += kQs)
#pragma unroll
      for (int j = 0; j < C::FN; j += kPair) {
        const int el = renewed(lane), h = el >> 5, c = el & 31, r = el / kLanes, c8 = el % kLanes * 8;
#pragma unroll
        for (int q = 0; q < kQs; ++q)
#pragma unroll
          for (int u = 0; u < kPair; ++u)
#pragma unroll
            for (int s = 0; s < 4; ++s) t[(8 * q + 4 * h + s) * kPitch + 32 * u + c] = acc[i][j + u][4 * (q0 + q) + s];
        wave_sync();
        float v[8];
        const float4 lo = *reinterpret_cast<const float4*>(t + r * kPitch + c8);
        const float4 hi = *reinterpret_cast<const float4*>(t + r * kPitch + c8 + 4);
        v[0] = lo.x; v[1] = lo.y; v[2] = lo.z; v[3] = lo.w;
        v[4] = hi.x; v[5] = hi.y; v[6] = hi.z; v[7] = hi.w;
        const int64_t row = m0 + (wm * C::FM + i) * 32 + 8 * q0 + r, col = n0 + (wn * C::FN + j) * 32 + c8;
        if (row < g.M && col < g.N) {
          const int64_t at = row * g.N + col;
          const int n = g.N - col < 8 ? (int)(g.N - col) : 8;
          if constexpr (PART) store8u(part + at, n, v);
          else put8<OT>(g, at, n, v);
        }
        wave_sync();
        __builtin_amdgcn_sched_barrier(0);
      }
}

template <class C, Dt OT, bool PART>
__global__ __launch_bounds__(C::kThreads, C::kWaves / 4) void tile8_kernel(const Args a) {
  constexpr bool kExact = OT == Dt::F32;
  __shared__ __attribute__((aligned(16))) uint8_t smem[C::kLds];
  // one contiguous run of units an XCD
  const int x = (int)blockIdx.x % kXcds;
  const int end = (int)((int64_t)(x + 1) * a.units / kXcds);
  int unit = (int)((int64_t)x * a.units / kXcds) + (int)blockIdx.x / kXcds;
  if (unit >= end) return;
  const int lane = threadIdx.x & 63, r = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / C::WN, wn = wave % C::WN;
  uint8_t* scratch = smem + C::NST * C::kStage + wave * C::kScratch;

  floatx16 acc[C::FM][C::FN];
  Loads<C> next;
  next.start(a, unit, wave, lane);
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_addr(smem));
  constexpr int kLoads = Loads<C>::kLoads, kReads = C::FN + 2 * C::FM, kMul = C::FM * C::FN;
  uint32_t qo[4], po[4];
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    qo[s] = (uint32_t)(r * 128 + 16 * ((4 * h + s) ^ swizzle(r)));
    po[s] = (uint32_t)(r * 128 + 16 * ((2 * s + h) ^ swizzle(r)));
  }
  const uint32_t so = (uint32_t)(r * 8 + 4 * h);
  Frags<C> f0, f1;
  Scales<C> sc;
  // all but the newest NST - 2 stages' loads of this wave have landed
  auto wait_loads = [&] { asm volatile("s_waitcnt vmcnt(%0)" ::"n"((C::NST - 2) * kLoads) : "memory"); };

  // NST - 1 stages in flight before the first is read, then always NST
#pragma unroll 1
  for (int s = 0; s < C::NST - 1; ++s) {
#pragma unroll
    for (int k = 0; k < kLoads; ++k) next.load(lds0 + s * C::kStage, wave, k);
    next.advance(a, end, wave, lane);
  }
  wait_loads();
  all_waves();
#pragma unroll
  for (int k = 0; k < kLoads; ++k) next.load(lds0 + (C::NST - 1) * C::kStage, wave, k);
#pragma unroll
  for (int k = 0; k < kReads; ++k) {
    read_scale<C>(smem, so, wm, wn, k, sc);
    read_frag<C>(smem, qo[0], po[0], wm, wn, k, f0);
  }

  int cur = 0;
  for (; unit < end; unit += a.slots) {
    int I, J, part;
    place_of(a, unit, I, J, part);
    const int n = a.panels - part * a.per < a.per ? a.panels - part * a.per : a.per;
#pragma unroll
    for (int i = 0; i < C::FM; ++i)
#pragma unroll
      for (int j = 0; j < C::FN; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
    for (int g = 0; g < n; ++g) {
      // here, not behind the loads: a branch behind the matrix instructions
      // would let the compiler sink them past it
      next.advance(a, end, wave, lane);
      const uint8_t* st = smem + cur * C::kStage;
      auto ahead = [&](int s, Frags<C>& f) {
        return [&, s](int k) {
#pragma unroll
          for (int n = share(kReads, k, kMul); n < share(kReads, k + 1, kMul); ++n)
            read_frag<C>(st, qo[s], po[s], wm, wn, n, f);
        };
      };
      step<C, kExact, 0>(f0, sc, acc, ahead(1, f1));
      step<C, kExact, 1>(f1, sc, acc, ahead(2, f0));
      step<C, kExact, 2>(f0, sc, acc, ahead(3, f1));
      // every read of this stage has returned: its buffer is free once all
      // waves are here, and the next stage's loads have landed
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      wait_loads();
      all_waves();
      const uint32_t freed = lds0 + cur * C::kStage;
      cur = cur + 1 == C::NST ? 0 : cur + 1;
      const uint8_t* nst = smem + cur * C::kStage;
      Scales<C> nsc;
      step<C, kExact, 3>(f1, sc, acc, [&](int k) {
#pragma unroll
        for (int n = share(kReads, k, kMul); n < share(kReads, k + 1, kMul); ++n) {
          read_scale<C>(nst, so, wm, wn, n, nsc);
          read_frag<C>(nst, qo[0], po[0], wm, wn, n, f0);
        }
#pragma unroll
        for (int n = share(kLoads, k, kMul); n < share(kLoads, k + 1, kMul); ++n) next.load(freed, wave, n);
      });
      sc = nsc;
    }
    const Product8& p = product_again();
    epilogue<C, OT, PART>(p, PART ? a.partials + part * p.M * p.N : nullptr, acc, (int64_t)I * C::BM, (int64_t)J * C::BN, wm,
                          wn, renewed(lane), scratch);
  }
  // the loads behind the last stage write LDS until they land
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

// ---- large tiles ----------------------------------------------------------------
// 256 x 256 a workgroup, eight waves of 64 x 128: two thirds of the bytes from
// LDS an instruction that the tiles above read, and three quarters of the bytes
// into it.  LDS holds two panels of Q's rows and scales, and of P's rows two
// halves of a panel (blocks 4 u to 4 u + 3, a line of 128 bytes a row), which
// follow each other: while half u is multiplied, the other half lands.  Step s
// of a half multiplies blocks 4 u + 2 s (slot 0) and 4 u + 2 s + 1 (slot 1).
// 8192 x 11008 x 4096, BF16 out: 739 GFLOP in 284 us (304 in the first hundred calls
// after a pause), 67% of the 3.87 PFLOP/s that the bare instruction reaches on
// random codes; the matrix units are busy 73% of the cycles.  FP32 out 520 us.  With half of the loads into LDS left out it
// took 14% less, with operands that stay in L2 8% less.
namespace wide {
constexpr int B = 256, kWaves = 8, WN = 2, FM = 2, FN = 4;
constexpr int kHalf = B * 128, kQ = 2 * kHalf, kPanelQ = B * 128, kScales = kQ + 2 * kPanelQ, kPanelS = 2 * B * 8;
constexpr int kScratch = 2304, kLds = kScales + 2 * kPanelS + kWaves * kScratch;
constexpr int kLoads = 4, kScaleLoads = 2;       // a wave's of a half of P or a panel of Q, and of a panel's scales

// The next panel of a workgroup's stream of tiles: of P's rows, or of Q's rows and
// both operands' scales.  Behind the last panel the same again.
template <bool P>
struct Cursor {
  int t, g;
  const uint8_t *data, *s;
  uint32_t code[kLoads], scale[P ? 1 : kScaleLoads];

  __device__ __forceinline__ void start(const Args& a, int tile, int wave, int lane) {
    int I, J, part;
    place_of(a, tile, I, J, part);
    t = tile;
    g = 0;
    const int64_t m0 = (int64_t)I * B, n0 = (int64_t)J * B;
    // rows past an operand's end: its last row, into values that are not written
    const int pm = (int)(a.g.M - m0 < B ? a.g.M - m0 : B) - 1, qm = (int)(a.g.N - n0 < B ? a.g.N - n0 : B) - 1;
    data = P ? a.g.p + m0 * kPanelBytes8 : a.g.q + n0 * kPanelBytes;
    const int last = P ? pm : qm;
#pragma unroll
    for (int k = 0; k < kLoads; ++k) {
      const int r = 8 * (wave * kLoads + k) + (lane >> 3);
      code[k] = (uint32_t)(r < last ? r : last) * (P ? kPanelBytes8 : kPanelBytes) + 16u * (uint32_t)((lane & 7) ^ swizzle(r));
    }
    if constexpr (!P) {
      // groups of 32 rows: P's eight, then Q's
      const int slast = wave < 4 ? pm : qm;
      s = wave < 4 ? a.g.p_scales + m0 * kPanelScales : a.g.q_scales + n0 * kPanelScales;
#pragma unroll
      for (int k = 0; k < kScaleLoads; ++k) {
        const int r = 32 * ((wave & 3) * kScaleLoads + k) + (lane >> 1);
        scale[k] = (uint32_t)(r < slast ? r : slast) * kPanelScales + 4u * (uint32_t)(lane & 1);
      }
    }
  }
  __device__ __forceinline__ void advance(const Args& a, int end, int wave, int lane) {
    if (g + 1 < a.panels) {
      ++g;
      data += P ? a.g.M * kPanelBytes8 : a.g.N * kPanelBytes;
      if constexpr (!P) s += (wave < 4 ? a.g.M : a.g.N) * kPanelScales;
    } else if (t + a.slots < end) {
      start(a, t + a.slots, wave, renewed(lane));
    }
  }
  // Load number k of half u of P, or of Q's panel and the scales into buffer b.
  __device__ __forceinline__ void load(uint32_t lds0, int ub, int wave, int k) const {
    if constexpr (P) dma16(data + 128 * ub, code[k], lds0 + (uint32_t)(ub * kHalf + (wave * kLoads + k) * 1024));
    else if (k < kLoads) dma16(data, code[k], lds0 + (uint32_t)(kQ + ub * kPanelQ + (wave * kLoads + k) * 1024));
    else dma4(s, scale[k - kLoads], lds0 + (uint32_t)(kScales + ub * kPanelS + (wave * kScaleLoads + k - kLoads) * 256));
  }
};

struct Blocks {                          // of a wave, for the epilogue
  static constexpr int FM = wide::FM, FN = wide::FN;
};
struct Frags {
  intx4 q[FN], p[FM][2];
};

template <bool EXACT, int S, class F>
__device__ __forceinline__ void step(const Frags& f, const uint32_t (&sc)[FN + FM], floatx16 (&acc)[FM][FN], F&& between) {
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const intx8 x = __builtin_shufflevector(f.p[i][0], f.p[i][1], 0, 1, 2, 3, 4, 5, 6, 7);
    intx8 high, low;
    if constexpr (EXACT) two_parts(x, high, low);
#pragma unroll
    for (int j = 0; j < FN; ++j) {
      if constexpr (EXACT) {
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(high, four_bits(f.q[j]), acc[i][j], 0, 4, 2 * S, (int)sc[FN + i], 2 * S, (int)sc[j]);
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(low, four_bits(f.q[j]), acc[i][j], 0, 4, 2 * S, (int)sc[FN + i], 2 * S, (int)sc[j]);
      } else {
        acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, four_bits(f.q[j]), acc[i][j], 0, 4, 2 * S, (int)sc[FN + i], 2 * S, (int)sc[j]);
      }
      __builtin_amdgcn_sched_barrier(0);
      between(i * FN + j);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
}

template <Dt OT>
__global__ __launch_bounds__(64 * kWaves, 2) void wide8_kernel(const Args a) {
  constexpr bool kExact = OT == Dt::F32;
  constexpr int kReads = FN + 2 * FM, kMul = FM * FN;
  __shared__ __attribute__((aligned(16))) uint8_t smem[kLds];
  const int x = (int)blockIdx.x % kXcds;
  const int end = (int)((int64_t)(x + 1) * a.units / kXcds);
  int tile = (int)((int64_t)x * a.units / kXcds) + (int)blockIdx.x / kXcds;
  if (tile >= end) return;
  const int lane = threadIdx.x & 63, r = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_addr(smem));
  floatx16 acc[FM][FN];
  Frags f0, f1;
  uint32_t sc[FN + FM];
  // a lane's chunks: of Q 4 u + 2 s + h; of P 4 s + h (slot 0) and 4 s + 2 + h
  const uint32_t line = (uint32_t)(r * 128), sw = (uint32_t)swizzle(r);
  auto read_frag = [&](int u, int s, int b, int k, Frags& f) {
    if (k < FN) {
      f.q[k] = *reinterpret_cast<const intx4*>(smem + kQ + b * kPanelQ + (wn * FN + k) * 4096 + line + 16 * ((4 * u + 2 * s + h) ^ sw));
    } else {
      const int i = (k - FN) >> 1, slot = (k - FN) & 1;
      f.p[i][slot] = *reinterpret_cast<const intx4*>(smem + u * kHalf + (wm * FM + i) * 4096 + line + 16 * ((4 * s + 2 * slot + h) ^ sw));
    }
  };
  // bytes 2 s of what a lane gets are its slot's scales in step s of half u
  auto read_scale = [&](int u, int b, int k) {
    const int row = (k < FN ? B + (wn * FN + k) * 32 : (wm * FM + k - FN) * 32) + r;
    return *reinterpret_cast<const uint32_t*>(smem + kScales + b * kPanelS + row * 8 + 4 * u) >> (8 * h);
  };
  Cursor<true> np;
  Cursor<false> nq;
  np.start(a, tile, wave, lane);
  nq.start(a, tile, wave, lane);
#pragma unroll
  for (int k = 0; k < kLoads; ++k) np.load(lds0, 0, wave, k);
#pragma unroll
  for (int k = 0; k < kLoads + kScaleLoads; ++k) nq.load(lds0, 0, wave, k);
#pragma unroll
  for (int k = 0; k < kLoads; ++k) np.load(lds0, 1, wave, k);
  nq.advance(a, end, wave, lane);
#pragma unroll
  for (int k = 0; k < kLoads + kScaleLoads; ++k) nq.load(lds0, 1, wave, k);
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(2 * kLoads + kScaleLoads) : "memory");
  all_waves();
#pragma unroll
  for (int k = 0; k < kReads; ++k) {
    if (k < FN + FM) sc[k] = read_scale(0, 0, k);
    read_frag(0, 0, 0, k, f0);
  }
  int b = 0;                              // buffer of this panel's Q and scales
  for (; tile < end; tile += a.slots) {
#pragma unroll
    for (int i = 0; i < FM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[i][j][e] = 0.0f;
    for (int g = 0; g < a.panels; ++g) {
      np.advance(a, end, wave, lane);     // to the next panel
      nq.advance(a, end, wave, lane);     // to the one behind it
      uint32_t nsc[FN + FM];
      step<kExact, 0>(f0, sc, acc, [&](int k) {
#pragma unroll
        for (int n = share(kReads, k, kMul); n < share(kReads, k + 1, kMul); ++n) read_frag(0, 1, b, n, f1);
      });
      // every read of P's first half has returned, in all waves, and its second
      // half has landed (behind it only the next panel's Q and scales are under way)
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kLoads + kScaleLoads) : "memory");
      all_waves();
      step<kExact, 1>(f1, sc, acc, [&](int k) {
#pragma unroll
        for (int n = share(kReads, k, kMul); n < share(kReads, k + 1, kMul); ++n) {
          if (n < FN + FM) nsc[n] = read_scale(1, b, n);
          read_frag(1, 0, b, n, f0);
        }
#pragma unroll
        for (int n = share(kLoads, k, kMul); n < share(kLoads, k + 1, kMul); ++n) np.load(lds0, 0, wave, n);
      });
      step<kExact, 0>(f0, nsc, acc, [&](int k) {
#pragma unroll
        for (int n = share(kReads, k, kMul); n < share(kReads, k + 1, kMul); ++n) read_frag(1, 1, b, n, f1);
      });
      // every read of this panel has returned, and the next one's first half of
      // P, its Q and its scales have landed
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      all_waves();
      step<kExact, 1>(f1, nsc, acc, [&](int k) {
#pragma unroll
        for (int n = share(kReads, k, kMul); n < share(kReads, k + 1, kMul); ++n) {
          if (n < FN + FM) sc[n] = read_scale(0, b ^ 1, n);
          read_frag(0, 0, b ^ 1, n, f0);
        }
        constexpr int kAll = 2 * kLoads + kScaleLoads;
#pragma unroll
        for (int n = share(kAll, k, kMul); n < share(kAll, k + 1, kMul); ++n) {
          if (n < kLoads) np.load(lds0, 1, wave, n);
          else nq.load(lds0, b, wave, n - kLoads);
        }
      });
      b ^= 1;
    }
    int I, J, part;
    place_of(a, tile, I, J, part);
    epilogue<Blocks, OT, false>(product_again(), nullptr, acc, (int64_t)I * B, (int64_t)J * B, wm, wn, renewed(lane),
                               smem + kScales + 2 * kPanelS + wave * kScratch);
  }
  // the loads behind the last panel write LDS until they land
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

template <Dt OT>
hipError_t launch(const Product8& g, hipStream_t s) {
  const int panels = (int)((g.K + kPanel - 1) / kPanel);
  Args a{g, panels, panels, (int)((g.M + B - 1) / B), (int)((g.N + B - 1) / B), 0, 0, kCusPerXcd, nullptr};
  a.tiles = a.units = a.TM * a.TN;
  const int most = (a.units + kXcds - 1) / kXcds;
  wide8_kernel<OT><<<dim3((unsigned)(most < a.slots ? most : a.slots) * kXcds), 64 * kWaves, 0, s>>>(a);
  return hipGetLastError();
}
}  // namespace wide

// The parts of a product's sums, in part order.
template <Dt OT>
__global__ __launch_bounds__(256) void parts_kernel(const Product8 g, const float* partials, int parts) {
  const int64_t count = g.M * g.N, at = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 8;
  if (at >= count) return;
  const int n = count - at < 8 ? (int)(count - at) : 8;
  float v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = 0.0f;
#pragma unroll 4
  for (int p = 0; p < parts; ++p) {
    Raw8<float> o;
    o.load(partials + p * count + at, n);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] += o.get(e);
  }
  put8<OT>(g, at, n, v);
}

// Microseconds that tiles of one shape take, from measured BF16 products (K 4096
// unless stated): a round of 256 workgroups and 1.2 a round, and a panel's
// time, which grows from `low` to `high` with the CUs at work.
//   M x N              64x64  64x128  128x128  128x256  256x256
//   64 x 4096           10.6   11.7    16.4     24.8
//   256 x 4096          11.5   12.8    17.2     26.0
//   512 x 4096          19.5   14.0    17.6     26.5
//   1024 x 4096         34.6   24.5    21.0     27.6
//   2048 x 4096         65.7   43.6    36.5     31.5     42.8
//   256 x 11008         26.7   21.9    17.9     26.7
//   4096 x 300, K 1000   8.8    6.8     8.3     11.9
//   4096 x 4096                                 59.0     52.2
//   8192 x 4096                                114       98.8
// K in parts (few tiles, long K) adds their FP32 values' way and a launch.
// FP32 outputs, whose P goes in two parts, take 1.8 times as long a panel.
struct Shape {
  int BM, BN;
  double low, high;
};
constexpr int kWide = 4;
constexpr Shape kShapes[] = {{64, 64, 0.53, 0.60}, {64, 128, 0.60, 0.75}, {128, 128, 0.95, 1.15}, {128, 256, 1.45, 1.90}, {256, 256, 2.40, 3.05}};
using Tile0 = Tile<64, 64, 2, 2, 3>;
using Tile1 = Tile<64, 128, 2, 4, 3>;
using Tile2 = Tile<128, 128, 4, 2, 2>;
using Tile3 = Tile<128, 256, 4, 2, 2>;

double rounds_cost(const Shape& h, int64_t units, int per, bool exact) {
  const double t = (exact ? 1.8 : 1.0) * (h.low + (h.high - h.low) * (units < 256 ? units / 256.0 : 1.0));
  return ((units + 255) / 256) * (1.2 + per * t);
}

struct Plan {
  int shape, parts, per;
};
Plan plan(int64_t M, int64_t N, int64_t K, bool exact, bool split) {
  const int panels = (int)((K + kPanel - 1) / kPanel);
  Plan best{0, 1, panels};
  double least = 0.0;
  for (int i = 0; i <= kWide; ++i) {
    const Shape& h = kShapes[i];
    const int64_t tiles = ((M + h.BM - 1) / h.BM) * ((N + h.BN - 1) / h.BN);
    for (int wanted : {1, 2, 4, 8}) {
      if (wanted > 1 && (!split || i == kWide || tiles * wanted > 256 || panels < 2 * wanted)) break;
      const int per = (panels + wanted - 1) / wanted, parts = (panels + per - 1) / per;
      double us = rounds_cost(h, tiles * parts, per, exact);
      if (parts > 1) us += 3.0 + parts * 2e-6 * (double)(M * N);
      if (least == 0.0 || us < least) {
        least = us;
        best = Plan{i, parts, per};
      }
    }
  }
  return best;
}

template <class C, Dt OT>
hipError_t tiled(const Product8& g, const Plan& p, float* ws, hipStream_t s) {
  Args a{g, (int)((g.K + kPanel - 1) / kPanel), p.per, (int)((g.M + C::BM - 1) / C::BM), (int)((g.N + C::BN - 1) / C::BN), 0, 0, kCusPerXcd, ws};
  a.tiles = a.TM * a.TN;
  a.units = a.tiles * p.parts;
  const int most = (a.units + kXcds - 1) / kXcds;
  const dim3 grid((unsigned)(most < a.slots ? most : a.slots) * kXcds);
  if (p.parts == 1) {
    tile8_kernel<C, OT, false><<<grid, C::kThreads, 0, s>>>(a);
    return hipGetLastError();
  }
  tile8_kernel<C, OT, true><<<grid, C::kThreads, 0, s>>>(a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  parts_kernel<OT><<<dim3((unsigned)((g.M * g.N + 2047) / 2048)), 256, 0, s>>>(g, ws, p.parts);
  return hipGetLastError();
}
// Up to 16 rows of P wait for Q alone (1 x 11008 x 4096 8.0 us; in two groups of
// 16 rows, 32 of them take 17.5, on tiles 11.0).
constexpr int64_t kFewRows = 16;

template <Dt OT>
hipError_t product(const Product8& g, float* ws, hipStream_t s) {
  if (g.M <= kFewRows) return few<OT>(g, s);
  const Plan p = plan(g.M, g.N, g.K, OT == Dt::F32, ws != nullptr);
  switch (p.shape) {
    case 0: return tiled<Tile0, OT>(g, p, ws, s);
    case 1: return tiled<Tile1, OT>(g, p, ws, s);
    case 2: return tiled<Tile2, OT>(g, p, ws, s);
    case 3: return tiled<Tile3, OT>(g, p, ws, s);
    default: return wide::launch<OT>(g, s);
  }
}

}  // namespace

size_t mx8_workspace(int64_t M, int64_t N, int64_t K) {
  if (M <= kFewRows) return 0;
  const int parts = std::max(plan(M, N, K, false, true).parts, plan(M, N, K, true, true).parts);
  return parts > 1 ? (size_t)parts * (size_t)(M * N) * sizeof(float) : 0;
}

hipError_t launch_mx8_product(const Product8& g, void* ws, hipStream_t s) {
  float* w = static_cast<float*>(ws);
  return g.ot == Dt::F32 ? product<Dt::F32>(g, w, s) : product<Dt::BF16>(g, w, s);
}

}  // namespace nvfp4

// C = P Q^T on panel operands (panel.hpp): MXFP4 on the block-scaled matrix
// instruction v_mfma_scale_f32_32x32x64_f8f6f4, f16 on
// v_mfma_f32_32x32x16_f16, both with FP32 accumulation.
//
// The two share everything but the instruction: a row's panel is 128 bytes,
// eight 16-byte chunks, and a chunk is exactly one lane's operand of one
// instruction -- 32 E2M1 codes, which is one MXFP4 block with its own scale,
// or 8 f16 values.  Lane l holds row l % 32, chunk 4 (l / 32) + s in step s of
// the panel (a product sums over K, so any assignment of K to steps serves as
// long as both operands share it).
//
// A stage is one panel of the tile's rows: DMA loads bring whole 128-byte
// lines into LDS (eight rows an instruction; a tile's panel is one contiguous
// run of memory), chunk c of row r at position c ^ swizzle(r), so that 32
// lanes reading one chunk of 32 rows hit distinct banks.  MXFP4 scales come
// by the dword, one for a lane's four steps.
//
// Workgroups stay for as many tiles as there are per slot (a slot is one
// resident workgroup).  The stages of a workgroup's tiles form one stream
// through a ring of buffers, so that a tile's first panels load while the
// tile before still multiplies and leaves; a tile leaves through 2.5 KB of
// LDS of each wave's own, without a barrier.
//
// Tiles left over after an equal number per slot are split along K into
// parts whose FP32 partials a second kernel sums in part order.
#include <cstddef>

#include "dma.hpp"
#include "mxfp4_device.hpp"
#include "panel.hpp"

namespace nvfp4 {
namespace {

typedef float floatx16 __attribute__((ext_vector_type(16)));
typedef int intx4 __attribute__((ext_vector_type(4)));
typedef int intx8 __attribute__((ext_vector_type(8)));
typedef _Float16 halfx8 __attribute__((ext_vector_type(8)));
typedef _Float16 halfx2 __attribute__((ext_vector_type(2)));

constexpr int kXcds = 8;          // workgroups go round-robin to 8 XCDs
constexpr int kCusPerXcd = 32;

constexpr int kScratch = 2560;    // bytes of LDS a wave's epilogue uses

template <int B_, int WM_, int WN_, int NST_, int BLOCKS_>
struct Tile {
  static constexpr int B = B_;                 // rows and columns
  static constexpr int WM = WM_, WN = WN_, NST = NST_, kBlocks = BLOCKS_;
  static constexpr int kWaves = WM * WN, kThreads = 64 * kWaves;
  static constexpr int FM = B / (32 * WM), FN = B / (32 * WN);
  static constexpr int kRows = 2 * B;          // operand rows of a stage
  static constexpr int kCodeBytes = kRows * 128;
  static constexpr int kCodeLoads = kRows / 8 / kWaves;        // DMA instructions a wave and stage
  static constexpr int kScaleLoads = kRows * 2 / 64 / kWaves;  // MXFP4: 4 bytes a lane
  static_assert(kCodeLoads * 8 * kWaves == kRows && kScaleLoads * 32 * kWaves == kRows, "uneven loads");
  static constexpr int kAcc = FM * FN * 16;
};
using Tile256 = Tile<256, 2, 4, 2, 1>;
using Tile128 = Tile<128, 2, 2, 2, 2>;
using Tile64 = Tile<64, 2, 2, 3, 2>;

struct Args {
  PanelOperand p, q;
  int M, N, panels;
  int TM, TN, tiles, batch, slots, sym;          // slots: per XCD
  int parts;
  uint32_t parts_inv;           // 2^16 / parts, rounded up: exact below 2^16 / parts units
  float* partials;
  // epilogue
  float alpha, beta, ca, cb, cc;
  const float* dalpha;
  const float* addend;
  uint8_t* out;
  uint8_t* out_t;
  const uint8_t* a;
  const float* din;
  const float* da;
  float* dout;
  int din_cols;
  int wave_blocks;              // panel_poly_kernel: 32-row blocks of the other operand
  int64_t bstride;
};

// The run of tiles of one XCD (see "schedule").
struct alignas(16) Run {
  int t0, whole, units, split0;   // first tile; whole units; units in all; split tiles of the runs before
};

// What the kernels look up by index: the runs, and the row-major outputs of a
// batch with their factors on alpha (n > 0).  The first argument, so that it
// sits at the start of the kernel-argument segment: an entry is then a scalar
// load from there.
struct Each {
  Run run[kXcds];
  int n;
  float alpha[kMaxPanelBatch];
  void* out[kMaxPanelBatch];
};

template <class T>
__device__ __forceinline__ T looked_up(size_t offset, int i) {
  typedef const __attribute__((address_space(4))) uint8_t* KBytes;
  typedef const __attribute__((address_space(4))) T* KT;
  return ((KT)((KBytes)__builtin_amdgcn_kernarg_segment_ptr() + offset))[i];
}
__device__ __forceinline__ Run run_at(int x) {
  const intx4 v = looked_up<intx4>(offsetof(Each, run), x);
  return Run{v[0], v[1], v[2], v[3]};
}

template <class T>
__device__ __forceinline__ T* moved(T* p, int64_t off) {
  return p ? reinterpret_cast<T*>(reinterpret_cast<uintptr_t>(p) + off) : p;
}

// ---- schedule ----------------------------------------------------------------
// The tiles of all problems are cut into kXcds contiguous runs, one per XCD,
// in an order that keeps a run's tiles in a compact patch (they share the
// XCD's L2).  A run's first n / slots * slots tiles are whole units, the rest,
// when parts > 1, K-parts; the workgroup in slot l of an XCD takes units l,
// l + slots, ... of its run.

struct Unit {
  int tile, part, split;        // split: index among the split tiles, -1 for a whole tile
};

// Unit l of a run; false when there is none.
__device__ __forceinline__ bool unit_of(const Args& a, const Run& run, int l, Unit& u) {
  u.part = 0;
  u.split = -1;
  u.tile = run.t0 + l;
  if (l < run.whole) return true;
  if (l >= run.units) return false;
  const int r = l - run.whole;
  const int s = (int)(((uint32_t)r * a.parts_inv) >> 16);      // r / parts
  u.tile = run.t0 + run.whole + s;
  u.part = r - s * a.parts;
  u.split = run.split0 + s;
  return true;
}

// First panel of K-part p of n.
__device__ __forceinline__ int part_panel(const Args& a, int p, int n) {
  return n == 1 ? p * a.panels : __builtin_amdgcn_readfirstlane((int)((uint32_t)(a.panels * p) / (uint32_t)n));
}

// Strips of kStrip tile rows, column by column within a strip; symmetric
// products list I <= J only, a strip's diagonal triangle first.
constexpr int kStrip = 4;
__device__ __forceinline__ void tile_of(const Args& a, int t, int& I, int& J) {
  if (a.sym) {
    for (int s = 0;; s += kStrip) {
      const int w = a.TM - s < kStrip ? a.TM - s : kStrip;
      const int tri = w * (w + 1) / 2, cnt = tri + w * (a.TM - s - w);
      if (t >= cnt) {
        t -= cnt;
        continue;
      }
      if (t < tri) {
        int j = 0;
        while (t > j) t -= ++j;          // column j holds j + 1 tiles
        I = s + t;
        J = s + j;
      } else {
        t -= tri;
        I = s + t % w;
        J = s + w + t / w;
      }
      return;
    }
  }
  const int s = t / (kStrip * a.TN) * kStrip;
  const int w = a.TM - s < kStrip ? a.TM - s : kStrip;
  t -= s * a.TN;
  I = s + t % w;
  J = t / w;
}

// Problem, row block and column block of a tile of the batch, in scalar
// registers (the divisions run on the vector unit).
__device__ __forceinline__ void place_of(const Args& a, int t, int& y, int& I, int& J) {
  y = a.batch == 1 ? 0 : __builtin_amdgcn_readfirstlane(t / a.tiles);
  int i, j;
  tile_of(a, t - y * a.tiles, i, j);
  I = __builtin_amdgcn_readfirstlane(i);
  J = __builtin_amdgcn_readfirstlane(j);
}

// ---- loads -------------------------------------------------------------------
// Where a workgroup's loads stand: the next panel of the unit being loaded,
// the wave's operand of it, and the byte offsets of a lane's loads inside a
// panel.  Rows past the operand's end read its last row: they feed only
// outputs that the epilogue does not write.  A wave's share of a stage never
// straddles the operands: B rows are a multiple of it.
template <class C, bool FP4>
struct Loads {
  static constexpr int kLoads = C::kCodeLoads + (FP4 ? C::kScaleLoads : 0);
  int l, g, g1;                         // unit of the run, next panel, end
  const uint8_t *data, *scales;         // panel g of the wave's operand
  int64_t pitch;                        // bytes of a panel's codes
  uint32_t code[C::kCodeLoads];
  uint32_t scale[FP4 ? C::kScaleLoads : 1];

  __device__ __forceinline__ void start(const Args& a, const Unit& u, int wave, int lane) {
    int y, I, J;
    place_of(a, u.tile, y, I, J);
    const int nparts = u.split < 0 ? 1 : a.parts;
    g = part_panel(a, u.part, nparts);
    g1 = part_panel(a, u.part + 1, nparts);
    const bool isP = wave * C::kCodeLoads * 8 < C::B;
    const int64_t rows = isP ? a.p.rows : a.q.rows;
    pitch = rows * 128;
    data = (isP ? a.p.data : a.q.data) + (int64_t)y * a.bstride + (int64_t)g * pitch;
    if constexpr (FP4) scales = (isP ? a.p.scales : a.q.scales) + (int64_t)g * rows * 8;
    const int lim = isP ? a.M : a.N;
    // operand row of the wave's first stage row
    const int r0 = (isP ? I * C::B : J * C::B - C::B) + 8 * wave * C::kCodeLoads;
#pragma unroll
    for (int i = 0; i < C::kCodeLoads; ++i) {
      int row = r0 + 8 * i + (lane >> 3);
      row = row < lim ? row : lim - 1;
      code[i] = (uint32_t)row * 128u + 16u * (uint32_t)((lane & 7) ^ swizzle(8 * i + 8 * wave * C::kCodeLoads + (lane >> 3)));
    }
    if constexpr (FP4) {
#pragma unroll
      for (int i = 0; i < C::kScaleLoads; ++i) {
        int row = r0 + 32 * i + (lane >> 1);
        row = row < lim ? row : lim - 1;
        scale[i] = (uint32_t)row * 8u + 4u * (uint32_t)(lane & 1);
      }
    }
  }
  // Load number k of the wave's share into the stage at LDS address `stage`.
  __device__ __forceinline__ void load(uint32_t stage, int wave, int k) const {
    if (k < C::kCodeLoads)
      dma16(data, code[k], stage + (uint32_t)(wave * C::kCodeLoads + k) * 1024u);
    else if constexpr (FP4)
      dma4(scales, scale[k - C::kCodeLoads],
           stage + (uint32_t)C::kCodeBytes + (uint32_t)(wave * C::kScaleLoads + k - C::kCodeLoads) * 256u);
  }
  // To the next panel: of this unit, of the workgroup's next unit, or, behind
  // the last, the same again (into a buffer that nothing reads).
  __device__ __forceinline__ void advance(const Args& a, const Run& run, int wave, int lane) {
    if (g + 1 < g1) {
      ++g;
      data += pitch;
      if constexpr (FP4) scales += pitch / 16;
      return;
    }
    Unit u;
    if (unit_of(a, run, l + a.slots, u)) {
      l += a.slots;
      start(a, u, wave, renewed(lane));
    }
  }
};

// ---- multiply ------------------------------------------------------------------
template <int S>
__device__ __forceinline__ floatx16 mfma_fp4(intx4 a, intx4 b, floatx16 c, uint32_t sa, uint32_t sb) {
  // 4-bit operands are four registers; the rest of the builtin's eight is not read
  const intx8 x = __builtin_shufflevector(a, a, 0, 1, 2, 3, -1, -1, -1, -1);
  const intx8 y = __builtin_shufflevector(b, b, 0, 1, 2, 3, -1, -1, -1, -1);
  return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, y, c, 4, 4, S, (int)sa, S, (int)sb);
}
__device__ __forceinline__ floatx16 mfma_f16(intx4 a, intx4 b, floatx16 c) {
  union { intx4 i; halfx8 h; } x{a}, y{b};
  return __builtin_amdgcn_mfma_f32_32x32x16_f16(x.h, y.h, c, 0, 0, 0);
}

// One step's operands of a wave, and a stage's scales (four steps).
template <class C>
struct Frags {
  intx4 q[C::FN], p[C::FM];
};
template <class C>
struct Scales {
  uint32_t q[C::FN], p[C::FM];
};

// Read number k of a step: Q's fragments, then P's, in the order of use.
template <class C>
__device__ __forceinline__ void read_frag(const uint8_t* st, uint32_t off, int wm, int wn, int k, Frags<C>& f) {
  if (k < C::FN)
    f.q[k] = *reinterpret_cast<const intx4*>(st + off + (C::B / 32 + wn * C::FN + k) * 4096);
  else
    f.p[k - C::FN] = *reinterpret_cast<const intx4*>(st + off + (wm * C::FM + k - C::FN) * 4096);
}
template <class C>
__device__ __forceinline__ void read_scale(const uint8_t* st, uint32_t off, int wm, int wn, int k, Scales<C>& f) {
  st += C::kCodeBytes;
  if (k < C::FN)
    f.q[k] = *reinterpret_cast<const uint32_t*>(st + off + (C::B / 32 + wn * C::FN + k) * 256);
  else
    f.p[k - C::FN] = *reinterpret_cast<const uint32_t*>(st + off + (wm * C::FM + k - C::FN) * 256);
}

// One step's MFMAs; `between(k)` puts memory operations behind the k-th, and
// the compiler keeps this order: a step's fragments are read while the step
// before multiplies.
template <class C, bool FP4, int S, class F>
__device__ __forceinline__ void step(const Frags<C>& f, const Scales<C>& sc, floatx16 (&acc)[C::FM][C::FN],
                                     F&& between) {
#pragma unroll
  for (int i = 0; i < C::FM; ++i)
#pragma unroll
    for (int j = 0; j < C::FN; ++j) {
      if constexpr (FP4)
        acc[i][j] = mfma_fp4<S>(f.p[i], f.q[j], acc[i][j], sc.p[i], sc.q[j]);
      else
        acc[i][j] = mfma_f16(f.p[i], f.q[j], acc[i][j]);
      __builtin_amdgcn_sched_barrier(0);
      between(i * C::FN + j);
      __builtin_amdgcn_sched_barrier(0);
    }
}

// Part k of n of the work 0 .. total - 1.
__device__ __forceinline__ constexpr int share(int total, int k, int n) { return total * k / n; }

// ---- epilogues -----------------------------------------------------------------
// acc[i][j][4 q + t] of a lane is row (wm FM + i) 32 + 8 q + 4 (lane / 32) + t,
// column (wn FN + j) 32 + lane % 32 of the tile.

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  union { halfx2 h; uint32_t u; } r;
  r.h[0] = (_Float16)lo;
  r.h[1] = (_Float16)hi;
  return r.u;
}
__device__ __forceinline__ float f16_lo(uint32_t w) {
  union { uint32_t u; halfx2 h; } r{w};
  return (float)r.h[0];
}
__device__ __forceinline__ float f16_hi(uint32_t w) {
  union { uint32_t u; halfx2 h; } r{w};
  return (float)r.h[1];
}

// Eight neighbours of a row-major matrix, or the first n of them.
template <Dt T>
__device__ __forceinline__ void load8(const void* p, int64_t at, float (&v)[8]) {
  if constexpr (T == Dt::F32) {
    const float* f = static_cast<const float*>(p) + at;
    const float4 a = *reinterpret_cast<const float4*>(f), b = *reinterpret_cast<const float4*>(f + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  } else {
    const uint4 a = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + at);
    v[0] = mx::bf16_lo(a.x); v[1] = mx::bf16_hi(a.x); v[2] = mx::bf16_lo(a.y); v[3] = mx::bf16_hi(a.y);
    v[4] = mx::bf16_lo(a.z); v[5] = mx::bf16_hi(a.z); v[6] = mx::bf16_lo(a.w); v[7] = mx::bf16_hi(a.w);
  }
}
// Rows that do not begin on 16 bytes: eight neighbours still move as such
// (global memory takes any alignment of the element type); the last of a row
// one by one (1000 x 777 x 1501 with an FP32 addend: 10.2 us with single
// elements throughout, 7.4 us so).
template <Dt T>
__device__ __forceinline__ void load_n(const void* p, int64_t at, int n, float (&v)[8]) {
  if constexpr (T == Dt::F32) {
    const float* f = static_cast<const float*>(p) + at;
    if (n == 8) {
      const mx::float4u a = *reinterpret_cast<const mx::float4u*>(f), b = *reinterpret_cast<const mx::float4u*>(f + 4);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = a[i];
        v[4 + i] = b[i];
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = i < n ? f[i] : 0.0f;
    }
  } else {
    const uint16_t* f = static_cast<const uint16_t*>(p) + at;
    if (n == 8) {
      const mx::bf16x8u a = *reinterpret_cast<const mx::bf16x8u*>(f);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __uint_as_float((uint32_t)a[i] << 16);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = i < n ? __uint_as_float((uint32_t)f[i] << 16) : 0.0f;
    }
  }
}
template <Dt T>
__device__ __forceinline__ void store8(void* p, int64_t at, const float (&v)[8]) {
  if constexpr (T == Dt::F32) {
    float* f = static_cast<float*>(p) + at;
    *reinterpret_cast<float4*>(f) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(f + 4) = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + at) =
        make_uint4(mx::pack_bf16(v[0], v[1]), mx::pack_bf16(v[2], v[3]), mx::pack_bf16(v[4], v[5]),
                   mx::pack_bf16(v[6], v[7]));
  }
}
template <Dt T>
__device__ __forceinline__ void store_n(void* p, int64_t at, int n, const float (&v)[8]) {
  if constexpr (T == Dt::F32) {
    float* f = static_cast<float*>(p) + at;
    if (n == 8) {
      *reinterpret_cast<mx::float4u*>(f) = mx::float4u{v[0], v[1], v[2], v[3]};
      *reinterpret_cast<mx::float4u*>(f + 4) = mx::float4u{v[4], v[5], v[6], v[7]};
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) f[i] = v[i];
    }
  } else {
    uint16_t* f = static_cast<uint16_t*>(p) + at;
    if (n == 8) {
      mx::bf16x8u w;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t u = mx::pack_bf16(v[2 * i], v[2 * i + 1]);
        w[2 * i] = (uint16_t)u;
        w[2 * i + 1] = (uint16_t)(u >> 16);
      }
      *reinterpret_cast<mx::bf16x8u*>(f) = w;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) f[i] = (uint16_t)mx::pack_bf16(v[i], 0.0f);
    }
  }
}

// Factors on a tile's values: alpha, and per row or per column where an array
// gives them.  A lane's are loaded together, before the blocks that use them:
// the accumulators stay as they are (scaled in place they would be kept twice,
// and spill).
template <class C>
struct Factors {
  float row[C::FM][2];          // by_rows: row 16 half + lane / 4 of block row i
  float col[C::FN][8];          // and the lane's eight columns of block column j

  // din: the tile's first row or column
  __device__ __forceinline__ Factors(float alpha, const float* din, bool cols, int wm, int wn, int lane) {
#pragma unroll
    for (int i = 0; i < C::FM; ++i) row[i][0] = row[i][1] = alpha;
#pragma unroll
    for (int j = 0; j < C::FN; ++j)
#pragma unroll
      for (int e = 0; e < 8; ++e) col[j][e] = 1.0f;
    if (din && !cols) {
#pragma unroll
      for (int i = 0; i < C::FM; ++i)
#pragma unroll
        for (int h = 0; h < 2; ++h) row[i][h] *= din[(wm * C::FM + i) * 32 + 16 * h + (lane >> 2)];
    } else if (din) {
#pragma unroll
      for (int j = 0; j < C::FN; ++j)
#pragma unroll
        for (int e = 0; e < 8; ++e) col[j][e] = din[(wn * C::FN + j) * 32 + (lane & 3) * 8 + e];
    }
  }
};

// f(row, column, v): eight neighbouring values of a tile row, each lane its
// own; the wave's 32 x 32 blocks pass through LDS sixteen rows at a time.
template <class C, class F>
__device__ __forceinline__ void by_rows(const floatx16 (&acc)[C::FM][C::FN], const Factors<C>& k, int wm, int wn, int lane,
                                        uint8_t* lds, F&& f) {
  constexpr int kPitch = 36;             // floats; 16 rows are 2304 bytes
  float* t = reinterpret_cast<float*>(lds);
#pragma unroll
  for (int i = 0; i < C::FM; ++i)
#pragma unroll
    for (int j = 0; j < C::FN; ++j)
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const int el = renewed(lane), h = el >> 5, c = el & 31, r = el >> 2, c8 = (el & 3) * 8;
#pragma unroll
        for (int q = 0; q < 2; ++q)
#pragma unroll
          for (int s = 0; s < 4; ++s) t[(8 * q + 4 * h + s) * kPitch + c] = acc[i][j][8 * half + 4 * q + s];
        wave_sync();
        float v[8];
        const float4 lo = *reinterpret_cast<const float4*>(t + r * kPitch + c8);
        const float4 hi = *reinterpret_cast<const float4*>(t + r * kPitch + c8 + 4);
        v[0] = lo.x; v[1] = lo.y; v[2] = lo.z; v[3] = lo.w;
        v[4] = hi.x; v[5] = hi.y; v[6] = hi.z; v[7] = hi.w;
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= k.row[i][half] * k.col[j][e];
        f((wm * C::FM + i) * 32 + 16 * half + r, (wn * C::FN + j) * 32 + c8, v);
        wave_sync();
        __builtin_amdgcn_sched_barrier(0);
      }
}

// f(column, row, w): eight neighbouring values of a tile column as f16, times
// alpha and din[row], whose values load one block row ahead (din null: alpha).
template <class C, class F>
__device__ __forceinline__ void by_cols(const floatx16 (&acc)[C::FM][C::FN], float alpha, const float* din, int wm, int wn,
                                        int lane, uint8_t* lds, F&& f) {
  constexpr int kPitch = 80;             // bytes; 32 columns of 32 rows
  float4 k[2][4];
  auto load = [&](int i) {
#pragma unroll
    for (int q = 0; q < 4; ++q)
      k[i & 1][q] = din ? *reinterpret_cast<const float4*>(din + (wm * C::FM + i) * 32 + 8 * q + 4 * (lane >> 5))
                        : make_float4(1.0f, 1.0f, 1.0f, 1.0f);
  };
  load(0);
#pragma unroll
  for (int i = 0; i < C::FM; ++i) {
    if (i + 1 < C::FM) load(i + 1);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int j = 0; j < C::FN; ++j) {
      const int el = renewed(lane), h = el >> 5, c = el & 31, r = el >> 2, c8 = (el & 3) * 8;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const float4 d = k[i & 1][q];
        *reinterpret_cast<uint2*>(lds + c * kPitch + 2 * (8 * q + 4 * h)) =
            make_uint2(pack_f16(alpha * d.x * acc[i][j][4 * q], alpha * d.y * acc[i][j][4 * q + 1]),
                       pack_f16(alpha * d.z * acc[i][j][4 * q + 2], alpha * d.w * acc[i][j][4 * q + 3]));
      }
      wave_sync();
#pragma unroll
      for (int half = 0; half < 2; ++half) {
        const uint4 w = *reinterpret_cast<const uint4*>(lds + (16 * half + r) * kPitch + 2 * c8);
        f((wn * C::FN + j) * 32 + 16 * half + r, (wm * C::FM + i) * 32 + c8, w);
      }
      wave_sync();
      __builtin_amdgcn_sched_barrier(0);
    }
  }
}

// The diagonal of a 32 x 32 block on it: the lanes whose column c is one of
// their rows (lane / 32 == c / 4 % 2) hold it at 4 (c / 8) + c % 4.
__device__ __forceinline__ bool on_diagonal(int lane) { return (lane >> 5) == ((lane >> 2) & 1); }
__device__ __forceinline__ float diagonal_of(const floatx16& v, int lane) {
  const int c = lane & 31, at = 4 * (c >> 3) + (c & 3);
  float d = v[0];
#pragma unroll
  for (int r = 1; r < 16; ++r) d = r == at ? v[r] : d;
  return d;
}

// What B's row is multiplied by for its diagonal's sake, B_ii / f16(B_ii): within
// 2^-11 of 1 while f16 holds B_ii as a normal number.  Below that the quotient
// may be anything from 0.5 to 1.5 and would scale the entries that carry the row,
// for a loss of 2^-25 at most: such a row is left alone.
__device__ __forceinline__ float row_factor(float v) {
  const float r = (float)(_Float16)v;
  return fabsf(r) >= 0x1p-14f ? v / r : 1.0f;
}

// Eight neighbours of an f16 panel operand: row r, columns from c (a multiple
// of 8) of an operand with `rows` rows a panel.
__device__ __forceinline__ uint8_t* panel_at(uint8_t* p, int rows, int r, int c) {
  return p + ((int64_t)(c >> 6) * rows + r) * 128 + (c & 63) * 2;
}

// The factors of a tile's rows, or of its columns.
__device__ __forceinline__ const float* tile_din(const Args& a, int y, int m0, int n0) {
  return a.din ? moved(a.din, (int64_t)y * a.bstride) + (a.din_cols ? n0 : m0) : nullptr;
}

// lds: this wave's kScratch bytes.  y: problem of the batch.  din: tile_din
// (Poly takes a.din itself).
template <class C, PanelEp EP, Dt OT, bool VEC>
__device__ __forceinline__ void epilogue(const Args& a, int neach, floatx16 (&acc)[C::FM][C::FN], int y, int I, int J,
                                         int wm, int wn, int lane, uint8_t* lds, const float* din) {
  const int m0 = I * C::B, n0 = J * C::B;
  const int64_t off = (int64_t)y * a.bstride;
  float alpha = a.alpha;
  if (a.dalpha) alpha *= *moved(a.dalpha, off);
  uint8_t* out = a.out + off;
  if (neach) {
    out = static_cast<uint8_t*>(looked_up<void*>(offsetof(Each, out), y));
    alpha *= looked_up<float>(offsetof(Each, alpha), y);
  }
  if constexpr (EP == PanelEp::Step || EP == PanelEp::Out) {
    // VEC: rows of whole 16-byte units, so that eight neighbours are in or out
    // together and move as such
    const Factors<C> k(alpha, din, a.din_cols != 0, wm, wn, lane);
    by_rows<C>(acc, k, wm, wn, lane, lds, [&](int dr, int dc, float (&v)[8]) {
      const int row = m0 + dr, col = n0 + dc;
      if (row >= a.M || col >= a.N) return;
      const int64_t at = (int64_t)row * a.N + col;
      const int n = a.N - col < 8 ? a.N - col : 8;
      float o[8];                        // the addend, or the weights
      if constexpr (EP == PanelEp::Step) {
        if constexpr (VEC) load8<OT>(out, at, o);
        else load_n<OT>(out, at, n, o);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = fmaf(a.beta, o[e], -v[e]);
      } else if (a.addend) {
        if constexpr (VEC) load8<Dt::F32>(a.addend, at, o);
        else load_n<Dt::F32>(a.addend, at, n, o);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = fmaf(a.beta, o[e], v[e]);
      }
      if constexpr (VEC) store8<OT>(out, at, v);
      else store_n<OT>(out, at, n, v);
    });
  } else {
    if constexpr (EP == PanelEp::Poly) {
      // A is symmetric: four neighbours of a column are four of a row; a
      // batch's loads go out before the first is used
      const uint8_t* A = a.a + off;
      const float* D = moved(a.din, off);
      constexpr int kBatch = C::FM * C::FN > 4 ? 2 : C::FM;      // block rows at a time
      const int h = lane >> 5, c = lane & 31;
#pragma unroll
      for (int i0 = 0; i0 < C::FM; i0 += kBatch) {
        uint2 w[kBatch][C::FN][4];
#pragma unroll
        for (int i = i0; i < i0 + kBatch && i < C::FM; ++i)
#pragma unroll
          for (int j = 0; j < C::FN; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              // outside A (whole blocks: M is a multiple of 64) anything
              // finite does, nothing of it is stored
              int row = m0 + (wm * C::FM + i) * 32, col = n0 + (wn * C::FN + j) * 32;
              row = (row < a.M ? row : 0) + 8 * q;
              col = col < a.M ? col : 0;
              w[i - i0][j][q] = *reinterpret_cast<const uint2*>(
                  A + (int64_t)(row >> 6) * a.M * 128 + (int64_t)col * 128 + (row & 63) * 2 + (uint32_t)(c * 128 + 8 * h));
            }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = i0; i < i0 + kBatch && i < C::FM; ++i)
#pragma unroll
          for (int j = 0; j < C::FN; ++j) {
            // row - column of the lane's first value
            const int d = m0 - n0 + (wm * C::FM + i) * 32 - (wn * C::FN + j) * 32 + 4 * h - c;
            const float dj = D[n0 + (wn * C::FN + j) * 32 + c];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const float4 d4 = *reinterpret_cast<const float4*>(D + m0 + (wm * C::FM + i) * 32 + 8 * q + 4 * h);
              const float di[4] = {d4.x, d4.y, d4.z, d4.w};
              const uint2 u = w[i - i0][j][q];
              const float av[4] = {f16_lo(u.x), f16_hi(u.x), f16_lo(u.y), f16_hi(u.y)};
#pragma unroll
              for (int t = 0; t < 4; ++t) {
                const float v = fmaf(a.cc, fmaf(di[t] + dj, av[t], acc[i][j][4 * q + t]), a.cb * av[t]);
                acc[i][j][4 * q + t] = d + 8 * q + t == 0 ? v + fmaf(a.cb, dj, a.ca) : v;
              }
            }
            // here, not where the stores need it (with A's values kept till then)
            asm volatile("" : "+v"(acc[i][j]));
          }
      }
    }
    if constexpr (EP != PanelEp::Iter) {
      if (I == J) {
        float* dout = moved(a.dout, off);
#pragma unroll
        for (int i = 0; i < C::FM; ++i)
#pragma unroll
          for (int j = 0; j < C::FN; ++j) {
            const int row = m0 + (wm * C::FM + i) * 32 + (lane & 31);
            if (wm * C::FM + i != wn * C::FN + j || !on_diagonal(lane) || row >= a.M) continue;
            const float v = (EP == PanelEp::Poly ? 1.0f : alpha) * diagonal_of(acc[i][j], lane);
            dout[row] = EP == PanelEp::Gram ? v - (float)(_Float16)v : row_factor(v);
          }
      }
    }
    // the transpose; a symmetric product's mirror (a diagonal tile is its own)
    constexpr bool kIter = EP == PanelEp::Iter;
    uint8_t* tdst = kIter ? a.out_t + off : out;
    const float mul = EP == PanelEp::Poly ? 1.0f : alpha;
    if (!kIter) din = nullptr;
    by_cols<C>(acc, mul, din, wm, wn, lane, lds, [&](int dc, int dr, uint4 w) {
      if (n0 + dc < a.N && m0 + dr < a.M) *reinterpret_cast<uint4*>(panel_at(tdst, a.N, n0 + dc, m0 + dr)) = w;
    });
    if (kIter || I != J) {
      const Factors<C> k(mul, din, false, wm, wn, lane);
      by_rows<C>(acc, k, wm, wn, lane, lds, [&](int dr, int dc, float (&v)[8]) {
        if (m0 + dr < a.M && n0 + dc < a.N)
          *reinterpret_cast<uint4*>(panel_at(out, a.M, m0 + dr, n0 + dc)) =
              make_uint4(pack_f16(v[0], v[1]), pack_f16(v[2], v[3]), pack_f16(v[4], v[5]), pack_f16(v[6], v[7]));
      });
    }
  }
}

// FP32 partials of a K-part: per block and quad a run of kThreads float4.
template <class C>
__device__ __forceinline__ size_t part_index(int b, int q, int thread) {
  return ((size_t)(b * 4 + q) * C::kThreads + thread) * 4;
}

template <class C, bool FP4>
constexpr int stage_bytes() { return C::kCodeBytes + (FP4 ? C::kRows * 8 : 0); }

template <class C>
__device__ __forceinline__ void clear(floatx16 (&acc)[C::FM][C::FN]) {
#pragma unroll
  for (int i = 0; i < C::FM; ++i)
#pragma unroll
    for (int j = 0; j < C::FN; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
}

template <class C, bool FP4, PanelEp EP, Dt OT, bool VEC>
__global__ __launch_bounds__(C::kThreads, C::kBlocks* C::kWaves / 4) void panel_kernel(const Each e, Args a) {
  constexpr int kStage = stage_bytes<C, FP4>();
  __shared__ __attribute__((aligned(16))) uint8_t smem[C::NST * kStage + C::kWaves * kScratch];
  const Run run = run_at((int)blockIdx.x % kXcds);
  int l = (int)blockIdx.x / kXcds;
  Unit un;
  if (!unit_of(a, run, l, un)) return;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / C::WN, wn = wave % C::WN;
  uint8_t* scratch = smem + C::NST * kStage + wave * kScratch;

  floatx16 acc[C::FM][C::FN];
  Loads<C, FP4> next;
  next.l = l;
  next.start(a, un, wave, lane);
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_addr(smem));
  constexpr int kLoads = Loads<C, FP4>::kLoads, kReads = C::FM + C::FN, kMul = C::FM * C::FN;
  uint32_t off[4];
#pragma unroll
  for (int s = 0; s < 4; ++s)
    off[s] = (uint32_t)((lane & 31) * 128 + 16 * ((4 * (lane >> 5) + s) ^ swizzle(lane & 31)));
  const uint32_t soff = (uint32_t)((lane & 31) * 8 + 4 * (lane >> 5));
  Frags<C> f0, f1;
  Scales<C> sc;
  // all but the newest NST - 2 stages' loads of this wave have landed
  auto wait_loads = [&] { asm volatile("s_waitcnt vmcnt(%0)" ::"n"((C::NST - 2) * kLoads) : "memory"); };

  // NST - 1 stages in flight before the first is read, then always NST
#pragma unroll 1
  for (int s = 0; s < C::NST - 1; ++s) {
#pragma unroll
    for (int k = 0; k < kLoads; ++k) next.load(lds0 + s * kStage, wave, k);
    next.advance(a, run, wave, lane);
  }
  wait_loads();
  all_waves();
#pragma unroll
  for (int k = 0; k < kLoads; ++k) next.load(lds0 + (C::NST - 1) * kStage, wave, k);
#pragma unroll
  for (int k = 0; k < kReads; ++k) {
    if constexpr (FP4) read_scale<C>(smem, soff, wm, wn, k, sc);
    read_frag<C>(smem, off[0], wm, wn, k, f0);
  }

  int cur = 0;
  do {
    clear<C>(acc);
    const int nparts = un.split < 0 ? 1 : a.parts;
    const int g0 = part_panel(a, un.part, nparts), g1 = part_panel(a, un.part + 1, nparts);
    for (int g = g0; g < g1; ++g) {
      // here, not behind the loads: a branch behind the MFMAs would let the
      // compiler sink them past it
      next.advance(a, run, wave, lane);
      const uint8_t* st = smem + cur * kStage;
      auto ahead = [&](int s, Frags<C>& f) {
        return [&, s](int k) {
#pragma unroll
          for (int r = share(kReads, k, kMul); r < share(kReads, k + 1, kMul); ++r)
            read_frag<C>(st, off[s], wm, wn, r, f);
        };
      };
      step<C, FP4, 0>(f0, sc, acc, ahead(1, f1));
      step<C, FP4, 1>(f1, sc, acc, ahead(2, f0));
      step<C, FP4, 2>(f0, sc, acc, ahead(3, f1));
      // every read of this stage has returned: its buffer is free once all
      // waves are here, and the next stage's loads have landed
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      wait_loads();
      all_waves();
      const uint32_t freed = lds0 + cur * kStage;
      cur = cur + 1 == C::NST ? 0 : cur + 1;
      const uint8_t* nst = smem + cur * kStage;
      Scales<C> nsc;
      step<C, FP4, 3>(f1, sc, acc, [&](int k) {
#pragma unroll
        for (int r = share(kReads, k, kMul); r < share(kReads, k + 1, kMul); ++r) {
          if constexpr (FP4) read_scale<C>(nst, soff, wm, wn, r, nsc);
          read_frag<C>(nst, off[0], wm, wn, r, f0);
        }
#pragma unroll
        for (int r = share(kLoads, k, kMul); r < share(kLoads, k + 1, kMul); ++r) next.load(freed, wave, r);
      });
      if constexpr (FP4) sc = nsc;
    }
    if (un.split >= 0) {
      float* part = a.partials + ((size_t)un.split * a.parts + un.part) * C::kAcc * C::kThreads;
#pragma unroll
      for (int i = 0; i < C::FM; ++i)
#pragma unroll
        for (int j = 0; j < C::FN; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q)
            *reinterpret_cast<float4*>(part + part_index<C>(i * C::FN + j, q, threadIdx.x)) = make_float4(
                acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]);
    } else {
      int y, I, J;
      place_of(a, un.tile, y, I, J);
      epilogue<C, EP, OT, VEC>(a, e.n, acc, y, I, J, wm, wn, renewed(lane), scratch,
                               tile_din(a, y, I * C::B, J * C::B));
    }
    l += a.slots;
  } while (unit_of(a, run, l, un));
  // the loads behind the last stage write LDS until they land
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

// A tile whose waves hold one 32 x 32 block each.
template <class C>
struct OneBlock : C {
  static constexpr int FM = 1, FN = 1;
};

// The split tiles: block number b of every wave's sub-tile a workgroup, its
// parts' partials summed in part order.
template <class C, PanelEp EP, Dt OT, bool VEC>
__global__ __launch_bounds__(C::kThreads) void panel_sum_kernel(const Each e, Args a) {
  __shared__ __attribute__((aligned(16))) uint8_t smem[C::kWaves * kScratch];
  constexpr int kBlocks = C::FM * C::FN;
  const int split = (int)blockIdx.x / kBlocks, b = (int)blockIdx.x % kBlocks;
  Run run = run_at(0);
  for (int x = 1; x < kXcds; ++x) {
    const Run r = run_at(x);
    if (r.split0 <= split) run = r;        // runs without split tiles share the next one's split0
  }
  int y, I, J;
  place_of(a, run.t0 + run.whole + split - run.split0, y, I, J);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  floatx16 acc[1][1];
  const float* part = a.partials + (size_t)split * a.parts * C::kAcc * C::kThreads;
#pragma unroll
  for (int r = 0; r < 16; ++r) acc[0][0][r] = 0.0f;
#pragma unroll 4
  for (int p = 0; p < a.parts; ++p)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const float4 v = *reinterpret_cast<const float4*>(part + (size_t)p * C::kAcc * C::kThreads +
                                                        part_index<C>(b, q, threadIdx.x));
      acc[0][0][4 * q] += v.x;
      acc[0][0][4 * q + 1] += v.y;
      acc[0][0][4 * q + 2] += v.z;
      acc[0][0][4 * q + 3] += v.w;
    }
  epilogue<OneBlock<C>, EP, OT, VEC>(a, e.n, acc, y, I, J, wave / C::WN * C::FM + b / C::FN, wave % C::WN * C::FN + b % C::FN,
                                     lane, smem + wave * kScratch,
                                   tile_din(a, y, I * C::B, J * C::B));
}

// Small products: one 32 x 32 tile a workgroup, its eight waves dividing the
// panels of K, each through a double buffer of LDS of its own: no barriers
// until the waves' sums meet, in wave order.  The whole of a product's time is
// then one or two trips to memory.  (Fragments loaded straight into registers
// touch 32 lines an instruction and fetch each line for every quarter of it.)
struct Tile32 {
  static constexpr int B = 32, WM = 1, WN = 1, FM = 1, FN = 1, kWaves = 8, kThreads = 512, kBlocks = 2, kAcc = 16;
};

template <bool FP4, PanelEp EP, Dt OT, bool VEC>
__global__ __launch_bounds__(512, 2) void panel_direct_kernel(const Each e, Args a) {
  constexpr int kBuf = 2 * 4096 + (FP4 ? 512 : 0);      // 32 rows of either operand, and their scales
  constexpr int kLoads = FP4 ? 10 : 8;
  __shared__ __attribute__((aligned(16))) uint8_t smem[Tile32::kWaves * 2 * kBuf];
  int y, I, J;
  place_of(a, (int)blockIdx.x, y, I, J);
  const int lane = threadIdx.x & 63, r = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int g0 = a.panels * wave / Tile32::kWaves, g1 = a.panels * (wave + 1) / Tile32::kWaves;
  uint8_t* mine = smem + wave * 2 * kBuf;
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_addr(mine));
  const int64_t off = (int64_t)y * a.bstride;
  // rows behind an operand's end read its last row: the epilogue drops them
  auto row_of = [&](int first, int lim) { return (uint32_t)(first < lim ? first : lim - 1); };
  auto load = [&](int g, int buf) {
    const uint32_t to = lds0 + (uint32_t)(buf * kBuf);
    const uint8_t* p = a.p.data + off + (int64_t)g * a.p.rows * 128;
    const uint8_t* q = a.q.data + off + (int64_t)g * a.q.rows * 128;
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // what the buffer held has been read
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int dr = 8 * k + (lane >> 3);
      const uint32_t chunk = (uint32_t)(((lane & 7) ^ swizzle(dr)) << 4);
      dma16(p, row_of(I * 32 + dr, a.M) * 128u + chunk, to + (uint32_t)(k * 1024));
      dma16(q, row_of(J * 32 + dr, a.N) * 128u + chunk, to + (uint32_t)(4096 + k * 1024));
    }
    if constexpr (FP4) {
      const uint32_t word = 4u * (uint32_t)(lane & 1);
      dma4(a.p.scales + (int64_t)g * a.p.rows * 8, row_of(I * 32 + (lane >> 1), a.M) * 8u + word, to + 8192u);
      dma4(a.q.scales + (int64_t)g * a.q.rows * 8, row_of(J * 32 + (lane >> 1), a.N) * 8u + word, to + 8448u);
    }
  };
  floatx16 acc[1][1];
  clear<Tile32>(acc);
  if (g0 < g1) load(g0, 0);
  for (int g = g0; g < g1; ++g) {
    const int buf = (g - g0) & 1;
    if (g + 1 < g1) {
      load(g + 1, buf ^ 1);
      asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kLoads) : "memory");
    } else {
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    }
    const uint8_t* st = mine + buf * kBuf + r * 128;
    uint2 sx = make_uint2(0, 0), sw = make_uint2(0, 0);
    if constexpr (FP4) {
      sx = *reinterpret_cast<const uint2*>(mine + buf * kBuf + 8192 + r * 8);
      sw = *reinterpret_cast<const uint2*>(mine + buf * kBuf + 8448 + r * 8);
    }
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const int at = ((2 * s + h) ^ swizzle(r)) << 4;
      const intx4 x = *reinterpret_cast<const intx4*>(st + at), w = *reinterpret_cast<const intx4*>(st + 4096 + at);
      const int shift = 16 * (s & 1) + 8 * h;      // byte 2 s + h of the eight
      if constexpr (FP4)
        acc[0][0] = mfma_fp4<0>(x, w, acc[0][0], (s < 2 ? sx.x : sx.y) >> shift, (s < 2 ? sw.x : sw.y) >> shift);
      else
        acc[0][0] = mfma_f16(x, w, acc[0][0]);
    }
  }
  // the sums take the first buffers' place, the epilogue wave 0's second
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  wave_sync();
#pragma unroll
  for (int k = 0; k < 4; ++k)
    *reinterpret_cast<float4*>(mine + (k * 64 + lane) * 16) =
        make_float4(acc[0][0][4 * k], acc[0][0][4 * k + 1], acc[0][0][4 * k + 2], acc[0][0][4 * k + 3]);
  __syncthreads();
  if (wave != 0) return;
#pragma unroll
  for (int v = 1; v < Tile32::kWaves; ++v)
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float4 o = *reinterpret_cast<const float4*>(smem + v * 2 * kBuf + (k * 64 + lane) * 16);
      acc[0][0][4 * k] += o.x;
      acc[0][0][4 * k + 1] += o.y;
      acc[0][0][4 * k + 2] += o.z;
      acc[0][0][4 * k + 3] += o.w;
    }
  epilogue<Tile32, EP, OT, VEC>(a, e.n, acc, y, I, J, 0, 0, lane, smem + kBuf, tile_din(a, y, I * 32, J * 32));
}

// Small matrices: B's rows are made where they are used, by every workgroup
// for itself, and never leave LDS -- one launch for B = a I + b A + c A^2 and
// the product with it.  A workgroup has 32 rows of B: the whole of A comes
// into LDS, eight waves divide the rows' 32 x 32 blocks, and then take one
// 32-row block of the other operand each.  B's blocks are computed transposed,
// so that a lane's four neighbours are neighbours of B's row.  Bound by its
// launch and two or three trips to memory, 5 to 8 us.
// FLIP: B is the product's right operand.
template <PanelEp EP, Dt OT, bool VEC, bool FLIP>
__global__ __launch_bounds__(512, 2) void panel_poly_kernel(const Each e, Args a) {
  // A, then (where both fit, behind it) each wave's block of the other
  // operand, whose place becomes the wave's epilogue scratch: all of the
  // largest A and one wave's block, so that a wave with A's time to load its
  // own does (256 x 512: 67.6 us with the block loaded afterwards, 66.0 so).
  // With B's rows that is the whole LDS; their factors go where A was.
  constexpr int kRoom = kPolyPanels * kPolyPanels * 8192 + kPolyPanels * 4096;
  __shared__ __attribute__((aligned(16))) uint8_t smem[kRoom + kPolyPanels * 4096];
  uint8_t* bt = smem + kRoom;
  const int lane = threadIdx.x & 63, r = lane & 31, h = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int stripes = FLIP ? a.TN : a.TM, blocks = FLIP ? a.TM : a.TN, groups = (blocks + a.wave_blocks - 1) / a.wave_blocks;
  const int S = (int)blockIdx.x % stripes, rest = (int)blockIdx.x / stripes;
  const int y = rest / groups, T = rest % groups * a.wave_blocks + wave;
  const int64_t off = (int64_t)y * a.bstride;
  const int panels = a.panels, lim = FLIP ? a.M : a.N;
  const PanelOperand& o = FLIP ? a.p : a.q;
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_addr(smem));
  const int asize = panels * panels * 8192, xsize = panels * 4096;       // bytes; xsize: of a wave's block
  const bool both = asize + a.wave_blocks * xsize <= kRoom;
  const int x0 = (both ? asize : 0) + wave * xsize;
  float* factor = reinterpret_cast<float*>(smem + (both ? 0 : kRoom - 128));

  const uint8_t* A = a.a + off;
  {
    const uint32_t src = (uint32_t)((lane >> 3) * 128 + (((lane & 7) ^ swizzle(8 * wave + (lane >> 3))) << 4));
    for (int i = wave; i < panels * panels * 8; i += 8) dma16(A, src + i * 1024u, lds0 + i * 1024u);
  }
  const bool mine = wave < a.wave_blocks && T < blocks;
  auto load_x = [&] {
    const uint8_t* data = o.data + off;
    for (int g = 0; g < panels; ++g, data += o.rows * 128)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        // rows behind the operand's end read its last row: the epilogue drops them
        int row = T * 32 + 8 * k + (lane >> 3);
        row = row < lim ? row : lim - 1;
        dma16(data, (uint32_t)row * 128u + (uint32_t)(((lane & 7) ^ swizzle(8 * k + (lane >> 3))) << 4),
              lds0 + (uint32_t)(x0 + (g * 4 + k) * 1024));
      }
  };
  if (both && mine) load_x();
  const float* D = moved(a.da, off);
  const float ds = D[S * 32 + r];
  float4 dj[4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    dj[k] = *reinterpret_cast<const float4*>(D + (wave < 2 * panels ? wave : 0) * 32 + 8 * k + 4 * h);
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  all_waves();

  // a 32-row block's fragment of step s, chunk 2 s + h of each row
  auto frag = [&](const uint8_t* block, int s) {
    return *reinterpret_cast<const intx4*>(block + r * 128 + (((2 * s + h) ^ swizzle(r)) << 4));
  };
  floatx16 acc[1][1];
  float mine_factor = 0.0f;
  static_assert(2 * kPolyPanels <= 8, "a block of B each");
  if (wave < 2 * panels) {
    const int j = wave;
    clear<Tile32>(acc);
    for (int g = 0; g < panels; ++g)
#pragma unroll
      for (int s = 0; s < 4; ++s)
        acc[0][0] = mfma_f16(frag(smem + g * panels * 8192 + j * 4096, s), frag(smem + g * panels * 8192 + S * 4096, s), acc[0][0]);
    // value 4 k + t: column 32 j + 8 k + 4 h + t of B's row 32 S + r
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int chunk = (((j & 1) * 4 + k) ^ swizzle(r)) << 4;
      const uint2 w = *reinterpret_cast<const uint2*>(smem + (j >> 1) * panels * 8192 + (S * 32 + r) * 128 + chunk + 8 * h);
      const float dv[4] = {dj[k].x, dj[k].y, dj[k].z, dj[k].w};
      const float av[4] = {f16_lo(w.x), f16_hi(w.x), f16_lo(w.y), f16_hi(w.y)};
#pragma unroll
      for (int t = 0; t < 4; ++t) {
        const float v = fmaf(a.cc, fmaf(dv[t] + ds, av[t], acc[0][0][4 * k + t]), a.cb * av[t]);
        acc[0][0][4 * k + t] = j == S && 8 * k + 4 * h + t == r ? v + fmaf(a.cb, ds, a.ca) : v;
      }
      *reinterpret_cast<uint2*>(bt + (j >> 1) * 4096 + r * 128 + chunk + 8 * h) =
          make_uint2(pack_f16(acc[0][0][4 * k], acc[0][0][4 * k + 1]),
                     pack_f16(acc[0][0][4 * k + 2], acc[0][0][4 * k + 3]));
    }
    if (j == S && on_diagonal(lane)) mine_factor = row_factor(diagonal_of(acc[0][0], lane));
  }
  // B is there, and nobody reads A any more
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  all_waves();
  if (wave == S && on_diagonal(lane)) factor[r] = mine_factor;
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  all_waves();
  if (!mine) return;
  if (!both) {
    load_x();
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  }
  clear<Tile32>(acc);
  for (int g = 0; g < panels; ++g)
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      const intx4 b = frag(bt + g * 4096, s), x = frag(smem + x0 + g * 4096, s);
      acc[0][0] = FLIP ? mfma_f16(x, b, acc[0][0]) : mfma_f16(b, x, acc[0][0]);
    }
  wave_sync();
  epilogue<Tile32, EP, OT, VEC>(a, e.n, acc, y, FLIP ? T : S, FLIP ? S : T, 0, 0, lane, smem + x0, factor);
}

template <class C, bool FP4, PanelEp EP, Dt OT, bool VEC>
hipError_t launch_one(const Each& e, const Args& a, const PanelPlan& p, hipStream_t s) {
  if constexpr (C::B == 32 && !FP4 && (EP == PanelEp::Out || EP == PanelEp::Step || EP == PanelEp::Iter))
    if (a.da) return launch_poly<EP, OT, VEC>(e, a, s);
  if constexpr (C::B == 32) {
    panel_direct_kernel<FP4, EP, OT, VEC><<<dim3((unsigned)p.groups), C::kThreads, 0, s>>>(e, a);
    return hipGetLastError();
  } else {
    panel_kernel<C, FP4, EP, OT, VEC><<<dim3((unsigned)p.groups), C::kThreads, 0, s>>>(e, a);
    const hipError_t r = hipGetLastError();
    if (r != hipSuccess || p.split_tiles == 0) return r;
    panel_sum_kernel<C, EP, OT, VEC><<<dim3((unsigned)(p.split_tiles * C::FM * C::FN)), C::kThreads, 0, s>>>(e, a);
    return hipGetLastError();
  }
}

template <class C, bool FP4, PanelEp EP, Dt OT>
hipError_t launch(const Each& e, const Args& a, const PanelPlan& p, hipStream_t s) {
  if constexpr (EP == PanelEp::Out || EP == PanelEp::Step)
    if (a.N % 8 != 0) return launch_one<C, FP4, EP, OT, false>(e, a, p, s);
  return launch_one<C, FP4, EP, OT, true>(e, a, p, s);
}

// Workgroups of panel_poly_kernel: `stripes` of B's rows, each with the other
// operand's `blocks`, `each` to a workgroup.
int64_t poly_groups(int64_t stripes, int64_t blocks, int each, int batch) {
  return stripes * ((blocks + each - 1) / each) * batch;
}

template <PanelEp EP, Dt OT, bool VEC>
hipError_t launch_poly(const Each& e, Args a, hipStream_t s) {
  const int stripes = a.din_cols ? a.TN : a.TM, blocks = a.din_cols ? a.TM : a.TN;
  // the fewest blocks a workgroup that leave one workgroup to a CU (256 x 512:
  // 67 us with 1, 73 with 8; 128 x 4096: 108 with 1, in two rounds, 89 with 4)
  a.wave_blocks = 1;
  while (a.wave_blocks < 8 && poly_groups(stripes, blocks, a.wave_blocks, a.batch) > kXcds * kCusPerXcd) a.wave_blocks *= 2;
  const dim3 grid((unsigned)poly_groups(stripes, blocks, a.wave_blocks, a.batch));
  if constexpr (EP != PanelEp::Iter)
    if (a.din_cols) {
      panel_poly_kernel<EP, OT, VEC, true><<<grid, 512, 0, s>>>(e, a);
      return hipGetLastError();
    }
  panel_poly_kernel<EP, OT, VEC, false><<<grid, 512, 0, s>>>(e, a);
  return hipGetLastError();
}

template <class C>
hipError_t launch_tile(const PanelProblem& g, const Each& e, const Args& a, const PanelPlan& p, bool fp4,
                       hipStream_t s) {
  if (fp4)                               // MXFP4 products have the plain epilogue only
    return g.ot == Dt::F32 ? launch<C, true, PanelEp::Out, Dt::F32>(e, a, p, s)
                           : launch<C, true, PanelEp::Out, Dt::BF16>(e, a, p, s);
  switch (g.ep) {
    case PanelEp::Out:
      return g.ot == Dt::F32 ? launch<C, false, PanelEp::Out, Dt::F32>(e, a, p, s)
                             : launch<C, false, PanelEp::Out, Dt::BF16>(e, a, p, s);
    case PanelEp::Step:
      return g.ot == Dt::F32 ? launch<C, false, PanelEp::Step, Dt::F32>(e, a, p, s)
                             : launch<C, false, PanelEp::Step, Dt::BF16>(e, a, p, s);
    case PanelEp::Gram: return launch<C, false, PanelEp::Gram, Dt::F32>(e, a, p, s);
    case PanelEp::Poly:
      if constexpr (C::B < 256) return launch<C, false, PanelEp::Poly, Dt::F32>(e, a, p, s);
      break;
    case PanelEp::Iter: return launch<C, false, PanelEp::Iter, Dt::F32>(e, a, p, s);
  }
  return hipErrorInvalidValue;
}

// The runs of a plan's tiles.  split: K-parts of the tiles that do not fill a
// round of the slots.
void runs_of(int tiles, int slots, int parts, Run (&run)[kXcds]) {
  int split0 = 0;
  for (int x = 0; x < kXcds; ++x) {
    Run& r = run[x];
    r.t0 = (int)((int64_t)x * tiles / kXcds);
    const int n = (int)((int64_t)(x + 1) * tiles / kXcds) - r.t0;
    r.whole = parts > 1 ? n / slots * slots : n;
    r.units = r.whole + (n - r.whole) * parts;
    r.split0 = split0;
    split0 += n - r.whole;
  }
}

template <class C>
PanelPlan plan_tile(int64_t M, int64_t N, bool sym, int batch, int parts) {
  PanelPlan p;
  p.tile = C::B;
  p.parts = parts;
  p.ws_bytes = 0;
  p.TM = (int)((M + C::B - 1) / C::B);
  p.TN = (int)((N + C::B - 1) / C::B);
  p.tiles = sym ? p.TM * (p.TM + 1) / 2 : p.TM * p.TN;
  p.slots = C::kBlocks * kCusPerXcd;
  Run run[kXcds];
  runs_of(p.tiles * batch, p.slots, parts, run);
  int most = 0;
  p.split_tiles = 0;
  for (const Run& r : run) {
    most = r.units > most ? r.units : most;
    if (parts > 1) p.split_tiles += (r.units - r.whole) / parts;
  }
  p.groups = C::B == 32 ? p.tiles * batch : (most < p.slots ? most : p.slots) * kXcds;
  p.ws_bytes = (size_t)p.split_tiles * parts * C::kAcc * C::kThreads * sizeof(float);
  return p;
}

PanelPlan plan_at(int tile, int64_t M, int64_t N, bool sym, int batch, int parts) {
  switch (tile) {
    case 256: return plan_tile<Tile256>(M, N, sym, batch, parts);
    case 128: return plan_tile<Tile128>(M, N, sym, batch, parts);
    case 64: return plan_tile<Tile64>(M, N, sym, batch, parts);
    default: return plan_tile<Tile32>(M, N, sym, batch, parts);
  }
}

// Microseconds that a plan takes, from measured products of random operands
// (256 CUs; MXFP4 and f16 cost the same per panel).  A round is one tile per
// slot; its time per panel grows with the tiles in it, since a full chip's
// matrix units run at a lower clock:
//   tile  slots  tiles: us per panel       once a round  once
//    256    256    64: 1.20   256: 1.75          3         6
//    128    512   256: 0.62   512: 1.10          2         4
//     64    512   256: 0.36   512: 0.47          1         3
//     32    256   0.55 per panel of a wave (an eighth of them), 2.3 a round, 0.8 once
// Measured against this: 4096^2 x 4096 38 us on 256 (43 on 128, 73 on 64),
// 2048^2 x 4096 16 us on 128 (27 on 256, 20 on 64), 1024^2 x 4096 9 us on 64
// (26 and 14).  A split adds its partials' traffic and the second kernel:
// 1024^2 x 16384 takes 43 us on 128 whole, 23 in 4 parts.  Tiles of 32 against
// 64: 64^2 with 32 panels 5.5 us (9.0), 512 x 768 with 16 panels 7.9 (10.9), with
// 2 panels 6.0 (4.6), 1024^2 with 16 panels 15.0 (11.8).
double plan_cost(const PanelPlan& p, int64_t panels, int batch) {
  if (p.tile == 32) return 0.8 + ((int64_t)p.tiles * batch + 255) / 256 * (2.3 + 0.55 * ((panels + 7) / 8));
  const double slots = p.slots * kXcds;
  const int few = p.tile == 256 ? 64 : 256;
  const double low = p.tile == 256 ? 1.20 : p.tile == 128 ? 0.62 : 0.36;
  const double high = p.tile == 256 ? 1.75 : p.tile == 128 ? 1.10 : 0.47;
  const double round = p.tile == 256 ? 3 : p.tile == 128 ? 2 : 1;
  auto per_panel = [&](double tiles) {
    if (tiles <= few) return low;
    return tiles >= slots ? high : low + (high - low) * (tiles - few) / (slots - few);
  };
  const int64_t all = (int64_t)p.tiles * batch;
  const int64_t whole = p.parts > 1 ? all - p.split_tiles : all;
  auto rounds = [&](int64_t units, double g) {
    const int64_t full = units / (int64_t)slots, rest = units % (int64_t)slots;
    return full * (round + g * high) + (rest ? round + g * per_panel((double)rest) : 0.0);
  };
  double us = round * 2 + rounds(whole, (double)panels);
  if (p.split_tiles)
    us += rounds((int64_t)p.split_tiles * p.parts, (double)panels / p.parts) + 2.0 + 2.0 * (double)p.ws_bytes / 5e6;
  return us;
}

}  // namespace

bool poly_in_product(int64_t mp, int64_t np, int batch) {
  return mp <= 64 * kPolyPanels && poly_groups(mp / 32, np / 32, 8, batch) <= kXcds * kCusPerXcd;
}
PanelPlan plan_panel_poly(int64_t M, int64_t N, int batch) { return plan_tile<Tile32>(M, N, false, batch, 1); }

PanelPlan plan_panel(int64_t M, int64_t N, int64_t panels, bool sym, int batch, bool allow_split, bool poly) {
  PanelPlan best{};
  double least = 0.0;
  for (int tile : {256, 128, 64, 32}) {
    if (tile == 256 && poly) continue;
    for (int parts : {1, 2, 4, 8}) {
      if (parts > 1 && (!allow_split || parts > panels || tile == 32)) break;
      const PanelPlan p = plan_at(tile, M, N, sym, batch, parts);
      const double us = plan_cost(p, panels, batch);
      if (least == 0.0 || us < least) {
        least = us;
        best = p;
      }
    }
  }
  return best;
}

hipError_t launch_panel(const PanelProblem& g, const PanelPlan& p, bool fp4, void* ws, hipStream_t s) {
  if (g.batch < 1 || g.batch > kMaxPanelBatch) return hipErrorInvalidValue;
  Args a{};
  a.p = g.p;
  a.q = g.q;
  a.M = (int)g.M;
  a.N = (int)g.N;
  a.panels = (int)g.panels;
  a.TM = p.TM;
  a.TN = p.TN;
  a.tiles = p.tiles;
  a.batch = g.batch;
  a.parts = p.parts;
  a.parts_inv = (65536u + (uint32_t)p.parts - 1) / (uint32_t)p.parts;
  a.slots = p.slots;
  a.sym = g.sym ? 1 : 0;
  a.partials = static_cast<float*>(ws);
  a.alpha = g.alpha;
  a.beta = g.beta;
  a.ca = g.ca;
  a.cb = g.cb;
  a.cc = g.cc;
  a.dalpha = g.dalpha;
  a.addend = g.addend;
  a.out = static_cast<uint8_t*>(g.out);
  a.out_t = static_cast<uint8_t*>(g.out_t);
  a.a = g.a;
  a.din = g.din;
  a.da = g.da;
  a.dout = g.dout;
  a.din_cols = g.din_cols ? 1 : 0;
  a.bstride = g.bstride;
  Each e;
  runs_of(p.tiles * g.batch, p.slots, p.parts, e.run);
  e.n = g.out_each ? g.batch : 0;
  for (int i = 0; i < kMaxPanelBatch; ++i) {
    e.out[i] = i < e.n ? g.out_each[i] : nullptr;
    e.alpha[i] = i < e.n && g.alpha_each ? g.alpha_each[i] : 1.0f;
  }
  switch (p.tile) {
    case 256: return launch_tile<Tile256>(g, e, a, p, fp4, s);
    case 128: return launch_tile<Tile128>(g, e, a, p, fp4, s);
    case 64: return launch_tile<Tile64>(g, e, a, p, fp4, s);
    default: return launch_tile<Tile32>(g, e, a, p, fp4, s);
  }
}

}  // namespace nvfp4

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
// by the dword, one for a lane's four steps.  Stages alternate between two
// buffers: while one is multiplied the next loads.
//
// Tiles left over after an equal number per CU are split along K into parts
// whose FP32 partials a second kernel sums in part order.
#include <cstddef>

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
using Tile64 = Tile<64, 2, 2, 3, 3>;

struct Args {
  PanelOperand p, q;
  int M, N, panels;
  int TM, TN, tiles, parts, slots, sym;
  float* partials;
  int64_t part_stride;          // bytes between the problems' partials
  // epilogue
  float alpha, beta, ca, cb, cc;
  const float* dalpha;
  const float* addend;
  uint8_t* out;
  uint8_t* out_t;
  const uint8_t* a;
  int64_t bstride;
};

// Row-major outputs of a batch, one by one (n > 0).  The first argument of
// the kernels, so that it sits at the start of the kernel-argument segment:
// the entry of problem y is then two scalar loads from there.
struct Each {
  int n;
  float alpha[kMaxPanelBatch];
  void* out[kMaxPanelBatch];
};
static_assert(offsetof(Each, alpha) == 4 && offsetof(Each, out) == 8 + 4 * kMaxPanelBatch, "Each layout");

__device__ __forceinline__ void pick_output(Args& a, int y) {
  typedef const __attribute__((address_space(4))) uint8_t* KBytes;
  typedef uint8_t* const __attribute__((address_space(4)))* KPtr;
  typedef const __attribute__((address_space(4))) float* KFloat;
  const KBytes k = (KBytes)__builtin_amdgcn_kernarg_segment_ptr();
  a.out = ((KPtr)(k + offsetof(Each, out)))[y];
  a.alpha *= ((KFloat)(k + offsetof(Each, alpha)))[y];
}

template <class T>
__device__ __forceinline__ T* moved(T* p, int64_t off) {
  return p ? reinterpret_cast<T*>(reinterpret_cast<uintptr_t>(p) + off) : p;
}

__device__ __forceinline__ void pick_problem(Args& a, int nout) {
  const int y = (int)blockIdx.y;
  const int64_t off = (int64_t)y * a.bstride;
  a.p.data = moved(a.p.data, off);
  a.q.data = moved(a.q.data, off);
  a.dalpha = moved(a.dalpha, off);
  a.a = moved(a.a, off);
  a.out_t = moved(a.out_t, off);
  a.partials = moved(a.partials, (int64_t)y * a.part_stride);
  if (nout)
    pick_output(a, y);
  else
    a.out = moved(a.out, off);
}

// ---- schedule ----------------------------------------------------------------
// The tiles are cut into kXcds contiguous runs, one per XCD, in an order that
// keeps a run's tiles in a compact patch (they share the XCD's L2).  Of a
// run's n tiles the first n / slots * slots run whole (slots: workgroups
// resident on an XCD) and the rest, when parts > 1, in K-parts.

struct Unit {
  int tile, part, split;        // split: index among the split tiles, -1 for a whole tile
};

__host__ __device__ inline void run_of(int tiles, int slots, int parts, int x, int& t0, int& n, int& whole) {
  t0 = (int)((int64_t)x * tiles / kXcds);
  n = (int)((int64_t)(x + 1) * tiles / kXcds) - t0;
  whole = parts > 1 ? n / slots * slots : n;
}

__device__ __forceinline__ bool unit_of(const Args& a, int b, Unit& u) {
  const int x = b % kXcds, l = b / kXcds;
  int t0, n, whole;
  run_of(a.tiles, a.slots, a.parts, x, t0, n, whole);
  u.part = 0;
  u.split = -1;
  u.tile = t0 + l;
  if (l < whole) return true;
  const int r = l - whole;
  if (r >= (n - whole) * a.parts) return false;
  int base = 0;
  for (int y = 0; y < x; ++y) {
    int ty, ny, wy;
    run_of(a.tiles, a.slots, a.parts, y, ty, ny, wy);
    base += ny - wy;
  }
  u.tile = t0 + whole + r / a.parts;
  u.part = r % a.parts;
  u.split = base + r / a.parts;
  return true;
}

__device__ __forceinline__ int split_tile(const Args& a, int s) {
  for (int x = 0; x < kXcds; ++x) {
    int t0, n, whole;
    run_of(a.tiles, a.slots, a.parts, x, t0, n, whole);
    if (s < n - whole) return t0 + whole + s;
    s -= n - whole;
  }
  return 0;
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

// ---- loads -------------------------------------------------------------------
// Global -> LDS DMA: lane l's bytes land at lds + 16 l (4 l).  Inline asm, so
// that the compiler does not take the LDS write as pending before every later
// LDS read; ordered by s_waitcnt vmcnt and the stage's barrier.  There are no
// register results, and the address operands are read at issue.
__device__ __forceinline__ uint32_t lds_addr(const void* p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)p;
}
__device__ __forceinline__ void dma16(const uint8_t* base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\tglobal_load_lds_dwordx4 %0, %1" ::"v"(off), "s"(base), "s"(lds) : "memory", "m0");
}
__device__ __forceinline__ void dma4(const uint8_t* base, uint32_t off, uint32_t lds) {
  asm volatile("s_mov_b32 m0, %2\n\tglobal_load_lds_dword %0, %1" ::"v"(off), "s"(base), "s"(lds) : "memory", "m0");
}

// Depends on r % 32 alone, so that a fragment's LDS address is one per-lane
// offset for each step plus a constant for its 32-row block.
__device__ __forceinline__ int swizzle(int r) { return (r ^ ((r & 31) >> 3)) & 7; }

// Byte offsets of a lane's loads inside a panel.  Rows past the operand's end
// read its last row: they feed only outputs that the epilogue does not write.
template <class C, bool FP4>
struct Src {
  uint32_t code[C::kCodeLoads];
  uint32_t scale[FP4 ? C::kScaleLoads : 1];
};

template <class C, bool FP4>
__device__ __forceinline__ void init_src(const Args& a, int m0, int n0, int wave, int lane, Src<C, FP4>& s) {
#pragma unroll
  for (int i = 0; i < C::kCodeLoads; ++i) {
    const int r = 8 * (wave * C::kCodeLoads + i) + (lane >> 3);      // operand row of the stage
    int row = r < C::B ? m0 + r : n0 + r - C::B;
    const int lim = r < C::B ? a.M : a.N;
    row = row < lim ? row : lim - 1;
    s.code[i] = (uint32_t)row * 128u + 16u * (uint32_t)((lane & 7) ^ swizzle(r));
  }
  if constexpr (FP4) {
#pragma unroll
    for (int i = 0; i < C::kScaleLoads; ++i) {
      const int r = 32 * (wave * C::kScaleLoads + i) + (lane >> 1);
      int row = r < C::B ? m0 + r : n0 + r - C::B;
      const int lim = r < C::B ? a.M : a.N;
      row = row < lim ? row : lim - 1;
      s.scale[i] = (uint32_t)row * 8u + 4u * (uint32_t)(lane & 1);
    }
  }
}

// Load number k of a wave's share of a stage.  A share never straddles the
// operands: B rows are a multiple of it.
template <class C, bool FP4>
struct Issue {
  static constexpr int kLoads = C::kCodeLoads + (FP4 ? C::kScaleLoads : 0);
  const uint8_t *data, *scales;        // the wave's operand
  int64_t rows;
  uint32_t code0, scale0;              // LDS offsets of the wave's share in a stage

  __device__ __forceinline__ Issue(const Args& a, int wave) {
    const bool isP = wave * C::kCodeLoads * 8 < C::B;
    data = isP ? a.p.data : a.q.data;
    scales = isP ? a.p.scales : a.q.scales;
    rows = isP ? a.p.rows : a.q.rows;
    code0 = (uint32_t)(wave * C::kCodeLoads) * 1024u;
    scale0 = (uint32_t)C::kCodeBytes + (uint32_t)(wave * C::kScaleLoads) * 256u;
  }
  __device__ __forceinline__ void load(const Src<C, FP4>& s, int g, uint32_t stage, int k) const {
    if (k < C::kCodeLoads)
      dma16(data + (int64_t)g * rows * 128, s.code[k], stage + code0 + 1024u * k);
    else if constexpr (FP4)
      dma4(scales + (int64_t)g * rows * 8, s.scale[k - C::kCodeLoads], stage + scale0 + 256u * (k - C::kCodeLoads));
  }
};

// ---- multiply ------------------------------------------------------------------
template <int S>
__device__ __forceinline__ floatx16 mfma_fp4(intx4 a, intx4 b, floatx16 c, uint32_t sa, uint32_t sb) {
  const intx8 x = {a[0], a[1], a[2], a[3], 0, 0, 0, 0}, y = {b[0], b[1], b[2], b[3], 0, 0, 0, 0};
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

// Two lanes that hold columns c and c + 1 of four rows (lo: rows 0 and 1
// packed, hi: rows 2 and 3) exchange halves: the even lane ends with the
// column pairs of rows 0 and 1, the odd one with those of rows 2 and 3.
__device__ __forceinline__ void pair_columns(uint32_t lo, uint32_t hi, bool odd, uint32_t& first, uint32_t& second) {
  const uint32_t give = odd ? lo : hi, keep = odd ? hi : lo;
  const uint32_t got = (uint32_t)__builtin_amdgcn_mov_dpp((int)give, 0xB1, 0xF, 0xF, true);
  const uint32_t a = odd ? got : keep, b = odd ? keep : got;     // a: column c, b: column c + 1
  first = __builtin_amdgcn_perm(b, a, 0x05040100u);
  second = __builtin_amdgcn_perm(b, a, 0x07060302u);
}

// The tile as 16-bit values in LDS, row-major with a padded pitch; `words`
// holds, per block and quad, the lane's four rows packed in pairs.
template <class C>
struct Stage16 {
  static constexpr int kPitch = C::B * 2 + 16;
  static constexpr int kBytes = C::B * kPitch;
};

template <class C>
struct Words {
  uint32_t w[C::FM][C::FN][4][2];
};
template <class C, Dt T>
__device__ __forceinline__ void pack_tile(const floatx16 (&acc)[C::FM][C::FN], Words<C>& w) {
#pragma unroll
  for (int i = 0; i < C::FM; ++i)
#pragma unroll
    for (int j = 0; j < C::FN; ++j) {
#pragma unroll
      for (int q = 0; q < 8; ++q)
        w.w[i][j][q >> 1][q & 1] = T == Dt::BF16 ? mx::pack_bf16(acc[i][j][2 * q], acc[i][j][2 * q + 1])
                                                 : pack_f16(acc[i][j][2 * q], acc[i][j][2 * q + 1]);
      __builtin_amdgcn_sched_barrier(0);
    }
}

template <class C>
__device__ __forceinline__ void stage_rows(uint8_t* lds, int wm, int wn, int lane, const Words<C>& w) {
  const int h = lane >> 5, c = lane & 31;
  const bool odd = lane & 1;
#pragma unroll
  for (int i = 0; i < C::FM; ++i)
#pragma unroll
    for (int j = 0; j < C::FN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint32_t first, second;
        pair_columns(w.w[i][j][q][0], w.w[i][j][q][1], odd, first, second);
        const int row = (wm * C::FM + i) * 32 + 8 * q + 4 * h + (odd ? 2 : 0);
        const int col = (wn * C::FN + j) * 32 + (c & ~1);
        *reinterpret_cast<uint32_t*>(lds + row * Stage16<C>::kPitch + col * 2) = first;
        *reinterpret_cast<uint32_t*>(lds + (row + 1) * Stage16<C>::kPitch + col * 2) = second;
      }
}

// The transposed tile: row = the tile's column.
template <class C>
__device__ __forceinline__ void stage_cols(uint8_t* lds, int wm, int wn, int lane, const Words<C>& w) {
  const int h = lane >> 5, c = lane & 31;
#pragma unroll
  for (int i = 0; i < C::FM; ++i)
#pragma unroll
    for (int j = 0; j < C::FN; ++j)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int row = (wn * C::FN + j) * 32 + c, col = (wm * C::FM + i) * 32 + 8 * q + 4 * h;
        *reinterpret_cast<uint2*>(lds + row * Stage16<C>::kPitch + col * 2) =
            make_uint2(w.w[i][j][q][0], w.w[i][j][q][1]);
      }
}

// A staged tile to f16 panels: rows r0 .. of an operand with `rows` rows a
// panel, columns from c0 (a multiple of 64) up to `cols` (likewise).
template <class C>
__device__ __forceinline__ void store_panels(const uint8_t* lds, uint8_t* dst, int r0, int rows, int c0, int cols) {
  for (int k = (int)threadIdx.x; k < C::B * C::B / 8; k += C::kThreads) {
    const int ch = k & 7, r = (k >> 3) % C::B, g = (k >> 3) / C::B;      // chunk, row, panel of the tile
    if (r0 + r < rows && c0 + 64 * g < cols)
      *reinterpret_cast<uint4*>(dst + ((int64_t)(c0 / 64 + g) * rows + r0 + r) * 128 + 16 * ch) =
          *reinterpret_cast<const uint4*>(lds + r * Stage16<C>::kPitch + 128 * g + 16 * ch);
  }
}

// Barrier after this wave's LDS accesses (global stores stay in flight).
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

template <class C, PanelEp EP, Dt OT>
__device__ __forceinline__ void epilogue(const Args& a, floatx16 (&acc)[C::FM][C::FN], int I, int J, int wm, int wn,
                                         int lane, uint8_t* lds) {
  const int m0 = I * C::B, n0 = J * C::B, h = lane >> 5, c = lane & 31;
  const float alpha = a.dalpha ? a.alpha * *a.dalpha : a.alpha;
  const bool inside = m0 + C::B <= a.M && n0 + C::B <= a.N;
  if constexpr (EP == PanelEp::Step || EP == PanelEp::Out) {
    // element by element: 32 lanes cover 32 neighbouring columns
    const int64_t base = (int64_t)(m0 + wm * C::FM * 32 + 4 * h) * a.N + n0 + wn * C::FN * 32 + c;
    constexpr bool kStaged = EP == PanelEp::Out && OT == Dt::BF16;
#pragma unroll
    for (int i = 0; i < C::FM; ++i)
#pragma unroll
      for (int j = 0; j < C::FN; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) {
          const int dr = i * 32 + 8 * (r >> 2) + (r & 3), dc = j * 32;
          const int64_t at = base + (int64_t)dr * a.N + dc;
          const bool ok = inside || (m0 + wm * C::FM * 32 + 4 * h + dr < a.M && n0 + wn * C::FN * 32 + c + dc < a.N);
          float v = alpha * acc[i][j][r];
          if constexpr (EP == PanelEp::Out) {
            if (a.addend && ok) v = fmaf(a.beta, a.addend[at], v);
            if constexpr (kStaged) acc[i][j][r] = v;
            else if (ok) reinterpret_cast<float*>(a.out)[at] = v;
          } else if (ok) {
            if constexpr (OT == Dt::F32) {
              float* w = reinterpret_cast<float*>(a.out) + at;
              *w = fmaf(a.beta, *w, -v);
            } else {
              uint16_t* w = reinterpret_cast<uint16_t*>(a.out) + at;
              *w = (uint16_t)mx::pack_bf16(fmaf(a.beta, __uint_as_float((uint32_t)*w << 16), -v), 0.0f);
            }
          }
        }
    if constexpr (kStaged) {
      Words<C> w;
      pack_tile<C, Dt::BF16>(acc, w);
      lds_barrier();
      stage_rows<C>(lds, wm, wn, lane, w);
      lds_barrier();
      uint16_t* out = reinterpret_cast<uint16_t*>(a.out);
      const bool vec = a.N % 8 == 0;
      for (int k = (int)threadIdx.x; k < C::B * C::B / 8; k += C::kThreads) {
        const int ch = k % (C::B / 8), r = k / (C::B / 8);
        const int row = m0 + r, col = n0 + 8 * ch;
        if (row >= a.M || col >= a.N) continue;
        const uint4 v = *reinterpret_cast<const uint4*>(lds + r * Stage16<C>::kPitch + 16 * ch);
        uint16_t* o = out + (int64_t)row * a.N + col;
        if (vec) {
          *reinterpret_cast<uint4*>(o) = v;
        } else {
          const uint32_t e[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int t = 0; t < 8; ++t)
            if (col + t < a.N) o[t] = (uint16_t)(e[t >> 1] >> (16 * (t & 1)));
        }
      }
    }
  } else {
    if constexpr (EP == PanelEp::Poly) {
      // A is symmetric: rows 4 .. 7 of a column are four neighbours of a row
#pragma unroll
      for (int i = 0; i < C::FM; ++i)
#pragma unroll
        for (int j = 0; j < C::FN; ++j)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            const int row = m0 + (wm * C::FM + i) * 32 + 8 * q + 4 * h, col = n0 + (wn * C::FN + j) * 32 + c;
            uint2 w = make_uint2(0u, 0u);
            if (inside || (row < a.M && col < a.N))
              w = *reinterpret_cast<const uint2*>(a.a + ((int64_t)(row >> 6) * a.M + col) * 128 + (row & 63) * 2);
            const float av[4] = {f16_lo(w.x), f16_hi(w.x), f16_lo(w.y), f16_hi(w.y)};
#pragma unroll
            for (int t = 0; t < 4; ++t) {
              float v = fmaf(a.cc, acc[i][j][4 * q + t], a.cb * av[t]);
              acc[i][j][4 * q + t] = row + t == col ? v + a.ca : v;
            }
            if (q == 3) __builtin_amdgcn_sched_barrier(0);
          }
    } else {
#pragma unroll
      for (int i = 0; i < C::FM; ++i)
#pragma unroll
        for (int j = 0; j < C::FN; ++j)
#pragma unroll
          for (int r = 0; r < 16; ++r) acc[i][j][r] *= alpha;
    }
    Words<C> w;
    pack_tile<C, Dt::F32>(acc, w);                       // f16
    constexpr bool kIter = EP == PanelEp::Iter;
    uint8_t* tdst = kIter ? a.out_t : a.out;
    lds_barrier();
    stage_cols<C>(lds, wm, wn, lane, w);
    lds_barrier();
    // the transpose: rows n0 .., columns m0 ..; a symmetric product's mirror
    // (a diagonal tile is its own)
    store_panels<C>(lds, tdst, n0, a.N, m0, a.M);
    if (kIter || I != J) {
      lds_barrier();
      stage_rows<C>(lds, wm, wn, lane, w);
      lds_barrier();
      store_panels<C>(lds, a.out, m0, a.M, n0, a.N);
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

template <class C, bool FP4, PanelEp EP, Dt OT>
__global__ __launch_bounds__(C::kThreads, C::kBlocks* C::kWaves / 4) void panel_kernel(const Each e, Args a) {
  constexpr int kStage = stage_bytes<C, FP4>();
  __shared__ __attribute__((aligned(16)))
  uint8_t smem[C::NST * kStage > Stage16<C>::kBytes ? C::NST * kStage : Stage16<C>::kBytes];
  pick_problem(a, e.n);
  Unit un;
  if (!unit_of(a, (int)blockIdx.x, un)) return;
  int I, J;
  tile_of(a, un.tile, I, J);
  const int nparts = un.split < 0 ? 1 : a.parts;
  const int g0 = (int)((int64_t)a.panels * un.part / nparts), g1 = (int)((int64_t)a.panels * (un.part + 1) / nparts);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / C::WN, wn = wave % C::WN;

  floatx16 acc[C::FM][C::FN];
#pragma unroll
  for (int i = 0; i < C::FM; ++i)
#pragma unroll
    for (int j = 0; j < C::FN; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

  Src<C, FP4> src;
  init_src<C, FP4>(a, I * C::B, J * C::B, wave, lane, src);
  const Issue<C, FP4> dma(a, wave);
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane(lds_addr(smem));
  constexpr int kLoads = Issue<C, FP4>::kLoads, kReads = C::FM + C::FN, kMul = C::FM * C::FN;
  uint32_t off[4];
#pragma unroll
  for (int s = 0; s < 4; ++s)
    off[s] = (uint32_t)((lane & 31) * 128 + 16 * ((4 * (lane >> 5) + s) ^ swizzle(lane & 31)));
  const uint32_t soff = (uint32_t)((lane & 31) * 8 + 4 * (lane >> 5));
  Frags<C> f0, f1;
  Scales<C> sc;
  auto wait_loads = [&] { asm volatile("s_waitcnt vmcnt(%0)" ::"n"((C::NST - 2) * kLoads) : "memory"); };
  auto read_first = [&](const uint8_t* st) {
#pragma unroll
    for (int k = 0; k < kReads; ++k) {
      if constexpr (FP4) read_scale<C>(st, soff, wm, wn, k, sc);
      read_frag<C>(st, off[0], wm, wn, k, f0);
    }
  };
  // Stages g0 .. g0 + NST - 2 in flight, then always one more: a panel past
  // the last is the last again, into a buffer that nothing reads.
  auto panel = [&](int g) { return g < g1 ? g : g1 - 1; };
#pragma unroll
  for (int s = 0; s < C::NST - 1; ++s)
#pragma unroll
    for (int k = 0; k < kLoads; ++k) dma.load(src, panel(g0 + s), lds0 + s * kStage, k);
  wait_loads();
  __builtin_amdgcn_s_barrier();
  read_first(smem);
#pragma unroll
  for (int k = 0; k < kLoads; ++k) dma.load(src, panel(g0 + C::NST - 1), lds0 + (C::NST - 1) * kStage, k);

  int cur = 0;
  auto first_three = [&](const uint8_t* st) {
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
  };
  for (int g = g0; g + 1 < g1; ++g) {
    first_three(smem + cur * kStage);
    // every read of this stage has returned: its buffer is free once all
    // waves are here, and the next stage's loads have landed
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    wait_loads();
    __builtin_amdgcn_s_barrier();
    const uint32_t freed = lds0 + cur * kStage;
    cur = cur + 1 == C::NST ? 0 : cur + 1;
    const uint8_t* st = smem + cur * kStage;
    const int gn = panel(g + C::NST);
    Scales<C> nsc;
    step<C, FP4, 3>(f1, sc, acc, [&](int k) {
#pragma unroll
      for (int r = share(kReads, k, kMul); r < share(kReads, k + 1, kMul); ++r) {
        if constexpr (FP4) read_scale<C>(st, soff, wm, wn, r, nsc);
        read_frag<C>(st, off[0], wm, wn, r, f0);
      }
#pragma unroll
      for (int r = share(kLoads, k, kMul); r < share(kLoads, k + 1, kMul); ++r) dma.load(src, gn, freed, r);
    });
    if constexpr (FP4) sc = nsc;
  }
  first_three(smem + cur * kStage);
  step<C, FP4, 3>(f1, sc, acc, [](int) {});
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");       // the loads past the end, before LDS serves the epilogue

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
    return;
  }
  epilogue<C, EP, OT>(a, acc, I, J, wm, wn, lane, smem);
}

// One split tile a workgroup: its parts' partials, summed in part order.
template <class C, PanelEp EP, Dt OT>
__global__ __launch_bounds__(C::kThreads) void panel_sum_kernel(const Each e, Args a) {
  __shared__ __attribute__((aligned(16))) uint8_t smem[Stage16<C>::kBytes];
  pick_problem(a, e.n);
  const int split = (int)blockIdx.x;
  int I, J;
  tile_of(a, split_tile(a, split), I, J);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  floatx16 acc[C::FM][C::FN];
#pragma unroll
  for (int i = 0; i < C::FM; ++i)
#pragma unroll
    for (int j = 0; j < C::FN; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
  const float* part = a.partials + (size_t)split * a.parts * C::kAcc * C::kThreads;
  for (int p = 0; p < a.parts; ++p, part += (size_t)C::kAcc * C::kThreads) {
#pragma unroll
    for (int i = 0; i < C::FM; ++i)
#pragma unroll
      for (int j = 0; j < C::FN; ++j)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const float4 v = *reinterpret_cast<const float4*>(part + part_index<C>(i * C::FN + j, q, threadIdx.x));
          acc[i][j][4 * q] += v.x;
          acc[i][j][4 * q + 1] += v.y;
          acc[i][j][4 * q + 2] += v.z;
          acc[i][j][4 * q + 3] += v.w;
        }
  }
  epilogue<C, EP, OT>(a, acc, I, J, wave / C::WN, wave % C::WN, lane, smem);
}

template <class C, bool FP4, PanelEp EP, Dt OT>
hipError_t launch(const Each& e, const Args& a, const PanelPlan& p, int batch, hipStream_t s) {
  panel_kernel<C, FP4, EP, OT><<<dim3((unsigned)p.units, (unsigned)batch), C::kThreads, 0, s>>>(e, a);
  const hipError_t r = hipGetLastError();
  if (r != hipSuccess || p.split_tiles == 0) return r;
  panel_sum_kernel<C, EP, OT><<<dim3((unsigned)p.split_tiles, (unsigned)batch), C::kThreads, 0, s>>>(e, a);
  return hipGetLastError();
}

template <class C>
hipError_t launch_tile(const PanelProblem& g, const Each& e, const Args& a, const PanelPlan& p, bool fp4,
                       hipStream_t s) {
  const int b = g.batch;
  if (fp4)                               // MXFP4 products have the plain epilogue only
    return g.ot == Dt::F32 ? launch<C, true, PanelEp::Out, Dt::F32>(e, a, p, b, s)
                           : launch<C, true, PanelEp::Out, Dt::BF16>(e, a, p, b, s);
  switch (g.ep) {
    case PanelEp::Out:
      return g.ot == Dt::F32 ? launch<C, false, PanelEp::Out, Dt::F32>(e, a, p, b, s)
                             : launch<C, false, PanelEp::Out, Dt::BF16>(e, a, p, b, s);
    case PanelEp::Step:
      return g.ot == Dt::F32 ? launch<C, false, PanelEp::Step, Dt::F32>(e, a, p, b, s)
                             : launch<C, false, PanelEp::Step, Dt::BF16>(e, a, p, b, s);
    case PanelEp::Gram: return launch<C, false, PanelEp::Gram, Dt::F32>(e, a, p, b, s);
    case PanelEp::Poly: return launch<C, false, PanelEp::Poly, Dt::F32>(e, a, p, b, s);
    case PanelEp::Iter: return launch<C, false, PanelEp::Iter, Dt::F32>(e, a, p, b, s);
  }
  return hipErrorInvalidValue;
}

template <class C>
PanelPlan plan_tile(int64_t M, int64_t N, bool sym, int parts) {
  PanelPlan p;
  p.tile = C::B;
  p.parts = parts;
  p.TM = (int)((M + C::B - 1) / C::B);
  p.TN = (int)((N + C::B - 1) / C::B);
  p.tiles = sym ? p.TM * (p.TM + 1) / 2 : p.TM * p.TN;
  p.split_tiles = 0;
  int most = 0;
  for (int x = 0; x < kXcds; ++x) {
    int t0, n, whole;
    run_of(p.tiles, C::kBlocks * kCusPerXcd, parts, x, t0, n, whole);
    const int u = whole + (n - whole) * parts;
    most = u > most ? u : most;
    if (parts > 1) p.split_tiles += n - whole;
  }
  p.units = most * kXcds;
  p.ws_bytes = (size_t)p.split_tiles * parts * C::kAcc * C::kThreads * sizeof(float);
  return p;
}

PanelPlan plan_at(int tile, int64_t M, int64_t N, bool sym, int parts) {
  return tile == 256 ? plan_tile<Tile256>(M, N, sym, parts)
                     : tile == 128 ? plan_tile<Tile128>(M, N, sym, parts) : plan_tile<Tile64>(M, N, sym, parts);
}

}  // namespace

PanelPlan plan_panel(int64_t M, int64_t N, int64_t panels, bool sym, int batch, bool allow_split,
                     bool fp4) {
  (void)panels;
  (void)fp4;
  (void)allow_split;
  const int64_t big = (M < N ? M : N);
  const int tile = big >= 1024 ? 256 : big >= 256 ? 128 : 64;
  (void)batch;
  return plan_at(tile, M, N, sym, 1);
}

hipError_t launch_panel(const PanelProblem& g, const PanelPlan& p, bool fp4, void* ws, int64_t ws_stride,
                        hipStream_t s) {
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
  a.parts = p.parts;
  a.sym = g.sym ? 1 : 0;
  a.partials = static_cast<float*>(ws);
  a.part_stride = ws_stride;
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
  a.bstride = g.bstride;
  Each e;
  e.n = g.out_each ? g.batch : 0;
  for (int i = 0; i < kMaxPanelBatch; ++i) {
    e.out[i] = i < e.n ? g.out_each[i] : nullptr;
    e.alpha[i] = i < e.n && g.alpha_each ? g.alpha_each[i] : 1.0f;
  }
  switch (p.tile) {
    case 256: a.slots = Tile256::kBlocks * kCusPerXcd; return launch_tile<Tile256>(g, e, a, p, fp4, s);
    case 128: a.slots = Tile128::kBlocks * kCusPerXcd; return launch_tile<Tile128>(g, e, a, p, fp4, s);
    default: a.slots = Tile64::kBlocks * kCusPerXcd; return launch_tile<Tile64>(g, e, a, p, fp4, s);
  }
}

}  // namespace nvfp4

// MXFP4 quantizers and dequantizers: one pass over the data, since a block's
// scale depends on its own 32 values alone.  All are bound by memory; the
// kernels below only arrange that every global access moves whole lines.
#include "mxfp4_device.hpp"
#include "panel.hpp"

namespace nvfp4 {
namespace {
using namespace mx;

// ---- blocks along the rows --------------------------------------------------
// A lane owns 8 consecutive elements, four lanes a block, 32 lanes one row's
// panel (512 bytes of BF16 in, one 128-byte line of codes out).

template <class T> struct Io;
template <> struct Io<float> {
  static constexpr int kVec = 4;   // elements that must divide the pitch for 16-byte accesses
  static __device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
  static __device__ __forceinline__ float load1(const float* p) { return *p; }
  static __device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
  }
  static __device__ __forceinline__ void store1(float* p, float v) { *p = v; }
  // two neighbouring columns
  static __device__ __forceinline__ void store2(float* p, float a, float b) {
    *reinterpret_cast<float2*>(p) = make_float2(a, b);
  }
};
template <> struct Io<uint16_t> {   // BF16 bits
  static constexpr int kVec = 8;
  static __device__ __forceinline__ void load8(const uint16_t* p, float (&v)[8]) {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    v[0] = bf16_lo(a.x); v[1] = bf16_hi(a.x); v[2] = bf16_lo(a.y); v[3] = bf16_hi(a.y);
    v[4] = bf16_lo(a.z); v[5] = bf16_hi(a.z); v[6] = bf16_lo(a.w); v[7] = bf16_hi(a.w);
  }
  static __device__ __forceinline__ float load1(const uint16_t* p) { return __uint_as_float((uint32_t)*p << 16); }
  static __device__ __forceinline__ void store8(uint16_t* p, const float (&v)[8]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]),
                                              pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7]));
  }
  static __device__ __forceinline__ void store1(uint16_t* p, float v) { *p = (uint16_t)pack_bf16(v, 0.0f); }
  static __device__ __forceinline__ void store2(uint16_t* p, float a, float b) {
    *reinterpret_cast<uint32_t*>(p) = pack_bf16(a, b);
  }
};

constexpr int kRowsPerPass = 8;    // 256 threads: 8 rows of one panel
constexpr int kPasses = 4;         // row groups a workgroup handles

template <bool VEC, class T>
__device__ __forceinline__ void load_chunk(const T* x, int64_t row, int64_t cols, int64_t c, float (&v)[8]) {
  const T* p = x + row * cols + c;
  if (VEC) {
    if (c < cols) {                // a multiple of 8 elements is all in or all out
      Io<T>::load8(p, v);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0.0f;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c + i < cols ? Io<T>::load1(p + i) : 0.0f;
  }
}

// Largest magnitude of the four lanes of a block.
__device__ __forceinline__ uint32_t quad_max(uint32_t a) {
  a = umax(a, (uint32_t)__builtin_amdgcn_mov_dpp((int)a, 0xB1, 0xF, 0xF, true));   // lane ^ 1
  return umax(a, (uint32_t)__builtin_amdgcn_mov_dpp((int)a, 0x4E, 0xF, 0xF, true)); // lane ^ 2
}

template <class T, bool VEC>
__global__ __launch_bounds__(256) void quant_rows_kernel(const T* __restrict__ x, int64_t rows, int64_t cols,
                                                         uint32_t panels,
                                                         uint8_t* __restrict__ codes,
                                                         uint8_t* __restrict__ scales) {
  const int t = threadIdx.x, lane32 = t & 31;
  const int64_t g = blockIdx.x % panels;
  const int64_t r0 = (int64_t)(blockIdx.x / panels) * (kRowsPerPass * kPasses) + (t >> 5);
  const int64_t c = g * kPanel + 8 * lane32;
  float v[kPasses][8];
#pragma unroll
  for (int p = 0; p < kPasses; ++p)
    if (r0 + p * kRowsPerPass < rows) load_chunk<VEC>(x, r0 + p * kRowsPerPass, cols, c, v[p]);
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int64_t r = r0 + p * kRowsPerPass;
    if (r >= rows) break;          // whole 32-lane groups leave together
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) a = umax(a, mag_bits(v[p][i]));
    const uint32_t byte = scale_byte(quad_max(a));
    *reinterpret_cast<uint32_t*>(codes + (g * rows + r) * kPanelBytes + 4 * lane32) = encode8(v[p], byte);
    if ((lane32 & 3) == 0) scales[(g * rows + r) * kPanelScales + (lane32 >> 2)] = (uint8_t)byte;
  }
}

template <class T, bool VEC>
__global__ __launch_bounds__(256) void dequant_rows_kernel(const uint8_t* __restrict__ codes,
                                                           const uint8_t* __restrict__ scales, int64_t rows,
                                                           int64_t cols, uint32_t panels, T* __restrict__ out) {
  const int t = threadIdx.x, lane32 = t & 31;
  const int64_t g = blockIdx.x % panels;
  const int64_t r0 = (int64_t)(blockIdx.x / panels) * (kRowsPerPass * kPasses) + (t >> 5);
  const int64_t c = g * kPanel + 8 * lane32;
  uint32_t w[kPasses], b[kPasses];
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int64_t r = r0 + p * kRowsPerPass;
    if (r < rows) {
      w[p] = *reinterpret_cast<const uint32_t*>(codes + (g * rows + r) * kPanelBytes + 4 * lane32);
      b[p] = scales[(g * rows + r) * kPanelScales + (lane32 >> 2)];
    }
  }
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int64_t r = r0 + p * kRowsPerPass;
    if (r >= rows || c >= cols) break;
    float v[8];
    decode8(w[p], b[p], v);
    T* o = out + r * cols + c;
    if (VEC) {
      Io<T>::store8(o, v);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (c + i < cols) Io<T>::store1(o + i, v[i]);
    }
  }
}

// ---- blocks down the columns (and both at once) -----------------------------
// A workgroup takes 256 rows (one panel of x^T) x 128 columns: wave w the
// 32-row block w, a lane two neighbouring columns of it, so that a row of the
// tile is one coalesced access and a column block's 32 values sit in one
// lane.  Codes and scales of the 128 columns go through LDS, so that each
// column's 128-byte line leaves whole.
//
// BOTH: the wave's 32 x 128 values also pass through LDS of its own, sixteen
// rows at a time, from where a lane takes 32 neighbours of a row -- one row
// block -- and encodes them like a column's.  (Reducing the rows' maxima
// across lanes instead costs four times the vector instructions: 62 us for
// 8192 x 4096 BF16, against 19 us so, the time of the bytes.)
//
// BF16 stays packed: maxima by 16-bit integer pairs, codes straight from
// pairs.

constexpr int kTileCols = 128;

// Two neighbouring columns of a row, and a block's 32 values.
template <class T> struct Pair;
template <> struct Pair<float> {
  float a, b;
  static __device__ __forceinline__ Pair zero() { return {0.0f, 0.0f}; }
};
template <> struct Pair<uint16_t> {
  uint32_t w;
  static __device__ __forceinline__ Pair zero() { return {0u}; }
};

template <bool VEC>
__device__ __forceinline__ Pair<float> load_pair(const float* p, int n) {
  if constexpr (VEC) {
    const float2 v = *reinterpret_cast<const float2*>(p);
    return {v.x, v.y};
  } else {
    return {p[0], n > 1 ? p[1] : 0.0f};
  }
}
template <bool VEC>
__device__ __forceinline__ Pair<uint16_t> load_pair(const uint16_t* p, int n) {
  if constexpr (VEC) return {*reinterpret_cast<const uint32_t*>(p)};
  else return {(uint32_t)p[0] | (n > 1 ? (uint32_t)p[1] << 16 : 0u)};
}

// Both columns of a lane: codes (16 bytes) and scale byte of each.
__device__ __forceinline__ void encode_cols(const Pair<float> (&v)[32], uint4& c0, uint4& c1, uint32_t& b0, uint32_t& b1) {
  uint32_t a0 = 0, a1 = 0;
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    a0 = umax(a0, mag_bits(v[i].a));
    a1 = umax(a1, mag_bits(v[i].b));
  }
  b0 = scale_byte(a0);
  b1 = scale_byte(a1);
  uint32_t w0[4], w1[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    float e0[8], e1[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      e0[i] = v[8 * q + i].a;
      e1[i] = v[8 * q + i].b;
    }
    w0[q] = encode8(e0, b0);
    w1[q] = encode8(e1, b1);
  }
  c0 = make_uint4(w0[0], w0[1], w0[2], w0[3]);
  c1 = make_uint4(w1[0], w1[1], w1[2], w1[3]);
}
__device__ __forceinline__ void encode_cols(const Pair<uint16_t> (&v)[32], uint4& c0, uint4& c1, uint32_t& b0,
                                            uint32_t& b1) {
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < 32; ++i) a = max_u16x2(a, v[i].w & 0x7FFF7FFFu);
  b0 = scale_byte(a << 16);
  b1 = scale_byte(a & 0xFFFF0000u);
  uint32_t w0[4], w1[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint32_t e0[4], e1[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {        // rows 2 i and 2 i + 1 of either column
      const uint32_t lo = v[8 * q + 2 * i].w, hi = v[8 * q + 2 * i + 1].w;
      e0[i] = __builtin_amdgcn_perm(hi, lo, 0x05040100u);
      e1[i] = __builtin_amdgcn_perm(hi, lo, 0x07060302u);
    }
    w0[q] = encode8_bf16(e0, b0);
    w1[q] = encode8_bf16(e1, b1);
  }
  c0 = make_uint4(w0[0], w0[1], w0[2], w0[3]);
  c1 = make_uint4(w1[0], w1[1], w1[2], w1[3]);
}

// A row block of 32 neighbours in LDS.
__device__ __forceinline__ void encode_row(const float* p, uint4& c, uint32_t& byte) {
  float v[32];
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const float4 f = *reinterpret_cast<const float4*>(p + 4 * q);
    v[4 * q] = f.x; v[4 * q + 1] = f.y; v[4 * q + 2] = f.z; v[4 * q + 3] = f.w;
  }
  uint32_t a = 0;
#pragma unroll
  for (int i = 0; i < 32; ++i) a = umax(a, mag_bits(v[i]));
  byte = scale_byte(a);
  uint32_t w[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    float e[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) e[i] = v[8 * q + i];
    w[q] = encode8(e, byte);
  }
  c = make_uint4(w[0], w[1], w[2], w[3]);
}
__device__ __forceinline__ void encode_row(const uint16_t* p, uint4& c, uint32_t& byte) {
  uint32_t v[4][4];
  uint32_t a = 0;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const uint4 f = *reinterpret_cast<const uint4*>(p + 8 * q);
    v[q][0] = f.x; v[q][1] = f.y; v[q][2] = f.z; v[q][3] = f.w;
#pragma unroll
    for (int i = 0; i < 4; ++i) a = max_u16x2(a, v[q][i] & 0x7FFF7FFFu);
  }
  byte = scale_byte(umax(a << 16, a & 0xFFFF0000u));
  c = make_uint4(encode8_bf16(v[0], byte), encode8_bf16(v[1], byte), encode8_bf16(v[2], byte), encode8_bf16(v[3], byte));
}

// Orders a wave's own LDS writes before its reads of other lanes' values.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

template <class T, bool VEC, bool BOTH>
__global__ __launch_bounds__(512) void quant_cols_kernel(const T* __restrict__ x, int64_t rows, int64_t cols,
                                                         uint32_t tiles, uint8_t* __restrict__ codes_c,
                                                         uint8_t* __restrict__ scales_c,
                                                         uint8_t* __restrict__ codes_r,
                                                         uint8_t* __restrict__ scales_r) {
  constexpr int kPitch = kTileCols * (int)sizeof(T) + 16;      // spreads a lane quad's rows over the banks
  __shared__ __attribute__((aligned(16))) uint8_t lc[kTileCols * 128];
  __shared__ __attribute__((aligned(16))) uint8_t ls[kTileCols * 8];
  __shared__ __attribute__((aligned(16))) uint8_t lr[BOTH ? 8 * 16 * kPitch : 16];
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int64_t c0 = (int64_t)(blockIdx.x % tiles) * kTileCols, gr = blockIdx.x / tiles;
  const int64_t r0 = gr * kPanel + 32 * wave;
  const int64_t c = c0 + 2 * lane;
  Pair<T> v[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    v[i] = Pair<T>::zero();
    if (r0 + i < rows && c < cols) v[i] = load_pair<VEC>(x + (r0 + i) * cols + c, (int)(cols - c < 2 ? 1 : 2));
  }
  uint4 w0, w1;
  uint32_t b0, b1;
  encode_cols(v, w0, w1, b0, b1);
  // column j's line: chunk `wave` at position wave ^ (j / 2 % 8), so that the
  // 64 lanes' 16-byte writes spread over the banks
  const int pos = 16 * (wave ^ (lane & 7));
  *reinterpret_cast<uint4*>(lc + (2 * lane) * 128 + pos) = w0;
  *reinterpret_cast<uint4*>(lc + (2 * lane + 1) * 128 + pos) = w1;
  ls[(2 * lane) * 8 + wave] = (uint8_t)b0;
  ls[(2 * lane + 1) * 8 + wave] = (uint8_t)b1;
  if constexpr (BOTH) {
    uint8_t* buf = lr + wave * 16 * kPitch;
    const int64_t gc = c0 / kPanel;
    const int half = (int)(c0 / kTileCols) & 1;     // which half of the rows' panel
    const int r = lane >> 2, b = lane & 3;          // row of sixteen, block of four
#pragma unroll
    for (int k = 0; k < 2; ++k) {
#pragma unroll
      for (int i = 0; i < 16; ++i) *reinterpret_cast<Pair<T>*>(buf + i * kPitch + (int)sizeof(Pair<T>) * lane) = v[16 * k + i];
      wave_sync();
      uint4 w;
      uint32_t byte;
      encode_row(reinterpret_cast<const T*>(buf + r * kPitch) + 32 * b, w, byte);
      // the quad's four bytes in its first lane
      uint32_t quad = byte;
      quad |= (uint32_t)__builtin_amdgcn_mov_dpp((int)quad, 0xB1, 0xF, 0xF, true) << 8;    // lanes 0 and 2: own | next << 8
      quad = (quad & 0xFFFFu) | (uint32_t)__builtin_amdgcn_mov_dpp((int)quad, 0x4E, 0xF, 0xF, true) << 16;
      const int64_t row = r0 + 16 * k + r;
      if (row < rows) {
        *reinterpret_cast<uint4*>(codes_r + (gc * rows + row) * kPanelBytes + 64 * half + 16 * b) = w;
        if (b == 0) *reinterpret_cast<uint32_t*>(scales_r + (gc * rows + row) * kPanelScales + 4 * half) = quad;
      }
      wave_sync();
    }
  }
  __syncthreads();
  for (int k = t; k < kTileCols * 8; k += 512) {
    const int j = k >> 3, p = k & 7;                 // column, 16-byte position
    if (c0 + j < cols)
      *reinterpret_cast<uint4*>(codes_c + (gr * cols + c0 + j) * kPanelBytes + 16 * (p ^ ((j >> 1) & 7))) =
          *reinterpret_cast<const uint4*>(lc + j * 128 + 16 * p);
  }
  if (t < kTileCols && c0 + t < cols)
    *reinterpret_cast<uint2*>(scales_c + (gr * cols + c0 + t) * kPanelScales) =
        *reinterpret_cast<const uint2*>(ls + t * 8);
}

template <class T, bool VEC>
__global__ __launch_bounds__(512) void dequant_cols_kernel(const uint8_t* __restrict__ codes,
                                                           const uint8_t* __restrict__ scales, int64_t rows,
                                                           int64_t cols, uint32_t tiles, T* __restrict__ out) {
  __shared__ __attribute__((aligned(16))) uint8_t lc[kTileCols * 128];
  __shared__ __attribute__((aligned(16))) uint8_t ls[kTileCols * 8];
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int64_t c0 = (int64_t)(blockIdx.x % tiles) * kTileCols, gr = blockIdx.x / tiles;
  for (int k = t; k < kTileCols * 8; k += 512) {
    const int j = k >> 3, p = k & 7;
    if (c0 + j < cols)
      *reinterpret_cast<uint4*>(lc + j * 128 + 16 * p) = *reinterpret_cast<const uint4*>(
          codes + (gr * cols + c0 + j) * kPanelBytes + 16 * (p ^ ((j >> 1) & 7)));
  }
  if (t < kTileCols && c0 + t < cols)
    *reinterpret_cast<uint2*>(ls + t * 8) =
        *reinterpret_cast<const uint2*>(scales + (gr * cols + c0 + t) * kPanelScales);
  __syncthreads();
  const int64_t c = c0 + 2 * lane, r0 = gr * kPanel + 32 * wave;
  if (c >= cols) return;
  const int pos = 16 * (wave ^ (lane & 7));
  const uint4 w0 = *reinterpret_cast<const uint4*>(lc + (2 * lane) * 128 + pos);
  const uint4 w1 = *reinterpret_cast<const uint4*>(lc + (2 * lane + 1) * 128 + pos);
  const uint32_t b0 = ls[(2 * lane) * 8 + wave], b1 = ls[(2 * lane + 1) * 8 + wave];
  const uint32_t q0[4] = {w0.x, w0.y, w0.z, w0.w}, q1[4] = {w1.x, w1.y, w1.z, w1.w};
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    float e0[8], e1[8];
    decode8(q0[q], b0, e0);
    decode8(q1[q], b1, e1);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int64_t r = r0 + 8 * q + i;
      if (r < rows) {
        T* o = out + r * cols + c;
        if (VEC) {
          Io<T>::store2(o, e0[i], e1[i]);
        } else {
          Io<T>::store1(o, e0[i]);
          if (c + 1 < cols) Io<T>::store1(o + 1, e1[i]);
        }
      }
    }
  }
}

// BOTH writes row lines by halves: when an odd number of 128-column tiles
// covers the columns, the last panel's second half is all padding and no
// tile writes it, so one more (empty) tile is launched.
uint32_t col_tiles(int64_t cols, bool both) {
  const int64_t n = (cols + kTileCols - 1) / kTileCols;
  return (uint32_t)(both ? (n + 1) / 2 * 2 : n);
}
uint32_t panels_of(int64_t n) { return (uint32_t)((n + kPanel - 1) / kPanel); }
// Workgroups in one dimension (the API bounds the product below 2^31).
dim3 rows_grid(int64_t rows, uint32_t panels) {
  return dim3((unsigned)((rows + kRowsPerPass * kPasses - 1) / (kRowsPerPass * kPasses) * panels));
}

template <class T>
hipError_t quantize(const T* x, int64_t rows, int64_t cols, int ways, uint8_t* cr, uint8_t* sr, uint8_t* cc,
                    uint8_t* sc, hipStream_t s) {
  if (ways == kMxRows) {
    const uint32_t p = panels_of(cols);
    if (cols % 8 == 0)
      quant_rows_kernel<T, true><<<rows_grid(rows, p), 256, 0, s>>>(x, rows, cols, p, cr, sr);
    else
      quant_rows_kernel<T, false><<<rows_grid(rows, p), 256, 0, s>>>(x, rows, cols, p, cr, sr);
    return hipGetLastError();
  }
  const bool both = ways == (kMxRows | kMxCols);
  const uint32_t n = col_tiles(cols, both);
  const dim3 grid(n * panels_of(rows));
  if (cols % 2 == 0) {
    if (both)
      quant_cols_kernel<T, true, true><<<grid, 512, 0, s>>>(x, rows, cols, n, cc, sc, cr, sr);
    else
      quant_cols_kernel<T, true, false><<<grid, 512, 0, s>>>(x, rows, cols, n, cc, sc, nullptr, nullptr);
  } else {
    if (both)
      quant_cols_kernel<T, false, true><<<grid, 512, 0, s>>>(x, rows, cols, n, cc, sc, cr, sr);
    else
      quant_cols_kernel<T, false, false><<<grid, 512, 0, s>>>(x, rows, cols, n, cc, sc, nullptr, nullptr);
  }
  return hipGetLastError();
}

template <class T>
hipError_t dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, bool down, T* out,
                      hipStream_t s) {
  if (!down) {
    const uint32_t p = panels_of(cols);
    if (cols % 8 == 0)
      dequant_rows_kernel<T, true><<<rows_grid(rows, p), 256, 0, s>>>(codes, scales, rows, cols, p, out);
    else
      dequant_rows_kernel<T, false><<<rows_grid(rows, p), 256, 0, s>>>(codes, scales, rows, cols, p, out);
    return hipGetLastError();
  }
  const uint32_t n = col_tiles(cols, false);
  const dim3 grid(n * panels_of(rows));
  if (cols % 2 == 0)
    dequant_cols_kernel<T, true><<<grid, 512, 0, s>>>(codes, scales, rows, cols, n, out);
  else
    dequant_cols_kernel<T, false><<<grid, 512, 0, s>>>(codes, scales, rows, cols, n, out);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_mx_quantize(const void* x, Dt xt, int64_t rows, int64_t cols, int ways, uint8_t* codes_r,
                              uint8_t* scales_r, uint8_t* codes_c, uint8_t* scales_c, hipStream_t s) {
  return xt == Dt::F32 ? quantize(static_cast<const float*>(x), rows, cols, ways, codes_r, scales_r, codes_c, scales_c, s)
                       : quantize(static_cast<const uint16_t*>(x), rows, cols, ways, codes_r, scales_r, codes_c, scales_c, s);
}

hipError_t launch_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, bool down,
                                void* out, Dt ot, hipStream_t s) {
  return ot == Dt::F32 ? dequantize(codes, scales, rows, cols, down, static_cast<float*>(out), s)
                       : dequantize(codes, scales, rows, cols, down, static_cast<uint16_t*>(out), s);
}

}  // namespace nvfp4

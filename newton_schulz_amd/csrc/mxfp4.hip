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
  static __device__ __forceinline__ void load2(const float* p, float& a, float& b) {
    const float2 w = *reinterpret_cast<const float2*>(p);
    a = w.x; b = w.y;
  }
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
  static __device__ __forceinline__ void load2(const uint16_t* p, float& a, float& b) {
    const uint32_t w = *reinterpret_cast<const uint32_t*>(p);
    a = bf16_lo(w); b = bf16_hi(w);
  }
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
// 32-row block w, a lane two neighbouring columns of it, so a column block's
// 32 values sit in one lane's registers and a row of the tile is one
// coalesced access.  Codes and scales of the 128 columns go through LDS, so
// that each column's 128-byte line leaves whole.
//
// BOTH: the row blocks of the same tile (32 columns = 16 lanes) from the same
// registers: the maximum by DPP over the 16 lanes, one byte of codes a lane
// and row, gathered in LDS into 64-byte halves of the rows' lines.

constexpr int kTileCols = 128;

// Maximum over the 16 lanes of a DPP row, left in every lane (rotations by
// 8, 4, 2, 1).
__device__ __forceinline__ uint32_t row16_max(uint32_t a) {
  a = umax(a, (uint32_t)__builtin_amdgcn_mov_dpp((int)a, 0x128, 0xF, 0xF, true));
  a = umax(a, (uint32_t)__builtin_amdgcn_mov_dpp((int)a, 0x124, 0xF, 0xF, true));
  a = umax(a, (uint32_t)__builtin_amdgcn_mov_dpp((int)a, 0x122, 0xF, 0xF, true));
  return umax(a, (uint32_t)__builtin_amdgcn_mov_dpp((int)a, 0x121, 0xF, 0xF, true));
}

template <class T, bool VEC, bool BOTH>
__global__ __launch_bounds__(512) void quant_cols_kernel(const T* __restrict__ x, int64_t rows, int64_t cols,
                                                         uint32_t tiles,
                                                         uint8_t* __restrict__ codes_c,
                                                         uint8_t* __restrict__ scales_c,
                                                         uint8_t* __restrict__ codes_r,
                                                         uint8_t* __restrict__ scales_r) {
  __shared__ __attribute__((aligned(16))) uint8_t lc[kTileCols * 128];
  __shared__ __attribute__((aligned(16))) uint8_t ls[kTileCols * 8];
  __shared__ __attribute__((aligned(16))) uint8_t lr[BOTH ? 256 * 64 : 16];
  __shared__ __attribute__((aligned(16))) uint8_t lrs[BOTH ? 256 * 4 : 16];
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int64_t c0 = (int64_t)(blockIdx.x % tiles) * kTileCols, gr = blockIdx.x / tiles;
  const int64_t r0 = gr * kPanel + 32 * wave;
  const int64_t c = c0 + 2 * lane;
  float v0[32], v1[32];
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    v0[i] = v1[i] = 0.0f;
    if (r0 + i < rows) {
      const T* p = x + (r0 + i) * cols + c;
      if (VEC) {
        if (c < cols) Io<T>::load2(p, v0[i], v1[i]);
      } else {
        if (c < cols) v0[i] = Io<T>::load1(p);
        if (c + 1 < cols) v1[i] = Io<T>::load1(p + 1);
      }
    }
  }
  uint32_t a0 = 0, a1 = 0;
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    a0 = umax(a0, mag_bits(v0[i]));
    a1 = umax(a1, mag_bits(v1[i]));
  }
  const uint32_t b0 = scale_byte(a0), b1 = scale_byte(a1);
  uint32_t w0[4], w1[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    float e0[8], e1[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      e0[i] = v0[8 * q + i];
      e1[i] = v1[8 * q + i];
    }
    w0[q] = encode8(e0, b0);
    w1[q] = encode8(e1, b1);
  }
  // column j's line: chunk `wave` at position wave ^ (j / 2 % 8), so that the
  // 64 lanes' 16-byte writes spread over the banks
  const int pos = 16 * (wave ^ (lane & 7));
  *reinterpret_cast<uint4*>(lc + (2 * lane) * 128 + pos) = make_uint4(w0[0], w0[1], w0[2], w0[3]);
  *reinterpret_cast<uint4*>(lc + (2 * lane + 1) * 128 + pos) = make_uint4(w1[0], w1[1], w1[2], w1[3]);
  ls[(2 * lane) * 8 + wave] = (uint8_t)b0;
  ls[(2 * lane + 1) * 8 + wave] = (uint8_t)b1;
  if constexpr (BOTH) {
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const uint32_t b = scale_byte(row16_max(umax(mag_bits(v0[i]), mag_bits(v1[i]))));
      const uint32_t w = encode2<0>(0u, v0[i], v1[i], scale_value(b));
      lr[(32 * wave + i) * 64 + lane] = (uint8_t)(b == 255u ? 0u : w);
      if ((lane & 15) == 0) lrs[(32 * wave + i) * 4 + (lane >> 4)] = (uint8_t)b;
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
  if constexpr (BOTH) {
    const int64_t gc = c0 / kPanel;
    const int half = (int)(c0 / kTileCols) & 1;       // which half of the row's panel
    for (int k = t; k < 256 * 4; k += 512) {
      const int r = k >> 2, p = k & 3;
      const int64_t row = gr * kPanel + r;
      if (row < rows)
        *reinterpret_cast<uint4*>(codes_r + (gc * rows + row) * kPanelBytes + 64 * half + 16 * p) =
            *reinterpret_cast<const uint4*>(lr + r * 64 + 16 * p);
    }
    if (t < 256 && gr * kPanel + t < rows)
      *reinterpret_cast<uint32_t*>(scales_r + (gc * rows + gr * kPanel + t) * kPanelScales + 4 * half) =
          *reinterpret_cast<const uint32_t*>(lrs + t * 4);
  }
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

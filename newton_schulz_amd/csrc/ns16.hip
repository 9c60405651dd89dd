// Passes around the products of the 16-bit Newton–Schulz iteration: the
// source's norm (with the momentum update of a Muon step in the same pass),
// and X_0's f16 panels together with those of its transpose.
#include <type_traits>

#include "mxfp4_device.hpp"
#include "panel.hpp"

namespace nvfp4 {
namespace {
using namespace mx;

// Eight neighbouring elements, at any alignment; `n` < 8 at the end of a row
// or of the data.
template <Dt T>
__device__ __forceinline__ void load8(const void* p, int64_t at, int n, float (&v)[8]) {
  if constexpr (T == Dt::F32) {
    const float* f = static_cast<const float*>(p) + at;
    if (n == 8) {
      const float4u a = *reinterpret_cast<const float4u*>(f), b = *reinterpret_cast<const float4u*>(f + 4);
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
      const bf16x8u a = *reinterpret_cast<const bf16x8u*>(f);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = __uint_as_float((uint32_t)a[i] << 16);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = i < n ? __uint_as_float((uint32_t)f[i] << 16) : 0.0f;
    }
  }
}

// v as it reads back after it was stored as T, and the store itself.
template <Dt T>
__device__ __forceinline__ void store8(void* p, int64_t at, int n, float (&v)[8]) {
  if constexpr (T == Dt::F32) {
    float* f = static_cast<float*>(p) + at;
    if (n == 8) {
      *reinterpret_cast<float4*>(f) = make_float4(v[0], v[1], v[2], v[3]);
      *reinterpret_cast<float4*>(f + 4) = make_float4(v[4], v[5], v[6], v[7]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) f[i] = v[i];
    }
  } else {
    uint16_t* f = static_cast<uint16_t*>(p) + at;
    const uint32_t w[4] = {pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]), pack_bf16(v[4], v[5]), pack_bf16(v[6], v[7])};
    if (n == 8) {
      *reinterpret_cast<uint4*>(f) = make_uint4(w[0], w[1], w[2], w[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) f[i] = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = bf16_lo(w[i]);
      v[2 * i + 1] = bf16_hi(w[i]);
    }
  }
}

__device__ __forceinline__ float clamp_keep_nan(float v, float clip) {
  return v > clip ? clip : (v < -clip ? -clip : v);
}

// Sum of a workgroup's doubles, in a fixed order, left in every thread.
template <int THREADS>
__device__ __forceinline__ double block_sum(double v, double* lds) {
#pragma unroll
  for (int d = 32; d >= 1; d >>= 1) v += __shfl_down(v, d, 64);
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  v = lds[0];
#pragma unroll
  for (int w = 1; w < THREADS / 64; ++w) v += lds[w];
  return v;
}

// One workgroup a CU, bound by the reads: four 16-byte loads of G are in
// flight in each of a CU's 512 lanes (11008 x 4096 BF16: 61 us with one in
// each of 256, 25 us so).  The momentum form has three streams and one load
// of each (8 x 1024 x 4096, 335 MB: 67 us with 256 lanes, 56 us so).
constexpr int kNormThreads = 512;
template <Dt GT, Dt MT, bool MOM>
__global__ __launch_bounds__(kNormThreads) void norm_kernel(const Ns16Inputs in, int64_t count, float mu, int nesterov,
                                                            double* part, int64_t bstride) {
  constexpr int kAhead = MOM ? 1 : 4;
  constexpr int64_t kStep = (int64_t)kNs16Parts * kNormThreads * 8;
  __shared__ double lds[kNormThreads / 64];
  const int y = (int)blockIdx.y;
  const void* g = in.g[y];
  void* mom = in.mom[y];
  const float clip = in.clip[y];
  double sum = 0.0;
  int64_t at = ((int64_t)blockIdx.x * kNormThreads + threadIdx.x) * 8;
  auto one = [&](int64_t i0, int n, float (&v)[8]) {
    if constexpr (MOM) {
      float m[8];
      load8<MT>(mom, i0, n, m);
#pragma unroll
      for (int i = 0; i < 8; ++i) m[i] = fmaf(mu, m[i], v[i]);
      store8<MT>(mom, i0, n, m);
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = nesterov ? fmaf(mu, m[i], v[i]) : m[i];
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = clamp_keep_nan(v[i], clip);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) sum += (double)v[i] * (double)v[i];
  };
  for (; at + (kAhead - 1) * kStep + 8 <= count; at += kAhead * kStep) {
    float v[kAhead][8];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) load8<GT>(g, at + k * kStep, 8, v[k]);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int k = 0; k < kAhead; ++k) one(at + k * kStep, 8, v[k]);
  }
  for (; at < count; at += kStep) {
    const int n = count - at < 8 ? (int)(count - at) : 8;
    float v[8];
    load8<GT>(g, at, n, v);
    one(at, n, v);
  }
  sum = block_sum<kNormThreads>(sum, lds);
  if (threadIdx.x == 0)
    reinterpret_cast<double*>(reinterpret_cast<uint8_t*>(part) + (int64_t)y * bstride)[blockIdx.x] = sum;
}

// One 64 x 64 tile of the source a workgroup: lines along its rows go to
// `along` ([columns / 64][rows_p][64]), lines down its columns to `down`.
template <Dt GT, Dt MT, bool MOM>
__global__ __launch_bounds__(256) void start_kernel(const Ns16Inputs in, int64_t rows, int64_t cols, float mu,
                                                    int nesterov, const double* part, uint8_t* along, uint8_t* down,
                                                    int64_t rows_p, int64_t cols_p, float* fac, int64_t bstride) {
  __shared__ double lds[4];
  __shared__ _Float16 tile[64][66];
  const int y = (int)blockIdx.y, t = threadIdx.x;
  const int64_t off = (int64_t)y * bstride;
  const double* pp = reinterpret_cast<const double*>(reinterpret_cast<const uint8_t*>(part) + off);
  const double norm = sqrt(block_sum<256>(pp[t], lds)) + 1e-7;      // kNs16Parts == 256 threads
  const double s = (double)kNs16Scale / norm;
  const bool ok = isfinite(norm);
  const int e = ok ? ilogb(s) : 0;                             // 2^e <= s < 2^(e + 1)
  const uint32_t tc = (uint32_t)(cols_p / 64);
  const int64_t R = (int64_t)(blockIdx.x / tc) * 64, C = (int64_t)(blockIdx.x % tc) * 64;
  if (blockIdx.x == 0 && t == 0) {
    float* f = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(fac) + off);
    const float k = ok ? (float)ldexp(s, -e) : __uint_as_float(0x7FC00000u);
    f[0] = k;
    f[1] = k * k;
  }
  const void* g = in.g[y];
  const void* mom = in.mom[y];
  const float clip = in.clip[y];
  const int r = t >> 2, c = (t & 3) * 16;
  union { _Float16 h[16]; uint4 w[2]; } v;
  float x[2][8], m[2][8];
#pragma unroll
  for (int b = 0; b < 2; ++b) {
    const int64_t col = C + c + 8 * b, at = (R + r) * cols + col;
    const int n = R + r < rows && col < cols ? (cols - col < 8 ? (int)(cols - col) : 8) : 0;
    load8<GT>(g, at, n, x[b]);
    if constexpr (MOM) load8<MT>(mom, at, n, m[b]);
  }
#pragma unroll
  for (int b = 0; b < 2; ++b) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float u;
      if constexpr (MOM) u = nesterov ? fmaf(mu, m[b][i], x[b][i]) : m[b][i];
      else u = clamp_keep_nan(x[b][i], clip);
      v.h[8 * b + i] = (_Float16)ldexpf(u, e);
    }
  }
  uint8_t* a = along + off + ((C / 64) * rows_p + R + r) * 128 + c * 2;
  *reinterpret_cast<uint4*>(a) = v.w[0];
  *reinterpret_cast<uint4*>(a + 16) = v.w[1];
#pragma unroll
  for (int i = 0; i < 16; ++i) tile[r][c + i] = v.h[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 16; ++i) v.h[i] = tile[c + i][r];
  uint8_t* d = down + off + ((R / 64) * cols_p + C + r) * 128 + c * 2;
  *reinterpret_cast<uint4*>(d) = v.w[0];
  *reinterpret_cast<uint4*>(d + 16) = v.w[1];
}

template <class F>
hipError_t by_type(Dt gt, Dt mt, bool mom, F&& f) {
  if (!mom) {
    if (gt == Dt::F32) f(std::integral_constant<Dt, Dt::F32>{}, std::integral_constant<Dt, Dt::F32>{}, std::false_type{});
    else f(std::integral_constant<Dt, Dt::BF16>{}, std::integral_constant<Dt, Dt::F32>{}, std::false_type{});
  } else if (gt == Dt::F32) {
    if (mt == Dt::F32) f(std::integral_constant<Dt, Dt::F32>{}, std::integral_constant<Dt, Dt::F32>{}, std::true_type{});
    else f(std::integral_constant<Dt, Dt::F32>{}, std::integral_constant<Dt, Dt::BF16>{}, std::true_type{});
  } else {
    if (mt == Dt::F32) f(std::integral_constant<Dt, Dt::BF16>{}, std::integral_constant<Dt, Dt::F32>{}, std::true_type{});
    else f(std::integral_constant<Dt, Dt::BF16>{}, std::integral_constant<Dt, Dt::BF16>{}, std::true_type{});
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_ns16_norm(const Ns16Inputs& in, int batch, Dt gt, Dt mt, int64_t count, float mu, int nesterov,
                            double* part, int64_t bstride, hipStream_t s) {
  const dim3 grid(kNs16Parts, (unsigned)batch);
  return by_type(gt, mt, in.mom[0] != nullptr, [&](auto G, auto M, auto mom) {
    norm_kernel<decltype(G)::value, decltype(M)::value, decltype(mom)::value>
        <<<grid, kNormThreads, 0, s>>>(in, count, mu, nesterov, part, bstride);
  });
}

hipError_t launch_ns16_start(const Ns16Inputs& in, int batch, Dt gt, Dt mt, int64_t rows, int64_t cols, bool tr,
                             float mu, int nesterov, const double* part, uint8_t* X, uint8_t* XT, int64_t mp,
                             int64_t np, float* fac, int64_t bstride, hipStream_t s) {
  const int64_t rows_p = tr ? np : mp, cols_p = tr ? mp : np;
  const dim3 grid((unsigned)(rows_p / 64 * (cols_p / 64)), (unsigned)batch);
  return by_type(gt, mt, in.mom[0] != nullptr, [&](auto G, auto M, auto mom) {
    start_kernel<decltype(G)::value, decltype(M)::value, decltype(mom)::value><<<grid, 256, 0, s>>>(
        in, rows, cols, mu, nesterov, part, tr ? XT : X, tr ? X : XT, rows_p, cols_p, fac, bstride);
  });
}

}  // namespace nvfp4

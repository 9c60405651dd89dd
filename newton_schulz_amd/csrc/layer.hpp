// What runs between two 4-bit linear layers: the root-mean-square norm with
// the residual's addition and dropout (norm.hip), MXFP8 and its products with
// MXFP4 (mxfp8.hip, mxfp8_gemm.hip), and products with NVFP4 weights
// (nvfp4_linear.hip).  Every launcher only enqueues on `s` and returns
// hipGetLastError().
#pragma once
#include "launch.hpp"

namespace nvfp4 {

// ---- dropout ------------------------------------------------------------------
// rng: device, seed and offset; null: no dropout.  Element kept where its 16
// random bits are at least `cut`, and then multiplied by `scale`.
struct Drop {
  const uint64_t* rng;
  uint32_t cut;
  float scale;
};
hipError_t launch_dropout(const void* x, Dt t, int64_t rows, int64_t cols, const Drop& d, void* out, hipStream_t s);

// ---- norm ---------------------------------------------------------------------
// Row width: what a workgroup of 1024 keeps in registers.
constexpr int64_t kNormMaxCols = 32768;
struct NormForward {
  const void* x;            // [T][C]
  const void* residual;     // [T][C] of ht, or null
  const void* w;            // [C]
  void* h;                  // [T][C], or null: x itself is normed
  void* y;                  // [T][C], or null
  uint8_t *codes8, *scales8, *codes4, *scales4;   // operands along the rows, or null
  float* rstd;              // [T], or null
  int64_t T;
  int C;
  double eps;
  Dt xt, ht, wt, yt;
  Drop drop;
};
hipError_t launch_norm(const NormForward& n, hipStream_t s);
// The normed rows in MXFP4 blocked along the tokens (operand of C rows): from
// h and rstd as launch_norm wrote them.
hipError_t launch_norm_cols(const void* h, Dt ht, const float* rstd, const void* w, Dt wt, int64_t T, int64_t C,
                            uint8_t* codes, uint8_t* scales, hipStream_t s);

struct NormBackward {
  const void* dy;           // [T][C]
  const void* h;            // [T][C] of ht
  const float* rstd;        // [T]
  const void* w;            // [C]
  const void* dh_in;        // [T][C] of ht, or null
  void* dh;                 // [T][C] of ht
  void* dx;                 // [T][C] of xt, or null
  float* dw;                // [C], or null
  float beta;               // dw = beta dw + ...
  float* partials;          // norm_partials(T, C) * C floats, with dw
  int64_t T;
  int C;
  Dt dyt, ht, wt, xt;
  Drop drop;
};
int64_t norm_partials(int64_t T, int64_t C);      // rows of partial sums
hipError_t launch_norm_backward(const NormBackward& n, hipStream_t s);

// ---- MXFP8 --------------------------------------------------------------------
hipError_t launch_mx8_quantize(const void* x, Dt xt, int64_t rows, int64_t cols, uint8_t* codes, uint8_t* scales,
                               hipStream_t s);
hipError_t launch_mx8_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, void* out,
                                 Dt ot, hipStream_t s);

// out [M][N] = beta addend + alpha P Q^T, P in MXFP8 and Q in MXFP4, both
// blocked along K.  addend null: none.
struct Product8 {
  const uint8_t *p, *p_scales, *q, *q_scales;
  int64_t M, N, K;
  float alpha, beta;
  const float* addend;
  void* out;
  Dt ot;
};
size_t mx8_workspace(int64_t M, int64_t N, int64_t K);
hipError_t launch_mx8_product(const Product8& g, void* ws, hipStream_t s);

// ---- NVFP4 weights --------------------------------------------------------------
// y [T][N] = x [T][K] W^T, W [N][K] in NVFP4 blocked along its rows.
hipError_t launch_nv_linear(const void* x, Dt xt, int64_t T, int64_t K, const uint8_t* codes, const uint8_t* scales,
                            const float* sg, int64_t N, void* y, Dt yt, hipStream_t s);

}  // namespace nvfp4

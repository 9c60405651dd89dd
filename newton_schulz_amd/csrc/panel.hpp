// Products of panel operands (panel.hip) and the passes around them that the
// 16-bit Newton–Schulz iteration needs (ns16.hip).  Every launcher only
// enqueues on `s` and returns hipGetLastError().
#pragma once
#include "launch.hpp"

namespace nvfp4 {

// A panel operand: rows x K cut along K into panels of 128 bytes a row --
// 256 E2M1 codes or 64 f16 values -- stored [panel][rows][128]; MXFP4 scales
// [panel][rows][8].  What lies behind a row's end in the last panel is zero.
struct PanelOperand {
  const uint8_t* data;
  const uint8_t* scales;   // E8M0, MXFP4 only
  int64_t rows;            // rows in each panel
};

// What becomes of acc = P Q^T.
enum class PanelEp : int {
  Out,    // out = beta addend + alpha acc, row-major FP32 or BF16
  Gram,   // f16 panels of alpha acc, both triangles of a symmetric product
  Poly,   // f16 panels of a I + b A + c acc, likewise (A symmetric, f16 panels)
  Iter,   // f16 panels of alpha acc and of its transpose
  Step,   // w = decay w - alpha acc, row-major FP32 or BF16, in place
};

struct PanelProblem {
  PanelOperand p, q;
  int64_t M = 0, N = 0;             // rows of out / columns of out
  int64_t panels = 0;
  bool sym = false;                 // P and Q are the same tensor
  PanelEp ep = PanelEp::Out;
  float alpha = 1.0f, beta = 0.0f;
  const float* dalpha = nullptr;    // device factor on alpha (may be null)
  const float* addend = nullptr;    // [M][N] FP32 (Out), may be out itself
  void* out = nullptr;              // Out, Step: [M][N]; Gram, Poly, Iter: panels of M rows
  void* out_t = nullptr;            // Iter: panels of N rows
  Dt ot = Dt::F32;
  const uint8_t* a = nullptr;       // Poly: A, panels of M rows
  float ca = 0, cb = 0, cc = 0;     // Poly
  // What f16 takes from the diagonals, which carry most of A's and B's norm,
  // is put back in FP32: Gram writes d = A_ii - f16(A_ii) to dout; Poly takes
  // it as din -- A^2 is A~^2 + (d_i + d_j) A~_ij to first order -- and writes
  // B_ii / f16(B_ii) to dout (1 where f16 holds B_ii as a subnormal number);
  // Iter, Out and Step multiply their rows by din (columns when din_cols),
  // which is B's diagonal put right as long as that dominates its rows.  Halves
  // the error of five steps where singular values are of one size (a 92 x 868
  // gradient: 2.0e-3 -> 1.05e-3).  Arrays of M rounded up to 256 rows; null:
  // none.
  const float* din = nullptr;
  float* dout = nullptr;
  bool din_cols = false;
  // Iter, Out and Step with `da` given: the left operand (the right one when
  // din_cols) is a I + b A + c A^2 with the coefficients above, made from A's
  // panels `a` and da = its d, and din's factors come from it; p (or q) is not
  // read.  Only with a plan_panel_poly plan.
  const float* da = nullptr;
  // `batch` problems, each with its pointers moved by `bstride` bytes; the
  // row-major outputs may be given one by one, with their own alpha
  int batch = 1;
  int64_t bstride = 0;
  void* const* out_each = nullptr;      // host, `batch` entries
  const float* alpha_each = nullptr;    // host, `batch` entries (factors on alpha)
};
constexpr int kMaxPanelBatch = 32;

struct PanelPlan {
  int tile;                // rows and columns of a tile: 256, 128, 64 or 32
  int parts;               // K-parts of each tile left over after equal rounds (1: none)
  int TM, TN, tiles;       // of one problem
  int slots;               // workgroups per XCD
  int split_tiles, groups; // of the whole batch
  size_t ws_bytes;         // FP32 partials of the whole batch
};
// poly: for the Poly epilogue, which has no 256 x 256 tiles: A's values next to
// the 128 accumulators of a lane spill there (4 x 2048^2: 73 us,
// 50 us on 128).
PanelPlan plan_panel(int64_t M, int64_t N, int64_t panels, bool sym, int batch, bool allow_split, bool poly);
// Whether the products with B (mp x mp, times mp x np) make it on the way:
// while A fits LDS and one round of workgroups does it, a launch less per step
// is worth more than B computed once.  Five steps (us, there / B by itself):
// 50 x 512: 47 / 65, 128 x 1000: 55 / 69, 256 x 512: 61 / 68, four of
// 256 x 2048: 112 / 124; the worst are 256 x 4096: 114 / 111 and sixteen of
// 192 x 300: 94 / 87.  In two rounds: 256 x 16384 218 / 202, four of 256 x 4096
// 182 / 160.
constexpr int kPolyPanels = 4;
bool poly_in_product(int64_t mp, int64_t np, int batch);
PanelPlan plan_panel_poly(int64_t M, int64_t N, int batch);
hipError_t launch_panel(const PanelProblem& g, const PanelPlan& p, bool fp4, void* ws, hipStream_t s);

// ---- MXFP4 quantizers (mxfp4.hip) -------------------------------------------
constexpr int kMxRows = 1, kMxCols = 2;
hipError_t launch_mx_quantize(const void* x, Dt xt, int64_t rows, int64_t cols, int ways, uint8_t* codes_r,
                              uint8_t* scales_r, uint8_t* codes_c, uint8_t* scales_c, hipStream_t s);
hipError_t launch_mx_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, bool down,
                                void* out, Dt ot, hipStream_t s);

// ---- MXFP4 products with few rows (mxfp4_few.hip) -------------------------------
// Whether a product of T rows goes there: one launch that reads w once, against
// a pass over x and a tiled product that reuses w.  Measured (us, x in BF16,
// there / tiled) on the GPU: 11008 x 4096 weights, T = 1: 6.1 / 9.4, 8: 8.9 / 9.4,
// 16: 12.0 / 9.8, 32: 22 / 11; 4096 x 4096, T = 16: 6.1 / 6.6, 32: 8.4 / 7.5; launched
// one by one from Python 11 / 16, which decides up to 16.
constexpr int64_t kMxFewRows = 32;
inline bool mx_few(int64_t T, int64_t N, int64_t K) {
  return T <= 16 || (T <= kMxFewRows && N * K <= (int64_t)1 << 24);
}
// out[T][N] = beta addend + alpha x w^T; x [T][K] FP32 or BF16, quantized along
// K, or codes with x_scales (then xt is not used).  addend null: none.
hipError_t launch_mx_few(const void* x, Dt xt, const uint8_t* x_scales, int64_t T, int64_t K, const uint8_t* w,
                         const uint8_t* w_scales, int64_t N, float alpha, float beta, const float* addend, void* out,
                         Dt ot, hipStream_t s);

// ---- 16-bit Newton–Schulz prologue (ns16.hip) --------------------------------
constexpr int kNs16Parts = 256;     // partial sums of squares per matrix
struct Ns16Inputs {                 // host pointer tables of one batch, by value
  const void* g[kMaxPanelBatch];
  void* mom[kMaxPanelBatch];        // Muon: momentum, updated in place (null: none)
  float clip[kMaxPanelBatch];
};
// Sums of squares of the iterate's source u -- clamp(G), or with momentum
// M <- mu M + g and u = g + mu M (nesterov) or M, M as stored -- into `part`
// [batch][kNs16Parts] doubles at stride `bstride`.
hipError_t launch_ns16_norm(const Ns16Inputs& in, int batch, Dt gt, Dt mt, int64_t count, float mu, int nesterov,
                            double* part, int64_t bstride, hipStream_t s);
// X_0's f16 panels and those of its transpose, zero-padded to mp x np:
// 2^e u with 2^e the power of two that brings the norm to (kNs16Scale / 2,
// kNs16Scale], so that BF16 sources are not rounded; t = kNs16Scale /
// (2^e (|u| + eps)) goes to fac[0] and t^2 to fac[1].  Sources are rows x cols row-major,
// transposed when `tr` (then X is cols x rows).
constexpr float kNs16Scale = 256.0f;
hipError_t launch_ns16_start(const Ns16Inputs& in, int batch, Dt gt, Dt mt, int64_t rows, int64_t cols, bool tr,
                             float mu, int nesterov, const double* part, uint8_t* X, uint8_t* XT, int64_t mp,
                             int64_t np, float* fac, int64_t bstride, hipStream_t s);

}  // namespace nvfp4

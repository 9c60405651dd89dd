// C ABI of the MXFP4 operators and of the 16-bit Newton–Schulz operators
// (declared in include/nvfp4ns.h): argument validation, workspace planning
// and launch sequences.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "api_common.hpp"
#include "mxfp4_device.hpp"
#include "panel.hpp"

using nvfp4::Dt;
using nvfp4::PanelEp;
using nvfp4::PanelOperand;
using nvfp4::PanelPlan;
using nvfp4::PanelProblem;

namespace {

// Offsets inside a panel are 32-bit and row numbers int.
constexpr int64_t kMaxDim = (int64_t)1 << 24;
inline bool mx_dim(int64_t a) { return a > 0 && a <= kMaxDim; }
// Elements of one matrix: keeps every launch's thread count below 2^32.
constexpr int64_t kMaxCount = (int64_t)1 << 36;
inline bool mx_dims(int64_t rows, int64_t cols) { return mx_dim(rows) && mx_dim(cols) && rows * cols <= kMaxCount; }
inline bool mx_dims(int64_t M, int64_t N, int64_t K) { return mx_dims(M, N) && mx_dims(M, K) && mx_dims(N, K); }
inline bool axis_ok(int a) { return a == NVFP4_ROWS || a == NVFP4_COLS; }
inline int64_t mx_panels(int64_t n) { return (n + nvfp4::mx::kPanel - 1) / nvfp4::mx::kPanel; }
// Bytes of an operand of `rows` rows blocked along `cols`.
inline size_t mx_codes(int64_t rows, int64_t cols) { return (size_t)rows * mx_panels(cols) * nvfp4::mx::kPanelBytes; }
inline size_t mx_scales(int64_t rows, int64_t cols) { return (size_t)rows * mx_panels(cols) * nvfp4::mx::kPanelScales; }
inline PanelOperand mx_operand(const uint8_t* codes, const uint8_t* scales, int64_t rows) {
  return PanelOperand{codes, scales, rows};
}

PanelProblem mx_product(const uint8_t* pc, const uint8_t* ps, const uint8_t* qc, const uint8_t* qs, int64_t M,
                        int64_t N, int64_t K, float alpha, float beta, const float* addend, void* out, Dt ot) {
  PanelProblem g;
  g.p = mx_operand(pc, ps, M);
  g.q = mx_operand(qc, qs, N);
  g.M = M;
  g.N = N;
  g.panels = mx_panels(K);
  g.alpha = alpha;
  g.beta = beta;
  g.addend = beta != 0.0f ? addend : nullptr;
  g.out = out;
  g.ot = ot;
  return g;
}

inline PanelPlan mx_plan(int64_t M, int64_t N, int64_t K, bool split) {
  if (nvfp4::mx_few(M, N, K)) return PanelPlan{};      // launch_mx_few: no plan, no workspace
  return nvfp4::plan_panel(M, N, mx_panels(K), false, 1, split, false);
}

// One product of operands in MXFP4, whichever way its rows call for.
hipError_t mx_multiply(const uint8_t* pc, const uint8_t* ps, const uint8_t* qc, const uint8_t* qs, int64_t M, int64_t N,
                       int64_t K, float alpha, float beta, const float* addend, void* out, Dt ot, void* ws,
                       hipStream_t s) {
  if (nvfp4::mx_few(M, N, K))
    return nvfp4::launch_mx_few(pc, Dt::F32, ps, M, K, qc, qs, N, alpha, beta, beta != 0.0f ? addend : nullptr, out, ot, s);
  return nvfp4::launch_panel(mx_product(pc, ps, qc, qs, M, N, K, alpha, beta, addend, out, ot),
                             mx_plan(M, N, K, ws != nullptr), true, ws, s);
}

}  // namespace

extern "C" {

size_t mxfp4_codes_bytes(int64_t rows, int64_t cols, nvfp4_axis axis) {
  if (!mx_dims(rows, cols) || !axis_ok(axis)) return 0;
  return axis == NVFP4_ROWS ? mx_codes(rows, cols) : mx_codes(cols, rows);
}

size_t mxfp4_scales_bytes(int64_t rows, int64_t cols, nvfp4_axis axis) {
  if (!mx_dims(rows, cols) || !axis_ok(axis)) return 0;
  return axis == NVFP4_ROWS ? mx_scales(rows, cols) : mx_scales(cols, rows);
}

ns_status mxfp4_quantize(const void* x, ns_dtype xt, int64_t rows, int64_t cols, nvfp4_axis axis, uint8_t* codes,
                         uint8_t* scales, void* stream) {
  if (!x || !codes || !scales || !dtype_ok(xt) || !axis_ok(axis)) return NS_ERR_ARG;
  if (!mx_dims(rows, cols)) return NS_ERR_SHAPE;
  if (!al(x, 16) || !al(codes, 16) || !al(scales, 16)) return NS_ERR_ARG;
  const Span X{x, (size_t)(rows * cols) * dtype_size(xt)}, C{codes, mxfp4_codes_bytes(rows, cols, axis)},
      S{scales, mxfp4_scales_bytes(rows, cols, axis)};
  if (hits(C, {X, S}) || hits(S, {X})) return NS_ERR_ARG;
  const bool r = axis == NVFP4_ROWS;
  NS_TRY(nvfp4::launch_mx_quantize(x, (Dt)xt, rows, cols, r ? nvfp4::kMxRows : nvfp4::kMxCols, r ? codes : nullptr,
                                   r ? scales : nullptr, r ? nullptr : codes, r ? nullptr : scales,
                                   as_stream(stream)));
  return NS_OK;
}

ns_status mxfp4_quantize_both(const void* x, ns_dtype xt, int64_t rows, int64_t cols, uint8_t* codes_rows,
                              uint8_t* scales_rows, uint8_t* codes_cols, uint8_t* scales_cols, void* stream) {
  if (!x || !codes_rows || !scales_rows || !codes_cols || !scales_cols || !dtype_ok(xt)) return NS_ERR_ARG;
  if (!mx_dims(rows, cols)) return NS_ERR_SHAPE;
  if (!al(x, 16) || !al(codes_rows, 16) || !al(scales_rows, 16) || !al(codes_cols, 16) || !al(scales_cols, 16))
    return NS_ERR_ARG;
  const Span X{x, (size_t)(rows * cols) * dtype_size(xt)}, C{codes_rows, mx_codes(rows, cols)},
      S{scales_rows, mx_scales(rows, cols)}, D{codes_cols, mx_codes(cols, rows)}, T{scales_cols, mx_scales(cols, rows)};
  if (hits(C, {X, S, D, T}) || hits(S, {X, D, T}) || hits(D, {X, T}) || hits(T, {X})) return NS_ERR_ARG;
  NS_TRY(nvfp4::launch_mx_quantize(x, (Dt)xt, rows, cols, nvfp4::kMxRows | nvfp4::kMxCols, codes_rows, scales_rows,
                                   codes_cols, scales_cols, as_stream(stream)));
  return NS_OK;
}

ns_status mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, nvfp4_axis axis,
                           void* out, ns_dtype ot, void* stream) {
  if (!codes || !scales || !out || !dtype_ok(ot) || !axis_ok(axis)) return NS_ERR_ARG;
  if (!mx_dims(rows, cols)) return NS_ERR_SHAPE;
  if (!al(codes, 16) || !al(scales, 16) || !al(out, 16)) return NS_ERR_ARG;
  const Span O{out, (size_t)(rows * cols) * dtype_size(ot)};
  if (hits(O, {Span{codes, mxfp4_codes_bytes(rows, cols, axis)}, Span{scales, mxfp4_scales_bytes(rows, cols, axis)}}))
    return NS_ERR_ARG;
  NS_TRY(nvfp4::launch_mx_dequantize(codes, scales, rows, cols, axis == NVFP4_COLS, out, (Dt)ot, as_stream(stream)));
  return NS_OK;
}

size_t mxfp4_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  if (!mx_dims(M, N, K)) return 0;
  return mx_plan(M, N, K, true).ws_bytes;
}

ns_status mxfp4_gemm(const uint8_t* codes_p, const uint8_t* scales_p, const uint8_t* codes_q, const uint8_t* scales_q,
                     int64_t M, int64_t N, int64_t K, float alpha, float beta, const float* addend, void* out,
                     ns_dtype ot, void* ws, size_t ws_bytes, void* stream) {
  if (!codes_p || !scales_p || !codes_q || !scales_q || !out || !dtype_ok(ot)) return NS_ERR_ARG;
  if (!std::isfinite(alpha) || !std::isfinite(beta) || (beta != 0.0f && !addend)) return NS_ERR_ARG;
  if (!mx_dims(M, N, K)) return NS_ERR_SHAPE;
  const PanelPlan plan = mx_plan(M, N, K, ws != nullptr);
  if (ws && ws_bytes < plan.ws_bytes) return NS_ERR_WORKSPACE;
  if (!al(codes_p, 16) || !al(scales_p, 16) || !al(codes_q, 16) || !al(scales_q, 16) || !al(out, 16) ||
      !al(addend, 16) || !al(ws, 16))
    return NS_ERR_ARG;
  const size_t mn = (size_t)(M * N);
  const bool in_place = beta != 0.0f && static_cast<const void*>(addend) == out && ot == NS_F32;
  const Span O{out, mn * dtype_size(ot)}, P{codes_p, mx_codes(M, K)}, PS{scales_p, mx_scales(M, K)},
      Q{codes_q, mx_codes(N, K)}, QS{scales_q, mx_scales(N, K)},
      A{beta != 0.0f && !in_place ? addend : nullptr, mn * sizeof(float)}, W{ws, ws ? ws_bytes : 0};
  if (hits(O, {P, PS, Q, QS, A, W}) || hits(W, {P, PS, Q, QS, A})) return NS_ERR_ARG;
  NS_TRY(mx_multiply(codes_p, scales_p, codes_q, scales_q, M, N, K, alpha, beta, addend, out, (Dt)ot, ws,
                     as_stream(stream)));
  return NS_OK;
}

// ---- linear layer --------------------------------------------------------------

}  // extern "C" (reopened below)

namespace {

// Workspace of the linear layer's calls: the quantized operands they make,
// then the products' partials (the products run one after another).
struct LinearLayout {
  size_t c0, s0, c1, s1, part, total;
};
LinearLayout forward_layout(int64_t T, int64_t N, int64_t K) {
  LinearLayout L{};
  if (nvfp4::mx_few(T, N, K)) return L;    // quantized in the product's registers
  size_t o = 0;
  auto take = [&](size_t b) { const size_t at = o; o = align_up(o + b); return at; };
  L.c0 = take(mx_codes(T, K));
  L.s0 = take(mx_scales(T, K));
  L.part = take(mx_plan(T, N, K, true).ws_bytes);
  L.total = o;
  return L;
}
LinearLayout backward_layout(int64_t T, int64_t N, int64_t K) {
  LinearLayout L{};
  size_t o = 0;
  auto take = [&](size_t b) { const size_t at = o; o = align_up(o + b); return at; };
  L.c0 = take(mx_codes(T, N));     // dy along N
  L.s0 = take(mx_scales(T, N));
  L.c1 = take(mx_codes(N, T));     // dy^T along the tokens
  L.s1 = take(mx_scales(N, T));
  const size_t a = mx_plan(T, K, N, true).ws_bytes, b = mx_plan(N, K, T, true).ws_bytes;
  L.part = take(a > b ? a : b);
  L.total = o;
  return L;
}

}  // namespace

extern "C" {

size_t mxfp4_linear_workspace_bytes(int64_t T, int64_t N, int64_t K) {
  if (!mx_dims(T, N, K)) return 0;
  return forward_layout(T, N, K).total;
}

ns_status mxfp4_linear(const void* x, ns_dtype xt, int64_t T, int64_t K, const uint8_t* w_codes,
                       const uint8_t* w_scales, int64_t N, void* y, ns_dtype yt, uint8_t* kept_codes,
                       uint8_t* kept_scales, void* ws, size_t ws_bytes, void* stream) {
  if (!x || !w_codes || !w_scales || !y || !dtype_ok(xt) || !dtype_ok(yt)) return NS_ERR_ARG;
  if ((kept_codes == nullptr) != (kept_scales == nullptr)) return NS_ERR_ARG;
  if (!mx_dims(T, N, K)) return NS_ERR_SHAPE;
  const LinearLayout L = forward_layout(T, N, K);
  if (ws_bytes < L.total || (L.total && !ws)) return NS_ERR_WORKSPACE;
  if (!al(x, 16) || !al(w_codes, 16) || !al(w_scales, 16) || !al(y, 16) || !al(kept_codes, 16) ||
      !al(kept_scales, 16) || !al(ws, 16))
    return NS_ERR_ARG;
  const Span X{x, (size_t)(T * K) * dtype_size(xt)}, W{w_codes, mx_codes(N, K)}, WS{w_scales, mx_scales(N, K)},
      Y{y, (size_t)(T * N) * dtype_size(yt)}, C{kept_codes, mx_codes(K, T)}, S{kept_scales, mx_scales(K, T)},
      Z{ws, ws ? ws_bytes : 0};
  if (hits(Y, {X, W, WS, C, S, Z}) || hits(C, {X, W, WS, S, Z}) || hits(S, {X, W, WS, Z}) || hits(Z, {X, W, WS}))
    return NS_ERR_ARG;
  hipStream_t s = as_stream(stream);
  uint8_t* b = static_cast<uint8_t*>(ws);
  if (nvfp4::mx_few(T, N, K)) {
    if (kept_codes)
      NS_TRY(nvfp4::launch_mx_quantize(x, (Dt)xt, T, K, nvfp4::kMxCols, nullptr, nullptr, kept_codes, kept_scales, s));
    NS_TRY(nvfp4::launch_mx_few(x, (Dt)xt, nullptr, T, K, w_codes, w_scales, N, 1.0f, 0.0f, nullptr, y, (Dt)yt, s));
    return NS_OK;
  }
  NS_TRY(nvfp4::launch_mx_quantize(x, (Dt)xt, T, K, kept_codes ? nvfp4::kMxRows | nvfp4::kMxCols : nvfp4::kMxRows,
                                   b + L.c0, b + L.s0, kept_codes, kept_scales, s));
  NS_TRY(mx_multiply(b + L.c0, b + L.s0, w_codes, w_scales, T, N, K, 1.0f, 0.0f, nullptr, y, (Dt)yt, b + L.part, s));
  return NS_OK;
}

size_t mxfp4_linear_backward_workspace_bytes(int64_t T, int64_t N, int64_t K) {
  if (!mx_dims(T, N, K)) return 0;
  return backward_layout(T, N, K).total;
}

ns_status mxfp4_linear_backward(const void* dy, ns_dtype dyt, int64_t T, int64_t N, int64_t K,
                                const uint8_t* wt_codes, const uint8_t* wt_scales, const uint8_t* kept_codes,
                                const uint8_t* kept_scales, void* dx, ns_dtype dxt, void* dw, ns_dtype dwt,
                                float beta, void* ws, size_t ws_bytes, void* stream) {
  if (!dy || !dtype_ok(dyt) || !dtype_ok(dxt) || !dtype_ok(dwt) || (!dx && !dw)) return NS_ERR_ARG;
  if (dx && (!wt_codes || !wt_scales)) return NS_ERR_ARG;
  if (dw && (!kept_codes || !kept_scales)) return NS_ERR_ARG;
  if (!std::isfinite(beta) || (beta != 0.0f && (!dw || dwt != NS_F32))) return NS_ERR_ARG;
  if (!mx_dims(T, N, K)) return NS_ERR_SHAPE;
  const LinearLayout L = backward_layout(T, N, K);
  if (!ws || ws_bytes < L.total) return NS_ERR_WORKSPACE;
  if (!al(dy, 16) || !al(wt_codes, 16) || !al(wt_scales, 16) || !al(kept_codes, 16) || !al(kept_scales, 16) ||
      !al(dx, 16) || !al(dw, 16) || !al(ws, 16))
    return NS_ERR_ARG;
  const Span Y{dy, (size_t)(T * N) * dtype_size(dyt)}, W{dx ? wt_codes : nullptr, mx_codes(K, N)},
      WS{dx ? wt_scales : nullptr, mx_scales(K, N)}, C{dw ? kept_codes : nullptr, mx_codes(K, T)},
      S{dw ? kept_scales : nullptr, mx_scales(K, T)}, X{dx, (size_t)(T * K) * dtype_size(dxt)},
      D{dw, (size_t)(N * K) * dtype_size(dwt)}, Z{ws, ws_bytes};
  if (hits(X, {Y, W, WS, C, S, D, Z}) || hits(D, {Y, W, WS, C, S, Z}) || hits(Z, {Y, W, WS, C, S}))
    return NS_ERR_ARG;
  hipStream_t s = as_stream(stream);
  uint8_t* b = static_cast<uint8_t*>(ws);
  NS_TRY(nvfp4::launch_mx_quantize(dy, (Dt)dyt, T, N, (dx ? nvfp4::kMxRows : 0) | (dw ? nvfp4::kMxCols : 0), b + L.c0,
                                   b + L.s0, b + L.c1, b + L.s1, s));
  if (dx)
    NS_TRY(mx_multiply(b + L.c0, b + L.s0, wt_codes, wt_scales, T, K, N, 1.0f, 0.0f, nullptr, dx, (Dt)dxt, b + L.part, s));
  if (dw)
    NS_TRY(mx_multiply(b + L.c1, b + L.s1, kept_codes, kept_scales, N, K, T, 1.0f, beta, static_cast<const float*>(dw), dw,
                       (Dt)dwt, b + L.part, s));
  return NS_OK;
}

}  // extern "C" (reopened below)

// ---- 16-bit Newton–Schulz --------------------------------------------------------

namespace {

constexpr int64_t kMaxElems16 = (int64_t)1 << 31;

// Workspace of one matrix: the iterate X [mp][np] (mp <= np, both padded to
// whole panels of 64) as f16 panels, its transpose twice (the update reads
// one while it writes the other), A and B, partials and scalars.
struct Ns16Layout {
  int64_t mp, np;
  size_t x, xt[2], a, b, da, rb, part, fac, total;   // of one matrix
  size_t split;                              // the batch's split tiles' partials, behind its matrices
  bool fused;                                // B made by the products that use it
  PanelPlan gram, poly, iter, last;
};

Ns16Layout ns16_layout(int64_t m, int64_t n, int batch) {
  Ns16Layout L;
  const int64_t xm = m < n ? m : n, xn = m < n ? n : m;
  L.mp = (xm + 63) / 64 * 64;
  L.np = (xn + 63) / 64 * 64;
  L.gram = nvfp4::plan_panel(L.mp, L.mp, L.np / 64, true, batch, true, false);
  L.poly = nvfp4::plan_panel(L.mp, L.mp, L.mp / 64, true, batch, true, true);
  L.iter = nvfp4::plan_panel(L.mp, L.np, L.mp / 64, false, batch, true, false);
  L.last = nvfp4::plan_panel(m, n, L.mp / 64, false, batch, true, false);
  L.fused = nvfp4::poly_in_product(L.mp, L.np, batch);
  if (L.fused) {
    L.iter = nvfp4::plan_panel_poly(L.mp, L.np, batch);
    L.last = nvfp4::plan_panel_poly(m, n, batch);
  }
  size_t part = 0;
  for (const PanelPlan* p : {&L.gram, &L.poly, &L.iter, &L.last}) part = p->ws_bytes > part ? p->ws_bytes : part;
  size_t o = 0;
  auto take = [&](size_t bytes) { const size_t at = o; o = align_up(o + bytes); return at; };
  L.x = take((size_t)(L.mp * L.np) * 2);
  L.xt[0] = take((size_t)(L.mp * L.np) * 2);
  L.xt[1] = take((size_t)(L.mp * L.np) * 2);
  L.a = take((size_t)(L.mp * L.mp) * 2);
  L.b = take((size_t)(L.mp * L.mp) * 2);
  // per row: what f16 takes from A's diagonal, and B's over its rounding (read
  // by whole tiles, so up to 255 rows further than they are written)
  L.da = take((size_t)(L.mp + 256) * sizeof(float));
  L.rb = take((size_t)(L.mp + 256) * sizeof(float));
  L.part = take(nvfp4::kNs16Parts * sizeof(double));
  L.fac = take(2 * sizeof(float));
  L.total = o;
  L.split = align_up(part);
  return L;
}

// What a batch of matrices of one shape is given besides its sources.
struct Ns16Call {
  Dt gt, mt, ot;
  const float* coeffs;
  int k;
  float mu = 0.0f, decay = 0.0f, lr = 0.0f;
  int nesterov = 0;
  bool step = false;              // outputs are weights to update
};

// `batch` matrices m x n: X_0, then per step A = X X^T, B = a I + b A + c A^2,
// X <- B X; the last update goes to the outputs.  X is held times kNs16Scale.
// The first step works on X_0 / t (see launch_ns16_start): its A takes t^2
// and its update t.
hipError_t ns16_batch(const nvfp4::Ns16Inputs& in, void* const* out, const float* alpha_each, int batch, int64_t m,
                      int64_t n, const Ns16Call& c, uint8_t* ws, hipStream_t s) {
  const Ns16Layout L = ns16_layout(m, n, batch);
  const bool tr = m > n;
  const int64_t stride = (int64_t)L.total;
  uint8_t *X = ws + L.x, *A = ws + L.a, *B = ws + L.b;
  double* part = reinterpret_cast<double*>(ws + L.part);
  float* fac = reinterpret_cast<float*>(ws + L.fac);
  float *da = reinterpret_cast<float*>(ws + L.da), *rb = reinterpret_cast<float*>(ws + L.rb);
  hipError_t e = nvfp4::launch_ns16_norm(in, batch, c.gt, c.mt, m * n, c.mu, c.nesterov, part, stride, s);
  if (e != hipSuccess) return e;
  e = nvfp4::launch_ns16_start(in, batch, c.gt, c.mt, m, n, tr, c.mu, c.nesterov, part, X, ws + L.xt[0], L.mp, L.np,
                               fac, stride, s);
  if (e != hipSuccess) return e;
  const PanelOperand ox{X, nullptr, L.mp}, oa{A, nullptr, L.mp}, ob{B, nullptr, L.mp};
  for (int it = 0; it < c.k; ++it) {
    uint8_t *XT = ws + L.xt[it & 1], *XN = ws + L.xt[1 - (it & 1)];
    const PanelOperand oxt{XT, nullptr, L.np};
    PanelProblem g;
    g.batch = batch;
    g.bstride = stride;
    g.p = g.q = ox;
    g.M = g.N = L.mp;
    g.panels = L.np / 64;
    g.sym = true;
    g.ep = PanelEp::Gram;
    g.alpha = 1.0f / (nvfp4::kNs16Scale * nvfp4::kNs16Scale);
    g.dalpha = it == 0 ? fac + 1 : nullptr;
    g.out = A;
    g.dout = da;
    e = nvfp4::launch_panel(g, L.gram, false, ws + (size_t)batch * L.total, s);
    if (e != hipSuccess) return e;
    g.p = g.q = oa;
    g.panels = L.mp / 64;
    g.ep = PanelEp::Poly;
    g.alpha = 1.0f;
    g.dalpha = nullptr;
    g.a = A;
    g.ca = c.coeffs[3 * it];
    g.cb = c.coeffs[3 * it + 1];
    g.cc = c.coeffs[3 * it + 2];
    g.out = B;
    g.din = da;
    g.dout = rb;
    if (!L.fused) {
      e = nvfp4::launch_panel(g, L.poly, false, ws + (size_t)batch * L.total, s);
      if (e != hipSuccess) return e;
    }
    PanelProblem u;
    u.batch = batch;
    u.bstride = stride;
    u.panels = L.mp / 64;
    u.dalpha = it == 0 ? fac : nullptr;
    u.din = rb;
    if (L.fused) {
      u.da = da;
      u.a = A;
      u.ca = g.ca;
      u.cb = g.cb;
      u.cc = g.cc;
    }
    if (it + 1 < c.k) {
      u.p = ob;
      u.q = oxt;
      u.M = L.mp;
      u.N = L.np;
      u.ep = PanelEp::Iter;
      u.out = X;
      u.out_t = XN;
      e = nvfp4::launch_panel(u, L.iter, false, ws + (size_t)batch * L.total, s);
    } else {
      // rows of the output are rows of X, or of its transpose when m > n
      u.p = tr ? oxt : ob;
      u.q = tr ? ob : oxt;
      u.din_cols = tr;
      u.M = m;
      u.N = n;
      u.ep = c.step ? PanelEp::Step : PanelEp::Out;
      u.alpha = (c.step ? c.lr : 1.0f) / nvfp4::kNs16Scale;
      u.beta = c.step ? c.decay : 0.0f;
      u.ot = c.ot;
      u.out_each = out;
      u.alpha_each = alpha_each;
      e = nvfp4::launch_panel(u, L.last, false, ws + (size_t)batch * L.total, s);
    }
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// A batch of a group: matrices of one shape, in call order.  Matrix j is taken
// with the first matrix of its shape, kMaxPanelBatch at a time.
struct Ns16Batch {
  int count, index[nvfp4::kMaxPanelBatch];
};
bool same_shape(const int64_t* m, const int64_t* n, int i, int j) { return m[i] == m[j] && n[i] == n[j]; }

template <class F>
ns_status for_batches(int count, const int64_t* m, const int64_t* n, F&& f) {
  for (int i = 0; i < count; ++i) {
    bool seen = false;
    for (int j = 0; j < i && !seen; ++j) seen = same_shape(m, n, i, j);
    if (seen) continue;
    Ns16Batch b{0, {}};
    for (int j = i; j < count; ++j) {
      if (!same_shape(m, n, i, j)) continue;
      b.index[b.count++] = j;
      if (b.count == nvfp4::kMaxPanelBatch) {
        const ns_status st = f(b);
        if (st != NS_OK) return st;
        b.count = 0;
      }
    }
    if (b.count) {
      const ns_status st = f(b);
      if (st != NS_OK) return st;
    }
  }
  return NS_OK;
}

ns_status ns16_shapes(int count, const int64_t* m, const int64_t* n) {
  for (int i = 0; i < count; ++i)
    if (!mx_dim(m[i]) || !mx_dim(n[i]) || m[i] * n[i] >= kMaxElems16) return NS_ERR_SHAPE;
  return NS_OK;
}

ns_status coeffs_ok(const float* coeffs, int k) {
  if (!coeffs || k <= 0) return NS_ERR_ARG;
  for (int i = 0; i < 3 * k; ++i)
    if (!std::isfinite(coeffs[i])) return NS_ERR_ARG;
  return NS_OK;
}

// One array of each matrix of a group.
struct Arrays {
  const void* const* p;
  ns_dtype t;
  bool written;
};
// Whether no array that is written shares a byte with another, and none with
// the workspace: the ranges in order of their starts, each against the
// furthest end before it (of all ranges if it is written itself, else of the
// written ones).  NS_ERR_ARG if some do.
ns_status group_clear(int count, const int64_t* m, const int64_t* n, std::initializer_list<Arrays> arrays, Span ws) {
  struct Range {
    uintptr_t from, to;
    bool written;
  };
  constexpr size_t kStack = 64;
  const size_t total = arrays.size() * (size_t)count + 1;
  Range few[kStack];
  Range* r = few;
  if (total > kStack) {
    r = static_cast<Range*>(std::malloc(total * sizeof(Range)));
    if (!r) return NS_ERR_ARG;
  }
  size_t k = 0;
  auto add = [&](const void* p, size_t bytes, bool written) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    r[k++] = Range{at, at + bytes, written};
  };
  add(ws.p, ws.n, true);
  for (const Arrays& a : arrays)
    for (int i = 0; i < count; ++i) add(a.p[i], (size_t)(m[i] * n[i]) * dtype_size(a.t), a.written);
  std::sort(r, r + k, [](const Range& x, const Range& y) { return x.from < y.from; });
  uintptr_t all = 0, written = 0;
  bool clear = true;
  for (size_t i = 0; i < k && clear; ++i) {
    clear = r[i].from >= (r[i].written ? all : written);
    all = r[i].to > all ? r[i].to : all;
    if (r[i].written) written = r[i].to > written ? r[i].to : written;
  }
  if (r != few) std::free(r);
  return clear ? NS_OK : NS_ERR_ARG;
}

}  // namespace

extern "C" {

size_t ns_f16_workspace_bytes(int count, const int64_t* m, const int64_t* n) {
  if (count <= 0 || !m || !n || ns16_shapes(count, m, n) != NS_OK) return 0;
  size_t most = 0;
  (void)for_batches(count, m, n, [&](const Ns16Batch& b) {
    const Ns16Layout L = ns16_layout(m[b.index[0]], n[b.index[0]], b.count);
    const size_t need = (size_t)b.count * L.total + L.split;
    most = need > most ? need : most;
    return NS_OK;
  });
  return most;
}

ns_status ns_orthogonalize_f16_grouped(int count, const void* const* G, const int64_t* m, const int64_t* n,
                                       ns_dtype gt, const float* coeffs, int k, const float* clip, void* const* out,
                                       ns_dtype ot, void* ws, size_t ws_bytes, void* stream) {
  if (count <= 0 || !G || !m || !n || !out || !dtype_ok(gt) || !dtype_ok(ot)) return NS_ERR_ARG;
  if (coeffs_ok(coeffs, k) != NS_OK) return NS_ERR_ARG;
  for (int i = 0; i < count; ++i) {
    if (!G[i] || !out[i]) return NS_ERR_ARG;
    if (clip && !(clip[i] > 0.0f)) return NS_ERR_ARG;
  }
  ns_status st = ns16_shapes(count, m, n);
  if (st != NS_OK) return st;
  if (!ws || ws_bytes < ns_f16_workspace_bytes(count, m, n)) return NS_ERR_WORKSPACE;
  if (!al(ws, 16)) return NS_ERR_ARG;
  for (int i = 0; i < count; ++i)
    if (!al(G[i], 16) || !al(out[i], 16)) return NS_ERR_ARG;
  st = group_clear(count, m, n, {{G, gt, false}, {out, ot, true}}, Span{ws, ws_bytes});
  if (st != NS_OK) return st;
  Ns16Call c{};
  c.gt = (Dt)gt;
  c.mt = Dt::F32;
  c.ot = (Dt)ot;
  c.coeffs = coeffs;
  c.k = k;
  return for_batches(count, m, n, [&](const Ns16Batch& b) {
    nvfp4::Ns16Inputs in{};
    void* o[nvfp4::kMaxPanelBatch];
    for (int i = 0; i < b.count; ++i) {
      in.g[i] = G[b.index[i]];
      in.clip[i] = clip ? clip[b.index[i]] : INFINITY;
      o[i] = out[b.index[i]];
    }
    NS_TRY(ns16_batch(in, o, nullptr, b.count, m[b.index[0]], n[b.index[0]], c, static_cast<uint8_t*>(ws),
                      as_stream(stream)));
    return NS_OK;
  });
}

ns_status ns_orthogonalize_f16(const void* G, ns_dtype gt, int64_t m, int64_t n, const float* coeffs, int k, float clip,
                               void* out, ns_dtype ot, void* ws, size_t ws_bytes, void* stream) {
  return ns_orthogonalize_f16_grouped(1, &G, &m, &n, gt, coeffs, k, &clip, &out, ot, ws, ws_bytes, stream);
}

ns_status ns_muon_step(int count, void* const* W, ns_dtype wt, void* const* M, ns_dtype mt, const void* const* G,
                       ns_dtype gt, const int64_t* m, const int64_t* n, const float* coeffs, int k,
                       const ns_muon_options* opt, const float* scale, void* ws, size_t ws_bytes, void* stream) {
  if (count <= 0 || !W || !M || !G || !m || !n || !opt || !dtype_ok(wt) || !dtype_ok(mt) || !dtype_ok(gt))
    return NS_ERR_ARG;
  if (coeffs_ok(coeffs, k) != NS_OK) return NS_ERR_ARG;
  if (!std::isfinite(opt->lr) || !std::isfinite(opt->momentum) || !std::isfinite(opt->weight_decay)) return NS_ERR_ARG;
  for (int i = 0; i < count; ++i)
    if (!W[i] || !M[i] || !G[i] || (scale && !std::isfinite(scale[i]))) return NS_ERR_ARG;
  ns_status st = ns16_shapes(count, m, n);
  if (st != NS_OK) return st;
  if (!ws || ws_bytes < ns_f16_workspace_bytes(count, m, n)) return NS_ERR_WORKSPACE;
  if (!al(ws, 16)) return NS_ERR_ARG;
  for (int i = 0; i < count; ++i)
    if (!al(W[i], 16) || !al(M[i], 16) || !al(G[i], 16)) return NS_ERR_ARG;
  st = group_clear(count, m, n, {{W, wt, true}, {M, mt, true}, {G, gt, false}}, Span{ws, ws_bytes});
  if (st != NS_OK) return st;
  Ns16Call c{};
  c.gt = (Dt)gt;
  c.mt = (Dt)mt;
  c.ot = (Dt)wt;
  c.coeffs = coeffs;
  c.k = k;
  c.mu = opt->momentum;
  c.nesterov = opt->nesterov != 0;
  c.lr = opt->lr;
  c.decay = (float)(1.0 - (double)opt->lr * (double)opt->weight_decay);
  c.step = true;
  return for_batches(count, m, n, [&](const Ns16Batch& b) {
    nvfp4::Ns16Inputs in{};
    void* o[nvfp4::kMaxPanelBatch];
    float sc[nvfp4::kMaxPanelBatch];
    for (int i = 0; i < b.count; ++i) {
      in.g[i] = G[b.index[i]];
      in.mom[i] = M[b.index[i]];
      o[i] = W[b.index[i]];
      sc[i] = scale ? scale[b.index[i]] : 1.0f;
    }
    NS_TRY(ns16_batch(in, o, sc, b.count, m[b.index[0]], n[b.index[0]], c, static_cast<uint8_t*>(ws),
                      as_stream(stream)));
    return NS_OK;
  });
}

}  // extern "C"

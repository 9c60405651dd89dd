// C ABI of the operators between 4-bit linear layers (declared in
// include/nvfp4ns.h): argument validation and launch sequences.
#include <hip/hip_runtime.h>

#include "api_common.hpp"
#include "layer.hpp"
#include "mx8_device.hpp"

using nvfp4::Drop;
using nvfp4::Dt;

namespace {

constexpr int64_t kMaxDim = (int64_t)1 << 24, kMaxCount = (int64_t)1 << 36;
// A launch has fewer than 2^32 threads.  The norm's have a workgroup of up to 1024
// for a row.  The NVFP4 product's are workgroups of 512 (1024 where there are up
// to 256 of them): ceil(N / 8) for one or two tokens, 2^30 threads at most, else at
// most ceil(N / 16) ceil(T / 16) <= T N / 256 + N / 16 + T / 16 + 1, with T and N up to
// 2^24 and T N up to 2^30 no more than 2^22 + 2^21 + 1.
constexpr int64_t kMaxWideRows = (int64_t)1 << 22, kMaxNvOutputs = (int64_t)1 << 30;
// 2^-254: up to there r of a row without values is finite in FP32, and y zero.
constexpr double kMinEps = 0x1p-254;
inline bool dim_ok(int64_t a) { return a > 0 && a <= kMaxDim; }
inline bool dims_ok(int64_t r, int64_t c) { return dim_ok(r) && dim_ok(c) && r * c <= kMaxCount; }
inline int64_t panels(int64_t n) { return (n + nvfp4::mx::kPanel - 1) / nvfp4::mx::kPanel; }
inline size_t codes4(int64_t rows, int64_t cols) { return (size_t)(rows * panels(cols)) * nvfp4::mx::kPanelBytes; }
inline size_t codes8(int64_t rows, int64_t cols) { return (size_t)(rows * panels(cols)) * nvfp4::mx::kPanelBytes8; }
inline size_t block_scales(int64_t rows, int64_t cols) { return (size_t)(rows * panels(cols)) * nvfp4::mx::kPanelScales; }

// Dropout's probability as the generator's 16 bits have it: kept where they
// are at least `cut`.  False for a probability that keeps nothing or none.
bool drop_of(double p, const void* rng, Drop& d) {
  d = Drop{nullptr, 0, 1.0f};
  if (!(p >= 0.0) || p >= 1.0) return false;
  const uint32_t cut = (uint32_t)std::floor(p * 65536.0 + 0.5);
  if (cut >= 65536u) return false;
  if (p == 0.0) return true;
  if (!rng || !al(rng, 8)) return false;
  d.rng = static_cast<const uint64_t*>(rng);
  d.cut = cut;
  d.scale = (float)(65536.0 / (65536.0 - cut));
  return true;
}

}  // namespace

extern "C" {

// ---- dropout ------------------------------------------------------------------

ns_status mx_dropout(const void* x, ns_dtype xt, int64_t rows, int64_t cols, double p, const void* rng, void* out,
                     void* stream) {
  Drop d;
  if (!x || !out || !dtype_ok(xt) || !rng || !al(rng, 8) || !drop_of(p, rng, d)) return NS_ERR_ARG;
  if (!dims_ok(rows, cols)) return NS_ERR_SHAPE;
  if (!al(x, 16) || !al(out, 16)) return NS_ERR_ARG;
  const size_t n = (size_t)(rows * cols) * dtype_size(xt);
  if ((x != out && hits(Span{out, n}, {Span{x, n}})) || hits(Span{out, n}, {Span{rng, 16}})) return NS_ERR_ARG;
  if (!d.rng) {                       // p = 0 keeps everything as it is
    d.rng = static_cast<const uint64_t*>(rng);
  }
  NS_TRY(nvfp4::launch_dropout(x, (Dt)xt, rows, cols, d, out, as_stream(stream)));
  return NS_OK;
}

// ---- norm ---------------------------------------------------------------------

ns_status mx_rms_norm(const mx_norm_args* a, void* stream) {
  Drop d;
  if (!a || !a->x || !a->weight || !dtype_ok(a->xt) || !dtype_ok(a->ht) || !dtype_ok(a->wt) || !dtype_ok(a->yt))
    return NS_ERR_ARG;
  if (!std::isfinite(a->eps) || !(a->eps >= kMinEps) || !drop_of(a->drop, a->rng, d)) return NS_ERR_ARG;
  const bool own_h = a->residual || d.rng;             // h is not x itself
  if (own_h ? !a->h : a->h != nullptr || a->ht != a->xt) return NS_ERR_ARG;
  if ((a->codes8 == nullptr) != (a->scales8 == nullptr) || (a->codes4 == nullptr) != (a->scales4 == nullptr) ||
      (a->kept_codes == nullptr) != (a->kept_scales == nullptr))
    return NS_ERR_ARG;
  if (!a->h && !a->y && !a->codes8 && !a->codes4 && !a->kept_codes && !a->rstd) return NS_ERR_ARG;
  if (a->kept_codes && !a->rstd) return NS_ERR_ARG;
  const int64_t T = a->T, C = a->C;
  if (!dims_ok(T, C) || C > nvfp4::kNormMaxCols || (C > 1024 && T >= kMaxWideRows)) return NS_ERR_SHAPE;
  for (const void* p : {a->x, a->residual, a->weight, (const void*)a->h, (const void*)a->y, (const void*)a->codes8,
                        (const void*)a->scales8, (const void*)a->codes4, (const void*)a->scales4,
                        (const void*)a->kept_codes, (const void*)a->kept_scales, (const void*)a->rstd})
    if (!al(p, 16)) return NS_ERR_ARG;
  const size_t n = (size_t)(T * C), nh = n * dtype_size(a->ht);
  // h may take the residual's place
  const Span X{a->x, n * dtype_size(a->xt)}, R{a->residual == a->h ? nullptr : a->residual, nh},
      W{a->weight, (size_t)C * dtype_size(a->wt)}, G{d.rng, 16}, H{a->h, nh}, Y{a->y, n * dtype_size(a->yt)},
      C8{a->codes8, codes8(T, C)}, S8{a->scales8, block_scales(T, C)}, C4{a->codes4, codes4(T, C)},
      S4{a->scales4, block_scales(T, C)}, KC{a->kept_codes, codes4(C, T)}, KS{a->kept_scales, block_scales(C, T)},
      RS{a->rstd, (size_t)T * sizeof(float)};
  if (hits(H, {X, R, W, G, Y, C8, S8, C4, S4, KC, KS, RS}) || hits(Y, {X, R, W, G, C8, S8, C4, S4, KC, KS, RS}) ||
      hits(C8, {X, R, W, G, S8, C4, S4, KC, KS, RS}) || hits(S8, {X, R, W, G, C4, S4, KC, KS, RS}) ||
      hits(C4, {X, R, W, G, S4, KC, KS, RS}) || hits(S4, {X, R, W, G, KC, KS, RS}) || hits(KC, {X, R, W, G, KS, RS}) ||
      hits(KS, {X, R, W, G, RS}) || hits(RS, {X, R, W, G}))
    return NS_ERR_ARG;
  nvfp4::NormForward f{a->x, a->residual, a->weight, a->h, a->y, a->codes8, a->scales8, a->codes4, a->scales4, a->rstd,
                       T, (int)C, a->eps, (Dt)a->xt, (Dt)a->ht, (Dt)a->wt, (Dt)a->yt, d};
  hipStream_t s = as_stream(stream);
  NS_TRY(nvfp4::launch_norm(f, s));
  if (a->kept_codes)
    NS_TRY(nvfp4::launch_norm_cols(a->h ? a->h : a->x, (Dt)a->ht, a->rstd, a->weight, (Dt)a->wt, T, C, a->kept_codes,
                                   a->kept_scales, s));
  return NS_OK;
}

size_t mx_rms_norm_backward_workspace_bytes(int64_t T, int64_t C) {
  if (!dims_ok(T, C) || C > nvfp4::kNormMaxCols) return 0;
  return (size_t)(nvfp4::norm_partials(T, C) * C) * sizeof(float);
}

ns_status mx_rms_norm_backward(const mx_norm_backward_args* a, void* ws, size_t ws_bytes, void* stream) {
  Drop d;
  if (!a || !a->dy || !a->h || !a->rstd || !a->weight || !a->dh || !dtype_ok(a->dyt) || !dtype_ok(a->ht) ||
      !dtype_ok(a->wt) || !dtype_ok(a->xt))
    return NS_ERR_ARG;
  if (!std::isfinite(a->beta) || !drop_of(a->drop, a->rng, d)) return NS_ERR_ARG;
  const int64_t T = a->T, C = a->C;
  if (!dims_ok(T, C) || C > nvfp4::kNormMaxCols) return NS_ERR_SHAPE;
  const size_t need = a->dweight ? mx_rms_norm_backward_workspace_bytes(T, C) : 0;
  if (need && (!ws || ws_bytes < need)) return NS_ERR_WORKSPACE;
  for (const void* p : {a->dy, a->h, (const void*)a->rstd, a->weight, a->dh_in, (const void*)a->dh, (const void*)a->dx,
                        (const void*)a->dweight, (const void*)ws})
    if (!al(p, 16)) return NS_ERR_ARG;
  const size_t n = (size_t)(T * C), nh = n * dtype_size(a->ht);
  // dh may take dh_in's place
  const Span DY{a->dy, n * dtype_size(a->dyt)}, H{a->h, nh}, RS{a->rstd, (size_t)T * sizeof(float)},
      W{a->weight, (size_t)C * dtype_size(a->wt)}, DI{a->dh_in == a->dh ? nullptr : a->dh_in, nh}, G{d.rng, 16}, DH{a->dh, nh},
      DX{a->dx, n * dtype_size(a->xt)}, DW{a->dweight, (size_t)C * sizeof(float)}, Z{need ? ws : nullptr, ws_bytes};
  if (hits(DH, {DY, H, RS, W, DI, G, DX, DW, Z}) || hits(DX, {DY, H, RS, W, DI, G, DW, Z}) ||
      hits(DW, {DY, H, RS, W, DI, G, Z}) || hits(Z, {DY, H, RS, W, DI, G}))
    return NS_ERR_ARG;
  const nvfp4::NormBackward b{a->dy, a->h, a->rstd, a->weight, a->dh_in, a->dh, a->dx, a->dweight, a->beta,
                              static_cast<float*>(ws), T, (int)C, (Dt)a->dyt, (Dt)a->ht, (Dt)a->wt, (Dt)a->xt, d};
  NS_TRY(nvfp4::launch_norm_backward(b, as_stream(stream)));
  return NS_OK;
}

// ---- MXFP8 --------------------------------------------------------------------

size_t mxfp8_codes_bytes(int64_t rows, int64_t cols) { return dims_ok(rows, cols) ? codes8(rows, cols) : 0; }
size_t mxfp8_scales_bytes(int64_t rows, int64_t cols) { return dims_ok(rows, cols) ? block_scales(rows, cols) : 0; }

ns_status mxfp8_quantize(const void* x, ns_dtype xt, int64_t rows, int64_t cols, uint8_t* codes, uint8_t* scales,
                         void* stream) {
  if (!x || !codes || !scales || !dtype_ok(xt)) return NS_ERR_ARG;
  if (!dims_ok(rows, cols)) return NS_ERR_SHAPE;
  if (!al(x, 16) || !al(codes, 16) || !al(scales, 16)) return NS_ERR_ARG;
  const Span X{x, (size_t)(rows * cols) * dtype_size(xt)}, C{codes, codes8(rows, cols)}, S{scales, block_scales(rows, cols)};
  if (hits(C, {X, S}) || hits(S, {X})) return NS_ERR_ARG;
  NS_TRY(nvfp4::launch_mx8_quantize(x, (Dt)xt, rows, cols, codes, scales, as_stream(stream)));
  return NS_OK;
}

ns_status mxfp8_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t cols, void* out,
                           ns_dtype ot, void* stream) {
  if (!codes || !scales || !out || !dtype_ok(ot)) return NS_ERR_ARG;
  if (!dims_ok(rows, cols)) return NS_ERR_SHAPE;
  if (!al(codes, 16) || !al(scales, 16) || !al(out, 16)) return NS_ERR_ARG;
  const Span O{out, (size_t)(rows * cols) * dtype_size(ot)};
  if (hits(O, {Span{codes, codes8(rows, cols)}, Span{scales, block_scales(rows, cols)}})) return NS_ERR_ARG;
  NS_TRY(nvfp4::launch_mx8_dequantize(codes, scales, rows, cols, out, (Dt)ot, as_stream(stream)));
  return NS_OK;
}

size_t mxfp8_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K) {
  if (!dims_ok(M, N) || !dims_ok(M, K) || !dims_ok(N, K)) return 0;
  return nvfp4::mx8_workspace(M, N, K);
}

ns_status mxfp8_gemm(const uint8_t* codes_p, const uint8_t* scales_p, const uint8_t* codes_q, const uint8_t* scales_q,
                     int64_t M, int64_t N, int64_t K, float alpha, float beta, const float* addend, void* out,
                     ns_dtype ot, void* ws, size_t ws_bytes, void* stream) {
  if (!codes_p || !scales_p || !codes_q || !scales_q || !out || !dtype_ok(ot)) return NS_ERR_ARG;
  if (!std::isfinite(alpha) || !std::isfinite(beta) || (beta != 0.0f && !addend)) return NS_ERR_ARG;
  if (!dims_ok(M, N) || !dims_ok(M, K) || !dims_ok(N, K)) return NS_ERR_SHAPE;
  if (ws && ws_bytes < nvfp4::mx8_workspace(M, N, K)) return NS_ERR_WORKSPACE;
  if (beta == 0.0f) addend = nullptr;
  if (!al(codes_p, 16) || !al(scales_p, 16) || !al(codes_q, 16) || !al(scales_q, 16) || !al(out, 16) ||
      !al(addend, 16) || !al(ws, 16))
    return NS_ERR_ARG;
  const size_t mn = (size_t)(M * N);
  const bool in_place = static_cast<const void*>(addend) == out && ot == NS_F32;
  const Span O{out, mn * dtype_size(ot)}, P{codes_p, codes8(M, K)}, PS{scales_p, block_scales(M, K)},
      Q{codes_q, codes4(N, K)}, QS{scales_q, block_scales(N, K)}, A{in_place ? nullptr : addend, mn * sizeof(float)},
      W{ws, ws ? ws_bytes : 0};
  if (hits(O, {P, PS, Q, QS, A, W}) || hits(W, {P, PS, Q, QS, A})) return NS_ERR_ARG;
  const nvfp4::Product8 g{codes_p, scales_p, codes_q, scales_q, M, N, K, alpha, beta, addend, out, (Dt)ot};
  NS_TRY(nvfp4::launch_mx8_product(g, ws, as_stream(stream)));
  return NS_OK;
}

// ---- NVFP4 weights --------------------------------------------------------------

ns_status nvfp4_linear(const void* x, ns_dtype xt, int64_t T, int64_t K, const uint8_t* w_codes,
                       const uint8_t* w_scales, const float* w_global_scale, int64_t N, void* y, ns_dtype yt,
                       void* stream) {
  if (!x || !w_codes || !w_scales || !w_global_scale || !y || !dtype_ok(xt) || !dtype_ok(yt)) return NS_ERR_ARG;
  if (!dims_ok(T, N) || !dims_ok(T, K) || !dims_ok(N, K) || K % 16 != 0 || T * N > kMaxNvOutputs) return NS_ERR_SHAPE;
  if (!al(x, 16) || !al(w_codes, 16) || !al(w_scales, 16) || !al(w_global_scale, 4) || !al(y, 16)) return NS_ERR_ARG;
  const Span Y{y, (size_t)(T * N) * dtype_size(yt)};
  if (hits(Y, {Span{x, (size_t)(T * K) * dtype_size(xt)}, Span{w_codes, (size_t)(N * K) / 2},
               Span{w_scales, (size_t)(N * K) / 16}, Span{w_global_scale, 4}}))
    return NS_ERR_ARG;
  NS_TRY(nvfp4::launch_nv_linear(x, (Dt)xt, T, K, w_codes, w_scales, w_global_scale, N, y, (Dt)yt, as_stream(stream)));
  return NS_OK;
}

}  // extern "C"

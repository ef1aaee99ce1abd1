// C ABI of the sparse FP8 row-wise linear layer: argument validation and
// dispatch to the gfx950 kernels.  The contract of every entry point is
// documented in include/sparse_fp8_row.h.
#include "sparse_fp8_row.h"

#include "sfr_launch.hpp"

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool fp8_ok(int dt) { return dt == SFR_E4M3 || dt == SFR_E5M2; }
bool scale_ok(int kind) { return kind == SFR_SCALE_ROW || kind == SFR_SCALE_TENSOR; }
// Bound on rows * cols of any one tensor, keeping every grid within HIP's limits.
constexpr int64_t kMaxElems = (int64_t)1 << 40;

bool act_ok(int act) { return act == SFR_ACT_SILU || act == SFR_ACT_GELU_TANH || act == SFR_ACT_RELU; }
bool out_ok(int dt) { return dt == SFR_OUT_BF16 || dt == SFR_OUT_F32; }
bool save_ok(int s) { return s >= SFR_SAVE_NONE && s <= SFR_SAVE_E5M2; }
bool save8(int s) { return s == SFR_SAVE_E4M3 || s == SFR_SAVE_E5M2; }
bool block_dim(int64_t d, int64_t multiple) { return d > 0 && d <= SFR_MAX_BLOCK_DIM && d % multiple == 0; }
bool gated_dim(int64_t f) { return block_dim(f, 32) && 2 * f <= SFR_MAX_BLOCK_DIM; }
// An output of the dense products: its tiles make one grid.
bool dense_ok(int64_t rows, int64_t cols) {
  const int64_t t = rows > 64 ? 128 : 64;
  return ((rows + t - 1) / t) * ((cols + t - 1) / t) <= ((int64_t)1 << 21);
}
bool gated_shape(int64_t m, int64_t k, int64_t f) {
  return m >= 0 && m <= SFR_MAX_DIM && block_dim(k, 32) && gated_dim(f) && dense_ok(m, 2 * f) &&
         dense_ok(m, k) && dense_ok(2 * f, k);
}

sfr_status launch_status(hipError_t e) { return e == hipSuccess ? SFR_OK : SFR_ERR_LAUNCH; }

}  // namespace

extern "C" {

sfr_status quantize_rowwise_fp8(const uint16_t* x, int64_t rows, int64_t cols, sfr_fp8_t dt, uint8_t* q,
                                float* scale, void* stream) {
  if (!fp8_ok(dt)) return SFR_ERR_DTYPE;
  if (rows < 0 || rows > SFR_MAX_DIM || cols <= 0 || cols > SFR_MAX_DIM || cols % 8 != 0 ||
      rows * cols > kMaxElems)
    return SFR_ERR_SHAPE;
  if (rows == 0) return SFR_OK;
  if (!x || !q || !scale) return SFR_ERR_NULL;
  if (!aligned16(x) || !aligned16(q) || !aligned16(scale)) return SFR_ERR_ALIGN;
  return launch_status(sfr::launch_quantize(x, rows, cols, dt, q, scale, static_cast<hipStream_t>(stream)));
}

int64_t sfr_quantize_tensorwise_workspace_bytes(int64_t rows, int64_t cols) {
  if (rows <= 0 || rows > SFR_MAX_DIM || cols <= 0 || cols > SFR_MAX_DIM || cols % 8 != 0 || rows * cols > kMaxElems)
    return 0;
  return sfr::tensor_workspace_bytes(rows, cols);
}

sfr_status quantize_tensorwise_fp8(const uint16_t* x, int64_t rows, int64_t cols, sfr_fp8_t dt, uint8_t* q,
                                   float* scale, void* workspace, int64_t workspace_bytes, void* stream) {
  if (!fp8_ok(dt)) return SFR_ERR_DTYPE;
  if (rows < 0 || rows > SFR_MAX_DIM || cols <= 0 || cols > SFR_MAX_DIM || cols % 8 != 0 ||
      rows * cols > kMaxElems)
    return SFR_ERR_SHAPE;
  if (rows == 0) return SFR_OK;
  if (workspace_bytes < sfr::tensor_workspace_bytes(rows, cols)) return SFR_ERR_SHAPE;
  if (!x || !q || !scale || !workspace) return SFR_ERR_NULL;
  if (!aligned16(x) || !aligned16(q) || !aligned16(scale) || !aligned16(workspace)) return SFR_ERR_ALIGN;
  return launch_status(
      sfr::launch_quantize_tensor(x, rows, cols, dt, q, scale, workspace, static_cast<hipStream_t>(stream)));
}

sfr_status quantize_tensorwise_fp8_noalloc(const uint16_t* x, int64_t rows, int64_t cols, sfr_fp8_t dt, uint8_t* q,
                                           float* scale, void* stream) {
  if (!fp8_ok(dt)) return SFR_ERR_DTYPE;
  if (rows < 0 || rows > SFR_MAX_DIM || cols <= 0 || cols > SFR_MAX_DIM || cols % 8 != 0 ||
      rows * cols > kMaxElems)
    return SFR_ERR_SHAPE;
  if (rows == 0) return SFR_OK;
  if (sfr::tensor_workspace_bytes(rows, cols) > sfr::noalloc_workspace_bytes()) return SFR_ERR_SHAPE;
  if (!x || !q || !scale) return SFR_ERR_NULL;
  if (!aligned16(x) || !aligned16(q) || !aligned16(scale)) return SFR_ERR_ALIGN;
  return launch_status(
      sfr::launch_quantize_tensor_noalloc(x, rows, cols, dt, q, scale, static_cast<hipStream_t>(stream)));
}

sfr_status compress_2to4_fp8(const uint8_t* w, int64_t n, int64_t k, sfr_fp8_t dt, uint8_t* values, uint8_t* meta,
                             void* stream) {
  if (!fp8_ok(dt)) return SFR_ERR_DTYPE;
  if (n < 0 || n > SFR_MAX_DIM || k <= 0 || k > SFR_MAX_DIM || k % 128 != 0 || n * k > kMaxElems)
    return SFR_ERR_SHAPE;
  if (n == 0) return SFR_OK;
  if (!w || !values || !meta) return SFR_ERR_NULL;
  if (!aligned16(w) || !aligned16(values) || !aligned16(meta)) return SFR_ERR_ALIGN;
  return launch_status(sfr::launch_compress(w, n, k, values, meta, static_cast<hipStream_t>(stream)));
}

sfr_status prune_2to4_bf16(const uint16_t* w, int64_t n, int64_t k, uint16_t* out, void* stream) {
  if (n < 0 || n > SFR_MAX_DIM || k <= 0 || k > SFR_MAX_DIM || k % 8 != 0 || n * k > kMaxElems)
    return SFR_ERR_SHAPE;
  if (n == 0) return SFR_OK;
  if (!w || !out) return SFR_ERR_NULL;
  if (!aligned16(w) || !aligned16(out)) return SFR_ERR_ALIGN;
  return launch_status(sfr::launch_prune_bf16(w, n, k, out, static_cast<hipStream_t>(stream)));
}

int sfr_linear_algo_count(void) { return sfr::ALGO_COUNT; }

int sfr_linear_algo_valid(int algo) { return sfr::linear_algo_valid(algo) ? 1 : 0; }

const char* sfr_linear_algo_name(int algo) { return sfr::linear_algo_name(algo); }

int sfr_linear_algo_supported(int algo, int64_t m, int64_t n, int64_t k) {
  if (m <= 0 || n <= 0 || n % 16 != 0 || k <= 0 || k % 128 != 0) return 0;
  return sfr::linear_algo_supported(algo, m, n, k) ? 1 : 0;
}

int sfr_linear_default_algo(int64_t m, int64_t n, int64_t k) { return sfr::linear_default_algo(m, n, k); }

sfr_status sparse_fp8_scaled_linear_algo(const uint8_t* xq, sfr_fp8_t x_dt, const float* xs, sfr_scale_t xs_kind,
                                         int64_t m, int64_t k, const uint8_t* values, const uint8_t* meta,
                                         sfr_fp8_t w_dt, const float* ws, sfr_scale_t ws_kind, int64_t n,
                                         const uint16_t* bias, void* out, sfr_out_t out_dt, int algo,
                                         void* stream) {
  if (!fp8_ok(x_dt) || !fp8_ok(w_dt) || (out_dt != SFR_OUT_BF16 && out_dt != SFR_OUT_F32) || !scale_ok(xs_kind) ||
      !scale_ok(ws_kind) || (algo != SFR_ALGO_DEFAULT && !sfr::linear_algo_valid(algo)))
    return SFR_ERR_DTYPE;
  if (m < 0 || m > SFR_MAX_DIM || n < 0 || n > SFR_MAX_DIM || n % 16 != 0 || k <= 0 || k > SFR_MAX_DIM ||
      k % 128 != 0 || m * k > kMaxElems || n * k > kMaxElems || m * n > kMaxElems)
    return SFR_ERR_SHAPE;
  if (m == 0 || n == 0) return SFR_OK;
  if (algo != SFR_ALGO_DEFAULT && !sfr::linear_algo_supported(algo, m, n, k)) return SFR_ERR_SHAPE;
  if (!xq || !xs || !values || !meta || !ws || !out) return SFR_ERR_NULL;
  if (!aligned16(xq) || !aligned16(xs) || !aligned16(values) || !aligned16(meta) || !aligned16(ws) ||
      !aligned16(out) || (bias && !aligned16(bias)))
    return SFR_ERR_ALIGN;
  sfr::LinearArgs a{xq, xs, values, meta, ws, bias, out, m, n, k, (int)x_dt, (int)w_dt, (int)out_dt,
                    xs_kind == SFR_SCALE_ROW ? 1 : 0, ws_kind == SFR_SCALE_ROW ? 1 : 0};
  return launch_status(sfr::launch_linear_algo(a, algo, static_cast<hipStream_t>(stream)));
}

sfr_status sparse_fp8_scaled_linear(const uint8_t* xq, sfr_fp8_t x_dt, const float* xs, sfr_scale_t xs_kind, int64_t m,
                                    int64_t k, const uint8_t* values, const uint8_t* meta, sfr_fp8_t w_dt,
                                    const float* ws, sfr_scale_t ws_kind, int64_t n, const uint16_t* bias, void* out,
                                    sfr_out_t out_dt, void* stream) {
  return sparse_fp8_scaled_linear_algo(xq, x_dt, xs, xs_kind, m, k, values, meta, w_dt, ws, ws_kind, n, bias, out,
                                       out_dt, SFR_ALGO_DEFAULT, stream);
}

sfr_status sparse_fp8_rowwise_linear_dynamic_algo(const uint16_t* x, sfr_fp8_t x_dt, int64_t m, int64_t k,
                                                  const uint8_t* values, const uint8_t* meta, sfr_fp8_t w_dt,
                                                  const float* ws, sfr_scale_t ws_kind, int64_t n,
                                                  const uint16_t* bias, void* out, sfr_out_t out_dt, uint8_t* xq,
                                                  float* xs, int algo, void* stream) {
  if (!fp8_ok(x_dt) || !fp8_ok(w_dt) || (out_dt != SFR_OUT_BF16 && out_dt != SFR_OUT_F32) || !scale_ok(ws_kind) ||
      (algo != SFR_ALGO_DEFAULT && !sfr::linear_algo_valid(algo)))
    return SFR_ERR_DTYPE;
  if (m < 0 || m > SFR_MAX_DIM || n < 0 || n > SFR_MAX_DIM || n % 16 != 0 || k <= 0 || k > SFR_MAX_DIM ||
      k % 128 != 0 || m * k > kMaxElems || n * k > kMaxElems || m * n > kMaxElems)
    return SFR_ERR_SHAPE;
  if (m == 0 || n == 0) return SFR_OK;
  if (algo != SFR_ALGO_DEFAULT && !sfr::linear_algo_supported(algo, m, n, k)) return SFR_ERR_SHAPE;
  if (!x || !values || !meta || !ws || !out || !xq || !xs) return SFR_ERR_NULL;
  if (!aligned16(x) || !aligned16(values) || !aligned16(meta) || !aligned16(ws) || !aligned16(out) ||
      !aligned16(xq) || !aligned16(xs) || (bias && !aligned16(bias)))
    return SFR_ERR_ALIGN;
  sfr::LinearArgs a{xq, xs, values, meta, ws, bias, out, m, n, k, (int)x_dt, (int)w_dt, (int)out_dt, 1,
                    ws_kind == SFR_SCALE_ROW ? 1 : 0};
  return launch_status(sfr::launch_linear_dynamic(x, xq, xs, a, algo, static_cast<hipStream_t>(stream)));
}

sfr_status sparse_fp8_rowwise_linear_dynamic(const uint16_t* x, sfr_fp8_t x_dt, int64_t m, int64_t k,
                                             const uint8_t* values, const uint8_t* meta, sfr_fp8_t w_dt,
                                             const float* ws, sfr_scale_t ws_kind, int64_t n, const uint16_t* bias,
                                             void* out, sfr_out_t out_dt, uint8_t* xq, float* xs, void* stream) {
  return sparse_fp8_rowwise_linear_dynamic_algo(x, x_dt, m, k, values, meta, w_dt, ws, ws_kind, n, bias, out, out_dt,
                                                xq, xs, SFR_ALGO_DEFAULT, stream);
}

sfr_status sparse_fp8_rowwise_linear(const uint8_t* xq, sfr_fp8_t x_dt, const float* xs, int64_t m, int64_t k,
                                     const uint8_t* values, const uint8_t* meta, sfr_fp8_t w_dt, const float* ws,
                                     int64_t n, const uint16_t* bias, void* out, sfr_out_t out_dt, void* stream) {
  return sparse_fp8_scaled_linear(xq, x_dt, xs, SFR_SCALE_ROW, m, k, values, meta, w_dt, ws, SFR_SCALE_ROW, n, bias,
                                  out, out_dt, stream);
}

sfr_status bsr_count_bf16(const uint16_t* w, int64_t n, int64_t k, int32_t* crow, void* stream) {
  if (n < 0 || n > SFR_MAX_DIM || n % SFR_BSR_BLOCK != 0 || k <= 0 || k > SFR_MAX_DIM || k % SFR_BSR_BLOCK != 0 ||
      n * k > kMaxElems)
    return SFR_ERR_SHAPE;
  if (!crow || (n > 0 && !w)) return SFR_ERR_NULL;
  if ((reinterpret_cast<uintptr_t>(crow) & 3u) || (w && !aligned16(w))) return SFR_ERR_ALIGN;
  return launch_status(sfr::launch_bsr_count(w, n, k, crow, static_cast<hipStream_t>(stream)));
}

sfr_status bsr_fill_bf16(const uint16_t* w, int64_t n, int64_t k, const int32_t* crow, int32_t* col,
                         uint16_t* values, void* stream) {
  if (n < 0 || n > SFR_MAX_DIM || n % SFR_BSR_BLOCK != 0 || k <= 0 || k > SFR_MAX_DIM || k % SFR_BSR_BLOCK != 0 ||
      n * k > kMaxElems)
    return SFR_ERR_SHAPE;
  if (n == 0) return SFR_OK;
  if (!w || !crow) return SFR_ERR_NULL;
  if (!aligned16(w) || (reinterpret_cast<uintptr_t>(crow) & 3u) || (reinterpret_cast<uintptr_t>(col) & 3u) ||
      (values && !aligned16(values)))
    return SFR_ERR_ALIGN;
  return launch_status(sfr::launch_bsr_fill(w, n, k, crow, col, values, static_cast<hipStream_t>(stream)));
}

sfr_status bsr_linear_bf16(const uint16_t* x, int64_t m, int64_t k, const int32_t* crow, const int32_t* col,
                           const uint16_t* values, int64_t n, const uint16_t* bias, void* out, sfr_out_t out_dt,
                           void* stream) {
  if (out_dt != SFR_OUT_BF16 && out_dt != SFR_OUT_F32) return SFR_ERR_DTYPE;
  if (m < 0 || m > SFR_MAX_DIM || n < 0 || n > SFR_MAX_DIM || n % SFR_BSR_BLOCK != 0 || k <= 0 ||
      k > SFR_MAX_DIM || k % SFR_BSR_BLOCK != 0 || m * k > kMaxElems || n * k > kMaxElems || m * n > kMaxElems ||
      (n / 16) * ((m + 15) / 16) > INT32_MAX)
    return SFR_ERR_SHAPE;
  if (m == 0 || n == 0) return SFR_OK;
  if (!x || !crow || !out) return SFR_ERR_NULL;
  if (!aligned16(x) || (reinterpret_cast<uintptr_t>(crow) & 3u) || (reinterpret_cast<uintptr_t>(col) & 3u) ||
      (values && !aligned16(values)) || !aligned16(out) || (bias && !aligned16(bias)))
    return SFR_ERR_ALIGN;
  return launch_status(sfr::launch_bsr_linear(x, m, k, crow, col, values, n, bias, out, (int)out_dt,
                                              static_cast<hipStream_t>(stream)));
}

sfr_status quantize_mx(const uint16_t* x, int64_t rows, int64_t cols, sfr_mx_t dt, uint8_t* q, uint8_t* scale,
                       void* stream) {
  if (dt < SFR_MX_E4M3 || dt > SFR_MX_E2M1) return SFR_ERR_DTYPE;
  if (rows < 0 || rows > SFR_MAX_DIM || cols <= 0 || cols > SFR_MAX_DIM || cols % SFR_MX_BLOCK != 0 ||
      rows * cols > kMaxElems)
    return SFR_ERR_SHAPE;
  if (rows == 0) return SFR_OK;
  if (!x || !q || !scale) return SFR_ERR_NULL;
  if (!aligned16(x) || !aligned16(q) || !aligned16(scale)) return SFR_ERR_ALIGN;
  return launch_status(sfr::launch_quantize_mx(x, rows, cols, dt, q, scale, static_cast<hipStream_t>(stream)));
}

sfr_status dequantize_mx(const uint8_t* q, const uint8_t* scale, int64_t rows, int64_t cols, sfr_mx_t dt,
                         uint16_t* out, void* stream) {
  if (dt < SFR_MX_E4M3 || dt > SFR_MX_E2M1) return SFR_ERR_DTYPE;
  if (rows < 0 || rows > SFR_MAX_DIM || cols <= 0 || cols > SFR_MAX_DIM || cols % SFR_MX_BLOCK != 0 ||
      rows * cols > kMaxElems)
    return SFR_ERR_SHAPE;
  if (rows == 0) return SFR_OK;
  if (!q || !scale || !out) return SFR_ERR_NULL;
  if (!aligned16(q) || !aligned16(scale) || !aligned16(out)) return SFR_ERR_ALIGN;
  return launch_status(sfr::launch_dequantize_mx(q, scale, rows, cols, dt, out, static_cast<hipStream_t>(stream)));
}

sfr_status gated_linear_bf16(const uint16_t* x, int64_t m, int64_t k, const uint16_t* w, int64_t f, sfr_act_t act,
                             uint16_t* h, sfr_save_t save, void* gu, uint8_t* gu_scale, void* stream) {
  if (!act_ok(act) || !save_ok(save)) return SFR_ERR_DTYPE;
  if (!gated_shape(m, k, f)) return SFR_ERR_SHAPE;
  if (m == 0) return SFR_OK;
  if (!x || !w || !h || (save != SFR_SAVE_NONE && !gu) || (save8(save) && !gu_scale)) return SFR_ERR_NULL;
  if (!aligned16(x) || !aligned16(w) || !aligned16(h) || (save != SFR_SAVE_NONE && !aligned16(gu)) ||
      (save8(save) && !aligned16(gu_scale)))
    return SFR_ERR_ALIGN;
  const sfr::GatedArgs a{x, w, nullptr, m, k, f, (int)act, h, (int)save, gu, gu_scale};
  return launch_status(sfr::launch_gated(a, static_cast<hipStream_t>(stream)));
}

int64_t sfr_gated_backward_workspace_bytes(int64_t m, int64_t k, int64_t f, sfr_save_t x_save) {
  if (!save_ok(x_save) || x_save == SFR_SAVE_NONE || !gated_shape(m, k, f)) return 0;
  return sfr::gated_backward_workspace_bytes(m, k, f, save8(x_save));
}

sfr_status gated_linear_bf16_backward(const uint16_t* dh, int64_t m, int64_t k, int64_t f, sfr_act_t act,
                                      const void* gu, const uint8_t* gu_scale, sfr_save_t gu_save, const void* x,
                                      const uint8_t* x_scale, sfr_save_t x_save, const uint16_t* w, uint16_t* dx,
                                      uint16_t* dw, void* workspace, int64_t workspace_bytes, void* stream) {
  if (!act_ok(act) || !save_ok(gu_save) || gu_save == SFR_SAVE_NONE || !save_ok(x_save) || x_save == SFR_SAVE_NONE)
    return SFR_ERR_DTYPE;
  if (!gated_shape(m, k, f)) return SFR_ERR_SHAPE;
  if (workspace_bytes < sfr::gated_backward_workspace_bytes(m, k, f, save8(x_save))) return SFR_ERR_SHAPE;
  if (!dx && !dw) return SFR_OK;
  if (m > 0 && (!dh || !gu || !workspace || (save8(gu_save) && !gu_scale) || (dx && !w) ||
                (dw && (!x || (save8(x_save) && !x_scale)))))
    return SFR_ERR_NULL;
  if (!aligned16(dh) || !aligned16(gu) || !aligned16(workspace) || !aligned16(dx) || !aligned16(dw) ||
      (save8(gu_save) && !aligned16(gu_scale)) || (dx && !aligned16(w)) ||
      (dw && (!aligned16(x) || (save8(x_save) && !aligned16(x_scale)))))
    return SFR_ERR_ALIGN;
  const sfr::GatedBackwardArgs a{dh,          w,  m,       k,           f, (int)act, (int)gu_save, gu, gu_scale,
                                 (int)x_save, x,  x_scale, dx,          dw};
  return launch_status(sfr::launch_gated_backward(a, workspace, static_cast<hipStream_t>(stream)));
}

int64_t sfr_mxfp4_workspace_bytes(int64_t m, int64_t n, int64_t k) {
  if (m <= 0 || m > SFR_MAX_DIM || !block_dim(n, 16) || !block_dim(k, 32) || !dense_ok(m, n)) return 0;
  return sfr::mxfp4_workspace_bytes(m, n, k);
}

sfr_status mxfp4_linear(const uint16_t* x, int64_t m, int64_t k, const uint8_t* wq, const uint8_t* ws, int64_t n,
                        const uint16_t* bias, void* out, sfr_out_t out_dt, void* workspace, int64_t workspace_bytes,
                        void* stream) {
  if (!out_ok(out_dt)) return SFR_ERR_DTYPE;
  if (m < 0 || m > SFR_MAX_DIM || (n != 0 && !block_dim(n, 16)) || !block_dim(k, 32) || !dense_ok(m, n))
    return SFR_ERR_SHAPE;
  if (m == 0 || n == 0) return SFR_OK;
  const int64_t need = sfr::mxfp4_workspace_bytes(m, n, k);
  if (workspace_bytes < need) return SFR_ERR_SHAPE;
  if (!x || !wq || !ws || !out || (need > 0 && !workspace)) return SFR_ERR_NULL;
  if (!aligned16(x) || !aligned16(wq) || !aligned16(ws) || !aligned16(out) || (bias && !aligned16(bias)) ||
      (need > 0 && !aligned16(workspace)))
    return SFR_ERR_ALIGN;
  const sfr::StreamArgs a{x, wq, ws, m, k, n, false, 0, bias, out, (int)out_dt};
  return launch_status(sfr::launch_mxfp4(a, workspace, static_cast<hipStream_t>(stream)));
}

sfr_status mxfp4_gated_linear(const uint16_t* x, int64_t m, int64_t k, const uint8_t* wq, const uint8_t* ws, int64_t f,
                              sfr_act_t act, uint16_t* h, void* stream) {
  if (!act_ok(act)) return SFR_ERR_DTYPE;
  if (m < 0 || m > SFR_MAX_DIM || !gated_dim(f) || !block_dim(k, 32) || !dense_ok(m, 2 * f))
    return SFR_ERR_SHAPE;
  if (m == 0) return SFR_OK;
  if (!x || !wq || !ws || !h) return SFR_ERR_NULL;
  if (!aligned16(x) || !aligned16(wq) || !aligned16(ws) || !aligned16(h)) return SFR_ERR_ALIGN;
  const sfr::StreamArgs a{x, wq, ws, m, k, f, true, (int)act, nullptr, h, (int)SFR_OUT_BF16};
  return launch_status(sfr::launch_mxfp4(a, nullptr, static_cast<hipStream_t>(stream)));
}

const char* sfr_block_kernel(sfr_product_t product, int64_t m, int64_t k, int64_t f, int32_t* slices) {
  static_assert((int)SFR_PRODUCT_GATED == sfr::PRODUCT_GATED &&
                    (int)SFR_PRODUCT_MXFP4_GATED == sfr::PRODUCT_MXFP4_GATED,
                "the same numbers");
  if (product < SFR_PRODUCT_GATED || product > SFR_PRODUCT_MXFP4_GATED || m <= 0 || m > SFR_MAX_DIM) return nullptr;
  if (product == SFR_PRODUCT_MXFP4       ? !block_dim(f, 16) || !block_dim(k, 32) || !dense_ok(m, f)
      : product == SFR_PRODUCT_MXFP4_GATED ? !gated_dim(f) || !block_dim(k, 32) || !dense_ok(m, 2 * f)
                                         : !gated_shape(m, k, f))
    return nullptr;
  const sfr::DenseKernel c = sfr::block_kernel((int)product, m, k, f);
  if (slices) *slices = c.slices;
  return c.name;
}

const char* sfr_status_string(sfr_status s) {
  switch (s) {
    case SFR_OK: return "ok";
    case SFR_ERR_NULL: return "null pointer";
    case SFR_ERR_SHAPE: return "invalid shape";
    case SFR_ERR_ALIGN: return "pointer not 16-byte aligned";
    case SFR_ERR_DTYPE: return "invalid dtype";
    case SFR_ERR_LAUNCH: return "kernel launch failed";
  }
  return "unknown status";
}

int sfr_format_version(void) { return SFR_FORMAT_VERSION; }

}  // extern "C"

// Host-side launchers of the gfx950 kernels (internal; the C ABI validates
// arguments before calling these).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace sfr {

hipError_t launch_quantize(const uint16_t* x, int64_t rows, int64_t cols, int fmt, uint8_t* q,
                           float* scale, hipStream_t stream);

// Tensor-wise quantization: workspace of tensor_workspace_bytes(rows, cols).
int64_t tensor_workspace_bytes(int64_t rows, int64_t cols);
hipError_t launch_quantize_tensor(const uint16_t* x, int64_t rows, int64_t cols, int fmt, uint8_t* q, float* scale,
                                  void* workspace, hipStream_t stream);
// The same on the library's own per-device workspace of noalloc_workspace_bytes().
int64_t noalloc_workspace_bytes();
hipError_t launch_quantize_tensor_noalloc(const uint16_t* x, int64_t rows, int64_t cols, int fmt, uint8_t* q,
                                          float* scale, hipStream_t stream);

hipError_t launch_compress(const uint8_t* w, int64_t n, int64_t k, uint8_t* values, uint8_t* meta,
                           hipStream_t stream);

// 2:4 pruning of a bf16 matrix (k % 8 == 0); out may be w.
hipError_t launch_prune_bf16(const uint16_t* w, int64_t n, int64_t k, uint16_t* out, hipStream_t stream);

struct LinearArgs {
  const uint8_t* xq;
  const float* xs;
  const uint8_t* values;
  const uint8_t* meta;
  const float* ws;
  const uint16_t* bias;  // may be null
  void* out;
  int64_t m, n, k;
  int x_fmt, w_fmt, out_fmt;
  int xs_stride, ws_stride;  // 1: one scale per row; 0: one scale for the operand
};

hipError_t launch_linear(const LinearArgs& a, hipStream_t stream);

// Kernel configurations of the linear layer.  algo < 0: the built-in choice.
enum LinearAlgo {
  ALGO_DECODE_LDS = 0,     // m <= 16, k % 1024 == 0: 16 weight rows per workgroup, one 1024-k unit per wavefront via LDS
  ALGO_DECODE_REG = 1,     // m <= 16: 16 weight rows per workgroup, streamed to registers
  ALGO_TILED_64 = 2,       // 64 x 64 tiles, 4 wavefronts
  ALGO_TILED_128 = 3,      // 128 x 128 tiles, 4 wavefronts
  ALGO_TILED_256 = 4,      // 256 x 256 tiles, 8 wavefronts
  ALGO_WIDE_256 = 5,       // 256 x 256 tiles, 4 software-pipelined wavefronts (k >= 512)
  ALGO_DECODE_LDS_32 = 6,  // as ALGO_DECODE_LDS with 32 weight rows per workgroup (n % 32 == 0)
  ALGO_TILED_256x128 = 7,  // 256 (n) x 128 (m) tiles, 8 wavefronts, one workgroup per CU
  ALGO_COUNT = 8
};
// Flag of an algorithm id: FP8 matrix-instruction accumulation (products of
// one instruction added 13 bits below the largest) instead of the default
// binary32-grade accumulation on exactly widened operands.
constexpr int ALGO_ACC_F8_FLAG = 0x100;
bool linear_algo_valid(int algo);
const char* linear_algo_name(int algo);
bool linear_algo_supported(int algo, int64_t m, int64_t n, int64_t k);
int linear_default_algo(int64_t m, int64_t n, int64_t k);
hipError_t launch_linear_algo(const LinearArgs& a, int algo, hipStream_t stream);

// Row-wise quantization of x into (xq, xs) and the linear layer on them (a's
// xq / xs are ignored) with algorithm `algo` (< 0: the built-in choice): one
// fused launch for small decode shapes on the built-in configuration, else two.
hipError_t launch_linear_dynamic(const uint16_t* x, uint8_t* xq, float* xs, const LinearArgs& a, int algo,
                                 hipStream_t stream);

// Block-sparse (BSR, 64 x 64 blocks) bf16 weight.
hipError_t launch_bsr_count(const uint16_t* w, int64_t n, int64_t k, int32_t* crow, hipStream_t stream);
hipError_t launch_bsr_fill(const uint16_t* w, int64_t n, int64_t k, const int32_t* crow, int32_t* col,
                           uint16_t* values, hipStream_t stream);
hipError_t launch_bsr_linear(const uint16_t* x, int64_t m, int64_t k, const int32_t* crow, const int32_t* col,
                             const uint16_t* values, int64_t n, const uint16_t* bias, void* out, int out_fmt,
                             hipStream_t stream);

// MX block formats (fmt: MX_E4M3, MX_E5M2, MX_E2M1); cols % 32 == 0.
hipError_t launch_quantize_mx(const uint16_t* x, int64_t rows, int64_t cols, int fmt, uint8_t* q, uint8_t* scale,
                              hipStream_t stream);
hipError_t launch_dequantize_mx(const uint8_t* q, const uint8_t* scale, int64_t rows, int64_t cols, int fmt,
                                uint16_t* out, hipStream_t stream);

// How activations are saved for the backward pass.
enum { GU_NONE = 0, GU_BF16 = 1, GU_E4M3 = 2, GU_E5M2 = 3 };

struct GatedArgs {
  const uint16_t* x;       // [m, k]
  const void* w;           // [2 f, k]: bf16, or 4-bit codes
  const uint8_t* w_scale;  // the codes' scales; null for bf16
  int64_t m, k, f;
  int act;
  uint16_t* h;  // [m, f]
  int gu_fmt;
  void* gu;           // [m, 2 f]
  uint8_t* gu_scale;  // [m, 2 f / 32]
};
hipError_t launch_gated(const GatedArgs& a, hipStream_t stream);
hipError_t launch_gated_dense(const GatedArgs& a, hipStream_t stream);  // the matrix-core form, any m

struct GatedBackwardArgs {
  const uint16_t *dh, *w;
  int64_t m, k, f;
  int act;
  int gu_fmt;
  const void* gu;
  const uint8_t* gu_scale;
  int x_fmt;
  const void* x;
  const uint8_t* x_scale;
  uint16_t *dx, *dw;  // either may be null
};
int64_t gated_backward_workspace_bytes(int64_t m, int64_t k, int64_t f, bool x_mx);
hipError_t launch_gated_backward(const GatedBackwardArgs& a, void* workspace, hipStream_t stream);

// Dense products with binary32 sums: dx = dgu w; dw = dgu^T x.
int64_t dense_dx_workspace_bytes(int64_t m, int64_t k, int64_t f2);
hipError_t launch_dense_dx(const uint16_t* dgu, const uint16_t* w, int64_t m, int64_t k, int64_t f2, uint16_t* dx,
                           void* workspace, hipStream_t stream);
hipError_t launch_dense_dw(const uint16_t* dgu, const uint16_t* x, int64_t m, int64_t k, int64_t f2, uint16_t* dw,
                           hipStream_t stream);

// Products of few activation rows: a bf16 weight (w_scale null, gated only)
// or a 4-bit one.  rows: n, or f when gated.
struct StreamArgs {
  const uint16_t* x;
  const void* w;
  const uint8_t* w_scale;
  int64_t m, k, rows;
  bool gated;
  int act;
  const uint16_t* bias;
  void* out;
  int out_fmt;
  const float *xs, *ws;  // ws not null: x and w are 8-bit integers with these scales
};
bool stream_rows(int64_t m, int64_t n, int64_t k, bool fp4, bool gated);  // n: weight rows (2 f when gated)
hipError_t launch_stream(const StreamArgs& a, hipStream_t stream);
const char* stream_name(const StreamArgs& a);  // of the form that launch_stream takes
// Modelled time of the matrix-core form, us.
double dense_us(int64_t m, int64_t n, int64_t k, bool fp4, bool gated);
// The matrix-core form of the 4-bit linear layer (not gated), any m.
int64_t dense_nt_workspace_bytes(int64_t m, int64_t n, int64_t k);
hipError_t launch_mxfp4_dense(const StreamArgs& a, void* workspace, hipStream_t stream);

// The matrix-core kernel that a product takes: its name and the slices of its sum.
struct DenseKernel {
  const char* name;
  int slices;
};
DenseKernel dense_gated_kernel(int64_t m, int64_t k, int64_t f);
DenseKernel dense_mxfp4_kernel(int64_t m, int64_t n, int64_t k);
DenseKernel dense_dx_kernel(int64_t m, int64_t k, int64_t f2);
DenseKernel dense_dw_kernel(int64_t m, int64_t k, int64_t f2);
// The same of any product of the block, streamed forms among them (f: n for PRODUCT_MXFP4).
enum { PRODUCT_GATED = 0, PRODUCT_GATED_SAVING, PRODUCT_DX, PRODUCT_DW, PRODUCT_MXFP4, PRODUCT_MXFP4_GATED };
DenseKernel block_kernel(int product, int64_t m, int64_t k, int64_t f);

// Rows of one launch with a wavefront per row: a grid has fewer than 2^32 threads.
constexpr int64_t kGridRows = (int64_t)1 << 25;

// 8-bit integers with a scale per row: the quantizer, and the product of two
// quantized matrices (or of a bf16 x, quantized into the workspace first).
hipError_t launch_quantize_int8(const uint16_t* x, int64_t rows, int64_t cols, int8_t* q, float* scale,
                                hipStream_t stream);
struct Int8Args {
  const uint16_t* x;  // bf16, or null where xq and xs are given
  const int8_t* xq;
  const float* xs;
  const int8_t* wq;
  const float* ws;
  const uint16_t* bias;  // may be null
  void* out;
  int64_t m, n, k;
  int out_fmt;
};
bool stream_rows_int8(int64_t m, int64_t n, int64_t k);
double dense_int8_us(int64_t m, int64_t n, int64_t k);
int64_t dense_int8_workspace_bytes(int64_t m, int64_t n, int64_t k);
hipError_t launch_int8_dense(const Int8Args& a, void* workspace, hipStream_t stream);
DenseKernel dense_int8_kernel(int64_t m, int64_t n, int64_t k);
int64_t int8_workspace_bytes(int64_t m, int64_t n, int64_t k, bool dynamic);
hipError_t launch_int8(const Int8Args& a, void* workspace, hipStream_t stream);
DenseKernel int8_kernel(int64_t m, int64_t n, int64_t k, bool dynamic);

int64_t mxfp4_workspace_bytes(int64_t m, int64_t n, int64_t k);  // of the linear layer; the gated block needs none
hipError_t launch_mxfp4(const StreamArgs& a, void* workspace, hipStream_t stream);

// The mixture of gated feed-forward blocks.
enum { ROUTE_SOFTMAX = 0, ROUTE_SIGMOID = 1 };
enum { EXPERT_BF16 = 0, EXPERT_INT8 = 1, EXPERT_FP4 = 2 };
constexpr int kMoeExperts = 1024, kMoeTop = 16, kMoeTokens = 64;  // most experts, choices; tokens of one pass
struct RouteArgs {
  const uint16_t *x, *w;
  int64_t m;
  int k, experts;
  const float* bias;  // may be null
  int top, score, renormalize;
  float* logits;   // [m, experts]
  int32_t* ids;    // [m, top]
  float* weights;  // [m, top]
};
hipError_t launch_moe_route(const RouteArgs& a, hipStream_t stream);
struct MoeArgs {
  const uint16_t* x;
  int m, k, f, experts, top;  // m: tokens of one pass
  const int32_t* ids;
  const float* weights;
  int form;
  const void *w_gu, *s_gu;      // [experts, 2 f, k]; scales: a float per row (INT8), a byte per 32 (FP4)
  const void *w_down, *s_down;  // [experts, k, f]
  int act;
  uint16_t* h;  // workspace [m, top, f]
  float* y;     // workspace [m, top, k]
  uint16_t* out;
};
int64_t moe_workspace_bytes(int64_t m, int64_t k, int64_t f, int top);
hipError_t launch_moe_layer(const MoeArgs& a, int64_t m, hipStream_t stream);

}  // namespace sfr

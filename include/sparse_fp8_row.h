/*
 * sparse_fp8_row.h -- C ABI of the MI355X (gfx950) row-wise-scaled FP8 linear
 * layer with a 2:4 semi-structured sparse weight.
 *
 * The operation (pytorch/ao PR #1671, "Add CUTLASS-based row-wise scaled
 * sparse FP8 kernel", ready-for-review comment, item 1: a converter of FP8
 * data to a 2:4 sparse format, and a row-wise scaled linear operator for a
 * sparse FP8 weight and an FP8 activation; item 4: the activation is quantized
 * dynamically) is, with torch `linear` conventions (weight [N, K]):
 *
 *     out[m, n] = bf16( xs[m] * ws[n] * sum_k xq[m, k] * wq[n, k]  (+ bias[n]) )
 *
 * where xq/xs is the FP8 activation with one binary32 scale per row, wq/ws the
 * FP8 weight with one binary32 scale per output row, and wq keeps at most two
 * non-zeros in every group of four consecutive k.  Either operand may be OCP
 * e4m3 ("fn": max 448, no infinities) or e5m2 (max 57344); the four dtype
 * pairs are the four instantiations the pages list (pytorch/ao issue #3516,
 * "Making torchao ABI compatible ...", file table).  A plain C ABI, free of
 * any framework's C++ types, is the point that issue makes.
 *
 * Conventions shared by every entry point:
 *  - All tensor pointers are DEVICE pointers to contiguous row-major data and
 *    must be 16-byte aligned.  The caller owns all memory; the library never
 *    allocates, frees or synchronizes.
 *  - `stream` is a hipStream_t (NULL = the default stream).  Work is enqueued
 *    on it and the call returns without waiting.  The library keeps no state
 *    between calls and may be called from several host threads at once.
 *  - Arguments are validated on the host before anything is launched.  On an
 *    error nothing is launched and no output is touched.  Device faults (bad
 *    pointers that pass validation) surface at the caller's next
 *    synchronization, as usual in HIP.
 *  - Outputs must not alias inputs.
 *  - Inputs must be finite.  NaN or infinite inputs give unspecified results.
 */
#ifndef SPARSE_FP8_ROW_H
#define SPARSE_FP8_ROW_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* FP8 formats (OCP 8-bit floating point). */
typedef enum { SFR_E4M3 = 0, SFR_E5M2 = 1 } sfr_fp8_t;

/* Output formats of the linear layer.  SFR_OUT_F32 writes the binary32 value
 * before the final bf16 rounding (for accuracy checks). */
typedef enum { SFR_OUT_BF16 = 0, SFR_OUT_F32 = 1 } sfr_out_t;

/* Scale granularity of one operand of sparse_fp8_scaled_linear: one binary32
 * scale per row (per token for the activation, per output row for the
 * weight), or one for the whole operand. */
typedef enum { SFR_SCALE_ROW = 0, SFR_SCALE_TENSOR = 1 } sfr_scale_t;

typedef enum {
    SFR_OK = 0,
    SFR_ERR_NULL = 1,   /* a required pointer is NULL                         */
    SFR_ERR_SHAPE = 2,  /* a size is negative, too large or not a multiple    */
    SFR_ERR_ALIGN = 3,  /* a pointer is not 16-byte aligned                   */
    SFR_ERR_DTYPE = 4,  /* an enum argument is out of range                   */
    SFR_ERR_LAUNCH = 5  /* the HIP runtime rejected a kernel launch           */
} sfr_status;

/* Version of the compressed-weight layout described at compress_2to4_fp8. */
#define SFR_FORMAT_VERSION 1

/* Largest accepted row count / column count / K of any entry point. */
#define SFR_MAX_DIM ((int64_t)1 << 30)

/*
 * quantize_rowwise_fp8 -- dynamic row-wise FP8 quantization.
 * Source: PR #1671 (row-wise scaled FP8 activation, quantized dynamically;
 * FP16->FP8 quantization must not produce NaN) and pytorch/ao PR #1455
 * ("[float8nocompile] ... atomic_max-based algo ...", review thread: the split
 * reduction is worth keeping because it is deterministic).
 *
 * For every row r of x (bf16 bits, [rows, cols]):
 *     amax     = max_k |x[r, k]|                      (exact)
 *     scale[r] = fl32(amax / fmax)                    (IEEE binary32 division;
 *                                                      fmax 448 or 57344)
 *     q[r, k]  = sat_rne_fp8(fl32(x[r, k] / scale[r]))
 * sat_rne_fp8 rounds to nearest, ties to even, keeps the sign of zero, and
 * clamps magnitudes above fmax to fmax.  A row whose amax is 0 gets
 * scale 0 and codes 0x00 / 0x80 that keep each zero's sign.  The result is
 * deterministic and exact: the same bytes on every run and every launch shape.
 *
 *   x      [rows, cols] bf16 bits, device, read.
 *   dt     format of q.
 *   q      [rows, cols] FP8 bytes, device, written.
 *   scale  [rows] binary32, device, written.
 * Sizes: 0 <= rows <= SFR_MAX_DIM, 0 < cols <= SFR_MAX_DIM, cols % 8 == 0.
 * rows == 0 is a no-op; cols == 0 is rejected (SFR_ERR_SHAPE) because a row
 * without elements has no amax.
 */
sfr_status quantize_rowwise_fp8(const uint16_t* x, int64_t rows, int64_t cols, sfr_fp8_t dt,
                                uint8_t* q, float* scale, void* stream);

/*
 * quantize_tensorwise_fp8 -- dynamic tensor-wise FP8 quantization: the
 * quantization of quantize_rowwise_fp8 with one scale for the whole tensor
 * (as if the tensor were a single row of rows*cols elements).  Source:
 * pytorch/ao PR #1455 ("[float8nocompile] Add alternate Triton kernels for
 * FP8 conversion which use atomic_max-based algo instead of reduction-based
 * algo", review thread): tensor-wise FP8 conversion whose global amax must
 * stay a deterministic reduction.  Here it is computed in two launches --
 * per-block maxima written to fixed workspace slots, then every block of the
 * cast kernel reduces all slots itself -- with no atomics; the amax is an
 * exact integer maximum, so the result is bit-exact and deterministic.
 *
 *     amax     = max_{r,k} |x[r, k]|                   (exact)
 *     scale[0] = fl32(amax / fmax)                     (IEEE binary32 division)
 *     q[r, k]  = sat_rne_fp8(fl32(x[r, k] / scale[0]))
 * An all-zero tensor gets scale 0 and sign-keeping zero codes.
 *
 *   x          [rows, cols] bf16 bits, device, read.
 *   dt         format of q.
 *   q          [rows, cols] FP8 bytes, device, written.
 *   scale      [1] binary32, device, written.
 *   workspace  device scratch of at least workspace_bytes =
 *              sfr_quantize_tensorwise_workspace_bytes(rows, cols) bytes,
 *              owned by the caller, overwritten; calls that may run at the
 *              same time need distinct workspaces.
 * Sizes as quantize_rowwise_fp8.  rows == 0 is a no-op; a workspace smaller
 * than required is SFR_ERR_SHAPE.
 */
sfr_status quantize_tensorwise_fp8(const uint16_t* x, int64_t rows, int64_t cols, sfr_fp8_t dt,
                                   uint8_t* q, float* scale, void* workspace, int64_t workspace_bytes,
                                   void* stream);

/* Workspace bytes quantize_tensorwise_fp8 needs for a [rows, cols] tensor
 * (at most 4 KB); 0 for sizes it rejects. */
int64_t sfr_quantize_tensorwise_workspace_bytes(int64_t rows, int64_t cols);

/*
 * quantize_tensorwise_fp8_noalloc -- quantize_tensorwise_fp8 for callers that
 * cannot allocate device memory (code under HIP graph capture, tight serving
 * loops, harnesses that forbid allocation): no workspace argument, and the
 * call allocates nothing.  The workspace is the library's own 4 KB device
 * array, one copy per GPU, held until the process ends; its address is
 * looked up on the first call on each device.  Results are bit-identical to
 * quantize_tensorwise_fp8's.
 *
 * Every call on one GPU uses that GPU's array, which keeps the last call's
 * contents (each call writes every slot it reads before reading it).  Calls
 * that may overlap on one GPU (different streams, or host threads) race on
 * the array and must be serialized by the caller.
 *
 * Arguments, sizes and errors as quantize_tensorwise_fp8 without the
 * workspace; a size whose workspace would exceed the array is SFR_ERR_SHAPE
 * (no accepted size does), and a failed lookup of the array SFR_ERR_LAUNCH.
 */
sfr_status quantize_tensorwise_fp8_noalloc(const uint16_t* x, int64_t rows, int64_t cols, sfr_fp8_t dt,
                                           uint8_t* q, float* scale, void* stream);

/*
 * compress_2to4_fp8 -- 2:4 semi-structured compression of an FP8 matrix.
 * Source: PR #1671 (converter to the 2:4 sparse format; testing found that
 * the compressor must treat -0.0 as zero, the issue the PR works around in
 * `from_plain()` and fixes upstream).
 *
 * For every row n and every group g of four consecutive k (k = 4g .. 4g+3)
 * of w ([n, k] FP8 bytes), the two entries of largest magnitude are kept;
 * ties go to the lower index and +0 / -0 have equal (zero) magnitude.  With
 * i0 < i1 the kept positions:
 *     values[n, 2g]   = w[n, 4g + i0]     values[n, 2g+1] = w[n, 4g + i1]
 *     (a kept -0.0, byte 0x80, is stored as 0x00)
 *     meta[n, g / 2]  bits 4*(g%2) .. 4*(g%2)+3  =  i0 | (i1 << 2)
 * so a little-endian 32-bit word of meta holds the nibbles of eight
 * consecutive groups, even group in the low nibble (layout version
 * SFR_FORMAT_VERSION).  Magnitude order is the unsigned order of the low
 * seven bits, identical for e4m3 and e5m2; `dt` is validated and otherwise
 * does not change the result.  Output is bit-exact and deterministic.
 *
 *   w      [n, k] FP8 bytes, device, read.
 *   values [n, k/2] bytes, device, written.
 *   meta   [n, k/8] bytes, device, written.
 * Sizes: 0 <= n <= SFR_MAX_DIM, 0 < k <= SFR_MAX_DIM, k % 128 == 0.
 * n == 0 is a no-op.
 */
sfr_status compress_2to4_fp8(const uint8_t* w, int64_t n, int64_t k, sfr_fp8_t dt,
                             uint8_t* values, uint8_t* meta, void* stream);

/*
 * prune_2to4_bf16 -- 2:4 magnitude pruning of a bf16 matrix, the weight's
 * first preparation step (before FP8 quantization and compress_2to4_fp8).
 * Source: PR #1671 (the weight is 2:4 semi-structured sparse; zeros of
 * either sign count as zero, the -0.0 issue that PR fixes in the converter).
 *
 * For every row and every group of four consecutive k of w ([n, k] bf16
 * bits), the two entries of largest magnitude keep their bits and the other
 * two become +0.0 (0x0000); ties go to the lower index and +0.0 / -0.0 have
 * equal (zero) magnitude.  A row's largest magnitude always survives, so its
 * row-wise FP8 scale is the same before and after pruning.  Finite inputs
 * only.  Output is bit-exact and deterministic.
 *
 *   w    [n, k] bf16 bits, device, read.
 *   out  [n, k] bf16 bits, device, written; may be w (in place).
 * Sizes: 0 <= n <= SFR_MAX_DIM, 0 < k <= SFR_MAX_DIM, k % 8 == 0.
 * n == 0 is a no-op.
 */
sfr_status prune_2to4_bf16(const uint16_t* w, int64_t n, int64_t k, uint16_t* out, void* stream);

/*
 * sparse_fp8_rowwise_linear -- the row-wise scaled linear layer with a 2:4
 * sparse FP8 weight.  Source: PR #1671 (row-wise scaled linear operator for a
 * sparse FP8 weight and an FP8 activation, one instantiation per dtype pair,
 * issue #3516's file table).
 *
 *     acc[m, n] = sum_k xq[m, k] * wq[n, k]          (binary32-grade accumulation
 *                                                    of exact products, any order)
 *     y[m, n]   = acc[m, n] * (xs[m] * ws[n]) (+ bias[n])   (binary32)
 *     out[m, n] = bf16_rne(y[m, n])   or   y[m, n] with SFR_OUT_F32
 * wq is the weight that (values, meta) encode in the compress_2to4_fp8
 * layout.  Any accumulation order is a correct result; the library's order is
 * fixed, so repeated calls give identical bits.
 *
 *   xq     [m, k] FP8 bytes (format x_dt), device, read.
 *   xs     [m] binary32, device, read.
 *   values [n, k/2], meta [n, k/8]: compressed weight (format w_dt), device, read.
 *   ws     [n] binary32, device, read.
 *   bias   [n] bf16 bits, device, read; may be NULL (no bias).
 *   out    [m, n] bf16 bits (SFR_OUT_BF16) or binary32 (SFR_OUT_F32), device, written.
 * Sizes: 0 <= m <= SFR_MAX_DIM, 0 <= n <= SFR_MAX_DIM, n % 16 == 0,
 * 0 < k <= SFR_MAX_DIM, k % 128 == 0.  m == 0 or n == 0 is a no-op.
 */
sfr_status sparse_fp8_rowwise_linear(const uint8_t* xq, sfr_fp8_t x_dt, const float* xs,
                                     int64_t m, int64_t k,
                                     const uint8_t* values, const uint8_t* meta, sfr_fp8_t w_dt,
                                     const float* ws, int64_t n, const uint16_t* bias,
                                     void* out, sfr_out_t out_dt, void* stream);

/*
 * sparse_fp8_scaled_linear -- sparse_fp8_rowwise_linear with the scale
 * granularity of each operand chosen: xs_kind / ws_kind SFR_SCALE_ROW reads
 * xs[m] / ws[n] as above, SFR_SCALE_TENSOR reads the single xs[0] / ws[0] for
 * every row (the tensor-wise scaling of quantize_tensorwise_fp8).  Everything
 * else -- arguments, sizes, accumulation, epilogue, errors -- is as
 * sparse_fp8_rowwise_linear, which is this call with both kinds
 * SFR_SCALE_ROW.  An unknown kind is SFR_ERR_DTYPE.
 */
sfr_status sparse_fp8_scaled_linear(const uint8_t* xq, sfr_fp8_t x_dt, const float* xs,
                                    sfr_scale_t xs_kind, int64_t m, int64_t k,
                                    const uint8_t* values, const uint8_t* meta, sfr_fp8_t w_dt,
                                    const float* ws, sfr_scale_t ws_kind, int64_t n,
                                    const uint16_t* bias, void* out, sfr_out_t out_dt,
                                    void* stream);

/*
 * Accumulation.  The products xq * wq are exact in binary32 (at most 8
 * significant bits each).  By default the library widens the FP8 codes
 * exactly to bf16 in registers and multiplies them on gfx950's 16-bit sparse
 * matrix instruction, which adds each product 24 bits below the largest term
 * of the instruction (the running sum included) and truncates toward zero:
 * a binary32-grade sum, whose error is that of a binary32 sum with
 * truncation in place of rounding.  An algorithm id with
 * SFR_ALGO_ACC_F8 set (see below) runs the FP8 sparse matrix instruction
 * instead, at twice the instruction rate; that instruction adds the 64
 * products of one 128-k step 13 bits below the largest of them, so a product
 * under 2^-13 of the step's largest is dropped.  On dot products that cancel
 * heavily next to large products (outlier channels, short K) its error can
 * exceed the bound above.
 */

/*
 * sparse_fp8_rowwise_linear_dynamic -- the layer from the bf16 activation:
 * quantize_rowwise_fp8 of x into (xq, xs), then sparse_fp8_scaled_linear with
 * row activation scales.  Source: PR #1671, item 4 (the activation is
 * quantized dynamically, per call).  xq and xs receive exactly the bytes
 * quantize_rowwise_fp8 writes; out is as sparse_fp8_scaled_linear.
 *
 * For 1 to 4 activation rows with k a multiple of 1024, both steps run in
 * ONE launch where that is faster: every workgroup quantizes the rows itself
 * (no workgroup waits for another), so the redundant work grows with rows x
 * workgroups.  One launch is taken for 1 or 2 rows with k up to 4096, or up
 * to 16384 while n / 16 does not exceed the device's CU count; for 3 or 4
 * rows with k up to 4096 and n / 16 at most the CU count.  Other shapes
 * take two launches (quantization, then the linear layer).  Both paths write
 * the same bytes.
 *
 *   x      [m, k] bf16 bits, device, read.
 *   xq     [m, k] FP8 bytes (format x_dt), device, written.
 *   xs     [m] binary32, device, written.
 * Other arguments, sizes and errors as sparse_fp8_scaled_linear (ws_kind
 * selects row or tensor weight scales).
 */
sfr_status sparse_fp8_rowwise_linear_dynamic(const uint16_t* x, sfr_fp8_t x_dt, int64_t m, int64_t k,
                                             const uint8_t* values, const uint8_t* meta, sfr_fp8_t w_dt,
                                             const float* ws, sfr_scale_t ws_kind, int64_t n,
                                             const uint16_t* bias, void* out, sfr_out_t out_dt,
                                             uint8_t* xq, float* xs, void* stream);

/*
 * sparse_fp8_rowwise_linear_dynamic_algo -- sparse_fp8_rowwise_linear_dynamic
 * with the linear layer's algorithm id given (SFR_ALGO_DEFAULT = the built-in
 * choice; ids as for sparse_fp8_scaled_linear_algo below).  The single-launch
 * path runs when the id's kernel configuration is the built-in one for the
 * shape; the accumulation follows the id.  Errors as
 * sparse_fp8_scaled_linear_algo.
 */
sfr_status sparse_fp8_rowwise_linear_dynamic_algo(const uint16_t* x, sfr_fp8_t x_dt, int64_t m, int64_t k,
                                                  const uint8_t* values, const uint8_t* meta, sfr_fp8_t w_dt,
                                                  const float* ws, sfr_scale_t ws_kind, int64_t n,
                                                  const uint16_t* bias, void* out, sfr_out_t out_dt,
                                                  uint8_t* xq, float* xs, int algo, void* stream);

/*
 * Kernel configurations ("algorithms") of the linear layer, and the choice
 * among them.  Source: pytorch/ao PR #4432 ("Add algorithm search to FP8
 * sparse linear benchmark": the best kernel configuration depends on the
 * shape, so it is searched per shape) and PR #1671 (remaining tasks: a
 * meaningful config selection).  Every algorithm computes the same function
 * (same result rules; the order of the binary32 sum differs between them).
 *
 * An algorithm id is a kernel configuration (low 8 bits) optionally or-ed
 * with SFR_ALGO_ACC_F8 (FP8 matrix-instruction accumulation, see
 * "Accumulation" above); without the flag the accumulation is binary32-grade.
 *
 *   sfr_linear_algo_count()      number of kernel configurations (ids
 *                                0 .. count-1, each with or without the flag).
 *   sfr_linear_algo_valid(a)     1 if a names an algorithm, else 0.
 *   sfr_linear_algo_name(a)      static name (configurations with the flag
 *                                end in "+f8acc"), NULL for an unknown id.
 *   sfr_linear_algo_supported(a, m, n, k)
 *                                1 if algorithm a can run the shape, else 0.
 *   sfr_linear_default_algo(m, n, k)
 *                                the library's built-in choice for the shape
 *                                on the current device (it counts rounds of
 *                                tiles over the device's compute units, so it
 *                                can differ between GPUs; 256 units are
 *                                assumed when no device is present).
 *   sparse_fp8_scaled_linear_algo(..., algo, stream)
 *                                sparse_fp8_scaled_linear with the given
 *                                algorithm; SFR_ALGO_DEFAULT (-1) = built-in
 *                                choice.  An unknown id is SFR_ERR_DTYPE; an
 *                                algorithm that cannot run the shape is
 *                                SFR_ERR_SHAPE.
 * Configurations: 0 decode_lds (m <= 64, k % 1024 == 0), 1 decode_reg
 * (m <= 16), 2 tiled_64x64, 3 tiled_128x128, 4 tiled_256x256,
 * 5 wide_256x256 (k >= 512, only with SFR_ALGO_ACC_F8), 6 decode_lds_32
 * (m <= 64, k % 1024 == 0, n % 32 == 0), 7 tiled_256x128 (tiles of 256
 * output columns n by 128 rows m).
 */
#define SFR_ALGO_DEFAULT (-1)
#define SFR_ALGO_ACC_F8 0x100
int sfr_linear_algo_count(void);
int sfr_linear_algo_valid(int algo);
const char* sfr_linear_algo_name(int algo);
int sfr_linear_algo_supported(int algo, int64_t m, int64_t n, int64_t k);
int sfr_linear_default_algo(int64_t m, int64_t n, int64_t k);
sfr_status sparse_fp8_scaled_linear_algo(const uint8_t* xq, sfr_fp8_t x_dt, const float* xs,
                                         sfr_scale_t xs_kind, int64_t m, int64_t k,
                                         const uint8_t* values, const uint8_t* meta, sfr_fp8_t w_dt,
                                         const float* ws, sfr_scale_t ws_kind, int64_t n,
                                         const uint16_t* bias, void* out, sfr_out_t out_dt, int algo,
                                         void* stream);

/*
 * Block-sparse (BSR) bf16 weight and its linear layer.
 * Source: pytorch/ao PR #1734 ("promote blocksparse from prototype, make it
 * faster"): the weight is stored in blocks of 64 x 64, most of them zero
 * (its measurements use sparsity level 0.9), and multiplied by a dense
 * activation whose row count is padded to 16 for decode.  The page names no
 * number format; here weight, activation and output are bf16, the sum is
 * binary32 (every bf16 product is exact in it), the result rounded once to
 * bf16 (nearest, ties to even) or returned in binary32.
 *
 * Layout (compressed-sparse-row over blocks, as torch's BSR tensors):
 *   crow   int32 [n/64 + 1]: crow[0] = 0, crow[i+1] - crow[i] = kept blocks of
 *          block row i (rows 64 i .. 64 i + 63); nnz = crow[n/64].
 *   col    int32 [nnz]: block column of each kept block, ascending within a
 *          block row.
 *   values bf16 bits [nnz][64][64]: each kept block, row-major.
 * A block is kept when any element is non-zero by value (+0.0 and -0.0 are
 * zero; NaN, infinities and subnormals are non-zero).
 *
 * bsr_count_bf16(w, n, k, crow, stream): two launches write crow for the
 *   dense bf16 w [n, k] (row-major, 16-byte aligned).  The caller reads
 *   crow[n/64] (nnz) to size col and values.
 * bsr_fill_bf16(w, n, k, crow, col, values, stream): writes col and values
 *   for the crow that bsr_count_bf16 wrote for the same w.  col and values
 *   may be NULL only when nnz = 0.
 * bsr_linear_bf16(x, m, k, crow, col, values, n, bias, out, out_dt, stream):
 *   out[m, n] = sum_k x[i, k] W[j, k] (+ bias[j]) for bf16 x [m, k]
 *   (row-major), the BSR weight W [n, k] and optional bf16 bias [n]; out is
 *   bf16 or binary32 [m, n], row-major.  Deterministic (fixed summation
 *   order).  Every block column index is clamped to the matrix, but crow and
 *   the values array must be the ones bsr_count_bf16 / bsr_fill_bf16 wrote
 *   (they are read as given).
 * Sizes: 0 <= n, m <= SFR_MAX_DIM; 0 < k <= SFR_MAX_DIM; n % 64 == 0,
 * k % 64 == 0.  Alignment: w, x, values, bias, out 16 bytes; crow, col 4.
 * Errors: SFR_ERR_SHAPE, SFR_ERR_NULL, SFR_ERR_ALIGN, SFR_ERR_DTYPE (out_dt),
 * SFR_ERR_LAUNCH.  All pointers are device memory owned by the caller; the
 * calls are asynchronous on `stream` (NULL = the default stream).
 */
#define SFR_BSR_BLOCK 64
sfr_status bsr_count_bf16(const uint16_t* w, int64_t n, int64_t k, int32_t* crow, void* stream);
sfr_status bsr_fill_bf16(const uint16_t* w, int64_t n, int64_t k, const int32_t* crow, int32_t* col,
                         uint16_t* values, void* stream);
sfr_status bsr_linear_bf16(const uint16_t* x, int64_t m, int64_t k, const int32_t* crow, const int32_t* col,
                           const uint16_t* values, int64_t n, const uint16_t* bias, void* out, sfr_out_t out_dt,
                           void* stream);

/*
 * ---------------------------------------------------------------------------
 * The gated feed-forward block and its 8-bit and 4-bit forms.
 *
 *     h[m, j] = act(sum_k x[m, k] w[j, k]) * sum_k x[m, k] w[f + j, k]
 *
 * for bf16 x [m, k] and one weight w [2 f, k] whose first f rows are the gate
 * projection and last f rows the up projection.  Activations saved for the
 * backward pass, and weights for decoding, may be held in MX block formats
 * (OCP Microscaling Formats v1.0: blocks of 32 values along a row share one
 * power-of-two scale, a byte E8M0), which gfx950 converts in hardware.
 *
 * Unlike the FP8 entry points above, these carry NaN and infinities through as
 * binary32 arithmetic does (an MX block that holds one decodes to NaN).
 *
 * Sizes: 0 <= m <= SFR_MAX_DIM; 0 < k, 2 f, n <= SFR_MAX_BLOCK_DIM; k % 32 == 0,
 * f % 32 == 0, n % 16 == 0; a call one of whose products has more than 2^21 tiles
 * of 128 x 128 outputs (64 x 64 up to 64 rows) is SFR_ERR_SHAPE.  Results do not depend on anything
 * but the arguments: the order of every sum is fixed, no atomics.
 * ---------------------------------------------------------------------------
 */
#define SFR_MAX_BLOCK_DIM ((int64_t)1 << 20)
#define SFR_MX_BLOCK 32

/* Element formats of the MX blocks.  E2M1 (4 bits: 0, .5, 1, 1.5, 2, 3, 4, 6 and
 * their negatives) packs two values a byte, the even column in the low half. */
typedef enum { SFR_MX_E4M3 = 0, SFR_MX_E5M2 = 1, SFR_MX_E2M1 = 2 } sfr_mx_t;

/* Activation of the gated block: x s(x), the tanh form of GELU, max(x, 0).  The
 * logistic factor s may be 0 where it lies below 2^-126 (SiLU: x < -87.3). */
typedef enum { SFR_ACT_SILU = 0, SFR_ACT_GELU_TANH = 1, SFR_ACT_RELU = 2 } sfr_act_t;

/* How an activation is saved for the backward pass. */
typedef enum { SFR_SAVE_NONE = 0, SFR_SAVE_BF16 = 1, SFR_SAVE_E4M3 = 2, SFR_SAVE_E5M2 = 3 } sfr_save_t;

/*
 * quantize_mx / dequantize_mx -- bf16 rows to MX blocks and back.
 * For every block b of 32 columns of every row (fmax = 448, 57344 or 6):
 *     amax        = max |x|                              (exact)
 *     scale[r, b] = e + 127, e the smallest whole number >= -110 with
 *                   amax <= fmax * 2^e                   (17 for a zero block)
 *     q           = rne(x * 2^-e)                        (sign of zero kept; an
 *                   element that would stand for 2^128 is the one below)
 * A block with a NaN or an infinity gets scale 255 and zero codes.
 * dequantize_mx writes q * 2^e, exactly (every such value is a bf16 number),
 * and NaN for a block of scale 255.  Deterministic, bit-exact.
 * Blocks from elsewhere may have any scale byte s and element code: one stands
 * for q * 2^(s - 127), rounded to the nearest bf16 number, ties to even (inexact
 * only for e4m3 elements below s = 3 and e5m2 elements below s = 10, which reach
 * under bf16's smallest step; infinite from 2^128 on), NaN and infinity codes
 * for themselves.  Every call that reads MX blocks takes them so.
 *
 *   x, out  [rows, cols] bf16 bits.
 *   q       [rows, cols] bytes, or [rows, cols / 2] for SFR_MX_E2M1.
 *   scale   [rows, cols / 32] bytes.
 * Sizes: 0 <= rows <= SFR_MAX_DIM, 0 < cols <= SFR_MAX_DIM, cols % 32 == 0.
 * rows == 0 is a no-op.
 */
sfr_status quantize_mx(const uint16_t* x, int64_t rows, int64_t cols, sfr_mx_t dt, uint8_t* q, uint8_t* scale,
                       void* stream);
sfr_status dequantize_mx(const uint8_t* q, const uint8_t* scale, int64_t rows, int64_t cols, sfr_mx_t dt,
                         uint16_t* out, void* stream);

/*
 * gated_linear_bf16 -- the gated block's forward pass in one launch: both
 * projections accumulate in binary32, h is formed from the unrounded sums g, u
 * and rounded once to bf16.  With a checkpoint, [g | u] is written as well:
 * bf16 values, or MX blocks quantized from the binary32 sums by the rule of
 * quantize_mx.
 *
 *   x        [m, k], w [2 f, k], h [m, f]: bf16 bits.
 *   save     SFR_SAVE_NONE: gu and gu_scale are not used (NULL).
 *   gu       [m, 2 f] bf16 bits (SFR_SAVE_BF16) or bytes (SFR_SAVE_E4M3 / _E5M2).
 *   gu_scale [m, 2 f / 32] bytes for the 8-bit forms, else not used.
 * m == 0 is a no-op.
 */
sfr_status gated_linear_bf16(const uint16_t* x, int64_t m, int64_t k, const uint16_t* w, int64_t f, sfr_act_t act,
                             uint16_t* h, sfr_save_t save, void* gu, uint8_t* gu_scale, void* stream);

/*
 * gated_linear_bf16_backward -- its gradients, from the saved [g | u] and x:
 *     dg = dh * u * act'(g),  du = dh * act(g)        (binary32, rounded to bf16)
 *     dx[m, k] = sum_j dg[m, j] w[j, k] + du[m, j] w[f + j, k]
 *     dw[j, k] = sum_m dg[m, j] x[m, k],  dw[f + j, k] = sum_m du[m, j] x[m, k]
 * (binary32 sums, rounded once to bf16).  relu' is 1 above 0 and 0 elsewhere, at
 * NaN too.  The rounding of dg and du, which the matrix instructions read in
 * bf16, makes the gradients' relative error 0.0024 (root mean square) where
 * the last rounding alone would leave 0.0017.
 *
 *   dh        [m, f] bf16 bits.
 *   gu, gu_scale, gu_save   as gated_linear_bf16 wrote them.
 *   x, x_scale, x_save      [m, k]: bf16 bits (SFR_SAVE_BF16, x_scale not used)
 *                           or quantize_mx's codes and scales.
 *   dx [m, k], dw [2 f, k]  bf16 bits, written; either may be NULL (not computed;
 *                           x is not read without dw, w not without dx).
 *   workspace  device scratch of at least sfr_gated_backward_workspace_bytes(
 *              m, k, f, x_save) bytes, overwritten; calls that may run at the
 *              same time need distinct workspaces.
 * m == 0 writes zeros to dw.  SFR_SAVE_NONE is SFR_ERR_DTYPE; a small
 * workspace is SFR_ERR_SHAPE.
 */
sfr_status gated_linear_bf16_backward(const uint16_t* dh, int64_t m, int64_t k, int64_t f, sfr_act_t act,
                                      const void* gu, const uint8_t* gu_scale, sfr_save_t gu_save, const void* x,
                                      const uint8_t* x_scale, sfr_save_t x_save, const uint16_t* w, uint16_t* dx,
                                      uint16_t* dw, void* workspace, int64_t workspace_bytes, void* stream);

/* Workspace bytes of gated_linear_bf16_backward; 0 for sizes it rejects. */
int64_t sfr_gated_backward_workspace_bytes(int64_t m, int64_t k, int64_t f, sfr_save_t x_save);

/*
 * mxfp4_linear -- the linear layer for a 4-bit weight with one scale per 32
 * values, as quantize_mx(SFR_MX_E2M1) writes it:
 *     out[m, n] = sum_k x[m, k] wq[n, k] (+ bias[n])
 * The weight's values are exact in bf16 (those of 2^128 and more, scale bytes
 * 253 and 254, are infinities); sums are binary32, rounded once to bf16 or
 * returned in binary32.
 * mxfp4_gated_linear -- the gated block for such a weight [2 f, k]; h bf16.
 *
 *   x   [m, k] bf16 bits.
 *   wq  [n, k / 2] (gated [2 f, k / 2]) bytes, ws [n, k / 32] bytes.
 *   bias [n] bf16 bits or NULL;  out [m, n] bf16 bits or binary32;  h [m, f].
 *   workspace  device scratch of at least sfr_mxfp4_workspace_bytes(m, n, k)
 *              bytes (0 for many sizes; then it may be NULL), overwritten; calls
 *              that may run at the same time need distinct workspaces.
 * m == 0 or n == 0 is a no-op; a small workspace is SFR_ERR_SHAPE.
 */
sfr_status mxfp4_linear(const uint16_t* x, int64_t m, int64_t k, const uint8_t* wq, const uint8_t* ws, int64_t n,
                        const uint16_t* bias, void* out, sfr_out_t out_dt, void* workspace, int64_t workspace_bytes,
                        void* stream);
sfr_status mxfp4_gated_linear(const uint16_t* x, int64_t m, int64_t k, const uint8_t* wq, const uint8_t* ws, int64_t f,
                              sfr_act_t act, uint16_t* h, void* stream);

/* Workspace bytes of mxfp4_linear; 0 for sizes it rejects. */
int64_t sfr_mxfp4_workspace_bytes(int64_t m, int64_t n, int64_t k);

/* The matrix products of the calls above, by what decides their kernel: the
 * forward pass without and with a checkpoint, dx, dw, and the two 4-bit calls. */
typedef enum {
    SFR_PRODUCT_GATED = 0,
    SFR_PRODUCT_GATED_SAVING = 1,
    SFR_PRODUCT_DX = 2,
    SFR_PRODUCT_DW = 3,
    SFR_PRODUCT_MXFP4 = 4,
    SFR_PRODUCT_MXFP4_GATED = 5
} sfr_product_t;

/*
 * sfr_block_kernel -- name of the kernel that a product takes (a static string;
 * for profiles and tests), NULL for sizes its call rejects and for a call
 * without rows.  f: n for SFR_PRODUCT_MXFP4.  slices (may be NULL) receives the
 * number of slices of its sum, 1 for an unsliced one.
 */
const char* sfr_block_kernel(sfr_product_t product, int64_t m, int64_t k, int64_t f, int32_t* slices);

/* Human-readable name of a status code (static string, never NULL). */
const char* sfr_status_string(sfr_status s);

/* The compressed-weight layout version this library reads and writes. */
int sfr_format_version(void);

#ifdef __cplusplus
}
#endif

#endif /* SPARSE_FP8_ROW_H */

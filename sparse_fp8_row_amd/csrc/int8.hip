// The linear layer in 8-bit integers with one scale per activation row and
// weight row: the row quantizer, and which kernels a call runs.
//
//     q = rne(127 x / amax),  scale = amax / 127         (a row at a time)
//     out[m, n] = xs[m] ws[n] sum_k xq[m, k] wq[n, k]  (+ bias[n])
//
// The sum is exact (32-bit integers on v_mfma_i32_16x16x64_i8; the entry points
// bound k), so no kernel, tile or slicing changes a result.
#include "sfr_launch.hpp"
#include "sfr_quant.hpp"

namespace sfr {
namespace {

// Codes of a row are those of the exact quotient 127 x / amax.  With x = a 2^p
// and amax = b 2^q (a, b whole, under 2^8) the quotient is a half-integer
// exactly or at least 2^-16 of itself away from one, so a quotient within 2^-20
// that is exact on half-integers decides every code.  Here it is one binary32
// product by the reciprocal, corrected once: t = t0 + r y with r = 127 x - t0 amax
// exact.  Where the true quotient t* is a half-integer the correction leaves
// |r| 2^-23, below half a step of t*, so t* is returned.  Rows are taken by the
// exponent of amax (x 2^-e, amax 2^-e in [1, 2)), so nothing over- or underflows
// that could reach code 1.
struct RowScale {
  float an, y;  // amax 2^-e and its reciprocal
  int e;
  bool live;  // false: a row of zeros, or one that is not finite
};

__device__ __forceinline__ RowScale row_scale(uint32_t amax_bits) {
  RowScale s;
  const float amax = bf16_to_f32(amax_bits);
  s.live = amax_bits != 0 && amax_bits < 0x7F80u;
  s.e = s.live ? __builtin_amdgcn_frexp_expf(amax) - 1 : 0;
  s.an = s.live ? ldexpf(amax, -s.e) : 1.0f;
  s.y = 1.0f / s.an;
  return s;
}

// The row's scale: 0 for zeros, NaN for a row that holds a NaN or an infinity.
__device__ __forceinline__ float scale_value(uint32_t amax_bits) {
  return amax_bits < 0x7F80u ? bf16_to_f32(amax_bits) / 127.0f : __builtin_nanf("");
}

// Low byte of the result: the code.  Adding 1.5 * 2^23 rounds to a whole number,
// ties to even, and leaves it in the low bits.
__device__ __forceinline__ uint32_t code(uint32_t bf16, const RowScale& s) {
  const float a = 127.0f * ldexpf(bf16_to_f32(bf16), -s.e);
  const float t0 = a * s.y;
  const float t = __builtin_fmaf(__builtin_fmaf(-t0, s.an, a), s.y, t0);
  return __float_as_uint(t + 12582912.0f);
}

__device__ __forceinline__ uint2 cast8_int8(const uint4& c, const RowScale& s) {
  if (!s.live) return make_uint2(0, 0);
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
  uint32_t pair[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    pair[i] = __builtin_amdgcn_perm(code(w[i] >> 16, s), code(w[i] & 0xFFFFu, s), 0x0C0C0400u);
  return make_uint2(pair[0] | pair[1] << 16, pair[2] | pair[3] << 16);
}

// One wavefront (BLOCK false, four rows a workgroup) or one workgroup of NT
// threads per row.  A thread's first CPT chunks of eight values stay in
// registers between the sweeps for the maximum and for the codes; what a longer
// row has beyond them is read again (from the caches).
template <int CPT, int NT, bool BLOCK>
__global__ __launch_bounds__(NT) void quantize_int8_kernel(const uint16_t* __restrict__ x, int64_t rows, int cols,
                                                           int8_t* __restrict__ q, float* __restrict__ scale) {
  constexpr int T = BLOCK ? NT : 64;  // threads of a row
  const int tid = BLOCK ? threadIdx.x : threadIdx.x & 63;
  const int64_t row = BLOCK ? blockIdx.x : (int64_t)blockIdx.x * (NT / 64) + (threadIdx.x >> 6);
  if (row >= rows) return;
  const int chunks = cols >> 3;
  const uint4* const xr = reinterpret_cast<const uint4*>(x + row * cols);
  uint2* const qr = reinterpret_cast<uint2*>(q + row * cols);
  uint4 held[CPT];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < CPT; ++i) {
    const int c = tid + T * i;
    held[i] = c < chunks ? xr[c] : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < CPT; ++i) m = mag_max8(held[i], m);
  for (int c = tid + T * CPT; c < chunks; c += T) m = mag_max8(xr[c], m);
  m = wave_max(m);
  if constexpr (BLOCK) {
    __shared__ uint32_t red[NT / 64];
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
    __syncthreads();
    m = red[0];
#pragma unroll
    for (int w = 1; w < NT / 64; ++w) m = max(m, red[w]);
  }
  const RowScale s = row_scale(m);
  if (tid == 0) scale[row] = scale_value(m);
#pragma unroll
  for (int i = 0; i < CPT; ++i) {
    const int c = tid + T * i;
    if (c < chunks) qr[c] = cast8_int8(held[i], s);
  }
  for (int c = tid + T * CPT; c < chunks; c += T) qr[c] = cast8_int8(xr[c], s);
}

int64_t align256(int64_t b) { return (b + 255) / 256 * 256; }

StreamArgs stream_args(const Int8Args& a) {
  StreamArgs s{};
  s.x = reinterpret_cast<const uint16_t*>(a.xq);
  s.w = a.wq;
  s.m = a.m;
  s.k = a.k;
  s.rows = a.n;
  s.bias = a.bias;
  s.out = a.out;
  s.out_fmt = a.out_fmt;
  s.xs = a.xs;
  s.ws = a.ws;
  return s;
}

}  // namespace

hipError_t launch_quantize_int8(const uint16_t* x, int64_t rows, int64_t cols, int8_t* q, float* scale,
                                hipStream_t stream) {
  const int c = (int)cols;
  if (rows < 1024) {
    const dim3 grid((unsigned)rows);
    if (cols <= 2048) quantize_int8_kernel<1, 256, true><<<grid, dim3(256), 0, stream>>>(x, rows, c, q, scale);
    else if (cols <= 8192) quantize_int8_kernel<2, 512, true><<<grid, dim3(512), 0, stream>>>(x, rows, c, q, scale);
    else quantize_int8_kernel<2, 1024, true><<<grid, dim3(1024), 0, stream>>>(x, rows, c, q, scale);
    return hipGetLastError();
  }
  const dim3 grid((unsigned)((rows + 3) / 4)), block(256);
  if (cols <= 2048) quantize_int8_kernel<4, 256, false><<<grid, block, 0, stream>>>(x, rows, c, q, scale);
  else if (cols <= 4096) quantize_int8_kernel<8, 256, false><<<grid, block, 0, stream>>>(x, rows, c, q, scale);
  else quantize_int8_kernel<16, 256, false><<<grid, block, 0, stream>>>(x, rows, c, q, scale);
  return hipGetLastError();
}

// Workspace: the partial sums of a sliced product; of a bf16 x its codes and scales.
int64_t int8_workspace_bytes(int64_t m, int64_t n, int64_t k, bool dynamic) {
  return (stream_rows_int8(m, n, k) ? 0 : align256(dense_int8_workspace_bytes(m, n, k))) +
         (dynamic ? align256(m * k) + align256(4 * m) : 0);
}

hipError_t launch_int8(const Int8Args& args, void* workspace, hipStream_t stream) {
  Int8Args a = args;
  uint8_t* at = static_cast<uint8_t*>(workspace);
  if (a.x) {
    int8_t* const q = reinterpret_cast<int8_t*>(at);
    float* const scale = reinterpret_cast<float*>(at + align256(a.m * a.k));
    at += align256(a.m * a.k) + align256(4 * a.m);
    const hipError_t e = launch_quantize_int8(a.x, a.m, a.k, q, scale, stream);
    if (e != hipSuccess) return e;
    a.xq = q;
    a.xs = scale;
  }
  if (stream_rows_int8(a.m, a.n, a.k)) return launch_stream(stream_args(a), stream);
  return launch_int8_dense(a, at, stream);
}

DenseKernel int8_kernel(int64_t m, int64_t n, int64_t k, bool dynamic) {
  if (!stream_rows_int8(m, n, k)) return dense_int8_kernel(m, n, k);
  static const float some = 0;  // ws: tells this product from the others, not read
  Int8Args a{};
  a.ws = &some;
  a.m = m;
  a.n = n;
  a.k = k;
  return {stream_name(stream_args(a)), 1};
}

}  // namespace sfr

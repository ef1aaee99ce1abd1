// MX block formats on gfx950: quantization of bf16 rows to FP8 (e4m3, e5m2) or
// 4-bit (e2m1) elements with one power-of-two scale per 32 values, and back.
//
// One pass over the data, memory bound: 2 bytes read and 33/32 (FP8) or 17/32
// (e2m1) written per value, and the reverse.  A row is a whole number of
// blocks and rows are contiguous, so the tensor is one run of blocks: a lane
// holds 8 values (a 16-byte load), four lanes a block, and the block's maximum
// is two lane exchanges inside those four.
#include "sfr_launch.hpp"
#include "sfr_mx.hpp"

namespace sfr {
namespace {

constexpr int kThreads = 256;
// Chunks of 8 values per lane: loads in flight per wavefront (4 x 1 KB).
constexpr int kChunks = 4;

template <int FMT>
__global__ __launch_bounds__(kThreads) void quantize_mx_kernel(const uint4* __restrict__ x, int64_t chunks,
                                                               uint8_t* __restrict__ q, uint8_t* __restrict__ scale) {
  const int64_t base = (int64_t)blockIdx.x * (kThreads * kChunks) + threadIdx.x;
  uint4 c[kChunks];
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    const int64_t at = base + i * kThreads;
    c[i] = at < chunks ? x[at] : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    const int64_t at = base + i * kThreads;
    const uint32_t w[4] = {c[i].x, c[i].y, c[i].z, c[i].w};
    uint32_t a = 0;  // |bf16| order is the unsigned order of the low 15 bits, NaN above infinity
#pragma unroll
    for (int j = 0; j < 4; ++j) a = max(a, max(w[j] & 0x7FFFu, (w[j] >> 16) & 0x7FFFu));
    a = max(a, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)a, 0xB1, 0xF, 0xF, false));  // quad lanes 1,0,3,2
    a = max(a, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)a, 0x4E, 0xF, 0xF, false));  // quad lanes 2,3,0,1
    const int code = mx_scale_code<FMT>(a << 16);
    const float inv = mx_inverse(code), limit = mx_limit<FMT>(code);
    float v[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      v[2 * j] = mx_scaled(bf16_to_f32(w[j] & 0xFFFFu), inv, limit);
      v[2 * j + 1] = mx_scaled(bf16_to_f32(w[j] >> 16), inv, limit);
    }
    if (at < chunks) {
      if constexpr (FMT == MX_E2M1) {
        reinterpret_cast<uint32_t*>(q)[at] = mx_pack8_e2m1(v);
      } else {
        reinterpret_cast<uint2*>(q)[at] =
            make_uint2(mx_pack4<FMT>(v[0], v[1], v[2], v[3]), mx_pack4<FMT>(v[4], v[5], v[6], v[7]));
      }
      if ((threadIdx.x & 3) == 0) scale[at >> 2] = (uint8_t)code;
    }
  }
}

template <int FMT>
__global__ __launch_bounds__(kThreads) void dequantize_mx_kernel(const uint8_t* __restrict__ q,
                                                                 const uint8_t* __restrict__ scale, int64_t chunks,
                                                                 uint4* __restrict__ out) {
  const int64_t base = (int64_t)blockIdx.x * (kThreads * kChunks) + threadIdx.x;
  uint2 c[kChunks];
  uint32_t s[kChunks];
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    const int64_t at = base + i * kThreads;
    c[i] = make_uint2(0, 0);
    s[i] = 0;
    if (at < chunks) {
      if constexpr (FMT == MX_E2M1) c[i].x = reinterpret_cast<const uint32_t*>(q)[at];
      else c[i] = reinterpret_cast<const uint2*>(q)[at];
      s[i] = scale[at >> 2];
    }
  }
#pragma unroll
  for (int i = 0; i < kChunks; ++i) {
    const int64_t at = base + i * kThreads;
    uint4 v;
    if constexpr (FMT == MX_E2M1) v = mx_widen8_e2m1(c[i].x, mx_scale_value(s[i]));
    else v = mx_widen8_fp8<FMT>(c[i], s[i]);
    if (at < chunks) out[at] = v;
  }
}

unsigned blocks_of(int64_t chunks) { return (unsigned)((chunks + kThreads * kChunks - 1) / (kThreads * kChunks)); }

}  // namespace

hipError_t launch_quantize_mx(const uint16_t* x, int64_t rows, int64_t cols, int fmt, uint8_t* q, uint8_t* scale,
                              hipStream_t stream) {
  const int64_t chunks = rows * (cols / 8);
  const uint4* in = reinterpret_cast<const uint4*>(x);
  const dim3 grid(blocks_of(chunks)), block(kThreads);
  if (fmt == MX_E4M3) quantize_mx_kernel<MX_E4M3><<<grid, block, 0, stream>>>(in, chunks, q, scale);
  else if (fmt == MX_E5M2) quantize_mx_kernel<MX_E5M2><<<grid, block, 0, stream>>>(in, chunks, q, scale);
  else quantize_mx_kernel<MX_E2M1><<<grid, block, 0, stream>>>(in, chunks, q, scale);
  return hipGetLastError();
}

hipError_t launch_dequantize_mx(const uint8_t* q, const uint8_t* scale, int64_t rows, int64_t cols, int fmt,
                                uint16_t* out, hipStream_t stream) {
  const int64_t chunks = rows * (cols / 8);
  uint4* o = reinterpret_cast<uint4*>(out);
  const dim3 grid(blocks_of(chunks)), block(kThreads);
  if (fmt == MX_E4M3) dequantize_mx_kernel<MX_E4M3><<<grid, block, 0, stream>>>(q, scale, chunks, o);
  else if (fmt == MX_E5M2) dequantize_mx_kernel<MX_E5M2><<<grid, block, 0, stream>>>(q, scale, chunks, o);
  else dequantize_mx_kernel<MX_E2M1><<<grid, block, 0, stream>>>(q, scale, chunks, o);
  return hipGetLastError();
}

}  // namespace sfr

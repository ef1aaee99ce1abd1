// The gated feed-forward block h = act(x Wg^T) * (x Wu^T): which kernels its
// forward and backward calls run, and the elementwise part of the gradients.
#include "sfr_launch.hpp"
#include "sfr_mx.hpp"

namespace sfr {
namespace {

// Eight saved values (bf16, or FP8 with their scale) as bf16.
template <int FMT>
__device__ __forceinline__ uint4 load_saved8(const void* p, const uint8_t* scale, int64_t at) {
  if constexpr (FMT == GU_BF16) {
    return *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + at);
  } else {
    constexpr int F = FMT == GU_E4M3 ? MX_E4M3 : MX_E5M2;
    return mx_widen8_fp8<F>(*reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(p) + at), scale[at / MX_BLOCK]);
  }
}

__device__ __forceinline__ void unpack8(const uint4& c, float (&v)[8]) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_to_f32(w[i] & 0xFFFFu);
    v[2 * i + 1] = bf16_to_f32(w[i] >> 16);
  }
}

struct GradParams {
  const uint4* dh;
  const void* gu;
  const uint8_t* gu_scale;
  uint4* dgu;
  int64_t m;
  int f8;  // f / 8
  // an 8-bit x to decode to bf16 for dW (0 chunks: none)
  const void* x;
  const uint8_t* x_scale;
  uint4* x_out;
  int64_t x_chunks;  // of 8 values
  int x_fmt;
};

// dgu[m] = [dh u act'(g) | dh act(g)] from the saved g and u: one pass, memory
// bound (per f: 2 bytes of dh, two saved values, 4 bytes written; 6.1 TB/s at m =
// 8192, f = 14336).  A lane holds 8 f.  The gradients are formed in binary32
// and rounded once to bf16, the type in which the two products read them: more
// bits would take a second pair of products (of what the rounding left), twice
// the time at the matrix cores' bound, to lower dx's and dw's relative error
// from 0.0024 to the 0.0017 of their own rounding.  An
// 8-bit x is decoded by the same threads first (a launch of its own cost the
// host 3 of a small call's 22 us; workgroups of their own 20 us at m = 8192).
template <int FMT, int ACT>
__global__ __launch_bounds__(256) void gated_grad_kernel(GradParams p) {
  const int64_t step = (int64_t)gridDim.x * gridDim.y * 256;
  for (int64_t i = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 256 + threadIdx.x; i < p.x_chunks; i += step)
    p.x_out[i] = p.x_fmt == GU_E4M3 ? load_saved8<GU_E4M3>(p.x, p.x_scale, i * 8)
                                    : load_saved8<GU_E5M2>(p.x, p.x_scale, i * 8);
  const int f8 = p.f8, c = blockIdx.x * 256 + threadIdx.x;
  if (c >= f8) return;
  for (int64_t r = blockIdx.y; r < p.m; r += gridDim.y) {
    float d[8], g[8], u[8], og[8], ou[8];
    const int64_t at = (2 * r * f8 + c) * 8;
    const uint4 d4 = p.dh[r * f8 + c], g4 = load_saved8<FMT>(p.gu, p.gu_scale, at),
                u4 = load_saved8<FMT>(p.gu, p.gu_scale, at + (int64_t)f8 * 8);
    unpack8(d4, d);
    unpack8(g4, g);
    unpack8(u4, u);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float a, slope;
      act_grad<ACT>(g[i], a, slope);
      og[i] = d[i] * u[i] * slope;
      ou[i] = d[i] * a;
    }
    p.dgu[2 * r * f8 + c] = make_uint4(pack_bf16x2(og[0], og[1]), pack_bf16x2(og[2], og[3]),
                                       pack_bf16x2(og[4], og[5]), pack_bf16x2(og[6], og[7]));
    p.dgu[(2 * r + 1) * f8 + c] = make_uint4(pack_bf16x2(ou[0], ou[1]), pack_bf16x2(ou[2], ou[3]),
                                             pack_bf16x2(ou[4], ou[5]), pack_bf16x2(ou[6], ou[7]));
  }
}

template <int FMT>
hipError_t run_grad(const GradParams& p, int act, hipStream_t stream) {
  const dim3 grid((unsigned)((p.f8 + 255) / 256), (unsigned)(p.m < 16384 ? p.m : 16384)), block(256);
  if (act == ACT_SILU) gated_grad_kernel<FMT, ACT_SILU><<<grid, block, 0, stream>>>(p);
  else if (act == ACT_GELU_TANH) gated_grad_kernel<FMT, ACT_GELU_TANH><<<grid, block, 0, stream>>>(p);
  else gated_grad_kernel<FMT, ACT_RELU><<<grid, block, 0, stream>>>(p);
  return hipGetLastError();
}

int64_t align256(int64_t b) { return (b + 255) / 256 * 256; }

}  // namespace

hipError_t launch_gated(const GatedArgs& a, hipStream_t stream) {
  if (a.gu_fmt == GU_NONE && stream_rows(a.m, 2 * a.f, a.k, false, true)) {
    StreamArgs s{};
    s.x = a.x;
    s.w = a.w;
    s.m = a.m;
    s.k = a.k;
    s.rows = a.f;
    s.gated = true;
    s.act = a.act;
    s.out = a.h;
    s.out_fmt = OUT_BF16;
    return launch_stream(s, stream);
  }
  return launch_gated_dense(a, stream);
}

// Workspace: dgu [m, 2 f] bf16, an 8-bit x [m, k] decoded to bf16, dx's partial sums.
int64_t gated_backward_workspace_bytes(int64_t m, int64_t k, int64_t f, bool x_mx) {
  if (m == 0) return 0;
  return align256(m * 2 * f * 2) + (x_mx ? align256(m * k * 2) : 0) + align256(dense_dx_workspace_bytes(m, k, 2 * f));
}

hipError_t launch_gated_backward(const GatedBackwardArgs& a, void* workspace, hipStream_t stream) {
  if (a.m == 0) return a.dw ? launch_dense_dw(nullptr, nullptr, 0, a.k, 2 * a.f, a.dw, stream) : hipSuccess;  // zeros
  uint8_t* at = static_cast<uint8_t*>(workspace);
  uint16_t* const dgu = reinterpret_cast<uint16_t*>(at);
  at += align256(a.m * 2 * a.f * 2);
  const uint16_t* x = static_cast<const uint16_t*>(a.x);
  GradParams p{};
  p.dh = reinterpret_cast<const uint4*>(a.dh);
  p.gu = a.gu;
  p.gu_scale = a.gu_scale;
  p.dgu = reinterpret_cast<uint4*>(dgu);
  p.m = a.m;
  p.f8 = (int)(a.f / 8);
  if (a.x_fmt != GU_BF16) {
    if (a.dw) {
      p.x = a.x;
      p.x_scale = a.x_scale;
      p.x_out = reinterpret_cast<uint4*>(at);
      p.x_chunks = a.m * (a.k / 8);
      p.x_fmt = a.x_fmt;
    }
    x = reinterpret_cast<const uint16_t*>(at);
    at += align256(a.m * a.k * 2);
  }
  hipError_t e = a.gu_fmt == GU_BF16   ? run_grad<GU_BF16>(p, a.act, stream)
                 : a.gu_fmt == GU_E4M3 ? run_grad<GU_E4M3>(p, a.act, stream)
                                       : run_grad<GU_E5M2>(p, a.act, stream);
  if (e == hipSuccess && a.dx) e = launch_dense_dx(dgu, a.w, a.m, a.k, 2 * a.f, a.dx, at, stream);
  if (e == hipSuccess && a.dw) e = launch_dense_dw(dgu, x, a.m, a.k, 2 * a.f, a.dw, stream);
  return e;
}

int64_t mxfp4_workspace_bytes(int64_t m, int64_t n, int64_t k) {
  return stream_rows(m, n, k, true, false) ? 0 : align256(dense_nt_workspace_bytes(m, n, k));
}

hipError_t launch_mxfp4(const StreamArgs& a, void* workspace, hipStream_t stream) {
  if (stream_rows(a.m, a.gated ? 2 * a.rows : a.rows, a.k, true, a.gated)) return launch_stream(a, stream);
  if (!a.gated) return launch_mxfp4_dense(a, workspace, stream);
  GatedArgs g{};
  g.x = a.x;
  g.w = a.w;
  g.w_scale = a.w_scale;
  g.m = a.m;
  g.k = a.k;
  g.f = a.rows;
  g.act = a.act;
  g.h = static_cast<uint16_t*>(a.out);
  g.gu_fmt = GU_NONE;
  return launch_gated_dense(g, stream);
}

DenseKernel block_kernel(int product, int64_t m, int64_t k, int64_t f) {
  if (product == PRODUCT_GATED_SAVING) return dense_gated_kernel(m, k, f);
  if (product == PRODUCT_DX) return dense_dx_kernel(m, k, 2 * f);
  if (product == PRODUCT_DW) return dense_dw_kernel(m, k, 2 * f);
  const bool fp4 = product != PRODUCT_GATED, gated = product != PRODUCT_MXFP4;
  if (!stream_rows(m, gated ? 2 * f : f, k, fp4, gated))
    return gated ? dense_gated_kernel(m, k, f) : dense_mxfp4_kernel(m, f, k);
  static const uint8_t some = 0;  // w_scale: tells a 4-bit weight from a bf16 one, not read
  StreamArgs a{};
  a.w_scale = fp4 ? &some : nullptr;
  a.m = m;
  a.k = k;
  a.rows = f;
  a.gated = gated;
  return {stream_name(a), 1};
}

}  // namespace sfr

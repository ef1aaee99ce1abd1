// The gated feed-forward block h = act(x Wg^T) * (x Wu^T): which kernels its
// forward and backward calls run, and the elementwise part of the gradients.
#include "sfr_launch.hpp"
#include "sfr_mx.hpp"

namespace sfr {
namespace {

// dgu[m] = [dh u act'(g) | dh act(g)] from the saved g and u: one pass, memory
// bound (per f: 2 bytes of dh, two saved values, 4 bytes written).  A lane
// holds 8 f.  The gradients are formed in binary32 and rounded once to bf16,
// the type in which the two products read them.
template <int FMT>
__device__ __forceinline__ void load_saved8(const void* gu, const uint8_t* scale, int64_t at, float (&v)[8]) {
  uint32_t w[4];
  if constexpr (FMT == GU_BF16) {
    const uint4 c = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(gu) + at);
    w[0] = c.x;
    w[1] = c.y;
    w[2] = c.z;
    w[3] = c.w;
  } else {
    constexpr int F = FMT == GU_E4M3 ? MX_E4M3 : MX_E5M2;
    const uint2 c = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint8_t*>(gu) + at);
    const float s = mx_scale_value(scale[at / MX_BLOCK]);
    w[0] = mx_widen2<F, false>(c.x, s);
    w[1] = mx_widen2<F, true>(c.x, s);
    w[2] = mx_widen2<F, false>(c.y, s);
    w[3] = mx_widen2<F, true>(c.y, s);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = bf16_to_f32(w[i] & 0xFFFFu);
    v[2 * i + 1] = bf16_to_f32(w[i] >> 16);
  }
}

template <int FMT, int ACT>
__global__ __launch_bounds__(256) void gated_grad_kernel(const uint4* __restrict__ dh, const void* __restrict__ gu,
                                                         const uint8_t* __restrict__ scale, int64_t m, int f8,
                                                         uint4* __restrict__ dgu) {
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= f8) return;
  for (int64_t r = blockIdx.y; r < m; r += gridDim.y) {
    const uint4 d4 = dh[r * f8 + c];
    const uint32_t d[4] = {d4.x, d4.y, d4.z, d4.w};
    float g[8], u[8];
    const int64_t at = (2 * r * f8 + c) * 8;
    load_saved8<FMT>(gu, scale, at, g);
    load_saved8<FMT>(gu, scale, at + (int64_t)f8 * 8, u);
    uint32_t og[4], ou[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float d0 = bf16_to_f32(d[i] & 0xFFFFu), d1 = bf16_to_f32(d[i] >> 16);
      float a0, a1, p0, p1;
      act_grad<ACT>(g[2 * i], a0, p0);
      act_grad<ACT>(g[2 * i + 1], a1, p1);
      og[i] = pack_bf16x2(d0 * u[2 * i] * p0, d1 * u[2 * i + 1] * p1);
      ou[i] = pack_bf16x2(d0 * a0, d1 * a1);
    }
    dgu[2 * r * f8 + c] = make_uint4(og[0], og[1], og[2], og[3]);
    dgu[(2 * r + 1) * f8 + c] = make_uint4(ou[0], ou[1], ou[2], ou[3]);
  }
}

template <int FMT>
hipError_t run_grad(const GatedBackwardArgs& a, uint16_t* dgu, hipStream_t stream) {
  const int f8 = (int)(a.f / 8);
  const dim3 grid((unsigned)((f8 + 255) / 256), (unsigned)(a.m < 16384 ? a.m : 16384)), block(256);
  const uint4* dh = reinterpret_cast<const uint4*>(a.dh);
  uint4* o = reinterpret_cast<uint4*>(dgu);
  if (a.act == ACT_SILU) gated_grad_kernel<FMT, ACT_SILU><<<grid, block, 0, stream>>>(dh, a.gu, a.gu_scale, a.m, f8, o);
  else if (a.act == ACT_GELU_TANH)
    gated_grad_kernel<FMT, ACT_GELU_TANH><<<grid, block, 0, stream>>>(dh, a.gu, a.gu_scale, a.m, f8, o);
  else gated_grad_kernel<FMT, ACT_RELU><<<grid, block, 0, stream>>>(dh, a.gu, a.gu_scale, a.m, f8, o);
  return hipGetLastError();
}

int64_t align256(int64_t b) { return (b + 255) / 256 * 256; }

}  // namespace

hipError_t launch_gated(const GatedArgs& a, hipStream_t stream) {
  if (a.gu_fmt == GU_NONE && stream_rows(a.m, 2 * a.f, a.k, false)) {
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

// Workspace: dgu [m, 2 f] bf16, then what one of the products needs at a time:
// dx its partial sums, dW (8-bit x) x [m, k] decoded to bf16.
int64_t gated_backward_workspace_bytes(int64_t m, int64_t k, int64_t f, bool x_mx) {
  if (m == 0) return 0;
  const int64_t partial = dense_dx_workspace_bytes(m, k, 2 * f), decoded = x_mx ? m * k * 2 : 0;
  return align256(m * 2 * f * 2) + align256(partial > decoded ? partial : decoded);
}

hipError_t launch_gated_backward(const GatedBackwardArgs& a, void* workspace, hipStream_t stream) {
  uint16_t* dgu = static_cast<uint16_t*>(workspace);
  void* more = static_cast<uint8_t*>(workspace) + align256(a.m * 2 * a.f * 2);
  if (a.m == 0) return a.dw ? launch_dense_dw(dgu, nullptr, 0, a.k, 2 * a.f, a.dw, stream) : hipSuccess;  // zeros
  hipError_t e = a.gu_fmt == GU_BF16   ? run_grad<GU_BF16>(a, dgu, stream)
                 : a.gu_fmt == GU_E4M3 ? run_grad<GU_E4M3>(a, dgu, stream)
                                       : run_grad<GU_E5M2>(a, dgu, stream);
  if (e != hipSuccess) return e;
  if (a.dx) {
    e = launch_dense_dx(dgu, a.w, a.m, a.k, 2 * a.f, a.dx, more, stream);
    if (e != hipSuccess) return e;
  }
  if (a.dw) {
    const uint16_t* x = static_cast<const uint16_t*>(a.x);
    if (a.x_fmt != GU_BF16) {
      uint16_t* const xw = static_cast<uint16_t*>(more);
      e = launch_dequantize_mx(static_cast<const uint8_t*>(a.x), a.x_scale, a.m, a.k,
                               a.x_fmt == GU_E4M3 ? MX_E4M3 : MX_E5M2, xw, stream);
      if (e != hipSuccess) return e;
      x = xw;
    }
    e = launch_dense_dw(dgu, x, a.m, a.k, 2 * a.f, a.dw, stream);
  }
  return e;
}

int64_t mxfp4_workspace_bytes(int64_t m, int64_t n, int64_t k, bool gated) {
  return gated || stream_rows(m, n, k, true) ? 0 : align256(dense_nt_workspace_bytes(m, n, k));
}

hipError_t launch_mxfp4(const StreamArgs& a, void* workspace, hipStream_t stream) {
  if (stream_rows(a.m, a.gated ? 2 * a.rows : a.rows, a.k, true)) return launch_stream(a, stream);
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

}  // namespace sfr

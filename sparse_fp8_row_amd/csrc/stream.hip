// Products of a few activation rows with a weight that is read once: the
// decode forms of the gated block (bf16 or 4-bit weight) and of the 4-bit
// linear layer.  Bound by reading the weight.
//
// A workgroup owns 16 RT weight rows and up to 16 activation rows (grid y); its
// wavefronts take steps of 128 k in turn, so together they read whole lines of
// each row, and their binary32 sums are added in a fixed order through LDS.
// The product runs on v_mfma_f32_16x16x32_bf16 with the weight as A operand:
// lane l holds weight row l % 16.  The order of k inside a step is free as long
// as both operands agree, so each lane loads 16 contiguous bytes of its row:
//   4-bit: 32 codes, one block of the format with one scale; instruction j of
//     the step takes codes 8 j .. 8 j + 7, decoded (exactly) to bf16 with the
//     scale applied by the converter: k = 32 (l / 16) + 8 j ..;
//   bf16: four loads of 8 values, k = 32 j + 8 (l / 16) ...
// Gated: row tiles alternate between gate and up rows, so act(g) * u is
// formed from the sums before anything is rounded.
#include "sfr_dense.hpp"

namespace sfr {
namespace {

template <bool FP4, bool GATED, int RT, int NW, int U>
__global__ __launch_bounds__(64 * NW) void stream_kernel(StreamArgs p) {
  static_assert(!GATED || RT % 2 == 0, "row tiles come in pairs");
  __shared__ __attribute__((aligned(16))) float red[NW][RT][16][16];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, lg = lane >> 4;
  const int64_t m0 = (int64_t)blockIdx.y * 16;
  const int mr = (int)min(p.m - m0, (int64_t)16);
  const int64_t n0 = (int64_t)blockIdx.x * (GATED ? RT / 2 : RT) * 16;
  const int K = (int)p.k;
  const int steps = (K + 127) / 128;

  // rows past the end read the last row (and are not stored)
  const uint16_t* x = p.x + (m0 + min(r16, mr - 1)) * K;
  const uint8_t* w[RT];
  const uint8_t* ws[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    const int64_t tile = GATED ? t >> 1 : t;
    const int64_t row = min(n0 + tile * 16 + r16, p.rows - 1) + (GATED && (t & 1) ? p.rows : 0);
    w[t] = static_cast<const uint8_t*>(p.w) + (FP4 ? row * (K / 2) : row * 2 * K);
    ws[t] = FP4 ? p.w_scale + row * (K / 32) : nullptr;
  }

  v4f acc[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) acc[t] = v4f{0.f, 0.f, 0.f, 0.f};

  for (int s0 = wave; s0 < steps; s0 += NW * U) {
    uint4 xv[U][4], wv[U][RT][FP4 ? 1 : 4];
    uint32_t sv[U][RT];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int s = s0 + i * NW;
      if (s < steps) {
        if constexpr (FP4) {
          // a lane whose block lies past the end of the row reads block 0 and
          // multiplies it by zero activations and a zero scale
          const int blk = s * 4 + lg;
          const bool in = blk * 32 < K;
          const int b = in ? blk : 0;
#pragma unroll
          for (int t = 0; t < RT; ++t) {
            wv[i][t][0] = *reinterpret_cast<const uint4*>(w[t] + b * 16);
            sv[i][t] = ws[t][b];
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            xv[i][j] = *reinterpret_cast<const uint4*>(x + b * 32 + 8 * j);
            if (!in) xv[i][j] = make_uint4(0, 0, 0, 0);
          }
#pragma unroll
          for (int t = 0; t < RT; ++t)
            if (!in) {
              sv[i][t] = 0;
              wv[i][t][0] = make_uint4(0, 0, 0, 0);
            }
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int k = s * 128 + 32 * j;
            const bool in = k < K;  // the same for every lane
#pragma unroll
            for (int t = 0; t < RT; ++t)
              wv[i][t][j] = in ? *reinterpret_cast<const uint4*>(w[t] + 2 * (k + 8 * lg)) : make_uint4(0, 0, 0, 0);
            xv[i][j] = in ? *reinterpret_cast<const uint4*>(x + k + 8 * lg) : make_uint4(0, 0, 0, 0);
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < U; ++i) {
      if (s0 + i * NW < steps) {
#pragma unroll
        for (int t = 0; t < RT; ++t) {
          if constexpr (FP4) {
            const float f = mx_scale_value(sv[i][t]);
            const uint32_t c[4] = {wv[i][t][0].x, wv[i][t][0].y, wv[i][t][0].z, wv[i][t][0].w};
#pragma unroll
            for (int j = 0; j < 4; ++j)
              acc[t] = mfma16(__builtin_bit_cast(v8bf, mx_widen8_e2m1(c[j], f)), __builtin_bit_cast(v8bf, xv[i][j]),
                              acc[t]);
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              acc[t] = mfma16(__builtin_bit_cast(v8bf, wv[i][t][j]), __builtin_bit_cast(v8bf, xv[i][j]), acc[t]);
          }
        }
      }
    }
  }

#pragma unroll
  for (int t = 0; t < RT; ++t)
    if (r16 < mr) *reinterpret_cast<v4f*>(&red[wave][t][r16][4 * lg]) = acc[t];
  __syncthreads();
  constexpr int OT = GATED ? RT / 2 : RT;
  for (int i = threadIdx.x; i < OT * 16 * mr; i += 64 * NW) {
    const int n = i % 16, t = i / 16 % OT, m = i / (16 * OT);
    const int64_t col = n0 + t * 16 + n;
    float y = 0.f, u = 0.f;
#pragma unroll
    for (int v = 0; v < NW; ++v) {
      y += red[v][GATED ? 2 * t : t][m][n];
      if constexpr (GATED) u += red[v][2 * t + 1][m][n];
    }
    if constexpr (GATED) {
      y = u * (p.act == ACT_SILU        ? act_value<ACT_SILU>(y)
               : p.act == ACT_GELU_TANH ? act_value<ACT_GELU_TANH>(y)
                                        : act_value<ACT_RELU>(y));
    }
    if (col < p.rows) {
      if (p.bias) y += bf16_to_f32(p.bias[col]);
      const int64_t at = (m0 + m) * p.rows + col;
      if (p.out_fmt == OUT_F32) static_cast<float*>(p.out)[at] = y;
      else static_cast<uint16_t*>(p.out)[at] = (uint16_t)pack_bf16x2(y, 0.f);
    }
  }
}

template <bool FP4, bool GATED, int RT, int NW, int U>
hipError_t run_stream(const StreamArgs& a, hipStream_t stream) {
  constexpr int cover = (GATED ? RT / 2 : RT) * 16;
  const dim3 grid((unsigned)((a.rows + cover - 1) / cover), (unsigned)((a.m + 15) / 16));
  stream_kernel<FP4, GATED, RT, NW, U><<<grid, dim3(64 * NW), 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace

bool stream_rows(int64_t m) { return m <= 32; }

hipError_t launch_stream(const StreamArgs& a, hipStream_t stream) {
  if (!a.w_scale) return run_stream<false, true, 2, 8, 1>(a, stream);
  if (a.gated) return run_stream<true, true, 2, 8, 2>(a, stream);
  return run_stream<true, false, 1, 8, 2>(a, stream);
}

}  // namespace sfr

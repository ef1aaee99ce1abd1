// Dense bf16 products of the gated feed-forward block on the matrix cores:
//   forward      P = x [Wg; Wu]^T, with h = act(g) * u (and the checkpoint of
//                g, u) formed from the accumulators;
//   input grad   dx = [dg du] [Wg; Wu];
//   weight grad  dW = [dg du]^T x;
// and the product with a decoded 4-bit weight.  Bound by the matrix cores for
// many rows (4 m k f operations forward, twice that backward), by reading the
// weight for few.
#include "sfr_dense.hpp"

namespace sfr {
namespace {

enum { EPI_PLAIN = 0, EPI_GATED = 1 };

struct DenseParams {
  const uint16_t *x, *w;
  int64_t ldx, ldw;
  int64_t rows_m, rows_n;  // rows of X; rows of W (GATED: of one half)
  int64_t k;
  int64_t k_per_split;  // multiple of BK; k of one slice of the sum
  int64_t tiles_m, tiles_n;
  int group;
  float* partial;  // with several slices: binary32 [slices, m, n], summed by dense_reduce_kernel
  PlainOut plain;
  GatedOut gated;
};

// ---------------------------------------------------------------------------
// Tiled kernel: BN x BM outputs per workgroup, WN x WM wavefronts of 64 (n) x
// BM / WM (m), S stages of BK in LDS.
// ---------------------------------------------------------------------------
template <int LX, int LW, int EPI, int BN, int BM, int WN, int WM, int S>
__global__ __launch_bounds__(64 * WN * WM) void dense_tile_kernel(DenseParams p) {
  constexpr int NW = WN * WM, FM = BM / WM / 16, FN = 4;
  constexpr bool PAIR = EPI == EPI_GATED;
  constexpr int WB = BN * BK * 2, XB = BM * BK * 2, STAGE = WB + XB;
  constexpr int LPS = BN / 8 / NW + BM / 8 / NW;  // loads per wavefront and stage
  static_assert(BN == WN * 64, "64 weight rows per wavefront");
  static_assert(NW * FM * 16 * 128 <= S * STAGE, "epilogue regions fit");
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];

  int64_t tm, tn;
  if (!tile_of(blockIdx.x, p.tiles_m, p.tiles_n, p.group, tm, tn)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wn = wave / WM, wm = wave % WM;
  const int64_t m0 = tm * BM, n0 = tn * (PAIR ? BN / 2 : BN);
  const int64_t k0 = blockIdx.y * p.k_per_split;
  const int kdim = (int)min(p.k - k0, p.k_per_split);
  const int KT = (kdim + BK - 1) / BK;

  Loader<LW, BN, NW, PAIR> lw(p.w, p.ldw, n0, p.rows_n, k0, p.k, wave, lane);
  Loader<LX, BM, NW, false> lx(p.x, p.ldx, m0, p.rows_m, k0, p.k, wave, lane);
  const Reader<LW, BN> rw(lane);
  const Reader<LX, BM> rx(lane);
  auto load = [&](int kt) __attribute__((always_inline)) {
    uint8_t* s = smem + (kt % S) * STAGE;
    lw.stage(s, kdim - kt * BK);
    lx.stage(s + WB, kdim - kt * BK);
  };

  v4f acc[FN][FM];
#pragma unroll
  for (int i = 0; i < FN; ++i)
#pragma unroll
    for (int j = 0; j < FM; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};

#pragma unroll
  for (int s = 0; s < S - 1; ++s)
    if (s < KT) load(s);
  for (int kt = 0; kt < KT; ++kt) {
    // stage kt has landed once only the later stages' loads are pending
    if (kt + S - 2 < KT) wait_vm<(S - 2) * LPS>();
    else wait_vm<0>();
    wait_lds();  // this wavefront's reads of the slot to be refilled are done
    wg_barrier();
    if (kt + S - 1 < KT) load(kt + S - 1);
    const uint8_t* tw = smem + (kt % S) * STAGE;
    const uint8_t* tx = tw + WB;
#pragma unroll
    for (int kk = 0; kk < BK / 32; ++kk) {
      v8bf a[FN], b[FM];
#pragma unroll
      for (int i = 0; i < FN; ++i) a[i] = rw.read(tw, wn * FN + i, kk);
#pragma unroll
      for (int j = 0; j < FM; ++j) b[j] = rx.read(tx, wm * FM + j, kk);
#pragma unroll
      for (int i = 0; i < FN; ++i)
#pragma unroll
        for (int j = 0; j < FM; ++j) acc[i][j] = mfma16(a[i], b[j], acc[i][j]);
    }
  }
  wait_lds();
  wg_barrier();  // every wavefront is done with the stages: their LDS becomes the epilogue's

  uint8_t* region = smem + wave * (FM * 16 * 128);
  const int64_t mb = m0 + wm * (FM * 16);
  if constexpr (EPI == EPI_GATED) {
    const v4f(&g0)[FM] = acc[0], (&u0)[FM] = acc[1], (&g1)[FM] = acc[2], (&u1)[FM] = acc[3];
    v4f g[2][FM], u[2][FM];
#pragma unroll
    for (int j = 0; j < FM; ++j) {
      g[0][j] = g0[j];
      g[1][j] = g1[j];
      u[0][j] = u0[j];
      u[1][j] = u1[j];
    }
    gated_epilogue<FM>(g, u, p.gated, mb, n0 + wn * 32, lane, region);
  } else {
    PlainOut o = p.plain;
    if (p.partial) {
      o.out = p.partial + (int64_t)blockIdx.y * o.m * o.n;
      o.bias = nullptr;
      o.out_fmt = OUT_F32;
    }
    plain_epilogue<FM>(acc, o, mb, n0 + wn * 64, lane, region);
  }
}

// Sums the slices in order, adds the bias, rounds once.
__global__ __launch_bounds__(256) void dense_reduce_kernel(const float* __restrict__ partial, int slices, PlainOut o) {
  const int64_t quads = o.m * o.n / 4;
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (at >= quads) return;
  const v4f* p = reinterpret_cast<const v4f*>(partial);
  v4f s = p[at];
  for (int i = 1; i < slices; ++i) s += p[at + i * quads];
  if (o.bias) {
    const uint2 b = *reinterpret_cast<const uint2*>(o.bias + at * 4 % o.n);
    s[0] += bf16_to_f32(b.x & 0xFFFFu);
    s[1] += bf16_to_f32(b.x >> 16);
    s[2] += bf16_to_f32(b.y & 0xFFFFu);
    s[3] += bf16_to_f32(b.y >> 16);
  }
  if (o.out_fmt == OUT_F32) reinterpret_cast<v4f*>(o.out)[at] = s;
  else reinterpret_cast<uint2*>(o.out)[at] = make_uint2(pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3]));
}

template <int LX, int LW, int EPI, int BN, int BM, int WN, int WM, int S>
hipError_t run_tile(DenseParams p, int slices, hipStream_t stream) {
  constexpr int bytes = S * (BN + BM) * BK * 2;
  auto* kernel = dense_tile_kernel<LX, LW, EPI, BN, BM, WN, WM, S>;
  if (bytes > 65536) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != hipSuccess) return e;
  }
  constexpr int cover = EPI == EPI_GATED ? BN / 2 : BN;
  p.tiles_m = (p.rows_m + BM - 1) / BM;
  p.tiles_n = (p.rows_n + cover - 1) / cover;
  p.group = 8;
  const int64_t grid = (p.tiles_m * p.tiles_n + 7) / 8 * 8;
  if (grid > (1 << 24)) return hipErrorInvalidValue;
  kernel<<<dim3((unsigned)grid, (unsigned)slices), dim3(64 * WN * WM), bytes, stream>>>(p);
  return hipGetLastError();
}

template <int LX, int LW, int EPI>
hipError_t run_dense(const DenseParams& p, int slices, hipStream_t stream) {
  if (p.rows_m > 64) return run_tile<LX, LW, EPI, 128, 128, 2, 2, 2>(p, slices, stream);
  return run_tile<LX, LW, EPI, 64, 64, 1, 4, 3>(p, slices, stream);
}

}  // namespace



hipError_t launch_gated_dense(const GatedArgs& a, hipStream_t stream) {
  DenseParams p{};
  p.x = a.x;
  p.w = a.w;
  p.ldx = p.ldw = a.k;
  p.rows_m = a.m;
  p.rows_n = a.f;
  p.k = p.k_per_split = a.k;
  p.gated = GatedOut{a.h, a.gu, a.gu_scale, a.m, a.f, a.act, a.gu_fmt};
  return run_dense<ROWS, ROWS, EPI_GATED>(p, 1, stream);
}

hipError_t launch_dense_nt(const uint16_t* x, const uint16_t* w, int64_t m, int64_t n, int64_t k, const uint16_t* bias,
                           void* out, int out_fmt, hipStream_t stream) {
  DenseParams p{};
  p.x = x;
  p.w = w;
  p.ldx = p.ldw = k;
  p.rows_m = m;
  p.rows_n = n;
  p.k = p.k_per_split = k;
  p.plain = PlainOut{out, bias, m, n, out_fmt};
  return run_dense<ROWS, ROWS, EPI_PLAIN>(p, 1, stream);
}

hipError_t launch_dense_dx(const uint16_t* dgu, const uint16_t* w, int64_t m, int64_t k, int64_t f2, uint16_t* dx,
                           hipStream_t stream) {
  DenseParams p{};
  p.x = dgu;
  p.w = w;
  p.ldx = f2;
  p.ldw = k;
  p.rows_m = m;
  p.rows_n = k;
  p.k = p.k_per_split = f2;
  p.plain = PlainOut{dx, nullptr, m, k, OUT_BF16};
  return run_dense<ROWS, COLS, EPI_PLAIN>(p, 1, stream);
}

hipError_t launch_dense_dw(const uint16_t* dgu, const uint16_t* x, int64_t m, int64_t k, int64_t f2, uint16_t* dw,
                           hipStream_t stream) {
  DenseParams p{};
  p.x = dgu;
  p.w = x;
  p.ldx = f2;
  p.ldw = k;
  p.rows_m = f2;
  p.rows_n = k;
  p.k = p.k_per_split = m;
  p.plain = PlainOut{dw, nullptr, f2, k, OUT_BF16};
  return run_dense<COLS, COLS, EPI_PLAIN>(p, 1, stream);
}

}  // namespace sfr

// Dense bf16 products of the gated feed-forward block on the matrix cores:
//   forward      P = x [Wg; Wu]^T, with h = act(g) * u (and the checkpoint of
//                g, u) formed from the accumulators;
//   input grad   dx = [dg du] [Wg; Wu];
//   weight grad  dW = [dg du]^T x;
// and the products with a decoded 4-bit weight and of 8-bit integers.  Bound by the matrix cores for
// many rows (4 m k f operations forward, twice that backward), by reading the
// weight for few.
#include <type_traits>

#include "sfr_dense.hpp"

namespace sfr {
namespace {

enum { EPI_PLAIN = 0, EPI_GATED = 1, EPI_INT8 = 2 };

template <int EPI>
using Sum = std::conditional_t<EPI == EPI_INT8, v4i, v4f>;

struct DenseParams {
  const uint16_t *x, *w;
  const uint8_t* w_scale;  // CODES: w holds the codes
  int64_t ldx, ldw;
  int64_t rows_m, rows_n;  // rows of X; rows of W (GATED: of one half)
  int64_t k;
  int64_t k_per_split;  // multiple of BK; k of one slice of the sum
  int slices, tiles_m, tiles_n, group;
  float* partial;  // with several slices: binary32 [slices, m, n], summed by dense_reduce_kernel
  PlainOut plain;
  GatedOut gated;
  Int8Scales scales;  // EPI_INT8: x, w and every count of k stand for pairs of 8-bit integers
};

// Where this workgroup's outputs go: the output, or its slice's partial sums.
__device__ __forceinline__ PlainOut plain_of(const DenseParams& p, uint32_t slice) {
  PlainOut o = p.plain;
  if (p.partial) {
    o.out = p.partial + (int64_t)slice * o.m * o.n;
    o.bias = nullptr;
    o.out_fmt = OUT_F32;
  }
  return o;
}

// A workgroup's scales in LDS (EPI_INT8), nothing otherwise.
template <int EPI, int BM, int BN>
struct TileScales {
  Int8Tile<BM, BN> t;
};
template <int BM, int BN>
struct TileScales<EPI_PLAIN, BM, BN> {};
template <int BM, int BN>
struct TileScales<EPI_GATED, BM, BN> {};

// The W operand's loader in the three forms.
template <int LW, int BR, int NW, bool PAIR, int DEPTH = 1>
struct WLoader {
  Loader<LW, BR, NW, PAIR> rows;
  __device__ __forceinline__ WLoader(const DenseParams& p, int64_t r0, int64_t k0, int wave, int lane)
      : rows(p.w, p.ldw, r0, p.rows_n, k0, wave, lane) {}
};
template <int BR, int NW, bool PAIR, int DEPTH>
struct WLoader<CODES, BR, NW, PAIR, DEPTH> {
  CodeLoader<BR, NW, PAIR, DEPTH> codes;
  __device__ __forceinline__ WLoader(const DenseParams& p, int64_t r0, int64_t k0, int wave, int lane)
      : codes(p.w, p.w_scale, p.k, r0, p.rows_n, k0, wave, lane) {}
};

// ---------------------------------------------------------------------------
// Tiled kernel: BN x BM outputs per workgroup, WN x WM wavefronts of 64 (n) x
// BM / WM (m), S stages of BK in LDS.  KS = 2: two such groups of wavefronts in
// the workgroup, each with half of k and stages of its own; the second's sums
// are added to the first's through LDS.  With few tiles, where a CU would hold
// one group and every stage waits out its latencies, two of them overlap (m =
// 140, k = f = 4096: forward 29.6 -> 23.6 us, with a 4-bit weight 36.7 -> 29.3).
// ---------------------------------------------------------------------------
template <int LX, int LW, int EPI, int BN, int BM, int WN, int WM, int S, int KS>
__global__ __launch_bounds__(64 * WN * WM * KS) void dense_tile_kernel(DenseParams p) {
  constexpr int NW = WN * WM, FM = BM / WM / 16, FN = 4;
  constexpr bool PAIR = EPI == EPI_GATED;
  constexpr int WB = BN * BK * 2, XB = BM * BK * 2, STAGE = WB + XB;
  constexpr bool FP4 = LW == CODES;
  // loads per wavefront and stage into LDS; of codes
  constexpr int LPS = (FP4 ? 0 : BN / 8 / NW) + BM / 8 / NW, LPC = FP4 ? CodeLoader<BN, NW, PAIR, 1>::LOADS : 0;
  static_assert(BN == WN * 64, "64 weight rows per wavefront");
  static_assert(NW * FM * 16 * 128 <= S * STAGE, "epilogue regions fit");
  static_assert(NW * FN * FM * 1024 <= S * STAGE, "the second group's sums fit in its stages");
  extern __shared__ __attribute__((aligned(1024))) uint8_t all_smem[];

  uint32_t slice;
  int64_t tm, tn;
  if (!tile_of(blockIdx.x, p.slices, p.tiles_m, p.tiles_n, p.group, slice, tm, tn)) return;
  const int lane = threadIdx.x & 63, wave_id = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kg = KS == 1 ? 0 : wave_id / NW, wave = KS == 1 ? wave_id : wave_id % NW;
  uint8_t* const smem = all_smem + kg * (S * STAGE);
  const int wn = wave / WM, wm = wave % WM;
  const int64_t m0 = tm * BM, n0 = tn * (PAIR ? BN / 2 : BN);
  const int64_t ks = slice * p.k_per_split;
  const int kslice = (int)min(p.k - ks, p.k_per_split);
  // every group runs the same number of stages; k past the slice reads zeros
  const int KT = ((kslice + BK - 1) / BK + KS - 1) / KS;
  const int64_t k0 = ks + kg * KT * BK;
  const int kdim = min(kslice - kg * KT * BK, KT * BK);

  WLoader<LW, BN, NW, PAIR> lw(p, n0, k0, wave, lane);
  Loader<LX, BM, NW, false> lx(p.x, p.ldx, m0, p.rows_m, k0, wave, lane);
  const Reader<FP4 ? ROWS : LW, BN, FN> rw(wn * FN, lane);
  const Reader<LX, BM, FM> rx(wm * FM, lane);
  // Puts stage kt in flight.  CODES: its codes were fetched one stage ago; they
  // go to LDS and the next stage's are fetched.
  auto load = [&](int kt) __attribute__((always_inline)) {
    uint8_t* s = smem + (kt % S) * STAGE;
    lx.stage(s + WB, kdim - kt * BK);
    if constexpr (FP4) {
      lw.codes.template put<0>(s);
      lw.codes.template fetch<0>(kdim - (kt + 1) * BK);
    } else {
      lw.rows.stage(s, kdim - kt * BK);
    }
  };
  Sum<EPI> acc[FN][FM];
#pragma unroll
  for (int i = 0; i < FN; ++i)
#pragma unroll
    for (int j = 0; j < FM; ++j) acc[i][j] = Sum<EPI>{};

  __shared__ TileScales<EPI, BM, BN> scales;
  Int8Fetched fetched{};
  if constexpr (EPI == EPI_INT8)
    if (!p.partial) fetched = fetch_scales<BM, BN>(p.scales, p.plain, m0, n0, threadIdx.x, 64 * NW * KS);
  if constexpr (FP4) lw.codes.template fetch<0>(kdim);
#pragma unroll
  for (int s = 0; s < S - 1; ++s)
    if (s < KT) load(s);
  if constexpr (EPI == EPI_INT8)
    if (!p.partial) put_scales<BM, BN>(scales.t, fetched, p.plain.bias, threadIdx.x, 64 * NW * KS);
  for (int kt = 0; kt < KT; ++kt) {
    // stage kt has landed once only the later stages' loads (and the codes
    // fetched with and after it) are pending
    if (kt + S - 2 < KT) wait_vm<(S - 2) * LPS + (S - 1) * LPC>();
    else wait_vm<0>();
    wait_lds();  // this wavefront's reads of the slot to be refilled are done
    wg_barrier();
    if (kt + S - 1 < KT) load(kt + S - 1);
    const uint8_t* tw = smem + (kt % S) * STAGE;
    const uint8_t* tx = tw + WB;
    v8bf a[2][FN], b[2][FM];
    rw.read(a, tw);
    rx.read(b, tx);
#pragma unroll
    for (int kk = 0; kk < 2; ++kk)
#pragma unroll
      for (int i = 0; i < FN; ++i)
#pragma unroll
        for (int j = 0; j < FM; ++j) acc[i][j] = mfma16(a[kk][i], b[kk][j], acc[i][j]);
  }
  wait_lds();
  wg_barrier();  // every wavefront is done with the stages: their LDS becomes the epilogue's

  if constexpr (KS == 2) {
    Sum<EPI>* const sums = reinterpret_cast<Sum<EPI>*>(all_smem + S * STAGE) + wave * (FN * FM * 64) + lane;
    if (kg == 1) {
#pragma unroll
      for (int i = 0; i < FN; ++i)
#pragma unroll
        for (int j = 0; j < FM; ++j) sums[(i * FM + j) * 64] = acc[i][j];
      wait_lds();
    }
    wg_barrier();
    if (kg == 1) return;
#pragma unroll
    for (int i = 0; i < FN; ++i)
#pragma unroll
      for (int j = 0; j < FM; ++j) acc[i][j] += sums[(i * FM + j) * 64];
  }

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
  } else if constexpr (EPI == EPI_INT8) {
    const Int8Tile<BM, BN>& t = scales.t;
    int8_epilogue<FM>(acc, p.partial ? nullptr : t.x + wm * (FM * 16), t.w + wn * 64, t.bias + wn * 64,
                      plain_of(p, slice), mb, n0 + wn * 64, lane, region);
  } else {
    plain_epilogue<FM>(acc, plain_of(p, slice), mb, n0 + wn * 64, lane, region);
  }
}

// ---------------------------------------------------------------------------
// Wide kernel: 128 WH x 64 XF outputs (256 x 256, 256 x 192, 384 x 192), eight
// wavefronts in two groups of four (one wavefront of each group per SIMD), two
// stages of BK in LDS.
//
// W's stage is WH part tiles of 128 rows, of which a wavefront owns 64 rows each
// (group g: rows 64 g ..); it owns 16 XF of X's 64 XF rows.  One step of k is WH
// phases, each: read operands from LDS and put tiles of later stages in flight;
// barrier; 8 XF matrix instructions; barrier.  The second group runs one
// barrier behind, so on every SIMD one wavefront reads while the other
// multiplies.
//
//   phase  LDS reads   loads issued                    outputs
//     0    W0, X       last part of W, step t + 1      W0 x X
//     1    W1          W0 and X of t + 2               W1 x X
//     2    W2          W1 of t + 2                     W2 x X      (WH = 3)
// (CODES: W's codes are fetched one or two steps earlier still; "issued" means
// decoded into LDS, and each part tile's fetch is two loads like its ROWS form.)
// A tile is refilled no earlier than the phase after its last read: every
// wavefront waits for its LDS reads before the barrier that ends its reading
// part, and the other group is one barrier away.  `pending` loads per
// wavefront (issued after the ones that the next phase needs) stay in flight
// when a phase waits.  Loads past the last step read zeros (they are masked)
// and keep the counts.
//
// Measured at m = 8192, k = 4096, f = 14336 (256 x 256): 1.37 - 1.45 PFLOP/s
// forward, 1.50 dx, 1.38 dW (median of a run, the best 2 - 6% higher), with the matrix
// units busy 80% of the cycles at a clock that power holds near 1.5 GHz.  On one
// box, where the forward pass took 1485 us (1.30): without the global loads 1272,
// without the LDS reads 1470, with phases of 16 instructions 1693.
// ---------------------------------------------------------------------------
template <int LX, int LW, int EPI, int WH, int XF>
__global__ __launch_bounds__(512, 2) void dense_wide_kernel(DenseParams p) {
  constexpr bool PAIR = EPI == EPI_GATED, FP4 = LW == CODES;
  // X in LDS: one tile of all its rows, or (COLS) tiles of 128
  constexpr int XT = LX == COLS ? XF / 2 : 1, XR = 64 * XF / XT, XFT = XF / XT;
  constexpr int WPART = 128 * BK * 2, XPART = XR * BK * 2, STAGE = WH * WPART + XT * XPART;
  static_assert(XR % 64 == 0 && (LX != COLS || XR == 128), "tile layouts");
  constexpr int LOADS_X = XF, LOADS_W = 2;  // per wavefront: X's stage, a part of W
  // Steps in pairs, their LDS addresses fixed: dx at m = 8192 1566 -> 1506 us, m =
  // 64 525 -> 442; a 4-bit weight (then fetched two steps ahead) in tiles of 256 x
  // 192 at m = 300 89 -> 82 us, but in 256 x 256 104 -> 106.  The forward pass
  // with a bf16 weight gains nothing (86 -> 88).
  constexpr bool PAIRS = LW == COLS || (FP4 && WH * XF <= 6);
  constexpr int DEPTH = FP4 && PAIRS ? 2 : 1;
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];

  uint32_t slice;
  int64_t tm, tn;
  if (!tile_of(blockIdx.x, p.slices, p.tiles_m, p.tiles_n, p.group, slice, tm, tn)) return;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wn = wave >> 2, wm = wave & 3;
  constexpr int HN = PAIR ? 64 : 128;  // W rows (of one of the pair) per part
  const int64_t m0 = tm * (64 * XF), n0 = tn * (WH * HN);
  const int64_t k0 = slice * p.k_per_split;
  const int kdim = (int)min(p.k - k0, p.k_per_split), KT = (kdim + BK - 1) / BK;

  WLoader<LW, 128, 8, PAIR, DEPTH> lw0(p, n0, k0, wave, lane);
  WLoader<LW, 128, 8, PAIR, DEPTH> lw1(p, n0 + HN, k0, wave, lane);
  WLoader<LW, 128, 8, PAIR, DEPTH> lw2(p, n0 + 2 * HN, k0, wave, lane);  // WH = 3
  Loader<LX, XR, 8, false> lx0(p.x, p.ldx, m0, p.rows_m, k0, wave, lane);
  Loader<LX, XR, 8, false> lx1(p.x, p.ldx, m0 + XR, p.rows_m, k0, wave, lane);  // XT = 2
  const Reader<FP4 ? ROWS : LW, 128, 4> rw(wn * 4, lane);
  const Reader<LX, XR, XFT> rx(wm * XFT, lane);

  Sum<EPI> acc[WH][XT][4][XFT];
#pragma unroll
  for (int h = 0; h < WH; ++h)
#pragma unroll
    for (int q = 0; q < XT; ++q)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < XFT; ++j) acc[h][q][i][j] = Sum<EPI>{};

  auto load_x = [&](int t) __attribute__((always_inline)) {
    uint8_t* s = smem + (t & 1) * STAGE + WH * WPART;
    lx0.stage(s, kdim - t * BK);
    if constexpr (XT == 2) lx1.stage(s + XPART, kdim - t * BK);
  };
  // Part `part` of W of step t, whose stage is `slot` (a constant in pairs of
  // steps); CODES: the codes fetched DEPTH steps ago go to LDS and those of step
  // t + DEPTH are fetched.
  using Even = std::integral_constant<int, 0>;
  using Odd = std::integral_constant<int, 1>;
  auto load_w = [&](auto slot, auto& l, int part, int t) __attribute__((always_inline)) {
    uint8_t* tile = smem + slot * STAGE + part * WPART;
    if constexpr (DEPTH == 2) {
      l.codes.template put<decltype(slot)::value>(tile);
      l.codes.template fetch<decltype(slot)::value>(kdim - (t + 2) * BK);
    } else if constexpr (FP4) {
      l.codes.template put<0>(tile);
      l.codes.template fetch<0>(kdim - (t + 1) * BK);
    } else {
      l.rows.stage(tile, kdim - t * BK);
    }
  };
  // the loads in the order of the phases
  if constexpr (FP4) {
    auto ahead = [&](auto& l) __attribute__((always_inline)) {
      l.codes.template fetch<0>(kdim);
      if constexpr (DEPTH == 2) l.codes.template fetch<1>(kdim - BK);
    };
    ahead(lw0);
    ahead(lw1);
    if constexpr (WH == 3) ahead(lw2);
  }
  __shared__ TileScales<EPI, 64 * XF, 128 * WH> scales;
  Int8Fetched fetched{};
  if constexpr (EPI == EPI_INT8)
    if (!p.partial) fetched = fetch_scales<64 * XF, 128 * WH>(p.scales, p.plain, m0, n0, threadIdx.x, 512);
  load_w(Even{}, lw0, 0, 0);
  load_x(0);
  load_w(Even{}, lw1, 1, 0);
  if constexpr (WH == 3) load_w(Even{}, lw2, 2, 0);
  load_w(Odd{}, lw0, 0, 1);
  load_x(1);
  if constexpr (WH == 3) load_w(Odd{}, lw1, 1, 1);
  if constexpr (EPI == EPI_INT8)
    if (!p.partial) put_scales<64 * XF, 128 * WH>(scales.t, fetched, p.plain.bias, threadIdx.x, 512);
  // W0 and X of step 0 have landed
  wait_vm<(WH == 3 ? 4 : 2) * LOADS_W + LOADS_X>();
  wait_lds();
  wg_barrier();
  if (wn == 1) wg_barrier();

  v8bf w[2][4], x[XT][2][XFT];
  auto multiply = [&](auto pending, Sum<EPI>(&c)[XT][4][XFT]) __attribute__((always_inline)) {
    wait_vm<pending.value>();
    wait_lds();
    wg_barrier();
    __builtin_amdgcn_sched_barrier(0);
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int kk = 0; kk < 2; ++kk)
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int q = 0; q < XT; ++q)
#pragma unroll
          for (int j = 0; j < XFT; ++j) c[q][i][j] = mfma16(w[kk][i], x[q][kk][j], c[q][i][j]);
    __builtin_amdgcn_s_setprio(0);
    __builtin_amdgcn_sched_barrier(0);
    wg_barrier();
  };
  // loads issued after the ones that the phase after 0, after 1 (WH = 3) and after the last needs
  constexpr std::integral_constant<int, (WH == 3 ? 4 : 2) * LOADS_W + LOADS_X> after0{}, after_last{};
  constexpr std::integral_constant<int, 4 * LOADS_W + 2 * LOADS_X> after1{};
  auto step = [&](auto slot, auto other, int t) __attribute__((always_inline)) {
    const uint8_t* s = smem + slot * STAGE;
    if constexpr (XT == 2) rx.read2(x[0], x[1], s + WH * WPART, XPART);
    else rx.read(x[0], s + WH * WPART);
    rw.read(w, s);
    if constexpr (WH == 3) load_w(other, lw2, 2, t + 1);
    else load_w(other, lw1, 1, t + 1);
    multiply(after0, acc[0]);

    rw.read(w, s + WPART);
    load_w(slot, lw0, 0, t + 2);
    load_x(t + 2);
    if constexpr (WH == 3) {
      multiply(after1, acc[1]);
      rw.read(w, s + 2 * WPART);
      load_w(slot, lw1, 1, t + 2);
    }
    multiply(after_last, acc[WH - 1]);
  };
  if constexpr (PAIRS) {
    int t = 0;
    for (; t + 1 < KT; t += 2) {
      step(Even{}, Odd{}, t);
      step(Odd{}, Even{}, t + 1);
    }
    if (t < KT) step(Even{}, Odd{}, t);
  } else {
    for (int t = 0; t < KT; ++t) step(t & 1, (t + 1) & 1, t);
  }
  if (wn == 0) wg_barrier();
  wait_vm<0>();
  wg_barrier();  // every load has landed: the stages become the epilogue's

  uint8_t* region = smem + wave * (XFT * 2048);
#pragma unroll
  for (int h = 0; h < WH; ++h)
#pragma unroll
    for (int q = 0; q < XT; ++q) {
      const int64_t mb = m0 + q * XR + wm * (XFT * 16);
      Sum<EPI>(&a)[4][XFT] = acc[h][q];
      if constexpr (EPI == EPI_GATED) {
        v4f g[2][XFT], u[2][XFT];
#pragma unroll
        for (int j = 0; j < XFT; ++j) {
          g[0][j] = a[0][j];
          u[0][j] = a[1][j];
          g[1][j] = a[2][j];
          u[1][j] = a[3][j];
        }
        gated_epilogue<XFT>(g, u, p.gated, mb, n0 + h * 64 + wn * 32, lane, region);
      } else if constexpr (EPI == EPI_INT8) {
        const Int8Tile<64 * XF, 128 * WH>& t = scales.t;
        const int c = h * 128 + wn * 64;
        int8_epilogue<XFT>(a, p.partial ? nullptr : t.x + q * XR + wm * (XFT * 16), t.w + c, t.bias + c,
                           plain_of(p, slice), mb, n0 + c, lane, region);
      } else {
        plain_epilogue<XFT>(a, plain_of(p, slice), mb, n0 + h * 128 + wn * 64, lane, region);
      }
    }
}

// Sums the slices in order (V = v4i: exactly, then the scales), adds the bias, rounds once.
template <class V>
__global__ __launch_bounds__(256) void dense_reduce_kernel(const float* __restrict__ partial, int slices, PlainOut o,
                                                           Int8Scales sc) {
  const int64_t quads = o.m * o.n / 4;
  const int64_t at = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (at >= quads) return;
  const V* p = reinterpret_cast<const V*>(partial);
  V total = p[at];
  int i = 1;
  for (; i + 4 <= slices; i += 4) {  // four loads in flight
    const V a = p[at + i * quads], b = p[at + (i + 1) * quads], c = p[at + (i + 2) * quads],
              d = p[at + (i + 3) * quads];
    total += a;
    total += b;
    total += c;
    total += d;
  }
  for (; i < slices; ++i) total += p[at + i * quads];
  v4f s;
  if constexpr (std::is_same_v<V, v4i>) {
    const float xs = sc.x[at * 4 / o.n];
    const v4f ws = *reinterpret_cast<const v4f*>(sc.w + at * 4 % o.n), bias = bias4(o.bias, at * 4 % o.n);
#pragma unroll
    for (int j = 0; j < 4; ++j) s[j] = int8_value(total[j], xs, ws[j], bias[j]);
  } else {
    s = total;
  }
  if (std::is_same_v<V, v4f> && o.bias) {
    const uint2 b = *reinterpret_cast<const uint2*>(o.bias + at * 4 % o.n);
    s[0] += bf16_to_f32(b.x & 0xFFFFu);
    s[1] += bf16_to_f32(b.x >> 16);
    s[2] += bf16_to_f32(b.y & 0xFFFFu);
    s[3] += bf16_to_f32(b.y >> 16);
  }
  if (o.out_fmt == OUT_F32) reinterpret_cast<v4f*>(o.out)[at] = s;
  else reinterpret_cast<uint2*>(o.out)[at] = make_uint2(pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3]));
}

// Tiles of bm x `cover` rows; the workgroups of the grid, or -1 where the tiles
// pass what the kernels index (the entry points refuse such sizes).
int64_t set_tiles(DenseParams& p, int64_t bm, int64_t cover, int slices) {
  const int64_t tm = (p.rows_m + bm - 1) / bm, tn = (p.rows_n + cover - 1) / cover;
  const int64_t items = tm * tn * slices;
  if (items > ((int64_t)1 << 23) - 8) return -1;
  p.slices = slices;
  p.tiles_m = (int)tm;
  p.tiles_n = (int)tn;
  p.group = 8;
  return (items + 7) / 8 * 8;
}

template <int LX, int LW, int EPI, int BN, int BM, int WN, int WM, int S, int KS = 1>
hipError_t run_tile(DenseParams p, int slices, hipStream_t stream) {
  constexpr int bytes = KS * S * (BN + BM) * BK * 2;
  static_assert(bytes <= 160 * 1024, "LDS of a CU");
  auto* kernel = dense_tile_kernel<LX, LW, EPI, BN, BM, WN, WM, S, KS>;
  if (bytes > 65536) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != hipSuccess) return e;
  }
  constexpr int cover = EPI == EPI_GATED ? BN / 2 : BN;
  const int64_t grid = set_tiles(p, BM, cover, slices);
  if (grid < 0) return hipErrorInvalidValue;
  kernel<<<dim3((unsigned)grid), dim3(64 * WN * WM * KS), bytes, stream>>>(p);
  return hipGetLastError();
}

template <int LX, int LW, int EPI, int WH, int XF>
hipError_t run_wide(DenseParams p, int slices, hipStream_t stream) {
  constexpr int bytes = 2 * (WH * 128 + XF * 64) * BK * 2;
  static_assert(bytes <= 160 * 1024, "LDS of a CU");
  auto* kernel = dense_wide_kernel<LX, LW, EPI, WH, XF>;
  const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                           hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e != hipSuccess) return e;
  constexpr int cover = EPI == EPI_GATED ? 64 * WH : 128 * WH;
  const int64_t grid = set_tiles(p, 64 * XF, cover, slices);
  if (grid < 0) return hipErrorInvalidValue;
  kernel<<<dim3((unsigned)grid), dim3(512), bytes, stream>>>(p);
  return hipGetLastError();
}

// ---------------------------------------------------------------------------
// Choice of kernel and of the number of slices of the sum: the smallest
// modelled time.  A configuration covers bn x bm outputs per workgroup, per_cu
// workgroups fit on a CU.  us per stage of k of one round of tiles, measured
// (forward, k = 4096, 64 stages): `one` with few tiles, `all` with one on each of
// 256 CUs, `full` with every CU full; `lasting` in place of `full` in a run past
// 250 us, where power lowers the clock of the wide kernels; `cols` times as long with a
// COLS W operand (dx).  Examples (measured, us):
//   m = 300, f = 14336: 256x192 71, 256x256 86, 128x128 97, 128x64 108, 384x192 98
//   m = 517, f = 14336: 384x192 107, 256x192 135, 128x128 158, 256x256 161
//   m = 128, f = 14336: 128x64 48, 128x128 49 (KS = 2: 44), 256x256 76
//   m = 140, f = 4096: 64x64 30 (KS = 2: 25), 128x64 32 (25), 128x128 41 (35)
//   m = 33, k = f = 512: 64x64 5.3 (KS = 2: 4.6), 128x64 6.6 (5.8)
//   m = 8192, f = 14336: 256x256 1485, 256x192 1618, 384x192 1662, 128x128 1868 (one
//     box; the clock decides: others run the first in 1310 - 1410, and the model,
//     which only has to rank them, gives it 1566)
//   dx m = 1000, k = 2048, f = 5632: 128x128 in 1, 2, 4, 8 slices 118, 73, 55, 67,
//     256x256 211, 122, 76, 59;  m = 4096, k = f = 2048: 128x128 63, 256x192 85
// Slices (plain outputs only) add a pass over their binary32 partial sums.
// ---------------------------------------------------------------------------
// _K2: two groups of wavefronts, each with half of k (KS = 2)
enum {
  CFG_WIDE = 0,
  CFG_WIDE_192,
  CFG_WIDE_384,
  CFG_128,
  CFG_128x64,
  CFG_64,
  CFG_128_K2,
  CFG_128x64_K2,
  CFG_64_K2,
  CFG_64_K2_DEEP,  // four stages instead of two; 8-bit integers only
  CFG_COUNT
};
struct Config {
  const char* name;
  int bn, bm, per_cu;
  bool rows_x;  // built for X by rows only
  double one, all, full, lasting, fixed, cols;
};
constexpr Config kConfigs[CFG_COUNT] = {
    {"wide_256x256", 256, 256, 1, false, 0.95, 1.37, 1.37, 1.66, 5.6, 1.0},
    {"wide_256x192", 256, 192, 1, true, 0.80, 1.06, 1.06, 1.34, 5.0, 1.06},
    {"wide_384x192", 384, 192, 1, true, 1.16, 1.60, 1.60, 2.06, 7.0, 1.04},
    {"tile_128x128", 128, 128, 2, false, 0.58, 0.76, 1.05, 1.05, 3.7, 1.0},
    {"tile_128x64", 128, 64, 2, false, 0.45, 0.51, 0.67, 0.67, 3.8, 1.0},
    {"tile_64x64", 64, 64, 3, false, 0.36, 0.40, 0.59, 0.59, 3.0, 1.0},
    {"tile_128x128_k2", 128, 128, 1, true, 0.45, 0.58, 0.58, 0.58, 4.0, 1.0},
    {"tile_128x64_k2", 128, 64, 1, true, 0.30, 0.34, 0.34, 0.34, 4.0, 1.0},
    {"tile_64x64_k2", 64, 64, 2, true, 0.23, 0.32, 0.42, 0.42, 3.0, 1.0},
    {}};
// The same kernels on 8-bit integers (stages of 128 k), measured with 64, 256 and full
// rounds of tiles at k = 4096 and 12288; the epilogue's share of `fixed` is larger, as
// the tiles of a given k take half as many stages.  With half the stages a tile waits
// out more of its latencies, so the 64 x 64 tiles with two groups of wavefronts have a
// form of four stages (m = 128, n = k = 4096 15.2 -> 11.6 us in a graph, 100 x 5648 x 2080 10.9
// -> 10.0, 60 x 14336 x 4096 14.9 -> 13.4).
constexpr Config kInt8Configs[CFG_COUNT] = {
    {"wide_256x256", 256, 256, 1, false, 0.98, 1.50, 1.50, 1.50, 9.5, 1.0},
    {"wide_256x192", 256, 192, 1, true, 0.82, 1.20, 1.20, 1.25, 8.5, 1.0},
    {"wide_384x192", 384, 192, 1, true, 1.32, 1.90, 1.90, 1.90, 8.5, 1.0},
    {"tile_128x128", 128, 128, 2, false, 0.68, 0.70, 1.30, 1.45, 6.0, 1.0},
    {"tile_128x64", 128, 64, 2, false, 0.41, 0.43, 0.62, 0.70, 5.5, 1.0},
    {"tile_64x64", 64, 64, 3, false, 0.31, 0.32, 0.62, 0.70, 4.5, 1.0},
    {"tile_128x128_k2", 128, 128, 1, true, 0.52, 0.54, 0.54, 0.60, 7.0, 1.0},
    {"tile_128x64_k2", 128, 64, 1, true, 0.33, 0.35, 0.35, 0.40, 5.5, 1.0},
    {"tile_64x64_k2", 64, 64, 2, true, 0.35, 0.35, 0.40, 0.45, 3.5, 1.0},
    {"tile_64x64_k2_deep", 64, 64, 1, true, 0.17, 0.23, 0.23, 0.26, 3.6, 1.0}};
struct Choice {
  int config, slices;
  int64_t k_per_split;
  double us;  // modelled
};

double model_us(const Config& g, uint32_t tiles, uint32_t stages, bool cols_w) {
  const uint32_t slots = 256 * g.per_cu, rounds = tiles / slots, rest = tiles % slots;
  const double tail = rest == 0     ? 0
                      : rest <= 256 ? g.one + (g.all - g.one) * rest / 256
                                    : g.all + (g.full - g.all) * (rest - 256) / (slots - 256);
  const double fixed = g.fixed * (rounds + (rest != 0));
  const double us = (cols_w ? g.cols : 1.0) * stages;
  const double t = (rounds * g.full + tail) * us;
  return fixed + (t < 250 ? t : t * g.lasting / g.full);
}

// n: columns of the output's tiles (2 f when gated).  lx, lw: the operands'
// layouts.  can_slice: a plain output.  (On the way of every call: 32-bit
// divisions, and no slices where the tiles alone make four rounds.)
Choice choose(int64_t m, int64_t n, int64_t k, int lx, int lw, bool can_slice, const Config* configs = kConfigs) {
  const uint32_t stages = (uint32_t)((k + BK - 1) / BK);
  uint32_t tiles[CFG_COUNT];
  const int count = configs == kInt8Configs ? CFG_COUNT : CFG_64_K2_DEEP;
  for (int c = 0; c < count; ++c) {
    const uint32_t bm = configs[c].bm, bn = configs[c].bn;
    tiles[c] = (((uint32_t)m + bm - 1) / bm) * (((uint32_t)n + bn - 1) / bn);
  }
  Choice best{CFG_64, 1, k, 1e300};
  const uint32_t most = can_slice && m * n <= ((int64_t)1 << 30) ? 16 : 1;
  for (uint32_t s = 1; s <= most; ++s) {
    const uint32_t per = s == 1 ? stages : (stages + s - 1) / s;
    if (s > 1 && per < 8) break;
    if (s > 1 && (stages + per - 1) / per != s) continue;
    const double join = s > 1 ? 3.0 + 8.0 * s * m * n / 6e6 : 0.0;
    if (join >= best.us) break;
    for (int c = 0; c < count; ++c) {
      const Config& g = configs[c];
      if ((g.rows_x && lx != ROWS) || (s > 1 && tiles[c] * s > 1024)) continue;
      if (c >= CFG_128_K2 && per < 2) continue;  // nothing for the second group
      // with few stages the stores are most of the time, and only where a CU
      // holds several workgroups does another's work go on meanwhile (128x128
      // against 256x256, m = 8192, f = 14336, k = 64: 92, 111 us; dW k = 4096, f =
      // 14336: m = 64 51, 57; m = 190 75, 79; m = 250 84, 82..90; m = 300 98, 91)
      if (c <= CFG_WIDE_384 && per < 4) continue;
      const double t = model_us(g, tiles[c] * s, per, lw == COLS) + join;
      if (t < best.us) best = Choice{c, (int)s, s == 1 ? k : (int64_t)per * BK, t};
    }
  }
  return best;
}

template <int LX, int LW, int EPI>
hipError_t run_dense(DenseParams p, const Choice& c, void* workspace, hipStream_t stream) {
  p.k_per_split = c.k_per_split;
  p.partial = c.slices > 1 ? static_cast<float*>(workspace) : nullptr;
  hipError_t e = hipErrorInvalidValue;
  switch (c.config) {
    case CFG_WIDE: e = run_wide<LX, LW, EPI, 2, 4>(p, c.slices, stream); break;
    case CFG_WIDE_192:
      if constexpr (LX == ROWS) e = run_wide<LX, LW, EPI, 2, 3>(p, c.slices, stream);
      break;
    case CFG_WIDE_384:
      if constexpr (LX == ROWS) e = run_wide<LX, LW, EPI, 3, 3>(p, c.slices, stream);
      break;
    case CFG_128_K2:
      if constexpr (LX == ROWS) e = run_tile<LX, LW, EPI, 128, 128, 2, 2, 2, 2>(p, c.slices, stream);
      break;
    case CFG_128x64_K2:
      if constexpr (LX == ROWS) e = run_tile<LX, LW, EPI, 128, 64, 2, 2, 3, 2>(p, c.slices, stream);
      break;
    case CFG_64_K2:
      if constexpr (LX == ROWS) e = run_tile<LX, LW, EPI, 64, 64, 1, 4, 2, 2>(p, c.slices, stream);
      break;
    case CFG_64_K2_DEEP:
      if constexpr (EPI == EPI_INT8) e = run_tile<LX, LW, EPI, 64, 64, 1, 4, 4, 2>(p, c.slices, stream);
      break;
    case CFG_128: e = run_tile<LX, LW, EPI, 128, 128, 2, 2, 2>(p, c.slices, stream); break;
    case CFG_128x64: e = run_tile<LX, LW, EPI, 128, 64, 2, 2, 3>(p, c.slices, stream); break;
    default: e = run_tile<LX, LW, EPI, 64, 64, 1, 4, 3>(p, c.slices, stream);
  }
  if (e != hipSuccess || c.slices == 1) return e;
  const int64_t quads = p.plain.m * p.plain.n / 4;
  dense_reduce_kernel<Sum<EPI>>
      <<<dim3((unsigned)((quads + 255) / 256)), dim3(256), 0, stream>>>(p.partial, c.slices, p.plain, p.scales);
  return hipGetLastError();
}

// The choice of each product, for its launch, its workspace and its name.
Choice choose_gated(int64_t m, int64_t k, int64_t f) { return choose(m, 2 * f, k, ROWS, ROWS, false); }
Choice choose_mxfp4(int64_t m, int64_t n, int64_t k) { return choose(m, n, k, ROWS, CODES, true); }
Choice choose_int8(int64_t m, int64_t n, int64_t k) { return choose(m, n, k / 2, ROWS, ROWS, true, kInt8Configs); }
Choice choose_dx(int64_t m, int64_t k, int64_t f2) { return choose(m, k, f2, ROWS, COLS, true); }
Choice choose_dw(int64_t m, int64_t k, int64_t f2) { return choose(f2, k, m, COLS, COLS, false); }

int64_t slice_bytes(const Choice& c, int64_t m, int64_t n) { return c.slices > 1 ? c.slices * m * n * 4 : 0; }

DenseKernel named(const Choice& c, const Config* configs = kConfigs) { return {configs[c.config].name, c.slices}; }

}  // namespace

DenseKernel dense_gated_kernel(int64_t m, int64_t k, int64_t f) { return named(choose_gated(m, k, f)); }
DenseKernel dense_mxfp4_kernel(int64_t m, int64_t n, int64_t k) { return named(choose_mxfp4(m, n, k)); }
DenseKernel dense_dx_kernel(int64_t m, int64_t k, int64_t f2) { return named(choose_dx(m, k, f2)); }
DenseKernel dense_dw_kernel(int64_t m, int64_t k, int64_t f2) { return named(choose_dw(m, k, f2)); }

DenseKernel dense_int8_kernel(int64_t m, int64_t n, int64_t k) { return named(choose_int8(m, n, k), kInt8Configs); }

double dense_us(int64_t m, int64_t n, int64_t k, bool fp4, bool gated) {
  return choose(m, n, k, ROWS, fp4 ? CODES : ROWS, !gated).us;
}

double dense_int8_us(int64_t m, int64_t n, int64_t k) { return choose_int8(m, n, k).us; }

// Workspace: the slices' partial sums.
int64_t dense_nt_workspace_bytes(int64_t m, int64_t n, int64_t k) { return slice_bytes(choose_mxfp4(m, n, k), m, n); }
int64_t dense_dx_workspace_bytes(int64_t m, int64_t k, int64_t f2) { return slice_bytes(choose_dx(m, k, f2), m, k); }

int64_t dense_int8_workspace_bytes(int64_t m, int64_t n, int64_t k) { return slice_bytes(choose_int8(m, n, k), m, n); }

hipError_t launch_gated_dense(const GatedArgs& a, hipStream_t stream) {
  DenseParams p{};
  p.x = a.x;
  p.w = static_cast<const uint16_t*>(a.w);
  p.w_scale = a.w_scale;
  p.ldx = p.ldw = a.k;
  p.rows_m = a.m;
  p.rows_n = a.f;
  p.k = a.k;
  p.gated = GatedOut{a.h, a.gu, a.gu_scale, a.m, a.f, a.act, a.gu_fmt};
  const Choice c = choose_gated(a.m, a.k, a.f);
  return a.w_scale ? run_dense<ROWS, CODES, EPI_GATED>(p, c, nullptr, stream)
                   : run_dense<ROWS, ROWS, EPI_GATED>(p, c, nullptr, stream);
}

hipError_t launch_mxfp4_dense(const StreamArgs& a, void* workspace, hipStream_t stream) {
  DenseParams p{};
  p.x = a.x;
  p.w = static_cast<const uint16_t*>(a.w);
  p.w_scale = a.w_scale;
  p.ldx = a.k;
  p.rows_m = a.m;
  p.rows_n = a.rows;
  p.k = a.k;
  p.plain = PlainOut{a.out, a.bias, a.m, a.rows, a.out_fmt};
  return run_dense<ROWS, CODES, EPI_PLAIN>(p, choose_mxfp4(a.m, a.rows, a.k), workspace, stream);
}

hipError_t launch_int8_dense(const Int8Args& a, void* workspace, hipStream_t stream) {
  DenseParams p{};
  p.x = reinterpret_cast<const uint16_t*>(a.xq);
  p.w = reinterpret_cast<const uint16_t*>(a.wq);
  p.ldx = p.ldw = a.k / 2;
  p.rows_m = a.m;
  p.rows_n = a.n;
  p.k = a.k / 2;
  p.plain = PlainOut{a.out, a.bias, a.m, a.n, a.out_fmt};
  p.scales = Int8Scales{a.xs, a.ws};
  return run_dense<ROWS, ROWS, EPI_INT8>(p, choose_int8(a.m, a.n, a.k), workspace, stream);
}

hipError_t launch_dense_dx(const uint16_t* dgu, const uint16_t* w, int64_t m, int64_t k, int64_t f2, uint16_t* dx,
                           void* workspace, hipStream_t stream) {
  DenseParams p{};
  p.x = dgu;
  p.w = w;
  p.ldx = f2;
  p.ldw = k;
  p.rows_m = m;
  p.rows_n = k;
  p.k = f2;
  p.plain = PlainOut{dx, nullptr, m, k, OUT_BF16};
  return run_dense<ROWS, COLS, EPI_PLAIN>(p, choose_dx(m, k, f2), workspace, stream);
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
  p.k = m;
  p.plain = PlainOut{dw, nullptr, f2, k, OUT_BF16};
  return run_dense<COLS, COLS, EPI_PLAIN>(p, choose_dw(m, k, f2), nullptr, stream);
}

}  // namespace sfr

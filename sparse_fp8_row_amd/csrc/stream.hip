// Products of a few activation rows with a weight that is read once: the
// decode forms of the gated block (bf16 or 4-bit weight) and of the 4-bit
// linear layer, and the linear layer in 8-bit integers.  Bound by reading the weight.
//
// A workgroup owns 16 RT weight rows and up to 16 activation rows (grid y).
// Its wavefronts take units of UK k in turn and add their binary32 sums in a
// fixed order through LDS at the end.  A wavefront streams its units through
// LDS of its own, D - 1 units ahead, with global -> LDS loads in which
// neighbouring lanes read neighbouring 16 bytes, and waits only for its own
// loads: there is no barrier before the end.  (Loads straight into the operand
// layout, with 16 rows under 16 neighbouring lanes, make one cache access per
// lane: 64 of them per 1 KB of weight and four times that for 16 activation
// rows, which held the 4-bit kernels to 1.5 - 3.3 TB/s.)
//
// The product runs on v_mfma_f32_16x16x32_bf16 with the weight as A operand:
// lane l holds weight row l % 16.  The order of k inside a step is free as long
// as both operands agree, so each lane takes contiguous 16-byte chunks:
//   4-bit: 32 codes, one block with one scale, per step of 128 k; instruction j
//     takes codes 8 j .. 8 j + 7, decoded (exactly) to bf16 with the scale applied
//     by the converter: k = 32 (l / 16) + 8 j ..;
//   bf16: k = 32 j + 8 (l / 16) ..
//   8-bit integers (weight and activation): as bf16 rows of half as many elements.
// Gated: row tiles alternate between gate and up rows, so act(g) * u is
// formed from the sums before anything is rounded.
#include <type_traits>

#include "sfr_dense.hpp"

namespace sfr {
namespace {

// R: activation rows in LDS (a power of two, at least the workgroup's).
template <bool FP4, int RT, int R, int NW, int D>
struct Stream {
  static constexpr int UK = FP4 ? 256 : 128;      // k of one unit
  static constexpr int WROW = FP4 ? UK / 2 : UK * 2, XROW = UK * 2;
  static constexpr int WL = 16 * WROW / 1024;     // loads of a row tile
  static constexpr int SL = FP4 ? 16 * (UK / 32) / 64 : 0;
  static constexpr int XL = (R * XROW + 1023) / 1024;
  static constexpr int LOADS = RT * (WL + SL) + XL;
  static constexpr int TILE = WL * 1024 + SL * 256, UNIT = RT * TILE + XL * 1024;
  static constexpr int RED = NW * RT * R * 16 * 4;
  static constexpr int BYTES = NW * D * UNIT > RED ? NW * D * UNIT : RED;
  static_assert((D - 1) * LOADS < 64, "wait counts");
};

template <bool FP4, bool GATED, int RT, int R, int NW, int D, bool NT, bool I8>
__global__ __launch_bounds__(64 * NW) void stream_kernel(StreamArgs p) {
  using S = Stream<FP4, RT, R, NW, D>;
  using Sum = std::conditional_t<I8, v4i, v4f>;
  using Part = std::conditional_t<I8, int, float>;
  static_assert(!I8 || (!FP4 && !GATED), "8-bit integers: the linear layer");
  static_assert(!GATED || RT % 2 == 0, "row tiles come in pairs");
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, lg = lane >> 4;
  const int64_t m0 = (int64_t)blockIdx.y * 16;
  const int mr = (int)min(p.m - m0, (int64_t)16);
  const int K = (int)(I8 ? p.k / 2 : p.k), wrow = FP4 ? K / 2 : K * 2;
  const int64_t tile0 = (int64_t)blockIdx.x * (GATED ? RT / 2 : RT), tiles = p.rows / 16;

  // tiles past the last one read the last one (and are not stored)
  __amdgpu_buffer_rsrc_t rw[RT], rs[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    const int64_t row = min(tile0 + (GATED ? t >> 1 : t), tiles - 1) * 16 + (GATED && (t & 1) ? p.rows : 0);
    rw[t] = buf_rsrc(static_cast<const uint8_t*>(p.w) + row * wrow, kPastRange);
    if constexpr (FP4) rs[t] = buf_rsrc(p.w_scale + row * (K / 32), kPastRange);
  }
  const __amdgpu_buffer_rsrc_t rx = buf_rsrc(p.x + m0 * K, kPastRange);

  uint8_t* const mine = smem + wave * (D * S::UNIT);
  // unit u into buffer slot; what lies past K (or the last activation row) reads zeros
  auto issue = [&](int slot, int u) __attribute__((always_inline)) {
    uint8_t* b = mine + slot * S::UNIT;
    const int left = K - u * S::UK;  // may be negative: every lane masked
    constexpr int WC = S::WROW / 16, WPL = 64 / WC;  // chunks per row, rows per load
#pragma unroll
    for (int t = 0; t < RT; ++t) {
#pragma unroll
      for (int j = 0; j < S::WL; ++j) {
        const int row = j * WPL + lane / WC, c = (lane % WC) ^ (row & 7);
        buf_to_lds<NT>(rw[t], b + t * S::TILE + j * 1024,
                   c * (FP4 ? 32 : 8) < left ? row * wrow + u * S::WROW + c * 16 : kPastRange);
      }
#pragma unroll
      for (int j = 0; j < S::SL; ++j) {
        const int row = j * 8 + (lane >> 3), c = lane & 7;
        buf_byte_to_lds(rs[t], b + t * S::TILE + S::WL * 1024 + j * 256,
                        c * 32 < left ? row * (K / 32) + u * 8 + c : kPastRange);
      }
    }
    constexpr int XC = S::XROW / 16, XPL = 64 / XC;
#pragma unroll
    for (int j = 0; j < S::XL; ++j) {
      const int row = j * XPL + lane / XC, c = (lane % XC) ^ (row & 7);
      buf_to_lds(rx, b + RT * S::TILE + j * 1024,
                 row < mr && c * 8 < left ? row * (K * 2) + u * S::XROW + c * 16 : kPastRange);
    }
  };

  Sum acc[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) acc[t] = Sum{};

  const int units = (K + S::UK - 1) / S::UK;
#pragma unroll
  for (int i = 0; i < D - 1; ++i) issue(i, wave + i * NW);
  const int xr = min(r16, R - 1);
  int slot = 0;
  for (int u = wave; u < units; u += NW) {
    wait_lds();  // the slot to be refilled has been read
    issue(slot == 0 ? D - 1 : slot - 1, u + (D - 1) * NW);
    wait_vm<(D - 1) * S::LOADS>();
    asm volatile("" ::: "memory");
    const uint8_t* b = mine + slot * S::UNIT;
    const uint8_t* xb = b + RT * S::TILE + xr * S::XROW;
#pragma unroll
    for (int s = 0; s < S::UK / 128; ++s) {
      v8bf x[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = FP4 ? 16 * s + 4 * lg + j : 4 * j + lg;
        x[j] = *reinterpret_cast<const v8bf*>(xb + 16 * (c ^ (xr & 7)));
      }
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        const uint8_t* wb = b + t * S::TILE + r16 * S::WROW;
        if constexpr (FP4) {
          const v4i q = *reinterpret_cast<const v4i*>(wb + 16 * ((4 * s + lg) ^ (r16 & 7)));
          const uint32_t e = *reinterpret_cast<const uint32_t*>(b + t * S::TILE + S::WL * 1024 +
                                                                4 * (r16 * 8 + 4 * s + lg));
          const float f = mx_scale_value(e);
#pragma unroll
          for (int j = 0; j < 4; ++j)
            acc[t] = mfma16(__builtin_bit_cast(v8bf, mx_widen8_e2m1((uint32_t)q[j], f)), x[j], acc[t]);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            acc[t] = mfma16(*reinterpret_cast<const v8bf*>(wb + 16 * ((4 * j + lg) ^ (r16 & 7))), x[j], acc[t]);
        }
      }
    }
    slot = slot == D - 1 ? 0 : slot + 1;
  }
  wait_vm<0>();
  wait_lds();
  wg_barrier();  // no load in flight, no read pending: the buffers become the sums'

  Part* const red = reinterpret_cast<Part*>(smem);  // [NW][RT][R][16]
#pragma unroll
  for (int t = 0; t < RT; ++t)
    if (r16 < mr) *reinterpret_cast<Sum*>(red + ((wave * RT + t) * R + r16) * 16 + 4 * lg) = acc[t];
  wait_lds();
  wg_barrier();
  constexpr int OT = GATED ? RT / 2 : RT;
  for (int i = threadIdx.x; i < OT * 16 * mr; i += 64 * NW) {
    const int n = i % 16, t = i / 16 % OT, m = i / (16 * OT);
    const int64_t col = (tile0 + t) * 16 + n;
    Part sum = 0;
    float u = 0.f;
#pragma unroll
    for (int v = 0; v < NW; ++v) {
      sum += red[((v * RT + (GATED ? 2 * t : t)) * R + m) * 16 + n];
      if constexpr (GATED) u += red[((v * RT + 2 * t + 1) * R + m) * 16 + n];
    }
    float y = (float)sum;
    if constexpr (GATED) {
      y = u * (p.act == ACT_SILU        ? act_value<ACT_SILU>(y)
               : p.act == ACT_GELU_TANH ? act_value<ACT_GELU_TANH>(y)
                                        : act_value<ACT_RELU>(y));
    }
    if (col < p.rows) {
      if constexpr (I8) y = int8_value(sum, p.xs[m0 + m], p.ws[col], p.bias ? bf16_to_f32(p.bias[col]) : -0.f);
      if (!I8 && p.bias) y += bf16_to_f32(p.bias[col]);
      const int64_t at = (m0 + m) * p.rows + col;
      if (p.out_fmt == OUT_F32) static_cast<float*>(p.out)[at] = y;
      else static_cast<uint16_t*>(p.out)[at] = (uint16_t)pack_bf16x2(y, 0.f);
    }
  }
}

template <bool FP4, bool GATED, int RT, int R, int NW, int D, bool NT = false, bool I8 = false>
hipError_t run_stream(const StreamArgs& a, hipStream_t stream) {
  constexpr int cover = (GATED ? RT / 2 : RT) * 16, bytes = Stream<FP4, RT, R, NW, D>::BYTES;
  static_assert(bytes <= 160 * 1024, "LDS of a CU");
  auto* kernel = stream_kernel<FP4, GATED, RT, R, NW, D, NT, I8>;
  if constexpr (bytes > 65536) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != hipSuccess) return e;
  }
  const dim3 grid((unsigned)((a.rows + cover - 1) / cover), (unsigned)((a.m + 15) / 16));
  kernel<<<grid, dim3(64 * NW), bytes, stream>>>(a);
  return hipGetLastError();
}

}  // namespace

// Whether the weight is streamed per 16 activation rows or multiplied in tiles
// that hold every row: up to 8 rows always, up to eight passes over the weight
// where the modelled time is less than the tiles' (us: what each 16 weight rows
// and each byte of the weight cost a pass, within a quarter of what 12 sizes
// from k = 704 to 8192 took; the tiles walk all of k by themselves, but read the
// weight once).
// Measured, stream against tiles, us:
//   bf16, k = 4096, f = 4096: 17 rows 15.9, 22.1; 33 rows 25.8, 22.2
//         k = 704, f = 9248: 17 rows 11.9, 8.7
//   4-bit linear, k = 4096, n = 8192: 32 rows 9.6, 15.6; 100 rows 25.9, 22.9
//   4-bit gated, k = 4096, f = 4096: 64 rows 15.3, 19.6; 100 rows 27.0, 20.7
//         k = 704, f = 9248: 16 rows 5.4, 8.6; 48 rows 12.5, 8.6
bool stream_rows(int64_t m, int64_t n, int64_t k, bool fp4, bool gated) {
  const int64_t passes = (m + 15) / 16;
  if (m <= 8) return true;
  if (passes > 8) return false;
  const double bytes = (double)n * k * (fp4 ? 0.5 : 2.0);
  const double pass = fp4 ? 0.0015 / 16 * n + bytes / 5.6e6 : bytes / 9e6;
  const double tiles = dense_us(m, n, k, fp4, gated), read = bytes / 4.8e6 + 3;
  return 3 + passes * pass <= (tiles > read ? tiles : read);
}

// The same for 8-bit integers (streamed, less 2.5 us of a graph's launch: 12 rows, n = k
// = 4096 3.9 us; 24, 8192 x 4096 11.5; 40, 14336 x 2080 19.4; 100, 1040 x 8192 11.5; 128, 4096 x
// 4096 16.6).  Stream against tiles, us: 20 rows, 4096 x 4096 6.8, 9.7; 40, 2080 x 2080 5.6, 7.3;
// 100, 1040 x 8192 14.0, 10.7; 128, 4096 x 4096 19.1, 11.5.
bool stream_rows_int8(int64_t m, int64_t n, int64_t k) {
  const int64_t passes = (m + 15) / 16;
  if (m <= 8) return true;
  if (passes > 8) return false;
  return 1.5 + passes * ((double)n * k / 6.2e6) <= dense_int8_us(m, n, k);
}

namespace {

// One form of the kernel, with its name.
struct Form {
  const char* name;
  hipError_t (*run)(const StreamArgs&, hipStream_t);
};

// Two buffers everywhere: more workgroups on a CU gain more than deeper ones.
constexpr Form kBf16R2{"stream_bf16_r2", run_stream<false, true, 2, 2, 3, 2, true>};
constexpr Form kBf16R8{"stream_bf16_r8", run_stream<false, true, 2, 8, 3, 2, true>};
constexpr Form kBf16R16{"stream_bf16_r16", run_stream<false, true, 2, 16, 3, 2, true>};
constexpr Form kBf16Passes{"stream_bf16_passes", run_stream<false, true, 2, 16, 3, 2>};
constexpr Form kGatedR2{"stream_4bit_gated_r2", run_stream<true, true, 2, 2, 4, 2>};
constexpr Form kGatedR8{"stream_4bit_gated_r8", run_stream<true, true, 2, 8, 4, 2>};
constexpr Form kGatedT2W4{"stream_4bit_gated_t2w4", run_stream<true, true, 2, 16, 4, 2>};
constexpr Form kGatedT4W3{"stream_4bit_gated_t4w3", run_stream<true, true, 4, 16, 3, 2>};
constexpr Form kGatedT2W2{"stream_4bit_gated_t2w2", run_stream<true, true, 2, 16, 2, 2>};
constexpr Form kGatedT4W2{"stream_4bit_gated_t4w2", run_stream<true, true, 4, 16, 2, 2>};
constexpr Form kR2T1W8{"stream_4bit_r2_t1w8", run_stream<true, false, 1, 2, 8, 2>};
constexpr Form kR2T1W4{"stream_4bit_r2_t1w4", run_stream<true, false, 1, 2, 4, 2>};
constexpr Form kR8T1W8{"stream_4bit_r8_t1w8", run_stream<true, false, 1, 8, 8, 2>};
constexpr Form kR8T2W4{"stream_4bit_r8_t2w4", run_stream<true, false, 2, 8, 4, 2>};
constexpr Form kT1W4{"stream_4bit_t1w4", run_stream<true, false, 1, 16, 4, 2>};
constexpr Form kT2W4{"stream_4bit_t2w4", run_stream<true, false, 2, 16, 4, 2>};
constexpr Form kT2W3{"stream_4bit_t2w3", run_stream<true, false, 2, 16, 3, 2>};
constexpr Form kT2W2{"stream_4bit_t2w2", run_stream<true, false, 2, 16, 2, 2>};
constexpr Form kI8R2{"stream_int8_r2", run_stream<false, false, 1, 2, 8, 3, false, true>};
constexpr Form kI8R8T1W8{"stream_int8_r8_t1w8", run_stream<false, false, 1, 8, 8, 2, false, true>};
constexpr Form kI8R8T2W3{"stream_int8_r8_t2w3", run_stream<false, false, 2, 8, 3, 2, false, true>};
constexpr Form kI8T1W4{"stream_int8_t1w4", run_stream<false, false, 1, 16, 4, 2, false, true>};
constexpr Form kI8T2W3{"stream_int8_t2w3", run_stream<false, false, 2, 16, 3, 2, false, true>};

// The form of a call.
//
// R by the rows of a workgroup: the activation's share of LDS and its loads
// grow with R, so 2 and 8 rows have forms of their own (n = 4096, k = 4096,
// 4-bit: 3.3, 3.9, 4.7 us for 1, 8, 16 rows; 8 rows in the 16-row form 4.6).
//
// A bf16 weight, read once, is loaded non-temporally (k = 4096, f = 14336: one
// row 41.5 -> 38.3 us, 16 rows 44.4 -> 39.6; with more rows later passes find
// it in the caches).  A 4-bit weight is not: 16 rows 16.9 -> 18.8 us where the
// caches hold it, 20.6 -> 20.1 where they do not.
//
// Row tiles and wavefronts of a workgroup for a 4-bit weight by the number of
// (pairs of) row tiles: as many wavefronts per tile as fit where each CU has one
// workgroup at most, else fewer of them, so that two or three workgroups fit on
// a CU, and two tiles to share an activation's loads.  (The gated forms of up
// to 8 rows and the bf16 forms are one for every number of tiles: they were
// timed at k = 4096, f = 14336 alone.)  Measured, us, the first form against the
// one taken: linear n = 28672, k = 4096: 1 row 12.8, 11.2; 8 rows 20.9, 13.8; 16
// rows 25.3, 18.1;  n = 8192, k = 4096: 8 rows 12.3, 8.2 (n = 16384); 16 rows
// 8.3, 6.3, 32 rows 15.0, 9.7;  n = 4096: 8 rows 4.0 against 4.9, 16 rows 4.7
// against 5.7;  gated k = 4096, 16 rows: f = 4096 6.4 against 9.2, f = 8192 10.4, 10.0;
// k = 704, f = 9248: 8.5, 5.4;  k = 4096, f = 4096, 64 rows: 19.4, 15.5.
//
// 8-bit integers, by the same rule, us: 16 rows, n = 4096, k = 14336: one tile and four
// wavefronts 12.0, two tiles and three 12.8; n = 14336, k = 4096: 15.2, 13.0 (two and four
// 16.7); 8 rows: one and eight 11.7, two and three 12.0; 15.6, 12.3.  Up to two rows one
// tile and eight, three buffers: n = 4096, k = 28672 22.8 (two buffers 24.2), n = 14336
// 72.7 (76.0).
const Form& stream_form(const StreamArgs& a) {
  if (a.ws) {
    const bool few = a.rows / 16 * ((a.m + 15) / 16) <= 256;
    return a.m <= 2 ? kI8R2 : a.m <= 8 ? (few ? kI8R8T1W8 : kI8R8T2W3) : few ? kI8T1W4 : kI8T2W3;
  }
  if (!a.w_scale) return a.m <= 2 ? kBf16R2 : a.m <= 8 ? kBf16R8 : a.m <= 16 ? kBf16R16 : kBf16Passes;
  const int64_t tiles = a.rows / 16 * ((a.m + 15) / 16);
  if (a.gated) {
    if (a.m <= 2) return kGatedR2;
    if (a.m <= 8) return kGatedR8;
    return tiles <= 256 ? kGatedT2W4 : tiles <= 512 ? kGatedT4W3 : tiles <= 768 ? kGatedT2W2 : kGatedT4W2;
  }
  if (a.m <= 2) return tiles <= 256 ? kR2T1W8 : kR2T1W4;
  if (a.m <= 8) return tiles <= 256 ? kR8T1W8 : kR8T2W4;
  return tiles <= 256 ? kT1W4 : tiles <= 512 ? kT2W4 : tiles <= 1024 ? kT2W3 : kT2W2;
}

}  // namespace

const char* stream_name(const StreamArgs& a) { return stream_form(a).name; }

hipError_t launch_stream(const StreamArgs& a, hipStream_t stream) { return stream_form(a).run(a, stream); }

}  // namespace sfr

// Device building blocks of the dense bf16 products: operand tiles staged in
// LDS by global -> LDS buffer loads, read as matrix-instruction operands, and
// the epilogues that finish a wavefront's block.
//
// Every product is P[m][n] = sum_k X[m, k] W[n, k].  The W rows are the A
// operand of v_mfma_f32_16x16x32_bf16 and the X rows its B operand, so lane l
// holds P[m = l % 16][n = 4 (l / 16) .. + 3] of a 16 x 16 block: four
// consecutive outputs of one row.  Each operand is stored in one of two ways:
//   ROWS: row-major [rows][k] (k contiguous);
//   COLS: row-major [k][rows] (its transpose; rows contiguous).
// A ROWS operand is read from LDS with 16-byte reads, a COLS operand with the
// transposing 8-byte reads of gfx950 (lane i of 16 receives column i of a 4 x
// 16 block), so the gradients need no transposed copy of anything.
#pragma once

#include "sfr_launch.hpp"
#include "sfr_mx.hpp"

namespace sfr {

//   CODES: a 4-bit weight, row-major codes and block scales; decoded into the
//     ROWS layout of LDS by the wavefronts that load it.
enum { ROWS = 0, COLS = 1, CODES = 2 };

typedef __attribute__((address_space(3))) void* lds_void_t;

constexpr int BK = 64;  // k of one stage

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buf_rsrc(const void* base, int bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, bytes, 0x00020000);
}

// Lane l's 16 bytes at `voff` land at lds + 16 l.  The range check covers the
// whole offset (it is all in the vector offset): a lane past the range writes zeros.
// NT: non-temporal (data read once).
template <bool NT = false>
__device__ __forceinline__ void buf_to_lds(__amdgpu_buffer_rsrc_t r, uint8_t* lds, int voff) {
  const uint32_t a = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_void_t)lds);
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void_t)(uintptr_t)a, 16, voff, 0, 0, NT ? 2 : 0);
}
// One byte per active lane -> one dword in LDS at lds + 4 lane.
__device__ __forceinline__ void buf_byte_to_lds(__amdgpu_buffer_rsrc_t r, uint8_t* lds, int voff) {
  const uint32_t a = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_void_t)lds);
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void_t)(uintptr_t)a, 1, voff, 0, 0, 0);
}
constexpr int kPastRange = 0x7FFFFFF0;  // an offset past every descriptor's range

// s_waitcnt with only the vector-memory counter constrained.
template <int N>
__device__ __forceinline__ void wait_vm() {
  static_assert(N >= 0 && N < 64, "vmcnt");
  __builtin_amdgcn_s_waitcnt((N & 0xF) | ((N >> 4) << 14) | (0x7 << 4) | (0xF << 8));
}
__device__ __forceinline__ void wait_lds() { __builtin_amdgcn_s_waitcnt(0xC07F); }
// Workgroup barrier that keeps global loads in flight.
__device__ __forceinline__ void wg_barrier() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// ---------------------------------------------------------------------------
// LDS layouts of one operand tile of BR rows x BK.
//   ROWS: 128 bytes per row; 16-byte chunk c of row r at c ^ (r % 8), so the 8
//     lanes of one 128-byte LDS cycle (8 rows, one chunk) take all banks once.
//   COLS: BR * 2 bytes per k; 32 lanes of a transposing read take 32 bytes of
//     each of eight k (0 .. 3 and 8 .. 11 from a multiple of 16), so the
//     32-byte unit u of k sits at u ^ cols_swizzle(k): eight different units of
//     a 256-byte line of banks (BR = 64: a line holds two k, four units each).
// A 1 KB load covers 8 rows (ROWS) or 512 / BR of k (COLS); the swizzles are
// applied to the global address of each lane.
// ---------------------------------------------------------------------------
template <int BR>
__device__ __forceinline__ int cols_swizzle(int k) {
  return BR >= 128 ? (k & 3) | (((k >> 3) & 1) << 2) : ((k >> 1) & 1) | (((k >> 3) & 1) << 1);
}

// One operand's loads, shared evenly by NW wavefronts; load j = wave + q * NW.
// PAIR (ROWS only): the tile's rows alternate in groups of 16 between rows of
// the two halves of the weight ([Wg; Wu], `half` rows apart): gate rows f0 ..
// in groups 0, 2, .. and the same up rows in groups 1, 3, ..
template <int L, int BR, int NW, bool PAIR>
struct Loader {
  static constexpr int PER = BR / 8 / NW;
  static_assert(BR / 8 % NW == 0, "loads split evenly");
  static_assert(!PAIR || (L == ROWS && NW % 4 == 0), "a wavefront's loads stay in one half");
  const uint8_t* base;
  int64_t step;   // bytes per stage of k
  int voff[PER];  // past the range for rows that do not exist
  int first[PER];  // the load's first k in the stage
  int wave;

  // rows r0 .. of `rows`; ld elements between stored rows; k from k0 on
  __device__ __forceinline__ Loader(const uint16_t* p, int64_t ld, int64_t r0, int64_t rows, int64_t k0, int wave_,
                                    int lane)
      : wave(wave_) {
    const int n = (int)min(rows - r0, (int64_t)BR);
    if constexpr (L == ROWS) {
      const int part = PAIR ? (wave >> 1) & 1 : 0;
      base = reinterpret_cast<const uint8_t*>(p + (part * rows + r0) * ld + k0);
      step = BK * 2;
      const int chunk = (lane & 7) ^ (lane >> 3);
#pragma unroll
      for (int q = 0; q < PER; ++q) {
        const int j = wave + q * NW;
        const int row = (PAIR ? (j >> 2) * 16 + (j & 1) * 8 : j * 8) + (lane >> 3);
        voff[q] = row < n ? row * (int)(ld * 2) + chunk * 16 : kPastRange;
        first[q] = chunk * 8;
      }
    } else {
      static_assert(L != COLS || 512 % BR == 0, "whole k per load");
      constexpr int RPL = 512 / BR, CPR = 64 / RPL;  // k per load, 16-byte chunks per k
      base = reinterpret_cast<const uint8_t*>(p + k0 * ld + r0);
      step = BK * 2 * ld;
#pragma unroll
      for (int q = 0; q < PER; ++q) {
        const int k = (wave + q * NW) * RPL + lane / CPR;
        const int chunk = (lane % CPR) ^ (cols_swizzle<BR>(k) << 1);
        voff[q] = chunk * 8 < n ? k * (int)(ld * 2) + 16 * chunk : kPastRange;
        first[q] = k;
      }
    }
  }
  // Puts the next stage's loads in flight and moves on.  k_left: k not yet
  // loaded; what lies past it reads zeros.  Every lane that is not masked reads
  // inside the operand (rows are a multiple of 8 long), so the range is fixed.
  __device__ __forceinline__ void stage(uint8_t* lds, int k_left) {
    const __amdgpu_buffer_rsrc_t r = buf_rsrc(base, 0x7FFFFF00);
#pragma unroll
    for (int q = 0; q < PER; ++q) buf_to_lds(r, lds + (wave + q * NW) * 1024, first[q] < k_left ? voff[q] : kPastRange);
    base += step;
  }
};

// A 4-bit weight's loads: every thread of NW wavefronts holds E codes of one
// row, decodes them (exactly) to bf16 and writes them to LDS in the ROWS layout.
// fetch puts the next stage's codes in flight in register set P of DEPTH, put
// writes them: with two sets, taken in turn, codes are fetched two stages
// before they are written.  A fetch is exactly two loads (codes; scale), which
// the wait counts rely on.
template <int BR, int NW, bool PAIR, int DEPTH>
struct CodeLoader {
  static constexpr int E = BR * BK / (64 * NW), LOADS = 2;
  static_assert(E == 16 || E == 32, "8 or 16 bytes of codes, one block's scale");
  __amdgpu_buffer_rsrc_t rq, rs;
  int voff, soff, first, lds;
  bool exists;
  uint32_t xor1;
  v4i code[DEPTH];
  uint32_t scale[DEPTH];

  __device__ __forceinline__ CodeLoader(const void* q, const uint8_t* sc, int64_t k, int64_t r0, int64_t rows,
                                        int64_t k0, int wave, int lane) {
    constexpr int TPR = BK / E, G = 4 / TPR;  // threads per row, groups of 16 rows per wavefront
    first = lane % TPR * E;
    // PAIR: a wavefront's rows all belong to half wave % 2 of the weight
    const int part = PAIR ? wave & 1 : 0, group = (PAIR ? wave >> 1 : wave) * G + lane / (16 * TPR);
    const int row = group * 16 + lane / TPR % 16;  // from r0
    const int r = PAIR ? (2 * group + part) * 16 + lane / TPR % 16 : row;
    const int64_t at = part * rows + r0;
    rq = buf_rsrc(static_cast<const uint8_t*>(q) + at * (k / 2) + k0 / 2, kPastRange);
    rs = buf_rsrc(sc + at * (k / 32) + k0 / 32, kPastRange);
    exists = row < rows - r0;
    voff = row * (int)(k / 2) + first / 2;
    soff = row * (int)(k / 32) + first / 32;
    lds = r * 128;
    xor1 = (uint32_t)(r & 7);
  }
  template <int P>
  __device__ __forceinline__ void fetch(int k_left) {
    const bool in = exists && first < k_left;
    const int v = in ? voff : kPastRange;  // past the range: zeros
    if constexpr (E == 16) {
      typedef int v2i __attribute__((ext_vector_type(2)));
      const v2i c = __builtin_bit_cast(v2i, __builtin_amdgcn_raw_buffer_load_b64(rq, v, 0, 0));
      code[P][0] = c[0];
      code[P][1] = c[1];
    } else {
      code[P] = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(rq, v, 0, 0));
    }
    scale[P] = __builtin_amdgcn_raw_buffer_load_b8(rs, in ? soff : kPastRange, 0, 0);
    voff += BK / 2;
    soff += BK / 32;
  }
  // Written by asm: before an ordinary LDS store the compiler waits for the
  // global -> LDS loads in flight.  The caller waits for its LDS writes
  // (wait_lds) before the barrier that publishes them.
  template <int P>
  __device__ __forceinline__ void put(uint8_t* tile) const {
    const float f = mx_scale_value(scale[P] & 0xFFu);
    const uint32_t row = (uint32_t)(uintptr_t)(lds_void_t)tile + lds;
#pragma unroll
    for (int i = 0; i < E / 8; ++i) {
      typedef uint32_t v4u __attribute__((ext_vector_type(4)));
      const uint4 v = mx_widen8_e2m1((uint32_t)code[P][i], f);
      asm volatile("ds_write_b128 %0, %1" ::"v"(row + 16 * ((uint32_t)(first / 8 + i) ^ xor1)),
                   "v"(v4u{v.x, v.y, v.z, v.w})
                   : "memory");
    }
  }
};

// Transposing reads from LDS, four (at offsets O0 .. O3) from each of N
// addresses, and the wait for them.  One asm block: the builtin makes the
// compiler wait for every global -> LDS load in flight before each such read,
// which would end the prefetch; inside the block the reads have landed before
// anything uses their registers.
typedef uint32_t v2u __attribute__((ext_vector_type(2)));
template <int N, int O0, int O1, int O2, int O3>
__device__ __forceinline__ void read_tr(v2u (&r)[N][4], const uint32_t (&a)[N]) {
  static_assert(N == 1 || N == 2 || N == 4, "blocks written out below");
  if constexpr (N == 1) {
    asm volatile(
        "ds_read_b64_tr_b16 %0, %4 offset:%5\n\t"
        "ds_read_b64_tr_b16 %1, %4 offset:%6\n\t"
        "ds_read_b64_tr_b16 %2, %4 offset:%7\n\t"
        "ds_read_b64_tr_b16 %3, %4 offset:%8\n\t"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(r[0][0]), "=&v"(r[0][1]), "=&v"(r[0][2]), "=&v"(r[0][3])
        : "v"(a[0]), "n"(O0), "n"(O1), "n"(O2), "n"(O3)
        : "memory");
  } else if constexpr (N == 2) {
    asm volatile(
        "ds_read_b64_tr_b16 %0, %8 offset:%10\n\t"
        "ds_read_b64_tr_b16 %1, %8 offset:%11\n\t"
        "ds_read_b64_tr_b16 %2, %8 offset:%12\n\t"
        "ds_read_b64_tr_b16 %3, %8 offset:%13\n\t"
        "ds_read_b64_tr_b16 %4, %9 offset:%10\n\t"
        "ds_read_b64_tr_b16 %5, %9 offset:%11\n\t"
        "ds_read_b64_tr_b16 %6, %9 offset:%12\n\t"
        "ds_read_b64_tr_b16 %7, %9 offset:%13\n\t"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(r[0][0]), "=&v"(r[0][1]), "=&v"(r[0][2]), "=&v"(r[0][3]), "=&v"(r[1][0]), "=&v"(r[1][1]),
          "=&v"(r[1][2]), "=&v"(r[1][3])
        : "v"(a[0]), "v"(a[1]), "n"(O0), "n"(O1), "n"(O2), "n"(O3)
        : "memory");
  } else {
    asm volatile(
        "ds_read_b64_tr_b16 %0, %16 offset:%20\n\t"
        "ds_read_b64_tr_b16 %1, %16 offset:%21\n\t"
        "ds_read_b64_tr_b16 %2, %16 offset:%22\n\t"
        "ds_read_b64_tr_b16 %3, %16 offset:%23\n\t"
        "ds_read_b64_tr_b16 %4, %17 offset:%20\n\t"
        "ds_read_b64_tr_b16 %5, %17 offset:%21\n\t"
        "ds_read_b64_tr_b16 %6, %17 offset:%22\n\t"
        "ds_read_b64_tr_b16 %7, %17 offset:%23\n\t"
        "ds_read_b64_tr_b16 %8, %18 offset:%20\n\t"
        "ds_read_b64_tr_b16 %9, %18 offset:%21\n\t"
        "ds_read_b64_tr_b16 %10, %18 offset:%22\n\t"
        "ds_read_b64_tr_b16 %11, %18 offset:%23\n\t"
        "ds_read_b64_tr_b16 %12, %19 offset:%20\n\t"
        "ds_read_b64_tr_b16 %13, %19 offset:%21\n\t"
        "ds_read_b64_tr_b16 %14, %19 offset:%22\n\t"
        "ds_read_b64_tr_b16 %15, %19 offset:%23\n\t"
        "s_waitcnt lgkmcnt(0)"
        : "=&v"(r[0][0]), "=&v"(r[0][1]), "=&v"(r[0][2]), "=&v"(r[0][3]), "=&v"(r[1][0]), "=&v"(r[1][1]),
          "=&v"(r[1][2]), "=&v"(r[1][3]), "=&v"(r[2][0]), "=&v"(r[2][1]), "=&v"(r[2][2]), "=&v"(r[2][3]),
          "=&v"(r[3][0]), "=&v"(r[3][1]), "=&v"(r[3][2]), "=&v"(r[3][3])
        : "v"(a[0]), "v"(a[1]), "v"(a[2]), "v"(a[3]), "n"(O0), "n"(O1), "n"(O2), "n"(O3)
        : "memory");
  }
}

__device__ __forceinline__ v8bf join8(v2u lo, v2u hi) {
  typedef uint32_t v4u __attribute__((ext_vector_type(4)));
  return __builtin_bit_cast(v8bf, v4u{lo[0], lo[1], hi[0], hi[1]});
}

// Operand reads of NF 16-row fragments from `first` on of a tile of BR rows.
template <int L, int BR, int NF>
struct Reader {
  uint32_t at[NF];  // ROWS: the lane's row (the chunk is XORed in); COLS: the lane's whole address, kk = 0
  int lg, c;
  static constexpr int HI = 4 * BR * 2, KK = 32 * BR * 2;  // COLS: from lower to upper four k; from kk = 0 to 1
  __device__ __forceinline__ Reader(int first, int lane) {
    const int r16 = lane & 15;
    lg = lane >> 4;
    c = r16 & 7;
#pragma unroll
    for (int i = 0; i < NF; ++i) {
      if constexpr (L == ROWS) {
        at[i] = (first + i) * 2048 + r16 * 128;
      } else {
        const int k = 8 * lg + (r16 >> 2);
        at[i] = k * (BR * 2) + 32 * ((first + i) ^ cols_swizzle<BR>(k)) + 16 * ((r16 & 3) >> 1) + 8 * (r16 & 1);
      }
    }
  }
  // out[kk][i]: fragment i with k 32 kk .. 32 kk + 31 of the stage
  __device__ __forceinline__ void read(v8bf (&out)[2][NF], const uint8_t* tile) const {
    if constexpr (L == ROWS) {
#pragma unroll
      for (int kk = 0; kk < 2; ++kk)
#pragma unroll
        for (int i = 0; i < NF; ++i)
          out[kk][i] = *reinterpret_cast<const v8bf*>(tile + at[i] + 16 * ((kk * 4 + lg) ^ c));
    } else {
      const uint32_t base = (uint32_t)(uintptr_t)(lds_void_t)tile;
      uint32_t a[NF];
      v2u r[NF][4];
#pragma unroll
      for (int i = 0; i < NF; ++i) a[i] = base + at[i];
      read_tr<NF, 0, HI, KK, KK + HI>(r, a);
#pragma unroll
      for (int i = 0; i < NF; ++i) {
        out[0][i] = join8(r[i][0], r[i][1]);
        out[1][i] = join8(r[i][2], r[i][3]);
      }
    }
  }
  // COLS: the same of two tiles, `apart` bytes apart, in one block.
  __device__ __forceinline__ void read2(v8bf (&o0)[2][NF], v8bf (&o1)[2][NF], const uint8_t* tile, int apart) const {
    static_assert(L == COLS, "transposing reads");
    const uint32_t base = (uint32_t)(uintptr_t)(lds_void_t)tile;
    uint32_t a[2 * NF];
    v2u r[2 * NF][4];
#pragma unroll
    for (int i = 0; i < NF; ++i) {
      a[i] = base + at[i];
      a[NF + i] = a[i] + apart;
    }
    read_tr<2 * NF, 0, HI, KK, KK + HI>(r, a);
#pragma unroll
    for (int i = 0; i < NF; ++i) {
      o0[0][i] = join8(r[i][0], r[i][1]);
      o0[1][i] = join8(r[i][2], r[i][3]);
      o1[0][i] = join8(r[NF + i][0], r[NF + i][1]);
      o1[1][i] = join8(r[NF + i][2], r[NF + i][3]);
    }
  }
};

__device__ __forceinline__ v4f mfma16(v8bf a, v8bf b, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}
// The same 16 bytes per lane as sixteen 8-bit integers, summed exactly: twice
// the k (64) in the same time.  The kernels that stage bf16 operands carry 8-bit
// rows as rows of half as many bf16 elements; only this product and the
// epilogue know the difference.
__device__ __forceinline__ v4i mfma16(v8bf a, v8bf b, v4i c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(v4i, a), __builtin_bit_cast(v4i, b), c, 0, 0, 0);
}

// ---------------------------------------------------------------------------
// Epilogues of a wavefront's block, FM x 16 rows m.  `region`: LDS of its own,
// free for use; rows are staged there so that stores write whole row segments.
// ---------------------------------------------------------------------------

// Writes FM * 16 staged rows of SEG bytes (SEG / 16 chunks, chunk c of row r
// at c ^ (r % chunks)) to out + m * ld_bytes, rows below m_end.
template <int FM, int SEG>
__device__ __forceinline__ void write_rows(const uint8_t* region, uint8_t* out, int64_t ld_bytes, int64_t m0,
                                           int64_t m_end, int lane) {
  constexpr int CPR = SEG / 16, RPI = 64 / CPR, N = (FM * 16 + RPI - 1) / RPI;
  wait_lds();
#pragma unroll
  for (int t = 0; t < N; ++t) {
    const int row = t * RPI + lane / CPR, c = lane % CPR;
    if (row < FM * 16 && m0 + row < m_end) {
      const uint4 v = *reinterpret_cast<const uint4*>(region + row * SEG + 16 * (c ^ (row & (CPR - 1))));
      *reinterpret_cast<uint4*>(out + (m0 + row) * ld_bytes + c * 16) = v;
    }
  }
  wait_lds();
}

struct GatedOut {
  uint16_t* h;        // [m, f]
  void* gu;           // checkpoint [m, 2 f]: bf16 or FP8; null for none
  uint8_t* gu_scale;  // [m, 2 f / 32] for FP8
  int64_t m, f;
  int act, fmt;  // fmt: GU_NONE ..
};

// One half (g or u) of the block into an FP8 checkpoint: 32 columns are one
// MX block, spread over the four 16-lane groups.
template <int FMT, int FM>
__device__ __forceinline__ void save_mx(const v4f (&v)[2][FM], uint8_t* q, uint8_t* scale, int64_t ld, int64_t m0,
                                        int64_t m_end, int64_t col, int lane, uint8_t* region) {
  const int r16 = lane & 15, lg = lane >> 4;
#pragma unroll
  for (int fm = 0; fm < FM; ++fm) {
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      a = max(a, max(__float_as_uint(v[0][fm][i]) & 0x7FFFFFFFu, __float_as_uint(v[1][fm][i]) & 0x7FFFFFFFu));
    a = max(a, (uint32_t)__shfl_xor((int)a, 16));
    a = max(a, (uint32_t)__shfl_xor((int)a, 32));
    const int code = mx_scale_code<FMT>(a);
    const float inv = mx_inverse(code), limit = mx_limit<FMT>(code);
    const int row = fm * 16 + r16;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const v4f& y = v[j][fm];
      const uint32_t w = mx_pack4<FMT>(mx_scaled(y[0], inv, limit), mx_scaled(y[1], inv, limit),
                                       mx_scaled(y[2], inv, limit), mx_scaled(y[3], inv, limit));
      *reinterpret_cast<uint32_t*>(region + row * 32 + 16 * (j ^ (row & 1)) + 4 * lg) = w;
    }
    if (lg == 0 && m0 + row < m_end) scale[(m0 + row) * (ld / MX_BLOCK) + col / MX_BLOCK] = (uint8_t)code;
  }
  write_rows<FM, 32>(region, q + col, ld, m0, m_end, lane);
}

template <int FM>
__device__ __forceinline__ void stage_bf16x32(const v4f (&v)[2][FM], int lane, uint8_t* region) {
  const int r16 = lane & 15, lg = lane >> 4;
#pragma unroll
  for (int fm = 0; fm < FM; ++fm) {
    const int row = fm * 16 + r16;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int c = (2 * j + (lg >> 1)) ^ (row & 3);
      *reinterpret_cast<uint2*>(region + row * 64 + c * 16 + 8 * (lg & 1)) =
          make_uint2(pack_bf16x2(v[j][fm][0], v[j][fm][1]), pack_bf16x2(v[j][fm][2], v[j][fm][3]));
    }
  }
}

template <int FM>
__device__ __forceinline__ void apply_gate(v4f (&h)[2][FM], const v4f (&g)[2][FM], const v4f (&u)[2][FM], int act) {
  auto all = [&](auto fn) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int fm = 0; fm < FM; ++fm)
#pragma unroll
        for (int i = 0; i < 4; ++i) h[j][fm][i] = fn(g[j][fm][i]) * u[j][fm][i];
  };
  if (act == ACT_SILU) all([](float t) { return act_value<ACT_SILU>(t); });
  else if (act == ACT_GELU_TANH) all([](float t) { return act_value<ACT_GELU_TANH>(t); });
  else all([](float t) { return act_value<ACT_RELU>(t); });
}

// g, u: columns col .. col + 31 (two groups of 16) of rows m0 .. m0 + 16 FM - 1.
// region: FM * 16 * 64 bytes.  h is formed from the binary32 g and u; the
// checkpoint rounds each of them once.
template <int FM>
__device__ __forceinline__ void gated_epilogue(const v4f (&g)[2][FM], const v4f (&u)[2][FM], const GatedOut& o,
                                               int64_t m0, int64_t col, int lane, uint8_t* region) {
  if (col >= o.f) return;
  v4f h[2][FM];
  apply_gate<FM>(h, g, u, o.act);
  stage_bf16x32<FM>(h, lane, region);
  write_rows<FM, 64>(region, reinterpret_cast<uint8_t*>(o.h + col), o.f * 2, m0, o.m, lane);
  if (o.fmt == GU_NONE) return;
  if (o.fmt == GU_BF16) {
    uint16_t* gu = reinterpret_cast<uint16_t*>(o.gu);
    stage_bf16x32<FM>(g, lane, region);
    write_rows<FM, 64>(region, reinterpret_cast<uint8_t*>(gu + col), o.f * 4, m0, o.m, lane);
    stage_bf16x32<FM>(u, lane, region);
    write_rows<FM, 64>(region, reinterpret_cast<uint8_t*>(gu + o.f + col), o.f * 4, m0, o.m, lane);
    return;
  }
  uint8_t* q = reinterpret_cast<uint8_t*>(o.gu);
  if (o.fmt == GU_E4M3) {
    save_mx<MX_E4M3, FM>(g, q, o.gu_scale, 2 * o.f, m0, o.m, col, lane, region);
    save_mx<MX_E4M3, FM>(u, q, o.gu_scale, 2 * o.f, m0, o.m, o.f + col, lane, region);
  } else {
    save_mx<MX_E5M2, FM>(g, q, o.gu_scale, 2 * o.f, m0, o.m, col, lane, region);
    save_mx<MX_E5M2, FM>(u, q, o.gu_scale, 2 * o.f, m0, o.m, o.f + col, lane, region);
  }
}

struct PlainOut {
  void* out;             // [m, n] bf16 or binary32
  const uint16_t* bias;  // [n] bf16 or null
  int64_t m, n;
  int out_fmt;
};

// acc: columns col .. col + 63 of rows m0 .. m0 + 16 FM - 1; n is a multiple
// of 8.  region: FM * 16 * 128 bytes (bf16 output).
template <int FM>
__device__ __forceinline__ void plain_epilogue(v4f (&acc)[4][FM], const PlainOut& o, int64_t m0, int64_t col, int lane,
                                               uint8_t* region) {
  const int r16 = lane & 15, lg = lane >> 4;
  if (col >= o.n) return;
  if (o.bias) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t n = min(col + 16 * j + 4 * lg, o.n - 4);
      const uint2 b = *reinterpret_cast<const uint2*>(o.bias + n);
#pragma unroll
      for (int fm = 0; fm < FM; ++fm) {
        acc[j][fm][0] += bf16_to_f32(b.x & 0xFFFFu);
        acc[j][fm][1] += bf16_to_f32(b.x >> 16);
        acc[j][fm][2] += bf16_to_f32(b.y & 0xFFFFu);
        acc[j][fm][3] += bf16_to_f32(b.y >> 16);
      }
    }
  }
  if (o.out_fmt == OUT_F32) {
    float* out = reinterpret_cast<float*>(o.out);
#pragma unroll
    for (int fm = 0; fm < FM; ++fm) {
      const int64_t m = m0 + fm * 16 + r16;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int64_t n = col + 16 * j + 4 * lg;
        if (m < o.m && n < o.n) *reinterpret_cast<v4f*>(out + m * o.n + n) = acc[j][fm];
      }
    }
    return;
  }
#pragma unroll
  for (int fm = 0; fm < FM; ++fm) {
    const int row = fm * 16 + r16;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int c = (2 * j + (lg >> 1)) ^ (row & 7);
      *reinterpret_cast<uint2*>(region + row * 128 + c * 16 + 8 * (lg & 1)) =
          make_uint2(pack_bf16x2(acc[j][fm][0], acc[j][fm][1]), pack_bf16x2(acc[j][fm][2], acc[j][fm][3]));
    }
  }
  wait_lds();
  uint16_t* out = reinterpret_cast<uint16_t*>(o.out);
#pragma unroll
  for (int t = 0; t < FM * 2; ++t) {
    const int row = t * 8 + (lane >> 3), c = lane & 7;
    const uint4 v = *reinterpret_cast<const uint4*>(region + row * 128 + 16 * (c ^ (row & 7)));
    const int64_t m = m0 + row, n = col + 8 * c;
    if (m < o.m && n < o.n) *reinterpret_cast<uint4*>(out + m * o.n + n) = v;
  }
}

// Scales of an 8-bit integer product: one per activation row and weight row.
struct Int8Scales {
  const float *x, *w;
};

// An output of an 8-bit integer product from its exact sum, by the same four
// roundings in every kernel: the sum to binary32, the scales' product, the fused
// multiply-add with the bias, and the caller's to the output type.
__device__ __forceinline__ float int8_value(int sum, float xs, float ws, float bias) {
  return __builtin_fmaf((float)sum, xs * ws, bias);
}

// Four biases from column n on (n a multiple of 4); zeros (-0, which leaves a
// product as it is) without one.
__device__ __forceinline__ v4f bias4(const uint16_t* bias, int64_t n) {
  if (!bias) return v4f{-0.f, -0.f, -0.f, -0.f};
  const uint2 b = *reinterpret_cast<const uint2*>(bias + n);
  return v4f{bf16_to_f32(b.x & 0xFFFFu), bf16_to_f32(b.x >> 16), bf16_to_f32(b.y & 0xFFFFu), bf16_to_f32(b.y >> 16)};
}

// The scales and biases of a workgroup's BM rows and BN columns, in LDS.  They are
// read at the start of its work (BM + BN is at most twice the threads, BN at most as many):
// read in the epilogue they held every tile up by 5 us.
template <int BM, int BN>
struct Int8Tile {
  float x[BM], w[BN], bias[BN];
};
struct Int8Fetched {
  float v[2];
  uint32_t bias;
};
// Rows m0 .. and columns n0 .. ; past the ends the last one's (not stored).
template <int BM, int BN>
__device__ __forceinline__ Int8Fetched fetch_scales(const Int8Scales& sc, const PlainOut& o, int64_t m0, int64_t n0,
                                                    int tid, int threads) {
  Int8Fetched f{};
  if (o.bias && tid < BN) f.bias = o.bias[min(n0 + tid, o.n - 1)];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int at = tid + i * threads;
    if (at < BM) f.v[i] = sc.x[min(m0 + at, o.m - 1)];
    else if (at < BM + BN) f.v[i] = sc.w[min(n0 + at - BM, o.n - 1)];
  }
  return f;
}
template <int BM, int BN>
__device__ __forceinline__ void put_scales(Int8Tile<BM, BN>& t, const Int8Fetched& f, bool biased, int tid,
                                           int threads) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int at = tid + i * threads;
    if (at < BM) t.x[at] = f.v[i];
    else if (at < BM + BN) t.w[at - BM] = f.v[i];
  }
  if (tid < BN) t.bias[tid] = biased ? bf16_to_f32(f.bias) : -0.f;
}

// Columns col .. col + 63 of rows m0 .. from their exact sums; xs, ws, bias: in LDS,
// of the first of these rows and columns (null for a slice's partial sums, which
// are kept as integers).
template <int FM>
__device__ __forceinline__ void int8_epilogue(const v4i (&acc)[4][FM], const float* xs, const float* ws,
                                              const float* bias, PlainOut o, int64_t m0, int64_t col, int lane,
                                              uint8_t* region) {
  const int r16 = lane & 15, lg = lane >> 4;
  if (col >= o.n) return;
  v4f y[4][FM];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    if (!xs) {
#pragma unroll
      for (int fm = 0; fm < FM; ++fm) y[j][fm] = __builtin_bit_cast(v4f, acc[j][fm]);
      continue;
    }
    const v4f w = *reinterpret_cast<const v4f*>(ws + 16 * j + 4 * lg);
    const v4f b = *reinterpret_cast<const v4f*>(bias + 16 * j + 4 * lg);
#pragma unroll
    for (int fm = 0; fm < FM; ++fm) {
      const float x = xs[fm * 16 + r16];
#pragma unroll
      for (int i = 0; i < 4; ++i) y[j][fm][i] = int8_value(acc[j][fm][i], x, w[i], b[i]);
    }
  }
  if (xs) o.bias = nullptr;
  plain_epilogue<FM>(y, o, m0, col, lane, region);
}

// Slice and tile of workgroup `id` of 8 * ceil(slices * T / 8): XCD id % 8 (each
// has its own L2) owns a contiguous run of them, slice by slice, the tiles of a
// slice in groups of `group` n tiles.  False past the last.  (32-bit: the
// launchers bound slices * T by 2^23.)  With every slice over all XCDs, each of
// which then reads most of both operands: dx of m = 73, k = 1408, f = 11584 42.8
// us against 21.3.
__device__ __forceinline__ bool tile_of(uint32_t id, uint32_t slices, uint32_t tiles_m, uint32_t tiles_n,
                                        uint32_t group, uint32_t& slice, int64_t& tm, int64_t& tn) {
  const uint32_t T = tiles_m * tiles_n, items = slices * T, per = (items + 7) / 8;
  uint32_t lid = (id % 8) * per + id / 8;
  if (id / 8 >= per || lid >= items) return false;
  slice = slices == 1 ? 0 : lid / T;
  lid -= slice * T;
  const uint32_t g = lid / (group * tiles_m), first = g * group;
  const uint32_t size = min(tiles_n - first, group), within = lid - first * tiles_m;
  tn = first + within % size;
  tm = within / size;
  return true;
}

}  // namespace sfr

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

enum { ROWS = 0, COLS = 1 };

typedef __bf16 v4bf __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void* lds_void_t;

constexpr int BK = 64;  // k of one stage

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buf_rsrc(const void* base, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, (int)(bytes > 0 ? bytes : 0), 0x00020000);
}

// Lane l's 16 bytes at `voff` land at lds + 16 l.  The range check covers the
// whole offset (it is all in the vector offset): a lane past the range writes zeros.
__device__ __forceinline__ void buf_to_lds(__amdgpu_buffer_rsrc_t r, uint8_t* lds, int voff) {
  const uint32_t a = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(lds_void_t)lds);
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_void_t)(uintptr_t)a, 16, voff, 0, 0, 0);
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
//   COLS: BR * 2 bytes per k; a transposing read takes 32 bytes of each of four
//     k (per 16 lanes), whose rows start at the same bank, so the 32-byte unit
//     u of row k sits at u ^ cols_swizzle(k).
// A 1 KB load covers 8 rows (ROWS) or 512 / BR of k (COLS); the swizzles are
// applied to the global address of each lane.
// ---------------------------------------------------------------------------
template <int BR>
__device__ __forceinline__ int cols_swizzle(int k) {
  return BR >= 128 ? (k & 3) | (((k >> 3) & 1) << 2) : (k & 3);
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
  int64_t left;  // bytes from base to the end of what may be read
  int64_t step;  // bytes per stage of k
  int voff[PER];
  int wave, chunk;

  // rows r0 .. of `rows`; ld elements between stored rows; k from k0 (a multiple of BK) of `kdim`
  __device__ __forceinline__ Loader(const uint16_t* p, int64_t ld, int64_t r0, int64_t rows, int64_t k0, int64_t kdim,
                                    int wave_, int lane)
      : wave(wave_) {
    if constexpr (L == ROWS) {
      const int part = PAIR ? (wave >> 1) & 1 : 0;
      const int64_t first = part * rows + r0;
      const int64_t n = min(rows - r0, (int64_t)(PAIR ? BR / 2 : BR));
      base = reinterpret_cast<const uint8_t*>(p + first * ld + k0);
      left = (n * ld - k0) * 2;
      step = BK * 2;
      chunk = (lane & 7) ^ (lane >> 3);
#pragma unroll
      for (int q = 0; q < PER; ++q) {
        const int j = wave + q * NW;
        const int row = (PAIR ? (j >> 2) * 16 + (j & 1) * 8 : j * 8) + (lane >> 3);
        voff[q] = row * (int)(ld * 2) + chunk * 16;
      }
    } else {
      constexpr int RPL = 512 / BR, CPR = 64 / RPL;  // k per load, 16-byte chunks per k
      base = reinterpret_cast<const uint8_t*>(p + k0 * ld + r0);
      left = ((kdim - k0) * ld - r0) * 2;
      step = BK * 2 * ld;
      chunk = 0;
#pragma unroll
      for (int q = 0; q < PER; ++q) {
        const int k = (wave + q * NW) * RPL + lane / CPR;
        voff[q] = k * (int)(ld * 2) + 16 * ((lane % CPR) ^ (cols_swizzle<BR>(k) << 1));
      }
    }
  }
  // Puts the next stage's loads in flight and moves on.  k_left: k not yet
  // loaded; in a ROWS operand's last stage the chunks past it read zeros (a
  // COLS operand's lie past the range by themselves).
  __device__ __forceinline__ void stage(uint8_t* lds, int k_left) {
    const __amdgpu_buffer_rsrc_t r = buf_rsrc(base, min(left, (int64_t)0x7FFFFF00));
#pragma unroll
    for (int q = 0; q < PER; ++q) {
      int v = voff[q];
      if constexpr (L == ROWS) v = chunk * 8 < k_left ? v : kPastRange;
      buf_to_lds(r, lds + (wave + q * NW) * 1024, v);
    }
    base += step;
    left -= step;
  }
};

// Operand reads of 16-row fragments from a tile of BR rows.
template <int L, int BR>
struct Reader {
  int a, b, c;  // lane parts of the address
  __device__ __forceinline__ Reader(int lane) {
    const int r16 = lane & 15, lg = lane >> 4;
    if constexpr (L == ROWS) {
      a = r16 * 128;
      b = lg;
      c = r16 & 7;
    } else {
      a = (8 * lg + (r16 >> 2)) * (BR * 2) + 16 * ((r16 & 3) >> 1) + 8 * (r16 & 1);
      b = cols_swizzle<BR>(8 * lg + (r16 >> 2));
      c = 0;
    }
  }
  // fragment frag (rows 16 frag ..), k 32 kk .. 32 kk + 31 of the stage
  __device__ __forceinline__ v8bf read(const uint8_t* tile, int frag, int kk) const {
    if constexpr (L == ROWS) {
      return *reinterpret_cast<const v8bf*>(tile + a + frag * 2048 + 16 * ((kk * 4 + b) ^ c));
    } else {
      const uint8_t* p = tile + a + kk * (32 * BR * 2) + 32 * (frag ^ b);
      typedef __attribute__((address_space(3))) v4bf* lds_v4_t;
      const v4bf lo = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_v4_t)(p));
      const v4bf hi = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_v4_t)(p + 4 * BR * 2));
      return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
    }
  }
};

__device__ __forceinline__ v4f mfma16(v8bf a, v8bf b, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
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

// Tile of workgroup `id` of 8 * ceil(T / 8): XCD id % 8 (each has its own L2)
// owns a contiguous run of the tiles, taken in groups of `group` n tiles.
// False past the last tile.
__device__ __forceinline__ bool tile_of(int64_t id, int64_t tiles_m, int64_t tiles_n, int group, int64_t& tm,
                                        int64_t& tn) {
  const int64_t T = tiles_m * tiles_n, per = (T + 7) / 8;
  const int64_t lid = (id % 8) * per + id / 8;
  if (id / 8 >= per || lid >= T) return false;
  const int64_t g = lid / (group * tiles_m), first = g * group;
  const int64_t size = min(tiles_n - first, (int64_t)group), within = lid - first * tiles_m;
  tn = first + within % size;
  tm = within / size;
  return true;
}

}  // namespace sfr

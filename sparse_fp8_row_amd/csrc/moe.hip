// A mixture of gated feed-forward blocks for a few tokens: the router, and the
// layer
//     out[t] = sum_s weights[t, s] (act(x[t] Wg[e]^T) * (x[t] Wu[e]^T)) Wd[e]^T,  e = ids[t, s]
// in two launches.  Bound by reading the chosen experts' weights once.
#include "sfr_dense.hpp"

namespace sfr {
namespace {

// ---------------------------------------------------------------------------
// Router
// ---------------------------------------------------------------------------

constexpr int kTokens = 4;  // of one workgroup of the logits

// logits[t, e] = x[t] . w[e] + bias[e], summed in binary64 and rounded once to
// binary32: every product of two bf16 values is exact in binary32, so the sum's
// rounding (2^-53) is all there is before the last, and which of two nearly equal
// experts a token takes does not depend on the batch, the tiling or the order.
__global__ __launch_bounds__(256) void route_logits_kernel(const uint16_t* __restrict__ x, int64_t m, int k,
                                                           const uint16_t* __restrict__ w, int experts,
                                                           const float* __restrict__ bias, float* __restrict__ logits) {
  __shared__ double red[4][kTokens];
  const int tid = threadIdx.x, e = blockIdx.x;
  const int64_t t0 = (int64_t)blockIdx.y * kTokens;
  double sum[kTokens] = {};
  for (int c = tid; c < k / 8; c += 256) {
    const uint4 b = reinterpret_cast<const uint4*>(w + (int64_t)e * k)[c];
    const uint32_t bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int t = 0; t < kTokens; ++t) {
      const uint4 a = reinterpret_cast<const uint4*>(x + min(t0 + t, m - 1) * k)[c];
      const uint32_t aw[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        sum[t] += (double)(bf16_to_f32(aw[i] & 0xFFFFu) * bf16_to_f32(bw[i] & 0xFFFFu));
        sum[t] += (double)(bf16_to_f32(aw[i] >> 16) * bf16_to_f32(bw[i] >> 16));
      }
    }
  }
#pragma unroll
  for (int t = 0; t < kTokens; ++t) {
#pragma unroll
    for (int d = 32; d >= 1; d /= 2) sum[t] += __shfl_xor(sum[t], d);
    if ((tid & 63) == 0) red[tid >> 6][t] = sum[t];
  }
  __syncthreads();
  if (tid < kTokens && t0 + tid < m) {
    double s = ((red[0][tid] + red[1][tid]) + red[2][tid]) + red[3][tid];
    if (bias) s += (double)bias[e];
    logits[(t0 + tid) * experts + e] = (float)s;
  }
}

// Whole numbers in the order of binary32 values, -0 and +0 one value, NaN above
// +infinity; 0 for -infinity, which is never chosen.
__device__ __forceinline__ uint32_t order_of(float v) {
  if (v != v) return 0xFFFFFFFFu;
  if (v == -__builtin_inff()) return 0;
  const uint32_t u = __float_as_uint(v + 0.0f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// A wavefront per token: `top` rounds of a wavefront-wide maximum over (value,
// lower index first); lane j then holds the j-th choice.  The weights are formed
// relative to the best, so no exponential overflows.
template <int PER>  // experts per lane
__global__ __launch_bounds__(256) void route_select_kernel(const float* __restrict__ logits, int64_t m, int experts,
                                                           int top, int score, int renormalize, int32_t* __restrict__ ids,
                                                           float* __restrict__ weights) {
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= m) return;
  float v[PER];
  uint64_t key[PER];  // order of the value, then of the lower index
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = lane + 64 * i;
    v[i] = e < experts ? logits[t * experts + e] : -__builtin_inff();
    const uint32_t o = order_of(v[i]);
    key[i] = o ? (uint64_t)o << 32 | (uint32_t)~e : 0;
  }
  float chosen = -__builtin_inff(), best = 0.0f;
  int id = -1;
  for (int j = 0; j < top; ++j) {
    uint64_t k = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) k = max(k, key[i]);
#pragma unroll
    for (int d = 1; d < 64; d *= 2) k = max(k, (uint64_t)__shfl_xor((unsigned long long)k, d));
    if (k == 0) break;  // nothing left: lanes j .. keep id -1
    const int e = (int)~(uint32_t)k;
    float mine = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (key[i] == k) {
        key[i] = 0;
        mine = v[i];
      }
    const float value = __shfl(mine, e & 63);
    if (j == 0) best = value;
    if (lane == j) {
      id = e;
      chosen = value;
    }
  }
  float p = 0.0f, total = 0.0f;
  if (score == ROUTE_SOFTMAX) {
    if (id >= 0) p = expf(chosen - best);
    if (!renormalize) {
#pragma unroll
      for (int i = 0; i < PER; ++i) total += v[i] == -__builtin_inff() ? 0.0f : expf(v[i] - best);
    }
  } else if (renormalize) {
    // s(l) / sum s(l) by differences of log s, which stay finite where s underflows
    auto log_s = [](float l) { return fminf(l, 0.0f) - log1pf(expf(-fabsf(l))); };
    if (id >= 0) p = chosen != chosen ? chosen : expf(log_s(chosen) - log_s(best));
  } else {
    if (id >= 0) p = 1.0f / (1.0f + expf(-chosen));
  }
  if (renormalize) total = p;
  if (renormalize || score == ROUTE_SOFTMAX) {
#pragma unroll
    for (int d = 1; d < 64; d *= 2) total += __shfl_xor(total, d);
    p = id >= 0 ? p / total : 0.0f;
  }
  if (lane < top) {
    ids[t * top + lane] = id;
    weights[t * top + lane] = p;
  }
}

// ---------------------------------------------------------------------------
// The layer
//
// Both kernels stream weight rows the way the few-row products do (stream.hip):
// wavefronts take units of UK k in LDS buffers of their own, D - 1 units ahead,
// 16 RT weight rows a workgroup, and add their sums in a fixed order at the end.
//
// Up: a workgroup owns RT / 2 pairs of gate and up row tiles of one expert, and
//   runs them on that expert's tokens, R at a time, gathered by their rows of x.
//   h = act(g) u goes to the workspace, rounded to bf16, at row (token, first
//   slot of the expert).  A workgroup reads ids by itself: a bit per chosen
//   expert in LDS, the blockIdx.y-th of which is its own.
// Down: a workgroup owns 16 RT columns of out for all tokens and walks all chosen
//   experts in ascending order; its wavefronts take even shares of their units.
//   Tokens are the columns of the product, zeros where a token did not choose the
//   expert; at the end of an expert a token's sums are added to its total with
//   its weight, and only where it did choose it, so that an infinity in a weight
//   stays with the tokens that met it.
// ---------------------------------------------------------------------------

struct Choices {
  int ids[kMoeTokens * kMoeTop];
  uint32_t bits[kMoeExperts / 32];  // chosen experts
};

// Reads ids: values outside [0, experts) are no choice (-1).
__device__ __forceinline__ void read_choices(Choices& c, const MoeArgs& p) {
  for (int i = threadIdx.x; i < kMoeExperts / 32; i += blockDim.x) c.bits[i] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < p.m * p.top; i += blockDim.x) {
    const int id = p.ids[i];
    const bool in = id >= 0 && id < p.experts;
    c.ids[i] = in ? id : -1;
    if (in) atomicOr(&c.bits[id / 32], 1u << (id & 31));
  }
  __syncthreads();
}

// The chosen experts in ascending order, found by a wavefront.
struct Chosen {
  uint32_t word;  // lane l < 32: bits of experts 32 l ..
  int upto;       // chosen experts up to this word's end
  int count;
  __device__ __forceinline__ Chosen(const Choices& c, int lane) {
    static_assert(kMoeExperts <= 64 * 32, "a word per lane");
    word = lane < kMoeExperts / 32 ? c.bits[lane] : 0;
    upto = __popc(word);
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int before = __shfl_up(upto, d);
      if (lane >= d) upto += before;
    }
    count = __builtin_amdgcn_readlane(upto, 63);
  }
  // The i-th (i < count), uniform.
  __device__ __forceinline__ int expert(int i) const {
    const uint64_t past = __ballot(upto > i);
    const int l = __builtin_ctzll(past);
    uint32_t w = (uint32_t)__builtin_amdgcn_readlane((int)word, l);
    int skip = i - (__builtin_amdgcn_readlane(upto, l) - __popc(w));
    for (; skip > 0; --skip) w &= w - 1;
    return 32 * l + __builtin_ctz(w);
  }
};

// Lane t's first slot with expert e, or -1.
__device__ __forceinline__ int slot_of(const Choices& c, const MoeArgs& p, int e, int t) {
  int slot = -1;
  if (t < p.m)
    for (int s = p.top - 1; s >= 0; --s) slot = c.ids[t * p.top + s] == e ? s : slot;
  return slot;
}

// R: activation rows in LDS.
template <int WF, int RT, int R, int NW, int D>
struct Unit {
  static constexpr int UK = WF == EXPERT_BF16 ? 128 : 256;
  static constexpr int WROW = WF == EXPERT_BF16 ? UK * 2 : WF == EXPERT_INT8 ? UK : UK / 2, XROW = UK * 2;
  static constexpr int WL = 16 * WROW / 1024, SL = WF == EXPERT_FP4 ? 16 * (UK / 32) / 64 : 0;
  static constexpr int XL = (R * XROW + 1023) / 1024;
  static constexpr int LOADS = RT * (WL + SL) + XL;
  static constexpr int TILE = WL * 1024 + SL * 256, BYTES = RT * TILE + XL * 1024;
  static constexpr int RED = NW * RT * R * 16 * 4;
  static constexpr int LDS = NW * D * BYTES > RED ? NW * D * BYTES : RED;
  static_assert((D - 1) * LOADS < 64, "wait counts");
};

template <int WF>
__device__ __forceinline__ int row_bytes(int k) {
  return WF == EXPERT_BF16 ? k * 2 : WF == EXPERT_INT8 ? k : k / 2;
}

// Puts a unit's 16 weight rows and (4-bit) scales in flight: k from u UK on, of
// which `left` exist (zeros past them; none for left <= 0).
template <int WF, bool NT, class U>
__device__ __forceinline__ void issue_weight(__amdgpu_buffer_rsrc_t rw, __amdgpu_buffer_rsrc_t rs, uint8_t* b, int u,
                                             int left, int k, int lane) {
  constexpr int WC = U::WROW / 16, WPL = 64 / WC, PER = U::UK / WC;  // chunks per row, rows per load, k per chunk
#pragma unroll
  for (int j = 0; j < U::WL; ++j) {
    const int row = j * WPL + lane / WC, c = (lane % WC) ^ (row & 7);
    buf_to_lds<NT>(rw, b + j * 1024, c * PER < left ? row * row_bytes<WF>(k) + u * U::WROW + c * 16 : kPastRange);
  }
#pragma unroll
  for (int j = 0; j < U::SL; ++j) {
    const int row = j * 8 + (lane >> 3), c = lane & 7;
    buf_byte_to_lds(rs, b + U::WL * 1024 + j * 256, c * 32 < left ? row * (k / 32) + u * 8 + c : kPastRange);
  }
}

// Eight 8-bit integers as bf16 values (exact).
__device__ __forceinline__ v8bf widen8_int8(uint32_t lo, uint32_t hi) {
  typedef uint32_t v4u __attribute__((ext_vector_type(4)));
  v4u r;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t w = i ? hi : lo;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      r[2 * i + h] = pack_bf16x2((float)(int8_t)(w >> (16 * h)), (float)(int8_t)(w >> (16 * h + 8)));
  }
  return __builtin_bit_cast(v8bf, r);
}

// acc[t][b] += (weight tile t) (activation rows 16 b ..) over one unit.
template <int WF, int RT, int RB, int R, class U>
__device__ __forceinline__ void multiply_unit(v4f (&acc)[RT][RB], const uint8_t* b, int lane) {
  const int r16 = lane & 15, lg = lane >> 4;
  const uint8_t* const xb = b + RT * U::TILE;
#pragma unroll
  for (int s = 0; s < U::UK / 128; ++s) {
    v8bf x[RB][4];
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
      const int row = min(16 * rb + r16, R - 1);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = WF == EXPERT_BF16 ? 4 * j + lg : 16 * s + 4 * lg + j;
        x[rb][j] = *reinterpret_cast<const v8bf*>(xb + row * U::XROW + 16 * (c ^ (row & 7)));
      }
    }
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      const uint8_t* wb = b + t * U::TILE + r16 * U::WROW;
      v8bf w[4];
      if constexpr (WF == EXPERT_BF16) {
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = *reinterpret_cast<const v8bf*>(wb + 16 * ((4 * j + lg) ^ (r16 & 7)));
      } else if constexpr (WF == EXPERT_INT8) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const v4i q = *reinterpret_cast<const v4i*>(wb + 16 * ((8 * s + 2 * lg + h) ^ (r16 & 7)));
          w[2 * h] = widen8_int8((uint32_t)q[0], (uint32_t)q[1]);
          w[2 * h + 1] = widen8_int8((uint32_t)q[2], (uint32_t)q[3]);
        }
      } else {
        const v4i q = *reinterpret_cast<const v4i*>(wb + 16 * ((4 * s + lg) ^ (r16 & 7)));
        const float f = mx_scale_value(
            *reinterpret_cast<const uint32_t*>(b + t * U::TILE + U::WL * 1024 + 4 * (r16 * 8 + 4 * s + lg)));
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = __builtin_bit_cast(v8bf, mx_widen8_e2m1((uint32_t)q[j], f));
      }
#pragma unroll
      for (int rb = 0; rb < RB; ++rb)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[t][rb] = mfma16(w[j], x[rb][j], acc[t][rb]);
    }
  }
}

// Row tile's descriptors: weight rows from `row` on of the stacked experts.
template <int WF>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t weight_rows(const void* w, int64_t row, int k) {
  return buf_rsrc(static_cast<const uint8_t*>(w) + row * row_bytes<WF>(k), kPastRange);
}
template <int WF>
__device__ __forceinline__ __amdgpu_buffer_rsrc_t scale_rows(const void* s, int64_t row, int k) {
  return buf_rsrc(static_cast<const uint8_t*>(s) + (WF == EXPERT_FP4 ? row * (k / 32) : 0), kPastRange);
}

template <int WF, int RT, int R, int NW, int D, bool NT>
__global__ __launch_bounds__(64 * NW) void moe_up_kernel(MoeArgs p) {
  using U = Unit<WF, RT, R, NW, D>;
  static_assert(RT % 2 == 0, "row tiles come in pairs");
  constexpr int RB = (R + 15) / 16;
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  __shared__ Choices choices;
  __shared__ int rows[kMoeTokens], pairs[kMoeTokens];  // the expert's tokens, and their rows of h
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, lg = lane >> 4;

  read_choices(choices, p);
  const Chosen chosen(choices, lane);
  if ((int)blockIdx.y >= chosen.count) return;
  const int e = chosen.expert(blockIdx.y);
  const int slot = slot_of(choices, p, e, lane);
  const uint64_t takers = __ballot(slot >= 0);
  const int count = __popcll(takers);
  if (wave == 0 && slot >= 0) {
    const int r = __popcll(takers & (((uint64_t)1 << lane) - 1));
    rows[r] = lane;
    pairs[r] = lane * p.top + slot;
  }
  __syncthreads();

  const int K = p.k, tile0 = blockIdx.x * (RT / 2), tiles = p.f / 16;
  // tiles past the last one read the last one (and are not stored)
  __amdgpu_buffer_rsrc_t rw[RT], rs[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    const int64_t row = (int64_t)e * 2 * p.f + min(tile0 + (t >> 1), tiles - 1) * 16 + (t & 1 ? p.f : 0);
    rw[t] = weight_rows<WF>(p.w_gu, row, K);
    rs[t] = scale_rows<WF>(p.s_gu, row, K);
  }
  const __amdgpu_buffer_rsrc_t rx = buf_rsrc(p.x, kPastRange);
  uint8_t* const mine = smem + wave * (D * U::BYTES);
  const int units = (K + U::UK - 1) / U::UK;
  constexpr int XC = U::XROW / 16, XPL = 64 / XC;

  for (int r0 = 0; r0 < count; r0 += R) {
    const int mr = min(count - r0, R);
    int xoff[U::XL];
#pragma unroll
    for (int j = 0; j < U::XL; ++j) {
      const int row = j * XPL + lane / XC;
      xoff[j] = row < mr ? rows[r0 + row] * (K * 2) + 16 * ((lane % XC) ^ (row & 7)) : kPastRange;
    }
    auto issue = [&](int at, int u) __attribute__((always_inline)) {
      uint8_t* b = mine + at * U::BYTES;
      const int left = K - u * U::UK;  // may be negative: every lane masked
#pragma unroll
      for (int t = 0; t < RT; ++t) issue_weight<WF, NT, U>(rw[t], rs[t], b + t * U::TILE, u, left, K, lane);
#pragma unroll
      for (int j = 0; j < U::XL; ++j) {
        const int c = (lane % XC) ^ ((j * XPL + lane / XC) & 7);
        const bool in = c * 8 < left && xoff[j] != kPastRange;
        buf_to_lds(rx, b + RT * U::TILE + j * 1024, in ? xoff[j] + u * U::XROW : kPastRange);
      }
    };
    v4f acc[RT][RB];
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
      for (int b = 0; b < RB; ++b) acc[t][b] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < D - 1; ++i) issue(i, wave + i * NW);
    int at = 0;
    for (int u = wave; u < units; u += NW) {
      wait_lds();  // the buffer to be refilled has been read
      issue(at == 0 ? D - 1 : at - 1, u + (D - 1) * NW);
      wait_vm<(D - 1) * U::LOADS>();
      asm volatile("" ::: "memory");
      multiply_unit<WF, RT, RB, R, U>(acc, mine + at * U::BYTES, lane);
      at = at == D - 1 ? 0 : at + 1;
    }
    wait_vm<0>();
    wait_lds();
    wg_barrier();  // no load in flight, no read pending: the buffers become the sums'

    float* const red = reinterpret_cast<float*>(smem);  // [NW][RT][R][16]
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
      for (int b = 0; b < RB; ++b)
        if (16 * b + r16 < mr)
          *reinterpret_cast<v4f*>(red + ((wave * RT + t) * R + 16 * b + r16) * 16 + 4 * lg) = acc[t][b];
    wait_lds();
    wg_barrier();
    constexpr int OT = RT / 2;
    for (int i = threadIdx.x; i < OT * 16 * mr; i += 64 * NW) {
      const int n = i % 16, t = i / 16 % OT, r = i / (16 * OT);
      const int col = (tile0 + t) * 16 + n;
      if (col >= p.f) continue;
      float g = 0.f, u = 0.f;
#pragma unroll
      for (int v = 0; v < NW; ++v) {
        g += red[((v * RT + 2 * t) * R + r) * 16 + n];
        u += red[((v * RT + 2 * t + 1) * R + r) * 16 + n];
      }
      if constexpr (WF == EXPERT_INT8) {
        const float* s = static_cast<const float*>(p.s_gu) + (int64_t)e * 2 * p.f + col;
        g *= s[0];
        u *= s[p.f];
      }
      const float h = u * (p.act == ACT_SILU        ? act_value<ACT_SILU>(g)
                           : p.act == ACT_GELU_TANH ? act_value<ACT_GELU_TANH>(g)
                                                    : act_value<ACT_RELU>(g));
      p.h[(int64_t)pairs[r0 + r] * p.f + col] = (uint16_t)pack_bf16x2(h, 0.f);
    }
    if (r0 + R < count) {
      wait_lds();
      wg_barrier();  // the sums are read: the buffers are free again
    }
  }
}

template <int WF, int RT, int R, int NW, int D, bool NT>
__global__ __launch_bounds__(64 * NW) void moe_down_kernel(MoeArgs p) {
  using U = Unit<WF, RT, R, NW, D>;
  constexpr int RB = (R + 15) / 16;
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  __shared__ Choices choices;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, lg = lane >> 4;
  const int F = p.f, tile0 = blockIdx.x * RT, tiles = p.k / 16;

  read_choices(choices, p);
  const Chosen chosen(choices, lane);
  const int each = (F + U::UK - 1) / U::UK, units = chosen.count * each;
  const int share = (units + NW - 1) / NW, first = min(wave * share, units), last = min(first + share, units);

  const __amdgpu_buffer_rsrc_t rh = buf_rsrc(p.h, kPastRange);
  uint8_t* const mine = smem + wave * (D * U::BYTES);
  constexpr int XC = U::XROW / 16, XPL = 64 / XC;
  __amdgpu_buffer_rsrc_t rw[RT], rs[RT];
  int hoff[U::XL];
  // the expert whose units are put in flight
  auto enter = [&](int i) __attribute__((always_inline)) {
    const int e = chosen.expert(i);
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      const int64_t row = (int64_t)e * p.k + min(tile0 + t, tiles - 1) * 16;
      rw[t] = weight_rows<WF>(p.w_down, row, F);
      rs[t] = scale_rows<WF>(p.s_down, row, F);
    }
    const int slot = slot_of(choices, p, e, lane);
    const int pair = slot < 0 ? -1 : lane * p.top + slot;
#pragma unroll
    for (int j = 0; j < U::XL; ++j) {
      const int row = j * XPL + lane / XC, from = __shfl(pair, row);
      hoff[j] = from < 0 ? kPastRange : from * (F * 2) + 16 * ((lane % XC) ^ (row & 7));
    }
  };
  int next = first, expert_in = 0, unit_in = 0;
  if (first < last) {
    expert_in = first / each;
    unit_in = first - expert_in * each;
    enter(expert_in);
  }
  // Puts the next unit in flight; past the wavefront's last, loads that are all masked.
  auto issue = [&](int at) __attribute__((always_inline)) {
    uint8_t* b = mine + at * U::BYTES;
    if (next < last && unit_in == each) {
      ++expert_in;
      unit_in = 0;
      enter(expert_in);
    }
    const int left = next < last ? F - unit_in * U::UK : 0;
#pragma unroll
    for (int t = 0; t < RT; ++t) issue_weight<WF, NT, U>(rw[t], rs[t], b + t * U::TILE, unit_in, left, F, lane);
#pragma unroll
    for (int j = 0; j < U::XL; ++j) {
      const int c = (lane % XC) ^ ((j * XPL + lane / XC) & 7);
      const bool in = c * 8 < left && hoff[j] != kPastRange;
      buf_to_lds(rh, b + RT * U::TILE + j * 1024, in ? hoff[j] + unit_in * U::XROW : kPastRange);
    }
    ++next;
    ++unit_in;
  };

  v4f acc[RT][RB], total[RT][RB];
#pragma unroll
  for (int t = 0; t < RT; ++t)
#pragma unroll
    for (int b = 0; b < RB; ++b) acc[t][b] = total[t][b] = v4f{0.f, 0.f, 0.f, 0.f};

  if (first < last) {
    int expert_at = first / each, unit_at = first - expert_at * each, at = 0;
#pragma unroll
    for (int i = 0; i < D - 1; ++i) issue(i);
    for (int u = first; u < last; ++u) {
      wait_lds();  // the buffer to be refilled has been read
      issue(at == 0 ? D - 1 : at - 1);
      wait_vm<(D - 1) * U::LOADS>();
      asm volatile("" ::: "memory");
      multiply_unit<WF, RT, RB, R, U>(acc, mine + at * U::BYTES, lane);
      at = at == D - 1 ? 0 : at + 1;
      if (++unit_at == each || u + 1 == last) {  // the expert's end, or this share's
        const int e = chosen.expert(expert_at);
        float weight = 0.f;  // lane t: token t's, over all its slots with this expert
        bool taker = false;
        if (lane < p.m)
          for (int s = 0; s < p.top; ++s)
            if (choices.ids[lane * p.top + s] == e) {
              weight += p.weights[lane * p.top + s];
              taker = true;
            }
        const uint64_t takers = __ballot(taker);
#pragma unroll
        for (int b = 0; b < RB; ++b) {
          const int col = 16 * b + r16;
          const float wt = __shfl(weight, col);
          const bool add = takers >> col & 1;
#pragma unroll
          for (int t = 0; t < RT; ++t) {
            v4f s = v4f{1.f, 1.f, 1.f, 1.f};
            if constexpr (WF == EXPERT_INT8)
              s = *reinterpret_cast<const v4f*>(static_cast<const float*>(p.s_down) + (int64_t)e * p.k +
                                                min(tile0 + t, tiles - 1) * 16 + 4 * lg);
#pragma unroll
            for (int i = 0; i < 4; ++i)
              total[t][b][i] = add ? total[t][b][i] + acc[t][b][i] * s[i] * wt : total[t][b][i];
            acc[t][b] = v4f{0.f, 0.f, 0.f, 0.f};
          }
        }
        ++expert_at;
        unit_at = 0;
      }
    }
  }
  wait_vm<0>();
  wait_lds();
  wg_barrier();  // no load in flight, no read pending: the buffers become the sums'

  float* const red = reinterpret_cast<float*>(smem);  // [NW][RT][R][16]
#pragma unroll
  for (int t = 0; t < RT; ++t)
#pragma unroll
    for (int b = 0; b < RB; ++b)
      if (16 * b + r16 < p.m)
        *reinterpret_cast<v4f*>(red + ((wave * RT + t) * R + 16 * b + r16) * 16 + 4 * lg) = total[t][b];
  wait_lds();
  wg_barrier();
  for (int i = threadIdx.x; i < RT * 16 * p.m; i += 64 * NW) {
    const int n = i % 16, t = i / 16 % RT, r = i / (16 * RT);
    const int col = (tile0 + t) * 16 + n;
    if (col >= p.k) continue;
    float y = 0.f;
#pragma unroll
    for (int v = 0; v < NW; ++v) y += red[((v * RT + t) * R + r) * 16 + n];
    p.out[(int64_t)r * p.k + col] = (uint16_t)pack_bf16x2(y, 0.f);
  }
}

template <class K>
hipError_t allow_lds(K* kernel, int bytes) {
  return bytes > 49152 ? hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, bytes)
                       : hipSuccess;
}

constexpr int kLdsLeft = 160 * 1024 - (int)sizeof(Choices) - 2 * kMoeTokens * 4;

template <int WF, int RT, int R, int NW, int D, bool NT>
hipError_t run_up(const MoeArgs& p, hipStream_t stream) {
  constexpr int bytes = Unit<WF, RT, R, NW, D>::LDS, cover = RT / 2 * 16;
  static_assert(bytes <= kLdsLeft, "LDS of a CU");
  auto* kernel = moe_up_kernel<WF, RT, R, NW, D, NT>;
  const hipError_t e = allow_lds(kernel, bytes);
  if (e != hipSuccess) return e;
  const dim3 grid((unsigned)((p.f + cover - 1) / cover), (unsigned)min(p.experts, p.m * p.top));
  kernel<<<grid, dim3(64 * NW), bytes, stream>>>(p);
  return hipGetLastError();
}

template <int WF, int RT, int R, int NW, int D, bool NT>
hipError_t run_down(const MoeArgs& p, hipStream_t stream) {
  constexpr int bytes = Unit<WF, RT, R, NW, D>::LDS, cover = RT * 16;
  static_assert(bytes <= kLdsLeft, "LDS of a CU");
  auto* kernel = moe_down_kernel<WF, RT, R, NW, D, NT>;
  const hipError_t e = allow_lds(kernel, bytes);
  if (e != hipSuccess) return e;
  kernel<<<dim3((unsigned)((p.k + cover - 1) / cover)), dim3(64 * NW), bytes, stream>>>(p);
  return hipGetLastError();
}

template <int WF>
hipError_t run_layer(const MoeArgs& p, hipStream_t stream) {
  hipError_t e = p.m <= 2    ? run_up<WF, 2, 2, 3, 2, true>(p, stream)
                 : p.m <= 8  ? run_up<WF, 2, 8, 3, 2, true>(p, stream)
                 : p.m <= 16 ? run_up<WF, 2, 16, 3, 2, true>(p, stream)
                             : run_up<WF, 2, 32, 2, 2, false>(p, stream);
  if (e != hipSuccess) return e;
  return p.m <= 2    ? run_down<WF, 1, 2, 8, 2, true>(p, stream)
         : p.m <= 8  ? run_down<WF, 1, 8, 6, 2, true>(p, stream)
         : p.m <= 16 ? run_down<WF, 1, 16, 4, 2, true>(p, stream)
         : p.m <= 32 ? run_down<WF, 1, 32, 2, 2, true>(p, stream)
                     : run_down<WF, 1, 64, 2, 2, true>(p, stream);
}

}  // namespace

hipError_t launch_moe_route(const RouteArgs& a, hipStream_t stream) {
  const int64_t groups = (a.m + kTokens - 1) / kTokens;
  for (int64_t g = 0; g < groups; g += 65535) {  // grid y
    const int64_t t = g * kTokens, n = groups - g < 65535 ? groups - g : 65535;
    route_logits_kernel<<<dim3(a.experts, (unsigned)n), dim3(256), 0, stream>>>(
        a.x + t * a.k, a.m - t, a.k, a.w, a.experts, a.bias, a.logits + t * a.experts);
  }
  const dim3 grid((unsigned)((a.m + 3) / 4)), block(256);
  auto* select = a.experts <= 64    ? route_select_kernel<1>
                 : a.experts <= 128 ? route_select_kernel<2>
                 : a.experts <= 256 ? route_select_kernel<4>
                                    : route_select_kernel<kMoeExperts / 64>;
  select<<<grid, block, 0, stream>>>(a.logits, a.m, a.experts, a.top, a.score, a.renormalize, a.ids, a.weights);
  return hipGetLastError();
}

// h of the tokens of one pass
int64_t moe_workspace_bytes(int64_t m, int64_t f, int top) {
  return (m < kMoeTokens ? m : kMoeTokens) * top * f * 2;
}

// kMoeTokens tokens at a time (a lane of a wavefront each).
hipError_t launch_moe_layer(const MoeArgs& args, int64_t m, hipStream_t stream) {
  MoeArgs p = args;
  for (int64_t t = 0; t < m; t += kMoeTokens) {
    p.m = (int)(m - t < kMoeTokens ? m - t : kMoeTokens);
    p.x = args.x + t * p.k;
    p.ids = args.ids + t * p.top;
    p.weights = args.weights + t * p.top;
    p.out = args.out + t * p.k;
    const hipError_t e = p.form == EXPERT_BF16   ? run_layer<EXPERT_BF16>(p, stream)
                         : p.form == EXPERT_INT8 ? run_layer<EXPERT_INT8>(p, stream)
                                                 : run_layer<EXPERT_FP4>(p, stream);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace sfr

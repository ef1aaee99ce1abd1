// A mixture of gated feed-forward blocks for a few tokens: the router, and the
// layer
//     out[t] = sum_s weights[t, s] (act(x[t] Wg[e]^T) * (x[t] Wu[e]^T)) Wd[e]^T,  e = ids[t, s]
// in two launches for a few tokens and three for up to 64, the tokens of one pass.
// Bound by reading the chosen experts' weights once.
#include <type_traits>

#include "sfr_dense.hpp"
#include "sfr_quant.hpp"

namespace sfr {
namespace {

// ---------------------------------------------------------------------------
// Router
// ---------------------------------------------------------------------------

// logits[t, e] = x[t] . w[e] + bias[e], summed in binary64 and rounded once to
// binary32: every product of two bf16 values is exact in binary64 (in binary32 it can
// overflow, vanish or be rounded among the subnormals).
//
// All kernels add in the same order, so a token's logits, and which of two nearly
// equal experts it takes, depend on nothing but its row and the experts': k is taken in
// steps of 32; chain s % 32 adds step s's products by fused multiply-adds, in the order
// j = 0 .. 7, lg = 0 .. 3 of k = 8 lg + j (the binary64 matrix instructions do just that
// over their own k, lg here, in both shapes); chains w, w + 8, w + 16, w + 24 join in this
// order to the sum of w = 0 .. 7, and these as waves_joined says.
constexpr int kChains = 4, kRouteWaves = 8;

__device__ __forceinline__ double bf16_to_f64(const uint4& v, int i) {
  const uint32_t w = i < 2 ? v.x : i < 4 ? v.y : i < 6 ? v.z : v.w;
  return (double)(i & 1 ? __uint_as_float(w & 0xFFFF0000u) : bf16_to_f32(w & 0xFFFFu));
}

template <class F>  // of(w): the sum of w
__device__ __forceinline__ auto waves_joined(F of) {
  auto s = of(0) + of(4);
#pragma unroll
  for (int w = 1; w < kRouteWaves / 2; ++w) s += of(w) + of(w + 4);
  return s;
}

// Few tokens: on v_mfma_f64_4x4x4_4b_f64 (lane l holds row l % 4 of both operands at k
// l / 16, of block l / 4 % 4, and row l / 16, column l % 4 of that block of D).  The
// blocks are the chains of one w, and its rows
//   4 tokens and 4 experts, with a w for each of eight wavefronts, or
//   ONE: four w of one token and one expert, in two wavefronts; of D only the diagonal
//     counts.  That takes four times the instructions, on sixteen times the
//     workgroups, and serves so few logits that CUs are idle (up to kOneLogits).
// A wavefront streams four rows of each operand, a step of every chain at a time, through
// LDS buffers of its own, kRouteDepth - 1 ahead (three and four buffers: 1 to 5% slower).  Bound
// by the conversions to binary64 (16 cycles each, two an instruction), for one token by
// the two launches.
constexpr int kRouteDepth = 2;

template <bool ONE>
__global__ __launch_bounds__(ONE ? 128 : 64 * kRouteWaves) void route_few_kernel(RouteArgs p) {
  static_assert(kChains == 4 && kRouteWaves == 8, "the blocks and rows of the instruction, the order of the joins");
  constexpr int D = kRouteDepth, N = ONE ? 1 : 4;
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  __shared__ double red[kRouteWaves][N * N];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int row = lane & 3, block = lane >> 2 & 3, lg = lane >> 4;
  const int e0 = blockIdx.x * N;
  const int64_t t0 = (int64_t)blockIdx.y * N;
  const __amdgpu_buffer_rsrc_t rx = buf_rsrc(p.x + t0 * p.k, kPastRange);
  const __amdgpu_buffer_rsrc_t rw = buf_rsrc(p.w + (int64_t)e0 * p.k, kPastRange);
  uint8_t* const mine = smem + wave * (D * 2048);
  // lane l loads row l / 16, block l / 4 % 4, lg l % 4 ^ row: what eight lanes read of LDS at
  // once (two blocks, four rows) then lies in different banks
  const int ahead = 8 * block + (ONE ? lg : 0);  // the lane's step, from the wavefront's first one on
  const int from = (ONE ? 0 : lg * p.k * 2) + ahead * 64 + 16 * (row ^ lg);
  const int at = 16 * (16 * row + 4 * block + (lg ^ row));
  const int steps = p.k / 32;
  const bool token = ONE || lg < p.m - t0, expert = ONE || lg < p.experts - e0;
  auto issue = [&](int buf, int s0) __attribute__((always_inline)) {
    const bool in = s0 + ahead < steps;  // past the ends zeros, which leave a sum as it is
    buf_to_lds(rx, mine + buf * 2048, in && token ? from + s0 * 64 : kPastRange);
    buf_to_lds(rw, mine + buf * 2048 + 1024, in && expert ? from + s0 * 64 : kPastRange);
  };
  const int first = ONE ? 4 * wave : wave;
#pragma unroll
  for (int i = 0; i < D - 1; ++i) issue(i, first + 32 * i);
  double sum = 0;
  int buf = 0;
  for (int s0 = first; s0 < steps; s0 += 32) {
    wait_lds();  // the buffer to be refilled has been read
    issue(buf == 0 ? D - 1 : buf - 1, s0 + 32 * (D - 1));
    wait_vm<2 * (D - 1)>();
    asm volatile("" ::: "memory");
    const uint4 a = *reinterpret_cast<const uint4*>(mine + buf * 2048 + at);
    const uint4 b = *reinterpret_cast<const uint4*>(mine + buf * 2048 + 1024 + at);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      sum = __builtin_amdgcn_mfma_f64_4x4x4f64(bf16_to_f64(a, j), bf16_to_f64(b, j), sum, 0, 0, 0);
    buf = buf == D - 1 ? 0 : buf + 1;
  }
  wait_vm<0>();  // the loads past the last step (zeros) end before the workgroup's LDS does
  sum = ((sum + __shfl_xor(sum, 4)) + __shfl_xor(sum, 8)) + __shfl_xor(sum, 12);  // (right where block is 0)
  if constexpr (ONE) {
    if (block == 0 && row == lg) red[4 * wave + row][0] = sum;
  } else {
    if (block == 0) red[wave][4 * lg + row] = sum;
  }
  __syncthreads();
  const int64_t t = t0 + threadIdx.x / N;
  const int e = e0 + threadIdx.x % N;
  if (threadIdx.x < N * N && t < p.m && e < p.experts) {
    const double s = waves_joined([&](int w) { return red[w][threadIdx.x]; });
    p.logits[t * p.experts + e] = (float)(s + (p.bias ? (double)p.bias[e] : -0.0));
  }
}

// More tokens: on v_mfma_f64_16x16x4_f64 (lane l holds A row and B column l % 16 at
// k l / 16, and rows 4 i + l / 16 of D's column l % 16).  A workgroup owns 16 TB tokens
// x 16 EB experts and each of its eight wavefronts the chains of one w: a lane loads
// eight values of each operand, whose j-th go into the j-th instruction.  Bound by the
// binary64 rate (64 cycles an instruction) and, at a third of that again, by the
// conversions of its operands.
//
// The forms, logits and choice in a graph, us:
//   ONE and 4 x 4: 64 logits of k = 2048 5.4, 5.6; 256 of k = 4096 7.1, 7.6; 256 (4 x 64) of
//     k = 2048 5.4, 5.6; 512 (8 x 64) 5.9, 5.9; 2048 (16 x 128) of k = 4096 8.7, 7.3;
//   4 x 4 and one block of 16 x 16, k = 4096: 64 x 256 12.7, 17.2; 384 x 64 13.8, 15.5; 192 x 160
//     17.8, 17.0; 128 x 256 18.2, 17.3; k = 1024: 96 x 160 8.8, 9.6; 192 x 160 10.9, 9.7;
//   one block fills the CUs evenly, 2 x 2 halve the conversions, from 1024 blocks on, k =
//     4096: 1000 x 161 37.6, 43.3; 1024 x 256 47.6, 44.0; 4096 x 128 86, 78; 8192 x 256 321,
//     286; a rule of their number alone, it is wrong where 2 x 2 leave a last round nearly
//     empty (1100 x 250 57, 78) or cover experts that are not there (16384 x 16 51, 81).
constexpr int64_t kOneLogits = 256, kFewLogits = 24576;
typedef double v4d __attribute__((ext_vector_type(4)));

template <int TB, int EB>  // blocks of 16 tokens and experts
__global__ __launch_bounds__(64 * kRouteWaves) void route_many_kernel(RouteArgs p) {
  constexpr int NW = kRouteWaves, H = NW / 2;
  __shared__ v4d red[H][TB * EB][64];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, lg = lane >> 4;
  const int e0 = blockIdx.x * 16 * EB;
  const int64_t t0 = (int64_t)blockIdx.y * 16 * TB;
  // rows past the ends read the last one (and are not stored)
  const uint16_t *px[TB], *pw[EB];
#pragma unroll
  for (int i = 0; i < TB; ++i) px[i] = p.x + min(t0 + 16 * i + r16, p.m - 1) * p.k + 8 * lg;
#pragma unroll
  for (int i = 0; i < EB; ++i) pw[i] = p.w + (int64_t)min(e0 + 16 * i + r16, p.experts - 1) * p.k + 8 * lg;
  const int steps = p.k / 32;
  uint4 x[TB], w[EB];
  auto load = [&](int s) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < TB; ++i) x[i] = *reinterpret_cast<const uint4*>(px[i] + s * 32);
#pragma unroll
    for (int i = 0; i < EB; ++i) w[i] = *reinterpret_cast<const uint4*>(pw[i] + s * 32);
  };
  if (wave < steps) load(wave);
  v4d sum[TB * EB];
#pragma unroll
  for (int b = 0; b < TB * EB; ++b) sum[b] = v4d{0, 0, 0, 0};
  // chain by chain, so that one chain's sums are all that is held beside the joined ones'
  for (int c = 0; c < kChains; ++c) {
    v4d acc[TB][EB];
#pragma unroll
    for (int i = 0; i < TB; ++i)
#pragma unroll
      for (int j = 0; j < EB; ++j) acc[i][j] = v4d{0, 0, 0, 0};
    for (int s = wave + NW * c; s < steps; s += NW * kChains) {
      uint4 a[TB], b[EB];
#pragma unroll
      for (int i = 0; i < TB; ++i) a[i] = x[i];
#pragma unroll
      for (int i = 0; i < EB; ++i) b[i] = w[i];
      const int on = s + NW * kChains, next = on < steps ? on : wave + NW * (c + 1);
      if (next < steps) load(next);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        double xa[TB], wb[EB];
#pragma unroll
        for (int i = 0; i < TB; ++i) xa[i] = bf16_to_f64(a[i], k);
#pragma unroll
        for (int i = 0; i < EB; ++i) wb[i] = bf16_to_f64(b[i], k);
#pragma unroll
        for (int i = 0; i < TB; ++i)
#pragma unroll
          for (int j = 0; j < EB; ++j)
            acc[i][j] = __builtin_amdgcn_mfma_f64_16x16x4f64(xa[i], wb[j], acc[i][j], 0, 0, 0);
      }
    }
#pragma unroll
    for (int i = 0; i < TB; ++i)
#pragma unroll
      for (int j = 0; j < EB; ++j) sum[i * EB + j] += acc[i][j];
  }
  if (wave >= H) {
#pragma unroll
    for (int b = 0; b < TB * EB; ++b) red[wave - H][b][lane] = sum[b];
  }
  __syncthreads();
  if (wave < H) {
#pragma unroll
    for (int b = 0; b < TB * EB; ++b) red[wave][b][lane] += sum[b];
  }
  __syncthreads();
  for (int b = wave; b < TB * EB; b += NW) {
    v4d s = red[0][b][lane];  // in the order of waves_joined
#pragma unroll
    for (int h = 1; h < H; ++h) s += red[h][b][lane];
    const int e = e0 + 16 * (b % EB) + r16;
    if (e >= p.experts) continue;
    const double bias = p.bias ? (double)p.bias[e] : -0.0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t t = t0 + 16 * (b / EB) + 4 * i + lg;
      if (t < p.m) p.logits[t * p.experts + e] = (float)(s[i] + bias);
    }
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

// A wavefront per token: `top` rounds of a wavefront-wide maximum, of whose lanes
// the lowest expert is taken; lane j then holds the j-th choice.  The weights are
// formed relative to the best, so no exponential overflows.
template <int PER>  // experts per lane
__global__ __launch_bounds__(256) void route_select_kernel(RouteArgs a) {
  const int lane = threadIdx.x & 63;
  const int64_t t = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  if (t >= a.m) return;
  const int top = a.top, score = a.score;
  const bool renormalize = a.renormalize;
  float v[PER];
  uint32_t key[PER];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = lane + 64 * i;
    v[i] = e < a.experts ? a.logits[t * a.experts + e] : -__builtin_inff();
    key[i] = order_of(v[i]);
  }
  float chosen = -__builtin_inff(), best = 0.0f;
  int id = -1;
  for (int j = 0; j < top; ++j) {
    uint32_t k = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) k = max(k, key[i]);
    k = wave_max(k);
    if (k == 0) break;  // nothing left: lanes j .. keep id -1
    bool found = false;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const uint64_t at = __ballot(key[i] == k);
      if (!found && at != 0) {
        found = true;
        const int l = __builtin_ctzll(at);
        const float value = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(v[i]), l));
        if (lane == l) key[i] = 0;
        if (j == 0) best = value;
        if (lane == j) {
          id = l + 64 * i;
          chosen = value;
        }
      }
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
    a.ids[t * top + lane] = id;
    a.weights[t * top + lane] = p;
  }
}

// ---------------------------------------------------------------------------
// The layer
//
// Every workgroup reads ids by itself and finds its expert's tokens; a weight in
// any of its forms is staged in LDS as it is stored and becomes bf16 operands there
// (exactly: 8-bit integers and 4-bit floats with their scale are bf16 numbers;
// the 8-bit form's row scales multiply the sums).  h = act(g) u is formed from
// binary32 sums and rounded to bf16 in the workspace, at row (token, first slot of
// the expert).
// ---------------------------------------------------------------------------

// What a workgroup knows of the tokens' choices, in two forms with the same calls.
// ids outside [0, experts) are no choice.
//   count          chosen experts
//   expert(i)      the i-th of them (uniform)
//   slot(e)        in lane t: token t's first slot with expert e, or -1
//   weight(e)      in lane t: the sum of its weights over its slots with e

// Up to 64 slots in all: a lane holds one (lane = t * top + s), and ballots do the
// rest, without LDS or a barrier (one token, 6 of 64 experts: 21.5 us a layer with the
// form below, 19.9).  Experts in the order of their first slots.
struct FewChoices {
  const MoeArgs& p;
  int id;
  float w;
  uint64_t firsts;  // slots that name an expert first
  int count;
  template <bool WEIGHTS>
  __device__ __forceinline__ FewChoices(const MoeArgs& p_, int lane, std::bool_constant<WEIGHTS>)
      : p(p_), id(-1), w(0.f), firsts(0) {
    if (lane < p.m * p.top) {
      const int v = p.ids[lane];
      if constexpr (WEIGHTS) w = p.weights[lane];
      if (v >= 0 && v < p.experts) id = v;
    }
    for (uint64_t rest = __ballot(id >= 0); rest != 0;) {
      const int first = __builtin_ctzll(rest);
      firsts |= (uint64_t)1 << first;
      rest &= ~__ballot(id == __builtin_amdgcn_readlane(id, first));
    }
    count = __popcll(firsts);
  }
  __device__ __forceinline__ int expert(int i) const {
    uint64_t f = firsts;
    for (; i > 0; --i) f &= f - 1;
    return __builtin_amdgcn_readlane(id, __builtin_ctzll(f));
  }
  // token t's bits of a mask over slots, for lane t
  __device__ __forceinline__ uint32_t mine(uint64_t slots, int lane) const {
    return lane < p.m ? (uint32_t)(slots >> (lane * p.top)) & ((1u << p.top) - 1) : 0;
  }
  __device__ __forceinline__ int slot(int e, int lane) const {
    const uint32_t s = mine(__ballot(id == e), lane);
    return s ? __builtin_ctz(s) : -1;
  }
  __device__ __forceinline__ float weight(int e, int lane) const {
    const uint32_t slots = mine(__ballot(id == e), lane);
    float sum = 0.f;
    for (int s = 0; s < p.top; ++s) {
      const float v = __shfl(w, lane * p.top + s & 63);
      sum += slots >> s & 1 ? v : 0.f;
    }
    return sum;
  }
};

// Any number: ids in LDS, and a bit per chosen expert, whose words a wavefront's
// lanes then hold.  Experts in ascending order.
struct ManyChoices {
  struct Shared {
    int ids[kMoeTokens * kMoeTop];
    uint32_t bits[kMoeExperts / 32];
  };
  const MoeArgs& p;
  const int* ids;
  uint32_t word;  // lane l < 32: bits of experts 32 l ..
  int upto;       // chosen experts up to this word's end
  int count;
  __device__ __forceinline__ ManyChoices(const MoeArgs& p_, Shared& c, int lane) : p(p_), ids(c.ids) {
    static_assert(kMoeExperts <= 64 * 32, "a word per lane");
    for (int i = threadIdx.x; i < kMoeExperts / 32; i += blockDim.x) c.bits[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < p.m * p.top; i += blockDim.x) {
      const int id = p.ids[i];
      const bool in = id >= 0 && id < p.experts;
      c.ids[i] = in ? id : -1;
      if (in) atomicOr(&c.bits[id / 32], 1u << (id & 31));
    }
    __syncthreads();
    word = lane < kMoeExperts / 32 ? c.bits[lane] : 0;
    upto = __popc(word);
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
      const int before = __shfl_up(upto, d);
      if (lane >= d) upto += before;
    }
    count = __builtin_amdgcn_readlane(upto, 63);
  }
  __device__ __forceinline__ int expert(int i) const {
    const int l = __builtin_ctzll(__ballot(upto > i));
    uint32_t w = (uint32_t)__builtin_amdgcn_readlane((int)word, l);
    for (int skip = i - (__builtin_amdgcn_readlane(upto, l) - __popc(w)); skip > 0; --skip) w &= w - 1;
    return 32 * l + __builtin_ctz(w);
  }
  __device__ __forceinline__ int slot(int e, int lane) const {
    int found = -1;
    if (lane < p.m)
      for (int s = p.top - 1; s >= 0; --s) found = ids[lane * p.top + s] == e ? s : found;
    return found;
  }
  __device__ __forceinline__ float weight(int e, int lane) const {
    float sum = 0.f;
    if (lane < p.m)
      for (int s = 0; s < p.top; ++s)
        if (ids[lane * p.top + s] == e) sum += p.weights[lane * p.top + s];
    return sum;
  }
};

// Sizes of a unit: UK_ k of RT weight tiles of 16 rows, and of R activation rows.
template <int WF, int RT, int R, int UK_>
struct Unit {
  static constexpr int UK = UK_;
  static constexpr int WROW = WF == EXPERT_BF16 ? UK * 2 : WF == EXPERT_INT8 ? UK : UK / 2, XROW = UK * 2;
  static constexpr int WL = 16 * WROW / 1024, SL = WF == EXPERT_FP4 ? (16 * (UK / 32) + 63) / 64 : 0;  // loads
  static constexpr int XL = (R * XROW + 1023) / 1024;
  static constexpr int TILE = WL * 1024 + SL * 256, WBYTES = RT * TILE, XBYTES = XL * 1024;
  // 16-byte chunk c of weight row r lies at chunk c ^ swizzle(r): eight rows of one
  // chunk take the 128 bytes of an LDS cycle once
  __device__ static __forceinline__ int swizzle(int r) { return WROW >= 128 ? r & 7 : r >> 1 & 3; }
};
// k of a unit where a wavefront streams both operands by itself
constexpr int stream_k(int form) { return form == EXPERT_BF16 ? 128 : 256; }

template <int WF>
__device__ __forceinline__ int row_bytes(int k) {
  return WF == EXPERT_BF16 ? k * 2 : WF == EXPERT_INT8 ? k : k / 2;
}

// Puts a unit's 16 weight rows and (4-bit) scales in flight: k from u UK on, of
// which `left` exist (zeros past them; none for left <= 0).  Non-temporal: the weight is read once.
template <int WF, class U>
__device__ __forceinline__ void issue_weight(__amdgpu_buffer_rsrc_t rw, __amdgpu_buffer_rsrc_t rs, uint8_t* b, int u,
                                             int left, int k, int lane) {
  constexpr int WC = U::WROW / 16, WPL = 64 / WC, PER = U::UK / WC;  // chunks per row, rows per load, k per chunk
#pragma unroll
  for (int j = 0; j < U::WL; ++j) {
    const int row = j * WPL + lane / WC, c = (lane % WC) ^ U::swizzle(row);
    buf_to_lds<true>(rw, b + j * 1024, c * PER < left ? row * row_bytes<WF>(k) + u * U::WROW + c * 16 : kPastRange);
  }
#pragma unroll
  for (int j = 0; j < U::SL; ++j) {
    constexpr int BC = U::UK / 32;  // blocks per row
    const int row = j * (64 / BC) + lane / BC, c = lane % BC;
    buf_byte_to_lds(rs, b + U::WL * 1024 + j * 256, c * 32 < left ? row * (k / 32) + u * BC + c : kPastRange);
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

// acc[t][b] += (weight tile t, at w) (activation rows 16 b .., at xb) over one unit.
template <int WF, int RT, int RB, int R, class U>
__device__ __forceinline__ void multiply_unit(v4f (&acc)[RT][RB], const uint8_t* b, const uint8_t* xb, int lane) {
  const int r16 = lane & 15, lg = lane >> 4, sw = U::swizzle(r16);
#pragma unroll
  for (int s = 0; s < U::UK / 128; ++s) {
    v8bf x[RB][4];
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
      const int row = min(16 * rb + r16, R - 1);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = 16 * s + (WF == EXPERT_BF16 ? 4 * j + lg : 4 * lg + j);
        x[rb][j] = *reinterpret_cast<const v8bf*>(xb + row * U::XROW + 16 * (c ^ (row & 7)));
      }
    }
    // two weight tiles at a time: a product's wait for its sum is the other's turn
    constexpr int P = RT % 2 == 0 ? 2 : 1;
#pragma unroll
    for (int t0 = 0; t0 < RT; t0 += P) {
      v8bf w[P][4];
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const uint8_t* const tile = b + (t0 + i) * U::TILE;
        const uint8_t* const wb = tile + r16 * U::WROW;
        if constexpr (WF == EXPERT_BF16) {
#pragma unroll
          for (int j = 0; j < 4; ++j) w[i][j] = *reinterpret_cast<const v8bf*>(wb + 16 * ((16 * s + 4 * j + lg) ^ sw));
        } else if constexpr (WF == EXPERT_INT8) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const v4i q = *reinterpret_cast<const v4i*>(wb + 16 * ((8 * s + 2 * lg + h) ^ sw));
            w[i][2 * h] = widen8_int8((uint32_t)q[0], (uint32_t)q[1]);
            w[i][2 * h + 1] = widen8_int8((uint32_t)q[2], (uint32_t)q[3]);
          }
        } else {
          const v4i q = *reinterpret_cast<const v4i*>(wb + 16 * ((4 * s + lg) ^ sw));
          const float f = mx_scale_value(
              *reinterpret_cast<const uint32_t*>(tile + U::WL * 1024 + 4 * (r16 * (U::UK / 32) + 4 * s + lg)));
#pragma unroll
          for (int j = 0; j < 4; ++j) w[i][j] = __builtin_bit_cast(v8bf, mx_widen8_e2m1((uint32_t)q[j], f));
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < P; ++i)
#pragma unroll
          for (int rb = 0; rb < RB; ++rb) acc[t0 + i][rb] = mfma16(w[i][j], x[rb][j], acc[t0 + i][rb]);
    }
  }
}

__device__ __forceinline__ float gate_value(int act, float g) {
  return act == ACT_SILU        ? act_value<ACT_SILU>(g)
         : act == ACT_GELU_TANH ? act_value<ACT_GELU_TANH>(g)
                                : act_value<ACT_RELU>(g);
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

// ---------------------------------------------------------------------------
// Few tokens: the weight rows are streamed the way the few-row products do
// (stream.hip): wavefronts take units of UK k in LDS buffers of their own, D - 1
// units ahead, 16 RT weight rows a workgroup, and add their sums in a fixed order
// at the end.  The weight is loaded non-temporally, being read once.
//
// Up: a workgroup owns RT / 2 pairs of gate and up row tiles of one expert, and
//   runs them on that expert's tokens (at most R), gathered by their rows of x.
// Down: a workgroup owns 16 RT columns of out for all tokens and walks all chosen
//   experts; its wavefronts take even shares of their units.  Tokens are the
//   columns of the product, zeros where a token did not choose the expert; at the
//   end of an expert a token's sums are added to its total with its weight, and
//   only where it did choose it, so that an infinity in a weight stays with the
//   tokens that met it.
//
// One token, 2 of 8 experts, k = 4096, f = 14336, bf16: up 72 us, down 37, 6.4 TB/s; 8-bit
// 70 us together, 4-bit 43.  With little to read the two launches' latencies are
// most of the time: 6 of 64, k = 2048, f = 1408, 8-bit 10.1 + 7.6 us for 52 MB.
// ---------------------------------------------------------------------------

// LDS of these kernels.
template <int WF, int RT, int R, int NW, int D>
struct Streamed : Unit<WF, RT, R, stream_k(WF)> {
  using U = Unit<WF, RT, R, stream_k(WF)>;
  static constexpr int LOADS = RT * (U::WL + U::SL) + U::XL, BYTES = U::WBYTES + U::XBYTES;
  static constexpr int RED = NW * RT * R * 16 * 4;
  static constexpr int LDS = NW * D * BYTES > RED ? NW * D * BYTES : RED;
  static_assert((D - 1) * LOADS < 64, "wait counts");
};

template <int WF, int RT, int R, int NW, int D>
__global__ __launch_bounds__(64 * NW) void moe_up_kernel(MoeArgs p) {
  using U = Unit<WF, RT, R, stream_k(WF)>;
  using L = Streamed<WF, RT, R, NW, D>;
  static_assert(RT % 2 == 0, "row tiles come in pairs");
  constexpr int RB = (R + 15) / 16;
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  __shared__ int rows[kMoeTokens], pairs[kMoeTokens];  // the expert's tokens, and their rows of h
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, lg = lane >> 4;

  const FewChoices chosen(p, lane, std::false_type{});
  if ((int)blockIdx.y >= chosen.count) return;
  const int e = chosen.expert(blockIdx.y), slot = chosen.slot(e, lane);
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
  uint8_t* const mine = smem + wave * (D * L::BYTES);
  const int units = (K + U::UK - 1) / U::UK;
  constexpr int XC = U::XROW / 16, XPL = 64 / XC;

  int xoff[U::XL];
#pragma unroll
  for (int j = 0; j < U::XL; ++j) {
    const int row = j * XPL + lane / XC;
    xoff[j] = row < count ? rows[row] * (K * 2) + 16 * ((lane % XC) ^ (row & 7)) : kPastRange;
  }
  auto issue = [&](int at, int u) __attribute__((always_inline)) {
    uint8_t* b = mine + at * L::BYTES;
    const int left = K - u * U::UK;  // may be negative: every lane masked
#pragma unroll
    for (int t = 0; t < RT; ++t) issue_weight<WF, U>(rw[t], rs[t], b + t * U::TILE, u, left, K, lane);
#pragma unroll
    for (int j = 0; j < U::XL; ++j) {
      const int c = (lane % XC) ^ ((j * XPL + lane / XC) & 7);
      const bool in = c * 8 < left && xoff[j] != kPastRange;
      buf_to_lds(rx, b + U::WBYTES + j * 1024, in ? xoff[j] + u * U::XROW : kPastRange);
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
    wait_vm<(D - 1) * L::LOADS>();
    asm volatile("" ::: "memory");
    multiply_unit<WF, RT, RB, R, U>(acc, mine + at * L::BYTES, mine + at * L::BYTES + U::WBYTES, lane);
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
      if (16 * b + r16 < count)
        *reinterpret_cast<v4f*>(red + ((wave * RT + t) * R + 16 * b + r16) * 16 + 4 * lg) = acc[t][b];
  wait_lds();
  wg_barrier();
  constexpr int OT = RT / 2;
  for (int i = threadIdx.x; i < OT * 16 * count; i += 64 * NW) {
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
    const float h = u * gate_value(p.act, g);
    p.h[(int64_t)pairs[r] * p.f + col] = (uint16_t)pack_bf16x2(h, 0.f);
  }
}

template <int WF, int RT, int R, int NW, int D>
__global__ __launch_bounds__(64 * NW) void moe_down_kernel(MoeArgs p) {
  using U = Unit<WF, RT, R, stream_k(WF)>;
  using L = Streamed<WF, RT, R, NW, D>;
  constexpr int RB = (R + 15) / 16;
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, lg = lane >> 4;
  const int F = p.f, tile0 = blockIdx.x * RT, tiles = p.k / 16;

  const FewChoices chosen(p, lane, std::true_type{});
  const int each = (F + U::UK - 1) / U::UK, units = chosen.count * each;
  const int share = (units + NW - 1) / NW, first = min(wave * share, units), last = min(first + share, units);

  const __amdgpu_buffer_rsrc_t rh = buf_rsrc(p.h, kPastRange);
  uint8_t* const mine = smem + wave * (D * L::BYTES);
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
    const int slot = chosen.slot(e, lane);
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
    uint8_t* b = mine + at * L::BYTES;
    if (next < last && unit_in == each) {
      ++expert_in;
      unit_in = 0;
      enter(expert_in);
    }
    const int left = next < last ? F - unit_in * U::UK : 0;
#pragma unroll
    for (int t = 0; t < RT; ++t) issue_weight<WF, U>(rw[t], rs[t], b + t * U::TILE, unit_in, left, F, lane);
#pragma unroll
    for (int j = 0; j < U::XL; ++j) {
      const int c = (lane % XC) ^ ((j * XPL + lane / XC) & 7);
      const bool in = c * 8 < left && hoff[j] != kPastRange;
      buf_to_lds(rh, b + U::WBYTES + j * 1024, in ? hoff[j] + unit_in * U::XROW : kPastRange);
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
      wait_vm<(D - 1) * L::LOADS>();
      asm volatile("" ::: "memory");
      multiply_unit<WF, RT, RB, R, U>(acc, mine + at * L::BYTES, mine + at * L::BYTES + U::WBYTES, lane);
      at = at == D - 1 ? 0 : at + 1;
      if (++unit_at == each || u + 1 == last) {  // the expert's end, or this share's
        const int e = chosen.expert(expert_at);
        const float weight = chosen.weight(e, lane);
        const uint64_t takers = __ballot(chosen.slot(e, lane) >= 0);
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

// ---------------------------------------------------------------------------
// More tokens: a workgroup owns NW wavefronts' weight tiles of one expert and all
// of k, and its wavefronts share the expert's activation rows, gathered: each
// puts its own weight tiles and a share of the activation in flight, D - 1 units
// ahead, and one barrier a unit publishes them.  The weight, read once, is loaded
// non-temporally (a layer for 64 tokens, 2 of 8 experts, k = 4096, f = 14336, 8-bit 297 -> 256
// us, bf16 501 -> 458; 16 tokens, 8 of 64, k = 2048, f = 1408, bf16 139 -> 127).  The
// number of 16-row blocks of the expert's tokens picks the loop (NB), and with it how
// many units fit LDS.
// The groups of NW wavefronts' tiles of all chosen experts are split evenly over as
// many workgroups as the CUs hold.  A group of an expert with many tokens takes longer
// where the weight has to be converted, so 8- and 4-bit groups are dealt out one by one
// when an expert can have more than 16 tokens; else in runs, whose units stay in flight
// from one group to the next (us, dealt against runs: 64 tokens, 2 of 8 experts, k = 4096,
// f = 14336, 8-bit 251, 298; 8 of 64, k = 2048, f = 1408, 8-bit 102, 123, 4-bit 88, 103, bf16 179,
// 166; 16 tokens, bf16 128, 118, 4-bit 65, 61).
//
// Up: RT / 2 pairs of gate and up tiles a wavefront; h as above.
// Down: RT tiles of 16 columns; weight times the sums go to the workspace in
//   binary32, a row per (token, first slot of the expert), which
//   moe_combine_kernel adds in the order of the slots: a token's result then
//   depends on nothing but the token.
// ---------------------------------------------------------------------------
struct TileShared {
  int rows[kMoeTokens], pairs[kMoeTokens];  // the expert's tokens, and their rows of h
  float weights[kMoeTokens];                // DOWN: over all the token's slots with the expert
};

template <int WF, bool DOWN, int RT, int NW, int UK, int POOL, int NB>
__device__ __forceinline__ void moe_tiles(const MoeArgs& p, const TileShared& sh, int e, int count, int g0, int g1,
                                          uint8_t* smem, int lane, int wave) {
  using U = Unit<WF, RT, 16 * NB, UK>;
  // every wavefront the same number of the activation's loads; those past its end write zeros
  constexpr int XL = (U::XL + NW - 1) / NW, LOADS = RT * (U::WL + U::SL) + XL, STAGE = NW * (U::WBYTES + XL * 1024);
  constexpr int D = POOL / STAGE < 6 ? POOL / STAGE : 6;
  static_assert(D >= 2 && (D - 2) * LOADS < 64, "units in LDS, wait counts");
  const int r16 = lane & 15, lg = lane >> 4;
  const int K = DOWN ? p.f : p.k, N = DOWN ? p.k : p.f;  // N: columns of the result
  constexpr int CT = DOWN ? RT : RT / 2;                 // its tiles of a wavefront
  const int tiles = N / 16;
  __amdgpu_buffer_rsrc_t rw[RT], rs[RT];
  // the tiles of group g; past the last one, the last one again (and not stored)
  auto enter = [&](int g) __attribute__((always_inline)) {
    const int tile0 = (g * NW + wave) * CT;
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      const int64_t row = DOWN ? (int64_t)e * N + min(tile0 + t, tiles - 1) * 16
                               : (int64_t)e * 2 * N + min(tile0 + t / 2, tiles - 1) * 16 + (t & 1 ? N : 0);
      rw[t] = weight_rows<WF>(DOWN ? p.w_down : p.w_gu, row, K);
      rs[t] = scale_rows<WF>(DOWN ? p.s_down : p.s_gu, row, K);
    }
  };
  const __amdgpu_buffer_rsrc_t rx = buf_rsrc(DOWN ? p.h : p.x, kPastRange);
  const int units = (K + U::UK - 1) / U::UK;
  constexpr int XC = U::XROW / 16, XPL = 64 / XC;
  int xoff[XL];
#pragma unroll
  for (int j = 0; j < XL; ++j) {
    const int row = (wave * XL + j) * XPL + lane / XC;
    xoff[j] = row < count ? (DOWN ? sh.pairs : sh.rows)[row] * (K * 2) + 16 * ((lane % XC) ^ (row & 7)) : kPastRange;
  }
  int group_in = g0, unit_in = 0;  // what is put in flight next
  enter(g0);
  auto issue = [&](int at) __attribute__((always_inline)) {
    if (unit_in == units && group_in + 1 < g1) {
      ++group_in;
      unit_in = 0;
      enter(group_in);
    }
    uint8_t* const b = smem + at * STAGE;
    const int left = K - unit_in * U::UK;  // not positive past the last unit: every lane masked
#pragma unroll
    for (int t = 0; t < RT; ++t)
      issue_weight<WF, U>(rw[t], rs[t], b + wave * U::WBYTES + t * U::TILE, unit_in, left, K, lane);
#pragma unroll
    for (int j = 0; j < XL; ++j) {
      const int row = (wave * XL + j) * XPL + lane / XC, c = (lane % XC) ^ (row & 7);
      const bool in = c * 8 < left && xoff[j] != kPastRange;
      buf_to_lds(rx, b + NW * U::WBYTES + (wave * XL + j) * 1024, in ? xoff[j] + unit_in * U::XROW : kPastRange);
    }
    ++unit_in;
  };
#pragma unroll
  for (int i = 0; i < D - 1; ++i) issue(i);
  int at = 0;
  for (int g = g0; g < g1; ++g) {
    v4f acc[RT][NB];
#pragma unroll
    for (int t = 0; t < RT; ++t)
#pragma unroll
      for (int b = 0; b < NB; ++b) acc[t][b] = v4f{0.f, 0.f, 0.f, 0.f};
    for (int u = 0; u < units; ++u) {
      wait_vm<(D - 2) * LOADS>();  // the oldest unit of this wavefront in flight has landed
      wait_lds();                  // and its reads of the stage to be refilled are done
      wg_barrier();
      issue(at == 0 ? D - 1 : at - 1);
      const uint8_t* const b = smem + at * STAGE;
      multiply_unit<WF, RT, NB, 16 * NB, U>(acc, b + wave * U::WBYTES, b + NW * U::WBYTES, lane);
      at = at == D - 1 ? 0 : at + 1;
    }
    // rows of the result: lane r16 of block b, four columns from 4 lg on
    const int tile0 = (g * NW + wave) * CT;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
      const int r = 16 * b + r16;
      if (r >= count) continue;
      const int64_t pair = sh.pairs[r];
#pragma unroll
      for (int t = 0; t < CT; ++t) {
        if (tile0 + t >= tiles) continue;
        const int col = (tile0 + t) * 16 + 4 * lg;
        if constexpr (DOWN) {
          v4f y = acc[t][b];
          if constexpr (WF == EXPERT_INT8)
            y *= *reinterpret_cast<const v4f*>(static_cast<const float*>(p.s_down) + (int64_t)e * N + col);
          *reinterpret_cast<v4f*>(p.y + pair * N + col) = y * sh.weights[r];
        } else {
          v4f g4 = acc[2 * t][b], v = acc[2 * t + 1][b];
          if constexpr (WF == EXPERT_INT8) {
            const float* s = static_cast<const float*>(p.s_gu) + (int64_t)e * 2 * N + col;
            g4 *= *reinterpret_cast<const v4f*>(s);
            v *= *reinterpret_cast<const v4f*>(s + N);
          }
          float h[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) h[i] = gate_value(p.act, g4[i]) * v[i];
          *reinterpret_cast<uint2*>(p.h + pair * N + col) =
              make_uint2(pack_bf16x2(h[0], h[1]), pack_bf16x2(h[2], h[3]));
        }
      }
    }
  }
  wait_vm<0>();  // the loads past the last unit (zeros) end before the LDS is used for anything else
}

template <int WF, bool DOWN, int RT, int NW, int UK, int POOL>
__global__ __launch_bounds__(64 * NW) void moe_tile_kernel(MoeArgs p) {
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  __shared__ ManyChoices::Shared shared;
  __shared__ TileShared sh;
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const ManyChoices chosen(p, shared, lane);
  constexpr int cover = NW * (DOWN ? RT : RT / 2) * 16;
  const int groups = ((DOWN ? p.k : p.f) + cover - 1) / cover, tasks = chosen.count * groups;
  const int blocks = gridDim.x, share = (tasks + blocks - 1) / blocks;
  const bool deal = WF != EXPERT_BF16 && p.m > 16;
  const int last = deal ? tasks : min((int)(blockIdx.x + 1) * share, tasks);
  for (int task = deal ? blockIdx.x : blockIdx.x * share; task < last;) {
    const int i = task / groups, g0 = task - i * groups, g1 = deal ? g0 + 1 : min(groups, g0 + last - task);
    task += deal ? blocks : g1 - g0;
    const int e = chosen.expert(i), slot = chosen.slot(e, lane);
    const uint64_t takers = __ballot(slot >= 0);
    __syncthreads();  // the expert before is done with its lists and the stages
    if (wave == 0) {
      const float w = DOWN ? chosen.weight(e, lane) : 0.f;
      if (slot >= 0) {
        const int r = __popcll(takers & (((uint64_t)1 << lane) - 1));
        sh.rows[r] = lane;
        sh.pairs[r] = lane * p.top + slot;
        sh.weights[r] = w;
      }
    }
    __syncthreads();
    const int count = __popcll(takers);
    if (count <= 16) moe_tiles<WF, DOWN, RT, NW, UK, POOL, 1>(p, sh, e, count, g0, g1, smem, lane, wave);
    else if (count <= 32) moe_tiles<WF, DOWN, RT, NW, UK, POOL, 2>(p, sh, e, count, g0, g1, smem, lane, wave);
    else if (count <= 48) moe_tiles<WF, DOWN, RT, NW, UK, POOL, 3>(p, sh, e, count, g0, g1, smem, lane, wave);
    else moe_tiles<WF, DOWN, RT, NW, UK, POOL, 4>(p, sh, e, count, g0, g1, smem, lane, wave);
  }
}

// out[t] = the sum of its experts' parts in the order of the slots, rounded once.
__global__ __launch_bounds__(256) void moe_combine_kernel(MoeArgs p) {
  const int t = blockIdx.y, c = blockIdx.x * 256 + threadIdx.x, lane = threadIdx.x & 63;
  int id = lane < p.top ? p.ids[t * p.top + lane] : -1;
  if (id >= p.experts) id = -1;
  uint32_t firsts = 0;  // slots that name an expert first
  for (uint64_t rest = __ballot(id >= 0); rest != 0;) {
    const int first = __builtin_ctzll(rest);
    firsts |= 1u << first;
    rest &= ~__ballot(id == __builtin_amdgcn_readlane(id, first));
  }
  if (c >= p.k / 4) return;
  const v4f* const y = reinterpret_cast<const v4f*>(p.y + (int64_t)t * p.top * p.k) + c;
  v4f s = v4f{0.f, 0.f, 0.f, 0.f};
  for (int i = 0; i < p.top; i += 4) {  // four loads in flight
    v4f v[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      v[j] = firsts >> (i + j) & 1 ? y[(int64_t)(i + j) * (p.k / 4)] : v4f{-0.f, -0.f, -0.f, -0.f};
#pragma unroll
    for (int j = 0; j < 4; ++j) s += v[j];
  }
  reinterpret_cast<uint2*>(p.out + (int64_t)t * p.k)[c] = make_uint2(pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3]));
}

template <class K>
hipError_t allow_lds(K* kernel, int bytes) {
  return bytes > 49152 ? hipFuncSetAttribute(reinterpret_cast<const void*>(kernel),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, bytes)
                       : hipSuccess;
}

int64_t align256(int64_t b) { return (b + 255) / 256 * 256; }

constexpr int kWhole = 148 * 1024, kHalf = 74 * 1024, kLess = 50 * 1024, kThird = 48 * 1024;
constexpr int kLdsLeft = 160 * 1024 - (int)sizeof(ManyChoices::Shared) - (int)sizeof(TileShared);
// Whether the layer is two launches of the streaming kernels, or three of the tiled
// ones.  Every workgroup that streams loads all tokens' activation for 16 or 32
// weight rows, where the tiled ones share it, so it is for few tokens on few
// experts (us, streamed against tiled: 8 tokens E8 8-bit 182, 208, bf16 351, 345; 5 tokens
// E8 4-bit 105, 126; 4 tokens on 4 of 16 experts of 1024 x 512 8-bit 14.1, 16.9; but 4
// tokens E64 bf16 89, 88, 8-bit 59, 48; 8 tokens E64 8-bit 87, 63).  The rule looks at
// neither k, f nor the weight's form.  Over 305 layers of one to eight tokens it loses 4.6%
// against the better of the two in the mean: up to two tokens 0.9% (at most 35%); three to
// eight with top <= 4 5.3%, of k < 1100 and f > 3000 27% (5 tokens, 8-bit, k = 320, f = 6752
// 68, 40), since streaming the down rows keeps k / 16 workgroups busy; with top > 4 6.8%, of k
// >= 2000 9.8% (4 tokens on 8 of 23 experts, 4-bit, 4064 x 1120 48, 68).
bool streamed(int64_t m, int top) { return m <= 2 || (m <= 8 && top <= 4); }

template <int WF, int RT, int R, int NW, int D>
hipError_t run_up(const MoeArgs& p, hipStream_t stream) {
  constexpr int bytes = Streamed<WF, RT, R, NW, D>::LDS, cover = RT / 2 * 16;
  static_assert(bytes <= kLdsLeft, "LDS of a CU");
  auto* kernel = moe_up_kernel<WF, RT, R, NW, D>;
  const hipError_t e = allow_lds(kernel, bytes);
  if (e != hipSuccess) return e;
  const dim3 grid((unsigned)((p.f + cover - 1) / cover), (unsigned)min(p.experts, p.m * p.top));
  kernel<<<grid, dim3(64 * NW), bytes, stream>>>(p);
  return hipGetLastError();
}

template <int WF, int RT, int R, int NW, int D>
hipError_t run_down(const MoeArgs& p, hipStream_t stream) {
  constexpr int bytes = Streamed<WF, RT, R, NW, D>::LDS, cover = RT * 16;
  static_assert(bytes <= kLdsLeft, "LDS of a CU");
  auto* kernel = moe_down_kernel<WF, RT, R, NW, D>;
  const hipError_t e = allow_lds(kernel, bytes);
  if (e != hipSuccess) return e;
  kernel<<<dim3((unsigned)((p.k + cover - 1) / cover)), dim3(64 * NW), bytes, stream>>>(p);
  return hipGetLastError();
}

template <int WF, bool DOWN, int RT, int NW, int UK, int POOL>
hipError_t run_tile(const MoeArgs& p, hipStream_t stream) {
  constexpr int cover = NW * (DOWN ? RT : RT / 2) * 16;
  static_assert(POOL <= kLdsLeft, "LDS of a CU");
  auto* kernel = moe_tile_kernel<WF, DOWN, RT, NW, UK, POOL>;
  const hipError_t e = allow_lds(kernel, POOL);
  if (e != hipSuccess) return e;
  // as many workgroups as the CUs hold, fewer where there are not so many groups of tiles
  const int n = DOWN ? p.k : p.f, most = min(p.experts, p.m * p.top) * ((n + cover - 1) / cover);
  constexpr int fit = 256 * (160 * 1024 / (POOL + (int)sizeof(ManyChoices::Shared) + (int)sizeof(TileShared)));
  kernel<<<dim3((unsigned)min(most, fit)), dim3(64 * NW), POOL, stream>>>(p);
  return hipGetLastError();
}

// The tiled forms, by tiles, wavefronts and k of a unit; LDS for one workgroup of a CU
// (kWhole), two (kHalf, kLess: fewer units ahead) or three (kThird).  Where there are
// few tiles, small workgroups: more of them, and the last round of groups wastes less;
// where there are many, large ones, which read the tokens' rows from LDS and memory less
// often.  `most` bounds the tiles of 16 result columns over the experts that can be
// chosen.  Measured on 300 layers of 4 to 128 experts, k and f from 256 to 4096 and 14336, 3
// to 64 tokens (lengths over the best of ten forms, in the mean), and on 24 large ones:
//   up   bf16  2, 2, 128 kHalf 0.9%, 2, 4, 128 kWhole 4.8%, parted at 45 tokens 0.7%; of 64
//              tokens, 8 of 32 experts, k = 7168, f = 2048 505 us and 465, of 24 403 and 465
//        8-bit 2, 4, 128 kHalf 2.6%, 2, 2, 128 kLess 2.9%, parted at 640 tiles 2.1%; before,
//              4, 4, 128 kWhole, 16% (equal for 64 tokens, 2 of 8 experts, k = 4096, f = 14336)
//        4-bit 2, 8, 256 kWhole 7.3%, 2, 2, 128 kLess 4.0%, parted at 1700 tiles 1.0%; of 64
//              tokens, 2 of 8 experts 220 us and 289
//   down bf16  1, 2, 128 kHalf 3.2%, 1, 4, 256 kWhole 5.1%, 2, 4, 128 kWhole 12%, parted as
//              below 2.0%; of the large layers with up to 16 tokens 1, 4, 256 is the faster one
//              (16 of 4096 x 4096, 16 tokens 149 us, 2, 4, 128 166), with 64 2, 4, 128 (531, 562)
//        8-bit 1, 4, 128 kThird 1.9%, 1, 8, 128 kHalf 8.7%, parted at 2048 tiles 1.4%; with more
//              than 16 tokens 1, 4, 128 kHalf 1.6%, kThird 4.0%, 1, 8, 128 kHalf 9.5% and of the
//              large layers 2.0%, 7.9%, 1.7%, parted at 4000 tiles 1.3% and 1.5%
//        4-bit 1, 4, 128 kThird 2.4%, 1, 8, 256 kWhole 8.8%, parted at 2048 tiles 2.1%; with more
//              than 16 tokens 1, 4, 128 kHalf 2.0%, kThird 4.0%, 1, 8, 256 kWhole 8.3% and of the
//              large layers 4.3%, 9.3%, 2.7%
// All of them add a sum's terms in the same order, so the choice, which depends on the
// number of tokens, leaves a token's bits as they are.
template <int WF>
hipError_t run_tiled_up(const MoeArgs& p, hipStream_t stream) {
  const int most = min(p.experts, p.m * p.top) * (p.f / 16);
  if constexpr (WF == EXPERT_BF16)
    return p.m > 44 && most >= 500 ? run_tile<WF, false, 2, 4, 128, kWhole>(p, stream)
                                   : run_tile<WF, false, 2, 2, 128, kHalf>(p, stream);
  else if constexpr (WF == EXPERT_INT8)
    return most <= 640 ? run_tile<WF, false, 2, 2, 128, kLess>(p, stream)
                       : run_tile<WF, false, 2, 4, 128, kHalf>(p, stream);
  else
    return most <= 1700 ? run_tile<WF, false, 2, 2, 128, kLess>(p, stream)
                        : run_tile<WF, false, 2, 8, 256, kWhole>(p, stream);
}

template <int WF>
hipError_t run_tiled_down(const MoeArgs& p, hipStream_t stream) {
  const int most = min(p.experts, p.m * p.top) * (p.k / 16);
  if constexpr (WF == EXPERT_BF16)
    return most <= 1000   ? run_tile<WF, true, 1, 2, 128, kHalf>(p, stream)
           : most <= 2000 ? run_tile<WF, true, 1, 4, 128, kHalf>(p, stream)
           : p.m <= 16    ? run_tile<WF, true, 1, 4, 256, kWhole>(p, stream)
                          : run_tile<WF, true, 2, 4, 128, kWhole>(p, stream);
  else if constexpr (WF == EXPERT_INT8)
    return most >= (p.m > 16 ? 4000 : 2048) ? run_tile<WF, true, 1, 8, 128, kHalf>(p, stream)
           : p.m > 16                       ? run_tile<WF, true, 1, 4, 128, kHalf>(p, stream)
                                            : run_tile<WF, true, 1, 4, 128, kThird>(p, stream);
  else
    return most >= 2048 ? run_tile<WF, true, 1, 8, 256, kWhole>(p, stream)
           : p.m > 16   ? run_tile<WF, true, 1, 4, 128, kHalf>(p, stream)
                        : run_tile<WF, true, 1, 4, 128, kThird>(p, stream);
}

// The streamed forms, by wavefronts, each with what it measured (us a layer in a graph;
// E8: 2 of 8 experts, k = 4096, f = 14336, E64: 8 of 64, k = 2048, f = 1408); three and four
// units in LDS are slower than two (one token, E64 8-bit 19.8, 21.8, 22.2):
//   up: up to two tokens four, where each has four units of k or more, else two (E8
//     4-bit 42.7, two 45.6; E64 8-bit, 6 of 64, 20.6, two 20.3); up to eight three, and two for
//     4-bit (8 tokens E8 bf16 326, two 331; 4-bit 131, two 125)
//   down: twelve up to two tokens (E64 19.9, four 20.7), eight up to eight (8 tokens E8
//     4-bit 125, four 130).
template <int WF>
hipError_t run_layer(const MoeArgs& p, bool few, hipStream_t stream) {
  if (!few) {
    hipError_t e = run_tiled_up<WF>(p, stream);
    if (e == hipSuccess) e = run_tiled_down<WF>(p, stream);
    if (e != hipSuccess) return e;
    moe_combine_kernel<<<dim3((unsigned)((p.k / 4 + 255) / 256), (unsigned)p.m), dim3(256), 0, stream>>>(p);
    return hipGetLastError();
  }
  const hipError_t e = p.m > 2 ? run_up<WF, 2, 8, WF == EXPERT_FP4 ? 2 : 3, 2>(p, stream)
                       : p.k >= 16 * stream_k(WF) ? run_up<WF, 2, 2, 4, 2>(p, stream)
                                                  : run_up<WF, 2, 2, 2, 2>(p, stream);
  if (e != hipSuccess) return e;
  return p.m <= 2 ? run_down<WF, 1, 2, 12, 2>(p, stream) : run_down<WF, 1, 8, 8, 2>(p, stream);
}

template <int TB, int EB>
void run_many(const RouteArgs& a, hipStream_t stream) {
  for (int64_t t = 0; t < a.m; t += 65535 * 16 * TB) {  // grid y
    RouteArgs p = a;
    p.x = a.x + t * a.k;
    p.logits = a.logits + t * a.experts;
    p.m = a.m - t;
    const int64_t groups = (p.m + 16 * TB - 1) / (16 * TB);
    const dim3 grid((unsigned)((a.experts + 16 * EB - 1) / (16 * EB)), (unsigned)(groups < 65535 ? groups : 65535));
    route_many_kernel<TB, EB><<<grid, dim3(64 * kRouteWaves), 0, stream>>>(p);
  }
}

}  // namespace

hipError_t launch_moe_route(const RouteArgs& a, hipStream_t stream) {
  const int64_t blocks = ((a.m + 15) / 16) * ((a.experts + 15) / 16);
  if (a.m * a.experts <= kOneLogits)
    route_few_kernel<true><<<dim3(a.experts, (unsigned)a.m), dim3(128), 2 * kRouteDepth * 2048, stream>>>(a);
  else if (a.m * a.experts <= kFewLogits)
    route_few_kernel<false><<<dim3((a.experts + 3) / 4, (unsigned)((a.m + 3) / 4)), dim3(64 * kRouteWaves),
                              kRouteWaves * kRouteDepth * 2048, stream>>>(a);
  else if (blocks < 1024) run_many<1, 1>(a, stream);
  else run_many<2, 2>(a, stream);
  auto* select = a.experts <= 64    ? route_select_kernel<1>
                 : a.experts <= 128 ? route_select_kernel<2>
                 : a.experts <= 256 ? route_select_kernel<4>
                                    : route_select_kernel<kMoeExperts / 64>;
  for (int64_t t = 0; t < a.m; t += kGridRows) {
    RouteArgs p = a;
    p.logits = a.logits + t * a.experts;
    p.ids = a.ids + t * a.top;
    p.weights = a.weights + t * a.top;
    p.m = a.m - t < kGridRows ? a.m - t : kGridRows;
    select<<<dim3((unsigned)((p.m + 3) / 4)), dim3(256), 0, stream>>>(p);
  }
  return hipGetLastError();
}

// Workspace: h of the tokens of one pass, bf16; the experts' parts of their results, binary32.
int64_t moe_workspace_bytes(int64_t m, int64_t k, int64_t f, int top) {
  const int64_t pairs = (m < kMoeTokens ? m : kMoeTokens) * top;
  return align256(pairs * f * 2) + (streamed(m, top) ? 0 : pairs * k * 4);
}

// kMoeTokens tokens at a time (a lane of a wavefront each).  The last of several
// passes takes the tiled kernels too, however short: a token's result is the same
// wherever in the call it stands.
hipError_t launch_moe_layer(const MoeArgs& args, int64_t m, hipStream_t stream) {
  MoeArgs p = args;
  const bool few = streamed(m, p.top);
  p.y = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(p.h) +
                                 align256((m < kMoeTokens ? m : kMoeTokens) * p.top * p.f * 2));
  for (int64_t t = 0; t < m; t += kMoeTokens) {
    p.m = (int)(m - t < kMoeTokens ? m - t : kMoeTokens);
    p.x = args.x + t * p.k;
    p.ids = args.ids + t * p.top;
    p.weights = args.weights + t * p.top;
    p.out = args.out + t * p.k;
    const hipError_t e = p.form == EXPERT_BF16   ? run_layer<EXPERT_BF16>(p, few, stream)
                         : p.form == EXPERT_INT8 ? run_layer<EXPERT_INT8>(p, few, stream)
                                                 : run_layer<EXPERT_FP4>(p, few, stream);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace sfr

// The linear layer in 8-bit integers with one scale per activation row and
// weight row: the row quantizer, and which kernels a call runs.
//
//     q = rne(127 x / amax),  scale = amax / 127         (a row at a time)
//     out[m, n] = xs[m] ws[n] sum_k xq[m, k] wq[n, k]  (+ bias[n])
//
// The sum is exact (32-bit integers on v_mfma_i32_16x16x64_i8; the entry points
// bound k), so no kernel, tile or slicing changes a result.
#include "sfr_dense.hpp"
#include "sfr_int8.hpp"

namespace sfr {
namespace {

// One wavefront (BLOCK false, four rows a workgroup) or one workgroup of NT
// threads per row.  A thread's first CPT chunks of eight values stay in
// registers between the sweeps for the maximum and for the codes; what a longer
// row has beyond them is read again (from the caches).
template <int CPT, int NT, bool BLOCK>
__global__ __launch_bounds__(NT) void quantize_int8_kernel(const uint16_t* __restrict__ x, int64_t rows, int cols,
                                                           int8_t* __restrict__ q, float* __restrict__ scale) {
  constexpr int T = BLOCK ? NT : 64;  // threads of a row
  const int tid = BLOCK ? threadIdx.x : threadIdx.x & 63;
  const int64_t row = BLOCK ? blockIdx.x : (int64_t)blockIdx.x * (NT / 64) + (threadIdx.x >> 6);
  if (row >= rows) return;
  const int chunks = cols >> 3;
  const uint4* const xr = reinterpret_cast<const uint4*>(x + row * cols);
  uint2* const qr = reinterpret_cast<uint2*>(q + row * cols);
  uint4 held[CPT];
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < CPT; ++i) {
    const int c = tid + T * i;
    held[i] = c < chunks ? xr[c] : make_uint4(0, 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < CPT; ++i) m = mag_max8(held[i], m);
  for (int c = tid + T * CPT; c < chunks; c += T) m = mag_max8(xr[c], m);
  m = wave_max(m);
  if constexpr (BLOCK) {
    __shared__ uint32_t red[NT / 64];
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = m;
    __syncthreads();
    m = red[0];
#pragma unroll
    for (int w = 1; w < NT / 64; ++w) m = max(m, red[w]);
  }
  const RowScale s = row_scale(m);
  if (tid == 0) scale[row] = scale_value(m);
#pragma unroll
  for (int i = 0; i < CPT; ++i) {
    const int c = tid + T * i;
    if (c < chunks) qr[c] = cast8_int8(held[i], s);
  }
  for (int c = tid + T * CPT; c < chunks; c += T) qr[c] = cast8_int8(xr[c], s);
}

// ---------------------------------------------------------------------------
// A few bf16 rows in one launch: every workgroup quantizes the activation for
// itself while its first weight units are in flight, keeps all of its codes in
// LDS, and streams weight rows against them, 16 at a time: wavefronts take units
// of 256 k in buffers of their own, D - 1 ahead and on into the next 16 rows, and
// add their sums at the end of each.  The activation is read by every workgroup,
// so this is for so few values that a launch costs more (fused()), and there are
// no more workgroups than the CUs hold.  Against the quantizer and the product in
// two launches, in a graph, us: one row, n = k = 4096 6.8, 7.9; n = 14336 12.7, 15.2; n =
// 28672 24.0, 28.6; 4 rows, n = 14336 13.7, 15.3; 2 rows, n = 14336, k = 8192 24.4, 29.6 (D =
// 2: 6.8, 13.2, 24.8, 14.3, 24.7); an eager call also saves the second launch's 3 us.
// ---------------------------------------------------------------------------
// chunks: of 8 values, per thread
constexpr int kFusedWaves = 8, kFusedDepth = 3, kFusedThreads = 64 * kFusedWaves, kFusedChunks = 4;

// Bytes between the rows' codes in LDS: whole units, and 16 so that rows lie in different banks.
constexpr int kFusedUnit = 256;
__host__ __device__ constexpr int codes_stride(int k) { return (k + kFusedUnit - 1) / kFusedUnit * kFusedUnit + 16; }

__global__ __launch_bounds__(kFusedThreads) void int8_fused_kernel(Int8Args p) {
  constexpr int NW = kFusedWaves, T = kFusedThreads, D = kFusedDepth, TILE = 16 * kFusedUnit, LOADS = TILE / 1024, R = kFusedChunks;
  extern __shared__ __attribute__((aligned(1024))) uint8_t smem[];
  __shared__ uint32_t maxes[NW][kFusedChunks];
  __shared__ int red[2][NW][R][16];  // of this tile and the one before
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r16 = lane & 15, lg = lane >> 4;
  const int K = (int)p.k, m = (int)p.m, chunks = K / 8, J = (chunks + T - 1) / T;  // J: chunks of a thread and row
  const int tiles = (int)(p.n / 16), units = (K + kFusedUnit - 1) / kFusedUnit;

  uint4 held[kFusedChunks];  // q: chunk threadIdx.x + T (q % J) of row q / J
#pragma unroll
  for (int q = 0; q < kFusedChunks; ++q) {
    const int r = q / J, c = threadIdx.x + T * (q - r * J);
    held[q] = r < m && c < chunks ? reinterpret_cast<const uint4*>(p.x + (int64_t)r * K)[c] : make_uint4(0, 0, 0, 0);
  }

  uint8_t* const mine = smem + wave * (D * TILE);
  int tile_in = blockIdx.x, unit_in = wave;  // what is put in flight next
  auto issue = [&](int at) __attribute__((always_inline)) {
    const int left = tile_in < tiles ? K - unit_in * kFusedUnit : 0;  // not positive: every lane masked
    const __amdgpu_buffer_rsrc_t rw = buf_rsrc(p.wq + (int64_t)min(tile_in, tiles - 1) * 16 * K, kPastRange);
#pragma unroll
    for (int j = 0; j < LOADS; ++j) {
      const int row = j * 4 + (lane >> 4), c = (lane & 15) ^ (row & 7);
      buf_to_lds(rw, mine + at * TILE + j * 1024, c * 16 < left ? row * K + unit_in * kFusedUnit + c * 16 : kPastRange);
    }
    unit_in += NW;
    if (unit_in >= units) {
      unit_in = wave;
      tile_in += gridDim.x;
    }
  };
#pragma unroll
  for (int i = 0; i < D - 1; ++i) issue(i);

  uint8_t* const codes = smem + NW * D * TILE;
  const int stride = codes_stride(K);
#pragma unroll
  for (int q = 0; q < kFusedChunks; ++q) {
    const uint32_t a = wave_max(mag_max8(held[q], 0));
    if (lane == 0) maxes[wave][q] = a;
  }
  wait_lds();
  wg_barrier();
  auto row_max = [&](int r) {
    uint32_t a = 0;
    for (int q = r * J; q < (r + 1) * J; ++q)
#pragma unroll
      for (int w = 0; w < NW; ++w) a = max(a, maxes[w][q]);
    return a;
  };
#pragma unroll
  for (int q = 0; q < kFusedChunks; ++q) {
    const int r = q / J, c = threadIdx.x + T * (q - r * J);
    if (r < m && c < chunks)
      *reinterpret_cast<uint2*>(codes + r * stride + 8 * c) = cast8_int8(held[q], row_scale(row_max(r)));
  }
  wait_lds();
  wg_barrier();

  const uint8_t* const xb = codes + min(r16, m - 1) * stride + 16 * lg;
  const float xs = scale_value(row_max(min(threadIdx.x / 16, m - 1)));  // of the row that this thread stores
  int at = 0, parity = 0;
  for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x, parity ^= 1) {
    v4i acc = v4i{0, 0, 0, 0};
    for (int u = wave; u < units; u += NW) {
      wait_lds();  // the buffer to be refilled has been read
      issue(at == 0 ? D - 1 : at - 1);
      wait_vm<(D - 1) * LOADS>();
      asm volatile("" ::: "memory");
      // what lies past K in the codes is not defined, and meets zeros of the weight
      const uint8_t* wb = mine + at * TILE + r16 * kFusedUnit;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        acc = mfma16(*reinterpret_cast<const v8bf*>(wb + 16 * ((4 * j + lg) ^ (r16 & 7))),
                     *reinterpret_cast<const v8bf*>(xb + u * kFusedUnit + 64 * j), acc);
      at = at == D - 1 ? 0 : at + 1;
    }
    if (r16 < m) *reinterpret_cast<v4i*>(&red[parity][wave][r16][4 * lg]) = acc;
    wait_lds();
    wg_barrier();  // and every wavefront has read what the tile before left here
    const int n = threadIdx.x % 16, r = threadIdx.x / 16;
    if (r < m) {
      const int64_t col = (int64_t)tile * 16 + n;
      int sum = 0;
#pragma unroll
      for (int v = 0; v < NW; ++v) sum += red[parity][v][r][n];
      const float y = int8_value(sum, xs, p.ws[col], p.bias ? bf16_to_f32(p.bias[col]) : -0.f);
      const int64_t to = r * p.n + col;
      if (p.out_fmt == OUT_F32) static_cast<float*>(p.out)[to] = y;
      else static_cast<uint16_t*>(p.out)[to] = (uint16_t)pack_bf16x2(y, 0.f);
    }
  }
  wait_vm<0>();  // the loads past the last unit (zeros) end before the workgroup's LDS does
}

// Whether a bf16 x of m rows is quantized in the product's own launch.
bool fused(int64_t m, int64_t k) { return m * ((k / 8 + kFusedThreads - 1) / kFusedThreads) <= kFusedChunks; }

// Bytes of LDS of m rows of k, and the most of any call that fused() admits: the
// kernel's limit is shared by all host threads, so every call sets it to the same.
constexpr int fused_bytes(int m, int k) { return kFusedWaves * kFusedDepth * 16 * kFusedUnit + m * codes_stride(k); }
constexpr int most_fused_bytes() {
  int most = 0;
  for (int m = 1; m <= kFusedChunks; ++m) {
    const int bytes = fused_bytes(m, kFusedChunks / m * kFusedThreads * 8);
    if (bytes > most) most = bytes;
  }
  return most;
}

hipError_t launch_fused(const Int8Args& a, hipStream_t stream) {
  constexpr int limit = most_fused_bytes();
  static_assert(limit + 5 * 1024 <= 160 * 1024, "LDS of a CU");
  const int bytes = fused_bytes((int)a.m, (int)a.k);
  const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void*>(int8_fused_kernel),
                                           hipFuncAttributeMaxDynamicSharedMemorySize, limit);
  if (e != hipSuccess) return e;
  // as many workgroups as the CUs hold, each the same number of tiles, or one fewer
  const int tiles = (int)(a.n / 16), most = 256 * (160 * 1024 / (bytes + 5 * 1024)), each = (tiles + most - 1) / most;
  int8_fused_kernel<<<dim3((unsigned)((tiles + each - 1) / each)), dim3(kFusedThreads), bytes, stream>>>(a);
  return hipGetLastError();
}

int64_t align256(int64_t b) { return (b + 255) / 256 * 256; }

StreamArgs stream_args(const Int8Args& a) {
  StreamArgs s{};
  s.x = reinterpret_cast<const uint16_t*>(a.xq);
  s.w = a.wq;
  s.m = a.m;
  s.k = a.k;
  s.rows = a.n;
  s.bias = a.bias;
  s.out = a.out;
  s.out_fmt = a.out_fmt;
  s.xs = a.xs;
  s.ws = a.ws;
  return s;
}

}  // namespace

hipError_t launch_quantize_int8(const uint16_t* x, int64_t rows, int64_t cols, int8_t* q, float* scale,
                                hipStream_t stream) {
  const int c = (int)cols;
  if (rows < 1024) {
    const dim3 grid((unsigned)rows);
    if (cols <= 2048) quantize_int8_kernel<1, 256, true><<<grid, dim3(256), 0, stream>>>(x, rows, c, q, scale);
    else if (cols <= 8192) quantize_int8_kernel<2, 512, true><<<grid, dim3(512), 0, stream>>>(x, rows, c, q, scale);
    else quantize_int8_kernel<2, 1024, true><<<grid, dim3(1024), 0, stream>>>(x, rows, c, q, scale);
    return hipGetLastError();
  }
  auto* kernel = cols <= 2048   ? quantize_int8_kernel<4, 256, false>
                 : cols <= 4096 ? quantize_int8_kernel<8, 256, false>
                                : quantize_int8_kernel<16, 256, false>;
  for (int64_t r = 0; r < rows; r += kGridRows) {
    const int64_t n = rows - r < kGridRows ? rows - r : kGridRows;
    kernel<<<dim3((unsigned)((n + 3) / 4)), dim3(256), 0, stream>>>(x + r * cols, n, c, q + r * cols, scale + r);
  }
  return hipGetLastError();
}

// Workspace: the partial sums of a sliced product; of a bf16 x its codes and scales.
int64_t int8_workspace_bytes(int64_t m, int64_t n, int64_t k, bool dynamic) {
  if (dynamic && fused(m, k)) return 0;
  return (stream_rows_int8(m, n, k) ? 0 : align256(dense_int8_workspace_bytes(m, n, k))) +
         (dynamic ? align256(m * k) + align256(4 * m) : 0);
}

hipError_t launch_int8(const Int8Args& args, void* workspace, hipStream_t stream) {
  if (args.x && fused(args.m, args.k)) return launch_fused(args, stream);
  Int8Args a = args;
  uint8_t* at = static_cast<uint8_t*>(workspace);
  if (a.x) {
    int8_t* const q = reinterpret_cast<int8_t*>(at);
    float* const scale = reinterpret_cast<float*>(at + align256(a.m * a.k));
    at += align256(a.m * a.k) + align256(4 * a.m);
    const hipError_t e = launch_quantize_int8(a.x, a.m, a.k, q, scale, stream);
    if (e != hipSuccess) return e;
    a.xq = q;
    a.xs = scale;
  }
  if (stream_rows_int8(a.m, a.n, a.k)) return launch_stream(stream_args(a), stream);
  return launch_int8_dense(a, at, stream);
}

DenseKernel int8_kernel(int64_t m, int64_t n, int64_t k, bool dynamic) {
  if (dynamic && fused(m, k)) return {"fused_int8", 1};
  if (!stream_rows_int8(m, n, k)) return dense_int8_kernel(m, n, k);
  static const float some = 0;  // ws: tells this product from the others, not read
  Int8Args a{};
  a.ws = &some;
  a.m = m;
  a.n = n;
  a.k = k;
  return {stream_name(stream_args(a)), 1};
}

}  // namespace sfr

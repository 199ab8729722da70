// int8_matmul.hip -- the product of 8-bit integers with a scale for each token
// and each channel, on gfx950:
//   y[m][n] = sx[m] sw[n] sum_k x[m][k] w[n][k] + bias[n]
// The sums are exact (32-bit integers; K <= 65536 values of at most 2^7 each);
// what is rounded is the sum's conversion to fp32, the products with the
// scales and the output.
//
// The weights are the matrix instruction's first operand and the tokens its
// second, so that a lane ends with four consecutive channels of one token.
#include <algorithm>

#include "norm_device.h"

namespace gdr {

namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));

struct MatArgs {
  const int8_t* x;
  const int8_t* w;
  const float* xs;
  const float* ws;
  const void* bias;   // nullable
  void* y;
  int64_t x_stride;   // bytes between tokens
  int M, N, K;
  int bias_dtype;
  int tiles_m, tiles_n;
};

// 16 bytes at any address
__device__ __forceinline__ i32x4 load16(const int8_t* p) {
  struct __attribute__((packed, aligned(1))) Raw {
    int u[4];
  };
  const Raw r = *reinterpret_cast<const Raw*>(p);
  return i32x4{r.u[0], r.u[1], r.u[2], r.u[3]};
}
// Bytes [k, k + 16) of a row of K; those past its end are zero, and none past
// it is read.
__device__ __forceinline__ i32x4 load16_of_row(const int8_t* row, int k, int K) {
  if (k + 16 <= K) return load16(row + k);
  unsigned __int128 v = 0;
  if (K >= 16) {  // the row's last 16 bytes, moved down
    const int down = k - (K - 16);
    if (down < 16) v = __builtin_bit_cast(unsigned __int128, load16(row + (K - 16))) >> (8 * down);
  } else {
    for (int e = K - 1; e >= k; --e) v = v << 8 | (uint8_t)row[e];
  }
  return __builtin_bit_cast(i32x4, v);
}

template <typename O>
__device__ __forceinline__ O scaled(int acc, float xs, float ws, float bias) {
  return from_f<O>(__builtin_fmaf((float)acc * ws, xs, bias));
}

// ---- few tokens ---------------------------------------------------------------
// A workgroup forms 16 NB channels of 16 MB tokens: its eight waves take an
// eighth of K each, read operands straight from memory to registers and add
// up their sums in LDS.
constexpr int kSplit = 8;
template <int NB, int MB, typename O>
__global__ __launch_bounds__(64 * kSplit) void int8_few_kernel(MatArgs a) {
  constexpr int BN = 16 * NB, BM = 16 * MB;
  __shared__ __align__(16) int part[kSplit][BM][BN + 4];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int r = lane & 15, kq = 16 * (lane >> 4);
  const int n0 = blockIdx.x * BN, m0 = blockIdx.y * BM;
  const int steps = (a.K + 63) / 64, per = (steps + kSplit - 1) / kSplit;
  const int k_begin = 64 * min(steps, wave * per), k_end = 64 * min(steps, (wave + 1) * per);
  const int8_t* wrow[NB];
  const int8_t* xrow[MB];
  // (rows past the end read the last one again; their sums are not stored)
#pragma unroll
  for (int i = 0; i < NB; ++i) wrow[i] = a.w + (int64_t)min(n0 + 16 * i + r, a.N - 1) * a.K;
#pragma unroll
  for (int j = 0; j < MB; ++j) xrow[j] = a.x + (int64_t)min(m0 + 16 * j + r, a.M - 1) * a.x_stride;
  i32x4 acc[NB][MB];
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int j = 0; j < MB; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
  const int whole = min(k_end, a.K / 64 * 64);
  int k = k_begin;
  for (; k < whole; k += 64) {
    i32x4 fw[NB], fx[MB];
#pragma unroll
    for (int i = 0; i < NB; ++i) fw[i] = load16(wrow[i] + k + kq);
#pragma unroll
    for (int j = 0; j < MB; ++j) fx[j] = load16(xrow[j] + k + kq);
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int j = 0; j < MB; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[i], fx[j], acc[i][j], 0, 0, 0);
  }
  if (k < k_end) {  // the row's end
    i32x4 fw[NB], fx[MB];
#pragma unroll
    for (int i = 0; i < NB; ++i) fw[i] = load16_of_row(wrow[i], k + kq, a.K);
#pragma unroll
    for (int j = 0; j < MB; ++j) fx[j] = load16_of_row(xrow[j], k + kq, a.K);
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int j = 0; j < MB; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[i], fx[j], acc[i][j], 0, 0, 0);
  }
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int j = 0; j < MB; ++j)
      *reinterpret_cast<i32x4*>(&part[wave][16 * j + r][16 * i + 4 * (lane >> 4)]) = acc[i][j];
  __syncthreads();
  for (int t = threadIdx.x; t < BM * BN; t += 64 * kSplit) {
    const int n = t % BN, m = t / BN;
    if (m0 + m >= a.M || n0 + n >= a.N) continue;
    int s = 0;
#pragma unroll
    for (int q = 0; q < kSplit; ++q) s += part[q][m][n];
    const float b = a.bias ? load_scalar(a.bias, n0 + n, a.bias_dtype) : 0.f;
    reinterpret_cast<O*>(a.y)[(int64_t)(m0 + m) * a.N + n0 + n] =
        scaled<O>(s, a.xs[m0 + m], a.ws[n0 + n], b);
  }
}

// ---- many tokens --------------------------------------------------------------
// A workgroup of WN x WM waves forms 32 NB WN channels of 32 MB WM tokens in
// steps of 128 bytes of K.  Tiles lie in LDS as rows of 128 bytes, the 16-byte
// piece j of row r at j ^ ((r / 2) % 8): 16 rows read at one column hit
// different banks.  While a step's products run, the next one's tiles arrive
// in the other buffer and the operands of the next quarter step in registers;
// there is one barrier a step, before its last quarter.
//
// DMA: rows of 16-byte pieces (K, strides and addresses multiples of 16) go
// straight to LDS, by raw buffer loads that return zero past the range;
// otherwise pieces pass through registers.
template <int WN, int WM, int NB, int MB, bool DMA, typename O>
__global__ __launch_bounds__(64 * WN * WM) void int8_tile_kernel(MatArgs a) {
  constexpr int NW = WN * WM, NT = 64 * NW;
  constexpr int BN = 32 * NB * WN, BM = 32 * MB * WM;
  constexpr int ROWS = BN + BM;              // of a buffer: the weights' rows, then the tokens'
  constexpr int PER = ROWS / 8 / NW;         // 1 KiB pieces of a wave
  static_assert(BN % (8 * PER) == 0, "a wave loads rows of one operand");
  static_assert(WM * 32 * BN * (int)sizeof(O) <= ROWS * 128, "the epilogue's rows fit a buffer");
  // two objects, so that a read of one does not wait for the other's loads
  __shared__ __align__(1024) uint8_t buf0[ROWS * 128];
  __shared__ __align__(1024) uint8_t buf1[ROWS * 128];
  __shared__ float col[2][BN];               // the channels' scales and biases
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)(threadIdx.x >> 6));
  const int wn = wave % WN, wm = wave / WN;

  // Workgroups go to the 8 XCDs in turn: each XCD takes consecutive tiles, and
  // eight rows of tiles are walked together, so that the tiles in flight in an
  // XCD share operands in its L2.
  const int total = a.tiles_m * a.tiles_n;
  int tile;
  {
    const int id = blockIdx.x, xcd = id % 8, per = total / 8, more = total % 8;
    tile = xcd * per + min(xcd, more) + id / 8;
  }
  const int band = 8 * a.tiles_n, b0 = tile / band * 8;
  const int high = min(8, a.tiles_m - b0);
  const int m0 = (b0 + tile % band % high) * BM, n0 = tile % band / high * BN;

  // this wave's rows of the buffers
  const int row0 = wave * 8 * PER;
  const bool is_w = row0 < BN;
  const int64_t stride = is_w ? (int64_t)a.K : a.x_stride;
  const int first = is_w ? n0 : m0, rows = min(is_w ? BN : BM, (is_w ? a.N : a.M) - first);
  const int in_tile = is_w ? row0 : row0 - BN;
  const int8_t* src = (is_w ? a.w : a.x) + (int64_t)first * stride;
  const int lrow = lane >> 3, lpos = lane & 7;
  const int piece[2] = {lpos ^ (lane >> 4), lpos ^ (4 + (lane >> 4))};
  const __amdgpu_buffer_rsrc_t rs = buf_rsrc(src, (int64_t)(rows - 1) * stride + a.K);
  i32x4 staged[DMA ? 1 : PER];

  auto request = [&](uint8_t* buf, int k0) {
#pragma unroll
    for (int t = 0; t < PER; ++t) {
      const int r = in_tile + 8 * t + lrow, k = k0 + 16 * piece[t & 1];
      if (DMA) {
        // past the row's end: an offset past the range, which reads as zero
        const int off = k < a.K ? r * (int)stride + k : 0x7ffffff0;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            rs, (__attribute__((address_space(3))) void*)(buf + (row0 + 8 * t) * 128), 16, off, 0,
            0, 0);
      } else {
        staged[DMA ? 0 : t] = load16_of_row(src + min(r, rows - 1) * stride, k, a.K);
      }
    }
  };
  auto deliver = [&](uint8_t* buf) {
    if (!DMA) {
#pragma unroll
      for (int t = 0; t < PER; ++t)
        *reinterpret_cast<i32x4*>(buf + (row0 + 8 * t) * 128 + 16 * lane) = staged[DMA ? 0 : t];
    }
  };

  // a barrier does not wait for a wave's loads to LDS: the wave does
  auto arrive = [&]() {
    if (DMA) __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
    __syncthreads();
  };

  i32x16 acc[NB][MB];
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int j = 0; j < MB; ++j)
#pragma unroll
      for (int e = 0; e < 16; ++e) acc[i][j][e] = 0;
  i32x4 fw[2][NB], fx[2][MB];
  const int lr = lane & 31, lh = lane >> 5, sw = (lr >> 1) & 7;
  const int w_at = (wn * NB * 32 + lr) * 128, x_at = (BN + wm * MB * 32 + lr) * 128;
  auto operands = [&](const uint8_t* buf, int q, int set) {
    const int p = 16 * ((2 * q + lh) ^ sw);
#pragma unroll
    for (int i = 0; i < NB; ++i)
      fw[set][i] = *reinterpret_cast<const i32x4*>(buf + w_at + 32 * 128 * i + p);
#pragma unroll
    for (int j = 0; j < MB; ++j)
      fx[set][j] = *reinterpret_cast<const i32x4*>(buf + x_at + 32 * 128 * j + p);
  };
  const int steps = (a.K + 127) / 128;
  auto step = [&](uint8_t* cur, uint8_t* next, int s) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (q < 3) {
        operands(cur, q + 1, (q + 1) & 1);
        if (!DMA && q == 0 && s + 1 < steps) request(next, (s + 1) * 128);
      } else if (s + 1 < steps) {
        deliver(next);
        arrive();  // the next step's tiles have arrived, this one's are read
        operands(next, 0, 0);
        if (DMA && s + 2 < steps) request(cur, (s + 2) * 128);
      }
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int j = 0; j < MB; ++j)
          acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fw[q & 1][i], fx[q & 1][j], acc[i][j],
                                                            0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  request(buf0, 0);
  deliver(buf0);
  arrive();
  operands(buf0, 0, 0);
  if (DMA && steps > 1) request(buf1, 128);
  for (int s = 0; s < steps; s += 2) {
    step(buf0, buf1, s);
    if (s + 1 < steps) step(buf1, buf0, s + 1);
  }

  // The outputs pass through LDS, 32 tokens of every wave at a time, so that a
  // row of the tile is stored in one piece; the 16-byte piece j of row r lies
  // at j ^ (r % 16).
  for (int t = threadIdx.x; t < BN; t += NT) {
    const int n = min(n0 + t, a.N - 1);
    col[0][t] = a.ws[n];
    col[1][t] = a.bias ? load_scalar(a.bias, n, a.bias_dtype) : 0.f;
  }
  __syncthreads();
  constexpr int V = 16 / (int)sizeof(O), PIECES = BN / V;
#pragma unroll
  for (int j = 0; j < MB; ++j) {
    uint8_t* buf = j & 1 ? buf1 : buf0;
    const int m = m0 + (wm * MB + j) * 32 + lr;
    const float xs = a.xs[min(m, a.M - 1)];
    uint8_t* out = buf + (wm * 32 + lr) * (BN * (int)sizeof(O));
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        const int c = (wn * NB + i) * 32 + 8 * g + 4 * lh;  // four channels of the tile
        O v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e)
          v[e] = scaled<O>(acc[i][j][4 * g + e], xs, col[0][c + e], col[1][c + e]);
        const int at = c * (int)sizeof(O);
        uint8_t* p = out + 16 * ((at >> 4) ^ (lr & 15)) + (at & 15);
        struct __attribute__((aligned(4 * sizeof(O)))) Four {
          O v[4];
        };
        *reinterpret_cast<Four*>(p) = Four{{v[0], v[1], v[2], v[3]}};
      }
    __syncthreads();
    for (int t = threadIdx.x; t < WM * 32 * PIECES; t += NT) {
      const int r = t / PIECES, p = t % PIECES;
      const int mm = m0 + ((r >> 5) * MB + j) * 32 + (r & 31), n = n0 + p * V;
      if (mm < a.M && n < a.N) {
        const Vec<O> v = *reinterpret_cast<const Vec<O>*>(buf + r * (BN * (int)sizeof(O)) +
                                                          16 * (p ^ (r & 15)));
        v.store_part(reinterpret_cast<O*>(a.y) + (int64_t)mm * a.N + n, a.N - n);
      }
    }
  }
}

template <typename F>
void by_out(const gdr_int8_matmul_problem* p, F f) {
  if (p->out_dtype == GDR_BF16) f(__bf16());
  else if (p->out_dtype == GDR_FP16) f(_Float16());
  else f(float());
}

}  // namespace

gdr_status launch_int8_matmul(const gdr_int8_matmul_problem* p, const void* x, const float* x_scale,
                              const void* w, const float* w_scale, const void* bias, void* y,
                              hipStream_t st) {
  MatArgs a{};
  a.x = reinterpret_cast<const int8_t*>(x);
  a.w = reinterpret_cast<const int8_t*>(w);
  a.xs = x_scale; a.ws = w_scale; a.bias = bias; a.y = y;
  a.x_stride = p->x_stride;
  a.M = p->M; a.N = p->N; a.K = p->K;
  a.bias_dtype = (int)p->bias_dtype;
  const bool aligned = p->K % 16 == 0 && p->x_stride % 16 == 0 && (uintptr_t)x % 16 == 0 &&
                       (uintptr_t)w % 16 == 0;
  by_out(p, [&](auto o) {
    using O = decltype(o);
    auto few = [&](auto nb, auto mb) {
      constexpr int NB = nb.value, MB = mb.value;
      const dim3 grid((p->N + 16 * NB - 1) / (16 * NB), (p->M + 16 * MB - 1) / (16 * MB));
      GDR_LAUNCH("int8_few", (int8_few_kernel<NB, MB, O>), grid, dim3(64 * kSplit), st, a);
    };
    auto tiles = [&](auto wn, auto wm, auto nb, auto mb) {
      constexpr int WN = wn.value, WM = wm.value, NB = nb.value, MB = mb.value;
      a.tiles_n = (p->N + 32 * NB * WN - 1) / (32 * NB * WN);
      a.tiles_m = (p->M + 32 * MB * WM - 1) / (32 * MB * WM);
      const dim3 grid((unsigned)((int64_t)a.tiles_m * a.tiles_n)), block(64 * WN * WM);
      if (aligned)
        GDR_LAUNCH("int8_tile", (int8_tile_kernel<WN, WM, NB, MB, true, O>), grid, block, st, a);
      else
        GDR_LAUNCH("int8_tile", (int8_tile_kernel<WN, WM, NB, MB, false, O>), grid, block, st, a);
    };
    const std::integral_constant<int, 1> c1;
    const std::integral_constant<int, 2> c2;
    const std::integral_constant<int, 4> c4;
    if (p->M <= 16) few(c1, c1);
    else if (p->M <= 32) few(c1, c2);
    else if (p->M <= 64 || (int64_t)p->M * p->N <= 128 * 128 * 128) few(c2, c4);
    else if ((int64_t)p->M * p->N < 256 * 256 * 256) tiles(c2, c2, c2, c2);
    else tiles(c4, c2, c2, c4);
  });
  return launch_status("int8_matmul");
}

}  // namespace gdr

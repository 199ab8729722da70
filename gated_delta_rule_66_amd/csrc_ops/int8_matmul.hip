// int8_matmul.hip -- the product of 8-bit integers with a scale for each token
// and each channel, on gfx950:
//   y[m][n] = sx[m] sw[n] sum_k x[m][k] w[n][k] + bias[n]
// The sums are exact (32-bit integers; K <= 65536 values of at most 2^7 each);
// what is rounded is the sum's conversion to fp32, the products with the
// scales and the output.
//
// 18,062 tokens by 12,288 channels of K = 4096 take 845 to 890 us (2.1 to 2.15
// POPS with random values; a library's product with 32-bit sums as its output
// 810 to 870), 2903 x 5003 of K = 2505 59, 48 of them the product; with the weights
// in the caches 64 x 12,288 11, 1 x 12,288 10 (5 TB/s), from memory 8 x 12,288 14.
//
// The weights are the matrix instruction's first operand and the tokens its
// second, so that a lane ends with four consecutive channels of one token.
#include <algorithm>
#include <cmath>

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
  int64_t w_stride;   // bytes between channels
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
// The same from two aligned reads: a read at an odd address takes several times
// as long.  (Bytes before p or past p + 16 share a word with the first or the
// last byte that is asked for.)
__device__ __forceinline__ i32x4 load16_shifted(const int8_t* p) {
  struct __attribute__((aligned(4))) Raw {
    int u[4];
  };
  const int shift = (int)((uintptr_t)p & 3);
  const int8_t* q = p - shift;
  const Raw r = *reinterpret_cast<const Raw*>(q);
  const int end = *reinterpret_cast<const int*>(q + (shift ? 16 : 12));
  return i32x4{(int)__builtin_amdgcn_alignbyte(r.u[1], r.u[0], shift),
               (int)__builtin_amdgcn_alignbyte(r.u[2], r.u[1], shift),
               (int)__builtin_amdgcn_alignbyte(r.u[3], r.u[2], shift),
               (int)__builtin_amdgcn_alignbyte(end, r.u[3], shift)};
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
// ODD: some row begins inside a word.
template <int NB, int MB, bool ODD, typename O>
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
  for (int i = 0; i < NB; ++i) wrow[i] = a.w + (int64_t)min(n0 + 16 * i + r, a.N - 1) * a.w_stride;
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
    for (int i = 0; i < NB; ++i) fw[i] = ODD ? load16_shifted(wrow[i] + k + kq) : load16(wrow[i] + k + kq);
#pragma unroll
    for (int j = 0; j < MB; ++j) fx[j] = ODD ? load16_shifted(xrow[j] + k + kq) : load16(xrow[j] + k + kq);
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

// A raw buffer resource of `bytes` bytes (below 2^31) in scalar registers.
__device__ __forceinline__ u32x4 tile_rsrc(const void* base, int64_t bytes) {
  const uint64_t b = (uint64_t)base;
  return u32x4{(unsigned)__builtin_amdgcn_readfirstlane((int)(uint32_t)b),
               (unsigned)__builtin_amdgcn_readfirstlane((int)((b >> 32) & 0xffff)),
               (unsigned)__builtin_amdgcn_readfirstlane((int)bytes), 0x00020000u};
}
__device__ __forceinline__ int lds_address(const void* p) {
  return __builtin_amdgcn_readfirstlane(
      (int)(uintptr_t)(const __attribute__((address_space(3))) void*)p);
}
// 16 bytes a lane from byte `off` of the range to 1 KiB of LDS at byte `at`, lane by lane;
// past the range's end zeros.  Written in assembly because the compiler, which
// cannot tell the buffers apart, waits for the builtin's loads before the next
// read of LDS.  There is no register to wait for: the wave waits on its vector
// memory counter before the barrier that hands the tile over.  (m0, which holds
// the address in LDS, is a register that the compiler reserves, and warns of in a
// list of clobbered ones; nothing else here reads or writes it.)
__device__ __forceinline__ void load_to_lds(u32x4 rs, int at, int off) {
  asm volatile(
      "s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(at),
      "v"(off), "s"(rs)
      : "memory");
}

// ---- many tokens --------------------------------------------------------------
// A workgroup of WN x WM waves forms 32 NB WN channels of 32 MB WM tokens in
// steps of KB bytes of K.  A step's tiles lie in LDS as rows of KB bytes, the
// 16-byte piece j of row r at j ^ swizzle(r), so that 16 rows read at one column
// hit different banks; rows and pieces past the operand's end are zero.
// Loads go straight to LDS, up to STEPS - 1 steps ahead of the products; the
// operands of the next 32 bytes arrive in registers while these ones' products
// run.  One barrier a step, before its last products: by then every wave has
// read this step's tiles, whose place the request for STEPS steps on takes, and
// waited for its own loads of the next one's.
//
// What bounds 256 x 256 tiles is power: 18,062 x 12,288 x 4096 take 850 us with
// random values and 678 with zeros, at matrix units busy for half of the cycles
// of a clock that falls to 1.6 GHz.  Left out in copies, the loads to LDS cost 130
// us of the 850, the reads of operands 50; products alone take 670.  The loads
// alone take 621 (22 bytes a cycle and CU, whatever the order of a row's pieces).
// Steps of 64 bytes, four in flight: 913 us.  Small problems wait for loads:
// there tiles of 64 x 64 keep four steps in flight (512 x 4096 x 4096 15 us; two
// steps 17, 128 x 128 tiles 23).
constexpr int KB = 128;
__device__ __forceinline__ int swizzle(int r) { return (r >> 1) & 7; }
template <int WN, int WM, int NB, int MB, int STEPS, typename O>
__global__ __launch_bounds__(64 * WN * WM) void int8_tile_kernel(MatArgs a) {
  constexpr int NW = WN * WM, NT = 64 * NW;
  constexpr int BN = 32 * NB * WN, BM = 32 * MB * WM;
  constexpr int ROWS = BN + BM;              // of a step: the weights' rows, then the tokens'
  constexpr int RPL = 1024 / KB;             // rows of a wave's load
  constexpr int PER = ROWS / RPL / NW;       // loads of a wave
  constexpr int STEP = ROWS * KB;            // bytes
  constexpr int Q = KB / 32;                 // parts of a step
  static_assert(BN % (RPL * PER) == 0, "a wave loads rows of one operand");
  static_assert(2 * WM * 32 * BN * (int)sizeof(O) <= STEPS * STEP, "two of the epilogue's parts fit");
  __shared__ __align__(1024) uint8_t buf[STEPS * STEP];
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

  // this wave's rows of a step
  const int row0 = wave * RPL * PER;
  const bool is_w = row0 < BN;
  const int64_t stride = is_w ? a.w_stride : a.x_stride;
  const int first = is_w ? n0 : m0, rows = min(is_w ? BN : BM, (is_w ? a.N : a.M) - first);
  const int8_t* src = (is_w ? a.w : a.x) + (int64_t)first * stride;
  const int lrow = lane / (KB / 16), lpos = lane % (KB / 16);
  const int piece[2] = {16 * (lpos ^ swizzle(lrow)), 16 * (lpos ^ swizzle(RPL + lrow))};
  u32x4 rs = tile_rsrc(src, (int64_t)(rows - 1) * stride + a.K);
  const int to = lds_address(buf) + row0 * KB;
  int from[PER];
#pragma unroll
  for (int t = 0; t < PER; ++t)
    from[t] = ((is_w ? row0 : row0 - BN) + RPL * t + lrow) * (int)stride + piece[t & 1];
  int k_next = 0;  // of the step that is requested next; rs begins there
  int slot_next = 0;

  auto request_one = [&](int t) {
    // past the row's end: an offset past the range, which reads as zero
    load_to_lds(rs, to + slot_next * STEP + 1024 * t,
                k_next + piece[t & 1] < a.K ? from[t] : 0x7ffffff0);
  };
  auto advance = [&]() {
    k_next += KB;
    slot_next = slot_next + 1 == STEPS ? 0 : slot_next + 1;
    const uint64_t base = ((uint64_t)rs[1] << 32 | rs[0]) + KB;
    rs[0] = (unsigned)base;
    rs[1] = (unsigned)(base >> 32);
    rs[2] -= KB;  // (used while some of a row is left)
  };
  // Waits until the wave's loads are done but for those of `ahead` steps, then
  // for the other waves (whose barrier does not wait for loads to LDS).
  auto arrive = [&](int ahead) {
    static_assert(STEPS == 2 || STEPS == 4, "steps ahead");
    if (STEPS == 4 && ahead == 2) __builtin_amdgcn_s_waitcnt(vmcnt_imm(2 * PER));
    else if (STEPS == 4 && ahead == 1) __builtin_amdgcn_s_waitcnt(vmcnt_imm(PER));
    else __builtin_amdgcn_s_waitcnt(vmcnt_imm(0));
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
  const int lr = lane & 31, lh = lane >> 5, sw = swizzle(lr);
  const int w_at = (wn * NB * 32 + lr) * KB, x_at = (BN + wm * MB * 32 + lr) * KB;
  auto operands = [&](int at, int q) {
    const uint8_t* p = buf + at + 16 * ((2 * q + lh) ^ sw);
#pragma unroll
    for (int i = 0; i < NB; ++i)
      fw[q & 1][i] = *reinterpret_cast<const i32x4*>(p + w_at + 32 * KB * i);
#pragma unroll
    for (int j = 0; j < MB; ++j)
      fx[q & 1][j] = *reinterpret_cast<const i32x4*>(p + x_at + 32 * KB * j);
  };
  auto product = [&](int q, int i, int j) {
    acc[i][j] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fw[q][i], fx[q][j], acc[i][j], 0, 0, 0);
  };
  // all parts of a step but the last, whose operands are left in registers
  auto parts = [&](int at) {
#pragma unroll
    for (int q = 0; q + 1 < Q; ++q) {
      operands(at, q + 1);
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_setprio(1);  // over the wave that reads operands
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int j = 0; j < MB; ++j) product(q & 1, i, j);
      __builtin_amdgcn_s_setprio(0);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  const int steps = (a.K + KB - 1) / KB;
  for (int s = 0; s < min(steps, STEPS); ++s) {
#pragma unroll
    for (int t = 0; t < PER; ++t) request_one(t);
    advance();
  }
  arrive(min(STEPS - 2, min(steps, STEPS) - 1));
  operands(0, 0);
  int at = 0;
  for (int s = 0; s + 1 < steps; ++s) {
    const int next = at + STEP == STEPS * STEP ? 0 : at + STEP;
    parts(at);
    // requested so far: steps up to s + STEPS - 1; s + 1 has to be there
    const int ahead = min(STEPS - 2, steps - 2 - s);
    arrive(ahead);
    operands(next, 0);
    __builtin_amdgcn_sched_barrier(0);
    const bool more = s + STEPS < steps;
#pragma unroll
    for (int i = 0; i < NB; ++i)
#pragma unroll
      for (int j = 0; j < MB; ++j) {
        product(1, i, j);
        __builtin_amdgcn_sched_barrier(0);
        if (more)
#pragma unroll
          for (int t = (i * MB + j) * PER / (NB * MB); t < (i * MB + j + 1) * PER / (NB * MB); ++t)
            request_one(t);
      }
    if (more) advance();
    at = next;
  }
  parts(at);
#pragma unroll
  for (int i = 0; i < NB; ++i)
#pragma unroll
    for (int j = 0; j < MB; ++j) product(1, i, j);

  // The outputs pass through LDS, 32 tokens of every wave at a time, so that a
  // row of the tile is stored in one piece; the 16-byte piece j of row r lies
  // at j ^ (r % 16), in rows of 8 pieces at j ^ (r / 2 % 8).
  for (int t = threadIdx.x; t < BN; t += NT) {
    const int n = min(n0 + t, a.N - 1);
    col[0][t] = a.ws[n];
    col[1][t] = a.bias ? load_scalar(a.bias, n, a.bias_dtype) : 0.f;
  }
  __syncthreads();
  constexpr int V = 16 / (int)sizeof(O), PIECES = BN / V;
  static_assert(PIECES % 16 == 0 || PIECES == 8, "pieces of a row");
  auto place = [](int r) { return PIECES == 8 ? (r >> 1) & 7 : r & 15; };
#pragma unroll
  for (int j = 0; j < MB; ++j) {
    uint8_t* rowsbuf = buf + (j & 1) * (WM * 32 * BN * (int)sizeof(O));
    const int m = m0 + (wm * MB + j) * 32 + lr;
    const float xs = a.xs[min(m, a.M - 1)];
    uint8_t* out = rowsbuf + (wm * 32 + lr) * (BN * (int)sizeof(O));
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
        uint8_t* p = out + 16 * ((at >> 4) ^ place(lr)) + (at & 15);
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
        const Vec<O> v = *reinterpret_cast<const Vec<O>*>(rowsbuf + r * (BN * (int)sizeof(O)) +
                                                          16 * (p ^ place(r)));
        v.store_part(reinterpret_cast<O*>(a.y) + (int64_t)mm * a.N + n, a.N - n);
      }
    }
  }
}

// Rows of K bytes at any address, copied to rows that begin at multiples of 128
// bytes (with ones at odd multiples of 16 the product takes 15 % longer) and end
// with zeros up to one of 16: up to two matrices, a wave a row.
struct PadArgs {
  const int8_t* src[2];
  int8_t* dst[2];
  int64_t stride[2];
  int rows[2];
  int K, padded, row;
};
__global__ __launch_bounds__(256) void int8_pad_kernel(PadArgs a) {
  int64_t r = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int which = r >= a.rows[0];
  if (which) r -= a.rows[0];
  if (which && r >= a.rows[1]) return;
  const int8_t* src = a.src[which] + r * a.stride[which];
  int8_t* dst = a.dst[which] + r * (int64_t)a.row;
  for (int k = 16 * (threadIdx.x & 63); k < a.padded; k += 1024)
    *reinterpret_cast<i32x4*>(dst + k) =
        k + 16 <= a.K ? load16_shifted(src + k) : load16_of_row(src, k, a.K);
}

// What a problem runs as, from its sizes.
struct MatPlan {
  enum { kFew16, kFew32, kFew64, kTile64, kTile128, kTile256 } kernel;
  bool pad_x, pad_w;  // tiles of rows whose pieces of 16 bytes are not aligned
  int row;            // bytes from one padded row to the next
};
// The kernel of the least estimated time, in us; bf16 outputs of random values.
// Tiles: the card holds `slots` workgroups; a round of them takes `full` per 128
// bytes of K, one of a workgroup a CU (half of them) or, with one of 256 x 256
// a CU, of half the CUs `half`.  Measured at K = 4096: 64 x 64 tiles 10.3 us
// for 192, 15.9 for 512; 128 x 128 20.6 for 64, 28 for 256, 41.5 for 512; 256 x
// 256 45 for 16, 73 for 256.  So 512 x 4096 outputs take 16, 23 and 48 us, 2048 x
// 4096 58, 42 and 52, 4096 x 4096 (80 in 128 x 128) 73.
// Few tokens: the weights' bytes (4.5 us for 1 x 4096 of K = 4096, 10 for 1 x
// 12288) and the tokens' from L2 for every 16 channels (5.9 and 14.1 for 16
// tokens, against 10.2 and 11.1 in 64 x 64 tiles).  All of these with operands that
// stay in the caches from call to call.
MatPlan plan_of(const gdr_int8_matmul_problem* p) {
  const double M = p->M, N = p->N, K = p->K, never = 1e30;
  auto tile_us = [&](double edge, double slots, double full, double half) {
    const double tiles = std::ceil(M / edge) * std::ceil(N / edge);
    const double rounds = std::floor(tiles / slots), rest = tiles - rounds * slots;
    const double last = rest == 0 ? 0 : rest <= slots / 2 ? half : full;
    return 1 + std::ceil(K / 128) * (rounds * full + last);
  };
  MatPlan q{};
  q.row = (p->K + 127) / 128 * 128;
  q.pad_w = p->K % 16 != 0;
  q.pad_x = q.pad_w || p->x_stride % 16 != 0;
  const double pad = q.pad_x ? 3 + (q.pad_w ? N + M : M) * K / 2.8e6 : 0;
  // what a launch holds: 2^32 threads, 65535 rows of workgroups
  const double few = std::ceil(N / 32) * std::ceil(M / 64);
  const double small = std::ceil(N / 64) * std::ceil(M / 64);
  const double odd = (p->K | p->x_stride) % 4 != 0 ? 1.65 : 1;
  const double us[6] = {
      M <= 16 ? 2 + odd * N * K / 5e6 * (0.8 + M / 40) : never,
      M <= 32 ? 2 + odd * N * K / 5e6 * 1.7 : never,
      few < 1 << 22 && M < 1 << 21 ? 1 + odd * K / 4096 * 12.5 * std::ceil(few / 256) : never,
      small < 1 << 23 ? pad + tile_us(64, 512, 0.44, 0.29) : never,
      pad + tile_us(128, 512, 1.28, 0.75),
      pad + tile_us(256, 256, 2.2, 1.45),
  };
  int best = 0;
  for (int i = 1; i < 6; ++i)
    if (us[i] < us[best]) best = i;
  q.kernel = (decltype(q.kernel))best;
  if (best <= MatPlan::kFew64) q.pad_x = q.pad_w = false;
  return q;
}

template <typename F>
void by_out(const gdr_int8_matmul_problem* p, F f) {
  if (p->out_dtype == GDR_BF16) f(__bf16());
  else if (p->out_dtype == GDR_FP16) f(_Float16());
  else f(float());
}

}  // namespace

size_t int8_matmul_workspace(const gdr_int8_matmul_problem* p) {
  const MatPlan q = plan_of(p);
  return (q.pad_w ? align256((size_t)q.row * p->N) : 0) +
         (q.pad_x ? align256((size_t)q.row * p->M) : 0);
}

gdr_status launch_int8_matmul(const gdr_int8_matmul_problem* p, const void* x, const float* x_scale,
                              const void* w, const float* w_scale, const void* bias, void* y,
                              void* ws, hipStream_t st) {
  MatArgs a{};
  a.x = reinterpret_cast<const int8_t*>(x);
  a.w = reinterpret_cast<const int8_t*>(w);
  a.xs = x_scale; a.ws = w_scale; a.bias = bias; a.y = y;
  a.x_stride = p->x_stride;
  a.w_stride = p->K;
  a.M = p->M; a.N = p->N; a.K = p->K;
  a.bias_dtype = (int)p->bias_dtype;
  const MatPlan q = plan_of(p);
  if (q.pad_x) {
    int8_t* at = reinterpret_cast<int8_t*>(ws);
    PadArgs pad{};
    pad.K = p->K;
    pad.padded = (p->K + 15) / 16 * 16;
    pad.row = q.row;
    if (q.pad_w) {
      pad.src[0] = a.w; pad.dst[0] = at; pad.stride[0] = p->K; pad.rows[0] = p->N;
      a.w = at;
      a.w_stride = q.row;
      at += align256((size_t)q.row * p->N);
    }
    pad.src[1] = a.x; pad.dst[1] = at; pad.stride[1] = p->x_stride; pad.rows[1] = p->M;
    a.x = at;
    a.x_stride = q.row;
    a.K = pad.padded;
    const int64_t rows = (int64_t)pad.rows[0] + pad.rows[1];
    GDR_LAUNCH("int8_pad", int8_pad_kernel, dim3((unsigned)((rows + 3) / 4)), dim3(256), st, pad);
  }
  by_out(p, [&](auto o) {
    using O = decltype(o);
    auto few = [&](auto nb, auto mb) {
      constexpr int NB = nb.value, MB = mb.value;
      const dim3 grid((p->N + 16 * NB - 1) / (16 * NB), (p->M + 16 * MB - 1) / (16 * MB));
      const bool odd = (a.x_stride | a.w_stride | (intptr_t)a.x | (intptr_t)a.w) & 3;
      if (odd)
        GDR_LAUNCH("int8_few", (int8_few_kernel<NB, MB, true, O>), grid, dim3(64 * kSplit), st, a);
      else
        GDR_LAUNCH("int8_few", (int8_few_kernel<NB, MB, false, O>), grid, dim3(64 * kSplit), st, a);
    };
    auto tiles = [&](auto wn, auto wm, auto nb, auto mb, auto steps) {
      constexpr int WN = wn.value, WM = wm.value, NB = nb.value, MB = mb.value;
      a.tiles_n = (p->N + 32 * NB * WN - 1) / (32 * NB * WN);
      a.tiles_m = (p->M + 32 * MB * WM - 1) / (32 * MB * WM);
      GDR_LAUNCH("int8_tile", (int8_tile_kernel<WN, WM, NB, MB, steps.value, O>),
                 dim3((unsigned)((int64_t)a.tiles_m * a.tiles_n)), dim3(64 * WN * WM), st, a);
    };
    const std::integral_constant<int, 1> c1;
    const std::integral_constant<int, 2> c2;
    const std::integral_constant<int, 4> c4;
    switch (q.kernel) {
      case MatPlan::kFew16: return few(c1, c1);
      case MatPlan::kFew32: return few(c1, c2);
      case MatPlan::kFew64: return few(c2, c4);
      case MatPlan::kTile64: return tiles(c2, c2, c1, c1, c4);
      case MatPlan::kTile128: return tiles(c2, c2, c2, c2, c2);
      case MatPlan::kTile256: return tiles(c4, c2, c2, c4, c2);
    }
  });
  return launch_status("int8_matmul");
}

}  // namespace gdr

// conv1d.hip -- the short causal depthwise convolution in front of a linear
// recurrence, on gfx950.  Per channel d and token t of a sequence,
//   z[t] = b + sum_{j < W} w[j] x[t - (W-1) + j],   y[t] = z[t] or silu(z[t]),
// rows before the sequence's first token being the state's W - 1 rows (the
// last inputs of what came before) or zero.
//
// Every operand is touched once and there are about 2 W flops per element, so
// memory bounds all three kernels.  A thread owns 16 bytes of channels (8 bytes
// in small gradients) and walks a run of tokens with the last W - 1 rows in
// registers, so x is read once plus W - 1 rows per run; the rows of the next
// group are requested before the current group is computed.  Runs have 64
// tokens where the chip is full with them, and fewer, to 8, where it is not (512
// tokens of 4096 channels: 10 us against 25 with runs of 64); narrow tensors
// take fewer channels and more runs per block (60,000 tokens of 24 channels:
// 9 us against 26 with 64 channel vectors per block).  Where the width
// is no multiple of the vector, the last vector of a row is moved back to end
// with the row: it repeats some channels, with the same bits, and the loop
// has no partial accesses.
#include <algorithm>
#include <type_traits>

#include "ops_device.h"
#include "ops_internal.h"

namespace gdr {

namespace {

constexpr int kThreads = 256;
constexpr int U = 4;  // tokens requested ahead per thread

struct ConvArgs {
  const void* x;
  const void* w;
  const void* bias;  // nullable
  const void* s0;    // nullable
  void* y;
  void* s1;          // nullable
  const void* dy;
  const void* ds1;   // nullable
  void* dx;
  void* ds0;         // nullable
  float* part;       // [token blocks][W + 1][D]
  const int32_t* cu;
  int64_t x_stride;
  int N, T, D, wdt;
  int tokens;        // B * T
  int cv;            // channel vectors per block (a power of two); kThreads / cv token runs
  int ts;            // tokens per run
  int xblocks;       // channel blocks (the fast part of the block index)
  int blocks;        // token blocks; the rows of blocks past them handle empty sequences
  int empty_rows;    // rows of blocks that walk the sequences for empty ones
};

// The part of a sequence that a run covers: tokens [ta, tb) of sequence n,
// which spans [s, e).
struct Run {
  int n, s, e;
};

__device__ __forceinline__ Run find_run(const ConvArgs& a, int t) {
  Run r;
  if (a.cu) {
    r.n = find_seq(a.cu, a.N, t);
    r.s = a.cu[r.n];
    r.e = a.cu[r.n + 1];
  } else {
    r.n = t / a.T;
    r.s = r.n * a.T;
    r.e = r.s + a.T;
  }
  return r;
}

// Where a thread's channels start: the last vector ends with the row.  PART:
// rows narrower than a vector, of which a thread has m elements.
template <int N>
__device__ __forceinline__ int channel_of(int vi, int D) {
  return max(0, min(vi * N, D - N));
}

template <typename T, int N, bool PART>
__device__ __forceinline__ void load_row(const T* p, int m, Vec<T, N>& v) {
  if (PART) v.load_part(p, m);
  else v.load(p);
}
template <typename T, int N, bool PART>
__device__ __forceinline__ void store_row(T* p, int m, const Vec<T, N>& v) {
  if (PART) v.store_part(p, m);
  else v.store(p);
}

// Input row of token t of run r, or the state's row before the sequence.
template <typename T, int N, int W, bool PART>
__device__ __forceinline__ void row_before(const ConvArgs& a, const Run& r, int t, int c, int m,
                                           Vec<T, N>& v) {
  const T* x = reinterpret_cast<const T*>(a.x);
  const T* s0 = reinterpret_cast<const T*>(a.s0);
  if (t >= r.s)
    load_row<T, N, PART>(x + t * a.x_stride + c, m, v);
  else if (s0)
    load_row<T, N, PART>(s0 + ((int64_t)r.n * (W - 1) + (t - r.s + W - 1)) * a.D + c, m, v);
  else
    v.zero();
}

// The state after a sequence: its last W - 1 inputs (older state rows first
// when the sequence is shorter).
template <typename T, int N, int W, bool PART>
__device__ __forceinline__ void write_state(const ConvArgs& a, const Run& r, int c, int m) {
  T* s1 = reinterpret_cast<T*>(a.s1);
#pragma unroll
  for (int i = 0; i < W - 1; ++i) {
    Vec<T, N> v;
    row_before<T, N, W, PART>(a, r, r.e - (W - 1) + i, c, m, v);
    store_row<T, N, PART>(s1 + ((int64_t)r.n * (W - 1) + i) * a.D + c, m, v);
  }
}

template <int N, int W, bool PART>
struct Taps {
  float w[W][N], b[N];
  __device__ __forceinline__ void load(const ConvArgs& a, int c, int m) {
    if (!PART) {
      float f[N * W];
      load_params<N * W>(a.w, (int64_t)c * W, a.wdt, f);
      if (a.bias) load_params<N>(a.bias, c, a.wdt, b);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        if (!a.bias) b[e] = 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j) w[j][e] = f[e * W + j];
      }
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e) {
        b[e] = (a.bias && e < m) ? load_scalar(a.bias, c + e, a.wdt) : 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j)
          w[j][e] = e < m ? load_scalar(a.w, (int64_t)(c + e) * W + j, a.wdt) : 0.f;
      }
    }
  }
};

// The forward: 8192 tokens of 12,288 bf16 channels take 75 us, 5.4 TB/s, what
// a large copy reaches (fp32, half as many channels: 77).  18,062 tokens of 2505
// fp16 channels take 44 us for 181 MB, 4.1 TB/s (37 where they come from the
// caches): rows start at every alignment, and neighbouring blocks of channels
// and of tokens, which share lines and the W - 1 rows before a run, run on
// different XCDs.
template <typename T, int N, int W, bool SILU, bool PART>
__global__ __launch_bounds__(kThreads) void conv_fwd_kernel(ConvArgs a) {
  const int cvi = threadIdx.x & (a.cv - 1), sub = threadIdx.x / a.cv;
  const int bx = blockIdx.x % a.xblocks, by = blockIdx.x / a.xblocks;
  const int vi = bx * a.cv + cvi;
  if (vi * N >= a.D) return;
  const int c = channel_of<N>(vi, a.D), m = PART ? a.D : N;
  if (by >= a.blocks) {  // sequences without tokens keep their state
    const int runs = kThreads / a.cv;
    for (int n = (by - a.blocks) * runs + sub; n < a.N; n += a.empty_rows * runs) {
      const Run r{n, a.cu[n], a.cu[n + 1]};
      if (r.s == r.e) write_state<T, N, W, PART>(a, r, c, m);
    }
    return;
  }
  Taps<N, W, PART> tap;
  tap.load(a, c, m);
  const int64_t first = ((int64_t)by * (kThreads / a.cv) + sub) * a.ts;
  if (first >= a.tokens) return;
  const int last = (int)min((int64_t)a.tokens, first + a.ts);

  auto out = [&](const float (*ext)[N], T* y) {
    Vec<T, N> o;
#pragma unroll
    for (int e = 0; e < N; ++e) {
      float z = tap.b[e];
#pragma unroll
      for (int j = 0; j < W; ++j) z += tap.w[j][e] * ext[j][e];
      o.v[e] = from_f<T>(SILU ? z * sigmoid(z) : z);
    }
    store_row<T, N, PART>(y, m, o);
  };
  for (int ta = (int)first; ta < last;) {
    const Run r = find_run(a, ta);
    const int tb = min(last, r.e);
    const T* x = reinterpret_cast<const T*>(a.x) + ta * a.x_stride + c;
    T* y = reinterpret_cast<T*>(a.y) + (int64_t)ta * a.D + c;
    const int full = (tb - ta) / U;
    Vec<T, N> next[U];
    if (full > 0) {
#pragma unroll
      for (int i = 0; i < U; ++i) load_row<T, N, PART>(x + i * a.x_stride, m, next[i]);
      x += U * a.x_stride;
    }
    float ext[W - 1 + U][N];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      Vec<T, N> v;
      row_before<T, N, W, PART>(a, r, ta - (W - 1) + j, c, m, v);
#pragma unroll
      for (int e = 0; e < N; ++e) ext[j][e] = to_f(v.v[e]);
    }
    for (int g = 0; g < full; ++g) {
#pragma unroll
      for (int i = 0; i < U; ++i)
#pragma unroll
        for (int e = 0; e < N; ++e) ext[W - 1 + i][e] = to_f(next[i].v[e]);
      if (g + 1 < full) {
#pragma unroll
        for (int i = 0; i < U; ++i) load_row<T, N, PART>(x + i * a.x_stride, m, next[i]);
        x += U * a.x_stride;
      }
#pragma unroll
      for (int i = 0; i < U; ++i) out(&ext[i], y + (int64_t)i * a.D);
      y += (int64_t)U * a.D;
#pragma unroll
      for (int j = 0; j < W - 1; ++j)
#pragma unroll
        for (int e = 0; e < N; ++e) ext[j][e] = ext[j + U][e];
    }
    for (int t = ta + full * U; t < tb; ++t) {
      load_row<T, N, PART>(x, m, next[0]);
      x += a.x_stride;
#pragma unroll
      for (int e = 0; e < N; ++e) ext[W - 1][e] = to_f(next[0].v[e]);
      out(&ext[0], y);
      y += a.D;
#pragma unroll
      for (int j = 0; j < W - 1; ++j)
#pragma unroll
        for (int e = 0; e < N; ++e) ext[j][e] = ext[j + 1][e];
    }
    if (tb == r.e && a.s1) write_state<T, N, W, PART>(a, r, c, m);
    ta = tb;
  }
}

// The gradient.  With dz = dy act'(z), zero past the sequence's end,
//   dx[u] = sum_j w[j] dz[u + (W-1) - j]  (+ the state's gradient where x[u]
//   became one of its rows),  dw[j] = sum_t dz[t] x[t - (W-1) + j],
//   db = sum_t dz[t],
// so the walk recomputes z from x, keeps the last W - 1 rows of dz as well,
// and writes dx W - 1 tokens behind; a run reads W - 1 rows past its end.
// dw and db are summed in fp32 per run, over the block's runs through LDS in
// a fixed order, and over the blocks by conv_reduce_kernel: no atomics.
// 8192 tokens of 12,288 bf16 channels take 146 us, 4.1 TB/s: some 30 vector
// operations per element, an exponential and a reciprocal at a quarter of the
// rate among them, take about 115 us by themselves.
template <typename T, int N, int W, bool SILU, bool PART>
__global__ __launch_bounds__(kThreads) void conv_bwd_kernel(ConvArgs a) {
  __shared__ float red[kThreads * N];
  const int cvi = threadIdx.x & (a.cv - 1), sub = threadIdx.x / a.cv;
  const int bx = blockIdx.x % a.xblocks, by = blockIdx.x / a.xblocks;
  const int vi = bx * a.cv + cvi;
  const bool mine = vi * N < a.D;
  const int c = channel_of<N>(vi, a.D), m = PART ? a.D : N;
  const T* ds1 = reinterpret_cast<const T*>(a.ds1);
  T* ds0 = reinterpret_cast<T*>(a.ds0);
  if (by >= a.blocks) {  // a sequence without tokens passes its state's gradient through
    const int runs = kThreads / a.cv;
    for (int n = (by - a.blocks) * runs + sub; n < a.N && mine; n += a.empty_rows * runs) {
      if (a.cu[n] != a.cu[n + 1]) continue;
#pragma unroll
      for (int i = 0; i < W - 1; ++i) {
        const int64_t o = ((int64_t)n * (W - 1) + i) * a.D + c;
        Vec<T, N> v;
        if (ds1) load_row<T, N, PART>(ds1 + o, m, v);
        else v.zero();
        store_row<T, N, PART>(ds0 + o, m, v);
      }
    }
    return;
  }
  float dw[W][N], db[N];
#pragma unroll
  for (int e = 0; e < N; ++e) {
    db[e] = 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j) dw[j][e] = 0.f;
  }
  const int64_t first = ((int64_t)by * (kThreads / a.cv) + sub) * a.ts;
  if (mine && first < a.tokens) {
    Taps<N, W, PART> tap;
    tap.load(a, c, m);
    const int last = (int)min((int64_t)a.tokens, first + a.ts);
    // dz of the token whose window ext holds, its shares of dw and db
    auto grad = [&](const float (*ext)[N], const Vec<T, N>& gy, float* dz, bool own) {
#pragma unroll
      for (int e = 0; e < N; ++e) {
        float g = to_f(gy.v[e]);
        if (SILU) {
          float z = tap.b[e];
#pragma unroll
          for (int j = 0; j < W; ++j) z += tap.w[j][e] * ext[j][e];
          const float sg = sigmoid(z);
          g *= sg * (1.f + z * (1.f - sg));
        }
        dz[e] = g;
        if (own) {
          db[e] += g;
#pragma unroll
          for (int j = 0; j < W; ++j) dw[j][e] += g * ext[j][e];
        }
      }
    };
    for (int ta = (int)first; ta < last;) {
      const Run r = find_run(a, ta);
      const int tb = min(last, r.e);
      const int low = ta == r.s ? r.s - (W - 1) : ta;  // first row whose gradient is written
      // dx (or the state's gradient) of row u, from dz[0 .. W-1] of tokens u ..
      auto back = [&](const float (*dz)[N], int u, bool near_end) {
        float g[N];
#pragma unroll
        for (int e = 0; e < N; ++e) {
          g[e] = 0.f;
#pragma unroll
          for (int j = 0; j < W; ++j) g[e] += tap.w[j][e] * dz[W - 1 - j][e];
        }
        if (near_end && ds1 && u >= r.e - (W - 1)) {
          Vec<T, N> v;
          load_row<T, N, PART>(ds1 + ((int64_t)r.n * (W - 1) + (u - r.e + W - 1)) * a.D + c, m, v);
#pragma unroll
          for (int e = 0; e < N; ++e) g[e] += to_f(v.v[e]);
        }
        Vec<T, N> o;
#pragma unroll
        for (int e = 0; e < N; ++e) o.v[e] = from_f<T>(g[e]);
        if (u >= r.s)
          store_row<T, N, PART>(reinterpret_cast<T*>(a.dx) + (int64_t)u * a.D + c, m, o);
        else if (ds0)
          store_row<T, N, PART>(ds0 + ((int64_t)r.n * (W - 1) + (u - r.s + W - 1)) * a.D + c, m, o);
      };
      const T* x = reinterpret_cast<const T*>(a.x) + ta * a.x_stride + c;
      const T* dy = reinterpret_cast<const T*>(a.dy) + (int64_t)ta * a.D + c;
      const int full = (tb - ta) / U;
      Vec<T, N> nx[U], ny[U];
      if (full > 0) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
          load_row<T, N, PART>(x + i * a.x_stride, m, nx[i]);
          load_row<T, N, PART>(dy + (int64_t)i * a.D, m, ny[i]);
        }
        x += U * a.x_stride;
        dy += (int64_t)U * a.D;
      }
      float ext[W - 1 + U][N], dz[W - 1 + U][N];
#pragma unroll
      for (int j = 0; j < W - 1; ++j) {
        Vec<T, N> v;
        row_before<T, N, W, PART>(a, r, ta - (W - 1) + j, c, m, v);
#pragma unroll
        for (int e = 0; e < N; ++e) {
          ext[j][e] = to_f(v.v[e]);
          dz[j][e] = 0.f;
        }
      }
      for (int k = 0; k < full; ++k) {
        Vec<T, N> gy[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
          gy[i] = ny[i];
#pragma unroll
          for (int e = 0; e < N; ++e) ext[W - 1 + i][e] = to_f(nx[i].v[e]);
        }
        if (k + 1 < full) {
#pragma unroll
          for (int i = 0; i < U; ++i) {
            load_row<T, N, PART>(x + i * a.x_stride, m, nx[i]);
            load_row<T, N, PART>(dy + (int64_t)i * a.D, m, ny[i]);
          }
          x += U * a.x_stride;
          dy += (int64_t)U * a.D;
        }
        const int u0 = ta + k * U - (W - 1);
#pragma unroll
        for (int i = 0; i < U; ++i) {
          grad(&ext[i], gy[i], dz[W - 1 + i], true);
          if (u0 + i >= low) back(&dz[i], u0 + i, false);  // u0 + i + W - 1 < tb <= the end
        }
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
#pragma unroll
          for (int e = 0; e < N; ++e) {
            ext[j][e] = ext[j + U][e];
            dz[j][e] = dz[j + U][e];
          }
      }
      for (int t = ta + full * U; t < tb + W - 1; ++t) {
        if (t < r.e) {
          load_row<T, N, PART>(x, m, nx[0]);
          load_row<T, N, PART>(dy, m, ny[0]);
          x += a.x_stride;
          dy += a.D;
#pragma unroll
          for (int e = 0; e < N; ++e) ext[W - 1][e] = to_f(nx[0].v[e]);
          grad(&ext[0], ny[0], dz[W - 1], t < tb);
        } else {
#pragma unroll
          for (int e = 0; e < N; ++e) ext[W - 1][e] = dz[W - 1][e] = 0.f;
        }
        const int u = t - (W - 1);
        if (u >= low) back(&dz[0], u, true);
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
#pragma unroll
          for (int e = 0; e < N; ++e) {
            ext[j][e] = ext[j + 1][e];
            dz[j][e] = dz[j + 1][e];
          }
      }
      ta = tb;
    }
  }
  // the block's sums, runs in order
  const int cols = a.cv * N, runs = kThreads / a.cv;
#pragma unroll
  for (int j = 0; j <= W; ++j) {
    __syncthreads();
#pragma unroll
    for (int e = 0; e < N; ++e) red[sub * cols + cvi * N + e] = j < W ? dw[j < W ? j : 0][e] : db[e];
    __syncthreads();
    for (int k = threadIdx.x; k < cols; k += kThreads) {
      const int kv = bx * a.cv + k / N, d = channel_of<N>(kv, a.D) + k % N;
      if (kv * N < a.D && d < a.D) {
        float s = 0.f;
        for (int q = 0; q < runs; ++q) s += red[q * cols + k];
        a.part[((int64_t)by * (W + 1) + j) * a.D + d] = s;
      }
    }
  }
}

// dw[d][j] and db[d] from the blocks' sums: 64 columns by 16 shares of the
// blocks (fixed order).  6 to 8 us, mostly latency; at most 512 blocks' sums
// (2048 of them cost the gradient 190 instead of 157 us).
__global__ __launch_bounds__(1024) void conv_reduce_kernel(const float* part, int blocks, int D,
                                                           int W, void* dw, void* db, int wdt) {
  __shared__ float red[16][64];
  const int64_t cols = (int64_t)(W + 1) * D;
  const int l = threadIdx.x & 63, q = threadIdx.x >> 6;
  const int64_t k = (int64_t)blockIdx.x * 64 + l;
  float s = 0.f;
  if (k < cols)
#pragma unroll 8
    for (int b = q; b < blocks; b += 16) s += part[b * cols + k];
  red[q][l] = s;
  __syncthreads();
  if (q == 0 && k < cols) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) s += red[i][l];
    const int j = (int)(k / D), d = (int)(k % D);
    if (j < W)
      store_scalar(dw, (int64_t)d * W + j, wdt, s);
    else if (db)
      store_scalar(db, d, wdt, s);
  }
}

// One or a few tokens per sequence on a cached state, updated in place: the
// thread that reads a state column writes it, so vectors do not overlap and
// the last one of a row may be partial (TAIL).  256 sequences of 12,288 bf16
// channels: 50 MB in 8.8 us from the caches, 10 us from memory.
template <typename T, int N, int W, bool SILU, bool TAIL>
__global__ __launch_bounds__(kThreads) void conv_update_kernel(ConvArgs a) {
  const int bx = blockIdx.x % a.xblocks, n = blockIdx.x / a.xblocks;
  const int c = (bx * kThreads + threadIdx.x) * N;
  const int m = min(N, a.D - c);
  if (m <= 0) return;
  const T* x = reinterpret_cast<const T*>(a.x) + (int64_t)n * a.T * a.x_stride + c;
  T* st = reinterpret_cast<T*>(a.s1) + (int64_t)n * (W - 1) * a.D + c;
  T* y = reinterpret_cast<T*>(a.y) + (int64_t)n * a.T * a.D + c;
  Vec<T, N> row[W];
#pragma unroll
  for (int j = 0; j < W - 1; ++j) load_row<T, N, TAIL>(st + (int64_t)j * a.D, m, row[j]);
  load_row<T, N, TAIL>(x, m, row[W - 1]);
  float w[W][N], b[N];
  if (!TAIL || m == N) {
    Taps<N, W, false> tap;
    tap.load(a, c, N);
    __builtin_memcpy(w, tap.w, sizeof(w));
    __builtin_memcpy(b, tap.b, sizeof(b));
  } else {
    Taps<N, W, true> tap;
    tap.load(a, c, m);
    __builtin_memcpy(w, tap.w, sizeof(w));
    __builtin_memcpy(b, tap.b, sizeof(b));
  }
  for (int t = 0;;) {
    Vec<T, N> o;
#pragma unroll
    for (int e = 0; e < N; ++e) {
      float z = b[e];
#pragma unroll
      for (int j = 0; j < W; ++j) z += w[j][e] * to_f(row[j].v[e]);
      o.v[e] = from_f<T>(SILU ? z * sigmoid(z) : z);
    }
    store_row<T, N, TAIL>(y + (int64_t)t * a.D, m, o);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) row[j] = row[j + 1];
    if (++t >= a.T) break;
    load_row<T, N, TAIL>(x + t * a.x_stride, m, row[W - 1]);
  }
#pragma unroll
  for (int j = 0; j < W - 1; ++j) store_row<T, N, TAIL>(st + (int64_t)j * a.D, m, row[j]);
}

struct Shape {
  int cv, ts, xblocks, yblocks;
};

// cv channel vectors (of N channels) by 256 / cv runs of ts tokens per block.
// Narrow tensors take fewer channels and more runs, so that every lane has
// work; runs shorten until the launch has `want` blocks, and lengthen while
// there are more than `most` token blocks (whose partial sums the weight
// gradient has to read back).
Shape shape_of(const gdr_conv_problem* p, int N, int want, int most) {
  const int nv = (p->D + N - 1) / N;
  Shape s;
  s.cv = 64;
  while (s.cv > 4 && s.cv / 2 >= nv) s.cv /= 2;
  s.xblocks = (nv + s.cv - 1) / s.cv;
  const int64_t tokens = (int64_t)p->B * p->T;
  const int runs = kThreads / s.cv;
  auto yb = [&](int ts) { return (tokens + (int64_t)ts * runs - 1) / ((int64_t)ts * runs); };
  s.ts = 64;
  while (s.ts > 8 && yb(s.ts) * s.xblocks < want) s.ts /= 2;
  while (yb(s.ts) > most) s.ts *= 2;
  s.yblocks = (int)yb(s.ts);
  return s;
}

constexpr int kFwdBlocks = 1024, kBwdBlocks = 768, kMostParts = 512, kMostGridY = 32768;

ConvArgs args_of(const gdr_conv_problem* p, const Shape& s) {
  ConvArgs a{};
  a.cu = p->cu_seqlens_dev;
  a.x_stride = p->x_stride;
  a.N = p->N;
  a.T = p->T;
  a.D = p->D;
  a.wdt = (int)p->w_dtype;
  a.tokens = p->B * p->T;
  a.cv = s.cv;
  a.ts = s.ts;
  a.xblocks = s.xblocks;
  a.blocks = s.yblocks;
  return a;
}

// Rows of blocks for the sequences without tokens, when there are any.
int empty_rows(const gdr_conv_problem* p, int runs) {
  if (!p->cu_seqlens_host) return 0;
  for (int n = 0; n < p->N; ++n)
    if (p->cu_seqlens_host[n + 1] == p->cu_seqlens_host[n])
      return std::min(1024, (p->N + runs - 1) / runs);
  return 0;
}

// Channels per thread: 16 bytes of the type.  In the gradient, whose rows,
// weights and sums take 142 registers for four channels and 250 for eight, 16
// bytes where that still leaves a run of 64 tokens to every thread (8192
// tokens of 12,288 bf16 channels: 146 us against 157), else four channels
// (512 tokens of 4096: 15 us against 21; 4096 of 64: 11 against 15).
int fwd_channels(const gdr_conv_problem* p) { return p->dtype == GDR_FP32 ? 4 : 8; }
int bwd_channels(const gdr_conv_problem* p) {
  const int wide = fwd_channels(p);
  return shape_of(p, wide, kBwdBlocks, kMostParts).ts >= 64 ? wide : 4;
}

// The type, the width, the activation and whether some access is partial.
template <typename F>
void by_type(const gdr_conv_problem* p, bool part, F f) {
  auto width = [&](auto t) {
    using T = decltype(t);
    auto act = [&](auto w) {
      constexpr int W = decltype(w)::value;
      const std::integral_constant<int, W> wc;
      if (p->activation) {
        if (part) f(T(), wc, std::true_type(), std::true_type());
        else f(T(), wc, std::true_type(), std::false_type());
      } else {
        if (part) f(T(), wc, std::false_type(), std::true_type());
        else f(T(), wc, std::false_type(), std::false_type());
      }
    };
    if (p->W == 2) act(std::integral_constant<int, 2>());
    else if (p->W == 3) act(std::integral_constant<int, 3>());
    else act(std::integral_constant<int, 4>());
  };
  if (p->dtype == GDR_BF16) width(__bf16());
  else if (p->dtype == GDR_FP16) width(_Float16());
  else width(float());
}

}  // namespace

gdr_status launch_status(const char* what) {
  const hipError_t e = hipGetLastError();
  if (e == hipSuccess) return GDR_OK;
  set_error("%s launch failed: %s", what, hipGetErrorString(e));
  return GDR_ERR_HIP;
}

gdr_status launch_conv_fwd(const gdr_conv_problem* p, const void* x, const void* weight,
                           const void* bias, const void* s0, void* y, void* s1, hipStream_t st) {
  const int N = fwd_channels(p);
  const Shape s = shape_of(p, N, kFwdBlocks, kMostGridY);
  ConvArgs a = args_of(p, s);
  a.x = x; a.w = weight; a.bias = bias; a.s0 = s0; a.y = y; a.s1 = s1;
  a.empty_rows = s1 ? empty_rows(p, kThreads / s.cv) : 0;
  const dim3 grid((unsigned)s.xblocks * (unsigned)(s.yblocks + a.empty_rows));
  by_type(p, p->D < N, [&](auto t, auto w, auto silu, auto part) {
    using T = decltype(t);
    GDR_LAUNCH("conv_fwd",
               (conv_fwd_kernel<T, 16 / (int)sizeof(T), w.value, silu.value, part.value>), grid,
               dim3(kThreads), st, a);
  });
  return launch_status("conv_fwd");
}

size_t conv_bwd_workspace(const gdr_conv_problem* p) {
  const Shape s = shape_of(p, bwd_channels(p), kBwdBlocks, kMostParts);
  return align256((size_t)s.yblocks * (p->W + 1) * p->D * sizeof(float));
}

gdr_status launch_conv_bwd(const gdr_conv_problem* p, const void* x, const void* weight,
                           const void* bias, const void* dy, const void* ds1, const void* s0,
                           void* dx, void* dw, void* db, void* ds0, void* ws, hipStream_t st) {
  const int N = bwd_channels(p);
  const Shape s = shape_of(p, N, kBwdBlocks, kMostParts);
  ConvArgs a = args_of(p, s);
  a.x = x; a.w = weight; a.bias = bias; a.s0 = s0; a.dy = dy; a.ds1 = ds1;
  a.dx = dx; a.ds0 = ds0; a.part = reinterpret_cast<float*>(ws);
  a.empty_rows = ds0 ? empty_rows(p, kThreads / s.cv) : 0;
  const dim3 grid((unsigned)s.xblocks * (unsigned)(s.yblocks + a.empty_rows));
  by_type(p, p->D < N, [&](auto t, auto w, auto silu, auto part) {
    using T = decltype(t);
    constexpr int wide = 16 / (int)sizeof(T);
    if (N == 4)
      GDR_LAUNCH("conv_bwd", (conv_bwd_kernel<T, 4, w.value, silu.value, part.value>), grid,
                 dim3(kThreads), st, a);
    else
      GDR_LAUNCH("conv_bwd", (conv_bwd_kernel<T, wide, w.value, silu.value, part.value>), grid,
                 dim3(kThreads), st, a);
  });
  const int64_t cols = (int64_t)(p->W + 1) * p->D;
  GDR_LAUNCH("conv_reduce", conv_reduce_kernel, dim3((unsigned)((cols + 63) / 64)), dim3(1024), st,
             a.part, s.yblocks, p->D, p->W, dw, db, (int)p->w_dtype);
  return launch_status("conv_bwd");
}

gdr_status launch_conv_update(const gdr_conv_problem* p, const void* x, void* state,
                              const void* weight, const void* bias, void* y, hipStream_t st) {
  const int N = fwd_channels(p);
  const int nv = (p->D + N - 1) / N;
  ConvArgs a = args_of(p, Shape{1, 1, (nv + kThreads - 1) / kThreads, 0});
  a.x = x; a.w = weight; a.bias = bias; a.y = y; a.s1 = state;
  const dim3 grid((unsigned)a.xblocks * (unsigned)p->B);
  by_type(p, p->D % N != 0, [&](auto t, auto w, auto silu, auto part) {
    using T = decltype(t);
    GDR_LAUNCH("conv_update",
               (conv_update_kernel<T, 16 / (int)sizeof(T), w.value, silu.value, part.value>), grid,
               dim3(kThreads), st, a);
  });
  return launch_status("conv_update");
}

}  // namespace gdr

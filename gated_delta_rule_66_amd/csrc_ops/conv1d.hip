// conv1d.hip -- the short causal depthwise convolution in front of a linear
// recurrence, on gfx950.  Per channel d and token t of a sequence,
//   z[t] = b + sum_{j < W} w[j] x[t - (W-1) + j],   y[t] = z[t] or silu(z[t]),
// rows before the sequence's first token being the state's W - 1 rows (the
// last inputs of what came before) or zero.
//
// Every operand is touched once and there are about 2 W flops per element, so
// memory bounds all three kernels.  A thread owns 16 bytes of channels (one
// load per token row) and walks a run of tokens with the last W - 1 rows in
// registers, so x is read once plus W - 1 rows per run; the rows of the next
// group are requested before the current group is computed.
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

// Input row of token t of run r, or the state's row before the sequence.
template <typename T, int W>
__device__ __forceinline__ void row_before(const ConvArgs& a, const Run& r, int t, int c, int m,
                                           Vec<T>& v) {
  const T* x = reinterpret_cast<const T*>(a.x);
  const T* s0 = reinterpret_cast<const T*>(a.s0);
  if (t >= r.s) {
    v.load_part(x + t * a.x_stride + c, m);
  } else if (s0) {
    v.load_part(s0 + ((int64_t)r.n * (W - 1) + (t - r.s + W - 1)) * a.D + c, m);
  } else {
#pragma unroll
    for (int e = 0; e < Vec<T>::n; ++e) v.v[e] = (T)0.f;
  }
}

// The state after a sequence: its last W - 1 inputs (older state rows first
// when the sequence is shorter).
template <typename T, int W>
__device__ __forceinline__ void write_state(const ConvArgs& a, const Run& r, int c, int m) {
  T* s1 = reinterpret_cast<T*>(a.s1);
#pragma unroll
  for (int i = 0; i < W - 1; ++i) {
    Vec<T> v;
    row_before<T, W>(a, r, r.e - (W - 1) + i, c, m, v);
    v.store_part(s1 + ((int64_t)r.n * (W - 1) + i) * a.D + c, m);
  }
}

template <typename T, int W>
struct Taps {
  float w[W][Vec<T>::n], b[Vec<T>::n];
  __device__ __forceinline__ void load(const ConvArgs& a, int c, int m) {
#pragma unroll
    for (int e = 0; e < Vec<T>::n; ++e) {
      b[e] = (a.bias && e < m) ? load_param(a.bias, c + e, a.wdt) : 0.f;
#pragma unroll
      for (int j = 0; j < W; ++j)
        w[j][e] = e < m ? load_param(a.w, (int64_t)(c + e) * W + j, a.wdt) : 0.f;
    }
  }
};

template <typename T, int W, bool SILU>
__global__ __launch_bounds__(kThreads) void conv_fwd_kernel(ConvArgs a) {
  constexpr int V = Vec<T>::n;
  const int cvi = threadIdx.x & (a.cv - 1), sub = threadIdx.x / a.cv;
  const int bx = blockIdx.x % a.xblocks, by = blockIdx.x / a.xblocks;
  const int c = (bx * a.cv + cvi) * V;
  const int m = min(V, a.D - c);
  if (m <= 0) return;
  if (by >= a.blocks) {  // sequences without tokens keep their state
    const int runs = kThreads / a.cv;
    for (int n = (by - a.blocks) * runs + sub; n < a.N; n += a.empty_rows * runs) {
      const Run r{n, a.cu[n], a.cu[n + 1]};
      if (r.s == r.e) write_state<T, W>(a, r, c, m);
    }
    return;
  }
  Taps<T, W> tap;
  tap.load(a, c, m);
  const T* x = reinterpret_cast<const T*>(a.x);
  T* y = reinterpret_cast<T*>(a.y);
  const int64_t first = ((int64_t)by * (kThreads / a.cv) + sub) * a.ts;
  if (first >= a.tokens) return;
  const int last = (int)min((int64_t)a.tokens, first + a.ts);

  for (int ta = (int)first; ta < last;) {
    const Run r = find_run(a, ta);
    const int tb = min(last, r.e);
    float ext[W - 1 + U][V];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      Vec<T> v;
      row_before<T, W>(a, r, ta - (W - 1) + j, c, m, v);
#pragma unroll
      for (int e = 0; e < V; ++e) ext[j][e] = to_f(v.v[e]);
    }
    Vec<T> next[U];
#pragma unroll
    for (int i = 0; i < U; ++i)
      if (ta + i < tb) next[i].load_part(x + (ta + i) * a.x_stride + c, m);
    for (int t = ta; t < tb; t += U) {
#pragma unroll
      for (int i = 0; i < U; ++i)
#pragma unroll
        for (int e = 0; e < V; ++e) ext[W - 1 + i][e] = to_f(next[i].v[e]);
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (t + U + i < tb) next[i].load_part(x + (t + U + i) * a.x_stride + c, m);
#pragma unroll
      for (int i = 0; i < U; ++i) {
        if (t + i < tb) {
          Vec<T> o;
#pragma unroll
          for (int e = 0; e < V; ++e) {
            float z = tap.b[e];
#pragma unroll
            for (int j = 0; j < W; ++j) z += tap.w[j][e] * ext[i + j][e];
            o.v[e] = from_f<T>(SILU ? z * sigmoid(z) : z);
          }
          o.store_part(y + (int64_t)(t + i) * a.D + c, m);
        }
      }
#pragma unroll
      for (int j = 0; j < W - 1; ++j)
#pragma unroll
        for (int e = 0; e < V; ++e) ext[j][e] = ext[j + U][e];
    }
    if (tb == r.e && a.s1) write_state<T, W>(a, r, c, m);
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
template <typename T, int W, bool SILU>
__global__ __launch_bounds__(kThreads) void conv_bwd_kernel(ConvArgs a) {
  constexpr int V = Vec<T>::n;
  __shared__ float red[kThreads * V];
  const int cvi = threadIdx.x & (a.cv - 1), sub = threadIdx.x / a.cv;
  const int bx = blockIdx.x % a.xblocks, by = blockIdx.x / a.xblocks;
  const int c = (bx * a.cv + cvi) * V;
  const int m = min(V, a.D - c);
  const T* x = reinterpret_cast<const T*>(a.x);
  const T* dy = reinterpret_cast<const T*>(a.dy);
  const T* ds1 = reinterpret_cast<const T*>(a.ds1);
  T* dx = reinterpret_cast<T*>(a.dx);
  T* ds0 = reinterpret_cast<T*>(a.ds0);
  if (by >= a.blocks) {  // a sequence without tokens passes its state's gradient through
    const int runs = kThreads / a.cv;
    for (int n = (by - a.blocks) * runs + sub; n < a.N && m > 0; n += a.empty_rows * runs) {
      if (a.cu[n] != a.cu[n + 1]) continue;
#pragma unroll
      for (int i = 0; i < W - 1; ++i) {
        const int64_t o = ((int64_t)n * (W - 1) + i) * a.D + c;
        Vec<T> v;
        if (ds1) {
          v.load_part(ds1 + o, m);
        } else {
#pragma unroll
          for (int e = 0; e < V; ++e) v.v[e] = (T)0.f;
        }
        v.store_part(ds0 + o, m);
      }
    }
    return;
  }
  float dw[W][V], db[V];
#pragma unroll
  for (int e = 0; e < V; ++e) {
    db[e] = 0.f;
#pragma unroll
    for (int j = 0; j < W; ++j) dw[j][e] = 0.f;
  }
  const int64_t first = ((int64_t)by * (kThreads / a.cv) + sub) * a.ts;
  if (m > 0 && first < a.tokens) {
    Taps<T, W> tap;
    tap.load(a, c, m);
    const int last = (int)min((int64_t)a.tokens, first + a.ts);
    for (int ta = (int)first; ta < last;) {
      const Run r = find_run(a, ta);
      const int tb = min(last, r.e);
      const int lend = min(r.e, tb + W - 1);         // rows that are read
      const int low = ta == r.s ? r.s - (W - 1) : ta;  // first row whose gradient is written
      float ext[W - 1 + U][V], dz[W - 1 + U][V];
#pragma unroll
      for (int j = 0; j < W - 1; ++j) {
        Vec<T> v;
        row_before<T, W>(a, r, ta - (W - 1) + j, c, m, v);
#pragma unroll
        for (int e = 0; e < V; ++e) {
          ext[j][e] = to_f(v.v[e]);
          dz[j][e] = 0.f;
        }
      }
      Vec<T> nx[U], ny[U];
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (ta + i < lend) {
          nx[i].load_part(x + (ta + i) * a.x_stride + c, m);
          ny[i].load_part(dy + (int64_t)(ta + i) * a.D + c, m);
        }
      for (int t = ta; t < tb + W - 1; t += U) {
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const bool live = t + i < lend, own = t + i < tb;
#pragma unroll
          for (int e = 0; e < V; ++e) {
            ext[W - 1 + i][e] = live ? to_f(nx[i].v[e]) : 0.f;
            float g = live ? to_f(ny[i].v[e]) : 0.f;
            if (SILU) {
              float z = tap.b[e];
#pragma unroll
              for (int j = 0; j < W; ++j) z += tap.w[j][e] * ext[i + j][e];
              const float sg = sigmoid(z);
              g = live ? g * (sg * (1.f + z * (1.f - sg))) : 0.f;
            }
            dz[W - 1 + i][e] = g;
            if (own) {
              db[e] += g;
#pragma unroll
              for (int j = 0; j < W; ++j) dw[j][e] += g * ext[i + j][e];
            }
          }
        }
#pragma unroll
        for (int i = 0; i < U; ++i)
          if (t + U + i < lend) {
            nx[i].load_part(x + (t + U + i) * a.x_stride + c, m);
            ny[i].load_part(dy + (int64_t)(t + U + i) * a.D + c, m);
          }
#pragma unroll
        for (int i = 0; i < U; ++i) {
          const int u = t + i - (W - 1);
          if (u >= low && u < tb) {
            float g[V];
#pragma unroll
            for (int e = 0; e < V; ++e) {
              g[e] = 0.f;
#pragma unroll
              for (int j = 0; j < W; ++j) g[e] += tap.w[j][e] * dz[i + W - 1 - j][e];
            }
            if (ds1 && u >= r.e - (W - 1)) {
              Vec<T> v;
              v.load_part(ds1 + ((int64_t)r.n * (W - 1) + (u - r.e + W - 1)) * a.D + c, m);
#pragma unroll
              for (int e = 0; e < V; ++e) g[e] += to_f(v.v[e]);
            }
            Vec<T> o;
#pragma unroll
            for (int e = 0; e < V; ++e) o.v[e] = from_f<T>(g[e]);
            if (u >= r.s)
              o.store_part(dx + (int64_t)u * a.D + c, m);
            else if (ds0)
              o.store_part(ds0 + ((int64_t)r.n * (W - 1) + (u - r.s + W - 1)) * a.D + c, m);
          }
        }
#pragma unroll
        for (int j = 0; j < W - 1; ++j)
#pragma unroll
          for (int e = 0; e < V; ++e) {
            ext[j][e] = ext[j + U][e];
            dz[j][e] = dz[j + U][e];
          }
      }
      ta = tb;
    }
  }
  // the block's sums, runs in order
  const int cols = a.cv * V, runs = kThreads / a.cv;
#pragma unroll
  for (int j = 0; j <= W; ++j) {
    __syncthreads();
#pragma unroll
    for (int e = 0; e < V; ++e) red[sub * cols + cvi * V + e] = j < W ? dw[j < W ? j : 0][e] : db[e];
    __syncthreads();
    for (int k = threadIdx.x; k < cols; k += kThreads) {
      const int d = bx * cols + k;
      if (d < a.D) {
        float s = 0.f;
        for (int q = 0; q < runs; ++q) s += red[q * cols + k];
        a.part[((int64_t)by * (W + 1) + j) * a.D + d] = s;
      }
    }
  }
}

// dw[d][j] and db[d] from the blocks' sums: 64 columns per workgroup, the
// blocks split over its four waves (fixed order).
__global__ __launch_bounds__(256) void conv_reduce_kernel(const float* part, int blocks, int D, int W,
                                                          void* dw, void* db, int wdt) {
  __shared__ float red[4][64];
  const int64_t cols = (int64_t)(W + 1) * D;
  const int l = threadIdx.x & 63, q = threadIdx.x >> 6;
  const int64_t k = (int64_t)blockIdx.x * 64 + l;
  float s = 0.f;
  if (k < cols)
#pragma unroll 8
    for (int b = q; b < blocks; b += 4) s += part[b * cols + k];
  red[q][l] = s;
  __syncthreads();
  if (q == 0 && k < cols) {
    s = (red[0][l] + red[1][l]) + (red[2][l] + red[3][l]);
    const int j = (int)(k / D), d = (int)(k % D);
    if (j < W)
      store_scalar(dw, (int64_t)d * W + j, wdt, s);
    else if (db)
      store_scalar(db, d, wdt, s);
  }
}

// One or a few tokens per sequence on a cached state, updated in place: the
// thread that reads a state column writes it.
template <typename T, int W, bool SILU>
__global__ __launch_bounds__(kThreads) void conv_update_kernel(ConvArgs a) {
  constexpr int V = Vec<T>::n;
  const int c = (blockIdx.x * kThreads + threadIdx.x) * V;
  const int m = min(V, a.D - c);
  if (m <= 0) return;
  const int n = blockIdx.y;
  const T* x = reinterpret_cast<const T*>(a.x) + (int64_t)n * a.T * a.x_stride + c;
  T* st = reinterpret_cast<T*>(a.s1) + (int64_t)n * (W - 1) * a.D + c;
  T* y = reinterpret_cast<T*>(a.y) + (int64_t)n * a.T * a.D + c;
  Vec<T> row[W];
#pragma unroll
  for (int j = 0; j < W - 1; ++j) row[j].load_part(st + (int64_t)j * a.D, m);
  row[W - 1].load_part(x, m);
  Taps<T, W> tap;
  tap.load(a, c, m);
  for (int t = 0;;) {
    Vec<T> o;
#pragma unroll
    for (int e = 0; e < V; ++e) {
      float z = tap.b[e];
#pragma unroll
      for (int j = 0; j < W; ++j) z += tap.w[j][e] * to_f(row[j].v[e]);
      o.v[e] = from_f<T>(SILU ? z * sigmoid(z) : z);
    }
    o.store_part(y + (int64_t)t * a.D, m);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) row[j] = row[j + 1];
    if (++t >= a.T) break;
    row[W - 1].load_part(x + t * a.x_stride, m);
  }
#pragma unroll
  for (int j = 0; j < W - 1; ++j) row[j].store_part(st + (int64_t)j * a.D, m);
}

struct Shape {
  int cv, ts, xblocks, yblocks;
};

// cv channel vectors (16 bytes each) by 256 / cv runs of ts tokens per block.
// Narrow tensors take fewer channels and more runs, so that every lane has
// work; runs shorten until the launch has `want` blocks, and lengthen while
// there are more than `most` token blocks (whose partial sums the weight
// gradient has to read back).
Shape shape_of(const gdr_conv_problem* p, int want, int most) {
  const int V = p->dtype == GDR_FP32 ? 4 : 8;
  const int nv = (p->D + V - 1) / V;
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

template <typename F>
void by_type(const gdr_conv_problem* p, F f) {
  auto width = [&](auto t) {
    using T = decltype(t);
    auto act = [&](auto w) {
      constexpr int W = decltype(w)::value;
      if (p->activation) f(T(), std::integral_constant<int, W>(), std::true_type());
      else f(T(), std::integral_constant<int, W>(), std::false_type());
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
  const Shape s = shape_of(p, kFwdBlocks, kMostGridY);
  ConvArgs a = args_of(p, s);
  a.x = x; a.w = weight; a.bias = bias; a.s0 = s0; a.y = y; a.s1 = s1;
  a.empty_rows = s1 ? empty_rows(p, kThreads / s.cv) : 0;
  const dim3 grid((unsigned)s.xblocks * (unsigned)(s.yblocks + a.empty_rows));
  by_type(p, [&](auto t, auto w, auto silu) {
    GDR_LAUNCH("conv_fwd", (conv_fwd_kernel<decltype(t), w.value, silu.value>), grid,
               dim3(kThreads), st, a);
  });
  return launch_status("conv_fwd");
}

size_t conv_bwd_workspace(const gdr_conv_problem* p) {
  const Shape s = shape_of(p, kBwdBlocks, kMostParts);
  return align256((size_t)s.yblocks * (p->W + 1) * p->D * sizeof(float));
}

gdr_status launch_conv_bwd(const gdr_conv_problem* p, const void* x, const void* weight,
                           const void* bias, const void* dy, const void* ds1, const void* s0,
                           void* dx, void* dw, void* db, void* ds0, void* ws, hipStream_t st) {
  const Shape s = shape_of(p, kBwdBlocks, kMostParts);
  ConvArgs a = args_of(p, s);
  a.x = x; a.w = weight; a.bias = bias; a.s0 = s0; a.dy = dy; a.ds1 = ds1;
  a.dx = dx; a.ds0 = ds0; a.part = reinterpret_cast<float*>(ws);
  a.empty_rows = ds0 ? empty_rows(p, kThreads / s.cv) : 0;
  const dim3 grid((unsigned)s.xblocks * (unsigned)(s.yblocks + a.empty_rows));
  by_type(p, [&](auto t, auto w, auto silu) {
    GDR_LAUNCH("conv_bwd", (conv_bwd_kernel<decltype(t), w.value, silu.value>), grid,
               dim3(kThreads), st, a);
  });
  const int64_t cols = (int64_t)(p->W + 1) * p->D;
  GDR_LAUNCH("conv_reduce", conv_reduce_kernel, dim3((unsigned)((cols + 63) / 64)), dim3(256), st,
             a.part, s.yblocks, p->D, p->W, dw, db, (int)p->w_dtype);
  return launch_status("conv_bwd");
}

gdr_status launch_conv_update(const gdr_conv_problem* p, const void* x, void* state,
                              const void* weight, const void* bias, void* y, hipStream_t st) {
  const int V = p->dtype == GDR_FP32 ? 4 : 8;
  const int nv = (p->D + V - 1) / V;
  ConvArgs a = args_of(p, Shape{1, 1, 1, 0});
  a.x = x; a.w = weight; a.bias = bias; a.y = y; a.s1 = state;
  const dim3 grid((nv + kThreads - 1) / kThreads, p->B);
  by_type(p, [&](auto t, auto w, auto silu) {
    GDR_LAUNCH("conv_update", (conv_update_kernel<decltype(t), w.value, silu.value>), grid,
               dim3(kThreads), st, a);
  });
  return launch_status("conv_update");
}

}  // namespace gdr

// rms_norm.hip -- root-mean-square norm with the residual's addition, on
// gfx950: h = x + r (rounded to the residual's type, the stream that the next
// layer adds to), y = w h / sqrt(mean h^2 + eps), y in the input's type or in
// 8 bits with a scale per row or per 128 columns; and its gradient.
//
// Memory bounds it: every operand is touched once.  A row stays in the
// registers of its threads, 8 elements each per step, from its load through
// the sum of squares to the store.
#include <algorithm>
#include <type_traits>

#include "norm_device.h"

namespace gdr {

namespace {

struct NormArgs {
  const void* x;
  const void* res;     // nullable
  const void* w;
  void* y;
  float* scale;
  void* h;             // stored when a residual is added
  float* rstd;         // nullable
  int64_t x_stride;    // elements between rows of x
  int rows, D, wdt, group, quant;
  float eps;
  // backward
  const void* dy;
  const void* dh;      // nullable: the gradient of the stored stream
  void* dx;
  void* dres;          // nullable
  float* part;         // [blocks][D]
  int blocks;
};

// The forward.  RES: the residual's type, void without one.  Memory bounds it:
// 16,384 rows of 4096 bf16 columns with a residual to e4m3 take 89 us for 472
// MB (5.3 TB/s; to int8 the same), 8192 of them to bf16 46 us for 268 MB (5.8);
// eight rows take 5 us, the latency of a load and two reductions.
template <typename T, typename RES, bool QUANT, int NT, int VPT, bool PART>
__global__ __launch_bounds__(block_of<NT>()) void norm_fwd_kernel(NormArgs a) {
  constexpr bool kRes = !std::is_void<RES>::value;
  typedef typename std::conditional<kRes, RES, T>::type R;
  __shared__ __align__(8) float lds[32];
  const int tid = NT == 64 ? (threadIdx.x & 63) : threadIdx.x;
  const int64_t row = NT == 64 ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6) : (int64_t)blockIdx.x;
  if (row >= a.rows) return;  // a whole wave; the barriers below are for NT > 64 only
  const T* x = reinterpret_cast<const T*>(a.x) + row * a.x_stride;
  const R* res = reinterpret_cast<const R*>(a.res) + row * a.D;
  R* h = reinterpret_cast<R*>(a.h) + row * a.D;
  float f[VPT][8], r[kRes ? VPT : 1][8];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = column_of<PART>(i * NT + tid, a.D);
    load8<T, PART>(x + c, a.D, f[i]);
    if (kRes) load8<R, PART>(res + c, a.D, r[kRes ? i : 0]);
  }
  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v0 = (i * NT + tid) * 8, c = column_of<PART>(i * NT + tid, a.D);
    if (kRes) {
      // the norm is of the stored stream, so that the gradient, which reads
      // it, is the gradient of what was computed
#pragma unroll
      for (int e = 0; e < 8; ++e) f[i][e] = to_f(from_f<R>(f[i][e] + r[kRes ? i : 0][e]));
      if (v0 < a.D) store8<R, PART>(h + c, a.D, f[i]);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const double v = c + e >= v0 ? f[i][e] : 0.f;
      sum = __builtin_fma(v, v, sum);
    }
  }
  // squares, mean and root in 64 bits: fp32 values beyond 2^64 have squares
  // past fp32's range and values below 2^-63 none at all, and the row's
  // statistic is the same for any width and any split of the row
  sum = row_sum<NT>(sum, reinterpret_cast<double*>(lds));
  const float rstd = (float)(1.0 / __builtin_sqrt(sum / a.D + (double)a.eps));
  if (a.rstd && tid == 0) a.rstd[row] = rstd;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v0 = (i * NT + tid) * 8, c = column_of<PART>(i * NT + tid, a.D);
    float w[8];
    load_weight<PART>(a.w, c, a.D, a.wdt, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[i][e] = f[i][e] * rstd * w[e];
    if (!QUANT && v0 < a.D)
      store8<T, PART>(reinterpret_cast<T*>(a.y) + row * a.D + c, a.D, f[i]);
  }
  if (!QUANT) return;

  quantise_row<NT, VPT, PART>(f, row, tid, a.D, a.quant, a.group, reinterpret_cast<uint8_t*>(a.y),
                              a.scale, lds);
}

// With u = h rstd (the unit row) and du = w dy:
//   dh = rstd (du - u mean(du u)) + (gradient of the stored stream),
//   dw = sum_rows dy u.
// A block walks rows blockIdx.x, + blocks, ... with dw in registers and
// leaves its sum in `part`; norm_reduce_kernel adds the blocks in order.
// Memory bounds it up to 8192 columns: 8192 rows of 4096 bf16 columns take 55
// us for 285 MB (5.2 TB/s).  Beyond, registers do, since five arrays of the row
// are held in them: 32 MB of columns with a bf16 residual take 84 us at 16,384
// columns (3.2 TB/s; up to 45 spilled registers at one wave per SIMD), 351 at
// 32,768 (0.8; 219 to 312) and 870 at 65,536 (0.3; 620 to 747).
template <typename T, typename RES, int NT, int VPT, bool PART>
__global__ __launch_bounds__(block_of<NT>()) void norm_bwd_kernel(NormArgs a) {
  constexpr bool kRes = !std::is_void<RES>::value;
  typedef typename std::conditional<kRes, RES, T>::type R;
  __shared__ float lds[16];
  __shared__ float wsum[NT == 64 ? 4 : 1][NT == 64 ? 64 * 8 * VPT : 1];
  const int tid = NT == 64 ? (threadIdx.x & 63) : threadIdx.x;
  const int q = NT == 64 ? (threadIdx.x >> 6) : 0;
  constexpr int RPB = NT == 64 ? 4 : 1;
  float dw[VPT][8], w[VPT][8];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[i][e] = 0.f;
    load_weight<PART>(a.w, column_of<PART>(i * NT + tid, a.D), a.D, a.wdt, w[i]);
  }
  for (int64_t row = (int64_t)blockIdx.x * RPB + q; row < a.rows; row += (int64_t)a.blocks * RPB) {
    const R* h = reinterpret_cast<const R*>(a.x) + row * a.x_stride;
    const T* dy = reinterpret_cast<const T*>(a.dy) + row * a.D;
    const R* dh = reinterpret_cast<const R*>(a.dh) + row * a.D;
    float u[VPT][8], du[VPT][8], g[VPT][8];
    const float rstd = a.rstd[row];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = column_of<PART>(i * NT + tid, a.D);
      load8<R, PART>(h + c, a.D, u[i]);
      load8<T, PART>(dy + c, a.D, du[i]);
      if (kRes && a.dh) {
        load8<R, PART>(dh + c, a.D, g[i]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) g[i][e] = 0.f;
      }
    }
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v0 = (i * NT + tid) * 8, c = column_of<PART>(i * NT + tid, a.D);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        u[i][e] *= rstd;
        dw[i][e] += du[i][e] * u[i][e];
        du[i][e] *= w[i][e];
        dot += c + e >= v0 ? du[i][e] * u[i][e] : 0.f;
      }
    }
    dot = row_reduce<NT, false>(dot, lds) / (float)a.D;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v0 = (i * NT + tid) * 8, c = column_of<PART>(i * NT + tid, a.D);
      if (v0 < a.D) {
#pragma unroll
        for (int e = 0; e < 8; ++e) g[i][e] += rstd * (du[i][e] - u[i][e] * dot);
        store8<T, PART>(reinterpret_cast<T*>(a.dx) + row * a.D + c, a.D, g[i]);
        if (kRes && a.dres)
          store8<R, PART>(reinterpret_cast<R*>(a.dres) + row * a.D + c, a.D, g[i]);
      }
    }
  }
  float* part = a.part + (int64_t)blockIdx.x * a.D;
  if (NT > 64) {
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      if ((i * NT + tid) * 8 < a.D)
        store8<float, PART>(part + column_of<PART>(i * NT + tid, a.D), a.D, dw[i]);
  } else {
    // columns of the block's four rows, each at its vector's place
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) wsum[q][(i * 64 + tid) * 8 + e] = dw[i][e];
    __syncthreads();
    for (int k = threadIdx.x; k < ((a.D + 7) / 8) * 8; k += 256) {
      const int c = column_of<PART>(k / 8, a.D) + k % 8;
      if (c < a.D)
        part[c] = (wsum[0][k] + wsum[NT == 64 ? 1 : 0][k]) +
                  (wsum[NT == 64 ? 2 : 0][k] + wsum[NT == 64 ? 3 : 0][k]);
    }
  }
}

// dweight over the blocks: 16 columns by 16 shares of the blocks.  6 us for
// 4096 columns and 1024 blocks, mostly latency.
__global__ __launch_bounds__(256) void norm_reduce_kernel(const float* part, int blocks, int D,
                                                          void* dw, int wdt) {
  __shared__ float red[16][17];
  const int l = threadIdx.x & 15, q = threadIdx.x >> 4;
  const int c = blockIdx.x * 16 + l;
  float s = 0.f;
  if (c < D)
#pragma unroll 8
    for (int b = q; b < blocks; b += 16) s += part[(int64_t)b * D + c];
  red[q][l] = s;
  __syncthreads();
  if (q == 0 && c < D) {
    s = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) s += red[i][l];
    store_scalar(dw, c, wdt, s);
  }
}

// Threads per row and 8-element steps per thread, by width: one wave up to
// 1024 columns, 256 threads up to 16384, 1024 up to 65536.  One wave for wider
// rows would need no barriers but holds more of a row per thread: 16384 rows
// of 4096 columns to e4m3 take 125 us with one wave a row and 88 us with 256
// threads, 8192 rows with a residual 54 and 47 us.  Beyond 16384 columns 256
// threads would hold more than 64 elements each of a row; with 1024, which leave
// a thread 128 registers, the forward spills at most 23 (8-bit outputs and fp32
// beyond 32,768 columns), the gradient many (see there).
template <typename F>
void by_width(int D, F f) {
  const int nv = (D + 7) / 8;
  const std::false_type whole;
#define GDR_W(NT, VPT) \
  if (nv <= NT * VPT)  \
  return f(std::integral_constant<int, NT>(), std::integral_constant<int, VPT>(), whole)
  if (D < 8)
    return f(std::integral_constant<int, 64>(), std::integral_constant<int, 1>(), std::true_type());
  GDR_W(64, 1);
  GDR_W(64, 2);
  GDR_W(256, 1);
  GDR_W(256, 2);
  GDR_W(256, 4);
  GDR_W(256, 8);
  GDR_W(1024, 4);
  GDR_W(1024, 8);
#undef GDR_W
}

// The input's and the residual's types (a pointer to either, for void).
template <typename F>
void by_type(const gdr_norm_problem* p, F f) {
  auto res = [&](auto t) {
    using T = decltype(t);
    if (!p->has_residual) f(t, (void*)nullptr);
    else if (p->res_dtype == GDR_FP32) f(t, (float*)nullptr);
    else f(t, (T*)nullptr);
  };
  if (p->dtype == GDR_BF16) res(__bf16());
  else if (p->dtype == GDR_FP16) res(_Float16());
  else res(float());
}

int bwd_blocks(const gdr_norm_problem* p) {
  // the partial weight gradients cost blocks * D * 8 bytes of traffic, the
  // rows rows * D * (6 or more): at least 8 rows a block, at most 1024 blocks
  const int rpb = p->D <= 1024 ? 4 : 1;
  const int64_t want = ((int64_t)p->rows + 8 * rpb - 1) / (8 * rpb);
  return (int)std::max<int64_t>(1, std::min<int64_t>(want, 1024));
}

NormArgs args_of(const gdr_norm_problem* p) {
  NormArgs a{};
  a.x_stride = p->x_stride;
  a.rows = p->rows;
  a.D = p->D;
  a.wdt = (int)p->w_dtype;
  a.group = p->group_size;
  a.eps = p->eps;
  return a;
}

}  // namespace

void launch_reduce_rows(const float* part, int rows, int cols, void* out, int dtype,
                        hipStream_t st) {
  GDR_LAUNCH("norm_reduce", norm_reduce_kernel, dim3((cols + 15) / 16), dim3(256), st, part, rows,
             cols, out, dtype);
}

gdr_status launch_norm_fwd(const gdr_norm_problem* p, const void* x, const void* res,
                           const void* weight, void* y, void* scale, void* h, float* rstd,
                           hipStream_t st) {
  NormArgs a = args_of(p);
  a.x = x; a.res = res; a.w = weight; a.y = y; a.scale = reinterpret_cast<float*>(scale);
  a.h = h; a.rstd = rstd;
  a.quant = p->quant;
  by_type(p, [&](auto t, auto r) {
    by_width(p->D, [&](auto nt, auto vpt, auto part) {
      using T = decltype(t);
      using R = typename std::remove_pointer<decltype(r)>::type;
      constexpr int NT = nt.value, VPT = vpt.value;
      const dim3 grid((unsigned)(NT == 64 ? (p->rows + 3) / 4 : p->rows));
      const dim3 block(block_of<NT>());
      if (p->quant)
        GDR_LAUNCH("norm_fwd", (norm_fwd_kernel<T, R, true, NT, VPT, part.value>), grid, block, st, a);
      else
        GDR_LAUNCH("norm_fwd", (norm_fwd_kernel<T, R, false, NT, VPT, part.value>), grid, block, st, a);
    });
  });
  return launch_status("norm_fwd");
}

size_t norm_bwd_workspace(const gdr_norm_problem* p) {
  return align256((size_t)bwd_blocks(p) * p->D * sizeof(float));
}

gdr_status launch_norm_bwd(const gdr_norm_problem* p, const void* dy, const void* h,
                           const void* weight, const float* rstd, const void* dh_out, void* dx,
                           void* dres, void* dw, void* ws, hipStream_t st) {
  NormArgs a = args_of(p);
  // with a residual the normalised stream is h, in its type and contiguous
  a.x = h; a.w = weight; a.dy = dy; a.dh = dh_out; a.rstd = const_cast<float*>(rstd);
  a.dx = dx; a.dres = dres; a.part = reinterpret_cast<float*>(ws);
  a.blocks = bwd_blocks(p);
  if (p->has_residual) a.x_stride = p->D;
  by_type(p, [&](auto t, auto r) {
    by_width(p->D, [&](auto nt, auto vpt, auto part) {
      using T = decltype(t);
      using R = typename std::remove_pointer<decltype(r)>::type;
      constexpr int NT = nt.value, VPT = vpt.value;
      GDR_LAUNCH("norm_bwd", (norm_bwd_kernel<T, R, NT, VPT, part.value>), dim3(a.blocks),
                 dim3(block_of<NT>()), st, a);
    });
  });
  launch_reduce_rows(a.part, a.blocks, p->D, dw, (int)p->w_dtype, st);
  return launch_status("norm_bwd");
}

}  // namespace gdr

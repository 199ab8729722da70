// rms_norm.hip -- root-mean-square norm with the residual's addition, on
// gfx950: h = x + r (rounded to the residual's type, the stream that the next
// layer adds to), y = w h / sqrt(mean h^2 + eps), y in the input's type or in
// 8 bits with a scale per row or per 128 columns; and its gradient.
//
// Memory bounds it: every operand is touched once.  A row stays in the
// registers of its threads, 8 elements each per step, from its load through
// the sum of squares to the store.  Where the width is no multiple of 8 the
// row's last vector is moved back to end with the row: loads need no bounds,
// the elements that it repeats are left out of sums and maxima, and its
// stores repeat their bits.
#include <algorithm>
#include <type_traits>

#include "ops_device.h"
#include "ops_internal.h"

namespace gdr {

namespace {

constexpr float kTinyScale = 1.1754943508222875e-38f;  // 2^-126

// Where vector vi of a row starts (PART: rows of fewer than 8 elements).
template <bool PART>
__device__ __forceinline__ int column_of(int vi, int D) {
  return PART ? 0 : min(vi * 8, D - 8);
}

// Eight consecutive elements of any of the types, in fp32.
template <typename T, bool PART>
__device__ __forceinline__ void load8(const T* p, int D, float* f) {
  constexpr int V = Vec<T>::n;
#pragma unroll
  for (int k = 0; k < 8; k += V) {
    Vec<T> v;
    if (PART) v.load_part(p + k, max(0, D - k));
    else v.load(p + k);
#pragma unroll
    for (int e = 0; e < V; ++e) f[k + e] = to_f(v.v[e]);
  }
}
template <typename T, bool PART>
__device__ __forceinline__ void store8(T* p, int D, const float* f) {
  constexpr int V = Vec<T>::n;
#pragma unroll
  for (int k = 0; k < 8; k += V) {
    Vec<T> v;
#pragma unroll
    for (int e = 0; e < V; ++e) v.v[e] = from_f<T>(f[k + e]);
    if (PART) v.store_part(p + k, max(0, D - k));
    else v.store(p + k);
  }
}
template <bool PART>
__device__ __forceinline__ void load_weight(const void* p, int c, int D, int dtype, float* f) {
  if (dtype == GDR_BF16) load8<__bf16, PART>(reinterpret_cast<const __bf16*>(p) + c, D, f);
  else if (dtype == GDR_FP16) load8<_Float16, PART>(reinterpret_cast<const _Float16*>(p) + c, D, f);
  else load8<float, PART>(reinterpret_cast<const float*>(p) + c, D, f);
}

// Largest magnitude that keeps a NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
  return (a > b || a != a) ? a : b;
}
// over the 16 lanes of a lane group; over the wave
__device__ __forceinline__ float max16(float v) {
  v = max_nan(v, dpp_mov<0xB1>(v));
  v = max_nan(v, dpp_mov<0x4E>(v));
  v = max_nan(v, dpp_mov<0x141>(v));
  return max_nan(v, dpp_mov<0x140>(v));
}
__device__ __forceinline__ float wave_max(float v) {
  v = max16(v);
  v = max_nan(v, __shfl_xor(v, 16, 64));
  return max_nan(v, __shfl_xor(v, 32, 64));
}

// Sum (or largest) of v over the NT threads of a row; every thread of the
// row gets the same bits.  Rows of one wave share a block, four at a time.
template <int NT, bool MAX>
__device__ __forceinline__ float row_reduce(float v, float* lds) {
  v = MAX ? wave_max(v) : wave_sum(v);
  if (NT == 64) return v;
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = lds[0];
#pragma unroll
  for (int i = 1; i < NT / 64; ++i) s = MAX ? max_nan(s, lds[i]) : s + lds[i];
  return s;
}

// The same for a sum in 64 bits.
template <int CTRL>
__device__ __forceinline__ double dpp_mov2(double v) {
  const uint2 u = __builtin_bit_cast(uint2, v);
  const uint2 r{__builtin_bit_cast(uint32_t, dpp_mov<CTRL>(__builtin_bit_cast(float, u.x))),
                __builtin_bit_cast(uint32_t, dpp_mov<CTRL>(__builtin_bit_cast(float, u.y)))};
  return __builtin_bit_cast(double, r);
}
template <int NT>
__device__ __forceinline__ double row_sum(double v, double* lds) {
  v += dpp_mov2<0xB1>(v);
  v += dpp_mov2<0x4E>(v);
  v += dpp_mov2<0x141>(v);
  v += dpp_mov2<0x140>(v);
  v += __shfl_xor(v, 16, 64);
  v += __shfl_xor(v, 32, 64);
  if (NT == 64) return v;
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  double s = lds[0];
#pragma unroll
  for (int i = 1; i < NT / 64; ++i) s += lds[i];
  return s;
}

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

__device__ __forceinline__ uint32_t pack_fp8(float a, float b, float c, float d) {
  int r = 0;
  r = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, r, false);
  r = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, r, true);
  return (uint32_t)r;
}
__device__ __forceinline__ uint32_t int8_of(float v) {
  return v != v ? 0u : (uint32_t)(int)rintf(v) & 0xffu;
}

// Threads of a block: one row of NT threads, or (NT == 64) four rows of one
// wave each.
template <int NT>
constexpr int block_of() {
  return NT == 64 ? 256 : NT;
}

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

  // 8 bits: scale = max |y| / top, at least 2^-126 so that rows of zeros stay
  // zeros; the quotient is rounded to nearest even
  const bool fp8 = a.quant == 1;
  const float top = fp8 ? 448.f : 127.f;
  const int ngroups = (a.D + 127) / 128;
  float row_scale = 0.f;
  if (a.group == 0) {
    float mx = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) mx = max_nan(mx, fabsf(f[i][e]));
    mx = row_reduce<NT, true>(mx, lds) / top;
    row_scale = mx < kTinyScale ? kTinyScale : mx;
    if (tid == 0) a.scale[row] = row_scale;
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v0 = (i * NT + tid) * 8, c = column_of<PART>(i * NT + tid, a.D);
    float s = row_scale;
    if (a.group) {  // 16 consecutive lanes hold a group's 128 columns
      float mx = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) mx = c + e >= v0 ? max_nan(mx, fabsf(f[i][e])) : mx;
      mx = max16(mx) / top;
      s = mx < kTinyScale ? kTinyScale : mx;
      if ((tid & 15) == 0 && v0 < a.D) a.scale[row * ngroups + v0 / 128] = s;
    }
    if (v0 < a.D) {
      float q[8];
      // (an infinite scale leaves the product's 0 or NaN as they are)
      const float inv = 1.f / s, fin = s < __builtin_inff() ? s : 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        // the product with the reciprocal may lie on the other side of a tie,
        // a whole step off in 8 bits: the residual makes it the fp32 quotient
        q[e] = f[i][e] * inv;
        q[e] = __builtin_fmaf(__builtin_fmaf(-q[e], fin, f[i][e]), inv, q[e]);
        // a NaN passes both comparisons
        q[e] = q[e] > top ? top : q[e] < -top ? -top : q[e];
      }
      uint32_t b[2];
      if (fp8) {
        b[0] = pack_fp8(q[0], q[1], q[2], q[3]);
        b[1] = pack_fp8(q[4], q[5], q[6], q[7]);
      } else {
#pragma unroll
        for (int k = 0; k < 2; ++k)
          b[k] = int8_of(q[4 * k]) | int8_of(q[4 * k + 1]) << 8 | int8_of(q[4 * k + 2]) << 16 |
                 int8_of(q[4 * k + 3]) << 24;
      }
      uint8_t* y = reinterpret_cast<uint8_t*>(a.y) + row * a.D + c;
      if (!PART && c == v0) {
        struct __attribute__((packed, aligned(1))) Raw {
          uint32_t u[2];
        };
        *reinterpret_cast<Raw*>(y) = Raw{{b[0], b[1]}};
      } else {  // what the vector repeats may belong to another scale
        for (int e = v0 - c; e < min(8, a.D); ++e) y[e] = (uint8_t)(b[e >> 2] >> (8 * (e & 3)));
      }
    }
  }
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
  GDR_LAUNCH("norm_reduce", norm_reduce_kernel, dim3((p->D + 15) / 16), dim3(256), st, a.part,
             a.blocks, p->D, dw, (int)p->w_dtype);
  return launch_status("norm_bwd");
}

}  // namespace gdr

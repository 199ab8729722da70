// rms_norm.hip -- root-mean-square norm with the residual's addition, on
// gfx950: h = x + r (rounded to the residual's type, the stream that the next
// layer adds to), y = w h / sqrt(mean h^2 + eps), y in the input's type or in
// 8 bits with a scale per row or per 128 columns; and its gradient.
//
// Memory bounds it: every operand is touched once.  A row stays in the
// registers of its threads (16 to 1024 threads by width, 8 elements each per
// step) from its load through the sum of squares to the store.
#include <algorithm>
#include <type_traits>

#include "ops_device.h"
#include "ops_internal.h"

namespace gdr {

namespace {

constexpr float kTinyScale = 1.1754943508222875e-38f;  // 2^-126

// Eight consecutive elements of any of the types, in fp32.
template <typename T>
__device__ __forceinline__ void load8(const T* p, int m, float* f) {
  constexpr int V = Vec<T>::n;
#pragma unroll
  for (int k = 0; k < 8; k += V) {
    Vec<T> v;
    v.load_part(p + k, m - k);
#pragma unroll
    for (int e = 0; e < V; ++e) f[k + e] = to_f(v.v[e]);
  }
}
template <typename T>
__device__ __forceinline__ void store8(T* p, int m, const float* f) {
  constexpr int V = Vec<T>::n;
#pragma unroll
  for (int k = 0; k < 8; k += V) {
    Vec<T> v;
#pragma unroll
    for (int e = 0; e < V; ++e) v.v[e] = from_f<T>(f[k + e]);
    v.store_part(p + k, m - k);
  }
}
__device__ __forceinline__ void load8_any(const void* p, int64_t i, int m, int dtype, float* f) {
  if (dtype == GDR_BF16) load8(reinterpret_cast<const __bf16*>(p) + i, m, f);
  else if (dtype == GDR_FP16) load8(reinterpret_cast<const _Float16*>(p) + i, m, f);
  else load8(reinterpret_cast<const float*>(p) + i, m, f);
}
__device__ __forceinline__ void store8_any(void* p, int64_t i, int m, int dtype, const float* f) {
  if (dtype == GDR_BF16) store8(reinterpret_cast<__bf16*>(p) + i, m, f);
  else if (dtype == GDR_FP16) store8(reinterpret_cast<_Float16*>(p) + i, m, f);
  else store8(reinterpret_cast<float*>(p) + i, m, f);
}

// Largest magnitude that keeps a NaN.
__device__ __forceinline__ float max_nan(float a, float b) {
  return (a > b || a != a) ? a : b;
}

// Sum (or largest) of v over the NT threads of a row; every thread of the
// row gets the same bits.  Rows narrower than a wave's worth share a block,
// one wave each.
template <int NT, bool MAX>
__device__ __forceinline__ float row_reduce(float v, float* lds) {
  if (MAX) {
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) v = max_nan(v, __shfl_xor(v, o, 64));
  } else {
    v = wave_sum(v);
  }
  if (NT == 64) return v;
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  float s = lds[0];
#pragma unroll
  for (int i = 1; i < NT / 64; ++i) s = MAX ? max_nan(s, lds[i]) : s + lds[i];
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
  int rows, D, xdt, rdt, wdt, group;
  float eps;
  // backward
  const void* dy;
  const void* dh;      // nullable: the gradient of the stored stream
  void* dx;
  void* dres;          // nullable
  float* part;         // [blocks][D]
  int blocks;
};

enum { OUT_SAME = 0, OUT_FP8 = 1, OUT_INT8 = 2 };

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

template <typename T, int NT, int VPT, int OUT>
__global__ __launch_bounds__(block_of<NT>()) void norm_fwd_kernel(NormArgs a) {
  __shared__ float lds[16];
  const int tid = NT == 64 ? (threadIdx.x & 63) : threadIdx.x;
  const int64_t row = NT == 64 ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6) : (int64_t)blockIdx.x;
  if (row >= a.rows) return;  // a whole wave; the barriers below are for NT > 64 only
  const T* x = reinterpret_cast<const T*>(a.x) + row * a.x_stride;
  float f[VPT][8];
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (i * NT + tid) * 8;
    if (c < a.D) {
      load8(x + c, a.D - c, f[i]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) f[i][e] = 0.f;
    }
  }
  if (a.res) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (i * NT + tid) * 8;
      if (c < a.D) {
        float r[8];
        load8_any(a.res, row * a.D + c, a.D - c, a.rdt, r);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          // the norm is of the stored stream, so that the gradient, which
          // reads it, is the gradient of what was computed
          const float s = f[i][e] + r[e];
          f[i][e] = a.rdt == GDR_FP32 ? s : a.rdt == GDR_BF16 ? (float)(__bf16)s : (float)(_Float16)s;
        }
        store8_any(a.h, row * a.D + c, a.D - c, a.rdt, f[i]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) ss += f[i][e] * f[i][e];
  ss = row_reduce<NT, false>(ss, lds);
  const float rstd = 1.f / sqrtf(ss / (float)a.D + a.eps);
  if (a.rstd && tid == 0) a.rstd[row] = rstd;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (i * NT + tid) * 8;
    if (c < a.D) {
      float w[8];
      load8_any(a.w, c, a.D - c, a.wdt, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[i][e] = f[i][e] * rstd * w[e];
      if (OUT == OUT_SAME) store8(reinterpret_cast<T*>(a.y) + row * a.D + c, a.D - c, f[i]);
    }
  }
  if (OUT == OUT_SAME) return;

  // 8 bits: scale = max |y| / top, at least 2^-126 so that rows of zeros stay
  // zeros; the quotient is rounded to nearest even
  const float top = OUT == OUT_FP8 ? 448.f : 127.f;
  const int ngroups = (a.D + 127) / 128;
  float row_scale = 0.f;
  if (a.group == 0) {
    float mx = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) mx = max_nan(mx, fabsf(f[i][e]));
    mx = row_reduce<NT, true>(mx, lds + 0) / top;
    row_scale = mx < kTinyScale ? kTinyScale : mx;
    if (tid == 0) a.scale[row] = row_scale;
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (i * NT + tid) * 8;
    float s = row_scale;
    if (a.group) {  // 16 consecutive lanes hold a group's 128 columns
      float mx = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) mx = max_nan(mx, fabsf(f[i][e]));
#pragma unroll
      for (int o = 1; o < 16; o <<= 1) mx = max_nan(mx, __shfl_xor(mx, o, 64));
      mx /= top;
      s = mx < kTinyScale ? kTinyScale : mx;
      if ((tid & 15) == 0 && c < a.D) a.scale[row * ngroups + c / 128] = s;
    }
    if (c < a.D) {
      float q[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        q[e] = f[i][e] / s;
        // a NaN passes both comparisons
        q[e] = q[e] > top ? top : q[e] < -top ? -top : q[e];
      }
      uint32_t b[2];
      if (OUT == OUT_FP8) {
        b[0] = pack_fp8(q[0], q[1], q[2], q[3]);
        b[1] = pack_fp8(q[4], q[5], q[6], q[7]);
      } else {
#pragma unroll
        for (int k = 0; k < 2; ++k)
          b[k] = int8_of(q[4 * k]) | int8_of(q[4 * k + 1]) << 8 | int8_of(q[4 * k + 2]) << 16 |
                 int8_of(q[4 * k + 3]) << 24;
      }
      uint8_t* y = reinterpret_cast<uint8_t*>(a.y) + row * a.D + c;
      if (c + 8 <= a.D) {
        struct __attribute__((packed, aligned(1))) Raw {
          uint32_t u[2];
        };
        *reinterpret_cast<Raw*>(y) = Raw{{b[0], b[1]}};
      } else {
        for (int e = 0; e < a.D - c; ++e) y[e] = (uint8_t)(b[e >> 2] >> (8 * (e & 3)));
      }
    }
  }
}

// With u = h rstd (the unit row) and du = w dy:
//   dh = rstd (du - u mean(du u)) + (gradient of the stored stream),
//   dw = sum_rows dy u.
// A block walks rows blockIdx.x, + blocks, ... with dw in registers and
// leaves its sum in `part`; norm_reduce_kernel adds the blocks in order.
template <typename T, int NT, int VPT>
__global__ __launch_bounds__(block_of<NT>()) void norm_bwd_kernel(NormArgs a) {
  __shared__ float lds[16];
  __shared__ float wsum[NT == 64 ? 4 : 1][NT == 64 ? 64 * 8 * VPT : 1];
  const int tid = NT == 64 ? (threadIdx.x & 63) : threadIdx.x;
  const int q = NT == 64 ? (threadIdx.x >> 6) : 0;
  constexpr int RPB = NT == 64 ? 4 : 1;
  float dw[VPT][8], w[VPT][8];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = (i * NT + tid) * 8;
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[i][e] = w[i][e] = 0.f;
    if (c < a.D) load8_any(a.w, c, a.D - c, a.wdt, w[i]);
  }
  for (int64_t row = (int64_t)blockIdx.x * RPB + q; row < a.rows; row += (int64_t)a.blocks * RPB) {
    float u[VPT][8], du[VPT][8];
    const float rstd = a.rstd[row];
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (i * NT + tid) * 8;
      if (c < a.D) {
        load8_any(a.x, row * a.x_stride + c, a.D - c, a.xdt, u[i]);
        load8(reinterpret_cast<const T*>(a.dy) + row * a.D + c, a.D - c, du[i]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) u[i][e] = du[i][e] = 0.f;
      }
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        u[i][e] *= rstd;
        dw[i][e] += du[i][e] * u[i][e];
        du[i][e] *= w[i][e];
        dot += du[i][e] * u[i][e];
      }
    dot = row_reduce<NT, false>(dot, lds) / (float)a.D;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (i * NT + tid) * 8;
      if (c < a.D) {
        float g[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] = 0.f;
        if (a.dh) load8_any(a.dh, row * a.D + c, a.D - c, a.rdt, g);
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] += rstd * (du[i][e] - u[i][e] * dot);
        store8(reinterpret_cast<T*>(a.dx) + row * a.D + c, a.D - c, g);
        if (a.dres) store8_any(a.dres, row * a.D + c, a.D - c, a.rdt, g);
      }
    }
  }
  float* part = a.part + (int64_t)blockIdx.x * a.D;
  if (NT > 64) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = (i * NT + tid) * 8;
      if (c < a.D) store8(part + c, a.D - c, dw[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) wsum[q][(i * 64 + tid) * 8 + e] = dw[i][e];
    __syncthreads();
    for (int c = threadIdx.x; c < a.D; c += 256)
      part[c] = (wsum[0][c] + wsum[NT == 64 ? 1 : 0][c]) +
                (wsum[NT == 64 ? 2 : 0][c] + wsum[NT == 64 ? 3 : 0][c]);
  }
}

__global__ __launch_bounds__(256) void norm_reduce_kernel(const float* part, int blocks, int D,
                                                          void* dw, int wdt) {
  __shared__ float red[4][64];
  const int l = threadIdx.x & 63, q = threadIdx.x >> 6;
  const int c = blockIdx.x * 64 + l;
  float s = 0.f;
  if (c < D)
#pragma unroll 8
    for (int b = q; b < blocks; b += 4) s += part[(int64_t)b * D + c];
  red[q][l] = s;
  __syncthreads();
  if (q == 0 && c < D)
    store_scalar(dw, c, wdt, (red[0][l] + red[1][l]) + (red[2][l] + red[3][l]));
}

// Threads per row and 8-element steps per thread, by width: one wave up to
// 1024 columns, then 256 threads up to 16384, 1024 up to 65536.
template <typename F>
void by_width(int D, F f) {
  const int nv = (D + 7) / 8;
  auto go = [&](auto nt, auto vpt) { f(nt, vpt); };
#define GDR_W(NT, VPT) \
  if (nv <= NT * VPT) return go(std::integral_constant<int, NT>(), std::integral_constant<int, VPT>())
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

template <typename F>
void by_type(const gdr_norm_problem* p, F f) {
  if (p->dtype == GDR_BF16) f(__bf16());
  else if (p->dtype == GDR_FP16) f(_Float16());
  else f(float());
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
  a.xdt = (int)p->dtype;
  a.rdt = (int)p->res_dtype;
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
  by_type(p, [&](auto t) {
    by_width(p->D, [&](auto nt, auto vpt) {
      using T = decltype(t);
      constexpr int NT = nt.value, VPT = vpt.value;
      const dim3 grid((unsigned)(NT == 64 ? (p->rows + 3) / 4 : p->rows));
      const dim3 block(block_of<NT>());
      if (p->quant == 0)
        GDR_LAUNCH("norm_fwd", (norm_fwd_kernel<T, NT, VPT, OUT_SAME>), grid, block, st, a);
      else if (p->quant == 1)
        GDR_LAUNCH("norm_fwd", (norm_fwd_kernel<T, NT, VPT, OUT_FP8>), grid, block, st, a);
      else
        GDR_LAUNCH("norm_fwd", (norm_fwd_kernel<T, NT, VPT, OUT_INT8>), grid, block, st, a);
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
  if (p->has_residual) {
    a.xdt = (int)p->res_dtype;
    a.x_stride = p->D;
  }
  by_type(p, [&](auto t) {
    by_width(p->D, [&](auto nt, auto vpt) {
      using T = decltype(t);
      constexpr int NT = nt.value, VPT = vpt.value;
      GDR_LAUNCH("norm_bwd", (norm_bwd_kernel<T, NT, VPT>), dim3(a.blocks), dim3(block_of<NT>()),
                 st, a);
    });
  });
  GDR_LAUNCH("norm_reduce", norm_reduce_kernel, dim3((p->D + 63) / 64), dim3(256), st, a.part,
             a.blocks, p->D, dw, (int)p->w_dtype);
  return launch_status("norm_bwd");
}

}  // namespace gdr

// sandwich_norm.hip -- from one block to the next on gfx950: the norm of a
// block's output, its gate, the residual scale, the residual's addition and
// the next block's norm in one pass,
//   n = w1 u(x)  (x without w1),   h = residual + alpha s act(g) n,
//   y = w2 u(h),                   u(v) = v / sqrt(mean v^2 + eps)
// with h rounded to the residual's type before it is normalised; y in the
// input's type or in 8 bits; and the gradient.
//
// Memory bounds it: a row of every operand stays in the registers of the row's
// threads from its load to its stores, so each is touched once.
#include <algorithm>

#include "norm_device.h"

namespace gdr {

namespace {

struct SandwichArgs {
  const void* x;
  const void* res;
  const void* gate;    // nullable
  const void* post;    // w1, nullable
  const void* scale;   // s, nullable
  const void* pre;     // w2
  void* y;
  float* q_scale;
  void* h;
  float* rstd_x;       // nullable in the forward
  float* rstd_h;
  int64_t x_stride, gate_stride;
  int rows, D, wdt, act, quant, group;
  float eps, alpha;
  // backward
  const void* dy;
  const void* dh;      // nullable
  void* dx;
  void* dres;
  void* dgate;
  float* part;         // [2][blocks][D]: dw2, and what dw1 and ds come from
  int blocks;
};

// One over the root of the row's mean square, in 64 bits as the norm without a
// gate has it.  `v0` excludes what a moved-back vector repeats.
template <int NT, int VPT, bool PART>
__device__ __forceinline__ float row_rstd(const float (&f)[VPT][8], int tid, int D, float eps,
                                          float* lds) {
  const int nt = row_threads<NT>();
  double sum = 0.0;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v0 = (i * nt + tid) * 8, c = column_of<PART>(i * nt + tid, D);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const double v = c + e >= v0 ? f[i][e] : 0.f;
      sum = __builtin_fma(v, v, sum);
    }
  }
  sum = row_sum<NT>(sum, reinterpret_cast<double*>(lds));
  return inverse_root(sum / D + (double)eps);
}

// The forward.  8192 rows of 4096 bf16 columns with a gate take 72 to 75 us for 336
// MB (4.5 to 4.7 TB/s), 4099 of 5003 fp16 columns with a residual in fp32 56 us for
// 246 MB (4.4): two sums over the row one after the other.  18,062 rows of 4096 to
// int8 take 174 us for 666 MB (3.8), eight 6 us.
template <typename T, typename R, bool QUANT, int NT, int VPT, bool PART>
__global__ __launch_bounds__(block_of<NT>()) void sandwich_fwd_kernel(SandwichArgs a) {
  __shared__ __align__(8) float lds[32];
  const int tid = NT == 64 ? (threadIdx.x & 63) : threadIdx.x, nt = row_threads<NT>();
  const int64_t row = NT == 64 ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6) : (int64_t)blockIdx.x;
  if (row >= a.rows) return;  // a whole wave; the barriers below are for rows of a block
  const T* x = reinterpret_cast<const T*>(a.x) + row * a.x_stride;
  const T* gate = reinterpret_cast<const T*>(a.gate) + row * a.gate_stride;
  const R* res = reinterpret_cast<const R*>(a.res) + row * a.D;
  R* h = reinterpret_cast<R*>(a.h) + row * a.D;
  float f[VPT][8], r[VPT][8], g[VPT][8];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = column_of<PART>(i * nt + tid, a.D);
    load8<T, PART>(x + c, a.D, f[i]);
    load8<R, PART>(res + c, a.D, r[i]);
    if (a.gate) load8<T, PART>(gate + c, a.D, g[i]);
  }
  if (a.post) {
    const float rstd = row_rstd<NT, VPT, PART>(f, tid, a.D, a.eps, lds);
    if (a.rstd_x && tid == 0) a.rstd_x[row] = rstd;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      float w[8];
      load_weight<PART>(a.post, column_of<PART>(i * nt + tid, a.D), a.D, a.wdt, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[i][e] = f[i][e] * rstd * w[e];
    }
  }
  if (a.gate) {
    by_activation<true>(a.act, [&](auto act) {
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) f[i][e] *= gate_value<act.value>(g[i][e]);
    });
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v0 = (i * nt + tid) * 8, c = column_of<PART>(i * nt + tid, a.D);
    if (a.scale) {
      float s[8];
      load_weight<PART>(a.scale, c, a.D, a.wdt, s);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[i][e] *= s[e];
    }
    // the norm is of the stored stream, so that the gradient, which reads it,
    // is the gradient of what was computed
#pragma unroll
    for (int e = 0; e < 8; ++e)
      f[i][e] = to_f(from_f<R>(__builtin_fmaf(f[i][e], a.alpha, r[i][e])));
    if (v0 < a.D) store8<R, PART>(h + c, a.D, f[i]);
  }
  const float rstd = row_rstd<NT, VPT, PART>(f, tid, a.D, a.eps, lds);
  if (a.rstd_h && tid == 0) a.rstd_h[row] = rstd;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v0 = (i * nt + tid) * 8, c = column_of<PART>(i * nt + tid, a.D);
    float w[8];
    load_weight<PART>(a.pre, c, a.D, a.wdt, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) f[i][e] = f[i][e] * rstd * w[e];
    if (!QUANT && v0 < a.D)
      store8<T, PART>(reinterpret_cast<T*>(a.y) + row * a.D + c, a.D, f[i]);
  }
  if (QUANT)
    quantise_row<NT, VPT, PART>(f, row, tid, a.D, a.quant, a.group,
                                reinterpret_cast<uint8_t*>(a.y), a.q_scale, lds);
}

// The gradient.  With the unit rows uh of h and ux of x (x itself without w1),
// A = act(g):
//   dH = dh + rh (dy w2 - uh mean(dy w2 uh)) = dresidual,   dw2 = sum dy uh
//   P = sum dH A ux,   dw1 = alpha s P,   ds = alpha w1 P
//   dg = dH alpha s w1 ux A',   du = dH alpha s A w1
//   dx = rx (du - ux mean(du ux))     (du without w1)
// A block walks rows blockIdx.x, + blocks, ... with dw2 and P in registers and
// leaves its sums in `part`.  8192 x 4096 with a gate take 115 us for 537 MB (4.7
// TB/s): eight streams, two sums, 104 registers and so two rows of 512 threads a
// CU.  Beyond 8192 columns dw2 and P lie in LDS and some 32 registers are spilled
// (33.5 million elements: 170 us of 16,384 columns, 129 of 8192).
template <typename T, typename R, int NT, int VPT, bool PART>
__global__ __launch_bounds__(block_of<NT>(), 4) void sandwich_bwd_kernel(SandwichArgs a) {
  constexpr int RPB = NT == 64 ? 4 : 1;
  constexpr int COLS = 64 * VPT * 8;  // of a wave's row
  constexpr bool kWeights = VPT == 1;  // LDS holds them beside the rows
  __shared__ float lds[16];
  __shared__ float wsum[NT == 64 ? 4 * COLS : 1];
  const int tid = NT == 64 ? (threadIdx.x & 63) : threadIdx.x, nt = row_threads<NT>();
  const int q = NT == 64 ? (threadIdx.x >> 6) : 0;
  // w2 and alpha s w1 by columns, in fp32
  extern __shared__ __align__(16) float weights[];
  float* w2 = weights;
  float* sw1 = weights + a.D;
  if (kWeights) {
    for (int c = threadIdx.x; c < a.D; c += blockDim.x) {
      w2[c] = load_scalar(a.pre, c, a.wdt);
      float v = a.alpha;
      if (a.scale) v *= load_scalar(a.scale, c, a.wdt);
      if (a.post) v *= load_scalar(a.post, c, a.wdt);
      sw1[c] = v;
    }
    __syncthreads();
  }
  // dw2 and P: in registers, or (two steps a thread) at the thread's place in LDS
  __shared__ __align__(16) float sums[VPT == 2 ? 2 * 1024 * 2 * 8 : 1];
  float dw[kWeights ? VPT : 1][8], P[kWeights ? VPT : 1][8];
  auto kept = [&](int k, int i) { return sums + ((k * VPT + i) * 1024 + tid) * 8; };
  if (kWeights) {
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) dw[kWeights ? i : 0][e] = P[kWeights ? i : 0][e] = 0.f;
  } else {
    for (int j = 0; j < 2 * VPT; ++j)
      for (int e = 0; e < 8; ++e) kept(0, j)[e] = 0.f;
  }
  for (int64_t row = (int64_t)blockIdx.x * RPB + q; row < a.rows; row += (int64_t)a.blocks * RPB) {
    const T* x = reinterpret_cast<const T*>(a.x) + row * a.x_stride;
    const T* gate = reinterpret_cast<const T*>(a.gate) + row * a.gate_stride;
    const T* dy = reinterpret_cast<const T*>(a.dy) + row * a.D;
    const R* h = reinterpret_cast<const R*>(a.h) + row * a.D;
    const R* dh = reinterpret_cast<const R*>(a.dh) + row * a.D;
    const float rh = a.rstd_h[row], rx = a.post ? a.rstd_x[row] : 1.f;
    float u[VPT][8], d[VPT][8], g[VPT][8], ux[VPT][8], s[VPT][8];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = column_of<PART>(i * nt + tid, a.D);
      load8<R, PART>(h + c, a.D, u[i]);
      load8<T, PART>(dy + c, a.D, d[i]);
      load8<T, PART>(x + c, a.D, ux[i]);
      if (a.gate) load8<T, PART>(gate + c, a.D, s[i]);
      if (a.dh) {
        load8<R, PART>(dh + c, a.D, g[i]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) g[i][e] = 0.f;
      }
    }
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v0 = (i * nt + tid) * 8, c = column_of<PART>(i * nt + tid, a.D);
      float w[8];
      if (kWeights) load8<float, PART>(w2 + c, a.D, w);
      else load_weight<PART>(a.pre, c, a.D, a.wdt, w);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        u[i][e] *= rh;
        if (kWeights) dw[kWeights ? i : 0][e] += d[i][e] * u[i][e];
        else kept(0, i)[e] += d[i][e] * u[i][e];
        d[i][e] *= w[e];
        dot += c + e >= v0 ? d[i][e] * u[i][e] : 0.f;
      }
    }
    dot = row_reduce<NT, false>(dot, lds) / (float)a.D;
    float dot2 = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v0 = (i * nt + tid) * 8, c = column_of<PART>(i * nt + tid, a.D);
      float w[8];
      if (kWeights) {
        load8<float, PART>(sw1 + c, a.D, w);
      } else {
        float t[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) w[e] = a.alpha;
        for (int k = 0; k < 2; ++k) {
          const void* p = k ? a.post : a.scale;
          if (!p) continue;
          load_weight<PART>(p, c, a.D, a.wdt, t);
#pragma unroll
          for (int e = 0; e < 8; ++e) w[e] *= t[e];
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) g[i][e] += rh * (d[i][e] - u[i][e] * dot);
      if (v0 < a.D)
        store8<R, PART>(reinterpret_cast<R*>(a.dres) + row * a.D + c, a.D, g[i]);
      Gate t[8];
      if (a.gate) {
        by_activation<true>(a.act, [&](auto act) {
#pragma unroll
          for (int e = 0; e < 8; ++e) t[e] = gate_and_slope<act.value>(s[i][e]);
        });
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) t[e] = {1.f, 0.f};
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        ux[i][e] *= rx;
        const float b = g[i][e] * ux[i][e];
        if (kWeights) P[kWeights ? i : 0][e] += b * t[e].value;
        else kept(1, i)[e] += b * t[e].value;
        s[i][e] = b * w[e] * t[e].slope;
        d[i][e] = g[i][e] * t[e].value * w[e];
        dot2 += c + e >= v0 ? d[i][e] * ux[i][e] : 0.f;
      }
      if (a.gate && v0 < a.D)
        store8<T, PART>(reinterpret_cast<T*>(a.dgate) + row * a.D + c, a.D, s[i]);
    }
    if (a.post) {
      dot2 = row_reduce<NT, false>(dot2, lds) / (float)a.D;
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) d[i][e] = rx * (d[i][e] - ux[i][e] * dot2);
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      if ((i * nt + tid) * 8 < a.D)
        store8<T, PART>(reinterpret_cast<T*>(a.dx) + row * a.D +
                            column_of<PART>(i * nt + tid, a.D), a.D, d[i]);
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    float* part = a.part + ((int64_t)k * a.blocks + blockIdx.x) * a.D;
    if (NT == 0) {
#pragma unroll
      for (int i = 0; i < VPT; ++i)
        if ((i * nt + tid) * 8 < a.D)
          store8<float, PART>(part + column_of<PART>(i * nt + tid, a.D), a.D,
                              !kWeights ? kept(k, i) : k ? P[kWeights ? i : 0] : dw[kWeights ? i : 0]);
    } else {
      // columns of the block's four rows, each at its vector's place
      __syncthreads();
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e)
          wsum[q * COLS + (i * 64 + tid) * 8 + e] =
              k ? P[kWeights ? i : 0][e] : dw[kWeights ? i : 0][e];
      __syncthreads();
      for (int j = threadIdx.x; j < ((a.D + 7) / 8) * 8; j += 256) {
        const int c = column_of<PART>(j / 8, a.D) + j % 8;
        if (c < a.D)
          part[c] = (wsum[j] + wsum[(NT == 64 ? 1 : 0) * COLS + j]) +
                    (wsum[(NT == 64 ? 2 : 0) * COLS + j] + wsum[(NT == 64 ? 3 : 0) * COLS + j]);
      }
    }
  }
}

// The parameters' gradients over the blocks, 16 columns by 16 shares of the
// blocks: dw2 (blockIdx.y 0), and dw1 and ds from P.
__global__ __launch_bounds__(256) void sandwich_reduce_kernel(SandwichArgs a, void* dpost,
                                                              void* dscale, void* dpre) {
  __shared__ float red[16][17];
  const int l = threadIdx.x & 15, q = threadIdx.x >> 4;
  const int c = blockIdx.x * 16 + l;
  const float* part = a.part + (int64_t)blockIdx.y * a.blocks * a.D;
  float s = 0.f;
  if (c < a.D)
#pragma unroll 8
    for (int b = q; b < a.blocks; b += 16) s += part[(int64_t)b * a.D + c];
  red[q][l] = s;
  __syncthreads();
  if (q || c >= a.D) return;
  s = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) s += red[i][l];
  if (blockIdx.y == 0) {
    store_scalar(dpre, c, a.wdt, s);
    return;
  }
  s *= a.alpha;
  if (dpost) store_scalar(dpost, c, a.wdt, a.scale ? s * load_scalar(a.scale, c, a.wdt) : s);
  if (dscale) store_scalar(dscale, c, a.wdt, a.post ? s * load_scalar(a.post, c, a.wdt) : s);
}

// The input's and the residual's types.
template <typename F>
void by_type(const gdr_sandwich_norm_problem* p, F f) {
  auto res = [&](auto t) {
    if (p->res_dtype == GDR_FP32) f(t, float());
    else f(t, t);
  };
  if (p->dtype == GDR_BF16) res(__bf16());
  else if (p->dtype == GDR_FP16) res(_Float16());
  else f(float(), float());
}

// Rows of several arrays: one 8-element step a thread as far as a block reaches
// (as they were first built, the forward of 8192 x 4096 bf16 with a gate: 70 us, with
// two steps 77; the gradient 117 and, with 193 registers, 139).
template <typename F>
void by_steps(int D, F f) {
  if (D <= 8192) return by_row<1>(D, f);
  f(dim3(64 * ((D + 1023) / 1024)), 1, std::integral_constant<int, 0>(),
    std::integral_constant<int, 2>(), std::false_type());
}

int bwd_blocks(const gdr_sandwich_norm_problem* p) {
  // 4096 waves fill the card; at least 8 rows a block, against its partial sums
  int64_t blocks = 1;
  by_steps(p->D, [&](dim3 block, int rows, auto, auto, auto) {
    blocks = std::min<int64_t>(4096 * 64 / block.x, ((int64_t)p->rows + 8 * rows - 1) / (8 * rows));
  });
  return (int)std::max<int64_t>(1, blocks);
}

SandwichArgs args_of(const gdr_sandwich_norm_problem* p) {
  SandwichArgs a{};
  a.x_stride = p->x_stride;
  a.gate_stride = p->gate_stride;
  a.rows = p->rows;
  a.D = p->D;
  a.wdt = (int)p->w_dtype;
  a.act = p->activation;
  a.quant = p->quant;
  a.group = p->group_size;
  a.eps = p->eps;
  a.alpha = p->alpha;
  return a;
}

int64_t blocks_of(const gdr_sandwich_norm_problem* p, int rows) {
  return ((int64_t)p->rows + rows - 1) / rows;
}

}  // namespace

int64_t sandwich_norm_threads(const gdr_sandwich_norm_problem* p) {
  int64_t threads = 0;
  by_steps(p->D, [&](dim3 block, int rows, auto, auto, auto) {
    threads = blocks_of(p, rows) * block.x;
  });
  return threads;
}

gdr_status launch_sandwich_norm_fwd(const gdr_sandwich_norm_problem* p, const void* x,
                                    const void* residual, const void* gate, const void* post,
                                    const void* res_scale, const void* pre, void* y, float* scale,
                                    void* h, float* rstd_x, float* rstd_h, hipStream_t st) {
  SandwichArgs a = args_of(p);
  a.x = x; a.res = residual; a.gate = gate; a.post = post; a.scale = res_scale; a.pre = pre;
  a.y = y; a.q_scale = scale; a.h = h; a.rstd_x = rstd_x; a.rstd_h = rstd_h;
  by_type(p, [&](auto t, auto r) {
    using T = decltype(t);
    using R = decltype(r);
    by_steps(p->D, [&](dim3 block, int rows, auto nt, auto vpt, auto part) {
      constexpr int NT = nt.value, VPT = vpt.value;
      const dim3 grid((unsigned)blocks_of(p, rows));
      if (p->quant)
        GDR_LAUNCH("sandwich_fwd", (sandwich_fwd_kernel<T, R, true, NT, VPT, part.value>), grid,
                   block, st, a);
      else
        GDR_LAUNCH("sandwich_fwd", (sandwich_fwd_kernel<T, R, false, NT, VPT, part.value>), grid,
                   block, st, a);
    });
  });
  return launch_status("sandwich_norm_fwd");
}

size_t sandwich_norm_bwd_workspace(const gdr_sandwich_norm_problem* p) {
  return align256((size_t)2 * bwd_blocks(p) * p->D * sizeof(float));
}

gdr_status launch_sandwich_norm_bwd(const gdr_sandwich_norm_problem* p, const void* dy,
                                    const void* dh, const void* x, const void* h, const void* gate,
                                    const void* post, const void* res_scale, const void* pre,
                                    const float* rstd_x, const float* rstd_h, void* dx,
                                    void* dresidual, void* dgate, void* dpost, void* dscale,
                                    void* dpre, void* ws, hipStream_t st) {
  SandwichArgs a = args_of(p);
  a.x = x; a.gate = gate; a.post = post; a.scale = res_scale; a.pre = pre;
  a.h = const_cast<void*>(h);
  a.rstd_x = const_cast<float*>(rstd_x);
  a.rstd_h = const_cast<float*>(rstd_h);
  a.dy = dy; a.dh = dh; a.dx = dx; a.dres = dresidual; a.dgate = dgate;
  a.part = reinterpret_cast<float*>(ws);
  a.blocks = bwd_blocks(p);
  by_type(p, [&](auto t, auto r) {
    using T = decltype(t);
    using R = decltype(r);
    by_steps(p->D, [&](dim3 block, int, auto nt, auto vpt, auto part) {
      constexpr int NT = nt.value, VPT = vpt.value;
      GDR_LAUNCH_LDS("sandwich_bwd", (sandwich_bwd_kernel<T, R, NT, VPT, part.value>),
                     dim3(a.blocks), block, VPT == 1 ? 2 * p->D * sizeof(float) : 0, st, a);
    });
  });
  GDR_LAUNCH("sandwich_reduce", sandwich_reduce_kernel,
             dim3((p->D + 15) / 16, dpost || dscale ? 2 : 1), dim3(256), st, a, dpost, dscale, dpre);
  return launch_status("sandwich_norm_bwd");
}

}  // namespace gdr

// gated_norm.hip -- the root-mean-square norm of a recurrence's output with
// its gate, on gfx950: over each group of columns (a head), a = act(z),
//   norm first:  y = w u(x) a        gate first:  y = w u(x a)
// with u(v) = v / sqrt(mean v^2 + eps); y in the input's type or in 8 bits; and
// the gradient.
//
// Memory bounds it: x and z are read once and y is written once.  Two layouts
// of the same kernels:
//   lanes: groups of 8 L columns, L = 1, 2, 4 ... 64.  A row of all groups
//     lies in the registers of its threads, and L neighbouring lanes of a wave
//     hold a group, whose sum needs no barrier;
//   whole: any other width.  A group is a row of its own (blockIdx.y names the
//     group), in the registers of its threads.
// 8-bit outputs whose scale spans several groups of the second kind go through
// LDS (gated_quant_kernel).
#include <algorithm>

#include "norm_device.h"

namespace gdr {

namespace {

struct GatedArgs {
  const void* x;
  const void* z;
  const void* w;
  void* y;
  float* scale;
  float* rstd;        // [rows][groups], nullable in the forward
  int64_t x_stride, z_stride;  // elements between rows
  int rows, D;        // columns of a row
  int width;          // columns that a row's threads hold: D, or a group
  int lanes;          // lanes of a group, 0 where the threads hold one group
  int size;           // columns of a group
  int groups;         // groups of a row
  int wdt, shared;    // shared: one group's weights for all
  int gate_first, act;  // act 1: silu, 2: sigmoid
  int quant, scale_group;
  float eps;
  // backward
  const void* dy;
  void* dx;
  void* dz;
  float* part;        // [blocks][shared ? size : D], whole: [blocks][D]
  int blocks;
};

// Sum over `lanes` (a power of two) neighbouring lanes, the same bits in each.
__device__ __forceinline__ double lanes_sum(double v, int lanes) {
  if (lanes > 1) v += dpp_mov2<0xB1>(v);
  if (lanes > 2) v += dpp_mov2<0x4E>(v);
  if (lanes > 4) v += dpp_mov2<0x141>(v);
  if (lanes > 8) v += dpp_mov2<0x140>(v);
  if (lanes > 16) v += __shfl_xor(v, 16, 64);
  if (lanes > 32) v += __shfl_xor(v, 32, 64);
  return v;
}
__device__ __forceinline__ float lanes_sum(float v, int lanes) {
  if (lanes > 1) v += dpp_mov<0xB1>(v);
  if (lanes > 2) v += dpp_mov<0x4E>(v);
  if (lanes > 4) v += dpp_mov<0x141>(v);
  if (lanes > 8) v += dpp_mov<0x140>(v);
  if (lanes > 16) v += __shfl_xor(v, 16, 64);
  if (lanes > 32) v += __shfl_xor(v, 32, 64);
  return v;
}

// Where a thread's weights stand: its column, or the column within its group
// (a power of two in the lanes layout) where the groups share them.
__device__ __forceinline__ int weight_at(const GatedArgs& a, int c) {
  return a.shared && a.lanes ? c & (a.size - 1) : c;
}

// The forward.
template <typename T, bool QUANT, int NT, int VPT, bool PART>
__global__ __launch_bounds__(block_of<NT>()) void gated_fwd_kernel(GatedArgs a) {
  __shared__ __align__(8) float lds[32];
  const int tid = NT == 64 ? (threadIdx.x & 63) : threadIdx.x;
  const int64_t row = NT == 64 ? (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6) : (int64_t)blockIdx.x;
  if (row >= a.rows) return;  // a whole wave; the barriers below are for NT > 64 only
  const int g = blockIdx.y;   // the group of the whole layout
  const int64_t first = (int64_t)g * a.width;
  const T* x = reinterpret_cast<const T*>(a.x) + row * a.x_stride + first;
  const T* z = reinterpret_cast<const T*>(a.z) + row * a.z_stride + first;
  float f[VPT][8], t[VPT][8];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = column_of<PART>(i * NT + tid, a.width);
    load8<T, PART>(x + c, a.width, f[i]);
    load8<T, PART>(z + c, a.width, t[i]);
  }
  // squares, mean and root in 64 bits, as the norm without a gate has them
  double sum[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v0 = (i * NT + tid) * 8, c = column_of<PART>(i * NT + tid, a.width);
    sum[i] = 0.0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      t[i][e] = gate_of(t[i][e], a.act);
      if (a.gate_first) f[i][e] *= t[i][e];
      const double v = c + e >= v0 ? f[i][e] : 0.f;
      sum[i] = __builtin_fma(v, v, sum[i]);
    }
  }
  float rstd[VPT];
  if (a.lanes) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v0 = (i * NT + tid) * 8;
      rstd[i] = (float)(1.0 / __builtin_sqrt(lanes_sum(sum[i], a.lanes) / a.size + (double)a.eps));
      if (a.rstd && v0 < a.D && (tid & (a.lanes - 1)) == 0)
        a.rstd[row * a.groups + v0 / a.size] = rstd[i];
    }
  } else {
#pragma unroll
    for (int i = 1; i < VPT; ++i) sum[0] += sum[i];
    const double all = row_sum<NT>(sum[0], reinterpret_cast<double*>(lds));
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      rstd[i] = (float)(1.0 / __builtin_sqrt(all / a.size + (double)a.eps));
    if (a.rstd && tid == 0) a.rstd[row * a.groups + g] = rstd[0];
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v0 = (i * NT + tid) * 8, c = column_of<PART>(i * NT + tid, a.width);
    float w[8];
    load_weight<PART>(a.w, weight_at(a, c) + (a.shared ? 0 : (int)first), a.width, a.wdt, w);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      f[i][e] = f[i][e] * rstd[i] * w[e];
      if (!a.gate_first) f[i][e] *= t[i][e];
      // (past the row's end the lanes layout holds groups that are none)
      if (QUANT && a.lanes && v0 >= a.D) f[i][e] = 0.f;
    }
    if (!QUANT && v0 < a.width)
      store8<T, PART>(reinterpret_cast<T*>(a.y) + row * a.D + first + c, a.width, f[i]);
  }
  if (QUANT)
    quantise_row<NT, VPT, PART>(f, row, tid, a.D, a.quant, a.scale_group,
                                reinterpret_cast<uint8_t*>(a.y), a.scale, lds);
}

// 8-bit outputs of rows of several groups that the lanes layout does not take.
// The row's values pass through LDS between the norm, where a wave walks one
// group at a time, and the quantisation, where a thread holds 8 columns.
constexpr int kQuantCols = 16384;
template <typename T>
__global__ __launch_bounds__(256) void gated_quant_kernel(GatedArgs a) {
  __shared__ __align__(16) float val[kQuantCols];
  __shared__ float red[16];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t row = blockIdx.x;
  const T* x = reinterpret_cast<const T*>(a.x) + row * a.x_stride;
  const T* z = reinterpret_cast<const T*>(a.z) + row * a.z_stride;
  float mx = 0.f;
  for (int g = wave; g < a.groups; g += 4) {
    const int c0 = g * a.size;
    double sum = 0.0;
    for (int c = lane; c < a.size; c += 64) {
      const float s = gate_of(to_f(z[c0 + c]), a.act);
      float f = to_f(x[c0 + c]);
      if (a.gate_first) f *= s;
      sum = __builtin_fma((double)f, (double)f, sum);
      val[c0 + c] = f;
    }
    const float rstd =
        (float)(1.0 / __builtin_sqrt(lanes_sum(sum, 64) / a.size + (double)a.eps));
    for (int c = lane; c < a.size; c += 64) {
      float f = val[c0 + c] * rstd * load_scalar(a.w, a.shared ? c : c0 + c, a.wdt);
      if (!a.gate_first) f *= gate_of(to_f(z[c0 + c]), a.act);
      val[c0 + c] = f;
      mx = max_nan(mx, fabsf(f));
    }
  }
  const bool fp8 = a.quant == 1;
  const float top = fp8 ? 448.f : 127.f;
  mx = row_reduce<256, true>(mx, red) / top;  // (its barriers hand `val` over, too)
  const float row_scale = mx < kTinyScale ? kTinyScale : mx;
  if (!a.scale_group && threadIdx.x == 0) a.scale[row] = row_scale;
  uint8_t* y = reinterpret_cast<uint8_t*>(a.y) + row * a.D;
  const int scales = (a.D + 127) / 128;
  for (int c0 = threadIdx.x * 8; c0 < scales * 128; c0 += 2048) {  // whole groups of 16 lanes
    float f[8], s = row_scale;
    float big = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      f[e] = c0 + e < a.D ? val[c0 + e] : 0.f;
      big = max_nan(big, fabsf(f[e]));
    }
    if (a.scale_group) {
      big = max16(big) / top;
      s = big < kTinyScale ? kTinyScale : big;
      if ((threadIdx.x & 15) == 0) a.scale[row * scales + c0 / 128] = s;
    }
    uint32_t b[2];
    quantise8(f, s, fp8, b);
    if (c0 + 8 <= a.D) store_bytes8(y + c0, b);
    else
      for (int e = 0; e < a.D - c0; ++e) y[c0 + e] = (uint8_t)(b[e >> 2] >> (8 * (e & 3)));
  }
}

// The gradient.  norm first, with u the unit rows:
//   du = dy w a,  dx = r (du - u mean(du u)),  dz = dy w u a',  dw = sum dy u a
// gate first, with v = x a and u its unit rows:
//   du = dy w,  dv = r (du - u mean(du u)),  dx = dv a,  dz = dv x a',
//   dw = sum dy u
// A block walks rows blockIdx.x, + blocks, ... with dw in registers and leaves
// its sum in `part`, which reduce_rows_kernel adds in order.  Where the groups
// of a row share their weights the block adds up its groups first.
template <typename T, int NT, int VPT, bool PART>
__global__ __launch_bounds__(block_of<NT>()) void gated_bwd_kernel(GatedArgs a) {
  constexpr int RPB = NT == 64 ? 4 : 1;
  constexpr int COLS = NT * VPT * 8;
  constexpr int WAVES = block_of<NT>() / 64;
  __shared__ float lds[16];
  // columns of four rows, or (shared weights) each wave's group
  __shared__ float wsum[NT == 64 ? 4 * COLS : WAVES * 512];
  const int tid = NT == 64 ? (threadIdx.x & 63) : threadIdx.x;
  const int q = NT == 64 ? (threadIdx.x >> 6) : 0;
  const int g = blockIdx.y;
  const int64_t first = (int64_t)g * a.width;
  float dw[VPT][8], w[VPT][8];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = column_of<PART>(i * NT + tid, a.width);
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[i][e] = 0.f;
    load_weight<PART>(a.w, weight_at(a, c) + (a.shared ? 0 : (int)first), a.width, a.wdt, w[i]);
  }
  for (int64_t row = (int64_t)blockIdx.x * RPB + q; row < a.rows; row += (int64_t)a.blocks * RPB) {
    const T* x = reinterpret_cast<const T*>(a.x) + row * a.x_stride + first;
    const T* z = reinterpret_cast<const T*>(a.z) + row * a.z_stride + first;
    const T* dy = reinterpret_cast<const T*>(a.dy) + row * a.D + first;
    float u[VPT][8], s[VPT][8], du[VPT][8], r[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = column_of<PART>(i * NT + tid, a.width);
      load8<T, PART>(x + c, a.width, u[i]);
      load8<T, PART>(z + c, a.width, s[i]);
      load8<T, PART>(dy + c, a.width, du[i]);
      r[i] = a.rstd[row * a.groups + (a.lanes ? c / a.size : g)];
    }
    float dot[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v0 = (i * NT + tid) * 8, c = column_of<PART>(i * NT + tid, a.width);
      const bool live = !a.lanes || v0 < a.D;
      dot[i] = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float act = gate_of(s[i][e], a.act);
        const float unit = u[i][e] * r[i] * (a.gate_first ? act : 1.f);
        const float k = a.gate_first ? 1.f : act;
        if (live) dw[i][e] += du[i][e] * unit * k;
        const float d = du[i][e] * w[i][e] * k;
        dot[i] += c + e >= v0 ? d * unit : 0.f;
      }
    }
    if (a.lanes) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) dot[i] = lanes_sum(dot[i], a.lanes) / (float)a.size;
    } else {
#pragma unroll
      for (int i = 1; i < VPT; ++i) dot[0] += dot[i];
      dot[0] = row_reduce<NT, false>(dot[0], lds) / (float)a.size;
#pragma unroll
      for (int i = 1; i < VPT; ++i) dot[i] = dot[0];
    }
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v0 = (i * NT + tid) * 8, c = column_of<PART>(i * NT + tid, a.width);
      if (v0 >= a.width) continue;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const Gate t = gate_and_slope(s[i][e], a.act);
        const float xr = u[i][e] * r[i];
        if (a.gate_first) {
          const float dv = r[i] * (du[i][e] * w[i][e] - xr * t.value * dot[i]);
          s[i][e] = dv * u[i][e] * t.slope;
          u[i][e] = dv * t.value;
        } else {
          const float d = du[i][e] * w[i][e];
          s[i][e] = d * xr * t.slope;
          u[i][e] = r[i] * (d * t.value - xr * dot[i]);
        }
      }
      store8<T, PART>(reinterpret_cast<T*>(a.dx) + row * a.D + first + c, a.width, u[i]);
      store8<T, PART>(reinterpret_cast<T*>(a.dz) + row * a.D + first + c, a.width, s[i]);
    }
  }
  if (a.shared && a.lanes) {
    // over the thread's steps, the wave's groups and the block's waves
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float v = dw[0][e];
#pragma unroll
      for (int i = 1; i < VPT; ++i) v += dw[i][e];
      for (int m = a.lanes; m < 64; m *= 2) v += __shfl_xor(v, m, 64);
      const int lane = threadIdx.x & 63;
      if (lane < a.lanes) wsum[(threadIdx.x >> 6) * 512 + lane * 8 + e] = v;
    }
    __syncthreads();
    for (int k = threadIdx.x; k < a.size; k += block_of<NT>()) {
      float v = wsum[k];
#pragma unroll
      for (int i = 1; i < WAVES; ++i) v += wsum[i * 512 + k];
      a.part[(int64_t)blockIdx.x * a.size + k] = v;
    }
    return;
  }
  float* part = a.part + (int64_t)blockIdx.x * a.D + first;
  if (NT > 64) {
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      if ((i * NT + tid) * 8 < a.width)
        store8<float, PART>(part + column_of<PART>(i * NT + tid, a.width), a.width, dw[i]);
  } else {
    // columns of the block's four rows, each at its vector's place
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) wsum[q * COLS + (i * 64 + tid) * 8 + e] = dw[i][e];
    __syncthreads();
    for (int k = threadIdx.x; k < ((a.width + 7) / 8) * 8; k += 256) {
      const int c = column_of<PART>(k / 8, a.width) + k % 8;
      if (c < a.width)
        part[c] = (wsum[k] + wsum[(NT == 64 ? 1 : 0) * COLS + k]) +
                  (wsum[(NT == 64 ? 2 : 0) * COLS + k] + wsum[(NT == 64 ? 3 : 0) * COLS + k]);
    }
  }
}

// Groups of 8 L columns, L a power of two up to a wave's 64 lanes.
bool in_lanes(int size) { return size % 8 == 0 && size <= 512 && (size & (size - 1)) == 0; }

// Threads per row and 8-element steps per thread, as the norm without a gate
// has them up to its 16,384 columns.
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
#undef GDR_W
}

template <typename F>
void by_type(const gdr_gated_norm_problem* p, F f) {
  if (p->dtype == GDR_BF16) f(__bf16());
  else if (p->dtype == GDR_FP16) f(_Float16());
  else f(float());
}

GatedArgs args_of(const gdr_gated_norm_problem* p) {
  GatedArgs a{};
  a.x_stride = p->x_stride;
  a.z_stride = p->gate_stride;
  a.rows = p->rows;
  a.D = p->D;
  a.size = p->norm_size;
  a.groups = p->D / p->norm_size;
  a.lanes = in_lanes(p->norm_size) ? p->norm_size / 8 : 0;
  a.width = a.lanes ? p->D : p->norm_size;
  a.wdt = (int)p->w_dtype;
  a.shared = p->shared_weight;
  a.gate_first = p->gate_first;
  a.act = p->activation;
  a.quant = p->quant;
  a.scale_group = p->scale_group;
  a.eps = p->eps;
  return a;
}

int bwd_blocks(const GatedArgs& a) {
  // as the norm without a gate: at least 8 rows a block, at most 1024 blocks
  const int rpb = a.width <= 1024 ? 4 : 1, across = a.lanes ? 1 : a.groups;
  const int64_t want = ((int64_t)a.rows + 8 * rpb - 1) / (8 * rpb);
  return (int)std::max<int64_t>(1, std::min<int64_t>(want, std::max(1, 1024 / across)));
}

}  // namespace

gdr_status launch_gated_norm_fwd(const gdr_gated_norm_problem* p, const void* x, const void* gate,
                                 const void* weight, void* y, float* scale, float* rstd,
                                 hipStream_t st) {
  GatedArgs a = args_of(p);
  a.x = x; a.z = gate; a.w = weight; a.y = y; a.scale = scale; a.rstd = rstd;
  by_type(p, [&](auto t) {
    using T = decltype(t);
    if (p->quant && !a.lanes && a.groups > 1) {
      GDR_LAUNCH("gated_quant", gated_quant_kernel<T>, dim3(a.rows), dim3(256), st, a);
      return;
    }
    by_width(a.width, [&](auto nt, auto vpt, auto part) {
      constexpr int NT = nt.value, VPT = vpt.value;
      const dim3 grid((unsigned)(NT == 64 ? (a.rows + 3) / 4 : a.rows), a.lanes ? 1 : a.groups);
      const dim3 block(block_of<NT>());
      if (p->quant)
        GDR_LAUNCH("gated_fwd", (gated_fwd_kernel<T, true, NT, VPT, part.value>), grid, block, st, a);
      else
        GDR_LAUNCH("gated_fwd", (gated_fwd_kernel<T, false, NT, VPT, part.value>), grid, block, st, a);
    });
  });
  return launch_status("gated_norm_fwd");
}

size_t gated_norm_bwd_workspace(const gdr_gated_norm_problem* p) {
  const GatedArgs a = args_of(p);
  return align256((size_t)bwd_blocks(a) * a.D * sizeof(float));
}

gdr_status launch_gated_norm_bwd(const gdr_gated_norm_problem* p, const void* dy, const void* x,
                                 const void* gate, const void* weight, const float* rstd, void* dx,
                                 void* dgate, void* dweight, void* ws, hipStream_t st) {
  GatedArgs a = args_of(p);
  a.x = x; a.z = gate; a.w = weight; a.rstd = const_cast<float*>(rstd);
  a.dy = dy; a.dx = dx; a.dz = dgate;
  a.part = reinterpret_cast<float*>(ws);
  a.blocks = bwd_blocks(a);
  by_type(p, [&](auto t) {
    using T = decltype(t);
    by_width(a.width, [&](auto nt, auto vpt, auto part) {
      constexpr int NT = nt.value, VPT = vpt.value;
      GDR_LAUNCH("gated_bwd", (gated_bwd_kernel<T, NT, VPT, part.value>),
                 dim3(a.blocks, a.lanes ? 1 : a.groups), dim3(block_of<NT>()), st, a);
    });
  });
  // [blocks][D] is [blocks * groups][size] where the groups share their weights
  const int cols = a.shared ? a.size : a.D;
  const int rows = a.shared && !a.lanes ? a.blocks * a.groups : a.blocks;
  launch_reduce_rows(a.part, rows, cols, dweight, a.wdt, st);
  return launch_status("gated_norm_bwd");
}

}  // namespace gdr

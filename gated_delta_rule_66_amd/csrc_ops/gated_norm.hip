// gated_norm.hip -- the root-mean-square norm of a recurrence's output with
// its gate, on gfx950: over each group of columns (a head), a = act(z),
//   norm first:  y = w u(x) a        gate first:  y = w u(x a)
// with u(v) = v / sqrt(mean v^2 + eps); y in the input's type or in 8 bits; and
// the gradient.
//
// Memory bounds it: x and z are read once and y is written once.  A row lies in
// the registers of its threads, and a group's sum is formed
//   lanes:    groups of 8 L columns, L = 1, 2, 4 ... 64, by the L neighbouring
//             lanes that hold them, without a barrier;
//   units:    a group is a row of its own, held by a wave or a block;
//   segments: groups of any width from 8 columns on, through LDS: a thread's 8
//             columns belong to two groups at most.
#include <algorithm>

#include "norm_device.h"

namespace gdr {

namespace {

// Narrower groups (of a width that lanes do not take) are summed as segments.
constexpr int kUnitColumns = 224;
// Columns of a row that a block's threads hold in the gradient of lanes, a
// multiple of every group's.
constexpr int kLanePiece = 8192;

enum Sums { kLanes, kUnits, kSegments };

struct GatedArgs {
  const void* x;
  const void* z;
  const void* w;
  void* y;
  float* scale;
  float* rstd;        // [rows][groups], nullable in the forward
  int64_t x_stride, z_stride;  // elements between rows
  int rows, D;
  int lanes;          // lanes of a group: that hold it (kLanes) or add it (kSegments)
  int size, groups;   // columns of a group, groups of a row
  int wdt, shared;    // shared: one group's weights for all
  int gate_first, act;  // act 1: silu, 2: sigmoid
  int quant, scale_group;
  float eps;
  double share;       // 1 / size
  // backward
  const void* dy;
  void* dx;
  void* dz;
  float* part;        // [sets][D], or [sets][size] of shared weights in lanes
  int sets;           // walkers of rows, each with a row of `part`
  // threads hold rows in pieces of so many columns: a group each (kUnits), or
  // up to kLanePiece (the gradient in lanes)
  int pieces, piece;
};

// The row and the columns that the u-th team of threads holds.
struct Unit {
  int64_t row;
  int piece, first, width;
};
__device__ __forceinline__ Unit unit_of(const GatedArgs& a, unsigned u) {
  if (a.pieces == 1) return {(int64_t)u, 0, 0, a.D};
  const unsigned row = u / (unsigned)a.pieces, piece = u - row * (unsigned)a.pieces;
  const int first = (int)piece * a.piece;
  return {(int64_t)row, (int)piece, first, min(a.piece, a.D - first)};
}

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

// The groups of the columns [c, c + 8): the first up to `bound`, and the next.
struct Span {
  int group, bound;
};
__device__ __forceinline__ Span span_of(const GatedArgs& a, int c) {
  const int g = c / a.size;
  return {g, (g + 1) * a.size};
}

// kSegments: the sums of all groups of a row from each vector's parts (a: of
// its first group, b: of the next), to total[group] in LDS for all threads.
// `part` holds two values a vector.  A group's vectors are added in a fixed
// order by as many lanes as hold them, up to a wave.
template <typename S, int VPT>
__device__ __forceinline__ void segment_sums(const GatedArgs& a, const Span* sp, const S* va,
                                             const S* vb, S* part, S* total) {
  const int nv = (a.D + 7) / 8;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int vi = i * blockDim.x + threadIdx.x;
    if (vi < nv) part[2 * vi] = va[i], part[2 * vi + 1] = vb[i];
  }
  __syncthreads();
  const int lane = threadIdx.x & (a.lanes - 1), teams = blockDim.x / a.lanes;
  for (int g = threadIdx.x / a.lanes; g < a.groups; g += teams) {
    const int c0 = g * a.size, c1 = c0 + a.size;
    S s = 0;
    for (int vi = c0 / 8 + lane; vi * 8 < c1; vi += a.lanes) {
      // the part that belongs to this group: the vector begins in it, or the
      // one before
      const int c = min(vi * 8, a.D - 8);
      s += part[2 * vi + (c >= c0 ? 0 : 1)];
    }
    s = lanes_sum(s, a.lanes);
    if (lane == 0) total[g] = s;
  }
  __syncthreads();
}

// Most vectors, and groups, of a row in segments of VPT steps a thread.
template <int VPT>
constexpr int most_vectors() {
  return 1024 * VPT;
}

// f(the order as a constant): one branch for all elements of a row.
template <typename F>
__device__ __forceinline__ void by_order(int gate_first, F f) {
  if (gate_first) f(std::true_type());
  else f(std::false_type());
}

// The forward.  Memory bounds it: 8192 rows of 4096 bf16 columns in heads of 128
// take 43 us for 201 MB (4.7 TB/s), 4099 of 5005 fp16 columns in groups of 715
// 36 us for 123 MB (3.4: a wave's second step is two fifths full).  To 8 bits
// 18,062 x 4096 take 98 us for 370 MB (3.8): exact gates (8 us) and quotients, the
// kernel's text holds 1371 vector instructions for a thread's 16 elements with
// both 8-bit types' and both activations' branches, 931 without the 8-bit types.
// Eight rows take 5 us.
template <typename T, bool QUANT, Sums SUMS, int NT, int VPT, bool PART>
__global__ __launch_bounds__(block_of<NT>()) void gated_fwd_kernel(GatedArgs a) {
  __shared__ __align__(8) float lds[32];
  constexpr bool kSeg = SUMS == kSegments;
  __shared__ double part[kSeg ? 2 * most_vectors<VPT>() : 1], total[kSeg ? most_vectors<VPT>() : 1];
  const int tid = NT == 64 ? (threadIdx.x & 63) : threadIdx.x, nt = row_threads<NT>();
  const Unit unit = unit_of(a, NT == 64 ? blockIdx.x * 4 + (threadIdx.x >> 6) : blockIdx.x);
  const int64_t row = unit.row;
  if (row >= a.rows) return;  // a whole wave; the barriers below are for rows of a block
  const int width = unit.width, first = unit.first;
  const T* x = reinterpret_cast<const T*>(a.x) + row * a.x_stride + first;
  const T* z = reinterpret_cast<const T*>(a.z) + row * a.z_stride + first;
  float f[VPT][8], t[VPT][8];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = column_of<PART>(i * nt + tid, width);
    load8<T, PART>(x + c, width, f[i]);
    load8<T, PART>(z + c, width, t[i]);
  }
  by_activation<false>(a.act, [&](auto act) {
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) t[i][e] = gate_value<act.value>(t[i][e]);
  });
  if (a.gate_first) {
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) f[i][e] *= t[i][e], t[i][e] = 1.f;
  }
  // squares, mean and root in 64 bits, as the norm without a gate has them
  double sum[VPT], next[kSeg ? VPT : 1];
  Span sp[kSeg ? VPT : 1];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v0 = (i * nt + tid) * 8, c = column_of<PART>(i * nt + tid, width);
    sum[i] = 0.0;
    if (kSeg) next[i] = 0.0, sp[i] = span_of(a, c);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const double v = c + e >= v0 ? f[i][e] : 0.f;
      if (kSeg && c + e >= sp[i].bound) next[i] = __builtin_fma(v, v, next[i]);
      else sum[i] = __builtin_fma(v, v, sum[i]);
    }
  }
  float rstd[VPT], rnext[kSeg ? VPT : 1];
  if (SUMS == kLanes) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v0 = (i * nt + tid) * 8;
      rstd[i] = inverse_root(lanes_sum(sum[i], a.lanes) * a.share + (double)a.eps);
      if (a.rstd && v0 < a.D && (tid & (a.lanes - 1)) == 0)
        a.rstd[row * a.groups + v0 / a.size] = rstd[i];
    }
  } else if (SUMS == kUnits) {
#pragma unroll
    for (int i = 1; i < VPT; ++i) sum[0] += sum[i];
    const double all = row_sum<NT>(sum[0], reinterpret_cast<double*>(lds));
    rstd[0] = inverse_root(all * a.share + (double)a.eps);
#pragma unroll
    for (int i = 1; i < VPT; ++i) rstd[i] = rstd[0];
    if (a.rstd && tid == 0) a.rstd[row * a.groups + unit.piece] = rstd[0];
  } else {
    segment_sums<double, VPT>(a, sp, sum, next, part, total);
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      rstd[i] = inverse_root(total[sp[i].group] * a.share + (double)a.eps);
      rnext[i] = inverse_root(total[min(sp[i].group + 1, a.groups - 1)] * a.share + (double)a.eps);
    }
    if (a.rstd)
      for (int g = tid; g < a.groups; g += nt)
        a.rstd[row * a.groups + g] = inverse_root(total[g] * a.share + (double)a.eps);
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v0 = (i * nt + tid) * 8, c = column_of<PART>(i * nt + tid, width);
    float w[8];
    if (!kSeg || !a.shared) {
      // (a power of two of columns in the lanes' groups)
      const int at = !a.shared ? first + c : SUMS == kLanes ? c & (a.size - 1) : c;
      load_weight<PART>(a.w, at, width, a.wdt, w);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        w[e] = load_scalar(a.w, c + e - sp[i].bound + (c + e >= sp[i].bound ? 0 : a.size), a.wdt);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      f[i][e] = f[i][e] * (kSeg && c + e >= sp[i].bound ? rnext[i] : rstd[i]) * w[e] * t[i][e];
      // (past the row's end the lanes hold groups that are none)
      if (QUANT && SUMS == kLanes && v0 >= a.D) f[i][e] = 0.f;
    }
    if (!QUANT && v0 < width)
      store8<T, PART>(reinterpret_cast<T*>(a.y) + row * a.D + first + c, width, f[i]);
  }
  if (QUANT)
    quantise_row<NT, VPT, PART>(f, row, tid, a.D, a.quant, a.scale_group,
                                reinterpret_cast<uint8_t*>(a.y), a.scale, lds);
}

// The gradient.  norm first, with u the unit rows:
//   du = dy w a,  dx = r (du - u mean(du u)),  dz = dy w u a',  dw = sum dy u a
// gate first, with v = x a and u its unit rows:
//   du = dy w,  dv = r (du - u mean(du u)),  dx = dv a,  dz = dv x a',
//   dw = sum dy u
// A block walks rows blockIdx.x, + blocks, ... with dw in registers and leaves
// its sum in `part`, which launch_reduce_rows adds in order.  Where lanes hold
// groups that share their weights the block adds up its groups first.
// 8192 x 4096 in heads of 128 take 62 us for 336 MB (5.4 TB/s), 4099 x 5005 in
// groups of 715 58 us for 205 MB (3.5: waves of two steps hold 204 registers, two
// of them a SIMD).  Beyond 8192 columns two steps of 1024 threads spill: one group
// of 16,384 some 160 registers (33.5 million elements 218 us, of 8192 69), segments
// some 480 (16,380 columns in groups of 12 302 us, 12,288 in 96 404; 4995 in 45,
// which spill none, 125).
template <typename T, Sums SUMS, int NT, int VPT, bool PART>
__global__ __launch_bounds__(block_of<NT>(), NT == 64 && VPT == 2 ? 2 : 4) void gated_bwd_kernel(GatedArgs a) {
  constexpr int RPB = NT == 64 ? 4 : 1;
  constexpr int COLS = 64 * VPT * 8;  // of a wave's row
  constexpr bool kSeg = SUMS == kSegments;
  __shared__ float lds[16];
  // columns of four rows, or (shared weights in lanes) each wave's group
  __shared__ float wsum[NT == 64 ? 4 * COLS : SUMS == kLanes ? 16 * 512 : 1];
  __shared__ float segs[kSeg ? 2 * most_vectors<VPT>() : 1], total[kSeg ? most_vectors<VPT>() : 1];
  const int tid = NT == 64 ? (threadIdx.x & 63) : threadIdx.x, nt = row_threads<NT>();
  const int q = NT == 64 ? (threadIdx.x >> 6) : 0;
  const Unit unit = unit_of(a, blockIdx.x * RPB + q);  // (its row: the walker)
  const int width = unit.width, first = unit.first;
  float dw[VPT][8], w[VPT][8];
  Span sp[kSeg ? VPT : 1];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int c = column_of<PART>(i * nt + tid, width);
    if (kSeg) sp[i] = span_of(a, c);
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[i][e] = 0.f;
    if (!kSeg || !a.shared) {
      const int at = !a.shared ? first + c : SUMS == kLanes ? c & (a.size - 1) : c;
      load_weight<PART>(a.w, at, width, a.wdt, w[i]);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        w[i][e] = load_scalar(a.w, c + e - sp[i].bound + (c + e >= sp[i].bound ? 0 : a.size), a.wdt);
    }
  }
  for (int64_t row = unit.row < a.sets ? unit.row : a.rows; row < a.rows; row += a.sets) {
    const T* x = reinterpret_cast<const T*>(a.x) + row * a.x_stride + first;
    const T* z = reinterpret_cast<const T*>(a.z) + row * a.z_stride + first;
    const T* dy = reinterpret_cast<const T*>(a.dy) + row * a.D + first;
    const float* rs = a.rstd + row * a.groups;
    float u[VPT][8], act[VPT][8], s[VPT][8], du[VPT][8], r[VPT], rnext[kSeg ? VPT : 1];
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int c = column_of<PART>(i * nt + tid, width);
      load8<T, PART>(x + c, width, u[i]);
      load8<T, PART>(z + c, width, act[i]);
      load8<T, PART>(dy + c, width, du[i]);
      r[i] = rs[kSeg ? sp[i].group : SUMS == kLanes ? (first + c) / a.size : unit.piece];
      if (kSeg) rnext[i] = rs[min(sp[i].group + 1, a.groups - 1)];
    }
    by_activation<false>(a.act, [&](auto which) {
#pragma unroll
      for (int i = 0; i < VPT; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const Gate g = gate_and_slope<which.value>(act[i][e]);
          act[i][e] = g.value;
          s[i][e] = g.slope;
        }
    });
    float dot[VPT], dnext[kSeg ? VPT : 1];
    by_order(a.gate_first, [&](auto gate_first) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int v0 = (i * nt + tid) * 8, c = column_of<PART>(i * nt + tid, width);
        const bool live = SUMS != kLanes || v0 < width;
        dot[i] = 0.f;
        if (kSeg) dnext[i] = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const bool second = kSeg && c + e >= sp[i].bound;
          const float re = second ? rnext[i] : r[i];
          const float unit = gate_first.value ? u[i][e] * act[i][e] * re : u[i][e] * re;
          const float k = gate_first.value ? 1.f : act[i][e];
          if (live) dw[i][e] += du[i][e] * unit * k;
          du[i][e] *= w[i][e];
          const float term = c + e >= v0 ? du[i][e] * k * unit : 0.f;
          if (second) dnext[i] += term;
          else dot[i] += term;
        }
      }
    });
    if (SUMS == kLanes) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) dot[i] = lanes_sum(dot[i], a.lanes) / (float)a.size;
    } else if (SUMS == kUnits) {
#pragma unroll
      for (int i = 1; i < VPT; ++i) dot[0] += dot[i];
      dot[0] = row_reduce<NT, false>(dot[0], lds) / (float)a.size;
#pragma unroll
      for (int i = 1; i < VPT; ++i) dot[i] = dot[0];
    } else {
      segment_sums<float, VPT>(a, sp, dot, dnext, segs, total);
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        dot[i] = total[sp[i].group] / (float)a.size;
        dnext[i] = total[min(sp[i].group + 1, a.groups - 1)] / (float)a.size;
      }
    }
    by_order(a.gate_first, [&](auto gate_first) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        const int c = column_of<PART>(i * nt + tid, width);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const bool second = kSeg && c + e >= sp[i].bound;
          const float re = second ? rnext[i] : r[i], mean = second ? dnext[i] : dot[i];
          const float d = du[i][e];
          if (gate_first.value) {
            // (with eps = 0 re may be as large as the activation is small: their
            // product comes first)
            const float dv = d - u[i][e] * act[i][e] * re * mean;
            s[i][e] = re * s[i][e] * dv * u[i][e];
            u[i][e] = re * act[i][e] * dv;
          } else {
            const float xr = u[i][e] * re;
            s[i][e] = d * xr * s[i][e];
            u[i][e] = re * (d * act[i][e] - xr * mean);
          }
        }
      }
    });
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v0 = (i * nt + tid) * 8, c = column_of<PART>(i * nt + tid, width);
      if (v0 >= width) continue;
      store8<T, PART>(reinterpret_cast<T*>(a.dx) + row * a.D + first + c, width, u[i]);
      store8<T, PART>(reinterpret_cast<T*>(a.dz) + row * a.D + first + c, width, s[i]);
    }
  }
  if (SUMS == kLanes && a.shared) {
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
    for (int k = threadIdx.x; k < a.size; k += blockDim.x) {
      float v = wsum[k];
      for (int i = 1; i < (int)blockDim.x >> 6; ++i) v += wsum[i * 512 + k];
      a.part[(int64_t)blockIdx.x * a.size + k] = v;
    }
    return;
  }
  if (NT == 0 || a.pieces > 1) {
    float* part = a.part + unit.row * a.D + first;
    if (unit.row < a.sets)
#pragma unroll
      for (int i = 0; i < VPT; ++i)
        if ((i * nt + tid) * 8 < width)
          store8<float, PART>(part + column_of<PART>(i * nt + tid, width), width, dw[i]);
  } else {
    // columns of the block's four rows, each at its vector's place
    float* part = a.part + (int64_t)blockIdx.x * a.D;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) wsum[q * COLS + (i * 64 + tid) * 8 + e] = dw[i][e];
    __syncthreads();
    for (int k = threadIdx.x; k < ((a.D + 7) / 8) * 8; k += 256) {
      const int c = column_of<PART>(k / 8, a.D) + k % 8;
      if (c < a.D)
        part[c] = (wsum[k] + wsum[(NT == 64 ? 1 : 0) * COLS + k]) +
                  (wsum[(NT == 64 ? 2 : 0) * COLS + k] + wsum[(NT == 64 ? 3 : 0) * COLS + k]);
    }
  }
}

template <typename F>
void by_type(const gdr_gated_norm_problem* p, F f) {
  if (p->dtype == GDR_BF16) f(__bf16());
  else if (p->dtype == GDR_FP16) f(_Float16());
  else f(float());
}

// How the sums of a problem's groups are formed.  Units hold a wave or a block a
// group, wherever no scale spans several groups and a wave's lanes are busy
// enough: (33.5 million bf16 elements, forward and gradient, as units and as
// segments: groups of 336 66 + 83 and 86 + 120 us, of 240 87 + 110 and 86 + 115, of
// 208 97 + 123 and 85 + 118, of 143 136 + 170 and 93 + 130, of 96 188 + 239 and 85 +
// 116).
Sums sums_of(const gdr_gated_norm_problem* p) {
  const int n = p->norm_size;
  if (n % 8 == 0 && n <= 512 && (n & (n - 1)) == 0) return kLanes;
  return n == p->D || (!p->quant && n >= kUnitColumns) ? kUnits : kSegments;
}
template <Sums SUMS>
using SumsTag = std::integral_constant<Sums, SUMS>;
using Zero = std::integral_constant<int, 0>;
using One = std::integral_constant<int, 1>;
using Two = std::integral_constant<int, 2>;

// Threads of a row in segments: a block's, also where a wave could hold it.
template <typename F>
void by_segments(int D, F f) {
  auto form = [&](auto vpt) {
    constexpr int C = 512 * vpt.value;
    f(dim3(64 * ((D + C - 1) / C)), 1, SumsTag<kSegments>(), Zero(), vpt, std::false_type());
  };
  if (D <= 8192) form(One());
  else form(Two());
}
// f(threads of a block, its rows, SUMS, NT, VPT, PART)
template <typename F>
void by_form(const gdr_gated_norm_problem* p, F f) {
  const Sums sums = sums_of(p);
  if (sums == kSegments) return by_segments(p->D, f);
  by_row<2>(sums == kLanes ? p->D : p->norm_size, [&](dim3 block, int rows, auto nt, auto vpt, auto part) {
    if constexpr (!part.value) {
      if (sums == kLanes) return f(block, rows, SumsTag<kLanes>(), nt, vpt, part);
    }
    f(block, rows, SumsTag<kUnits>(), nt, vpt, part);
  });
}
// The gradient holds six arrays of a row: one step a thread as far as a block
// reaches (as it was first built, 4096 columns by 256 threads of two steps took 193
// registers and 75 us, by 512 threads of one 111 and 61; now 103 and 62), two for a
// wave's units.
template <typename F>
void by_form_bwd(const gdr_gated_norm_problem* p, F f) {
  const Sums sums = sums_of(p);
  if (sums == kSegments) return by_segments(p->D, f);
  const int width = sums == kLanes ? std::min(p->D, kLanePiece) : p->norm_size;
  auto form = [&](dim3 block, int rows, auto nt, auto vpt, auto part) {
    if constexpr (!part.value) {
      if (sums == kLanes) return f(block, rows, SumsTag<kLanes>(), nt, vpt, part);
    }
    f(block, rows, SumsTag<kUnits>(), nt, vpt, part);
  };
  if (sums == kUnits && width > 512 && width <= 1024)
    return f(dim3(256), 4, SumsTag<kUnits>(), std::integral_constant<int, 64>(), Two(),
             std::false_type());
  if (width <= 8192) return by_row<1>(width, form);
  f(dim3(64 * ((width + 1023) / 1024)), 1, SumsTag<kUnits>(), Zero(), Two(), std::false_type());
}

GatedArgs args_of(const gdr_gated_norm_problem* p) {
  GatedArgs a{};
  a.x_stride = p->x_stride;
  a.z_stride = p->gate_stride;
  a.rows = p->rows;
  a.D = p->D;
  a.size = p->norm_size;
  a.groups = p->D / p->norm_size;
  a.lanes = p->norm_size / 8;
  if (sums_of(p) == kSegments) {
    a.lanes = 2;  // a group's vectors, one more at either end
    while (a.lanes < 64 && a.lanes < p->norm_size / 8 + 2) a.lanes *= 2;
  }
  a.wdt = (int)p->w_dtype;
  a.shared = p->shared_weight;
  a.gate_first = p->gate_first;
  a.act = p->activation;
  a.quant = p->quant;
  a.scale_group = p->scale_group;
  a.eps = p->eps;
  a.share = 1.0 / p->norm_size;
  a.piece = sums_of(p) == kLanes ? kLanePiece : p->norm_size;
  return a;
}

int pieces_of(const gdr_gated_norm_problem* p, bool backward) {
  const Sums sums = sums_of(p);
  return sums == kUnits               ? p->D / p->norm_size
         : sums == kLanes && backward ? (p->D + kLanePiece - 1) / kLanePiece
                                      : 1;
}
// Blocks of the gradient, and their walkers of rows (sets).  4096 waves fill the
// card; a block (a wave of units) walks at least 8 rows, against its partial
// sums.
struct Walk {
  int blocks, sets;
  int parts;  // rows of partial sums
};
Walk walk_of(const gdr_gated_norm_problem* p) {
  Walk w{};
  const int64_t groups = pieces_of(p, true);
  by_form_bwd(p, [&](dim3 block, int rows, auto, auto, auto, auto) {
    // `rows` walkers a block
    const int64_t most = std::max<int64_t>(1, 4096 * 64 / block.x * rows / groups);
    int64_t sets = std::max<int64_t>(1, std::min<int64_t>(most, ((int64_t)p->rows + 7) / 8));
    if (groups == 1) sets = (sets + rows - 1) / rows * rows;
    w.sets = (int)sets;
    w.blocks = (int)((sets * groups + rows - 1) / rows);
    // a block's own row of sums, or its walker's
    const bool own = groups == 1 || (sums_of(p) == kLanes && p->shared_weight);
    w.parts = own ? w.blocks : w.sets;
  });
  return w;
}

// Blocks of the forward: `rows` rows or, as units, groups each.
int64_t blocks_of(const gdr_gated_norm_problem* p, int rows) {
  return ((int64_t)p->rows * pieces_of(p, false) + rows - 1) / rows;
}

}  // namespace

int64_t gated_norm_threads(const gdr_gated_norm_problem* p) {
  int64_t threads = 0;
  by_form(p, [&](dim3 block, int rows, auto, auto, auto, auto) {
    threads = blocks_of(p, rows) * block.x;
  });
  return threads;
}

gdr_status launch_gated_norm_fwd(const gdr_gated_norm_problem* p, const void* x, const void* gate,
                                 const void* weight, void* y, float* scale, float* rstd,
                                 hipStream_t st) {
  GatedArgs a = args_of(p);
  a.x = x; a.z = gate; a.w = weight; a.y = y; a.scale = scale; a.rstd = rstd;
  a.pieces = pieces_of(p, false);
  by_type(p, [&](auto t) {
    using T = decltype(t);
    by_form(p, [&](dim3 block, int rows, auto sums, auto nt, auto vpt, auto part) {
      constexpr Sums SUMS = sums.value;
      constexpr int NT = nt.value, VPT = vpt.value;
      const dim3 grid((unsigned)blocks_of(p, rows));
      if (p->quant)
        GDR_LAUNCH("gated_fwd", (gated_fwd_kernel<T, true, SUMS, NT, VPT, part.value>), grid, block,
                   st, a);
      else
        GDR_LAUNCH("gated_fwd", (gated_fwd_kernel<T, false, SUMS, NT, VPT, part.value>), grid, block,
                   st, a);
    });
  });
  return launch_status("gated_norm_fwd");
}

size_t gated_norm_bwd_workspace(const gdr_gated_norm_problem* p) {
  // a row more for the groups' own sums
  return align256(((size_t)walk_of(p).parts + 1) * p->D * sizeof(float));
}

gdr_status launch_gated_norm_bwd(const gdr_gated_norm_problem* p, const void* dy, const void* x,
                                 const void* gate, const void* weight, const float* rstd, void* dx,
                                 void* dgate, void* dweight, void* ws, hipStream_t st) {
  GatedArgs a = args_of(p);
  a.x = x; a.z = gate; a.w = weight; a.rstd = const_cast<float*>(rstd);
  a.dy = dy; a.dx = dx; a.dz = dgate;
  a.part = reinterpret_cast<float*>(ws);
  const Walk walk = walk_of(p);
  a.pieces = pieces_of(p, true);
  a.sets = walk.sets;
  by_type(p, [&](auto t) {
    using T = decltype(t);
    by_form_bwd(p, [&](dim3 block, int, auto sums, auto nt, auto vpt, auto part) {
      GDR_LAUNCH("gated_bwd",
                 (gated_bwd_kernel<T, sums.value, nt.value, vpt.value, part.value>),
                 dim3(walk.blocks), block, st, a);
    });
  });
  if (a.shared && a.groups > 1 && sums_of(p) != kLanes) {
    float* sums = a.part + (int64_t)walk.parts * a.D;
    launch_reduce_rows(a.part, walk.parts, a.D, sums, GDR_FP32, st);
    launch_reduce_rows(sums, a.groups, a.size, dweight, a.wdt, st);
  } else {
    launch_reduce_rows(a.part, walk.parts, a.shared ? a.size : a.D, dweight, a.wdt, st);
  }
  return launch_status("gated_norm_bwd");
}

}  // namespace gdr

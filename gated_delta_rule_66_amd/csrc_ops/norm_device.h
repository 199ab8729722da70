// norm_device.h -- what the operators on rows share: a row in the registers of
// its threads, sums over it, and its quantisation to 8 bits.
//
// A row's threads hold 8 elements each per step.  Where the width is no
// multiple of 8 the row's last vector is moved back to end with the row: loads
// need no bounds, the elements that it repeats are left out of sums and
// maxima, and its stores repeat their bits.
#pragma once

#include <type_traits>

#include "ops_device.h"
#include "ops_internal.h"

namespace gdr {

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

// Threads of a row: NT, or the whole block where that is 0.
template <int NT>
__device__ __forceinline__ int row_threads() {
  return NT ? NT : (int)blockDim.x;
}

// Sum (or largest) of v over the threads of a row; every thread of the row gets
// the same bits.  Rows of one wave share a block, four at a time.
template <int NT, bool MAX>
__device__ __forceinline__ float row_reduce(float v, float* lds) {
  v = MAX ? wave_max(v) : wave_sum(v);
  if (NT == 64) return v;
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  if (NT == 0) {  // up to 16 waves, a lane each
    const int l = threadIdx.x & 15;
    v = l < (int)blockDim.x >> 6 ? lds[l] : 0.f;
    return MAX ? max16(v) : sum16(v);
  }
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
__device__ __forceinline__ double sum16(double v) {
  v += dpp_mov2<0xB1>(v);
  v += dpp_mov2<0x4E>(v);
  v += dpp_mov2<0x141>(v);
  v += dpp_mov2<0x140>(v);
  return v;
}
template <int NT>
__device__ __forceinline__ double row_sum(double v, double* lds) {
  v = sum16(v);
  v += __shfl_xor(v, 16, 64);
  v += __shfl_xor(v, 32, 64);
  if (NT == 64) return v;
  __syncthreads();
  if ((threadIdx.x & 63) == 0) lds[threadIdx.x >> 6] = v;
  __syncthreads();
  if (NT == 0) {
    const int l = threadIdx.x & 15;
    return sum16(l < (int)blockDim.x >> 6 ? lds[l] : 0.0);
  }
  double s = lds[0];
#pragma unroll
  for (int i = 1; i < NT / 64; ++i) s += lds[i];
  return s;
}

__device__ __forceinline__ uint32_t pack_fp8(float a, float b, float c, float d) {
  int r = 0;
  r = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, r, false);
  r = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, r, true);
  return (uint32_t)r;
}

// 1 / sqrt(a) to more than fp32's precision: the instruction's estimate and one
// step of Newton's (0 for an infinity, as the quotient has it).
__device__ __forceinline__ float inverse_root(double a) {
  const double y = __builtin_amdgcn_rsq(a);
  const double z = y * __builtin_fma(-0.5 * a * y, y, 1.5);
  return (float)(a < __builtin_inf() && a > 0.0 ? z : y);
}

// A gate's activations (kNone: z itself) and their derivatives, from
//   e = e^-|z|  and  r = 1 / (1 + e)
// to fp32's precision: the power of the exponent's fraction, which has an error
// of 2^-25 only, scaled by its whole part (subnormal numbers, too); the
// reciprocal's estimate gets a step of Newton's (with the instructions alone a
// 16-bit stream's roundings fell the other way twice as often as an exact
// gate's).  |z| is taken at 128 at the most, where e^-|z| is less than half of
// fp32's smallest number.  (minimum and maximum pass a NaN.)
enum Activation { kNone, kSilu, kSigmoid };
struct Tail {
  float e, r;
};
__device__ __forceinline__ Tail gate_tail(float z) {  // |z| <= 128
  constexpr float kLog2e = 1.4426950408889634f, kRest = 1.9259629911e-8f;
  constexpr float kWhole = 12582912.f;  // 1.5 2^23: its last bits count whole numbers
  const float m = fabsf(z);
  const float k = __builtin_fmaf(-m, kLog2e, kWhole), n = k - kWhole;
  const float f = __builtin_fmaf(-m, kRest, __builtin_fmaf(-m, kLog2e, -n));
  const float e = __builtin_ldexpf(__builtin_amdgcn_exp2f(f), __builtin_bit_cast(int, k) - 0x4b400000);
  const float d = 1.f + e, r = fast_rcp(d);
  return {e, __builtin_fmaf(__builtin_fmaf(-d, r, 1.f), r, r)};
}
template <Activation ACT>
__device__ __forceinline__ float gate_value(float z) {
  if (ACT == kNone) return z;
  z = __builtin_elementwise_maximum(z, -128.f);  // an infinity times 0 would be a NaN
  const Tail t = gate_tail(__builtin_elementwise_minimum(z, 128.f));
  const float s = (z < 0.f ? t.e : 1.f) * t.r;
  return ACT == kSilu ? z * s : s;
}
struct Gate {
  float value, slope;
};
// With t = e r, the smaller of the sigmoid and its complement: the larger is one
// less it (the other way round nothing would be left of an open gate's
// complement), their product the sigmoid's slope p, and silu's s + z p.
template <Activation ACT>
__device__ __forceinline__ Gate gate_and_slope(float z) {
  if (ACT == kNone) return {z, 1.f};
  z = __builtin_elementwise_maximum(z, -128.f);
  const float zc = __builtin_elementwise_minimum(z, 128.f);
  const Tail tail = gate_tail(zc);
  const float t = tail.e * tail.r, big = 1.f - t, p = t * big, s = z < 0.f ? t : big;
  if (ACT == kSilu) return {z * s, __builtin_fmaf(zc, p, s)};
  return {s, p};
}
// f(the activation as a constant): one branch for all elements of a row.
template <bool NONE, typename F>
__device__ __forceinline__ void by_activation(int act, F f) {
  if (act == 1) f(std::integral_constant<Activation, kSilu>());
  else if (!NONE || act == 2) f(std::integral_constant<Activation, kSigmoid>());
  else f(std::integral_constant<Activation, kNone>());
}

// Threads of a block (the most, where NT is 0): one row of NT threads, or (NT ==
// 64) four rows of one wave each.
template <int NT>
constexpr int block_of() {
  return NT == 64 ? 256 : NT == 0 ? 1024 : NT;
}

// Eight values over the scale s, rounded to nearest even: e4m3 or int8.  With s
// from the largest of them a quotient passes the type's largest value by a
// rounding at most, which the conversion's takes away.
__device__ __forceinline__ void quantise8(const float (&f)[8], float s, bool fp8, uint32_t (&b)[2]) {
  float q[8];
  // (an infinite scale leaves the product's 0 or NaN as they are)
  const bool finite = s < __builtin_inff();
  const float inv = 1.f / s, fin = finite ? s : 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    // the product with the reciprocal may lie on the other side of a tie,
    // a whole step off in 8 bits: the residual makes it the fp32 quotient
    q[e] = f[e] * inv;
    q[e] = __builtin_fmaf(__builtin_fmaf(-q[e], fin, f[e]), inv, q[e]);
  }
  if (fp8) {
    b[0] = pack_fp8(q[0], q[1], q[2], q[3]);
    b[1] = pack_fp8(q[4], q[5], q[6], q[7]);
  } else {
    // 1.5 2^23 + q holds q's nearest whole number in its lowest byte; a scale
    // that is no number or infinite leaves 0
    uint32_t u[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) u[e] = __builtin_bit_cast(uint32_t, q[e] + 12582912.f);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint32_t lo = __builtin_amdgcn_perm(u[4 * k + 1], u[4 * k], 0x0c0c0400u);
      const uint32_t hi = __builtin_amdgcn_perm(u[4 * k + 3], u[4 * k + 2], 0x04000c0cu);
      b[k] = finite ? lo | hi : 0u;
    }
  }
}
// Eight bytes to any address.
__device__ __forceinline__ void store_bytes8(uint8_t* y, const uint32_t (&b)[2]) {
  struct __attribute__((packed, aligned(1))) Raw {
    uint32_t u[2];
  };
  *reinterpret_cast<Raw*>(y) = Raw{{b[0], b[1]}};
}

// A row's values f to 8 bits (`quant` 1: e4m3, 2: int8): scale = max |f| / top,
// at least 2^-126 so that rows of zeros stay zeros, over the row (`group` 0) or
// over each 128 columns; the quotient is rounded to nearest even.  `lds`: 16
// floats that the row's threads share.
template <int NT, int VPT, bool PART>
__device__ __forceinline__ void quantise_row(const float (&f)[VPT][8], int64_t row, int tid, int D,
                                             int quant, int group, uint8_t* q_out, float* scale,
                                             float* lds) {
  const int nt = row_threads<NT>();
  const bool fp8 = quant == 1;
  const float top = fp8 ? 448.f : 127.f;
  const int ngroups = (D + 127) / 128;
  float row_scale = 0.f;
  if (group == 0) {
    float mx = 0.f;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) mx = max_nan(mx, fabsf(f[i][e]));
    mx = row_reduce<NT, true>(mx, lds) / top;
    row_scale = mx < kTinyScale ? kTinyScale : mx;
    if (tid == 0) scale[row] = row_scale;
  }
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v0 = (i * nt + tid) * 8, c = column_of<PART>(i * nt + tid, D);
    float s = row_scale;
    if (group) {  // 16 consecutive lanes hold a group's 128 columns
      float mx = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) mx = c + e >= v0 ? max_nan(mx, fabsf(f[i][e])) : mx;
      mx = max16(mx) / top;
      s = mx < kTinyScale ? kTinyScale : mx;
      if ((tid & 15) == 0 && v0 < D) scale[row * ngroups + v0 / 128] = s;
    }
    if (v0 < D) {
      uint32_t b[2];
      quantise8(f[i], s, fp8, b);
      uint8_t* y = q_out + row * D + c;
      if (!PART && c == v0) {
        store_bytes8(y, b);
      } else {  // what the vector repeats may belong to another scale
        for (int e = v0 - c; e < min(8, D); ++e) y[e] = (uint8_t)(b[e >> 2] >> (8 * (e & 3)));
      }
    }
  }
}

// How a row of D columns is held: by one wave (four rows a block) or by a block
// of just as many waves as it takes, MOST 8-element steps a thread (one where
// the row is as short as that).  f(threads of the block, rows of a block, NT,
// VPT, PART).
template <int MOST, typename F>
void by_row(int D, F f) {
  const int nv = (D + 7) / 8;
  const std::false_type whole;
  const std::integral_constant<int, 1> one;
  const std::integral_constant<int, MOST> most;
  const std::integral_constant<int, 64> wave;
  const std::integral_constant<int, 0> block;
  auto threads = [&](int steps) { return dim3(64 * ((nv + 64 * steps - 1) / (64 * steps))); };
  if (D < 8) f(dim3(256), 4, wave, one, std::true_type());
  else if (nv <= 64) f(dim3(256), 4, wave, one, whole);
  else if (MOST == 2 && nv <= 128) f(dim3(256), 4, wave, most, whole);
  else f(threads(MOST), 1, block, most, whole);
}

}  // namespace gdr

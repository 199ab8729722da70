// ops_device.h -- device-side building blocks of the layer operators.
#pragma once

#include "../csrc/gdr_device.h"
#include "../csrc/gdr_internal.h"

namespace gdr {

// N consecutive elements, 8 or 16 bytes (by default 16).  Rows of odd width
// start at any element, so the access promises only the element's own
// alignment: global memory takes 16-byte loads and stores at any address (the
// compiler emits one global_load_dwordx4 either way).
template <typename T, int N = 16 / (int)sizeof(T)>
struct Vec {
  static constexpr int n = N;
  struct __attribute__((packed, aligned(sizeof(T)))) Raw {
    uint32_t u[N * sizeof(T) / 4];
  };
  T v[n];

  __device__ __forceinline__ void load(const T* p) {
    const Raw r = *reinterpret_cast<const Raw*>(p);
    *this = __builtin_bit_cast(Vec, r);
  }
  __device__ __forceinline__ void store(T* p) const {
    *reinterpret_cast<Raw*>(p) = __builtin_bit_cast(Raw, *this);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int e = 0; e < n; ++e) v[e] = (T)0.f;
  }
  // the first m elements (the row's end); the others are zero
  __device__ __forceinline__ void load_part(const T* p, int m) {
    if (m >= n) {
      load(p);
      return;
    }
#pragma unroll
    for (int e = 0; e < n; ++e) v[e] = e < m ? p[e] : (T)0.f;
  }
  __device__ __forceinline__ void store_part(T* p, int m) const {
    if (m >= n) {
      store(p);
      return;
    }
#pragma unroll
    for (int e = 0; e < n; ++e)
      if (e < m) p[e] = v[e];
  }
};

// COUNT (a multiple of 4) consecutive values of a parameter held in 16 bits
// or fp32
template <typename T, int COUNT>
__device__ __forceinline__ void load_values(const T* p, float* f) {
#pragma unroll
  for (int k = 0; k < COUNT; k += 4) {
    Vec<T, 4> v;
    v.load(p + k);
#pragma unroll
    for (int e = 0; e < 4; ++e) f[k + e] = to_f(v.v[e]);
  }
}
template <int COUNT>
__device__ __forceinline__ void load_params(const void* p, int64_t i, int dtype, float* f) {
  if (dtype == GDR_BF16) load_values<__bf16, COUNT>(reinterpret_cast<const __bf16*>(p) + i, f);
  else if (dtype == GDR_FP16) load_values<_Float16, COUNT>(reinterpret_cast<const _Float16*>(p) + i, f);
  else load_values<float, COUNT>(reinterpret_cast<const float*>(p) + i, f);
}

__device__ __forceinline__ float fast_rcp(float x) { return __builtin_amdgcn_rcpf(x); }
__device__ __forceinline__ float sigmoid(float z) { return fast_rcp(1.f + __expf(-z)); }

// Sum over a whole wave (every lane ends with the same bits).
__device__ __forceinline__ float wave_sum(float v) { return sum4g(sum16(v)); }

}  // namespace gdr

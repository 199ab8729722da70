// ssm_device.h -- what the selective-scan kernels share: the segments that
// sequences are cut into, a chunk's gate, the tiles in LDS and the state in
// registers.
//
// Per sequence and head, with a K x V fp32 state S, dt_t = softplus(raw_t +
// bias) (or raw_t + bias) and g_t = -exp(A_log) dt_t:
//     S_t = e^{g_t} S_{t-1} + dt_t B_t x_t^T        y_t = S_t^T C_t + D x_t
// Chunk by chunk (64 tokens, gamma the inclusive cumsum of g in the chunk):
//     Y   = diag(e^gamma) C S + (C B^T o L diag(dt)) X,  L_ri = e^{gamma_r - gamma_i}, i <= r
//     S  <- e^{gamma_end} S + B^T diag(dt e^{gamma_end - gamma}) X
// Unlike the delta rule, a chunk's effect on the state does not depend on the
// state, so a sequence can be cut into segments whose effects are formed in
// parallel and added up with one scalar decay each.
#pragma once

#include <type_traits>

#include "ops_device.h"
#include "ops_internal.h"

namespace gdr {

struct SsmArgs {
  const void* x;
  const void* dt;
  const void* A_log;
  const void* B;
  const void* C;
  const void* D;        // nullable
  const void* dt_bias;  // nullable
  const float* h0;      // nullable
  void* y;
  float* ht;            // nullable
  // workspace: per (segment id, head) the state that the segment adds, then
  // the state at the segment's end; and the segment's summed log decay
  float* seg_state;
  float* seg_decay;
  const int32_t* cu;
  int64_t xs, bs, cs;   // elements between tokens of x, B, C
  int N, T, H, G;
  int seg;              // tokens per segment (a multiple of 64)
  int nids;             // segment ids
  int dt_dtype, p_dtype, softplus;
};

// Segment ids: dense batches number each sequence's ceil(T / seg) segments
// one after the other; packed sequence n starts at id n + floor(cu[n] / seg),
// which leaves it at least ceil(length / seg) ids, so that the id's sequence
// is found by bisection in cu alone.  Ids beyond a sequence's segments are
// unused.
struct Segment {
  int n, j, count;        // sequence, segment in it, segments of it (0: unused id)
  int64_t start, end;     // the sequence's tokens
  int64_t t0, t1;         // the segment's tokens
};

__device__ __forceinline__ Segment segment_of(const SsmArgs& a, int id) {
  Segment s;
  if (a.cu) {
    int lo = 0, hi = a.N - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (mid + a.cu[mid] / a.seg <= id) lo = mid;
      else hi = mid - 1;
    }
    s.n = lo;
    s.start = a.cu[lo];
    s.end = a.cu[lo + 1];
    s.j = id - (lo + a.cu[lo] / a.seg);
  } else {
    const int m = (a.T + a.seg - 1) / a.seg;
    s.n = id / m;
    s.j = id % m;
    s.start = (int64_t)s.n * a.T;
    s.end = s.start + a.T;
  }
  s.count = (int)((s.end - s.start + a.seg - 1) / a.seg);
  s.t0 = s.start + (int64_t)s.j * a.seg;
  s.t1 = min(s.end, s.t0 + a.seg);
  // a sequence without tokens keeps one (empty) segment, which passes its state on
  if (s.count == 0) s.count = s.j == 0 ? 1 : 0;
  if (s.j >= s.count) s.count = 0;
  return s;
}

// Logical block of hardware block b: consecutive logical blocks (the heads of
// one segment, which read the same B and C) run on one XCD and share its L2.
__device__ __forceinline__ int xcd_order(int b, int nb) {
  const int x = b & 7, q = nb >> 3, r = nb & 7;
  return x * q + min(x, r) + (b >> 3);
}

__device__ __forceinline__ float ssm_step_size(float raw, float bias, int softplus) {
  const float z = raw + bias;
  return softplus ? fmaxf(z, 0.f) + log1pf(__expf(-fabsf(z))) : z;
}

__device__ __forceinline__ float param(const void* p, int i, int dtype) {
  return p ? load_scalar(p, i, dtype) : 0.f;
}

// Exclusive suffix sum over the wave's lanes: sum of x over the lanes above.
__device__ __forceinline__ float wave_suffix_excl(float x) {
  const int l = lane_id();
  float s = __shfl_down(x, 1, 64);
  if (l == 63) s = 0.f;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const float y = __shfl_down(s, off, 64);
    if (l + off < 64) s += y;
  }
  return s;
}

// Transposed operand fragment with its rows in pair order: lane (grp, col)
// receives X[k0 + 8 grp + e][m0 + 8 (col / 4) + col % 4] of a row-major LDS
// matrix (base = &X[k0][m0]).  The D tiles of two such operands, m0 and m0 + 4,
// then hold rows 8 grp + e and 8 grp + 4 + e of a 32-row block: packed side by
// side they are an operand in contiguous k order with no data movement, and
// the other operand is one 16-byte read (frag_row).
template <typename T>
__device__ __forceinline__ typename VT<T>::x8 frag_tr_pair(const T* base, int ld) {
  const int l = lane_id();
  const int grp = l >> 4, j = l & 15;
  const T* p0 = base + (8 * grp + (j >> 2)) * ld + 8 * (j & 3);
  const T* p1 = p0 + 4 * ld;
  typedef __attribute__((address_space(3))) i16x4 lds_i16x4;
  const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(p0));
  const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4*)(p1));
  const i16x8 r = i16x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
  return __builtin_bit_cast(typename VT<T>::x8, r);
}

// Exponent e such that the largest |v| of the lane's column (the four lanes
// with its l % 16) times 2^e lies in [2^13, 2^14): fp16 operand pairs then
// keep 22 bits of every value that matters next to it, however small step
// sizes make them, and overflow never.  bf16 has fp32's range and needs no
// scale.
__device__ __forceinline__ int column_exponent(float m) {
  m = fmaxf(m, __shfl_xor(m, 16, 64));
  m = fmaxf(m, __shfl_xor(m, 32, 64));
  const int e = 14 - __builtin_amdgcn_frexp_expf(m);
  return m > 0.f && m < __builtin_inff() ? min(max(e, -100), 100) : 0;
}

// fp32 values as the sum of two 16-bit ones: hi is v rounded, lo the rest
// rounded, so that hi + lo is v to 2^-18 (bf16) relative; two products with
// them keep a state as exact as fp32 inputs would.
template <typename T>
__device__ __forceinline__ void split8(const float* v, typename VT<T>::x8& hi,
                                       typename VT<T>::x8& lo) {
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    hi[e] = from_f<T>(v[e]);
    lo[e] = from_f<T>(v[e] - to_f(hi[e]));
  }
}

template <typename T>
__device__ __forceinline__ typename VT<T>::x8 pack8(f32x4 a, f32x4 b) {
  return typename VT<T>::x8{from_f<T>(a[0]), from_f<T>(a[1]), from_f<T>(a[2]), from_f<T>(a[3]),
                            from_f<T>(b[0]), from_f<T>(b[1]), from_f<T>(b[2]), from_f<T>(b[3])};
}

// 64 rows of COLS elements from global memory into registers and from there
// to LDS (rows past `rows` are zero); NT threads, 16-byte pieces at any
// alignment.
template <typename T, int COLS, int NT>
struct Rows64 {
  static constexpr int kPer = 64 * COLS / 8 / NT;
  Vec<T> r[kPer];
  __device__ __forceinline__ void load(const T* g, int64_t stride, int rows) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int p = i * NT + threadIdx.x, row = p / (COLS / 8), c = p % (COLS / 8) * 8;
      if (row < rows) {
        r[i].load(g + row * stride + c);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) r[i].v[e] = (T)0.f;
      }
    }
  }
  __device__ __forceinline__ void store(T* lds, int ld) const {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int p = i * NT + threadIdx.x, row = p / (COLS / 8), c = p % (COLS / 8) * 8;
      *reinterpret_cast<uint4*>(lds + row * ld + c) = __builtin_bit_cast(uint4, r[i]);
    }
  }
};

// State element (k, v) of register e of tile nt, column tile pt, for wave w of
// 4 whose columns start at w V / 4: pair order along k (frag_tr_pair).
template <int V>
__device__ __forceinline__ int state_k(int nt, int e) {
  const int l = lane_id();
  return 32 * (nt >> 1) + 8 * (l >> 4) + 4 * (nt & 1) + e;
}
template <int V>
__device__ __forceinline__ int state_v(int w, int pt) {
  return w * (V / 4) + 16 * pt + (lane_id() & 15);
}

// Host side: the problem's arguments, its element type and sizes as types.
SsmArgs ssm_args(const gdr_ssm_problem* p, const SsmPlan& pl);
void launch_ssm_states(const gdr_ssm_problem* p, const SsmArgs& a, bool grad, hipStream_t st);

template <typename F>
inline void ssm_by_shape(const gdr_ssm_problem* p, F f) {
  auto type = [&](auto t) {
    using T = decltype(t);
    auto c64 = std::integral_constant<int, 64>();
    auto c128 = std::integral_constant<int, 128>();
    if (p->K == 64 && p->V == 64) f(T(), c64, c64);
    else if (p->K == 64) f(T(), c64, c128);
    else if (p->V == 64) f(T(), c128, c64);
    else f(T(), c128, c128);
  };
  if (p->in_dtype == GDR_BF16) type(__bf16());
  else type(_Float16());
}

}  // namespace gdr

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

// A value that the compiler takes to be new at this point: what depends on it
// is formed here again and not kept in registers across the chunk loop.
__device__ __forceinline__ int fresh_v(int x) {
  asm volatile("" : "+v"(x));
  return x;
}
__device__ __forceinline__ int fresh_s(int x) {
  asm volatile("" : "+s"(x));
  return x;
}

constexpr float kLog2e = 1.44269504088896340736f;
__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// softplus(z) = max(z, 0) + log(1 + u), u = e^{-|z|}, to a few units of fp32's
// last place: a step size's relative error is multiplied by the exponent that
// the decay has summed up.  e^t is 2^h (1 + ln 2 r) with t log2(e) = h + r, the
// product's rounding being r; log(1 + u) = 2 atanh(s), s = u / (2 + u) <= 1/3, by
// its series (the first term left out is below 2^-25 of the sum).
__device__ __forceinline__ float ssm_step_size(float raw, float bias, int softplus) {
  const float z = raw + bias, t = fmaxf(-fabsf(z), -120.f);
  const float h = t * kLog2e, r = __builtin_fmaf(t, kLog2e, -h);
  const float e = exp2_fast(h);
  const float u = __builtin_fmaf(e, r * 0.69314718f, e);
  const float s = u * fast_rcp(2.f + u), q = s * s;
  float p = 1.f / 15.f;
  p = __builtin_fmaf(p, q, 1.f / 13.f);
  p = __builtin_fmaf(p, q, 1.f / 11.f);
  p = __builtin_fmaf(p, q, 1.f / 9.f);
  p = __builtin_fmaf(p, q, 1.f / 7.f);
  p = __builtin_fmaf(p, q, 1.f / 5.f);
  p = __builtin_fmaf(p, q, 1.f / 3.f);
  p = __builtin_fmaf(p, q, 1.f);
  return softplus && z == z ? __builtin_fmaf(2.f * s, p, fmaxf(z, 0.f)) : z;
}

__device__ __forceinline__ float param(const void* p, int i, int dtype) {
  return p ? load_scalar(p, i, dtype) : 0.f;
}

// Prefix (inclusive) and suffix (exclusive) sums over the wave's lanes: DPP
// shifts within the rows of 16, then the rows' totals through scalars.
template <int CTRL>
__device__ __forceinline__ float dpp_zero(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL,
                                                               0xF, 0xF, true));
}
__device__ __forceinline__ float lane_value(float v, int lane) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}
__device__ __forceinline__ float wave_prefix(float x) {
  x += dpp_zero<0x111>(x);
  x += dpp_zero<0x112>(x);
  x += dpp_zero<0x114>(x);
  x += dpp_zero<0x118>(x);
  const float a = lane_value(x, 15), b = lane_value(x, 31), c = lane_value(x, 47);
  const int row = lane_id() >> 4;
  return x + (row == 0 ? 0.f : row == 1 ? a : row == 2 ? a + b : (a + b) + c);
}
__device__ __forceinline__ float wave_suffix_excl(float x) {
  x = __shfl_down(x, 1, 64);
  if (lane_id() == 63) x = 0.f;
  x += dpp_zero<0x101>(x);
  x += dpp_zero<0x102>(x);
  x += dpp_zero<0x104>(x);
  x += dpp_zero<0x108>(x);
  const float a = lane_value(x, 48), b = lane_value(x, 32), c = lane_value(x, 16);
  const int row = lane_id() >> 4;
  return x + (row == 3 ? 0.f : row == 2 ? a : row == 1 ? a + b : (a + b) + c);
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
    // v as one fp32 number: from the product it came from the compiler forms
    // hi twice, once rounded straight to fp16 (v_fma_mixlo_f16) and once by
    // way of fp32, which now and then are not the same
    float t = v[e];
    asm("" : "+v"(t));
    hi[e] = from_f<T>(t);
    lo[e] = from_f<T>(t - to_f(hi[e]));
  }
}

// Tiles in LDS have unpadded rows with their 16-byte pieces permuted (sw_off).
// All operands are read 8 bytes a lane, rows in split k order or transposed:
// measured, both then run at the rate of linear reads (a wave's 512 bytes in
// 1.7 counter ticks), while 16-byte row operands (4.5 against 2.7 linear) and
// tiles permuted by 8-byte units (2.8 against 1.7) do not.
// Operand reads.  The lane's byte offsets for the patterns are formed once; a
// tile's column offset is a multiple of 16 elements and enters by an
// exclusive or, its rows by an addition, so an address costs at most one
// instruction.  hide() keeps the compiler from forming all of them ahead of
// the chunk loop, which spills registers.
template <int COLS>
struct Sw {
  int split, tr;
  __device__ __forceinline__ Sw() {
    const int l = lane_id(), g = l >> 4, j = l & 15;
    split = 2 * sw_off<COLS>(j, 4 * g);
    tr = 2 * sw_off<COLS>(4 * g + (j >> 2), 4 * (j & 3));
  }
  __device__ __forceinline__ void hide() { asm volatile("" : "+v"(split), "+v"(tr)); }
};
// four elements of row r0 + lane % 16 from column c0 + 4 (lane / 16)
template <typename T, int COLS>
__device__ __forceinline__ const typename VT<T>::x4* row4(const T* X, const Sw<COLS>& o, int r0,
                                                          int c0) {
  return reinterpret_cast<const typename VT<T>::x4*>(reinterpret_cast<const char*>(X) +
                                                     2 * COLS * r0 + (o.split ^ (2 * c0)));
}
template <typename T, int COLS>
__device__ __forceinline__ typename VT<T>::x4* row4(T* X, const Sw<COLS>& o, int r0, int c0) {
  return reinterpret_cast<typename VT<T>::x4*>(reinterpret_cast<char*>(X) + 2 * COLS * r0 +
                                               (o.split ^ (2 * c0)));
}
// rows r0 + lane % 16 as an operand in split k order
template <typename T, int COLS>
__device__ __forceinline__ typename VT<T>::x8 split_frag(const T* X, const Sw<COLS>& o, int r0,
                                                         int k0) {
  typedef typename VT<T>::x4 x4;
  const char* p = reinterpret_cast<const char*>(X) + 2 * COLS * r0;
  const x4 lo = *reinterpret_cast<const x4*>(p + (o.split ^ (2 * k0)));
  const x4 hi = *reinterpret_cast<const x4*>(p + (o.split ^ (2 * k0 + 32)));
  return typename VT<T>::x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
}
// columns m0 + lane % 16, the 32 rows from k0 in split k order
template <typename T, int COLS>
__device__ __forceinline__ typename VT<T>::x8 tr_frag(const T* X, const Sw<COLS>& o, int k0, int m0) {
  const char* p = reinterpret_cast<const char*>(X) + 2 * COLS * k0 + (o.tr ^ (2 * m0));
  const i16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_t*)(p));
  const i16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_i16x4_t*)(p + 32 * COLS));
  return __builtin_bit_cast(typename VT<T>::x8,
                            i16x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]});
}

// Exponent e, the same in the wave, such that the largest |S| times 2^e lies in
// [2^13, 2^14); for fp16 operands.
template <int NT>
__device__ __forceinline__ int state_exponent(const f32x4* S) {
  float m = 0.f;
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int e = 0; e < 4; ++e) m = fmaxf(m, fabsf(S[nt][e]));
  m = fmaxf(m, dpp_mov<0xB1>(m));
  m = fmaxf(m, dpp_mov<0x4E>(m));
  m = fmaxf(m, dpp_mov<0x141>(m));
  m = fmaxf(m, dpp_mov<0x140>(m));
  m = fmaxf(m, __shfl_xor(m, 16, 64));
  m = fmaxf(m, __shfl_xor(m, 32, 64));
  const int e = 14 - __builtin_amdgcn_frexp_expf(m);
  return m > 0.f && m < __builtin_inff() ? min(max(e, -100), 100) : 100;
}

// The largest of the wave's v >= 0, in a scalar.
__device__ __forceinline__ float wave_largest(float v) {
  v = fmaxf(v, dpp_zero<0x111>(v));
  v = fmaxf(v, dpp_zero<0x112>(v));
  v = fmaxf(v, dpp_zero<0x114>(v));
  v = fmaxf(v, dpp_zero<0x118>(v));
  v = fmaxf(v, dpp_zero<0x142>(v));  // row 0's to row 1, 2's to 3; then both to row 3
  v = fmaxf(v, dpp_zero<0x143>(v));
  return lane_value(v, 63);
}

__device__ __forceinline__ float largest4(f32x4 v) {
  return fmaxf(fmaxf(fabsf(v[0]), fabsf(v[1])), fmaxf(fabsf(v[2]), fabsf(v[3])));
}

// Decayed scores as fp16 operands.  A wave scales a tile of 16 x 16 of them (the
// forward: the tiles of a column block) by a power of two such that the largest
// lies in [2^13, 2^14): whatever step sizes and gradients make of the scores,
// none overflows, and those down to 2^-27 of the largest keep the type's 11
// bits; `down` undoes the scale in the fp32 sums.  Tiles with scales of their
// own take products of 16 tokens instead of 32 (8 x 4096 tokens of 64 heads in
// 8 groups, K = 128, V = 64: 12 % of the outputs' 460 us, 2 and 7 % of the
// gradient's walks, 604 and 731).
__device__ __forceinline__ float tile_scale(float m, float& down) {
  m = wave_largest(m);
  const int e = 14 - __builtin_amdgcn_frexp_expf(m);
  const int s = m > 0.f && m < __builtin_inff() ? min(max(e, -120), 120) : 0;
  down = ldexpf(1.f, -s);
  return ldexpf(1.f, s);
}
__device__ __forceinline__ f16x4 tile_f16(f32x4 v, float& down) {
  const float up = tile_scale(largest4(v), down);
  return f16x4{from_f<_Float16>(v[0] * up), from_f<_Float16>(v[1] * up), from_f<_Float16>(v[2] * up),
               from_f<_Float16>(v[3] * up)};
}

template <typename T>
__device__ __forceinline__ typename VT<T>::x4 round4(f32x4 v) {
  return typename VT<T>::x4{from_f<T>(v[0]), from_f<T>(v[1]), from_f<T>(v[2]), from_f<T>(v[3])};
}

// Products over 16 tokens, of the halves (0 or 1) of operands in split k order.
// They are not chained with products over 32 through one accumulator: measured,
// a 32-token product right behind a 16-token one took two of its four sums
// before they were written.
__device__ __forceinline__ f32x4 mfma_half(f16x4 a, f16x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x16f16(a, b, c, 0, 0, 0);
}
__device__ __forceinline__ f32x4 mfma_half(bf16x4 a, bf16x4 b, f32x4 c) {
  return __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(__builtin_bit_cast(i16x4, a),
                                                   __builtin_bit_cast(i16x4, b), c, 0, 0, 0);
}
template <int HALF>
__device__ __forceinline__ f16x4 half_of(f16x8 v) {
  return f16x4{v[4 * HALF], v[4 * HALF + 1], v[4 * HALF + 2], v[4 * HALF + 3]};
}
template <int HALF>
__device__ __forceinline__ bf16x4 half_of(bf16x8 v) {
  return bf16x4{v[4 * HALF], v[4 * HALF + 1], v[4 * HALF + 2], v[4 * HALF + 3]};
}
// c + a b down over one half
template <int HALF>
__device__ __forceinline__ f32x4 mfma_tile(f16x8 a, f16x8 b, float down, f32x4 c) {
  return c + mfma_half(half_of<HALF>(a), half_of<HALF>(b), zero4()) * down;
}

// The weighted values of block tb of a chunk: column operand xf (split k order)
// times its tokens' weights.
template <typename T>
__device__ __forceinline__ void weighted(const typename VT<T>::x8& xf, const float* wt, int tb,
                                         int g4, float scale, float* v) {
  const f32x4 w0 = *reinterpret_cast<const f32x4*>(wt + 32 * tb + 4 * g4) * scale;
  const f32x4 w1 = *reinterpret_cast<const f32x4*>(wt + 32 * tb + 16 + 4 * g4) * scale;
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] = to_f(xf[e]) * (e < 4 ? w0[e & 3] : w1[e & 3]);
}

// S <- decay S + A^T diag(wt) x over a chunk's 64 tokens, for PT blocks of 16
// columns: A a swizzled 64 x K tile, xf[tb][pt] the lane's column of x in two
// blocks of 32 tokens, wt in LDS.  The weighted values go in as 16-bit operands
// that sum to them: a pair with fp16 (22 bits, the columns scaled to fit) and
// with bf16 (16 bits and a sign), or, EXACT, three with bf16.  States that are
// handed on (to a caller, to other segments) take EXACT: a pair's 2^-18 is 50
// times the error of fp32 sums.  Where a walk's states end in 16-bit outputs
// and 2^-16 sums (the gradient's forward walk) the pair is enough, and saves
// 5 % of the walk's time.
template <typename T, int K, bool EXACT, int PT>
__device__ __forceinline__ void update_state(f32x4 (&S)[PT][K / 16], const T* A, const Sw<K>& o,
                                             const typename VT<T>::x8 (&xf)[2][PT], const float* wt,
                                             int g4, float decay) {
  constexpr int NT = K / 16;
  constexpr bool kScaled = !__is_same(T, __bf16), kThree = EXACT && !kScaled;
  float scale[PT];
#pragma unroll
  for (int pt = 0; pt < PT; ++pt) {
    scale[pt] = 1.f;
    if (kScaled) {
      float m = 0.f;
#pragma unroll
      for (int tb = 0; tb < 2; ++tb) {
        float v[8];
        weighted<T>(xf[tb][pt], wt, tb, g4, 1.f, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) m = fmaxf(m, fabsf(v[e]));
      }
      scale[pt] = ldexpf(1.f, column_exponent(m));
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) S[pt][nt] *= kScaled ? decay * scale[pt] : decay;
  }
#pragma unroll
  for (int tb = 0; tb < 2; ++tb) {
    typename VT<T>::x8 hi[PT], lo[PT], rest[kThree ? PT : 1];
#pragma unroll
    for (int pt = 0; pt < PT; ++pt) {
      float v[8];
      weighted<T>(xf[tb][pt], wt, tb, g4, scale[pt], v);
      split8<T>(v, hi[pt], lo[pt]);
      if (kThree) {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          rest[pt][e] = from_f<T>(v[e] - to_f(hi[pt][e]) - to_f(lo[pt][e]));
      }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const auto f = tr_frag(A, o, 32 * tb, 16 * nt);
#pragma unroll
      for (int pt = 0; pt < PT; ++pt) {
        S[pt][nt] = mfma16(f, hi[pt], S[pt][nt]);
        S[pt][nt] = mfma16(f, lo[pt], S[pt][nt]);
        if (kThree) S[pt][nt] = mfma16(f, rest[pt], S[pt][nt]);
      }
      // a few operands in flight, not all of them: registers
      if (nt % (4 / PT) == 4 / PT - 1) __builtin_amdgcn_sched_barrier(0);
    }
  }
  if (kScaled) {
#pragma unroll
    for (int pt = 0; pt < PT; ++pt) {
      const float back = 1.f / scale[pt];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) S[pt][nt] *= back;
    }
  }
}

// 64 rows of COLS elements: NT threads hold them in registers between the
// global loads and the swizzled LDS tile (sw_off), so that the next chunk's
// loads are in flight while this one computes.  The range check of the
// buffer loads makes rows past the chunk's end zero.
template <typename T, int COLS, int NT>
struct Rows64 {
  static constexpr int kPer = 64 * COLS / 8 / NT, kRow = COLS / 8, kStep = NT / kRow;
  static_assert(kStep % 16 == 0, "a thread's rows share their swizzle");
  uint4 r[kPer];
  // `cols` of a row's COLS elements exist (the others of the last row read as
  // zero, of the rows before it as whatever follows)
  __device__ __forceinline__ void load(const T* g, int64_t stride, int rows, int cols = COLS) {
    const auto rs = buf_rsrc(g, ((rows - 1) * stride + cols) * (int64_t)sizeof(T));
    const int sb = (int)stride * (int)sizeof(T);
    int off = (int)threadIdx.x / kRow * sb + (int)threadIdx.x % kRow * 16;
    asm volatile("" : "+v"(off));
#pragma unroll
    for (int i = 0; i < kPer; ++i) r[i] = buf_load16(rs, off + i * (kStep * sb));
  }
  __device__ __forceinline__ void store(T* lds) const {
    T* p = lds + sw_off<COLS>((int)threadIdx.x / kRow, (int)threadIdx.x % kRow * 8);
#pragma unroll
    for (int i = 0; i < kPer; ++i) *reinterpret_cast<uint4*>(p + i * kStep * COLS) = r[i];
  }
};

// State element (k, v) of register e of tile nt in column block ct: k = 16 nt +
// 4 (lane / 16) + e, v = 16 ct + lane % 16 (the accumulator layout; two stacked
// tiles are an operand in split k order).
__device__ __forceinline__ int state_at(int ct, int nt, int e, int V) {
  const int l = lane_id();
  return (16 * nt + 4 * (l >> 4) + e) * V + 16 * ct + (l & 15);
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

// ssm_bwd.h -- the selective scan's gradient on gfx950: the walks along the
// segments, one instantiation unit per type (ssm_bwd_bf16.hip,
// ssm_bwd_fp16.hip); ssm_bwd.hip holds the small kernels and the launches.
//
// With P the gradient of the state after token t (P_t = C_t dy_t^T +
// e^{g_{t+1}} P_{t+1}), u_t = P_t^T B_t:
//     dx_t = dt_t u_t + D dy_t            dD = sum dy_t . x_t
//     dB_t = dt_t P_t x_t                 dC_t = S_t dy_t
//     ddt_t = rate dg_t + x_t . u_t       dA_log = sum g_t dg_t
// and dg_t, the gradient of the log decay, is the sum over all pairs i < t <=
// r of E_ri = e^{g_{i+1} + .. + g_r} dt_i (C_r . B_i)(dy_r . x_i).  Over a
// chunk these are the pairs inside it, those that end in it, those that begin
// in it and those that span it, with A the sum over the pairs that span the
// chunk's end, <S, P> there:
//     dg_t = (A - sum_{i in chunk} dt_i far_i) + sum_{i < t} dt_i far_i
//            + sum_{r >= t} (row_r - dt_r q_r)
//   row_r = sum_{i < r, in the chunk} E_ri + e^{gamma_r} dy_r . S^T C_r,
//   dt_i q_i = sum_{r > i, in the chunk} E_ri,   far_i = e^{gamma_end - gamma_i} x_i . P^T B_i
// (The pair i = r spans no decay; it is part of u_i . x_i = q_i + far_i + own_i
// only.)  dg at the chunk's first token is the A of the chunk before: a chain
// along the segment, from <S_end, P_end> at its end, that would add rounding
// errors up without limit, since what spans a chunk is a difference of sums.
// Two things end it.  Where a chunk decays by more than e^-24 nothing spans
// it; and every kMid chunks the forward walk leaves its fp32 state, which the
// backward walk multiplies by its own (one head of 4096 tokens, emulated: dA_log
// off by 0.5 to 8 % of the root of its summed squares with one plain suffix
// sum, by 0.03 % or less so).  No other state is stored: two walks, one forward
// with S, one backward with P, keep them in accumulators.
//   forward walk:  row_t, dC = diag(e^gamma) dY S^T + W B,   W = (dY X^T) o L diag(dt)
//   backward walk: u     = (C B^T o L)^T dY + diag(e^{gamma_end - gamma}) B P
//                  dB    = diag(dt e^{gamma_end - gamma}) X P^T + W^T C
// The scores' row and column sums are taken in fp32 before any rounding, and
// the state's share in them uses its 16-bit pair (hi + lo): up to kMid chunks
// of them are added up, so these must be near fp32.  W, one rounding of which
// would be shared by a row of dB or dC, is a pair of operands too (dB and dC of a
// short sequence 2.4 times as far from the definition with one), and C B^T o L
// gives dx its diagonal in fp32.  The other products round one operand (C B^T o
// L, S, P) to 16 bits, as their outputs are.
//
// One workgroup walks a segment for up to HPW heads of one group at once: they
// share the B and C tiles and C B^T, and their dB and dC are summed in
// registers.  Each wave holds 16 PT state columns of one head and, for that
// head, forms the state's products and update; the ten score tiles and the
// tiles of dB or dC are dealt over all waves, for which the states are passed
// through LDS once, rounded.  The order within a chunk keeps few registers
// live at once (at K = V = 128 a wave's states take 64 of its 256): scores go to
// LDS as they are formed.  The next chunk is requested as soon as this one is
// in LDS, where registers allow (K = 64, V = 128, two heads, backward: 90
// against 93 us; K = 128, V = 64: 82 against 86), and in the backward walk
// with K = V = 128 after dx is stored; with two heads of that size the second
// one's rows follow later, since all of them at once are spilled as they arrive
// (bf16 132 -> 113 and 172 -> 165 us, fp16 140 -> 123 and 201 -> 198).  With 8192
// tokens, 32 heads in 16 groups, K = V = 128 the walks take 113 and 165 us (fp16
// 123 and 198): matrix units busy 16 to 18 % and LDS 25 % of the time, none and 84
// bytes of spilled registers a lane (fp16 20 and 152), two waves per SIMD that wait
// for each other at three or four barriers a chunk.
#pragma once

#include "ssm_device.h"

namespace gdr {

// Chunks between the states that meet their gradients inside a segment.  Each
// costs 4 K V bytes written and read, 32 to 128 a token (8 x 4096 uncut tokens
// of 64 heads, K = 128, V = 64: 6 and 7 % of the walks' 555 and 671 us).
constexpr int kMid = 8;

struct SsmGradArgs {
  SsmArgs f;            // the forward's inputs, the segments, their start states
  const void* dy;
  const float* dht;     // nullable
  const float* seg_grad;   // per (id, head): the state's gradient at the segment's start
  void* dx;
  void* dB;
  void* dC;
  float* dh0;           // nullable
  // fp32 [slots][tokens][G][K] when a group's heads take more than one workgroup
  float* part_dB;
  float* part_dC;
  // [H][tokens], the sums above
  float* row;
  float* q;
  float* far;
  float* own;
  // the states kMid chunks apart inside segments (register order) and their
  // products with their gradients, in 8 waves' parts, at (tokens before) / (64 kMid)
  float* mid_state;     // nullable: no segment has more than kMid chunks
  float* mid;
  int mid_parts;        // waves of a head
  float* span;          // [nids][H]: <S_end, P_end>
  float* part_dD;       // [nids][H]
  int slots;            // workgroups per group
  int64_t tokens;
};

template <typename T, int K, int V, int HPW, bool REV>
void launch_ssm_grad(const SsmGradArgs& a, unsigned grid, hipStream_t st);

#ifdef GDR_SSM_GRAD_KERNELS

namespace {

// Heads whose state columns are in LDS at once: all of them where they fit
// (with K = V = 128 two heads' tiles leave room for one).
template <int K, int V, int HPW>
constexpr int kPublished = K * V == 128 * 128 ? 1 : HPW;

template <typename T, int K, int V, int HPW, int NW, bool REV>
struct GradSmem {
  T C[64 * K];
  T B[64 * K];
  T X[HPW][64 * V];
  T Y[HPW][64 * V];
  T R[kPublished<K, V, HPW> * V * K];  // state columns [V][K]
  T W[64 * 64];
  T GL[REV ? HPW : 0][64 * 64];  // the decayed scores
  T Wd[REV ? 0 : 64 * 16];  // the rest of W's diagonal tiles (backward: in GL)
  float od[REV ? HPW : 0][64];  // the rest of GL's diagonal
  // fp16: what undoes the scales of W's and GL's tiles
  float wd[__is_same(T, __bf16) ? 0 : 16], gd[REV && !__is_same(T, __bf16) ? HPW : 0][16];
  float gam[HPW][64];  // in powers of two
  float eg[HPW][64], es[REV ? HPW : 0][64], wt[HPW][64], dts[HPW][64], decay[HPW];
  float pe[HPW][160], pa[NW][64], po[REV ? HPW : 0][64];  // pe: sum_at
  int ex[NW];
  float fin[HPW][NW];
};

// The ten 16 x 16 tiles on or below the diagonal of a chunk's 64 x 64 matrix
// over NW waves: tile s of wave w as row block * 4 + column block, -1 past the
// wave's share (3, 3, 2, 2 of four waves; 2, 2 and six times 1 of eight).
template <int NW>
constexpr int kMostTiles = NW == 4 ? 3 : 2;
template <int NW>
__device__ __forceinline__ int tri_tile(int w, int s) {
  constexpr uint64_t all = 0xFEDCA98405ull;  // tiles 5, 0, 4, 8, 9, A, C, D, E, F
  const int i = NW == 4 ? w + 4 * s : s == 0 ? w + 2 : w;
  const bool in = NW == 4 ? i < 10 : s == 0 || w < 2;
  return in ? (int)(all >> (4 * i)) & 15 : -1;
}

// Token a's sum over the tokens of block bb: on and below the diagonal of a
// chunk's 64 x 4 such sums (backward: above it).
template <bool REV>
__device__ __forceinline__ int sum_at(int bb, int a) {
  return REV ? 8 * bb * (bb + 1) + a : 56 * bb - 8 * bb * bb + a;
}

// The two walks are mirror images: with (P, Q, p, q) = (C, B, dY, X) forward
// and (B, C, X, dY) backward, a the token a result belongs to and b the one
// it sums over (b <= a forward, b >= a backward), both form the scores P_a .
// Q_b and p_a . q_b, the state's product with P and its dot with p, the
// gradient of P from the state and W, and update the state with Q^T q.
template <typename T, int K, int V, int HPW, int PT, bool REV>
__global__ __launch_bounds__(4 * HPW * V / PT, REV && K == 128 && HPW * V / PT == 64 ? 1 : 2) void ssm_grad_kernel(
    SsmGradArgs ga) {
  typedef typename VT<T>::x8 x8;
  typedef typename VT<T>::x4 x4;
  constexpr int NW = HPW * V / (16 * PT), WPH = NW / HPW, NTH = 64 * NW, NT = K / 16;
  constexpr int TPW = 4 * NT / NW, MT = kMostTiles<NW>, RB = kPublished<K, V, HPW>;
  constexpr bool kScaled = !__is_same(T, __bf16), kEarly = !REV || K * V < 128 * 128;
  constexpr bool kSplit = RB < HPW;
  static_assert(TPW >= 1 && (NW == 4 || NW == 8), "tiles are dealt to all waves");
  __shared__ __align__(16) GradSmem<T, K, V, HPW, NW, REV> s;
  const SsmArgs& a = ga.f;
  const int R = a.H / a.G;
  const int L = xcd_order(blockIdx.x, gridDim.x);
  const int slot = L % ga.slots, grp = L / ga.slots % a.G, id = L / (ga.slots * a.G);
  const int head0 = grp * R + slot * HPW, nh = min(HPW, R - slot * HPW);
  const Segment sg = segment_of(a, id);
  if (sg.count == 0) {
    if (REV && threadIdx.x < (unsigned)nh) ga.part_dD[(int64_t)id * a.H + head0 + threadIdx.x] = 0.f;
    return;
  }
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = lane_id();
  const int ct0 = w % WPH * PT, h = head0 + min(w / WPH, nh - 1);
  const bool active = w / WPH < nh;

  // start states: the forward walk's from the segment before (or h0), the
  // backward walk's from the segment after (or dht)
  f32x4 S[PT][NT];
  const int64_t KV = (int64_t)K * V;
  auto load_slot = [&](const float* p, int id_, int pt, f32x4* dst) {
    const float* src = p + ((int64_t)id_ * a.H + h) * KV;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
      dst[nt] = *reinterpret_cast<const f32x4*>(src + (((ct0 + pt) * NT + nt) * 64 + l) * 4);
  };
  auto load_user = [&](const float* p, int pt, f32x4* dst) {
    const float* src = p ? p + ((int64_t)sg.n * a.H + h) * KV : nullptr;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) dst[nt][e] = src ? src[state_at(ct0 + pt, nt, e, V)] : 0.f;
  };
  auto end_grad = [&](int pt, f32x4* dst) {  // the state's gradient at the segment's end
    if (sg.j + 1 < sg.count) load_slot(ga.seg_grad, id + 1, pt, dst);
    else load_user(ga.dht, pt, dst);
  };
  auto exponent = [&]() {
    int e = state_exponent<NT>(S[0]);
#pragma unroll
    for (int pt = 1; pt < PT; ++pt) e = min(e, state_exponent<NT>(S[pt]));
    return e;
  };
#pragma unroll
  for (int pt = 0; pt < PT; ++pt) {
    if (REV) end_grad(pt, S[pt]);
    else if (sg.j > 0) load_slot(a.seg_state, id - 1, pt, S[pt]);
    else load_user(a.h0, pt, S[pt]);
  }
  if (kScaled) {
    const int e = exponent();
    if (l == 0) s.ex[w] = e;
  }

  const float skip = param(a.D, h, a.p_dtype);
  // the head whose gate this wave forms, if it is one of the last waves
  const int gh = NW - 1 - w, ghead = head0 + min(gh, nh - 1);
  const bool gates = gh < nh;
  const float rate = -expf(load_scalar(a.A_log, ghead, a.p_dtype));
  const float bias = param(a.dt_bias, ghead, a.p_dtype);
  float dsum[HPW];
#pragma unroll
  for (int hh = 0; hh < HPW; ++hh) dsum[hh] = 0.f;
  const T* xg = reinterpret_cast<const T*>(a.x) + (int64_t)head0 * V;
  const T* yg = reinterpret_cast<const T*>(ga.dy) + (int64_t)head0 * V;
  const T* bg = reinterpret_cast<const T*>(a.B) + (int64_t)grp * K;
  const T* cg = reinterpret_cast<const T*>(a.C) + (int64_t)grp * K;
  const int64_t ys = (int64_t)a.H * V;

  Rows64<T, K, NTH> rb, rc;
  Rows64<T, V, NTH> rx[HPW], ry[HPW];
  float raw = 0.f;
  const int nch = (int)((sg.t1 - sg.t0 + 63) / 64);
  auto token = [&](int c) { return sg.t0 + 64ll * (REV ? nch - 1 - c : c); };
  auto rows_of = [&](int64_t t) { return (int)min((int64_t)64, sg.t1 - t); };
  // chunk c's heads h0 <= hh < h1, with the first one B and C
  auto request = [&](int c, int h0, int h1) {
    const int64_t t = token(c);
    const int rows = rows_of(t);
    if (h0 == 0) {
      rb.load(bg + t * a.bs, a.bs, rows);
      rc.load(cg + t * a.cs, a.cs, rows);
    }
#pragma unroll
    for (int hh = 0; hh < HPW; ++hh)
      if (hh >= h0 && hh < h1 && hh < nh) {
        rx[hh].load(xg + t * a.xs + hh * V, a.xs, rows);
        ry[hh].load(yg + t * ys + hh * V, ys, rows);
      }
  };
  auto request_dt = [&](int c) {
    const int64_t t = token(c);
    raw = l < rows_of(t) ? load_scalar(a.dt, (t + l) * a.H + ghead, a.dt_dtype) : 0.f;
  };
  auto gate = [&](int c) {  // one token per lane
    const float step = l < rows_of(token(c)) ? ssm_step_size(raw, bias, a.softplus) : 0.f;
    const float g = rate * step;
    const float gam = wave_prefix(g), es = __expf(wave_suffix_excl(g));
    s.gam[gh][l] = gam * kLog2e;
    s.eg[gh][l] = __expf(gam);
    if (REV) s.es[REV ? gh : 0][l] = es;
    s.wt[gh][l] = step * es;
    s.dts[gh][l] = step;
    if (l == 0) s.decay[gh] = __expf(lane_value(gam, 63));
  };
  if (nch > 0) {
    request(0, 0, HPW);
    if (gates) request_dt(0);
  }

  const T* P = REV ? s.B : s.C;
  const T* Q = REV ? s.C : s.B;
  Sw<K> ok;
  Sw<V> ov;
  Sw<64> om;
  __syncthreads();
  for (int c = 0; c < nch; ++c) {
    const int64_t t = token(c);
    const int rows = rows_of(t);
    const int lf = fresh_v(l), wf = fresh_s(w), g4 = lf >> 4, col = lf & 15;
    const int hw = wf / WPH, v0 = wf % WPH * (16 * PT);
    const int hr = min(hw, nh - 1);  // inactive waves read what exists
    const T* p = REV ? s.X[hr] : s.Y[hr];
    const T* q = REV ? s.Y[hr] : s.X[hr];
    ok.hide();
    ov.hide();
    om.hide();
    rb.store(s.B);
    rc.store(s.C);
#pragma unroll
    for (int hh = 0; hh < HPW; ++hh)
      if (hh < nh) {
        rx[hh].store(s.X[hh]);
        ry[hh].store(s.Y[hh]);
      }
    // fp16: one exponent per head for its state columns as operands
    float up = 1.f, down = 1.f, hdown[HPW];
#pragma unroll
    for (int hh = 0; hh < HPW; ++hh) {
      hdown[hh] = 1.f;
      if (kScaled) {
        int e = s.ex[hh * WPH];
#pragma unroll
        for (int i = 1; i < WPH; ++i) e = min(e, s.ex[hh * WPH + i]);
        hdown[hh] = ldexpf(1.f, -e);
        if (hh == hw) {
          up = ldexpf(1.f, e);
          down = hdown[hh];
        }
      }
    }
    // this wave's state columns, rounded, for the other waves
    auto publish = [&](T* dst) {
#pragma unroll
      for (int pt = 0; pt < PT; ++pt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          x4 z;
#pragma unroll
          for (int e = 0; e < 4; ++e) z[e] = from_f<T>(kScaled ? S[pt][nt][e] * up : S[pt][nt][e]);
          *row4(dst, ok, v0 + 16 * pt, 16 * nt) = z;
        }
    };
    if (active && hw < RB) publish(s.R + hw * V * K);
    if (gates) {
      gate(c);
      if (c + 1 < nch) request_dt(c + 1);
    }
    __syncthreads();  // A: tiles, gates and the first state columns are in LDS
    const bool more = c + 1 < nch;
    if (kEarly && more) request(c + 1, 0, kSplit ? 1 : HPW);

    // W is a pair of operands: the second one's tiles lie across the diagonal
    // from the first's, those on it in tiles that nothing else uses (backward:
    // on GL's empty side)
    auto rest_of_w = [&](int ab, int bb) -> x4* {
      if (ab != bb) return row4(s.W, om, 16 * bb, 16 * ab);
      if (REV) return row4(s.GL[0], om, ab < 3 ? 48 : 32, ab < 3 ? 16 * ab : 0);
      return reinterpret_cast<x4*>(s.Wd + 16 * (16 * ab + col) + 4 * g4);
    };

    // scores (transposed: rows b, columns a), their sums over b, and W summed
    // over the heads
#pragma unroll
    for (int k = 0; k < MT; ++k) {
      const int ti = tri_tile<NW>(wf, k);
      if (ti >= 0) {
        const int ab = REV ? ti & 3 : ti >> 2, bb = REV ? ti >> 2 : ti & 3;
        f32x4 gt = zero4(), wsum = zero4();
#pragma unroll
        for (int kb = 0; kb < K / 32; ++kb)
          gt = mfma16(split_frag(Q, ok, 16 * bb, 32 * kb), split_frag(P, ok, 16 * ab, 32 * kb), gt);
        const int ia = 16 * ab + col, ib = 16 * bb + 4 * g4;
#pragma unroll
        for (int hh = 0; hh < HPW; ++hh) {
          if (hh >= nh) continue;
          const T* ph = REV ? s.X[hh] : s.Y[hh];
          const T* qh = REV ? s.Y[hh] : s.X[hh];
          f32x4 vt = zero4();
#pragma unroll
          for (int kv = 0; kv < V / 32; ++kv)
            vt = mfma16(split_frag(qh, ov, 16 * bb, 32 * kv), split_frag(ph, ov, 16 * ab, 32 * kv), vt);
          const float gam_a = s.gam[hh][ia], dt_a = s.dts[hh][ia];
          const f32x4 gam_b = *reinterpret_cast<const f32x4*>(&s.gam[hh][ib]);
          const f32x4 dt_b = *reinterpret_cast<const f32x4*>(&s.dts[hh][ib]);
          float sum = 0.f, own = 0.f;  // own: the pair of a token with itself
          f32x4 gl;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const bool in = REV ? ib + e >= ia : ib + e <= ia, self = ib + e == ia;
            const float lx = exp2_fast(REV ? gam_b[e] - gam_a : gam_a - gam_b[e]);
            const float lm = in ? lx : 0.f;
            const float f = vt[e] * lm;
            const float fd = f * (REV ? dt_a : dt_b[e]);
            wsum[e] += fd;
            if (REV) {
              gl[e] = gt[e] * lm;
              const float one = gt[e] * f;
              sum += self ? 0.f : one;
              own += self ? one : 0.f;
              dsum[hh] += self ? vt[e] : 0.f;
            } else {
              sum += self ? 0.f : gt[e] * fd;
            }
          }
          sum = sum4g(sum);
          if (g4 == 0) s.pe[hh][sum_at<REV>(bb, ia)] = sum;
          if (REV && ab == bb) {
            own = sum4g(own);
            if (g4 == 0) s.po[REV ? hh : 0][ia] = own;
          }
          if (REV) {
            float back = 1.f;
            x4 z;
            if constexpr (kScaled) {
              z = tile_f16(gl, back);
              if (l == 0) s.gd[hh][4 * ab + bb] = back;
            } else {
              z = round4<T>(gl);
            }
            *row4(s.GL[hh], om, 16 * ab, 16 * bb) = z;
            if (ab == bb && g4 == col >> 2) {  // what rounding took from the diagonal
              float d = 0.f;
#pragma unroll
              for (int e = 0; e < 4; ++e) d += ib + e == ia ? gl[e] - to_f(z[e]) * back : 0.f;
              s.od[REV ? hh : 0][ia] = d;
            }
          }
        }
        if constexpr (kScaled) {
          float back;
          wsum *= tile_scale(largest4(wsum), back);
          if (l == 0) s.wd[4 * ab + bb] = back;
        }
        x4 hi, lo;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          float t = wsum[e];
          asm("" : "+v"(t));  // one fp32 number (as in split8)
          hi[e] = from_f<T>(t);
          lo[e] = from_f<T>(t - to_f(hi[e]));
        }
        *row4(s.W, om, 16 * ab, 16 * bb) = hi;
        *rest_of_w(ab, bb) = lo;
      }
      __builtin_amdgcn_sched_barrier(0);
    }

    // P's gradient, transposed: head hh's state's part, rows k, columns a
    f32x4 acc[TPW];
#pragma unroll
    for (int i = 0; i < TPW; ++i) acc[i] = zero4();
    auto inter = [&](int hh) {
      const T* ph = REV ? s.X[hh] : s.Y[hh];
      const T* src = s.R + (RB == 1 ? 0 : hh * V * K);
      const float* sc = REV ? s.wt[hh] : s.eg[hh];
      constexpr int PER = TPW < 4 ? TPW : 4;   // tiles that share the state's operand
#pragma unroll
      for (int j = 0; j < TPW / PER; ++j) {
        const int idx = wf * TPW + j * PER, nt = idx >> 2, a0 = idx & 3;
        f32x4 tmp[PER];
#pragma unroll
        for (int i = 0; i < PER; ++i) tmp[i] = zero4();
#pragma unroll
        for (int kv = 0; kv < V / 32; ++kv) {
          const x8 af = tr_frag(src, ok, 32 * kv, 16 * nt);
#pragma unroll
          for (int i = 0; i < PER; ++i)
            tmp[i] = mfma16(af, split_frag(ph, ov, 16 * (a0 + i), 32 * kv), tmp[i]);
        }
#pragma unroll
        for (int i = 0; i < PER; ++i)
          acc[j * PER + i] += tmp[i] * (sc[16 * (a0 + i) + col] * hdown[hh]);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
#pragma unroll
    for (int hh = 0; hh < RB; ++hh)
      if (hh < nh) inter(hh);

    // the state's product with P, its pair of operands, rows v, columns a; its
    // dot with p goes into a's sum
    f32x4 u[PT][4];
#pragma unroll
    for (int pt = 0; pt < PT; ++pt)
#pragma unroll
      for (int r = 0; r < 4; ++r) u[pt][r] = zero4();
    if (active) {
#pragma unroll
      for (int kb = 0; kb < K / 32; ++kb) {
        x8 hi[PT], lo[PT];
#pragma unroll
        for (int pt = 0; pt < PT; ++pt) {
          float v[8];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            v[e] = kScaled ? S[pt][2 * kb][e] * up : S[pt][2 * kb][e];
            v[4 + e] = kScaled ? S[pt][2 * kb + 1][e] * up : S[pt][2 * kb + 1][e];
          }
          split8<T>(v, hi[pt], lo[pt]);
        }
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const x8 f = split_frag(P, ok, 16 * r, 32 * kb);
#pragma unroll
          for (int pt = 0; pt < PT; ++pt) {
            u[pt][r] = mfma16(hi[pt], f, u[pt][r]);
            u[pt][r] = mfma16(lo[pt], f, u[pt][r]);
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float sc = (REV ? s.es[REV ? hw : 0] : s.eg[hw])[16 * r + col] * down;
        float dot = 0.f;
#pragma unroll
        for (int pt = 0; pt < PT; ++pt) {
          u[pt][r] *= sc;
          const x4 o = *row4(p, ov, 16 * r, v0 + 16 * pt);
#pragma unroll
          for (int e = 0; e < 4; ++e) dot += u[pt][r][e] * to_f(o[e]);
        }
        dot = sum4g(dot);
        if (g4 == 0) s.pa[wf][16 * r + col] = dot;
      }
    }
    x8 xf[2][PT];
#pragma unroll
    for (int tb = 0; tb < 2; ++tb)
#pragma unroll
      for (int pt = 0; pt < PT; ++pt) xf[tb][pt] = tr_frag(q, ov, 32 * tb, v0 + 16 * pt);
    __syncthreads();  // B: W, the scores and the sums are in LDS, the state columns read

    if (RB < HPW && nh > 1) {  // the second head's columns take the first one's place
      if (active && hw == 1) publish(s.R);
      __syncthreads();
    }
    if (REV && active) {
      T* dx = reinterpret_cast<T*>(ga.dx) + t * ys + (int64_t)h * V;
      const int yb = (int)ys * (int)sizeof(T);
      const auto rs = buf_rsrc(dx, (int64_t)(rows - 1) * yb + V * (int)sizeof(T));
#pragma unroll
      for (int r = 0; r < 4; ++r) {
#pragma unroll
        for (int sb = r >> 1; sb < 2; ++sb) {
          const x8 f = split_frag(s.GL[hw], om, 16 * r, 32 * sb);
#pragma unroll
          for (int pt = 0; pt < PT; ++pt) {
            if constexpr (kScaled) {
              if (2 * sb >= r) u[pt][r] = mfma_tile<0>(xf[sb][pt], f, s.gd[hw][4 * r + 2 * sb], u[pt][r]);
              u[pt][r] = mfma_tile<1>(xf[sb][pt], f, s.gd[hw][4 * r + 2 * sb + 1], u[pt][r]);
            } else {
              if (r % 2 == 0) {
                u[pt][r] = mfma16(xf[sb][pt], f, u[pt][r]);
              } else {
                if (2 * sb >= r) u[pt][r] = mfma_half(half_of<0>(xf[sb][pt]), half_of<0>(f), u[pt][r]);
                u[pt][r] = mfma_half(half_of<1>(xf[sb][pt]), half_of<1>(f), u[pt][r]);
              }
            }
          }
        }
        const int row = 16 * r + col;
        const float di = s.dts[hw][row], dd = skip + di * s.od[hw][row];
#pragma unroll
        for (int pt = 0; pt < PT; ++pt) {
          const x4 yv = *row4(s.Y[hr], ov, 16 * r, v0 + 16 * pt);
          x4 z;
#pragma unroll
          for (int e = 0; e < 4; ++e) z[e] = from_f<T>(di * u[pt][r][e] + dd * to_f(yv[e]));
          buf_store8(rs, row * yb + (v0 + 16 * pt + 4 * g4) * (int)sizeof(T),
                     __builtin_bit_cast(u32x2, z));
        }
      }
    }
    __builtin_amdgcn_sched_barrier(0);
    if (!kEarly && more) request(c + 1, 0, kSplit ? 1 : HPW);
    if (kEarly && kSplit && more) request(c + 1, 1, HPW);
    if (RB < HPW && nh > 1) inter(HPW - 1);
    if (active)
      update_state<T, K, REV>(S, Q, ok, xf, REV ? s.eg[hw] : s.wt[hw], g4, s.decay[hw]);
    if (!kEarly && kSplit && more) request(c + 1, 1, HPW);
    if (kScaled) {
      const int e = exponent();
      if (l == 0) s.ex[w] = e;
    }
    if (w < nh && l < rows) {  // wave hh: head hh's sums
      const int blk = l >> 4;
      float v = 0.f, far = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (REV ? i >= blk : i <= blk) v += s.pe[w][sum_at<REV>(i, l)];
#pragma unroll
      for (int i = 0; i < WPH; ++i) far += s.pa[w * WPH + i][l];
      const int64_t o = (int64_t)(head0 + w) * ga.tokens + t + l;
      if (REV) {
        ga.q[o] = v;
        ga.far[o] = far;
        ga.own[o] = s.po[REV ? w : 0][l];
      } else {
        ga.row[o] = v + far;
      }
    }
    {
      const int row_bytes = a.G * K * (ga.slots == 1 ? (int)sizeof(T) : 4);
      const int64_t o = (t * a.G + grp) * K;
      char* base = ga.slots == 1
                       ? reinterpret_cast<char*>(reinterpret_cast<T*>(REV ? ga.dB : ga.dC) + o)
                       : reinterpret_cast<char*>((REV ? ga.part_dB : ga.part_dC) +
                                                 (int64_t)slot * ga.tokens * a.G * K + o);
      const auto rs = buf_rsrc(base, (int64_t)(rows - 1) * row_bytes + K * (ga.slots == 1 ? 2 : 4));
#pragma unroll
      for (int i = 0; i < TPW; ++i) {
        const int idx = wf * TPW + i, nt = idx >> 2, ab = idx & 3;
#pragma unroll
        for (int sb = 0; sb < 2; ++sb)
          if (REV ? sb >= (ab >> 1) : sb <= (ab >> 1)) {
            const x8 qf = tr_frag(Q, ok, 32 * sb, 16 * nt), wt = split_frag(s.W, om, 16 * ab, 32 * sb);
            // of the two tiles one may be beyond the diagonal
            if (!REV || 2 * sb >= ab) {
              const f32x4 w2 = mfma_half(half_of<0>(qf), *rest_of_w(ab, 2 * sb),
                                         mfma_half(half_of<0>(qf), half_of<0>(wt), kScaled ? zero4() : acc[i]));
              if constexpr (kScaled) acc[i] += w2 * s.wd[4 * ab + 2 * sb];
              else acc[i] = w2;
            }
            if (REV || 2 * sb + 1 <= ab) {
              const f32x4 w2 = mfma_half(half_of<1>(qf), *rest_of_w(ab, 2 * sb + 1),
                                         mfma_half(half_of<1>(qf), half_of<1>(wt), kScaled ? zero4() : acc[i]));
              if constexpr (kScaled) acc[i] += w2 * s.wd[4 * ab + 2 * sb + 1];
              else acc[i] = w2;
            }
          }
        const int off = (16 * ab + col) * row_bytes, k0 = 16 * nt + 4 * g4;
        if (ga.slots == 1) {
          const x4 z{from_f<T>(acc[i][0]), from_f<T>(acc[i][1]), from_f<T>(acc[i][2]),
                     from_f<T>(acc[i][3])};
          buf_store8(rs, off + 2 * k0, __builtin_bit_cast(u32x2, z));
        } else {
          buf_store16(rs, off + 4 * k0, __builtin_bit_cast(uint4, acc[i]));
        }
      }
    }
    __syncthreads();  // D: the tiles may be overwritten
    // every kMid chunks the forward walk's state meets the backward one's (here,
    // where the chunk's other registers are free)
    const int edge = REV ? nch - 1 - c : c + 1;
    if (ga.mid_state && active && edge % kMid == 0 && edge > 0 && edge < nch) {
      const int64_t at = (sg.t0 + 64ll * edge) / (64 * kMid) * a.H + h;
      const auto rs = buf_rsrc(ga.mid_state + at * KV + ct0 * (16 * K), 64ll * PT * K);
      float d = 0.f;
#pragma unroll
      for (int pt = 0; pt < PT; ++pt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const int off = 16 * lf + 1024 * (pt * NT + nt);
          if (REV) {
            const f32x4 v = __builtin_bit_cast(f32x4, buf_load16(rs, off));
#pragma unroll
            for (int e = 0; e < 4; ++e) d += S[pt][nt][e] * v[e];
          } else {
            buf_store16(rs, off, __builtin_bit_cast(uint4, S[pt][nt]));
          }
        }
      if (REV) {
        d = wave_sum(d);
        if (l == 0) ga.mid[at * 8 + w % WPH] = d;
      }
    }
  }

  // what spans the segment's end; the gradient of h0; dy . x
  if (REV) {
    if (active && ga.dh0 && sg.j == 0) {
#pragma unroll
      for (int pt = 0; pt < PT; ++pt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            ga.dh0[((int64_t)sg.n * a.H + h) * KV + state_at(ct0 + pt, nt, e, V)] = S[pt][nt][e];
    }
#pragma unroll
    for (int hh = 0; hh < HPW; ++hh) {
      const float d = wave_sum(dsum[hh]);
      if (l == 0) s.fin[hh][w] = d;
    }
  } else {
    float d = 0.f;
#pragma unroll
    for (int pt = 0; pt < PT; ++pt) {
      f32x4 E[NT];
      end_grad(pt, E);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) d += S[pt][nt][e] * E[nt][e];
    }
    d = wave_sum(d);
    if (l == 0) {
#pragma unroll
      for (int hh = 0; hh < HPW; ++hh) s.fin[hh][w] = hh == w / WPH ? d : 0.f;
    }
  }
  __syncthreads();
  if (threadIdx.x < (unsigned)nh) {
    float d = 0.f;
    for (int i = 0; i < NW; ++i) d += s.fin[threadIdx.x][i];
    (REV ? ga.part_dD : ga.span)[(int64_t)id * a.H + head0 + threadIdx.x] = d;
  }
}

}  // namespace

// Columns of a wave, in blocks of 16: 32 where two heads of V = 128 share a
// workgroup (16 waves of 16 columns would have 128 registers each).
template <int V, int HPW>
constexpr int kGradColumns = V == 128 && HPW == 2 ? 2 : 1;

template <typename T, int K, int V, int HPW, bool REV>
void launch_ssm_grad(const SsmGradArgs& a, unsigned grid, hipStream_t st) {
  constexpr int PT = kGradColumns<V, HPW>;
  GDR_LAUNCH(REV ? "ssm_grad_rev" : "ssm_grad_fwd", (ssm_grad_kernel<T, K, V, HPW, PT, REV>),
             dim3(grid), dim3(4 * HPW * V / PT), st, a);
}

#define GDR_INSTANTIATE(T, K, V)                                                            \
  template void launch_ssm_grad<T, K, V, 1, false>(const SsmGradArgs&, unsigned, hipStream_t); \
  template void launch_ssm_grad<T, K, V, 1, true>(const SsmGradArgs&, unsigned, hipStream_t);  \
  template void launch_ssm_grad<T, K, V, 2, false>(const SsmGradArgs&, unsigned, hipStream_t); \
  template void launch_ssm_grad<T, K, V, 2, true>(const SsmGradArgs&, unsigned, hipStream_t);

#endif  // GDR_SSM_GRAD_KERNELS

}  // namespace gdr

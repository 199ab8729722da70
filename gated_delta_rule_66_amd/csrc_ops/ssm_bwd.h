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
// r of E_ri = e^{g_{i+1} + .. + g_r} dt_i (C_r . B_i)(dy_r . x_i).  A pair
// counts with + in its row r and - in its column i, so dg is a suffix sum of
//     row_t - dt_t q_t,   row_r = sum_i E_ri,   q_i = x_i . u_i,
// plus, at a segment's end, the pairs that span it: <S_end, P_end>.  No state
// has to meet its gradient at every chunk, and none is stored: two walks, one
// forward with S, one backward with P, keep them in accumulators.
//   forward walk:  row_t = sum_{i <= t} (in the chunk) E_ti + e^{gamma_t} dy_t . S^T C_t
//                  dC    = diag(e^gamma) dY S^T + W B,   W = (dY X^T) o L diag(dt)
//   backward walk: u     = (C B^T o L)^T dY + diag(e^{gamma_end - gamma}) B P
//                  dB    = diag(dt e^{gamma_end - gamma}) X P^T + W^T C
// The scores' row and column sums are taken in fp32 before any rounding, and
// the state's share in them uses its 16-bit pair (hi + lo): the suffix sum
// adds rounding errors up, so these must be near fp32.  The other products
// round one operand (W, C B^T o L, S, P) to 16 bits, as their outputs are.
//
// One workgroup walks a segment for up to HPW heads of one group: they share
// the B and C tiles and C B^T, and their dB and dC are summed in registers.
// V / 16 waves, each with 16 state columns of every head; per chunk and head
// every wave also takes its share of dB's or dC's tiles, for which the states
// are passed through LDS once, rounded.
#pragma once

#include "ssm_device.h"

namespace gdr {

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
  float* row;           // [H][tokens]
  float* q;             // [H][tokens]
  float* span;          // [nids][H]: <S_end, P_end>
  float* part_dD;       // [nids][H]
  int slots;            // workgroups per group
  int64_t tokens;
};

constexpr int kGradHeads = 2;  // heads per workgroup, at most

template <typename T, int K, int V, int HPW, bool REV>
void launch_ssm_grad(const SsmGradArgs& a, unsigned grid, hipStream_t st);

#ifdef GDR_SSM_GRAD_KERNELS

namespace {

template <typename T, int K, int V>
struct GradSmem {
  T C[64 * K];
  T B[64 * K];
  T X[64 * V];
  T Y[64 * V];
  T R[V * K > 2 * 64 * 64 ? V * K : 2 * 64 * 64];  // state columns [V][K], then W and the scores
  float gam[2][64];  // in powers of two
  float eg[2][64], es[2][64], wt[2][64], dts[2][64], decay[2];
  float pe[4][64], pa[V / 16][64];
  int ex[kGradHeads][V / 16];
  float fin[kGradHeads][V / 16];
};

// The two walks are mirror images: with (P, Q, p, q) = (C, B, dY, X) forward
// and (B, C, X, dY) backward, a the token a result belongs to and b the one
// it sums over (b <= a forward, b >= a backward), both form the scores P_a .
// Q_b and p_a . q_b, the state's product with P and its dot with p, the
// gradient of P from the state and W, and update the state with Q^T q.
template <typename T, int K, int V, int HPW, bool REV>
__global__ __launch_bounds__(4 * V, K * V >= 8192 ? 2 : (V == 64 ? 3 : 4)) void ssm_grad_kernel(
    SsmGradArgs ga) {
  typedef typename VT<T>::x8 x8;
  typedef typename VT<T>::x4 x4;
  constexpr int NW = V / 16, NTH = 64 * NW, NT = K / 16, TPW = 4 * NT / NW;
  constexpr int MT = kMostTiles<NW>;
  constexpr bool kScaled = !__is_same(T, __bf16);
  __shared__ __align__(16) GradSmem<T, K, V> s;
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
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int l = lane_id();

  // start states: the forward walk's from the segment before (or h0), the
  // backward walk's from the segment after (or dht)
  f32x4 S[HPW][1][NT];
  const int64_t KV = (int64_t)K * V;
  auto load_slot = [&](const float* p, int id_, int h, f32x4* dst) {
    const float* src = p + ((int64_t)id_ * a.H + h) * KV;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
      dst[nt] = *reinterpret_cast<const f32x4*>(src + ((w * NT + nt) * 64 + l) * 4);
  };
  auto load_user = [&](const float* p, int h, f32x4* dst) {
    const float* src = p ? p + ((int64_t)sg.n * a.H + h) * KV : nullptr;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) dst[nt][e] = src ? src[state_at(w, nt, e, V)] : 0.f;
  };
  auto end_grad = [&](int h, f32x4* dst) {  // the state's gradient at the segment's end
    if (sg.j + 1 < sg.count) load_slot(ga.seg_grad, id + 1, h, dst);
    else load_user(ga.dht, h, dst);
  };
#pragma unroll
  for (int hh = 0; hh < HPW; ++hh) {
    if (hh < nh) {
      const int h = head0 + hh;
      if (REV) end_grad(h, S[hh][0]);
      else if (sg.j > 0) load_slot(a.seg_state, id - 1, h, S[hh][0]);
      else load_user(a.h0, h, S[hh][0]);
      if (kScaled) {
        const int e = state_exponent<NT>(S[hh][0]);
        if (l == 0) s.ex[hh][w] = e;
      }
    } else {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) S[hh][0][nt] = zero4();
    }
  }

  float rate[HPW], bias[HPW], skip[HPW], dsum[HPW];
#pragma unroll
  for (int hh = 0; hh < HPW; ++hh) {
    const int h = head0 + min(hh, nh - 1);
    rate[hh] = -expf(load_scalar(a.A_log, h, a.p_dtype));
    bias[hh] = param(a.dt_bias, h, a.p_dtype);
    skip[hh] = param(a.D, h, a.p_dtype);
    dsum[hh] = 0.f;
  }
  const T* xg = reinterpret_cast<const T*>(a.x) + (int64_t)head0 * V;
  const T* yg = reinterpret_cast<const T*>(ga.dy) + (int64_t)head0 * V;
  const T* bg = reinterpret_cast<const T*>(a.B) + (int64_t)grp * K;
  const T* cg = reinterpret_cast<const T*>(a.C) + (int64_t)grp * K;
  const int64_t ys = (int64_t)a.H * V;

  Rows64<T, K, NTH> rb, rc;
  Rows64<T, V, NTH> rx, ry;
  float raw = 0.f;
  const int nch = (int)((sg.t1 - sg.t0 + 63) / 64);
  auto token = [&](int c) { return sg.t0 + 64ll * (REV ? nch - 1 - c : c); };
  auto rows_of = [&](int64_t t) { return (int)min((int64_t)64, sg.t1 - t); };
  auto request_bc = [&](int c) {
    const int64_t t = token(c);
    rb.load(bg + t * a.bs, a.bs, rows_of(t));
    rc.load(cg + t * a.cs, a.cs, rows_of(t));
  };
  auto request_xy = [&](int c, int hh) {
    const int64_t t = token(c);
    rx.load(xg + t * a.xs + hh * V, a.xs, rows_of(t));
    ry.load(yg + t * ys + hh * V, ys, rows_of(t));
  };
  auto request_dt = [&](int c, int hh) {
    const int64_t t = token(c);
    raw = l < rows_of(t) ? load_scalar(a.dt, (t + l) * a.H + head0 + hh, a.dt_dtype) : 0.f;
  };
  auto gate = [&](int c, int hh, int b) {  // one token per lane
    const float step =
        l < rows_of(token(c)) ? ssm_step_size(raw, bias[hh], a.softplus) : 0.f;
    const float g = rate[hh] * step;
    const float gam = wave_prefix(g), es = __expf(wave_suffix_excl(g));
    s.gam[b][l] = gam * kLog2e;
    s.eg[b][l] = __expf(gam);
    s.es[b][l] = es;
    s.wt[b][l] = step * es;
    s.dts[b][l] = step;
    if (l == 0) s.decay[b] = __expf(lane_value(gam, 63));
  };
  if (nch > 0) {
    request_bc(0);
    request_xy(0, 0);
    if (w == NW - 1) {
      request_dt(0, 0);
      gate(0, 0, 0);
      if (nh > 1) request_dt(0, 1);
      else if (nch > 1) request_dt(1, 0);
    }
  }
  if (kScaled) __syncthreads();

  const T* P = REV ? s.B : s.C;
  const T* Q = REV ? s.C : s.B;
  const T* p = REV ? s.X : s.Y;
  const T* q = REV ? s.Y : s.X;
  T* const W = s.R;
  T* const GL = s.R + 64 * 64;
  Sw<K> ok;
  Sw<V> ov;
  Sw<64> om;
  int b = 0;  // the gate's buffer
  for (int c = 0; c < nch; ++c) {
    const int64_t t = token(c);
    const int rows = rows_of(t);
    f32x4 gt[MT], wsum[MT], acc[TPW];
#pragma unroll
    for (int k = 0; k < MT; ++k) gt[k] = wsum[k] = zero4();
#pragma unroll
    for (int i = 0; i < TPW; ++i) acc[i] = zero4();
#pragma unroll
    for (int hh = 0; hh < HPW; ++hh) {
      if (hh >= nh) continue;
      const bool last = hh + 1 == nh;
      const int lf = fresh_v(l), wf = fresh_s(w), g4 = lf >> 4, col = lf & 15, v0 = 16 * wf;
      ok.hide();
      ov.hide();
      om.hide();
      if (hh == 0) {
        rb.store(s.B);
        rc.store(s.C);
      }
      rx.store(s.X);
      ry.store(s.Y);
      // the state's columns, rounded, for the other waves
      float up = 1.f, down = 1.f;
      if (kScaled) {
        int e = s.ex[hh][0];
#pragma unroll
        for (int i = 1; i < NW; ++i) e = min(e, s.ex[hh][i]);
        up = ldexpf(1.f, e);
        down = ldexpf(1.f, -e);
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        x4 z;
#pragma unroll
        for (int e = 0; e < 4; ++e) z[e] = from_f<T>(kScaled ? S[hh][0][nt][e] * up : S[hh][0][nt][e]);
        *row4(s.R, ok, v0, 16 * nt) = z;
      }
      __syncthreads();  // A: tiles, gate and state columns are in LDS

      // scores (transposed: rows b, columns a), their sums over b, and W
      // summed over the heads
      f32x4 gl[MT];
#pragma unroll
      for (int k = 0; k < MT; ++k) {
        const int ti = tri_tile<NW>(wf, k);
        gl[k] = zero4();
        if (ti >= 0) {
          const int ab = REV ? ti & 3 : ti >> 2, bb = REV ? ti >> 2 : ti & 3;
          if (hh == 0) {
#pragma unroll
            for (int kb = 0; kb < K / 32; ++kb)
              gt[k] = mfma16(split_frag(Q, ok, 16 * bb, 32 * kb), split_frag(P, ok, 16 * ab, 32 * kb),
                             gt[k]);
          }
          f32x4 vt = zero4();
#pragma unroll
          for (int kv = 0; kv < V / 32; ++kv)
            vt = mfma16(split_frag(q, ov, 16 * bb, 32 * kv), split_frag(p, ov, 16 * ab, 32 * kv), vt);
          const int ia = 16 * ab + col, ib = 16 * bb + 4 * g4;
          const float gam_a = s.gam[b][ia], dt_a = s.dts[b][ia];
          const f32x4 gam_b = *reinterpret_cast<const f32x4*>(&s.gam[b][ib]);
          const f32x4 dt_b = *reinterpret_cast<const f32x4*>(&s.dts[b][ib]);
          float sum = 0.f;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const bool in = REV ? ib + e >= ia : ib + e <= ia;
            const float lx = exp2_fast(fminf(REV ? gam_b[e] - gam_a : gam_a - gam_b[e], 0.f));
            const float lm = in ? lx : 0.f;
            const float f = vt[e] * lm;
            const float fd = f * (REV ? dt_a : dt_b[e]);
            wsum[k][e] += fd;
            if (REV) {
              gl[k][e] = gt[k][e] * lm;
              sum += gt[k][e] * f;
              if (ib + e == ia) dsum[hh] += vt[e];
            } else {
              sum += gt[k][e] * fd;
            }
          }
          sum = sum4g(sum);
          if (g4 == 0) s.pe[bb][ia] = sum;
        }
        __builtin_amdgcn_sched_barrier(0);
      }

      // P's gradient, transposed: the state's part, rows k, columns a
      {
        const float* sc = REV ? s.wt[b] : s.eg[b];
        constexpr int PER = TPW < 4 ? TPW : 4;   // tiles that share the state's operand
#pragma unroll
        for (int j = 0; j < TPW / PER; ++j) {
          const int idx = wf * TPW + j * PER, nt = idx >> 2, a0 = idx & 3;
          f32x4 tmp[PER];
#pragma unroll
          for (int i = 0; i < PER; ++i) tmp[i] = zero4();
#pragma unroll
          for (int kv = 0; kv < V / 32; ++kv) {
            const x8 af = tr_frag(s.R, ok, 32 * kv, 16 * nt);
#pragma unroll
            for (int i = 0; i < PER; ++i)
              tmp[i] = mfma16(af, split_frag(p, ov, 16 * (a0 + i), 32 * kv), tmp[i]);
          }
#pragma unroll
          for (int i = 0; i < PER; ++i)
            acc[j * PER + i] += tmp[i] * (sc[16 * (a0 + i) + col] * down);
          __builtin_amdgcn_sched_barrier(0);
        }
      }

      // the state's product with P, its pair of operands, rows v, columns a;
      // its dot with p goes into a's sum
      f32x4 u[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) u[r] = zero4();
#pragma unroll
      for (int kb = 0; kb < K / 32; ++kb) {
        float v[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[e] = kScaled ? S[hh][0][2 * kb][e] * up : S[hh][0][2 * kb][e];
          v[4 + e] = kScaled ? S[hh][0][2 * kb + 1][e] * up : S[hh][0][2 * kb + 1][e];
        }
        x8 hi, lo;
        split8<T>(v, hi, lo);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const x8 f = split_frag(P, ok, 16 * r, 32 * kb);
          u[r] = mfma16(hi, f, u[r]);
          u[r] = mfma16(lo, f, u[r]);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        u[r] *= (REV ? s.es[b] : s.eg[b])[16 * r + col] * down;
        const x4 o = *row4(p, ov, 16 * r, v0);
        float dot = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) dot += u[r][e] * to_f(o[e]);
        dot = sum4g(dot);
        if (g4 == 0) s.pa[w][16 * r + col] = dot;
      }

      // the state's update
      x8 xf[2][1];
#pragma unroll
      for (int tb = 0; tb < 2; ++tb) xf[tb][0] = tr_frag(q, ov, 32 * tb, v0);
      update_state<T, K, 1>(S[hh], Q, ok, xf, REV ? s.eg[b] : s.wt[b], g4, s.decay[b]);
      __syncthreads();  // B: the state columns are read, the partial sums written

      if (!last) request_xy(c, hh + 1);
      else if (c + 1 < nch) request_xy(c + 1, 0);
      if (last && c + 1 < nch) request_bc(c + 1);
      if (kScaled) {
        const int e = state_exponent<NT>(S[hh][0]);
        if (l == 0) s.ex[hh][w] = e;
      }
      if (w == 0 && l < rows) {
        const int blk = l >> 4;
        float v = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (REV ? i >= blk : i <= blk) v += s.pe[i][l];
#pragma unroll
        for (int i = 0; i < NW; ++i) v += s.pa[i][l];
        (REV ? ga.q : ga.row)[(int64_t)(head0 + hh) * ga.tokens + t + l] = v;
      }
      if (last || REV) {
#pragma unroll
        for (int k = 0; k < MT; ++k) {
          const int ti = tri_tile<NW>(wf, k);
          if (ti >= 0) {
            const int ab = REV ? ti & 3 : ti >> 2, bb = REV ? ti >> 2 : ti & 3;
            x4 z;
            if (last) {
#pragma unroll
              for (int e = 0; e < 4; ++e) z[e] = from_f<T>(wsum[k][e]);
              *row4(W, om, 16 * ab, 16 * bb) = z;
            }
            if (REV) {
#pragma unroll
              for (int e = 0; e < 4; ++e) z[e] = from_f<T>(gl[k][e]);
              *row4(GL, om, 16 * ab, 16 * bb) = z;
            }
          }
        }
        // the tiles beyond the diagonal that the products read: (a, b) = (0, 1)
        // and (2, 3) forward, (1, 0) and (3, 2) backward
        for (int i = threadIdx.x; i < 128; i += NTH) {
          const int r0 = (i >> 6) * 32, ar = r0 + (REV ? 16 : 0) + ((i >> 2) & 15),
                    bc = r0 + (REV ? 0 : 16) + 4 * (i & 3);
          const x4 z{};
          *reinterpret_cast<x4*>(W + sw_off<64>(ar, bc)) = z;
          *reinterpret_cast<x4*>(GL + sw_off<64>(ar, bc)) = z;
        }
        __syncthreads();  // C: W and the decayed scores are in LDS

        if (last) {
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
              if (REV ? sb >= (ab >> 1) : sb <= (ab >> 1))
                acc[i] = mfma16(tr_frag(Q, ok, 32 * sb, 16 * nt), split_frag(W, om, 16 * ab, 32 * sb),
                                acc[i]);
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
        if (REV) {
          T* dx = reinterpret_cast<T*>(ga.dx) + t * ys + (int64_t)(head0 + hh) * V;
          const int yb = (int)ys * (int)sizeof(T);
          const auto rs = buf_rsrc(dx, (int64_t)(rows - 1) * yb + V * (int)sizeof(T));
#pragma unroll
          for (int r = 0; r < 4; ++r) {
#pragma unroll
            for (int sb = r >> 1; sb < 2; ++sb)
              u[r] = mfma16(xf[sb][0], split_frag(GL, om, 16 * r, 32 * sb), u[r]);
            const int row = 16 * r + col;
            const float di = s.dts[b][row];
            const x4 yv = *row4(s.Y, ov, 16 * r, v0);
            x4 z;
#pragma unroll
            for (int e = 0; e < 4; ++e) z[e] = from_f<T>(di * u[r][e] + skip[hh] * to_f(yv[e]));
            buf_store8(rs, row * yb + (v0 + 4 * g4) * (int)sizeof(T), __builtin_bit_cast(u32x2, z));
          }
        }
      }
      if (w == NW - 1) {  // the gate of the next head or chunk, whose dt is here already
        const int hn = last ? 0 : hh + 1, cn = last ? c + 1 : c;
        if (cn < nch) {
          gate(cn, last ? 0 : (hh + 1 < HPW ? hh + 1 : 0), b ^ 1);
          const int h2 = hn + 1 < nh ? hn + 1 : 0, c2 = hn + 1 < nh ? cn : cn + 1;
          if (c2 < nch) request_dt(c2, h2);
        }
      }
      b ^= 1;
      __syncthreads();  // D: the tiles may be overwritten
    }
  }

  // what spans the segment's end; the gradient of h0; dy . x
#pragma unroll
  for (int hh = 0; hh < HPW; ++hh) {
    if (hh >= nh) continue;
    const int h = head0 + hh;
    if (REV) {
      if (ga.dh0 && sg.j == 0) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e)
            ga.dh0[((int64_t)sg.n * a.H + h) * KV + state_at(w, nt, e, V)] = S[hh][0][nt][e];
      }
      const float d = wave_sum(dsum[hh]);
      if (l == 0) s.fin[hh][w] = d;
    } else {
      f32x4 E[NT];
      end_grad(h, E);
      float d = 0.f;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) d += S[hh][0][nt][e] * E[nt][e];
      d = wave_sum(d);
      if (l == 0) s.fin[hh][w] = d;
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

template <typename T, int K, int V, int HPW, bool REV>
void launch_ssm_grad(const SsmGradArgs& a, unsigned grid, hipStream_t st) {
  GDR_LAUNCH(REV ? "ssm_grad_rev" : "ssm_grad_fwd", (ssm_grad_kernel<T, K, V, HPW, REV>),
             dim3(grid), dim3(4 * V), st, a);
}

#define GDR_INSTANTIATE(T, K, V)                                                            \
  template void launch_ssm_grad<T, K, V, 1, false>(const SsmGradArgs&, unsigned, hipStream_t); \
  template void launch_ssm_grad<T, K, V, 1, true>(const SsmGradArgs&, unsigned, hipStream_t);  \
  template void launch_ssm_grad<T, K, V, 2, false>(const SsmGradArgs&, unsigned, hipStream_t); \
  template void launch_ssm_grad<T, K, V, 2, true>(const SsmGradArgs&, unsigned, hipStream_t);

#endif  // GDR_SSM_GRAD_KERNELS

}  // namespace gdr

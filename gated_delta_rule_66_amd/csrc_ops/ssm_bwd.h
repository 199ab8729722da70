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
  static constexpr int LK = K + 8, LV = V + 8, LM = 64 + 8;
  static constexpr int kR = V * LK > 2 * 64 * LM ? V * LK : 2 * 64 * LM;
  T C[64 * LK];
  T B[64 * LK];
  T X[64 * LV];
  T Y[64 * LV];
  T R[kR];  // a head's state columns [V][LK], then W and C B^T o L [64][LM]
  float gam[64], eg[64], es[64], wt[64], dts[64];
  float pe[4][64], pa[V / 16][64];
  int ex[kGradHeads][V / 16];
  float fin[2][V / 16];
};

// The ten tiles on or below the diagonal over NW waves, tile s of wave w
// (row block * 4 + column block), -1 past its share.
template <int NW>
__device__ __forceinline__ int grad_tile(int w, int s) {
  if (NW == 4) {
    constexpr uint64_t t = 0xC | (0xDull << 4) | (0x0ull << 8) | (0xEull << 12) | (0xFull << 16) |
                           (0x5ull << 20) | (0x8ull << 24) | (0x9ull << 28) | (0xAull << 36) |
                           (0x4ull << 40);
    return s < (w < 2 ? 3 : 2) ? (int)(t >> (12 * w + 4 * s)) & 15 : -1;
  }
  // eight waves: the first two take a second tile
  constexpr uint64_t t = 0xFEDCA984ull;             // waves 0 .. 7
  if (s == 0) return (int)(t >> (4 * w)) & 15;
  return s == 1 && w < 2 ? (w == 0 ? 0x0 : 0x5) : -1;
}

template <typename T, int K, int V, int HPW, bool REV>
__global__ __launch_bounds__(4 * V, V == 64 ? 2 : 1) void ssm_grad_kernel(SsmGradArgs ga) {
  typedef typename VT<T>::x8 x8;
  typedef typename VT<T>::x4 x4;
  typedef GradSmem<T, K, V> Smem;
  constexpr int LK = Smem::LK, LV = Smem::LV, LM = Smem::LM;
  constexpr int NW = V / 16, NTH = 64 * NW, NT = K / 16, TPW = 4 * NT / NW;
  constexpr int MT = NW == 4 ? 3 : 2;  // most tiles of a wave
  constexpr bool kScaled = !__is_same(T, __bf16);
  struct __attribute__((packed, aligned(sizeof(T)))) Raw8 {
    uint32_t u[2];
  };
  __shared__ Smem s;
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
  const int w = threadIdx.x >> 6, l = lane_id(), g4 = l >> 4, col = l & 15;
  const int v0 = 16 * w;

  // start states: the forward walk's from the segment before (or h0), the
  // backward walk's from the segment after (or dht)
  f32x4 S[HPW][NT];
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
      for (int e = 0; e < 4; ++e)
        dst[nt][e] = src ? src[(int64_t)state_k<V>(nt, e) * V + v0 + col] : 0.f;
  };
  auto end_grad = [&](int h, f32x4* dst) {  // the state's gradient at the segment's end
    if (sg.j + 1 < sg.count) load_slot(ga.seg_grad, id + 1, h, dst);
    else load_user(ga.dht, h, dst);
  };
  auto exponent = [&](const f32x4* p) {  // wave-wide: largest |S| 2^e in [2^13, 2^14)
    float m = 0.f;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int e = 0; e < 4; ++e) m = fmaxf(m, fabsf(p[nt][e]));
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) m = fmaxf(m, __shfl_xor(m, o, 64));
    const int e = 14 - __builtin_amdgcn_frexp_expf(m);
    return m > 0.f && m < __builtin_inff() ? min(max(e, -100), 100) : 100;
  };
#pragma unroll
  for (int hh = 0; hh < HPW; ++hh) {
    if (hh < nh) {
      const int h = head0 + hh;
      if (REV) end_grad(h, S[hh]);
      else if (sg.j > 0) load_slot(a.seg_state, id - 1, h, S[hh]);
      else load_user(a.h0, h, S[hh]);
      if (kScaled) {
        const int e = exponent(S[hh]);
        if (l == 0) s.ex[hh][w] = e;
      }
    } else {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) S[hh][nt] = zero4();
    }
  }
  if (kScaled) __syncthreads();

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
  auto request_bc = [&](int c) {
    const int64_t t = token(c);
    const int rows = (int)min((int64_t)64, sg.t1 - t);
    rb.load(bg + t * a.bs, a.bs, rows);
    rc.load(cg + t * a.cs, a.cs, rows);
  };
  auto request_xy = [&](int c, int hh) {
    const int64_t t = token(c);
    const int rows = (int)min((int64_t)64, sg.t1 - t);
    rx.load(xg + t * a.xs + hh * V, a.xs, rows);
    ry.load(yg + t * ys + hh * V, ys, rows);
    raw = l < rows ? load_scalar(a.dt, (t + l) * a.H + head0 + hh, a.dt_dtype) : 0.f;
  };
  if (nch > 0) {
    request_bc(0);
    request_xy(0, 0);
  }

  for (int c = 0; c < nch; ++c) {
    const int64_t t = token(c);
    const int rows = (int)min((int64_t)64, sg.t1 - t);
    f32x4 gt[MT], wsum[MT], acc[TPW];
#pragma unroll
    for (int k = 0; k < MT; ++k) gt[k] = wsum[k] = zero4();
#pragma unroll
    for (int i = 0; i < TPW; ++i) acc[i] = zero4();
#pragma unroll
    for (int hh = 0; hh < HPW; ++hh) {
      if (hh >= nh) continue;
      const bool last = hh + 1 == nh;
      // gate, one token per lane
      const float step = l < rows ? ssm_step_size(raw, bias[hh], a.softplus) : 0.f;
      const float g = rate[hh] * step;
      const float gam = wave_inclusive_scan(g), suf = wave_suffix_excl(g);
      const float decay = __expf(__shfl(gam, 63, 64));
      if (w == 0) {
        const float es = __expf(suf);
        s.gam[l] = gam;
        s.eg[l] = __expf(gam);
        s.es[l] = es;
        s.wt[l] = step * es;
        s.dts[l] = step;
      }
      if (hh == 0) {
        rb.store(s.B, LK);
        rc.store(s.C, LK);
      }
      rx.store(s.X, LV);
      ry.store(s.Y, LV);
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
      for (int kb = 0; kb < NT / 2; ++kb)
        *reinterpret_cast<x8*>(s.R + (v0 + col) * LK + 32 * kb + 8 * g4) =
            pack8<T>(S[hh][2 * kb] * up, S[hh][2 * kb + 1] * up);
      __syncthreads();  // A: tiles, gate and state columns are in LDS

      if (!last) request_xy(c, hh + 1);
      else if (c + 1 < nch) request_xy(c + 1, 0);
      if (hh == 0 && c + 1 < nch) request_bc(c + 1);

      // scores, their row or column sums, and W summed over the heads
      f32x4 gl[MT];
#pragma unroll
      for (int k = 0; k < MT; ++k) {
        const int ti = grad_tile<NW>(w, k);
        gl[k] = zero4();
        if (ti >= 0) {
          const int rbk = ti >> 2, cbk = ti & 3;
          if (hh == 0) {
#pragma unroll
            for (int kb = 0; kb < K / 32; ++kb)
              gt[k] = mfma16(frag_row(s.C + 16 * rbk * LK + 32 * kb, LK),
                             frag_row(s.B + 16 * cbk * LK + 32 * kb, LK), gt[k]);
          }
          f32x4 vt = zero4();
#pragma unroll
          for (int kv = 0; kv < V / 32; ++kv)
            vt = mfma16(frag_row(s.Y + 16 * rbk * LV + 32 * kv, LV),
                        frag_row(s.X + 16 * cbk * LV + 32 * kv, LV), vt);
          const int i = 16 * cbk + col;
          const float gi = s.gam[i], di = s.dts[i];
          float cs = 0.f;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int r = 16 * rbk + 4 * g4 + e;
            const float lm = r >= i ? __expf(s.gam[r] - gi) : 0.f;
            const float f = vt[e] * lm;
            wsum[k][e] += f * di;
            if (REV) {
              gl[k][e] = gt[k][e] * lm;
              cs += gt[k][e] * f;
              if (r == i) dsum[hh] += vt[e];
            } else {
              const float rs = sum16(gt[k][e] * f * di);
              if (col == 0) s.pe[cbk][r] = rs;
            }
          }
          if (REV) {
            cs = sum4g(cs);
            if (g4 == 0) s.pe[rbk][i] = cs;
          }
        }
      }

      // dC^T (dB^T): the state's part, rows k, columns t
      {
        const T* rows_lds = REV ? s.X : s.Y;
        const float* sc = REV ? s.wt : s.eg;
        constexpr int PER = TPW < 4 ? TPW : 4;   // tiles that share a column of the state
#pragma unroll
        for (int q = 0; q < TPW / PER; ++q) {
          const int idx = w * TPW + q * PER, nt = idx >> 2, rb0 = idx & 3;
          f32x4 tmp[PER];
#pragma unroll
          for (int i = 0; i < PER; ++i) tmp[i] = zero4();
#pragma unroll
          for (int kv = 0; kv < V / 32; ++kv) {
            const x8 af = frag_tr(s.R + 32 * kv * LK + 16 * nt, LK);
#pragma unroll
            for (int i = 0; i < PER; ++i)
              tmp[i] = mfma16(af, frag_row(rows_lds + 16 * (rb0 + i) * LV + 32 * kv, LV), tmp[i]);
          }
#pragma unroll
          for (int i = 0; i < PER; ++i)
            acc[q * PER + i] += tmp[i] * (sc[16 * (rb0 + i) + col] * down);
        }
      }

      // S^T C^T (P^T B^T) with the state's pair, rows v, columns t; its dot
      // with dy (x) goes into the row (column) sums
      f32x4 u[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) u[r] = zero4();
#pragma unroll
      for (int kb = 0; kb < NT / 2; ++kb) {
        float v[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[e] = S[hh][2 * kb][e] * up;
          v[4 + e] = S[hh][2 * kb + 1][e] * up;
        }
        x8 hi, lo;
        split8<T>(v, hi, lo);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const x8 f = frag_row((REV ? s.B : s.C) + 16 * r * LK + 32 * kb, LK);
          u[r] = mfma16(hi, f, u[r]);
          u[r] = mfma16(lo, f, u[r]);
        }
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int row = 16 * r + col;
        u[r] *= (REV ? s.es : s.eg)[row] * down;
        const x4 o = *reinterpret_cast<const x4*>((REV ? s.X : s.Y) + row * LV + v0 + 4 * g4);
        float dot = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) dot += u[r][e] * to_f(o[e]);
        dot = sum4g(dot);
        if (g4 == 0) s.pa[w][row] = dot;
      }

      // the state's update
      x8 xf[2];
      {
        const T* src = REV ? s.Y : s.X;
        const T* mat = REV ? s.C : s.B;
        float wt[2][8];
        float m = 0.f;
#pragma unroll
        for (int tb = 0; tb < 2; ++tb) {
          xf[tb] = frag_tr(src + 32 * tb * LV + v0, LV);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            wt[tb][e] = (REV ? s.eg : s.wt)[32 * tb + 8 * g4 + e];
            if (kScaled) m = fmaxf(m, fabsf(to_f(xf[tb][e]) * wt[tb][e]));
          }
        }
        const float scale = kScaled ? ldexpf(1.f, column_exponent(m)) : 1.f;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) S[hh][nt] *= decay * scale;
#pragma unroll
        for (int tb = 0; tb < 2; ++tb) {
          float v[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] = to_f(xf[tb][e]) * wt[tb][e] * scale;
          x8 hi, lo;
          split8<T>(v, hi, lo);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            const x8 bf = frag_tr_pair(mat + 32 * tb * LK + 32 * (nt >> 1) + 4 * (nt & 1), LK);
            S[hh][nt] = mfma16(bf, hi, S[hh][nt]);
            S[hh][nt] = mfma16(bf, lo, S[hh][nt]);
          }
        }
        if (kScaled) {
          const float back = 1.f / scale;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) S[hh][nt] *= back;
        }
      }
      __syncthreads();  // B: the state columns are read, the partial sums written

      if (kScaled) {
        const int e = exponent(S[hh]);
        if (l == 0) s.ex[hh][w] = e;
      }
      if (threadIdx.x < 64 && l < rows) {
        const int blk = l >> 4;
        float v = 0.f;
#pragma unroll
        for (int b = 0; b < 4; ++b)
          if (REV ? b >= blk : b <= blk) v += s.pe[b][l];
#pragma unroll
        for (int b = 0; b < NW; ++b) v += s.pa[b][l];
        (REV ? ga.q : ga.row)[(int64_t)(head0 + hh) * ga.tokens + t + l] = v;
      }
      if (last || REV) {
        T* W = s.R;
        T* GL = s.R + 64 * LM;
#pragma unroll
        for (int k = 0; k < MT; ++k) {
          const int ti = grad_tile<NW>(w, k);
          if (ti >= 0) {
            const int o = (16 * (ti >> 2) + 4 * g4) * LM + 16 * (ti & 3) + col;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              if (last) W[o + e * LM] = from_f<T>(wsum[k][e]);
              if (REV) GL[o + e * LM] = from_f<T>(gl[k][e]);
            }
          }
        }
        // the tiles above the diagonal that the products read: (0, 1), (2, 3)
        for (int i = threadIdx.x; i < 512; i += NTH) {
          const int o = ((i >> 8) * 32 + ((i >> 4) & 15)) * LM + (i >> 8) * 32 + 16 + (i & 15);
          W[o] = (T)0.f;
          GL[o] = (T)0.f;
        }
        __syncthreads();  // C: W and C B^T o L are in LDS

        if (last) {
#pragma unroll
          for (int i = 0; i < TPW; ++i) {
            const int idx = w * TPW + i, nt = idx >> 2, blk = idx & 3;
            if (!REV) {
              for (int ib = 0; ib <= (blk >> 1); ++ib)
                acc[i] = mfma16(frag_tr(s.B + 32 * ib * LK + 16 * nt, LK),
                                frag_row(W + 16 * blk * LM + 32 * ib, LM), acc[i]);
            } else {
              for (int rk = blk >> 1; rk < 2; ++rk)
                acc[i] = mfma16(frag_tr(s.C + 32 * rk * LK + 16 * nt, LK),
                                frag_tr(W + 32 * rk * LM + 16 * blk, LM), acc[i]);
            }
            const int row = 16 * blk + col;
            if (row < rows) {
              const int64_t o = ((t + row) * a.G + grp) * K + 16 * nt + 4 * g4;
              if (ga.slots == 1) {
                x4 z{from_f<T>(acc[i][0]), from_f<T>(acc[i][1]), from_f<T>(acc[i][2]),
                     from_f<T>(acc[i][3])};
                *reinterpret_cast<Raw8*>(reinterpret_cast<T*>(REV ? ga.dB : ga.dC) + o) =
                    __builtin_bit_cast(Raw8, z);
              } else {
                float* p = (REV ? ga.part_dB : ga.part_dC) + (int64_t)slot * ga.tokens * a.G * K + o;
                *reinterpret_cast<f32x4*>(p) = acc[i];
              }
            }
          }
        }
        if (REV) {
          T* dx = reinterpret_cast<T*>(ga.dx) + t * ys + (int64_t)(head0 + hh) * V;
#pragma unroll
          for (int r = 0; r < 4; ++r) {
#pragma unroll
            for (int rk = r >> 1; rk < 2; ++rk)
              u[r] = mfma16(xf[rk], frag_tr(GL + 32 * rk * LM + 16 * r, LM), u[r]);
            const int row = 16 * r + col;
            if (row < rows) {
              const float di = s.dts[row];
              const x4 yv = *reinterpret_cast<const x4*>(s.Y + row * LV + v0 + 4 * g4);
              x4 z;
#pragma unroll
              for (int e = 0; e < 4; ++e) z[e] = from_f<T>(di * u[r][e] + skip[hh] * to_f(yv[e]));
              *reinterpret_cast<Raw8*>(dx + row * ys + v0 + 4 * g4) = __builtin_bit_cast(Raw8, z);
            }
          }
        }
      }
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
            ga.dh0[((int64_t)sg.n * a.H + h) * KV + (int64_t)state_k<V>(nt, e) * V + v0 + col] =
                S[hh][nt][e];
      }
      const float d = wave_sum(dsum[hh]);
      if (l == 0) s.fin[hh][w] = d;
    } else {
      f32x4 P[NT];
      end_grad(h, P);
      float d = 0.f;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) d += S[hh][nt][e] * P[nt][e];
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

// ssm_fwd.hip -- the selective state space scan on gfx950: prompts chunk by
// chunk on matrix instructions, single tokens on cached states.
//
// A prompt moves 4 V bytes of x and y per token and head (16 bits) and needs
// about 2 K V multiply-adds, 5 K V with the pairs and triples that keep the
// state exact: on this card memory and the matrix units take about the same
// time, and few heads leave CUs idle.  So sequences are cut into segments until
// the launch fills the chip: one walk forms what every segment but the last
// adds to the state (reads x and B only), ssm_combine_kernel adds these up
// along each sequence, and a second walk goes through each segment from its
// start state.
//
// Measured at 65,536 tokens, 32 heads in 8 groups, K = 128, V = 64, bf16: the
// state walk 133 us for 402 MB (3.0 TB/s; 104 us with the update left out), the
// outputs' 280 us for 841 MB, the sums in between 17 us.  Both walks are
// bound by their loads and, little less, by the vector and matrix
// instructions of the update; two chunks in flight instead of one took as long.
#include <algorithm>
#include <cmath>

#include "ssm_device.h"

namespace gdr {

namespace {

template <typename T, int K, int V, int HPW, bool OUT>
struct WalkSmem {
  T C[OUT ? 64 * K : 0];
  T B[64 * K];
  T X[64 * HPW * V];
  T M[OUT ? HPW : 0][64 * 64];
  float md[OUT && !__is_same(T, __bf16) ? HPW : 0][4];  // fp16: what undoes the scales of M's column blocks
  float od[OUT ? HPW : 0][64];                          // what rounding took from M's diagonal
  float gam[HPW][2][64];  // in powers of two
  float eg[HPW][2][64], wt[HPW][2][64], dts[HPW][2][64], decay[HPW][2];
};

// kOut: the segment's outputs from its start state.  kState: what it adds to
// the state.  kGrad: what it adds to the state's gradient at its start, the
// same with dy and C for x and B (the caller passes them so), e^gamma for the
// weights, and the chunks from the last to the first.
//
// A workgroup walks HPW heads of one group, which share the B and C tiles and
// the scores C B^T; each wave holds 16 PT columns of one head's state in
// accumulators and reads every operand of B and C once for them: 32 columns
// for outputs, whose LDS reads count (65,536 tokens as above: 437 us with 16,
// 384 with 32), 16 for states, where twice the waves hide more latency
// (136 us with 32, 133 with 16).  Per chunk,
// the tiles of the next one are in registers (in flight), those of this one
// in LDS, swizzled so that operands are read as fast as linear rows (LDS is
// active 29 % of the outputs' time, a third of that for conflicts, and 20 % of
// the states', without any); the last waves, which have the fewest score tiles,
// form the next chunk's gates.
enum { kOut, kState, kGrad };
template <typename T, int K, int V, int HPW, int PT, int MODE>
__global__ __launch_bounds__(4 * HPW * V / PT, MODE != kOut ? 4 : HPW * PT == 1 ? 3 : 2) void ssm_walk_kernel(SsmArgs a) {
  typedef typename VT<T>::x8 x8;
  typedef typename VT<T>::x4 x4;
  constexpr int NW = HPW * V / (16 * PT), WPH = NW / HPW, NTH = 64 * NW, NT = K / 16;
  constexpr int XC = HPW * V;  // columns of the x tile
  constexpr bool OUT = MODE == kOut;
  constexpr bool kScaled = !__is_same(T, __bf16);
  static_assert(!OUT || NW == 4, "each wave forms one column of score tiles");
  __shared__ __align__(16) WalkSmem<T, K, V, HPW, OUT> s;
  const int R = a.H / a.G, slots = (R + HPW - 1) / HPW;
  const int L = xcd_order(blockIdx.x, gridDim.x);
  const int part = L % slots, grp_h = L / slots % a.G, id = L / (slots * a.G);
  const int head0 = grp_h * R + part * HPW, nh = min(HPW, R - part * HPW);
  const Segment sg = segment_of(a, id);
  if (sg.count == 0) return;
  if (MODE == kState && sg.j + 1 >= sg.count) return;
  if (MODE == kGrad && sg.j == 0) return;
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), l = lane_id();
  const int hw = w / WPH, ct0 = w % WPH * PT, h = head0 + min(hw, nh - 1);
  const bool active = hw < nh;

  const T* xg = reinterpret_cast<const T*>(a.x) + (int64_t)head0 * V;
  const T* bg = reinterpret_cast<const T*>(a.B) + (int64_t)grp_h * K;
  const T* cg = reinterpret_cast<const T*>(a.C) + (int64_t)grp_h * K;
  const float skip = param(a.D, h, a.p_dtype);
  // the head whose gate this wave forms, if it is one of the last waves
  const int gh = NW - 1 - w, ghead = head0 + min(gh, nh - 1);
  const bool gates = gh < nh;
  const float rate = -expf(load_scalar(a.A_log, ghead, a.p_dtype));
  const float bias = param(a.dt_bias, ghead, a.p_dtype);

  f32x4 S[PT][NT];
  const int64_t unit = ((int64_t)sg.n * a.H + h) * K * V;
  const int64_t slot = ((int64_t)id * a.H + h) * K * V;
#pragma unroll
  for (int pt = 0; pt < PT; ++pt) {
    if (OUT && sg.j > 0) {
      const float* src = a.seg_state + slot - (int64_t)a.H * K * V;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        S[pt][nt] = *reinterpret_cast<const f32x4*>(src + (((ct0 + pt) * NT + nt) * 64 + l) * 4);
    } else {
      const bool from = OUT && a.h0;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          S[pt][nt][e] = from ? a.h0[unit + state_at(ct0 + pt, nt, e, V)] : 0.f;
    }
  }
  if (OUT) {  // tiles above the diagonal that the product with M reads: (0, 1) and (2, 3)
    for (int i = threadIdx.x; i < 512 * HPW; i += NTH) {
      const int k = i & 511;
      s.M[i >> 9][sw_off<64>((k >> 8) * 32 + ((k >> 4) & 15), (k >> 8) * 32 + 16 + (k & 15))] =
          (T)0.f;
    }
  }

  const int nch = (int)((sg.t1 - sg.t0 + 63) / 64);
  auto token = [&](int c) { return sg.t0 + 64ll * (MODE == kGrad ? nch - 1 - c : c); };
  auto rows_of = [&](int64_t t) { return (int)min((int64_t)64, sg.t1 - t); };
  Rows64<T, K, NTH> rb, rc;
  Rows64<T, XC, NTH> rx;
  float raw = 0.f, total = 0.f;
  auto request = [&](int64_t t) {
    const int rows = rows_of(t);
    rx.load(xg + t * a.xs, a.xs, rows, nh * V);
    rb.load(bg + t * a.bs, a.bs, rows);
    if (OUT) rc.load(cg + t * a.cs, a.cs, rows);
  };
  auto request_dt = [&](int64_t t) {
    raw = l < rows_of(t) ? load_scalar(a.dt, (t + l) * a.H + ghead, a.dt_dtype) : 0.f;
  };
  // a chunk's gate, one token per lane; tokens past the end have step size 0
  auto gate = [&](int64_t t, int b) {
    const float step = l < rows_of(t) ? ssm_step_size(raw, bias, a.softplus) : 0.f;
    const float g = rate * step;
    const float gam = wave_prefix(g);
    const float all = lane_value(gam, 63);
    total += all;
    s.gam[gh][b][l] = gam * kLog2e;
    s.eg[gh][b][l] = __expf(gam);
    s.wt[gh][b][l] = MODE == kGrad ? __expf(gam) : step * __expf(wave_suffix_excl(g));
    s.dts[gh][b][l] = step;
    if (l == 0) s.decay[gh][b] = __expf(all);
  };
  if (nch > 0) {
    request(token(0));
    if (gates) {
      request_dt(token(0));
      gate(token(0), 0);
      if (nch > 1) request_dt(token(1));
    }
  }

  Sw<K> ok;
  Sw<XC> ov;
  Sw<64> om;
  for (int c = 0; c < nch; ++c) {
    const int64_t t = token(c);
    const int b = c & 1;
    const int lf = fresh_v(l), wf = fresh_s(w), g4 = lf >> 4, col = lf & 15;
    const int hf = wf / WPH, v0 = hf * V + wf % WPH * (16 * PT);  // column in the x tile
    ok.hide();
    ov.hide();
    om.hide();
    rx.store(s.X);
    rb.store(s.B);
    if (OUT) rc.store(s.C);
    __syncthreads();
    if (c + 1 < nch) request(token(c + 1));

    f32x4 acc[PT][4];
    if (OUT) {
      // The state's part of the output, transposed (rows v, columns t), and
      // the scores of the wave's column block of tokens: they share C's
      // operands.
      f32x4 sc[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        sc[r] = zero4();
#pragma unroll
        for (int pt = 0; pt < PT; ++pt) acc[pt][r] = zero4();
      }
      float up = 1.f, down = 1.f;
      if (kScaled) {
        int e = state_exponent<NT>(S[0]);
#pragma unroll
        for (int pt = 1; pt < PT; ++pt) e = min(e, state_exponent<NT>(S[pt]));
        up = ldexpf(1.f, e);
        down = ldexpf(1.f, -e);
      }
      const int cb = wf;  // wave w: the score tiles of column block w, on and below the diagonal
#pragma unroll
      for (int kb = 0; kb < K / 32; ++kb) {
        x8 sf[PT];
#pragma unroll
        for (int pt = 0; pt < PT; ++pt)
          sf[pt] = kScaled ? pack_split<T>(S[pt][2 * kb] * up, S[pt][2 * kb + 1] * up)
                           : pack_split<T>(S[pt][2 * kb], S[pt][2 * kb + 1]);
        const x8 bf = split_frag(s.B, ok, 16 * cb, 32 * kb);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const x8 cf = split_frag(s.C, ok, 16 * r, 32 * kb);
#pragma unroll
          for (int pt = 0; pt < PT; ++pt) acc[pt][r] = mfma16(sf[pt], cf, acc[pt][r]);
          sc[r] = mfma16(bf, cf, sc[r]);  // needed or not: branches would cut the schedule up
        }
        if (PT > 1 || kb % 2 == 1) __builtin_amdgcn_sched_barrier(0);
      }
      // M = (C B^T) o L diag(dt), rounded to T as an operand; its tiles are
      // transposed, so that a lane holds four neighbours of a row
      const int i = 16 * cb + 4 * g4;
      auto put_m = [&](int hh, int r, int c, f32x4 v, f32x4 scaled, float back) {
        const x4 z = round4<T>(scaled);
        *row4(s.M[hh], om, 16 * r, 16 * c) = z;
        if (r == c && g4 == col >> 2) {
          float d = 0.f;
#pragma unroll
          for (int e = 0; e < 4; ++e) d += 4 * g4 + e == col ? v[e] - to_f(z[e]) * back : 0.f;
          s.od[hh][16 * r + col] = d;
        }
      };
#pragma unroll
      for (int hh = 0; hh < HPW; ++hh) {
        if (hh >= nh) continue;
        const f32x4 gi = *reinterpret_cast<const f32x4*>(&s.gam[hh][b][i]);
        const f32x4 di = *reinterpret_cast<const f32x4*>(&s.dts[hh][b][i]);
        f32x4 o[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          if (kScaled) o[r] = zero4();
          if (r >= cb) {
            const int row = 16 * r + col;
            const float gr = s.gam[hh][b][row];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float v = sc[r][e] * exp2_fast(gr - gi[e]) * di[e];
              o[r][e] = row >= i + e ? v : 0.f;
            }
            if (!kScaled) put_m(hh, r, cb, o[r], o[r], 1.f);
          }
        }
        if constexpr (kScaled) {
          float back;
          const float scale = tile_scale(
              fmaxf(fmaxf(largest4(o[0]), largest4(o[1])), fmaxf(largest4(o[2]), largest4(o[3]))), back);
          if (l == 0) s.md[hh][cb] = back;
#pragma unroll
          for (int r = 0; r < 4; ++r)
            if (r >= cb) put_m(hh, r, cb, o[r], o[r] * scale, back);
        }
      }
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const float eg = s.eg[hf][b][16 * r + col] * down;
#pragma unroll
        for (int pt = 0; pt < PT; ++pt) acc[pt][r] *= eg;
      }
      __syncthreads();
    }

    if (active) {
      // x^T fragments serve the product with M and, weighted, the state's
      // update; with fp16 the state's columns are scaled while it is added
      x8 xf[2][PT];
#pragma unroll
      for (int tb = 0; tb < 2; ++tb)
#pragma unroll
        for (int pt = 0; pt < PT; ++pt) xf[tb][pt] = tr_frag(s.X, ov, 32 * tb, v0 + 16 * pt);
      if (OUT) {
#pragma unroll
        for (int tb = 0; tb < 2; ++tb)
#pragma unroll
          for (int r = 2 * tb; r < 4; ++r) {
            const x8 mf = split_frag(s.M[hf], om, 16 * r, 32 * tb);
#pragma unroll
            for (int pt = 0; pt < PT; ++pt) {
              if constexpr (kScaled) {
                acc[pt][r] = mfma_tile<0>(xf[tb][pt], mf, s.md[hf][2 * tb], acc[pt][r]);
                if (2 * tb + 1 <= r)
                  acc[pt][r] = mfma_tile<1>(xf[tb][pt], mf, s.md[hf][2 * tb + 1], acc[pt][r]);
              } else {
                acc[pt][r] = mfma16(xf[tb][pt], mf, acc[pt][r]);
              }
            }
          }
        __builtin_amdgcn_sched_barrier(0);
      }
      if (OUT) {
        T* y = reinterpret_cast<T*>(a.y) + (t * a.H + head0) * V;
        const int ys = a.H * V * (int)sizeof(T);
        const auto rs = buf_rsrc(y, (int64_t)(rows_of(t) - 1) * ys + nh * V * (int)sizeof(T));
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int row = 16 * r + col;
          const float dd = skip + s.od[hf][row];
#pragma unroll
          for (int pt = 0; pt < PT; ++pt) {
            const x4 xv = *row4(s.X, ov, 16 * r, v0 + 16 * pt);
            x4 o;
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] = from_f<T>(acc[pt][r][e] + dd * to_f(xv[e]));
            buf_store8(rs, row * ys + (v0 + 16 * pt + 4 * g4) * (int)sizeof(T),
                       __builtin_bit_cast(u32x2, o));
          }
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      update_state<T, K, true>(S, s.B, ok, xf, s.wt[hf][b], g4, s.decay[hf][b]);
    }
    if (gates && c + 1 < nch) {
      gate(token(c + 1), b ^ 1);
      if (c + 2 < nch) request_dt(token(c + 2));
    }
    __syncthreads();
  }

  if (!active && !(gates && !OUT)) return;
  if (!OUT) {
    if (gates && l == 0) a.seg_decay[(int64_t)id * a.H + ghead] = total;
    if (!active) return;
    float* dst = a.seg_state + slot;
#pragma unroll
    for (int pt = 0; pt < PT; ++pt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
        *reinterpret_cast<f32x4*>(dst + (((ct0 + pt) * NT + nt) * 64 + l) * 4) = S[pt][nt];
  } else if (a.ht && sg.j + 1 == sg.count) {
#pragma unroll
    for (int pt = 0; pt < PT; ++pt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          a.ht[unit + state_at(ct0 + pt, nt, e, V)] = S[pt][nt][e];
  }
}

// The walk's shape: V = 64 takes two heads of a group at once (32 columns a
// wave) where a group has two (65,536 tokens, 32 heads in 8 groups, K = 128:
// outputs 268 us, states 133; with one head a workgroup 303 and 150); V = 128
// one head on four waves of 32 columns.
int walk_heads(const gdr_ssm_problem* p) { return p->V == 64 && p->H / p->G >= 2 ? 2 : 1; }
template <int MODE>
void launch_walk(const gdr_ssm_problem* p, const SsmArgs& a, const char* name, hipStream_t st) {
  const int R = p->H / p->G, heads = walk_heads(p);
  const dim3 grid((unsigned)((int64_t)a.nids * p->G * ((R + heads - 1) / heads)));
  ssm_by_shape(p, [&](auto t, auto k, auto v) {
    using T = decltype(t);
    constexpr int K = k.value, V = v.value, PT = MODE == kOut ? 2 : 1;
    if constexpr (V == 128) {
      GDR_LAUNCH(name, (ssm_walk_kernel<T, K, V, 1, PT, MODE>), grid, dim3(512 / PT), st, a);
    } else {
      if (heads == 2)
        GDR_LAUNCH(name, (ssm_walk_kernel<T, K, V, 2, PT, MODE>), grid, dim3(512 / PT), st, a);
      else
        GDR_LAUNCH(name, (ssm_walk_kernel<T, K, V, 1, 1, MODE>), grid, dim3(256), st, a);
    }
  });
}

// Segment j's end state over what it added, E_j = e^{decay_j} E_{j-1} +
// add_j with E_{-1} the initial state, for all but the last segment; REV: the
// state's gradient at segment j's start, F_j = e^{decay_j} F_{j+1} + add_j
// with F past the last segment the final state's gradient, for all but the
// first.  One thread walks four state elements along the sequence.  Bound by
// the states' bytes, read and written once: 57 MB each way in 20 us (5.8 TB/s).
template <int K, int V, bool REV>
__global__ __launch_bounds__(256) void ssm_combine_kernel(SsmArgs a) {
  constexpr int parts = K * V / 1024;
  const int part = blockIdx.x % parts;
  const int u = blockIdx.x / parts, n = u / a.H, h = u % a.H;
  int id0;
  int64_t len;
  if (a.cu) {
    id0 = n + a.cu[n] / a.seg;
    len = a.cu[n + 1] - a.cu[n];
  } else {
    id0 = n * ((a.T + a.seg - 1) / a.seg);
    len = a.T;
  }
  const int m = (int)((len + a.seg - 1) / a.seg);
  if (m < 2) return;
  const int at = (part * 256 + threadIdx.x) * 4;      // element in the register order
  f32x4 E = zero4();
  if (a.h0) {
    // register order: [16-column tile][nt][lane][e]
    constexpr int NT = K / 16;
    const int lane = (at >> 2) & 63, q = at >> 8, nt = q % NT, ct = q / NT;
    const int v = 16 * ct + (lane & 15);
    const int k = 16 * nt + 4 * (lane >> 4);
#pragma unroll
    for (int e = 0; e < 4; ++e) E[e] = a.h0[((int64_t)n * a.H + h) * K * V + (int64_t)(k + e) * V + v];
  }
  const int first = REV ? id0 + m - 1 : id0;
  const int64_t dir = REV ? -1 : 1, step = dir * a.H * K * V;
  float* p = a.seg_state + ((int64_t)first * a.H + h) * K * V + at;
  const float* dec = a.seg_decay + (int64_t)first * a.H + h;
  // eight segments' loads at a time: the chain itself is a few operations
  for (int j = 0; j + 1 < m; j += 8) {
    f32x4 add[8];
    float d[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (j + i + 1 < m) {
        add[i] = *reinterpret_cast<const f32x4*>(p + i * step);
        d[i] = dec[dir * (j + i) * a.H];
      }
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (j + i + 1 < m) {
        E = E * __expf(d[i]) + add[i];
        *reinterpret_cast<f32x4*>(p + i * step) = E;
      }
    p += 8 * step;
  }
}

// Single tokens (or a few) on a cached state: 256 threads hold 32 columns of
// one head's state, read once and written once; thread (c, r) has columns
// 4 c .. 4 c + 3 of rows r, r + 32, ...  The state's bytes bound it: 256
// sequences of 32 heads with K = V = 128 take 211 us for 1.08 GB (5.1 TB/s, a
// large copy's rate), one sequence with V = 64 takes 4 us.
template <typename T, int K, int V>
__global__ __launch_bounds__(256) void ssm_step_kernel(SsmArgs a) {
  constexpr int R = K / 32;
  __shared__ f32x4 red[2][4][8];
  const int blocks = V / 32;
  const int vb = blockIdx.x % blocks, u = blockIdx.x / blocks, n = u / a.H, h = u % a.H;
  const int grp_h = h / (a.H / a.G);
  const int c = threadIdx.x & 7, r = threadIdx.x >> 3, w = threadIdx.x >> 6;
  const int64_t base = ((int64_t)n * a.H + h) * K * V + 32 * vb + 4 * c;
  int64_t t0, t1;
  if (a.cu) {
    t0 = a.cu[n];
    t1 = a.cu[n + 1];
  } else {
    t0 = (int64_t)n * a.T;
    t1 = t0 + a.T;
  }
  f32x4 S[R];
#pragma unroll
  for (int i = 0; i < R; ++i)
    S[i] = a.h0 ? *reinterpret_cast<const f32x4*>(a.h0 + base + (int64_t)(r + 32 * i) * V) : zero4();
  const float rate = -expf(load_scalar(a.A_log, h, a.p_dtype));
  const float bias = param(a.dt_bias, h, a.p_dtype), skip = param(a.D, h, a.p_dtype);
  const T* xg = reinterpret_cast<const T*>(a.x) + (int64_t)h * V + 32 * vb + 4 * c;
  const T* bg = reinterpret_cast<const T*>(a.B) + (int64_t)grp_h * K + r;
  const T* cg = reinterpret_cast<const T*>(a.C) + (int64_t)grp_h * K + r;
  T* yg = reinterpret_cast<T*>(a.y) + (int64_t)h * V + 32 * vb + 4 * c;
  for (int64_t t = t0; t < t1; ++t) {
    const float step = ssm_step_size(load_scalar(a.dt, t * a.H + h, a.dt_dtype), bias, a.softplus);
    const float decay = __expf(rate * step);
    f32x4 x, y = zero4();
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = to_f(xg[t * a.xs + e]);
#pragma unroll
    for (int i = 0; i < R; ++i) {
      const float b = step * to_f(bg[t * a.bs + 32 * i]), q = to_f(cg[t * a.cs + 32 * i]);
      S[i] = S[i] * decay + b * x;
      y += q * S[i];
    }
    // over the 8 row groups of the wave, then over the waves
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float v = y[e];
      v += __shfl_xor(v, 8, 64);
      v = sum4g(v);
      y[e] = v;
    }
    const int par = (int)(t & 1);
    if ((threadIdx.x & 63) < 8) red[par][w][c] = y;
    __syncthreads();
    if (threadIdx.x < 8) {
      const f32x4 o = (red[par][0][c] + red[par][1][c]) + (red[par][2][c] + red[par][3][c]);
#pragma unroll
      for (int e = 0; e < 4; ++e) yg[t * a.H * V + e] = from_f<T>(o[e] + skip * x[e]);
    }
  }
  if (a.ht) {
#pragma unroll
    for (int i = 0; i < R; ++i)
      *reinterpret_cast<f32x4*>(a.ht + base + (int64_t)(r + 32 * i) * V) = S[i];
  }
}

}  // namespace

SsmArgs ssm_args(const gdr_ssm_problem* p, const SsmPlan& pl) {
  SsmArgs a{};
  a.cu = p->cu_seqlens_dev;
  a.xs = p->x_stride;
  a.bs = p->b_stride;
  a.cs = p->c_stride;
  a.N = p->N;
  a.T = p->T;
  a.H = p->H;
  a.G = p->G;
  a.seg = pl.seg;
  a.nids = pl.nids;
  a.dt_dtype = (int)p->dt_dtype;
  a.p_dtype = (int)p->p_dtype;
  a.softplus = p->dt_softplus;
  return a;
}

// How sequences are cut for a launch with `per_seg` workgroups for each
// segment, of which `slots` run at once: the segment length, in chunks, of
// least cost.  Workgroups run in rounds of `slots`; a round takes its
// segments' chunks and about 1.5 chunks for the states at both ends, a last
// round that fills a share f of the slots (0.45 + 0.55 f) of that (a CU's
// workgroups share its units.  Outputs, K = 128, V = 64, bf16: of one head one
// workgroup alone takes 4.3 us a chunk, two 6.4, three 8.4; of two heads one
// takes 6.2 and two 8.9; fp16 up to 1 more).  Cut, every chunk's x and B are read
// once more for 0.4 of a chunk, and two launches are added, worth about four
// chunks.
SsmPlan ssm_plan(const gdr_ssm_problem* p, int64_t per_seg, int64_t slots) {
  int64_t longest = 0, tokens = 0;
  const int seqs = p->cu_seqlens_host ? p->N : 1;
  auto chunks_of = [&](int n) {
    const int64_t len = p->cu_seqlens_host
                            ? (int64_t)p->cu_seqlens_host[n + 1] - p->cu_seqlens_host[n]
                            : p->T;
    return (len + 63) / 64;
  };
  for (int n = 0; n < seqs; ++n) longest = std::max(longest, chunks_of(n));
  if (p->cu_seqlens_host) tokens = p->T;
  longest = std::max<int64_t>(1, longest);
  const int64_t copies = p->cu_seqlens_host ? 1 : p->B;
  auto rounds = [&](double wgs) {
    const double full = std::floor(wgs / slots), f = wgs / slots - full;
    return full + (f > 0.0 ? 0.45 + 0.55 * f : 0.0);
  };
  // every length up to 32 chunks, then steps of about an eighth, and no cut
  int64_t best_sc = longest;
  double best = 1e300;
  for (int64_t sc = std::min<int64_t>(4, longest);;) {
    int64_t segs = 0, work = 0;
    for (int n = 0; n < seqs; ++n) {
      const int64_t c = chunks_of(n);
      segs += std::max<int64_t>(1, (c + sc - 1) / sc);
      work += c;
    }
    const double wgs = (double)(segs * copies * per_seg);
    const bool cut = sc < longest;
    // unequal segments: no shorter than the longest, no less than the work
    const double mean = (double)work / (double)segs;
    const double r = rounds(wgs);
    const double one = std::max((double)sc, r * mean) + 1.5 * std::max(1.0, r);
    const double cost = (r <= 1.0 ? r * (sc + 1.5) : one) * (cut ? 1.4 : 1.0) + (cut ? 4.0 : 0.0);
    if (cost < best) {
      best = cost;
      best_sc = sc;
    }
    if (sc == longest) break;
    // (of many sequences fewer lengths: each costs the host a look at all of them)
    sc = std::min(longest, seqs > 64 ? sc + sc / 2 : sc < 32 ? sc + 1 : sc + sc / 8);
  }
  SsmPlan pl;
  pl.split = best_sc < longest;
  pl.seg = (int)(best_sc * 64);
  pl.nids = p->cu_seqlens_host ? (int)(p->N + tokens / pl.seg)
                               : (int)(p->B * ((p->T + (int64_t)pl.seg - 1) / pl.seg));
  return pl;
}

SsmPlan ssm_fwd_plan(const gdr_ssm_problem* p) {
  if (p->keep_states) return ssm_grad_cut(p);
  const int R = p->H / p->G, heads = walk_heads(p);
  return ssm_plan(p, (int64_t)p->G * ((R + heads - 1) / heads), p->V == 64 && heads == 1 ? 768 : 512);
}

size_t ssm_fwd_workspace(const gdr_ssm_problem* p, const SsmPlan& pl) {
  if (!pl.split) return 0;
  return align256((size_t)pl.nids * p->H * p->K * p->V * sizeof(float)) +
         align256((size_t)pl.nids * p->H * sizeof(float));
}

// Every segment's end states (grad: the gradients at its start) in
// a.seg_state; for the gradient a holds dy, C and dht for x, B and h0.
void launch_ssm_states(const gdr_ssm_problem* p, const SsmArgs& a, bool grad, hipStream_t st) {
  if (grad) launch_walk<kGrad>(p, a, "ssm_state_grad", st);
  else launch_walk<kState>(p, a, "ssm_state", st);
  ssm_by_shape(p, [&](auto, auto k, auto v) {
    constexpr int K = k.value, V = v.value;
    const dim3 grid((unsigned)((int64_t)p->N * p->H * (K * V / 1024)));
    if (grad) GDR_LAUNCH("ssm_combine", (ssm_combine_kernel<K, V, true>), grid, dim3(256), st, a);
    else GDR_LAUNCH("ssm_combine", (ssm_combine_kernel<K, V, false>), grid, dim3(256), st, a);
  });
}

gdr_status launch_ssm_fwd(const gdr_ssm_problem* p, const SsmPlan& pl, const void* x,
                          const void* dt, const void* A_log, const void* B, const void* C,
                          const void* D, const void* dt_bias, const float* h0, void* y, float* ht,
                          void* ws, hipStream_t st) {
  SsmArgs a = ssm_args(p, pl);
  a.x = x; a.dt = dt; a.A_log = A_log; a.B = B; a.C = C; a.D = D; a.dt_bias = dt_bias;
  a.h0 = h0; a.y = y; a.ht = ht;
  if (pl.split) {
    a.seg_state = reinterpret_cast<float*>(ws);
    a.seg_decay = reinterpret_cast<float*>(
        reinterpret_cast<char*>(ws) + align256((size_t)pl.nids * p->H * p->K * p->V * sizeof(float)));
  }
  if (pl.split) launch_ssm_states(p, a, false, st);
  launch_walk<kOut>(p, a, "ssm_out", st);
  return launch_status("ssm_fwd");
}

gdr_status launch_ssm_step(const gdr_ssm_problem* p, const void* x, const void* dt,
                           const void* A_log, const void* B, const void* C, const void* D,
                           const void* dt_bias, const float* h0, void* y, float* ht,
                           hipStream_t st) {
  SsmArgs a = ssm_args(p, SsmPlan{64, 0, false});
  a.x = x; a.dt = dt; a.A_log = A_log; a.B = B; a.C = C; a.D = D; a.dt_bias = dt_bias;
  a.h0 = h0; a.y = y; a.ht = ht;
  ssm_by_shape(p, [&](auto t, auto k, auto v) {
    constexpr int K = k.value, V = v.value;
    GDR_LAUNCH("ssm_step", (ssm_step_kernel<decltype(t), K, V>),
               dim3((unsigned)((int64_t)p->N * p->H * (V / 32))), dim3(256), st, a);
  });
  return launch_status("ssm_step");
}

}  // namespace gdr

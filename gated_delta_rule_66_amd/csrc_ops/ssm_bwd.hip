// ssm_bwd.hip -- the selective scan's gradient: the step sizes' part, the sums
// over segments and workgroups, and the launches (the walks: ssm_bwd.h).
#include <algorithm>

#include "ssm_bwd.h"

namespace gdr {

namespace {

// Sums over the 16 lanes of a chunk: of the lanes behind, of the lanes before.
__device__ __forceinline__ float behind16(float x) {
  x = dpp_zero<0x101>(x);
  x += dpp_zero<0x101>(x);
  x += dpp_zero<0x102>(x);
  x += dpp_zero<0x104>(x);
  return x + dpp_zero<0x108>(x);
}
__device__ __forceinline__ float before16(float x) {
  x = dpp_zero<0x111>(x);
  x += dpp_zero<0x111>(x);
  x += dpp_zero<0x112>(x);
  x += dpp_zero<0x114>(x);
  return x + dpp_zero<0x118>(x);
}
__device__ __forceinline__ double wave_sum2(double v) {
#pragma unroll
  for (int m = 1; m < 64; m *= 2) v += __shfl_xor(v, m, 64);
  return v;
}

// dg from the walks' sums (ssm_bwd.h), the raw step sizes' gradient and the
// segment's shares of dA_log and ddt_bias.  One workgroup per (segment, head),
// 16 chunks at a time from the end, four tokens per thread: sums inside a chunk
// in fp32, the chain over the chunks and the shares in 64 bits.  12 us for 8192
// tokens of 32 heads: latency, and reads of dt one head apart.
template <typename DT>
__global__ __launch_bounds__(256) void ssm_dt_kernel(SsmGradArgs ga, DT* ddt, float* part_dA,
                                                     float* part_db) {
  __shared__ float ends[16], begins[16], spans[16];
  __shared__ int how[16];  // 0: from the chunk behind, 1: nothing spans the chunk, 2: from a kept state
  __shared__ double red[2][4];
  const SsmArgs& a = ga.f;
  const int id = blockIdx.x / a.H, h = blockIdx.x % a.H;
  const Segment sg = segment_of(a, id);
  const int64_t out = (int64_t)id * a.H + h;
  if (sg.count == 0) {
    if (threadIdx.x == 0) part_dA[out] = part_db[out] = 0.f;
    return;
  }
  const int l = lane_id(), w = threadIdx.x >> 6, c = threadIdx.x >> 4, i16 = threadIdx.x & 15;
  const float rate = -expf(load_scalar(a.A_log, h, a.p_dtype));
  const float bias = param(a.dt_bias, h, a.p_dtype);
  const int64_t first = (int64_t)h * ga.tokens;
  const int64_t len = sg.t1 - sg.t0;
  const int nch = (int)((len + 63) / 64);
  double chain = ga.span[out], dA = 0.0, db = 0.0;
  for (int64_t b = (len - 1) / 1024; b >= 0; --b) {
    const int64_t t0 = sg.t0 + 1024 * b + 4 * threadIdx.x;
    const int edge = (int)(16 * b) + c + 1;  // the chunk ends where chunk `edge` begins
    float raw[4], step[4], u[4], sum[4], pre[4], g = 0.f;
#pragma unroll
    for (int e = 3; e >= 0; --e) {
      const bool live = t0 + e < sg.t1;
      const int64_t o = first + t0 + e;
      raw[e] = live ? load_scalar(a.dt, (t0 + e) * a.H + h, a.dt_dtype) : 0.f;
      step[e] = live ? ssm_step_size(raw[e], bias, a.softplus) : 0.f;
      const float q = live ? ga.q[o] : 0.f, far = live ? ga.far[o] : 0.f;
      u[e] = (q + far) + (live ? ga.own[o] : 0.f);
      sum[e] = (live ? ga.row[o] - step[e] * q : 0.f) + (e < 3 ? sum[e < 3 ? e + 1 : 3] : 0.f);
      pre[e] = step[e] * far;
      g += rate * step[e];
    }
    const float here = (pre[0] + pre[1]) + (pre[2] + pre[3]);
    const float behind = behind16(sum[0]), before = before16(here);
    const bool kept = ga.mid_state && edge % kMid == 0 && edge < nch;
    float mid = 0.f;
    if (kept && i16 < ga.mid_parts)
      mid = ga.mid[((sg.t0 + 64ll * edge) / (64 * kMid) * a.H + h) * 8 + i16];
    mid = sum16(mid);
    g = sum16(g);
    if (i16 == 0) {
      ends[c] = behind + sum[0];
      spans[c] = mid;
      how[c] = g < -24.f ? 1 : kept ? 2 : 0;
    }
    if (i16 == 15) begins[c] = before + here;
    __syncthreads();
    float over = 0.f;  // what spans this thread's chunk
#pragma unroll
    for (int i = 15; i >= 0; --i) {
      if (how[i] == 2) chain = spans[i];
      chain = how[i] == 1 ? 0.0 : chain - begins[i];
      if (i == c) over = (float)chain;
      chain += ends[i];
    }
    float prefix = before;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (t0 + e < sg.t1) {
        const float dg = over + prefix + (behind + sum[e]);
        float d = rate * dg + u[e];
        if (a.softplus) d *= sigmoid(raw[e] + bias);
        ddt[(t0 + e) * a.H + h] = from_f<DT>(d);
        dA += (double)dg * (rate * step[e]);
        db += d;
      }
      prefix += pre[e];
    }
    __syncthreads();
  }
  dA = wave_sum2(dA);
  db = wave_sum2(db);
  if (l == 0) {
    red[0][w] = dA;
    red[1][w] = db;
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    part_dA[out] = (float)((red[0][0] + red[0][1]) + (red[0][2] + red[0][3]));
    part_db[out] = (float)((red[1][0] + red[1][1]) + (red[1][2] + red[1][3]));
  }
}

// The parameters' gradients over all segments: one workgroup per head and
// parameter (A_log, dt_bias, D).
__global__ __launch_bounds__(256) void ssm_param_kernel(const float* part, int64_t stride, int nids,
                                                        int H, void* dA, void* db, void* dD,
                                                        int dtype) {
  __shared__ float red[4];
  const int which = blockIdx.x / H, h = blockIdx.x % H;
  void* out = which == 0 ? dA : which == 1 ? db : dD;
  if (!out) return;
  const float* p = part + which * stride + h;
  float v = 0.f;
  for (int64_t i = threadIdx.x; i < nids; i += 256) v += p[i * H];
  v = wave_sum(v);
  if (lane_id() == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  if (threadIdx.x == 0) store_scalar(out, h, dtype, (red[0] + red[1]) + (red[2] + red[3]));
}

// dB and dC over a group's workgroups, in order, four values per thread.
// Bound by the partial sums' bytes: 8192 tokens, 4 groups of 8 heads (four
// workgroups each), K = 128, 134 MB, take 29 us.
template <typename T>
__global__ __launch_bounds__(256) void ssm_group_kernel(const float* pB, const float* pC, int slots,
                                                        int64_t n, T* dB, T* dC) {
  struct __attribute__((packed, aligned(sizeof(T)))) Raw {
    uint32_t u[2];
  };
  for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4; i < 2 * n;
       i += (int64_t)gridDim.x * 1024) {
    const bool second = i >= n;
    const int64_t k = second ? i - n : i;
    const float* p = (second ? pC : pB) + k;
    f32x4 v = *reinterpret_cast<const f32x4*>(p);
    for (int s = 1; s < slots; ++s) v += *reinterpret_cast<const f32x4*>(p + s * n);
    const typename VT<T>::x4 o{from_f<T>(v[0]), from_f<T>(v[1]), from_f<T>(v[2]), from_f<T>(v[3])};
    *reinterpret_cast<Raw*>((second ? dC : dB) + k) = __builtin_bit_cast(Raw, o);
  }
}

// Heads per workgroup (those of one group share its B, C and C B^T and add
// their dB, dC in registers), workgroups per group and the cut.  A pair of
// heads fills a CU (8192 tokens, 32 heads, K = V = 128: 502 us for the whole
// gradient step with segments for 256 workgroups, 569 for 512); one head at
// V = 64 leaves room for two (K = 64: 273 us for 512, 350 for 256).
struct GradPlan {
  int heads, slots;
  SsmPlan cut;
};
GradPlan grad_plan(const gdr_ssm_problem* p) {
  GradPlan g;
  const int R = p->H / p->G;
  g.heads = R >= 2 ? 2 : 1;
  g.slots = (R + g.heads - 1) / g.heads;
  g.cut = ssm_plan(p, (int64_t)p->G * g.slots, g.heads == 1 && p->V == 64 ? 512 : 256);
  return g;
}

// Byte offsets in the workspace.
struct GradLayout {
  size_t state, grad, sdec, gdec, row, q, far, own, mid_state, mid, span, params, pB, pC, total;
};
GradLayout layout(const gdr_ssm_problem* p, const GradPlan& g) {
  GradLayout o{};
  const size_t tokens = (size_t)p->B * p->T, ids = (size_t)g.cut.nids * p->H;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += align256(bytes);
    return here;
  };
  if (g.cut.split) {
    if (!p->keep_states) {
      o.state = take(ids * p->K * p->V * sizeof(float));
      o.sdec = take(ids * sizeof(float));
    }
    o.grad = take(ids * p->K * p->V * sizeof(float));
    o.gdec = take(ids * sizeof(float));
  }
  o.row = take(tokens * p->H * sizeof(float));
  o.q = take(tokens * p->H * sizeof(float));
  o.far = take(tokens * p->H * sizeof(float));
  o.own = take(tokens * p->H * sizeof(float));
  if (g.cut.seg > 64 * kMid) {
    const size_t edges = (tokens / (64 * kMid) + 1) * p->H;
    o.mid_state = take(edges * p->K * p->V * sizeof(float));
    o.mid = take(edges * 8 * sizeof(float));
  }
  o.span = take(ids * sizeof(float));
  o.params = take(3 * ids * sizeof(float));
  if (g.slots > 1) {
    o.pB = take(tokens * p->G * p->K * g.slots * sizeof(float));
    o.pC = take(tokens * p->G * p->K * g.slots * sizeof(float));
  }
  o.total = at;
  return o;
}

}  // namespace

SsmPlan ssm_grad_cut(const gdr_ssm_problem* p) { return grad_plan(p).cut; }

size_t ssm_bwd_workspace(const gdr_ssm_problem* p) { return layout(p, grad_plan(p)).total; }

gdr_status launch_ssm_bwd(const gdr_ssm_problem* p, const void* x, const void* dt,
                          const void* A_log, const void* B, const void* C, const void* D,
                          const void* dt_bias, const void* dy, const float* dht, const float* h0,
                          const void* kept, void* dx, void* ddt, void* dA_log, void* dB, void* dC, void* dD,
                          void* ddt_bias, float* dh0, void* ws, hipStream_t st) {
  const GradPlan g = grad_plan(p);
  const GradLayout o = layout(p, g);
  char* base = reinterpret_cast<char*>(ws);
  auto f32 = [&](size_t off) { return reinterpret_cast<float*>(base + off); };
  SsmGradArgs a{};
  a.f = ssm_args(p, g.cut);
  a.f.x = x; a.f.dt = dt; a.f.A_log = A_log; a.f.B = B; a.f.C = C; a.f.D = D; a.f.dt_bias = dt_bias;
  a.f.h0 = h0;
  if (g.cut.split) {
    if (p->keep_states) {
      a.f.seg_state = reinterpret_cast<float*>(const_cast<void*>(kept));  // only read
    } else {
      a.f.seg_state = f32(o.state);
      a.f.seg_decay = f32(o.sdec);
      launch_ssm_states(p, a.f, false, st);
    }
    SsmArgs r = a.f;
    r.x = dy; r.xs = (int64_t)p->H * p->V;
    r.B = C; r.bs = p->c_stride;
    r.h0 = dht;
    r.seg_state = f32(o.grad);
    r.seg_decay = f32(o.gdec);
    launch_ssm_states(p, r, true, st);
    a.seg_grad = r.seg_state;
  }
  const int64_t ids = (int64_t)g.cut.nids * p->H;
  float* params = f32(o.params);
  a.dy = dy; a.dht = dht; a.dx = dx; a.dB = dB; a.dC = dC; a.dh0 = dh0;
  if (g.slots > 1) {
    a.part_dB = f32(o.pB);
    a.part_dC = f32(o.pC);
  }
  a.row = f32(o.row);
  a.q = f32(o.q);
  a.far = f32(o.far);
  a.own = f32(o.own);
  if (g.cut.seg > 64 * kMid) {
    a.mid_state = f32(o.mid_state);
    a.mid = f32(o.mid);
  }
  a.mid_parts = p->V == 128 && g.heads == 1 ? 8 : 4;
  a.span = f32(o.span);
  a.part_dD = params + 2 * ids;
  a.slots = g.slots;
  a.tokens = (int64_t)p->B * p->T;
  const unsigned grid = (unsigned)((int64_t)g.cut.nids * p->G * g.slots);
  ssm_by_shape(p, [&](auto t, auto k, auto v) {
    using T = decltype(t);
    constexpr int K = k.value, V = v.value;
    if (g.heads == 2) {
      launch_ssm_grad<T, K, V, 2, false>(a, grid, st);
      launch_ssm_grad<T, K, V, 2, true>(a, grid, st);
    } else {
      launch_ssm_grad<T, K, V, 1, false>(a, grid, st);
      launch_ssm_grad<T, K, V, 1, true>(a, grid, st);
    }
    const dim3 dgrid((unsigned)ids);
    if (p->dt_dtype == GDR_FP32)
      GDR_LAUNCH("ssm_dt", (ssm_dt_kernel<float>), dgrid, dim3(256), st, a,
                 reinterpret_cast<float*>(ddt), params, params + ids);
    else
      GDR_LAUNCH("ssm_dt", (ssm_dt_kernel<T>), dgrid, dim3(256), st, a, reinterpret_cast<T*>(ddt),
                 params, params + ids);
    if (g.slots > 1) {
      const int64_t n = a.tokens * p->G * K;
      GDR_LAUNCH("ssm_group", (ssm_group_kernel<T>), dim3((unsigned)std::min<int64_t>((2 * n / 4 + 255) / 256, 1 << 20)),
                 dim3(256), st, a.part_dB, a.part_dC, g.slots, n, reinterpret_cast<T*>(dB),
                 reinterpret_cast<T*>(dC));
    }
  });
  GDR_LAUNCH("ssm_param", ssm_param_kernel, dim3(3 * p->H), dim3(256), st, params, ids, g.cut.nids,
             p->H, dA_log, ddt_bias, dD, (int)p->p_dtype);
  return launch_status("ssm_bwd");
}

}  // namespace gdr

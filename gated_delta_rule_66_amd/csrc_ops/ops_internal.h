// ops_internal.h -- host-side interface between the C ABI of the layer
// operators (short convolution, selective scan, residual RMS norm, gated and
// sandwich norm, rows and products in 8 bits) and their launchers.
#pragma once

#include "../csrc/gdr_internal.h"

namespace gdr {

// GDR_LAUNCH with `lds` bytes (up to 64 KiB) that the kernel declares extern.
#define GDR_LAUNCH_LDS(name, kernel, grid, block, lds, st, ...)        \
  do {                                                                 \
    if (::gdr::g_profiling) ::gdr::profile_begin(st, name);            \
    hipLaunchKernelGGL(kernel, grid, block, lds, st, __VA_ARGS__);     \
    if (::gdr::g_profiling) ::gdr::profile_end(st);                    \
  } while (0)

// Launch failures become a status; `what` names the operator.
gdr_status launch_status(const char* what);

// --- short causal convolution (conv1d.hip) ---
size_t conv_bwd_workspace(const gdr_conv_problem* p);
gdr_status launch_conv_fwd(const gdr_conv_problem* p, const void* x, const void* weight,
                           const void* bias, const void* s0, void* y, void* s1, hipStream_t st);
gdr_status launch_conv_bwd(const gdr_conv_problem* p, const void* x, const void* weight,
                           const void* bias, const void* dy, const void* ds1, const void* s0,
                           void* dx, void* dw, void* db, void* ds0, void* ws, hipStream_t st);
gdr_status launch_conv_update(const gdr_conv_problem* p, const void* x, void* state,
                              const void* weight, const void* bias, void* y, hipStream_t st);

// --- residual RMS norm (rms_norm.hip) ---
size_t norm_bwd_workspace(const gdr_norm_problem* p);
gdr_status launch_norm_fwd(const gdr_norm_problem* p, const void* x, const void* res,
                           const void* weight, void* y, void* scale, void* h, float* rstd,
                           hipStream_t st);
gdr_status launch_norm_bwd(const gdr_norm_problem* p, const void* dy, const void* h,
                           const void* weight, const float* rstd, const void* dh_out, void* dx,
                           void* dres, void* dw, void* ws, hipStream_t st);

// out[c] = the sum of part[r][c] over the rows, in a fixed order.
void launch_reduce_rows(const float* part, int rows, int cols, void* out, int dtype,
                        hipStream_t st);

// --- gated RMS norm (gated_norm.hip) ---
// threads of the forward's launch (the gradient's is bounded)
int64_t gated_norm_threads(const gdr_gated_norm_problem* p);
gdr_status launch_gated_norm_fwd(const gdr_gated_norm_problem* p, const void* x, const void* gate,
                                 const void* weight, void* y, float* scale, float* rstd,
                                 hipStream_t st);
size_t gated_norm_bwd_workspace(const gdr_gated_norm_problem* p);
gdr_status launch_gated_norm_bwd(const gdr_gated_norm_problem* p, const void* dy, const void* x,
                                 const void* gate, const void* weight, const float* rstd, void* dx,
                                 void* dgate, void* dweight, void* ws, hipStream_t st);

// --- sandwich RMS norm (sandwich_norm.hip) ---
int64_t sandwich_norm_threads(const gdr_sandwich_norm_problem* p);  // the forward's
gdr_status launch_sandwich_norm_fwd(const gdr_sandwich_norm_problem* p, const void* x,
                                    const void* residual, const void* gate, const void* post,
                                    const void* res_scale, const void* pre, void* y, float* scale,
                                    void* h, float* rstd_x, float* rstd_h, hipStream_t st);
size_t sandwich_norm_bwd_workspace(const gdr_sandwich_norm_problem* p);
gdr_status launch_sandwich_norm_bwd(const gdr_sandwich_norm_problem* p, const void* dy,
                                    const void* dh, const void* x, const void* h, const void* gate,
                                    const void* post, const void* res_scale, const void* pre,
                                    const float* rstd_x, const float* rstd_h, void* dx,
                                    void* dresidual, void* dgate, void* dpost, void* dscale,
                                    void* dpre, void* ws, hipStream_t st);

// --- rows and products in 8 bits (quantize.hip, int8_matmul.hip) ---
gdr_status launch_quantize_rows(const gdr_quantize_problem* p, const void* x, void* q, float* scale,
                                hipStream_t st);
size_t int8_matmul_workspace(const gdr_int8_matmul_problem* p);
gdr_status launch_int8_matmul(const gdr_int8_matmul_problem* p, const void* x, const float* x_scale,
                              const void* w, const float* w_scale, const void* bias, void* y,
                              void* ws, hipStream_t st);

// --- selective state space scan (ssm_fwd.hip, ssm_bwd.hip) ---
struct SsmPlan {
  int seg;     // tokens per segment, a multiple of 64
  int nids;    // segment ids
  bool split;  // some sequence has more than one segment
};
SsmPlan ssm_plan(const gdr_ssm_problem* p, int64_t per_seg, int64_t slots);
SsmPlan ssm_fwd_plan(const gdr_ssm_problem* p);
SsmPlan ssm_grad_cut(const gdr_ssm_problem* p);
size_t ssm_fwd_workspace(const gdr_ssm_problem* p, const SsmPlan& pl);
gdr_status launch_ssm_fwd(const gdr_ssm_problem* p, const SsmPlan& pl, const void* x,
                          const void* dt, const void* A_log, const void* B, const void* C,
                          const void* D, const void* dt_bias, const float* h0, void* y, float* ht,
                          void* ws, hipStream_t st);
gdr_status launch_ssm_step(const gdr_ssm_problem* p, const void* x, const void* dt,
                           const void* A_log, const void* B, const void* C, const void* D,
                           const void* dt_bias, const float* h0, void* y, float* ht,
                           hipStream_t st);

size_t ssm_bwd_workspace(const gdr_ssm_problem* p);
gdr_status launch_ssm_bwd(const gdr_ssm_problem* p, const void* x, const void* dt,
                          const void* A_log, const void* B, const void* C, const void* D,
                          const void* dt_bias, const void* dy, const float* dht, const float* h0,
                          const void* kept, void* dx, void* ddt, void* dA_log, void* dB, void* dC, void* dD,
                          void* ddt_bias, float* dh0, void* ws, hipStream_t st);

}  // namespace gdr

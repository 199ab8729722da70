// ops_internal.h -- host-side interface between the C ABI of the layer
// operators (short convolution, selective scan, residual RMS norm) and their
// launchers.
#pragma once

#include "../csrc/gdr_internal.h"

namespace gdr {

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

// ops_api.cpp -- the C ABI of the layer operators: argument validation and
// workspace sizes.  Host code; validation finishes before the first HIP call.
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <cstring>

#include "ops_internal.h"

namespace gdr {

static gdr_status fail(gdr_status s, char* reason, size_t len, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  set_error("%s", buf);
  if (reason && len) {
    strncpy(reason, buf, len - 1);
    reason[len - 1] = '\0';
  }
  return s;
}

static bool is_type(gdr_dtype d) { return d == GDR_BF16 || d == GDR_FP16 || d == GDR_FP32; }
static bool is_flag(int32_t v) { return v == 0 || v == 1; }

// Sequences: B dense rows of T tokens, or N packed ones in [0, T).
static gdr_status check_seqs(int B, int T, int N, const int32_t* dev, const int32_t* host,
                             char* reason, size_t len) {
  if ((dev != nullptr) != (host != nullptr))
    return fail(GDR_ERR_VARLEN, reason, len, "cu_seqlens needs both the device and the host copy");
  if (!dev) {
    if (N != B) return fail(GDR_ERR_SHAPE, reason, len, "dense input needs N == B (N=%d B=%d)", N, B);
    return GDR_OK;
  }
  if (B != 1) return fail(GDR_ERR_VARLEN, reason, len, "packed input needs B == 1, got %d", B);
  if (N < 1) return fail(GDR_ERR_VARLEN, reason, len, "N must be >= 1 with cu_seqlens");
  if (host[0] != 0) return fail(GDR_ERR_VARLEN, reason, len, "cu_seqlens[0] must be 0");
  for (int n = 0; n < N; ++n)
    if (host[n + 1] < host[n])
      return fail(GDR_ERR_VARLEN, reason, len, "cu_seqlens decreases at %d", n + 1);
  if (host[N] != T)
    return fail(GDR_ERR_VARLEN, reason, len, "cu_seqlens[N]=%d must equal T=%d", host[N], T);
  return GDR_OK;
}

static gdr_status need_workspace(size_t need, const void* ws, size_t have, const char* what) {
  if (need > 0 && (!ws || have < need))
    return fail(GDR_ERR_WORKSPACE, nullptr, 0, "%s workspace needs %zu bytes, got %zu", what, need,
                ws ? have : (size_t)0);
  return GDR_OK;
}

static gdr_status validate(const gdr_conv_problem* p, char* reason, size_t len) {
  if (!p) return fail(GDR_ERR_NULL, reason, len, "problem descriptor is NULL");
  if (!is_type(p->dtype))
    return fail(GDR_ERR_DTYPE, reason, len, "x must be bf16, fp16 or fp32 (got code %d)",
                (int)p->dtype);
  if (p->w_dtype != p->dtype && p->w_dtype != GDR_FP32)
    return fail(GDR_ERR_DTYPE, reason, len, "the weight must have x's dtype or fp32 (got code %d)",
                (int)p->w_dtype);
  if (p->B < 1 || p->T < 1 || p->D < 1)
    return fail(GDR_ERR_SHAPE, reason, len, "sizes must be positive (B=%d T=%d D=%d)", p->B, p->T,
                p->D);
  if (p->W < 2 || p->W > 4)
    return fail(GDR_ERR_SHAPE, reason, len, "the convolution's width must be 2, 3 or 4, got %d",
                p->W);
  if (p->D > 65536) return fail(GDR_ERR_SHAPE, reason, len, "at most 65536 channels, got %d", p->D);
  // the last block's runs begin up to 2^23 tokens past the last one, in 32-bit
  // arithmetic
  if ((int64_t)p->B * p->T > 0x7f000000)
    return fail(GDR_ERR_SHAPE, reason, len, "problem too large");
  if (p->x_stride < p->D)
    return fail(GDR_ERR_SHAPE, reason, len, "x_stride=%lld is below D=%d", (long long)p->x_stride,
                p->D);
  if (!is_flag(p->activation))
    return fail(GDR_ERR_ARG, reason, len, "activation must be 0 (none) or 1 (silu)");
  return check_seqs(p->B, p->T, p->N, p->cu_seqlens_dev, p->cu_seqlens_host, reason, len);
}

static gdr_status validate(const gdr_norm_problem* p, char* reason, size_t len) {
  if (!p) return fail(GDR_ERR_NULL, reason, len, "problem descriptor is NULL");
  if (!is_type(p->dtype))
    return fail(GDR_ERR_DTYPE, reason, len, "x must be bf16, fp16 or fp32 (got code %d)",
                (int)p->dtype);
  if (p->w_dtype != p->dtype && p->w_dtype != GDR_FP32)
    return fail(GDR_ERR_DTYPE, reason, len, "the weight must have x's dtype or fp32 (got code %d)",
                (int)p->w_dtype);
  if (!is_flag(p->has_residual))
    return fail(GDR_ERR_ARG, reason, len, "has_residual must be 0 or 1");
  if (p->has_residual && p->res_dtype != p->dtype && p->res_dtype != GDR_FP32)
    return fail(GDR_ERR_DTYPE, reason, len, "the residual must have x's dtype or fp32 (got code %d)",
                (int)p->res_dtype);
  if (p->rows < 1 || p->D < 1)
    return fail(GDR_ERR_SHAPE, reason, len, "sizes must be positive (rows=%d D=%d)", p->rows, p->D);
  if (p->D > 65536) return fail(GDR_ERR_SHAPE, reason, len, "at most 65536 columns, got %d", p->D);
  // a launch holds fewer than 2^32 threads: 64, 256 or 1024 a row
  if ((int64_t)p->rows * (p->D <= 1024 ? 64 : p->D <= 16384 ? 256 : 1024) > 0xffff0000ll)
    return fail(GDR_ERR_SHAPE, reason, len, "too many rows (%d of %d columns)", p->rows, p->D);
  if (p->x_stride < p->D)
    return fail(GDR_ERR_SHAPE, reason, len, "x_stride=%lld is below D=%d", (long long)p->x_stride,
                p->D);
  if (p->quant < 0 || p->quant > 2)
    return fail(GDR_ERR_ARG, reason, len, "quant must be 0 (none), 1 (e4m3) or 2 (int8)");
  if (p->group_size != 0 && p->group_size != 128)
    return fail(GDR_ERR_ARG, reason, len, "group_size must be 0 (the row) or 128, got %d",
                p->group_size);
  if (!p->quant && p->group_size)
    return fail(GDR_ERR_ARG, reason, len, "group_size is for quantised outputs");
  if (!std::isfinite(p->eps) || p->eps < 0.f)
    return fail(GDR_ERR_ARG, reason, len, "eps must be finite and >= 0");
  return GDR_OK;
}

static gdr_status validate(const gdr_ssm_problem* p, char* reason, size_t len) {
  if (!p) return fail(GDR_ERR_NULL, reason, len, "problem descriptor is NULL");
  if ((p->K != 64 && p->K != 128) || (p->V != 64 && p->V != 128))
    return fail(GDR_ERR_HEAD_DIM, reason, len, "K and V must be 64 or 128, got K=%d V=%d", p->K,
                p->V);
  if (p->in_dtype != GDR_BF16 && p->in_dtype != GDR_FP16)
    return fail(GDR_ERR_DTYPE, reason, len, "x, B and C must be bf16 or fp16 (got code %d)",
                (int)p->in_dtype);
  if (p->dt_dtype != p->in_dtype && p->dt_dtype != GDR_FP32)
    return fail(GDR_ERR_DTYPE, reason, len, "dt must have x's dtype or fp32 (got code %d)",
                (int)p->dt_dtype);
  if (p->p_dtype != p->in_dtype && p->p_dtype != GDR_FP32)
    return fail(GDR_ERR_DTYPE, reason, len,
                "A_log, D and dt_bias must have x's dtype or fp32 (got code %d)", (int)p->p_dtype);
  if (p->B < 1 || p->T < 1 || p->H < 1 || p->G < 1)
    return fail(GDR_ERR_SHAPE, reason, len, "sizes must be positive (B=%d T=%d H=%d G=%d)", p->B,
                p->T, p->H, p->G);
  if (p->G > p->H || p->H % p->G != 0)
    return fail(GDR_ERR_HEADS, reason, len, "heads must be a multiple of groups (H=%d G=%d)", p->H,
                p->G);
  // launches hold fewer than 2^32 threads: at most 4096 for the states of a
  // sequence's head, 512 for each of a head's segments, which have 256 tokens
  // or more unless the sequence is shorter
  if ((int64_t)p->B * p->T > 0x7f000000 || p->H > 32768 || (int64_t)p->N * p->H > (1 << 19) ||
      (int64_t)p->B * p->T * p->H > (1 << 30))
    return fail(GDR_ERR_SHAPE, reason, len,
                "problem too large (B * T * H up to 2^30, N * H up to 2^19, H up to 32768)");
  if (p->x_stride < (int64_t)p->H * p->V || p->b_stride < (int64_t)p->G * p->K ||
      p->c_stride < (int64_t)p->G * p->K)
    return fail(GDR_ERR_SHAPE, reason, len,
                "token strides must cover a token's heads (x %lld, B %lld, C %lld)",
                (long long)p->x_stride, (long long)p->b_stride, (long long)p->c_stride);
  // 64 rows of a tile lie within 2^31 bytes
  if (p->x_stride > (1 << 23) || p->b_stride > (1 << 23) || p->c_stride > (1 << 23))
    return fail(GDR_ERR_SHAPE, reason, len,
                "token strides must be at most 2^23 (x %lld, B %lld, C %lld)",
                (long long)p->x_stride, (long long)p->b_stride, (long long)p->c_stride);
  if (!is_flag(p->dt_softplus) || !is_flag(p->keep_states))
    return fail(GDR_ERR_ARG, reason, len, "dt_softplus and keep_states must be 0 or 1");
  return check_seqs(p->B, p->T, p->N, p->cu_seqlens_dev, p->cu_seqlens_host, reason, len);
}

// What the operators on rows share: sizes, types, strides, 8-bit outputs.
static gdr_status check_rows(int rows, int D, int most, gdr_dtype dtype, int quant, int group,
                             char* reason, size_t len) {
  if (!is_type(dtype))
    return fail(GDR_ERR_DTYPE, reason, len, "x must be bf16, fp16 or fp32 (got code %d)", (int)dtype);
  if (rows < 1 || D < 1)
    return fail(GDR_ERR_SHAPE, reason, len, "sizes must be positive (rows=%d D=%d)", rows, D);
  if (D > most) return fail(GDR_ERR_SHAPE, reason, len, "at most %d columns, got %d", most, D);
  if (quant < 0 || quant > 2)
    return fail(GDR_ERR_ARG, reason, len, "quant must be 0 (none), 1 (e4m3) or 2 (int8)");
  if (group != 0 && group != 128)
    return fail(GDR_ERR_ARG, reason, len, "columns per scale must be 0 (the row) or 128, got %d",
                group);
  if (!quant && group)
    return fail(GDR_ERR_ARG, reason, len, "columns per scale are for quantised outputs");
  return GDR_OK;
}
// A launch holds fewer than 2^32 threads.
static gdr_status check_threads(int64_t threads, int rows, int D, char* reason, size_t len) {
  if (threads > 0xffff0000ll)
    return fail(GDR_ERR_SHAPE, reason, len, "too many rows (%d of %d columns)", rows, D);
  return GDR_OK;
}
static gdr_status check_stride(const char* name, int64_t stride, int D, char* reason, size_t len) {
  if (stride < D)
    return fail(GDR_ERR_SHAPE, reason, len, "%s_stride=%lld is below D=%d", name, (long long)stride,
                D);
  return GDR_OK;
}

static gdr_status validate(const gdr_gated_norm_problem* p, char* reason, size_t len) {
  if (!p) return fail(GDR_ERR_NULL, reason, len, "problem descriptor is NULL");
  gdr_status s = check_rows(p->rows, p->D, 16384, p->dtype, p->quant, p->scale_group, reason, len);
  if (s != GDR_OK) return s;
  if (p->w_dtype != p->dtype && p->w_dtype != GDR_FP32)
    return fail(GDR_ERR_DTYPE, reason, len, "the weight must have x's dtype or fp32 (got code %d)",
                (int)p->w_dtype);
  if (p->norm_size < 1 || p->D % p->norm_size != 0)
    return fail(GDR_ERR_SHAPE, reason, len, "D must be a multiple of norm_size (D=%d norm_size=%d)",
                p->D, p->norm_size);
  if (p->norm_size < 8 && p->norm_size != p->D)
    return fail(GDR_ERR_SHAPE, reason, len, "norm_size must be D or at least 8, got %d",
                p->norm_size);
  if ((s = check_threads(gated_norm_threads(p), p->rows, p->D, reason, len)) != GDR_OK) return s;
  if (!is_flag(p->shared_weight) || !is_flag(p->gate_first))
    return fail(GDR_ERR_ARG, reason, len, "shared_weight and gate_first must be 0 or 1");
  if (p->activation != 1 && p->activation != 2)
    return fail(GDR_ERR_ARG, reason, len, "activation must be 1 (silu) or 2 (sigmoid)");
  if (!std::isfinite(p->eps) || p->eps < 0.f)
    return fail(GDR_ERR_ARG, reason, len, "eps must be finite and >= 0");
  if ((s = check_stride("x", p->x_stride, p->D, reason, len)) != GDR_OK) return s;
  return check_stride("gate", p->gate_stride, p->D, reason, len);
}

static gdr_status validate(const gdr_sandwich_norm_problem* p, char* reason, size_t len) {
  if (!p) return fail(GDR_ERR_NULL, reason, len, "problem descriptor is NULL");
  gdr_status s = check_rows(p->rows, p->D, 16384, p->dtype, p->quant, p->group_size, reason, len);
  if (s != GDR_OK) return s;
  if ((s = check_threads(sandwich_norm_threads(p), p->rows, p->D, reason, len)) != GDR_OK) return s;
  if (p->res_dtype != p->dtype && p->res_dtype != GDR_FP32)
    return fail(GDR_ERR_DTYPE, reason, len, "the residual must have x's dtype or fp32 (got code %d)",
                (int)p->res_dtype);
  if (p->w_dtype != p->dtype && p->w_dtype != GDR_FP32)
    return fail(GDR_ERR_DTYPE, reason, len, "the weights must have x's dtype or fp32 (got code %d)",
                (int)p->w_dtype);
  if (p->activation < 0 || p->activation > 2)
    return fail(GDR_ERR_ARG, reason, len, "activation must be 0 (none), 1 (silu) or 2 (sigmoid)");
  if (!std::isfinite(p->eps) || p->eps < 0.f)
    return fail(GDR_ERR_ARG, reason, len, "eps must be finite and >= 0");
  if (!std::isfinite(p->alpha)) return fail(GDR_ERR_ARG, reason, len, "alpha must be finite");
  if ((s = check_stride("x", p->x_stride, p->D, reason, len)) != GDR_OK) return s;
  return check_stride("gate", p->gate_stride, p->D, reason, len);
}

static gdr_status validate(const gdr_quantize_problem* p, char* reason, size_t len) {
  if (!p) return fail(GDR_ERR_NULL, reason, len, "problem descriptor is NULL");
  gdr_status s = check_rows(p->rows, p->D, 65536, p->dtype, p->quant, p->group_size, reason, len);
  if (s != GDR_OK) return s;
  // 64, 256 or 1024 a row
  const int a_row = p->D <= 1024 ? 64 : p->D <= 16384 ? 256 : 1024;
  if ((s = check_threads((int64_t)p->rows * a_row, p->rows, p->D, reason, len)) != GDR_OK) return s;
  if (p->quant == 0)
    return fail(GDR_ERR_ARG, reason, len, "quant must be 1 (e4m3) or 2 (int8)");
  return check_stride("x", p->x_stride, p->D, reason, len);
}

static gdr_status validate(const gdr_int8_matmul_problem* p, char* reason, size_t len) {
  if (!p) return fail(GDR_ERR_NULL, reason, len, "problem descriptor is NULL");
  if (!is_type(p->out_dtype))
    return fail(GDR_ERR_DTYPE, reason, len, "the output must be bf16, fp16 or fp32 (got code %d)",
                (int)p->out_dtype);
  if (p->bias_dtype != p->out_dtype && p->bias_dtype != GDR_FP32)
    return fail(GDR_ERR_DTYPE, reason, len, "the bias must have the output's dtype or fp32 (got code %d)",
                (int)p->bias_dtype);
  if (p->M < 1 || p->N < 1 || p->K < 1)
    return fail(GDR_ERR_SHAPE, reason, len, "sizes must be positive (M=%d N=%d K=%d)", p->M, p->N,
                p->K);
  // 65536 products of at most 2^14 stay below 2^31
  if (p->K > 65536) return fail(GDR_ERR_SHAPE, reason, len, "at most K = 65536, got %d", p->K);
  // a launch holds fewer than 2^32 threads: 256 for 128 x 128 outputs, 512 for 16
  // channels of a few tokens
  if ((((int64_t)p->M + 127) / 128) * (((int64_t)p->N + 127) / 128) > (1 << 23) ||
      p->N > (1 << 26))
    return fail(GDR_ERR_SHAPE, reason, len, "problem too large (M=%d N=%d)", p->M, p->N);
  // rows that are no multiple of 16 bytes may be copied, by 64 threads each
  if ((p->K % 16 != 0 || p->x_stride % 16 != 0) && 64 * ((int64_t)p->M + p->N) > 0xffff0000ll)
    return fail(GDR_ERR_SHAPE, reason, len, "problem too large (M=%d N=%d)", p->M, p->N);
  // the rows of a tile lie within 2^31 bytes
  if (p->x_stride < p->K || p->x_stride > (1 << 22))
    return fail(GDR_ERR_SHAPE, reason, len, "x_stride=%lld must be K=%d to 2^22",
                (long long)p->x_stride, p->K);
  return GDR_OK;
}

static bool misaligned(const void* p) { return ((uintptr_t)p & 15) != 0; }

}  // namespace gdr

using namespace gdr;

extern "C" {

gdr_status gdr_conv1d_check(const gdr_conv_problem* p, char* reason, size_t reason_len) {
  const gdr_status s = validate(p, reason, reason_len);
  if (s == GDR_OK && reason && reason_len) reason[0] = '\0';
  return s;
}

gdr_status gdr_conv1d_fwd(const gdr_conv_problem* p, const void* x, const void* weight,
                          const void* bias, const void* initial_state, void* y,
                          void* final_state, void* stream) {
  gdr_status s = validate(p, nullptr, 0);
  if (s != GDR_OK) return s;
  if (!x || !weight || !y)
    return fail(GDR_ERR_NULL, nullptr, 0, "a required convolution pointer is NULL");
  if (final_state && final_state == initial_state)
    return fail(GDR_ERR_ARG, nullptr, 0,
                "final_state may not be initial_state (gdr_conv1d_update works in place)");
  if ((s = gdr_check_device()) != GDR_OK) return s;
  return launch_conv_fwd(p, x, weight, bias, initial_state, y, final_state, (hipStream_t)stream);
}

size_t gdr_conv1d_bwd_workspace_size(const gdr_conv_problem* p) {
  return validate(p, nullptr, 0) == GDR_OK ? conv_bwd_workspace(p) : 0;
}

gdr_status gdr_conv1d_bwd(const gdr_conv_problem* p, const void* x, const void* weight,
                          const void* bias, const void* dy, const void* dfinal_state,
                          const void* initial_state, void* dx, void* dweight, void* dbias,
                          void* dinitial_state, void* workspace, size_t workspace_bytes,
                          void* stream) {
  gdr_status s = validate(p, nullptr, 0);
  if (s != GDR_OK) return s;
  if (!x || !weight || !dy || !dx || !dweight)
    return fail(GDR_ERR_NULL, nullptr, 0, "a required convolution-gradient pointer is NULL");
  if (dinitial_state && !initial_state)
    return fail(GDR_ERR_ARG, nullptr, 0, "dinitial_state needs initial_state");
  s = need_workspace(conv_bwd_workspace(p), workspace, workspace_bytes, "convolution-gradient");
  if (s != GDR_OK) return s;
  if ((s = gdr_check_device()) != GDR_OK) return s;
  return launch_conv_bwd(p, x, weight, bias, dy, dfinal_state, initial_state, dx, dweight, dbias,
                         dinitial_state, workspace, (hipStream_t)stream);
}

gdr_status gdr_conv1d_update(const gdr_conv_problem* p, const void* x, void* state,
                             const void* weight, const void* bias, void* y, void* stream) {
  gdr_status s = validate(p, nullptr, 0);
  if (s != GDR_OK) return s;
  if (p->cu_seqlens_dev)
    return fail(GDR_ERR_VARLEN, nullptr, 0, "gdr_conv1d_update takes dense sequences");
  if (p->B > 65535)
    return fail(GDR_ERR_SHAPE, nullptr, 0, "gdr_conv1d_update takes at most 65535 sequences, got %d",
                p->B);
  if (!x || !state || !weight || !y)
    return fail(GDR_ERR_NULL, nullptr, 0, "a required convolution-update pointer is NULL");
  if ((s = gdr_check_device()) != GDR_OK) return s;
  return launch_conv_update(p, x, state, weight, bias, y, (hipStream_t)stream);
}

gdr_status gdr_ssm_check(const gdr_ssm_problem* p, char* reason, size_t reason_len) {
  const gdr_status s = validate(p, reason, reason_len);
  if (s == GDR_OK && reason && reason_len) reason[0] = '\0';
  return s;
}

size_t gdr_ssm_fwd_workspace_size(const gdr_ssm_problem* p) {
  return validate(p, nullptr, 0) == GDR_OK ? ssm_fwd_workspace(p, ssm_fwd_plan(p)) : 0;
}

gdr_status gdr_ssm_fwd(const gdr_ssm_problem* p, const void* x, const void* dt, const void* A_log,
                       const void* B, const void* C, const void* D, const void* dt_bias,
                       const float* initial_state, void* y, float* final_state, void* workspace,
                       size_t workspace_bytes, void* stream) {
  gdr_status s = validate(p, nullptr, 0);
  if (s != GDR_OK) return s;
  if (!x || !dt || !A_log || !B || !C || !y)
    return fail(GDR_ERR_NULL, nullptr, 0, "a required scan pointer is NULL");
  if (final_state && final_state == initial_state)
    return fail(GDR_ERR_ARG, nullptr, 0,
                "final_state may not be initial_state (gdr_ssm_step works in place)");
  if (misaligned(initial_state) || misaligned(final_state) || misaligned(workspace))
    return fail(GDR_ERR_ARG, nullptr, 0, "states and workspace must be 16-byte aligned");
  const SsmPlan pl = ssm_fwd_plan(p);
  s = need_workspace(ssm_fwd_workspace(p, pl), workspace, workspace_bytes, "scan");
  if (s != GDR_OK) return s;
  if ((s = gdr_check_device()) != GDR_OK) return s;
  return launch_ssm_fwd(p, pl, x, dt, A_log, B, C, D, dt_bias, initial_state, y, final_state,
                        workspace, (hipStream_t)stream);
}

size_t gdr_ssm_bwd_workspace_size(const gdr_ssm_problem* p) {
  return validate(p, nullptr, 0) == GDR_OK ? ssm_bwd_workspace(p) : 0;
}

gdr_status gdr_ssm_bwd(const gdr_ssm_problem* p, const void* x, const void* dt, const void* A_log,
                       const void* B, const void* C, const void* D, const void* dt_bias,
                       const void* dy, const float* dfinal_state, const float* initial_state,
                       const void* kept_states, void* dx, void* ddt, void* dA_log, void* dB, void* dC, void* dD,
                       void* ddt_bias, float* dinitial_state, void* workspace,
                       size_t workspace_bytes, void* stream) {
  gdr_status s = validate(p, nullptr, 0);
  if (s != GDR_OK) return s;
  if (!x || !dt || !A_log || !B || !C || !dy || !dx || !ddt || !dA_log || !dB || !dC)
    return fail(GDR_ERR_NULL, nullptr, 0, "a required scan-gradient pointer is NULL");
  if ((dD && !D) || (ddt_bias && !dt_bias) || (dinitial_state && !initial_state))
    return fail(GDR_ERR_ARG, nullptr, 0, "dD, ddt_bias and dinitial_state need their inputs");
  if (misaligned(initial_state) || misaligned(dfinal_state) || misaligned(dinitial_state) ||
      misaligned(workspace))
    return fail(GDR_ERR_ARG, nullptr, 0, "states and workspace must be 16-byte aligned");
  if (misaligned(kept_states))
    return fail(GDR_ERR_ARG, nullptr, 0, "kept states must be 16-byte aligned");
  if (kept_states ? !p->keep_states
                  : p->keep_states && ssm_fwd_workspace(p, ssm_fwd_plan(p)) > 0)
    return fail(GDR_ERR_NULL, nullptr, 0, "kept_states come with keep_states, and only then");
  s = need_workspace(ssm_bwd_workspace(p), workspace, workspace_bytes, "scan-gradient");
  if (s != GDR_OK) return s;
  if ((s = gdr_check_device()) != GDR_OK) return s;
  return launch_ssm_bwd(p, x, dt, A_log, B, C, D, dt_bias, dy, dfinal_state, initial_state,
                        kept_states, dx, ddt, dA_log, dB, dC, dD, ddt_bias, dinitial_state, workspace,
                        (hipStream_t)stream);
}

gdr_status gdr_ssm_step(const gdr_ssm_problem* p, const void* x, const void* dt, const void* A_log,
                        const void* B, const void* C, const void* D, const void* dt_bias,
                        const float* initial_state, void* y, float* final_state, void* stream) {
  gdr_status s = validate(p, nullptr, 0);
  if (s != GDR_OK) return s;
  if (!x || !dt || !A_log || !B || !C || !y)
    return fail(GDR_ERR_NULL, nullptr, 0, "a required scan pointer is NULL");
  if (misaligned(initial_state) || misaligned(final_state))
    return fail(GDR_ERR_ARG, nullptr, 0, "states must be 16-byte aligned");
  if ((s = gdr_check_device()) != GDR_OK) return s;
  return launch_ssm_step(p, x, dt, A_log, B, C, D, dt_bias, initial_state, y, final_state,
                         (hipStream_t)stream);
}

gdr_status gdr_rms_norm_check(const gdr_norm_problem* p, char* reason, size_t reason_len) {
  const gdr_status s = validate(p, reason, reason_len);
  if (s == GDR_OK && reason && reason_len) reason[0] = '\0';
  return s;
}

gdr_status gdr_rms_norm_fwd(const gdr_norm_problem* p, const void* x, const void* residual,
                            const void* weight, void* y, float* scale, void* h, float* rstd,
                            void* stream) {
  gdr_status s = validate(p, nullptr, 0);
  if (s != GDR_OK) return s;
  if (!x || !weight || !y) return fail(GDR_ERR_NULL, nullptr, 0, "a required norm pointer is NULL");
  if ((residual != nullptr) != (p->has_residual == 1) || (h != nullptr) != (p->has_residual == 1))
    return fail(GDR_ERR_NULL, nullptr, 0, "residual and h come with has_residual, and only then");
  if ((scale != nullptr) != (p->quant != 0))
    return fail(GDR_ERR_NULL, nullptr, 0, "scale comes with a quantised output, and only then");
  if ((s = gdr_check_device()) != GDR_OK) return s;
  return launch_norm_fwd(p, x, residual, weight, y, scale, h, rstd, (hipStream_t)stream);
}

size_t gdr_rms_norm_bwd_workspace_size(const gdr_norm_problem* p) {
  return validate(p, nullptr, 0) == GDR_OK ? norm_bwd_workspace(p) : 0;
}

gdr_status gdr_rms_norm_bwd(const gdr_norm_problem* p, const void* dy, const void* h,
                            const void* weight, const float* rstd, const void* dh, void* dx,
                            void* dresidual, void* dweight, void* workspace,
                            size_t workspace_bytes, void* stream) {
  gdr_status s = validate(p, nullptr, 0);
  if (s != GDR_OK) return s;
  if (p->quant) return fail(GDR_ERR_ARG, nullptr, 0, "a quantised output has no gradient");
  if (!dy || !h || !weight || !rstd || !dx || !dweight)
    return fail(GDR_ERR_NULL, nullptr, 0, "a required norm-gradient pointer is NULL");
  if (!p->has_residual && (dh || dresidual))
    return fail(GDR_ERR_ARG, nullptr, 0, "dh and dresidual come with has_residual");
  s = need_workspace(norm_bwd_workspace(p), workspace, workspace_bytes, "norm-gradient");
  if (s != GDR_OK) return s;
  if ((s = gdr_check_device()) != GDR_OK) return s;
  return launch_norm_bwd(p, dy, h, weight, rstd, dh, dx, dresidual, dweight, workspace,
                         (hipStream_t)stream);
}

gdr_status gdr_gated_norm_check(const gdr_gated_norm_problem* p, char* reason, size_t reason_len) {
  const gdr_status s = validate(p, reason, reason_len);
  if (s == GDR_OK && reason && reason_len) reason[0] = '\0';
  return s;
}

gdr_status gdr_gated_norm_fwd(const gdr_gated_norm_problem* p, const void* x, const void* gate,
                              const void* weight, void* y, float* scale, float* rstd,
                              void* stream) {
  gdr_status s = validate(p, nullptr, 0);
  if (s != GDR_OK) return s;
  if (!x || !gate || !weight || !y)
    return fail(GDR_ERR_NULL, nullptr, 0, "a required gated-norm pointer is NULL");
  if ((scale != nullptr) != (p->quant != 0))
    return fail(GDR_ERR_NULL, nullptr, 0, "scale comes with a quantised output, and only then");
  if (rstd && p->quant)
    return fail(GDR_ERR_ARG, nullptr, 0, "rstd is for the gradient, which a quantised output has not");
  if ((s = gdr_check_device()) != GDR_OK) return s;
  return launch_gated_norm_fwd(p, x, gate, weight, y, scale, rstd, (hipStream_t)stream);
}

size_t gdr_gated_norm_bwd_workspace_size(const gdr_gated_norm_problem* p) {
  return validate(p, nullptr, 0) == GDR_OK ? gated_norm_bwd_workspace(p) : 0;
}

gdr_status gdr_gated_norm_bwd(const gdr_gated_norm_problem* p, const void* dy, const void* x,
                              const void* gate, const void* weight, const float* rstd, void* dx,
                              void* dgate, void* dweight, void* workspace, size_t workspace_bytes,
                              void* stream) {
  gdr_status s = validate(p, nullptr, 0);
  if (s != GDR_OK) return s;
  if (p->quant) return fail(GDR_ERR_ARG, nullptr, 0, "a quantised output has no gradient");
  if (!dy || !x || !gate || !weight || !rstd || !dx || !dgate || !dweight)
    return fail(GDR_ERR_NULL, nullptr, 0, "a required gated-norm-gradient pointer is NULL");
  s = need_workspace(gated_norm_bwd_workspace(p), workspace, workspace_bytes, "gated-norm-gradient");
  if (s != GDR_OK) return s;
  if ((s = gdr_check_device()) != GDR_OK) return s;
  return launch_gated_norm_bwd(p, dy, x, gate, weight, rstd, dx, dgate, dweight, workspace,
                               (hipStream_t)stream);
}

gdr_status gdr_sandwich_norm_check(const gdr_sandwich_norm_problem* p, char* reason,
                                   size_t reason_len) {
  const gdr_status s = validate(p, reason, reason_len);
  if (s == GDR_OK && reason && reason_len) reason[0] = '\0';
  return s;
}

gdr_status gdr_sandwich_norm_fwd(const gdr_sandwich_norm_problem* p, const void* x,
                                 const void* residual, const void* gate, const void* post_weight,
                                 const void* res_scale, const void* pre_weight, void* y,
                                 float* scale, void* h, float* rstd_x, float* rstd_h,
                                 void* stream) {
  gdr_status s = validate(p, nullptr, 0);
  if (s != GDR_OK) return s;
  if (!x || !residual || !pre_weight || !y || !h)
    return fail(GDR_ERR_NULL, nullptr, 0, "a required sandwich-norm pointer is NULL");
  if ((scale != nullptr) != (p->quant != 0))
    return fail(GDR_ERR_NULL, nullptr, 0, "scale comes with a quantised output, and only then");
  if (rstd_x && !post_weight)
    return fail(GDR_ERR_ARG, nullptr, 0, "rstd_x comes with post_weight");
  if (h == residual) return fail(GDR_ERR_ARG, nullptr, 0, "h may not be residual");
  if ((s = gdr_check_device()) != GDR_OK) return s;
  return launch_sandwich_norm_fwd(p, x, residual, gate, post_weight, res_scale, pre_weight, y, scale,
                                  h, rstd_x, rstd_h, (hipStream_t)stream);
}

size_t gdr_sandwich_norm_bwd_workspace_size(const gdr_sandwich_norm_problem* p) {
  return validate(p, nullptr, 0) == GDR_OK ? sandwich_norm_bwd_workspace(p) : 0;
}

gdr_status gdr_sandwich_norm_bwd(const gdr_sandwich_norm_problem* p, const void* dy, const void* dh,
                                 const void* x, const void* h, const void* gate,
                                 const void* post_weight, const void* res_scale,
                                 const void* pre_weight, const float* rstd_x, const float* rstd_h,
                                 void* dx, void* dresidual, void* dgate, void* dpost_weight,
                                 void* dres_scale, void* dpre_weight, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  gdr_status s = validate(p, nullptr, 0);
  if (s != GDR_OK) return s;
  if (p->quant) return fail(GDR_ERR_ARG, nullptr, 0, "a quantised output has no gradient");
  if (!dy || !x || !h || !pre_weight || !rstd_h || !dx || !dresidual || !dpre_weight)
    return fail(GDR_ERR_NULL, nullptr, 0, "a required sandwich-norm-gradient pointer is NULL");
  if ((gate != nullptr) != (dgate != nullptr))
    return fail(GDR_ERR_NULL, nullptr, 0, "dgate comes with gate, and only then");
  if ((post_weight != nullptr) != (rstd_x != nullptr))
    return fail(GDR_ERR_NULL, nullptr, 0, "rstd_x comes with post_weight, and only then");
  if ((dpost_weight && !post_weight) || (dres_scale && !res_scale))
    return fail(GDR_ERR_ARG, nullptr, 0, "dpost_weight and dres_scale need their inputs");
  s = need_workspace(sandwich_norm_bwd_workspace(p), workspace, workspace_bytes,
                     "sandwich-norm-gradient");
  if (s != GDR_OK) return s;
  if ((s = gdr_check_device()) != GDR_OK) return s;
  return launch_sandwich_norm_bwd(p, dy, dh, x, h, gate, post_weight, res_scale, pre_weight, rstd_x,
                                  rstd_h, dx, dresidual, dgate, dpost_weight, dres_scale,
                                  dpre_weight, workspace, (hipStream_t)stream);
}

gdr_status gdr_quantize_check(const gdr_quantize_problem* p, char* reason, size_t reason_len) {
  const gdr_status s = validate(p, reason, reason_len);
  if (s == GDR_OK && reason && reason_len) reason[0] = '\0';
  return s;
}

gdr_status gdr_quantize_rows(const gdr_quantize_problem* p, const void* x, void* q, float* scale,
                             void* stream) {
  gdr_status s = validate(p, nullptr, 0);
  if (s != GDR_OK) return s;
  if (!x || !q || !scale)
    return fail(GDR_ERR_NULL, nullptr, 0, "a required quantisation pointer is NULL");
  if ((s = gdr_check_device()) != GDR_OK) return s;
  return launch_quantize_rows(p, x, q, scale, (hipStream_t)stream);
}

gdr_status gdr_int8_matmul_check(const gdr_int8_matmul_problem* p, char* reason,
                                 size_t reason_len) {
  const gdr_status s = validate(p, reason, reason_len);
  if (s == GDR_OK && reason && reason_len) reason[0] = '\0';
  return s;
}

size_t gdr_int8_matmul_workspace_size(const gdr_int8_matmul_problem* p) {
  return validate(p, nullptr, 0) == GDR_OK ? int8_matmul_workspace(p) : 0;
}

gdr_status gdr_int8_matmul(const gdr_int8_matmul_problem* p, const void* x, const float* x_scale,
                           const void* weight, const float* w_scale, const void* bias, void* y,
                           void* workspace, size_t workspace_bytes, void* stream) {
  gdr_status s = validate(p, nullptr, 0);
  if (s != GDR_OK) return s;
  if (!x || !x_scale || !weight || !w_scale || !y)
    return fail(GDR_ERR_NULL, nullptr, 0, "a required matrix-product pointer is NULL");
  if (p->K % 16 == 0 && (misaligned(weight) || (p->x_stride % 16 == 0 && misaligned(x))))
    return fail(GDR_ERR_ARG, nullptr, 0, "rows of a multiple of 16 bytes must be 16-byte aligned");
  s = need_workspace(int8_matmul_workspace(p), workspace, workspace_bytes, "matrix-product");
  if (s != GDR_OK) return s;
  if (misaligned(workspace))
    return fail(GDR_ERR_ARG, nullptr, 0, "the workspace must be 16-byte aligned");
  if ((s = gdr_check_device()) != GDR_OK) return s;
  return launch_int8_matmul(p, x, x_scale, weight, w_scale, bias, y, workspace,
                            (hipStream_t)stream);
}

}  // extern "C"

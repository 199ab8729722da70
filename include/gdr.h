/*
 * gdr.h -- C ABI of libgdr: the chunked gated delta rule (GDN chunked prefill)
 * forward and backward on AMD Instinct MI355X (gfx950).
 *
 * The operation
 * -------------
 * FlashQLA pages ("flashqla-linear-attention", Core API; "FlashQLA
 * Documentation", forward / backward) define the tensors; the recurrence is
 * the gated delta rule of Gated Delta Networks (Yang, Kautz, Hatamizadeh,
 * 2024).  For every sequence n and value head h (q/k head hq = h / (Hv/Hq),
 * grouped value attention), with a K x V fp32 state S:
 *
 *     S_t = exp(g_t) S_{t-1} + beta_t k_t (v_t - exp(g_t) S_{t-1}^T k_t)^T
 *     o_t = scale * S_t^T q_t
 *
 * computed chunk by chunk (64 tokens) in the WY form: per chunk, gamma is the
 * chunk-local inclusive cumsum of g, A = (I + strict_lower(diag(beta) K K^T o
 * exp(gamma_r - gamma_i)))^{-1} is unit lower triangular, and the state moves
 * from chunk to chunk by S <- e^{gamma_L} S + K^T diag(e^{gamma_L-gamma})
 * A (diag(beta) V - diag(beta e^gamma) K S).
 *
 * Tensor layouts (row-major, contiguous, tokens of all sequences flattened):
 *   q, k          [B, T, Hq, K]           in_dtype
 *   v, o, do, dv  [B, T, Hv, V]           in_dtype
 *   g, dg         [B, T, Hv]              g_dtype (natural-log decay, or the
 *                                         gate's raw input with use_gate)
 *   beta, dbeta   [B, T, Hv]              in_dtype
 *   g_cum         [B, T, Hv]              fp32: chunk-local inclusive cumsum of g
 *   A             [B, T, Hv, 64]          in_dtype: row r of a chunk's inverse
 *                                         at token chunk_start + r; columns past
 *                                         a partial chunk are 0
 *   h             [NC, Hv, K, V]          in_dtype: state at the start of each
 *                                         chunk, chunk c of sequence n at row
 *                                         chunk_offsets[n] + c
 *   states        [N, Hv, K, V]           fp32: initial_state, final_state,
 *                                         dht, dh0
 * With state_v_first != 0 every state tensor (h included) is [.., V, K]
 * instead; the results are then bit-identical transposes of the default.
 * Packed variable-length input (cu_seqlens != NULL) has B == 1 and T the total
 * token count; N = number of sequences.  K and V must be 128.
 *
 * Conventions
 * -----------
 * - The caller owns every buffer and the stream.  The library allocates no
 *   device memory, keeps no pointer after a call returns and never
 *   synchronises: work is enqueued on `stream` (a hipStream_t; NULL = the
 *   null stream) and buffers must stay alive until the stream reaches it.
 * - Outputs are overwritten, never accumulated.  Inputs and outputs must not
 *   alias.  Device pointers must be 16-byte aligned.
 * - Every argument is validated on the host before any HIP call; a failure
 *   returns a status (never aborts) and gdr_last_error() describes it.
 * - Results are deterministic: no floating-point atomics, fixed reduction
 *   orders, and a context-parallel plan that depends only on shapes.
 */
#ifndef GDR_H
#define GDR_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  GDR_OK = 0,
  GDR_ERR_NULL = 1,      /* a required pointer is NULL */
  GDR_ERR_SHAPE = 2,     /* non-positive or inconsistent sizes */
  GDR_ERR_HEAD_DIM = 3,  /* K != 128 or V != 128 */
  GDR_ERR_DTYPE = 4,     /* q/k/v not bf16/fp16, or g not in_dtype/fp32 */
  GDR_ERR_HEADS = 5,     /* Hq > Hv or Hv % Hq != 0 */
  GDR_ERR_VARLEN = 6,    /* malformed cu_seqlens */
  GDR_ERR_WORKSPACE = 7, /* workspace missing or too small */
  GDR_ERR_DEVICE = 8,    /* no gfx950 device current */
  GDR_ERR_HIP = 9,       /* a HIP launch failed */
  GDR_ERR_ARG = 10       /* another bad argument (scale, chunk size, flags) */
} gdr_status;

typedef enum { GDR_BF16 = 0, GDR_FP16 = 1, GDR_FP32 = 2 } gdr_dtype;

typedef struct {
  int32_t B, T, Hq, Hv, K, V;
  int32_t N;                      /* sequences: B, or len(cu_seqlens) - 1 */
  const int32_t* cu_seqlens_dev;  /* device [N+1] token offsets, or NULL (dense) */
  const int32_t* cu_seqlens_host; /* host copy of the same; used to plan launches
                                     without a device-to-host copy; NULL iff the
                                     device pointer is NULL */
  gdr_dtype in_dtype;             /* q, k, v, beta, do, o, A, h and their grads */
  gdr_dtype g_dtype;              /* raw g and dg: in_dtype or GDR_FP32 */
  float scale;                    /* output scale, usually K^-0.5 */
  int32_t state_v_first;          /* 0: states [.., K, V]; 1: [.., V, K] */
  int32_t cp_segments;            /* intra-GPU context parallelism along T:
                                     0 = automatic plan, 1 = off, s > 1 = split
                                     every sequence into up to s segments */
  int32_t wave_tiles;             /* 16-column state tiles per wave in the scans:
                                     0 = automatic, 1 or 2 */
  int32_t use_qk_l2norm;          /* 1: every kernel scales q and k per (token,
                                     head) to unit length over K before use,
                                     x / sqrt(sum x^2 + 1e-6) in fp32, and the
                                     backward's dq, dk are with respect to the
                                     raw q, k; 0: q and k are used as given.
                                     The option the FLA backend pull request
                                     ("[GDN] Add FlashQLA backend dispatch",
                                     the dispatch's argument list) passes as
                                     use_qk_l2norm_in_kernel. */
  int32_t beta_sigmoid;           /* 1: the beta input is a logit and the
                                     recurrence uses sigmoid(beta); dbeta is with
                                     respect to the logit (the PR page's
                                     use_beta_sigmoid_in_kernel) */
  int32_t neg_eigval;             /* 1: the recurrence uses 2 beta (after the
                                     sigmoid when both are set), so the
                                     transition I - beta k k^T may have a
                                     negative eigenvalue; dbeta is with respect
                                     to the input (the PR page's
                                     allow_neg_eigval) */
  int32_t use_gate;               /* 1: g holds the gate's raw input x and the
                                     recurrence's log decay is, per token and
                                     value head h, computed in fp32:
                                       -exp(gate_A_log[h]) * softplus(x + gate_dt_bias[h])
                                     (the Mamba-2 discretisation that Gated
                                     DeltaNet layers use for their decay; the PR
                                     page's use_gate_in_kernel).  g_cum is the
                                     cumsum of that log decay; the backward
                                     then goes through gdr_chunk_bwd_gate. */
  const float* gate_A_log;        /* device [Hv] fp32: required iff use_gate */
  const float* gate_dt_bias;      /* device [Hv] fp32, or NULL for a zero bias;
                                     NULL unless use_gate */
  int32_t h_packed;               /* 1: gdr_chunk_fwd writes the chunk-start
                                     states h in the packed layout that
                                     gdr_chunk_bwd_states reads (below),
                                     whatever state_v_first says; 0: h is
                                     [NC, Hv, K, V] (or [NC, Hv, V, K] with
                                     state_v_first) */
} gdr_problem;

/* Status name ("GDR_ERR_SHAPE", ...). */
const char* gdr_status_string(gdr_status s);

/* Description of the last failure in the calling thread ("" if none). */
const char* gdr_last_error(void);

/* Host-only argument check, the analogue of the verifier in the FLA backend
 * pull request ("[GDN] Add FlashQLA backend dispatch", Changes and review
 * threads: K != 128, V != 128 and unsupported dtypes are rejected with a
 * reason).  Writes a NUL-terminated reason into `reason` (may be NULL). */
gdr_status gdr_check_supported(const gdr_problem* p, char* reason, size_t reason_len);

/* Device check: the current HIP device is a gfx950.  GDR_ERR_DEVICE if not. */
gdr_status gdr_check_device(void);

/* Bytes of device workspace gdr_chunk_fwd / gdr_chunk_bwd (and
 * gdr_chunk_bwd_gate) / gdr_chunk_bwd_states need for `p` (0 if `p` is
 * invalid).  Depends only on the problem's shapes.  With use_qk_l2norm the
 * forward (h_packed = 1) and the states backward size for both of their
 * forms: given the forward's unit rows they run as problems without the
 * option, whose plans may differ. */
size_t gdr_chunk_fwd_workspace_size(const gdr_problem* p);
size_t gdr_chunk_bwd_workspace_size(const gdr_problem* p);
size_t gdr_chunk_bwd_states_workspace_size(const gdr_problem* p);

/* Forward ("flashqla-linear-attention", Low-Level API; "FlashQLA
 * Documentation", forward pass returning g, A, o, h, final_state).
 *   in : q, k, v, g, beta; initial_state (nullable, fp32 state layout)
 *   out: g_cum, A, o (required); h (nullable: chunk-start states);
 *        final_state (nullable: output_final_state == False)
 *   workspace: device buffer of gdr_chunk_fwd_workspace_size(p) bytes.  With
 *   use_qk_l2norm and h NULL or packed, its tail holds the q and k rows
 *   normalised once (fwd_prep) for the rest of the forward, which then runs
 *   as a problem without the option. */
gdr_status gdr_chunk_fwd(const gdr_problem* p, const void* q, const void* k, const void* v,
                         const void* g, const void* beta, const float* initial_state,
                         float* g_cum, void* A, void* o, void* h, float* final_state,
                         void* workspace, size_t workspace_bytes, void* stream);

/* Forward that keeps what the backward needs (the pages' autograd
 * integration, "flashqla-linear-attention", Integration with PyTorch
 * Autograd: the forward saves what its backward takes).  gdr_chunk_fwd with
 * p->h_packed = 1, plus:
 *   out: h (required), the packed chunk-start states gdr_chunk_bwd_states
 *        reads
 *        trans: when the plan splits sequences into T-segments, each
 *        segment's state transition T_seg (S_end = T_seg S_start + B_seg),
 *        fp32 [N * Hv][cp_segments][K][K], gdr_chunk_trans_size(p) bytes;
 *        required when that size is nonzero, ignored (may be NULL) when it
 *        is zero; trans_bytes is its size (GDR_ERR_WORKSPACE when smaller).
 *        Entries of the first and last segment of each sequence are never
 *        written or read.  With p->use_qk_l2norm the buffer also keeps,
 *        after the transitions (256-byte aligned), the q and k rows scaled
 *        to unit length (in_dtype, q's layout) and their fp32 1 / |x| per
 *        (token, q head): the forward normalises the rows once, runs the
 *        rest as a problem without the option, and gdr_chunk_bwd_states
 *        given the buffer does the same, mapping dq, dk back through the
 *        normalisation; gdr_chunk_trans_size is then nonzero whatever the
 *        plan.
 * A forward with h_packed = 1 and the backward that takes its states plan
 * together (one segment count for both, gdr_plan_info), so that the
 * backward applies the transposed T_seg instead of forming its own
 * transitions.  Errors: GDR_ERR_ARG when h_packed != 1, GDR_ERR_NULL for a
 * missing h or trans, else as gdr_chunk_fwd. */
size_t gdr_chunk_trans_size(const gdr_problem* p);
gdr_status gdr_chunk_fwd_states(const gdr_problem* p, const void* q, const void* k,
                                const void* v, const void* g, const void* beta,
                                const float* initial_state, float* g_cum, void* A, void* o,
                                void* h, float* trans, size_t trans_bytes, float* final_state,
                                void* workspace, size_t workspace_bytes, void* stream);

/* Forward without allocation, for callers that cannot call hipMalloc or take
 * a caller-owned workspace: code under HIP graph capture, tight serving
 * loops, harnesses that forbid allocation.  Same arguments, results and
 * errors as gdr_chunk_fwd (bit-identical outputs: same plan, same kernels),
 * with no workspace: the library uses a static device array of 64 MiB per
 * GPU (GDR_NOALLOC_SCRATCH_BYTES), allocated when the library's code object
 * loads on that GPU and held until the process ends.  Problems whose
 * gdr_chunk_fwd_workspace_size exceeds it are rejected with
 * GDR_ERR_WORKSPACE before any device work (a single 65,536-token sequence
 * with 32 value heads needs 48 MiB; short and dense problems need none).
 * Every call on a GPU shares that GPU's array: calls that overlap on one GPU
 * (on different streams, or from several threads) race and must not be
 * issued.  Nothing in the array needs to start at zero: each call writes
 * every byte it later reads. */
#define GDR_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20)
gdr_status gdr_chunk_fwd_noalloc(const gdr_problem* p, const void* q, const void* k,
                                 const void* v, const void* g, const void* beta,
                                 const float* initial_state, float* g_cum, void* A, void* o,
                                 void* h, float* final_state, void* stream);

/* Backward ("FlashQLA Documentation", backward pass: takes q, k, v, the g
 * returned by the forward, beta, A, do, dht, scale, initial_state, cu_seqlens
 * and returns dq, dk, dv, db, dg, dh0).
 *   in : q, k, v, g_cum (the forward's fp32 g output), beta, A (forward
 *        output), do; dht (nullable = zero); initial_state (nullable = zero)
 *   out: dq, dk (in_dtype, [B,T,Hq,K]); dv; dbeta; dg (g_dtype, gradient with
 *        respect to the raw g); dh0 (fp32, written iff initial_state != NULL,
 *        may be NULL otherwise)
 *   Problems with use_gate are rejected (GDR_ERR_ARG): see gdr_chunk_bwd_gate.
 *   workspace: device buffer of gdr_chunk_bwd_workspace_size(p) bytes. */
gdr_status gdr_chunk_bwd(const gdr_problem* p, const void* q, const void* k, const void* v,
                         const float* g_cum, const void* beta, const void* A, const void* do_,
                         const float* dht, const float* initial_state, void* dq, void* dk,
                         void* dv, void* dbeta, void* dg, float* dh0, void* workspace,
                         size_t workspace_bytes, void* stream);

/* Backward with the in-kernel gate (problem->use_gate == 1; gdr_chunk_bwd
 * rejects such problems).  The arguments of gdr_chunk_bwd, plus:
 *   in : g, the gate's raw input x the forward took (g_dtype [B,T,Hv])
 *   out: dg is the gradient with respect to x (g_dtype);
 *        dA_log, ddt_bias (fp32 [Hv], each nullable = not written): the
 *        gradients of gate_A_log and gate_dt_bias, sums over every token of
 *        every sequence, in a fixed order (deterministic)
 * The workspace (gdr_chunk_bwd_workspace_size) includes 8 bytes per chunk
 * and value head for the per-chunk partial sums of those two gradients. */
gdr_status gdr_chunk_bwd_gate(const gdr_problem* p, const void* q, const void* k, const void* v,
                              const float* g_cum, const void* g, const void* beta, const void* A,
                              const void* do_, const float* dht, const float* initial_state,
                              void* dq, void* dk, void* dv, void* dbeta, void* dg, float* dh0,
                              float* dA_log, float* ddt_bias, void* workspace,
                              size_t workspace_bytes, void* stream);

/* Backward given the forward's chunk-start states: the backward the pages'
 * autograd integration ("flashqla-linear-attention", Integration with
 * PyTorch Autograd) runs after a forward that kept its states.  The
 * arguments and results of gdr_chunk_bwd (gdr_chunk_bwd_gate when
 * p->use_gate), plus:
 *   in : h, the chunk-start states gdr_chunk_fwd computed for the same
 *        problem and inputs with h_packed = 1: per chunk row and value head
 *        the 128 x 128 state in in_dtype as [V/16][K/32][64][8]: element
 *        ((vb * 4 + kb) * 64 + 16 * g + c) * 8 + e holds the state at value
 *        16 vb + c and key 32 kb + 4 g + e (e < 4), 32 kb + 16 + 4 g + e - 4
 *        (e >= 4) -- the order the kernels hold it in, so that it is written
 *        and read in 1 KiB contiguous pieces
 *        trans (nullable), the segment transitions gdr_chunk_fwd_states
 *        kept for the same problem and inputs, trans_bytes its size
 *        (GDR_ERR_WORKSPACE when below gdr_chunk_trans_size); when the plan
 *        splits sequences the state-gradient scan then applies them
 *        transposed (the gradient's transition over a segment is T_seg^T)
 *        instead of forming its own, which halves its transition pass;
 *        NULL: it forms them (ignored when the plan splits nothing).
 *        With p->use_qk_l2norm the buffer's unit rows are used instead of
 *        normalising q and k again (q and k are then not read); NULL: the
 *        backward normalises them itself
 *        g, the gate's raw input (use_gate only; NULL otherwise, and so are
 *        dA_log, ddt_bias)
 * The states are not recomputed: only the reverse state-gradient scan runs
 * before the per-chunk gradients, and the workspace
 * (gdr_chunk_bwd_states_workspace_size) holds no state buffer.  States or
 * transitions from another problem or other inputs give meaningless
 * gradients. */
gdr_status gdr_chunk_bwd_states(const gdr_problem* p, const void* q, const void* k,
                                const void* v, const float* g_cum, const void* g,
                                const void* beta, const void* A, const void* do_,
                                const float* dht, const float* initial_state, const void* h,
                                const float* trans, size_t trans_bytes, void* dq, void* dk,
                                void* dv, void* dbeta, void* dg, float* dh0, float* dA_log,
                                float* ddt_bias, void* workspace, size_t workspace_bytes,
                                void* stream);

/* Token-by-token forward for short inputs: decode steps, a few speculative
 * tokens, or a prefill continued from a cached state (the "state-cached
 * continuation" the "flashqla-linear-attention" page lists among its
 * topics).  The same o and final_state as gdr_chunk_fwd, from the same
 * recurrence, but one token at a time with the fp32 state of each
 * (sequence, value head) held on chip: the state is read once and written
 * once, so a step costs about two state transfers (128 KiB per head).
 *   in : q, k [B,T,Hq,K]; v [B,T,Hv,V]; g (raw log decay, g_dtype) and beta
 *        [B,T,Hv]; initial_state fp32 [N,Hv,K,V] ([N,Hv,V,K] with
 *        state_v_first), nullable = zeros
 *   out: o [B,T,Hv,V] in in_dtype; final_state fp32, same layout as
 *        initial_state, nullable.  final_state may be the same buffer as
 *        initial_state (the state is updated in place); no other argument
 *        may alias another.
 * Honours cu_seqlens, state_v_first, scale, use_qk_l2norm, the beta options
 * and use_gate (g is then the gate's raw input).  Needs no
 * workspace.  Costs grow linearly with T; past a few chunks gdr_chunk_fwd is
 * faster.  Errors as gdr_chunk_fwd (validation on the host first). */
gdr_status gdr_recurrent_fwd(const gdr_problem* p, const void* q, const void* k, const void* v,
                             const void* g, const void* beta, const float* initial_state,
                             void* o, float* final_state, void* stream);

/* Variable-length helpers (host, pure integer, bit-exact), after the
 * utilities of the "FlashQLA Documentation" page.  `cu` holds n_plus_1
 * non-decreasing offsets starting at 0.  Each returns GDR_ERR_VARLEN for a
 * malformed `cu`, GDR_ERR_ARG for chunk_size < 1.
 *
 * prepare_lens: lens[i] = cu[i+1] - cu[i]   (n_plus_1 - 1 entries). */
gdr_status gdr_prepare_lens_i32(const int32_t* cu, int64_t n_plus_1, int32_t* lens);
gdr_status gdr_prepare_lens_i64(const int64_t* cu, int64_t n_plus_1, int64_t* lens);

/* prepare_chunk_indices: one row per chunk, in sequence order, holding
 * [sequence index n, chunk index j within sequence n]; the chunk's first
 * token is cu[n] + j * chunk_size.  `out` ([num_chunks, 2]) may be NULL to
 * query *num_chunks only. */
gdr_status gdr_prepare_chunk_indices_i32(const int32_t* cu, int64_t n_plus_1, int64_t chunk_size,
                                         int32_t* out, int64_t* num_chunks);
gdr_status gdr_prepare_chunk_indices_i64(const int64_t* cu, int64_t n_plus_1, int64_t chunk_size,
                                         int64_t* out, int64_t* num_chunks);

/* prepare_chunk_offsets: offsets[0] = 0, offsets[i+1] = offsets[i] +
 * ceil(lens[i] / chunk_size) (n_plus_1 entries, the shape of cu), and
 * *total = offsets[n_plus_1 - 1]: the row of chunk c of sequence n in a
 * global per-chunk buffer such as h is offsets[n] + c. */
gdr_status gdr_prepare_chunk_offsets_i32(const int32_t* cu, int64_t n_plus_1, int64_t chunk_size,
                                         int32_t* offsets, int64_t* total);
gdr_status gdr_prepare_chunk_offsets_i64(const int64_t* cu, int64_t n_plus_1, int64_t chunk_size,
                                         int64_t* offsets, int64_t* total);

/* The literal reading of the chunk-index description: one row per chunk
 * holding [first token of the chunk, global chunk id]. */
gdr_status gdr_prepare_chunk_token_starts_i64(const int64_t* cu, int64_t n_plus_1,
                                              int64_t chunk_size, int64_t* out,
                                              int64_t* num_chunks);

/* The launch plan the library picks for `p` in one direction (backward != 0:
 * gdr_chunk_bwd, or gdr_chunk_bwd_states when p->h_packed; else
 * gdr_chunk_fwd / gdr_chunk_fwd_states); it depends only on shapes and those
 * flags.  With p->h_packed both directions share one segment count:
 * *cp_segments = T-segments per sequence (1 = no context parallelism),
 * *wave_tiles = 16-column state tiles per wave in the scans (1 or 2).
 * A nonzero cp_segments / wave_tiles in `p` fixes that choice for both. */
gdr_status gdr_plan_info(const gdr_problem* p, int backward, int32_t* cp_segments,
                         int32_t* wave_tiles);

/* The pipelined backward gdr_chunk_bwd_states runs for `p` (a diagnostic;
 * shapes only).  With at most 128 (sequence, head) units of a dense batch,
 * or 256 of packed sequences without grouped heads, and 16 or more chunks
 * in the longest sequence: *slices = 1: one launch holds the state-gradient
 * scan and the gradient workgroups of every chunk, the chunks nearest their
 * sequence's end first, each starting once the scan has stored its chunk's
 * state gradient (bounds = 0, chunks of the longest sequence).  With
 * use_qk_l2norm (reported for the backward that normalises q and k itself;
 * given the forward's unit rows it runs as without the option), at most 64
 * units of a dense batch and no grouped heads, *slices >= 2: the scan runs in ranges of
 * chunks, the last range first, each launch pairing one range's scan with
 * the per-chunk gradients of the range the launch before finished; the last
 * launch runs the gradients of chunks [bounds[0], bounds[1]) of every
 * sequence alone.  *slices = 0: one scan launch, then one gradient launch.
 * bounds (nullable) receives up to max_bounds of the *slices + 1 range
 * starts (bounds[*slices] = chunks per sequence). */
gdr_status gdr_bwd_pipeline_info(const gdr_problem* p, int32_t* slices, int32_t* bounds,
                                 int32_t max_bounds);

/* Kernel timing for benchmarks and diagnostics (not part of the pages' API).
 * While enabled, every kernel the library launches is bracketed by a pair of
 * HIP events recorded on its stream.  gdr_profile_enable clears the records
 * (and creates events lazily afterwards); gdr_profile_read waits for the
 * recorded events, adds up the elapsed time per kernel name (names such as
 * "fwd_prep", "scan_out", "scan_aug", "scan_state", "cp_combine",
 * "dh_scan_out", "dh_scan_aug", "grad", "gva_reduce", "chunk_offsets"),
 * writes up to max_entries of them (names: NUL-terminated, name_stride bytes
 * apart; total_ms; launches -- each may be NULL), clears the records and
 * returns the number of entries written. */
gdr_status gdr_profile_enable(int enable);
int gdr_profile_read(char* names, size_t name_stride, double* total_ms, int* launches,
                     int max_entries);

/* ==== The operators around the recurrence in a layer =======================
 * The short causal convolution in front of it, the selective state space scan
 * (its sibling with one decay per head and no delta term), the RMS norm with
 * the residual's addition; and at the layer's ends the norm of the output with
 * its gate, the norms on both sides of the residual's addition, rows in 8 bits
 * and their product.  The conventions above hold: the caller owns
 * buffers and streams, every argument is validated on the host before any HIP
 * call, nothing is allocated or kept, results are deterministic.  Two calls
 * may run at once on different streams if they share no output or workspace.
 * Where a problem states a token stride, consecutive tokens' rows of that
 * input lie so many elements apart (a slice of a wider tensor); every other
 * tensor is contiguous.  Outputs overlap no input unless a function says so.
 * These operators ask only for the alignment of one element unless a function
 * says otherwise. */

/* ---- short causal depthwise convolution ----
 * Per channel d and token t of a sequence, with x[t'] for t' before the
 * sequence taken from the state's W - 1 rows (zero without a state):
 *     z[t] = bias[d] + sum_{j < W} weight[d][j] x[t - (W-1) + j][d]
 *     y[t] = z[t], or z[t] / (1 + e^-z[t]) with activation = 1
 *   x, y, dy, dx    [B, T, D]        dtype; x with a token stride
 *   weight          [D, W]           w_dtype, W = 2, 3 or 4
 *   bias            [D]              w_dtype, nullable
 *   states          [N, W - 1, D]    dtype: the last W - 1 inputs, oldest
 *                                    first (a shorter sequence keeps the
 *                                    younger rows of its initial state) */
typedef struct {
  int32_t B, T, D, W;
  int32_t N;                      /* sequences: B, or len(cu_seqlens) - 1 */
  const int32_t* cu_seqlens_dev;  /* as in gdr_problem */
  const int32_t* cu_seqlens_host;
  gdr_dtype dtype;                /* bf16, fp16 or fp32 */
  gdr_dtype w_dtype;              /* dtype or GDR_FP32 */
  int32_t activation;             /* 0: none, 1: silu */
  int64_t x_stride;               /* elements between tokens of x, >= D */
} gdr_conv_problem;

/* Host-only argument check (as gdr_check_supported). */
gdr_status gdr_conv1d_check(const gdr_conv_problem* p, char* reason, size_t reason_len);

/*   in : x, weight, bias (nullable), initial_state (nullable = zeros)
 *   out: y; final_state (nullable = not written) */
gdr_status gdr_conv1d_fwd(const gdr_conv_problem* p, const void* x, const void* weight,
                          const void* bias, const void* initial_state, void* y,
                          void* final_state, void* stream);

/* The gradient: dfinal_state (nullable = zero) is the gradient of
 * final_state.  out: dx, dweight; dbias (nullable = not written);
 * dinitial_state (nullable = not written; only with initial_state). */
size_t gdr_conv1d_bwd_workspace_size(const gdr_conv_problem* p);
gdr_status gdr_conv1d_bwd(const gdr_conv_problem* p, const void* x, const void* weight,
                          const void* bias, const void* dy, const void* dfinal_state,
                          const void* initial_state, void* dx, void* dweight, void* dbias,
                          void* dinitial_state, void* workspace, size_t workspace_bytes,
                          void* stream);

/* One or a few tokens per sequence (dense, B sequences of T tokens, B <=
 * 65535) on cached states: y as above, and `state` [B, W-1, D] is updated in
 * place. */
gdr_status gdr_conv1d_update(const gdr_conv_problem* p, const void* x, void* state,
                             const void* weight, const void* bias, void* y, void* stream);

/* ---- selective state space scan ----
 * Per sequence and head h (group h / (H / G)), with a K x V fp32 state S,
 * rate = -exp(A_log[h]), dt_t = softplus(raw_t + dt_bias[h]) with dt_softplus
 * (raw_t + dt_bias[h] without):
 *     S_t = exp(rate dt_t) S_{t-1} + dt_t B_t x_t^T
 *     y_t = S_t^T C_t + D[h] x_t
 * the recurrence of Mamba-2 layers: the gated delta rule's sibling with the
 * same gate and no delta term (C, B and x in the places of q, k and v).
 *   x, y, dy, dx   [B, T, H, V]   in_dtype; x with a token stride
 *   B, C, dB, dC   [B, T, G, K]   in_dtype; B, C with a token stride
 *   dt, ddt        [B, T, H]      dt_dtype
 *   A_log, D, dt_bias [H]         p_dtype; D and dt_bias nullable (zero)
 *   states         [N, H, K, V]   fp32, 16-byte aligned
 * K and V are 64 or 128.  Products run on 16-bit operands with fp32 sums; the
 * states and their gradients are as exact as fp32 inputs would make them, the
 * products inside a chunk (64 tokens) round their decayed scores to in_dtype,
 * with fp16 after scaling them to its range: only inputs and results have to
 * fit the type.  A chunk's decays are formed from prefix sums of the log
 * decays in fp32.  A sum passes through up to 7 additions, is multiplied by
 * log2(e), and a decay is the exponential of two sums' difference: with the
 * roundings of step sizes and rates (a few 2^-24 of each term) a decay is
 * within 2^-19 of the largest |sum| of its chunk, relatively, if the log
 * decays have one sign, and within twice that otherwise.
 * Step sizes may be negative without softplus (the state then grows).  An
 * infinity or NaN in x may reach every output of its sequence from the start
 * of its chunk on, other inputs' from their own token on; other sequences
 * stay as they are. */
typedef struct {
  int32_t B, T, H, G, K, V;
  int32_t N;                      /* sequences: B, or len(cu_seqlens) - 1 */
  const int32_t* cu_seqlens_dev;  /* as in gdr_problem */
  const int32_t* cu_seqlens_host;
  gdr_dtype in_dtype;             /* bf16 or fp16 */
  gdr_dtype dt_dtype;             /* in_dtype or GDR_FP32 */
  gdr_dtype p_dtype;              /* in_dtype or GDR_FP32 */
  int32_t dt_softplus;            /* 0 or 1 */
  int32_t keep_states;            /* 1: the forward's workspace is kept for the gradient */
  int64_t x_stride;               /* elements between tokens, H * V to 2^23 */
  int64_t b_stride, c_stride;     /* the same for B and C, G * K to 2^23 */
} gdr_ssm_problem;

gdr_status gdr_ssm_check(const gdr_ssm_problem* p, char* reason, size_t reason_len);

/* Forward over whole sequences: initial_state (nullable = zeros), y,
 * final_state (nullable = not written; not initial_state).  Long sequences
 * are cut into segments that run in parallel; the cuts depend on the shapes
 * and lengths only.  With keep_states the cut is the gradient's, and the
 * workspace (of the size that the problem with keep_states asks for, possibly
 * 0) holds the states at the segments' ends afterwards. */
size_t gdr_ssm_fwd_workspace_size(const gdr_ssm_problem* p);
gdr_status gdr_ssm_fwd(const gdr_ssm_problem* p, const void* x, const void* dt, const void* A_log,
                       const void* B, const void* C, const void* D, const void* dt_bias,
                       const float* initial_state, void* y, float* final_state, void* workspace,
                       size_t workspace_bytes, void* stream);

/* The gradient of the forward.
 *   in : the forward's inputs; dy; dfinal_state (nullable = zero);
 *        kept_states: with keep_states, the workspace of the forward of the
 *        same problem and inputs (NULL if its size was 0); without, NULL, and
 *        everything is recomputed from the inputs
 *   out: dx, ddt (with respect to the raw step sizes), dA_log, dB, dC; dD,
 *        ddt_bias, dinitial_state (each nullable = not written, and only with
 *        its input).  Parameters' gradients are in p_dtype, sums over all
 *        tokens in a fixed order.
 * dx, dB and dC round one operand of their products in a chunk to in_dtype, as
 * y does.  ddt, dA_log and ddt_bias come from fp32 sums, of which at most 512
 * tokens' rounding errors add up: dA_log is within 2^-10 of the root of the
 * summed squares of its terms g_t dg_t.  (The workspace holds fp32 states every
 * 512 tokens of segments longer than that.) */
size_t gdr_ssm_bwd_workspace_size(const gdr_ssm_problem* p);
gdr_status gdr_ssm_bwd(const gdr_ssm_problem* p, const void* x, const void* dt, const void* A_log,
                       const void* B, const void* C, const void* D, const void* dt_bias,
                       const void* dy, const float* dfinal_state, const float* initial_state,
                       const void* kept_states, void* dx, void* ddt, void* dA_log, void* dB,
                       void* dC, void* dD, void* ddt_bias, float* dinitial_state, void* workspace,
                       size_t workspace_bytes, void* stream);

/* Token by token for decode steps: the same y and final_state, the state read
 * once and written once; final_state may be initial_state (updated in
 * place). */
gdr_status gdr_ssm_step(const gdr_ssm_problem* p, const void* x, const void* dt, const void* A_log,
                        const void* B, const void* C, const void* D, const void* dt_bias,
                        const float* initial_state, void* y, float* final_state, void* stream);

/* ---- root-mean-square norm with the residual's addition ----
 * Per row, with h = x + residual rounded to res_dtype (h = x without one):
 *     y = weight h / sqrt(mean(h^2) + eps)
 * in dtype, or quantised to 8 bits: scale = max(max|y| / top, 2^-126) over the
 * row or over each 128 columns (the last group of a row may be narrower),
 * q = the fp32 quotient y / scale rounded to nearest even; top = 448 (e4m3,
 * OCP) or 127 (int8).
 * A NaN in a group makes its scale NaN (and an int8 value 0).
 *   x, y, dy, dx [rows, D] dtype (x with a row stride); residual, h, dh,
 *   dresidual [rows, D] res_dtype; weight, dweight [D] w_dtype; q [rows, D]
 *   8 bits; scale [rows] or [rows, ceil(D / 128)] fp32; rstd [rows] fp32
 * D <= 65536. */
typedef struct {
  int32_t rows, D;
  gdr_dtype dtype;                /* bf16, fp16 or fp32 */
  gdr_dtype res_dtype;            /* dtype or GDR_FP32 (read when has_residual) */
  gdr_dtype w_dtype;              /* dtype or GDR_FP32 */
  int32_t has_residual;
  int32_t quant;                  /* 0: y in dtype, 1: e4m3, 2: int8 */
  int32_t group_size;             /* columns per scale: 0 = the row, or 128 */
  float eps;                      /* finite, >= 0 */
  int64_t x_stride;               /* elements between rows of x, >= D */
} gdr_norm_problem;

gdr_status gdr_rms_norm_check(const gdr_norm_problem* p, char* reason, size_t reason_len);

/*   in : x, weight, residual (iff has_residual)
 *   out: y (q when quantised); scale (iff quantised); h (iff has_residual);
 *        rstd (nullable: 1 / sqrt(mean h^2 + eps), which the gradient takes) */
gdr_status gdr_rms_norm_fwd(const gdr_norm_problem* p, const void* x, const void* residual,
                            const void* weight, void* y, float* scale, void* h, float* rstd,
                            void* stream);

/* The gradient (quant = 0).  h is what the forward normalised: its h with a
 * residual, else x (with x's row stride).
 *   in : dy, h, weight, rstd; dh (nullable = zero; iff has_residual allowed):
 *        the gradient of the stored h
 *   out: dx; dresidual (nullable; the same gradient in res_dtype, for
 *        residuals of another type than x); dweight */
size_t gdr_rms_norm_bwd_workspace_size(const gdr_norm_problem* p);
gdr_status gdr_rms_norm_bwd(const gdr_norm_problem* p, const void* dy, const void* h,
                            const void* weight, const float* rstd, const void* dh, void* dx,
                            void* dresidual, void* dweight, void* workspace,
                            size_t workspace_bytes, void* stream);

/* ---- root-mean-square norm with a gate ----
 * Of a recurrence's output, over each group of norm_size consecutive columns
 * (a head).  With u(v) = v / sqrt(mean(v^2) + eps) over the group:
 *     y = weight u(x) act(gate), or weight u(x act(gate)) with gate_first
 * in dtype, or quantised as gdr_rms_norm_fwd does it, with a scale per row or
 * per 128 columns of the row of all groups.
 *   x, gate, y, dy, dx, dgate [rows, D] dtype (x and gate with a row stride);
 *   weight, dweight [D] w_dtype, or [norm_size] with shared_weight; q [rows, D]
 *   8 bits; scale [rows] or [rows, ceil(D / 128)] fp32; rstd [rows, D /
 *   norm_size] fp32
 * D <= 16384, a multiple of norm_size, which is D or at least 8.  An infinite
 * gate has silu's and the sigmoid's limit; sigmoids below fp32's normal range (of
 * gates below -87) have the precision of its subnormal numbers.  With eps = 0 a
 * group's root mean square has to have an inverse in fp32 (2^-126 or more).  A
 * NaN or an infinity in x reaches its group only, and in 8 bits what its scale
 * covers. */
typedef struct {
  int32_t rows, D, norm_size;
  gdr_dtype dtype;                /* bf16, fp16 or fp32 */
  gdr_dtype w_dtype;              /* dtype or GDR_FP32 */
  int32_t shared_weight;          /* 1: weight [norm_size], for every group */
  int32_t gate_first;
  int32_t activation;             /* 1: silu, 2: sigmoid */
  int32_t quant;                  /* 0: y in dtype, 1: e4m3, 2: int8 */
  int32_t scale_group;            /* columns per scale: 0 = the row, or 128 */
  float eps;                      /* finite, >= 0 */
  int64_t x_stride, gate_stride;  /* elements between rows, >= D */
} gdr_gated_norm_problem;

gdr_status gdr_gated_norm_check(const gdr_gated_norm_problem* p, char* reason, size_t reason_len);

/*   in : x, gate, weight
 *   out: y (q when quantised); scale (iff quantised); rstd (nullable, not when
 *        quantised: one over the root of each group's mean square, which the
 *        gradient takes) */
gdr_status gdr_gated_norm_fwd(const gdr_gated_norm_problem* p, const void* x, const void* gate,
                              const void* weight, void* y, float* scale, float* rstd,
                              void* stream);

/* The gradient (quant = 0).  in: dy and the forward's x, gate, weight, rstd;
 * out: dx, dgate, dweight (a sum over the rows in a fixed order). */
size_t gdr_gated_norm_bwd_workspace_size(const gdr_gated_norm_problem* p);
gdr_status gdr_gated_norm_bwd(const gdr_gated_norm_problem* p, const void* dy, const void* x,
                              const void* gate, const void* weight, const float* rstd, void* dx,
                              void* dgate, void* dweight, void* workspace, size_t workspace_bytes,
                              void* stream);

/* ---- the norms on both sides of a residual's addition ----
 * From a block's output x to the next block's input, with u as above over the
 * row:
 *     n = post_weight u(x)                     (x without post_weight)
 *     h = residual + alpha res_scale act(gate) n, rounded to res_dtype
 *     y = pre_weight u(h)
 * (a factor that is not given is 1), y in dtype or quantised as
 * gdr_rms_norm_fwd does it.
 *   x, gate, y, dy, dx, dgate [rows, D] dtype (x and gate with a row stride);
 *   residual, h, dh, dresidual [rows, D] res_dtype; post_weight, res_scale,
 *   pre_weight and their gradients [D] w_dtype; q, scale as for
 *   gdr_rms_norm_fwd; rstd_x, rstd_h [rows] fp32
 * D <= 16384. */
typedef struct {
  int32_t rows, D;
  gdr_dtype dtype;                /* bf16, fp16 or fp32 */
  gdr_dtype res_dtype;            /* dtype or GDR_FP32 */
  gdr_dtype w_dtype;              /* dtype or GDR_FP32 */
  int32_t activation;             /* of the gate; 0: none, 1: silu, 2: sigmoid */
  int32_t quant;                  /* 0: y in dtype, 1: e4m3, 2: int8 */
  int32_t group_size;             /* columns per scale: 0 = the row, or 128 */
  float eps;                      /* finite, >= 0 */
  float alpha;                    /* finite */
  int64_t x_stride, gate_stride;  /* elements between rows, >= D */
} gdr_sandwich_norm_problem;

gdr_status gdr_sandwich_norm_check(const gdr_sandwich_norm_problem* p, char* reason,
                                   size_t reason_len);

/*   in : x, residual, pre_weight; gate, post_weight, res_scale (nullable)
 *   out: y (q when quantised), h; scale (iff quantised); rstd_x (nullable, only
 *        with post_weight) and rstd_h (nullable), which the gradient takes */
gdr_status gdr_sandwich_norm_fwd(const gdr_sandwich_norm_problem* p, const void* x,
                                 const void* residual, const void* gate, const void* post_weight,
                                 const void* res_scale, const void* pre_weight, void* y,
                                 float* scale, void* h, float* rstd_x, float* rstd_h,
                                 void* stream);

/* The gradient (quant = 0).
 *   in : dy; dh (nullable = zero): the gradient of the stored h; the forward's
 *        x, h, gate, post_weight, res_scale, pre_weight, rstd_x (iff
 *        post_weight), rstd_h
 *   out: dx, dresidual, dpre_weight; dgate (iff gate); dpost_weight and
 *        dres_scale (each nullable = not written, and only with its input) */
size_t gdr_sandwich_norm_bwd_workspace_size(const gdr_sandwich_norm_problem* p);
gdr_status gdr_sandwich_norm_bwd(const gdr_sandwich_norm_problem* p, const void* dy, const void* dh,
                                 const void* x, const void* h, const void* gate,
                                 const void* post_weight, const void* res_scale,
                                 const void* pre_weight, const float* rstd_x, const float* rstd_h,
                                 void* dx, void* dresidual, void* dgate, void* dpost_weight,
                                 void* dres_scale, void* dpre_weight, void* workspace,
                                 size_t workspace_bytes, void* stream);

/* ---- rows to 8 bits ----
 * q and scale of x as gdr_rms_norm_fwd forms them of its y: weights as they are
 * loaded (a scale per channel), activations that come from no norm.  An
 * infinity makes its scale infinite and what the scale covers 0 (itself NaN in
 * e4m3); a NaN makes its scale NaN.
 *   x [rows, D] dtype with a row stride; q [rows, D] 8 bits; scale [rows] or
 *   [rows, ceil(D / 128)] fp32.   D <= 65536. */
typedef struct {
  int32_t rows, D;
  gdr_dtype dtype;                /* bf16, fp16 or fp32 */
  int32_t quant;                  /* 1: e4m3, 2: int8 */
  int32_t group_size;             /* columns per scale: 0 = the row, or 128 */
  int64_t x_stride;               /* elements between rows, >= D */
} gdr_quantize_problem;

gdr_status gdr_quantize_check(const gdr_quantize_problem* p, char* reason, size_t reason_len);
gdr_status gdr_quantize_rows(const gdr_quantize_problem* p, const void* x, void* q, float* scale,
                             void* stream);

/* ---- product of 8-bit integers ----
 *     y[m][n] = x_scale[m] w_scale[n] sum_k x[m][k] weight[n][k] + bias[n]
 * a projection of tokens quantised with a scale each by a weight quantised
 * with a scale per channel.  The sums are exact; a scale or bias that is no
 * number reaches its token or channel only.
 *   x [M, K] int8 with a token stride; weight [N, K] int8; x_scale [M],
 *   w_scale [N] fp32; bias [N] bias_dtype (nullable); y [M, N] out_dtype
 * K <= 65536; M + N below 2^26 where rows are copied (below). */
typedef struct {
  int32_t M, N, K;
  gdr_dtype out_dtype;            /* bf16, fp16 or fp32 */
  gdr_dtype bias_dtype;           /* out_dtype or GDR_FP32 */
  int64_t x_stride;               /* bytes between tokens, K to 2^22 */
} gdr_int8_matmul_problem;

gdr_status gdr_int8_matmul_check(const gdr_int8_matmul_problem* p, char* reason, size_t reason_len);

/* Weights of rows of a multiple of 16 bytes (K) begin at a multiple of 16
 * bytes, and so does x if its stride is one, too.  The workspace (of size 0
 * where K and x_stride are multiples of 16, and possibly elsewhere) is 16-byte
 * aligned: rows of other lengths are copied there. */
size_t gdr_int8_matmul_workspace_size(const gdr_int8_matmul_problem* p);
gdr_status gdr_int8_matmul(const gdr_int8_matmul_problem* p, const void* x, const float* x_scale,
                           const void* weight, const float* w_scale, const void* bias, void* y,
                           void* workspace, size_t workspace_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* GDR_H */

/*
 * ssd.h -- C ABI of libssd: the Mamba-2 selective state-space (SSD) layer's
 * chunked scan, forward and backward, on one NVIDIA GB300 (sm_103a).
 *
 * The operation (page "llm-mamba-200" (gigipick.blogspot.com), sections 1-2:
 * a selective linear recurrence whose steps combine associatively; the
 * equations are lost from the page text and are taken in their Mamba-2 form
 * with one scalar decay per head):
 *
 *   dt_eff[t,h] = softplus(dt[t,h] + dt_bias[h])
 *   h_t         = exp(dt_eff[t,h] * A[h]) * h_{t-1} + dt_eff[t,h] * x_t (outer) B_t
 *   y_t         = h_t . C_t + D[h] * x_t
 *
 * per batch row and head, with h_{-1} = initial_states (or 0).  When seq_idx
 * is given, a token whose id differs from the previous token's starts a new
 * sequence with a zero state; initial_states feeds only the first one.
 * final_states is the state after the last token.
 *
 * It is evaluated by chunks of chunk_size tokens (page "llm-mamba-200",
 * section 3: carry-out state of one chunk is the carry-in of the next), with
 * the cross-chunk state passing, forward and backward, done as an associative
 * scan (page "B200 Helion Mamba-2" (aitrends.kr/articles/109906), section
 * "Helion based B200 kernel redesign").
 *
 * Shapes (b = batch, L = seqlen, H = nheads, P = headdim, N = dstate,
 * G = ngroups; head h reads group floor(h*G/H), i.e. G contiguous blocks of
 * H/G heads).  Every tensor is dense row-major, device memory:
 *
 *   x, y, dy, dx            (b, L, H, P)   dtype
 *   dt, ddt                 (b, L, H)      dtype
 *   B, C, dB, dC            (b, L, G, N)   dtype
 *   dt_bias, A, D and grads (H)            fp32
 *   initial_states, final_states, dfinal_states, dinitial_states
 *                           (b, H, P, N)   fp32
 *   seq_idx                 (b, L)         int32, nondecreasing along each row
 *
 * where dtype is SSD_F32 (fp32) or SSD_BF16 (bf16; fp32 accumulation inside).
 * Every pointer must be 16-byte aligned.
 *
 * Ownership: the caller allocates every buffer, the workspace included, and
 * keeps them alive until the stream work completes.  The library never
 * allocates, never synchronises (except the two status readers and
 * ssd_profile_stop) and keeps no mutable global state other than a
 * per-device cache of device attributes, the optional timing records and
 * the one exception below: the fixed device array behind ssd_fwd_noalloc
 * (SSD_NOALLOC_SCRATCH_BYTES on every GPU that loads the library) with a
 * per-device cache of its address, shared by all ssd_fwd_noalloc calls --
 * calls of it that overlap on the GPU race on that array (see there).
 * Calls enqueue work on the given stream and return before it completes.
 *
 * Errors: every entry point validates its arguments before enqueuing
 * anything and returns an ssd_status; nothing is thrown across the ABI.
 * Errors detected on the device (a bounded wait that expired) are recorded
 * in a status word at the start of the workspace; read it with
 * ssd_read_device_status (ssd_fwd_noalloc_read_device_status for
 * ssd_fwd_noalloc, whose workspace is the library's own array).
 */
#ifndef SSD_H_
#define SSD_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* ssd_stream_t; /* a cudaStream_t; NULL = legacy default stream */

typedef enum {
  SSD_OK = 0,
  SSD_ERR_INVALID_ARGUMENT = 1, /* null required pointer, bad dims, misaligned pointer */
  SSD_ERR_UNSUPPORTED = 2,      /* shape/dtype outside the compiled set, or not an sm_103 device */
  SSD_ERR_WORKSPACE_TOO_SMALL = 3,
  SSD_ERR_CUDA = 4,             /* a CUDA runtime error while enqueuing */
  SSD_ERR_TIMEOUT = 5,          /* a device-side bounded wait expired (read via the status word) */
  SSD_ERR_NO_KEPT_STATES = 6    /* ssd_bwd with SSD_KEEP_FWD_STATES found no forward intermediates of
                                   this problem in the workspace (read via the status word) */
} ssd_status;

typedef enum { SSD_F32 = 0, SSD_BF16 = 1 } ssd_dtype;

enum {
  SSD_HAS_INIT = 1,      /* initial_states is given */
  SSD_HAS_SEQ_IDX = 2,   /* seq_idx is given */
  SSD_HAS_DFINAL = 4,    /* ssd_bwd: dfinal_states (upstream gradient of final_states) is given */
  SSD_WANT_DINIT = 8,    /* ssd_bwd: write dinitial_states */
  /* Keep the forward's intermediates for the backward (the usual training
   * step: forward, then backward on the same inputs).  ssd_fwd with this
   * flag leaves in its workspace what the backward would otherwise
   * recompute -- dt_eff, the chunk-local cumsums of dt_eff * A, the per-chunk
   * decays and the carry-in state of every chunk (in the problem's dtype) --
   * and stamps the workspace with the problem's signature; ssd_fwd without it
   * clears the stamp.  A forward on the separate kernels also keeps the fp32
   * carry-in states (its scan writes them over the fp32 chunk states) and
   * says so in the stamp.  ssd_bwd with this flag, given that same
   * workspace, takes them from there instead of recomputing them: where it
   * runs its single-pass state chains, from either forward; where it runs
   * the separate kernels, from a forward on the separate kernels (if the
   * same problem's forward takes the single-pass kernel, that backward
   * recomputes as usual and ignores the flag).  The inputs must be the ones
   * that forward saw: the stamp covers the problem's shape, not its values.
   * A workspace without the stamp this backward needs makes it report
   * SSD_ERR_NO_KEPT_STATES in the device status word (its results are then
   * garbage).  Forward results do not depend on the flag; backward results
   * agree with the recomputing backward to rounding (bit for bit on the
   * separate kernels, which keep exactly what they would recompute). */
  SSD_KEEP_FWD_STATES = 16,
  /* Testing only: the first scan tile of the first state chain never
   * publishes its prefix, so the tiles after it exhaust their bounded wait
   * (0.1 s with this flag, 2 s otherwise) and the call ends with
   * SSD_ERR_TIMEOUT in the device status word instead of hanging.  Results
   * of such a call are garbage. */
  SSD_TEST_DROP_SCAN_PUBLISH = 1 << 16,
  /* Path selection (comparisons and tests; results agree to rounding).  By
   * default the library takes its single-pass kernels -- in ssd_fwd one
   * persistent CTA per (batch row, head) that keeps the carry on chip, in
   * ssd_bwd one such CTA per chain for the forward and the reverse state
   * chains (bf16, headdim 64, d_state 64 or 128) -- when there are at least
   * about three chains per four SMs, and otherwise its separate kernels
   * (chunk cumsum, chunk states, state-passing scan, chunk output).
   * SSD_PATH_MULTI_KERNEL forces the separate kernels; SSD_PATH_SINGLE_PASS
   * forces the single-pass kernels wherever their shape set allows. */
  SSD_PATH_MULTI_KERNEL = 1 << 17,
  SSD_PATH_SINGLE_PASS = 1 << 18,
  /* Testing only: the persistent token-gradient kernel runs on at most two
   * CTAs, so that a small problem walks several work units per CTA.  Results
   * are the same bits as without the flag. */
  SSD_TEST_FEW_CTAS = 1 << 19,
  /* Comparison: the separate kernels' forward state-passing scan takes each
   * segment's local scan across the lanes of a warp (Hillis-Steele steps of
   * warp shuffles, lane k holding chunk k) instead of sequentially inside
   * each thread; the join of the segments is the same.  Results agree to
   * rounding. */
  SSD_SCAN_WARP_SHUFFLE = 1 << 20
};

typedef struct {
  int64_t batch, seqlen, nheads, headdim, dstate, ngroups, chunk_size;
  int32_t dtype; /* ssd_dtype */
  int32_t flags; /* SSD_HAS_* / SSD_WANT_* */
} ssd_problem;

/* Limits of the compiled kernels (checked by every entry point):
 *   1 <= chunk_size <= 256, chunk_size % 16 == 0
 *   headdim in {16, 32, 64, 128}; dstate in {16, 32, 64, 128};
 *   headdim * dstate <= 8192
 *   nheads % ngroups == 0; batch, seqlen >= 1                              */

/* Bytes of device workspace ssd_fwd / ssd_bwd need for this problem
 * (a pure function of the problem; 0 if the problem is invalid). */
size_t ssd_fwd_workspace_bytes(const ssd_problem* prob);
size_t ssd_bwd_workspace_bytes(const ssd_problem* prob);

/* Forward.  Writes y and (if non-NULL) final_states.  initial_states must be
 * non-NULL iff SSD_HAS_INIT, seq_idx iff SSD_HAS_SEQ_IDX.  Enqueues on
 * `stream` and returns without waiting. */
int ssd_fwd(const ssd_problem* prob, const void* x, const void* dt, const float* dt_bias,
            const float* A, const void* B, const void* C, const float* D,
            const float* initial_states, const int32_t* seq_idx, void* y, float* final_states,
            void* workspace, size_t workspace_bytes, ssd_stream_t stream);

/* Backward (reverse mode of ssd_fwd for the upstream gradients dy and,
 * if SSD_HAS_DFINAL, dfinal_states).  The forward intermediates are
 * recomputed inside (the call is stateless).  Gradients are overwritten, not
 * accumulated: dx, ddt, dB, dC in dtype; ddt_bias, dA, dD (H) fp32;
 * dinitial_states (fp32) iff SSD_WANT_DINIT.  All reductions (dA, dD,
 * ddt_bias over tokens, dB and dC over the heads of a group) are taken in a
 * fixed order: results are bitwise reproducible run to run. */
int ssd_bwd(const ssd_problem* prob, const void* x, const void* dt, const float* dt_bias,
            const float* A, const void* B, const void* C, const float* D,
            const float* initial_states, const int32_t* seq_idx, const void* dy,
            const float* dfinal_states, void* dx, void* ddt, float* ddt_bias, float* dA,
            void* dB, void* dC, float* dD, float* dinitial_states, void* workspace,
            size_t workspace_bytes, ssd_stream_t stream);

/* Human-readable name of a status code (static string). */
const char* ssd_status_string(int status);

/* Synchronises `stream`, then reads the device status word of the last call
 * that used `workspace` (SSD_OK, SSD_ERR_TIMEOUT or SSD_ERR_NO_KEPT_STATES;
 * a timeout is reported first).  Returns SSD_ERR_CUDA if the
 * synchronisation or the copy fails. */
int ssd_read_device_status(const void* workspace, ssd_stream_t stream);

/* Allocation-free forward.  The pages have no counterpart: this is a
 * library convenience for callers that cannot allocate device memory where
 * they call the layer -- a plain C host with no handle on the framework's
 * caching allocator, or a latency-critical loop where an allocation (and
 * the synchronisation cudaMalloc implies) is not allowed.  Same arguments
 * and results as ssd_fwd, minus the workspace: the workspace is a
 * library-owned device array of SSD_NOALLOC_SCRATCH_BYTES (32 MiB) that
 * every GPU loading libssd holds until the process exits.  Problems whose
 * ssd_fwd_workspace_bytes exceeds it are rejected with
 * SSD_ERR_WORKSPACE_TOO_SMALL.  The call allocates nothing.  Its first call
 * on a device looks up the array's device address (cudaGetSymbolAddress,
 * with that device current) and caches it; make that first call before any
 * stream capture.  All calls share the one array and it keeps the last
 * call's contents (each call re-zeroes what must start at zero): calls that
 * can overlap on the GPU -- on different streams or from different host
 * threads -- race on it.  Its device status word is read with
 * ssd_fwd_noalloc_read_device_status. */
#define SSD_NOALLOC_SCRATCH_BYTES (32u << 20)
int ssd_fwd_noalloc(const ssd_problem* prob, const void* x, const void* dt, const float* dt_bias,
                    const float* A, const void* B, const void* C, const float* D,
                    const float* initial_states, const int32_t* seq_idx, void* y,
                    float* final_states, ssd_stream_t stream);

/* Status of the last ssd_fwd_noalloc call on the current device: the
 * counterpart of ssd_read_device_status for the library-owned array, whose
 * address callers never see.  Synchronises `stream`, then returns SSD_OK or
 * SSD_ERR_TIMEOUT (a device-side bounded wait of that call expired; its
 * results are then garbage), or SSD_ERR_CUDA if the synchronisation or the
 * copy fails.  No counterpart on the pages either. */
int ssd_fwd_noalloc_read_device_status(ssd_stream_t stream);

/* ---------------------------------------------------------------------------
 * Context parallelism: the sequence split into contiguous shards (one per
 * rank, or run one after another on one GPU), each shard run through
 * ssd_fwd / ssd_bwd as a problem of its own, the shards joined by two
 * exclusive folds.  Page "B200 Helion Mamba-2" (aitrends.kr/articles/109906)
 * names context parallelism as the module's integration goal without a
 * method; it follows from the recurrence: a shard maps the state h entering
 * it to dec * h + final(0) (dec = product of its per-token decays
 * exp(dt_eff * A), 0 when a sequence starts after its first token; final(0)
 * = its final state from a zero start), and its dinitial_states is affine
 * in the gradient g at its final state, dinit(g) = dec * g + dinit(0).
 *
 * Forward: every shard runs from a zero state (its final_states = local),
 * ssd_shard_decay gives dec and the segment ids of its first and last
 * tokens; after the exchange of (dec, local, ids) of all shards,
 * ssd_shard_fold (reverse = 0, boundary = initial_states or NULL) gives the
 * state entering every shard (out) and the layer's final state (total);
 * every shard runs again from its entering state.  Backward: every shard's
 * dinitial_states with no upstream final gradient (local), exchanged,
 * folded with reverse = 1 (boundary = dfinal_states or NULL) gives every
 * shard its upstream dfinal_states (out); each shard then runs its backward;
 * dA, dD and ddt_bias are sums over the shards.  A shard whose first token
 * starts a new sequence enters from zero and sends no gradient back. */

/* dec (b, H) fp32 of one shard (prob: the shard as a problem; only batch,
 * seqlen, nheads, dtype and SSD_HAS_SEQ_IDX are read) and, if first_ids /
 * last_ids (b) int32 are non-NULL (both or neither), the segment ids of the
 * shard's first and last tokens (0 without seq_idx).  dt (b, Ls, H) dtype;
 * dt_bias, A (H) fp32; seq_idx (b, Ls) iff SSD_HAS_SEQ_IDX. */
int ssd_shard_decay(const ssd_problem* prob, const void* dt, const float* dt_bias, const float* A,
                    const int32_t* seq_idx, float* decay, int32_t* first_ids, int32_t* last_ids,
                    ssd_stream_t stream);

/* The exclusive fold over nshards shards, in order (reverse = 0) or from
 * the right (reverse = 1).  decay (R, b, H) fp32; local, out (R, b, H, P, N)
 * fp32; first_ids, last_ids (R, b) int32 or both NULL (no sequence starts on
 * shard boundaries); boundary (b, H, P, N) fp32 or NULL (zero); total
 * (b, H, P, N) fp32 or NULL.  Forward: h = boundary; for r: h = 0 if shard
 * r > 0 starts a new sequence; out[r] = h; h = decay[r] h + local[r];
 * total = h.  Reverse: g = boundary; for r = R-1 .. 0: out[r] = g;
 * g = decay[r] g + local[r]; g = 0 if shard r > 0 starts a new sequence;
 * total = g.  Device pointers, 16-byte aligned; enqueue only. */
int ssd_shard_fold(int64_t nshards, int64_t batch, int64_t nheads, int64_t headdim, int64_t dstate,
                   const float* decay, const float* local, const int32_t* first_ids,
                   const int32_t* last_ids, const float* boundary, float* out, float* total,
                   int reverse, ssd_stream_t stream);

/* ---------------------------------------------------------------------------
 * Gated RMSNorm of the Mamba-2 block: the normalisation the block applies to
 * the scan's output y, gated by the block's z branch.  Page "B200 Helion
 * Mamba-2" (aitrends.kr/articles/109906) measures its backward
 * (`_layer_norm_bwd`, a memory-bound row reduction) at batch 2, seqlen 8192,
 * bf16, without writing out the operation; it is read as
 *
 *   g[r,j]    = y[r,j] * silu(z[r,j])        (g = y without SSD_NORM_HAS_Z)
 *   rstd[r,k] = 1 / sqrt(mean_{j in group k} g[r,j]^2 + eps)
 *   out[r,j]  = g[r,j] * rstd[r,k] * weight[j]
 *
 * over rows r (tokens) and groups k of group_size contiguous columns (in the
 * Mamba-2 block: dim = nheads * headdim, group_size = dim / ngroups).  The
 * backward gives dy, dz and dweight = sum over rows of dout * g * rstd; that
 * sum is folded across thread blocks in a fixed order (page "Cake RMSNorm",
 * blog.secrett2633.cloud, flashinfer PR 6997, section "Fixed-order tree fold
 * reduction"), so dweight is bitwise reproducible run to run on one device.
 *
 * Layouts (dense row-major, device memory, 16-byte aligned):
 *   y, z, out, dout, dy, dz   (rows, dim)   dtype
 *   weight, dweight           (dim)         fp32
 *   rstd                      (rows, dim / group_size) fp32
 * Limits: dim % group_size == 0; group_size a multiple of 8 (bf16) or 4
 * (fp32) and at most 4096 (bf16) or 2048 (fp32); eps >= 0.
 * Ownership, errors and stream semantics as above.  The calls have no
 * device-side waits and use no status word. */
enum { SSD_NORM_HAS_Z = 1 /* z (the gate) is given */ };

typedef struct {
  int64_t rows, dim, group_size;
  float eps;
  int32_t dtype; /* ssd_dtype of y, z, out, dout, dy, dz */
  int32_t flags; /* SSD_NORM_HAS_Z */
} ssd_norm_problem;

/* Forward: writes out and, if non-NULL, rstd.  z must be non-NULL iff
 * SSD_NORM_HAS_Z. */
int ssd_gated_rmsnorm_fwd(const ssd_norm_problem* prob, const void* y, const void* z,
                          const float* weight, void* out, float* rstd, ssd_stream_t stream);

/* Bytes of device workspace ssd_gated_rmsnorm_bwd needs (the per-block
 * dweight partials; a pure function of the problem, 0 if it is invalid). */
size_t ssd_gated_rmsnorm_bwd_workspace_bytes(const ssd_norm_problem* prob);

/* Backward for the upstream gradient dout (rstd is recomputed from y and z).
 * Overwrites dy, dz (non-NULL iff SSD_NORM_HAS_Z) and dweight. */
int ssd_gated_rmsnorm_bwd(const ssd_norm_problem* prob, const void* y, const void* z,
                          const float* weight, const void* dout, void* dy, void* dz,
                          float* dweight, void* workspace, size_t workspace_bytes,
                          ssd_stream_t stream);

/* ---------------------------------------------------------------------------
 * The norm that takes in the residual, as it stands before a layer's input
 * projection, with its output in the type or in 8 bits:
 *
 *   h[r,j]   = x[r,j] + residual[r,j]      rounded to residual_dtype (h = x without a residual)
 *   rstd[r]  = 1 / sqrt(mean_j h[r,j]^2 + eps)
 *   out[r,j] = h[r,j] * rstd[r] * weight[j]
 *
 * 8-bit output by the state cache's rule (below), a row of out to a scale:
 * out stands for code * scales[r]; a row that holds an infinity or a NaN gets
 * the scale NaN, one of values below 2^-118 zeros.  The squares are summed in
 * fp32: |h| beyond about 1e18 overflows them, and out is then 0.
 *
 * The backward, for the upstream gradients dout of out (of the values that the
 * codes stand for, if they are 8 bits: their rounding passes it through) and,
 * if non-NULL, dh of h, writes
 *   dx = dresidual = dh + the norm's own,  dweight[j] = sum_r dout h rstd
 * with dresidual NULL where dx is enough (the same type).  It recomputes rstd
 * from h.  dweight is summed in a fixed order: bitwise reproducible run to run
 * on one device.
 *
 * Layouts (device memory, 16-byte aligned, dense but for x):
 *   x                (rows, dim)  dtype, x_stride elements from row to row (0: dense)
 *   dout, dx         (rows, dim)  dtype;  out: dtype, or one byte a value
 *   residual, h, dh, dresidual   (rows, dim)  residual_dtype
 *   weight, dweight  (dim) fp32;  scales (rows) fp32, iff out_format is not SSD_OUT_PLAIN
 * residual_dtype is dtype, or SSD_F32 for bf16 layers on an fp32 stream.  h may
 * be NULL (not wanted) or the residual itself (updated in place).  dim <=
 * 16384; eps > 0.  Ownership, errors and stream semantics as above; no
 * device-side waits. */
enum { SSD_NORM_HAS_RESIDUAL = 2 /* residual is given */ };
typedef enum { SSD_OUT_PLAIN = 0, SSD_OUT_INT8 = 1, SSD_OUT_E4M3 = 2 } ssd_out_format;

typedef struct {
  int64_t rows, dim, x_stride;
  float eps;
  int32_t dtype;          /* ssd_dtype of x, out (SSD_OUT_PLAIN), dout, dx */
  int32_t residual_dtype; /* ssd_dtype of residual, h, dh, dresidual */
  int32_t out_format;     /* ssd_out_format; the backward does not read it */
  int32_t flags;          /* SSD_NORM_HAS_RESIDUAL */
} ssd_add_norm_problem;

int ssd_add_rmsnorm_fwd(const ssd_add_norm_problem* prob, const void* x, const void* residual,
                        const float* weight, void* h, void* out, float* scales,
                        ssd_stream_t stream);

/* Bytes of device workspace ssd_add_rmsnorm_bwd needs (partial dweights; a
 * pure function of the problem, 0 if it is invalid). */
size_t ssd_add_rmsnorm_bwd_workspace_bytes(const ssd_add_norm_problem* prob);

int ssd_add_rmsnorm_bwd(const ssd_add_norm_problem* prob, const void* h, const float* weight,
                        const void* dout, const void* dh, void* dx, void* dresidual,
                        float* dweight, void* workspace, size_t workspace_bytes,
                        ssd_stream_t stream);

/* ---------------------------------------------------------------------------
 * The gated delta rule: the recurrence of a layer whose state is corrected
 * by what it already holds, instead of only added to.  Per batch row and
 * head, with a state S (headdim x dstate), a log decay g and a strength beta:
 *
 *   S'  = exp(g_t) S_{t-1}
 *   u_t = beta_t (v_t - S' k_t)
 *   S_t = S' + u_t (outer) k_t
 *   y_t = scale * S_t q_t
 *
 * with S_{-1} = initial_states (or 0).  q and k take the places of the SSD
 * layer's C and B (ngroups heads of dstate values; head h reads group
 * floor(h * ngroups / nheads)), v and y those of x and y.  A token whose
 * seq_idx differs from its predecessor's starts from S' = 0.  Nothing is
 * normalised inside: with |k| = 1 and 0 <= beta <= 2 the state stays bounded.
 *
 * Shapes (b = batch, L = seqlen, H = nheads, P = headdim, N = dstate,
 * G = ngroups), device memory, 16-byte aligned:
 *   q, k             (b, L, G, N)   dtype, q_stride / k_stride elements from
 *                                   token to token (0: dense, G * N)
 *   v                (b, L, H, P)   dtype, v_stride (0: dense, H * P)
 *   g, beta          (b, L, H)      dtype
 *   y, dy            (b, L, H, P)   dtype, dense; dq, dk, dv, dg, dbeta dense
 *   initial_states, final_states, dfinal_states, dinitial_states
 *                    (b, H, P, N)   state_dtype
 *   seq_idx          (b, L)         int32
 * The strides let q, k and v be column blocks of one projection's output.
 * g may be -inf (the state is forgotten); a g below -100 counts as one.
 *
 * Precision: fp32 problems compute in fp32 throughout.  bf16 problems hold
 * states, sums and decays in fp32; where the tensor cores form the products
 * (headdim a multiple of 64, dstate 64 or 128, strides multiples of 8) their
 * operands -- the carried state among them -- are rounded to bf16, and a value
 * that is not finite may reach the y of tokens before it (dv: after it), within
 * its own sequence and its own chunk of 64 tokens.  In no problem does it reach y,
 * dv, the final state or the initial state's gradient through a sequence's start
 * or a decay that forgets.  dq, dk, dg and dbeta may take it up in every token of
 * the chunks (64 tokens; fp32 kernels: 32) in which its sequence has one.
 *
 * Limits: headdim, dstate <= 256; nheads % ngroups == 0; ownership, errors
 * and stream semantics as above; device-side waits are bounded, and one that
 * expired is recorded in the status word at the start of the call's workspace
 * (ssd_read_device_status; the step has no waits and no workspace).  Results
 * are bitwise reproducible run to run. */
typedef struct {
  int64_t batch, seqlen, nheads, headdim, dstate, ngroups;
  int64_t q_stride, k_stride, v_stride; /* elements from token to token; 0 = dense */
  float scale;
  int32_t dtype;       /* ssd_dtype of q, k, v, g, beta, y and their gradients */
  int32_t state_dtype; /* ssd_dtype of the states at the boundary */
  int32_t flags;       /* SSD_HAS_INIT, SSD_HAS_SEQ_IDX, SSD_HAS_DFINAL, SSD_WANT_DINIT */
} ssd_delta_problem;

/* Device bytes of the workspaces and of the buffer in which the forward
 * leaves what the backward reads (pure functions of the problem, whatever its
 * flags; 0 if it is invalid). */
size_t ssd_delta_fwd_workspace_bytes(const ssd_delta_problem* prob);
size_t ssd_delta_bwd_workspace_bytes(const ssd_delta_problem* prob);
size_t ssd_delta_saved_bytes(const ssd_delta_problem* prob);

/* Forward over whole sequences.  Writes y and, if non-NULL, final_states;
 * with `saved` (ssd_delta_saved_bytes) also what ssd_delta_bwd needs. */
int ssd_delta_fwd(const ssd_delta_problem* prob, const void* q, const void* k, const void* v,
                  const void* g, const void* beta, const void* initial_states,
                  const int32_t* seq_idx, void* y, void* final_states, void* saved,
                  size_t saved_bytes, void* workspace, size_t workspace_bytes,
                  ssd_stream_t stream);

/* Backward of the forward that wrote `saved` from the same problem and
 * inputs, for the upstream gradients dy and, if SSD_HAS_DFINAL,
 * dfinal_states.  Gradients are overwritten; dq and dk are sums over the
 * heads of their group, taken in a fixed order; dinitial_states iff
 * SSD_WANT_DINIT.  `saved` is only read. */
int ssd_delta_bwd(const ssd_delta_problem* prob, const void* q, const void* k, const void* v,
                  const void* g, const void* beta, const int32_t* seq_idx, const void* dy,
                  const void* dfinal_states, void* dq, void* dk, void* dv, void* dg, void* dbeta,
                  void* dinitial_states, const void* saved, size_t saved_bytes, void* workspace,
                  size_t workspace_bytes, ssd_stream_t stream);

/* The recurrent form for serving: every sequence of the batch takes seqlen
 * tokens (one, or a few drafted ones) from its state in a pool of nslots
 * states (nslots, H, P, N), fp32 (state_dtype must be SSD_F32; flags 0).
 * slots (b) int32 or NULL gives each sequence's place in the pool (NULL: b's
 * own index, nslots >= batch); one outside [0, nslots) is padding: its y is
 * zero and no state is read or written.  Writes y for all tokens unless y is
 * NULL, and unless states_out is NULL the state after the first lengths[b]
 * tokens of each sequence (lengths (b) int32 or NULL: all; clamped to
 * [0, seqlen]).  states_out may be states_in.  Two sequences of one call must
 * not write the same slot.  All arithmetic is fp32. */
int ssd_delta_step(const ssd_delta_problem* prob, const void* q, const void* k, const void* v,
                   const void* g, const void* beta, int64_t nslots, const float* states_in,
                   float* states_out, const int32_t* slots, const int32_t* lengths, void* y,
                   ssd_stream_t stream);

/* ---------------------------------------------------------------------------
 * Verification of drafted tokens: which of a draft's tokens a sequence keeps,
 * and the token that follows them, so that the result is distributed as the
 * target's own samples.  With the target's probabilities p (b, ndraft + 1,
 * vocab), the draft's q (b, ndraft, vocab), both dtype, and given random
 * numbers: token i of a sequence's first lengths[b] is kept while
 *   uniform[b, i] * q_i(token_i) < p_i(token_i)        (in fp32)
 * and the first that fails ends the draft.  With n kept, the next token is
 *   argmax_v  w(v) / noise[b, v],   w = max(p_n - q_n, 0)  after a refusal,
 *                                   w = p_n                after a whole draft
 * (noise (b, vocab) fp32: independent standard exponentials make that a draw
 * from w; ties go to the lowest index).  Where no w is positive, w = p_n; if
 * none of those is either, the token is 0.  NaN weights and ratios are passed
 * over.  draft_probs may be NULL for drafts chosen without a distribution
 * (q_i = 1 at the token, 0 elsewhere).  lengths (b) int32 or NULL (all
 * ndraft), clamped to [0, ndraft]; a drafted token outside [0, vocab) is
 * refused.  uniform (b, ndraft) fp32, draft_tokens (b, ndraft) int32.
 * Writes out_tokens (b, ndraft + 1) int32 -- the kept tokens, the next one,
 * then -1 -- and accepted (b) int32, the number kept.  ndraft may be 0 (then
 * the draft's arrays may be NULL).  1 <= vocab < 2^31. */
typedef struct {
  int64_t batch, ndraft, vocab;
  int32_t dtype; /* ssd_dtype of both probabilities */
  int32_t flags; /* 0 */
} ssd_verify_problem;

int ssd_verify_draft(const ssd_verify_problem* prob, const void* target_probs,
                     const void* draft_probs, const int32_t* draft_tokens, const int32_t* lengths,
                     const float* uniform, const float* noise, int32_t* out_tokens,
                     int32_t* accepted, ssd_stream_t stream);

/* ---------------------------------------------------------------------------
 * The 8-bit cache of recurrent states: prefixes' states (of the SSD layer or
 * of the delta rule) put away at a quarter of their size.  Each row of N
 * values has one fp32 scale: with a = max |x| of the row and t = 127 (int8)
 * or 448 (e4m3), scale = a * (1 / t) and each value is x * ((1 / a) * t)
 * rounded to nearest, ties to even (fp32, every operation rounded).  A row
 * whose a is below 2^-118 is stored as zeros with scale 0 (a bound chosen for
 * both formats: (1 / a) * t is finite from about 2^-119.2 on for e4m3 and 2^-121
 * for int8); a row that holds an infinity or a NaN reads back as NaN throughout.
 * cache (nslots, H, P, N) bytes, scales (nslots, H, P)
 * fp32.  slots (b) int32 or NULL as for ssd_delta_step; the store passes over
 * slots outside the pool (and must not get one twice), the load gives zeros
 * for them (and may read one slot into many sequences). */
typedef enum { SSD_CACHE_INT8 = 0, SSD_CACHE_E4M3 = 1 } ssd_cache_format;

typedef struct {
  int64_t batch, nheads, headdim, dstate, nslots;
  int32_t format; /* ssd_cache_format */
  int32_t flags;  /* 0 */
} ssd_cache_problem;

int ssd_state_cache_store(const ssd_cache_problem* prob, const float* states, const int32_t* slots,
                          void* cache, float* scales, ssd_stream_t stream);
int ssd_state_cache_load(const ssd_cache_problem* prob, const void* cache, const float* scales,
                         const int32_t* slots, float* states, ssd_stream_t stream);

/* ---------------------------------------------------------------------------
 * The product of 8-bit codes, as the norm above writes them, with weights of
 * the same form:
 *
 *   out[m,n] = a_scales[m] * w_scales[n] * sum_k a[m,k] * w[n,k]  + bias[n]
 *
 * a (m, k), w (n, k): int8 (all 256 values) or e4m3, dense; a_scales (m),
 * w_scales (n), bias (n; or NULL) fp32; out (m, n) out_dtype, dense.  Device
 * memory, 16-byte aligned.  The sums are fp32: those of int8 codes are exact
 * while their partial sums stay below 2^24 (always for k <= 1024).  A NaN or an
 * infinity in a token's scale or codes stays in its row of out, one in a
 * channel's in its column.  m, n <= 2^22, k <= 2^20.  Ownership, errors and stream
 * semantics as above; device-side waits are bounded, and one that expired is
 * recorded in the status word at the start of the workspace
 * (ssd_read_device_status).  Results are bitwise reproducible run to run. */
typedef struct {
  int64_t m, n, k;
  int32_t format;    /* ssd_cache_format of a and w */
  int32_t out_dtype; /* ssd_dtype of out */
  int32_t flags;     /* 0 */
} ssd_matmul_problem;

/* Bytes of device workspace ssd_scaled_matmul needs (a pure function of the
 * problem, at least 256; 0 if it is invalid). */
size_t ssd_scaled_matmul_workspace_bytes(const ssd_matmul_problem* prob);

int ssd_scaled_matmul(const ssd_matmul_problem* prob, const void* a, const float* a_scales,
                      const void* w, const float* w_scales, const float* bias, void* out,
                      void* workspace, size_t workspace_bytes, ssd_stream_t stream);

/* ---------------------------------------------------------------------------
 * Log probabilities of given tokens, the entropy and the top alternatives of
 * their distributions, and the gradient to the logits.  Per row, with
 * z = scale * logits:
 *
 *   lse = log sum_v exp z_v      logprob = z[token] - lse
 *   entropy = -sum_v p_v log p_v,  p = exp(z - lse)
 *
 * and the ntop words of the largest logits in descending order, ties to the
 * lower index, with their log probabilities.
 *
 * logits (rows, vocab) dtype, logit_stride elements from row to row (0:
 * dense); tokens (rows) int32; logprobs, entropy, lse (rows) fp32; stats
 * (rows, 2) fp32, what the backward needs of the rows: the largest logit m, and
 * log sum exp(z - scale m); top_tokens int32 and top_logprobs fp32 (rows, ntop).
 * A token outside [0, vocab) is padding: its logprob is 0 and has no gradient.
 * A logit of -inf excludes its word: it is no alternative, its log probability
 * is -inf, and its gradient 0 unless it is the given token (then the formula's
 * below with p = 0, scale * dlogprob: such a row wants a dlogprob of 0); places
 * for which no word is left hold -1 and -inf.  A row that excludes every word
 * has lse -inf, logprob -inf, entropy 0 and no gradient.  A NaN or +inf in a row
 * makes its lse, logprob (of a token), entropy and gradient NaN; the alternatives
 * are then those of the values that are not NaN.  Of logprobs (given with
 * tokens), entropy, lse, stats and the alternatives each may be NULL, but not all.
 *
 * The backward takes stats and, for dentropy, entropy from the forward, and the
 * upstream gradients dlogprobs (given with tokens) and dentropy (rows) fp32 --
 * either may be NULL -- and writes dlogits (rows, vocab) dtype, grad_stride
 * elements from row to row (0: dense):
 *   dlogits_v = scale * (dlogprob * (1[v = token] - p_v)
 *                        - dentropy * p_v * (log p_v + entropy))
 * A row into which no gradient comes -- padding, or no dlogprobs, with dentropy 0
 * or NULL -- has dlogits 0, whatever its logits hold.  dlogits may be logits
 * itself (then with the same stride).
 *
 * Device memory, 16-byte aligned (strides are free).  scale from 2^-120 on, with
 * scale * log2(e) finite (scale <= 2.358e38); ntop <= 32; 1 <= vocab < 2^31.
 * All sums are fp32.  Ownership, errors and stream semantics as above; no
 * workspace.  Results are bitwise reproducible run to run. */
typedef struct {
  int64_t rows, vocab;
  int64_t logit_stride, grad_stride; /* elements from row to row; 0 = dense */
  float scale;
  int32_t ntop;
  int32_t dtype; /* ssd_dtype of logits and dlogits */
  int32_t flags; /* 0 */
} ssd_logprob_problem;

int ssd_token_logprobs(const ssd_logprob_problem* prob, const void* logits, const int32_t* tokens,
                       float* logprobs, float* entropy, float* lse, float* stats,
                       int32_t* top_tokens, float* top_logprobs, ssd_stream_t stream);
int ssd_token_logprobs_bwd(const ssd_logprob_problem* prob, const void* logits,
                           const int32_t* tokens, const float* stats, const float* entropy,
                           const float* dlogprobs, const float* dentropy, void* dlogits,
                           ssd_stream_t stream);

/* Library build/version string, e.g. "libssd 0.1 sm_103a". */
const char* ssd_version(void);

/* Per-kernel timing, a measurement aid.  ssd_profile_start (re)starts
 * recording on the current device: from then on every kernel launched by
 * ssd_fwd/ssd_bwd is bracketed by two CUDA events recorded on the call's
 * stream.  ssd_profile_stop ends recording and waits for the recorded events
 * (it synchronises), folding them into per-kernel totals that
 * ssd_profile_count/ssd_profile_get report (name is a static string).  The
 * event pool holds 32768 launches; ssd_profile_stop returns
 * SSD_ERR_WORKSPACE_TOO_SMALL if launches beyond it went unrecorded.  Use
 * from one host thread. */
int ssd_profile_start(void);
int ssd_profile_stop(void);
int ssd_profile_count(void);
int ssd_profile_get(int index, const char** name, int* launches, double* total_ms);

#ifdef __cplusplus
}
#endif
#endif /* SSD_H_ */

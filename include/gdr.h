/*
 * gdr.h -- C ABI of the B200 gated delta-rule library (libgdr.so).
 *
 * The recurrence, per (sequence n, value head h), with the state held
 * transposed as H = S^T of shape [dk][dv] (dv contiguous):
 *
 *     u_t = beta_t (v_t - alpha_t H_{t-1}^T k_t)
 *     H_t = alpha_t H_{t-1} + k_t u_t^T,            alpha_t = exp(g_t)
 *     post-write read  o_t = scale * H_t^T q_t
 *     pre-write read   o_t = scale * H_{t-1}^T q_t
 *
 * (Prizma "seq/delta.py", module docstring: the same update on the untransposed
 * state, and the strictly causal read from the state before the token's write;
 * sparse_delta_memory/layer.py, SparseDeltaMemory docstring: the memory decays by
 * the gate's exponential, then takes a write of beta times the key and the
 * prediction error; tiny_gdn/fugue.py, BidirectionalGatedDeltaNet2 docstring: the
 * forward scan reads the state after the token's write.)
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * - Every tensor argument is a DEVICE pointer owned by the caller.  The
 *   library never allocates, frees or synchronises; every call only enqueues
 *   kernels on `stream` (a cudaStream_t passed as void*; NULL = legacy default
 *   stream) and returns.  Calls hold no host state between them.
 * - All tensors are dense and row-major in the index order given.  Pointers
 *   must be 16-byte aligned (GDR_ERR_ALIGNMENT otherwise).
 * - Arguments are validated on the host before anything is enqueued; a call
 *   that returns anything but GDR_OK has enqueued nothing (except
 *   GDR_ERR_CUDA, returned when a launch itself fails).
 * - Inconsistencies only visible on the device (a cu_seqlens array that is not
 *   non-decreasing, does not start at 0 or does not end at T) are recorded in
 *   an error word inside the workspace; the kernels then skip the work.  Read
 *   it with gdr_read_device_error.  No kernel traps or waits without a bound
 *   (the one wait not on a timer: in gdr_chunk_fwd_bidir the two CTAs of a
 *   cluster meet at a cluster barrier before they exit, and each bounds every
 *   wait that could keep it from getting there).
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
    GDR_ERR_INVALID_ARG = 1,   /* null pointer, bad size, Hv % Hk != 0, bad enum ... */
    GDR_ERR_UNSUPPORTED = 2,   /* valid, but no kernel for this (dk, dv, chunk, dtype) */
    GDR_ERR_ALIGNMENT = 3,     /* a pointer is not 16-byte aligned */
    GDR_ERR_WORKSPACE = 4,     /* workspace missing or smaller than the required size */
    GDR_ERR_CUDA = 5,          /* a CUDA launch failed (cudaGetLastError after launch) */
    GDR_ERR_DEVICE_CHECK = 6,  /* device-side check failed (bad cu_seqlens) */
    GDR_ERR_TIMEOUT = 7,       /* a bounded device-side wait gave up */
    GDR_ERR_RANGE = 8          /* tensor-core path: an internal operand left the fp16 range
                                  (|x| >= 65000 or not finite); the outputs are not valid */
} gdr_status;

typedef enum { GDR_F32 = 0, GDR_BF16 = 1 } gdr_dtype;

/* Read mode.  POST: o_t = scale * S_t q_t (tiny_gdn/fugue.py forward scan,
 * q_t^T S_t).  PRE: o_t = scale * S_{t-1} q_t (Prizma "seq/delta.py", the
 * strictly causal pre-write read). */
typedef enum { GDR_READ_POST = 0, GDR_READ_PRE = 1 } gdr_read_mode;

/*
 * Arguments of the chunk-parallel forward (training / prefill).
 *
 * The forward is evaluated in the exact chunk-wise WY/UT form (Prizma
 * "seq/delta.py", chunked_delta: per chunk a unit-lower-triangular solve
 * (I + A) U = ..., then the chunk-to-chunk state carry;
 * sparse_delta_memory/layer.py module docstring: the chunk size changes the
 * result only through floating-point rounding).
 */
typedef struct {
    int B;                 /* rows; with cu_seqlens B must be 1 */
    int T;                 /* tokens per row (with cu_seqlens: total packed tokens) */
    int Hk, Hv;            /* key/query heads and value heads, Hv % Hk == 0; value head h
                              reads key head h / (Hv / Hk)  (tiny_gdn/fugue.py `heads`) */
    int dk, dv;            /* head dims; GPU kernels: dk, dv in {32, 64, 128} */
    int n_seqs;            /* == B without cu_seqlens, else number of packed sequences */
    int chunk;             /* 16, 32, 64 or 128 (64: the contract of flashrt fused_layer.py
                              `_prefill_chain`); chunks restart at every sequence start */
    gdr_dtype io_dtype;    /* dtype of q, k, v and o */
    gdr_dtype gate_dtype;  /* dtype of g and beta */
    gdr_read_mode read_mode;
    float scale;           /* multiplies the read in both modes */
    int qk_l2norm;         /* 1: q, k <- x / max(||x||_2, 1e-6) in fp32 inside the kernels
                              (use_qk_l2norm_in_kernel of tiny_gdn/fugue.py `scan`) */
    int reverse;           /* 1: scan every sequence from its last token to its first, in
                              place (tiny_gdn/fugue.py `scan`, direction 1); o is written at
                              each token's own position, S_final is the state after the
                              sequence's FIRST token */
    int o_accumulate;      /* 1: o += result (o is read, the sum written back in io_dtype);
                              0: o = result */
    /* Fused gating prologue (sparse_delta_memory/layer.py `compute_gates`: A = -exp(A_log),
     * g = A * softplus(a + dt_bias), beta = sigmoid(b); tiny_gdn/fugue.py `project`: beta
     * doubled to allow negative eigenvalues; flashrt fused_layer.py `gdn_gating`).
     *   gate_raw = 0: g and beta are the gates themselves; the three fields below are unused.
     *   gate_raw = 1: the g and beta arguments hold the raw per-token projections a and b
     *                 (same shape and gate_dtype), and the kernels form, in fp32,
     *                   g    = gate_A[h] * softplus(a + gate_dt_bias[h])
     *                   beta = beta_scale * sigmoid(b)
     *                 with softplus(x) = x for x > 20 (as torch's softplus threshold). */
    int gate_raw;
    const float* gate_A;        /* [Hv] fp32 device array, A = -exp(A_log) (<= 0 for a decay);
                                   4-byte aligned; required when gate_raw */
    const float* gate_dt_bias;  /* [Hv] fp32 device array; 4-byte aligned; required when
                                   gate_raw */
    float beta_scale;           /* 1, or 2 for negative eigenvalues; must be finite */
    /* GDN-2 decoupled gates (tiny_gdn/fugue.py BidirectionalGatedDeltaNet2:
     * S_t = (I - k_t (b_t * k_t)^T) Diag(exp g_t) S_{t-1} + k_t (w_t * v_t)^T).
     *   gdn2 = 0: scalar gates, g and beta of one value per token and value head.
     *   gdn2 = 1: g is the per-key-channel log decay [.., Hv, dk], beta the per-key-channel
     *             erase gate b [.., Hv, dk], and gdn2_w the per-value-channel write gate
     *             [.., Hv, dv], all gate_dtype and 16-byte aligned.  With g = log(alpha),
     *             b = w = beta on every channel this is the scalar rule.  Not combined with
     *             gate_raw.  bf16 inputs and gates with dk = dv = 128, chunk 64 and forward
     *             scans take the tensor cores (a preparation kernel over every chunk and
     *             head, then the recursion); a chunk whose per-channel decay grows by more
     *             than 2^100 within 16 tokens is refused there with GDR_ERR_RANGE. */
    int gdn2;
    const void* gdn2_w;
    /* Optional device status word (NULL: none).  A device int owned by the caller, who
     * sets it to GDR_OK (0) before the call.  When a device-side check of the call fails
     * (GDR_ERR_DEVICE_CHECK, GDR_ERR_TIMEOUT, GDR_ERR_RANGE), the call's last kernel stores
     * that status here if the word still holds GDR_OK; the library never clears it.  The
     * caller reads it whenever it likes (e.g. cudaMemcpyAsync into pinned host memory on
     * the same stream), with no synchronisation inside the library, so one word can
     * collect the status of many calls.  4-byte aligned.  Serves every entry point that
     * takes these arguments, gdr_chunk_fwd_noalloc included. */
    int* status;
} gdr_chunk_args;

/* Bytes of device workspace gdr_chunk_fwd needs for these arguments (0 on invalid
 * arguments).  Depends on B, T, Hv, dk, dv, n_seqs, chunk and the dtypes only. */
size_t gdr_chunk_fwd_workspace_size(const gdr_chunk_args* args);

/*
 * Chunk-parallel forward over every sequence and value head.
 *
 *   q, k        [B, T, Hk, dk]   io_dtype
 *   v           [B, T, Hv, dv]   io_dtype
 *   g, beta     [B, T, Hv]       gate_dtype; g = log(alpha) (<= 0 for a decay), beta
 *                                 unrestricted (beta in (0, 2) gives negative
 *                                 eigenvalues, tiny_gdn/fugue.py `project`)
 *   S0          [n_seqs, Hv, dk, dv] fp32 initial state, or NULL for zero
 *   cu_seqlens  [n_seqs + 1] int32 device offsets into the packed row (B == 1), or
 *               NULL for B rows of T tokens (tiny_gdn/fugue.py `segment_layout`)
 *   o           [B, T, Hv, dv]   io_dtype output (rounded to nearest even for bf16)
 *   S_final     [n_seqs, Hv, dk, dv] fp32 final state, or NULL; may alias S0
 *               (each state is read completely before its final value is written)
 *   workspace   device scratch of at least gdr_chunk_fwd_workspace_size(args) bytes,
 *               256-byte aligned; its contents need no initialisation
 *
 * Empty sequences are allowed (their S_final is S0, or zero).
 */
gdr_status gdr_chunk_fwd(const gdr_chunk_args* args,
                         const void* q, const void* k, const void* v,
                         const void* g, const void* beta,
                         const float* S0, const int32_t* cu_seqlens,
                         void* o, float* S_final,
                         void* workspace, size_t workspace_bytes, void* stream);

/*
 * gdr_chunk_fwd without a caller-provided workspace.  (No counterpart on the pages: this is
 * a convenience of this library.)
 *
 * For callers that cannot allocate device memory: a serving process whose GPU memory is
 * reserved up front by its own pool (cudaMalloc may fail there, and it synchronises the
 * device), code inside a framework hook or callback where the CUDA allocator may not be
 * called, or a plain-C caller without a device allocator.  The caller still passes the
 * inputs and outputs exactly as for gdr_chunk_fwd; the scratch is a static device array of
 * GDR_NOALLOC_SCRATCH_BYTES that every GPU loading this library holds until exit.
 *
 * - Calls whose scratch need (gdr_chunk_fwd_workspace_size) exceeds the array return
 *   GDR_ERR_WORKSPACE and enqueue nothing.  The tensor-core path needs only
 *   256 + 8 (n_seqs + 1) + 4 (ceil(B*T / chunk) + n_seqs) bytes (with gdn2 another 74240
 *   bytes per chunk and value head); the CUDA-core path
 *   additionally 4 B*T Hv (dk + dv + 1) bytes (4 B*T Hv (2 dk + dv) with gdn2), and for
 *   chunk <= 64 with dk a multiple of 32 up to 128 another 8 B*T Hv dk +
 *   4 (ceil(B*T / chunk) + n_seqs) Hv chunk^2 bytes, so it fits only small problems.
 * - The first call on a device looks up the array's device address (cudaGetSymbolAddress)
 *   with that device current; make that first call before any stream capture.
 * - All calls on a device share the one array: calls that overlap on the GPU (different
 *   streams, or different host threads, without ordering between them) race and may
 *   corrupt each other's results.  Each call rewrites every scratch field it reads, so a
 *   previous call's contents never leak into the next.
 * - The device error word lives in the shared array: read it with
 *   gdr_noalloc_read_device_error (which synchronises), or give args->status a device word
 *   of the caller's to have it set without a synchronisation.
 * - The array's address is cached per device and CUDA context; a call made after the
 *   device's primary context was reset (cudaDeviceReset) looks it up again.
 * - Arguments that are valid but have no kernel path return GDR_ERR_UNSUPPORTED, invalid
 *   ones the status gdr_chunk_fwd would return; neither enqueues anything.
 */
#define GDR_NOALLOC_SCRATCH_BYTES (4u << 20)
gdr_status gdr_chunk_fwd_noalloc(const gdr_chunk_args* args,
                                 const void* q, const void* k, const void* v,
                                 const void* g, const void* beta,
                                 const float* S0, const int32_t* cu_seqlens,
                                 void* o, float* S_final, void* stream);

/* Test/diagnostic helper for gdr_chunk_fwd_noalloc, NOT for the hot path: copies the device
 * error word out of the static scratch array of the current device (as the last
 * gdr_chunk_fwd_noalloc call on `stream` left it), SYNCHRONISES `stream`, and returns GDR_OK
 * or the recorded device-side status. */
gdr_status gdr_noalloc_read_device_error(void* stream);

/* Name of the kernel path gdr_chunk_fwd takes for these arguments: "tc" (tcgen05
 * tensor-core kernels), "simt" (fp32 CUDA-core kernels) or NULL if unsupported. */
const char* gdr_chunk_fwd_path(const gdr_chunk_args* args);

/*
 * Bidirectional forward (Rondo-Exp tiny_gdn/fugue.py, the bidirectional token mixer): one
 * forward scan with (g_fwd, beta_fwd) and one scan over each sequence's tokens in reverse
 * order with (g_bwd, beta_bwd), both from a zero state with the same q, k, v, read mode and
 * scale, their outputs summed into o:  o = o_fwd + o_bwd  (o_bwd at each token's own
 * position).  No state is returned.
 *
 *   args        as for gdr_chunk_fwd, with reverse = 0 and o_accumulate = 0
 *   g_*, beta_* [B, T, Hv] gate_dtype, or the raw projections with gate_raw (both
 *               directions share gate_A, gate_dt_bias, beta_scale); GDN-2 layouts with gdn2
 *               (both directions share gdn2_w)
 *   o           [B, T, Hv, dv] io_dtype; on the tensor-core path the two directions are
 *               summed in fp32 and the sum rounded once (two gdr_chunk_fwd calls, the second
 *               with reverse and o_accumulate, round each direction first)
 *   workspace   at least gdr_chunk_fwd_bidir_workspace_size(args) bytes, 256-byte aligned
 *
 * On the tensor-core path one grid runs both scans: the two scans of a (sequence, head) are
 * the two CTAs of a thread-block cluster.  The reverse scan's 64-token chunks are aligned
 * with the forward scan's (its first chunk holds the sequence's last T mod 64 tokens), so
 * both produce the output of the same 64 tokens per chunk; the scan that gets to a chunk
 * first leaves its fp32 output there in the workspace, and the other adds it to its own and
 * writes o.  The two CTAs read the same q, k, v tiles within one residency, so the second
 * read is served mostly from L2.  The CUDA-core path runs the reverse scan after the forward
 * one, accumulating into o.  Errors: as gdr_chunk_fwd.
 */
size_t gdr_chunk_fwd_bidir_workspace_size(const gdr_chunk_args* args);
gdr_status gdr_chunk_fwd_bidir(const gdr_chunk_args* args,
                               const void* q, const void* k, const void* v,
                               const void* g_fwd, const void* beta_fwd,
                               const void* g_bwd, const void* beta_bwd,
                               const int32_t* cu_seqlens, void* o,
                               void* workspace, size_t workspace_bytes, void* stream);

/*
 * Backward pass of gdr_chunk_fwd: the gradients of
 *     L = <dO, o> + <dS_final, S_final>
 * with respect to q, k, v, g, beta and S0, for the same arguments (Prizma "seq/delta.py",
 * module docstring: the chunk-parallel form agrees with the per-token recurrence on the
 * forward and on the gradients; the gradient is the per-token recurrence's).  The forward's
 * intermediate values are recomputed from the inputs; nothing from a forward call is kept.
 *
 *   args        as for gdr_chunk_fwd, with gate_raw = 0, gdn2 = 0, o_accumulate = 0;
 *               kernels: chunk in {16, 32, 64}, dk <= 128, dv a multiple of 32 up to 128
 *   q .. cu_seqlens   the forward's inputs, layouts as for gdr_chunk_fwd
 *   dO          [B, T, Hv, dv]   io_dtype, gradient of o
 *   dS_final    [n_seqs, Hv, dk, dv] fp32 gradient of S_final, or NULL for zero
 *   dq, dk      [B, T, Hk, dk]   io_dtype outputs (summed over the v-heads of a key head)
 *   dv          [B, T, Hv, dv]   io_dtype output
 *   dg, dbeta   [B, T, Hv]       gate_dtype outputs (dg is the gradient of g = log alpha)
 *   dS0         [n_seqs, Hv, dk, dv] fp32 output, or NULL
 *   workspace   device scratch of at least gdr_chunk_bwd_workspace_size(args) bytes,
 *               256-byte aligned, no initialisation needed
 *
 * Kernels.  bf16, dk = dv = 128, chunk 64 ("tc"): the tensor-core forward kernel runs twice,
 * once leaving the in-chunk decay, the state at every chunk start and V', once as the adjoint
 * recurrence from dS_final back to dS0 (dH+ at every chunk, dV'); two per-(chunk, head)
 * tcgen05 kernels then form dq, dk, dv, dg and dbeta, the second forming W and U~ again from
 * its own solve.  With one v-head per key head they write dq and dk themselves; otherwise a
 * last kernel sums them over each key head's v-heads.  Their operands are fp16, each row
 * (or tile) scaled by a power of two; an fp16 operand of the recurrences that leaves its range
 * (|dO| or a gradient of the state beyond 65504) is reported as GDR_ERR_RANGE through the
 * workspace, as in gdr_chunk_fwd.  Other sizes and fp32 ("simt"): fp32 CUDA-core kernels.
 *
 * Outputs are written, never accumulated.  Errors: as gdr_chunk_fwd; GDR_ERR_UNSUPPORTED
 * for sizes or options outside the kernels' range.
 */
size_t gdr_chunk_bwd_workspace_size(const gdr_chunk_args* args);
gdr_status gdr_chunk_bwd(const gdr_chunk_args* args,
                         const void* q, const void* k, const void* v,
                         const void* g, const void* beta,
                         const float* S0, const int32_t* cu_seqlens,
                         const void* dO, const float* dS_final,
                         void* dq, void* dk, void* dv, void* dg, void* dbeta, float* dS0,
                         void* workspace, size_t workspace_bytes, void* stream);

/* Name of the kernel path gdr_chunk_bwd takes for these arguments: "tc" (tcgen05
 * tensor-core kernels), "simt" (fp32 CUDA-core kernels) or NULL if unsupported. */
const char* gdr_chunk_bwd_path(const gdr_chunk_args* args);

/*
 * One-token recurrent decode step (flashrt fused_layer.py `_decode_one`, the
 * recurrent core that reads and writes the cached state once per token).
 */
typedef struct {
    int N;                 /* independent sequences, one token each */
    int Hk, Hv, dk, dv;    /* as in gdr_chunk_args; GPU kernel: dk in {32,64,128},
                              dv a multiple of 32 up to 128 */
    gdr_dtype io_dtype, gate_dtype;
    gdr_read_mode read_mode;
    float scale;
    int qk_l2norm;
    int gate_raw;               /* fused gating prologue, exactly as in gdr_chunk_args */
    const float* gate_A;
    const float* gate_dt_bias;
    float beta_scale;
    /* Fused output epilogue of the decode chain (flashrt fused_layer.py `_decode_one`:
     * rms_norm_gated_silu(core_out, z, norm.weight, eps) applied per head to the
     * recurrent core's output).
     *   out_norm = 0: o is the recurrent output itself; the three fields below are unused.
     *   out_norm = 1: o_j = c_j / sqrt(mean_j(c_j^2) + norm_eps) * norm_weight[j] * silu(z_j)
     *                 per (sequence, head), c the recurrent output in fp32, the mean over the
     *                 dv values of the head, silu(x) = x / (1 + e^-x). */
    int out_norm;
    const void* norm_z;         /* [N, Hv, dv] io_dtype; 16-byte aligned; required when
                                   out_norm */
    const float* norm_weight;   /* [dv] fp32, shared by the heads; 4-byte aligned; required
                                   when out_norm */
    float norm_eps;             /* >= 0, finite */
    /* GDN-2 decoupled gates (tiny_gdn/fugue.py BidirectionalGatedDeltaNet2:
     * S_t = (I - k_t (b_t * k_t)^T) Diag(exp g_t) S_{t-1} + k_t (w_t * v_t)^T).
     *   gdn2 = 0: scalar gates, g and beta of one value per token and value head.
     *   gdn2 = 1: g is the per-key-channel log decay [N, Hv, dk], beta the per-key-channel
     *             erase gate b [N, Hv, dk], and gdn2_w the per-value-channel write gate
     *             [N, Hv, dv], all gate_dtype and 16-byte aligned.  With g = log(alpha),
     *             b = w = beta on every channel this is the scalar rule.  Not combined with
     *             gate_raw. */
    int gdn2;
    const void* gdn2_w;
} gdr_decode_args;

/*
 *   q, k     [N, Hk, dk]  io_dtype      v, o  [N, Hv, dv]  io_dtype
 *   g, beta  [N, Hv]      gate_dtype
 *   S_inout  [N, Hv, dk, dv] fp32, updated in place: every block reads its whole slice
 *            of the state into registers before it writes any of it back, so no scratch
 *            state is needed.
 */
gdr_status gdr_decode_step(const gdr_decode_args* args,
                           const void* q, const void* k, const void* v,
                           const void* g, const void* beta,
                           float* S_inout, void* o, void* stream);

/*
 * ---- Operators around the recurrence --------------------------------------------------------
 *
 * The rest of a recurrent layer: the short causal convolution in front of the delta rule, the
 * gated linear recurrence (diagonal: one state per channel) that can stand beside it or in its
 * place, and the group norm behind either.  They follow the conventions above, with these
 * additions:
 * - The tokens are B rows of T, or with cu_seqlens (B == 1) packed sequences of T tokens
 *   together; sequences of no or one token are allowed.
 * - reverse = 1 runs every sequence from its last token to its first, in place: "scan order"
 *   below is that order, and outputs stand at each token's own position.
 * - No workspace except where a `_workspace_size` is declared.  A cu_seqlens that does not
 *   start at 0, decreases or does not end at T is reported as GDR_ERR_DEVICE_CHECK in
 *   args->status (an optional device int as in gdr_chunk_args); the outputs are then
 *   unspecified, but no access leaves the tensors.  gdr_scan_fwd and gdr_scan_bwd report there
 *   too (GDR_ERR_TIMEOUT) if a bounded wait between the blocks of a cluster ran out; with or
 *   without a status word, every value that misses what was waited for is then NaN.
 * - Channel arrays (weights, biases, their gradients) are fp32 and 4-byte aligned, everything
 *   else 16-byte aligned.  An output (or workspace) that shares bytes with an input or another
 *   output is GDR_ERR_INVALID_ARG unless it is said that it may be that array; then it has to be
 *   the whole of it.
 * - Sums, states and statistics are fp32; results are rounded once.  Repeated calls give the
 *   same bits.  Calls that overlap on the GPU share nothing but their arguments.
 */

/*
 * Gated linear recurrence over D independent channels, alpha_t = exp(g_t):
 *
 *     h_t = alpha_t h_{t-1} + b_t,    o_t = h_t
 *     b_t = v_t                  write = GDR_WRITE_PLAIN
 *     b_t = beta_t v_t           write = GDR_WRITE_GATE
 *     b_t = (1 - alpha_t) v_t    write = GDR_WRITE_TIED
 *
 * g may be -inf (alpha = 0: a finite state is dropped).  Where decays grow (g > 0), their product
 * over any run of tokens of a sequence has to stay in the fp32 range, since runs of tokens are
 * formed at once and joined by it.  A sequence never sees another one's values, infinities and
 * NaN included.
 */
typedef enum { GDR_WRITE_PLAIN = 0, GDR_WRITE_GATE = 1, GDR_WRITE_TIED = 2 } gdr_write;

typedef struct {
    int B, T;              /* rows and tokens per row (with cu_seqlens B must be 1);
                              B * T <= 2^31 - 2^16 */
    int D;                 /* channels (heads times head size), any number >= 1 */
    int n_seqs;            /* == B without cu_seqlens */
    gdr_dtype io_dtype;    /* v, o and their gradients */
    gdr_dtype gate_dtype;  /* g, beta and their gradients */
    gdr_write write;
    int reverse;
    int* status;
} gdr_scan_args;

/*
 *   v, o         [B, T, D] io_dtype
 *   g, beta      [B, T, D] gate_dtype (beta with GDR_WRITE_GATE only, else NULL)
 *   h0           [n_seqs, D] fp32 or NULL for zero
 *   h_final      [n_seqs, D] fp32 or NULL; may alias h0.  An empty sequence keeps its h0.
 */
gdr_status gdr_scan_fwd(const gdr_scan_args* args, const void* v, const void* g,
                        const void* beta, const float* h0, const int32_t* cu_seqlens,
                        void* o, float* h_final, void* stream);

/*
 * Gradients of <dO, o> + <dh_final, h_final> with respect to v, g, beta and h0:
 *     lam_t = dO_t + m_{t+1},  m_t = alpha_t lam_t,  m behind the last token = dh_final
 *     dv = lam | beta lam | (1 - alpha) lam      dbeta = v lam
 *     dg = m h_{t-1}  (TIED: m (h_{t-1} - v))    dh0 = m of the first token
 * h_{t-1} is read from o, as gdr_scan_fwd wrote it (for bf16, with that rounding).
 *   v            not read with GDR_WRITE_PLAIN (may be NULL there)
 *   dh_final     [n_seqs, D] fp32 or NULL for zero;  dh0 [n_seqs, D] fp32 or NULL; may alias
 *                dh_final
 *   dv, dg, dbeta   outputs, shaped and typed as v, g, beta
 */
gdr_status gdr_scan_bwd(const gdr_scan_args* args, const void* v, const void* g,
                        const void* beta, const void* o, const void* dO, const float* h0,
                        const int32_t* cu_seqlens, const float* dh_final, void* dv, void* dg,
                        void* dbeta, float* dh0, void* stream);

/*
 * One token for each of B sequences (T == 1, n_seqs == B): v, g, beta, o [B, D]; the state h
 * [B, D] fp32 is read and the new one written to h_out, which may be h itself.
 */
gdr_status gdr_scan_step(const gdr_scan_args* args, const void* v, const void* g,
                         const void* beta, const float* h, float* h_out, void* o, void* stream);

/*
 * Short causal depthwise convolution with an activation, over scan order:
 *
 *     p_t = bias + sum_{j < width} w[c][width - 1 - j] x_{t-j},   y_t = act(p_t)
 *
 * with the inputs before a sequence's first token taken from its state, or zero.
 */
typedef enum { GDR_ACT_NONE = 0, GDR_ACT_SILU = 1, GDR_ACT_SIGMOID = 2 } gdr_activation;

typedef struct {
    int B, T, D, n_seqs;   /* as in gdr_scan_args */
    int width;             /* 2, 3 or 4 */
    gdr_dtype io_dtype;    /* x, y, the states and their gradients */
    gdr_activation activation;  /* GDR_ACT_NONE or GDR_ACT_SILU */
    int reverse;
    int* status;
} gdr_conv_args;

/*
 *   x, y         [B, T, D] io_dtype;  w [D, width] fp32;  bias [D] fp32 or NULL
 *   state        [n_seqs, width - 1, D] io_dtype, oldest input first, or NULL for zero
 *   state_out    [n_seqs, width - 1, D] io_dtype or NULL: every sequence's last width - 1
 *                inputs (its state's behind them where it is shorter); must not overlap state
 */
gdr_status gdr_conv_fwd(const gdr_conv_args* args, const void* x, const float* w,
                        const float* bias, const void* state, const int32_t* cu_seqlens,
                        void* y, void* state_out, void* stream);

/*
 * Gradients of <dy, y>; p is formed again from x.  dw [D, width], dbias [D] (or NULL), dx
 * [B, T, D], dstate [n_seqs, width - 1, D] io_dtype (or NULL).
 *   workspace    at least gdr_conv_bwd_workspace_size(args) bytes, 256-byte aligned, no
 *                initialisation needed
 */
size_t gdr_conv_bwd_workspace_size(const gdr_conv_args* args);
gdr_status gdr_conv_bwd(const gdr_conv_args* args, const void* x, const float* w,
                        const float* bias, const void* dy, const void* state,
                        const int32_t* cu_seqlens, void* dx, float* dw, float* dbias,
                        void* dstate, void* workspace, size_t workspace_bytes, void* stream);

/*
 * One token for each of B sequences (T == 1, n_seqs == B): x, y [B, D]; state
 * [B, width - 1, D]; state_out receives the state with x appended, and may be state itself.
 */
gdr_status gdr_conv_step(const gdr_conv_args* args, const void* x, const float* w,
                         const float* bias, const void* state, void* state_out, void* y,
                         void* stream);

/*
 * Group norm with an activation, channels last: the H groups are the heads of x [B, T, H, d].
 *
 *     n = (x - mean) / sqrt(var + eps)        center = 1
 *     n = x / sqrt(mean(x^2) + eps)           center = 0
 *     u = n w + bias,    y = u act(z) with a gate z, y = act(u) without
 *
 * The statistics of a group are over the d channels of one token (per_sequence = 0: the output
 * norm of gated_rmsnorm kind, as gdr_decode_step fuses it), or over those of all tokens of a
 * sequence (per_sequence = 1).
 */
typedef struct {
    int B, T, H, d, n_seqs;
    gdr_dtype io_dtype;    /* x, z, y and their gradients */
    int per_sequence;
    int center;
    gdr_activation activation;
    int shared_weight;     /* 1: w, bias and their gradients are [d], for every head; 0: [H, d] */
    float eps;             /* finite, >= 0 */
    int* status;
} gdr_norm_args;

/*
 *   x, z, y      [B, T, H, d] io_dtype; z NULL for no gate
 *   w, bias      fp32 [H, d] or [d]; NULL for ones and zeros
 *   cu_seqlens   read with per_sequence only
 *   stats        [n_seqs, H, 2] fp32 or NULL, per_sequence only: mean (0 without center) and
 *                1 / sqrt(var + eps) of every group, for the backward pass
 *   workspace    at least gdr_norm_fwd_workspace_size(args) bytes (0 unless per_sequence; then
 *                NULL is allowed), 256-byte aligned, no initialisation needed
 * Sizes: d up to 1024 where d elements are a multiple of 16 bytes, else up to 256.
 */
size_t gdr_norm_fwd_workspace_size(const gdr_norm_args* args);
gdr_status gdr_norm_fwd(const gdr_norm_args* args, const void* x, const float* w,
                        const float* bias, const void* z, const int32_t* cu_seqlens, void* y,
                        float* stats, void* workspace, size_t workspace_bytes, void* stream);

/*
 * Gradients of <dy, y>; the normalised values are formed again from x.
 *   stats        as gdr_norm_fwd wrote them; required with per_sequence, else ignored
 *   dx, dz       [B, T, H, d] (dz with z only); dw, dbias shaped as w, bias, or NULL
 */
size_t gdr_norm_bwd_workspace_size(const gdr_norm_args* args);
gdr_status gdr_norm_bwd(const gdr_norm_args* args, const void* x, const float* w,
                        const float* bias, const void* z, const void* dy,
                        const int32_t* cu_seqlens, const float* stats, void* dx, float* dw,
                        float* dbias, void* dz, void* workspace, size_t workspace_bytes,
                        void* stream);

/* Human-readable name of a status. */
const char* gdr_status_string(gdr_status status);

/* Test/diagnostic helper, NOT for the hot path: copies the device error word out of a
 * workspace last used by gdr_chunk_fwd with `args`, SYNCHRONISES `stream`, and returns
 * GDR_OK or the recorded device-side status. */
gdr_status gdr_read_device_error(const gdr_chunk_args* args, const void* workspace,
                                 void* stream);

/* Library version string (also names the target architecture). */
const char* gdr_version(void);

#ifdef __cplusplus
}
#endif

#endif /* GDR_H */

/*
 * kda.h -- C ABI of the GB300 (sm_103a) library for KDA: the forward passes and
 * the recurrence's backward.
 *
 * KDA (Kimi Delta Attention) is a gated delta rule with a per-channel diagonal
 * decay.  Per (sequence n, value head hv), with q/k taken from head
 * h = hv / (HV / H), an fp32 state S of shape [K, V] evolves as
 *
 *     S_t = (I - beta_t k_t k_t^T) Diag(2^{g_t}) S_{t-1} + beta_t k_t v_t^T
 *     o_t = scale * S_t^T q_t,            scale = K^{-1/2} unless given,
 *
 * with g_t <= 0 a base-2 log decay per channel (kernel-fun 0.2.0.dev1 sdist,
 * ALGORITHM.md, preamble; attention-gym PR #317 "Add fused recurrent_kda for
 * decode and inference prefill", PR description).
 *
 * Operations:
 *   kda_gate_cumsum    chunk-local gate cumsum (ALGORITHM.md, Stage 1)
 *   kda_chunk_fwd      chunked forward, BT = 64 (ALGORITHM.md, Stages 1-4)
 *   kda_recurrent_fwd  token-by-token forward for decode (PR #317)
 * each also as an *_act variant that applies the gate and beta activations to
 * raw inputs inside the op (kda_activation below), and
 *   kda_recurrent_bwd  the gradients of the recurrence (ALGORITHM.md, Backward),
 *                      also as kda_recurrent_bwd_act (gradients of the raw inputs)
 *   kda_chunk_bwd      the same gradients in the chunked form on the tensor cores
 *                      (ALGORITHM.md, Backward, the seven launches), also as
 *                      kda_chunk_bwd_act, and after kda_chunk_fwd_save (a forward
 *                      that keeps the backward's recomputed state) without the
 *                      recompute
 *
 * Beside KDA itself, the rest of a recurrent block (see "The recurrent block"):
 *   kda_short_conv_fwd / _bwd / _step   the short causal convolution
 *   kda_ssm_scan_fwd / _bwd, kda_ssm_step   the selective state-space scan
 *   kda_add_rmsnorm_fwd / _bwd          residual addition and RMS norm, 8-bit outputs
 *   kda_gdn_fwd / _bwd / _step          the gated delta rule with one decay per head
 *   kda_gated_rmsnorm_fwd / _bwd        RMS norm in groups with an activated gate
 *   kda_sandwich_norm_fwd / _bwd        the norms after a block and before the next, around the
 *                                       gated, scaled residual stream
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 * Memory.  Every tensor pointer is a DEVICE pointer owned by the caller, on
 * the current CUDA device.  The library allocates no memory and keeps no
 * global state beyond a per-process cache of device attributes and, once a
 * pipelined call has run on a device, streams and events there: one stream and
 * two events for kda_chunk_fwd (KDA_FLAG_SERIAL), up to four streams of the lowest
 * priority with four events each for kda_gdn_fwd and kda_gdn_bwd.  All work is
 * enqueued on `stream` (NULL = the legacy default stream), or ordered by events
 * between what `stream` holds and what comes on it next; calls return without
 * synchronising, except kda_read_device_status.
 *
 * Layouts (all C-contiguous, row-major):
 *   q, k        [B, T, H, K]     dtype `shape->dtype`
 *   v, o        [B, T, HV, V]    dtype `shape->dtype`  (o has q's dtype)
 *   g, g_cum    [B, T, HV, K]    fp32 (the gate is per VALUE head)
 *   beta        [B, T, HV]       dtype `shape->dtype`
 *   h0, ht      [N, HV, K, V]    fp32, K-major state, one entry per sequence
 *   cu_seqlens  [N + 1]          int32, device resident
 * With cu_seqlens == NULL the batch is dense: N = B and row b is one sequence
 * of T tokens.  With cu_seqlens != NULL the batch is packed: B must be 1, T is
 * the physical capacity, and sequence n occupies rows [cu[n], cu[n+1]).
 * Packed-sequence contract (attention-gym PR #317, PR description; review
 * comments on offset validation): offsets must satisfy cu[0] == 0,
 * cu[n] <= cu[n+1] and cu[N] <= T.  Repeated offsets are empty slots whose
 * final state is h0 copied bit for bit (+0.0 when h0 is NULL).  Rows at or
 * beyond cu[N] are outside the contract: never written, and their input values
 * (NaN included) never reach any output.
 *
 * Errors.  Arguments the host can check are checked before anything is
 * enqueued; a failing call returns KDA_ERR_INVALID_ARG or KDA_ERR_UNSUPPORTED,
 * enqueues nothing, and kda_last_error_message() says why.  Offsets live on
 * the device and are validated there on every call (graph replay included):
 * invalid offsets never trap and never cause an out-of-bounds access; the
 * work they govern is skipped and bit KDA_DEVICE_BAD_CU_SEQLENS is OR-ed into
 * *dev_status (when dev_status is not NULL).  Outputs are unspecified for a
 * call whose status word reports an error.  The status word is only written
 * by OR; clear it with kda_clear_device_status.
 */
#ifndef KDA_H_
#define KDA_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Binary-compatible with cudaStream_t. */
typedef struct CUstream_st *kda_stream_t;

typedef enum {
    KDA_OK = 0,
    KDA_ERR_INVALID_ARG = 1,      /* malformed arguments (host-detected)         */
    KDA_ERR_UNSUPPORTED = 2,      /* well-formed but outside the supported set    */
    KDA_ERR_BAD_CU_SEQLENS = 3,   /* reported via the device status word          */
    KDA_ERR_CUDA = 4,             /* a CUDA runtime call or a launch failed        */
    KDA_ERR_TIMEOUT = 5           /* a bounded on-device wait gave up              */
} kda_status;

typedef enum {
    KDA_DTYPE_F32 = 0,            /* q, k, v, beta, o in fp32                     */
    KDA_DTYPE_BF16 = 1            /* q, k, v, beta, o in bf16                     */
} kda_dtype;

/* shape->flags */
#define KDA_FLAG_QK_L2NORM   (1u << 0)  /* L2-normalise q and k rows inside the op:
                                           x / sqrt(sum x^2 + 1e-6)  (kernel-fun
                                           0.2.0.dev1 wheel, kda/autograd.py,
                                           use_qk_l2norm)                          */
#define KDA_FLAG_G_IS_CUMSUM (1u << 1)  /* kda_chunk_fwd only: g already holds the
                                           chunk-local cumsum (kda_gate_cumsum
                                           output with chunk_size 64)             */
#define KDA_FLAG_SPLIT_SCAN  (1u << 2)  /* kda_chunk_fwd, bf16 tensor-core path: for
                                           few long sequences (num_seqs * HV * V / 32
                                           <= 64, T >= 1024, V % 64 == 0) run each
                                           sequence's inter-chunk scan as two
                                           segments at once and compose them after
                                           (h_end = P h_start + E: context parallel
                                           within one GPU).  Needs a larger
                                           workspace (size it with the same flags);
                                           ignored elsewhere.                      */
#define KDA_FLAG_SERIAL      (1u << 3)  /* kda_chunk_fwd: run every launch on the
                                           caller's stream, one after the other.
                                           Without it, a dense bf16 input whose
                                           scan leaves at least half of the SMs
                                           idle is pipelined: while the scan of
                                           each sequence's first chunks runs on
                                           the caller's stream, the prep of the
                                           remaining chunks runs on a library-
                                           owned low-priority stream (forked from
                                           and joined back to the caller's stream
                                           with events, so graph capture sees one
                                           fork and one join) on the other SMs.    */

#define KDA_FLAG_BWD_SAVED   (1u << 4)  /* kda_chunk_bwd: the workspace holds what
                                           kda_chunk_fwd_save stored for the same
                                           inputs, shape and options, so the
                                           forward is not run again (the saved
                                           per-chunk tiles and states are read as
                                           they are; h0 is not read).  Refused by
                                           kda_chunk_fwd_save, ignored by the
                                           other entry points.                     */

#define KDA_FLAG_TEST_WAIT_TIMEOUT (1u << 31)
                                        /* Test hook, kda_chunk_fwd on the bf16
                                           tensor-core path: the scan kernel's MMA
                                           issuer first waits on a barrier that
                                           nothing signals, with a 2 us limit.  The
                                           wait gives up, KDA_DEVICE_TIMEOUT is set,
                                           and the kernel takes the path of any
                                           wait that runs out: no further MMA is
                                           issued, the copies already in flight are
                                           drained (bounded), every warp finishes
                                           its rounds and the kernel returns.  The
                                           outputs of such a call are unspecified;
                                           the context stays usable.  Ignored by
                                           the other kernels.                      */

/* Bits of the device status word. */
#define KDA_DEVICE_BAD_CU_SEQLENS (1 << 0)
#define KDA_DEVICE_TIMEOUT        (1 << 1)
#define KDA_DEVICE_INTERNAL       (1 << 2)  /* a launch found an internal invariant broken
                                               (e.g. the alignment of its shared memory)
                                               and skipped its work; reported as
                                               KDA_ERR_CUDA                            */
#define KDA_DEVICE_GATE_RANGE     (1 << 3)  /* kda_chunk_bwd: a chunk's gate range
                                               max |g2| (log2, chunk-local cumsum of
                                               g_scale g) exceeds 100, or is not
                                               finite; that chunk's gradients were not
                                               computed.  Reported as
                                               KDA_ERR_UNSUPPORTED                     */
#define KDA_DEVICE_BAD_INDEX      (1 << 4)  /* a state index past the last slot (the step
                                               entry points); that row was skipped.
                                               Reported as KDA_ERR_INVALID_ARG         */

typedef struct {
    int32_t B, T, H, HV, K, V;  /* see Layouts; HV % H == 0                         */
    int32_t num_seqs;           /* N: B when dense, len(cu_seqlens) - 1 when packed  */
    kda_dtype dtype;            /* of q, k, v, beta and o                           */
    float scale;                /* readout scale; <= 0 selects K^{-1/2}             */
    float g_scale;              /* multiplier applied to g before use: 1 for base-2
                                   log gates, 1/ln 2 for natural-log gates          */
    uint32_t flags;             /* KDA_FLAG_*                                       */
} kda_shape;

/*
 * Input activations applied inside the op (the *_act entry points).  Defined in
 * kernel-fun 0.2.0.dev1 wheel, kda/chain.py, gate_cumsum, and kda/ops.py,
 * chunk_kda (use_gate_in_kernel, use_beta_sigmoid_in_kernel, allow_neg_eigval);
 * sdist ALGORITHM.md, "Stage 1" note on the fused gate activation.
 *   A_log       [HV] fp32 device pointer, or NULL.  When set, g holds the raw
 *               gate pre-activation and the op uses, in g's place, the
 *               natural-log decay
 *                   -exp(A_log[hv]) * softplus(g[t, hv, d] + dt_bias[hv, d])
 *               (times shape->g_scale as always: 1/ln 2 for this form).
 *               softplus(x) = ln(1 + e^x), evaluated as x itself above 20.
 *   dt_bias     [HV, K] fp32 device pointer, or NULL (no bias); needs A_log.
 *   beta_scale  0: beta is the gate as given.  > 0: beta holds logits and the
 *               op uses sigmoid(beta) * beta_scale (1, or 2 to allow negative
 *               eigenvalues), rounded to the input dtype as the pages cast it to
 *               q's dtype.
 * The pages' lower_bound option has no formula there and is not provided.
 * A NULL kda_activation, or one with A_log == NULL and beta_scale == 0, is the
 * plain op.  The activation cannot be combined with KDA_FLAG_G_IS_CUMSUM.
 */
typedef struct {
    const float *A_log;
    const float *dt_bias;
    float beta_scale;
} kda_activation;

/*
 * kda_gate_cumsum -- chunk-local inclusive cumsum of the gate.
 * Defined in kernel-fun 0.2.0.dev1 sdist, ALGORITHM.md, "Stage 1 -- cumsum":
 *     g_cum[t, hv, d] = g_scale * sum_{s = c(t)}^{t} g[s, hv, d]
 * where c(t) is the first row of t's chunk, chunks of `chunk_size` rows being
 * counted from the first row of t's own sequence.  chunk_size == 1 is the
 * identity (times g_scale), as with attention-gym's bounded_gate_cumsum with
 * chunk_size=1 (PR #317, PR description).
 *   g, g_cum   [B, T, HV, K] fp32; must not alias; rows outside every sequence
 *              of g_cum are not written.
 *   chunk_size 1 <= chunk_size <= 64.
 *   Only B, T, H, HV, K, num_seqs and g_scale of *shape are used (H >= 1).
 */
kda_status kda_gate_cumsum(const float *g, float *g_cum, const int32_t *cu_seqlens,
                           const kda_shape *shape, int32_t chunk_size, int32_t *dev_status,
                           kda_stream_t stream);
/* kda_gate_cumsum with the gate activation of *act applied to g first (its
 * beta_scale is ignored). */
kda_status kda_gate_cumsum_act(const float *g, float *g_cum, const int32_t *cu_seqlens,
                               const kda_shape *shape, const kda_activation *act,
                               int32_t chunk_size, int32_t *dev_status, kda_stream_t stream);

/*
 * kda_chunk_fwd -- the chunked forward with chunks of BT = 64 rows.
 * Defined in kernel-fun 0.2.0.dev1 sdist, ALGORITHM.md, "Forward" (Stage 1
 * cumsum, Stage 2 intra/WY, Stage 3+4 scan + o); arguments and return contract
 * of kernel-fun 0.2.0.dev1 wheel, kda/ops.py, chunk_kda (o in q's dtype, ht
 * only when asked for, a NULL initial state meaning zeros).  Reaches the
 * result of the token recurrence above up to rounding.
 *   q, k, v, g, beta   inputs (Layouts).  g is the per-token log decay unless
 *                      KDA_FLAG_G_IS_CUMSUM is set.
 *   h0                 [N, HV, K, V] fp32 or NULL (zeros).
 *   o                  [B, T, HV, V] output, dtype of q.
 *   ht                 [N, HV, K, V] fp32 final state, or NULL (not stored).
 *                      May alias h0.
 *   workspace          device scratch of at least kda_chunk_workspace_size()
 *                      bytes, 256-byte aligned; its contents on entry do not
 *                      matter and on return are unspecified.  Calls that share
 *                      one workspace must be ordered on the GPU.
 *   stream             the call's work follows earlier work on `stream` and
 *                      later work on it sees the results.  Unless
 *                      KDA_FLAG_SERIAL is set, a dense bf16 call may run some
 *                      launches on a library stream forked from `stream` and
 *                      joined back to it with events (see KDA_FLAG_SERIAL);
 *                      such calls take a host-side lock while they enqueue.
 * Supported: K in {64, 128} with 1 <= V <= 256 (K, V multiples of 16 for bf16);
 * for bf16 also any K that is a multiple of 8 up to 128 when V is a multiple of
 * 32 up to 256 (the tensor-core kernels run such K padded with zero channels).
 */
kda_status kda_chunk_fwd(const void *q, const void *k, const void *v, const float *g,
                         const void *beta, const float *h0, const int32_t *cu_seqlens,
                         const kda_shape *shape, void *o, float *ht, void *workspace,
                         size_t workspace_bytes, int32_t *dev_status, kda_stream_t stream);
/* kda_chunk_fwd on raw g / beta with the activations of *act (see above). */
kda_status kda_chunk_fwd_act(const void *q, const void *k, const void *v, const float *g,
                             const void *beta, const float *h0, const int32_t *cu_seqlens,
                             const kda_shape *shape, const kda_activation *act, void *o,
                             float *ht, void *workspace, size_t workspace_bytes,
                             int32_t *dev_status, kda_stream_t stream);

/* Bytes of workspace kda_chunk_fwd needs for *shape (0 on invalid shapes).  For
 * shapes that may be pipelined it depends on the current device's SM count:
 * size the workspace with the device that will run the call current. */
size_t kda_chunk_workspace_size(const kda_shape *shape);
/* The same number under the name the boundary was first specified with. */
size_t kda_workspace_size(const kda_shape *shape);

/*
 * kda_chunk_fwd_noalloc -- kda_chunk_fwd for callers that cannot allocate
 * device memory at call time (a runtime that owns a fixed, pre-planned memory
 * budget, a plugin host that forbids allocations outside its pool, or a
 * latency-critical loop that cannot afford cudaMalloc's implicit device
 * synchronisation).  The pages have no counterpart to it: it is a property of
 * this library's interface, not of the method.
 *   Arguments, layouts, results and errors are those of kda_chunk_fwd, minus
 *   the workspace: the call uses a scratch array of KDA_NOALLOC_SCRATCH_BYTES
 *   built into the library, which every GPU that loads the library holds until
 *   the process exits.  Shapes whose kda_chunk_workspace_size exceeds it are
 *   rejected with KDA_ERR_UNSUPPORTED and a message; nothing is enqueued.
 *   The call allocates nothing and runs every launch on `stream`, one after
 *   the other (as with KDA_FLAG_SERIAL).  Its first call on a device looks up the
 *   array's device address (cudaGetSymbolAddress) and caches it.  With lazy
 *   module loading (the CUDA default) that lookup is what loads the array onto
 *   the device and reserves its 32 MiB, so it can fail for lack of device
 *   memory (KDA_ERR_CUDA with a message saying so) or wait on the device: make
 *   the first call on each device during set-up, before any stream capture.
 *   Every call on a device shares the one array, so calls that overlap on the
 *   GPU (different streams without ordering) race and give wrong results;
 *   serialise them.  The array keeps the last call's contents; nothing in it
 *   needs to start at zero.
 */
#define KDA_NOALLOC_SCRATCH_BYTES (32u << 20)
kda_status kda_chunk_fwd_noalloc(const void *q, const void *k, const void *v, const float *g,
                                 const void *beta, const float *h0, const int32_t *cu_seqlens,
                                 const kda_shape *shape, void *o, float *ht, int32_t *dev_status,
                                 kda_stream_t stream);

/*
 * kda_recurrent_fwd -- token-by-token forward for decode and inference prefill.
 * Defined in attention-gym PR #317, PR description: one sequential scan over
 * the tokens of each (sequence, head, value block) with the [K, BV] fp32 state
 * held in registers, fp32 arithmetic whatever the input dtype, queries scaled
 * by 1/sqrt(K); work flattened onto grid x so that N * HV beyond 65535 works
 * (PR #317, review comment on grid Y).
 *   g         per-token log decay (KDA_FLAG_G_IS_CUMSUM is rejected).
 *   h0, ht    as for kda_chunk_fwd; ht == h0 (in-place decode) is allowed.
 * Supported: 1 <= K <= 256, 1 <= V (any size; value blocks of 128 columns).
 */
kda_status kda_recurrent_fwd(const void *q, const void *k, const void *v, const float *g,
                             const void *beta, const float *h0, const int32_t *cu_seqlens,
                             const kda_shape *shape, void *o, float *ht, int32_t *dev_status,
                             kda_stream_t stream);
/* kda_recurrent_fwd on raw g / beta with the activations of *act (see above). */
kda_status kda_recurrent_fwd_act(const void *q, const void *k, const void *v, const float *g,
                                 const void *beta, const float *h0, const int32_t *cu_seqlens,
                                 const kda_shape *shape, const kda_activation *act, void *o,
                                 float *ht, int32_t *dev_status, kda_stream_t stream);

/*
 * kda_recurrent_bwd -- gradients of the token recurrence: given do = dL/do and
 * dht = dL/dht, dq, dk, dv, dbeta, dg (with respect to the per-token gate g, the
 * same g kda_recurrent_fwd takes) and dh0.  The contract is kernel-fun
 * 0.2.0.dev1 sdist, ALGORITHM.md, "Backward" (kernel-fun wheel, kda/chain.py,
 * backward: dq, dk, dv, dbeta, dg, dh0; GVA gradients of q and k summed over the
 * value heads that share them); the result is computed for the recurrence the
 * chunked form reaches exactly, in fp32 whatever the input dtype.
 *   q, k, v, g, beta, h0, cu_seqlens, shape   as for kda_recurrent_fwd.
 *   dout               [B, T, HV, V], dtype of q.
 *   dht                [N, HV, K, V] fp32, or NULL (zero).
 *   dq, dk             [B, T, H, K] fp32 outputs; dv [B, T, HV, V]; dg [B, T, HV, K];
 *                      dbeta [B, T, HV]; dh0 [N, HV, K, V] or NULL (not stored).
 *                      Rows outside every sequence are zero.  dq, dk, dg and dbeta
 *                      are summed with atomic adds: their rounding order varies.
 *   workspace          kda_recurrent_bwd_workspace_size() bytes, 16-byte aligned:
 *                      the state at the start of every 8 tokens.
 *   flags              KDA_FLAG_QK_L2NORM: q, k are normalised inside the op (as in
 *                      the forward) and dq, dk are the gradients of the raw rows.
 * Supported: K <= 128, any V; not with KDA_FLAG_G_IS_CUMSUM.
 */
kda_status kda_recurrent_bwd(const void *q, const void *k, const void *v, const float *g,
                             const void *beta, const float *h0, const int32_t *cu_seqlens,
                             const kda_shape *shape, const void *dout, const float *dht,
                             float *dq, float *dk, float *dv, float *dg, float *dbeta, float *dh0,
                             void *workspace, size_t workspace_bytes, int32_t *dev_status,
                             kda_stream_t stream);
/*
 * kda_recurrent_bwd on raw g / beta with the activations of *act (see
 * kda_activation): the forward is kda_recurrent_fwd_act's (or kda_chunk_fwd_act's)
 * and the gradients are those of its inputs.  The chain rule through the
 * activations (kernel-fun 0.2.0.dev1 wheel, kda/chain.py, gate_backward):
 *   dg       with respect to the raw gate g;
 *   dbeta    with respect to the raw beta logits when beta_scale > 0 (the
 *            rounding of the activated beta to the input dtype passes the
 *            gradient through);
 *   dA_log   [HV] fp32, required when act->A_log is set: sum over tokens and
 *            channels of dL/dg' * g', g' the activated gate (zeroed, then summed);
 *   ddt_bias [HV, K] fp32, required when act->dt_bias is set: the sum over tokens
 *            of dg (zeroed, then summed).
 * Both may be NULL when the corresponding input is not set; their rounding
 * order varies (atomic adds).
 */
kda_status kda_recurrent_bwd_act(const void *q, const void *k, const void *v, const float *g,
                                 const void *beta, const float *h0, const int32_t *cu_seqlens,
                                 const kda_shape *shape, const kda_activation *act,
                                 const void *dout, const float *dht, float *dq, float *dk,
                                 float *dv, float *dg, float *dbeta, float *dh0, float *dA_log,
                                 float *ddt_bias, void *workspace, size_t workspace_bytes,
                                 int32_t *dev_status, kda_stream_t stream);
/* Bytes of workspace kda_recurrent_bwd needs for *shape (0 on invalid shapes). */
size_t kda_recurrent_bwd_workspace_size(const kda_shape *shape);

/*
 * kda_chunk_bwd -- the same gradients as kda_recurrent_bwd, computed in the chunked
 * form of kernel-fun 0.2.0.dev1 sdist, ALGORITHM.md, "Backward" (the seven launches:
 * recompute, re-scan, dAv, dhu, wy_dqkg, intra, dg cumsum; kernel-fun wheel,
 * kda/chain.py, backward) on the tensor cores: the forward's prep and scan run again
 * and store, per (chunk, value head), w, Akk, the state at the chunk's start and v';
 * a reverse scan forms dL/dv' and dL/dh per chunk; one kernel per (chunk, value
 * head) then forms dq, dk, dv, dbeta and dg.  Operands are bf16 (the inputs, the
 * checkpoints and the intermediate gradients), accumulation fp32.
 *   q, k, v, g, beta, h0, cu_seqlens, shape   as for kda_chunk_fwd.
 *   dout, dht, dq, dk, dv, dg, dbeta, dh0     as for kda_recurrent_bwd.  With
 *                      HV > H, dq and dk are summed over the value heads that share
 *                      a q/k head with atomic adds (their rounding order varies);
 *                      with HV == H every element is stored once and the result is
 *                      deterministic.  With cu_seqlens, rows outside every sequence
 *                      are zero.  A chunk refused for its gate range gets zero
 *                      gradients (and KDA_DEVICE_GATE_RANGE).
 *   workspace          kda_chunk_bwd_workspace_size() bytes, 256-byte aligned.
 *   flags              KDA_FLAG_QK_L2NORM (q, k normalised inside the op; dq, dk
 *                      are the raw rows' gradients), KDA_FLAG_SERIAL and
 *                      KDA_FLAG_BWD_SAVED (the workspace holds kda_chunk_fwd_save's
 *                      stores for these inputs: the recompute and re-scan are
 *                      skipped); a cumsummed gate takes kda_recurrent_bwd.
 * Supported: bf16, K = V = 128.  A chunk whose gate range is too wide raises
 * KDA_DEVICE_GATE_RANGE in *dev_status.  Tensors 16-byte aligned.
 */
kda_status kda_chunk_bwd(const void *q, const void *k, const void *v, const float *g,
                         const void *beta, const float *h0, const int32_t *cu_seqlens,
                         const kda_shape *shape, const void *dout, const float *dht, float *dq,
                         float *dk, float *dv, float *dg, float *dbeta, float *dh0,
                         void *workspace, size_t workspace_bytes, int32_t *dev_status,
                         kda_stream_t stream);
/*
 * kda_chunk_bwd on raw g / beta with the activations of *act (see kda_activation), the
 * forward being kda_chunk_fwd_act's: the gradients of the raw inputs, dA_log and
 * ddt_bias as for kda_recurrent_bwd_act.  With KDA_FLAG_QK_L2NORM (either entry point)
 * the rows are normalised inside the op and dq, dk are the raw rows' gradients.  The
 * kernels form the gradients of the normalised rows and the activated gate and beta;
 * the chain rules follow in two elementwise passes (the ones kda_recurrent_bwd uses).
 */
kda_status kda_chunk_bwd_act(const void *q, const void *k, const void *v, const float *g,
                             const void *beta, const float *h0, const int32_t *cu_seqlens,
                             const kda_shape *shape, const kda_activation *act, const void *dout,
                             const float *dht, float *dq, float *dk, float *dv, float *dg,
                             float *dbeta, float *dh0, float *dA_log, float *ddt_bias,
                             void *workspace, size_t workspace_bytes, int32_t *dev_status,
                             kda_stream_t stream);
/*
 * kda_chunk_fwd_save -- the chunked forward of kda_chunk_fwd_act (act may be NULL:
 * kda_chunk_fwd), the same o and ht bit for bit, that also leaves in `workspace`
 * what kda_chunk_bwd re-derives in its first two stages (recompute and re-scan of
 * kernel-fun 0.2.0.dev1 sdist, ALGORITHM.md, "Backward"): per (chunk, value head)
 * the operand tiles, w, Akk, the state at the chunk's start and v', and every
 * sequence's final state.  A later kda_chunk_bwd (or _act) of the same inputs,
 * shape, options and workspace with KDA_FLAG_BWD_SAVED then starts at the reverse
 * scan: memory (kda_chunk_bwd_workspace_size bytes held from the forward to the
 * backward) for the forward's second run.
 *   arguments          as for kda_chunk_fwd_act; ht may be NULL.
 *   workspace          kda_chunk_bwd_workspace_size() bytes, 256-byte aligned,
 *                      owned by the caller and left untouched until the backward.
 *   flags              KDA_FLAG_QK_L2NORM and KDA_FLAG_SERIAL.
 * Supported: bf16, K = V = 128 (as kda_chunk_bwd).
 */
kda_status kda_chunk_fwd_save(const void *q, const void *k, const void *v, const float *g,
                              const void *beta, const float *h0, const int32_t *cu_seqlens,
                              const kda_shape *shape, const kda_activation *act, void *o,
                              float *ht, void *workspace, size_t workspace_bytes,
                              int32_t *dev_status, kda_stream_t stream);

/* Bytes of workspace kda_chunk_bwd needs for *shape (0 on invalid shapes).  As for
 * kda_chunk_workspace_size, a shape that may be packed (B == 1) is sized for packed
 * input, which covers a dense call of the same shape too. */
size_t kda_chunk_bwd_workspace_size(const kda_shape *shape);

/* ------------------------------------------------------------------------------
 * The recurrent block around KDA: the short causal convolution in front of the state
 * update, the selective state-space scan (the delta rule's sibling: one decay per head
 * and no delta correction), and the residual RMS norm at the block's entry.
 *
 * Conventions are those above (device pointers, streams, errors, packed sequences),
 * with these additions.
 * Strides.  Inputs that a layer cuts out of one projection may be column ranges of a
 * wider tensor: x_stride etc. are the elements between the rows of consecutive tokens
 * (0: contiguous rows); the columns of a row are contiguous and row (b, t) is row
 * b * T + t.  A call takes up to 2^31 - 256 rows (B T).  Outputs are contiguous.  Any
 * alignment of the element type is taken; rows that start on 16-byte boundaries are faster.
 * Outputs must not overlap inputs, or each other, but where an entry says that they may.
 * State caches.  The step entry points update one row of a cache per batch row, in
 * place: state_indices[n] is row n's slot (NULL: slot n).  A negative entry marks an
 * unused batch row: no state is touched and its output is zero.  An entry past the last
 * slot sets KDA_DEVICE_BAD_INDEX, and its row is skipped like an unused one.  Entries must
 * be distinct: two rows of one slot race.
 * Non-finite inputs make the outputs that depend on them non-finite, and of the forward
 * functions, the steps, the convolution's and the norm's gradients no others.  In the scan's
 * gradients they may reach further: to all rows of their chunk (up to 128 rows of the same
 * sequence) in the same head, and in dB and dC in the same group.  In the gated delta rule's
 * chunked forward and in its gradients they may reach every row of their sequence in the same value
 * head from their chunk's first row on (the gradients: any row), and in dq and dk in the heads that
 * share a q/k head with it.
 */

/* flags of kda_conv_shape */
#define KDA_CONV_FLAG_SILU (1u << 0)      /* y = pre * sigmoid(pre); without it y = pre */

typedef struct {
    int32_t B, T, C, W;         /* W taps: 2, 3 or 4                                    */
    int32_t num_seqs;           /* N: B when dense, len(cu_seqlens) - 1 when packed      */
    kda_dtype dtype;            /* of x, y, the states and their gradients              */
    int64_t x_stride;           /* elements between x's rows (0: C)                     */
    uint32_t flags;             /* KDA_CONV_FLAG_*                                      */
} kda_conv_shape;

/*
 * kda_short_conv_fwd -- y_t[c] = act(bias[c] + sum_{k < W} w[c, k] x_{t-W+1+k}[c]), rows
 * before a sequence's first being its carried state (or zero).
 *   x          [B, T, C];  w [C, W] fp32;  bias [C] fp32 or NULL
 *   state_in   [N, W-1, C] or NULL (zeros): the rows before each sequence, oldest first
 *   y          [B, T, C]; rows outside every sequence are not written
 *   state_out  [N, W-1, C] or NULL: the last W-1 rows of (state_in, x) per sequence (an
 *              empty sequence keeps its state).  Must not alias state_in.
 */
kda_status kda_short_conv_fwd(const void *x, const float *w, const float *bias,
                              const void *state_in, const int32_t *cu_seqlens,
                              const kda_conv_shape *shape, void *y, void *state_out,
                              int32_t *dev_status, kda_stream_t stream);
/*
 * kda_short_conv_bwd -- the gradients for dy = dL/dy and dstate_out = dL/dstate_out (or
 * NULL): dx [B, T, C] and dstate_in [N, W-1, C] (or NULL, not stored) in the shape's type, dw [C, W] and
 * dbias [C] (or NULL) fp32, summed in a fixed order.  With cu_seqlens, dx is zero in rows
 * outside every sequence.
 *   workspace  kda_short_conv_bwd_workspace_size() bytes, 16-byte aligned.
 */
kda_status kda_short_conv_bwd(const void *x, const float *w, const float *bias,
                              const void *state_in, const int32_t *cu_seqlens,
                              const kda_conv_shape *shape, const void *dy, const void *dstate_out,
                              void *dx, float *dw, float *dbias, void *dstate_in, void *workspace,
                              size_t workspace_bytes, int32_t *dev_status, kda_stream_t stream);
size_t kda_short_conv_bwd_workspace_size(const kda_conv_shape *shape);
/*
 * kda_short_conv_step -- one token for each of shape->B batch rows (T = 1): y [B, C] and
 * the state cache [num_slots, W-1, C] moved on by one row, in place.
 */
kda_status kda_short_conv_step(const void *x, const float *w, const float *bias, void *state,
                               const int32_t *state_indices, int32_t num_slots,
                               const kda_conv_shape *shape, void *y, int32_t *dev_status,
                               kda_stream_t stream);

/* flags of kda_ssm_shape */
#define KDA_SSM_FLAG_DT_SOFTPLUS (1u << 0) /* the step is softplus(dt + dt_bias), not
                                              dt + dt_bias                              */
#define KDA_SSM_FLAG_NO_SAVE (1u << 2)     /* of a forward: its workspace will not be given
                                              to the backward as `saved`, and is smaller */

typedef struct {
    int32_t B, T, H, G, N, P;   /* H heads in G groups (H % G == 0), N state rows and P
                                   columns per head: 1 <= N, P <= 256                   */
    int32_t num_seqs;           /* B when dense, len(cu_seqlens) - 1 when packed        */
    kda_dtype dtype;            /* of x, dt, Bm, Cm, y and their gradients              */
    int64_t x_stride, dt_stride, b_stride, c_stride;  /* elements between rows (0:
                                   contiguous: H P, H, G N, G N)                        */
    uint32_t flags;             /* KDA_SSM_FLAG_*                                       */
} kda_ssm_shape;

/*
 * kda_ssm_scan_fwd -- the selective state-space scan.  Per sequence and head h, with B_t,
 * C_t from group h / (H / G), step d_t (see the flag) and A = -exp(A_log[h]):
 *     S_t = exp(d_t A) S_{t-1} + d_t B_t x_t^T,      y_t = S_t^T C_t + D[h] x_t
 *   x          [B, T, H, P];  dt [B, T, H];  Bm, Cm [B, T, G, N]
 *   A_log      [H] fp32;  D, dt_bias [H] fp32 or NULL
 *   h0, ht     [num_seqs, H, N, P] fp32 or NULL, as for kda_chunk_fwd; ht may alias h0
 *   y          [B, T, H, P]; rows outside every sequence are not written
 *   workspace  kda_ssm_workspace_size() bytes, 256-byte aligned.  It holds the state at
 *              each chunk's start on return: kda_ssm_scan_bwd takes it as `saved` (not
 *              with KDA_SSM_FLAG_NO_SAVE, which leaves out what only the backward reads).
 * Steps that are >= 0 keep every decay <= 1; they are not checked.
 */
kda_status kda_ssm_scan_fwd(const void *x, const void *dt, const float *A_log, const void *Bm,
                            const void *Cm, const float *D, const float *dt_bias, const float *h0,
                            const int32_t *cu_seqlens, const kda_ssm_shape *shape, void *y,
                            float *ht, void *workspace, size_t workspace_bytes,
                            int32_t *dev_status, kda_stream_t stream);
size_t kda_ssm_workspace_size(const kda_ssm_shape *shape);
/*
 * kda_ssm_scan_bwd -- the gradients for dy = dL/dy and dht = dL/dht (or NULL): dx, ddt,
 * dB, dC in the shape's type and the inputs' (contiguous) layouts; dA_log, dD, ddt_bias
 * [H] fp32 (dD, ddt_bias may be NULL: not stored); dh0 [num_seqs, H, N, P] fp32 or NULL.
 * dB and dC are summed over a group's heads, the [H] gradients over all tokens, each in a
 * fixed order.  With cu_seqlens, rows outside every sequence are zero.
 * KDA_SSM_FLAG_NO_SAVE is refused.
 *   saved      the workspace of kda_ssm_scan_fwd for the same inputs and shape, untouched
 *              since, or NULL: the chunk states are formed again
 *   workspace  kda_ssm_bwd_workspace_size(shape, saved != NULL) bytes, 256-byte aligned.
 */
kda_status kda_ssm_scan_bwd(const void *x, const void *dt, const float *A_log, const void *Bm,
                            const void *Cm, const float *D, const float *dt_bias, const float *h0,
                            const int32_t *cu_seqlens, const kda_ssm_shape *shape, const void *dy,
                            const float *dht, void *dx, void *ddt, void *dB, void *dC,
                            float *dA_log, float *dD, float *ddt_bias, float *dh0,
                            const void *saved, void *workspace, size_t workspace_bytes,
                            int32_t *dev_status, kda_stream_t stream);
size_t kda_ssm_bwd_workspace_size(const kda_ssm_shape *shape, int saved);
/*
 * kda_ssm_step -- one token for each of shape->B batch rows (T = 1): y [B, H, P] and the
 * state cache [num_slots, H, N, P] fp32 advanced in place.
 */
kda_status kda_ssm_step(const void *x, const void *dt, const float *A_log, const void *Bm,
                        const void *Cm, const float *D, const float *dt_bias, float *state,
                        const int32_t *state_indices, int32_t num_slots,
                        const kda_ssm_shape *shape, void *y, int32_t *dev_status,
                        kda_stream_t stream);

typedef enum {
    KDA_NORM_SAME = 0,          /* y in the input's type                                */
    KDA_NORM_E4M3 = 1,          /* 8-bit floats (4 exponent bits, 3 fraction bits), top 448 */
    KDA_NORM_INT8 = 2           /* 8-bit integers, top 127                              */
} kda_norm_out;

typedef struct {
    int64_t rows;
    int32_t cols;               /* 1 .. 16384                                           */
    kda_dtype dtype;            /* of x, residual, h and their gradients                */
    kda_norm_out out;
    int32_t group;              /* 8-bit outputs: columns per scale: 0 (the row) or 128 */
    float eps;                  /* >= 0                                                 */
} kda_norm_shape;

/*
 * kda_add_rmsnorm_fwd -- h = x + residual (residual NULL: h = x),
 *     y = h w / sqrt(mean(h^2) + eps),
 * and for the 8-bit outputs, per row or group of columns, scale = max|y| / top (1 where
 * every y is 0, at least the smallest normal number elsewhere, and not a number where a y
 * is not) and q = y (1 / scale), the reciprocal and the product each rounded in fp32, then
 * rounded to the output's type, ties to even.
 *   x, residual, h  [rows, cols] (h may be NULL: not stored); the norm takes the unrounded sum
 *   w               [cols] fp32
 *   y               [rows, cols]: the shape's type, or one byte per element
 *   scale           [rows, groups] fp32, groups = ceil(cols / group) (1 without); 8-bit only
 */
kda_status kda_add_rmsnorm_fwd(const void *x, const void *residual, const float *w,
                               const kda_norm_shape *shape, void *h, void *y, float *scale,
                               kda_stream_t stream);
/*
 * kda_add_rmsnorm_bwd -- the gradients at the stored h for dy = dL/dy and dh = dL/dh of
 * the residual stream (or NULL): dx [rows, cols] (x's and the residual's alike) in the
 * shape's type, dw [cols] fp32 summed in a fixed order.  shape->out and group are ignored.
 *   workspace  kda_add_rmsnorm_bwd_workspace_size() bytes, 16-byte aligned.
 */
kda_status kda_add_rmsnorm_bwd(const void *dy, const void *h, const float *w, const void *dh,
                               const kda_norm_shape *shape, void *dx, float *dw, void *workspace,
                               size_t workspace_bytes, kda_stream_t stream);
size_t kda_add_rmsnorm_bwd_workspace_size(const kda_norm_shape *shape);

/* ------------------------------------------------------------------------------
 * The gated delta rule with one decay per head.  KDA's sibling with a scalar gate: per
 * (sequence, value head hv), with q and k of head hv / (HV / H) and a base-2 log decay g_t,
 *     S_t = 2^{g_t} S_{t-1} + beta_t k_t (v_t - (2^{g_t} S_{t-1})^T k_t)^T,   o_t = scale S_t^T q_t.
 * Every exponent is a difference of cumulative decays taken before the exponential, so that
 * no range of g <= 0 is refused in either direction; g = -inf drops the state before the row.
 * The conventions are the recurrent block's.
 */

/* flags of kda_gdn_shape */
#define KDA_GDN_FLAG_QK_L2NORM (1u << 0)   /* q and k rows normalised inside the op:
                                              x / sqrt(sum x^2 + 1e-6)                  */
#define KDA_GDN_FLAG_NO_SAVE (1u << 1)     /* of a forward: its workspace will not be given
                                              to the backward as `saved`, and may be smaller */
#define KDA_GDN_FLAG_TEST_WAIT_TIMEOUT (1u << 31)  /* test hook of kda_gdn_fwd and kda_gdn_bwd: the
                                              kernels' waits for copies give up at once,
                                              KDA_DEVICE_TIMEOUT is set and they take the path of
                                              any wait that runs out.  Outputs are undefined;
                                              never set it in use.                           */

typedef struct {
    int32_t B, T, H, HV, K, V;  /* HV % H == 0; 1 <= K, V <= 256                        */
    int32_t num_seqs;           /* B when dense, len(cu_seqlens) - 1 when packed        */
    kda_dtype dtype;            /* of q, k, v, beta, o and their gradients              */
    float scale;                /* readout scale; <= 0 selects K^{-1/2}                 */
    float g_scale;              /* multiplier of g: 1 for base-2, 1/ln 2 for natural    */
    int64_t q_stride, k_stride, v_stride;  /* elements between rows (0: contiguous: H K,
                                   H K, HV V)                                           */
    uint32_t flags;             /* KDA_GDN_FLAG_*                                       */
} kda_gdn_shape;

/*
 * kda_gdn_fwd -- the chunked forward.  Dense calls of long sequences and few heads, outside a
 * stream capture, run in two parts that overlap on a stream of the library's own, which waits
 * for `stream` and is waited for on it.  A call never waits for another stream's: where every
 * stream of the library's still has some of another's work, it runs in one part, with the same bits.
 *   q, k       [B, T, H, K];  v [B, T, HV, V];  beta [B, T, HV]
 *   g          [B, T, HV] fp32
 *   h0, ht     [num_seqs, HV, K, V] fp32 or NULL, as for kda_chunk_fwd; ht may alias h0
 *   o          [B, T, HV, V]; rows outside every sequence are not written
 *   workspace  kda_gdn_workspace_size() bytes, 256-byte aligned.  On return it holds what
 *              kda_gdn_bwd takes as `saved` (not with KDA_GDN_FLAG_NO_SAVE).
 */
kda_status kda_gdn_fwd(const void *q, const void *k, const void *v, const float *g, const void *beta,
                       const float *h0, const int32_t *cu_seqlens, const kda_gdn_shape *shape, void *o,
                       float *ht, void *workspace, size_t workspace_bytes, int32_t *dev_status,
                       kda_stream_t stream);
size_t kda_gdn_workspace_size(const kda_gdn_shape *shape);
/*
 * kda_gdn_bwd -- the gradients for dout = dL/do and dht = dL/dht (or NULL): dq, dk, dv, dbeta in
 * the shape's type and the inputs' (contiguous) layouts, dg [B, T, HV] fp32, dh0 [num_seqs, HV,
 * K, V] fp32 or NULL.  dq and dk are summed over the value heads that share them in a fixed
 * order.  With cu_seqlens, rows outside every sequence are zero.  KDA_GDN_FLAG_NO_SAVE is refused.
 * No gradient may alias an input; dh0 may alias dht.
 *   saved      the workspace of kda_gdn_fwd for the same inputs and shape, untouched since, or
 *              NULL: the forward's states are formed again
 *   workspace  kda_gdn_bwd_workspace_size(shape, saved != NULL) bytes, 256-byte aligned.
 */
kda_status kda_gdn_bwd(const void *q, const void *k, const void *v, const float *g, const void *beta,
                       const float *h0, const int32_t *cu_seqlens, const kda_gdn_shape *shape,
                       const void *dout, const float *dht, void *dq, void *dk, void *dv, float *dg,
                       void *dbeta, float *dh0, const void *saved, void *workspace,
                       size_t workspace_bytes, int32_t *dev_status, kda_stream_t stream);
size_t kda_gdn_bwd_workspace_size(const kda_gdn_shape *shape, int saved);
/*
 * kda_gdn_step -- one token for each of shape->B batch rows (T = 1): o [B, HV, V] and the state
 * cache [num_slots, HV, K, V] fp32 advanced in place.  o must not alias q, k or v.
 */
kda_status kda_gdn_step(const void *q, const void *k, const void *v, const float *g, const void *beta,
                        float *state, const int32_t *state_indices, int32_t num_slots,
                        const kda_gdn_shape *shape, void *o, int32_t *dev_status, kda_stream_t stream);

/* ------------------------------------------------------------------------------
 * The norms around a gated block.  rms(x) = x / sqrt(mean(x^2) + eps).  The conventions are the
 * recurrent block's: outputs overlap neither inputs nor each other.  Values that are not finite reach
 * their row (in the gated norm their group of it) and, in the gradients, the weights' gradients
 * of its columns.
 */
typedef enum {
    KDA_GATE_SIGMOID = 0,       /* act(z) = sigmoid(z)                                  */
    KDA_GATE_SILU = 1           /* act(z) = z sigmoid(z)                                */
} kda_gate_act;

typedef struct {
    int64_t rows;
    int32_t cols;               /* a multiple of group, up to 131072                    */
    int32_t group;              /* columns normalised together (a head): 1 .. 16384     */
    kda_dtype dtype;            /* of x, gate, y and their gradients                    */
    kda_gate_act act;
    int32_t gate_first;         /* 0: rms(x) w act(gate); 1: rms(x act(gate)) w         */
    int32_t shared_weight;      /* 1: w [group], the same in every group; 0: w [cols]   */
    float eps;                  /* >= 0                                                 */
    int64_t x_stride, gate_stride;  /* elements between rows (0: cols)                  */
} kda_gated_norm_shape;

/* kda_gated_rmsnorm_fwd -- y [rows, cols] from x, gate [rows, cols] and w (fp32). */
kda_status kda_gated_rmsnorm_fwd(const void *x, const void *gate, const float *w,
                                 const kda_gated_norm_shape *shape, void *y, kda_stream_t stream);
/*
 * kda_gated_rmsnorm_bwd -- the gradients for dy = dL/dy [rows, cols]: dx and dgate (contiguous) in the
 * shape's type, dw fp32 in w's shape, summed in a fixed order.
 *   workspace  kda_gated_rmsnorm_bwd_workspace_size() bytes, 16-byte aligned.
 */
kda_status kda_gated_rmsnorm_bwd(const void *dy, const void *x, const void *gate, const float *w,
                                 const kda_gated_norm_shape *shape, void *dx, void *dgate, float *dw,
                                 void *workspace, size_t workspace_bytes, kda_stream_t stream);
size_t kda_gated_rmsnorm_bwd_workspace_size(const kda_gated_norm_shape *shape);

typedef struct {
    int64_t rows;
    int32_t cols;               /* 1 .. 16384                                           */
    kda_dtype dtype;            /* of x, residual, gate, h, y and their gradients       */
    kda_gate_act act;           /* of the gate, if there is one                         */
    float eps;                  /* >= 0, of both norms                                  */
} kda_sandwich_shape;

/*
 * kda_sandwich_norm_fwd -- what stands between a block's output x and the next block's input y:
 *     h = residual_scale residual + act(gate) rms(x) w_post,      y = rms(h) w_pre
 *   x, residual, gate, h, y  [rows, cols] (gate may be NULL: 1); the second norm takes the
 *                            unrounded h
 *   w_post, w_pre            [cols] fp32;  residual_scale [cols] fp32 or NULL (1)
 */
kda_status kda_sandwich_norm_fwd(const void *x, const void *residual, const void *gate,
                                 const float *w_post, const float *w_pre, const float *residual_scale,
                                 const kda_sandwich_shape *shape, void *h, void *y, kda_stream_t stream);
/*
 * kda_sandwich_norm_bwd -- the gradients for dy = dL/dy and dh = dL/dh of the residual stream (or
 * NULL), at the unrounded h (formed again): dx, dresidual and dgate (with a gate) in the shape's
 * type; dw_post, dw_pre and dresidual_scale (with a scale) [cols] fp32, summed in a fixed order.
 *   workspace  kda_sandwich_norm_bwd_workspace_size() bytes, 16-byte aligned.
 */
kda_status kda_sandwich_norm_bwd(const void *dy, const void *dh, const void *x, const void *residual,
                                 const void *gate, const float *w_post, const float *w_pre,
                                 const float *residual_scale, const kda_sandwich_shape *shape, void *dx,
                                 void *dresidual, void *dgate, float *dw_post, float *dw_pre,
                                 float *dresidual_scale, void *workspace, size_t workspace_bytes,
                                 kda_stream_t stream);
size_t kda_sandwich_norm_bwd_workspace_size(const kda_sandwich_shape *shape);

/*
 * kda_read_device_status -- synchronise `stream`, copy the status word to
 * *host_bits (may be NULL) and map it to a status: KDA_OK when no bit is set,
 * KDA_ERR_BAD_CU_SEQLENS, KDA_ERR_TIMEOUT or, for KDA_DEVICE_BAD_INDEX,
 * KDA_ERR_INVALID_ARG otherwise.  Does not clear it.
 */
kda_status kda_read_device_status(const int32_t *dev_status, int32_t *host_bits,
                                  kda_stream_t stream);

/* kda_clear_device_status -- enqueue a reset of the status word to 0. */
kda_status kda_clear_device_status(int32_t *dev_status, kda_stream_t stream);

/*
 * Stage timing for benchmarks (not needed for correct use).  While enabled,
 * every kernel the library enqueues is bracketed by two CUDA events recorded
 * on the caller's stream; do not enable it around stream capture.
 * kda_profile_report synchronises the recorded events and writes up to
 * max_entries rows: the kernel's name (NUL-separated into names, at most
 * names_len bytes), its summed duration in milliseconds and its launch count.
 * It returns the number of rows (or -1 on a CUDA error).  Reset clears the
 * totals.  Process-wide, guarded by a mutex.
 */
kda_status kda_profile_enable(int enable);
int kda_profile_report(char *names, size_t names_len, double *total_ms, int64_t *launches,
                       int max_entries);
void kda_profile_reset(void);

/*
 * Peak fp32 FMA throughput of the current device, measured: a kernel of 16
 * independent FMA chains per thread on 8 x 256 threads per SM, timed with CUDA
 * events on `stream` (best of three after a warm-up launch), in TFLOP/s (two
 * flops per FMA).  The roofline denominator for the fp32-bound kernels (the
 * recurrent prefill and backward).  Synchronises the stream.
 */
kda_status kda_measure_fp32_fma_peak(double *tflops, kda_stream_t stream);

/* Static text for a status code. */
const char *kda_status_string(kda_status status);

/* Reason for the most recent non-OK return on the calling host thread. */
const char *kda_last_error_message(void);

/* Library version, "major.minor.patch". */
const char *kda_version(void);

#ifdef __cplusplus
}
#endif

#endif /* KDA_H_ */

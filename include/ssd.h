/*
 * ssd.h — C ABI of the GB300 (sm_103a) selective state-space scan library.
 *
 * The library computes one selective state-space scan and its vector-Jacobian
 * product (VJP) on the GPU, for three forms of the recurrence:
 *
 *   Mamba-2 (SSD_MAMBA2), one scalar decay per head, B and C shared by the
 *   heads of a group:
 *       dt'_t = softplus(dt_raw_t)
 *       s_t   = exp(dt'_t * A_h) * s_{t-1} + dt'_t * x_t (outer) B_t
 *       y_t   = s_t . C_t                     (the updated state s_t)
 *   Mamba-1 (SSD_MAMBA1), one decay per state:
 *       s_t[n] = exp(dt'_t * A[d,n]) * s_{t-1}[n] + dt'_t * x_t * B_t[n]
 *       y_t    = sum_n s_t[n] * C_t[n]
 *   MIMO rank R (SSD_MIMO), the form of one pass of the Mamba-3 scan:
 *       s_t     = exp(da_t) * s_{t-1} + sum_r v_{t,r} (outer) B_{t,r}
 *       y_{t,r} = s_t . C_{t,r}
 *
 * Sources (the pages the method is taken from):
 *   - "S1-31: SSM_SCAN_BACK — Mamba has a backward" (llama.cpp PR text),
 *     opening paragraph: the reverse recurrence, the Mamba-2 and Mamba-1
 *     branches and the five gradients; "Two things that are easy to get
 *     wrong", item 1: the final-state gradient is a nonzero seed; item 2:
 *     the backward needs s_{t-1} and recomputes the states; verification
 *     table: the softplus derivative belongs in d(dt_raw).
 *   - burn-mamba "combined_backward.rs" (Mamba-3 double-SSD, serial
 *     recalculated): CombinedGrads (one gradient per input, including the
 *     initial state), the chunkwise K1..K5 forward and the recompute backward
 *     (replay K1..K4 from the saved leaf inputs, reverse per-chunk loop
 *     fusing the K5 and K4 backwards, then batched K3/K2/K1 backwards).
 *
 * Conventions for every call:
 *   - All tensor arguments are DEVICE pointers to contiguous row-major
 *     arrays owned by the caller.  The library allocates nothing: scratch
 *     memory is the caller's workspace, sized by ssd_workspace_size().
 *   - Work is enqueued asynchronously on `cuda_stream` (a cudaStream_t; NULL
 *     is the legacy default stream).  A call returns once its kernels are
 *     enqueued.  Buffers must stay valid until the stream reaches them.
 *   - Arguments are validated before anything is launched; on any error no
 *     kernel runs and no output is written.
 *   - Results are bitwise reproducible: the same inputs on the same GPU give
 *     the same bits on every call (all reductions run in a fixed order; no
 *     floating-point atomics).
 *   - Calls on different streams with different buffers (including different
 *     workspaces) may run concurrently.  A workspace must not be shared by
 *     calls that may overlap on the GPU.
 */
#ifndef SSD_GB300_H
#define SSD_GB300_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  SSD_OK = 0,
  SSD_ERR_INVALID_ARG = 1, /* NULL where a buffer is required, unknown enum, negative size */
  SSD_ERR_SHAPE = 2,       /* sizes the method does not allow (H % G, limits of this build) */
  SSD_ERR_DTYPE = 3,       /* io dtype not supported for this variant */
  SSD_ERR_ALIGNMENT = 4,   /* a pointer is not 16-byte aligned */
  SSD_ERR_WORKSPACE = 5,   /* ws_bytes smaller than ssd_workspace_size() */
  SSD_ERR_CUDA = 6,        /* a CUDA runtime call or kernel launch failed */
  SSD_ERR_TIMEOUT = 7,     /* the device status word is nonzero: a bounded device-side wait gave up */
  SSD_ERR_INTERNAL = 8,    /* a device-side consistency check failed */
  SSD_ERR_TOO_LARGE = 9    /* ssd_forward_static: the problem needs more scratch than its fixed array */
} ssd_status;

typedef enum { SSD_MAMBA2 = 0, SSD_MAMBA1 = 1, SSD_MIMO = 2 } ssd_variant;

typedef enum { SSD_F32 = 0, SSD_BF16 = 1 } ssd_dtype;

/*
 * Problem description.
 *   variant    ssd_variant.
 *   io_dtype   ssd_dtype of x, B, C, y, dy, dx, dB, dC (and of v, dv for
 *              MIMO).  dt_raw, A, s0, s_final, ds_final, ds0, ddt_raw, dA are
 *              always fp32.  Mamba-1 supports SSD_F32 only.
 *   batch      b >= 1 independent sequences.
 *   seqlen     T >= 1 steps.
 *   nheads     H heads (Mamba-2, MIMO) or D channels (Mamba-1).
 *   headdim    P (Mamba-2, MIMO); must be 1 for Mamba-1.
 *   dstate     N state size.
 *   ngroups    G groups of consecutive heads sharing B and C (Mamba-2;
 *              H % G == 0, head h reads group h / (H/G)).  Ignored for
 *              Mamba-1 (B, C are shared by all channels) and MIMO (B, C are
 *              per head).
 *   chunk      L, the chunk length of the chunkwise algorithm (Mamba-2,
 *              MIMO), 1 <= L <= 256.  Mamba-1 has no chunkwise form: its
 *              kernels walk the sequence step by step (checkpointing the
 *              state every 8 steps in the backward) and accept any
 *              1 <= L <= 256 here.  T need not be a multiple of L: the sequence is cut
 *              into nc = ceil(T / L) chunks, and the last one holds the
 *              remaining T - (nc - 1) L steps (a tail chunk).  The kernels
 *              treat its missing steps as steps with dt' = 0 (da = 0) and
 *              x = B = C = dy = 0, which leave the state unchanged, and store
 *              nothing for them, so every output equals the serial recurrence
 *              over the T real steps.  The chunked layout of the pages builds T
 *              as nchunks * chunk_len; the tail chunk is this library's
 *              widening, which lets a caller stream a sequence in pieces of
 *              any length through s0 / ds_final.
 *   mimo_rank  R (MIMO); must be 1 for the other variants.
 * Limits of this build: P <= 256, N <= 256, L * R <= 256 (Mamba-2, MIMO);
 * N <= 32, L <= 256 (Mamba-1).  Larger sizes return SSD_ERR_SHAPE.
 */
typedef struct {
  int32_t variant;
  int32_t io_dtype;
  int64_t batch;
  int64_t seqlen;
  int64_t nheads;
  int64_t headdim;
  int64_t dstate;
  int64_t ngroups;
  int64_t chunk;
  int64_t mimo_rank;
} ssd_problem;

/*
 * Bytes of device workspace that ssd_forward (backward == 0) or ssd_backward
 * (backward != 0) needs for `prob`.  Writes *bytes and returns SSD_OK, or
 * returns a validation error and leaves *bytes untouched.  Host-only; touches
 * no device.
 */
ssd_status ssd_workspace_size(const ssd_problem* prob, int backward, size_t* bytes);

/*
 * Forward scan: y and s_final from (x, dt_raw, A, B, C, s0).
 *
 * Layouts (row-major):
 *   Mamba-2: x, y [b,T,H,P]; dt_raw [b,T,H]; A [H]; B, C [b,T,G,N];
 *            s0, s_final [b,H,P,N].
 *   Mamba-1: x, y, dt_raw [b,T,D]; A [D,N]; B, C [b,T,N]; s0, s_final [b,D,N].
 *   MIMO:    the x slot carries v [b,T,R,H,P]; the dt_raw slot carries the
 *            pre-combined decay exponent da [b,T,H] (no softplus is applied);
 *            A must be NULL; B, C [b,T,R,H,N]; y [b,T,R,H,P];
 *            s0, s_final [b,H,P,N].
 * s0 may be NULL (a zero initial state).  Every other pointer is required
 * (except A for MIMO) and must be 16-byte aligned.
 * ws / ws_bytes: caller-owned device workspace of at least
 * ssd_workspace_size(prob, 0) bytes (always >= 256, never NULL).  Its first
 * 4 bytes are a device status word (int32): the call resets it to 0, and a
 * kernel whose bounded wait on an internal barrier gives up writes a nonzero
 * code there (the outputs are then invalid).  Read it after the stream
 * reaches the call if that check is wanted.
 */
ssd_status ssd_forward(const ssd_problem* prob, const void* x, const float* dt_raw, const float* A,
                       const void* B, const void* C, const float* s0, void* y, float* s_final, void* ws,
                       size_t ws_bytes, void* cuda_stream);

/*
 * Backward (VJP) of ssd_forward.  Inputs: the upstream gradients dy (layout
 * and dtype of y) and ds_final (fp32, layout of s_final; required, it is the
 * nonzero seed of the reverse recurrence), and the saved leaf inputs of the
 * forward (x, dt_raw, A, B, C, s0 exactly as passed to ssd_forward).  No
 * forward intermediate is needed: the backward recomputes the chunk states.
 *
 * Outputs (each takes its primal's layout and dtype):
 *   dx [like x], ddt_raw [like dt_raw, fp32], dA [like A, fp32],
 *   dB [like B], dC [like C], ds0 [like s0, fp32].
 * dB, dC (Mamba-2: over the heads of each group; Mamba-1: over all
 * channels) and dA (over batch and time) are full reductions written once.
 * MIMO: dx returns dv, ddt_raw returns d(da), and dA must be NULL.
 * s0 may be NULL (zero initial state); ds0 is still written.
 * ws / ws_bytes: at least ssd_workspace_size(prob, 1) bytes, with the same
 * device status word in its first 4 bytes as for ssd_forward.
 */
ssd_status ssd_backward(const ssd_problem* prob, const void* dy, const float* ds_final, const void* x,
                        const float* dt_raw, const float* A, const void* B, const void* C, const float* s0,
                        void* dx, float* ddt_raw, float* dA, void* dB, void* dC, float* ds0, void* ws,
                        size_t ws_bytes, void* cuda_stream);

/*
 * Stashed chunk states: a forward that keeps every chunk-input state S_c for
 * the backward, and a backward that reads them instead of replaying the
 * forward scan (the "Two things that are easy to get wrong" section, item 2,
 * of the "S1-31: SSM_SCAN_BACK" page: the backward needs the states the
 * forward overwrote; storing all of them is the reference, a cheaper scheme
 * must give the same bits).  The stash holds the same bf16 tiles the
 * recompute path writes to its workspace, produced by the same kernel from the
 * same inputs, so ssd_backward_stashed returns bit for bit what ssd_backward
 * returns for the same leaf inputs.  It saves the backward one pass of the
 * state scan (about an eighth of a forward + backward step at the Mamba-2
 * 2.7B layer shape) for b*H*ceil(T/L)*N*P*2 bytes of device memory held from the
 * forward to the backward.
 *
 * Available where the tensor-core path runs: Mamba-2, bf16 io, chunk 64,
 * headdim 64, dstate 128 (other problems return SSD_ERR_SHAPE).
 *
 * ssd_states_size: bytes of the stash for `prob` (bf16 [b, H, ceil(T/L)][N][P],
 *   row-major; tile (b, h, c) is the state entering chunk c, S_0 = s0 rounded
 *   to bf16).  Host-only.
 * ssd_forward_stash: ssd_forward, plus the stash written to `states`
 *   (caller-owned device buffer of at least ssd_states_size bytes, 16-byte
 *   aligned; a smaller states_bytes returns SSD_ERR_WORKSPACE).  y and s_final
 *   are bit for bit those of ssd_forward.  ws as for ssd_forward.
 * ssd_backward_stashed: ssd_backward without s0, reading `states` as written
 *   by ssd_forward_stash for the same x, dt_raw, A, B, s0 (the caller keeps
 *   the buffer unchanged in between; nothing checks it).  ws as for
 *   ssd_backward.
 * Errors and the device status word are those of ssd_forward / ssd_backward.
 */
ssd_status ssd_states_size(const ssd_problem* prob, size_t* bytes);
ssd_status ssd_forward_stash(const ssd_problem* prob, const void* x, const float* dt_raw, const float* A,
                             const void* B, const void* C, const float* s0, void* y, float* s_final, void* states,
                             size_t states_bytes, void* ws, size_t ws_bytes, void* cuda_stream);
ssd_status ssd_backward_stashed(const ssd_problem* prob, const void* dy, const float* ds_final, const void* x,
                                const float* dt_raw, const float* A, const void* B, const void* C,
                                const void* states, size_t states_bytes, void* dx, float* ddt_raw, float* dA,
                                void* dB, void* dC, float* ds0, void* ws, size_t ws_bytes, void* cuda_stream);

/*
 * Checkpoint every K chunks: a forward that keeps the fp32 chain state at
 * every K-th chunk boundary, and a backward that replays the chunk states from
 * those checkpoints in independent segments of K chunks instead of one
 * sequential scan over the whole sequence (the "Two things that are easy to
 * get wrong" section, item 2, of the "S1-31: SSM_SCAN_BACK" page: checkpoints
 * every K steps are the cheaper scheme, and must give the bits of storing every
 * state).  The checkpoints are the exact fp32 states of the forward's scan, and
 * each segment applies the same operations to them as the whole-sequence
 * replay, so ssd_backward_checkpointed returns bit for bit what ssd_backward
 * returns, for any K.  Memory held from the forward to the backward:
 * b*H*ceil(nc/K)*P*N*4 bytes (nc = ceil(T/L); 84 MB at K = 8 for the Mamba-2
 * 2.7B layer shape, against 336 MB for the stash of every state).
 *
 * Available where the tensor-core path runs: Mamba-2, bf16 io, chunk 64,
 * headdim 64, dstate 128 (other problems return SSD_ERR_SHAPE).  every = K,
 * 1 <= K <= 2^30 (SSD_ERR_INVALID_ARG otherwise); K >= nc keeps only s0.
 *
 * ssd_checkpoints_size: bytes of the checkpoints (fp32 [b, H, ceil(nc/K)][P][N],
 *   row-major; entry (b, h, k) is the state entering chunk k*K, entry 0 = s0,
 *   zeros for a NULL s0).  Host-only.
 * ssd_forward_checkpointed: ssd_forward, plus the checkpoints written to
 *   `ckpt` (caller-owned device buffer of at least ssd_checkpoints_size bytes,
 *   16-byte aligned; a smaller ckpt_bytes returns SSD_ERR_WORKSPACE).  y and
 *   s_final are bit for bit those of ssd_forward.  ws as for ssd_forward.
 * ssd_backward_checkpointed: ssd_backward without s0, reading the checkpoints
 *   written by ssd_forward_checkpointed with the same K for the same x,
 *   dt_raw, A, B, s0 (the caller keeps the buffer unchanged in between; nothing
 *   checks it).  ws as for ssd_backward.
 * Errors and the device status word are those of ssd_forward / ssd_backward.
 */
ssd_status ssd_checkpoints_size(const ssd_problem* prob, int64_t every, size_t* bytes);
ssd_status ssd_forward_checkpointed(const ssd_problem* prob, const void* x, const float* dt_raw, const float* A,
                                    const void* B, const void* C, const float* s0, void* y, float* s_final,
                                    int64_t every, float* ckpt, size_t ckpt_bytes, void* ws, size_t ws_bytes,
                                    void* cuda_stream);
ssd_status ssd_backward_checkpointed(const ssd_problem* prob, const void* dy, const float* ds_final, const void* x,
                                     const float* dt_raw, const float* A, const void* B, const void* C,
                                     int64_t every, const float* ckpt, size_t ckpt_bytes, void* dx, float* ddt_raw,
                                     float* dA, void* dB, void* dC, float* ds0, void* ws, size_t ws_bytes,
                                     void* cuda_stream);

/*
 * Forward scan without a caller workspace, for callers that cannot allocate
 * device memory.  (The pages describe no such call; it is an addition of this
 * library.)
 *
 * Who needs it: code that runs where device allocation is not available or
 * not allowed once it has started, for example an inference engine or plugin
 * whose host framework owns all GPU memory and hands out only the tensors, or
 * a latency-critical loop that has a rule of no allocation after start-up.
 * ssd_forward needs a workspace from ssd_workspace_size(); this call takes
 * none.  Its scratch is one fixed array of 32 MiB in device memory, declared
 * at file scope in the library, so every GPU that loads the library keeps
 * those 32 MiB until the process exits.
 *
 * Arguments, layouts, results and validation are those of ssd_forward,
 * without ws / ws_bytes.  A problem whose ssd_workspace_size(prob, 0) exceeds
 * 32 MiB is rejected with SSD_ERR_TOO_LARGE before anything runs.  The call
 * allocates nothing (no cudaMalloc, no allocating library routine).
 *
 * Start-up: the array belongs to this library's device module, which the
 * CUDA runtime loads on a device the first time the library needs it there
 * (lazy loading, the default).  Loading reserves the 32 MiB, so a caller that
 * forbids device allocation after start-up calls
 * ssd_forward_static_status(NULL, stream) once per device at start-up, with
 * that device current and before any stream capture: it loads the module and
 * looks up the array's address and does nothing else.  Later calls allocate
 * nothing.
 *
 * All calls share the one array, which keeps the last call's contents (its
 * first 4 bytes are the device status word, reset to 0 by every call):
 * calls that may overlap on the GPU, on any streams, race on it and must be
 * serialized by the caller.
 *
 * ssd_forward_static_status(code, stream): with code == NULL, the start-up
 * step above only.  Otherwise it also copies the status word into *code (a
 * caller-owned host int32) on `stream`, after the work already enqueued
 * there, and waits for that stream.  Returns SSD_OK when the word is 0,
 * SSD_ERR_TIMEOUT when a bounded wait of the last call gave up (its outputs
 * are then invalid; *code holds the code), SSD_ERR_CUDA if a CUDA call fails.
 */
ssd_status ssd_forward_static(const ssd_problem* prob, const void* x, const float* dt_raw, const float* A,
                              const void* B, const void* C, const float* s0, void* y, float* s_final,
                              void* cuda_stream);
ssd_status ssd_forward_static_status(int32_t* code, void* cuda_stream);

/*
 * The device status word of a workspace, and a test of the bounded waits.
 *
 * Every wait of a kernel of this library on one of its barriers is bounded
 * (two seconds).  One that runs out writes a nonzero code into the status
 * word (the first 4 bytes of the call's workspace), stops issuing work and
 * returns; the host learns of it only from the word, since the call itself
 * returned before the GPU ran it.  (The pages ask for none of this; it is the
 * failure detection of this library.)
 *
 * ssd_read_status(ws, code, stream): copies the status word at the start of
 * the device workspace `ws` into *code (host int32) on `stream`, after the
 * work already enqueued there, and waits for that stream.  Returns SSD_OK for
 * 0, SSD_ERR_TIMEOUT for a nonzero word, SSD_ERR_INVALID_ARG for NULL
 * arguments, SSD_ERR_CUDA if a CUDA call fails.  Allocates nothing.
 *
 * ssd_wait_selftest(ws, limit_us, stream): resets the status word of `ws`
 * (device, 16-byte aligned, at least 4 bytes) and launches one warp in which
 * one thread waits on a barrier that nothing ever completes, with a limit of
 * limit_us microseconds (1 .. 2 000 000) instead of two seconds.  The wait
 * runs out, writes code 1 into the word and the kernel returns: a following
 * ssd_read_status returns SSD_ERR_TIMEOUT with *code == 1, and the stream and
 * context stay usable.  Returns SSD_ERR_INVALID_ARG for a NULL ws or a limit
 * outside the range, SSD_ERR_ALIGNMENT, or SSD_ERR_CUDA if the launch fails.
 */
ssd_status ssd_read_status(const void* ws, int32_t* code, void* cuda_stream);
ssd_status ssd_wait_selftest(void* ws, uint32_t limit_us, void* cuda_stream);

/*
 * KDA: the gated delta-rule recurrence of the notes page "sec-10.tex"
 * (section "反向传播推导"), a second workload beside the selective scan, and
 * its BPTT backward (the page's reverse-time steps 1-6).  fp32 io and
 * arithmetic.  Per batch element and value head, with state S [K, V]:
 *     S_dec = exp(g_t) (.) S_{t-1}     (one log-decay per key row)
 *     r_t   = v_t - k_t^T S_dec
 *     S_t   = S_dec + beta_t k_t (x) r_t
 *     o_t   = (scale q_t)^T S_t
 * Value head hv reads query / key head hv / G, G = value_heads / nheads (the
 * page's grouped value heads); dq, dk of a query / key head are the sums over
 * its G value heads.
 *
 * Layouts (row-major, fp32, 16-byte aligned): q, k, dq, dk [b,T,H,K];
 * v, o, do, dv [b,T,HV,V]; g, dg [b,T,HV,K]; beta, dbeta [b,T,HV];
 * s0, s_final, ds_final, ds0 [b,HV,K,V].  s0 may be NULL (zeros).
 * Limits of this build: key_dim <= 128, value_dim <= 128 (SSD_ERR_SHAPE);
 * value_heads a multiple of nheads (SSD_ERR_SHAPE).
 *
 * ssd_kda_workspace_size: device workspace of the forward (backward == 0) or
 *   backward; host-only.  The backward's holds fp32 checkpoints of the state
 *   every 8 steps (b*HV*ceil(T/8)*K*V*4 bytes), the per-step row sums of its
 *   CTAs and the per-value-head dq, dk.  Its first 4 bytes are the device
 *   status word, as for ssd_forward.
 * ssd_kda_forward: o and s_final.
 * ssd_kda_backward: dq, dk, dv, dg, dbeta and ds0 of <do, o> + <ds_final,
 *   s_final> (ds_final required); recomputes the states from the leaf inputs
 *   (no forward intermediate is needed).  Deterministic: every sum has a
 *   fixed order.
 * Errors as for ssd_forward; every error is returned before anything is
 * enqueued.
 */
typedef struct {
  int64_t batch;
  int64_t seqlen;
  int64_t nheads;      /* H: query / key heads */
  int64_t value_heads; /* HV: a multiple of H */
  int64_t key_dim;     /* K */
  int64_t value_dim;   /* V */
} ssd_kda_problem;

ssd_status ssd_kda_workspace_size(const ssd_kda_problem* prob, int backward, size_t* bytes);
ssd_status ssd_kda_forward(const ssd_kda_problem* prob, const float* q, const float* k, const float* v,
                           const float* g, const float* beta, const float* s0, float scale, float* o, float* s_final,
                           void* ws, size_t ws_bytes, void* cuda_stream);
ssd_status ssd_kda_backward(const ssd_kda_problem* prob, const float* dout, const float* ds_final, const float* q,
                            const float* k, const float* v, const float* g, const float* beta, const float* s0,
                            float scale, float* dq, float* dk, float* dv, float* dg, float* dbeta, float* ds0,
                            void* ws, size_t ws_bytes, void* cuda_stream);

/*
 * The gated delta rule with one log-decay per head, by chunks on the tensor
 * cores and step by step on a cache of states.  Per sequence and value head,
 * with state S [K, V]:
 *     S_dec = exp(g_t) S_{t-1}
 *     r_t   = beta_t (v_t - S_dec^T k_t)
 *     S_t   = S_dec + k_t (x) r_t
 *     o_t   = scale S_t^T q_t
 * (the KDA recurrence above with the same decay for every key row, on bf16
 * tensors).  Value head hv reads query / key head hv / G, G = value_heads /
 * nheads; dq, dk of a query / key head are the sums over its G value heads.
 *
 * ssd_delta_problem:
 *   io_dtype    of q, k, v, o and their gradients: SSD_BF16; ssd_delta_step
 *               also takes SSD_F32 (the others return SSD_ERR_DTYPE).
 *   gate_dtype  of g, beta, dg, dbeta: SSD_F32 or SSD_BF16.  (g <= 0 in
 *               earnest; -inf forgets the state.)
 *   packed      0: batch sequences of seqlen steps each, q [b,T,H,K] and so
 *               on.  1: batch sequences of lengths of their own, one after
 *               another on one axis of seqlen steps in all, q [T,H,K] and so
 *               on; the call's cu_seqlens (device, int32 [batch + 1], 4-byte
 *               aligned) holds 0, the ends of the first sequences, seqlen.
 *               Empty sequences are allowed.  The kernels clamp its values to
 *               0 .. seqlen and to ascending order.  Steps that belong to no
 *               sequence (before the first value, past the last one of an axis
 *               that is padded) take no part; o and the gradients are zero
 *               there.  ssd_delta_step takes packed = 0.
 *   batch, seqlen, nheads (H), value_heads (HV, a multiple of H), key_dim (K),
 *   value_dim (V): >= 1.  Limits of this build: K, V <= 128, HV <= 65535, steps
 *               and b*HV below 2^31 (SSD_ERR_SHAPE).
 *   q_stride, k_stride, v_stride: elements from a step to the next, for
 *               tensors that lie inside wider ones; 0 = dense (H*K, H*K,
 *               HV*V).  Batches follow one another at T strides.  Everything
 *               else is dense.
 * Layouts (row-major): q, k, dq, dk [b,T,H,K]; v, o, do, dv [b,T,HV,V];
 * g, beta, dg, dbeta [b,T,HV]; s0, s_final, ds_final, ds0 [b,HV,K,V] fp32.
 * q, k, v need the alignment of their type (rows of whole 16-byte pieces that
 * start on 16 bytes are read faster); every other pointer of the chunked calls
 * is 16-byte aligned.
 *
 * Precision.  The state is held and summed in fp32 over any length, and what
 * the chunk products read of it enters the tensor cores as two bf16 numbers,
 * which keep 16 bits: s_final and ds0 are good to about 1e-5 of the terms that
 * they are sums of (some 4e-6 of their own size as a rule, where fp32 products
 * would give 3e-7; 7e-5 was seen of ds0 at one key a head, whose terms cancel),
 * and o and dv are rounded once to bf16.  The other gradients are sums of
 * products of bf16-rounded tiles: their relative error is about 2^-8 whatever
 * type they are stored in, also for fp32 gates.  A NaN or
 * infinity in q, k, v, g or beta may reach every step of its chunk of 64 steps
 * and every later one of its sequence; other sequences and steps past a sequence's end take
 * nothing from it.
 *
 * ssd_delta_workspace_size: device workspace of ssd_delta_forward (backward ==
 *   0) or ssd_delta_backward; stashed != 0: of the call with a stash, which
 *   needs less.  Host-only.  Its first 4 bytes are the device status word, as
 *   for ssd_forward.
 * ssd_delta_stash_size: bytes of the stash that a training forward may keep
 *   for its backward: per chunk and value head the bf16 state that enters it
 *   (V16*KP*2 bytes, V16 = V rounded up to 16, KP = K rounded up to 64 or
 *   128), the written rows r (64*V16*2) and the chunk's triangular inverse,
 *   scores and decays (33.25 KiB).  Host-only.
 * ssd_delta_forward: o, and s_final unless it is NULL, from s0 (NULL: zeros).
 *   stash NULL, or a device buffer (16-byte aligned) that is filled.
 * ssd_delta_backward: dq, dk, dv, dg, dbeta and (unless NULL) ds0 of <do, o> +
 *   <ds_final, s_final> (ds_final NULL: zeros) from the leaf inputs, exactly as
 *   passed to the forward.  With the stash that a forward of the same problem
 *   and inputs filled it reads the chunk states instead of making them again;
 *   the results are the same bit for bit.
 * ssd_delta_step: seqlen >= 1 steps of each of batch sequences on `state`
 *   [num_slots,HV,K,V] (fp32, 16-byte aligned), updated in place.  Sequence n
 *   uses slot slots[n] (device, int32 [batch]; NULL: slot n, num_slots >=
 *   batch).  A slot number outside 0 .. num_slots - 1 marks a place without a
 *   sequence: its o is zero and no state is touched.  Two sequences of a call
 *   must not share a slot.  fp32 arithmetic, no workspace.  Other pointers
 *   need the alignment of their type.
 * Errors as for ssd_forward; every error is returned before anything is
 * enqueued.  Results are bitwise reproducible.
 */
typedef struct {
  int32_t io_dtype;
  int32_t gate_dtype;
  int32_t packed;
  int32_t reserved; /* 0 */
  int64_t batch;
  int64_t seqlen;
  int64_t nheads;
  int64_t value_heads;
  int64_t key_dim;
  int64_t value_dim;
  int64_t q_stride;
  int64_t k_stride;
  int64_t v_stride;
} ssd_delta_problem;

ssd_status ssd_delta_workspace_size(const ssd_delta_problem* prob, int backward, int stashed, size_t* bytes);
ssd_status ssd_delta_stash_size(const ssd_delta_problem* prob, size_t* bytes);
ssd_status ssd_delta_forward(const ssd_delta_problem* prob, const void* q, const void* k, const void* v, const void* g,
                             const void* beta, const float* s0, const int32_t* cu_seqlens, float scale, void* o,
                             float* s_final, void* stash, size_t stash_bytes, void* ws, size_t ws_bytes,
                             void* cuda_stream);
ssd_status ssd_delta_backward(const ssd_delta_problem* prob, const void* dout, const float* ds_final, const void* q,
                              const void* k, const void* v, const void* g, const void* beta, const float* s0,
                              const int32_t* cu_seqlens, float scale, void* dq, void* dk, void* dv, void* dg,
                              void* dbeta, float* ds0, const void* stash, size_t stash_bytes, void* ws,
                              size_t ws_bytes, void* cuda_stream);
ssd_status ssd_delta_step(const ssd_delta_problem* prob, const void* q, const void* k, const void* v, const void* g,
                          const void* beta, float* state, const int32_t* slots, int64_t num_slots, float scale, void* o,
                          void* cuda_stream);

/*
 * Layer norm over the last dimension and its backward: the norm in front of a
 * mixer (rows of the model's width) and of its heads' outputs (rows of a head).
 *     mean = sum x / D, var = sum (x - mean)^2 / D, rstd = (var + eps)^-1/2,
 *     y = (x - mean) rstd * weight + bias
 *
 * ssd_norm_problem: io_dtype of x, y, dy, dx and weight_dtype of weight, bias,
 * dw, db (SSD_F32 or SSD_BF16 each; sums are fp32); rows >= 1 (< 2^31), dim
 * 1 .. 16384 (SSD_ERR_SHAPE), x_stride: elements from a row of x to the next
 * (0 = dense).  y, dy, dx are dense [rows, dim]; mean, rstd fp32 [rows].  x,
 * mean and rstd need the alignment of their type, every other pointer 16
 * bytes.
 *
 * ssd_norm_forward: y, and mean and rstd unless NULL.  weight NULL: ones, bias
 *   NULL: zeros; eps >= 0.
 * ssd_norm_backward: dx, and dw and db (summed over the rows in a fixed order)
 *   unless NULL, from the forward's x, mean, rstd and weight.  ws (at least
 *   ssd_norm_workspace_size bytes) may be NULL where dw and db are.
 * Errors as for ssd_forward.  Results are bitwise reproducible.
 */
typedef struct {
  int32_t io_dtype;
  int32_t weight_dtype;
  int64_t rows;
  int64_t dim;
  int64_t x_stride;
} ssd_norm_problem;

ssd_status ssd_norm_workspace_size(const ssd_norm_problem* prob, size_t* bytes);
ssd_status ssd_norm_forward(const ssd_norm_problem* prob, const void* x, const void* weight, const void* bias, float eps,
                            void* y, float* mean, float* rstd, void* cuda_stream);
ssd_status ssd_norm_backward(const ssd_norm_problem* prob, const void* dy, const void* x, const float* mean,
                             const float* rstd, const void* weight, void* dx, void* dw, void* db, void* ws,
                             size_t ws_bytes, void* cuda_stream);

/*
 * The gated linear recurrence with one decay per channel: whole sequences with
 * gradients, packed prompts, and single steps on a cache of states.  Per
 * sequence and channel, with s the sigmoid:
 *     g_t = -scale softplus(lam) s(r_t),   a_t = exp(g_t)
 *     h_t = a_t h_{t-1} + sqrt(1 - a_t^2) s(i_t) x_t,   y_t = h_t
 *
 * ssd_glr_problem:
 *   io_dtype    of x, r, i, y and their gradients: SSD_F32 or SSD_BF16.  lam,
 *               states and their gradients are fp32, as all arithmetic.
 *   packed      0: batch sequences of seqlen steps each, x [b,T,D].  1: batch
 *               sequences one after another on one axis of seqlen steps, x
 *               [T,D], with cu_seqlens as for the delta rule above (ascending;
 *               values are clamped to 0 .. seqlen; empty sequences are allowed:
 *               their h_final is their h0).  y and the gradients are zero at
 *               steps of no sequence.  ssd_glr_step takes packed = 0.
 *   batch, seqlen, dim (D): >= 1.  Limits of this build (SSD_ERR_SHAPE): T up
 *               to 2^31 - 65536 and below 2^31 steps in all, D and strides up to
 *               2^24, batch below 2^29, and up to 65535 where not packed.
 *   x_stride, r_stride, i_stride: elements from a step to the next, for
 *               tensors that lie inside wider ones; 0 = dense.  Batches follow
 *               one another at T strides.  Everything else is dense.
 * Layouts: x, r, i, y, dy, dx, dr, di [b,T,D]; lam, dlam [D]; h0, h_final,
 * dh_final, dh0 [b,D] fp32.  x, r, i, dy and fp32 arrays need the alignment of
 * their type (rows of whole 16-byte pieces that start on 16 bytes are read
 * faster), y, dx, dr, di, the stash and the workspace 16 bytes.  Outputs must
 * not overlap inputs.
 *
 * A NaN or infinity reaches the later steps of its channel and sequence only
 * (the earlier ones' gradients); other sequences take nothing from it.
 * ssd_glr_forward takes a gate s(i) below 2^-64 as 0 (i below about -44), and
 * ssd_glr_backward gates below 1e-30 as 1e-30 (below about -69).
 *
 * ssd_glr_stash_size: bytes of the stash a training forward may keep for its
 *   backward: the fp32 state that enters every eighth step (bf16), or every
 *   fourth (fp32).  Host-only.
 * ssd_glr_workspace_size: device workspace of ssd_glr_backward (the forward
 *   needs none); stashed != 0: of the call with a stash.  Host-only.
 * ssd_glr_forward: y, and h_final unless NULL, from h0 (NULL: zeros); the stash
 *   is filled unless NULL.  scale >= 0.
 * ssd_glr_backward: dx, dr, di, dlam and (unless NULL) dh0 of <dy, y> +
 *   <dh_final, h_final> (dh_final NULL: zeros) from the leaf inputs, as passed
 *   to the forward.  Without the stash of a forward of the same problem and
 *   inputs the states are made again; the results are the same bit for bit.
 * ssd_glr_step: seqlen >= 1 steps of each of batch sequences on `state`
 *   [num_slots,D] (fp32), updated in place; slots as for ssd_delta_step.
 * Errors as for ssd_forward; every error is returned before anything is
 * enqueued.  Results are bitwise reproducible.
 */
typedef struct {
  int32_t io_dtype;
  int32_t packed;
  int64_t batch;
  int64_t seqlen;
  int64_t dim;
  int64_t x_stride;
  int64_t r_stride;
  int64_t i_stride;
} ssd_glr_problem;

ssd_status ssd_glr_stash_size(const ssd_glr_problem* prob, size_t* bytes);
ssd_status ssd_glr_workspace_size(const ssd_glr_problem* prob, int stashed, size_t* bytes);
ssd_status ssd_glr_forward(const ssd_glr_problem* prob, const void* x, const void* r, const void* i, const float* lam,
                           const float* h0, const int32_t* cu_seqlens, float scale, void* y, float* h_final, void* stash,
                           size_t stash_bytes, void* cuda_stream);
ssd_status ssd_glr_backward(const ssd_glr_problem* prob, const void* dy, const float* dh_final, const void* x, const void* r,
                            const void* i, const float* lam, const float* h0, const int32_t* cu_seqlens, float scale,
                            void* dx, void* dr, void* di, float* dlam, float* dh0, const void* stash, size_t stash_bytes,
                            void* ws, size_t ws_bytes, void* cuda_stream);
ssd_status ssd_glr_step(const ssd_glr_problem* prob, const void* x, const void* r, const void* i, const float* lam,
                        float* state, const int32_t* slots, int64_t num_slots, float scale, void* y, void* cuda_stream);

/*
 * The causal short convolution of each channel (depthwise) with bias and
 * activation: whole sequences with gradients, packed prompts, and single steps
 * on a cache of inputs.  Per sequence and channel
 *     z_t = bias + sum over j < K of weight[K-1-j] x_{t-j},   y = z s(z) or z
 * where x before the first step is the sequence's taps: the last K - 1 inputs
 * of what came before it, oldest first (NULL: zeros).
 *
 * ssd_conv_problem:
 *   io_dtype     of x, y, the taps and their gradients; weight_dtype of weight,
 *                bias, dw, db (SSD_F32 or SSD_BF16 each; arithmetic is fp32).
 *   packed       0: x [b,T,D]; 1: x [T,D] and cu_seqlens, as for ssd_glr_forward.
 *                ssd_conv_step takes packed = 0.
 *   activation   SSD_ACT_NONE or SSD_ACT_SILU.
 *   batch, seqlen, dim (D), taps (K): >= 1.  Limits of this build
 *                (SSD_ERR_SHAPE): K 2 .. 4, D up to 2^20, steps below 2^31 -
 *                4095, batch below 2^29, and up to 65535 where not packed.
 *   x_stride     elements from a step of x to the next (0: dense); batches
 *                follow one another at T strides.  Everything else is dense.
 * Layouts: x, y, dy, dx [b,T,D]; weight, dw [D,K]; bias, db [D]; taps,
 * taps_final, dtaps [b,K-1,D].  Pointers need the alignment of their type, the
 * workspace 16 bytes; where D and the stride are multiples of four and every
 * pointer starts on four elements four channels are taken at a time.  Outputs
 * must not overlap inputs.
 *
 * ssd_conv_workspace_size: device workspace of ssd_conv_backward (the others
 *   need none).  Host-only.
 * ssd_conv_forward: y, and taps_final unless NULL (where a sequence has fewer
 *   than K - 1 steps, what is left of its taps comes first).  bias NULL: zeros.
 * ssd_conv_backward: dx, and dw, db (summed in a fixed order) and dtaps unless
 *   NULL, of <dy, y>.  taps_final hands on inputs: its gradient is the caller's.
 * ssd_conv_step: seqlen >= 1 steps of each of batch sequences on `state`
 *   [num_slots,K-1,D] (io_dtype), updated in place; slots as for
 *   ssd_delta_step.
 * Errors as for ssd_forward; every error is returned before anything is
 * enqueued.  Results are bitwise reproducible.
 */
typedef enum { SSD_ACT_NONE = 0, SSD_ACT_SILU = 1, SSD_ACT_GELU = 2 } ssd_activation;

typedef struct {
  int32_t io_dtype;
  int32_t weight_dtype;
  int32_t packed;
  int32_t activation;
  int64_t batch;
  int64_t seqlen;
  int64_t dim;
  int64_t taps;
  int64_t x_stride;
} ssd_conv_problem;

ssd_status ssd_conv_workspace_size(const ssd_conv_problem* prob, size_t* bytes);
ssd_status ssd_conv_forward(const ssd_conv_problem* prob, const void* x, const void* weight, const void* bias, const void* taps,
                            const int32_t* cu_seqlens, void* y, void* taps_final, void* cuda_stream);
ssd_status ssd_conv_backward(const ssd_conv_problem* prob, const void* dy, const void* x, const void* weight, const void* bias,
                             const void* taps, const int32_t* cu_seqlens, void* dx, void* dw, void* db, void* dtaps, void* ws,
                             size_t ws_bytes, void* cuda_stream);
ssd_status ssd_conv_step(const ssd_conv_problem* prob, const void* x, const void* weight, const void* bias, void* state,
                         const int32_t* slots, int64_t num_slots, void* y, void* cuda_stream);

/*
 * The gated feed-forward: both projections, the activation and the product in
 * one pass, and its gradients.
 *     G = x Wg^T,   U = x Wu^T,   h = act(G) U
 * with act SiLU (G s(G)) or GELU in its tanh form.
 *
 * ssd_ffn_problem:
 *   io_dtype    of every tensor: SSD_BF16 (SSD_F32 returns SSD_ERR_DTYPE).
 *               Products are summed in fp32.
 *   activation  SSD_ACT_SILU or SSD_ACT_GELU.
 *   rows (M), dim (D), hidden (F): >= 1.  Limits of this build (SSD_ERR_SHAPE):
 *               D and F multiples of 8 up to 2^20, M up to 2^24.
 *   x_stride    elements from a row of x to the next, a multiple of 8 (0:
 *               dense).  Everything else is dense.
 * Layouts: x, dx [M,D]; w_gate, w_up, dw_gate, dw_up [F,D]; h, dh [M,F].
 * Every pointer is 16-byte aligned.  Outputs must not overlap inputs.
 *
 * Precision.  h is rounded once.  The stash holds each number of G and U
 * rounded to 24 bits (2^-16 of it at most), and the backward's products read dG
 * and dU rounded to bf16: 2^-8 of each term at most, so the gradients are good
 * to that of their terms' size and rounded once more.  A NaN or infinity reaches
 * its own row of h and dx, and every element of the weights' gradients that sums
 * over that row.
 *
 * ssd_ffn_stash_size: bytes of the stash that a training forward may keep for
 *   its backward (6 F bytes for each of M rows, M rounded up to 128).
 *   Host-only.
 * ssd_ffn_workspace_size: device workspace of ssd_ffn_forward (backward == 0) or
 *   ssd_ffn_backward; stashed != 0: of the call with a stash, which needs less.
 *   Host-only.  Its first 4 bytes are the device status word, as for
 *   ssd_forward.
 * ssd_ffn_forward: h; the stash is filled unless NULL.
 * ssd_ffn_backward: dx, dw_gate and dw_up of <dh, h> from the leaf inputs, as
 *   passed to the forward.  Without the stash of a forward of the same problem
 *   and inputs G and U are made again; the results are the same bit for bit.
 * Errors as for ssd_forward; every error is returned before anything is
 * enqueued.  Results are bitwise reproducible.
 */
typedef struct {
  int32_t io_dtype;
  int32_t activation;
  int64_t rows;
  int64_t dim;
  int64_t hidden;
  int64_t x_stride;
} ssd_ffn_problem;

ssd_status ssd_ffn_stash_size(const ssd_ffn_problem* prob, size_t* bytes);
ssd_status ssd_ffn_workspace_size(const ssd_ffn_problem* prob, int backward, int stashed, size_t* bytes);
ssd_status ssd_ffn_forward(const ssd_ffn_problem* prob, const void* x, const void* w_gate, const void* w_up, void* h,
                           void* stash, size_t stash_bytes, void* ws, size_t ws_bytes, void* cuda_stream);
ssd_status ssd_ffn_backward(const ssd_ffn_problem* prob, const void* dh, const void* x, const void* w_gate, const void* w_up,
                            void* dx, void* dw_gate, void* dw_up, const void* stash, size_t stash_bytes, void* ws,
                            size_t ws_bytes, void* cuda_stream);

/*
 * Per-launch timing, for diagnostics and roofline measurement.
 *
 * ssd_profile_start(capacity): every later ssd_forward / ssd_backward call
 * (from any host thread) records a pair of CUDA events around each kernel it
 * enqueues, on that call's stream, for up to `capacity` launches.  Returns
 * SSD_ERR_INVALID_ARG if capacity < 1.  Events are created with
 * cudaEventCreate on the current device; no device memory is allocated.
 *
 * ssd_profile_stop(out, capacity, count): waits for the recorded events,
 * writes one {kernel name, milliseconds} record per launch in launch order
 * (at most `capacity`), sets *count to the number written, destroys the
 * events and turns recording off.  The names are static strings.  Returns
 * SSD_ERR_CUDA if an event query fails.
 */
typedef struct {
  const char* kernel;
  float ms;
} ssd_kernel_time;

ssd_status ssd_profile_start(int capacity);
ssd_status ssd_profile_stop(ssd_kernel_time* out, int capacity, int* count);

/* Static, human-readable name of a status code (never NULL). */
const char* ssd_status_string(ssd_status status);

/* Version of this library as MAJOR*10000 + MINOR*100 + PATCH. */
int ssd_version(void);

#ifdef __cplusplus
}
#endif

#endif /* SSD_GB300_H */

/*
 * gdn.h -- C ABI of the GB300 (sm_103a) chunked Gated DeltaNet prefill library.
 *
 * The operation.  The pages name a "chunked Gated DeltaNet prefill" as one of the
 * fused operations of their native Qwen3.5 prefill workers and test it against
 * float64 references ("Cua-S1 4B 0.2 native text worker", kernel-test paragraph;
 * "Open-Jev-27B-v1.1 native text worker", section "Validation and optimization
 * scope").  They print no equations; the library computes the gated delta rule
 * per (sequence, value head):
 *
 *     S_t = alpha_t S_{t-1} (I - beta_t k_t k_t^T) + beta_t v_t k_t^T,   alpha_t = exp(g_t)
 *     o_t = S_t q_t / sqrt(dk)
 *
 * with S a dv x dk fp32 state (S_0 = init_state, or zeros) and the last S
 * returned as the final state.  q and k are expected to be L2-normalised per
 * token by the caller (the pages do this in a separate fused norm operation).
 * Internally the tokens of each sequence are processed in chunks of 64 with
 * the WY / UT-transform form of the recurrence.
 *
 * Versioning.  Like the pages' library ("ABI 4", later "CUDA ABI is 5"), the
 * ABI carries a version number; callers built against another version must be
 * rebuilt together with the library.
 */
#ifndef GDN_H
#define GDN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define GDN_ABI_VERSION 5

/* Status codes (0 = success, negative = error). */
#define GDN_OK 0
#define GDN_ERR_ARG (-1)    /* null required pointer, bad size, Hv % Hk != 0, unsupported dk/dv */
#define GDN_ERR_ALIGN (-2)  /* a pointer is not 16-byte aligned */
#define GDN_ERR_ALLOC (-3)  /* the library's device workspace could not be grown */
#define GDN_ERR_LAUNCH (-4) /* a CUDA call or kernel launch failed (see gdn_last_cuda_error) */
#define GDN_ERR_SCRATCH (-5) /* the problem needs more scratch than the fixed or caller-given workspace */

/* Flags of gdn_prefill_ex. */
#define GDN_FLAG_L2NORM_QK 1u /* normalise q and k per token inside the kernels: x / max(||x||, 1e-6) */
#define GDN_FLAG_TWO_LEVEL 2u /* use the two-level chunk scan (dense batches only) */
#define GDN_FLAG_ONE_LEVEL 4u /* never use the two-level chunk scan */
/* Segments per sequence for GDN_FLAG_TWO_LEVEL (2..255; 0 or absent = chosen by the library). */
#define GDN_FLAG_SEGMENTS(n) ((((unsigned)(n)) & 0xffu) << 8)
#define GDN_FLAG_SLICE32 0x10000u /* state carry: 32 state rows per CTA */
#define GDN_FLAG_SLICE16 0x40000u /* state carry: 16 state rows per CTA */
#define GDN_FLAG_SLICE64 0x20000u /* state carry: 64 state rows per CTA (dv a multiple of 64) */
#define GDN_FLAG_WIDE_RANGE 0x80000u /* state carry on bf16 hi + lo operand pairs (fp32 range; slower) */

/* Size of the fixed device scratch array behind gdn_prefill_static (64 MiB per device). */
#define GDN_STATIC_SCRATCH_BYTES (128u << 20)

/* Returns GDN_ABI_VERSION of the loaded library. */
int gdn_abi_version(void);

/* Human-readable text for a status code (static storage, never NULL). */
const char *gdn_strerror(int status);

/* The cudaError_t of the most recent GDN_ERR_LAUNCH / GDN_ERR_ALLOC on this thread (0 if none). */
int gdn_last_cuda_error(void);

/*
 * gdn_prefill -- chunked Gated DeltaNet prefill on the GPU, asynchronous on `stream`.
 *
 * Pointers (all DEVICE memory, owned by the caller, not retained after return,
 * each 16-byte aligned):
 *   q, k        bf16 [Ttot, Hk, dk]   queries and keys (L2-normalised per token)
 *   v           bf16 [Ttot, Hv, dv]   values
 *   g           fp32 [Ttot, Hv]       log decay, g <= 0 (alpha = exp(g))
 *   beta        fp32 [Ttot, Hv]       write strength in (0, 1)
 *   cu_seqlens  int32 [B + 1] or NULL packed sequence boundaries (see below)
 *   init_state  fp32 [B, Hv, dv, dk] or NULL (NULL = zero initial states)
 *   out         bf16 [Ttot, Hv, dv]   outputs o_t (written; must not alias any input)
 *   final_state fp32 [B, Hv, dv, dk] or NULL (NULL = not written); may alias init_state
 *
 * Sizes.  With cu_seqlens == NULL there are B sequences of T tokens each and
 * Ttot = B * T.  Otherwise B is the number of packed sequences, sequence b covers
 * tokens [cu_seqlens[b], cu_seqlens[b + 1]), cu_seqlens[0] = 0, cu_seqlens[B] =
 * T = Ttot, entries non-decreasing; zero-length sequences are allowed and return
 * their initial state.  The contents of cu_seqlens are not checked on the host
 * (that would need a synchronisation); out-of-range entries are clamped to
 * [0, T] on the device so no access leaves the buffers, and a malformed array sets
 * GDN_STATUS_BAD_CU_SEQLENS (see gdn_device_status).  Value head h reads key head
 * h / (Hv / Hk).  dk and dv must each be 32, 64 or 128.
 *
 * Precision and range.  The chunk products run on the tensor cores with fp32
 * accumulation and fp16 operands: k and q (converted from bf16, exact for
 * magnitudes 2^-17 .. 65504), the chunk's UT transform and score product, and the
 * state-side operands rounded from the fp32 state (2^-11 relative).  The state
 * itself is carried in fp32.  Operands beyond fp16's range (about 65504: values of
 * that size, or a state that grows to it) make the state non-finite, which sets
 * GDN_STATUS_NONFINITE_STATE.  Below it, fp16 keeps full precision only down to 2^-14:
 * with values of order 1e-5 and less the operands lose accuracy, and a single-level
 * call whose final state for some (sequence, head, row block) is nonzero but below
 * 2^-12 sets GDN_STATUS_SMALL_STATE.  gdn_prefill_ex with GDN_FLAG_WIDE_RANGE carries
 * the state-side operands as bf16 hi + lo pairs instead (fp32 range, 2^-16, slower).
 *
 * Memory.  The library keeps a per-device, grow-only workspace (allocated on the
 * first call that needs more; about 16 KB per 64-token chunk and value head, plus
 * 32 KB per chunk and key head for dk = 128, 16 KB for dk <= 64).
 * After a call at the largest size, later calls allocate nothing.  gdn_prefill,
 * gdn_prefill_ex and gdn_prefill_host calls on one device share that workspace
 * (and gdn_prefill_host's staging area): calls whose GPU work could overlap
 * (different streams, or host threads without ordering) must be ordered by the
 * caller, or use gdn_prefill_ws with a workspace each.
 *
 * Long prompts with few heads.  The chunks of a sequence are processed in order,
 * so a dense batch (cu_seqlens == NULL) whose B * Hv * dv / 32 state-carry blocks
 * leave most SMs idle is cut into P segments on 64-token boundaries and run as a
 * two-level scan instead: every segment's state transition and zero-start end
 * state at once, a short fp32 combine of the segment start states, then every
 * segment again from its true start state.  This applies when at least three
 * segments of four or more chunks fit one wave of B * P * Hv * (dv + dk) / 32
 * blocks (for example one 16,384-token prompt with 4 value heads of 128).  It
 * uses a second library-owned buffer (two bf16 [Ttot, Hv, dk] tensors and a few
 * fp32 state sets, also grow-only) and a library-owned second stream joined back
 * into `stream` by events.  Its results agree with the single-level path to the
 * stated tolerances, not bit for bit.  gdn_prefill_ex can force or forbid it.
 *
 * Returns GDN_OK, or an error code before anything is launched (argument and
 * alignment errors), or GDN_ERR_LAUNCH / GDN_ERR_ALLOC.  B == 0 returns GDN_OK
 * and does nothing.  The call does not synchronise the stream.
 */
int gdn_prefill(const void *q, const void *k, const void *v,
                const float *g, const float *beta,
                const int32_t *cu_seqlens, const float *init_state,
                void *out, float *final_state,
                int B, int T, int Hk, int Hv, int dk, int dv,
                void *stream /* cudaStream_t; NULL = legacy default stream */);

/*
 * gdn_prefill_host -- the same operation on HOST buffers (same layouts; any
 * alignment).  Copies the inputs to the library's device staging area, runs
 * gdn_prefill on `stream`, copies out and final_state back and synchronises
 * `stream` before returning.  Page-locked host buffers give the fastest copies.
 * cu_seqlens, init_state and final_state may be NULL as above.  For problems of
 * 8 MB or more (q, k and v together) the copies overlap the kernels, on
 * library-owned streams that are joined back into `stream`:
 *   - equal-length batches: 2 to 8 windows of whole 64-token chunks (about 16
 *     chunks each, the last one half as many).  The copies of one window overlap the kernels of the previous
 *     one and the copy-back of earlier ones; each window's state carry starts from
 *     the state the previous window left (kept on the device in fp32);
 *   - packed batches: up to four groups of whole key heads, whose state carries
 *     run side by side.
 * Either way the results are bit for bit those of gdn_prefill.
 */
int gdn_prefill_host(const void *q, const void *k, const void *v,
                     const float *g, const float *beta,
                     const int32_t *cu_seqlens, const float *init_state,
                     void *out, float *final_state,
                     int B, int T, int Hk, int Hv, int dk, int dv,
                     void *stream);

/*
 * gdn_prefill_ex -- gdn_prefill with option flags.
 *
 * GDN_FLAG_L2NORM_QK: q and k are taken as they come out of the projections and
 * L2-normalised per token inside the kernels (the pages run this normalisation
 * as a separate fused "norm ... QK" operation before the prefill; "Open-Jev-27B-v1.1
 * native text worker", "Validation and optimization scope").  The norms are summed
 * in fp32 from the bf16 inputs and applied as row scalings of the fp32 products, so
 * no normalised copy of q or k is written.
 *
 * GDN_FLAG_TWO_LEVEL: use the two-level chunk scan described under gdn_prefill
 * whenever the batch is dense and has at least two chunks per sequence, with
 * GDN_FLAG_SEGMENTS(n) segments per sequence (capped at the chunk count) or, without
 * it, the library's choice (at least 3).  GDN_FLAG_ONE_LEVEL: never use it.  Both
 * together, or unknown flag bits, are GDN_ERR_ARG.
 *
 * GDN_FLAG_SLICE16 / GDN_FLAG_SLICE32 / GDN_FLAG_SLICE64: each state-carry CTA owns
 * 16, 32 or 64 rows of the dv x dk state.  Without one, the library takes 64 when dv is
 * a multiple of 64 and 1.5 x the waves (of one CTA per SM) of 64-row CTAs are fewer
 * than those of 32-row CTAs (many sequences or heads), 16 when twice as many 32-row
 * CTAs would still fit one wave (few heads), else 32.  More than one of them, or
 * GDN_FLAG_SLICE64 with dv = 32, is GDN_ERR_ARG.
 * The results are the same for every width.
 *
 * GDN_FLAG_WIDE_RANGE: the state carry takes its state-side tensor-core operands as
 * bf16 hi + lo pairs (fp32 range, ~2^-16 relative) and the chunk's UT transform and
 * score product as bf16, instead of fp16 throughout.  For inputs or states beyond
 * fp16's range (see "Precision and range" under gdn_prefill); slower.  Everything
 * else as gdn_prefill.
 */
int gdn_prefill_ex(const void *q, const void *k, const void *v,
                   const float *g, const float *beta,
                   const int32_t *cu_seqlens, const float *init_state,
                   void *out, float *final_state,
                   int B, int T, int Hk, int Hv, int dk, int dv,
                   unsigned flags, void *stream);

/*
 * gdn_prefill_ws -- gdn_prefill with a caller-owned workspace.
 *
 * Same arguments, layouts, alignment rules and status codes as gdn_prefill, plus
 * `workspace` (device memory, 256-byte aligned, at least gdn_workspace_bytes(B, T,
 * Hk, Hv, dk, dv, cu_seqlens != NULL) bytes, not shared with concurrent calls) and
 * its size.  The call allocates nothing and never synchronises the host, so a
 * caller can record it into a CUDA graph and replay it with new input values in
 * the same buffers -- the calling convention behind the pages' per-prompt-length
 * CUDA Graph replay ("Cua-S1 4B 0.2 native text worker", CUDA Graph paragraph).
 * Returns GDN_ERR_SCRATCH when the workspace is too small, GDN_ERR_ALIGN when it
 * is not 256-byte aligned.  Always the single-level path (no second stream, no
 * library buffers).
 */
int gdn_prefill_ws(const void *q, const void *k, const void *v,
                   const float *g, const float *beta,
                   const int32_t *cu_seqlens, const float *init_state,
                   void *out, float *final_state,
                   int B, int T, int Hk, int Hv, int dk, int dv,
                   void *workspace, size_t workspace_bytes, void *stream);

/*
 * gdn_decode -- one token per sequence on a carried state, the state updated in place.
 *
 *   q, k   bf16 [B, Hk, dk];  v bf16 [B, Hv, dv];  g, beta fp32 [B, Hv]
 *   state  fp32 [B, Hv, dv, dk]  read as S_{t-1}, overwritten with S_t
 *   out    bf16 [B, Hv, dv]      o_t = S_t q_t / sqrt(dk)
 *
 * The same recurrence as gdn_prefill applied to a single token, so a prefill of
 * T tokens followed by gdn_decode of token T+1 matches a prefill of T+1 tokens.
 * All pointers device memory, 16-byte aligned; out must not alias the inputs.
 * Asynchronous on `stream`; allocates nothing.  Returns GDN_OK or an argument /
 * alignment / launch error.
 */
int gdn_decode(const void *q, const void *k, const void *v, const float *g, const float *beta,
               float *state, void *out, int B, int Hk, int Hv, int dk, int dv, void *stream);

/*
 * gdn_set_phase_events -- timing hook for the NEXT gdn_prefill call on this host
 * thread.  ev_begin, ev_mid and ev_end are cudaEvent_t handles created by the
 * caller; they are recorded on the call's stream before the chunk-preparation
 * kernel, between it and the state-carry kernel, and after the state-carry
 * kernel.  The hook is consumed by that one call (pass NULLs to clear it).
 */
void gdn_set_phase_events(void *ev_begin, void *ev_mid, void *ev_end);

/*
 * gdn_prefill_static -- gdn_prefill for callers that cannot allocate device memory.
 *
 * The pages have no counterpart to this entry point.  It exists for callers that
 * are not allowed to call cudaMalloc: a plugin whose host engine owns all device
 * memory, a service with a memory budget fixed at start-up, or code that must not
 * take the implicit device synchronisation of cudaMalloc / cudaFree.  Same
 * arguments, layouts, alignment rules and status codes as gdn_prefill; the caller
 * still passes the inputs and outputs.  Instead of the grow-only workspace it uses
 * a fixed array of GDN_STATIC_SCRATCH_BYTES in device memory that every GPU
 * loading the library holds until the process exits; it calls no allocator.
 *   - Returns GDN_ERR_SCRATCH, before launching anything, when the problem needs
 *     more scratch than that.  gdn_workspace_bytes gives the need: 16 KiB per
 *     (64-token chunk, value head) pair, 32.5 KiB per (chunk, key head) pair for
 *     dk = 128 (16.5 KiB for dk <= 64) and a small table -- for example 64.5 MiB for
 *     one 4,096-token sequence with 32 value heads over 16 key heads.
 *   - All calls on a device share the array and it keeps the last call's contents.
 *     Calls whose GPU work overlaps (other streams, other host threads) race on it:
 *     the caller must order them.
 *   - The first call on each device looks the array's address up (with that device
 *     current); make that first call before capturing the stream into a CUDA graph.
 *   - Always the single-level path (no two-level scan).
 *   - Status bits of its kernels go to the array's first word; gdn_device_status reads
 *     and clears them with the workspace's.  gdn_set_phase_events applies as to
 *     gdn_prefill, and gdn_last_cuda_error reports its launch errors.
 */
int gdn_prefill_static(const void *q, const void *k, const void *v,
                       const float *g, const float *beta,
                       const int32_t *cu_seqlens, const float *init_state,
                       void *out, float *final_state,
                       int B, int T, int Hk, int Hv, int dk, int dv,
                       void *stream);

/*
 * Device status bits.  Every wait inside the kernels (on an MMA completion or a
 * TMA load) is bounded; a wait that runs out sets one of these bits in the first
 * word of the workspace, lets its copies and MMAs in flight land (bounded again),
 * frees its tensor memory and returns, so the context stays usable.  With
 * gdn_prefill_ws the word is the first 4 bytes of the caller's workspace; with
 * gdn_prefill_static it is the first word of the fixed array.
 */
#define GDN_STATUS_MMA_TIMEOUT 1       /* the state-carry kernel (or gdn_ssm_scan's, gdn_attn's) gave up waiting for an MMA phase */
#define GDN_STATUS_LOAD_TIMEOUT 2      /* the same, waiting for a tile load */
#define GDN_STATUS_PREP_LOAD_TIMEOUT 4 /* the preparation kernel gave up waiting (tile load or Gram product) */
#define GDN_STATUS_BAD_CU_SEQLENS 8    /* cu_seqlens was not 0 = cu[0] <= ... <= cu[B] = T (entries clamped) */
#define GDN_STATUS_NONFINITE_STATE 16  /* a final state of the fp16 state carry was not finite (see gdn_prefill) */
#define GDN_STATUS_SMALL_STATE 32      /* a final state of the fp16 state carry stayed below 2^-12 (see gdn_prefill) */
#define GDN_STATUS_BAD_PAGE 64         /* gdn_attn_step met a block that the cache does not have (unseen) */

/*
 * gdn_device_status -- synchronise the current device, return the status bits
 * accumulated since the last call (in *status: the OR of the words of the library's
 * workspaces, gdn_prefill's, gdn_ssm_scan's and the attention's, and, once gdn_prefill_static has run
 * on the device, the fixed array's) and clear them.  Returns GDN_OK or GDN_ERR_LAUNCH.
 */
int gdn_device_status(int *status);

/*
 * gdn_selftest_wait_timeout -- run the bounded-wait path on purpose: one CTA
 * waits on an mbarrier that nothing completes, gives up after `max_polls` polls,
 * and records GDN_STATUS_MMA_TIMEOUT, exactly as the kernels do.  *status gets
 * the recorded bits (synchronous).  Used to test failure detection without a GPU
 * fault.
 */
int gdn_selftest_wait_timeout(int max_polls, int *status);

/*
 * gdn_selftest_static_wait_timeout -- the same bounded wait, but recording its bit in
 * the status word of gdn_prefill_static's fixed array, where a wait that runs out
 * inside that entry point would; gdn_device_status then reports it.  Synchronous;
 * allocates nothing.  Returns GDN_OK, GDN_ERR_ARG (max_polls < 1) or GDN_ERR_LAUNCH.
 */
int gdn_selftest_static_wait_timeout(int max_polls);

/*
 * gdn_debug_fail_allocations -- test hook for failure handling: the next `count`
 * device allocations the library would make (workspace, staging or scan buffers)
 * fail as if cudaMalloc had run out of memory, so the call returns GDN_ERR_ALLOC
 * before launching anything and keeps its previous buffers.  0 switches it off.
 * Returns the count that was pending.  Needs no GPU.
 */
int gdn_debug_fail_allocations(int count);

/* Segments per sequence that gdn_prefill_ex with these flags (gdn_prefill: flags = 0)
 * would use on the current device: 1 for the single-level path, P >= 2 for the
 * two-level chunk scan.  0 on bad arguments or unknown flags. */
int gdn_scan_segments(int B, int T, int Hk, int Hv, int dk, int dv, int packed, unsigned flags);

/* Bytes of device workspace gdn_prefill needs for these sizes (0 on bad arguments). */
size_t gdn_workspace_bytes(int B, int T, int Hk, int Hv, int dk, int dv, int packed);

/* Release the calling device's workspace and staging buffers (synchronises the device). */
void gdn_release_workspace(void);

/* ---------------------------------------------------------------------------------------
 * The operators around the recurrence in a hybrid layer: the short causal convolution over
 * the channels that feed it, the selective state space scan (the other recurrence of such
 * layers), each for prompts and for single tokens, and the norm that opens a layer.
 *
 * All pointers are DEVICE memory, owned by the caller and not retained; every call is
 * asynchronous on `stream`, never synchronises the host (but for a gdn_ssm_scan, gdn_attn or
 * gdn_attn_step that has to make or enlarge the library's own workspace), and returns GDN_OK or, before anything is launched,
 * GDN_ERR_ARG / GDN_ERR_ALIGN (or GDN_ERR_LAUNCH from a launch).
 * Activations are bf16; sums, states of the scan and softplus / exp values are fp32.  A
 * `*_stride` is the distance between consecutive tokens in elements, so that an operand can
 * be a slice of a wider projection or convolution output; within a token the elements are
 * contiguous.  bf16 activations start on 16 bytes and, with more than one token, their
 * strides are multiples of 8 elements (GDN_ERR_ALIGN otherwise); dt has no such rule.
 * Outputs are contiguous and must not overlap the inputs unless stated.  Each call takes its
 * arguments in a struct, read before it returns.
 * ------------------------------------------------------------------------------------- */

/* Flags of gdn_conv and gdn_conv_step. */
#define GDN_CONV_SILU 1u /* out = silu(convolution), else the convolution itself */

/*
 * gdn_conv -- short causal convolution of every channel over the tokens of its sequence:
 *
 *     y[t, c] = act( bias[c] + sum_{k < K} weight[c, k] x[t - K + 1 + k, c] )
 *
 *   x            bf16 [Ttot, C], token stride x_stride
 *   weight       bf16 [C, K];  bias bf16 [C] or NULL
 *   cu_seqlens   int32 [B + 1] or NULL, as for gdn_prefill (dense: B sequences of T tokens;
 *                packed: T tokens in all; out-of-order entries read and write nothing out of
 *                range, their results are unspecified)
 *   init_state   bf16 [B, K - 1, C] or NULL: the inputs before each sequence, oldest first
 *                (NULL = zeros)
 *   out          bf16 [Ttot, C];  must not overlap x
 *   final_state  bf16 [B, K - 1, C] or NULL: the last K - 1 inputs of each sequence (of its
 *                state, where it is shorter); must not overlap init_state (GDN_ERR_ARG)
 *
 * K is 2, 3 or 4, C a multiple of 8.  Sums in fp32, one rounding to bf16.
 */
typedef struct gdn_conv_args {
  const void *x;
  long long x_stride;
  const void *weight, *bias;
  const int32_t *cu_seqlens;
  const void *init_state;
  void *out, *final_state;
  int B, T, C, K;
  unsigned flags;
  void *stream;
} gdn_conv_args;
int gdn_conv(const gdn_conv_args *args);

/*
 * gdn_conv_step -- gdn_conv for one token per sequence: x and out [B, C], state bf16
 * [B, K - 1, C] read and overwritten with the last K - 1 inputs.
 */
typedef struct gdn_conv_step_args {
  const void *x;
  long long x_stride;
  const void *weight, *bias;
  void *state, *out;
  int B, C, K;
  unsigned flags;
  void *stream;
} gdn_conv_step_args;
int gdn_conv_step(const gdn_conv_step_args *args);

/* Flags of gdn_ssm_scan and gdn_ssm_step. */
#define GDN_SSM_SOFTPLUS 1u /* the step is softplus(dt + dt_bias), else dt + dt_bias */
#define GDN_SSM_DT_F32 2u   /* dt is fp32, else bf16 */

/*
 * gdn_ssm_scan -- selective state space scan of a prompt, one decay per (token, value head):
 *
 *     S_t = exp(s_t A_h) S_{t-1} + s_t x_t B_t^T        s_t = softplus(dt_t + dt_bias_h)
 *     y_t = (S_t C_t + D_h x_t) silu(z_t)
 *
 * with S a dv x dk fp32 state.  B and C belong to key heads: value head h reads key head
 * h / (Hv / Hk).
 *
 *   x            bf16 [Ttot, Hv, dv];  dt [Ttot, Hv] bf16 or fp32 (any alignment of its type)
 *   A            fp32 [Hv] (negative: a decay);  Bm, Cm bf16 [Ttot, Hk, dk]
 *   D            fp32 [Hv] or NULL (no skip term);  dt_bias fp32 [Hv] or NULL
 *   z            bf16 [Ttot, Hv, dv] or NULL (no gate)
 *   cu_seqlens   as for gdn_conv; malformed entries also set GDN_STATUS_BAD_CU_SEQLENS
 *   init_state   fp32 [B, Hv, dv, dk] or NULL (zeros)
 *   out          bf16 [Ttot, Hv, dv]
 *   final_state  fp32 [B, Hv, dv, dk] or NULL; may alias init_state.  A sequence of no tokens
 *                returns its initial state.
 *
 * dk and dv are 32, 64 or 128 each.  A sequence's results do not depend on the values of other
 * sequences of a packed batch, infinities and NaN included.  Within a sequence the tokens are
 * worked on in chunks of 128 with products of matrices, so a value that is not finite makes the
 * outputs of its chunk before it not finite too.  Without softplus a step may be below zero; like a
 * decay rate A above 0 it grows the state, which may overflow.
 *
 * The state is fp32 throughout.  For a prompt's outputs it, and the weights between the tokens of
 * a chunk, are rounded to bf16 as operands of the matrix products (2^-9 of each term); the sums
 * are fp32.  gdn_ssm_step rounds nothing but its output.
 *
 * workspace: gdn_ssm_workspace_bytes(...) bytes of device memory for the sizes of the call,
 * 256-byte aligned, not shared with concurrent calls, or NULL for the library's own grow-only one
 * (shared by the calls on a device: order calls whose work could overlap, as for gdn_prefill;
 * enlarging it frees and allocates, which synchronises).  The bytes do not grow with the sizes:
 * few sequences and heads are cut into segments, whose sums they hold, and more are not, so a
 * smaller batch may need more.  A buffer kept over calls is sized for the largest need among them.
 * With a workspace the call allocates nothing and can be captured into a CUDA graph;
 * GDN_ERR_SCRATCH when it is too small.  Its first word, which the caller clears, collects status
 * bits; gdn_device_status reports those of the library's own.
 */
typedef struct gdn_ssm_scan_args {
  const void *x;
  long long x_stride;
  const void *dt;
  long long dt_stride;
  const float *A;
  const void *Bm;
  long long b_stride;
  const void *Cm;
  long long c_stride;
  const float *D;
  const void *z;
  long long z_stride;
  const float *dt_bias;
  const int32_t *cu_seqlens;
  const float *init_state;
  void *out;
  float *final_state;
  int B, T, Hk, Hv, dk, dv;
  unsigned flags;
  void *workspace;
  size_t workspace_bytes;
  void *stream;
} gdn_ssm_scan_args;
int gdn_ssm_scan(const gdn_ssm_scan_args *args);

/* Bytes of workspace gdn_ssm_scan needs for these sizes on the current device (0 on bad arguments). */
size_t gdn_ssm_workspace_bytes(int B, int T, int Hk, int Hv, int dk, int dv, int packed);

/*
 * gdn_debug_ssm_wait_polls -- test hook for the waits of gdn_ssm_scan's kernels: how often the
 * thread that issues copies and products looks before it gives up (0: at once; negative: the
 * usual limit, about a second; what waits for that thread keeps this one).  A call whose waits
 * give up ends, with GDN_STATUS_MMA_TIMEOUT or GDN_STATUS_LOAD_TIMEOUT in its status word and
 * nothing to be read in its outputs.  Returns the limit before.  Needs no GPU.
 */
int gdn_debug_ssm_wait_polls(int polls);

/*
 * gdn_ssm_step -- gdn_ssm_scan for one token per sequence (x, z, out [B, Hv, dv], dt [B, Hv],
 * Bm, Cm [B, Hk, dk]); state fp32 [B, Hv, dv, dk], 16-byte aligned, updated in place.
 */
typedef struct gdn_ssm_step_args {
  const void *x;
  long long x_stride;
  const void *dt;
  long long dt_stride;
  const float *A;
  const void *Bm;
  long long b_stride;
  const void *Cm;
  long long c_stride;
  const float *D;
  const void *z;
  long long z_stride;
  const float *dt_bias;
  float *state;
  void *out;
  int B, Hk, Hv, dk, dv;
  unsigned flags;
  void *stream;
} gdn_ssm_step_args;
int gdn_ssm_step(const gdn_ssm_step_args *args);

/* Flags of gdn_add_norm. */
#define GDN_NORM_E4M3 1u /* out is e4m3 with scales, else bf16 */

/*
 * gdn_add_norm -- root-mean-square norm with the residual's addition:
 *
 *     r = x + residual;   y = r / sqrt(mean(r^2) + eps) weight
 *
 *   x         bf16 [rows, D], row stride x_stride;  residual bf16 [rows, D] or NULL (r = x)
 *   weight    bf16 [D]
 *   residual_out  bf16 [rows, D] or NULL: r, rounded; may be `residual` itself
 *   out       bf16 [rows, D], or with GDN_NORM_E4M3 8-bit [rows, D] (y / scale, saturated)
 *   scales    fp32 [rows, ceil(D / group)] with GDN_NORM_E4M3: max(max |y|, 2^-96) / 448 over each
 *             `group` of columns (32, 64 or 128; 0: one scale per row)
 *
 * D is a multiple of 8 up to 32,768.  y is computed from the unrounded sum and rounded once.  A NaN
 * in a group makes its scale NaN.
 */
typedef struct gdn_add_norm_args {
  const void *x;
  long long x_stride;
  const void *residual, *weight;
  void *residual_out, *out;
  float *scales;
  int rows, D, group;
  float eps;
  unsigned flags;
  void *stream;
} gdn_add_norm_args;
int gdn_add_norm(const gdn_add_norm_args *args);

/* ---------------------------------------------------------------------------------------
 * Attention, the other kind of layer between the recurrences, and its paged key-value cache.
 * A server's step: gdn_cache_plan (blocks and slots of the new tokens), then in every layer
 * gdn_cache_append and gdn_attn (prompts) or gdn_attn_step (one token of every request).
 *
 * What is said above of pointers, streams, strides, alignment and return codes holds here too.
 * The cache of a layer is two tensors, k_cache and v_cache, [blocks, Hkv, page, d]: blocks of
 * `page` tokens (a multiple of 16), a head's tokens of a block one after the other; bf16, or
 * e4m3 with a scale a head (GDN_CACHE_E4M3: a value is its 8 bits times k_scale or v_scale of
 * its head, fp32 [Hkv]).  A `*_block_stride` is the distance between blocks in elements, a
 * multiple of 16.  A token's slot is block * page + its place in the block, below 2^31.
 *
 * Heads: query head h reads key head h / (Hq / Hkv); d is a multiple of 8 up to 128.
 * ------------------------------------------------------------------------------------- */

/* Flags of gdn_cache_append and gdn_attn_step. */
#define GDN_CACHE_E4M3 1u /* the cache is e4m3 with scales, else bf16 */

/*
 * gdn_cache_plan -- new blocks for the requests that need them, and a slot for every new token.
 *
 *   lens         int32 [B]: tokens that each request has in the cache; below 0: an idle row
 *   block_table  int32 [B, W], row stride table_stride: its blocks; new ones are put behind
 *   free_blocks  int32 [capacity], the stack of free blocks; free_count int32 [1], its height
 *   cu_seqlens   int32 [B + 1] or NULL: boundaries of the requests' new tokens among T (NULL: one
 *                each, T = B); out-of-order entries read and write nothing out of range
 *   slots        int32 [T]: slot of every new token; -1 for those of a request that is idle or
 *                refused, for those behind the last request, and where the table is out of range
 *   new_lens     int32 [B]: lens with the new tokens (may be `lens`)
 *   new_count    int32 [1]: the stack's height after the call (may be `free_count`)
 *   refused      int32 [1] or NULL: requests that got nothing
 *
 * Request b has ceil(lens / page) blocks and wants ceil((lens + new) / page).  Blocks go out from
 * the top of the stack in the requests' order.  A request is refused as a whole (its length, its
 * table and its blocks stay) when it would need more than W blocks, or when it needs blocks and
 * those before it and it want more than there are; so one refused for lack of blocks takes those
 * behind it that need blocks with it, not those that still have room.  B is at most 16,384.
 */
typedef struct gdn_cache_plan_args {
  const int32_t *lens;
  int32_t *block_table;
  long long table_stride;
  const int32_t *free_blocks, *free_count, *cu_seqlens;
  int32_t *slots, *new_lens, *new_count, *refused;
  int B, T, W, capacity, page;
  void *stream;
} gdn_cache_plan_args;
int gdn_cache_plan(const gdn_cache_plan_args *args);

/*
 * gdn_cache_append -- the keys and values of T tokens, bf16 [T, Hkv, d], to their slots.
 *
 * Slots below 0 or past the cache are passed over.  With e4m3 a value is x / scale, rounded once and
 * saturated (a NaN stays one).  Two tokens must not have the same slot: which of them each piece of
 * eight values comes from is then unspecified.
 */
typedef struct gdn_cache_append_args {
  const void *k;
  long long k_stride;
  const void *v;
  long long v_stride;
  void *k_cache;
  long long k_block_stride;
  void *v_cache;
  long long v_block_stride;
  const float *k_scale, *v_scale;
  const int32_t *slots;
  int T, Hkv, d, page, blocks;
  unsigned flags;
  void *stream;
} gdn_cache_append_args;
int gdn_cache_append(const gdn_cache_append_args *args);

/*
 * gdn_attn -- attention of prompts: causal, with an optional window and sinks:
 *
 *     o_i = sum_j w_ij v_j / sum_j w_ij,   w_ij = exp(scale q_i.k_j),   over the keys j that i sees
 *
 * The queries of a sequence are its last tokens: query i of n, with m keys, is at position
 * p = m - n + i.  It sees the keys j <= p; with window > 0, of those the j > p - window and the
 * j < sinks.  A query that sees no key gives 0 and an lse of minus infinity.
 *
 *   q, out        bf16 [T, Hq, d], [T, Hq, d];  k, v bf16 [Tk, Hkv, d];  token strides as above
 *   cu_seqlens    int32 [B + 1] or NULL (dense: B sequences of T queries and Tk keys each; packed: T
 *                 and Tk in all); rows of out behind the last sequence are left as they were
 *   cu_seqlens_k  int32 [B + 1] or NULL: boundaries of the keys, where they are not the queries'
 *   lse           fp32 [T, Hq] or NULL: log sum_j w_ij
 *
 * Hq / Hkv is at most 128, and there are at most 2^31 - 1,024 queries, and keys, in all.  What unseen
 * keys and values hold, infinities and NaN included, does not reach a query (where a value is not finite, the
 * queries of the tiles beside it that do not see it are worked out apart, more slowly and with other roundings;
 * those that see it are not).  Weights are rounded to bf16 as operands of the second product (2^-9 of each term);
 * scores, sums and the running maximum are fp32.
 *
 * workspace: gdn_attn_workspace_bytes(...) bytes of device memory, 256-byte aligned, not shared with
 * concurrent calls, or NULL for the library's own, of which each of up to 16 streams has one (another takes
 * over the one longest unused, and synchronises the device for it), so that calls on different streams may
 * overlap.  With a workspace the call allocates nothing and can be captured into a CUDA graph; without one
 * the capture of a gdn_attn_step, and of a device's first call, is refused with GDN_ERR_SCRATCH (a graph of
 * a gdn_attn without one holds the library's status words, which gdn_release_workspace frees).
 * The caller clears all of it once, before its first call; its first word collects status bits, and
 * gdn_device_status reports those of the library's own.
 */
typedef struct gdn_attn_args {
  const void *q;
  long long q_stride;
  const void *k;
  long long k_stride;
  const void *v;
  long long v_stride;
  const int32_t *cu_seqlens, *cu_seqlens_k;
  void *out;
  float *lse;
  int B, T, Tk, Hq, Hkv, d, window, sinks;
  float scale;
  unsigned flags; /* 0 */
  void *workspace;
  size_t workspace_bytes;
  void *stream;
} gdn_attn_args;
int gdn_attn(const gdn_attn_args *args);

/*
 * gdn_debug_attn_smem_base -- test hook: gdn_attn's kernels are made for devices whose system keeps 1,024
 * bytes of a block's shared memory, and the call is refused elsewhere (GDN_ERR_LAUNCH, before anything is
 * launched).  With bytes > 0 the library takes that for what the device says, until a call with 0.  Returns
 * what was set before.  Needs no GPU.
 */
int gdn_debug_attn_smem_base(int bytes);

/* Bytes of workspace that gdn_attn and gdn_attn_step need for these sizes on the current device, whatever
 * the lengths (0 on bad arguments). */
size_t gdn_attn_workspace_bytes(int B, int Hq, int Hkv, int d);

/*
 * gdn_attn_step -- gdn_attn for one token of each of B requests over the paged cache.
 *
 *   q, out       bf16 [B, Hq, d]
 *   block_table  int32 [B, W], row stride table_stride;  lens int32 [B]: tokens in the cache, the new
 *                one included (its query is at position lens - 1); below 1: gives 0; above W * page:
 *                counts as that
 *   lse          fp32 [B, Hq] or NULL
 *
 * A block outside [0, blocks) counts as unseen and sets GDN_STATUS_BAD_PAGE; the table's entries behind
 * a request's blocks are not read.  What the cache holds in places that are not seen changes nothing.
 * Weights keep 16 bits over a bf16 cache, 11 over an e4m3 one.
 */
typedef struct gdn_attn_step_args {
  const void *q;
  long long q_stride;
  const void *k_cache;
  long long k_block_stride;
  const void *v_cache;
  long long v_block_stride;
  const float *k_scale, *v_scale;
  const int32_t *block_table;
  long long table_stride;
  const int32_t *lens;
  void *out;
  float *lse;
  int B, Hq, Hkv, d, page, blocks, W, window, sinks;
  float scale;
  unsigned flags;
  void *workspace;
  size_t workspace_bytes;
  void *stream;
} gdn_attn_step_args;
int gdn_attn_step(const gdn_attn_step_args *args);

#ifdef __cplusplus
}
#endif

#endif /* GDN_H */

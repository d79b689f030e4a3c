/*
 * gdn.h — C ABI of the MI355X (gfx950) chunked gated-delta-rule training kernel.
 *
 * The operation (Gated DeltaNet training, forward and backward, on packed variable-length
 * sequences; flashinfer PR #8172 "non-deterministic context-parallel Cake GDN chunked
 * autograd backend", PR description) is, per document n and value head h, with q/k head
 * j = h / (HV / H):
 *
 *     qh, kh = l2norm(q_t), l2norm(k_t)        (only when l2norm_qk; l2norm(x) = x / sqrt(x.x + 1e-6))
 *     S_t    = exp(g_t) S_{t-1} + beta_t kh (v_t - exp(g_t) S_{t-1}^T kh)^T
 *     o_t    = S_t^T qh
 *
 * with S_0 = h0[n,h] (or 0) a d x d FP32 state (row = key index) and ht[n,h] = S_last.
 * g is the log decay and beta the write strength, both used as given. Documents never share
 * state. The argument set (q, k, v, g, beta, cu_seqlens, optional h0, optional in-kernel
 * q/k L2 norm, light/full saved set) follows the pages' problem statement (flashinfer PR #8542
 * description and README saved-set table quoted in its review).
 *
 * Layouts (row-major, token-major, all pointers 16-byte aligned device pointers):
 *   q, k        [T, H,  d]   io dtype (bf16 or f32)
 *   v, o        [T, HV, d]   io dtype
 *   dO, dv      [T, HV, d]   io dtype
 *   dq, dk      [T, H,  d]   io dtype
 *   g, beta     [T, HV]      f32;  dg, dbeta [T, HV] f32
 *   h0, ht      [N, HV, d, d] f32 (key index, value index); dht, dh0 the same
 *   cu_seqlens  [N + 1]      int32, cu_seqlens[0] = 0, nondecreasing, cu_seqlens[N] = T
 *
 * Ownership: the caller allocates every buffer (outputs, the saved set, the workspace) and
 * owns every stream. The library never allocates or frees device memory, never creates a
 * stream and never synchronises the host (gdn_status, a query, is the one call that waits).
 * Work is enqueued on `stream` (a hipStream_t; NULL = the default stream) and, when the
 * problem names one, on the caller's auxiliary stream problem->aux_stream: all of it runs
 * after the work enqueued on `stream` before the call and before the work enqueued there
 * after it (the auxiliary stream is forked from and joined back into `stream` with events).
 * With aux_stream = NULL every launch goes to `stream`. Inputs are not modified. Calls are
 * reentrant; calls that share a workspace or a saved buffer must not overlap. Concurrent calls
 * may name the same auxiliary stream: their auxiliary work then runs there one call after the
 * other.
 *
 * Errors: every entry returns GDN_OK or an error code; gdn_last_error() gives a message for
 * the calling thread. Host validation (shapes, cu_seqlens, sizes, pointers, alignment) runs
 * before the first launch, so a call it rejects writes nothing. A launch failure returns
 * GDN_EHIP. Two conditions can only be seen on the device, by the first kernel of a call:
 * a device cu_seqlens that disagrees with the host copy in the problem, and (gdn_bwd) a saved
 * buffer whose 256-byte tag does not name this problem, save mode and ABI version. Then every
 * kernel of the call skips its work, the call's floating-point outputs are filled with NaN,
 * and gdn_status() reports GDN_EINVAL or GDN_ESAVED. Faults inside kernels surface at the
 * caller's next synchronisation.
 */
#ifndef GDN_H_
#define GDN_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define GDN_ABI_VERSION 2

/* return codes */
#define GDN_OK 0
#define GDN_EINVAL 1       /* bad shape, cu_seqlens, null required pointer, misalignment */
#define GDN_EUNSUPPORTED 2 /* d not 64 or 128, or an unsupported dtype */
#define GDN_ESAVED 3       /* saved buffer not written by gdn_fwd/gdn_fwd_recompute for this problem */
#define GDN_EWORKSPACE 4   /* workspace smaller than gdn_workspace_bytes() */
#define GDN_EHIP 5         /* a HIP launch or runtime call failed */

/* io dtypes (q, k, v, o, dO, dq, dk, dv) */
#define GDN_DTYPE_BF16 0
#define GDN_DTYPE_F32 1

/* Saved-set forms (README saved-set table quoted in the review of flashinfer PR #8542; the
 * kept-tape form follows the `reuse_recompute_tapes` row of the option table quoted in the
 * review of flashinfer PR #8172).
 * LIGHT keeps Akk (the inverse of I + L per chunk, bf16 [T, HV, 64]), gcum (f32 [HV, T]) and
 * gamma (f32 [NT, HV]); the backward replays the state tape. FULL also keeps the state tape
 * (bf16 [NT, HV, d, d]), v_new (bf16 [T, HV, d]), w and u (bf16 [T, HV, d]) and Aqk
 * (bf16 [T, HV, 64]). TAPE keeps LIGHT plus the state tape only: a checkpointed step runs
 * gdn_fwd in LIGHT form, then gdn_fwd_recompute and gdn_bwd in TAPE form, so the backward binds
 * the tape that the recompute's walk wrote instead of replaying it. FULL and TAPE backwards
 * skip the replay walk. All forms give bitwise identical outputs and gradients. */
#define GDN_SAVE_LIGHT 0
#define GDN_SAVE_FULL 1
#define GDN_SAVE_TAPE 2

/* operations, for gdn_workspace_bytes and gdn_status */
#define GDN_OP_FWD 0
#define GDN_OP_RECOMPUTE 1
#define GDN_OP_BWD 2

typedef struct gdn_problem {
  int32_t n_seqs;                 /* N >= 1 documents (zero-length documents allowed) */
  int32_t h_qk;                   /* H q/k heads */
  int32_t h_v;                    /* HV value heads, a multiple of H */
  int32_t d;                      /* head dim, d_k = d_v = 64 or 128 */
  int64_t n_tokens;               /* T = cu_seqlens[N] */
  int32_t dtype;                  /* GDN_DTYPE_* of the io tensors */
  int32_t l2norm_qk;              /* 1: L2-normalise q and k rows inside the kernel */
  int32_t has_h0;                 /* 1: h0 is given (and gdn_bwd writes dh0) */
  int32_t want_ht;                /* 1: gdn_fwd writes ht */
  int32_t save_mode;              /* GDN_SAVE_LIGHT, GDN_SAVE_FULL or GDN_SAVE_TAPE */
  int32_t deterministic;          /* 1: fixed-order dq/dk reduction over the HV/H value heads
                                     of each q/k head (bitwise reproducible); 0: FP32 atomics */
  const int32_t* cu_seqlens_host; /* host copy of cu_seqlens, read during each call only */
  void* aux_stream;               /* optional second stream (hipStream_t) of the caller on the
                                     device of `stream`; NULL: every launch on `stream` */
  int32_t segments;               /* walk segments per document (the PR #8172 README option
                                     table's `segments` / `walk_seg` and its plan policy):
                                     1 = each document's state walk is one serial chain;
                                     P >= 2 = documents of at least 16 chunks are walked as up to
                                     P segments (transfer walks, a carry merge, then the
                                     segments' walks side by side); 0 = the library's count,
                                     from the shape and the device's CU count (segments only
                                     when the chains fill at most half of the CUs). At P > 1
                                     the saved set ends with the segments' start states */
  int32_t reserved0;              /* must be 0 */
} gdn_problem;

/* Bytes of the saved buffer for this problem and save_mode: a 256-byte tag plus the saved
 * tensors, each 256-byte aligned (per-token figures of the README saved-set table quoted in
 * the review of flashinfer PR #8542: light 6,339 B/token and full +67,584 B/token at
 * HV = 48, d = 128, all chunks full). 0 if the problem is invalid (see gdn_last_error). */
size_t gdn_saved_bytes(const gdn_problem* p);

/* Bytes of device workspace one call of `op` needs: chunk tables, the status word, inverse q/k
 * norms, the per-value-head decayed q.k tiles, the replayed state tape, the end-state-gradient
 * tape and the chunk-gradient work-queue counters (backward), FP32 dq/dk accumulators (atomic
 * reduction), the segment carry states. The
 * pages' byte queries (flashinfer PR #8172 description: saved, workspace and communication
 * byte-accounting APIs) are the model. 0 if the problem is invalid. */
size_t gdn_workspace_bytes(const gdn_problem* p, int op);

/* Forward (flashinfer PR #8172 description: the chunked training kernel's forward call; the
 * chunk programs it runs are those the commit messages of flashinfer PR #7097 name: prep,
 * intra, WY and the state walk). Writes o [T, HV, d], ht [N, HV, d, d] (if want_ht) and the
 * saved set. h0 may be NULL iff has_h0 = 0; ht may be NULL iff want_ht = 0. */
int gdn_fwd(const gdn_problem* p, const void* q, const void* k, const void* v, const float* g,
            const float* beta, const int32_t* cu_seqlens, const float* h0, void* o, float* ht,
            void* saved, void* workspace, size_t workspace_bytes, void* stream);

/* Checkpoint re-run of the forward (flashinfer PR #8172 description: the checkpointed call;
 * README option table: `recompute_output`, the re-run that launches no output program).
 * Writes the saved set only (no o, no ht), bitwise equal to the saved set gdn_fwd writes for
 * the same inputs and save_mode. */
int gdn_fwd_recompute(const gdn_problem* p, const void* q, const void* k, const void* v,
                      const float* g, const float* beta, const int32_t* cu_seqlens,
                      const float* h0, void* saved, void* workspace, size_t workspace_bytes,
                      void* stream);

/* Backward (flashinfer PR #8172 description: the backward call, with its gradient-state
 * traversal and gradient programs; the deterministic and float-atomic dq/dk reductions are
 * the pages' deterministic and non-deterministic packages). Reads the saved set of the
 * matching forward or recompute (same problem and save_mode), dO and optional dht (NULL = 0),
 * and writes dq, dk, dv, dg, dbeta and (if has_h0) dh0. */
int gdn_bwd(const gdn_problem* p, const void* q, const void* k, const void* v, const float* g,
            const float* beta, const int32_t* cu_seqlens, const float* h0, const void* saved,
            const void* dO, const float* dht, void* dq, void* dk, void* dv, float* dg,
            float* dbeta, float* dh0, void* workspace, size_t workspace_bytes, void* stream);

/* Device-side status of the last call of `op` that used this workspace (the refusals of
 * flashinfer PR #8542's description: a saved set that does not match is refused). Enqueues a
 * copy of the status word on `stream` and waits for `stream`: this query synchronises the
 * host. Returns GDN_OK, GDN_EINVAL (the device cu_seqlens disagreed with the host copy) or
 * GDN_ESAVED (gdn_bwd was given a saved buffer whose tag does not name this problem, save
 * mode and ABI version); a copy failure returns GDN_EHIP. */
int gdn_status(const gdn_problem* p, int op, const void* workspace, void* stream);

/* Size of the fixed device scratch array behind gdn_fwd_noalloc (64 MiB per device). */
#define GDN_NOALLOC_SCRATCH_BYTES (64u << 20)

/* gdn_fwd for callers that cannot allocate device memory (code under HIP graph capture, tight
 * serving loops, harnesses that forbid hipMalloc): the same forward, with its workspace in a
 * fixed device array of GDN_NOALLOC_SCRATCH_BYTES that the library holds on each device until
 * the process ends, instead of a caller's buffer. Every launch goes to `stream` (aux_stream is
 * ignored); no device memory is allocated or freed and no event is created. A problem whose
 * forward workspace (gdn_workspace_bytes(p, GDN_OP_FWD)) exceeds the array is refused with
 * GDN_EWORKSPACE. Calls on one device share the array: calls that overlap there (two streams,
 * two threads) race and must not be issued. */
int gdn_fwd_noalloc(const gdn_problem* p, const void* q, const void* k, const void* v, const float* g,
                    const float* beta, const int32_t* cu_seqlens, const float* h0, void* o, float* ht,
                    void* saved, void* stream);

/* ---- Short causal conv1d + SiLU front-end ------------------------------------------------
 * The depthwise causal convolution that the pages run over the packed q/k/v channels together
 * with the gated delta rule (flashinfer PR #8542 "Conventions": shape B23 runs the short causal
 * convolution over the 10,240 packed q/k/v channels on every timed call; flashinfer PR #7117: the
 * causal conv1d + SiLU training backend of the same kernel family; the README saved-set table
 * keeps at most 3 history rows, a window of 4 taps). Per document (cu_seqlens as above), channel
 * c and token t:
 *
 *     pre[t, c] = bias[c] + sum_{i<W} weight[c, i] x[t - (W-1) + i, c]   (x = 0 before the document)
 *     y[t, c]   = SiLU(pre[t, c]) = pre / (1 + exp(-pre))                 (pre when silu = 0)
 *
 * x is [T, C] in the io dtype; weight f32 [C, W] (tap W-1 multiplies the current token); bias f32
 * [C] or NULL. The output channels are written split into n_groups tensors y[g] of
 * [T, group_channels[g]] (e.g. q, k, v: 2048, 2048, 6144 channels), so the gated delta rule reads
 * them without a copy; the backward takes the upstream gradients split the same way and writes dx
 * [T, C], dweight f32 [C, W] and dbias f32 [C] (if non-NULL). The weight and bias gradients are
 * summed in a fixed order (bitwise reproducible). Ownership, streams and errors as above; these
 * calls use `stream` only. */
typedef struct gdn_conv_problem {
  int32_t n_seqs;                 /* N >= 1 documents */
  int32_t channels;               /* C = sum of group_channels, a multiple of 8 */
  int64_t n_tokens;               /* T = cu_seqlens[N] */
  int32_t width;                  /* W taps, 1..4 */
  int32_t dtype;                  /* GDN_DTYPE_* of x, y, dy, dx */
  int32_t silu;                   /* 1: y = SiLU(pre); 0: y = pre */
  int32_t n_groups;               /* 1..4 output tensors */
  int32_t group_channels[4];      /* channels of each output tensor, multiples of 8 */
  const int32_t* cu_seqlens_host; /* host copy of cu_seqlens, read during each call only */
} gdn_conv_problem;

/* Bytes of device workspace gdn_conv_bwd needs (the per-workgroup partial sums of dweight and
 * dbias). 0 if the problem is invalid. */
size_t gdn_conv_workspace_bytes(const gdn_conv_problem* p);

/* Forward: y[g] for every group. */
int gdn_conv_fwd(const gdn_conv_problem* p, const void* x, const float* weight, const float* bias,
                 const int32_t* cu_seqlens, void* const* y, void* stream);

/* Backward: dx, dweight and (if non-NULL) dbias from x and the split upstream gradients dy[g]. */
int gdn_conv_bwd(const gdn_conv_problem* p, const void* x, const float* weight, const float* bias,
                 const int32_t* cu_seqlens, const void* const* dy, void* dx, float* dweight, float* dbias,
                 void* workspace, size_t workspace_bytes, void* stream);

/* ---- The gated delta rule, recurrent: one serving step on cached states --------------------
 * The operation at the top of this file, token by token, on states that live in a cache between
 * calls: one token a sequence when decoding, a few when drafted tokens are checked or a prompt is
 * extended (whole prompts go through gdn_fwd, whose h0 and ht have the layout of cached states. It is
 * faster from about 256 tokens on with one sequence, 85 with 4, 32 with 12 ((16, 48) heads, d = 128,
 * bf16), and rounds its products' operands to bf16: an error of 2.4e-3 in the state after 512 tokens,
 * where FP32 here leaves 1.6e-7).
 * Sequence n starts from states[slot_in[n]] (from zero if slot_in[n] = -1), runs its tokens in
 * order and leaves its last state in states[slot_out[n]] (nowhere if -1; a sequence of no tokens
 * leaves its start state). slot_in[n] = slot_out[n] updates a state in place. slot_tok, if given,
 * names for each token the slot that keeps the state after it (-1: none), so that a run of drafted
 * tokens can be rolled back to any of them. All arithmetic is FP32. Longer sequences (by the host's
 * lengths; without slot_tok) are taken 16 tokens at a time; where that ends in a state that is not
 * finite, once more token by token, so an infinity or NaN reaches what the recurrence takes it to and
 * no earlier token, and log decays may rise as far as the recurrence itself stays in FP32's range.
 * The order of the sums follows from the call's sizes and lengths, so the same call gives the same bits, and a
 * sequence in calls of different sizes may differ by rounding.
 *
 *   q, k      [T, H, d], v [T, HV, d]  io dtype; a token's heads are contiguous, tokens are
 *                                      q_stride, k_stride, v_stride elements apart
 *   g, beta   [T, HV] f32;  o [T, HV, d] io dtype (contiguous)
 *   states    [n_slots, HV, d, d] f32 (key index, value index)
 *   slot_in, slot_out  [N] int32;  slot_tok [T] int32 or NULL
 *   cu_seqlens [N + 1] int32, or NULL (with cu_seqlens_host NULL): one token a sequence, T = N
 *
 * A state is read whole before any state of its sequence is written, and sequences run side by
 * side: a slot that one sequence writes must not be read or written by another in the same call.
 * The call may be captured into a graph; the device arrays are read at each replay. They are
 * checked on the device: a sequence with a token range outside [0, T] or a slot outside
 * [-1, n_slots) writes no state and fills its o rows (those inside [0, T]) with NaN, as does a
 * token with such a slot_tok for its own state and row. Lengths on the device may differ from the
 * host's (a graph replayed with other lengths, or a shorter batch: T and N stay, sequences may be
 * empty): rows of o that no sequence covers are not written and keep what the buffer held. */
typedef struct gdn_recurrent_problem {
  int32_t n_seqs;                 /* N >= 1 sequences (of zero tokens or more); N and T at most 2^31 - 2^20 */
  int32_t h_qk;                   /* H q/k heads */
  int32_t h_v;                    /* HV value heads, a multiple of H */
  int32_t d;                      /* head dim, 64 or 128 */
  int64_t n_tokens;               /* T */
  int32_t dtype;                  /* GDN_DTYPE_* of q, k, v, o */
  int32_t l2norm_qk;              /* 1: L2-normalise q and k rows inside the kernel */
  int32_t n_slots;                /* states in the cache, >= 1 */
  int32_t reserved0;              /* must be 0 */
  int64_t q_stride;               /* elements from one token's q to the next (0: H * d, at most */
  int64_t k_stride;               /* 2^24); the same for k (0: H * d) and v (0: HV * d). Rows are */
  int64_t v_stride;               /* 16-byte aligned */
  const int32_t* cu_seqlens_host; /* host copy of cu_seqlens, read during each call only; NULL: one
                                     token a sequence */
} gdn_recurrent_problem;

int gdn_recurrent(const gdn_recurrent_problem* p, const void* q, const void* k, const void* v, const float* g,
                  const float* beta, const int32_t* cu_seqlens, const int32_t* slot_in, const int32_t* slot_out,
                  const int32_t* slot_tok, float* states, void* o, void* stream);

/* ---- Norms of the q and k heads with the position rotation ---------------------------------
 * What stands between a layer's q/k projections (or the conv front-end) and the rule or an
 * attention over the same heads, in one pass over q and k. For each head row x of a token at
 * position p (d values, weight w or all ones):
 *
 *   n = x / sqrt(mean(x^2) + eps)      (GDN_NORM_RMS)
 *       x / sqrt(sum(x^2) + eps)       (GDN_NORM_L2)
 *       x                              (GDN_NORM_NONE: the rotation alone)
 *   z = n w
 *   y = z with the pairs (z_a, z_b) of its first rotary_dim values turned by the angle p f_i:
 *       y_a = m (z_a cos - z_b sin),  y_b = m (z_b cos + z_a sin),  i = 0 .. rotary_dim / 2 - 1
 *       pairs (i, i + rotary_dim / 2), or with interleaved = 1 (2 i, 2 i + 1)
 *
 * freqs holds f_i as an unsigned 64-bit fraction of a turn per position, f_i / (2 pi) 2^64, so that
 * the angle modulo a turn is exact at every position: gdn_rope_frequencies makes it. m is the
 * magnitude. The backward takes the gradients of y and the forward's inputs and gives those of
 * x and of the weights (summed over tokens and heads in a fixed order: bitwise reproducible).
 * Outputs may be the inputs' own buffers (q_out = q, k_out = k; dq = dq_out, dk = dk_out): each
 * row is read before it is written, by the same lanes. */
#define GDN_NORM_NONE 0
#define GDN_NORM_L2 1
#define GDN_NORM_RMS 2

typedef struct gdn_qk_rope_problem {
  int64_t n_tokens;    /* T >= 0 */
  int32_t h_q;         /* q heads, 1 .. 16384 */
  int32_t h_k;         /* k heads, 0 .. 16384 (0: no k tensors) */
  int32_t d;           /* head dim, a multiple of 8, 8 .. 256 */
  int32_t dtype;       /* GDN_DTYPE_* of q, k and their outputs and gradients */
  int32_t norm;        /* GDN_NORM_* */
  int32_t rotary_dim;  /* values of each head that are rotated: a multiple of 8, 0 .. d */
  int32_t interleaved; /* 0: pairs half the rotary dim apart; 1: neighbours */
  float eps;           /* added under the norm's root */
  float magnitude;     /* m */
  int32_t reserved0;   /* must be 0 */
  int64_t q_stride;    /* elements between the tokens of q (0: contiguous), */
  int64_t k_stride;    /* of k, */
  int64_t qo_stride;   /* of q_out and dq_out, */
  int64_t ko_stride;   /* of k_out and dk_out, */
  int64_t dq_stride;   /* of dq */
  int64_t dk_stride;   /* and of dk (the backward's). At most 2^27; rows are 16-byte aligned */
} gdn_qk_rope_problem;

/* Frequencies of the rotation, on the host: freqs[i] (rotary_dim / 2 of them) and the magnitude,
 * from the base b and one of
 *   GDN_ROPE_PLAIN  f_i = b^(-2 i / rotary_dim)
 *   GDN_ROPE_LINEAR f_i / factor (every position divided by factor)
 *   GDN_ROPE_NTK    the base raised to b factor^(rotary_dim / (rotary_dim - 2))
 *   GDN_ROPE_YARN   f_i (1 - r_i) + f_i / factor r_i, r_i rising from 0 to 1 over the indices i between
 *                   those that make `fast` and `slow` turns in original_length positions (rounded
 *                   outwards); magnitude 0.1 ln(factor) + 1 for factor > 1
 *   GDN_ROPE_BANDS  the same blend with r_i = 1 - (turns_i - slow) / (fast - slow), cut to [0, 1], where
 *                   turns_i = original_length f_i / (2 pi); magnitude 1
 * (YaRN: Peng et al. 2023, the blend by index and the blend by turns of its section 3.2.) */
#define GDN_ROPE_PLAIN 0
#define GDN_ROPE_LINEAR 1
#define GDN_ROPE_NTK 2
#define GDN_ROPE_YARN 3
#define GDN_ROPE_BANDS 4

typedef struct gdn_rope_scaling {
  int32_t kind;           /* GDN_ROPE_* */
  int32_t rotary_dim;     /* even, >= 2 */
  double base;            /* > 1 */
  double factor;          /* > 0 (not read by GDN_ROPE_PLAIN) */
  double original_length; /* > 0 (GDN_ROPE_YARN and GDN_ROPE_BANDS) */
  double fast;            /* turns: fast > slow > 0 (GDN_ROPE_YARN and GDN_ROPE_BANDS) */
  double slow;
} gdn_rope_scaling;

int gdn_rope_frequencies(const gdn_rope_scaling* s, uint64_t* freqs_host, float* magnitude);

/* Bytes of device workspace gdn_qk_rope_bwd needs (the workgroups' partial sums of the weight
 * gradients). 0 if the problem is invalid. */
size_t gdn_qk_rope_workspace_bytes(const gdn_qk_rope_problem* p);

/* Forward: q_out, k_out. positions [T] int32 (any sign) and freqs [rotary_dim / 2] uint64 on the
 * device, NULL iff rotary_dim = 0; q_weight, k_weight f32 [d] or NULL (NULL with GDN_NORM_NONE). */
int gdn_qk_rope_fwd(const gdn_qk_rope_problem* p, const void* q, const void* k, const int32_t* positions,
                    const uint64_t* freqs, const float* q_weight, const float* k_weight, void* q_out, void* k_out,
                    void* stream);

/* Backward: dq, dk from q, k (not read, may be NULL, with GDN_NORM_NONE) and the upstream
 * gradients dq_out, dk_out; dq_weight, dk_weight f32 [d] iff the weight is given. */
int gdn_qk_rope_bwd(const gdn_qk_rope_problem* p, const void* q, const void* k, const int32_t* positions,
                    const uint64_t* freqs, const float* q_weight, const float* k_weight, const void* dq_out,
                    const void* dk_out, void* dq, void* dk, float* dq_weight, float* dk_weight, void* workspace,
                    size_t workspace_bytes, void* stream);

/* ---- The conv front-end's serving step ------------------------------------------------------
 * gdn_conv_fwd's operation on sequences whose last W - 1 inputs live in a cache between calls:
 * windows [n_slots, W - 1, C] in the io dtype, oldest row first (the last W - 1 rows of a prompt's
 * x, zeros before its first token, are its window). Slots, cu_seqlens, in-place updates and the
 * checks on the device are those of gdn_recurrent: a sequence reads windows[slot_in[n]] (zeros if
 * -1), writes its last window to windows[slot_out[n]], and slot_tok keeps the window after each
 * token. Where gdn_recurrent fills o rows with NaN, the rows of every y[g] are, and rows that no
 * sequence covers are not written. */
typedef struct gdn_conv_step_problem {
  int32_t n_seqs;                 /* N >= 1 sequences */
  int32_t channels;               /* C = sum of group_channels, a multiple of 8 */
  int64_t n_tokens;               /* T */
  int32_t width;                  /* W taps, 1..4 (at 1 there is no window: windows may be NULL) */
  int32_t dtype;                  /* GDN_DTYPE_* of x, y and windows */
  int32_t silu;                   /* 1: y = SiLU(pre); 0: y = pre */
  int32_t n_groups;               /* 1..4 output tensors */
  int32_t group_channels[4];      /* channels of each output tensor, multiples of 8 */
  int32_t n_slots;                /* windows in the cache, >= 1 */
  int32_t reserved0;              /* must be 0 */
  int64_t x_stride;               /* elements from one token's x to the next (0: C); 16-byte rows */
  const int32_t* cu_seqlens_host; /* host copy of cu_seqlens; NULL: one token a sequence */
} gdn_conv_step_problem;

int gdn_conv_step(const gdn_conv_step_problem* p, const void* x, const float* weight, const float* bias,
                  const int32_t* cu_seqlens, const int32_t* slot_in, const int32_t* slot_out,
                  const int32_t* slot_tok, void* windows, void* const* y, void* stream);

/* ---- Linear attention with a decay for each head ---------------------------------------------
 * The layer without the delta rule: per document n and value head h, with q/k head j = h / (HV / H),
 *
 *     S_t = exp(g_t) S_{t-1} + k_t v_t^T,   o_t = scale S_t^T q_t
 *
 * S_0 = h0[n,h] (or 0) and ht[n,h] = S_last as in gdn_fwd. The log decays g are one for each token and
 * head (GDN_DECAY_TOKEN, [T, HV]) or one for each head (GDN_DECAY_HEAD, [HV]). Layouts as at the top of
 * this file (g may start at any of its values); q, k and v may be parts of one row (their strides in the
 * problem). o, ht and the gradients are contiguous and no buffers of the inputs (ht over h0, and dh0 over h0 or
 * dht, are refused). States, decays and sums are FP32 (the sums of the log decays 64-bit); for bf16 the decayed
 * products of a chunk and the state that they meet are rounded once to bf16 for o, dv and, without dg, dq and dk,
 * which are rounded to it themselves (2.3e-3 instead of 1.7e-3 off); of a group's value heads each head's dq and dk
 * are rounded to 11 bits before their sum. ht, dh0 and dg keep FP32's accuracy. With f32 rows nothing is rounded
 * to fewer bits. All sums have a fixed order: the same call gives the same bits.
 *
 * A document goes in chunks of 64 tokens, and what is not finite in a token reaches, through zeros of
 * masked products, all tokens of its chunk (forward also earlier ones), then what depends on the state;
 * other documents never. A log decay of minus infinity drops the state (as any under -10000), and dg is 0 there
 * (as at any under -104). Log decays may be positive while their sums over a chunk, and over the tokens that a
 * state other than zero passes, stay in FP32's range.
 *
 * The launch is planned from the host's lengths; the device's cu_seqlens may hold others (a graph that is
 * replayed with other lengths, or a shorter batch: T and N stay), as long as it rises from 0 or more to
 * at most T. Values that do not are cut to that range, and the rows of such documents are then not
 * specified. Rows of o and of gradients that no document covers are not written. */
#define GDN_DECAY_TOKEN 0
#define GDN_DECAY_HEAD 1

typedef struct gdn_linear_problem {
  int32_t n_seqs;                 /* N documents, 1 .. 65535 (of zero tokens or more) */
  int32_t h_qk;                   /* H q/k heads */
  int32_t h_v;                    /* HV value heads, a multiple of H, at most 65535; HV d at most 2^22 */
  int32_t d;                      /* head dim, 64 or 128 */
  int64_t n_tokens;               /* T = cu_seqlens[N], at most 2^31 - 2^20 */
  int32_t dtype;                  /* GDN_DTYPE_* of q, k, v, o and their gradients */
  int32_t decay;                  /* GDN_DECAY_* */
  int32_t has_h0;                 /* 1: h0 is given (and gdn_linear_bwd writes dh0) */
  int32_t want_ht;                /* 1: gdn_linear_fwd writes ht */
  float scale;                    /* of the outputs */
  int32_t reserved0;              /* must be 0 */
  int64_t q_stride;               /* elements from one token's q to the next (0: H * d), at most */
  int64_t k_stride;               /* 2^22; the same for k and v (0: HV * d). Rows are 16-byte */
  int64_t v_stride;               /* aligned */
  const int32_t* cu_seqlens_host; /* host copy of cu_seqlens, read during each call only */
} gdn_linear_problem;

/* Bytes of device workspace a call of `op` (GDN_OP_FWD, GDN_OP_BWD) needs: the states that long documents'
 * segments start from, and in the backward their gradients, row products for dg and, with shared heads,
 * dq and dk before their sums over a group. 0 if the problem is invalid. */
size_t gdn_linear_workspace_bytes(const gdn_linear_problem* p, int op);

/* Forward: o, and ht if want_ht. */
int gdn_linear_fwd(const gdn_linear_problem* p, const void* q, const void* k, const void* v, const float* g,
                   const int32_t* cu_seqlens, const float* h0, void* o, float* ht, void* workspace,
                   size_t workspace_bytes, void* stream);

/* Backward, from the forward's inputs alone (no saved set): dq, dk, dv from dO and optional dht (NULL = 0);
 * dg (g's layout) if not NULL; dh0 iff has_h0. Without dg the products that it alone needs are left out. */
int gdn_linear_bwd(const gdn_linear_problem* p, const void* q, const void* k, const void* v, const float* g,
                   const int32_t* cu_seqlens, const float* h0, const void* dO, const float* dht, void* dq, void* dk,
                   void* dv, float* dg, float* dh0, void* workspace, size_t workspace_bytes, void* stream);

/* Its serving step on cached states, token by token in FP32: slots, cu_seqlens, slot_tok and the checks on
 * the device are gdn_recurrent's. From runs of about 12 tokens on gdn_linear_fwd is faster, whose h0 and ht have
 * the layout of cached states. */
typedef struct gdn_linear_step_problem {
  int32_t n_seqs;                 /* N >= 1 sequences (of zero tokens or more); N and T at most 2^31 - 2^20 */
  int32_t h_qk;                   /* H q/k heads */
  int32_t h_v;                    /* HV value heads, a multiple of H */
  int32_t d;                      /* head dim, 64 or 128 */
  int64_t n_tokens;               /* T */
  int32_t dtype;                  /* GDN_DTYPE_* of q, k, v, o */
  int32_t decay;                  /* GDN_DECAY_* */
  float scale;                    /* of the outputs */
  int32_t n_slots;                /* states in the cache, >= 1 */
  int32_t reserved0;              /* must be 0 */
  int64_t q_stride;               /* as in gdn_recurrent_problem */
  int64_t k_stride;
  int64_t v_stride;
  const int32_t* cu_seqlens_host; /* host copy of cu_seqlens; NULL: one token a sequence */
} gdn_linear_step_problem;

int gdn_linear_step(const gdn_linear_step_problem* p, const void* q, const void* k, const void* v, const float* g,
                    const int32_t* cu_seqlens, const int32_t* slot_in, const int32_t* slot_out, const int32_t* slot_tok,
                    float* states, void* o, void* stream);

/* ---- RMS norm of rows with the residual's addition --------------------------------------------
 * What stands before a layer's projections. For each row of d values (weight w, or ones):
 *
 *     x' = x + residual                  (FP32; x without a residual)
 *     residual_out = x'                  (rounded to the io type)
 *     y  = w x' / sqrt(mean(x'^2) + eps) (of x' before that rounding)
 *
 * y is in the io type (GDN_OUT_IO), or in 8 bits (GDN_OUT_E4M3: sign, 4 exponent and 3 mantissa bits, largest
 * value 448) with an FP32 scale for each row (group = 0) or each `group` values of it: scale = the largest
 * magnitude / 448 (1 where all are zero, at least 2^-126) and y the value nearest to that of the FP32 row over scale,
 * ties to even (for scales of 2^-90 and more; below, of FP32's quotient). y and residual_out may be the inputs'
 * own buffers (of the same row layout): each row is read before it is written. The squares' sum has to stay in
 * FP32's range: below its largest number, and with eps = 0 not under its smallest (a row of zeros then gives NaN). What
 * is not finite stays in its row (and in dweight). */
#define GDN_OUT_IO 0
#define GDN_OUT_E4M3 1

typedef struct gdn_rms_norm_problem {
  int64_t n_rows;          /* >= 0 */
  int32_t d;               /* a multiple of 8, 8 .. 16384 */
  int32_t dtype;           /* GDN_DTYPE_* of x, residual, y (GDN_OUT_IO) and gradients */
  int32_t out;             /* GDN_OUT_* */
  int32_t group;           /* GDN_OUT_E4M3: values that share a scale: 0 (the row), 32, 64 or 128 */
  float eps;               /* added under the root */
  int32_t reserved0;       /* must be 0 */
  int64_t x_stride;        /* elements between the rows of x (0: contiguous) */
  int64_t residual_stride; /* and of residual (backward: of d_residual). Rows are 16-byte aligned */
} gdn_rms_norm_problem;

/* Bytes of device workspace gdn_rms_norm_bwd needs (workgroups' sums of dweight). 0 if the problem is invalid. */
size_t gdn_rms_norm_workspace_bytes(const gdn_rms_norm_problem* p);

/* Forward: y [n_rows, d]; scales f32 [n_rows, d / group] with GDN_OUT_E4M3; residual_out [n_rows, d] iff residual. */
int gdn_rms_norm_fwd(const gdn_rms_norm_problem* p, const void* x, const float* weight, const void* residual, void* y,
                     float* scales, void* residual_out, void* stream);

/* Backward of the GDN_OUT_IO form at x' = x (what the forward left in residual_out): dx = the gradient of x'
 * through y plus d_residual (that of residual_out; NULL: 0), which is the gradient of the forward's x and
 * residual alike; dweight f32 [d] (NULL: not wanted), summed in a fixed order. dx may be dy or a contiguous d_residual or x. */
int gdn_rms_norm_bwd(const gdn_rms_norm_problem* p, const void* x, const float* weight, const void* dy,
                     const void* d_residual, void* dx, float* dweight, void* workspace, size_t workspace_bytes, void* stream);

/* ---- What a serving step reads, from the requests' lengths -------------------------------------
 * N requests with contexts[n] tokens in the caches and lengths[n] new ones. Caches are cut into blocks of
 * `block` tokens; block_table[n, b] names the block that holds tokens b block .. of request n. Blocks that new
 * tokens enter are taken from the end of free_list[0 .. free_count), in the requests' order, and written to the
 * table (its other entries stay). Made for the step:
 *
 *   granted [N]       tokens that the request gets: lengths[n], or 0 from the first request on whose tokens or
 *                     blocks do not fit any more (n_tokens, free_count); also 0, for that request alone, where
 *                     lengths[n] or contexts[n] is negative or the table has no room for them
 *   cu_seqlens [N+1]  running sums of granted, from 0
 *   positions [T]     the position of each token in its request (0 behind the last)
 *   token_slots [T]   its row in a cache of blocks, block_table[n, p / block] block + p % block (-1 behind the last)
 *   slot_in [N]       the block of the request's last token in the caches (-1 with none): the state that it starts from
 *   slot_out [N]      the block of its last token after the step (slot_in without new tokens): where its state goes
 *   slot_tok [T]      for each token that ends a block and is not the step's last of its request that block, else -1:
 *                     states after whole blocks stay behind, as starts for requests that share the tokens so far
 *   contexts [N]      contexts + granted; free_count [1] what is left (both may be the inputs' own buffers)
 *
 * With slots that are blocks, gdn_recurrent, gdn_linear_step and gdn_conv_step read cu_seqlens, slot_in, slot_out and
 * slot_tok, and gdn_qk_rope positions, as they are. Any output may be NULL. A free_count outside
 * [0, n_free] is cut to that. The call may be captured; all of its arrays are read at each replay. */
typedef struct gdn_step_maps_problem {
  int32_t n_seqs;     /* N requests, 1 .. 4096 */
  int32_t block;      /* tokens of a block, >= 1 */
  int64_t n_tokens;   /* T: room for new tokens, 0 .. 2^31 - 2^20 */
  int32_t max_blocks; /* columns of block_table, >= 1 */
  int32_t n_free;     /* entries of free_list, >= 0 */
  int32_t reserved0;  /* must be 0 */
} gdn_step_maps_problem;

typedef struct gdn_step_maps_out {
  int32_t* cu_seqlens;
  int32_t* positions;
  int64_t* token_slots;
  int32_t* granted;
  int32_t* slot_in;
  int32_t* slot_out;
  int32_t* slot_tok;
  int32_t* contexts;
  int32_t* free_count;
} gdn_step_maps_out;

int gdn_step_maps(const gdn_step_maps_problem* p, const int32_t* lengths, const int32_t* contexts, int32_t* block_table,
                  const int32_t* free_list, const int32_t* free_count, const gdn_step_maps_out* out, void* stream);

/* Message of the calling thread's last error ("" if none). */
const char* gdn_last_error(void);

/* GDN_ABI_VERSION of the loaded library. */
int gdn_abi_version(void);

/* Kernel timing, for benchmarks. While enabled (on = 1), every kernel launch of the library is
 * bracketed by two hipEvents recorded on the stream it is launched on (no synchronisation at
 * launch). gdn_timing_collect waits for all recorded events, adds their elapsed times to
 * per-kernel totals and returns the number of distinct kernels; for the first `max` (in name
 * order) it fills names (valid until the next collect on this thread), total_ms and launch
 * counts (any array may be NULL). gdn_timing_launches (call it before gdn_timing_collect, which
 * drops the pending events) waits for them as well and fills, for up to `max` launches in
 * launch order, the kernel name and the start and end times in ms after the earliest start;
 * it returns the number of pending launches. gdn_timing_reset drops totals and pending events. */
void gdn_timing_enable(int on);
int gdn_timing_collect(int max, const char** names, double* total_ms, int* launches);
int gdn_timing_launches(int max, const char** names, double* start_ms, double* end_ms);
void gdn_timing_reset(void);

#ifdef __cplusplus
}
#endif

#endif /* GDN_H_ */

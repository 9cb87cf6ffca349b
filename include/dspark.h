/*
 * dspark.h -- C ABI of the DSpark proposal head and the greedy verify step.
 *
 * The method (llama.cpp commit 6fed9f6, src/models/dflash.cpp, squash log of
 * "spec: add DSpark speculative decoding", the proposal formula):
 *
 *   logits(i)  = h[b, i] . lm_head^T (+ lm_bias)
 *   logits'(i) = logits(i) + markov_w2^T . markov_w1[prev(i)]
 *   prev(0)    = the block's anchor token,  prev(i > 0) = argmax logits'(i - 1)
 *
 * run greedily over the slots of a block and in parallel over the blocks of a batch,
 * followed by DFlash's unchanged greedy verify/accept.  The confidence head
 * conf = sigmoid(h . w_conf + b_conf) truncates each block at its first slot below
 * conf_min ("spec: add confidence-based draft pruning for DSpark").  Block layouts:
 * anchor-first (every slot predicts) and the 1+N bonus-anchor layout of
 * speculators-format drafts (llama.cpp PR #26275, "Format differences": slot 0 holds
 * the bonus token and is not a prediction slot).  Reduced draft vocabularies come in
 * the two forms PR #26275 describes: an lm_head expanded to the full vocabulary with a
 * -1e9 bias on rows the draft cannot emit, or a compact head plus a d2t table of
 * absolute target ids.
 *
 * Conventions shared by every entry point:
 *   - Pointers named "device" must point to device memory of the current device;
 *     "host" pointers to host memory.  The caller owns every buffer; the library keeps
 *     no pointer after a call returns and allocates no device memory.
 *   - Arrays are dense and row-major with the shapes given; element types are the
 *     config's dtype for the tensors marked "dtype", int32 / fp32 otherwise.
 *   - Calls are asynchronous on `stream` (a cudaStream_t; NULL = the legacy default
 *     stream) unless stated otherwise.
 *   - dspark_propose and dspark_verify can be captured into a CUDA graph (stream
 *     capture) and replayed; a replay reads the buffers the captured call was given, so
 *     refill them in place between replays.  Make one direct call on the device before
 *     the first capture: it does the library's one-time per-device set-up.
 *   - Argument errors detectable on the host return before anything is launched and
 *     leave every output untouched.  Problems only the device can see (an anchor
 *     outside [0, V), a bounded wait that gave up, a prepared buffer made for another
 *     head) set bits of an error word in the workspace.  Each dspark_propose call clears
 *     that word when it starts, so it describes the latest call on that workspace; read
 *     it with dspark_device_status().
 *   - dspark_last_error() returns a message for the calling thread's last failure.
 */
#ifndef DSPARK_H_
#define DSPARK_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum dspark_status {
  DSPARK_OK = 0,
  DSPARK_ERR_INVALID_ARG = 1,  /* a NULL required pointer, a bad size, a bad flag */
  DSPARK_ERR_UNSUPPORTED = 2,  /* valid in principle but outside what the kernels take */
  DSPARK_ERR_WORKSPACE = 3,    /* workspace NULL, misaligned or too small */
  DSPARK_ERR_CUDA = 4,         /* a CUDA runtime call failed (message has the details) */
  DSPARK_ERR_DEVICE = 5,       /* a kernel saw bad data (e.g. an anchor outside [0, V)) */
  DSPARK_ERR_TIMEOUT = 6       /* a bounded device-side wait gave up */
} dspark_status;

typedef enum dspark_dtype {
  DSPARK_F32 = 0,   /* fp32 operands, fp32 FMA arithmetic */
  DSPARK_BF16 = 1   /* bf16 operands, fp32 accumulation on the tensor cores */
} dspark_dtype;

/* Sizes and knobs of one call. */
typedef struct dspark_config {
  int32_t B;                  /* blocks in the batch, >= 1 */
  int32_t L_in;               /* slots per block in `hidden`, >= 1 (>= 2 for 1+N) */
  int32_t H;                  /* hidden size, >= 1 (multiple of 8 for bf16) */
  int32_t V;                  /* vocabulary: token ids are in [0, V) */
  int32_t r;                  /* Markov rank, >= 1 */
  int32_t top_k;              /* candidates kept per slot, 1 .. min(32, V_head) */
  int32_t sample_from_anchor; /* 1: anchor-first, N = L_in prediction slots reading
                                 hidden rows 0..L_in-1;
                                 0: 1+N bonus anchor, N = L_in - 1 slots reading
                                 hidden rows 1..L_in-1 (row 0 is the bonus token) */
  int32_t topk_markov;        /* 1: top-k ranks the corrected logits (the lattice
                                 candidates get the Markov bias, lucebox PR #626);
                                 0: top-k ranks the base logits */
  float conf_min;             /* truncate at the first slot with conf < conf_min;
                                 <= 0 disables truncation (n_draft = N) */
  int32_t dtype;              /* dspark_dtype of hidden, lm_head, markov_w1/w2, w_conf */
  int32_t skip_truncated;     /* 0: every slot is drafted; n_draft only marks the cut.
                                 1: adaptive block length -- the confidences and n_draft
                                 are computed first, and the slots of block b from
                                 n_draft[b] on are not drafted: draft and topk_ids read
                                 -1 there, topk_vals NaN (llama.cpp DSpark log,
                                 confidence-based draft pruning: verify reads nothing
                                 past the cut).  bf16 with a prepared head and no logits
                                 output only (DSPARK_ERR_UNSUPPORTED otherwise). */
} dspark_config;

/* The drafter head's weights (device memory, not modified). */
typedef struct dspark_head {
  const void* lm_head;        /* device [V_head, H], dtype */
  const float* lm_bias;       /* device [V_head] fp32, or NULL.  A bias <= -1e8 marks a
                                 row the draft cannot emit (never chosen while any
                                 other row is finite) */
  const int32_t* d2t;         /* device [V_head] int32, strictly increasing token ids in
                                 [0, V): row j of lm_head / column j of markov_w2 is
                                 token d2t[j].  NULL: row j is token j and V_head == V */
  int32_t V_head;             /* rows of lm_head = columns of markov_w2 (multiple of 8
                                 for bf16) */
  const void* markov_w1;      /* device [V, r], dtype; row p is gathered for prev = p */
  const void* markov_w2;      /* device [r, V_head], dtype */
  const void* w_conf;         /* device [H], dtype, or NULL (no confidence head:
                                 conf output is not written, n_draft = N) */
  float b_conf;
  const void* prepared;       /* device buffer filled by dspark_prepare_head() for these
                                 weights, or NULL.  With it (bf16 only), the chain runs
                                 the exact-bound pruned form: same results, the Markov
                                 term evaluated only where it can change them.  Without
                                 it, or when the logits output is requested, the chain
                                 evaluates every head row (dense form). */
} dspark_head;

/* Outputs of dspark_propose (device memory).  N = dspark_num_slots(cfg). */
typedef struct dspark_outputs {
  int32_t* draft;             /* required [B, N]: the greedy chain's tokens; all N slots
                                 are filled and truncation only sets n_draft, except
                                 with skip_truncated = 1 (-1 from n_draft[b] on) */
  int32_t* n_draft;           /* required [B]: truncated draft length, 0..N */
  int32_t* topk_ids;          /* [B, N, top_k] token ids by value descending, ties to
                                 the lower id; or NULL */
  float* topk_vals;           /* [B, N, top_k] the ranked logits of topk_ids; or NULL */
  float* conf;                /* [B, N] confidences; or NULL */
  float* logits;              /* [B, N, V_head] corrected logits (column j = head row
                                 j); or NULL.  Costs a full write; meant for tests */
} dspark_outputs;

/* N, the prediction slots per block (L_in or L_in - 1); 0 on invalid input. */
int32_t dspark_num_slots(const dspark_config* cfg);

/* Bytes of device workspace dspark_propose needs for this config and head; 0 on
   invalid input.  The workspace must be 256-byte aligned.  Its contents need no
   initialisation and are scratch between calls; each call clears the error word that
   dspark_device_status() reads, so that word describes the latest call. */
size_t dspark_propose_workspace_size(const dspark_config* cfg, const dspark_head* head);

/*
 * dspark_propose -- the whole proposal of one batch.
 *
 * hidden  device [B, L_in, H] dtype: the drafter's final hidden states
 * anchors device [B] int32: token 0 of every block (the dedicated anchor input of the
 *         llama.cpp squash log; in the 1+N layout the bonus token), each in [0, V)
 * conf_hidden device [B, L_in, H] dtype, or NULL: a separate input of the confidence
 *         head (lucebox PR #626, summary: a calibrated confidence export taken before
 *         the final norm).  When given, the confidence head reads it in place of
 *         `hidden`, slot for slot; the logits and the chain still read `hidden`.  NULL:
 *         the confidence head reads `hidden`.
 * out     the outputs above
 *
 * Steps, all on the device: (a) emittable-row handling from lm_bias / d2t;
 * (b) base logits of every prediction slot over the head's rows; (c) the confidence
 * head and the truncation length; (d) the Markov-corrected greedy chain over the N
 * slots, vectorised over blocks; (e) top-k per slot.  Not reentrant on one workspace:
 * calls that share a workspace must be ordered on the GPU.
 */
dspark_status dspark_propose(const dspark_config* cfg, const dspark_head* head,
                             const void* hidden, const int32_t* anchors,
                             const void* conf_hidden, const dspark_outputs* out,
                             void* workspace, size_t workspace_bytes, void* stream);

/*
 * dspark_verify -- DFlash's greedy verify/accept (unchanged by DSpark).
 *
 * draft    device [B, N] int32      n_draft device [B] int32 (values outside [0, N] are
 *                                    clamped to that range)
 * target   device [B, N + 1] int32: the target model's argmax after the anchor and after
 *          each drafted slot
 * accepted device [B] int32: a = the longest prefix j <= n_draft[b] with
 *          draft[b, 0..j-1] == target[b, 0..j-1]
 * bonus    device [B] int32: target[b, a]
 * emitted  device [B, N + 1] int32 or NULL: draft[b, 0..a-1], then the bonus token, then
 *          -1; with greedy decoding this equals the target's own argmax sequence.
 */
dspark_status dspark_verify(int32_t B, int32_t N, const int32_t* draft,
                            const int32_t* n_draft, const int32_t* target,
                            int32_t* accepted, int32_t* bonus, int32_t* emitted,
                            void* stream);

/*
 * dspark_tree_verify -- greedy verify of the top-k candidate lattice (the tree consumer
 * of the per-slot candidates; lucebox PR #626, description: the DDTree's candidate
 * top-k gets the Markov bias; onnxruntime-genai PR #2490, DFlash 2 / DSpark builder
 * commits: the runtime walks the drafter's candidate lattice greedily).
 *
 * The tree is the whole lattice: every candidate of slot i is a child of every candidate
 * of slot i - 1, down to depth n_draft[b] (the pages define no other construction).  A
 * greedy target accepts the child equal to its argmax after the accepted prefix; as that
 * prefix is always the target's own tokens, the argmax at depth i is target[b, i].
 *
 * topk_ids device [B, N, top_k] int32: the candidates of dspark_propose (topk_ids)
 * n_draft  device [B] int32 (clamped to [0, N])
 * target   device [B, N + 1] int32: the target model's argmax tokens along its own
 *          greedy continuation
 * accepted device [B] int32: a = the largest j <= n_draft[b] such that target[b, i] is
 *          among topk_ids[b, i, :] for every i < j
 * bonus    device [B] int32: target[b, a]
 * emitted  device [B, N + 1] int32 or NULL: target[b, 0..a], then -1 (greedy lossless)
 * path     device [B, N] int32 or NULL: for i < a the rank q with
 *          topk_ids[b, i, q] == target[b, i] (the first such q), -1 from a on
 *
 * With top_k = 1 it equals dspark_verify on the greedy draft.  Host-detectable errors
 * (sizes, NULL required pointers) return before any launch.
 */
dspark_status dspark_tree_verify(int32_t B, int32_t N, int32_t top_k,
                                 const int32_t* topk_ids, const int32_t* n_draft,
                                 const int32_t* target, int32_t* accepted, int32_t* bonus,
                                 int32_t* emitted, int32_t* path, void* stream);

/* Bytes of the buffer dspark_prepare_head() fills for this head (bf16 only; 0 on invalid
   input or fp32).  Layout: a 256-byte header recording what the buffer was prepared for
   (V, V_head, r and the markov_w1 / markov_w2 addresses), markov_w2 transposed
   [round_up(V_head, 128)][r] bf16, the fp32 Euclidean norm of every markov_w2 column,
   their maximum over each 128-row tile, and the largest Euclidean norm of a markov_w1
   row.
   A head in the bias form of a reduced draft vocabulary (lm_bias given, d2t NULL,
   V_head == V, and 1 <= n_emit < V rows with bias > -1e8) is prepared in its compact
   form instead (llama.cpp PR #26275, the reduced draft vocabulary as an expanded head
   and as a d2t map): a 256-byte header (V, H, r, n_emit, the padded row count
   n_pad = round_up(n_emit, 8) and the lm_head, lm_bias, markov_w1, markov_w2
   addresses), the emittable rows in increasing order [n_pad] int32 (padded with copies
   of the last), per-chunk counts, their lm_head rows [n_pad][H] bf16, markov_w2
   columns [r][n_pad] bf16 and biases [n_pad] fp32 (padding rows: zero weights, bias
   -1e30), then the layout above for that compact head.  To size it, this call counts
   the emittable rows on the device and waits for the count (current device, default
   stream). */
size_t dspark_prepare_head_size(const dspark_config* cfg, const dspark_head* head);

/*
 * dspark_prepare_head -- one-time preparation of a head's Markov weights for the pruned
 * chain (the weights are constant across calls, like a converted checkpoint).
 *
 * prepared  device buffer of dspark_prepare_head_size() bytes, 256-byte aligned, owned by
 *           the caller; pass it as head->prepared to later dspark_propose calls.  It must
 *           be prepared again whenever markov_w1 or markov_w2 changes, in place or by
 *           address: the pruned chain's bounds come from both (the column norms of
 *           markov_w2 and the largest row norm of markov_w1), and stale bounds can drop
 *           the true argmax or top-k rows without any error.  head->prepared itself is
 *           ignored here.
 *
 * A dspark_propose call whose V, V_head, r, markov_w1 or markov_w2 address differ from
 * those the buffer was prepared for reads nothing past the buffer's header: it drafts
 * nothing and dspark_device_status() then reports DSPARK_ERR_DEVICE with that reason.
 * (Contents changed in place at the same addresses cannot be detected; re-prepare.)
 *
 * Bias form (see dspark_prepare_head_size): the emittable rows are counted (this call
 * waits for the count on `stream`), found and gathered on the device into the compact
 * head; later dspark_propose calls with this head run on those rows only (the GEMM, the
 * chain and the top-k), with the same outputs as over the full head.  That holds while
 * top_k <= n_emit and the logits output is not requested; otherwise a call uses the
 * full head (the dense chain over every row).  It must be prepared again when lm_head or
 * lm_bias changes too.  A process that did not prepare the buffer itself reads its
 * header once, synchronously, on first use: make that first call outside stream
 * capture.
 */
dspark_status dspark_prepare_head(const dspark_config* cfg, const dspark_head* head,
                                  void* prepared, size_t prepared_bytes, void* stream);

/* Stages of dspark_propose, in launch order, for dspark_propose_timed(). */
enum {
  DSPARK_STAGE_CONF = 0,    /* confidence head + truncation length */
  DSPARK_STAGE_LOGITS = 1,  /* base logits of every prediction slot (the lm_head GEMM) */
  DSPARK_STAGE_CHAIN = 2,   /* Markov-corrected greedy chain and per-slot candidates */
  DSPARK_STAGE_TOPK = 3,    /* final top-k ordering */
  DSPARK_NUM_STAGES = 4
};

/* dspark_propose that also records events[s] (cudaEvent_t, created by the caller) on
   `stream` as stage s begins, and events[DSPARK_NUM_STAGES] after the last stage.
   A stage with no kernel for this config records its event right before the next
   one's.  The work done is identical to dspark_propose's. */
dspark_status dspark_propose_timed(const dspark_config* cfg, const dspark_head* head,
                                   const void* hidden, const int32_t* anchors,
                                   const void* conf_hidden, const dspark_outputs* out,
                                   void* workspace, size_t workspace_bytes, void* stream,
                                   void* const* events);

/* Number of kernels one dspark_propose call launches for this config, head and set of
   requested outputs, the kernel that resets the workspace's control block included; -1
   on invalid input. */
int32_t dspark_propose_kernel_count(const dspark_config* cfg, const dspark_head* head,
                                    const dspark_outputs* out);

/* Bytes of device workspace dspark_step_host needs: dspark_propose's plus staging for
   the host inputs and outputs.  256-byte aligned; 0 on invalid input. */
size_t dspark_step_host_workspace_size(const dspark_config* cfg, const dspark_head* head);

/*
 * dspark_step_host -- one draft step from and to HOST memory: copies hidden, anchors
 * and target in, runs dspark_propose and dspark_verify, copies the results out.
 *
 * hidden_h  host [B, L_in, H] dtype      anchors_h host [B] int32
 * conf_hidden_h host [B, L_in, H] dtype, or NULL: the confidence head's separate input
 *           (see dspark_propose); copied in like hidden_h
 * target_h  host [B, N + 1] int32 (the target's argmax tokens for the verify step)
 * draft_h   host [B, N] int32            n_draft_h host [B] int32
 * accepted_h, bonus_h host [B] int32
 * topk_ids_h / topk_vals_h host [B, N, top_k] or NULL
 *
 * hidden_h is copied with cudaMemcpyAsync on `stream`.  The other buffers are read or
 * written by the kernels in place when they are page-locked host memory the device can
 * address (cudaHostAlloc, or cudaHostRegister with a mapping; cudaPointerGetAttributes
 * reports them as host memory with a device pointer); otherwise they too are copied
 * through workspace staging.  Page-locked buffers throughout are the fast case.  The
 * call returns once everything is queued: synchronise `stream` before reading the
 * outputs.
 */
dspark_status dspark_step_host(const dspark_config* cfg, const dspark_head* head,
                               const void* hidden_h, const int32_t* anchors_h,
                               const void* conf_hidden_h,
                               const int32_t* target_h, int32_t* draft_h,
                               int32_t* n_draft_h, int32_t* accepted_h, int32_t* bonus_h,
                               int32_t* topk_ids_h, float* topk_vals_h,
                               void* workspace, size_t workspace_bytes, void* stream);

/*
 * dspark_propose_noalloc -- dspark_propose for callers that cannot allocate device memory.
 *
 * (No counterpart on the pages: an interface addition of this library.)  Some callers
 * cannot call cudaMalloc or any allocating routine: code that runs inside a host
 * framework owning every allocation, allocator-free plugins, or callers that must not
 * touch the allocator while the device is in use elsewhere.  This entry point takes the
 * same arguments as dspark_propose minus the workspace: its scratch is a fixed 16 MiB
 * array of device memory built into the library, which every GPU that loads the library
 * holds until the process exits.  It allocates nothing itself.
 *
 *   - Calls whose dspark_propose_workspace_size() exceeds 16 MiB return
 *     DSPARK_ERR_WORKSPACE before launching anything (small batches and vocabularies
 *     only; larger ones need dspark_propose and a caller workspace).
 *   - The scratch's device address belongs to the CUDA context current at the call.  A
 *     call that is not being captured looks it up (with the device current) and keeps it
 *     for that context; a call made while `stream` is capturing uses the address kept
 *     for the current context and is refused if there is none.  So make one call on each
 *     device (and again after a cudaDeviceReset) before any stream capture.
 *   - Every call on a device shares the one scratch array, which keeps the contents the
 *     last call left (each call clears what has to start at zero).  Calls that overlap on
 *     the GPU -- on different streams, or from different host threads without ordering --
 *     race on it and give wrong results: order them on one stream.
 *   - Problems only the device can see (an anchor outside [0, V), a bounded wait that
 *     gave up) are recorded in the scratch's error word; read them with
 *     dspark_noalloc_device_status() before the next call on the device clears them.
 */
dspark_status dspark_propose_noalloc(const dspark_config* cfg, const dspark_head* head,
                                     const void* hidden, const int32_t* anchors,
                                     const void* conf_hidden, const dspark_outputs* out,
                                     void* stream);

/* Synchronises `stream`, reads the device error word of a workspace used by
   dspark_propose (it describes the latest call on that workspace), and clears it.
   DSPARK_OK when no kernel flagged anything; DSPARK_ERR_DEVICE or DSPARK_ERR_TIMEOUT
   otherwise, with the reason in dspark_last_error(). */
dspark_status dspark_device_status(void* workspace, void* stream);

/* Synchronises `stream` and reads three counters of the latest dspark_propose call on
   `workspace` (they restart at zero with every call).  Instrumentation of the cost of
   the two chain forms; the method on the pages has no counterpart.  Any output pointer
   may be NULL.
     on_the_fly:     (slot, block) pairs the exact-bound pruned chain could not look up
                     in its tables and evaluated on the fly (loose Cauchy-Schwarz bounds:
                     too many candidate rows or possible previous rows);
     every_row:      of those, the pairs whose candidate list overflowed, so that every
                     head row was evaluated;
     dense_overflow: (slot, block) pairs of the dense chain whose top-k candidate lists
                     overflowed (massive ties) and were recomputed over every head row.
   DSPARK_ERR_INVALID_ARG for a NULL workspace; DSPARK_ERR_CUDA if the read fails. */
dspark_status dspark_pass_stats(void* workspace, void* stream, int32_t* on_the_fly,
                                int32_t* every_row, int32_t* dense_overflow);

/* dspark_device_status() for the built-in scratch of dspark_propose_noalloc() on the
   current device: synchronises `stream`, reads the error word of the latest no-alloc call
   on this device and clears it.  (No counterpart on the pages, like the entry point it
   serves.)  Call it on the stream of that call, outside stream capture. */
dspark_status dspark_noalloc_device_status(void* stream);

/*
 * dspark_wait_selftest -- makes one bounded device-side wait run out, on purpose.
 *
 * (No counterpart on the pages: a test hook of this library's failure detection.)  Every
 * wait inside the library's kernels (a pipeline stage waiting for its copy, the MMA
 * waiting for a free accumulator, a grid barrier) gives up after a clock budget of about
 * one second, raises the timeout bit of the workspace's error word and lets the kernel
 * return, so that the CUDA context stays usable.  This call launches one small kernel that
 * waits, through the same bounded-wait routine, on a barrier that nothing ever completes.
 *
 *   workspace        device, >= 256 bytes, 256-byte aligned; only its first word (the
 *                    error word) is written.  A dspark_propose workspace qualifies.
 *   budget_cycles    SM clock cycles to wait before giving up, in [1, 2e9].
 *   pre_abort        1 = the abort flag is already set, so the wait gives up at its first
 *                    check; 0 = it gives up when the budget runs out.
 *   stream           the CUDA stream (cudaStream_t), may be NULL.
 *
 * Host-detectable errors (above) return before any launch.  Afterwards,
 * dspark_device_status() on the same workspace reports DSPARK_ERR_TIMEOUT and clears it.
 */
dspark_status dspark_wait_selftest(void* workspace, size_t workspace_bytes,
                                   int64_t budget_cycles, int32_t pre_abort, void* stream);

/* ---------------------------------------------------------------------------------
 * Training the head.  dspark_block_norm makes the head's inputs from a drafter block's
 * output, dspark_head_loss scores teacher-forced slots and gives the gradients of
 * everything their logits are made of, dspark_block_norm_backward carries them through
 * the norm, and dspark_clip_grads bounds the step.  Every array is aligned to its elements
 * at least; a call refuses one that is not.  (The pages describe the head these
 * calls train, not its training: the operators are this library's own.)
 * ------------------------------------------------------------------------------- */

typedef enum dspark_reduction {
  DSPARK_LOSS_SUM = 0,   /* total = loss_scale * sum_t w_t loss_t */
  DSPARK_LOSS_MEAN = 1   /* that over the sum of w_t of the rows that carry a loss */
} dspark_reduction;

/* Sizes and knobs of dspark_head_loss. */
typedef struct dspark_loss_config {
  int32_t T;             /* rows (slots of all blocks), 1 .. 2^20 */
  int32_t H;             /* hidden size, 1 .. 2^16 (multiple of 8 for bf16) */
  int32_t V;             /* vocabulary, at most 2^24: token ids are in [0, V) */
  int32_t r;             /* Markov rank, 1 .. 512; 0: a head without the Markov term */
  int32_t dtype;         /* dspark_dtype of hidden, the head's weights and the gradients */
  int32_t reduction;     /* dspark_reduction */
  int32_t vocab_pieces;  /* the gradients are computed over the vocabulary in this many
                            pieces, >= 1; 0: chosen by size.  One piece keeps the
                            softmax numerators of the whole vocabulary in the workspace
                            (2 bytes each for bf16, 4 for fp32); with more, only a piece's
                            are held, and each piece's logits are computed a second time.
                            At most ceil(V_head / 256) pieces are made.  No effect when no
                            gradient is asked for: nothing is kept then.  Besides, the rows
                            of [hidden | markov_w1[prev]] are held once in dtype and, for
                            d_hidden or d_markov_w1, in fp32 at least once (in bf16 up to
                            512 MB of partial sums where once takes less). */
  float loss_scale;      /* factor of the total and of every gradient; finite */
} dspark_loss_config;

/* Outputs of dspark_head_loss (device memory).  Gradients are of `total`, have the
   config's dtype and are overwritten, not added to. */
typedef struct dspark_loss_outputs {
  float* loss;           /* required [T]: the negative log-likelihood of each row's label;
                            0 for a row that carries no loss */
  float* total;          /* required [1]; 0 when no row carries a loss */
  int32_t* n_rows;       /* [1] rows that carry a loss; or NULL */
  void* d_hidden;        /* [T, H] (0 for rows without a loss); or NULL */
  void* d_lm_head;       /* [V_head, H]; or NULL (a frozen lm_head) */
  void* d_markov_w1;     /* [V, r]; or NULL */
  void* d_markov_w2;     /* [r, V_head]; or NULL */
} dspark_loss_outputs;

/* Bytes of device workspace dspark_head_loss needs for this config, head and set of
   requested gradients; 0 on invalid input.  256-byte aligned; needs no initialisation. */
size_t dspark_head_loss_workspace_size(const dspark_loss_config* cfg,
                                       const dspark_head* head,
                                       const dspark_loss_outputs* out);

/*
 * dspark_head_loss -- softmax cross entropy of the Markov-corrected logits over the
 * head's vocabulary, with its gradients:
 *
 *   z[t, v] = hidden[t] . lm_head[v] + lm_bias[v] + markov_w1[prev[t]] . markov_w2[:, v]
 *   loss[t] = log sum_v exp z[t, v] - z[t, label[t]]
 *
 * hidden  device [T, H] dtype.  Rows of blocks [B, L_in, H] are passed as T = B * L_in
 *         (in the 1+N layout with a negative label at slot 0)
 * prev    device [T] int32: the token before each slot, in [0, V); NULL when r = 0
 * labels  device [T] int32: the target token of each slot.  A negative label, or a token
 *         the head cannot emit (absent from d2t, or masked by lm_bias <= -1e8), marks a
 *         row without a loss: nothing of that row is read into any result
 * weights device [T] fp32 >= 0, or NULL (all 1): w_t
 *
 * The head's lm_head, lm_bias, d2t, V_head, markov_w1 and markov_w2 are read (the last
 * two NULL when r = 0); w_conf, b_conf and prepared are not.  Masked head rows take no
 * part: their probability is 0, their gradients are 0, and their weights are not read.
 * lm_bias itself gets no gradient.  For bf16, lm_head, markov_w2 and the gradients of the
 * weights are 16-byte aligned.  A label at or above V, or a prev outside [0, V) on a
 * row with a loss, drops the row and raises the error word (dspark_device_status).
 *
 * bf16: products on the tensor cores with fp32 accumulation; the softmax statistics,
 * losses and sums are fp32.  With the vocabulary in one piece the logits are kept as 16-bit
 * distances from a maximum, in steps of 1/896: a probability in the gradient is off by at
 * most 0.06% (with several pieces they are computed again, and are not).  The gradient of the
 * logits is rounded to bf16 before the gradient products; d_hidden and d_markov_w1 get back
 * what the label's entry lost, and when at most 64 of at most 128 rows carry a loss every
 * entry's rounding is carried along.  Each gradient is rounded once more on output.
 *
 * A row whose logits are not all numbers (or are +infinity) has NaN in its loss and its
 * gradients, and so have the total and the weights' gradients.  No atomics decide an order of
 * summation: the same call gives the same bits.  d_markov_w1 compares every row's prev with
 * the earlier ones': with T^2 (0.2 s at 2^20 rows, all different).  Not reentrant on one
 * workspace.  Can be captured into a CUDA graph.
 */
dspark_status dspark_head_loss(const dspark_loss_config* cfg, const dspark_head* head,
                               const void* hidden, const int32_t* prev,
                               const int32_t* labels, const float* weights,
                               const dspark_loss_outputs* out, void* workspace,
                               size_t workspace_bytes, void* stream);

/* What a teacher says of every row: its listed tokens (dspark_top_logits makes such a list). */
typedef struct dspark_teacher {
  const int32_t* ids;    /* device [T, k]: token ids; a negative one is absent */
  const float* logits;   /* device [T, k] fp32: their logits; -infinity: absent, whatever the id */
  const float* lse;      /* device [T] fp32: the log-sum-exp of scale * logits over the
                            teacher's whole vocabulary, or NULL: over the listed tokens */
  int32_t k;             /* listed tokens a row, 1 .. 256 */
  float scale;           /* factor of the teacher's logits (1 / temperature); finite */
} dspark_teacher;

/* Bytes of device workspace dspark_distill_loss needs: dspark_head_loss's, and about 12 bytes
   for each listed token; 0 on invalid input.  256-byte aligned; needs no initialisation. */
size_t dspark_distill_loss_workspace_size(const dspark_loss_config* cfg,
                                          const dspark_head* head,
                                          const dspark_teacher* teacher,
                                          const dspark_loss_outputs* out);

/*
 * dspark_distill_loss -- the divergence of the head from a teacher's listed tokens, with its
 * gradients.  With z as for dspark_head_loss and log p = z - log sum_v exp z:
 *
 *   log q[t, k] = scale * logits[t, k] - L[t]
 *   loss[t]     = sum_k q[t, k] (log q[t, k] - log p[t, ids[t, k]])
 *
 * Listed tokens that the head cannot emit (absent from d2t, or masked by lm_bias) are left out.
 * L is the log-sum-exp of the ones that are not, so that their q sum to 1; or, with
 * teacher->lse, that of the teacher's whole vocabulary: q are then the teacher's own
 * probabilities, and the rest of them takes no part.  A row with no token left carries no loss:
 * nothing of it is read into any result.  A token at or above V, or listed twice in a row, or
 * a prev outside [0, V) on a row with a loss, drops the row and raises the error word.
 *
 * config, head, hidden, prev, weights, outputs (n_rows: rows with a loss), precision, workspace
 * and capture are as for dspark_head_loss.  The listed tokens' logits are taken by fp32 dot
 * products, and their entries of the logits' gradient by themselves, each off by what its log q
 * and log p are; the most probable listed token's by as little of themselves where both are
 * near 0 (log q: without teacher->lse), so that a loss near 0 keeps its gradient.  In bf16 these
 * entries are rounded to 8 bits before the products, with what the most probable listed token's
 * lost given back to d_hidden and d_markov_w1.
 */
dspark_status dspark_distill_loss(const dspark_loss_config* cfg, const dspark_head* head,
                                  const void* hidden, const int32_t* prev,
                                  const dspark_teacher* teacher, const float* weights,
                                  const dspark_loss_outputs* out, void* workspace,
                                  size_t workspace_bytes, void* stream);

/* Sizes and knobs of dspark_block_norm and its gradient. */
typedef struct dspark_norm_config {
  int32_t T;             /* rows (tokens), 1 .. 2^30 */
  int32_t H;             /* features, 1 .. 8192 */
  int32_t dtype;         /* dspark_dtype of every tensor */
  int32_t gate_span;     /* consecutive rows that share one gate row, >= 1; T or more: all
                            rows share one */
  float eps;             /* > 0 */
  float residual_scale;  /* s below; finite */
  float weight_offset;   /* added to the norm weights (1 for weights stored about 0) */
} dspark_norm_config;

/*
 * dspark_block_norm -- the norms around the end of a drafter block:
 *
 *   u = y / rms(y) * (weight_offset + w_post)       (u = y when w_post is NULL)
 *   x_out = x + s * gate * u                        (gate = 1 when NULL)
 *   h = x_out / rms(x_out) * (weight_offset + w_pre),   rms(a) = sqrt(mean(a^2) + eps)
 *
 * x, y    device [T, H]: the residual stream and the block's output.  y NULL: x_out = x
 * gate    device [ceil(T / gate_span), H] or NULL
 * w_post, w_pre device [H]; w_pre is required
 * x_out   device [T, H] or NULL: the stream after the block (the head's conf_hidden);
 *         may be x itself
 * h       device [T, H]: the head's hidden; may be y itself
 *
 * Arithmetic in fp32; h is computed from x_out before its rounding.
 */
dspark_status dspark_block_norm(const dspark_norm_config* cfg, const void* x, const void* y,
                                const void* gate, const void* w_post, const void* w_pre,
                                void* x_out, void* h, void* stream);

/* Bytes of device workspace dspark_block_norm_backward needs; 0 on invalid input. */
size_t dspark_block_norm_workspace_size(const dspark_norm_config* cfg);

/*
 * dspark_block_norm_backward -- the gradients of dspark_block_norm, from its inputs:
 *
 * d_h     device [T, H]: the gradient of h       d_x_out device [T, H] or NULL: of x_out
 * d_x     device [T, H]                          d_y     device [T, H]; NULL with y
 * d_gate  device, gate's shape (summed over the rows that share a gate row); NULL with gate
 * d_w_post, d_w_pre device [H]: summed over the rows; d_w_post NULL with w_post
 *
 * Every gradient is overwritten, and must not overlap an input or another one.  The
 * sums over rows are taken in a fixed order.
 */
dspark_status dspark_block_norm_backward(const dspark_norm_config* cfg, const void* x,
                                         const void* y, const void* gate,
                                         const void* w_post, const void* w_pre,
                                         const void* d_h, const void* d_x_out, void* d_x,
                                         void* d_y, void* d_gate, void* d_w_post,
                                         void* d_w_pre, void* workspace,
                                         size_t workspace_bytes, void* stream);

/* One gradient of dspark_clip_grads. */
typedef struct dspark_grad {
  const void* in;        /* device [n] */
  void* out;             /* device [n]: in itself, or memory that overlaps no gradient */
  int64_t n;             /* elements, >= 0 */
  int32_t dtype;         /* dspark_dtype */
} dspark_grad;

/* Bytes of device workspace dspark_clip_grads needs for `count` gradients; 0 on invalid
   input. */
size_t dspark_clip_grads_workspace_size(int32_t count, const dspark_grad* grads);

/*
 * dspark_clip_grads -- the global norm of a list of gradients, and the clipped list:
 *
 *   norm = sqrt(sum over all elements of in^2),   out = in * min(1, max_norm / (norm + 1e-6))
 *
 * grads    host [count]: read during the call only
 * max_norm >= 0
 * norm     device [1] fp32
 *
 * Squares are summed in fp32, in a fixed order.  When the norm is not finite (or its
 * square leaves fp32's range), out = in: the norm says so, and the caller skips the step.
 * Where out is in and the factor is 1 nothing is written.
 */
dspark_status dspark_clip_grads(int32_t count, const dspark_grad* grads, float max_norm,
                                float* norm, void* workspace, size_t workspace_bytes,
                                void* stream);

/* ---------------------------------------------------------------------------------
 * Tokens in and out: the drafter's input rows and their gradient, and the tokens of a
 * target's logits.  dspark_sample draws the tokens that dspark_verify takes as `target`
 * (a draft is then accepted exactly where it is what the target would have drawn, so the
 * output is the target's own distribution); dspark_top_logits lists what a teacher says.
 * (The pages verify greedily: the operators are this library's own.)
 * ------------------------------------------------------------------------------- */

/* Sizes and settings of dspark_sample. */
typedef struct dspark_sample_config {
  int32_t T;             /* rows, 1 .. 2^20 */
  int32_t V;             /* tokens of a row, 1 .. 2^24 */
  int64_t ld;            /* elements from a row of logits to the next, >= V */
  int32_t dtype;         /* dspark_dtype of the logits */
  int32_t top_k;         /* <= 0: off */
  float temperature;     /* <= 0: the largest logit, whatever the filters say */
  float top_p;           /* >= 1: off; <= 0: the largest */
  float min_p;           /* <= 0: off; >= 1: those equal to the largest */
} dspark_sample_config;

/* Settings of single rows (device arrays [T]), each in its config value's place; or NULL. */
typedef struct dspark_sample_rows {
  const int32_t* top_k;
  const float* temperature;
  const float* top_p;
  const float* min_p;
} dspark_sample_rows;

/*
 * dspark_sample -- a token of every row of logits, by one given uniform number each.
 *
 * A row's order is by falling logit, equal ones by rising id.  With weights
 * w = exp((z - max) / temperature), one after the other:
 *   top_k  keeps the first top_k tokens of the order
 *   top_p  keeps its shortest prefix whose weight is at least top_p of the weight kept so far
 *   min_p  keeps the tokens with w >= min_p
 * and the token is the first by id for which the weight of the kept tokens up to it exceeds
 * uniform times the weight of all kept ones.
 *
 * logits  device [T, ld] dtype.  A logit of -infinity or NaN is never drawn; a row without any
 *         other has token -1 and log-probability -infinity.  With +infinity in a row, only those
 *         are drawn, all alike
 * rows    host struct of device arrays, or NULL.  A row's NaN setting: temperature as 0, top_p
 *         and min_p off
 * uniform device [T] fp32 in [0, 1) (below, or NaN: 0; above: the last kept one
 *         that has a weight)
 * tokens  device [T] int32
 * logp    device [T] fp32 or NULL: the token's log-probability among the kept ones
 *
 * Weights are cut to whole multiples of 2^-S of the largest, S = 62 - ceil(log2 V) (44 for
 * 151936 tokens), and off by at most 2^-27 of themselves besides.  The token is that of their exact
 * sums, whatever the call's other rows; the mass that logp is made of may be V of those units too
 * large.  tokens and logp overlap nothing else.  Needs no workspace; calls may run at once.  Can be
 * captured into a CUDA graph.
 */
dspark_status dspark_sample(const dspark_sample_config* cfg, const dspark_sample_rows* rows,
                            const void* logits, const float* uniform, int32_t* tokens,
                            float* logp, void* stream);

/*
 * dspark_top_logits -- the k largest logits of every row, and the row's log-sum-exp.
 *
 * logits  device [T, ld] dtype, T in 1 .. 2^20, V in 1 .. 2^24, ld >= V
 * k       1 .. min(V, 1024)
 * ids     device [T, k] int32, values device [T, k] fp32: by falling logit, equal ones by rising
 *         id.  -infinity and NaN are not listed: where fewer than k others are left, -1 and
 *         -infinity stand (absent, for dspark_distill_loss)
 * lse     device [T] fp32 or NULL: log sum exp of the row (NaN left out), off by at most 2^-17 and
 *         2^-22 of itself whatever V is (the roundings' sum; as a rule some 1e-7)
 *
 * The outputs overlap nothing else.  Needs no workspace; calls may run at once.  Can be captured
 * into a CUDA graph.
 */
dspark_status dspark_top_logits(int32_t T, int32_t V, int64_t ld, int32_t dtype, int32_t k,
                                const void* logits, int32_t* ids, float* values, float* lse,
                                void* stream);

/* Sizes and settings of dspark_embed and its gradient. */
typedef struct dspark_embed_config {
  int32_t T;             /* rows (tokens), 1 .. 2^20 */
  int32_t V;             /* rows of the table, 1 .. 2^24 */
  int32_t H;             /* features, 1 .. 2^16 */
  int32_t dtype;         /* dspark_dtype of every tensor */
  float scale;           /* finite */
} dspark_embed_config;

/*
 * dspark_embed -- out[t] = scale * table[ids[t]].
 *
 * table   device [V, H]      ids  device [T] int32; a row whose id is outside [0, V) is zeros
 * out     device [T, H]: the fp32 product, in bf16 rounded to it; overlaps nothing else
 */
dspark_status dspark_embed(const dspark_embed_config* cfg, const void* table,
                           const int32_t* ids, void* out, void* stream);

/* Bytes of device workspace dspark_embed_backward needs; 0 on invalid input.  256-byte
   aligned; needs no initialisation. */
size_t dspark_embed_workspace_size(const dspark_embed_config* cfg);

/*
 * dspark_embed_backward -- d_table[v] = add[v] + scale * sum of d_out[t] over ids[t] = v.
 *
 * ids     device [T] int32.  A negative id is no token; one at or above V is none either, and
 *         raises the error word (dspark_device_status)
 * d_out   device [T, H]
 * add     device [V, H] or NULL (zeros): what the gradient is added to, as the gradient of a
 *         tied lm_head.  May be d_table itself: then only rows that occur are read and written
 * d_table device [V, H], overwritten; overlaps nothing else
 *
 * Sums are fp32, over a token's rows in their order, in parts of at most max(32, ceil(T / 2432))
 * rows that are joined with their rounding errors; scale times the sum (with add: fused with it) is
 * rounded to fp32, and in bf16 that to bf16.  The same call gives the same bits.  Not reentrant on
 * one workspace.  Can be captured into a CUDA graph.
 */
dspark_status dspark_embed_backward(const dspark_embed_config* cfg, const int32_t* ids,
                                    const void* d_out, const void* add, void* d_table,
                                    void* workspace, size_t workspace_bytes, void* stream);

/* Static description of a status code. */
const char* dspark_status_string(int32_t status);

/* Message describing the calling thread's most recent failed call ("" if none). */
const char* dspark_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* DSPARK_H_ */

/*
 * libtpoverlap -- tensor-parallel linear layers whose GEMM overlaps the movement
 * of its operand or result chunks, on one GB300 (sm_103a).
 *
 * The tp "ranks" of a tensor-parallel group are simulated as tp chunk buffers in
 * one GPU's memory.  Three operations are provided:
 *
 *   AG+GEMM   Y = allgather_rows(X_0 .. X_tp-1) . W^T, rows in rank order.
 *             TransformerEngine issue "curious about atomic_gemm_overlap_ag",
 *             listing of CommOverlapP2PBase::atomic_gemm_overlap_ag: a ring of
 *             chunk send/recv steps fills the gathered buffer, a per-chunk
 *             producer counter marks each chunk ready, and one GEMM consumes
 *             the chunks as their counters flip.
 *   GEMM+RS   Y = sum_r X_r . W_r^T, rank b receives row block b.
 *             TransformerEngine PR "Comm+GEMM overlap API updated to support
 *             cuBlasMp backend", sequence diagram, GEMM + reduce-scatter path.
 *   GEMM+AR   Y = sum_r X_r . W_r^T in full, produced in row chunks.
 *             nvFuser PR "Reference implementation for Linear+Allreduce with
 *             overlapping": row-parallel linear, per-chunk matmul then
 *             all-reduce SUM.
 *
 * Conventions (TN layout, as the listing's transa/transb and m/n naming):
 *   n  rows of Y (tokens), m  columns of Y (output features),
 *   k  the GLOBAL contraction length.  For AG every X_r is [n/tp, k]; for RS and
 *      AR every rank holds a K-slice, X_r [n, k/tp] and W_r [m, k/tp].
 *   All matrices are dense row-major; X and W are "K-major" (the contraction
 *   index is contiguous); Y is always bf16.
 *   bf16 buffers hold IEEE bfloat16, e4m3 buffers OCP FP8 E4M3 codes.
 *
 * Ownership: the caller owns every X, W, Y buffer and the stream.  The context
 * owns the staging buffer (the gathered X), the per-chunk counters, the device
 * error word and the trace buffer; all are allocated by tpo_ctx_create and
 * nothing is allocated by the per-call entry points.
 *
 * Calls are stream-ordered and asynchronous: they validate their arguments on
 * the host, enqueue work on `stream` (a cudaStream_t passed as void*, NULL for
 * the legacy default stream) and return.  Inputs must stay valid until the
 * stream reaches the call.  Argument errors are reported synchronously before
 * anything is enqueued.  A device-side failure (a bounded wait that ran out) is
 * recorded in the context's error word and reported by the next
 * tpo_sync_status; until then the word is sticky and later calls on the
 * context abort early.  Every entry point sets a thread-local message readable
 * through tpo_last_error when it fails.
 *
 * A context is not thread-safe: calls on one context must come from one host
 * thread at a time.  Calls that overlap on the GPU (different streams) must use
 * different contexts.
 */
#ifndef TPOVERLAP_H
#define TPOVERLAP_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct tpo_ctx tpo_ctx; /* opaque */

/* Input element type (Y is always bf16).  TPO_F32 is a type of tpo_layer_norm
 * and tpo_layer_norm_bwd only. */
typedef enum { TPO_BF16 = 0, TPO_FP8_E4M3 = 1, TPO_F32 = 2 } tpo_dtype;

typedef enum {
  TPO_OK = 0,
  TPO_ERR_INVALID_ARG = 1, /* bad pointer, size, alignment or option */
  TPO_ERR_UNSUPPORTED = 2, /* valid request outside what the library supports */
  TPO_ERR_CUDA = 3,        /* a CUDA runtime/driver call failed */
  TPO_ERR_TIMEOUT = 4,     /* a bounded device-side wait ran out */
  TPO_ERR_OOM = 5          /* device allocation failed in tpo_ctx_create */
} tpo_status;

/* Operation limits of the library. */
#define TPO_MAX_TP 16
#define TPO_MAX_ROW_CHUNKS 64
#define TPO_BLOCK_M 128 /* rows of one output tile */
#define TPO_BLOCK_N 256 /* columns of one output tile */
/* Sizes need not be multiples of the tile: the last tile of a slot, block or
 * part loads zeros past its edge and stores only the rows and columns that
 * exist.  Row pitches must be multiples of 16 bytes. */

/*
 * Create a context for one problem size on the current CUDA device.
 *   tp     number of simulated ranks, 1..16
 *   n      rows of Y, a multiple of tp (every rank holds n/tp rows)
 *   k      global contraction length: a multiple of 8 (bf16) or 16 (e4m3);
 *          for RS/AR also k % tp == 0 and k/tp a multiple of 8 (16 for e4m3)
 *   m      columns of Y, a multiple of 8
 *   dtype  a tpo_dtype value
 * Allocates the staging buffer (n*k elements), counters, error word and trace
 * buffer on the current device.  Returns NULL on any error (no half-built
 * context is ever returned); tpo_last_error says why.
 * The signature follows the context-handle pattern of the cuBLASMp backend in
 * TransformerEngine PR "Comm+GEMM overlap API updated to support cuBlasMp
 * backend" (nvte_comm_gemm_ctx_create ... nvte_comm_gemm_ctx_destroy).
 */
tpo_ctx* tpo_ctx_create(int tp, int64_t n, int64_t k, int64_t m, int dtype);

/* Release everything the context owns (synchronises with its pending work).
 * tpo_ctx_destroy(NULL) is a no-op returning TPO_OK. */
tpo_status tpo_ctx_destroy(tpo_ctx* ctx);

/*
 * AG+GEMM: Y[n, m] = gather(X_0..X_tp-1)[n, k] . W[m, k]^T, Y rows in rank order.
 *   x      host array of tp device pointers; x[r] is rank r's chunk [n/tp, k]
 *   w      device pointer, [m, k]
 *   y      device pointer, [n, m] bf16
 *   d_scale_inv_x, d_scale_inv_w
 *          e4m3 contexts: device pointers to one fp32 each (the per-tensor
 *          scale_inv of all X_r together and of W); the product is multiplied
 *          by both in fp32 before rounding.  bf16 contexts: must be NULL.
 *   stream cudaStream_t
 * Semantics (listing of atomic_gemm_overlap_ag): the observer rank `self_rank`
 * (option, default 0) holds its own chunk and receives the others in ring
 * order self-1, self-2, ... (mod tp).  A producer role copies each arriving
 * chunk into its rank-order slot of the staging buffer and publishes the
 * slot's counter with release semantics; the GEMM role acquire-waits on that
 * counter before its first tensor-memory load of the slot.  Y is written in
 * rank order directly (no rotation buffer).  All pointers 16-byte aligned.
 * The result is bit-identical in every mode (option "mode").
 */
tpo_status tpo_ag_gemm(tpo_ctx* ctx, const void* const* x, const void* w, void* y,
                       const float* d_scale_inv_x, const float* d_scale_inv_w, void* stream);

/*
 * GEMM+RS: y[b] = rows [b*n/tp, (b+1)*n/tp) of sum_r X_r . W_r^T.
 *   x   host array of tp device pointers, X_r [n, k/tp]
 *   w   host array of tp device pointers, W_r [m, k/tp]
 *   y   host array of tp device pointers, y[b] [n/tp, m] bf16
 * The partial products are summed in a fixed ring order inside one GEMM:
 * the output rows owned by rank b accumulate ranks b+1, b+2, ..., b (mod tp),
 * the order of a ring reduce-scatter that ends at the owner, in fp32, with a
 * single rounding to bf16 in the epilogue.  e4m3 contexts take their scales
 * from tpo_set_fp8_scales.  Blocks are produced in order (block 0 first);
 * after every tile of block b is stored, block b's done counter (see
 * tpo_done_counters) reaches its target with release semantics.
 */
tpo_status tpo_gemm_rs(tpo_ctx* ctx, const void* const* x, const void* const* w, void* const* y,
                       void* stream);

/*
 * GEMM+AR (row-parallel linear): Y[n, m] = sum_r X_r . W_r^T.
 *   x, w          as tpo_gemm_rs
 *   y             device pointer [n, m] bf16
 *   n_row_chunks  1..64; n must be a multiple of n_row_chunks*tp
 * Output tiles are produced chunk by chunk (row chunk 0 first).  Inside row
 * chunk c, the rows of the chunk's i-th of tp equal parts sum ranks i+1, ...,
 * i (mod tp), the per-part order of a ring all-reduce of that chunk.  After
 * every tile of chunk c is stored, the chunk's done counter (see
 * tpo_done_counters) reaches its target with release semantics.  e4m3
 * contexts as tpo_gemm_rs.
 */
tpo_status tpo_gemm_ar(tpo_ctx* ctx, const void* const* x, const void* const* w, void* y,
                       int n_row_chunks, void* stream);

/*
 * Scales for GEMM+RS / GEMM+AR on an e4m3 context: device pointers to one fp32
 * each, the scale_inv shared by all X_r and the one shared by all W_r (one
 * per-tensor scale across the ranks' K-slices, as the gathered AG input
 * carries one).  The accumulated sum is multiplied by both in fp32 before the
 * bf16 rounding.  The pointers are read by every later RS/AR call (they must
 * stay valid); required before the first RS/AR call of an e4m3 context;
 * TPO_ERR_INVALID_ARG on a bf16 context or NULL pointers.
 */
tpo_status tpo_set_fp8_scales(tpo_ctx* ctx, const float* d_scale_inv_x, const float* d_scale_inv_w);

/*
 * Options (integers).  Keys:
 *   "producer_sms"     CTAs given to the chunk producer in overlapped AG; 0 (the
 *                      default) picks, from a model of the copy and GEMM rates
 *                      and the round-robin tile schedule, the fewest CTAs
 *                      whose copy does not delay the GEMM (at most 32; even
 *                      for pairs); with tail_split 1, the smallest count from
 *                      4 whose copy stays ahead of the split schedule; an odd
 *                      count for pairs is rounded up
 *   "gemm_ctas"        CTAs given to the GEMM (0 = all SMs not producing)
 *   "tail_split"       AG, modes 0-2 (default 0: whole tiles only, and every
 *                      grid, mode and producer count gives the same bits).
 *                      1: the tiles left over after the GEMM CTAs' whole
 *                      rounds go first and are divided along K among them;
 *                      2: the producer CTAs join the GEMM once their copy is
 *                      done, and the last tiles are divided along K between
 *                      the GEMM CTAs (a short share each) and them (the rest),
 *                      sized from a model of both rates; 3: as 1 but the
 *                      leftover tiles come after the whole rounds.  Each later K part of
 *                      a split tile is an fp32 partial in the context's
 *                      workspace, added in K order to the first part before
 *                      the bf16 rounding, so the result depends on the plan:
 *                      modes 1 and 2 then run mode 0's launch shape and plan
 *                      (same bits in all three); other producer counts,
 *                      gemm_ctas values and mode 4 (never split) may round
 *                      split tiles differently.
 *   "mode"             AG schedule: 0 overlapped (one launch, producer and GEMM
 *                      co-resident), 1 sequential (copy to completion, then the
 *                      same GEMM), 2 GEMM only (staging and counters must hold a
 *                      previous call's chunks), 3 producer only (no GEMM; y is
 *                      not written), 4 split: per ring step one chunk copy on a
 *                      side stream and one GEMM launch over that slot after it
 *                      (no counters; the multi-launch design of the split
 *                      all-gather overlap in TransformerEngine PR "Comm+GEMM
 *                      overlap API updated to support cuBlasMp backend" and the
 *                      ring decomposition of nvFuser PR "Ring-based
 *                      decomposition for Allgather+GEMM overlap ATen
 *                      implementation"), for comparison
 *   "seq_copy_ctas"    CTAs of the copy in sequential mode (0 = all SMs)
 *   "self_rank"        observer rank for the ring order, 0..tp-1
 *   "wait_timeout_ms"  bound of every device-side wait (default 2000)
 *   "trace"            1 = record device timestamps (tpo_read_trace)
 *   "debug_skip_chunk" slot whose counter the producer never publishes (-1 off)
 *   "debug_delay_ns"   producer spin before each publish
 *   "debug_last_step"  mode 3 only: the producer stops after this ring step
 *                      (-1 = all steps)
 *   "debug_skip_partial" GEMM CTA (index among the GEMM CTAs) that never
 *                      publishes its split-tile partial (-1 off): the tile's
 *                      finisher times out
 *   "stage_kblocks"    128-byte K blocks per shared-memory pipeline stage of
 *                      the CTA-pair variant: 1 (default; six stages of one
 *                      K block, each released as soon as its MMAs are done)
 *                      or 2 (three stages of two, one barrier test per eight
 *                      MMAs; used only where every accumulation unit has an
 *                      even number of K blocks).  Results are identical; one
 *                      block per stage measured 1.4-2.6 % faster on 4096^3.
 *   "col_split"        column tiles per tile group (AG ring step, RS owner
 *                      block, AR row chunk), the group's 32-column strips
 *                      split evenly among them: -1 the fewest tiles of at
 *                      most 256 columns; 0 (default) automatic: the fewest,
 *                      unless the launch has at most half as many tiles as
 *                      it can have GEMM CTA groups (the SMs, less 32 for the
 *                      AG producers, per MMA variant), then as many narrower
 *                      tiles per group (down to 32 columns) as still fit in
 *                      one round; otherwise 4 bits per group g < 16
 *                      ((v >> 4g) & 15) of extra tiles.  The GEMM grid
 *                      follows the plan's tile count.  Results are identical
 *                      (the MMA computes every output element the same way
 *                      whatever the tile width).  A K block of a narrower
 *                      tile costs less, but not in proportion (at 192
 *                      columns ~0.86 of a 256-column one: the operand loads
 *                      bound it), so more tiles pay only where they all fit
 *                      in one round: each tile's epilogue is then shorter.
 *   "sched"            which CTA group computes which tile: 1 round robin
 *                      (group g takes tiles g, g+G, g+2G, ...); 2 dynamic
 *                      (each group claims its next tile from a launch-wide
 *                      counter, so that faster groups take more tiles and
 *                      the tiles in flight stay a contiguous run of the tile
 *                      order); 0 (default) automatic: dynamic for launches of
 *                      at least 8 rounds, round robin otherwise and with the
 *                      AG tail split.  Results are identical either way.
 *   "cta_group"        MMA variant: 0 automatic, 1 single-SM 128x256 tiles,
 *                      2 CTA pairs (2-SM MMA, 256x256 tiles; needs every tile
 *                      group a multiple of 256 rows).  Results are identical.
 *   "cooperative"      0 (default): overlapped AG is a plain launch whose grid
 *                      never exceeds the co-resident CTA count, so once no
 *                      other work holds SMs every producer and GEMM CTA runs at
 *                      once (if other work does, a GEMM CTA's wait for a chunk
 *                      is bounded: TPO_ERR_TIMEOUT, never a hang); 1: a
 *                      cooperative launch, whose co-residency the driver
 *                      guarantees, but which cannot start before the launch
 *                      ahead of it has ended (no "pdl" overlap)
 *   "pdl"              1 (default): every kernel launch is marked for
 *                      programmatic dependent launch: its CTAs may start their
 *                      set-up (barriers, tensor memory) on SMs the previous
 *                      launch on the stream has left and wait (griddepcontrol)
 *                      for that launch's completion before touching global
 *                      memory.  Measured on back-to-back 4096^3 AG calls:
 *                      2.8-3.6 % faster.  0: ordinary stream order.
 *   "reduce"           GEMM+RS / GEMM+AR sum of the ranks' partial products:
 *                      0 (default) chain every rank's K-slice, in ring order,
 *                      into one fp32 accumulator; 1 compute each rank's partial
 *                      on its own and add the partials in ring order in the
 *                      epilogue (fp32); 2 as 1 but round every partial and
 *                      every running sum to bf16, the arithmetic of a bf16
 *                      ring reduce-scatter such as the bf16 ring all-reduce in
 *                      nvFuser PR "Reference implementation for Linear+Allreduce
 *                      with overlapping".  In modes 1 and 2 each rank's
 *                      partial takes one of the two tensor-memory accumulators
 *                      and the running sum lives in a context-owned workspace
 *                      (one 128 x 256 block per SM, fp32 in mode 1, bf16 in
 *                      mode 2), so the MMAs never wait for the additions.
 * Read-only keys for tpo_get_opt: "last_producer_ctas", "last_gemm_ctas",
 * "last_cta_group", "last_stage_kblocks", "last_split_tiles",
 * "last_late_groups", "last_col_plan", "last_sched" (shape of the context's latest kernel
 * launch: producer CTAs, GEMM CTAs, 1 or 2 CTAs per MMA, K blocks per
 * pipeline stage, tiles split along K, producer CTA groups that joined the
 * GEMM, extra column tiles per group in the col_split encoding, each
 * group's count capped at 15 in the report, 1 round robin or 2 dynamic tiles),
 * "coop_clusters" (0 once the driver refused a cooperative cluster launch),
 * "tp", "n", "k", "m", "dtype" (the sizes the context was created for).
 * Environment variables TPO_<KEY in upper case> override the defaults at
 * create time.  Unknown keys or out-of-range values: TPO_ERR_INVALID_ARG.
 */
tpo_status tpo_set_opt(tpo_ctx* ctx, const char* key, int64_t value);
tpo_status tpo_get_opt(tpo_ctx* ctx, const char* key, int64_t* value);

/* Wait for all work this context enqueued, read and clear the device error
 * word.  Returns TPO_OK or the recorded failure (TPO_ERR_TIMEOUT); after a
 * failure the counters are re-zeroed so the context is usable again. */
tpo_status tpo_sync_status(tpo_ctx* ctx);

/* Details of the last device failure seen by tpo_sync_status: code, site,
 * block index, slot (4 words). */
tpo_status tpo_last_device_error(tpo_ctx* ctx, uint32_t out[4]);

/* Thread-local message of the last failing call on this thread ("" if none). */
const char* tpo_last_error(void);

/* Read-only device pointer to the staging buffer [n, k] (the gathered X in rank
 * order), for inspection after a synchronised AG call. */
const void* tpo_staging_ptr(tpo_ctx* ctx);

/* Device pointer to the done counters (TPO_MAX_ROW_CHUNKS uint32 words), one
 * per output group of the latest tpo_gemm_rs (group b = owner block y[b]) or
 * tpo_gemm_ar (group c = row chunk c) call, and the value every group's counter
 * reaches once that call has stored all of the group's rows.  The GEMM raises
 * them with release semantics as it finishes each tile, so a consumer that
 * acquire-loads a counter equal to *target may read the group's rows while
 * the rest of the output is still being computed: the signal the
 * communication side of an atomic GEMM+RS (or of a chunked all-reduce) waits
 * on.  The counters restart from zero when the operation or the group count
 * changes between calls. */
const uint32_t* tpo_done_counters(tpo_ctx* ctx, uint32_t* target);

/* Trace words (uint64 nanoseconds of the device global timer), valid after
 * tpo_sync_status when option "trace" was 1; reset by each traced call. */
#define TPO_TRACE_START 0      /* earliest CTA start */
#define TPO_TRACE_END 1        /* latest CTA end */
#define TPO_TRACE_PUBLISH 2    /* + slot: latest producer publish of the slot */
#define TPO_TRACE_ACQUIRE 18   /* + slot: earliest GEMM acquire of the slot */
#define TPO_TRACE_WAIT_NS 34   /* total ns GEMM CTAs spent waiting on counters */
#define TPO_TRACE_CHUNK_DONE 35 /* + group: completion time of an RS block / AR row chunk */
/* Pipeline diagnosis (SM clock cycles summed over GEMM CTAs): */
#define TPO_TRACE_CYC_TMA_EMPTY 100  /* TMA issuer blocked on a free stage */
#define TPO_TRACE_CYC_MMA_FULL 101   /* MMA issuer blocked on a loaded stage */
#define TPO_TRACE_CYC_MMA_TEMPTY 102 /* MMA issuer blocked on a drained accumulator */
#define TPO_TRACE_CYC_EPI_TFULL 103  /* epilogue warps blocked on a finished accumulator */
#define TPO_TRACE_CYC_GEMM 104       /* GEMM CTAs' total cycles (set-up to tear-down) */
#define TPO_TRACE_KBLOCKS 105        /* 128-byte K blocks issued to the tensor cores */
#define TPO_TRACE_WORDS 128
tpo_status tpo_read_trace(tpo_ctx* ctx, uint64_t* out, int cap);

/* Library build string (compiler, target architecture). */
const char* tpo_version(void);

/*
 * AG+GEMM that allocates no device memory.  The pages have no counterpart of
 * this entry point; it exists for callers that cannot call cudaMalloc when they
 * run the layer: a serving process that reserved all device memory for its own
 * pool at start-up, a runtime whose allocator forbids raw device allocations
 * after initialisation so that its memory use stays fixed, or any code that
 * only owns the buffers it is handed.  tpo_ctx_create allocates, so these
 * callers cannot hold a context.
 *
 * Computes what tpo_ag_gemm computes for observer rank 0 in one overlapped
 * launch with the launch shape tpo_ag_gemm picks under default options (CTA
 * pairs wherever n/tp is a multiple of 256, the automatic column plan, the
 * schedule model's producer count, 2 s wait bound).  The result is
 * bit-identical to tpo_ag_gemm's whenever that call computes whole
 * tiles (option tail_split 0, the default), in any mode and with either MMA
 * variant; the tail-split schedules (tail_split 1 to 3) add K-split partials
 * in an order that depends on their launch shape and agree with it only
 * within the parity tolerance.  Arguments as tpo_ctx_create (tp, n, k, m,
 * dtype) plus tpo_ag_gemm (x, w, y, scale_inv pointers, stream).
 *
 * Scratch (the gathered staging buffer, the chunk counters and the error word)
 * lives in a static device array of the library: TPO_NOALLOC_MAX_STAGING_BYTES
 * plus TPO_NOALLOC_WORDS_BYTES (the kernel's word block rounded up to 256
 * bytes), held by every GPU that loads the library until the process exits.
 * n*k*element size above TPO_NOALLOC_MAX_STAGING_BYTES is rejected with
 * TPO_ERR_INVALID_ARG and a message naming the limit.
 * The first call on a device sets that device up (looks up the array's device
 * address, configures the kernel); make it before any stream capture.
 * Every call shares the array and clears its counters and error word on
 * `stream` first; calls whose GPU work could overlap (other streams, other host
 * threads) race on the array.  The call blocks until its work on `stream` has
 * finished, then returns TPO_OK or TPO_ERR_TIMEOUT if a device wait ran out.
 * If it returns TPO_ERR_CUDA after its launch (the error word could not be
 * read back), it first tries to wait for `stream`; should that fail as well,
 * the kernel may still be running and the array's contents stay undefined
 * until the device is reset.
 */
#define TPO_NOALLOC_MAX_STAGING_BYTES (32ull << 20) /* 32 MiB */
#define TPO_NOALLOC_WORDS_BYTES 5632ull             /* counters, error word, trace: 5.5 KiB */
tpo_status tpo_ag_gemm_noalloc(int tp, int64_t n, int64_t k, int64_t m, int dtype, const void* const* x,
                               const void* w, void* y, const float* d_scale_inv_x,
                               const float* d_scale_inv_w, void* stream);

/*
 * Block operators: the parts of a transformer sublayer that sit next to its
 * tensor-parallel projections.  Layer norm, a linear layer with bias,
 * activation and residual in the product's epilogue, and the gated
 * feed-forward projections, each with its backward pass.
 *
 * They run on a tpo_block handle, which owns a workspace and a device error
 * word; the rules are the context's.  A call validates its arguments on the
 * host, enqueues kernels on `stream` and returns; nothing is allocated, and a
 * call may be captured into a CUDA graph.  The current device must be the
 * handle's.  A handle is not thread-safe, and calls that overlap on the GPU
 * (different streams) need different handles.  A device-side wait that runs
 * out is sticky until tpo_block_sync_status reports it.
 *
 * Layout: n counts rows (tokens), k input features, m output features.  Every
 * matrix is row-major with its own row pitch `ld` in elements (at least the
 * row's length).  Pitches of the matrix products are multiples of 16 bytes and
 * their addresses 16-byte aligned (a matrix of at most one row needs no
 * pitch); k and m themselves may be any number from 1.  The layer norm takes
 * any pitch and any address that its element type allows.  n = 0 is an empty
 * batch: forward calls and input gradients write nothing, weight gradients
 * become zero.  Outputs must not overlap inputs except where a call says so.
 *
 * Arithmetic: sums, norms, biases, activations and their derivatives are
 * computed in fp32 from the inputs' values, and an output is rounded once, to
 * its own type.  The backward products take the gradient of the
 * pre-activation as a matrix operand, so it is rounded to bf16 in between (the
 * gradient of the bias is summed before that rounding).  No call uses atomics
 * on data: calls with the same values, sizes, pitches, address alignments and
 * options on the same kind of device give the same bits.  (Pitches, alignments
 * and the number of SMs enter the choice of kernel and with it the order in
 * which fp32 terms are added.)
 * NaN and infinities in the inputs spread as the formulas say, and only there:
 * a row of the output never sees another row's input.
 */
typedef struct tpo_block tpo_block; /* opaque */

/* Activations.  GELU is x Phi(x), GELU_TANH its tanh form
 * x/2 (1 + tanh(sqrt(2/pi) (x + 0.044715 x^3))), SILU x / (1 + exp(-x)).
 * RELU's derivative at 0 is 0.  At NaN every activation is NaN, and so is every
 * derivative but NONE's. */
typedef enum { TPO_ACT_NONE = 0, TPO_ACT_RELU = 1, TPO_ACT_GELU = 2, TPO_ACT_GELU_TANH = 3, TPO_ACT_SILU = 4 } tpo_act;

/* The block operators, as tpo_block_workspace names them. */
typedef enum {
  TPO_OP_LAYER_NORM = 0,
  TPO_OP_LAYER_NORM_BWD = 1,
  TPO_OP_LINEAR = 2,
  TPO_OP_LINEAR_BWD = 3,
  TPO_OP_GATED = 4,
  TPO_OP_GATED_BWD = 5
} tpo_block_op;

/* Bytes of workspace that one call of `op` with up to n rows needs (m is not
 * used by the norms), or -1 with tpo_last_error set for sizes out of range.
 * Forward calls need none; needs no GPU. */
int64_t tpo_block_workspace(int op, int64_t n, int64_t k, int64_t m);

/* Create a handle with `workspace_bytes` (0 or more) of workspace on the
 * current CUDA device: the largest need of the calls it will serve.  A call
 * whose need is larger returns TPO_ERR_INVALID_ARG and names it.  NULL on any
 * error; tpo_last_error says why. */
tpo_block* tpo_block_create(int64_t workspace_bytes);

/* Release the handle (its pending work must have been synchronised or may
 * still run: the release waits for the device).  NULL is a no-op. */
tpo_status tpo_block_destroy(tpo_block* blk);

/*
 * Options (integers).  The first two choose how the products run; results agree
 * within the rounding of fp32 sums.
 *   "path"   0 (default) by rule; 1 CTA pairs (256-row tiles); 2 clusters that
 *            cut the contraction (for few rows, or small weights' gradients)
 *   "split"  CTAs of such a cluster, 1..8; 0 (default) by rule
 *   "wait_timeout_ms"  bound of every device-side wait, 1..600000 (default 2000)
 * Unknown keys or values out of range: TPO_ERR_INVALID_ARG.
 */
tpo_status tpo_block_set_opt(tpo_block* blk, const char* key, int64_t value);
tpo_status tpo_block_get_opt(tpo_block* blk, const char* key, int64_t* value);

/* Wait for the work on `stream`, read and clear the handle's error word. */
tpo_status tpo_block_sync_status(tpo_block* blk, void* stream);

/*
 * Layer norm over the last dimension, row by row:
 *   mean = sum x / k,  rstd = 1 / sqrt(sum (x - mean)^2 / k + eps)
 *   y = (x - mean) rstd gamma + beta
 *   dtype    of x and y: TPO_BF16 or TPO_F32
 *   wdtype   of gamma and beta [k]: TPO_BF16 or TPO_F32; either pointer may be
 *            NULL (gamma 1, beta 0)
 *   mean, rstd  [n] fp32, written for the backward pass; NULL to skip
 * The variance is the mean of squared differences (no cancellation of
 * sums of squares).  y may be x itself, with the same pitch.
 */
tpo_status tpo_layer_norm(tpo_block* blk, int64_t n, int64_t k, int dtype, int wdtype, const void* x, int64_t ldx,
                          const void* gamma, const void* beta, float eps, void* y, int64_t ldy, float* mean,
                          float* rstd, void* stream);

/*
 * Gradient of tpo_layer_norm, with xhat = (x - mean) rstd and a = dy gamma:
 *   dx = rstd (a - mean(a) - xhat mean(a xhat)) [+ dres]
 *   dgamma = sum over rows of dy xhat,  dbeta = sum over rows of dy
 * dres [n, k] (NULL: none) is the gradient that reaches x past the norm, as on
 * a residual branch.  dx, dgamma and dbeta (of wdtype) may each be NULL; gamma
 * NULL means 1.  dx may be dy or dres itself, with the same pitch.
 */
tpo_status tpo_layer_norm_bwd(tpo_block* blk, int64_t n, int64_t k, int dtype, int wdtype, const void* dy,
                              int64_t lddy, const void* x, int64_t ldx, const void* gamma, const float* mean,
                              const float* rstd, const void* dres, int64_t lddres, void* dx, int64_t lddx,
                              void* dgamma, void* dbeta, void* stream);

/*
 * Linear layer with its epilogue:  y = act(z) + residual,  z = x w^T + bias
 *   dtype      of x [n, k] and w [m, k]: TPO_BF16 or TPO_FP8_E4M3
 *   bias       [m] bf16 or NULL;  act: a tpo_act
 *   residual   [n, m] bf16 or NULL; may be y itself, with the same pitch
 *   z          [n, m] bf16, the pre-activation for the backward pass, or NULL
 *   y          [n, m] bf16
 *   d_scale_inv_x, d_scale_inv_w  e4m3: device pointers to one fp32 each, the
 *              product is multiplied by both before the bias; bf16: NULL
 */
tpo_status tpo_linear(tpo_block* blk, int64_t n, int64_t k, int64_t m, int dtype, const void* x, int64_t ldx,
                      const void* w, int64_t ldw, const void* bias, int act, const void* residual, int64_t ldr,
                      void* z, int64_t ldz, void* y, int64_t ldy, const float* d_scale_inv_x,
                      const float* d_scale_inv_w, void* stream);

/*
 * Gradient of tpo_linear (bf16):  dz = dy act'(z);
 *   dx [n, k] = dz w,  dw [m, k] = dz^T x,  db [m] = sum over rows of dz
 * z is the forward call's (TPO_ACT_NONE: NULL).  dx, dw and db may each be
 * NULL; without dx, w may be NULL, and without dw, x.  The residual's gradient
 * is dy itself.
 */
tpo_status tpo_linear_bwd(tpo_block* blk, int64_t n, int64_t k, int64_t m, int act, const void* dy, int64_t lddy,
                          const void* z, int64_t ldz, const void* x, int64_t ldx, const void* w, int64_t ldw,
                          void* dx, int64_t lddx, void* dw, int64_t lddw, void* db, void* stream);

/*
 * Gated feed-forward projections:  h = act(g) * u,  g = x wg^T,  u = x wu^T
 * (SILU: SwiGLU, GELU: GeGLU, RELU: ReGLU, NONE: bilinear).
 *   x [n, k], wg and wu [m, k] of dtype; h [n, m] bf16
 *   g, u       [n, m] bf16 for the backward pass, both or neither NULL
 *   scales     e4m3: device pointers for x, wg and wu; bf16: NULL
 */
tpo_status tpo_gated(tpo_block* blk, int64_t n, int64_t k, int64_t m, int dtype, const void* x, int64_t ldx,
                     const void* wg, int64_t ldwg, const void* wu, int64_t ldwu, int act, void* g, int64_t ldg,
                     void* u, int64_t ldu, void* h, int64_t ldh, const float* d_scale_inv_x,
                     const float* d_scale_inv_wg, const float* d_scale_inv_wu, void* stream);

/*
 * Gradient of tpo_gated (bf16):  dg = dh u act'(g),  du = dh act(g);
 *   dx [n, k] = dg wg + du wu,  dwg [m, k] = dg^T x,  dwu [m, k] = du^T x
 * dx may be NULL (wg and wu may then be, too), and dwg and dwu together (x may
 * then be, too).
 */
tpo_status tpo_gated_bwd(tpo_block* blk, int64_t n, int64_t k, int64_t m, int act, const void* dh, int64_t lddh,
                         const void* g, int64_t ldg, const void* u, int64_t ldu, const void* x, int64_t ldx,
                         const void* wg, int64_t ldwg, const void* wu, int64_t ldwu, void* dx, int64_t lddx,
                         void* dwg, int64_t lddwg, void* dwu, int64_t lddwu, void* stream);

/*
 * The attention sublayer: what lies between a column-parallel projection of
 * queries, keys and values and the row-parallel output projection.  Rotary
 * positions and attention with grouped heads, on the same handle and under the
 * same rules as the block operators above.
 *
 * Layout: q and its like are [n, heads, dim], k and v [nk, kv_heads, dim], bf16,
 * with unit stride in dim, a pitch `ld` from one row (token) to the next and a
 * pitch `h` from one head to the next, in elements.  A slice of a fused
 * projection's output, a cache of rows and a cache of heads are all of this
 * form.  A pitch that a single row or a single head does not need is ignored.
 */

/* How a head's first `rot` elements form pairs: element i with i + rot / 2, or
 * 2 i with 2 i + 1. */
typedef enum { TPO_ROTARY_HALVES = 0, TPO_ROTARY_PAIRS = 1 } tpo_rotary_layout;
/* Frequencies for contexts longer than the trained one: as they are, all
 * divided by `factor`, or each by how many turns it makes over the trained
 * context of `original` positions: kept from `high` turns on, divided by
 * `factor` up to `low`, and a linear blend of the two between. */
typedef enum { TPO_ROTARY_UNSCALED = 0, TPO_ROTARY_LINEAR = 1, TPO_ROTARY_BY_PARTS = 2 } tpo_rotary_scaling;

/*
 * Writes the rot / 2 entries of a table in host memory (the caller copies it to
 * the device; needs no GPU).  Pair i turns by f_i = base^(-2 i / rot) radians a
 * position, scaled as above; its entry is 2^64 f_i / (2 pi) modulo 2^64, the
 * turns per position as a 64-bit fraction.  Any other frequencies may be put
 * into a table in the same form.  TPO_ERR_INVALID_ARG, and nothing is written,
 * if base and factor make a frequency that is not finite.
 */
tpo_status tpo_rotary_table(int64_t rot, double base, int scaling, double factor, double low, double high,
                            int64_t original, uint64_t* table);

/*
 * Rotary positions: each pair (a, b) of the first `rot` elements of a head
 * becomes magnitude (a cos t - b sin t, a sin t + b cos t), t = position times
 * the pair's frequency; the other elements are copied.
 *   dtype      of x and y: TPO_BF16 or TPO_F32; pitches and addresses as their
 *              element type allows
 *   inverse    not 0: turns the other way, which is the gradient (of dy to dx)
 *   pos        [n] positions, any of 32 bits; NULL: the row's number
 *   table      [rot / 2] in device memory, as tpo_rotary_table writes it
 *   rows       [n] the row of y that each row goes to (as into a cache), NULL:
 *              its own, with ny = n.  Rows that are negative or at least ny are
 *              left out; no two may be the same.
 * The angle is exact for every position (64-bit arithmetic); sine, cosine and
 * the turn are computed in fp32, and the result is rounded once.  y may be x,
 * with the same pitches and without rows, and overlaps it in no other way.
 * rot = 0 copies.
 */
tpo_status tpo_rotary(tpo_block* blk, int64_t n, int64_t heads, int64_t dim, int64_t rot, int dtype, int layout,
                      int inverse, float magnitude, const int32_t* pos, const uint64_t* table, const void* x,
                      int64_t ldx, int64_t hx, const int32_t* rows, int64_t ny, void* y, int64_t ldy, int64_t hy,
                      void* stream);

/* Bytes of workspace that a call with up to n and nk rows needs (batch does not
 * enter), or -1 with tpo_last_error set; need no GPU. */
int64_t tpo_attention_workspace(int64_t n, int64_t nk, int64_t heads, int64_t kv_heads, int64_t dim);
int64_t tpo_attention_bwd_workspace(int64_t n, int64_t nk, int64_t heads, int64_t kv_heads, int64_t dim);

/*
 * Attention, sequence by sequence:
 *   out = softmax(scale q k^T) v
 *   lse = log sum exp(scale q k^T)  (natural logarithm)
 * heads is a multiple of kv_heads (up to 128 times); query head h reads key head
 * h / (heads / kv_heads).  dim is a multiple of 8 up to 128.  Addresses are
 * 16-byte aligned and pitches multiples of 16 bytes.
 *   q_start    [batch + 1] device, not decreasing: sequence i has the queries of
 *              rows q_start[i] up to q_start[i + 1]; batch is at least 1
 *   k_start, k_len  device: its keys are k_len[i] rows from k_start[i] on, or
 *              with k_len NULL (k_start then has batch + 1 entries) the rows
 *              up to k_start[i + 1], or with both NULL the queries' rows.
 *              With one sequence each may be NULL: all rows, k_len of them.
 *   causal     not 0: the sequence's last query sees all of its keys, each
 *              earlier one a key less (query t of nq sees t + 1 + nk - nq)
 *   scale      positive, at most 1e38
 *   lse        [n, heads] fp32 for the backward pass, or NULL
 * Lengths are read on the device: a captured call follows them as they change.
 * Starts and lengths are held inside the tensors, so that no call reads or
 * writes outside them.  A sequence may have no queries or no keys; a query that
 * sees no key gets zeros and lse = -infinity.  Rows of no sequence are left as
 * they were, and what they or the unused rows of a cache hold is never used.
 * Scores, weights and sums are held in fp32; the weights are rounded to bf16
 * as operands of the product with v (their sum is taken before that).
 * A call's work is counted in steps.  A tile is 2 floor(128 / group) tokens of a
 * sequence with the group = heads / kv_heads heads that share a key head; it has
 * a step for every 128 keys that its last token sees, at least one, and four
 * more.  (In the gradient: tiles of floor(128 / group) tokens over keys and, for
 * dk and dv, tiles of 128 keys over those of tokens, each with two more; each of
 * the two counts by itself.)  There may be 2^31 - 2 steps.  One sequence without
 * arrays that has more is refused with TPO_ERR_UNSUPPORTED; where lengths are on
 * the device, nothing is computed and tpo_block_sync_status reports the same
 * error.
 * What stores a tile waits for as long as its block works on it, about 1.5 us for
 * every 128 keys, and the way past a million slots without queries takes some
 * 10 ms: from 10^8 of either on, option "wait_timeout_ms" has to follow.
 * Outputs overlap no input.
 */
tpo_status tpo_attention(tpo_block* blk, int64_t batch, int64_t n, int64_t nk, int64_t heads, int64_t kv_heads,
                         int64_t dim, const int32_t* q_start, const int32_t* k_start, const int32_t* k_len,
                         int causal, float scale, const void* q, int64_t ldq, int64_t hq, const void* k, int64_t ldk,
                         int64_t hk, const void* v, int64_t ldv, int64_t hv, void* out, int64_t ldo, int64_t ho,
                         float* lse, void* stream);

/*
 * Gradient of tpo_attention, with p = exp(scale q k^T - lse) and
 * delta = sum over dim of dout out:
 *   ds = p (dout v^T - delta);  dq = scale ds k,  dk = scale ds^T q,  dv = p^T dout
 * dk and dv are summed over the query heads that share a key head.  out and lse
 * are the forward call's.  The sequences' keys must not overlap, nor an output
 * an input.  A key that no
 * query sees gets zeros.  p and ds are rounded to bf16 as operands of the
 * products.  Rows of no sequence are left as they were, in dq, dk and dv too.
 * Rows of other sequences and of none never reach a gradient; within
 * a sequence a value that is not finite may also reach gradients that it has no
 * part in, of rows that share a product of 128 by 128 with it.
 */
tpo_status tpo_attention_bwd(tpo_block* blk, int64_t batch, int64_t n, int64_t nk, int64_t heads, int64_t kv_heads,
                             int64_t dim, const int32_t* q_start, const int32_t* k_start, const int32_t* k_len,
                             int causal, float scale, const void* dout, int64_t lddo, int64_t hdo, const void* q,
                             int64_t ldq, int64_t hq, const void* k, int64_t ldk, int64_t hk, const void* v,
                             int64_t ldv, int64_t hv, const void* out, int64_t ldo, int64_t ho, const float* lse,
                             void* dq, int64_t lddq, int64_t hdq, void* dk, int64_t lddk, int64_t hdk, void* dv,
                             int64_t lddv, int64_t hdv, void* stream);

#ifdef __cplusplus
}
#endif
#endif /* TPOVERLAP_H */

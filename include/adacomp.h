/*
 * adacomp.h -- C ABI of the AdaComp compressor for AMD Instinct MI355X (gfx950).
 *
 * AdaComp ("AdaComp (Adaptive Residual Gradient Compression)", AIMech curated
 * page, definition paragraph and the Mechanism claim on local-bin soft
 * threshold and mean-g_max quantization, Algorithm 2) compresses each layer's
 * gradient dW against a residue carried from step to step:
 *
 *   G = residue + dW,  H = G + dW                       (float32, no contraction)
 *   bins of L_T consecutive elements; g_max(i) = max |G| over bin i
 *   transmit every element with |H| >= g_max(its bin) and G != 0
 *   s = mean of g_max over the layer's bins             (one scale per layer)
 *   G_q = sign(G) * s for transmitted elements
 *   residue <- G - G_q (transmitted), residue <- G (all others)
 *
 * The transmitted elements are packed as sparse-indexed ternary words, 8-bit
 * when L_T < 64 and 16-bit otherwise (Application claim, Table 2; Curated
 * Limitations), into a message whose length varies from step to step
 * (Limitation claim).  decode_accumulate sums several such messages, one per
 * learner of a data-parallel job, into a dense float32 gradient.
 *
 * Conventions common to every call:
 *   - Every pointer named residue, dW, out, msg, msgs[k] or ws is a DEVICE
 *     pointer on the device that was current when the plan was created; that
 *     device must be current at the call.  Pointers to plain structs and to
 *     the msgs array are HOST pointers.  The caller owns every buffer.
 *   - The flat float32 buffers (residue, dW, out) hold every layer of the
 *     segment table at its element offset; they must be 16-byte aligned and
 *     hold at least info.span elements (the end of the last layer rounded up
 *     to a multiple of 4).  Elements outside every segment may be read but
 *     are never written.
 *   - msg and ws must be 16-byte aligned and at least as large as the plan
 *     reports.  Buffers given to one call must not overlap.
 *   - Calls are asynchronous on `stream` (a hipStream_t; NULL is the default
 *     stream) and return once the work is enqueued.  Argument errors are
 *     detected on the host before anything is enqueued, and then nothing is
 *     written.  Results are deterministic: the same inputs give the same bits.
 *   - Return value: ADACOMP_OK (0) or a negative status; adacomp_status_str()
 *     names it.  No C++ exception crosses this interface.
 *
 * Message layout (all little-endian, every region 16-byte aligned, padding
 * bytes zero; w = 8 if L_T < 64 else 16):
 *   header, 32 bytes: u32 magic 0x43414441 ("ADAC"), u16 version 1, u16 0,
 *     u32 nseg, u32 plan_hash, u64 total_bytes, u64 total_survivors;
 *   directory at byte 32: nseg x 16 bytes {f32 s, u32 nsurv, u64 entries_offset};
 *   count regions, one per segment in table order, at positions fixed by the
 *     plan: B words of w bits, the number of transmitted elements per bin;
 *   entry regions, one per segment in table order, packed after the count
 *     regions: nsurv words of w bits, bin-major with ascending in-bin index,
 *     each word = sign << (w-1) | in_bin_index, sign = 1 iff G < 0.
 */
#ifndef ADACOMP_H
#define ADACOMP_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Status codes. */
#define ADACOMP_OK 0
#define ADACOMP_ERR_INVALID_ARGUMENT (-1) /* null pointer, empty table, numel 0, unknown flags, wrong device, aliasing */
#define ADACOMP_ERR_UNSUPPORTED_BIN (-2)  /* L_T = 0 or L_T > 32768 (a 16-bit word holds a 15-bit index) */
#define ADACOMP_ERR_MISALIGNED (-3)       /* segment offset not a multiple of 4, or a buffer not 16-byte aligned */
#define ADACOMP_ERR_OVERLAP (-4)          /* two segments share an element */
#define ADACOMP_ERR_CAPACITY (-5)         /* a buffer is smaller than the plan requires */
#define ADACOMP_ERR_HIP (-6)              /* a HIP runtime call or kernel launch failed */
#define ADACOMP_ERR_TOO_LARGE (-7)        /* numel >= 2^32 in one segment, or the table exceeds launch limits */
#define ADACOMP_ERR_SCRATCH_LIMIT (-8)    /* adacomp_compress_noalloc: the plan's workspace exceeds its scratch */

#define ADACOMP_MAX_BIN_LEN 32768u

/* Segment flag: hard Local Selection (LS) instead of AdaComp's soft threshold.
 * The baseline the same page's Mechanism claim "self-adjusting sparsity
 * prevents residual explosion" (Figures 4-6) contrasts AdaComp with: per bin
 * only the first element (lowest index) whose |G| equals the bin maximum is
 * transmitted, none when the maximum is 0; s, the residue update and the
 * message format are those of AdaComp. */
#define ADACOMP_SEG_LS 1u
#define ADACOMP_MAX_MESSAGES 256u         /* most messages one decode_accumulate call sums */

/* One layer: numel consecutive elements of the flat buffers starting at
 * element `offset` (a multiple of 4), compressed with bins of bin_len = L_T
 * elements over its flattened storage order.  flags: 0 (AdaComp) or
 * ADACOMP_SEG_LS. */
typedef struct adacomp_segment {
    uint64_t offset;
    uint64_t numel;
    uint32_t bin_len;
    uint32_t flags;
} adacomp_segment;

/* Sizes a caller needs to allocate buffers for a segment table. */
typedef struct adacomp_plan_info {
    uint32_t nseg;
    uint32_t plan_hash;                 /* FNV-1a 32 of the table, as in message headers */
    uint64_t total_numel;               /* sum of numel */
    uint64_t span;                      /* max(offset + numel) rounded up to a multiple of 4:
                                           the minimum length of residue, dW and out */
    uint64_t total_bins;                /* sum over segments of ceil(numel / bin_len) */
    uint64_t ntiles;                    /* work tiles (whole bins of one segment each) */
    uint64_t header_bytes;              /* 32 + 16*nseg: read this much to learn a message's size */
    uint64_t message_capacity;          /* largest possible message: every element transmitted */
    uint64_t compress_workspace_bytes;
    uint64_t decode_workspace_bytes_per_message;
    uint64_t decode_workspace_bytes_fixed; /* decode ws for K messages = fixed + K * per_message */
    uint64_t compress_launches;         /* kernel launches of one adacomp_compress call */
} adacomp_plan_info;

typedef struct adacomp_plan adacomp_plan;   /* opaque, immutable once created */
typedef struct adacomp_timer adacomp_timer; /* opaque per-kernel device timer */

/* Host-only: validate a segment table and report the sizes its plan would
 * have.  Touches no GPU.  Returns a status; fills *info on success. */
int adacomp_plan_query(const adacomp_segment* segs, uint32_t nseg, adacomp_plan_info* info);

/* Validate the table, build the work tiles and copy the small tile tables to
 * the current device.  The plan owns that device memory until
 * adacomp_plan_destroy.  An immutable plan may be used from several streams
 * at once (with separate buffers).
 *
 * Compress is one tile-pass launch per tile shape used (bins up to 2045,
 * up to 4093, longer), then the finish: survivor offsets, s, header and
 * directory, entry words and residue of the sent elements.  For a small
 * table -- span <= ADACOMP_SMALL_TABLE_MAX_SPAN elements and at most
 * ADACOMP_SMALL_TABLE_MAX_SEGMENTS segments -- the finish is one launch
 * whose every workgroup holds the table's tile counts in LDS.  Otherwise, for
 * a table of at most ADACOMP_SMALL_TABLE_MAX_SEGMENTS segments and at most
 * ADACOMP_CHUNK_FINISH_MAX_TILES tiles (info.ntiles), it is two: the chunk
 * scan, then one kernel whose every workgroup computes s and the entry
 * regions from the chunk sums in LDS and encodes its share.  Any other table
 * takes three (chunk scan, finalize, encode).  info.compress_launches reports
 * the total.  Every path writes the same bytes.  plan_query reports the sizes
 * of a plan made with no flags. */
#define ADACOMP_SMALL_TABLE_MAX_SPAN (1u << 21)
#define ADACOMP_SMALL_TABLE_MAX_SEGMENTS 256u
#define ADACOMP_CHUNK_FINISH_MAX_TILES (1u << 20)
int adacomp_plan_create(const adacomp_segment* segs, uint32_t nseg, adacomp_plan** plan);

/* Plan flags (adacomp_plan_create_ex).
 * SEPARATE_FINISH: finish with the three kernels whatever the table.
 * SINGLE_LAUNCH: compress a small table whose bins are all <= 4093 in one
 *   launch: the workgroup that finishes its tile last completes the message
 *   alone.  Correct, but slower on MI355X than the default (the release of
 *   every tile and one CU's scattered stores cost more than the launches it
 *   saves); built for comparison.  Other tables ignore it.
 * The two flags are exclusive.
 * DECODE_RECORDS: plain sums (adacomp_decode_accumulate with accumulate = 0)
 *   of at most 16 messages over bins of at most 4093 elements always take the
 *   entry-record decode (a per-tile record pass, then tiles that read their
 *   count and entry words in one round trip).  By default only tables of at
 *   least 65536 such tiles, all of 16-bit words, take it; smaller tables and
 *   8-bit words measured faster without it.  Combines with either flag above. */
#define ADACOMP_PLAN_SEPARATE_FINISH 1u
#define ADACOMP_PLAN_SINGLE_LAUNCH 2u
#define ADACOMP_PLAN_DECODE_RECORDS 4u
/* adacomp_plan_create with plan flags (0, or an OR of the above with at most
 * one of SEPARATE_FINISH and SINGLE_LAUNCH; any other value is
 * ADACOMP_ERR_INVALID_ARGUMENT). */
int adacomp_plan_create_ex(const adacomp_segment* segs, uint32_t nseg, uint32_t plan_flags,
                           adacomp_plan** plan);
int adacomp_plan_destroy(adacomp_plan* plan);
int adacomp_plan_get_info(const adacomp_plan* plan, adacomp_plan_info* info);

/* One AdaComp compression step over every segment (the definition above).
 *   residue  [span] float32, read and updated in place.
 *   dW       [span] float32, read only.
 *   n_elems  elements in residue and in dW (>= info.span).
 *   msg      message output, msg_bytes >= info.message_capacity.  Its length
 *            is the header's total_bytes (read it after the stream syncs).
 *   ws       workspace, ws_bytes >= info.compress_workspace_bytes; no
 *            initial contents required, contents undefined afterwards, except
 *            that with ADACOMP_PLAN_SINGLE_LAUNCH its first 8 bytes hold a
 *            ticket counter: a 48-bit tag above a 16-bit count, left with
 *            count 0.  Any other initial value is accepted; only the tag with
 *            a nonzero count (a call stopped part way) would miscount.
 *   bin_max_out  nullable device float32[total_bins]: every g_max, segments
 *            in table order, bins in order (a testing aid).
 * Determinism: s is the bin maxima summed in float64 in a fixed order, divided
 * by B in float64 and rounded once to float32; everything else is exact. */
int adacomp_compress(const adacomp_plan* plan, float* residue, const float* dW,
                     uint64_t n_elems, void* msg, uint64_t msg_bytes, void* ws,
                     uint64_t ws_bytes, float* bin_max_out, void* stream);

/* For callers that cannot allocate device memory (code under HIP graph
 * capture, tight serving loops, harnesses that forbid allocation): one
 * compression step exactly as adacomp_compress, with the workspace taken
 * from a scratch array the library holds on each GPU it runs on, from the
 * first call on that GPU until the process ends.  The call allocates nothing
 * (no hipMalloc, hipFree or other allocating routine).
 *   Arguments as for adacomp_compress, without ws and ws_bytes; the current
 *   device must be the plan's.
 *   The plan's info.compress_workspace_bytes must be at most
 *   ADACOMP_NOALLOC_SCRATCH_BYTES (128 MiB: tables of up to about 33 million
 *   elements); larger plans return ADACOMP_ERR_SCRATCH_LIMIT before any work.
 *   Every call on one GPU shares that GPU's scratch and it keeps the last
 *   call's contents (compress needs no initial contents): calls that may
 *   overlap on one GPU -- on different streams, or from different threads
 *   without ordering -- race and must not be issued. */
#define ADACOMP_NOALLOC_SCRATCH_BYTES (128ull << 20)
int adacomp_compress_noalloc(const adacomp_plan* plan, float* residue, const float* dW,
                             uint64_t n_elems, void* msg, uint64_t msg_bytes, float* bin_max_out,
                             void* stream);

/* Sum K messages made by adacomp_compress with this same segment table into
 * out, in message order: for k = 0..K-1 and every element j message k
 * transmits, out[j] = out[j] + sign * s (float32, rounded each time).
 *   msgs        HOST array of K device pointers; 1 <= K <= ADACOMP_MAX_MESSAGES.
 *   out         [span] float32.  accumulate = 0: every element of every
 *               segment starts from +0; accumulate = 1: starts from out.
 *               An element no message transmits gets no addition.
 *   ws          ws_bytes >= fixed + K * per_message (see plan info).
 * Each msgs[k] must point to at least the header's total_bytes readable
 * bytes (at least 32).  A message is checked on the device before any entry
 * word is read, and is refused -- it contributes nothing, the other messages
 * are summed as if it were absent -- when its header does not match the plan
 * (magic, version, nseg, plan_hash; total_bytes a multiple of 16 between the
 * start of the entry regions and info.message_capacity), or when a segment's
 * directory entry disagrees with the count words (entry offset not 16-byte
 * aligned or before the entry regions; survivors more than the segment's
 * elements or unequal to the sum of its count words; a tile counting more
 * survivors than it has elements; the padded entry region past total_bytes).
 * Entry words whose in-bin index lies outside the bin are ignored.  The
 * number of refused messages is written as a uint32 at byte 0 of ws; the
 * call itself still returns ADACOMP_OK. */
int adacomp_decode_accumulate(const adacomp_plan* plan, const void* const* msgs, uint32_t K,
                              float* out, uint64_t n_elems, int accumulate, void* ws,
                              uint64_t ws_bytes, void* stream);

/* One step of SGD with momentum (no dampening, no Nesterov), the optimizer the
 * paper's abstract names for its training runs, taken on the summed messages:
 *   g = scale * sum (+ weight_decay * w when weight_decay != 0)
 *   m = momentum * m + g
 *   w = w - lr * m
 * each operation one float32 operation rounded to nearest. */
typedef struct adacomp_sgd {
    float lr;
    float momentum;
    float weight_decay;
    float scale;    /* e.g. 1/K to average the learners' gradients */
} adacomp_sgd;

/* Sum K messages exactly as adacomp_decode_accumulate with accumulate = 0 and
 * take one adacomp_sgd step on every element of every segment, without
 * writing the sum to memory (one dense pass instead of decode + optimizer).
 *   weights, momentum  [span] float32 each, updated in place; elements
 *               outside every segment are not written.
 *   sgd         HOST pointer to the step's parameters.
 *   ws          ws_bytes >= adacomp_decode_sgd_workspace_bytes(plan, K); plans
 *               with bins longer than 4093 elements need a dense scratch of
 *               4 * span bytes in it.
 * Messages are checked, refused and counted at byte 0 of ws as in
 * adacomp_decode_accumulate. */
int adacomp_decode_sgd(const adacomp_plan* plan, const void* const* msgs, uint32_t K,
                       float* weights, float* momentum, uint64_t n_elems, const adacomp_sgd* sgd,
                       void* ws, uint64_t ws_bytes, void* stream);
int adacomp_decode_sgd_workspace_bytes(const adacomp_plan* plan, uint32_t K, uint64_t* bytes);

/* One Adam step with bias-corrected moments (the other optimizer the paper's
 * abstract names), in its textbook form, each operation one float32
 * operation rounded to nearest (division and square root correctly rounded):
 *   g = scale * sum (+ weight_decay * w when weight_decay != 0)
 *   m = beta1 * m + (1 - beta1) * g;   v = beta2 * v + (1 - beta2) * (g * g)
 *   w = w - lr * ((m / c1) / (sqrt(v / c2) + eps))
 * c1 = 1 - beta1^step, c2 = 1 - beta2^step, each computed in double on the
 * host and rounded once to float; 1 - beta1 and 1 - beta2 are float
 * operations.  step >= 1 counts the calls made so far, this one included. */
typedef struct adacomp_adam {
    float lr;
    float beta1;
    float beta2;
    float eps;
    float weight_decay;
    float scale;
    uint32_t step;
} adacomp_adam;

/* As adacomp_decode_sgd, with one Adam step on weights, m and v ([span]
 * float32 each, updated in place).  ws as for adacomp_decode_sgd
 * (adacomp_decode_sgd_workspace_bytes).  step = 0 is an invalid argument. */
int adacomp_decode_adam(const adacomp_plan* plan, const void* const* msgs, uint32_t K,
                        float* weights, float* m, float* v, uint64_t n_elems,
                        const adacomp_adam* adam, void* ws, uint64_t ws_bytes, void* stream);

/* Same calls with a timer: device time of each kernel stage is recorded with
 * HIP events on `stream` and summed in the timer.  timer may be NULL. */
int adacomp_compress_timed(const adacomp_plan* plan, float* residue, const float* dW,
                           uint64_t n_elems, void* msg, uint64_t msg_bytes, void* ws,
                           uint64_t ws_bytes, float* bin_max_out, void* stream,
                           adacomp_timer* timer);
int adacomp_decode_accumulate_timed(const adacomp_plan* plan, const void* const* msgs,
                                    uint32_t K, float* out, uint64_t n_elems, int accumulate,
                                    void* ws, uint64_t ws_bytes, void* stream,
                                    adacomp_timer* timer);
int adacomp_decode_sgd_timed(const adacomp_plan* plan, const void* const* msgs, uint32_t K,
                             float* weights, float* momentum, uint64_t n_elems,
                             const adacomp_sgd* sgd, void* ws, uint64_t ws_bytes, void* stream,
                             adacomp_timer* timer);
int adacomp_decode_adam_timed(const adacomp_plan* plan, const void* const* msgs, uint32_t K,
                              float* weights, float* m, float* v, uint64_t n_elems,
                              const adacomp_adam* adam, void* ws, uint64_t ws_bytes, void* stream,
                              adacomp_timer* timer);

/* Kernel stages a timer reports, in this order. */
#define ADACOMP_STAGE_TILE_PASS 0   /* dense pass: G, H, bin maxima, selection, counts */
#define ADACOMP_STAGE_CHUNK_SCAN 1  /* per-chunk survivor offsets and scale partial sums */
#define ADACOMP_STAGE_FINALIZE 2    /* s per segment, message header and directory (three-kernel finish) */
#define ADACOMP_STAGE_ENCODE 3      /* entry words and residue of transmitted elements */
#define ADACOMP_STAGE_DECODE_COUNT 4
#define ADACOMP_STAGE_DECODE_BASE 5
#define ADACOMP_STAGE_DECODE_APPLY 6
#define ADACOMP_STAGE_COMPRESS_CALL 7  /* a whole adacomp_compress call, gaps between kernels included
                                          (a small-table or two-kernel finish's last kernel is
                                          recorded under stage 3, a single launch only here) */
#define ADACOMP_STAGE_DECODE_CALL 8    /* a whole adacomp_decode_accumulate call */
#define ADACOMP_STAGE_DECODE_SGD_CALL 9  /* a whole adacomp_decode_sgd call (its kernels: stages 4-6) */
#define ADACOMP_STAGE_DECODE_ADAM_CALL 10 /* a whole adacomp_decode_adam call (its kernels: stages 4-6) */
#define ADACOMP_NUM_STAGES 11

/* A timer keeps the HIP events of every call recorded since the last read
 * (one per stage boundary); one timer may serve calls on several streams,
 * from one host thread at a time (it has no lock). */
int adacomp_timer_create(adacomp_timer** timer);
int adacomp_timer_destroy(adacomp_timer* timer);
/* Wait for every recorded event, then report per stage the summed
 * milliseconds and the number of launches since the last reset.  On
 * ADACOMP_ERR_HIP the calls read so far stay counted and the call whose
 * events failed is dropped. */
int adacomp_timer_read(adacomp_timer* timer, double* ms, uint64_t* launches, uint32_t nstages);
int adacomp_timer_reset(adacomp_timer* timer);

/* ------------------------------------------------------------------------
 * Operators of the training step around the compressor: the optimizer step on
 * the flat buffers decode writes, layer norm and the gated linear recurrence,
 * each with its gradient.  The conventions above hold (device pointers of the
 * current device, asynchronous on `stream`, errors found on the host before
 * anything is enqueued, nothing allocated, deterministic); additions are
 * named at each call.  An output buffer must not overlap any other buffer of
 * the call; views of the gated scan may be parts of the same rows. */

/* Element types of the operators' activations and gradients. */
#define ADACOMP_FLOAT 0
#define ADACOMP_BFLOAT 1
#define ADACOMP_HALF 2

/* One tensor of an optimizer's table: numel consecutive elements of the flat
 * buffers from element `offset` (a multiple of 4), its decoupled weight decay
 * and its factor on the learning rate. */
typedef struct adacomp_tensor {
    uint64_t offset;
    uint64_t numel;
    float weight_decay;
    float lr_scale;
} adacomp_tensor;

typedef struct adacomp_optimizer_info {
    uint64_t ntensors;
    uint64_t total_numel;
    uint64_t span;                 /* max(offset + numel) rounded up to a multiple of 4 */
    uint64_t nblocks;              /* sum over tensors of ceil(numel / ADACOMP_MOMENT_BLOCK) */
    uint64_t norm_workspace_bytes; /* ws of adacomp_grad_norm */
} adacomp_optimizer_info;

typedef struct adacomp_optimizer adacomp_optimizer; /* opaque, immutable once created */

/* Host-only: validate a table and report its sizes.  ERR_INVALID_ARGUMENT for
 * an empty table, a tensor without elements or a factor that is not finite;
 * ERR_MISALIGNED, ERR_OVERLAP and ERR_TOO_LARGE as for a segment table. */
int adacomp_optimizer_query(const adacomp_tensor* tensors, uint32_t ntensors,
                            adacomp_optimizer_info* info);
/* Validate the table and copy its work tiles to the current device. */
int adacomp_optimizer_create(const adacomp_tensor* tensors, uint32_t ntensors,
                             adacomp_optimizer** optimizer);
int adacomp_optimizer_destroy(adacomp_optimizer* optimizer);
int adacomp_optimizer_get_info(const adacomp_optimizer* optimizer, adacomp_optimizer_info* info);

/* Norm of the scaled gradient over every tensor of the table, and the factor
 * that brings it down to max_norm:
 *   clip[0] = scale * sqrt(sum g^2),  clip[1] = clip[0] > max_norm ? max_norm / clip[0] : 1
 * summed, divided and compared in float64, each rounded once to float32.  A
 * norm of NaN gives the factor 1, an infinite one 0.
 *   grad  [span] of grad_type, read only; 16-byte aligned; elements outside
 *         every tensor do not count.
 *   clip  device float32[2] (8-byte aligned).
 *   ws    16-byte aligned, ws_bytes >= info.norm_workspace_bytes; no initial
 *         contents required. */
int adacomp_grad_norm(const adacomp_optimizer* optimizer, const void* grad, int grad_type,
                      uint64_t n_elems, float max_norm, float scale, float* clip, void* ws,
                      uint64_t ws_bytes, void* stream);

/* One AdamW step.  Per element of tensor i, with lr_i = lr * lr_scale_i:
 *   g = grad * scale * (clip ? clip[1] : 1)
 *   m = beta1 * m + (1 - beta1) * g;   v = beta2 * v + (1 - beta2) * (g * g)
 *   w = w * (1 - lr_i * weight_decay_i)
 *         - lr_i / (1 - beta1^step) * (m / (sqrt(v) / sqrt(1 - beta2^step) + eps))
 * 1 - beta, the bias corrections, lr_i, the step size lr_i / (1 - beta1^step)
 * and the decay factor are formed in float64, each rounded once.  step >= 1
 * counts the calls made so far, this one included; it and lr are values of the
 * call, so a captured step replays with the same ones. */
typedef struct adacomp_adamw {
    float lr;
    float beta1;
    float beta2;
    float eps;
    float scale;
    uint32_t step;
} adacomp_adamw;

/* The step with float32 moments.
 *   weights, m, v  [span] float32, updated in place.
 *   grad           [span] of grad_type, read only.
 *   weights_bf16   nullable [span] bfloat16: the new weights rounded once.
 *   clip           nullable device float32[2], as adacomp_grad_norm writes it.
 * Every [span] buffer is 16-byte aligned; elements outside every tensor are
 * not written. */
int adacomp_adamw_step(const adacomp_optimizer* optimizer, float* weights, const void* grad,
                       int grad_type, float* m, float* v, void* weights_bf16, uint64_t n_elems,
                       const adacomp_adamw* adamw, const float* clip, void* stream);

/* The step with moments in 8 bits: blocks of ADACOMP_MOMENT_BLOCK consecutive
 * elements of one tensor (the last one shorter) share one power-of-two scale
 * for each moment, and an element holds an e4m3 code of m and one of v.
 *   m_codes, v_codes  [span] bytes, 16-byte aligned: value = e4m3(code) * 2^(scale - 127).
 *   scales            [2 * info.nblocks] bytes, 16-byte aligned: of block b (tensors
 *                     in table order), m's at 2b and v's at 2b + 1.  All zeros
 *                     is the state before the first step.
 * g, m and v are formed in float64 (the weights' step from them in float32, its
 * root and quotient to a unit in the last place each) and rounded once: the scale is the smallest in 0..254 under which the
 * block's largest magnitude, cut to 20 fraction bits, is at most 448; each
 * magnitude, cut to a multiple of 2^-17 of its code's step, is rounded up with
 * the probability of its remainder.  The random bits of an element are a hash
 * of its index, seed and step, so the same call gives the same codes whatever
 * the table around it.  A v above zero never becomes zero; what no code
 * holds, and NaN, becomes NaN. */
#define ADACOMP_MOMENT_BLOCK 32u
int adacomp_adamw_packed_step(const adacomp_optimizer* optimizer, float* weights,
                              const void* grad, int grad_type, void* m_codes, void* v_codes,
                              void* scales, void* weights_bf16, uint64_t n_elems,
                              const adacomp_adamw* adamw, uint32_t seed, const float* clip,
                              void* stream);

/* Layer norm over the last axis of `rows` rows of `cols` elements:
 *   mean = sum x / cols,  rstd = 1 / sqrt(sum (x - mean)^2 / cols + eps)
 *   y = (x - mean) * rstd * weight + bias
 * in float32 whatever the type, y rounded once.
 *   x, y          rows of `type`, x_stride and y_stride (>= cols) elements apart;
 *                 aligned to their element.
 *   weight, bias  nullable [cols] float32 (absent: 1, 0).
 *   mean, rstd    nullable [rows] float32 outputs, as the backward pass takes them.
 * rows = 0 is no work.  ERR_TOO_LARGE for more than ADACOMP_NORM_MAX_COLS
 * columns, 2^32 rows and more, 2^22 rows and more of over 16384 columns, or a
 * matrix that reaches past 2^40 elements. */
#define ADACOMP_NORM_MAX_COLS 65536u
int adacomp_layer_norm(const void* x, uint64_t x_stride, const float* weight, const float* bias,
                       void* y, uint64_t y_stride, float* mean, float* rstd, uint64_t rows,
                       uint32_t cols, int type, float eps, void* stream);

/* Its gradients, with xhat = (x - mean) * rstd and g = dy * weight:
 *   dx = rstd * (g - sum g / cols - xhat * sum (g * xhat) / cols)
 *   dweight = sum over rows of dy * xhat,  dbias = sum over rows of dy
 * in float32, the sums over rows joined in float64 in a fixed order.
 *   weight          nullable (1).
 *   dweight, dbias  [cols] float32, both or neither (NULL: not computed);
 *                   with rows = 0 they become zero.
 *   ws              16-byte aligned, ws_bytes >= adacomp_layer_norm_workspace_bytes(rows,
 *                   cols); not used, and may be NULL, without dweight and dbias.  No
 *                   initial contents required.
 * ERR_TOO_LARGE as above, but from over 8192 columns on for 2^22 rows. */
int adacomp_layer_norm_backward(const void* dy, uint64_t dy_stride, const void* x,
                                uint64_t x_stride, const float* weight, const float* mean,
                                const float* rstd, void* dx, uint64_t dx_stride, float* dweight,
                                float* dbias, uint64_t rows, uint32_t cols, int type, void* ws,
                                uint64_t ws_bytes, void* stream);
int adacomp_layer_norm_workspace_bytes(uint64_t rows, uint32_t cols, uint64_t* bytes);

/* Gated linear recurrence along the sequence, per sequence b and channel c:
 *   h_t = a_t * h_(t-1) + k_t * x_t,   t = 0 .. n_b - 1
 *   sigmoid = 1:  a = 1 / (1 + exp(-gate)),  k = 1 / (1 + exp(gate))  (= 1 - a)
 *   sigmoid = 0:  a = gate,  k = 1
 * states in float32, and a and k within 8 of its half units in the last place
 * (a no smaller than 1.6e-38 whatever the gate, k 0 below 1.2e-38).  The
 * sequence is cut into tiles whose gate products are formed and joined, so with
 * sigmoid = 0 the products of consecutive gates, however many, have to stay
 * below float32's largest number (gates in [-1, 1] always do).  Products below
 * its normal numbers keep an absolute error of 2^-149, and are 0 only where a
 * gate is.
 * ERR_TOO_LARGE: length or batch * channels from 2^31 on, batch or channels
 * from 2^24 on, time strides from 2^32 or batch strides from 2^40 on, or 2^32
 * work-items and more: one for each 8 steps (backward with the sigmoid) or 16
 * of 4 bytes of adjacent channels, whole tiles counted. */
typedef struct adacomp_scan_shape {
    uint64_t length;      /* steps, n_b <= length; may be 0 */
    uint32_t batch;       /* sequences; may be 0 */
    uint32_t channels;    /* >= 1 */
    int type;             /* element type of gate, x, h and their gradients */
    int sigmoid;          /* 0 or 1 */
} adacomp_scan_shape;

/* A [batch, length, channels] tensor whose channels are adjacent; strides in
 * elements, time_stride >= channels.  Aligned to its element. */
typedef struct adacomp_view {
    void* data;
    uint64_t batch_stride;
    uint64_t time_stride;
} adacomp_view;

/* Forward.
 *   gate, x   inputs;  h  output, zero at steps from n_b on.
 *   h0        nullable [batch, channels] float32: the state before step 0 (NULL: 0).
 *   h_last    nullable [batch, channels] float32 output: the state after the
 *             last step (h0 for an empty sequence).
 *   lengths   nullable device int32[batch]: n_b, taken into 0 .. length; what lies at
 *             steps from n_b on is not used, whatever it holds.  NULL: length.
 *   ws        16-byte aligned, ws_bytes >= adacomp_gated_scan_workspace_bytes(shape);
 *             no initial contents required. */
int adacomp_gated_scan(const adacomp_scan_shape* shape, const adacomp_view* gate,
                       const adacomp_view* x, const adacomp_view* h, const float* h0,
                       float* h_last, const int32_t* lengths, void* ws, uint64_t ws_bytes,
                       void* stream);

/* Gradients, from the states h that the forward call wrote:
 *   l_t = dh_t + a_(t+1) * l_(t+1),  dh_last added at the last step
 *   dx = l * k;  sigmoid = 1: dgate = l * (h_(t-1) - x) * a * k, 0: dgate = l * h_(t-1)
 *   dh0 = a_0 * l_0   (dh_last for an empty sequence)
 *   x        not read, and may be NULL, with sigmoid = 0.
 *   dgate, dx  outputs, zero at steps from n_b on.
 *   h0, dh_last  nullable (0);  dh0  nullable output. */
int adacomp_gated_scan_backward(const adacomp_scan_shape* shape, const adacomp_view* gate,
                                const adacomp_view* x, const adacomp_view* h,
                                const adacomp_view* dh, const adacomp_view* dgate,
                                const adacomp_view* dx, const float* h0, const float* dh_last,
                                float* dh0, const int32_t* lengths, void* ws, uint64_t ws_bytes,
                                void* stream);
int adacomp_gated_scan_workspace_bytes(const adacomp_scan_shape* shape, uint64_t* bytes);

const char* adacomp_status_str(int status);

#ifdef __cplusplus
}
#endif

#endif /* ADACOMP_H */

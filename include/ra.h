/*
 * ra.h -- C ABI of the GB300 ring-attention forward library (libra.so).
 *
 * What the library computes (ring attention, forward):
 *   Q, K and V are split along the sequence into N shards.  Shard p keeps its
 *   query block; at ring step t = 0..N-1 it meets the K/V block of shard
 *   r = (p - t) mod N ("device i -> i+1" rotation: "3.6 Distributed Training II",
 *   section "Ring Attention"; the Q&A page "Explain ring attention ...", section
 *   "The ring").  Each block is folded into a running max m, running sum l and
 *   output accumulator o by the online-softmax update of "Module 23: Distributed
 *   Training", section "The Math: One Block at a Time"; at the end O = o / l.
 *   Causal attention skips blocks strictly in the future of a query tile and
 *   masks the rest key by key on global positions (Module 23, "Exact by
 *   Construction"); the diagonal is kept (key position <= query position).
 *
 *   One GPU runs all N shards: the ring rotation becomes the order in which
 *   each query tile visits K/V tiles.  There are no inter-GPU transfers.
 *
 * Tensor conventions shared by every entry point:
 *   - Q, O:   [B, Hq,  S, d] row-major, contiguous.
 *   - K, V:   [B, Hkv, S, d] row-major, contiguous.
 *   - LSE:    [B, Hq,  S] float32, natural-log log-sum-exp of the scaled,
 *             masked scores of each row (the pages return O only; the LSE is
 *             what lets partial results be merged).
 *   - The S axis is in LAYOUT ORDER: shard p occupies rows [p*S/N, (p+1)*S/N),
 *     and row p*S/N + i holds the token at natural position pos(p, i):
 *       contiguous: p*S/N + i
 *       striped:    i*N + p                 (Module 23, "The Causal Imbalance --
 *                                            and the Striped Fix")
 *       zigzag:     with c = S/(2N): i < c ? p*c + i : (2N-1-p)*c + (i - c)
 *                   (reading of "the same idea, paired up block-by-block": chunk p
 *                   paired with chunk 2N-1-p)
 *     ra_layout_perm converts natural order <-> layout order.
 *   - GQA: query head h reads key/value head h / (Hq/Hkv).
 *   - Scores are s = scale * q.k with scale = 1/sqrt(d) unless given.
 *
 * Ownership: the caller owns every device buffer passed in.  A plan owns its
 * host tables, its device work tables (whole forward, one per ring step, backward),
 * its device status word, a stream for its own allocations and frees, three CUDA
 * events for ra_ring_fwd, and one event per stream its kernels were launched on;
 * ra_fwd, ra_fwd_step, ra_ring_rotate, ra_ring_fwd, ra_bwd, ra_merge_partials and
 * ra_layout_perm allocate no device memory ("allocates nothing" below: the first
 * launch of a plan on a stream it has not used creates that stream's event) and are
 * asynchronous on the given stream (a cudaStream_t passed as void*; NULL = legacy
 * default).
 *
 * Errors: every call returns an ra_status; on failure ra_last_error() returns a
 * thread-local message.  Arguments are checked before anything is launched.
 * Every device buffer must be memory of the CURRENT device (or managed memory)
 * and every stream must belong to it: the kernels run on the current device, so
 * a buffer of another device or a host pointer is rejected with
 * RA_ERR_INVALID_ARG before any launch (RA_ERR_NO_DEVICE when no device exists).
 * Uneven shards are rejected, never padded (Module 23, "Common Pitfalls":
 * reject uneven shards rather than silently bias the result).
 */
#ifndef RA_H_
#define RA_H_

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  RA_OK = 0,
  RA_ERR_INVALID_ARG = 1,  /* null/misaligned pointer, bad size, uneven shards */
  RA_ERR_UNSUPPORTED = 2,  /* valid problem outside what the kernels handle      */
  RA_ERR_CUDA = 3,         /* a CUDA runtime call or launch failed               */
  RA_ERR_TIMEOUT = 4,      /* a device-side wait exceeded its budget (~1 s)      */
  RA_ERR_NO_DEVICE = 5,    /* the plan has no device state (no GPU at plan time) */
  RA_ERR_BOUNDS = 6        /* debug build only: a kernel's bounds check failed    */
} ra_status;

typedef enum {
  RA_LAYOUT_CONTIGUOUS = 0,
  RA_LAYOUT_STRIPED = 1,
  RA_LAYOUT_ZIGZAG = 2
} ra_layout;

typedef enum {
  RA_DTYPE_F32 = 0,   /* float32 Q/K/V/O; SIMT kernel, d <= 128              */
  RA_DTYPE_BF16 = 1   /* bfloat16 Q/K/V/O; tensor-core kernel, d == 128      */
} ra_dtype;

/* One attention problem.  All sizes are element counts. */
typedef struct {
  int64_t batch;     /* B  >= 1                                            */
  int64_t seq;       /* S  >= 1, multiple of n_shards (2*n_shards: zigzag) */
  int32_t heads_q;   /* Hq >= 1, multiple of heads_kv                      */
  int32_t heads_kv;  /* Hkv >= 1                                           */
  int32_t head_dim;  /* d: 128 for BF16; 1..128 for F32                    */
  int32_t n_shards;  /* N >= 1                                             */
  int32_t layout;    /* ra_layout                                          */
  int32_t causal;    /* 0 or 1                                             */
  int32_t dtype;     /* ra_dtype                                           */
  float scale;       /* score scale; 0 selects 1/sqrt(head_dim)            */
} ra_problem;

typedef struct ra_plan_s* ra_plan_t;

/*
 * ra_plan -- validate a problem and build its ring schedule.
 * Builds, on the host, the per-shard tile classification (FULL / PARTIAL / SKIP,
 * see ra_plan_tile_counts) and, for BF16 problems, the work lists of the
 * tensor-core kernels: the whole forward (ra_fwd), one list per ring step
 * (ra_fwd_step), the gathered forward (ra_fwd_gathered) and the two backward
 * passes (ra_bwd), each in longest-first order with key/value heads grouped.  It
 * also picks each kernel's schedule: synchronised rounds when one key/value head's
 * K and V exceed 32 MiB, otherwise items handed out as CTAs free up.  When a CUDA
 * device is current, it uploads the work tables and allocates the plan's device
 * status word (stream-ordered, on a stream of the plan's own; the call returns once
 * they are in place), and creates the three events ra_ring_fwd orders its streams
 * with.  Without a
 * device the plan is host-only: tile counts work, the compute calls return
 * RA_ERR_NO_DEVICE.
 * *out receives the plan; release it with ra_plan_destroy.
 * Errors: RA_ERR_INVALID_ARG (null pointers, sizes < 1, S % N, zigzag S % 2N,
 * Hq % Hkv, bad enum), RA_ERR_UNSUPPORTED (BF16 with d != 128, F32 with d > 128,
 * more than 2^31 rows, more than 32767 shards; a plan too large to build on the
 * host: N^2 x query tiles per shard above 2^30, BF16 work lists above 2^27
 * entries, or a host allocation that failed), RA_ERR_CUDA (device upload failed).
 */
ra_status ra_plan(const ra_problem* prob, ra_plan_t* out);

/*
 * ra_plan_window -- a plan in which a query sees only the last `window` keys up to its
 * own position and the first `sinks` keys of the sequence: key j is visible to query i
 * (global positions) when j <= i and (j > i - window or j < sinks).  The pages' causal
 * attention sees the whole prefix; this is its windowed form for sequences whose full
 * prefix is not wanted.  Every entry point that takes a plan accepts it, with the same
 * tensors: ra_fwd (fused and partials), ra_fwd_step, ra_ring_fwd, ra_fwd_gathered,
 * ra_bwd.  Key tiles that no query of a query tile sees are neither read nor computed.
 * prob: as for ra_plan, with causal 1.
 * window: >= 1; a window of at least seq is the whole causal prefix.
 * sinks: >= 0; any value from seq on is the whole causal prefix as well.
 * ra_plan_tile_counts on it: FULL when every query of the tile sees every key, PARTIAL
 * for the other key tiles within reach of the query tile, SKIP for the rest.
 * K and V (and Q and dO in ra_bwd) must be finite: a key that a query does not see
 * enters its products with weight zero where it shares a tile with keys that are seen,
 * and zero times an infinity or a NaN is a NaN.  A row of Q that is not finite leaves its
 * own row of O and LSE undefined, in ra_fwd as under ra_plan, and no other.
 * Its LSE is that of the unrounded weights.  Its kernels hold no counters: calls that
 * share the plan may be captured into graphs (keep the plan while a graph of them lives).
 * Errors: as ra_plan, and RA_ERR_INVALID_ARG (causal 0, window < 1, sinks < 0),
 * RA_ERR_UNSUPPORTED (seq above 2^30; BF16: window + sinks, within seq, above 2^24 over
 * max(1, Hq / Hkv / 2)).
 */
ra_status ra_plan_window(const ra_problem* prob, int64_t window, int64_t sinks, ra_plan_t* out);

/* Release a plan and its device memory.  NULL is accepted.  It does not wait:
 * kernels queued with this plan may still read its tables, so the plan records
 * an event on every stream it launched on (after its latest launch there), and
 * the frees of its device memory are queued in stream order behind those events
 * only (cudaFreeAsync on the plan's own stream; the plan allocated its tables
 * with cudaMallocAsync).  Other streams' work and other plans' kernels are not
 * waited for.  Do not use the plan after this call.  It does not clear a pending
 * CUDA error. */
ra_status ra_plan_destroy(ra_plan_t plan);

/*
 * ra_plan_tile_counts -- per-shard causal tile classification of the schedule.
 * For one (batch entry, query head), counts over all N ring steps the pairs
 * (128-row query tile of shard p, 128-row key tile of the block met at step t)
 * that are FULL (every (q,k) pair causal), PARTIAL (some) or SKIP (none),
 * following Module 23's per-device causal work count ("The Causal Imbalance")
 * at tile granularity.  The last tile of a shard may be shorter than 128.
 * Non-causal problems count every tile FULL.  full, partial and skip are
 * caller-owned host arrays of n_shards int64 each (any may be NULL).
 */
ra_status ra_plan_tile_counts(ra_plan_t plan, int64_t* full, int64_t* partial, int64_t* skip);

/*
 * ra_fwd -- ring-attention forward on the plan's problem.
 * q, k, v: device pointers, layout order, dtype of the plan, 16-byte aligned.
 * Fused mode (o_parts == lse_parts == NULL):
 *   o   [B, Hq, S, d] in the plan's dtype (required);
 *   lse [B, Hq, S] float32 (may be NULL).
 * Partials mode (o_parts and lse_parts non-NULL, o == lse == NULL):
 *   o_parts   [N, B, Hq, S, d] float32 and lse_parts [N, B, Hq, S] float32;
 *   entry t of a row of shard p is attention of that row over the key block of
 *   shard (p - t) mod N alone, normalised by its own sum; a block with no causal
 *   key gives O_t = 0, LSE_t = -inf.  ra_merge_partials combines them.
 * Asynchronous on stream; allocates nothing.  A device-side wait that runs out
 * of budget makes the kernel return early and sets the plan's status word;
 * ra_sync_status reports it.  Calls that share a plan must not overlap on the
 * GPU (the plan's device words hold the status and the work-item counter).
 * Errors: RA_ERR_INVALID_ARG (null/misaligned pointers, mixed modes),
 * RA_ERR_NO_DEVICE, RA_ERR_CUDA (launch failure).
 */
ra_status ra_fwd(ra_plan_t plan, const void* q, const void* k, const void* v,
                 void* o, float* lse, float* o_parts, float* lse_parts, void* stream);

/*
 * ra_fwd_step -- one ring step for every shard, run as the device holding the shard
 * runs it: each shard attends to the K/V block it holds at that step.
 * At step t shard p holds the block that started on shard (p - t) mod N, passed
 * on one device per step (device i -> i+1: "3.6 Distributed Training II",
 * section "Ring Attention"; the Q&A page, section "The ring").
 * step: t in [0, N).
 * q: [B, Hq, S, d] in layout order.
 * k_blk, v_blk: [B, Hkv, S, d] receive buffers.  The rows of shard p, [p*S/N, (p+1)*S/N),
 *   hold the block shard p holds at step t: K/V themselves at t = 0, then what t
 *   calls of ra_ring_rotate have passed along.
 * o_part [B, Hq, S, d] float32 and lse_part [B, Hq, S] float32 receive the
 *   attention of every row over that block alone, with the conventions of
 *   ra_fwd's partials mode: normalised by its own sum; O_t = 0 and LSE_t = -inf
 *   where the block has no causal key.  The result equals entry t of ra_fwd's
 *   partials.
 * Device pointers in the plan's dtype (o_part/lse_part float32), 16-byte aligned.
 * Asynchronous on stream; allocates nothing; the plan holds one work list per step.
 * Calls that share a plan must not overlap on the GPU.
 * Errors: RA_ERR_INVALID_ARG (step out of range, null/misaligned pointers),
 * RA_ERR_NO_DEVICE, RA_ERR_CUDA.
 */
ra_status ra_fwd_step(ra_plan_t plan, int32_t step, const void* q, const void* k_blk,
                      const void* v_blk, float* o_part, float* lse_part, void* stream);

/*
 * ra_ring_rotate -- the ring's exchange, in which every shard passes its K/V block on
 * to the next: for each [S, d] matrix of K and V ([B, Hkv, S, d], plan dtype), the
 * rows of shard (p + 1) mod N in the destination receive the rows of shard p in the
 * source (device i -> i+1; "3.6 Distributed Training II", "Ring Attention").
 * The copies are copy-engine transfers, two per tensor (strided over B*Hkv), so
 * they can run on a second stream while a forward kernel occupies every SM.  That
 * is one GPU's stand-in for the send/receive that overlaps compute between devices.
 * k_src, v_src, k_dst, v_dst: device pointers.  A destination must not overlap its
 * source or the other destination.  Asynchronous on stream; allocates nothing.
 * Errors: RA_ERR_INVALID_ARG (null pointers, overlap), RA_ERR_NO_DEVICE, RA_ERR_CUDA.
 */
ra_status ra_ring_rotate(ra_plan_t plan, const void* k_src, const void* v_src, void* k_dst,
                         void* v_dst, void* stream);

/*
 * ra_ring_fwd -- the explicit ring driver.  It runs N calls of ra_fwd_step on
 * `stream`.  While step t computes, ra_ring_rotate passes the block of step t on
 * to the receive buffer of step t+1, on `comm_stream`: the overlap of
 * communication with compute that "3.6 Distributed Training II", "Ring
 * Attention", describes.  Then it merges the N partials with ra_merge_partials
 * (Module 23, "The Math: One Block at a Time": the fold is order independent).
 * q, k, v: as for ra_fwd.
 * o [B, Hq, S, d] (plan dtype) and lse [B, Hq, S] float32 (may be NULL) receive
 *   the fused result.
 * k_buf, v_buf: caller-owned scratch, two receive buffers each: [2, B, Hkv, S, d]
 *   in the plan's dtype.  They must not overlap each other or K/V.  May be NULL
 *   when N == 1.
 * o_parts [N, B, Hq, S, d] and lse_parts [N, B, Hq, S]: caller-owned float32
 *   scratch for the per-step partials; they hold them after the call.
 * stream: the compute stream.  comm_stream: the rotation stream; it may equal
 *   stream, and then nothing overlaps.  The driver orders both streams with three
 *   events that the plan owns.  Work already queued on stream comes before the
 *   rotations; later work on stream comes after the driver's work on both streams.
 * Asynchronous; allocates nothing.  Calls that share a plan must not overlap.
 * Errors: as ra_fwd_step, ra_ring_rotate and ra_merge_partials.
 */
ra_status ra_ring_fwd(ra_plan_t plan, const void* q, const void* k, const void* v, void* o,
                      float* lse, void* k_buf, void* v_buf, float* o_parts, float* lse_parts,
                      void* stream, void* comm_stream);

/*
 * ra_bwd -- gradients of the ring-attention forward (dQ, dK, dV from dO).
 * The pages present ring attention as a way to train on long sequences (the
 * activations of every layer are kept for the backward pass: "3.6 Distributed
 * Training II", section "Ring Attention") but print no backward pass; this one
 * differentiates the forward's definition O = softmax(scale * Q K^T + M) V:
 *   P = exp(scale * Q K^T + M - LSE)   (recomputed from the forward's LSE)
 *   dV = P^T dO,  dP = dO V^T,  dS = P * (dP - D),  D = rowsum(dO * O),
 *   dQ = scale * dS K,  dK = scale * dS^T Q,
 * with a key/value head's dK and dV summed over the query heads that read it.
 * The work follows the ring: a query tile of shard p meets the key blocks of
 * shards (p - t) mod N (as in the forward); a key block of shard r meets the
 * queries of shard (r + t) mod N at step t, so its gradients gather where the
 * block travels.
 * q, k, v, o, dout (dO): as for ra_fwd (layout order, plan dtype); o and lse
 *   are the forward's outputs for the same q, k, v.
 * dq [B, Hq, S, d], dk and dv [B, Hkv, S, d]: outputs, plan dtype.
 * scratch: caller-owned float32 device buffer of ra_bwd_scratch_size bytes (per
 *   query row LSE * log2(e) and D, in blocks of 64 rows of one shard).
 * Device pointers, 16-byte aligned.  Asynchronous on stream; allocates nothing.
 * A device-side wait that runs out of budget is reported by ra_sync_status.
 * Calls that share a plan must not overlap on the GPU.
 * Errors: RA_ERR_INVALID_ARG (null/misaligned pointers), RA_ERR_NO_DEVICE,
 * RA_ERR_CUDA.
 */
ra_status ra_bwd(ra_plan_t plan, const void* q, const void* k, const void* v, const void* o,
                 const float* lse, const void* dout, void* dq, void* dk, void* dv, float* scratch,
                 void* stream);

/*
 * ra_bwd_scratch_size -- bytes of the scratch buffer ra_bwd needs for this plan:
 * 512 bytes per 64-row block of every (batch, query head, shard), about
 * 8 * B * Hq * S bytes; for a windowed BF16 plan also the fp32 partial sums of the key
 * tiles that are cut (those that hold sinks, and all of a small problem's).  Host only.  Errors: RA_ERR_INVALID_ARG (null arguments).
 */
ra_status ra_bwd_scratch_size(ra_plan_t plan, int64_t* bytes);

/*
 * ra_allgather_kv -- the all-gather of the all-gather variant of context parallelism:
 * every device gathers the K/V blocks of all shards instead of passing them around
 * a ring ("3.6 Distributed Training II", section "Ring Attention": the Llama 3
 * paper's context parallelism for long-context training, with an all-gather of K/V
 * rather than a ring).  One GPU keeps one gathered copy: k_all, v_all
 * [B, Hkv, S, d] receive K and V in NATURAL order (row = token position).
 * k, v: [B, Hkv, S, d] in layout order.  Device pointers, plan dtype, 16-byte
 * aligned; a destination must not overlap its source or the other destination.
 * Asynchronous on stream; allocates nothing.
 * Errors: RA_ERR_INVALID_ARG (null/misaligned pointers, overlap), RA_ERR_NO_DEVICE,
 * RA_ERR_CUDA.
 */
ra_status ra_allgather_kv(ra_plan_t plan, const void* k, const void* v, void* k_all, void* v_all,
                          void* stream);

/*
 * ra_fwd_gathered -- the forward of the all-gather variant: every query row of
 * shard p attends over the gathered K/V in one step, causal by position (the keys
 * at or before its own position; Module 23, "Exact by Construction").  The result
 * is the same attention as ra_fwd; only the data movement differs.
 * q: [B, Hq, S, d] in layout order; k_all, v_all: [B, Hkv, S, d] in natural order
 * (ra_allgather_kv); o [B, Hq, S, d] (plan dtype) and lse [B, Hq, S] float32 (may be
 * NULL) in layout order.  Device pointers, 16-byte aligned.  Asynchronous on stream;
 * allocates nothing.  Calls that share a plan must not overlap on the GPU.
 * Errors: RA_ERR_INVALID_ARG (null/misaligned pointers), RA_ERR_NO_DEVICE, RA_ERR_CUDA.
 */
ra_status ra_fwd_gathered(ra_plan_t plan, const void* q, const void* k_all, const void* v_all,
                          void* o, float* lse, void* stream);

/*
 * ra_ulysses_a2a -- DeepSpeed-Ulysses' all-to-all for N devices (the Q&A page
 * "Explain ring attention ...", section "Related approaches": split by attention
 * heads with an all-to-all instead of a ring).  Each device starts with its
 * sequence shard of every head; the exchange hands device p' every token, by
 * position, of heads p'*H/N .. (p'+1)*H/N - 1, where it runs ordinary attention over
 * the whole sequence (ra_fwd with a plan of batch N*B, H/N heads, one shard); the
 * reverse exchange returns O (and the LSE) to the sequence shards.
 * direction 0 (sequence -> heads): src [B, H, S, row] in layout order (shard p =
 *   rows [p*S/N, (p+1)*S/N)), dst [N, B, H/N, S, row] (device p', natural order).
 * direction 1 (heads -> sequence): src [N, B, H/N, S, row], dst [B, H, S, row].
 * row_bytes: 256 (d = 128 bf16) or 4 (the float32 LSE).  heads: H, a multiple of N.
 * Device pointers, 16-byte aligned, not overlapping.  Asynchronous; allocates nothing.
 * Errors: RA_ERR_INVALID_ARG (uneven shards, heads % N, direction, pointers),
 * RA_ERR_UNSUPPORTED (row_bytes, more than 2^31-1 rows), RA_ERR_CUDA.
 */
ra_status ra_ulysses_a2a(int32_t direction, int32_t layout, int64_t seq, int32_t n_shards,
                         int64_t batch, int32_t heads, int32_t row_bytes, const void* src, void* dst,
                         void* stream);

/*
 * ra_merge_partials -- exact combination of partial attention results.
 * For each of `rows` rows: LSE = ln sum_t e^(LSE_t), O = sum_t e^(LSE_t - LSE) O_t
 * (order independence of the online-softmax fold, Module 23, "The Math: One
 * Block at a Time").  Parts with LSE_t = -inf are ignored; a row whose parts are
 * all -inf gets O = 0 and LSE = -inf.
 * o_parts [n_parts, rows, d] float32, lse_parts [n_parts, rows] float32, o [rows, d]
 * in o_dtype (F32 or BF16, round-to-nearest-even), lse [rows] float32 or NULL.
 * Device pointers, 16-byte aligned.  Asynchronous on stream; allocates nothing.
 * Errors: RA_ERR_INVALID_ARG (sizes < 1, d > 1024, null/misaligned pointers),
 * RA_ERR_CUDA.
 */
ra_status ra_merge_partials(int32_t n_parts, int64_t rows, int32_t d,
                            const float* o_parts, const float* lse_parts,
                            void* o, int32_t o_dtype, float* lse, void* stream);

/*
 * ra_layout_perm -- move whole rows between natural order and layout order.
 * src and dst are [rows_outer, seq, row_bytes] (e.g. Q as [B*Hq, S, d*2] bytes).
 * inverse == 0: dst[o, j] = src[o, pos(j)]   (natural -> layout order)
 * inverse != 0: dst[o, pos(j)] = src[o, j]   (layout -> natural order)
 * with pos the layout map above.  row_bytes must be a multiple of 4; pointers
 * 16-byte aligned; src and dst must not overlap.  Asynchronous; allocates nothing.
 * Errors: RA_ERR_INVALID_ARG (uneven shards, bad sizes, overlap, alignment),
 * RA_ERR_UNSUPPORTED (seq above 2^31-1, n_shards above 32767, more than 2^63-1 bytes),
 * RA_ERR_CUDA.
 */
ra_status ra_layout_perm(int32_t layout, int64_t seq, int32_t n_shards, int32_t inverse,
                         int64_t rows_outer, int32_t row_bytes,
                         const void* src, void* dst, void* stream);

/*
 * ra_layout_index -- host helper: pos_out[j] = natural position of layout row j,
 * for j in [0, seq).  pos_out is a caller-owned host array of seq int64.
 * Errors: RA_ERR_INVALID_ARG (uneven shards, null pointer, bad layout).
 */
ra_status ra_layout_index(int32_t layout, int64_t seq, int32_t n_shards, int64_t* pos_out);

/*
 * ra_sync_status -- synchronize `stream`, then read and clear the plan's device
 * status word.  Returns RA_ERR_TIMEOUT if a kernel launched with this plan gave
 * up on a device-side wait since the last call, RA_ERR_BOUNDS if (in the debug
 * build, libra_debug.so, compiled with RA_DEBUG_BOUNDS) one of its bounds checks
 * failed, RA_ERR_CUDA on a CUDA error, RA_OK otherwise.
 */
ra_status ra_sync_status(ra_plan_t plan, void* stream);

/*
 * ra_fwd_static -- the bf16 fused forward for callers that cannot allocate.
 * The pages have no counterpart to this entry point; it exists for callers that
 * must not allocate device memory at run time (code running under an allocator
 * or memory pool it may not bypass, or with a device footprint fixed at load
 * time) and therefore cannot create a plan, since ra_plan allocates the work
 * table and status word.  It computes exactly what ra_fwd computes in fused mode
 * for a bf16, head_dim 128 problem, without a plan and without allocating:
 * no cudaMalloc, cudaFree or other allocating routine is called.
 *   - Scratch: the work table and status word live in one file-scope device
 *     array of 4 MiB + 256 B, held on every GPU that loads the library until the
 *     process exits.  Problems needing more than 131072 work items (one item per
 *     pair of 128-row query tiles; e.g. 1M tokens x 32 query heads is exactly
 *     131072), or more than 2^30 (item, ring step) pairs to cost, are rejected
 *     with RA_ERR_UNSUPPORTED.
 *   - Set-up: the first call on a device (with that device current) looks up the
 *     array's device address (a host-side runtime query, made once per device).
 *   - Sharing: every call reuses the array; the status word is cleared at the
 *     start of each call.  Calls whose kernels overlap on the GPU race on the
 *     array and must not be issued; calls from several host threads are
 *     serialised on the host.  Device-side wait timeouts are recorded in the
 *     array's status word, which ra_fwd_static_status reports.
 * prob: the problem (dtype RA_DTYPE_BF16, head_dim 128).  q, k, v, o, lse: as for
 * ra_fwd in fused mode (lse may be NULL), device pointers, 16-byte aligned.
 * Asynchronous on stream.
 * Errors: RA_ERR_INVALID_ARG, RA_ERR_UNSUPPORTED (dtype, head_dim, size),
 * RA_ERR_NO_DEVICE, RA_ERR_CUDA.
 */
ra_status ra_fwd_static(const ra_problem* prob, const void* q, const void* k, const void* v,
                        void* o, float* lse, void* stream);

/*
 * ra_fwd_static_status -- the device-wait status of the latest ra_fwd_static
 * call on the current device.  Like ra_fwd_static, no counterpart on the pages.
 * Synchronizes `stream` (the stream that call ran on), then reads and clears the
 * status word in the static array: RA_ERR_TIMEOUT if that call's kernel gave up
 * on a device-side wait (its O/LSE are then incomplete), RA_ERR_BOUNDS if a
 * bounds check of the debug build failed, RA_OK otherwise or when ra_fwd_static
 * has not run on this device.  It allocates nothing.  The next ra_fwd_static call
 * clears the word, so read it before issuing another.
 * Errors: RA_ERR_TIMEOUT, RA_ERR_BOUNDS, RA_ERR_NO_DEVICE, RA_ERR_CUDA.
 */
ra_status ra_fwd_static_status(void* stream);

/*
 * ra_wait_selftest -- check the failure-detection path of the tensor-core kernels.
 * Not a step of the method.  Every mbarrier wait in the tensor-core kernels gives
 * up after about one second, records a bit in a device status word and lets its
 * kernel return, so that a handshake that never comes ends in RA_ERR_TIMEOUT
 * (ra_sync_status) instead of a hung GPU.  This call runs that wait routine once
 * in a one-warp kernel against an mbarrier that nothing ever arrives on.
 * *status_out (host) receives the status word the wait left: 2 (the MMA-side bit
 * of ra_sync_status's message) when it gave up as designed, 0 if it never did.
 * Later launches in the same context are unaffected.
 * Synchronous, on the legacy default stream of the current device; it takes
 * about one second.  It allocates one 4-byte device word and frees it.
 * Errors: RA_ERR_INVALID_ARG (null status_out), RA_ERR_NO_DEVICE, RA_ERR_CUDA.
 */
ra_status ra_wait_selftest(uint32_t* status_out);

/*
 * ra_kv4_*: a paged key/value cache held in 4 bits, and the attention of new tokens over
 * it.  No counterpart on the pages: after a prompt has gone through ring attention, its
 * keys and values are kept here and the sequence is continued token by token.
 *
 * The cache is one caller-owned device buffer of ra_kv4_cache_size bytes, a pool of
 * `pages` pages of `page_rows` tokens.  Position x of sequence b lies in page
 * page_table[b][x / page_rows] of the pool, at row x % page_rows of it.  Page tables,
 * lengths and counts are device arrays of int32, read by the kernels, so that a captured
 * graph follows them.  Sequences may share pages for reading; a place is written by one
 * row of a call only.
 *
 * Format.  A page holds, for each key/value head, page_rows / 16 blocks of 16 tokens; a
 * block is 20 * d bytes: 16 rows of d/2 bytes of key codes, 16 rows of d/8 bytes of key
 * parameters, the same for the values.  Every 32 channels of a row form a group with two
 * bf16 parameters, scale then low (4 bytes a group, groups in order), computed in float32
 * from the group's values x:
 *   low = bf16(min x),  scale = bf16((max x - low) * r), 0 when that is below 2^-100, with
 *   r the float32 next to 1/15,
 *   code = floor((x - low) / scale + 1/2) in exact arithmetic, held to 0..15 (0 when
 *   scale is 0),  value = low + scale * code.
 * A group with an infinity, a NaN or a range beyond float32 gets scale 0 and low NaN: all
 * of it reads back as NaN.  Codes lie in little-endian nibbles of their row:
 *   keys:   channel c is nibble c % 8 of 32-bit word (c % 32 / 8) * (d/32) + c / 32,
 *   values: channel c is nibble c % 4 of 16-bit word (c % 32 / 4) * (d/32) + c / 32,
 * the order in which the attention kernel's lanes take them.
 *
 * Page indices outside the pool, positions outside the page table and lengths or counts
 * out of range are found by the kernels: such rows are not written, not read back and not
 * attended to, and ra_kv4_sync_status reports
 * them.
 */
typedef struct {
  int64_t pages;      /* pages of the pool, >= 1                                    */
  int32_t page_rows;  /* tokens of a page: a multiple of 16, 16..65536              */
  int32_t heads_q;    /* Hq >= 1, multiple of heads_kv (ra_kv4_attend)              */
  int32_t heads_kv;   /* Hkv >= 1                                                   */
  int32_t head_dim;   /* d: 64 or 128                                               */
  int32_t dtype;      /* ra_dtype of K, V, Q and O                                  */
  int64_t window;     /* as ra_plan_window's; 0: the whole prefix                   */
  int64_t sinks;      /* as ra_plan_window's                                        */
  float scale;        /* score scale; 0 selects 1/sqrt(head_dim)                    */
} ra_kv4_problem;

typedef struct ra_kv4_s* ra_kv4_t;

/*
 * ra_kv4_plan -- validate a cache's description and create its handle, which owns a
 * device status word and one event per stream its kernels were launched on (host-only
 * without a device, as ra_plan).  Release it with ra_kv4_destroy, after the graphs that
 * captured its calls.  One host thread at a time may use a handle; its calls may overlap
 * on the GPU.
 * Errors: RA_ERR_INVALID_ARG (null arguments, sizes < 1, page_rows, Hq % Hkv, window or
 * sinks < 0, bad enum or scale), RA_ERR_UNSUPPORTED (head_dim, more than 2^31-1 pages,
 * a cache beyond 2^62 bytes), RA_ERR_CUDA.
 */
ra_status ra_kv4_plan(const ra_kv4_problem* prob, ra_kv4_t* out);

/* Release a handle (NULL is accepted).  It does not wait, as ra_plan_destroy. */
ra_status ra_kv4_destroy(ra_kv4_t kv);

/* Bytes of the cache buffer: pages * heads_kv * page_rows * d * 5/4.  Host only.
 * Errors: RA_ERR_INVALID_ARG (null arguments). */
ra_status ra_kv4_cache_size(ra_kv4_t kv, int64_t* bytes);

/*
 * ra_kv4_write -- quantise new keys and values into the cache.
 * k, v: [batch, Hkv, rows, d] in the handle's dtype.  Row t of sequence b goes to
 * position first[b] + t, for t < count[b] (count NULL: every row); later rows of a padded
 * batch are not read.  Nothing else of the cache changes.
 * page_table: [batch, table_width] int32; first, count: [batch] int32.
 * Device pointers, 16-byte aligned (page_table, first, count: 4-byte).  Asynchronous on
 * stream; allocates nothing.
 * Errors: RA_ERR_INVALID_ARG (null/misaligned pointers, sizes < 1), RA_ERR_UNSUPPORTED
 * (batch * Hkv * rows above 2^31-1, table_width * page_rows above 2^30),
 * RA_ERR_NO_DEVICE, RA_ERR_CUDA.
 */
ra_status ra_kv4_write(ra_kv4_t kv, void* cache, int64_t batch, int64_t rows, const void* k, const void* v,
                       const int32_t* page_table, int64_t table_width, const int32_t* first,
                       const int32_t* count, void* stream);

/*
 * ra_kv4_read -- read keys and values back as what they stand for: low + scale * code in
 * float32 (the product is exact, the sum rounded), then rounded to the handle's dtype.
 * k, v: [batch, Hkv, rows, d]; row t of sequence b receives position first[b] + t for
 * t < count[b] (count NULL: every row).  Later rows stay as they were (zero_rest 0) or
 * become zeros (1), and so do rows whose page or position is out of range.
 * Everything else as for ra_kv4_write (zero_rest other than 0 or 1: RA_ERR_INVALID_ARG).
 */
ra_status ra_kv4_read(ra_kv4_t kv, const void* cache, int64_t batch, int64_t rows, const int32_t* page_table,
                      int64_t table_width, const int32_t* first, const int32_t* count, int32_t zero_rest,
                      void* k, void* v, void* stream);

/*
 * ra_kv4_attend -- attention of the last `rows` tokens of every sequence over its cached
 * keys and values (the tokens' own among them: write them first).
 * q, o: [batch, Hq, rows, d] in the handle's dtype; lse [batch, Hq, rows] float32 (may be
 * NULL).  length: [batch] int32, the tokens of sequence b that the cache holds; query t
 * sits at position length[b] - rows + t and sees the positions up to its own, within the
 * handle's window and sinks.  A query that sees nothing (length 0, or a position before
 * the first) gets O = 0, LSE = -inf.  Keys beyond a sequence's length are not looked at:
 * what pages hold there does not matter.
 * bf16: Q enters the products as it is and the softmax weights rounded to bf16, each
 * times its value's scale; sums are fp32.  float32: both are split into three bf16 terms,
 * which keep their 24 bits; the fp32 sums run over codes, so that O is off by 5e-7 to 7e-7
 * (relative) where sums over the values themselves give 1e-7 to 3e-7.  A value group's
 * scale (its range / 15) times the largest weight must stay below 2^58, and its values
 * below 2^89 (their weighted sum, not yet divided, is an fp32 number); groups of scales
 * below 2^-52 lose precision relative to themselves.
 * scratch: ra_kv4_attend_scratch_size bytes (NULL when that is 0), not shared by calls
 * that may overlap.  Device pointers, 16-byte aligned (page_table, length: 4-byte).
 * Asynchronous on stream; allocates nothing.
 * Errors: as ra_kv4_write (batch, or Hkv times the 8-row query tiles, above 65535:
 * RA_ERR_UNSUPPORTED).
 */
ra_status ra_kv4_attend(ra_kv4_t kv, const void* cache, int64_t batch, int64_t rows, const void* q,
                        const int32_t* page_table, int64_t table_width, const int32_t* length, void* o,
                        float* lse, float* scratch, void* stream);

/* Bytes of ra_kv4_attend's scratch for these sizes (0 when it needs none).  Host only.
 * Errors: RA_ERR_INVALID_ARG, RA_ERR_UNSUPPORTED as ra_kv4_attend. */
ra_status ra_kv4_attend_scratch_size(ra_kv4_t kv, int64_t batch, int64_t rows, int64_t table_width,
                                     int64_t* bytes);

/*
 * ra_kv4_sync_status -- synchronize `stream`, then read and clear the handle's status
 * word: RA_ERR_INVALID_ARG when a call since the last one met a page index, position,
 * length or count out of range, RA_ERR_CUDA on a CUDA error, RA_ERR_BOUNDS when a bounds
 * check of the debug build failed, RA_OK otherwise.
 */
ra_status ra_kv4_sync_status(ra_kv4_t kv, void* stream);

/*
 * ra_rope_*: rotary positions.  No counterpart on the pages, whose attention takes queries and
 * keys as they come: a model that uses the ring rotates them by their positions in the whole
 * sequence first, which a shard's rows do not show by their place.
 *
 * The first rotary_dim channels of a row form pairs: channels j and j + rotary_dim/2, or
 * interleaved 2j and 2j + 1 (j < rotary_dim/2).  At position n the pair (x1, x2) becomes
 *   A (x1 cos a - x2 sin a),  A (x1 sin a + x2 cos a),  a = n * w_j,
 * and the other channels are copied.  w_j = base^(-2j / rotary_dim), scaled for contexts longer
 * than `original` tokens:
 *   NONE    as it is;
 *   LINEAR  w_j / factor (positions interpolated);
 *   BASE    base * factor^(rotary_dim / (rotary_dim - 2)) in place of base (rotary_dim 2: as it is);
 *   BANDS   t_j w_j + (1 - t_j) w_j / factor, t_j = (r_j - low) / (high - low) held to 0..1, where
 *           r_j = original * w_j / 2 pi are the pair's turns within `original` tokens;
 *   RAMP    (1 - t_j) w_j + t_j w_j / factor, t_j = (j - j0) / (j1 - j0) held to 0..1, where j0 =
 *           max(floor(i(high)), 0), j1 = min(ceil(i(low)), rotary_dim - 1), j1 - j0 at least 0.001,
 *           and i(r) = rotary_dim * ln(original / 2 pi r) / (2 ln base).
 * Speeds are float64, a few 2^-53 of themselves off; position * speed is taken modulo a turn in
 * integers (64-bit fractions of a turn) and cut to 2^-33 of it; products and sums are float32, with
 * one rounding to the dtype.
 */
typedef enum {
  RA_ROPE_NONE = 0,
  RA_ROPE_LINEAR = 1,
  RA_ROPE_BASE = 2,
  RA_ROPE_BANDS = 3,
  RA_ROPE_RAMP = 4
} ra_rope_scaling;

typedef struct {
  int32_t head_dim;     /* d, 2..1024                                           */
  int32_t rotary_dim;   /* channels that are rotated, the first ones: even, <= d */
  int32_t interleaved;  /* 0: channels j and j + rotary_dim/2; 1: 2j and 2j + 1  */
  int32_t dtype;        /* ra_dtype of the rows                                 */
  double base;          /* > 1                                                  */
  int32_t scaling;      /* ra_rope_scaling                                      */
  double factor;        /* >= 1 (scaling other than NONE)                       */
  int64_t original;     /* >= 1 (BANDS, RAMP)                                   */
  double low, high;     /* turns within `original` tokens, 0 < low < high (BANDS, RAMP) */
  double amplitude;     /* A, 2^-126 .. the largest float32; 0 selects 1        */
} ra_rope_problem;

typedef struct ra_rope_s* ra_rope_t;

/*
 * ra_rope_plan -- validate a rotation's description and compute its speeds (in float64).  The
 * handle owns a small device table and one event per stream it was used on (host-only without
 * a device, as ra_plan).  Release it with ra_rope_destroy, after the graphs that captured its
 * calls.  One host thread at a time may use a handle; its calls may overlap on the GPU.
 * Errors: RA_ERR_INVALID_ARG (null arguments, sizes, bad enum, factor or amplitude),
 * RA_ERR_UNSUPPORTED (head_dim above 1024), RA_ERR_CUDA.
 */
ra_status ra_rope_plan(const ra_rope_problem* prob, ra_rope_t* out);

/* Release a handle (NULL is accepted).  It does not wait, as ra_plan_destroy. */
ra_status ra_rope_destroy(ra_rope_t rope);

/*
 * ra_rope -- rotate queries and keys in one launch.
 * q, q_out: [batch, heads_q, seq, d]; k, k_out: [batch, heads_kv, seq, d] (heads_kv 0: none, and
 * NULL pointers).  Each has its own strides (host arrays of 3: batch, head, row, in elements, not
 * negative; the d channels of a row follow each other), so that projections' outputs are read
 * where they lie and the ring's tensors are written in order.  Rows are written once: strides of
 * an output that put two rows in one place are refused, and an output may be its own input (the
 * same pointer and strides), but not overlap an input otherwise.
 * position: [batch, seq] int32, any value; NULL: row i of shard p stands at pos(p, i) of the
 * layout (see above; seq has to divide into its shards), the natural position.
 * Device pointers aligned to their elements (position: 4 bytes); 16-byte aligned rows of
 * rotary_dim and d multiples of 32 bytes go 16 bytes at a time.  Asynchronous on stream;
 * allocates nothing.
 * Errors: RA_ERR_INVALID_ARG (null/misaligned pointers, sizes, strides, layout),
 * RA_ERR_UNSUPPORTED (batch * seq * d above 2^38, more than 2^20 heads), RA_ERR_NO_DEVICE,
 * RA_ERR_CUDA.
 */
ra_status ra_rope(ra_rope_t rope, int64_t batch, int64_t seq, int32_t heads_q, int32_t heads_kv, int32_t layout,
                  int32_t n_shards, const int32_t* position, const void* q, const int64_t* q_strides, const void* k,
                  const int64_t* k_strides, void* q_out, const int64_t* q_out_strides, void* k_out,
                  const int64_t* k_out_strides, void* stream);

/*
 * ra_rope_bwd -- gradients with respect to what ra_rope was given, from those with respect to
 * what it returned: the transposed rotation, A (y1 cos a + y2 sin a), A (y2 cos a - y1 sin a).
 * Everything else as for ra_rope.
 */
ra_status ra_rope_bwd(ra_rope_t rope, int64_t batch, int64_t seq, int32_t heads_q, int32_t heads_kv, int32_t layout,
                      int32_t n_shards, const int32_t* position, const void* dq, const int64_t* dq_strides,
                      const void* dk, const int64_t* dk_strides, void* dq_out, const int64_t* dq_out_strides,
                      void* dk_out, const int64_t* dk_out_strides, void* stream);

/*
 * ra_paged_*: a paged key/value cache in the tensors' own type, filled chunk by chunk, the
 * attention of new tokens over it, and its eviction by accumulated attention weight.  No
 * counterpart on the pages: prompts that arrive in pieces, and sequences continued from them.
 *
 * The cache is one caller-owned device buffer [pages, 2, Hkv, page_rows, d]: a page's keys, then
 * its values.  Slot x of sequence b lies in page page_table[b][x / page_rows], at row
 * x % page_rows.
 *
 * A call takes a packed batch: the new tokens of `batch` sequences one after the other, tensors
 * [tokens, heads, d] with strides of their own (host arrays of 2: token, head, in elements,
 * multiples of 16 bytes).  Sequence b has the tokens offset[b] .. offset[b+1] - 1 (none is fine)
 * and, those among them, length[b] slots in use: its i-th new token has slot length[b] -
 * (offset[b+1] - offset[b]) + i.  Tokens before offset[0] and from offset[batch] on belong to no
 * sequence; nothing is read or written for them.
 * page_table: [batch, table_width] int32; offset: [batch + 1] int32; length: [batch] int32, all
 * on the device and read by the kernels, so that a captured graph follows them.  Sequences may
 * share pages for reading; a place is written by one row of a call only.
 *
 * Offsets that fall or leave 0..tokens, lengths that are negative, smaller than the sequence's
 * new tokens or beyond its page table, and page indices outside the pool are found by the
 * kernels: such sequences are left out (their rows stay as they were), the slots of such pages
 * are not written, not moved and not attended to, and ra_paged_sync_status reports them.
 * (Offsets that fall can name a token twice: ra_paged_append writes it for the first of its
 * sequences, and what the other calls leave for it is that of either.)
 * Entries of the page table for slots that no token of the call sees are not read.
 */
typedef struct {
  int64_t pages;      /* pages of the pool, >= 1                                    */
  int32_t page_rows;  /* slots of a page: a multiple of 16, 16..65536               */
  int32_t heads_q;    /* Hq >= 1, multiple of heads_kv                              */
  int32_t heads_kv;   /* Hkv >= 1                                                   */
  int32_t head_dim;   /* d: 64 or 128                                               */
  int32_t dtype;      /* ra_dtype of the cache, Q, K, V and O                       */
  int64_t window;     /* as ra_plan_window's, counted in slots; 0: the whole prefix */
  int64_t sinks;      /* as ra_plan_window's                                        */
  float scale;        /* score scale, 2^-100..2^100; 0 selects 1/sqrt(head_dim)     */
} ra_paged_problem;

typedef struct ra_paged_s* ra_paged_t;

/*
 * ra_paged_plan -- validate a cache's description and create its handle, which owns a device
 * status word and one event per stream its kernels were launched on (host-only without a
 * device, as ra_plan).  Release it with ra_paged_destroy, after the graphs that captured its
 * calls.  One host thread at a time may use a handle; its calls may overlap on the GPU.
 * Errors: RA_ERR_INVALID_ARG (null arguments, sizes < 1, page_rows, Hq % Hkv, window or sinks
 * < 0, bad enum or scale), RA_ERR_UNSUPPORTED (head_dim, more than 65535 key/value heads, more
 * than 2^31-1 rows of d channels), RA_ERR_CUDA.
 */
ra_status ra_paged_plan(const ra_paged_problem* prob, ra_paged_t* out);

/* Release a handle (NULL is accepted).  It does not wait, as ra_plan_destroy. */
ra_status ra_paged_destroy(ra_paged_t kv);

/*
 * ra_paged_append -- the new tokens' keys and values into the cache, in one launch with the
 * rotation of their keys and queries.
 * k, v: [tokens, Hkv, d]; q, q_out: [tokens, Hq, d], or both NULL.
 * rope: the rotation of keys and queries (of the cache's dtype and head_dim); NULL: keys are
 * written as they are, and q has to be NULL.  Results are those of ra_rope, bit for bit.
 * position: [tokens] int32, the tokens' positions in the rotation; NULL: their slots (the same
 * until an eviction has moved slots together).
 * q_out may be q with the same strides; no output may overlap an input otherwise.
 * Device pointers, 16-byte aligned (page_table, offset, length, position: 4-byte).
 * Asynchronous on stream; allocates nothing.
 * Errors: RA_ERR_INVALID_ARG (null/misaligned pointers, sizes < 1, strides, a rotation of
 * another type), RA_ERR_UNSUPPORTED (table_width * page_rows above 2^30, more than 4096
 * sequences, tokens * (Hq + 2 Hkv) above 2^30), RA_ERR_NO_DEVICE, RA_ERR_CUDA.
 */
ra_status ra_paged_append(ra_paged_t kv, ra_rope_t rope, void* cache, int64_t batch, int64_t tokens, const void* k,
                          const int64_t* k_strides, const void* v, const int64_t* v_strides, const void* q,
                          const int64_t* q_strides, void* q_out, const int64_t* q_out_strides,
                          const int32_t* page_table, int64_t table_width, const int32_t* offset,
                          const int32_t* length, const int32_t* position, void* stream);

/*
 * ra_paged_attend -- attention of the new tokens over their sequences' slots (their own among
 * them: append them first).  A token at slot s sees the slots j <= s, within the handle's
 * window and sinks (j > s - window or j < sinks).
 * q, o: [tokens, Hq, d], no two rows in one place; lse: [tokens, Hq] float32, contiguous (may be NULL).  A token all of
 * whose slots lie in pages out of range gets O = 0, LSE = -inf.
 * Slots that no token of the call sees may hold anything.  Values that some of them see must be
 * finite: they enter the products of the others with weight zero.
 * bf16: the softmax weights are rounded to bf16 for the second product; sums are fp32.  A chunk's
 * O is divided by the sum with the largest weight of every 128 slots as rounded, so that where one
 * slot has nearly all the weight its rounding cancels; the LSE is that of the exact sum.
 * bf16 chunks of calls of more than 2048 sequences, of tables of more than 2^25 slots
 * (table_width * page_rows) or of more than 128 query heads a key/value head are read 16 query rows at a
 * time, as float32 is, which takes them several times as long.
 * scratch: ra_paged_attend_scratch_size bytes (NULL when that is 0), not shared by calls that
 * may overlap.  o may not overlap an input.
 * Device pointers, 16-byte aligned (page_table, offset, length, lse: 4-byte).  Asynchronous on
 * stream; allocates nothing.
 * Errors: as ra_paged_append.
 */
ra_status ra_paged_attend(ra_paged_t kv, const void* cache, int64_t batch, int64_t tokens, const void* q,
                          const int64_t* q_strides, const int32_t* page_table, int64_t table_width,
                          const int32_t* offset, const int32_t* length, void* o, const int64_t* o_strides,
                          float* lse, float* scratch, void* stream);

/* Bytes of ra_paged_attend's scratch for these sizes (0 when it needs none).  Host only.
 * Errors: RA_ERR_INVALID_ARG, RA_ERR_UNSUPPORTED as ra_paged_attend. */
ra_status ra_paged_attend_scratch_size(ra_paged_t kv, int64_t batch, int64_t tokens, int64_t table_width,
                                       int64_t* bytes);

/*
 * ra_paged_weigh -- the attention weight that every slot receives from the new tokens, added to
 * what it received before: for slot j < length[b] of key/value head h,
 *   weight[b, h, j] = (weight_in[b, h, j] for slots before the call's tokens, else 0)
 *                     + sum over the tokens and query heads of the group that see j of
 *                       e^(scale q.k_j - LSE).
 * q: [tokens, Hq, d] as in ra_paged_attend; lse: [tokens, Hq] float32, what that call returned.
 * weight_in, weight: [batch, Hkv, weight_width] float32, contiguous; weight_in may be weight, or
 * NULL (zeros).  Slots from length[b] on stay as they were, and so do slots in pages out of
 * range; slots from weight_width on are reported (ra_paged_sync_status).  Deterministic.
 * scratch: ra_paged_weigh_scratch_size bytes (NULL when that is 0), not shared by calls that
 * may overlap.
 * Device pointers, 16-byte aligned (tables, lse and weights: 4-byte).  Asynchronous on stream;
 * allocates nothing.
 * Errors: as ra_paged_attend (weight_width outside 1..2^30: RA_ERR_INVALID_ARG).
 */
ra_status ra_paged_weigh(ra_paged_t kv, const void* cache, int64_t batch, int64_t tokens, const void* q,
                         const int64_t* q_strides, const float* lse, const int32_t* page_table,
                         int64_t table_width, const int32_t* offset, const int32_t* length,
                         const float* weight_in, float* weight, int64_t weight_width, float* scratch,
                         void* stream);

/* Bytes of ra_paged_weigh's scratch for these sizes (0 when it needs none).  Host only.
 * Errors: RA_ERR_INVALID_ARG, RA_ERR_UNSUPPORTED as ra_paged_weigh. */
ra_status ra_paged_weigh_scratch_size(ra_paged_t kv, int64_t batch, int64_t tokens, int64_t table_width,
                                      int64_t* bytes);

/*
 * ra_paged_evict -- keep at most `keep` slots of every sequence and key/value head: its `first`
 * first ones, its `recent` last ones, and of the others the heaviest; ties go to the lowest slot,
 * NaN counts as lighter than anything.  A sequence of up to `keep` slots keeps them all.  The
 * slots that stay move together in their order, each head by itself: slot kept[b, h, i] becomes
 * slot i.
 * length: [batch] int32.  weight_in: [batch, Hkv, weight_width] float32, weight (may be weight_in
 * or NULL) receives the weights of the slots that stay; other entries stay as they were.
 * new_table: [batch, new_width] int32, the pages that the sequences have afterwards: page_table
 * itself (in place; no page of it may be another sequence's), an array with the same entries, or
 * pages that no sequence of the call has (the old pages then keep what they hold, for others that
 * share them).
 * kept: [batch, Hkv, keep] int32, -1 behind the last; new_length: [batch] int32 (not length).
 * A sequence whose length is beyond the page table or weight_width, or whose slots do not fit in
 * new_width pages, is left as it is, with new_length 0, and reported.
 * Rotated keys stay valid: they keep the positions that they were rotated by; later tokens are
 * appended with positions of their own.
 * Device pointers, 16-byte aligned (tables and weights: 4-byte).  Asynchronous on stream;
 * allocates nothing.
 * Errors: as ra_paged_append (keep, first, recent, new_width, weight_width: RA_ERR_INVALID_ARG).
 */
ra_status ra_paged_evict(ra_paged_t kv, void* cache, int64_t batch, const int32_t* page_table, int64_t table_width,
                         const int32_t* length, const float* weight_in, float* weight, int64_t weight_width,
                         int64_t keep, int64_t first, int64_t recent, const int32_t* new_table, int64_t new_width,
                         int32_t* kept, int32_t* new_length, void* stream);

/*
 * ra_paged_sync_status -- synchronize `stream`, then read and clear the handle's status word:
 * RA_ERR_INVALID_ARG when a call since the last one met a page index, offset, length or slot out
 * of range, RA_ERR_TIMEOUT when a device-side wait ran out of budget, RA_ERR_CUDA on a CUDA
 * error, RA_ERR_BOUNDS when a bounds check of the debug build failed, RA_OK otherwise.
 */
ra_status ra_paged_sync_status(ra_paged_t kv, void* stream);

/* Thread-local message describing the last failure on this thread ("" if none). */
const char* ra_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* RA_H_ */

/*
 * scute.h -- C ABI of libscute.so: the adapted linear layer in normal form,
 * evaluated for a heterogeneous batch in which every token carries its own
 * adapter id, on one NVIDIA GB300 (sm_103a).
 *
 * What is computed.  For a token x (row vector, [d_in]) routed to adapter a,
 *
 *     F_a(x) = ((x R) W) * s + b + sum_k c_k (((x A_k) * d_k) B_k * e_k)
 *
 * the "normal form" of the article "Scute: Exact Batched Serving for PEFT
 * Adapters Beyond LoRA" (paper-daily.com), section "The big picture: six extra
 * slots in the LoRA computation".  W is the layer's shared base weight.  LoRA,
 * DoRA, (IA)^3, VeRA and OFT adapters are written into the slots at
 * registration; the fold rule of section "Which slots can be merged at load?"
 * multiplies every slot next to a tensor the adapter owns into that tensor, and
 * keeps live the slots next to shared tensors (s, b, R next to W; VeRA's d and
 * e next to the shared VeRA pair).  Tokens with id -1 get x W.
 *
 * Conventions used by every call below.
 *   - Row-major, row-vector orientation: x [n, d_in], W [d_in, d_out],
 *     A [d_in, rank], B [rank, d_out], out [n, d_out].
 *   - Matrices (W, A, B, R, shared VeRA A/B, x, out) are in the context dtype
 *     (bf16 or fp32).  A bf16 context may also write an fp32 `out`.
 *     Vectors (s, b, d, e, DoRA magnitude, (IA)^3 l) are always float32.
 *   - OFT rotations are explicit 32x32 blocks: R [d_in/32, 32, 32]; block k
 *     acts on input features [32k, 32k+32).
 *   - Setup calls (create, add_layer, set_shared, register, unregister) accept
 *     host or device pointers (the library copies through unified addressing)
 *     and may synchronise the device.  The library owns every tensor it keeps:
 *     caller buffers may be freed as soon as a setup call returns.
 *   - scute_linear is asynchronous on the caller's stream, allocates nothing,
 *     never synchronises and can be captured in a CUDA graph.  Errors the device
 *     detects (an id that names no adapter, a wait that timed out) are recorded
 *     in a status word read by scute_sync_status.  No call traps or hangs.
 *   - A context is thread-compatible, not thread-safe: calls on one context
 *     must be serialised by the caller, and its scute_linear calls must be
 *     ordered on the device (one stream, or streams joined by events), because
 *     they share the context's workspace.
 */
#ifndef SCUTE_H
#define SCUTE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct scute_ctx scute_ctx;

/* Adapter methods.  The order is also the order tokens are grouped in. */
typedef enum {
    SCUTE_LORA = 0, /* owned A, B and scalar c                                   */
    SCUTE_DORA = 1, /* owned A, B, c and learned column lengths (magnitude)      */
    SCUTE_IA3  = 2, /* l on key / value / up projections (the s slot)           */
    SCUTE_VERA = 3, /* per-adapter d, e around the layer's shared VeRA pair     */
    SCUTE_OFT  = 4, /* block-diagonal input rotation R (32x32 blocks)           */
    SCUTE_NF   = 5  /* raw normal-form slots: s, b, R and one owned term        */
} scute_method;

typedef enum { SCUTE_BF16 = 0, SCUTE_FP32 = 1 } scute_dtype;

typedef enum {
    SCUTE_OK = 0,
    SCUTE_ERR_ARG = 1,          /* null pointer, bad enum, out-of-range id/layer   */
    SCUTE_ERR_SHAPE = 2,        /* dimension not allowed (see each call)          */
    SCUTE_ERR_DTYPE = 3,        /* dtype combination not allowed                   */
    SCUTE_ERR_OOM = 4,          /* device allocation failed                        */
    SCUTE_ERR_BAD_ADAPTER = 5,  /* a token id named no registered adapter          */
    SCUTE_ERR_CUDA = 6,         /* a CUDA runtime call failed (see last_error)     */
    SCUTE_ERR_TIMEOUT = 7,      /* a bounded device-side wait gave up              */
    SCUTE_ERR_UNSUPPORTED = 8,  /* valid but outside what this build supports      */
    SCUTE_ERR_NO_DEVICE = 9,    /* no usable sm_103 device                        */
    SCUTE_ERR_PAGES = 10        /* cache pages ran out, or a page, slot or length is out of range */
} scute_status;

/* Limits of this build. */
#define SCUTE_MAX_TOKENS    16384  /* tokens per scute_linear call                 */
#define SCUTE_MAX_ADAPTERS  8192   /* registered adapters per context              */
#define SCUTE_MAX_RANK      64     /* rank of an owned low-rank term               */
#define SCUTE_MAX_SHARED_RANK 1024 /* rank of a layer's shared VeRA pair           */
#define SCUTE_OFT_BLOCK     32

/* Library version as MAJOR*10000 + MINOR*100 + PATCH. */
int scute_version(void);

/* Create a context on CUDA device `device`.
 *   dtype          storage/compute dtype of matrices and activations;
 *   max_tokens     largest n of a scute_linear call (1..SCUTE_MAX_TOKENS);
 *   max_adapters   adapter ids are 0..max_adapters-1 (1..SCUTE_MAX_ADAPTERS);
 *   max_layers     layer ids are 0..max_layers-1.
 * The context allocates its workspace here and grows it in scute_add_layer and
 * scute_set_shared.  Returns SCUTE_ERR_NO_DEVICE when the device is not sm_103. */
scute_status scute_create(scute_ctx **ctx, int device, scute_dtype dtype, int max_tokens,
                          int max_adapters, int max_layers);

/* Free every device allocation of the context (synchronises the device). */
void scute_destroy(scute_ctx *ctx);

/* Last error message of this context (static storage owned by the context). */
const char *scute_last_error(const scute_ctx *ctx);

/* Add base layer `layer` with shared weight W [d_in, d_out] (row-major, context
 * dtype).  The base GEMM h = xW is computed once for the whole batch (article,
 * "The big picture").  d_in and d_out must be positive multiples of 32
 * (SCUTE_ERR_SHAPE otherwise).  The library keeps a K-major copy of W. */
scute_status scute_add_layer(scute_ctx *ctx, int layer, int d_in, int d_out, const void *W);

/* Set the shared VeRA pair of `layer`: A_sh [d_in, rank], B_sh [rank, d_out]
 * (context dtype), shared by every VeRA adapter on that layer (article, "Which
 * slots can be merged at load?": VeRA's A and B are shared, rank 256 there).
 * rank must be a positive multiple of 32 and at most SCUTE_MAX_SHARED_RANK. */
scute_status scute_set_shared(scute_ctx *ctx, int layer, int rank, const void *A_sh,
                              const void *B_sh);

/* One layer's raw (unfolded) tensors of an adapter.  NULL = slot absent
 * (identity).  Which fields a method reads:
 *   LORA  A [d_in, rank], B [rank, d_out], c (= alpha / rank), rank
 *   DORA  A, B, c, rank, magnitude [d_out] (learned column length m)
 *   IA3   l [d_out]
 *   VERA  d [shared rank], e [d_out], c  (the layer must have a shared pair;
 *         c scales the shared term and is applied as given, like every other
 *         term's c: 1 for plain VeRA, 0 switches the term off)
 *   OFT   R [d_in/32, 32, 32]
 *   NF    any of s [d_out], b [d_out], R, and one owned term A, B, rank, c with
 *         optional d [rank] and e [d_out]
 * Layers of an adapter that are not listed get identity slots (n_layers may
 * be 0: the adapter then leaves every layer unchanged). */
typedef struct {
    int layer;
    int rank;
    float c;
    const void *A;
    const void *B;
    const float *d;
    const float *e;
    const float *s;
    const float *b;
    const void *R;
    const float *magnitude;
    const float *l;
} scute_layer_tensors;

/* Register an adapter: validate, copy to the device and apply the fold rule
 * (article, "Which slots can be merged at load?" and "How does Scute plug
 * into vLLM?"):
 *   - c and d of an owned term go into A:  A' = c A diag(d);
 *   - e of an owned term goes into B:      B' = B diag(e);
 *   - DoRA: s = m / ||column of (W + cAB)|| (L2 over d_in, accumulated in
 *     float64) stays live on the base path, and the same factor is folded into
 *     B as its e;  a zero column norm returns SCUTE_ERR_ARG;
 *   - (IA)^3: l becomes the live s slot;
 *   - VeRA: d and e stay live next to the shared pair;
 *   - OFT: the blocks of R stay live (they sit next to W).
 * Writes the new adapter id (lowest free id) to *adapter_id_out.
 * Errors: SCUTE_ERR_ARG (bad method / missing tensor / unknown layer / no free
 * id), SCUTE_ERR_SHAPE, SCUTE_ERR_UNSUPPORTED (rank > SCUTE_MAX_RANK, or R
 * combined with a VeRA term), SCUTE_ERR_OOM.  On error nothing is registered. */
scute_status scute_register_adapter(scute_ctx *ctx, scute_method method,
                                    const scute_layer_tensors *t, int n_layers,
                                    int32_t *adapter_id_out);

/* Remove an adapter and free its tensors.  Synchronises the device first, so
 * no in-flight call can still read them.  Its id becomes free. */
scute_status scute_unregister_adapter(scute_ctx *ctx, int32_t adapter_id);

/* The adapted linear layer for a heterogeneous batch (the hot path).
 *   x            device [n, d_in], context dtype;
 *   adapter_ids  device int32 [n]; -1 = base only.  An id that names no
 *                registered adapter is treated as -1 and recorded as
 *                SCUTE_ERR_BAD_ADAPTER in the status word;
 *   n            0..max_tokens (n = 0 returns SCUTE_OK without launching);
 *   out          device [n, d_out] in out_dtype (FP32 or, for a bf16 context,
 *                BF16); overwritten.
 *   stream       a cudaStream_t (NULL = legacy default stream).
 * Steps, all on the device: token indexing (stable grouping by method and
 * adapter id), the OFT input rotation into a workspace copy of x, the base
 * GEMM on tcgen05 tensor cores with the s / b epilogue gathered by adapter,
 * the owned low-rank shrink and expand, and the VeRA shared-pair GEMMs.  A
 * decode batch (bf16 context, n <= 128) runs all of them in one persistent
 * launch (scute_linear_batch with one call).
 * Returns after enqueueing; x, adapter_ids and out must stay valid until the
 * stream reaches the call. */
scute_status scute_linear(scute_ctx *ctx, const void *x, const int32_t *adapter_ids, int64_t n,
                          int layer, void *out, scute_dtype out_dtype, void *stream);

/* scute_linear with HOST buffers: copies x and adapter_ids from host memory
 * into context-owned device staging, runs scute_linear and copies `out` back,
 * all enqueued on `stream`; a bf16-context batch of at most 128 tokens stores
 * into a pinned, mapped, 16-byte-aligned `out_host` directly (unless the
 * separate s pass of scute_set_variant is on).  Pinned host memory keeps it
 * asynchronous; the caller synchronises the stream before reading
 * `out_host`. */
scute_status scute_linear_host(scute_ctx *ctx, const void *x_host, const int32_t *ids_host,
                               int64_t n, int layer, void *out_host, scute_dtype out_dtype,
                               void *stream);

/* Several layers over the same tokens in one call: for each i < n_calls,
 * calls[i].out receives the adapted layer calls[i].layer applied to
 * calls[i].x, all with the one adapter_ids vector (the projections of a
 * transformer block that read the same batch, such as q, k and v, or gate and
 * up).  The results are those of n_calls scute_linear calls up to the order of
 * floating-point sums.
 *   calls    HOST array of n_calls entries (0..SCUTE_MAX_CALLS); each x and out
 *            as for scute_linear (device, 16-byte aligned); an out may not
 *            overlap any call's x or out.  A layer may appear more than once.
 * A decode batch (bf16 context, n <= 128) runs as ONE persistent cooperative
 * launch that streams every listed layer's weights once, split over all SMs
 * in contiguous runs of 64-wide K blocks (section "Where is the cheapest place
 * to compute the remaining slots?" of the article prices the extra slots in
 * bytes moved; this launch keeps the one large byte stream, the base weights,
 * continuous).  Other batches run the calls one after another.  Errors as for
 * scute_linear; nothing is enqueued when an argument is rejected.  Calls on one
 * context must be ordered on the device (they share its workspace). */
#define SCUTE_MAX_CALLS 8
typedef struct scute_call {
    const void *x;   /* [n, d_in of layer] */
    int layer;
    void *out;       /* [n, d_out of layer] */
} scute_call;
scute_status scute_linear_batch(scute_ctx *ctx, const scute_call *calls, int n_calls,
                                const int32_t *adapter_ids, int64_t n, scute_dtype out_dtype,
                                void *stream);

/* scute_linear_batch with HOST buffers (every x and out, and adapter_ids, in
 * host memory): the inputs are copied into context-owned device staging, the
 * batch runs, the outputs are copied back, all enqueued on `stream`.  When
 * every input buffer is pinned and mapped, one kernel launch moves all of
 * them through their device addresses; otherwise each is one asynchronous
 * copy.  A bf16-context batch of at most 128 tokens whose output buffers are
 * all pinned, mapped and 16-byte aligned has its outputs stored straight
 * into them by the step (unless the separate s pass of scute_set_variant is
 * on); other pinned, mapped outputs take one scatter launch after the batch,
 * and any other output one copy each.  The caller synchronises the stream
 * before reading the outputs. */
scute_status scute_linear_batch_host(scute_ctx *ctx, const scute_call *calls, int n_calls,
                                     const int32_t *ids_host, int64_t n, scute_dtype out_dtype,
                                     void *stream);

/* Synchronise the device and return (then clear) the device status word:
 * SCUTE_OK, SCUTE_ERR_TIMEOUT, SCUTE_ERR_BAD_ADAPTER or SCUTE_ERR_PAGES (the
 * first of these that was recorded, in this order). */
scute_status scute_sync_status(scute_ctx *ctx);

/* Token indexing alone, for inspection.  Runs the same kernel scute_linear
 * runs and copies its results into caller device buffers on `stream`:
 *   perm       int32 [n]     sorted position -> token index;
 *   aid_sorted int32 [n]     adapter of each sorted row (-1 = base);
 *   seg_start  int32 [n + 1] first sorted row of each segment, then n;
 *   seg_aid    int32 [n]     adapter of each segment;
 *   counts     int32 [22]    n_seg, rows per method (7: LoRA, DoRA, (IA)^3,
 *                            VeRA, OFT, NF, base), first row per method (7),
 *                            segments per method (7).
 * Only the first n_seg entries of seg_aid and n_seg + 1 of seg_start are set. */
scute_status scute_debug_index(scute_ctx *ctx, const int32_t *adapter_ids, int64_t n,
                               int32_t *perm, int32_t *aid_sorted, int32_t *seg_start,
                               int32_t *seg_aid, int32_t *counts, void *stream);

/* ---------------------------------------------------------------- token indexing without a context
 * The article has no counterpart of this call: it is a service of this
 * library for callers that cannot allocate device memory.  Typical ones: a
 * batch scheduler or router in a process whose serving engine has already
 * reserved its device memory pool (most of HBM goes to the KV cache), where a
 * new allocation fails or takes memory the pool counts on; and code on a
 * latency-critical path, where cudaMalloc and cudaFree may synchronise the
 * device.  Such callers still want the adapter segments a batch forms, but
 * cannot create a context (scute_create allocates its workspaces).
 *
 * Runs the kernel scute_debug_index runs, on the CURRENT device and `stream`,
 * with the same outputs (perm, aid_sorted, seg_start, seg_aid, counts: layout
 * as for scute_debug_index; all device buffers of the caller), and
 *   method_of_adapter  HOST int8 [n_adapters]: the scute_method of each
 *                      adapter id, or -1 where the id names no adapter;
 *                      copied with cudaMemcpyAsync (pageable memory may be
 *                      reused when the call returns; pinned memory must stay
 *                      unchanged until the stream has passed the call);
 *   flags              device int32 [1] or NULL: nonzero when an id in
 *                      adapter_ids named no adapter (those tokens become
 *                      base-only rows, as in scute_linear).
 * Scratch: a file-scope device array of SCUTE_NOALLOC_SCRATCH_BYTES (the method
 * table and a status word), located once per device with cudaGetSymbolAddress
 * on the first call made while that device is current.  That first call may
 * load the library's module, so make it before any stream capture.  The
 * address is kept for the life of the process: do not use this call on a
 * device after cudaDeviceReset (or any teardown of its primary context) in
 * the same process.  Nothing
 * is allocated: no cudaMalloc, cudaFree or allocating library routine.
 * Overlapping calls on one device (other streams, other host threads) share
 * the array and race; order them on the device.
 * Errors (nothing is launched): SCUTE_ERR_ARG for a null output, n < 0,
 * n_adapters < 1 or a method code outside -1..5; SCUTE_ERR_UNSUPPORTED for
 * n > SCUTE_MAX_TOKENS or n_adapters > SCUTE_NOALLOC_MAX_ADAPTERS (the static
 * table's size); SCUTE_ERR_NO_DEVICE when the current device is not sm_103;
 * SCUTE_ERR_CUDA when a CUDA call fails. */
#define SCUTE_NOALLOC_MAX_ADAPTERS 8192
#define SCUTE_NOALLOC_SCRATCH_BYTES (256 + SCUTE_NOALLOC_MAX_ADAPTERS)
scute_status scute_index_tokens_noalloc(const int8_t *method_of_adapter, int32_t n_adapters,
                                        const int32_t *adapter_ids, int64_t n, int32_t *perm,
                                        int32_t *aid_sorted, int32_t *seg_start, int32_t *seg_aid,
                                        int32_t *counts, int32_t *flags, void *stream);

/* ---------------------------------------------------------------- the decoder block's other operators
 * The adapted layer computes a transformer block's projections; the calls of
 * this section do what a serving step needs between them, on the context's
 * device and in its dtype: cache pages and slots for every request's new
 * tokens (scute_kv_resize), rotary positions and the cache write
 * (scute_kv_append), attention of one new token of each request over the
 * paged cache (scute_paged_attention), and the norms, gate and residual that
 * close a sub-block (scute_residual_norm).  The article leaves these to the
 * serving engine; they have no counterpart in it.
 *
 * All four are asynchronous on `stream`, allocate nothing and can be captured
 * in a CUDA graph.  They read lengths, tables and slots on the device, so a
 * captured step stays valid while those change.  Arguments the host can see
 * are checked before anything is enqueued; what only the device can see (a
 * length beyond the block table, a page outside the pool, too few free pages)
 * never reads or writes out of range and is recorded in the status word:
 * scute_sync_status then returns SCUTE_ERR_PAGES.  Calls on one context must
 * be ordered on the device (they share its workspace, 30 MB on 152 SMs, which
 * scute_create allocates). */

/* Element type of a cache: BF16 or E4M3 (8-bit float, 4 exponent and 3
 * mantissa bits) in a bf16 context, FP32 in an fp32 context. */
typedef enum { SCUTE_KV_BF16 = 0, SCUTE_KV_FP32 = 1, SCUTE_KV_E4M3 = 2 } scute_kv_dtype;

/* A paged key/value cache.  The pools and tables are the caller's; the library
 * keeps nothing of them.  Cache slot p * page_size + t is token t of page p;
 * its key of head h is the head_dim consecutive elements at
 *     k + p * page_stride + t * token_stride + h * head_stride
 * and its value the same place of v (strides in elements).  Head-major pages
 * ([page][head][token][dim]) and token-major ones ([page][token][head][dim])
 * are both strides of this form.  Token t of request r lies in page
 * block_table[r * table_stride + t / page_size].
 *   k, v            16-byte aligned; strides multiples of 16 bytes, at least head_dim;
 *   head_dim        a multiple of 16, 16..256;
 *   n_pages * page_size  at most 2^31 - 1; offsets are computed in 64 bits;
 *   k_scale, v_scale  NULL, or device float [kv_heads]: a stored element stands
 *                   for itself times its head's scale (an E4M3 cache is
 *                   written as value / scale, rounded to nearest, saturated);
 *   block_table     needed by scute_paged_attention only. */
typedef struct {
    void *k, *v;
    int32_t dtype;                /* scute_kv_dtype */
    int32_t n_pages, page_size, kv_heads, head_dim;
    int64_t page_stride, token_stride, head_stride;
    const int32_t *block_table;   /* device [n_req][table_stride] */
    int64_t table_stride;
    int32_t table_cols;           /* entries of a row that may be read */
    const float *k_scale, *v_scale;
} scute_kv_cache;

#define SCUTE_MAX_REQUESTS 16384
#define SCUTE_MAX_HEAD_DIM 256

/* Give each request the pages of its new length, and each new token its slot.
 * Request r has len_in[r] cached tokens in pages block_table[r][0 ..
 * ceil(len_in[r] / page_size)) and shall have len_new[r].
 *   - A request that shrinks (to 0: it has ended) gives up its last pages.
 *     They go on top of the free list, in the order of requests and, within
 *     one, of its table.  Its table row is left as it is.
 *   - A request that grows takes its pages from the top of the free list (the
 *     ones just given up included), in the order of requests; they are
 *     written behind its old ones in its row.  Requests are served while both
 *     last: a request that needs pages is refused when it and those before it
 *     need more than there are; then, of the rest, one is refused when its new
 *     tokens and those before it (of requests not refused for pages) are more
 *     than max_new.
 *     A refused request keeps its length and takes nothing
 *     (SCUTE_ERR_PAGES); a request that grows within its last page is never
 *     refused for want of pages.
 *   - The new tokens of served requests, in order, are the step's token rows:
 *     slot_map[i], positions[i] and token_req[i] are row i's cache slot, its
 *     position in its request and its request.  Rows beyond them, up to
 *     max_new, get -1, 0 and -1 (scute_kv_append skips slot -1), so that a
 *     captured step can have a fixed number of rows.  A row whose page number
 *     (of the table or the free list) is negative, or so large that no slot of
 *     31 bits comes of it, gets INT32_MIN and is recorded (SCUTE_ERR_PAGES).
 *   - cu_new [n_req + 1]: request r's rows are cu_new[r] .. cu_new[r + 1).
 * len_in, len_new, len_out  device int32 [n_req]; len_out may be len_in.  A
 *     length outside 0 .. table_cols * page_size is an error
 *     (SCUTE_ERR_PAGES): as len_in it counts as the nearest one inside, as
 *     len_new the request keeps its length;
 * free_pages  device int32 [n_free_max], the free list: pages free_pages[0 ..
 *     *free_in), the top last.  Entries from the new count on keep what they
 *     held;
 * free_in, free_out  device int32: the list's count; free_out may be free_in.
 * n_req is 0..SCUTE_MAX_REQUESTS, n_req * table_cols and n_free_max at most
 * 2^31 - 1, max_new 0..2^30.  A step's pages are fixed by
 * the arguments alone, whatever order the device works in. */
scute_status scute_kv_resize(scute_ctx *ctx, const int32_t *len_in, const int32_t *len_new, int n_req,
                             int32_t *block_table, int64_t table_stride, int table_cols, int page_size,
                             int32_t *free_pages, int64_t n_free_max, const int32_t *free_in,
                             int32_t *free_out, int32_t *len_out, int32_t *cu_new, int32_t *slot_map,
                             int32_t *positions, int32_t *token_req, int64_t max_new, void *stream);

/* Rotary positions.  Pair i of a head's first rotary_dim elements is turned by
 * the angle whose cosine and sine stand in row p of the table:
 *     (a, b) -> (a cos - b sin, b cos + a sin),
 *     cos = cos_sin[p][i], sin = cos_sin[p][rotary_dim / 2 + i].
 * Pair i is elements i and i + rotary_dim / 2, or 2i and 2i + 1 when
 * `interleaved`; elements from rotary_dim on pass unchanged.  With several axes
 * (time, height, width of an image or video token) the pairs are cut into
 * consecutive sections, and p is the token's position on its section's axis.
 *   cos_sin     device float [n_pos][rotary_dim] (scute_rope_table);
 *   positions   device int32, axis a of token t at a * axis_stride + t; a
 *               position outside 0..n_pos-1 counts as the nearest one inside
 *               and is recorded (SCUTE_ERR_PAGES);
 *   n_axes      1..4; section[a] pairs each, rotary_dim / 2 in all (with one
 *               axis, section is not read);
 *   rotary_dim  even, 2..head_dim. */
typedef struct {
    const float *cos_sin;
    int32_t n_pos, rotary_dim, interleaved, n_axes;
    int32_t section[4];
    const int32_t *positions;
    int64_t axis_stride;
} scute_rope;

/* Fill a rotary table: cos_sin[p][i] = cos(p f_i), cos_sin[p][rotary_dim / 2 + i]
 * = sin(p f_i), computed in 64 bits, with f_i = inv_freq[i] (device double
 * [rotary_dim / 2]: a stretched context's own frequencies) or, when inv_freq is
 * NULL, theta^(-2i / rotary_dim). */
scute_status scute_rope_table(scute_ctx *ctx, float *cos_sin, int n_pos, int rotary_dim, double theta,
                              const double *inv_freq, void *stream);

/* Write the keys and values of n token rows into the cache, keys (and queries)
 * turned by their positions.
 *   slot_map  device int32 [n]: row t's cache slot, or -1 for none; a slot
 *             outside the pool is skipped and recorded (SCUTE_ERR_PAGES).  Two
 *             rows may not name one slot;
 *   k, v      context dtype, head h of row t at t * k_stride + h * head_dim
 *             (v_stride); q [q_heads heads] the same way, written to q_out
 *             (which may be q) for every row, those without a slot too;
 *             q NULL: keys and values only;
 *   rope      NULL: no turning (q must then be NULL).
 * Strides are in elements, at least heads * head_dim; no alignment beyond the
 * element's is needed (16-byte aligned rows are fastest).  Sums are in 32 bits,
 * rounded once.  n is 0..2^24. */
scute_status scute_kv_append(scute_ctx *ctx, const scute_kv_cache *kv, const int32_t *slot_map, int64_t n,
                             const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                             const void *q, int64_t q_stride, int q_heads, void *q_out,
                             int64_t q_out_stride, const scute_rope *rope, void *stream);

/* Attention of one new token of each request over its cached tokens:
 *     out[r][h] = sum_t p_t v_t,  p = softmax over t of score(q[r][h] . k_t),
 * over the last kv_len[r] cached tokens (with window > 0: the last
 * min(kv_len[r], window) of them), k_t and v_t of key/value head h / (q_heads /
 * kv_heads).  score(x) = scale x, or softcap tanh(scale x / softcap) with
 * softcap > 0.  A request without tokens gets zeros (and an lse of -infinity).
 *   q, out    context dtype [n_req][q_heads * head_dim], rows q_stride and
 *             out_stride elements apart; 16-byte aligned, strides multiples of
 *             16 bytes; out may be q;
 *   kv_len    device int32 [n_req]; more than table_cols * page_size counts as
 *             that many and is recorded; so is a table entry outside the pool,
 *             whose tokens are left out (SCUTE_ERR_PAGES).  Nothing beyond a
 *             request's length is read;
 *   lse       NULL, or device float [n_req][q_heads]: log sum exp of the scores
 *             (joins this result with one over other tokens);
 *   scale     0: 1 / sqrt(head_dim).
 * n_req is 0..SCUTE_MAX_REQUESTS; table_cols * page_size at most 2^30, and 2^33
 * over all requests; q_heads a multiple of kv_heads.  Scores, softmax
 * statistics and sums are held in 32 bits.  What is rounded to fewer on the way:
 * a weight as it is multiplied with a value, to 16 bits with a BF16 cache (an error
 * of 2^-17 of it), 22 with an E4M3 one, none with FP32; and queries before an E4M3
 * cache's keys, below 2^-22 of their head's largest element.  The work is cut over the
 * whole batch's tokens, whatever request they belong to, and joined in a fixed
 * order: the same call gives the same bits. */
typedef struct {
    const void *q;
    int64_t q_stride;
    void *out;
    int64_t out_stride;
    float *lse;
    const int32_t *kv_len;
    int32_t n_req, q_heads;
    float scale, softcap;
    int32_t window;
} scute_attention;
scute_status scute_paged_attention(scute_ctx *ctx, const scute_kv_cache *kv, const scute_attention *a,
                                   void *stream);

/* The end of a sub-block and the beginning of the next, for n token rows:
 *     h = residual + scale * gate * post(y),   out = pre(h).
 * post and pre are norms over a row of d: x / sqrt(mean(x^2) + eps) * w + b, or
 * with `layer` the same of x - mean(x).  Everything between is held in 32 bits;
 * out and residual_out are each rounded once (pre reads h before its rounding).
 *   y, residual, out, residual_out   context dtype, rows of d elements their
 *              stride apart; residual NULL counts as zeros; residual_out
 *              (NULL: not written) may be residual; out may be y (NULL: no norm
 *              after);
 *   post_w, post_b, pre_w, pre_b   device float [d]; post_w NULL: no norm of
 *              y (post_b must then be NULL); pre_w NULL: ones; biases NULL: zeros;
 *   gate_vec   NULL, or device float [d]; gate_rows NULL, or context dtype
 *              [n][d], rows gate_stride apart; at most one of the two;
 *   n 0..2^24, d 1..SCUTE_MAX_NORM_DIM, eps >= 0; no alignment beyond the
 *   element's is needed (16-byte aligned rows are fastest). */
#define SCUTE_MAX_NORM_DIM 32768
typedef struct {
    const void *y;
    int64_t y_stride;
    const void *residual;
    int64_t residual_stride;
    void *residual_out;
    int64_t residual_out_stride;
    void *out;
    int64_t out_stride;
    const float *post_w, *post_b, *pre_w, *pre_b;
    const float *gate_vec;
    const void *gate_rows;
    int64_t gate_stride;
    float scale, eps;
    int32_t layer;
} scute_norm;
scute_status scute_residual_norm(scute_ctx *ctx, const scute_norm *a, int64_t n, int d, void *stream);

/* ---------------------------------------------------------------- byte model
 * Zero-parameter byte and time model (article, section "Where is the cheapest
 * place to compute the remaining slots?": added time = extra bytes / memory
 * bandwidth + extra launches x launch cost; bytes are what adapter work is
 * measured in).
 *
 * For one call it lists every kernel launch the library makes for it, with the
 * bytes that launch must move to and from device memory (each operand read
 * once, each result written once; intermediates a launch keeps to itself are
 * not counted: a lower bound that measured DRAM bytes are compared against)
 * and its floating-point operations, plus the call's algorithmic bytes: W once,
 * each distinct adapter's live (post-fold) tensors once, the shared VeRA pair
 * once when a VeRA token is present, x read, out written and the ids read.
 * Launch plans: a bf16 batch of at most 128 tokens is ONE launch ("step") over
 * every layer of the call, with "oft_pass" before it and "s_pass" after it
 * when the variant flags place those slots in passes of their own
 * (scute_set_variant; the step's own bytes then lose R, or the DoRA and
 * (IA)^3 s vectors); otherwise each layer takes the per-kernel plan
 * ("index", "rotate", "base_gemm", "lr_shrink", "lr_expand", "vera_shrink",
 * "vera_expand"; in a bf16 context above 256 tokens "lr_shrink" and, for a
 * shared rank that is a multiple of 64, "vera_shrink" come before
 * "base_gemm", which takes in the owned expand).  Pure host arithmetic: no device work, no context needed for
 * scute_byte_model and scute_byte_model_batch. */
#define SCUTE_BM_MAX_KERNELS 64
typedef struct {
    int n_kernels;                          /* launches of the call            */
    char name[SCUTE_BM_MAX_KERNELS][24];    /* kernel names                    */
    int64_t bytes[SCUTE_BM_MAX_KERNELS];    /* bytes read + written per launch */
    int64_t flops[SCUTE_BM_MAX_KERNELS];    /* 2 x multiply-adds per launch    */
    int64_t algorithmic_bytes;              /* minimal bytes of the call       */
    int64_t adapter_bytes;                  /* live adapter tensors + shared pair */
    int64_t base_weight_bytes;              /* W                               */
    int32_t distinct_adapters;              /* distinct valid ids in the batch */
} scute_byte_report;

/* One registered adapter as the byte model sees one layer of it.
 * method = -1 marks an unregistered id. */
typedef struct {
    int method;
    int rank;          /* owned low-rank rank on this layer (0 = none) */
    int has_s, has_b, has_R, has_vera, has_vera_e;
} scute_bm_adapter;

typedef struct {
    scute_dtype dtype;        /* context dtype                                 */
    scute_dtype out_dtype;
    int d_in, d_out;
    int shared_rank;          /* 0 = no shared VeRA pair                       */
    int lowrank_launched;     /* the per-kernel plan launches the owned-term kernels */
    int vera_launched;        /* the per-kernel plan launches the VeRA kernels */
    int max_adapters;
    const scute_bm_adapter *adapters;  /* [max_adapters]                       */
    int variant;              /* SCUTE_VARIANT_* flags of the call (0: none)   */
} scute_bm_layer;

/* One call of one layer (scute_linear). */
scute_status scute_byte_model(const scute_bm_layer *layer, const int32_t *ids_host, int64_t n,
                              scute_byte_report *rep);

/* One batched call (scute_linear_batch) over n_layers (1..SCUTE_MAX_CALLS)
 * layers that read the same ids; all in one dtype.  SCUTE_ERR_UNSUPPORTED when
 * the per-kernel plan needs more than SCUTE_BM_MAX_KERNELS launches. */
scute_status scute_byte_model_batch(const scute_bm_layer *layers, int n_layers, const int32_t *ids_host,
                                    int64_t n, scute_byte_report *rep);

/* The same for layer `layer` of a context, from its registered adapters. */
scute_status scute_predict_bytes(const scute_ctx *ctx, const int32_t *ids_host, int64_t n,
                                 int layer, scute_dtype out_dtype, scute_byte_report *rep);

/* The same for a batched call of a context (only calls[i].layer is read). */
scute_status scute_predict_batch(const scute_ctx *ctx, const scute_call *calls, int n_calls,
                                 const int32_t *ids_host, int64_t n, scute_dtype out_dtype,
                                 scute_byte_report *rep);

/* Predicted time of a launch list, in microseconds:
 *     sum over launches of max(bytes / hbm_gbs, flops / tensor_tflops)
 *     + launches x launch_us.
 * With tensor_tflops <= 0 the flops term is dropped and this is the article's
 * model as it stands (bytes / bandwidth + launches x launch cost); the flops
 * term extends it to launches bound by the tensor cores (prefill GEMMs).  The
 * three constants are measured on the device, never fitted. */
scute_status scute_predict_time(const scute_byte_report *rep, double hbm_gbs, double tensor_tflops,
                                double launch_us, double *us_out);

/* ---------------------------------------------------------------- counters
 * Device kernels enqueued by this context since creation. */
int64_t scute_launch_count(const scute_ctx *ctx);

/* Kernel timing with CUDA events on the launching stream.  While enabled,
 * every launch of the hot path (the decode step; or, on the per-kernel plan,
 * the indexing, rotation, base GEMM, low-rank shrink + expand pair and the two
 * VeRA GEMMs) is bracketed by an event pair, stored in a ring of
 * `SCUTE_TIMING_SLOTS` slots in launch order and tagged with its kind
 * (SCUTE_KIND_*).  Event records made during stream capture become graph
 * nodes and are re-recorded on every replay.  Timing puts an event record
 * between launches that would otherwise overlap their start and end
 * (programmatic dependent launch), so a timed call can be slightly slower.
 * scute_timing_read synchronises the device and writes the elapsed
 * milliseconds of the first `max` used slots; scute_timing_kinds writes their
 * kinds. */
#define SCUTE_TIMING_SLOTS 256
enum {
    SCUTE_KIND_STEP = 0,         /* the batched decode step (one launch)       */
    SCUTE_KIND_INDEX = 1,        /* token indexing                             */
    SCUTE_KIND_ROTATE = 2,       /* OFT rotation / gather of the token operand */
    SCUTE_KIND_BASE_GEMM = 3,    /* base GEMM with the s / b epilogue          */
    SCUTE_KIND_LOWRANK = 4,      /* owned low-rank shrink and expand (2 launches) */
    SCUTE_KIND_VERA_SHRINK = 5,  /* VeRA shared shrink GEMM                    */
    SCUTE_KIND_VERA_EXPAND = 6,  /* VeRA shared expand GEMM                    */
    SCUTE_KIND_OFT_PASS = 7,     /* rotation as its own pass (scute_set_variant) */
    SCUTE_KIND_S_PASS = 8,       /* s as its own pass (scute_set_variant)      */
    SCUTE_KIND_KV_RESIZE = 9,    /* scute_kv_resize                            */
    SCUTE_KIND_KV_APPEND = 10,   /* scute_kv_append                            */
    SCUTE_KIND_ATTENTION = 11,   /* scute_paged_attention                      */
    SCUTE_KIND_NORM = 12         /* scute_residual_norm                        */
};
scute_status scute_timing_enable(scute_ctx *ctx, int enable);
scute_status scute_timing_reset(scute_ctx *ctx);
scute_status scute_timing_read(scute_ctx *ctx, float *ms_out, int max, int *n_out);
scute_status scute_timing_kinds(const scute_ctx *ctx, int *kinds_out, int max, int *n_out);

/* Test hook for the failure path (no counterpart in the article).  With
 * what = SCUTE_INJECT_STALL, the context's next decode launch (bf16, n <= 128)
 * waits for a count that no CTA ever reaches: its bounded waits run out (about
 * 2 s), every CTA drains what it issued, frees TMEM and returns, and
 * scute_sync_status then reports SCUTE_ERR_TIMEOUT.  The context stays usable;
 * the hook applies to that one launch only.  Nothing traps or faults.
 * SCUTE_INJECT_STALL_ATTENTION does the same to the context's next
 * scute_paged_attention: its fetching warps never get a stage of cached tokens
 * back, so that their waits and the computing warps' run out (where a CTA's
 * share of the tokens is more than its stages hold); its outputs are then
 * undefined.  what = 0 takes either hook back. */
#define SCUTE_INJECT_STALL 1
#define SCUTE_INJECT_STALL_ATTENTION 2
scute_status scute_debug_inject(scute_ctx *ctx, int what);

/* Separate-pass placements of two live slots, for validating the byte and
 * time model (article, section "Where is the cheapest place to compute the
 * remaining slots?": the model is checked there on OFT's input rotation and
 * on applying DoRA's s outside the expand).  With flags = 0 (the default) the
 * decode step applies every slot inside its one launch.  Otherwise a bf16
 * decode batch (n <= 128) of this context adds, around its step launch:
 *   SCUTE_VARIANT_OFT_PASS  one launch before the step that writes x R for
 *                           the rotated tokens (x for the others) into a
 *                           context-owned copy, which the step then reads;
 *   SCUTE_VARIANT_S_PASS    one launch after the step that multiplies the
 *                           output rows of DoRA and (IA)^3 tokens by their s,
 *                           which the step then leaves out (DoRA expanding
 *                           with B' whose s is not folded in).
 * Results stay those of the normal form up to rounding order.  Other batches
 * (fp32 contexts, more than 128 tokens) ignore the flags.  A setup call:
 * SCUTE_VARIANT_OFT_PASS allocates the rotated-copy workspace here, so do not
 * make it during stream capture.  scute_predict_batch describes the launches
 * of the flags in force. */
#define SCUTE_VARIANT_OFT_PASS 1
#define SCUTE_VARIANT_S_PASS 2
scute_status scute_set_variant(scute_ctx *ctx, int flags);

/* Test hook for the out-of-memory path (no counterpart in the article).  The
 * k-th device allocation the library makes after this call (counted over
 * every context of the process) fails as if the device were out of memory:
 * nothing is allocated for it and the call that needed it returns
 * SCUTE_ERR_OOM, having freed what it had allocated itself and leaving the
 * context as it was.  k <= 0 switches the hook off.  Host-side only: no
 * device work is involved. */
void scute_debug_fail_alloc(int k);

/* The plan of the context's last decode-step launch (the host values that
 * launch was given), so that the kernel's index arithmetic can be checked
 * against its buffers on the host.  The article has no counterpart.  Writes at
 * most `cap` int64 values to the HOST array `out`:
 *   SCUTE_PLAN_HEAD values: n_calls, n, bn (tokens per tile), stages, grid,
 *     n_units (VeRA shrink units), vs_ch (K blocks per unit), n_tiles,
 *     n_items (low-rank shrink items), rmax, t_main (main K blocks), hold,
 *     smem_bytes (before the one-CTA-per-SM floor), smem_optin,
 *     part_floats (partial-tile workspace), xs_cols and u_cols (row pitch of
 *     the token-operand and VeRA-intermediate slots), sync_ints, pre_floats
 *     (the owned low-rank rows b + v B', all call slots);
 *   then SCUTE_PLAN_CALL_FIELDS values per call: blk0, d_in, kdim, d_out,
 *     krv, rv, kblocks, vkb, n_ft, n_vt, vs_chunks, vs_unit0, tile0, lr_rmax,
 *     lr_items, lr_item0, vs_x, xs_direct;
 *   then grid + 1 values: the stream-K range bounds start[0..grid].
 * *n_out = the number of values the plan has (only the first cap written).
 * SCUTE_ERR_ARG when no decode step has been launched on the context. */
#define SCUTE_PLAN_HEAD 19
#define SCUTE_PLAN_CALL_FIELDS 18
scute_status scute_debug_step_plan(const scute_ctx *ctx, int64_t *out, int cap, int *n_out);

#ifdef __cplusplus
}
#endif
#endif /* SCUTE_H */

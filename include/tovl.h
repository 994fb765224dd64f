/*
 * tovl.h -- C ABI of the tovl library: token-row movement fused with a bf16
 * tensor-core GEMM on one NVIDIA GB300 (sm_103a).
 *
 * The method: producer CTAs move token rows into one gathered buffer while
 * consumer CTAs run a GEMM that starts on each 128-row block as soon as its
 * rows are complete.  Completion follows the single-writer slot protocol of
 * the Astro Bear page "Fused compute/communication operators (4): cross-GPU
 * sync protocols on PCIe -- single writer, election and watermarks":
 *   section 2  slots hold monotonically increasing sequence numbers that are
 *              never reset; round k waits for a value >= k;
 *   section 3  many writers are counted with a local acq_rel atomic and the
 *              last arrival is elected to publish with a release store;
 *   section 4  one watermark slot per 64-row chunk;
 *   section 5  row-block counters take release reductions and are pre-seeded
 *              with the padding count, so real arrivals reach 128 exactly.
 * The "ranks" of the pages are logical shards held in this GPU's memory; the
 * library uses no peer memory and no collectives.
 *
 * Conventions for every entry point:
 *   - Pointers named as device pointers must point to device memory of the
 *     handle's GPU, 16-byte aligned; host pointers are ordinary host memory.
 *   - bf16 tensors are row-major with unit stride in the last dimension.
 *   - The caller owns every buffer and stream; the handle owns only its
 *     control plane (counters, slots, status word, plan scratch) and its
 *     sequence number.
 *   - `stream` is a cudaStream_t (NULL = legacy default stream).  Calls are
 *     asynchronous; one call is one protocol round.  Calls on one handle must
 *     be issued from one host thread, in order, on one stream.
 *   - Return value: TOVL_OK, or an error code from tovl_status.  Argument
 *     errors are detected on the host before anything is enqueued and leave
 *     the handle unchanged.  Errors found on the device (a wait that timed
 *     out, an expert id out of range) are sticky in the handle's status word
 *     and read with tovl_sync_status(); device code never traps.
 *   - There is no CPU fallback: on a machine without a compute-capability
 *     10.3 GPU, tovl_create returns TOVL_ERR_UNSUPPORTED.
 */
#ifndef TOVL_H
#define TOVL_H

#ifdef __cplusplus
extern "C" {
#endif

typedef struct tovl_ctx* tovl_handle;

typedef enum {
    TOVL_OK = 0,
    TOVL_ERR_INVALID = 1,      /* bad argument, shape, alignment or routing */
    TOVL_ERR_UNSUPPORTED = 2,  /* shape or device the kernels do not support */
    TOVL_ERR_CUDA = 3,         /* a CUDA runtime call failed; see tovl_last_error */
    TOVL_ERR_TIMEOUT = 4,      /* a device wait gave up (sticky, from tovl_sync_status) */
    TOVL_ERR_OOM = 5           /* device allocation failed in tovl_create */
} tovl_status;

/* Row-copy mechanism of tovl_gated_copy.  The producers of the fused
 * kernels use 16 warps per CTA; their copy path is option 14. */
typedef enum {
    TOVL_COPY_VECTOR = 0,      /* 16-byte vector loads/stores by warps */
    TOVL_COPY_BULK = 1,        /* bulk asynchronous copies through a shared-memory ring */
    TOVL_COPY_AUTO = 2         /* vector below 8 KB rows, bulk from 8 KB (the default) */
} tovl_copy_mode;

typedef struct {
    int device;                /* CUDA device ordinal */
    int chunk_rows;            /* watermark chunk; must be 64 (or 0 for 64) -- section 4 */
    int gate_rows;             /* GEMM row-block gate; must be 128 (or 0 for 128) -- section 5 */
    int producer_ctas;         /* P; 0 = chosen per call: copy and GEMM time balanced,
                                  then grown while the GEMM keeps its wave count */
    int consumer_ctas;         /* C; 0 = all remaining SMs */
    long long wait_timeout_ns; /* bound of every device wait; 0 = 2 s */
    int copy_mode;             /* tovl_copy_mode of tovl_gated_copy; the default is
                                  TOVL_COPY_AUTO (measured on GB300, gated: 71-91 % of
                                  the HBM copy bandwidth with vector copies from 256 B
                                  to 4 KB rows, 94-96 % with bulk copies at 8-16 KB) */
    long long max_rows;        /* capacity in rows of gathered/dispatched buffers and copies */
    int max_pairs;             /* largest T*k of a dispatch call */
    int max_experts;           /* largest E of a dispatch call (<= 512) */
    int k_slices;              /* 1..8 (0 = 1): each 64-row chunk watermark (and each
                                  128-row block counter) is split into this many
                                  K-ranges, published separately, so a GEMM tile may
                                  start on the first K-range of its rows; 1 = one
                                  watermark per chunk (sections 4-5 exactly) */
} tovl_config;

/* Fills `cfg` with defaults for `device`. */
void tovl_default_config(tovl_config* cfg, int device);

/* Creates a handle: validates `cfg`, checks the device (compute capability
 * 10.3), allocates and zeroes the control plane (chunk slots and counters for
 * max_rows/64 chunks, row-block counters for max_rows/128 blocks, status
 * word, plan scratch).  Sequence number starts at 0.  On failure *out is
 * NULL and nothing stays allocated. */
int tovl_create(tovl_handle* out, const tovl_config* cfg);

/* Frees the handle's device memory after synchronising its last stream.
 * NULL is accepted.  The handle must not be used afterwards. */
int tovl_destroy(tovl_handle h);

/* All-gather of S logical shards followed by a GEMM (the tensor-parallel
 * all-gather + GEMM of the platform page "know your platform", section 3,
 * with the completion protocol of sections 2-5 of the sync page).
 *   shards      host array of S device pointers; shard s is bf16 [R][K]
 *   num_shards  S, 1..64
 *   rows_per_shard R >= 1; M = S*R <= max_rows
 *   K           multiple of 64, at most 32768
 *   W           device, bf16 [K][N]
 *   N           multiple of 256
 *   gathered    device, bf16 [M][K]: receives G[s*R + i] = shard s row i
 *   out         device, bf16 [M][N]: out = G x W, fp32 accumulation,
 *               rounded to nearest even
 * One round: producers copy every row and publish each 64-row chunk; each
 * consumer tile waits for its chunks' slots to reach this round's sequence. */
int tovl_gather_gemm(tovl_handle h, const void* const* shards, int num_shards, int rows_per_shard, int K,
                     const void* W, int N, void* gathered, void* out, void* stream);

/* Rows a dispatch buffer needs: T*k + E*127 rounded up to a multiple of 128. */
long long tovl_dispatch_rows(int T, int k, int E);

/* The same bound for expert segments aligned to `align` rows (128, or 256 with
 * option 17): T*k + E*(align-1) rounded up to a multiple of align; 0 for any
 * other align. */
long long tovl_dispatch_rows_aligned(int T, int k, int E, int align);

/* Dispatch scatter of top-k routed tokens into padded per-expert segments,
 * followed by a grouped GEMM per expert (notify-stage counting of the DeepEP
 * FIFO-pipeline page; row-block counters with padding seeds of section 5).
 *   x           device, bf16 [T][H] (may be null when T = 0)
 *   topk_idx    device, int32 [T][k]: expert of pair (t, j), each in [0, E);
 *               not the -1 that tovl_route_topk leaves in a masked slot
 *               (may be null when T = 0: a round without tokens, whose plan
 *               is empty and whose call still counts as one round)
 *   H           multiple of 64, at most 32768 (the GEMM K)
 *   W           device, bf16 [E][H][N], N multiple of 256
 *   dispatched  device, bf16 [tovl_dispatch_rows(T,k,E)][H]: rows of expert e
 *               occupy [off[e], off[e] + count[e]) in ascending (t, j) order;
 *               the segment is padded with zero rows to a multiple of 128
 *   expert_offsets device, int32 [E+1]: receives off[]; off[E] = padded total
 *   out         device, bf16 [tovl_dispatch_rows(T,k,E)][N]: rows [off[e],
 *               off[e+1]) = dispatched rows x W[e]; padding rows are zero;
 *               rows >= off[E] are not written
 * Padding rows of `dispatched` are re-zeroed whenever the segment layout or
 * the buffer differs from the previous dispatch call on this handle.  An
 * expert id outside [0, E) makes the round a no-op that sets
 * TOVL_ERR_INVALID in the status word. */
int tovl_dispatch_grouped_gemm(tovl_handle h, const void* x, int T, int H, const int* topk_idx, int k, int E,
                               const void* W, int N, void* dispatched, int* expert_offsets, void* out,
                               void* stream);

/* GEMM + reduce-scatter over logical shards (a row-parallel layer: ReduceScatter
 * is the collective the platform page benchmarks beside AllGather, section
 * 3).  Shard s holds the K-slice X_s [M][Ks] of the activations and W_s
 * [Ks][N] of the weights; its partial P_s = X_s x W_s is computed by the
 * consumer CTAs (fp32 accumulation, rounded to bf16) and every partial tile
 * is published with the single-writer protocol: its epilogue warps arrive on
 * the tile's counter (acq_rel) once their stores are in global memory, and
 * the last arrival release-stores the sequence into the tile's slot.  The
 * reducers poll the S slots of an output tile (acquire) and write
 *   out[m][n] = bf16( sum_s f32(P_s[m][n]) ), fp32 sums in ascending s.
 * By default producer CTAs reduce; with option 19 = 1 (and no producer count
 * set) the reducer of output tile o is the CTA pair that computes shard
 * (o mod S)'s partial of it.
 *   X           device, bf16 [S][M][Ks]
 *   num_shards  S, 1..64
 *   M           rows, a multiple of 128
 *   Ks          multiple of 64, at most 32768
 *   W           device, bf16 [S][Ks][N], N a multiple of 256
 *   partials    device, bf16 [S][M][N]: receives P_s
 *   out         device, bf16 [M][N]: receives the reduced rows
 * Partial tiles (S x (M/128) x (N/256), or half that with CTA pairs) must
 * not exceed max_rows/64 x k_slices, the handle's counter capacity.  One
 * round (one sequence number). */
int tovl_gemm_reduce_scatter(tovl_handle h, const void* X, int num_shards, int M, int Ks, const void* W, int N,
                             void* partials, void* out, void* stream);

/* Combine: the reverse of the last dispatch round on this handle ("cross-GPU
 * sync protocols on PCIe", section 3, the layer-1 combine: every expert
 * output row goes back to its token's staging row; each 64-row staging chunk
 * is counted with acq_rel atomics and published by the elected last writer;
 * reducers poll the chunk slots with acquire loads).
 *   y           device, bf16 [rows][N]: expert outputs in the dispatched layout
 *               of the last tovl_dispatch_grouped_gemm call (its `out`)
 *   N           row length of y, multiple of 64, at most 32768
 *   gate_w      device, fp32 [T][k]: weight of pair (t, j)
 *   staging     device, bf16 [T*k][N]: receives staging[t*k + j] = y[dst(t, j)]
 *   combined    device, bf16 [T][N]: receives round-to-nearest-even of
 *               sum_j gate_w[t][j] * staging[t*k + j], every product and every
 *               partial sum rounded to fp32, j ascending
 *   stream      cudaStream_t, ordered after the dispatch call
 * T, k and the routing plan are the last dispatch call's; T*k <= max_rows.
 * Without an earlier dispatch on the handle the call returns
 * TOVL_ERR_INVALID; after a dispatch whose plan was rejected (bad expert id)
 * the round is a no-op that sets TOVL_ERR_INVALID in the status word; after
 * a dispatch round without tokens (T = 0) the call returns TOVL_OK and does
 * nothing (no round).  Otherwise one round (one sequence number), like the
 * other calls.  With option 18 on (the default) and no producer count set,
 * every CTA copies in 10 of its 16 warps and reduces in the other 6;
 * otherwise producer CTAs copy (option 1, default 7/12 of the SMs) and the
 * remaining SMs reduce. */
int tovl_combine(tovl_handle h, const void* y, int N, const float* gate_w, void* staging, void* combined,
                 void* stream);

/* ---------------------------------------------------------------- no-allocation plan
 * The pages have no counterpart to this entry point; it serves callers that
 * must not allocate device memory themselves (code inside another
 * framework's memory budget, latency-critical loops that cannot afford
 * cudaMalloc's device-wide synchronisation, plugins whose host owns every
 * allocation).
 *
 * tovl_dispatch_plan_noalloc computes the routing plan of a dispatch round
 * -- the same kernels and results as tovl_dispatch_grouped_gemm's plan --
 * without a handle and without allocating: its scratch is one fixed device
 * array inside the library (about 0.3 MB, held by every GPU that loads the
 * library until the process exits).
 *   topk_idx        device, int32 [T][k], expert of each pair in [0, E)
 *   expert_offsets  device, int32 [E+1]: padded segment starts (multiples of
 *                   128); all zero if an expert id is out of range (the only
 *                   report of that error: this entry point has no status word)
 *   dst_rows        device, int32 [T*k]: destination row of each pair, rows
 *                   of one expert in ascending (t, j) order; not written when
 *                   an expert id is out of range
 *   stream          cudaStream_t; the call is asynchronous
 * Limits: T*k <= TOVL_NOALLOC_MAX_PAIRS and E <= TOVL_NOALLOC_MAX_EXPERTS;
 * larger sizes return TOVL_ERR_UNSUPPORTED before anything is enqueued.
 * It runs on the calling thread's current device.  The first call on a
 * device looks up the scratch array's device address (cudaGetSymbolAddress)
 * and keeps it for the life of the process; make that first call before any
 * stream capture.  The kept address does not survive a reset of the device
 * (cudaDeviceReset, or a reset of its primary context): after one, this
 * entry point must not be called again in that process.  All calls
 * on a device share the one array and it keeps the previous call's
 * contents, so calls whose kernels overlap on the GPU (other streams, other
 * threads) race and must be serialised by the caller. */
#define TOVL_NOALLOC_MAX_PAIRS 32768
#define TOVL_NOALLOC_MAX_EXPERTS 64
int tovl_dispatch_plan_noalloc(const int* topk_idx, int T, int k, int E, int* expert_offsets, int* dst_rows,
                               void* stream);

/* ---------------------------------------------------------------- decode step
 * Operators of a serving step around the experts, for few tokens as well as
 * many: the norm before the layer, the router, the whole expert layer for up
 * to 64 tokens, and products of up to 64 rows with 4-bit weights.  Longer
 * batches have no gated layer here: tovl_dispatch_grouped_gemm multiplies
 * scattered rows by one bf16 matrix per expert and tovl_combine adds its rows
 * up, with no activation between and no slots without an expert.  None of the
 * calls below is a protocol round: the sequence number stays.  T = 0 is
 * accepted everywhere, does nothing and reads no tensor.
 *
 * Packed 4-bit weights of a matrix W [K][N] (N contiguous): 32-bit words
 * [K/8][N]; the word of (r, n) holds rows 8r .. 8r+7 of column n, row 8r+2i in
 * bits 4i .. 4i+3 and row 8r+2i+1 in bits 16+4i .. 16+4i+3.  A group is
 * `group` rows (32, 64 or 128; K a multiple of it) of one column:
 *   W[k][n] = (nibble - zero[k/group][n]) * scale[k/group][n],
 * scale bf16 [K/group][N], zero uint8 [K/group][N] with values 0 .. 15, or a
 * null pointer for zero = 8 throughout.  N is a multiple of 8, with zeros of
 * 16; all pointers are 16-byte aligned.  Stacked matrices (one per expert)
 * are contiguous. */

/* Element types of the calls below. */
typedef enum {
    TOVL_BF16 = 0,
    TOVL_F32 = 1,
    TOVL_E4M3 = 2              /* 8-bit float, 4 exponent and 3 mantissa bits, largest value 448 */
} tovl_type;

/* Residual addition, root-mean-square norm and 8-bit output in one pass:
 *   r = x + residual                        (fp32)
 *   y = r * rsqrt(mean(r^2) + eps) * weight (fp32, mean over the row)
 *   residual_out = r, out = y, each rounded once to its type;
 *   per group of columns: scale = max(max |y|, 1e-12) / 448,
 *   q = e4m3(y / scale), rounded to nearest even.
 *   x           device, bf16 [T][H], rows ldx elements apart
 *   residual    device, [T][H] of residual_type (TOVL_BF16 or TOVL_F32), rows
 *               ldr elements apart; null = none (r = x; residual_out unused)
 *   residual_out device, type and row distance of residual; may be residual
 *   weight      device, bf16 [H]
 *   out         device, bf16 [T][H], rows ldo apart (may be x); null = not wanted
 *   q           device, e4m3 [T][H] contiguous; null = not wanted (then
 *               q_scale and group are ignored).  One of out and q is given.
 *   q_scale     device, fp32 [T][ceil(H/group)]
 *   group       32, 64 or 128, or 0 for one scale per row; the last group of
 *               a row may be shorter
 * H is 1 .. 32768; pointers need the alignment of their element type only
 * (rows of 16-byte multiples and alignment are fastest, then tensors whose
 * rows start equally far from a 16-byte boundary).  A NaN in a row
 * shows in all of its outputs. */
int tovl_add_rmsnorm(tovl_handle h, const void* x, long long ldx, const void* residual, void* residual_out,
                     int residual_type, long long ldr, const void* weight, float eps, int T, int H, void* out,
                     long long ldo, void* q, float* q_scale, int group, void* stream);

/* Softmax routing: the k largest logits of each token, the lowest expert
 * first among equal ones, and their softmax weights.
 *   logits      device, bf16 or fp32 (type) [T][E], rows ld elements apart
 *   E, k        E 1 .. 512, k 1 .. 32
 *   renormalize 1: weights over the chosen experts (they sum to 1); 0: over all
 *   topk_idx    device, int32 [T][k], in descending logits
 *   gate_w      device, fp32 [T][k]
 * An expert whose logit is -inf or NaN is masked: never chosen, weight 0.
 * Slots that no expert is left for hold -1 with weight 0 (a token whose
 * logits are all masked has nothing but those); +inf counts as the largest
 * finite logit does.  tovl_moe_decode takes the -1; tovl_dispatch_grouped_gemm
 * does not: routing for it needs k experts that are not masked per token. */
int tovl_route_topk(tovl_handle h, const void* logits, int type, long long ld, int T, int E, int k, int renormalize,
                    int* topk_idx, float* gate_w, void* stream);

/* Bytes of workspace that tovl_moe_decode[_q4] needs for these sizes on the
 * handle's device; -1 if the sizes are not supported. */
long long tovl_moe_decode_workspace(tovl_handle h, int T, int k, int H, int I);

/* The gated expert layer for a few tokens:
 *   h(t, e) = silu(x[t] W13[e][:, 0:I]) * (x[t] W13[e][:, I:2I]),
 *   out[t]  = sum over j of gate_w[t][j] * (h(t, e) W2[e]), e = topk_idx[t][j]
 * with fp32 sums, rounded once to bf16.  Between the two products h is kept as
 * two bf16 numbers, which leave 2^-16 of it (an h over bf16's largest number
 * is infinite).  Weights are finite; a sum with an infinite one may be
 * infinite or NaN.
 *   x           device, bf16 [T][H], rows ldx elements apart (a multiple of 8),
 *               16-byte aligned; T 0 .. 64, H a multiple of 8 up to 32768
 *   topk_idx    device, int32 [T][k]: experts, or -1 for a slot without one
 *               (masked, or an expert that lives elsewhere); k 1 .. 16.
 *               Other ids outside [0, E) make the call a no-op that sets
 *               TOVL_ERR_INVALID in the status word.
 *   gate_w      device, fp32 [T][k]; weights of -1 slots are not read
 *   E           1 .. 512
 *   W13         device, bf16 [E][H][2I]: gate columns, then up columns
 *   W2          device, bf16 [E][I][H]; I a multiple of 8 up to 32768
 *   out         device, bf16 [T][H], rows ldo apart; a token without experts
 *               gets zeros
 *   workspace   device, 256-byte aligned, tovl_moe_decode_workspace bytes of
 *               any content; free again when the call's kernels have ended
 * The weights of experts that no token names are not read.  Small layers take
 * two kernels, others one whose grid meets at three barriers: all its CTAs (one
 * per SM) must be resident together, and option 13 keeps the guarantee.
 * Results are the same bits on every call with the same arguments. */
int tovl_moe_decode(tovl_handle h, const void* x, long long ldx, int T, int H, const int* topk_idx,
                    const float* gate_w, int k, int E, const void* W13, const void* W2, int I, void* out,
                    long long ldo, void* workspace, long long workspace_bytes, void* stream);

/* The same layer with packed 4-bit experts: W13 [E] matrices [H][2I], W2 [E]
 * matrices [I][H], with zeros for both or for neither; H and I multiples of
 * group.  Scales are applied to fp32 sums.  h is rounded to fp16 times a power
 * of two per 128 columns of I: 2^-11 of it at most, and below 2^-28 of the
 * largest of the 128 an absolute 2^-39 of that. */
int tovl_moe_decode_q4(tovl_handle h, const void* x, long long ldx, int T, int H, const int* topk_idx,
                       const float* gate_w, int k, int E, const void* W13_q, const void* W13_scale,
                       const void* W13_zero, const void* W2_q, const void* W2_scale, const void* W2_zero, int group,
                       int I, void* out, long long ldo, void* workspace, long long workspace_bytes, void* stream);

/* Bytes of workspace that tovl_matvec_q4 needs; -1 if not supported. */
long long tovl_matvec_q4_workspace(tovl_handle h, int T, int N);

/* Few rows times one packed 4-bit matrix: out[t] = x[t] W, fp32 sums, rounded
 * once to bf16.
 *   x           device, [T][K], rows ldx elements apart, 16-byte aligned rows:
 *               bf16, or e4m3 (x_type) with x_scale; T 0 .. 64, K up to 32768
 *   x_scale     device, fp32 [T][ceil(K/128)]: x[t][k] stands for
 *               x * x_scale[t][k/128] (the q and q_scale of tovl_add_rmsnorm
 *               with group 128); null for bf16
 *   wq, w_scale, w_zero, group  the packed matrix [K][N], N up to 2^24
 *   out         device, bf16 [T][N], rows ldo apart
 *   workspace   device, 256-byte aligned, tovl_matvec_q4_workspace bytes of
 *               any content */
int tovl_matvec_q4(tovl_handle h, const void* x, int x_type, const float* x_scale, long long ldx, int T, int K,
                   const void* wq, const void* w_scale, const void* w_zero, int group, int N, void* out,
                   long long ldo, void* workspace, long long workspace_bytes, void* stream);

/* Quantises bf16 matrices W [E][K][N] into the packed form, rounding to
 * nearest: without zeros (w_zero null) scale = max |w| / 7, with zeros scale =
 * (max(w, 0) - min(w, 0)) / 15 and zero = round(-min(w, 0) / scale), the scale
 * rounded to bf16 first; 1 (and nothing but zeros) where that rounds to 0.
 * Any finite weights. */
int tovl_quantize_q4(tovl_handle h, const void* W, int E, int K, int N, int group, void* wq, void* w_scale,
                     void* w_zero, void* stream);

/* ---------------------------------------------------------------- paged attention step
 * Operators of a serving step around the key-value cache: pages and cache
 * slots for the step's new tokens, their rotary embedding with the cache
 * writes, and attention of one new token per request.  A cache is pages of
 * `page` slots that requests own through a block table: token t of request b
 * lies in slot t % page of page table[b][t / page].  The calls take their
 * arguments in a struct, read before they return (one pointer to pass where a
 * short call's time is the host's).  None of them is a protocol round; a batch
 * of 0 requests or tokens does nothing.  Tensors do not overlap unless said so. */

/* Element (page p, slot s, head g, column d) of the keys and of the values is
 * p * page_stride + s * slot_stride + g * head_stride + d elements from k and
 * v.  An e4m3 cache has one fp32 scale per slot and head for each of the two:
 * a row stands for its elements times k_scale (v_scale) [p][g][s], not negative
 * and contiguous.  k and v are 16-byte aligned, dim and the strides multiples
 * of 16 bytes, strides at least dim (those of extents of 1 are not used). */
typedef struct {
    void* k;
    void* v;
    float* k_scale;            /* [pages][heads][page]; null for bf16 */
    float* v_scale;
    int type;                  /* TOVL_BF16 or TOVL_E4M3 */
    int pages;                 /* pages * page < 2^31 */
    int page;                  /* slots of a page, any number */
    int heads;
    int dim;                   /* columns, up to 256 */
    long long page_stride, slot_stride, head_stride;   /* elements */
} tovl_kv_cache;

/* Pages, cache slots and positions of a step's new tokens, in one kernel.
 *   length      device, int32 [B]: tokens that each request holds; B 0 .. 4096
 *   add         device, int32 [B]: new tokens (0 for none), or -1 for a request
 *               that has ended and gives its pages back
 *   table       device, int32 [B][width], rows ldt apart: pages of each request,
 *               ceil(length / page) of them in use; receives the new ones behind
 *   ring        device, int32 [pages]: free pages, from entry state[0] on (it
 *               goes on at entry 0 behind the last); given-back pages are
 *               written behind the free ones
 *   state       device, int32 [4]: first free entry, number of free pages; the
 *               other two are not read
 *   length_out  device, int32 [B]: length + add, 0 for a request that has ended;
 *               may be length
 *   state_out   device, int32 [4]: the new state, then the number of new tokens
 *               and of lacking pages; may be state
 *   slots, positions device, int32 [cap], cap up to 2^30: for the new tokens of
 *               request 0, 1, ... in the order of their positions page *
 *               table[b][position / page] + position % page and position; behind
 *               the last -1 and 0
 *   starts      device, int32 [B+1]: first new token of each request in slots,
 *               and their number
 * New pages are taken from the ring in the order of requests and positions;
 * pages that a call gives back serve from the next call on, in the same order.
 * A page is one request's: given back by two that share it, it is in the ring twice.
 * With too few free pages nothing changes: no new tokens (slots all -1),
 * length_out = length, state_out[3] = the pages that are lacking.  Counts that
 * cannot be (a length below 0 or add below -1, more tokens than width pages or
 * cap hold, more free pages than there are) leave everything as it was too, with
 * state_out[3] = -1, and set TOVL_ERR_INVALID in the status word. */
typedef struct {
    const int* length;
    const int* add;
    int* table;
    int* ring;
    const int* state;
    int* length_out;
    int* state_out;
    int* slots;
    int* positions;
    int* starts;
    long long ldt;
    int B, width, pages, page, cap;
} tovl_page_plan_args;
int tovl_page_plan(tovl_handle h, const tovl_page_plan_args* args, void* stream);

/* Rotary embedding of queries and keys; keys and values to their cache slots.
 * With c and s the cosine and sine of pair i at the token's position,
 *   (x, y) -> (x c - y s, y c + x s), i = 0 .. rot/2 - 1,
 * of columns (i, i + rot/2), or (2 i, 2 i + 1) with interleaved; columns from
 * rot on stay.  In fp32, rounded once to bf16; to an e4m3 cache
 *   scale = max(max |x|, 1e-12) / 448 of the row, e4m3(x / scale), ties to even.
 *   q           device, bf16 [T][Hq][dim], tokens ldq elements apart
 *   k, v        device, bf16 [T][heads][dim], ldk and ldv apart
 *   positions   device, int32 [T], in [0, max_pos)
 *   slots       device, int32 [T]: page * page id + slot, all different; -1: the
 *               token is not written (its position is not checked, its q_out
 *               means nothing if it is out of range)
 *   cos_sin     device, fp32 [max_pos][rot]: rot/2 cosines, rot/2 sines
 *   rot         a multiple of 16 up to dim, 0 for none (cos_sin unused)
 *   q_out       device, bf16 [T][Hq][dim], ldqo apart; may be q
 * Token rows are 16-byte aligned, their distances multiples of 8 elements.
 * Another slot or position sets TOVL_ERR_INVALID in the status word; its keys
 * and values are not written.  A NaN in a row of an e4m3 cache makes its scale
 * NaN. */
typedef struct {
    const void* q;
    const void* k;
    const void* v;
    void* q_out;
    const int* positions;
    const int* slots;
    const float* cos_sin;
    const tovl_kv_cache* cache;
    long long ldq, ldk, ldv, ldqo;
    int T, Hq, max_pos, rot, interleaved;
} tovl_rope_append_args;
int tovl_rope_append(tovl_handle h, const tovl_rope_append_args* args, void* stream);

/* Bytes of workspace that tovl_attn_decode needs on the handle's device, any
 * batch and lengths; -1 if the sizes are not supported. */
long long tovl_attn_decode_workspace(tovl_handle h, int Hq, int heads, int dim);

/* Attention of one new token per request over its cached tokens, the new one
 * among them:
 *   z[t] = scale * q[b][g] . k[t], t from max(0, length - window) (0 without a
 *   window) to length - 1, k and v of head g / (Hq / heads),
 *   out[b][g] = sum of softmax(z)[t] v[t], lse[b][g] = ln sum exp z[t]
 * with fp32 sums of weights, up to 2^8 each, times values, rounded once to bf16.
 * Weights are off by 2^-15 of themselves with a bf16 cache (0 below 2^-126 of a
 * row's largest), with an e4m3 one by 2^-11, and where weight times v_scale is
 * below 2^-14 of a row's largest by 2^-25 of that, or by 2^-73 where the largest
 * is below 2^-48.  With an e4m3 cache scores are up to 2^26 in magnitude.
 *   q           device, bf16 [B][Hq][dim], requests ldq elements apart (a
 *               multiple of 8), 16-byte aligned; Hq a multiple of heads
 *   table       device, int32 [B][width], rows ldt apart
 *   length      device, int32 [B], 0 .. width * page, below 2^31 - 63; B 0 .. 65536
 *   window      the last tokens that are seen; 0 = all
 *   out         device, bf16 [B][Hq][dim], ldo apart, like q; a request of
 *               length 0 gets zeros and an lse of -inf
 *   lse         device, fp32 [B][Hq]; null = not wanted
 *   workspace   device, 256-byte aligned, any content; free again when the
 *               call's kernel has ended
 * Entries of the table outside the pages that hold seen tokens are not read;
 * what slots of those pages hold that no seen token lies in does not matter.
 * A page outside [0, pages) or a length out of range sets TOVL_ERR_INVALID in
 * the status word, and 2^31 - 1 tiles or more (of 16 to 64 tokens of a key head
 * for 8 or 16 of its query heads) set TOVL_ERR_UNSUPPORTED; the result of the
 * request, or of all, means nothing then.
 * Infinite and NaN keys and values that are seen show in the results that see
 * them (an infinite value as infinite, or as NaN where its weight is 0 and in an
 * e4m3 cache, where its scale is infinite); seen tokens whose scores are all
 * -infinite give zeros and an lse of -inf.  The result of a call depends on its
 * arguments alone (the same bits on every call on the same device). */
typedef struct {
    const void* q;
    void* out;
    float* lse;
    const int* table;
    const int* length;
    const tovl_kv_cache* cache;
    void* workspace;
    long long ldq, ldo, ldt, workspace_bytes;
    int B, Hq, width, window;
    float scale;
} tovl_attn_decode_args;
int tovl_attn_decode(tovl_handle h, const tovl_attn_decode_args* args, void* stream);

/* ---------------------------------------------------------------- controls
 * The acceptance method of the platform page, section 5, compares the fused
 * kernel with its parts run alone on the same SM counts. */

/* GEMM-only control: the consumer CTAs of tovl_gather_gemm (same count C)
 * with gates disabled, on an already filled A.  A: device bf16 [M][K],
 * W: device bf16 [K][N], out: device bf16 [M][N].  Not a protocol round. */
int tovl_gemm_only(tovl_handle h, const void* A, int M, int K, const void* W, int N, void* out, void* stream);

/* Copy-only control: the producer CTAs of tovl_gather_gemm (same count P)
 * with the full protocol and no consumers.  Arguments as tovl_gather_gemm.
 * A protocol round. */
int tovl_copy_only(tovl_handle h, const void* const* shards, int num_shards, int rows_per_shard, int K,
                   void* gathered, void* stream);

/* Permuted row copy dst[perm[i]] = src[i] over 64-row destination chunks.
 *   src, dst    device, n_rows x row_bytes each (row_bytes multiple of 16)
 *   perm        device, int32 [n_rows], a permutation of [0, n_rows)
 *   gated       1: every row is an arrival on its destination chunk, the last
 *               arrival publishes the chunk slot, waiter CTAs observe the
 *               slots (a protocol round); 0: the same copy with no
 *               protocol (not a round)
 *   stamps      1: record publish and first-observe times per chunk
 *               (read them with tovl_read_latency)
 * The copy mechanism is the handle's copy mode (option 3): vector copies, bulk
 * copies (rows up to 24 KB; larger rows return TOVL_ERR_UNSUPPORTED), or the
 * default automatic choice by row size.  Results are identical in every mode. */
int tovl_gated_copy(tovl_handle h, const void* src, void* dst, long long n_rows, int row_bytes, const int* perm,
                    int gated, int stamps, void* stream);

/* ---------------------------------------------------------------- diagnostics */

/* Synchronises the handle's last stream, returns the sticky device status
 * (TOVL_OK if none) and clears it. */
int tovl_sync_status(tovl_handle h);

/* Lengths of the control-plane arrays: chunk slots/counters
 * (max_rows/64 chunks x k_slices, index chunk*k_slices + slice) and
 * row-block counters (max_rows/128 blocks x k_slices). */
int tovl_ctrl_sizes(tovl_handle h, int* n_chunks, int* n_blocks);

/* Copies the control plane to host arrays (after synchronising): slots and
 * cnts [n_chunks], rbcnts [n_blocks] (lengths from tovl_ctrl_sizes);
 * *seq = calls that were protocol rounds.
 * Any pointer may be NULL. */
int tovl_read_ctrl(tovl_handle h, int* slots, int* cnts, int* rbcnts, long long* seq);

/* Copies the last dispatch round's plan to host arrays (after
 * synchronising): counts [E], dst [T*k], src_of_dst [m_pad] (token of each
 * row, -1 for padding), pad [m_pad/128], blk_expert [m_pad/128], *m_pad.
 * Any pointer may be NULL. */
int tovl_read_plan(tovl_handle h, int* counts, int* dst, int* src_of_dst, int* pad, int* blk_expert, int* m_pad);

/* Options for sweeps: 1 = producer CTAs (0 = automatic split; reads back
 * the count the last call used), 2 = consumer CTAs, 3 = copy mode,
 * 4 = statistics on/off, 5 = wait timeout in ns, 6 = copy-sweep CTAs,
 * 7 = copy-sweep waiter CTAs, 9 = k_slices (read only),
 * 10 = CTA-pair consumers for gather calls (1 = on, the default: two CTAs of a
 * cluster compute a 256x256 tile with cta_group::2 MMAs; 0 = one CTA per
 * 128x256 tile; reads back 0 if the device cannot co-schedule pairs),
 * 11 = co-resident CTA pairs on the device (read only), 12 = 1 if
 * cooperative launches are accepted with pairs (read only), 13 = fused
 * launches request the cooperative co-residency guarantee (1, the default;
 * 0 launches the same kernel without it, for tools that cannot replay
 * cooperative launches -- the grid still fits one CTA per SM; the same
 * switch applies to the combine kernel and to gated copies),
 * 14 = producer copy path of the fused kernels: 0 = 16-byte vector loads and
 * stores through registers (the default), 1 = bulk asynchronous loads of each
 * row segment into a per-warp shared-memory buffer, then 16-byte vector
 * stores (results are identical),
 * 15 = programmatic dependent launch between the library's own kernels
 * (1, the default: a kernel's launch and prologue overlap the end of the
 * kernel before it -- plan counting, plan finalisation, the fused kernel,
 * combine -- and every kernel waits for its predecessor before it reads
 * memory; 0 = plain stream order; reads back 0 if the device refused it),
 * 16 = role switch (1, the default; 0 = fixed roles; 2 = also for CTA-pair
 * tiles): in tovl_dispatch_grouped_gemm with producer CTAs (option 18 = 0)
 * consumer tiles are handed out by a ticket counter and producer CTAs take
 * tiles once their copies are done
 * (the automatic split then gives the copy twice its balance share); with
 * 256-row segments this applies at 2 only (a CTA pair takes one ticket for
 * both CTAs; measured about 1 % slower than fixed pair roles on the uniform
 * and Zipf workloads, whose last wave the joining producers cannot fill); in
 * tovl_gemm_reduce_scatter consumer CTAs that have finished their partial
 * tiles take reduction items beside the producer CTAs,
 * 17 = expert segment alignment of tovl_dispatch_grouped_gemm in rows: 128
 * (the default: segments padded to the 128-row block, the layout the oracle
 * defines) or 256 (segments padded to two blocks, so CTA pairs compute
 * 256-row tiles inside one expert; the padded rows are zero and their
 * block counters are seeded like any padding; buffers then need
 * tovl_dispatch_rows_aligned(T, k, E, 256) rows; with embedded producers
 * CTA pairs run 128-row segments as well, two blocks of a segment per pair
 * tile, a segment's odd last block beside a phantom half that is computed
 * but never stored, so 256 no longer buys speed there),
 * 18 = embedded producers (1, the default: in tovl_dispatch_grouped_gemm and
 * tovl_combine;
 * 2 = also in tovl_gather_gemm; 0 = off): the call launches no producer
 * CTAs; every SM (every co-resident CTA pair) is a consumer and the
 * consumer CTAs' four spare warps copy the rows, in the producers' order and
 * with their counters and seeds (16-byte vector copies whatever option 14
 * says; the role switch does not apply; CTA pairs on 128-row segments, see
 * 17).  Measured on GB300: dispatch calls 16-17 % shorter than with
 * producer CTAs and single-CTA tiles (uniform 141.5 -> 118 us, Zipf 793 ->
 * 670 us), the TP gather 4-6 % slower (its three tile waves
 * stay three; the copy warps share the SMs),
 * 19 = where tovl_gemm_reduce_scatter sums the partials: 0 (the default) =
 * producer CTAs reduce, consumers join them when option 16 is on; 1 (when no
 * producer count is set) = every SM computes partial tiles and the CTA pair
 * that computes shard (o mod S)'s partial of output tile o sums that tile's S
 * partials in five otherwise idle warps, once all S partial tiles' slots are
 * published,
 * 20 = L2 eviction priorities of the fused calls' memory streams, a bit mask:
 * 1 producer source loads evict-last, 32 evict-first; 16 producer
 * destination stores evict-last; 4 A tensor loads evict-first; 8 weight
 * tensor loads evict-last; 2 output tensor stores evict-first; 0 = no
 * priorities; -1 (the default) = each call's measured choice: 32 | 8 for
 * tovl_gather_gemm, 8 for tovl_dispatch_grouped_gemm, 0 otherwise (results
 * are identical whatever the mask),
 * 23 = tile width of tovl_dispatch_grouped_gemm's CTA-pair tiles with
 * embedded producers (128- or 256-row segments): 1 (the default)
 * = 256 x 512 tiles when N is a multiple of 512 (one 512-column accumulator,
 * half the activation loads per MMA), else 256 x 256; 0 = always 256 x 256
 * (results agree within the GEMM tolerance either way),
 * 8 = fault injection for tests: consumer gates
 * wait for sequence seq + value, which no producer publishes, so every gate
 * expires after the wait timeout and the call ends with TOVL_ERR_TIMEOUT in
 * the status word (0 = off). */
int tovl_set_option(tovl_handle h, int option, long long value);
int tovl_get_option(tovl_handle h, int option, long long* value);

/* Statistics of the last call with statistics on: [0] gate polls,
 * [1] earliest consumer start ns, [2] latest consumer end ns, [3] earliest
 * producer start ns, [4] latest producer end ns. */
int tovl_read_stats(tovl_handle h, unsigned long long* stats, int n);

/* Timeline of the last fused call made with statistics on (%globaltimer ns):
 *   what 0: publish time of each chunk slice [n_chunks], index chunk*k_slices + slice
 *           (0 where no producer thread published it)
 *   what 1: time the consumer's gate passed each (tile, slice) [tiles*k_slices]
 *   what 2: time each tile's output was stored [tiles]
 *   what 3: time each tile's accumulator was complete (epilogue start) [tiles]
 * Tiles are numbered row block * (N/256) + column block; for dispatch calls
 * the tile count is the bound tovl_dispatch_rows/128 * N/256 (unused tiles
 * read 0), with 512-column pair tiles (option 23) N/512 column blocks.
 * n must not exceed the stated length. */
int tovl_read_trace(tovl_handle h, int what, long long* out, long long n);

/* Publish and first-observe %globaltimer stamps of the first n chunks of the
 * last stamped tovl_gated_copy. */
int tovl_read_latency(tovl_handle h, long long* pub_ns, long long* obs_ns, int n);

/* Number of SMs of the handle's device. */
int tovl_num_sms(tovl_handle h);

const char* tovl_error_string(int code);

/* Text of the last CUDA error seen by this handle ("" if none). */
const char* tovl_last_error(tovl_handle h);

#ifdef __cplusplus
}
#endif

#endif /* TOVL_H */

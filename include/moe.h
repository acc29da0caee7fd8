/*
 * moe.h - C ABI of the GB300 (sm_103a) mixture-of-experts FFN block with
 * MLX-style group-64 affine quantised weights.
 *
 * The block (page "TurboFieldfare - System design"):
 *   1. router: logits[t, e] = sum_k W_r[e, k] x[t, k], W_r 8-bit affine,
 *      no softcap (section "Why the runtime has this shape"; section
 *      "Decode", router description);
 *   2. top-k (k = 8 of E = 128) with ties to the lower expert id, softmax
 *      over the k selected logits (section "Decode");
 *   3. per selected expert a 4-bit affine GeGLU FFN
 *      o = W_down (gelu_tanh(W_gate x) * (W_up x)) (section "Metal
 *      execution": fused affine decode + GeGLU + weighted reduction);
 *   4. y = sum_j w_j o_j + o_shared, the dense shared expert added with no
 *      routing weight (section "Why the runtime has this shape").
 * Prefill handles chunks of at most 128 rows (section "Prefill"), so every
 * call takes 1 <= n_tokens <= 128.
 *
 * Quantised matrix format (section "Why the runtime has this shape"): a
 * matrix W[N, K] is three arrays
 *   q      : packed codes, row-major, little-endian uint32 words; code i of a
 *            row at bits 4*(i%8) of word i/8 (4-bit) or 8*(i%4) of word i/4
 *            (8-bit, i.e. plain byte order);
 *   scales : bf16 [N, K/64], row-major;
 *   biases : bf16 [N, K/64], row-major;
 * and W[n, k] = q[n, k] * scales[n, k/64] + biases[n, k/64].
 *
 * Expert storage (section ".gturbo directory": fixed-stride, page-aligned
 * expert blobs whose sub-tensors sit at their own offsets): routed expert e
 * is the blob at experts + e * expert_stride; inside a blob the nine
 * sub-tensors (gate/up [I, H], down [H, I]; q, scales, biases each) sit at
 * the byte offsets of moe_blob_layout.  The shared expert is one more blob
 * with the same layout.
 *
 * Conventions for every call
 *   - Returns MOE_OK (0) or a MOE_ERR_* code; nothing throws across the ABI.
 *   - All tensor pointers are DEVICE pointers owned by the caller; the
 *     library never frees them.  The workspace `ws` is caller-owned device
 *     memory of at least moe_workspace_bytes() bytes, 256-byte aligned, and
 *     must not be shared by calls that may run concurrently.
 *   - Launches are asynchronous on `stream` (a cudaStream_t; NULL = the
 *     legacy default stream); no call synchronises the host except
 *     moe_get_error.  Inputs must stay valid until the stream reaches the
 *     call.
 *   - Arguments are checked on the host before anything is launched:
 *     null pointers, n_tokens outside [1, 128], dims the kernels do not
 *     support, pointers not 16-byte aligned (tensor data) or offsets not
 *     256-byte aligned -> MOE_ERR_INVALID_ARG / MOE_ERR_UNSUPPORTED and no
 *     launch.  Faults found on the device (an expert id out of range in
 *     moe_expert_ffn / moe_route_sort, non-finite router logits) never trap:
 *     the offending item is skipped and a device error word is set, read
 *     back by moe_get_error.
 *   - A handle may be used from one stream at a time (it owns the device
 *     error word and the router's completion counter).
 *   - The layer calls run one persistent launch per layer (one block per
 *     SM, blocks that wait for one another at grid barriers).  Their blocks
 *     must all be resident at once: while such a call runs, no other work
 *     may hold SMs of the device (a kernel on another stream, another
 *     process under MPS, a green context).  Otherwise blocks wait at a
 *     barrier until the bounded wait (2 s) gives up, the call records
 *     MOE_ERR_TIMEOUT and its outputs are not valid; moe_get_error then
 *     reports the timeout and restores the barrier state for the next call.
 *     Handles created with MOE_DECODE_FUSED=0 / MOE_PREFILL_FUSED=0 in the
 *     environment run separate launches that never wait for one another.
 */
#ifndef MOE_AFFINE_H
#define MOE_AFFINE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st *moe_stream_t; /* == cudaStream_t */

enum moe_status {
  MOE_OK = 0,
  MOE_ERR_INVALID_ARG = 1,   /* null pointer, bad size or alignment          */
  MOE_ERR_UNSUPPORTED = 2,   /* dims outside what the kernels implement       */
  MOE_ERR_CUDA = 3,          /* a CUDA runtime call failed                    */
  MOE_ERR_BAD_EXPERT_ID = 4, /* device: expert id outside [0, E) was skipped  */
  MOE_ERR_TIMEOUT = 5,       /* device: a bounded wait gave up                */
  MOE_ERR_NONFINITE = 6,     /* device: a router logit was NaN or infinite    */
  MOE_ERR_WORKSPACE = 7      /* workspace smaller than moe_workspace_bytes    */
};

/* Shapes.  Supported: group == 64; hidden, inter multiples of 64 with
 * 64 <= hidden <= 4096 and 64 <= inter <= 2048; 1 <= top_k <= 8;
 * top_k <= n_experts <= 128.  The target workload is hidden 2816,
 * inter 704, 128 experts, top-8. */
typedef struct {
  int hidden;    /* H: model width, input/output features of the block      */
  int inter;     /* I: expert intermediate width                            */
  int n_experts; /* E: routed experts                                       */
  int top_k;     /* k: experts selected per token                           */
  int group;     /* quantisation group along K; must be 64                  */
} moe_dims;

/* One quantised matrix: device pointers to codes, scales, biases. */
typedef struct {
  const void *q;
  const void *scales;
  const void *biases;
} moe_qmat;

/* Byte offsets of the nine sub-tensors inside one expert blob; each must be
 * a multiple of 256. */
typedef struct {
  size_t gate_q, gate_s, gate_b;
  size_t up_q, up_s, up_b;
  size_t down_q, down_s, down_b;
} moe_blob_layout;

/* Weights of one MoE layer (all device pointers). */
typedef struct {
  moe_dims dims;
  moe_qmat router;          /* 8-bit [E, H]                                   */
  const void *experts;      /* E routed blobs, fixed stride                   */
  size_t expert_stride;     /* bytes between blobs; multiple of 256           */
  moe_blob_layout layout;   /* sub-tensor offsets (routed and shared blobs)   */
  const void *shared;       /* the shared expert's blob                       */
  const float *logit_bias;  /* nullable [E]: added to the logits before top-k */
  /* The router's learned scales (section "Decode", router description),
   * both nullable (null: identity):
   *   router_scale      bf16 [H], 16-byte aligned: the router projects
   *                     x * router_scale / sqrt(H) instead of x (the experts
   *                     still take x);
   *   per_expert_scale  fp32 [E]: the routing weight of a selected expert e
   *                     is softmax(...) * per_expert_scale[e]. */
  const void *router_scale;
  const float *per_expert_scale;
  /* The layer tail (section "Decode", cb2 phase: post-FFN norm, residual,
   * learned layer scalar), both nullable; read only by the residual calls
   * (moe_layer_forward_residual, moe_layer_forward_stack):
   *   post_norm     bf16 [H], 16-byte aligned: norm weight g of
   *                 z = bf16(y / sqrt(mean(y^2) + 1e-6) * g) (null: z = y);
   *   layer_scalar  fp32 [1] on the device: h <- bf16(layer_scalar * bf16(h + z))
   *                 (null: h <- bf16(h + z)). */
  const void *post_norm;
  const float *layer_scalar;
} moe_layer_weights;

typedef struct moe_handle moe_handle;

/* Human-readable name of a status code (static string). */
const char *moe_status_string(int status);

/* Create / destroy a handle on the current CUDA device.  moe_create
 * allocates a few bytes of device memory (error word, counters) and sets
 * kernel attributes; it is the only call that allocates. */
int moe_create(moe_handle **out);
int moe_destroy(moe_handle *h);

/* Host-side validation of a layer description (no device access). */
int moe_check_weights(const moe_layer_weights *w);

/* Workspace bytes needed by moe_router_topk / moe_expert_ffn /
 * moe_layer_forward / moe_layer_forward_residual for n_tokens rows;
 * 0 if dims are unsupported or n_tokens is outside [1, 128]. */
size_t moe_workspace_bytes(const moe_dims *dims, int n_tokens);

/* Steps 1-2 (router projection, top-k, softmax weights).
 *   x        bf16 [T, H] row-major, the block input (already normalised)
 *   logits   nullable fp32 [T, E]: raw logits + logit_bias
 *   ids      int32 [T, k]: selected experts, by descending logit, ties to
 *            the lower id
 *   weights  fp32 [T, k]: softmax over the selected logits
 * Also leaves the token->expert grouping of step 3 in the workspace. */
int moe_router_topk(moe_handle *h, const void *x, int n_tokens, const moe_layer_weights *w,
                    float *logits, int32_t *ids, float *weights, void *ws, size_t ws_bytes,
                    moe_stream_t stream);

/* Step 3 on its own: stable counting sort of the pairs p = t*k + j by
 * expert id (section "Prefill": token/expert pairs grouped per expert).
 *   ids      int32 [T, k] device
 *   counts   int32 [E]       pairs per expert
 *   offsets  int32 [E + 1]   exclusive prefix sums of counts
 *   perm     int32 [T*k]     pair index at each sorted position
 *   pos      int32 [T*k]     sorted position of each pair (-1 if its id was
 *                            out of range; such pairs are dropped and
 *                            MOE_ERR_BAD_EXPERT_ID is recorded)
 * Runs one thread block; needs no workspace. */
int moe_route_sort(moe_handle *h, const int32_t *ids, int n_tokens, const moe_dims *dims,
                   int32_t *counts, int32_t *offsets, int32_t *perm, int32_t *pos,
                   moe_stream_t stream);

/* Steps 3-4 with caller-given routing (e.g. forced ids).
 *   x        bf16 [T, H];  ids int32 [T, k];  weights fp32 [T, k]
 *   include_shared  1: add the shared expert; 0: routed sum only
 *   y        bf16 [T, H] output
 * Out-of-range ids are skipped on the device (MOE_ERR_BAD_EXPERT_ID). */
int moe_expert_ffn(moe_handle *h, const void *x, int n_tokens, const int32_t *ids,
                   const float *weights, const moe_layer_weights *w, int include_shared, void *y,
                   void *ws, size_t ws_bytes, moe_stream_t stream);

/* The whole block, steps 1-4: y = MoE(x).
 *   x bf16 [T, H] in;  y bf16 [T, H] out;
 *   ids_out (int32 [T, k]), logits_out (fp32 [T, E]), weights_out
 *   (fp32 [T, k]) are nullable copies of the routing. */
int moe_layer_forward(moe_handle *h, const void *x, int n_tokens, const moe_layer_weights *w,
                      void *y, int32_t *ids_out, float *logits_out, float *weights_out, void *ws,
                      size_t ws_bytes, moe_stream_t stream);

/* One layer of a residual stack (the decode/prefill harness around the
 * block): x = bf16(h / sqrt(mean(h^2) + 1e-6)) (rmsnorm without scale, as
 * the router's input normalisation in section "Decode"); y = MoE(x);
 * h <- bf16(h + y) in place.  With a layer tail in w (post_norm and/or
 * layer_scalar set), h <- bf16(lambda * bf16(h + bf16(g * y / rms(y))))
 * instead, by one more launch after the block.
 *   hidden   bf16 [T, H] in/out
 *   y_out    nullable bf16 [T, H]: the block output before the add (and
 *            before the tail)
 *   x_out    nullable bf16 [T, H]: the normalised block input */
int moe_layer_forward_residual(moe_handle *h, void *hidden, int n_tokens,
                               const moe_layer_weights *w, void *y_out, void *x_out,
                               int32_t *ids_out, float *logits_out, void *ws, size_t ws_bytes,
                               moe_stream_t stream);

/* ---- whole-prompt layer (section "Prefill": layer-major execution; the
 * token/expert pairs grouped into bounded routed-MoE work; experts streamed
 * in tiles of at most eight, the next tile fetched while the current tile's
 * work is queued; shared and routed branches combined before the tail).
 *
 * The same function as moe_layer_forward_residual, for a prompt of up to
 * MOE_PROMPT_MAX_ROWS rows in one call:
 *   hidden <- bf16(hidden + MoE(rmsnorm(hidden)))   (or the layer's tail)
 * row by row.  Rows are routed independently; all rows' token/expert pairs
 * are grouped per expert and cut into chunks of at most 256 rows of one
 * expert, and every (chunk, 128 weight rows) is one unit of a persistent
 * tensor-core GEMM (tcgen05.mma, weights dequantised once per unit into fp16
 * on chip: w = q * s + b rounded once to fp16).  Units run the shared
 * expert first, then experts in ascending id, i.e. tile after tile of eight
 * experts, so an expert's weights come from HBM about once per layer and
 * its later chunks read them from L2; each SM prefetches its next unit's
 * weights into L2 while the current one runs.
 *   hidden    bf16 [n_rows, H] in/out
 *   n_rows    1 <= n_rows <= MOE_PROMPT_MAX_ROWS
 *   y_out, x_out, ids_out, logits_out: nullable, as in
 *             moe_layer_forward_residual ([n_rows, ...])
 *   ws        moe_prompt_workspace_bytes(dims, n_rows) bytes, 256-aligned
 *             (about 0.7 GB at 4096 rows of the target shape: the operand,
 *             h and fp32 expert-output rows of every sorted position)
 * Six launches (router, grouping, operand gather, gate/up GEMM, down GEMM,
 * combine; a seventh for a layer tail), none of which waits for another
 * block, so the call may share the device.  Errors as for the other layer
 * calls; MOE_ERR_UNSUPPORTED when the shape's tiles do not fit on chip.
 * Capturable in a CUDA graph (the tensor maps are kernel parameters). */
#define MOE_PROMPT_MAX_ROWS 4096
size_t moe_prompt_workspace_bytes(const moe_dims *dims, int n_rows);
int moe_layer_forward_prompt(moe_handle *h, void *hidden, int n_rows, const moe_layer_weights *w,
                             void *y_out, void *x_out, int32_t *ids_out, float *logits_out,
                             void *ws, size_t ws_bytes, moe_stream_t stream);

/* n_layers single-token layers of a residual stack in one call (the decode
 * step of the section "Decode": every layer's router input is the residual
 * stream normalised, its block output is added back):
 *   for l in 0 .. n_layers-1:  hidden <- bf16(hidden + MoE_l(rmsnorm(hidden)))
 * (or layer l's tail around it, as in moe_layer_forward_residual)
 * with MoE_l the block of layers[l] (all with the same dims); the same
 * launches as n_layers calls of moe_layer_forward_residual with n_tokens = 1.
 *   hidden   bf16 [H] in/out;  layers: host array of n_layers weight sets;
 *   ws       workspace of moe_workspace_bytes(dims, 1)
 * Validates every layer before the first launch; capturable. */
int moe_layer_forward_stack(moe_handle *h, void *hidden, int n_layers, const moe_layer_weights *layers,
                            void *ws, size_t ws_bytes, moe_stream_t stream);

/* ---- Expert offload (sections "Resource split", "Load and ownership" and
 * "Decode": every opened layer owns 16 routed-expert slots; after the router
 * (cb1) the host looks the selected experts up in the layer's cache, fills
 * only the missing slots (io), then the routed branch runs on the slots
 * (cb2); eviction is least frequently used, recency breaking ties).  Here
 * the routed experts stay in pinned host memory and the slots are device
 * memory, filled over the host link.
 *
 * moe_expert_cache is the host-side policy state of n_layers layers of
 * n_slots slots each (n_slots <= MOE_CACHE_MAX_SLOTS); it owns no device
 * memory.  Readings of the policy: an expert's use count starts at 1 when it
 * enters a slot and grows by 1 at each step that selects it; recency is the
 * step of its last selection; empty slots are taken first (lowest index);
 * a step's own experts are never evicted by its misses; remaining ties go to
 * the lower slot. */
#define MOE_CACHE_MAX_SLOTS 64
typedef struct moe_expert_cache moe_expert_cache;
int moe_cache_create(int n_layers, int n_slots, moe_expert_cache **out);
void moe_cache_destroy(moe_expert_cache *c);
/* One step of the policy for `n` selected experts `ids` (host int32) of
 * `layer`: slots[j] (host int32 [n]) = the slot holding ids[j] afterwards;
 * load_slots / load_ids (nullable host int32 [n]) = the slots to fill and
 * their experts, *n_loads of them.  MOE_ERR_UNSUPPORTED if the step has more
 * distinct experts than slots, MOE_ERR_BAD_EXPERT_ID for a negative id. */
int moe_cache_lookup(moe_expert_cache *c, int layer, const int32_t *ids, int n, int32_t *slots,
                     int32_t *load_slots, int32_t *load_ids, int *n_loads);
/* Hits and misses of a layer so far (a hit: a selected expert already in a slot). */
int moe_cache_stats(const moe_expert_cache *c, int layer, long long *hits, long long *misses);
/* The expert in a slot (-1: empty; -2: bad arguments). */
int moe_cache_slot_expert(const moe_expert_cache *c, int layer, int slot);
int moe_cache_slots(const moe_expert_cache *c);

/* One single-token layer of a residual stack with its routed experts in host
 * memory: the router on the device (rmsnorm of hidden, logits, top-k), the
 * ids copied to the host (one stream synchronisation: the CPU handoff of the
 * pages), moe_cache_lookup, one host-to-device copy per missing expert into
 * its slot, then the block (shared expert + the routed experts on their
 * slots) with hidden <- bf16(hidden + y) in place.  Results equal those of
 * moe_layer_forward_residual on resident experts with the chained launches
 * (the same kernels, the experts relabelled by slot).
 *   w        the layer: router and shared expert in device memory; w->experts
 *            pinned host memory of the E expert blobs (w->expert_stride apart)
 *   slots    device memory of this layer's slots: moe_cache_slots(c) blobs at
 *            w->expert_stride bytes each, 256-byte aligned, owned by the caller
 *   ws       workspace of moe_workspace_bytes(dims, 1)
 * No layer tail (MOE_ERR_UNSUPPORTED); not capturable in a CUDA graph (it
 * waits on the stream). */
int moe_layer_forward_offload(moe_handle *h, moe_expert_cache *c, int layer, void *hidden,
                              const moe_layer_weights *w, void *slots, void *ws, size_t ws_bytes,
                              moe_stream_t stream);

/* Single-token layer call that allocates nothing (the pages have no
 * counterpart: it exists for hosts that cannot allocate device memory,
 * e.g. a program whose own pool owns the whole device, or a per-token loop
 * where an allocation would stall the device and cannot be captured).
 * Same computation as moe_layer_forward with n_tokens = 1 on the fused
 * single-token kernel, but with no handle and no workspace.  Its scratch
 * lives in two static device arrays that every GPU loading this library
 * holds until the process exits:
 *   - 16 KiB: h, the logits when logits_out is NULL, the grid-barrier
 *     counter and the device error word;
 *   - 160 KiB: the logit mailboxes, 128 64-bit words per block of the grid
 *     (one block per SM, so devices with at most 160 SMs).
 *   x    bf16 [H] in;  y bf16 [H] out;  ids_out int32 [k], logits_out
 *        fp32 [E], weights_out fp32 [k] nullable.
 * Limits: (top_k + 1) * inter * 2 <= 15 KiB (top-8 of inter 704 uses
 * 12,672 B), at most 160 SMs, and the fused kernel's conditions
 * (n_experts <= SM count, its shared memory fits); otherwise
 * MOE_ERR_UNSUPPORTED and nothing is launched.  The first call on a device
 * looks up the arrays' device addresses and sets kernel attributes, so make
 * it before any stream capture.  The grid-barrier counter only grows (its
 * value gives each launch the epoch that tags its logits); the arrays keep
 * the last call's contents.  Calls that overlap on the GPU (different
 * streams, or the same arrays from two threads) race on the shared scratch.
 * Device-side errors (bounded-wait timeouts, non-finite values) accumulate
 * in the static error word until moe_static_get_error reads them. */
int moe_layer_forward_static(const void *x, const moe_layer_weights *w, void *y, int32_t *ids_out,
                             float *logits_out, float *weights_out, moe_stream_t stream);

/* The error word of moe_layer_forward_static on the current device: waits
 * for all work on the device, returns (in *status) the first device-side
 * error recorded since the last read (MOE_OK if none, or if no static call
 * ran on this device) and clears it.  After a timeout it also puts the
 * static grid-barrier counter and mailboxes back to zero, so the next static
 * call starts from a consistent state.  Allocates nothing. */
int moe_static_get_error(int *status);

/* ---- The tied 4-bit head and embedding (section "Why the runtime has this
 * shape": the embedding and the language-model head share one 4-bit affine
 * matrix, and the model ends with a logit softcap of 30; section "Decode":
 * the head returns the argmax token in a pure-greedy configuration, else the
 * full logits vector). */
typedef struct {
  int vocab;   /* V rows: a multiple of 16, at most 2^28                       */
  int hidden;  /* H columns: 64 .. 4096, a multiple of 64                      */
  moe_qmat w;  /* q uint32 [V, H/8] (code i at bits 4*(i%8) of word i/8),
                  scales and biases bf16 [V, H/64]; all 16-byte aligned        */
} moe_head_weights;

/* The head on up to 8 rows:
 *   logits[t, v] = cap * tanh((W x_t)[v] / cap)   (cap <= 0: no softcap)
 *   tokens[t]    = argmax_v logits[t, v], ties to the lower id
 *   x        bf16 [T, H], 16-byte aligned, T in [1, 8]
 *   logits   nullable fp32 [T, V];  tokens nullable int32 [T]; not both null
 * One kernel launch, graph-capturable.  The argmax state lives in the
 * handle (cleared by the launch that used it), so head calls on one handle
 * must not overlap on the GPU.  A non-finite logit is skipped by the argmax
 * and records MOE_ERR_NONFINITE. */
int moe_head_forward(moe_handle *h, const void *x, int n_tokens, const moe_head_weights *w, float softcap,
                     float *logits, int32_t *tokens, moe_stream_t stream);

/* A dense 4-bit affine projection in the same matrix format (section ".gturbo
 * directory": the production manifest stores the attention weights 4-bit
 * affine, group 64, like the embedding; section "Metal execution": single-
 * token decode runs projections as custom GEMV kernels), e.g. the
 * attention's Q/K/V and output projections:
 *   y[t, n] = sum_k W[n, k] x[t, k]
 *   w        W [N, K] as moe_head_weights (vocab = N rows, a multiple of 16;
 *            hidden = K columns, 64 .. 4096, a multiple of 64)
 *   x        bf16 [T, K], 16-byte aligned, T in [1, 8]
 *   y        nullable bf16 [T, N] (the fp32 sum rounded to nearest even)
 *   y32      nullable fp32 [T, N]; not both null
 * One launch of the head kernel with no softcap and no argmax, graph-
 * capturable; it does not touch the head's greedy state. */
int moe_dense_forward(moe_handle *h, const void *x, int n_tokens, const moe_head_weights *w, void *y, float *y32,
                      moe_stream_t stream);

/* The tied embedding: out[i] = bf16(q[ids[i], :] * scale + bias), the
 * dequantised row rounded once to bf16 (no scale factor).
 *   ids int32 [n] on the device, n >= 1;  out bf16 [n, H], 16-byte aligned.
 * An id outside [0, V) gives a zero row and records MOE_ERR_BAD_EXPERT_ID. */
int moe_embed(moe_handle *h, const int32_t *ids, int n, const moe_head_weights *w, void *out,
              moe_stream_t stream);

/* ---- From the residual stream to the next token, for a batch of rows.
 * Three calls that a decode loop over many sequences makes around the layers:
 * the residual addition and norm with 8-bit rows, the 8-bit projection that
 * takes them (an attention-like projection, or a head with its softcap for
 * more rows than moe_head_forward takes), and the processing of the logits.
 * Each is one or two launches, allocates nothing, and can be captured in a
 * CUDA graph.  The handle's device has to be the current one. */

/* Residual addition, root-mean-square norm and 8-bit rows.  Per row:
 *   s = bf16(hidden + y)                   (s = hidden without y)
 *   u = s * norm                           (u = s without norm)
 *   r = 1 / sqrt(mean(s^2) + eps),  m = max |u|
 *   q = rint(127 u / m)  (ties to even; zero for m = 0),  scale = m r / 127
 * so q * scale stands for the normalised row u r.  The codes are those of
 * exact arithmetic on the stored bf16 values (products below 2^-126 round to
 * fp32).
 *   hidden      bf16 [n_rows, width];  y nullable bf16 [n_rows, width]
 *   norm        nullable bf16 [width]
 *   eps         0 .. 1 (the layers use 1e-6; below 1e-30, rows whose values all
 *               lie below 2^-50 lose accuracy to the range of fp32)
 *   hidden_out  nullable bf16 [n_rows, width]: s; may be hidden itself;
 *               only with y
 *   q           int8 [n_rows, width], -127 .. 127;  scales fp32 [n_rows]
 *   x_out       nullable bf16 [n_rows, width]: bf16(u r)
 * width: a multiple of 16, 16 .. 16384; n_rows 1 .. MOE_NORM_MAX_ROWS;
 * matrices and norm 16-byte aligned.  Other outputs must not overlap an
 * input.  A row of zeros has codes and scale 0.  A row with a NaN or an
 * infinity in s or u, or whose sum of squares passes the range of fp32 (also
 * below, with eps = 0), or whose largest normalised value m r passes it (where
 * x_out is given that of bf16), gets codes 0, scale NaN and x_out NaN (s is
 * written all the same) and records MOE_ERR_NONFINITE. */
#define MOE_NORM_MAX_ROWS (1 << 20)
int moe_norm_quant(moe_handle *h, const void *hidden, const void *y, int n_rows, int width, const void *norm,
                   float eps, void *hidden_out, int8_t *q, float *scales, void *x_out, moe_stream_t stream);

/* An 8-bit matrix with a scale per output channel: W[n, k] = q[n, k] * scales[n]. */
typedef struct {
  int channels;         /* N: 1 .. 2^28                                        */
  int width;            /* K: a multiple of 16, 16 .. 16384                    */
  const int8_t *q;      /* [N, K] row-major, 16-byte aligned                   */
  const float *scales;  /* [N]                                                 */
} moe_qdense_weights;

/* Workspace of moe_qdense_forward for n_rows rows (0: none needed, and for
 * arguments that the call refuses): room for the rows in 2 bytes a value, from
 * 9 rows on.  It depends on n_rows and the width alone.  A call that widens its
 * rows without a launch of their own, which depends on the device too, takes
 * the workspace all the same and leaves it as it was. */
size_t moe_qdense_workspace_bytes(const moe_qdense_weights *w, int n_rows);

/* Dense projection of 8-bit rows:
 *   y[t, n] = cap(x_scales[t] * scales[n] * sum_k x[t, k] q[n, k])
 *   cap(z) = softcap * tanh(z / softcap), or z for softcap <= 0 (finite)
 *   x         int8 [n_rows, K], 16-byte aligned;  x_scales fp32 [n_rows]
 *   n_rows    1 .. MOE_QDENSE_MAX_ROWS
 *   y         nullable bf16 [n_rows, N];  y32 nullable fp32 [n_rows, N];
 *             not both null
 *   ws        moe_qdense_workspace_bytes(w, n_rows) bytes, 256-byte aligned
 *             (null where that is 0)
 * Outputs must not overlap an input or each other.  Up to 8 rows the sums are
 * exact 32-bit integers; more rows are summed in fp32, exact while the partial
 * sums stay below 2^24 (always, for K up to 1024).  Calls that may run at the
 * same time need a workspace each. */
#define MOE_QDENSE_MAX_ROWS 65536
int moe_qdense_forward(moe_handle *h, const int8_t *x, const float *x_scales, int n_rows, const moe_qdense_weights *w,
                       float softcap, void *y, float *y32, void *ws, size_t ws_bytes, moe_stream_t stream);

/* The rules of moe_logits_process (all device pointers; a part whose first
 * pointer is null is left out). */
typedef struct {
  /* Tokens of each row so far, prompt first: history [n_rows, history_stride],
   * of which the first history_len[t] count (clamped to 0 .. history_stride;
   * history_stride 1 .. 2^24), the first prompt_len[t] of those (null: 0) the
   * prompt.  The penalties are per row, null: none. */
  const int32_t *history;
  const int32_t *history_len;
  const int32_t *prompt_len;
  int history_stride;
  const float *repetition;  /* of tokens anywhere in the history: l > 0 ? l / p : l * p  */
  const float *presence;    /* subtracted once from tokens after the prompt              */
  const float *frequency;   /* subtracted per occurrence after the prompt                */
  /* Added to single logits: [n_rows, bias_stride], the first bias_len[t] of a
   * row (clamped to 0 .. bias_stride; bias_stride 1 .. 2^24).  Of several
   * entries for one token the last counts. */
  const int32_t *bias_ids;
  const float *bias_values;
  const int32_t *bias_len;
  int bias_stride;
  /* Allowed tokens: bit v % 32 of word v / 32, [n_rows, mask_stride] words;
   * mask_stride 0: one mask for every row. */
  const uint32_t *mask;
  int mask_stride;
} moe_logit_rules;

/* Penalties, biases and a mask on logits, and the greedy token of the result.
 * In this order, each rounded to fp32: repetition; frequency times the count;
 * presence; bias; -inf where the mask does not allow the token.
 *   logits   fp32 [n_rows, logits_stride], the first vocab (1 .. 2^28) of a
 *            row; n_rows 1 .. MOE_LOGITS_MAX_ROWS; logits_stride >= vocab
 *   out      nullable fp32 [n_rows, out_stride]; may be logits itself (with
 *            the same stride), else must not overlap it; columns from vocab on are left as they are
 *   tokens   nullable int32 [n_rows]: argmax, ties to the lower id; -1 where
 *            no logit is above -inf;  out and tokens not both null
 * A NaN or +inf that the mask does not remove is passed on, skipped by the
 * argmax and records MOE_ERR_NONFINITE; ids outside the vocabulary are
 * skipped and record MOE_ERR_BAD_EXPERT_ID.  One launch.  The greedy state
 * lives in the handle (cleared by the launch that used it), so calls on one
 * handle must not overlap on the GPU. */
#define MOE_LOGITS_MAX_ROWS 4096
int moe_logits_process(moe_handle *h, const float *logits, size_t logits_stride, int n_rows, int vocab,
                       const moe_logit_rules *rules, float *out, size_t out_stride, int32_t *tokens,
                       moe_stream_t stream);

/* ---- Attention of a decode loop, over a paged cache of keys and values, and
 * the choice of the next token.  As above: a launch each, nothing allocated,
 * capturable in a CUDA graph, the handle's device the current one. */

/* A cache of keys and values.  The rows of a sequence's positions lie in pages
 * of page_rows positions: position p of sequence s is row p % page_rows of page
 * table[s * table_stride + p / page_rows].  Sequences may share pages, and
 * a table may name a page again (the oldest page of a sliding window taken up
 * anew), as long as no call reads a position whose row holds another's values.
 * A page holds, per head, page_rows rows of head_dim values: bf16, or where
 * k_scales and v_scales are given 8-bit codes with a scale per row (value =
 * code * scale). */
typedef struct {
  int n_pages;           /* 1 ..; n_pages * kv_heads * page_rows up to 2^31 - 256    */
  int kv_heads;          /* 1 .. 128                                                 */
  int page_rows;         /* 16, 32, 64, 128 or 256                                   */
  int head_dim;          /* a multiple of 16, 16 .. 256                              */
  void *k, *v;           /* [n_pages, kv_heads, page_rows, head_dim], 16-byte aligned */
  float *k_scales, *v_scales; /* both null (bf16), or [n_pages, kv_heads, page_rows], 16-byte aligned */
  const int32_t *table;  /* [n_seqs, table_stride]                                   */
  int n_seqs;            /* 1 .. MOE_KV_MAX_SEQS                                     */
  int table_stride;      /* 1 ..; table_stride * page_rows up to 2^30                */
} moe_kv_cache;
#define MOE_KV_MAX_SEQS 4096
#define MOE_KV_MAX_ROWS (1 << 20)

/* Rotary positions, and new rows into the cache.  Row t is position row_pos[t]
 * of sequence row_seq[t] (row_seq null: of sequence t).  With rot_dims = r > 0
 * the first r dimensions of every head of q and k turn by the position's
 * angles, a pair j, j + r/2 by a = row_pos[t] * inv_freq[j]:
 *   x_j cos a - x_{j+r/2} sin a,  x_{j+r/2} cos a + x_j sin a     (j < r/2)
 * (the angle is reduced in 64 bits: positions may be far).  Then
 *   q_out[t]  bf16 of q's turned row
 *   cache     bf16 of k's turned and v's row; in 8 bits, with m the largest
 *             magnitude of a head's row: rint(127 x / m) (zero for m = 0) and
 *             the scale m / 127, of k's turned row before any rounding to bf16
 *   q         nullable bf16 [n_rows, q_heads, head_dim]; q_out only with q, may
 *             be q itself (with the same stride)
 *   k, v      bf16 [n_rows, kv_heads, head_dim]
 *   strides   of q, k, v, q_out: values from row to row, multiples of 8 (the
 *             parts of one projection's output can be given as they lie)
 *   row_pos   int32 [n_rows]; row_seq nullable int32 [n_rows]
 *   inv_freq  fp32 [rot_dims / 2] (null: rot_dims 0)
 *   rot_dims  0, or a multiple of 16 up to head_dim
 * n_rows 1 .. MOE_KV_MAX_ROWS, q_heads 1 .. 1024; all bf16 data 16-byte
 * aligned.  A row of a negative position is left out: nothing is written for
 * it.  A row of a sequence, a position or a page that is not there is not
 * written to the cache (its q_out is) and records MOE_ERR_BAD_EXPERT_ID.  In 8
 * bits a head's row with a NaN or an infinity gets codes 0 and the scale NaN
 * and records MOE_ERR_NONFINITE.  No two rows of a call may go to one place of
 * the cache (its row would hold values of both).  Outputs must not overlap
 * inputs otherwise. */
int moe_kv_append(moe_handle *h, const void *q, size_t q_stride, int q_heads, const void *k, size_t k_stride,
                  const void *v, size_t v_stride, int n_rows, const int32_t *row_seq, const int32_t *row_pos,
                  const moe_kv_cache *cache, const float *inv_freq, int rot_dims, void *q_out, size_t q_out_stride,
                  moe_stream_t stream);

/* Rows of the cache as bf16 (8-bit rows: the fp32 product code * scale,
 * rounded): row t is position row_pos[t] of sequence row_seq[t] (null: of sequence
 * t), as above; positions may be named again.
 *   k_out, v_out  nullable bf16 [n_rows, kv_heads, head_dim] with strides of
 *                 multiples of 8 values from row to row, 16-byte aligned; not
 *                 both null
 * Outputs must not overlap the cache or each other.  A row of a negative
 * position is left as it was; one that is not there is all zeros and records
 * MOE_ERR_BAD_EXPERT_ID. */
int moe_kv_read(moe_handle *h, const moe_kv_cache *cache, const int32_t *row_seq, const int32_t *row_pos, int n_rows,
                void *k_out, size_t k_stride, void *v_out, size_t v_stride, moe_stream_t stream);

/* Workspace of moe_kv_attend: the same for any lengths (0 for arguments that
 * the call refuses). */
size_t moe_kv_attend_workspace_bytes(const moe_kv_cache *cache, int q_heads);

/* Attention of one new token per sequence (whose own key and value are in the
 * cache already).  Query head i of sequence s looks at the keys of head
 * i / (q_heads / kv_heads) at the positions p with
 *   max(0, lengths[s] - window) <= p < lengths[s]       (window 0: from 0 on)
 *   z_p = cap(scale * sum_d q[d] k_p[d]),  cap(z) = softcap * tanh(z / softcap),
 *         or z for softcap 0
 *   out = sum_p e^(z_p - L) v_p,  L = log sum_p e^(z_p)
 * and lengths outside 0 .. table_stride * page_rows count as the nearer end.
 *   q        bf16 [n_seqs, q_heads, head_dim], rows q_stride values apart;
 *   out      the same with out_stride (strides multiples of 8, 16-byte aligned)
 *   lse      nullable fp32 [n_seqs, q_heads]: L
 *   lengths  int32 [n_seqs]
 *   q_heads  a multiple of kv_heads, up to 64 times as many; n_seqs *
 *            table_stride * page_rows / 16 * kv_heads (for each 16 query heads
 *            of a key head, or part of them) below 2^31
 *   scale    finite;  softcap 0 or above, finite;  window 0 or above
 *   ws       moe_kv_attend_workspace_bytes(cache, q_heads) bytes, 256-byte aligned
 * Outputs must not overlap inputs (a query is read by several blocks).  A
 * sequence without a position to look at gets zeros and L = -inf.  Positions
 * of a page that is not there are left out, and one among those looked at
 * records MOE_ERR_BAD_EXPERT_ID; what the cache holds from the length on, or
 * ahead of the window, does not matter.  Sums and statistics are fp32; a weight
 * e^(z - max) is rounded once, to bf16 with a bf16 cache and to fp16 (with its
 * value row's scale) with an 8-bit one, where a weight and scale below 2^-28 of
 * the largest keep fewer bits (2^-39 of the largest scale).  Finished-block
 * counters live in the handle, so calls on one handle must not overlap on the
 * GPU; calls that may run at the same time need a handle and a workspace each. */
int moe_kv_attend(moe_handle *h, const void *q, size_t q_stride, const moe_kv_cache *cache, const int32_t *lengths,
                  int q_heads, float scale, float softcap, int window, void *out, size_t out_stride, float *lse,
                  void *ws, size_t ws_bytes, moe_stream_t stream);

/* The filters of moe_sample, a value per row (device pointers; null: the value
 * in brackets for every row). */
typedef struct {
  const float *uniform;      /* the random numbers, 0 <= u < 1 (never null)              */
  const float *temperature;  /* [1]; not above 0: the greedy token                       */
  const int32_t *top_k;      /* [0]; not above 0: off                                    */
  const float *top_p;        /* [1]; from 1 on: off                                      */
  const float *min_p;        /* [0]; not above 0: off; 1 at most                         */
} moe_sample_rules;

/* A token drawn from each row's logits.  With M the largest logit and the
 * tokens in the order of their logits, the lower id first of equal ones, those
 * that remain are
 *   of all tokens with a logit above -inf those with (l - M) / temperature >= ln(min_p),
 *   of these the first top_k,
 *   of these the fewest first ones whose weights w = e^((l - M) / temperature)
 *   sum to top_p of the sum or more, one at least.
 * The token is the first by id whose running sum of the remaining weights is
 * above u times their whole sum.
 *   logits    fp32 [n_rows, logits_stride], the first vocab (1 .. 2^28) of a
 *             row; n_rows 1 .. MOE_LOGITS_MAX_ROWS; logits_stride >= vocab
 *   tokens    int32 [n_rows]: the token; -1 where no logit is above -inf
 *   logprobs  nullable fp32 [n_rows]: the log of the token's share of the
 *             remaining weights (0 for a greedy row; -inf with token -1)
 * u counts as 0 below 0 or NaN, and as the last remaining token from 1 on.  A
 * NaN filter is off, a NaN temperature is greedy.  A NaN or +inf among the
 * logits counts as -inf and records MOE_ERR_NONFINITE.  A row whose logits did
 * not land in time gets token -1 and records MOE_ERR_TIMEOUT.  The sums are exact
 * over weights within 2^-21 of their values, rounded to whole units of
 * 2^-(31 + the leading zeros of vocab's 32 bits) of the largest (2^-44 for
 * 262144 tokens, 2^-34 for the most), the same whatever their order and
 * whatever else is in the call.  Nothing but the error stays in the handle:
 * calls may overlap. */
int moe_sample(moe_handle *h, const float *logits, size_t logits_stride, int n_rows, int vocab,
               const moe_sample_rules *rules, int32_t *tokens, float *logprobs, moe_stream_t stream);

/* Launch tracing (diagnostics).  With a non-null device buffer of
 * 4 * n_launches u64, each subsequent kernel launch by this handle takes the
 * next 4 slots (wrapping) and records %globaltimer values, combined with
 * atomicMax so a zeroed buffer is the reset state:
 *   [0] bitwise NOT of the first block's entry time
 *   [1] bitwise NOT of the time that block passed its dependency wait
 *   [2] latest time a block had its weights in shared memory (0: n/a)
 *   [3] latest block exit time (the router: its last block's exit).
 * A call launches 3 (T == 1) or 4 kernels; slot groups are reserved as
 * router 1, gate/up 1, down (+ combine) 2, sort 1; moe_norm_quant,
 * moe_logits_process, moe_kv_append, moe_kv_read, moe_kv_attend and moe_sample
 * 1, moe_qdense_forward 1, or 2 where a launch of its own
 * widens the rows.  Buffer owned by the caller; NULL turns tracing off.
 * Tracing adds a few atomics per block. */
int moe_set_trace(moe_handle *h, unsigned long long *buffer, int n_launches);

/* Self-test of the device-side bounded waits (failure detection without a
 * GPU fault): launches one thread that waits on a barrier nothing ever
 * completes; after limit_ns (1 .. 2e9 ns) of device time it gives up and
 * records MOE_ERR_TIMEOUT in the error word, which moe_get_error then
 * reports.  Every wait in the kernels above uses the same bounded wait. */
int moe_selftest_wait_timeout(moe_handle *h, unsigned long long limit_ns, moe_stream_t stream);

/* Self-test of a grid barrier that never completes (failure detection
 * without a GPU fault): arms the handle's next fused single-token launch so
 * that block `block` (0 <= block < SM count) withholds its arrival at the
 * barrier between the gate/up and down phases, and every bounded wait of
 * that launch gives up after limit_ns (1 .. 2e9 ns) of device time.  The
 * blocks then record MOE_ERR_TIMEOUT and leave (the launch's outputs are not
 * valid); moe_get_error reports it and restores the barrier state, so the
 * next call is correct again.  Host-side only: launches nothing itself. */
int moe_selftest_skip_arrival(moe_handle *h, int block, unsigned long long limit_ns);

/* Waits for all work on the device, then returns (in *status) the first
 * device-side error recorded since the last call (MOE_OK if none) and
 * clears it.  After a timeout it also resets the handle's grid-barrier
 * counters, tickets and logit mailboxes (a launch whose blocks did not all
 * arrive leaves its counter out of step).  The return value reports
 * failures of the call itself. */
int moe_get_error(moe_handle *h, int *status);

#ifdef __cplusplus
}
#endif
#endif /* MOE_AFFINE_H */

/*
 * moe_ep.h -- C ABI of the MI355X (gfx950) rank-major MoE expert-parallel
 * dispatch/combine library (libmoe_ep.so).
 *
 * One process holds a whole expert-parallel (EP) group of ep_size logical
 * ranks.  Each rank's receive region and combine input region is a partition
 * of one caller-owned device workspace, so dispatch and combine are on-device
 * scatter / gather-reduce kernels on one GPU.  Every per-rank argument of the
 * FlashInfer API becomes an array indexed by rank.
 *
 * Sources of the contract (FlashInfer API pages for flashinfer.moe_ep):
 *   MoEEpCommunication       class description, is_platform_supported(),
 *                            dispatch(), combine(), get_combine_input_buffer(),
 *                            destroy()
 *   NVLinkOneSidedAlltoAll   class description (rank-major placement and
 *                            invalid rows), active_rank_mask(), dispatch()
 *                            (mask and weights rules), combine() (mask rule),
 *                            get_combine_input_buffer()
 *   CakeAlltoAll             class description (rows beyond a source's count)
 *
 * Conventions for every entry point:
 *   - Pointers named "device" point to GPU memory of the current HIP device;
 *     all other pointers are host memory and are read only during the call.
 *   - Validation happens on the host before anything is enqueued.  On any
 *     error no device work is queued and the handle's state is unchanged.
 *   - Device work is enqueued on `stream` (a hipStream_t; NULL = the null
 *     stream of the current device) and is asynchronous: inputs must stay
 *     valid, and outputs must not be read, until the stream has passed the
 *     call.  No entry point synchronizes the device or allocates device
 *     memory.  A stream on another device than the workspace's makes
 *     dispatch and combine fail with MOE_EP_ERR_INVALID_ARG.
 *   - A handle serves one in-flight dispatch/combine pair and is not
 *     thread-safe.
 *   - Every entry point returns a moe_ep_status (0 = success) unless stated.
 *     moe_ep_last_error() describes the most recent failure of this thread.
 */
#ifndef MOE_EP_H
#define MOE_EP_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Symbols of this header are the library's only exports. */
#define MOE_EP_API __attribute__((visibility("default")))

/* A uint64 bitmask names the active ranks, so a group has at most 64 ranks
 * (NVLinkOneSidedAlltoAll, active_rank_mask()). */
#define MOE_EP_MAX_RANKS 64
/* active_rank_mask value meaning "no mask passed": every rank is active. */
#define MOE_EP_ALL_RANKS (~(uint64_t)0)

typedef enum moe_ep_status {
  MOE_EP_OK = 0,
  MOE_EP_ERR_INVALID_ARG = -1,  /* bad pointer, size, dtype, or weights/scales passed by some ranks only */
  MOE_EP_ERR_STATE = -2,        /* call out of the dispatch -> combine -> dispatch order */
  MOE_EP_ERR_CAPACITY = -3,     /* tokens_per_rank outside [largest local count, capacity] */
  MOE_EP_ERR_MASK = -4,         /* mask without enable_rank_mask, bits >= ep_size, or combine mask != dispatch mask */
  MOE_EP_ERR_ALIGN = -5,        /* an int32/float/workspace pointer not aligned to its element */
  MOE_EP_ERR_HIP = -6,          /* a HIP runtime call failed (launch or device query) */
  MOE_EP_ERR_UNSUPPORTED = -7   /* no virtual memory management on the device, or a checkpoint
                                   call on a handle whose workspace the caller owns */
} moe_ep_status;

/* Order in which dispatch writes the receive rows (moe_ep_params.dispatch_order).
 * Both write the same bytes; they differ only in speed:
 *  SOURCE_ROW:  a workgroup reads one token row once and writes it to every
 *               destination in turn (best for large groups and fan-out).
 *  DESTINATION: a workgroup writes one (destination, row) pair; rows are
 *               pinned to XCDs so the other destinations' re-reads of a row
 *               hit that XCD's L2, and each destination's region is written
 *               as one sequential sweep (best for groups of a few ranks
 *               whose rows are mostly real tokens).
 *  AUTO:        DESTINATION when ep_size <= 16, ep_size^2 * tokens_per_rank
 *               <= 16384 and the ep_size * tokens_per_rank source rows do
 *               not fill the chip on their own (MI355X runs 256 CUs x 32
 *               waves at once); also when ep_size <= 8 and at least 80% of
 *               the ep_size * tokens_per_rank rows are real tokens (host
 *               counts only: a step with device-resident counts uses the
 *               first rule); else SOURCE_ROW.
 * An explicit DESTINATION request whose grid would pass 2^31 - 1 workgroups
 * makes moe_ep_dispatch fail with MOE_EP_ERR_INVALID_ARG (nothing launched);
 * AUTO then takes SOURCE_ROW instead. */
typedef enum moe_ep_dispatch_order {
  MOE_EP_ORDER_AUTO = 0,
  MOE_EP_ORDER_SOURCE_ROW = 1,
  MOE_EP_ORDER_DESTINATION = 2
} moe_ep_dispatch_order;

/* Element type of combine's input and output rows (both use the same one;
 * MoEEpCommunication, get_combine_input_buffer() takes any torch dtype).
 * Combine widens every element exactly to float32, adds in float32, and
 * rounds the sum once to the type, to nearest even. */
typedef enum moe_ep_dtype {
  MOE_EP_F32 = 0,
  MOE_EP_BF16 = 1,
  MOE_EP_F16 = 2                  /* IEEE binary16 */
} moe_ep_dtype;

/* Static sizes of one EP group (the pages' MoEEpCommParams plus the
 * enable_rank_mask switch of the backend config). */
typedef struct moe_ep_params {
  int32_t ep_size;                /* ranks in the group, 1..64 */
  int32_t num_experts;            /* global experts, a multiple of ep_size; rank d owns
                                     experts [d*E/ep, (d+1)*E/ep) (contiguous blocks) */
  int32_t top_k;                  /* experts per token, >= 1 */
  int32_t max_tokens_per_rank;    /* capacity: the largest local_num_tokens of any rank */
  int32_t hidden_size;            /* elements of a combine row */
  int32_t combine_max_elem_bytes; /* element size the combine input buffer is sized for: 2 (bf16,
                                     f16) or 4 (also f32) */
  int64_t hidden_row_bytes;       /* bytes of one dispatched hidden_states row (opaque) */
  int64_t scale_row_bytes;        /* bytes of one hidden_states_scale row; 0 = no scales */
  int32_t invalid_expert_id;      /* written into every top_k slot of an invalid receive row */
  int32_t enable_rank_mask;       /* nonzero: dispatch/combine accept an active_rank_mask */
  int64_t eplb_stats_bytes;       /* bytes of one rank's expert-load statistics row, gathered
                                     by dispatch (MoEEpCommunication, dispatch(),
                                     eplb_local_stats); 0 = not supported */
  int32_t dispatch_order;         /* moe_ep_dispatch_order; 0 = AUTO */
} moe_ep_params;

/* Inputs of one dispatch, per SOURCE rank s < ep_size
 * (MoEEpCommunication, dispatch()).  Entries at s >= ep_size are ignored. */
typedef struct moe_ep_dispatch_args {
  const void*    hidden[MOE_EP_MAX_RANKS];        /* device [n_s, hidden_row_bytes], rows contiguous */
  const void*    hidden_scale[MOE_EP_MAX_RANKS];  /* device [n_s, scale_row_bytes] or NULL */
  const int32_t* topk_ids[MOE_EP_MAX_RANKS];      /* device [n_s, top_k] global expert ids */
  const float*   topk_weights[MOE_EP_MAX_RANKS];  /* device [n_s, top_k] or NULL */
  int32_t        local_num_tokens[MOE_EP_MAX_RANKS]; /* n_s, 0..capacity */
  uint64_t       weights_present;  /* bit s: rank s passed topk_weights (an empty [0, top_k]
                                      tensor counts).  Must be none or all ranks. */
  uint64_t       scales_present;   /* bit s: rank s passed hidden_states_scale.  None or all. */
  int32_t        runtime_max_tokens_per_rank; /* < 0 = None = capacity; else in [max n_s, capacity] */
  uint64_t       active_rank_mask; /* MOE_EP_ALL_RANKS = no mask; else needs enable_rank_mask
                                      and only bits < ep_size */
  const void*    eplb_local_stats[MOE_EP_MAX_RANKS]; /* device [eplb_stats_bytes] per rank, or NULL */
  uint64_t       eplb_present;     /* bit s: rank s passed eplb_local_stats.  None or all; needs
                                      eplb_stats_bytes > 0 */
  const int32_t* local_num_tokens_device; /* optional device int32 [ep_size]: the token counts,
                                      read by the kernels when they run (so a captured graph
                                      replays ragged steps).  When set, local_num_tokens is
                                      ignored, each count is clamped to [0, tokens_per_rank],
                                      every rank's hidden / ids / weights / scale buffers must
                                      hold tokens_per_rank rows, and so must every combine
                                      output buffer.  NULL = use local_num_tokens. */
} moe_ep_dispatch_args;

/* What destination rank d received: views into its workspace partition,
 * valid until the next moe_ep_dispatch on the handle. */
typedef struct moe_ep_dispatch_result {
  void*    hidden;          /* device [num_rows, hidden_row_bytes] */
  void*    hidden_scale;    /* device [num_rows, scale_row_bytes], NULL when no scales passed */
  int32_t* topk_ids;        /* device [num_rows, top_k] */
  float*   topk_weights;    /* device [num_rows, top_k], NULL when no weights passed */
  int32_t  tokens_per_rank; /* tpr of this step */
  int32_t  num_rows;        /* ep_size * tokens_per_rank */
  void*    eplb_global_stats; /* device [ep_size, eplb_stats_bytes]: row s holds rank s's
                                 eplb_local_stats; NULL when none were passed */
  int32_t  dispatch_order;  /* order the kernel ran in: MOE_EP_ORDER_SOURCE_ROW or
                               MOE_EP_ORDER_DESTINATION (AUTO resolved), same for every rank */
} moe_ep_dispatch_result;

/* Inputs of one combine (MoEEpCommunication, combine()). */
typedef struct moe_ep_combine_args {
  const void* expert_output[MOE_EP_MAX_RANKS]; /* per rank d: device [ep*tpr, hidden_size] (the same
                                                  memory as [ep, tpr, hidden_size]); NULL = rank d's
                                                  combine input buffer */
  void*       output[MOE_EP_MAX_RANKS];        /* per source rank s: device [n_s, hidden_size] */
  int32_t     dtype;                           /* moe_ep_dtype of expert_output and output */
  uint64_t    active_rank_mask;                /* must equal the dispatch's mask */
} moe_ep_combine_args;

typedef struct moe_ep_handle_s* moe_ep_handle;

/* 1 when the current HIP device is a gfx950 (MI355X-class) GPU, else 0.
 * Needs no handle and does no device work
 * (MoEEpCommunication, is_platform_supported()). */
MOE_EP_API int moe_ep_is_platform_supported(void);

/* Bytes of device workspace a group with these params needs (receive
 * regions, combine input regions, and the per-token destination masks and
 * records that dispatch leaves for combine, for capacity-sized steps).
 * *out_bytes is set on success. */
MOE_EP_API int moe_ep_workspace_bytes(const moe_ep_params* params, size_t* out_bytes);

/* Creates a handle over a caller-owned device workspace of at least
 * moe_ep_workspace_bytes() bytes, aligned to 256 bytes.  The workspace is
 * borrowed until moe_ep_destroy and needs no initialisation.  Host-only: no
 * device work (it asks HIP which device holds the workspace, so dispatch
 * and combine can refuse a stream on another device). */
MOE_EP_API int moe_ep_create(const moe_ep_params* params, void* workspace, size_t workspace_bytes,
                  moe_ep_handle* out_handle);

/* Sends every token to the ranks that own its selected experts
 * (MoEEpCommunication, dispatch()) with rank-major placement
 * (NVLinkOneSidedAlltoAll, class description): on destination d, row
 * s*tpr + t holds token t of source s -- its hidden row, scale row, topk_ids
 * and topk_weights, verbatim -- when d owns one of its experts and d is
 * active.  Every other row (token not routed to d, d masked off, or
 * t >= n_s) gets invalid_expert_id in all top_k slots and weight 0.0; its
 * hidden and scale bytes are left unspecified.  tpr is
 * runtime_max_tokens_per_rank, or the capacity when it is < 0.
 * When every rank passes eplb_local_stats, each rank's statistics row is
 * also gathered into row s of a [ep_size, eplb_stats_bytes] region on every
 * rank (MoEEpCommunication, dispatch(), eplb_local_stats), in the same launch.
 * Fills results[0 .. ep_size-1] (host array) with views into the workspace.
 * Needs the IDLE state; leaves the handle DISPATCHED.  One kernel launch. */
MOE_EP_API int moe_ep_dispatch(moe_ep_handle handle, const moe_ep_dispatch_args* args,
                    moe_ep_dispatch_result* results, void* stream);

/* Rank `rank`'s combine input buffer: device [ep_size*tpr, hidden_size] of
 * `dtype`, in its workspace partition, for the expert computation to write
 * into (MoEEpCommunication and NVLinkOneSidedAlltoAll,
 * get_combine_input_buffer()).  Valid only between dispatch and combine
 * (ERR_STATE otherwise); dtype's size must not exceed
 * combine_max_elem_bytes. */
MOE_EP_API int moe_ep_get_combine_input_buffer(moe_ep_handle handle, int32_t rank, int32_t dtype,
                                    void** out_ptr);

/* For every source rank s and token t < n_s: output[s][t] = sum, over the
 * ranks d that token was dispatched to in ascending d, of
 * expert_output[d][s*tpr + t], accumulated in float32 from +0.0 and rounded
 * once to dtype (bfloat16, float16: round to nearest even).  A token that reached no
 * rank gets zeros.  Rows of tokens not dispatched to d are never read, nor is
 * any row of a masked-off rank (MoEEpCommunication, combine();
 * NVLinkOneSidedAlltoAll, combine() mask rule).  Needs the DISPATCHED state;
 * leaves the handle IDLE.  One kernel launch.  After a host-count dispatch,
 * when the read ranks' expert_output rows and the non-empty outputs each lie
 * at one constant stride (the combine input buffers do; so do outputs sliced
 * from one [ep_size, n, hidden_size] allocation), the launch carries only
 * scalar arguments, which the HIP runtime enqueues ~0.6 us faster. */
MOE_EP_API int moe_ep_combine(moe_ep_handle handle, const moe_ep_combine_args* args, void* stream);

/* Releases the handle's host state; a workspace passed to moe_ep_create
 * stays the caller's, one made by moe_ep_create_vmm is unmapped and freed
 * (after waiting for the device).  NULL is a no-op.  Device work already
 * enqueued with the handle must have finished before a caller-owned
 * workspace is reused (MoEEpCommunication, destroy()). */
MOE_EP_API int moe_ep_destroy(moe_ep_handle handle);

/* Creates a handle whose workspace the library maps itself with HIP virtual
 * memory management on the current device: a reserved virtual address range
 * backed by one physical allocation.  Only such a handle can release its
 * physical memory for a process checkpoint while its addresses stay put
 * (NVLinkOneSidedAlltoAll and CakeAlltoAll, checkpoint_prepare() and
 * checkpoint_restore()).  ERR_UNSUPPORTED when the device lacks virtual
 * memory management; ERR_HIP when a mapping call fails (nothing is left
 * allocated). */
MOE_EP_API int moe_ep_create_vmm(const moe_ep_params* params, moe_ep_handle* out_handle);

/* Device address and size of the handle's workspace.  For a handle from
 * moe_ep_create_vmm the address is the same for the handle's whole life,
 * across checkpoints, but must not be touched while the memory is released. */
MOE_EP_API int moe_ep_workspace(moe_ep_handle handle, void** out_ptr, size_t* out_bytes);

/* Before a process checkpoint: waits for the device, then unmaps and
 * releases the workspace's physical memory, keeping its virtual addresses
 * reserved so that HIP graphs captured on the workspace replay once
 * moe_ep_checkpoint_restore has backed it again.  Only between rounds
 * (ERR_STATE after a dispatch without its combine).  A second call does
 * nothing.  Until the restore, dispatch, combine and
 * get_combine_input_buffer return ERR_STATE.  ERR_UNSUPPORTED for handles
 * from moe_ep_create.  If unmapping fails part-way the handle is unusable
 * (every later call but destroy returns ERR_STATE). */
MOE_EP_API int moe_ep_checkpoint_prepare(moe_ep_handle handle);

/* After the checkpoint: backs the reserved addresses with new physical
 * memory (contents undefined; the workspace needs no initialisation).  Does
 * nothing when the workspace is mapped.  If mapping fails part-way the
 * handle is unusable, as above. */
MOE_EP_API int moe_ep_checkpoint_restore(moe_ep_handle handle);

/* Receive rows (ep_size * tokens_per_rank) of the largest step
 * moe_ep_dispatch_noalloc takes: the size of the library's fixed record area
 * (24 bytes per row plus 256, 1.5 MiB, held on each GPU the library runs on
 * until the process ends). */
#define MOE_EP_NOALLOC_MAX_ROWS 65536

/* For callers that cannot allocate device memory (code under HIP graph
 * capture, tight serving loops, harnesses that forbid hipMalloc): the same
 * dispatch as moe_ep_dispatch -- same arguments, results, state change and
 * errors -- except that the per-token routing records dispatch leaves for
 * combine (destination masks, token positions, token counts) go to a fixed
 * device array inside the library instead of the workspace.  The handle's
 * next moe_ep_combine reads them from there.  Nothing is allocated or freed:
 * the array's device address is looked up once per device (at moe_ep_create
 * when the workspace's device is known, else at the first call on a device).
 * ERR_CAPACITY when ep_size * tokens_per_rank exceeds MOE_EP_NOALLOC_MAX_ROWS
 * (nothing enqueued); ERR_HIP when the lookup fails.
 * Every handle on a GPU shares that GPU's one array, and it keeps only the
 * last noalloc dispatch's records: a noalloc dispatch must not run between
 * another handle's noalloc dispatch and that handle's combine on the same
 * GPU (in stream order), and calls that overlap on one GPU, from several
 * streams or threads, race. */
MOE_EP_API int moe_ep_dispatch_noalloc(moe_ep_handle handle, const moe_ep_dispatch_args* args,
                                       moe_ep_dispatch_result* results, void* stream);

/* Bitmask with bit r set for each of the n listed ranks, all in [0, 64)
 * (NVLinkOneSidedAlltoAll, active_rank_mask()).  ERR_MASK for a rank out of
 * range. */
MOE_EP_API int moe_ep_active_rank_mask(const int32_t* ranks, int32_t n, uint64_t* out_mask);

/* ------------------------------------------------------------------------
 * Expert-side operators: what a decode step computes around dispatch and
 * combine.  A router's logits become the topk_ids and topk_weights that
 * dispatch takes (moe_ep_route); the experts' matrices are applied to the
 * rows of their tokens (moe_ep_expert_linear, one matrix; moe_ep_layer, the
 * whole gated feed-forward summed over a token's experts).  They need no
 * handle.  Activations and dense weights are MOE_EP_BF16 or MOE_EP_F16,
 * sums float32, and a result is rounded once.  Results do not depend on
 * timing: the same inputs give the same bits.
 *
 * The stream must belong to the current HIP device (ERR_INVALID_ARG
 * otherwise), and so must every device pointer.  Pointers to 16-bit
 * elements, to int32 and to float must be aligned to their element
 * (ERR_ALIGN otherwise); 4-bit weights and their scales to 16 bytes.  Row
 * strides are in elements.
 * ------------------------------------------------------------------------ */

/* Most experts of a router, a linear product or a layer. */
#define MOE_EP_MAX_EXPERTS 1024
/* Most experts per token of a router or a layer. */
#define MOE_EP_MAX_TOPK 64
/* Most groups of a router. */
#define MOE_EP_MAX_GROUPS 64

typedef enum moe_ep_score {
  MOE_EP_SCORE_SOFTMAX = 0,       /* softmax over the experts */
  MOE_EP_SCORE_SIGMOID = 1        /* each expert's own sigmoid */
} moe_ep_score;

/* How a token's logits l[0 .. num_experts) choose its top_k experts.
 *
 *   score   s = softmax(l) or sigmoid(l)
 *   choice  c = s + bias with a bias, else s (without bias and groups c = l,
 *           which has the same order and no ties from rounding)
 *   groups  with num_groups > 1 the experts form num_groups equal blocks; a
 *           group counts the sum of its group_top best open choices, and
 *           only the top_groups best groups stay open
 *   ids     the top_k best open choices, best first
 *   weights s[ids], divided by their sum when renormalize is set, times scale
 *
 * Equal choices and equal groups go to the lower index.  Choices are
 * compared in float64.  An expert whose logit or bias is -inf or NaN is
 * closed: it has no share in the softmax and is never chosen.  A logit of
 * +inf counts as the largest float32.  Slots that no open expert is left
 * for get invalid_expert_id and weight 0; so does every weight of a token
 * whose chosen scores sum to 0 under renormalize. */
typedef struct moe_ep_router {
  int32_t num_experts;            /* 1..MOE_EP_MAX_EXPERTS */
  int32_t top_k;                  /* 1..min(num_experts, MOE_EP_MAX_TOPK) */
  int32_t score;                  /* moe_ep_score */
  int32_t num_groups;             /* 1..MOE_EP_MAX_GROUPS, divides num_experts; 1 = no groups */
  int32_t top_groups;             /* 1..num_groups, holding at least top_k experts */
  int32_t group_top;              /* 1 or 2 */
  int32_t renormalize;
  int32_t invalid_expert_id;
  float scale;
  const float* bias;              /* device [num_experts], or NULL */
} moe_ep_router;

/* Chooses the experts of num_tokens tokens: logits device [num_tokens,
 * num_experts] of logits_dtype (any moe_ep_dtype), rows logits_stride apart;
 * topk_ids device int32 and topk_weights device float, both [num_tokens,
 * top_k], as moe_ep_dispatch takes them.  One kernel launch per 2^24 tokens. */
MOE_EP_API int moe_ep_route(const moe_ep_router* router, const void* logits, int32_t logits_dtype,
                            int64_t logits_stride, int32_t num_tokens, int32_t* topk_ids,
                            float* topk_weights, void* stream);

/* The matrices [N, K] of a set of experts.
 *
 * group_size 0: dense, data is [experts, N, K] of the activations' type and
 * scales is ignored.
 *
 * group_size g = 32, 64 or 128: 4-bit integers q in 0..15 with
 *   W[n][k] = (q - 8) * scale[n][k / g]
 * in tiles of 16 rows by 128 columns, 1024 bytes each:
 *   data    uint8 [experts, ceil(N/16), ceil(K/128), 1024]
 *   scales  of the activations' type [experts, ceil(N/16),
 *           ceil(K/128) * 128 / g, 16], a tile's 16 rows side by side
 * In a tile, row r's columns c = 32 j + 8 i + e (j, i < 4, e < 8) are in the
 * 4 bytes at (16 i + r) * 16 + 4 j: byte e of them holds column e < 4 in its
 * low half and column e + 4 in its high half.  Rows past N and columns past
 * K are padding of any value.  A token whose activations hold an infinity
 * gets NaN from 4-bit weights, and so may one whose activations' sums times
 * 15 are beyond float32 (q x and 8 x are summed apart). */
typedef struct moe_ep_weight {
  const void* data;
  const void* scales;
  int32_t group_size;
} moe_ep_weight;

typedef struct moe_ep_linear_args {
  const void* x;                  /* device [num_rows, in_features] of dtype */
  int64_t x_stride;               /* >= 0; 0 repeats one row */
  const int32_t* expert_ids;      /* device [num_rows], or NULL: every row is expert 0's */
  void* out;                      /* device [num_rows, out_features] of out_dtype */
  int64_t out_stride;             /* >= out_features */
  moe_ep_weight weight;           /* N = out_features, K = in_features */
  int32_t dtype;                  /* MOE_EP_BF16 or MOE_EP_F16 */
  int32_t out_dtype;              /* dtype, or MOE_EP_F32 */
  int32_t num_rows;
  int32_t num_experts;            /* 1..MOE_EP_MAX_EXPERTS */
  int32_t expert_offset;          /* expert_ids of the first expert, >= 0 */
  int32_t in_features;            /* 8..2^22 */
  int32_t out_features;           /* 1..2^22 */
} moe_ep_linear_args;

/* out[r] = W[expert_ids[r] - expert_offset] x[r].  Rows whose id is outside
 * [expert_offset, expert_offset + num_experts) get zeros.  Made for the few
 * rows of a decode step: a used expert's weights are gone through once for
 * every 4 (4-bit) or 8 (dense) of its rows, or for every 48 where it has many,
 * after the first time from a cache where they fit.  One kernel launch per
 * 2048 rows.  x and out, each from its first element to its last, must not
 * overlap. */
MOE_EP_API int moe_ep_expert_linear(const moe_ep_linear_args* args, void* stream);

typedef struct moe_ep_layer_args {
  const void* hidden;             /* device [num_tokens, hidden_size] of dtype */
  int64_t hidden_stride;          /* >= 0; 0 repeats one row */
  const int32_t* topk_ids;        /* device [num_tokens, top_k]; NULL with router */
  const float* topk_weights;      /* device [num_tokens, top_k], or NULL: all 1 */
  const moe_ep_router* router;    /* host; chooses ids and weights from router_logits, or NULL */
  const void* router_logits;      /* device [num_tokens, router->num_experts], with router */
  int64_t logits_stride;
  void* out;                      /* device [num_tokens, hidden_size] of out_dtype */
  int64_t out_stride;             /* >= hidden_size */
  moe_ep_weight gate_up;          /* N = 2 * intermediate_size (gate rows, then up rows), K = hidden_size */
  moe_ep_weight down;             /* N = hidden_size, K = intermediate_size */
  void* workspace;                /* device, moe_ep_layer_workspace_bytes() bytes, 256-byte aligned */
  size_t workspace_bytes;
  int32_t dtype;                  /* MOE_EP_BF16 or MOE_EP_F16 */
  int32_t out_dtype;              /* dtype, or MOE_EP_F32 */
  int32_t logits_dtype;           /* any moe_ep_dtype */
  int32_t num_tokens;
  int32_t top_k;                  /* 1..MOE_EP_MAX_TOPK; the router's with router */
  int32_t num_experts;            /* experts whose weights are here, 1..MOE_EP_MAX_EXPERTS */
  int32_t expert_offset;          /* id of the first of them, >= 0 */
  int32_t hidden_size;            /* 8..2^22 */
  int32_t intermediate_size;      /* 8..2^22 */
} moe_ep_layer_args;

/* Bytes of device workspace moe_ep_layer needs for these sizes (the sizes,
 * gate_up.group_size and whether a router is set are read; pointers are not
 * followed).  What serves a number of tokens serves any smaller one.  It is
 * for a pass of up to 2048 tokens and counts every (token, slot) pair, its
 * expert here or not: 6 bytes for each column of intermediate_size, and with
 * many tokens to an expert 4 for each of hidden_size (1024 rows, top_k 8,
 * hidden 7168, intermediate 2048: 320 MiB). */
MOE_EP_API int moe_ep_layer_workspace_bytes(const moe_ep_layer_args* args, size_t* out_bytes);

/* The experts of a mixture-of-experts layer, whole:
 *   out[t] = sum_j topk_weights[t][j] * down_e( silu(gate_e hidden[t]) * (up_e hidden[t]) ),
 *   e = topk_ids[t][j] - expert_offset,
 * over the slots j whose e is in [0, num_experts); a token with none gets
 * zeros.  An expert named twice by a token counts with both weights.  With
 * all experts here this is a whole layer; with one rank's experts on the
 * rows dispatch left that rank it is the expert computation between
 * dispatch and combine, and out may be the rank's combine input buffer.
 *
 * Per 2048 tokens two kernel launches, or three for many tokens to an expert;
 * one more for the router's choice, which the first of the two makes itself
 * for at most 8 tokens, 64 slots and 256 experts.  out may be hidden itself
 * (same address, stride and type) but not overlap it otherwise, each taken
 * from its first element to its last.  The workspace holds nothing between
 * calls; calls that may overlap in time (other streams, graphs replayed side
 * by side) need one each.
 *
 * Between the products an activation is a float32 value, whole: what is
 * small or large beside float16's own range keeps its 24 bits.  An infinite
 * weight in down may give NaN where the formula has an infinity. */
MOE_EP_API int moe_ep_layer(const moe_ep_layer_args* args, void* stream);

/* ------------------------------------------------------------------------
 * Dense operators: what a block computes on all of its tokens beside the
 * routed experts.  The residual's addition and the norm that make the rows
 * dispatch takes, in 16 bits or in 8 bits with scales (moe_ep_rms_norm); the
 * first half of a shared expert's gated feed-forward and its gradients
 * (moe_ep_gated, moe_ep_gated_grad); a projection that the requests of a
 * batch share, with a low-rank adapter of each one's own
 * (moe_ep_adapter_linear).  They need no handle; streams, devices, strides
 * and alignment are as for the expert-side operators.  Sums are float32 or
 * wider, and results do not depend on timing.
 * ------------------------------------------------------------------------ */

/* out_dtype of moe_ep_rms_norm for 8-bit rows: OCP e4m3 (largest value 448). */
#define MOE_EP_E4M3 8

typedef struct moe_ep_norm_args {
  const void* x;                  /* device [num_rows, hidden_size] of dtype */
  int64_t x_stride;               /* >= 0; 0 repeats one row */
  const void* residual;           /* device [num_rows, hidden_size] of dtype, or NULL */
  int64_t residual_stride;        /* >= 0; 0 repeats one row */
  const void* weight;             /* device [hidden_size] of weight_dtype */
  void* out;                      /* device [num_rows, hidden_size] of out_dtype */
  int64_t out_stride;             /* >= hidden_size */
  float* scales;                  /* device [num_rows, groups], MOE_EP_E4M3 only */
  int64_t scales_stride;          /* >= groups */
  void* residual_out;             /* device [num_rows, hidden_size] of dtype, with residual only */
  int64_t residual_out_stride;    /* >= hidden_size */
  int32_t dtype;                  /* MOE_EP_BF16 or MOE_EP_F16 */
  int32_t weight_dtype;           /* dtype, or MOE_EP_F32 */
  int32_t out_dtype;              /* dtype, or MOE_EP_E4M3 */
  int32_t group_size;             /* MOE_EP_E4M3: columns of a scale, 32, 64 or 128; 0: a whole row */
  int32_t num_rows;
  int32_t hidden_size;            /* 8..2^22 */
  float eps;                      /* >= 0, finite */
} moe_ep_norm_args;

/* With s = x + residual (float32; x without a residual) and m = mean(s^2)
 * over a row:
 *   residual_out = s, rounded to dtype
 *   y            = s / sqrt(m + eps) * weight
 *   out          = y, rounded to dtype; or, in 8 bits,
 *   scales       = max|y| / 448 over a group of columns (the last may be short)
 *   out          = y / scale, rounded to e4m3, ties to even
 * y is made from the float32 sum, not from its rounding, and m is summed in
 * float64, so no square overflows.  The 8-bit values are the nearest ones to
 * 448 s w / max|s w| of the group, without the roundings of y and scale (groups
 * with a scale below 2^-64 apart).  A group whose scale is 0 holds zeros.  An
 * infinity or NaN in a row makes NaN of the row's y that it reaches by the
 * formula, and a group with NaN has the scale NaN and NaN throughout.
 *
 * groups is ceil(hidden_size / group_size), or 1: with group_size 128 the
 * rows and scales are what dispatch forwards as hidden and scale rows.  out
 * and residual_out may each be x or residual itself (same address, stride
 * and element size); otherwise no output may overlap an input or another
 * output, each taken from its first element to its last.  One kernel launch,
 * and one more for each 2^21 rows after the first. */
MOE_EP_API int moe_ep_rms_norm(const moe_ep_norm_args* args, void* stream);

typedef struct moe_ep_gated_args {
  const void* x;                  /* device [num_rows, hidden_size] of dtype */
  int64_t x_stride;               /* >= 0; 0 repeats one row */
  const void* gate_up;            /* device [2 * intermediate_size, hidden_size] of dtype: gate rows, then up rows */
  int64_t gate_up_stride;         /* >= hidden_size */
  void* out;                      /* device [num_rows, intermediate_size] of out_dtype */
  int64_t out_stride;             /* >= intermediate_size */
  float* pre;                     /* device [num_rows, 2 * intermediate_size], or NULL; see below */
  int32_t dtype;                  /* MOE_EP_BF16 or MOE_EP_F16 */
  int32_t out_dtype;              /* dtype, or MOE_EP_F32 */
  int32_t num_rows;
  int32_t hidden_size;            /* 8..2^22 */
  int32_t intermediate_size;      /* 8..2^22 */
} moe_ep_gated_args;

/* The first half of a gated feed-forward, whose weights lie as moe_ep_layer's
 * gate_up of one expert:
 *   g = gate_up[:I] x, u = gate_up[I:] x, out = silu(g) * u = g / (1 + exp(-g)) * u
 * in one kernel launch; g and u stay float32 until out is rounded.  Results of
 * 2^23 or more tiles of 128 x 128 (of gate and up) are refused, there and in
 * the two functions below.  With pre
 * they are kept for moe_ep_gated_grad as they are, g in the first I columns
 * and u in the others.  Outputs must not overlap inputs or one another, each
 * taken from its first element to its last. */
MOE_EP_API int moe_ep_gated(const moe_ep_gated_args* args, void* stream);

typedef struct moe_ep_gated_grad_args {
  const void* dout;               /* device [num_rows, intermediate_size] of dout_dtype */
  int64_t dout_stride;            /* >= 0; 0 repeats one row */
  const void* x;                  /* as moe_ep_gated's */
  int64_t x_stride;
  const void* gate_up;
  int64_t gate_up_stride;
  const float* pre;               /* what moe_ep_gated kept */
  void* dx;                       /* device [num_rows, hidden_size] of dtype, or NULL */
  int64_t dx_stride;              /* >= hidden_size */
  void* dgate_up;                 /* device [2 * intermediate_size, hidden_size] of dtype, or NULL */
  int64_t dgate_up_stride;        /* >= hidden_size */
  void* workspace;                /* device, moe_ep_gated_grad_workspace_bytes() bytes, 256-byte aligned */
  size_t workspace_bytes;
  int32_t dtype;                  /* MOE_EP_BF16 or MOE_EP_F16 */
  int32_t dout_dtype;             /* dtype, or MOE_EP_F32 */
  int32_t num_rows;
  int32_t hidden_size;            /* 8..2^22 */
  int32_t intermediate_size;      /* 8..2^22 */
  int32_t d_parts;                /* numbers of dtype that each of dg and du goes into the products as: 1 (or 0), 2 */
} moe_ep_gated_grad_args;

/* Bytes of device workspace moe_ep_gated_grad needs for these sizes (the
 * sizes, dtype and d_parts are read; pointers are not followed): 4 for each
 * element of dout (8 with two parts), and 8 MiB. */
MOE_EP_API int moe_ep_gated_grad_workspace_bytes(const moe_ep_gated_grad_args* args, size_t* out_bytes);

/* The gradients of moe_ep_gated's inputs:
 *   dg = dout * u * s * (1 + g * (1 - s)), s = 1 / (1 + exp(-g));  du = dout * g * s
 *   dx = dg gate_up[:I] + du gate_up[I:],  dgate_up = [dg^T x; du^T x]
 * each written whole, not added to (without rows dgate_up is zeros).  dg and
 * du are made in float32.  With one part they are rounded once to dtype before
 * the products, which adds to the results' error about as much as their own
 * rounding does; with two they go in as the rounding and the rounding of what it
 * leaves, 16 bits for bfloat16 and 22 for float16, and the products take twice
 * as long.  float16 ones are multiplied with a power of two that brings the
 * largest finite one to 2^14..2^15 first, so that none overflows.  x is read for dgate_up only and gate_up for dx only; the other
 * may be NULL.  One kernel launch (float16: two) and one or two for each
 * gradient.  Outputs must not overlap inputs or one another.  The workspace
 * holds nothing between calls; calls that may overlap in time need one each. */
MOE_EP_API int moe_ep_gated_grad(const moe_ep_gated_grad_args* args, void* stream);

typedef struct moe_ep_adapter_args {
  const void* x;                  /* device [num_rows, in_features] of dtype */
  int64_t x_stride;               /* >= 0; 0 repeats one row */
  const void* weight;             /* device [out_features, in_features] of dtype */
  int64_t weight_stride;          /* >= in_features */
  const void* lora_a;             /* device [num_adapters, rank, in_features] of dtype */
  const void* lora_b;             /* device [num_adapters, out_features, rank] of dtype */
  const int32_t* adapter_ids;     /* device [num_rows] */
  const float* scales;            /* device [num_adapters], or NULL: all 1 */
  void* out;                      /* device [num_rows, out_features] of out_dtype */
  int64_t out_stride;             /* >= out_features */
  void* workspace;                /* device, moe_ep_adapter_workspace_bytes() bytes, 256-byte aligned */
  size_t workspace_bytes;
  int32_t dtype;                  /* MOE_EP_BF16 or MOE_EP_F16 */
  int32_t out_dtype;              /* dtype, or MOE_EP_F32 */
  int32_t num_rows;               /* 0..2^25 */
  int32_t in_features;            /* 8..2^22 */
  int32_t out_features;           /* 1..2^22 */
  int32_t num_adapters;           /* 1..MOE_EP_MAX_EXPERTS */
  int32_t rank;                   /* 1..MOE_EP_MAX_RANK; smaller adapters are padded with zeros */
} moe_ep_adapter_args;

/* Largest rank of an adapter. */
#define MOE_EP_MAX_RANK 1024

/* Bytes of device workspace moe_ep_adapter_linear needs for these sizes (the
 * sizes are read; pointers are not followed): 6 for each row and rank (rounded
 * up to 32), 16 (rounded up to 8) up to 64 rows. */
MOE_EP_API int moe_ep_adapter_workspace_bytes(const moe_ep_adapter_args* args, size_t* out_bytes);

/* A projection that all rows share, with a low-rank adapter of each row's own:
 *   out[r] = weight x[r] + scales[a] * lora_b[a] (lora_a[a] x[r]), a = adapter_ids[r];
 * rows whose id is outside [0, num_adapters) have no adapter.  lora_a[a] x is
 * kept as float32, whole, and the sum of both products is rounded once.  What
 * is in an adapter that a row does not name does not reach the row; infinities
 * and NaN in its own give what the formula gives (but an infinity in lora_b
 * times a low value below 2^-100 may give NaN).  out must not overlap an input,
 * each taken from its first element to its last.  The workspace holds nothing
 * between calls; calls that may overlap in time need one each.  Two kernel
 * launches. */
MOE_EP_API int moe_ep_adapter_linear(const moe_ep_adapter_args* args, void* stream);

/* Static text for a status code. */
MOE_EP_API const char* moe_ep_status_string(int status);

/* Description of this thread's most recent failed call ("" if none). */
MOE_EP_API const char* moe_ep_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* MOE_EP_H */

/*
 * recsa_dense.h - dense operators over a RecSA token cache, for NVIDIA B200 (sm_100a):
 * attention over every visible token (a chunk of new tokens or single decode tokens),
 * the same with a sliding window and a few first tokens that stay visible (sinks), the
 * attention weight each cache slot receives, and the eviction of slots by that weight.
 *
 * They read the token caches of recsa.h's recsa_tree (contiguous or paged, keys stored
 * before RoPE, equal or per-sequence lengths) for the layers of a model that stay dense or
 * windowed, and keep a cache bounded.  The conventions of recsa.h hold: device pointers,
 * 16-byte alignment, asynchronous calls, nothing allocated, argument errors reported with a
 * status and nothing launched, per-sequence lengths clamped and flagged, page-table entries
 * outside the pool never dereferenced (such a token is skipped and flagged).
 * Outputs may not overlap the call's queries, weights or kept slots (refused); what the pages
 * of one pool or another name is the caller's.
 *
 * A cache without a tree: in every call here tree->k_node, tree->v_node and tree->pooler may
 * be NULL together.  Calls that add tokens update the tree when there is one, and write the
 * token rows alone when there is none.
 *
 * Tokens and positions.  L is a sequence's token count and slot t holds the key of position
 * t.  A query at position p sees the tokens t < p, or with a window only
 * t < sinks and p - window <= t < p.  Scores are softmax_scale * <R_p q, R_t k_t> with the
 * rotate-half RoPE R of recsa.h; a sink that lies outside the window is scored at its rank
 * among the visible tokens (the query then sits at sinks + window), or at its token position.
 * So p counts the tokens that a query sees, as in recsa_decode: a query that sees its own
 * token, at position p - 1, still sits one past it.  A causal RoPE layer has the query at its
 * own token instead, <R_i q_i, R_t k_t> for t <= i: recsa_view.own_token = 2.  The query of
 * bound p then sits at p - 1 (for the sinks at sinks + window - 1), in every call here.
 * The output is the softmax-weighted mean of the visible values; a query that sees nothing
 * outputs zeros.  Rows that a query does not see never reach its output, whatever they hold.
 */
#ifndef RECSA_DENSE_H
#define RECSA_DENSE_H

#include "recsa.h"

#ifdef __cplusplus
extern "C" {
#endif

/* Which tokens a query sees (NULL stands for all zeros: every token, decode positions).
 *   sinks          : first tokens that stay visible beside the window (ignored without one).
 *   window         : 0 = no window; else the query's last `window` tokens are visible.
 *   sink_positions : 0 = a sink outside the window is scored at its rank among the visible
 *                    tokens; 1 = at its token position.
 *   causal         : 0 = every query sits at p = L (decode); 1 = the n queries belong to the
 *                    last n tokens of the cache: query i sits at p = L - n + i.
 *   own_token      : with causal: 1 or 2 = a query also sees its own token
 *                    (p = L - n + i + 1); 0 is the position convention of recsa_prefill_chunk.
 *                    2, causal or not: a query sits at p - 1, its own token's position (that
 *                    of the cache's last token for queries at the end, and in a decode step):
 *                    the attention of a dense or windowed RoPE layer.
 *   kernel         : launch-shape override of the attention calls: 0 = automatic by the sizes;
 *                    1 = the rows kernel (8 or 16 query rows a block; every output type);
 *                    2 = the chunk kernel (256 query rows a block on tcgen05; bf16 outputs,
 *                    else RECSA_ERR_UNSUPPORTED).  Results agree up to their rounding.
 * A query whose p is 0 or less (a sequence shorter than the chunk) sees nothing. */
typedef struct recsa_view {
  int32_t sinks;
  int32_t window;
  int32_t sink_positions;
  int32_t causal;
  int32_t own_token;
  int32_t kernel;
} recsa_view;

/* Bytes of the workspace (about 48 MB, and up to 320 MB - for sequences of more than 1.2 million
 * tokens up to 1.25 GB - for the rotated rows of long chunks) of the dense calls on caches of `batch` sequences of up to
 * `capacity` tokens (host only).  Unlike recsa_decode's, this workspace is written by every
 * call (partial sums of sequences that several thread blocks share), so calls whose GPU work
 * can overlap - other streams, two captured graphs replayed side by side - each need their
 * own; calls ordered on one stream share one. */
RECSA_API recsa_status recsa_dense_workspace_size(const recsa_params *params, int32_t batch, int64_t capacity,
                                                  size_t *bytes_out);

/* Fill a workspace of ws_bytes >= recsa_dense_workspace_size() bytes (device pointer,
 * 16-byte aligned): the rotation tables of params->rope_base, zeroed counters, cleared error
 * word.  Call once before the first dense call that uses it.  recsa_check_device_errors
 * reads and clears its error word. */
RECSA_API recsa_status recsa_dense_workspace_init(const recsa_params *params, int32_t batch, int64_t capacity,
                                                  void *ws, size_t ws_bytes, recsa_stream_t stream);

/* Attention of num_queries queries per sequence over the tokens that are in the cache.
 *   q   : bf16 [batch][num_queries][Hq][128], pre-RoPE.
 *   out : [batch][num_queries][Hq][128], fp32 if out_is_fp32 else bf16.
 * Accuracy.  fp32 outputs come from two fp16 parts of rotated rows (22 bits) and three bf16 parts
 * of probabilities on the tensor cores, as accurate as fp32 arithmetic; rows with elements that
 * those parts do not hold (keys beyond 4094, queries beyond about 8000 at the default scale) are
 * computed in fp32, two to three times slower.  bf16 outputs of the rows kernel come from two bf16
 * parts: a score is off by at most 3 * 2^-16 softmax_scale |q| |k|, an output by twice that, 2^-16
 * of the largest value seen and its own rounding.  The chunk kernel rounds rotated rows to fp16 and
 * probabilities to bf16: 2^-10 softmax_scale |q| |k|, and 2^-8 beside the output's own rounding.
 * Errors so grow with the scores; measured on random rows, as shares of the output's norm (and of
 * the worst row's):
 *   spread of the scores        1                    5                    20
 *   fp32 output           1.8e-7 (4e-7)        4.5e-7 (2.4e-6)      1.6e-6 (7e-6)
 *   bf16, rows kernel     1.7e-3 (2.2e-3)      1.7e-3 (2.3e-3)      1.4e-3 (2.2e-3)
 *   bf16, chunk kernel    2.4e-3 (3.6e-3)      2.4e-3 (5.0e-3)      2.4e-3 (1.2e-2)
 * The automatic choice goes by the sizes of the whole call; view->kernel = 1 keeps a query's
 * accuracy the same whatever it is batched with. */
RECSA_API recsa_status recsa_dense_attend(const recsa_params *params, const recsa_tree *tree, const recsa_view *view,
                                          const void *q, int32_t num_queries, void *out, int32_t out_is_fp32,
                                          void *ws, size_t ws_bytes, recsa_stream_t stream);

/* recsa_prefill_chunk's dense counterpart: appends `chunk` tokens to every sequence
 * (k_new / v_new: bf16 [batch][chunk][Hkv][128]), advances the lengths, and attends the
 * chunk's queries causally (view->causal is taken as 1).  On success tree->length becomes
 * L + chunk. */
RECSA_API recsa_status recsa_dense_prefill_chunk(const recsa_params *params, recsa_tree *tree, const recsa_view *view,
                                                 const void *k_new, const void *v_new, const void *q, int32_t chunk,
                                                 void *out, int32_t out_is_fp32, void *ws, size_t ws_bytes,
                                                 recsa_stream_t stream);

/* recsa_decode_step's dense counterpart: per sequence appends one token at its device length,
 * advances the length and attends that token's query over the tokens it then holds (its own
 * included).  Every launch parameter comes from the capacity, so the call can be captured into
 * a CUDA graph.  Needs tree->seq_len; tree->length is neither read nor written (the other calls
 * take it as the lengths' bound: the caller sets it before them).  A sequence
 * with no room keeps its tokens and length and is flagged (RECSA_ERR_DEVICE_CHECK).
 * view->causal is not used; own_token = 2 puts the query at its own token's position. */
RECSA_API recsa_status recsa_dense_decode_step(const recsa_params *params, const recsa_tree *tree,
                                               const recsa_view *view, const void *k_new, const void *v_new,
                                               const void *q, void *out, int32_t out_is_fp32, void *ws,
                                               size_t ws_bytes, recsa_stream_t stream);

/* The softmax weight that each cache slot receives from the queries, summed over the queries
 * and over the query heads of its KV group, in fp32.
 * Weights are as accurate as fp32 outputs above.  (With more than 8 query rows a KV group, a head
 * with elements beyond the parts' range is scored from two bf16 parts, 2^-16, instead.)
 *   weights : fp32 [batch][Hkv][capacity]; slots [0, L) are overwritten (accumulate = 0) or
 *             added to (accumulate = 1), slots at or past a sequence's L are left as they are.
 * Views with a window are RECSA_ERR_UNSUPPORTED, and so are more than 8 query rows a KV group
 * over sequences of more than about 100 million tokens (their partial sums do not fit). */
RECSA_API recsa_status recsa_accumulate_weights(const recsa_params *params, const recsa_tree *tree,
                                                const recsa_view *view, const void *q, int32_t num_queries,
                                                float *weights, int32_t accumulate, void *ws, size_t ws_bytes,
                                                recsa_stream_t stream);

/* Cut every (sequence, KV head) of a cache to its `keep` most attended slots.
 * A sequence of L <= keep tokens keeps them all.  Otherwise slots [0, sinks) and the last
 * `recent` slots are kept, and of the others those with the largest weights up to `keep`
 * slots in all (ties to the lower slot; a weight that is NaN ranks below every number).
 * The kept rows move, in slot order, to slots 0 .. min(L, keep) - 1: a kept key's position
 * becomes its rank among the kept ones.
 *   weights      : fp32 [batch][Hkv][tree->capacity], read.
 *   kept         : int32 [batch][Hkv][keep], written: the kept slots ascending, -1 past them.
 *   into         : the cache that receives the rows (its capacity >= min(keep, tree->length);
 *                  the same batch and heads), or NULL to compact `tree` in place.  Its length
 *                  (and its seq_len, which it needs when `tree` has one) become those of the
 *                  kept rows; its tree, when it has one, is rebuilt over them.  A separate
 *                  cache may not share rows with `tree`.  In place, every page belongs to one
 *                  sequence.  Slots past the kept rows are left as they are.
 *   into_weights : NULL, or fp32 [batch][Hkv][capacity of the receiving cache] that receives
 *                  the kept slots' weights in the same order; in place it may be `weights`.
 *                  In place the slots from the kept ones up to the old length become 0, so that
 *                  tokens appended there start from 0 in recsa_accumulate_weights.  Beside
 *                  another cache, slots past the kept ones are left as they are: a buffer that
 *                  holds an earlier cache's weights is cleared by the caller before this call.
 * The call takes no workspace: a length outside [0, tree->length] (clamped), and a row that
 * moves from or to a page outside the pool, are flagged in the library's own error word, which
 * recsa_check_device_errors reads and clears with any workspace.  A row from such a page
 * arrives as zeros; a row to such a page is not written.
 * Needs keep >= 1 and sinks + recent <= keep. */
RECSA_API recsa_status recsa_evict(const recsa_params *params, recsa_tree *tree, const float *weights, int32_t keep,
                                   int32_t sinks, int32_t recent, int32_t *kept, recsa_tree *into,
                                   float *into_weights, recsa_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* RECSA_DENSE_H */

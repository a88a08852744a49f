// Host side of the dense cache operators: argument checks and the launches behind each call.
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>

#include "recsa_dense_internal.h"
#include "recsa_evict.h"

using namespace recsa;

namespace {

recsa_status check_cache(const recsa_params *p, const recsa_tree *t, TreeGeom *g) {
  recsa_status s = check_params(p);
  if (s != RECSA_OK) return s;
  if (!t) return fail(RECSA_ERR_INVALID_ARGUMENT, "tree is NULL");
  const int have = (t->k_node != nullptr) + (t->v_node != nullptr) + (t->pooler != nullptr);
  if (have != 0 && have != 3)
    return fail(RECSA_ERR_INVALID_ARGUMENT, "tree->k_node, v_node and pooler are all given or all NULL");
  return check_tree(p, t, g, have == 0);
}

bool has_tree(const recsa_tree *t) { return t->k_node != nullptr; }

recsa_status check_view(const recsa_view *v) {
  if (!v) return RECSA_OK;
  if (v->sinks < 0 || v->window < 0) return fail(RECSA_ERR_INVALID_ARGUMENT, "sinks %d, window %d", v->sinks, v->window);
  if ((int64_t)v->sinks + v->window > ((int64_t)1 << 30))
    return fail(RECSA_ERR_UNSUPPORTED, "sinks %d + window %d > 2^30", v->sinks, v->window);
  if (v->kernel < 0 || v->kernel > 2) return fail(RECSA_ERR_INVALID_ARGUMENT, "kernel %d (0 .. 2)", v->kernel);
  if (v->sink_positions != 0 && v->sink_positions != 1)
    return fail(RECSA_ERR_INVALID_ARGUMENT, "sink_positions %d (0 or 1)", v->sink_positions);
  if (v->own_token < 0 || v->own_token > 2) return fail(RECSA_ERR_INVALID_ARGUMENT, "own_token %d (0 .. 2)", v->own_token);
  return RECSA_OK;
}

recsa_status check_buffer(const void *p, const char *name) {
  if (!p) return fail(RECSA_ERR_INVALID_ARGUMENT, "%s is NULL", name);
  if (!aligned16(p)) return fail(RECSA_ERR_INVALID_ARGUMENT, "%s is not 16-byte aligned", name);
  return RECSA_OK;
}

recsa_status check_dense_ws(const recsa_params *p, const recsa_tree *t, const void *ws, size_t ws_bytes) {
  recsa_status s = check_buffer(ws, "workspace");
  if (s != RECSA_OK) return s;
  size_t need = 0;
  s = recsa_dense_workspace_size(p, t->batch, t->capacity, &need);
  if (s != RECSA_OK) return s;
  if (ws_bytes < need)
    return fail(RECSA_ERR_WORKSPACE_TOO_SMALL, "workspace %zu bytes < %zu needed", ws_bytes, need);
  return RECSA_OK;
}

// Buffers that one call reads in some blocks and writes in others may not overlap.
struct Extent {
  const void *p;
  size_t bytes;
  const char *name;
};
recsa_status check_apart(const Extent &a, const Extent &b) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
  if (a.p && b.p && x < y + b.bytes && y < x + a.bytes)
    return fail(RECSA_ERR_INVALID_ARGUMENT, "%s overlaps %s", a.name, b.name);
  return RECSA_OK;
}
size_t query_bytes(const recsa_params *p, const recsa_tree *t, int32_t nq) {
  return (size_t)t->batch * nq * p->num_q_heads * kRowBytes;
}
recsa_status check_out(const recsa_params *p, const recsa_tree *t, const void *q, int32_t nq, const void *out,
                       int32_t out_is_fp32) {
  const size_t bytes = query_bytes(p, t, nq);
  return check_apart({out, bytes * (out_is_fp32 ? 2 : 1), "out"}, {q, bytes, "q"});
}

DenseArgs dense_args(const recsa_params *p, const recsa_tree *t, const recsa_view *v, const void *q, int32_t nq,
                     int64_t length, bool causal, bool own, void *ws) {
  DenseArgs a = {};
  a.k = reinterpret_cast<const uint16_t *>(t->k_tok);
  a.v = reinterpret_cast<const uint16_t *>(t->v_tok);
  a.q = reinterpret_cast<const uint16_t *>(q);
  a.seq_len = t->seq_len;
  a.capacity = t->capacity;
  if (t->page_table) {
    a.pages = t->page_table;
    a.page_shift = __builtin_ctz((unsigned)t->page_size);
    a.pages_per_seq = (int32_t)(t->capacity / t->page_size);
    a.num_pages = t->num_pages;
  }
  a.batch = t->batch;
  a.hkv = p->num_kv_heads;
  a.group_shift = __builtin_ctz((unsigned)(p->num_q_heads / p->num_kv_heads));
  a.nq = nq;
  a.length = (int32_t)length;
  if (v && v->window > 0) {
    a.sinks = v->sinks;
    a.window = v->window;
    a.rank_sinks = v->sink_positions == 0;
  }
  a.causal = causal;
  a.own = causal && own;
  a.back = v && v->own_token == 2;
  a.nsplit = a.tiles = 1;
  a.qscale = (p->softmax_scale > 0.f ? p->softmax_scale : 1.0f / std::sqrt((float)kD)) * kLog2e;
  a.rope_base = p->rope_base;
  a.hdr = reinterpret_cast<WsHeader *>(ws);
  return a;
}

// Whether a bf16 output takes the chunk kernel.  With K keys in all (sequences x KV heads x keys
// seen) and t tiles of 16 query rows a group, the rows kernel measured 18 us + 0.12 ns K t, the
// chunk kernel (up to 256 rows) 38 us + 0.2 ns K: at 32 heads of 8192 keys they cross at 2 tiles
// (85 and 89 us), at 8 heads of 8192 between 4 and 6 (48 and 57, 60 and 57 us), at 2 heads of 2000
// the rows kernel is ahead at 32 (31 and 44 us).
bool chunk_pays(int64_t keys, int64_t rows) {
  return (double)keys * (double)(12 * ceil_div(rows, 16) - 20) > 2e6;
}

// The work items of the launch fit its grid.
recsa_status check_rows(const DenseArgs &a) {
  const int64_t rows = ((int64_t)a.nq << a.group_shift) * a.hkv * a.batch;
  if (rows > ((int64_t)1 << 31) - 16 * (int64_t)a.batch * a.hkv)
    return fail(RECSA_ERR_UNSUPPORTED, "%lld query rows", (long long)rows);
  return RECSA_OK;
}

// The most keys any query tile of the launch can see.
int64_t max_keys(const DenseArgs &a) {
  const int64_t n = a.length;
  if (!a.window) return n;
  return std::min<int64_t>(n, (int64_t)a.sinks + a.window + (a.causal ? std::min(a.nq, 256 >> a.group_shift) : 0));
}

// The kernel a call asks for, before anything is queued.
recsa_status check_kernel(const recsa_view *v, int32_t out_is_fp32) {
  if (v && v->kernel == 2 && out_is_fp32) return fail(RECSA_ERR_UNSUPPORTED, "the chunk kernel writes bf16 outputs");
  return RECSA_OK;
}

recsa_status attend(DenseArgs a, const recsa_view *v, void *out, int32_t out_is_fp32, size_t ws_bytes, void *stream) {
  a.out = out;
  a.out_fp32 = out_is_fp32 ? 1 : 0;
  const int kernel = v ? v->kernel : 0;
  const int64_t rows = (int64_t)a.nq << a.group_shift;  // of a KV group
  int rc = kNoRoom;
  if (!a.out_fp32 && (kernel == 2 || (kernel == 0 && chunk_pays((int64_t)a.batch * a.hkv * max_keys(a), rows))))
    rc = launch_dense_chunk(a, max_keys(a), (int64_t)(ws_bytes - kDenseImages), stream);
  if (rc == kNoRoom) rc = launch_dense_rows(a, max_keys(a), nullptr, stream);
  return rc != 0 ? cuda_fail(rc, "dense attend") : RECSA_OK;
}

}  // namespace

extern "C" {

RECSA_API recsa_status recsa_dense_workspace_size(const recsa_params *params, int32_t batch, int64_t capacity,
                                                  size_t *bytes_out) {
  const recsa_status s = check_params(params);
  if (s != RECSA_OK) return s;
  if (batch < 1) return fail(RECSA_ERR_INVALID_ARGUMENT, "batch %d < 1", batch);
  if (capacity < 1) return fail(RECSA_ERR_INVALID_ARGUMENT, "capacity %lld < 1", (long long)capacity);
  if (capacity > ((int64_t)1 << 30))
    return fail(RECSA_ERR_UNSUPPORTED, "capacity %lld > 2^30 tokens", (long long)capacity);
  if (!bytes_out) return fail(RECSA_ERR_INVALID_ARGUMENT, "bytes_out is NULL");
  // rotated rows of the chunk kernel: all heads' keys and queries up to kMaxDenseImages, or else
  // one head's keys (and an eighth of the room for its queries)
  const int64_t rows = std::min<int64_t>((capacity + 127) / 128 * 128 * batch, 1 << 20);
  const int64_t all = rows * (params->num_kv_heads + 2 * (int64_t)params->num_q_heads) * kRowBytes * 9 / 8 + (1 << 20);
  const int64_t head = (capacity + 127) / 128 * (128 * kRowBytes + 16) / 7 * 8 + (1 << 20);
  const int64_t most = std::max<int64_t>(kMaxDenseImages, std::min<int64_t>(head, kMaxHeadImages));
  *bytes_out = kDenseImages + (size_t)(std::min(all, most) + 255) / 256 * 256;
  return RECSA_OK;
}

RECSA_API recsa_status recsa_dense_workspace_init(const recsa_params *params, int32_t batch, int64_t capacity,
                                                  void *ws, size_t ws_bytes, recsa_stream_t stream) {
  size_t need = 0;
  recsa_status s = recsa_dense_workspace_size(params, batch, capacity, &need);
  if (s != RECSA_OK) return s;
  s = check_buffer(ws, "workspace");
  if (s != RECSA_OK) return s;
  if (ws_bytes < need) return fail(RECSA_ERR_WORKSPACE_TOO_SMALL, "workspace %zu bytes < %zu needed", ws_bytes, need);
  const int rc = launch_dense_init(ws, (double)params->rope_base, stream);
  return rc != 0 ? cuda_fail(rc, "dense workspace") : RECSA_OK;
}

RECSA_API recsa_status recsa_dense_attend(const recsa_params *params, const recsa_tree *tree, const recsa_view *view,
                                          const void *q, int32_t num_queries, void *out, int32_t out_is_fp32,
                                          void *ws, size_t ws_bytes, recsa_stream_t stream) {
  TreeGeom g;
  recsa_status s = check_cache(params, tree, &g);
  if (s == RECSA_OK) s = check_view(view);
  if (s == RECSA_OK) s = check_kernel(view, out_is_fp32);
  if (s != RECSA_OK) return s;
  if (num_queries < 1) return fail(RECSA_ERR_INVALID_ARGUMENT, "num_queries %d < 1", num_queries);
  s = check_buffer(q, "q");
  if (s == RECSA_OK) s = check_buffer(out, "out");
  if (s == RECSA_OK) s = check_dense_ws(params, tree, ws, ws_bytes);
  if (s != RECSA_OK) return s;
  const DenseArgs a = dense_args(params, tree, view, q, num_queries, tree->length, view && view->causal,
                                 view && view->own_token, ws);
  s = check_rows(a);
  if (s == RECSA_OK) s = check_out(params, tree, q, num_queries, out, out_is_fp32);
  if (s != RECSA_OK) return s;
  return attend(a, view, out, out_is_fp32, ws_bytes, stream);
}

RECSA_API recsa_status recsa_dense_prefill_chunk(const recsa_params *params, recsa_tree *tree, const recsa_view *view,
                                                 const void *k_new, const void *v_new, const void *q, int32_t chunk,
                                                 void *out, int32_t out_is_fp32, void *ws, size_t ws_bytes,
                                                 recsa_stream_t stream) {
  TreeGeom g;
  recsa_status s = check_cache(params, tree, &g);
  if (s == RECSA_OK) s = check_view(view);
  if (s == RECSA_OK) s = check_kernel(view, out_is_fp32);
  if (s != RECSA_OK) return s;
  if (chunk < 1) return fail(RECSA_ERR_INVALID_ARGUMENT, "chunk %d < 1", chunk);
  s = check_buffer(k_new, "k_new");
  if (s == RECSA_OK) s = check_buffer(v_new, "v_new");
  if (s == RECSA_OK) s = check_buffer(q, "q");
  if (s == RECSA_OK) s = check_buffer(out, "out");
  if (s != RECSA_OK) return s;
  const int64_t L = tree->length, L2 = L + chunk;
  if (L2 > tree->capacity)
    return fail(RECSA_ERR_CAPACITY, "length %lld + chunk %d > capacity %lld", (long long)L, chunk,
                (long long)tree->capacity);
  s = check_dense_ws(params, tree, ws, ws_bytes);
  if (s != RECSA_OK) return s;
  const DenseArgs a = dense_args(params, tree, view, q, chunk, L2, true, view && view->own_token, ws);
  s = check_rows(a);
  if (s == RECSA_OK) s = check_out(params, tree, q, chunk, out, out_is_fp32);
  if (s != RECSA_OK) return s;
  int rc;
  if (has_tree(tree)) {
    s = extend_tree(g, *tree, k_new, v_new, L, chunk, stream, &a.hdr->err);
    if (s != RECSA_OK) return s;
  } else {
    rc = launch_append_tokens(a, tree->k_tok, tree->v_tok, k_new, v_new, L, chunk, L2, stream);
    if (rc != 0) return cuda_fail(rc, "append");
  }
  if (tree->seq_len) {
    rc = launch_advance_lengths(tree->seq_len, tree->batch, chunk, L2, stream);
    if (rc != 0) return cuda_fail(rc, "advance of the sequence lengths");
  }
  s = attend(a, view, out, out_is_fp32, ws_bytes, stream);
  if (s == RECSA_OK) tree->length = L2;
  return s;
}

RECSA_API recsa_status recsa_dense_decode_step(const recsa_params *params, const recsa_tree *tree,
                                               const recsa_view *view, const void *k_new, const void *v_new,
                                               const void *q, void *out, int32_t out_is_fp32, void *ws,
                                               size_t ws_bytes, recsa_stream_t stream) {
  TreeGeom g;
  recsa_status s = check_cache(params, tree, &g);
  if (s == RECSA_OK) s = check_view(view);
  if (s == RECSA_OK) s = check_kernel(view, out_is_fp32);
  if (s != RECSA_OK) return s;
  if (!tree->seq_len)
    return fail(RECSA_ERR_INVALID_ARGUMENT, "a decode step needs per-sequence lengths (tree->seq_len)");
  s = check_buffer(k_new, "k_new");
  if (s == RECSA_OK) s = check_buffer(v_new, "v_new");
  if (s == RECSA_OK) s = check_buffer(q, "q");
  if (s == RECSA_OK) s = check_buffer(out, "out");
  if (s == RECSA_OK) s = check_dense_ws(params, tree, ws, ws_bytes);
  if (s != RECSA_OK) return s;
  // every bound comes from the capacity, none from the current lengths
  const int64_t cap = tree->capacity;
  const DenseArgs a = dense_args(params, tree, view, q, 1, cap, false, false, ws);
  s = check_rows(a);
  if (s == RECSA_OK) s = check_out(params, tree, q, 1, out, out_is_fp32);
  if (s != RECSA_OK) return s;
  uint32_t *const err = &a.hdr->err;
  int rc = has_tree(tree) ? launch_extend(g, *tree, k_new, v_new, cap - 1, 1, levels_for(cap, g.b), stream, err, err)
                          : launch_append_tokens(a, tree->k_tok, tree->v_tok, k_new, v_new, 0, 1, cap, stream);
  if (rc != 0) return cuda_fail(rc, "append");
  rc = launch_advance_lengths(tree->seq_len, tree->batch, 1, cap, stream);
  if (rc != 0) return cuda_fail(rc, "advance of the sequence lengths");
  return attend(a, view, out, out_is_fp32, ws_bytes, stream);
}

RECSA_API recsa_status recsa_accumulate_weights(const recsa_params *params, const recsa_tree *tree,
                                                const recsa_view *view, const void *q, int32_t num_queries,
                                                float *weights, int32_t accumulate, void *ws, size_t ws_bytes,
                                                recsa_stream_t stream) {
  TreeGeom g;
  recsa_status s = check_cache(params, tree, &g);
  if (s == RECSA_OK) s = check_view(view);
  if (s != RECSA_OK) return s;
  if (view && view->window > 0) return fail(RECSA_ERR_UNSUPPORTED, "attention weights of a windowed view");
  if (num_queries < 1) return fail(RECSA_ERR_INVALID_ARGUMENT, "num_queries %d < 1", num_queries);
  s = check_buffer(q, "q");
  if (s == RECSA_OK) s = check_buffer(weights, "weights");
  if (s == RECSA_OK) s = check_dense_ws(params, tree, ws, ws_bytes);
  if (s != RECSA_OK) return s;
  const DenseArgs a = dense_args(params, tree, view, q, num_queries, tree->length, view && view->causal,
                                 view && view->own_token, ws);
  s = check_rows(a);
  if (s == RECSA_OK)
    s = check_apart({weights, (size_t)tree->batch * params->num_kv_heads * tree->capacity * sizeof(float), "weights"},
                    {q, query_bytes(params, tree, num_queries), "q"});
  if (s != RECSA_OK) return s;
  float *lse = reinterpret_cast<float *>(reinterpret_cast<char *>(ws) + kDenseLse);
  const int rc = launch_dense_weights(a, lse, weights, accumulate ? 1 : 0, (int64_t)(ws_bytes - kDenseImages), stream);
  if (rc == kNoRoom)
    return fail(RECSA_ERR_UNSUPPORTED, "the partial sums of a sequence of %lld tokens do not fit a workspace",
                (long long)tree->length);
  return rc != 0 ? cuda_fail(rc, "attention weights") : RECSA_OK;
}

static EvictCache evict_cache(const recsa_tree *t) {
  EvictCache c = {};
  c.k = reinterpret_cast<uint4 *>(t->k_tok);
  c.v = reinterpret_cast<uint4 *>(t->v_tok);
  c.capacity = t->capacity;
  if (t->page_table) {
    c.pages = t->page_table;
    c.page_shift = __builtin_ctz((unsigned)t->page_size);
    c.pages_per_seq = (int32_t)(t->capacity / t->page_size);
    c.num_pages = t->num_pages;
  }
  return c;
}

RECSA_API recsa_status recsa_evict(const recsa_params *params, recsa_tree *tree, const float *weights, int32_t keep,
                                   int32_t sinks, int32_t recent, int32_t *kept, recsa_tree *into,
                                   float *into_weights, recsa_stream_t stream) {
  TreeGeom g, gi;
  recsa_status s = check_cache(params, tree, &g);
  if (s != RECSA_OK) return s;
  s = check_buffer(weights, "weights");
  if (s == RECSA_OK) s = check_buffer(kept, "kept");
  if (s != RECSA_OK) return s;
  if (keep < 1) return fail(RECSA_ERR_INVALID_ARGUMENT, "keep %d < 1", keep);
  if (sinks < 0 || recent < 0 || (int64_t)sinks + recent > keep)
    return fail(RECSA_ERR_INVALID_ARGUMENT, "sinks %d + recent %d outside [0, keep %d]", sinks, recent, keep);
  const bool in_place = !into || into == tree;
  recsa_tree *const to = in_place ? tree : into;
  const int64_t most = std::min<int64_t>(keep, tree->length);
  gi = g;
  if (!in_place) {
    s = check_cache(params, into, &gi);
    if (s != RECSA_OK) return s;
    if (into->batch != tree->batch)
      return fail(RECSA_ERR_INVALID_ARGUMENT, "into->batch %d, tree->batch %d", into->batch, tree->batch);
    if (into->capacity < most)
      return fail(RECSA_ERR_CAPACITY, "into->capacity %lld < %lld kept slots", (long long)into->capacity,
                  (long long)most);
    if (tree->seq_len && !into->seq_len)
      return fail(RECSA_ERR_INVALID_ARGUMENT, "into needs per-sequence lengths (seq_len), as tree has them");
    if (tree->seq_len && into->seq_len == tree->seq_len)
      return fail(RECSA_ERR_INVALID_ARGUMENT, "into->seq_len is tree->seq_len");
    if (into->k_tok == tree->k_tok || into->v_tok == tree->v_tok || into->k_tok == tree->v_tok ||
        into->v_tok == tree->k_tok)
      return fail(RECSA_ERR_INVALID_ARGUMENT, "into shares its rows with tree (pass NULL to compact in place)");
  }
  // Rows that are read and written.  (The pages of two pools may interleave without sharing a row:
  // what a page table names is the caller's.)
  const size_t slots = (size_t)tree->batch * params->num_kv_heads;
  const Extent from[2] = {{tree->k_tok, tree->page_table ? 0 : slots * tree->capacity * kRowBytes, "tree->k_tok"},
                          {tree->v_tok, tree->page_table ? 0 : slots * tree->capacity * kRowBytes, "tree->v_tok"}};
  const Extent dest[2] = {{to->k_tok, to->page_table ? 0 : slots * to->capacity * kRowBytes, "into->k_tok"},
                          {to->v_tok, to->page_table ? 0 : slots * to->capacity * kRowBytes, "into->v_tok"}};
  if (!to->page_table) s = check_apart(dest[0], dest[1]);
  for (int i = 0; i < 4 && s == RECSA_OK && !in_place && !tree->page_table && !to->page_table; ++i)
    s = check_apart(dest[i & 1], from[i >> 1]);
  const Extent old_weights = {weights, slots * tree->capacity * sizeof(float), "weights"},
               new_weights = {into_weights, slots * to->capacity * sizeof(float), "into_weights"},
               slots_kept = {kept, slots * keep * sizeof(int32_t), "kept"};
  if (s == RECSA_OK && !(in_place && into_weights == weights)) s = check_apart(new_weights, old_weights);
  if (s == RECSA_OK) s = check_apart(slots_kept, old_weights);
  if (s == RECSA_OK) s = check_apart(slots_kept, new_weights);
  if (s != RECSA_OK) return s;
  if (into_weights) {
    s = check_buffer(into_weights, "into_weights");
    if (s != RECSA_OK) return s;
    if (!in_place && into_weights == weights)
      return fail(RECSA_ERR_INVALID_ARGUMENT, "into_weights is weights, but into is another cache");
  }
  if ((int64_t)tree->batch * params->num_kv_heads > 0x7fffffff / 16)
    return fail(RECSA_ERR_UNSUPPORTED, "%d sequences of %d KV heads", tree->batch, params->num_kv_heads);
  EvictArgs a = {};
  a.from = evict_cache(tree);
  a.to = evict_cache(to);
  a.weights = weights;
  a.to_weights = into_weights;
  a.kept = kept;
  a.seq_len = tree->seq_len;
  a.capacity = tree->capacity;
  a.to_capacity = to->capacity;
  a.batch = tree->batch;
  a.hkv = params->num_kv_heads;
  a.length = (int32_t)tree->length;
  a.keep = keep;
  a.sinks = sinks;
  a.recent = recent;
  const int rc = launch_evict(a, in_place, to->seq_len, stream);
  if (rc != 0) return cuda_fail(rc, "evict");
  if (has_tree(to) && most > 0) {
    recsa_tree now = *to;
    now.length = most;
    s = build_range(gi, now, most, 0, false, stream);
    if (s != RECSA_OK) return s;
  }
  to->length = most;
  return RECSA_OK;
}

}  // extern "C"

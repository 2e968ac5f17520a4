// C ABI of the paged cache's data (declared in include/smcsd.h): argument
// checks and launches.  No allocation, no synchronisation.
#include <cmath>

#include "cache_ops.h"
#include "kernels.h"
#include "smcsd.h"

namespace smcsd {

static bool cache_ok(const smc_cache *c) {
  if (!c || !c->k || !c->v) return false;
  if (c->layers < 1 || c->blocks < 1 || c->block_size < 1 || c->kv_heads < 1 || c->head_dim < 1) {
    return false;
  }
  if (c->layers > 32767 || c->block_size > (1 << 20) || c->kv_heads > (1 << 16) ||
      c->head_dim > (1 << 16)) {
    return false;
  }
  // the elements of one block are counted in 32 bits
  if (static_cast<double>(c->block_size) * c->kv_heads * c->head_dim >= 536870912.0) return false;
  if (c->layer_stride < 0 || c->block_stride < 0 || c->token_stride < 0 || c->head_stride < 0) {
    return false;
  }
  const int esz = dtype_bytes(c->dtype);
  return reinterpret_cast<uintptr_t>(c->k) % esz == 0 && reinterpret_cast<uintptr_t>(c->v) % esz == 0;
}

static bool dtype_ok(int dtype) { return dtype == SMC_F32 || dtype == SMC_BF16 || dtype == SMC_F16; }

static bool batch_ok(const smc_batch *b) {
  if (!b || !b->tables || !b->seq_len) return false;
  if (b->S < 1 || b->T < 1 || b->rows < 0 || b->max_new < 1 || b->max_new > SMC_MAX_NEW) return false;
  if (b->group < 1 || b->S % b->group != 0) return false;
  if (!b->row_start && static_cast<int64_t>(b->S) * b->max_new != b->rows) return false;
  return true;
}

// (a path's places, and those of the threads past its end, are counted in 32 bits)
static bool path_ok(const int32_t *path, const int32_t *n_path, int32_t max_path) {
  return path && n_path && max_path >= 1 && max_path <= (1 << 30);
}

// The stride of an axis of length 1 is never used: it counts as an aligned one.
static int64_t stride_of(int64_t stride, int32_t length) { return length > 1 ? stride : 128; }

static CacheArgs to_cache(const smc_cache *c, int layer) {
  const int64_t at = layer * c->layer_stride * dtype_bytes(c->dtype);
  return {static_cast<char *>(c->k) + at, static_cast<char *>(c->v) + at,
          stride_of(c->layer_stride, c->layers), stride_of(c->block_stride, c->blocks),
          stride_of(c->token_stride, c->block_size), stride_of(c->head_stride, c->kv_heads),
          c->layers, c->blocks, c->block_size, c->kv_heads, c->head_dim, c->dtype};
}

static BatchArgs to_batch(const smc_batch *b) {
  return {b->tables, b->seq_len, b->row_start, b->S, b->T, b->rows, b->max_new, b->group};
}

static bool attention_shape_ok(const smc_cache *c, const smc_batch *b, int q_heads) {
  if (q_heads < 1 || q_heads > (1 << 16) || q_heads % c->kv_heads != 0) return false;
  // a token's number, and that of one up to 32 tiles on, is counted in 32 bits
  if (static_cast<double>(b->T) * c->block_size > SMC_MAX_TABLE_TOKENS) return false;
  // tiles of 64 tokens and at least one row of a key head, counted in 32 bits
  const double tiles = (static_cast<double>(b->T) * c->block_size / 64 + 1) * c->kv_heads * b->S *
                       (static_cast<double>(b->max_new) * (q_heads / c->kv_heads) / 128 + 1);
  return tiles < 536870912.0 &&
         static_cast<double>(b->rows) * q_heads < 2147483647.0 &&
         q_heads / c->kv_heads <= 128 &&
         static_cast<double>(b->max_new) * b->group * (q_heads / c->kv_heads) < 1073741824.0;
}

static size_t cache_ws_bytes(const smc_cache *c, const smc_batch *b, int q_heads) {
  if (!b) return kCacheStatusBytes;
  return attention_workspace_bytes(to_cache(c, 0), to_batch(b), q_heads);
}

static int32_t check_ws(const void *workspace, size_t have, size_t need) {
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255u) || have < need) {
    return SMC_ERR_WORKSPACE;
  }
  return SMC_OK;
}

cudaError_t launch_early(const void *fn, dim3 grid, unsigned block, size_t dyn, void **args,
                         cudaStream_t st) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = dyn;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelExC(&cfg, fn, args);
}

static bool cache8_ok(const smc_cache8 *c) {
  if (!cache_ok(&c->data) || !c->k_scale || !c->v_scale) return false;
  if (c->scale_layer_stride < 0 || c->scale_block_stride < 0 || c->scale_head_stride < 0) return false;
  return reinterpret_cast<uintptr_t>(c->k_scale) % 4 == 0 && reinterpret_cast<uintptr_t>(c->v_scale) % 4 == 0;
}

static ScaleArgs to_scales(const smc_cache8 *c, int layer) {
  const int64_t at = layer * c->scale_layer_stride;
  return {c->k_scale + at, c->v_scale + at, c->scale_layer_stride, c->scale_block_stride, c->scale_head_stride};
}

static size_t cache8_ws_bytes(const smc_cache8 *c, const smc_batch *b, int q_heads) {
  if (!b) return kCacheStatusBytes;
  return attention8_workspace_bytes(to_cache(&c->data, 0), to_batch(b), q_heads);
}

static bool multiple_of_16(const void *p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

// The checks and arguments that smc_tree_attention and smc_tree_attention8
// share; the cache's strides in multiples of `unit` elements.
static bool attention_args(const smc_attn_params *p, const smc_cache *cache, int32_t layer,
                           const smc_batch *batch, const void *q, const uint32_t *mask, void *out,
                           float *lse, void *workspace, int unit, AttnArgs *to) {
  if (!cache_ok(cache) || !batch_ok(batch) || layer < 0 || layer >= cache->layers) return false;
  if (p->reserved != 0 || !attention_shape_ok(cache, batch, p->q_heads)) return false;
  if (batch->rows > 0 && (!q || !out)) return false;
  if (!(std::isfinite(p->scale) && p->scale > 0.f)) return false;
  if (p->mask_words < 0 || (mask && p->mask_words < 1)) return false;
  if (cache->head_dim % unit != 0 || cache->head_dim > 128) return false;
  const CacheArgs c = to_cache(cache, layer);
  const int rows = batch->rows;
  for (const int64_t stride : {c.block_stride, c.token_stride, c.head_stride}) {
    if (stride < 0 || stride % unit != 0) return false;
  }
  for (const int64_t stride :
       {stride_of(p->q_row_stride, rows), stride_of(p->q_head_stride, p->q_heads),
        stride_of(p->out_row_stride, rows), stride_of(p->out_head_stride, p->q_heads)}) {
    if (stride < 0 || stride % 8 != 0) return false;
  }
  // an axis is not a broadcast one
  if (stride_of(p->q_row_stride, rows) == 0 || stride_of(p->q_head_stride, p->q_heads) == 0) return false;
  if (!multiple_of_16(c.k) || !multiple_of_16(c.v) || !multiple_of_16(q) || !multiple_of_16(out)) {
    return false;
  }
  AttnArgs a{};
  a.c = c;
  a.b = to_batch(batch);
  a.q = static_cast<const char *>(q);
  a.mask = mask;
  a.out = static_cast<char *>(out);
  a.lse = lse;
  a.q_heads = p->q_heads;
  a.mask_words = p->mask_words;
  a.scale = p->scale;
  a.q_row = stride_of(p->q_row_stride, rows);
  a.q_head = stride_of(p->q_head_stride, p->q_heads);
  a.o_row = p->out_row_stride;
  a.o_head = p->out_head_stride;
  a.status = static_cast<unsigned *>(workspace);
  *to = a;
  return true;
}

// Those of smc_qk_norm_rope and smc_qk_norm_rope8; rows of `dtype`.
static bool qk_args(const smc_qk_params *p, const smc_cache *cache, int32_t layer,
                    const smc_batch *batch, int dtype, const void *q, const void *k, const void *v,
                    const void *q_weight, const void *k_weight, const int32_t *positions,
                    const float *rope, void *q_out, void *workspace, QkArgs *to) {
  if (!cache_ok(cache) || !batch_ok(batch) || layer < 0 || layer >= cache->layers) return false;
  if (batch->rows > 0 && (!q || !k || !v || !q_out)) return false;
  if (p->q_heads < 1 || p->q_heads > (1 << 16)) return false;
  if (cache->head_dim > 256 || p->rot_dim < 0 || p->rot_dim > cache->head_dim || p->rot_dim % 2 != 0) {
    return false;
  }
  if (p->max_pos < 1 || (p->rot_dim > 0 && !rope)) return false;
  if (p->interleaved != 0 && p->interleaved != 1) return false;
  if (!(std::isfinite(p->eps) && p->eps >= 0.f) || !std::isfinite(p->weight_offset)) return false;
  for (const int64_t stride : {p->q_row_stride, p->q_head_stride, p->k_row_stride, p->k_head_stride,
                               p->v_row_stride, p->v_head_stride, p->out_row_stride,
                               p->out_head_stride}) {
    if (stride < 0) return false;
  }
  const uintptr_t esz = dtype_bytes(dtype);
  for (const void *ptr : {q, k, v, q_weight, k_weight, static_cast<const void *>(q_out)}) {
    if (reinterpret_cast<uintptr_t>(ptr) % esz != 0) return false;
  }
  QkArgs a{};
  a.c = to_cache(cache, layer);
  a.b = to_batch(batch);
  a.q = static_cast<const char *>(q);
  a.k = static_cast<const char *>(k);
  a.v = static_cast<const char *>(v);
  a.qw = static_cast<const char *>(q_weight);
  a.kw = static_cast<const char *>(k_weight);
  a.positions = positions;
  a.rope = rope;
  a.out = static_cast<char *>(q_out);
  a.q_heads = p->q_heads;
  a.rot = p->rot_dim;
  a.max_pos = p->max_pos;
  a.interleaved = p->interleaved;
  a.eps = p->eps;
  a.w0 = p->weight_offset;
  a.q_row = p->q_row_stride; a.q_head = p->q_head_stride;
  a.k_row = p->k_row_stride; a.k_head = p->k_head_stride;
  a.v_row = p->v_row_stride; a.v_head = p->v_head_stride;
  a.o_row = p->out_row_stride; a.o_head = p->out_head_stride;
  a.status = static_cast<unsigned *>(workspace);
  *to = a;
  return true;
}

}  // namespace smcsd

using namespace smcsd;

extern "C" {

size_t smc_cache_workspace_bytes(const smc_cache *cache, const smc_batch *batch, int32_t q_heads) {
  if (!cache || !dtype_ok(cache->dtype) || !cache_ok(cache)) return 0;
  if (batch && (!batch_ok(batch) || !attention_shape_ok(cache, batch, q_heads))) return 0;
  return cache_ws_bytes(cache, batch, q_heads);
}

int32_t smc_tree_attention(const smc_attn_params *p, const smc_cache *cache, int32_t layer,
                           const smc_batch *batch, const void *q, const uint32_t *mask, void *out,
                           float *lse, void *workspace, size_t ws_bytes, void *stream) {
  if (!p || !cache) return SMC_ERR_ARG;
  if (cache->dtype != SMC_BF16 && cache->dtype != SMC_F16) return SMC_ERR_DTYPE;
  AttnArgs a;
  if (!attention_args(p, cache, layer, batch, q, mask, out, lse, workspace, 8, &a)) return SMC_ERR_ARG;
  const int32_t rc = check_ws(workspace, ws_bytes, cache_ws_bytes(cache, batch, p->q_heads));
  if (rc != SMC_OK) return rc;
  return launch_tree_attention(a, workspace, static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? SMC_OK : SMC_ERR_LAUNCH;
}

int32_t smc_qk_norm_rope(const smc_qk_params *p, const smc_cache *cache, int32_t layer,
                         const smc_batch *batch, const void *q, const void *k, const void *v,
                         const void *q_weight, const void *k_weight, const int32_t *positions,
                         const float *rope, void *q_out, void *workspace, size_t ws_bytes,
                         void *stream) {
  if (!p || !cache) return SMC_ERR_ARG;
  if (!dtype_ok(cache->dtype)) return SMC_ERR_DTYPE;
  QkArgs a;
  if (!qk_args(p, cache, layer, batch, cache->dtype, q, k, v, q_weight, k_weight, positions, rope, q_out,
               workspace, &a)) {
    return SMC_ERR_ARG;
  }
  const int32_t rc = check_ws(workspace, ws_bytes, kCacheStatusBytes);
  if (rc != SMC_OK) return rc;
  return launch_qk_norm_rope(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? SMC_OK
                                                                                 : SMC_ERR_LAUNCH;
}

int32_t kv_copy_blocks(const smc_cache *cache, const int32_t *pairs, const int32_t *counts,
                       int32_t lists, int32_t max_pairs, void *workspace, size_t ws_bytes,
                       void *stream) {
  if (!cache) return SMC_ERR_ARG;
  if (!dtype_ok(cache->dtype)) return SMC_ERR_DTYPE;
  if (!cache_ok(cache) || !pairs || !counts || lists < 1 || max_pairs < 1 ||
      static_cast<int64_t>(lists) * max_pairs > (1 << 30)) {
    return SMC_ERR_ARG;
  }
  const int32_t rc = check_ws(workspace, ws_bytes, kCacheStatusBytes);
  if (rc != SMC_OK) return rc;
  return launch_copy_blocks(to_cache(cache, 0), pairs, counts, lists, max_pairs,
                            static_cast<unsigned *>(workspace),
                            static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? SMC_OK : SMC_ERR_LAUNCH;
}

int32_t kv_compact_tokens(const smc_cache *cache, const smc_batch *batch, const int32_t *path,
                          const int32_t *n_path, int32_t max_path, void *workspace,
                          size_t ws_bytes, void *stream) {
  if (!cache) return SMC_ERR_ARG;
  if (!dtype_ok(cache->dtype)) return SMC_ERR_DTYPE;
  if (!cache_ok(cache) || !batch_ok(batch) || !path_ok(path, n_path, max_path)) return SMC_ERR_ARG;
  const int32_t rc = check_ws(workspace, ws_bytes, kCacheStatusBytes);
  if (rc != SMC_OK) return rc;
  return launch_compact_tokens(to_cache(cache, 0), to_batch(batch), path, n_path, max_path,
                               static_cast<unsigned *>(workspace),
                               static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? SMC_OK : SMC_ERR_LAUNCH;
}

int32_t kv_truncate(const smc_params *p, const smc_kv *kv, const int32_t *new_len, void *workspace,
                    size_t ws_bytes, void *stream) {
  Workspace ws{};
  const int32_t rc = prepare_kv_call(p, kv, new_len, workspace, ws_bytes, &ws);
  if (rc != SMC_OK) return rc;
  const KvArgs k{kv->tables, kv->seq_len, kv->refcount, kv->free_list, kv->free_top,
                 kv->cow_pairs, kv->n_cow, kv->T, kv->block_size, kv->P};
  return launch_kv_truncate(p->B, p->N, k, new_len, ws, static_cast<cudaStream_t>(stream)) ==
                 cudaSuccess ? SMC_OK : SMC_ERR_LAUNCH;
}

size_t smc_cache8_workspace_bytes(const smc_cache8 *cache, const smc_batch *batch, int32_t q_heads) {
  if (!cache || cache->data.dtype != SMC_E4M3 || !cache8_ok(cache)) return 0;
  if (batch && (!batch_ok(batch) || !attention_shape_ok(&cache->data, batch, q_heads))) return 0;
  return cache8_ws_bytes(cache, batch, q_heads);
}

int32_t smc_tree_attention8(const smc_attn_params *p, const smc_cache8 *cache, int32_t layer,
                            const smc_batch *batch, int32_t dtype, const void *q, const uint32_t *mask,
                            void *out, float *lse, void *workspace, size_t ws_bytes, void *stream) {
  if (!p || !cache) return SMC_ERR_ARG;
  if (cache->data.dtype != SMC_E4M3 || (dtype != SMC_BF16 && dtype != SMC_F16)) return SMC_ERR_DTYPE;
  AttnArgs a;
  if (!cache8_ok(cache) ||
      !attention_args(p, &cache->data, layer, batch, q, mask, out, lse, workspace, 16, &a)) {
    return SMC_ERR_ARG;
  }
  const int32_t rc = check_ws(workspace, ws_bytes, cache8_ws_bytes(cache, batch, p->q_heads));
  if (rc != SMC_OK) return rc;
  return launch_tree_attention8(a, to_scales(cache, layer), dtype, workspace,
                                static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? SMC_OK : SMC_ERR_LAUNCH;
}

int32_t smc_qk_norm_rope8(const smc_qk_params *p, const smc_cache8 *cache, int32_t layer,
                          const smc_batch *batch, int32_t dtype, const void *q, const void *k,
                          const void *v, const void *q_weight, const void *k_weight,
                          const int32_t *positions, const float *rope, void *q_out, void *workspace,
                          size_t ws_bytes, void *stream) {
  if (!p || !cache) return SMC_ERR_ARG;
  if (cache->data.dtype != SMC_E4M3 || !dtype_ok(dtype)) return SMC_ERR_DTYPE;
  QkArgs a;
  // (a CTA takes a key head, one more the queries, on the grid's second axis; rows are counted in 32 bits, as far as
  // a CTA's last one past the arrays' end)
  if (!cache8_ok(cache) || cache->data.kv_heads > 65534 || !batch || batch->rows > (1 << 30) ||
      !qk_args(p, &cache->data, layer, batch, dtype, q, k, v, q_weight, k_weight, positions, rope, q_out,
               workspace, &a)) {
    return SMC_ERR_ARG;
  }
  const int32_t rc = check_ws(workspace, ws_bytes, kCacheStatusBytes);
  if (rc != SMC_OK) return rc;
  return launch_qk_norm_rope8(a, to_scales(cache, layer), dtype, static_cast<cudaStream_t>(stream)) ==
                 cudaSuccess ? SMC_OK : SMC_ERR_LAUNCH;
}

int32_t kv_copy_blocks8(const smc_cache8 *cache, const int32_t *pairs, const int32_t *counts,
                        int32_t lists, int32_t max_pairs, void *workspace, size_t ws_bytes, void *stream) {
  if (!cache) return SMC_ERR_ARG;
  if (cache->data.dtype != SMC_E4M3) return SMC_ERR_DTYPE;
  if (!cache8_ok(cache) || !pairs || !counts || lists < 1 || max_pairs < 1 ||
      static_cast<int64_t>(lists) * max_pairs > (1 << 30)) {
    return SMC_ERR_ARG;
  }
  const int32_t rc = check_ws(workspace, ws_bytes, kCacheStatusBytes);
  if (rc != SMC_OK) return rc;
  return launch_copy_blocks8(to_cache(&cache->data, 0), to_scales(cache, 0), pairs, counts, lists, max_pairs,
                             static_cast<unsigned *>(workspace), static_cast<cudaStream_t>(stream)) ==
                 cudaSuccess ? SMC_OK : SMC_ERR_LAUNCH;
}

int32_t kv_compact_tokens8(const smc_cache8 *cache, const smc_batch *batch, const int32_t *path,
                           const int32_t *n_path, int32_t max_path, void *workspace, size_t ws_bytes,
                           void *stream) {
  if (!cache) return SMC_ERR_ARG;
  if (cache->data.dtype != SMC_E4M3) return SMC_ERR_DTYPE;
  if (!cache8_ok(cache) || !batch_ok(batch) || !path_ok(path, n_path, max_path)) return SMC_ERR_ARG;
  if (cache->data.block_size > kMostCompactBlock || cache->data.kv_heads > 65535) return SMC_ERR_ARG;
  const int32_t rc = check_ws(workspace, ws_bytes, kCacheStatusBytes);
  if (rc != SMC_OK) return rc;
  return launch_compact_tokens8(to_cache(&cache->data, 0), to_scales(cache, 0), to_batch(batch), path, n_path,
                                max_path, static_cast<unsigned *>(workspace),
                                static_cast<cudaStream_t>(stream)) == cudaSuccess
             ? SMC_OK : SMC_ERR_LAUNCH;
}

}  // extern "C"

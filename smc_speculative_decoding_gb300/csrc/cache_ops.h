// Internal interface between the cache entry points (cache_api.cu) and their
// kernels (tree_attention.cu, qk_norm_rope.cu, cache_pages.cu).
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "kernels.h"
#include "smcsd.h"

namespace smcsd {

// One layer of the cache (k, v at the layer's first element) or, with
// layer_stride and layers, all of them.  Strides in elements.
struct CacheArgs {
  char *k, *v;
  int64_t layer_stride, block_stride, token_stride, head_stride;
  int32_t layers, blocks, block_size, kv_heads, head_dim, dtype;
};

struct BatchArgs {
  const int32_t *tables, *seq_len, *row_start;
  int32_t S, T, rows, max_new, group;
};

inline int dtype_bytes(int dtype) { return dtype == SMC_F32 ? 4 : 2; }

struct QkArgs {
  CacheArgs c;
  BatchArgs b;
  const char *q, *k, *v;
  const char *qw, *kw;
  const int32_t *positions;
  const float *rope;
  char *out;
  int32_t q_heads, rot, max_pos, interleaved;
  float eps, w0;
  int64_t q_row, q_head, k_row, k_head, v_row, v_head, o_row, o_head;
  unsigned *status;
};

struct AttnArgs {
  CacheArgs c;
  BatchArgs b;
  const char *q;
  const uint32_t *mask;
  char *out;
  float *lse;
  int32_t q_heads, mask_words;
  float scale;
  int64_t q_row, q_head, o_row, o_head;
  unsigned *status;
};

// Launches with programmatic stream serialisation: a kernel's CTAs may start
// while the kernel ahead of it in the stream drains, and wait for it in full
// (wait_for_stream) before they touch global memory.  About 3 us of a small
// attention call that follows another.
cudaError_t launch_early(const void *fn, dim3 grid, unsigned block, size_t dyn, void **args,
                         cudaStream_t st);

// Workspace of the cache entry points: the status word first (256 bytes).
constexpr size_t kCacheStatusBytes = 256;
size_t attention_workspace_bytes(const CacheArgs &c, const BatchArgs &b, int q_heads);

cudaError_t launch_tree_attention(const AttnArgs &a, void *workspace, cudaStream_t st);
cudaError_t launch_qk_norm_rope(const QkArgs &a, cudaStream_t st);
cudaError_t launch_copy_blocks(const CacheArgs &c, const int32_t *pairs, const int32_t *counts,
                               int lists, int max_pairs, unsigned *status, cudaStream_t st);
cudaError_t launch_compact_tokens(const CacheArgs &c, const BatchArgs &b, const int32_t *path,
                                  const int32_t *n_path, int max_path, unsigned *status,
                                  cudaStream_t st);
cudaError_t launch_kv_truncate(int B, int N, const KvArgs &kv, const int32_t *new_len,
                               const Workspace &ws, cudaStream_t st);

}  // namespace smcsd

// Attention of each sequence's new tokens over its paged cache, under a tree
// mask (smc_tree_attention in smcsd.h).
#include "cache_common.cuh"

namespace smcsd {

constexpr int kAttnThreads = 256;

// One warp per (row, head): the online softmax, a token at a time.
template <typename T>
__global__ void __launch_bounds__(kAttnThreads) tree_attention_kernel(const AttnArgs a) {
  const int64_t unit = static_cast<int64_t>(blockIdx.x) * (kAttnThreads / 32) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (unit >= static_cast<int64_t>(a.b.rows) * a.q_heads) return;
  const int row = static_cast<int>(unit / a.q_heads), h = static_cast<int>(unit % a.q_heads);
  const int s = seq_of_row(a.b, row);
  if (s < 0) return;
  const SeqInfo si = seq_info(a.b, a.c.block_size, s);
  const int i = row - si.row0;
  if (i < 0 || i >= si.n) {
    if (lane == 0 && si.bits) raise_status(a.status, si.bits);
    return;
  }
  const int D = a.c.head_dim;
  const T *q = reinterpret_cast<const T *>(a.q) + row * a.q_row + h * a.q_head;
  float qv[4], acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int e = 0; e < 4; ++e) qv[e] = lane + 32 * e < D ? to_f32(q[lane + 32 * e]) : 0.f;
  const int kh = h / (a.q_heads / a.c.kv_heads);
  const int32_t *table = a.b.tables + static_cast<int64_t>(s) * a.b.T;
  const int ctx = si.len - si.n;
  float m = -INFINITY, l = 0.f;
  for (int t = 0; t < si.len; ++t) {
    if (t >= ctx) {
      const int j = t - ctx;
      bool sees = j <= i;
      if (a.mask) {
        sees = (j >> 5) < a.mask_words &&
               (a.mask[static_cast<int64_t>(row) * a.mask_words + (j >> 5)] >> (j & 31) & 1u);
      }
      if (!sees) continue;
    }
    const int block = table[t / a.c.block_size];
    if (block < 0 || block >= a.c.blocks) {
      if (lane == 0) raise_status(a.status, SMC_DEV_BAD_BLOCK);
      continue;
    }
    const int64_t off = block * a.c.block_stride + (t % a.c.block_size) * a.c.token_stride +
                        kh * a.c.head_stride;
    const T *k = reinterpret_cast<const T *>(a.c.k) + off;
    const T *v = reinterpret_cast<const T *>(a.c.v) + off;
    float z = 0.f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (lane + 32 * e < D) z = fmaf(qv[e], to_f32(k[lane + 32 * e]), z);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
    z *= a.scale;
    const float mn = fmaxf(m, z);
    const float f = m == -INFINITY ? 0.f : __expf(m - mn), p = mn == -INFINITY ? 0.f : __expf(z - mn);
    l = l * f + p;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (lane + 32 * e < D) acc[e] = fmaf(p, to_f32(v[lane + 32 * e]), acc[e] * f);
    }
    m = mn;
  }
  T *out = reinterpret_cast<T *>(a.out) + row * a.o_row + h * a.o_head;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (lane + 32 * e < D) out[lane + 32 * e] = from_f32<T>(l == 0.f ? 0.f : acc[e] / l);
  }
  if (a.lse && lane == 0) a.lse[unit] = l == 0.f ? -INFINITY : m + logf(l);
}

size_t attention_workspace_bytes(const CacheArgs &, const BatchArgs &, int) {
  return kCacheStatusBytes;
}

cudaError_t launch_tree_attention(const AttnArgs &a, void *, cudaStream_t st) {
  const int64_t units = static_cast<int64_t>(a.b.rows) * a.q_heads;
  if (units == 0) return cudaSuccess;
  const unsigned grid = static_cast<unsigned>((units + kAttnThreads / 32 - 1) / (kAttnThreads / 32));
  if (a.c.dtype == SMC_BF16) tree_attention_kernel<__nv_bfloat16><<<grid, kAttnThreads, 0, st>>>(a);
  else tree_attention_kernel<__half><<<grid, kAttnThreads, 0, st>>>(a);
  return cudaGetLastError();
}

}  // namespace smcsd

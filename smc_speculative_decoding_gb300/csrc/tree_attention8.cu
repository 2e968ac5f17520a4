// Attention of each sequence's new tokens over its paged 8-bit cache, under a
// tree mask (smc_tree_attention8 in smcsd.h).
#include "cache_common.cuh"

namespace smcsd {

size_t attention8_workspace_bytes(const CacheArgs &, const BatchArgs &, int) { return kCacheStatusBytes; }

constexpr int kThreads8 = 128;
constexpr int kWarps8 = kThreads8 / 32;

// A CTA takes one row of one query head; its warps every fourth token, each
// with a running maximum, sum and accumulator, joined at the end.
template <typename T>
__global__ void __launch_bounds__(kThreads8)
attention8_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ ScaleArgs sc) {
  __shared__ float s_m[kWarps8], s_l[kWarps8], s_o[kWarps8][128];
  const int row = blockIdx.x, qh = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int D = a.c.head_dim, bs = a.c.block_size, h = qh / (a.q_heads / a.c.kv_heads);
  wait_for_stream();
  const int s = seq_of_row(a.b, row);
  if (s < 0 || s >= a.b.S) return;
  const SeqInfo si = seq_info(a.b, bs, s);
  const int i = row - si.row0;
  if (i < 0 || i >= si.n) {
    if (si.bits && threadIdx.x == 0) raise_status(a.status, si.bits);
    return;
  }
  const T *q = reinterpret_cast<const T *>(a.q) + row * a.q_row + qh * a.q_head;
  float x[4], o[4] = {0.f, 0.f, 0.f, 0.f}, m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e) x[e] = 4 * lane + e < D ? to_f32(q[4 * lane + e]) : 0.f;
  const int32_t *table = a.b.tables + static_cast<int64_t>(s) * a.b.T;
  const uint32_t *mask = a.mask ? a.mask + static_cast<int64_t>(row) * a.mask_words : nullptr;
  for (int t = warp; t < si.len; t += kWarps8) {
    const int j = t - (si.len - si.n);
    if (j >= 0 && (mask ? j / 32 >= a.mask_words || !(mask[j / 32] >> (j % 32) & 1u) : j > i)) continue;
    const int block = table[t / bs];
    if (block < 0 || block >= a.c.blocks) {
      if (lane == 0) raise_status(a.status, SMC_DEV_BAD_BLOCK);
      continue;
    }
    const int64_t at = block * a.c.block_stride + (t % bs) * a.c.token_stride + h * a.c.head_stride + 4 * lane;
    float k[4] = {0.f, 0.f, 0.f, 0.f}, v[4] = {0.f, 0.f, 0.f, 0.f};
    if (4 * lane < D) {
      const uint32_t kb = *reinterpret_cast<const uint32_t *>(a.c.k + at), vb = *reinterpret_cast<const uint32_t *>(a.c.v + at);
#pragma unroll
      for (int e = 0; e < 4; e += 2) {
        const uint32_t kh = from_e4m3x2(kb >> (8 * e)), vh = from_e4m3x2(vb >> (8 * e));
        const float2 kf = __half22float2(*reinterpret_cast<const __half2 *>(&kh));
        const float2 vf = __half22float2(*reinterpret_cast<const __half2 *>(&vh));
        k[e] = kf.x; k[e + 1] = kf.y;
        v[e] = vf.x; v[e + 1] = vf.y;
      }
    }
    const float ks = scale_of(sc.k[block * sc.block + h * sc.head]), vs = scale_of(sc.v[block * sc.block + h * sc.head]);
    float z = x[0] * k[0] + x[1] * k[1] + x[2] * k[2] + x[3] * k[3];
#pragma unroll
    for (int step = 16; step > 0; step >>= 1) z += __shfl_xor_sync(0xffffffffu, z, step);
    z *= a.scale * ks;
    const float top = fmaxf(m, z), f = m == -INFINITY ? 0.f : expf(m - top), w = expf(z - top);
    m = top;
    l = l * f + w;
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = o[e] * f + w * vs * v[e];
  }
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) s_o[warp][4 * lane + e] = o[e];
  __syncthreads();
  float top = s_m[0], sum = 0.f, r = 0.f;
  for (int w = 1; w < kWarps8; ++w) top = fmaxf(top, s_m[w]);
  const int d = threadIdx.x;
  for (int w = 0; w < kWarps8; ++w) {
    if (s_m[w] == -INFINITY && s_l[w] == 0.f) continue;
    const float f = expf(s_m[w] - top);
    sum += f * s_l[w];
    r += f * s_o[w][d];
  }
  if (d < D) {
    reinterpret_cast<T *>(a.out)[row * a.o_row + qh * a.o_head + d] = from_f32<T>(sum == 0.f ? 0.f : r / sum);
  }
  if (a.lse && d == 0) {
    a.lse[static_cast<int64_t>(row) * a.q_heads + qh] = sum == 0.f ? -INFINITY : top + logf(sum);
  }
}

cudaError_t launch_tree_attention8(const AttnArgs &a, const ScaleArgs &s, int dtype, void *, cudaStream_t st) {
  if (a.b.rows == 0) return cudaSuccess;
  ScaleArgs scales = s;
  void *args[] = {const_cast<AttnArgs *>(&a), &scales};
  return launch_early(dtype == SMC_BF16 ? reinterpret_cast<const void *>(attention8_kernel<__nv_bfloat16>)
                                        : reinterpret_cast<const void *>(attention8_kernel<__half>),
                      dim3(a.b.rows, a.q_heads), kThreads8, 0, args, st);
}

}  // namespace smcsd

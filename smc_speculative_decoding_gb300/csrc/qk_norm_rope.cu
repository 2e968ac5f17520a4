// Per-head RMS norms of queries and keys, the position rotation, and the write
// of keys and values into the cache's blocks (smc_qk_norm_rope in smcsd.h).
#include "cache_common.cuh"

namespace smcsd {

constexpr int kQkThreads = 256;
constexpr int kQkMaxPerLane = 8;  // head_dim <= 256 over 32 lanes

// One CTA per row; a warp per head, each lane elements lane, lane + 32, ...
template <typename T>
__global__ void __launch_bounds__(kQkThreads) qk_rows_kernel(const QkArgs a) {
  const int row = blockIdx.x;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int s = seq_of_row(a.b, row);
  if (s < 0) return;
  const SeqInfo si = seq_info(a.b, a.c.block_size, s);
  const int i = row - si.row0;
  if (i < 0 || i >= si.n) {
    if (threadIdx.x == 0 && si.bits) raise_status(a.status, si.bits);
    return;
  }
  const int at = si.len - si.n + i;
  const int block = a.b.tables[static_cast<int64_t>(s) * a.b.T + at / a.c.block_size];
  const int pos = a.positions ? a.positions[row] : at;
  unsigned bits = 0;
  if (block < 0 || block >= a.c.blocks) bits |= SMC_DEV_BAD_BLOCK;
  if (pos < 0 || pos >= a.max_pos) bits |= SMC_DEV_BAD_ROWS;
  if (bits) {
    if (threadIdx.x == 0) raise_status(a.status, bits);
    return;
  }
  const int D = a.c.head_dim, Hk = a.c.kv_heads, half = a.rot / 2;
  const int64_t slot = block * a.c.block_stride + (at % a.c.block_size) * a.c.token_stride;
  const float *cs = a.rope + static_cast<int64_t>(pos) * a.rot;
  for (int h = warp; h < a.q_heads + 2 * Hk; h += kQkThreads / 32) {
    const T *src;
    T *dst;
    const T *w = nullptr;
    bool value = false;
    if (h < a.q_heads) {
      src = reinterpret_cast<const T *>(a.q) + row * a.q_row + h * a.q_head;
      dst = reinterpret_cast<T *>(a.out) + row * a.o_row + h * a.o_head;
      w = reinterpret_cast<const T *>(a.qw);
    } else if (h < a.q_heads + Hk) {
      const int g = h - a.q_heads;
      src = reinterpret_cast<const T *>(a.k) + row * a.k_row + g * a.k_head;
      dst = reinterpret_cast<T *>(a.c.k) + slot + g * a.c.head_stride;
      w = reinterpret_cast<const T *>(a.kw);
    } else {
      const int g = h - a.q_heads - Hk;
      src = reinterpret_cast<const T *>(a.v) + row * a.v_row + g * a.v_head;
      dst = reinterpret_cast<T *>(a.c.v) + slot + g * a.c.head_stride;
      value = true;
    }
    T raw[kQkMaxPerLane], out[kQkMaxPerLane];
    float sum = 0.f;
#pragma unroll
    for (int e = 0; e < kQkMaxPerLane; ++e) {
      const int d = lane + 32 * e;
      if (d < D) {
        raw[e] = src[d];
        const float x = to_f32(raw[e]);
        sum = fmaf(x, x, sum);
      }
    }
    if (value) {
#pragma unroll
      for (int e = 0; e < kQkMaxPerLane; ++e) {
        if (lane + 32 * e < D) dst[lane + 32 * e] = raw[e];
      }
      continue;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const float r = w ? rsqrtf(sum / D + a.eps) : 1.f;
    auto normed = [&](int d) {
      const float x = to_f32(src[d]) * r;
      return w ? x * (to_f32(w[d]) + a.w0) : x;
    };
#pragma unroll
    for (int e = 0; e < kQkMaxPerLane; ++e) {
      const int d = lane + 32 * e;
      if (d >= D) continue;
      float y = normed(d);
      if (d < a.rot) {
        const bool second = a.interleaved ? (d & 1) : d >= half;
        const int j = a.interleaved ? d >> 1 : (second ? d - half : d);
        const int other = a.interleaved ? d ^ 1 : (second ? d - half : d + half);
        const float z = normed(other), c = cs[j], sn = cs[half + j];
        y = second ? fmaf(z, sn, y * c) : fmaf(-z, sn, y * c);
      }
      out[e] = from_f32<T>(y);
    }
    __syncwarp();  // q_out may be q: every lane has read its pairs
#pragma unroll
    for (int e = 0; e < kQkMaxPerLane; ++e) {
      if (lane + 32 * e < D) dst[lane + 32 * e] = out[e];
    }
  }
}

cudaError_t launch_qk_norm_rope(const QkArgs &a, cudaStream_t st) {
  if (a.b.rows == 0) return cudaSuccess;
  switch (a.c.dtype) {
    case SMC_F32: qk_rows_kernel<float><<<a.b.rows, kQkThreads, 0, st>>>(a); break;
    case SMC_BF16: qk_rows_kernel<__nv_bfloat16><<<a.b.rows, kQkThreads, 0, st>>>(a); break;
    default: qk_rows_kernel<__half><<<a.b.rows, kQkThreads, 0, st>>>(a); break;
  }
  return cudaGetLastError();
}

}  // namespace smcsd

// Per-head RMS norms of queries and keys, the position rotation, and the write
// of keys and values into an 8-bit cache (smc_qk_norm_rope8 in smcsd.h).
#include "cache_common.cuh"

namespace smcsd {

constexpr int kThreads8 = 256;
constexpr int kWarps8 = kThreads8 / 32;

// Work: a *run* is the new tokens of one sequence that lie in one block; its
// keys and values of one head share a scale.  CTA (x, h) takes the runs that
// begin in rows [x * per, (x + 1) * per): for each, key head h's keys and
// values, and the query heads h, h + kv_heads, ...
struct Run {
  int row, n;      // rows [row, row + n)
  int seq, at;     // the first one's place in its table
};

// The first run that begins at row `r` or later and before `end`; n = 0: none.
__device__ __forceinline__ Run next_run(const QkArgs &a, int r, int end) {
  const int bs = a.c.block_size;
  while (r < end) {
    const int s = seq_of_row(a.b, r);
    if (s < 0 || s >= a.b.S) break;  // rows past the last sequence
    const SeqInfo si = seq_info(a.b, bs, s);
    const int i = r - si.row0;
    if (i < 0 || i >= si.n) {
      if (si.bits && blockIdx.y == 0 && threadIdx.x == 0) raise_status(a.status, si.bits);
      ++r;
      continue;
    }
    const int at = si.len - si.n + i, off = at % bs, n = min(bs - off, si.n - i);
    if (i == 0 || off == 0) return {r, n, s, at};
    r += n;
  }
  return {0, 0, 0, 0};
}

// Element d of a vector after norm (r = rsqrt of the mean square) and rotation.
template <typename T>
__device__ __forceinline__ float turned(const QkArgs &a, const T *src, const T *w, float r, const float *cs, int d) {
  auto normed = [&](int e) {
    const float x = to_f32(src[e]) * r;
    return w ? x * (to_f32(w[e]) + a.w0) : x;
  };
  const float y = normed(d);
  if (d >= a.rot) return y;
  const int half = a.rot / 2;
  const bool second = a.interleaved ? (d & 1) : d >= half;
  const int j = a.interleaved ? d >> 1 : (second ? d - half : d);
  const float z = normed(a.interleaved ? d ^ 1 : (second ? d - half : d + half));
  return second ? fmaf(z, cs[half + j], y * cs[j]) : fmaf(-z, cs[half + j], y * cs[j]);
}

// rsqrt(mean(x^2) + eps) of a vector, or 1 without weights: a warp's lanes.
template <typename T>
__device__ __forceinline__ float norm_of(const QkArgs &a, const T *src, const T *w) {
  if (!w) return 1.f;
  float sum = 0.f;
  for (int d = threadIdx.x & 31; d < a.c.head_dim; d += 32) {
    const float x = to_f32(src[d]);
    sum = fmaf(x, x, sum);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return rsqrtf(sum / a.c.head_dim + a.eps);
}

// Any sizes, strides and alignment: a warp per vector, each lane elements lane,
// lane + 32, ...; keys are computed for the block's scale and again to be stored.
template <typename T>
__global__ void __launch_bounds__(kThreads8)
append8_kernel(const __grid_constant__ QkArgs a, const __grid_constant__ ScaleArgs sc, int per) {
  __shared__ int s_top[2];
  __shared__ float s_old[2], s_new[2];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, h = blockIdx.y;
  const int bs = a.c.block_size, D = a.c.head_dim;
  wait_for_stream();
  const int r0 = blockIdx.x * per, end = min(r0 + per, a.b.rows);
  for (Run run = next_run(a, r0, end); run.n > 0; run = next_run(a, run.row + run.n, end)) {
    const int block = a.b.tables[static_cast<int64_t>(run.seq) * a.b.T + run.at / bs], off = run.at % bs;
    if (block < 0 || block >= a.c.blocks) {
      if (h == 0 && tid == 0) raise_status(a.status, SMC_DEV_BAD_BLOCK);
      continue;
    }
    auto position = [&](int i) {
      const int p = a.positions ? a.positions[run.row + i] : run.at + i;
      return p >= 0 && p < a.max_pos ? p : -1;
    };
    auto key = [&](int i) { return reinterpret_cast<const T *>(a.k) + (run.row + i) * a.k_row + h * a.k_head; };
    auto value = [&](int i) { return reinterpret_cast<const T *>(a.v) + (run.row + i) * a.v_row + h * a.v_head; };
    const T *kw = reinterpret_cast<const T *>(a.kw), *qw = reinterpret_cast<const T *>(a.qw);
    __syncthreads();
    if (tid < 2) s_top[tid] = 0;
    __syncthreads();
    float top_k = 0.f, top_v = 0.f;
    for (int i = warp; i < run.n; i += kWarps8) {
      const int pos = position(i);
      if (pos < 0) {
        if (h == 0 && lane == 0) raise_status(a.status, SMC_DEV_BAD_ROWS);
        continue;
      }
      const float *cs = a.rope + static_cast<int64_t>(pos) * a.rot;
      const float r = norm_of(a, key(i), kw);
      for (int d = lane; d < D; d += 32) {
        const float y = fabsf(turned(a, key(i), kw, r, cs, d)), v = fabsf(to_f32(value(i)[d]));
        if (y < INFINITY) top_k = fmaxf(top_k, y);
        if (v < INFINITY) top_v = fmaxf(top_v, v);
      }
    }
    atomicMax(&s_top[0], __float_as_int(top_k));  // of positive numbers: their bits' order
    atomicMax(&s_top[1], __float_as_int(top_v));
    __syncthreads();
    if (tid < 2) {
      float *at = (tid ? sc.v : sc.k) + block * sc.block + h * sc.head;
      const float need = least_scale(__int_as_float(s_top[tid]));
      s_old[tid] = off ? scale_of(*at) : need;
      s_new[tid] = fmaxf(need, s_old[tid]);
      *at = s_new[tid];
    }
    __syncthreads();
    uint8_t *const k0 = reinterpret_cast<uint8_t *>(a.c.k) + block * a.c.block_stride + h * a.c.head_stride;
    uint8_t *const v0 = reinterpret_cast<uint8_t *>(a.c.v) + block * a.c.block_stride + h * a.c.head_stride;
    for (int which = 0; which < 2; ++which) {  // tokens ahead of the new ones
      const float f = s_old[which] / s_new[which];
      if (f == 1.f) continue;
      for (int t = warp; t < off; t += kWarps8) {
        uint8_t *x = (which ? v0 : k0) + t * a.c.token_stride;
        for (int d = lane; d < D; d += 32) x[d] = static_cast<uint8_t>(rescale_e4m3x4(x[d], f));
      }
    }
    for (int i = warp; i < run.n; i += kWarps8) {
      const int pos = position(i);
      if (pos < 0) continue;
      const float *cs = a.rope + static_cast<int64_t>(pos) * a.rot;
      const float r = norm_of(a, key(i), kw);
      const int64_t token = (off + i) * a.c.token_stride;
      for (int d = lane; d < D; d += 32) {
        const float y = finite_or_nan(turned(a, key(i), kw, r, cs, d));
        k0[token + d] = static_cast<uint8_t>(to_e4m3x2(y / s_new[0], 0.f));
        v0[token + d] = static_cast<uint8_t>(to_e4m3x2(finite_or_nan(to_f32(value(i)[d])) / s_new[1], 0.f));
      }
      for (int g = h; g < a.q_heads; g += a.c.kv_heads) {
        const T *src = reinterpret_cast<const T *>(a.q) + (run.row + i) * a.q_row + g * a.q_head;
        T *dst = reinterpret_cast<T *>(a.out) + (run.row + i) * a.o_row + g * a.o_head;
        const float rq = norm_of(a, src, qw);
        T out[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (lane + 32 * e < D) out[e] = from_f32<T>(turned(a, src, qw, rq, cs, lane + 32 * e));
        }
        __syncwarp();  // q_out may be q: every lane has read its pairs
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (lane + 32 * e < D) dst[lane + 32 * e] = out[e];
        }
        __syncwarp();
      }
    }
  }
}

cudaError_t launch_qk_norm_rope8(const QkArgs &a, const ScaleArgs &s, int dtype, cudaStream_t st) {
  if (a.b.rows == 0) return cudaSuccess;
  int per = a.c.block_size < a.b.max_new ? a.c.block_size : a.b.max_new;
  ScaleArgs scales = s;
  const void *fn = dtype == SMC_F32    ? reinterpret_cast<const void *>(append8_kernel<float>)
                   : dtype == SMC_BF16 ? reinterpret_cast<const void *>(append8_kernel<__nv_bfloat16>)
                                       : reinterpret_cast<const void *>(append8_kernel<__half>);
  void *args[] = {const_cast<QkArgs *>(&a), &scales, &per};
  return launch_early(fn, dim3((a.b.rows + per - 1) / per, a.c.kv_heads), kThreads8, 0, args, st);
}

}  // namespace smcsd

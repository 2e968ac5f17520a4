// Per-head RMS norms of queries and keys, the position rotation, and the write
// of keys and values into the cache's blocks (smc_qk_norm_rope in smcsd.h).
#include "qk_turn.cuh"

namespace smcsd {

constexpr int kQkThreads = 64;
constexpr int kQkMaxPerLane = 8;  // head_dim <= 256 over 32 lanes

// Any sizes, strides and alignment: one CTA per row; a warp per head, each lane
// elements lane, lane + 32, ...
template <typename T>
__global__ void __launch_bounds__(kQkThreads) qk_rows_kernel(const __grid_constant__ QkArgs a) {
  const int row = blockIdx.x;
  wait_for_stream();
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

// The same with 16-byte accesses.  A head is a group of kLanes lanes with one
// vector each; a CTA takes a row.  With y the dims that x's turn with,
//   out = r (x (w cos) + y (w' (-+ sin))),  w' the weights of y,
// so a lane folds the weights and signs into its dims' angles once a row, and a
// head costs two packed products, one packed sum and the scaling by
// r = rsqrt(mean(x^2) + eps) per pair of dims.  The first heads' loads are
// under way before the row's place in the cache and its angles are known: for
// one row the time is two dependent loads, for many the bytes'.
//   Measured, 12 535 rows of 56 heads of 96 in fp16 (309 MB): scalar arithmetic
// with run-time selects 138 us, bound by the instructions issued (389 per
// vector and warp); this form 102 us with 256 threads a row, 75 us with 128, 66
// with 64, and 63 since (4.9 TB/s): what a warp does once a row is shared by more heads.
constexpr int kAhead = 4;  // q heads of a group whose loads are under way at once

template <typename T, int kLanes, bool kInter>
__global__ void __launch_bounds__(kQkThreads, 16) qk_vectors_kernel(const __grid_constant__ QkArgs a) {
  const int row = blockIdx.x;
  const int group = threadIdx.x / kLanes, vec = threadIdx.x % kLanes, groups = blockDim.x / kLanes;
  const int Hk = a.c.kv_heads;
  Turn<T, kLanes, kInter> turn;
  turn.place(a);
  const bool has = turn.has;
  auto at_head = [&](const char *base, int64_t row_stride, int64_t head_stride, int h) {
    return base + (row * row_stride + h * head_stride) * static_cast<int64_t>(sizeof(T)) + vec * 16;
  };
  auto fetch = [&](const char *base, int64_t row_stride, int64_t head_stride, int heads, int h) {
    return has && h < heads ? *reinterpret_cast<const uint4 *>(at_head(base, row_stride, head_stride, h))
                            : make_uint4(0, 0, 0, 0);
  };
  // k's heads start at the first group, v's at the last one
  const int v0 = groups - 1 - group;
  wait_for_stream();
  uint4 rq[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i) rq[i] = fetch(a.q, a.q_row, a.q_head, a.q_heads, group + i * groups);
  uint4 rk = fetch(a.k, a.k_row, a.k_head, Hk, group), rv = fetch(a.v, a.v_row, a.v_head, Hk, v0);
  // The row's sequence is the guessed one when every sequence has max_new rows
  // (else it is searched for).  What the guess needs is loaded in one go; its
  // block and the angles are the second dependent load.
  int s = min(row / a.b.max_new, a.b.S - 1);
  int pos = a.positions ? a.positions[row] : 0;
  SeqInfo si = seq_info(a.b, a.c.block_size, s);
  if (row < si.row0 || row >= si.row0 + si.n) {
    s = a.b.row_start ? seq_of_row(a.b, row) : -1;
    if (s >= 0) si = seq_info(a.b, a.c.block_size, s);
    if (s < 0 || row < si.row0 || row >= si.row0 + si.n) {
      if (threadIdx.x == 0 && si.bits) raise_status(a.status, si.bits);
      return;
    }
  }
  const int at = si.len - si.n + row - si.row0;
  if (!a.positions) pos = at;
  const int block = a.b.tables[static_cast<int64_t>(s) * a.b.T + at / a.c.block_size];
  if (pos < 0 || pos >= a.max_pos) {
    if (threadIdx.x == 0) raise_status(a.status, SMC_DEV_BAD_ROWS);
    return;
  }
  const float *table = a.rope + static_cast<int64_t>(pos) * a.rot;
  turn.load(a, table, a.qw);
  if (block < 0 || block >= a.c.blocks) {
    if (threadIdx.x == 0) raise_status(a.status, SMC_DEV_BAD_BLOCK);
    return;
  }
  const float inv_dim = 1.f / a.c.head_dim;
  for (int i0 = 0; i0 * groups < a.q_heads; i0 += kAhead) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if ((i0 + i) * groups >= a.q_heads) break;  // for the whole CTA
      const int h = group + (i0 + i) * groups;
      const uint4 z = turn.apply(rq[i], a.qw != nullptr, inv_dim, a.eps);
      if (has && h < a.q_heads) {
        *reinterpret_cast<uint4 *>(const_cast<char *>(at_head(a.out, a.o_row, a.o_head, h))) = z;
      }
    }
    if ((i0 + kAhead) * groups < a.q_heads) {
#pragma unroll
      for (int i = 0; i < kAhead; ++i) {
        rq[i] = fetch(a.q, a.q_row, a.q_head, a.q_heads, group + (i0 + kAhead + i) * groups);
      }
    }
  }
  const int64_t slot = block * a.c.block_stride + (at % a.c.block_size) * a.c.token_stride;
  auto in_cache = [&](char *base, int h) {
    return reinterpret_cast<uint4 *>(base + (slot + h * a.c.head_stride) * static_cast<int64_t>(sizeof(T)) + vec * 16);
  };
  turn.load(a, table, a.kw);
  for (int h0 = 0; h0 < Hk; h0 += groups) {
    const int hk = group + h0, hv = v0 + h0;
    const uint4 z = turn.apply(rk, a.kw != nullptr, inv_dim, a.eps);
    if (has && hk < Hk) *in_cache(a.c.k, hk) = z;
    if (has && hv < Hk) *in_cache(a.c.v, hv) = rv;
    if (h0 + groups < Hk) {
      rk = fetch(a.k, a.k_row, a.k_head, Hk, hk + groups);
      rv = fetch(a.v, a.v_row, a.v_head, Hk, hv + groups);
    }
  }
}

// Whether every address is a multiple of 16 bytes and every vector turns as a
// whole.
static bool vectors_ok(const QkArgs &a) {
  const int esz = dtype_bytes(a.c.dtype), E = 16 / esz;
  uint64_t all = reinterpret_cast<uintptr_t>(a.q) | reinterpret_cast<uintptr_t>(a.k) |
                 reinterpret_cast<uintptr_t>(a.v) | reinterpret_cast<uintptr_t>(a.out) |
                 reinterpret_cast<uintptr_t>(a.c.k) | reinterpret_cast<uintptr_t>(a.c.v) |
                 reinterpret_cast<uintptr_t>(a.qw) | reinterpret_cast<uintptr_t>(a.kw) |
                 reinterpret_cast<uintptr_t>(a.rope);
  const int rows = a.b.rows, Hk = a.c.kv_heads;
  auto stride = [&](int64_t s, int n) { if (n > 1) all |= static_cast<uint64_t>(s) * esz; };
  stride(a.q_row, rows); stride(a.k_row, rows); stride(a.v_row, rows); stride(a.o_row, rows);
  stride(a.q_head, a.q_heads); stride(a.o_head, a.q_heads);
  stride(a.k_head, Hk); stride(a.v_head, Hk);
  stride(a.c.head_stride, Hk); stride(a.c.token_stride, a.c.block_size); stride(a.c.block_stride, a.c.blocks);
  return all % 16 == 0 && a.c.head_dim % E == 0 && a.c.head_dim <= 32 * E && a.rot % E == 0 &&
         (a.interleaved || a.rot / 2 % E == 0);
}

template <typename T, bool kInter>
static cudaError_t launch_vectors(const QkArgs &a, cudaStream_t st) {
  const int vectors = a.c.head_dim * static_cast<int>(sizeof(T)) / 16, heads = a.q_heads + 2 * a.c.kv_heads;
  const int lanes = vectors <= 8 ? 8 : vectors <= 16 ? 16 : 32;
  // no more threads than heads to start on
  const int threads = heads * lanes < kQkThreads ? (heads * lanes + 31) / 32 * 32 : kQkThreads;
  const void *fn = lanes == 8    ? reinterpret_cast<const void *>(qk_vectors_kernel<T, 8, kInter>)
                   : lanes == 16 ? reinterpret_cast<const void *>(qk_vectors_kernel<T, 16, kInter>)
                                 : reinterpret_cast<const void *>(qk_vectors_kernel<T, 32, kInter>);
  void *args[] = {const_cast<QkArgs *>(&a)};
  return launch_early(fn, dim3(a.b.rows), threads, 0, args, st);
}

cudaError_t launch_qk_norm_rope(const QkArgs &a, cudaStream_t st) {
  if (a.b.rows == 0) return cudaSuccess;
  if (vectors_ok(a)) {
    switch (a.c.dtype) {
      case SMC_F32: return a.interleaved ? launch_vectors<float, true>(a, st) : launch_vectors<float, false>(a, st);
      case SMC_BF16:
        return a.interleaved ? launch_vectors<__nv_bfloat16, true>(a, st) : launch_vectors<__nv_bfloat16, false>(a, st);
      default: return a.interleaved ? launch_vectors<__half, true>(a, st) : launch_vectors<__half, false>(a, st);
    }
  }
  const void *fn = a.c.dtype == SMC_F32    ? reinterpret_cast<const void *>(qk_rows_kernel<float>)
                   : a.c.dtype == SMC_BF16 ? reinterpret_cast<const void *>(qk_rows_kernel<__nv_bfloat16>)
                                           : reinterpret_cast<const void *>(qk_rows_kernel<__half>);
  void *args[] = {const_cast<QkArgs *>(&a)};
  return launch_early(fn, dim3(a.b.rows), kQkThreads, 0, args, st);
}

}  // namespace smcsd

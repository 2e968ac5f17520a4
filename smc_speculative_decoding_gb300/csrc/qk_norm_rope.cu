// Per-head RMS norms of queries and keys, the position rotation, and the write
// of keys and values into the cache's blocks (smc_qk_norm_rope in smcsd.h).
#include "cache_common.cuh"

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

template <typename T>
__device__ __forceinline__ void unpack16(const uint4 &v, float *x) {
  const T *e = reinterpret_cast<const T *>(&v);
#pragma unroll
  for (int i = 0; i < static_cast<int>(16 / sizeof(T)); ++i) x[i] = to_f32(e[i]);
}
template <>
__device__ __forceinline__ void unpack16<__nv_bfloat16>(const uint4 &v, float *x) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(w[i] << 16);
    x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
template <typename T>
__device__ __forceinline__ uint4 pack16(const float *x);
template <>
__device__ __forceinline__ uint4 pack16<float>(const float *x) {
  return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
}
template <>
__device__ __forceinline__ uint4 pack16<__nv_bfloat16>(const float *x) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
template <>
__device__ __forceinline__ uint4 pack16<__half>(const float *x) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(x[2 * i + 1]), "f"(x[2 * i]));
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// A lane's dims of a row: the vector it holds, its partner lane, and the
// factors of x and of y.
template <typename T, int kLanes, bool kInter>
struct Turn {
  static constexpr int E = 16 / sizeof(T);
  unsigned long long cw[E / 2], sw[E / 2];
  bool has, turns, second;
  int other;  // lane of the warp whose vector holds the partners

  __device__ __forceinline__ void place(const QkArgs &a) {
    const int d0 = threadIdx.x % kLanes * E, half = a.rot / 2, lane = threadIdx.x & 31;
    has = d0 < a.c.head_dim;
    turns = has && d0 < a.rot;
    second = !kInter && d0 >= half;
    other = turns && !kInter ? lane + (second ? -half / E : half / E) : lane;
  }
  __device__ __forceinline__ void load(const QkArgs &a, const float *table, const char *weight) {
    const int vec = threadIdx.x % kLanes, d0 = vec * E, half = a.rot / 2;
    float c[E], n[E], w[E], wy[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      c[e] = w[e] = wy[e] = 1.f;
      n[e] = 0.f;
    }
    if (turns) {
      if (kInter) {
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          c[e] = c[e + 1] = table[(d0 + e) / 2];
          n[e + 1] = table[half + (d0 + e) / 2];
          n[e] = -n[e + 1];
        }
      } else {
        const float4 *c4 = reinterpret_cast<const float4 *>(table + (second ? d0 - half : d0));
#pragma unroll
        for (int e = 0; e < E; e += 4) {
          const float4 x = c4[e / 4], y = c4[half / 4 + e / 4];
          c[e] = x.x; c[e + 1] = x.y; c[e + 2] = x.z; c[e + 3] = x.w;
          n[e] = y.x; n[e + 1] = y.y; n[e + 2] = y.z; n[e + 3] = y.w;
        }
        if (!second) {
#pragma unroll
          for (int e = 0; e < E; ++e) n[e] = -n[e];
        }
      }
    }
    if (weight && has) {
      const uint4 *v = reinterpret_cast<const uint4 *>(weight);
      unpack16<T>(v[vec], w);
      unpack16<T>(v[kInter || !turns ? vec : vec + (second ? -half / E : half / E)], wy);
#pragma unroll
      for (int e = 0; e < E; ++e) {
        w[e] += a.w0;
        wy[e] += a.w0;
      }
    }
#pragma unroll
    for (int e = 0; e < E; e += 2) {
      cw[e / 2] = f2pack(c[e] * w[e], c[e + 1] * w[e + 1]);
      sw[e / 2] = kInter ? f2pack(n[e] * wy[e + 1], n[e + 1] * wy[e]) : f2pack(n[e] * wy[e], n[e + 1] * wy[e + 1]);
    }
  }
  // One head's vector, turned and (norm) scaled.  All lanes of the warp call it.
  __device__ __forceinline__ uint4 apply(const uint4 &raw, bool norm, float inv_dim, float eps) const {
    float x[E], z[E];
    unpack16<T>(raw, x);
    unsigned long long x2[E / 2], r2 = 0;
#pragma unroll
    for (int e = 0; e < E / 2; ++e) x2[e] = f2pack(x[2 * e], x[2 * e + 1]);
    if (norm) {
      unsigned long long sum2 = mul2(x2[0], x2[0]);
#pragma unroll
      for (int e = 1; e < E / 2; ++e) sum2 = fma2(x2[e], x2[e], sum2);
      float a, b;
      f2unpack(sum2, a, b);
      a += b;
#pragma unroll
      for (int o = kLanes / 2; o > 0; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o, kLanes);
      r2 = f2dup(rsqrtf(fmaf(a, inv_dim, eps)));
    }
#pragma unroll
    for (int e = 0; e < E / 2; ++e) {
      float ya, yb;
      if (kInter) {
        ya = x[2 * e + 1];
        yb = x[2 * e];
      } else {
        ya = __shfl_sync(0xffffffffu, x[2 * e], other);
        yb = __shfl_sync(0xffffffffu, x[2 * e + 1], other);
      }
      if (!turns) ya = yb = 0.f;  // an infinity there is no partner
      unsigned long long t = fma2(x2[e], cw[e], mul2(f2pack(ya, yb), sw[e]));
      if (norm) t = mul2(t, r2);
      f2unpack(t, z[2 * e], z[2 * e + 1]);
    }
    return pack16<T>(z);
  }
};

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

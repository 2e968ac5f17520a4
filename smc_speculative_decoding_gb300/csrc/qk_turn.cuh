// A vector of a head per lane: unpacking, packing, and the norm and rotation of
// qk_norm_rope.cu on it.
#pragma once

#include "cache_common.cuh"

namespace smcsd {

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

}  // namespace smcsd

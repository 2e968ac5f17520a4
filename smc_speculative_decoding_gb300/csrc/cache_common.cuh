// Device helpers shared by the cache kernels: a sequence's rows and tokens,
// checked, and the address of a token in its block.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "cache_ops.h"
#include "device_common.cuh"

namespace smcsd {

// The kernels ahead in the stream have ended and their writes are visible.
__device__ __forceinline__ void wait_for_stream() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <typename T>
__device__ __forceinline__ float to_f32(T x);
template <>
__device__ __forceinline__ float to_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ float to_f32<__half>(__half x) { return __half2float(x); }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 x) {
  return __bfloat162float(x);
}
// Rounded to nearest even.
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}

// Two numbers rounded to nearest even, a in the low half.
template <typename T>
__device__ __forceinline__ uint32_t pack2(float a, float b);
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float a, float b) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float a, float b) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
  return r;
}

// ---- 8 bits ----------------------------------------------------------------
constexpr float kLeastScale = 0x1p-100f, kMostScale = 0x1p100f;

// A stored scale as it counts: within [2^-100, 2^100], NaN as the least.
__device__ __forceinline__ float scale_of(float s) { return fminf(fmaxf(s, kLeastScale), kMostScale); }

// The least 2^t with top <= 448 * 2^t = 1.75 * 2^(t + 8), t within [-kRange, kRange]; top >= 0.
template <int kRange = 100>
__device__ __forceinline__ float least_scale(float top) {
  const uint32_t bits = __float_as_uint(top);
  const int t = static_cast<int>(bits >> 23) - 127 - ((bits & 0x7fffffu) <= 0x600000u ? 8 : 7);
  return __uint_as_float(static_cast<uint32_t>(min(max(t, -kRange), kRange) + 127) << 23);
}
// Two numbers to e4m3, a in the low byte: to nearest, ties to even; past 448
// to 448, NaN to NaN.
__device__ __forceinline__ uint32_t to_e4m3x2(float a, float b) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
  return r;
}
// Infinities are stored as NaN.
__device__ __forceinline__ float finite_or_nan(float x) {
  return fabsf(x) < INFINITY ? x : __uint_as_float(0x7fffffffu);
}
// Two e4m3 numbers (the low 16 bits) as fp16, exactly.
__device__ __forceinline__ uint32_t from_e4m3x2(uint32_t x) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(x)));
  return r;
}
// Four e4m3 numbers under another scale: each times f, rounded again.
__device__ __forceinline__ uint32_t rescale_e4m3x4(uint32_t x, float f) {
  uint32_t r = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint32_t h = from_e4m3x2(x >> (16 * i));
    const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&h));
    r |= to_e4m3x2(v.x * f, v.y * f) << (16 * i);
  }
  return r;
}

// A sequence's rows [row0, row0 + n) and the tokens it holds.  n = 0 and bits
// set when its offsets or its token count are out of range, so that a caller
// which honours n touches nothing outside the arrays.
struct SeqInfo {
  int row0, n, len;
  unsigned bits;
};

__device__ __forceinline__ SeqInfo seq_info(const BatchArgs &b, int block_size, int s) {
  SeqInfo i;
  i.bits = 0;
  i.len = b.seq_len[s];
  int row1;
  if (b.row_start) {
    i.row0 = b.row_start[s];
    row1 = b.row_start[s + 1];
  } else {
    i.row0 = s * b.max_new;
    row1 = i.row0 + b.max_new;
  }
  i.n = row1 - i.row0;
  if (i.row0 < 0 || row1 < i.row0 || row1 > b.rows || i.n > b.max_new) {
    i.bits |= SMC_DEV_BAD_ROWS;
    i.n = 0;
    i.row0 = 0;
  }
  if (i.len < i.n || i.len > static_cast<int64_t>(b.T) * block_size) {
    i.bits |= SMC_DEV_BAD_BLOCK;
    i.n = 0;
    i.len = 0;
  }
  return i;
}

// The sequence that row `r` belongs to, or -1 past the last one.
__device__ __forceinline__ int seq_of_row(const BatchArgs &b, int r) {
  if (!b.row_start) return r / b.max_new;
  int lo = 0, hi = b.S;  // the first s with row_start[s + 1] > r
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (b.row_start[mid + 1] > r) hi = mid; else lo = mid + 1;
  }
  return lo < b.S ? lo : -1;
}

}  // namespace smcsd

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

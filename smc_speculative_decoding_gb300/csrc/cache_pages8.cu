// An accepted path of an 8-bit cache moved to the front of its sequence's new
// tokens (kv_compact_tokens8 in smcsd.h).
#include "cache_common.cuh"
#include "path_places.h"

namespace smcsd {

constexpr int kThreads8 = 256;
constexpr int kMoves8 = kMostCompactBlock;  // places found at a time: whole blocks that tokens move into
constexpr int kAhead8 = 8;     // loads of a thread under way before their stores

template <typename U>
__device__ __forceinline__ U rescaled(U x, float f) {
  if (f == 1.f) return x;
  if constexpr (sizeof(U) == 16) {
    return make_uint4(rescale_e4m3x4(x.x, f), rescale_e4m3x4(x.y, f), rescale_e4m3x4(x.z, f),
                      rescale_e4m3x4(x.w, f));
  } else {
    return static_cast<U>(rescale_e4m3x4(x, f));
  }
}

// A CTA takes one sequence, K or V of one layer, and `heads` key heads; a
// thread owns a column (sizeof(U) bytes of a head) of all tokens.  The blocks
// that tokens move into are taken in ascending order.  A source is never ahead
// of its place, so it lies in the block itself or in a later one, which still
// is as it was: per block, first its new scales from those of the sources, then
// the moves in their order (a place that is written is no later source, as the
// path ascends), then, where a scale has grown, the tokens that stayed.
//   Bytes bound it where there are many: 64 paths in 32 layers, 76 MB, 26 us, 2.9
// TB/s, in three dependent round trips (places, scales, elements); with a CTA for
// each block, and its threads over tokens and columns, 68.
template <typename U>
__global__ void __launch_bounds__(kThreads8)
compact_tokens8_kernel(CacheArgs c, ScaleArgs sc, BatchArgs b, const int32_t *path, const int32_t *n_path,
                       int max_path, int heads, unsigned *status) {
  __shared__ int s_block[kMoves8], s_token[kMoves8];  // where a place's token comes from; block -1: it stays
  __shared__ int s_top[kThreads8];                    // new scales of the heads, as their bits
  __shared__ int s_warp[kThreads8 / 32], s_last, s_any;
  const int s = blockIdx.x, tid = threadIdx.x, lane = tid & 31, threads = blockDim.x;
  wait_for_stream();
  const SeqInfo si = seq_info(b, c.block_size, s);
  const int n = n_path[s];
  const bool reports = blockIdx.y == 0 && blockIdx.z == 0;
  if (si.bits || n < 0 || n > max_path) {
    if (reports && tid == 0) raise_status(status, si.bits | (n < 0 || n > max_path ? SMC_DEV_BAD_ROWS : 0));
    return;
  }
  const int32_t *p = path + static_cast<int64_t>(s) * max_path;
  const int32_t *table = b.tables + static_cast<int64_t>(s) * b.T;
  const int layer = blockIdx.y >> 1, head0 = blockIdx.z * heads, here = min(heads, c.kv_heads - head0);
  char *base = ((blockIdx.y & 1) ? c.v : c.k) + layer * c.layer_stride + head0 * c.head_stride;
  float *scale = ((blockIdx.y & 1) ? sc.v : sc.k) + layer * sc.layer + head0 * sc.head;
  const int bs = c.block_size, first = si.len - si.n, per_head = c.head_dim / static_cast<int>(sizeof(U));
  const int cols = per_head * here;
  const PathPlaces places{first, si.n, n, bs};
  if (tid == 0) s_last = -1;
  for (int i0 = 0; i0 < n;) {
    const int i1 = places.end(i0, kMoves8);
    __syncthreads();  // s_last is set; the last places have been read
    for (int r = i0; r < i1; r += threads) {
      const int i = r + tid;
      // an index counts when it is in range, past every one in range before it
      // and not ahead of its place
      const int mine = i < i1 ? p[i] : -1;
      const bool in = mine >= 0 && mine < si.n;
      int top = in ? mine : -1;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, top, o);
        if (lane >= o) top = max(top, up);
      }
      if (lane == 31) s_warp[tid >> 5] = top;
      int before = __shfl_up_sync(0xffffffffu, top, 1);
      if (lane == 0) before = -1;
      __syncthreads();
      before = max(before, s_last);
      for (int w = 0; w < (tid >> 5); ++w) before = max(before, s_warp[w]);
      __syncthreads();
      if (tid == threads - 1) s_last = max(before, in ? mine : -1);
      if (i < i1) {
        const bool good = in && mine > before && mine >= i;
        unsigned bits = good ? 0 : SMC_DEV_BAD_ROWS;
        int block = -1, token = 0;
        if (good && mine != i) {
          const int to = table[(first + i) / bs];
          block = table[(first + mine) / bs];
          token = (first + mine) % bs;
          if (to < 0 || to >= c.blocks || block < 0 || block >= c.blocks) {
            bits |= SMC_DEV_BAD_BLOCK;
            block = -1;
          }
        }
        if (bits && reports) raise_status(status, bits);
        s_block[i - i0] = block;
        s_token[i - i0] = token;
      }
      __syncthreads();
    }
    // the blocks that tokens move into
    for (int from = i0, last = places.moves_end(i1); from < last;) {
      const int slot = places.slot(from), to = places.slot_end(from, last), off = first + from - slot * bs;
      const int moves = to - from, at = from - i0;
      const int block = table[slot];
      from = to;
      if (block < 0 || block >= c.blocks) continue;  // raised above where a token moves
      __syncthreads();
      if (tid == 0) s_any = 0;
      for (int h = tid; h < here; h += threads) {
        s_top[h] = __float_as_int(scale_of(scale[block * sc.block + h * sc.head]));
      }
      __syncthreads();
      for (int e = tid; e < moves * here; e += threads) {
        const int j = e / here, h = e - j * here, src = s_block[at + j];
        if (src >= 0) {
          s_any = 1;
          if (src != block) atomicMax(&s_top[h], __float_as_int(scale_of(scale[src * sc.block + h * sc.head])));
        }
      }
      __syncthreads();
      if (!s_any) continue;
      char *const dst = base + block * c.block_stride;
      for (int col = tid; col < cols; col += threads) {
        const int h = col / per_head;
        const int64_t column = h * c.head_stride + (col - h * per_head) * static_cast<int64_t>(sizeof(U));
        const float now = __int_as_float(s_top[h]);
        for (int j = 0; j < moves; j += kAhead8) {
          U x[kAhead8];
          float f[kAhead8];
#pragma unroll
          for (int e = 0; e < kAhead8; ++e) {
            const int src = j + e < moves ? s_block[at + j + e] : -1;
            if (src >= 0) {
              x[e] = *reinterpret_cast<const U *>(base + src * c.block_stride + s_token[at + j + e] * c.token_stride + column);
              f[e] = scale_of(scale[src * sc.block + h * sc.head]) / now;
            }
          }
#pragma unroll
          for (int e = 0; e < kAhead8; ++e) {
            if (j + e < moves && s_block[at + j + e] >= 0) {
              *reinterpret_cast<U *>(dst + (off + j + e) * c.token_stride + column) = rescaled(x[e], f[e]);
            }
          }
        }
        const float old = scale_of(scale[block * sc.block + h * sc.head]);
        if (old != now) {
          const int held = min(bs, si.len - slot * bs);
          for (int t = 0; t < held; ++t) {
            if (t >= off && t < off + moves && s_block[at + t - off] >= 0) continue;
            U *stays = reinterpret_cast<U *>(dst + t * c.token_stride + column);
            *stays = rescaled(*stays, old / now);
          }
        }
      }
      __syncthreads();  // every thread has read the block's old scales
      for (int h = tid; h < here; h += threads) scale[block * sc.block + h * sc.head] = __int_as_float(s_top[h]);
    }
    i0 = i1;
  }
}

// Widest access that every address of the cache is a multiple of.
static int access_bytes8(const CacheArgs &c) {
  const uint64_t bits = reinterpret_cast<uintptr_t>(c.k) | reinterpret_cast<uintptr_t>(c.v) |
                        static_cast<uint64_t>(c.layer_stride) | static_cast<uint64_t>(c.block_stride) |
                        static_cast<uint64_t>(c.token_stride) | static_cast<uint64_t>(c.head_stride) |
                        static_cast<uint64_t>(c.head_dim);
  return bits % 16 == 0 ? 16 : bits % 4 == 0 ? 4 : 1;
}

cudaError_t launch_compact_tokens8(const CacheArgs &c, const ScaleArgs &s, const BatchArgs &b,
                                   const int32_t *path, const int32_t *n_path, int max_path,
                                   unsigned *status, cudaStream_t st) {
  CacheArgs cache = c;
  ScaleArgs scales = s;
  BatchArgs batch = b;
  const int width = access_bytes8(c), per_head = c.head_dim / width;
  int heads = kThreads8 / per_head;
  heads = heads < 1 ? 1 : heads > c.kv_heads ? c.kv_heads : heads;
  const void *fn = width == 16  ? reinterpret_cast<const void *>(compact_tokens8_kernel<uint4>)
                   : width == 4 ? reinterpret_cast<const void *>(compact_tokens8_kernel<uint32_t>)
                                : reinterpret_cast<const void *>(compact_tokens8_kernel<uint8_t>);
  void *args[] = {&cache, &scales, &batch, &path, &n_path, &max_path, &heads, &status};
  // a thread per column, as far as a CTA goes; at least two warps, which find the places
  const int cols = per_head * heads, threads = cols >= kThreads8 ? kThreads8 : cols <= 64 ? 64 : (cols + 31) / 32 * 32;
  return launch_early(fn, dim3(b.S, 2 * c.layers, (c.kv_heads + heads - 1) / heads), threads, 0, args, st);
}

}  // namespace smcsd

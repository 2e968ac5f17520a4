// Blocks of the cache: copying them (kv_copy_blocks), moving a drafted tree's
// accepted path to the front (kv_compact_tokens), and giving blocks back
// (kv_truncate).  Declared in smcsd.h.
#include "cache_common.cuh"

namespace smcsd {

constexpr int kPageThreads = 256;
constexpr int kInFlight = 8;  // loads of a thread under way before their stores

// A block seen as rows of contiguous elements: block b, row r (of `rows`, the
// tokens and heads that are not contiguous with one another).
struct BlockRows {
  int32_t rows_outer, rows_inner;      // rows = outer * inner
  int64_t outer_stride, inner_stride;  // elements
  int32_t row_elems;
};

// Collapses (token, head, d) of one block into as few contiguous rows as its
// strides allow.
static BlockRows block_rows(const CacheArgs &c) {
  BlockRows r{c.block_size, c.kv_heads, c.token_stride, c.head_stride, c.head_dim};
  if (c.head_stride == c.head_dim || c.kv_heads == 1) {  // heads of a token lie side by side
    r = {1, c.block_size, 0, c.token_stride, c.head_dim * c.kv_heads};
    if (c.token_stride == r.row_elems) r = {1, 1, 0, 0, r.row_elems * c.block_size};
  } else if (c.token_stride == c.head_dim || c.block_size == 1) {  // tokens of a head do
    r = {1, c.kv_heads, 0, c.head_stride, c.head_dim * c.block_size};
    if (c.head_stride == r.row_elems) r = {1, 1, 0, 0, r.row_elems * c.kv_heads};
  }
  return r;
}

// A CTA copies one pair's K or V of one layer; a thread has eight loads under
// way before their stores.  Bound by DRAM: the pairs of 256 particles in 32
// layers, blocks of 16 tokens of 8 heads of 128 in bf16, 641 MB, take 95.5 us
// (6.7 TB/s).
template <typename U>
__global__ void __launch_bounds__(kPageThreads)
copy_blocks_kernel(CacheArgs c, BlockRows br, const int32_t *pairs, const int32_t *counts,
                   int max_pairs, int esz, unsigned *status) {
  const int list = blockIdx.x / max_pairs, i = blockIdx.x % max_pairs;
  wait_for_stream();
  const int n = counts[list];
  if (n < 0 || n > max_pairs) {
    if (threadIdx.x == 0) raise_status(status, SMC_DEV_BAD_ROWS);
    return;
  }
  if (i >= n) return;
  const int src = pairs[2 * static_cast<int64_t>(blockIdx.x)];
  const int dst = pairs[2 * static_cast<int64_t>(blockIdx.x) + 1];
  if (src < 0 || src >= c.blocks || dst < 0 || dst >= c.blocks) {
    if (threadIdx.x == 0) raise_status(status, SMC_DEV_BAD_BLOCK);
    return;
  }
  const int layer = blockIdx.y >> 1;
  char *base = ((blockIdx.y & 1) ? c.v : c.k) + layer * c.layer_stride * esz;
  const char *from = base + src * c.block_stride * esz;
  char *to = base + dst * c.block_stride * esz;
  const int per_row = static_cast<int>(static_cast<int64_t>(br.row_elems) * esz / sizeof(U));
  const int rows = br.rows_outer * br.rows_inner;
  for (int r = 0; r < rows; ++r) {
    const int64_t off = ((r / br.rows_inner) * br.outer_stride +
                         (r % br.rows_inner) * br.inner_stride) * esz;
    const U *src_row = reinterpret_cast<const U *>(from + off);
    U *dst_row = reinterpret_cast<U *>(to + off);
    for (int e0 = threadIdx.x; e0 < per_row; e0 += kInFlight * kPageThreads) {
      U x[kInFlight];
#pragma unroll
      for (int i = 0; i < kInFlight; ++i) {
        const int e = e0 + i * kPageThreads;
        if (e < per_row) x[i] = src_row[e];
      }
#pragma unroll
      for (int i = 0; i < kInFlight; ++i) {
        const int e = e0 + i * kPageThreads;
        if (e < per_row) dst_row[e] = x[i];
      }
    }
  }
}

// Thread t owns column t of a token's (head, d) elements for the whole path.
// A path ascends, so path[i] >= i; behind a skipped entry that is asked for, as
// a place past its token may lie past the new tokens and the table.  Taken in
// order, with a batch's loads before its stores, no move then overwrites a later
// source, and no thread touches another's column.  The places of 64 moves at a time are found by as many
// threads; a CTA's time is then three dependent loads (the path, the blocks,
// the first batch) and the bytes'.  64 paths of up to 9 tokens in 32 layers, 8
// heads of 128 in bf16, 151 MB: 26.3 us (5.7 TB/s).
constexpr int kMoves = 64;

template <typename U>
__global__ void __launch_bounds__(kPageThreads)
compact_tokens_kernel(CacheArgs c, BatchArgs b, const int32_t *path, const int32_t *n_path,
                      int max_path, int esz, unsigned *status) {
  __shared__ int64_t s_from[kMoves], s_to[kMoves];
  __shared__ int s_before[kMoves / 32 + 1], s_last;
  const int s = blockIdx.x, tid = threadIdx.x;
  wait_for_stream();
  const int32_t *p = path + static_cast<int64_t>(s) * max_path;
  int mine = tid < kMoves && tid < max_path ? p[tid] : -1;
  const SeqInfo si = seq_info(b, c.block_size, s);
  const int n = n_path[s];
  const bool reports = blockIdx.y == 0;
  if (si.bits || n < 0 || n > max_path) {
    if (reports && tid == 0) raise_status(status, si.bits | (n < 0 || n > max_path ? SMC_DEV_BAD_ROWS : 0));
    return;
  }
  const int layer = blockIdx.y >> 1;
  char *base = ((blockIdx.y & 1) ? c.v : c.k) + layer * c.layer_stride * esz;
  const int per_head = static_cast<int>(static_cast<int64_t>(c.head_dim) * esz / sizeof(U));
  const int cols = per_head * c.kv_heads;
  const int first = si.len - si.n;
  const int32_t *table = b.tables + static_cast<int64_t>(s) * b.T;
  if (tid == 0) s_last = -1;
  for (int i0 = 0; i0 < n; i0 += kMoves) {
    __syncthreads();  // the last moves' places have been read; s_last is set
    if (tid < kMoves) {
      const int i = i0 + tid, lane = tid & 31;
      if (i0 > 0) mine = i < n ? p[i] : -1;
      // an index counts when it is in range, past every one in range before it
      // (a running maximum over the warp, the warps and the moves before) and
      // not ahead of its place
      const bool in = i < n && mine >= 0 && mine < si.n;
      int top = in ? mine : -1;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int up = __shfl_up_sync(0xffffffffu, top, o);
        if (lane >= o) top = max(top, up);
      }
      if (lane == 31) s_before[tid >> 5] = top;
      int before = __shfl_up_sync(0xffffffffu, top, 1);
      if (lane == 0) before = -1;
      asm volatile("bar.sync 1, 64;" ::: "memory");
      before = max(before, s_last);
      for (int w = 0; w < (tid >> 5); ++w) before = max(before, s_before[w]);
      asm volatile("bar.sync 1, 64;" ::: "memory");
      if (tid == kMoves - 1) s_last = max(before, in ? mine : -1);
      int64_t from = -1, to = -1;
      const bool good = in && mine > before && mine >= i;
      unsigned bits = i < n && !good ? SMC_DEV_BAD_ROWS : 0;
      if (good && mine != i) {
        const int ft = first + mine, tt = first + i;
        const int fb = table[ft / c.block_size], tb = table[tt / c.block_size];
        if (fb < 0 || fb >= c.blocks || tb < 0 || tb >= c.blocks) {
          bits |= SMC_DEV_BAD_BLOCK;
        } else {
          from = (fb * c.block_stride + (ft % c.block_size) * c.token_stride) * esz;
          to = (tb * c.block_stride + (tt % c.block_size) * c.token_stride) * esz;
        }
      }
      if (bits && reports) raise_status(status, bits);
      s_from[tid] = from;
      s_to[tid] = to;
    }
    __syncthreads();
    const int moves = min(n - i0, kMoves);
    for (int col = tid; col < cols; col += blockDim.x) {
      char *column = base + (col / per_head) * c.head_stride * esz +
                     static_cast<int64_t>(col % per_head) * sizeof(U);
      for (int j = 0; j < moves; j += kInFlight) {
        U x[kInFlight];
#pragma unroll
        for (int e = 0; e < kInFlight; ++e) {
          if (j + e < moves && s_from[j + e] >= 0) x[e] = *reinterpret_cast<const U *>(column + s_from[j + e]);
        }
#pragma unroll
        for (int e = 0; e < kInFlight; ++e) {
          if (j + e < moves && s_from[j + e] >= 0) *reinterpret_cast<U *>(column + s_to[j + e]) = x[e];
        }
      }
    }
  }
}

// One CTA per prompt: references of the slots past the kept blocks are
// dropped, freed blocks collected in the workspace's bitmap, then pushed in
// ascending id order; the bitmap is left clear.
__global__ void __launch_bounds__(kPageThreads)
kv_truncate_kernel(int N, KvArgs kv, const int32_t *new_len, Workspace ws) {
  __shared__ int s_warp[kPageThreads / 32];
  __shared__ int s_top;
  const int b = blockIdx.x, tid = threadIdx.x;
  const int words = (kv.P + 31) / 32;
  unsigned *bitmap = ws.kv_bitmap + static_cast<int64_t>(b) * words;
  const int base = b * kv.P;
  for (int n = 0; n < N; ++n) {
    const int64_t at = static_cast<int64_t>(b) * N + n;
    const int len = kv.seq_len[at], keep = new_len[at];
    if (keep < 0 || keep > len || len > static_cast<int64_t>(kv.T) * kv.block_size) {
      if (tid == 0) raise_status(ws.status, SMC_DEV_BAD_BLOCK);
      continue;
    }
    const int from = static_cast<int>((static_cast<int64_t>(keep) + kv.block_size - 1) / kv.block_size);
    const int to = static_cast<int>((static_cast<int64_t>(len) + kv.block_size - 1) / kv.block_size);
    for (int t = from + tid; t < to; t += kPageThreads) {
      int32_t *slot = kv.tables + at * kv.T + t;
      const int id = *slot;
      if (id < base || id >= base + kv.P) {
        raise_status(ws.status, SMC_DEV_BAD_BLOCK);
        continue;
      }
      *slot = -1;
      const int old = atomicSub(&kv.refcount[id], 1);
      if (old <= 0) {
        atomicAdd(&kv.refcount[id], 1);
        raise_status(ws.status, SMC_DEV_BAD_BLOCK);
      } else if (old == 1) {
        atomicOr(&bitmap[(id - base) >> 5], 1u << ((id - base) & 31));
      }
    }
    __syncthreads();  // every thread has read this particle's length
    if (tid == 0) kv.seq_len[at] = keep;
  }
  if (tid == 0) s_top = kv.free_top[b];
  __syncthreads();
  for (int w0 = 0; w0 < words; w0 += kPageThreads) {
    const int w = w0 + tid;
    unsigned m = 0;
    if (w < words) {
      m = __ldcg(&bitmap[w]);
      if (m) bitmap[w] = 0;
    }
    const int mine = __popc(m);
    int incl = mine;
    const int lane = tid & 31, warp = tid >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    if (lane == 31) s_warp[warp] = incl;
    __syncthreads();
    int before = s_top, total = 0;
    for (int k = 0; k < kPageThreads / 32; ++k) {
      if (k < warp) before += s_warp[k];
      total += s_warp[k];
    }
    int at = before + incl - mine;
    while (m) {
      const int bit = __ffs(m) - 1;
      m &= m - 1;
      if (at >= 0 && at < kv.P) kv.free_list[static_cast<int64_t>(base) + at] = base + 32 * w + bit;
      else raise_status(ws.status, SMC_DEV_BAD_BLOCK);
      ++at;
    }
    __syncthreads();
    if (tid == 0) s_top += total;
    __syncthreads();
  }
  if (tid == 0) kv.free_top[b] = s_top;
}

// Widest access that every address of the cache is a multiple of.
static int access_bytes(const CacheArgs &c) {
  const int esz = dtype_bytes(c.dtype);
  const uint64_t bits = reinterpret_cast<uintptr_t>(c.k) | reinterpret_cast<uintptr_t>(c.v) |
                        static_cast<uint64_t>(c.layer_stride * esz) |
                        static_cast<uint64_t>(c.block_stride * esz) |
                        static_cast<uint64_t>(c.token_stride * esz) |
                        static_cast<uint64_t>(c.head_stride * esz) |
                        static_cast<uint64_t>(c.head_dim) * esz;
  if (bits % 16 == 0) return 16;
  return bits % 4 == 0 ? 4 : 2;
}

cudaError_t launch_copy_blocks(const CacheArgs &c, const int32_t *pairs, const int32_t *counts,
                               int lists, int max_pairs, unsigned *status, cudaStream_t st) {
  CacheArgs cache = c;
  BlockRows rows = block_rows(c);
  int esz = dtype_bytes(c.dtype);
  const int width = access_bytes(c);
  const void *fn = width == 16  ? reinterpret_cast<const void *>(copy_blocks_kernel<uint4>)
                   : width == 4 ? reinterpret_cast<const void *>(copy_blocks_kernel<uint32_t>)
                                : reinterpret_cast<const void *>(copy_blocks_kernel<uint16_t>);
  void *args[] = {&cache, &rows, &pairs, &counts, &max_pairs, &esz, &status};
  return launch_early(fn, dim3(lists * max_pairs, 2 * c.layers), kPageThreads, 0, args, st);
}

cudaError_t launch_compact_tokens(const CacheArgs &c, const BatchArgs &b, const int32_t *path,
                                  const int32_t *n_path, int max_path, unsigned *status,
                                  cudaStream_t st) {
  CacheArgs cache = c;
  BatchArgs batch = b;
  int esz = dtype_bytes(c.dtype);
  const int width = access_bytes(c);
  // a thread per column, as far as a CTA goes; at least those that find places
  const int64_t cols = static_cast<int64_t>(c.kv_heads) * c.head_dim * esz / width;
  const int threads = cols >= kPageThreads ? kPageThreads
                      : cols > kMoves      ? static_cast<int>((cols + 31) / 32 * 32)
                                           : kMoves;
  const void *fn = width == 16  ? reinterpret_cast<const void *>(compact_tokens_kernel<uint4>)
                   : width == 4 ? reinterpret_cast<const void *>(compact_tokens_kernel<uint32_t>)
                                : reinterpret_cast<const void *>(compact_tokens_kernel<uint16_t>);
  void *args[] = {&cache, &batch, &path, &n_path, &max_path, &esz, &status};
  return launch_early(fn, dim3(b.S, 2 * c.layers), threads, 0, args, st);
}

cudaError_t launch_kv_truncate(int B, int N, const KvArgs &kv, const int32_t *new_len,
                               const Workspace &ws, cudaStream_t st) {
  kv_truncate_kernel<<<B, kPageThreads, 0, st>>>(N, kv, new_len, ws);
  return cudaGetLastError();
}

}  // namespace smcsd

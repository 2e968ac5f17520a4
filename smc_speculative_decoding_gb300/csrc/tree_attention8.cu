// Attention of each sequence's new tokens over its paged 8-bit cache, under a
// tree mask (smc_tree_attention8 in smcsd.h).  The calls' work and the joins of
// parts are those of attention_work.cuh; the kernel here is its own.
//
// Mathematics.  The cache's bytes go to the tensor cores as they are, by TMA and
// with no conversion on the way, so that a tile costs the CUDA cores nothing but
// its softmax.  The other operands are cut into 8-bit pieces whose products add
// up in the fp32 accumulators:
//  - a row of q, under one power of two, into e4m3 pieces q1 = e4m3(q), q2 =
//    e4m3(q - q1), for fp16 a third: each takes four significant bits and a sign,
//    so two hold bf16's eight and three fp16's eleven (down to 2^-10 beside a
//    largest element of 224 to 448);
//  - a weight w <= 2^15, as fp16, into three e5m2 pieces: three significant bits
//    and a sign each hold fp16's eleven down to w = 2^-6.  The least piece is
//    2^-16; what a smaller weight has below that is rounded up or down by the
//    token's place (small_part), so that many tokens of one small weight come to
//    their sum.  (Rounded to nearest, all of them would be off to the same side:
//    20000 tokens of 2^-21.6 of the largest weight by 17 %, of 2^-24.5 by all that
//    they add.)  What fp16 drops is 2^-25, 2^-33 of a largest weight of 2^8.
//    (e4m3 has two bits more in two pieces, but ends at 2^-9: beside a weight of
//    2^8, tokens of 2^-18 and less of the largest weight would be lost, and a
//    long context has many.)
// The scales of k go to the scores.  Those of v go into the weights' exponents,
//   w_j = 2^(z_j + log2 s_v(j) - M + 8),  out = sum w_j v8_j / sum w_j / s_v(j),
// with M a running maximum of z + log2 s_v, so that weights stay in range
// whatever the scales.
//   The products are the transposed ones, S^T = K Q^T and O^T = V^T P^T: a tile's
// 128 tokens, and the head's dims, are the 128 rows that a tensor-core tile has,
// and the rows of q its columns, of which there are as few as there are.  A
// softmax thread holds one token's scores: a token's two scales are two registers,
// and every thread has work whatever the number of rows.  What must agree
// between tokens, the maximum, is only looked at for a rise (a vote a tile).
#include <atomic>

#include "attention_work.cuh"
#include "tensor_core.cuh"

namespace smcsd {

constexpr int kTile8 = 128;    // tokens per tile
constexpr int kMaxCtas8 = 384; // slots for continuations
static_assert(kMaxCtas8 <= kMostCtas, "tickets");
constexpr int kCtasPerSm = 2;
constexpr int kThreads8 = 320;
constexpr int kSegs8 = 4;      // segments found ahead
constexpr int kTileBytes8 = kTile8 * 128;

template <typename T>
struct Rows8;  // most rows of a unit, pieces of q
template <>
struct Rows8<__nv_bfloat16> { static constexpr int kRows = 64, kPieces = 2; };
template <>
struct Rows8<__half> { static constexpr int kRows = 48, kPieces = 3; };

template <typename T>
struct Units8 {
  static constexpr int kTile = kTile8, kRowTiles = 1, kUnitRows = Rows8<T>::kRows;
  static constexpr bool kParts = true;
};

size_t attention8_workspace_bytes(const CacheArgs &c, const BatchArgs &b, int q_heads) {
  return carve(c, b, q_heads, kMaxCtas8, 64, nullptr, nullptr);
}

struct Kernel8Args : WorkArgs {
  ScaleArgs sc8;
};

constexpr float kTop = 15.f;      // weights are at most 2^kTop (as fp16: 0x7800) ...
constexpr uint32_t kPastTop = 0x07ff07ff;  // adds up to 0x8000 with what is more, as fp16
constexpr float kTopFresh = 8.f; // ... and the largest one 2^kTopFresh when the maximum is taken
constexpr float kUnset = 3e38f;   // of a row that has seen nothing yet, in place of kTopFresh - M: past kTop with any score
constexpr float kSumScale = 0x1p-32f;  // sums of w / s_v: centres their range

// ---------------------------------------------------------------------------
// attention8_kernel.  Two CTAs to a multiprocessor, each: warps 0-7 the softmax
// (thread = token of a tile; warps w and w + 4 take the even and the odd chunks of
// 16 rows; ahead of a segment they cut its rows of q into pieces, four threads a
// row), warp 8 issues the matrix products, warp 9 finds the CTA's segments (parts
// of units), copies K and V and prepares their scales.  Shared memory: two slots
// each of K and V tiles, q's pieces, the weights' pieces.  Tensor memory, 64
// columns each: two tiles' scores, the accumulator, the sums of w / s_v (each
// lane's tokens).
//   A softmax thread's loop takes 16 rows at a time and keeps nothing of them in
// registers.  64 trees of 16 tokens over up to 8192: 64 rows unrolled with the
// sums in registers, 4 warps a CTA, 391 us; so, with 8 warps, 291; with the rows'
// pieces cut by the same warps and so 96 registers each, 256 (a largest weight of
// 2^8 and not 2^7 since, 261).  Other ways:
// chunks of 8 rows 289, two chunks unrolled 320, the next chunk's scores loaded
// ahead 274, 4 warps 277.
//   Weights are taken on trust that none passes 2^kTop, and written ahead of the
// vote that says so; the products start behind it.  Where a maximum has risen, what
// the tile added to the sums of those chunks is taken off again, maxima, sums and
// accumulator are brought up, and the chunks are taken anew (once: they cannot pass
// again).  (Of an earlier form that took 322 us, a timing copy whose maxima never
// rose took 262.)
//   What bounds it: the softmax, half of the issue slots and waits for tensor
// memory, exponentials and the vote between them.  A tile's products keep the
// tensor cores for 980 cycles (a product of 64 columns is bound by its operands'
// way from shared memory, 49 cycles), its bytes the memory for 1400; a
// multiprocessor takes 2500 cycles a tile.
//   Measured: those 64 trees, 812 MB, 258 to 265 us, 3.1 TB/s; 131072 tokens of
// one sequence, 269 MB, 102 to 108 us, of which 14 us start it; one token over 513,
// 12.5 us.  DRAM reads 1.21 GB for the 64 trees: a head's token is 128 bytes, and
// what comes with it to L2 is the next head's, which another CTA reads later.
//   Every wait is bounded, and on a barrier all of whose turns the waiting
// thread follows.
// ---------------------------------------------------------------------------
struct alignas(16) Seg8 {  // read and written in 16-byte words
  int row0, rows;  // first row of the unit, rows of it
  int i0;          // new token of the first row (own parts)
  int seq, head;   // head unit
  int t0, n;       // first token, tiles
  int ctx, kv1;    // tokens before ctx are seen by all; end of the entry's tokens
  int flags;
  int join;        // of a cut unit: the owner CTA, and continuations << 16
  int pad;
};
constexpr int kWhole8 = 4, kBase8 = 8, kEnd8 = 16;  // with kShared: final result, first tiles, none left

struct Tail8 {
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2];
  uint64_t s_full[2], p_full, pv_done, q_full, o_full, o_free, drained;
  uint64_t seg_full[kSegs8], seg_empty[kSegs8], group;
  Seg8 seg[kSegs8];
  float4 token[2][kTile8];  // of a tile's tokens: scale * log2 e * s_k, log2 s_v, kSumScale / s_v
  float4 col[32];     // of two rows each: scale of q, and kTopFresh - M
  alignas(16) int top[64];  // maxima of a tile, then factors
  uint32_t rise[3];   // chunks of 16 rows in which a weight passed 2^kTop, of three votes
  unsigned nonfinite; // the last segment (from 1) with a new token whose NaN were zeroed
  uint32_t tmem;
  volatile int abort;
  int joins;          // this CTA stored the last part of the unit
};

static_assert(sizeof(Seg8) == 48 && offsetof(Tail8, seg) % 16 == 0 && offsetof(Tail8, col) % 16 == 0, "16-byte words");

template <typename T>
struct Smem8 {
  static constexpr int kRows = Rows8<T>::kRows;
  static constexpr int kPiece = kRows * 128;  // bytes of one piece of q, or of a tile's weights
  static constexpr int kK = 0, kV = 2 * kTileBytes8, kQ = 4 * kTileBytes8;
  static constexpr int kP = kQ + Rows8<T>::kPieces * kPiece;
  static constexpr int kTail = kP + 3 * kPiece;
  static constexpr int kBytes = kTail + static_cast<int>(sizeof(Tail8));
};
// an SM's 228 KB less 1 KB of the system's for each CTA
static_assert(Smem8<__nv_bfloat16>::kBytes <= 228 * 1024 / kCtasPerSm - 1024, "shared memory");
static_assert(Smem8<__half>::kBytes <= 228 * 1024 / kCtasPerSm - 1024, "shared memory");
static_assert(Smem8<__half>::kPiece % 1024 == 0, "the swizzle counts from 1 KB boundaries");

__device__ __forceinline__ bool take_segment8(Tail8 *s, uint32_t seg, Seg8 *to, unsigned *status) {
  if (!warp_wait(s, &s->seg_full[seg % kSegs8], seg / kSegs8 & 1u, status)) return false;
  const int4 *from = reinterpret_cast<const int4 *>(&s->seg[seg % kSegs8]);
  const int4 a = from[0], b = from[1], c = from[2];
  *to = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w, c.x, c.y, c.z, c.w};
  return !(to->flags & kEnd8);
}

// Of a scale.  (Where log2's last bit is off, both a token's weight and what
// its weight adds to the sum are by the same factor: a score off by 2^-22 of it.)
__device__ __forceinline__ float fast_log2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float fast_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// What is added to a weight's last fp16 part (twice) before its lower byte is
// dropped, so that it is rounded to e5m2: 0 to 255 by a token's place, the
// golden ratio's multiples, which any run of places covers evenly.  A part that
// e5m2 holds has a lower byte of 0 and stays as it is.
__device__ __forceinline__ uint32_t small_part(int place) {
  return (static_cast<uint32_t>(place) * 40503u >> 8 & 0xffu) * 0x00010001u;
}

// The order of floats in that of ints (and back: its own inverse).
__device__ __forceinline__ int ordered(int bits) { return bits ^ (bits >> 31 & 0x7fffffff); }

// Which rows of a unit see token `at` (at or past w.ctx): bits [i * heads, (i + 1)
// * heads) for new token w.i0 + i.
template <typename T>
__device__ __forceinline__ uint64_t rows_that_see(const WorkArgs &k, const Seg8 &w, int at) {
  if (at < w.ctx) return ~0ull;
  if (at >= w.kv1) return 0;
  const int heads = unit_heads<Units8<T>>(k, w.head).n;
  const int j = at - w.ctx, tokens = w.rows / heads, word = j >> 5;
  const uint64_t one = heads >= 64 ? ~0ull : (1ull << heads) - 1;
  uint64_t see = 0;
  if (!k.a.mask) {  // a chain: new tokens j and later
#pragma unroll 1
    for (int i = max(j - w.i0, 0); i < tokens; ++i) see |= one << (i * heads);
    return see;
  }
  if (word >= k.a.mask_words) return 0;
  const uint32_t *mask = k.a.mask + static_cast<int64_t>(w.row0) * k.a.mask_words + word;
#pragma unroll 4
  for (int i = 0; i < tokens; ++i) {
    if (__ldg(mask + static_cast<int64_t>(i) * k.a.mask_words) >> (j & 31) & 1u) see |= one << (i * heads);
  }
  return see;
}

// Rows that see a new token whose element d of v is NaN get NaN there: the
// products met it as 0.
template <typename T>
__device__ __forceinline__ void patch_nan8(const WorkArgs &k, const Seg8 &w, const UnitHeads &heads, int d, char *const *to,
                                           bool whole) {
  const int32_t *table = k.a.b.tables + static_cast<int64_t>(w.seq) * k.a.b.T;
  const int t1 = min(w.t0 + w.n * kTile8, w.kv1);
#pragma unroll 1
  for (int at = max(w.t0, w.ctx); at < t1; ++at) {
    const int block = table[block_of(k, at)];
    if (block < 0 || block >= k.a.c.blocks) continue;
    const char *v = k.a.c.v + block * k.a.c.block_stride + (at % k.a.c.block_size) * k.a.c.token_stride +
                    heads.key * k.a.c.head_stride;
    if ((v[d] & 0x7f) != 0x7f) continue;
    const uint64_t see = rows_that_see<T>(k, w, at);
#pragma unroll 1
    for (int r = 0; r < w.rows; ++r) {
      if (!(see >> r & 1)) continue;
      const float nan = __uint_as_float(0x7fffffffu);
      if (whole) reinterpret_cast<T *>(to[r])[d] = from_f32<T>(nan);
      else reinterpret_cast<float *>(to[r])[d] = nan;
    }
  }
}

// Sums v[0..15] over the warp's lanes; lane l gets that of v[l % 16].
__device__ __forceinline__ float transposed_sum(const uint32_t *x) {
  const int lane = threadIdx.x & 31;
  float v[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) v[j] = __uint_as_float(x[j]);
#pragma unroll
  for (int s = 8; s > 0; s >>= 1) {
    const bool up = lane & s;
#pragma unroll
    for (int j = 0; j < s; ++j) {
      const float send = up ? v[j] : v[j + s], keep = up ? v[j + s] : v[j];
      v[j] = keep + __shfl_xor_sync(0xffffffffu, send, s);
    }
  }
  return v[0] + __shfl_xor_sync(0xffffffffu, v[0], 16);
}

// The maximum of v[0..15] over the warp's lanes, NaN as -inf; lane l gets that of v[l % 16].
__device__ __forceinline__ float transposed_max(const uint32_t *x) {
  const int lane = threadIdx.x & 31;
  float v[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) v[j] = fmaxf(__uint_as_float(x[j]), -INFINITY);
#pragma unroll
  for (int s = 8; s > 0; s >>= 1) {
    const bool up = lane & s;
#pragma unroll
    for (int j = 0; j < s; ++j) {
      const float send = up ? v[j] : v[j + s], keep = up ? v[j + s] : v[j];
      v[j] = fmaxf(keep, __shfl_xor_sync(0xffffffffu, send, s));
    }
  }
  return fmaxf(v[0], __shfl_xor_sync(0xffffffffu, v[0], 16));
}

// 64 of a token's 128 bytes of a V tile: all become 0, or (not `all`) those that
// are NaN, of which it says whether there were any.
__device__ __forceinline__ bool clear_row8(char *row, bool all) {
  bool found = false;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    uint4 *x16 = reinterpret_cast<uint4 *>(row) + ((e + threadIdx.x) & 3);
    uint4 x = make_uint4(0, 0, 0, 0);
    bool change = all;
    if (!all) {
      x = *x16;
      uint32_t *words = reinterpret_cast<uint32_t *>(&x);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t bad = __vcmpeq4(words[j] & 0x7f7f7f7fu, 0x7f7f7f7fu);
        if (bad) {
          words[j] &= ~bad;
          change = found = true;
        }
      }
    }
    if (change) *x16 = x;
  }
  return found;
}

template <typename T, bool kTma>
__global__ void __launch_bounds__(kThreads8, kCtasPerSm)
attention8_kernel(const __grid_constant__ Kernel8Args k, const __grid_constant__ CUtensorMap map_k,
                  const __grid_constant__ CUtensorMap map_v) {
  using M = Smem8<T>;
  constexpr int kRows = Rows8<T>::kRows, kPieces = Rows8<T>::kPieces;
  extern __shared__ __align__(1024) char smem[];
  Tail8 *const s = reinterpret_cast<Tail8 *>(smem + M::kTail);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const CacheArgs &c8 = k.a.c;
  const int D = c8.head_dim;
  unsigned *const status = k.a.status;

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s->k_full[i], 1);
      mbar_init(&s->k_empty[i], 1);
      mbar_init(&s->v_full[i], 1);
      mbar_init(&s->v_empty[i], 1);
      mbar_init(&s->s_full[i], 2);  // the products, and the tokens' scales
    }
    mbar_init(&s->p_full, 1);
    mbar_init(&s->pv_done, 1);
    mbar_init(&s->q_full, 8);
    mbar_init(&s->o_full, 1);
    mbar_init(&s->o_free, 8);
    mbar_init(&s->drained, 1);
    mbar_init(&s->group, 8);
    s->rise[0] = s->rise[1] = s->rise[2] = 0;
    for (int i = 0; i < kSegs8; ++i) {
      mbar_init(&s->seg_full[i], 1);
      mbar_init(&s->seg_empty[i], 9);  // every warp but the one that fills it
    }
    s->nonfinite = 0;
    s->abort = (smem_addr(smem) & 1023u) != 0;
    mbar_init_fence();
  }
  if (warp == 8) tmem_alloc<256>(&s->tmem);
  if (kTma && warp == 9 && elect_one()) {
    prefetch_map(&map_k);
    prefetch_map(&map_v);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s->tmem;
  wait_for_stream();
  if (k.more_kernels) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  if (s->abort) {
    if (tid == 0) raise_status(status, SMC_DEV_TIMEOUT);
  } else if (warp < 8) {
    // ---- softmax --------------------------------------------------------------
    const int half = warp >> 2, token = tid & 127;  // chunks half, half + 2; token of a tile
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(warp & 3) << 21), t_o = t_lane + 128, t_sum = t_lane + 192;
    char *const p_at = smem + M::kP + (token >> 3) * 128 + (token & 7) * 16;
    uint32_t seg = 0, tile = 0, turns = 0, votes = 0;
    bool ok = true;
    // all softmax warps, and the bits that any of them names.  Vote v goes into word v % 3, which was cleared behind
    // vote v - 2: all had read it then, and no one writes it before the one who clears it has come to vote v - 1.
    auto group_or = [&](uint32_t mine) {
      uint32_t *const word = s->rise + votes;
      if (mine) atomicOr(word, mine);
      warp_arrive(&s->group, lane);
      ++turns;
      ok = warp_wait(s, &s->group, (turns - 1) & 1u, status);
      const uint32_t all = *reinterpret_cast<volatile uint32_t *>(word);
      votes = votes == 2 ? 0 : votes + 1;
      if (tid == 0) s->rise[votes == 2 ? 0 : votes + 1] = 0;  // word v + 2 = v - 1
      return all;
    };
    auto group_sync = [&] {
      warp_arrive(&s->group, lane);
      ++turns;
      return warp_wait(s, &s->group, (turns - 1) & 1u, status);
    };
    while (ok && warp_wait(s, &s->seg_full[seg % kSegs8], seg / kSegs8 & 1u, status)) {
      const Seg8 &w = s->seg[seg % kSegs8];  // (released behind the segment: what is rarely looked at stays there)
      if (w.flags & kEnd8) break;
      const int tiles = w.n, ctx = w.flags & kShared ? INT32_MAX : w.ctx, kv1 = w.kv1;
      const int chunks = (w.rows + 15) >> 4;
      int at = w.t0 + token;
      {
        uint32_t zero[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) zero[e] = 0;
        __syncwarp();
        for (int cb = half; cb < chunks; cb += 2) tmem_st16(t_sum + cb * 16, zero);
        tmem_wait_st();
      }
      // the rows' pieces and scales, maxima not set (the products of the last segment are done)
      {
        const UnitHeads heads = unit_heads<Units8<T>>(k, w.head);
        const int r = tid >> 2, part = tid & 3, in = r / heads.n, rows = w.rows;  // 32 dims each
        const uint4 *q = reinterpret_cast<const uint4 *>(
            k.a.q + ((w.row0 + in) * k.a.q_row + (heads.first + r - in * heads.n) * k.a.q_head) * static_cast<int64_t>(sizeof(T)));
        uint4 v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          v[e] = r < rows && part * 4 + e < D / 8 ? q[part * 4 + e] : make_uint4(0, 0, 0, 0);
        }
        const T *x = reinterpret_cast<const T *>(v);
        float top = 0.f;
#pragma unroll
        for (int j = 0; j < 32; ++j) {
          const float a = fabsf(to_f32(x[j]));
          if (a < INFINITY) top = fmaxf(top, a);
        }
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // (a row of bf16 may be of any size: the range is that of 2^t and 2^-t both)
        const float scale = least_scale<126>(top), inv = __uint_as_float((254u << 23) - __float_as_uint(scale));  // 1 / 2^t
        if (r < 16 * chunks) {
          char *const to = smem + M::kQ + r * 128;
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t words[kPieces][4] = {};
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
              float a = finite_or_nan(to_f32(x[c * 16 + j])) * inv, b = finite_or_nan(to_f32(x[c * 16 + j + 1])) * inv;
#pragma unroll
              for (int piece = 0; piece < kPieces; ++piece) {
                const uint32_t e = to_e4m3x2(a, b), h = from_e4m3x2(e);
                words[piece][j / 4] |= e << (j & 2) * 8;
                const float2 taken = __half22float2(*reinterpret_cast<const __half2 *>(&h));
                a -= taken.x;
                b -= taken.y;
              }
            }
#pragma unroll
            for (int piece = 0; piece < kPieces; ++piece) {
              *reinterpret_cast<uint4 *>(to + piece * M::kPiece + (((part * 2 + c) ^ (r & 7)) << 4)) =
                  make_uint4(words[piece][0], words[piece][1], words[piece][2], words[piece][3]);
            }
          }
        }
        if (part == 0) {
          float *const col = reinterpret_cast<float *>(&s->col[r >> 1]) + (r & 1);
          col[0] = r < rows ? scale : 0.f;
          col[2] = r < rows ? kUnset : -INFINITY;
        }
        fence_proxy_async_smem();
        warp_arrive(&s->q_full, lane);
      }
      ++seg;
      if (!(ok = group_sync())) break;  // (every row's scale)

      for (int i = 0; i < tiles; ++i, ++tile, at += kTile8) {
        const bool edge = at - token + kTile8 > ctx;
        const uint64_t see = edge ? rows_that_see<T>(k, w, at) : ~0ull;
        const uint32_t buf = tile & 1u, t_s = t_lane + buf * 64;
        if (!(ok = warp_wait(s, &s->s_full[buf], tile >> 1 & 1u, status))) break;
        tc_fence_after();
        const float4 scales = s->token[buf][token];
        const unsigned long long a2 = f2dup(scales.x), b2 = f2dup(scales.y), c2 = f2dup(scales.z);
        const uint32_t last = small_part(at);
        uint32_t todo = ~0u;  // chunks to take; at first all, then those with a new maximum (once)
        uint32_t over = 0;    // of this warp: those where one of its weights passed 2^kTop
        for (bool known = i > 0, again = false;; known = true) {
          if (known) {
#pragma unroll 1
            for (int cb = half; cb < chunks; cb += 2) {
              if (!(todo >> cb & 1)) continue;
              uint32_t most = 0;  // the largest weights, fp16, of even and of odd rows
              unsigned long long z[8], sum[8];
              __syncwarp();
              tmem_get16x2(t_s + cb * 16, t_sum + cb * 16, z, sum);
              const float4 *col = s->col + cb * 8;
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float4 c = col[e];
                // (less M behind the maximum's own rounding)
                z[e] = add2(fma2(z[e], mul2(a2, f2pack(c.x, c.y)), b2), f2pack(c.z, c.w));
              }
              if (edge) {
                const uint32_t some = static_cast<uint32_t>(see >> (cb * 16));
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  float y0, y1;
                  f2unpack(z[e], y0, y1);
                  z[e] = f2pack(some >> 2 * e & 1 ? y0 : -INFINITY, some >> (2 * e + 1) & 1 ? y1 : -INFINITY);
                }
              }
              uint32_t h[8], p[4];
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                float w0, w1;
                f2unpack(z[e], w0, w1);
                w0 = fast_exp2(w0);
                w1 = fast_exp2(w1);
                h[e] = pack2<__half>(w0, w1);
                sum[e] = fma2(f2pack(w0, w1), c2, sum[e]);
                asm("max.f16x2 %0, %0, %1;" : "+r"(most) : "r"(h[e]));
              }
              // the weights' slots are free when the last product is done
              if (cb == half && tile > 0 && !(ok = warp_wait(s, &s->pv_done, (tile - 1) & 1u, status))) break;
              // pieces: e5m2 is fp16's upper byte, rounded by adding half of its step (the last one: see small_part)
#pragma unroll
              for (int piece = 0; piece < 3; ++piece) {
#pragma unroll
                for (int e = 0; e < 8; e += 2) {
                  const uint32_t u = h[e] + (piece < 2 ? 0x00800080u : last), v = h[e + 1] + (piece < 2 ? 0x00800080u : last);
                  p[e / 2] = __byte_perm(u, v, 0x7531);
                  if (piece < 2) {
                    const uint32_t hu = u & 0xff00ff00u, hv = v & 0xff00ff00u;
                    asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(h[e]) : "r"(hu));
                    asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(h[e + 1]) : "r"(hv));
                  }
                }
                *reinterpret_cast<uint4 *>(p_at + piece * M::kPiece + cb * 2048) = make_uint4(p[0], p[1], p[2], p[3]);
              }
              const bool past = __any_sync(0xffffffffu, (most + kPastTop) & 0x80008000u);
              // (the sums go without weights that may be of any size; the second time none is)
              if (again || !past) {
                __syncwarp();
                tmem_put16(t_sum + cb * 16, sum);
              } else {
                over |= 1u << cb;
              }
            }
            if (!ok) break;
            if (edge) {
              // the tile reaches past the committed tokens: rows of V past the last
              // token become 0 (they may hold anything), and so do NaN of new tokens,
              // which patch_nan8 puts back
              if (!(ok = warp_wait(s, &s->v_full[buf], tile >> 1 & 1u, status))) break;
              if (at >= ctx && clear_row8(smem + M::kV + buf * kTileBytes8 + token * 128 + half * 64, at >= kv1)) {
                s->nonfinite = seg;
              }
            }
            fence_proxy_async_smem();
            __syncwarp();
            tmem_wait_st();
            tc_fence_before();
            todo = group_or(again || lane ? 0 : over);
            if (!ok || !todo) break;
            tc_fence_after();
            again = true;
          }
          // New maxima in these chunks, of every row whose weights would pass 2^kTopFresh while at it: a tile's largest
          // z + log2 s_v.  What the warp added to the sums is taken off again; it counts once more under the new
          // maximum, so that its rounding here is small beside the sum.
          if (tid < 64) s->top[tid] = INT32_MIN;
          if (!(ok = group_sync())) break;
#pragma unroll 1
          for (int cb = half; cb < chunks; cb += 2) {
            if (!(todo >> cb & 1)) continue;
            const bool added = known && !(over >> cb & 1);
            uint32_t x[16], sum[16];
            __syncwarp();
            tmem_ld16(t_s + cb * 16, x);
            tmem_ld16(t_sum + cb * 16, sum);
            tmem_wait_all();
            tmem_tie16(x);
            tmem_tie16(sum);
            const uint32_t some = static_cast<uint32_t>(see >> (cb * 16));
#pragma unroll
            for (int e = 0; e < 16; e += 2) {
              const float4 c = s->col[cb * 8 + e / 2];
              const unsigned long long y =
                  fma2(f2pack(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), mul2(a2, f2pack(c.x, c.y)), b2);
              float y0, y1, w0, w1, s0, s1;
              f2unpack(y, y0, y1);
              f2unpack(add2(y, f2pack(c.z, c.w)), w0, w1);
              x[e] = some >> e & 1 ? __float_as_uint(y0) : 0xff800000u;
              x[e + 1] = some >> (e + 1) & 1 ? __float_as_uint(y1) : 0xff800000u;
              w0 = some >> e & 1 ? fast_exp2(w0) : 0.f;
              w1 = some >> (e + 1) & 1 ? fast_exp2(w1) : 0.f;
              f2unpack(fma2(f2pack(-w0, -w1), c2, f2pack(__uint_as_float(sum[e]), __uint_as_float(sum[e + 1]))), s0, s1);
              sum[e] = __float_as_uint(s0);
              sum[e + 1] = __float_as_uint(s1);
            }
            if (added) tmem_st16(t_sum + cb * 16, sum);
            const float top = transposed_max(x);
            if (lane < 16) atomicMax(&s->top[cb * 16 + lane], ordered(__float_as_int(top)));
          }
          tmem_wait_st();
          if (!(ok = group_sync())) break;
          if (tid < 64) {
            float f = 1.f;  // the factor's root: a factor itself may be less than fp32 holds, beside a sum of 2^76
            if (tid < w.rows && todo >> (tid >> 4) & 1) {
              const float top = __int_as_float(ordered(s->top[tid]));
              float *less = reinterpret_cast<float *>(&s->col[tid >> 1]) + 2 + (tid & 1);
              if (top > -INFINITY && top + *less > kTopFresh) {
                f = *less == kUnset ? 0.f : fast_exp2(0.5f * (kTopFresh - top - *less));
                const float fresh = kTopFresh - top;
                *less = top + fresh > kTop ? -top : fresh;  // where a step of fp32 is more than kTop - kTopFresh
              }
            }
            s->top[tid] = __float_as_int(f);
          }
          if (!(ok = group_sync())) break;
          if (i > 0) {  // (the last product is in the accumulator: the weights' slots were free)
#pragma unroll 1
            for (int cb = half; cb < chunks; cb += 2) {
              if (!(todo >> cb & 1)) continue;
              uint32_t o[16], sum[16];
              __syncwarp();
              tmem_ld16(t_o + cb * 16, o);
              tmem_ld16(t_sum + cb * 16, sum);
              tmem_wait_all();
              tmem_tie16(o);
              tmem_tie16(sum);
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const float f = __int_as_float(s->top[cb * 16 + e]);
                o[e] = __float_as_uint(__uint_as_float(o[e]) * f * f);
                sum[e] = __float_as_uint(__uint_as_float(sum[e]) * f * f);
              }
              tmem_st16(t_o + cb * 16, o);
              tmem_st16(t_sum + cb * 16, sum);
            }
            tmem_wait_st();
          }
        }
        if (!ok) break;
        if (tid == 0) mbar_arrive(&s->p_full);  // behind the vote, for all: the scores have been read, too
        __syncwarp();
      }
      if (!ok) break;
      // ---- the unit's result --------------------------------------------------
      if (!(ok = warp_wait(s, &s->o_full, (seg - 1) & 1u, status))) break;
      tc_fence_after();
      // (the weights' slots are free: the sums of four warps, factors and rows' addresses)
      float *const sums = reinterpret_cast<float *>(smem + M::kP), *const inverse = sums + 4 * 64;
      char **const to = reinterpret_cast<char **>(inverse + 64);
#pragma unroll 1
      for (int cb = half; cb < chunks; cb += 2) {
        uint32_t x[16];
        __syncwarp();
        tmem_ld16(t_sum + cb * 16, x);
        tmem_wait_all();
        tmem_tie16(x);
        const float sum = transposed_sum(x);
        if (lane < 16) sums[(warp & 3) * 64 + cb * 16 + lane] = sum;
      }
      if (!(ok = group_sync())) break;
      const UnitHeads heads = unit_heads<Units8<T>>(k, w.head);
      const bool whole = w.flags & kWhole8, base = w.flags & kBase8;
      const int kind = w.flags & kShared ? 1 : 0;
      if (tid < w.rows) {
        const float l = (sums[tid] + sums[64 + tid]) + (sums[128 + tid] + sums[192 + tid]);
        const int in = tid / heads.n, row = w.row0 + in, qh = heads.first + tid - in * heads.n;
        const int64_t rh = static_cast<int64_t>(row) * k.a.q_heads + qh;
        const int64_t cont = static_cast<int64_t>(blockIdx.x) * kRows + tid;
        const float less = *(reinterpret_cast<const float *>(&s->col[tid >> 1]) + 2 + (tid & 1));
        const float lse2 = l == 0.f ? -INFINITY : log2f(l) + (32.f - less);
        inverse[tid] = l == 0.f ? 0.f : 1.f / l * kSumScale;
        if (whole) {
          if (k.a.lse) k.a.lse[rh] = lse2 * 0.69314718055994531f;
          to[tid] = k.a.out + (row * k.a.o_row + qh * k.a.o_head) * static_cast<int64_t>(sizeof(T));
        } else if (base) {
          k.w.lse[kind][rh] = lse2;
          to[tid] = reinterpret_cast<char *>(k.w.o[kind] + rh * D);
        } else {
          k.w.lse_c[cont] = lse2;
          to[tid] = reinterpret_cast<char *>(k.w.o_c + cont * D);
        }
      }
      if (!(ok = group_sync())) break;
      const bool bad = *reinterpret_cast<volatile unsigned *>(&s->nonfinite) == seg;
      const int rows = w.rows;
#pragma unroll 1
      for (int cb = half; cb < chunks; cb += 2) {
        uint32_t o[16];
        __syncwarp();
        tmem_ld16(t_o + cb * 16, o);
        tmem_wait_all();
        tmem_tie16(o);
        if (token < D) {
          const int some = min(rows - cb * 16, 16);
          auto value = [&](int e) {
            const float f = inverse[cb * 16 + e];
            return f == 0.f ? 0.f : __uint_as_float(o[e]) * f;
          };
          if (whole) {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              if (e < some) reinterpret_cast<T *>(to[cb * 16 + e])[token] = from_f32<T>(value(e));
            }
          } else {
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              if (e < some) reinterpret_cast<float *>(to[cb * 16 + e])[token] = value(e);
            }
          }
        }
      }
      tc_fence_before();
      warp_arrive(&s->o_free, lane);  // the accumulator may be written again
      if (bad) {
        if (!(ok = group_sync())) break;  // both halves' rows are written
        if (tid < D) patch_nan8<T>(k, w, heads, tid, to, whole);
      }
      __syncwarp();
      if (k.join_inside && !whole) {
        // the CTA that stores a cut unit's last part joins them, in their order
        const int owner = w.join & 0xffff, more = w.join >> 16;
        if (!(ok = group_sync())) break;
        if (tid == 0) {
          __threadfence();  // what the CTA stored, ahead of the count
          const bool all = atomicAdd(&k.w.tickets[owner], 1u) == static_cast<unsigned>(more);
          if (all) k.w.tickets[owner] = 0;
          s->joins = all;
          __threadfence();
        }
        if (!(ok = group_sync())) break;
        if (s->joins) {
          for (int slot = warp; slot < w.rows; slot += 8) {
            const int in = slot / heads.n, qh = heads.first + slot - in * heads.n;
            const int64_t rh = static_cast<int64_t>(w.row0 + in) * k.a.q_heads + qh;
            write_row<T>(k, rh, w.row0 + in, qh, join_parts<Units8<T>>(k, 0, rh, owner, more, slot));
          }
        }
        __syncwarp();
      }
      // (the next segment's first weights are written behind a turn of `group`, and so behind all of this)
      warp_arrive(&s->seg_empty[(seg - 1) % kSegs8], lane);
    }
    __syncwarp();
    tmem_wait_all();  // (a warp that gave up may have left some under way)
    tmem_wait_st();
  } else {
    if (warp == 8) {
      // ---- matrix products ----------------------------------------------------
      const int k_steps = (D + 31) / 32;
      const uint32_t k0 = smem_desc(smem_addr(smem + M::kK), 16), v0 = smem_desc(smem_addr(smem + M::kV), 16);
      const uint32_t q0 = smem_desc(smem_addr(smem + M::kQ), 16);
      // weights: 8 tokens x 16 rows of 16 bytes each, 128 bytes to the next tokens, 2048 to the next rows
      const uint32_t p0 = smem_desc(smem_addr(smem + M::kP), 128);
      constexpr uint32_t kHighP = 2048u >> 4 | 1u << 14;
      uint32_t seg = 0, tile = 0;
      bool ok = true;
      Seg8 w;
      while (ok && take_segment8(s, seg, &w, status)) {
        warp_arrive(&s->seg_empty[seg % kSegs8], lane);
        const int n = w.n, columns = (w.rows + 15) & ~15;
        const uint32_t id_s = instr_desc8(columns, false, false, false), id_o = instr_desc8(columns, true, true, true);
        if (elect_one()) {
          // the scores of tile i, then the product with V of the tile before
          ok = guarded_wait(s, &s->q_full, seg & 1u, status);
          for (int i = 0; ok && i <= n; ++i) {
            if (i < n) {  // (their buffer's last ones have been read: the weights of two tiles ago were there)
              const uint32_t at = (tile + i) & 1u;
              if (!(ok = guarded_wait(s, &s->k_full[at], (tile + i) >> 1 & 1u, status))) break;
              tc_fence_after();
              const uint32_t ka = k0 + at * (kTileBytes8 >> 4);
#pragma unroll 1
              for (int piece = 0; piece < kPieces; ++piece) {
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                  if (c < k_steps) {
                    mma8_ss(tmem + at * 64, ka + c * 32 / 16, q0 + (piece * M::kPiece + c * 32) / 16, kDescHigh, id_s,
                            piece > 0 || c > 0);
                  }
                }
              }
              tc_commit(&s->s_full[at]);
              tc_commit(&s->k_empty[at]);
            }
            if (i == 0) continue;
            const uint32_t last = tile + i - 1, at = last & 1u;
            // the last segment's result has been read
            if (i == 1 && seg > 0 && !(ok = guarded_wait(s, &s->o_free, (seg - 1) & 1u, status))) break;
            if (!(ok = guarded_wait(s, &s->v_full[at], last >> 1 & 1u, status) && guarded_wait(s, &s->p_full, last & 1u, status))) break;
            tc_fence_after();
            const uint32_t va = v0 + at * (kTileBytes8 >> 4);
#pragma unroll 1
            for (int piece = 0; piece < 3; ++piece) {
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                mma8_ss(tmem + 128, va + c * 4096 / 16, p0 + (piece * M::kPiece + c * 512) / 16, kHighP, id_o,
                        i > 1 || piece > 0 || c > 0);
              }
            }
            tc_commit(&s->v_empty[at]);
            tc_commit(&s->pv_done);
          }
          if (ok) tc_commit(&s->o_full);
        }
        ok = __all_sync(0xffffffffu, ok);
        tile += n;
        ++seg;
      }
      if (elect_one()) {
        tc_commit(&s->drained);  // nothing of this CTA runs on when it ends
        if (!mbar_wait(&s->drained, 0, kWaitPolls)) raise_status(status, SMC_DEV_TIMEOUT);
      }
      __syncwarp();
    } else {
      // ---- segments, K and V ----------------------------------------------------
      Walk<Units8<T>> walk;
      walk.start(k);
      unsigned bits = 0;
      uint32_t tile = 0;
      bool ok = true, begun = false;
      for (uint32_t seg = 0; ok; ++seg) {
        if (seg >= kSegs8 && !(ok = warp_wait(s, &s->seg_empty[seg % kSegs8], (seg / kSegs8 - 1) & 1u, status))) break;
        const bool more = walk.next(k);
        if (!begun && lane == 0 && !k.join_inside) {
          const bool cut = more && walk.first_cut;
          int4 *rec = reinterpret_cast<int4 *>(&k.w.cuts[blockIdx.x]);
          rec[0] = cut ? make_int4(walk.t.row0 + walk.tokens0, walk.rows, walk.head, walk.more) : make_int4(0, 0, 0, 0);
          rec[1] = make_int4(more ? walk.t.flags : 0, 0, 0, 0);
        }
        begun = true;
        Seg8 w{};
        w.flags = kEnd8;
        if (more) {
          w = {walk.t.row0 + walk.tokens0, walk.rows, walk.tokens0, walk.t.seq, walk.head, walk.t.kv0 + walk.i0 * kTile8,
               walk.n, walk.t.ctx, walk.t.kv1, 0, walk.owner | walk.more << 16, 0};
          w.flags = (walk.t.flags & kShared) | ((walk.t.flags & kSolo) && walk.n == walk.t.tiles ? kWhole8 : 0) |
                    (walk.i0 == 0 ? kBase8 : 0);
        }
        if (lane == 0) {
          int4 *to = reinterpret_cast<int4 *>(&s->seg[seg % kSegs8]);
          to[0] = make_int4(w.row0, w.rows, w.i0, w.seq);
          to[1] = make_int4(w.head, w.t0, w.n, w.ctx);
          to[2] = make_int4(w.kv1, w.flags, w.join, 0);
        }
        warp_arrive(&s->seg_full[seg % kSegs8], lane);
        if (!more) break;
        // the tiles
        const int head = unit_heads<Units8<T>>(k, w.head).key, t_end = min(w.t0 + w.n * kTile8, w.kv1);
        const int32_t *table = k.a.b.tables + static_cast<int64_t>(w.seq) * k.a.b.T;
        auto place = [&](int t) {  // (block, token in it)
          const int slot = block_of(k, t);
          int id = table[slot];
          if (id < 0 || id >= c8.blocks) {
            bits |= SMC_DEV_BAD_BLOCK;
            id = 0;
          }
          return make_int2(id, t - slot * c8.block_size);
        };
        // places of 32 boxes, a lane each, and of the 32 after them
        const int box_log2 = 31 - __clz(k.box), per_tile = kTile8 >> box_log2;
        int2 here = make_int2(0, 0), ahead = make_int2(0, 0);
        int from = -32;
        if constexpr (kTma) {
          if (lane * k.box < t_end - w.t0) ahead = place(w.t0 + lane * k.box);
        }
        for (int i = 0; i < w.n; ++i, ++tile) {
          const uint32_t slot = tile & 1u, turn = tile >> 1 & 1u;
          const int t0 = w.t0 + i * kTile8, t1 = min(t0 + kTile8, t_end);
          char *const to_k = smem + M::kK + slot * kTileBytes8, *const to_v = smem + M::kV + slot * kTileBytes8;
          // scales of tokens lane, lane + 32, ...: on their way while slots are waited for
          float ks[4], vs[4];
          auto scales_of = [&](int e, int block) {
            const int64_t from = block * k.sc8.block + head * k.sc8.head;
            ks[e] = k.sc8.k[from];
            vs[e] = k.sc8.v[from];
          };
          if constexpr (kTma) {
            if ((i + 1) * per_tile > from + 32) {
              from = i * per_tile;
              here = ahead;
              const int on = (32 + lane) * k.box;  // (t0 + on may be past what 32 bits count)
              if (on < t_end - t0) ahead = place(t0 + on);
            }
            const int boxes = (t1 - t0 + k.box - 1) / k.box, mine = i * per_tile - from + lane;
            const int block = __shfl_sync(0xffffffffu, here.x, mine & 31), token = __shfl_sync(0xffffffffu, here.y, mine & 31);
            // (a token past the last one has its box's block, or the one of some box before: a block of the cache)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              scales_of(e, __shfl_sync(0xffffffffu, here.x, (i * per_tile - from + ((lane + 32 * e) >> box_log2)) & 31));
            }
#pragma unroll
            for (int which = 0; which < 2; ++which) {
              uint64_t *full = which ? &s->v_full[slot] : &s->k_full[slot];
              if (!(ok = warp_wait(s, which ? &s->v_empty[slot] : &s->k_empty[slot], turn ^ 1u, status))) break;
              if (lane == 0) mbar_arrive_expect_tx(full, boxes * k.box * 128);
              __syncwarp();
              if (lane < boxes) {
                tma_load_4d((which ? to_v : to_k) + lane * k.box * 128, which ? &map_v : &map_k, 0, token, head, block, full);
              }
              __syncwarp();
            }
          } else {
            // lane l finds rows l, l + 32, ...; a copy's lanes take their rows' places
            int64_t off[4] = {0, 0, 0, 0};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const bool in = t0 + lane + 32 * e < t1;
              const int2 p = in ? place(t0 + lane + 32 * e) : make_int2(0, 0);
              scales_of(e, p.x);
              if (in) {
                off[e] = p.x * c8.block_stride + p.y * c8.token_stride + head * c8.head_stride;
              }
            }
            const int chunk = lane & 7;
            const bool take = chunk * 16 < D;
#pragma unroll
            for (int which = 0; which < 2; ++which) {
              if (!(ok = warp_wait(s, which ? &s->v_empty[slot] : &s->k_empty[slot], turn ^ 1u, status))) break;
              const char *column = (which ? c8.v : c8.k) + (take ? chunk * 16 : 0);
              const uint32_t to = smem_addr(which ? to_v : to_k);
#pragma unroll
              for (int e = 0; e < 4; ++e) {
#pragma unroll
                for (int r = lane >> 3; r < 32; r += 4) {
                  const int64_t from_row = __shfl_sync(0xffffffffu, off[e], r);
                  const int row = r + 32 * e;
                  if (t0 + row < t1) cp_async16(to + row * 128 + ((chunk ^ (row & 7)) << 4), column + from_row, take);
                }
              }
              asm volatile("cp.async.commit_group;" ::: "memory");
              if (which) {  // K has arrived
                asm volatile("cp.async.wait_group 1;" ::: "memory");
                fence_proxy_async_smem();
                warp_arrive(&s->k_full[slot], lane);
                asm volatile("cp.async.wait_group 0;" ::: "memory");
                fence_proxy_async_smem();
                warp_arrive(&s->v_full[slot], lane);
              }
            }
            if (!ok) asm volatile("cp.async.wait_all;" ::: "memory");
          }
          if (!ok) break;
          // (V's slot is free when all of the softmax has read the scales of its last tile)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float sv = scale_of(vs[e]);
            s->token[slot][lane + 32 * e] = make_float4(k.sc * scale_of(ks[e]), fast_log2(sv), kSumScale * fast_rcp(sv), 0.f);
          }
          warp_arrive(&s->s_full[slot], lane);
        }
      }
      if (kTma && s->abort) {  // copies that may be under way
        for (uint32_t t = tile < 2 ? 0 : tile - 2; t <= tile; ++t) {
          mbar_wait(&s->k_full[t & 1u], t >> 1 & 1u, 1u << 12);
          mbar_wait(&s->v_full[t & 1u], t >> 1 & 1u, 1u << 12);
        }
      }
      if (bits) raise_status(status, bits);
    }
  }
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_free<256>(tmem);
  }
}

// ---------------------------------------------------------------------------
// Launch.
// ---------------------------------------------------------------------------
// [blocks][kv_heads][block_size][head_dim] in boxes of 128 bytes x `box` tokens;
// columns past head_dim read as 0.
static bool make_map8(CUtensorMap *map, const CacheArgs &c, void *base, int box) {
  const EncodeFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(c.head_dim), static_cast<cuuint64_t>(c.block_size),
                              static_cast<cuuint64_t>(c.kv_heads), static_cast<cuuint64_t>(c.blocks)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(c.token_stride), static_cast<cuuint64_t>(c.head_stride),
                                 static_cast<cuuint64_t>(c.block_stride)};
  const cuuint32_t boxes[4] = {128, static_cast<cuuint32_t>(box), 1, 1};
  const cuuint32_t steps[4] = {1, 1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, base, dims, strides, boxes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T>
static const void *attention8_fn(bool tma) {
  return tma ? reinterpret_cast<const void *>(attention8_kernel<T, true>)
             : reinterpret_cast<const void *>(attention8_kernel<T, false>);
}

static cudaError_t configure8(int *ctas) {
  constexpr int kMaxDev = 64;
  static std::atomic<int> known[kMaxDev];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const int slot = dev < kMaxDev ? dev : kMaxDev - 1;
  *ctas = dev < kMaxDev ? known[slot].load(std::memory_order_acquire) : 0;
  if (*ctas) return cudaSuccess;
  for (const bool tma : {false, true}) {
    e = cudaFuncSetAttribute(attention8_fn<__nv_bfloat16>(tma), cudaFuncAttributeMaxDynamicSharedMemorySize,
                             Smem8<__nv_bfloat16>::kBytes);
    if (e != cudaSuccess) return e;
    e = cudaFuncSetAttribute(attention8_fn<__half>(tma), cudaFuncAttributeMaxDynamicSharedMemorySize,
                             Smem8<__half>::kBytes);
    if (e != cudaSuccess) return e;
  }
  int n = 0;
  e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  n *= kCtasPerSm;
  *ctas = n < kMaxCtas8 ? n : kMaxCtas8;
  if (dev < kMaxDev) known[slot].store(*ctas, std::memory_order_release);
  return cudaSuccess;
}

template <typename T>
static cudaError_t launch8(const AttnArgs &a, const ScaleArgs &s, void *workspace, int most_ctas, cudaStream_t st) {
  constexpr int kRows = Rows8<T>::kRows;
  Kernel8Args k{};
  k.a = a;
  k.sc8 = s;
  // as for 16 bits: shared blocks are read once where reading them again would not be the L2 cache's work
  const double table_bytes = static_cast<double>(a.b.S) * a.b.T * a.c.block_size * a.c.kv_heads * a.c.head_dim * 2;
  if (table_bytes < 96e6) k.a.b.group = 1;
  carve(a.c, k.a.b, a.q_heads, kMaxCtas8, 64, static_cast<char *>(workspace), &k.w);
  k.rep = a.q_heads / a.c.kv_heads;
  const int parts = (k.rep + kRows - 1) / kRows;
  k.head_units = a.c.kv_heads * parts;
  k.unit_rep = (k.rep + parts - 1) / parts;
  k.tile_tokens = kRows / k.unit_rep;
  k.sc = a.scale * 1.4426950408889634f;
  divide_by(a.c.block_size, &k);
  // a box is a run of tokens inside one block and one tile; the swizzle repeats every eight rows, so a box
  // starts on a multiple of eight.  Blocks of other sizes are copied by a warp's lanes, 16 bytes each
  int box = kTile8;
  while (a.c.block_size % box) box >>= 1;
  CUtensorMap map_k{}, map_v{};
  const bool tma = box >= 8 && make_map8(&map_k, a.c, a.c.k, box) && make_map8(&map_v, a.c, a.c.v, box);
  k.box = box;
  // no more CTAs than tiles there can be
  const int64_t units = a.b.S * ((static_cast<int64_t>(a.b.max_new) + k.tile_tokens - 1) / k.tile_tokens);
  const int64_t most = (static_cast<int64_t>(a.b.T) * a.c.block_size + kTile8 - 1) / kTile8 * k.head_units * units;
  const int ctas = most < most_ctas ? static_cast<int>(most) : most_ctas;
  k.planned = k.w.groups > 0 || a.b.S > 256;
  const int64_t most_rows = static_cast<int64_t>(a.b.max_new) * k.a.b.group * k.unit_rep;
  const int unit_rows = static_cast<int>(most_rows < kRows ? most_rows : kRows);
  k.join_inside = !k.w.groups && unit_rows * (ctas / k.head_units + 2) <= 1024;
  k.more_kernels = k.w.groups > 0 || (ctas > 1 && !k.join_inside);
  cudaError_t e;
  void *work[] = {static_cast<WorkArgs *>(&k)};
  if (k.planned) {
    int n = ctas;
    void *args[] = {static_cast<WorkArgs *>(&k), &n};
    e = launch_early(reinterpret_cast<const void *>(plan_kernel<Units8<T>>), dim3(k.w.groups ? k.w.groups : 1),
                     kPlanThreads, 0, args, st);
    if (e != cudaSuccess) return e;
  }
  void *args[] = {&k, &map_k, &map_v};
  e = launch_early(attention8_fn<T>(tma), dim3(ctas), kThreads8, Smem8<T>::kBytes, args, st);
  if (e != cudaSuccess) return e;
  if (ctas > 1 && !k.join_inside) {
    e = launch_early(reinterpret_cast<const void *>(join_cut_units_kernel<T, Units8<T>>),
                     dim3(ctas - 1, (unit_rows + kJoinWarps - 1) / kJoinWarps), 32 * kJoinWarps, 0, work, st);
    if (e != cudaSuccess) return e;
  }
  if (!k.w.groups) return cudaSuccess;
  return launch_early(reinterpret_cast<const void *>(join_shared_kernel<T>), dim3(a.b.rows), 32 * kJoinWarps, 0, work, st);
}

cudaError_t launch_tree_attention8(const AttnArgs &a, const ScaleArgs &s, int dtype, void *workspace, cudaStream_t st) {
  if (a.b.rows == 0) return cudaSuccess;
  int ctas = 0;
  const cudaError_t e = configure8(&ctas);
  if (e != cudaSuccess) return e;
  return dtype == SMC_BF16 ? launch8<__nv_bfloat16>(a, s, workspace, ctas, st) : launch8<__half>(a, s, workspace, ctas, st);
}

}  // namespace smcsd

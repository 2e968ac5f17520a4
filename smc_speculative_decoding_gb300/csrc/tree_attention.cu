// Attention of each sequence's new tokens over its paged cache, under a tree
// mask (smc_tree_attention in smcsd.h).
//
// Three kernels, chained by programmatic dependent launch:
//   plan_kernel       lists the call's work in tiles of 64 tokens;
//   attention_kernel  persistent, one CTA per SM, on the 5th-generation tensor
//                     cores; every CTA takes an equal run of the tiles;
//   join_cut_units_kernel  joins the rows that several CTAs contributed to
//                     (with few rows the last of these CTAs does);
//   join_shared_kernel  behind it, joins a shared and an own part.
// Measured (bf16, 8 key heads of 128): 64 trees of 16 tokens over up to 8192,
// 32 heads, 264 to 270 us (6.1 to 6.3 TB/s); 8 tokens of 64 heads over 131072,
// 93 us (5.8 TB/s); 16 trees of 64 tokens over up to 4096, 90 us, bound by the
// softmax; one token over 513, 12 us, bound by latency.
#include <cuda.h>

#include <atomic>

#include "cache_common.cuh"

namespace smcsd {

// ---------------------------------------------------------------------------
// Work.  An *entry* is a run of consecutive rows and a range of tokens that
// they all attend: the own part of one sequence, or the part that the
// sequences of a prompt share (their leading equal table slots).  Per key
// head and per two row tiles an entry makes one *unit* of ceil(tokens / 64)
// tiles.  A row tile is floor(128 / rep) new tokens times the rep query heads
// of the key head, so a tile starts on a token.  The units' tiles form one
// line; CTA c takes tiles [c * per, (c + 1) * per) of it, so ragged lengths
// load every SM alike.  A unit's first tiles' CTA owns the unit's result;
// every later CTA of the unit has exactly one such continuation (its first
// segment) and stores it in its own slot.
// ---------------------------------------------------------------------------
constexpr int kTile = 64;         // tokens per tile
constexpr int kRows = 128;        // rows of a tensor-core tile
constexpr int kUnitRows = 256;    // most rows of a unit: two tensor-core tiles of 128
constexpr int kMaxCtas = 192;     // slots for continuations
constexpr int kPlanThreads = 1024;
constexpr uint32_t kWaitPolls = 1u << 17;  // each may suspend up to 20 us

struct Entry {
  int row0;    // first row
  int tokens;  // rows of one query head
  int seq;     // whose table
  int kv0, kv1;
  int ctx;     // tokens before ctx are seen by every row
  int tiles;   // per unit
  int flags;
};
constexpr int kShared = 1, kSolo = 2;  // a shared part; the rows have no other part

// The unit that the boundary before a CTA is the first to cut.
struct Cut {
  int row0, rows, head, more;  // first row, rows of the unit (0: no such unit), key head,
  int flags, pad[3];           // continuations; the entry's flags
};

struct PlanHeader {
  unsigned ticket;  // plan CTAs done; returns to zero
  int total, per;   // tiles, tiles per CTA
};

struct AttnWorkspace {
  PlanHeader *head;
  unsigned *tickets;  // [kMaxCtas] parts stored of the unit that a CTA's end cuts; return to zero
  int *common;     // [groups] shared tokens
  int *ref;        // [groups] the sequence by whose table they are read
  int *tile0;      // [entries + 1]
  Entry *entries;  // shared parts of the groups (when group > 1), then the sequences
  float *lse[2];   // own, shared: [rows * q_heads], log2
  float *o[2];     // [rows * q_heads][head_dim], normalised
  Cut *cuts;       // [kMaxCtas]
  float *lse_c;    // [kMaxCtas][kUnitRows] continuations
  float *o_c;      // [kMaxCtas][kUnitRows][head_dim]
  int groups;      // 0 when group == 1
  int n_entries;
};

static size_t carve(const CacheArgs &c, const BatchArgs &b, int q_heads, char *base,
                    AttnWorkspace *w) {
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off = (off + bytes + 255) / 256 * 256;
    return base + at;
  };
  AttnWorkspace t{};
  const size_t rh = static_cast<size_t>(b.rows) * q_heads, D = c.head_dim;
  t.groups = b.group > 1 ? b.S / b.group : 0;
  t.n_entries = b.S + t.groups;
  take(kCacheStatusBytes);
  t.head = reinterpret_cast<PlanHeader *>(take(sizeof(PlanHeader)));
  t.tickets = reinterpret_cast<unsigned *>(take(sizeof(unsigned) * kMaxCtas));
  t.common = reinterpret_cast<int *>(take(sizeof(int) * t.groups));
  t.ref = reinterpret_cast<int *>(take(sizeof(int) * t.groups));
  t.tile0 = reinterpret_cast<int *>(take(sizeof(int) * (static_cast<size_t>(t.n_entries) + 1)));
  t.entries = reinterpret_cast<Entry *>(take(sizeof(Entry) * t.n_entries));
  for (int k = 0; k < 2; ++k) {
    const size_t n = k == 0 || t.groups ? rh : 0;
    t.lse[k] = reinterpret_cast<float *>(take(sizeof(float) * n));
    t.o[k] = reinterpret_cast<float *>(take(sizeof(float) * n * D));
  }
  t.cuts = reinterpret_cast<Cut *>(take(sizeof(Cut) * kMaxCtas));
  t.lse_c = reinterpret_cast<float *>(take(sizeof(float) * kMaxCtas * kUnitRows));
  t.o_c = reinterpret_cast<float *>(take(sizeof(float) * kMaxCtas * kUnitRows * D));
  if (w) *w = t;
  return off;
}

size_t attention_workspace_bytes(const CacheArgs &c, const BatchArgs &b, int q_heads) {
  return carve(c, b, q_heads, nullptr, nullptr);
}

struct KernelArgs {
  AttnArgs a;
  AttnWorkspace w;
  int rep;      // query heads per key head, at most 128
  int tile_tokens;  // new tokens of a row tile: floor(128 / rep)
  int q_box;    // new tokens of a copied box of Q
  int planned;      // plan_kernel has run (else each CTA finds its own work)
  int more_kernels; // joins follow (a call's last kernel lets nothing start before its end)
  int join_inside;  // the last CTA of a cut unit joins its parts
  int box;      // tokens per copied box
  uint32_t magic, shift;  // t / block_size == umulhi(t, magic) >> shift
  float sc;     // scale * log2 e
};

// ---------------------------------------------------------------------------
// plan_kernel: the tokens that each prompt's sequences share, then (the last
// CTA to finish) the entries and the prefix of their tiles.
// ---------------------------------------------------------------------------
__device__ int block_scan_excl(int v, int *warps, int *total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += up;
  }
  if (lane == 31) warps[warp] = incl;
  __syncthreads();
  int before = 0, all = 0;
  for (int k = 0; k < kPlanThreads / 32; ++k) {
    if (k < warp) before += warps[k];
    all += warps[k];
  }
  __syncthreads();
  *total = all;
  return before + incl - v;
}

// Units of one key head: row tiles of an entry, two by two.
__device__ __forceinline__ int unit_tiles(const KernelArgs &k, int tokens) {
  return (tokens + 2 * k.tile_tokens - 1) / (2 * k.tile_tokens);
}

__device__ __forceinline__ int entry_tiles(const KernelArgs &k, int tokens, int kv0, int kv1,
                                           int *per_unit) {
  *per_unit = (kv1 - kv0 + kTile - 1) / kTile;
  if (tokens <= 0 || kv1 <= kv0) return 0;
  return *per_unit * k.a.c.kv_heads * unit_tiles(k, tokens);
}

__device__ int make_entry(const KernelArgs &k, int e, Entry *out) {
  const BatchArgs &b = k.a.b;
  const int bs = k.a.c.block_size;
  Entry t{};
  int tiles;
  if (e < k.w.groups) {
    const int s0 = e * b.group;
    const int shared = __ldcg(&k.w.common[e]);
    if (shared > 0) {  // every sequence is in order, so the rows are consecutive
      const SeqInfo first = seq_info(b, bs, s0), last = seq_info(b, bs, s0 + b.group - 1);
      // (a sequence without rows has no part in what the others share: the first one's table may be another)
      t = {first.row0, last.row0 + last.n - first.row0, __ldcg(&k.w.ref[e]), 0, shared, shared, 0, kShared};
    }
    tiles = entry_tiles(k, t.tokens, 0, shared, &t.tiles);
  } else {
    const int s = e - k.w.groups;
    const SeqInfo si = seq_info(b, bs, s);
    if (si.bits) raise_status(k.a.status, si.bits);
    const int shared = k.w.groups ? __ldcg(&k.w.common[s / b.group]) : 0;
    t = {si.row0, si.n, s, shared, si.len, si.len - si.n, 0, shared ? 0 : kSolo};
    tiles = entry_tiles(k, t.tokens, t.kv0, t.kv1, &t.tiles);
  }
  if (out) *out = t;
  return tiles;
}

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const __grid_constant__ KernelArgs k, int ctas) {
  __shared__ int warps[kPlanThreads / 32];
  __shared__ int s_slots, s_limit, s_seqs, s_bad, s_ref;
  __shared__ bool s_last;
  const int tid = threadIdx.x;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  wait_for_stream();
  const BatchArgs &b = k.a.b;
  const int bs = k.a.c.block_size;
  if (k.w.groups) {
    const int s0 = blockIdx.x * b.group;
    if (tid == 0) {
      s_limit = 0x7fffffff;
      s_seqs = s_bad = 0;
      s_ref = 0x7fffffff;
    }
    __syncthreads();
    for (int i = tid; i < b.group; i += kPlanThreads) {
      const SeqInfo si = seq_info(b, bs, s0 + i);
      if (si.bits) s_bad = 1;
      if (si.n > 0) {
        atomicMin(&s_limit, si.len - si.n);
        atomicAdd(&s_seqs, 1);
        atomicMin(&s_ref, s0 + i);
      }
    }
    __syncthreads();
    if (tid == 0) s_slots = s_seqs > 1 && !s_bad ? s_limit / bs : 0;
    __syncthreads();
    const int slots = s_slots;
    if (slots > 0) {  // a warp per sequence, against the first one that has rows
      const int32_t *ref = b.tables + static_cast<int64_t>(s_ref) * b.T;
      int mine = slots;
      for (int i = s_ref - s0 + 1 + (tid >> 5); i < b.group; i += kPlanThreads / 32) {
        if (b.row_start && b.row_start[s0 + i] == b.row_start[s0 + i + 1]) continue;  // no rows
        const int32_t *row = b.tables + static_cast<int64_t>(s0 + i) * b.T;
#pragma unroll 4
        for (int t = tid & 31; t < slots; t += 32) {
          if (row[t] != ref[t]) mine = min(mine, t);
        }
      }
      if (mine < slots) atomicMin(&s_slots, mine);
    }
    __syncthreads();
    if (tid == 0) {
      const int64_t tokens = static_cast<int64_t>(s_slots) * bs;
      k.w.common[blockIdx.x] = static_cast<int>(tokens / kTile * kTile);
      k.w.ref[blockIdx.x] = s_ref;
      __threadfence();
      s_last = atomicAdd(&k.w.head->ticket, 1) + 1 == gridDim.x;
    }
    __syncthreads();
    if (!s_last) return;
    if (tid == 0) k.w.head->ticket = 0;
    __threadfence();
  }
  // the prefix of the tiles: thread t takes a run of entries
  const int run = (k.w.n_entries + kPlanThreads - 1) / kPlanThreads;
  const int e0 = min(tid * run, k.w.n_entries), e1 = min(e0 + run, k.w.n_entries);
  int mine = 0;
  for (int e = e0; e < e1; ++e) {
    Entry t;
    mine += make_entry(k, e, &t);
    k.w.entries[e] = t;
  }
  int total;
  int at = block_scan_excl(mine, warps, &total);
  for (int e = e0; e < e1; ++e) {
    k.w.tile0[e] = at;
    const Entry &t = k.w.entries[e];
    int unused;
    at += entry_tiles(k, t.tokens, t.kv0, t.kv1, &unused);
  }
  if (tid == 0) {
    k.w.tile0[k.w.n_entries] = total;
    k.w.head->total = total;
    k.w.head->per = max(1, (total + ctas - 1) / ctas);
  }
}

// ---------------------------------------------------------------------------
// Tensor-core and tensor-memory primitives (PTX for sm_103a).
// ---------------------------------------------------------------------------
__device__ __forceinline__ void tmem_alloc_512(uint32_t *dst) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(
                   smem_addr(dst))
               : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free_512(uint32_t base) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(base) : "memory");
}
__device__ __forceinline__ void tc_fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_commit(uint64_t *bar) {
  asm volatile(
      "tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
          smem_addr(bar))
      : "memory");
}
// Shared-memory operand in 128-byte-swizzled rows of 64 elements: `lbo` bytes
// between 64-element panels (of the contiguous axis, MN-major operands only),
// 1024 bytes between groups of eight rows.  Only the low word of a descriptor
// varies.  The products take it as 32 bits and are issued by an elected
// thread: with 64-bit descriptors in an unrolled `lane == 0` branch the
// compiled code used wrong addresses for all but the first step.
constexpr uint32_t kDescHigh = 1024u >> 4 | 1u << 14 | 2u << 29;  // version, swizzle
__device__ __forceinline__ uint32_t smem_desc(uint32_t addr, uint32_t lbo) {  // low word
  return (addr & 0x3ffffu) >> 4 | (lbo >> 4) << 16;
}
// D[tmem] (+)= A[smem] * B[smem]
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 da, db;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 da, {%1, %5};\n\tmov.b64 db, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], da, db, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"(kDescHigh)
      : "memory");
}
// D[tmem] (+)= A[tmem] * B[smem]
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 db;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 db, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], db, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"(kDescHigh)
      : "memory");
}
__device__ __forceinline__ bool elect_one() {
  uint32_t yes;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(yes));
  return yes != 0;
}
#define SMC_R8(r, i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3]), "=r"(r[i + 4]), \
                     "=r"(r[i + 5]), "=r"(r[i + 6]), "=r"(r[i + 7])
#define SMC_I8(r, i) "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3]), "r"(r[i + 4]), \
                     "r"(r[i + 5]), "r"(r[i + 6]), "r"(r[i + 7])
// 32 columns of the calling warp's 32 lanes: thread = lane, register = column.
__device__ __forceinline__ void tmem_ld32(uint32_t addr, uint32_t *r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : SMC_R8(r, 0), SMC_R8(r, 8), SMC_R8(r, 16), SMC_R8(r, 24)
      : "r"(addr));
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::
          SMC_I8(r, 0),
      SMC_I8(r, 8), SMC_I8(r, 16), SMC_I8(r, 24), "r"(addr)
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::SMC_I8(r, 0),
      SMC_I8(r, 8), "r"(addr)
      : "memory");
}
// Waits for the warp's loads.  The registers of a load count as written only
// here, so that no use of them moves ahead of the wait.
#define SMC_T8(r, i) "+r"(r[i]), "+r"(r[i + 1]), "+r"(r[i + 2]), "+r"(r[i + 3]), "+r"(r[i + 4]), \
                     "+r"(r[i + 5]), "+r"(r[i + 6]), "+r"(r[i + 7])
__device__ __forceinline__ void tmem_wait_ld(uint32_t *r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : SMC_T8(r, 0), SMC_T8(r, 8), SMC_T8(r, 16), SMC_T8(r, 24)::"memory");
}
__device__ __forceinline__ void tmem_tie(uint32_t *r) {
  asm volatile("" : SMC_T8(r, 0), SMC_T8(r, 8), SMC_T8(r, 16), SMC_T8(r, 24));
}
__device__ __forceinline__ void tmem_wait_st() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
// kind::f16 with 128 rows, n columns, fp32 accumulators; b_mn: B is stored
// with its n axis contiguous.
__host__ __device__ constexpr uint32_t instr_desc(bool bf16, int n, bool b_mn) {
  return 1u << 4 | (bf16 ? 1u << 7 | 1u << 10 : 0u) | (b_mn ? 1u << 16 : 0u) |
         static_cast<uint32_t>(n >> 3) << 17 | (128u >> 4) << 24;
}
__device__ __forceinline__ void tma_load_4d(void *dst, const CUtensorMap *map, int d, int token,
                                            int head, int block, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_addr(dst)),
      "l"(map), "r"(smem_addr(bar)), "r"(d), "r"(token), "r"(head), "r"(block)
      : "memory");
}
__device__ __forceinline__ void prefetch_map(const CUtensorMap *map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
__device__ __forceinline__ void tma_load_3d(void *dst, const CUtensorMap *map, int d, int head,
                                            int row, uint64_t *bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_addr(dst)),
      "l"(map), "r"(smem_addr(bar)), "r"(d), "r"(head), "r"(row)
      : "memory");
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool take) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(take ? 16 : 0)
               : "memory");
}

// Eight words to a 32-byte boundary, one whole sector a thread.
__device__ __forceinline__ void store_32_bytes(void *dst, const uint32_t *x) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(x[0]),
               "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
               : "memory");
}

template <typename T>
struct Weights;
template <>
struct Weights<__nv_bfloat16> {
  static constexpr bool kBf16 = true;
  // weights are 2^(z - m), m at most kLazy below the running maximum
  static constexpr float kOffset = 0.f;
  static constexpr uint32_t kExpMask = 0x7f807f80u;
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
  }
};
template <>
struct Weights<__half> {
  static constexpr bool kBf16 = false;
  // fp16 has 2^-24 .. 65504: weights are scaled by 2^7, so that with kLazy
  // they stay below 2^15 and small ones keep 7 more bits
  static constexpr float kOffset = 7.f;
  static constexpr uint32_t kExpMask = 0x7c007c00u;
  static __device__ __forceinline__ uint32_t pack(float a, float b) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
  }
};
// The accumulators are rescaled only when the running maximum (log2) rises
// by more than this; until then weights may reach 2^kLazy.
constexpr float kLazy = 8.f;

// ---------------------------------------------------------------------------
// attention_kernel.  Warps 0-3 and 4-7: two softmax groups (thread = row of a
// row tile); warps 8 and 9: the threads that issue either group's matrix
// products; warp 10 finds the CTA's segments (parts of units) for all and
// copies K; warp 11 copies Q and V.  Shared memory: two Q tiles and a ring
// each of K and V tiles.  Tensor memory, per group: a tile's scores (64
// columns), two tiles' weights (32 each) and the accumulator (128).
//   Units of one row tile: the groups take alternate tiles of the unit, each
//   with its own running maximum, sum and accumulator, joined at the end.
//   Two such units about as long, one after the other: a group each, so that
//   their ends overlap and nothing is joined.  With 20 of the tile's 128 rows
//   in use a tile takes the one softmax warp 2900 cycles and a segment's end
//   10000, whatever its length: 256 sequences of 300 to 640 own tokens took 382
//   us one by one and 273 so; 256 of one token and 100 to 1024 tokens 276 and
//   197; 512 of 150 to 300 tokens 375 and 260.
//   Units of two: each group has its own row tile; a tile of K and V serves
//   both.
// A group takes its scores to registers at once, so the next tile's scores are
// computed beside its softmax (and the next segment's beside the write of a
// result), and the product with V of one tile beside the softmax of the next:
// a group waits for no product's latency.  With the weights in place of the
// scores, and the next scores behind the product with V, a tile of 256 rows
// took 2700 cycles, of which 1100 were that wait.
//   Every wait is on a barrier all of whose turns the waiting thread follows:
// a slot is one group's for good (see Geometry), and before both groups use a
// tile, all earlier tiles are done with.  tests/test_attention_protocol.py runs
// the roles and their barriers on the CPU.
// ---------------------------------------------------------------------------
constexpr int kAttnThreads = 384;
constexpr int kRingBytes = 160 * 1024;
constexpr int kSegs = 4;  // segments found ahead
// Two segments go side by side where their tiles differ by at most this: the
// serving workload 315, 323 and 332 us at 1, 3 and 8 in their first form,
// batches of 8k tokens 270, 270 and 294 us at 3, 8 and 64.
constexpr int kTwoGap = 3;

template <int kHalves>  // 64-element panels of the head dim
struct Geometry {
  static constexpr int kTileBytes = kHalves * kTile * 128;
  // Slots of K and of V: V waits for its weights, K does not.  Tile i of a
  // segment takes one of group i % 2's half of the slots (the even or the odd
  // ones) in turn.
  static constexpr int kSlotsK = 6 * (2 / kHalves), kSlotsV = 4 * (2 / kHalves);
  static constexpr int kQTile = kHalves * kRows * 128;
  static constexpr int kQBytes = 2 * kQTile;
  static constexpr int kTail = kQBytes + kRingBytes;
};

struct Seg {
  int row0, rows;  // first row of the unit, rows of it
  int i0;          // new token of the first row (own parts)
  int seq, head;
  int t0, n;       // first token, tiles
  int ctx, kv1;    // tokens before ctx are seen by all; end of the entry's tokens
  int n_new;       // new tokens of the sequence (own parts)
  int flags;
  int join;        // of a cut unit: the owner CTA, and continuations << 16; with kTwo the other's tiles
};
// with kShared: final result, first tiles, none left, two segments side by side, the last one was
constexpr int kWhole = 4, kBase = 8, kEnd = 16, kTwo = 32, kBehindTwo = 64;

struct AttnTail {
  uint64_t full[2][12], empty[2][12];  // K, V
  uint64_t seg_full[kSegs], seg_empty[kSegs];
  uint64_t q_full[2], q_free[2], scores[2], s_free[2], weights[2][2], o_full[2], o_free, stats, stored, counted;
  uint64_t drained[2];
  Seg seg[kSegs][2];  // either group's
  float2 stat[2][kRows];  // either group's (max, sum) of a row
  uint32_t tmem;
  unsigned nonfinite[2];  // segment number (from 1) of the last odd or even one with such a value
  volatile int abort;
  int joins;              // this CTA stored the last part of the unit
};

// A CTA's walk over its tiles: one segment (part of a unit) at a time.  All
// lanes of a warp walk together.
//   Without a plan, and with no more units than CTAs, the line may be laid out
// so that a CTA's run never crosses a unit: every unit's tiles are rounded up
// to a multiple of the run `per`, the least for which the runs suffice.  Each
// CTA then has one segment, and no unit is cut more often than it must.  It is
// taken where it lengthens the longest run by at most a tenth and two tiles.
// Measured, with equal runs and so: 8 sequences of 8 key heads and 11 tiles
// 26.9 and 18.8 us; 5 of 12 heads, 0 to 13 tiles, 21.9 and 16.3 us; one of 8
// heads and 2049 tiles 98.6 and 93.5 us.
struct Walk {
  int x, x1, per, e;
  Entry t;
  int base;       // tiles of the line before entry e
  int span;       // tiles of the line of each of its units
  bool aligned;
  int head, rt;   // unit
  int i0, n;      // tiles [i0, i0 + n) of the unit
  int tokens0;    // new token of the unit's first row
  int rows;       // rows of the unit

  __device__ __forceinline__ int span_of(int tiles) const {
    return aligned ? (tiles + per - 1) / per * per : tiles;
  }
  // units and tiles per unit of sequence e
  __device__ __forceinline__ int2 sequence_units(const KernelArgs &k, int e, unsigned *bits) {
    if (e >= k.w.n_entries) return make_int2(0, 0);
    const SeqInfo si = seq_info(k.a.b, k.a.c.block_size, e);
    *bits |= si.bits;
    if (si.n <= 0) return make_int2(0, 0);
    return make_int2(k.a.c.kv_heads * unit_tiles(k, si.n), (si.len + kTile - 1) / kTile);
  }
  __device__ __forceinline__ void start(const KernelArgs &k) {
    const int lane = threadIdx.x & 31;
    aligned = false;
    int total;
    if (k.planned) {
      per = __ldcg(&k.w.head->per);
      total = __ldcg(&k.w.head->total);
      x = min(static_cast<int>(blockIdx.x) * per, total);
      x1 = min(x + per, total);
      if (x >= x1) return;
      int lo = 0, hi = k.w.n_entries - 1;  // the last entry with tile0 <= x
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (__ldcg(&k.w.tile0[mid]) <= x) lo = mid; else hi = mid - 1;
      }
      e = lo;
    } else {
      // the entries are the sequences: a lane each, 32 at a time
      unsigned bits = 0;
      const int entries = k.w.n_entries, ctas = gridDim.x;
      int2 mine = make_int2(0, 0);
      int units = 0;
      total = 0;
      for (int s0 = 0; s0 < entries; s0 += 32) {
        mine = sequence_units(k, s0 + lane, &bits);
        units += mine.x;
        total += mine.x * mine.y;
      }
      units = __reduce_add_sync(0xffffffffu, units);
      total = __reduce_add_sync(0xffffffffu, total);
      if (bits && blockIdx.x == 0) raise_status(k.a.status, bits);
      per = max(1, (total + ctas - 1) / ctas);
      if (units <= ctas) {
        for (int run = max(per, 2); 10 * run <= 11 * per + 20; run += 1 + run / 32) {
          int runs = 0;
          for (int s0 = 0; s0 < entries; s0 += 32) {
            if (entries > 32) mine = sequence_units(k, s0 + lane, &bits);
            runs += mine.x * ((mine.y + run - 1) / run);
          }
          runs = __reduce_add_sync(0xffffffffu, runs);
          if (runs <= ctas) {
            per = run;
            total = runs * run;
            aligned = true;
            break;
          }
        }
      }
      x = min(static_cast<int>(blockIdx.x) * per, total);
      x1 = min(x + per, total);
      if (x >= x1) return;
      base = 0;
      for (int s0 = 0;; s0 += 32) {
        if (entries > 32) mine = sequence_units(k, s0 + lane, &bits);
        const int tiles = mine.x * span_of(mine.y);
        int incl = tiles;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int up = __shfl_up_sync(0xffffffffu, incl, o);
          if (lane >= o) incl += up;
        }
        const unsigned past = __ballot_sync(0xffffffffu, base + incl > x);
        if (past) {
          const int first = __ffs(past) - 1;
          e = s0 + first;
          base += __shfl_sync(0xffffffffu, incl - tiles, first);
          break;
        }
        base += __shfl_sync(0xffffffffu, incl, 31);
      }
    }
    load(k);
  }
  __device__ __forceinline__ void load(const KernelArgs &k) {
    if (k.planned) {
      const int4 *p = reinterpret_cast<const int4 *>(&k.w.entries[e]);
      const int4 a = __ldcg(p), b = __ldcg(p + 1);
      t = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
      base = __ldcg(&k.w.tile0[e]);
    } else {
      const SeqInfo si = seq_info(k.a.b, k.a.c.block_size, e);
      t = {si.row0, si.n, e, 0, si.len, si.len - si.n, (si.len + kTile - 1) / kTile, kSolo};
    }
    span = span_of(t.tiles);
  }
  __device__ __forceinline__ bool next(const KernelArgs &k) {
    if (x >= x1) return false;
    int rts;
    for (;;) {
      rts = unit_tiles(k, t.tokens);
      const int tiles = t.tokens > 0 && t.kv1 > t.kv0 ? rts * k.a.c.kv_heads * span : 0;
      if (x - base < tiles) break;
      base += tiles;
      ++e;
      load(k);
    }
    const int local = x - base, u = local / span;
    i0 = local - u * span;
    n = min(t.tiles - i0, x1 - x);
    head = u / rts;
    rt = u - head * rts;
    tokens0 = rt * 2 * k.tile_tokens;
    rows = min(t.tokens - tokens0, 2 * k.tile_tokens) * k.rep;
    // the unit's place on the line, in CTAs
    const int unit0 = x - i0;
    owner = unit0 / per;
    more = (unit0 + span - 1) / per - owner;
    first_cut = i0 > 0 && i0 <= per;
    x = aligned ? x1 : x + n;
    return true;
  }
  int owner, more;  // the CTA of the unit's first tiles; the CTAs after it
  bool first_cut;   // this segment begins at the first cut of its unit
};

// A ring's slots, tile by tile.  Either half of the slots (the even and the odd
// ones) is used in turn; `pos` and `parity` are the half's next slot and the
// parity of that slot's barriers.
template <int kSlots>
struct Ring {
  static constexpr uint32_t kHalf = kSlots / 2;
  uint32_t pos[2] = {0, 0}, parity[2] = {0, 0};
  __device__ __forceinline__ uint32_t at(bool odd) const {
    return odd ? 2 * pos[1] + 1 : 2 * pos[0];
  }
  __device__ __forceinline__ uint32_t par(bool odd) const { return odd ? parity[1] : parity[0]; }
  __device__ __forceinline__ void step(bool odd) {
    uint32_t &p = odd ? pos[1] : pos[0], &q = odd ? parity[1] : parity[0];
    if (++p == kHalf) {
      p = 0;
      q ^= 1u;
    }
  }
  // past n tiles of one half that this thread does not use
  __device__ __forceinline__ void skip(bool odd, uint32_t n) {
    uint32_t &p = odd ? pos[1] : pos[0], &q = odd ? parity[1] : parity[0];
    p += n;
    const uint32_t turns = p / kHalf;
    p -= turns * kHalf;
    q ^= turns & 1u;
  }
};

// Waits.  Every one is bounded, and gives up for the whole CTA: the one that
// ran out raises the status bit and the abort flag, at which the others end.
// What is done when a barrier has already completed is kept to a few
// instructions: each role's code runs once a tile, after other roles' code has
// displaced it from the instruction cache, and is paid for by its length.
__device__ __noinline__ bool wait_slowly(AttnTail *s, uint64_t *bar, uint32_t parity, unsigned *status) {
  for (uint32_t i = 0; i < kWaitPolls; ++i) {
    if (mbar_try_wait(bar, parity)) return true;
    if (s->abort) return false;
  }
  s->abort = 1;
  raise_status(status, SMC_DEV_TIMEOUT);
  return false;
}
__device__ __forceinline__ bool guarded_wait(AttnTail *s, uint64_t *bar, uint32_t parity, unsigned *status) {
  return mbar_try_wait(bar, parity) || wait_slowly(s, bar, parity, status);
}
// The same for a whole warp, in step: every lane polls and takes the same
// branch, so that the warp is converged for the .aligned instructions that
// follow.
__device__ __noinline__ bool warp_wait_slowly(AttnTail *s, uint64_t *bar, uint32_t parity, unsigned *status) {
  for (uint32_t i = 0; i < kWaitPolls; ++i) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    if (__any_sync(0xffffffffu, s->abort)) return false;
  }
  s->abort = 1;
  raise_status(status, SMC_DEV_TIMEOUT);
  return false;
}
__device__ __forceinline__ bool warp_wait(AttnTail *s, uint64_t *bar, uint32_t parity, unsigned *status) {
  return __all_sync(0xffffffffu, mbar_try_wait(bar, parity)) || warp_wait_slowly(s, bar, parity, status);
}
// One arrival for a warp (lane 0's), by predicate and not by a branch, for
// the same reason.  What the other lanes did before is ordered by __syncwarp.
__device__ __forceinline__ void warp_arrive(uint64_t *bar, int lane) {
  __syncwarp();
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.eq.s32 p, %1, 0;\n\t"
      "@p mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(smem_addr(bar)),
      "r"(lane)
      : "memory");
}

// Bits of a row's view of new tokens j0 .. j0 + 31: 1 for committed tokens
// (j < 0), the mask's bit or the chain's for new ones, 0 past them.
__device__ __forceinline__ uint32_t view_bits(const uint32_t *mask, int words, int i, int n_new,
                                              int j0) {
  if (j0 + 32 <= 0) return 0xffffffffu;
  if (j0 >= n_new) return 0u;
  uint32_t bits;
  if (mask) {
    const int w = j0 >> 5;
    const uint32_t lo = w < 0 ? 0xffffffffu : (w < words ? __ldg(mask + w) : 0u);
    const uint32_t hi = w + 1 < 0 ? 0xffffffffu : (w + 1 < words ? __ldg(mask + w + 1) : 0u);
    bits = __funnelshift_r(lo, hi, j0 & 31);
  } else {
    const int c = i - j0 + 1;  // new tokens 0..i
    bits = c <= 0 ? 0u : (c >= 32 ? 0xffffffffu : (1u << c) - 1u);
  }
  const int left = n_new - j0;
  if (left < 32) bits &= (1u << left) - 1u;
  return bits;
}

// A new token that holds an infinity or NaN had it zeroed in the products, as
// rows that do not see the token must not meet it.  Rows that see it get it
// here: columns [c0, c1) of the row's result whose visible new tokens in
// [t0, t1) hold such values become the sum of these.
template <typename T, typename Out>
__device__ __noinline__ void patch_nonfinite(const KernelArgs &k, int seq, int ctx, int n_new,
                                             int head, int row, int i, int t0, int t1, int c0,
                                             int c1, Out *o) {
  const uint32_t *mask = k.a.mask ? k.a.mask + static_cast<int64_t>(row) * k.a.mask_words : nullptr;
  const int32_t *table = k.a.b.tables + static_cast<int64_t>(seq) * k.a.b.T;
  for (int d = c0; d < c1; ++d) {
    float sum = 0.f;
    for (int at = max(t0, ctx); at < t1; ++at) {
      if (!(view_bits(mask, k.a.mask_words, i, n_new, at - ctx) & 1u)) continue;
      const int block = table[at / k.a.c.block_size];
      if (block < 0 || block >= k.a.c.blocks) continue;
      const T *v = reinterpret_cast<const T *>(k.a.c.v) + block * k.a.c.block_stride +
                   (at % k.a.c.block_size) * k.a.c.token_stride + head * k.a.c.head_stride;
      const float x = to_f32(v[d]);
      if (!(fabsf(x) < INFINITY)) sum += x;
    }
    if (sum != 0.f) o[d] = from_f32<Out>(sum);
  }
}

// ---------------------------------------------------------------------------
// Joining a row's parts: each part p has a log-sum-exp L_p (log2) and a
// normalised result o_p;
//   out = sum 2^(L_p - M) o_p / sum 2^(L_p - M),  M = max L_p.
// A warp joins a row, with as many parts' loads under way as it can.
// ---------------------------------------------------------------------------
constexpr int kJoinWarps = 8;

struct Joined {
  float top = -INFINITY, sum = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  __device__ __forceinline__ void raise(float to) {
    const float f = top == -INFINITY ? 0.f : fast_exp2(top - to);
    sum *= f;
    acc.x *= f;
    acc.y *= f;
    acc.z *= f;
    acc.w *= f;
    top = to;
  }
  __device__ __forceinline__ void add(float lse, float4 x) {  // lse <= top
    const float f = lse == -INFINITY ? 0.f : fast_exp2(lse - top);
    sum += f;
    acc.x = fmaf(f, x.x, acc.x);
    acc.y = fmaf(f, x.y, acc.y);
    acc.z = fmaf(f, x.z, acc.z);
    acc.w = fmaf(f, x.w, acc.w);
  }
  __device__ __forceinline__ float lse2() const { return sum == 0.f ? -INFINITY : top + log2f(sum); }
  __device__ __forceinline__ float4 result() const {
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    return make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
  }
};

__device__ __forceinline__ float4 load_part(const float *o, bool live) {
  return live ? __ldcg(reinterpret_cast<const float4 *>(o) + (threadIdx.x & 31))
              : make_float4(0.f, 0.f, 0.f, 0.f);
}

template <typename T>
__device__ __forceinline__ void write_row(const KernelArgs &k, int64_t rh, int row, int qh, const Joined &j) {
  const int lane = threadIdx.x & 31;
  const float4 x = j.result();
  if (4 * lane < k.a.c.head_dim) {
    T *dst = reinterpret_cast<T *>(k.a.out) + row * k.a.o_row + qh * k.a.o_head + 4 * lane;
    *reinterpret_cast<uint2 *>(dst) = make_uint2(Weights<T>::pack(x.x, x.y), Weights<T>::pack(x.z, x.w));
  }
  if (k.a.lse && lane == 0) k.a.lse[rh] = j.lse2() * 0.69314718055994531f;
}

// A row of a cut unit: its owner's part, and a continuation each of CTAs
// cta + 1 .. cta + more at row `slot` of their slots.
__device__ __forceinline__ Joined join_parts(const KernelArgs &k, int kind, int64_t rh, int cta, int more,
                                             int slot) {
  const int D = k.a.c.head_dim;
  const bool live = 4 * static_cast<int>(threadIdx.x & 31) < D;
  Joined j;
  float l = __ldcg(&k.w.lse[kind][rh]);
  float4 x = load_part(k.w.o[kind] + rh * D, live);
  const int64_t slot0 = static_cast<int64_t>(cta + 1) * kUnitRows + slot;
  constexpr int kBatch = 8;
  for (int p = 0; p < more; p += kBatch) {
    float ls[kBatch];
    float4 xs[kBatch];
    float top = fmaxf(j.top, l);
#pragma unroll
    for (int e = 0; e < kBatch; ++e) {
      const int64_t at = slot0 + static_cast<int64_t>(p + e) * kUnitRows;
      const bool in = p + e < more;
      ls[e] = in ? __ldcg(&k.w.lse_c[at]) : -INFINITY;
      xs[e] = load_part(k.w.o_c + at * D, live && in);
    }
#pragma unroll
    for (int e = 0; e < kBatch; ++e) top = fmaxf(top, ls[e]);
    j.raise(top);
    j.add(l, x);
    l = -INFINITY;
#pragma unroll
    for (int e = 0; e < kBatch; ++e) j.add(ls[e], xs[e]);
  }
  return j;
}

// Segment number `seg` (from 0) of a group as warp 10 left it.  False when the wait gave
// up or no segment is left.
__device__ __forceinline__ bool take_segment(AttnTail *s, uint32_t seg, int g, Seg *to, unsigned *status) {
  if (!warp_wait(s, &s->seg_full[seg % kSegs], seg / kSegs & 1u, status)) return false;
  const int4 *from = reinterpret_cast<const int4 *>(&s->seg[seg % kSegs][g]);
  const int4 a = from[0], b = from[1], c = from[2];
  *to = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w, c.x, c.y, c.z, c.w};
  return !(to->flags & kEnd);
}

// Copies the tiles of a segment, of K or of V, into their ring; with kTwo those
// of two segments, in turn.  `seg` is where warp 10 left either group's.
template <int kHalves, bool kTma, int kSlots>
__device__ __forceinline__ bool copy_tiles(const KernelArgs &k, const CUtensorMap *map, const char *src,
                                           char *slots, uint64_t *full, uint64_t *empty, AttnTail *s,
                                           Ring<kSlots> &ring, const Seg *seg, bool pair,
                                           unsigned *bits, uint32_t *filled, uint32_t *parities) {
  using G = Geometry<kHalves>;
  const int lane = threadIdx.x & 31;
  const CacheArgs &c = k.a.c;
  const uint32_t bs = c.block_size;
  const int per_tile = kTile / k.box;
  const bool two = seg->flags & kTwo;
  // (block, token in it) of token t of a segment's sequence
  auto place = [&](const Seg *of, uint32_t t) {
    const uint32_t b = bs == 1 ? t : __umulhi(t, k.magic) >> k.shift;
    int id = k.a.b.tables[static_cast<int64_t>(of->seq) * k.a.b.T + b];
    if (id < 0 || id >= c.blocks) {
      *bits |= SMC_DEV_BAD_BLOCK;
      id = 0;
    }
    return make_int2(id, t - b * bs);
  };
  // the places of boxes `from` + lane, of two segments half the lanes each
  int2 ahead = make_int2(0, 0);
  int from = -64;
  const int span = two ? 16 : 32;
  int unseen = -1;  // the slot whose element copies may still be under way
  bool ok = true;
  const int turns = two ? 2 * max(seg[0].n, seg[1].n) : seg->n;
  for (int turn = 0; turn < turns; ++turn) {
    const bool odd = turn & 1;
    const int i = two ? turn >> 1 : turn;
    const Seg *const mine = seg + odd;
    const int n = mine->n, head = mine->head, begin = mine->t0, end = min(begin + n * kTile, mine->kv1);
    const int t0 = begin + i * kTile, t1 = min(t0 + kTile, end);
    const uint32_t slot = ring.at(odd);
    char *dst = slots + slot * G::kTileBytes;
    if constexpr (kTma) {
      if ((i + 1) * per_tile > from + span) {
        from = i * per_tile;
        const Seg *const of = seg + (two ? lane >> 4 : 0);
        const int t = of->t0 + i * kTile + (lane & (span - 1)) * k.box;
        if (t < min(of->t0 + of->n * kTile, of->kv1)) ahead = place(of, t);
      }
    }
    if (i >= n) continue;
    // (the first turn of a fresh barrier passes for the one before it)
    if (!(ok = warp_wait(s, &empty[slot], ring.par(odd) ^ 1u, k.a.status))) break;
    if (!pair) warp_arrive(&empty[slot], lane);  // one group uses it
    *filled |= 1u << slot;
    *parities = (*parities & ~(1u << slot)) | ring.par(odd) << slot;
    ring.step(odd);
    if constexpr (kTma) {
      const int boxes = (t1 - t0 + k.box - 1) / k.box;
      const int at = i * per_tile - from + (two && odd ? 16 : 0);
      if (elect_one()) mbar_arrive_expect_tx(&full[slot], boxes * kHalves * k.box * 128);
      __syncwarp();
      for (int b = 0; b < boxes; ++b) {
        const int block = __shfl_sync(0xffffffffu, ahead.x, at + b);
        const int token = __shfl_sync(0xffffffffu, ahead.y, at + b);
        if (elect_one()) {
#pragma unroll
          for (int half = 0; half < kHalves; ++half) {
            tma_load_4d(dst + half * (kTile * 128) + b * k.box * 128, map, half * 64, token, head,
                        block, &full[slot]);
          }
        }
        __syncwarp();
      }
    } else {
      // lane l finds rows l and l + 32; a copy's lanes take their rows' places
      constexpr int kChunks = 8 * kHalves, kStep = 32 / kChunks;
      const int ch = lane % kChunks, r0 = lane / kChunks;
      const bool take = ch * 8 < c.head_dim;
      int64_t off[2] = {0, 0};
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        if (t0 + lane + 32 * e < t1) {
          const int2 at_block = place(mine, t0 + lane + 32 * e);
          off[e] = (at_block.x * c.block_stride + at_block.y * c.token_stride + head * c.head_stride) * 2;
        }
      }
      const char *column = src + (take ? ch * 16 : 0);
      const uint32_t d0 = smem_addr(dst) + (ch >> 3) * (kTile * 128);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll 8
        for (int r = r0; r < 32; r += kStep) {
          const int64_t from_row = __shfl_sync(0xffffffffu, off[e], r);
          const int row = r + 32 * e;
          if (t0 + row < t1) cp_async16(d0 + row * 128 + (((ch & 7) ^ (row & 7)) << 4), column + from_row, take);
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
      if (unseen >= 0) {  // the tile before this one has arrived
        asm volatile("cp.async.wait_group 1;" ::: "memory");
        fence_proxy_async_smem();
        warp_arrive(&full[unseen], lane);
      }
      unseen = slot;
    }
  }
  if constexpr (!kTma) {
    asm volatile("cp.async.wait_all;" ::: "memory");
    if (unseen >= 0) {
      fence_proxy_async_smem();
      warp_arrive(&full[unseen], lane);
    }
  }
  return ok;
}

// Waits until the last copy into each of a ring's slots has landed: a CTA that
// gave up may have left some under way.
__device__ __noinline__ void wait_landed(uint64_t *full, uint32_t filled, uint32_t parities) {
  for (uint32_t slot = 0; slot < 12; ++slot) {
    if (filled >> slot & 1u) mbar_wait(&full[slot], parities >> slot & 1u, 1u << 12);
  }
}

template <typename T, int kHalves, bool kTma>
__global__ void __launch_bounds__(kAttnThreads, 1)
attention_kernel(const __grid_constant__ KernelArgs k, const __grid_constant__ CUtensorMap map_q,
                 const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v) {
  using G = Geometry<kHalves>;
  using Wt = Weights<T>;
  extern __shared__ __align__(1024) char smem[];
  char *const s_q = smem;
  char *const s_k = smem + G::kQBytes, *const s_v = s_k + G::kSlotsK * G::kTileBytes;
  AttnTail *const s = reinterpret_cast<AttnTail *>(smem + G::kTail);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int D = k.a.c.head_dim;
  const int tile_rows = k.tile_tokens * k.rep;
  unsigned *const status = k.a.status;

  if (tid == 0) {
    for (int v = 0; v < 2; ++v) {
      for (int i = 0; i < (v ? G::kSlotsV : G::kSlotsK); ++i) {
        mbar_init(&s->full[v][i], 1);
        mbar_init(&s->empty[v][i], 2);  // both groups, or one and the copying warp
      }
    }
    for (int i = 0; i < kSegs; ++i) {
      mbar_init(&s->seg_full[i], 1);
      mbar_init(&s->seg_empty[i], 11);  // every warp but the one that fills it
    }
    for (int g = 0; g < 2; ++g) {
      mbar_init(&s->q_full[g], 1);
      mbar_init(&s->q_free[g], 2);
      for (int b = 0; b < 2; ++b) mbar_init(&s->weights[g][b], 4);
      mbar_init(&s->scores[g], 1);
      mbar_init(&s->s_free[g], 4);
      mbar_init(&s->o_full[g], 1);
      mbar_init(&s->drained[g], 1);
    }
    mbar_init(&s->o_free, 8);
    mbar_init(&s->stats, 8);
    mbar_init(&s->stored, 8);
    mbar_init(&s->counted, 1);
    s->nonfinite[0] = s->nonfinite[1] = 0;
    s->abort = (smem_addr(smem) & 1023u) != 0;  // the swizzle counts from 1 KB boundaries
    mbar_init_fence();
  }
  if (warp == 8) tmem_alloc_512(&s->tmem);
  if (warp == 9 && elect_one()) {
    prefetch_map(&map_q);
    if (kTma) {
      prefetch_map(&map_k);
      prefetch_map(&map_v);
    }
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
    // ---- softmax groups ---------------------------------------------------
    const int g = warp >> 2, wq = warp & 3;
    const int r = wq * 32 + lane;  // row of the group's tile
    const int r_tok = r / k.rep, r_head = r - r_tok * k.rep;
    const uint32_t lanes = static_cast<uint32_t>(wq * 32) << 16;
    const uint32_t t_s = tmem + lanes + g * 128, t_o = tmem + lanes + 256 + g * 128;
    uint32_t seg = 0, turn = 0, cuts = 0;  // segments, tiles of this group, cut units so far
    Ring<G::kSlotsV> ring_v;
    bool ok = true;
    Seg w;
    while (ok && take_segment(s, seg, g, &w, status)) {
      warp_arrive(&s->seg_empty[seg % kSegs], lane);
      ++seg;
      const bool pair = w.rows > tile_rows, two_segs = w.flags & kTwo;
      const bool apart = pair || two_segs;  // either group has a result of its own
      const int rows = pair ? (g == 0 ? tile_rows : w.rows - tile_rows) : w.rows;  // of this group
      const bool live = r < rows, warp_live = wq * 32 < rows;
      const int tok = (pair && g ? k.tile_tokens : 0) + (live ? r_tok : 0);
      const int i_new = w.i0 + tok;  // new token of a sequence's own part
      const int row = w.row0 + tok, qh = w.head * k.rep + (live ? r_head : 0);
      const bool own = !(w.flags & kShared);
      float m = -INFINITY, l = 0.f;
      // the releases of the V slots of the group's last tile and the one before
      uint64_t *last = nullptr, *before = nullptr;
      uint32_t last_par = 0, before_par = 0;
      const int tiles = two_segs ? 2 * w.n : w.n;
      for (int i = pair ? 0 : g; i < tiles; i += pair ? 1 : 2) {
        const int t0 = w.t0 + (two_segs ? i >> 1 : i) * kTile;
        const uint32_t buf = turn & 1u;
        if (!(ok = warp_wait(s, &s->scores[g], buf, status))) break;
        ++turn;
        tc_fence_after();
        const bool edge = own && t0 + kTile > w.ctx;
        uint32_t z[64];
        if (warp_live) {
          __syncwarp();
          tmem_ld32(t_s, z);
          tmem_ld32(t_s + 32, z + 32);
        }
        // beside the load: the product with V of the tile before the last, which
        // had this tile's weight columns, is done
        ok = !before || warp_wait(s, before, before_par, status);
        tc_fence_after();
        if (warp_live) {
          tmem_wait_ld(z);
          tmem_tie(z + 32);
        }
        if (!ok) break;
        tc_fence_before();
        warp_arrive(&s->s_free[g], lane);
        const bool odd = i & 1;
        if (warp_live) {
          if (edge) {
            const uint32_t *mask =
                k.a.mask ? k.a.mask + static_cast<int64_t>(row) * k.a.mask_words : nullptr;
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              const uint32_t see = view_bits(mask, k.a.mask_words, i_new, w.n_new, t0 + 32 * b - w.ctx);
#pragma unroll
              for (int c = 0; c < 32; ++c) {
                if (!(see >> c & 1u)) z[32 * b + c] = 0xff800000u;
              }
            }
            __syncwarp();
          }
          float mx[4];
#pragma unroll
          for (int b = 0; b < 4; ++b) mx[b] = __uint_as_float(z[b]);
#pragma unroll
          for (int c = 4; c < 60; c += 8) {
#pragma unroll
            for (int b = 0; b < 4; ++b) {
              mx[b] = fmaxf(fmaxf(mx[b], __uint_as_float(z[c + b])), __uint_as_float(z[c + 4 + b]));
            }
          }
#pragma unroll
          for (int b = 0; b < 4; ++b) mx[b] = fmaxf(mx[b], __uint_as_float(z[60 + b]));
          const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * k.sc;
          const bool rise = top > m + kLazy;
          if (!last) {
            m = top;
          } else if (__any_sync(0xffffffffu, rise)) {
            // the last product with V is in the accumulator when its slot is free
            if (!(ok = warp_wait(s, last, last_par, status))) break;
            tc_fence_after();
            const float mn = rise ? top : m;
            const float f = m == -INFINITY ? 0.f : fast_exp2(m - mn);
            l *= f;
            m = mn;
#pragma unroll 1
            for (int c = 0; c < D; c += 32) {
              uint32_t o[32];
              tmem_ld32(t_o + c, o);
              tmem_wait_ld(o);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tmem_st32(t_o + c, o);
            }
            tmem_wait_st();
          }
          const float sub = Wt::kOffset - (m == -INFINITY ? 0.f : m);
          const unsigned long long sc2 = f2dup(k.sc), sub2 = f2dup(sub);
          unsigned long long sum2[2] = {f2dup(0.f), f2dup(0.f)};
          uint32_t p[32];
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            if (c == 16) {  // half the weights: fewer live registers
              __syncwarp();
              tmem_st16(t_s + 64 + 32 * buf, p);
            }
            const unsigned long long y = fma2(
                f2pack(__uint_as_float(z[2 * c]), __uint_as_float(z[2 * c + 1])), sc2, sub2);
            float a, b;
            f2unpack(y, a, b);
            a = fast_exp2(a);
            b = fast_exp2(b);
            sum2[c & 1] = add2(sum2[c & 1], f2pack(a, b));
            p[c] = Wt::pack(a, b);
          }
          __syncwarp();
          tmem_st16(t_s + 64 + 32 * buf + 16, p + 16);
          // (the product takes weights in the cache's type, each off by at most half a step
          // of it; their sum is of the unrounded ones)
          float sa, sb;
          f2unpack(add2(sum2[0], sum2[1]), sa, sb);
          l += sa + sb;
          tmem_wait_st();
        }
        if (edge) {
          // the tile reaches past the committed tokens: V rows past the last
          // token become 0 (they may hold anything), and so do infinities
          // and NaN of new tokens, which patch_nonfinite puts back
          if (!(ok = warp_wait(s, &s->full[1][ring_v.at(odd)], ring_v.par(odd), status))) break;
          const int t = t0 + (r & (kTile - 1));
          if (t >= w.ctx) {
            char *v = s_v + ring_v.at(odd) * G::kTileBytes + (r & (kTile - 1)) * 128;
            bool found = false;
            const int c0 = (r / kTile) * 4 * kHalves;
#pragma unroll 4
            for (int c = c0; c < c0 + 4 * kHalves; ++c) {
              uint4 *at16 = reinterpret_cast<uint4 *>(v + (c >> 3) * (kTile * 128) +
                                                      (((c + lane) & 7) << 4));
              uint4 x = make_uint4(0, 0, 0, 0);
              bool change = t >= w.kv1;
              if (!change) {
                x = *at16;
                uint32_t *words = reinterpret_cast<uint32_t *>(&x);
#pragma unroll
                for (int b = 0; b < 4; ++b) {
                  const uint32_t bad = __vcmpeq2(words[b] & Wt::kExpMask, Wt::kExpMask);
                  if (bad) {
                    words[b] &= ~bad;
                    change = found = true;
                  }
                }
              }
              if (change) *at16 = x;
            }
            if (found) s->nonfinite[seg & 1u] = seg;
          }
          fence_proxy_async_smem();
        }
        tc_fence_before();
        warp_arrive(&s->weights[g][buf], lane);
        before = last;
        before_par = last_par;
        last = &s->empty[1][ring_v.at(odd)];
        last_par = ring_v.par(odd);
        ring_v.step(odd);
      }
      if (!ok) break;
      if (!pair) ring_v.skip(g == 0, two_segs ? w.join : (w.n + g) >> 1);  // the other group's tiles
      // ---- the unit's result -----------------------------------------------
      const uint32_t par = (seg - 1) & 1u;
      ok = warp_wait(s, &s->o_full[g], par, status) && (apart || warp_wait(s, &s->o_full[1 - g], par, status));
      if (!ok) break;
      tc_fence_after();
      s->stat[g][r] = make_float2(m, l);
      warp_arrive(&s->stats, lane);
      // (for two row tiles too: the group that zeroes a value of V which is not finite tells the other)
      if (!two_segs && !(ok = warp_wait(s, &s->stats, par, status))) break;
      const bool bad = s->nonfinite[seg & 1u] == seg;
      const bool two = !apart && w.n > 1;
      float f0 = 1.f, f1 = 0.f;
      if (!apart) {
        const float2 s0 = s->stat[0][r], s1 = s->stat[1][r];
        m = fmaxf(s0.x, s1.x);
        f0 = s0.x == -INFINITY ? 0.f : fast_exp2(s0.x - m);
        f1 = s1.x == -INFINITY ? 0.f : fast_exp2(s1.x - m);
        l = s0.y * f0 + s1.y * f1;
      }
      const float inv = l == 0.f ? 0.f : 1.f / l;
      f0 *= inv;
      f1 *= inv;
      const bool whole = w.flags & kWhole, base = w.flags & kBase;
      const int kind = own ? 0 : 1;
      const int64_t rh = static_cast<int64_t>(row) * k.a.q_heads + qh;
      const int64_t cont = static_cast<int64_t>(blockIdx.x) * kUnitRows + (pair && g ? tile_rows : 0) + r;
      if (live && (apart || g == 0)) {
        const float lse2 = l == 0.f ? -INFINITY : m - Wt::kOffset + log2f(l);
        if (whole) {
          if (k.a.lse) k.a.lse[rh] = lse2 * 0.69314718055994531f;
        } else if (base) {
          k.w.lse[kind][rh] = lse2;
        } else {
          k.w.lse_c[cont] = lse2;
        }
      }
      __syncwarp();
      const int half_cols = 32 * kHalves;
      const int c_begin = apart ? 0 : g * half_cols;
      const int c_end = min(apart ? 2 * half_cols : c_begin + half_cols, D);
      T *const out = reinterpret_cast<T *>(k.a.out) + row * k.a.o_row + qh * k.a.o_head;
      float *const part = base ? k.w.o[kind] + rh * D : k.w.o_c + cont * D;
      if (warp_live) {
        const uint32_t t_a = tmem + lanes + 256 + (apart ? g * 128 : 0);
#pragma unroll 1
        for (int c = c_begin; c < c_end; c += 32) {
          uint32_t x[32], y[32];
          tmem_ld32(t_a + c, x);
          if (two) tmem_ld32(t_a + 128 + c, y);
          tmem_wait_ld(x);
          if (two) {
            tmem_tie(y);
#pragma unroll
            for (int e = 0; e < 32; ++e) {
              x[e] = __float_as_uint(fmaf(__uint_as_float(y[e]), f1, __uint_as_float(x[e]) * f0));
            }
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) x[e] = __float_as_uint(__uint_as_float(x[e]) * f0);
          }
          if (c + 32 >= c_end) {  // the accumulators may be written again
            tc_fence_before();
            warp_arrive(&s->o_free, lane);
          }
          if (live) {
            if (whole) {
#pragma unroll
              for (int e = 0; e < 32; e += 8) {
                if (c + e < D) {
                  uint4 v;
                  uint32_t *words = reinterpret_cast<uint32_t *>(&v);
#pragma unroll
                  for (int j = 0; j < 4; ++j) {
                    words[j] = Wt::pack(__uint_as_float(x[e + 2 * j]), __uint_as_float(x[e + 2 * j + 1]));
                  }
                  *reinterpret_cast<uint4 *>(out + c + e) = v;
                }
              }
            } else {
#pragma unroll
              for (int e = 0; e < 32; e += 8) {
                if (c + e < D) store_32_bytes(part + c + e, x + e);
              }
            }
          }
          __syncwarp();
        }
      }
      if (!warp_live || c_begin >= c_end) warp_arrive(&s->o_free, lane);
      if (bad && live) {
        const int t1 = min(w.t0 + w.n * kTile, w.kv1);
        if (whole) {
          patch_nonfinite<T>(k, w.seq, w.ctx, w.n_new, w.head, row, i_new, w.t0, t1, c_begin, c_end, out);
        } else {
          patch_nonfinite<T>(k, w.seq, w.ctx, w.n_new, w.head, row, i_new, w.t0, t1, c_begin, c_end, part);
        }
      }
      __syncwarp();
      if (k.join_inside && !whole) {
        // the CTA that stores a cut unit's last part joins them, in their order
        const int owner = w.join & 0xffff, more = w.join >> 16;
        warp_arrive(&s->stored, lane);
        if (warp == 0) {
          if (!(ok = warp_wait(s, &s->stored, cuts & 1u, status))) break;
          if (lane == 0) {
            __threadfence();  // what the CTA stored, ahead of the count
            const bool all = atomicAdd(&k.w.tickets[owner], 1u) == static_cast<unsigned>(more);
            if (all) k.w.tickets[owner] = 0;
            s->joins = all;
            __threadfence();
          }
          warp_arrive(&s->counted, lane);
        }
        if (!(ok = warp_wait(s, &s->counted, cuts & 1u, status))) break;
        ++cuts;
        if (s->joins) {
          for (int slot = warp; slot < w.rows; slot += 8) {
            const int tok_in = slot / k.rep, head = w.head * k.rep + slot - tok_in * k.rep;
            const int64_t to = static_cast<int64_t>(w.row0 + tok_in) * k.a.q_heads + head;
            write_row<T>(k, to, w.row0 + tok_in, head, join_parts(k, 0, to, owner, more, slot));
          }
        }
        __syncwarp();
      }
    }
  } else if (warp < 10) {
    // ---- matrix products: warp 8 for group 0, warp 9 for group 1 --------------
    const int g = warp - 8;
    const uint32_t id_qk = instr_desc(Wt::kBf16, kTile, false);
    const uint32_t id_pv = instr_desc(Wt::kBf16, (D + 15) / 16 * 16, true);
    const int k_steps = (D + 15) / 16;
    // descriptors of the first bytes; a step's offset is added to the address field
    const uint32_t q0 = smem_desc(smem_addr(s_q), 16), k0 = smem_desc(smem_addr(s_k), 16);
    const uint32_t v0 = smem_desc(smem_addr(s_v), kTile * 128);
    const uint32_t t_s = tmem + g * 128, t_o = tmem + 256 + g * 128;
    uint32_t seg = 0, q_turn = 0;           // segments and Q tiles so far
    uint32_t tiles = 0, asked = 0, given = 0;  // tiles of the group so far: scores, products with V
    Ring<G::kSlotsK> ring_k;
    Ring<G::kSlotsV> ring_v;
    bool ok = true;
    Seg w;
    while (ok && take_segment(s, seg, g, &w, status)) {
      warp_arrive(&s->seg_empty[seg % kSegs], lane);
      const bool pair = w.rows > tile_rows, two_segs = w.flags & kTwo;
      const bool apart = pair || two_segs;  // either group has a Q of its own
      const int n = two_segs ? 2 * w.n : w.n, step = pair ? 1 : 2, first = pair ? 0 : g;
      const Ring<G::kSlotsK> k_before = ring_k;
      const Ring<G::kSlotsV> v_before = ring_v;
      const uint32_t q_at = q_turn + (apart ? g : 0), q_other = q_turn + 1 - g;
      q_turn += apart ? 2 : 1;
      if (elect_one()) {
        const uint32_t qa = q0 + (q_at & 1u) * (G::kQTile >> 4);
        // scores of tile i, once the last ones are taken and its K is there
        auto scores = [&](int i) {
          const bool odd = i & 1;
          const uint32_t at = ring_k.at(odd);
          // (the first turn of a fresh barrier passes for the one before it)
          if (!guarded_wait(s, &s->s_free[g], ~asked & 1u, status) ||
              !guarded_wait(s, &s->full[0][at], ring_k.par(odd), status)) {
            return false;
          }
          ++asked;
          ring_k.step(odd);
          tc_fence_after();
          const uint32_t ka = k0 + at * (G::kTileBytes >> 4);
#pragma unroll
          for (int c = 0; c < 4 * kHalves; ++c) {
            if (c < k_steps) {
              mma_ss(t_s, qa + ((c >> 2) * (kRows * 128) + (c & 3) * 32) / 16,
                     ka + ((c >> 2) * (kTile * 128) + (c & 3) * 32) / 16, id_qk, c > 0);
            }
          }
          tc_commit(&s->scores[g]);
          tc_commit(&s->empty[0][at]);
          return true;
        };
        auto free_q = [&] {  // after the segment's last scores
          tc_commit(&s->q_free[q_at & 1u]);
          if (apart) tc_commit(&s->q_free[q_other & 1u]);
        };
        // both of two tiles, as both issuing threads free both
        ok = guarded_wait(s, &s->q_full[q_at & 1u], q_at >> 1 & 1u, status) &&
             (!apart || guarded_wait(s, &s->q_full[q_other & 1u], q_other >> 1 & 1u, status));
        // Groups side by side do not end together, and a unit of two row tiles takes either half
        // of V's slots.  So its softmax, which waits on these, starts when both results before
        // it have been read: else a wait could be two turns ahead of the other group's slot, and
        // pass.  (Here and not in the softmax warps: there the wait's code cost calls that never
        // take it: the serving workload 275 us against 272, trees of 80 wide heads 132 against 128.)
        if (ok && pair && (w.flags & kBehindTwo)) ok = guarded_wait(s, &s->o_free, (seg - 1) & 1u, status);
        if (ok && first < n) ok = scores(first);
        if (ok && first + step >= n) free_q();
        for (int i = first; ok && i < n; i += step) {
          if (i + step < n) {
            if (!(ok = scores(i + step))) break;
            if (i + 2 * step >= n) free_q();
          }
          // the last segment's result has been read
          if (i == first && seg > 0 && !(ok = guarded_wait(s, &s->o_free, (seg - 1) & 1u, status))) break;
          const bool odd = i & 1;
          const uint32_t at = ring_v.at(odd);
          const uint32_t buf = given & 1u, va = v0 + at * (G::kTileBytes >> 4);
          ok = guarded_wait(s, &s->full[1][at], ring_v.par(odd), status) &&
               guarded_wait(s, &s->weights[g][buf], given >> 1 & 1u, status);
          if (!ok) break;
          ++given;
          ring_v.step(odd);
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < kTile / 16; ++c) {
            mma_ts(t_o, t_s + 64 + 32 * buf + c * 8, va + c * 2048 / 16, id_pv, i >= step || c > 0);
          }
          tc_commit(&s->empty[1][at]);
        }
        // a group without tiles keeps the others' pace
        if (ok && first >= n && seg > 0) ok = guarded_wait(s, &s->o_free, (seg - 1) & 1u, status);
        if (ok) tc_commit(&s->o_full[g]);
      }
      // what the elected lane counted, for all: its tiles, and the other group's
      ok = __all_sync(0xffffffffu, ok);
      asked = given = tiles += pair ? n : (n + 1 - g) >> 1;
      ring_k = k_before;
      ring_v = v_before;
      for (int odd = 0; odd < 2; ++odd) {
        const int half = !two_segs ? (n + 1 - odd) >> 1 : odd == g ? w.n : w.join;
        ring_k.skip(odd, half);
        ring_v.skip(odd, half);
      }
      ++seg;
    }
    if (elect_one()) {
      tc_commit(&s->drained[g]);  // nothing of this CTA runs on when it ends
      if (!mbar_wait(&s->drained[g], 0, kWaitPolls)) raise_status(status, SMC_DEV_TIMEOUT);
    }
    __syncwarp();
  } else if (warp == 10) {
    // ---- segments, K ------------------------------------------------------------
    Walk w;
    w.start(k);
    Ring<G::kSlotsK> ring;
    unsigned bits = 0;
    uint32_t filled = 0, parities = 0;
    bool ok = true;
    Seg next{};
    bool begun = false, held = false;  // next is found and not yet taken
    int behind = 0;                    // kBehindTwo, behind two segments side by side
    for (uint32_t seg = 0; ok; ++seg) {
      if (seg >= kSegs &&
          !(ok = warp_wait(s, &s->seg_empty[seg % kSegs], (seg / kSegs - 1) & 1u, status))) {
        break;
      }
      // the next segment, and the one after it beside it where both have one
      // row tile and are about as long
      Seg *const to = s->seg[seg % kSegs];
      int n = 0;
      bool pair = false;
      for (int g = 0; g < 2; ++g) {
        if (!held) {
          const bool more = w.next(k);
          if (!begun && lane == 0 && !k.join_inside) {
            const bool cut = more && w.first_cut;
            int4 *rec = reinterpret_cast<int4 *>(&k.w.cuts[blockIdx.x]);
            rec[0] = cut ? make_int4(w.t.row0 + w.tokens0, w.rows, w.head, w.more) : make_int4(0, 0, 0, 0);
            rec[1] = make_int4(more ? w.t.flags : 0, 0, 0, 0);
          }
          begun = held = true;
          next.flags = kEnd;
          if (more) {
            next = {w.t.row0 + w.tokens0, w.rows, w.tokens0, w.t.seq, w.head, w.t.kv0 + w.i0 * kTile, w.n,
                    w.t.ctx, w.t.kv1, w.t.tokens, 0, w.owner | w.more << 16};
            next.flags = (w.t.flags & kShared) | ((w.t.flags & kSolo) && w.n == w.t.tiles ? kWhole : 0) |
                         (w.i0 == 0 ? kBase : 0);
          }
        }
        // (a join inside is for one unit at a time)
        const bool may = !(next.flags & kEnd) && next.rows <= tile_rows && (!k.join_inside || (next.flags & kWhole));
        if (g) {
          if (!may || abs(n - next.n) > kTwoGap) break;
          if (lane == 0) {
            to->flags |= kTwo;
            to->join = next.n;
          }
          next.flags |= kTwo;
          next.join = n;
        }
        if (lane < 2 && lane >= g) {
          int4 *at = reinterpret_cast<int4 *>(to + lane);
          at[0] = make_int4(next.row0, next.rows, next.i0, next.seq);
          at[1] = make_int4(next.head, next.t0, next.n, next.ctx);
          at[2] = make_int4(next.kv1, next.n_new, next.flags | behind, next.join);
        }
        n = next.n;
        pair = next.rows > tile_rows;
        held = false;
        if (!may) break;
      }
      warp_arrive(&s->seg_full[seg % kSegs], lane);
      if (to->flags & kEnd) break;
      behind = to->flags & kTwo ? kBehindTwo : 0;
      ok = copy_tiles<kHalves, kTma, G::kSlotsK>(k, &map_k, k.a.c.k, s_k, s->full[0], s->empty[0], s, ring,
                                                 to, pair, &bits, &filled, &parities);
    }
    if (kTma && s->abort) wait_landed(s->full[0], filled, parities);
    if (bits) raise_status(status, bits);
  } else {
    // ---- Q and V ----------------------------------------------------------------
    Ring<G::kSlotsV> ring;
    uint32_t seg = 0, q_turn = 0;
    unsigned bits = 0;
    uint32_t filled = 0, parities = 0;
    bool ok = true;
    Seg w;
    while (ok && take_segment(s, seg, 0, &w, status)) {
      const Seg *const at_seg = s->seg[seg % kSegs];
      const bool pair = w.rows > tile_rows, two_segs = w.flags & kTwo;
      for (int j = 0; ok && j < (pair || two_segs ? 2 : 1); ++j, ++q_turn) {
        const uint32_t at = q_turn & 1u;
        if (q_turn >= 2 && !(ok = warp_wait(s, &s->q_free[at], ((q_turn >> 1) - 1) & 1u, status))) break;
        const int row0 = pair ? w.row0 + j * k.tile_tokens : at_seg[j].row0;
        const int head0 = at_seg[j].head * k.rep;
        if (elect_one()) {
          mbar_arrive_expect_tx(&s->q_full[at], kHalves * k.q_box * k.rep * 128);
#pragma unroll
          for (int half = 0; half < kHalves; ++half) {
            tma_load_3d(s_q + at * G::kQTile + half * (kRows * 128), &map_q, half * 64, head0, row0,
                        &s->q_full[at]);
          }
        }
        __syncwarp();
      }
      if (!ok) break;
      ok = copy_tiles<kHalves, kTma, G::kSlotsV>(k, &map_v, k.a.c.v, s_v, s->full[1], s->empty[1], s, ring,
                                                 at_seg, pair, &bits, &filled, &parities);
      warp_arrive(&s->seg_empty[seg % kSegs], lane);
      ++seg;
    }
    if (s->abort) {
      if (kTma) wait_landed(s->full[1], filled, parities);
      for (uint32_t q = q_turn > 2 ? q_turn - 2 : 0; q < q_turn; ++q) {
        mbar_wait(&s->q_full[q & 1u], q >> 1 & 1u, 1u << 12);
      }
    }
    if (bits) raise_status(status, bits);
  }
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_free_512(tmem);
  }
}

// The units that a CTA's range cuts: CTA (c, chunk) takes eight rows of the
// unit that the boundary between CTAs c and c + 1 is the first to cut (CTA
// c + 1 left its record): its owner's part and a continuation each of CTAs
// c + 1 .. c + more.  Rows that have another unit too get their joined part
// back for join_shared_kernel.
template <typename T>
__global__ void __launch_bounds__(32 * kJoinWarps)
join_cut_units_kernel(const __grid_constant__ KernelArgs k) {
  // the last kernel of a call lets nothing start before it has ended
  if (k.w.groups) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  wait_for_stream();
  const int cta = blockIdx.x, lane = threadIdx.x & 31;
  const int4 *cut = reinterpret_cast<const int4 *>(&k.w.cuts[cta + 1]);
  const int4 c = __ldcg(cut);  // row0, rows, head, more
  const int flags = __ldcg(cut + 1).x;
  const int slot = blockIdx.y * kJoinWarps + (threadIdx.x >> 5);
  if (slot >= c.y) return;
  const int D = k.a.c.head_dim, i = slot / k.rep, row = c.x + i, qh = c.z * k.rep + slot - i * k.rep;
  const int64_t rh = static_cast<int64_t>(row) * k.a.q_heads + qh;
  const bool live = 4 * lane < D;
  const int kind = flags & kShared;
  const Joined j = join_parts(k, kind, rh, cta, c.w, slot);
  if (flags & kSolo) {
    write_row<T>(k, rh, row, qh, j);
  } else {
    const float4 y = j.result();
    if (live) reinterpret_cast<float4 *>(k.w.o[kind] + rh * D)[lane] = y;
    if (lane == 0) k.w.lse[kind][rh] = j.lse2();
  }
}

// The rows of prompts with a shared part: its result and the own part's.  A
// CTA per row, four heads a warp at a time.
constexpr int kJoinHeads = 4;
template <typename T>
__global__ void __launch_bounds__(32 * kJoinWarps)
join_shared_kernel(const __grid_constant__ KernelArgs k) {
  const BatchArgs &b = k.a.b;
  const int row = blockIdx.x;
  wait_for_stream();
  int seq = min(row / b.max_new, b.S - 1);  // right when every sequence has max_new rows
  if (b.row_start && !(b.row_start[seq] <= row && row < b.row_start[seq + 1])) seq = seq_of_row(b, row);
  // without a shared part the row is written already; its rows are in order with one
  if (seq < 0 || __ldcg(&k.w.common[seq / b.group]) == 0) return;
  const int D = k.a.c.head_dim, lane = threadIdx.x & 31;
  const bool live = 4 * lane < D;
  for (int q0 = (threadIdx.x >> 5) * kJoinHeads; q0 < k.a.q_heads; q0 += kJoinWarps * kJoinHeads) {
    float l[kJoinHeads][2];
    float4 x[kJoinHeads][2];
#pragma unroll
    for (int e = 0; e < kJoinHeads; ++e) {
      const int64_t rh = static_cast<int64_t>(row) * k.a.q_heads + q0 + e;
      const bool in = q0 + e < k.a.q_heads;
#pragma unroll
      for (int p = 0; p < 2; ++p) {
        l[e][p] = in ? __ldcg(&k.w.lse[p][rh]) : -INFINITY;
        x[e][p] = load_part(k.w.o[p] + rh * D, live && in);
      }
    }
#pragma unroll
    for (int e = 0; e < kJoinHeads; ++e) {
      if (q0 + e >= k.a.q_heads) break;
      Joined j;
      j.top = fmaxf(l[e][0], l[e][1]);
      j.add(l[e][0], x[e][0]);
      j.add(l[e][1], x[e][1]);
      write_row<T>(k, static_cast<int64_t>(row) * k.a.q_heads + q0 + e, row, q0 + e, j);
    }
  }
}

// ---------------------------------------------------------------------------
// Launch.
// ---------------------------------------------------------------------------
using EncodeFn = decltype(&cuTensorMapEncodeTiled);

static EncodeFn encode_fn() {
  static EncodeFn fn = [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess) {
      p = nullptr;
    }
    return reinterpret_cast<EncodeFn>(p);
  }();
  return fn;
}

// [rows][q_heads][head_dim] in boxes of 64 elements x the heads of a key head x
// a row tile's tokens; rows past the last read as 0.
static bool make_q_map(CUtensorMap *map, const KernelArgs &k) {
  const EncodeFn fn = encode_fn();
  if (!fn) return false;
  const AttnArgs &a = k.a;
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(a.c.head_dim), static_cast<cuuint64_t>(a.q_heads),
                              static_cast<cuuint64_t>(a.b.rows)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(a.q_head) * 2, static_cast<cuuint64_t>(a.q_row) * 2};
  const cuuint32_t boxes[3] = {64, static_cast<cuuint32_t>(k.rep), static_cast<cuuint32_t>(k.q_box)};
  const cuuint32_t steps[3] = {1, 1, 1};
  return fn(map, a.c.dtype == SMC_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
            3, const_cast<char *>(a.q), dims, strides, boxes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// [blocks][kv_heads][block_size][head_dim] in boxes of 64 elements x `box`
// tokens; columns past head_dim read as 0.
static bool make_map(CUtensorMap *map, const CacheArgs &c, void *base, int box) {
  const EncodeFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(c.head_dim), static_cast<cuuint64_t>(c.block_size),
                              static_cast<cuuint64_t>(c.kv_heads), static_cast<cuuint64_t>(c.blocks)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(c.token_stride) * 2,
                                 static_cast<cuuint64_t>(c.head_stride) * 2,
                                 static_cast<cuuint64_t>(c.block_stride) * 2};
  const cuuint32_t boxes[4] = {64, static_cast<cuuint32_t>(box), 1, 1};
  const cuuint32_t steps[4] = {1, 1, 1, 1};
  return fn(map, c.dtype == SMC_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16,
            4, base, dims, strides, boxes, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename T>
static const void *attention_fn(bool wide, bool tma) {
  if (wide) {
    return tma ? reinterpret_cast<const void *>(attention_kernel<T, 2, true>)
               : reinterpret_cast<const void *>(attention_kernel<T, 2, false>);
  }
  return tma ? reinterpret_cast<const void *>(attention_kernel<T, 1, true>)
             : reinterpret_cast<const void *>(attention_kernel<T, 1, false>);
}

constexpr size_t kAttnSmem = Geometry<2>::kTail + sizeof(AttnTail);
static_assert(Geometry<1>::kTail <= Geometry<2>::kTail && kAttnSmem <= 227 * 1024, "shared memory");
static_assert(Geometry<1>::kSlotsV <= 12 &&
              (Geometry<2>::kSlotsK + Geometry<2>::kSlotsV) * Geometry<2>::kTileBytes == kRingBytes,
              "rings");

static cudaError_t configure(int *sms) {
  constexpr int kMaxDev = 64;
  static std::atomic<int> known[kMaxDev];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const int slot = dev < kMaxDev ? dev : kMaxDev - 1;
  *sms = dev < kMaxDev ? known[slot].load(std::memory_order_acquire) : 0;
  if (*sms) return cudaSuccess;
  for (const bool wide : {false, true}) {
    for (const bool tma : {false, true}) {
      for (const void *fn : {attention_fn<__nv_bfloat16>(wide, tma), attention_fn<__half>(wide, tma)}) {
        e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(kAttnSmem));
        if (e != cudaSuccess) return e;
      }
    }
  }
  int n = 0;
  e = cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  *sms = n < kMaxCtas ? n : kMaxCtas;
  if (dev < kMaxDev) known[slot].store(*sms, std::memory_order_release);
  return cudaSuccess;
}

cudaError_t launch_tree_attention(const AttnArgs &a, void *workspace, cudaStream_t st) {
  if (a.b.rows == 0) return cudaSuccess;
  int sms = 0;
  cudaError_t e = configure(&sms);
  if (e != cudaSuccess) return e;
  KernelArgs k{};
  k.a = a;
  // Reading shared blocks once takes two more kernels and a second part of
  // every row.  While all that the sequences' tables have room for is less than
  // what the L2 cache holds, reading it again costs less than that.  The host
  // knows the tables' room, not the tokens held (they are on the device): tables
  // with much room to spare are read once though they hold little.  Measured,
  // once and again: 8 sequences that share 512 of 700 tokens 27.4 and 20.2 us
  // (room for 96 MB and more, and for 24 to 92 MB); 16 x 16 that share 2048 of
  // 2690 272 and 437 us.
  const double table_bytes = static_cast<double>(a.b.S) * a.b.T * a.c.block_size * a.c.kv_heads * a.c.head_dim * 4;
  if (table_bytes < 96e6) k.a.b.group = 1;
  carve(a.c, k.a.b, a.q_heads, static_cast<char *>(workspace), &k.w);
  k.rep = a.q_heads / a.c.kv_heads;
  k.tile_tokens = kRows / k.rep;
  k.q_box = a.b.rows < k.tile_tokens ? a.b.rows : k.tile_tokens;
  k.sc = a.scale * 1.4426950408889634f;
  // with 2^s the power of two at or above the block size, 2^(31 + s) / size
  // rounded up divides every t < 2^31 exactly
  const uint64_t bs = a.c.block_size;
  uint32_t log2 = 0;
  while ((1ull << log2) < bs) ++log2;
  k.magic = static_cast<uint32_t>(((1ull << (31 + log2)) + bs - 1) / bs);
  k.shift = log2 ? log2 - 1 : 0;
  // a box is a run of tokens inside one block and one tile; the swizzle
  // repeats every eight rows, so a box starts on a multiple of eight.  Blocks
  // of other sizes are copied by the lanes, 16 bytes each: 34 trees of 64 rows,
  // 16 heads over 8, 7379 tokens in blocks of 20 take 328 us, 2.1 times their
  // bytes' time
  int box = kTile;
  while (a.c.block_size % box) box >>= 1;
  CUtensorMap map_q{}, map_k{}, map_v{};
  if (!make_q_map(&map_q, k)) return cudaErrorInvalidValue;
  const bool tma = box >= 8 && make_map(&map_k, a.c, a.c.k, box) && make_map(&map_v, a.c, a.c.v, box);
  k.box = box;
  // no more CTAs than tiles there can be
  const int64_t units = a.b.S * ((static_cast<int64_t>(a.b.max_new) + 2 * k.tile_tokens - 1) / (2 * k.tile_tokens));
  const int64_t most = (static_cast<int64_t>(a.b.T) * a.c.block_size + kTile - 1) / kTile * a.c.kv_heads * units;
  const int ctas = most < sms ? static_cast<int>(most) : sms;
  // Up to 256 sequences, each CTA counts the tiles itself: a few loads a lane,
  // against a launch.  Measured, so and planned: one sequence 12.0 and 13.7 us,
  // 256 of them 126.4 and 126.8, 1024 347 and 329.  Shared parts need the
  // tables compared.
  k.planned = k.w.groups > 0 || a.b.S > 256;
  // Few parts: the last CTA of a cut unit joins them, against another launch:
  // one token 12.0 and 12.9 us, 256 sequences of one 126 and 137 us; about even
  // at 400 parts (18.9 us by a kernel, 19.4).  A CTA takes about 8 us for 1344
  // parts (64 rows of 21), so more of them take a kernel that spreads them over
  // the machine.  A unit
  // spans at most 1 / kv_heads of the line, as its sequence has as many.
  const int64_t most_rows = static_cast<int64_t>(a.b.max_new) * k.a.b.group * k.rep;
  const int unit_rows = static_cast<int>(most_rows < kUnitRows ? most_rows : kUnitRows);
  k.join_inside = !k.w.groups && unit_rows * (ctas / a.c.kv_heads + 2) <= 1024;
  k.more_kernels = k.w.groups > 0 || (ctas > 1 && !k.join_inside);
  if (k.planned) {
    int n = ctas;
    void *pargs[] = {&k, &n};
    e = launch_early(reinterpret_cast<const void *>(plan_kernel), dim3(k.w.groups ? k.w.groups : 1), kPlanThreads,
                     0, pargs, st);
    if (e != cudaSuccess) return e;
  }
  const bool bf16 = a.c.dtype == SMC_BF16, wide = a.c.head_dim > 64;
  void *args[] = {&k, &map_q, &map_k, &map_v};
  e = launch_early(bf16 ? attention_fn<__nv_bfloat16>(wide, tma) : attention_fn<__half>(wide, tma),
                 dim3(ctas), kAttnThreads, kAttnSmem, args, st);
  if (e != cudaSuccess) return e;
  void *jargs[] = {&k};
  if (ctas > 1 && !k.join_inside) {  // with one CTA nothing is cut
    e = launch_early(bf16 ? reinterpret_cast<const void *>(join_cut_units_kernel<__nv_bfloat16>)
                        : reinterpret_cast<const void *>(join_cut_units_kernel<__half>),
                   dim3(ctas - 1, (unit_rows + kJoinWarps - 1) / kJoinWarps), 32 * kJoinWarps, 0, jargs, st);
    if (e != cudaSuccess) return e;
  }
  if (!k.w.groups) return cudaSuccess;
  return launch_early(bf16 ? reinterpret_cast<const void *>(join_shared_kernel<__nv_bfloat16>)
                         : reinterpret_cast<const void *>(join_shared_kernel<__half>),
                    dim3(a.b.rows), 32 * kJoinWarps, 0, jargs, st);
}

}  // namespace smcsd

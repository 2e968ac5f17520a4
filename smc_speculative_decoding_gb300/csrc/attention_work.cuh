// What the attention kernels over the paged cache share: their work as a line
// of tiles, the joins of parts, and the launch of either.
#pragma once

#include <cuda.h>

#include "cache_common.cuh"

namespace smcsd {

// ---------------------------------------------------------------------------
// Work.  An *entry* is a run of consecutive rows and a range of tokens that
// they all attend: the own part of one sequence, or the part that the
// sequences of a prompt share (their leading equal table slots).  A *unit* is
// what a CTA computes at a time: one or two row tiles of an entry, over its
// tokens in tiles of kTile.  A row tile is `tile_tokens` consecutive new tokens
// times the query heads of a key head, or where these are more than it has rows
// for a part of them (kParts).  The units' tiles form one
// line; CTA c takes tiles [c * per, (c + 1) * per) of it, so ragged lengths
// load every SM alike.  A unit's first tiles' CTA owns the unit's result;
// every later CTA of the unit has exactly one such continuation (its first
// segment) and stores it in its own slot.
// ---------------------------------------------------------------------------
constexpr int kPlanThreads = 1024;
// Most CTAs of either kernel.  What has to be zero between calls (the header and
// the tickets) lies alike in every layout, so that calls of other shapes, and of
// the other cache's width, may follow one another in a workspace.
constexpr int kMostCtas = 384;

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
  int row0, rows, head, more;  // first row, rows of the unit (0: no such unit), head unit,
  int flags, pad[3];           // continuations; the entry's flags
};

struct PlanHeader {
  unsigned ticket;  // plan CTAs done; returns to zero
  int total, per;   // tiles, tiles per CTA
};

struct AttnWorkspace {
  PlanHeader *head;
  unsigned *tickets;  // [kMostCtas] parts stored of the unit that a CTA's end cuts; return to zero
  int *common;     // [groups] shared tokens
  int *ref;        // [groups] the sequence by whose table they are read
  int *tile0;      // [entries + 1]
  Entry *entries;  // shared parts of the groups (when group > 1), then the sequences
  float *lse[2];   // own, shared: [rows * q_heads], log2
  float *o[2];     // [rows * q_heads][head_dim], normalised
  Cut *cuts;       // [ctas]
  float *lse_c;    // [ctas][unit_rows] continuations
  float *o_c;      // [ctas][unit_rows][head_dim]
  int groups;      // 0 when group == 1
  int n_entries;
};

inline size_t carve(const CacheArgs &c, const BatchArgs &b, int q_heads, int ctas, int unit_rows,
                    char *base, AttnWorkspace *w) {
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
  t.tickets = reinterpret_cast<unsigned *>(take(sizeof(unsigned) * kMostCtas));
  t.common = reinterpret_cast<int *>(take(sizeof(int) * t.groups));
  t.ref = reinterpret_cast<int *>(take(sizeof(int) * t.groups));
  t.tile0 = reinterpret_cast<int *>(take(sizeof(int) * (static_cast<size_t>(t.n_entries) + 1)));
  t.entries = reinterpret_cast<Entry *>(take(sizeof(Entry) * t.n_entries));
  for (int k = 0; k < 2; ++k) {
    const size_t n = k == 0 || t.groups ? rh : 0;
    t.lse[k] = reinterpret_cast<float *>(take(sizeof(float) * n));
    t.o[k] = reinterpret_cast<float *>(take(sizeof(float) * n * D));
  }
  t.cuts = reinterpret_cast<Cut *>(take(sizeof(Cut) * ctas));
  const size_t slots = static_cast<size_t>(ctas) * unit_rows;
  t.lse_c = reinterpret_cast<float *>(take(sizeof(float) * slots));
  t.o_c = reinterpret_cast<float *>(take(sizeof(float) * slots * D));
  if (w) *w = t;
  return off;
}

struct WorkArgs {
  AttnArgs a;
  AttnWorkspace w;
  int rep;      // query heads per key head
  int tile_tokens;  // new tokens of a row tile
  int q_box;    // new tokens of a copied box of Q
  int planned;      // plan_kernel has run (else each CTA finds its own work)
  int more_kernels; // joins follow (a call's last kernel lets nothing start before its end)
  int join_inside;  // the last CTA of a cut unit joins its parts
  int box;      // tokens per copied box of K and V
  uint32_t magic, shift;  // t / block_size == umulhi(t, magic) >> shift
  float sc;     // scale * log2 e
  int head_units;   // with kParts: units of heads, a multiple of the key heads,
  int unit_rep;     // and the rows that a new token has in one (the last of a key head may have fewer)
};

// S: kTile, tokens per tile; kRowTiles, row tiles of a unit; kUnitRows, most
// rows of one; kParts, whether a key head may have several head units.
// The query heads [first, first + n) of a head unit:
struct UnitHeads {
  int key, first, n;
};
template <class S>
__device__ __forceinline__ UnitHeads unit_heads(const WorkArgs &k, int unit) {
  if (!S::kParts) return {unit, unit * k.rep, k.rep};
  const int parts = k.head_units / k.a.c.kv_heads, key = unit / parts, from = (unit - key * parts) * k.unit_rep;
  return {key, key * k.rep + from, min(k.unit_rep, k.rep - from)};
}

// t / block_size by a multiplication: with 2^s the power of two at or above the
// block size, 2^(31 + s) / size rounded up divides every t < 2^31 exactly.
inline void divide_by(int block_size, WorkArgs *k) {
  const uint64_t bs = block_size;
  uint32_t log2 = 0;
  while ((1ull << log2) < bs) ++log2;
  k->magic = static_cast<uint32_t>(((1ull << (31 + log2)) + bs - 1) / bs);
  k->shift = log2 ? log2 - 1 : 0;
}
__device__ __forceinline__ uint32_t block_of(const WorkArgs &k, uint32_t t) {
  return k.a.c.block_size == 1 ? t : __umulhi(t, k.magic) >> k.shift;
}

// ---------------------------------------------------------------------------
// plan_kernel: the tokens that each prompt's sequences share, then (the last
// CTA to finish) the entries and the prefix of their tiles.
// ---------------------------------------------------------------------------
static __device__ int block_scan_excl(int v, int *warps, int *total) {
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

// Units of an entry in one head unit.
template <class S>
__device__ __forceinline__ int token_units(const WorkArgs &k, int tokens) {
  return (tokens + S::kRowTiles * k.tile_tokens - 1) / (S::kRowTiles * k.tile_tokens);
}
template <class S>
__device__ __forceinline__ int head_units(const WorkArgs &k) {
  return S::kParts ? k.head_units : k.a.c.kv_heads;
}

template <class S>
__device__ __forceinline__ int entry_tiles(const WorkArgs &k, int tokens, int kv0, int kv1,
                                           int *per_unit) {
  *per_unit = (kv1 - kv0 + S::kTile - 1) / S::kTile;
  if (tokens <= 0 || kv1 <= kv0) return 0;
  return *per_unit * head_units<S>(k) * token_units<S>(k, tokens);
}

template <class S>
__device__ int make_entry(const WorkArgs &k, int e, Entry *out) {
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
    tiles = entry_tiles<S>(k, t.tokens, 0, shared, &t.tiles);
  } else {
    const int s = e - k.w.groups;
    const SeqInfo si = seq_info(b, bs, s);
    if (si.bits) raise_status(k.a.status, si.bits);
    const int shared = k.w.groups ? __ldcg(&k.w.common[s / b.group]) : 0;
    t = {si.row0, si.n, s, shared, si.len, si.len - si.n, 0, shared ? 0 : kSolo};
    tiles = entry_tiles<S>(k, t.tokens, t.kv0, t.kv1, &t.tiles);
  }
  if (out) *out = t;
  return tiles;
}

template <class S>
__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const __grid_constant__ WorkArgs k, int ctas) {
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
      k.w.common[blockIdx.x] = static_cast<int>(tokens / S::kTile * S::kTile);
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
    mine += make_entry<S>(k, e, &t);
    k.w.entries[e] = t;
  }
  int total;
  int at = block_scan_excl(mine, warps, &total);
  for (int e = e0; e < e1; ++e) {
    k.w.tile0[e] = at;
    const Entry &t = k.w.entries[e];
    int unused;
    at += entry_tiles<S>(k, t.tokens, t.kv0, t.kv1, &unused);
  }
  if (tid == 0) {
    k.w.tile0[k.w.n_entries] = total;
    k.w.head->total = total;
    k.w.head->per = max(1, (total + ctas - 1) / ctas);
  }
}

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
template <class S>
struct Walk {
  int x, x1, per, e;
  Entry t;
  int base;       // tiles of the line before entry e
  int span;       // tiles of the line of each of its units
  bool aligned;
  int head, rt;   // unit: its head unit, and which of the token units
  int i0, n;      // tiles [i0, i0 + n) of the unit
  int tokens0;    // new token of the unit's first row
  int rows;       // rows of the unit

  __device__ __forceinline__ int span_of(int tiles) const {
    return aligned ? (tiles + per - 1) / per * per : tiles;
  }
  // units and tiles per unit of sequence e
  __device__ __forceinline__ int2 sequence_units(const WorkArgs &k, int e, unsigned *bits) {
    if (e >= k.w.n_entries) return make_int2(0, 0);
    const SeqInfo si = seq_info(k.a.b, k.a.c.block_size, e);
    *bits |= si.bits;
    if (si.n <= 0) return make_int2(0, 0);
    return make_int2(head_units<S>(k) * token_units<S>(k, si.n), (si.len + S::kTile - 1) / S::kTile);
  }
  __device__ __forceinline__ void start(const WorkArgs &k) {
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
  __device__ __forceinline__ void load(const WorkArgs &k) {
    if (k.planned) {
      const int4 *p = reinterpret_cast<const int4 *>(&k.w.entries[e]);
      const int4 a = __ldcg(p), b = __ldcg(p + 1);
      t = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
      base = __ldcg(&k.w.tile0[e]);
    } else {
      const SeqInfo si = seq_info(k.a.b, k.a.c.block_size, e);
      t = {si.row0, si.n, e, 0, si.len, si.len - si.n, (si.len + S::kTile - 1) / S::kTile, kSolo};
    }
    span = span_of(t.tiles);
  }
  __device__ __forceinline__ bool next(const WorkArgs &k) {
    if (x >= x1) return false;
    int rts;
    for (;;) {
      rts = token_units<S>(k, t.tokens);
      const int tiles = t.tokens > 0 && t.kv1 > t.kv0 ? rts * head_units<S>(k) * span : 0;
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
    tokens0 = rt * S::kRowTiles * k.tile_tokens;
    rows = min(t.tokens - tokens0, S::kRowTiles * k.tile_tokens) * unit_heads<S>(k, head).n;
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
__device__ __forceinline__ void write_row(const WorkArgs &k, int64_t rh, int row, int qh, const Joined &j) {
  const int lane = threadIdx.x & 31;
  const float4 x = j.result();
  if (4 * lane < k.a.c.head_dim) {
    T *dst = reinterpret_cast<T *>(k.a.out) + row * k.a.o_row + qh * k.a.o_head + 4 * lane;
    *reinterpret_cast<uint2 *>(dst) = make_uint2(pack2<T>(x.x, x.y), pack2<T>(x.z, x.w));
  }
  if (k.a.lse && lane == 0) k.a.lse[rh] = j.lse2() * 0.69314718055994531f;
}

// A row of a cut unit: its owner's part, and a continuation each of CTAs
// cta + 1 .. cta + more at row `slot` of their slots.
template <class S>
__device__ __forceinline__ Joined join_parts(const WorkArgs &k, int kind, int64_t rh, int cta, int more,
                                             int slot) {
  const int D = k.a.c.head_dim;
  const bool live = 4 * static_cast<int>(threadIdx.x & 31) < D;
  Joined j;
  float l = __ldcg(&k.w.lse[kind][rh]);
  float4 x = load_part(k.w.o[kind] + rh * D, live);
  const int64_t slot0 = static_cast<int64_t>(cta + 1) * S::kUnitRows + slot;
  constexpr int kBatch = 8;
  for (int p = 0; p < more; p += kBatch) {
    float ls[kBatch];
    float4 xs[kBatch];
    float top = fmaxf(j.top, l);
#pragma unroll
    for (int e = 0; e < kBatch; ++e) {
      const int64_t at = slot0 + static_cast<int64_t>(p + e) * S::kUnitRows;
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

// The units that a CTA's range cuts: CTA (c, chunk) takes eight rows of the
// unit that the boundary between CTAs c and c + 1 is the first to cut (CTA
// c + 1 left its record): its owner's part and a continuation each of CTAs
// c + 1 .. c + more.  Rows that have another unit too get their joined part
// back for join_shared_kernel.
template <typename T, class S>
__global__ void __launch_bounds__(32 * kJoinWarps)
join_cut_units_kernel(const __grid_constant__ WorkArgs k) {
  // the last kernel of a call lets nothing start before it has ended
  if (k.w.groups) asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  wait_for_stream();
  const int cta = blockIdx.x, lane = threadIdx.x & 31;
  const int4 *cut = reinterpret_cast<const int4 *>(&k.w.cuts[cta + 1]);
  const int4 c = __ldcg(cut);  // row0, rows, head unit, more
  const int flags = __ldcg(cut + 1).x;
  const int slot = blockIdx.y * kJoinWarps + (threadIdx.x >> 5);
  if (slot >= c.y) return;
  const UnitHeads heads = unit_heads<S>(k, c.z);
  const int D = k.a.c.head_dim, i = slot / heads.n, row = c.x + i, qh = heads.first + slot - i * heads.n;
  const int64_t rh = static_cast<int64_t>(row) * k.a.q_heads + qh;
  const bool live = 4 * lane < D;
  const int kind = flags & kShared;
  const Joined j = join_parts<S>(k, kind, rh, cta, c.w, slot);
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
join_shared_kernel(const __grid_constant__ WorkArgs k) {
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

using EncodeFn = decltype(&cuTensorMapEncodeTiled);

inline EncodeFn encode_fn() {
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

}  // namespace smcsd

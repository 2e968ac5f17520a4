// Per-head RMS norms of queries and keys, the position rotation, and the write
// of keys and values into an 8-bit cache (smc_qk_norm_rope8 in smcsd.h).
#include "qk_turn.cuh"

namespace smcsd {

constexpr int kThreads8 = 256;
constexpr int kWarps8 = kThreads8 / 32;

// Work: a *run* is the new tokens of one sequence that lie in one block; its
// keys and values of one head share a scale.  CTA (x, h) takes the runs that
// begin in rows [x * per, (x + 1) * per): for each, key head h's keys and
// values, and query heads (the scalar kernel's) or, in CTAs of their own past
// those of the key heads, query heads alone (the vectors').
struct Run {
  int row, n;      // rows [row, row + n)
  int seq, at;     // the first one's place in its table
};

// The first sequence whose rows end behind row r (S: none): a warp probes 32
// places at a time, so that 1024 sequences take two dependent loads.
__device__ __forceinline__ int find_seq(const BatchArgs &b, int r) {
  int lo = 0, hi = b.S;  // in [lo, hi]
  while (lo < hi) {
    const int step = (hi - lo + 32) / 32, at = lo + (static_cast<int>(threadIdx.x & 31) + 1) * step - 1;
    const unsigned past = __ballot_sync(0xffffffffu, at >= hi || b.row_start[at + 1] > r);
    const int first = __ffs(past) - 1;  // (at least the last lane's is)
    hi = min(hi, lo + (first + 1) * step - 1);
    lo += first * step;
    if (step == 1) break;
  }
  return lo;
}

// The runs that begin in rows [r, end), one after the other.
struct Runs {
  int s, r, end;
  __device__ __forceinline__ Runs(const QkArgs &a, int r0, int r1) : s(min(r0 / a.b.max_new, a.b.S - 1)), r(r0), end(r1) {
    // (the guess is right where every sequence has max_new rows)
    if (!a.b.row_start) s = r0 / a.b.max_new;
    else if (!(a.b.row_start[s] <= r0 && r0 < a.b.row_start[s + 1])) s = find_seq(a.b, r0);
  }
  __device__ __forceinline__ Run next(const QkArgs &a) {
    const int bs = a.c.block_size;
    while (r < end && s < a.b.S) {
      const SeqInfo si = seq_info(a.b, bs, s);
      const int i = r - si.row0;
      if (si.bits || i >= si.n) {  // the next sequence
        if (si.bits && blockIdx.y == 0 && threadIdx.x == 0) raise_status(a.status, si.bits);
        ++s;
        continue;
      }
      if (i < 0) {  // (rows of a sequence that is out of order)
        r = min(end, si.row0);
        continue;
      }
      const int at = si.len - si.n + i, off = at % bs, n = min(bs - off, si.n - i);
      const Run run{r, n, s, at};
      r += n;
      if (i == 0 || off == 0) return run;
    }
    return {0, 0, 0, 0};
  }
};

// Keys are rounded step by step, x r, then w, then the rotation's products, as
// plain fp32 does, and the sum of a norm is taken in one order (eight or four
// neighbours each lane, then across the lanes) by both kernels below: where a
// block's largest key lies beside a power of two, its last bit decides the scale,
// and neither alignment nor strides have a say in it.

// Element d of a vector after norm (r = rsqrt of the mean square) and rotation.
template <typename T>
__device__ __forceinline__ float turned(const QkArgs &a, const T *src, const T *w, float r, const float *cs, int d) {
  auto normed = [&](int e) {
    const float x = to_f32(src[e]);
    return w ? __fmul_rn(__fmul_rn(x, r), to_f32(w[e]) + a.w0) : x;
  };
  const float y = normed(d);
  if (d >= a.rot) return y;
  const int half = a.rot / 2;
  const bool second = a.interleaved ? (d & 1) : d >= half;
  const int j = a.interleaved ? d >> 1 : (second ? d - half : d);
  const float z = normed(a.interleaved ? d ^ 1 : (second ? d - half : d + half));
  const float p = __fmul_rn(y, cs[j]), q = __fmul_rn(z, cs[half + j]);
  return second ? __fadd_rn(q, p) : __fsub_rn(p, q);
}

// rsqrt(mean(x^2) + eps) of a vector, or 1 without weights: a warp's lanes.
template <typename T>
__device__ __forceinline__ float norm_of(const QkArgs &a, const T *src, const T *w) {
  if (!w) return 1.f;
  constexpr int E = 16 / sizeof(T);
  float sum = 0.f;
  for (int d0 = static_cast<int>(threadIdx.x & 31) * E; d0 < a.c.head_dim; d0 += 32 * E) {
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float x = d0 + e < a.c.head_dim ? to_f32(src[d0 + e]) : 0.f;
      sum = fmaf(x, x, sum);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  return rsqrtf(fmaf(sum, 1.f / a.c.head_dim, a.eps));
}

// Any sizes, strides and alignment: a warp per vector, each lane elements lane,
// lane + 32, ...; keys are computed for the block's scale and again to be stored.
// (1280 rows of 32 + 8 + 8 heads of 128 58 us, 12535 rows of 40 + 8 + 8 heads of 96
// 358 us; with the vectors below 21 and 135.)
template <typename T>
__global__ void __launch_bounds__(kThreads8)
append8_kernel(const __grid_constant__ QkArgs a, const __grid_constant__ ScaleArgs sc, int per) {
  __shared__ int s_top[2];
  __shared__ float s_old[2], s_new[2];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, h = blockIdx.y;
  const int bs = a.c.block_size, D = a.c.head_dim;
  wait_for_stream();
  const int r0 = blockIdx.x * per;
  Runs runs(a, r0, min(r0 + per, a.b.rows));
  for (Run run = runs.next(a); run.n > 0; run = runs.next(a)) {
    const int block = a.b.tables[static_cast<int64_t>(run.seq) * a.b.T + run.at / bs], off = run.at % bs;
    if (block < 0 || block >= a.c.blocks) {
      if (h == 0 && tid == 0) raise_status(a.status, SMC_DEV_BAD_BLOCK);
      continue;
    }
    auto position = [&](int i) {
      const int p = a.positions ? a.positions[run.row + i] : run.at + i;
      return p >= 0 && p < a.max_pos ? p : -1;
    };
    auto key = [&](int i) { return reinterpret_cast<const T *>(a.k) + (run.row + i) * a.k_row + h * a.k_head; };
    auto value = [&](int i) { return reinterpret_cast<const T *>(a.v) + (run.row + i) * a.v_row + h * a.v_head; };
    const T *kw = reinterpret_cast<const T *>(a.kw), *qw = reinterpret_cast<const T *>(a.qw);
    __syncthreads();
    if (tid < 2) s_top[tid] = 0;
    __syncthreads();
    float top_k = 0.f, top_v = 0.f;
    for (int i = warp; i < run.n; i += kWarps8) {
      const int pos = position(i);
      if (pos < 0) {
        if (h == 0 && lane == 0) raise_status(a.status, SMC_DEV_BAD_ROWS);
        continue;
      }
      const float *cs = a.rope + static_cast<int64_t>(pos) * a.rot;
      const float r = norm_of(a, key(i), kw);
      for (int d = lane; d < D; d += 32) {
        const float y = fabsf(turned(a, key(i), kw, r, cs, d)), v = fabsf(to_f32(value(i)[d]));
        if (y < INFINITY) top_k = fmaxf(top_k, y);
        if (v < INFINITY) top_v = fmaxf(top_v, v);
      }
    }
    atomicMax(&s_top[0], __float_as_int(top_k));  // of positive numbers: their bits' order
    atomicMax(&s_top[1], __float_as_int(top_v));
    __syncthreads();
    if (tid < 2) {
      float *at = (tid ? sc.v : sc.k) + block * sc.block + h * sc.head;
      const float need = least_scale(__int_as_float(s_top[tid]));
      s_old[tid] = off ? scale_of(*at) : need;
      s_new[tid] = fmaxf(need, s_old[tid]);
      *at = s_new[tid];
    }
    __syncthreads();
    uint8_t *const k0 = reinterpret_cast<uint8_t *>(a.c.k) + block * a.c.block_stride + h * a.c.head_stride;
    uint8_t *const v0 = reinterpret_cast<uint8_t *>(a.c.v) + block * a.c.block_stride + h * a.c.head_stride;
    for (int which = 0; which < 2; ++which) {  // tokens ahead of the new ones
      const float f = s_old[which] / s_new[which];
      if (f == 1.f) continue;
      for (int t = warp; t < off; t += kWarps8) {
        uint8_t *x = (which ? v0 : k0) + t * a.c.token_stride;
        for (int d = lane; d < D; d += 32) x[d] = static_cast<uint8_t>(rescale_e4m3x4(x[d], f));
      }
    }
    for (int i = warp; i < run.n; i += kWarps8) {
      const int pos = position(i);
      if (pos < 0) continue;
      const float *cs = a.rope + static_cast<int64_t>(pos) * a.rot;
      const float r = norm_of(a, key(i), kw);
      const int64_t token = (off + i) * a.c.token_stride;
      for (int d = lane; d < D; d += 32) {
        const float y = finite_or_nan(turned(a, key(i), kw, r, cs, d));
        k0[token + d] = static_cast<uint8_t>(to_e4m3x2(y / s_new[0], 0.f));
        v0[token + d] = static_cast<uint8_t>(to_e4m3x2(finite_or_nan(to_f32(value(i)[d])) / s_new[1], 0.f));
      }
      for (int g = h; g < a.q_heads; g += a.c.kv_heads) {
        const T *src = reinterpret_cast<const T *>(a.q) + (run.row + i) * a.q_row + g * a.q_head;
        T *dst = reinterpret_cast<T *>(a.out) + (run.row + i) * a.o_row + g * a.o_head;
        const float rq = norm_of(a, src, qw);
        T out[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (lane + 32 * e < D) out[e] = from_f32<T>(turned(a, src, qw, rq, cs, lane + 32 * e));
        }
        __syncwarp();  // q_out may be q: every lane has read its pairs
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (lane + 32 * e < D) dst[lane + 32 * e] = out[e];
        }
        __syncwarp();
      }
    }
  }
}

// ---------------------------------------------------------------------------
// The same with 16-byte accesses: a vector per group of kLanes lanes.  A run's
// keys and values are dealt to the groups, computed once, and stay in registers
// while the largest of them is found (kKept vectors a group; what is more is
// computed again).  The queries, which need no scale, are other CTAs' work, where
// a row's angles and weights serve several heads.
//   A run is a chain of dependent loads (offsets, lengths, table, rows, the block's
// scale), and what hides one is other runs: the registers are bound to what 32
// warps a multiprocessor have, though some go to local memory.  12535 rows of 32 +
// 8 + 8 heads, 300 MB: 135 us, 2.2 TB/s (24 warps 156, 16 without a spill 195; keys,
// values and queries in one CTA, 16 warps, 185; CTAs of 512 threads 135).  1280
// rows, 29 MB: 21 us, with CTAs of 256 threads throughout 46.
// ---------------------------------------------------------------------------
constexpr int kKept = 2;
constexpr int kQueryCtas = 912;  // (with 24 warps: half as many 22.9 and 156 us, these 20.3 and 156, four times as many 21.6 and 162)
constexpr int kAhead8 = 4;  // queries of a group whose loads are under way at once

template <typename T, int kLanes, bool kInter>
__global__ void __launch_bounds__(kThreads8, 4)
append8_vectors_kernel(const __grid_constant__ QkArgs a, const __grid_constant__ ScaleArgs sc, int per) {
  constexpr int E = 16 / sizeof(T);
  __shared__ int s_top[2];
  __shared__ float s_old[2], s_new[2];
  const int tid = threadIdx.x, h = blockIdx.y, vec = tid % kLanes, group = tid / kLanes, groups = blockDim.x / kLanes;
  const int bs = a.c.block_size, d0 = vec * E, half = a.rot / 2;
  Turn<T, kLanes, kInter> turn;
  turn.place(a);
  const bool has = turn.has;
  const float inv_dim = 1.f / a.c.head_dim;
  // CTAs past those of the key heads take query heads h0, h0 + parts, ...
  const bool queries = h >= a.c.kv_heads;
  const int parts = gridDim.y - a.c.kv_heads, h0 = h - a.c.kv_heads, nq = (a.q_heads - h0 + parts - 1) / parts;
  wait_for_stream();
  const int r0 = blockIdx.x * per;
  Runs runs(a, r0, min(r0 + per, a.b.rows));
  for (Run run = runs.next(a); run.n > 0; run = runs.next(a)) {
    const int block = a.b.tables[static_cast<int64_t>(run.seq) * a.b.T + run.at / bs], off = run.at % bs, n = run.n;
    if (block < 0 || block >= a.c.blocks) {
      if (h == 0 && tid == 0) raise_status(a.status, SMC_DEV_BAD_BLOCK);
      continue;
    }
    auto position = [&](int i) {  // a row's, -1 out of range
      const int p = a.positions ? a.positions[run.row + i] : run.at + i;
      return p >= 0 && p < a.max_pos ? p : -1;
    };
    auto table_of = [&](int pos) { return a.rope + static_cast<int64_t>(pos) * a.rot; };
    auto fetch = [&](const char *base, int64_t row_stride, int64_t head_stride, int i, int head) {
      return has ? *reinterpret_cast<const uint4 *>(base + ((run.row + i) * row_stride + head * head_stride) *
                                                               static_cast<int64_t>(sizeof(T)) + vec * 16)
                 : make_uint4(0, 0, 0, 0);
    };
    if (queries) {
      // Queries: a group takes rows group, group + groups, ..., and with fewer rows than groups, as many groups share a row's heads.
      const int share = n < groups ? groups / n : 1, phase = n < groups ? group / n : 0;
      const int q_row0 = n < groups ? group - phase * n : group, q_step = groups;
      const int64_t head_step = static_cast<int64_t>(share) * parts * a.q_head * static_cast<int64_t>(sizeof(T)),
                    out_step = static_cast<int64_t>(share) * parts * a.o_head * static_cast<int64_t>(sizeof(T));
      const bool any_q = phase < share && has;
      auto query_at = [&](int i) {
        return a.q + ((run.row + i) * a.q_row + (h0 + phase * parts) * a.q_head) * static_cast<int64_t>(sizeof(T)) + vec * 16;
      };
      for (int i0 = 0; i0 < n; i0 += q_step) {
        const int i = i0 + q_row0, pos = i < n ? position(i) : -1;
        const bool writes = any_q && pos >= 0;
        char *out = a.out + ((run.row + i) * a.o_row + (h0 + phase * parts) * a.o_head) * static_cast<int64_t>(sizeof(T)) + vec * 16;
        const char *q = query_at(i);
        for (int g0 = 0; g0 < nq; g0 += kAhead8 * share) {  // (of phase 0: the same number of turns for all lanes)
          uint4 rq[kAhead8];
#pragma unroll
          for (int t = 0; t < kAhead8; ++t) {
            rq[t] = any_q && i < n && g0 + phase + t * share < nq ? *reinterpret_cast<const uint4 *>(q + t * head_step)
                                                                   : make_uint4(0, 0, 0, 0);
          }
          if (g0 == 0 && pos >= 0) turn.load(a, table_of(pos), a.qw);
#pragma unroll
          for (int t = 0; t < kAhead8; ++t) {
            if (g0 + t * share >= nq) break;  // for the whole CTA
            const uint4 z = turn.apply(rq[t], a.qw != nullptr, inv_dim, a.eps);
            if (writes && g0 + phase + t * share < nq) *reinterpret_cast<uint4 *>(out + t * out_step) = z;
          }
          q += kAhead8 * head_step;
          out += kAhead8 * out_step;
        }
      }
      continue;
    }
    // (read early: its use is at the end of a chain of loads)
    float *const scale_at = (tid == 1 ? sc.v : sc.k) + block * sc.block + h * sc.head;
    const float before = tid < 2 && off ? *scale_at : 0.f;
    // item j < n: key of row j; j < 2n: value of row j - n.  All lanes of a warp call it.
    auto item = [&](int j, float *z) {
      const bool key = j < n;
      const int i = key ? j : j - n;
      const bool in = j < 2 * n;
      const uint4 raw = in ? (key ? fetch(a.k, a.k_row, a.k_head, i, h) : fetch(a.v, a.v_row, a.v_head, i, h)) : make_uint4(0, 0, 0, 0);
      const int pos = in ? position(i) : -1;
      float x[E], y[E];
      unpack16<T>(raw, x);
#pragma unroll
      for (int e = 0; e < E; ++e) z[e] = x[e];
      if (__any_sync(0xffffffffu, key)) {
        if (a.kw) {
          float sum = 0.f, w[E];
#pragma unroll
          for (int e = 0; e < E; ++e) sum = fmaf(x[e], x[e], sum);
#pragma unroll
          for (int o = kLanes / 2; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o, kLanes);
          const float r = rsqrtf(fmaf(sum, inv_dim, a.eps));
          if (has) unpack16<T>(reinterpret_cast<const uint4 *>(a.kw)[vec], w);
#pragma unroll
          for (int e = 0; e < E; ++e) {
            if (key && has) z[e] = x[e] = __fmul_rn(__fmul_rn(x[e], r), w[e] + a.w0);
          }
        }
#pragma unroll
        for (int e = 0; e < E; ++e) y[e] = kInter ? x[e ^ 1] : __shfl_sync(0xffffffffu, x[e], turn.other);
        if (key && pos >= 0 && turn.turns) {
          const float *cs = table_of(pos) + (kInter ? d0 / 2 : turn.second ? d0 - half : d0);
          constexpr int kAngles = kInter ? E / 2 : E;
          alignas(16) float c[kAngles], sn[kAngles];
          if constexpr (kAngles % 4 == 0) {
#pragma unroll
            for (int e = 0; e < kAngles; e += 4) {
              *reinterpret_cast<float4 *>(c + e) = *reinterpret_cast<const float4 *>(cs + e);
              *reinterpret_cast<float4 *>(sn + e) = *reinterpret_cast<const float4 *>(cs + half + e);
            }
          } else {
#pragma unroll
            for (int e = 0; e < kAngles; ++e) {
              c[e] = cs[e];
              sn[e] = cs[half + e];
            }
          }
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const bool second = kInter ? e & 1 : turn.second;
            const float p = __fmul_rn(x[e], c[kInter ? e / 2 : e]), q = __fmul_rn(y[e], sn[kInter ? e / 2 : e]);
            z[e] = second ? __fadd_rn(q, p) : __fsub_rn(p, q);
          }
        }
      }
      return has && pos >= 0;
    };
    auto largest = [&](const float *z) {
      float top = 0.f;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const float v = fabsf(z[e]);
        if (v < INFINITY) top = fmaxf(top, v);
      }
      return top;
    };
    __syncthreads();
    if (tid < 2) s_top[tid] = 0;
    if (tid < n && h == 0 && position(tid) < 0) raise_status(a.status, SMC_DEV_BAD_ROWS);
    for (int i = tid + blockDim.x; i < n; i += blockDim.x) {
      if (h == 0 && position(i) < 0) raise_status(a.status, SMC_DEV_BAD_ROWS);
    }
    float kept[kKept][E];
    bool live[kKept];
    float top[2] = {0.f, 0.f};
#pragma unroll
    for (int t = 0; t < kKept; ++t) {
      live[t] = false;
      if (t * groups >= 2 * n) break;  // for the whole CTA
      const int j = group + t * groups;
      live[t] = item(j, kept[t]);
      const float m = live[t] ? largest(kept[t]) : 0.f;
      if (j < n) top[0] = fmaxf(top[0], m); else top[1] = fmaxf(top[1], m);
    }
    for (int j0 = kKept * groups; j0 < 2 * n; j0 += groups) {
      float z[E];
      const int j = j0 + group;
      const float m = item(j, z) ? largest(z) : 0.f;
      if (j < n) top[0] = fmaxf(top[0], m); else top[1] = fmaxf(top[1], m);
    }
    __syncthreads();  // s_top is clear
#pragma unroll
    for (int w = 0; w < 2; ++w) {
      const int m = __reduce_max_sync(0xffffffffu, __float_as_int(top[w]));  // of positive numbers: their bits' order
      if ((tid & 31) == 0 && m) atomicMax(&s_top[w], m);
    }
    __syncthreads();
    if (tid < 2) {
      const float need = least_scale(__int_as_float(s_top[tid]));
      s_old[tid] = off ? scale_of(before) : need;
      s_new[tid] = fmaxf(need, s_old[tid]);
      *scale_at = s_new[tid];
    }
    __syncthreads();
    char *const to[2] = {a.c.k + block * a.c.block_stride + h * a.c.head_stride,
                         a.c.v + block * a.c.block_stride + h * a.c.head_stride};
    auto store = [&](int j, const float *z) {
      const int which = j >= n;
      const float scale = s_new[which];
      uint32_t words[E / 4];
      // a power of two's reciprocal is exact
      const bool power = (__float_as_uint(scale) & 0x7fffffu) == 0;
      const float inv = __uint_as_float((254u << 23) - __float_as_uint(scale));
#pragma unroll
      for (int e = 0; e < E; e += 4) {
        float v[4];
#pragma unroll
        for (int f = 0; f < 4; ++f) v[f] = power ? finite_or_nan(z[e + f]) * inv : finite_or_nan(z[e + f]) / scale;
        words[e / 4] = to_e4m3x2(v[0], v[1]) | to_e4m3x2(v[2], v[3]) << 16;
      }
      char *dst = to[which] + (off + (which ? j - n : j)) * a.c.token_stride + d0;
      if constexpr (E == 8) *reinterpret_cast<uint2 *>(dst) = make_uint2(words[0], words[1]);
      else *reinterpret_cast<uint32_t *>(dst) = words[0];
    };
#pragma unroll
    for (int t = 0; t < kKept; ++t) {
      if (live[t]) store(group + t * groups, kept[t]);
    }
    for (int j0 = kKept * groups; j0 < 2 * n; j0 += groups) {
      float z[E];
      if (item(j0 + group, z)) store(j0 + group, z);
    }
    for (int which = 0; which < 2; ++which) {  // tokens ahead of the new ones
      const float f = s_old[which] / s_new[which];
      if (f == 1.f || !has) continue;
      for (int t = group; t < off; t += groups) {
        uint32_t *x = reinterpret_cast<uint32_t *>(to[which] + t * a.c.token_stride + d0);
#pragma unroll
        for (int e = 0; e < E / 4; ++e) x[e] = rescale_e4m3x4(x[e], f);
      }
    }
  }
}

// Whether rows and weights are 16-byte vectors that turn as a whole, and the
// cache's are aligned to what becomes of one.
static bool vectors8_ok(const QkArgs &a, int dtype) {
  const int esz = dtype_bytes(dtype), E = 16 / esz;
  uint64_t all = reinterpret_cast<uintptr_t>(a.q) | reinterpret_cast<uintptr_t>(a.k) |
                 reinterpret_cast<uintptr_t>(a.v) | reinterpret_cast<uintptr_t>(a.out) |
                 reinterpret_cast<uintptr_t>(a.qw) | reinterpret_cast<uintptr_t>(a.kw) |
                 reinterpret_cast<uintptr_t>(a.rope);
  uint64_t cache = reinterpret_cast<uintptr_t>(a.c.k) | reinterpret_cast<uintptr_t>(a.c.v);
  const int rows = a.b.rows, Hk = a.c.kv_heads;
  auto stride = [&](int64_t s, int n) { if (n > 1) all |= static_cast<uint64_t>(s) * esz; };
  stride(a.q_row, rows); stride(a.k_row, rows); stride(a.v_row, rows); stride(a.o_row, rows);
  stride(a.q_head, a.q_heads); stride(a.o_head, a.q_heads);
  stride(a.k_head, Hk); stride(a.v_head, Hk);
  cache |= static_cast<uint64_t>(a.c.head_stride) | static_cast<uint64_t>(a.c.token_stride) |
           static_cast<uint64_t>(a.c.block_stride);
  return all % 16 == 0 && cache % E == 0 && a.c.head_dim % E == 0 && a.c.head_dim <= 32 * E && a.rot % E == 0 &&
         (a.interleaved || a.rot / 2 % E == 0);
}

template <typename T, bool kInter>
static const void *vectors8_fn(int lanes) {
  return lanes == 8    ? reinterpret_cast<const void *>(append8_vectors_kernel<T, 8, kInter>)
         : lanes == 16 ? reinterpret_cast<const void *>(append8_vectors_kernel<T, 16, kInter>)
                       : reinterpret_cast<const void *>(append8_vectors_kernel<T, 32, kInter>);
}

template <typename T>
static const void *vectors8_fn(const QkArgs &a, int lanes) {
  return a.interleaved ? vectors8_fn<T, true>(lanes) : vectors8_fn<T, false>(lanes);
}

cudaError_t launch_qk_norm_rope8(const QkArgs &a, const ScaleArgs &s, int dtype, cudaStream_t st) {
  if (a.b.rows == 0) return cudaSuccess;
  int per = a.c.block_size < a.b.max_new ? a.c.block_size : a.b.max_new;
  ScaleArgs scales = s;
  if (vectors8_ok(a, dtype)) {
    const int vectors = a.c.head_dim * dtype_bytes(dtype) / 16, lanes = vectors <= 8 ? 8 : vectors <= 16 ? 16 : 32;
    const void *fn = dtype == SMC_F32    ? vectors8_fn<float>(a, lanes)
                     : dtype == SMC_BF16 ? vectors8_fn<__nv_bfloat16>(a, lanes)
                                         : vectors8_fn<__half>(a, lanes);
    // a group of lanes for every row, whose key and value it keeps: with few rows a CTA is a small one, so that more
    // of their chains of dependent loads run side by side
    const int64_t most = static_cast<int64_t>(per) * lanes;
    const int threads = most >= kThreads8 ? kThreads8 : most <= 64 ? 64 : static_cast<int>((most + 31) / 32 * 32);
    // queries: CTAs to fill the multiprocessors, and no more: a row's angles and weights serve all heads of a CTA
    const int groups = (a.b.rows + per - 1) / per, most_parts = a.q_heads < a.c.kv_heads ? a.q_heads : a.c.kv_heads;
    int parts = (kQueryCtas + groups - 1) / groups;
    parts = parts > most_parts ? most_parts : parts;
    parts = parts > 65535 - a.c.kv_heads ? 65535 - a.c.kv_heads : parts;  // (the grid's second axis)
    void *args[] = {const_cast<QkArgs *>(&a), &scales, &per};
    return launch_early(fn, dim3(groups, a.c.kv_heads + parts), threads, 0, args, st);
  }
  const void *fn = dtype == SMC_F32    ? reinterpret_cast<const void *>(append8_kernel<float>)
                   : dtype == SMC_BF16 ? reinterpret_cast<const void *>(append8_kernel<__nv_bfloat16>)
                                       : reinterpret_cast<const void *>(append8_kernel<__half>);
  void *args[] = {const_cast<QkArgs *>(&a), &scales, &per};
  return launch_early(fn, dim3((a.b.rows + per - 1) / per, a.c.kv_heads), kThreads8, 0, args, st);
}

}  // namespace smcsd

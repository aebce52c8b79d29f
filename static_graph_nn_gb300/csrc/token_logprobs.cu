// Log probabilities of given tokens, the entropy of each row's distribution and
// its most likely tokens, and their gradient.
//
// With z = x / T over a row x of logits, m = max x and L = log sum exp((x - m) / T):
//   logp    = (x[id] - m) / T - L
//   entropy = L - sum_v p_v (x_v - m) / T        p_v = exp((x_v - m) / T - L)
//   dx_v    = (g (1[v = id] - p_v) - h p_v (log p_v + entropy)) / T
//
// Forward: one read of the logits.  A thread keeps the maximum of its own elements
// and, relative to it and in base 2, the sums of 2^t and of 2^t t; the block joins
// them.  A block takes a row; few rows are split over a cluster of up to eight
// blocks, whose results meet in the first one's shared memory.
//
// The k most likely: the k-th largest of the threads' maxima (of 64 groups of them) is
// at most the k-th largest element, and few elements are as large.  The four units
// that hold a thread's maximum, or all of its units where its other maxima are as large
// too, are read again by all threads side by side, what is at least that large is
// listed, and the list is ranked.  Where equal values make the list too long, the
// smaller ones are left out and found in order of their places.
//
// Bound by DRAM: 16384 x 32000 bf16 with a tenth of padding 144 us (6.5 TB/s; with one
// chunk of four units on its way to a thread instead of two 152), its gradient 300 us
// (6.65 TB/s); without padding 155 us, with 5 alternatives 186, with 32 226.  1037 x 50021
// fp32, 5 alternatives: 37.5 us (5.3 TB/s; all rows at once, so their ends meet).
#include <cmath>

#include "common.cuh"
#include "f32x2.cuh"
#include "kernels.h"
#include "op_checks.h"

namespace mg {
namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kNothing = -1000.0f;     // as an exponent of 2: 0, and finite
constexpr int kLogpList = 512;           // candidates that are ranked
constexpr int kLogpOwners = 64;          // threads whose elements are read again
constexpr int kMaxCluster = 8;
constexpr int kLogpShort = 384;          // units of 16 bytes of a short row

struct LogpArgs {
  const void* logits;
  long long stride;
  int vocab;
  const void* ids;
  int id64;
  float inv_t;
  float* logp;
  float* stats;
  float* entropy;
  int k;
  int* top_ids;
  float* top_logp;
};

struct LogpGradArgs {
  const void* logits;
  long long stride;
  int vocab;
  const void* ids;
  int id64;
  float inv_t;
  const float* stats;
  const float* entropy;
  const float* dlogp;
  const float* dentropy;
  void* dlogits;
  long long dstride;
};

// The given token of row r; -1 for one outside the vocabulary.
__device__ __forceinline__ int token_of(const void* ids, int id64, int vocab, size_t r) {
  const long long id = id64 ? static_cast<const long long*>(ids)[r] : static_cast<const int*>(ids)[r];
  return id >= 0 && id < vocab ? (int)id : -1;
}

// An integer that orders floats: NaN least, then -inf; -0 equals +0.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0;
  const uint32_t b = __float_as_uint(x + 0.0f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

__device__ __forceinline__ float key_value(uint32_t key) {
  return __uint_as_float(key & 0x80000000u ? key & 0x7fffffffu : ~key);   // (of 0, which is NaN's: NaN)
}
// A value and its place in one integer: larger values first, of equal ones the lower place.
__device__ __forceinline__ unsigned long long place_key(float x, int c) {
  return (unsigned long long)order_key(x) << 32 | (uint32_t)~c;
}

__device__ __forceinline__ float exp2_near(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
// The larger one, NaN if one is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

// ---- a part of a row: whole 16-byte units, and single elements before and behind them
template <typename T>
struct Part {
  static constexpr int kPer = 16 / (int)sizeof(T);
  const T* x;        // its first element
  int at;            // that element's place in the row
  int head, units, tail;
  __device__ __forceinline__ const uint4* unit(int u) const { return reinterpret_cast<const uint4*>(x + head) + u; }
  __device__ __forceinline__ int unit_place(int u) const { return at + head + u * kPer; }
  __device__ __forceinline__ const T* behind() const { return x + head + (size_t)units * kPer; }
  __device__ __forceinline__ int count() const { return head + units * kPer + tail; }
};
// The part of rank `rank` of `ranks`: the units split evenly, the row's ends with the outer ones.
template <typename T>
__device__ __forceinline__ Part<T> part_of(const T* row, int n, int rank, int ranks) {
  Part<T> p;
  const int off = (int)((16 - reinterpret_cast<uintptr_t>(row) % 16) % 16 / sizeof(T));
  const int head = min(off, n), units = (n - head) / Part<T>::kPer, tail = n - head - units * Part<T>::kPer;
  const int begin = (int)((long long)units * rank / ranks), end = (int)((long long)units * (rank + 1) / ranks);
  p.units = end - begin;
  p.head = rank == 0 ? head : 0;
  p.tail = rank == ranks - 1 ? tail : 0;
  p.at = rank == 0 ? 0 : head + begin * Part<T>::kPer;
  p.x = row + p.at;
  return p;
}
__device__ __forceinline__ void widen(const uint4& u, f32x2 (&f)[4]) {
  f[0] = widen2(u.x);
  f[1] = widen2(u.y);
  f[2] = widen2(u.z);
  f[3] = widen2(u.w);
}
__device__ __forceinline__ void widen(const uint4& u, f32x2 (&f)[2]) {
  f[0] = both(__uint_as_float(u.x), __uint_as_float(u.y));
  f[1] = both(__uint_as_float(u.z), __uint_as_float(u.w));
}
__device__ __forceinline__ uint4 narrow(const f32x2 (&f)[4]) {
  return make_uint4(narrow2(f[0]), narrow2(f[1]), narrow2(f[2]), narrow2(f[3]));
}
__device__ __forceinline__ uint4 narrow(const f32x2 (&f)[2]) {
  const float2 a = parts(f[0]), b = parts(f[1]);
  return make_uint4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x), __float_as_uint(b.y));
}
// The largest of N units' values (a NaN only if all are).
template <int N>
__device__ __forceinline__ float units_max(const uint4 (&u)[N], bf16) {
  __nv_bfloat162 m = *reinterpret_cast<const __nv_bfloat162*>(&u[0].x);
#pragma unroll
  for (int q = 0; q < N; ++q) {
    const uint32_t w[4] = {u[q].x, u[q].y, u[q].z, u[q].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) m = __hmax2(m, *reinterpret_cast<const __nv_bfloat162*>(&w[i]));
  }
  const float2 f = __bfloat1622float2(m);
  return fmaxf(f.x, f.y);
}
template <int N>
__device__ __forceinline__ float units_max(const uint4 (&u)[N], float) {
  float m = __uint_as_float(u[0].x);
#pragma unroll
  for (int q = 0; q < N; ++q)
    m = fmaxf(fmaxf(fmaxf(m, __uint_as_float(u[q].x)), fmaxf(__uint_as_float(u[q].y), __uint_as_float(u[q].z))),
              __uint_as_float(u[q].w));
  return m;
}

// The maximum m of some elements, and with t = (x - m) / T in base 2 the sums of 2^t and of 2^t t.
struct RowSums {
  float m, s, q;
  // relative to a larger maximum
  __device__ __forceinline__ void lift(float to, float c) {
    const float d = max_nan((m - (to == -INFINITY ? 0.0f : to)) * c, kNothing), f = exp2_near(d);
    q = f * fmaf(s, d, q);
    s *= f;
    m = to;
  }
  __device__ __forceinline__ void one(float x, float c) {
    if (x > m) lift(x, c);
    const float t = max_nan((x - (m == -INFINITY ? 0.0f : m)) * c, kNothing), e = exp2_near(t);
    s += e;
    q = fmaf(e, t, q);
  }
};

// The block's sums of both, relative to one maximum.
__device__ __forceinline__ void block_sums(RowSums& t, float (&red)[2][32]) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, nw = blockDim.x >> 5;
  t.s = warp_sum(t.s);
  t.q = warp_sum(t.q);
  if (lane == 0) {
    red[0][w] = t.s;
    red[1][w] = t.q;
  }
  __syncthreads();
  t.s = warp_sum(lane < nw ? red[0][lane] : 0.0f);
  t.q = warp_sum(lane < nw ? red[1][lane] : 0.0f);
}

// Where a thread's maximum is: in its chunk (of four units) of this number, -1 for one of the
// row's single elements; and the largest of its other chunks' maxima.
struct RowBest {
  int chunk;
  float others;
};
// Four units of the part from u0 on, a block's width apart; -inf behind the part.
template <typename T>
__device__ __forceinline__ void fetch_chunk(const Part<T>& p, int u0, uint4 (&u)[4]) {
  constexpr uint32_t kNone = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;
  const int step = blockDim.x;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    u[i] = u0 + i * step < p.units ? *p.unit(u0 + i * step) : make_uint4(kNone, kNone, kNone, kNone);
}
// A thread's sums; one: its first chunk.
template <typename T>
__device__ __forceinline__ RowSums row_sums(const Part<T>& p, float c, uint4 (&one)[4], RowBest& best) {
  constexpr int pairs = Part<T>::kPer / 2;
  RowSums r = {-INFINITY, 0.0f, 0.0f};
  best = {-1, -INFINITY};
  const int step = blockDim.x;
  const f32x2 cc = both(c);
  int chunk = 0;
  const auto add = [&](const uint4 (&u)[4]) {
    const float top = units_max(u, T());
    best.others = fmaxf(best.others, fminf(top, r.m));
    if (top > r.m) {
      best.chunk = chunk;
      r.lift(top, c);
    }
    const f32x2 minus = both(r.m == -INFINITY ? 0.0f : -r.m);
    f32x2 s = both(0.0f), q = both(0.0f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f32x2 f[pairs];
      widen(u[i], f);
#pragma unroll
      for (int j = 0; j < pairs; ++j) {
        const float2 d = parts(mul2(add2(f[j], minus), cc));
        const float a = max_nan(d.x, kNothing), b = max_nan(d.y, kNothing);
        const f32x2 e = both(exp2_near(a), exp2_near(b));
        s = add2(s, e);
        q = fma2(e, both(a, b), q);
      }
    }
    const float2 ss = parts(s), qq = parts(q);
    r.s += ss.x + ss.y;
    r.q += qq.x + qq.y;
    ++chunk;
  };
  // two chunks on their way at any time
  uint4 two[4];
  fetch_chunk(p, threadIdx.x + 4 * step, two);
  for (int u0 = threadIdx.x; u0 < p.units; u0 += 8 * step) {
    add(one);
    fetch_chunk(p, u0 + 8 * step, one);
    if (u0 + 4 * step >= p.units) break;
    add(two);
    fetch_chunk(p, u0 + 12 * step, two);
  }
  const auto single = [&](float x) {
    if (x > r.m) {
      best.others = fmaxf(best.others, r.m);
      best.chunk = -1;
    }
    r.one(x, c);
  };
  if ((int)threadIdx.x < p.head) single(ld_elem(p.x, threadIdx.x));
  if ((int)threadIdx.x < p.tail) single(ld_elem(p.behind(), threadIdx.x));
  return r;
}

// ---- the most likely ------------------------------------------------------------
constexpr uint32_t kLeastKey = 0x007fffffu;   // of -inf

struct TopShared {
  alignas(16) uint32_t groups[64];            // maxima of groups of threads: keys, their last six bits the group's
  uint32_t maxima[512];                       // the threads', as keys
  unsigned long long list[kLogpList];
  int owner[kLogpOwners];                     // of all of whose units may hold some
  int2 chunk[kLogpOwners];                    // the only ones that may: a thread's
  int n_owners, n_chunks, n_list, n_more;
  uint32_t threshold;
  unsigned long long best[MG_MAX_TOP];        // in order; 0 where there are fewer
};

// A little below the k-th largest of the G groups' maxima: each of G threads counts those above its own.
template <int G>
__device__ __forceinline__ void kth_group(TopShared& t, int k) {
  if (threadIdx.x >= G) return;
  const uint32_t v = t.groups[threadIdx.x];
  int above = 0;
#pragma unroll
  for (int j = 0; j < G; j += 4) {
    const uint4 w = *reinterpret_cast<const uint4*>(t.groups + j);
    above += (w.x > v) + (w.y > v) + (w.z > v) + (w.w > v);
  }
  if (above == k - 1) t.threshold = v & ~63u;
}
// Exactly the k-th largest of the threads' maxima.
__device__ __forceinline__ void kth_maximum(TopShared& t, int k) {
  const uint32_t v = t.maxima[threadIdx.x];
  int before = 0;
  for (int j = 0; j < (int)blockDim.x; ++j) before += t.maxima[j] > v || (t.maxima[j] == v && j < (int)threadIdx.x);
  if (before == k - 1) t.threshold = v;
}

// Every element of the part: f(value, place in the row).
template <typename T, typename F>
__device__ __forceinline__ void each_of_unit(const Part<T>& p, int u, const uint4& w, F&& f) {
  f32x2 v[Part<T>::kPer / 2];
  widen(w, v);
#pragma unroll
  for (int j = 0; j < Part<T>::kPer / 2; ++j) {
    const float2 d = parts(v[j]);
    f(d.x, p.unit_place(u) + 2 * j);
    f(d.y, p.unit_place(u) + 2 * j + 1);
  }
}
template <typename T, typename F>
__device__ __forceinline__ void each_element(const Part<T>& p, F&& f) {
  for (int u = threadIdx.x; u < p.units; u += blockDim.x) each_of_unit(p, u, *p.unit(u), f);
  if ((int)threadIdx.x < p.head) f(ld_elem(p.x, threadIdx.x), p.at + threadIdx.x);
  if ((int)threadIdx.x < p.tail) f(ld_elem(p.behind(), threadIdx.x), p.at + p.count() - p.tail + threadIdx.x);
}

// Lists the elements whose keys are at least `least` (that of -inf or more), of the
// threads whose maxima are; false if there are more than the list holds.  The counts
// are 0 before.
template <typename T>
__device__ bool list_from(const Part<T>& p, TopShared& t, const RowBest& best, uint32_t least) {
  const bool mine = t.maxima[threadIdx.x] >= least;
  if (mine && order_key(best.others) >= least) {
    const int i = atomicAdd(&t.n_owners, 1);
    if (i < kLogpOwners) t.owner[i] = threadIdx.x;
  } else if (mine && best.chunk >= 0) {
    const int i = atomicAdd(&t.n_chunks, 1);
    if (i < kLogpOwners) t.chunk[i] = make_int2(threadIdx.x, best.chunk);
  }
  __syncthreads();
  const int owners = t.n_owners, chunks = t.n_chunks;
  if (owners > kLogpOwners || chunks > kLogpOwners) return false;
  const float from = key_value(least);
  const auto add = [&](float x, int c) {
    if (!(x >= from)) return;
    const int i = atomicAdd(&t.n_list, 1);
    if (i < kLogpList) t.list[i] = place_key(x, c);
  };
  const auto look = [&](int u) {
    if (u >= p.units) return;
    const uint4 w[1] = {*p.unit(u)};
    if (units_max(w, T()) >= from) each_of_unit(p, u, w[0], add);
  };
  for (int i = threadIdx.x; i < 4 * chunks; i += blockDim.x) {
    const int2 at = t.chunk[i / 4];
    look(at.x + (4 * at.y + i % 4) * (int)blockDim.x);
  }
  const int rounds = (p.units + blockDim.x - 1) / blockDim.x;   // units of a thread at most
  // a thread takes every blockDim.x-th of the owners' units, one owner after the other
  if (rounds && owners) {
    const int skip = blockDim.x / rounds, rest = blockDim.x % rounds;
    for (int o = threadIdx.x / rounds, j = threadIdx.x % rounds; o < owners;) {
      look(t.owner[o] + j * (int)blockDim.x);
      o += skip;
      j += rest;
      if (j >= rounds) {
        j -= rounds;
        ++o;
      }
    }
  }
  if (mine) {
    if ((int)threadIdx.x < p.head) add(ld_elem(p.x, threadIdx.x), p.at + threadIdx.x);
    if ((int)threadIdx.x < p.tail) add(ld_elem(p.behind(), threadIdx.x), p.at + p.count() - p.tail + threadIdx.x);
  }
  __syncthreads();
  return t.n_list <= kLogpList;
}

// The listed keys in order to t.best[0 .. k-1]; returns after a barrier.
__device__ __forceinline__ void rank_list(TopShared& t, int n, int k) {
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const unsigned long long v = t.list[i];
    int above = 0;
    for (int j = 0; j < n; ++j) above += t.list[j] > v;
    if (above < k) t.best[above] = v;
  }
  __syncthreads();
}

// The part's k largest (fewer if it has fewer) in order in t.best.
template <typename T, int N>
__device__ void top_of_part(const Part<T>& p, TopShared& t, int k, float maximum, const RowBest& best) {
  k = min(k, p.count());
  const bool any = (int)threadIdx.x < p.units || (int)threadIdx.x < p.head || (int)threadIdx.x < p.tail;
  constexpr int G = N < 64 ? N : 64;
  uint32_t key = any ? order_key(maximum) : 0u;
  t.maxima[threadIdx.x] = key;
#pragma unroll
  for (int o = 1; o < N / G; o *= 2) key = max(key, __shfl_xor_sync(0xffffffffu, key, o));
  if (threadIdx.x % (N / G) == 0) t.groups[threadIdx.x / (N / G)] = (key & ~63u) | threadIdx.x / (N / G);
  if (threadIdx.x < MG_MAX_TOP) t.best[threadIdx.x] = 0;
  if (threadIdx.x == 0) t.n_owners = t.n_chunks = t.n_list = 0;
  __syncthreads();
  if (k == 0) return;
  kth_group<G>(t, k);
  __syncthreads();
  uint32_t th = t.threshold;
  if (th > kLeastKey && list_from(p, t, best, th) && t.n_list >= k) {
    rank_list(t, t.n_list, k);
    return;
  }
  // Too many equal ones, few that are not -inf, or (behind maxima of -inf that are NaN)
  // too few: those above the exact threshold, then equal ones in order of their places.
  __syncthreads();
  kth_maximum(t, k);
  if (threadIdx.x == 0) t.n_owners = t.n_chunks = t.n_list = 0;
  __syncthreads();
  th = t.threshold;
  if (!list_from(p, t, best, max(th + 1, kLeastKey))) {
    // Many large values in few threads' hands: the exact k-th largest, bit by bit.
    uint32_t lo = 0;
    for (int bit = 31; bit >= 0; --bit) {
      const uint32_t mid = lo | 1u << bit;
      if (threadIdx.x == 0) t.n_more = 0;
      __syncthreads();
      int n = 0;
      each_element(p, [&](float x, int) { n += order_key(x) >= mid; });
      n = __reduce_add_sync(0xffffffffu, n);
      if ((threadIdx.x & 31) == 0) atomicAdd(&t.n_more, n);
      __syncthreads();
      if (t.n_more >= k) lo = mid;
      __syncthreads();
    }
    th = lo;
    if (threadIdx.x == 0) t.n_list = 0;
    __syncthreads();
    each_element(p, [&](float x, int c) {
      if (order_key(x) > th) t.list[atomicAdd(&t.n_list, 1)] = place_key(x, c);   // fewer than k
    });
    __syncthreads();
  }
  const int above = min(t.n_list, k);
  rank_list(t, t.n_list, k);
  // equal ones: of each step's elements in order, until there are enough
  int have = above;
  for (int round = 0; round < 2 && have < k; ++round, th = 0) {   // (the second: NaN)
    for (int c0 = 0; c0 < p.count() && have < k; c0 += blockDim.x) {
      const int i = c0 + threadIdx.x;
      const bool is = i < p.count() && order_key(ld_elem(p.x, i)) == th;
      const unsigned votes = __ballot_sync(0xffffffffu, is);
      const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
      if (lane == 0) t.owner[warp] = __popc(votes);
      __syncthreads();
      int before = have, all = have;
      for (int w = 0; w < (int)blockDim.x / 32; ++w) {
        if (w < warp) before += t.owner[w];
        all += t.owner[w];
      }
      before += __popc(votes & ((1u << lane) - 1));
      if (is && before < k) t.best[before] = (unsigned long long)th << 32 | (uint32_t)~(p.at + i);
      have = min(all, k);
      __syncthreads();
    }
    if (th == 0) break;
  }
}

// ---- clusters ---------------------------------------------------------------------
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Another block's shared memory at the place of p in this one's.
template <typename V>
__device__ __forceinline__ const V* of_rank(const V* p, int rank) {
  uint64_t r;
  asm("mapa.u64 %0, %1, %2;" : "=l"(r) : "l"((uint64_t)p), "r"(rank));
  return reinterpret_cast<const V*>(r);
}

// A row per cluster of blocks of N threads.
template <typename T, bool TOP, int N>
__global__ void __launch_bounds__(N) logp_kernel(LogpArgs a, int ranks) {
  __shared__ float red[32], red2[2][32];
  __shared__ RowSums mine;
  __shared__ TopShared top[1];   // (nothing refers to it without TOP)
  const size_t r = blockIdx.x / ranks;
  const int rank = blockIdx.x % ranks;
  const T* x = static_cast<const T*>(a.logits) + r * a.stride;
  const Part<T> p = part_of(x, a.vocab, rank, ranks);
  uint4 next[4];
  fetch_chunk(p, threadIdx.x, next);   // under way before the id says whether the row counts
  const int id = a.ids ? token_of(a.ids, a.id64, a.vocab, r) : 0;
  if (id < 0) {   // (in all blocks of the cluster)
    if (rank) return;
    if (threadIdx.x == 0) {
      a.logp[r] = 0.0f;
      if (a.stats) a.stats[2 * r] = a.stats[2 * r + 1] = 0.0f;
      if (a.entropy) a.entropy[r] = 0.0f;
    }
    for (int i = threadIdx.x; i < a.k; i += blockDim.x) {
      a.top_ids[r * a.k + i] = -1;
      a.top_logp[r * a.k + i] = 0.0f;
    }
    return;
  }
  const float given = threadIdx.x == 0 && rank == 0 && a.logp ? ld_elem(x, id) : 0.0f;   // (ahead of the row)
  const float c = a.inv_t * kLog2e;
  RowBest best;
  RowSums t = row_sums(p, c, next, best);
  const float maximum = t.m;
  t.lift(block_max(t.m, red), c);
  block_sums(t, red2);
  if (TOP) top_of_part<T, N>(p, top[0], a.k, maximum, best);
  if (ranks > 1) {
    if (threadIdx.x == 0) mine = t;
    cluster_sync();
    if (rank == 0) {
      RowSums all[kMaxCluster];
      float m = -INFINITY;
#pragma unroll
      for (int i = 0; i < kMaxCluster; ++i) {
        if (i < ranks) all[i] = *of_rank(&mine, i);
        m = i < ranks ? fmaxf(m, all[i].m) : m;
      }
      t = {m, 0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < kMaxCluster; ++i) {
        if (i >= ranks) continue;
        all[i].lift(m, c);
        t.s += all[i].s;
        t.q += all[i].q;
      }
      if (TOP) {
        for (int i = threadIdx.x; i < ranks * a.k; i += blockDim.x) top[0].list[i] = *of_rank(&top[0].best[i % a.k], i / a.k);
        __syncthreads();
        // (absent ones are 0, less than every element's key: their rank is not written)
        rank_list(top[0], ranks * a.k, a.k);
      }
    }
    cluster_sync();
    if (rank) return;
  }
  const float m = t.m == -INFINITY ? 0.0f : t.m, ls = logf(t.s);
  const bool none = t.s == 0.0f;   // every logit is -inf
  if (threadIdx.x == 0) {
    if (a.logp) a.logp[r] = none ? -INFINITY : (given - m) * a.inv_t - ls;
    if (a.stats) *reinterpret_cast<float2*>(a.stats + 2 * r) = make_float2(t.m, ls);
    if (a.entropy) a.entropy[r] = none ? 0.0f : ls - t.q / t.s * kLn2;
  }
  if (TOP) {
    for (int i = threadIdx.x; i < a.k; i += blockDim.x) {
      const unsigned long long v = top[0].best[i];
      a.top_ids[r * a.k + i] = (int)~(uint32_t)v;
      a.top_logp[r * a.k + i] = none ? -INFINITY : (key_value((uint32_t)(v >> 32)) - m) * a.inv_t - ls;
    }
  }
}

// ---- gradient -----------------------------------------------------------------------
// A block takes a row, or one of `ranks` parts of it.
template <typename T>
__global__ void __launch_bounds__(256) logp_grad_kernel(LogpGradArgs a, int ranks) {
  constexpr int per = Part<T>::kPer, pairs = per / 2;
  const size_t r = blockIdx.x / ranks;
  const T* x = static_cast<const T*>(a.logits) + r * a.stride;
  T* dx = static_cast<T*>(a.dlogits) + r * a.dstride;
  const int id = a.ids ? token_of(a.ids, a.id64, a.vocab, r) : 0;
  const float g = a.dlogp && id >= 0 ? a.dlogp[r] * a.inv_t : 0.0f;
  const float h = a.dentropy && id >= 0 ? a.dentropy[r] * a.inv_t : 0.0f;
  const float2 st = *reinterpret_cast<const float2*>(a.stats + 2 * r);
  // by the places of the gradient's units; the logits' are the same, or they are taken one by one
  const bool same = (reinterpret_cast<uintptr_t>(x) ^ reinterpret_cast<uintptr_t>(dx)) % 16 == 0;
  const Part<T> p = part_of(static_cast<const T*>(dx), a.vocab, blockIdx.x % ranks, ranks);
  T* const to = dx + p.at;
  const T* const from = x + p.at;
  const int step = blockDim.x, behind = p.head + p.units * per;
  // (every logit is -inf: the sum of none is 0; beside a NaN it is NaN, and the maximum may be -inf too)
  if ((g == 0.0f && h == 0.0f) || (st.x == -INFINITY && st.y == -INFINITY)) {
    for (int u = threadIdx.x; u < p.units; u += step) reinterpret_cast<uint4*>(to + p.head)[u] = make_uint4(0, 0, 0, 0);
    if ((int)threadIdx.x < p.head) st_elem(to, threadIdx.x, 0.0f);
    if ((int)threadIdx.x < p.tail) st_elem(to, behind + threadIdx.x, 0.0f);
    return;
  }
  // in base 2: l = (x - m) c - L, p = 2^l, dx = p (k0 + k1 l) (+ g at the given token)
  const float ent = a.dentropy ? a.entropy[r] : 0.0f, k0 = -fmaf(h, ent, g), k1 = -h * kLn2;
  const f32x2 minus = both(-st.x), c = both(a.inv_t * kLog2e), l0 = both(-st.y * kLog2e), c0 = both(k0), c1 = both(k1);
  const auto slope = [&](f32x2 v) {
    const float2 d = parts(fma2(add2(v, minus), c, l0));
    const float l = max_nan(d.x, kNothing), n = max_nan(d.y, kNothing);
    return mul2(both(exp2_near(l), exp2_near(n)), fma2(c1, both(l, n), c0));
  };
  const int at_id = a.dlogp ? id - p.at : -1;   // the given token's place in the part
  const auto single = [&](int i) {
    const float d = parts(slope(both(ld_elem(from, i)))).x;
    st_elem(to, i, i == at_id ? d + g : d);
  };
  if (same) {
    const uint4* in = reinterpret_cast<const uint4*>(from + p.head);
    uint4* out = reinterpret_cast<uint4*>(to + p.head);
    const int id_unit = at_id >= p.head ? (at_id - p.head) / per : -1, id_in = (at_id - p.head) % per;
    for (int u0 = threadIdx.x; u0 < p.units; u0 += 4 * step) {
      uint4 w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = u0 + i * step < p.units ? in[u0 + i * step] : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int u = u0 + i * step;
        if (u >= p.units) continue;
        f32x2 f[pairs];
        widen(w[i], f);
#pragma unroll
        for (int j = 0; j < pairs; ++j) f[j] = slope(f[j]);
        if (u == id_unit) {
#pragma unroll
          for (int j = 0; j < pairs; ++j) f[j] = add2(f[j], both(id_in == 2 * j ? g : 0.0f, id_in == 2 * j + 1 ? g : 0.0f));
        }
        out[u] = narrow(f);
      }
    }
  } else {
    for (int i = p.head + threadIdx.x; i < behind; i += step) single(i);
  }
  if ((int)threadIdx.x < p.head) single(threadIdx.x);
  if ((int)threadIdx.x < p.tail) single(behind + threadIdx.x);
}

// Many rows: 128 threads each, so that a row's sums are joined by few warps, or one
// warp for the shortest without alternatives (4096 x 1000 bf16: 9.0 us against 11.6; with
// 20 alternatives 26 against 22).  Four blocks to a multiprocessor keep the memory
// busy, fewer are enough for rows of up to 64 KB (450 x 32000 bf16, 20 alternatives: 11.1
// us against 14.1 with 512 threads; 450 x 131072 fp32: 61 against 49).  Few rows: 512
// threads, and as many blocks to a row, up to eight, as fill the multiprocessors while a
// thread still has two units (32 x 32000 bf16, 20 alternatives: four blocks 7.4 us, eight 11.5).
template <typename T>
cudaError_t logp_forward(const LogpArgs& a, int rows, cudaStream_t s) {
  const int sms = device_sms();
  const int units = (int)((long long)a.vocab * (int)sizeof(T) / 16);
  int threads = units < kLogpShort && !a.k ? 32 : 128, ranks = 1;
  if (rows < sms || (rows < 4 * sms && units > 4096)) {
    threads = units < kLogpShort ? 128 : 512;
    while (ranks < kMaxCluster && 2 * ranks * rows <= 2 * sms && units >= 4 * ranks * threads) ranks *= 2;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((long long)rows * ranks));
  cfg.blockDim = dim3(threads);
  cfg.stream = s;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = ranks;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  cudaError_t e;
  if (threads == 32)
    e = cudaLaunchKernelEx(&cfg, logp_kernel<T, false, 32>, a, ranks);
  else if (threads == 128)
    e = a.k ? cudaLaunchKernelEx(&cfg, logp_kernel<T, true, 128>, a, ranks) : cudaLaunchKernelEx(&cfg, logp_kernel<T, false, 128>, a, ranks);
  else
    e = a.k ? cudaLaunchKernelEx(&cfg, logp_kernel<T, true, 512>, a, ranks) : cudaLaunchKernelEx(&cfg, logp_kernel<T, false, 512>, a, ranks);
  return e != cudaSuccess ? e : cudaGetLastError();
}
template <typename T>
cudaError_t logp_backward(const LogpGradArgs& a, int rows, cudaStream_t s) {
  int ranks = 1;
  const int sms = device_sms();
  while (2ll * ranks * rows <= 8 * sms && (long long)a.vocab * (int)sizeof(T) / 16 >= 512ll * ranks) ranks *= 2;
  logp_grad_kernel<T><<<(unsigned)((long long)rows * ranks), 256, 0, s>>>(a, ranks);
  return cudaGetLastError();
}

}  // namespace
}  // namespace mg

using mg::op_fail;

static mg_status check_logits(const char* fn, int dtype, int id_kind, long long rows, int vocab, long long stride,
                              float temperature) {
  if ((dtype != 0 && dtype != 1) || (id_kind != 0 && id_kind != 1))
    return op_fail(MG_ERR_INVALID_ARG, "%s: dtype and id_kind must be 0 or 1", fn);
  if (rows < 0 || rows > 0x7fffffff || vocab < 1 || vocab > mg::kMaxWidth || stride < vocab || stride > (1ll << 31))
    return op_fail(MG_ERR_SHAPE, "%s: rows %lld, vocab %d, row stride %lld", fn, rows, vocab, stride);
  if (!(temperature > 0.0f) || !std::isfinite(temperature) || !std::isfinite(mg::kLog2e * (1.0f / temperature)))
    return op_fail(MG_ERR_INVALID_ARG, "%s: the temperature must be positive and finite, log2(e) over it finite", fn);
  return MG_OK;
}

// Whether the rows of two matrices of one stride and width lie beside one another: between their starts are whole
// strides, and a rest that leaves room for one row and, up to the next stride, for the other.
static bool rows_beside(const void* a, const void* b, int vocab, long long stride, int dtype) {
  const size_t es = dtype ? 2 : 4, line = stride * es, wide = vocab * es;
  const uintptr_t p = reinterpret_cast<uintptr_t>(a), q = reinterpret_cast<uintptr_t>(b);
  const size_t rest = (p < q ? q - p : p - q) % line;
  return rest >= wide && line - rest >= wide;
}

// Bytes from the first element to the last one's end.
static size_t rows_bytes(long long rows, int vocab, long long stride, int dtype) {
  return rows ? ((size_t)(rows - 1) * stride + vocab) * (dtype ? 2 : 4) : 0;
}

extern "C" mg_status mg_token_logprobs(int dtype, const void* logits, long long rows, int vocab, long long row_stride,
                                       int id_kind, const void* ids, float temperature, float* logp, float* stats,
                                       float* entropy, int k, int* top_ids, float* top_logp, mg_stream_t stream) {
  const char* fn = "mg_token_logprobs";
  mg_status st = check_logits(fn, dtype, id_kind, rows, vocab, row_stride, temperature);
  if (st != MG_OK) return st;
  if (k < 0 || k > MG_MAX_TOP || k > vocab)
    return op_fail(MG_ERR_SHAPE, "%s: k = %d of a vocabulary of %d, at most %d", fn, k, vocab, MG_MAX_TOP);
  if (rows && (!logits || !ids != !logp || (k && (!top_ids || !top_logp)) || !(logp || stats || entropy || k)))
    return op_fail(MG_ERR_INVALID_ARG,
                   "%s: logits must be non-NULL, ids with logp, top_ids and top_logp with k, and one output at least", fn);
  const unsigned es = dtype ? 2 : 4;
  st = mg::op_begin(fn, {{logits, es}, {ids, id_kind ? 8u : 4u}, {logp, 4}, {stats, 8}, {entropy, 4}, {k ? top_ids : nullptr, 4},
                         {k ? top_logp : nullptr, 4}});
  if (st != MG_OK) return st;
  const size_t n = (size_t)rows, nk = n * k * 4;
  st = mg::op_disjoint(fn, {{logits, rows_bytes(rows, vocab, row_stride, dtype), false, false}, {ids, n * (id_kind ? 8 : 4), false, false},
                            {logp, n * 4, true, false}, {stats, n * 8, true, false}, {entropy, n * 4, true, false},
                            {top_ids, nk, true, false}, {top_logp, nk, true, false}});
  if (st != MG_OK || !rows) return st;
  mg::LogpArgs a = {logits, row_stride, vocab, ids, id_kind, 1.0f / temperature, logp, stats, entropy, k, top_ids, top_logp};
  return mg::op_end(fn, dtype ? mg::logp_forward<mg::bf16>(a, (int)rows, (cudaStream_t)stream)
                              : mg::logp_forward<float>(a, (int)rows, (cudaStream_t)stream));
}

extern "C" mg_status mg_token_logprobs_backward(int dtype, const void* logits, long long rows, int vocab,
                                                long long row_stride, int id_kind, const void* ids, float temperature,
                                                const float* stats, const float* entropy, const float* dlogp,
                                                const float* dentropy, void* dlogits, long long dlogits_stride,
                                                mg_stream_t stream) {
  const char* fn = "mg_token_logprobs_backward";
  mg_status st = check_logits(fn, dtype, id_kind, rows, vocab, row_stride, temperature);
  if (st == MG_OK) st = check_logits(fn, dtype, id_kind, rows, vocab, dlogits_stride, temperature);
  if (st != MG_OK) return st;
  if (rows && (!logits || !stats || !dlogits || (!dlogp && !dentropy) || (dlogp && !ids) || (dentropy && !entropy)))
    return op_fail(MG_ERR_INVALID_ARG,
                   "%s: logits, stats, dlogits and one of dlogp (with ids) and dentropy (with entropy) must be non-NULL", fn);
  const unsigned es = dtype ? 2 : 4;
  st = mg::op_begin(fn, {{logits, es}, {ids, id_kind ? 8u : 4u}, {stats, 8}, {entropy, 4}, {dlogp, 4}, {dentropy, 4}, {dlogits, es}});
  if (st != MG_OK) return st;
  const size_t n = (size_t)rows;
  const bool beside = row_stride == dlogits_stride && rows_beside(logits, dlogits, vocab, row_stride, dtype);
  st = mg::op_disjoint(fn, {{beside ? nullptr : logits, rows_bytes(rows, vocab, row_stride, dtype), false, false},
                            {ids, n * (id_kind ? 8 : 4), false, false}, {stats, n * 8, false, false},
                            {entropy, n * 4, false, false}, {dlogp, n * 4, false, false}, {dentropy, n * 4, false, false},
                            {dlogits, rows_bytes(rows, vocab, dlogits_stride, dtype), true,
                             logits == dlogits && row_stride == dlogits_stride}});
  if (st != MG_OK || !rows) return st;
  mg::LogpGradArgs a = {logits, row_stride, vocab, ids, id_kind, 1.0f / temperature, stats, entropy, dlogp, dentropy, dlogits,
                        dlogits_stride};
  return mg::op_end(fn, dtype ? mg::logp_backward<mg::bf16>(a, (int)rows, (cudaStream_t)stream)
                              : mg::logp_backward<float>(a, (int)rows, (cudaStream_t)stream));
}

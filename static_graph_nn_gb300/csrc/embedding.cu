// Token embedding: lookup with scaling, and its gradient by sorted tokens.
//
//   forward   out[i] = scale * table[id_i]               (0 for an id outside [0, V))
//   backward  dtable[v] = scale * sum_{i: id_i = v} dout[i]   (dense, fp32)
//
// The forward is a gather: it reads the rows that the ids name and writes n
// rows, nothing else.  A thread moves 16 bytes of one row and has several rows'
// loads in flight.  A few tokens are bound by one launch; many by the chain of
// two loads (an id, then its row) of blocks that end after one round: 16384 bf16
// rows of 2048, about 5800 of them distinct, take 21 us, and their bytes 13.4 at
// the DRAM's rate.
//
// The backward must write all V rows, and sums the rows of dout that share an
// id.  Adding with atomics would need a zeroed table, a read-modify-write of
// every touched row, and would change results from run to run.  Instead:
//
//   1. the positions are sorted by id with a stable counting sort (positions of
//      one id stay ascending).  Up to 65536 ids one cluster of four or eight CTAs
//      sorts them in shared memory, exchanging counts and elements through DSMEM;
//      meanwhile the other CTAs of the launch write the zero rows, each
//      finding the ids of its own range of rows with one scan of the ids, so
//      the sort's latency hides under bandwidth-bound stores;
//   2. the sorted order is cut into equal windows, one thread group each, so
//      that frequent ids cost no more than rare ones.  A group streams its
//      window's rows of dout, eight in flight, and writes a row of the table
//      whenever the id changes.  A sum that crosses windows leaves one partial
//      per window;
//   3. a third launch joins those partials, a block per sum, in a fixed order.
//
// Every row of the table is written once, and the order of every addition is
// fixed by the ids alone: the same bits in every run.  Wide rows are bound by
// DRAM (V d fp32 written, n d read), narrow ones by the three launches in a row.
#include <algorithm>
#include <cstdio>

#include "../../include/mg.h"
#include "common.cuh"
#include "kernels.h"
#include "op_checks.h"

namespace mg {
namespace {

constexpr int kRadixBits = 9;
constexpr int kRadix = 1 << kRadixBits;
constexpr int kSortThreads = 256;
constexpr int kSortItems = 16;                            // per thread
constexpr int kSortTile = kSortThreads * kSortItems;      // 4096 keys per block
constexpr int kWarps = kSortThreads / 32;
constexpr int kSumThreads = 152 * 2 * 256;  // threads that sum: windows of the sorted order times threads a row
constexpr int kSmallThreads = 1024;
constexpr long long kSmallMax = 64 * kSmallThreads;   // ids that a cluster sorts
constexpr int kZeroRange = 65536;   // rows whose presence one block holds as bits

// ---------------------------------------------------------------- forward

template <typename T>
struct Vec16;   // 16 bytes of T as floats
template <>
struct Vec16<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void load(const float* p, float* f) {
    const float4 v = __ldg(reinterpret_cast<const float4*>(p));
    f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
  }
};
template <>
struct Vec16<bf16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ void load(const bf16* p, float* f) {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(p));
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 t = __bfloat1622float2(h[i]);
      f[2 * i] = t.x;
      f[2 * i + 1] = t.y;
    }
  }
};

template <int N>
__device__ __forceinline__ void store_vec(float* p, const float* f) {
#pragma unroll
  for (int q = 0; q < N / 4; ++q)
    reinterpret_cast<float4*>(p)[q] = make_float4(f[4 * q], f[4 * q + 1], f[4 * q + 2], f[4 * q + 3]);
}
template <int N>
__device__ __forceinline__ void store_vec(bf16* p, const float* f) {
  uint32_t w[N / 2];
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t*>(&h);
  }
  if (N == 8) {
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
  }
}

// One thread: column chunk c (C elements) of U rows.  tpr threads per row.
template <typename TT, typename TO, typename TI, bool VEC, int U>
__global__ void __launch_bounds__(256) embed_fwd_kernel(const TT* table, int V, int d, const TI* ids,
                                                        long long n, float scale, TO* out, int tpr) {
  constexpr int C = VEC ? Vec16<TT>::N : 1;
  const int rpb = 256 / tpr;
  const int lane = threadIdx.x % tpr, sub = threadIdx.x / tpr;
  const long long stride = (long long)gridDim.x * rpb;
  for (long long r0 = (long long)blockIdx.x * rpb + sub; r0 < n; r0 += stride * U) {
    long long id[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long r = r0 + u * stride;
      id[u] = r < n ? (long long)ids[r] : -1;
    }
    for (int c = lane * C; c < d; c += tpr * C) {
      float f[U][C];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (id[u] >= 0 && id[u] < V) {
          const TT* p = table + (size_t)id[u] * d + c;
          if (VEC) Vec16<TT>::load(p, f[u]);
          else f[u][0] = ld_elem(p, 0);
        } else {
#pragma unroll
          for (int i = 0; i < C; ++i) f[u][i] = 0.0f;
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const long long r = r0 + u * stride;
        if (r >= n) continue;
        const bool ok = id[u] >= 0 && id[u] < V;   // padding stays +0 under any scale
#pragma unroll
        for (int i = 0; i < C; ++i) f[u][i] = ok ? f[u][i] * scale : 0.0f;
        TO* o = out + (size_t)r * d + c;
        if constexpr (VEC) store_vec<C>(o, f[u]);
        else st_elem(o, 0, f[u][0]);
      }
    }
  }
}

int threads_per_row(int chunks) {
  int t = 1;
  while (t < chunks && t < 256) t *= 2;
  return t;
}

template <typename TT, typename TO, typename TI>
cudaError_t fwd_launch(const void* table, int V, int d, const void* ids, long long n, float scale,
                       void* out, cudaStream_t s) {
  constexpr int C = Vec16<TT>::N;
  const bool vec = d % C == 0;
  const int tpr = threads_per_row(vec ? d / C : d);
  const long long blocks = (n + 256 / tpr - 1) / (256 / tpr);
  // four rows in flight per thread once the rows fill the GPU; below that one
  // row per thread spreads the few rows over more SMs
  const bool deep = blocks >= 4 * 152 * 4;
  long long grid = deep ? (blocks + 3) / 4 : blocks;
  if (grid > 152 * 64) grid = 152 * 64;
  const TT* t = (const TT*)table;
  const TI* id = (const TI*)ids;
  TO* o = (TO*)out;
  const dim3 g((unsigned)grid);
  if (vec && deep) embed_fwd_kernel<TT, TO, TI, true, 4><<<g, 256, 0, s>>>(t, V, d, id, n, scale, o, tpr);
  else if (vec) embed_fwd_kernel<TT, TO, TI, true, 1><<<g, 256, 0, s>>>(t, V, d, id, n, scale, o, tpr);
  else if (deep) embed_fwd_kernel<TT, TO, TI, false, 4><<<g, 256, 0, s>>>(t, V, d, id, n, scale, o, tpr);
  else embed_fwd_kernel<TT, TO, TI, false, 1><<<g, 256, 0, s>>>(t, V, d, id, n, scale, o, tpr);
  return cudaGetLastError();
}

// ---------------------------------------------------------------- sort
// Stable least-significant-digit counting sort of (id, position), 9 bits a
// pass.  Invalid ids sort last under the key V.

template <typename TI>
__device__ __forceinline__ uint32_t key_of(const TI* ids, long long i, int V) {
  const long long id = (long long)ids[i];
  return id >= 0 && id < V ? (uint32_t)id : (uint32_t)V;
}

struct KeysIn {   // first pass: the ids themselves; later passes: the previous output
  const void* ids;
  int id64;
  int V;
  const uint32_t* key;
  const uint32_t* pos;
  __device__ __forceinline__ uint32_t k(uint32_t i) const {
    if (key) return key[i];
    return id64 ? key_of((const long long*)ids, i, V) : key_of((const int*)ids, i, V);
  }
  __device__ __forceinline__ uint32_t p(uint32_t i) const { return pos ? pos[i] : i; }
};

// counts[digit * gridDim.x + block]
__global__ void __launch_bounds__(kSortThreads) sort_count_kernel(KeysIn in, uint32_t n, int shift,
                                                                  uint32_t* counts) {
  __shared__ uint32_t h[kRadix];
  for (int i = threadIdx.x; i < kRadix; i += kSortThreads) h[i] = 0;
  __syncthreads();
  const uint32_t base = blockIdx.x * (uint32_t)kSortTile;
  for (int j = 0; j < kSortItems; ++j) {
    const uint32_t i = base + j * kSortThreads + threadIdx.x;
    if (i < n) atomicAdd(&h[(in.k(i) >> shift) & (kRadix - 1)], 1u);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < kRadix; i += kSortThreads) counts[(size_t)i * gridDim.x + blockIdx.x] = h[i];
}

// exclusive scan of m counts in place, one block
__global__ void __launch_bounds__(1024) sort_scan_kernel(uint32_t* counts, uint32_t m) {
  __shared__ uint32_t wsum[32];
  __shared__ uint32_t carry;
  if (threadIdx.x == 0) carry = 0;
  __syncthreads();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  for (uint32_t b = 0; b < m; b += 4096) {
    const uint32_t i0 = b + threadIdx.x * 4;
    uint32_t v[4], s = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      v[q] = i0 + q < m ? counts[i0 + q] : 0;
      s += v[q];
    }
    uint32_t x = s;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) wsum[w] = x;
    __syncthreads();
    if (w == 0) {
      uint32_t t = wsum[lane];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, t, o);
        if (lane >= o) t += y;
      }
      wsum[lane] = t;
    }
    __syncthreads();
    uint32_t e = carry + (w ? wsum[w - 1] : 0) + x - s;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (i0 + q < m) counts[i0 + q] = e;
      e += v[q];
    }
    __syncthreads();
    if (threadIdx.x == 0) carry += wsum[31];
    __syncthreads();
  }
}

// The lanes with ok and this lane's digit, bit by bit: by __match_any_sync the
// sort of 32768 ids by four CTAs took 58 us, this way 42; a whole gradient of 1000003 ids in
// rows of 32 took 213 us and 208.
__device__ __forceinline__ uint32_t same_digit(bool ok, uint32_t dg, int bits) {
  uint32_t same = __ballot_sync(0xffffffffu, ok);
#pragma unroll
  for (int b = 0; b < kRadixBits; ++b) {
    if (b >= bits) break;
    const uint32_t set = __ballot_sync(0xffffffffu, dg >> b & 1);
    same &= dg >> b & 1 ? set : ~set;
  }
  return same;
}

// Each warp owns kSortItems * 32 consecutive keys; a key's place is its
// digit's base of this block (scanned counts), plus the earlier warps' keys of
// that digit, plus the warp's own earlier ones: stable.
__global__ void __launch_bounds__(kSortThreads) sort_scatter_kernel(KeysIn in, uint32_t n, int shift,
                                                                    const uint32_t* bases,
                                                                    uint32_t* key_out, uint32_t* pos_out) {
  __shared__ uint32_t cnt[kWarps][kRadix];
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  for (int i = threadIdx.x; i < kWarps * kRadix; i += kSortThreads) (&cnt[0][0])[i] = 0;
  __syncthreads();
  const uint32_t base = blockIdx.x * (uint32_t)kSortTile + w * (kSortItems * 32);
  uint32_t k[kSortItems], rank[kSortItems];
#pragma unroll
  for (int j = 0; j < kSortItems; ++j) {
    const uint32_t i = base + j * 32 + lane;
    k[j] = i < n ? in.k(i) : 0xffffffffu;
  }
#pragma unroll
  for (int j = 0; j < kSortItems; ++j) {
    const uint32_t i = base + j * 32 + lane;
    const bool ok = i < n;
    const uint32_t dg = (k[j] >> shift) & (kRadix - 1);
    const uint32_t same = same_digit(ok, dg, kRadixBits);
    const uint32_t before = __popc(same & ((1u << lane) - 1));
    uint32_t c = 0;
    if (ok) c = cnt[w][dg];
    __syncwarp();
    if (ok && before == 0) cnt[w][dg] = c + __popc(same);
    __syncwarp();
    rank[j] = c + before;
  }
  __syncthreads();
  for (int dgt = threadIdx.x; dgt < kRadix; dgt += kSortThreads) {
    uint32_t run = bases[(size_t)dgt * gridDim.x + blockIdx.x];
#pragma unroll
    for (int q = 0; q < kWarps; ++q) {
      const uint32_t c = cnt[q][dgt];
      cnt[q][dgt] = run;
      run += c;
    }
  }
  __syncthreads();
#pragma unroll
  for (int j = 0; j < kSortItems; ++j) {
    const uint32_t i = base + j * 32 + lane;
    if (i >= n) continue;
    const uint32_t o = cnt[w][(k[j] >> shift) & (kRadix - 1)] + rank[j];
    key_out[o] = k[j];
    pos_out[o] = in.p(i);
  }
}

// Segment bounds of every id that occurs, from the sorted keys.
__global__ void __launch_bounds__(256) sort_bounds_kernel(const uint32_t* key, uint32_t n, uint32_t V, uint2* seg) {
  const uint32_t i = blockIdx.x * 256u + threadIdx.x;
  if (i >= n) return;
  const uint32_t k = key[i];
  if (k >= V) return;
  if (i == 0 || key[i - 1] != k) seg[k].x = i;
  if (i + 1 == n || key[i + 1] != k) seg[k].y = i + 1;
}

// Zeros of one row; aligned 16-byte stores between a scalar head and tail.
__device__ __forceinline__ void zero_row(float* row, int d, int lane) {
  const int head = min(d, (int)((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / 4);
  if (lane < head) row[lane] = 0.0f;
  float4* body = reinterpret_cast<float4*>(row + head);
  const int n4 = (d - head) / 4;
  for (int i = lane; i < n4; i += 32) body[i] = make_float4(0.f, 0.f, 0.f, 0.f);
  const int t = head + n4 * 4 + lane;
  if (t < d) row[t] = 0.0f;
}

// Rows that no id names, after a sort that cleared seg: one warp per row.
__global__ void __launch_bounds__(256) zero_rows_kernel(const uint2* seg, uint32_t V, int d, float* dtable) {
  const int lane = threadIdx.x & 31;
  for (uint32_t v = blockIdx.x * 8 + (threadIdx.x >> 5); v < V; v += gridDim.x * 8)
    if (seg[v].y == 0) zero_row(dtable + (size_t)v * d, d, lane);
}

// ---- one launch for up to kSmallMax ids: the first cluster sorts, the others zero
struct SmallArgs {
  KeysIn in;
  uint32_t n, V;
  int d, digit_bits, passes;   // of the sort
  uint32_t* key;
  uint32_t* pos;
  uint2* seg;
  float* dtable;
};

__device__ __forceinline__ uint32_t cluster_addr(const void* p, uint32_t cta) {
  uint32_t a = static_cast<uint32_t>(__cvta_generic_to_shared(p)), out;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(out) : "r"(a), "r"(cta));
  return out;
}
__device__ __forceinline__ uint32_t ld_cluster(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void st_cluster(uint32_t a, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ void cluster_barrier() {
  __syncwarp();
  asm volatile("barrier.cluster.arrive.aligned;\nbarrier.cluster.wait.aligned;" ::: "memory");
}

template <int IPT>
struct SmallSmem {
  uint16_t cnt[32][kRadix];              // per warp and digit; then the exclusive prefix over warps
  uint32_t tot[kRadix];                  // this CTA's digit counts, read by the cluster
  uint32_t base[kRadix];                 // first place of this CTA's keys of a digit
  uint32_t key[kSmallThreads * IPT];     // this CTA's part of the order, written by the cluster
  uint32_t pos[kSmallThreads * IPT];
  uint32_t wsum[32];
};

template <int IPT, int CL>
__global__ void __cluster_dims__(CL, 1, 1) __launch_bounds__(kSmallThreads, 1)
    sort_small_kernel(const SmallArgs A) {
  extern __shared__ __align__(16) uint8_t raw[];
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  dependents_start();
  if (blockIdx.x >= CL) {
    // ---- zero rows of a contiguous range of the table
    uint32_t* bits = reinterpret_cast<uint32_t*>(raw);
    const uint32_t nz = gridDim.x - CL, z = blockIdx.x - CL;
    const uint32_t lo = (uint32_t)((unsigned long long)A.V * z / nz);
    const uint32_t hi = (uint32_t)((unsigned long long)A.V * (z + 1) / nz);
    for (uint32_t r0 = lo; r0 < hi; r0 += kZeroRange) {
      const uint32_t nr = min(hi - r0, (uint32_t)kZeroRange), nw = (nr + 31) / 32;
      for (uint32_t i = tid; i < nw; i += kSmallThreads) bits[i] = 0;
      __syncthreads();
      for (uint32_t i0 = tid; i0 < A.n; i0 += 8 * kSmallThreads) {
        uint32_t k[8];                        // eight loads in flight
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const uint32_t i = i0 + q * kSmallThreads;
          k[q] = i < A.n ? A.in.k(i) - r0 : 0xffffffffu;    // below r0 wraps to a large value
        }
#pragma unroll
        for (int q = 0; q < 8; ++q)
          if (k[q] < nr) atomicOr(&bits[k[q] >> 5], 1u << (k[q] & 31));
      }
      __syncthreads();
      for (uint32_t r = w; r < nr; r += 32)
        if (!(bits[r >> 5] >> (r & 31) & 1)) zero_row(A.dtable + (size_t)(r0 + r) * A.d, A.d, lane);
      __syncthreads();
    }
    return;
  }
  SmallSmem<IPT>& S = *reinterpret_cast<SmallSmem<IPT>*>(raw);
  const uint32_t cta = blockIdx.x;
  constexpr uint32_t kChunk = kSmallThreads * IPT;
  const int bins = 1 << A.digit_bits;
  const uint32_t first = cta * kChunk + w * (32 * IPT) + lane;
  uint32_t k[IPT], p[IPT], rank[IPT];
#pragma unroll
  for (int j = 0; j < IPT; ++j) {
    const uint32_t i = first + j * 32;
    k[j] = i < A.n ? A.in.k(i) : 0;
    p[j] = i;
  }
  for (int pass = 0; pass < A.passes; ++pass) {
    const int shift = pass * A.digit_bits;
    for (int i = lane; i < bins / 2; i += 32) reinterpret_cast<uint32_t*>(S.cnt[w])[i] = 0;
    __syncwarp();
#pragma unroll
    for (int j = 0; j < IPT; ++j) {
      const bool ok = first + j * 32 < A.n;     // the places behind the last id stay behind it
      const uint32_t dg = (k[j] >> shift) & (bins - 1);
      const uint32_t same = same_digit(ok, dg, A.digit_bits);
      const uint32_t before = __popc(same & ((1u << lane) - 1));
      uint32_t c = 0;
      if (ok) c = S.cnt[w][dg];
      __syncwarp();
      if (ok && before == 0) S.cnt[w][dg] = (uint16_t)(c + __popc(same));
      __syncwarp();
      rank[j] = c + before;
    }
    __syncthreads();
    if (tid < bins) {
      uint32_t run = 0;
#pragma unroll 8
      for (int q = 0; q < 32; ++q) {
        const uint32_t c = S.cnt[q][tid];
        S.cnt[q][tid] = (uint16_t)run;
        run += c;
      }
      S.tot[tid] = run;
    }
    cluster_barrier();                          // every CTA's counts are there
    uint32_t all = 0, before = 0;
    if (tid < bins) {
#pragma unroll
      for (uint32_t c = 0; c < CL; ++c) {
        const uint32_t t = ld_cluster(cluster_addr(&S.tot[tid], c));
        if (c < cta) before += t;
        all += t;
      }
    }
    uint32_t x = all;                           // exclusive scan over the digits
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) S.wsum[w] = x;
    __syncthreads();
    if (w == 0) {
      uint32_t t = S.wsum[lane];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, t, o);
        if (lane >= o) t += y;
      }
      S.wsum[lane] = t;
    }
    __syncthreads();
    if (tid < bins) S.base[tid] = (w ? S.wsum[w - 1] : 0) + x - all + before;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < IPT; ++j) {
      if (first + j * 32 >= A.n) continue;
      const uint32_t dg = (k[j] >> shift) & (bins - 1);
      const uint32_t o = S.base[dg] + S.cnt[w][dg] + rank[j];
      const uint32_t c = o / kChunk, at = o % kChunk;
      st_cluster(cluster_addr(&S.key[at], c), k[j]);
      st_cluster(cluster_addr(&S.pos[at], c), p[j]);
    }
    cluster_barrier();                          // the order of this pass is complete
#pragma unroll
    for (int j = 0; j < IPT; ++j) {
      const uint32_t i = w * (32 * IPT) + lane + j * 32;
      k[j] = S.key[i];
      p[j] = S.pos[i];
    }
  }
#pragma unroll
  for (int j = 0; j < IPT; ++j) {
    const uint32_t i = first + j * 32;
    if (i >= A.n) continue;
    A.key[i] = k[j];
    A.pos[i] = p[j];
    if (k[j] >= A.V) continue;
    const uint32_t at = i % kChunk;
    const uint32_t prev = i == 0 ? 0xffffffffu
                                 : at ? S.key[at - 1] : ld_cluster(cluster_addr(&S.key[kChunk - 1], cta - 1));
    const uint32_t next = i + 1 == A.n ? 0xffffffffu
                                       : at + 1 < kChunk ? S.key[at + 1] : ld_cluster(cluster_addr(&S.key[0], cta + 1));
    if (prev != k[j]) A.seg[k[j]].x = i;
    if (next != k[j]) A.seg[k[j]].y = i + 1;
  }
  cluster_barrier();                            // no CTA leaves while another reads its keys
}

// ---------------------------------------------------------------- sums
struct SumArgs {
  const void* dout;
  float* dtable;
  const uint2* seg;
  const uint32_t* key;
  const uint32_t* pos;
  float* part;            // [windows][2][d]
  uint32_t n, V;
  int d;
  float scale;
  uint32_t window, n_windows;
  int col_tiles, tpr;
  int v32;   // rows of dtable and part are 32-byte aligned
};

// One thread's columns of a row.  VEC: NCH chunks of 16 bytes, tpr chunks apart
// (16 columns), each copied to a slot of shared memory that only this thread
// reads (cp.async, no barrier); fp32 rows of any width: 8 columns, tpr apart, the
// same way in 4-byte copies; bf16 rows of odd width: 4 columns through
// registers.  Keys, addresses and comparisons are paid once per row and thread,
// and eight columns a thread spent most of the kernel on them: 16384 bf16 rows
// of 2048 took 41 us with 8 columns a thread, 33 with 16, and 24 with 32-byte
// stores (two 16-byte ones write each sector in halves).  Rows are fetched in
// batches of kBatch, two batches in flight.
constexpr int kBatch = 4;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

template <typename T, bool VEC>
struct Fetch {   // VEC
  static constexpr int E = 16 / sizeof(T), NCH = 16 / E, C = 16;
  static constexpr int SMEM = 2 * kBatch * NCH * 256 * 16;
  __device__ __forceinline__ void start(uint4* ring, int slot, const T* row, int lane, int d, int tpr) {
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int c = (lane + i * tpr) * E;
      if (c < d)
        cp_async16(static_cast<uint32_t>(__cvta_generic_to_shared(ring + (slot * NCH + i) * 256 + threadIdx.x)),
                   row + c);
    }
  }
  // columns beyond d add what their slot holds; they are not stored
  __device__ __forceinline__ void add(const uint4* ring, int slot, float* acc) const {
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const uint4 u = ring[(slot * NCH + i) * 256 + threadIdx.x];
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if (E == 8) {
          acc[i * 8 + 2 * q] += __uint_as_float(w[q] << 16);
          acc[i * 8 + 2 * q + 1] += __uint_as_float(w[q] & 0xffff0000u);
        } else {
          acc[i * 4 + q] += __uint_as_float(w[q]);
        }
      }
    }
  }
  static __device__ __forceinline__ void put(float* row, int lane, int d, int tpr, const float* f, float scale,
                                             int v32) {
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
      const int c = (lane + i * tpr) * E;
      if (c < d) {
        float g[E];
#pragma unroll
        for (int q = 0; q < E; ++q) g[q] = f[i * E + q] * scale;
        // 16-byte stores 32 bytes apart would be two half-written sectors a lane
        if (E == 8 && v32) st8f32(row + c, g);
        else store_vec<E>(row + c, g);
      }
    }
  }
};
template <>
struct Fetch<float, false> {   // 4-byte copies, 8 columns
  static constexpr int C = 8, SMEM = 2 * kBatch * C * 256 * 4;
  __device__ __forceinline__ void start(uint4* ring, int slot, const float* row, int lane, int d, int tpr) {
    const uint32_t dst = static_cast<uint32_t>(__cvta_generic_to_shared(ring)) + (slot * C * 256 + threadIdx.x) * 4;
#pragma unroll
    for (int i = 0; i < C; ++i)
      if (lane + i * tpr < d)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst + i * 1024), "l"(row + lane + i * tpr)
                     : "memory");
  }
  __device__ __forceinline__ void add(const uint4* ring, int slot, float* acc) const {
    const float* f = reinterpret_cast<const float*>(ring) + slot * C * 256 + threadIdx.x;
#pragma unroll
    for (int i = 0; i < C; ++i) acc[i] += f[i * 256];
  }
  static __device__ __forceinline__ void put(float* row, int lane, int d, int tpr, const float* f, float scale, int) {
#pragma unroll
    for (int i = 0; i < C; ++i)
      if (lane + i * tpr < d) row[lane + i * tpr] = f[i] * scale;
  }
};
template <>
struct Fetch<bf16, false> {
  static constexpr int C = 4, SMEM = 0;
  float f[2 * kBatch][C];
  __device__ __forceinline__ void start(uint4*, int slot, const bf16* row, int lane, int d, int tpr) {
#pragma unroll
    for (int i = 0; i < C; ++i) f[slot][i] = lane + i * tpr < d ? ld_elem(row, lane + i * tpr) : 0.0f;
  }
  __device__ __forceinline__ void add(const uint4*, int slot, float* acc) const {
#pragma unroll
    for (int i = 0; i < C; ++i) acc[i] += f[slot][i];
  }
  static __device__ __forceinline__ void put(float* row, int lane, int d, int tpr, const float* f, float scale, int) {
#pragma unroll
    for (int i = 0; i < C; ++i)
      if (lane + i * tpr < d) row[lane + i * tpr] = f[i] * scale;
  }
};

template <typename T, bool VEC>
__global__ void __launch_bounds__(256, 2) embed_sum_kernel(const SumArgs A) {
  using L = Fetch<T, VEC>;
  constexpr int C = L::C, B = kBatch;
  extern __shared__ __align__(16) uint4 ring[];
  const int lane = threadIdx.x % A.tpr, sub = threadIdx.x / A.tpr, rpb = 256 / A.tpr;
  const uint32_t items = A.n_windows * (uint32_t)A.col_tiles;
  dependency_wait();
  for (uint32_t base = blockIdx.x * rpb; base < items; base += gridDim.x * rpb) {
    const uint32_t it = base + sub;
    const uint32_t win = it / A.col_tiles;
    const int tile = it % A.col_tiles;
    // this tile's columns: pointers moved by c0, width d
    const int c0 = tile * A.tpr * C, d = A.d - c0;
    const T* dout = static_cast<const T*>(A.dout) + c0;
    float* dtable = A.dtable + c0;
    float* part = A.part + (size_t)win * 2 * A.d + c0;
    uint32_t kfirst = A.V, klast = A.V;
    uint2 sfirst = {0, 0}, slast = {0, 0};
    bool left = false, right = false;
    if (it < items) {
      uint32_t wb = win * A.window, we = min(A.n, wb + A.window);
      kfirst = A.key[wb];
      klast = A.key[we - 1];
      const uint32_t kprev = wb > 0 ? A.key[wb - 1] : 0xffffffffu, knext = we < A.n ? A.key[we] : 0xffffffffu;
      left = kprev == kfirst && kfirst < A.V;       // the first sum began in an earlier window
      right = knext == klast && klast < A.V;        // the last one goes on in a later one
      if (left) sfirst = A.seg[kfirst];
      if (right) slast = A.seg[klast];
      // a segment of at most a window's length belongs to the window it begins
      // in; only longer ones are cut
      if (right && slast.y - slast.x <= A.window) {
        right = false;
        if (slast.x >= wb) we = slast.y;
      }
      if (left && sfirst.y - sfirst.x <= A.window) {
        left = false;
        wb = min(sfirst.y, we);
      }
      uint32_t cur = A.V;
      bool from_left = left;
      float acc[C];
      L rows;
      uint32_t kk[2][B];
      // keys and fetches of the batch at j (a multiple of 4) into half h
      auto fetch = [&](uint32_t j, int h) {
        if (j < we) {
          const uint4 k4 = *reinterpret_cast<const uint4*>(A.key + j);
          const uint4 p4 = *reinterpret_cast<const uint4*>(A.pos + j);
          const uint32_t kq[4] = {k4.x, k4.y, k4.z, k4.w}, pq[4] = {p4.x, p4.y, p4.z, p4.w};
#pragma unroll
          for (int q = 0; q < B; ++q) {
            kk[h][q] = j + q >= wb && j + q < we ? kq[q] : A.V;
            if (kk[h][q] < A.V) rows.start(ring, h * B + q, dout + (size_t)pq[q] * A.d, lane, d, A.tpr);
          }
        }
        if (L::SMEM) asm volatile("cp.async.commit_group;" ::: "memory");
      };
      auto flush = [&] {
        if (cur < A.V) {
          if (from_left) L::put(part, lane, d, A.tpr, acc, 1.0f, A.v32);
          else L::put(dtable + (size_t)cur * A.d, lane, d, A.tpr, acc, A.scale, A.v32);
          from_left = false;
        }
      };
      const uint32_t j0 = wb & ~3u;
      fetch(j0, 0);
      fetch(j0 + B, 1);
      for (uint32_t j = j0; j < we; j += 2 * B) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (j + h * B >= we) break;
          if (L::SMEM) asm volatile("cp.async.wait_group 1;" ::: "memory");   // all but the youngest batch
#pragma unroll
          for (int q = 0; q < B; ++q) {
            const uint32_t k = kk[h][q];
            if (k >= A.V) continue;      // outside the window, or padding (sorted behind every id)
            if (k != cur) {
              flush();
#pragma unroll
              for (int i = 0; i < C; ++i) acc[i] = 0.0f;
              cur = k;
            }
            rows.add(ring, h * B + q, acc);
          }
          fetch(j + (2 + h) * B, h);
        }
      }
      if (L::SMEM) asm volatile("cp.async.wait_group 0;" ::: "memory");
      if (cur < A.V) {
        if (right && !from_left) L::put(part + A.d, lane, d, A.tpr, acc, 1.0f, A.v32);
        else flush();
      }
    }
  }
}

// The sums that cross windows, from their partials: slot 1 of the window in which
// a segment begins, slot 0 of the later ones.  An id with a tenth of all
// positions has a tenth of the windows' partials, so a block gives its 256
// threads to one segment and 128 threads' columns at a time: each group of
// threads adds a run of consecutive windows, and the runs are added in order.
// (Joined by the last group to arrive in the kernel above, one by one, half of
// 16384 positions under one id, 1024 columns, took 141 us for the whole
// gradient, this way 60; of 1000003 in rows of 32, 2834 us and 244; frequencies
// as in text, 16384 rows of 2048, 66 us and 69.)
constexpr int kJoinCols = 128;  // threads a row at most
constexpr int kJoinBlocks = 8;  // blocks per SM at most

// Block (x, y): the windows x, x + gridDim.x, ...; the column tiles y, y + gridDim.y, ...
template <int VEC>
__global__ void __launch_bounds__(256) embed_join_kernel(const SumArgs A) {
  constexpr int U = 8;                   // partials in flight a thread
  __shared__ uint4 found[256];           // first window, windows, id
  __shared__ uint32_t n_found;
  __shared__ float red[256][VEC];
  const int tid = threadIdx.x, lane = tid % A.tpr, grp = tid / A.tpr, groups = 256 / A.tpr;
  dependency_wait();
  for (uint32_t base = blockIdx.x; base < A.n_windows; base += 256 * gridDim.x) {
    if (tid == 0) n_found = 0;
    __syncthreads();
    const uint32_t win = base + tid * gridDim.x, we = (win + 1) * A.window;
    if (win < A.n_windows && we < A.n) {
      const uint32_t k = A.key[we - 1], next = A.key[we];
      if (k < A.V && next == k) {
        const uint2 s = A.seg[k];
        if (s.y - s.x > A.window && s.x >= win * A.window)
          found[atomicAdd(&n_found, 1u)] = make_uint4(win, (s.y - 1) / A.window - win + 1, k, 0);
      }
    }
    __syncthreads();
    const uint32_t n = n_found;
    for (uint32_t j = 0; j < n; ++j) {
      const uint32_t w0 = found[j].x, count = found[j].y;
      const uint32_t run = (count + groups - 1) / groups, lo = grp * run, hi = min(count, lo + run);
      for (int tile = blockIdx.y; tile < A.col_tiles; tile += gridDim.y) {
        const int c = (tile * A.tpr + lane) * VEC;
        float acc[VEC];
#pragma unroll
        for (int i = 0; i < VEC; ++i) acc[i] = 0.0f;
        if (c < A.d) {
          const float* part = A.part + (size_t)w0 * 2 * A.d + c;
#pragma unroll 1
          for (uint32_t q = lo; q < hi; q += U) {
            float f[U][VEC];
#pragma unroll
            for (int u = 0; u < U; ++u) {
              if (q + u >= hi) continue;
              const float* p = part + ((size_t)(q + u) * 2 + (q + u == 0)) * A.d;
              if constexpr (VEC == 4) {
                const float4 v = __ldcg(reinterpret_cast<const float4*>(p));
                f[u][0] = v.x; f[u][1] = v.y; f[u][2] = v.z; f[u][3] = v.w;
              } else {
                f[u][0] = __ldcg(p);
              }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
              if (q + u >= hi) continue;
#pragma unroll
              for (int i = 0; i < VEC; ++i) acc[i] += f[u][i];
            }
          }
        }
#pragma unroll
        for (int i = 0; i < VEC; ++i) red[tid][i] = acc[i];
        __syncthreads();
        if (grp == 0 && c < A.d) {
          for (int q = 1; q < groups && q * run < count; ++q)
#pragma unroll
            for (int i = 0; i < VEC; ++i) acc[i] += red[q * A.tpr + lane][i];
#pragma unroll
          for (int i = 0; i < VEC; ++i) acc[i] *= A.scale;
          float* o = A.dtable + (size_t)found[j].z * A.d + c;
          if constexpr (VEC == 4) store_vec<4>(o, acc);
          else *o = acc[0];
        }
        __syncthreads();
      }
    }
    __syncthreads();     // the list has been read
  }
}

// ---------------------------------------------------------------- workspace
struct Ws {
  size_t key[2], pos[2], seg, counts, part, bytes;
  uint32_t window, n_windows, sort_blocks;
  int passes, digit_bits;
};

Ws ws_layout(long long n, int V, int d) {
  Ws w = {};
  // as many windows (of 8 entries at least) as give kSumThreads threads at 16
  // columns each: 608 for rows of 2048, 9728 for rows of 128 (two blocks per SM; of
  // fp32 rows in multiples of 8, which hold 128 KB of copies a block, one fits, and
  // they run in two waves).  Multiples of 4: a
  // window's keys are read four at a time
  const long long windows = kSumThreads / threads_per_row((d + 15) / 16);
  const long long win = ((n + windows - 1) / windows + 3) / 4 * 4;
  w.window = (uint32_t)(win > 8 ? win : 8);
  w.n_windows = (uint32_t)((n + w.window - 1) / w.window);
  w.sort_blocks = (uint32_t)((n + kSortTile - 1) / kSortTile);
  int key_bits = 1;
  while (((long long)V >> key_bits) != 0) ++key_bits;     // keys are 0 .. V
  w.passes = (key_bits + kRadixBits - 1) / kRadixBits;
  w.digit_bits = (key_bits + w.passes - 1) / w.passes;
  if (w.digit_bits < 5) w.digit_bits = 5;
  size_t top = 0;
  auto take = [&](size_t bytes) {
    const size_t o = top;
    top += (bytes + 255) / 256 * 256;
    return o;
  };
  for (int i = 0; i < 2; ++i) {
    w.key[i] = take((size_t)n * 4);
    w.pos[i] = take((size_t)n * 4);
  }
  w.seg = take((size_t)V * 8);
  w.counts = take((size_t)kRadix * w.sort_blocks * 4);
  w.part = take((size_t)std::min(windows, (n + 7) / 8) * 2 * d * 4);   // at most, so that no smaller n needs more
  w.bytes = top;
  return w;
}

}  // namespace

size_t embedding_ws_bytes(long long n, int V, int d) { return ws_layout(n, V, d).bytes; }

int embedding_bwd_launches(long long n, int V, int d) {
  if (n == 0) return 1;
  const Ws w = ws_layout(n, V, d);
  return (n <= kSmallMax ? 1 : 3 * w.passes + 2) + (w.n_windows > 1 ? 2 : 1);
}

cudaError_t embedding_fwd(DType tt, const void* table, int V, int d, int id64, const void* ids, long long n,
                          float scale, DType ot, void* out, cudaStream_t s) {
  if (n == 0) return cudaSuccess;
#define MG_EMBED_FWD(TT, TO)                                                                  \
  return id64 ? fwd_launch<TT, TO, long long>(table, V, d, ids, n, scale, out, s)             \
              : fwd_launch<TT, TO, int>(table, V, d, ids, n, scale, out, s)
  if (tt == DT_F32 && ot == DT_F32) { MG_EMBED_FWD(float, float); }
  if (tt == DT_F32) { MG_EMBED_FWD(float, bf16); }
  if (ot == DT_F32) { MG_EMBED_FWD(bf16, float); }
  MG_EMBED_FWD(bf16, bf16);
#undef MG_EMBED_FWD
}

template <int IPT, int CL>
static cudaError_t sort_small(const SmallArgs& A, cudaStream_t s) {
  constexpr size_t smem = sizeof(SmallSmem<IPT>) > kZeroRange / 8 ? sizeof(SmallSmem<IPT>) : kZeroRange / 8;
  const cudaError_t attr =    // of this device's context: set in every call
      cudaFuncSetAttribute(sort_small_kernel<IPT, CL>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (attr != cudaSuccess) return attr;
  // clusters that run at once (a cluster's CTAs share a GPC, so some SMs may
  // stay out): a later one would start when the first zeroing ones end
  static const int slots = [&] {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(CL * (device_sms() / CL));
    cfg.blockDim = dim3(kSmallThreads);
    cfg.dynamicSmemBytes = smem;
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = CL;
    at.val.clusterDim.y = at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    int c = 0;
    if (cudaOccupancyMaxActiveClusters(&c, sort_small_kernel<IPT, CL>, &cfg) != cudaSuccess || c < 2) {
      cudaGetLastError();
      c = 2;
    }
    return c;
  }();
  // a block's rows are worth its scan of the ids only if they are many
  const long long most = slots - 1, rows = (long long)A.V * A.d / (CL * 65536);
  const unsigned grid = CL + CL * (unsigned)(rows < 1 ? 1 : rows < most ? rows : most);
  sort_small_kernel<IPT, CL><<<grid, kSmallThreads, smem, s>>>(A);
  return cudaGetLastError();
}

cudaError_t embedding_bwd_sort(int id64, const void* ids, long long n, int V, int d, float* dtable, void* workspace,
                               cudaStream_t s) {
  const Ws w = ws_layout(n, V, d);
  char* base = static_cast<char*>(workspace);
  auto u32 = [&](size_t off) { return reinterpret_cast<uint32_t*>(base + off); };
  uint2* seg = reinterpret_cast<uint2*>(base + w.seg);
  KeysIn in{ids, id64, V, nullptr, nullptr};
  if (n <= kSmallMax) {
    SmallArgs A{in, (uint32_t)n, (uint32_t)V, d, w.digit_bits, w.passes, u32(w.key[0]), u32(w.pos[0]), seg,
                dtable};
    // Eight CTAs sort faster than four, but fewer clusters of eight run at once (15
    // of 19: 112 CTAs write the zero rows instead of 140), so up to 16384 ids four
    // sort where the zeros take longer than the sort.  us, by eight and by four:
    // 32768 ids x 2048, vocabulary 32000, 89 and 117; x 64, 37 and 71; 16384 ids x
    // 2048, 73 and 70; x 768, 36 and 43; 5000 ids x 768, 33 and 31; x 256, 23 and 25.
    if (n > 16 * kSmallThreads || (n > 4 * kSmallThreads && (long long)V * d <= 2048 * n)) {
      if (n <= 8 * kSmallThreads) return sort_small<1, 8>(A, s);
      if (n <= 16 * kSmallThreads) return sort_small<2, 8>(A, s);
      if (n <= 32 * kSmallThreads) return sort_small<4, 8>(A, s);
      return sort_small<8, 8>(A, s);
    }
    if (n <= 4 * kSmallThreads) return sort_small<1, 4>(A, s);
    if (n <= 8 * kSmallThreads) return sort_small<2, 4>(A, s);
    return sort_small<4, 4>(A, s);
  }
  cudaError_t e = cudaMemsetAsync(seg, 0, (size_t)V * sizeof(uint2), s);
  if (e != cudaSuccess) return e;
  for (int p = 0; p < w.passes; ++p) {
    const int shift = p * kRadixBits;
    const int dst = (w.passes - 1 - p) & 1;   // the last pass writes buffer 0
    sort_count_kernel<<<w.sort_blocks, kSortThreads, 0, s>>>(in, (uint32_t)n, shift, u32(w.counts));
    sort_scan_kernel<<<1, 1024, 0, s>>>(u32(w.counts), (uint32_t)kRadix * w.sort_blocks);
    sort_scatter_kernel<<<w.sort_blocks, kSortThreads, 0, s>>>(in, (uint32_t)n, shift, u32(w.counts),
                                                               u32(w.key[dst]), u32(w.pos[dst]));
    in.key = u32(w.key[dst]);
    in.pos = u32(w.pos[dst]);
  }
  sort_bounds_kernel<<<(unsigned)((n + 255) / 256), 256, 0, s>>>(u32(w.key[0]), (uint32_t)n, (uint32_t)V, seg);
  const long long zblocks = ((long long)V + 7) / 8;
  zero_rows_kernel<<<(unsigned)(zblocks < 152 * 8 ? zblocks : 152 * 8), 256, 0, s>>>(seg, (uint32_t)V, d, dtable);
  return cudaGetLastError();
}

template <typename T, bool VEC>
static cudaError_t sum_launch(const SumArgs& A, unsigned grid, cudaStream_t s) {
  constexpr int smem = Fetch<T, VEC>::SMEM;
  const cudaError_t attr =
      cudaFuncSetAttribute(embed_sum_kernel<T, VEC>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (attr != cudaSuccess) return attr;
  return launch_dependent(embed_sum_kernel<T, VEC>, grid, 256, smem, s, A);
}

cudaError_t embedding_bwd_sum(DType t, const void* dout, long long n, int V, int d, float scale, float* dtable,
                              void* workspace, cudaStream_t s) {
  if (n == 0) return cudaSuccess;
  const Ws w = ws_layout(n, V, d);
  char* base = static_cast<char*>(workspace);
  SumArgs A;
  A.dout = dout;
  A.dtable = dtable;
  A.seg = reinterpret_cast<uint2*>(base + w.seg);
  A.key = reinterpret_cast<uint32_t*>(base + w.key[0]);
  A.pos = reinterpret_cast<uint32_t*>(base + w.pos[0]);
  A.part = reinterpret_cast<float*>(base + w.part);
  A.n = (uint32_t)n;
  A.V = (uint32_t)V;
  A.d = d;
  A.scale = scale;
  A.window = w.window;
  A.n_windows = w.n_windows;
  // columns a thread: see Fetch; at most 256 threads (a block) a row
  const int per = d % 8 == 0 ? 16 : t == DT_F32 ? 8 : 4;
  A.tpr = threads_per_row((d + per - 1) / per);
  A.col_tiles = (d + A.tpr * per - 1) / (A.tpr * per);
  A.v32 = (reinterpret_cast<uintptr_t>(dtable) & 31) == 0 && (reinterpret_cast<uintptr_t>(A.part) & 31) == 0;
  const int rpb = 256 / A.tpr;
  const long long blocks = ((long long)w.n_windows * A.col_tiles + rpb - 1) / rpb;
  const unsigned grid = (unsigned)(blocks < 152 * 16 ? blocks : 152 * 16);
  const bool vec = d % 8 == 0;
  cudaError_t e;
  if (t == DT_F32) e = vec ? sum_launch<float, true>(A, grid, s) : sum_launch<float, false>(A, grid, s);
  else e = vec ? sum_launch<bf16, true>(A, grid, s) : sum_launch<bf16, false>(A, grid, s);
  if (e != cudaSuccess || w.n_windows == 1) return e;
  const int cols = d % 4 == 0 ? d / 4 : d;
  A.tpr = std::min(threads_per_row(cols), kJoinCols);
  A.col_tiles = (cols + A.tpr - 1) / A.tpr;
  const unsigned ty = (unsigned)std::min(A.col_tiles, 152);
  const dim3 join_grid(std::min(w.n_windows, std::max(1u, 152 * kJoinBlocks / ty)), ty);
  return d % 4 == 0 ? launch_dependent(embed_join_kernel<4>, join_grid, 256, 0, s, A)
                    : launch_dependent(embed_join_kernel<1>, join_grid, 256, 0, s, A);
}

}  // namespace mg

// ============================================================================
namespace {

using mg::op_fail;

constexpr long long kMaxIds = 0x7fffff00ll;   // positions and segment bounds are 32-bit

mg_status check_embedding(const char* fn, int dtype, int id_kind, long long n, int vocab, int dim, float scale) {
  if ((dtype != 0 && dtype != 1) || (id_kind != 0 && id_kind != 1))
    return op_fail(MG_ERR_INVALID_ARG, "%s: dtypes and id_kind must be 0 or 1", fn);
  if (vocab < 1 || vocab == 0x7fffffff || dim < 1 || dim > mg::kMaxWidth)
    return op_fail(MG_ERR_SHAPE, "%s: vocab and dim must be positive, dim at most 2^30 (got %d, %d)", fn, vocab, dim);
  if (n < 0 || n > kMaxIds)
    return op_fail(MG_ERR_SHAPE, "%s: n must be in [0, %lld] (got %lld)", fn, kMaxIds, n);
  if (!(scale - scale == 0.0f)) return op_fail(MG_ERR_INVALID_ARG, "%s: scale is not finite", fn);
  return MG_OK;
}

}  // namespace

extern "C" size_t mg_embedding_workspace_bytes(long long n, int vocab, int dim) {
  if (n < 0 || n > kMaxIds || vocab < 1 || vocab == 0x7fffffff || dim < 1 || dim > mg::kMaxWidth) return 0;
  return mg::embedding_ws_bytes(n, vocab, dim);
}

extern "C" mg_status mg_embedding_forward(int table_dtype, const void* table, int vocab, int dim, int id_kind,
                                          const void* ids, long long n, float scale, int out_dtype, void* out,
                                          mg_stream_t stream) {
  const char* fn = "mg_embedding_forward";
  mg_status st = check_embedding(fn, table_dtype, id_kind, n, vocab, dim, scale);
  if (st != MG_OK) return st;
  if (out_dtype != 0 && out_dtype != 1) return op_fail(MG_ERR_INVALID_ARG, "%s: out_dtype must be 0 or 1", fn);
  if (!table || (n && (!ids || !out)))
    return op_fail(MG_ERR_INVALID_ARG, "%s: table, ids and out must be non-NULL", fn);
  if ((st = mg::op_begin(fn, {{table, 16}, {ids, id_kind ? 8u : 4u}, {out, 16}})) != MG_OK) return st;
  return mg::op_end(fn, mg::embedding_fwd((mg::DType)table_dtype, table, vocab, dim, id_kind, ids, n, scale,
                                          (mg::DType)out_dtype, out, (cudaStream_t)stream));
}

extern "C" mg_status mg_embedding_backward(int dtype, const void* dout, int vocab, int dim, int id_kind,
                                           const void* ids, long long n, float scale, float* dtable,
                                           void* workspace, size_t workspace_bytes, mg_stream_t stream) {
  const char* fn = "mg_embedding_backward";
  mg_status st = check_embedding(fn, dtype, id_kind, n, vocab, dim, scale);
  if (st != MG_OK) return st;
  if (!dtable || !workspace || (n && (!ids || !dout)))
    return op_fail(MG_ERR_INVALID_ARG, "%s: dout, ids, dtable and workspace must be non-NULL", fn);
  const size_t need = mg::embedding_ws_bytes(n, vocab, dim);
  if (workspace_bytes < need)
    return op_fail(MG_ERR_INVALID_ARG, "%s: the workspace needs %zu bytes, %zu given", fn, need, workspace_bytes);
  if ((st = mg::op_begin(fn, {{dout, 16}, {ids, id_kind ? 8u : 4u}, {dtable, 16}, {workspace, 16}})) != MG_OK) return st;
  cudaError_t e = mg::embedding_bwd_sort(id_kind, ids, n, vocab, dim, dtable, workspace, (cudaStream_t)stream);
  if (e == cudaSuccess)
    e = mg::embedding_bwd_sum((mg::DType)dtype, dout, n, vocab, dim, scale, dtable, workspace,
                              (cudaStream_t)stream);
  return mg::op_end(fn, e);
}

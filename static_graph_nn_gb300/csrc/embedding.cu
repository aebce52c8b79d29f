// Token embedding: lookup with scaling, and its gradient by sorted tokens.
//
//   forward   out[i] = scale * table[id_i]               (0 for an id outside [0, V))
//   backward  dtable[v] = scale * sum_{i: id_i = v} dout[i]   (dense, fp32)
//
// The forward is a gather: it reads n rows and writes n rows, nothing else, so
// it is bound by DRAM (and, for a few tokens, by one launch).  A thread moves
// 16 bytes of one row and has several rows' loads in flight.
//
// The backward must write all V rows, and sums the rows of dout that share an
// id.  Adding with atomics would need a zeroed table, a read-modify-write of
// every touched row, and would change results from run to run.  Instead the
// positions are sorted by id with a stable counting sort (positions of one id
// stay ascending), which leaves each id's positions as one segment; then every
// row of the table is written exactly once: zeros where the segment is empty,
// else the fp32 sum in ascending position order.  Text has a few very frequent
// ids; a segment longer than kHot entries is summed by many blocks, each over
// one fixed window of the sorted order, and the last block to finish adds the
// windows' partials in order.  The order of every addition is fixed by the ids
// alone, so the result is the same in every run.
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
constexpr int kWindowMin = 64;      // sorted entries per window of a hot segment
constexpr int kMaxWindows = 2048;   // windows of any call: bounds a hot row's partials

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
    const uint32_t dg = ok ? (k[j] >> shift) & (kRadix - 1) : kRadix + lane;   // unique when absent
    const uint32_t same = __match_any_sync(0xffffffffu, dg);
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

// start[v] = first sorted entry with key >= v, for v in [0, V]; also clears the
// hot rows' arrival counters.  An entry fills the rows between its
// predecessor's key and its own; long runs of absent ids are filled by the
// whole block.
__global__ void __launch_bounds__(256) sort_bounds_kernel(const uint32_t* key, uint32_t n, uint32_t V,
                                                          uint32_t* start, uint32_t* arrivals,
                                                          uint32_t n_arrivals) {
  __shared__ uint32_t big_lo[256], big_hi[256], big_at[256];
  __shared__ int nbig;
  const uint32_t gtid = blockIdx.x * 256u + threadIdx.x;
  for (uint32_t a = gtid; a < n_arrivals; a += gridDim.x * 256u) arrivals[a] = 0;
  if (threadIdx.x == 0) nbig = 0;
  __syncthreads();
  const uint32_t i = gtid;
  if (i <= n) {
    const uint32_t lo = i == 0 ? 0 : key[i - 1] + 1;      // first row not yet filled
    const uint32_t hi = i == n ? V : key[i];              // last row this entry fills
    if (lo <= hi && hi - lo < 8) {
      for (uint32_t v = lo; v <= hi && v <= V; ++v) start[v] = i;
    } else if (lo <= hi) {
      const int b = atomicAdd(&nbig, 1);
      big_lo[b] = lo;
      big_hi[b] = hi;
      big_at[b] = i;
    }
  }
  __syncthreads();
  for (int b = 0; b < nbig; ++b)
    for (uint32_t v = big_lo[b] + threadIdx.x; v <= big_hi[b]; v += 256) start[v] = big_at[b];
}

// ---------------------------------------------------------------- sums
struct SumArgs {
  const void* dout;
  float* dtable;
  const uint32_t* start;
  const uint32_t* key;
  const uint32_t* pos;
  float* part;            // [windows][2][d]
  uint32_t* arrivals;     // [windows][column tiles]
  uint32_t n, V;
  int d;
  float scale;
  uint32_t window, n_windows;
  int col_tiles, tpr;
  int hot_blocks;         // leading blocks: one (window, column tile) each
};

// Column layout of one thread: VEC: 8 consecutive columns; else 4 columns, tpr apart.
template <typename T, bool VEC>
struct Cols {
  static constexpr int C = VEC ? 8 : 4;
  static __device__ __forceinline__ int first(int tile, int lane, int tpr) {
    return tile * tpr * C + (VEC ? lane * C : lane);
  }
  static __device__ __forceinline__ void add(const T* row, int c0, int d, int tpr, float* acc) {
    float f[C];
    get(row, c0, d, tpr, f);
#pragma unroll
    for (int i = 0; i < C; ++i) acc[i] += f[i];
  }
  static __device__ __forceinline__ void get(const T* row, int c0, int d, int tpr, float* f) {
    if constexpr (VEC) {
      if (c0 < d) {
        Vec16<T>::load(row + c0, f);
        if (sizeof(T) == 4) Vec16<T>::load(row + c0 + 4, f + 4);
      }
    } else {
#pragma unroll
      for (int i = 0; i < C; ++i) f[i] = c0 + i * tpr < d ? ld_elem(row, c0 + i * tpr) : 0.0f;
    }
  }
  static __device__ __forceinline__ void put(float* row, int c0, int d, int tpr, const float* f) {
    if constexpr (VEC) {
      if (c0 < d) {
        store_vec<8>(row + c0, f);
      }
    } else {
#pragma unroll
      for (int i = 0; i < C; ++i)
        if (c0 + i * tpr < d) row[c0 + i * tpr] = f[i];
    }
  }
};

// Sum of sorted entries [b, e) at this thread's columns, ascending, four rows
// of dout in flight.
template <typename T, bool VEC>
__device__ __forceinline__ void sum_entries(const SumArgs& A, uint32_t b, uint32_t e, int c0, float* acc) {
  using L = Cols<T, VEC>;
  const T* dout = static_cast<const T*>(A.dout);
#pragma unroll
  for (int i = 0; i < L::C; ++i) acc[i] = 0.0f;
  uint32_t j = b;
  for (; j + 4 <= e; j += 4) {
    float f[4][L::C];
#pragma unroll
    for (int q = 0; q < 4; ++q) L::get(dout + (size_t)A.pos[j + q] * A.d, c0, A.d, A.tpr, f[q]);
#pragma unroll
    for (int q = 0; q < 4; ++q)
#pragma unroll
      for (int i = 0; i < L::C; ++i) acc[i] += f[q][i];
  }
  for (; j < e; ++j) L::add(dout + (size_t)A.pos[j] * A.d, c0, A.d, A.tpr, acc);
}

template <typename T, bool VEC>
__global__ void __launch_bounds__(256) embed_sum_kernel(const SumArgs A) {
  using L = Cols<T, VEC>;
  const int lane = threadIdx.x % A.tpr, sub = threadIdx.x / A.tpr, rpb = 256 / A.tpr;
  if ((int)blockIdx.x < A.hot_blocks) {
    // ---- one window of the sorted order, for the hot segments it meets
    __shared__ int last;
    const uint32_t j = blockIdx.x / A.col_tiles;
    const int tile = blockIdx.x % A.col_tiles;
    const uint32_t wb = j * A.window, we = min(A.n, wb + A.window);
    const uint32_t k0 = A.key[wb], k1 = A.key[we - 1];
    for (int slot = 0; slot < 2; ++slot) {
      const uint32_t k = slot ? k1 : k0;
      if (k >= A.V || (slot && k1 == k0)) continue;
      const uint32_t sb = A.start[k], se = A.start[k + 1];
      if (se - sb <= 2 * A.window) continue;
      const int c0 = L::first(tile, lane, A.tpr);
      float acc[L::C];
      if (sub == 0) {
        sum_entries<T, VEC>(A, max(sb, wb), min(se, we), c0, acc);
        L::put(A.part + ((size_t)j * 2 + slot) * A.d, c0, A.d, A.tpr, acc);
      }
      __threadfence();
      __syncthreads();
      const uint32_t w0 = sb / A.window, w1 = (se - 1) / A.window;
      if (threadIdx.x == 0)
        last = atomicAdd(&A.arrivals[(size_t)w0 * A.col_tiles + tile], 1u) == w1 - w0;
      __syncthreads();
      if (last && sub == 0) {
        // every window's partial is there: add them in order
        __threadfence();
#pragma unroll
        for (int i = 0; i < L::C; ++i) acc[i] = 0.0f;
        for (uint32_t w = w0; w <= w1; ++w) {
          const int sl = (w == w0 && sb % A.window) ? 1 : 0;
          const float* p = A.part + ((size_t)w * 2 + sl) * A.d;
          float f[L::C];
          if constexpr (VEC) {
            if (c0 < A.d) {
              const float4 a = __ldcg(reinterpret_cast<const float4*>(p + c0));
              const float4 b = __ldcg(reinterpret_cast<const float4*>(p + c0) + 1);
              f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
              f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
            }
          } else {
#pragma unroll
            for (int i = 0; i < L::C; ++i) f[i] = c0 + i * A.tpr < A.d ? __ldcg(p + c0 + i * A.tpr) : 0.0f;
          }
#pragma unroll
          for (int i = 0; i < L::C; ++i) acc[i] += f[i];
        }
#pragma unroll
        for (int i = 0; i < L::C; ++i) acc[i] *= A.scale;
        L::put(A.dtable + (size_t)k * A.d, c0, A.d, A.tpr, acc);
      }
      __syncthreads();
    }
    return;
  }
  // ---- rows of the table, each written once (hot rows by the blocks above)
  const long long items = (long long)A.V * A.col_tiles;
  const long long stride = (long long)(gridDim.x - A.hot_blocks) * rpb;
  for (long long it = (long long)(blockIdx.x - A.hot_blocks) * rpb + sub; it < items; it += stride) {
    const uint32_t v = (uint32_t)(it / A.col_tiles);
    const int c0 = L::first((int)(it % A.col_tiles), lane, A.tpr);
    const uint32_t b = A.start[v], e = A.start[v + 1];
    if (e - b > 2 * A.window) continue;
    float acc[L::C];
    sum_entries<T, VEC>(A, b, e, c0, acc);
#pragma unroll
    for (int i = 0; i < L::C; ++i) acc[i] *= A.scale;
    L::put(A.dtable + (size_t)v * A.d, c0, A.d, A.tpr, acc);
  }
}

// ---------------------------------------------------------------- workspace
struct Ws {
  size_t key[2], pos[2], start, counts, arrivals, part, bytes;
  uint32_t window, n_windows, sort_blocks;
  int tpr, col_tiles, passes;
};

Ws ws_layout(long long n, int V, int d) {
  Ws w = {};
  // d % 8 decides the column layout; both cover at most 256 threads a row
  const bool vec = d % 8 == 0;
  const int per = vec ? 8 : 4;
  w.tpr = threads_per_row((d + per - 1) / per);
  w.col_tiles = (d + w.tpr * per - 1) / (w.tpr * per);
  long long win = (n + kMaxWindows - 1) / kMaxWindows;
  w.window = (uint32_t)(win > kWindowMin ? win : kWindowMin);
  w.n_windows = (uint32_t)((n + w.window - 1) / w.window);
  w.sort_blocks = (uint32_t)((n + kSortTile - 1) / kSortTile);
  int bits = 1;
  while (((long long)V >> bits) != 0) ++bits;
  w.passes = (bits + kRadixBits - 1) / kRadixBits;
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
  w.start = take(((size_t)V + 1) * 4);
  w.counts = take((size_t)kRadix * w.sort_blocks * 4);
  w.arrivals = take((size_t)w.n_windows * w.col_tiles * 4);
  w.part = take((size_t)w.n_windows * 2 * d * 4);
  w.bytes = top;
  return w;
}

}  // namespace

size_t embedding_ws_bytes(long long n, int V, int d) { return ws_layout(n, V, d).bytes; }

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

cudaError_t embedding_bwd_sort(int id64, const void* ids, long long n, int V, int d, void* workspace,
                               cudaStream_t s) {
  const Ws w = ws_layout(n, V, d);
  char* base = static_cast<char*>(workspace);
  auto u32 = [&](size_t off) { return reinterpret_cast<uint32_t*>(base + off); };
  KeysIn in{ids, id64, V, nullptr, nullptr};
  for (int p = 0; p < w.passes && n > 0; ++p) {
    const int shift = p * kRadixBits;
    // the last pass writes buffer 0
    const int dst = (w.passes - 1 - p) & 1;
    sort_count_kernel<<<w.sort_blocks, kSortThreads, 0, s>>>(in, (uint32_t)n, shift, u32(w.counts));
    sort_scan_kernel<<<1, 1024, 0, s>>>(u32(w.counts), (uint32_t)kRadix * w.sort_blocks);
    sort_scatter_kernel<<<w.sort_blocks, kSortThreads, 0, s>>>(in, (uint32_t)n, shift, u32(w.counts),
                                                               u32(w.key[dst]), u32(w.pos[dst]));
    in.key = u32(w.key[dst]);
    in.pos = u32(w.pos[dst]);
  }
  const unsigned grid = (unsigned)((n + 1 + 255) / 256);
  sort_bounds_kernel<<<grid, 256, 0, s>>>(u32(w.key[0]), (uint32_t)n, (uint32_t)V, u32(w.start),
                                          u32(w.arrivals), w.n_windows * (uint32_t)w.col_tiles);
  return cudaGetLastError();
}

cudaError_t embedding_bwd_sum(DType t, const void* dout, long long n, int V, int d, float scale, float* dtable,
                              void* workspace, cudaStream_t s) {
  const Ws w = ws_layout(n, V, d);
  char* base = static_cast<char*>(workspace);
  SumArgs A;
  A.dout = dout;
  A.dtable = dtable;
  A.start = reinterpret_cast<uint32_t*>(base + w.start);
  A.key = reinterpret_cast<uint32_t*>(base + w.key[0]);
  A.pos = reinterpret_cast<uint32_t*>(base + w.pos[0]);
  A.part = reinterpret_cast<float*>(base + w.part);
  A.arrivals = reinterpret_cast<uint32_t*>(base + w.arrivals);
  A.n = (uint32_t)n;
  A.V = (uint32_t)V;
  A.d = d;
  A.scale = scale;
  A.window = w.window;
  A.n_windows = w.n_windows;
  A.col_tiles = w.col_tiles;
  A.tpr = w.tpr;
  // a segment can be hot only if all tokens could fill one
  A.hot_blocks = n > 2ll * w.window ? (int)w.n_windows * w.col_tiles : 0;
  const int rpb = 256 / w.tpr;
  const long long items = ((long long)V * w.col_tiles + rpb - 1) / rpb;
  const long long rows_grid = items < 152 * 16 ? items : 152 * 16;
  const unsigned grid = (unsigned)(rows_grid + A.hot_blocks);
  const bool vec = d % 8 == 0;
  if (t == DT_F32) {
    if (vec) embed_sum_kernel<float, true><<<grid, 256, 0, s>>>(A);
    else embed_sum_kernel<float, false><<<grid, 256, 0, s>>>(A);
  } else {
    if (vec) embed_sum_kernel<bf16, true><<<grid, 256, 0, s>>>(A);
    else embed_sum_kernel<bf16, false><<<grid, 256, 0, s>>>(A);
  }
  return cudaGetLastError();
}

}  // namespace mg

// ============================================================================
namespace {

using mg::op_fail;

constexpr long long kMaxIds = 0x7fffff00ll;   // positions and segment bounds are 32-bit

mg_status check_embedding(const char* fn, int dtype, int id_kind, long long n, int vocab, int dim, float scale) {
  if ((dtype != 0 && dtype != 1) || (id_kind != 0 && id_kind != 1))
    return op_fail(MG_ERR_INVALID_ARG, "%s: dtypes and id_kind must be 0 or 1", fn);
  if (vocab < 1 || vocab == 0x7fffffff || dim < 1)
    return op_fail(MG_ERR_SHAPE, "%s: vocab and dim must be positive (got %d, %d)", fn, vocab, dim);
  if (n < 0 || n > kMaxIds)
    return op_fail(MG_ERR_SHAPE, "%s: n must be in [0, %lld] (got %lld)", fn, kMaxIds, n);
  if (!(scale - scale == 0.0f)) return op_fail(MG_ERR_INVALID_ARG, "%s: scale is not finite", fn);
  return MG_OK;
}

}  // namespace

extern "C" size_t mg_embedding_workspace_bytes(long long n, int vocab, int dim) {
  if (n < 0 || n > kMaxIds || vocab < 1 || vocab == 0x7fffffff || dim < 1) return 0;
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
  cudaError_t e = mg::embedding_bwd_sort(id_kind, ids, n, vocab, dim, workspace, (cudaStream_t)stream);
  if (e == cudaSuccess)
    e = mg::embedding_bwd_sum((mg::DType)dtype, dout, n, vocab, dim, scale, dtable, workspace,
                              (cudaStream_t)stream);
  return mg::op_end(fn, e);
}

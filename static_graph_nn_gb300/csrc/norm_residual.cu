// The step between two blocks of a residual network: the block's output y is
// normalised, gated and added to the scaled residual stream, and the sum is
// normalised for the next block.
//   u = y r1 g1,  r1 = 1 / sqrt(mean(y^2) + eps)        (u = y without g1)
//   x' = s x + a u                                      (a: one gate for all rows, or one for each run of rows)
//   h = x' r2 g2, r2 = 1 / sqrt(mean(x'^2) + eps)
// Backward, from the gradients dx' and dh:
//   t = dx' + r2 (dh g2 - r2 x' mean(dh g2 r2 x'))      dx = s t
//   w = a t,  dy = r1 (w g1 - r1 y mean(w g1 r1 y))
//   dg2 = sum dh x' r2,  dg1 = sum w y r1,  da = sum t u (over the gate's rows)
//
// Bound by DRAM: four row vectors a row forward, six backward.  A block (a warp for
// narrow rows, a cluster for wide ones) works on consecutive rows, so that the gammas
// and the gate stay in its registers and the columns' sums too; the next row is on
// its way through shared memory meanwhile.  The backward needs one exchange a row:
// mean(w g1 y) is split into two sums that do not need t, which itself needs a mean.
// Each block's column sums go to the workspace (two fp32 rows), and a second launch
// adds them in order.
//
// 16384 x 2048 bf16: forward 46 us (5.8 TB/s), backward 76 (5.3 TB/s with the second
// launch, 4.3 us of it); more rows on their way or more blocks are slower (forward,
// blocks of 128 threads on a multiprocessor x rows in shared memory: 4 x 2 46.2 us,
// 3 x 2 49.6, 6 x 2 50.3, 4 x 3 49.6, 5 x 3 51.5; backward 4 x 2 78.7, 3 x 2 80.4, 3 x 3 81.9,
// 4 x 3 84.4), and holding x' and q in registers between the sums and the
// gradients, which leaves three blocks, is no faster (in a loop of the backward alone 75
// against 73).
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "f32x2.cuh"
#include "kernels.h"
#include "op_checks.h"

namespace mg {
namespace {

constexpr int kNrThreads = 256;   // of the kernels for any width

struct NormResArgs {
  const void* y;
  const void* x;
  const float* g1;
  const float* gate;
  const float* g2;
  int rows, dim, gate_rows;   // gate_rows: rows that share a gate
  float scale, eps;
  void* xo;
  void* h;
  float* rstd;
  int block_rows;             // consecutive rows of a block
  int stages;                 // rows in shared memory at once
  int row_units;              // 16-byte units of a row there
  int ranks, part;            // blocks that share a row, columns of each
};

struct NormResGradArgs {
  const void* dxo;
  const void* dh;
  const void* y;
  const void* x;
  const float* rstd;
  const float* g1;
  const float* gate;
  const float* g2;
  int rows, dim, gate_rows, gates;
  float scale;
  void* dy;
  void* dx;
  float* dg1;
  float* dgate;
  float* dg2;
  float* ws;                  // [blocks][2][dim]
  // blocks: `parts` for each gate (block_rows rows each), or, where parts is 1, one for each block_gates gates
  int parts, block_rows, block_gates;
  int stages, row_units;
  int ranks, part;            // blocks that share a row, columns of each
};

// ---- a row in a block's registers --------------------------------------------
// The next rows are copied ahead into a ring in shared memory, 16 bytes at a time.
// Where rows begin on 16 bytes (OWN) a thread holds U such units of each row, a
// block's width apart, and copies those itself, so that it waits for nothing but its
// own copies; units beyond the row, and rows that are not given, are zeros from the
// start.  Else all threads copy the 16-byte units that a row touches, with zeros for the
// bytes behind it, and after a barrier a thread takes words of four bytes, a warp's
// width apart.  bf16 rows that begin within a word have theirs shifted out of two, and
// stored with the lane before's half.  (14124 x 2124 bf16: forward 56 us, backward 112; by
// single elements 92 and 196; by units of 16 bytes, shifted out of two, 2.4 times the
// aligned rows' instructions and 193.)  The arithmetic takes two elements at a time.
template <typename T>
struct Unit {
  static constexpr int kPer = 16 / (int)sizeof(T);   // elements
  static constexpr int kPairs = kPer / 2;
};
// The column of a thread's element e.
template <typename T, bool OWN, int U>
__device__ __forceinline__ int column(int e) {
  constexpr int per = OWN ? Unit<T>::kPer : Unit<T>::kPer / 4;
  if (OWN) return ((int)threadIdx.x + e / per * (int)blockDim.x) * per + e % per;
  return ((int)threadIdx.x / 32 * U * 128 + (int)threadIdx.x % 32) * per + e / per * 32 * per + e % per;
}
// The fp32 vector's values at columns e and e + 1 of this thread, `other` where there are none.
template <typename T, bool OWN, int U>
__device__ __forceinline__ f32x2 vector_at(const float* v, int dim, float other, int e) {
  const int c = column<T, OWN, U>(e), d = column<T, OWN, U>(e + 1);
  if (OWN) {
    if (!v || c >= dim) return both(other);
    const float2 f = *reinterpret_cast<const float2*>(v + c);
    return both(f.x, f.y);
  }
  return both(v && c < dim ? v[c] : other, v && d < dim ? v[d] : other);
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
// N pairs of elements from e on of a row, which begins `at` bytes into its copy.
template <typename T, int U, int N>
__device__ __forceinline__ void pairs_at(const uint4* copy, int at, int e, f32x2* v) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(copy) + at / 4 + threadIdx.x / 32 * U * 128 + threadIdx.x % 32;
  if (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < N; ++i)
      v[i] = both(__uint_as_float(w[(e + 2 * i) * 32]), __uint_as_float(w[(e + 2 * i + 1) * 32]));
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      uint32_t u = w[(e / 2 + i) * 32];
      if (at & 2) u = __funnelshift_r(u, w[(e / 2 + i) * 32 + 1], 16);
      v[i] = widen2(u);
    }
  }
}
// Writes them to the row; by whole warps.
template <int U, int N>
__device__ __forceinline__ void store_pairs(float* row, int, int dim, int e, const f32x2* v) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int c = column<float, false, U>(e + 2 * i), d = column<float, false, U>(e + 2 * i + 1);
    const float2 f = parts(v[i]);
    if (c < dim) row[c] = f.x;
    if (d < dim) row[d] = f.y;
  }
}
template <int U, int N>
__device__ __forceinline__ void store_pairs(bf16* row, int at, int dim, int e, const f32x2* v) {
  const int lane = threadIdx.x & 31;
  if (at & 2) {   // words are the last lane's second element and this one's first
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = column<bf16, false, U>(e + 2 * i);
      uint16_t* half = reinterpret_cast<uint16_t*>(row) + c;
      const uint32_t w = narrow2(v[i]), last = __shfl_up_sync(~0u, w, 1);
      if (lane > 0 && c < dim)
        *reinterpret_cast<uint32_t*>(half - 1) = __funnelshift_r(last, w, 16);
      else if (c < dim)
        half[0] = (uint16_t)w;
      if (c + 1 < dim && (lane == 31 || c + 2 >= dim)) half[1] = (uint16_t)(w >> 16);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int c = column<bf16, false, U>(e + 2 * i);
      uint16_t* half = reinterpret_cast<uint16_t*>(row) + c;
      const uint32_t w = narrow2(v[i]);
      if (c + 1 < dim)
        *reinterpret_cast<uint32_t*>(half) = w;
      else if (c < dim)
        half[0] = (uint16_t)w;
    }
  }
}
template <typename T, int U>
__device__ __forceinline__ void copy_row(uint4* to, const T* p, int dim) {
#pragma unroll
  for (int j = 0; j < U; ++j) {
    const int u = threadIdx.x + j * blockDim.x;
    if (u * Unit<T>::kPer < dim)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                       (uint32_t)__cvta_generic_to_shared(to + j * blockDim.x + threadIdx.x)),
                   "l"(p + (size_t)u * Unit<T>::kPer)
                   : "memory");
  }
}
// The n elements of a matrix from element e on, with all of the 16-byte units that they
// touch, by all threads; zeros for the bytes behind them, up to the end of the next unit.
template <typename T>
__device__ __forceinline__ void copy_span(uint4* to, const T* m, size_t e, int n) {
  const int begin = (int)(e * sizeof(T) % 16), end = begin + n * (int)sizeof(T);
  const char* from = reinterpret_cast<const char*>(m + e) - begin;
  for (int b = threadIdx.x * 16; b < end + 16; b += blockDim.x * 16) {
    const int size = max(0, min(16, end - b));
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(to) + b),
                 "l"(size ? from + b : from), "r"(size)
                 : "memory");
  }
}
// Zeros in the units that no copy writes: those beyond the row, and all of a row that is not given.
template <typename T, int U>
__device__ __forceinline__ void clear_row(uint4* to, bool given, int dim) {
#pragma unroll
  for (int j = 0; j < U; ++j)
    if (!given || (int)(threadIdx.x + j * blockDim.x) * Unit<T>::kPer >= dim)
      to[j * blockDim.x + threadIdx.x] = make_uint4(0, 0, 0, 0);
}

// Zeros in all units, before the first copy.
__device__ __forceinline__ void clear_ring(uint4* ring, int units) {
  for (int i = threadIdx.x; i < units; i += blockDim.x) ring[i] = make_uint4(0, 0, 0, 0);
  __syncthreads();
}

constexpr int kNrWarps = 16;   // of a block, at most
constexpr int kNrRanks = 8;   // blocks that share wide rows, at most
// A block's place in its cluster, and its columns.
struct NormResPart {
  int block, rank, c0, dim;
};
template <typename A>
__device__ __forceinline__ NormResPart part_of(const A& a) {
  NormResPart p;
  p.block = blockIdx.x / a.ranks;
  p.rank = blockIdx.x % a.ranks;
  p.c0 = p.rank * a.part;
  p.dim = min(a.part, a.dim - p.c0);
  return p;
}
// Sums of N values over a row's blocks, the same in every thread.  `turn` alternates from
// call to call: the barrier of one call lies between the reads of the call before it
// and the writes of the call after it.  A block writes its sums to every block of its
// cluster; after the last call's barrier none is written to any more.
template <int N>
struct RowSums {
  alignas(16) float warp[2][N][kNrWarps];
  float block[2][kNrRanks][N];
};
template <int N>
__device__ __forceinline__ void row_sums(float (&v)[N], RowSums<N>& red, int& turn, int rank, int ranks) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
#pragma unroll
  for (int n = 0; n < N; ++n) v[n] = warp_sum(v[n]);
  if (warps == 1) return;
  const int now = turn;
  turn ^= 1;
  if (lane == 0) {
#pragma unroll
    for (int n = 0; n < N; ++n) red.warp[now][n][warp] = v[n];
  }
  __syncthreads();
#pragma unroll
  for (int n = 0; n < N; ++n) v[n] = 0.0f;
  for (int w = 0; w < warps; w += 4) {
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const float4 f = *reinterpret_cast<const float4*>(&red.warp[now][n][w]);   // (zeros beyond the warps)
      v[n] += (f.x + f.y) + (f.z + f.w);
    }
  }
  if (ranks == 1) return;
  if ((int)threadIdx.x < ranks) {
    uint64_t to;
    asm("mapa.u64 %0, %1, %2;" : "=l"(to) : "l"((uint64_t)&red.block[now][rank][0]), "r"(threadIdx.x));
#pragma unroll
    for (int n = 0; n < N; ++n) reinterpret_cast<float*>(to)[n] = v[n];
  }
  asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
#pragma unroll
  for (int n = 0; n < N; ++n) {
    v[n] = 0.0f;
    for (int i = 0; i < ranks; ++i) v[n] += *reinterpret_cast<volatile float*>(&red.block[now][i][n]);
  }
}
// Zeros beyond the warps (the first sums' barrier lies between them and their reads); in
// a cluster, every block is there before one writes to it.
template <int N>
__device__ __forceinline__ void clear_sums(RowSums<N>& red, int ranks) {
  const int warps = blockDim.x >> 5;
  for (int i = threadIdx.x; i < 2 * kNrWarps * N; i += blockDim.x)
    if (i % kNrWarps >= warps) (&red.warp[0][0][0])[i] = 0.0f;
  if (ranks > 1) asm volatile("barrier.cluster.arrive.release.aligned;\nbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// 1 / sqrt(x): an estimate and one step of Newton's method.
__device__ __forceinline__ float inverse_root(float x) {
  const float r = rsqrtf(x);
  return r > 0.0f ? fmaf(r, 0.5f * fmaf(-x * r, r, 1.0f), r) : r;   // (0 of infinity, NaN of NaN)
}

// Rows in shared memory, one of them in use.  The kernels get the number as an argument: as a constant it made the aligned
// backward slower, whose registers the compiler then fills with addresses (fp32, 256 wide: 94 us against 81, 4096: 82
// against 75).
constexpr int kNrStages = 2;
// All but the youngest N groups of copies are there.
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <typename T, int U, bool OWN, int T0>
__global__ void __launch_bounds__(T0, T0 == 32 ? 24 : (U * Unit<T>::kPer == 8 ? 768 : T0 == 320 ? 640 : 512) / T0) norm_res_kernel(NormResArgs a) {
  constexpr int per = Unit<T>::kPer, pairs = Unit<T>::kPairs, E = U * per, P = E / 2;
  extern __shared__ __align__(16) uint4 ring[];   // [stage][y, x][U][threads]
  __shared__ RowSums<1> red;
  const NormResPart my = part_of(a);
  const int dim = my.dim;
  clear_sums<1>(red, a.ranks);
  const int array = OWN ? U * blockDim.x : a.row_units, stage = 2 * array;
  const int first = my.block * a.block_rows, end = min(first + a.block_rows, a.rows);
  const T *ys = static_cast<const T*>(a.y), *xs = static_cast<const T*>(a.x);
  const auto row_at = [&](int r) { return (size_t)r * a.dim + my.c0; };
  int fill = 0;
  const auto ahead = [&](int r) {
    uint4* to = ring + fill * stage;
    if (r < end && OWN) {
      copy_row<T, U>(to, ys + row_at(r), dim);
      copy_row<T, U>(to + array, xs + row_at(r), dim);
    } else if (r < end) {
      copy_span(to, ys, row_at(r), dim);
      copy_span(to + array, xs, row_at(r), dim);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    fill = fill + 1 == a.stages ? 0 : fill + 1;
  };
  // (the vectors' loads and the first rows' copies are under way together)
  f32x2 w[P], g2[P];
#pragma unroll
  for (int p = 0; p < P; ++p) g2[p] = vector_at<T, OWN, U>(a.g2 ? a.g2 + my.c0 : nullptr, dim, 0.0f, 2 * p);
  if (!OWN) clear_ring(ring, a.stages * stage);
  for (int i = 0; i < a.stages - 1; ++i) ahead(first + i);
  if (OWN)
    for (int i = 0; i < 2 * a.stages; ++i) clear_row<T, U>(ring + i * array, true, dim);
  const float inv_dim = 1.0f / a.dim;
  const f32x2 scale = both(a.scale);
  int gate_end = first, slot = 0, turn = 0;
  for (int r = first; r < end; ++r) {
    if (r == gate_end) {   // the product of the post norm's factors and the gate, kept for the gate's rows
      const int gi = r / a.gate_rows;
      const float* gate = a.gate ? a.gate + (size_t)gi * a.dim + my.c0 : nullptr;
#pragma unroll
      for (int p = 0; p < P; ++p)
        w[p] = mul2(vector_at<T, OWN, U>(a.g1 ? a.g1 + my.c0 : nullptr, dim, 1.0f, 2 * p), vector_at<T, OWN, U>(gate, dim, 1.0f, 2 * p));
      gate_end = (gi + 1) * a.gate_rows;
    }
    f32x2 y[P], x[P];
    const int at = (int)(row_at(r) * sizeof(T) % 16);
    const uint4* in = ring + slot * stage;
    slot = slot + 1 == a.stages ? 0 : slot + 1;
    if (OWN) {
      ahead(r + a.stages - 1);
      copies_wait<kNrStages - 1>();
      in += threadIdx.x;
#pragma unroll
      for (int j = 0; j < U; ++j) {
        widen(in[j * blockDim.x], reinterpret_cast<f32x2(&)[pairs]>(y[j * pairs]));
        widen(in[array + j * blockDim.x], reinterpret_cast<f32x2(&)[pairs]>(x[j * pairs]));
      }
    } else {
      copies_wait<kNrStages - 2>();
      __syncthreads();             // row r is there, and the row before it has been read
      ahead(r + a.stages - 1);
      pairs_at<T, U, P>(in, at, 0, y);
      pairs_at<T, U, P>(in + array, at, 0, x);
    }
    float r1 = 1.0f, r2 = 1.0f;
    const auto root_of = [&](const f32x2 (&v)[P]) {
      f32x2 s = both(0.0f);
#pragma unroll
      for (int p = 0; p < P; ++p) s = fma2(v[p], v[p], s);
      const float2 t = parts(s);
      float q[1] = {t.x + t.y};
      row_sums<1>(q, red, turn, my.rank, a.ranks);
      return inverse_root(fmaf(q[0], inv_dim, a.eps));
    };
    if (a.g1) r1 = root_of(y);
    const f32x2 rr = both(r1);
#pragma unroll
    for (int p = 0; p < P; ++p) x[p] = fma2(scale, x[p], mul2(mul2(y[p], w[p]), rr));
    if (a.g2) r2 = root_of(x);
    T* xo = static_cast<T*>(a.xo) + row_at(r);
    T* h = a.h ? static_cast<T*>(a.h) + row_at(r) : nullptr;
    const f32x2 rq = both(r2);
    if (OWN) {
#pragma unroll
      for (int j = 0; j < U; ++j) {
        const int c = column<T, OWN, U>(j * per);
        if (c >= dim) continue;
        f32x2 f[pairs];
#pragma unroll
        for (int i = 0; i < pairs; ++i) f[i] = x[j * pairs + i];
        *reinterpret_cast<uint4*>(xo + c) = narrow(f);
        if (!h) continue;
#pragma unroll
        for (int i = 0; i < pairs; ++i) f[i] = mul2(f[i], mul2(rq, g2[j * pairs + i]));
        *reinterpret_cast<uint4*>(h + c) = narrow(f);
      }
    } else {
      store_pairs<U, P>(xo, at, dim, 0, x);
      if (h) {
#pragma unroll
        for (int p = 0; p < P; ++p) x[p] = mul2(x[p], mul2(rq, g2[p]));
        store_pairs<U, P>(h, at, dim, 0, x);
      }
    }
    if (a.rstd && my.rank == 0 && threadIdx.x == 0) *reinterpret_cast<float2*>(a.rstd + 2 * (size_t)r) = make_float2(r1, r2);
  }
}

// A block's rows, gate by gate: rows [first, end) of gate g.
struct NormResSpan {
  int g, first, end;
};
__device__ __forceinline__ bool next_span(const NormResGradArgs& a, int block, NormResSpan& s) {
  if (a.parts > 1) {
    if (s.g >= 0) return false;
    s.g = block / a.parts;
    s.first = s.g * a.gate_rows + block % a.parts * a.block_rows;
    s.end = min(s.first + a.block_rows, (s.g + 1) * a.gate_rows);
    return s.first < s.end;
  }
  s.g = s.g < 0 ? block * a.block_gates : s.g + 1;
  s.first = s.g * a.gate_rows;
  s.end = s.first + a.gate_rows;
  return s.g < min((block + 1) * a.block_gates, a.gates);
}
// A column's sums over a span.  P = sum t y r1 gives both the gate's gradient, g1 P,
// and, times the gate, the post norm's.  Where a block has whole gates it writes
// their gradients and keeps the post norm's; else it keeps P.
__device__ __forceinline__ void span_sums(const NormResGradArgs& a, int block, const NormResSpan& s, bool first, int c, float P) {
  float* keep = a.ws + (size_t)block * 2 * a.dim + c;
  if (a.parts > 1) {
    *keep = P;
    return;
  }
  if (a.dgate) a.dgate[(size_t)s.g * a.dim + c] = a.g1 ? a.g1[c] * P : P;
  if (a.gate) P *= a.gate[(size_t)s.g * a.dim + c];
  *keep = first ? P : *keep + P;
}

// The three sums of a row in one exchange.  With b = w y (w = gate g1) and q = dx' + r2 dh g2: m1 = r2 mean(dh g2 x') and
// sum w t y = sum b q - m1 r2^2 sum b x'.  With m2 = r1 mean(w t y), t = dx' + r2 (dh g2 - r2 m1 x') and dy = r1 (w t -
// r1 m2 y): r1 y, r2 x', m1 and m2 stay near the gradients' and vectors' size whatever the rows' magnitude, and no power
// of a root is formed.  (The cube of one leaves fp32's range where rows are 1e13 or 1e-13, and where they are 0 under an eps
// below 1e-25.)
template <typename T, int U, bool OWN, int T0>
__global__ void __launch_bounds__(T0, T0 == 32 ? 24 : (U * Unit<T>::kPer == 8 ? 768 : 512) / T0) norm_res_grad_kernel(NormResGradArgs a) {
  constexpr int per = Unit<T>::kPer, pairs = Unit<T>::kPairs, E = U * per, P = E / 2;
  constexpr int N = sizeof(T) == 4 ? 1 : pairs;   // at any offset: pairs of a row at a time, as registers allow
  extern __shared__ __align__(16) uint4 ring[];   // [stage][y, x, dx_out, dh][U][threads]
  __shared__ RowSums<3> red;
  const NormResPart my = part_of(a);
  const int dim = my.dim;
  clear_sums<3>(red, a.ranks);
  const int array = OWN ? U * blockDim.x : a.row_units, stage = 4 * array;
  const T *ys = static_cast<const T*>(a.y), *xs = static_cast<const T*>(a.x);
  const T *os = static_cast<const T*>(a.dxo), *hs = static_cast<const T*>(a.dh);
  const float inv_dim = 1.0f / a.dim;
  const f32x2 scale = both(a.scale);
  f32x2 sp[P], s2[P], w[P], g2[P];
#pragma unroll
  for (int p = 0; p < P; ++p) {
    s2[p] = both(0.0f);
    g2[p] = vector_at<T, OWN, U>(hs ? a.g2 + my.c0 : nullptr, dim, 0.0f, 2 * p);
  }
  const auto clear = [&] {
    if (OWN)
      for (int i = 0; i < a.stages; ++i) {
        clear_row<T, U>(ring + i * stage, true, dim);
        clear_row<T, U>(ring + i * stage + array, true, dim);
        clear_row<T, U>(ring + i * stage + 2 * array, os != nullptr, dim);
        clear_row<T, U>(ring + i * stage + 3 * array, hs != nullptr, dim);
      }
  };
  NormResSpan s = {-1, 0, 0};
  bool any = false;
  int turn = 0;
  while (next_span(a, my.block, s)) {
    const float* gate = a.gate ? a.gate + (size_t)s.g * a.dim + my.c0 : nullptr;
    int fill = 0, slot = 0;
    const auto ahead = [&](int r) {
      uint4* to = ring + fill * stage;
      const size_t at = (size_t)r * a.dim + my.c0;
      if (r < s.end && OWN) {
        copy_row<T, U>(to, ys + at, dim);
        copy_row<T, U>(to + array, xs + at, dim);
        if (os) copy_row<T, U>(to + 2 * array, os + at, dim);
        if (hs) copy_row<T, U>(to + 3 * array, hs + at, dim);
      } else if (r < s.end) {
        copy_span(to, ys, at, dim);
        copy_span(to + array, xs, at, dim);
        if (os) copy_span(to + 2 * array, os, at, dim);
        if (hs) copy_span(to + 3 * array, hs, at, dim);
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
      fill = fill + 1 == a.stages ? 0 : fill + 1;
    };
    if (!OWN && any) __syncthreads();   // the last span's rows have been read
    if (!OWN && !any) clear_ring(ring, a.stages * stage);
    // (the vectors' loads and the first rows' copies are under way together)
    const float2* roots = reinterpret_cast<const float2*>(a.rstd);
    float2 root = roots[s.first];
    f32x2 g1[P], ga[P];
#pragma unroll
    for (int p = 0; p < P; ++p) {
      g1[p] = vector_at<T, OWN, U>(a.g1 ? a.g1 + my.c0 : nullptr, dim, 1.0f, 2 * p);
      ga[p] = vector_at<T, OWN, U>(gate, dim, 1.0f, 2 * p);
    }
    for (int i = 0; i < a.stages - 1; ++i) ahead(s.first + i);
    if (!any) clear();
#pragma unroll
    for (int p = 0; p < P; ++p) {
      sp[p] = both(0.0f);
      w[p] = mul2(g1[p], ga[p]);
    }
    for (int r = s.first; r < s.end; ++r) {
      const size_t at = (size_t)r * a.dim + my.c0;
      const float r1 = a.g1 ? root.x : 1.0f, r2 = hs ? root.y : 1.0f;
      const f32x2 rr1 = both(r1), rr2 = both(r2);
      const int off = (int)(at * sizeof(T) % 16);
      const uint4* in = ring + slot * stage;
      slot = slot + 1 == a.stages ? 0 : slot + 1;
      if (OWN) {
        ahead(r + a.stages - 1);
        copies_wait<kNrStages - 1>();
        in += threadIdx.x;
      } else {
        copies_wait<kNrStages - 2>();
        __syncthreads();             // row r is there, and the row before it has been read
        ahead(r + a.stages - 1);
      }
      if (r + 1 < s.end) root = roots[r + 1];
      const auto unit = [&](int j, f32x2 (&y)[pairs], f32x2 (&x)[pairs], f32x2 (&o)[pairs], f32x2 (&h)[pairs]) {
        if (OWN) {
          widen(in[j * blockDim.x], y);
          widen(in[array + j * blockDim.x], x);
          widen(in[2 * array + j * blockDim.x], o);
          widen(in[3 * array + j * blockDim.x], h);
        } else {
#pragma unroll
          for (int i = 0; i < pairs; i += N) {
            const int e = j * per + 2 * i;
            pairs_at<T, U, N>(in, off, e, y + i);
            pairs_at<T, U, N>(in + array, off, e, x + i);
            pairs_at<T, U, N>(in + 2 * array, off, e, o + i);
            pairs_at<T, U, N>(in + 3 * array, off, e, h + i);
          }
        }
      };
      f32x2 t1 = both(0.0f), t2 = t1, t3 = t1;
#pragma unroll
      for (int j = 0; j < U; ++j) {
        f32x2 y[pairs], x[pairs], o[pairs], h[pairs];
        unit(j, y, x, o, h);
#pragma unroll
        for (int i = 0; i < pairs; ++i) {
          const int p = j * pairs + i;
          const f32x2 b = mul2(w[p], y[i]), xo = fma2(rr1, b, mul2(scale, x[i])), v = mul2(h[i], g2[p]);
          t1 = fma2(v, xo, t1);
          t2 = fma2(b, fma2(rr2, v, o[i]), t2);
          t3 = fma2(b, xo, t3);
        }
      }
      const float2 u1 = parts(t1), u2 = parts(t2), u3 = parts(t3);
      float sum[3] = {u1.x + u1.y, u2.x + u2.y, u3.x + u3.y};
      row_sums<3>(sum, red, turn, my.rank, a.ranks);
      const float m1 = hs ? r2 * (sum[0] * inv_dim) : 0.0f;
      const float m2 = a.g1 ? r1 * ((hs ? fmaf(-m1, r2 * (r2 * sum[2]), sum[1]) : sum[1]) * inv_dim) : 0.0f;
      const f32x2 n1 = both(-r2 * m1), n2 = both(-r1 * m2);
#pragma unroll
      for (int j = 0; j < U; ++j) {
        f32x2 y[pairs], x[pairs], o[pairs], h[pairs];
        unit(j, y, x, o, h);
#pragma unroll
        for (int i = 0; i < pairs; ++i) {
          const int p = j * pairs + i;
          const f32x2 wp = w[p], xo = fma2(rr1, mul2(wp, y[i]), mul2(scale, x[i]));
          const f32x2 t = fma2(rr2, fma2(n1, xo, mul2(h[i], g2[p])), o[i]);
          sp[p] = fma2(t, mul2(y[i], rr1), sp[p]);
          s2[p] = fma2(mul2(h[i], rr2), xo, s2[p]);
          x[i] = mul2(scale, t);
          y[i] = mul2(rr1, fma2(n2, y[i], mul2(wp, t)));
        }
        if (OWN) {
          const int c = column<T, OWN, U>(j * per);
          if (c >= dim) continue;
          *reinterpret_cast<uint4*>(static_cast<T*>(a.dy) + at + c) = narrow(y);
          *reinterpret_cast<uint4*>(static_cast<T*>(a.dx) + at + c) = narrow(x);
        } else {
#pragma unroll
          for (int i = 0; i < pairs; i += N) {
            store_pairs<U, N>(static_cast<T*>(a.dy) + at, off, dim, j * per + 2 * i, y + i);
            store_pairs<U, N>(static_cast<T*>(a.dx) + at, off, dim, j * per + 2 * i, x + i);
          }
        }
      }
    }
    if (a.parts > 1) dependents_start();   // (the join waits for the whole grid all the same)
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const float2 f = parts(sp[p]);
      const int c = column<T, OWN, U>(2 * p), d = column<T, OWN, U>(2 * p + 1);
      if (c < dim) span_sums(a, my.block, s, !any, my.c0 + c, f.x);
      if (d < dim) span_sums(a, my.block, s, !any, my.c0 + d, f.y);
    }
    any = true;
  }
  float* keep = a.ws + (size_t)my.block * 2 * a.dim + my.c0;
#pragma unroll
  for (int p = 0; p < P; ++p) {
    const float2 f = parts(s2[p]);
    const int c = column<T, OWN, U>(2 * p), d = column<T, OWN, U>(2 * p + 1);
    if (c < dim) keep[a.dim + c] = f.x;
    if (d < dim) keep[a.dim + d] = f.y;
  }
}

// ---- rows of any width: read again for every sum -------------------------------
template <typename T>
__global__ void __launch_bounds__(kNrThreads) norm_res_wide_kernel(NormResArgs a) {
  __shared__ float red[32];
  const size_t row = (size_t)blockIdx.x * a.dim;
  const T *y = static_cast<const T*>(a.y) + row, *x = static_cast<const T*>(a.x) + row;
  const float* gate = a.gate ? a.gate + (size_t)(blockIdx.x / a.gate_rows) * a.dim : nullptr;
  float r1 = 1.0f, r2 = 1.0f;
  if (a.g1) {
    float s = 0.0f;
    for (int c = threadIdx.x; c < a.dim; c += kNrThreads) s += ld_elem(y, c) * ld_elem(y, c);
    r1 = 1.0f / sqrtf(block_sum(s, red) / a.dim + a.eps);
  }
  auto out = [&](int c) {
    float u = ld_elem(y, c);
    if (a.g1) u *= r1 * a.g1[c];
    if (gate) u *= gate[c];
    return a.scale * ld_elem(x, c) + u;
  };
  if (a.g2) {
    float s = 0.0f;
    for (int c = threadIdx.x; c < a.dim; c += kNrThreads) {
      const float v = out(c);
      s += v * v;
    }
    r2 = 1.0f / sqrtf(block_sum(s, red) / a.dim + a.eps);
  }
  for (int c = threadIdx.x; c < a.dim; c += kNrThreads) {
    const float v = out(c);
    st_elem(static_cast<T*>(a.xo) + row, c, v);
    if (a.h) st_elem(static_cast<T*>(a.h) + row, c, v * r2 * a.g2[c]);
  }
  if (a.rstd && threadIdx.x == 0) {
    a.rstd[2 * (size_t)blockIdx.x] = r1;
    a.rstd[2 * (size_t)blockIdx.x + 1] = r2;
  }
}

template <typename T>
__global__ void __launch_bounds__(kNrThreads) norm_res_grad_wide_kernel(NormResGradArgs a) {
  __shared__ float red[32];
  float* sums = a.ws + (size_t)blockIdx.x * 2 * a.dim;   // the post norm's (or P), the pre norm's
  for (int c = threadIdx.x; c < a.dim; c += kNrThreads) sums[c] = sums[(size_t)a.dim + c] = 0.0f;   // (2 dim may pass 2^31)
  __syncthreads();
  NormResSpan span = {-1, 0, 0};
  while (next_span(a, blockIdx.x, span)) {
    const float* gate = a.gate ? a.gate + (size_t)span.g * a.dim : nullptr;
    for (int r = span.first; r < span.end; ++r) {
      const size_t row = (size_t)r * a.dim;
      const T *y = static_cast<const T*>(a.y) + row, *x = static_cast<const T*>(a.x) + row;
      const T* dxo = a.dxo ? static_cast<const T*>(a.dxo) + row : nullptr;
      const T* dh = a.dh ? static_cast<const T*>(a.dh) + row : nullptr;
      const float r1 = a.g1 ? a.rstd[2 * (size_t)r] : 1.0f, r2 = dh ? a.rstd[2 * (size_t)r + 1] : 1.0f;
      auto w = [&](int c) { return (a.g1 ? a.g1[c] : 1.0f) * (gate ? gate[c] : 1.0f); };
      auto sum = [&](int c) { return a.scale * ld_elem(x, c) + r1 * (w(c) * ld_elem(y, c)); };
      float s1 = 0.0f;
      if (dh) {
        for (int c = threadIdx.x; c < a.dim; c += kNrThreads) s1 += ld_elem(dh, c) * a.g2[c] * sum(c);
        s1 = block_sum(s1, red) / a.dim;
      }
      auto total = [&](int c) {
        float t = dxo ? ld_elem(dxo, c) : 0.0f;
        if (dh) t += r2 * (ld_elem(dh, c) * a.g2[c] - sum(c) * r2 * r2 * s1);
        return t;
      };
      float s2 = 0.0f;
      if (a.g1) {
        for (int c = threadIdx.x; c < a.dim; c += kNrThreads) s2 += w(c) * total(c) * ld_elem(y, c);
        s2 = block_sum(s2, red) / a.dim;
      }
      for (int c = threadIdx.x; c < a.dim; c += kNrThreads) {
        const float t = total(c), yc = ld_elem(y, c), g = a.parts == 1 && gate ? gate[c] : 1.0f;
        const float P = t * yc * r1;
        sums[c] += g * P;
        if (a.parts == 1 && a.dgate) {
          float* d = a.dgate + (size_t)span.g * a.dim + c;
          *d = (r == span.first ? 0.0f : *d) + (a.g1 ? a.g1[c] * P : P);
        }
        if (dh) sums[a.dim + c] += ld_elem(dh, c) * sum(c) * r2;
        const float d = r1 * w(c) * t - yc * r1 * r1 * r1 * s2;
        st_elem(static_cast<T*>(a.dy) + row, c, d);
        st_elem(static_cast<T*>(a.dx) + row, c, a.scale * t);
      }
    }
  }
}

// The blocks' sums in order: `wide` columns a block, for each of them runs of blocks
// added side by side and then in order.  blockIdx.y: 0 the post norm's (and that of a
// gate for all rows, which is made of the same sums), 1 the pre norm's, beyond the gates'
// (blocks have parts of them).
__global__ void __launch_bounds__(1024) norm_res_join_kernel(NormResGradArgs a, int blocks, int wide) {
  __shared__ float red[1024 + 128];
  const int col = threadIdx.x % wide, run = threadIdx.x / wide, runs = blockDim.x / wide, c = blockIdx.x * wide + col;
  const bool in = c < a.dim, gated = blockIdx.y == 0 && a.gate && a.parts > 1 && a.gates > 1;
  dependency_wait();
  const auto add = [&](int which, size_t from, int n) {
    const int per = (n + runs - 1) / runs, begin = min(n, run * per), end = min(n, begin + per);
    const float* v = a.ws + (from * 2 + which) * a.dim + c;
    float s = 0.0f;
    const auto some = [&](int from_block, int to_block) {   // eight loads under way at once
      float t = 0.0f;
      for (int i0 = from_block; i0 < to_block; i0 += 8) {
        float u[8];
#pragma unroll
        for (int q = 0; q < 8; ++q) u[q] = i0 + q < to_block ? v[(size_t)(i0 + q) * 2 * a.dim] : 0.0f;
#pragma unroll
        for (int q = 0; q < 8; ++q) t += u[q];
      }
      return t;
    };
    if (in && gated)   // gate by gate
      for (int g = begin / a.parts, i = begin; i < end; i = (++g) * a.parts)
        s = fmaf(a.gate[(size_t)g * a.dim + c], some(i, min(end, (g + 1) * a.parts)), s);
    else if (in)
      s = some(begin, end);
    red[run * (wide + 1) + col] = s;
    __syncthreads();
    float t = 0.0f;
    if (run == 0)
      for (int i = 0; i < runs; ++i) t += red[i * (wide + 1) + col];
    __syncthreads();
    return t;
  };
  const bool writes = run == 0 && in;
  if (blockIdx.y == 0) {
    if (!a.dg1 && !(a.dgate && a.gates == 1)) return;
    const float t = add(0, 0, blocks);
    const bool one = a.gates == 1 && a.parts > 1;   // then t is the sum of the P
    if (writes && a.dg1) a.dg1[c] = one && a.gate ? a.gate[c] * t : t;
    if (writes && a.dgate && one) a.dgate[c] = a.g1 ? a.g1[c] * t : t;
  } else if (blockIdx.y == 1) {
    if (!a.dg2) return;
    const float t = a.dh ? add(1, 0, blocks) : 0.0f;
    if (writes) a.dg2[c] = t;
  } else {
    for (int g = blockIdx.y - 2; g < a.gates; g += gridDim.y - 2) {
      const float t = add(0, (size_t)g * a.parts, a.parts);
      if (writes) a.dgate[(size_t)g * a.dim + c] = a.g1 ? a.g1[c] * t : t;
    }
  }
}
__global__ void __launch_bounds__(256) norm_res_zero_kernel(NormResGradArgs a) {
  const size_t i = (size_t)blockIdx.x * 256 + threadIdx.x, n = (size_t)a.gates * a.dim;
  if (a.dgate && i < n) a.dgate[i] = 0.0f;
  if (a.dg1 && i < (size_t)a.dim) a.dg1[i] = 0.0f;
  if (a.dg2 && i < (size_t)a.dim) a.dg2[i] = 0.0f;
}

// ---- which kernel ----------------------------------------------------------------
struct NormResShape {
  int threads = 0;   // 0: the kernels for any width
  int each = 0;      // elements a thread
  bool own = false;
  bool more = false;   // 640 threads on a multiprocessor instead of 512
  int row_units = 0, ranks = 1, part = 0;
  size_t smem = 0;
};
constexpr size_t kNrSmem = 220 * 1024;
constexpr int kNrMost = 512;
constexpr int kNrFew = 192;
// A warp of eight elements a lane for the narrowest rows, else sixteen elements a
// thread, which take fewer exchanges (32768 x 1024 bf16 backward: 76 us against 80), but
// eight up to 1024 where that leaves fewer threads without elements (16384 x 600 fp32:
// 52 us against 57) or where blocks have few rows each and their start counts (2000 x 1000
// bf16: 16.1 us against 18.6).  A cluster of blocks where a row is more than the threads
// of one hold, or two rows of it more than shared memory does: backward, of blocks of up
// to 192 threads, of which a multiprocessor has several (2142 x 14000 bf16 102 us, 1831 x
// 8192 fp32 91; of up to 512 threads 124 and 119), forward, of up to 512 (1500 x 20000 bf16
// 83 us against 94).  Rows that one block holds are faster so (6000 x 5000 bf16 backward 89
// us, by clusters 103).  Forward, 96 registers a thread are enough where they let one
// more block onto a multiprocessor (bf16 7322 x 4097 72 us against 103, 5859 x 5120 44 against 56,
// 10000 x 3000 45 against 50; fp32 3661 x 4097 46 against 55, but 5000 x 3000 44.6 against
// 42.5: where it doubles the blocks); backward they are not (6000 x 5000 bf16 113 against 89).
NormResShape norm_res_shape(int dtype, int rows, int dim, bool grad) {
  NormResShape s;
  const int es = dtype ? 2 : 4, per = 16 / es;
  s.own = (size_t)dim * es % 16 == 0;
  for (const int few : {kNrFew, kNrMost}) {
    for (s.ranks = 1; s.ranks <= kNrRanks; s.ranks *= 2) {
      const int most = grad && s.ranks > 1 ? few : kNrMost;
      s.part = (dim + s.ranks - 1) / s.ranks;
      if (s.own) s.part = (s.part + per - 1) / per * per;
      // (forward: 32 elements a thread before two blocks, which cost a row two exchanges)
      s.each = s.part <= 256 ? 8 : s.part <= 16 * 512 || grad ? 16 : 32;
      int threads = ((s.part + s.each - 1) / s.each + 31) / 32 * 32;
      if (s.each == 16 && s.part <= 1024) {
        const int eight = ((s.part + 7) / 8 + 31) / 32 * 32;
        if (20 * eight < 17 * 2 * threads || rows < 8 * device_sms() * 512 / threads) {
          s.each = 8;
          threads = eight;
        }
      }
      if (threads > most) continue;
      s.row_units = s.each * es * threads / 16 + (s.own ? 0 : 2);
      s.smem = (size_t)kNrStages * (grad ? 4 : 2) * s.row_units * 16;
      if (s.smem > kNrSmem) continue;
      s.threads = threads;
      s.more = !grad && s.each == 16 && threads > (dtype ? 128 : 256) && 640 / threads > 512 / threads;
      return s;
    }
  }
  s.ranks = 1;
  return s;
}
// Rows that are worked on at once: by registers (128 a thread; 80 in the narrowest) and by
// shared memory.  Clusters may be fewer, as they do not fill all multiprocessors: the
// launch asks how many run at once, or its last ones would wait for a second round (3125 x
// 9600 bf16 backward, 112 clusters where 110 run: 151 us against 100).
int norm_res_slots(const NormResShape& s) {
  if (!s.threads) return device_sms() * 4;
  int n = (s.each == 8 ? 768 : s.more ? 640 : 512) / s.threads;
  n = std::max(1, std::min(n, (int)(kNrSmem / (s.smem + 2048))));
  return std::max(1, device_sms() * n / s.ranks);
}

struct NormResSplit {
  int parts, block_rows, block_gates;
  long long blocks;
};
// Few gates: one round of blocks, whole parts of a gate each; more: four rounds, of
// which the last may be partly empty, at eight rows or more to a part (a block also
// writes two fp32 rows of sums).
NormResSplit norm_res_split(int rows, int gates, int slots) {
  NormResSplit p;
  const int per = rows / gates;
  int parts = slots / gates >= 4 ? slots / gates : std::min((4 * slots + gates - 1) / gates, (per + 7) / 8);
  parts = std::max(1, std::min(parts, per));
  p.block_rows = (per + parts - 1) / parts;
  p.parts = (per + p.block_rows - 1) / p.block_rows;
  p.block_gates = p.parts > 1 ? 1 : std::max(1, gates / (4 * slots));
  p.blocks = p.parts > 1 ? (long long)gates * p.parts : (gates + p.block_gates - 1) / p.block_gates;
  return p;
}

// At least the blocks of any split of these rows or fewer: one round of them, or (the
// split's four rounds, rounded up twice) eight.
long long norm_res_most_blocks(int rows, int dim, int gates) {
  long long most = 1;
  for (int dtype = 0; dtype < 2; ++dtype)
    for (int r : {1, rows}) {
      const NormResShape shape = norm_res_shape(dtype, r, dim, true);
      const int slots = norm_res_slots(shape);
      // (clusters: half the slots or more, see norm_res_clusters)
      most = std::max(most, slots / gates >= (shape.ranks > 1 ? 8 : 4) ? (long long)slots : 8ll * slots);
    }
  return std::min<long long>(most, std::max(rows, 1));
}

// The slots of a cluster's shape, of which `active` run at once.
int norm_res_clusters(int slots, int active) { return std::max((slots + 1) / 2, std::min(slots, active)); }

// Launches, or, with `active`, tells how many clusters run at once.
template <typename K, typename A>
cudaError_t norm_res_launch(K kernel, const A& a, long long blocks, int threads, size_t smem, cudaStream_t s, int ranks = 1, int* active = nullptr) {
  if (smem > 40 * 1024) {   // (the static part counts too)
    // the most of any call, not this call's: the limit is the kernel's, and another host thread may launch it
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kNrSmem);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(blocks * ranks));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = ranks;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = ranks > 1;
  if (active) return cudaOccupancyMaxActiveClusters(active, kernel, &cfg);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

template <typename T, bool OWN>
cudaError_t norm_res_forward(const NormResArgs& a, const NormResShape& s, long long blocks, cudaStream_t st, int* active) {
  constexpr int W = sizeof(T) == 4 ? 2 : 1;   // units of eight elements
  const auto go = [&](auto kernel) { return norm_res_launch(kernel, a, blocks, s.threads, s.smem, st, s.ranks, active); };
  if (s.each == 8) return s.threads == 32 ? go(norm_res_kernel<T, W, OWN, 32>) : go(norm_res_kernel<T, W, OWN, 128>);
  if (s.each == 32) return go(norm_res_kernel<T, 4 * W, OWN, 512>);
  if (s.threads <= 128) return go(norm_res_kernel<T, 2 * W, OWN, 128>);
  if (s.more) return go(norm_res_kernel<T, 2 * W, OWN, 320>);
  return go(norm_res_kernel<T, 2 * W, OWN, 512>);
}
template <typename T, bool OWN>
cudaError_t norm_res_backward(const NormResGradArgs& a, const NormResShape& s, long long blocks, cudaStream_t st, int* active) {
  constexpr int W = sizeof(T) == 4 ? 2 : 1;
  const auto go = [&](auto kernel) { return norm_res_launch(kernel, a, blocks, s.threads, s.smem, st, s.ranks, active); };
  if (s.each == 8) return s.threads == 32 ? go(norm_res_grad_kernel<T, W, OWN, 32>) : go(norm_res_grad_kernel<T, W, OWN, 128>);
  if (s.threads <= 128) return go(norm_res_grad_kernel<T, 2 * W, OWN, 128>);
  return go(norm_res_grad_kernel<T, 2 * W, OWN, 512>);
}

}  // namespace
}  // namespace mg

using mg::op_fail;

static mg_status check_norm_res(const char* fn, int dtype, int rows, int dim, const float* gate, int gates, float scale) {
  if (dtype != 0 && dtype != 1) return op_fail(MG_ERR_INVALID_ARG, "%s: dtype must be 0 or 1", fn);
  if (rows < 0 || rows > mg::kMaxWidth || dim < 1 || dim > mg::kMaxWidth)
    return op_fail(MG_ERR_SHAPE, "%s: rows %d, dim %d", fn, rows, dim);
  if (gate ? gates < 1 || rows % gates || (rows && gates > rows) : gates != 0)
    return op_fail(MG_ERR_SHAPE, "%s: %d gates for %d rows (0 without a gate; else a divisor of the rows)", fn, gates, rows);
  if (!std::isfinite(scale)) return op_fail(MG_ERR_INVALID_ARG, "%s: scale must be finite", fn);
  return MG_OK;
}

extern "C" size_t mg_norm_residual_workspace_bytes(int rows, int dim, int gates) {
  if (rows < 0 || rows > mg::kMaxWidth || dim < 1 || dim > mg::kMaxWidth || gates < 0 || (gates && rows % gates)) return 0;
  return ((size_t)mg::norm_res_most_blocks(rows, dim, gates ? gates : 1) * 2 * dim + 4) * sizeof(float);
}

extern "C" mg_status mg_norm_residual_forward(int dtype, const void* y, const void* x, int rows, int dim,
                                              const float* gamma_post, const float* gate, int gates, float scale,
                                              const float* gamma_pre, float eps, void* x_out, void* h, float* rstd,
                                              mg_stream_t stream) {
  const char* fn = "mg_norm_residual_forward";
  mg_status st = check_norm_res(fn, dtype, rows, dim, gate, gates, scale);
  if (st != MG_OK) return st;
  if (!(eps > 0.0f) || !std::isfinite(eps)) return op_fail(MG_ERR_INVALID_ARG, "%s: eps must be positive and finite", fn);
  if (rows && (!y || !x || !x_out || !h != !gamma_pre))
    return op_fail(MG_ERR_INVALID_ARG, "%s: y, x and x_out must be non-NULL, and h and gamma_pre be given together", fn);
  st = mg::op_begin(fn, {{y, 16}, {x, 16}, {gamma_post, 16}, {gate, 16}, {gamma_pre, 16}, {x_out, 16}, {h, 16}, {rstd, 16}});
  if (st != MG_OK) return st;
  const size_t n = (size_t)rows * dim * (dtype ? 2 : 4), v = (size_t)dim * 4;
  st = mg::op_disjoint(fn, {{y, n, false, false}, {x, n, false, false}, {gamma_post, v, false, false}, {gate, gates * v, false, false},
                            {gamma_pre, v, false, false}, {x_out, n, true, x_out == y || x_out == x},
                            {h, n, true, h == y || h == x}, {rstd, (size_t)rows * 8, true, false}});
  if (st != MG_OK || !rows) return st;
  const mg::NormResShape shape = mg::norm_res_shape(dtype, rows, dim, false);
  mg::NormResArgs a = {y, x, gamma_post, gate, gamma_pre, rows, dim, gates ? rows / gates : rows, scale, eps, x_out, h, rstd, 1, mg::kNrStages, shape.row_units,
                       shape.ranks, shape.part};
  cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e;
  if (!shape.threads) {
    e = dtype ? mg::norm_res_launch(mg::norm_res_wide_kernel<mg::bf16>, a, rows, mg::kNrThreads, 0, s)
              : mg::norm_res_launch(mg::norm_res_wide_kernel<float>, a, rows, mg::kNrThreads, 0, s);
  } else {
    const auto go = [&](long long blocks, int* active) {
      if (dtype)
        return shape.own ? mg::norm_res_forward<mg::bf16, true>(a, shape, blocks, s, active)
                         : mg::norm_res_forward<mg::bf16, false>(a, shape, blocks, s, active);
      return shape.own ? mg::norm_res_forward<float, true>(a, shape, blocks, s, active)
                       : mg::norm_res_forward<float, false>(a, shape, blocks, s, active);
    };
    int slots = mg::norm_res_slots(shape), active = slots;
    e = shape.ranks > 1 ? go(slots, &active) : cudaSuccess;
    slots = mg::norm_res_clusters(slots, active);
    a.block_rows = (rows + slots - 1) / slots;
    if (e == cudaSuccess) e = go((rows + a.block_rows - 1) / a.block_rows, nullptr);
  }
  return mg::op_end(fn, e);
}

extern "C" mg_status mg_norm_residual_backward(int dtype, const void* dx_out, const void* dh, const void* y,
                                               const void* x, const float* rstd, int rows, int dim,
                                               const float* gamma_post, const float* gate, int gates, float scale,
                                               const float* gamma_pre, void* dy, void* dx, float* dgamma_post,
                                               float* dgate, float* dgamma_pre, void* workspace,
                                               size_t workspace_bytes, mg_stream_t stream) {
  const char* fn = "mg_norm_residual_backward";
  mg_status st = check_norm_res(fn, dtype, rows, dim, gate, gates, scale);
  if (st != MG_OK) return st;
  if ((rows && (!y || !x || !rstd || !dy || !dx || (!dx_out && !dh))) || !workspace)
    return op_fail(MG_ERR_INVALID_ARG, "%s: y, x, rstd, dy, dx, workspace and one of dx_out and dh must be non-NULL", fn);
  if ((dh && !gamma_pre) || (dgamma_pre && !gamma_pre) || (dgamma_post && !gamma_post) || (dgate && !gate))
    return op_fail(MG_ERR_INVALID_ARG, "%s: dh and each gradient of a vector need that vector", fn);
  const size_t need = mg_norm_residual_workspace_bytes(rows, dim, gates);
  if (workspace_bytes < need)
    return op_fail(MG_ERR_INVALID_ARG, "%s: the workspace needs %zu bytes, %zu given", fn, need, workspace_bytes);
  st = mg::op_begin(fn, {{dx_out, 16}, {dh, 16}, {y, 16}, {x, 16}, {rstd, 16}, {gamma_post, 16}, {gate, 16}, {gamma_pre, 16},
                         {dy, 16}, {dx, 16}, {dgamma_post, 16}, {dgate, 16}, {dgamma_pre, 16}, {workspace, 16}});
  if (st != MG_OK) return st;
  const size_t n = (size_t)rows * dim * (dtype ? 2 : 4), v = (size_t)dim * 4;
  const auto over = [&](const void* p) { return p == dx_out || p == dh || p == y || p == x; };
  st = mg::op_disjoint(fn, {{dx_out, n, false, false}, {dh, n, false, false}, {y, n, false, false}, {x, n, false, false},
                            {rstd, (size_t)rows * 8, false, false}, {gamma_post, v, false, false}, {gate, gates * v, false, false},
                            {gamma_pre, v, false, false}, {dy, n, true, over(dy)}, {dx, n, true, over(dx)},
                            {dgamma_post, v, true, false}, {dgate, gates * v, true, false}, {dgamma_pre, v, true, false},
                            {workspace, need, true, false}});
  if (st != MG_OK) return st;
  mg::NormResGradArgs a = {dx_out, dh, y, x, rstd, gamma_post, gate, gamma_pre, rows, dim, 0, gates ? gates : 1, scale,
                           dy, dx, dgamma_post, dgate, dgamma_pre, static_cast<float*>(workspace), 1, 1, 1, 0, 0, 1, dim};
  cudaStream_t s = (cudaStream_t)stream;
  if (!rows) {
    const long long blocks = ((long long)a.gates * dim + 255) / 256;
    return mg::op_end(fn, mg::norm_res_launch(mg::norm_res_zero_kernel, a, blocks, 256, 0, s));
  }
  a.gate_rows = rows / a.gates;
  const mg::NormResShape shape = mg::norm_res_shape(dtype, rows, dim, true);
  const auto go = [&](long long blocks, int* active) {
    if (dtype)
      return shape.own ? mg::norm_res_backward<mg::bf16, true>(a, shape, blocks, s, active)
                       : mg::norm_res_backward<mg::bf16, false>(a, shape, blocks, s, active);
    return shape.own ? mg::norm_res_backward<float, true>(a, shape, blocks, s, active)
                     : mg::norm_res_backward<float, false>(a, shape, blocks, s, active);
  };
  const int most = mg::norm_res_slots(shape);
  int active = most;
  cudaError_t e = shape.ranks > 1 ? go(most, &active) : cudaSuccess;
  if (e != cudaSuccess) return mg::op_end(fn, e);
  const mg::NormResSplit split = mg::norm_res_split(rows, a.gates, mg::norm_res_clusters(most, active));
  a.stages = mg::kNrStages;
  a.row_units = shape.row_units;
  a.ranks = shape.ranks;
  a.part = shape.part;
  a.parts = split.parts;
  a.block_rows = split.block_rows;
  a.block_gates = split.block_gates;
  if (!shape.threads)
    e = dtype ? mg::norm_res_launch(mg::norm_res_grad_wide_kernel<mg::bf16>, a, split.blocks, mg::kNrThreads, 0, s)
              : mg::norm_res_launch(mg::norm_res_grad_wide_kernel<float>, a, split.blocks, mg::kNrThreads, 0, s);
  else
    e = go(split.blocks, nullptr);
  const int gate_blocks = dgate && a.parts > 1 && a.gates > 1 ? std::min(a.gates, 65533) : 0;
  if (e == cudaSuccess && (dgamma_post || dgamma_pre || (dgate && a.parts > 1))) {
    // (many blocks: narrow rows; eight columns of a sector each, and four times the runs)
    const int wide = split.blocks > 1024 ? 8 : 32;
    const unsigned threads = 32 * (unsigned)std::max(4ll, std::min(32ll, split.blocks / 12));
    e = mg::launch_dependent(mg::norm_res_join_kernel, dim3((dim + wide - 1) / wide, 2 + gate_blocks), threads, 0, s, a,
                             (int)split.blocks, wide);
  }
  return mg::op_end(fn, e);
}

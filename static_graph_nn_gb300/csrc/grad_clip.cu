// Global norm of many gradient tensors, and clipping by it.
//
//   norm = sqrt(sum over all tensors of sum_i g_i^2)
//   c    = max_norm / norm if norm > max_norm, else 1   (1 if norm is NaN or infinite)
//   out  = c g
//
// The list is cut into chunks of at most 32 KB of one tensor; a block holds a
// whole chunk in registers, eight 16-byte loads a thread.
//
// Up to three chunks per SM (15 MB) all fit on chip at once: one cooperative
// launch reads every gradient once, meets at a grid barrier for the norm, and
// writes the scaled values from the registers.  This is bound by latency (one
// launch, one DRAM round trip, the barrier).
//
// Larger lists take two launches, the sum of squares and the scaling, and are
// bound by DRAM: 12 bytes per fp32 element (two reads and a write; 334M
// elements in 586 us, 6.8 TB/s).  The second pass walks the chunks backwards, so
// that what the first one read last is still in L2, and is a dependent launch
// that loads its chunks before the norm is there.
//
// Sums: a thread squares and adds 32 elements at a time in fp32 (eight running
// sums of four) and adds that to an fp64 total, so that the error does not
// grow with the count; should an fp32 sum leave the range in which squares
// neither overflow nor lose bits to underflow, those elements are summed again
// in fp64 from registers.  Every block writes its total to its own slot and the
// slots are added in order: no atomic order enters the result.
#include <algorithm>
#include <cmath>
#include <cstdio>
#include <cstdlib>
#include <exception>
#include <iterator>
#include <memory>
#include <new>
#include <utility>
#include <vector>

#include "../../include/mg.h"
#include "common.cuh"
#include "kernels.h"
#include "op_checks.h"

namespace mg {
namespace {

constexpr int kClipThreads = 256;
constexpr int kClipVecs = 8;                                      // 16-byte loads a thread and chunk
constexpr int kClipBytes = kClipThreads * kClipVecs * 16;         // 32 KB
constexpr int kClipFusedPerSm = 3;   // resident blocks that hold a chunk each (84 registers a thread)
constexpr unsigned kClipSpin = 1u << 22;                          // bounded barrier wait

struct ClipChunk {
  const void* g;
  void* out;
  int len;
  int flags;   // bit 0: bf16, bit 1: g and out allow 16-byte accesses
};

struct ClipSync {
  unsigned long long calls;     // fused calls finished
  unsigned last;                // blocks that have written their partial sum (two-pass calls)
  unsigned failed;              // 1 from the first fused call on in which a block gave up waiting
};

// A block's sum with the number of the call it belongs to, written and read as
// one 16-byte word: a reader that finds its call's number has the sum.
struct alignas(16) ClipSum {
  double sum;
  unsigned long long call;
};
__device__ __forceinline__ void put_sum(ClipSum* p, double sum, unsigned long long call) {
  asm volatile("{\n.reg .b128 v;\nmov.b128 v, {%1, %2};\nst.relaxed.gpu.global.b128 [%0], v;\n}\n" ::"l"(p),
               "l"(__double_as_longlong(sum)), "l"(call)
               : "memory");
}
__device__ __forceinline__ bool get_sum(const ClipSum* p, unsigned long long call, double& sum) {
  long long lo;
  unsigned long long hi;
  asm volatile("{\n.reg .b128 v;\nld.relaxed.gpu.global.b128 v, [%2];\nmov.b128 {%0, %1}, v;\n}\n"
               : "=l"(lo), "=l"(hi)
               : "l"(p)
               : "memory");
  sum = __longlong_as_double(lo);
  return hi == call;
}

__device__ __forceinline__ double block_sum_f64(double v, double* red /* 32 */) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, nw = blockDim.x >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if (lane == 0) red[w] = v;
  __syncthreads();
  double t = lane < nw ? red[lane] : 0.0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
  return t;
}

// Sum of the squares of N values held in registers.
template <int N>
__device__ __forceinline__ double squares(const float (&x)[N]) {
  float s[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < N; ++i) s[i & 7] = fmaf(x[i], x[i], s[i & 7]);
  const float t = ((s[0] + s[1]) + (s[2] + s[3])) + ((s[4] + s[5]) + (s[6] + s[7]));
  // inside this range the largest square neither overflows nor is a value
  // whose neighbours' squares underflow by more than 2^-24 of the sum
  if (t < 1e37f && t > 1e-25f) return (double)t;
  if (t == 0.0f) {
    bool any = false;
#pragma unroll
    for (int i = 0; i < N; ++i) any = any || x[i] != 0.0f;
    if (!any) return 0.0;
  }
  double d = 0.0;
#pragma unroll
  for (int i = 0; i < N; ++i) d += (double)x[i] * (double)x[i];
  return d;
}

__device__ __forceinline__ void widen_bf16(const uint4& u, float* f) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

// A thread's part of a chunk: kClipVecs vectors of 16 bytes, a block's width
// apart; zeros behind the chunk's last whole vector.
struct ClipData {
  uint4 u[kClipVecs];
  __device__ __forceinline__ void load(const ClipChunk& c) {
    const int nv = c.flags & 2 ? c.len / (c.flags & 1 ? 8 : 4) : 0;
    const uint4* p = static_cast<const uint4*>(c.g);
#pragma unroll
    for (int q = 0; q < kClipVecs; ++q) {
      const int i = threadIdx.x + q * kClipThreads;
      u[q] = i < nv ? p[i] : make_uint4(0, 0, 0, 0);
    }
  }
  __device__ __forceinline__ double sum(const ClipChunk& c) const {
    double t = 0.0;
    if (c.flags & 1) {
#pragma unroll
      for (int q = 0; q < kClipVecs; q += 4) {
        float x[32];
#pragma unroll
        for (int j = 0; j < 4; ++j) widen_bf16(u[q + j], x + 8 * j);
        t += squares<32>(x);
      }
    } else {
      float x[32];
#pragma unroll
      for (int q = 0; q < kClipVecs; ++q) {
        x[4 * q] = __uint_as_float(u[q].x);
        x[4 * q + 1] = __uint_as_float(u[q].y);
        x[4 * q + 2] = __uint_as_float(u[q].z);
        x[4 * q + 3] = __uint_as_float(u[q].w);
      }
      t = squares<32>(x);
    }
    return t;
  }
  // c = 1 stores the bits as they are (a NaN keeps its payload)
  __device__ __forceinline__ void store(const ClipChunk& c, float f) const {
    const int nv = c.flags & 2 ? c.len / (c.flags & 1 ? 8 : 4) : 0;
    uint4* p = static_cast<uint4*>(c.out);
#pragma unroll
    for (int q = 0; q < kClipVecs; ++q) {
      const int i = threadIdx.x + q * kClipThreads;
      if (i >= nv) continue;
      uint4 v = u[q];
      if (f != 1.0f) {
        uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (c.flags & 1) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(__uint_as_float(w[j] << 16) * f,
                                                           __uint_as_float(w[j] & 0xffff0000u) * f);
            w[j] = *reinterpret_cast<const uint32_t*>(&h);
          } else {
            w[j] = __float_as_uint(__uint_as_float(w[j]) * f);
          }
        }
        v = make_uint4(w[0], w[1], w[2], w[3]);
      }
      __stcs(p + i, v);
    }
  }
};

// Elements outside the whole vectors: a chunk's tail, or all of an unaligned one.
template <typename F>
__device__ __forceinline__ void clip_rest(const ClipChunk& c, F&& f) {
  const int done = c.flags & 2 ? (c.flags & 1 ? c.len & ~7 : c.len & ~3) : 0;
  for (int i = done + threadIdx.x; i < c.len; i += kClipThreads) f(i);
}

__device__ __forceinline__ double chunk_squares(const ClipChunk& c, const ClipData& d) {
  double t = d.sum(c);
  clip_rest(c, [&](int i) {
    const float x[1] = {c.flags & 1 ? ld_elem(static_cast<const bf16*>(c.g), i)
                                    : ld_elem(static_cast<const float*>(c.g), i)};
    t += squares<1>(x);
  });
  return t;
}

__device__ __forceinline__ void chunk_store(const ClipChunk& c, const ClipData& d, float f) {
  d.store(c, f);
  clip_rest(c, [&](int i) {
    if (c.flags & 1) {
      const bf16 x = static_cast<const bf16*>(c.g)[i];
      static_cast<bf16*>(c.out)[i] = f == 1.0f ? x : __float2bfloat16_rn(__bfloat162float(x) * f);
    } else {
      const uint32_t x = static_cast<const uint32_t*>(c.g)[i];
      static_cast<uint32_t*>(c.out)[i] = f == 1.0f ? x : __float_as_uint(__uint_as_float(x) * f);
    }
  });
}

// The norm and the factor.
__device__ __forceinline__ float2 clip_factor(double sum, float max_norm) {
  const double norm = sqrt(sum);
  const bool finite = norm - norm == 0.0;
  return make_float2((float)norm, finite && norm > (double)max_norm ? (float)((double)max_norm / norm) : 1.0f);
}

// The same from the blocks' sums, added in order by one block.
__device__ __forceinline__ float2 clip_finish(const double* partial, int n, float max_norm, double* red) {
  double s = 0.0;
  for (int i = threadIdx.x; i < n; i += kClipThreads) s += __ldcg(partial + i);
  return clip_factor(block_sum_f64(s, red), max_norm);
}

// One chunk per block, all blocks resident (cooperative launch).  The barrier is
// the exchange of the sums itself: every block waits for every block's sum of
// this call and adds them in the same order.
//
// Block 0 writes the statistics, and a block that gave up waiting (its chunk is
// not written) makes them NaN, whichever comes first: the one sets the mark
// `failed`, fences and writes NaN; the other writes the numbers, fences and
// looks at the mark.  Of two such fences one is first: either block 0 sees the
// mark, or the NaN come after its numbers.  The mark stays: a block that began
// late may have left a sum under the next call's number.  (A count of the blocks that leave,
// with the last one writing, cost 231 atomics on one word: 14.4 -> 16.3 us for the MLP.)
__global__ void __launch_bounds__(kClipThreads, kClipFusedPerSm)
    clip_fused_kernel(const ClipChunk* chunks, ClipSum* sums, ClipSync* sync, float max_norm, float* stats,
                      unsigned spin_limit) {
  __shared__ double red[32];
  __shared__ unsigned long long s_call;
  const ClipChunk c = chunks[blockIdx.x];
  // one thread reads the number of calls and passes it on with the block's sum:
  // block 0, which writes the next number, does so with every block's sum at hand
  if (threadIdx.x == 0) s_call = *reinterpret_cast<volatile unsigned long long*>(&sync->calls) + 1;
  ClipData d;
  d.load(c);
  const double t = block_sum_f64(chunk_squares(c, d), red);
  const unsigned long long call = s_call;
  if (threadIdx.x == 0) put_sum(sums + blockIdx.x, t, call);
  double s = 0.0;
  bool ok = true;
  for (int i = threadIdx.x; i < (int)gridDim.x; i += kClipThreads) {
    double v;
    unsigned spin = 0;
    while (!get_sum(sums + i, call, v) && ++spin < spin_limit) {}
    ok = ok && spin < spin_limit;
    s += v;
  }
  ok = __syncthreads_and(ok);
  const float2 r = clip_factor(block_sum_f64(s, red), max_norm);
  if (threadIdx.x == 0 && (blockIdx.x == 0 || !ok)) {
    const float nan = __int_as_float(0x7fffffff);
    volatile unsigned* failed = &sync->failed;
    volatile float* st = stats;
    if (!ok) *failed = 1;
    st[0] = ok ? r.x : nan;
    st[1] = ok ? r.y : nan;
    asm volatile("fence.sc.gpu;" ::: "memory");
    if (*failed) st[0] = st[1] = nan;
    if (blockIdx.x == 0) sync->calls = call;   // each sum carries the number that its block's one reader read
  }
  if (ok && (r.y != 1.0f || c.out != c.g)) chunk_store(c, d, r.y);
}

__global__ void __launch_bounds__(kClipThreads, 4) clip_norm_kernel(const ClipChunk* chunks, int n_chunks,
                                                                    double* partial, ClipSync* sync,
                                                                    float max_norm, float* stats) {
  __shared__ double red[32];
  __shared__ bool last;
  double t = 0.0;
  dependents_start();        // the scaling blocks load their chunks as these leave
  ClipChunk next;
  if ((int)blockIdx.x < n_chunks) next = chunks[blockIdx.x];
  for (int i = blockIdx.x; i < n_chunks; i += gridDim.x) {
    const ClipChunk c = next;
    ClipData d;
    d.load(c);
    if (i + (int)gridDim.x < n_chunks) next = chunks[i + gridDim.x];
    t += chunk_squares(c, d);
  }
  t = block_sum_f64(t, red);
  if (threadIdx.x == 0) {
    partial[blockIdx.x] = t;
    __threadfence();
    last = atomicAdd(&sync->last, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  const float2 r = clip_finish(partial, gridDim.x, max_norm, red);
  if (threadIdx.x == 0) {
    stats[0] = r.x;
    stats[1] = r.y;
    sync->last = 0;   // for the next call
  }
}

__global__ void __launch_bounds__(kClipThreads, 4) clip_scale_kernel(const ClipChunk* chunks, int n_chunks,
                                                                     const float* stats) {
  const ClipChunk c = chunks[n_chunks - 1 - (int)blockIdx.x];
  ClipData d;
  d.load(c);           // in flight while the norm is finished
  dependency_wait();   // the norm is there, and every gradient has been read
  const float f = stats[1];
  if (f == 1.0f && c.out == c.g) return;
  chunk_store(c, d, f);
}

// ---- inside a training step: the flat gradient buffer's chunk table
__global__ void __launch_bounds__(kClipThreads) grad_squares_kernel(const Chunk* chunks, const float* g, double* sums) {
  __shared__ double red[32];
  const Chunk c = chunks[blockIdx.x];
  const float4* g4 = reinterpret_cast<const float4*>(g + c.start);
  double t = 0.0;
  for (int b = 0; b < c.len / 4; b += 2 * kClipThreads) {
    float4 v[2];
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int i = b + q * kClipThreads + threadIdx.x;
      v[q] = i < c.len / 4 ? g4[i] : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    const float x[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
    t += squares<8>(x);
  }
  const int i = (c.len & ~3) + threadIdx.x;
  if (i < c.len) {
    const float x[1] = {g[c.start + i]};
    t += squares<1>(x);
  }
  t = block_sum_f64(t, red);
  if (threadIdx.x == 0) sums[blockIdx.x] = t;
}

__global__ void __launch_bounds__(kClipThreads) grad_norm_kernel(const double* sums, int n, double* parts,
                                                                 unsigned* sync, float max_norm, float* stats) {
  __shared__ double red[32];
  __shared__ bool last;
  double t = 0.0;
  for (int i = blockIdx.x * kClipThreads + threadIdx.x; i < n; i += gridDim.x * kClipThreads) t += sums[i];
  t = block_sum_f64(t, red);
  if (threadIdx.x == 0) {
    parts[blockIdx.x] = t;
    __threadfence();
    last = atomicAdd(sync, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  const float2 r = clip_finish(parts, gridDim.x, max_norm, red);
  if (threadIdx.x == 0) {
    stats[0] = r.x;
    stats[1] = r.y;
    *sync = 0;
  }
}

}  // namespace

cudaError_t grad_squares(const Chunk* chunks, int n_chunks, const float* g, double* sums, cudaStream_t s) {
  if (n_chunks <= 0) return cudaSuccess;
  grad_squares_kernel<<<n_chunks, kClipThreads, 0, s>>>(chunks, g, sums);
  return cudaGetLastError();
}

cudaError_t grad_norm_finish(const double* sums, int n_chunks, double* parts, unsigned* sync, float max_norm,
                             float* stats, cudaStream_t s) {
  int grid = (n_chunks + kClipThreads - 1) / kClipThreads;
  grid = grid < 1 ? 1 : grid > kNormParts ? kNormParts : grid;
  grad_norm_kernel<<<grid, kClipThreads, 0, s>>>(sums, n_chunks, parts, sync, max_norm, stats);
  return cudaGetLastError();
}

}  // namespace mg

struct mg_grad_list {
  int device = 0;
  int n_chunks = 0;
  char* ws = nullptr;   // chunk table, partial sums, arrival counter
  size_t partial_off = 0, sync_off = 0;
  int sms = 0;
  bool fused = false;   // all chunks resident at once: one launch
  // the tensors' memory: begins in ascending order, and the largest end up to each
  std::vector<std::pair<uintptr_t, uintptr_t>> memory;
  unsigned spin = mg::kClipSpin;
};

using mg::op_fail;

static constexpr size_t kMaxChunks = 1u << 26;   // of a list: 2 TB of gradients, before the host allocates for them

extern "C" mg_status mg_grad_list_create(int n, const void* const* grads, void* const* out, const size_t* counts,
                                         const int* dtypes, mg_grad_list** list) {
  const char* fn = "mg_grad_list_create";
  if (!list) return op_fail(MG_ERR_INVALID_ARG, "%s: list is NULL", fn);
  *list = nullptr;
  if (n < 1 || !grads || !counts || !dtypes)
    return op_fail(MG_ERR_INVALID_ARG, "%s: n must be positive and grads, counts, dtypes non-NULL", fn);
  try {
    struct Span {
      uintptr_t lo, hi;
      int tensor;
      bool written;
    };
    std::vector<Span> spans;
    std::vector<mg::ClipChunk> table;
    for (int i = 0; i < n; ++i) {
      if (dtypes[i] != 0 && dtypes[i] != 1)
        return op_fail(MG_ERR_INVALID_ARG, "%s: dtype of tensor %d must be 0 or 1", fn, i);
      const size_t es = dtypes[i] ? 2 : 4;
      if (counts[i] == 0) continue;
      const char* g = static_cast<const char*>(grads[i]);
      char* o = out ? static_cast<char*>(out[i]) : const_cast<char*>(g);
      if (!g || !o) return op_fail(MG_ERR_INVALID_ARG, "%s: tensor %d is NULL", fn, i);
      const size_t step = mg::kClipBytes / es;
      if (counts[i] / step + table.size() > kMaxChunks)
        return op_fail(MG_ERR_SHAPE, "%s: tensor %d has %zu elements, too many", fn, i, counts[i]);
      mg_status st = mg::op_begin(fn, {{g, (unsigned)es}, {o, (unsigned)es}});
      if (st != MG_OK) return st;
      const uintptr_t gl = reinterpret_cast<uintptr_t>(g), ol = reinterpret_cast<uintptr_t>(o);
      const size_t bytes = counts[i] * es;
      if (gl != ol) spans.push_back({gl, gl + bytes, i, false});
      spans.push_back({ol, ol + bytes, i, true});
      const int flags = dtypes[i] | (gl % 16 == 0 && ol % 16 == 0 ? 2 : 0);
      for (size_t a = 0; a < counts[i]; a += step)
        table.push_back({g + a * es, o + a * es, (int)std::min<size_t>(step, counts[i] - a), flags});
    }
    // a written range may meet no other range (the same tensor twice, or an
    // output inside another tensor, would be scaled twice or read half scaled)
    std::sort(spans.begin(), spans.end(), [](const Span& a, const Span& b) { return a.lo < b.lo; });
    uintptr_t hi = 0, whi = 0;
    int ht = -1, wt = -1;
    for (const Span& s : spans) {
      if (s.lo < whi || (s.written && s.lo < hi))
        return op_fail(MG_ERR_INVALID_ARG, "%s: tensors %d and %d overlap in memory that is written", fn,
                       s.lo < whi ? wt : ht, s.tensor);
      if (s.hi > hi) { hi = s.hi; ht = s.tensor; }
      if (s.written && s.hi > whi) { whi = s.hi; wt = s.tensor; }
    }
    std::unique_ptr<mg_grad_list> l(new mg_grad_list());
    for (const Span& s : spans)
      l->memory.emplace_back(s.lo, std::max(s.hi, l->memory.empty() ? 0 : l->memory.back().second));
    l->n_chunks = (int)table.size();
    cudaError_t e = cudaGetDevice(&l->device);
    int coop = 0, per_sm = 0;
    l->sms = mg::device_sms();
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&coop, cudaDevAttrCooperativeLaunch, l->device);
    if (e == cudaSuccess)
      e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, mg::clip_fused_kernel, mg::kClipThreads, 0);
    if (const char* ev = getenv("MG_CLIP_WAIT"))
      if (const int v = atoi(ev); v > 0) l->spin = (unsigned)v;
    l->fused = coop && l->n_chunks > 0 && l->n_chunks <= l->sms * std::min(per_sm, mg::kClipFusedPerSm);
    const size_t blocks = std::max<size_t>(l->fused ? table.size() : 1, (size_t)l->sms * 4);
    l->partial_off = (table.size() * sizeof(mg::ClipChunk) + 255) / 256 * 256;
    l->sync_off = l->partial_off + blocks * sizeof(mg::ClipSum);
    const size_t bytes = l->sync_off + sizeof(mg::ClipSync);
    if (e == cudaSuccess) e = cudaMalloc((void**)&l->ws, bytes);
    if (e != cudaSuccess) {
      cudaGetLastError();
      return op_fail(e == cudaErrorMemoryAllocation ? MG_ERR_OOM : MG_ERR_CUDA, "%s: %zu bytes: %s", fn, bytes,
                     cudaGetErrorString(e));
    }
    if (!table.empty())
      e = cudaMemcpy(l->ws, table.data(), table.size() * sizeof(mg::ClipChunk), cudaMemcpyHostToDevice);
    if (e == cudaSuccess) e = cudaMemset(l->ws + l->partial_off, 0, bytes - l->partial_off);
    // both may still be on their way, and a caller's stream need not wait for
    // the default one
    if (e == cudaSuccess) e = cudaStreamSynchronize(nullptr);
    if (e != cudaSuccess) {
      cudaFree(l->ws);
      return mg::op_end(fn, e);
    }
    *list = l.release();
    return MG_OK;
  } catch (const std::exception&) {   // of the vectors: no exception leaves a C entry
    return op_fail(MG_ERR_OOM, "%s: host allocation failed", fn);
  }
}

extern "C" void mg_grad_list_destroy(mg_grad_list* l) {
  if (!l) return;
  int prev = -1;
  cudaGetDevice(&prev);
  cudaSetDevice(l->device);
  cudaFree(l->ws);   // waits for the device
  if (prev >= 0) cudaSetDevice(prev);
  delete l;
}

extern "C" mg_status mg_grad_list_clip(mg_grad_list* l, float max_norm, float* stats, mg_stream_t stream) {
  const char* fn = "mg_grad_list_clip";
  if (!l || !stats) return op_fail(MG_ERR_INVALID_ARG, "%s: list and stats must be non-NULL", fn);
  if (!(max_norm >= 0.0f)) return op_fail(MG_ERR_INVALID_ARG, "%s: max_norm must be at least 0", fn);
  int dev = -1;
  if (cudaGetDevice(&dev) == cudaSuccess && dev != l->device)
    return op_fail(MG_ERR_INVALID_ARG, "%s: the list belongs to device %d but device %d is current", fn, l->device, dev);
  mg_status st = mg::op_begin(fn, {{stats, 8}});
  if (st != MG_OK) return st;
  const uintptr_t at = reinterpret_cast<uintptr_t>(stats);
  const auto behind = std::lower_bound(l->memory.begin(), l->memory.end(), std::make_pair(at + 8, (uintptr_t)0));
  if (behind != l->memory.begin() && std::prev(behind)->second > at)
    return op_fail(MG_ERR_INVALID_ARG, "%s: stats lies in a tensor of the list", fn);
  cudaStream_t s = (cudaStream_t)stream;
  const auto* chunks = reinterpret_cast<const mg::ClipChunk*>(l->ws);
  mg::ClipSync* sync = reinterpret_cast<mg::ClipSync*>(l->ws + l->sync_off);
  cudaError_t e;
  if (l->fused) {
    mg::ClipSum* sums = reinterpret_cast<mg::ClipSum*>(l->ws + l->partial_off);
    void* args[] = {&chunks, &sums, &sync, &max_norm, &stats, &l->spin};
    e = cudaLaunchCooperativeKernel(reinterpret_cast<const void*>(mg::clip_fused_kernel), dim3(l->n_chunks),
                                    dim3(mg::kClipThreads), args, 0, s);
    return mg::op_end(fn, e);
  }
  double* partial = reinterpret_cast<double*>(l->ws + l->partial_off);
  const int blocks = std::max(1, std::min(l->n_chunks, 4 * l->sms));
  mg::clip_norm_kernel<<<blocks, mg::kClipThreads, 0, s>>>(chunks, l->n_chunks, partial, sync, max_norm, stats);
  e = cudaGetLastError();
  if (e == cudaSuccess && l->n_chunks) {
    e = mg::launch_dependent(mg::clip_scale_kernel, l->n_chunks, mg::kClipThreads, 0, s, chunks, l->n_chunks, stats);
  }
  return mg::op_end(fn, e);
}

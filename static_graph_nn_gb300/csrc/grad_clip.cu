// Global norm of many gradient tensors, and clipping by it.
//
//   norm = sqrt(sum over all tensors of sum_i g_i^2)
//   c    = max_norm / norm if norm > max_norm, else 1   (1 if norm is NaN or infinite)
//   out  = c g
//
// Two passes over a table of chunks (runs of at most kClipChunk elements of
// one tensor): the first sums squares, the second scales.  Both are bound by
// memory; the second pass reads what the first read last, walking the table
// backwards, so that the part of the gradients still in L2 is not read from
// DRAM again.
//
// Sums: a thread squares and adds 32 elements at a time in fp32 and adds that
// to an fp64 total, so that the error does not grow with the count; should an
// fp32 sum leave the range in which squares neither overflow nor lose bits to
// underflow, those 32 elements are summed again in fp64 from registers.  Every
// block writes its total to its own slot and the block that finishes last adds
// the slots in order: no atomic order enters the result.
#include <algorithm>
#include <cmath>
#include <cstdio>
#include <memory>
#include <new>
#include <vector>

#include "../../include/mg.h"
#include "common.cuh"
#include "kernels.h"
#include "op_checks.h"

namespace mg {
namespace {

constexpr int kClipChunk = 16384;
constexpr int kClipThreads = 256;

struct ClipChunk {
  const void* g;
  void* out;
  int len;
  int flags;   // bit 0: bf16, bit 1: g and out allow 16-byte accesses
};

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
  float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < N; ++i) s[i & 3] = fmaf(x[i], x[i], s[i & 3]);
  const float t = (s[0] + s[1]) + (s[2] + s[3]);
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

template <typename T>
__device__ __forceinline__ void load16(const T* p, float* f);
template <>
__device__ __forceinline__ void load16<float>(const float* p, float* f) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const float4 v = reinterpret_cast<const float4*>(p)[q];
    f[4 * q] = v.x; f[4 * q + 1] = v.y; f[4 * q + 2] = v.z; f[4 * q + 3] = v.w;
  }
}
template <>
__device__ __forceinline__ void load16<bf16>(const bf16* p, float* f) {
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const uint4 u = reinterpret_cast<const uint4*>(p)[q];
    const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&u);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 t = __bfloat1622float2(h[i]);
      f[8 * q + 2 * i] = t.x;
      f[8 * q + 2 * i + 1] = t.y;
    }
  }
}

template <typename T>
__device__ __forceinline__ double chunk_squares(const T* g, int len, bool vec) {
  double total = 0.0;
  const int step = kClipThreads * 16;
  int done = 0;
  if (vec) {
    for (int b = threadIdx.x * 16; b + 16 <= len; b += step) {
      float x[16];
      load16<T>(g + b, x);
      total += squares<16>(x);
    }
    done = len & ~15;
  }
  for (int i = done + threadIdx.x; i < len; i += kClipThreads) {
    float x[1] = {ld_elem(g, i)};
    total += squares<1>(x);
  }
  return total;
}

__global__ void __launch_bounds__(kClipThreads) clip_norm_kernel(const ClipChunk* chunks, int n_chunks,
                                                                 double* partial, unsigned* arrivals,
                                                                 float max_norm, float* stats) {
  __shared__ double red[32];
  __shared__ bool last;
  double t = 0.0;
  if ((int)blockIdx.x < n_chunks) {
    const ClipChunk c = chunks[blockIdx.x];
    t = c.flags & 1 ? chunk_squares(static_cast<const bf16*>(c.g), c.len, c.flags & 2)
                    : chunk_squares(static_cast<const float*>(c.g), c.len, c.flags & 2);
  }
  t = block_sum_f64(t, red);
  if (threadIdx.x == 0) {
    partial[blockIdx.x] = t;
    __threadfence();
    last = atomicAdd(arrivals, 1u) == gridDim.x - 1;
  }
  __syncthreads();
  if (!last) return;
  __threadfence();
  double s = 0.0;
  for (int i = threadIdx.x; i < (int)gridDim.x; i += kClipThreads) s += __ldcg(partial + i);
  s = block_sum_f64(s, red);
  if (threadIdx.x == 0) {
    const double norm = sqrt(s);
    const bool finite = norm - norm == 0.0;
    stats[0] = (float)norm;
    stats[1] = finite && norm > (double)max_norm ? (float)((double)max_norm / norm) : 1.0f;
    *arrivals = 0;   // for the next call
  }
}

template <typename T>
__device__ __forceinline__ void chunk_scale(const T* g, T* out, int len, bool vec, float c) {
  const int step = kClipThreads * 16;
  int done = 0;
  if (vec) {
    for (int b = threadIdx.x * 16; b + 16 <= len; b += step) {
      float x[16];
      load16<T>(g + b, x);
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] *= c;
      if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          reinterpret_cast<float4*>(out + b)[q] = make_float4(x[4 * q], x[4 * q + 1], x[4 * q + 2], x[4 * q + 3]);
      } else {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 h = __floats2bfloat162_rn(x[8 * q + 2 * i], x[8 * q + 2 * i + 1]);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
          }
          reinterpret_cast<uint4*>(out + b)[q] = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
    }
    done = len & ~15;
  }
  for (int i = done + threadIdx.x; i < len; i += kClipThreads) st_elem(out, i, ld_elem(g, i) * c);
}

// c = 1: the bits as they are (a NaN keeps its payload).
template <typename W>
__device__ __forceinline__ void chunk_copy(const W* g, W* out, int len, bool vec) {
  constexpr int N = 16 / sizeof(W);
  int done = 0;
  if (vec) {
    for (int b = threadIdx.x; b < len / N; b += kClipThreads)
      reinterpret_cast<uint4*>(out)[b] = reinterpret_cast<const uint4*>(g)[b];
    done = len / N * N;
  }
  for (int i = done + threadIdx.x; i < len; i += kClipThreads) out[i] = g[i];
}

__global__ void __launch_bounds__(kClipThreads) clip_scale_kernel(const ClipChunk* chunks, int n_chunks,
                                                                  const float* stats) {
  const float c = stats[1];
  const ClipChunk k = chunks[n_chunks - 1 - (int)blockIdx.x];
  if (c == 1.0f) {
    if (k.out == k.g) return;
    if (k.flags & 1)
      chunk_copy(static_cast<const uint16_t*>(k.g), static_cast<uint16_t*>(k.out), k.len, k.flags & 2);
    else
      chunk_copy(static_cast<const uint32_t*>(k.g), static_cast<uint32_t*>(k.out), k.len, k.flags & 2);
    return;
  }
  if (k.flags & 1)
    chunk_scale(static_cast<const bf16*>(k.g), static_cast<bf16*>(k.out), k.len, k.flags & 2, c);
  else
    chunk_scale(static_cast<const float*>(k.g), static_cast<float*>(k.out), k.len, k.flags & 2, c);
}

}  // namespace
}  // namespace mg

struct mg_grad_list {
  int device = 0;
  int n_chunks = 0;
  char* ws = nullptr;   // chunk table, partial sums, arrival counter
  size_t partial_off = 0, arrivals_off = 0;
};

using mg::op_fail;

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
      if (counts[i] > (size_t)1 << 46) return op_fail(MG_ERR_SHAPE, "%s: tensor %d has %zu elements", fn, i, counts[i]);
      mg_status st = mg::op_begin(fn, {{g, (unsigned)es}, {o, (unsigned)es}});
      if (st != MG_OK) return st;
      const uintptr_t gl = reinterpret_cast<uintptr_t>(g), ol = reinterpret_cast<uintptr_t>(o);
      const size_t bytes = counts[i] * es;
      if (gl != ol) spans.push_back({gl, gl + bytes, i, false});
      spans.push_back({ol, ol + bytes, i, true});
      const int flags = dtypes[i] | (gl % 16 == 0 && ol % 16 == 0 ? 2 : 0);
      for (size_t a = 0; a < counts[i]; a += mg::kClipChunk)
        table.push_back({g + a * es, o + a * es, (int)std::min<size_t>(mg::kClipChunk, counts[i] - a), flags});
    }
    if (table.size() > 0x7ffffff0u) return op_fail(MG_ERR_SHAPE, "%s: too many elements", fn);
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
    l->n_chunks = (int)table.size();
    cudaError_t e = cudaGetDevice(&l->device);
    const size_t blocks = std::max<size_t>(1, table.size());
    l->partial_off = (table.size() * sizeof(mg::ClipChunk) + 255) / 256 * 256;
    l->arrivals_off = l->partial_off + blocks * sizeof(double);
    const size_t bytes = l->arrivals_off + 16;
    if (e == cudaSuccess) e = cudaMalloc((void**)&l->ws, bytes);
    if (e != cudaSuccess) {
      cudaGetLastError();
      return op_fail(e == cudaErrorMemoryAllocation ? MG_ERR_OOM : MG_ERR_CUDA, "%s: %zu bytes: %s", fn, bytes,
                     cudaGetErrorString(e));
    }
    if (!table.empty())
      e = cudaMemcpy(l->ws, table.data(), table.size() * sizeof(mg::ClipChunk), cudaMemcpyHostToDevice);
    if (e == cudaSuccess) e = cudaMemset(l->ws + l->arrivals_off, 0, 16);
    if (e != cudaSuccess) {
      cudaFree(l->ws);
      return mg::op_end(fn, e);
    }
    *list = l.release();
    return MG_OK;
  } catch (const std::bad_alloc&) {
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
  cudaStream_t s = (cudaStream_t)stream;
  const auto* chunks = reinterpret_cast<const mg::ClipChunk*>(l->ws);
  const int blocks = std::max(1, l->n_chunks);
  mg::clip_norm_kernel<<<blocks, mg::kClipThreads, 0, s>>>(
      chunks, l->n_chunks, reinterpret_cast<double*>(l->ws + l->partial_off),
      reinterpret_cast<unsigned*>(l->ws + l->arrivals_off), max_norm, stats);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess && l->n_chunks) {
    mg::clip_scale_kernel<<<l->n_chunks, mg::kClipThreads, 0, s>>>(chunks, l->n_chunks, stats);
    e = cudaGetLastError();
  }
  return mg::op_end(fn, e);
}

// Log probabilities of given tokens, the entropy of each row's distribution and
// its most likely tokens, and their gradient.
//
// With z = x / T over a row x of logits, m = max x and L = log sum exp((x - m) / T):
//   logp    = (x[id] - m) / T - L
//   entropy = L - sum_v p_v (x_v - m) / T        p_v = exp((x_v - m) / T - L)
//   dx_v    = (g (1[v = id] - p_v) - h p_v (log p_v + entropy)) / T
#include <cmath>

#include "common.cuh"
#include "kernels.h"
#include "op_checks.h"

namespace mg {
namespace {

constexpr int kLogpThreads = 256;

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

__device__ __forceinline__ unsigned long long block_max_u64(unsigned long long v, unsigned long long* red) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, nw = blockDim.x >> 5;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const unsigned long long t = __shfl_xor_sync(0xffffffffu, v, o);
    v = t > v ? t : v;
  }
  __syncthreads();
  if (lane == 0) red[w] = v;
  __syncthreads();
  v = lane < nw ? red[lane] : 0;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const unsigned long long t = __shfl_xor_sync(0xffffffffu, v, o);
    v = t > v ? t : v;
  }
  return v;
}

// A row per block.
template <typename T>
__global__ void __launch_bounds__(kLogpThreads) logp_kernel(LogpArgs a) {
  __shared__ float red[32];
  __shared__ unsigned long long red64[32];
  const size_t r = blockIdx.x;
  const T* x = static_cast<const T*>(a.logits) + r * a.stride;
  const int id = a.ids ? token_of(a.ids, a.id64, a.vocab, r) : 0;
  if (id < 0) {
    if (threadIdx.x == 0) {
      a.logp[r] = 0.0f;
      if (a.stats) a.stats[2 * r] = a.stats[2 * r + 1] = 0.0f;
      if (a.entropy) a.entropy[r] = 0.0f;
    }
    for (int i = threadIdx.x; i < a.k; i += kLogpThreads) {
      a.top_ids[r * a.k + i] = -1;
      a.top_logp[r * a.k + i] = 0.0f;
    }
    return;
  }
  float m = -INFINITY;
  for (int c = threadIdx.x; c < a.vocab; c += kLogpThreads) m = fmaxf(m, ld_elem(x, c));
  m = block_max(m, red);
  const float mm = m == -INFINITY ? 0.0f : m;
  float s = 0.0f, q = 0.0f;
  for (int c = threadIdx.x; c < a.vocab; c += kLogpThreads) {
    const float t = (ld_elem(x, c) - mm) * a.inv_t, e = expf(t);
    s += e;
    if (e > 0.0f) q += e * t;
  }
  s = block_sum(s, red);
  q = block_sum(q, red);
  const float ls = logf(s);
  const bool none = s == 0.0f;   // every logit is -inf
  if (threadIdx.x == 0) {
    if (a.logp) a.logp[r] = none ? -INFINITY : (ld_elem(x, id) - mm) * a.inv_t - ls;
    if (a.stats) {
      a.stats[2 * r] = m;
      a.stats[2 * r + 1] = ls;
    }
    if (a.entropy) a.entropy[r] = none ? 0.0f : ls - q / s;
  }
  unsigned long long last = ~0ull;
  for (int i = 0; i < a.k; ++i) {
    unsigned long long best = 0;
    for (int c = threadIdx.x; c < a.vocab; c += kLogpThreads) {
      const unsigned long long v = (unsigned long long)order_key(ld_elem(x, c)) << 32 | (uint32_t)~c;
      if (v < last && v > best) best = v;
    }
    last = block_max_u64(best, red64);
    if (threadIdx.x == 0) {
      const int c = (int)~(uint32_t)last;
      a.top_ids[r * a.k + i] = c;
      a.top_logp[r * a.k + i] = none ? -INFINITY : (ld_elem(x, c) - mm) * a.inv_t - ls;
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(kLogpThreads) logp_grad_kernel(LogpGradArgs a) {
  const size_t r = blockIdx.x;
  const T* x = static_cast<const T*>(a.logits) + r * a.stride;
  T* dx = static_cast<T*>(a.dlogits) + r * a.dstride;
  const int id = a.ids ? token_of(a.ids, a.id64, a.vocab, r) : 0;
  const float g = a.dlogp && id >= 0 ? a.dlogp[r] : 0.0f;
  const float h = a.dentropy && id >= 0 ? a.dentropy[r] : 0.0f;
  const float m = a.stats[2 * r], ls = a.stats[2 * r + 1];
  if ((g == 0.0f && h == 0.0f) || m == -INFINITY) {
    for (int c = threadIdx.x; c < a.vocab; c += kLogpThreads) st_elem(dx, c, 0.0f);
    return;
  }
  const float ent = a.dentropy ? a.entropy[r] : 0.0f;
  for (int c = threadIdx.x; c < a.vocab; c += kLogpThreads) {
    const float lp = (ld_elem(x, c) - m) * a.inv_t - ls, p = expf(lp);
    float d = -g * p;
    if (p != 0.0f) d -= h * p * (lp + ent);
    if (c == id) d += g;
    st_elem(dx, c, d * a.inv_t);
  }
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
  if (!(temperature > 0.0f) || !std::isfinite(temperature) || !std::isfinite(1.0f / temperature))
    return op_fail(MG_ERR_INVALID_ARG, "%s: the temperature and its reciprocal must be positive and finite", fn);
  return MG_OK;
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
  if (dtype)
    mg::logp_kernel<mg::bf16><<<(unsigned)rows, mg::kLogpThreads, 0, (cudaStream_t)stream>>>(a);
  else
    mg::logp_kernel<float><<<(unsigned)rows, mg::kLogpThreads, 0, (cudaStream_t)stream>>>(a);
  return mg::op_end(fn, cudaGetLastError());
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
  st = mg::op_disjoint(fn, {{logits, rows_bytes(rows, vocab, row_stride, dtype), false, false},
                            {ids, n * (id_kind ? 8 : 4), false, false}, {stats, n * 8, false, false},
                            {entropy, n * 4, false, false}, {dlogp, n * 4, false, false}, {dentropy, n * 4, false, false},
                            {dlogits, rows_bytes(rows, vocab, dlogits_stride, dtype), true,
                             logits == dlogits && row_stride == dlogits_stride}});
  if (st != MG_OK || !rows) return st;
  mg::LogpGradArgs a = {logits, row_stride, vocab, ids, id_kind, 1.0f / temperature, stats, entropy, dlogp, dentropy, dlogits,
                        dlogits_stride};
  if (dtype)
    mg::logp_grad_kernel<mg::bf16><<<(unsigned)rows, mg::kLogpThreads, 0, (cudaStream_t)stream>>>(a);
  else
    mg::logp_grad_kernel<float><<<(unsigned)rows, mg::kLogpThreads, 0, (cudaStream_t)stream>>>(a);
  return mg::op_end(fn, cudaGetLastError());
}

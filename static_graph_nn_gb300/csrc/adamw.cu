// AdamW over many tensors at once, with moments in 32 or in 8 bits.
//
//   g' = c g                                  c = max_norm / norm where norm > max_norm, else 1
//   m  = b1 m + (1 - b1) g'
//   v  = b2 v + (1 - b2) g'^2
//   p  = p (1 - lr wd) - lr / (1 - b1^t) m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// Moments in 8 bits: m and sqrt(v) are e4m3 codes under one scale for each 256
// elements of a tensor.  A scale is the least power of two that keeps the
// block's largest magnitude at or below 446.7: e4m3 keeps the same three bits
// of mantissa under any scale, and a power of two leaves a value that does not
// change on its code, where a scale that follows the maximum would move all
// values of the block against their codes in every step.  The border lies just
// inside e4m3's 448, at a number that sums of short numbers do not hit, so that
// no rounding decides a scale.
// A code is rounded up or down at random with the probability of its distance:
// b2 = 0.999 changes sqrt(v) by at most one part in 2000 a step, far less than
// half a step of the code (one part in 16), so that rounding to nearest would
// keep a moment where it is forever.  The random bits are a function of the
// seed, t and the element's place in the list: 16 of a 64-bit word that
// SplitMix64 (Steele, Lea and Flood, OOPSLA 2014) gives for each four elements.
// The root of a second moment that is not 0 never gets the code 0 (an update
// would be divided by eps).  The update itself uses the moments before they are
// rounded.  Moments are computed one fp32 rounding an operation, so that a
// host that does the same finds the same codes.
#include <algorithm>
#include <cmath>
#include <exception>
#include <memory>
#include <vector>

#include "common.cuh"
#include "kernels.h"
#include "op_checks.h"

namespace mg {
namespace {

constexpr int kAdamwBlock = 256;       // elements under a scale
constexpr int kAdamwThreads = 256;
constexpr int kAdamwChunk = 8192;      // elements of one tensor that a block updates

struct AdamwChunk {
  void* p;
  const void* g;
  void* m;
  void* v;
  float* ms;
  float* vs;
  void* copy;
  unsigned long long place;   // of the chunk's first element in the list
  int len;
  int flags;                  // bit 0: p bf16, bit 1: g bf16
  float wd;
};

struct AdamwStep {
  const AdamwChunk* chunks;
  float b1, om1, b2, om2, ln_b1, ln_b2, eps;
  float lr, step_size, inv_root_bc2;   // from the host's lr and t
  const float* lr_dev;
  const int* step_dev;
  const float* norm;
  float max_norm;
  unsigned long long seed, step;
};

__host__ __device__ __forceinline__ unsigned long long mix64(unsigned long long z) {
  z = (z ^ (z >> 30)) * 0xBF58476D1CE4E5B9ull;
  z = (z ^ (z >> 27)) * 0x94D049BB133111EBull;
  return z ^ (z >> 31);
}

// Four elements' random bits; place a multiple of 4.
__device__ __forceinline__ unsigned long long adamw_random(unsigned long long key, unsigned long long place) {
  return mix64(key + (place / 4 + 1) * 0x9E3779B97F4A7C15ull);
}

// The scale of a block whose largest magnitude has these bits, and its reciprocal.
__device__ __forceinline__ float scale_of(uint32_t top) {
  const uint32_t b = (min(top, 0x7F800000u) + 0x20A3C4u) & 0x7F800000u;
  return __uint_as_float(b <= 9u << 23 ? 1u << 23 : b - (8u << 23));
}
__device__ __forceinline__ float reciprocal_of(float scale) {
  return __uint_as_float((254u << 23) - __float_as_uint(scale));
}

// e4m3 bits shifted to fp32's place are the value times 2^-120, subnormals too.
__device__ __forceinline__ float e4m3_value(uint32_t code) {
  if ((code & 0x7f) == 0x7f) return __int_as_float(0x7fffffff);
  return __uint_as_float((code & 0x7f) << 20 | (code & 0x80) << 24) * 0x1p120f;
}
// |x| is at most 448; rnd: 16 random bits.  What is not finite becomes NaN.
__device__ __forceinline__ uint32_t e4m3_code(float x, uint32_t rnd) {
  const uint32_t b = __float_as_uint(x * 0x1p-120f);
  return min(((b & 0x7fffffffu) + (rnd << 4)) >> 20, 0x7fu) | (b >> 31) << 7;
}

struct AdamwScalars {
  float c, lr, step_size, inv_root_bc2;
  unsigned long long key;
  bool skip;
};
__device__ __forceinline__ AdamwScalars adamw_scalars(const AdamwStep& a) {
  AdamwScalars s;
  const float norm = a.norm ? *a.norm : 0.0f;
  s.skip = !(norm - norm == 0.0f);
  s.c = norm > a.max_norm ? a.max_norm / norm : 1.0f;
  s.lr = a.lr_dev ? *a.lr_dev : a.lr;
  s.step_size = a.step_size;
  s.inv_root_bc2 = a.inv_root_bc2;
  unsigned long long t = a.step;
  if (a.step_dev) {
    t = max(*a.step_dev, 1);
    s.inv_root_bc2 = 1.0f / sqrtf(-expm1f((float)t * a.ln_b2));
  }
  if (a.step_dev || a.lr_dev)
    s.step_size = s.lr / (a.step_dev ? -expm1f((float)t * a.ln_b1) : a.step_size);   // (host t, device lr: the correction itself)
  s.key = mix64(a.seed * 1000003ull + t);
  return s;
}

__device__ __forceinline__ void adamw_moments(const AdamwStep& a, float g, float& m, float& v) {
  m = __fadd_rn(__fmul_rn(m, a.b1), __fmul_rn(g, a.om1));
  v = __fadd_rn(__fmul_rn(v, a.b2), __fmul_rn(__fmul_rn(g, g), a.om2));
}
__device__ __forceinline__ float adamw_param(const AdamwScalars& s, float eps, float wd, float p, float m, float root) {
  return p * (1.0f - s.lr * wd) - s.step_size * m / (root * s.inv_root_bc2 + eps);
}

// A chunk per block, a thread per element of a scale's block.
template <int BITS>
__global__ void __launch_bounds__(kAdamwThreads) adamw_kernel(AdamwStep a) {
  __shared__ float red[32];
  const AdamwScalars s = adamw_scalars(a);
  if (s.skip) return;
  const AdamwChunk k = a.chunks[blockIdx.x];
  for (int b = 0; b < k.len; b += kAdamwBlock) {
    const int i = b + threadIdx.x;
    const bool in = i < k.len;
    float p = 0.0f, g = 0.0f, m = 0.0f, v = 0.0f;
    if (in) {
      p = k.flags & 1 ? ld_elem(static_cast<const bf16*>(k.p), i) : ld_elem(static_cast<const float*>(k.p), i);
      g = k.flags & 2 ? ld_elem(static_cast<const bf16*>(k.g), i) : ld_elem(static_cast<const float*>(k.g), i);
      if (BITS == 32) {
        m = static_cast<const float*>(k.m)[i];
        v = static_cast<const float*>(k.v)[i];
      } else {
        m = e4m3_value(static_cast<const uint8_t*>(k.m)[i]) * k.ms[b / kAdamwBlock];
        v = e4m3_value(static_cast<const uint8_t*>(k.v)[i]) * k.vs[b / kAdamwBlock];
        v = __fmul_rn(v, v);
      }
      g = __fmul_rn(g, s.c);
      adamw_moments(a, g, m, v);
    }
    const float root = sqrtf(v);
    if (BITS == 8) {
      const uint32_t tm = __float_as_uint(block_max(fabsf(m), red)), tv = __float_as_uint(block_max(root, red));
      const float sm = scale_of(tm), sv = scale_of(tv);
      if (in) {
        const uint32_t rnd = (uint32_t)(adamw_random(s.key, (k.place + i) & ~3ull) >> (16 * (i & 3))) & 0xffffu;
        static_cast<uint8_t*>(k.m)[i] = e4m3_code(m * reciprocal_of(sm), rnd);
        static_cast<uint8_t*>(k.v)[i] = max(e4m3_code(root * reciprocal_of(sv), rnd), root != 0.0f ? 1u : 0u);
      }
      __syncthreads();
      if (threadIdx.x == 0) {
        k.ms[b / kAdamwBlock] = sm;
        k.vs[b / kAdamwBlock] = sv;
      }
    } else if (in) {
      static_cast<float*>(k.m)[i] = m;
      static_cast<float*>(k.v)[i] = v;
    }
    if (in) {
      p = adamw_param(s, a.eps, k.wd, p, m, root);
      if (k.flags & 1)
        st_elem(static_cast<bf16*>(k.p), i, p);
      else
        st_elem(static_cast<float*>(k.p), i, p);
      if (k.copy) st_elem(static_cast<bf16*>(k.copy), i, p);
    }
  }
}

}  // namespace
}  // namespace mg

struct mg_adamw {
  int device = 0, bits = 32;
  unsigned n_chunks = 0;
  mg::AdamwChunk* chunks = nullptr;
  double beta1 = 0, beta2 = 0, eps = 0;
  unsigned long long seed = 0;
};

using mg::op_fail;

static constexpr size_t kMaxAdamwChunks = 1u << 26;

extern "C" mg_status mg_adamw_create(int n, const mg_adamw_tensor* tensors, int state_bits, double beta1, double beta2,
                                     double eps, unsigned long long seed, mg_adamw** out) {
  const char* fn = "mg_adamw_create";
  if (!out) return op_fail(MG_ERR_INVALID_ARG, "%s: out is NULL", fn);
  *out = nullptr;
  if (n < 1 || !tensors) return op_fail(MG_ERR_INVALID_ARG, "%s: n must be positive and tensors non-NULL", fn);
  if (state_bits != 8 && state_bits != 32) return op_fail(MG_ERR_INVALID_ARG, "%s: state_bits must be 8 or 32", fn);
  if (!(beta1 >= 0.0 && (float)beta1 < 1.0f && beta2 >= 0.0 && (float)beta2 < 1.0f) || !((float)eps > 0.0f) || !std::isfinite(eps))
    return op_fail(MG_ERR_INVALID_ARG, "%s: betas must lie in [0, 1) and eps be positive", fn);
  try {
    struct Span {
      uintptr_t lo, hi;
      int tensor;
      bool written;
    };
    std::vector<Span> spans;
    std::vector<mg::AdamwChunk> table;
    unsigned long long place = 0;
    const size_t ss = state_bits == 8 ? 1 : 4;
    for (int i = 0; i < n; ++i) {
      const mg_adamw_tensor& t = tensors[i];
      if ((t.param_dtype != 0 && t.param_dtype != 1) || (t.grad_dtype != 0 && t.grad_dtype != 1))
        return op_fail(MG_ERR_INVALID_ARG, "%s: dtypes of tensor %d must be 0 or 1", fn, i);
      if (!(t.weight_decay >= 0.0f) || !std::isfinite(t.weight_decay))
        return op_fail(MG_ERR_INVALID_ARG, "%s: weight_decay of tensor %d must be finite and not negative", fn, i);
      if (t.count == 0) continue;
      if (!t.param || !t.grad || !t.m || !t.v || (state_bits == 8 && (!t.m_scales || !t.v_scales)))
        return op_fail(MG_ERR_INVALID_ARG, "%s: a pointer of tensor %d is NULL", fn, i);
      if (t.count / mg::kAdamwChunk + table.size() > kMaxAdamwChunks)
        return op_fail(MG_ERR_SHAPE, "%s: tensor %d has %zu elements, too many", fn, i, t.count);
      const size_t ps = t.param_dtype ? 2 : 4, gs = t.grad_dtype ? 2 : 4;
      const size_t blocks = (t.count + mg::kAdamwBlock - 1) / mg::kAdamwBlock;
      float* ms = state_bits == 8 ? t.m_scales : nullptr;
      float* vs = state_bits == 8 ? t.v_scales : nullptr;
      mg_status st = mg::op_begin(fn, {{t.param, (unsigned)ps}, {t.grad, (unsigned)gs}, {t.m, (unsigned)ss}, {t.v, (unsigned)ss},
                                       {ms, 4}, {vs, 4}, {t.copy, 2}});
      if (st != MG_OK) return st;
      const auto span = [&](const void* p, size_t bytes, bool written) {
        if (p) spans.push_back({reinterpret_cast<uintptr_t>(p), reinterpret_cast<uintptr_t>(p) + bytes, i, written});
      };
      span(t.param, t.count * ps, true);
      span(t.grad, t.count * gs, false);
      span(t.m, t.count * ss, true);
      span(t.v, t.count * ss, true);
      span(ms, blocks * 4, true);
      span(vs, blocks * 4, true);
      span(t.copy, t.count * 2, true);
      for (size_t a = 0; a < t.count; a += mg::kAdamwChunk) {
        mg::AdamwChunk k;
        k.p = static_cast<char*>(t.param) + a * ps;
        k.g = static_cast<const char*>(t.grad) + a * gs;
        k.m = static_cast<char*>(t.m) + a * ss;
        k.v = static_cast<char*>(t.v) + a * ss;
        k.ms = ms ? ms + a / mg::kAdamwBlock : nullptr;
        k.vs = vs ? vs + a / mg::kAdamwBlock : nullptr;
        k.copy = t.copy ? static_cast<char*>(t.copy) + a * 2 : nullptr;
        k.place = place + a;
        k.len = (int)std::min<size_t>(mg::kAdamwChunk, t.count - a);
        k.flags = t.param_dtype | t.grad_dtype << 1;
        k.wd = t.weight_decay;
        table.push_back(k);
      }
      place += (unsigned long long)blocks * mg::kAdamwBlock;
    }
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
    std::unique_ptr<mg_adamw> o(new mg_adamw());
    o->bits = state_bits;
    o->beta1 = beta1;
    o->beta2 = beta2;
    o->eps = eps;
    o->seed = seed;
    o->n_chunks = (unsigned)table.size();
    cudaError_t e = cudaGetDevice(&o->device);
    if (e == cudaSuccess && o->n_chunks) {
      const size_t bytes = table.size() * sizeof(mg::AdamwChunk);
      e = cudaMalloc((void**)&o->chunks, bytes);
      if (e != cudaSuccess) {
        cudaGetLastError();
        return op_fail(e == cudaErrorMemoryAllocation ? MG_ERR_OOM : MG_ERR_CUDA, "%s: %zu bytes: %s", fn, bytes,
                       cudaGetErrorString(e));
      }
      e = cudaMemcpy(o->chunks, table.data(), bytes, cudaMemcpyHostToDevice);
      // it may still be on its way, and a caller's stream need not wait for the
      // default one
      if (e == cudaSuccess) e = cudaStreamSynchronize(nullptr);
      if (e != cudaSuccess) cudaFree(o->chunks);
    }
    if (e != cudaSuccess) return mg::op_end(fn, e);
    *out = o.release();
    return MG_OK;
  } catch (const std::exception&) {   // of the vectors: no exception leaves a C entry
    return op_fail(MG_ERR_OOM, "%s: host allocation failed", fn);
  }
}

extern "C" void mg_adamw_destroy(mg_adamw* o) {
  if (!o) return;
  int prev = -1;
  cudaGetDevice(&prev);
  cudaSetDevice(o->device);
  cudaFree(o->chunks);   // waits for the device
  if (prev >= 0) cudaSetDevice(prev);
  delete o;
}

extern "C" mg_status mg_adamw_step(mg_adamw* o, double lr, long long step, const float* lr_device, const int* step_device,
                                   const float* norm, float max_norm, mg_stream_t stream) {
  const char* fn = "mg_adamw_step";
  if (!o) return op_fail(MG_ERR_INVALID_ARG, "%s: the optimizer is NULL", fn);
  if (!lr_device && !(lr >= 0.0 && std::isfinite((float)lr)))
    return op_fail(MG_ERR_INVALID_ARG, "%s: lr must be finite and not negative", fn);
  if (!step_device && step < 1) return op_fail(MG_ERR_INVALID_ARG, "%s: step must be at least 1", fn);
  if (norm && !(max_norm >= 0.0f)) return op_fail(MG_ERR_INVALID_ARG, "%s: max_norm must be at least 0", fn);
  int dev = -1;
  if (cudaGetDevice(&dev) == cudaSuccess && dev != o->device)
    return op_fail(MG_ERR_INVALID_ARG, "%s: the optimizer belongs to device %d but device %d is current", fn, o->device, dev);
  mg_status st = mg::op_begin(fn, {{lr_device, 4}, {step_device, 4}, {norm, 4}});
  if (st != MG_OK || !o->n_chunks) return st;
  mg::AdamwStep a;
  a.chunks = o->chunks;
  a.b1 = (float)o->beta1;
  a.om1 = (float)(1.0 - o->beta1);
  a.b2 = (float)o->beta2;
  a.om2 = (float)(1.0 - o->beta2);
  a.ln_b1 = (float)std::log(o->beta1);
  a.ln_b2 = (float)std::log(o->beta2);
  a.eps = (float)o->eps;
  const double bc1 = step_device ? 1.0 : -std::expm1((double)step * std::log(o->beta1));
  const double bc2 = step_device ? 1.0 : -std::expm1((double)step * std::log(o->beta2));
  a.lr = (float)lr;
  a.step_size = (float)(lr_device ? bc1 : lr / bc1);
  a.inv_root_bc2 = (float)(1.0 / std::sqrt(bc2));
  a.lr_dev = lr_device;
  a.step_dev = step_device;
  a.norm = norm;
  a.max_norm = max_norm;
  a.seed = o->seed;
  a.step = (unsigned long long)step;
  if (o->bits == 8)
    mg::adamw_kernel<8><<<o->n_chunks, mg::kAdamwThreads, 0, (cudaStream_t)stream>>>(a);
  else
    mg::adamw_kernel<32><<<o->n_chunks, mg::kAdamwThreads, 0, (cudaStream_t)stream>>>(a);
  return mg::op_end(fn, cudaGetLastError());
}

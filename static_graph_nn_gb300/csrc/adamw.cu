// AdamW over many tensors at once, with moments in 32 or in 8 bits.
//
//   g' = c g                                  c = max_norm / norm where norm > max_norm, else 1
//   m  = b1 m + (1 - b1) g'
//   v  = b2 v + (1 - b2) g'^2
//   p  = p (1 - lr wd) - lr / (1 - b1^t) m / (sqrt(v) / sqrt(1 - b2^t) + eps)
//
// Moments in 8 bits: m and sqrt(v) are e4m3 codes under one scale for each 256
// elements of a tensor.  A scale is the least power of two that keeps the
// block's largest finite magnitude at or below 446.7 (what is not finite becomes
// NaN under any scale): e4m3 keeps the same three bits of mantissa under any
// scale, and a power of two leaves a value that does not change on its code,
// where a scale that follows the maximum would move all values of the block
// against their codes in every step.  The border lies just
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
//
// Bound by DRAM: 28 bytes an fp32 element, 16 with 8-bit moments, 2 more for a bf16 copy.
// 334M elements with a copy: 1435 us (7.0 TB/s), with 8-bit moments 861 us (7.0 TB/s).
// With bf16 parameters and gradients, 10 bytes, by issue: 65 instructions an element (24M
// in 400 tensors: 57 us, 4.2 TB/s), about 45 of them the arithmetic of moments, roots and
// codes (random bits about 5); most of it is done on two elements at once.  Tensors at any
// address, one element an access: 100M fp32 in 429 us (aligned 404), with 8-bit moments 441
// (234), bf16 with 8-bit moments 691 (203).
// Blocks of 8-bit moments are copied ahead through shared memory: a warp's loads
// are under way while it computes (861 us against 1201).  In them a lane takes
// twice four neighbours, so that every access of a warp is contiguous; eight
// neighbours are two half used accesses of each sector (1091 us).
#include <algorithm>
#include <cmath>
#include <exception>
#include <iterator>
#include <memory>
#include <utility>
#include <vector>

#include <cuda_fp16.h>

#include "common.cuh"
#include "f32x2.cuh"
#include "kernels.h"
#include "op_checks.h"

namespace mg {
namespace {

constexpr int kAdamwBlock = 256;       // elements under a scale: eight for each lane of a warp
constexpr int kAdamwThreads = 256;
constexpr int kAdamwPass = kAdamwThreads * 8;   // elements that a block updates at once
constexpr int kAdamwChunk = 4 * kAdamwPass;     // of one tensor that it updates in all, in long lists

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
  int flags;                  // bit 0: p bf16, bit 1: g bf16, bit 2: eight elements of each allow one access
  float wd;
};
static_assert(sizeof(AdamwChunk) == 80, "the header states the table's bytes");

struct AdamwStep {
  const AdamwChunk* chunks;
  float b1, om1, b2, om2, ln_b1, ln_b2, eps;
  float one;                           // 1, unknown to the compiler
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

// Four elements' random bits are mix64 of this, place a multiple of 4.
constexpr unsigned long long kWeyl = 0x9E3779B97F4A7C15ull;
__device__ __forceinline__ unsigned long long random_state(unsigned long long key, unsigned long long place) {
  return key + (place / 4 + 1) * kWeyl;
}

// The scale of a block whose largest magnitude has these bits, and its reciprocal.
__device__ __forceinline__ float scale_of(uint32_t top) {
  const uint32_t b = (min(top, 0x7F800000u) + 0x20A3C4u) & 0x7F800000u;
  return __uint_as_float(b <= 9u << 23 ? 1u << 23 : b - (8u << 23));
}
__device__ __forceinline__ float reciprocal_of(float scale) {
  return __uint_as_float((254u << 23) - __float_as_uint(scale));
}

// Two e4m3 codes' values (NaN for its code).
__device__ __forceinline__ float2 e4m3_values(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((unsigned short)two));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// The larger of three magnitudes; NaN if one is.
__device__ __forceinline__ float max_abs3(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(fabsf(a)), "f"(fabsf(b)), "f"(fabsf(c)));
  return r;
}
__device__ __forceinline__ float rsqrt_near(float x) {
  float r;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}
__device__ __forceinline__ float reciprocal_near(float x) {
  float r;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
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

// The eight elements of a lane in a block of 256: neighbours, in one access
// (RUN); twice four neighbours, 128 apart (PAIR; of whole blocks); 32 apart (APART;
// for tensors at any address).
enum Lay { APART, RUN, PAIR };
template <Lay L>
__device__ __forceinline__ int element(int i0, int j) {
  return L == RUN ? i0 + j : L == PAIR ? i0 + j + (j < 4 ? 0 : 124) : i0 + 32 * j;
}
template <Lay L>
__device__ __forceinline__ int first_element(int b) {
  const int lane = threadIdx.x & 31;
  return b + (L == RUN ? 8 * lane : L == PAIR ? 4 * lane : lane);
}
__device__ __forceinline__ void ld8f32(const float* p, float (&f)[8]) {
  uint32_t w[8];
  asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]), "=r"(w[4]), "=r"(w[5]), "=r"(w[6]), "=r"(w[7])
               : "l"(p));
#pragma unroll
  for (int j = 0; j < 8; ++j) f[j] = __uint_as_float(w[j]);
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * j], f[2 * j + 1]);
    w[j] = *reinterpret_cast<const uint32_t*>(&h);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
template <Lay L>
__device__ __forceinline__ void load8(const void* p, bool narrow, int i0, int len, f32x2 (&o)[4]) {
  float f[8];
  if (L == RUN && i0 + 8 <= len) {
    if (narrow) {
      const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const bf16*>(p) + i0);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        f[2 * j] = __uint_as_float(w[j] << 16);
        f[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
      }
    } else {
      ld8f32(static_cast<const float*>(p) + i0, f);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int i = element<L>(i0, j);
      f[j] = i >= len ? 0.0f : narrow ? ld_elem(static_cast<const bf16*>(p), i) : ld_elem(static_cast<const float*>(p), i);
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) o[j] = both(f[2 * j], f[2 * j + 1]);
}
template <Lay L>
__device__ __forceinline__ void store8(void* p, bool narrow, int i0, int len, const f32x2 (&o)[4]) {
  float f[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 t = parts(o[j]);
    f[2 * j] = t.x;
    f[2 * j + 1] = t.y;
  }
  if (L == RUN && i0 + 8 <= len) {
    if (narrow)
      *reinterpret_cast<uint4*>(static_cast<bf16*>(p) + i0) = pack8(f);
    else
      st8f32(static_cast<float*>(p) + i0, f);
    return;
  }
  if constexpr (L == PAIR) {
    if (narrow) {
      const uint4 u = pack8(f);
      *reinterpret_cast<uint2*>(static_cast<bf16*>(p) + i0) = make_uint2(u.x, u.y);
      *reinterpret_cast<uint2*>(static_cast<bf16*>(p) + i0 + 128) = make_uint2(u.z, u.w);
    } else {
      *reinterpret_cast<float4*>(static_cast<float*>(p) + i0) = make_float4(f[0], f[1], f[2], f[3]);
      *reinterpret_cast<float4*>(static_cast<float*>(p) + i0 + 128) = make_float4(f[4], f[5], f[6], f[7]);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int i = element<L>(i0, j);
      if (i >= len) continue;
      if (narrow)
        st_elem(static_cast<bf16*>(p), i, f[j]);
      else
        st_elem(static_cast<float*>(p), i, f[j]);
    }
  }
}
// Eight codes in two words.
template <Lay L>
__device__ __forceinline__ uint2 load_codes(const uint8_t* p, int i0, int len) {
  if (L == RUN && i0 + 8 <= len) return *reinterpret_cast<const uint2*>(p + i0);
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int i = element<L>(i0, j);
    if (i < len) w[j / 4] |= (uint32_t)p[i] << (8 * (j % 4));
  }
  return make_uint2(w[0], w[1]);
}
template <Lay L>
__device__ __forceinline__ void store_codes(uint8_t* p, int i0, int len, uint2 c) {
  if (L == RUN && i0 + 8 <= len) {
    *reinterpret_cast<uint2*>(p + i0) = c;
    return;
  }
  if constexpr (L == PAIR) {
    *reinterpret_cast<uint32_t*>(p + i0) = c.x;
    *reinterpret_cast<uint32_t*>(p + i0 + 128) = c.y;
  } else {
    const uint32_t w[2] = {c.x, c.y};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const int i = element<L>(i0, j);
      if (i < len) p[i] = (uint8_t)(w[j / 4] >> (8 * (j % 4)));
    }
  }
}
// The moments and the root, eight elements of a lane.  Products with a scale, a
// power of two, round nowhere, so a scale goes into the factor that follows it
// (wide: not where that would leave the normal range).
__device__ __forceinline__ void moments8(const AdamwStep& a, float c, const f32x2 (&g)[4], f32x2 (&m)[4], f32x2 (&v)[4]) {
  // the sums as products with 1: the compiler makes one operation, with one
  // rounding, of a product and a sum
  const f32x2 cc = both(c), o1 = both(a.om1), o2 = both(a.om2), one = both(a.one);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const f32x2 t = mul2(g[j], cc);
    m[j] = fma2(m[j], one, mul2(t, o1));
    v[j] = fma2(v[j], one, mul2(mul2(t, t), o2));
  }
}
__device__ __forceinline__ void scaled_moments(const AdamwStep& a, f32x2 (&m)[4], f32x2 (&v)[4]) {
  const f32x2 b1 = both(a.b1), b2 = both(a.b2);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    m[j] = mul2(m[j], b1);
    v[j] = mul2(v[j], b2);
  }
}
// beta1 m and beta2 v from their codes.
__device__ __forceinline__ void decode8(const AdamwStep& a, uint2 mc, uint2 vc, float ms, float vs, f32x2 (&m)[4], f32x2 (&v)[4]) {
  const uint32_t mt[4] = {mc.x & 0xffffu, mc.x >> 16, mc.y & 0xffffu, mc.y >> 16};
  const uint32_t vt[4] = {vc.x & 0xffffu, vc.x >> 16, vc.y & 0xffffu, vc.y >> 16};
  const bool wide = (ms == 0.0f || (ms >= 0x1p-100f && ms <= 0x1p100f)) && (vs == 0.0f || (vs >= 0x1p-40f && vs <= 0x1p40f));
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 x = e4m3_values(mt[j]), y = e4m3_values(vt[j]);
    m[j] = both(x.x, x.y);
    v[j] = both(y.x, y.y);
  }
  if (wide) {
    const f32x2 fm = both(ms * a.b1), fv = both(vs * vs * a.b2);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      m[j] = mul2(m[j], fm);
      v[j] = mul2(mul2(v[j], v[j]), fv);   // (a code's square is exact)
    }
    return;
  }
  const f32x2 fm = both(ms), fv = both(vs);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    m[j] = mul2(m[j], fm);
    v[j] = mul2(v[j], fv);
    v[j] = mul2(v[j], v[j]);
  }
  scaled_moments(a, m, v);
}
// The largest magnitude's bits over the warp's 256 values (a NaN is larger than any number).
__device__ __forceinline__ uint32_t block_top(const f32x2 (&f)[4]) {
  const float2 p = parts(f[0]), q = parts(f[1]), r = parts(f[2]), t = parts(f[3]);
  const float top = max_abs3(max_abs3(p.x, p.y, q.x), max_abs3(q.y, r.x, r.y), max_abs3(t.x, t.y, 0.0f));
  return __reduce_max_sync(0xffffffffu, __float_as_uint(top));
}
// The same over those that are finite: what is not becomes NaN under any scale, and takes no part in it.
__device__ __forceinline__ uint32_t finite_top(const f32x2 (&f)[4]) {
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 x = parts(f[j]);
    const uint32_t a = __float_as_uint(fabsf(x.x)), b = __float_as_uint(fabsf(x.y));
    top = max(top, max(a < 0x7f800000u ? a : 0u, b < 0x7f800000u ? b : 0u));
  }
  return __reduce_max_sync(0xffffffffu, top);
}
// Square roots, rounded: an estimate and one step of Newton's method on it, whose
// residual is exact.  For values that are normal numbers or 0 (of smaller ones the root
// comes out too small).
__device__ __forceinline__ void roots8(f32x2 (&v)[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 x = parts(v[j]);
    const f32x2 y = both(rsqrt_near(fmaxf(x.x, 0x1p-126f)), rsqrt_near(fmaxf(x.y, 0x1p-126f)));
    const f32x2 r = mul2(v[j], y), e = fma2(mul2(r, both(-1.0f)), r, v[j]);
    v[j] = fma2(e, mul2(y, both(0.5f)), r);
  }
}
__device__ __forceinline__ void update8(const AdamwStep& a, const AdamwScalars& s, float wd, const f32x2 (&m)[4],
                                        const f32x2 (&root)[4], f32x2 (&p)[4]) {
  const f32x2 keep = both(1.0f - s.lr * wd), rate = both(-s.step_size), inv = both(s.inv_root_bc2), eps = both(a.eps);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 d = parts(fma2(root[j], inv, eps));
    p[j] = fma2(mul2(m[j], rate), both(reciprocal_near(d.x), reciprocal_near(d.y)), mul2(p[j], keep));
  }
}
// Codes of eight values under the scale, top the largest's bits; rnd: two elements' 16
// random bits in each word.  A value times 2^-120 over the scale has the bits of its
// e4m3 code, subnormals too, at fp32's place; the random bits are added below the
// code's last one, and the code is the top byte when all is shifted up by four (which
// drops the sign).  What is not finite becomes NaN.
__device__ __forceinline__ uint2 encode8(const f32x2 (&f)[4], float scale, uint32_t top, const uint32_t (&rnd)[4]) {
  const f32x2 inv = both(reciprocal_of(scale)), place = both(0x1p-120f);
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t t[4];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const float2 x = parts(mul2(mul2(f[2 * h + j], inv), place));
      t[2 * j] = (__float_as_uint(x.x) << 4) + __byte_perm(rnd[2 * h + j], 0, 0x4104);
      t[2 * j + 1] = (__float_as_uint(x.y) << 4) + __byte_perm(rnd[2 * h + j], 0, 0x4324);
    }
    w[h] = __byte_perm(__byte_perm(t[0], t[1], 0x0073), __byte_perm(t[2], t[3], 0x0073), 0x5410);
  }
  if (top >= 0x7f800000u) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 y = parts(f[j]);
      if (!(fabsf(y.x) < INFINITY)) w[j / 2] |= 0x7fu << (16 * (j % 2));
      if (!(fabsf(y.y) < INFINITY)) w[j / 2] |= 0x7fu << (16 * (j % 2) + 8);
    }
  }
  return make_uint2(w[0], w[1]);
}
// The signs of eight values, in the codes' places.
__device__ __forceinline__ uint2 signs8(const f32x2 (&f)[4]) {
  uint32_t w[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const float2 x = parts(f[2 * h]), y = parts(f[2 * h + 1]);
    w[h] = __byte_perm(__byte_perm(__float_as_uint(x.x), __float_as_uint(x.y), 0x0073),
                       __byte_perm(__float_as_uint(y.x), __float_as_uint(y.y), 0x0073), 0x5410) & 0x80808080u;
  }
  return make_uint2(w[0], w[1]);
}
// Codes of 0 of values that are not 0 become 1.
__device__ __forceinline__ void not_zero8(const f32x2 (&f)[4], uint2& c) {
  uint32_t w[2] = {c.x, c.y};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (((w[h] - 0x01010101u) & ~w[h] & 0x80808080u) == 0) continue;
    const float2 x = parts(f[2 * h]), y = parts(f[2 * h + 1]);
    const float e[4] = {x.x, x.y, y.x, y.y};
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if ((w[h] >> (8 * j) & 0xffu) == 0 && e[j] != 0.0f) w[h] |= 1u << (8 * j);
  }
  c = make_uint2(w[0], w[1]);
}
// A warp's 256 elements of a chunk, from element b on, that are there: p and g, and
// beta1 m and beta2 v.
template <int BITS, Lay L>
__device__ __forceinline__ void adamw_finish(const AdamwStep& a, const AdamwScalars& s, const AdamwChunk& k, int b,
                                             unsigned long long state, f32x2 (&p)[4], f32x2 (&g)[4], f32x2 (&m)[4],
                                             f32x2 (&v)[4]) {
  const int i0 = first_element<L>(b), blk = b / kAdamwBlock;
  moments8(a, s.c, g, m, v);
  if (BITS == 32) {
    store8<L>(k.m, false, i0, k.len, m);
    store8<L>(k.v, false, i0, k.len, v);
  }
  const uint32_t tm = BITS == 8 ? block_top(m) : 0, tv = BITS == 8 ? block_top(v) : 0;
  const bool finite = max(tm, tv) < 0x7f800000u;
  const float sm = scale_of(finite ? tm : finite_top(m));
  const float sv = scale_of(__float_as_uint(sqrtf(__uint_as_float(finite ? tv : finite_top(v)))));
  // (a root of a moment below the normal range is then far below eps, and its code the least)
  if (BITS == 8 && finite && sv >= 0x1p-30f && sv <= 0x1p60f && a.eps >= 1e-9f) {
    roots8(v);
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 x = parts(v[j]);
      v[j] = both(sqrtf(x.x), sqrtf(x.y));
    }
  }
  update8(a, s, k.wd, m, v, p);
  store8<L>(k.p, k.flags & 1, i0, k.len, p);
  if (k.copy) store8<L>(k.copy, true, i0, k.len, p);
  if (BITS == 8) {
    uint32_t rnd[4];
    if (L != APART) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const unsigned long long w = mix64(state + h * (element<L>(0, 4) / 4 * kWeyl));
        rnd[2 * h] = (uint32_t)w;
        rnd[2 * h + 1] = (uint32_t)(w >> 32);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const unsigned long long at = k.place + i0 + 32 * j;
        const uint32_t r = (uint32_t)(mix64(random_state(s.key, at)) >> (16 * (at & 3))) & 0xffffu;
        rnd[j / 2] = j % 2 ? rnd[j / 2] | r << 16 : r;
      }
    }
    const uint2 mc = encode8(m, sm, tm, rnd);
    uint2 vc = encode8(v, sv, tv, rnd);
    const uint2 signs = signs8(m);
    not_zero8(v, vc);
    store_codes<L>(static_cast<uint8_t*>(k.m), i0, k.len, make_uint2(mc.x | signs.x, mc.y | signs.y));
    store_codes<L>(static_cast<uint8_t*>(k.v), i0, k.len, vc);
    __syncwarp();   // every lane has read the scales
    if ((threadIdx.x & 31) == 0) {
      k.ms[blk] = sm;
      k.vs[blk] = sv;
    }
  }
}

template <int BITS, Lay L>
__device__ __forceinline__ void adamw_block(const AdamwStep& a, const AdamwScalars& s, const AdamwChunk& k, int b,
                                            unsigned long long state) {
  const int i0 = first_element<L>(b), blk = b / kAdamwBlock;
  f32x2 p[4], g[4], m[4], v[4];
  load8<L>(k.p, k.flags & 1, i0, k.len, p);
  load8<L>(k.g, k.flags & 2, i0, k.len, g);
  if (BITS == 32) {
    load8<L>(k.m, false, i0, k.len, m);
    load8<L>(k.v, false, i0, k.len, v);
    scaled_moments(a, m, v);
  } else {
    const uint2 mc = load_codes<L>(static_cast<const uint8_t*>(k.m), i0, k.len);
    const uint2 vc = load_codes<L>(static_cast<const uint8_t*>(k.v), i0, k.len);
    decode8(a, mc, vc, k.ms[blk], k.vs[blk], m, v);
  }
  adamw_finish<BITS, L>(a, s, k, b, state, p, g, m, v);
}

// ---- 8-bit moments: whole blocks through shared memory, copied ahead
constexpr int kAdamwStages = 2;          // (three, with room for three blocks: 855 us, but 61 against 57 for the bf16 list)
constexpr int kAdamwStageBytes = 2560;   // p, g: 1024 each; m, v: 256 each
constexpr int kAdamwSmem = kAdamwThreads / 32 * kAdamwStages * kAdamwStageBytes;

template <int N>
__device__ __forceinline__ void copy_ahead(uint32_t to, const void* from) {
  if (N == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to), "l"(from), "n"(N) : "memory");
}
// Every lane copies, and later reads, its own elements (PAIR: a warp's accesses are
// contiguous): nothing to wait for but its own copies.
__device__ __forceinline__ void copy_block(const AdamwChunk& k, int b, uint32_t stage) {
  const int lane = threadIdx.x & 31, i0 = first_element<PAIR>(b);
  const auto wide = [&](uint32_t to, const void* p, bool narrow) {
    if (narrow) {
      copy_ahead<8>(to + 8 * lane, static_cast<const bf16*>(p) + i0);
      copy_ahead<8>(to + 512 + 8 * lane, static_cast<const bf16*>(p) + i0 + 128);
    } else {
      copy_ahead<16>(to + 16 * lane, static_cast<const float*>(p) + i0);
      copy_ahead<16>(to + 512 + 16 * lane, static_cast<const float*>(p) + i0 + 128);
    }
  };
  wide(stage, k.p, k.flags & 1);
  wide(stage + 1024, k.g, k.flags & 2);
  copy_ahead<4>(stage + 2048 + 4 * lane, static_cast<const uint8_t*>(k.m) + i0);
  copy_ahead<4>(stage + 2176 + 4 * lane, static_cast<const uint8_t*>(k.m) + i0 + 128);
  copy_ahead<4>(stage + 2304 + 4 * lane, static_cast<const uint8_t*>(k.v) + i0);
  copy_ahead<4>(stage + 2432 + 4 * lane, static_cast<const uint8_t*>(k.v) + i0 + 128);
}
__device__ __forceinline__ void read_wide(const char* at, bool narrow, f32x2 (&o)[4]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (narrow) {
      const uint2 u = *reinterpret_cast<const uint2*>(at + 512 * h + 8 * lane);
      o[2 * h] = both(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u));
      o[2 * h + 1] = both(__uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
    } else {
      const float4 u = *reinterpret_cast<const float4*>(at + 512 * h + 16 * lane);
      o[2 * h] = both(u.x, u.y);
      o[2 * h + 1] = both(u.z, u.w);
    }
  }
}
__device__ __forceinline__ uint2 read_codes(const char* at) {
  const int lane = threadIdx.x & 31;
  return make_uint2(*reinterpret_cast<const uint32_t*>(at + 4 * lane), *reinterpret_cast<const uint32_t*>(at + 128 + 4 * lane));
}
__device__ __forceinline__ void adamw8_chunk(const AdamwStep& a, const AdamwScalars& s, const AdamwChunk& k) {
  extern __shared__ __align__(16) char buffer[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, first = warp * kAdamwBlock;
  char* mine = buffer + warp * kAdamwStages * kAdamwStageBytes;
  const uint32_t at = (uint32_t)__cvta_generic_to_shared(mine);
  const int whole = k.len < first + kAdamwBlock ? 0 : (k.len - first - kAdamwBlock) / kAdamwPass + 1;   // this warp's
#pragma unroll
  for (int i = 0; i < kAdamwStages - 1; ++i) {
    if (i < whole) copy_block(k, first + i * kAdamwPass, at + i * kAdamwStageBytes);
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  // lane i, and 16 + i, hold the scales of this warp's block i
  float scales = 0.0f;
  if ((lane & 15) < whole) scales = (lane < 16 ? k.ms : k.vs)[warp + (lane & 15) * (kAdamwPass / kAdamwBlock)];
  unsigned long long state = random_state(s.key, k.place + first_element<PAIR>(first));
  int slot = 0;
  for (int i = 0; i < whole; ++i) {
    asm volatile("cp.async.wait_group %0;" ::"n"(kAdamwStages - 2) : "memory");
    const char* in = mine + slot * kAdamwStageBytes;
    f32x2 p[4], g[4], m[4], v[4];
    read_wide(in, k.flags & 1, p);
    read_wide(in + 1024, k.flags & 2, g);
    const uint2 mc = read_codes(in + 2048), vc = read_codes(in + 2304);
    const int next = i + kAdamwStages - 1;
    if (next < whole)
      copy_block(k, first + next * kAdamwPass, at + (slot == 0 ? kAdamwStages - 1 : slot - 1) * kAdamwStageBytes);
    asm volatile("cp.async.commit_group;" ::: "memory");
    decode8(a, mc, vc, __shfl_sync(0xffffffffu, scales, i), __shfl_sync(0xffffffffu, scales, 16 + i), m, v);
    adamw_finish<8, PAIR>(a, s, k, first + i * kAdamwPass, state, p, g, m, v);
    state += kAdamwPass / 4 * kWeyl;
    slot = slot == kAdamwStages - 1 ? 0 : slot + 1;
  }
  const int b = first + whole * kAdamwPass;
  if (b < k.len) adamw_block<8, RUN>(a, s, k, b, random_state(s.key, k.place + first_element<RUN>(b)));   // the tensor's end
}

// A chunk per block, 256 elements at a time per warp.
template <int BITS>
__global__ void __launch_bounds__(kAdamwThreads, BITS == 8 ? 4 : 3) adamw_kernel(AdamwStep a) {
  const AdamwChunk k = a.chunks[blockIdx.x];
  const AdamwScalars s = adamw_scalars(a);
  if (s.skip) return;
  const int first = (threadIdx.x >> 5) * kAdamwBlock;
  if (!(k.flags & 4)) {
    for (int b = first; b < k.len; b += kAdamwPass) adamw_block<BITS, APART>(a, s, k, b, 0);
  } else if (BITS == 8) {
    adamw8_chunk(a, s, k);
  } else {
    for (int b = first; b < k.len; b += kAdamwPass) adamw_block<BITS, RUN>(a, s, k, b, 0);
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
  std::vector<std::pair<uintptr_t, uintptr_t>> written;   // the memory that a step writes: begins and ends, ascending
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
  if (!(beta1 >= 0.0 && (float)beta1 < 1.0f && beta2 >= 0.0 && (float)beta2 < 1.0f) || !((float)eps >= 0x1p-126f) || !std::isfinite((float)eps))
    return op_fail(MG_ERR_INVALID_ARG, "%s: betas must lie in [0, 1) and eps be a positive normal fp32 number", fn);
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
    // short lists in chunks of one pass, so that they spread over all multiprocessors
    double total = 0.0;
    for (int i = 0; i < n; ++i) total += (double)tensors[i].count;
    const size_t chunk = total < 8.0 * mg::device_sms() * mg::kAdamwChunk ? mg::kAdamwPass : mg::kAdamwChunk;
    for (int i = 0; i < n; ++i) {
      const mg_adamw_tensor& t = tensors[i];
      if ((t.param_dtype != 0 && t.param_dtype != 1) || (t.grad_dtype != 0 && t.grad_dtype != 1))
        return op_fail(MG_ERR_INVALID_ARG, "%s: dtypes of tensor %d must be 0 or 1", fn, i);
      if (!(t.weight_decay >= 0.0f) || !std::isfinite(t.weight_decay))
        return op_fail(MG_ERR_INVALID_ARG, "%s: weight_decay of tensor %d must be finite and not negative", fn, i);
      if (t.count == 0) continue;
      if (!t.param || !t.grad || !t.m || !t.v || (state_bits == 8 && (!t.m_scales || !t.v_scales)))
        return op_fail(MG_ERR_INVALID_ARG, "%s: a pointer of tensor %d is NULL", fn, i);
      if (t.count / chunk + table.size() > kMaxAdamwChunks)
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
      const auto at = [](const void* p, size_t align) { return reinterpret_cast<uintptr_t>(p) % align == 0; };
      const bool vec = at(t.param, 8 * ps) && at(t.grad, 8 * gs) && at(t.m, 8 * ss) && at(t.v, 8 * ss) && at(t.copy, 16);
      for (size_t a = 0; a < t.count; a += chunk) {
        mg::AdamwChunk k;
        k.p = static_cast<char*>(t.param) + a * ps;
        k.g = static_cast<const char*>(t.grad) + a * gs;
        k.m = static_cast<char*>(t.m) + a * ss;
        k.v = static_cast<char*>(t.v) + a * ss;
        k.ms = ms ? ms + a / mg::kAdamwBlock : nullptr;
        k.vs = vs ? vs + a / mg::kAdamwBlock : nullptr;
        k.copy = t.copy ? static_cast<char*>(t.copy) + a * 2 : nullptr;
        k.place = place + a;
        k.len = (int)std::min<size_t>(chunk, t.count - a);
        k.flags = t.param_dtype | t.grad_dtype << 1 | (vec ? 4 : 0);
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
    for (const Span& s : spans)
      if (s.written) o->written.emplace_back(s.lo, s.hi);
    o->bits = state_bits;
    o->beta1 = beta1;
    o->beta2 = beta2;
    o->eps = eps;
    o->seed = seed;
    o->n_chunks = (unsigned)table.size();
    cudaError_t e = cudaGetDevice(&o->device);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(mg::adamw_kernel<8>, cudaFuncAttributeMaxDynamicSharedMemorySize, mg::kAdamwSmem);
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
  for (const void* p : {(const void*)lr_device, (const void*)step_device, (const void*)norm}) {
    const uintptr_t at = reinterpret_cast<uintptr_t>(p);
    const auto behind = std::lower_bound(o->written.begin(), o->written.end(), std::make_pair(at + 4, (uintptr_t)0));
    if (p && behind != o->written.begin() && std::prev(behind)->second > at)
      return op_fail(MG_ERR_INVALID_ARG, "%s: lr_device, step_device or norm lies in memory that the step writes", fn);
  }
  mg::AdamwStep a;
  a.chunks = o->chunks;
  a.b1 = (float)o->beta1;
  a.om1 = (float)(1.0 - o->beta1);
  a.b2 = (float)o->beta2;
  a.om2 = (float)(1.0 - o->beta2);
  a.ln_b1 = (float)std::log(o->beta1);
  a.ln_b2 = (float)std::log(o->beta2);
  a.eps = (float)o->eps;
  a.one = 1.0f;
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
    mg::adamw_kernel<8><<<o->n_chunks, mg::kAdamwThreads, mg::kAdamwSmem, (cudaStream_t)stream>>>(a);
  else
    mg::adamw_kernel<32><<<o->n_chunks, mg::kAdamwThreads, 0, (cudaStream_t)stream>>>(a);
  return mg::op_end(fn, cudaGetLastError());
}

// Fused epilogue of a tensor-core GEMM: 32 accumulator columns of one row, as
// GemmArgs describes it.  Shared by the SM-pair GEMM and the grouped products.
#pragma once
#include "common.cuh"
#include "kernels.h"

namespace mg {

template <typename TO>
static __device__ __forceinline__ float rv(float v) {
  return sizeof(TO) == 2 ? __bfloat162float(__float2bfloat16_rn(v)) : v;
}

static __device__ __forceinline__ void ld8f(const bf16* p, float* f) {
  uint4 u = *reinterpret_cast<const uint4*>(p);
  const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float2 t = __bfloat1622float2(h[i]);
    f[2 * i] = t.x;
    f[2 * i + 1] = t.y;
  }
}

static __device__ __forceinline__ void st8f(bf16* p, const float* f) {
  uint4 u;
  uint32_t* w = reinterpret_cast<uint32_t*>(&u);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<uint32_t*>(&h);
  }
  *reinterpret_cast<uint4*>(p) = u;
}

// Epilogue of 32 columns of one row; identical arithmetic to gemm_tc.cu.  On
// return v holds the values stored (before their rounding to TO) at the
// columns below N.
template <typename TO>
static __device__ __forceinline__ void epi32(const GemmArgs& g, bool vec, bool vec32, int m, int n0,
                                      float (&v)[32]) {
  if (vec && n0 + 32 <= g.N) {
    if (g.bias) {
      const float4* b4 = reinterpret_cast<const float4*>(g.bias + n0);
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        float4 b = b4[q];
        v[4 * q] += b.x; v[4 * q + 1] += b.y; v[4 * q + 2] += b.z; v[4 * q + 3] += b.w;
      }
    }
    if (g.act || g.resid || g.out_z) {
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] = rv<TO>(v[j]);
    }
    if (g.out_z) {
      bf16* z = static_cast<bf16*>(g.out_z) + (size_t)m * g.ldz + n0;
      if (vec32) {
        st16bf(z, v);
        st16bf(z + 16, v + 16);
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) st8f(z + 8 * q, v + 8 * q);
      }
    }
    if (g.act) {
#pragma unroll
      for (int j = 0; j < 32; ++j) v[j] = apply_act(g.act, v[j]);
    }
    if (g.dact) {
      const bf16* sv = static_cast<const bf16*>(g.saved) + (size_t)m * g.lds + n0;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        float f[16];
        if (vec32) {
          ld16bf(sv + 16 * q, f);
        } else {
          ld8f(sv + 16 * q, f);
          ld8f(sv + 16 * q + 8, f + 8);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i)
          v[16 * q + i] = rv<TO>(v[16 * q + i]) * act_grad_from_saved(g.dact, f[i]);
      }
    }
    if (g.resid) {
      const bf16* rp = static_cast<const bf16*>(g.resid) + (size_t)m * g.ldr + n0;
#pragma unroll
      for (int q = 0; q < 2; ++q) {
        float f[16];
        if (vec32) {
          ld16bf(rp + 16 * q, f);
        } else {
          ld8f(rp + 16 * q, f);
          ld8f(rp + 16 * q + 8, f + 8);
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) v[16 * q + i] += f[i];
      }
    }
    TO* out = static_cast<TO*>(g.out) + (size_t)m * g.ldo + n0;
    if (vec32) {
      if (sizeof(TO) == 2) {
        st16bf(reinterpret_cast<bf16*>(out), v);
        st16bf(reinterpret_cast<bf16*>(out) + 16, v + 16);
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) st8f32(reinterpret_cast<float*>(out) + 8 * q, v + 8 * q);
      }
    } else if (sizeof(TO) == 2) {
#pragma unroll
      for (int q = 0; q < 4; ++q) st8f(reinterpret_cast<bf16*>(out) + 8 * q, v + 8 * q);
    } else {
#pragma unroll
      for (int q = 0; q < 8; ++q)
        reinterpret_cast<float4*>(out)[q] = make_float4(v[q * 4], v[q * 4 + 1], v[q * 4 + 2], v[q * 4 + 3]);
    }
    return;
  }
  const size_t rz = (size_t)m * g.ldz, rs = (size_t)m * g.lds, rr = (size_t)m * g.ldr;
#pragma unroll
  for (int j = 0; j < 32; ++j) {
    const int n = n0 + j;
    if (n >= g.N) continue;
    float x = v[j];
    if (g.bias) x += g.bias[n];
    if (g.act || g.resid || g.out_z) x = rv<TO>(x);
    if (g.out_z) static_cast<bf16*>(g.out_z)[rz + n] = __float2bfloat16_rn(x);
    if (g.act) x = apply_act(g.act, x);
    if (g.dact) {
      x = rv<TO>(x);
      x *= act_grad_from_saved(g.dact, __bfloat162float(static_cast<const bf16*>(g.saved)[rs + n]));
    }
    if (g.resid) x += __bfloat162float(static_cast<const bf16*>(g.resid)[rr + n]);
    st_elem(static_cast<TO*>(g.out), (size_t)m * g.ldo + n, x);
    v[j] = x;
  }
}

// The same where the 32 columns may end at N, a multiple of 8, and every row is
// 16-byte aligned: whole groups of 8 columns in 16-byte accesses.  (Element by
// element, the last 16 of 304 columns doubled a product's time.)  No bias.
template <typename TO>
static __device__ __forceinline__ void epi_by8(const GemmArgs& g, int m, int n0, float (&v)[32]) {
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int n = n0 + 8 * q;
    if (n >= g.N) break;
    float* x = v + 8 * q;
    if (g.act || g.resid || g.out_z) {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = rv<TO>(x[i]);
    }
    if (g.out_z) st8f(static_cast<bf16*>(g.out_z) + (size_t)m * g.ldz + n, x);
    if (g.act) {
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = apply_act(g.act, x[i]);
    }
    if (g.dact) {
      float f[8];
      ld8f(static_cast<const bf16*>(g.saved) + (size_t)m * g.lds + n, f);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = rv<TO>(x[i]) * act_grad_from_saved(g.dact, f[i]);
    }
    if (g.resid) {
      float f[8];
      ld8f(static_cast<const bf16*>(g.resid) + (size_t)m * g.ldr + n, f);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] += f[i];
    }
    TO* out = static_cast<TO*>(g.out) + (size_t)m * g.ldo + n;
    if (sizeof(TO) == 2) {
      st8f(reinterpret_cast<bf16*>(out), x);
    } else {
      reinterpret_cast<float4*>(out)[0] = make_float4(x[0], x[1], x[2], x[3]);
      reinterpret_cast<float4*>(out)[1] = make_float4(x[4], x[5], x[6], x[7]);
    }
  }
}

}  // namespace mg

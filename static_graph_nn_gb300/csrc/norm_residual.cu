// The step between two blocks of a residual network: the block's output y is
// normalised, gated and added to the scaled residual stream, and the sum is
// normalised for the next block.
//   u = y r1 g1,  r1 = 1 / sqrt(mean(y^2) + eps)        (u = y without g1)
//   x' = s x + a u                                      (a: one gate for all rows, or one for each run of rows)
//   h = x' r2 g2, r2 = 1 / sqrt(mean(x'^2) + eps)
// Backward, from the gradients dx' and dh:
//   t = dx' + r2 (dh g2) - x' r2^3 mean(dh g2 x')       dx = s t
//   w = a t,  dy = r1 (w g1) - y r1^3 mean(w g1 y)
//   dg2 = sum dh x' r2,  dg1 = sum w y r1,  da = sum t u (over the gate's rows)
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "kernels.h"
#include "op_checks.h"

namespace mg {
namespace {

constexpr int kNrThreads = 256;

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
  int rows, dim, gate_rows;
  float scale;
  void* dy;
  void* dx;
  float* dg1;
  float* dgate;
  float* dg2;
  float* ws;
};

template <typename T>
__global__ void __launch_bounds__(kNrThreads) norm_res_kernel(NormResArgs a) {
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
    for (int c = threadIdx.x; c < a.dim; c += kNrThreads) s += out(c) * out(c);
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

// One gate's rows, or a part of them, per block (blockIdx.y the part): the
// gradients of the rows, and the columns' sums over them into the workspace.
template <typename T>
__global__ void __launch_bounds__(kNrThreads) norm_res_grad_kernel(NormResGradArgs a, int part_rows) {
  __shared__ float red[32];
  const size_t part = (size_t)blockIdx.x * gridDim.y + blockIdx.y;
  const float* gate = a.gate ? a.gate + (size_t)blockIdx.x * a.dim : nullptr;
  float* sums = a.ws + part * 3 * a.dim;
  const int first = blockIdx.x * a.gate_rows;
  const int end = min(first + a.gate_rows, first + ((int)blockIdx.y + 1) * part_rows);
  for (int c = threadIdx.x; c < 3 * a.dim; c += kNrThreads) sums[c] = 0.0f;
  __syncthreads();
  for (int r = first + blockIdx.y * part_rows; r < end; ++r) {
    const size_t row = (size_t)r * a.dim;
    const T *y = static_cast<const T*>(a.y) + row, *x = static_cast<const T*>(a.x) + row;
    const T* dxo = a.dxo ? static_cast<const T*>(a.dxo) + row : nullptr;
    const T* dh = a.dh ? static_cast<const T*>(a.dh) + row : nullptr;
    const float r1 = a.g1 ? a.rstd[2 * (size_t)r] : 1.0f, r2 = dh ? a.rstd[2 * (size_t)r + 1] : 1.0f;
    auto branch = [&](int c) { return a.g1 ? ld_elem(y, c) * r1 * a.g1[c] : ld_elem(y, c); };
    auto sum = [&](int c) { return a.scale * ld_elem(x, c) + (gate ? gate[c] : 1.0f) * branch(c); };
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
      for (int c = threadIdx.x; c < a.dim; c += kNrThreads)
        s2 += (gate ? gate[c] : 1.0f) * total(c) * a.g1[c] * ld_elem(y, c);
      s2 = block_sum(s2, red) / a.dim;
    }
    for (int c = threadIdx.x; c < a.dim; c += kNrThreads) {
      const float t = total(c), w = (gate ? gate[c] : 1.0f) * t, yc = ld_elem(y, c);
      sums[c] += a.g1 ? w * yc * r1 : 0.0f;
      sums[a.dim + c] += t * branch(c);
      sums[2 * a.dim + c] += dh ? ld_elem(dh, c) * sum(c) * r2 : 0.0f;
      st_elem(static_cast<T*>(a.dy) + row, c, a.g1 ? r1 * (w * a.g1[c] - yc * r1 * r1 * s2) : w);
      st_elem(static_cast<T*>(a.dx) + row, c, a.scale * t);
    }
  }
}

// The parts' sums in order: of all of them for the two norms, of a gate's for
// its own (blockIdx.y; the norms' in the first).
__global__ void __launch_bounds__(kNrThreads) norm_res_join_kernel(NormResGradArgs a, int gates, int parts) {
  const int c = blockIdx.x * kNrThreads + threadIdx.x;
  if (c >= a.dim) return;
  auto add = [&](int which, size_t from, size_t n) {
    float s = 0.0f;
    for (size_t i = from; i < from + n; ++i) s += a.ws[(i * 3 + which) * a.dim + c];
    return s;
  };
  if (a.dgate)
    for (int g = blockIdx.y; g < gates; g += gridDim.y) a.dgate[(size_t)g * a.dim + c] = add(1, (size_t)g * parts, parts);
  if (blockIdx.y) return;
  if (a.dg1) a.dg1[c] = add(0, 0, (size_t)gates * parts);
  if (a.dg2) a.dg2[c] = add(2, 0, (size_t)gates * parts);
}

// Parts of each gate's rows.
int norm_res_parts(int rows, int gates) {
  const int per = rows / gates;
  int parts = (2 * 152 + gates - 1) / gates;
  if (parts > per) parts = per;
  return parts < 1 ? 1 : parts;
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
  const int g = gates ? gates : 1;
  return ((size_t)g * (rows ? mg::norm_res_parts(rows, g) : 1) * 3 * dim + 4) * sizeof(float);
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
  mg::NormResArgs a = {y, x, gamma_post, gate, gamma_pre, rows, dim, gates ? rows / gates : rows, scale, eps, x_out, h, rstd};
  if (dtype)
    mg::norm_res_kernel<mg::bf16><<<rows, mg::kNrThreads, 0, (cudaStream_t)stream>>>(a);
  else
    mg::norm_res_kernel<float><<<rows, mg::kNrThreads, 0, (cudaStream_t)stream>>>(a);
  return mg::op_end(fn, cudaGetLastError());
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
  mg::NormResGradArgs a = {dx_out, dh, y, x, rstd, gamma_post, gate, gamma_pre, rows, dim, 0, scale,
                           dy, dx, dgamma_post, dgate, dgamma_pre, static_cast<float*>(workspace)};
  cudaStream_t s = (cudaStream_t)stream;
  const int g = gates ? gates : 1;
  int parts = 0;
  cudaError_t e = cudaSuccess;
  if (rows) {
    a.gate_rows = rows / g;
    const int part_rows = (a.gate_rows + mg::norm_res_parts(rows, g) - 1) / mg::norm_res_parts(rows, g);
    parts = (a.gate_rows + part_rows - 1) / part_rows;
    if (dtype)
      mg::norm_res_grad_kernel<mg::bf16><<<dim3(g, parts), mg::kNrThreads, 0, s>>>(a, part_rows);
    else
      mg::norm_res_grad_kernel<float><<<dim3(g, parts), mg::kNrThreads, 0, s>>>(a, part_rows);
    e = cudaGetLastError();
  }
  if (e == cudaSuccess && (dgamma_post || dgate || dgamma_pre)) {
    mg::norm_res_join_kernel<<<dim3((dim + mg::kNrThreads - 1) / mg::kNrThreads, dgate ? std::min(g, 65535) : 1), mg::kNrThreads, 0,
                               s>>>(a, g, parts);
    e = cudaGetLastError();
  }
  return mg::op_end(fn, e);
}

// Matrix products grouped by expert (ragged row ranges), CUDA-core version and
// the entry points.
//
//   forward  y_e  = x_e  W_e        x [rows, d_in], W [E, d_in, d_out]
//   dX       dx_e = dy_e W_e^T
//   dW       dW_e = x_e^T dy_e      fp32, 0 for a group without rows
//
// The group boundaries are device data: every block reads them into shared
// memory and walks the same list of output tiles, so the host neither waits
// for the router nor launches one product per expert.
//
// This file's kernel runs fp32 (FFMA only), small bf16 products of widths that
// TMA cannot address (rows that are not multiples of 16 bytes), and every bf16
// product of a plan made with MG_GEMM=simt.  Bound by the FP32 units:
// 64x64 tiles (a group's last tile is half empty on average, so small ones) of
// 128 threads with 8x4 outputs each, two products per instruction.  fp32
// operands come by 4-byte asynchronous copies (any width and alignment,
// transposed on the way, zeros outside) two K steps ahead.  Shared memory is
// what limits it (three 16-byte reads per 32 products and thread): 4096 rows x
// 16 experts x 1001x517 in fp32 took 273 us with 4x4 outputs a thread and
// synchronous copies, 163 with 8x4 and the copies ahead, 140 with
// conflict-free transposed writes and no bounds in the inner tiles (30
// TFLOP/s); 8x8 outputs with 64 threads a tile read less but leave too few warps
// (161).
//
// A strict plan's forward carries the rounding errors of its sums, as the dense
// strict forward does (gemm_simt.cu): a ReLU behind it decides on the sign of
// the exact pre-activation.  The same tiles with 256 threads of 4x4 outputs; ten
// operations a product: 4096 rows x 16 x 1001x517 in 975 us, 123 plain.
//
// Where the tiles do not outnumber the resident blocks, each one's sum is split
// over several blocks through the workspace and joined in order by a
// second launch: 111 rows x 3148x1224, one group, dX in fp32: 126 us whole, 39 so.
#include <algorithm>
#include <cstdio>

#include "../../include/mg.h"
#include "common.cuh"
#include "group_epilogue.cuh"
#include "group_table.cuh"
#include "kernels.h"
#include "op_checks.h"

namespace mg {
namespace {

constexpr int S_T = 64;        // output tile
constexpr int S_K = 16;
constexpr int S_LD = S_T + 4;  // 16-byte aligned rows, transposed writes spread over the banks
constexpr int S_STAGES = 3;
// Threads of a block and resident blocks per SM: 8x4 outputs a thread, or 4x4
// whose sums carry their errors (4096 rows x 16 x 1001x517: 975 us; 8x4 of those at 12 warps an SM 1370).
constexpr int simt_threads(bool comp) { return comp ? 256 : 128; }
constexpr int simt_per_sm(bool comp) { return comp ? 3 : 4; }

struct SimtStage {
  float a[S_K][S_LD], b[S_K][S_LD];
};

// Fetch a K step of one operand into s[k][i]: element (i, k) is src[i * ld + k]
// (K_MAJOR) or src[k * ld + i]; zeros at i >= ni or k >= nk.
template <int NT, bool K_MAJOR, bool FULL>
__device__ __forceinline__ void simt_copy(float (&s)[S_K][S_LD], const float* src, long long ld, int ni, int nk) {
  // K_MAJOR: 8 k x 4 i per warp, whose transposed writes meet 32 banks
  const int k0 = K_MAJOR ? threadIdx.x % 8 : threadIdx.x / S_T;
  const int i0 = K_MAJOR ? threadIdx.x / 8 : threadIdx.x % S_T;
  constexpr int DI = NT / 8, DK = NT / S_T;   // steps of i (K_MAJOR) and of k
  const float* p = src + (K_MAJOR ? i0 * ld + k0 : k0 * ld + i0);
  const uint32_t dst = static_cast<uint32_t>(__cvta_generic_to_shared(&s[k0][i0]));
#pragma unroll
  for (int q = 0; q < S_T * S_K / NT; ++q) {
    constexpr int HALF = S_T / DI;                          // K_MAJOR: copies per 8 k
    const int dk = K_MAJOR ? q / HALF * 8 : q * DK, di = K_MAJOR ? q % HALF * DI : 0;
    const bool ok = FULL || (i0 + di < ni && k0 + dk < nk);
    const float* g = p + (K_MAJOR ? di * ld + dk : dk * ld);
    if (!FULL && !ok) g = src;
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst + (dk * S_LD + di) * 4), "l"(g),
                 "r"(ok ? 4 : 0)
                 : "memory");
  }
}
template <int NT, bool K_MAJOR>
__device__ __forceinline__ void simt_fetch(float (&s)[S_K][S_LD], const float* src, long long ld, int ni, int nk) {
  if (ni >= S_T && nk >= S_K) simt_copy<NT, K_MAJOR, true>(s, src, ld, ni, nk);
  else simt_copy<NT, K_MAJOR, false>(s, src, ld, ni, nk);
}
template <int NT, bool K_MAJOR>
__device__ __forceinline__ void simt_fetch(float (&s)[S_K][S_LD], const bf16* src, long long ld, int ni, int nk) {
#pragma unroll
  for (int q = 0; q < S_T * S_K / NT; ++q) {
    const int j = threadIdx.x + q * NT;
    const int k = K_MAJOR ? j % S_K : j / S_T, i = K_MAJOR ? j / S_K : j % S_T;
    s[k][i] = i < ni && k < nk ? __bfloat162float(K_MAJOR ? src[i * ld + k] : src[k * ld + i]) : 0.0f;
  }
}

__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  return (uint64_t)__float_as_uint(hi) << 32 | __float_as_uint(lo);
}
// Two fp32 FMAs in one instruction, each rounded as fmaf.
__device__ __forceinline__ void fma2(uint64_t& c, uint64_t a, uint64_t b) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(c) : "l"(a), "l"(b));
}

// The value of a compensated sum.  Where the sum itself has left the finite
// range its error term is no number, and the sum is the answer.
__device__ __forceinline__ float dot2_value(float s, float c) { return s - s == 0.0f ? __fadd_rn(s, c) : s; }

// splits > 1: part s of every tile's sum goes, as it is, to rows s * out_rows ..
// of g.ws.  COMP: sums that carry their rounding errors (dot2_step: ten
// operations a product instead of one; two values a part in g.ws, the sums and
// their errors).
template <typename T, int KIND, bool COMP>
__global__ void __launch_bounds__(simt_threads(COMP), simt_per_sm(COMP))
    group_simt_kernel(const GroupArgs g, int splits, long long out_rows) {
  constexpr int NT = simt_threads(COMP), RI = S_T * S_T / NT / 4;   // RI x 4 outputs a thread
  extern __shared__ int s_tab[];
  __shared__ __align__(16) SimtStage st[S_STAGES];
  GroupTable t;
  t.n = g.groups + (g.zero_rest ? 2 : 0);
  t.lo = s_tab;
  t.hi = s_tab + g.groups + 2;
  t.cum = s_tab + 2 * (g.groups + 2);
  if (threadIdx.x < 32) load_group_table(t, g.offsets, g.groups, g.rows, S_T);
  __syncthreads();
  const int K0 = KIND == GROUP_DX ? g.d_out : g.d_in;    // width of A's rows (FWD, DX)
  const int N = KIND == GROUP_DX ? g.d_in : g.d_out;
  const int tiles_n = (N + S_T - 1) / S_T;
  const int tiles_k = (g.d_in + S_T - 1) / S_T;          // DW: row tiles of each dW[e]
  const long long items = splits * (KIND == GROUP_DW ? (long long)g.groups * tiles_k * tiles_n
                                                     : (long long)t.cum[t.n - 1] * tiles_n);
  const T* A = static_cast<const T*>(g.A);
  const T* B = static_cast<const T*>(g.B);
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;   // rows ty*4.. (and 32+ty*4..), columns tx*4..
  int e = 0;
  for (long long item = blockIdx.x; item < items; item += gridDim.x) {
    const int part = (int)(item % splits);
    const long long tile = item / splits;
    const int mt = (int)(tile / tiles_n), n0 = (int)(tile % tiles_n) * S_T;
    int m0, m_end, K;
    long long krow0 = 0;
    if (KIND == GROUP_DW) {
      e = mt / tiles_k;
      m0 = (mt % tiles_k) * S_T;
      m_end = g.d_in;
      krow0 = t.lo[e];
      K = t.hi[e] - t.lo[e];
    } else {
      while (t.cum[e] <= mt) ++e;
      m0 = t.lo[e] + (mt - (e ? t.cum[e - 1] : 0)) * S_T;
      m_end = t.hi[e];
      K = e < g.groups ? K0 : 0;
    }
    const T* W = KIND == GROUP_DW || e >= g.groups ? B : B + (size_t)e * g.d_in * g.d_out;
    const int steps = (K + S_K - 1) / S_K;
    const int k_lo = (int)((long long)steps * part / splits) * S_K;
    K = min(K, (int)((long long)steps * (part + 1) / splits) * S_K);       // this part: [k_lo, K)
    auto fetch = [&](int k0) {
      SimtStage& q = st[k0 / S_K % S_STAGES];
      if (k0 < K) {
        if (KIND == GROUP_DW) {
          simt_fetch<NT, false>(q.a, A + (size_t)(krow0 + k0) * g.d_in + m0, g.d_in, m_end - m0, K - k0);
          simt_fetch<NT, false>(q.b, B + (size_t)(krow0 + k0) * g.d_out + n0, g.d_out, N - n0, K - k0);
        } else {
          simt_fetch<NT, true>(q.a, A + (size_t)m0 * K0 + k0, K0, m_end - m0, K - k0);
          if (KIND == GROUP_FWD) simt_fetch<NT, false>(q.b, W + (size_t)k0 * g.d_out + n0, g.d_out, N - n0, K - k0);
          else simt_fetch<NT, true>(q.b, W + (size_t)n0 * g.d_out + k0, g.d_out, N - n0, K - k0);
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    uint64_t acc2[4][4] = {};              // the thread's rows 2i and 2i + 1, column j
    float hi[4][4] = {}, lo[4][4] = {};    // COMP: sums and their errors
    __syncthreads();                       // the previous tile's last step has been read
    fetch(k_lo);
    fetch(k_lo + S_K);
    for (int k0 = k_lo; k0 < K; k0 += S_K) {
      asm volatile("cp.async.wait_group 1;" ::: "memory");
      __syncthreads();                     // this step is there for all, the one before is read
      fetch(k0 + 2 * S_K);
      const SimtStage& q = st[k0 / S_K % S_STAGES];
#pragma unroll
      for (int k = 0; k < S_K; ++k) {
        const float4 a0 = *reinterpret_cast<const float4*>(&q.a[k][ty * 4]);
        const float4 b0 = *reinterpret_cast<const float4*>(&q.b[k][tx * 4]);
        const float b[4] = {b0.x, b0.y, b0.z, b0.w};
        if constexpr (COMP) {
          const float a[4] = {a0.x, a0.y, a0.z, a0.w};
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) dot2_step(a[i], b[j], hi[i][j], lo[i][j]);
        } else {
          const float4 a1 = *reinterpret_cast<const float4*>(&q.a[k][32 + ty * 4]);
          const uint64_t a[4] = {pack2(a0.x, a0.y), pack2(a0.z, a0.w), pack2(a1.x, a1.y), pack2(a1.z, a1.w)};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint64_t bb = pack2(b[j], b[j]);
#pragma unroll
            for (int i = 0; i < 4; ++i) fma2(acc2[i][j], a[i], bb);
          }
        }
      }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
#pragma unroll
    for (int i = 0; i < RI; ++i) {
      const int m = m0 + (i & 4) * 8 + ty * 4 + (i & 3);
      if (m >= m_end) continue;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int n = n0 + tx * 4 + j;
        if (n >= N) continue;
        const size_t o = (size_t)((KIND == GROUP_DW ? (long long)e * g.d_in : 0) + m) * N + n;
        float x;
        if constexpr (COMP) {
          if (splits > 1) g.ws[(size_t)(splits + part) * out_rows * N + o] = lo[i][j];
          x = splits > 1 ? hi[i][j] : dot2_value(hi[i][j], lo[i][j]);
        } else {
          x = __uint_as_float((uint32_t)(acc2[i / 2][j] >> (i % 2 * 32)));
        }
        if (splits > 1) g.ws[(size_t)part * out_rows * N + o] = x;
        else if (KIND == GROUP_DW) static_cast<float*>(g.out)[o] = x;
        else group_epilogue<T>(g, o, x);
      }
    }
  }
}

// Tiles at most (every group may end inside one).
long long simt_tiles(int kind, int rows, int groups, int d_in, int d_out) {
  const long long tiles_n = ((kind == GROUP_DX ? d_in : d_out) + S_T - 1) / S_T;
  return tiles_n * (kind == GROUP_DW ? (long long)groups * ((d_in + S_T - 1) / S_T)
                                     : (long long)rows / S_T + std::min(groups, rows));
}

constexpr long long kSplitBlocks = 2 * 4 * 152;

// Parts of every tile's sum: as many as fill 4 x 152 blocks twice, of twelve K steps at
// least (on average over the groups in dW).
int simt_splits(int kind, int rows, int groups, int d_in, int d_out) {
  const long long tiles = simt_tiles(kind, rows, groups, d_in, d_out);
  const long long steps = (kind == GROUP_FWD ? d_in : kind == GROUP_DX ? d_out : rows / groups) / S_K;
  const long long s = std::min(std::min(kSplitBlocks / std::max(tiles, 1ll), steps / 12), 16ll);
  return s < 2 ? 1 : (int)s;
}

template <typename T, int KIND, bool COMP = false>
cudaError_t simt_launch(const GroupArgs& given, cudaStream_t s) {
  GroupArgs g = given;
  const int splits = g.ws ? simt_splits(KIND, g.rows, g.groups, g.d_in, g.d_out) : 1;
  if (splits > 1) g.zero_rest = 0;       // those rows are the join's
  const long long items = splits * (simt_tiles(KIND, g.rows, g.groups, g.d_in, g.d_out) +
                                    (g.zero_rest ? 2 : 0) * ((KIND == GROUP_DX ? g.d_in : g.d_out) / S_T + 1));
  const int slots = simt_per_sm(COMP) * device_sms();
  const int grid = (int)(items < slots ? items : slots);
  const size_t smem = (size_t)kGroupTableInts(g.groups) * sizeof(int);
  const long long out_rows = group_out_rows(KIND, g.rows, g.groups, g.d_in);
  group_simt_kernel<T, KIND, COMP><<<grid, simt_threads(COMP), smem, s>>>(g, splits, out_rows);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || splits == 1) return e;
  return group_join(given, splits, out_rows, KIND == GROUP_DX ? g.d_in : g.d_out, s);
}

template <typename T, int KIND>
__global__ void __launch_bounds__(256) group_join_kernel(const GroupArgs g, int splits, long long rows, int N) {
  dependency_wait();
  __shared__ int s_first, s_last;
  if (KIND != GROUP_DW) {
    if (threadIdx.x < 32) {
      int hi = 0;
      for (int e = threadIdx.x; e <= g.groups; e += 32) hi = max(hi, min(g.offsets[e], g.rows));
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) hi = max(hi, __shfl_xor_sync(0xffffffffu, hi, o));
      if (threadIdx.x == 0) {
        s_first = min(max(g.offsets[0], 0), g.rows);
        s_last = hi;
      }
    }
    __syncthreads();
  }
  const long long total = rows * N;
  for (long long i = blockIdx.x * 256ll + threadIdx.x; i < total; i += gridDim.x * 256ll) {
    bool inside = true;
    if (KIND != GROUP_DW) {
      const long long r = i / N;
      inside = r >= s_first && r < s_last;
      if (!inside && !g.zero_rest) continue;
    }
    float x = 0.0f;
    if (inside && g.compensated) {
      float err = 0.0f;
      for (int s = 0; s < splits; ++s) {
        const float h = g.ws[s * total + i], t = __fadd_rn(x, h), z = __fsub_rn(t, x);
        err = __fadd_rn(err, __fadd_rn(g.ws[(splits + s) * total + i],
                                       __fadd_rn(__fsub_rn(x, __fsub_rn(t, z)), __fsub_rn(h, z))));
        x = t;
      }
      x = dot2_value(x, err);
    } else if (inside) {
      for (int s = 0; s < splits; ++s) x += g.ws[s * total + i];
    }
    if (KIND == GROUP_DW) static_cast<float*>(g.out)[i] = x;
    else group_epilogue<T>(g, (size_t)i, x);
  }
}

template <typename T, int KIND>
cudaError_t join_launch(const GroupArgs& g, int splits, long long rows, int N, cudaStream_t s) {
  const long long blocks = (rows * N + 255) / 256;
  return launch_dependent(group_join_kernel<T, KIND>, (unsigned)std::min(blocks, 152ll * 8), 256, 0, s, g, splits, rows, N);
}

}  // namespace

// For these rows or fewer: in the forward and dX, s <= kSplitBlocks / tiles parts
// of at most S_T tiles / tiles_n rows; dW's parts grow with the rows.
size_t grouped_simt_split_bytes(int rows, int groups, int d_in, int d_out, bool compensated) {
  size_t most = 0;
  for (int kind : {GROUP_FWD, GROUP_DX, GROUP_DW}) {
    const bool dw = kind == GROUP_DW;
    const int s = simt_splits(kind, dw ? rows : std::min(rows, 1), groups, d_in, d_out);   // the most of any rows
    const int N = kind == GROUP_DX ? d_in : d_out;
    if (s < 2) continue;
    const long long part_rows = dw ? (long long)s * groups * d_in
                                   : std::min((long long)s * rows, kSplitBlocks * S_T / ((N + S_T - 1) / S_T));
    most = std::max<size_t>(most, (size_t)part_rows * N * (kind == GROUP_FWD && compensated ? 8 : 4));
  }
  return most;
}

cudaError_t group_join(const GroupArgs& g, int splits, long long rows, int N, cudaStream_t s) {
  if (g.kind == GROUP_DW) return join_launch<float, GROUP_DW>(g, splits, rows, N, s);
  if (g.type == DT_F32)
    return g.kind == GROUP_FWD ? join_launch<float, GROUP_FWD>(g, splits, rows, N, s)
                               : join_launch<float, GROUP_DX>(g, splits, rows, N, s);
  return g.kind == GROUP_FWD ? join_launch<bf16, GROUP_FWD>(g, splits, rows, N, s)
                             : join_launch<bf16, GROUP_DX>(g, splits, rows, N, s);
}

int grouped_launches(const GroupArgs& g) {
  if (g.rows == 0 && g.kind != GROUP_DW) return 0;
  if (grouped_tc_eligible(g)) return grouped_tc_launches(g);
  return g.ws && simt_splits(g.kind, g.rows, g.groups, g.d_in, g.d_out) > 1 ? 2 : 1;
}

cudaError_t grouped_gemm(const GroupArgs& g, cudaStream_t s) {
  if (g.rows == 0 && g.kind != GROUP_DW) return cudaSuccess;
  if (grouped_tc_eligible(g)) return grouped_gemm_tc(g, s);
  if (g.type == DT_F32) {
    if (g.kind == GROUP_FWD)
      return g.compensated ? simt_launch<float, GROUP_FWD, true>(g, s) : simt_launch<float, GROUP_FWD>(g, s);
    if (g.kind == GROUP_DX) return simt_launch<float, GROUP_DX>(g, s);
    return simt_launch<float, GROUP_DW>(g, s);
  }
  if (g.kind == GROUP_FWD) return simt_launch<bf16, GROUP_FWD>(g, s);
  if (g.kind == GROUP_DX) return simt_launch<bf16, GROUP_DX>(g, s);
  return simt_launch<bf16, GROUP_DW>(g, s);
}

}  // namespace mg

// ============================================================================
namespace {

using mg::op_fail;

constexpr size_t kErrorBytes = 256;   // of a workspace: begins with the error word; then the scratch

size_t workspace_bytes(int rows, int groups, int d_in, int d_out) {
  return kErrorBytes + mg::grouped_scratch_bytes(rows, groups, d_in, d_out, false);
}

mg_status grouped_call(const char* fn, mg::GroupKind kind, int dtype, const void* a, const void* b,
                       const int* offsets, int rows, int groups, int d_in, int d_out, void* out, void* ws,
                       size_t ws_bytes, mg_stream_t stream) {
  if (dtype != 0 && dtype != 1) return op_fail(MG_ERR_INVALID_ARG, "%s: dtype must be 0 or 1", fn);
  if (rows < 0 || groups < 1 || d_in < 1 || d_out < 1)
    return op_fail(MG_ERR_SHAPE, "%s: bad sizes (rows %d, groups %d, d_in %d, d_out %d)", fn, rows, groups, d_in,
                   d_out);
  if (rows > mg::kMaxWidth || d_in > mg::kMaxWidth || d_out > mg::kMaxWidth)
    return op_fail(MG_ERR_SHAPE, "%s: rows, d_in and d_out must be at most 2^30 (got %d, %d, %d)", fn, rows, d_in,
                   d_out);
  if (groups > mg::kMaxGroups)
    return op_fail(MG_ERR_UNSUPPORTED, "%s: at most %d groups (got %d)", fn, mg::kMaxGroups, groups);
  const bool rows_needed = rows > 0;
  const bool dw = kind == mg::GROUP_DW;
  if (!offsets || !ws || (rows_needed && !a) || (!b && (rows_needed || !dw)) || (!out && (rows_needed || dw)))
    return op_fail(MG_ERR_INVALID_ARG, "%s: a pointer is NULL", fn);
  const size_t need = workspace_bytes(rows, groups, d_in, d_out);
  if (ws_bytes < need)
    return op_fail(MG_ERR_INVALID_ARG, "%s: the workspace needs %zu bytes, %zu given", fn, need, ws_bytes);
  mg_status st = mg::op_begin(fn, {{a, 16}, {b, 16}, {offsets, 4}, {out, 16}, {ws, 16}});
  if (st != MG_OK) return st;
  mg::GroupArgs g;
  g.kind = kind;
  g.type = (mg::DType)dtype;
  g.rows = rows;
  g.groups = groups;
  g.d_in = d_in;
  g.d_out = d_out;
  g.offsets = offsets;
  g.A = a;
  g.B = b;
  g.out = out;
  g.err = static_cast<int*>(ws);
  g.ws = reinterpret_cast<float*>(static_cast<char*>(ws) + kErrorBytes);
  return mg::op_end(fn, mg::grouped_gemm(g, (cudaStream_t)stream));
}

}  // namespace

extern "C" size_t mg_grouped_linear_workspace_bytes(int rows, int groups, int d_in, int d_out) {
  if (rows < 0 || groups < 1 || groups > mg::kMaxGroups || d_in < 1 || d_out < 1 || rows > mg::kMaxWidth ||
      d_in > mg::kMaxWidth || d_out > mg::kMaxWidth)
    return 0;
  return workspace_bytes(rows, groups, d_in, d_out);
}

extern "C" mg_status mg_grouped_linear_forward(int dtype, const void* x, const int* offsets, int rows, int groups,
                                               int d_in, int d_out, const void* w, void* y, void* ws,
                                               size_t ws_bytes, mg_stream_t stream) {
  return grouped_call("mg_grouped_linear_forward", mg::GROUP_FWD, dtype, x, w, offsets, rows, groups, d_in, d_out,
                      y, ws, ws_bytes, stream);
}

extern "C" mg_status mg_grouped_linear_backward_input(int dtype, const void* dy, const int* offsets, int rows,
                                                      int groups, int d_in, int d_out, const void* w, void* dx,
                                                      void* ws, size_t ws_bytes, mg_stream_t stream) {
  return grouped_call("mg_grouped_linear_backward_input", mg::GROUP_DX, dtype, dy, w, offsets, rows, groups, d_in,
                      d_out, dx, ws, ws_bytes, stream);
}

extern "C" mg_status mg_grouped_linear_backward_weight(int dtype, const void* x, const void* dy, const int* offsets,
                                                       int rows, int groups, int d_in, int d_out, float* dw,
                                                       void* ws, size_t ws_bytes, mg_stream_t stream) {
  return grouped_call("mg_grouped_linear_backward_weight", mg::GROUP_DW, dtype, x, dy, offsets, rows, groups, d_in,
                      d_out, dw, ws, ws_bytes, stream);
}

extern "C" mg_status mg_grouped_linear_status(const void* ws, mg_stream_t stream) {
  const char* fn = "mg_grouped_linear_status";
  if (!ws) return op_fail(MG_ERR_INVALID_ARG, "%s: workspace is NULL", fn);
  const mg_status st = mg::op_begin(fn, {{ws, 16}});
  if (st != MG_OK) return st;
  int gave_up = 0;
  cudaError_t e = cudaMemcpyAsync(&gave_up, ws, sizeof gave_up, cudaMemcpyDeviceToHost, (cudaStream_t)stream);
  if (e == cudaSuccess) e = cudaStreamSynchronize((cudaStream_t)stream);
  if (e != cudaSuccess) return mg::op_end(fn, e);
  if (gave_up)
    return op_fail(MG_ERR_TIMEOUT, "%s: a device-side wait gave up in a call with this workspace: its results are invalid",
                   fn);
  return MG_OK;
}

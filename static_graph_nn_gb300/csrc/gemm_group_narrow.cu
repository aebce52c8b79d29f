// Products grouped by expert with a few rows per group (decoding): forward and
// input gradient.
//
// Such a call reads every used expert's weights once and does little else, so
// it is bound by DRAM.  The weights take the M side of the MMA (128 output
// columns on the accumulator's lanes) and up to 32 rows of the group the N
// side: D[n, t] = sum_k W[k, n] x[t, k], so that no tensor work is spent on
// rows that do not exist and the stages hold weights, not padding (16 of 20
// KB).  Seven stages, 112 KB of weights in flight per SM (24 rows x 8 experts x
// 2048x8192 with cold caches, a graph launch included: 52.0 us, and 52.3 with five).
//
// Where the tiles are fewer than half the SMs, a cluster of two or four CTAs
// shares a tile, each with a part of K; the partial sums go to the first CTA's
// shared memory and are added in CTA order: the same bits in every run.
// (Cutting all tiles' K blocks into even stretches, joined through global
// memory, lost more in the joins than the evenness gave: 34 against 21 us for 16
// experts x 2048x1024.)
//
// Called in a loop, where L2 keeps some of the weights, that product takes 42 us
// (6.1 TB/s); with cold caches 52, and 73 on the 256-row tiles of the pair kernel.
//
// Warps: 0 TMA producer, 1 MMA issuer, 2-5 epilogue (one accumulator lane
// quarter each).  Every wait is bounded.
#include <cuda.h>

#include "common.cuh"
#include "group_epilogue.cuh"
#include "group_table.cuh"
#include "group_tma.h"
#include "kernels.h"
#include "op_checks.h"
#include "tc_common.cuh"
#include "tc_pair.cuh"

namespace mg {
namespace {

using namespace tc;

constexpr int N_M = 128;           // output columns of a tile
constexpr int N_T = 32;            // rows of a tile
constexpr int N_BK = 64;
constexpr int N_STAGES = 7;
constexpr int N_THREADS = 192;
constexpr int N_SPLIT = 4;         // CTAs of a tile at most
constexpr int kMinBlocks = 8;      // K blocks per CTA worth a split
constexpr uint32_t N_W_BYTES = N_M * N_BK * 2;
constexpr uint32_t N_X_BYTES = N_T * N_BK * 2;
constexpr int N_PANEL = 64 * N_BK * 2;

struct NarrowParams {
  GroupArgs g;
  int N, tiles_n, k_blocks;
  int split;         // CTAs of a tile (a cluster)
};

struct NarrowTile {
  int e, m0, rows, n0;   // group, first row, rows (at most N_T), first column
};

__device__ __forceinline__ NarrowTile narrow_tile(const NarrowParams& P, const GroupTable& t, int tile, int& e) {
  NarrowTile r;
  const int mt = tile / P.tiles_n, nt = tile - mt * P.tiles_n;
  if (e >= t.n || (e > 0 && t.cum[e - 1] > mt)) e = 0;
  while (t.cum[e] <= mt) ++e;
  r.e = e;
  r.m0 = t.lo[e] + (mt - (e ? t.cum[e - 1] : 0)) * N_T;
  r.rows = min(N_T, t.hi[e] - r.m0);
  r.n0 = nt * N_M;
  return r;
}

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::
          "r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

template <int KIND>
__global__ void __launch_bounds__(N_THREADS, 1)
    group_narrow_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                        const NarrowParams P) {
  constexpr bool W_MN = KIND == GROUP_FWD;
  constexpr uint32_t TMEM_COLS = 2 * N_T;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sW = smem;
  uint8_t* sX = smem + N_STAGES * N_W_BYTES;
  float* s_out = reinterpret_cast<float*>(sX + N_STAGES * N_X_BYTES);   // [N_T][N_M], then the other CTAs' partials
  uint64_t* full = reinterpret_cast<uint64_t*>(s_out + P.split * N_T * N_M);
  uint64_t* empty = full + N_STAGES;
  uint64_t* tfull = empty + N_STAGES;
  uint64_t* tempty = tfull + 2;
  uint64_t* pfull = tempty + 2;        // first CTA: the others' partials are there
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(pfull + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  GroupTable t;
  t.n = P.g.groups;
  t.lo = reinterpret_cast<int*>(tmem_slot + 2);
  t.hi = t.lo + P.g.groups + 2;
  t.cum = t.hi + P.g.groups + 2;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < N_STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], 128);
    }
    mbar_init(pfull, 128 * (P.split > 1 ? P.split - 1 : 1));
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) tmem_alloc(tmem_slot, TMEM_COLS);
  if (warp == 2) load_group_table(t, P.g.offsets, P.g.groups, P.g.rows, N_T);
  tc_fence_before();
  __syncthreads();
  if (P.split > 1) cluster_sync();     // the other CTAs' barriers too
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int rank = blockIdx.x % P.split, n_tiles = t.cum[t.n - 1] * P.tiles_n;
  const int first = blockIdx.x / P.split, step = gridDim.x / P.split;
  const int k_lo = P.k_blocks * rank / P.split, k_hi = P.k_blocks * (rank + 1) / P.split;

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0, e = 0;
      uint32_t phase = 0;
      for (int tile = first; tile < n_tiles && !*abort_flag; tile += step) {
        const NarrowTile T = narrow_tile(P, t, tile, e);
        for (int k = k_lo; k < k_hi; ++k) {
          if (!mbar_wait(&empty[stage], phase ^ 1)) { *abort_flag = 1; atomicExch(P.g.err, 1); break; }
          mbar_expect_tx(&full[stage], N_W_BYTES + N_X_BYTES);
          uint8_t* w = sW + stage * N_W_BYTES;
          const int k0 = k * N_BK;
          if (W_MN) {
            tma_load_3d(w, &tmW, &full[stage], T.n0, k0, T.e);
            tma_load_3d(w + N_PANEL, &tmW, &full[stage], T.n0 + 64, k0, T.e);
          } else {
            tma_load_3d(w, &tmW, &full[stage], k0, T.n0, T.e);
          }
          tma_load_2d(sX + stage * N_X_BYTES, &tmX, &full[stage], k0, T.m0);
          if (++stage == N_STAGES) { stage = 0; phase ^= 1; }
        }
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t idesc = instr_desc(N_M, N_T, W_MN ? 1 : 0, 0);
      int stage = 0, it = 0;
      uint32_t phase = 0;
      for (int tile = first; tile < n_tiles && !*abort_flag; tile += step, ++it) {
        const int acc = it & 1;
        if (!mbar_wait(&tempty[acc], ((uint32_t)(it >> 1) & 1u) ^ 1)) { *abort_flag = 1; atomicExch(P.g.err, 1); break; }
        tc_fence_after();
        const uint32_t d = tmem_base + (uint32_t)(acc * N_T);
        bool ok = true;
        for (int k = k_lo; k < k_hi; ++k) {
          if (!mbar_wait(&full[stage], phase)) { ok = false; break; }
          tc_fence_after();
          const uint32_t w = smem_u32(sW + stage * N_W_BYTES);
          const uint32_t x = smem_u32(sX + stage * N_X_BYTES);
#pragma unroll
          for (int q = 0; q < N_BK / 16; ++q) {
            const uint64_t wd = W_MN ? smem_desc(w + q * 2048, N_PANEL, 1024) : smem_desc(w + q * 32, 16, 1024);
            mma_bf16(d, wd, smem_desc(x + q * 32, 16, 1024), idesc, (k > k_lo || q) ? 1u : 0u);
          }
          mma_commit(&empty[stage]);
          if (++stage == N_STAGES) { stage = 0; phase ^= 1; }
        }
        if (!ok) { *abort_flag = 1; atomicExch(P.g.err, 1); break; }
        mma_commit(&tfull[acc]);
      }
    }
  } else {
    const int quarter = warp & 3;                 // TMEM lanes this warp may access
    const int m = quarter * 32 + lane;            // output column in the tile
    if (P.g.zero_rest) {
      // rows of no group: the epilogue of a zero, the rows dealt over the CTAs
      const int first = t.lo[0], rest = first + P.g.rows - t.hi[t.n - 1];
      for (int r = blockIdx.x; r < rest; r += gridDim.x) {
        const int row = r < first ? r : t.hi[t.n - 1] + r - first;
        for (int c = (warp - 2) * 32 + lane; c < P.N; c += 128) group_epilogue<bf16>(P.g, (size_t)row * P.N + c, 0.0f);
      }
    }
    int it = 0, e = 0;
    for (int tile = first; tile < n_tiles; tile += step, ++it) {
      const NarrowTile T = narrow_tile(P, t, tile, e);
      const int acc = it & 1;
      uint32_t bad = !mbar_wait(&tfull[acc], (uint32_t)(it >> 1) & 1u) || *abort_flag;
      // the four warps leave together
      asm volatile(
          "{\n.reg .pred p, q;\nsetp.ne.u32 q, %0, 0;\nbar.red.or.pred p, 1, 128, q;\nselp.u32 %0, 1, 0, p;\n}\n"
          : "+r"(bad)
          :
          : "memory");
      if (bad) {
        *abort_flag = 1;
        if (lane == 0) atomicExch(P.g.err, 1);
        break;
      }
      tc_fence_after();
      float v[32];
      tmem_ld32(tmem_base + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(acc * N_T), v);
      tc_fence_before();
      mbar_arrive(&tempty[acc]);
      // this thread's column, row by row, in shared memory: the loops over the
      // rows stay loops (unrolled over registers, the epilogue's code was long
      // enough for its instruction fetches to cost 6 us)
      float* col = s_out + m;
#pragma unroll
      for (int q = 0; q < 32; ++q) col[q * N_M] = v[q];
      if (P.split > 1) {
        // (a cluster that shares a tile has no second one: the slots are used once)
        if (rank > 0) {
          const uint32_t dst = map_to(s_out + rank * N_T * N_M + m, 0);
          for (int q = 0; q < T.rows; ++q)
            asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(dst + q * N_M * 4), "f"(col[q * N_M]) : "memory");
          mbar_arrive_remote_release(map_to(pfull, 0));
          break;
        }
        if (!mbar_wait_cluster(pfull, 0)) {
          *abort_flag = 1;
          atomicExch(P.g.err, 1);
          break;
        }
        for (int q = 0; q < T.rows; ++q) {
          float sum = col[q * N_M];
          for (int c = 1; c < P.split; ++c) sum += col[(c * N_T + q) * N_M];
          col[q * N_M] = sum;
        }
      }
      if (T.n0 + m < P.N)
        for (int q = 0; q < T.rows; ++q)
          group_epilogue<bf16>(P.g, (size_t)(T.m0 + q) * P.N + T.n0 + m, col[q * N_M]);
    }
  }

  if (*abort_flag) drain_in_flight();
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (P.split > 1) cluster_sync();     // no CTA leaves while another writes to it
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, TMEM_COLS);
  }
}

size_t narrow_smem(int groups, int split) {
  return 1024 + (size_t)N_STAGES * (N_W_BYTES + N_X_BYTES) + (size_t)split * N_T * N_M * 4 +
         (2 * N_STAGES + 5) * 8 + 8 + (size_t)kGroupTableInts(groups) * 4;
}

template <int KIND>
cudaError_t launch_narrow(const GroupArgs& g, cudaStream_t s) {
  const int k = KIND == GROUP_FWD ? g.d_in : g.d_out;
  NarrowParams P;
  P.g = g;
  P.N = KIND == GROUP_FWD ? g.d_out : g.d_in;
  P.tiles_n = (P.N + N_M - 1) / N_M;
  P.k_blocks = (k + N_BK - 1) / N_BK;
  CUtensorMap mw, mx;
  const bool ok = (KIND == GROUP_FWD ? group_map(&mw, g.B, g.groups, g.d_in, g.d_out, g.ldb, 64, N_BK)
                                     : group_map(&mw, g.B, g.groups, g.d_in, g.d_out, g.ldb, N_BK, N_M)) &&
                  group_map(&mx, g.A, 0, g.rows, k, g.lda, N_BK, N_T);
  if (!ok) return cudaErrorInvalidValue;
  const cudaError_t attr = cudaFuncSetAttribute(    // of this device's context: set in every call
      group_narrow_kernel<KIND>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)narrow_smem(kMaxGroups, N_SPLIT));
  if (attr != cudaSuccess) return attr;
  const int sms = device_sms();
  // tiles at most: every group may end inside one (split > 1 relies on it: one
  // tile per cluster)
  const long long tiles = ((long long)g.rows / N_T + (g.groups < g.rows ? g.groups : g.rows)) * P.tiles_n;
  P.split = 1;
  while (P.split < N_SPLIT && tiles * P.split * 2 <= sms && P.k_blocks / (P.split * 2) >= kMinBlocks) P.split *= 2;
  const long long most = tiles * P.split;
  const int grid = most < sms ? (int)most : sms / P.split * P.split;
  const size_t smem = narrow_smem(g.groups, P.split);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(N_THREADS);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = P.split;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, group_narrow_kernel<KIND>, mw, mx, P);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace

// Up to 16 rows per group on average: a tile then holds most groups whole.  Up
// to there this kernel is 1.0 to 1.4 times as fast as the pair kernel (cold
// caches, 3, 8 and 16 rows per group: 52, 52, 53 against 73, 57, 58 us for 8 x
// 2048x8192; 22, 24, 25 against 26, 26, 26 for 64 x 1024x512); beyond, groups of
// several tiles read their weights again (32 rows: 66 against 59, 28 against 27).
bool grouped_narrow(const GroupArgs& g) {
  const long long n = g.kind == GROUP_FWD ? g.d_out : g.d_in;
  const bool fits = ((long long)g.rows / N_T + g.groups) * ((n + N_M - 1) / N_M) <= 0x3fffffff;   // 32-bit tiles
  return fits && g.kind != GROUP_DW && (long long)g.rows <= 16ll * g.groups;
}

cudaError_t grouped_gemm_narrow(const GroupArgs& g, cudaStream_t s) {
  return g.kind == GROUP_FWD ? launch_narrow<GROUP_FWD>(g, s) : launch_narrow<GROUP_DX>(g, s);
}

}  // namespace mg

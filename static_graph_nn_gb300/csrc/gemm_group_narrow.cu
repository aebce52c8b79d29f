// Products grouped by expert with a few rows per group (decoding): forward and
// input gradient.
//
// Such a call reads every used expert's weights once and does little else, so
// it is bound by DRAM.  The weights take the M side of the MMA (128 output
// columns on the accumulator's lanes) and up to 32 rows of the group the N
// side: D[n, t] = sum_k W[k, n] x[t, k], so that no tensor work is spent on
// rows that do not exist and the stages hold weights, not padding (16 of 20
// KB).  Seven stages, 112 KB of weights in flight per SM: with ten the same call
// took 58 us, with six 52, with seven 51.
//
// Work is cut evenly: as many rounds of whole tiles as every CTA can take (in
// a round the CTAs stream neighbouring columns), and the K blocks of the tiles
// left over form one line of which each CTA takes an equal stretch (at least
// kMinBlocks).  A tile that CTAs share is summed in fp32 from their partials in
// the workspace, by the CTA that arrives last, in CTA order: the same bits in
// every run.  The stretches come first, so that the sums hide under the rounds.
// 24 rows x 8 experts x 2048x8192 (512 tiles for 152 SMs), weights in DRAM,
// with a graph launch: 67 us on the pair kernel's whole tiles, 57.6 with the
// line over all tiles, 51 so.
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
constexpr int N_CTAS = 152;        // at most
constexpr int kMinBlocks = 8;      // K blocks per CTA worth a split
constexpr uint32_t N_W_BYTES = N_M * N_BK * 2;
constexpr uint32_t N_X_BYTES = N_T * N_BK * 2;
constexpr int N_PANEL = 64 * N_BK * 2;

struct NarrowParams {
  GroupArgs g;
  int N, tiles_n, k_blocks;
  int* counters;     // per tile, zero between calls
  float* part;       // [CTA][2][N_T][N_M]
};

// This CTA's pieces of work: its stretch of the shared tiles' line of K blocks,
// tile by tile, then a whole tile of every round.
struct Pieces {
  int kb, whole;            // K blocks per tile; tiles [0, whole) are not shared
  int ctas;                 // that share the line
  long long total, begin, end, at;
  int next_whole;
  int tile, k_lo, n;        // the current piece
  bool shared;
  __device__ __forceinline__ Pieces(int n_tiles, int kb_) : kb(kb_) {
    const int G = gridDim.x, c = blockIdx.x;
    whole = n_tiles / G * G;
    total = (long long)(n_tiles - whole) * kb;
    const long long most = total / kMinBlocks;
    ctas = (int)min((long long)G, most < 1 ? 1ll : most);
    begin = c < ctas ? start(c) : total;
    end = c < ctas ? start(c + 1) : total;
    at = begin;
    next_whole = c;
  }
  __device__ __forceinline__ long long start(int c) const { return total * c / ctas; }
  __device__ __forceinline__ int owner(long long block) const { return (int)(((block + 1) * ctas - 1) / total); }
  __device__ __forceinline__ bool next() {
    if (at < end) {
      const int t = (int)(at / kb);
      k_lo = (int)(at - (long long)t * kb);
      n = (int)min((long long)(kb - k_lo), end - at);
      tile = whole + t;
      shared = n < kb;
      at += n;
      return true;
    }
    if (next_whole >= whole) return false;
    tile = next_whole;
    next_whole += gridDim.x;
    k_lo = 0;
    n = kb;
    shared = false;
    return true;
  }
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
  uint64_t* full = reinterpret_cast<uint64_t*>(sX + N_STAGES * N_X_BYTES);
  uint64_t* empty = full + N_STAGES;
  uint64_t* tfull = empty + N_STAGES;
  uint64_t* tempty = tfull + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tempty + 2);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  int* s_last = reinterpret_cast<int*>(tmem_slot + 2);
  GroupTable t;
  t.n = P.g.groups;
  t.lo = s_last + 2;
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
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) tmem_alloc(tmem_slot, TMEM_COLS);
  if (warp == 2) load_group_table(t, P.g.offsets, P.g.groups, P.g.rows, N_T);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int kb = P.k_blocks;
  Pieces W(t.cum[t.n - 1] * P.tiles_n, kb);      // each warp walks its own copy

  if (warp == 0) {
    if (lane == 0) {
      int stage = 0, e = 0;
      uint32_t phase = 0;
      while (!*abort_flag && W.next()) {
        const NarrowTile T = narrow_tile(P, t, W.tile, e);
        for (int k = W.k_lo; k < W.k_lo + W.n; ++k) {
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
      for (; !*abort_flag && W.next(); ++it) {
        const int acc = it & 1;
        if (!mbar_wait(&tempty[acc], ((uint32_t)(it >> 1) & 1u) ^ 1)) { *abort_flag = 1; atomicExch(P.g.err, 1); break; }
        tc_fence_after();
        const uint32_t d = tmem_base + (uint32_t)(acc * N_T);
        bool ok = true;
        for (int k = 0; k < W.n; ++k) {
          if (!mbar_wait(&full[stage], phase)) { ok = false; break; }
          tc_fence_after();
          const uint32_t w = smem_u32(sW + stage * N_W_BYTES);
          const uint32_t x = smem_u32(sX + stage * N_X_BYTES);
#pragma unroll
          for (int q = 0; q < N_BK / 16; ++q) {
            const uint64_t wd = W_MN ? smem_desc(w + q * 2048, N_PANEL, 1024) : smem_desc(w + q * 32, 16, 1024);
            mma_bf16(d, wd, smem_desc(x + q * 32, 16, 1024), idesc, (k | q) ? 1u : 0u);
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
    for (; W.next(); ++it) {
      const NarrowTile T = narrow_tile(P, t, W.tile, e);
      const int acc = it & 1;
      uint32_t bad = mbar_wait(&tfull[acc], (uint32_t)(it >> 1) & 1u) ? *abort_flag != 0 : 1;
      // the four warps leave together: they meet at barriers below
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
      bool store = true;
      if (W.shared) {
        // a shared tile: leave the partial; the last of its CTAs adds them all
        const long long b0 = (long long)(W.tile - W.whole) * kb;      // the tile's part of the line
        float* mine = P.part + ((size_t)blockIdx.x * 2 + (W.begin >= b0 ? 0 : 1)) * N_T * N_M + m;
#pragma unroll
        for (int q = 0; q < 32; ++q)
          if (q < T.rows) mine[q * N_M] = v[q];
        __threadfence();
        asm volatile("bar.sync 1, 128;" ::: "memory");
        const int c0 = W.owner(b0), c1 = W.owner(b0 + kb - 1);
        if (warp == 2 && lane == 0) *s_last = atomicAdd(&P.counters[W.tile - W.whole], 1) == c1 - c0;
        asm volatile("bar.sync 1, 128;" ::: "memory");
        store = *s_last != 0;
        if (store) {
          __threadfence();
          if (warp == 2 && lane == 0) P.counters[W.tile - W.whole] = 0;
#pragma unroll
          for (int q = 0; q < 32; ++q) v[q] = 0.0f;
          for (int c = c0; c <= c1; ++c) {
            const int slot = W.start(c) >= b0 ? 0 : 1;   // the tile is c's first piece, or its last
            const float* p = P.part + ((size_t)c * 2 + slot) * N_T * N_M + m;
#pragma unroll
            for (int q = 0; q < 32; ++q)
              if (q < T.rows) v[q] += __ldcg(p + q * N_M);
          }
        }
      }
      if (store && T.n0 + m < P.N) {
#pragma unroll
        for (int q = 0; q < 32; ++q)
          if (q < T.rows) group_epilogue<bf16>(P.g, (size_t)(T.m0 + q) * P.N + T.n0 + m, v[q]);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem_base, TMEM_COLS);
  }
}

size_t narrow_smem(int groups) {
  return 1024 + (size_t)N_STAGES * (N_W_BYTES + N_X_BYTES) + (2 * N_STAGES + 4) * 8 + 16 +
         (size_t)kGroupTableInts(groups) * 4;
}

long long narrow_tiles(int rows, int groups, int N) {
  return ((long long)rows / N_T + groups) * ((N + N_M - 1) / N_M);
}

template <int KIND>
cudaError_t launch_narrow(const GroupArgs& g, cudaStream_t s) {
  const int k = KIND == GROUP_FWD ? g.d_in : g.d_out;
  NarrowParams P;
  P.g = g;
  P.N = KIND == GROUP_FWD ? g.d_out : g.d_in;
  P.tiles_n = (P.N + N_M - 1) / N_M;
  P.k_blocks = (k + N_BK - 1) / N_BK;
  P.counters = g.ws;
  const size_t n_counters = (size_t)narrow_tiles(g.rows, g.groups, g.d_in > g.d_out ? g.d_in : g.d_out);
  P.part = reinterpret_cast<float*>(reinterpret_cast<char*>(P.counters) + (n_counters * 4 + 255) / 256 * 256);
  CUtensorMap mw, mx;
  const bool ok = (KIND == GROUP_FWD ? group_map(&mw, g.B, g.groups, g.d_in, g.d_out, 64, N_BK)
                                     : group_map(&mw, g.B, g.groups, g.d_in, g.d_out, N_BK, N_M)) &&
                  group_map(&mx, g.A, 0, g.rows, k, N_BK, N_T);
  if (!ok) return cudaErrorInvalidValue;
  static const cudaError_t attr = cudaFuncSetAttribute(
      group_narrow_kernel<KIND>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)narrow_smem(kMaxGroups));
  if (attr != cudaSuccess) return attr;
  const int sms = device_sms();
  const long long most = narrow_tiles(g.rows, g.groups, P.N) * P.k_blocks / kMinBlocks;
  int grid = sms < N_CTAS ? sms : N_CTAS;
  if (most < grid) grid = most < 1 ? 1 : (int)most;
  group_narrow_kernel<KIND><<<grid, N_THREADS, narrow_smem(g.groups), s>>>(mw, mx, P);
  return cudaGetLastError();
}

}  // namespace

// Up to 16 rows per group on average: a tile then holds most groups whole.
// More rows make several tiles of one group re-read its weights from L2, and
// the 256-row tiles of the pair kernel win (@@).
bool grouped_narrow(const GroupArgs& g) {
  return g.kind != GROUP_DW && g.ws && (long long)g.rows <= 16ll * g.groups;
}

size_t grouped_narrow_ws_bytes(int rows, int groups, int d_in, int d_out) {
  if ((long long)rows > 16ll * groups) return 0;
  const size_t counters = (size_t)narrow_tiles(rows, groups, d_in > d_out ? d_in : d_out);
  return (counters * 4 + 255) / 256 * 256 + (size_t)N_CTAS * 2 * N_T * N_M * 4;
}

cudaError_t grouped_gemm_narrow(const GroupArgs& g, cudaStream_t s) {
  return g.kind == GROUP_FWD ? launch_narrow<GROUP_FWD>(g, s) : launch_narrow<GROUP_DX>(g, s);
}

}  // namespace mg

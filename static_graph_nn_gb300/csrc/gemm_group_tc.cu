// Matrix products grouped by expert on the tensor cores: 256x256 output tiles
// on CTA pairs (tcgen05 cta_group::2, bf16 operands, fp32 accumulators in
// TMEM), the arrangement of the dense SM-pair GEMM (gemm_tc2.cu) with a ragged
// list of tiles.
//
//   forward  y_e  = x_e  W_e      A = x  K-major,  B = W_e N-major
//   dX       dx_e = dy_e W_e^T    A = dy K-major,  B = W_e K-major
//   dW       dW_e = x_e^T dy_e    A = x  M-major,  B = dy  N-major, fp32 out
//
// Bound by the tensor cores (2 T K N flops against x + W + y bytes) once the
// groups have a few hundred rows.
//
// Ragged rows.  Every CTA reads the offsets into shared memory and walks the
// same list of tiles (group by group, columns fastest), so one persistent
// launch serves all groups.  A forward tile's last rows may belong to the next
// group: they are computed into accumulator rows of their own and not stored.
// W is addressed as a three-dimensional tensor, so a K block past its last row
// reads zeros, not the next expert's weights.  In dW the groups' rows are the
// K dimension, and the last 64-row block of a group may hold rows of the next
// one: that block has a buffer and barriers of its own beside the ring, and a
// warp of each CTA overwrites the foreign rows with zeros in shared memory (both
// operands: a NaN there would survive a zero factor), fences them to the async
// proxy and only then reports it full.  It is loaded while the tile's first
// blocks are multiplied and comes last in the sum, so its extra steps take no
// time.  (16384 rows x 8 experts x 2048x8192, ncu: in the producer's own loop 404
// us, by a warp of its own but in the ring 377, so 352; groups of whole blocks
// 350.)
//
// Long sums.  The tensor core truncates each addition to its fp32 accumulator,
// an error that grows with the number of additions: 2.3e-6 of the result at
// 2048 rows a group (in the 2-norm).  dW is stored in fp32, so there every G_SEG
// K blocks start a new accumulator, and the epilogue adds them in registers,
// rounding to nearest: segments of 8 and 12 blocks cost 8 and 4 % of the time
// and leave 0.5e-6 and 0.7e-6, however long the group; plain fp32 products are at
// 0.45e-6.  Outputs in bf16 round 1000 times as coarsely and keep one
// accumulator.
//
// dW's epilogue stores through shared memory: each warp puts 16 rows x 32
// columns into a swizzled 2 KB buffer and one lane hands it to the TMA, which
// also clips at d_in and d_out.  Stored row by row from the lanes' registers
// (32-byte pieces of 32 rows an instruction), the 256 KB of a tile took longer
// than the MMAs of the next two segments and held the tensor cores up: 429
// against 417 us, and 46 against 37 for 8192 rows into one 1024x2048 gradient.
//
// Widths that are no multiples of 8 (rows that TMA cannot address) are repacked
// into the workspace with padded rows first, and the outputs leave row by row
// through the epilogue's buffers, a warp's lanes beside each other: 16384 rows x
// 8 x 2047x8191 forward 518 us, dX 527, dW 591.  The CUDA-core kernel keeps what
// that is not worth (group_repacks).
//
// Few tiles.  Where they are at most half the pairs, each tile's K blocks
// are split over several pairs, which write fp32 partial tiles into the
// workspace; a second, dependent launch adds them in order and applies the
// epilogue (the same bits in every run): 16384 rows into one 512x512 weight
// gradient 30 us, 99 unsplit; 300 rows x 8192x256 23 us, 51 unsplit.
//
// Warp roles and pipeline as in gemm_tc2.cu: warp 0 TMA producer, warp 1 MMA
// issuer (leader CTA), warps 2-9 epilogue, in dW warp 10 zeroing; five 32 KB
// stages per CTA (a sixth gains nothing); two accumulators of 256 columns.  Every wait is bounded.
#include <cuda.h>

#include <algorithm>

#include "common.cuh"
#include "group_epilogue.cuh"
#include "group_table.cuh"
#include "group_tma.h"
#include "kernels.h"
#include "op_checks.h"
#include "tc_common.cuh"
#include "tc_epilogue.cuh"
#include "tc_pair.cuh"

namespace mg {
namespace {

using namespace tc;

constexpr int G_BM = 128;          // rows per CTA (256 per pair)
constexpr int G_BNH = 128;         // B columns per CTA (256 per pair)
constexpr int G_BN = 256;
constexpr int G_BK = 64;
constexpr int G_STAGES = 5;
constexpr int G_THREADS = 320;      // one more warp in dW

constexpr int group_threads(int kind) { return kind == GROUP_DW ? G_THREADS + 32 : G_THREADS; }
constexpr uint32_t G_A_BYTES = G_BM * G_BK * 2;
constexpr uint32_t G_B_BYTES = G_BNH * G_BK * 2;
constexpr int G_SEG = 12;          // K blocks (768 rows) per accumulator in dW
constexpr uint32_t G_TAIL_BYTES = G_A_BYTES + G_B_BYTES;   // dW: the ragged K block
constexpr uint32_t G_OUT_BYTES = 8 * 16 * 128;             // dW: a 16x32 fp32 buffer per epilogue warp
constexpr uint32_t group_extra_bytes(int kind, bool any) {  // shared memory behind the ring
  return (kind == GROUP_DW ? G_TAIL_BYTES : 0) + (kind == GROUP_DW || any ? G_OUT_BYTES : 0);
}
constexpr int G_PANEL = 64 * G_BK * 2;   // one 64-column panel of a stage

struct GroupTcParams {
  GemmArgs g;              // the epilogue: N, leading dimensions, outputs
  GroupArgs any;           // the same for widths that are no multiples of 8
  int plain;               // nothing but the sum is stored
  const int* offsets;
  int rows, groups, zero_rest;
  int d_in, d_out;
  int tiles_n;             // 256-column tiles of an output row
  int tiles_m;             // dW: 256-row tiles of one dW[e]
  int k_blocks;            // forward, dX
  int vec32;               // rows of the epilogue's matrices allow 32-byte accesses (16 always)
  int splits;              // parts of every tile's K blocks; part s writes rows s * split_rows ..
  int split_rows;
  int* err;
};

// One output tile of the list.
struct GroupTile {
  int e, m0, m_end, n0;
  int kb;        // K blocks (0: the result is zero)
  int k0;        // forward, dX: first of them
  int part;      // split of the K blocks
  int krow0;     // dW: first row of the group
  int tail;      // dW: rows of the last K block that belong to the group, 0 if all 64 do
};

template <int KIND>
__device__ __forceinline__ int tile_count(const GroupTcParams& P, const GroupTable& t) {
  return P.splits * (KIND == GROUP_DW ? P.groups * P.tiles_m * P.tiles_n : t.cum[t.n - 1] * P.tiles_n);
}

// e: cursor kept between calls (items ascend).
template <int KIND>
__device__ __forceinline__ GroupTile tile_at(const GroupTcParams& P, const GroupTable& t, int item, int& e) {
  GroupTile r;
  r.part = 0;
  if (P.splits > 1) {
    r.part = item % P.splits;
    item /= P.splits;
  }
  r.k0 = 0;
  if (KIND == GROUP_DW) {
    const int per = P.tiles_m * P.tiles_n;
    e = item / per;
    const int q = item - e * per;
    r.m0 = (q / P.tiles_n) * 2 * G_BM;
    r.n0 = (q % P.tiles_n) * G_BN;
    r.m_end = P.d_in;
    r.krow0 = t.lo[e];
    const int size = t.hi[e] - t.lo[e];
    r.kb = (size + G_BK - 1) / G_BK;
    r.tail = size % G_BK;
    if (P.splits > 1) {
      const int lo = r.kb * r.part / P.splits, hi = r.kb * (r.part + 1) / P.splits;
      if (hi < r.kb || hi == lo) r.tail = 0;     // the group's last block is another part's
      r.krow0 += lo * G_BK;
      r.kb = hi - lo;
    }
  } else {
    const int mt = item / P.tiles_n;
    r.n0 = (item - mt * P.tiles_n) * G_BN;
    while (t.cum[e] <= mt) ++e;
    r.m0 = t.lo[e] + (mt - (e ? t.cum[e - 1] : 0)) * 2 * G_BM;
    r.m_end = t.hi[e];
    r.kb = e < P.groups ? P.k_blocks : 0;
    r.krow0 = 0;
    r.tail = 0;
    if (P.splits > 1) {
      r.k0 = r.kb * r.part / P.splits;
      r.kb = r.kb * (r.part + 1) / P.splits - r.k0;
    }
  }
  r.e = e;
  return r;
}

__device__ __forceinline__ void tma_load_3d_to_leader(void* dst, const CUtensorMap* map, uint32_t bar_cluster,
                                                      int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar_cluster), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// A box of shared memory to global memory (clipped at the tensor's bounds), in a
// bulk group of its own.
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, const void* src, int x, int y, int z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(smem_u32(src)), "r"(x), "r"(y), "r"(z)
               : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

// 32 columns of a warp's 32 rows (lane = row), stored row by row with the lanes
// beside each other, through a buffer of 16 rows (rotated by the row: no bank
// conflicts).  Rows below m_end; base: rows before the output's row 0.
template <int KIND>
__device__ __forceinline__ void store_any(const GroupTcParams& P, float* buf, const float (&v)[32], int row0, int m_end,
                                          int base, int n0, int lane) {
#pragma unroll 1
  for (int h = 0; h < 2; ++h) {
    __syncwarp();
    if (lane >> 4 == h) {
      const int r = lane & 15;
#pragma unroll
      for (int j = 0; j < 32; ++j) buf[r * 32 + ((j + r) & 31)] = v[j];
    }
    __syncwarp();
    const int rows = min(16, m_end - row0 - 16 * h);
    if (n0 + lane >= P.g.N) continue;
    const size_t o = (size_t)(base + row0 + 16 * h) * P.g.N + n0 + lane;
    if (KIND == GROUP_DW || P.splits > 1) {
      float* out = static_cast<float*>(P.g.out) + o;
#pragma unroll 4
      for (int r = 0; r < rows; ++r) out[(size_t)r * P.g.N] = buf[r * 32 + ((lane + r) & 31)];
    } else if (P.plain) {
      bf16* out = static_cast<bf16*>(P.any.out) + o;
#pragma unroll 4
      for (int r = 0; r < rows; ++r) out[(size_t)r * P.g.N] = __float2bfloat16_rn(buf[r * 32 + ((lane + r) & 31)]);
    } else {
#pragma unroll 1
      for (int r = 0; r < rows; ++r) group_epilogue<bf16>(P.any, o + (size_t)r * P.g.N, buf[r * 32 + ((lane + r) & 31)]);
    }
  }
}

// ANY: outputs of any width and alignment.
template <int KIND, typename TO, bool ANY>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(group_threads(KIND), 1)
    group_pair_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                      const __grid_constant__ CUtensorMap tmO, const GroupTcParams P) {
  constexpr bool A_MN = KIND == GROUP_DW;
  constexpr bool B_MN = KIND != GROUP_DX;
  constexpr uint32_t TMEM_COLS = 2 * G_BN;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>(
      (reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  uint8_t* sA = smem;
  uint8_t* sB = smem + G_STAGES * G_A_BYTES;
  uint8_t* sT = sB + G_STAGES * G_B_BYTES;
  uint8_t* sO = sT + (KIND == GROUP_DW ? G_TAIL_BYTES : 0);
  uint64_t* full = reinterpret_cast<uint64_t*>(sT + group_extra_bytes(KIND, ANY));
  uint64_t* empty = full + G_STAGES;
  uint64_t* tfull = empty + G_STAGES;
  uint64_t* tempty = tfull + 2;
  uint64_t* tail_loaded = tempty + 2;      // ragged block: this CTA's part has arrived,
  uint64_t* tail_peer = tail_loaded + 1;   // leader: the peer's part is zeroed,
  uint64_t* tail_full = tail_peer + 1;     // leader: both are,
  uint64_t* tail_empty = tail_full + 1;    // it has been multiplied
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(tail_empty + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  GroupTable t;
  t.n = P.groups + (P.zero_rest ? 2 : 0);
  t.lo = reinterpret_cast<int*>(tmem_slot + 2);
  t.hi = t.lo + P.groups + 2;
  t.cum = t.hi + P.groups + 2;

  const uint32_t rank = cluster_rank();
  const bool leader = rank == 0;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;

  if (threadIdx.x == 0) {
    for (int s = 0; s < G_STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int i = 0; i < 4; ++i) mbar_init(&tail_loaded[i], 1);
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], 2 * 256);
    }
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(TMEM_COLS));
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
  }
  if (warp == 2) load_group_table(t, P.offsets, P.groups, P.rows, 2 * G_BM);
  tc_fence_before();
  cluster_sync();                      // barriers, tables and TMEM of both CTAs are ready
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot;
  const int n_items = tile_count<KIND>(P, t);

  if (warp == 0) {
    // ---------------- TMA producer (both CTAs) ----------------
    if (lane == 0) {
      int stage = 0, e = 0;
      uint32_t phase = 0, tail_phase = 0;
      for (int item = pair; item < n_items && !*abort_flag; item += npairs) {
        const GroupTile T = tile_at<KIND>(P, t, item, e);
        const int m0 = T.m0 + (int)rank * G_BM, n0 = T.n0 + (int)rank * G_BNH;
        const int plain = T.tail ? T.kb - 1 : T.kb;
        for (int kb = 0; kb <= plain; ++kb) {
          // the ragged block, once the ring has turned over: by then the one of
          // the tile before has been multiplied
          if (KIND == GROUP_DW && T.tail && kb == min(plain, G_STAGES)) {
            if (!mbar_wait_cluster(tail_empty, tail_phase ^ 1)) { *abort_flag = 1; atomicExch(P.err, 1); break; }
            tail_phase ^= 1;
            const int kr = T.krow0 + plain * G_BK;
            mbar_expect_tx(tail_loaded, G_TAIL_BYTES);
            tma_load_2d(sT, &tmA, tail_loaded, m0, kr);
            tma_load_2d(sT + G_PANEL, &tmA, tail_loaded, m0 + 64, kr);
            tma_load_2d(sT + G_A_BYTES, &tmB, tail_loaded, n0, kr);
            tma_load_2d(sT + G_A_BYTES + G_PANEL, &tmB, tail_loaded, n0 + 64, kr);
          }
          if (kb == plain) break;
          if (!mbar_wait_cluster(&empty[stage], phase ^ 1)) { *abort_flag = 1; atomicExch(P.err, 1); break; }
          uint8_t* a = sA + stage * G_A_BYTES;
          uint8_t* b = sB + stage * G_B_BYTES;
          const int k0 = (T.k0 + kb) * G_BK;
          if (leader) mbar_expect_tx(&full[stage], 2 * (G_A_BYTES + G_B_BYTES));
          const uint32_t fb = map_to(&full[stage], 0);
          if (A_MN) {
            tma_load_2d_to_leader(a, &tmA, fb, m0, T.krow0 + k0);
            tma_load_2d_to_leader(a + G_PANEL, &tmA, fb, m0 + 64, T.krow0 + k0);
          } else {
            tma_load_2d_to_leader(a, &tmA, fb, k0, m0);
          }
          if (KIND == GROUP_DW) {
            tma_load_2d_to_leader(b, &tmB, fb, n0, T.krow0 + k0);
            tma_load_2d_to_leader(b + G_PANEL, &tmB, fb, n0 + 64, T.krow0 + k0);
          } else if (B_MN) {
            tma_load_3d_to_leader(b, &tmB, fb, n0, k0, T.e);
            tma_load_3d_to_leader(b + G_PANEL, &tmB, fb, n0 + 64, k0, T.e);
          } else {
            tma_load_3d_to_leader(b, &tmB, fb, k0, n0, T.e);
          }
          if (++stage == G_STAGES) { stage = 0; phase ^= 1; }
        }
      }
    }
  } else if (KIND == GROUP_DW && warp == 10) {
    // ---------------- zeroing of the blocks that end inside a group's rows ----------------
    int e = 0;
    uint32_t ph = 0;
    for (int item = pair; item < n_items; item += npairs) {
      const GroupTile T = tile_at<KIND>(P, t, item, e);
      if (!T.tail) continue;
      int ok = __all_sync(0xffffffffu, mbar_wait(tail_loaded, ph));
      if (ok) {
        // a K row is one 128-byte line of each panel, whatever the swizzle inside it
        const int n16 = (G_BK - T.tail) * 8;
#pragma unroll
        for (int p = 0; p < 4; ++p) {
          uint4* q = reinterpret_cast<uint4*>(sT + p * G_PANEL + T.tail * 128);
          for (int i = lane; i < n16; i += 32) q[i] = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async();
        __syncwarp();
        if (lane == 0) {
          if (leader) {
            ok = mbar_wait_cluster(tail_peer, ph);
            if (ok) mbar_arrive(tail_full);
          } else {
            mbar_arrive_remote_release(map_to(tail_peer, 0));
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
      }
      ph ^= 1;
      if (!ok) {
        if (lane == 0) { *abort_flag = 1; atomicExch(P.err, 1); }
        break;
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && leader) {
      // ---------------- leader: MMA issuer for the pair ----------------
      constexpr uint32_t idesc = instr_desc(2 * G_BM, G_BN, A_MN ? 1 : 0, B_MN ? 1 : 0);
      int stage = 0, e = 0, it = 0;
      uint32_t phase = 0, tail_phase = 0;
      for (int item = pair; item < n_items && !*abort_flag; item += npairs) {
        const GroupTile T = tile_at<KIND>(P, t, item, e);
        bool ok = true;
        for (int kb = 0; ok && (kb < T.kb || kb == 0);) {
          // one accumulator: all K blocks, or a segment of them
          const int k_end = KIND == GROUP_DW ? min(T.kb, kb + G_SEG) : T.kb;
          const int k_begin = kb, acc = it & 1;
          const uint32_t use = (uint32_t)(it >> 1) & 1u;
          if (!mbar_wait_cluster(&tempty[acc], use ^ 1)) { ok = false; break; }
          tc_fence_after();
          const uint32_t d = tmem_base + (uint32_t)(acc * G_BN);
          for (; kb < k_end; ++kb) {
            const bool tail = KIND == GROUP_DW && T.tail && kb == T.kb - 1;
            if (!(tail ? mbar_wait_cluster(tail_full, tail_phase) : mbar_wait_cluster(&full[stage], phase))) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint32_t a = smem_u32(tail ? sT : sA + stage * G_A_BYTES);
            const uint32_t b = smem_u32(tail ? sT + G_A_BYTES : sB + stage * G_B_BYTES);
#pragma unroll
            for (int k = 0; k < G_BK / 16; ++k) {
              const uint64_t ad = A_MN ? smem_desc(a + k * 2048, G_PANEL, 1024) : smem_desc(a + k * 32, 16, 1024);
              const uint64_t bd = B_MN ? smem_desc(b + k * 2048, G_PANEL, 1024) : smem_desc(b + k * 32, 16, 1024);
              mma_bf16_pair(d, ad, bd, idesc, (kb > k_begin || k) ? 1u : 0u);
            }
            mma_commit_pair(tail ? tail_empty : &empty[stage]);
            if (tail) tail_phase ^= 1;
            else if (++stage == G_STAGES) { stage = 0; phase ^= 1; }
          }
          if (!ok) break;
          mma_commit_pair(&tfull[acc]);
          ++it;
          if (T.kb == 0) break;
        }
        if (!ok) { *abort_flag = 1; atomicExch(P.err, 1); break; }
      }
    }
  } else {
    // ---------------- epilogue (warps 2..9, both CTAs) ----------------
    const int quarter = warp & 3;
    const int half = (warp - 2) >> 2;
    const int row_in_tile = quarter * 32 + lane;
    const uint32_t leader_tempty[2] = {map_to(&tempty[0], 0), map_to(&tempty[1], 0)};
    int e = 0, it = 0;
    bool up = true;
    // the next accumulator is full (false: a wait gave up)
    auto wait_full = [&](int acc) {
      if (!mbar_wait(&tfull[acc], (uint32_t)(it >> 1) & 1u)) { *abort_flag = 1; atomicExch(P.err, 1); }
      up = !*abort_flag;
      up = __all_sync(0xffffffffu, up);
      tc_fence_after();
      return up;
    };
    for (int item = pair; item < n_items && up; item += npairs) {
      const GroupTile T = tile_at<KIND>(P, t, item, e);
      const int m = T.m0 + (int)rank * G_BM + row_in_tile;
      const bool row_ok = m < T.m_end;
      const int mo = m + T.part * P.split_rows;
      const uint32_t lanes = tmem_base + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(half * (G_BN / 2));
      const int n0 = T.n0 + half * (G_BN / 2);
      if (KIND == GROUP_DW) {
        float sum[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int i = 0; i < 32; ++i) sum[c][i] = 0.0f;
        const int segs = T.kb ? (T.kb + G_SEG - 1) / G_SEG : 1;
        for (int sg = 0; sg < segs; ++sg, ++it) {
          const int acc = it & 1;
          if (!wait_full(acc)) break;
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            uint32_t r[32];
            tmem_ld32_async(lanes + acc * G_BN + c * 32, r);
            tmem_wait_regs(r);
            if (c == 3) {
              tc_fence_before();
              mbar_arrive_remote(leader_tempty[acc]);
            }
            if (T.kb) {
#pragma unroll
              for (int i = 0; i < 32; ++i) sum[c][i] += __uint_as_float(r[i]);
            }
          }
        }
        if (!up) break;
        const int row0 = T.m0 + (int)rank * G_BM + quarter * 32;     // the warp's rows
        uint8_t* buf = sO + (warp - 2) * 2048;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int n = n0 + c * 32;
          if (n >= P.g.N) continue;                                  // warp-uniform, as below
          if constexpr (ANY) {
            store_any<KIND>(P, reinterpret_cast<float*>(buf), sum[c], row0, T.m_end,
                            T.e * P.d_in + T.part * P.split_rows, n, lane);
          } else {
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
              if (row0 + 16 * h >= T.m_end) continue;
              if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
              __syncwarp();
              if (lane >> 4 == h) {
#pragma unroll
                for (int q = 0; q < 8; ++q)
                  *reinterpret_cast<float4*>(buf + sw128(lane & 15, q)) =
                      make_float4(sum[c][4 * q], sum[c][4 * q + 1], sum[c][4 * q + 2], sum[c][4 * q + 3]);
                fence_proxy_async();
              }
              __syncwarp();
              if (lane == 0) tma_store_3d(&tmO, buf, n, row0 + 16 * h, T.part * P.groups + T.e);
            }
          }
        }
        continue;
      }
      const int acc = it & 1;
      if (!wait_full(acc)) break;
      ++it;
#pragma unroll 1
      for (int cp = 0; cp < 2; ++cp) {
        uint32_t r0[32], r1[32];
        tmem_ld32_async(lanes + acc * G_BN + cp * 64, r0);
        tmem_ld32_async(lanes + acc * G_BN + cp * 64 + 32, r1);
        tmem_wait_regs(r0);
        reg_fence(r1);
        if (cp == 1) {
          tc_fence_before();
          mbar_arrive_remote(leader_tempty[acc]);
        }
        auto chunk = [&](int n, uint32_t (&r)[32]) {
          if (n >= P.g.N || (!ANY && !row_ok)) return;
          float v[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = T.kb ? __uint_as_float(r[i]) : 0.0f;
          if (ANY)
            store_any<KIND>(P, reinterpret_cast<float*>(sO + (warp - 2) * 2048), v, m - lane, T.m_end, T.part * P.split_rows, n,
                            lane);
          else if (n + 32 <= P.g.N) epi32<TO>(P.g, true, P.vec32 != 0, mo, n, v);
          else epi_by8<TO>(P.g, mo, n, v);
        };
        chunk(n0 + cp * 64, r0);
        chunk(n0 + cp * 64 + 32, r1);
      }
    }
    if (KIND == GROUP_DW && !ANY && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }

  if (*abort_flag) drain_in_flight();
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync();                      // no remote arrive or MMA still targets either CTA
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(TMEM_COLS));
  }
}

// ---------------------------------------------------------------- host side
typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                  const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                  const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                  CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn group_encode_fn() {
  static EncodeTiledFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      return reinterpret_cast<EncodeTiledFn>(p);
    return static_cast<EncodeTiledFn>(nullptr);
  }();
  return fn;
}

// fp32 [outer][rows][cols], dense; 32x16 boxes, 128-byte swizzle.
bool group_out_map(CUtensorMap* map, void* base, long long outer, long long rows, long long cols) {
  EncodeTiledFn fn = group_encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)outer};
  cuuint64_t strides[2] = {(cuuint64_t)cols * 4, (cuuint64_t)cols * (cuuint64_t)rows * 4};
  cuuint32_t box[3] = {32, 16, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, base, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
         CUDA_SUCCESS;
}

size_t group_pair_smem(int kind, bool any, int groups) {
  return 1024 + (size_t)G_STAGES * (G_A_BYTES + G_B_BYTES) + group_extra_bytes(kind, any) + (2 * G_STAGES + 8) * 8 + 8 +
         (size_t)kGroupTableInts(groups) * 4;
}

// ---- few tiles
// Parts of the K blocks for these sizes: as many as keep 76 pairs busy, with at
// least eight blocks each (on average over the groups in dW).
int group_splits(int kind, int rows, int groups, int d_in, int d_out) {
  const int N = kind == GROUP_DX ? d_in : d_out, K = kind == GROUP_FWD ? d_in : d_out;
  const long long tiles_n = (N + G_BN - 1) / G_BN;
  const long long tiles = kind == GROUP_DW ? groups * ((d_in + 2ll * G_BM - 1) / (2 * G_BM)) * tiles_n
                                           : ((long long)rows / (2 * G_BM) + groups) * tiles_n;
  const long long kb = kind == GROUP_DW ? (long long)rows / groups / G_BK : (K + G_BK - 1) / G_BK;
  const long long s = std::min(std::min(76 / tiles, kb / 8), 16ll);
  return s < 2 ? 1 : (int)s;
}

// Their bytes for these rows or fewer (forward, dX: s <= 76 / tiles parts of at
// most 256 tiles / tiles_n rows; dW's parts grow with the rows).
size_t split_bytes(int kind, int rows, int groups, int d_in, int d_out) {
  const int N = kind == GROUP_DX ? d_in : d_out;
  long long part_rows;
  if (kind == GROUP_DW) {
    const int s = group_splits(kind, rows, groups, d_in, d_out);
    part_rows = s < 2 ? 0 : (long long)s * groups * d_in;
  } else {
    const int least = group_splits(kind, std::min(rows, 1), groups, d_in, d_out);   // the most parts of any rows
    part_rows = least < 2 ? 0 : std::min((long long)least * rows, 76ll * 2 * G_BM / ((N + G_BN - 1) / G_BN));
  }
  return (size_t)part_rows * N * 4;
}

template <int KIND, typename TO, bool ANY>
cudaError_t launch_group_pair(const GroupArgs& g, int splits, cudaStream_t s) {
  CUtensorMap ma, mb, mo = {};
  bool ok;
  if (KIND == GROUP_DW) {
    ok = (ANY || group_out_map(&mo, splits > 1 ? g.ws : g.out, (long long)splits * g.groups, g.d_in, g.d_out)) &&
         group_map(&ma, g.A, 0, g.rows, g.d_in, g.lda, 64, G_BK) &&
         group_map(&mb, g.B, 0, g.rows, g.d_out, g.ldb, 64, G_BK);
  } else {
    const int k = KIND == GROUP_FWD ? g.d_in : g.d_out;
    ok = group_map(&ma, g.A, 0, g.rows, k, g.lda, G_BK, G_BM) &&
         (KIND == GROUP_FWD ? group_map(&mb, g.B, g.groups, g.d_in, g.d_out, g.ldb, 64, G_BK)
                            : group_map(&mb, g.B, g.groups, g.d_in, g.d_out, g.ldb, G_BK, G_BNH));
  }
  if (!ok) return cudaErrorInvalidValue;
  GroupTcParams P;
  const int N = KIND == GROUP_DX ? g.d_in : g.d_out;
  P.any = g;
  P.plain = !g.act && !g.out_z && !g.dact && !g.resid;
  P.splits = splits;
  P.split_rows = (int)group_out_rows(g.kind, g.rows, g.groups, g.d_in);
  P.g.N = N;
  P.g.ldz = P.g.lds = P.g.ldr = P.g.ldo = N;
  if (splits == 1) {
    P.g.act = g.act;
    P.g.out_z = g.out_z;
    P.g.saved = g.saved; P.g.dact = g.dact;
    P.g.resid = g.resid;
  }
  P.g.aux_type = DT_BF16;
  P.g.out = splits > 1 ? g.ws : g.out;
  P.g.out_type = sizeof(TO) == 4 ? DT_F32 : DT_BF16;
  P.offsets = g.offsets;
  P.rows = g.rows;
  P.groups = g.groups;
  P.zero_rest = splits > 1 ? 0 : g.zero_rest;
  P.d_in = g.d_in;
  P.d_out = g.d_out;
  P.tiles_n = (N + G_BN - 1) / G_BN;
  P.tiles_m = (g.d_in + 2 * G_BM - 1) / (2 * G_BM);
  P.k_blocks = ((KIND == GROUP_FWD ? g.d_in : g.d_out) + G_BK - 1) / G_BK;
  P.err = g.err;
  auto al = [](const void* p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; };
  if (!ANY && !(al(P.g.out, 16) && al(P.g.out_z, 16) && al(P.g.saved, 16) && al(P.g.resid, 16)))
    return cudaErrorInvalidValue;
  P.vec32 = al(P.g.out, 32) && al(P.g.out_z, 32) && al(P.g.saved, 32) && al(P.g.resid, 32) && N % 16 == 0;
  auto kern = group_pair_kernel<KIND, TO, ANY>;
  const size_t smem = group_pair_smem(KIND, ANY, g.groups);
  const cudaError_t attr = cudaFuncSetAttribute(    // of this device's context: set in every call
      kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)group_pair_smem(KIND, ANY, kMaxGroups));
  if (attr != cudaSuccess) return attr;
  static const int slots = [&] {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * (device_sms() / 2));
    cfg.blockDim = dim3(group_threads(KIND));
    cfg.dynamicSmemBytes = group_pair_smem(KIND, ANY, kMaxGroups);
    cudaLaunchAttribute at;
    at.id = cudaLaunchAttributeClusterDimension;
    at.val.clusterDim.x = 2;
    at.val.clusterDim.y = 1;
    at.val.clusterDim.z = 1;
    cfg.attrs = &at;
    cfg.numAttrs = 1;
    int c = 0;
    if (cudaOccupancyMaxActiveClusters(&c, kern, &cfg) != cudaSuccess || c <= 0) {
      cudaGetLastError();
      c = device_sms() / 2;
    }
    return c;
  }();
  // tiles at most: every group may end inside one
  const long long items = splits * (KIND == GROUP_DW
                              ? (long long)g.groups * P.tiles_m * P.tiles_n
                              : ((long long)g.rows / (2 * G_BM) + g.groups + (P.zero_rest ? 2 : 0)) * P.tiles_n);
  if (items > 0x7fffffff) return cudaErrorInvalidValue;
  const int pairs = items < slots ? (int)items : slots;
  kern<<<2 * pairs, group_threads(KIND), smem, s>>>(ma, mb, mo, P);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || splits == 1) return e;
  return group_join(g, splits, P.split_rows, N, s);
}

// ---- operands of widths that are no multiples of 8
// Rows of L elements to rows of Lp (a multiple of 8), zeros behind; a thread per
// 16 bytes written.
__global__ void __launch_bounds__(256) group_repack_kernel(const bf16* src, uint4* dst, unsigned L, unsigned Lp8,
                                                           long long chunks) {
  for (long long i = blockIdx.x * 256ll + threadIdx.x; i < chunks; i += gridDim.x * 256ll) {
    const long long r = i / Lp8;
    const unsigned c = (unsigned)(i - r * Lp8) * 8;
    const unsigned short* p = reinterpret_cast<const unsigned short*>(src) + r * L + c;
    unsigned h[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) h[q] = c + q < L ? p[q] : 0;
    dst[i] = make_uint4(h[0] | h[1] << 16, h[2] | h[3] << 16, h[4] | h[5] << 16, h[6] | h[7] << 16);
  }
}

int pad8(int n) { return (n + 7) / 8 * 8; }

// An operand's rows and width, and the scratch its repacked copy takes.
struct Operand {
  long long rows;
  int width;
  size_t bytes() const { return width % 8 ? ((size_t)rows * pad8(width) * 2 + 255) / 256 * 256 : 0; }
};
Operand operand_a(int kind, int rows, int d_in, int d_out) { return {rows, kind == GROUP_DX ? d_out : d_in}; }
Operand operand_b(int kind, int rows, int groups, int d_in, int d_out) {
  return {kind == GROUP_DW ? (long long)rows : (long long)groups * d_in, d_out};
}

// Whether a product of such widths is worth the repacking against the CUDA-core
// kernel, whose time goes with the operations (64-row tiles) and with its steps
// along the sum: forward 30 against 80 us for 300 rows x 4 x 601x1003, 29 against
// 52 for 1000 x 8 x 333x333, 161 against 645 for 24 x 8 x 2047x8191.  A weight
// gradient of few rows per group only writes, which the plain kernel does better
// (24 rows: 193 against 334 us; 75 rows per group: 26 against 38).
bool group_repacks(int kind, int rows, int groups, int d_in, int d_out) {
  if (d_in % 8 == 0 && d_out % 8 == 0) return false;
  if (kind == GROUP_DW) return rows >= 32ll * groups && 2.0 * rows * d_in * d_out >= 1e8;
  const double tile_rows = std::max((double)rows, 64.0 * std::min(rows, groups));
  return 2.0 * tile_rows * d_in * d_out >= 1e8 || (kind == GROUP_FWD ? d_in : d_out) >= 128;
}

cudaError_t repack(const void*& p, int& ld, const Operand& o, char*& ws, cudaStream_t s) {
  if (o.width % 8 == 0) return cudaSuccess;
  ld = pad8(o.width);
  const long long chunks = o.rows * (ld / 8), blocks = (chunks + 255) / 256;
  group_repack_kernel<<<(unsigned)std::min(blocks, 152ll * 32), 256, 0, s>>>(
      static_cast<const bf16*>(p), reinterpret_cast<uint4*>(ws), (unsigned)o.width, (unsigned)(ld / 8), chunks);
  p = ws;
  ws += o.bytes();
  return cudaGetLastError();
}

}  // namespace

bool group_map(CUtensorMap* map, const void* base, long long outer, long long rows, long long cols, long long ld,
               int box_cols, int box_rows) {
  EncodeTiledFn fn = group_encode_fn();
  if (!fn) return false;
  cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)outer};
  if (!ld) ld = cols;
  cuuint64_t strides[2] = {(cuuint64_t)ld * 2, (cuuint64_t)ld * (cuuint64_t)rows * 2};
  cuuint32_t box[3] = {(cuuint32_t)box_cols, (cuuint32_t)box_rows, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, outer ? 3 : 2, const_cast<void*>(base), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool grouped_tc_eligible(const GroupArgs& g) {
  auto al = [](const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
  // mo = e * d_in + m and the tile counts are 32-bit
  if (!g.use_tc || g.type != DT_BF16 || g.rows == 0) return false;
  if ((g.d_in % 8 || g.d_out % 8) && !(g.ws && group_repacks(g.kind, g.rows, g.groups, g.d_in, g.d_out))) return false;
  if ((long long)g.groups * g.d_in > 0x7fff0000ll) return false;
  const long long tiles_n = ((g.kind == GROUP_DX ? g.d_in : g.d_out) + G_BN - 1) / G_BN;
  const long long tiles_m = g.kind == GROUP_DW ? (long long)g.groups * ((g.d_in + 255) / 256)
                                               : g.rows / 256 + g.groups + 2ll;
  if (tiles_m * tiles_n > 0x3fffffffll) return false;
  return al(g.A) && al(g.B) && group_encode_fn() != nullptr;
}

size_t grouped_scratch_bytes(int rows, int groups, int d_in, int d_out, bool compensated) {
  size_t most = grouped_simt_split_bytes(rows, groups, d_in, d_out, compensated);
  for (int kind : {GROUP_FWD, GROUP_DX, GROUP_DW}) {
    size_t n = split_bytes(kind, rows, groups, d_in, d_out);
    if (group_repacks(kind, rows, groups, d_in, d_out))
      n += operand_a(kind, rows, d_in, d_out).bytes() + operand_b(kind, rows, groups, d_in, d_out).bytes();
    most = std::max(most, n);
  }
  return most;
}

int grouped_tc_launches(const GroupArgs& g) {
  return 1 + (operand_a(g.kind, g.rows, g.d_in, g.d_out).width % 8 != 0) +
         (operand_b(g.kind, g.rows, g.groups, g.d_in, g.d_out).width % 8 != 0) +
         (g.ws && !grouped_narrow(g) && group_splits(g.kind, g.rows, g.groups, g.d_in, g.d_out) > 1);
}

cudaError_t grouped_gemm_tc(const GroupArgs& given, cudaStream_t s) {
  GroupArgs g = given;
  const bool any = g.d_in % 8 || g.d_out % 8;
  if (any) {
    char* ws = reinterpret_cast<char*>(g.ws);
    cudaError_t e = repack(g.A, g.lda, operand_a(g.kind, g.rows, g.d_in, g.d_out), ws, s);
    if (e == cudaSuccess) e = repack(g.B, g.ldb, operand_b(g.kind, g.rows, g.groups, g.d_in, g.d_out), ws, s);
    if (e != cudaSuccess) return e;
    g.ws = reinterpret_cast<float*>(ws);
  }
  if (grouped_narrow(g)) return grouped_gemm_narrow(g, s);
  const int splits = g.ws ? group_splits(g.kind, g.rows, g.groups, g.d_in, g.d_out) : 1;
  if (any) {
    if (g.kind == GROUP_DW) return launch_group_pair<GROUP_DW, float, true>(g, splits, s);
    return g.kind == GROUP_FWD ? launch_group_pair<GROUP_FWD, bf16, true>(g, splits, s)
                               : launch_group_pair<GROUP_DX, bf16, true>(g, splits, s);
  }
  if (g.kind == GROUP_DW) return launch_group_pair<GROUP_DW, float, false>(g, splits, s);
  if (g.kind == GROUP_FWD)
    return splits > 1 ? launch_group_pair<GROUP_FWD, float, false>(g, splits, s)
                      : launch_group_pair<GROUP_FWD, bf16, false>(g, 1, s);
  return splits > 1 ? launch_group_pair<GROUP_DX, float, false>(g, splits, s)
                    : launch_group_pair<GROUP_DX, bf16, false>(g, 1, s);
}

}  // namespace mg

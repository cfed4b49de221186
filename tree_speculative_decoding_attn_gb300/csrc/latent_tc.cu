// Tree attention over a cache of latent vectors on pairs of SMs (bf16 in,
// float32 softmax and accumulation).
//
// A key is a row c = [latent (LAT) ; rotary (64)], a value its latent part;
// a query row is (node, head), already in the latent space:
//   x_j = scale q . c_j over the LAT + 64 dims,  out = sum_j softmax(x)_j c_j[:LAT].
// All heads and nodes of a sequence share every key, so they are rows of one
// product: 2 (2 LAT + 64) flops a row and key for 2 (LAT + 64) bytes a key,
// tensor-bound from about 150 rows a sequence on, HBM-bound below.
//
// What fits decides the shape.  LAT = 512 output columns of 128 rows would
// fill one SM's TMEM and leave nothing for S, and 128 query rows of 576 dims
// are 144 KB of shared memory.  So a CTA holds 64 rows, and a pair MMA of M =
// 128 (cta_group::2) gives them the full rate: rows 0-63 of a pair lie in the
// even CTA, and each CTA's lanes 0-63 hold the columns of the first half of N,
// lanes 64-127 those of the second.  Measured: M128 N128 K16 33 cycles, M128
// N256 K16 65 (4096 bf16 multiply-adds a cycle and SM, the peak), issued by
// one elected thread; the single-CTA M = 64 forms run at half of that.
//   S(g)  = Q K(g)^T   N = 128 keys (64 in each CTA), K = LAT + 64
//   O    += P(g) V(g)  N = 256 dims (128 in each CTA), K = 128 keys, LAT/256
//                      of them; P in shared memory
// K and V are the same rows, but the pair splits S by keys and O by dims: a
// CTA needs its own 64 keys whole, and of the other 64 the half of the dims
// that it multiplies in PV.  Of its own keys the other half of the dims is
// done with after S, and that is where the other CTA's keys are loaded: each
// "place" (64 keys, 128 dims of every block of 256) holds in both CTAs what
// PV reads at one shared-memory offset, as the pair MMA asks.  104 KB a tile
// and SM instead of 136 with V in a place of its own, which an SM takes in at
// about 55 bytes a cycle at most (TMA boxes of 256 rows of 128 bytes).
//
// Shared memory (LAT 512): Q 72 KB, two tiles of latents 128, rotary columns
// 8, P 16.  TMEM: O LAT/2 columns, two S buffers of 64.
// Roles: warp 0 loads Q and K, warp 2 V; of the even CTA warp 1 issues S and
// warp 3 PV; warps 4-11 softmax and epilogue: a thread owns 32 keys of one row
// (lanes r and r + 64 of two warps share row r).  Two S buffers: the softmax of
// a tile runs under the next tile's S and the last one's PV.
// Work: all (sequence, 128-row tile) units, each its tree tiles and then its
// prefix tiles of 128 keys, go whole to the pairs or are cut into one equal
// range a pair; units cut between pairs leave float32 partials that a second
// kernel joins.
// What bounds it: a tile's MMAs are 2258 cycles, its shared-memory traffic
// (operands 245 KB, TMA 104, P 16) 2850 at 128 bytes a cycle, and it takes
// 2800 to 3200; 32 trees of 32 nodes x 64 heads over 4096 rows: 405-455 us, 1.29
// to 1.46 PFLOP/s, at 1370 W, where the power limit holds the clock at 1740 MHz.
// One token of 64 heads, batch 64 over 4096 rows: 73 us, of them 58 at 5.2 TB/s
// in the tiles of 64 pairs, the rest start (6.5) and epilogue (3.5).
// Tried and not kept: one warp for all MMAs (4400 cycles a tile: its waits are
// not covered), P announced through a warp that forwards at the cluster's
// scope (1400 cycles a hand-off, 540 us), S held back behind the last PV (490
// to 540), tiles of 64 keys for one row tile (0-4 %, and 46 -> 63 us at LAT
// 256), the next tiles' keys prefetched into L2 (0-15 % slower: TMA's time).
// Every wait is bounded.
#include <cuda.h>
#include <math.h>

#include "common.cuh"
#include "kernels.h"
#include "latent_work.cuh"
#include "tc_ptx.cuh"

namespace {

using namespace sv::ptx;

constexpr int kBN = 128, kRope = 64, kThreads = 384, kPairs = 76;
constexpr uint32_t kPiece = 64 * 128;  // 64 rows (or keys) x 64 elements, 128-byte swizzle
constexpr uint32_t kWaitLimit = 1u << 22;
constexpr int kSegW = 3;      // a unit's fixed cost, in tiles (ragged trees: 1 143 us, 2 132, 3 128, 5 129)
constexpr int kJoinW = 6;     // what a join costs, in tiles
using sv::kLow;
constexpr float kTau = 16.f;  // the maximum moves when a tile exceeds it by more than 2^kTau

template <int LAT> struct Cfg {
  static constexpr int D = LAT + kRope;
  static constexpr int VJ = LAT / 256;           // blocks of 256 dims
  static constexpr int NB = LAT == 512 ? 2 : 4;  // tiles of latent places
  static constexpr int NR = LAT == 512 ? 1 : 2;  // tiles of rotary columns
  static constexpr int QG = LAT == 512 ? 3 : 5;  // column groups of a box of Q
  static constexpr uint32_t q_bytes = (D / 64) * kPiece;
  static constexpr uint32_t place = 2 * VJ * kPiece;  // 64 keys x 128 dims of every block
  static constexpr uint32_t c_bytes = 2 * place;      // of one tile
};
static_assert(Cfg<512>::D / 64 % Cfg<512>::QG == 0 && Cfg<256>::D / 64 % Cfg<256>::QG == 0, "Q's boxes cover the row");

template <int LAT> struct Bars {
  using C = Cfg<LAT>;
  // (full, p, ofree: the even CTA's count for both)
  uint64_t kfull[C::NB * 2], kread[C::NB * 2], vfull[C::NB * 2], empty[C::NB * 2], rfull[C::NR], rempty[C::NR];
  uint64_t qfull, qempty, sfull[2], sread[2], p[2], pv[2], ofree, vland, drain[2];
  sv::LatentRange range;
  uint32_t tmem;
  volatile int abort;
  float xmax[2][2][128];
};
template <int LAT> constexpr uint32_t smem_bytes() {
  using C = Cfg<LAT>;
  return C::q_bytes + 2 * kPiece + C::NB * C::c_bytes + C::NR * kPiece + sizeof(Bars<LAT>);
}
static_assert(smem_bytes<512>() <= 232448 && smem_bytes<256>() <= 232448, "shared memory per CTA exceeds 227 KB");

constexpr uint32_t kIdescS = idesc_bf16_f32(128, 128, 0, 0);   // Q, K both K-major
constexpr uint32_t kIdescPV = idesc_bf16_f32(128, 256, 0, 1);  // V is MN-major (dims contiguous)
constexpr uint32_t kColS = 256;

__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
  return p != 0;
}
// TMA load into this CTA whose bytes count on a barrier of the pair's even CTA.
__device__ __forceinline__ void load_2d(void *dst, const CUtensorMap *map, int c0, int c1, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];"
      ::"r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void load_3d(void *dst, const CUtensorMap *map, int c0, int c1, int c2, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
      ::"r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void load_4d(void *dst, const CUtensorMap *map, int c0, int c1, int c2, int c3, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];"
      ::"r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void load_5d(void *dst, const CUtensorMap *map, int c0, int c1, int c2, int c3, int c4,
                                        uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, %6}], [%7];"
      ::"r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "r"(bar)
      : "memory");
}
// Arrive on a barrier of the cluster, after this thread's (and, behind a
// __syncwarp, its warp's) writes for every CTA of the cluster.
__device__ __forceinline__ void arrive_release(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool try_wait_acquire(uint64_t *bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
      " selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
// Bounded wait that also ends once another role of the CTA has given up; its
// outcome is one for the warp.  CLUSTER: threads of the other CTA arrive.
template <bool CLUSTER = false, class B> __device__ __forceinline__ bool wait(B *bars, uint64_t *bar, uint32_t parity) {
  bool ok = !CLUSTER && mbar_test(bar, parity);
  for (uint32_t i = 0; !ok && i < kWaitLimit; ++i) {
    if ((ok = CLUSTER ? try_wait_acquire(bar, parity) : mbar_try_wait(bar, parity))) break;
    if ((i & 63) == 63 && bars->abort) break;
  }
  ok = __all_sync(0xffffffffu, ok);
  if (!ok) bars->abort = 1;
  return ok;
}
// The same where the phase was tested before (a test that need not suspend
// the thread, done while other work was left, costs less than a wait that
// finds its phase complete).
template <class B> __device__ __forceinline__ bool wait_tested(bool done, B *bars, uint64_t *bar, uint32_t parity) {
  return __all_sync(0xffffffffu, done) || wait(bars, bar, parity);
}

using sv::pack_bf16;

using Work = sv::LatentWork<kBN, 128>;
using Walk = sv::LatentWalk<Work>;

template <int LAT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    latent_tc_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_c,
                     const __grid_constant__ CUtensorMap tm_r, const __grid_constant__ CUtensorMap tm_tc,
                     const __grid_constant__ CUtensorMap tm_tr, const Work w, const uint64_t *__restrict__ anc,
                     __nv_bfloat16 *__restrict__ out, float *__restrict__ ws, int4 *__restrict__ desc,
                     float scale_log2, int row_end, int32_t *status, const sv::KvPages pg) {
  using C = Cfg<LAT>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t *sQ = smem, *sP = sQ + C::q_bytes, *sC = sP + 2 * kPiece, *sR = sC + C::NB * C::c_bytes;
  Bars<LAT> *bars = reinterpret_cast<Bars<LAT> *>(sR + C::NR * kPiece);

  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_rank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const int R = w.N * w.hq;

  // The 128-byte swizzle needs 1024-byte aligned tiles; both CTAs of a
  // cluster see the same layout, so they leave together.
  if (smem_u32(smem) & 1023u) {
    if (threadIdx.x == 0) sv::report(status, SPEC_DEV_INTERNAL);
    return;
  }
  grid_dep_launch();
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::NB * 2; ++i) {
      mbar_init(&bars->kfull[i], 1);
      mbar_init(&bars->kread[i], 1);
      mbar_init(&bars->vfull[i], 1);
      mbar_init(&bars->empty[i], 1);
    }
    for (int i = 0; i < C::NR; ++i) {
      mbar_init(&bars->rfull[i], 1);
      mbar_init(&bars->rempty[i], 1);
    }
    mbar_init(&bars->qfull, 1);
    mbar_init(&bars->qempty, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->sfull[i], 1);
      mbar_init(&bars->sread[i], 16);  // the softmax warps of both CTAs
      mbar_init(&bars->p[i], 8);       // those of 64 keys
      mbar_init(&bars->pv[i], 1);
      mbar_init(&bars->drain[i], 1);
    }
    mbar_init(&bars->ofree, 16);
    mbar_init(&bars->vland, 1);
    bars->abort = 0;
    mbar_fence_init();
  }
  if (warp == 1) tmem_alloc_pair(&bars->tmem, 512);
  if (warp == 0) {
    const sv::LatentRange range = sv::latent_range(w, pair, pairs, kSegW, kJoinW, rank == 0 ? desc + pair : nullptr,
                                                   blockIdx.x == 0 ? status : nullptr);
    if (lane == 0) bars->range = range;
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = bars->tmem;
  Walk walk(bars->range, kSegW);
  bool ok = true;

  // The cache row of prefix key `key` (its 64 keys lie in one block; a bad
  // block reads rows past the end: zeros).
  auto cache_row = [&](int b, int key) {
    const int row = sv::kv_row(pg, b, 1, 0, w.s_max, key, status);
    return row < 0 ? row_end : row;
  };

  // 64 rows from `row` on, of every block of 256 dims the half h, into a place.
  auto load_place = [&](uint8_t *dst, bool tree, int row, int h, int b, uint32_t bar) {
    if (tree) load_5d(dst, &tm_tc, 0, row, 2 * h, 0, b, bar);
    else load_4d(dst, &tm_c, 0, row, 2 * h, 0, bar);
  };

  if (warp == 0) {
    // ---------------------------------------------------------------- Q, K
    const bool me = elect_one();
    if (me) {
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_c);
      tma_prefetch_desc(&tm_r);
      tma_prefetch_desc(&tm_tc);
      tma_prefetch_desc(&tm_tr);
    }
    int g = 0;
    // Q of a segment: behind its first K, which need not wait for the last
    // segment's S (the first segment's Q first)
    auto load_q = [&](int seg) -> bool {
      if (!wait(bars, &bars->qempty, (seg & 1) ^ 1)) return false;
      if (me) {
        if (rank == 0) mbar_expect_tx(&bars->qfull, 2 * C::q_bytes);
        const uint32_t bar = mapa_cluster(&bars->qfull, 0);
        for (int i = 0; i < C::D / 64; i += C::QG)
          load_4d(sQ + i * kPiece, &tm_q, 0, walk.rt * 128 + (int)rank * 64, i, walk.b, bar);
      }
      __syncwarp();
      return true;
    };
    for (int seg = 0; ok && walk.advance(w); ++seg) {
      if (seg == 0 && !(ok = load_q(seg))) break;
      for (int t = walk.t0; ok && t < walk.t1; ++t, ++g) {
        const bool tree = t < w.tree_tiles;
        const int row = tree ? t * kBN + (int)rank * 64 : cache_row(walk.b, (t - w.tree_tiles) * kBN + (int)rank * 64);
        const int buf = g % C::NB, rb = g % C::NR;
        if (!(ok = wait(bars, &bars->rempty[rb], ((g / C::NR) & 1) ^ 1))) break;
        if (me) {
          if (rank == 0) mbar_expect_tx(&bars->rfull[rb], 2 * kPiece);
          const uint32_t bar = mapa_cluster(&bars->rfull[rb], 0);
          if (tree) load_3d(sR + rb * kPiece, &tm_tr, LAT, row, walk.b, bar);
          else load_2d(sR + rb * kPiece, &tm_r, LAT, row, bar);
        }
        __syncwarp();
        for (int h = 0; ok && h < 2; ++h) {
          const int s = buf * 2 + h;
          if (!(ok = wait(bars, &bars->empty[s], ((g / C::NB) & 1) ^ 1))) break;
          if (me) {
            if (rank == 0) mbar_expect_tx(&bars->kfull[s], 2 * C::place);
            load_place(sC + s * C::place, tree, row, h, walk.b, mapa_cluster(&bars->kfull[s], 0));
          }
          __syncwarp();
        }
        if (ok && t == walk.t0 && seg > 0) ok = load_q(seg);
      }
    }
  } else if (warp == 2) {
    // ---------------------------------------------------------------- V
    // the half of the dims that this CTA multiplies of the other CTA's keys,
    // over the half that it does not of its own
    const bool me = elect_one();
    const int h = 1 - (int)rank;
    int g = 0;
    while (ok && walk.advance(w)) {
      for (int t = walk.t0; ok && t < walk.t1; ++t, ++g) {
        const bool tree = t < w.tree_tiles;
        const int row = (tree ? t * kBN : cache_row(walk.b, (t - w.tree_tiles) * kBN)) + h * 64;
        const int s = g % C::NB * 2 + h;
        if (!(ok = wait(bars, &bars->kread[s], (g / C::NB) & 1))) break;
        if (me) {
          if (rank == 0) {
            mbar_expect_tx(&bars->vfull[s], C::place);      // this CTA's load
            mbar_expect_tx(&bars->vfull[s ^ 1], C::place);  // the odd CTA's
          }
          load_place(sC + s * C::place, tree, row, (int)rank, walk.b, mapa_cluster(&bars->vfull[s], 0));
        }
        __syncwarp();
      }
    }
  } else if (warp == 1 && rank == 0) {
    // ---------------------------------------------------------------- S
    // (S and PV are issued by two warps: an MMA waits for room in a short
    // queue, so the waits of one warp run under the products of the other)
    const uint32_t qa = smem_u32(sQ), ca = smem_u32(sC), ra = smem_u32(sR);
    int g = 0;
    for (int seg = 0; ok && walk.advance(w); ++seg) {
      if (!(ok = wait(bars, &bars->qfull, seg & 1))) break;
      for (int t = walk.t0; ok && t < walk.t1; ++t, ++g) {
        const int s = g % C::NB * 2, rb = g % C::NR;
        const uint32_t par = (g / C::NB) & 1, d = tmem + kColS + (g & 1) * 64;
        bool there = mbar_test(&bars->rfull[rb], (g / C::NR) & 1);
        // the buffer's last S has been read
        if (g >= 2 && !(ok = wait(bars, &bars->sread[g & 1], ((g >> 1) & 1) ^ 1))) break;
        if (!(ok = wait_tested(there, bars, &bars->rfull[rb], (g / C::NR) & 1))) break;
        there = mbar_test(&bars->kfull[s], par);
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_ss_pair(d, smem_desc_sw128(qa + LAT / 64 * kPiece + k * 32, 16, 1024),
                        smem_desc_sw128(ra + rb * kPiece + k * 32, 16, 1024), kIdescS, k > 0);
          mma_commit_pair_mc(&bars->rempty[rb], 3);
        }
        __syncwarp();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (!ok || !(ok = wait_tested(there, bars, &bars->kfull[s + h], par))) break;
          if (h == 0) there = mbar_test(&bars->kfull[s + 1], par);
          tc_fence_after();
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < C::VJ * 8; ++k) {
              // 16 dims: block k / 8, column group 2 h + (k / 4) % 2 of it
              const uint32_t qo = ((k >> 3) * 4 + 2 * h + ((k >> 2) & 1)) * kPiece + (k & 3) * 32;
              mma_ss_pair(d, smem_desc_sw128(qa + qo, 16, 1024),
                          smem_desc_sw128(ca + (s + h) * C::place + (k >> 2) * kPiece + (k & 3) * 32, 16, 1024), kIdescS, 1);
            }
            mma_commit_pair_mc(&bars->kread[s + h], 3);
            if (h == 1) {
              mma_commit_pair_mc(&bars->sfull[g & 1], 3);
              if (t == walk.t1 - 1) mma_commit_pair_mc(&bars->qempty, 3);
            }
          }
          __syncwarp();
        }
      }
    }
    if (!ok) {  // let issued MMAs finish before TMEM is freed
      if (elect_one()) mma_commit_pair_mc(&bars->drain[0], 1);
      __syncwarp();
      mbar_wait(&bars->drain[0], 0, kWaitLimit);
    }
  } else if (warp == 3 && rank == 0) {
    // ---------------------------------------------------------------- PV
    const uint32_t ca = smem_u32(sC), pa = smem_u32(sP);
    int g = 0;
    for (int seg = 0; ok && walk.advance(w); ++seg) {
      for (int t = walk.t0; ok && t < walk.t1; ++t, ++g) {
        const bool start = t == walk.t0;
        const int keys = t < w.tree_tiles ? kBN : min(kBN, walk.P - (t - w.tree_tiles) * kBN);
        const int s = g % C::NB * 2;
        const uint32_t par = (g / C::NB) & 1;
        if (keys < kBN) {
          // the softmax warps clear the V rows past the last key, once they are there
          for (int kh = 0; ok && kh < 2; ++kh) ok = wait(bars, &bars->vfull[s + kh], par);
          if (!ok) break;
          if (elect_one()) {
            arrive_release(mapa_cluster(&bars->vland, 0));
            arrive_release(mapa_cluster(&bars->vland, 1));
          }
          __syncwarp();
        }
        // the last segment's O has been read
        if (start && seg > 0 && !(ok = wait(bars, &bars->ofree, (seg - 1) & 1))) break;
#pragma unroll
        for (int kh = 0; kh < 2; ++kh) {
          const bool there = mbar_test(&bars->vfull[s + kh], par);
          if (!ok || !(ok = wait(bars, &bars->p[kh], g & 1)) ||
              !(ok = wait_tested(there, bars, &bars->vfull[s + kh], par)))
            break;
          tc_fence_after();
          if (elect_one()) {
            const uint32_t vb = ca + (s + kh) * C::place, pb = pa + kh * kPiece;
#pragma unroll
            for (int j = 0; j < C::VJ; ++j)
#pragma unroll
              for (int k = 0; k < 4; ++k)
                mma_ss_pair(tmem + j * 128, smem_desc_sw128(pb + k * 32, 16, 1024),
                            smem_desc_sw128(vb + j * 2 * kPiece + k * 2048, kPiece, 1024), kIdescPV, !start || kh || k > 0);
            mma_commit_pair_mc(&bars->empty[s + kh], 3);
            mma_commit_pair_mc(&bars->pv[kh], 3);
          }
          __syncwarp();
        }
      }
    }
    if (!ok) {
      if (elect_one()) mma_commit_pair_mc(&bars->drain[1], 1);
      __syncwarp();
      mbar_wait(&bars->drain[1], 0, kWaitLimit);
    }
  } else if (warp >= 4) {
    // ---------------------------------------------------------------- softmax
    // Lane L of TMEM: row L % 64, keys [64 (L / 64), +64) of a tile; this
    // warp takes columns [32 h, +32) of its lanes.  The four threads of a row
    // exchange their maxima at a barrier of the four warps of 32 rows.
    const int quarter = warp & 3, h = (warp - 4) >> 2, L = quarter * 32 + lane, r = L & 63, half = L >> 6;
    const uint32_t lane_off = (uint32_t)(quarter * 32) << 16;
    auto row_sync = [&]() { asm volatile("bar.sync %0, 128;" ::"r"(1 + (quarter & 1)) : "memory"); };
    // the four threads' values of this row, in one order for all of them
    auto row_put = [&](int buf, float v) { bars->xmax[buf][h][L] = v; };
    const uint32_t sread_bar = mapa_cluster(&bars->sread[0], 0), p_bar = mapa_cluster(&bars->p[half], 0);
    const int words = SPEC_MASK_WORDS(w.N);
    int g = 0, ragged = 0;
    bool s_there = false;
    while (walk.advance(w)) {
      const int row = walk.rt * 128 + (int)rank * 64 + r;
      const bool row_ok = row < R;
      const uint64_t *mask = anc + ((int64_t)walk.b * w.N + (row_ok ? row / w.hq : 0)) * words;
      float m = kLow, l = 0.f;
      for (int t = walk.t0; t < walk.t1; ++t, ++g) {
        // which of this thread's 32 keys the row sees
        const bool tree = t < w.tree_tiles;
        const int first = half * 64 + h * 32;
        const int left = (tree ? w.N - t * kBN : walk.P - (t - w.tree_tiles) * kBN) - first;
        uint32_t vis = left >= 32 ? ~0u : left > 0 ? (1u << left) - 1 : 0u;
        if (tree && left > 0) vis &= row_ok ? (uint32_t)(mask[2 * t + half] >> (h * 32)) : 0u;
        if (ok) ok = wait_tested(s_there, bars, &bars->sfull[g & 1], (g >> 1) & 1);
        uint32_t x[32];
        if (ok) {
          tc_fence_after();
          tmem_ld32(tmem + lane_off + kColS + (g & 1) * 64 + h * 32, x);
          tmem_wait_ld();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(sread_bar + (g & 1) * 8);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) x[i] = 0;
        }
        if (__any_sync(0xffffffffu, vis != ~0u)) {
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (!((vis >> i) & 1)) x[i] = 0xff800000u;  // -inf
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int i = 0; i < 16; ++i)
          mx[i & 3] = fmax3(mx[i & 3], __uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1]));
        row_put(g & 1, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])));
        row_sync();
        const bool p_free = g > 0 && mbar_test(&bars->pv[half], (g - 1) & 1);
        const float mt = fmaxf(fmaxf(bars->xmax[g & 1][0][r], bars->xmax[g & 1][0][r + 64]),
                               fmaxf(bars->xmax[g & 1][1][r], bars->xmax[g & 1][1][r + 64])) * scale_log2;
        const bool need = mt > m + kTau;
        if (__any_sync(0xffffffffu, need)) {
          const float a = need ? ex2(m - mt) : 1.f;
          if (need) {
            m = mt;
            l *= a;
          }
          if (t > walk.t0) {
            if (ok && (ok = wait(bars, &bars->pv[1], (g - 1) & 1))) {
              tc_fence_after();
#pragma unroll 1
              for (int c = h * (LAT / 4); c < (h + 1) * (LAT / 4); c += 16) {
                uint32_t o[16];
                tmem_ld16(tmem + lane_off + c, o);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * a);
                tmem_st16(tmem + lane_off + c, o);
              }
              tmem_wait_st();
              tc_fence_before();
            }
            row_sync();  // PV of the first keys adds to what all four warps scale
          }
        }
        // P = 2^(x scale - m), rounded to bf16 for the product (2^-8 of each
        // weight, either way); the row sum takes it unrounded
        const float2 sc = make_float2(scale_log2, scale_log2), nm = make_float2(-m, -m);
        float2 acc[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
        uint32_t pk[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          float2 e = fma2(make_float2(__uint_as_float(x[2 * i]), __uint_as_float(x[2 * i + 1])), sc, nm);
          e = make_float2(ex2(e.x), ex2(e.y));
          acc[i & 3] = add2(acc[i & 3], e);
          pk[i] = pack_bf16(e.x, e.y);
        }
        const float2 sum = add2(add2(acc[0], acc[1]), add2(acc[2], acc[3]));
        l += sum.x + sum.y;
        if (g > 0 && ok) ok = wait_tested(p_free, bars, &bars->pv[half], (g - 1) & 1);  // the last P has been read
        if (ok) {
          uint8_t *dst = sP + half * kPiece + r * 128;
#pragma unroll
          for (int c = 0; c < 4; ++c)
            *reinterpret_cast<uint4 *>(dst + (((h * 4 + c) ^ (r & 7)) << 4)) =
                make_uint4(pk[4 * c], pk[4 * c + 1], pk[4 * c + 2], pk[4 * c + 3]);
        }
        const int keys = tree ? kBN : min(kBN, walk.P - (t - w.tree_tiles) * kBN);
        if (keys < kBN) {
          // rows past the prefix may hold anything, NaN among it: cleared
          if (ok) ok = wait<true>(bars, &bars->vland, ragged & 1);
          ++ragged;
          if (ok) {
            uint8_t *v = sC + (g % C::NB * 2 + half) * C::place;
            const int from = max(keys - half * 64, 0);  // among the 64 keys whose P these warps write
            const int n = max(64 - from, 0) * 16;        // 16-byte pieces of one block of 256 dims
            for (int e = h * 64 + r; e < n * C::VJ; e += 128) {
              const int j = e / n, f = e - j * n, c = f & 15;
              *reinterpret_cast<uint4 *>(v + (j * 2 + (c >> 3)) * kPiece + (from + (f >> 4)) * 128 +
                                         (c & 7) * 16) = make_uint4(0, 0, 0, 0);
            }
          }
        }
        s_there = mbar_test(&bars->sfull[(g + 1) & 1], ((g + 1) >> 1) & 1);
        if (ok) {
          fence_proxy_async_smem();
          tc_fence_before();
          __syncwarp();
          // What the odd CTA wrote is read by products that the even one issues.
          // Every thread's fence has its writes in shared memory before the arrival
          // leaves the SM; the arrival itself releases at the CTA's scope.  That
          // this orders them is an assumption: the PTX memory model wants the
          // cluster's scope, whose release drains the thread's memory operations
          // (800 to 1000 cycles a tile: the serving case 405 -> 540 us; an acquire
          // of that scope costs nothing, but has no release to meet).  The same
          // holds for S and O read (sread, ofree), behind the wait for the loads.
          if (lane == 0) mbar_arrive_cluster(p_bar);
        }
      }
      // the whole row's sum
      row_sync();
      row_put(g & 1, l);
      row_sync();
      const float lt = (bars->xmax[g & 1][0][r] + bars->xmax[g & 1][0][r + 64]) +
                       (bars->xmax[g & 1][1][r] + bars->xmax[g & 1][1][r + 64]);
      row_sync();
      if (ok) ok = wait(bars, &bars->pv[1], (g - 1) & 1);
      if (ok) {
        tc_fence_after();
        const bool whole = walk.t0 == 0 && walk.t1 == walk.T;
        const float inv = whole ? (lt == 0.f ? 0.f : 1.f / lt) : 1.f;  // a row that sees nothing: zeros
        __nv_bfloat16 *o = out + ((int64_t)walk.b * R + row) * LAT + half * 128;
        float *slot = ws + (size_t)(2 * pair + (walk.t0 > 0 ? 0 : 1)) * sv::latent_slot_floats(LAT, 128);
        const int lr = (int)rank * 64 + r;
#pragma unroll 1
        for (int c = h * (LAT / 4); c < (h + 1) * (LAT / 4); c += 32) {
          uint32_t v[32];
          tmem_ld32(tmem + lane_off + c, v);
          tmem_wait_ld();
          const int d = (c >> 7) * 256 + (c & 127);  // (+ half * 128)
          if (whole) {
            // rows to pieces of 64 bytes of a row (lanes of 32 rows would touch 32
            // lines with each store), over the part of P that the four warps of
            // these rows write next behind a barrier of theirs
            uint8_t *st = sP + half * kPiece + (quarter & 1) * 4096 + h * 2048;
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint4 u;
              u.x = pack_bf16(__uint_as_float(v[8 * i]) * inv, __uint_as_float(v[8 * i + 1]) * inv);
              u.y = pack_bf16(__uint_as_float(v[8 * i + 2]) * inv, __uint_as_float(v[8 * i + 3]) * inv);
              u.z = pack_bf16(__uint_as_float(v[8 * i + 4]) * inv, __uint_as_float(v[8 * i + 5]) * inv);
              u.w = pack_bf16(__uint_as_float(v[8 * i + 6]) * inv, __uint_as_float(v[8 * i + 7]) * inv);
              *reinterpret_cast<uint4 *>(st + lane * 64 + ((i ^ ((lane >> 1) & 3)) << 4)) = u;
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int to = i * 8 + (lane >> 2), piece = lane & 3;  // row among the warp's 32
              if (row - lane + to < R)
                *reinterpret_cast<uint4 *>(o + (to - lane) * LAT + d + 8 * piece) =
                    *reinterpret_cast<const uint4 *>(st + to * 64 + ((piece ^ ((to >> 1) & 3)) << 4));
            }
          } else if (row_ok) {
            float *dst = slot + sv::latent_at<LAT, 128>(lr, half * 128 + d);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              *reinterpret_cast<uint4 *>(dst + i * 4 * 128) = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
          }
        }
        if (!whole && row_ok && half == 0 && h == 0)
          *reinterpret_cast<float2 *>(slot + 128 * (size_t)LAT + 2 * lr) = make_float2(m, lt);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(mapa_cluster(&bars->ofree, 0));
      }
    }
  }

  // Nothing leaves while its pair may still copy into it, multiply from it
  // or arrive on it (after a wait that gave up: copies in flight land long
  // before the other roles' waits run out).
  __syncwarp();
  if (!ok && lane == 0) sv::report(status, SPEC_DEV_TIMEOUT);
  tc_fence_before();
  __syncthreads();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
using sv::MapDim;

// Pairs to run: two tiles (at max_prefix) each or more.  5000 keys of one
// token: 41 pairs 21.8 us, 21: 18.9, 14: 19.4, 11: 18.8 (parts to join).
int pairs_of(const SvLatentShape &s) {
  const long long units = (long long)s.batch * (((long long)s.n_nodes * s.hq + 127) / 128);
  const long long tiles = units * ((s.max_prefix + kBN - 1) / kBN + (s.n_nodes + kBN - 1) / kBN);
  return (int)((tiles + 1) / 2 < kPairs ? (tiles + 1) / 2 : kPairs);
}

template <int LAT>
int launch(const SvLatentShape &s, const void *q, const void *cache, const void *tree, const int32_t *prefix_len,
           const uint64_t *anc, void *out, float scale, void *ws, int32_t *status, cudaStream_t stream) {
  using C = Cfg<LAT>;
  const int pairs = pairs_of(s), R = s.n_nodes * s.hq;
  const long long row = C::D * 2, groups = C::D / 64, N = s.n_nodes;
  const long long cached = s.block_table ? (long long)s.num_blocks * s.block_size : (long long)s.batch * s.s_max;
  const long long rows = cached > 0 ? cached : 1;
  CUtensorMap mq, mc, mr, mtc, mtr;
  const MapDim in{64, 0, 64}, all{C::D, 0, 64}, none{0, 0, 0};
  // (the coordinates: element, row, column group; of a place the groups of a block, blocks)
  if (sv::make_map(&mq, q, {in, {R, row, 64}, {groups, 128, C::QG}, {s.batch, row * R, 1}, none}) != SPEC_OK ||
      sv::make_map(&mc, cache, {in, {rows, row, 64}, {4, 128, 2}, {C::VJ, 512, C::VJ}, none}) != SPEC_OK ||
      sv::make_map(&mr, cache, {all, {rows, row, 64}, none, none, none}) != SPEC_OK ||
      sv::make_map(&mtc, tree, {in, {N, row, 64}, {4, 128, 2}, {C::VJ, 512, C::VJ}, {s.batch, row * N, 1}}) != SPEC_OK ||
      sv::make_map(&mtr, tree, {all, {N, row, 64}, {s.batch, row * N, 1}, none, none}) != SPEC_OK)
    return SPEC_ERR_CUDA;
  int4 *desc = static_cast<int4 *>(ws);
  float *slots = reinterpret_cast<float *>(desc + kPairs);
  const Work w(prefix_len, s.batch, s.n_nodes, s.hq, s.s_max, s.max_prefix, C::D * 2);
  if (cudaFuncSetAttribute(latent_tc_kernel<LAT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           (int)smem_bytes<LAT>()) != cudaSuccess)
    return SPEC_ERR_CUDA;
  latent_tc_kernel<LAT><<<2 * pairs, kThreads, smem_bytes<LAT>(), stream>>>(
      mq, mc, mr, mtc, mtr, w, anc, (__nv_bfloat16 *)out, slots, desc, scale * 1.4426950408889634f, (int)rows, status,
      sv::KvPages{s.block_table, s.block_size, s.max_blocks, s.num_blocks});
  if (cudaGetLastError() != cudaSuccess) return SPEC_ERR_CUDA;
  if (pairs == 1) return SPEC_OK;
  return sv::launch_latent_join<LAT, 128>(slots, desc, (__nv_bfloat16 *)out, R, pairs, (long long)s.batch * w.RT, stream);
}

}  // namespace

size_t sv_latent_tc_ws_bytes(const SvLatentShape &s) {
  return kPairs * sizeof(int4) + 2 * (size_t)pairs_of(s) * sv::latent_slot_floats(s.latent_dim, 128) * sizeof(float);
}

int sv_latent_tc(const SvLatentShape &s, const void *q, const void *cache, const void *tree, const int32_t *prefix_len,
                 const uint64_t *anc, void *out, float scale, void *ws, int32_t *status, cudaStream_t stream) {
  return (s.latent_dim == 512 ? launch<512> : launch<256>)(s, q, cache, tree, prefix_len, anc, out, scale, ws, status,
                                                           stream);
}

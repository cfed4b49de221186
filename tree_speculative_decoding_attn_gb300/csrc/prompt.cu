// Causal attention of packed prompt tokens over expanded latent keys and
// values (bf16 in, float32 softmax and accumulation).
//
//   x_j = scale (q[0..127] . k_j + q[128..191] . rope_j),  out = sum_j softmax(x)_j v_j
// for the keys up to the query's own position.  2 (192 + 128) flops a query,
// key and head: tensor-bound for all but a few queries.
//
// A CTA takes 256 queries of one head as two tiles of 128, so that the softmax
// of one tile runs under the products of the other, and both share every
// key tile of 128:
//   S_i(j) = Q_i K(j)^T  (N = 128, K = 192; the rotary columns of K are one
//            64-column box shared by all heads)   768 cycles
//   O_i   += P_i(j) V(j) (N = 128 dims, K = 128; P in TMEM over S)  512 cycles
// P lies where S was, and S_i(j + 1) goes over it once PV_i(j) is done.
//   warp 0      loads Q, K and V, and clears the V rows past the sequence's
//               last key
//   warps 1, 2  the MMAs of tile 0 and 1 (an elected thread each); their S in
//               turns, or both tiles would multiply and then both wait
//   warps 4-19  softmax and output, eight warps a tile: a thread half a row;
//               P is announced in two parts, so that PV starts under the rest
// Shared memory behind Q holds three pairs of 16 KB pieces, taken in turn by
// the 128 dims of K(j), K(j + 1) and V(j) (V(j + 1) follows K(j), whose S is the
// first to be done, K(j + 2) follows V(j)), and two pieces for rotary columns.
// What bounds it: two tiles' MMAs are 2560 cycles a key tile (2660 by their
// shared-memory traffic), the chain S, softmax (1600), PV with its hand-offs
// 3100 to 3400.  8192 tokens of 32 heads 449 to 472 us, 1.46 to 1.53 PFLOP/s, 491
// (1.40) under sustained load, at the power limit (1365 W).  Steps: one MMA warp
// and eight softmax warps 4680 cycles, 527 us; a warp a tile 4060, 491; S in
// turns 3850, 483; P in two parts 476; V no longer waiting for its one place
// 470; one wait for several barriers, outputs through shared memory, and S(j + 1)
// behind a wait for PV(j) (without it 3 % less, 432 to 465, by an order of
// products that nothing promises) 450.  Without the exponentials (timing only) the same: not a
// limit of the exponential unit.  Not kept: scalar instead of two-wide float32
// arithmetic (+4 %), P in parts of 48 and 16 or 16 and 48 keys (+4 %).
// TMEM columns: S0 [0,128) S1 [128,256) O0 [256,384) O1 [384,512).
// Longest tiles are launched first.  Where CTAs are fewer than SMs (a chunk of
// few heads behind a long kept beginning) the keys are cut into parts, a CTA
// each, whose float32 partials a second kernel joins.  Every wait is bounded.
#include <cuda.h>
#include <math.h>

#include "common.cuh"
#include "kernels.h"
#include "latent_work.cuh"
#include "tc_ptx.cuh"

namespace {

using namespace sv::ptx;

constexpr int kBN = 128, kD = 128, kRope = 64, kThreads = 640, kTiles = 2, kSms = 152;
constexpr uint32_t kPiece = 128 * 128;  // 128 rows x 64 elements, 128-byte swizzle
constexpr uint32_t kQBytes = 3 * kPiece, kPair = 2 * kPiece, kRing = 3 * kPair + 2 * kPiece;
constexpr uint32_t kWaitLimit = 1u << 22;
using sv::kLow;
constexpr float kTau = 16.f;  // the maximum moves when a tile exceeds it by more than 2^kTau

struct Bars {
  uint64_t q[kTiles], kfull[2], kempty[2], vfull[2], vempty[2], vclear, sfull[kTiles], p[2][kTiles], pv[kTiles], turn[kTiles], drain[kTiles];
  uint32_t tmem;
  volatile int abort;
  // by half of the keys and row (one buffer: S(j + 1) comes after both halves' P(j))
  float xmax[2][kTiles * 128];
};
constexpr uint32_t kSmemBytes = kTiles * kQBytes + kRing + sizeof(Bars);
static_assert(kSmemBytes <= 232448, "shared memory per CTA exceeds 227 KB");

constexpr uint32_t kIdescS = idesc_bf16_f32(128, 128, 0, 0);   // Q, K both K-major
constexpr uint32_t kIdescPV = idesc_bf16_f32(128, 128, 0, 1);  // V is MN-major (dims contiguous)

__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
  return p != 0;
}
// Bounded wait that also ends once another role has given up; its outcome is
// one for the warp.
__device__ __forceinline__ bool wait(Bars *bars, uint64_t *bar, uint32_t parity) {
  bool ok = false;
  for (uint32_t i = 0; i < kWaitLimit; ++i) {
    if ((ok = mbar_try_wait(bar, parity))) break;
    if ((i & 63) == 63 && bars->abort) break;
  }
  ok = __all_sync(0xffffffffu, ok);
  if (!ok) bars->abort = 1;
  return ok;
}
// The same for several, whose tries overlap (one of a completed barrier takes
// some 180 cycles beside busy softmax warps).
struct Phase {
  uint64_t *bar;
  uint32_t parity;
};
template <int N> __device__ __forceinline__ bool wait(Bars *bars, const Phase (&ph)[N]) {
  bool ok = false;
  for (uint32_t i = 0; i < kWaitLimit; ++i) {
    ok = true;
#pragma unroll
    for (int k = 0; k < N; ++k) ok &= mbar_try_wait(ph[k].bar, ph[k].parity);
    if (ok) break;
    if ((i & 63) == 63 && bars->abort) break;
  }
  ok = __all_sync(0xffffffffu, ok);
  if (!ok) bars->abort = 1;
  return ok;
}
using sv::pack_bf16;

// A partial: 256 rows of 128 float32 sums, four dims by four ([32][256][4]: a
// thread that writes them holds a row, and a warp's store is one piece), then
// 256 pairs (maximum in log2 units, sum).
__host__ __device__ constexpr size_t slot_floats() { return 256 * (size_t)(kD + 2); }
__device__ __forceinline__ int slot_at(int row, int dim) { return ((dim >> 2) * 256 + row) * 4; }

__global__ void __launch_bounds__(kThreads, 1)
    prompt_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                  const __grid_constant__ CUtensorMap tm_r, const __grid_constant__ CUtensorMap tm_v,
                  const int32_t *__restrict__ q_off, const int32_t *__restrict__ kv_off, __nv_bfloat16 *__restrict__ out,
                  float *__restrict__ ws, int hq, int parts, int total_q, int total_kv, int max_q, float scale_log2,
                  int32_t *status) {
  const int head = blockIdx.x / parts, part = blockIdx.x - head * parts, b = blockIdx.y;
  if (parts > 1) grid_dep_launch();
  const int q_first = q_off[b], q_end = q_off[b + 1], k_first = kv_off[b], k_end = kv_off[b + 1];
  if (q_first < 0 || k_first < 0 || q_end < q_first || k_end < k_first || q_end > total_q || k_end > total_kv ||
      q_end - q_first > max_q) {
    if (threadIdx.x == 0) sv::report(status, SPEC_DEV_CAPACITY);
    return;
  }
  const int n = q_end - q_first, m_keys = k_end - k_first;
  const int q0 = (int)(gridDim.z - 1 - blockIdx.z) * kTiles * 128;  // first query of this CTA
  if (q0 >= n) return;

  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023u) {  // the 128-byte swizzle needs it
    if (threadIdx.x == 0) sv::report(status, SPEC_DEV_INTERNAL);
    return;
  }
  uint8_t *sQ = smem, *ring = sQ + kTiles * kQBytes, *sR = ring + 3 * kPair;
  Bars *bars = reinterpret_cast<Bars *>(ring + kRing);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;

  // key tiles of each query tile: up to its last query's position; of them
  // this part's, from tile j0 on
  int tiles[kTiles], all = 0;
#pragma unroll
  for (int i = 0; i < kTiles; ++i) {
    const int last = min(n, q0 + (i + 1) * 128) - 1;  // last query of the tile
    const int seen = q0 + i * 128 < n ? m_keys - n + last + 1 : 0;
    tiles[i] = seen > 0 ? (seen + kBN - 1) / kBN : 0;
    all = max(all, tiles[i]);
  }
  const int j0 = (int)((int64_t)all * part / parts);
  all = (int)((int64_t)all * (part + 1) / parts) - j0;
#pragma unroll
  for (int i = 0; i < kTiles; ++i) tiles[i] = max(0, min(tiles[i] - j0, all));
  const int keys_left = m_keys - j0 * kBN;  // from tile j0 on

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars->q[i], 1);
      mbar_init(&bars->kfull[i], 1);
      mbar_init(&bars->kempty[i], kTiles);
      mbar_init(&bars->vfull[i], 1);
      mbar_init(&bars->vempty[i], kTiles);
      mbar_init(&bars->sfull[i], 1);
      mbar_init(&bars->p[0][i], 8);
      mbar_init(&bars->p[1][i], 8);
      mbar_init(&bars->pv[i], 1);
      mbar_init(&bars->turn[i], 1);
      mbar_init(&bars->drain[i], 1);
    }
    mbar_init(&bars->vclear, 1);
    bars->abort = 0;
    mbar_fence_init();
  }
  if (warp == 1) tmem_alloc(&bars->tmem, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bars->tmem;
  bool ok = true;

  if (warp == 0) {
    // ---------------------------------------------------------------- loads
    const bool me = elect_one();
    if (me && all > 0) {
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_r);
      tma_prefetch_desc(&tm_v);
    }
    int k_done = 0, v_done = 0, at = 0;  // at: j mod 3
    auto rope = [&](int j) {
      mbar_expect_tx(&bars->kfull[j & 1], 3 * kPiece);
      tma_load_2d(sR + (j & 1) * kPiece, &tm_r, 0, k_first + (j0 + j) * kBN, &bars->kfull[j & 1]);
    };
    auto load_q = [&](int i) {
      if (tiles[i] == 0) return;
      mbar_expect_tx(&bars->q[i], kQBytes);
      for (int c = 0; c < 3; ++c)
        tma_load_3d(sQ + i * kQBytes + c * kPiece, &tm_q, c * 64, head, q_first + q0 + i * 128, &bars->q[i]);
    };
    for (int j = 0; ok && j < all; ++j) {
      const int row = k_first + (j0 + j) * kBN;
      if (j > 1 && !(ok = wait(bars, &bars->vempty[j & 1], ((j >> 1) & 1) ^ 1))) break;
      if (me) {
        if (j == 0) load_q(0);
        if (j < 2) rope(j);
        tma_load_3d(ring + at * kPair, &tm_k, 0, head, row, &bars->kfull[j & 1]);
        tma_load_3d(ring + at * kPair + kPiece, &tm_k, 64, head, row, &bars->kfull[j & 1]);
        if (j == 0) load_q(1);  // (S of tile 0 is first)
      }
      ++k_done;
      __syncwarp();
      if (j > 0 && !(ok = wait(bars, &bars->kempty[(j - 1) & 1], ((j - 1) >> 1) & 1))) break;
      at = at == 0 ? 2 : at - 1;  // (j + 2) mod 3
      if (me) {
        uint64_t *bar = &bars->vfull[j & 1];
        mbar_expect_tx(bar, kPair);
        tma_load_3d(ring + at * kPair, &tm_v, 0, head, row, bar);
        tma_load_3d(ring + at * kPair + kPiece, &tm_v, 64, head, row, bar);
        if (j > 0 && j + 1 < all) rope(j + 1);
      }
      at = at == 0 ? 2 : at - 1;  // (j + 1) mod 3
      ++v_done;
      __syncwarp();
    }
    if (ok && all > 0 && (ok = wait(bars, &bars->vfull[(all - 1) & 1], ((all - 1) >> 1) & 1))) {
      uint8_t *sV = ring + (all + 1) % 3 * kPair;
      // what follows the sequence's last key belongs to others: cleared
      const int keys = keys_left - (all - 1) * kBN;
      if (keys < kBN) {
        for (int e = lane; e < (kBN - keys) * 16; e += 32)
          *reinterpret_cast<uint4 *>(sV + (e & 8 ? kPiece : 0) + (keys + (e >> 4)) * 128 + (e & 7) * 16) =
              make_uint4(0, 0, 0, 0);
        fence_proxy_async_smem();
        __syncwarp();
        if (me) mbar_arrive(&bars->vclear);
      }
    }
    if (!ok) {  // let the copies into this CTA land before it exits
      for (int i = 0; i < kTiles; ++i)
        if (k_done > 0 && tiles[i] > 0) mbar_wait(&bars->q[i], 0, kWaitLimit);
      for (int j = k_done > 2 ? k_done - 2 : 0; j < k_done; ++j) mbar_wait(&bars->kfull[j & 1], (j >> 1) & 1, kWaitLimit);
      for (int j = v_done > 2 ? v_done - 2 : 0; j < v_done; ++j) mbar_wait(&bars->vfull[j & 1], (j >> 1) & 1, kWaitLimit);
    }
  } else if (warp < 1 + kTiles) {
    // ---------------------------------------------------------------- MMAs
    // (a warp a tile: an MMA waits for room in a short queue, so the waits of
    // one warp run under the products of the other)
    const int i = warp - 1;
    const uint32_t qa = smem_u32(sQ) + i * kQBytes, ring_a = smem_u32(ring), ra = smem_u32(sR);
    uint32_t ka = ring_a, va = ring_a + 2 * kPair;  // K(j) and V(j)
    const uint32_t s_col = tmem + i * 128, o_col = tmem + 256 + i * 128;
    const int nt = i == 0 ? tiles[0] : tiles[1];
    if (nt > 0) ok = wait(bars, &bars->q[i], 0);
    auto scores = [&](int j) {  // (the elected thread)
#pragma unroll
      for (int k = 0; k < 12; ++k) {
        const uint32_t off = (k >> 2) * kPiece + (k & 3) * 32;
        const uint32_t key = k < 8 ? ka + off : ra + (j & 1) * kPiece + (k & 3) * 32;
        mma_ss(s_col, smem_desc_sw128(qa + off, 16, 1024), smem_desc_sw128(key, 16, 1024), kIdescS, k > 0);
      }
      mma_commit(&bars->sfull[i]);
      mma_commit(&bars->kempty[j & 1]);
      mbar_arrive(&bars->turn[i]);
    };
    // What S(j) waits for: its keys, and its turn (issued side by side, both
    // tiles' products and then both their softmaxes would run at the same time).
    auto keys = [&](int j) { return Phase{&bars->kfull[j & 1], (uint32_t)(j >> 1) & 1}; };
    auto turn = [&](int j) {  // (of tile 0's first: none, a phase that is over)
      return Phase{&bars->turn[1 - i], (uint32_t)(i == 1 ? j : j - 1) & 1};
    };
    for (int j = -1; ok && j < all; ++j) {
      // P(j) V(j), then S(j + 1) over P(j), behind a wait for the products that
      // read it: products with different accumulators have no order that the
      // instruction set promises, although one thread issues both.
      // P comes in two parts, the first 32 keys of each half of 64 and the rest.
      auto values = [&](int c) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int k = (e >> 1) * 4 + c * 2 + (e & 1);
          mma_ts(o_col, s_col + k * 8, smem_desc_sw128(va + k * 2048, kPiece, 1024), kIdescPV, j > 0 || c > 0 || e > 0);
        }
      };
      const bool mine = j >= 0 && j < nt, next = j + 1 < all;
      if (mine) {
        if (keys_left - j * kBN < kBN && !(ok = wait(bars, &bars->vclear, 0))) break;
        if (!(ok = wait(bars, {{&bars->vfull[j & 1], (uint32_t)(j >> 1) & 1}, {&bars->p[0][i], (uint32_t)j & 1}}))) break;
        tc_fence_after();
        if (elect_one()) values(0);
        __syncwarp();
        if (!(ok = wait(bars, &bars->p[1][i], j & 1))) break;
        tc_fence_after();
        if (elect_one()) {
          values(1);
          mma_commit(&bars->pv[i]);
          mma_commit(&bars->vempty[j & 1]);
        }
        __syncwarp();
      } else if (j >= 0) {
        if (!(ok = wait(bars, &bars->vfull[j & 1], (j >> 1) & 1))) break;
        if (elect_one()) mbar_arrive(&bars->vempty[j & 1]);
        __syncwarp();
      }
      if (next) {
        if (j >= 0 && j + 1 < nt) ok = wait(bars, {keys(j + 1), turn(j + 1), {&bars->pv[i], (uint32_t)j & 1}});
        else ok = wait(bars, {keys(j + 1), turn(j + 1)});
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
          if (j + 1 < nt) {
            scores(j + 1);
          } else {
            mbar_arrive(&bars->kempty[(j + 1) & 1]);
            mbar_arrive(&bars->turn[i]);
          }
        }
      }
      __syncwarp();
      if (j >= 0) va = va == ring_a + 2 * kPair ? ring_a : va + kPair;
      ka = ka == ring_a + 2 * kPair ? ring_a : ka + kPair;
    }
    if (!ok) {  // let issued MMAs finish before TMEM is freed
      if (elect_one()) mma_commit(&bars->drain[i]);
      __syncwarp();
      mbar_wait(&bars->drain[i], 0, kWaitLimit);
    }
  } else if (warp >= 4) {
    // ---------------------------------------------------------------- softmax
    // Warps 4-11 tile 0, 12-19 tile 1; two warps share 32 rows, half h of the
    // keys (and of the output's dims) each.
    const int i = (warp - 4) >> 3, h = ((warp - 4) >> 2) & 1, quarter = warp & 3;
    const int r = quarter * 32 + lane, qi = q0 + i * 128 + r;  // this thread's query
    const int seen = qi < n ? keys_left - n + qi + 1 : 0;       // keys that it sees from tile j0 on (<= 0: none)
    const uint32_t s_addr = tmem + ((uint32_t)(quarter * 32) << 16) + i * 128, o_addr = s_addr + 256 + h * 64;
    const int nt = i == 0 ? tiles[0] : tiles[1];
    auto row_sync = [&]() { asm volatile("bar.sync %0, 64;" ::"r"(1 + i * 4 + quarter) : "memory"); };
    float m = kLow, l = 0.f;
    for (int j = 0; j < nt; ++j) {
      if (ok) ok = wait(bars, &bars->sfull[i], j & 1);
      uint32_t x[2][32];
      if (ok) {
        tc_fence_after();
        tmem_ld32(s_addr + h * 64, x[0]);
        tmem_ld32(s_addr + h * 64 + 32, x[1]);
        tmem_wait_ld();
      } else {
#pragma unroll
        for (int e = 0; e < 64; ++e) x[e >> 5][e & 31] = 0;
      }
      const int left = seen - j * kBN - h * 64;  // visible keys among this thread's 64
      if (__any_sync(0xffffffffu, left < 64)) {
#pragma unroll
        for (int e = 0; e < 64; ++e)
          if (e >= left) x[e >> 5][e & 31] = 0xff800000u;  // -inf
      }
      float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int e = 0; e < 32; ++e)
        mx[e & 3] = fmax3(mx[e & 3], __uint_as_float(x[e >> 4][(2 * e) & 31]), __uint_as_float(x[e >> 4][(2 * e + 1) & 31]));
      mx[0] = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
      bars->xmax[h][i * 128 + r] = mx[0];
      row_sync();  // also: both halves of S have been read, P may lie over them
      const float mt = fmaxf(mx[0], bars->xmax[1 - h][i * 128 + r]) * scale_log2;
      const bool need = mt > m + kTau;
      if (__any_sync(0xffffffffu, need)) {
        const float a = need ? ex2(m - mt) : 1.f;
        if (need) {
          m = mt;
          l *= a;
        }
        if (j > 0 && ok && (ok = wait(bars, &bars->pv[i], (j - 1) & 1))) {
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < 64; c += 16) {
            uint32_t o[16];
            tmem_ld16(o_addr + c, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * a);
            tmem_st16(o_addr + c, o);
          }
        }
      }
      // P = 2^(x scale - m) rounded to bf16 for the product (2^-8 of each
      // weight), the row sum takes it unrounded
      const float2 sc = make_float2(scale_log2, scale_log2), nm = make_float2(-m, -m);
      float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        uint32_t pk[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          float2 v = fma2(make_float2(__uint_as_float(x[c][2 * e]), __uint_as_float(x[c][2 * e + 1])), sc, nm);
          v = make_float2(ex2(v.x), ex2(v.y));
          acc[e & 1] = add2(acc[e & 1], v);
          pk[e] = pack_bf16(v.x, v.y);
        }
        if (ok) {
          tmem_st16(s_addr + h * 32 + c * 16, pk);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bars->p[c][i]);
        }
      }
      const float2 sum = add2(acc[0], acc[1]);
      l += sum.x + sum.y;
    }
    row_sync();
    bars->xmax[h][i * 128 + r] = l;
    row_sync();
    l = bars->xmax[0][i * 128 + r] + bars->xmax[1][i * 128 + r];
    if (ok && nt > 0) ok = wait(bars, &bars->pv[i], (nt - 1) & 1);
    if (ok) {
      tc_fence_after();
      if (parts > 1) {
        // a part that shows the row nothing leaves a sum of 0, and no O
        float *slot = ws + slot_floats() * (((size_t)blockIdx.z * gridDim.y + b) * gridDim.x + blockIdx.x);
        const int row = i * 128 + r;
        if (h == 0 && qi < n) *reinterpret_cast<float2 *>(slot + 256 * kD + 2 * row) = make_float2(m, l);
#pragma unroll 1
        for (int c = 0; nt > 0 && c < 2; ++c) {
          uint32_t v[32];
          tmem_ld32(o_addr + c * 32, v);
          tmem_wait_ld();
          if (qi >= n) continue;
          float *dst = slot + slot_at(row, h * 64 + c * 32);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            *reinterpret_cast<uint4 *>(dst + e * 4 * 256) = make_uint4(v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]);
        }
      } else {
        const float inv = l == 0.f ? 0.f : 1.f / l;  // a query that sees nothing: zeros
        // rows to pieces of 128 bytes of a row (32 lanes of 32 rows would touch 32
        // lines with each store), where this tile's Q lay
        uint8_t *st = sQ + i * kQBytes + ((warp - 4) & 7) * 4096;
#pragma unroll 1
        for (int c = 0; c < 2; ++c) {
          uint32_t v[32];
          if (nt > 0) {
            tmem_ld32(o_addr + c * 32, v);
            tmem_wait_ld();
          }
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint4 u = make_uint4(0, 0, 0, 0);
            if (nt > 0) {
              u.x = pack_bf16(__uint_as_float(v[8 * e]) * inv, __uint_as_float(v[8 * e + 1]) * inv);
              u.y = pack_bf16(__uint_as_float(v[8 * e + 2]) * inv, __uint_as_float(v[8 * e + 3]) * inv);
              u.z = pack_bf16(__uint_as_float(v[8 * e + 4]) * inv, __uint_as_float(v[8 * e + 5]) * inv);
              u.w = pack_bf16(__uint_as_float(v[8 * e + 6]) * inv, __uint_as_float(v[8 * e + 7]) * inv);
            }
            *reinterpret_cast<uint4 *>(st + lane * 128 + (((c * 4 + e) ^ (lane & 7)) << 4)) = u;
          }
        }
        __syncwarp();
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int to = e * 4 + (lane >> 3), piece = lane & 7, qt = qi - lane + to;  // row among the warp's 32
          if (qt < n)
            *reinterpret_cast<uint4 *>(out + ((int64_t)(q_first + qt) * hq + head) * kD + h * 64 + piece * 8) =
                *reinterpret_cast<const uint4 *>(st + to * 128 + ((piece ^ (to & 7)) << 4));
        }
      }
    }
  }

  __syncwarp();
  if (!ok && lane == 0) sv::report(status, SPEC_DEV_TIMEOUT);
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Joins the parts of a unit: block (8 queries, unit), the queries side by side as
// they lie, a thread four dims of one.
__global__ void __launch_bounds__(256)
    prompt_join_kernel(const float *__restrict__ ws, const int32_t *__restrict__ q_off,
                       const int32_t *__restrict__ kv_off, __nv_bfloat16 *__restrict__ out, int hq, int parts,
                       int total_q, int total_kv, int max_q) {
  __shared__ float s_a[8][sv::kMostParts], s_l[8];
  static_assert(sv::kMostParts >= kSms, "a part a CTA at most");
  grid_dep_wait();
  const int per = 256 / 8;  // blocks of a unit
  const int unit = blockIdx.x / per, row0 = (blockIdx.x - unit * per) * 8, head = unit % hq, b = blockIdx.y;
  const int q_first = q_off[b], q_end = q_off[b + 1], k_first = kv_off[b], k_end = kv_off[b + 1];
  if (q_first < 0 || k_first < 0 || q_end < q_first || k_end < k_first || q_end > total_q || k_end > total_kv ||
      q_end - q_first > max_q)
    return;  // reported by the main kernel
  const int z = unit / hq, qi0 = (int)(gridDim.x / (per * hq) - 1 - z) * kTiles * 128 + row0;
  if (qi0 >= q_end - q_first) return;
  const float *slot = ws + slot_floats() * ((((size_t)z * gridDim.y + b) * hq + head) * parts);
  {
    const int r = threadIdx.x >> 5;
    const bool there = qi0 + r < q_end - q_first;
    const float l = sv::latent_weights<sv::kMostParts>(parts, s_a[r], [&](int p) {
      const float2 ml = there ? *reinterpret_cast<const float2 *>(slot + p * slot_floats() + 256 * kD + 2 * (row0 + r))
                              : make_float2(0.f, 0.f);
      return ml.y == 0.f ? make_float2(-INFINITY, 0.f) : ml;  // (a part of nothing: no weight, and no sums to read)
    });
    if ((threadIdx.x & 31) == 0) s_l[r] = l;
  }
  __syncthreads();
  const int r = threadIdx.x & 7, dim = (threadIdx.x >> 3) * 4;
  if (qi0 + r >= q_end - q_first) return;
  constexpr int B = 8;  // parts in flight
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int p0 = 0; p0 < parts; p0 += B) {
    float4 x[B];
#pragma unroll
    for (int i = 0; i < B; ++i)
      if (p0 + i < parts && s_a[r][p0 + i] != 0.f)
        x[i] = *reinterpret_cast<const float4 *>(slot + (p0 + i) * slot_floats() + slot_at(row0 + r, dim));
#pragma unroll
    for (int i = 0; i < B; ++i)
      if (p0 + i < parts && s_a[r][p0 + i] != 0.f) sv::fma4(acc, s_a[r][p0 + i], x[i]);
  }
  sv::store4(out + ((int64_t)(q_first + qi0 + r) * hq + head) * kD + dim, acc, s_l[r]);
}

int q_tiles_of(const SvPromptShape &s) {
  const int longest = s.max_q < s.total_q ? s.max_q : s.total_q;
  return longest ? (longest + kTiles * 128 - 1) / (kTiles * 128) : 1;  // (none allowed: some may be there, to report)
}
// Parts of a unit's keys: as many as fill the SMs, of four tiles at least
// where sequences have the mean length.
int parts_of(const SvPromptShape &s) {
  const long long units = (long long)s.hq * s.batch * q_tiles_of(s);
  if (2 * units > kSms) return 1;
  const long long most = s.total_kv / (4ll * kBN * s.batch), n = kSms / units;
  return (int)(n < most ? n : most > 1 ? most : 1);
}

}  // namespace

size_t sv_prompt_ws_bytes(const SvPromptShape &s) {
  const int parts = parts_of(s);
  return parts > 1 ? slot_floats() * sizeof(float) * parts * s.hq * s.batch * q_tiles_of(s) : 0;
}

int sv_prompt_attn(const SvPromptShape &s, const void *q, const void *k, const void *k_rope, const void *v,
                   const int32_t *q_offsets, const int32_t *kv_offsets, void *out, float scale, void *ws, int32_t *status,
                   cudaStream_t stream) {
  const int q_tiles = q_tiles_of(s), parts = parts_of(s);
  CUtensorMap mq, mk, mr, mv;
  const sv::MapDim q_dims{kD + kRope, 0, 64}, dims{kD, 0, 64}, rope{kRope, 0, 64}, none{0, 0, 0};
  const long long q_head = (kD + kRope) * 2;
  // (the coordinates: element, head, token)
  if (sv::make_map(&mq, q, {q_dims, {s.hq, q_head, 1}, {s.total_q, s.hq * q_head, 128}, none, none}) != SPEC_OK ||
      sv::make_map(&mk, k, {dims, {s.hq, s.k_head * 2, 1}, {s.total_kv, s.k_token * 2, 128}, none, none}) != SPEC_OK ||
      sv::make_map(&mr, k_rope, {rope, {s.total_kv, s.rope_token * 2, 128}, none, none, none}) != SPEC_OK ||
      sv::make_map(&mv, v, {dims, {s.hq, s.v_head * 2, 1}, {s.total_kv, s.v_token * 2, 128}, none, none}) != SPEC_OK)
    return SPEC_ERR_CUDA;
  if (cudaFuncSetAttribute(prompt_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmemBytes) != cudaSuccess)
    return SPEC_ERR_CUDA;
  prompt_kernel<<<dim3(s.hq * parts, s.batch, q_tiles), kThreads, kSmemBytes, stream>>>(
      mq, mk, mr, mv, q_offsets, kv_offsets, (__nv_bfloat16 *)out, (float *)ws, s.hq, parts, s.total_q, s.total_kv,
      s.max_q, scale * 1.4426950408889634f, status);
  if (cudaGetLastError() != cudaSuccess) return SPEC_ERR_CUDA;
  if (parts == 1) return SPEC_OK;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(s.hq * q_tiles * (256 / 8), s.batch);
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, prompt_join_kernel, (const float *)ws, q_offsets, kv_offsets, (__nv_bfloat16 *)out,
                            s.hq, parts, s.total_q, s.total_kv, s.max_q) == cudaSuccess
             ? SPEC_OK
             : SPEC_ERR_CUDA;
}

// Tree attention over a cache of latent vectors for few rows a sequence, or few
// tiles in all (bf16 in, float32 softmax and accumulation): a token of a few
// heads, a short chain, a short cache.
//
//   x_j = scale q . c_j over the LAT + 64 dims,  out = sum_j softmax(x)_j c_j[:LAT].
// With 16 rows a key's 1152 bytes meet 35 kflop: HBM-bound, and a tcgen05 tile
// of 128 rows would be seven eighths padding, loaded by pairs that read every
// value twice.  Here a CTA streams whole rows once, 64 keys a tile (72 KB at
// LAT 512) through a ring of three, and multiplies with the warp-level matrix
// product (m16n8k16), whose shape fits 16 rows:
//   S: warp i of 8 takes keys [8 i, +8) of the tile; the 16 queries' fragments
//      of all 576 dims stay in its registers (144 of them)
//   softmax: S goes through shared memory, warp i takes rows 2 i and 2 i + 1,
//      keeps their running maximum and sum, and leaves P and what the rows'
//      outputs are scaled by
//   PV: warp i takes dims [64 i, +64) (LAT 256: 32), 64 keys deep
// Two barriers a tile; the load of the tile after next is issued behind the
// first, when every warp is done with the tile before.  A tile whose data are
// there is 2700 to 3000 cycles of work; in a long stream a CTA takes 1.53 to 1.63
// us a tile (3200 to 3400 cycles at 2.07 GHz), which is HBM's read rate (6.9 to 7.3
// TB/s in all).  Batch 64 of 16 heads over 4096 rows 59 us: 27 tiles a CTA 44, the
// rest start, partials and the join; one sequence of 5000 rows 11.4 (start 4, one
// tile a CTA 2, partial 1, join 3).
// Work: equal ranges of all (sequence, 16 rows) units, or whole units, a CTA each;
// cut units leave float32 partials for a second kernel.  Every wait is bounded.
#include <math.h>

#include "common.cuh"
#include "kernels.h"
#include "latent_work.cuh"
#include "tc_ptx.cuh"

namespace {

using namespace sv::ptx;
using sv::kLow;
using sv::pack_bf16;

constexpr int kRows = 16, kBN = 64, kRope = 64, kThreads = 256, kWarps = 8, kCtas = 152;
constexpr uint32_t kPiece = 64 * 128;  // 64 keys x 64 elements, 128-byte swizzle
constexpr uint32_t kWaitLimit = 1u << 22;
constexpr int kSegW = 2;  // a unit's fixed cost, in tiles
constexpr int kJoinW = 4;  // what a join costs, in tiles

using Work = sv::LatentWork<kBN, kRows>;
using Walk = sv::LatentWalk<Work>;

template <int LAT> struct Cfg {
  static constexpr int D = LAT + kRope;
  static constexpr int ST = LAT == 512 ? 3 : 5;  // tiles in the ring
  static constexpr int NT = LAT / kWarps / 8;    // n-tiles of 8 dims of a warp
  static constexpr uint32_t tile = D / 64 * kPiece;
};

struct Rest {
  uint64_t full[5];
  sv::LatentRange range;
  volatile int abort;
  alignas(16) float s[kRows][kBN + 4];
  float alpha[kRows], l[kRows], m[kRows];
};
template <int LAT> constexpr uint32_t smem_bytes() {
  return Cfg<LAT>::ST * Cfg<LAT>::tile + 2048 + sizeof(Rest);  // tiles, P, the rest
}
static_assert(smem_bytes<512>() <= 232448 && smem_bytes<256>() <= 232448, "shared memory per CTA exceeds 227 KB");

__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t *a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int LAT>
__global__ void __launch_bounds__(kThreads, 1)
    latent_few_kernel(const __grid_constant__ CUtensorMap tm_c, const __grid_constant__ CUtensorMap tm_t, const Work w,
                      const __nv_bfloat16 *__restrict__ q, const uint64_t *__restrict__ anc,
                      __nv_bfloat16 *__restrict__ out, float *__restrict__ ws, int4 *__restrict__ desc,
                      float scale_log2, int row_end, int32_t *status, const sv::KvPages pg) {
  using C = Cfg<LAT>;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t *sP = smem + C::ST * C::tile;
  Rest *rest = reinterpret_cast<Rest *>(sP + 2048);
  if (smem_u32(smem) & 1023u) {  // the 128-byte swizzle needs it
    if (threadIdx.x == 0) sv::report(status, SPEC_DEV_INTERNAL);
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int R = w.N * w.hq, words = SPEC_MASK_WORDS(w.N);
  grid_dep_launch();
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::ST; ++i) mbar_init(&rest->full[i], 1);
    rest->abort = 0;
    mbar_fence_init();
    tma_prefetch_desc(&tm_c);
    tma_prefetch_desc(&tm_t);
  }
  if (warp == 0) {
    const sv::LatentRange r =
        sv::latent_range(w, blockIdx.x, gridDim.x, kSegW, kJoinW, desc + blockIdx.x, blockIdx.x == 0 ? status : nullptr);
    if (lane == 0) rest->range = r;
  }
  __syncthreads();
  Walk walk(rest->range, kSegW);

  // Thread 0 loads ahead: its own walk over the tiles.  A tile's block is looked
  // up when the tile before it is issued, so that nothing waits for the table,
  // and divisions are left to a segment's start (they are 300 cycles of the
  // path from one barrier to the next).
  Walk far(rest->range, kSegW);
  bool far_more = false;
  int far_t = 0, far_g = 0, far_blk = 0, far_row = 0;  // block, and row in it (contiguous: in the cache)
  const int32_t *far_table = pg.table;
  auto far_segment = [&]() {
    far_more = far.advance(w);
    far_t = far.t0;
    const int key = max(0, far_t - w.tree_tiles) * kBN;
    if (!pg.table) {
      far_row = far.b * w.s_max + key;
    } else if (far_more) {
      far_table = pg.table + (int64_t)far.b * pg.max_blocks + key / pg.block_size;
      far_row = key % pg.block_size;
      if (far_t >= w.tree_tiles) far_blk = __ldg(far_table);
    }
  };
  if (threadIdx.x == 0) far_segment();
  auto load_next = [&]() {  // (thread 0)
    if (!far_more) return;
    uint64_t *bar = &rest->full[far_g % C::ST];
    uint8_t *dst = smem + far_g % C::ST * C::tile;
    mbar_expect_tx(bar, C::tile);
    if (far_t < w.tree_tiles) {
      tma_load_4d(dst, &tm_t, 0, far_t * kBN, 0, far.b, bar);
    } else {
      int row = far_row;
      if (pg.table) {
        row += far_blk * pg.block_size;
        if (far_blk < 0 || far_blk >= pg.num_blocks) {
          sv::report(status, SPEC_DEV_BAD_BLOCK);
          row = row_end;  // past the pool: zeros
        }
      }
      tma_load_3d(dst, &tm_c, 0, row, 0, bar);
      far_row += kBN;
    }
    ++far_g;
    if (++far_t >= far.t1) {
      far_segment();
    } else if (pg.table && far_t >= w.tree_tiles) {
      if (far_row >= pg.block_size) {
        far_row = 0;
        ++far_table;
      }
      far_blk = __ldg(far_table);
    }
  };

  const int r0 = lane >> 2, c2 = (lane & 3) * 2;  // fragment row (and + 8), first of two columns
  int g = 0;
  bool ok = true;
  for (int seg = 0; ok && walk.advance(w); ++seg) {
    const int row0 = walk.rt * kRows;
    const int64_t qrow = (int64_t)walk.b * R + row0;
    // the 16 queries (rows past the last: zeros) through the stage that the
    // ring fills next, behind the first barrier below, into fragments
    uint32_t a[C::D / 16][4];
    {
      constexpr int PER = kRows * (C::D / 8) / kThreads, REST = kRows * (C::D / 8) % kThreads;
      uint8_t *sQ = smem + (g + C::ST - 1) % C::ST * C::tile;
      uint4 v[PER + (REST > 0)];
      auto at = [&](int i) { return threadIdx.x + i * kThreads; };
#pragma unroll
      for (int i = 0; i < PER + (REST > 0); ++i) {
        const int r = at(i) / (C::D / 8), c = at(i) % (C::D / 8);
        v[i] = make_uint4(0, 0, 0, 0);
        if (r < kRows && row0 + r < R) v[i] = sv::ldg_stream(q + (qrow + r) * C::D + c * 8);
      }
      // (the first tiles' loads behind them: they fill the memory's queues)
      if (seg == 0 && threadIdx.x == 0)
        for (int i = 0; i < C::ST - 1; ++i) load_next();
#pragma unroll
      for (int i = 0; i < PER + (REST > 0); ++i) {
        const int r = at(i) / (C::D / 8), c = at(i) % (C::D / 8);
        if (r < kRows)
          *reinterpret_cast<uint4 *>(sQ + (c >> 3) * (kRows * 128) + r * 128 + (((c & 7) ^ (r & 7)) << 4)) = v[i];
      }
      fence_proxy_async_smem();  // a TMA copy is next there
      __syncthreads();
      const uint32_t base = smem_u32(sQ);
      const int r = lane & 15;
#pragma unroll
      for (int k = 0; k < C::D / 16; ++k)
        ldsm4(base + (k >> 2) * (kRows * 128) + r * 128 + ((((2 * k & 7) + (lane >> 4)) ^ (r & 7)) << 4), a[k]);
    }
    float o[C::NT][4];
#pragma unroll
    for (int n = 0; n < C::NT; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) o[n][i] = 0.f;
    float m = kLow, l = 0.f;  // of row 2 warp + lane / 16
    for (int t = walk.t0; t < walk.t1; ++t, ++g) {
      uint8_t *tile = smem + g % C::ST * C::tile;
      const uint32_t base = smem_u32(tile);
      const bool tree = t < w.tree_tiles;
      const int left = tree ? w.N - t * kBN : walk.P - (t - w.tree_tiles) * kBN;  // keys there are
      if (!mbar_wait(&rest->full[g % C::ST], (g / C::ST) & 1, kWaitLimit)) rest->abort = 1;
      if (!tree && left < kBN) {
        // rows past the prefix may hold anything, NaN among it: cleared
        for (int e = threadIdx.x; e < (kBN - left) * (LAT / 8); e += kThreads) {
          const int k = left + e / (LAT / 8), c = e % (LAT / 8);
          *reinterpret_cast<uint4 *>(tile + (c >> 3) * kPiece + k * 128 + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async_smem();
      }
      // S: 16 rows x this warp's 8 keys, in four sums
      float s[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
      {
        const int key = warp * 8 + (lane & 7);
        const uint32_t row = base + key * 128;
        // a load: this key's dims [32 k2, +32), 8 of them a group of 8 lanes;
        // three loads in flight
        static_assert(C::D / 32 % 3 == 0 || C::D / 32 % 2 == 0, "whole batches");
        constexpr int B = C::D / 32 % 3 == 0 ? 3 : 2;
#pragma unroll
        for (int k2 = 0; k2 < C::D / 32; k2 += B) {
          uint32_t b[B][4];
#pragma unroll
          for (int i = 0; i < B; ++i)
            ldsm4(row + ((k2 + i) >> 1) * kPiece + ((((((k2 + i) & 1) << 2) + (lane >> 3)) ^ (key & 7)) << 4), b[i]);
#pragma unroll
          for (int i = 0; i < B; ++i) {
            mma16816(s[(2 * (k2 + i)) & 3], a[2 * (k2 + i)], b[i][0], b[i][1]);
            mma16816(s[(2 * (k2 + i) + 1) & 3], a[2 * (k2 + i) + 1], b[i][2], b[i][3]);
          }
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j)
        rest->s[r0 + (j >> 1) * 8][warp * 8 + c2 + (j & 1)] = (s[0][j] + s[1][j]) + (s[2][j] + s[3][j]);
      __syncthreads();
      if (rest->abort) {
        ok = false;
        break;
      }
      if (threadIdx.x == 0) load_next();  // over the tile before this one
      // softmax: half a warp a row, four keys a lane
      {
        const int r = warp * 2 + (lane >> 4), row = row0 + r, k0 = (lane & 15) * 4;
        uint32_t see = left >= k0 + 4 ? 15u : left > k0 ? (1u << (left - k0)) - 1 : 0u;
        if (tree)
          see &= row < R ? (uint32_t)(anc[((int64_t)walk.b * w.N + row / w.hq) * words + t] >> k0) : 0u;
        const float4 x = *reinterpret_cast<const float4 *>(&rest->s[r][k0]);
        float p[4] = {x.x, x.y, x.z, x.w}, mt = m;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          p[i] = (see >> i) & 1 ? p[i] * scale_log2 : -INFINITY;
          mt = fmaxf(mt, p[i]);
        }
#pragma unroll
        for (int o = 8; o; o >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, o));
        const float al = ex2(m - mt);
        m = mt;
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = ex2(p[i] - mt);
        // P rounded to bf16 for the product (2^-8 of each weight), the row
        // sum (each lane's share of it) takes it unrounded
        l = l * al + ((p[0] + p[1]) + (p[2] + p[3]));
        *reinterpret_cast<uint2 *>(sP + r * 128 + ((((lane & 15) >> 1) ^ (r & 7)) << 4) + (lane & 1) * 8) =
            make_uint2(pack_bf16(p[0], p[1]), pack_bf16(p[2], p[3]));
        if ((lane & 15) == 0) rest->alpha[r] = al;
      }
      __syncthreads();
      const float al0 = rest->alpha[r0], al8 = rest->alpha[r0 + 8];
      if (__any_sync(0xffffffffu, al0 != 1.f || al8 != 1.f)) {
#pragma unroll
        for (int n = 0; n < C::NT; ++n) {
          o[n][0] *= al0;
          o[n][1] *= al0;
          o[n][2] *= al8;
          o[n][3] *= al8;
        }
      }
      // PV: 16 rows x this warp's dims, four loads in flight
#pragma unroll
      for (int k = 0; k < kBN / 16; ++k) {
        uint32_t p[4], b[C::NT / 2][4];
        const int pr = lane & 15, key = 16 * k + (lane & 15);
        ldsm4(smem_u32(sP) + pr * 128 + (((2 * k + (lane >> 4)) ^ (pr & 7)) << 4), p);
#pragma unroll
        for (int n = 0; n < C::NT / 2; ++n) {
          const int col = warp * (C::NT * 8) + n * 16;  // of 16 dims: 8 a half of the lanes
          ldsm4t(base + (col >> 6) * kPiece + key * 128 + (((((col & 63) >> 3) + (lane >> 4)) ^ (key & 7)) << 4), b[n]);
        }
#pragma unroll
        for (int n = 0; n < C::NT / 2; ++n) {
          mma16816(o[2 * n], p, b[n][0], b[n][1]);
          mma16816(o[2 * n + 1], p, b[n][2], b[n][3]);
        }
      }
    }
    if (!ok) break;
#pragma unroll
    for (int o2 = 8; o2; o2 >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o2);
    if ((lane & 15) == 0) {
      rest->l[warp * 2 + (lane >> 4)] = l;
      rest->m[warp * 2 + (lane >> 4)] = m;
    }
    __syncthreads();
    const bool whole = walk.t0 == 0 && walk.t1 == walk.T;
    float *slot = ws + (size_t)(2 * blockIdx.x + (walk.t0 > 0 ? 0 : 1)) * sv::latent_slot_floats(LAT, kRows);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = r0 + 8 * h;
      if (row0 + r >= R) continue;
      const float lr = rest->l[r], inv = lr == 0.f ? 0.f : 1.f / lr;  // a row that sees nothing: zeros
      const int col = warp * (C::NT * 8) + c2;
#pragma unroll
      for (int n = 0; n < C::NT; ++n) {
        if (whole)
          *reinterpret_cast<uint32_t *>(out + (qrow + r) * LAT + col + n * 8) =
              pack_bf16(o[n][2 * h] * inv, o[n][2 * h + 1] * inv);
        else
          *reinterpret_cast<float2 *>(slot + r * LAT + col + n * 8) = make_float2(o[n][2 * h], o[n][2 * h + 1]);
      }
    }
    if (!whole && threadIdx.x < kRows && row0 + (int)threadIdx.x < R)
      *reinterpret_cast<float2 *>(slot + kRows * LAT + 2 * threadIdx.x) =
          make_float2(rest->m[threadIdx.x], rest->l[threadIdx.x]);
    // (the next segment writes l and m behind two barriers at least)
  }
  if (!ok && threadIdx.x == 0) {
    sv::report(status, SPEC_DEV_TIMEOUT);
    // let the copies into this CTA land before it exits
    for (int i = far_g > C::ST ? far_g - C::ST : 0; i < far_g; ++i)
      mbar_wait(&rest->full[i % C::ST], (i / C::ST) & 1, kWaitLimit);
  }
}

// CTAs to run: no more than tiles (at max_prefix).
int ctas_of(const SvLatentShape &s) {
  const long long units = (long long)s.batch * (((long long)s.n_nodes * s.hq + kRows - 1) / kRows);
  const long long tiles = units * ((s.max_prefix + kBN - 1) / kBN + (s.n_nodes + kBN - 1) / kBN);
  return (int)(tiles < kCtas ? tiles : kCtas);
}

template <int LAT>
int launch(const SvLatentShape &s, const void *q, const void *cache, const void *tree, const int32_t *prefix_len,
           const uint64_t *anc, void *out, float scale, void *ws, int32_t *status, cudaStream_t stream) {
  using C = Cfg<LAT>;
  const int ctas = ctas_of(s), R = s.n_nodes * s.hq;
  const long long row = C::D * 2, groups = C::D / 64, N = s.n_nodes;
  const long long cached = s.block_table ? (long long)s.num_blocks * s.block_size : (long long)s.batch * s.s_max;
  const long long rows = cached > 0 ? cached : 1;
  CUtensorMap mc, mt;
  const sv::MapDim in{64, 0, 64}, none{0, 0, 0};
  // (the coordinates: element, row, column group, sequence)
  if (sv::make_map(&mc, cache, {in, {rows, row, kBN}, {groups, 128, (int)groups}, none, none}) != SPEC_OK ||
      sv::make_map(&mt, tree, {in, {N, row, kBN}, {groups, 128, (int)groups}, {s.batch, row * N, 1}, none}) != SPEC_OK)
    return SPEC_ERR_CUDA;
  int4 *desc = static_cast<int4 *>(ws);
  float *slots = reinterpret_cast<float *>(desc + kCtas);
  const Work w(prefix_len, s.batch, s.n_nodes, s.hq, s.s_max, s.max_prefix, C::D * 2);
  if (cudaFuncSetAttribute(latent_few_kernel<LAT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           (int)smem_bytes<LAT>()) != cudaSuccess)
    return SPEC_ERR_CUDA;
  latent_few_kernel<LAT><<<ctas, kThreads, smem_bytes<LAT>(), stream>>>(
      mc, mt, w, (const __nv_bfloat16 *)q, anc, (__nv_bfloat16 *)out, slots, desc, scale * 1.4426950408889634f,
      (int)rows, status, sv::KvPages{s.block_table, s.block_size, s.max_blocks, s.num_blocks});
  if (cudaGetLastError() != cudaSuccess) return SPEC_ERR_CUDA;
  return sv::launch_latent_join<LAT, kRows>(slots, desc, (__nv_bfloat16 *)out, R, ctas, (long long)s.batch * w.RT, stream);
}

}  // namespace

size_t sv_latent_few_ws_bytes(const SvLatentShape &s) {
  return kCtas * sizeof(int4) + 2 * (size_t)ctas_of(s) * sv::latent_slot_floats(s.latent_dim, kRows) * sizeof(float);
}

int sv_latent_few(const SvLatentShape &s, const void *q, const void *cache, const void *tree, const int32_t *prefix_len,
                  const uint64_t *anc, void *out, float scale, void *ws, int32_t *status, cudaStream_t stream) {
  return (s.latent_dim == 512 ? launch<512> : launch<256>)(s, q, cache, tree, prefix_len, anc, out, scale, ws, status,
                                                           stream);
}

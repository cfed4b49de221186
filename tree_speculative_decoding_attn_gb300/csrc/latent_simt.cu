// Tree attention over a cache of latent vectors on CUDA cores (float32).
//
// Row (node, head) has a query q in the latent space, a key is a cache or
// tree row c = [latent ; rotary], a value its latent part:
//   out = sum_j softmax_j(scale q . c_j) c_j[:LAT].
// One CTA takes 8 rows and a range of the keys, 32 at a time.  Scores: a
// warp holds four key rows in registers (lanes over their dims) and multiplies
// them with the 8 queries in shared memory.  Softmax: one warp a row, running
// maximum and sum.  Values: a thread owns one or two of the latent dims for
// all 8 rows.  Key ranges are joined by a second kernel.  What bounds it is
// the float32 FMA rate (every key row is read once per 8 rows, from L1 the
// second time); float32 caches are for exactness, not for speed.  A small call
// is a row's chain of loads, scores and the join: a tree of 5 nodes x 4 heads
// over 129 rows 8.3 us (18.8 with a warp's keys one after another, 13.0 with the
// join as an ordinary launch, 11.9 with the queries loaded behind the length, the
// join's ranges one after another and ranges of 32 keys).
#include <math.h>

#include "common.cuh"
#include "kernels.h"
#include "latent_work.cuh"
#include "tc_ptx.cuh"

namespace {

constexpr int kRows = 8, kKeys = 32, kThreads = 256, kRope = 64;
using sv::kLow;
constexpr int kMaxSplits = 128, kGrain = 16;  // ranges of keys, and what their lengths are multiples of

// A partial: LAT unnormalised sums, the maximum (log2 units), the sum of P.
constexpr int partial_floats(int lat) { return lat + 4; }

template <int LAT>
__global__ void __launch_bounds__(kThreads)
    latent_simt_kernel(const float *__restrict__ q, const float *__restrict__ cache, const float *__restrict__ tree,
                       const int32_t *__restrict__ prefix_len, const uint64_t *__restrict__ anc,
                       float *__restrict__ out, float *__restrict__ ws, int N, int hq, int s_max, int max_prefix,
                       int chunk, float scale_log2, int32_t *status, const sv::KvPages pg) {
  constexpr int D = LAT + kRope, PER = D / 32, VD = LAT / kThreads;
  __shared__ alignas(16) float s_q[kRows][D];
  __shared__ float s_p[kRows][kKeys];
  __shared__ float s_alpha[kRows], s_l[kRows], s_m[kRows];
  __shared__ int s_row[kKeys];  // cache row of a prefix key, -1 outside the pool
  const int R = N * hq, b = blockIdx.z, split = blockIdx.y, row0 = blockIdx.x * kRows;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  sv::ptx::grid_dep_launch();
  const int P = prefix_len[b];
  // (the queries before anything waits for the length)
#pragma unroll
  for (int i = 0; i < kRows * D / 4 / kThreads + 1; ++i) {
    const int e = threadIdx.x + i * kThreads, r = e / (D / 4);
    if (r >= kRows) break;
    reinterpret_cast<float4 *>(&s_q[0][0])[e] =
        row0 + r < R ? reinterpret_cast<const float4 *>(q + ((int64_t)b * R + row0) * D)[e] : make_float4(0.f, 0.f, 0.f, 0.f);
  }
  if (P < 0 || P > max_prefix || P > s_max) {
    if (threadIdx.x == 0) sv::report(status, SPEC_DEV_CAPACITY);
    return;
  }
  const int words = SPEC_MASK_WORDS(N), last = P + N;
  const int k0 = split * chunk, k1 = min(last, k0 + chunk);
  float acc[kRows][VD];
#pragma unroll
  for (int r = 0; r < kRows; ++r)
#pragma unroll
    for (int v = 0; v < VD; ++v) acc[r][v] = 0.f;
  float m = kLow, l = 0.f;  // of row `warp`
  for (int j0 = k0; j0 < k1; j0 += kKeys) {
    const int n = min(kKeys, k1 - j0);
    __syncthreads();  // the last tile's rows and P have been read
    if (threadIdx.x < n) {
      const int j = j0 + threadIdx.x;
      s_row[threadIdx.x] = j < P ? sv::kv_row(pg, b, 1, 0, s_max, j, status) : 0;
    }
    __syncthreads();
    auto key_row = [&](int j) -> const float * {
      if (j0 + j >= P) return tree + ((int64_t)b * N + (j0 + j - P)) * D;
      return s_row[j] < 0 ? nullptr : cache + (int64_t)s_row[j] * D;
    };
    constexpr int KW = kKeys / (kThreads / 32);  // keys of a warp: warp, warp + 8, ..
    float k[KW][PER], dot[KW][kRows];
#pragma unroll
    for (int j = 0; j < KW; ++j) {
      const float *c = warp + 8 * j < n ? key_row(warp + 8 * j) : nullptr;
#pragma unroll
      for (int i = 0; i < PER; ++i) k[j][i] = c ? c[lane + 32 * i] : 0.f;
    }
#pragma unroll
    for (int r = 0; r < kRows; ++r) {
#pragma unroll
      for (int j = 0; j < KW; ++j) dot[j][r] = 0.f;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const float x = s_q[r][lane + 32 * i];
#pragma unroll
        for (int j = 0; j < KW; ++j) dot[j][r] = fmaf(k[j][i], x, dot[j][r]);
      }
    }
#pragma unroll
    for (int j = 0; j < KW; ++j) {
      // eight sums over 32 lanes, one left in each group of four lanes
#pragma unroll
      for (int step = 0; step < 3; ++step) {
        const int o = 16 >> step, half = 4 >> step;
#pragma unroll
        for (int r = 0; r < half; ++r) {
          const bool up = lane & o;
          const float give = up ? dot[j][r] : dot[j][r + half];
          dot[j][r] = (up ? dot[j][r + half] : dot[j][r]) + __shfl_xor_sync(0xffffffffu, give, o);
        }
      }
      dot[j][0] += __shfl_xor_sync(0xffffffffu, dot[j][0], 2);
      dot[j][0] += __shfl_xor_sync(0xffffffffu, dot[j][0], 1);
      const int r = lane >> 2, key = warp + 8 * j;
      if ((lane & 3) == 0 && key < n) {
        bool see = row0 + r < R;
        if (see && j0 + key >= P) {
          const int t = j0 + key - P, node = (row0 + r) / hq;
          see = (anc[((int64_t)b * N + node) * words + (t >> 6)] >> (t & 63)) & 1ull;
        }
        s_p[r][key] = see ? dot[j][0] * scale_log2 : -INFINITY;
      }
    }
    __syncthreads();
    {
      const float x = lane < n ? s_p[warp][lane] : -INFINITY;
      const float mt = fmaxf(sv::warp_max(x), m);
      const float p = exp2f(x - mt), a = exp2f(m - mt);
      l = l * a + sv::warp_sum(p);
      m = mt;
      s_p[warp][lane] = p;
      if (lane == 0) s_alpha[warp] = a;
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < kRows; ++r)
#pragma unroll
      for (int v = 0; v < VD; ++v) acc[r][v] *= s_alpha[r];
#pragma unroll 8
    for (int j = 0; j < n; ++j) {
      const float *c = key_row(j);
#pragma unroll
      for (int v = 0; v < VD; ++v) {
        const float x = c ? c[threadIdx.x + v * kThreads] : 0.f;
#pragma unroll
        for (int r = 0; r < kRows; ++r) acc[r][v] = fmaf(s_p[r][j], x, acc[r][v]);
      }
    }
  }
  if (lane == 0) {
    s_l[warp] = l;
    s_m[warp] = m;
  }
  __syncthreads();
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    const int64_t row = (int64_t)b * R + row0 + r;
    if (row0 + r >= R) break;
    if (gridDim.y == 1) {
      const float inv = s_l[r] == 0.f ? 0.f : 1.f / s_l[r];  // a row that sees nothing: zeros
#pragma unroll
      for (int v = 0; v < VD; ++v) out[row * LAT + threadIdx.x + v * kThreads] = acc[r][v] * inv;
    } else {
      float *w = ws + (row * gridDim.y + split) * partial_floats(LAT);
#pragma unroll
      for (int v = 0; v < VD; ++v) w[threadIdx.x + v * kThreads] = acc[r][v];
      if (threadIdx.x == 0) {
        w[LAT] = s_m[r];
        w[LAT + 1] = s_l[r];
      }
    }
  }
}

// One CTA a row: the key ranges' sums, weighted by their maxima; eight in
// flight (a loop of one after another: 12 us more with 63 ranges).
template <int LAT>
__global__ void __launch_bounds__(128)
    latent_simt_join_kernel(const float *__restrict__ ws, float *__restrict__ out, const int32_t *__restrict__ prefix_len,
                            int R, int splits, int s_max, int max_prefix) {
  __shared__ float s_a[kMaxSplits], s_l;
  sv::ptx::grid_dep_wait();
  const int64_t row = blockIdx.x;
  const int P = prefix_len[row / R];
  const float *w = ws + row * splits * partial_floats(LAT);
  if (threadIdx.x < 32) {
    const float l = sv::latent_weights<kMaxSplits>(splits, s_a, [&](int s) {
      return *reinterpret_cast<const float2 *>(w + (int64_t)s * partial_floats(LAT) + LAT);
    });
    if (threadIdx.x == 0) s_l = l;
  }
  __syncthreads();
  if (P < 0 || P > max_prefix || P > s_max) return;  // reported by the main kernel
  constexpr int V = LAT / 128, B = 8;
  float acc[V];
#pragma unroll
  for (int v = 0; v < V; ++v) acc[v] = 0.f;
  for (int s0 = 0; s0 < splits; s0 += B) {
    float x[B][V];
#pragma unroll
    for (int i = 0; i < B; ++i)
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (s0 + i < splits) x[i][v] = w[(int64_t)(s0 + i) * partial_floats(LAT) + threadIdx.x + 128 * v];
#pragma unroll
    for (int i = 0; i < B; ++i)
#pragma unroll
      for (int v = 0; v < V; ++v)
        if (s0 + i < splits) acc[v] = fmaf(s_a[s0 + i], x[i][v], acc[v]);
  }
  const float inv = s_l == 0.f ? 0.f : 1.f / s_l;
#pragma unroll
  for (int v = 0; v < V; ++v) out[row * LAT + threadIdx.x + 128 * v] = acc[v] * inv;
}

// Ranges of keys: as many as fill the GPU's 152 SMs once (LAT 256: two CTAs an
// SM, by their registers; a few more than that would run a second time round:
// 16 heads, 2000 keys 15 us in 126 CTAs, 27 in 252).
int splits_of(const SvLatentShape &s, int *chunk) {
  const long long ctas = (long long)s.batch * ((s.n_nodes * s.hq + kRows - 1) / kRows);
  const int tiles = (s.max_prefix + s.n_nodes + kGrain - 1) / kGrain;
  long long n = (s.latent_dim == 512 ? 152 : 304) / ctas;
  n = n > tiles ? tiles : n;
  n = n > kMaxSplits ? kMaxSplits : n < 1 ? 1 : n;  // (what the join holds)
  const int each = (tiles + (int)n - 1) / (int)n;  // tiles of a range
  *chunk = each * kGrain;
  return (tiles + each - 1) / each;  // (in tiles: keys and a range's length together may pass 32 bits)
}

template <int LAT>
int launch(const SvLatentShape &s, const void *q, const void *cache, const void *tree, const int32_t *prefix_len,
           const uint64_t *anc, void *out, float scale, void *ws, int32_t *status, cudaStream_t stream) {
  int chunk;
  const int splits = splits_of(s, &chunk), R = s.n_nodes * s.hq;
  latent_simt_kernel<LAT><<<dim3((R + kRows - 1) / kRows, splits, s.batch), kThreads, 0, stream>>>(
      (const float *)q, (const float *)cache, (const float *)tree, prefix_len, anc, (float *)out, (float *)ws,
      s.n_nodes, s.hq, s.s_max, s.max_prefix, chunk, scale * 1.4426950408889634f, status,
      sv::KvPages{s.block_table, s.block_size, s.max_blocks, s.num_blocks});
  if (cudaGetLastError() != cudaSuccess) return SPEC_ERR_CUDA;
  if (splits == 1) return SPEC_OK;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(s.batch * R);
  cfg.blockDim = dim3(128);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, latent_simt_join_kernel<LAT>, (const float *)ws, (float *)out, prefix_len, R, splits,
                            s.s_max, s.max_prefix) == cudaSuccess
             ? SPEC_OK
             : SPEC_ERR_CUDA;
}

}  // namespace

size_t sv_latent_simt_ws_bytes(const SvLatentShape &s) {
  int chunk;
  const int splits = splits_of(s, &chunk);
  return splits == 1 ? 0 : (size_t)s.batch * s.n_nodes * s.hq * splits * partial_floats(s.latent_dim) * 4;
}

int sv_latent_simt(const SvLatentShape &s, const void *q, const void *cache, const void *tree,
                   const int32_t *prefix_len, const uint64_t *anc, void *out, float scale, void *ws, int32_t *status,
                   cudaStream_t stream) {
  return (s.latent_dim == 512 ? launch<512> : launch<256>)(s, q, cache, tree, prefix_len, anc, out, scale, ws, status,
                                                           stream);
}

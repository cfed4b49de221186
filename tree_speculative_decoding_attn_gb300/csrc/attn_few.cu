// Window tree attention of few rows, in one launch: a decode step, a short
// chain, a small tree.
//
// out = sum_k 2^(s_k - M) v_k / sum_k 2^(s_k - M) with s = scale log2(e) q.k
// over the sinks, the window and the tree's keys that the row's position and
// ancestor mask show it.  Sums and accumulators are float32, and P is too (bf16
// inputs: to 2^-17, below).
//
// What bounds it: latency in small calls, the cache's bytes in large ones.  A
// decode step in bf16 (32/8 heads of 128, window 1024, paged) takes 7.5 us from
// a graph, five float32 nodes of 4 heads over a window of 333 5.4: the launch
// 2 of it, then prefix length, block table and keys one after another, and a
// cluster barrier.  The step at batch 64 takes 53 us (270 MB, 5.1 TB/s), over a
// window of 4000 166 (1.05 GB, 6.3 TB/s).
//
// Work split: one cluster per (16 query rows, KV head, sequence), whose CTAs
// share its visible keys evenly, key by key (no tiles: every key's row is
// looked up by itself, so pages and cut windows need no care).  The partial
// results are pushed into the shared memory of the CTAs that own slices of the
// output (one cluster barrier; a pull would add a trip), which weigh and write
// them.
//
// float32 (CUDA cores): a CTA's keys are few enough to be in flight at once: K
// into registers (four lanes a key, two keys a lane group), V by asynchronous
// copies into shared memory.  So the softmax needs one pass and no running
// max: scores to shared memory, a warp a row for max, exp2 and sum, then P V
// with two dims and four rows a thread.  Measured against this, decode step:
// 512 threads and eight lanes a key 8.6 to 7.1 us, the next round's K ahead in
// registers 7.7, tiles of 32 keys and a second launch 22.
//
// bf16: 16 rows are one operand of the warp-level matrix product, whatever
// part of them is used; CUDA cores cost 14 us where these take 8 (4 nodes, 16
// rows), and 92 instead of 53 at batch 64.  The SM-pair kernel's tiles of 256
// rows take 0.8 us per 128 keys for any number of rows: 15 and 87 us.
#include <math.h>

#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "tc_ptx.cuh"

namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kRows = 16;                // query rows of a cluster
constexpr int kLanes = 4;                // that share a key
constexpr int kGroups = kThreads / kLanes;  // keys taken at once, half of a round
constexpr int kMaxCtas = 16;
constexpr int kSms = 152;
constexpr int kMaxKeys = 264;            // of a float32 CTA: 256 with a few sinks and nodes

__device__ __forceinline__ void copy16(void *dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(sv::ptx::smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cluster_arrive_relaxed() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The outputs that this CTA owns, from the partial results pushed to it:
// in [CTA][per] pieces of four dims, ml [CTA] the rows' max and sum.
template <typename T, int D, typename RowAt>
__device__ __forceinline__ void join(const float4 *in, const float2 (*ml)[kRows], int pieces, int per, RowAt row_at,
                                     T *out) {
  const int C = gridDim.x, rank = blockIdx.x;
  for (int j = threadIdx.x; j < min(per, pieces - rank * per); j += kThreads) {
    const int i = rank * per + j, rr = i / (D / 4), c = i % (D / 4) * 4;
    float M = -INFINITY, L = 0.f;
    for (int s = 0; s < C; ++s) M = fmaxf(M, ml[s][rr].x);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int s = 0; s < C; ++s) {
      const float2 v = ml[s][rr];
      const float f = v.x == -INFINITY ? 0.f : exp2f(v.x - M);  // (a CTA that saw no key of the row)
      const float4 x = in[s * per + j];
      L = fmaf(f, v.y, L);
      o.x = fmaf(f, x.x, o.x);
      o.y = fmaf(f, x.y, o.y);
      o.z = fmaf(f, x.z, o.z);
      o.w = fmaf(f, x.w, o.w);
    }
    const float inv = L > 0.f ? 1.f / L : 0.f;  // (a row that sees nothing: zeros)
    T *to = out + row_at(rr) + c;
    if constexpr (sizeof(T) == 2) {
      const __nv_bfloat162 w0 = __floats2bfloat162_rn(o.x * inv, o.y * inv);
      const __nv_bfloat162 w1 = __floats2bfloat162_rn(o.z * inv, o.w * inv);
      *reinterpret_cast<uint2 *>(to) =
          make_uint2(*reinterpret_cast<const uint32_t *>(&w0), *reinterpret_cast<const uint32_t *>(&w1));
    } else {
      *reinterpret_cast<float4 *>(to) = make_float4(o.x * inv, o.y * inv, o.z * inv, o.w * inv);
    }
  }
}
__device__ __forceinline__ void push(float4 *dst, int to, const float4 &x) {
  asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(sv::ptx::mapa_cluster(dst, to)), "f"(x.x),
               "f"(x.y), "f"(x.z), "f"(x.w)
               : "memory");
}
__device__ __forceinline__ void push(float2 *dst, int to, const float2 &x) {
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(sv::ptx::mapa_cluster(dst, to)), "f"(x.x), "f"(x.y)
               : "memory");
}

__device__ __forceinline__ float dot4(const float4 &x, const float4 &y, float a) {
  return fmaf(x.x, y.x, fmaf(x.y, y.y, fmaf(x.z, y.z, fmaf(x.w, y.w, a))));
}

template <int D>
__global__ void __launch_bounds__(kThreads, 2)
    attn_few_kernel(const float *__restrict__ q, const float *__restrict__ kc, const float *__restrict__ vc,
                    const float *__restrict__ kt, const float *__restrict__ vt, const int32_t *__restrict__ prefix_len,
                    const uint64_t *__restrict__ anc, float *__restrict__ out, int N, int Hq, int Hkv, int s_max,
                    int max_prefix, int cap, float scale_log2, int32_t *status, const sv::KvPages pg,
                    const sv::Window win) {
  constexpr int VEC = 4;                 // values of a 16-byte piece
  constexpr int LC = D / VEC / kLanes;      // 16-byte pieces of a key that a lane holds
  constexpr int PG = kThreads / (D / 2);  // thread groups of P V
  constexpr int MW = SPEC_MAX_NODES / 64;
  extern __shared__ uint4 dyn[];
  __shared__ __align__(16) float s_q[kRows][D];
  __shared__ __align__(16) float s_acc[PG][4][D];
  __shared__ float4 s_in[kRows * D / 4 + kMaxCtas];   // [CTA][its slice of this CTA's outputs]
  __shared__ float2 s_ml[kMaxCtas][kRows];            // the CTAs' max and sum of each row
  __shared__ float2 s_own[kRows];
  __shared__ uint64_t s_anc[kRows][MW];
  __shared__ int s_pos[kRows];
  float *sV = reinterpret_cast<float *>(dyn);         // [cap][D]
  float *sS = sV + (size_t)cap * D;                   // [kRows][ld]
  const int ld = cap + 4;

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int C = gridDim.x, rank = blockIdx.x, b = blockIdx.z / Hkv, kvh = blockIdx.z % Hkv;
  const int G = Hq / Hkv, r0 = blockIdx.y * kRows, nr = min(kRows, N * G - r0);
  const int P = prefix_len[b];
  if (P < 0 || P > max_prefix || P > s_max) {  // (the whole cluster)
    if (tid == 0) sv::report(status, SPEC_DEV_CAPACITY);
    return;
  }
  const auto row_at = [&](int rr) {  // element of the row's first dim, in q and out
    return (((int64_t)b * N + (r0 + rr) / G) * Hq + kvh * G + (r0 + rr) % G) * D;
  };
  cluster_arrive_relaxed();  // (waited for before the first push: the partners run)

  // the rows: queries, positions, ancestors
  for (int e = tid; e < nr * (D / VEC); e += kThreads) {
    const int rr = e / (D / VEC), c = e % (D / VEC);
    *reinterpret_cast<float4 *>(&s_q[rr][c * VEC]) = *reinterpret_cast<const float4 *>(q + row_at(rr) + c * VEC);
  }
  const int nw = (N + 63) >> 6;
  for (int e = tid; e < nr * nw; e += kThreads) {
    const int rr = e / nw;
    const int64_t node = (int64_t)b * N + (r0 + rr) / G;
    s_anc[rr][e - rr * nw] = anc[node * nw + e - rr * nw];
    if (e == rr * nw) s_pos[rr] = P + sv::win_depth(win, node, N);
  }

  // the visible keys: sinks [0, n_sink), window [lo, P), tree
  const int lo = max(0, P - win.window + 1), n_sink = min(win.sinks, lo), n_prefix = n_sink + P - lo;
  const int total = n_prefix + N, per_cta = (total + C - 1) / C;
  const int first = rank * per_cta, n = max(0, min(per_cta, total - first)), n4 = (n + 3) & ~3;
  const int group = tid / kLanes, l = tid % kLanes;
  const int nq = (nr + 3) >> 2;
  bool synced = false;
  for (int base = 0; base < n4; base += 2 * kGroups) {
    float4 kv[2][LC];
    int pos[2], node[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int i = base + h * kGroups + group, slot = first + i;
      pos[h] = 0;
      node[h] = -1;
#pragma unroll
      for (int j = 0; j < LC; ++j) kv[h][j] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (i >= n4) continue;
      const float *kp = nullptr, *vp = nullptr;
      if (i < n && slot < n_prefix) {
        pos[h] = slot < n_sink ? slot : lo + slot - n_sink;
        const int row = sv::kv_row(pg, b, Hkv, kvh, s_max, pos[h], status);
        if (row >= 0) {
          kp = kc + (int64_t)row * D;
          vp = vc + (int64_t)row * D;
        }
      } else if (i < n) {
        node[h] = slot - n_prefix;
        const int64_t row = ((int64_t)b * Hkv + kvh) * N + node[h];
        kp = kt + row * D;
        vp = vt + row * D;
        pos[h] = P + sv::win_depth(win, (int64_t)b * N + node[h], N);
      }
      // (a key past the CTA's, or of a bad block: zeros)
#pragma unroll
      for (int j = 0; j < LC; ++j) {
        const int c = (l + kLanes * j) * VEC;
        if (kp) kv[h][j] = *reinterpret_cast<const float4 *>(kp + c);
      }
#pragma unroll
      for (int j = 0; j < LC; ++j) {
        const int c = (l + kLanes * j) * VEC;
        if (vp)
          copy16(sV + (size_t)i * D + c, vp + c);
        else
          *reinterpret_cast<float4 *>(sV + (size_t)i * D + c) = make_float4(0.f, 0.f, 0.f, 0.f);
      }
    }
    if (!synced) __syncthreads();  // the rows are in place
    synced = true;
    // four rows at a time, two keys a lane group (one, where the second is
    // past the end)
    const int i0 = base + warp * (32 / kLanes);
    auto scores = [&](auto two) {
      constexpr int H = decltype(two)::value;
      for (int qd = 0; qd < nq; ++qd) {
        float a[2][4] = {};
#pragma unroll
        for (int j = 0; j < LC; ++j)
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float4 x = *reinterpret_cast<const float4 *>(&s_q[qd * 4 + r][(l + kLanes * j) * VEC]);
#pragma unroll
            for (int h = 0; h < H; ++h) a[h][r] = dot4(x, kv[h][j], a[h][r]);
          }
        // sums over the lanes of a key: one row each
        const bool up = l & 2, odd = l & 1;
        const int rr = qd * 4 + l;
#pragma unroll
        for (int h = 0; h < H; ++h) {
          const float x0 = (up ? a[h][2] : a[h][0]) + __shfl_xor_sync(0xffffffffu, up ? a[h][0] : a[h][2], 2);
          const float x1 = (up ? a[h][3] : a[h][1]) + __shfl_xor_sync(0xffffffffu, up ? a[h][1] : a[h][3], 2);
          const float y = (odd ? x1 : x0) + __shfl_xor_sync(0xffffffffu, odd ? x0 : x1, 1);
          const int i = base + h * kGroups + group;
          if (i >= n4 || rr >= nr) continue;
          bool vis = i < n && (pos[h] < win.sinks || s_pos[rr] - pos[h] < win.window);
          if (node[h] >= 0) vis = vis && ((s_anc[rr][node[h] >> 6] >> (node[h] & 63)) & 1ull);
          sS[rr * ld + i] = vis ? y * scale_log2 : -INFINITY;
        }
      }
    };
    if (i0 + kGroups < n4)
      scores(std::integral_constant<int, 2>{});
    else if (i0 < n4)
      scores(std::integral_constant<int, 1>{});
  }
  __syncthreads();
  // softmax over the CTA's keys, a warp a row
  for (int rr = warp; rr < nr; rr += kWarps) {
    float *s = sS + rr * ld;
    float m = -INFINITY, sum = 0.f;
#pragma unroll 2
    for (int i = lane; i < n4; i += 32) m = fmaxf(m, s[i]);
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
#pragma unroll 2
    for (int i = lane; i < n4; i += 32) {
      const float x = s[i], p = x == -INFINITY ? 0.f : exp2f(x - m);
      s[i] = p;
      sum += p;
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (lane == 0) s_own[rr] = make_float2(m, sum);
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
  // P V: two dims and four rows a thread; the groups that are left over share
  // out the keys
  const int quads = nq > 2 ? 4 : nq, parts = PG / quads;
  const int pg_i = tid / (D / 2), quad = pg_i % quads, d = tid % (D / 2) * 2;
  {
    float acc[4][2] = {};
    if (quad < nq) {
      const float *sp = sS + quad * 4 * ld;
#pragma unroll 2
      for (int k = pg_i / quads * 4; k < n4; k += parts * 4) {
        float4 p[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) p[r] = *reinterpret_cast<const float4 *>(sp + r * ld + k);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 v = *reinterpret_cast<const float2 *>(sV + (size_t)(k + i) * D + d);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const float w = i == 0 ? p[r].x : i == 1 ? p[r].y : i == 2 ? p[r].z : p[r].w;
            acc[r][0] = fmaf(w, v.x, acc[r][0]);
            acc[r][1] = fmaf(w, v.y, acc[r][1]);
          }
        }
      }
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) *reinterpret_cast<float2 *>(&s_acc[pg_i][r][d]) = make_float2(acc[r][0], acc[r][1]);
  }
  __syncthreads();
  cluster_wait();
  // push: slices of the outputs to the CTAs that own them, the rows' max and
  // sum to everyone
  const int pieces = nr * (D / 4), per = (pieces + C - 1) / C;
  for (int i = tid; i < pieces; i += kThreads) {
    const int rr = i / (D / 4), c = i % (D / 4) * 4;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int p = 0; p < parts; ++p) {
      const float4 y = *reinterpret_cast<const float4 *>(&s_acc[p * quads + (rr >> 2)][rr & 3][c]);
      x.x += y.x;
      x.y += y.y;
      x.z += y.z;
      x.w += y.w;
    }
    const int to = i / per;
    push(&s_in[rank * per + i - to * per], to, x);
  }
  if (tid < nr * C) {
    const int rr = tid / C, to = tid % C;
    push(&s_ml[rank][rr], to, s_own[rr]);
  }
  __syncwarp();
  cluster_arrive();
  cluster_wait();
  join<float, D>(s_in, s_ml, pieces, per, row_at, out);
}

// bf16, for any number of keys: a CTA's warps stream blocks of 16 keys, each
// through buffers of its own (no CTA barrier on the way), with a running max,
// and their results are weighed at the end.
// The next block's K is under way from the moment that the scores are done,
// its V from the end of P V.  P goes into the second product as the sum of
// two bf16 numbers, so that it is rounded to 2^-17 of itself.
constexpr int kBlock = 16;
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], const void *p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(sv::ptx::smem_u32(p))
               : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t (&r)[4], const void *p) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(sv::ptx::smem_u32(p))
               : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
               "{%0, %1, %2, %3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  const __nv_bfloat162 w = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&w);
}

template <int D>
struct Stream {
  static constexpr int kChunks = D / 8;              // 16-byte pieces of a row
  static constexpr int kOut = D + 8;                 // floats of a row of a warp's result
  static constexpr int kBuf = kBlock * D * 2;        // bytes of a block's K or V
  static constexpr int kWarpBytes = kRows * kOut * 4 > 2 * kBuf ? kRows * kOut * 4 : 2 * kBuf;
  // address of chunk c of row r: rows are 2 D bytes, the chunks of eight rows spread over the banks
  static __device__ __forceinline__ __nv_bfloat16 *at(void *buf, int r, int c) {
    return reinterpret_cast<__nv_bfloat16 *>(buf) + r * D + ((c ^ (r & 7)) * 8);
  }
};

template <int D>
__global__ void __launch_bounds__(kThreads, 2)
    attn_stream_kernel(const __nv_bfloat16 *__restrict__ q, const __nv_bfloat16 *__restrict__ kc,
                       const __nv_bfloat16 *__restrict__ vc, const __nv_bfloat16 *__restrict__ kt,
                       const __nv_bfloat16 *__restrict__ vt, const int32_t *__restrict__ prefix_len,
                       const uint64_t *__restrict__ anc, __nv_bfloat16 *__restrict__ out, int N, int Hq, int Hkv,
                       int s_max, int max_prefix, float scale_log2, int32_t *status, const sv::KvPages pg,
                       const sv::Window win) {
  using S = Stream<D>;
  constexpr int LC = S::kChunks / 4;  // pieces of a key that a lane copies
  constexpr int MW = SPEC_MAX_NODES / 64;
  extern __shared__ uint4 dyn[];
  __shared__ uint4 s_q[kRows * S::kChunks];
  __shared__ float4 s_in[kRows * D / 4 + kMaxCtas];
  __shared__ float2 s_ml[kMaxCtas][kRows];
  __shared__ float2 s_warp[kWarps][kRows];
  __shared__ uint64_t s_anc[kRows][MW];
  __shared__ int s_pos[kRows];

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int C = gridDim.x, rank = blockIdx.x, b = blockIdx.z / Hkv, kvh = blockIdx.z % Hkv;
  const int G = Hq / Hkv, r0 = blockIdx.y * kRows, nr = min(kRows, N * G - r0);
  const int P = prefix_len[b];
  if (P < 0 || P > max_prefix || P > s_max) {  // (the whole cluster)
    if (tid == 0) sv::report(status, SPEC_DEV_CAPACITY);
    return;
  }
  const auto row_at = [&](int rr) {  // element of the row's first dim, in q and out
    return (((int64_t)b * N + (r0 + rr) / G) * Hq + kvh * G + (r0 + rr) % G) * D;
  };
  cluster_arrive_relaxed();  // (waited for before the first push: the partners run)

  const int lo = max(0, P - win.window + 1), n_sink = min(win.sinks, lo), n_prefix = n_sink + P - lo;
  const int total = n_prefix + N, per_cta = (total + C - 1) / C;
  const int first = rank * per_cta, n = max(0, min(per_cta, total - first));
  uint8_t *mine = reinterpret_cast<uint8_t *>(dyn) + warp * S::kWarpBytes;
  void *sK = mine, *sV = mine + S::kBuf;
  const int group = lane >> 2, t = lane & 3;
  // a lane's two keys of a block, group and group + 8: rows to copy, and
  // position and node (-1: a prefix key, -2: none) for the masks
  struct Keys {
    const __nv_bfloat16 *k[2], *v[2];
    int pos[2], node[2];
  };
  auto look = [&](int block, Keys &x) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int i = block * kBlock + h * 8 + group, slot = first + i;
      x.k[h] = x.v[h] = nullptr;
      x.pos[h] = 0;
      x.node[h] = -2;
      if (i >= n) continue;
      if (slot < n_prefix) {
        x.pos[h] = slot < n_sink ? slot : lo + slot - n_sink;
        x.node[h] = -1;
        const int row = sv::kv_row(pg, b, Hkv, kvh, s_max, x.pos[h], status);
        if (row >= 0) {
          x.k[h] = kc + (int64_t)row * D;
          x.v[h] = vc + (int64_t)row * D;
        }
      } else {
        x.node[h] = slot - n_prefix;
        x.pos[h] = P + sv::win_depth(win, (int64_t)b * N + x.node[h], N);
        const int64_t row = ((int64_t)b * Hkv + kvh) * N + x.node[h];
        x.k[h] = kt + row * D;
        x.v[h] = vt + row * D;
      }
    }
  };
  auto copy = [&](void *buf, const __nv_bfloat16 *const (&src)[2]) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int j = 0; j < LC; ++j) {
        const int c = t + 4 * j;
        __nv_bfloat16 *dst = S::at(buf, h * 8 + group, c);
        if (src[h])
          copy16(dst, src[h] + c * 8);
        else  // (no key, or of a bad block: zeros)
          *reinterpret_cast<uint4 *>(dst) = make_uint4(0, 0, 0, 0);
      }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  const int blocks = (n + kBlock - 1) / kBlock;
  Keys keys;
  if (warp < blocks) {
    look(warp, keys);
    copy(sK, keys.k);
    copy(sV, keys.v);
  }

  // the rows: queries (zeros past the last), positions, ancestors
  for (int e = tid; e < kRows * S::kChunks; e += kThreads) {
    const int rr = e / S::kChunks, c = e % S::kChunks;
    *reinterpret_cast<uint4 *>(S::at(s_q, rr, c)) =
        rr < nr ? *reinterpret_cast<const uint4 *>(q + row_at(rr) + c * 8) : make_uint4(0, 0, 0, 0);
  }
  const int nw = (N + 63) >> 6;
  for (int e = tid; e < nr * nw; e += kThreads) {
    const int rr = e / nw;
    const int64_t node = (int64_t)b * N + (r0 + rr) / G;
    s_anc[rr][e - rr * nw] = anc[node * nw + e - rr * nw];
    if (e == rr * nw) s_pos[rr] = P + sv::win_depth(win, node, N);
  }
  __syncthreads();

  float acc[D / 8][4] = {}, m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  // (rows past the last mask as row 0 and are not written)
  const int row[2] = {group < nr ? group : 0, group + 8 < nr ? group + 8 : 0};
  const int at[2] = {s_pos[row[0]], s_pos[row[1]]};
  const int deepest = __reduce_max_sync(0xffffffffu, max(at[0], at[1]));
  for (int blk = warp; blk < blocks; blk += kWarps) {
    // ldmatrix's lane-to-row maps: A and V^T take rows lane & 15, K rows of eight keys
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    __syncwarp();
    float s[2][4] = {};
#pragma unroll
    for (int kk = 0; kk < D / 32; ++kk) {
      uint32_t a0[4], a1[4], k0[4], k1[4];
      ldsm4(a0, S::at(s_q, lane & 15, kk * 4 + (lane >> 4)));
      ldsm4(a1, S::at(s_q, lane & 15, kk * 4 + 2 + (lane >> 4)));
      ldsm4(k0, S::at(sK, lane & 7, kk * 4 + (lane >> 3)));
      ldsm4(k1, S::at(sK, 8 + (lane & 7), kk * 4 + (lane >> 3)));
      mma16816(s[0], a0, k0[0], k0[1]);
      mma16816(s[1], a0, k1[0], k1[1]);
      mma16816(s[0], a1, k0[2], k0[3]);
      mma16816(s[1], a1, k1[2], k1[3]);
    }
    Keys next;
    const bool more = blk + kWarps < blocks;
    if (more) look(blk + kWarps, next);
    __syncwarp();  // K is read
    if (more) copy(sK, next.k);
    // masks: element (i, e) of s is row `row[e / 2]`, key 8 i + 2 t + e % 2
    bool whole = true;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      whole = whole && keys.node[h] == -1 && (keys.pos[h] < win.sinks || deepest - keys.pos[h] < win.window);
    whole = __all_sync(0xffffffffu, whole);
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        s[i][e] *= scale_log2;
        s[i][e + 2] *= scale_log2;
        if (whole) continue;
        const int from = (2 * t + e) * 4;
        const int pos = __shfl_sync(0xffffffffu, keys.pos[i], from);
        const int node = __shfl_sync(0xffffffffu, keys.node[i], from);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          bool vis = node != -2 && (pos < win.sinks || at[h] - pos < win.window);
          if (node >= 0) vis = vis && ((s_anc[row[h]][node >> 6] >> (node & 63)) & 1ull);
          if (!vis) s[i][e + 2 * h] = -INFINITY;
        }
      }
    float p[2][4];
    bool moved = false;
    float corr[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float mx = fmaxf(fmaxf(s[0][2 * h], s[0][2 * h + 1]), fmaxf(s[1][2 * h], s[1][2 * h + 1]));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const float mn = fmaxf(m[h], mx), z = mn == -INFINITY ? 0.f : mn;  // (nothing seen yet: every p is 0)
      corr[h] = exp2f(m[h] - z);
      moved = moved || mn != m[h];
      m[h] = mn;
      float sum = 0.f;
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 2; ++e) sum += p[i][2 * h + e] = exp2f(s[i][2 * h + e] - z);
      l[h] = fmaf(l[h], corr[h], sum);
    }
    if (__any_sync(0xffffffffu, moved)) {
#pragma unroll
      for (int d = 0; d < D / 8; ++d)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[d][e] *= corr[e >> 1];
    }
    uint32_t hi[4], rest[4];
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float x = p[i][2 * h], y = p[i][2 * h + 1];
        const uint32_t w = pack(x, y);
        hi[2 * i + h] = w;
        rest[2 * i + h] = pack(x - __uint_as_float(w << 16), y - __uint_as_float(w & 0xFFFF0000u));
      }
    if (more)
      asm volatile("cp.async.wait_group 1;" ::: "memory");
    else
      asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncwarp();
#pragma unroll
    for (int d = 0; d < D / 16; ++d) {
      uint32_t v[4];
      ldsm4_trans(v, S::at(sV, lane & 15, d * 2 + (lane >> 4)));
      mma16816(acc[2 * d], hi, v[0], v[1]);
      mma16816(acc[2 * d + 1], hi, v[2], v[3]);
      mma16816(acc[2 * d], rest, v[0], v[1]);
      mma16816(acc[2 * d + 1], rest, v[2], v[3]);
    }
    __syncwarp();  // V is read
    if (more) copy(sV, next.v);
    keys = next;
  }
  // the warps' results, in their own buffers
  float *res = reinterpret_cast<float *>(mine);
#pragma unroll
  for (int d = 0; d < D / 8; ++d)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      *reinterpret_cast<float2 *>(res + (group + 8 * h) * S::kOut + d * 8 + 2 * t) =
          make_float2(acc[d][2 * h], acc[d][2 * h + 1]);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
    if (t == 0) s_warp[warp][group + 8 * h] = make_float2(m[h], l[h]);
  }
  __syncthreads();
  cluster_wait();
  // push: slices of the outputs to the CTAs that own them, the rows' max and
  // sum to everyone
  const int pieces = nr * (D / 4), per = (pieces + C - 1) / C;
  const auto weigh = [&](int rr, float (&f)[kWarps]) {
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, f[w] = s_warp[w][rr].x);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) f[w] = f[w] == -INFINITY ? 0.f : exp2f(f[w] - M);
    return M;
  };
  for (int i = tid; i < pieces; i += kThreads) {
    const int rr = i / (D / 4), c = i % (D / 4) * 4;
    float f[kWarps];
    weigh(rr, f);
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float4 y = *reinterpret_cast<const float4 *>(reinterpret_cast<const uint8_t *>(dyn) + w * S::kWarpBytes +
                                                         (rr * S::kOut + c) * 4);
      x.x = fmaf(f[w], y.x, x.x);
      x.y = fmaf(f[w], y.y, x.y);
      x.z = fmaf(f[w], y.z, x.z);
      x.w = fmaf(f[w], y.w, x.w);
    }
    const int to = i / per;
    push(&s_in[rank * per + i - to * per], to, x);
  }
  if (tid < nr * C) {
    const int rr = tid / C, to = tid % C;
    float f[kWarps], L = 0.f;
    const float M = weigh(rr, f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) L = fmaf(f[w], s_warp[w][rr].y, L);
    push(&s_ml[rank][rr], to, make_float2(M, L));
  }
  __syncwarp();
  cluster_arrive();
  cluster_wait();
  join<__nv_bfloat16, D>(s_in, s_ml, pieces, per, row_at, out);
}

template <int D>
constexpr int kStreamBytes = kWarps *Stream<D>::kWarpBytes;
template <int D>
constexpr int few_bytes(int cap) {
  return cap * D * 4 + kRows * (cap + 4) * 4;
}

// Gives a kernel its cluster and shared-memory sizes, once per device, and
// tells the largest cluster that the device runs: 16 CTAs is more than every
// device has to take (a partition whose GPCs have fewer SMs does not).
template <typename K>
int prepare(K kern, int most_bytes, std::atomic<uint64_t> (&known)[2]) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) {
    (void)cudaGetLastError();
    return kMaxCtas;  // (no device: the call's own launch tells)
  }
  if (dev <= 63 && (known[0].load() >> dev & 1)) return known[1].load() >> dev & 1 ? kMaxCtas : kMaxCtas / 2;
  bool wide = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most_bytes) == cudaSuccess &&
              cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess;
  if (wide) {
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kMaxCtas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kMaxCtas);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = most_bytes;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    wide = cudaOccupancyMaxActiveClusters(&n, kern, &cfg) == cudaSuccess && n > 0;
  }
  if (!wide) (void)cudaGetLastError();
  if (dev <= 63) {
    if (wide) known[1].fetch_or(1ull << dev);
    known[0].fetch_or(1ull << dev);
  }
  return wide ? kMaxCtas : kMaxCtas / 2;
}
template <typename T, int D>
int prepare_few() {
  static std::atomic<uint64_t> known[2];
  if constexpr (sizeof(T) == 2)
    return prepare(attn_stream_kernel<D>, kStreamBytes<D>, known);
  else
    return prepare(attn_few_kernel<D>, few_bytes<D>(kMaxKeys), known);
}

// One cluster of p.splits CTAs per 16 rows, KV head and sequence.
template <typename... P, typename... A>
int launch_clusters(void (*kern)(P...), const SvAttnShape &s, const SvAttnPlan &p, int bytes, cudaStream_t stream,
                    A... args) {
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = p.splits;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  const int R = s.n_nodes * (s.hq / s.hkv);
  cfg.gridDim = dim3(p.splits, (R + kRows - 1) / kRows, s.batch * s.hkv);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = bytes;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...) == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

template <typename T, int D>
int launch_few(const SvAttnShape &s, const SvAttnPlan &p, const void *q, const void *kc, const void *vc,
               const void *kt, const void *vt, const int32_t *prefix_len, const uint64_t *anc, void *out, float scale,
               int32_t *status, cudaStream_t stream) {
  const sv::KvPages pg{s.block_table, s.block_size, s.max_blocks, s.num_blocks};
  const sv::Window win{s.depth, s.window, s.sinks};
  const float scale_log2 = scale * 1.4426950408889634f;
  const auto run = [&](auto kern, int bytes, auto... cap) {
    return launch_clusters(kern, s, p, bytes, stream, (const T *)q, (const T *)kc, (const T *)vc, (const T *)kt,
                           (const T *)vt, prefix_len, anc, (T *)out, s.n_nodes, s.hq, s.hkv, s.s_max, s.max_prefix,
                           cap..., scale_log2, status, pg, win);
  };
  if constexpr (sizeof(T) == 2)
    return run(attn_stream_kernel<D>, kStreamBytes<D>);
  else
    return run(attn_few_kernel<D>, few_bytes<D>(p.chunk), p.chunk);
}

}  // namespace

// CTAs a cluster: enough for 32 keys each (bf16: 64), but no more than run at
// once (two a SM, in float32 while a CTA's share is below some 150 keys of 128
// dims; clusters of 16 fit a GPC each, so that 256 CTAs in sixteens
// took 16 us where eights took 10).  Taken for every shape that the SM-pair
// kernel does not take, as far as a f32 CTA's keys fit, and else by an
// estimate of both kernels, ns: a wave of clusters costs its start and 21 a
// key of a CTA; the SM-pair kernel about eight tiles' time beside its tiles
// (830 each), shared out in parts of eight or more where its row groups are
// few.  Measured this / the SM-pair kernel, bf16, 32/8 heads of
// 128, us: one node, batch 1, window 256: 6.0 / 10.5, 1024: 6.9 / 15.3, 4000:
// 9.9 / 14.5; batch 8: 6.9 / 12.4, 11 / 18, 27 / 39; batch 64: 21 / 60, 53 /
// 87, 166 / 216; 8 nodes, batch 1: 7.3 / 10.8, 9.9 / 15.6, 15.1 / 15.0; batch
// 8: 10.3 / 12.3, 16.8 / 17.7 (the estimate errs); 16 nodes, batch 8: 13.9 /
// 12.4, 26 / 18; 60 nodes, batch 1: 10.1 / 11.2, 17.1 / 15.9, 41 / 21.  Other
// heads of 128, window 1024: 64/8, one node, batch 1: 7.7 / 16.6, batch 64: 57
// / 90; 32 nodes, batch 1: 18.3 / 16.9; 16/16, 60 nodes, batch 1: 13.1 / 16.6,
// batch 8: 56 / 30; 28/4, 8 nodes, batch 8: 17.9 / 17.1.  At head_dim 64 a key
// has half the bytes and the other side's tile costs the same: 32/8, one node,
// batch 64: 38 / 88, window 4000: 110 / 216.  The estimate is of 128 dims and
// gives up too early there: 32/8, 8 nodes, batch 8: 13.3 / 18.1 (it takes the
// SM pairs), batch 64: 74 / 88; 60 nodes, batch 1: 13.1 / 16.7.  f32
// against the CUDA-core tiles: 5 nodes, 4 heads of 64, window 333: 5.4 / 12.6,
// 4000: 9.5 / 28; 32/8 heads of 128, window 1024: one node 7.7 / 21.4, 60
// nodes 72 / 92, batch 64 162 / 362.
int sv_attn_few_ctas(const SvAttnShape &s) {
  if (s.dtype == SPEC_BF16) return s.head_dim == 128 ? prepare_few<__nv_bfloat16, 128>() : prepare_few<__nv_bfloat16, 64>();
  return s.head_dim == 128 ? prepare_few<float, 128>() : prepare_few<float, 64>();
}

bool sv_attn_few_plan(const SvAttnShape &s, bool pairs, int most_ctas, SvAttnPlan *p) {
  const bool stream = s.dtype == SPEC_BF16;
  const long long seen = (long long)s.window - 1 + s.sinks;
  const long long keys = (seen < s.max_prefix ? seen : s.max_prefix) + s.n_nodes;  // at most
  const int R = s.n_nodes * (s.hq / s.hkv);
  const long long clusters = (long long)s.batch * s.hkv * ((R + kRows - 1) / kRows);
  const auto at_once = [](int c) { return c == kMaxCtas ? kSms : 2 * kSms; };
  int c = 1;
  while (c < most_ctas && (long long)c * (stream ? 64 : 32) < keys) c *= 2;
  while (c > 1 && clusters * c > at_once(c) && (stream || keys <= (long long)c / 2 * kMaxKeys)) c /= 2;
  const long long each = (keys + c - 1) / c;
  if (!stream && each > kMaxKeys) return false;
  *p = SvAttnPlan{};
  p->few = true;
  p->splits = c;
  p->chunk = stream ? 0 : (int)(each + 7) / 8 * 8;
  if (!pairs) return true;
  const long long waves = (clusters * c + at_once(c) - 1) / at_once(c);
  const long long few = waves * (5500 + 21 * each);
  const long long groups = (long long)s.batch * s.hkv * ((R + 255) / 256), tiles = (keys + 127) / 128 + 1;
  const long long pair = groups >= kSms / 2   ? 1500 + (6500 + 830 * tiles) * groups / (kSms / 2)
                         : groups > kSms / 4 ? 8000 + 830 * tiles
                                             : 8000 + 830 * (tiles < 8 ? tiles : 8);
  return few <= pair;
}

int sv_attn_few(const SvAttnShape &s, const SvAttnPlan &p, const void *q, const void *kc, const void *vc,
                const void *kt, const void *vt, const int32_t *prefix_len, const uint64_t *anc, void *out, float scale,
                int32_t *status, cudaStream_t stream) {
  auto run = [&](auto launch) { return launch(s, p, q, kc, vc, kt, vt, prefix_len, anc, out, scale, status, stream); };
  if (s.dtype == SPEC_BF16)
    return s.head_dim == 128 ? run(launch_few<__nv_bfloat16, 128>) : run(launch_few<__nv_bfloat16, 64>);
  return s.head_dim == 128 ? run(launch_few<float, 128>) : run(launch_few<float, 64>);
}

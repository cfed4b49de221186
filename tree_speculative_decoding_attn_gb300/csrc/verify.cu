// Verification of drafted tokens from given probabilities and given uniform
// numbers (spec_verify_probs).
//
// "Drafters: ...", section "Why the answer does not change": keep a draft
// with min(1, p/q), otherwise sample the target with the drafter's
// probabilities subtracted; over a tree, the siblings of a node in turn.
//
// Mathematics.  At node v the residual after j rejected siblings is
//   deterministic siblings:  r_j = p without the rejected tokens, mass W_j = 1 - sum of theirs
//   siblings drawn from q:   r_j = max(0, p - c_j q), mass D_j = sum of it,
//                            c_0 = 0, D_0 = 1, c_{j+1} = c_j + D_j
// (the closed form of r <- norm(max(0, r - q))), and sibling c is kept iff
// u_c * mass * q(t_c) < r_j(t_c) (q = 1 for deterministic siblings).  So a
// test needs one probability of p and one of q; a whole row is read only for
// D_j (a rejected sibling with another behind it) and for the bonus: the
// lowest token x with sum_{y <= x} r(y) > u * sum r.
//
// Exactness.  The answer is a set of integers, so no sum may depend on its
// order.  Probabilities are turned into 64-bit fixed point in units of 2^-60
// (exact from 2^-37 up, cut below), and every sum is an integer sum: the
// same for any split over lanes, warps and CTAs, and within V * 2^-60 of the
// real one, where float32 sums would move the border of every token by up to
// 2^-24.  The tests of single drafts use float64 (one thread, a few products).
//
// What bounds it: nothing but latency at batch 1 (two dependent gathers, the
// walk in shared memory, one row, one cluster exchange), the rows' bytes at
// large batch.  One cluster per sequence; each warp owns one contiguous piece
// of the row, so the bonus is found from the per-warp sums by rereading one
// warp's piece (at most a few KB, in L2).
#include <cooperative_groups.h>

#include "common.cuh"
#include "kernels.h"
#include "tc_ptx.cuh"

namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 16;
constexpr int kInFlight = 4;  // 16-byte loads of one lane in flight (twice that with a drafter's row)
typedef unsigned long long u64;
constexpr u64 kOne = 1ull << 60;

// x in [0, 1] in units of 2^-60, cut; anything else (NaN too) sets *bad and
// counts as 0.
__device__ __forceinline__ u64 fixed60(float x, bool *bad) {
  if (!(x >= 0.f && x <= 1.f)) {
    *bad = true;
    return 0;
  }
  const uint32_t b = __float_as_uint(x) & 0x7FFFFFFFu;
  const u64 m = (b & 0x7FFFFFu) | 0x800000u;
  const int sh = (int)(b >> 23) - 90;  // x = m * 2^(e - 150)
  return sh >= 0 ? m << sh : sh > -24 ? m >> -sh : 0;
}
// A uniform number as the rule takes it: in [0, 1).
__device__ __forceinline__ float uniform(float u) { return u >= 0.f ? fminf(u, 0.99999994f) : 0.f; }
// floor(u * s) for u in [0, 1), exactly.
__device__ __forceinline__ u64 part_of(float u, u64 s) {
  const uint32_t b = __float_as_uint(u);
  const int e = (int)(b >> 23);
  if (e == 0) return 0;  // below 2^-126: u * s < 1
  const u64 m = (b & 0x7FFFFFu) | 0x800000u;
  const u64 lo = m * s, hi = __umul64hi(m, s);
  const int sh = 150 - e;  // >= 24
  if (sh < 64) return (lo >> sh) | (hi << (64 - sh));
  return sh < 128 ? hi >> (sh - 64) : 0;
}
__device__ __forceinline__ u64 warp_sum_u64(u64 v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ u64 warp_incl_u64(u64 v) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  return v;
}

struct Shared {
  int fc[SPEC_MAX_NODES], ns[SPEC_MAX_NODES], tok[SPEC_MAX_NODES], par[SPEC_MAX_NODES];
  float u[SPEC_MAX_NODES], p[SPEC_MAX_NODES], q[SPEC_MAX_NODES];
  int removed[SPEC_MAX_NODES];  // deterministic siblings: distinct rejected tokens of the current node
  int path[SPEC_MAX_NODES + 1];
  u64 wsum[kWarps];
  u64 part[2];                  // this CTA's sum, double-buffered by exchange
  u64 all[kMaxCluster];
  // the walk's next pass over a row: node, c = ci + cf * 2^-60, whether it is the bonus
  int node, n_removed, last, len;
  uint32_t ci;
  u64 cf;
};

// A row of probabilities, cut into 16-byte vectors aligned in memory: vector
// k holds the elements k * VEC - mis ..; the part of the first and the last
// one outside the row reads as zero (and is not touched).
template <typename T>
struct Row {
  static constexpr int VEC = 16 / (int)sizeof(T);
  const T *row;
  int V, mis;
  __device__ Row(const T *base, int64_t off, int V_) : row(base + off), V(V_) {
    mis = (int)((reinterpret_cast<uintptr_t>(row) & 15) / sizeof(T));
  }
  __device__ int vectors() const { return (V + mis + VEC - 1) / VEC; }
  __device__ uint4 load(int k) const {
    const int e0 = k * VEC - mis;
    if (e0 >= 0 && e0 + VEC <= V) return *reinterpret_cast<const uint4 *>(row + e0);
    uint32_t w[4] = {0, 0, 0, 0};
    for (int i = 0; i < VEC; ++i)
      if (e0 + i >= 0 && e0 + i < V) {
        if constexpr (sizeof(T) == 4)
          w[i] = __float_as_uint(row[e0 + i]);
        else
          w[i >> 1] |= (uint32_t)__bfloat16_as_ushort(row[e0 + i]) << (16 * (i & 1));
      }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  __device__ static float at(const uint4 &v, int i) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if constexpr (sizeof(T) == 4) return __uint_as_float(w[i]);
    return __uint_as_float((i & 1) ? w[i >> 1] & 0xFFFF0000u : w[i >> 1] << 16);
  }
};

// max(0, p - c q), c = ci + cf * 2^-60.
template <bool DRAFT>
__device__ __forceinline__ u64 weight(float p, float q, uint32_t ci, u64 cf, bool *bad) {
  const u64 fp = fixed60(p, bad);
  if constexpr (DRAFT) {
    if (ci | cf) {
      const u64 fq = fixed60(q, bad);
      const u64 cq = fq * ci + (cf ? __umul64hi(cf << 4, fq) : 0);
      return fp > cq ? fp - cq : 0;
    }
  }
  return fp;
}

template <typename T, bool DRAFT>
__global__ void __launch_bounds__(kThreads)
    verify_kernel(const T *__restrict__ p_all, const T *__restrict__ q_all, int N, int V,
                  const int32_t *__restrict__ tok, const int32_t *__restrict__ parents,
                  const int32_t *__restrict__ first_child, const int32_t *__restrict__ next_sibling,
                  const float *__restrict__ u_accept, const float *__restrict__ u_bonus, int path_cap,
                  int32_t *acc_len, int32_t *acc_path, int32_t *bonus, int32_t *status) {
  constexpr int VEC = 16 / (int)sizeof(T);
  __shared__ Shared sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int nc = gridDim.x, rank = blockIdx.x, b = blockIdx.y;  // the cluster spans x
  cg::cluster_group cluster = cg::this_cluster();
  bool bad = false;

  // every node's test needs one value of its parent's row (every CTA of the
  // cluster walks the tree itself, from the same values)
  if (tid < N) {
    const int64_t i = (int64_t)b * N + tid;
    const int par = parents[i], t = tok[i];
    sh.fc[tid] = first_child[i];
    sh.ns[tid] = next_sibling[i];
    sh.u[tid] = uniform(u_accept[i]);
    sh.par[tid] = par;
    sh.tok[tid] = t;
    if (par >= 0 && par < N && t >= 0 && t < V) {
      const int64_t at = ((int64_t)b * N + par) * V + t;
      const float pv = sv::to_f32(p_all[at]);
      const float qv = DRAFT ? sv::to_f32(q_all[at]) : 1.f;
      bad = !(pv >= 0.f && pv <= 1.f) || !(qv >= 0.f && qv <= 1.f);
      sh.p[tid] = pv >= 0.f && pv <= 1.f ? pv : 0.f;
      sh.q[tid] = qv >= 0.f && qv <= 1.f ? qv : 0.f;
    }
  }
  __syncthreads();

  // thread 0's walk, kept across the passes it asks for
  int v = 0, child = sh.fc[0], len = 0, steps = 0, n_removed = 0;
  uint32_t ci = 0;
  u64 cf = 0, D = kOne;       // drafter: c, and the residual's mass
  double W = 1.0;             // deterministic: what the removals have left
  if (tid == 0) sh.path[0] = 0;

  auto row_sum = [&](int node, uint32_t rci, u64 rcf, int removals) {
    // this warp's piece of the row: its sum
    const int64_t off = ((int64_t)b * N + node) * V;
    const Row<T> rp(p_all, off, V), rq(DRAFT ? q_all : p_all, off, V);
    const bool with_q = DRAFT && (rci | rcf);
    const int nvec = rp.vectors(), pieces = nc * kWarps;
    const int seg = ((nvec + pieces - 1) / pieces + 31) / 32 * 32;
    const int w = rank * kWarps + warp;
    const int k1 = min(nvec, (w + 1) * seg);
    u64 s = 0;
    for (int k0 = w * seg; k0 < k1; k0 += 32 * kInFlight) {
      uint4 a[kInFlight], c[kInFlight];
#pragma unroll
      for (int j = 0; j < kInFlight; ++j) {
        const int k = k0 + 32 * j + lane;
        a[j] = k < k1 ? rp.load(k) : make_uint4(0, 0, 0, 0);
        if (DRAFT) c[j] = with_q && k < k1 ? rq.load(k) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int j = 0; j < kInFlight; ++j)
#pragma unroll
        for (int i = 0; i < VEC; ++i)
          s += weight<DRAFT>(Row<T>::at(a[j], i), DRAFT ? Row<T>::at(c[j], i) : 0.f, rci, rcf, &bad);
    }
    if (!DRAFT) {
      for (int r = lane; r < removals; r += 32) {
        const int t = sh.removed[r], k = (t + rp.mis) / VEC;
        bool ignore;
        if (k >= w * seg && k < k1) s -= fixed60(sv::to_f32(rp.row[t]), &ignore);
      }
    }
    s = warp_sum_u64(s);
    if (lane == 0) sh.wsum[warp] = s;
  };
  // the cluster's sum of the CTAs' wsum; sh.all holds the CTAs' own
  int parity = 0;
  auto cluster_total = [&]() -> u64 {
    __syncthreads();
    if (warp == 0) {
      const u64 s = warp_sum_u64(lane < kWarps ? sh.wsum[lane] : 0);
      if (lane == 0) sh.part[parity] = s;
    }
    cluster.sync();
    if (tid < nc) sh.all[tid] = *cluster.map_shared_rank(&sh.part[parity], tid);
    parity ^= 1;
    __syncthreads();
    u64 s = 0;
    for (int i = 0; i < nc; ++i) s += sh.all[i];
    return s;
  };

  u64 total;
  for (;;) {
    if (tid == 0) {
      // walk until a row has to be read
      bool want = false;
      while (!want && child >= 0) {
        if (child >= N || sh.par[child] != v || ++steps > N) {
          if (rank == 0) sv::report(status, SPEC_DEV_BAD_PARENTS);
          break;  // broken links: the node is taken as having no further child
        }
        const int t = sh.tok[child];
        bool keep = false, counted = false;
        if (t < 0 || t >= V) {
          if (rank == 0) sv::report(status, SPEC_DEV_BAD_TOKEN);
        } else if (DRAFT) {
          const double c = (double)ci + (double)cf * 0x1p-60;
          const double q = (double)sh.q[child], w = fmax(0.0, (double)sh.p[child] - c * q);
          keep = D > 0 && (double)sh.u[child] * q * ((double)D * 0x1p-60) < w;
          counted = true;
        } else {
          bool again = false;
          for (int r = 0; r < n_removed; ++r) again = again || sh.removed[r] == t;
          const double w = again ? 0.0 : (double)sh.p[child];
          keep = (double)sh.u[child] * W < w;
          if (!keep && !again) {
            sh.removed[n_removed++] = t;
            W = fmax(0.0, W - w);
          }
        }
        if (keep) {
          if (len + 1 >= path_cap) {
            if (rank == 0) sv::report(status, SPEC_DEV_CAPACITY);
            break;
          }
          v = child;
          sh.path[++len] = v;
          child = sh.fc[v];
          ci = 0;
          cf = 0;
          D = kOne;
          W = 1.0;
          n_removed = 0;
          continue;
        }
        child = sh.ns[child];
        if (counted) {
          cf += D;  // c += D (below 2 in a row that sums to 1)
          ci += (uint32_t)(cf >> 60);
          cf &= kOne - 1;
          want = child >= 0;  // its test needs the mass of the new residual
        }
      }
      sh.node = v;
      sh.ci = ci;
      sh.cf = cf;
      sh.n_removed = n_removed;
      sh.last = !want;
      sh.len = len;
    }
    __syncthreads();
    row_sum(sh.node, sh.ci, sh.cf, sh.n_removed);
    total = cluster_total();
    if (sh.last) break;
    D = total;  // (thread 0's)
    __syncthreads();
  }
  // an empty residual (p = q but for roundings, or every token removed): the target's own row
  uint32_t bci = sh.ci;
  u64 bcf = sh.cf;
  int removals = sh.n_removed;
  const int node = sh.node;
  if (total == 0 && ((bci | bcf) || removals)) {
    bci = 0;
    bcf = 0;
    removals = 0;
    __syncthreads();
    row_sum(node, 0, 0, 0);
    total = cluster_total();
  }

  // the bonus: the CTA, then the warp, then the element whose sum passes u * total
  const u64 thr = part_of(uniform(u_bonus[b]), total);
  u64 before = 0;
  for (int i = 0; i < rank; ++i) before += sh.all[i];
  if (total > 0 && before <= thr && thr < before + sh.all[rank]) {
    for (int i = 0; i < warp; ++i) before += sh.wsum[i];
    if (before <= thr && thr < before + sh.wsum[warp]) {
      const int64_t off = ((int64_t)b * N + node) * V;
      const Row<T> rp(p_all, off, V), rq(DRAFT ? q_all : p_all, off, V);
      const int nvec = rp.vectors(), pieces = nc * kWarps;
      const int seg = ((nvec + pieces - 1) / pieces + 31) / 32 * 32;
      const int w = rank * kWarps + warp;
      const int k1 = min(nvec, (w + 1) * seg);
      for (int k0 = w * seg; k0 < k1; k0 += 32) {
        const int k = k0 + lane;
        const uint4 a = k < k1 ? rp.load(k) : make_uint4(0, 0, 0, 0);
        const uint4 c = DRAFT && (bci | bcf) && k < k1 ? rq.load(k) : make_uint4(0, 0, 0, 0);
        u64 x[VEC], s = 0;
#pragma unroll
        for (int i = 0; i < VEC; ++i) {
          x[i] = weight<DRAFT>(Row<T>::at(a, i), Row<T>::at(c, i), bci, bcf, &bad);
          if (!DRAFT)
            for (int r = 0; r < removals; ++r)
              if (sh.removed[r] == k * VEC - rp.mis + i) x[i] = 0;
          s += x[i];
        }
        const u64 incl = warp_incl_u64(s);
        if (__any_sync(0xffffffffu, before + incl > thr)) {
          u64 run = before + incl - s;
          if (run <= thr && thr < before + incl) {
            int hit = -1;
#pragma unroll
            for (int i = 0; i < VEC; ++i) {
              run += x[i];
              if (hit < 0 && run > thr) hit = k * VEC - rp.mis + i;
            }
            bonus[b] = hit;
          }
          break;
        }
        before += __shfl_sync(0xffffffffu, incl, 31);
      }
    }
  }
  if (rank == 0) {
    if (tid == 0) {
      acc_len[b] = sh.len;
      if (total == 0) {  // a row without any probability
        bonus[b] = 0;
        bad = true;
      }
    }
    for (int i = tid; i < path_cap; i += kThreads) acc_path[(int64_t)b * path_cap + i] = i <= sh.len ? sh.path[i] : -1;
  }
  if (bad) sv::report(status, SPEC_DEV_BAD_PROB);
  cluster.sync();  // the partners' reads of this CTA's sums are done
}

// CTAs per sequence: as many as give every warp a full load round of its
// piece, up to 16 (a size the device may refuse: then 8), and no more than
// keep the whole batch resident at once.
template <typename T, bool DRAFT>
int launch_verify(const void *p, const void *q, int batch, int N, int V, const int32_t *tok, const int32_t *parents,
                  const int32_t *first_child, const int32_t *next_sibling, const float *u_accept, const float *u_bonus,
                  int path_cap, int32_t *acc_len, int32_t *acc_path, int32_t *bonus, int32_t *status,
                  cudaStream_t stream) {
  constexpr int VEC = 16 / (int)sizeof(T);
  auto kern = verify_kernel<T, DRAFT>;
  int nc = 8;
  while (nc > 1 && (batch * nc > 304 || (nc / 2) * kThreads * VEC >= V)) nc /= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(nc, batch);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = nc;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, (const T *)p, (const T *)q, N, V, tok, parents, first_child, next_sibling,
                            u_accept, u_bonus, path_cap, acc_len, acc_path, bonus, status) == cudaSuccess
             ? SPEC_OK
             : SPEC_ERR_CUDA;
}

}  // namespace

int sv_verify_probs(const void *p, const void *q, int dtype, int batch, int n_nodes, int vocab, const int32_t *tok,
                    const int32_t *parents, const int32_t *first_child, const int32_t *next_sibling,
                    const float *u_accept, const float *u_bonus, int path_cap, int32_t *acc_len, int32_t *acc_path,
                    int32_t *bonus, int32_t *status, cudaStream_t stream) {
  auto run = [&](auto launch) {
    return launch(p, q, batch, n_nodes, vocab, tok, parents, first_child, next_sibling, u_accept, u_bonus, path_cap,
                  acc_len, acc_path, bonus, status, stream);
  };
  if (dtype == SPEC_BF16)
    return q ? run(launch_verify<__nv_bfloat16, true>) : run(launch_verify<__nv_bfloat16, false>);
  return q ? run(launch_verify<float, true>) : run(launch_verify<float, false>);
}

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
// order.  Probabilities are turned into 64-bit fixed point in units of 2^-58
// (exact from 2^-35 up, cut below), and every sum is an integer sum: the
// same for any split over lanes, warps and CTAs, and within V * 2^-58 of the
// real one, where float32 sums would move the border of every token by up to
// 2^-24.  The tests of single drafts use float64 (one thread, a few products).
//
// What bounds it: latency.  One sequence of a six-node chain over 32000 tokens
// takes 6.3 us (two dependent gathers 1.3, the walk in shared memory 0.6, its
// row 1.2, the exchange 0.6, the bonus 1.1, the launch the rest); 64 trees of
// 32 nodes over 128256 bf16 tokens 14.7 us (16.8 MB, 1.1 TB/s: the two dependent
// gathers then miss the TLB, 2.6, and the rows' integer sums, ten 32-bit
// operations a value, take 3 to 6 where a SM holds two CTAs); eight trees of
// 60 nodes whose siblings a drafter drew 19 to 21 with the numbers drawn (a
// rejected sibling costs 3.7 us: its row pair 2.2, the exchange 0.7, the next
// test 0.8; keeping the rows in shared memory from pass to pass gains
// nothing), in bf16 28 (eight products a vector, 132 bytes of them spilled at
// 64 registers).  Kept: all the tests that need no row at once, one thread a
// child (serial float64 tests cost 0.9 each); the whole CTA on the piece that
// holds the bonus (its own warp alone took up to 20).  One cluster per
// sequence; each warp owns one contiguous piece of the row, so the bonus is
// found from the per-warp sums by rereading one warp's piece (a few KB, in
// L2), a vector a thread.
#include <type_traits>

#include "common.cuh"
#include "kernels.h"
#include "tc_ptx.cuh"

namespace {

using namespace sv::ptx;

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 16;
constexpr int kInFlight = 4;  // 16-byte loads of one lane in flight (twice that with a drafter's row)
typedef unsigned long long u64;
constexpr int kBits = 58;
constexpr u64 kOne = 1ull << kBits;
// Sums stop below a mass of 4: a row that gets there is no distribution (its
// bonus is token 0, reported), and no sum of a million ones wraps: between
// two stops lie the 32 values of a load round, or 16 stopped sums.
constexpr u64 kMost = 4 * kOne - 1;

// Cluster barrier in two halves.  It tells that the CTAs run and have their
// barriers set up (fenced), later that they are done; the sums are ordered by
// their mbarriers, so the arrival need not wait for memory (0.2 us each).
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// Writes v to another CTA's shared memory and counts its 8 bytes on a barrier there.
__device__ __forceinline__ void send_u64(uint32_t dst, u64 v, uint32_t bar) {
  asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.u64 [%0], %1, [%2];" ::"r"(dst), "l"(v), "r"(bar)
               : "memory");
}
// Waits (bounded) for the 8-byte sums of the other CTAs that a barrier counts:
// they are read right after, so the wait acquires at the cluster's scope.
__device__ __forceinline__ bool sums_wait(uint64_t *bar, uint32_t parity) {
  constexpr uint32_t kWaitLimit = 1u << 22;
  for (uint32_t i = 0; i < kWaitLimit; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    if (ok) return true;
  }
  return false;
}

// The bits of a float in [0, 1] as a number of units of 2^-58, cut: the 24
// bits of the significand at the top of 64, shifted right by what the
// exponent leaves (m 2^(e - 150) = (m 2^40 >> (132 - e)) 2^-58; PTX gives 0
// for shifts past 63).
__device__ __forceinline__ u64 fixed(uint32_t b) {
  const u64 m = (u64)(((b & 0x7FFFFFu) | 0x800000u) << 8) << 32;
  u64 r;
  asm("shr.u64 %0, %1, %2;" : "=l"(r) : "l"(m), "r"(132u - (b >> 23)));
  return r;
}
constexpr uint32_t kOneBits = 0x3F800000u;  // 1.f: bits of the floats in [0, 1] are at most these
// Anything but a float in [0, 1] (NaN too) sets *bad and counts as 0.
__device__ __forceinline__ uint32_t checked(uint32_t b, bool *bad) {
  if (b <= kOneBits) return b;
  if (b != 0x80000000u) *bad = true;  // (-0 is 0)
  return 0;
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
  for (int o = 16; o > 1; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  v = min(v, kMost);
  return min(v + __shfl_xor_sync(0xffffffffu, v, 1), kMost);
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
  uint8_t keep[SPEC_MAX_NODES];    // kept if the walk gets to it (drafter's siblings: to it first)
  uint8_t again[SPEC_MAX_NODES];   // its token is an earlier sibling's
  int removed[SPEC_MAX_NODES];     // the distinct rejected tokens of the last node
  int path[SPEC_MAX_NODES + 1];
  u64 wsum[kWarps];
  u64 all[2][kMaxCluster];      // the CTAs' sums, double-buffered by exchange, and
  uint64_t bar[2];              // the barriers that count their arrival
  // the walk's next pass over a row: node, c = ci + cf * 2^-58, whether it is the bonus
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
  // float32 bits of element i; values outside [0, 1] are made 0 and reported
  __device__ static uint32_t at(const uint4 &v, int i) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if constexpr (sizeof(T) == 4) return w[i];
    return (i & 1) ? w[i >> 1] & 0xFFFF0000u : w[i >> 1] << 16;
  }
  __device__ static void unpack(const uint4 &v, uint32_t (&x)[VEC], bool *bad) {
    uint32_t most = 0;
#pragma unroll
    for (int i = 0; i < VEC; ++i) most = max(most, x[i] = at(v, i));
    if (most > kOneBits) {
#pragma unroll
      for (int i = 0; i < VEC; ++i) x[i] = checked(x[i], bad);
    }
  }
};

// floor(c q) in units of 2^-58 for the bits b of a q in [0, 1] and c2 = c 2^59
// < 2^63: (c2 * (24-bit significand * 2^8) >> 32) >> (127 - e), half the
// instructions of a product of two 64-bit numbers.
__device__ __forceinline__ u64 scaled(uint32_t b, u64 c2) {
  const uint32_t m = ((b & 0x7FFFFFu) | 0x800000u) << 8;
  const u64 t = (u64)(uint32_t)(c2 >> 32) * m + ((u64)(uint32_t)c2 * m >> 32);
  u64 r;
  asm("shr.u64 %0, %1, %2;" : "=l"(r) : "l"(t), "r"(127u - (b >> 23)));
  return r;
}

// max(0, p - c q) of a vector's elements, c = ci + cf * 2^-58.  MODE: 0
// c = 0, 1 c = 1, 2 c < 16, 3 any c (c q past 4 is past any p).
template <int MODE, int VEC>
__device__ __forceinline__ void weights(const uint32_t (&p)[VEC], const uint32_t (&q)[VEC], uint32_t ci, u64 cf,
                                        u64 (&x)[VEC]) {
#pragma unroll
  for (int i = 0; i < VEC; ++i) {
    x[i] = fixed(p[i]);
    if (MODE == 0) continue;
    u64 fq = MODE == 2 ? scaled(q[i], ((u64)ci << kBits | cf) << 1) : fixed(q[i]);
    if (MODE == 3) {
      fq = min(fq, kMost / ci);
      fq = fq * ci + __umul64hi(cf << (64 - kBits), fq);
    }
    x[i] = x[i] > fq ? x[i] - fq : 0;
  }
}

template <typename T, bool DRAFT>
__global__ void __launch_bounds__(kThreads, 2)
    verify_kernel(const T *__restrict__ p_all, const T *__restrict__ q_all, int N, int V,
                  const int32_t *__restrict__ tok, const int32_t *__restrict__ parents,
                  const int32_t *__restrict__ first_child, const int32_t *__restrict__ next_sibling,
                  const float *__restrict__ u_accept, const float *__restrict__ u_bonus, int path_cap,
                  int32_t *acc_len, int32_t *acc_path, int32_t *bonus, int32_t *status) {
  constexpr int VEC = 16 / (int)sizeof(T);
  __shared__ Shared sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int nc = gridDim.x, rank = blockIdx.x, b = blockIdx.y;  // the cluster spans x
  bool bad = false, odd = false;  // odd: of this thread's node, whether the walk tests it or not
  if (tid == 0) {
    mbar_init(&sh.bar[0], 1);
    mbar_init(&sh.bar[1], 1);
    mbar_fence_init();
  }
  __syncthreads();
  cluster_arrive();  // (waited for before the first sum is sent)

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
      sh.p[tid] = __uint_as_float(checked(__float_as_uint(sv::to_f32(p_all[at])), &odd));
      sh.q[tid] = DRAFT ? __uint_as_float(checked(__float_as_uint(sv::to_f32(q_all[at])), &odd)) : 1.f;
      // drafter's siblings: the test of a first sibling
      sh.keep[tid] = (double)sh.u[tid] * (double)sh.q[tid] < (double)sh.p[tid];
    }
  }
  __syncthreads();
  if constexpr (!DRAFT) {
    // The walk gets to a child only past its rejected earlier siblings, so
    // what they have left is known without walking: every child is tested at
    // once (a thread each), and the walk below reads the answers.  (Children
    // of a node are numbered in the order of their links; links that are not
    // a tree's are found by the walk.)
    const int par = tid < N ? sh.par[tid] : -1;
    const bool real = par >= 0 && par < N && sh.tok[tid] >= 0 && sh.tok[tid] < V;
    auto siblings = [&](auto f) {  // the ones before this child, in order
      int c = sh.fc[par];
      for (int n = 0; n < N && c >= 0 && c < N && c != tid; ++n) {
        if (sh.par[c] == par && sh.tok[c] >= 0 && sh.tok[c] < V) f(c);
        c = sh.ns[c];
      }
    };
    if (real) {
      bool again = false;
      siblings([&](int c) { again = again || sh.tok[c] == sh.tok[tid]; });
      sh.again[tid] = again;
    }
    __syncthreads();
    if (real) {
      double W = 1.0;
      siblings([&](int c) {
        if (!sh.again[c]) W = fmax(0.0, W - (double)sh.p[c]);
      });
      sh.keep[tid] = !sh.again[tid] && (double)sh.u[tid] * W < (double)sh.p[tid];
    }
    __syncthreads();
  }

  // thread 0's walk, kept across the passes it asks for
  int v = 0, child = sh.fc[0], len = 0, steps = 0, n_removed = 0;
  uint32_t ci = 0;
  u64 cf = 0, D = kOne;       // drafter: c, and the residual's mass
  if (tid == 0) sh.path[0] = 0;

  // vectors of a warp's piece of a row (all rows are cut alike)
  auto piece_of = [&](int nvec) { return ((nvec + nc * kWarps - 1) / (nc * kWarps) + 31) / 32 * 32; };
  // this warp's piece of the row: its sum, in sh.wsum
  auto row_sum = [&](auto mode, int node, uint32_t rci, u64 rcf, int removals) {
    constexpr int MODE = decltype(mode)::value;
    const int64_t off = ((int64_t)b * N + node) * V;
    const Row<T> rp(p_all, off, V), rq(MODE ? q_all : p_all, off, V);
    const int nvec = rp.vectors(), seg = piece_of(nvec);
    const int w = rank * kWarps + warp;
    const int k1 = min(nvec, (w + 1) * seg);
    u64 s = 0;
    for (int k0 = w * seg; k0 < k1; k0 += 32 * kInFlight) {
      uint4 a[kInFlight], c[kInFlight];
#pragma unroll
      for (int j = 0; j < kInFlight; ++j) {
        const int k = k0 + 32 * j + lane;
        a[j] = k < k1 ? rp.load(k) : make_uint4(0, 0, 0, 0);
        if (MODE) c[j] = k < k1 ? rq.load(k) : make_uint4(0, 0, 0, 0);
      }
      u64 xs = 0;
#pragma unroll
      for (int j = 0; j < kInFlight; ++j) {
        uint32_t pb[VEC], qb[VEC] = {};
        Row<T>::unpack(a[j], pb, &bad);
        if (MODE) Row<T>::unpack(c[j], qb, &bad);
        u64 x[VEC];
        weights<MODE>(pb, qb, rci, rcf, x);
#pragma unroll
        for (int i = 0; i < VEC; ++i) xs += x[i];
      }
      s = min(s + xs, kMost);
    }
    s = warp_sum_u64(s);
    if (!DRAFT && removals) {
      u64 gone = 0;
      for (int r = lane; r < removals; r += 32) {
        const int t = sh.removed[r], k = (t + rp.mis) / VEC;
        bool ignore;
        if (k >= w * seg && k < k1) gone += fixed(checked(__float_as_uint(sv::to_f32(rp.row[t])), &ignore));
      }
      gone = warp_sum_u64(gone);
      s = s > gone ? s - gone : 0;
    }
    if (lane == 0) sh.wsum[warp] = s;
  };
  auto with_mode = [&](uint32_t rci, u64 rcf, auto f) {
    if (!DRAFT || !(rci | rcf)) return f(std::integral_constant<int, 0>{});
    if constexpr (DRAFT) {
      if (rci == 1 && rcf == 0) return f(std::integral_constant<int, 1>{});
      if (rci < 16) return f(std::integral_constant<int, 2>{});
      f(std::integral_constant<int, 3>{});
    }
  };
  // The cluster's sum of the CTAs' wsum; all[] holds the CTAs' own.  Each CTA
  // sends its sum to every CTA and waits for theirs: one trip, where a cluster
  // barrier and a read of the others' memory take two (1.1 us).
  int turn = 0;
  const u64 *all = nullptr;
  auto cluster_total = [&]() -> u64 {
    const int buf = turn & 1;
    const uint32_t parity = (turn >> 1) & 1;
    __syncthreads();
    if (turn == 0) cluster_wait();  // every CTA's barriers exist
    ++turn;
    if (warp == 0) {
      const u64 s = warp_sum_u64(lane < kWarps ? sh.wsum[lane] : 0);
      if (lane == 0) mbar_expect_tx(&sh.bar[buf], nc * (uint32_t)sizeof(u64));
      __syncwarp();
      if (lane < nc) send_u64(mapa_cluster(&sh.all[buf][rank], lane), s, mapa_cluster(&sh.bar[buf], lane));
    }
    if (!sums_wait(&sh.bar[buf], parity)) sv::report(status, SPEC_DEV_TIMEOUT);
    __syncwarp();  // (the cluster barriers take whole warps)
    all = sh.all[buf];
    u64 s = 0;
    for (int i = 0; i < nc; ++i) s += all[i];
    return min(s, kMost);
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
          if (!(ci | cf)) {
            keep = sh.keep[child];
          } else {
            const double c = (double)ci + (double)cf * 0x1p-58;
            const double q = (double)sh.q[child], w = fmax(0.0, (double)sh.p[child] - c * q);
            keep = D > 0 && (double)sh.u[child] * q * ((double)D * 0x1p-58) < w;
          }
          counted = true;
        } else {
          keep = sh.keep[child];
          if (!keep && !sh.again[child]) sh.removed[n_removed++] = t;
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
          n_removed = 0;
          continue;
        }
        child = sh.ns[child];
        if (counted) {
          cf += D;  // c += D (below 2 in a row that sums to 1)
          ci += (uint32_t)(cf >> kBits);
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
    with_mode(sh.ci, sh.cf, [&](auto mode) { row_sum(mode, sh.node, sh.ci, sh.cf, sh.n_removed); });
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
    row_sum(std::integral_constant<int, 0>{}, node, 0, 0, 0);
    total = cluster_total();
  }

  if (total == kMost) total = 0;
  cluster_arrive();  // no more is sent; at the kernel's end every CTA has got this far
  // the bonus: the CTA, then the warp whose piece's sum passes u * total; its
  // piece is read again by the whole CTA, a vector a thread
  const u64 thr = part_of(uniform(u_bonus[b]), total);
  u64 before = 0;
  for (int i = 0; i < rank; ++i) before += all[i];
  if (total > 0 && before <= thr && thr < before + all[rank]) {
    int owner = 0;
    while (owner < kWarps - 1 && before + sh.wsum[owner] <= thr) before += sh.wsum[owner++];
    __syncthreads();  // wsum is read; it takes the warps' sums of the piece's rounds from here on
    with_mode(bci, bcf, [&](auto mode) {
      constexpr int MODE = decltype(mode)::value;
      const int64_t off = ((int64_t)b * N + node) * V;
      const Row<T> rp(p_all, off, V), rq(MODE ? q_all : p_all, off, V);
      const int nvec = rp.vectors(), seg = piece_of(nvec);
      const int w = rank * kWarps + owner;
      const int k1 = min(nvec, (w + 1) * seg);
      for (int k0 = w * seg; k0 < k1; k0 += kThreads) {
        const int k = k0 + tid;
        uint32_t pb[VEC], qb[VEC] = {};
        Row<T>::unpack(k < k1 ? rp.load(k) : make_uint4(0, 0, 0, 0), pb, &bad);
        if (MODE) Row<T>::unpack(k < k1 ? rq.load(k) : make_uint4(0, 0, 0, 0), qb, &bad);
        u64 x[VEC], s = 0;
        weights<MODE>(pb, qb, bci, bcf, x);
        if (!DRAFT) {
          for (int r = 0; r < removals; ++r) {
            const int at = sh.removed[r] + rp.mis - k * VEC;
#pragma unroll
            for (int i = 0; i < VEC; ++i)
              if (i == at) x[i] = 0;
          }
        }
#pragma unroll
        for (int i = 0; i < VEC; ++i) s += x[i];
        const u64 incl = warp_incl_u64(s);
        if (lane == 31) sh.wsum[warp] = incl;
        __syncthreads();
        u64 run = before + incl - s, round = 0;
        for (int i = 0; i < kWarps; ++i) {
          if (i < warp) run += sh.wsum[i];
          round += sh.wsum[i];
        }
        if (run <= thr && thr < run + s) {
          int hit = -1;
#pragma unroll
          for (int i = 0; i < VEC; ++i) {
            run += x[i];
            if (hit < 0 && run > thr) hit = k * VEC - rp.mis + i;
          }
          bonus[b] = hit;
        }
        before += round;
        if (before > thr) break;
        __syncthreads();
      }
    });
  }
  if (rank == 0) {
    if (tid == 0) {
      acc_len[b] = sh.len;
      if (total == 0) {  // a row without any probability, or with far too much
        bonus[b] = 0;
        bad = true;
      }
    }
    for (int i = tid; i < path_cap; i += kThreads) acc_path[(int64_t)b * path_cap + i] = i <= sh.len ? sh.path[i] : -1;
  }
  if (odd && rank == 0) {  // reported if the walk has tested the node: a child of the path's, not past the kept one
    const int par = sh.par[tid];
    for (int i = 0; i <= sh.len; ++i) {
      if (sh.path[i] != par) continue;
      int c = sh.fc[par];
      for (int n = 0; n < N && c >= 0 && c < N; ++n) {
        bad = bad || c == tid;
        if (i < sh.len && c == sh.path[i + 1]) break;
        c = sh.ns[c];
      }
    }
  }
  if (bad) sv::report(status, SPEC_DEV_BAD_PROB);
  __syncwarp();
  cluster_wait();
}

// CTAs per sequence: up to 16 (a size the device may refuse: then 8), no more
// than give every warp a full load round of its piece, and no more than keep
// the whole batch resident at two CTAs a SM.
template <typename T, bool DRAFT>
int launch_verify(const void *p, const void *q, int batch, int N, int V, const int32_t *tok, const int32_t *parents,
                  const int32_t *first_child, const int32_t *next_sibling, const float *u_accept, const float *u_bonus,
                  int path_cap, int32_t *acc_len, int32_t *acc_path, int32_t *bonus, int32_t *status,
                  cudaStream_t stream) {
  constexpr int VEC = 16 / (int)sizeof(T);
  auto kern = verify_kernel<T, DRAFT>;
  int nc = kMaxCluster;
  while (nc > 1 && (batch * nc > 2 * 152 || (nc / 2) * kThreads * VEC >= V)) nc /= 2;
  if (nc > 8 && cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) {
    (void)cudaGetLastError();
    nc = 8;
  }
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
  auto launch = [&]() {
    return cudaLaunchKernelEx(&cfg, kern, (const T *)p, (const T *)q, N, V, tok, parents, first_child, next_sibling,
                              u_accept, u_bonus, path_cap, acc_len, acc_path, bonus, status);
  };
  cudaError_t e = launch();
  if (e == cudaErrorInvalidClusterSize && nc > 8) {
    (void)cudaGetLastError();
    attr[0].val.clusterDim.x = 8;
    cfg.gridDim = dim3(8, batch);
    e = launch();
  }
  return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
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

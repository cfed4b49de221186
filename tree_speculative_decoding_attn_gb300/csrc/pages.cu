// The pages of a paged K/V cache: forking, reserving (with copy-on-write),
// freeing and compacting.  "5.3 Medusa、EAGLE 与 MTP", section 8, closing
// remarks (block tables of paged KV); what the commit leaves to "the caller's
// allocator".
//
// State, all in device memory and owned by the caller: block tables [batch,
// max_blocks] (negative entry: no block) and one reference count per block
// (the table entries that name it, plus whatever the caller adds).  A block
// of count 0 is free; there is no free list, so the lowest free ids are found
// by a scan and every result is a function of the inputs alone: integer
// atomics count, their order changes nothing.
//
// fork and free move no rows: 4 bytes per table entry and per block, a few
// microseconds of latency.  reserve and compact plan in one cluster (counts,
// scans, a list of moves) and copy in a second launch over the whole GPU, a
// programmatic dependent of the first; that one is bound by HBM: two bytes
// moved per byte copied.
#include <cooperative_groups.h>

#include "common.cuh"
#include "kernels.h"
#include "tc_ptx.cuh"

namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 1024;
constexpr int kMaxBatch = 4096;   // rows of a table (a shared-memory word each)
constexpr int kRange = 1024;      // blocks whose counts one CTA owns
constexpr long long kScanEntries = 8192;  // table entries up to which every CTA scans the whole table

__device__ __forceinline__ int ld_relaxed(const int32_t *p) {
  int v;
  asm volatile("ld.relaxed.gpu.global.s32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
  return v;
}

// Does a page of positions [r0, r0 + block_size) of a sequence of P rows
// stay: does it begin below P + spare and, in a window, hold a sink or a
// position that a node at P sees or that comes after it?
__device__ __forceinline__ bool page_stays(long long r0, int block_size, long long P, int window, int sinks,
                                           int spare) {
  if (r0 >= P + spare) return false;
  return window <= 0 || r0 < sinks || r0 + block_size > P - window + 1;
}

// How many of the new sequences continue each old one.
__device__ __forceinline__ void count_parents(const int32_t *__restrict__ parent, int batch, int batch_out,
                                              int *s_mult, int32_t *status) {
  for (int i = threadIdx.x; i < batch; i += kThreads) s_mult[i] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < batch_out; i += kThreads) {
    const int p = parent[i];
    if (p >= batch) {
      sv::report(status, SPEC_DEV_BAD_PARENTS);
    } else if (p >= 0) {
      atomicAdd(&s_mult[p], 1);
    }
  }
  __syncthreads();
}
// The new tables' entries and lengths, this thread's share of them.
__device__ __forceinline__ void fork_rows(const int32_t *table, const int32_t *prefix_len,
                                          const int32_t *__restrict__ parent, int batch, int batch_out,
                                          int max_blocks, int num_blocks, int32_t *table_out, int32_t *prefix_out,
                                          uint32_t first, uint32_t step) {
  const uint32_t fresh = (uint32_t)batch_out * max_blocks;
#pragma unroll 4
  for (uint32_t e = first; e < fresh; e += step) {
    const uint32_t i = e / max_blocks;
    const int p = parent[i];
    int blk = p >= 0 && p < batch ? table[(uint32_t)p * max_blocks + (e - i * max_blocks)] : -1;
    if (blk < 0 || blk >= num_blocks) blk = -1;
    table_out[e] = blk;
  }
  for (uint32_t i = first; i < (uint32_t)batch_out; i += step) {
    const int p = parent[i];
    prefix_out[i] = p >= 0 && p < batch ? prefix_len[p] : 0;
  }
}

// fork (FORK) and free.  CTA c owns the counts of blocks [c kRange, +kRange):
// it scans the whole table once, collects its blocks' changes in shared
// memory and writes their counts.  free: the owner of an entry's block also
// writes the entry, so the table may be changed in place: another CTA sees
// the block's id, which is not its own, or -1.
template <bool FORK>
__global__ void __launch_bounds__(kThreads)
    pages_refs_kernel(const int32_t *table, const int32_t *prefix_len, const int32_t *__restrict__ parent, int batch,
                      int batch_out, int max_blocks, int block_size, int num_blocks, int window, int sinks, int spare,
                      const int32_t *ref, int32_t *table_out, int32_t *prefix_out, int32_t *ref_out, int32_t *status) {
  __shared__ int s_delta[kRange];
  __shared__ int s_mult[FORK ? kMaxBatch : 1];  // continuations of an old sequence
  const int lo = blockIdx.x * kRange, n = min(kRange, num_blocks - lo);
  for (int i = threadIdx.x; i < n; i += kThreads) s_delta[i] = 0;
  __syncthreads();
  if constexpr (FORK) {
    count_parents(parent, batch, batch_out, s_mult, status);
    fork_rows(table, prefix_len, parent, batch, batch_out, max_blocks, num_blocks, table_out, prefix_out,
              blockIdx.x * kThreads + threadIdx.x, gridDim.x * kThreads);
  }
  const uint32_t total = (uint32_t)batch * max_blocks;
#pragma unroll 4
  for (uint32_t e = threadIdx.x; e < total; e += kThreads) {
    const int blk = FORK ? table[e] : ld_relaxed(table + e);
    const uint32_t b = e / max_blocks;
    const bool mine = blk >= lo && blk < lo + n;
    if (blk >= num_blocks) sv::report(status, SPEC_DEV_BAD_BLOCK);
    if constexpr (FORK) {
      const int d = s_mult[b] - 1;
      if (mine && d) atomicAdd(&s_delta[blk - lo], d);
    } else {
      if (mine) {
        const bool stays =
            page_stays((long long)(e - b * max_blocks) * block_size, block_size, prefix_len[b], window, sinks, spare);
        if (!stays) atomicSub(&s_delta[blk - lo], 1);
        table_out[e] = stays ? blk : -1;
      } else if (blockIdx.x == 0 && (blk < 0 || blk >= num_blocks)) {
        table_out[e] = -1;
      }
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kThreads) ref_out[lo + i] = ref[lo + i] + s_delta[i];
}

// The same for tables of more entries than a CTA scans quickly: every entry
// is looked at once, and its block's count changed by an atomic (in ref_out,
// which holds the old counts by then: counts_copy_kernel, where it is not
// changed in place).
__global__ void __launch_bounds__(kThreads)
    counts_copy_kernel(const int32_t *__restrict__ ref, int32_t *__restrict__ ref_out, int num_blocks) {
  const int i = blockIdx.x * kThreads + threadIdx.x;
  if (i < num_blocks) ref_out[i] = ref[i];
}
template <bool FORK>
__global__ void __launch_bounds__(kThreads)
    pages_refs_spread_kernel(const int32_t *table, const int32_t *prefix_len, const int32_t *__restrict__ parent,
                             int batch, int batch_out, int max_blocks, int block_size, int num_blocks, int window,
                             int sinks, int spare, int32_t *table_out, int32_t *prefix_out, int32_t *ref_out,
                             int32_t *status) {
  __shared__ int s_mult[FORK ? kMaxBatch : 1];
  const uint32_t first = blockIdx.x * kThreads + threadIdx.x, step = gridDim.x * kThreads;
  if constexpr (FORK) {
    count_parents(parent, batch, batch_out, s_mult, status);
    fork_rows(table, prefix_len, parent, batch, batch_out, max_blocks, num_blocks, table_out, prefix_out, first, step);
  }
  const uint32_t total = (uint32_t)batch * max_blocks;
#pragma unroll 4
  for (uint32_t e = first; e < total; e += step) {
    const int blk = table[e];
    const uint32_t b = e / max_blocks;
    const bool good = blk >= 0 && blk < num_blocks;
    if (blk >= num_blocks) sv::report(status, SPEC_DEV_BAD_BLOCK);
    if constexpr (FORK) {
      const int d = s_mult[b] - 1;
      if (good && d) atomicAdd(&ref_out[blk], d);
    } else {
      const bool stays = good && page_stays((long long)(e - b * max_blocks) * block_size, block_size, prefix_len[b],
                                            window, sinks, spare);
      if (good && !stays) atomicSub(&ref_out[blk], 1);
      table_out[e] = stays ? blk : -1;
    }
  }
}

// ---------------------------------------------------------------------------
// reserve and compact
// ---------------------------------------------------------------------------
struct Move {
  int src, dst, rows, pad;
};
// The workspace: header (number of moves), moves, then words per block and
// per table entry.
struct Space {
  int *n_moves;
  Move *moves;
  int *a, *b, *c;  // [num_blocks] each
  int *flag;       // [batch * max_blocks]
};
__host__ __device__ inline size_t space_layout(Space *s, void *base, long long batch, long long max_blocks,
                                               long long num_blocks) {
  uint8_t *p = static_cast<uint8_t *>(base);
  size_t off = 16;
  const size_t moves = off;
  off += (size_t)(num_blocks > batch ? num_blocks : batch) * sizeof(Move);
  const size_t words = off;
  off += (size_t)num_blocks * 3 * 4;
  const size_t flag = off;
  off += (size_t)batch * max_blocks * 4;
  if (s) {
    s->n_moves = reinterpret_cast<int *>(p);
    s->moves = reinterpret_cast<Move *>(p + moves);
    s->a = reinterpret_cast<int *>(p + words);
    s->b = s->a + num_blocks;
    s->c = s->b + num_blocks;
    s->flag = reinterpret_cast<int *>(p + flag);
  }
  return (off + 15) / 16 * 16;
}

// Exclusive prefix sum of v over the CTA's threads and the CTA's total.
template <typename V>
__device__ V cta_scan(V v, V *total) {
  __shared__ V s_warp[kThreads / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  V x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const V y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  if (warp == 0) {
    V w = s_warp[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const V y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    s_warp[lane] = w;
  }
  __syncthreads();
  *total = s_warp[kThreads / 32 - 1];
  return x - v + (warp ? s_warp[warp - 1] : V(0));
}

// The plans run on one cluster: CTA c owns the contiguous blocks [lo, hi) of
// the pool, so a pool of a million blocks is read by eight SMs and a small
// one by a single CTA.
constexpr int kPlanCtas = 8;
constexpr int kPlanBlocks = 8192;  // blocks that a CTA of a plan takes on before the cluster grows
struct Span {
  int lo, hi;
};
__device__ __forceinline__ Span my_span(int num_blocks) {
  const int per = (num_blocks + (int)gridDim.x - 1) / (int)gridDim.x;
  const int lo = min(num_blocks, (int)blockIdx.x * per);
  return Span{lo, min(num_blocks, lo + per)};
}
__device__ __forceinline__ void plan_sync(cg::cluster_group &cluster) {
  if (gridDim.x > 1)
    cluster.sync();
  else
    __syncthreads();
}
// Sums a number of each CTA over the cluster: the CTAs before this one, and all.
__device__ void cluster_sums(cg::cluster_group &cluster, int *s_mine, int mine, int *before, int *all) {
  *before = 0;
  *all = mine;
  if (gridDim.x == 1) return;
  if (threadIdx.x == 0) *s_mine = mine;
  cluster.sync();
  int b = 0, a = 0;
  for (int i = 0; i < (int)gridDim.x; ++i) {
    const int v = *cluster.map_shared_rank(s_mine, i);
    a += v;
    if (i < (int)blockIdx.x) b += v;
  }
  *before = b;
  *all = a;
}
// Sum over the CTA of f(i), i in [lo, hi).
template <typename F>
__device__ int cta_count(int lo, int hi, F f) {
  if (lo >= hi) return 0;
  int v = 0, total;
#pragma unroll 8
  for (int i = lo + (int)threadIdx.x; i < hi; i += kThreads) v += f(i);
  cta_scan(v, &total);
  return total;
}

// The entries a call writes: the pages holding rows P .. P + need - 1 of each
// sequence, numbered in (sequence, page) order.
struct Writes {
  const int *off;  // [batch + 1] in shared memory
  int batch;
  __device__ int seq_of(int i) const {  // the last sequence whose first entry is <= i (and that has any)
    int lo = 0, hi = batch;
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (off[mid] <= i) lo = mid; else hi = mid;
    }
    return lo;
  }
};

constexpr int kKeep = 0, kFresh = 1, kCopy = 2;

__global__ void __launch_bounds__(kThreads)
    reserve_plan_kernel(const int32_t *table, int32_t *table_out, int batch, int max_blocks, int block_size,
                        int num_blocks, const int32_t *__restrict__ prefix_len, const int32_t *__restrict__ need,
                        const int32_t *ref, int32_t *ref_out, const Space ws, int32_t *status) {
  __shared__ int s_off[kMaxBatch + 1];
  __shared__ int s_moves, s_free;
  cg::cluster_group cluster = cg::this_cluster();
  sv::ptx::grid_dep_launch();
  const int tid = threadIdx.x;
  const Span own = my_span(num_blocks);
  if (tid == 0) s_moves = 0;

  // 1. how many entries each sequence writes (a thread takes consecutive
  // ones; every CTA counts them all)
  const int sper = (batch + kThreads - 1) / kThreads;
  const int b0 = min(batch, tid * sper), b1 = min(batch, b0 + sper);
  auto writes_of = [&](int b, bool tell) -> int {
    const int nd = need[b];
    if (nd <= 0) return 0;
    const long long P = prefix_len[b], end = P + nd;
    if (P < 0 || end > (long long)max_blocks * block_size) {
      if (tell) sv::report(status, SPEC_DEV_CAPACITY);
      return 0;
    }
    return (int)((uint32_t)(end - 1) / (uint32_t)block_size - (uint32_t)P / (uint32_t)block_size) + 1;
  };
  // (in the same scan: the free ones among this CTA's first kThreads blocks;
  // on the way over its blocks: the writers' counts at their start, and the
  // counts as they were, where they are not changed in place)
  auto visit = [&](int i) -> int {
    const int r = ref[i];
    ws.a[i] = 0;
    ws.b[i] = -1;
    if (ref_out != ref) ref_out[i] = r;
    return r <= 0;
  };
  const int first = own.lo + tid;
  const int first_free = first < own.hi ? visit(first) : 0;
  unsigned long long v = first_free, sums;
  for (int b = b0; b < b1; ++b) v += (unsigned long long)writes_of(b, true) << 32;
  const unsigned long long sofar = cta_scan(v, &sums);
  const int n = (int)(sums >> 32);
  int at = (int)(sofar >> 32);
  for (int b = b0; b < b1; ++b) {
    s_off[b] = at;
    at += writes_of(b, false);
  }
  if (tid == 0) s_off[batch] = n;
  const int nfree = (int)(uint32_t)sums + cta_count(own.lo + kThreads, own.hi, visit);
  if (table_out != table)
    for (int64_t e = (int64_t)blockIdx.x * kThreads + tid; e < (int64_t)batch * max_blocks;
         e += (int64_t)gridDim.x * kThreads)
      table_out[e] = table[e];
  int base, all_free;
  cluster_sums(cluster, &s_free, nfree, &base, &all_free);
  // the lowest free blocks in order, as many as could be wanted
  const int k0 = base + (int)(uint32_t)sofar;
  if (first_free && k0 < n) ws.c[k0] = first;
  base += (int)(uint32_t)sums;
  for (int i0 = own.lo + kThreads; i0 < own.hi && base < n; i0 += kThreads) {
    const int i = i0 + tid;
    const bool f = i < own.hi && ref[i] <= 0;
    int sum;
    const int k = base + cta_scan((int)f, &sum);
    if (f && k < n) ws.c[k] = i;
    base += sum;
  }
  plan_sync(cluster);  // the CTAs' parts are in place (and their sums read)
  if (blockIdx.x != 0) return;
  const Writes wr{s_off, batch};
  struct Entry {
    int b, j, blk, r;  // sequence, page, its block (-1: none) and that block's count
    int64_t e;
  };
  auto entry = [&](int i) -> Entry {
    Entry x;
    x.b = wr.seq_of(i);
    x.j = prefix_len[x.b] / block_size + (i - s_off[x.b]);
    x.e = (int64_t)x.b * max_blocks + x.j;
    x.blk = table[x.e];
    if (x.blk >= num_blocks) sv::report(status, SPEC_DEV_BAD_BLOCK);
    if (x.blk < 0 || x.blk >= num_blocks) x.blk = -1;
    x.r = x.blk < 0 ? 0 : ref[x.blk];
    return x;
  };
  // 2. the writers of each shared block: how many, and which is the last
  // (a thread's first entry stays in its registers through all steps)
  const Entry mine = tid < n ? entry(tid) : Entry{0, 0, -1, 0, 0};
  for (int i = tid; i < n; i += kThreads) {
    const Entry x = i == tid ? mine : entry(i);
    if (x.r > 1) {
      atomicAdd(&ws.a[x.blk], 1);
      atomicMax(&ws.b[x.blk], i);
    }
  }
  __syncthreads();
  // 3. what becomes of each entry, and its number among those that get a
  // block.  Taken in order, a writer copies a block that others still hold:
  // all of them if some other holder does not write, else all but the last.
  int wanted = 0, my_flag = kKeep, my_rank = 0;
  for (int i0 = 0; i0 < n; i0 += kThreads) {
    const int i = i0 + tid;
    int f = kKeep;
    if (i < n) {
      const Entry x = i0 == 0 ? mine : entry(i);
      if (x.blk < 0)
        f = kFresh;
      else if (x.r > 1 && !(__ldcg(&ws.a[x.blk]) >= x.r && __ldcg(&ws.b[x.blk]) == i))
        f = kCopy;
    }
    int sum;
    const int rank = wanted + cta_scan((int)(f != kKeep), &sum);
    wanted += sum;
    if (i0 == 0) {
      my_flag = f;
      my_rank = rank;
    } else if (i < n) {
      ws.flag[i] = rank << 2 | f;
    }
  }
  const bool fits = wanted <= all_free;
  if (!fits && tid == 0) sv::report(status, SPEC_DEV_CAPACITY);
  // 4. hand the blocks out in entry order
  if (fits) {
    for (int i = tid; i < n; i += kThreads) {
      const int f = i == tid ? my_flag : ws.flag[i] & 3, rank = i == tid ? my_rank : ws.flag[i] >> 2;
      if (f == kKeep) continue;
      const Entry x = i == tid ? mine : entry(i);
      const int blk = __ldcg(&ws.c[rank]);
      table_out[x.e] = blk;
      ref_out[blk] = 1;
      if (f == kCopy) {
        atomicSub(&ref_out[x.blk], 1);
        const int P = prefix_len[x.b], rows = P % block_size;
        if (x.j == P / block_size && rows > 0)  // rows in use before the first new one
          ws.moves[atomicAdd(&s_moves, 1)] = Move{x.blk, blk, rows, 0};
      }
    }
  }
  __syncthreads();
  if (tid == 0) *ws.n_moves = s_moves;
}

__global__ void __launch_bounds__(kThreads)
    compact_plan_kernel(int block_size, int num_blocks, const int32_t *ref, int32_t *ref_out, int32_t *n_used,
                        int32_t *remap, const Space ws) {
  __shared__ int s_sum[2];
  cg::cluster_group cluster = cg::this_cluster();
  sv::ptx::grid_dep_launch();
  const int tid = threadIdx.x;
  const Span own = my_span(num_blocks);
  // U, and the used blocks before this CTA's (the first kThreads of its
  // blocks by a scan that is needed later anyway)
  int before, U, low_before, low, first_sum;
  const int first = own.lo + tid, first_r = first < own.hi ? ref[first] : 0;
  const int first_ub = cta_scan((int)(first_r > 0), &first_sum);
  const int used = first_sum + cta_count(own.lo + kThreads, own.hi, [&](int i) { return (int)(ref[i] > 0); });
  cluster_sums(cluster, &s_sum[0], used, &before, &U);
  // used blocks below U
  if (num_blocks <= kThreads) {
    if (first == U) s_sum[1] = first_ub;
    __syncthreads();
    low = U < num_blocks && U < kThreads ? s_sum[1] : U;
  } else {
    const int mine = cta_count(own.lo, min(own.hi, max(own.lo, U)), [&](int i) { return (int)(ref[i] > 0); });
    cluster_sums(cluster, &s_sum[1], mine, &low_before, &low);
  }
  const int m = U - low;  // holes below U, and as many used blocks from U on
  for (int i0 = own.lo; i0 < own.hi; i0 += kThreads) {
    const int i = i0 + tid;
    const int r = i < own.hi ? ref[i] : 0;
    int sum = first_sum;
    const int ub = before + (i0 == own.lo ? first_ub : cta_scan((int)(r > 0), &sum));  // used blocks before block i
    before += sum;
    if (i < own.hi) {
      if (r <= 0 && i < U) ws.moves[i - ub].dst = i;
      if (r > 0 && i >= U) {
        ws.moves[ub - low].rows = block_size;
        ws.moves[ub - low].src = i;
      }
      ws.a[i] = r > 0 ? i : -1;  // the new id of block i (those that move: below)
      ref_out[i] = max(r, 0);
    }
  }
  plan_sync(cluster);
  for (int k = (int)blockIdx.x * kThreads + tid; k < m; k += (int)gridDim.x * kThreads) {
    const int src = __ldcg(&ws.moves[k].src), dst = __ldcg(&ws.moves[k].dst);
    ws.a[src] = dst;
    ref_out[dst] = __ldcg(&ref[src]);
    ref_out[src] = 0;
  }
  if (tid == 0 && blockIdx.x == 0) {
    *ws.n_moves = m;
    *n_used = U;
  }
  if (remap) {
    plan_sync(cluster);
    for (int i = own.lo + tid; i < own.hi; i += kThreads) remap[i] = __ldcg(&ws.a[i]);
  }
  plan_sync(cluster);  // the partners' reads of this CTA's sums are done
}

// Copies the planned rows of every layer and KV head, K and V, 16 bytes a
// thread and load; REMAP: also renames the table's entries.  A unit is up to
// kPiece vectors of one (move, K or V, layer, head); the CTAs take them in
// turn.  Measured with the plan, eight loads in flight, streaming accesses and
// up to sixteen CTAs a SM in the grid (four of them resident: 64 registers a
// thread) against four loads, plain accesses and eight: a compaction that
// reads and writes 0.73 GB 113 us (6.5 TB/s, 0.96 of a plain copy's rate)
// against 121, a reservation whose copies are 0.11 GB 20.6 against 23.4.
constexpr int kCopyThreads = 256;
constexpr int kInFlight = 8;
constexpr int kPiece = kCopyThreads * kInFlight;
template <bool REMAP>
__global__ void __launch_bounds__(kCopyThreads)
    pages_copy_kernel(uint4 *k_pages, uint4 *v_pages, int n_layers, int hkv, int block_size, int num_blocks,
                      int vec_per_row, const Space ws, const int32_t *table, int32_t *table_out, int64_t n_entries,
                      int32_t *status) {
  sv::ptx::grid_dep_wait();
  const int n_moves = *ws.n_moves;
  const int64_t page_vec = (int64_t)block_size * vec_per_row;
  const int pieces = (int)((page_vec + kPiece - 1) / kPiece);
  const int pools = v_pages ? 2 : 1;  // (a cache of one pool: K alone)
  const int64_t units = (int64_t)n_moves * pools * n_layers * hkv * pieces;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int piece = (int)(u % pieces);
    int64_t x = u / pieces;
    const int h = (int)(x % hkv);
    x /= hkv;
    const int layer = (int)(x % n_layers);
    x /= n_layers;
    const bool is_v = v_pages && (x & 1);
    const Move mv = ws.moves[v_pages ? x >> 1 : x];
    const int64_t n = (int64_t)mv.rows * vec_per_row;
    uint4 *pool = is_v ? v_pages : k_pages;
    const int64_t layer0 = (int64_t)layer * num_blocks;
    const uint4 *src = pool + ((layer0 + mv.src) * hkv + h) * page_vec;
    uint4 *dst = pool + ((layer0 + mv.dst) * hkv + h) * page_vec;
    const int64_t i0 = (int64_t)piece * kPiece + threadIdx.x;
    uint4 r[kInFlight];
#pragma unroll
    for (int j = 0; j < kInFlight; ++j)
      if (i0 + j * kCopyThreads < n) r[j] = __ldcs(src + i0 + j * kCopyThreads);
#pragma unroll
    for (int j = 0; j < kInFlight; ++j)
      if (i0 + j * kCopyThreads < n) __stcs(dst + i0 + j * kCopyThreads, r[j]);
  }
  if constexpr (REMAP) {
    for (int64_t e = (int64_t)blockIdx.x * kCopyThreads + threadIdx.x; e < n_entries;
         e += (int64_t)gridDim.x * kCopyThreads) {
      const int blk = table[e];
      int to = -1;
      if (blk >= 0) {
        to = blk < num_blocks ? ws.a[blk] : -1;
        if (to < 0) sv::report(status, SPEC_DEV_BAD_BLOCK);
      }
      table_out[e] = to;
    }
  }
}

template <bool REMAP>
int launch_copy(void *k, void *v, int n_layers, int hkv, int block_size, int num_blocks, int vec_per_row,
                long long most_moves, const Space &ws, const int32_t *table, int32_t *table_out, int64_t n_entries,
                int32_t *status, cudaStream_t stream) {
  const long long page_vec = (long long)block_size * vec_per_row;
  const long long units = most_moves * 2 * n_layers * hkv * ((page_vec + kPiece - 1) / kPiece);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(units < 1 ? 1 : units > 152 * 16 ? 152 * 16 : units));
  cfg.blockDim = dim3(kCopyThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, pages_copy_kernel<REMAP>, (uint4 *)k, (uint4 *)v, n_layers, hkv, block_size,
                            num_blocks, vec_per_row, ws, table, table_out, n_entries, status) == cudaSuccess
             ? SPEC_OK
             : SPEC_ERR_CUDA;
}

// Launches a plan kernel on a cluster as the pool needs it.
template <typename... P, typename... A>
int launch_plan(void (*kern)(P...), int num_blocks, cudaStream_t stream, A... args) {
  int nc = 1;
  while (nc < kPlanCtas && (long long)nc * kPlanBlocks < num_blocks) nc *= 2;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = nc;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(nc);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, args...) == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

// fork and free.  A CTA that owns its blocks' counts has one launch to do and
// no atomics in memory, but looks at every entry; measured fork / free, us,
// against one look and an atomic per entry (two launches out of place): 64
// entries 3.0 / 1.9 against 3.3 / 2.3, 4096: 3.6 / 3.9 against 5.3 / 5.7,
// 8192: 4.5 / 6.2 against 5.4 / 5.7, 16384: 6.0 / 9.4 against 5.5 / 5.8,
// 262144: 79 / 77 against 6.8 / 6.8.
template <bool FORK>
int launch_refs(const int32_t *table, const int32_t *prefix_len, const int32_t *parent, int batch, int batch_out,
                int max_blocks, int block_size, int num_blocks, int window, int sinks, int spare, const int32_t *ref,
                int32_t *table_out, int32_t *prefix_out, int32_t *ref_out, int32_t *status, cudaStream_t stream) {
  const long long entries = (long long)(batch_out > batch ? batch_out : batch) * max_blocks;
  if (entries <= kScanEntries) {
    pages_refs_kernel<FORK><<<(num_blocks + kRange - 1) / kRange, kThreads, 0, stream>>>(
        table, prefix_len, parent, batch, batch_out, max_blocks, block_size, num_blocks, window, sinks, spare, ref,
        table_out, prefix_out, ref_out, status);
    return sv_launch_status();
  }
  if (ref_out != ref) {
    counts_copy_kernel<<<(num_blocks + kThreads - 1) / kThreads, kThreads, 0, stream>>>(ref, ref_out, num_blocks);
    if (cudaGetLastError() != cudaSuccess) return SPEC_ERR_CUDA;
  }
  const long long ctas = (entries + 4 * kThreads - 1) / (4 * kThreads);
  pages_refs_spread_kernel<FORK><<<(unsigned)(ctas < 304 ? ctas : 304), kThreads, 0, stream>>>(
      table, prefix_len, parent, batch, batch_out, max_blocks, block_size, num_blocks, window, sinks, spare, table_out,
      prefix_out, ref_out, status);
  return sv_launch_status();
}

}  // namespace

size_t sv_pages_ws_bytes(int batch, int max_blocks, int num_blocks) {
  return space_layout(nullptr, nullptr, batch, max_blocks, num_blocks);
}

static_assert(kMaxBatch == SPEC_PAGES_MAX_BATCH, "the header's limit");

int sv_pages_fork(const int32_t *table, const int32_t *prefix_len, const int32_t *parent, int batch, int batch_out,
                  int max_blocks, int num_blocks, const int32_t *ref, int32_t *table_out, int32_t *prefix_out,
                  int32_t *ref_out, int32_t *status, cudaStream_t stream) {
  return launch_refs<true>(table, prefix_len, parent, batch, batch_out, max_blocks, 1, num_blocks, 0, 0, 0, ref,
                           table_out, prefix_out, ref_out, status, stream);
}

int sv_pages_free(const int32_t *table, const int32_t *prefix_len, int batch, int max_blocks, int block_size,
                  int num_blocks, int window, int sinks, int spare, const int32_t *ref, int32_t *table_out,
                  int32_t *ref_out, int32_t *status, cudaStream_t stream) {
  return launch_refs<false>(table, prefix_len, nullptr, batch, 0, max_blocks, block_size, num_blocks, window, sinks,
                            spare, ref, table_out, nullptr, ref_out, status, stream);
}

int sv_pages_reserve(void *k, void *v, int vec_per_row, int n_layers, int hkv, int block_size, int num_blocks,
                     const int32_t *table, int32_t *table_out, int batch, int max_blocks, const int32_t *prefix_len,
                     const int32_t *need, const int32_t *ref, int32_t *ref_out, void *workspace, int32_t *status,
                     cudaStream_t stream) {
  Space ws;
  space_layout(&ws, workspace, batch, max_blocks, num_blocks);
  const int rc = launch_plan(reserve_plan_kernel, num_blocks, stream, table, table_out, batch, max_blocks, block_size,
                             num_blocks, prefix_len, need, ref, ref_out, ws, status);
  if (rc != SPEC_OK) return rc;
  return launch_copy<false>(k, v, n_layers, hkv, block_size, num_blocks, vec_per_row, batch, ws, nullptr, nullptr, 0,
                            status, stream);
}

int sv_pages_compact(void *k, void *v, int vec_per_row, int n_layers, int hkv, int block_size, int num_blocks,
                     const int32_t *table, int32_t *table_out, int batch, int max_blocks, const int32_t *ref,
                     int32_t *ref_out, int32_t *n_used, int32_t *remap, void *workspace, int32_t *status,
                     cudaStream_t stream) {
  Space ws;
  space_layout(&ws, workspace, batch, max_blocks, num_blocks);
  const int rc = launch_plan(compact_plan_kernel, num_blocks, stream, block_size, num_blocks, ref, ref_out, n_used,
                             remap, ws);
  if (rc != SPEC_OK) return rc;
  return launch_copy<true>(k, v, n_layers, hkv, block_size, num_blocks, vec_per_row, (num_blocks + 1) / 2, ws, table,
                           table_out, (int64_t)batch * max_blocks, status, stream);
}

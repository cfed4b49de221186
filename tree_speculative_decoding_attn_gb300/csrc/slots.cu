// Where packed tokens lie in a paged cache, and their rows' way in and out.
//
// Token t of a batch of packed requests belongs to the request b with
// off[b] <= t < off[b + 1], off the running sum of the requests' lengths; it
// sits at position prefix_len[b] + t - off[b], whose row of the pool follows
// from the block table.  Every CTA sums the lengths for itself (at most 4096,
// one pass of a block scan) and looks its tokens' requests up in the sums in
// shared memory: one launch, no order between CTAs, and the call is as long
// as a launch and three dependent loads (64 requests of one token 5 us with
// the rows' write behind it).
#include "common.cuh"
#include "kernels.h"
#include "tc_ptx.cuh"

namespace {

constexpr int kThreads = 256, kMaxBatch = SPEC_PAGES_MAX_BATCH;

__global__ void __launch_bounds__(kThreads)
    slots_kernel(const int32_t *__restrict__ table, const int32_t *__restrict__ prefix_len,
                 const int32_t *__restrict__ new_len, int batch, int max_blocks, int block_size, int num_blocks,
                 int room, int32_t *__restrict__ offsets, int32_t *__restrict__ slots, int32_t *__restrict__ positions,
                 int32_t *status) {
  __shared__ int s_off[kMaxBatch + 1];
  __shared__ long long s_warp[kThreads / 32];
  sv::ptx::grid_dep_launch();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  // lengths of this thread's requests, summed in 64 bits
  const int per = (batch + kThreads - 1) / kThreads, b0 = threadIdx.x * per;
  long long sum = 0;
  for (int i = 0; i < per; ++i)
    if (b0 + i < batch) sum += max(0, new_len[b0 + i]);
  long long up = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, up, o);
    if (lane >= o) up += v;
  }
  if (lane == 31) s_warp[warp] = up;
  __syncthreads();
  long long at = up - sum, all = 0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) {
    if (w < warp) at += s_warp[w];
    all += s_warp[w];
  }
  // (sums past the room stop at it: those tokens are dropped)
  for (int i = 0; i < per; ++i)
    if (b0 + i < batch) {
      s_off[b0 + i] = (int)min(at, (long long)room);
      at += max(0, new_len[b0 + i]);
    }
  if (threadIdx.x == 0) {
    s_off[batch] = (int)min(all, (long long)room);
    if (all > room && blockIdx.x == 0) sv::report(status, SPEC_DEV_CAPACITY);
  }
  __syncthreads();
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i <= batch; i += kThreads) offsets[i] = s_off[i];
  const int total = s_off[batch];
  for (int64_t t = blockIdx.x * kThreads + threadIdx.x; t < room; t += (int64_t)gridDim.x * kThreads) {
    int slot = -1, pos = -1;
    if (t < total) {
      int lo = 0, hi = batch;  // s_off[lo] <= t < s_off[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_off[mid] <= t) lo = mid;
        else hi = mid;
      }
      const int P = prefix_len[lo];
      const long long p = (long long)P + (t - s_off[lo]);
      if (P < 0 || p >= (long long)max_blocks * block_size) {
        sv::report(status, SPEC_DEV_CAPACITY);
      } else {
        pos = (int)p;
        const int blk = table[(int64_t)lo * max_blocks + pos / block_size];
        if (blk < 0 || blk >= num_blocks) sv::report(status, SPEC_DEV_BAD_BLOCK);
        else slot = blk * block_size + pos % block_size;
      }
    }
    slots[t] = slot;
    if (positions) positions[t] = pos;
  }
}

// Rows [T, hkv, dim] to (WRITE) or from their places in a pool [num_blocks,
// hkv, block_size, dim].  A CTA takes a run of rows, about 32 KB: their places
// are looked up once, into shared memory, and then every thread has kVecs
// 16-byte vectors in flight.  HBM-bound for long runs: 28400 rows of 576
// bf16 out of a pool 13.4 us, of them 9.7 at the copy rate, the rest the
// start.  Launched as a programmatic dependent, since it mostly follows
// slots_kernel.
constexpr int kVecs = 4, kRun = 256;
template <bool WRITE>
__global__ void __launch_bounds__(kThreads)
    rows_kernel(uint4 *__restrict__ pages, uint4 *__restrict__ rows, const int32_t *__restrict__ slots, int n_rows,
                int hkv, int block_size, int num_blocks, int vec, int run, int32_t *status) {
  __shared__ int64_t s_at[kRun];  // first vector of a row's place, -1: none
  sv::ptx::grid_dep_wait();
  const int row0 = blockIdx.x * run, n = min(run, n_rows - row0);
  if (threadIdx.x < n) {
    const int row = row0 + threadIdx.x, t = row / hkv, h = row - t * hkv;
    const int slot = slots[t], blk = slot / block_size;
    int64_t at = -1;
    if (slot >= num_blocks * block_size) sv::report(status, SPEC_DEV_BAD_BLOCK);
    else if (slot >= 0) at = (((int64_t)blk * hkv + h) * block_size + (slot - blk * block_size)) * vec;
    s_at[threadIdx.x] = at;
  }
  __syncthreads();
  uint4 *mine = rows + (int64_t)row0 * vec;
  const int total = n * vec;
  for (int e0 = threadIdx.x; e0 < total; e0 += kVecs * kThreads) {
    uint4 v[kVecs];
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int e = e0 + i * kThreads, r = e / vec;
      v[i] = make_uint4(0, 0, 0, 0);
      if (e >= total) continue;
      const int64_t at = s_at[r];
      if (WRITE) v[i] = __ldcs(mine + e);
      else if (at >= 0) v[i] = __ldcs(pages + at + (e - r * vec));
    }
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int e = e0 + i * kThreads, r = e / vec;
      if (e >= total) continue;
      const int64_t at = s_at[r];
      if (!WRITE) mine[e] = v[i];
      else if (at >= 0) pages[at + (e - r * vec)] = v[i];
    }
  }
}

template <bool WRITE>
int launch_rows(void *pages, void *rows, const int32_t *slots, int n_rows, int hkv, int block_size, int num_blocks,
                int vec, int32_t *status, cudaStream_t stream) {
  // (few rows: spread over the SMs rather than in long runs)
  int run = kVecs * kThreads / vec, spread = (n_rows + 303) / 304;
  run = run > spread ? spread : run;
  run = run < 1 ? 1 : run > kRun ? kRun : run;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((n_rows + run - 1) / run);
  cfg.blockDim = dim3(kThreads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, rows_kernel<WRITE>, (uint4 *)pages, (uint4 *)rows, slots, n_rows, hkv, block_size,
                            num_blocks, vec, run, status) == cudaSuccess
             ? SPEC_OK
             : SPEC_ERR_CUDA;
}

}  // namespace

int sv_pages_slots(const int32_t *table, const int32_t *prefix_len, const int32_t *new_len, int batch, int max_blocks,
                   int block_size, int num_blocks, int room, int32_t *offsets, int32_t *slots, int32_t *positions,
                   int32_t *status, cudaStream_t stream) {
  const int ctas = (room + kThreads - 1) / kThreads;
  slots_kernel<<<ctas < 608 ? ctas : 608, kThreads, 0, stream>>>(
      table, prefix_len, new_len, batch, max_blocks, block_size, num_blocks, room, offsets, slots, positions, status);
  return sv_launch_status();
}

int sv_slots_rows(bool write, void *pages, void *rows, const int32_t *slots, int T, int hkv, int block_size,
                  int num_blocks, int vec, int32_t *status, cudaStream_t stream) {
  return (write ? launch_rows<true> : launch_rows<false>)(pages, rows, slots, T * hkv, hkv, block_size, num_blocks, vec,
                                                          status, stream);
}

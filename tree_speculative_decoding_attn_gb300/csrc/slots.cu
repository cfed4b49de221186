// Where packed tokens lie in a paged cache, and their rows' way in and out.
//
// Token t of a batch of packed requests belongs to the request b with
// off[b] <= t < off[b + 1], off the running sum of the requests' lengths; it
// sits at position prefix_len[b] + t - off[b], whose row of the pool follows
// from the block table.  Every CTA sums the lengths for itself (at most 4096,
// one pass of a block scan) and looks its tokens' requests up in the sums in
// shared memory: one launch, no order between CTAs, and the call is as long
// as a launch and three dependent loads.
#include "common.cuh"
#include "kernels.h"

namespace {

constexpr int kThreads = 256, kMaxBatch = SPEC_PAGES_MAX_BATCH;

__global__ void __launch_bounds__(kThreads)
    slots_kernel(const int32_t *__restrict__ table, const int32_t *__restrict__ prefix_len,
                 const int32_t *__restrict__ new_len, int batch, int max_blocks, int block_size, int num_blocks,
                 int room, int32_t *__restrict__ offsets, int32_t *__restrict__ slots, int32_t *__restrict__ positions,
                 int32_t *status) {
  __shared__ int s_off[kMaxBatch + 1];
  __shared__ long long s_warp[kThreads / 32];
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
// hkv, block_size, dim], a 16-byte vector a thread, kVecs of them in flight.
constexpr int kVecs = 4;
template <bool WRITE>
__global__ void __launch_bounds__(kThreads)
    rows_kernel(uint4 *__restrict__ pages, uint4 *__restrict__ rows, const int32_t *__restrict__ slots, int T, int hkv,
                int block_size, int num_blocks, int vec, int32_t *status) {
  const int64_t total = (int64_t)T * hkv * vec, step = (int64_t)gridDim.x * kThreads;
  const int per = hkv * vec;
  const int limit = num_blocks * block_size;
  for (int64_t e0 = blockIdx.x * kThreads + threadIdx.x; e0 < total; e0 += kVecs * step) {
    uint4 v[kVecs];
    int64_t at[kVecs];
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int64_t e = e0 + i * step;
      at[i] = -1;
      v[i] = make_uint4(0, 0, 0, 0);
      if (e >= total) continue;
      const int t = (int)(e / per), r = (int)(e - (int64_t)t * per), h = r / vec, c = r - h * vec;
      const int slot = __ldg(slots + t);
      if (slot >= limit) sv::report(status, SPEC_DEV_BAD_BLOCK);
      if (slot >= 0 && slot < limit) {
        const int blk = slot / block_size;
        at[i] = (((int64_t)blk * hkv + h) * block_size + (slot - blk * block_size)) * vec + c;
        v[i] = WRITE ? sv::ldg_stream(rows + e) : pages[at[i]];
      }
    }
#pragma unroll
    for (int i = 0; i < kVecs; ++i) {
      const int64_t e = e0 + i * step;
      if (WRITE) {
        if (at[i] >= 0) pages[at[i]] = v[i];
      } else if (e < total) {
        rows[e] = v[i];
      }
    }
  }
}

}  // namespace

int sv_pages_slots(const int32_t *table, const int32_t *prefix_len, const int32_t *new_len, int batch, int max_blocks,
                   int block_size, int num_blocks, int room, int32_t *offsets, int32_t *slots, int32_t *positions,
                   int32_t *status, cudaStream_t stream) {
  const int ctas = (room + 4 * kThreads - 1) / (4 * kThreads);
  slots_kernel<<<ctas < 1 ? 1 : ctas < 608 ? ctas : 608, kThreads, 0, stream>>>(
      table, prefix_len, new_len, batch, max_blocks, block_size, num_blocks, room, offsets, slots, positions, status);
  return sv_launch_status();
}

int sv_slots_rows(bool write, void *pages, void *rows, const int32_t *slots, int T, int hkv, int block_size,
                  int num_blocks, int vec, int32_t *status, cudaStream_t stream) {
  const int64_t n = ((int64_t)T * hkv * vec + kThreads * kVecs - 1) / (kThreads * kVecs);
  const unsigned ctas = (unsigned)(n < 152 * 8 ? n : 152 * 8);
  if (write)
    rows_kernel<true><<<ctas, kThreads, 0, stream>>>((uint4 *)pages, (uint4 *)rows, slots, T, hkv, block_size, num_blocks,
                                                     vec, status);
  else
    rows_kernel<false><<<ctas, kThreads, 0, stream>>>((uint4 *)pages, (uint4 *)rows, slots, T, hkv, block_size,
                                                      num_blocks, vec, status);
  return sv_launch_status();
}

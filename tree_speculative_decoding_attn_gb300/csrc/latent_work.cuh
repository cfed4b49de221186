// What the kernels of latent attention share: the work's division into equal
// ranges, the joining of units that a range's end cuts, tensor maps.
//
// A unit is (sequence, ROWS query rows): its tree tiles, then its prefix
// tiles, TILE keys each.  All units of all sequences, in order, each with its
// tiles' weight (1) and a fixed one, are cut into one equal range per part (a
// CTA, or a pair), computed on the device since prefix lengths are device
// data that change inside a captured graph.
#pragma once
#include <cuda.h>

#include "common.cuh"
#include "tc_ptx.cuh"

namespace sv {

constexpr float kLow = -3.0e38f;  // running maximum before the first key

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t *>(&v);
}

template <int TILE, int ROWS> struct LatentWork {
  const int32_t *prefix_len;
  int batch, N, hq, s_max, max_prefix, RT, tree_tiles;
  LatentWork(const int32_t *prefix_len, int batch, int N, int hq, int s_max, int max_prefix)
      : prefix_len(prefix_len), batch(batch), N(N), hq(hq), s_max(s_max), max_prefix(max_prefix),
        RT((N * hq + ROWS - 1) / ROWS), tree_tiles((N + TILE - 1) / TILE) {}
  __device__ int prefix(int b) const { return __ldg(prefix_len + b); }
  __device__ bool fits(int P) const { return P >= 0 && P <= max_prefix && P <= s_max; }
  // tiles of a unit of sequence b (0: its prefix length is refused)
  __device__ int tiles(int b) const {
    const int P = prefix(b);
    return fits(P) ? tree_tiles + (P + TILE - 1) / TILE : 0;
  }
};

struct LatentRange {
  long long lo, hi, b0;  // the range of weights, and where sequence b begins
  int b;                 // the sequence that holds lo
};

// a / b of whole numbers >= 0: in 32 bits where they fit (a 64-bit division is
// some hundred instructions).
__device__ __forceinline__ long long quotient(long long a, long long b) {
  return (a | b) >> 32 ? a / b : (long long)((unsigned)a / (unsigned)b);
}

// One warp: the range of part `part` of `parts`.  desc (may be null): the
// first range end inside a cut unit names it and its parts (sequence, unit,
// parts, 1).  status (may be null): refused prefix lengths are reported.
template <class Work>
__device__ __forceinline__ LatentRange latent_range(const Work &w, int part, int parts, int fixed, int4 *desc,
                                                    int32_t *status) {
  const int lane = threadIdx.x & 31;
  long long total = 0;
  int T0 = 0;  // of sequence `lane`
  for (int s = 0; s < w.batch; s += 32) {
    const int b = s + lane;
    if (b < w.batch) {
      const int T = w.tiles(b);
      if (s == 0) T0 = T;
      total += (long long)w.RT * (T + fixed);
      if (T == 0) report(status, SPEC_DEV_CAPACITY);
    }
  }
  for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  // (no more ranges than weight: each that begins inside a unit has a tile)
  const long long n = total < parts ? total : parts;
  LatentRange r{0, 0, 0, 0};
  if (part >= n) {
    if (desc && lane == 0) *desc = make_int4(0, 0, 0, 0);
    return r;
  }
  const long long lo = quotient(total * part, n), hi = quotient(total * (part + 1), n);
  long long base = 0;
  for (int s = 0; s < w.batch; s += 32) {
    const int b = s + lane;
    const int T = b >= w.batch ? 0 : s == 0 ? T0 : w.tiles(b);
    const long long mine = b < w.batch ? (long long)w.RT * (T + fixed) : 0;
    long long up = mine;
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, up, o);
      if (lane >= o) up += v;
    }
    const long long first = base + up - mine;
    const bool here = b < w.batch && first <= lo && lo < first + mine;
    if (here && desc) {
      int4 d = make_int4(0, 0, 0, 0);
      const int unit = (int)quotient(lo - first, T + fixed);
      const long long start = first + (long long)unit * (T + fixed) + fixed;  // where the unit's first tile weighs
      if (T > 0 && lo > start && quotient(total * (part - 1), n) <= start) {
        // the last range that begins before the unit's end: the largest e
        // with floor(total e / n) < start + T, that is total e < (start + T) n
        const long long e = quotient((start + T) * n + total - 1, total) - 1;
        d = make_int4(b, unit, (int)(e < n ? e : n - 1) - part + 2, 1);
      }
      *desc = d;
    }
    const unsigned who = __ballot_sync(0xffffffffu, here);
    if (who) {
      const int l = __ffs(who) - 1;
      r.lo = lo;
      r.hi = hi;
      r.b0 = __shfl_sync(0xffffffffu, first, l);
      r.b = s + l;
      return r;
    }
    base += __shfl_sync(0xffffffffu, up, 31);
  }
  return r;
}

// The segments of a range in order: tiles [t0, t1) of T of unit rt of
// sequence b, whose prefix is P.
template <class Work> struct LatentWalk {
  long long pos, end, b0;
  int b, next_b, rt, t0, t1, T, P, fixed;
  __device__ LatentWalk(const LatentRange &r, int fixed)
      : pos(r.lo), end(r.hi), b0(r.b0), b(r.b), next_b(r.b), rt(0), t0(0), t1(0), T(0), P(0), fixed(fixed) {}
  __device__ bool advance(const Work &w) {
    while (pos < end && next_b < w.batch) {
      b = next_b;
      T = w.tiles(b);
      P = w.prefix(b);
      const int wu = T + fixed;
      rt = (int)quotient(pos - b0, wu);
      const long long u0 = b0 + (long long)rt * wu, u1 = u0 + wu, stop = end < u1 ? end : u1;
      t0 = (int)max(0ll, pos - u0 - fixed);
      t1 = T ? (int)max(0ll, stop - u0 - fixed) : 0;
      pos = stop;
      if (stop == u1 && rt == w.RT - 1) {
        ++next_b;
        b0 = u1;
      }
      if (t1 > t0) return true;
    }
    return false;
  }
};

// A part's partial: ROWS rows of LAT float32 sums, then ROWS pairs (maximum in
// log2 units, sum).  Part p has two: 2p for a segment cut at its start, 2p + 1
// for one cut at its end alone.
__host__ __device__ constexpr size_t latent_slot_floats(int lat, int rows) { return rows * (size_t)(lat + 2); }

// Joins the parts of cut units: block (row, cut unit, dims).  The 128 threads
// are GROUPS groups, each with its share of the parts, a thread four dims of
// 512 / GROUPS; all groups' sums go through shared memory.  Many parts (one
// long sequence) take more groups and blocks of fewer dims.
template <int LAT, int ROWS, int GROUPS>
__global__ void __launch_bounds__(128)
    latent_join_kernel(const float *__restrict__ ws, const int4 *__restrict__ desc, int parts,
                       __nv_bfloat16 *__restrict__ out, int R) {
  constexpr int MOST = 160, PER = 128 / GROUPS, B = 8;  // parts; threads a group; loads in flight
  __shared__ float s_a[MOST], s_l;
  __shared__ float4 s_acc[GROUPS][PER];
  __shared__ int s_part;
  const int lane = threadIdx.x & 31, lr = blockIdx.x;
  if (threadIdx.x == 0) s_part = 0;
  ptx::grid_dep_wait();
  __syncthreads();
  // the cut unit blockIdx.y of those that there are, by its first range end
  if (threadIdx.x < 32) {
    int seen = 0;
    for (int p = 1; p < parts; p += 32) {
      const unsigned cut = __ballot_sync(0xffffffffu, p + lane < parts && desc[p + lane].w != 0);
      const int mine = seen + __popc(cut & ((1u << lane) - 1));
      if ((cut >> lane & 1) && mine == (int)blockIdx.y) s_part = p + lane;
      seen += __popc(cut);
    }
  }
  __syncthreads();
  const int part0 = s_part;
  if (part0 == 0) return;
  const int4 d = desc[part0];
  const int row = d.y * ROWS + lr;
  if (row >= R) return;
  // the first part ends its range (slot 1), the others begin theirs (slot 0)
  auto part = [&](int i) {
    return ws + (size_t)(i == 0 ? 2 * (part0 - 1) + 1 : 2 * (part0 - 1 + i)) * latent_slot_floats(LAT, ROWS);
  };
  if (threadIdx.x < 32) {
    float2 ml[MOST / 32];
    float m = kLow, l = 0.f;
#pragma unroll
    for (int i = 0; i < MOST / 32; ++i) {
      const int p = i * 32 + lane;
      ml[i] = p < d.z ? *reinterpret_cast<const float2 *>(part(p) + ROWS * (size_t)LAT + 2 * lr) : make_float2(kLow, 0.f);
      m = fmaxf(m, ml[i].x);
    }
    m = warp_max(m);
#pragma unroll
    for (int i = 0; i < MOST / 32; ++i) {
      const float a = exp2f(ml[i].x - m);
      s_a[i * 32 + lane] = a;
      l = fmaf(a, ml[i].y, l);
    }
    l = warp_sum(l);
    if (lane == 0) s_l = l;
  }
  const int group = threadIdx.x / PER, at = threadIdx.x % PER, dim = blockIdx.z * (PER * 4) + at * 4;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  bool first = true;
  for (int p0 = group; p0 < d.z || first; p0 += B * GROUPS) {
    float4 x[B];
#pragma unroll
    for (int i = 0; i < B; ++i)
      x[i] = __ldcs(reinterpret_cast<const float4 *>(part(min(p0 + i * GROUPS, d.z - 1)) + (size_t)lr * LAT + dim));
    if (first) __syncthreads();  // the weights, behind the first loads
    first = false;
#pragma unroll
    for (int i = 0; i < B; ++i) {
      if (p0 + i * GROUPS >= d.z) continue;
      const float a = s_a[p0 + i * GROUPS];
      acc.x = fmaf(a, x[i].x, acc.x);
      acc.y = fmaf(a, x[i].y, acc.y);
      acc.z = fmaf(a, x[i].z, acc.z);
      acc.w = fmaf(a, x[i].w, acc.w);
    }
  }
  if (GROUPS > 1) {
    s_acc[group][at] = acc;
    __syncthreads();
    if (group > 0) return;
#pragma unroll
    for (int i = 1; i < GROUPS; ++i) {
      const float4 o = s_acc[i][at];
      acc.x += o.x;
      acc.y += o.y;
      acc.z += o.z;
      acc.w += o.w;
    }
  }
  const float inv = s_l == 0.f ? 0.f : 1.f / s_l;  // a row that sees nothing: zeros
  *reinterpret_cast<uint2 *>(out + ((int64_t)d.x * R + row) * LAT + dim) =
      make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
}
template <int LAT, int ROWS>
int launch_latent_join(const float *slots, const int4 *desc, __nv_bfloat16 *out, int R, int parts, long long units,
                       cudaStream_t stream) {
  if (parts == 1) return SPEC_OK;
  constexpr int FEW = 512 / LAT, MANY = 4 * FEW;
  const bool many = parts > 4 * units;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(R < ROWS ? R : ROWS, units < parts - 1 ? (unsigned)units : parts - 1, many ? 4 : 1);
  cfg.blockDim = dim3(128);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t e = many ? cudaLaunchKernelEx(&cfg, latent_join_kernel<LAT, ROWS, MANY>, slots, desc, parts, out, R)
                             : cudaLaunchKernelEx(&cfg, latent_join_kernel<LAT, ROWS, FEW>, slots, desc, parts, out, R);
  return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

// ---------------------------------------------------------------- tensor maps
typedef CUresult (*EncodeTiledFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                  const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                  CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// cuTensorMapEncodeTiled through the runtime (no link against libcuda);
// resolved once per process.
inline EncodeTiledFn encode_tiled() {
  static EncodeTiledFn fn = [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    const bool ok = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
                        cudaSuccess && q == cudaDriverEntryPointSuccess;
    return ok ? reinterpret_cast<EncodeTiledFn>(p) : nullptr;
  }();
  return fn;
}

// A bf16 map with 128-byte swizzle; a dim of size 0 is left out.  Rows of
// 64-element column groups come in boxes of rows x groups, which lie in shared
// memory group by group.  (A TMA box of 64 rows of 128 bytes takes 186 cycles
// of an SM, one of 128 rows 311: 44 and 53 bytes a cycle, measured.)
struct MapDim {
  long long size, stride;  // (bytes)
  int box;
};
inline int make_map(CUtensorMap *m, const void *base, const MapDim (&d)[5]) {
  EncodeTiledFn enc = encode_tiled();
  if (!enc) return SPEC_ERR_CUDA;
  cuuint64_t dims[5], strides[4];
  cuuint32_t box[5], es[5] = {1, 1, 1, 1, 1}, rank = 0;
  for (const MapDim &x : d) {
    if (x.size == 0) continue;
    dims[rank] = (cuuint64_t)x.size;
    box[rank] = (cuuint32_t)x.box;
    if (rank > 0) strides[rank - 1] = (cuuint64_t)x.stride;
    ++rank;
  }
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void *>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? SPEC_OK
             : SPEC_ERR_CUDA;
}

}  // namespace sv

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
  int far;  // so many tiles of all sequences together do not stay in L2
  LatentWork(const int32_t *prefix_len, int batch, int N, int hq, int s_max, int max_prefix, int row_bytes)
      : prefix_len(prefix_len), batch(batch), N(N), hq(hq), s_max(s_max), max_prefix(max_prefix),
        RT((N * hq + ROWS - 1) / ROWS), tree_tiles((N + TILE - 1) / TILE), far((100 << 20) / (TILE * row_bytes)) {}
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
// Where whole units share out nearly as evenly, none is cut: the longest part
// is then no more than a fifth and `join` weights (about what partials and their
// join cost) above the mean.  us cut / whole: one token of 64 heads, batch 64, 4096
// keys 84 / 72, 500 keys 35 / 21; 64 heads x 32 nodes, 4 trees over 4096 keys 80
// / 60, 32 trees 439 / 406, over 8192 keys 902 / 790 (whole units of a sequence
// run side by side, in L2); one token of 16 heads, batch 140, 2048 keys 68 / 61.
// Not whole: 64 heads x 9 nodes, 8 trees over 6000 keys 68 / 89; one token of 64
// heads, 64 sequences of 1000 to 8000 keys 86 / 98; 32 heads, 16 sequences of
// 1000 keys 19 / 23.
template <class Work>
__device__ __forceinline__ LatentRange latent_range(const Work &w, int part, int parts, int fixed, int join, int4 *desc,
                                                    int32_t *status) {
  const int lane = threadIdx.x & 31;
  long long total = 0;
  int T0 = 0, most = 0;  // tiles of sequence `lane`, of the longest
  for (int s = 0; s < w.batch; s += 32) {
    const int b = s + lane;
    if (b < w.batch) {
      const int T = w.tiles(b);
      if (s == 0) T0 = T;
      most = max(most, T);
      total += (long long)w.RT * (T + fixed);
      if (T == 0) report(status, SPEC_DEV_CAPACITY);
    }
  }
  most = __reduce_max_sync(0xffffffffu, most) + fixed;
  for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
  LatentRange r{0, 0, 0, 0};
  long long base = 0;  // weight of the sequences before the 32 that are looked at
  // sequence b = s + lane: its tiles, its weight, and where it begins
  auto look = [&](int s, int &T, long long &mine, long long &first) {
    const int b = s + lane;
    T = b >= w.batch ? 0 : s == 0 ? T0 : w.tiles(b);
    mine = b < w.batch ? (long long)w.RT * (T + fixed) : 0;
    long long up = mine;
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(0xffffffffu, up, o);
      if (lane >= o) up += v;
    }
    first = base + up - mine;
    base += __shfl_sync(0xffffffffu, up, 31);
  };
  int T;
  long long mine, first;
  const long long units = (long long)w.batch * w.RT, each = units <= parts ? 1 : quotient(units + parts - 1, parts);
  if (5 * each * most * parts <= 6 * total + 5ll * join * parts) {  // whole units, `each` a part
    const long long i0 = each * part, i1 = i0 + each;
    if (desc && lane == 0) *desc = make_int4(0, 0, 0, 0);
    if (i0 >= units) return r;
    const int b0 = (int)quotient(i0, w.RT), b1 = (int)quotient(i1, w.RT);
    r.b = b0;
    r.hi = total;
    for (int s = 0; s < w.batch && s <= b1; s += 32) {
      look(s, T, mine, first);
      const long long lo = first + (i0 - (long long)b0 * w.RT) * (T + fixed);
      const long long hi = first + (i1 - (long long)b1 * w.RT) * (T + fixed);
      if (b0 >> 5 == s >> 5) {
        r.b0 = __shfl_sync(0xffffffffu, first, b0 & 31);
        r.lo = __shfl_sync(0xffffffffu, lo, b0 & 31);
      }
      if (b1 < w.batch && b1 >> 5 == s >> 5) r.hi = __shfl_sync(0xffffffffu, hi, b1 & 31);
    }
    return r;
  }
  // (no more ranges than weight: each that begins inside a unit has a tile)
  long long n = total < parts ? total : parts;
  // The units of a sequence read the same rows.  Where those do not stay in L2,
  // parts in halves of a unit let pairs of units read them at the same time.  us
  // with all parts / in halves: 4 sequences of 4 units over 32768 keys 127 / 115
  // (76 and 72 parts, 4.5 a unit), 1 of 3 over 93000 80 / 75, 3 of 5 over 40000 125
  // / 120, 2 of 8 over 50000 163 / 157, 16 of 3 over 8000 105 / 103, 2 of 2 over
  // 60000 the same; 8 of 2 over 16384 72 / 78.  Lengths that differ (4 of 32000 to
  // 32768: 123) put the cuts elsewhere in each sequence.
  if (w.RT > 1 && units * most == total && (long long)most * w.batch > w.far) {
    const long long even = quotient(2ll * parts, units) * units / 2;
    if (10 * even >= 9ll * parts && even < n) n = even;
  }
  if (part >= n) {
    if (desc && lane == 0) *desc = make_int4(0, 0, 0, 0);
    return r;
  }
  const long long lo = quotient(total * part, n), hi = quotient(total * (part + 1), n);
  for (int s = 0; s < w.batch; s += 32) {
    const int b = s + lane;
    look(s, T, mine, first);
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
// Where dim `dim` of row `row` lies in it.  128 rows: [LAT / 4][128][4], since a
// thread that writes them holds a row, and a warp's store is 512 bytes in one
// piece (a row after another: 32 lines; 6.5 us for a pair's partial instead of 3).
template <int LAT, int ROWS> __host__ __device__ constexpr size_t latent_at(int row, int dim) {
  return ROWS == 128 ? ((size_t)(dim >> 2) * ROWS + row) * 4 + (dim & 3) : row * (size_t)LAT + dim;
}

constexpr int kMostParts = 160;
// The k-th cut unit of those that there are, by its first range end (part 0:
// fewer than k + 1).  One warp; all entries in flight at once.
__device__ __forceinline__ void latent_cut(const int4 *desc, int parts, int k, int *part, int4 *d) {
  const int lane = threadIdx.x & 31;
  int4 e[kMostParts / 32];
#pragma unroll
  for (int i = 0; i < kMostParts / 32; ++i) {
    const int p = 1 + i * 32 + lane;
    e[i] = p < parts ? desc[p] : make_int4(0, 0, 0, 0);
  }
  if (lane == 0) *part = 0;
  __syncwarp();
  int seen = 0;
#pragma unroll
  for (int i = 0; i < kMostParts / 32; ++i) {
    const unsigned cut = __ballot_sync(0xffffffffu, e[i].w != 0);
    if (e[i].w != 0 && seen + __popc(cut & ((1u << lane) - 1)) == k) {
      *part = 1 + i * 32 + lane;
      *d = e[i];
    }
    seen += __popc(cut);
  }
}
// What the n parts of a row weigh (into a[]), and the sum of all their sums.
// One warp; n <= MOST.
template <int MOST, class Stats>
__device__ __forceinline__ float latent_weights(int n, float *a, const Stats &stats) {
  const int lane = threadIdx.x & 31;
  float2 ml[MOST / 32];
  float m = kLow, l = 0.f;
#pragma unroll
  for (int i = 0; i < MOST / 32; ++i) {
    ml[i] = i * 32 + lane < n ? stats(i * 32 + lane) : make_float2(kLow, 0.f);
    m = fmaxf(m, ml[i].x);
  }
  m = warp_max(m);
#pragma unroll
  for (int i = 0; i < MOST / 32; ++i) {
    const float w = exp2f(ml[i].x - m);
    if (i * 32 + lane < n) a[i * 32 + lane] = w;
    l = fmaf(w, ml[i].y, l);
  }
  return warp_sum(l);
}
__device__ __forceinline__ void fma4(float4 &acc, float a, const float4 &x) {
  acc.x = fmaf(a, x.x, acc.x);
  acc.y = fmaf(a, x.y, acc.y);
  acc.z = fmaf(a, x.z, acc.z);
  acc.w = fmaf(a, x.w, acc.w);
}
__device__ __forceinline__ void store4(__nv_bfloat16 *p, const float4 &v, float l) {
  const float inv = l == 0.f ? 0.f : 1.f / l;  // a row that sees nothing: zeros
  *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf16(v.x * inv, v.y * inv), pack_bf16(v.z * inv, v.w * inv));
}

// Joins the parts of cut units, a thread four dims of a row at a time.
// BY_ROW (FORM 8, and partials of 16 rows): block (row, cut unit, LAT / FORM
// dims), ten parts in flight, shared out over groups of threads whose sums go
// through shared memory.  Otherwise block (8 rows, cut unit, FORM 1: 64 dims, FORM
// 0: all), the rows side by side as they lie.
template <int LAT, int ROWS, int FORM>
__global__ void __launch_bounds__(128)
    latent_join_kernel(const float *__restrict__ ws, const int4 *__restrict__ desc, int parts,
                       __nv_bfloat16 *__restrict__ out, int R) {
  constexpr bool BY_ROW = FORM == 8 || ROWS == 16;
  constexpr int RB = BY_ROW ? 1 : 8;  // rows of a block
  __shared__ float s_a[RB][kMostParts], s_l[RB];
  __shared__ int s_part;
  __shared__ int4 s_desc;
  const int warp = threadIdx.x >> 5;
  ptx::grid_dep_wait();
  if ((int)gridDim.y < parts - 1) {
    if (warp == 0) latent_cut(desc, parts, blockIdx.y, &s_part, &s_desc);
  } else if (threadIdx.x == 0) {  // as many blocks as range ends: each looks at its own
    s_desc = desc[blockIdx.y + 1];
    s_part = s_desc.w != 0 ? (int)blockIdx.y + 1 : 0;
  }
  __syncthreads();
  const int part0 = s_part;
  if (part0 == 0) return;
  const int4 d = s_desc;
  const int lr0 = blockIdx.x * RB, rows = min(min(RB, ROWS - lr0), R - d.y * ROWS - lr0);
  if (rows <= 0) return;
  // the first part ends its range (slot 1), the others begin theirs (slot 0)
  auto part = [&](int i) {
    return ws + (size_t)(i == 0 ? 2 * (part0 - 1) + 1 : 2 * (part0 - 1 + i)) * latent_slot_floats(LAT, ROWS);
  };
  // (beside the first of the sums)
  auto weights = [&]() {
    for (int r = warp; r < rows; r += 4) {
      const float l = latent_weights<kMostParts>(d.z, s_a[r], [&](int p) {
        return *reinterpret_cast<const float2 *>(part(p) + ROWS * (size_t)LAT + 2 * (lr0 + r));
      });
      if ((threadIdx.x & 31) == 0) s_l[r] = l;
    }
    __syncthreads();
  };
  __nv_bfloat16 *o = out + ((int64_t)d.x * R + d.y * ROWS + lr0) * LAT;
  auto load = [&](int p, int r, int dim) {
    return __ldcs(reinterpret_cast<const float4 *>(part(p) + latent_at<LAT, ROWS>(lr0 + r, dim)));
  };
  if constexpr (BY_ROW) {
    constexpr int DIMS = LAT / FORM, PER = DIMS / 4, GROUPS = 128 / PER, B = 10;  // B: loads in flight
    __shared__ float4 s_acc[GROUPS][PER];
    const int group = threadIdx.x / PER, at = threadIdx.x % PER, dim = blockIdx.z * DIMS + at * 4;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float4 x[B];
    auto fetch = [&](int p0) {
#pragma unroll
      for (int i = 0; i < B; ++i)
        if (p0 + i * GROUPS < d.z) x[i] = load(p0 + i * GROUPS, 0, dim);
    };
    fetch(group);
    weights();
    for (int p0 = group; p0 < d.z; p0 += B * GROUPS) {
      if (p0 != group) fetch(p0);
#pragma unroll
      for (int i = 0; i < B; ++i)
        if (p0 + i * GROUPS < d.z) fma4(acc, s_a[0][p0 + i * GROUPS], x[i]);
    }
    if (GROUPS > 1) {
      s_acc[group][at] = acc;
      __syncthreads();
      if (group > 0) return;
#pragma unroll
      for (int i = 1; i < GROUPS; ++i) fma4(acc, 1.f, s_acc[i][at]);
    }
    store4(o + dim, acc, s_l[0]);
  } else {
    constexpr int NI = FORM == 1 ? 1 : LAT / 64, B = FORM == 1 ? 8 : 2;  // pieces of a thread; parts in flight
    const int r = threadIdx.x & 7, dim0 = blockIdx.z * 64 + (threadIdx.x >> 3) * 4;
    float4 acc[NI], x[B][NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) acc[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    auto fetch = [&](int p) {
#pragma unroll
      for (int h = 0; h < B; ++h)
#pragma unroll
        for (int i = 0; i < NI; ++i)
          if (p + h < d.z && r < rows) x[h][i] = load(p + h, r, dim0 + i * 64);
    };
    fetch(0);
    weights();
    if (r >= rows) return;
    for (int p = 0; p < d.z; p += B) {
      if (p > 0) fetch(p);
#pragma unroll
      for (int h = 0; h < B; ++h)
#pragma unroll
        for (int i = 0; i < NI; ++i)
          if (p + h < d.z) fma4(acc[i], s_a[r][p + h], x[h][i]);
    }
#pragma unroll
    for (int i = 0; i < NI; ++i) store4(o + (size_t)r * LAT + dim0 + i * 64, acc[i], s_l[r]);
  }
}
template <int LAT, int ROWS>
int launch_latent_join(const float *slots, const int4 *desc, __nv_bfloat16 *out, int R, int parts, long long units,
                       cudaStream_t stream) {
  if (parts == 1) return SPEC_OK;
  const int rows = R < ROWS ? R : ROWS, cut = units < parts - 1 ? (int)units : parts - 1;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(128);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // (us of the whole call, FORM 8 / 1 / 0: 128 rows of 76 parts 38 / 60 / -, 512
  // rows of 19 parts 57 / 52 / -, 75 units of 128 rows - / 128 / 124)
  auto run = [&](auto kernel, dim3 grid) {
    cfg.gridDim = grid;
    return cudaLaunchKernelEx(&cfg, kernel, slots, desc, parts, out, R) == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
  };
  if (rows * cut <= 256) return run(latent_join_kernel<LAT, ROWS, 8>, dim3(rows, cut, 8));
  if constexpr (ROWS == 16) {
    return run(latent_join_kernel<LAT, ROWS, 1>, dim3(rows, cut));
  } else {
    if (rows * cut <= 4096) return run(latent_join_kernel<LAT, ROWS, 1>, dim3((rows + 7) / 8, cut, LAT / 64));
    return run(latent_join_kernel<LAT, ROWS, 0>, dim3((rows + 7) / 8, cut));
  }
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

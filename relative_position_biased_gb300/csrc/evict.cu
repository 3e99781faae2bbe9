// evict.cu -- shrinks a K / V cache to the keys that matter: per sequence and
// kv head it keeps the newest `recent` keys, the first `sink` keys and, of the
// rest, the heaviest by accumulated attention weight (key_weights.cu; equal
// weights: the lower index), and moves the kept rows, in order, into another
// cache.  NaN weighs less than every number.
//
// Select: a cluster of CTAs per (sequence, kv head).  The weights become
// 32-bit keys in their order; three histogram passes (11 + 11 + 10 bits, from
// the top) over distributed shared memory find the exact smallest kept key
// and how many of its equals are kept; a last pass ranks the kept keys by
// ballots and writes their rows.  Nothing is sorted, and every count is an
// integer, so the result does not depend on any order.  Bound by the latency
// of four dependent passes over the weights (which stay in L2): the cluster
// is as wide as the longest sequence asks for.
// Move: a flat copy of the kept rows' bytes, any number of planes (codes,
// scales, bf16 rows); bound by memory.
#include <cooperative_groups.h>

#include <algorithm>

#include "nvfp4.cuh"

namespace cg = cooperative_groups;

namespace relattn {
namespace {

constexpr int ET = 512, EW = ET / 32;
constexpr int EB = 8;                        // keys of a lane in a tile
constexpr int ETILE = ET * EB;
constexpr int EBINS = 2048;

// Order-preserving bits: larger weight, larger key; -0 as 0, NaN below -inf.
__device__ __forceinline__ uint32_t rank_bits(float w) {
  if (w != w) return 0;
  const uint32_t b = __float_as_uint(w == 0.f ? 0.f : w);
  return (b >> 31) ? ~b : b | 0x80000000u;
}

struct Segment {
  int b, h, n, keep, sink, recent, rest, mid;   // mid: keys that compete for `rest` places
  int k0, d0;
  bool ok;
};

__device__ __forceinline__ Segment segment(const EvictArgs &a, int unit) {
  Segment s;
  s.b = unit / a.Hkv;
  s.h = unit - s.b * a.Hkv;
  s.k0 = a.cu_k[s.b];
  s.d0 = a.cu_keep[s.b];
  const int k1 = a.cu_k[s.b + 1], d1 = a.cu_keep[s.b + 1];
  s.n = k1 - s.k0;
  s.keep = d1 - s.d0;
  s.ok = s.k0 >= 0 && s.d0 >= 0 && k1 >= s.k0 && d1 >= s.d0 && s.keep <= s.n && s.n <= a.max_k && d1 <= a.total_keep &&
         (a.src.block_table ? (long)s.n <= (long)a.src.max_pages * a.src.page_size : (long)k1 <= a.src.rows) &&
         (a.dst.block_table ? (long)s.keep <= (long)a.dst.max_pages * a.dst.page_size : (long)d1 <= a.dst.rows);
  s.recent = min(a.recent, s.keep);
  s.sink = min(a.sink, min(s.keep - s.recent, s.n - s.recent));
  s.rest = s.keep - s.recent - s.sink;
  s.mid = s.n - s.recent - s.sink;
  return s;
}

__device__ __forceinline__ uint32_t weight_key(const EvictArgs &a, const Segment &s, int p, long *row) {
  *row = a.src.row(s.b, s.k0, p);
  return *row >= 0 ? rank_bits(__ldg(a.weights + (long)s.h * a.src.rows + *row)) : 0;
}

__global__ void __launch_bounds__(ET) relattn_evict_select_kernel(const __grid_constant__ EvictArgs a) {
  __shared__ unsigned hist[EBINS];
  __shared__ unsigned scan[EW];
  __shared__ int counts[2];                  // kept above the border / equal to it, in this CTA's keys
  __shared__ unsigned found[2];              // digit, places left below it
  __shared__ int wabove[EW], wequal[EW];
  cg::cluster_group cl = cg::this_cluster();
  const int cs = cl.num_blocks(), rank = cl.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const Segment s = segment(a, blockIdx.x / cs);
  const unsigned full = 0xffffffffu;
  if (!s.ok) {                               // the same for every CTA of the cluster
    if (rank == 0 && tid == 0) atomicOr(a.err, kDevErrSeqlens);
    if (s.d0 >= 0 && s.d0 + (long)s.keep <= a.total_keep)
      for (int i = tid; i < s.keep; i += ET) {
        a.src_row[(long)s.h * a.total_keep + s.d0 + i] = -1;
        if (s.h == 0) a.dst_row[s.d0 + i] = -1;
      }
    return;
  }
  // this CTA's keys, a multiple of 32 each
  const int chunk = ((s.n + cs - 1) / cs + 31) & ~31;
  const int lo = min(s.n, rank * chunk), hi = min(s.n, lo + chunk);
  const int mlo = max(lo, s.sink), mhi = min(hi, s.n - s.recent);   // its competing keys

  // the border: keys above it are kept, and `equal` of those on it
  uint32_t border = 0, mask = 0;
  int left = s.rest;
  if (s.rest > 0 && s.rest < s.mid) {
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const int bins = pass == 2 ? 1024 : 2048;
      for (int i = tid; i < bins; i += ET) hist[i] = 0;
      __syncthreads();
      for (int p0 = mlo + warp * 32 * EB; p0 < mhi; p0 += ETILE) {
        uint32_t key[EB];
        long row;
#pragma unroll
        for (int i = 0; i < EB; ++i) {
          const int p = p0 + 32 * i + lane;
          key[i] = p < mhi ? weight_key(a, s, p, &row) : 0;
        }
#pragma unroll
        for (int i = 0; i < EB; ++i) {
          const bool in = p0 + 32 * i + lane < mhi && (key[i] & mask) == border;
          const unsigned bin = (key[i] >> shift) & (bins - 1);
          const unsigned who = __ballot_sync(full, in);
          if (!who) continue;
          // a warp of equal digits (ties are common) adds once
          const unsigned lead = __shfl_sync(full, bin, __ffs(who) - 1);
          if (__all_sync(full, !in || bin == lead)) {
            if (lane == 0) atomicAdd(&hist[lead], (unsigned)__popc(who));
          } else if (in) {
            atomicAdd(&hist[bin], 1u);
          }
        }
      }
      cl.sync();
      // every CTA adds the cluster's histograms; thread t holds bins from the top
      unsigned c[4], mine = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int bin = bins - 1 - (4 * tid + j);
        c[j] = 0;
        if (bin >= 0)
          for (int r = 0; r < cs; ++r) c[j] += cl.map_shared_rank(hist, r)[bin];
        mine += c[j];
      }
      unsigned inc = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned y = __shfl_up_sync(full, inc, o);
        if (lane >= o) inc += y;
      }
      if (lane == 31) scan[warp] = inc;
      __syncthreads();
      unsigned before = inc - mine;
      for (int w = 0; w < warp; ++w) before += scan[w];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (before < (unsigned)left && before + c[j] >= (unsigned)left) {
          found[0] = bins - 1 - (4 * tid + j);
          found[1] = left - before;
        }
        before += c[j];
      }
      cl.sync();                             // histograms are read, and `found` is written
      border |= found[0] << shift;
      mask |= (uint32_t)(bins - 1) << shift;
      left = (int)found[1];
    }
  }
  const bool all = s.rest == s.mid, none = s.rest == 0;
  // kept / equal keys of this CTA, then of the CTAs before it
  auto kind = [&](int p, uint32_t key) {     // 0 dropped, 1 kept, 2 on the border
    if (p < s.sink || p >= s.n - s.recent) return 1;
    if (all) return 1;
    if (none) return 0;
    return key > border ? 1 : key == border ? 2 : 0;
  };
  if (tid < 2) counts[tid] = 0;
  __syncthreads();
  int na = 0, ne = 0;
  for (int p0 = lo + warp * 32 * EB; p0 < hi; p0 += ETILE) {
    long row;
    uint32_t key[EB];
#pragma unroll
    for (int i = 0; i < EB; ++i) {
      const int p = p0 + 32 * i + lane;
      key[i] = p < hi ? weight_key(a, s, p, &row) : 0;
    }
#pragma unroll
    for (int i = 0; i < EB; ++i) {
      const int p = p0 + 32 * i + lane, k = p < hi ? kind(p, key[i]) : 0;
      na += k == 1;
      ne += k == 2;
    }
  }
  na = __reduce_add_sync(full, na);
  ne = __reduce_add_sync(full, ne);
  if (lane == 0) {
    atomicAdd(&counts[0], na);
    atomicAdd(&counts[1], ne);
  }
  cl.sync();
  int above = 0, equal = 0;                  // before the tile at hand
  for (int r = 0; r < rank; ++r) {
    above += cl.map_shared_rank(counts, r)[0];
    equal += cl.map_shared_rank(counts, r)[1];
  }
  const int places = all || none ? 0 : left; // border keys kept, lowest index first
  for (int t0 = lo; t0 < hi; t0 += ETILE) {
    const int p0 = t0 + warp * 32 * EB;
    uint32_t key[EB];
    long row[EB];
#pragma unroll
    for (int i = 0; i < EB; ++i) {
      const int p = p0 + 32 * i + lane;
      row[i] = -1;
      key[i] = p < hi ? weight_key(a, s, p, &row[i]) : 0;
    }
    unsigned ba[EB], be[EB];
    int wa = 0, we = 0;
#pragma unroll
    for (int i = 0; i < EB; ++i) {
      const int p = p0 + 32 * i + lane, k = p < hi ? kind(p, key[i]) : 0;
      ba[i] = __ballot_sync(full, k == 1);
      be[i] = __ballot_sync(full, k == 2);
      wa += __popc(ba[i]);
      we += __popc(be[i]);
    }
    __syncthreads();                         // the previous tile's counts are read
    if (lane == 0) wabove[warp] = wa, wequal[warp] = we;
    __syncthreads();
    int a0 = above, e0 = equal;
    for (int w = 0; w < EW; ++w) {
      if (w < warp) a0 += wabove[w], e0 += wequal[w];
      above += wabove[w];
      equal += wequal[w];
    }
    const unsigned below = (1u << lane) - 1;
#pragma unroll
    for (int i = 0; i < EB; ++i) {
      const int p = p0 + 32 * i + lane;
      const bool on = be[i] >> lane & 1;
      const int eb = e0 + __popc(be[i] & below);
      if ((ba[i] >> lane & 1) || (on && eb < places)) {
        const int j = a0 + __popc(ba[i] & below) + min(eb, places);
        const long at = (long)s.d0 + j;
        long dst = a.dst.row(s.b, s.d0, j);
        if (row[i] < 0 || dst < 0) atomicOr(a.err, kDevErrSeqlens);
        a.src_row[(long)s.h * a.total_keep + at] = (int)row[i];
        if (s.h == 0) a.dst_row[at] = (int)dst;
        if (dst >= 0) {
          const long o = (long)s.h * a.dst.rows + dst;
          const long src = (long)s.h * a.src.rows + row[i];
          if (a.pos_out) a.pos_out[o] = a.key_pos ? (row[i] >= 0 ? __ldg(a.key_pos + src) : -1) : p;
          if (a.w_out) a.w_out[o] = row[i] >= 0 ? __ldg(a.weights + src) : 0.f;
        }
      }
      a0 += __popc(ba[i]);
      e0 += __popc(be[i]);
    }
  }
  cl.sync();                                 // no CTA leaves while another reads its counts
}

// Copy units: 16 bytes where a plane's rows and addresses allow, else 8, 4 or 1.
struct MoveArgs {
  const int32_t *src_row, *dst_row, *cu_keep;
  int batch, total_keep, Hkv, planes, units;
  long src_rows, dst_rows;
  const uint8_t *from[kMaxPlanes];
  uint8_t *to[kMaxPlanes];
  int bytes[kMaxPlanes], width[kMaxPlanes], first[kMaxPlanes + 1];
};

constexpr int MT = 256, MU = 4;              // units in flight per thread

__global__ void __launch_bounds__(MT) relattn_evict_move_kernel(const __grid_constant__ MoveArgs a) {
  const long per_row = (long)a.Hkv * a.units, total = a.total_keep * per_row;
  const int used0 = a.cu_keep[0], used1 = a.cu_keep[a.batch];
  for (long i0 = (long)blockIdx.x * MT * MU + threadIdx.x; i0 < total; i0 += (long)gridDim.x * MT * MU) {
    uint4 v[MU];
    uint8_t *to[MU];
    int width[MU];
#pragma unroll
    for (int k = 0; k < MU; ++k) {
      const long i = i0 + (long)k * MT;
      width[k] = 0;
      if (i >= total) continue;
      const int j = (int)(i / per_row), hu = (int)(i - j * per_row), h = hu / a.units, un = hu - h * a.units;
      if (j < used0 || j >= used1) continue;   // rows of no sequence
      const long src = __ldg(a.src_row + (long)h * a.total_keep + j), dst = __ldg(a.dst_row + j);
      if (src < 0 || dst < 0 || src >= a.src_rows || dst >= a.dst_rows) continue;
      int pl = 0;
#pragma unroll
      for (int q = 1; q < kMaxPlanes; ++q) pl += q < a.planes && un >= a.first[q];
      const int w = a.width[pl], off = (un - a.first[pl]) * w;
      const uint8_t *from = a.from[pl] + (src * a.Hkv + h) * a.bytes[pl] + off;
      to[k] = a.to[pl] + (dst * a.Hkv + h) * a.bytes[pl] + off;
      width[k] = w;
      if (w == 16) v[k] = __ldg(reinterpret_cast<const uint4 *>(from));
      else if (w == 8) {
        const uint2 x = __ldg(reinterpret_cast<const uint2 *>(from));
        v[k].x = x.x, v[k].y = x.y;
      } else if (w == 4) v[k].x = __ldg(reinterpret_cast<const unsigned *>(from));
      else v[k].x = __ldg(from);
    }
#pragma unroll
    for (int k = 0; k < MU; ++k) {
      if (width[k] == 16) *reinterpret_cast<uint4 *>(to[k]) = v[k];
      else if (width[k] == 8) *reinterpret_cast<uint2 *>(to[k]) = make_uint2(v[k].x, v[k].y);
      else if (width[k] == 4) *reinterpret_cast<unsigned *>(to[k]) = v[k].x;
      else if (width[k] == 1) *to[k] = (uint8_t)v[k].x;
    }
  }
}

}  // namespace

cudaError_t launch_evict(const EvictArgs &a, cudaStream_t stream) {
  // CTAs per (sequence, kv head): one per 16K keys, at most the portable 8
  int cs = 1;
  while (cs < 8 && a.max_k > cs * 16384) cs *= 2;
  const long units = (long)a.batch * a.Hkv;
  if (units * cs > 0x7fffffffL) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(units * cs));
  cfg.blockDim = dim3(ET);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = cs;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  cudaError_t e = cudaLaunchKernelEx(&cfg, relattn_evict_select_kernel, a);
  if (e != cudaSuccess) return e;
  if (a.planes == 0 || a.total_keep == 0) return cudaSuccess;
  MoveArgs m = {};
  m.src_row = a.src_row;
  m.dst_row = a.dst_row;
  m.cu_keep = a.cu_keep;
  m.batch = a.batch;
  m.total_keep = a.total_keep;
  m.Hkv = a.Hkv;
  m.planes = a.planes;
  m.src_rows = a.src.rows;
  m.dst_rows = a.dst.rows;
  for (int i = 0; i < a.planes; ++i) {
    m.from[i] = static_cast<const uint8_t *>(a.from[i]);
    m.to[i] = static_cast<uint8_t *>(a.to[i]);
    m.bytes[i] = a.bytes[i];
    const uintptr_t bits = reinterpret_cast<uintptr_t>(a.from[i]) | reinterpret_cast<uintptr_t>(a.to[i]) | (uintptr_t)a.bytes[i];
    m.width[i] = !(bits & 15) ? 16 : !(bits & 7) ? 8 : !(bits & 3) ? 4 : 1;
    m.first[i] = m.units;
    m.units += a.bytes[i] / m.width[i];
  }
  m.first[a.planes] = m.units;
  const long total = (long)a.total_keep * a.Hkv * m.units;
  const long grid = std::min<long>((total + MT * MU - 1) / (MT * MU), 1L << 20);
  relattn_evict_move_kernel<<<(unsigned)grid, MT, 0, stream>>>(m);
  return cudaGetLastError();
}

}  // namespace relattn

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
// integer, so the result does not depend on any order.  Few long sequences are
// selected by all SMs instead (a million keys of two heads: 128 us of the call
// to 81): the same passes, with the counts in global memory.  The keys are read
// once where a CTA's share fits its shared memory, else from L2 in each pass.
// Move: the kept rows' bytes, any number of planes (codes, scales, bf16 rows);
// bound by memory (half of 64 sequences of 1 to 32 thousand 4-bit rows of two
// heads: selection 49 us, move 61 us at 6.1 TB/s of DRAM traffic).
#include <cooperative_groups.h>

#include <algorithm>

#include "nvfp4.cuh"

namespace cg = cooperative_groups;

namespace relattn {
namespace {

constexpr int EB = 8;                        // keys of a lane in a tile
constexpr int EBINS = 2048;
constexpr int ECOPY = 4;                     // copies of a histogram: equal digits of a warp collide less
constexpr int kMaxCluster = 16;              // CTAs of a cluster (above 8: opted into)
constexpr int kCacheKeys = 46 * 1024;        // keys of a CTA that shared memory holds
constexpr int kWideUnits = 8, kWideKeys = 32 * 1024;         // (evict_wide_bytes)

// Order-preserving bits: larger weight, larger key; -0 as 0, NaN below -inf.
__device__ __forceinline__ uint32_t rank_bits(float w) {
  const uint32_t b = __float_as_uint(w + 0.f);
  return w != w ? 0u : b ^ ((uint32_t)((int)b >> 31) | 0x80000000u);
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

// A warp takes 32 EB keys from p0 (a multiple of 32) at a time, key 32 i + lane
// in [i].  32 keys share a page, so lane i looks up row i's page: base[i] is
// the cache row of key 32 i, -1 outside the cache.
__device__ __forceinline__ void rows_of(const EvictArgs &a, const Segment &s, int p0, int hi, int lane, int (&base)[EB]) {
  if (!a.src.block_table) {                  // (the segment's rows lie inside the cache)
#pragma unroll
    for (int i = 0; i < EB; ++i) base[i] = s.k0 + p0 + 32 * i;
    return;
  }
  int r = -1;
  if (lane < EB && p0 + 32 * lane < hi) r = (int)a.src.row(s.b, s.k0, p0 + 32 * lane);
#pragma unroll
  for (int i = 0; i < EB; ++i) base[i] = __shfl_sync(0xffffffffu, r, i);
}

template <bool CACHED>
__device__ __forceinline__ void load_keys(const EvictArgs &a, const Segment &s, int p0, int hi, int lane,
                                          const uint32_t *cache, int lo, uint32_t (&key)[EB]) {
  if (CACHED) {
#pragma unroll
    for (int i = 0; i < EB; ++i) {
      const int p = p0 + 32 * i + lane;
      key[i] = p < hi ? cache[p - lo] : 0;
    }
    return;
  }
  int base[EB];
  rows_of(a, s, p0, hi, lane, base);
  const float *w0 = a.weights + (long)s.h * a.src.rows + lane;
  float w[EB];
#pragma unroll
  for (int i = 0; i < EB; ++i) {
    const bool in = p0 + 32 * i + lane < hi && base[i] >= 0;
    w[i] = in ? __ldg(w0 + base[i]) : __int_as_float(0x7fffffff);
  }
#pragma unroll
  for (int i = 0; i < EB; ++i) key[i] = rank_bits(w[i]);
}

// A wide selection: words of workspace per (sequence, kv head): the barrier's
// counter, three passes' histograms, two counts of every CTA.
constexpr int kWideHist = 32, kWideCounts = kWideHist + 3 * EBINS, kWideCtas = 512, kWideWords = kWideCounts + 2 * kWideCtas;

// All CTAs of a (sequence, kv head), which a cooperative launch keeps resident
// together; false after a timeout.
__device__ __forceinline__ bool unit_barrier(unsigned *counter, unsigned target, int *err, int *failed) {
  __syncthreads();
  if (threadIdx.x == 0) {
    __threadfence();
    atomicAdd(counter, 1u);
    const long long t0 = clock64();
    int bad = 0;
    while (*reinterpret_cast<volatile unsigned *>(counter) < target)
      if (clock64() - t0 > 2000000000ll) {
        record_timeout(err, 60);
        bad = 1;
        break;
      }
    __threadfence();
    *failed = bad;
  }
  __syncthreads();
  return *failed == 0;
}

// Dynamic shared memory: the CTA's keys when CACHED.
template <int ET, bool CACHED, bool WIDE>
__global__ void __launch_bounds__(ET, 1024 / ET) relattn_evict_select_kernel(const __grid_constant__ EvictArgs a) {
  constexpr int EW = ET / 32, ETILE = ET * EB, EPT = EBINS / ET;      // EPT: bins of a thread
  extern __shared__ uint32_t cache[];
  __shared__ __align__(16) unsigned hist[EBINS * ECOPY];              // this CTA's counts of the pass
  __shared__ unsigned scan[EW], lscan[EW];
  __shared__ unsigned found[2];              // digit, places left below it
  __shared__ int counts[2];                  // kept above the border / equal to it, in this CTA's keys
  __shared__ int wabove[EW], wequal[EW];
  __shared__ unsigned total[EBINS];          // the cluster's counts of the pass
  __shared__ int failed;
  cg::cluster_group cl = cg::this_cluster();
  const int cs = WIDE ? a.ctas : (int)cl.num_blocks(), rank = WIDE ? (int)(blockIdx.x % cs) : (int)cl.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const Segment s = segment(a, blockIdx.x / cs);
  unsigned *wide = WIDE ? a.wide + (long)(blockIdx.x / cs) * kWideWords : nullptr;
  unsigned arrivals = 0;
  auto meet = [&]() {                        // the CTAs of the (sequence, kv head)
    if (!WIDE) {
      cl.sync();
      return true;
    }
    return unit_barrier(wide, arrivals += cs, a.err, &failed);
  };
  const unsigned full = 0xffffffffu;
  if (!s.ok) {                               // the same for every CTA of the cluster
    if (rank == 0 && tid == 0) atomicOr(a.err, kDevErrSeqlens);
    // Nothing of it is moved: each of its places among the kept rows says so.
    // (Every place lies in a sequence whose start is not above and whose end is
    // above it, so none keeps what the workspace held.)
    if (rank == 0)
      for (long j = max(s.d0, 0) + (long)tid; j < min(a.cu_keep[s.b + 1], a.total_keep); j += ET) {
        a.src_row[(long)s.h * a.total_keep + j] = -1;
        if (s.h == 0) a.dst_row[j] = -1;
      }
    return;
  }
  // this CTA's keys, a multiple of 32 each
  const long chunk = (((long)s.n + cs - 1) / cs + 31) & ~31L;
  const int lo = (int)min((long)s.n, rank * chunk), hi = (int)min((long)s.n, lo + chunk);
  const int m0 = s.sink, m1 = s.n - s.recent;                       // the competing keys
  const int mlo = max(lo, m0 & ~31), mhi = min(hi, m1);             // from a multiple of 32 (or none)

  if (CACHED) {
    for (int p0 = lo + warp * 32 * EB; p0 < hi; p0 += ETILE) {
      uint32_t key[EB];
      load_keys<false>(a, s, p0, hi, lane, nullptr, 0, key);
#pragma unroll
      for (int i = 0; i < EB; ++i) {
        const int p = p0 + 32 * i + lane;
        if (p < hi) cache[p - lo] = key[i];
      }
    }
    __syncthreads();
  }

  if (WIDE) {
    // Should a barrier give up, rows that no CTA got to list are not moved.
    for (long j = s.d0 + (long)rank * ET + tid; j < s.d0 + s.keep; j += (long)cs * ET) {
      a.src_row[(long)s.h * a.total_keep + j] = -1;
      if (s.h == 0) a.dst_row[j] = -1;
    }
    if (rank == a.test_skip_cta) return;     // (test hook: never arrives)
  }

  // the border: keys above it are kept, and `left` of those on it
  uint32_t border = 0, mask = 0;
  int left = s.rest, na = 0, ne = 0;         // na / ne: this CTA's keys above / on the border
  const bool choose = s.rest > 0 && s.rest < s.mid;
  if (choose) {
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
      const int bins = pass == 2 ? 1024 : 2048;
      for (int i = tid; i < bins; i += ET) reinterpret_cast<uint4 *>(hist)[i] = make_uint4(0, 0, 0, 0);
      __syncthreads();
      for (int p0 = mlo + warp * 32 * EB; p0 < mhi; p0 += ETILE) {
        uint32_t key[EB];
        load_keys<CACHED>(a, s, p0, mhi, lane, cache, lo, key);
#pragma unroll
        for (int i = 0; i < EB; ++i) {
          const int p = p0 + 32 * i + lane;
          const bool in = p >= m0 && p < mhi && (key[i] & mask) == border;
          if (in) atomicAdd(&hist[((key[i] >> shift) & (bins - 1)) * ECOPY + (lane & (ECOPY - 1))], 1u);
        }
      }
      const unsigned *sums = total;
      if (WIDE) {
        // the CTAs' counts meet in global memory (integers: in any order)
        unsigned *g = wide + kWideHist + pass * EBINS;
        sums = g;
        __syncthreads();
        for (int i = tid; i < bins; i += ET) {
          const uint4 x = reinterpret_cast<const uint4 *>(hist)[i];
          const unsigned c = x.x + x.y + x.z + x.w;
          if (c) atomicAdd(g + i, c);
        }
        if (!meet()) return;
      } else {
        cl.sync();
        // every CTA adds one slice of the bins over the cluster and hands the
        // sums to all
        const int slice = bins / cs;
        for (int i = tid; i < slice; i += ET) {
          const int bin = rank * slice + i;
          unsigned c = 0;
          for (int r = 0; r < cs; ++r) {
            const uint4 x = reinterpret_cast<const uint4 *>(cl.map_shared_rank(hist, r))[bin];
            c += x.x + x.y + x.z + x.w;
          }
          for (int r = 0; r < cs; ++r) cl.map_shared_rank(total, r)[bin] = c;
        }
        cl.sync();
      }
      // thread t holds EPT bins, from the top
      unsigned c[EPT], own[EPT], mine = 0, lmine = 0;
#pragma unroll
      for (int j = 0; j < EPT; ++j) {
        const int bin = bins - 1 - (EPT * tid + j);
        c[j] = own[j] = 0;
        if (bin >= 0) {
          const uint4 x = reinterpret_cast<const uint4 *>(hist)[bin];
          c[j] = WIDE ? __ldcg(sums + bin) : sums[bin];
          own[j] = x.x + x.y + x.z + x.w;
        }
        mine += c[j];
        lmine += own[j];
      }
      unsigned inc = mine, linc = lmine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned y = __shfl_up_sync(full, inc, o), ly = __shfl_up_sync(full, linc, o);
        if (lane >= o) inc += y, linc += ly;
      }
      if (lane == 31) scan[warp] = inc, lscan[warp] = linc;
      __syncthreads();
      unsigned before = inc - mine, lbefore = linc - lmine;
      before += __reduce_add_sync(full, lane < warp && lane < EW ? scan[lane] : 0u);
      lbefore += __reduce_add_sync(full, lane < warp && lane < EW ? lscan[lane] : 0u);
#pragma unroll
      for (int j = 0; j < EPT; ++j) {
        if (before < (unsigned)left && before + c[j] >= (unsigned)left) {
          found[0] = bins - 1 - (EPT * tid + j);
          found[1] = left - before;
          counts[0] = (int)lbefore;          // this CTA's keys above the digit
          counts[1] = (int)own[j];           // and on it
        }
        before += c[j];
        lbefore += own[j];
      }
      __syncthreads();
      border |= found[0] << shift;
      mask |= (uint32_t)(bins - 1) << shift;
      left = (int)found[1];
      na += counts[0];
      ne = counts[1];
      __syncthreads();
    }
  }
  const bool all = s.rest == s.mid;
  const int places = choose ? left : 0;      // border keys kept, lowest index first
  // kept outright: protected keys of this CTA, all competing ones, or those above the border
  auto overlap = [&](int x0, int x1) { return max(0, min(hi, x1) - max(lo, x0)); };
  if (all) na = overlap(m0, m1);
  na += overlap(0, m0) + overlap(m1, s.n);
  if (!choose) ne = 0;
  int above = 0, equal = 0;                  // before the tile at hand
  if (WIDE) {
    int *all_counts = reinterpret_cast<int *>(wide + kWideCounts);
    if (tid == 0) all_counts[2 * rank] = na, all_counts[2 * rank + 1] = ne;
    if (!meet()) return;
    for (int r = lane; r < rank; r += 32) above += __ldcg(all_counts + 2 * r), equal += __ldcg(all_counts + 2 * r + 1);
    above = __reduce_add_sync(full, above);
    equal = __reduce_add_sync(full, equal);
  } else {
    if (tid == 0) counts[0] = na, counts[1] = ne;
    cl.sync();
    for (int r = 0; r < rank; ++r) {
      above += cl.map_shared_rank(counts, r)[0];
      equal += cl.map_shared_rank(counts, r)[1];
    }
  }
  static_assert(EBINS * ECOPY >= ETILE, "a tile's kept keys fit the histograms' place");
  int *list = reinterpret_cast<int *>(hist);
  int32_t *src_row = a.src_row + (long)s.h * a.total_keep + s.d0, *dst_row = a.dst_row + s.d0;
  int32_t *pos_out = a.pos_out ? a.pos_out + (long)s.h * a.dst.rows : nullptr;
  float *w_out = a.w_out ? a.w_out + (long)s.h * a.dst.rows : nullptr;
  for (int t0 = lo; t0 < hi; t0 += ETILE) {
    const int p0 = t0 + warp * 32 * EB;
    uint32_t key[EB];
    load_keys<CACHED>(a, s, p0, hi, lane, cache, lo, key);
    unsigned ba[EB], be[EB];
    int wa = 0, we = 0;
#pragma unroll
    for (int i = 0; i < EB; ++i) {
      const int p = p0 + 32 * i + lane;
      const bool in = p < hi, safe = p < m0 || p >= m1;
      ba[i] = __ballot_sync(full, in && (safe || all || (choose && key[i] > border)));
      be[i] = __ballot_sync(full, in && !safe && choose && key[i] == border);
      wa += __popc(ba[i]);
      we += __popc(be[i]);
    }
    __syncthreads();                         // the previous tile's counts are read
    if (lane == 0) wabove[warp] = wa, wequal[warp] = we;
    __syncthreads();
    const int va = lane < EW ? wabove[lane] : 0, ve = lane < EW ? wequal[lane] : 0;
    int a0 = above + __reduce_add_sync(full, lane < warp ? va : 0);
    int e0 = equal + __reduce_add_sync(full, lane < warp ? ve : 0);
    const int first = above + min(equal, places);
    above += __reduce_add_sync(full, va);
    equal += __reduce_add_sync(full, ve);
    const int kept = above + min(equal, places) - first;      // of this tile
    // the tile's kept keys, in order, into shared memory (the histograms' place) ...
    const unsigned below = (1u << lane) - 1;
    if (wa + we > 0) {                       // the same for the whole warp
#pragma unroll
      for (int i = 0; i < EB; ++i) {
        const int eb = e0 + __popc(be[i] & below);
        if ((ba[i] >> lane & 1) || ((be[i] >> lane & 1) && eb < places))
          list[a0 + __popc(ba[i] & below) + min(eb, places) - first] = p0 + 32 * i + lane;
        a0 += __popc(ba[i]);
        e0 += __popc(be[i]);
      }
    }
    __syncthreads();
    // ... and out from there with every lane at work (few keys of a warp are
    // kept: stores from the ranking itself took 4 us a tile)
    for (int k = tid; k < kept; k += ET) {
      const int p = list[k], j = first + k;
      const int row = a.src.block_table ? (int)a.src.row(s.b, s.k0, p) : s.k0 + p;
      const int dst = a.dst.block_table ? (int)a.dst.row(s.b, s.d0, j) : s.d0 + j;
      if (row < 0 || dst < 0) atomicOr(a.err, kDevErrSeqlens);
      src_row[j] = row;
      if (s.h == 0) dst_row[j] = dst;
      if (dst >= 0) {
        if (pos_out) pos_out[dst] = !a.key_pos ? p : row >= 0 ? __ldg(a.key_pos + (long)s.h * a.src.rows + row) : -1;
        if (w_out) w_out[dst] = row >= 0 ? __ldg(a.weights + (long)s.h * a.src.rows + row) : 0.f;
      }
    }
  }
  if (!WIDE) cl.sync();                      // no CTA leaves while another reads its counts
}

// Copies the kept rows of one plane (blockIdx.y) and head, in units of 16 bytes
// where the plane's rows and addresses allow, else 8, 4 or 1: a CTA takes as
// many rows as give each thread MU units, all in flight together.  The head is
// the fastest block index: the heads of a row share lines.
struct MoveArgs {
  const int32_t *src_row, *dst_row, *cu_keep;
  int batch, total_keep, Hkv;
  long src_rows, dst_rows;
  const uint8_t *from[kMaxPlanes];
  uint8_t *to[kMaxPlanes];
  int bytes[kMaxPlanes], width[kMaxPlanes], rows[kMaxPlanes];         // rows: of a CTA
};

constexpr int MT = 256, MU = 4, MROWS = MT * MU;

template <typename V>
__device__ __forceinline__ void move_rows(const uint8_t *from, uint8_t *to, long pitch, int units, int n, const int *src,
                                          const int *dst) {
  const int total = n * units;
  const int shift = (units & (units - 1)) == 0 ? 31 - __clz(units) : -1;
  for (int i0 = threadIdx.x; i0 < total; i0 += MT * MU) {
    V v[MU];
    long o[MU];
#pragma unroll
    for (int k = 0; k < MU; ++k) {
      const int i = i0 + k * MT;
      o[k] = -1;
      if (i >= total) continue;
      const int j = shift >= 0 ? i >> shift : i / units, off = (i - j * units) * (int)sizeof(V);
      if (src[j] < 0) continue;
      v[k] = __ldg(reinterpret_cast<const V *>(from + src[j] * pitch + off));
      o[k] = dst[j] * pitch + off;
    }
#pragma unroll
    for (int k = 0; k < MU; ++k)
      if (o[k] >= 0) *reinterpret_cast<V *>(to + o[k]) = v[k];
  }
}

__global__ void __launch_bounds__(MT) relattn_evict_move_kernel(const __grid_constant__ MoveArgs a) {
  __shared__ int src[MROWS], dst[MROWS];
  const int pl = blockIdx.y, rows = a.rows[pl];
  const int h = blockIdx.x % a.Hkv;
  const long j0 = (long)(blockIdx.x / a.Hkv) * rows;
  if (j0 >= a.total_keep) return;
  const int n = (int)min((long)rows, a.total_keep - j0);
  const int used0 = __ldg(a.cu_keep), used1 = __ldg(a.cu_keep + a.batch);
  for (int i = threadIdx.x; i < n; i += MT) {
    const int j = (int)j0 + i;
    int s = __ldg(a.src_row + (long)h * a.total_keep + j), d = __ldg(a.dst_row + j);
    if (j < used0 || j >= used1 || d < 0 || s >= a.src_rows || d >= a.dst_rows) s = -1;   // a row of no sequence
    src[i] = s;
    dst[i] = d;
  }
  __syncthreads();
  const int bytes = a.bytes[pl], width = a.width[pl];
  const uint8_t *from = a.from[pl] + (long)h * bytes;
  uint8_t *to = a.to[pl] + (long)h * bytes;
  const long pitch = (long)a.Hkv * bytes;
  if (width == 16) move_rows<uint4>(from, to, pitch, bytes / 16, n, src, dst);
  else if (width == 8) move_rows<uint2>(from, to, pitch, bytes / 8, n, src, dst);
  else if (width == 4) move_rows<unsigned>(from, to, pitch, bytes / 4, n, src, dst);
  else move_rows<unsigned char>(from, to, pitch, bytes, n, src, dst);
}

template <int ET, bool CACHED, bool WIDE>
cudaError_t launch_select(const EvictArgs &a, long units, int cs, int smem, cudaStream_t stream) {
  auto *kernel = relattn_evict_select_kernel<ET, CACHED, WIDE>;
  static std::atomic<bool> done[kMaxDevicesAttr], wide[kMaxDevicesAttr];
  if (CACHED) {
    const cudaError_t e = set_max_smem_once(reinterpret_cast<const void *>(kernel), kCacheKeys * 4, done);
    if (e != cudaSuccess) return e;
  }
  if (!WIDE && cs > 8) {
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevicesAttr) return cudaErrorInvalidDevice;
    if (!wide[dev].load(std::memory_order_acquire)) {
      const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
      if (e != cudaSuccess) return e;
      wide[dev].store(true, std::memory_order_release);
    }
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(units * cs));
  cfg.blockDim = dim3(ET);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  if (WIDE) {
    attr.id = cudaLaunchAttributeCooperative;          // its CTAs wait for one another
    attr.val.cooperative = 1;
  } else {
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = cs;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
  }
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace

// Few long sequences: clusters would leave most SMs idle, so all of them work
// on the selection, in a cooperative launch, and meet in global memory.
// Measured (us, this / clusters, of the whole call with half of the keys kept
// and one plane of 8 bytes): one head of 8 thousand keys 44 / 36, of 33 thousand 42 /
// 46, of a million 52 / 106; eight heads of 33 thousand 36 / 46, of a million 120 /
// 214.
size_t evict_wide_bytes(int batch, int Hkv, int max_k) {
  const long units = (long)batch * Hkv;
  return units <= kWideUnits && max_k >= kWideKeys ? (size_t)units * kWideWords * sizeof(unsigned) : 0;
}

cudaError_t clear_evicted(const EvictArgs &a, cudaStream_t stream) {
  const size_t bytes = (size_t)a.Hkv * a.dst.rows * 4;
  if (bytes == 0) return cudaSuccess;
  if (a.w_out) {
    const cudaError_t e = cudaMemsetAsync(a.w_out, 0, bytes, stream);
    if (e != cudaSuccess) return e;
  }
  return a.pos_out ? cudaMemsetAsync(a.pos_out, 0xff, bytes, stream) : cudaSuccess;
}

cudaError_t launch_evict(const EvictArgs &args, cudaStream_t stream) {
  EvictArgs a = args;
  if (a.clear) {
    const cudaError_t e = clear_evicted(a, stream);
    if (e != cudaSuccess) return e;
  }
  // CTAs per (sequence, kv head): one per 16K keys, up to 16; of 512 threads
  // while 16K keys are enough, else of 1024
  int cs = 1;
  while (cs < kMaxCluster && a.max_k > cs * 16384) cs *= 2;
  const long units = (long)a.batch * a.Hkv;   // (the host keeps units x kMaxCluster below 2^31)
  const long chunk = ((a.max_k + cs - 1) / cs + 31) & ~31L;
  cudaError_t e;
  if (a.wide) {
    a.ctas = std::min(kWideCtas, a.sms / (int)units);
    const long own = ((a.max_k + a.ctas - 1) / a.ctas + 31) & ~31L;
    e = cudaMemsetAsync(a.wide, 0, (size_t)units * kWideWords * sizeof(unsigned), stream);
    if (e != cudaSuccess) return e;
    e = own <= kCacheKeys ? launch_select<1024, true, true>(a, units, a.ctas, (int)own * 4, stream)
                          : launch_select<1024, false, true>(a, units, a.ctas, 0, stream);
  } else {
    e = chunk <= 16384       ? launch_select<512, true, false>(a, units, cs, (int)chunk * 4, stream)
        : chunk <= kCacheKeys ? launch_select<1024, true, false>(a, units, cs, (int)chunk * 4, stream)
                              : launch_select<1024, false, false>(a, units, cs, 0, stream);
  }
  if (e != cudaSuccess) return e;
  if (a.planes == 0 || a.total_keep == 0) return cudaSuccess;
  MoveArgs m = {};
  m.src_row = a.src_row;
  m.dst_row = a.dst_row;
  m.cu_keep = a.cu_keep;
  m.batch = a.batch;
  m.total_keep = a.total_keep;
  m.Hkv = a.Hkv;
  m.src_rows = a.src.rows;
  m.dst_rows = a.dst.rows;
  long grid = 0;
  for (int i = 0; i < a.planes; ++i) {
    m.from[i] = static_cast<const uint8_t *>(a.from[i]);
    m.to[i] = static_cast<uint8_t *>(a.to[i]);
    m.bytes[i] = a.bytes[i];
    const uintptr_t bits = reinterpret_cast<uintptr_t>(a.from[i]) | reinterpret_cast<uintptr_t>(a.to[i]) | (uintptr_t)a.bytes[i];
    m.width[i] = !(bits & 15) ? 16 : !(bits & 7) ? 8 : !(bits & 3) ? 4 : 1;
    const int units = a.bytes[i] / m.width[i];
    m.rows[i] = std::max(16, std::min(MROWS, MROWS / units));
    grid = std::max(grid, ((long)a.total_keep + m.rows[i] - 1) / m.rows[i] * a.Hkv);
  }
  if (grid > 0x7fffffffL) return cudaErrorInvalidValue;
  relattn_evict_move_kernel<<<dim3((unsigned)grid, (unsigned)a.planes), MT, 0, stream>>>(m);
  return cudaGetLastError();
}

}  // namespace relattn

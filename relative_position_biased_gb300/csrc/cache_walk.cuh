// cache_walk.cuh -- what the kernels that stream a K / V cache in warps of 32
// keys share: the sequences' rows, the order in which tiles are walked, and
// where a key's cache row lies.
#pragma once

#include "nvfp4.cuh"

namespace relattn {

struct Unit {
  SeqRows s;
  int b, h, rb;
  int qbase;       // position of the sequence's first query row
  int lo;          // first key, a multiple of 32
  int nrows;       // query rows of the block (<= 0: none)
};

// The sequence's rows and lengths; lo / tiles of its units.  Zero tiles where
// there is nothing to do or the lengths are inconsistent.
__device__ __forceinline__ int unit_tiles(const WalkArgs &p, int b, SeqRows *sp, int *lo) {
  const SeqRows s = seq_rows(p.a.cu_q, p.a.cu_k, b, p.a.total_q, p.pages);
  *sp = s;
  *lo = 0;
  if (!s.ok || s.lq > p.a.max_q || s.lk > p.a.max_k || first_query_pos(s, p.q_pos, b) < 0) return -1;
  if (s.lq == 0 && !p.idle) return 0;
  if (p.a.window > 0 && !p.key_pos) *lo = max(0, s.lk - s.lq - p.a.window + 1) & ~31;
  const int tile = kWalkTile / p.hp;
  return (s.lk - *lo + tile - 1) / tile;
}

// Tiles before the first one that meets the bias band, where those count more
// (band_extra > 0).
__device__ __forceinline__ int plain_tiles(const WalkArgs &p, const SeqRows &s, int lo, int tiles) {
  if (p.band_extra == 0 || s.lq == 0) return tiles;
  const int first = s.lk - s.lq - p.a.E + 1 - lo;       // the first key of the band, from lo
  return min(max(first, 0) / (kWalkTile / p.hp), tiles);
}

// A unit's tiles with their weights: a tile of the band counts 1 + band_extra
// times and belongs to the range that holds its first.
struct Weighted {
  int plain, extra, total;
  __device__ __forceinline__ int tile(int v) const { return v <= plain ? v : plain + (v - plain + extra) / (extra + 1); }
};
__device__ __forceinline__ Weighted weighted_tiles(const WalkArgs &p, const SeqRows &s, int lo, int tiles) {
  const int plain = plain_tiles(p, s, lo, tiles);
  return {plain, p.band_extra, tiles + p.band_extra * (tiles - plain)};
}

// Row n of the unit's block: its index among all (token, head) rows, and token.
__device__ __forceinline__ long unit_row(const WalkArgs &p, const Unit &u, int n, int *tok) {
  const int rr = u.rb * kFp4Rows + n;
  *tok = rr / p.a.group;
  return (long)(u.s.q0 + *tok) * p.a.Hq + u.h * p.a.group + (rr - *tok * p.a.group);
}

// First cache row of 32 keys from key0 (they share a page), -1 outside the cache.
__device__ __forceinline__ long group_row(const WalkArgs &p, const Unit &u, int key0) {
  if (key0 >= u.s.lk) return -1;
  const long r = p.pages.row(u.b, u.s.k0, key0);
  if (r < 0) atomicOr(p.a.err, kDevErrSeqlens);
  return r;
}

// Last i in [0, n) with v[i] <= x (0 if none): the sequence that holds x when v
// is its running start.
__device__ __forceinline__ int last_not_above(const int *v, int n, int x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (v[mid] <= x) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Sums of tile counts stop at kTooMany: cu_seqlens in order hold fewer than 2^31
// keys, 2^27 weighted tiles.  Lengths that each pass the checks may be more
// together (entries out of order, pages listed twice), and an int would overflow.
constexpr int kTooMany = 1 << 30;
__device__ __forceinline__ int add_tiles(int a, int b) { return (int)min((unsigned)a + (unsigned)b, (unsigned)kTooMany); }

// Running (weighted) tile counts of the sequences into prefix[0 .. batch] (batch <=
// kWalkBatch), by a CTA of THREADS; returns the total.  Inconsistent sequences
// hold no tile and are recorded once; with too many tiles there is nothing to do,
// which is recorded too.
template <int THREADS>
__device__ __forceinline__ int tile_prefix(const WalkArgs &p, int *prefix, int *wsum) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int base = 0;
  for (int b0 = 0; b0 < p.a.batch; b0 += THREADS) {
    const int b = b0 + tid;
    int n = 0;
    if (b < p.a.batch) {
      SeqRows s;
      int lo;
      n = unit_tiles(p, b, &s, &lo);
      if (n < 0) {
        n = 0;
        if (blockIdx.x == 0) atomicOr(p.a.err, kDevErrSeqlens);
      } else {
        n += p.band_extra * (n - plain_tiles(p, s, lo, n));
      }
    }
    int inc = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, inc, o);
      if (lane >= o) inc = add_tiles(inc, y);
    }
    if (lane == 31) wsum[warp] = inc;
    __syncthreads();
    int before = base, all = base;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
      if (w < warp) before = add_tiles(before, wsum[w]);
      all = add_tiles(all, wsum[w]);
    }
    if (b < p.a.batch) prefix[b] = before + inc - n;
    base = all;
    __syncthreads();
  }
  if (base == kTooMany) {
    if (blockIdx.x == 0 && tid == 0) atomicOr(p.a.err, kDevErrSeqlens);
    base = 0;
  }
  if (tid == 0) prefix[p.a.batch] = base;
  __syncthreads();
  return base;
}

// A CTA's way through the tiles of a decode, piece by piece.  The units' tiles
// are laid end to end and cut into ranges of C; CTA c takes ranges [c k, (c + 1) k),
// of at most `most` tiles each where the plan's k allows.  Or (p.whole) the CTA
// has one unit, whose `total` tiles are cut in the same way.
struct Ranges {
  unsigned x, end, C;                        // the next tile, the one past the last, tiles of a range
  __device__ __forceinline__ Ranges(const Fp4DecodeArgs &p, unsigned total, unsigned most) {
    if (p.whole) {
      x = 0, end = total;
      C = max(most, total / (unsigned)p.splits + 1);
      return;
    }
    const unsigned share = max((total + gridDim.x - 1) / gridDim.x, 1u);
    const unsigned k = min((share + most - 1) / most, (unsigned)p.waves);
    C = max((share + k - 1) / k, (unsigned)p.c_min);
    x = (unsigned)min((unsigned long long)blockIdx.x * k * C, (unsigned long long)total);
    end = x + (unsigned)min((unsigned long long)k * C, (unsigned long long)(total - x));
  }
};

// One piece: tiles [t0, t0 + tiles) of its unit (none where a range ends within a
// weighted tile), the slot it fills, and the slots that the unit's pieces use.
struct Piece {
  int t0, tiles, slot, used;
};

// The piece at at.x, which moves on past it.  `place` fills in the unit's head,
// rows and positions from the unit group's number; per: tiles of a unit group.
template <typename F>
__device__ __forceinline__ Piece next_piece(const Fp4DecodeArgs &p, Ranges &at, Unit &u, const int *prefix, unsigned per, F place) {
  Piece c;
  const unsigned left = min(at.end - at.x, at.C - at.x % at.C);      // to the end of the range
  if (p.whole) {
    c = {(int)at.x, (int)left, (int)(at.x / at.C), (int)((at.end - 1) / at.C + 1)};
    at.x += left;
    return c;
  }
  const unsigned hr = at.x / per;
  const int xb = (int)(at.x - hr * per);
  u.b = last_not_above(prefix, p.a.batch, xb);       // it holds tile xb
  const int real = unit_tiles(p, u.b, &u.s, &u.lo), v0 = xb - prefix[u.b];
  const Weighted w = weighted_tiles(p, u.s, u.lo, real);
  const int n = (int)min((unsigned)(w.total - v0), left);
  place((int)hr);
  const unsigned ustart = hr * per + prefix[u.b], first = ustart / at.C;
  c.t0 = w.tile(v0);
  c.tiles = w.tile(v0 + n) - c.t0;
  c.slot = (int)(at.x / at.C - first);
  c.used = (int)((ustart + w.total - 1) / at.C - first) + 1;
  at.x += n;
  return c;
}

__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds_u16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t lds_u8(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}

// Power of two that brings a magnitude to 2^14 .. 2^15 (from its fp32 bits),
// and its inverse: f16, whose last place is 2^-24, then holds a bf16 row (8 bits)
// exactly down to 2^-31 of its largest element, and smaller elements to within
// 2^-39 of it.
__device__ __forceinline__ float f16_row_scale(uint32_t top, float *back) {
  const int e = min(max((int)(top >> 23) - 127, -100), 127);
  *back = __uint_as_float((uint32_t)(e - 14 + 127) << 23);
  return __uint_as_float((uint32_t)(14 - e + 127) << 23);
}

}  // namespace relattn

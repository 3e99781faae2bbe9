// key_weights.cuh -- what the kernels of the key weights share.
#pragma once

#include "cache_walk.cuh"

namespace relattn {

// The bias table (P's columns in falling order of distance): row m holds
// distance origin - m, with kTablePad zero rows on either side of [0, E).
constexpr int kTablePad = 160;
__host__ __device__ __forceinline__ int rel_table_rows(int E) { return E + 2 * kTablePad; }
__host__ __device__ __forceinline__ int rel_table_origin(int E) { return E - 1 + kTablePad; }

// First token (a multiple of 32) that the tcgen05 kernel takes of a key tile:
// with a bias the first whose every distance to the tile's keys is at least E,
// without one the first that may see a key.
__device__ __forceinline__ int tc_first_token(const KeyWeightArgs &p, int qbase, int tile0) {
  if (p.a.E > 0) {
    const long t = (long)tile0 + kWalkTile - 1 + p.a.E - qbase;
    return (int)min((max(t, 0L) + 31) & ~31L, 0x7fffffe0L);
  }
  return max(tile0 - qbase, 0) & ~31;
}

// w_out of key `key` (cache row `row`) with the new weight `sum`.
__device__ __forceinline__ void write_weight(const KeyWeightArgs &p, const Unit &u, int key, long row, float sum) {
  const long at = (long)u.h * p.pages.rows + row;
  if (p.w_in && p.decay != 0.f && key < u.s.lk - u.s.lq) sum = fmaf(p.decay, __ldg(p.w_in + at), sum);
  p.w_out[at] = sum;
}

// The 128 keys from tile0 as bf16 rows: at(key, chunk) is where 8 dims go.  A
// 4-bit value without its head's factor has 6 bits, so bf16 holds it exactly.
// Keys past the sequence or outside the cache are zero.
template <int THREADS, typename F>
__device__ __forceinline__ void load_key_tile(const KeyWeightArgs &p, const Unit &u, int tile0, int tid, F at) {
  constexpr int N = kWalkTile * 8 / THREADS, B = N < 4 ? N : 4;     // 16-dim blocks of a thread, and in flight together
  static_assert(N * THREADS == kWalkTile * 8 && N % B == 0, "whole blocks");
  if (p.k) {
    for (int i0 = 0; i0 < N; i0 += B) {
      uint4 v[B][2];
#pragma unroll
      for (int i = 0; i < B; ++i) {
        const int x = tid + (i0 + i) * THREADS, key = tile0 + (x >> 3);
        const long row = key < u.s.lk ? p.pages.row(u.b, u.s.k0, key) : -1;
        v[i][0] = v[i][1] = make_uint4(0, 0, 0, 0);
        if (row >= 0) {
          const uint4 *src = reinterpret_cast<const uint4 *>(p.k + (row * p.a.Hkv + u.h) * kHeadDim + (x & 7) * 16);
          v[i][0] = __ldg(src), v[i][1] = __ldg(src + 1);
        }
      }
#pragma unroll
      for (int i = 0; i < B; ++i) {
        const int x = tid + (i0 + i) * THREADS;
        *reinterpret_cast<uint4 *>(at(x >> 3, 2 * (x & 7))) = v[i][0];
        *reinterpret_cast<uint4 *>(at(x >> 3, 2 * (x & 7) + 1)) = v[i][1];
      }
    }
    return;
  }
  for (int i0 = 0; i0 < N; i0 += B) {
    uint2 c[B];
    uint32_t sc[B];
#pragma unroll
    for (int i = 0; i < B; ++i) {
      const int x = tid + (i0 + i) * THREADS, key = tile0 + (x >> 3);
      const long row = key < u.s.lk ? p.pages.row(u.b, u.s.k0, key) : -1;
      c[i] = make_uint2(0, 0);
      sc[i] = 0;
      if (row >= 0) {
        const long hb = (row * p.a.Hkv + u.h) * kFp4Blocks + (x & 7);
        c[i] = __ldg(reinterpret_cast<const uint2 *>(p.kv.k + hb * 8));
        sc[i] = __ldg(p.kv.k_scale + hb);
      }
    }
#pragma unroll
    for (int i = 0; i < B; ++i) {
      const int x = tid + (i0 + i) * THREADS;
      const uint32_t s2 = __byte_perm(e4m3x2_to_f16(sc[i]), 0, 0x1010);
      uint32_t w[8];
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        uint32_t f[4];
        e2m1x8_to_f16(y ? c[i].y : c[i].x, f);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t v = hmul2(f[j], s2);
          float lo, hi;
          asm("cvt.f32.f16 %0, %1;" : "=f"(lo) : "h"((uint16_t)(v & 0xffffu)));
          asm("cvt.f32.f16 %0, %1;" : "=f"(hi) : "h"((uint16_t)(v >> 16)));
          w[4 * y + j] = pack_bf16x2(lo, hi);
        }
      }
      *reinterpret_cast<uint4 *>(at(x >> 3, 2 * (x & 7))) = make_uint4(w[0], w[1], w[2], w[3]);
      *reinterpret_cast<uint4 *>(at(x >> 3, 2 * (x & 7) + 1)) = make_uint4(w[4], w[5], w[6], w[7]);
    }
  }
}

}  // namespace relattn

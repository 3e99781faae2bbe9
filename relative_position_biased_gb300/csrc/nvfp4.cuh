// nvfp4.cuh -- the 4-bit cache format and the device helpers that its kernels
// share.  NVFP4: E2M1 codes (sign, two exponent bits, one mantissa bit: 0,
// 0.5, 1, 1.5, 2, 3, 4, 6), one E4M3 scale per 16 consecutive dims and one
// fp32 factor per kv head; value = code * scale * factor.  Two codes per
// byte, the lower dim in the low nibble.  A row of one head is 64 bytes of
// codes and 8 of scales.
#pragma once

#include "launch.h"
#include "mxfp8.cuh"

namespace relattn {

constexpr int kFp4RowBytes = kHeadDim / 2;    // code bytes of a (row, head)
constexpr int kFp4Blocks = kHeadDim / 16;     // scale bytes of a (row, head)

// Sequences up to this many are laid end to end by the walking kernels (their
// table leaves room for four decode CTAs per SM).  Past it a decode takes a CTA
// per unit, and key weights of few rows the tiles kernel.  Measured (384 / 512
// sequences of 512 to 4096 4-bit keys, one row, group 8, two kv heads): decode 123 /
// 168 us, the same rate; key weights 81 / 347, three times as long per key.
constexpr int kWalkBatch = 384;

// Four code bytes (one word, lowest byte first) as four f16 pairs, the low
// nibble of each byte in the low half.  Exact.
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&o)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
      : "r"(w));
}

// Two E4M3 bytes (low half of w) as an f16 pair.  Exact.
__device__ __forceinline__ uint32_t e4m3x2_to_f16(uint32_t w) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)w));
  return r;
}

__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// f16 pair of two floats, round to nearest: lo in the low half.
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// D += A * B, m16n8k16, f16 inputs, fp32 accumulate.
__device__ __forceinline__ void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                              uint32_t a3, uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};\n"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transpose of an 8 x 8 matrix of f16 held one pair a lane.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

// 8-byte async copy global->shared (zero fill, nothing read, when !pred).
__device__ __forceinline__ void cp_async8(uint32_t dst, const void *src, bool pred) {
  const int n = pred ? 8 : 0;
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;\n" ::"r"(dst), "l"(src), "r"(n));
}

// Rows of one sequence as the cache kernels see them; ok only when the
// cu_seqlens entries and lengths agree with the host's sizes.
struct SeqRows {
  int q0, lq, k0, lk;
  bool ok;
};

__device__ __forceinline__ SeqRows seq_rows(const int32_t *cu_q, const int32_t *cu_k, int b, int total_q,
                                            const CachePages &pg) {
  SeqRows s;
  s.q0 = cu_q[b];
  s.k0 = cu_k[b];
  const int q1 = cu_q[b + 1], k1 = cu_k[b + 1];
  s.lq = q1 - s.q0;
  s.lk = k1 - s.k0;
  s.ok = s.q0 >= 0 && s.k0 >= 0 && q1 >= s.q0 && k1 >= s.k0 && s.lk >= s.lq && q1 <= total_q &&
         (pg.block_table ? (long)s.lk <= (long)pg.max_pages * pg.page_size : (long)k1 <= pg.rows);
  return s;
}

// Position of the first query row of sequence b; -1 where q_pos is out of range.
__device__ __forceinline__ int first_query_pos(const SeqRows &s, const int32_t *q_pos, int b) {
  if (!q_pos) return s.lk - s.lq;
  const int p = __ldg(q_pos + b);
  return p >= 0 && p <= 0x7fffffff - s.lq ? p : -1;
}

}  // namespace relattn

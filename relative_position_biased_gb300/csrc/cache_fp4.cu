// cache_fp4.cu -- rows into and out of the 4-bit (NVFP4) K / V cache.
//
// The K / V rows of a chunk (the tail of every sequence) are quantised into
// the cache rows that the attention reads, contiguous or paged, or read back
// as bf16.  With t = x / factor (one fp32 rounding) the scale of 16 dims is
// E4M3(max |t| / 6), nearest, ties to even, at most 448, and each code is the
// E2M1 value nearest to t / scale, ties to even, at most 6.  Both are the
// roundings of the exact quotients: a border between two codes times the
// divisor has at most 7 bits, so a dividend that is not exactly on it is at
// least 2^-24 of it away, and the correctly rounded fp32 quotient then never
// lands on the border by rounding.
//
// Division.  16 elements share a divisor, so each quotient is made from the
// divisor's correctly rounded reciprocal and one residual step (Markstein's
// theorem: with y = RN(1/b), q = RN(a y) and the exact residual r = a - b q, RN(q
// + r y) is the correctly rounded a / b): three operations, where the divide
// function takes about ten (store and load of 4 x 8192 x 2 rows: 38 -> 28 us).
// Outside the range where residuals are exact, and for infinities, the divide
// function is called.
//
// No pipe is full: the store takes 15.6 us of those 28 with its issue slots 66 %
// busy and DRAM 27 %, the load 14.3 with 42 and 8 %.  Each thread searches its row's
// sequence and page itself and then waits for small loads (in all, 4 and 8 cycles an
// instruction).
//
// One thread takes 16 dims of K and of V: 32 bytes of bf16 on one side, 8 bytes
// of codes and a scale byte on the other, so a warp touches 1 KB and 256 + 32
// bytes without gaps.
#include "nvfp4.cuh"

namespace relattn {
namespace {

constexpr int kRowThreads = 256;

// a / b for a shared b: y = RN(1 / b), `plain` when the short form does not hold.
struct Divisor {
  float b, y;
  bool plain;
  // top: the largest |a|
  __device__ __forceinline__ Divisor(float b_, float top) : b(b_) {
    y = __frcp_rn(b);
    plain = !(b > 0x1p-60f && b < 0x1p60f && top < 0x1p60f);
  }
  // (Elements below 2^-60 may lose residual bits to underflow: they are far
  // below every border, the smallest being 2^-12.  The residual is taken as b q -
  // a: of a -0 it is +0, and -0 y - 0 stays -0; a - b q would end as +0.)
  __device__ __forceinline__ float quick(float a) const {
    const float q = __fmul_rn(a, y);
    return __fmaf_rn(-__fmaf_rn(q, b, -a), y, q);
  }
  __device__ __forceinline__ void operator()(float (&x)[16], float &top) const {
    if (!plain) {
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = quick(x[i]);
      top = quick(top);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = __fdiv_rn(x[i], b);
      top = __fdiv_rn(top, b);
    }
  }
};

// sequence of chunk row t: the last b with cu_q[b] <= t
__device__ __forceinline__ int find_seq(const int32_t *cu_q, int batch, int t) {
  int lo = 0, hi = batch;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(cu_q + mid) <= t) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Cache row of chunk row t; false when t belongs to no sequence (left alone).
__device__ __forceinline__ bool place_row(const Fp4RowArgs &a, int t, long *row) {
  const int b = find_seq(a.cu_q, a.batch, t);
  const SeqRows s = seq_rows(a.cu_q, a.cu_k, b, a.total_q, a.pages);
  if (t < s.q0 || t >= s.q0 + s.lq) {
    if (!s.ok) atomicOr(a.err, kDevErrSeqlens);
    return false;                 // behind the last sequence, or inconsistent
  }
  if (!s.ok) {
    atomicOr(a.err, kDevErrSeqlens);
    return false;
  }
  *row = a.pages.row(b, s.k0, s.lk - s.lq + (t - s.q0));
  if (*row < 0) atomicOr(a.err, kDevErrSeqlens);
  return true;
}

// What a thread takes of a call: block hb of a (row, head) grid of per_row.
// (32-bit: 2^32 blocks of K and V alone would fill the device's memory; the
// host refuses more.)
struct BlockPlace {
  unsigned t, hb;
  int h;
  __device__ __forceinline__ BlockPlace(int Hkv) {
    const unsigned idx = blockIdx.x * kRowThreads + threadIdx.x, per_row = Hkv * kFp4Blocks;
    t = idx / per_row;
    hb = idx - t * per_row;
    h = hb / kFp4Blocks;
  }
};

__device__ __forceinline__ void store_block(const uint4 *src, const float *gp, int h, uint8_t *codes_at, uint8_t *scale_at) {
  const float g = gp ? __ldg(gp + h) : 1.f;
  const uint4 w0 = __ldg(src), w1 = __ldg(src + 1);
  const uint32_t ws[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
  float x[16];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[2 * i] = __uint_as_float(ws[i] << 16);
    x[2 * i + 1] = __uint_as_float(ws[i] & 0xffff0000u);
    // largest magnitude as bits: a NaN is larger than every number
    top = max(top, max((ws[i] << 16) & 0x7fff0000u, ws[i] & 0x7fff0000u));
  }
  float amax = __uint_as_float(top);
  if (gp) Divisor(g, amax)(x, amax);
  const uint32_t sb = e4m3x2(0.f, __fdiv_rn(amax, 6.f)) & 0xffu;
  const uint32_t sh = e4m3x2_to_f16(sb);
  float s;
  asm("cvt.f32.f16 %0, %1;" : "=f"(s) : "h"((uint16_t)sh));
  uint32_t codes[2] = {0, 0};
  if (s > 0.f) {
    Divisor(s, amax)(x, amax);
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
      uint32_t c;
      asm("{\n\t.reg .b8 c;\n\tcvt.rn.satfinite.e2m1x2.f32 c, %1, %2;\n\tmov.b32 %0, {c, 0, 0, 0};\n\t}"
          : "=r"(c) : "f"(x[i + 1]), "f"(x[i]));
      codes[i / 8] |= c << (4 * (i & 7));
    }
  }
  *reinterpret_cast<uint2 *>(codes_at) = make_uint2(codes[0], codes[1]);
  *scale_at = (uint8_t)sb;
}

__global__ void __launch_bounds__(kRowThreads) relattn_store_fp4_kernel(const __grid_constant__ Fp4RowArgs a) {
  const BlockPlace x(a.Hkv);
  if (x.t >= (unsigned)a.total_q) return;
  long row;
  if (!place_row(a, (int)x.t, &row) || row < 0) return;
  const long per_row = a.Hkv * kFp4Blocks, from = ((long)x.t * per_row + x.hb) * 16, to = row * per_row + x.hb;
  store_block(reinterpret_cast<const uint4 *>(a.k + from), a.kv.k_global, x.h, const_cast<uint8_t *>(a.kv.k) + to * 8,
              const_cast<uint8_t *>(a.kv.k_scale) + to);
  store_block(reinterpret_cast<const uint4 *>(a.v + from), a.kv.v_global, x.h, const_cast<uint8_t *>(a.kv.v) + to * 8,
              const_cast<uint8_t *>(a.kv.v_scale) + to);
}

__device__ __forceinline__ void load_block(uint2 c, uint32_t sb, const float *gp, int h, uint4 *dst) {
  const float g = gp ? __ldg(gp + h) : 1.f;
  const uint32_t sh = e4m3x2_to_f16(sb);
  float s;
  asm("cvt.f32.f16 %0, %1;" : "=f"(s) : "h"((uint16_t)sh));
  uint32_t o[8];
#pragma unroll
  for (int w = 0; w < 2; ++w) {
    uint32_t f[4];
    e2m1x8_to_f16(w ? c.y : c.x, f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float lo, hi;
      asm("cvt.f32.f16 %0, %1;" : "=f"(lo) : "h"((uint16_t)(f[i] & 0xffffu)));
      asm("cvt.f32.f16 %0, %1;" : "=f"(hi) : "h"((uint16_t)(f[i] >> 16)));
      // code * scale is exact (6 bits); one fp32 product, then the bf16 rounding
      o[4 * w + i] = pack_bf16x2(lo * s * g, hi * s * g);
    }
  }
  dst[0] = make_uint4(o[0], o[1], o[2], o[3]);
  dst[1] = make_uint4(o[4], o[5], o[6], o[7]);
}

__global__ void __launch_bounds__(kRowThreads) relattn_load_fp4_kernel(const __grid_constant__ Fp4RowArgs a) {
  const BlockPlace x(a.Hkv);
  if (x.t >= (unsigned)a.total_q) return;
  long row;
  if (!place_row(a, (int)x.t, &row)) return;
  const long per_row = a.Hkv * kFp4Blocks, to = ((long)x.t * per_row + x.hb) * 16, from = row * per_row + x.hb;
  uint2 ck = make_uint2(0, 0), cv = ck;
  uint32_t sk = 0, sv = 0;
  if (row >= 0) {                 // a row outside the cache reads as zero
    ck = __ldg(reinterpret_cast<const uint2 *>(a.kv.k + from * 8));
    cv = __ldg(reinterpret_cast<const uint2 *>(a.kv.v + from * 8));
    sk = __ldg(a.kv.k_scale + from);
    sv = __ldg(a.kv.v_scale + from);
  }
  load_block(ck, sk, a.kv.k_global, x.h, reinterpret_cast<uint4 *>(const_cast<__nv_bfloat16 *>(a.k) + to));
  load_block(cv, sv, a.kv.v_global, x.h, reinterpret_cast<uint4 *>(const_cast<__nv_bfloat16 *>(a.v) + to));
}

cudaError_t row_grid(const Fp4RowArgs &a, dim3 *grid) {
  const unsigned long n = (unsigned long)a.total_q * a.Hkv * kFp4Blocks;
  if (n > 0xffffffffUL - kRowThreads) return cudaErrorInvalidValue;
  *grid = dim3((unsigned)((n + kRowThreads - 1) / kRowThreads));
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_store_fp4(const Fp4RowArgs &a, cudaStream_t stream) {
  dim3 grid;
  const cudaError_t e = row_grid(a, &grid);
  if (e != cudaSuccess) return e;
  relattn_store_fp4_kernel<<<grid, kRowThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_load_fp4(const Fp4RowArgs &a, cudaStream_t stream) {
  dim3 grid;
  const cudaError_t e = row_grid(a, &grid);
  if (e != cudaSuccess) return e;
  relattn_load_fp4_kernel<<<grid, kRowThreads, 0, stream>>>(a);
  return cudaGetLastError();
}

}  // namespace relattn

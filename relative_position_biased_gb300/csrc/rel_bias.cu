// rel_bias.cu -- R = r . P for query rows and distances, in the workspace of a
// kernel that gathers its relative bias by distance (the 4-bit decode, the
// key weights): rel_logits(t, h, d) = r_{t,h} . P[:, d] of the page "SGLang
// and Miles Add Day-0 Support for Inkling", section "Attention with Relative
// Positional Embedding".
//
// A [rows, r_dim] x [r_dim, E] product with r_dim <= 64: what it writes (4
// bytes a value) is many times what it reads, so it is bound by that and, at a
// decode step's sizes, by its launch (1024 rows x 1024 distances: 7 us).  A CTA
// takes 64 rows x 128 distances, a warp 16 rows; both operands are staged in
// shared memory, zero past r_dim, the rows and E, with 16-byte loads where the
// addresses allow and 2-byte ones elsewhere.
#include "launch.h"

namespace relattn {
namespace {

constexpr int RB_ROWS = 64, RB_DIST = 128, RB_THREADS = 128;
constexpr int RB_RS = 64 + 8, RB_PS = RB_DIST + 8;   // padded row lengths (elements)

__global__ void __launch_bounds__(RB_THREADS)
relattn_rel_bias_kernel(const __nv_bfloat16 *__restrict__ r, const __nv_bfloat16 *__restrict__ P, long rows,
                        int rd, int E, float *__restrict__ R) {
  asm volatile("griddepcontrol.launch_dependents;");
  __shared__ __align__(16) __nv_bfloat16 rs[RB_ROWS * RB_RS];
  __shared__ __align__(16) __nv_bfloat16 ps[64 * RB_PS];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long row0 = (long)blockIdx.x * RB_ROWS;
  const int rd_pad = (rd + 15) & ~15;
  const __nv_bfloat16 zero = __float2bfloat16_rn(0.f);
  if ((rd & 7) == 0 && (reinterpret_cast<uintptr_t>(r) & 15u) == 0) {
    const int cpr = rd_pad / 8;
    for (int i = tid; i < RB_ROWS * cpr; i += RB_THREADS) {
      const int y = i / cpr, c = (i - y * cpr) * 8;
      uint4 v = make_uint4(0, 0, 0, 0);
      if (row0 + y < rows && c < rd) v = *reinterpret_cast<const uint4 *>(r + (row0 + y) * rd + c);
      *reinterpret_cast<uint4 *>(rs + y * RB_RS + c) = v;
    }
  } else {
    for (int i = tid; i < RB_ROWS * rd_pad; i += RB_THREADS) {
      const int y = i / rd_pad, c = i - y * rd_pad;
      rs[y * RB_RS + c] = row0 + y < rows && c < rd ? r[(row0 + y) * rd + c] : zero;
    }
  }
  const bool p_vec = (E & 7) == 0 && (reinterpret_cast<uintptr_t>(P) & 15u) == 0;
  const int g = lane >> 2, t = lane & 3;
  for (int d0 = blockIdx.y * RB_DIST; d0 < E; d0 += gridDim.y * RB_DIST) {
    __syncthreads();                         // the previous slice of P is read
    if (p_vec) {
      for (int i = tid; i < rd_pad * (RB_DIST / 8); i += RB_THREADS) {
        const int c = i / (RB_DIST / 8), x = (i % (RB_DIST / 8)) * 8;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (c < rd && d0 + x < E) v = *reinterpret_cast<const uint4 *>(P + (size_t)c * E + d0 + x);
        *reinterpret_cast<uint4 *>(ps + c * RB_PS + x) = v;
      }
    } else {
      for (int i = tid; i < rd_pad * RB_DIST; i += RB_THREADS) {
        const int c = i / RB_DIST, x = i % RB_DIST;
        ps[c * RB_PS + x] = c < rd && d0 + x < E ? P[(size_t)c * E + d0 + x] : zero;
      }
    }
    __syncthreads();
    float acc[16][4];
#pragma unroll
    for (int n = 0; n < 16; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
    for (int kk = 0; kk < rd_pad; kk += 16) {
      const int srow = (lane & 7) + (((lane >> 3) & 1) << 3), scol = (lane >> 4) << 3;
      uint32_t a0, a1, a2, a3;
      ldsm_x4(smem_addr(rs + (warp * 16 + srow) * RB_RS + kk + scol), a0, a1, a2, a3);
#pragma unroll
      for (int n = 0; n < 8; ++n) {
        uint32_t b0, b1, b2, b3;
        ldsm_x4_t(smem_addr(ps + (kk + srow) * RB_PS + n * 16 + scol), b0, b1, b2, b3);
        mma_bf16_16816(acc[2 * n], a0, a1, a2, a3, b0, b1);
        mma_bf16_16816(acc[2 * n + 1], a0, a1, a2, a3, b2, b3);
      }
    }
    const bool even = (E & 1) == 0;          // float2 stores stay aligned
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      const long row = row0 + warp * 16 + g + 8 * half;
      if (row >= rows) continue;
      float *dst = R + row * E;
#pragma unroll
      for (int n = 0; n < 16; ++n) {
        const int d = d0 + n * 8 + 2 * t;
        const float x = acc[n][2 * half], y = acc[n][2 * half + 1];
        if (even && d + 1 < E) {
          *reinterpret_cast<float2 *>(dst + d) = make_float2(x, y);
        } else {
          if (d < E) dst[d] = x;
          if (d + 1 < E) dst[d + 1] = y;
        }
      }
    }
  }
}

}  // namespace

cudaError_t launch_rel_bias(const __nv_bfloat16 *r, const __nv_bfloat16 *P, long rows, int r_dim, int E,
                            float *R, cudaStream_t stream) {
  const long gx = (rows + RB_ROWS - 1) / RB_ROWS;
  if (gx > 0x7fffffffL) return cudaErrorInvalidValue;
  // few rows: the distances spread over CTAs too; many rows: a CTA walks them
  const int slices = (E + RB_DIST - 1) / RB_DIST;
  const dim3 grid((unsigned)gx, (unsigned)(gx >= 2048 ? 1 : slices < 1024 ? slices : 1024));
  relattn_rel_bias_kernel<<<grid, RB_THREADS, 0, stream>>>(r, P, rows, r_dim, E, R);
  return cudaGetLastError();
}

}  // namespace relattn

#include "launch.h"

namespace relattn {
namespace {

// out / lse of a row from its partials: lse = ln sum exp(lse_s), out = sum
// exp(lse_s - lse) o_s.  RW warps per (token, head) take the slots in turn; a slot
// without keys holds lse = -inf and is not read further.  Rows of no sequence,
// or of one whose lengths the kernels refused, are left as they are.
template <int RW>
__global__ void __launch_bounds__(256) relattn_extend_combine_kernel(const __grid_constant__ KernelArgs a, int slots) {
  __shared__ float red_z[8];
  __shared__ float4 red_o[8][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, wi = warp % RW;
  const long rows = (long)a.total_q * a.Hq, row = (long)blockIdx.x * (8 / RW) + warp / RW;
  const int t = (int)(min(row, rows - 1) / a.Hq), h = (int)(row - (long)t * a.Hq);
  int lo = 0, hi = a.batch - 1;                  // the sequence that holds token t
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.cu_q[mid] <= t) lo = mid;
    else hi = mid - 1;
  }
  const int cq = a.cu_q[lo], ck = a.cu_k[lo], Lq = a.cu_q[lo + 1] - cq, Lk = a.cu_k[lo + 1] - ck;
  const bool mine = row < rows && t >= cq && t < cq + Lq && Lk >= Lq && Lq <= a.max_q && Lk <= a.max_k &&
                    extend_rows_ok(a, cq, Lq, ck, Lk);
  // launched as a programmatic dependent: the partials are visible from here on
  asm volatile("griddepcontrol.wait;" ::: "memory");
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float m = -INFINITY, z = 0.f;
  if (mine) {
    for (int s = lane; s < slots; s += 32) m = fmaxf(m, a.lse_part[(long)s * rows + row]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
#pragma unroll 4
    for (int s = wi; s < slots; s += RW) {
      const float ls = a.lse_part[(long)s * rows + row];
      if (ls == -INFINITY) continue;
      const float4 v = *reinterpret_cast<const float4 *>(a.o_part + ((long)s * rows + row) * kHeadDim + lane * 4);
      const float w = exp2f((ls - m) * kLog2e);
      z += w;
      acc.x = fmaf(w, v.x, acc.x);
      acc.y = fmaf(w, v.y, acc.y);
      acc.z = fmaf(w, v.z, acc.z);
      acc.w = fmaf(w, v.w, acc.w);
    }
  }
  if (RW > 1) {
    red_o[warp][lane] = acc;
    if (lane == 0) red_z[warp] = z;
    __syncthreads();
    if (wi != 0) return;
#pragma unroll
    for (int i = 1; i < RW; ++i) {
      const float4 o = red_o[warp + i][lane];
      acc.x += o.x, acc.y += o.y, acc.z += o.z, acc.w += o.w;
      z += red_z[warp + i];
    }
  }
  if (!mine) return;
  const float inv = z == 0.f ? 0.f : 1.f / z;    // (a NaN sum stays one)
  uint2 packed;
  packed.x = pack_bf16x2(acc.x * inv, acc.y * inv);
  packed.y = pack_bf16x2(acc.z * inv, acc.w * inv);
  *reinterpret_cast<uint2 *>(a.out + row * kHeadDim + lane * 4) = packed;
  if (lane == 0) a.lse[(long)h * a.total_q + t] = z == 0.f ? -INFINITY : m + logf(z);
}

}  // namespace

cudaError_t launch_extend_combine(const KernelArgs &a, int slots, bool pdl, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  const bool wide = slots >= 16;                 // (few rows then: more loads of one in flight)
  cfg.gridDim = dim3((unsigned)(wide ? (long)a.total_q * a.Hq : ((long)a.total_q * a.Hq + 7) / 8));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return wide ? cudaLaunchKernelEx(&cfg, relattn_extend_combine_kernel<8>, a, slots)
              : cudaLaunchKernelEx(&cfg, relattn_extend_combine_kernel<1>, a, slots);
}

}  // namespace relattn

// bwd_sink.cu -- what the sinks of a sliding window add to the gradients.
//
// With a window W that keeps the first S keys, a row at position i sees the
// keys 0 <= i - j < W and, besides, the keys j < S with i - j >= W.  The two
// sets are disjoint and every gradient is a sum over the keys (or rows) that
// meet, so the kernels of bwd_mma.cu and bwd_tc.cu compute the window's part as
// they do without sinks, and this file the rest:
//     p = exp(l(i,j) - lse_i),  dl = p (dout_i . v_j - D_i),
//     dq_i += s_i alpha sum_j dl k_j,        dk_j += sum_i s_i alpha dl q_i,
//     dv_j += sum_i p dout_i,                dr_i += s_i sum_j dl P[:, i-j]
// (the last where i - j < E, which needs E > W).  Everything here stays fp32 and
// is added before the results' one rounding to bf16.
//
// What bounds it: every row past the window is read (q, dout: 512 bytes) and its
// dq part written (512 bytes), for 16 keys' five products: HBM (once for every 16
// sinks: beyond them dq and dr are read and added to as well).  4 x 8192 tokens of
// 16 heads, window 4096: 67 us for 268 MB, 4.0 TB/s (the sums 5 us); few rows are a
// chain of loads instead: 5 sequences of 90 to 1500 tokens of 8 heads take 20.  A warp takes 16
// rows (token, head of the group) at a time against 16 keys, in m16n8k16
// instructions; its rows come through a two-stage ring of its own; dk and dv of
// the 16 keys stay in its registers over all its rows.  P and dS are turned for
// dk and dv in registers (movmatrix).  The sums of the CTAs go to slots that a
// second kernel adds in order: no atomics, the same result every time.
#include <algorithm>

#include "launch.h"
#include "nvfp4.cuh"

namespace relattn {
namespace {

constexpr int SW = 8, ST = SW * 32;        // warps, threads
constexpr int SK = 16;                     // keys of a block
// (token, head) rows of a CTA: 1024 where that leaves two CTAs an SM and more, else
// fewer, down to one pass of the warps.  Each CTA's partial costs 16 KB: 4 x 8192
// tokens 67 us with 1024 rows, 112 with 128; 5 sequences of 90 - 1500 67 and 20.
constexpr int kRowsMax = 1024, kRowsMin = 16 * SW;
constexpr int kSinkRing = 2;
constexpr int STAGE = 2 * 16 * 256;        // a warp's 16 rows of q and dout
constexpr int OFF_K = 0, OFF_V = SK * 256, OFF_RING = 2 * SK * 256;
constexpr int PS_ROW = 66;                 // bf16 of a distance of a warp's P slice (33 words: no bank conflicts)
constexpr int PS_BYTES = 32 * PS_ROW * 2;
constexpr int OFF_PS = OFF_RING + SW * kSinkRing * STAGE;
constexpr int SMEM = OFF_PS + SW * PS_BYTES;
constexpr int PART = 2 * SK * kHeadDim;    // floats of a slot
static_assert(SW * 64 * 32 * 4 <= SW * kSinkRing * STAGE, "the merge reuses the ring");

__device__ __forceinline__ uint32_t swz(int row, int c) { return row * 256 + ((c ^ (row & 7)) << 4); }

struct SinkRows {
  int cq, Lq, ck, Lk, t0, n;               // first token with a sink outside its window, (token, head) rows from it
  bool ok;
};
__device__ __forceinline__ SinkRows sink_rows(const BwdArgs &a, int b) {
  SinkRows s;
  s.cq = a.cu_q[b], s.ck = a.cu_k[b];
  s.Lq = a.cu_q[b + 1] - s.cq, s.Lk = a.cu_k[b + 1] - s.ck;
  s.ok = s.Lq >= 0 && s.Lk >= s.Lq && s.Lq <= a.max_q && s.Lk <= a.max_k && s.cq >= 0 && s.cq + (long)s.Lq <= a.total_q &&
         s.ck >= 0 && s.ck + (long)s.Lk <= a.total_k;
  s.t0 = max(0, a.window - (s.Lk - s.Lq));
  s.n = s.ok ? max(0, s.Lq - s.t0) * a.group : 0;
  return s;
}
// first slot of a sequence: floor(x) + 1 >= ceil(x) leaves every sequence enough
__device__ __forceinline__ long first_slot(const BwdArgs &a, int rows, int b, int cq) { return (long)cq * a.group / rows + b; }
__device__ __forceinline__ long slot_at(const BwdArgs &a, long slots, int g, int kb, long slot) {
  return (((long)g * ((a.sink + SK - 1) / SK) + kb) * slots + slot) * PART;
}

__global__ void __launch_bounds__(ST, 1) relattn_bwd_sink_kernel(const __grid_constant__ BwdArgs a, int rows, long slots) {
  extern __shared__ __align__(128) uint8_t smem[];
  const uint32_t sbase = smem_addr(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, gq = lane >> 2, qq = lane & 3;
  const int g = blockIdx.y, b = blockIdx.z;
  const SinkRows s = sink_rows(a, b);
  if (!s.ok && tid == 0 && blockIdx.x == 0) atomicOr(a.err, kDevErrSeqlens);
  const int x0 = (int)min((long)blockIdx.x * rows, (long)s.n), x1 = min(x0 + rows, s.n);
  if (x0 >= x1) return;
  const int off = s.Lk - s.Lq, nkb = (a.sink + SK - 1) / SK;
  const uint32_t ring = sbase + OFF_RING + warp * kSinkRing * STAGE;
  const bool bias = a.sink_dr != nullptr;
  // row x of the list (clamped): token and head
  auto token = [&](int x) { return s.t0 + min(x, s.n - 1) / a.group; };
  auto head = [&](int x) { return g * a.group + min(x, s.n - 1) % a.group; };
  auto issue = [&](int x, int st) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int idx = i * 32 + lane, row = idx >> 4, c = idx & 15;
      const size_t at = ((size_t)(s.cq + token(x + row)) * a.Hq + head(x + row)) * kHeadDim + c * 8;
      cp_async16(ring + st * STAGE + swz(row, c), a.q + at, true);
      cp_async16(ring + st * STAGE + 16 * 256 + swz(row, c), a.dout + at, true);
    }
  };
  const int arow = (lane & 7) + (((lane >> 3) & 1) << 3);     // ldmatrix row of an A (or transposed B) operand

  for (int kb = 0; kb < nkb; ++kb) {
    const int j0 = kb * SK;
    __syncthreads();                       // the block before has been read
    for (int idx = tid; idx < SK * 16; idx += ST) {
      const int row = idx >> 4, c = idx & 15, j = j0 + row;
      const bool ok = j < a.sink && j < s.Lk;
      const size_t at = ((size_t)(s.ck + (ok ? j : 0)) * a.Hkv + g) * kHeadDim + c * 8;
      cp_async16(sbase + OFF_K + swz(row, c), a.k + at, ok);
      cp_async16(sbase + OFF_V + swz(row, c), a.v + at, ok);
    }
    cp_async_commit();
    cp_async_wait<0>();
    __syncthreads();

    float dk[16][4], dv[16][4];            // dk / dv [key][dim]: keys gq, gq + 8
#pragma unroll
    for (int n = 0; n < 16; ++n) {
      dk[n][0] = dk[n][1] = dk[n][2] = dk[n][3] = 0.f;
      dv[n][0] = dv[n][1] = dv[n][2] = dv[n][3] = 0.f;
    }
    int st = 0;
    if (x0 + 16 * warp < x1) issue(x0 + 16 * warp, 0);
    cp_async_commit();
    for (int x = x0 + 16 * warp; x < x1; x += 16 * SW, st ^= 1) {
      if (x + 16 * SW < x1) issue(x + 16 * SW, st ^ 1);
      cp_async_commit();
      cp_async_wait<1>();
      __syncwarp();
      const uint32_t qs = ring + st * STAGE, ds = qs + 16 * 256;
      // ---- S = Q K^T, dP = dout V^T: 16 rows x 16 keys
      float sc[2][4] = {}, dp[2][4] = {};
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        uint32_t qa[4], da[4], kf[4], vf[4];
        const int brow = (lane & 7) + ((lane >> 4) << 3), c = 2 * kk + ((lane >> 3) & 1);
        ldsm_x4(qs + swz(arow, 2 * kk + (lane >> 4)), qa[0], qa[1], qa[2], qa[3]);
        ldsm_x4(ds + swz(arow, 2 * kk + (lane >> 4)), da[0], da[1], da[2], da[3]);
        ldsm_x4(sbase + OFF_K + swz(brow, c), kf[0], kf[1], kf[2], kf[3]);
        ldsm_x4(sbase + OFF_V + swz(brow, c), vf[0], vf[1], vf[2], vf[3]);
        mma_bf16_16816(sc[0], qa[0], qa[1], qa[2], qa[3], kf[0], kf[1]);
        mma_bf16_16816(sc[1], qa[0], qa[1], qa[2], qa[3], kf[2], kf[3]);
        mma_bf16_16816(dp[0], da[0], da[1], da[2], da[3], vf[0], vf[1]);
        mma_bf16_16816(dp[1], da[0], da[1], da[2], da[3], vf[2], vf[3]);
      }
      // ---- the bias of the pairs within E (a sink outside the window lies there only
      // where E reaches past it), all loads in flight together
      float rb[2][4] = {};
      if (bias) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int xr = x + gq + 8 * r, t = token(xr);
          const size_t row = (size_t)(s.cq + t) * a.Hq + head(xr);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int d = off + t - (j0 + (i >> 1) * 8 + 2 * qq + (i & 1));
            const bool in = d >= a.window && d < a.E;
            if (a.rall_ok) {
              rb[r][i] = in ? __ldg(a.Rall + row * a.e_pad + d) : 0.f;
            } else if (in) {
              for (int c = 0; c < a.rd; ++c)
                rb[r][i] = fmaf(__bfloat162float(a.r[row * a.rd + c]), __bfloat162float(a.P[(size_t)c * a.E + d]), rb[r][i]);
            }
          }
        }
      }
      // ---- p and s alpha dl; a row's keys outside its window, of the sinks
      uint32_t pw[2][2], dw[2][2];         // [row half][key half], bf16 pairs of keys
      float rest[2][4];                    // s dl (for dr)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int xr = x + gq + 8 * r, t = token(xr), h = head(xr), pos = off + t;
        const bool live = xr < x1;
        const float srow = log_scale(pos, a.inv_ln_base);
        const size_t li = (size_t)h * a.total_q + s.cq + t;
        const float lse2 = a.lse[li] * kLog2e, Di = a.Dsum[li];
#pragma unroll
        for (int n = 0; n < 2; ++n) {
          float pv[2], dl[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int j = j0 + n * 8 + 2 * qq + e, d = pos - j;
            const bool vis = live && j < a.sink && d >= a.window;
            const float z = fmaf(sc[n][2 * r + e], a.alpha, rb[r][2 * n + e]);
            const float p = vis ? fast_exp2(fmaf(z, srow * kLog2e, -lse2)) : 0.f;
            pv[e] = p;
            const float w = vis ? p * (dp[n][2 * r + e] - Di) * srow : 0.f;
            rest[n][2 * r + e] = w;
            dl[e] = w * a.alpha;
          }
          pw[r][n] = pack_bf16x2(pv[0], pv[1]);
          dw[r][n] = pack_bf16x2(dl[0], dl[1]);
        }
      }
      // ---- dq = dS K (keys as the reduction), out in fp32
#pragma unroll
      for (int dpi = 0; dpi < 8; ++dpi) {
        uint32_t kf[4];
        ldsm_x4_t(sbase + OFF_K + swz(arow, 2 * dpi + (lane >> 4)), kf[0], kf[1], kf[2], kf[3]);
        float dq[2][4] = {};
        mma_bf16_16816(dq[0], dw[0][0], dw[1][0], dw[0][1], dw[1][1], kf[0], kf[1]);
        mma_bf16_16816(dq[1], dw[0][0], dw[1][0], dw[0][1], dw[1][1], kf[2], kf[3]);
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const int xr = x + gq + 8 * r;
          if (xr >= x1) continue;
          float *dst = a.sink_dq + ((size_t)(s.cq + token(xr)) * a.Hq + head(xr)) * kHeadDim + dpi * 16 + 2 * qq;
#pragma unroll
          for (int n = 0; n < 2; ++n) {
            float2 v = make_float2(dq[n][2 * r], dq[n][2 * r + 1]);
            if (kb > 0) {                  // (this thread wrote it for the keys before)
              const float2 o = *reinterpret_cast<const float2 *>(dst + 8 * n);
              v.x += o.x, v.y += o.y;
            }
            *reinterpret_cast<float2 *>(dst + 8 * n) = v;
          }
        }
      }
      // ---- dv += P^T dout, dk += dS^T q (rows as the reduction)
      const uint32_t p0 = transpose8x8(pw[0][0]), p1 = transpose8x8(pw[0][1]), p2 = transpose8x8(pw[1][0]),
                     p3 = transpose8x8(pw[1][1]);
      const uint32_t d0 = transpose8x8(dw[0][0]), d1 = transpose8x8(dw[0][1]), d2 = transpose8x8(dw[1][0]),
                     d3 = transpose8x8(dw[1][1]);
#pragma unroll
      for (int dpi = 0; dpi < 8; ++dpi) {
        uint32_t b0, b1, b2, b3;
        ldsm_x4_t(ds + swz(arow, 2 * dpi + (lane >> 4)), b0, b1, b2, b3);
        mma_bf16_16816(dv[2 * dpi], p0, p1, p2, p3, b0, b1);
        mma_bf16_16816(dv[2 * dpi + 1], p0, p1, p2, p3, b2, b3);
        ldsm_x4_t(qs + swz(arow, 2 * dpi + (lane >> 4)), b0, b1, b2, b3);
        mma_bf16_16816(dk[2 * dpi], d0, d1, d2, d3, b0, b1);
        mma_bf16_16816(dk[2 * dpi + 1], d0, d1, d2, d3, b2, b3);
      }
      // ---- dr of the rows whose bias reaches a sink outside the window: the columns
      // of P that the 16 rows meet turned into shared memory [distance][channel],
      // then two channels a lane (r_dim <= 64), s dl from the lane that holds it
      if (bias && sink_in_bias(a, off + token(x))) {              // (the first row's distances are the least)
        const int dmin = off + token(x) - (j0 + SK - 1);          // 31 distances at most
        __nv_bfloat16 *ps = reinterpret_cast<__nv_bfloat16 *>(smem + OFF_PS + warp * PS_BYTES);
        const bool col = dmin + lane >= a.window && dmin + lane < a.E;
#pragma unroll 8
        for (int c = 0; c < a.rd; ++c) ps[lane * PS_ROW + c] = col ? a.P[(size_t)c * a.E + dmin + lane] : __float2bfloat16(0.f);
        __syncwarp();
#pragma unroll
        for (int r = 0; r < 2; ++r) {
#pragma unroll 1
          for (int i = 0; i < 8; ++i) {
            const int xr = x + 8 * r + i, t = token(xr), pos = off + t;
            if (xr >= x1 || !sink_in_bias(a, pos)) continue;      // (warp-uniform)
            float acc0 = 0.f, acc1 = 0.f;
#pragma unroll
            for (int k = 0; k < SK; ++k) {
              const float v = __shfl_sync(0xffffffffu, rest[k >> 3][2 * r + (k & 1)], 4 * i + ((k & 7) >> 1));
              const int d = pos - (j0 + k);
              if (d < a.window || d >= a.E) continue;             // (no term, whatever s dl is)
              const float2 p = __bfloat1622float2(reinterpret_cast<const __nv_bfloat162 *>(ps + (d - dmin) * PS_ROW)[lane]);
              acc0 = fmaf(v, p.x, acc0);
              acc1 = fmaf(v, p.y, acc1);
            }
            float *dst = a.sink_dr + ((size_t)(s.cq + t) * a.Hq + head(xr)) * a.rd + 2 * lane;
            if (2 * lane < a.rd) dst[0] = kb > 0 ? dst[0] + acc0 : acc0;
            if (2 * lane + 1 < a.rd) dst[1] = kb > 0 ? dst[1] + acc1 : acc1;
          }
        }
      }
      __syncwarp();                        // the stage is read
    }
    cp_async_wait<0>();

    // ---- the warps' dk, then dv, through the ring into the CTA's slot
    float *part = a.sink_part + slot_at(a, slots, g, kb, first_slot(a, rows, b, s.cq) + blockIdx.x);
    float *red = reinterpret_cast<float *>(smem + OFF_RING);      // [warp][64][32 lanes]
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      __syncthreads();
#pragma unroll
      for (int n = 0; n < 16; ++n)
#pragma unroll
        for (int c = 0; c < 4; ++c) red[(warp * 64 + 4 * n + c) * 32 + lane] = which ? dv[n][c] : dk[n][c];
      __syncthreads();
      for (int e = tid; e < 64 * 32; e += ST) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < SW; ++w) v += red[w * 64 * 32 + e];
        const int l = e & 31, c = (e >> 5) & 3, n = e >> 7;
        const int key = (l >> 2) + 8 * (c >> 1), dim = 8 * n + 2 * (l & 3) + (c & 1);
        part[(which * SK + key) * kHeadDim + dim] = v;
      }
    }
  }
}

// sink_dkv[b][g][j] = the slots' sums in order (zero where no row has the sink)
__global__ void __launch_bounds__(2 * kHeadDim) relattn_bwd_sink_sum_kernel(const __grid_constant__ BwdArgs a, int rows, long slots) {
  const int j = blockIdx.x, g = blockIdx.y, b = blockIdx.z;
  const int which = threadIdx.x / kHeadDim, dim = threadIdx.x % kHeadDim;
  const SinkRows s = sink_rows(a, b);
  const int n = (s.n + rows - 1) / rows;
  const float *src = a.sink_part + (which * SK + j % SK) * kHeadDim + dim;
  float v = 0.f;
  for (int i = 0; i < n; ++i) v += src[slot_at(a, slots, g, j / SK, first_slot(a, rows, b, s.cq) + i)];
  a.sink_dkv[((((size_t)b * a.Hkv + g) * a.sink + j) * 2 + which) * kHeadDim + dim] = v;
}

// (152 SMs: the workspace's size follows from it and is given without a device)
int sink_rows_of_cta(int total_q, int Hq) {
  const long want = (long)total_q * Hq / (2 * 152) / kRowsMin * kRowsMin;
  return (int)std::min<long>(std::max<long>(want, kRowsMin), kRowsMax);
}
long sink_slots(int batch, int total_q, int group, int rows) { return (long)total_q * group / rows + batch; }

}  // namespace

size_t bwd_sink_part_bytes(int batch, int total_q, int Hkv, int group, int sink) {
  const int rows = sink_rows_of_cta(total_q, Hkv * group);
  return (size_t)Hkv * ((sink + SK - 1) / SK) * sink_slots(batch, total_q, group, rows) * PART * sizeof(float);
}

cudaError_t launch_bwd_sink(const BwdArgs &a, cudaStream_t stream) {
  static std::atomic<bool> done[kMaxDevicesAttr];
  cudaError_t e = set_max_smem_once(reinterpret_cast<const void *>(relattn_bwd_sink_kernel), SMEM, done);
  if (e != cudaSuccess) return e;
  const int rows = sink_rows_of_cta(a.total_q, a.Hq);
  const long slots = sink_slots(a.batch, a.total_q, a.group, rows);
  const unsigned chunks = (unsigned)(((long)std::min(a.max_q, a.total_q) * a.group + rows - 1) / rows);
  relattn_bwd_sink_kernel<<<dim3(chunks, a.Hkv, a.batch), ST, SMEM, stream>>>(a, rows, slots);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  relattn_bwd_sink_sum_kernel<<<dim3(a.sink, a.Hkv, a.batch), 2 * kHeadDim, 0, stream>>>(a, rows, slots);
  return cudaGetLastError();
}

}  // namespace relattn

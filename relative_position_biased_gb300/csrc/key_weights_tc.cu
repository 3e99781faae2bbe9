// key_weights_tc.cu -- the key weights of many query rows on tcgen05 / TMEM /
// TMA, for the rows of a key tile that carry no relative bias: those whose
// every distance to the tile's 128 keys is at least rel_extent (all rows when
// there is no bias).
//
// w[j] += sum_i exp(x_ij - lse_i), x_ij = s(i) alpha q_i . k_j.  A CTA holds
// the 128 keys of one (sequence, kv head) and walks the rows that see them,
// 256 at a time: S^T = K Q^T with the keys along the MMA's M (TMEM lanes) and
// the rows along N = 256, the widest form: one instruction for 16 dims reads
// the keys once for 256 rows.  With the keys along the lanes a thread owns a
// key, its sum never leaves its register, and a row's constants (s alpha
// log2 e, lse log2 e) are broadcast reads.  A step's rows are 8 sub-tiles of
// 32 tokens of one query head each, so its lse is contiguous and a window or
// a sequence end wastes at most 31 columns.
//
// What bounds it: per logit the tensor core takes 256 flops and a thread one
// fused multiply-add, one exponential and one add (the first and last in
// pairs), and half of an 16-byte shared read for 2 logits.
//
// Roles (12 warps): warp 0 the TMA producer (q, a ring of two steps of 64 KB),
// warp 1 the MMA issuer, warps 4-7 and 8-11 two warpgroups that take the steps
// in turn, each with a TMEM buffer of 256 columns; they also load the keys at
// the start (bf16 rows or 4-bit values as bf16, contiguous or paged) into the
// swizzled operand layout.  Every wait is bounded: a timeout sets the device
// error word, the roles stop, the issuer and the producer drain what they
// issued, and TMEM is freed.
#include <cudaTypedefs.h>

#include <algorithm>

#include "key_weights.cuh"
#include "tc_common.cuh"

namespace relattn {
namespace {

using namespace tc;

constexpr int KWT = 384;                     // threads: 4 role warps + 2 warpgroups
constexpr int SUB = 32, NSUB = 8;            // tokens of a sub-tile, sub-tiles of a step
constexpr int KW_STAGES = 2;
constexpr uint32_t KW_K = 0;                                   // 2 halves [128 keys x 128 B]
constexpr uint32_t KW_Q = KW_K + 32768;                        // stages x 2 halves [256 rows x 128 B]
constexpr uint32_t KW_C = KW_Q + KW_STAGES * 65536;            // per warpgroup: scale [256], -lse [256]
constexpr uint32_t KW_SUM = KW_C + 2 * 2 * 256 * 4;            // the second warpgroup's sums [128]
constexpr uint32_t KW_BAR = KW_SUM + 512;
enum { BK_FULL = 0, BQ_FULL = 1, BQ_EMPTY = BQ_FULL + KW_STAGES, BS_FULL = BQ_EMPTY + KW_STAGES, BS_EMPTY = BS_FULL + 2,
       B_DRAIN_KW = BS_EMPTY + 2, BKW_COUNT };
constexpr uint32_t KW_SLOT = KW_BAR + BKW_COUNT * 8;
constexpr uint32_t KW_ABORT = KW_SLOT + 8;
constexpr uint32_t KW_SMEM = KW_ABORT + 8 + 1024;
static_assert(KW_SMEM <= 227 * 1024, "shared memory budget");

__device__ __forceinline__ bool drain_wait(uint32_t bar, uint32_t parity) {
  const long long t0 = clock64();
  while (!mbar_test_wait(bar, parity))
    if (clock64() - t0 > 200000000ll) return false;
  return true;
}

__device__ __forceinline__ void add2(float &d0, float &d1, float a0, float a1) {
  asm("{\n .reg .b64 ra, rd;\n mov.b64 ra, {%2, %3};\n mov.b64 rd, {%0, %1};\n"
      " add.rn.f32x2 rd, rd, ra;\n mov.b64 {%0, %1}, rd;\n}\n"
      : "+f"(d0), "+f"(d1) : "f"(a0), "f"(a1));
}

__global__ void __launch_bounds__(KWT, 1)
relattn_key_weights_tc_kernel(const __grid_constant__ KeyWeightArgs p, const __grid_constant__ CUtensorMap map_q) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_addr(smem);
  auto bar = [&](int i) { return sb + KW_BAR + 8u * i; };
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + KW_ABORT);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const bool add = p.a.E > 0;                // the tiles kernel has written its part
  Unit u;
  u.rb = 0;
  u.b = blockIdx.y / p.a.Hkv;
  u.h = blockIdx.y - u.b * p.a.Hkv;
  const int ok = unit_tiles(p, u.b, &u.s, &u.lo);
  const int tile0 = blockIdx.x * kWalkTile;
  if (ok < 0) {
    if (blockIdx.x == 0 && u.h == 0 && tid == 0) atomicOr(p.a.err, kDevErrSeqlens);
    return;
  }
  if (tile0 >= u.s.lk) return;
  u.qbase = u.s.lk - u.s.lq;
  const int nkeys = min(kWalkTile, u.s.lk - tile0);
  const int tok0 = min(tc_first_token(p, u.qbase, tile0), u.s.lq);
  int tok1 = u.s.lq;
  if (p.a.window > 0) tok1 = (int)min((long)tok1, max((long)tile0 + nkeys - 1 + p.a.window - u.qbase, 0L));
  const int per_head = tok1 > tok0 ? (tok1 - tok0 + SUB - 1) / SUB : 0;
  const int subs = per_head * p.a.group, steps = (subs + NSUB - 1) / NSUB;
  if (steps == 0 && add) return;

  if (tid == 0) {
    mbar_init(bar(BK_FULL), 256);
    for (int s = 0; s < KW_STAGES; ++s) {
      mbar_init(bar(BQ_FULL + s), 1);
      mbar_init(bar(BQ_EMPTY + s), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(BS_FULL + i), 1);
      mbar_init(bar(BS_EMPTY + i), 128);
    }
    mbar_init(bar(B_DRAIN_KW), 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(sb + KW_SLOT, 512);
    tmem_relinquish();
  }
  if (warp == 0 && lane == 0) prefetch_tmap(&map_q);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + KW_SLOT);

  if (warp == 0) {
    // ======================================================== TMA producer
    if (lane == 0) {
      bool run = true;
      int issued = 0;
      for (int n = 0; n < steps && run; ++n) {
        const int st = n % KW_STAGES;
        if (n >= KW_STAGES && !(run = mbar_wait(bar(BQ_EMPTY + st), ((n / KW_STAGES) - 1) & 1, abort_flag, 21))) break;
        const int cnt = min(NSUB, subs - n * NSUB);
        mbar_arrive_expect_tx(bar(BQ_FULL + st), cnt * SUB * 256);
        for (int s = 0; s < cnt; ++s) {
          const int i = n * NSUB + s, hh = i / per_head, t0 = tok0 + (i - hh * per_head) * SUB;
          const uint32_t dst = sb + KW_Q + st * 65536 + s * (SUB * 128);
          tma_load_3d(dst, &map_q, 0, u.h * p.a.group + hh, u.s.q0 + t0, bar(BQ_FULL + st));
          tma_load_3d(dst + 32768, &map_q, 64, u.h * p.a.group + hh, u.s.q0 + t0, bar(BQ_FULL + st));
        }
        issued = n + 1;
      }
      if (*abort_flag)                       // let the copies this thread issued land before the CTA exits
        for (int m = max(0, issued - KW_STAGES); m < issued; ++m)
          drain_wait(bar(BQ_FULL + m % KW_STAGES), (m / KW_STAGES) & 1);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ======================================================== MMA issuer
    bool run = mbar_wait_warp(bar(BK_FULL), 0, abort_flag, 22);
    tc_fence_after();
    const uint64_t kd = smem_desc_sw128(sb + KW_K, 16, 1024);
    for (int n = 0; n < steps && run; ++n) {
      const int st = n % KW_STAGES, buf = n & 1;
      if (!(run = mbar_wait_warp(bar(BQ_FULL + st), (n / KW_STAGES) & 1, abort_flag, 23))) break;
      if (n >= 2 && !(run = mbar_wait_warp(bar(BS_EMPTY + buf), ((n >> 1) - 1) & 1, abort_flag, 24))) break;
      tc_fence_after();
      const int cnt = min(NSUB, subs - n * NSUB);
      const uint32_t id = idesc_bf16_f32(kWalkTile, cnt * SUB, 0, 0);
      const uint64_t qd = smem_desc_sw128(sb + KW_Q + st * 65536, 16, 1024);
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        const uint32_t ad = kk < 4 ? 2u * kk : 1024u + 2u * (kk - 4);      // the second 64 dims: 16 KB on
        const uint32_t bd = kk < 4 ? 2u * kk : 2048u + 2u * (kk - 4);      // 32 KB on
        mma_ss_e(tmem + 256u * buf, kd + ad, qd + bd, id, kk > 0 ? 1u : 0u);
      }
      mma_commit_e(bar(BQ_EMPTY + st));
      mma_commit_e(bar(BS_FULL + buf));
    }
    if (!run) {
      // stop: wait for the MMAs already issued before tensor memory is freed
      mma_commit_e(bar(B_DRAIN_KW));
      drain_wait(bar(B_DRAIN_KW), 0);
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ======================================================== the two warpgroups
    const int wg = (warp - 4) >> 2, wt = tid - 128 - wg * 128;     // thread = key of the tile
    load_key_tile(p, u, tile0, tid - 128, 256, [&](int k, int c) {
      return smem + KW_K + (c >> 3) * 16384 + k * 128 + (((c & 7) ^ (k & 7)) << 4);
    });
    fence_proxy_async_smem();
    mbar_arrive(bar(BK_FULL));
    const float kg = p.k == nullptr && p.kv.k_global ? __ldg(p.kv.k_global + u.h) : 1.f;
    const float a0 = p.a.alpha_log2e * kg;
    const unsigned wlim = p.a.window > 0 ? (unsigned)p.a.window : 0x80000000u;
    const int key = tile0 + wt;
    const uint32_t lane_off = (uint32_t)((wt >> 5) * 32) << 16;
    float *cs = reinterpret_cast<float *>(smem + KW_C) + wg * 512;  // scale [256], then -lse [256]
    // this thread's two columns of a step: 2 wt, 2 wt + 1 (one sub-tile)
    const int sub = wt >> 4, col = (2 * wt) & 31;
    auto constants = [&](int n, float2 &sc, float2 &z) {
      sc = make_float2(0.f, 0.f);
      z = make_float2(-INFINITY, -INFINITY);
      const int i = n * NSUB + sub;
      if (n >= steps || i >= subs) return;
      const int hh = i / per_head, tok = tok0 + (i - hh * per_head) * SUB + col;
      const float *l = p.lse + (long)(u.h * p.a.group + hh) * p.a.total_q + u.s.q0 + tok;
      if (tok < tok1) {
        const float v = __ldg(l);
        z.x = v == -INFINITY ? -INFINITY : -v * kLog2e;      // a row that saw nothing gives nothing
        sc.x = a0 * log_scale(u.qbase + tok, p.a.inv_ln_base);
      }
      if (tok + 1 < tok1) {
        const float v = __ldg(l + 1);
        z.y = v == -INFINITY ? -INFINITY : -v * kLog2e;
        sc.y = a0 * log_scale(u.qbase + tok + 1, p.a.inv_ln_base);
      }
    };
    float2 sc, z;
    constants(wg, sc, z);
    float s0 = 0.f, s1 = 0.f;
    bool run = true;
    for (int n = wg; n < steps; n += 2) {
      const int buf = wg;
      // the warpgroup's own constants: all have read the step before
      asm volatile("bar.sync %0, 128;" ::"r"(wg + 1) : "memory");
      *reinterpret_cast<float2 *>(cs + 2 * wt) = sc;
      *reinterpret_cast<float2 *>(cs + 256 + 2 * wt) = z;
      asm volatile("bar.sync %0, 128;" ::"r"(wg + 1) : "memory");
      constants(n + 2, sc, z);
      run = run && __all_sync(0xffffffffu, mbar_wait(bar(BS_FULL + buf), (n >> 1) & 1, abort_flag, 25));
      if (!run) continue;                    // (the barriers above stay matched)
      tc_fence_after();
      const int cnt = min(NSUB, subs - n * NSUB);
      const uint32_t taddr = tmem + lane_off + 256u * buf;
      uint32_t x[2][32];
      tmem_ld32(taddr, x[0]);
#pragma unroll
      for (int s = 0; s < NSUB; ++s) {
        if (s >= cnt) break;
        uint32_t(&v)[32] = x[s & 1];
        tmem_wait_ld(v);
        if (s + 1 < cnt) tmem_ld32(taddr + 32u * (s + 1), x[(s + 1) & 1]);
        const int i = n * NSUB + s, hh = i / per_head, t0 = tok0 + (i - hh * per_head) * SUB;
        const int pos0 = u.qbase + t0;
        // some (row, key) of the sub-tile out of sight, or a row past the range
        const bool edge = t0 + SUB > tok1 || pos0 < tile0 + nkeys - 1 || (unsigned)(pos0 + SUB - 1 - tile0) >= wlim;
        const float4 *c4 = reinterpret_cast<const float4 *>(cs + 32 * s);
        const float4 *z4 = reinterpret_cast<const float4 *>(cs + 256 + 32 * s);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const float4 c = c4[q], zz = z4[q];
          float y0, y1, y2, y3;
          ffma2(y0, y1, __uint_as_float(v[4 * q]), __uint_as_float(v[4 * q + 1]), c.x, c.y, zz.x, zz.y);
          ffma2(y2, y3, __uint_as_float(v[4 * q + 2]), __uint_as_float(v[4 * q + 3]), c.z, c.w, zz.z, zz.w);
          if (edge) {
            const int d = pos0 + 4 * q - key;
            const int left = tok1 - (t0 + 4 * q);
            if ((unsigned)d >= wlim || left < 1) y0 = -INFINITY;
            if ((unsigned)(d + 1) >= wlim || left < 2) y1 = -INFINITY;
            if ((unsigned)(d + 2) >= wlim || left < 3) y2 = -INFINITY;
            if ((unsigned)(d + 3) >= wlim || left < 4) y3 = -INFINITY;
          }
          add2(s0, s1, fast_exp2(y0), fast_exp2(y1));
          add2(s0, s1, fast_exp2(y2), fast_exp2(y3));
        }
      }
      tc_fence_before();
      mbar_arrive(bar(BS_EMPTY + buf));
    }
    // the two warpgroups' sums meet
    float *other = reinterpret_cast<float *>(smem + KW_SUM);
    if (wg == 1) other[wt] = s0 + s1;
    asm volatile("bar.sync 3, 256;" ::: "memory");
    if (wg == 0 && key < u.s.lk && !*abort_flag) {
      const float sum = s0 + s1 + other[wt];
      const long row = p.pages.row(u.b, u.s.k0, key);
      if (row < 0) {
        atomicOr(p.a.err, kDevErrSeqlens);
      } else if (add) {
        float *w = p.w_out + (long)u.h * p.pages.rows + row;
        *w += sum;
      } else {
        write_weight(p, u, key, row, sum);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && *abort_flag) record_timeout(p.a.err, *abort_flag);
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = []() -> PFN_cuTensorMapEncodeTiled_v12000 {
    cudaDriverEntryPointQueryResult q;
    void *f = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    return nullptr;
  }();
  return fn;
}

}  // namespace

// At least one 32-token box, and enough rows that 256 columns are worth a
// tile's set-up.
bool key_weights_tc_supported(const KeyWeightArgs &p) {
  return p.a.max_q >= 16 && p.a.total_q >= SUB && encoder() != nullptr;
}

cudaError_t launch_key_weights_tc(const KeyWeightArgs &p, cudaStream_t stream) {
  // q [total_q, Hq, 128] in boxes of 64 dims x 1 head x 32 tokens, 128-byte swizzle
  CUtensorMap mq;
  cuuint64_t dims[3] = {128, (cuuint64_t)p.a.Hq, (cuuint64_t)p.a.total_q};
  cuuint64_t strides[2] = {256, (cuuint64_t)p.a.Hq * 256};
  cuuint32_t box[3] = {64, 1, SUB};
  cuuint32_t es[3] = {1, 1, 1};
  auto fn = encoder();
  if (!fn || fn(&mq, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<__nv_bfloat16 *>(p.a.q), dims, strides, box, es,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  static std::atomic<bool> done[kMaxDevicesAttr];
  const cudaError_t e = set_max_smem_once(reinterpret_cast<const void *>(relattn_key_weights_tc_kernel), (int)KW_SMEM, done);
  if (e != cudaSuccess) return e;
  relattn_key_weights_tc_kernel<<<dim3((unsigned)((p.a.max_k + kWalkTile - 1) / kWalkTile),
                                       (unsigned)(p.a.batch * p.a.Hkv)), KWT, KW_SMEM, stream>>>(p, mq);
  return cudaGetLastError();
}

}  // namespace relattn

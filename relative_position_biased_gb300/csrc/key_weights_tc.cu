// key_weights_tc.cu -- the key weights of many query rows on tcgen05 / TMEM /
// TMA: w[j] += sum_i exp(x_ij - lse_i) over the rows (tokens and heads of a kv
// head's group) that see key j, x_ij = s(i) (alpha q_i . k_j + R_i[i - j]),
// R = r . P inside the band of rel_extent distances.
//
// A CTA holds the 128 keys of one (sequence, kv head) as the MMA's N and walks
// the rows that see them 128 at a time along M (TMEM lanes), rows ordered by
// token, then head.  So a thread owns a row slot and 32 keys: the row's
// constants (scale, lse) are registers, and each (lane, key) partial sum stays
// in a register over all steps; lanes meet once, at the end.  Per logit that
// leaves half a packed multiply-add, an exponential and half a packed add.
//
// Bias: R of a step's rows is a second product, [128 rows x r_dim] x [r_dim x
// (128 + tokens - 1) distances], its second operand consecutive rows of the
// bias table (P's columns in falling order), so key j and the step's token
// tau meet in column j + (tokens - 1 - tau).  A warp's 32 lanes hold at most
// 2^NB tokens: a lane reads a window of 16 + 2^NB - 1 columns and shifts it
// by its token's place with NB rounds of selects.  Nothing of size rows x E
// leaves the SM.
//
// What bounds it: the issue of N = 128 products (about 70 cycles each, 8 a
// step and 4 more in the band) outside the band, the consumers inside it.
//
// Roles (20 warps): warp 0 the TMA producer (q ring of three steps; r rows and
// table window of band steps, two), warp 1 the MMA issuer, warps 4-19 four
// warpgroups of 32 keys each (two of 64 keys left the exponentials waiting for
// TMEM loads: 618 against XXX us on a 4 x 8192 prompt); these also load the
// keys at the start (bf16 rows or 4-bit values as bf16, contiguous or paged)
// into the swizzled operand layout.  CTAs start longest first: early keys are
// seen by the most rows.  TMEM: S twice 128 columns, R up to 256.  Every wait is bounded: a
// timeout sets the device error word, the roles stop, the issuer and the
// producer drain what they issued, and TMEM is freed.
#include <cudaTypedefs.h>

#include <algorithm>

#include "key_weights.cuh"
#include "tc_common.cuh"

namespace relattn {
namespace {

using namespace tc;

constexpr int NWG = 4, KPW = kWalkTile / NWG;          // warpgroups, keys of each
constexpr int KWC = NWG * 128, KWT = 128 + KWC;        // consumer threads, all threads
constexpr int QST = 3, RST = 2;              // stages of q, of r and the table
constexpr uint32_t KW_K = 0;                                   // 2 halves [128 keys x 128 B]
constexpr uint32_t KW_Q = KW_K + 32768;                        // stages x 2 halves [128 rows x 128 B]
constexpr uint32_t KW_R = KW_Q + QST * 32768;                  // stages x [128 rows x 128 B]
constexpr uint32_t KW_T = KW_R + RST * 16384;                  // stages x [256 distances x 128 B]
constexpr uint32_t KW_BAR = KW_T + RST * 32768;
enum { BK_FULL = 0, BQ_FULL = 1, BQ_EMPTY = BQ_FULL + QST, BR_FULL = BQ_EMPTY + QST, BR_EMPTY = BR_FULL + RST,
       BS_FULL = BR_EMPTY + RST, BS_EMPTY = BS_FULL + 2, BB_FULL = BS_EMPTY + 2, BB_EMPTY, B_DRAIN_KW, BKW_COUNT };
constexpr uint32_t KW_SLOT = KW_BAR + BKW_COUNT * 8;
constexpr uint32_t KW_ABORT = KW_SLOT + 8;
constexpr uint32_t KW_SMEM = KW_ABORT + 8 + 1024;
static_assert(KW_SMEM <= 227 * 1024, "shared memory budget");
constexpr uint32_t TM_S = 0, TM_R = 256;     // TMEM columns

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

// Tokens of a step and columns of its R product.
__host__ __device__ __forceinline__ int step_tokens(int group) { return 128 / group; }
__host__ __device__ __forceinline__ int bias_columns(int group) { return (128 + step_tokens(group) - 1 + 15) & ~15; }

// The window w[0 .. CW - 1] moved left by shift < 2^NB places.  (The choices
// are bitwise: written as conditionals the compiler chooses between addresses
// and keeps w in local memory: 4 times the kernel's time.)
template <int NB, int CW, int N>
__device__ __forceinline__ void shift_window(uint32_t (&w)[N], int shift) {
  if constexpr (NB > 0) {
    constexpr int S = 1 << (NB - 1);
    const uint32_t far = shift & S ? 0xffffffffu : 0u;
#pragma unroll
    for (int k = 0; k < CW + S - 1; ++k) w[k] = (w[k + S] & far) | (w[k] & ~far);
    shift_window<NB - 1, CW>(w, shift);
  }
}

struct RowConst {
  float a, b, z;     // logit scale, bias scale, -lse (base 2)
  int pos;           // -1: no row here
};

// KPW keys of a step for one row slot.  BAND: with the bias; EDGE: with masks.
template <int NB, bool BAND, bool EDGE>
__device__ __forceinline__ void step_keys(uint32_t s_addr, uint32_t r_addr, int shift, uint32_t r_done, const RowConst &c,
                                          int key0, unsigned wlim, float (&acc)[KPW]) {
  constexpr int CW = 16, NC = KPW / CW, WIN = CW + (1 << NB) - 1;
  constexpr int W0 = NB == 5 ? 32 : 16, WX = NB <= 2 ? 4 : 16;  // the window's columns come in two loads
#pragma unroll
  for (int ch = 0; ch < NC; ++ch) {
    static_assert(!BAND || WIN <= W0 + WX, "window");
    uint32_t s[CW], lo[BAND ? W0 : 1], hi[BAND ? WX : 1], w[BAND ? W0 + WX : 1];
    tmem_ld16(s_addr + ch * CW, s);
    if constexpr (BAND) {
      if constexpr (W0 == 32) tmem_ld32(r_addr + ch * CW, lo);
      else tmem_ld16(r_addr + ch * CW, lo);
      if constexpr (WX == 4) tmem_ld4(r_addr + ch * CW + W0, hi);
      else tmem_ld16(r_addr + ch * CW + W0, hi);
    }
    tmem_wait_ld(s);
    if constexpr (BAND) {
      tmem_wait_ld(lo);
      tmem_wait_ld(hi);
      if (ch == NC - 1) {                    // R is read: the next step's may be made
        tc_fence_before();
        mbar_arrive(r_done);
      }
#pragma unroll
      for (int k = 0; k < W0; ++k) w[k] = lo[k];
#pragma unroll
      for (int k = 0; k < WX; ++k) w[W0 + k] = hi[k];
      shift_window<NB, CW>(w, shift);
    }
#pragma unroll
    for (int k = 0; k < CW; k += 2) {
      float y0, y1;
      ffma2(y0, y1, __uint_as_float(s[k]), __uint_as_float(s[k + 1]), c.a, c.a, c.z, c.z);
      if constexpr (BAND) ffma2(y0, y1, __uint_as_float(w[k]), __uint_as_float(w[k + 1]), c.b, c.b, y0, y1);
      if constexpr (EDGE) {
        const int d = c.pos - (key0 + ch * CW + k);
        if ((unsigned)d >= wlim || c.pos < 0) y0 = -INFINITY;
        if ((unsigned)(d - 1) >= wlim || c.pos < 0) y1 = -INFINITY;
      }
      add2(acc[ch * CW + k], acc[ch * CW + k + 1], fast_exp2(y0), fast_exp2(y1));
    }
  }
}

template <int NB>
__global__ void __launch_bounds__(KWT, 1)
relattn_key_weights_tc_kernel(const __grid_constant__ KeyWeightArgs p, const __grid_constant__ CUtensorMap map_q,
                              const __grid_constant__ CUtensorMap map_r, const __grid_constant__ CUtensorMap map_t) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_addr(smem);
  auto bar = [&](int i) { return sb + KW_BAR + 8u * i; };
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + KW_ABORT);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  Unit u;
  u.rb = 0;
  const int bh = blockIdx.x % (unsigned)(p.a.batch * p.a.Hkv);
  u.b = bh / p.a.Hkv;
  u.h = bh - u.b * p.a.Hkv;
  const int ok = unit_tiles(p, u.b, &u.s, &u.lo);
  const int tile0 = (int)(blockIdx.x / (unsigned)(p.a.batch * p.a.Hkv)) * kWalkTile;
  if (ok < 0) {
    if (tile0 == 0 && u.h == 0 && tid == 0) atomicOr(p.a.err, kDevErrSeqlens);
  }
  if (ok < 0 || tile0 >= u.s.lk) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }
  u.qbase = u.s.lk - u.s.lq;
  const int nkeys = min(kWalkTile, u.s.lk - tile0), group = p.a.group, ntok = step_tokens(group);
  // tokens that see a key of the tile
  const int tok0 = min(p.tc == 2 ? max(tile0 - u.qbase, 0) : tc_first_token(p, u.qbase, tile0), u.s.lq);
  int tok1 = u.s.lq;
  if (p.a.window > 0) tok1 = (int)min((long)tok1, max((long)tile0 + nkeys - 1 + p.a.window - u.qbase, 0L));
  const int steps = tok1 > tok0 ? (tok1 - tok0 + ntok - 1) / ntok : 0;
  const bool add = p.tc == 1;                // the tiles kernel has written the band's part
  if (steps == 0 && add) return;
  // steps whose rows meet the band (the first ones)
  int band_steps = 0;
  if (p.tc == 2 && p.a.E > 0) {
    const long first = (long)tile0 + kWalkTile - 1 + p.a.E - u.qbase - tok0;      // tokens from tok0 on with distances below E
    band_steps = (int)min((long)steps, max(first + ntok - 1, 0L) / ntok);
  }

  if (tid == 0) {
    mbar_init(bar(BK_FULL), KWC);
    for (int s = 0; s < QST; ++s) mbar_init(bar(BQ_FULL + s), 1), mbar_init(bar(BQ_EMPTY + s), 1);
    for (int s = 0; s < RST; ++s) mbar_init(bar(BR_FULL + s), 1), mbar_init(bar(BR_EMPTY + s), 1);
    for (int i = 0; i < 2; ++i) mbar_init(bar(BS_FULL + i), 1), mbar_init(bar(BS_EMPTY + i), KWC);
    mbar_init(bar(BB_FULL), 1);
    mbar_init(bar(BB_EMPTY), KWC);
    mbar_init(bar(B_DRAIN_KW), 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(sb + KW_SLOT, 512);
    tmem_relinquish();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&map_q);
    if (band_steps > 0) prefetch_tmap(&map_r), prefetch_tmap(&map_t);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + KW_SLOT);

  if (warp == 0) {
    // ======================================================== TMA producer
    if (lane == 0) {
      bool run = true;
      int issued = 0, issued_r = 0;
      const int row_bytes = ntok * group * 128, h0 = u.h * group;
      for (int n = 0; n < steps && run; ++n) {
        const int st = n % QST, t0 = tok0 + n * ntok;
        if (n >= QST && !(run = mbar_wait(bar(BQ_EMPTY + st), ((n / QST) - 1) & 1, abort_flag, 21))) break;
        mbar_arrive_expect_tx(bar(BQ_FULL + st), 2 * row_bytes);
        tma_load_3d(sb + KW_Q + st * 32768, &map_q, 0, h0, u.s.q0 + t0, bar(BQ_FULL + st));
        tma_load_3d(sb + KW_Q + st * 32768 + 16384, &map_q, 64, h0, u.s.q0 + t0, bar(BQ_FULL + st));
        issued = n + 1;
        if (n < band_steps) {
          if (n == 0) asm volatile("griddepcontrol.wait;" ::: "memory");      // the bias table
          const int rs = n % RST;
          if (n >= RST && !(run = mbar_wait(bar(BR_EMPTY + rs), ((n / RST) - 1) & 1, abort_flag, 22))) break;
          mbar_arrive_expect_tx(bar(BR_FULL + rs), row_bytes + bias_columns(group) * 128);
          tma_load_3d(sb + KW_R + rs * 16384, &map_r, 0, h0, u.s.q0 + t0, bar(BR_FULL + rs));
          tma_load_2d(sb + KW_T + rs * 32768, &map_t, 0,
                      rel_table_origin(p.a.E) - (u.qbase + t0 + ntok - 1) + tile0, bar(BR_FULL + rs));
          issued_r = n + 1;
        }
      }
      if (*abort_flag) {                     // let the copies this thread issued land before the CTA exits
        for (int m = max(0, issued - QST); m < issued; ++m) drain_wait(bar(BQ_FULL + m % QST), (m / QST) & 1);
        for (int m = max(0, issued_r - RST); m < issued_r; ++m) drain_wait(bar(BR_FULL + m % RST), (m / RST) & 1);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ======================================================== MMA issuer
    bool run = mbar_wait_warp(bar(BK_FULL), 0, abort_flag, 23);
    tc_fence_after();
    const uint64_t kd = smem_desc_sw128(sb + KW_K, 16, 1024);
    const uint32_t id_s = idesc_bf16_f32(128, kWalkTile, 0, 0), id_r = idesc_bf16_f32(128, bias_columns(group), 0, 0);
    for (int n = 0; n < steps && run; ++n) {
      const int st = n % QST, buf = n & 1;
      if (!(run = mbar_wait_warp(bar(BQ_FULL + st), (n / QST) & 1, abort_flag, 24))) break;
      if (n >= 2 && !(run = mbar_wait_warp(bar(BS_EMPTY + buf), ((n >> 1) - 1) & 1, abort_flag, 25))) break;
      tc_fence_after();
      const uint64_t qd = smem_desc_sw128(sb + KW_Q + st * 32768, 16, 1024);
#pragma unroll
      for (int kk = 0; kk < 8; ++kk) {
        const uint32_t o = kk < 4 ? 2u * kk : 1024u + 2u * (kk - 4);       // the second 64 dims: 16 KB on
        mma_ss_e(tmem + TM_S + 128u * buf, qd + o, kd + o, id_s, kk > 0 ? 1u : 0u);
      }
      mma_commit_e(bar(BQ_EMPTY + st));
      if (n < band_steps) {
        const int rs = n % RST;
        if (!(run = mbar_wait_warp(bar(BR_FULL + rs), (n / RST) & 1, abort_flag, 26))) break;
        if (n >= 1 && !(run = mbar_wait_warp(bar(BB_EMPTY), (n - 1) & 1, abort_flag, 27))) break;
        tc_fence_after();
        const uint64_t rd = smem_desc_sw128(sb + KW_R + rs * 16384, 16, 1024);
        const uint64_t td = smem_desc_sw128(sb + KW_T + rs * 32768, 16, 1024);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) mma_ss_e(tmem + TM_R, rd + 2u * kk, td + 2u * kk, id_r, kk > 0 ? 1u : 0u);
        mma_commit_e(bar(BR_EMPTY + rs));
        mma_commit_e(bar(BB_FULL));
      }
      mma_commit_e(bar(BS_FULL + buf));
    }
    if (!run) {
      // stop: wait for the MMAs already issued before tensor memory is freed
      mma_commit_e(bar(B_DRAIN_KW));
      drain_wait(bar(B_DRAIN_KW), 0);
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ======================================================== the warpgroups
    const int wg = (warp - 4) >> 2, wq = warp & 3, slot = wq * 32 + lane;   // slot = row of the step
    load_key_tile<KWC>(p, u, tile0, tid - 128, [&](int k, int c) {
      return smem + KW_K + (c >> 3) * 16384 + k * 128 + (((c & 7) ^ (k & 7)) << 4);
    });
    fence_proxy_async_smem();
    mbar_arrive(bar(BK_FULL));
    const float kg = p.k == nullptr && p.kv.k_global ? __ldg(p.kv.k_global + u.h) : 1.f;
    const unsigned wlim = p.a.window > 0 ? (unsigned)p.a.window : 0x80000000u;
    const int tau = slot / group, hh = slot - tau * group;
    const bool used = slot < ntok * group;
    const int tau_hi = min((wq * 32 + 31) / group, ntok - 1);              // last token of the warp
    const int shift = max(tau_hi - tau, 0);
    const uint32_t lanes = tmem + ((uint32_t)(wq * 32) << 16);
    const uint32_t r_addr = lanes + TM_R + KPW * wg + (ntok - 1 - tau_hi);
    const int key0 = tile0 + KPW * wg;
    const float *lse = p.lse + (long)(u.h * group + hh) * p.a.total_q + u.s.q0;
    auto load_lse = [&](int n) {
      const int tok = tok0 + n * ntok + tau;
      return n < steps && used && tok < tok1 ? __ldg(lse + tok) : -INFINITY;
    };
    float acc[KPW];
#pragma unroll
    for (int k = 0; k < KPW; ++k) acc[k] = 0.f;
    float z = load_lse(0);
    bool run = true;
    for (int n = 0; n < steps && run; ++n) {
      const int buf = n & 1, t0 = tok0 + n * ntok, tok = t0 + tau;
      RowConst c;
      const bool live = used && tok < tok1 && z != -INFINITY;     // a row that saw nothing gives nothing
      c.pos = live ? u.qbase + tok : -1;
      const float s = live ? log_scale(u.qbase + tok, p.a.inv_ln_base) : 0.f;
      c.a = p.a.alpha_log2e * s * kg;
      c.b = s * kLog2e;
      c.z = live ? -z * kLog2e : -INFINITY;
      z = load_lse(n + 1);
      const bool band = n < band_steps;
      // some pair out of sight, or some slot without a row
      const bool edge = __any_sync(0xffffffffu, !live) || u.qbase + t0 < tile0 + nkeys - 1 ||
                        (unsigned)(u.qbase + t0 + ntok - 1 - tile0) >= wlim;
      run = __all_sync(0xffffffffu, mbar_wait(bar(BS_FULL + buf), (n >> 1) & 1, abort_flag, 28) &&
                                        (!band || mbar_wait(bar(BB_FULL), n & 1, abort_flag, 29)));
      if (!run) break;
      tc_fence_after();
      const uint32_t s_addr = lanes + TM_S + 128u * buf + KPW * wg;
      if (band) {
        if (edge) step_keys<NB, true, true>(s_addr, r_addr, shift, bar(BB_EMPTY), c, key0, wlim, acc);
        else step_keys<NB, true, false>(s_addr, r_addr, shift, bar(BB_EMPTY), c, key0, wlim, acc);
      } else {
        if (edge) step_keys<NB, false, true>(s_addr, r_addr, shift, 0, c, key0, wlim, acc);
        else step_keys<NB, false, false>(s_addr, r_addr, shift, 0, c, key0, wlim, acc);
      }
      tc_fence_before();
      mbar_arrive(bar(BS_EMPTY + buf));
    }
    // the lanes' sums meet: lane k ends with key k
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      const bool up = lane & o;
#pragma unroll
      for (int k = 0; k < o; ++k) {
        const float give = up ? acc[k] : acc[k + o], keep = up ? acc[k + o] : acc[k];
        acc[k] = keep + __shfl_xor_sync(0xffffffffu, give, o);
      }
    }
    // the q ring is idle once every step has been read
    float *part = reinterpret_cast<float *>(smem + KW_Q) + wg * 128;        // [4 warps][32 keys]
    part[wq * 32 + lane] = acc[0];
    asm volatile("bar.sync %0, 128;" ::"r"(wg + 1) : "memory");
    const int key = key0 + lane;
    if (wq == 0 && key < u.s.lk && !*abort_flag) {
      const float sum = part[lane] + part[32 + lane] + part[64 + lane] + part[96 + lane];
      const long row = p.pages.row(u.b, u.s.k0, key);
      if (row < 0) {
        atomicOr(p.a.err, kDevErrSeqlens);
      } else if (add) {
        p.w_out[(long)u.h * p.pages.rows + row] += sum;
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
  asm volatile("griddepcontrol.wait;" ::: "memory");
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

// [tokens, heads, width] bf16 in boxes of 64 columns (zero past width) x a
// group's heads x a step's tokens, 128-byte swizzle
bool encode_rows(CUtensorMap *m, const void *base, int width, int heads, int tokens, int group) {
  auto fn = encoder();
  if (!fn) return false;
  cuuint64_t dims[3] = {(cuuint64_t)width, (cuuint64_t)heads, (cuuint64_t)tokens};
  cuuint64_t strides[2] = {(cuuint64_t)width * 2, (cuuint64_t)heads * width * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)group, (cuuint32_t)step_tokens(group)};
  cuuint32_t es[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int NB>
cudaError_t launch_nb(const KeyWeightArgs &p, cudaStream_t stream, const CUtensorMap &mq, const CUtensorMap &mr,
                      const CUtensorMap &mt) {
  static std::atomic<bool> done[kMaxDevicesAttr];
  auto *kernel = relattn_key_weights_tc_kernel<NB>;
  const cudaError_t e = set_max_smem_once(reinterpret_cast<const void *>(kernel), (int)KW_SMEM, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  const long grid = ((long)p.a.max_k + kWalkTile - 1) / kWalkTile * p.a.batch * p.a.Hkv;
  if (grid > 0x7fffffffL) return cudaErrorInvalidValue;
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(KWT);
  cfg.dynamicSmemBytes = KW_SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = p.tc == 2 && p.a.E > 0 ? 1 : 0;       // right behind the bias table's kernel
  return cudaLaunchKernelEx(&cfg, kernel, p, mq, mr, mt);
}

}  // namespace

// 0: the shape is not for this kernel; 2: it takes every row; 1: it takes the
// rows past the band (r's rows are not 16-byte multiples, or P's are not
// aligned), the tiles kernel the others.
int key_weights_tc_kind(const KeyWeightArgs &p) {
  const KernelArgs &a = p.a;
  if (a.group > 128 || a.max_q < 16 || a.total_q < step_tokens(a.group) || !encoder()) return 0;
  if (a.E == 0) return 2;
  return a.rd % 8 == 0 && (reinterpret_cast<uintptr_t>(a.r) & 15u) == 0 ? 2 : 1;
}

cudaError_t launch_key_weights_tc(const KeyWeightArgs &p, cudaStream_t stream) {
  CUtensorMap mq, mr, mt;
  const int group = p.a.group;
  if (!encode_rows(&mq, p.a.q, kHeadDim, p.a.Hq, p.a.total_q, group)) return cudaErrorInvalidValue;
  mr = mt = mq;                              // (unused without a bias)
  if (p.tc == 2 && p.a.E > 0) {
    if (!encode_rows(&mr, p.a.r, p.a.rd, p.a.Hq, p.a.total_q, group)) return cudaErrorInvalidValue;
    cuuint64_t dims[2] = {64, (cuuint64_t)rel_table_rows(p.a.E)};
    cuuint64_t strides[1] = {128};
    cuuint32_t box[2] = {64, (cuuint32_t)bias_columns(group)};
    cuuint32_t es[2] = {1, 1};
    if (encoder()(&mt, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<__nv_bfloat16 *>(p.table), dims, strides, box, es,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  // most tokens that 32 consecutive row slots may hold
  const int tokens = std::min(32, 31 / group + 2);
  const int exact = 32 % group == 0 ? 32 / group : tokens;
  if (exact <= 2) return launch_nb<1>(p, stream, mq, mr, mt);
  if (exact <= 4) return launch_nb<2>(p, stream, mq, mr, mt);
  if (exact <= 8) return launch_nb<3>(p, stream, mq, mr, mt);
  if (exact <= 16) return launch_nb<4>(p, stream, mq, mr, mt);
  return launch_nb<5>(p, stream, mq, mr, mt);
}

}  // namespace relattn

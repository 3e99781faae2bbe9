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
// step and 4 more in the band) outside the band, the consumers inside it; with
// a tile of only two steps (32 observing tokens of a group of 8) the consumers'
// turn from tile to tile, of which the lanes' shuffles are a third.  Measured: all
// rows of a 4 x 8192 prompt, window 4096, group 8: 575 us, 717 TFLOP/s.
//
// A CTA is given tiles until there are none left (cluster launch control), in
// the order in which CTAs would start, longest first: early keys are seen by
// the most rows.  The next tile's keys and query rows are on their way while
// this one is worked on.  With a CTA for each tile its start, the load of the
// keys and the last sums were 6 us of each: 140 us for 32 tokens of each of
// 4 sequences of 16 to 64 thousand keys, now 69.  A tile is taken only when
// at most kStepsAhead steps are left: taken as early as the slots allow, the
// CTAs were uneven at the end (682 against 575 us on a 4 x 8192 prompt, window
// 4096).
//
// Roles (20 warps): warp 0 the TMA producer (q ring of three steps; r rows and
// table window of a band step), warp 1 the MMA issuer, warp 2 the scheduler,
// which plans the tiles for all, warp 3 the producer of bf16 keys (two stages,
// 32 keys a load, contiguous or paged), warps 4-19 four warpgroups of 32 keys
// each (two of 64 keys left the exponentials waiting for TMEM loads: 618
// against 583 us on that prompt); these also load 4-bit keys, as bf16, into the
// swizzled operand layout.  TMEM: S twice 128 columns, R up to 256.  Every wait
// is bounded: a timeout sets the device error word, the roles stop, those that
// issued copies, products or requests await them, and TMEM is freed.
#include <cudaTypedefs.h>

#include <algorithm>

#include "key_weights.cuh"
#include "tc_common.cuh"

namespace relattn {
namespace {

using namespace tc;

constexpr int NWG = 4, KPW = kWalkTile / NWG;          // warpgroups, keys of each
constexpr int KWC = NWG * 128, KWT = 128 + KWC;        // consumer threads, all threads
constexpr int KST = 2, QST = 3, RST = 1;     // stages of the keys, of q, of r and the table
constexpr int UST = 3;                       // tiles planned and not yet finished
constexpr int kStepsAhead = 8;               // no further tile is taken while more steps than these are left
constexpr uint32_t KW_K = 0;                                   // stages x 2 halves [128 keys x 128 B]
constexpr uint32_t KW_Q = KW_K + KST * 32768;                  // stages x 2 halves [128 rows x 128 B]
constexpr uint32_t KW_R = KW_Q + QST * 32768;                  // stages x [128 rows x 128 B]
constexpr uint32_t KW_T = KW_R + RST * 16384;                  // stages x [256 distances x 128 B]
constexpr uint32_t KW_PART = KW_T + RST * 32768;               // [warpgroup][3 warps][32 keys] sums
constexpr uint32_t KW_UNIT = KW_PART + NWG * 96 * 4;           // stages x a planned tile
constexpr uint32_t KW_CLC = KW_UNIT + UST * 64;
constexpr uint32_t KW_BAR = KW_CLC + 16;
enum { BK_FULL = 0, BK_EMPTY = BK_FULL + KST, BU_FULL = BK_EMPTY + KST, BU_EMPTY = BU_FULL + UST,
       BC_FULL = BU_EMPTY + UST, BQ_FULL, BQ_EMPTY = BQ_FULL + QST, BR_FULL = BQ_EMPTY + QST, BR_EMPTY = BR_FULL + RST,
       BS_FULL = BR_EMPTY + RST, BS_EMPTY = BS_FULL + 2, BB_FULL = BS_EMPTY + 2, BB_EMPTY,
       BP_FULL, BP_EMPTY = BP_FULL + NWG, B_DRAIN_KW = BP_EMPTY + NWG, BKW_COUNT };
constexpr uint32_t KW_SLOT = KW_BAR + BKW_COUNT * 8;
constexpr uint32_t KW_ABORT = KW_SLOT + 8;
constexpr uint32_t KW_DONE = KW_ABORT + 4;   // steps that the issuer has begun
constexpr uint32_t KW_SMEM = KW_ABORT + 8 + 1024;
static_assert(KW_SMEM <= 227 * 1024, "shared memory budget");
constexpr uint32_t TM_S = 0, TM_R = 256;     // TMEM columns
// Waits for a planned tile last as long as the scheduler passes over units that
// have none: max_seqlen_k may be far above the lengths, a grid has up to 2^31
// units, and one takes 0.9 us of an SM (400 million: 2.4 s).  The scheduler's own
// waits are short, and one that gives up ends these too, so this is only the last
// resort: 40 s.
constexpr long long kPlanCycles = 80000000000ll;

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

// One unit of work: the 128 keys from tile0 of a (sequence, kv head).
struct alignas(16) Tile {
  int b, h, q0, lq, k0, lk;
  int qbase;                 // position of the sequence's first query row
  int tile0, nkeys;
  int tok0, tok1;            // tokens that see a key of the tile
  int steps, band_steps;     // steps of the tile; those whose rows meet the band (the first ones)
  int more, pad[2];          // 0: there was no further tile
};
static_assert(sizeof(Tile) == 64, "four 16-byte words");

// Unit `index` of the grid; false where the sequence has no such tile.
__device__ __forceinline__ bool plan_tile(const KeyWeightArgs &p, unsigned index, Tile &t) {
  const unsigned heads = (unsigned)(p.a.batch * p.a.Hkv);
  const int bh = index % heads;
  t.b = bh / p.a.Hkv;
  t.h = bh - t.b * p.a.Hkv;
  t.tile0 = (int)(index / heads) * kWalkTile;
  t.more = 1;
  SeqRows s;
  int lo;
  if (unit_tiles(p, t.b, &s, &lo) < 0) {
    if (t.tile0 == 0 && t.h == 0) atomicOr(p.a.err, kDevErrSeqlens);
    return false;
  }
  if (t.tile0 >= s.lk) return false;
  t.q0 = s.q0, t.lq = s.lq, t.k0 = s.k0, t.lk = s.lk;
  t.qbase = s.lk - s.lq;
  const int ntok = step_tokens(p.a.group);
  t.nkeys = min(kWalkTile, s.lk - t.tile0);
  t.tok0 = min(p.tc == 2 ? max(t.tile0 - t.qbase, 0) : tc_first_token(p, t.qbase, t.tile0), s.lq);
  t.tok1 = s.lq;
  if (p.a.window > 0) t.tok1 = (int)min((long)t.tok1, max((long)t.tile0 + t.nkeys - 1 + p.a.window - t.qbase, 0L));
  t.steps = t.tok1 > t.tok0 ? (t.tok1 - t.tok0 + ntok - 1) / ntok : 0;
  t.band_steps = 0;
  if (p.tc == 2 && p.a.E > 0) {
    const long first = (long)t.tile0 + kWalkTile - 1 + p.a.E - t.qbase - t.tok0;     // tokens from tok0 on with distances below E
    t.band_steps = (int)min((long)t.steps, max(first + ntok - 1, 0L) / ntok);
  }
  return true;
}

// Cluster launch control: a CTA asks for the index of one that has not begun
// and takes its work over, so that the hardware's order (longest first) holds
// while barriers, tensor memory and the loads of the next keys carry on.
__device__ __forceinline__ void ask_for_unit(uint32_t dst, uint32_t bar) {
  asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];\n" ::"r"(dst),
               "r"(bar)
               : "memory");
}
__device__ __forceinline__ bool given_unit(uint32_t src, unsigned *index) {
  uint32_t got, x;
  asm volatile(
      "{\n .reg .pred p;\n .reg .b128 w;\n ld.shared.b128 w, [%2];\n"
      " clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, w;\n selp.u32 %0, 1, 0, p;\n mov.u32 %1, 0;\n"
      " @p clusterlaunchcontrol.query_cancel.get_first_ctaid::x.b32.b128 %1, w;\n}\n"
      : "=r"(got), "=r"(x)
      : "r"(src)
      : "memory");
  *index = x;
  return got != 0;
}

template <int NB>
__global__ void __launch_bounds__(KWT, 1)
relattn_key_weights_tc_kernel(const __grid_constant__ KeyWeightArgs p, const __grid_constant__ CUtensorMap map_q,
                              const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_r,
                              const __grid_constant__ CUtensorMap map_t) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_addr(smem);
  auto bar = [&](int i) { return sb + KW_BAR + 8u * i; };
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + KW_ABORT);
  volatile int *begun = reinterpret_cast<volatile int *>(smem + KW_DONE);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int group = p.a.group, ntok = step_tokens(group);
  const bool add = p.tc == 1;                // the tiles kernel has written the band's part

  if (tid == 0) {
    for (int s = 0; s < KST; ++s) mbar_init(bar(BK_FULL + s), p.k ? 1 : KWC), mbar_init(bar(BK_EMPTY + s), 1);
    // a tile is read by the two producers' lanes, the issuer's and the consumers' warps
    for (int s = 0; s < UST; ++s) mbar_init(bar(BU_FULL + s), 1), mbar_init(bar(BU_EMPTY + s), 3 + KWC / 32);
    mbar_init(bar(BC_FULL), 1);
    for (int s = 0; s < QST; ++s) mbar_init(bar(BQ_FULL + s), 1), mbar_init(bar(BQ_EMPTY + s), 1);
    for (int s = 0; s < RST; ++s) mbar_init(bar(BR_FULL + s), 1), mbar_init(bar(BR_EMPTY + s), 1);
    for (int i = 0; i < 2; ++i) mbar_init(bar(BS_FULL + i), 1), mbar_init(bar(BS_EMPTY + i), KWC);
    mbar_init(bar(BB_FULL), 1);
    mbar_init(bar(BB_EMPTY), KWC);
    for (int i = 0; i < NWG; ++i) mbar_init(bar(BP_FULL + i), 96), mbar_init(bar(BP_EMPTY + i), 32);
    mbar_init(bar(B_DRAIN_KW), 1);
    *abort_flag = 0;
    *begun = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(sb + KW_SLOT, 512);
    tmem_relinquish();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&map_q);
    if (p.k) prefetch_tmap(&map_k);
    if (p.tc == 2 && p.a.E > 0) prefetch_tmap(&map_r), prefetch_tmap(&map_t);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + KW_SLOT);
  // A wait that may last a tile: it gives up a second after the issuer's last step.
  auto wait_long = [&](int b, uint32_t parity, int site, long long limit = 2000000000ll) {
    long long t0 = clock64();
    int seen = *begun;
    while (!mbar_try_wait(bar(b), parity, 2000u)) {
      if (*abort_flag) return false;
      if (*begun != seen) {
        seen = *begun;
        t0 = clock64();
      } else if (clock64() - t0 > limit) {
        *abort_flag = site;
        return false;
      }
    }
    return true;
  };
  // The k-th tile of this CTA, by a whole warp, or by one lane; false: there is none.
  auto next_tile = [&](int k, bool one_lane, Tile &t) {
    const int s = k % UST;
    bool got = wait_long(BU_FULL + s, (k / UST) & 1, 30, kPlanCycles);
    if (!one_lane) got = __all_sync(0xffffffffu, got);
    if (!got) return false;
    const uint4 *src = reinterpret_cast<const uint4 *>(smem + KW_UNIT + 64 * s);
    uint4 *dst = reinterpret_cast<uint4 *>(&t);
#pragma unroll
    for (int i = 0; i < 4; ++i) dst[i] = src[i];
    if (!one_lane) __syncwarp();
    if (one_lane || lane == 0) mbar_arrive(bar(BU_EMPTY + s));
    return t.more != 0;
  };

  if (warp < 4) {
    if (warp == 0) {
      // ====================================================== TMA producer
      if (lane == 0) {
        bool run = true, table = false;
        int g = 0, gr = 0;                   // steps, band steps issued
        const int row_bytes = ntok * group * 128;
        Tile t;
        for (int k = 0; run && next_tile(k, true, t); ++k) {
          const int h0 = t.h * group;
          for (int n = 0; n < t.steps && run; ++n) {
            const int st = g % QST, t0 = t.tok0 + n * ntok;
            if (g >= QST && !(run = mbar_wait(bar(BQ_EMPTY + st), ((g / QST) - 1) & 1, abort_flag, 21))) break;
            mbar_arrive_expect_tx(bar(BQ_FULL + st), 2 * row_bytes);
            tma_load_3d(sb + KW_Q + st * 32768, &map_q, 0, h0, t.q0 + t0, bar(BQ_FULL + st));
            tma_load_3d(sb + KW_Q + st * 32768 + 16384, &map_q, 64, h0, t.q0 + t0, bar(BQ_FULL + st));
            ++g;
            if (n < t.band_steps) {
              if (!table) asm volatile("griddepcontrol.wait;" ::: "memory");      // the bias table
              table = true;
              const int rs = gr % RST;
              if (gr >= RST && !(run = mbar_wait(bar(BR_EMPTY + rs), ((gr / RST) - 1) & 1, abort_flag, 22))) break;
              mbar_arrive_expect_tx(bar(BR_FULL + rs), row_bytes + bias_columns(group) * 128);
              tma_load_3d(sb + KW_R + rs * 16384, &map_r, 0, h0, t.q0 + t0, bar(BR_FULL + rs));
              tma_load_2d(sb + KW_T + rs * 32768, &map_t, 0,
                          rel_table_origin(p.a.E) - (t.qbase + t0 + ntok - 1) + t.tile0, bar(BR_FULL + rs));
              ++gr;
            }
          }
        }
        if (*abort_flag) {                   // let the copies this thread issued land before the CTA exits
          for (int m = max(0, g - QST); m < g; ++m) drain_wait(bar(BQ_FULL + m % QST), (m / QST) & 1);
          for (int m = max(0, gr - RST); m < gr; ++m) drain_wait(bar(BR_FULL + m % RST), (m / RST) & 1);
        }
      }
      __syncwarp();
    } else if (warp == 1) {
      // ====================================================== MMA issuer
      bool run = true;
      int g = 0, gr = 0, kt = 0;             // steps, band steps and tiles so far
      const uint32_t id_s = idesc_bf16_f32(128, kWalkTile, 0, 0), id_r = idesc_bf16_f32(128, bias_columns(group), 0, 0);
      Tile t;
      for (int k = 0; run && next_tile(k, false, t); ++k) {
        const int ks = kt % KST;
        if (t.steps > 0 && !(run = mbar_wait_warp(bar(BK_FULL + ks), (kt / KST) & 1, abort_flag, 23))) break;
        const uint64_t kd = smem_desc_sw128(sb + KW_K + ks * 32768, 16, 1024);
        for (int n = 0; n < t.steps; ++n) {
          const int st = g % QST, buf = g & 1;
          if (!(run = mbar_wait_warp(bar(BQ_FULL + st), (g / QST) & 1, abort_flag, 24))) break;
          if (g >= 2 && !(run = mbar_wait_warp(bar(BS_EMPTY + buf), ((g >> 1) - 1) & 1, abort_flag, 25))) break;
          tc_fence_after();
          const uint64_t qd = smem_desc_sw128(sb + KW_Q + st * 32768, 16, 1024);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            const uint32_t o = kk < 4 ? 2u * kk : 1024u + 2u * (kk - 4);       // the second 64 dims: 16 KB on
            mma_ss_e(tmem + TM_S + 128u * buf, qd + o, kd + o, id_s, kk > 0 ? 1u : 0u);
          }
          mma_commit_e(bar(BQ_EMPTY + st));
          if (lane == 0) *begun = g + 1;
          if (n < t.band_steps) {
            const int rs = gr % RST;
            if (!(run = mbar_wait_warp(bar(BR_FULL + rs), (gr / RST) & 1, abort_flag, 26))) break;
            if (gr >= 1 && !(run = mbar_wait_warp(bar(BB_EMPTY), (gr - 1) & 1, abort_flag, 27))) break;
            tc_fence_after();
            const uint64_t rd = smem_desc_sw128(sb + KW_R + rs * 16384, 16, 1024);
            const uint64_t td = smem_desc_sw128(sb + KW_T + rs * 32768, 16, 1024);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) mma_ss_e(tmem + TM_R, rd + 2u * kk, td + 2u * kk, id_r, kk > 0 ? 1u : 0u);
            mma_commit_e(bar(BR_EMPTY + rs));
            mma_commit_e(bar(BB_FULL));
            ++gr;
          }
          mma_commit_e(bar(BS_FULL + buf));
          ++g;
        }
        if (!run) break;
        if (t.steps > 0) {
          mma_commit_e(bar(BK_EMPTY + ks));
          ++kt;
        }
      }
      if (*abort_flag) {
        // stop: wait for the MMAs already issued before tensor memory is freed
        mma_commit_e(bar(B_DRAIN_KW));
        drain_wait(bar(B_DRAIN_KW), 0);
      }
      __syncwarp();
    } else if (warp == 2 && lane == 0) {
      // ====================================================== scheduler
      unsigned index = blockIdx.x;
      bool more = true, own = true;          // the first tile is the CTA's own
      int asked = 0, steps = 0;
      for (int k = 0; more; ++k) {
        const int s = k % UST;
        if (k >= UST && !wait_long(BU_EMPTY + s, ((k / UST) - 1) & 1, 31)) break;
        Tile t = {};
        do {
          if (!own) {
            // a tile taken early is one that an idler CTA cannot take
            long long t0 = clock64();
            for (int seen = *begun; steps - *begun > kStepsAhead && !*abort_flag;) {
              __nanosleep(100);
              if (*begun != seen) {
                seen = *begun;
                t0 = clock64();
              } else if (clock64() - t0 > 2000000000ll) {
                *abort_flag = 36;
              }
            }
            if (*abort_flag) {
              more = false;
              break;
            }
            fence_proxy_async_smem();        // the last answer has been read
            mbar_arrive_expect_tx(bar(BC_FULL), 16);
            ask_for_unit(sb + KW_CLC, bar(BC_FULL));
            // the answer is awaited whatever else went wrong
            if (!drain_wait(bar(BC_FULL), asked & 1)) {
              *abort_flag = 32;
              more = false;
              break;
            }
            ++asked;
            more = given_unit(sb + KW_CLC, &index);
          }
          own = false;
        } while (more && !plan_tile(p, index, t));
        if (!more) t.more = 0;
        steps += t.more ? t.steps : 0;
        *reinterpret_cast<Tile *>(smem + KW_UNIT + 64 * s) = t;
        mbar_arrive(bar(BU_FULL + s));
      }
    } else if (warp == 3 && lane == 0) {
      // ====================================================== the keys' producer (bf16)
      int kt = 0;
      Tile t;
      for (int k = 0; next_tile(k, true, t); ++k) {
        if (t.steps == 0 || !p.k) continue;
        const int ks = kt % KST;
        if (kt >= KST && !wait_long(BK_EMPTY + ks, ((kt / KST) - 1) & 1, 33)) break;
        if (kt++ == p.a.test_skip_k_tile) continue;     // (test hook: a skipped tile is never loaded)
        mbar_arrive_expect_tx(bar(BK_FULL + ks), 32768);
#pragma unroll
        for (int i = 0; i < kWalkTile / 32; ++i) {
          // 32 keys share a page; rows past the last key, which nothing counts, may be any, and outside the cache zeros
          const int key = t.tile0 + 32 * i;
          const long row = key < t.lk ? p.pages.row(t.b, t.k0, key) : -1;
          const int z = (int)(row >= 0 ? row : p.pages.rows);
          const uint32_t dst = sb + KW_K + ks * 32768 + i * 4096;
          tma_load_3d(dst, &map_k, 0, t.h, z, bar(BK_FULL + ks));
          tma_load_3d(dst + 16384, &map_k, 64, t.h, z, bar(BK_FULL + ks));
        }
      }
      if (*abort_flag)                       // the copies land before the CTA exits
        for (int m = max(0, kt - KST); m < kt; ++m) drain_wait(bar(BK_FULL + m % KST), (m / KST) & 1);
    }
  } else {
    // ======================================================== the warpgroups
    const int wg = (warp - 4) >> 2, wq = warp & 3, slot = wq * 32 + lane;   // slot = row of the step
    const unsigned wlim = p.a.window > 0 ? (unsigned)p.a.window : 0x80000000u;
    const int tau = slot / group, hh = slot - tau * group;
    const bool used = slot < ntok * group;
    const int tau_hi = min((wq * 32 + 31) / group, ntok - 1);              // last token of the warp
    const int shift = max(tau_hi - tau, 0);
    const uint32_t lanes = tmem + ((uint32_t)(wq * 32) << 16);
    const uint32_t r_addr = lanes + TM_R + KPW * wg + (ntok - 1 - tau_hi);
    float *part = reinterpret_cast<float *>(smem + KW_PART) + wg * 96;      // [3 warps][32 keys]
    bool run = true;
    int g = 0, gr = 0, sums = 0;
    // The k-th tile stays in its slot until this warp is done with it.
    auto tile_at = [&](int k) { return reinterpret_cast<const volatile Tile *>(smem + KW_UNIT + 64 * (k % UST)); };
    auto wait_tile = [&](int k) {
      return __all_sync(0xffffffffu, mbar_wait(bar(BU_FULL + k % UST), (k / UST) & 1, abort_flag, 30, kPlanCycles)) &&
             tile_at(k)->more;
    };
    auto unit_at = [&](const volatile Tile *t) {
      Unit u = {};
      u.s.q0 = t->q0, u.s.lq = t->lq, u.s.k0 = t->k0, u.s.lk = t->lk;
      u.b = t->b, u.h = t->h, u.qbase = t->qbase;
      return u;
    };
    auto lse_of = [&](const volatile Tile *t) {
      return p.lse + (long)(t->h * group + hh) * p.a.total_q + t->q0 + t->tok0 + tau;
    };
    int kt = 0;
    // 4-bit keys are made bf16 by these threads; the stage is free: every step of the tile before the last has been read
    auto load_keys = [&](int k) {
      if (p.k || tile_at(k)->steps == 0) return;
      const uint32_t ks = kt++ % KST * 32768;
      load_key_tile<KWC>(p, unit_at(tile_at(k)), tile_at(k)->tile0, tid - 128, [&](int key, int c) {
        return smem + KW_K + ks + (c >> 3) * 16384 + key * 128 + (((c & 7) ^ (key & 7)) << 4);
      });
      fence_proxy_async_smem();
      mbar_arrive(bar(BK_FULL + ks / 32768));
    };
    // lse of the row in the step n whose first token is `left` before the tile's last
    auto load_lse = [&](const float *lse, int n, int left) {
      return used && n * ntok + tau < left ? __ldg(lse + n * ntok) : -INFINITY;
    };
    bool more = wait_tile(0);
    float z = -INFINITY;
    if (more) {
      load_keys(0);
      z = load_lse(lse_of(tile_at(0)), 0, tile_at(0)->tok1 - tile_at(0)->tok0);
    }
    for (int k = 0; more; ++k) {
      const volatile Tile *t = tile_at(k);
      const float kg = p.k == nullptr && p.kv.k_global ? __ldg(p.kv.k_global + t->h) : 1.f;
      const float *lse = lse_of(t);
      const int tile0 = t->tile0, key0 = tile0 + KPW * wg, last = tile0 + t->nkeys - 1;
      const int steps = t->steps, band_steps = t->band_steps;
      const int pos0 = t->qbase + t->tok0, left = t->tok1 - t->tok0;       // first token's position; tokens
      float acc[KPW];
#pragma unroll
      for (int j = 0; j < KPW; ++j) acc[j] = 0.f;
      for (int n = 0; n < steps; ++n, ++g) {
        const int buf = g & 1, pos = pos0 + n * ntok;
        RowConst c;
        const bool live = used && n * ntok + tau < left && z != -INFINITY;     // a row that saw nothing gives nothing
        c.pos = live ? pos + tau : -1;
        const float s = live ? log_scale(pos + tau, p.a.inv_ln_base) : 0.f;
        c.a = p.a.alpha_log2e * s * kg;
        c.b = s * kLog2e;
        c.z = live ? -z * kLog2e : -INFINITY;
        z = n + 1 < steps ? load_lse(lse, n + 1, left) : -INFINITY;
        const bool band = n < band_steps;
        // some pair out of sight, or some slot without a row
        const bool edge = __any_sync(0xffffffffu, !live) || pos < last || (unsigned)(pos + ntok - 1 - tile0) >= wlim;
        run = __all_sync(0xffffffffu, mbar_wait(bar(BS_FULL + buf), (g >> 1) & 1, abort_flag, 28) &&
                                          (!band || mbar_wait(bar(BB_FULL), gr & 1, abort_flag, 29)));
        if (!run) break;
        tc_fence_after();
        const uint32_t s_addr = lanes + TM_S + 128u * buf + KPW * wg;
        if (band) {
          if (edge) step_keys<NB, true, true>(s_addr, r_addr, shift, bar(BB_EMPTY), c, key0, wlim, acc);
          else step_keys<NB, true, false>(s_addr, r_addr, shift, bar(BB_EMPTY), c, key0, wlim, acc);
          ++gr;
        } else {
          if (edge) step_keys<NB, false, true>(s_addr, r_addr, shift, 0, c, key0, wlim, acc);
          else step_keys<NB, false, false>(s_addr, r_addr, shift, 0, c, key0, wlim, acc);
        }
        tc_fence_before();
        mbar_arrive(bar(BS_EMPTY + buf));
      }
      if (!run) break;
      // the next tile's first lse is on its way while this one's sums meet
      more = wait_tile(k + 1);
      if (more) {
        load_keys(k + 1);
        z = load_lse(lse_of(tile_at(k + 1)), 0, tile_at(k + 1)->tok1 - tile_at(k + 1)->tok0);
      }
      if (t->steps > 0 || !add) {
        // lane j ends with key j
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
          const bool up = lane & o;
#pragma unroll
          for (int j = 0; j < o; ++j) {
            const float give = up ? acc[j] : acc[j + o], keep = up ? acc[j + o] : acc[j];
            acc[j] = keep + __shfl_xor_sync(0xffffffffu, give, o);
          }
        }
        // the sums of a warpgroup's four warps meet in its first (mbarriers: a
        // warp that gave up must not leave the others waiting)
        if (wq > 0) {
          if (sums > 0) run = __all_sync(0xffffffffu, mbar_wait(bar(BP_EMPTY + wg), (sums - 1) & 1, abort_flag, 34));
          if (!run) break;
          part[(wq - 1) * 32 + lane] = acc[0];
          mbar_arrive(bar(BP_FULL + wg));
        } else {
          run = __all_sync(0xffffffffu, mbar_wait(bar(BP_FULL + wg), sums & 1, abort_flag, 35));
          if (!run) break;
          acc[0] += part[lane] + part[32 + lane] + part[64 + lane];
          mbar_arrive(bar(BP_EMPTY + wg));
        }
        ++sums;
        const int key = t->tile0 + KPW * wg + lane;
        if (wq == 0 && key < t->lk) {
          const Unit u = unit_at(t);
          const float sum = acc[0];
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
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(BU_EMPTY + k % UST));
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

// [rows, heads, width] bf16 in boxes of 64 columns (zero past width) x
// box_heads x box_rows, 128-byte swizzle
bool encode_rows(CUtensorMap *m, const void *base, int width, int heads, long rows, int box_heads, int box_rows) {
  auto fn = encoder();
  if (!fn) return false;
  cuuint64_t dims[3] = {(cuuint64_t)width, (cuuint64_t)heads, (cuuint64_t)rows};
  cuuint64_t strides[2] = {(cuuint64_t)width * 2, (cuuint64_t)heads * width * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_rows};
  cuuint32_t es[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int NB>
cudaError_t launch_nb(const KeyWeightArgs &p, cudaStream_t stream, const CUtensorMap &mq, const CUtensorMap &mk,
                      const CUtensorMap &mr, const CUtensorMap &mt) {
  static std::atomic<bool> done[kMaxDevicesAttr];
  auto *kernel = relattn_key_weights_tc_kernel<NB>;
  const cudaError_t e = set_max_smem_once(reinterpret_cast<const void *>(kernel), (int)KW_SMEM, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  const long grid = ((long)p.a.max_k + kWalkTile - 1) / kWalkTile * p.a.batch * p.a.Hkv;      // (the host keeps it below 2^31)
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(KWT);
  cfg.dynamicSmemBytes = KW_SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = p.tc == 2 && p.a.E > 0 ? 1 : 0;       // right behind the bias table's kernel
  return cudaLaunchKernelEx(&cfg, kernel, p, mq, mk, mr, mt);
}

}  // namespace

// 0: the shape is not for this kernel; 2: it takes every row; 1: it takes the
// rows past the band (r's rows are not 16-byte multiples, or r is not aligned),
// the tiles kernel the others.  Few tokens leave most of a step's 128 rows empty.
// Measured (us, tiles kernel / this; group 8, two kv heads, E = 1024, 4-bit keys,
// then bf16), 3, 5, 9 and 15 tokens: 64 sequences of 1 to 32 thousand keys 292 / 483,
// 390 / 458, 493 / 461, 600 / 461; 302 / 411, 398 / 400, 499 / 407, 605 / 404; 4 of
// 16 to 64 thousand 57 / 57, 75 / 82, 95 / 82, 113 / 81; 62 / 62, 78 / 72, 97 / 72,
// 117 / 72.  (So this one would be the better from some 8 tokens on.)
int key_weights_tc_kind(const KeyWeightArgs &p) {
  const KernelArgs &a = p.a;
  if (a.group > 128 || a.max_q < 16 || a.total_q < step_tokens(a.group) || !encoder()) return 0;
  // rows are coordinates of the key loads, 32 of them a box
  if (p.k && (p.pages.rows > 0x7fffffffL || p.pages.rows < 32)) return 0;
  if (a.E == 0) return 2;
  return a.rd % 8 == 0 && (reinterpret_cast<uintptr_t>(a.r) & 15u) == 0 ? 2 : 1;
}

cudaError_t launch_key_weights_tc(const KeyWeightArgs &p, cudaStream_t stream) {
  CUtensorMap mq, mk, mr, mt;
  const int group = p.a.group;
  if (!encode_rows(&mq, p.a.q, kHeadDim, p.a.Hq, p.a.total_q, group, step_tokens(group))) return cudaErrorInvalidValue;
  mk = mr = mt = mq;                              // (unused with 4-bit keys, without a bias)
  if (p.k && !encode_rows(&mk, p.k, kHeadDim, p.a.Hkv, p.pages.rows, 1, 32)) return cudaErrorInvalidValue;
  if (p.tc == 2 && p.a.E > 0) {
    if (!encode_rows(&mr, p.a.r, p.a.rd, p.a.Hq, p.a.total_q, group, step_tokens(group))) return cudaErrorInvalidValue;
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
  if (exact <= 2) return launch_nb<1>(p, stream, mq, mk, mr, mt);
  if (exact <= 4) return launch_nb<2>(p, stream, mq, mk, mr, mt);
  if (exact <= 8) return launch_nb<3>(p, stream, mq, mk, mr, mt);
  if (exact <= 16) return launch_nb<4>(p, stream, mq, mk, mr, mt);
  return launch_nb<5>(p, stream, mq, mk, mr, mt);
}

}  // namespace relattn

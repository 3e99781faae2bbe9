// extend_tc.cu -- attention of many new tokens over a cache (relattn_extend) on
// 5th-generation tensor cores: the keys outside the relative-bias band (all of
// them without a bias), and the merge of partial results.
//
// Per row, x(i,j) = s(i) alpha q_i . k_j over the keys that the band kernel leaves
// (page "SGLang and Miles Add Day-0 Support for Inkling", section "Attention
// with Relative Positional Embedding"), softmax, P V.  The band kernel has, per
// row, the keys from a first one on (band_first below).
//
// The work of a CTA: up to 256 rows of one kv head, (token, head of the group)
// pairs in two tiles of 128 that share every K / V tile, against a range of
// 128-key tiles.  Rows packed this way fill the tiles from 16 tokens on (group 8),
// and a tile's rows span few positions, so that little is computed for masked
// keys at the diagonal and the window's edge.  Key tiles start at multiples of 128
// keys and hold whole pages or whole parts of pages: a copy per part, K by one
// warp and V by another.  The tiles of a window's sinks stand before its own.
// What bounds it: the exponentials and the products take 1.8 us for the two
// 128 x 128 tiles of a step (1.4 PFLOP/s over all SMs); with one K / V tile of 64
// KB a step that is also 5.4 TB/s of cache where the rows fill one CTA.
//
// Where the rows fill too few CTAs the keys are cut: each range leaves a
// normalised fp32 partial, which a second kernel merges with the band's.  In one
// piece the band's result (out, lse) is taken up as the start of the running
// maximum and sum, as in fwd_tc_main.cu, whose roles and tensor memory this
// kernel shares:
//   warp 0      q rows, K tiles; warp 2: V tiles; warp 3 idle
//   warp 1      tensor memory; issues S_w = Q_w K^T and O_w += P_w V
//   warps 4-7   softmax of row tile 0, warps 8-11 of row tile 1: thread = row
// Tensor memory: O_w at 128 w, S_w at 256 + 128 w, P_w (bf16) over S_w.
//
// Every wait is bounded; a timeout sets the device error word, the CTA drains
// its own copies / MMAs with bounded waits, frees tensor memory and exits.
#include <cudaTypedefs.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "launch.h"
#include "tc_common.cuh"

namespace relattn {
namespace {

using namespace tc;

constexpr int BM = 128, BN = kTcKeyTile;
constexpr int K_STAGES = 2, V_STAGES = 3;
constexpr int NTHREADS = 384;
constexpr float kRescaleThreshold = 8.f;   // log2 units
constexpr uint32_t TM_O = 0, TM_S = 256;   // O_w at 128 w, S_w at 256 + 128 w

constexpr uint32_t BOX_BYTES = 16384;                // [64 dims x 128 rows], 128-byte rows
constexpr uint32_t TILE_BYTES = 2 * BOX_BYTES;       // 128 dims
constexpr uint32_t SM_Q = 0;                         // Q_0, Q_1
constexpr uint32_t SM_K = SM_Q + 2 * TILE_BYTES;
constexpr uint32_t SM_V = SM_K + K_STAGES * TILE_BYTES;
constexpr uint32_t SM_BAR = SM_V + V_STAGES * TILE_BYTES;
constexpr int B_Q_FULL = 0, B_K_FULL = 1, B_K_EMPTY = B_K_FULL + K_STAGES, B_V_FULL = B_K_EMPTY + K_STAGES,
              B_V_EMPTY = B_V_FULL + V_STAGES, B_S_FULL = B_V_EMPTY + V_STAGES, B_P_FULL = B_S_FULL + 2,
              B_P_HALF = B_P_FULL + 2, B_PV_TAIL = B_P_HALF + 2, B_DRAIN = B_PV_TAIL + 2, B_COUNT = B_DRAIN + 1;
constexpr uint32_t SM_TMEM_SLOT = SM_BAR + B_COUNT * 8;
constexpr uint32_t SM_ABORT = SM_TMEM_SLOT + 8;
constexpr uint32_t SM_TOTAL = SM_ABORT + 8;
constexpr uint32_t SMEM_BYTES = SM_TOTAL + 1024;   // + alignment slack
static_assert(SMEM_BYTES <= 227 * 1024, "shared memory budget");

template <int N>
__device__ __forceinline__ float row_max(const float (&x)[N]) {
  if constexpr (N == 1) {
    return x[0];
  } else if constexpr (N == 2) {
    return fmaxf(x[0], x[1]);
  } else {
    constexpr int M = (N + 2) / 3;
    float t[M];
#pragma unroll
    for (int k = 0; k < M; ++k) {
      if (3 * k + 2 < N) t[k] = fmax3(x[3 * k], x[3 * k + 1], x[3 * k + 2]);
      else if (3 * k + 1 < N) t[k] = fmaxf(x[3 * k], x[3 * k + 1]);
      else t[k] = x[3 * k];
    }
    return row_max(t);
  }
}

__global__ void __launch_bounds__(NTHREADS, 1)
relattn_extend_main_kernel(const __grid_constant__ ExtendTcArgs x, const __grid_constant__ CUtensorMap map_q,
                           const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v) {
  const KernelArgs &a = x.a;
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~uintptr_t(1023));
  const uint32_t sb = smem_addr(smem);
  auto bar = [&](int i) { return sb + SM_BAR + 8u * i; };
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + SM_ABORT);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  // This kernel is launched as the band's programmatic dependent: its CTAs take SMs
  // as the band's leave them.  With partials they need nothing of the band (else
  // the softmax warps wait for it before they read its results), and the merge
  // may be launched behind them.  The first CTA ends after the band's grid, so
  // that whoever waits for this grid has waited for both.
  asm volatile("griddepcontrol.launch_dependents;");
  struct EndAfterBand {
    __device__ ~EndAfterBand() {
      if ((blockIdx.x | blockIdx.y | blockIdx.z) == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
    }
  } end_after_band;

  // ------------------------------------------------------------ work item
  const int kv_head = blockIdx.y, b = blockIdx.z;
  const int split = blockIdx.x % x.splits, tile = x.row_tiles - 1 - blockIdx.x / x.splits;   // longest first
  const int cq = a.cu_q[b], ck = a.cu_k[b];
  const int Lq = a.cu_q[b + 1] - cq, Lk = a.cu_k[b + 1] - ck;
  if (Lq < 0 || Lk < Lq || Lq > a.max_q || Lk > a.max_k || !extend_rows_ok(a, cq, Lq, ck, Lk)) {
    if (tid == 0) atomicOr(a.err, kDevErrSeqlens);
    return;
  }
  const int TT = x.tokens;                            // tokens of a row tile
  const int tok0 = 2 * TT * tile;
  if (tok0 >= Lq) return;
  const ExtendTiles T = extend_tiles(x, tok0, Lq, Lk);
  const int ntok = T.ntok, nw = ntok > TT ? 2 : 1, off = Lk - Lq, p0 = T.p0, p_last = T.p_last;
  const int b_first = T.b_first, far = T.far, w_lo = T.w_lo, n_sink = T.n_sink, n_all = T.n_all;
  auto key0 = [&](int v) { return BN * (v < n_sink ? v : w_lo + v - n_sink); };
  const int v_end = min(n_all, (split + 1) * x.chunk), n_main = max(0, v_end - split * x.chunk);
  auto tile_key = [&](int i) { return key0(v_end - 1 - i); };      // nearest first
  const bool partial = x.slots > 1;
  const bool init = x.band != 0 && !partial;                // go on from the band's out / lse
  const size_t rows_all = (size_t)a.total_q * a.Hq;
  if (n_main <= 0) {
    if (partial)                                                    // a range without keys
      for (int i = tid; i < ntok * a.group; i += NTHREADS)
        a.lse_part[split * rows_all + (size_t)(cq + tok0 + i / a.group) * a.Hq + kv_head * a.group + i % a.group] = -INFINITY;
    return;                                                         // (or the band's result is final)
  }

  // ------------------------------------------------------------ setup
  if (tid == 0) {
    mbar_init(bar(B_Q_FULL), 1);
    for (int i = 0; i < K_STAGES; ++i) {
      mbar_init(bar(B_K_FULL + i), 1);
      mbar_init(bar(B_K_EMPTY + i), 1);
    }
    for (int i = 0; i < V_STAGES; ++i) {
      mbar_init(bar(B_V_FULL + i), 1);
      mbar_init(bar(B_V_EMPTY + i), 1);
    }
    for (int w = 0; w < 2; ++w) {
      mbar_init(bar(B_S_FULL + w), 1);
      mbar_init(bar(B_P_FULL + w), 128);
      mbar_init(bar(B_P_HALF + w), 128);
      mbar_init(bar(B_PV_TAIL + w), 1);
    }
    mbar_init(bar(B_DRAIN), 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 1) {
    tmem_alloc(sb + SM_TMEM_SLOT, 512);
    tmem_relinquish();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&map_q);
    prefetch_tmap(&map_k);
    prefetch_tmap(&map_v);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + SM_TMEM_SLOT);
  int issued_k = 0, issued_v = 0;   // the copies (to drain them if the CTA gives up)
  bool q_issued = false;

  // the copies of the tile at key k0, one a lane (lane = part of the tile); a
  // part that no row needs, or whose page lies outside the pool, reads zeros
  auto part_needed = [&](int k0) -> bool {
    const int p = k0 + lane * x.box;
    return lane * x.box < BN && p <= p_last && (a.window <= 0 || p + x.box > p0 - a.window + 1 || p < a.sink);
  };
  auto part_page = [&](int k0) -> int {
    if (a.block_table == nullptr || !part_needed(k0)) return 0;
    return __ldg(a.block_table + (size_t)b * a.max_pages + (k0 + lane * x.box) / a.page_size);
  };
  auto copy_parts = [&](uint32_t dst, const CUtensorMap *map, int k0, int pg, uint32_t br) {
    const int p = k0 + lane * x.box;
    int row = -BN;
    if (part_needed(k0)) {
      if (a.block_table == nullptr) row = ck + p;
      else if ((unsigned)pg < (unsigned)a.num_pages) row = pg * a.page_size + p % a.page_size;
      else atomicOr(a.err, kDevErrSeqlens);
    }
    if (lane == 0) mbar_arrive_expect_tx(br, TILE_BYTES);
    __syncwarp();
    if (lane * x.box < BN) {
      tma_load_3d(dst + lane * x.box * 128, map, 0, kv_head, row, br);
      tma_load_3d(dst + BOX_BYTES + lane * x.box * 128, map, 64, kv_head, row, br);
    }
    __syncwarp();
  };

  if (warp < 4) {
    if (warp == 0) {
      // ====================================================== q rows and K tiles
      if (lane == 0) {
        // a box: TT tokens x the group's heads x 64 dims (rows past the tokens
        // hold other rows or zeros, rows past the box whatever was there)
        mbar_arrive_expect_tx(bar(B_Q_FULL), (uint32_t)(nw * x.q_bytes));
        for (int w = 0; w < nw; ++w) {
          tma_load_3d(sb + SM_Q + w * TILE_BYTES, &map_q, 0, kv_head * a.group, cq + tok0 + w * TT, bar(B_Q_FULL));
          tma_load_3d(sb + SM_Q + w * TILE_BYTES + BOX_BYTES, &map_q, 64, kv_head * a.group, cq + tok0 + w * TT,
                      bar(B_Q_FULL));
        }
        q_issued = true;
      }
      __syncwarp();
      int page = part_page(tile_key(0));
      for (int i = 0; i < n_main; ++i) {
        const int st = i % K_STAGES;
        if (i >= K_STAGES && !__all_sync(0xffffffffu, mbar_wait_suspend(bar(B_K_EMPTY + st), ((i / K_STAGES) - 1) & 1, abort_flag, 41)))
          break;
        // (test hook: a skipped tile is never loaded)
        if (i != a.test_skip_k_tile) copy_parts(sb + SM_K + st * TILE_BYTES, &map_k, tile_key(i), page, bar(B_K_FULL + st));
        issued_k = i + 1;
        if (i + 1 < n_main) page = part_page(tile_key(i + 1));
      }
    } else if (warp == 2) {
      // ====================================================== V tiles
      int page = part_page(tile_key(0));
      for (int i = 0; i < n_main; ++i) {
        const int st = i % V_STAGES;
        if (i >= V_STAGES && !__all_sync(0xffffffffu, mbar_wait_suspend(bar(B_V_EMPTY + st), ((i / V_STAGES) - 1) & 1, abort_flag, 42)))
          break;
        copy_parts(sb + SM_V + st * TILE_BYTES, &map_v, tile_key(i), page, bar(B_V_FULL + st));
        issued_v = i + 1;
        if (i + 1 < n_main) page = part_page(tile_key(i + 1));
      }
    } else if (warp == 1) {
      // ====================================================== MMA issuer
      // The whole warp runs this (descriptors stay warp-uniform); each MMA and
      // commit is issued by one elected lane.
      {
        const uint32_t id_s = idesc_bf16_f32(BM, BN, 0, 0);     // S: Q (smem, K-major) x K (smem, K-major)
        const uint32_t id_o = idesc_bf16_f32(BM, 128, 0, 1);    // O: P (tmem) x V (smem, MN-major)
        // descriptor bases: +2 per 32 bytes of a 128-byte row, +1024 per 16 KB
        // box, +128 per 16 V rows, +2048 per 32 KB tile
        const uint64_t qd0 = smem_desc_sw128(sb + SM_Q, 16, 1024);
        const uint64_t kd0 = smem_desc_sw128(sb + SM_K, 16, 1024);
        const uint64_t vd0 = smem_desc_sw128(sb + SM_V, BOX_BYTES, 1024);
        bool ok = mbar_wait_warp(bar(B_Q_FULL), 0, abort_flag, 43);
        auto issue_s = [&](int w, int i) -> bool {   // S_w of main tile i
          const int ks = i % K_STAGES;
          if (w == 0 && !mbar_wait_warp(bar(B_K_FULL + ks), (i / K_STAGES) & 1, abort_flag, 44)) return false;
          const uint64_t qd = qd0 + (uint64_t)(w * (TILE_BYTES >> 4));
          const uint64_t kd = kd0 + (uint64_t)(ks * (TILE_BYTES >> 4));
          const uint32_t d = tmem + TM_S + 128u * (uint32_t)w;
          mma_ss_e<0>(d, qd + 0, kd + 0, id_s);
          mma_ss_e<1>(d, qd + 2, kd + 2, id_s);
          mma_ss_e<1>(d, qd + 4, kd + 4, id_s);
          mma_ss_e<1>(d, qd + 6, kd + 6, id_s);
          mma_ss_e<1>(d, qd + 1024, kd + 1024, id_s);
          mma_ss_e<1>(d, qd + 1026, kd + 1026, id_s);
          mma_ss_e<1>(d, qd + 1028, kd + 1028, id_s);
          mma_ss_e<1>(d, qd + 1030, kd + 1030, id_s);
          mma_commit_e(bar(B_S_FULL + w));
          return true;
        };
        // O_w += P_w V of main tile i, keys 0..63 once the softmax has written
        // that half of P, keys 64..127 once it has written all of it
        auto issue_pv = [&](int w, int i) -> bool {
          const int vs = i % V_STAGES;
          if (w == 0 && !mbar_wait_warp(bar(B_V_FULL + vs), (i / V_STAGES) & 1, abort_flag, 45)) return false;
          if (!mbar_wait_warp(bar(B_P_HALF + w), i & 1, abort_flag, 50)) return false;
          tc_fence_after();
          const uint64_t vd = vd0 + (uint64_t)(vs * (TILE_BYTES >> 4));
          const uint32_t o = tmem + TM_O + 128u * (uint32_t)w, pa = tmem + TM_S + 128u * (uint32_t)w;
          if (i > 0 || init) mma_ts_e<1>(o, pa + 0, vd + 0, id_o);
          else mma_ts_e<0>(o, pa + 0, vd + 0, id_o);
          mma_ts_e<1>(o, pa + 8, vd + 128, id_o);
          mma_ts_e<1>(o, pa + 16, vd + 256, id_o);
          mma_ts_e<1>(o, pa + 24, vd + 384, id_o);
          if (!mbar_wait_warp(bar(B_P_FULL + w), i & 1, abort_flag, 46)) return false;
          tc_fence_after();
          mma_ts_e<1>(o, pa + 32, vd + 512, id_o);
          mma_ts_e<1>(o, pa + 40, vd + 640, id_o);
          mma_ts_e<1>(o, pa + 48, vd + 768, id_o);
          mma_ts_e<1>(o, pa + 56, vd + 896, id_o);
          if (i == n_main - 1) mma_commit_e(bar(B_PV_TAIL + w));
          return true;
        };
        if (ok) ok = issue_s(0, 0);
        if (ok && nw > 1) ok = issue_s(1, 0);
        // S_w(i+1) goes into the buffer whose P_w(i) PV_w(i) has just been
        // issued to read: the tensor core runs them in order
        for (int i = 0; i < n_main && ok; ++i) {
          for (int w = 0; w < nw && ok; ++w) {
            if (!(ok = issue_pv(w, i))) break;
            if (i + 1 < n_main) ok = issue_s(w, i + 1);
          }
        }
        // drain: every MMA issued above has finished before TMEM is released
        mma_commit_e(bar(B_DRAIN));
        volatile int keep_waiting = 0;
        mbar_wait(bar(B_DRAIN), 0, &keep_waiting, 47, 400000000ll);
      }
      __syncwarp();
    }
  } else {
    // ======================================================== softmax
    const int w = (warp - 4) >> 2;               // row tile
    const int wq = warp & 3;                     // lane quarter (TMEM lanes 32 wq ..)
    const int a_row = 32 * wq + lane;            // row == TMEM lane
    const uint32_t lane_base = (uint32_t)(32 * wq) << 16;
    // the row: a token and a head (rows past the tile's tokens repeat others).
    // Only its position stays in a register through the tiles.
    auto row_token = [&]() { return tok0 + min(w * TT + min(a_row / a.group, TT - 1), ntok - 1); };
    auto row_head = [&]() { return kv_head * a.group + a_row % a.group; };
    const int pos = off + row_token();
    const float sc = log_scale(pos, a.inv_ln_base);
    const float cqk = a.alpha_log2e * sc;        // > 0 (checked on the host)
    const bool releaser = (w == nw - 1) && (wq == 0) && (lane == 0);   // frees K / V stages
    const uint32_t obuf = tmem + lane_base + TM_O + 128u * (uint32_t)w;
    const uint32_t sbuf = tmem + lane_base + TM_S + 128u * (uint32_t)w;
    auto warp_wait = [&](uint32_t br, uint32_t parity, int site) -> bool {
      const bool r = mbar_wait(br, parity, abort_flag, site);
      return __all_sync(0xffffffffu, r);
    };

    float m_ref = -INFINITY, l = 0.f;
    if (init) {
      // the band's state: m = lse log2(e), l = 1, O = what it left in out
      asm volatile("griddepcontrol.wait;" ::: "memory");
      const int tok = row_token(), h = row_head();
      const float lse0 = a.lse[(size_t)h * a.total_q + cq + tok];
      const float2 ups = reinterpret_cast<const float2 *>(x.carry)[(size_t)(cq + tok) * a.Hq + h];
      if (lse0 != -INFINITY) {
        m_ref = lse0 * kLog2e;
        l = 1.f;
      }
      const uint4 *src = reinterpret_cast<const uint4 *>(a.out + ((size_t)(cq + tok) * a.Hq + h) * kHeadDim);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float up = c < 2 ? ups.x : ups.y;
        uint32_t r[32];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 v = src[4 * c + i];
          const uint32_t pr[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&pr[k]));
            r[8 * i + 2 * k] = __float_as_uint(f.x * up);
            r[8 * i + 2 * k + 1] = __float_as_uint(f.y * up);
          }
        }
        __syncwarp();
        tmem_st32(obuf + 32u * c, r);
      }
      tmem_wait_st();
    }

    bool ok = true;
    for (int i = 0; i < n_main && w < nw; ++i) {
      if (!(ok = warp_wait(bar(B_S_FULL + w), i & 1, 48))) break;
      if (releaser) {
        // S_1(i) landed: K(i) is read by both heads; S_1(i) was issued after
        // PV_1(i-1), so V(i-1) is free too
        mbar_arrive(bar(B_K_EMPTY + i % K_STAGES));
        if (i > 0) mbar_arrive(bar(B_V_EMPTY + (i - 1) % V_STAGES));
      }
      tc_fence_after();
      if (w == 0 && tile_key(i) + BN > Lk) {
        // values past the last key (rows of no key, of another sequence): zero, so
        // that a NaN there does not meet a weight of zero.  Tile 0's product is
        // issued first, so this half of its P guards tile 1's as well.
        if (!(ok = warp_wait(bar(B_V_FULL + i % V_STAGES), (i / V_STAGES) & 1, 51))) break;
        if (tile_key(i) + a_row >= Lk) {
          uint4 *v = reinterpret_cast<uint4 *>(smem + SM_V + (i % V_STAGES) * TILE_BYTES + a_row * 128);
#pragma unroll
          for (int k = 0; k < 8; ++k) v[k] = v[BOX_BYTES / 16 + k] = make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
      }
      float x_[128];   // raw scores; the scale is applied inside the exponent
      __syncwarp();
      tmem_ld32f<0>(sbuf + 0u, x_);
      tmem_ld32f<32>(sbuf + 32u, x_);
      tmem_ld32f<64>(sbuf + 64u, x_);
      tmem_ld32f<96>(sbuf + 96u, x_);
      tmem_wait_ld_f<0>(x_);
      reg_dep_f<32>(x_);
      reg_dep_f<64>(x_);
      reg_dep_f<96>(x_);
      const int j0 = tile_key(i);
      // (the CTA's rows see all of the tile unless it passes the first row's last
      // key or starts before the last row's window)
      const bool need_mask = j0 + BN - 1 > min(p0, b_first - 1) || (a.window > 0 && j0 < p_last - a.window + 1);
      if (need_mask) {
        // the row's keys: its window below the band's first, and the sinks that its
        // window has left behind, as a bit a key
        int pp = pos;
        asm volatile("" : "+r"(pp));             // (worked out here: kept, they would spill)
        const int first = extend_row_first(x, pp), lo = a.window > 0 ? max(0, pp - a.window + 1) : 0;
        const int kmin = lo - j0, kend = min(pp + 1, first) - j0;
        const int kfar = j0 < far ? min(min(a.sink, lo), first) - j0 : 0;
        auto below = [](int n) -> uint32_t { return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u; };
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint32_t seen = (below(kend - 32 * c) & ~below(kmin - 32 * c)) | below(kfar - 32 * c);
#pragma unroll
          for (int k = 0; k < 32; ++k) x_[32 * c + k] = (seen >> k) & 1u ? x_[32 * c + k] : -INFINITY;
        }
      }
      // P (bf16 pairs) of keys 32c .. 32c + 31 over S_w columns [16c, 16c + 16)
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
      auto p_chunk = [&](int c, float mu) {
        uint32_t pk[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          float y0, y1;
          ffma2(y0, y1, x_[32 * c + 2 * k], x_[32 * c + 2 * k + 1], cqk, cqk, -mu, -mu);
          const float e0 = fast_exp2(y0), e1 = fast_exp2(y1);
          ffma2(acc[2 * (k & 1)], acc[2 * (k & 1) + 1], e0, e1, 1.f, 1.f, acc[2 * (k & 1)], acc[2 * (k & 1) + 1]);
          pk[k] = pack_bf16x2(e0, e1);
        }
        __syncwarp();
        tmem_st16(sbuf + 16u * (uint32_t)c, pk);
      };
      // Where every row of the warp has a running max, the first half of P is
      // computed against it before the tile's own max is known: that max only
      // decides whether the running max moves (a rare rescale), and a warp in
      // which some row's does recomputes the half.  The values are the same as
      // computing the max first.
      const bool spec = __all_sync(0xffffffffu, m_ref != -INFINITY);
      if (spec) {
        p_chunk(0, m_ref);
        p_chunk(1, m_ref);
      }
      const float mx = row_max(x_) * cqk;
      float corr = 1.f;
      bool rescale_o = false, moved = false;
      if (mx > m_ref + kRescaleThreshold || (m_ref == -INFINITY && mx != -INFINITY)) {
        const float m_new = fmaxf(m_ref, mx);
        corr = (m_ref == -INFINITY) ? 0.f : fast_exp2(m_ref - m_new);
        rescale_o = (m_ref != -INFINITY) && (i > 0 || init);
        l *= corr;
        m_ref = m_new;
        moved = true;
      }
      const float m_use = (m_ref == -INFINITY) ? 0.f : m_ref;
      if (!spec || __any_sync(0xffffffffu, moved)) {
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[k] = 0.f;
        p_chunk(0, m_use);
        p_chunk(1, m_use);
      }
      // O_w is touched only when a row of this warp needs a rescale; PV_w(i-1)
      // has finished (S_w(i) was issued after it).  TMEM loads / stores are
      // warp-collective: the whole warp rescales (rows that need not: by 1).
      // It happens before the first half of P is handed over: PV_w(i) starts then.
      if (__any_sync(0xffffffffu, rescale_o)) {
        const float cf = rescale_o ? corr : 1.f;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t r[32];
          __syncwarp();
          tmem_ld32(obuf + 32u * c, r);
          tmem_wait_ld(r);
#pragma unroll
          for (int k = 0; k < 32; ++k) r[k] = __float_as_uint(__uint_as_float(r[k]) * cf);
          __syncwarp();
          tmem_st32(obuf + 32u * c, r);
        }
      }
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(bar(B_P_HALF + w));
      p_chunk(2, m_use);
      p_chunk(3, m_use);
      l += (acc[0] + acc[1]) + (acc[2] + acc[3]);
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(bar(B_P_FULL + w));
    }
    // ---- epilogue
    if (w < nw) {
      if (ok) ok = warp_wait(bar(B_PV_TAIL + w), 0, 49);
      if (ok) {
        tc_fence_after();
        const int tok = row_token(), h = row_head(), tt = a_row / a.group;
        const bool valid = tt < TT && w * TT + tt < ntok;
        const size_t qrow = (size_t)(cq + tok) * a.Hq + h;
        const float inv = l > 0.f ? 1.f / l : 0.f;
        const float row_lse = l > 0.f ? (m_ref + __log2f(l)) * kLn2 : -INFINITY;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t r[32];
          __syncwarp();
          tmem_ld32(obuf + 32u * c, r);
          tmem_wait_ld(r);
          if (valid && partial) {
            float4 *dst = reinterpret_cast<float4 *>(a.o_part + (split * rows_all + qrow) * kHeadDim + 32 * c);
#pragma unroll
            for (int k = 0; k < 8; ++k)
              dst[k] = make_float4(__uint_as_float(r[4 * k]) * inv, __uint_as_float(r[4 * k + 1]) * inv,
                                   __uint_as_float(r[4 * k + 2]) * inv, __uint_as_float(r[4 * k + 3]) * inv);
          } else if (valid) {
            __nv_bfloat16 *dst = a.out + qrow * kHeadDim + 32 * c;
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              uint4 v;
              v.x = pack_bf16x2(__uint_as_float(r[8 * k + 0]) * inv, __uint_as_float(r[8 * k + 1]) * inv);
              v.y = pack_bf16x2(__uint_as_float(r[8 * k + 2]) * inv, __uint_as_float(r[8 * k + 3]) * inv);
              v.z = pack_bf16x2(__uint_as_float(r[8 * k + 4]) * inv, __uint_as_float(r[8 * k + 5]) * inv);
              v.w = pack_bf16x2(__uint_as_float(r[8 * k + 6]) * inv, __uint_as_float(r[8 * k + 7]) * inv);
              *reinterpret_cast<uint4 *>(dst + 8 * k) = v;
            }
          }
        }
        if (valid) {
          if (partial) a.lse_part[split * rows_all + qrow] = row_lse;
          else a.lse[(size_t)h * a.total_q + cq + tok] = row_lse;
        }
      }
    }
  }

  // ------------------------------------------------------------ teardown
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && *abort_flag) record_timeout(a.err, *abort_flag);
  if (warp == 0 && lane == 0 && *abort_flag) {
    // the CTA gave up: let the producer's own copies land before shared memory
    // goes away (bounded waits, not cut short by the abort)
    volatile int keep_waiting = 0;
    if (q_issued) mbar_wait(bar(B_Q_FULL), 0, &keep_waiting, 2, 400000000ll);
    for (int i = max(0, issued_k - K_STAGES); i < issued_k; ++i)
      if (i != a.test_skip_k_tile)
        mbar_wait(bar(B_K_FULL + i % K_STAGES), (i / K_STAGES) & 1, &keep_waiting, 2, 400000000ll);
  }
  if (warp == 2 && lane == 0 && *abort_flag) {
    volatile int keep_waiting = 0;
    for (int i = max(0, issued_v - V_STAGES); i < issued_v; ++i)
      mbar_wait(bar(B_V_FULL + i % V_STAGES), (i / V_STAGES) & 1, &keep_waiting, 2, 400000000ll);
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

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
    // 32 slots at a time, those of them that hold something: four loads in flight
    for (int s0 = 32 * wi; s0 < slots; s0 += 32 * RW) {
      const float ls = s0 + lane < slots ? a.lse_part[(long)(s0 + lane) * rows + row] : -INFINITY;
      const float w = exp2f((ls - m) * kLog2e);
      for (unsigned full = __ballot_sync(0xffffffffu, ls != -INFINITY); full;) {
        float4 v[4];
        float f[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int i = full ? __ffs(full) - 1 : 0;
          f[k] = full ? __shfl_sync(0xffffffffu, w, i) : 0.f;
          v[k] = full ? *reinterpret_cast<const float4 *>(a.o_part + ((long)(s0 + i) * rows + row) * kHeadDim + lane * 4)
                      : make_float4(0.f, 0.f, 0.f, 0.f);
          full &= full - 1;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          z += f[k];
          acc.x = fmaf(f[k], v[k].x, acc.x);
          acc.y = fmaf(f[k], v[k].y, acc.y);
          acc.z = fmaf(f[k], v[k].z, acc.z);
          acc.w = fmaf(f[k], v[k].w, acc.w);
        }
      }
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

PFN_cuTensorMapEncodeTiled_v12000 encoder() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = []() -> PFN_cuTensorMapEncodeTiled_v12000 {
    cudaDriverEntryPointQueryResult q;
    void *p = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    return nullptr;
  }();
  return fn;
}

// [rows, heads, 128] bf16 -> box of 64 dims x box_heads heads x box_rows rows, 128-byte swizzle
bool encode_rows(CUtensorMap *m, const void *base, int heads, int rows, int box_heads, int box_rows) {
  auto fn = encoder();
  if (!fn) return false;
  cuuint64_t dims[3] = {128, (cuuint64_t)heads, (cuuint64_t)rows};
  cuuint64_t strides[2] = {256, (cuuint64_t)heads * 256};
  cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_rows};
  cuuint32_t es[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(base), dims, strides, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

cudaError_t launch_extend_main(const ExtendTcArgs &args, cudaStream_t stream) {
  ExtendTcArgs x = args;
  const KernelArgs &a = x.a;
  const int q_tokens = std::min(x.tokens, a.total_q);        // a box stays inside the tensor
  x.box = extend_box(a);
  x.q_bytes = 2 * 64 * 2 * a.group * q_tokens;
  CUtensorMap mq, mk, mv;
  if (!encode_rows(&mq, a.q, a.Hq, a.total_q, a.group, q_tokens) || !encode_rows(&mk, a.k, a.Hkv, a.kv_rows, 1, x.box) ||
      !encode_rows(&mv, a.v, a.Hkv, a.kv_rows, 1, x.box))
    return cudaErrorInvalidValue;
  static std::atomic<bool> attr_set[kMaxDevicesAttr];
  cudaError_t e = set_max_smem_once(reinterpret_cast<const void *>(relattn_extend_main_kernel), (int)SMEM_BYTES, attr_set);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(x.row_tiles * x.splits), a.Hkv, a.batch);
  cfg.blockDim = dim3(NTHREADS);
  cfg.dynamicSmemBytes = SMEM_BYTES;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = x.band != 0 ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, relattn_extend_main_kernel, x, mq, mk, mv);
}

cudaError_t launch_extend_combine(const KernelArgs &a, int slots, bool pdl, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  const bool wide = slots > 32;                  // (more loads of a row in flight: 8 warps a row, 32 slots each)
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

// extend_band.cu -- the relative-bias band of relattn_extend on 5th-generation
// tensor cores: for the row at position i the keys from extend_band_first (of its
// pair of row tiles in extend_tc.cu) to i, x(i,j) = s(i) (alpha q_i.k_j + [0 <= i-j
// < E] r_i . P[:, i-j]) (page "SGLang and Miles Add Day-0 Support for Inkling",
// section "Attention with Relative Positional Embedding"), softmax, P V.  The keys
// before are extend_tc.cu's.
//
// An item is up to 128 rows of one kv head, (token, head of the group) pairs of
// consecutive tokens, against 64-key steps from the diagonal backwards (or a
// piece of them).  A CTA per SM walks the items; its rings run on from item to
// item, so that the next item's copies and first products overlap the end of
// this one.  Per step: S = Q K^T (Q in tensor memory), R = r . P for the 64
// distances that the step adds, softmax, O += P V.
//
// The shear.  Row i needs R at the distances i - j of the step's keys, another
// offset for every token.  R goes from tensor memory to shared memory, [distance]
// [row] in a ring of 160 (or 192) distances: the lanes of a warp are rows, so
// that writing a distance and reading row by row at any offset are both free of
// bank conflicts, and one load a key replaces the six select stages of a shift in
// registers (fwd_tc.cu, where they are half of the instructions).  The first 32
// distances of the ring are held twice, behind its end: a thread's 32 keys are
// then 32 loads at constant offsets from one address.  A row is read and written
// by the two threads that share it, so their two warps meet, not the CTA.
// A step adds 64 distances and needs those of 64 keys and the block's tokens: 160
// hold up to 32 tokens (groups of 4 and more: 128 rows), 192 up to 64.  From step to
// step a row's two threads have met before either writes again; at an item's start they
// have not, and what both would write to the same place is written once (extend_ring.h).
//
// The list of items is counted from the lengths on the device, so that a batch whose
// sequences are far shorter than the longest has no empty ones (4096 tokens of one
// sequence and one of 63 others: the band 428 us with a place in the list for every
// block that a sequence might have, 117 so).
//
// Warps: 0: r rows, P slices and K tiles; 1: tensor memory, issues the products;
// 2: q rows and V tiles; 4-11: softmax, thread = row, warps 4-7 keys 0-31 of a
// step, warps 8-11 keys 32-63.
// Tensor memory: Q [0,64), O [64,192), S 2 x 64 [192,320) (P in bf16 over it),
// R 2 x 64 [320,448).
// What bounds it: a step's chain -- S and R out of tensor memory, R's way through
// shared memory, the exchange of the maximum between a row's two threads, the
// exponentials, P -- takes 2,000 cycles; issue slots 41 %, tensor pipe 25 % (4 x 8192
// tokens, Hq 16 / Hkv 2, r_dim 64, E 1024, window 4096: 553 us; R issued with its own
// step instead of one ahead 710, four softmax warpgroups or P before the step's
// maximum no faster).
//
// Every wait is bounded; a timeout sets the device error word, the CTA drains
// its own copies / MMAs with bounded waits, frees tensor memory and exits.
#include <cudaTypedefs.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "extend_ring.h"
#include "launch.h"
#include "tc_common.cuh"

namespace relattn {
namespace {

using namespace tc;

constexpr int BM = 128;          // rows of an item at most
constexpr int HN = 64;           // keys of a step, distances of an r.P chunk
constexpr int NTHREADS = 384;
constexpr uint32_t kRegsSupport = 88, kRegsSoftmax = 208;
static_assert(128 * kRegsSupport + 256 * kRegsSoftmax <= NTHREADS * 168, "register split");
constexpr float kRescaleThreshold = 8.f;   // log2 units
constexpr uint32_t TM_Q = 0, TM_O = 64, TM_S = 192, TM_R = 320;

constexpr uint32_t STAGE = 16384;          // 64 keys x 128 dims: two boxes of 64 dims; or 64 dims of 128 q rows
constexpr uint32_t KV_BOX = 8192;
constexpr int K_STAGES = 2, P_STAGES = 2;

template <bool WIDE>
struct Lay {
  static constexpr int RING = WIDE ? 192 : 160, SLOTS = RING / 32;
  static constexpr int V_STAGES = WIDE ? 2 : 3;
  static constexpr uint32_t SM_K = 0;
  static constexpr uint32_t SM_V = SM_K + K_STAGES * STAGE;
  static constexpr uint32_t SM_RT = SM_V + V_STAGES * STAGE;             // r rows, 128 bytes each
  static constexpr uint32_t SM_PS = SM_RT + 16384;                       // P slices
  static constexpr uint32_t SM_R = SM_PS + P_STAGES * 8192;              // fp32 [RING + 32][128]
  static constexpr uint32_t SM_XCH = SM_R + (RING + 32) * BM * 4;        // row exchange [2][2][128] f32
  static constexpr uint32_t SM_BAR = SM_XCH + 2 * 2 * 128 * 4;
};
constexpr int B_K_FULL = 0, B_K_EMPTY = B_K_FULL + K_STAGES, B_V_FULL = B_K_EMPTY + K_STAGES, B_V_EMPTY = B_V_FULL + 3,
              B_PS_FULL = B_V_EMPTY + 3, B_PS_EMPTY = B_PS_FULL + P_STAGES, B_RT_FULL = B_PS_EMPTY + P_STAGES,
              B_RT_EMPTY = B_RT_FULL + 1, B_S_FULL = B_RT_EMPTY + 1, B_P_FULL = B_S_FULL + 2, B_R_FULL = B_P_FULL + 2,
              B_R_FREE = B_R_FULL + 2, B_XCH = B_R_FREE + 2, B_RW = B_XCH + 4, B_TAIL = B_RW + 4, B_DRAIN = B_TAIL + 1,
              B_COUNT = B_DRAIN + 1;
template <bool WIDE>
constexpr uint32_t smem_bytes() { return Lay<WIDE>::SM_BAR + B_COUNT * 8 + 16 + 1024; }
static_assert(smem_bytes<false>() <= 227 * 1024 && smem_bytes<true>() <= 227 * 1024, "shared memory budget");

struct BandArgs {
  ExtendTcArgs x;
  int tokens;             // of an item
  int n_items;            // at most (sequences that do not overlap)
  int box, row_bytes;     // rows of a K / V copy; bytes of 64 dims (or channels) of an item's q (or r) rows
};

struct Item {
  int b, g, cq, ck, lk, p0, p_last, tok0, ntok;
  int first, steps;       // first 64-key block (the nearest), steps backwards
  int slot;
  int c_start, c_first;   // r.P chunks: the oldest that step 0 reads, the newest
};

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

template <bool WIDE>
__global__ void __launch_bounds__(NTHREADS, 1)
relattn_extend_band_kernel(const __grid_constant__ BandArgs ba, const __grid_constant__ CUtensorMap map_q,
                           const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                           const __grid_constant__ CUtensorMap map_r, const __grid_constant__ CUtensorMap map_p) {
  using L = Lay<WIDE>;
  constexpr int V_STAGES = L::V_STAGES;
  const KernelArgs &a = ba.x.a;
  extern __shared__ uint8_t smem_raw[];
  // (with partials the kernel of the other keys may run beside this one)
  asm volatile("griddepcontrol.launch_dependents;");
  uint8_t *smem = smem_raw + ((1024u - (smem_addr(smem_raw) & 1023u)) & 1023u);
  const uint32_t sb = smem_addr(smem);
  auto bar = [&](int i) { return sb + L::SM_BAR + 8u * i; };
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::SM_BAR + B_COUNT * 8 + 8);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  // ------------------------------------------------------------ work items
  // (sequence, token block from the last backwards, kv head, piece), the list without
  // gaps, every grid-th one from the CTA's number on.  Every role walks the same list
  // and its counters run on.  32 sequences at a time lie in the lanes of a warp.
  Item I{};
  int gs = 0, vb = 0, ob = 0, n_it = 0;   // steps, V slots, chunks and items (with steps) so far
  int c0 = -32, c_run = 0, c_all = 0;     // first of the sequences, items before them, theirs
  int s_cq = 0, s_ck = 0, s_Lq = 0, s_Lk = 0, s_upto = 0;      // lane's sequence, items up to its end
  const int per_block = a.Hkv * ba.x.band_pieces;
  auto next_item = [&](int n) -> bool {   // the list's n-th (n grows); its steps may be 0
    if (n >= ba.n_items) return false;
    while (n >= c_run + c_all) {
      c_run += c_all;
      c0 += 32;
      if (c0 >= a.batch) return false;
      s_Lq = 0;
      if (c0 + lane < a.batch) {
        s_cq = __ldg(a.cu_q + c0 + lane);
        s_ck = __ldg(a.cu_k + c0 + lane);
        s_Lq = __ldg(a.cu_q + c0 + lane + 1) - s_cq;
        s_Lk = __ldg(a.cu_k + c0 + lane + 1) - s_ck;
        if (s_Lq < 0 || s_Lk < s_Lq || s_Lq > a.max_q || s_Lk > a.max_k || !extend_rows_ok(a, s_cq, s_Lq, s_ck, s_Lk)) {
          atomicOr(a.err, kDevErrSeqlens);
          s_Lq = 0;
        }
      }
      s_upto = (s_Lq + ba.tokens - 1) / ba.tokens * per_block;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int u = __shfl_up_sync(0xffffffffu, s_upto, o);
        if (lane >= o) s_upto += u;
      }
      c_all = __shfl_sync(0xffffffffu, s_upto, 31);
    }
    const int i = __ffs(__ballot_sync(0xffffffffu, c_run + s_upto > n)) - 1;
    I.b = c0 + i;
    I.cq = __shfl_sync(0xffffffffu, s_cq, i);
    I.ck = __shfl_sync(0xffffffffu, s_ck, i);
    I.lk = __shfl_sync(0xffffffffu, s_Lk, i);
    const int Lq = __shfl_sync(0xffffffffu, s_Lq, i);
    const int left = c_run + __shfl_sync(0xffffffffu, s_upto, i) - 1 - n;      // items of the sequence behind it
    const int piece = ba.x.band_pieces - 1 - left % ba.x.band_pieces;
    I.g = a.Hkv - 1 - left / ba.x.band_pieces % a.Hkv;
    I.tok0 = left / per_block * ba.tokens;      // (last block first)
    I.ntok = min(ba.tokens, Lq - I.tok0);
    I.p0 = I.lk - Lq + I.tok0;
    I.p_last = I.p0 + I.ntok - 1;
    // keys from the band's first (or the window's, unless sinks lie in the band before it)
    // on; an item lies within a pair of row tiles, whose tokens are a multiple of its own
    const int j_lo = a.window > 0 ? max(0, I.p0 - a.window + 1) : 0;
    const int b0 = extend_band_first(a, I.p0 - I.tok0 % (2 * ba.x.tokens));
    const int low = (min(a.sink, j_lo) > b0 ? b0 : max(b0, j_lo)) / HN;
    I.first = I.p_last / HN - piece * ba.x.band_steps;
    I.steps = min(ba.x.band_steps, max(0, I.first - low + 1));
    I.slot = piece;
    const int D0 = I.p0 - HN * I.first;
    const BandChunks chunks = band_chunks(D0, I.ntok);
    I.c_first = chunks.first;
    I.c_start = chunks.start;
    return true;
  };
  auto finish_item = [&]() {
    if (I.steps == 0) return;
    gs += I.steps;
    vb += I.steps + 2;
    ob += I.c_first + I.steps - I.c_start;          // (a chunk a step)
    ++n_it;
  };

  // ------------------------------------------------------------ setup
  if (tid == 0) {
    for (int i = 0; i < K_STAGES; ++i) {
      mbar_init(bar(B_K_FULL + i), 1);
      mbar_init(bar(B_K_EMPTY + i), 1);
    }
    for (int i = 0; i < 3; ++i) {
      mbar_init(bar(B_V_FULL + i), 1);
      mbar_init(bar(B_V_EMPTY + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(B_PS_FULL + i), 1);
      mbar_init(bar(B_PS_EMPTY + i), 1);
      mbar_init(bar(B_S_FULL + i), 1);
      mbar_init(bar(B_P_FULL + i), 256);
      mbar_init(bar(B_R_FULL + i), 1);
      mbar_init(bar(B_R_FREE + i), 256);
    }
    mbar_init(bar(B_RT_FULL), 1);
    mbar_init(bar(B_RT_EMPTY), 1);
    for (int i = 0; i < 4; ++i) {
      mbar_init(bar(B_XCH + i), 64);
      mbar_init(bar(B_RW + i), 64);
    }
    mbar_init(bar(B_TAIL), 1);
    mbar_init(bar(B_DRAIN), 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  // P-slice rows r_dim .. rd_pad are zero (the copies cover r_dim rows)
  for (int i = tid; i < (a.rd_pad - a.rd) * 8 * P_STAGES; i += NTHREADS) {
    const int st = i / ((a.rd_pad - a.rd) * 8), rem = i % ((a.rd_pad - a.rd) * 8), ch = a.rd + (rem >> 3);
    *reinterpret_cast<uint4 *>(smem + L::SM_PS + st * 8192 + (ch >> 3) * 1024 + (ch & 7) * 128 + (rem & 7) * 16) =
        make_uint4(0u, 0u, 0u, 0u);
  }
  fence_proxy_async_smem();
  if (warp == 1) {
    tmem_alloc(sb + L::SM_BAR + B_COUNT * 8, 512);
    tmem_relinquish();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&map_q);
    prefetch_tmap(&map_k);
    prefetch_tmap(&map_v);
    prefetch_tmap(&map_r);
    prefetch_tmap(&map_p);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + L::SM_BAR + B_COUNT * 8);
  int issued_k = 0, issued_v = 0, issued_p = 0, issued_rt = 0;   // copies, drained if the CTA gives up

  // the copies of the 64 keys of a block, one a lane (lane = part); a part that no
  // row needs, or whose page lies outside the pool, reads zeros
  auto part_needed = [&](int blk) -> bool {
    const int p = HN * blk + lane * ba.box;
    return lane * ba.box < HN && p <= I.p_last && (a.window <= 0 || p + ba.box > I.p0 - a.window + 1 || p < a.sink);
  };
  auto part_page = [&](int blk) -> int {
    if (a.block_table == nullptr || blk < 0 || !part_needed(blk)) return 0;
    return __ldg(a.block_table + (size_t)I.b * a.max_pages + (HN * blk + lane * ba.box) / a.page_size);
  };
  auto copy_parts = [&](uint32_t dst, const CUtensorMap *map, int blk, int pg, uint32_t br) {
    const int p = HN * blk + lane * ba.box;
    int row = -HN;
    if (part_needed(blk)) {
      if (a.block_table == nullptr) row = I.ck + p;
      else if ((unsigned)pg < (unsigned)a.num_pages) row = pg * a.page_size + p % a.page_size;
      else atomicOr(a.err, kDevErrSeqlens);
    }
    if (lane == 0) mbar_arrive_expect_tx(br, STAGE);
    __syncwarp();
    if (lane * ba.box < HN) {
      tma_load_3d(dst + lane * ba.box * 128, map, 0, I.g, row, br);
      tma_load_3d(dst + KV_BOX + lane * ba.box * 128, map, 64, I.g, row, br);
    }
    __syncwarp();
  };
  // (parked, not polling: these warps share their sub-partitions with softmax warps)
  auto wait_parked = [&](uint32_t br, uint32_t parity, int site) -> bool {
    return __all_sync(0xffffffffu, mbar_wait_suspend(br, parity, abort_flag, site));
  };

  if (warp < 4) {
    regs_dec<kRegsSupport>();
    if (warp == 0) {
      // ====================================================== r rows, P slices, K tiles
      bool run = true;
      for (int n = blockIdx.x; run && next_item(n); n += gridDim.x) {
        if (I.steps == 0) continue;
        if (n_it > 0 && !(run = wait_parked(bar(B_RT_EMPTY), (n_it - 1) & 1, 61))) break;
        if (lane == 0) {
          mbar_arrive_expect_tx(bar(B_RT_FULL), (uint32_t)ba.row_bytes);
          tma_load_3d(sb + L::SM_RT, &map_r, 0, I.g * a.group, I.cq + I.tok0, bar(B_RT_FULL));
        }
        __syncwarp();
        issued_rt = n_it + 1;
        int c = I.c_start, page = part_page(I.first);
        for (int s = 0; s < I.steps && run; ++s) {
          // K before the chunks, as the issuer takes them: with it behind, S(0) would
          // wait for chunks whose stages only R, issued after S(0), frees
          const int k = gs + s, st = k % K_STAGES;
          if (k >= K_STAGES) run = wait_parked(bar(B_K_EMPTY + st), ((k / K_STAGES) - 1) & 1, 63);
          if (!run) break;
          // (test hook: a skipped tile is never loaded)
          if (k != a.test_skip_k_tile) copy_parts(sb + L::SM_K + st * STAGE, &map_k, I.first - s, page, bar(B_K_FULL + st));
          issued_k = k + 1;
          page = part_page(s + 1 < I.steps ? I.first - s - 1 : -1);
          for (; c <= min(I.c_first + s + 1, I.c_first + I.steps - 1); ++c) {   // (a step ahead, as R)
            const int o = ob + c - I.c_start, st = o % P_STAGES;
            if (o >= P_STAGES && !(run = wait_parked(bar(B_PS_EMPTY + st), ((o / P_STAGES) - 1) & 1, 62))) break;
            if (lane == 0) {
              mbar_arrive_expect_tx(bar(B_PS_FULL + st), 128u * (uint32_t)a.rd);
              tma_load_2d(sb + L::SM_PS + st * 8192, &map_p, HN * c, 0, bar(B_PS_FULL + st));
            }
            __syncwarp();
            issued_p = o + 1;
          }
        }
        finish_item();
      }
    } else if (warp == 2) {
      // ====================================================== q rows, V tiles
      bool run = true;
      for (int n = blockIdx.x; run && next_item(n); n += gridDim.x) {
        if (I.steps == 0) continue;
        int page = part_page(I.first);
        for (int h = 0; h < 2 && run; ++h) {        // 64 dims of the item's q rows a slot
          const int v = vb + h, st = v % V_STAGES;
          if (v >= V_STAGES) run = wait_parked(bar(B_V_EMPTY + st), ((v / V_STAGES) - 1) & 1, 64);
          if (!run) break;
          if (lane == 0) {
            mbar_arrive_expect_tx(bar(B_V_FULL + st), (uint32_t)ba.row_bytes);
            tma_load_3d(sb + L::SM_V + st * STAGE, &map_q, 64 * h, I.g * a.group, I.cq + I.tok0, bar(B_V_FULL + st));
          }
          __syncwarp();
          issued_v = v + 1;
        }
        for (int s = 0; s < I.steps && run; ++s) {
          const int v = vb + 2 + s, st = v % V_STAGES;
          if (v >= V_STAGES) run = wait_parked(bar(B_V_EMPTY + st), ((v / V_STAGES) - 1) & 1, 65);
          if (!run) break;
          copy_parts(sb + L::SM_V + st * STAGE, &map_v, I.first - s, page, bar(B_V_FULL + st));
          issued_v = v + 1;
          page = part_page(s + 1 < I.steps ? I.first - s - 1 : -1);
        }
        finish_item();
      }
    } else if (warp == 1) {
      // ====================================================== MMA issuer
      // The whole warp runs the issue code; each MMA, copy and commit is issued
      // by one elected lane.
      const uint32_t id_s = idesc_bf16_f32(BM, HN, 0, 0);       // S: Q (tmem) x K (smem, K-major)
      const uint32_t id_o = idesc_bf16_f32(BM, 128, 0, 1);      // O: P (tmem) x V (smem, MN-major)
      const uint32_t id_r = idesc_bf16_f32(BM, HN, 0, 1);       // R: r (smem) x P (smem, MN-major)
      const int r_ksteps = a.rd_pad / 16;
      const uint64_t kd0 = smem_desc_sw128(sb + L::SM_K, 16, 1024);
      const uint64_t vd0 = smem_desc_sw128(sb + L::SM_V, KV_BOX, 1024);
      const uint64_t qd0 = smem_desc_sw128(sb + L::SM_V, 16, 1024);
      const uint64_t rd0 = smem_desc_sw128(sb + L::SM_RT, 16, 1024);
      const uint64_t pd0 = smem_desc_sw128(sb + L::SM_PS, 8192, 1024);
      bool ok = true, r_in = false;
      auto issue_r = [&](int c) -> bool {           // R of chunk c into buffer o % 2
        const int o = ob + c - I.c_start, st = o % P_STAGES;
        if (!r_in) {
          if (!mbar_wait_warp(bar(B_RT_FULL), n_it & 1, abort_flag, 66)) return false;
          r_in = true;
        }
        if (o >= 2 && !mbar_wait_warp(bar(B_R_FREE + (o & 1)), ((o >> 1) - 1) & 1, abort_flag, 67)) return false;
        if (!mbar_wait_warp(bar(B_PS_FULL + st), (o / P_STAGES) & 1, abort_flag, 68)) return false;
        tc_fence_after();
        const uint32_t d = tmem + TM_R + 64u * (uint32_t)(o & 1);
        const uint64_t pd = pd0 + (uint64_t)((st * 8192) >> 4);
        mma_ss_e<0>(d, rd0, pd, id_r);
        if (r_ksteps > 1) mma_ss_e<1>(d, rd0 + 2, pd + 128, id_r);
        if (r_ksteps > 2) mma_ss_e<1>(d, rd0 + 4, pd + 256, id_r);
        if (r_ksteps > 3) mma_ss_e<1>(d, rd0 + 6, pd + 384, id_r);
        mma_commit_e(bar(B_R_FULL + (o & 1)));
        if (c == I.c_first + I.steps - 1) mma_commit_e(bar(B_RT_EMPTY));   // the item's last chunk
        return true;
      };
      auto issue_s = [&](int s) -> bool {
        const int k = gs + s, st = k % K_STAGES;
        if (!mbar_wait_warp(bar(B_K_FULL + st), (k / K_STAGES) & 1, abort_flag, 69)) return false;
        tc_fence_after();
        const uint64_t kd = kd0 + (uint64_t)((st * STAGE) >> 4);
        const uint32_t d = tmem + TM_S + 64u * (uint32_t)(k & 1), q = tmem + TM_Q;
        mma_ts_e<0>(d, q + 0, kd + 0, id_s);
        mma_ts_e<1>(d, q + 8, kd + 2, id_s);
        mma_ts_e<1>(d, q + 16, kd + 4, id_s);
        mma_ts_e<1>(d, q + 24, kd + 6, id_s);
        mma_ts_e<1>(d, q + 32, kd + 512, id_s);
        mma_ts_e<1>(d, q + 40, kd + 514, id_s);
        mma_ts_e<1>(d, q + 48, kd + 516, id_s);
        mma_ts_e<1>(d, q + 56, kd + 518, id_s);
        mma_commit_e(bar(B_S_FULL + (k & 1)));
        return true;
      };
      auto issue_pv = [&](int s) -> bool {
        const int k = gs + s, v = vb + 2 + s, st = v % V_STAGES;
        if (!mbar_wait_warp(bar(B_V_FULL + st), (v / V_STAGES) & 1, abort_flag, 70)) return false;
        if (!mbar_wait_warp(bar(B_P_FULL + (k & 1)), (k >> 1) & 1, abort_flag, 71)) return false;
        tc_fence_after();
        const uint64_t vd = vd0 + (uint64_t)((st * STAGE) >> 4);
        const uint32_t o = tmem + TM_O, p = tmem + TM_S + 64u * (uint32_t)(k & 1);
        if (s > 0) mma_ts_e<1>(o, p + 0, vd + 0, id_o);
        else mma_ts_e<0>(o, p + 0, vd + 0, id_o);
        mma_ts_e<1>(o, p + 8, vd + 128, id_o);
        mma_ts_e<1>(o, p + 16, vd + 256, id_o);
        mma_ts_e<1>(o, p + 24, vd + 384, id_o);
        mma_commit_e(bar(B_V_EMPTY + st));
        if (s == I.steps - 1) mma_commit_e(bar(B_TAIL));   // (that slot may take the next q rows before it is looked at)
        return true;
      };
      for (int n = blockIdx.x; ok && next_item(n); n += gridDim.x) {
        if (I.steps == 0) continue;
        r_in = false;
        // q rows: two V slots -> TMEM (in order behind the products that read the last ones)
        for (int h = 0; h < 2 && ok; ++h) {
          const int v = vb + h, st = v % V_STAGES;
          if (!(ok = mbar_wait_warp(bar(B_V_FULL + st), (v / V_STAGES) & 1, abort_flag, 72))) break;
          tc_fence_after();
          const uint64_t qd = qd0 + (uint64_t)((st * STAGE) >> 4);
          for (int k = 0; k < 4; ++k) tmem_cp_128x256b_e(tmem + TM_Q + 32u * h + 8u * k, qd + 2 * k);
          mma_commit_e(bar(B_V_EMPTY + st));
        }
        // S(0) first: it needs no r, and R's third chunk waits for the softmax.  R runs
        // a step ahead of S: behind it, the softmax waited half of a step for it.
        const int c_last = I.c_first + I.steps - 1;
        if (ok) ok = issue_s(0);
        for (int c = I.c_start; c <= min(I.c_first + 1, c_last) && ok; ++c) ok = issue_r(c);
        for (int s = 0; s < I.steps && ok; ++s) {
          if (s + 1 < I.steps && !(ok = issue_s(s + 1))) break;
          if (I.c_first + s + 2 <= c_last && !(ok = issue_r(I.c_first + s + 2))) break;
          ok = issue_pv(s);
        }
        finish_item();
      }
      // drain: every MMA issued above has finished before TMEM is released
      mma_commit_e(bar(B_DRAIN));
      volatile int keep_waiting = 0;
      mbar_wait(bar(B_DRAIN), 0, &keep_waiting, 73, 400000000ll);
    }
    __syncwarp();
  } else {
    regs_inc<kRegsSoftmax>();
    // ======================================================== softmax
    const int wg = (warp - 4) >> 2;
    const int wq = warp & 3;                     // lane quarter (TMEM lanes 32 wq ..)
    const int a_row = 32 * wq + lane;            // row == TMEM lane
    const bool leader = warp == 4 && lane == 0;  // (an arrival costs the issuer less than a commit)
    const uint32_t lane_base = (uint32_t)(32 * wq) << 16;
    const int row_tok = a_row / a.group;         // (rows past the item's tokens repeat its last one)
    float *ring = reinterpret_cast<float *>(smem + L::SM_R) + a_row;
    float *xbuf = reinterpret_cast<float *>(smem + L::SM_XCH);   // [2 parity][2 wg][128]
    auto warp_wait = [&](uint32_t br, uint32_t parity, int site) -> bool {
      const bool r = mbar_wait(br, parity, abort_flag, site);
      return __all_sync(0xffffffffu, r);
    };
    // the product of the item's step s is done: its V slot is free
    auto pv_wait = [&](int s, int site) -> bool {
      const int v = vb + 2 + s;
      return warp_wait(bar(B_V_EMPTY + v % V_STAGES), (v / V_STAGES) & 1, site);
    };
    int n_xch = 0, n_rw = 0;
    // this thread's value to the other warpgroup's thread of the same row, and its
    auto hand_over = [&](float v) {
      xbuf[(n_xch & 1) * 256 + wg * 128 + a_row] = v;
      mbar_arrive(bar(B_XCH + wq));
    };
    auto take_over = [&](bool &okx) -> float {
      okx = warp_wait(bar(B_XCH + wq), n_xch & 1, 74);
      return xbuf[(n_xch++ & 1) * 256 + (1 - wg) * 128 + a_row];
    };
    // this warpgroup's 32 distances of chunk c into the ring
    auto copy_chunk = [&](int c) -> bool {
      const int o = ob + c - I.c_start;
      if (!warp_wait(bar(B_R_FULL + (o & 1)), (o >> 1) & 1, 75)) return false;
      if (leader) mbar_arrive(bar(B_PS_EMPTY + o % P_STAGES));     // its P slice is read
      tc_fence_after();
      uint32_t w[32];
      __syncwarp();
      tmem_ld32(tmem + lane_base + TM_R + 64u * (uint32_t)(o & 1) + 32u * wg, w);
      tmem_wait_ld(w);
      tc_fence_before();
      mbar_arrive(bar(B_R_FREE + (o & 1)));
      if (!band_stored(c, wg, I.c_first, L::SLOTS)) return true;
      const int slot = band_slot(o, wg, L::SLOTS);
      float *dst = ring + slot * 32 * BM;
#pragma unroll
      for (int i = 0; i < 32; ++i) dst[i * BM] = __uint_as_float(w[i]);
      if (slot == 0) {                           // held twice
#pragma unroll
        for (int i = 0; i < 32; ++i) dst[(L::RING + i) * BM] = __uint_as_float(w[i]);
      }
      return true;
    };
    bool ok = true;
    for (int n = blockIdx.x; ok && next_item(n); n += gridDim.x) {
      const int tok = I.tok0 + min(row_tok, I.ntok - 1), h = I.g * a.group + a_row % a.group;
      const bool valid = row_tok < I.ntok;
      const int pos = I.p0 + (tok - I.tok0);
      const size_t qrow = (size_t)(I.cq + tok) * a.Hq + h;
      const bool partial = ba.x.slots > 1;
      const size_t part_row = (size_t)I.slot * a.total_q * a.Hq + qrow;
      if (I.steps == 0) {                        // a piece without keys
        if (valid && wg == 0) a.lse_part[part_row] = -INFINITY;
        continue;
      }
      const float sc = log_scale(pos, a.inv_ln_base);
      const float cqk = a.alpha_log2e * sc, cbias = kLog2e * sc, qk_over_bias = cqk / cbias;   // alpha > 0
      float m_ref = -INFINITY, l = 0.f;
      for (int c = I.c_start; c <= I.c_first && ok; ++c) ok = copy_chunk(c);
      mbar_arrive(bar(B_RW + wq));
      for (int s = 0; s < I.steps && ok; ++s) {
        const int k = gs + s, j0 = HN * (I.first - s);
        const uint32_t sbuf = tmem + lane_base + TM_S + 64u * (uint32_t)(k & 1);
        if (!(ok = warp_wait(bar(B_S_FULL + (k & 1)), (k >> 1) & 1, 76))) break;
        if (leader) mbar_arrive(bar(B_K_EMPTY + k % K_STAGES));      // its keys are read
        tc_fence_after();
        // the row's R at distances d - u of the thread's keys j0 + 32 wg + u
        float x[32];
        if (!(ok = warp_wait(bar(B_RW + wq), n_rw & 1, 77))) break;
        ++n_rw;
        uint32_t sr[32];
        __syncwarp();
        tmem_ld32(sbuf + 32u * wg, sr);
        {
          const int d = pos - j0 - 32 * wg;
          const int p = ((d >> 5) + 2 * (ob - I.c_start) + 4 * L::SLOTS * 64) % L::SLOTS * 32 + (d & 31);
          const float *src = ring + (p < 31 ? p + L::RING : p) * BM;
#pragma unroll
          for (int u = 0; u < 32; ++u) x[u] = src[-u * BM];
        }
        tmem_wait_ld(sr);
#pragma unroll
        for (int u = 0; u < 32; u += 2)
          ffma2(x[u], x[u + 1], __uint_as_float(sr[u]), __uint_as_float(sr[u + 1]), qk_over_bias, qk_over_bias,
                x[u], x[u + 1]);
        if (j0 + HN - 1 > I.p0 || (a.window > 0 && j0 < I.p_last - a.window + 1)) {
          // up to the row's own key, in its window or a sink: a bit a key
          const int jb = j0 + 32 * wg;
          auto below = [&](int key) -> uint32_t {   // the thread's keys below `key`
            const int n = key - jb;
            return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u;
          };
          uint32_t seen = below(pos + 1);
          if (a.window > 0) seen &= ~below(pos - a.window + 1) | below(a.sink);
#pragma unroll
          for (int i = 0; i < 32; ++i) x[i] = (seen >> i) & 1u ? x[i] : -INFINITY;
        }
        // x holds alpha S + bias; the logit in log2 units is x * cbias
        const float mloc = row_max(x) * cbias;
        hand_over(mloc);
        const float mo = take_over(ok);
        if (!ok) break;
        const float mx = fmaxf(mloc, mo);
        float corr = 1.f;
        bool rescale_o = false;
        if (mx > m_ref + kRescaleThreshold || (m_ref == -INFINITY && mx != -INFINITY)) {
          const float m_new = fmaxf(m_ref, mx);
          corr = (m_ref == -INFINITY) ? 0.f : fast_exp2(m_ref - m_new);
          rescale_o = (s > 0) && (m_ref != -INFINITY);
          l *= corr;
          m_ref = m_new;
        }
        // both threads of the row have read R for this step: the next step's chunk
        if (s + 1 < I.steps) {
          if (!(ok = copy_chunk(I.c_first + s + 1))) break;
          mbar_arrive(bar(B_RW + wq));
        }
        const float m_use = (m_ref == -INFINITY) ? 0.f : m_ref;
        uint32_t pk[16];
        float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          float y0, y1;
          ffma2(y0, y1, x[2 * i], x[2 * i + 1], cbias, cbias, -m_use, -m_use);
          const float e0 = fast_exp2(y0), e1 = fast_exp2(y1);
          ffma2(acc[2 * (i & 1)], acc[2 * (i & 1) + 1], e0, e1, 1.f, 1.f, acc[2 * (i & 1)], acc[2 * (i & 1) + 1]);
          pk[i] = pack_bf16x2(e0, e1);
        }
        l += (acc[0] + acc[1]) + (acc[2] + acc[3]);
        __syncwarp();
        tmem_st16(sbuf + 16u * wg, pk);          // P (bf16 pairs) over S columns [16 wg, 16 wg + 16)
        // O moves to a new maximum only when a row of the warp needs it (the whole
        // warp then, its half of the columns), once the last step's product is done
        if (__any_sync(0xffffffffu, rescale_o)) {
          if (!(ok = pv_wait(s - 1, 78))) break;
          tc_fence_after();
          const float cf = rescale_o ? corr : 1.f;
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t r[32];
            const uint32_t oaddr = tmem + lane_base + TM_O + 64u * wg + 32u * c;
            __syncwarp();
            tmem_ld32(oaddr, r);
            tmem_wait_ld(r);
#pragma unroll
            for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * cf);
            __syncwarp();
            tmem_st32(oaddr, r);
          }
        }
        if (j0 + HN > I.lk) {
          // values past the sequence's last key (rows of no key, of another
          // sequence): zero, so that a NaN there does not meet a weight of zero
          const int v = vb + 2 + s;
          if (!(ok = warp_wait(bar(B_V_FULL + v % V_STAGES), (v / V_STAGES) & 1, 79))) break;
          if (wg == 0 && a_row < HN && j0 + a_row >= I.lk) {
            uint4 *dst = reinterpret_cast<uint4 *>(smem + L::SM_V + (v % V_STAGES) * STAGE + a_row * 128);
#pragma unroll
            for (int i = 0; i < 8; ++i) dst[i] = dst[KV_BOX / 16 + i] = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(bar(B_P_FULL + (k & 1)));
      }
      if (!ok) break;
      // ---- epilogue (the issuer is on the next item already)
      if (!(ok = warp_wait(bar(B_TAIL), n_it & 1, 80))) break;
      hand_over(l);
      const float lt = l + take_over(ok);
      if (!ok) break;
      tc_fence_after();
      const float inv = row_inverse(lt), row_lse = row_logsumexp(m_ref, lt);
      float o[64];
      __syncwarp();
      tmem_ld32f<0>(tmem + lane_base + TM_O + 64u * wg, o);
      tmem_ld32f<32>(tmem + lane_base + TM_O + 64u * wg + 32u, o);
      tmem_wait_ld_f<0>(o);
      reg_dep_f<32>(o);
#pragma unroll
      for (int i = 0; i < 64; ++i) o[i] *= inv;
      if (partial) {
        if (valid) {
          float *dst = a.o_part + part_row * kHeadDim + 64 * wg;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            uint32_t v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = __float_as_uint(o[8 * i + k]);
            store32(dst + 8 * i, v, ba.x.part32);
          }
        }
      } else {
        // the row is done, or goes on over the keys before the band: then as f16,
        // each half of it scaled by the power of two that brings its largest element
        // to 2^14 .. 2^15.  f16 then has 8 bits and more of elements from 2^-17 on (its
        // unit below 2^-14 is 2^-24); a half with smaller ones, an infinity or a NaN
        // goes in bf16.
        const int Lq = I.lk - (I.p0 - I.tok0), pair = 2 * ba.x.tokens;
        const bool more = extend_tiles(ba.x, tok / pair * pair, Lq, I.lk).n_all > 0;
        uint4 *dst = reinterpret_cast<uint4 *>(a.out + qrow * kHeadDim + 64 * wg);
        if (more) {
          uint32_t top = 0u, least = ~0u;        // of the magnitudes' bits, zeros aside (less one: still a bound)
#pragma unroll
          for (int i = 0; i < 64; ++i) {
            const uint32_t m = __float_as_uint(o[i]) & 0x7fffffffu;
            top = max(top, m);
            least = min(least, m - 1u);
          }
          const int e = min(max((int)(top >> 23) - 127, -100), 127);
          const bool wide = top >= 0x7f800000u || (int)(least >> 23) - 127 < e - 31;
          const float down = __uint_as_float((uint32_t)(14 - e + 127) << 23);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t w[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              const __half2 hv = __floats2half2_rn(o[16 * i + 2 * k] * down, o[16 * i + 2 * k + 1] * down);
              w[k] = wide ? pack_bf16x2(o[16 * i + 2 * k], o[16 * i + 2 * k + 1]) : *reinterpret_cast<const uint32_t *>(&hv);
            }
            if (valid) store32(dst + 2 * i, w, ba.x.out32);
          }
          if (valid) ba.x.carry[2 * qrow + wg] = wide ? -1.f : __uint_as_float((uint32_t)(e - 14 + 127) << 23);
        } else if (valid) {
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t w[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) w[k] = pack_bf16x2(o[16 * i + 2 * k], o[16 * i + 2 * k + 1]);
            store32(dst + 2 * i, w, ba.x.out32);
          }
        }
      }
      tc_fence_before();                         // (before the next item's first P is handed over)
      if (valid && wg == 0) {
        if (partial) a.lse_part[part_row] = row_lse;
        else a.lse[(size_t)h * a.total_q + I.cq + tok] = row_lse;
      }
      finish_item();
    }
  }

  // ------------------------------------------------------------ teardown
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && *abort_flag) record_timeout(a.err, *abort_flag);
  if (*abort_flag && lane == 0) {
    // the CTA gave up: let the copies land before shared memory goes away
    // (bounded waits, not cut short by the abort)
    volatile int keep_waiting = 0;
    if (warp == 0) {
      for (int i = max(0, issued_k - K_STAGES); i < issued_k; ++i)
        if (i != a.test_skip_k_tile)
          mbar_wait(bar(B_K_FULL + i % K_STAGES), (i / K_STAGES) & 1, &keep_waiting, 2, 400000000ll);
      for (int i = max(0, issued_p - P_STAGES); i < issued_p; ++i)
        mbar_wait(bar(B_PS_FULL + i % P_STAGES), (i / P_STAGES) & 1, &keep_waiting, 2, 400000000ll);
      if (issued_rt > 0) mbar_wait(bar(B_RT_FULL), (issued_rt - 1) & 1, &keep_waiting, 2, 400000000ll);
    } else if (warp == 2) {
      for (int i = max(0, issued_v - V_STAGES); i < issued_v; ++i)
        mbar_wait(bar(B_V_FULL + i % V_STAGES), (i / V_STAGES) & 1, &keep_waiting, 2, 400000000ll);
    }
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
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

// [rows, heads, width] bf16 in boxes of 64 x box_heads x box_rows, 128-byte swizzle
bool encode_rows(CUtensorMap *m, const void *base, int width, int heads, int rows, int box_heads, int box_rows) {
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

template <bool WIDE>
cudaError_t launch_band(const BandArgs &ba, const CUtensorMap (&m)[5], cudaStream_t stream) {
  static std::atomic<bool> attr_set[kMaxDevicesAttr];
  cudaError_t e = set_max_smem_once(reinterpret_cast<const void *>(relattn_extend_band_kernel<WIDE>),
                                    (int)smem_bytes<WIDE>(), attr_set);
  if (e != cudaSuccess) return e;
  const KernelArgs &a = ba.x.a;
  const int ctas = a.sms > 0 ? std::min(ba.n_items, a.sms) : ba.n_items;
  relattn_extend_band_kernel<WIDE><<<ctas, NTHREADS, smem_bytes<WIDE>(), stream>>>(ba, m[0], m[1], m[2], m[3], m[4]);
  return cudaGetLastError();
}

}  // namespace

int extend_band_tokens(const KernelArgs &a) { return std::min(128 / a.group, a.group >= 4 ? 32 : 64); }

cudaError_t launch_extend_band(const ExtendTcArgs &x, cudaStream_t stream) {
  const KernelArgs &a = x.a;
  BandArgs ba = {};
  ba.x = x;
  ba.tokens = extend_band_tokens(a);
  ba.n_items = (int)(extend_band_items(a) * x.band_pieces);   // (pieces only where items are fewer than SMs)
  ba.box = std::min(extend_box(a), HN);
  const int q_tokens = std::min(ba.tokens, a.total_q);        // a box stays inside the tensor
  ba.row_bytes = 128 * a.group * q_tokens;
  CUtensorMap m[5];
  // P [r_dim, E]: boxes of 64 distances x r_dim channels; distances past E read as 0
  cuuint64_t dims[2] = {(cuuint64_t)a.E, (cuuint64_t)a.rd};
  cuuint64_t strides[1] = {(cuuint64_t)a.E * 2};
  cuuint32_t box[2] = {(cuuint32_t)HN, (cuuint32_t)a.rd}, es[2] = {1, 1};
  auto fn = encoder();
  if (!fn || !encode_rows(&m[0], a.q, 128, a.Hq, a.total_q, a.group, q_tokens) ||
      !encode_rows(&m[1], a.k, 128, a.Hkv, a.kv_rows, 1, ba.box) || !encode_rows(&m[2], a.v, 128, a.Hkv, a.kv_rows, 1, ba.box) ||
      !encode_rows(&m[3], a.r, a.rd, a.Hq, a.total_q, a.group, q_tokens) ||
      fn(&m[4], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<__nv_bfloat16 *>(a.P), dims, strides, box, es,
         CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
    return cudaErrorInvalidValue;
  return a.group >= 4 ? launch_band<false>(ba, m, stream) : launch_band<true>(ba, m, stream);
}

}  // namespace relattn

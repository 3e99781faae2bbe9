// extend_tc.cu -- attention of many new tokens over a cache (relattn_extend) on
// 5th-generation tensor cores: the keys outside the relative-bias band (all of
// them without a bias), and the merge of partial results.
//
// Per row, x(i,j) = s(i) alpha q_i . k_j over the keys that the band kernel leaves
// (page "SGLang and Miles Add Day-0 Support for Inkling", section "Attention
// with Relative Positional Embedding"), softmax, P V.  The band kernel has, per
// item, the keys from a first one on (extend_band_first).
//
// An item is up to 256 rows of one kv head, (token, head of the group) pairs in two
// tiles of 128 that share every K / V tile, against key tiles of 128 from the nearest
// backwards.  Rows packed this way fill the tiles from 16 tokens on (group 8), and a
// tile's rows span few positions, so that little is computed for masked keys at the
// diagonal and the window's edge.  Key tiles start at multiples of 128 keys and hold
// whole pages or whole parts of pages: a copy per part, K by one warp and V by
// another.  The tiles of a window's sinks stand before its own.
//
// A CTA per SM takes an equal share of all key tiles, found from the lengths on the
// device (walk_units): shares start and end inside row tiles, so that ragged batches
// and counts of tiles that are no multiple of the SMs leave none idle.  A tile within
// one share is final; of a cut one each piece leaves a normalised fp32 partial, two a
// CTA at most, and relattn_extend_join_kernel adds them.  (12 chunks of 4-88 tokens on
// 6.6k-50k keys: 166 us with ranges of equal length for every tile, 132 so; 4 chunks
// of 2048 under a window of 4096, 3.4 tiles an SM: 375 and 357.)  The band's row joins
// the piece with the nearest keys in its epilogue; where the band comes in pieces
// itself, all partials are kept by row and relattn_extend_combine_kernel adds them.
//
// What bounds it: a step of the two tiles takes 1.5 - 1.66 us (2048 tokens of 16 heads on
// 131072 keys: 1.41 PFLOP/s), the exponentials and the chain S, maximum, P, P V of
// each tile alternating with the other's; with one K / V tile of 64 KB a step that is
// also 6 TB/s of cache where the rows fill one item.  An item's start and end cost 4 -
// 6 us.  Everything is inlined: calls in this kernel cost 40 % of its speed.
//
// Roles (as in fwd_tc_main.cu):
//   warp 0      K tiles; warp 2: V tiles; warp 3: the list of items, q rows
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
constexpr int K_STAGES = 2, V_STAGES = 3, ITEMS = 4;
constexpr int NTHREADS = 384;
constexpr uint32_t kRegsSupport = 88, kRegsSoftmax = 208;
static_assert(128 * kRegsSupport + 256 * kRegsSoftmax <= NTHREADS * 168, "register split");
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
              B_P_HALF = B_P_FULL + 2, B_PV_TAIL = B_P_HALF + 2, B_Q_EMPTY = B_PV_TAIL + 2, B_I_FULL = B_Q_EMPTY + 1,
              B_I_EMPTY = B_I_FULL + ITEMS, B_DRAIN = B_I_EMPTY + ITEMS, B_COUNT = B_DRAIN + 1;
constexpr uint32_t SM_TMEM_SLOT = SM_BAR + B_COUNT * 8;
constexpr uint32_t SM_ABORT = SM_TMEM_SLOT + 8;
constexpr uint32_t SM_ITEM = (SM_ABORT + 8 + 15) & ~15u;
constexpr uint32_t SM_PLAN = SM_ITEM + ITEMS * 80;   // units and band items of every warp's sequences, begin and end of the share
constexpr uint32_t SM_TOTAL = SM_PLAN + 2 * 12 * 8 + 2 * 16;
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

// ---------------------------------------------------------------- the shares
// The work in units: a step of two row tiles 6, of one 5, and 21 a piece (fitted to
// the CTAs' times: 1.5 - 1.66 us, 1.3 us, 4 - 6 us).  In the order (sequence, pair of
// row tiles, kv head) all CTAs take equally many: a row tile that holds a share's end
// is cut there, at a step.
constexpr int kStep2 = 6, kStep1 = 5, kPiece = 21;

struct Seq {
  int cq, ck, Lq, Lk, tiles;     // tiles: pairs of row tiles, 0 if it has no rows or is refused
};
__device__ __forceinline__ Seq load_seq(const ExtendTcArgs &x, int b) {
  const KernelArgs &a = x.a;
  Seq s;
  s.cq = __ldg(a.cu_q + b);
  s.ck = __ldg(a.cu_k + b);
  s.Lq = __ldg(a.cu_q + b + 1) - s.cq;
  s.Lk = __ldg(a.cu_k + b + 1) - s.ck;
  s.tiles = 0;
  if (s.Lq < 0 || s.Lk < s.Lq || s.Lq > a.max_q || s.Lk > a.max_k || !extend_rows_ok(a, s.cq, s.Lq, s.ck, s.Lk))
    atomicOr(a.err, kDevErrSeqlens);
  else
    s.tiles = (int)(((long)s.Lq + 2 * x.tokens - 1) / (2 * x.tokens));
  return s;
}
__device__ __forceinline__ int step_units(const ExtendTcArgs &x, const ExtendTiles &t) {
  return t.ntok > x.tokens ? kStep2 : kStep1;
}
__device__ __forceinline__ int tile_units(const ExtendTcArgs &x, int tile, int Lq, int Lk) {
  const ExtendTiles t = extend_tiles(x, 2 * x.tokens * tile, Lq, Lk);
  return t.n_all > 0 ? t.n_all * step_units(x, t) + kPiece : 0;
}
__device__ __forceinline__ long warp_scan(long v) {       // inclusive
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}
// A warp's walk over the sequences [b0, b1): their units, or with a target (below
// the units, >= 0) its place as (sequence, pair of row tiles, kv head, steps before
// it): 0 steps or -1 for all of them, the tile is not cut there.  blocks: token
// blocks of the band's items.
__device__ __forceinline__ long walk_units(const ExtendTcArgs &x, int b0, int b1, long target, int4 *at, long &blocks) {
  const int lane = threadIdx.x & 31;
  const long heads = x.a.Hkv;
  long run = 0;
#pragma unroll 1
  for (int c0 = b0; c0 < b1; c0 += 32) {
    Seq s{};
    if (c0 + lane < b1) s = load_seq(x, c0 + lane);
    if (x.band != 0 && s.tiles > 0) blocks += (s.Lq + x.band_tokens - 1) / x.band_tokens;
    long mine = 0;
    if (__reduce_max_sync(0xffffffffu, s.tiles) <= 4) {
#pragma unroll 1
      for (int t = 0; t < s.tiles; ++t) mine += tile_units(x, t, s.Lq, s.Lk);
    } else {
#pragma unroll 1
      for (unsigned todo = __ballot_sync(0xffffffffu, s.tiles > 0); todo; todo &= todo - 1) {
        const int i = __ffs(todo) - 1, n = __shfl_sync(0xffffffffu, s.tiles, i);
        const int Lq = __shfl_sync(0xffffffffu, s.Lq, i), Lk = __shfl_sync(0xffffffffu, s.Lk, i);
        long u = 0;
#pragma unroll 1
        for (int t = lane; t < n; t += 32) u += tile_units(x, t, Lq, Lk);
        u = __shfl_sync(0xffffffffu, warp_scan(u), 31);
        if (lane == i) mine = u;
      }
    }
    mine *= heads;
    const long upto = warp_scan(mine);
    if (target >= 0) {
      const unsigned hit = __ballot_sync(0xffffffffu, run + upto > target);
      if (hit) {
        const int i = __ffs(hit) - 1, n = __shfl_sync(0xffffffffu, s.tiles, i);
        const int Lq = __shfl_sync(0xffffffffu, s.Lq, i), Lk = __shfl_sync(0xffffffffu, s.Lk, i);
        long rest = target - run - __shfl_sync(0xffffffffu, upto - mine, i);
#pragma unroll 1
        for (int t0 = 0; t0 < n; t0 += 32) {
          const long u = t0 + lane < n ? heads * tile_units(x, t0 + lane, Lq, Lk) : 0, to = warp_scan(u);
          const unsigned here = __ballot_sync(0xffffffffu, to > rest);
          if (here) {
            const int j = __ffs(here) - 1;
            rest -= __shfl_sync(0xffffffffu, to - u, j);
            const ExtendTiles T = extend_tiles(x, 2 * x.tokens * (t0 + j), Lq, Lk);
            const int w = step_units(x, T), units = T.n_all * w + kPiece, head = (int)(rest / units);
            int step = min(max(((int)(rest - (long)head * units) - kPiece + w / 2) / w, 0), T.n_all);
            if (x.cut == nullptr) step = 2 * step < T.n_all ? 0 : T.n_all;
            if (step < 2) step = 0;                        // (no piece of one step)
            else if (T.n_all - step < 2) step = T.n_all;
            if (lane == 0) *at = make_int4(c0 + i, t0 + j, head, step < T.n_all ? step : -1);
            return 0;
          }
          rest -= __shfl_sync(0xffffffffu, to, 31);
        }
      }
    }
    run += __shfl_sync(0xffffffffu, upto, 31);
  }
  return run;
}

// A piece of work: steps [s0, s0 + steps) of a pair of row tiles, nearest keys first
struct Item {
  int b, head, cq, ck, Lk, off, tok0, ntok;       // off: position of token 0
  int s0, steps, n_all, n_sink, w_lo, p0, p_last, far;
  int whole;                                      // 1: its steps are all of the tile's; 0: steps = 0 ends the list
  int pad[3];
};
static_assert(sizeof(Item) == 80, "ring of items");

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
  // as the band's leave them.  With the band in pieces they need nothing of it (else
  // the softmax warps wait for it before they read its results), and the merge
  // may be launched behind them.  The first CTA ends after the band's grid, so
  // that whoever waits for this grid has waited for both.
  asm volatile("griddepcontrol.launch_dependents;");
  struct EndAfterBand {
    __device__ ~EndAfterBand() {
      if (blockIdx.x == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
    }
  } end_after_band;

  // ------------------------------------------------------------ the CTA's share
  long *sum = reinterpret_cast<long *>(smem + SM_PLAN);
  int4 *edge = reinterpret_cast<int4 *>(smem + SM_PLAN + 2 * 12 * 8);
  const int seq0 = (int)((long)a.batch * warp / 12), seq1 = (int)((long)a.batch * (warp + 1) / 12);
  const long me = blockIdx.x;
  long mine = 0, before = 0, total = 0, shares = 0, early = 0, lead = 0;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {       // the units; the share's first, its end
    // the first unit of share c: CTAs from `early` on start `lead` units later
    const long c = me + pass - 1, late = max(shares - early, 0l);
    const long target = pass == 0 ? -1 : (total + late * lead) * c / shares - max(c - early, 0l) * lead;
    if (pass == 0 || (target >= before && target < before + mine)) {
      long blocks = 0;
      const long n = walk_units(x, seq0, seq1, pass == 0 ? -1 : target - before, edge + pass - 1, blocks);
      if (pass == 0) {
        mine = n;
        early = __reduce_add_sync(0xffffffffu, (int)blocks);
      }
    } else if (target == total && tid == 0) {
      edge[pass - 1] = make_int4(a.batch, 0, 0, 0);
    }
    if (pass > 0) continue;
    if (lane == 0) sum[warp] = mine, sum[12 + warp] = early;
    __syncthreads();
    long items = 0;
    for (int w = 0; w < 12; ++w) {
      if (w < warp) before += sum[w];
      total += sum[w];
      items += sum[12 + w];
    }
    shares = min((long)gridDim.x, max(total / x.min_share, 1l));
    // The band's items over its CTAs: this kernel's first CTAs get the SMs that have
    // one less, the others theirs up to an item later (0, 2/5, 1 of an item's time: 12
    // chunks of 4-88 tokens, one item an SM at most, 145, 141, 138 us; 4 chunks of 2048
    // with 6 or 7 366, 362, 372; 3 chunks 297, 289, 291).
    items *= a.Hkv * x.band_pieces;
    early = a.sms - items % a.sms;
    lead = min(items < a.sms ? (long)x.band_units : (long)x.band_units * 2 / 5, total / (2 * shares));
    if (total == 0 || me >= shares) {
      if (tid == 0 && x.cut) x.cut[me] = make_int4(0, 0, 0, 0);
      return;
    }
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
    mbar_init(bar(B_Q_EMPTY), 1);
    for (int i = 0; i < ITEMS; ++i) {
      mbar_init(bar(B_I_FULL + i), 1);
      mbar_init(bar(B_I_EMPTY + i), 11);     // K, V, products, eight warps of softmax
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
  int issued = 0, issued_q = 0;   // the copies (to drain them if the CTA gives up)
  if (tid == 0 && x.cut) x.cut[me] = edge[0].w > 0 ? edge[0] : make_int4(0, 0, 0, 0);

  // items come through a ring in shared memory; every warp takes each of them and
  // reads what it needs there.  (A wait for items before may last as long as their
  // steps: 2 s and 50 us a step.)
  auto patience = [](long steps) -> long long { return 4000000000ll + 100000ll * steps; };
  const Item *items = reinterpret_cast<const Item *>(smem + SM_ITEM);
  auto take = [&](int n, long steps) -> const volatile Item * {       // null: the list ends (or the CTA gives up)
    if (!__all_sync(0xffffffffu, mbar_wait_suspend(bar(B_I_FULL + n % ITEMS), (n / ITEMS) & 1, abort_flag, 52, patience(steps)))) return nullptr;
    const volatile Item *it = items + n % ITEMS;
    return it->steps > 0 ? it : nullptr;
  };
  auto taken = [&](int n) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(B_I_EMPTY + n % ITEMS));
  };
  auto key0 = [](int v, int n_sink, int w_lo) { return BN * (v < n_sink ? v : w_lo + v - n_sink); };   // of a tile's v-th key tile

  // the copies of the tile at key k0, one a lane (lane = part of the tile); a
  // part that no row needs, or whose page lies outside the pool, reads zeros
  struct Copy {
    int b, head, ck, p0, p_last, v, n_sink, w_lo;
  };
  auto copy_of = [](const volatile Item *it) -> Copy {
    return {it->b, it->head, it->ck, it->p0, it->p_last, it->n_all - 1 - it->s0, it->n_sink, it->w_lo};
  };
  auto part_needed = [&](const Copy &c, int k0) -> bool {
    const int p = k0 + lane * x.box;
    return lane * x.box < BN && p <= c.p_last && (a.window <= 0 || p + x.box > c.p0 - a.window + 1 || p < a.sink);
  };
  auto part_page = [&](const Copy &c, int k0) -> int {
    if (a.block_table == nullptr || !part_needed(c, k0)) return 0;
    return __ldg(a.block_table + (size_t)c.b * a.max_pages + (k0 + lane * x.box) / a.page_size);
  };
  auto copy_parts = [&](const Copy &c, uint32_t dst, const CUtensorMap *map, int k0, int pg, uint32_t br) {
    const int p = k0 + lane * x.box;
    int row = -BN;
    if (part_needed(c, k0)) {
      if (a.block_table == nullptr) row = c.ck + p;
      else if ((unsigned)pg < (unsigned)a.num_pages) row = pg * a.page_size + p % a.page_size;
      else atomicOr(a.err, kDevErrSeqlens);
    }
    if (lane == 0) mbar_arrive_expect_tx(br, TILE_BYTES);
    __syncwarp();
    if (lane * x.box < BN) {
      tma_load_3d(dst + lane * x.box * 128, map, 0, c.head, row, br);
      tma_load_3d(dst + BOX_BYTES + lane * x.box * 128, map, 64, c.head, row, br);
    }
    __syncwarp();
  };

  if (warp < 4) {
    regs_dec<kRegsSupport>();
    if (warp == 3) {
      // ====================================================== items and their q rows
      const int4 from = edge[0], to = edge[1];
      Item it;
      it.b = from.x;
      it.head = from.z;
      int tile = from.y, n = 0;
      bool past = from.w < 0;                              // (the share starts behind this tile)
      it.s0 = max(from.w, 0);
      Seq q = load_seq(x, it.b);
      bool run = true;
      long steps = 0;                                      // put so far
      auto put = [&]() -> bool {
        if (n >= ITEMS && !__all_sync(0xffffffffu, mbar_wait_suspend(bar(B_I_EMPTY + n % ITEMS), ((n / ITEMS) - 1) & 1, abort_flag, 53, patience(steps))))
          return false;
        if (lane == 0) {
          *reinterpret_cast<Item *>(smem + SM_ITEM + (n % ITEMS) * sizeof(Item)) = it;
          mbar_arrive(bar(B_I_FULL + n % ITEMS));
        }
        __syncwarp();
        return true;
      };
      while (run && it.b < a.batch) {
        const bool end = it.b == to.x && tile == to.y && it.head == to.z;
        const ExtendTiles T = extend_tiles(x, 2 * x.tokens * tile, q.Lq, q.Lk);
        const int s1 = end && to.w >= 0 ? to.w : T.n_all;
        if (!past && s1 > it.s0) {
          it.cq = q.cq, it.ck = q.ck, it.Lk = q.Lk, it.off = q.Lk - q.Lq;
          it.tok0 = 2 * x.tokens * tile, it.ntok = T.ntok;
          it.steps = s1 - it.s0, it.n_all = T.n_all, it.n_sink = T.n_sink, it.w_lo = T.w_lo;
          it.p0 = T.p0, it.p_last = T.p_last, it.far = T.far;
          it.whole = it.steps == T.n_all;
          if (!(run = put())) break;
          // a box: the tokens of a row tile x the group's heads x 64 dims (rows past the
          // tokens hold other rows or zeros, rows past the box whatever was there)
          if (n > 0 && !(run = __all_sync(0xffffffffu, mbar_wait_suspend(bar(B_Q_EMPTY), (n - 1) & 1, abort_flag, 54, patience(steps))))) break;
          const int nw = T.ntok > x.tokens ? 2 : 1;
          if (lane == 0) {
            mbar_arrive_expect_tx(bar(B_Q_FULL), (uint32_t)(nw * x.q_bytes));
            for (int w = 0; w < nw; ++w) {
              tma_load_3d(sb + SM_Q + w * TILE_BYTES, &map_q, 0, it.head * a.group, it.cq + it.tok0 + w * x.tokens, bar(B_Q_FULL));
              tma_load_3d(sb + SM_Q + w * TILE_BYTES + BOX_BYTES, &map_q, 64, it.head * a.group, it.cq + it.tok0 + w * x.tokens,
                          bar(B_Q_FULL));
            }
          }
          __syncwarp();
          issued_q = ++n;
          steps += it.steps;
        }
        if (end) break;
        past = false;
        it.s0 = 0;
        if (++it.head < a.Hkv) continue;
        // the next tile with steps, 32 tiles or sequences at a time
        it.head = 0;
        ++tile;
        unsigned left = 0;                                 // sequences of the 32 from c0 on that may have one
        Seq mine = q;
        int c0 = it.b + 1 - 32;
        for (;;) {
          unsigned hit = 0;
#pragma unroll 1
          for (; tile < q.tiles && !hit; tile += 32)
            hit = __ballot_sync(0xffffffffu, tile + lane < q.tiles && tile_units(x, tile + lane, q.Lq, q.Lk) > 0);
          if (hit) {
            tile += __ffs(hit) - 1 - 32;
            break;
          }
          while (!left && c0 + 32 < a.batch) {
            c0 += 32;
            mine = Seq{};
            if (c0 + lane < a.batch) mine = load_seq(x, c0 + lane);
            left = __ballot_sync(0xffffffffu, mine.tiles > 1 || (mine.tiles == 1 && tile_units(x, 0, mine.Lq, mine.Lk) > 0));
          }
          if (!left) {
            it.b = a.batch;
            break;
          }
          const int i = __ffs(left) - 1;
          left &= left - 1;
          it.b = c0 + i;
          tile = 0;
          q.cq = __shfl_sync(0xffffffffu, mine.cq, i);
          q.ck = __shfl_sync(0xffffffffu, mine.ck, i);
          q.Lq = __shfl_sync(0xffffffffu, mine.Lq, i);
          q.Lk = __shfl_sync(0xffffffffu, mine.Lk, i);
          q.tiles = __shfl_sync(0xffffffffu, mine.tiles, i);
        }
      }
      if (run) {
        it.steps = 0;
        put();
      }
    } else if (warp != 1) {
      // ====================================================== K tiles (warp 0), V tiles (warp 2)
      const bool is_v = warp == 2;
      const CUtensorMap *map = is_v ? &map_v : &map_k;
      const int stages = is_v ? V_STAGES : K_STAGES;
      const uint32_t ring = sb + (is_v ? SM_V : SM_K), full = bar(is_v ? B_V_FULL : B_K_FULL), empty = bar(is_v ? B_V_EMPTY : B_K_EMPTY);
      int kt = 0, st = 0;
      uint32_t parity = 1;                     // of the stage's release (none is waited for in the first round)
      bool run = true;
#pragma unroll 1
      for (int n = 0; run; ++n) {
        const volatile Item *it = take(n, kt);
        if (!it) break;
        const int steps = it->steps;
        const Copy c = copy_of(it);
        int k0 = key0(c.v, c.n_sink, c.w_lo), page = part_page(c, k0);
#pragma unroll 1
        for (int i = 0; i < steps; ++i) {
          if (kt >= stages && !(run = __all_sync(0xffffffffu, mbar_wait_suspend(empty + 8u * st, parity, abort_flag, is_v ? 42 : 41))))
            break;
          // (test hook: a skipped tile of K is never loaded)
          if (is_v || kt != a.test_skip_k_tile) copy_parts(c, ring + st * TILE_BYTES, map, k0, page, full + 8u * st);
          issued = ++kt;
          if (i + 1 < steps) page = part_page(c, k0 = key0(c.v - i - 1, c.n_sink, c.w_lo));
          if (++st == stages) st = 0, parity ^= 1;
        }
        taken(n);
      }
    } else {
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
        bool ok = true;
        int kt = 0, kt1 = 0;              // steps of the items before, of those with a second row tile
        int steps = 0, nw = 0;
        auto issue_s = [&](int w, int i) -> bool {   // S_w of the item's step i
          const int ks = (kt + i) % K_STAGES;
          if (w == 0 && !mbar_wait_warp(bar(B_K_FULL + ks), ((kt + i) / K_STAGES) & 1, abort_flag, 44)) return false;
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
          if (i == steps - 1 && w == nw - 1) mma_commit_e(bar(B_Q_EMPTY));
          return true;
        };
        // O_w += P_w V of the item's step i, keys 0..63 once the softmax has written
        // that half of P, keys 64..127 once it has written all of it (an item's first
        // also tells that the softmax has read the item before's O)
        auto issue_pv = [&](int w, int i) -> bool {
          const int vs = (kt + i) % V_STAGES, parity = ((w ? kt1 : kt) + i) & 1;
          if (w == 0 && !mbar_wait_warp(bar(B_V_FULL + vs), ((kt + i) / V_STAGES) & 1, abort_flag, 45)) return false;
          if (!mbar_wait_warp(bar(B_P_HALF + w), parity, abort_flag, 50)) return false;
          tc_fence_after();
          const uint64_t vd = vd0 + (uint64_t)(vs * (TILE_BYTES >> 4));
          const uint32_t o = tmem + TM_O + 128u * (uint32_t)w, pa = tmem + TM_S + 128u * (uint32_t)w;
          if (i > 0) mma_ts_e<1>(o, pa + 0, vd + 0, id_o);
          else mma_ts_e<0>(o, pa + 0, vd + 0, id_o);
          mma_ts_e<1>(o, pa + 8, vd + 128, id_o);
          mma_ts_e<1>(o, pa + 16, vd + 256, id_o);
          mma_ts_e<1>(o, pa + 24, vd + 384, id_o);
          if (!mbar_wait_warp(bar(B_P_FULL + w), parity, abort_flag, 46)) return false;
          tc_fence_after();
          mma_ts_e<1>(o, pa + 32, vd + 512, id_o);
          mma_ts_e<1>(o, pa + 40, vd + 640, id_o);
          mma_ts_e<1>(o, pa + 48, vd + 768, id_o);
          mma_ts_e<1>(o, pa + 56, vd + 896, id_o);
          if (i == steps - 1) mma_commit_e(bar(B_PV_TAIL + w));
          return true;
        };
        for (int n = 0; ok; ++n) {
          const volatile Item *it = take(n, kt);
          if (!it) break;
          steps = it->steps;
          nw = it->ntok > x.tokens ? 2 : 1;
          taken(n);
          if (!(ok = mbar_wait_warp(bar(B_Q_FULL), n & 1, abort_flag, 43))) break;
          // S_w(i+1) goes into the buffer whose P_w(i) PV_w(i) has just been
          // issued to read: the tensor core runs them in order
#pragma unroll 1
          for (int i = -1; i < steps && ok; ++i) {
#pragma unroll 1
            for (int w = 0; w < nw && ok; ++w) {
              if (i >= 0 && !(ok = issue_pv(w, i))) break;
              if (i + 1 < steps) ok = issue_s(w, i + 1);
            }
          }
          kt += steps;
          if (nw > 1) kt1 += steps;
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
    regs_inc<kRegsSoftmax>();
    const int w = (warp - 4) >> 2;               // row tile
    const int wq = warp & 3;                     // lane quarter (TMEM lanes 32 wq ..)
    const int a_row = 32 * wq + lane;            // row == TMEM lane
    const uint32_t lane_base = (uint32_t)(32 * wq) << 16;
    const uint32_t obuf = tmem + lane_base + TM_O + 128u * (uint32_t)w;
    const uint32_t sbuf = tmem + lane_base + TM_S + 128u * (uint32_t)w;
    auto warp_wait = [&](uint32_t br, uint32_t parity, int site) -> bool {
      const bool r = mbar_wait(br, parity, abort_flag, site);
      return __all_sync(0xffffffffu, r);
    };
    int kt = 0;                                  // steps so far
    uint32_t s_parity = 0, tail_parity = 0;      // of the row tile's S and last P V
    bool ok = true, band_done = false;
#pragma unroll 1
    for (int n = 0; ok; ++n) {
    const volatile Item *it = take(n, kt);
    if (!it) break;
    const int steps = it->steps;
    if (w * x.tokens >= it->ntok) {              // (this row tile has no rows)
      kt += steps;
      taken(n);
      continue;
    }
    const bool releaser = (w == 1 || it->ntok <= x.tokens) && wq == 0 && lane == 0;   // frees K / V stages
    // the row: a token and a head (rows past the tile's tokens repeat others).
    // Only its position stays in a register through the steps.
    auto row_token = [&]() { return it->tok0 + min(w * x.tokens + min(a_row / a.group, x.tokens - 1), it->ntok - 1); };
    auto row_head = [&]() { return it->head * a.group + a_row % a.group; };
    const int pos = it->off + row_token();
    const float cqk = a.alpha_log2e * log_scale(pos, a.inv_ln_base);   // > 0 (checked on the host)
    float m_ref = -INFINITY, l = 0.f;
    // (the item's rows see all of a key tile unless it passes the first row's last
    // key or starts before the last row's window)
    const int n_sink = it->n_sink, w_lo = it->w_lo, v0 = it->n_all - 1 - it->s0, Lk = it->Lk;
    const int all_to = it->p0 + 1 - BN, all_from = a.window > 0 ? it->p_last - a.window + 1 : 0;
#pragma unroll 1
    for (int v = v0; v > v0 - steps; --v) {
      if (!(ok = warp_wait(bar(B_S_FULL + w), s_parity, 48))) break;
      s_parity ^= 1;
      if (releaser) {
        // S_1 landed: K is read by both row tiles; S_1 was issued after the step
        // before's PV_1, so that step's V is free too
        mbar_arrive(bar(B_K_EMPTY + kt % K_STAGES));
        if (v < v0) mbar_arrive(bar(B_V_EMPTY + (kt - 1) % V_STAGES));
      }
      tc_fence_after();
      const int j0 = key0(v, n_sink, w_lo);
      if (w == 0 && j0 + BN > Lk) {
        // values past the last key (rows of no key, of another sequence): zero, so
        // that a NaN there does not meet a weight of zero.  Tile 0's product is
        // issued first, so this half of its P guards tile 1's as well.
        const int vs = kt % V_STAGES;
        if (!(ok = warp_wait(bar(B_V_FULL + vs), (kt / V_STAGES) & 1, 51))) break;
        if (j0 + a_row >= Lk) {
          uint4 *vr = reinterpret_cast<uint4 *>(smem + SM_V + vs * TILE_BYTES + a_row * 128);
#pragma unroll
          for (int k = 0; k < 8; ++k) vr[k] = vr[BOX_BYTES / 16 + k] = make_uint4(0u, 0u, 0u, 0u);
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
      const bool need_mask = j0 > all_to || j0 < all_from;
      if (need_mask) {
        // the row's keys: its window, and the sinks that its window has left behind, as
        // a bit a key
        int pp = pos;
        asm volatile("" : "+r"(pp));             // (worked out here: kept, they would spill)
        const int lo = a.window > 0 ? max(0, pp - a.window + 1) : 0;
        const int kmin = lo - j0, kend = pp + 1 - j0;
        const int kfar = j0 < it->far ? min(a.sink, lo) - j0 : 0;
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
        rescale_o = (m_ref != -INFINITY) && v < v0;
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
#pragma unroll 1
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
      ++kt;
    }
    // ---- epilogue: the row is done, or its piece goes to a partial -- the CTA's own
    // two, or (the band in pieces) the row's, for the piece with the nearest keys.
    // The band's row (in one piece) joins the piece with the nearest keys.
    const int tok = row_token(), h = row_head(), tt = a_row / a.group, s0 = it->s0;
    const bool valid = tt < x.tokens && w * x.tokens + tt < it->ntok;
    const size_t qrow = (size_t)(it->cq + tok) * a.Hq + h, lrow = (size_t)h * a.total_q + it->cq + tok;
    const bool by_row = x.slots > 1 && s0 == 0, own = !by_row && !(x.slots <= 1 && it->whole);
    const bool join = x.band != 0 && x.slots <= 1 && s0 == 0;
    uint32_t band[2][8] = {};                    // the next 32 dims of it
    const __nv_bfloat16 *src = a.out + qrow * kHeadDim;
    float band_lse = -INFINITY;
    float2 ups = make_float2(0.f, 0.f);
    if (join) {
      if (!band_done) asm volatile("griddepcontrol.wait;" ::: "memory");
      band_done = true;
#pragma unroll
      for (int i = 0; i < 2; ++i) load32(src + 16 * i, band[i], x.out32);
      band_lse = a.lse[lrow];
      ups = reinterpret_cast<const float2 *>(x.carry)[qrow];
    }
    if (ok) ok = warp_wait(bar(B_PV_TAIL + w), tail_parity, 49);
    tail_parity ^= 1;
    if (ok) {
      tc_fence_after();
      if (releaser) mbar_arrive(bar(B_V_EMPTY + (kt - 1) % V_STAGES));
      float inv = row_inverse(l), row_lse = row_logsumexp(m_ref, l);
      const bool wide0 = ups.x < 0.f, wide1 = ups.y < 0.f;       // (that half of the band's row is bf16)
      ups = make_float2(fabsf(ups.x), fabsf(ups.y));
      if (join && band_lse != -INFINITY) {
        const float top = fmaxf(row_lse, band_lse), wm = __expf(row_lse - top), wb = __expf(band_lse - top);
        inv *= wm / (wm + wb);
        ups.x *= wb / (wm + wb);
        ups.y *= wb / (wm + wb);
        row_lse = top + __logf(wm + wb);
      } else {
        ups = make_float2(0.f, 0.f);
      }
      const size_t at = by_row ? (size_t)x.band_pieces * a.total_q * a.Hq + qrow
                               : ((size_t)(2 * me + (s0 == 0 ? 1 : 0)) * x.piece_tokens + (tok - it->tok0)) * a.group + a_row % a.group;
      float *part = by_row ? a.o_part : x.piece, *part_lse = by_row ? a.lse_part : x.piece_lse;
#pragma unroll 1
      for (int c = 0; c < 4; ++c) {
        uint32_t r[32];
        __syncwarp();
        tmem_ld32(obuf + 32u * c, r);
        tmem_wait_ld(r);
        float o[32];
#pragma unroll
        for (int k = 0; k < 32; ++k) o[k] = __uint_as_float(r[k]) * inv;
        if (join) {
          const float up = c < 2 ? ups.x : ups.y;
          const bool wide = c < 2 ? wide0 : wide1;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&band[i][k]));
              if (wide) f = make_float2(__uint_as_float(band[i][k] << 16), __uint_as_float(band[i][k] & 0xffff0000u));
              o[16 * i + 2 * k] = fmaf(f.x, up, o[16 * i + 2 * k]);
              o[16 * i + 2 * k + 1] = fmaf(f.y, up, o[16 * i + 2 * k + 1]);
            }
            if (c < 3) load32(src + 32 * (c + 1) + 16 * i, band[i], x.out32);
          }
        }
        if (valid && (by_row || own)) {
          float *dst = part + at * kHeadDim + 32 * c;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t v[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) v[k] = __float_as_uint(o[8 * i + k]);
            store32(dst + 8 * i, v, x.part32);
          }
        } else if (valid) {
          uint4 *dst = reinterpret_cast<uint4 *>(a.out + qrow * kHeadDim + 32 * c);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint32_t w[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) w[k] = pack_bf16x2(o[16 * i + 2 * k], o[16 * i + 2 * k + 1]);
            store32(dst + 2 * i, w, x.out32);
          }
        }
      }
      tc_fence_before();                         // (before the next item's first P is handed over)
      if (valid) {
        if (by_row || own) part_lse[at] = row_lse;
        else a.lse[lrow] = row_lse;
      }
    }
    taken(n);
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
    for (int i = max(0, issued - K_STAGES); i < issued; ++i)
      if (i != a.test_skip_k_tile)
        mbar_wait(bar(B_K_FULL + i % K_STAGES), (i / K_STAGES) & 1, &keep_waiting, 2, 400000000ll);
  }
  if (warp == 2 && lane == 0 && *abort_flag) {
    volatile int keep_waiting = 0;
    for (int i = max(0, issued - V_STAGES); i < issued; ++i)
      mbar_wait(bar(B_V_FULL + i % V_STAGES), (i / V_STAGES) & 1, &keep_waiting, 2, 400000000ll);
  }
  if (warp == 3 && lane == 0 && *abort_flag && issued_q > 0) {
    volatile int keep_waiting = 0;
    mbar_wait(bar(B_Q_FULL), (issued_q - 1) & 1, &keep_waiting, 2, 400000000ll);
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Do two shares start in the same tile, behind its first step?
__device__ __forceinline__ bool same_tile(const int4 &u, const int4 &v) {
  return u.w > 0 && v.w > 0 && u.x == v.x && u.y == v.y && u.z == v.z;
}

// out / lse of a row from its partials: lse = ln sum exp(lse_s), out = sum
// exp(lse_s - lse) o_s.  RW warps per (token, head) take them in turn; one without
// keys holds lse = -inf and is not read further.  Rows of no sequence, or of one
// whose lengths the kernels refused, are left as they are.  The partials of a row:
// its slots in o_part and, where shares cut its tile, the pieces behind the cuts.
template <int RW>
__global__ void __launch_bounds__(256) relattn_extend_combine_kernel(const __grid_constant__ ExtendTcArgs x) {
  const KernelArgs &a = x.a;
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
  int own = x.slots, share = 0, cuts = 0;        // slots; first share that starts in the tile, such shares
  long in_tile = 0;
  // launched as a programmatic dependent: the partials are visible from here on
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (x.cut != nullptr && mine) {
    const int tile = (t - cq) / (2 * x.tokens), g = h / a.group;
    in_tile = (t - cq - 2 * x.tokens * tile) * a.group + h % a.group;
    if (extend_tiles(x, 2 * x.tokens * tile, Lq, Lk).n_all == 0) --own;      // (nothing but the band)
    const int4 c = make_int4(lo, tile, g, 1);
    for (int s0 = 0; s0 < x.ctas; s0 += 32) {
      const unsigned hit = __ballot_sync(0xffffffffu, s0 + lane < x.ctas && same_tile(c, x.cut[min(s0 + lane, x.ctas - 1)]));
      if (hit && cuts == 0) share = s0 + __ffs(hit) - 1;
      cuts += __popc(hit);
    }
  }
  const int n = own + cuts;
  auto place = [&](int s) -> long {              // of partial s, in rows of o_part or (s >= own) of piece
    return s < own ? (long)s * rows + row : (long)(2 * (share + s - own)) * x.piece_tokens * a.group + in_tile;
  };
  auto part_lse = [&](int s) { return s < own ? a.lse_part[place(s)] : x.piece_lse[place(s)]; };
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float m = -INFINITY, z = 0.f;
  if (mine) {
    for (int s = lane; s < n; s += 32) m = fmaxf(m, part_lse(s));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    // 32 partials at a time, those of them that hold something: four loads in flight
    for (int s0 = 32 * wi; s0 < n; s0 += 32 * RW) {
      const float ls = s0 + lane < n ? part_lse(s0 + lane) : -INFINITY;
      const float w = exp2f((ls - m) * kLog2e);
      for (unsigned full = __ballot_sync(0xffffffffu, ls != -INFINITY); full;) {
        float4 v[4];
        float f[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int i = full ? __ffs(full) - 1 : 0, s = s0 + i;
          f[k] = full ? __shfl_sync(0xffffffffu, w, i) : 0.f;
          v[k] = full ? *reinterpret_cast<const float4 *>((s < own ? a.o_part : x.piece) + place(s) * kHeadDim + lane * 4)
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

// The same for the rows of the tiles that shares cut, whose partials are the pieces
// before the first cut and behind each: a row of blocks for every share's start,
// which ends at once unless that is a tile's first cut.  A warp a row: a chain of
// loads (two pieces a row as a rule), which many short warps hide best until their
// instructions fill the issue slots (78 %): 12 chunks of 4-88 tokens on 6.6k-50k keys
// take 132 us, on the same GPU with two rows a warp 133, four 137, eight 153.
__global__ void __launch_bounds__(256) relattn_extend_join_kernel(const __grid_constant__ ExtendTcArgs x) {
  const KernelArgs &a = x.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, share = blockIdx.x + 1;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int4 c = x.cut[share], next = x.cut[min(share + lane, x.ctas - 1)];
  if (c.w <= 0 || same_tile(c, x.cut[share - 1])) return;
  int n = 1;                                     // partials: the piece before the cut, those behind
  for (int s0 = share; s0 < x.ctas; s0 += 32) {
    const int4 u = s0 == share ? next : x.cut[min(s0 + lane, x.ctas - 1)];
    const int k = __popc(__ballot_sync(0xffffffffu, s0 + lane < x.ctas && same_tile(c, u)));
    n += k;
    if (k < 32) break;
  }
  const int cq = a.cu_q[c.x], tok0 = 2 * x.tokens * c.y, r = blockIdx.y * 8 + warp;
  if (r >= min(x.piece_tokens, a.cu_q[c.x + 1] - cq - tok0) * a.group) return;
  const long stride = (long)x.piece_tokens * a.group;
  const long first = (long)(2 * (share - 1) + 1) * stride + r, behind = (long)(2 * share) * stride + r;
  float m = -INFINITY, z = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
  for (int s = 0; s < n; ++s) {
    const long at = s == 0 ? first : behind + 2 * stride * (s - 1);
    const float ls = x.piece_lse[at];
    const float4 v = *reinterpret_cast<const float4 *>(x.piece + at * kHeadDim + lane * 4);
    const float top = fmaxf(m, ls), old = m == -INFINITY ? 0.f : exp2f((m - top) * kLog2e);
    const float w = ls == -INFINITY ? 0.f : exp2f((ls - top) * kLog2e);
    m = top;
    z = fmaf(z, old, w);
    acc.x = fmaf(acc.x, old, w * v.x);
    acc.y = fmaf(acc.y, old, w * v.y);
    acc.z = fmaf(acc.z, old, w * v.z);
    acc.w = fmaf(acc.w, old, w * v.w);
  }
  const int t = cq + tok0 + r / a.group, h = c.z * a.group + r % a.group;
  const float inv = z == 0.f ? 0.f : 1.f / z;
  uint2 packed;
  packed.x = pack_bf16x2(acc.x * inv, acc.y * inv);
  packed.y = pack_bf16x2(acc.z * inv, acc.w * inv);
  *reinterpret_cast<uint2 *>(a.out + ((long)t * a.Hq + h) * kHeadDim + lane * 4) = packed;
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
  cfg.gridDim = dim3((unsigned)x.ctas);
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

cudaError_t launch_extend_combine(const ExtendTcArgs &x, int partials, cudaStream_t stream) {
  const KernelArgs &a = x.a;
  // 8 warps a row where it has more than a warp's round of partials (32 tokens on 65536
  // keys, 77 of them: 54 us, 58 with one; 100 tokens, 20 of them: 103, 93 with one)
  const bool wide = partials > 32;
  const long rows = (long)a.total_q * a.Hq;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (x.slots <= 1) {
    cfg.gridDim = dim3((unsigned)x.ctas - 1, (unsigned)((x.piece_tokens * a.group + 7) / 8));
    return cudaLaunchKernelEx(&cfg, relattn_extend_join_kernel, x);
  }
  cfg.gridDim = dim3((unsigned)(wide ? rows : (rows + 7) / 8));
  return wide ? cudaLaunchKernelEx(&cfg, relattn_extend_combine_kernel<8>, x)
              : cudaLaunchKernelEx(&cfg, relattn_extend_combine_kernel<1>, x);
}

}  // namespace relattn

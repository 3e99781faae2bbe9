// decode_fp4_tc.cu -- decode over the 4-bit (NVFP4) cache on tcgen05 / TMEM for
// steps with many query rows a kv head: verified drafts, short chunks.
//
// The computation is that of decode_fp4.cu, x(i,j) = s(i) (alpha q_i . k_j +
// [0 <= i - j < E] r_i . P[:, i - j]), out = softmax(x) v.  There a conversion
// of the cache's values feeds 16 query rows; here one feeds 128: 8 warps
// make f16 tiles of 128 keys in shared memory (a product code * scale has 6
// bits and is exact), one thread a row takes the softmax, and the products S =
// Q K^T, O += P V read Q and P from tensor memory.  72 rows of a million keys
// and two heads took five passes of the other kernel, 439 us; here 170 (1.8 TB/s).
//
// What bounds it: no pipe (tensor a quarter, issue two fifths busy) but the way
// of a tile through its steps, 1.3 us: conversion, product, a softmax warp of
// each scheduler that walks 128 columns alone, second product.  (An earlier form
// took 193 us for that case without a bias, 166 without the conversion, 142
// without the softmax, 117 without both.)  So two groups of conversion warps
// take tiles in turn, the next logits are made while these are worked on, and
// loops are kept short: unrolled, with P in registers, the softmax took 183 to
// 193 us instead of 178, as the roles' code then no longer fits the instruction
// cache together; with eight softmax warps, 64 keys and dims each, 205.  Tiles of
// the bias band are slow (a warp fetches 32 windows of R) and weigh more in the
// split of the work.
//
// q is f16 after a power-of-two scaling per row, P is rounded to f16 and held
// times 2^7, the factors of the head are folded into the logit scale and the
// output: as in the other kernel, and as exact.  The running maximum is raised
// only when a logit passes it by more than 8 (base 2), so O is rarely read back.
// A NaN scale of V is zeroed in the tile (0 * NaN would spoil rows that do not
// see the key) and its block of 16 dims written as NaN in the rows that do.
//
// Roles (16 warps): 0-3 softmax and the output (a thread a row), 4-11
// conversion (two groups, 32 keys of every other tile each, raw bytes in a ring
// of asynchronous copies of their own), 12 the products.  TMEM: S twice 128
// columns, O 128, Q 64, P 64.  Work is split as in the other kernel: units
// (sequence, kv head, 128-row block) of tiles laid end to end.  Every wait is
// bounded: a timeout sets the device error word and the roles stop.
#include <algorithm>

#include "cache_walk.cuh"
#include "tc_common.cuh"

namespace relattn {
namespace {

using namespace tc;

constexpr int SMW = 4, DQW = 4, DQG = 2, TDT = (SMW + DQG * DQW + 4) * 32;
constexpr int KST = 2, VST = 2, RAW = 2;     // stages: K tiles, V tiles, raw bytes
constexpr int DK = kWalkTile / DQW;          // keys of a conversion warp
static_assert(DK == 32, "a scale copy a lane");
constexpr int DJ = DK / 8;                   // keys of a lane
// a raw stage of a warp: K codes [4][32 keys][16 B], V codes, K scales [32][8 B], V scales
constexpr uint32_t RW_V = DK * kFp4RowBytes, RW_KS = 2 * RW_V, RW_VS = RW_KS + DK * kFp4Blocks;
constexpr uint32_t RW_BYTES = RW_VS + DK * kFp4Blocks;
constexpr uint32_t TILE = kWalkTile * kHeadDim * 2;                // 2 halves [128 keys x 128 B]
constexpr uint32_t TD_K = 0, TD_V = TD_K + KST * TILE, TD_RAW = TD_V + VST * TILE;
constexpr uint32_t TD_BIAS = TD_RAW + DQG * DQW * RAW * RW_BYTES;  // [softmax warp][2][32 rows][16 keys]
constexpr int BROW = 20;                     // floats of a row in it (8 rows' 16-byte reads meet no bank twice)
constexpr uint32_t TD_NAN = TD_BIAS + SMW * 2 * 32 * BROW * 4;     // 4 tiles x [128 keys][4]: NaN blocks
constexpr uint32_t TD_FLAG = TD_NAN + 4 * kWalkTile * 4;           // 4 tiles x [conversion warp]: any NaN
constexpr uint32_t TD_BAR = TD_FLAG + 4 * DQW * 4;
enum { DB_QF = 0, DB_KF, DB_KE = DB_KF + KST, DB_VF = DB_KE + KST, DB_VE = DB_VF + VST, DB_SF = DB_VE + VST,
       DB_PF = DB_SF + 2, DB_OD = DB_PF + 2, DB_DRAIN, DB_COUNT };
constexpr uint32_t TD_SLOT = TD_BAR + DB_COUNT * 8, TD_ABORT = TD_SLOT + 8;
constexpr uint32_t TD_SMEM = TD_ABORT + 8 + 1024;
static_assert(TD_SMEM + (kWalkBatch + 1 + 16) * 4 <= 227 * 1024, "shared memory budget");
constexpr uint32_t TM_S = 0, TM_O = 256, TM_Q = 384, TM_P = 448;   // TMEM columns
constexpr float kPShift = 7.f;               // P is held times 2^7
constexpr float kNone = -3.402823466e38f;    // running maximum before any visible key: finite
constexpr float kRaise = 8.f;                // the maximum is raised past this excess

// Instruction descriptor: f16 x f16 -> fp32, M = N = 128; b_mn: B is N-contiguous.
__host__ __device__ constexpr uint32_t idesc_f16(int b_mn) {
  return (1u << 4) | ((uint32_t)b_mn << 16) | ((128u >> 3) << 17) | ((128u >> 4) << 24);
}

__device__ __forceinline__ void add2(float &d0, float &d1, float a0, float a1) {
  asm("{\n .reg .b64 ra, rd;\n mov.b64 ra, {%2, %3};\n mov.b64 rd, {%0, %1};\n"
      " add.rn.f32x2 rd, rd, ra;\n mov.b64 {%0, %1}, rd;\n}\n"
      : "+f"(d0), "+f"(d1) : "f"(a0), "f"(a1));
}
__device__ __forceinline__ void sts128(uint32_t a, const uint32_t (&v)[4]) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
}

// A wait of many warps off the critical path: a probe, then suspended probes.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, volatile int *abort, int site) {
  return __all_sync(0xffffffffu, mbar_test_wait(bar, parity) || mbar_wait_suspend(bar, parity, abort, site));
}

// The pieces of this CTA, in order, as every role walks them: body(unit, first
// tile, tiles (none where a range ends within a tile), slot, slots used by the
// unit) until it returns false.
template <typename F>
__device__ __forceinline__ void for_pieces(const Fp4DecodeArgs &p, const int *prefix, int base, F body) {
  Unit u;
  auto place = [&](int hr) {
    u.rb = hr % p.row_blocks;
    u.h = hr / p.row_blocks;
    u.nrows = min(kFp4TcRows, u.s.lq * p.a.group - u.rb * kFp4TcRows);
    u.qbase = u.s.lk - u.s.lq;
  };
  unsigned total = (unsigned)base * (unsigned)(p.a.Hkv * p.row_blocks);      // (the plan keeps it below 2^31)
  if (p.whole) {                             // one CTA per unit
    const int hr = blockIdx.x / p.a.batch;
    u.b = blockIdx.x - hr * p.a.batch;
    const int n = unit_tiles(p, u.b, &u.s, &u.lo);
    if (n < 0 && threadIdx.x == 0) atomicOr(p.a.err, kDevErrSeqlens);
    total = max(n, 0);
    place(hr);
  }
  Ranges at(p, total, kFp4TcMostTiles);
  while (at.x < at.end) {
    const Piece c = next_piece(p, at, u, prefix, (unsigned)base, place);
    if (u.nrows > 0 && !body(u, c.t0, c.tiles, c.slot, c.used)) return;
  }
}

// 32 keys from cache row row0 into one raw stage of a conversion warp.  Codes
// are stored [chunk of 32 dims][key], so that 8 lanes of 8 keys read 128
// contiguous bytes.
__device__ __forceinline__ void copy_keys(const Fp4DecodeArgs &p, const Unit &u, uint32_t st, int key0, long row0,
                                          int lane) {
  const int n = row0 >= 0 ? u.s.lk - key0 : 0;          // keys to copy; the rest is zeroed
#pragma unroll
  for (int i = 0; i < DJ; ++i) {
    const int k = (lane >> 2) + 8 * i, c = lane & 3;
    const bool ok = k < n;
    const long o = ok ? ((row0 + k) * p.a.Hkv + u.h) * kFp4RowBytes + c * 16 : 0;
    cp_async16(st + c * (DK * 16) + k * 16, p.kv.k + o, ok);
    cp_async16(st + RW_V + c * (DK * 16) + k * 16, p.kv.v + o, ok);
  }
  const bool ok = lane < n;
  const long o = ok ? ((row0 + lane) * p.a.Hkv + u.h) * kFp4Blocks : 0;
  cp_async8(st + RW_KS + lane * kFp4Blocks, p.kv.k_scale + o, ok);
  cp_async8(st + RW_VS + lane * kFp4Blocks, p.kv.v_scale + o, ok);
}

// Two scale bytes, NaN ones as zero.
__device__ __forceinline__ uint32_t without_nan(uint32_t s) {
  return ((s & 0x7fu) == 0x7fu ? 0u : s & 0xffu) | ((s & 0x7f00u) == 0x7f00u ? 0u : s & 0xff00u);
}

// 32 dims of a key (chunk c) as f16 into the swizzled tile.
__device__ __forceinline__ void convert_chunk(uint32_t tile, int key, int c, const uint4 &raw, uint32_t scales) {
  const uint32_t s = e4m3x2_to_f16(scales);
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t m = __byte_perm(s, 0, i < 2 ? 0x1010 : 0x3232);
    uint32_t f[4];
    e2m1x8_to_f16(w[i], f);
#pragma unroll
    for (int j = 0; j < 4; ++j) f[j] = hmul2(f[j], m);
    sts128(tile + (c >> 1) * (TILE / 2) + key * 128 + (((4 * (c & 1) + i) ^ (key & 7)) << 4), f);
  }
}

__global__ void __launch_bounds__(TDT, 1) relattn_decode_fp4_tc_kernel(const __grid_constant__ Fp4DecodeArgs p) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ int prefix[kWalkBatch + 1];
  __shared__ int wsum[TDT / 32];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t sb = smem_addr(smem);
  auto bar = [&](int i) { return sb + TD_BAR + 8u * i; };
  volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + TD_ABORT);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const unsigned full = 0xffffffffu;
  // the merge kernel may take its place beside the last CTAs; it waits for this grid
  asm volatile("griddepcontrol.launch_dependents;");

  if (tid == 0) {
    mbar_init(bar(DB_QF), SMW * 32);
    for (int s = 0; s < KST; ++s) mbar_init(bar(DB_KF + s), DQW), mbar_init(bar(DB_KE + s), 1);
    for (int s = 0; s < VST; ++s) mbar_init(bar(DB_VF + s), DQW), mbar_init(bar(DB_VE + s), 1);
    for (int s = 0; s < 2; ++s) mbar_init(bar(DB_SF + s), 1), mbar_init(bar(DB_PF + s), SMW * 32);
    mbar_init(bar(DB_OD), 1);
    mbar_init(bar(DB_DRAIN), 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == SMW + DQG * DQW) {
    tmem_alloc(sb + TD_SLOT, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem + TD_SLOT);
  int base = 0;
  if (!p.whole) base = tile_prefix<TDT>(p, prefix, wsum);

  if (warp < SMW) {
    regs_inc<192>();
    // ======================================================== softmax, a thread a row
    const uint32_t lanes = tmem + ((uint32_t)(warp * 32) << 16);
    const int slot_row = warp * 32 + lane;
    const uint32_t stage = sb + TD_BIAS + warp * 2 * 32 * BROW * 4;
    const unsigned wlim = p.a.window > 0 ? (unsigned)p.a.window : 0x80000000u;
    const long rows_all = (long)p.a.total_q * p.a.Hq;
    int g = 0;                               // tiles so far
    bool waited = false;                     // for the kernel before this one: R
    for_pieces(p, prefix, base, [&](const Unit &u, int t0, int n, int slot, int used) {
      const bool live = slot_row < u.nrows, any_row = warp * 32 < u.nrows;
      const int rr = u.rb * kFp4TcRows + (live ? slot_row : 0), tok = rr / p.a.group;
      const int head = u.h * p.a.group + (rr - tok * p.a.group);
      const long grow = (long)(u.s.q0 + tok) * p.a.Hq + head;
      const int qp = u.qbase + tok;
      if (n == 0) {                          // a slot without a tile
        if (live) p.a.lse_part[(long)slot * rows_all + grow] = -INFINITY;
        return true;
      }
      const int qmin = u.qbase + u.rb * kFp4TcRows / p.a.group;
      const int qmax = u.qbase + (u.rb * kFp4TcRows + u.nrows - 1) / p.a.group;
      const float s = log_scale(qp, p.a.inv_ln_base);
      float coef, bscale = s * kLog2e;
      {
        // the row to f16, its sign such that the logit scale is not negative
        const float kg = p.kv.k_global ? __ldg(p.kv.k_global + u.h) : 1.f;
        const uint4 *src = reinterpret_cast<const uint4 *>(p.a.q + grow * kHeadDim);
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const uint4 v = live ? __ldg(src + i) : make_uint4(0, 0, 0, 0);
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) top = max(top, max((w[k] << 16) & 0x7fff0000u, w[k] & 0x7fff0000u));
        }
        float back;
        float up = f16_row_scale(top, &back);
        coef = p.a.alpha_log2e * s * kg * back;
        if (coef < 0.f) coef = -coef, up = -up;
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
          uint32_t f[32];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint4 v = live ? __ldg(src + 8 * h + i) : make_uint4(0, 0, 0, 0);
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int k = 0; k < 4; ++k)
              f[4 * i + k] = pack_f16x2(__uint_as_float(w[k] << 16) * up, __uint_as_float(w[k] & 0xffff0000u) * up);
          }
          __syncwarp();
          tmem_st32(lanes + TM_Q + 32 * h, f);
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(bar(DB_QF));
      }
      float m = kNone, l0 = 0.f, l1 = 0.f;
      unsigned nan_blocks = 0;
      for (int i = 0; i < n; ++i, ++g) {
        const int key0 = u.lo + (t0 + i) * kWalkTile, buf = g & 1;
        const uint32_t sa = lanes + TM_S + 128u * buf;
        const bool band = p.a.E > 0 && qmin - (key0 + kWalkTile - 1) < p.a.E && qmax >= key0;
        const bool edge = key0 + kWalkTile - 1 > qmin || (unsigned)max(qmax - key0, 0) >= wlim;
        // The rows' R of 16 keys into one of two buffers, two rows at a time, keys
        // along the lanes.
        auto fetch_bias = [&](int ch) {
          const int gr = (int)grow, k = key0 + 16 * ch + (lane & 15), half = lane >> 4;
#pragma unroll 4
          for (int r = 0; r < 16; ++r) {
            const int d = __shfl_sync(full, qp, 2 * r + half) - k;
            const long row = __shfl_sync(full, gr, 2 * r + half);
            const bool in = (unsigned)d < (unsigned)p.a.E;
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;\n" ::"r"(
                             stage + (((ch & 1) * 32 + 2 * r + half) * BROW + (lane & 15)) * 4),
                         "l"(p.a.rdec + (in ? row * p.a.E + d : 0)), "r"(in ? 4 : 0) : "memory");
          }
          cp_async_commit();
        };
        if (band && any_row) {
          if (!waited) asm volatile("griddepcontrol.wait;" ::: "memory");
          waited = true;
          fetch_bias(0);
          fetch_bias(1);
        }
        if (!__all_sync(full, mbar_wait(bar(DB_SF + buf), (g >> 1) & 1, abort_flag, 41))) return false;
        tc_fence_after();
        const uint32_t fl = sb + TD_FLAG + (g & 3) * DQW * 4;
        const uint4 fa = lds128(fl);
        if (any_row) {
          float cm = coef;
          if (band || edge) {
            // ---- the logits, with bias and mask, go back to tensor memory
            cm = 1.f;
#pragma unroll 1
            for (int ch = 0; ch < 8; ++ch) {
              const int d0 = qp - (key0 + 16 * ch);                // distance of the first key
              uint32_t x[16];
              tmem_ld16(sa + 16 * ch, x);
              if (band) {
                if (ch < 7) cp_async_wait<1>();
                else cp_async_wait<0>();
                __syncwarp();
              }
              tmem_wait_ld(x);
#pragma unroll
              for (int k = 0; k < 16; k += 4) {
                uint4 b = make_uint4(0, 0, 0, 0);
                if (band) b = lds128(stage + ((ch & 1) * 32 + lane) * BROW * 4 + k * 4);
                const uint32_t bb[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  float v = __uint_as_float(x[k + j]) * coef;
                  if (band) v = fmaf(__uint_as_float(bb[j]), bscale, v);
                  if (edge && (unsigned)(d0 - (k + j)) >= wlim) v = -INFINITY;
                  x[k + j] = __float_as_uint(v);
                }
              }
              tmem_st16(sa + 16 * ch, x);
              __syncwarp();
              if (band && ch < 6) fetch_bias(ch + 2);
            }
            tmem_wait_st();
          }
          // ---- P of the maximum so far; again, with a raised one, where a logit
          // passes it by too much (S stays as it is, P has its own columns)
          float z0, z1;
          bool free = i == 0;                // P's last product is through
#pragma unroll 1
          for (;;) {
            const float c = kPShift - m;
            float mx = -INFINITY;
            z0 = l0, z1 = l1;
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
              float x[64];
              uint32_t y[32];
              tmem_ld32f<0>(sa + 64 * h, x);
              tmem_ld32f<32>(sa + 64 * h + 32, x);
              tmem_wait_ld_f<0>(x);
              reg_dep_f<32>(x);
#pragma unroll
              for (int k = 0; k < 32; ++k) {
                float e0, e1;
                mx = fmax3(mx, x[2 * k], x[2 * k + 1]);
                ffma2(e0, e1, x[2 * k], x[2 * k + 1], cm, cm, c, c);
                e0 = fast_exp2(e0), e1 = fast_exp2(e1);
                add2(z0, z1, e0, e1);
                y[k] = pack_f16x2(e0, e1);
              }
              if (!free) {
                if (!__all_sync(full, mbar_wait(bar(DB_OD), (g - 1) & 1, abort_flag, 42))) return false;
                tc_fence_after();
                free = true;
              }
              tmem_st32(lanes + TM_P + 32 * h, y);
            }
            mx *= cm;
            if (!__any_sync(full, mx > m + kRaise)) break;
            const float to = fmaxf(m, mx), f = fast_exp2(m - to);
            m = to;
            l0 *= f, l1 *= f;
            if (i == 0) continue;
            // O as it stands, after the last tile's product
#pragma unroll 1
            for (int ch = 0; ch < 4; ++ch) {
              float x[32];
              uint32_t w[32];
              tmem_ld32f<0>(lanes + TM_O + 32 * ch, x);
              tmem_wait_ld_f<0>(x);
#pragma unroll
              for (int k = 0; k < 32; ++k) w[k] = __float_as_uint(x[k] * f);
              tmem_st32(lanes + TM_O + 32 * ch, w);
            }
          }
          l0 = z0, l1 = z1;
          tmem_wait_st();
        } else if (i > 0) {
          // (a warp without rows follows the products too, one phase at a time)
          if (!__all_sync(full, mbar_wait(bar(DB_OD), (g - 1) & 1, abort_flag, 43))) return false;
        }
        // ---- NaN blocks of V that the row sees
        if (fa.x | fa.y | fa.z | fa.w) {
          const uint32_t f4[4] = {fa.x, fa.y, fa.z, fa.w};
#pragma unroll
          for (int w = 0; w < DQW; ++w)
            if (f4[w])
              for (int k = DK * w; k < DK * (w + 1); ++k) {
                uint32_t b;
                asm volatile("ld.shared.b32 %0, [%1];" : "=r"(b) : "r"(sb + TD_NAN + ((g & 3) * kWalkTile + k) * 4));
                if ((unsigned)qp - (unsigned)(key0 + k) < wlim)
                  nan_blocks |= (b & 3u) | ((b >> 6) & 0xcu) | ((b >> 12) & 0x30u) | ((b >> 18) & 0xc0u);
              }
        }
        tc_fence_before();
        mbar_arrive(bar(DB_PF + buf));
      }
      // ---- the piece's result
      // (Every warp has seen the product before the last: in this piece's last tile, or
      // at the end of the piece before.  A parity wait tells only neighbouring
      // phases apart: one for that product, first polled after the last one too
      // has completed, would never pass.)
      if (!__all_sync(full, mbar_wait(bar(DB_OD), (g - 1) & 1, abort_flag, 44))) return false;
      tc_fence_after();
      const float z = l0 + l1;
      const float scale = z == 0.f ? 0.f : (p.kv.v_global ? __ldg(p.kv.v_global + u.h) : 1.f) / z;
      const float lse = z == 0.f ? -INFINITY : (m - kPShift + log2f(z)) * kLn2;
      if (live) {
        if (p.splits == 1) p.a.lse[(long)head * p.a.total_q + u.s.q0 + tok] = lse;
        else p.a.lse_part[(long)slot * rows_all + grow] = lse;
        if (t0 == 0)                         // mark the slots that no piece fills
          for (int k = used; k < p.splits; ++k) p.a.lse_part[(long)k * rows_all + grow] = -INFINITY;
      }
      __syncwarp();
      if (any_row) {
#pragma unroll
        for (int ch = 0; ch < 4; ++ch) {
          float x[32];
          tmem_ld32f<0>(lanes + TM_O + 32 * ch, x);
          tmem_wait_ld_f<0>(x);
#pragma unroll
          for (int k = 0; k < 32; ++k) {
            x[k] *= scale;
            if (nan_blocks >> (2 * ch + k / 16) & 1) x[k] = __int_as_float(0x7fffffff);
          }
          if (live && p.splits == 1) {
            uint4 *dst = reinterpret_cast<uint4 *>(p.a.out + grow * kHeadDim + 32 * ch);
#pragma unroll
            for (int k = 0; k < 4; ++k)
              dst[k] = make_uint4(pack_bf16x2(x[8 * k], x[8 * k + 1]), pack_bf16x2(x[8 * k + 2], x[8 * k + 3]),
                                  pack_bf16x2(x[8 * k + 4], x[8 * k + 5]), pack_bf16x2(x[8 * k + 6], x[8 * k + 7]));
          } else if (live) {
            float4 *dst = reinterpret_cast<float4 *>(p.a.o_part + ((long)slot * rows_all + grow) * kHeadDim + 32 * ch);
#pragma unroll
            for (int k = 0; k < 8; ++k) dst[k] = make_float4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]);
          }
          __syncwarp();
        }
      }
      return true;
    });
    cp_async_wait<0>();
  } else if (warp < SMW + DQG * DQW) {
    regs_dec<104>();
    // ======================================================== conversion
    const int dw = (warp - SMW) % DQW, turn = (warp - SMW) / DQW;
    const uint32_t ring = sb + TD_RAW + (warp - SMW) * RAW * RW_BYTES;
    int g0 = 0;                              // tiles before this piece
    for_pieces(p, prefix, base, [&](const Unit &u, int t0, int n, int slot, int used) {
      const int own = (turn - g0) & (DQG - 1), count = (n - own + DQG - 1) / DQG;      // first of this group's tiles; how many
      const int first = u.lo + (t0 + own) * kWalkTile + dw * DK;
      long next = count > 0 ? group_row(p, u, first) : -1;
      int rs = 0, cs = 0;                    // stages to read and to copy into
#pragma unroll 1
      for (int i = 1 - RAW; i < count; ++i) {
        __syncwarp();                        // the stage before this one has been read
        const int ahead = i + RAW - 1;
        if (ahead < count) copy_keys(p, u, ring + cs * RW_BYTES, first + ahead * DQG * kWalkTile, next, lane);
        cp_async_commit();
        cs = cs == RAW - 1 ? 0 : cs + 1;
        next = ahead + 1 < count ? group_row(p, u, first + (ahead + 1) * DQG * kWalkTile) : -1;
        if (i < 0) continue;
        cp_async_wait<RAW - 1>();
        __syncwarp();
        const uint32_t st = ring + rs * RW_BYTES;
        rs = rs == RAW - 1 ? 0 : rs + 1;
        const int g = g0 + own + i * DQG;
        const int c = lane >> 3, k = lane & 7, ks = g % KST, vs = g % VST;
        const uint32_t at = st + c * (DK * 16) + k * 16, sat = st + RW_KS + k * kFp4Blocks + 2 * c;
        // NaN scales of V are listed before the logits of their keys are known
        uint32_t bad[DJ], some = 0;
#pragma unroll
        for (int j = 0; j < DJ; ++j) {
          const uint32_t sv = lds_u16(sat + RW_VS - RW_KS + 8 * kFp4Blocks * j);
          bad[j] = ((sv & 0x7fu) == 0x7fu ? 1u : 0u) | ((sv & 0x7f00u) == 0x7f00u ? 2u : 0u);
          some |= bad[j];
        }
        const bool any = __any_sync(full, some);
        if (any) {
#pragma unroll
          for (int j = 0; j < DJ; ++j)
            smem[TD_NAN + ((g & 3) * kWalkTile + dw * DK + k + 8 * j) * 4 + c] = (uint8_t)bad[j];
        }
        if (lane == 0) *reinterpret_cast<int *>(smem + TD_FLAG + ((g & 3) * DQW + dw) * 4) = any;
        if (g >= KST && !wait_warp(bar(DB_KE + ks), ((g / KST) - 1) & 1, abort_flag, 45)) return false;
#pragma unroll 1
        for (int j = 0; j < DJ; ++j)
          convert_chunk(sb + TD_K + ks * TILE, dw * DK + k + 8 * j, c, lds128(at + 128 * j),
                        lds_u16(sat + 8 * kFp4Blocks * j));
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && g != p.a.test_skip_k_tile) mbar_arrive(bar(DB_KF + ks));    // (test hook: never told)
        if (g >= VST && !wait_warp(bar(DB_VE + vs), ((g / VST) - 1) & 1, abort_flag, 46)) return false;
#pragma unroll 1
        for (int j = 0; j < DJ; ++j)
          convert_chunk(sb + TD_V + vs * TILE, dw * DK + k + 8 * j, c, lds128(at + RW_V + 128 * j),
                        without_nan(lds_u16(sat + RW_VS - RW_KS + 8 * kFp4Blocks * j)));
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(DB_VF + vs));
      }
      g0 += n;
      cp_async_wait<0>();
      return true;
    });
    cp_async_wait<0>();
  } else {
    // ======================================================== the products (the warpgroup's first warp)
    regs_dec<112>();
    int g = 0, pieces = 0;
    bool run = true;
    const uint32_t q = tmem + TM_Q, o = tmem + TM_O, id_s = idesc_f16(0), id_o = idesc_f16(1);
    const uint64_t kd0 = smem_desc_sw128(sb + TD_K, 16, 1024), vd0 = smem_desc_sw128(sb + TD_V, TILE / 2, 1024);
    if (warp == SMW + DQG * DQW) for_pieces(p, prefix, base, [&](const Unit &u, int t0, int n, int slot, int used) {
      if (n == 0) return true;
      if (!(run = mbar_wait_warp(bar(DB_QF), pieces & 1, abort_flag, 47))) return false;
      ++pieces;
      auto pv = [&](int t, bool acc) {       // O += P V of tile t
        const int vs = t % VST;
        if (!(run = mbar_wait_warp(bar(DB_PF + (t & 1)), (t >> 1) & 1, abort_flag, 48))) return false;
        if (!(run = mbar_wait_warp(bar(DB_VF + vs), (t / VST) & 1, abort_flag, 49))) return false;
        tc_fence_after();
        const uint64_t vd = vd0 + (uint64_t)(vs * (TILE >> 4));
        const uint32_t pa = tmem + TM_P;
        if (acc) mma_ts_e<1>(o, pa, vd, id_o);
        else mma_ts_e<0>(o, pa, vd, id_o);
        mma_ts_e<1>(o, pa + 8, vd + 128, id_o);
        mma_ts_e<1>(o, pa + 16, vd + 256, id_o);
        mma_ts_e<1>(o, pa + 24, vd + 384, id_o);
        mma_ts_e<1>(o, pa + 32, vd + 512, id_o);
        mma_ts_e<1>(o, pa + 40, vd + 640, id_o);
        mma_ts_e<1>(o, pa + 48, vd + 768, id_o);
        mma_ts_e<1>(o, pa + 56, vd + 896, id_o);
        mma_commit_e(bar(DB_VE + vs));
        mma_commit_e(bar(DB_OD));
        return true;
      };
      for (int i = 0; i < n; ++i, ++g) {
        const int ks = g % KST;
        if (!(run = mbar_wait_warp(bar(DB_KF + ks), (g / KST) & 1, abort_flag, 50))) return false;
        tc_fence_after();
        const uint64_t kd = kd0 + (uint64_t)(ks * (TILE >> 4));
        const uint32_t d = tmem + TM_S + 128u * (g & 1);
        mma_ts_e<0>(d, q, kd, id_s);
        mma_ts_e<1>(d, q + 8, kd + 2, id_s);
        mma_ts_e<1>(d, q + 16, kd + 4, id_s);
        mma_ts_e<1>(d, q + 24, kd + 6, id_s);
        mma_ts_e<1>(d, q + 32, kd + 1024, id_s);
        mma_ts_e<1>(d, q + 40, kd + 1026, id_s);
        mma_ts_e<1>(d, q + 48, kd + 1028, id_s);
        mma_ts_e<1>(d, q + 56, kd + 1030, id_s);
        mma_commit_e(bar(DB_KE + ks));
        mma_commit_e(bar(DB_SF + (g & 1)));
        if (i > 0 && !pv(g - 1, i > 1)) return false;
      }
      return pv(g - 1, n > 1);
    });
    if (!run) {                              // (so only where products were issued)
      // stop: wait for the products already issued before tensor memory is freed
      mma_commit_e(bar(DB_DRAIN));
      const long long c0 = clock64();
      while (!mbar_test_wait(bar(DB_DRAIN), 0) && clock64() - c0 < 200000000ll) {
      }
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && *abort_flag) record_timeout(p.a.err, *abort_flag);
  if (warp == SMW + DQG * DQW) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

}  // namespace

cudaError_t launch_decode_fp4_tc(const Fp4DecodeArgs &p, cudaStream_t stream) {
  static std::atomic<bool> done[kMaxDevicesAttr];
  const cudaError_t e = set_max_smem_once(reinterpret_cast<const void *>(relattn_decode_fp4_tc_kernel), (int)TD_SMEM, done);
  if (e != cudaSuccess) return e;
  const long grid = p.whole ? (long)p.a.batch * p.a.Hkv * p.row_blocks : p.a.sms;
  if (grid > 0x7fffffffL) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(TDT);
  cfg.dynamicSmemBytes = TD_SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = p.a.E > 0 ? 1 : 0;          // behind the R kernel
  return cudaLaunchKernelEx(&cfg, relattn_decode_fp4_tc_kernel, p);
}

}  // namespace relattn

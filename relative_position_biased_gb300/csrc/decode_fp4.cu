// decode_fp4.cu -- split-KV decode of relative attention over the 4-bit
// (NVFP4) K / V cache.
//
// The computation of the other decodes (page "SGLang and Miles Add Day-0
// Support for Inkling", section "Attention with Relative Positional
// Embedding"; the split of the keys on the page "vLLM Day-0 support for TML
// Inkling"), x(i,j) = s(i) (alpha q_i . k_j + [0 <= d < E] r_i . P[:, d]),
// out = softmax(x) v, with k and v the values the cache stands for and d the
// difference of two positions: the rows' own indices, or (a cache that
// eviction has thinned out) positions given per row and kv head.
//
// What bounds it: a key of one head is 144 bytes and 256 values.  The bytes
// alone take 21 ps at the copy rate; each value has to become an f16 operand,
// and a conversion (two values a lane) runs at about 1.2 warp instructions a
// clock and SM against 2 for the f16 multiply by the scale and 0.5 for the
// matrix instruction.  So the kernel is written around few instructions a
// key, on warp-level matrix instructions fed from registers: with few rows the
// tcgen05 path's way through shared memory, 2 bytes a value, costs more than the
// products (decode_fp4_tc.cu takes it for many).
// Measured: 64 sequences of 1 to 32 thousand keys, group 8, two kv heads: 97 us
// (3.2 TB/s of the cache).  No pipe is full there: issue slots are 62 % busy, DRAM
// 47 %, and without any conversion the call still took 80 us.  The rest is CTAs of
// equal ranges that do not end together (62 to 82 us within one SM), R before
// and the merge after them (7 and 10 us each by themselves).
//   - Keys go along the matrix instruction's 16 rows, query rows along its 8
//     columns: S^T = K q^T, O^T += V^T P^T.  One token of a GQA-8 group fills
//     it; with 16 rows a unit takes two columns sets.
//   - The dims of a product may be summed in any order, so a lane's share of a
//     key is 16 contiguous bytes: 32 dims, two scales.  No value crosses
//     lanes, and q is laid out to match once per unit.
//   - For V the operand pairs two keys of one dim: the nibbles of two code
//     words are interleaved before the conversion (four logical operations
//     for 16 values), and a lane's 16 dims are one scale block.
//   - A product code * scale has 6 bits and is exact in f16; the factor of the
//     head is folded into the logit scale and the output.  q is bf16 and exact in
//     f16, after a power-of-two scaling per row, down to 2^-31 of its row's
//     maximum; below that it is rounded by at most 2^-39 of the maximum.  P is
//     rounded to f16 (11 bits, half a step 2^-12 of the value), scaled by 2^7 so
//     that what is lost below f16's range is 2^-31 of the largest; everything
//     else is fp32.
//
// A warp streams 32 keys at a time through its own ring of asynchronous
// copies: no barrier among warps until the end of a piece.  The running
// maximum is raised only when a logit passes it by more than 8 (base 2).
//
// Work split: the units (sequence, kv heads of a CTA, 16-row block) hold
// ceil(keys / tile) tiles each; they are laid end to end in ranges of C tiles, one
// a CTA, or several where one would sum over too many keys.  A piece of a unit
// writes its partial to slot (its range) - (first range of the unit); the unit's
// first piece marks the slots no piece fills.  With an even number of kv heads a
// CTA takes two of them, two warps each, over the same 64 keys: their rows share
// 128-byte lines, and lines fetched for one head only were read twice (538 MB for
// 311 MB of cache).
#include <algorithm>

#include "cache_walk.cuh"

namespace relattn {
namespace {

constexpr int FW = 4, FT = FW * 32;          // warps and threads of a CTA
constexpr int FK = kWalkTile / FW;         // keys a warp takes at a time
static_assert(FK == 32, "two 16-key groups");
constexpr int F_STAGES = 3;
// a stage of one warp: K codes, V codes, K scales, V scales
constexpr int FS_V = FK * kFp4RowBytes, FS_KS = 2 * FS_V, FS_VS = FS_KS + FK * kFp4Blocks;
constexpr int FS_BYTES = FS_VS + FK * kFp4Blocks;
constexpr int F_RING = FW * F_STAGES * FS_BYTES;
static_assert(F_RING >= FW * kFp4Rows * kHeadDim * 4 + 2 * FW * kFp4Rows * 4 + 2 * kFp4Rows * 8, "the merge reuses the ring");
constexpr float kPShift = 7.f;               // P is held times 2^7
constexpr float kNone = -3.402823466e38f;    // running maximum before any visible key: finite, so that
                                             // differences from it are never NaN
constexpr float kRaise = 8.f;                // the maximum is raised past this excess

constexpr int ctas_per_sm(int nt) { return nt == 1 ? 4 : 3; }

// Copies 32 keys into one stage of the warp's ring.  Within 16 keys, key k
// (k = i + 4 j, j in {0, 1}, +8) is row 2 i + j (+8) of the matrix operand: K
// is stored in operand order (a quarter warp then reads 128 contiguous
// bytes), V in key order with its 16-byte chunks exchanged every other pair
// of keys (a half warp reads keys t = 0..3 from distinct banks).
__device__ __forceinline__ void issue_group(const Fp4DecodeArgs &p, const Unit &u, uint32_t st, int key0, long row0,
                                            int lane) {
  const int n = row0 >= 0 ? u.s.lk - key0 : 0;          // keys to copy; the rest is zeroed
  const int k0 = lane >> 2, c = lane & 3;
  const long rb = (long)p.a.Hkv * kFp4RowBytes, step = 8 * rb;
  long off = (max(row0, 0L) + k0) * rb + u.h * kFp4RowBytes + c * 16;
  // rows 8 apart keep their place within 16 keys: 8 more, whole groups
  const uint32_t kdst = st + (2 * (k0 & 3) + (k0 >> 2)) * kFp4RowBytes + c * 16;
  const uint32_t vdst = st + FS_V + k0 * kFp4RowBytes + ((c ^ (((k0 >> 1) & 1) << 1)) << 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool ok = k0 + 8 * i < n;
    const long o = ok ? off : 0;
    cp_async16(kdst + 8 * i * kFp4RowBytes, p.kv.k + o, ok);
    cp_async16(vdst + 8 * i * kFp4RowBytes, p.kv.v + o, ok);
    off += step;
  }
  const bool ok = lane < n;
  const long soff = ok ? ((row0 + lane) * p.a.Hkv + u.h) * kFp4Blocks : 0;
  cp_async8(st + FS_KS + lane * kFp4Blocks, p.kv.k_scale + soff, ok);
  cp_async8(st + FS_VS + lane * kFp4Blocks, p.kv.v_scale + soff, ok);
}

// One piece: tiles [t0, t0 + n) of unit u, whose u.h is the warp's head;
// partial into `slot` (or the result itself when there is one slot).
template <int NT, bool POS>
__device__ __forceinline__ void run_piece(const Fp4DecodeArgs &p, const Unit &u, int t0, int n, int slot,
                                          uint8_t *smem) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const uint32_t ring = smem_addr(smem) + warp * (F_STAGES * FS_BYTES);
  const int tile = kWalkTile / p.hp;        // keys of a tile
  const int k_first = u.lo + t0 * tile + warp / p.hp * FK;
  const unsigned full = 0xffffffffu;

  // ---- the first copies, then the query rows while they fly
  long next_row = -1;                       // cache row of the next group to copy
  int pos_next = 0x7fffffff;                // its key's position (lane = key)
  int pos_q[F_STAGES];                      // positions of the groups in flight
  auto fetch_pos = [&](int key0, long row) {
    int kp = 0x7fffffff;                    // masked for every row
    if (POS && row >= 0 && key0 + lane < u.s.lk) {
      kp = __ldg(p.key_pos + (long)u.h * p.pages.rows + row + lane);
      if (kp < 0) kp = 0x7fffffff;
    }
    return kp;
  };
#pragma unroll
  for (int i = 0; i < F_STAGES - 1; ++i) {
    pos_q[i] = 0x7fffffff;
    if (i < n) {
      const int key0 = k_first + i * tile;
      const long row = group_row(p, u, key0);
      if (POS) pos_q[i] = fetch_pos(key0, row);
      issue_group(p, u, ring + i * FS_BYTES, key0, row, lane);
    }
    cp_async_commit();
  }
  bool waited = false;                      // for the kernel before this one: R
  if (F_STAGES - 1 < n) {
    next_row = group_row(p, u, k_first + (F_STAGES - 1) * tile);
    if (POS) pos_next = fetch_pos(k_first + (F_STAGES - 1) * tile, next_row);
  }

  uint32_t qf[NT][16];                      // row 8 nt + g, dims 32 t .. 32 t + 31
  float coef[NT][2], bscale[NT][2];         // of rows 8 nt + 2 t, + 1
  int qp[NT][2], gr_[NT][2];                // position, row of R
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int nrow = nt * 8 + g;
    int tok = 0;
    float back = 1.f;
    if (nrow < u.nrows) {
      const uint4 *src = reinterpret_cast<const uint4 *>(p.a.q + unit_row(p, u, nrow, &tok) * kHeadDim + t * 32);
      uint4 w[4];
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = __ldg(src + i);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t ws[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          qf[nt][4 * i + j] = ws[j];
          top = max(top, max((ws[j] << 16) & 0x7fff0000u, ws[j] & 0x7fff0000u));
        }
      }
      const unsigned quad = 0xfu << (lane & ~3);
      top = max(top, __shfl_xor_sync(quad, top, 1));
      top = max(top, __shfl_xor_sync(quad, top, 2));
      const float up = f16_row_scale(top, &back);
#pragma unroll
      for (int i = 0; i < 16; ++i)
        qf[nt][i] = pack_f16x2(__uint_as_float(qf[nt][i] << 16) * up, __uint_as_float(qf[nt][i] & 0xffff0000u) * up);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) qf[nt][i] = 0;
    }
    __syncwarp();
    const float kg = p.kv.k_global ? __ldg(p.kv.k_global + u.h) : 1.f;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int m = nt * 8 + 2 * t + c;
      const float bk = __shfl_sync(full, back, (2 * t + c) * 4);
      int tk;
      const bool live = m < u.nrows;
      gr_[nt][c] = (int)unit_row(p, u, live ? m : 0, &tk);
      const float s = live ? log_scale(u.qbase + tk, p.a.inv_ln_base) : 0.f;
      qp[nt][c] = live ? u.qbase + tk : -1;   // rows past the block see no key
      coef[nt][c] = p.a.alpha_log2e * s * kg * bk;
      bscale[nt][c] = s * kLog2e;
    }
  }
  int qmin, qmax;
  {
    int tk;
    unit_row(p, u, 0, &tk);
    qmin = u.qbase + tk;
    unit_row(p, u, u.nrows - 1, &tk);
    qmax = u.qbase + tk;
  }
  const unsigned wlim = p.a.window > 0 ? (unsigned)p.a.window : 0x80000000u;

  float acc[8][NT][4];                      // O^T: dims 16 g + 2 m (+1), rows 8 nt + 2 t (+1)
  float mref[NT][2], l[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
    for (int c = 0; c < 2; ++c) mref[nt][c] = kNone, l[nt][c] = 0.f;
#pragma unroll
    for (int m = 0; m < 8; ++m) acc[m][nt][0] = acc[m][nt][1] = acc[m][nt][2] = acc[m][nt][3] = 0.f;
  }

  int buf = 0;
  for (int it = 0; it < n; ++it) {
    const int key0 = k_first + it * tile;
    cp_async_wait<F_STAGES - 2>();
    __syncwarp();                            // the stage has landed; the one before it is read
    {
      const int nb = buf == 0 ? F_STAGES - 1 : buf - 1;
      if (it + F_STAGES - 1 < n) issue_group(p, u, ring + nb * FS_BYTES, key0 + (F_STAGES - 1) * tile, next_row, lane);
      cp_async_commit();
    }
    const int pos_lane = POS ? pos_q[0] : 0;
    if (POS) {
#pragma unroll
      for (int i = 0; i + 2 < F_STAGES; ++i) pos_q[i] = pos_q[i + 1];
      pos_q[F_STAGES - 2] = pos_next;
    }
    if (it + F_STAGES < n) {
      next_row = group_row(p, u, key0 + F_STAGES * tile);
      if (POS) pos_next = fetch_pos(key0 + F_STAGES * tile, next_row);
    }
    const uint32_t st = ring + buf * FS_BYTES;
    buf = buf == F_STAGES - 1 ? 0 : buf + 1;
    if (key0 >= u.s.lk) continue;            // past the sequence: nothing for this warp

    const bool edge = POS || key0 + FK - 1 > qmin || (unsigned)(qmax - key0) >= wlim;
    const bool band = p.a.E > 0 && (POS ? __any_sync(full, pos_lane != 0x7fffffff && qmin - pos_lane < p.a.E)
                                        : qmin - (key0 + FK - 1) < p.a.E);
#pragma unroll 1
    for (int gr = 0; gr < 2; ++gr) {
      int kp[2];                             // positions of the lane's keys
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const int k = gr * 16 + hf * 8 + (g >> 1) + 4 * (g & 1);
        kp[hf] = POS ? __shfl_sync(full, pos_lane, k) : key0 + k;
      }
      // With 8 rows the bias is loaded ahead of the products, which hide its
      // latency (64 x 1 rows: 4 us of 106); with 16 that costs more in spilled
      // registers than it gives (72 rows, which took this path then: 457 -> 482
      // us on a million keys).
      float bias[4];
      auto load_bias = [&](int nt) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const unsigned d = (unsigned)qp[nt][i & 1] - (unsigned)kp[i >> 1];
          bias[i] = d < (unsigned)p.a.E ? p.a.rdec[(long)gr_[nt][i & 1] * p.a.E + d] : 0.f;
        }
      };
      if (band) {
        if (!waited) {
          asm volatile("griddepcontrol.wait;" ::: "memory");
          waited = true;
        }
        if (NT == 1) load_bias(0);
      }
      // ---- S^T = K q^T, two chains of four products
      float x[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) x[nt][i] = 0.f;
      {
        const uint32_t kb = st + gr * 16 * kFp4RowBytes + t * 16;
        const uint4 w0 = lds128(kb + g * kFp4RowBytes), w1 = lds128(kb + (g + 8) * kFp4RowBytes);
        const int kg16 = (g >> 1) + 4 * (g & 1);
        const uint32_t sb = st + FS_KS + (gr * 16 + kg16) * kFp4Blocks + 2 * t;
        const uint32_t s0 = e4m3x2_to_f16(lds_u16(sb)), s1 = e4m3x2_to_f16(lds_u16(sb + 8 * kFp4Blocks));
        const uint32_t ww0[4] = {w0.x, w0.y, w0.z, w0.w}, ww1[4] = {w1.x, w1.y, w1.z, w1.w};
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const uint32_t m0 = __byte_perm(s0, 0, w < 2 ? 0x1010 : 0x3232);
          const uint32_t m1 = __byte_perm(s1, 0, w < 2 ? 0x1010 : 0x3232);
          uint32_t f0[4], f1[4];
          e2m1x8_to_f16(ww0[w], f0);
          e2m1x8_to_f16(ww1[w], f1);
#pragma unroll
          for (int i = 0; i < 4; ++i) f0[i] = hmul2(f0[i], m0), f1[i] = hmul2(f1[i], m1);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            mma_f16_16816(x[nt], f0[0], f1[0], f0[1], f1[1], qf[nt][4 * w], qf[nt][4 * w + 1]);
            mma_f16_16816(x[nt], f0[2], f1[2], f0[3], f1[3], qf[nt][4 * w + 2], qf[nt][4 * w + 3]);
          }
        }
      }

      // ---- logits: scale, bias, mask
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) x[nt][i] = x[nt][i] * coef[nt][i & 1];
      if (band) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          if (NT > 1) load_bias(nt);
#pragma unroll
          for (int i = 0; i < 4; ++i) x[nt][i] = fmaf(bias[i], bscale[nt][i & 1], x[nt][i]);
        }
      }
      if (edge) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if ((unsigned)qp[nt][i & 1] - (unsigned)kp[i >> 1] >= wlim) x[nt][i] = -INFINITY;
      }

      // ---- the running maximum, raised only when a logit passes it by more than kRaise
      bool need = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c = 0; c < 2; ++c) need |= fmaxf(x[nt][c], x[nt][c + 2]) > mref[nt][c] + kRaise;
      if (__any_sync(full, need)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float m = fmaxf(x[nt][c], x[nt][c + 2]);
            m = fmaxf(m, __shfl_xor_sync(full, m, 4));
            m = fmaxf(m, __shfl_xor_sync(full, m, 8));
            m = fmaxf(m, __shfl_xor_sync(full, m, 16));
            m = fmaxf(m, mref[nt][c]);
            const float f = fast_exp2(mref[nt][c] - m);
            mref[nt][c] = m;
            l[nt][c] *= f;
#pragma unroll
            for (int d = 0; d < 8; ++d) acc[d][nt][c] *= f, acc[d][nt][c + 2] *= f;
          }
      }
      uint32_t pb[NT][2];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float e[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) e[i] = fast_exp2(x[nt][i] - (mref[nt][i & 1] - kPShift));
        l[nt][0] += e[0] + e[2];
        l[nt][1] += e[1] + e[3];
        // key g x rows 2t, 2t+1  ->  row g x keys 2t, 2t+1
        pb[nt][0] = transpose8x8(pack_f16x2(e[0], e[1]));
        pb[nt][1] = transpose8x8(pack_f16x2(e[2], e[3]));
      }

      // ---- O^T += V^T P^T
      // the lane's keys, in operand order 2t, 2t+1, 2t+8, 2t+9: t, 4+t, 8+t, 12+t; dims 16 g ..
      const uint32_t vb = st + FS_V + (gr * 16 + t) * kFp4RowBytes + ((((g >> 1) ^ (((t >> 1) & 1) << 1))) << 4) + (g & 1) * 8;
      const uint32_t sb = st + FS_VS + (gr * 16 + t) * kFp4Blocks + g;
      uint2 w[4];
      uint32_t sc[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        w[j] = lds64(vb + 4 * j * kFp4RowBytes);
        sc[j] = lds_u8(sb + 4 * j * kFp4Blocks);
      }
      if (edge) {
        // Keys that no row sees: scale zero, so that their values (a NaN scale,
        // an unwritten row) do not reach the sum.  A NaN scale that some rows
        // see spoils its 16 dims of those rows, which the lane's quad holds; as
        // an operand it would spoil every row (0 * NaN).
        bool bad = false;
        int vk[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int k = gr * 16 + 4 * j + t;
          vk[j] = POS ? __shfl_sync(full, pos_lane, k) : key0 + k;
          if (vk[j] > qmax || (unsigned)max(qmin - vk[j], 0) >= wlim) sc[j] = 0;
          bad |= (sc[j] & 0x7f) == 0x7f;
        }
        if (__any_sync(full, bad)) {
#pragma unroll 1
          for (int src = 0; src < 4; ++src)
#pragma unroll 1
            for (int j = 0; j < 4; ++j) {
              const int mine = j == 0 ? vk[0] : j == 1 ? vk[1] : j == 2 ? vk[2] : vk[3];
              const uint32_t sj = j == 0 ? sc[0] : j == 1 ? sc[1] : j == 2 ? sc[2] : sc[3];
              const int v = __shfl_sync(full, mine, src, 4);
              const bool nan = (__shfl_sync(full, sj, src, 4) & 0x7f) == 0x7f;
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int c = 0; c < 2; ++c)
                  if (nan && (unsigned)qp[nt][c] - (unsigned)v < wlim)
#pragma unroll
                    for (int m = 0; m < 8; ++m) acc[m][nt][c] = acc[m][nt][c + 2] = __int_as_float(0x7fffffff);
            }
#pragma unroll
          for (int j = 0; j < 4; ++j)
            if ((sc[j] & 0x7f) == 0x7f) sc[j] = 0;
        }
      }
      const uint32_t s0 = e4m3x2_to_f16(sc[0] | (sc[1] << 8)), s1 = e4m3x2_to_f16(sc[2] | (sc[3] << 8));
#pragma unroll
      for (int hw = 0; hw < 2; ++hw) {
        const uint32_t A = hw ? w[0].y : w[0].x, B = hw ? w[1].y : w[1].x;
        const uint32_t C = hw ? w[2].y : w[2].x, E = hw ? w[3].y : w[3].x;
        const uint32_t nib = 0x0f0f0f0fu;
        uint32_t f0[4], f1[4], f2[4], f3[4];
        e2m1x8_to_f16((A & nib) | ((B << 4) & ~nib), f0);
        e2m1x8_to_f16(((A >> 4) & nib) | (B & ~nib), f1);
        e2m1x8_to_f16((C & nib) | ((E << 4) & ~nib), f2);
        e2m1x8_to_f16(((C >> 4) & nib) | (E & ~nib), f3);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          f0[i] = hmul2(f0[i], s0), f1[i] = hmul2(f1[i], s0);
          f2[i] = hmul2(f2[i], s1), f3[i] = hmul2(f3[i], s1);
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
            mma_f16_16816(acc[4 * hw + i][nt], f0[i], f1[i], f2[i], f3[i], pb[nt][0], pb[nt][1]);
        }
      }
    }
  }
  cp_async_wait<0>();

  // ---- merge the warps
  __syncthreads();                           // every ring is idle
  float *so = reinterpret_cast<float *>(smem);                   // [warp][row][128]
  float *sm = so + FW * kFp4Rows * kHeadDim, *sl = sm + FW * kFp4Rows;
  long *sg = reinterpret_cast<long *>(sl + FW * kFp4Rows);       // [head of the CTA][row]: output row
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      float z = l[nt][c];
      z += __shfl_xor_sync(full, z, 4);
      z += __shfl_xor_sync(full, z, 8);
      z += __shfl_xor_sync(full, z, 16);
      const int row = nt * 8 + 2 * t + c;
      if (g == 0) {
        sm[warp * kFp4Rows + row] = mref[nt][c];
        sl[warp * kFp4Rows + row] = z;
      }
#pragma unroll
      for (int m = 0; m < 8; ++m)
        *reinterpret_cast<float2 *>(so + (warp * kFp4Rows + row) * kHeadDim + 16 * g + 2 * m) =
            make_float2(acc[m][nt][c], acc[m][nt][c + 2]);
    }
  __syncthreads();
  // a thread per (head, row): the warps' factors, lse and the output row
  const long rows_all = (long)p.a.total_q * p.a.Hq;
  if (tid < kFp4Rows * p.hp) {
    const int hs = tid / kFp4Rows, row = tid % kFp4Rows, h = u.h - warp % p.hp + hs;
    float m = kNone, z = 0.f, f[FW];
#pragma unroll
    for (int w = 0; w < FW; ++w)
      if (w % p.hp == hs) m = fmaxf(m, sm[w * kFp4Rows + row]);
#pragma unroll
    for (int w = 0; w < FW; ++w) {
      f[w] = 0.f;
      if (w % p.hp == hs) {
        const float mw = sm[w * kFp4Rows + row], zw = sl[w * kFp4Rows + row];
        // (a warp without a visible key has an empty sum; a NaN sum stays one)
        f[w] = fast_exp2(mw - m);
        z = fmaf(zw, f[w], z);
      }
    }
    const float scale = z == 0.f ? 0.f : (p.kv.v_global ? __ldg(p.kv.v_global + h) : 1.f) / z;
#pragma unroll
    for (int w = 0; w < FW; ++w)
      if (w % p.hp == hs) sl[w * kFp4Rows + row] = f[w] * scale;
    const float lse = z == 0.f ? -INFINITY : (m - kPShift + log2f(z)) * kLn2;
    if (row < u.nrows) {
      const int rr = u.rb * kFp4Rows + row, tok = u.s.q0 + rr / p.a.group;
      const int head = h * p.a.group + rr % p.a.group;
      const long grow = (long)tok * p.a.Hq + head;
      sg[tid] = grow;
      if (p.splits == 1) p.a.lse[(long)head * p.a.total_q + tok] = lse;
      else p.a.lse_part[(long)slot * rows_all + grow] = lse;
    }
  }
  __syncthreads();
  for (int hs = 0; hs < p.hp; ++hs)
#pragma unroll 4
    for (int row = 0; row < u.nrows; ++row) {
      float o = 0.f;
#pragma unroll
      for (int w = 0; w < FW; ++w)
        if (w % p.hp == hs) o = fmaf(so[(w * kFp4Rows + row) * kHeadDim + tid], sl[w * kFp4Rows + row], o);
      const long grow = sg[hs * kFp4Rows + row];
      if (p.splits == 1) p.a.out[grow * kHeadDim + tid] = __float2bfloat16_rn(o);
      else p.a.o_part[((long)slot * rows_all + grow) * kHeadDim + tid] = o;
    }
  __syncthreads();                           // the merge buffers become rings again
}

template <int NT, bool POS>
__global__ void __launch_bounds__(FT, ctas_per_sm(NT)) relattn_decode_fp4_kernel(const __grid_constant__ Fp4DecodeArgs p) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int prefix[kWalkBatch + 1];
  __shared__ int wsum[FW];
  const int tid = threadIdx.x, hsub = (tid >> 5) % p.hp;
  // the merge kernel may take its place beside the last CTAs; it waits for this grid
  asm volatile("griddepcontrol.launch_dependents;");
  Unit u;
  // head group and row block of unit group hr; the warp's head
  auto place = [&](int hr) {
    u.rb = hr % p.row_blocks;
    u.h = hr / p.row_blocks * p.hp + hsub;
    u.nrows = min(kFp4Rows, u.s.lq * p.a.group - u.rb * kFp4Rows);
    u.qbase = first_query_pos(u.s, p.q_pos, u.b);
  };
  unsigned per = 0, total = 0;               // tiles of a unit group, and of all (the plan keeps them below 2^31)
  if (p.whole) {                             // one CTA per unit
    const int hr = blockIdx.x / p.a.batch;
    u.b = blockIdx.x - hr * p.a.batch;
    const int n = unit_tiles(p, u.b, &u.s, &u.lo);
    if (n < 0 && tid == 0) atomicOr(p.a.err, kDevErrSeqlens);
    total = max(n, 0);
    place(hr);
  } else {
    per = tile_prefix<FT>(p, prefix, wsum);
    total = per * (unsigned)(p.a.Hkv / p.hp * p.row_blocks);
  }
  Ranges at(p, total, kFp4MostTiles);
  while (at.x < at.end) {
    const Piece c = next_piece(p, at, u, prefix, per, place);
    if (u.nrows <= 0) continue;
    // mark slots without a piece: the first piece those past the last, a range within a tile its own
    const int from = c.tiles > 0 ? c.used : c.slot, to = c.tiles > 0 ? p.splits : c.slot + 1;
    if (c.t0 == 0 || c.tiles == 0)
      for (int i = tid; i < u.nrows * p.hp; i += FT) {
        const int hs = i / u.nrows, rr = u.rb * kFp4Rows + i % u.nrows;
        const long grow = (long)(u.s.q0 + rr / p.a.group) * p.a.Hq + (u.h - hsub + hs) * p.a.group + rr % p.a.group;
        for (int k = from; k < to; ++k) p.a.lse_part[(long)k * p.a.total_q * p.a.Hq + grow] = -INFINITY;
      }
    if (c.tiles > 0) run_piece<NT, POS>(p, u, c.t0, c.tiles, c.slot, smem);
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// out / lse of one row from its partials; rows of no (valid) sequence are left
// as they are.  A CTA per row, its warps taking the slots in turn.
__global__ void __launch_bounds__(FT) relattn_decode_fp4_combine_kernel(const __grid_constant__ Fp4DecodeArgs p) {
  __shared__ float red_m[FW], red_z[FW];
  __shared__ float4 red_o[FW][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long row = blockIdx.x, rows = (long)p.a.total_q * p.a.Hq;
  const int tq = (int)(row / p.a.Hq);
  SeqRows s;
  int first;
  const int tiles = unit_tiles(p, last_not_above(p.a.cu_q, p.a.batch, tq), &s, &first);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  if (tiles <= 0 || tq < s.q0 || tq >= s.q0 + s.lq) return;
  float m = -INFINITY;
  bool nan = false;
  for (int i = threadIdx.x; i < p.splits; i += FT) {
    const float v = p.a.lse_part[i * rows + row];
    m = fmaxf(m, v);
    nan |= v != v;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  if (lane == 0) red_m[warp] = m;
  nan = __syncthreads_or(nan);
#pragma unroll
  for (int w = 0; w < FW; ++w) m = fmaxf(m, red_m[w]);
  if (nan) m = 0.f;                          // the weights below turn NaN by themselves
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  float z = 0.f;
  if (m != -INFINITY)
    for (int i0 = warp; i0 < p.splits; i0 += 4 * FW) {       // four slots' loads in flight together
      float ls[4];
      float4 v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const int i = i0 + k * FW;
        ls[k] = i < p.splits ? p.a.lse_part[i * rows + row] : -INFINITY;
      }
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (ls[k] != -INFINITY)
          v[k] = *reinterpret_cast<const float4 *>(p.a.o_part + ((i0 + k * FW) * rows + row) * kHeadDim + lane * 4);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (ls[k] == -INFINITY) continue;
        const float f = exp2f((ls[k] - m) * kLog2e);
        z += f;
        acc.x = fmaf(f, v[k].x, acc.x);
        acc.y = fmaf(f, v[k].y, acc.y);
        acc.z = fmaf(f, v[k].z, acc.z);
        acc.w = fmaf(f, v[k].w, acc.w);
      }
    }
  red_o[warp][lane] = acc;
  if (lane == 0) red_z[warp] = z;
  __syncthreads();
  if (warp != 0) return;
#pragma unroll
  for (int w = 1; w < FW; ++w) {
    const float4 o = red_o[w][lane];
    acc.x += o.x, acc.y += o.y, acc.z += o.z, acc.w += o.w;
    z += red_z[w];
  }
  const float inv = z == 0.f ? 0.f : 1.f / z;
  uint2 packed;
  packed.x = pack_bf16x2(acc.x * inv, acc.y * inv);
  packed.y = pack_bf16x2(acc.z * inv, acc.w * inv);
  *reinterpret_cast<uint2 *>(p.a.out + row * kHeadDim + lane * 4) = packed;
  if (lane == 0) p.a.lse[(row - (long)tq * p.a.Hq) * p.a.total_q + tq] = z == 0.f ? -INFINITY : m + logf(z);
}

template <int NT, bool POS>
cudaError_t launch_main(const Fp4DecodeArgs &p, cudaStream_t stream) {
  static std::atomic<bool> done[kMaxDevicesAttr];
  auto *kernel = relattn_decode_fp4_kernel<NT, POS>;
  const cudaError_t e = set_max_smem_once(reinterpret_cast<const void *>(kernel), F_RING, done);
  if (e != cudaSuccess) return e;
  const long grid = p.whole ? (long)p.a.batch * (p.a.Hkv / p.hp) * p.row_blocks : (long)p.a.sms * ctas_per_sm(NT);
  if (grid > 0x7fffffffL) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(FT);
  cfg.dynamicSmemBytes = F_RING;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = p.a.E > 0 ? 1 : 0;          // behind the R kernel
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

// Rows of a kv head past which the tcgen05 kernel is taken.  It costs the same
// for 1 and 128 rows; here every 16 rows convert the cache again.  Measured (us,
// this / that; 2 kv heads, E = 1024), 32, 40 and 128 rows: one sequence of 16384
// keys 27 / 27, 28 / 27, 40 / 31; of 131072 64 / 43, 71 / 43, 111 / 48; 64
// of 8192 137 / 155, 177 / 158, 478 / 195.  From 40 rows on that one is the
// better throughout.  At 32 it depends on the keys of a CTA, which this rule does
// not look at: it keeps the batch at 137 and leaves one long sequence at 64.
constexpr int kTcMinRows = 32;
// Its tiles that meet the bias band take some seven times as long as the others:
// 175 us for 72 rows of a million keys and E = 1024, 208 with a weight of four.
// (This weight and the next were measured at E = 1024 only.)
constexpr int kTcBandExtra = 6;
// And of this kernel about twice as long (64 sequences of 1 to 32 thousand keys:
// 97 us, 104 without weights, 100 with three times).
constexpr int kBandExtra = 1;

bool two_columns(const KernelArgs &a) { return a.max_q * a.group > 8; }

}  // namespace

// Slots, workspace and the least tiles of a range.  A unit holds at most U
// tiles and meets at most ceil(U / C) + 1 ranges of C tiles, so C >= U /
// (slots - 1) keeps its pieces within the slots.  A unit meets no more ranges than
// there are (CTAs x waves), so as many slots do for any C: max_k may be a bound far
// above the lengths.  A unit that has a CTA of its own is cut into pieces only
// where it is too long for one, by its own length and the slots.  False when the
// sizes do not fit the kernel's index types.
bool plan_decode_fp4(const KernelArgs &a, long total_k, bool positions, int want_splits, Fp4DecodePlan *plan) {
  const int rows = a.max_q * a.group;
  plan->tc = rows > kTcMinRows && !positions;
  const int block = plan->tc ? kFp4TcRows : kFp4Rows;
  plan->row_blocks = (rows + block - 1) / block;
  long vis = a.max_k;
  if (a.window > 0 && !positions) vis = std::min<long>(vis, (long)a.window + a.max_q - 1 + FK - 1);
  plan->hp = a.Hkv % 2 == 0 && !plan->tc ? 2 : 1;
  const long tile = kWalkTile / plan->hp;
  long U = (vis + tile - 1) / tile;
  const long band = a.E > 0 ? std::min<long>(U, ((long)a.E + a.max_q) / tile + 2) : 0;
  plan->band_extra = a.E == 0 ? 0 : plan->tc ? kTcBandExtra : kBandExtra;
  U += plan->band_extra * band;              // (tiles of the band are weighted)
  const long keys = std::min<long>(total_k, (long)a.batch * vis);
  const long heads = (long)(a.Hkv / plan->hp) * plan->row_blocks;
  const long total = (keys / tile + a.batch * (1 + plan->band_extra * band)) * heads;
  const long grid = (long)a.sms * (plan->tc ? 1 : ctas_per_sm(two_columns(a) ? 2 : 1));
  // A piece's fixed cost is that of a few tiles, and partials cost a second
  // kernel: up to 8 tiles stay whole (one sequence of 8 tiles, caches cold: 18.6 us
  // whole, 22.7 in pieces of two; 12 tiles 25.7 and 24.7).
  const long kMinTiles = plan->tc ? 4 : 2, kWhole = plan->tc ? 0 : 8;
  const long most = plan->tc ? kFp4TcMostTiles : kFp4MostTiles;
  const long share = std::max<long>((total + grid - 1) / grid, kMinTiles), waves = (share + most - 1) / most;
  const long C = (share + waves - 1) / waves, ranges = grid * waves;
  // pieces that the longest sequence needs, which total_k bounds as well
  const long pieces = (std::min<long>(U, total_k / tile + 1 + plan->band_extra * band) + most - 1) / most;
  const long least = want_splits > 0 ? 1 : kMinTiles;
  long splits = std::max<long>(pieces, 1);
  plan->whole = a.batch > kWalkBatch || want_splits == 1 || (want_splits <= 0 && U <= std::max(C, kWhole));
  if (!plan->whole) {
    splits = want_splits > 0 ? std::max<long>(want_splits, pieces > 1 ? pieces + 1 : 2) : (U + C - 1) / C + 1;
    splits = std::min(std::min<long>(splits, U + 1), ranges);
    plan->whole = splits == 1;
  }
  plan->splits = (int)splits;
  plan->waves = (int)waves;
  plan->c_min = plan->whole ? 0 : splits == ranges ? (int)least : (int)std::max<long>((U + splits - 2) / (splits - 1), least);
  const size_t rows_all = (size_t)a.total_q * a.Hq;
  size_t end = 0;
  plan->lse_offset = 0;
  if (splits > 1) {
    plan->lse_offset = ((size_t)splits * rows_all * kHeadDim * sizeof(float) + 255) / 256 * 256;
    end = plan->lse_offset + (size_t)splits * rows_all * sizeof(float);
  }
  plan->rel_offset = (end + 255) / 256 * 256;
  plan->ws_bytes = a.E > 0 ? plan->rel_offset + rows_all * a.E * sizeof(float) : end;
  return rows_all <= 0x7fffffffUL && (long)a.batch * heads <= 0x7fffffffL &&
         ((long)a.batch * U + grid) * heads <= 0x7fffffffL;
}

cudaError_t launch_decode_fp4(const Fp4DecodeArgs &p, cudaStream_t stream) {
  if (p.a.E > 0) {
    const cudaError_t e = launch_rel_bias(p.a.r, p.a.P, (long)p.a.total_q * p.a.Hq, p.a.rd, p.a.E,
                                          const_cast<float *>(p.a.rdec), stream);
    if (e != cudaSuccess) return e;
  }
  cudaError_t e;
  if (p.tc) e = launch_decode_fp4_tc(p, stream);
  else if (two_columns(p.a)) e = p.key_pos ? launch_main<2, true>(p, stream) : launch_main<2, false>(p, stream);
  else e = p.key_pos ? launch_main<1, true>(p, stream) : launch_main<1, false>(p, stream);
  if (e != cudaSuccess || p.splits == 1) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((long)p.a.total_q * p.a.Hq));
  cfg.blockDim = dim3(FT);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, relattn_decode_fp4_combine_kernel, p);
}

}  // namespace relattn

// key_weights.cu -- the attention weight that every cached key receives,
//   w_out[h][j] = decay * w_in[h][j] + sum_{i, heads of group h} exp(x_ij - lse_i),
// from the saved logsumexp of the rows (x_ij as in the decode kernels: page
// "SGLang and Miles Add Day-0 Support for Inkling", section "Attention with
// Relative Positional Embedding").  It is what eviction ranks the keys by.
// With lse known there is no running maximum and no order among keys: a key's
// sum stays in registers from its first row to its last (fp32, one order, no
// atomics), and only K is read.
//
// Keys go along the matrix instruction's 16 rows, query rows along its 8
// columns, so a lane holds two keys' logits for two rows and a sum over rows
// is a sum in the lane and, once at the end, over four lanes.  K is bf16 (bf16
// products) or 4-bit (codes times scales, exact in f16, as in decode_fp4.cu).
//
//   few rows (at most 16 per kv head, a decode step): the walk of the decode,
//     a warp streams 32 keys at a time through its own ring.  64 sequences of 1 to 32
//     thousand keys, group 8: 4-bit keys 70 us, 2.5 TB/s of what must be read and
//     written, with no pipe full (issue slots 63 % busy, mostly conversions; DRAM
//     37 %); bf16 keys 122 us, 4.7 TB/s.
//   many rows: a CTA holds 128 keys as operands in registers and takes the
//     rows that see them 32 at a time through shared memory; bound by the
//     matrix instruction and the exponentials.  The bias is a product too:
//     key j and a row at position i meet column i - j of P, so a table of P's
//     columns in falling order makes the 16 keys' bias columns 16 consecutive
//     rows, and P^T r^T of one token's rows is 4 more instructions of the
//     same shape, its operand read from shared memory at the token's offset.
//     Nothing of size rows x E is ever stored.
//   many rows of the usual shapes: the tcgen05 kernel of key_weights_tc.cu
//     takes them all (32 tokens of 4 sequences of 16 to 64 thousand keys: 70 us,
//     240 here), or (r rows that TMA cannot read) those past the bias band and
//     adds to these sums.
#include <algorithm>

#include "key_weights.cuh"

namespace relattn {
namespace {

constexpr int WW = 4, WT = WW * 32, WK = kWalkTile / WW;
static_assert(WK == 32, "two 16-key groups");
constexpr int W_STAGES = 3;
constexpr int kColdKeys = 1024;              // keys out of every row's sight that a CTA takes at a time

template <bool FP4>
struct KStage {
  static constexpr int row = FP4 ? kFp4RowBytes : kHeadDim * 2;
  static constexpr int scales = WK * row;
  static constexpr int bytes = scales + (FP4 ? WK * kFp4Blocks : 0);
  static constexpr int ring = WW * W_STAGES * bytes;
};

// Key of row g of a 16-key operand (its other key is 8 further): the 4-bit
// layout of decode_fp4.cu, or the natural one.
template <bool FP4>
__device__ __forceinline__ int operand_key(int g) {
  return FP4 ? (g >> 1) + 4 * (g & 1) : g;
}

template <bool FP4>
__device__ __forceinline__ void issue_keys(const KeyWeightArgs &p, const Unit &u, uint32_t st, int key0, long row0,
                                           int lane) {
  if (FP4) {
    const long rb = (long)p.a.Hkv * kFp4RowBytes;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int k = (lane >> 2) + 8 * i, c = lane & 3, k16 = k & 15;
      const bool ok = row0 >= 0 && key0 + k < u.s.lk;
      const long off = ok ? (row0 + k) * rb + u.h * kFp4RowBytes + c * 16 : 0;
      const int slot = (k & 16) + (k16 & 8) + 2 * (k16 & 3) + ((k16 >> 2) & 1);
      cp_async16(st + slot * kFp4RowBytes + c * 16, p.kv.k + off, ok);
    }
    const bool ok = row0 >= 0 && key0 + lane < u.s.lk;
    cp_async8(st + KStage<true>::scales + lane * kFp4Blocks,
              p.kv.k_scale + (ok ? ((row0 + lane) * p.a.Hkv + u.h) * kFp4Blocks : 0), ok);
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const int k = (lane >> 4) + 2 * i, c = lane & 15;
      const bool ok = row0 >= 0 && key0 + k < u.s.lk;
      const long off = ok ? ((row0 + k) * p.a.Hkv + u.h) * kHeadDim + c * 8 : 0;
      cp_async16(st + k * 256 + ((c ^ (k & 7)) << 4), p.k + off, ok);
    }
  }
}

// The A operand of one 16-key group and 16-dim step s from a stage.
template <bool FP4>
__device__ __forceinline__ void key_operands(uint32_t st, int gr, int lane, uint32_t (&f)[8][4]) {
  const int g = lane >> 2, t = lane & 3;
  if (FP4) {
    const uint32_t kb = st + gr * 16 * kFp4RowBytes + t * 16;
    const uint4 w0 = lds128(kb + g * kFp4RowBytes), w1 = lds128(kb + (g + 8) * kFp4RowBytes);
    const uint32_t sb = st + KStage<true>::scales + (gr * 16 + operand_key<true>(g)) * kFp4Blocks + 2 * t;
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
      for (int i = 0; i < 2; ++i) {
        f[2 * w + i][0] = hmul2(f0[2 * i], m0);
        f[2 * w + i][1] = hmul2(f1[2 * i], m1);
        f[2 * w + i][2] = hmul2(f0[2 * i + 1], m0);
        f[2 * w + i][3] = hmul2(f1[2 * i + 1], m1);
      }
    }
  } else {
    const int row = gr * 16 + (lane & 7) + (((lane >> 3) & 1) << 3);
#pragma unroll
    for (int s = 0; s < 8; ++s)
      ldsm_x4(st + row * 256 + (((2 * s + (lane >> 4)) ^ (row & 7)) << 4), f[s][0], f[s][1], f[s][2], f[s][3]);
  }
}

template <bool FP4>
__device__ __forceinline__ void key_mma(float (&d)[4], const uint32_t (&f)[4], uint32_t b0, uint32_t b1) {
  if (FP4) mma_f16_16816(d, f[0], f[1], f[2], f[3], b0, b1);
  else mma_bf16_16816(d, f[0], f[1], f[2], f[3], b0, b1);
}

// Sum of v[0..3] over the quad's four lanes; lane t ends with v[t]'s.
__device__ __forceinline__ float quad_reduce(const float (&v)[4], int t) {
  const unsigned full = 0xffffffffu;
  const float a = (t & 1) ? v[0] : v[1], b = (t & 1) ? v[2] : v[3];      // given away
  const float x = ((t & 1) ? v[1] : v[0]) + __shfl_xor_sync(full, a, 1);
  const float y = ((t & 1) ? v[3] : v[2]) + __shfl_xor_sync(full, b, 1);
  return ((t & 2) ? y : x) + __shfl_xor_sync(full, (t & 2) ? x : y, 2);
}

// ------------------------------------------------------------------ few rows

template <int NT, bool POS, bool FP4>
__device__ __forceinline__ void weigh_piece(const KeyWeightArgs &p, const Unit &u, int t0, int n, uint8_t *smem) {
  constexpr int SB = KStage<FP4>::bytes;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const uint32_t ring = smem_addr(smem) + warp * (W_STAGES * SB);
  const int tile = kWalkTile / p.hp;        // keys of a tile
  const int k_first = u.lo + t0 * tile + warp / p.hp * WK;
  const unsigned full = 0xffffffffu;
  long rows_q[W_STAGES];                    // cache rows of the groups in flight, then the next to copy
#pragma unroll
  for (int i = 0; i < W_STAGES; ++i) {
    rows_q[i] = i < n ? group_row(p, u, k_first + i * tile) : -1;
    if (i < W_STAGES - 1) {
      if (i < n) issue_keys<FP4>(p, u, ring + i * SB, k_first + i * tile, rows_q[i], lane);
      cp_async_commit();
    }
  }
  bool waited = false;                      // for the kernel before this one: R

  uint32_t qf[NT][16];
  float coef[NT][2], bscale[NT][2], lse2[NT][2];
  int qp[NT][2], rrow[NT][2];               // position (-1: no row, or one that gives nothing), row of R
  bool whole = true;                        // every slot holds a row that gives something
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    const int nrow = nt * 8 + g;
    int tok = 0;
    float back = 1.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) qf[nt][i] = 0;
    if (nrow < u.nrows) {
      const __nv_bfloat16 *qrow = p.a.q + unit_row(p, u, nrow, &tok) * kHeadDim;
      if (FP4) {                            // dims 32 t .., f16
        const uint4 *src = reinterpret_cast<const uint4 *>(qrow + t * 32);
        uint32_t top = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 w = __ldg(src + i);
          const uint32_t ws[4] = {w.x, w.y, w.z, w.w};
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
      } else {                              // dims 16 s + 2 t (+1), + 8: bf16 as they are
        const uint32_t *src = reinterpret_cast<const uint32_t *>(qrow) + t;
#pragma unroll
        for (int s = 0; s < 8; ++s) {
          qf[nt][2 * s] = __ldg(src + 8 * s);
          qf[nt][2 * s + 1] = __ldg(src + 8 * s + 4);
        }
      }
    }
    __syncwarp();
    const float kg = FP4 && p.kv.k_global ? __ldg(p.kv.k_global + u.h) : 1.f;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int m = nt * 8 + 2 * t + c;
      const float bk = __shfl_sync(full, back, (2 * t + c) * 4);
      int tk;
      const bool live = m < u.nrows;
      const long grow = unit_row(p, u, live ? m : 0, &tk);
      rrow[nt][c] = (int)grow;
      const float s = live ? log_scale(u.qbase + tk, p.a.inv_ln_base) : 0.f;
      coef[nt][c] = p.a.alpha_log2e * s * kg * bk;
      bscale[nt][c] = s * kLog2e;
      // A row that saw nothing (lse -inf), and one past the block, give nothing:
      // masked, since 0 times an infinite or NaN key is not 0.
      const float z = live ? __ldg(p.lse + (grow % p.a.Hq) * p.a.total_q + grow / p.a.Hq) : -INFINITY;
      const bool gives = z != -INFINITY;
      whole = whole && gives;
      qp[nt][c] = gives ? u.qbase + tk : -1;
      lse2[nt][c] = gives ? z * kLog2e : INFINITY;
    }
  }
  int qmin, qmax, tk_;
  unit_row(p, u, 0, &tk_);
  qmin = u.qbase + tk_;
  unit_row(p, u, u.nrows - 1, &tk_);
  qmax = u.qbase + tk_;
  const unsigned wlim = p.a.window > 0 ? (unsigned)p.a.window : 0x80000000u;
  if (!__all_sync(full, whole)) qmax = -1;   // every key needs the mask

  int buf = 0;
  for (int it = 0; it < n; ++it) {
    const int key0 = k_first + it * tile;
    cp_async_wait<W_STAGES - 2>();
    __syncwarp();
    const long row0 = rows_q[0];
    {
      const int nb = buf == 0 ? W_STAGES - 1 : buf - 1;
      if (it + W_STAGES - 1 < n) issue_keys<FP4>(p, u, ring + nb * SB, key0 + (W_STAGES - 1) * tile, rows_q[W_STAGES - 1], lane);
      cp_async_commit();
    }
#pragma unroll
    for (int i = 0; i + 1 < W_STAGES; ++i) rows_q[i] = rows_q[i + 1];
    rows_q[W_STAGES - 1] = it + W_STAGES < n ? group_row(p, u, key0 + W_STAGES * tile) : -1;
    const uint32_t st = ring + buf * SB;
    buf = buf == W_STAGES - 1 ? 0 : buf + 1;
    if (key0 >= u.s.lk) continue;
    int kp_lane = 0x7fffffff;
    if (POS && row0 >= 0 && key0 + lane < u.s.lk) {
      kp_lane = __ldg(p.key_pos + (long)u.h * p.pages.rows + row0 + lane);
      if (kp_lane < 0) kp_lane = 0x7fffffff;
    }
    const bool edge = POS || key0 + WK - 1 > qmin || (unsigned)(qmax - key0) >= wlim;
    const bool band = p.a.E > 0 && (POS ? __any_sync(full, kp_lane != 0x7fffffff && qmin - kp_lane < p.a.E)
                                        : qmin - (key0 + WK - 1) < p.a.E);
    if (band && !waited) {
      asm volatile("griddepcontrol.wait;" ::: "memory");
      waited = true;
    }
    float v[4];                              // keys operand_key(g) + 8 hf + 16 gr at 2 gr + hf
#pragma unroll
    for (int gr = 0; gr < 2; ++gr) {
      int kp[2];
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        const int k = gr * 16 + hf * 8 + operand_key<FP4>(g);
        kp[hf] = POS ? __shfl_sync(full, kp_lane, k) : key0 + k;
        v[2 * gr + hf] = 0.f;
      }
      float x[NT][4], bias[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) x[nt][i] = bias[nt][i] = 0.f;
      if (band) {                            // ahead of the products, which hide its latency
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const unsigned d = (unsigned)qp[nt][i & 1] - (unsigned)kp[i >> 1];
            if (d < (unsigned)p.a.E) bias[nt][i] = p.a.rdec[(long)rrow[nt][i & 1] * p.a.E + d];
          }
      }
      uint32_t f[8][4];
      key_operands<FP4>(st, gr, lane, f);
#pragma unroll
      for (int s = 0; s < 8; ++s)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) key_mma<FP4>(x[nt], f[s], qf[nt][2 * s], qf[nt][2 * s + 1]);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float y = fmaf(x[nt][i], coef[nt][i & 1], -lse2[nt][i & 1]);
          if (band) y = fmaf(bias[nt][i], bscale[nt][i & 1], y);
          float e = fast_exp2(y);
          if (edge && (unsigned)qp[nt][i & 1] - (unsigned)kp[i >> 1] >= wlim) e = 0.f;
          v[2 * gr + (i >> 1)] += e;
        }
    }
    const float sum = quad_reduce(v, t);
    const int key = key0 + (t >> 1) * 16 + (t & 1) * 8 + operand_key<FP4>(g);
    if (row0 >= 0 && key < u.s.lk) write_weight(p, u, key, row0 + (key - key0), sum);
  }
  cp_async_wait<0>();
  __syncwarp();
}

// CTAs of an SM: bounded by registers (4-bit keys) or the ring (bf16 keys).
constexpr int rows_ctas(int nt, bool fp4) { return fp4 ? (nt == 1 ? 5 : 3) : 2; }

template <int NT, bool POS, bool FP4>
__global__ void __launch_bounds__(WT, rows_ctas(NT, FP4)) relattn_key_weights_rows_kernel(const __grid_constant__ KeyWeightArgs p) {
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int prefix[kWalkBatch + 1];
  __shared__ int wsum[WW];
  const int base = tile_prefix<WT>(p, prefix, wsum);
  const long per = base, total = per * (p.a.Hkv / p.hp);
  const long C = (total + gridDim.x - 1) / gridDim.x;
  long x = blockIdx.x * C;
  const long end = min(total, x + C);
  Unit u;
  u.rb = 0;
  while (x < end) {
    const int hg = (int)(x / per), xb = (int)(x - hg * per);
    u.h = hg * p.hp + (int)(threadIdx.x >> 5) % p.hp;
    u.b = last_not_above(prefix, p.a.batch, xb);
    const int real = unit_tiles(p, u.b, &u.s, &u.lo), v0 = xb - prefix[u.b];
    const Weighted w = weighted_tiles(p, u.s, u.lo, real);
    const int n = (int)min((long)(w.total - v0), end - x), t0 = w.tile(v0), tiles = w.tile(v0 + n) - t0;
    u.nrows = u.s.lq * p.a.group;
    u.qbase = first_query_pos(u.s, p.q_pos, u.b);
    if (tiles > 0) weigh_piece<NT, POS, FP4>(p, u, t0, tiles, smem);
    x += n;
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// ------------------------------------------------------------------ many rows

constexpr int QR = 32;                       // query rows staged at a time
constexpr int TR = 256;                      // rows of the bias table in shared memory, a ring
// shared memory: K as operands, then (its place) the ring; two stages of q and r rows
constexpr int ST_Q = WW * WK * 256, ST_R = ST_Q + 2 * QR * 256, ST_C = ST_R + 2 * QR * 128;
constexpr int ST_BYTES = ST_C + 2 * QR * 5 * 4;
static_assert(TR * 128 <= ST_Q && TR >= 128 + 2 * QR, "two stages' table rows fit the ring");

template <bool POS>
__global__ void __launch_bounds__(WT, 3) relattn_key_weights_tiles_kernel(const __grid_constant__ KeyWeightArgs p) {
  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, t = lane & 3;
  const unsigned full = 0xffffffffu;
  Unit u;
  u.rb = 0;
  u.b = blockIdx.y / p.a.Hkv;
  u.h = blockIdx.y - u.b * p.a.Hkv;
  const int ok = unit_tiles(p, u.b, &u.s, &u.lo);
  if (ok < 0 && blockIdx.x == 0 && u.h == 0 && tid == 0) atomicOr(p.a.err, kDevErrSeqlens);
  const int tile0 = blockIdx.x * kWalkTile, key0 = tile0 + warp * WK;
  if (ok < 0 || tile0 >= u.s.lk) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    return;
  }
  u.qbase = u.s.lq > 0 ? first_query_pos(u.s, p.q_pos, u.b) : 0;
  const unsigned wlim = p.a.window > 0 ? (unsigned)p.a.window : 0x80000000u;
  // tokens that may see a key of the tile, less those the tcgen05 kernel takes
  int tok0 = 0, tok1 = u.s.lq;
  if (!POS) {
    tok0 = max(0, tile0 - u.qbase);
    const long last = (long)min(tile0 + kWalkTile, u.s.lk) - 1 + wlim - u.qbase;   // first token past the window
    if (last < tok1) tok1 = (int)max(last, 0L);
    if (p.tc) tok1 = min(tok1, tc_first_token(p, u.qbase, tile0));
  }
  const long row0 = group_row(p, u, key0);
  uint32_t f[2][8][4];
  if (tok0 < tok1) {
    load_key_tile<WT>(p, u, tile0, tid, [&](int k, int c) { return smem + k * 256 + ((c ^ (k & 7)) << 4); });
    __syncthreads();
    const uint32_t sk = smem_addr(smem) + warp * WK * 256;
#pragma unroll
    for (int gr = 0; gr < 2; ++gr) {
      const int row = gr * 16 + (lane & 7) + (((lane >> 3) & 1) << 3);
#pragma unroll
      for (int s = 0; s < 8; ++s)
        ldsm_x4(sk + row * 256 + (((2 * s + (lane >> 4)) ^ (row & 7)) << 4), f[gr][s][0], f[gr][s][1], f[gr][s][2], f[gr][s][3]);
    }
    __syncthreads();                         // the table ring takes K's place
  }
  int kp[2][2], kp_lane = 0x7fffffff;
  if (POS && row0 >= 0 && key0 + lane < u.s.lk) {
    kp_lane = __ldg(p.key_pos + (long)u.h * p.pages.rows + row0 + lane);
    if (kp_lane < 0) kp_lane = 0x7fffffff;
  }
#pragma unroll
  for (int gr = 0; gr < 2; ++gr)
#pragma unroll
    for (int hf = 0; hf < 2; ++hf) {
      const int k = gr * 16 + hf * 8 + g;
      kp[gr][hf] = POS ? __shfl_sync(full, kp_lane, k) : key0 + k;
    }
  asm volatile("griddepcontrol.wait;" ::: "memory");   // the table, or R

  const uint32_t ring = smem_addr(smem), sq = ring + ST_Q, sr = ring + ST_R;
  float *sc = reinterpret_cast<float *>(smem + ST_C);  // [stage][coef, bias scale, lse, position, row][QR]
  const float kg = p.k == nullptr && p.kv.k_global ? __ldg(p.kv.k_global + u.h) : 1.f;
  const int ks = p.a.E > 0 && !POS ? (p.a.rd + 15) / 16 : 0;   // 16-channel steps of the bias product
  const bool r_vec = (p.a.rd & 7) == 0 && (reinterpret_cast<uintptr_t>(p.a.r) & 15u) == 0;
  const long rbeg = (long)tok0 * p.a.group, rend = (long)tok1 * p.a.group;
  const int m0 = rel_table_origin(p.a.E);
  int table_lo = 0x7fffffff;                 // table rows from here on have been copied
  auto stage = [&](long r0, int buf) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = (tid >> 4) + 8 * i, c = tid & 15;
      const long rr = r0 + n;
      const bool live = rr < rend;
      const int tok = (int)((live ? rr : rbeg) / p.a.group), hh = (int)((live ? rr : rbeg) - (long)tok * p.a.group);
      const __nv_bfloat16 *src = p.a.q + ((long)(u.s.q0 + tok) * p.a.Hq + u.h * p.a.group + hh) * kHeadDim + c * 8;
      cp_async16(sq + buf * QR * 256 + n * 256 + ((c ^ (n & 7)) << 4), src, live);
    }
    const int last = (int)((min(r0 + QR, rend) - 1) / p.a.group), first = (int)(r0 / p.a.group);
    if (ks > 0 && u.qbase + first - (tile0 + kWalkTile - 1) < p.a.E) {
      // r rows (zero past r_dim), and the table rows that these tokens add
      for (int i = tid; i < QR * 2 * ks; i += WT) {
        const int n = i / (2 * ks), c = i - n * 2 * ks;
        const long rr = r0 + n;
        const bool live = rr < rend;
        const int tok = (int)((live ? rr : rbeg) / p.a.group), hh = (int)((live ? rr : rbeg) - (long)tok * p.a.group);
        const __nv_bfloat16 *src = p.a.r + ((long)(u.s.q0 + tok) * p.a.Hq + u.h * p.a.group + hh) * p.a.rd;
        const uint32_t dst = sr + buf * QR * 128 + n * 128 + ((c ^ (n & 7)) << 4);
        if (r_vec) {
          cp_async16(dst, src + (c * 8 < p.a.rd ? c * 8 : 0), live && c * 8 < p.a.rd);
        } else {
          uint32_t w[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int e = c * 8 + 2 * j;
            const uint32_t lo = live && e < p.a.rd ? __bfloat16_as_ushort(src[e]) : 0;
            const uint32_t hi = live && e + 1 < p.a.rd ? __bfloat16_as_ushort(src[e + 1]) : 0;
            w[j] = lo | (hi << 16);
          }
          st_shared_v4(dst, w[0], w[1], w[2], w[3]);
        }
      }
      const int lo = m0 - (u.qbase + last) + tile0;
      const int hi = min(table_lo, m0 - (u.qbase + first) + tile0 + kWalkTile);
      for (int i = tid; i < (hi - lo) * 8; i += WT) {
        const int m = lo + (i >> 3), c = i & 7, slot = m & (TR - 1);
        const bool in = m >= 0 && m < rel_table_rows(p.a.E);
        cp_async16(ring + slot * 128 + ((c ^ (slot & 7)) << 4), p.table + (in ? (long)m * 64 + c * 8 : 0), in);
      }
      table_lo = lo;
    }
    if (tid < QR) {
      const long rr = r0 + tid;
      const bool live = rr < rend;
      const int tok = (int)((live ? rr : rbeg) / p.a.group), hh = (int)((live ? rr : rbeg) - (long)tok * p.a.group);
      const int head = u.h * p.a.group + hh;
      float *o = sc + buf * 5 * QR + tid;
      const float s = live ? log_scale(u.qbase + tok, p.a.inv_ln_base) : 0.f;
      const float z = live ? __ldg(p.lse + (long)head * p.a.total_q + u.s.q0 + tok) : -INFINITY;
      o[0] = p.a.alpha_log2e * s * kg;
      o[QR] = s * kLog2e;
      o[2 * QR] = z == -INFINITY ? INFINITY : z * kLog2e;
      o[3 * QR] = __int_as_float(live ? u.qbase + tok : -1);
      o[4 * QR] = __int_as_float(tok * p.a.group + hh);
    }
    cp_async_commit();
  };

  float v[4] = {0.f, 0.f, 0.f, 0.f};
  int buf = 0;
  if (rbeg < rend) stage(rbeg, 0);
  for (long r0 = rbeg; r0 < rend; r0 += QR, buf ^= 1) {
    cp_async_wait<0>();
    __syncthreads();                         // this stage has landed, the other one is read
    if (r0 + QR < rend) stage(r0 + QR, buf ^ 1);
    const float *c_coef = sc + buf * 5 * QR;
    const int qmin = __float_as_int(c_coef[3 * QR]);
    const int qlast = u.qbase + (int)((min(r0 + QR, rend) - 1) / p.a.group);
    const bool edge = POS || key0 + WK - 1 > qmin || (unsigned)(qlast - key0) >= wlim || r0 + QR > rend;
    const bool band = p.a.E > 0 && (POS ? __any_sync(full, kp_lane != 0x7fffffff && qmin - kp_lane < p.a.E)
                                        : qmin - (key0 + WK - 1) < p.a.E);
#pragma unroll 1
    for (int nt = 0; nt < QR / 8; ++nt) {
      uint32_t b[16];
      const int brow = nt * 8 + (lane & 7);
#pragma unroll
      for (int s = 0; s < 4; ++s)
        ldsm_x4(sq + buf * QR * 256 + brow * 256 + (((4 * s + (lane >> 3)) ^ (brow & 7)) << 4), b[4 * s], b[4 * s + 1],
                b[4 * s + 2], b[4 * s + 3]);
      float x[2][4], y[2][4];
#pragma unroll
      for (int gr = 0; gr < 2; ++gr) {
        x[gr][0] = x[gr][1] = x[gr][2] = x[gr][3] = 0.f;
        y[gr][0] = y[gr][1] = y[gr][2] = y[gr][3] = 0.f;
#pragma unroll
        for (int s = 0; s < 8; ++s)
          mma_bf16_16816(x[gr], f[gr][s][0], f[gr][s][1], f[gr][s][2], f[gr][s][3], b[2 * s], b[2 * s + 1]);
      }
      if (band && !POS) {
        // y = P^T r^T, one token's rows at a time: key j is table row m0 - i + j
        uint32_t rbf[8];
#pragma unroll
        for (int s = 0; s < 2; ++s)
          ldsm_x4(sr + buf * QR * 128 + brow * 128 + (((4 * s + (lane >> 3)) ^ (brow & 7)) << 4), rbf[4 * s],
                  rbf[4 * s + 1], rbf[4 * s + 2], rbf[4 * s + 3]);
        const int my_pos = __float_as_int(c_coef[3 * QR + nt * 8 + g]);       // of the row this lane holds
        const int lo_pos = __float_as_int(c_coef[3 * QR + nt * 8]);
        const int hi_pos = min(qlast, __shfl_sync(full, my_pos, 28) < 0 ? qlast : __shfl_sync(full, my_pos, 28));
        for (int pos = lo_pos; pos >= 0 && pos <= hi_pos; ++pos) {
          const bool mine = my_pos == pos;
#pragma unroll
          for (int gr = 0; gr < 2; ++gr) {
            const int m = m0 - pos + key0 + gr * 16 + (lane & 7) + (((lane >> 3) & 1) << 3);
            const uint32_t slot = (uint32_t)m & (TR - 1);
#pragma unroll
            for (int s = 0; s < 4; ++s)
              if (s < ks) {
                uint32_t a0, a1, a2, a3;
                ldsm_x4(ring + slot * 128 + (((2 * s + (lane >> 4)) ^ (slot & 7)) << 4), a0, a1, a2, a3);
                mma_bf16_16816(y[gr], a0, a1, a2, a3, mine ? rbf[2 * s] : 0u, mine ? rbf[2 * s + 1] : 0u);
              }
          }
        }
      }
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        const int m = nt * 8 + 2 * t + c;
        const float coef = c_coef[m], bs = c_coef[QR + m], lse2 = c_coef[2 * QR + m];
        const int qp = __float_as_int(c_coef[3 * QR + m]);
#pragma unroll
        for (int gr = 0; gr < 2; ++gr)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            float l = fmaf(x[gr][2 * hf + c], coef, -lse2);
            const unsigned d = (unsigned)qp - (unsigned)kp[gr][hf];
            if (POS) {
              if (band && d < (unsigned)p.a.E) {
                const int rr = __float_as_int(c_coef[4 * QR + m]), tok = rr / p.a.group;
                const long grow = (long)(u.s.q0 + tok) * p.a.Hq + u.h * p.a.group + (rr - tok * p.a.group);
                l = fmaf(p.a.rdec[grow * p.a.E + d], bs, l);
              }
            } else if (band) {
              l = fmaf(y[gr][2 * hf + c], bs, l);
            }
            if ((edge && d >= wlim) || lse2 == INFINITY) l = -INFINITY;   // (0 times a NaN key is not 0)
            v[2 * gr + hf] += fast_exp2(l);
          }
      }
    }
  }
  const float sum = quad_reduce(v, t);
  const int key = key0 + (t >> 1) * 16 + (t & 1) * 8 + g;
  if (row0 >= 0 && key < u.s.lk) write_weight(p, u, key, row0 + (key - key0), sum);
}

// The bias table: row m holds P[:, d] for d = origin - m, zero outside [0, E)
// and past r_dim.
__global__ void __launch_bounds__(256) relattn_rel_table_kernel(const __nv_bfloat16 *__restrict__ P, int rd, int E,
                                                                __nv_bfloat16 *__restrict__ table) {
  asm volatile("griddepcontrol.launch_dependents;");
  __shared__ __nv_bfloat16 tile[64][33];
  const int m0 = blockIdx.x * 32, rows = rel_table_rows(E), org = rel_table_origin(E);
  for (int i = threadIdx.x; i < 64 * 32; i += 256) {
    const int c = i >> 5, m = m0 + (i & 31), d = org - m;
    tile[c][i & 31] = c < rd && d >= 0 && d < E ? P[(size_t)c * E + d] : __float2bfloat16_rn(0.f);
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 64 * 32; i += 256) {
    const int m = m0 + (i >> 6), c = i & 63;
    if (m < rows) table[(long)m * 64 + c] = tile[c][i >> 6];
  }
}

// ------------------------------------------------------------------ keys out of sight

// Keys that the walk leaves out (past the window of every row): w_out = decay *
// w_in.
__global__ void __launch_bounds__(256) relattn_key_weights_cold_kernel(const __grid_constant__ KeyWeightArgs p) {
  Unit u;
  u.b = blockIdx.y / p.a.Hkv;
  u.h = blockIdx.y - u.b * p.a.Hkv;
  const int tiles = unit_tiles(p, u.b, &u.s, &u.lo);
  if (tiles < 0) return;
  const int end = u.lo;
  for (int key = blockIdx.x * kColdKeys + threadIdx.x; key < min(end, (int)(blockIdx.x + 1) * kColdKeys); key += 256) {
    const long row = p.pages.row(u.b, u.s.k0, key);
    if (row < 0) {
      atomicOr(p.a.err, kDevErrSeqlens);
      continue;
    }
    write_weight(p, u, key, row, 0.f);
  }
}

template <int NT, bool POS, bool FP4>
cudaError_t launch_rows(const KeyWeightArgs &p, cudaLaunchConfig_t cfg) {
  static std::atomic<bool> done[kMaxDevicesAttr];
  auto *kernel = relattn_key_weights_rows_kernel<NT, POS, FP4>;
  const cudaError_t e = set_max_smem_once(reinterpret_cast<const void *>(kernel), KStage<FP4>::ring, done);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3((unsigned)(p.a.sms * rows_ctas(NT, FP4)));
  cfg.blockDim = dim3(WT);
  cfg.dynamicSmemBytes = KStage<FP4>::ring;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <bool POS, bool FP4>
cudaError_t launch_few(const KeyWeightArgs &p, cudaLaunchConfig_t cfg) {
  return p.a.max_q * p.a.group <= 8 ? launch_rows<1, POS, FP4>(p, cfg) : launch_rows<2, POS, FP4>(p, cfg);
}

template <bool POS>
cudaError_t launch_tiles(const KeyWeightArgs &p, cudaLaunchConfig_t cfg) {
  static std::atomic<bool> done[kMaxDevicesAttr];
  auto *kernel = relattn_key_weights_tiles_kernel<POS>;
  const cudaError_t e = set_max_smem_once(reinterpret_cast<const void *>(kernel), ST_BYTES, done);
  if (e != cudaSuccess) return e;
  cfg.gridDim = dim3((unsigned)((p.a.max_k + kWalkTile - 1) / kWalkTile), (unsigned)(p.a.batch * p.a.Hkv));
  cfg.blockDim = dim3(WT);
  cfg.dynamicSmemBytes = ST_BYTES;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

// A call is walked (few rows) or takes tiles of keys; with positions, and when
// walked, the bias comes from R in the workspace, else from the bias table.
constexpr int kBandExtra = 1;                // a walked tile with a bias counts twice (64 sequences, 1 to 32 thousand
                                            // keys: 69 us; 75 counted once, 72 three times)
bool key_weights_walked(const KernelArgs &a) { return (long)a.max_q * a.group <= kFp4Rows && a.batch <= kWalkBatch; }

size_t key_weights_workspace(const KernelArgs &a, bool positions) {
  if (a.E <= 0) return 0;
  if (positions || key_weights_walked(a)) return (size_t)a.total_q * a.Hq * a.E * sizeof(float);
  return (size_t)rel_table_rows(a.E) * 64 * sizeof(__nv_bfloat16);
}

cudaError_t launch_key_weights(const KeyWeightArgs &args, cudaStream_t stream) {
  KeyWeightArgs p = args;
  const bool pos = p.key_pos != nullptr, fp4 = p.k == nullptr, walked = key_weights_walked(p.a);
  p.table = nullptr;
  p.hp = walked && p.a.Hkv % 2 == 0 ? 2 : 1;   // two heads share their rows' lines
  p.idle = 1;                                 // their keys' weights decay
  p.band_extra = walked && p.a.E > 0 ? kBandExtra : 0;
  if (p.a.E > 0) {
    cudaError_t e;
    if (pos || walked) {
      e = launch_rel_bias(p.a.r, p.a.P, (long)p.a.total_q * p.a.Hq, p.a.rd, p.a.E, const_cast<float *>(p.a.rdec), stream);
    } else {
      p.table = reinterpret_cast<const __nv_bfloat16 *>(p.a.rdec);
      relattn_rel_table_kernel<<<(rel_table_rows(p.a.E) + 31) / 32, 256, 0, stream>>>(
          p.a.P, p.a.rd, p.a.E, const_cast<__nv_bfloat16 *>(p.table));
      e = cudaGetLastError();
    }
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = p.a.E > 0 ? 1 : 0;          // behind the R or table kernel
  if (walked) {
    const cudaError_t e = pos ? (fp4 ? launch_few<true, true>(p, cfg) : launch_few<true, false>(p, cfg))
                              : (fp4 ? launch_few<false, true>(p, cfg) : launch_few<false, false>(p, cfg));
    // the walk leaves the keys past every row's window alone
    if (e != cudaSuccess || p.a.window <= 0 || pos || p.a.max_k <= p.a.window) return e;
    relattn_key_weights_cold_kernel<<<dim3((unsigned)((p.a.max_k + kColdKeys - 1) / kColdKeys),
                                           (unsigned)(p.a.batch * p.a.Hkv)), 256, 0, stream>>>(p);
    return cudaGetLastError();
  }
  p.tc = pos ? 0 : key_weights_tc_kind(p);
  cudaError_t e = cudaSuccess;
  if (p.tc != 2) e = pos ? launch_tiles<true>(p, cfg) : launch_tiles<false>(p, cfg);
  if (e != cudaSuccess || !p.tc) return e;
  return launch_key_weights_tc(p, stream);
}

}  // namespace relattn

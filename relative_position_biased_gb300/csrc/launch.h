// launch.h -- internal launchers called by the C ABI layer (api.cu).
#pragma once

#include <cudaTypedefs.h>

#include <atomic>
#include <mutex>

#include "common.cuh"

namespace relattn {

// The calling thread's current CUDA context (a CUcontext, as an opaque key),
// or null before the runtime has made one current.  Per-device addresses the
// library caches (device symbols) are keyed on it: after cudaDeviceReset the
// primary context is new, the module is loaded again and the symbols may
// move, so a cached address is looked up again when the context changes.
inline void *current_cu_context() {
  static const PFN_cuCtxGetCurrent_v4000 get = []() -> PFN_cuCtxGetCurrent_v4000 {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuCtxGetCurrent", &p, 4000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      return reinterpret_cast<PFN_cuCtxGetCurrent_v4000>(p);
    return nullptr;
  }();
  CUcontext c = nullptr;
  if (get && get(&c) != CUDA_SUCCESS) c = nullptr;
  return reinterpret_cast<void *>(c);
}

// Raise `func`'s dynamic shared-memory limit to `bytes` once per device.
// `done` holds one flag per device for that kernel; the first launch on a
// device sets the attribute under a process-wide lock, so host threads that
// launch concurrently neither race on the flag nor skip the call.
constexpr int kMaxDevicesAttr = 64;
inline cudaError_t set_max_smem_once(const void *func, int bytes,
                                     std::atomic<bool> (&done)[kMaxDevicesAttr]) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevicesAttr)
    return cudaErrorInvalidDevice;
  if (done[dev].load(std::memory_order_acquire)) return cudaSuccess;
  static std::mutex mu;
  std::lock_guard<std::mutex> lock(mu);
  if (done[dev].load(std::memory_order_relaxed)) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done[dev].store(true, std::memory_order_release);
  return e;
}

// Query rows per decode CTA for a given row count (max_seqlen_q * group).
int decode_warps_for_rows(int rows);

// Per-split key-chunk granularity (keys per tile) of the decode kernels.
constexpr int kDecodeKeyTile = 64;

size_t prefill_mma_smem_bytes(int rd_pad);
size_t decode_mma_smem_bytes(int warps, int rd_pad);

cudaError_t launch_prefill_mma(const KernelArgs &a, cudaStream_t stream);

// tcgen05 / TMA kernels: need 16-byte aligned q/k/v/out (and r/P), r_dim % 8 == 0,
// rel_extent % 8 == 0, r_dim <= 64 and at least one 128-key tile of K/V.
// Their key tiles (and decode split chunks) are kTcKeyTile keys.
constexpr int kTcKeyTile = 128;
bool tc_supported(const KernelArgs &a, int total_k);
cudaError_t launch_prefill_tc(const KernelArgs &a, int total_k, cudaStream_t stream);
// Prefill past the bias band (fwd_tc_main.cu): two query heads of one GQA
// group per CTA; needs an even group size, alpha > 0 and at least 128 query
// rows and keys.  With init_from_out it continues from the band kernel's
// out / lse (launched first with band_only).
bool tc_main_supported(const KernelArgs &a, int total_q, int total_k);
cudaError_t launch_prefill_tc_main(const KernelArgs &a, int total_k, cudaStream_t stream);
// decode on the same kernel: 128 rows of (token, head-in-group) per CTA; grid
// (num_splits, Hkv * row_blocks, batch); partials when num_splits > 1.
constexpr int kTcDecodeRows = 128;
cudaError_t launch_decode_tc(const KernelArgs &a, int total_k, cudaStream_t stream);
// decode of few rows (decode_tc.cu): keys along the MMA's M; an item is
// (split, sequence, kv head) and holds every row of the sequence's tokens for
// that kv head (max_q x group <= 16).  Needs 16-byte aligned q / k / v / out
// and at least 128 K / V rows.  With a bias it first computes R = r . P of the
// decode rows into a.rdec (decode_rel_bytes of workspace).  Partials when
// num_splits > 1.
constexpr int kFewRows = 16;
bool decode_few_rows_supported(const KernelArgs &a, int kv_rows);
size_t decode_rel_bytes(const KernelArgs &a);
cudaError_t launch_decode_few_rows(const KernelArgs &a, int kv_rows, cudaStream_t stream);
// The same decode on an MXFP8 K / V cache (decode_tc.cu): E4M3 codes k8 / v8
// [kv_rows, Hkv, 128] (16-byte aligned) with E8M0 scales ks / vs [kv_rows,
// Hkv, 4] (4-byte aligned); q quantised per item in the kernel, Q K^T as an
// E4M3 product per 32-dim block, V dequantised to bf16 for P V.  Contiguous
// K / V only.
bool decode_mxfp8_supported(const KernelArgs &a, const void *k8, const void *v8, const void *ks,
                            const void *vs, int kv_rows);
cudaError_t launch_decode_mxfp8(const KernelArgs &a, const void *k8, const void *v8, const void *ks,
                                const void *vs, int kv_rows, cudaStream_t stream);
// MXFP8 quantisation (mxfp8.cu): n_blocks blocks of 32 bf16 (x 16-byte
// aligned) -> 32 E4M3 codes (16-byte aligned) and one E8M0 scale byte each.
cudaError_t launch_quantize_mxfp8(const void *x, long n_blocks, void *codes, void *scales,
                                  cudaStream_t stream);
cudaError_t launch_decode_mma(const KernelArgs &a, int warps, cudaStream_t stream);
// pdl: launched as a programmatic dependent of the kernel before it on the
// stream (which lets it launch early; the combine waits for its results)
cudaError_t launch_combine(const float *o_part, const float *lse_part, int num_splits,
                           int total_q, int num_heads, __nv_bfloat16 *out, float *lse,
                           cudaStream_t stream, bool pdl = false);

// Backward pass (bwd_mma.cu): gradients of sum(dout * out) w.r.t. q, k, v, r.
struct BwdArgs {
  const __nv_bfloat16 *q, *k, *v, *r, *P, *out, *dout;
  const float *lse;            // [Hq, Tq] natural log (the forward's)
  const int32_t *cu_q, *cu_k;
  __nv_bfloat16 *dq, *dk, *dv, *dr;   // dr may be null (no bias)
  float *Dsum;                 // workspace [Hq, Tq]: dout . out
  float *Rall;                 // workspace [Tq, Hq, e_pad]: R = r . P for distances < E (bias only)
  int e_pad;                   // row stride of Rall: E rounded up to a multiple of 4
  int rall_ok;                 // 1: Rall has been written (the band's dq loads its R windows from it)
  float *dkv_part;             // workspace [2 halves][dk, dv][Tk, Hkv, 128] fp32 (GQA groups of 4, 6, 8 ...)
  int kv_split;                // 2: two tcgen05 dk / dv CTAs per key tile, each half the group's heads
  int test_skip_dkdv_step;     // test hooks: a step whose copies the tcgen05 dk / dv producer
  int test_skip_dq_step;       //   (or the tcgen05 dq producer) never issues (-1: off)
  float *dq_part;              // workspace [Tq, Hq, 128]: dq over the keys outside the bias band (fp32)
  int dq_split;                // 1: the tcgen05 dq takes the keys outside the band and writes
                               //    dq_part; the warp-MMA dq takes the band and adds dq_part
  int *err;
  int batch, total_q, total_k, max_q, max_k, Hq, Hkv, group;
  int rd, rd_pad, E, window;
  float alpha, alpha_log2e, inv_ln_base;
  int p_vec_ok;                // 16-byte vector loads of P allowed (E % 8 == 0)
  int q_tiles, k_tiles;        // 64-row / 64-key tiles per sequence (max)
};
size_t bwd_dq_smem_bytes(int rd_pad);
size_t bwd_dkdv_smem_bytes(int rd_pad);
cudaError_t launch_backward(const BwdArgs &a, int sms, cudaStream_t stream);
// dk / dv on tcgen05 (bwd_tc.cu): 16-byte aligned q / k / v / dout, r_dim <= 64,
// at least 128 keys and 64 query rows in total (the TMA boxes)
bool bwd_tc_supported(const BwdArgs &a);
cudaError_t launch_bwd_dkdv_tc(const BwdArgs &a, cudaStream_t stream);
// dq on tcgen05 (bwd_tc.cu) over the keys every row of a 128-row tile sees
// outside the bias band (all keys without a bias); also needs 128 query rows
bool bwd_dq_tc_supported(const BwdArgs &a);
cudaError_t launch_bwd_dq_tc(const BwdArgs &a, cudaStream_t stream);

// attention prologue (prologue.cu): ShortConv + Q/K RMSNorm + KV-cache rows;
// err = the device error word, sms = the SM count (sizes the grid),
// skip_tile = test hook (a token tile whose copies are never issued; -1 = off).
// mx: an MXFP8 cache to write as well (or instead, with null bf16 caches).
cudaError_t launch_prologue(const relattn_prologue_params *p, int *err, int sms, int skip_tile,
                            cudaStream_t stream, const relattn_kv_mxfp8_out *mx = nullptr);

// The 4-bit (NVFP4) K / V cache (nvfp4.cuh): codes [rows, Hkv, 64] (16-byte
// aligned), scales [rows, Hkv, 8] (8-byte aligned), factors [Hkv] or null (1).
struct Fp4Cache {
  const uint8_t *k, *v, *k_scale, *v_scale;
  const float *k_global, *v_global;
};

// Physical cache rows: contiguous rows cu_seqlens_k[b] + p, or (with a block
// table) row block_table[b * max_pages + p / page_size] * page_size + p % page_size.
struct CachePages {
  const int32_t *block_table;
  int page_size, max_pages, num_pages;
  long rows;   // rows of the cache arrays

  // row of key p of sequence b (k0 = cu_seqlens_k[b]), -1 when it lies outside the arrays
  __device__ __forceinline__ long row(int b, int k0, int p) const {
    if (block_table) {
      const int slot = p / page_size;
      if (slot >= max_pages) return -1;
      const int pg = __ldg(block_table + (long)b * max_pages + slot);
      return (unsigned)pg < (unsigned)num_pages ? (long)pg * page_size + (p - slot * page_size) : -1;
    }
    const long r = (long)k0 + p;
    return r < rows ? r : -1;
  }
};

// Chunk rows into / out of the 4-bit cache (cache_fp4.cu): k / v bf16
// [total_q, Hkv, 128], read by the store and written by the load.
struct Fp4RowArgs {
  const __nv_bfloat16 *k, *v;
  const int32_t *cu_q, *cu_k;
  int *err;
  int batch, total_q, Hkv;
  Fp4Cache kv;
  CachePages pages;
};
cudaError_t launch_store_fp4(const Fp4RowArgs &a, cudaStream_t stream);
cudaError_t launch_load_fp4(const Fp4RowArgs &a, cudaStream_t stream);

// R = r . P of every query row and distance < E (rel_bias.cu): fp32 [rows][E],
// any r_dim <= 64 and E.  A kernel launched behind it as its programmatic
// dependent may start early and waits for it with griddepcontrol.wait.
cudaError_t launch_rel_bias(const __nv_bfloat16 *r, const __nv_bfloat16 *P, long rows, int r_dim, int E,
                            float *R, cudaStream_t stream);

// Kernels that stream a cache: q, r, P, lengths, rdec and err in `a`; key_pos
// [Hkv, pages.rows] / q_pos [batch] are positions, or both null (row indices).
struct WalkArgs {
  KernelArgs a;
  CachePages pages;
  const int32_t *key_pos, *q_pos;
  int hp;                             // kv heads a walking CTA takes (1 or 2)
  int idle;                           // 1: sequences without query rows are walked too
  int band_extra;                     // a tile that meets the bias band counts as this many more
};
constexpr int kWalkTile = 128;        // keys a CTA takes at a time, over its kv heads

// Split-KV decode over the 4-bit cache (decode_fp4.cu, decode_fp4_tc.cu).
struct Fp4DecodeArgs : WalkArgs {
  Fp4Cache kv;
  int row_blocks;      // row blocks per (sequence, kv head)
  int splits;          // partial slots of a row; 1 = no partials
  int whole;           // 1: one CTA per unit
  int waves;           // else: most ranges a CTA takes
  int c_min;           // and least tiles of a range (keeps a unit within its slots)
  int tc;              // 1: the tcgen05 kernel (decode_fp4_tc.cu)
};
// Most tiles summed in one piece.  The matrix instructions add to an fp32
// accumulator by truncation: each takes about 1e-7 off it (measured, values of one
// sign: 72 rows of 2^27 keys, 880 thousand in a piece, lost 0.5 % of the result,
// 4 million in one piece 2.5 %).  4096 additions, 8 a tile on tcgen05 and 2 a tile in
// a warp of the other kernel, keep that below 2^-11.
constexpr int kFp4MostTiles = 2048, kFp4TcMostTiles = 512;
struct Fp4DecodePlan {
  int hp, row_blocks, splits, whole, waves, c_min, tc, band_extra;
  size_t lse_offset, rel_offset, ws_bytes;
};
constexpr int kFp4Rows = 16;          // query rows of a work unit
constexpr int kFp4TcRows = 128;       // and of one of the tcgen05 kernel
constexpr int kFp4PageUnit = 32;      // page sizes are multiples of it
bool plan_decode_fp4(const KernelArgs &a, long total_k, bool positions, int want_splits, Fp4DecodePlan *plan);
cudaError_t launch_decode_fp4(const Fp4DecodeArgs &a, cudaStream_t stream);
cudaError_t launch_decode_fp4_tc(const Fp4DecodeArgs &a, cudaStream_t stream);

// Attention weight per key (key_weights.cu): w_out[h][row] = decay w_in[h][row]
// (0 for the newest Lq keys) + sum over query rows and the group's heads of
// exp(x - lse).  K is bf16 (k) or 4-bit (kv.k, when k is null).
struct KeyWeightArgs : WalkArgs {
  const __nv_bfloat16 *k;
  Fp4Cache kv;
  const float *lse;    // [Hq, total_q]
  const float *w_in;   // [Hkv, pages.rows], null: zero
  float *w_out;
  float decay;
  const __nv_bfloat16 *table;   // bias table in the workspace (set by the launcher)
  int tc;                       // tcgen05 kernel (key_weights_tc.cu): 0 no, 1 the rows past the bias band, 2 all rows
};
bool key_weights_walked(const KernelArgs &a);
size_t key_weights_workspace(const KernelArgs &a, bool positions);
cudaError_t launch_key_weights(const KeyWeightArgs &a, cudaStream_t stream);
// Many rows on tcgen05 (key_weights_tc.cu), by p.tc: the value it supports for
// these arguments, and the launch (with 1 it adds to the tiles kernel's sums).
int key_weights_tc_kind(const KeyWeightArgs &a);
cudaError_t launch_key_weights_tc(const KeyWeightArgs &a, cudaStream_t stream);

// Eviction (evict.cu)
constexpr int kMaxPlanes = 8;
struct EvictArgs {
  const float *weights;          // [Hkv, src.rows]
  const int32_t *cu_k, *cu_keep, *key_pos;
  CachePages src, dst;
  int batch, total_keep, max_k, Hkv, sink, recent;
  float *w_out;                  // [Hkv, dst.rows] or null
  int32_t *pos_out;              // [Hkv, dst.rows] or null
  int clear;                     // both are cleared first
  int32_t *src_row;              // workspace [Hkv, total_keep]: cache row of every kept key
  int32_t *dst_row;              // workspace [total_keep]: its row in the new cache
  int planes;
  const void *from[kMaxPlanes];  // [src.rows, Hkv, bytes]
  void *to[kMaxPlanes];          // [dst.rows, Hkv, bytes]
  int bytes[kMaxPlanes];
  unsigned *wide;                // workspace of a wide selection (evict_wide_bytes), zeroed by the launcher
  int ctas;                      // CTAs per (sequence, kv head) in a wide selection (set by the launcher)
  int sms;
  int test_skip_cta;             // test hook: CTA of a wide selection that never arrives (-1: none)
  int *err;
};
size_t evict_wide_bytes(int batch, int Hkv, int max_k);       // 0: one cluster per (sequence, kv head)
cudaError_t clear_evicted(const EvictArgs &a, cudaStream_t stream);     // w_out to 0, pos_out to -1
cudaError_t launch_evict(const EvictArgs &a, cudaStream_t stream);

}  // namespace relattn

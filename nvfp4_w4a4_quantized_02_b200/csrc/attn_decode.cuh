// Attention over the block-scaled 8-bit cache for sequences with few new tokens.
//
// For a query row q (one head of one token) and the cached tokens j it sees,
//     x_j = scale log2(e) sK_j (q . k_j),   o = sum_j 2^{x_j} sV_j v_j / sum_j 2^{x_j},
// where k_j, v_j are E4M3 codes and sK_j, sV_j the scales of j's block.  One pass with a
// running maximum; the maximum is taken over x_j + log2 sV_j, so that the weights the
// matrix instruction sees,
//     P_j = 2^{x_j + log2 sV_j - M + kBoost},
// already hold the value scale, while the denominator adds P_j / sV_j.  M need not be the maximum
// itself: it follows when a P would exceed 2^(kBoost + kSlack), FP16's range being 2^16.  P is rounded
// to FP16, the operand type that E4M3 values are exact in: with 11 bits down to 2^-26 of 2^kBoost,
// FP16's smallest normal number, and below that to within half its smallest step, 2^-37 of 2^kBoost.
//
// Bound by HBM: a unit is eight query rows of a kv head (heads of a group, times tokens) and reads
// every cached byte of its sequence once, for 2 x 8 multiply-adds; 9 to 32 rows are two to four
// units and read the cache as often.  Each warp keeps its own ring of STAGES steps of K and V rows in shared
// memory, filled by TMA, so that about 190 KB (at 64 values per head half of that) are on their way to an SM
// whatever its warps do (loads straight into registers reached 3.3 TB/s on 32 sequences of up to
// 8192 tokens), and feeds mma.m16n8k16 from it:
//  * S^T = K Q^T has the cached tokens as its 16 rows and up to 8 query rows (the heads of
//    a group, times tokens) as its 8 columns.  The contraction runs over the head's
//    values in any order as long as K and Q agree, so a lane takes 16 consecutive bytes
//    of a token's row as its values of four k-steps.
//  * O^T = V^T P^T has 16 values as its rows and 16 tokens as its contraction: a lane
//    reads the same 16 values of four tokens and byte permutes pair the tokens.  The
//    accumulators' columns are query rows again, so rescaling is lane-local, and
//    movmatrix turns S^T's accumulators into the P^T operand.
// The 16 tokens of a tile may stand in any order in both products; with the 128-byte swizzle of
// the TMA and the order of token_of() every shared-memory read is free of bank conflicts.
// E4M3 is exact in FP16; q is scaled by a power of two per row to lie in FP16's range
// and keeps all of its BF16 bits within 2^-29 of the row's largest value.  Sums, maxima
// and accumulators are FP32.
//
// The cached tiles of all (sequence, kv head, 8-row group) units form one list that is
// cut evenly over the CTAs; a unit that several CTAs share leaves partial results
// (O, M, l) in the workspace and combine_kernel joins them in a fixed order.  Where the block table
// has room for kWholeTiles tiles at most, units stay whole: the second kernel would cost more (at six
// tiles, 700 tokens, whole units took 14.9 us and cut ones 11.2 us).
//
// Measured, 8-bit cache: 32 sequences of up to 8192 tokens, 8 kv heads of 128 values, groups of 6:
// 76 us, 4.5 TB/s; 2 of up to 131072, 4 kv heads of 256: 69 us, 4.4 TB/s; one of 700: 11 us, the latency of
// two launches and a short stream.
#pragma once

#include <cuda_fp16.h>

#include <type_traits>

#include "batch.cuh"
#include "ptx.cuh"

namespace nvfp4 {
namespace attn {

constexpr int kRows = 8;        // query rows of a unit
constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr float kBoost = 12.0f;
constexpr float kSlack = 3.0f;
constexpr int kWholeTiles = 3;
constexpr float kMinLogScale = -100.0f;  // log2 of the smallest value scale taken at its word
constexpr int kGroup = 16;      // tokens of one mma tile; a cache block holds a multiple of it

struct Args {
  const uint16_t *q;  // BF16 [tokens x ld_q], head h at column h * D
  int64_t ld_q;
  const int32_t *cu_seqlens;  // [n_seqs + 1]
  const int32_t *kv_lens;     // [n_seqs] tokens in the cache, the new ones included
  int64_t tokens;
  int n_seqs;
  int kv_heads, group;        // query head h reads kv head h / group
  const int32_t *table;       // [n_seqs x ld_table] cache block of tokens [b * block, (b + 1) * block)
  int64_t ld_table;
  int64_t max_kv;             // table columns * block size
  const uint8_t *k, *v;       // [num_blocks][kv_heads][block][D] E4M3
  const float *k_scales, *v_scales;  // [num_blocks][kv_heads]
  int64_t num_blocks;
  int log_block;
  float scale_log2;           // softmax scale * log2(e)
  int causal;
  void *out;
  int64_t ld_out;
  int out_fp32;
  // workspace
  int4 *desc;                 // per unit: sequence, kv head, row group, -; first and last CTA in desc2
  int2 *desc2;
  int *n_units;
  float *part;                // [2 * gridDim.x][kRows][D]
  float2 *part_ml;            // [2 * gridDim.x][kRows] (M, l)
  int whole;                  // units are not cut: no partial results, no combine kernel
  int splits;                 // prompt kernel: CTAs per item at most (prompt_part, prompt_ml: 1 + splits > 1)
  float *prompt_part;         // [items * splits][rows of an item][D]
  float2 *prompt_ml;          // [items * splits][rows of an item] (reference, l)
  int max_decode_rows;        // sequences with more query rows per kv head belong to the prompt kernel
};

// log2 of the tokens of a warp's step.
__host__ __device__ constexpr int step_log(int d) { return d == 256 ? 4 : 5; }

template <int D>
struct Cfg {
  static constexpr int TS = 1 << step_log(D);
  static constexpr int NG = TS / kGroup;
  static constexpr int STAGES = D == 256 ? 3 : 2;  // steps of a warp's ring
  static constexpr int CTAS = D == 256 ? 2 : 3;    // per SM
  static constexpr int TILE = TS * kWarps;       // tokens of a CTA's step
  static constexpr int SEGK = D / 64;            // 64-value segments of a K row
  static constexpr int VW = D >= 128 ? 4 : 2;    // 32-bit words of V per lane and token, per segment
  static constexpr int SEGV = D >= 128 ? D / 128 : 1;
  static constexpr int MB = D / 16;              // 16-value row blocks of O^T
  static constexpr int LD = D + 4;
  static constexpr int ROWB = D < 128 ? D : 128;  // bytes of a row of a panel
  static constexpr int PANELS = D / ROWB;
  static constexpr int PART = TS * D;            // bytes of a step's K (or V)
  static constexpr int RING = kWarps * STAGES * 2 * PART;
};

// Rows of a TMA box of codes: a power of two of tokens of one cache block, up to a step.
__host__ __device__ constexpr int box_log(int log_block, int d) { return log_block < step_log(d) ? log_block : step_log(d); }

// Token of row `slot` of a 16-token tile: 0 5 2 7 4 1 6 3, then the same plus 8.
__device__ __forceinline__ int token_of(int slot) { return slot & 1 ? (((slot & 6) ^ 4) + 1) | (slot & 8) : slot; }

// Byte offset of 16-byte piece c of row r in a panel, as the TMA's swizzle puts it.
template <int D>
__device__ __forceinline__ uint32_t swizzled(int r, int c) {
  return D < 128 ? r * 64 + ((c ^ ((r >> 1) & 3)) << 4) : r * 128 + ((c ^ (r & 7)) << 4);
}

__device__ __forceinline__ void tma_load_3d(void *smem_dst, const CUtensorMap *map, uint64_t *bar, int32_t x, int32_t y,
                                            int32_t z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
      : "memory");
}

__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two_bytes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(two_bytes)));
  return r;
}

// Four codes of a word as two FP16 pairs.
__device__ __forceinline__ void e4m3x4_to_f16x4(uint32_t w, uint32_t &lo, uint32_t &hi) {
  asm("{\n\t.reg .b16 l, h;\n\t"
      "mov.b32 {l, h}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, l;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
      : "=r"(lo), "=r"(hi)
      : "r"(w));
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}

__device__ __forceinline__ float ex2(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// log2 of a value scale, exact for powers of two; scales below 2^kMinLogScale count as that.
__device__ __forceinline__ float log_scale(float s) {
  const uint32_t b = __float_as_uint(s);
  if (b < (uint32_t(127 + int(kMinLogScale)) << 23)) return kMinLogScale;
  float f;
  asm("lg2.approx.f32 %0, %1;" : "=f"(f) : "f"(__uint_as_float((b & 0x7fffffu) | 0x3f800000u)));
  if ((b & 0x7fffffu) == 0) f = 0.0f;
  return b < 0x7f800000u ? float(int(b >> 23) - 127) + f : __int_as_float(0x7fffffff);
}
// 2^-18 / sV, the factor of a weight in the denominator.  A row has fewer than 2^31 tokens with weights of up
// to 2^15 (or 2^16 per tile of 128), and sV is at least 2^-100: with the 2^-18 their sum stays below 2^128.
constexpr float kSumUnit = 0x1p-18f;
__device__ __forceinline__ float inverse_scale(float s) { return kSumUnit / fmaxf(s, 0x1p-100f); }

// Power of two 2^e that brings a row's largest magnitude into [2^14, 2^15) when the row is
// multiplied by 2^-e; 0 for zero and non-finite rows.
__device__ __forceinline__ int row_exponent(float amax) {
  if (!(amax > 0.0f) || amax > 3.4e38f) return 0;
  int e;
  frexpf(amax, &e);  // amax = m 2^e, 0.5 <= m < 1
  return e - 15;
}

// One sequence of the batch; `high`: largest usable bound of the sequences before it.
struct Seq {
  int64_t start;
  int q_len, kv_len;
  bool ok;
};
__device__ __forceinline__ Seq make_seq(const Args &a, int64_t b, int64_t e, int64_t kv, int64_t high) {
  Seq r;
  r.ok = bounds_ok(b, e, a.tokens) && b >= high && kv >= 0 && kv <= a.max_kv;
  r.start = r.ok ? b : 0;
  r.q_len = r.ok ? static_cast<int>(e - b) : 0;
  r.kv_len = r.ok ? static_cast<int>(kv) : 0;
  return r;
}
// Sequence s by its own bounds.
__device__ __forceinline__ Seq load_seq(const Args &a, int s) {
  return make_seq(a, __ldg(a.cu_seqlens + s), __ldg(a.cu_seqlens + s + 1), __ldg(a.kv_lens + s), 0);
}
// Whether sequence s starts behind the usable bounds of those before, of which `high` (shared) is the largest; it
// takes up s's.  All threads call.
__device__ __forceinline__ bool in_order(const Args &a, int s, int &high) {
  const int b = __ldg(a.cu_seqlens + s), h = high;
  __syncthreads();
  if (threadIdx.x == 0 && b <= a.tokens) high = max(h, b);
  __syncthreads();
  return b >= h;
}
// Sequence s of this thread (nothing if s is behind the last) as it counts; all threads call, `high` and
// s_max as in bound_scan.
template <int THREADS>
__device__ __forceinline__ Seq scan_seq(const Args &a, int s, int &high, int (&s_max)[THREADS / 32]) {
  const bool have = s < a.n_seqs;
  const int64_t b = have ? __ldg(a.cu_seqlens + s) : 0, e = have ? __ldg(a.cu_seqlens + s + 1) : 0;
  return make_seq(a, b, e, have ? __ldg(a.kv_lens + s) : 0, bound_scan<THREADS>(have, b, a.tokens, high, s_max));
}

// Shared memory behind the rings; the warps' O are joined in the rings' place.
template <int D>
struct DecodeSmem {
  uint64_t full[kWarps][Cfg<D>::STAGES];
  float4 scales[kWarps][Cfg<D>::STAGES][Cfg<D>::NG];  // (sK, log2 sV, kSumUnit / sV, -) of each 16-token tile; sK < 0: no tokens there
  float m[kWarps][kRows], l[kWarps][kRows];
  int lim[kRows];
  int nan_first[D];  // first token, among those that some rows of the unit do not see, whose value is NaN
  int64_t scan_t[kWarps], scan_u[kWarps];
  int64_t base_t, base_u;
  int scan_b[kWarps], high;
  int odd;    // some sequence does not count by its own bounds or length
  int found;
};

// Work items per unit (its tiles, or one where units stay whole) and units of a sequence; (0, 0)
// where the prompt kernel takes it.
template <int D>
__device__ __forceinline__ void seq_work(const Args &a, const Seq &s, int &tiles, int &units) {
  const int64_t rows = int64_t(s.q_len) * a.group;
  if (rows == 0 || rows > a.max_decode_rows) {
    tiles = units = 0;
    return;
  }
  tiles = a.whole ? 1 : max(1, (s.kv_len + Cfg<D>::TILE - 1) / Cfg<D>::TILE);
  units = a.kv_heads * static_cast<int>((rows + kRows - 1) / kRows);
}

// Inclusive block scan of two 64-bit values.
__device__ __forceinline__ void block_scan(int64_t &t, int64_t &u, int64_t *st, int64_t *su) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(0xffffffffu, t, o), y = __shfl_up_sync(0xffffffffu, u, o);
    if (lane >= o) {
      t += x;
      u += y;
    }
  }
  if (lane == 31) {
    st[warp] = t;
    su[warp] = u;
  }
  __syncthreads();
  for (int w = 0; w < warp; ++w) {
    t += st[w];
    u += su[w];
  }
}

// A warp's ring.  Lane i < boxes looks up and copies box i of a step (R tokens of one block, K
// and V); it does so for step n + STAGES when step n is done, with the block number fetched one
// step earlier.  The box's scales are written at the end of step n + 1, when they have arrived.
template <int D>
struct Ring {
  using C = Cfg<D>;
  const Args &a;
  const CUtensorMap *k_map, *v_map;
  unsigned char *buf;  // STAGES steps of K, V
  uint64_t *full;
  float4 (*scales)[C::NG];
  int s, h, log_r, lane;
  int end;        // tokens from here on are not wanted
  bool mine;      // this lane has a box

  // Number of the block that holds this lane's box of the step at token `tok`; -1: not wanted.
  __device__ __forceinline__ int lookup(int tok) const {
    const int t = tok + (lane << log_r);
    return mine && t < end ? __ldg(a.table + s * a.ld_table + (t >> a.log_block)) : -1;
  }
  // Copies the step at token `tok`; returns the box's scales (sK < 0: no tokens there).
  __device__ __forceinline__ float2 copy(int stage, int tok, int id) const {
    float2 sc = make_float2(-1.0f, 1.0f);
    if (tok >= end) return sc;  // uniform over the warp
    const int t = tok + (lane << log_r);
    int blk = -1;
    if (mine && t < end) {
      if (id >= 0 && id < a.num_blocks) blk = id * a.kv_heads + h;
      else record_bad_index();
    }
    const uint32_t have = __ballot_sync(0xffffffffu, blk >= 0);
    if (lane == 0) mbar_arrive_expect_tx(full + stage, __popc(have) * ((2 * D) << log_r));
    __syncwarp();
    if (blk >= 0) {
      unsigned char *dst = buf + stage * 2 * C::PART + (lane << log_r) * C::ROWB;
      const int row = t & ((1 << a.log_block) - 1);
#pragma unroll
      for (int p = 0; p < C::PANELS; ++p) {
        tma_load_3d(dst + p * C::TS * C::ROWB, k_map, full + stage, p * C::ROWB, row, blk);
        tma_load_3d(dst + C::PART + p * C::TS * C::ROWB, v_map, full + stage, p * C::ROWB, row, blk);
      }
      sc = make_float2(__ldg(a.k_scales + blk), __ldg(a.v_scales + blk));
    }
    return sc;
  }
  __device__ __forceinline__ void write_scales(int stage, float2 sc) const {
    if (mine) {
      const float4 v = make_float4(sc.x, log_scale(sc.y), inverse_scale(sc.y), 0.0f);
      for (int g = 0; g < (1 << log_r) / kGroup; ++g) scales[stage][(lane << log_r) / kGroup + g] = v;
    }
  }
};

// One segment of a unit: cached tiles [tile0, tile0 + ntile) of (sequence s, kv head h,
// row group rg).  `slot` < 0: the segment is the whole unit and its result goes to `out`,
// else to partial `slot` of the workspace.
template <int D>
__device__ bool decode_segment(const Args &a, const CUtensorMap *k_map, const CUtensorMap *v_map, DecodeSmem<D> &sm,
                               unsigned char *rings, uint32_t &phases, const Seq &sq, int s, int h, int rg, int tile0,
                               int ntile, int slot) {
  using C = Cfg<D>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  unsigned char *buf = rings + warp * (Cfg<D>::STAGES * 2 * C::PART);
  bool ok = true;
  const int g = lane >> 2, q = lane & 3;
  const int n_rows = min(kRows, sq.q_len * a.group - rg * kRows);

  // Visible tokens of each row; the fewest and the most of the unit's rows.
  if (threadIdx.x < kRows) {
    const int R = rg * kRows + min(static_cast<int>(threadIdx.x), n_rows - 1);
    sm.lim[threadIdx.x] = a.causal ? min(sq.kv_len, sq.kv_len - sq.q_len + R / a.group + 1) : sq.kv_len;
  }
  for (int i = threadIdx.x; i < D; i += kThreads) sm.nan_first[i] = 0x7fffffff;

  const int last_row = rg * kRows + n_rows - 1;  // the unit's rows are in token order: it sees most
  const int kv_end = a.causal ? min(sq.kv_len, sq.kv_len - sq.q_len + last_row / a.group + 1) : sq.kv_len;
  const int tok_end = min((tile0 + ntile) * C::TILE, kv_end);
  const int log_r = box_log(a.log_block, D), tok0 = (tile0 * kWarps + warp) * C::TS;
  const Ring<D> ring{a, k_map, v_map, buf, sm.full[warp], sm.scales[warp], s, h, log_r, lane, tok_end, (lane << log_r) < C::TS};
  int id[C::STAGES + 1];
  float2 pending[C::STAGES];
#pragma unroll
  for (int i = 0; i <= C::STAGES; ++i) id[i] = ring.lookup(tok0 + i * C::TILE);
#pragma unroll
  for (int i = 0; i < C::STAGES; ++i) pending[i] = ring.copy(i, tok0 + i * C::TILE, id[i]);
  int next_id = id[C::STAGES];

  // Q fragments of row g: values 64 seg + 16 q + 4 j + {0, 1 | 2, 3}, scaled by 2^-e.
  uint32_t qf[C::SEGK][4][2];
  float rc;
  {
    const int R = rg * kRows + g;
    const bool ok = g < n_rows;
    const uint16_t *src = a.q + (sq.start + (ok ? R / a.group : 0)) * a.ld_q + int64_t(h * a.group + (ok ? R % a.group : 0)) * D;
    uint4 w[C::SEGK][2];
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < C::SEGK; ++i)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        w[i][k] = ok ? __ldg(reinterpret_cast<const uint4 *>(src + 64 * i + 16 * q + 8 * k)) : make_uint4(0, 0, 0, 0);
        const uint32_t x[4] = {w[i][k].x, w[i][k].y, w[i][k].z, w[i][k].w};
#pragma unroll
        for (int n = 0; n < 4; ++n)
          amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(x[n] << 16)), fabsf(__uint_as_float(x[n] & 0xFFFF0000u))));
      }
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    const int e = row_exponent(amax);
    // two factors: 2^-e alone can leave FP32's range.  An infinite value makes every score of the
    // row infinite or NaN: the row is NaN.
    const float f0 = amax <= 3.4e38f ? ldexpf(1.0f, -(e / 2)) : __int_as_float(0x7fffffff), f1 = ldexpf(1.0f, -(e - e / 2));
#pragma unroll
    for (int i = 0; i < C::SEGK; ++i)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t x[4] = {w[i][k].x, w[i][k].y, w[i][k].z, w[i][k].w};
#pragma unroll
        for (int n = 0; n < 4; ++n)
          qf[i][2 * k + (n >> 1)][n & 1] = pack_f16(__uint_as_float(x[n] << 16) * f0 * f1,
                                                    __uint_as_float(x[n] & 0xFFFF0000u) * f0 * f1);
      }
    rc = ldexpf(a.scale_log2, e);
  }
  const float rc0 = __shfl_sync(0xffffffffu, rc, 8 * q), rc1 = __shfl_sync(0xffffffffu, rc, 8 * q + 4);
  __syncthreads();
  const int lim0 = sm.lim[2 * q], lim1 = sm.lim[2 * q + 1];
  const int lim_min = min(sm.lim[0], tok_end);

  float o[C::MB][4];
#pragma unroll
  for (int i = 0; i < C::MB; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) o[i][j] = 0.0f;
  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.0f, l1 = 0.0f;

#pragma unroll
  for (int i = 0; i < C::STAGES; ++i) ring.write_scales(i, pending[i]);
  __syncwarp();
  int stage = 0, last = -1;  // last: stage of the scales on their way
  float2 sc_last = make_float2(0.0f, 0.0f);
  const int tk = token_of(g);
#pragma unroll 1
  for (int tok = tok0; tok < tok_end; tok += C::TILE) {
    ok = __all_sync(0xffffffffu, mbar_wait(&sm.full[warp][stage], (phases >> stage) & 1));
    if (!ok) break;
    phases ^= 1u << stage;
    const unsigned char *kb = buf + stage * 2 * C::PART, *vb = kb + C::PART;
    float4 sc[C::NG];
#pragma unroll
    for (int n = 0; n < C::NG; ++n) sc[n] = sm.scales[warp][stage][n];

    // A step whose tokens all rows see needs no masks.
    bool tail = tok + C::TS > lim_min;
#pragma unroll
    for (int n = 0; n < C::NG; ++n) tail |= sc[n].x < 0.0f;
    auto step = [&](auto masked) {
      constexpr bool MASK = decltype(masked)::value;
      float x[C::NG][4];
#pragma unroll
      for (int n = 0; n < C::NG; ++n) {
#pragma unroll
        for (int j = 0; j < 4; ++j) x[n][j] = 0.0f;
#pragma unroll
        for (int i = 0; i < C::SEGK; ++i) {
          const int panel = i * 64 / C::ROWB, piece = (i * 64 % C::ROWB) / 16 + q;
          const unsigned char *base = kb + panel * C::TS * C::ROWB;
          const uint4 lo = *reinterpret_cast<const uint4 *>(base + swizzled<D>(kGroup * n + tk, piece));
          const uint4 hi = *reinterpret_cast<const uint4 *>(base + swizzled<D>(kGroup * n + tk + 8, piece));
          const uint32_t ka[4] = {lo.x, lo.y, lo.z, lo.w}, kc[4] = {hi.x, hi.y, hi.z, hi.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t a0, a1, a2, a3;
            e4m3x4_to_f16x4(ka[j], a0, a2);
            e4m3x4_to_f16x4(kc[j], a1, a3);
            mma_f16(x[n], a0, a1, a2, a3, qf[i][j][0], qf[i][j][1]);
          }
        }
      }

      float mx0 = -INFINITY, mx1 = -INFINITY;
#pragma unroll
      for (int n = 0; n < C::NG; ++n) {
        const float c0 = sc[n].x * rc0, c1 = sc[n].x * rc1, e = sc[n].y;
        x[n][0] = fmaf(x[n][0], c0, e);
        x[n][1] = fmaf(x[n][1], c1, e);
        x[n][2] = fmaf(x[n][2], c0, e);
        x[n][3] = fmaf(x[n][3], c1, e);
        if constexpr (MASK) {
          const bool none = sc[n].x < 0.0f || tok + kGroup * n >= tok_end;
          const int t0 = none ? 0x7fffffff - 8 : tok + kGroup * n + tk;
          x[n][0] = t0 < lim0 ? x[n][0] : -INFINITY;
          x[n][1] = t0 < lim1 ? x[n][1] : -INFINITY;
          x[n][2] = t0 + 8 < lim0 ? x[n][2] : -INFINITY;
          x[n][3] = t0 + 8 < lim1 ? x[n][3] : -INFINITY;
        }
        mx0 = fmaxf(mx0, fmaxf(x[n][0], x[n][2]));
        mx1 = fmaxf(mx1, fmaxf(x[n][1], x[n][3]));
      }
      // The reference stays while no weight exceeds 2^(kBoost + kSlack).
      if (__any_sync(0xffffffffu, mx0 > m0 + kSlack || mx1 > m1 + kSlack)) {
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) {
          mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, w));
          mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, w));
        }
        const float f0 = mx0 > m0 ? ex2(m0 - mx0) : 1.0f, f1 = mx1 > m1 ? ex2(m1 - mx1) : 1.0f;
        m0 = fmaxf(m0, mx0), m1 = fmaxf(m1, mx1);
        l0 *= f0, l1 *= f1;
#pragma unroll
        for (int i = 0; i < C::MB; ++i) {
          o[i][0] *= f0, o[i][1] *= f1;
          o[i][2] *= f0, o[i][3] *= f1;
        }
      }
      const float b0 = (m0 == -INFINITY ? 0.0f : m0) - kBoost, b1 = (m1 == -INFINITY ? 0.0f : m1) - kBoost;
      uint32_t pf[C::NG][2];
#pragma unroll
      for (int n = 0; n < C::NG; ++n) {
        const float p0 = ex2(x[n][0] - b0), p1 = ex2(x[n][1] - b1), p2 = ex2(x[n][2] - b0), p3 = ex2(x[n][3] - b1);
        l0 = fmaf(p0 + p2, sc[n].z, l0);
        l1 = fmaf(p1 + p3, sc[n].z, l1);
        pf[n][0] = movmatrix_trans(pack_f16(p0, p1));
        pf[n][1] = movmatrix_trans(pack_f16(p2, p3));
      }
      // V: a lane's 16 (at 64 values 8) values of its four tokens of each tile.
#pragma unroll
      for (int n = 0; n < C::NG; ++n)
#pragma unroll
        for (int i = 0; i < C::SEGV; ++i) {
          uint32_t r[4][C::VW];
#pragma unroll
          for (int t = 0; t < 4; ++t) {
            const int row = kGroup * n + token_of(2 * q + (t & 1)) + 8 * (t >> 1);
            if constexpr (C::VW == 4) {
              const uint4 x4 = *reinterpret_cast<const uint4 *>(vb + i * C::TS * C::ROWB + swizzled<D>(row, g));
              r[t][0] = x4.x, r[t][1] = x4.y, r[t][2] = x4.z, r[t][3] = x4.w;
            } else {
              const uint2 x2 = *reinterpret_cast<const uint2 *>(vb + swizzled<D>(row, g >> 1) + 8 * (g & 1));
              r[t][0] = x2.x, r[t][1] = x2.y;
            }
            // Bytes that belong to no token never reach the product.  Nor do, among tokens that only some
            // of the rows see, NaN: the others' weight is 0, and 0 * NaN is NaN; its place is remembered.
            if constexpr (MASK) {
              const bool gone = sc[n].x < 0.0f || tok + row >= tok_end;
#pragma unroll
              for (int w = 0; w < C::VW; ++w) {
                uint32_t &word = r[t][w];
                if (gone) word = 0;
                if ((((word & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) == 0) continue;
                for (int b = 0; b < 4; ++b)
                  if (((word >> (8 * b)) & 0x7f) == 0x7f) {
                    atomicMin(&sm.nan_first[i * 128 + 4 * C::VW * g + 4 * w + b], tok + row);
                    word &= ~(0xffu << (8 * b));
                  }
              }
            }
          }
#pragma unroll
          for (int w = 0; w < C::VW; ++w) {
            // tokens (0, 1) and (2, 3) of values (0, 1), then (2, 3) of the word
#pragma unroll
            for (int v = 0; v < 2; ++v) {
              const uint32_t sel = v == 0 ? 0x5140 : 0x7362;
              uint32_t a0, a1, a2, a3;
              e4m3x4_to_f16x4(__byte_perm(r[0][w], r[1][w], sel), a0, a1);
              e4m3x4_to_f16x4(__byte_perm(r[2][w], r[3][w], sel), a2, a3);
              mma_f16(o[(i * C::VW + w) * 2 + v], a0, a1, a2, a3, pf[n][0], pf[n][1]);
            }
          }
        }
    };
    if (tail) step(std::true_type{});
    else step(std::false_type{});
    if (last >= 0) ring.write_scales(last, sc_last);
    __syncwarp();  // the stage has been read, and the scales are there before their step
    const int ahead = tok + C::STAGES * C::TILE;
    last = ahead < tok_end ? stage : -1;
    sc_last = ring.copy(stage, ahead, next_id);
    next_id = ring.lookup(ahead + C::TILE);
    stage = stage + 1 == Cfg<D>::STAGES ? 0 : stage + 1;
  }
  if (__syncthreads_or(!ok)) return false;  // a copy never came; the rings are in use no more

  // Join the warps: (O, M, l) of each through shared memory.
#pragma unroll
  for (int w = 4; w < 32; w <<= 1) {
    l0 += __shfl_xor_sync(0xffffffffu, l0, w);
    l1 += __shfl_xor_sync(0xffffffffu, l1, w);
  }
  float (*so)[kRows][C::LD] = reinterpret_cast<float (*)[kRows][C::LD]>(rings);
  if (g == 0) {
    sm.m[warp][2 * q] = m0, sm.m[warp][2 * q + 1] = m1;
    sm.l[warp][2 * q] = l0, sm.l[warp][2 * q + 1] = l1;
  }
#pragma unroll
  for (int i = 0; i < C::SEGV; ++i)
#pragma unroll
    for (int w = 0; w < C::VW; ++w)
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int j = 0; j < 4; ++j)  // accumulator (value 2 b + j / 2 of the word, row 2 q + j % 2)
          so[warp][2 * q + (j & 1)][i * 128 + 4 * C::VW * g + 4 * w + 2 * b + (j >> 1)] = o[(i * C::VW + w) * 2 + b][j];
  __syncthreads();
  for (int idx = threadIdx.x; idx < kRows * (D / 2); idx += kThreads) {
    const int r = idx / (D / 2), c = (idx % (D / 2)) * 2;
    if (r >= n_rows) break;
    float M = sm.m[0][r];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) M = fmaxf(M, sm.m[w][r]);
    const float base = M == -INFINITY ? 0.0f : M;
    float l = 0.0f, o0 = 0.0f, o1 = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = ex2(sm.m[w][r] - base);
      l = fmaf(sm.l[w][r], f, l);
      o0 = fmaf(so[w][r][c], f, o0);
      o1 = fmaf(so[w][r][c + 1], f, o1);
    }
    if (sm.nan_first[c] < sm.lim[r]) o0 = __int_as_float(0x7fffffff);
    if (sm.nan_first[c + 1] < sm.lim[r]) o1 = __int_as_float(0x7fffffff);
    if (slot >= 0) {
      *reinterpret_cast<float2 *>(a.part + (int64_t(slot) * kRows + r) * D + c) = make_float2(o0, o1);
      if (c == 0) a.part_ml[slot * kRows + r] = make_float2(M, l);
    } else {
      const float f = l == 0.0f ? 0.0f : kSumUnit / l;  // no visible token: the row is 0
      const int R = rg * kRows + r;
      const int64_t at = (sq.start + R / a.group) * a.ld_out + int64_t(h * a.group + R % a.group) * D + c;
      if (a.out_fp32)
        *reinterpret_cast<float2 *>(static_cast<float *>(a.out) + at) = make_float2(o0 * f, o1 * f);
      else
        *reinterpret_cast<__nv_bfloat162 *>(static_cast<uint16_t *>(a.out) + at) = __floats2bfloat162_rn(o0 * f, o1 * f);
    }
  }
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the rings are written by copies again
  __syncthreads();
  return true;
}

template <int D>
__global__ void __launch_bounds__(kThreads, Cfg<D>::CTAS)
    decode_kernel(const __grid_constant__ Args a, const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap v_map) {
  extern __shared__ unsigned char smem_raw[];
  unsigned char *rings = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  DecodeSmem<D> &sm = *reinterpret_cast<DecodeSmem<D> *>(rings + Cfg<D>::RING);
  if (threadIdx.x < kWarps * Cfg<D>::STAGES) mbar_init(&sm.full[0][0] + threadIdx.x, 1);
  fence_barrier_init();
  if (threadIdx.x == 0) sm.odd = 0;
  __syncthreads();
  uint32_t phases = 0;  // bit i: parity of the next phase of the warp's stage i
  grid_dep_wait();
  grid_dep_launch();

  // Total work.  Inclusive sums of the last batch of kThreads sequences stay in t_sum, u_sum.
  int64_t total = 0, total_u = 0, t_sum = 0, u_sum = 0;
  int tiles = 0, units = 0;
  int high = 0;
  auto batch_sums = [&](int s0) {
    tiles = units = 0;
    const int s = s0 + threadIdx.x;
    if (s < a.n_seqs) {
      const Seq q = load_seq(a, s);
      if (!q.ok) sm.odd = 1;
      seq_work<D>(a, q, tiles, units);
    }
    t_sum = int64_t(tiles) * units;
    u_sum = units;
    block_scan(t_sum, u_sum, sm.scan_t, sm.scan_u);
    if (sm.odd) {  // again, with what the earlier sequences' bounds leave
      const Seq q = scan_seq<kThreads>(a, s, high, sm.scan_b);
      if (s < a.n_seqs && !q.ok && blockIdx.x == 0) record_bad_index();
      seq_work<D>(a, q, tiles, units);
      t_sum = int64_t(tiles) * units;
      u_sum = units;
      block_scan(t_sum, u_sum, sm.scan_t, sm.scan_u);
    }
  };
  for (int s0 = 0; s0 < a.n_seqs; s0 += kThreads) {
    batch_sums(s0);
    if (threadIdx.x == kThreads - 1) {
      sm.base_t = t_sum;
      sm.base_u = u_sum;
    }
    __syncthreads();
    total += sm.base_t;
    total_u += sm.base_u;
    __syncthreads();
  }
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.n_units = static_cast<int>(total_u);
  const int64_t ctas = min(int64_t(gridDim.x), total);
  if (int64_t(blockIdx.x) >= ctas) return;
  const int64_t begin = blockIdx.x * total / ctas, end = (blockIdx.x + 1) * total / ctas;

  // The sequence that holds tile `begin`, and the tiles and units before it.
  int64_t before_t = 0;
  int before_u = 0;  // the units fit the combine kernel's grid
  int seq = 0;
  high = 0;
  for (int s0 = 0; s0 < a.n_seqs; s0 += kThreads) {
    if (threadIdx.x == 0) sm.found = -1;
    if (a.n_seqs > kThreads) batch_sums(s0);
    __syncthreads();
    const int64_t mine = int64_t(tiles) * units;
    if (before_t + t_sum > begin && before_t + t_sum - mine <= begin) {
      sm.found = s0 + threadIdx.x;
      sm.base_t = before_t + t_sum - mine;
      sm.base_u = before_u + u_sum - units;
    }
    __syncthreads();
    if (sm.found >= 0) {
      seq = sm.found;
      before_t = sm.base_t;
      before_u = static_cast<int>(sm.base_u);
      break;
    }
    if (threadIdx.x == kThreads - 1) {
      sm.base_t = before_t + t_sum;
      sm.base_u = before_u + u_sum;
    }
    __syncthreads();
    before_t = sm.base_t;
    before_u = static_cast<int>(sm.base_u);
    __syncthreads();
  }
  __syncthreads();

  int64_t at = begin;
  Seq sq = load_seq(a, seq);
  if (sm.odd) {
    if (threadIdx.x == 0) sm.high = static_cast<int>(sq.start);
    __syncthreads();
  }
  seq_work<D>(a, sq, tiles, units);
  while (at < end) {
    while (at >= before_t + int64_t(tiles) * units) {  // next sequence with work
      before_t += int64_t(tiles) * units;
      before_u += units;
      if (++seq >= a.n_seqs) return;
      sq = load_seq(a, seq);
      if (sm.odd && !in_order(a, seq, sm.high)) sq.q_len = 0;
      seq_work<D>(a, sq, tiles, units);
    }
    const int64_t local = at - before_t;
    const int unit = static_cast<int>(local / tiles), tile0 = static_cast<int>(local - int64_t(unit) * tiles);
    const int ntile = static_cast<int>(min(int64_t(tiles - tile0), end - at));
    const int h = unit % a.kv_heads, rg = unit / a.kv_heads;
    const bool whole = ntile == tiles;
    if (!a.whole && tile0 == 0 && threadIdx.x == 0) {
      const int64_t last = before_t + int64_t(unit + 1) * tiles - 1;
      a.desc[before_u + unit] = make_int4(seq, h, rg, 0);
      a.desc2[before_u + unit] = make_int2(blockIdx.x, static_cast<int>(((last + 1) * ctas - 1) / total));
    }
    if (!decode_segment<D>(a, &k_map, &v_map, sm, rings, phases, sq, seq, h, rg, tile0, a.whole ? kWholeTiles : ntile,
                           whole ? -1 : 2 * int(blockIdx.x) + (tile0 == 0)))
      return;
    at += ntile;
  }
}

template <int D>
constexpr int decode_smem_bytes() {
  return 1024 + Cfg<D>::RING + int(sizeof(DecodeSmem<D>));
}

// Joins the partial results of the units that several CTAs share.  Grid (units, kRows / ROWS): D / 4
// threads take four values each of a query row, for one in kJoin partials.
template <int D>
struct Join {
  static constexpr int PARTS = 4, ROWS = 2, PER_ROW = D / 4, THREADS = ROWS * PER_ROW * PARTS;
};
template <int D>
__global__ void __launch_bounds__(Join<D>::THREADS) combine_kernel(const __grid_constant__ Args a) {
  constexpr int kJoin = Join<D>::PARTS, ROWS = Join<D>::ROWS;
  __shared__ float4 so[kJoin][ROWS][D / 4];
  __shared__ float sl[kJoin][ROWS], smax[kJoin][ROWS];
  grid_dep_wait();
  grid_dep_launch();
  if (int(blockIdx.x) >= *a.n_units) return;
  const int2 c = a.desc2[blockIdx.x];
  if (c.x == c.y) return;  // one CTA wrote the result
  const int4 u = a.desc[blockIdx.x];
  const Seq sq = load_seq(a, u.x);
  const int part = threadIdx.x / (ROWS * D / 4), r = threadIdx.x / (D / 4) % ROWS, col = threadIdx.x % (D / 4);
  const int row = blockIdx.y * ROWS + r, R = u.z * kRows + row;
  const bool valid = R < sq.q_len * a.group;  // other rows' partials are not written
  // the first CTA's partial is its last segment, the others' their first
  auto slot = [&](int i) { return int64_t(2 * i + (i == c.x)) * kRows + row; };
  // every kJoin-th partial, with a running maximum; four loads in flight
  float M = -INFINITY, l = 0.0f;
  float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  for (int i0 = c.x + part; valid && i0 <= c.y; i0 += 4 * kJoin) {
    float2 ml[4];
    float4 v[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = i0 + k * kJoin;
      ml[k] = make_float2(-INFINITY, 0.0f);
      v[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (i <= c.y) {
        ml[k] = a.part_ml[slot(i)];
        v[k] = *reinterpret_cast<const float4 *>(a.part + slot(i) * D + 4 * col);
      }
    }
    float m = M;
#pragma unroll
    for (int k = 0; k < 4; ++k) m = fmaxf(m, ml[k].x);
    const float base = m == -INFINITY ? 0.0f : m, g = ex2(M - base);
    l *= g;
    o.x *= g, o.y *= g, o.z *= g, o.w *= g;
    M = m;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (i0 + k * kJoin > c.y) continue;
      const float f = ex2(ml[k].x - base);
      l = fmaf(ml[k].y, f, l);
      o.x = fmaf(v[k].x, f, o.x), o.y = fmaf(v[k].y, f, o.y), o.z = fmaf(v[k].z, f, o.z), o.w = fmaf(v[k].w, f, o.w);
    }
  }
  so[part][r][col] = o;
  if (col == 0) sl[part][r] = l, smax[part][r] = M;
  __syncthreads();
  if (part != 0 || !valid) return;
  float m = smax[0][r];
#pragma unroll
  for (int k = 1; k < kJoin; ++k) m = fmaxf(m, smax[k][r]);
  const float base = m == -INFINITY ? 0.0f : m;
  l = 0.0f;
  o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
  for (int k = 0; k < kJoin; ++k) {
    const float f = ex2(smax[k][r] - base);
    const float4 v = so[k][r][col];
    l = fmaf(sl[k][r], f, l);
    o.x = fmaf(v.x, f, o.x), o.y = fmaf(v.y, f, o.y), o.z = fmaf(v.z, f, o.z), o.w = fmaf(v.w, f, o.w);
  }
  const float f = l == 0.0f ? 0.0f : kSumUnit / l;
  const int64_t at = (sq.start + R / a.group) * a.ld_out + int64_t(u.y * a.group + R % a.group) * D + 4 * col;
  if (a.out_fp32) {
    *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + at) = make_float4(o.x * f, o.y * f, o.z * f, o.w * f);
  } else {
    __nv_bfloat162 p[2] = {__floats2bfloat162_rn(o.x * f, o.y * f), __floats2bfloat162_rn(o.z * f, o.w * f)};
    *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + at) = *reinterpret_cast<const uint2 *>(p);
  }
}

}  // namespace attn
}  // namespace nvfp4

// Attention over the block-scaled 8-bit cache for sequences with few new tokens.
//
// For a query row q (one head of one token) and the cached tokens j it sees,
//     x_j = scale log2(e) sK_j (q . k_j),   o = sum_j 2^{x_j} sV_j v_j / sum_j 2^{x_j},
// where k_j, v_j are E4M3 codes and sK_j, sV_j the scales of j's block.  One pass with a
// running maximum; the maximum is taken over x_j + log2 sV_j, so that the weights the
// matrix instruction sees,
//     P_j = 2^{x_j + log2 sV_j - M + kBoost},
// already hold the value scale and are at most 2^kBoost, while the denominator adds
// P_j / sV_j.  kBoost keeps weights down to 2^-36 of the largest above the FP16 subnormals.
//
// Bound by HBM: every cached byte is read once per kv head, for 2 x 8 multiply-adds.  So
// K and V go from global memory straight into registers in the layout that
// mma.m16n8k16 wants, with no trip through shared memory:
//  * S^T = K Q^T has the cached tokens as its 16 rows and up to 8 query rows (the heads of
//    a group, times tokens) as its 8 columns.  The contraction runs over the head's
//    values in any order as long as K and Q agree, so a lane takes 16 consecutive bytes
//    of a token's row as its values of four k-steps.
//  * O^T = V^T P^T has 16 values as its rows and 16 tokens as its contraction: a lane
//    reads the same 16 values of four tokens and byte permutes pair the tokens.  The
//    accumulators' columns are query rows again, so rescaling is lane-local, and
//    movmatrix turns S^T's accumulators into the P^T operand.
// E4M3 is exact in FP16; q is scaled by a power of two per row to lie in FP16's range
// and keeps all of its BF16 bits within 2^-29 of the row's largest value.  Sums, maxima
// and accumulators are FP32.
//
// The cached tiles of all (sequence, kv head, 8-row group) units form one list that is
// cut evenly over the CTAs; a unit that several CTAs share leaves partial results
// (O, M, l) in the workspace and combine_kernel joins them in a fixed order.
#pragma once

#include <cuda_fp16.h>

#include "ptx.cuh"

namespace nvfp4 {
namespace attn {

constexpr int kRows = 8;        // query rows of a unit
constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr float kBoost = 12.0f;
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
  int max_decode_rows;        // sequences with more query rows per kv head belong to the prompt kernel
};

template <int D>
struct Cfg {
  static constexpr int TS = D == 256 ? 16 : 32;  // tokens of a warp's step
  static constexpr int NG = TS / kGroup;
  static constexpr int TILE = TS * kWarps;       // tokens of a CTA's step
  static constexpr int SEGK = D / 64;            // 64-value segments of a K row
  static constexpr int VW = D >= 128 ? 4 : 2;    // 32-bit words of V per lane and token, per segment
  static constexpr int SEGV = D >= 128 ? D / 128 : 1;
  static constexpr int MB = D / 16;              // 16-value row blocks of O^T
  static constexpr int LD = D + 4;
};

__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two_bytes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(two_bytes)));
  return r;
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

__device__ __forceinline__ uint4 ld_stream(const void *p) {
  uint4 r;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}
__device__ __forceinline__ uint2 ld_stream2(const void *p) {
  uint2 r;
  asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(r.x), "=r"(r.y) : "l"(p));
  return r;
}

// log2 of a value scale, exact for powers of two.
__device__ __forceinline__ float log_scale(float s) { return fmaxf(log2f(s), kMinLogScale) + (s != s ? s : 0.0f); }

// Power of two 2^e that brings a row's largest magnitude into [2^14, 2^15) when the row is
// multiplied by 2^-e; 0 for zero and non-finite rows.
__device__ __forceinline__ int row_exponent(float amax) {
  if (!(amax > 0.0f) || amax > 3.4e38f) return 0;
  int e;
  frexpf(amax, &e);  // amax = m 2^e, 0.5 <= m < 1
  return e - 15;
}

// One sequence of the batch.
struct Seq {
  int64_t start;
  int q_len, kv_len;
  bool ok;
};
__device__ __forceinline__ Seq load_seq(const Args &a, int s) {
  Seq r;
  const int64_t b = __ldg(a.cu_seqlens + s), e = __ldg(a.cu_seqlens + s + 1);
  const int64_t kv = __ldg(a.kv_lens + s);
  r.ok = b >= 0 && e >= b && e <= a.tokens && kv >= 0 && kv <= a.max_kv;
  r.start = r.ok ? b : 0;
  r.q_len = r.ok ? static_cast<int>(e - b) : 0;
  r.kv_len = r.ok ? static_cast<int>(kv) : 0;
  return r;
}

template <int D>
struct DecodeSmem {
  float o[kWarps][kRows][Cfg<D>::LD];
  float m[kWarps][kRows], l[kWarps][kRows];
  int lim[kRows];
  int nan_first[D];  // first token, among those that some rows of the unit do not see, whose value is NaN
  int64_t scan_t[kWarps], scan_u[kWarps];
  int64_t base_t, base_u;
  int found;
};

// Tiles and units of a sequence; (0, 0) where the prompt kernel takes it.
template <int D>
__device__ __forceinline__ void seq_work(const Args &a, const Seq &s, int &tiles, int &units) {
  const int64_t rows = int64_t(s.q_len) * a.group;
  if (rows == 0 || rows > a.max_decode_rows) {
    tiles = units = 0;
    return;
  }
  tiles = max(1, (s.kv_len + Cfg<D>::TILE - 1) / Cfg<D>::TILE);
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

template <int D>
struct KStage {
  uint4 r[Cfg<D>::NG][2][Cfg<D>::SEGK];
};
template <int D>
struct VStage {
  uint32_t r[Cfg<D>::NG][4][Cfg<D>::SEGV][Cfg<D>::VW];
};

// Where a 16-token group lives: its block's (block, head) index, or -1.
template <int D>
__device__ __forceinline__ int64_t group_block(const Args &a, int s, int h, int tok, int kv_len) {
  if (tok >= kv_len) return -1;
  const int64_t id = __ldg(a.table + s * a.ld_table + (tok >> a.log_block));
  if (id < 0 || id >= a.num_blocks) {
    record_bad_index();
    return -1;
  }
  return id * a.kv_heads + h;
}

template <int D>
__device__ __forceinline__ void load_k(const Args &a, uint4 (&r)[2][Cfg<D>::SEGK], int64_t blk, int tok, int kv_len) {
  const int g = (threadIdx.x & 31) >> 2, q = threadIdx.x & 3;
  const int off = tok & ((1 << a.log_block) - 1);
  const uint8_t *p = a.k + ((blk << a.log_block) + off + g) * D + 16 * q;
#pragma unroll
  for (int i = 0; i < 2; ++i)
#pragma unroll
    for (int s = 0; s < Cfg<D>::SEGK; ++s)
      r[i][s] = blk >= 0 && tok + g + 8 * i < kv_len ? ld_stream(p + i * 8 * D + s * 64) : make_uint4(0, 0, 0, 0);
}

template <int D>
__device__ __forceinline__ void load_v(const Args &a, uint32_t (&r)[4][Cfg<D>::SEGV][Cfg<D>::VW], int64_t blk, int tok,
                                       int kv_len) {
  using C = Cfg<D>;
  const int g = (threadIdx.x & 31) >> 2, q = threadIdx.x & 3;
  const int off = tok & ((1 << a.log_block) - 1);
  const uint8_t *p = a.v + ((blk << a.log_block) + off) * D + 4 * C::VW * g;
#pragma unroll
  for (int t = 0; t < 4; ++t) {
    const int tt = 2 * q + (t & 1) + 8 * (t >> 1);  // tokens 2q, 2q + 1, 2q + 8, 2q + 9
    const bool ok = blk >= 0 && tok + tt < kv_len;  // bytes behind the sequence never reach the product
#pragma unroll
    for (int s = 0; s < C::SEGV; ++s) {
      if constexpr (C::VW == 4) {
        const uint4 x = ok ? ld_stream(p + int64_t(tt) * D + s * 128) : make_uint4(0, 0, 0, 0);
        r[t][s][0] = x.x, r[t][s][1] = x.y, r[t][s][2] = x.z, r[t][s][3] = x.w;
      } else {
        const uint2 x = ok ? ld_stream2(p + int64_t(tt) * D) : make_uint2(0, 0);
        r[t][s][0] = x.x, r[t][s][1] = x.y;
      }
    }
  }
}

// One segment of a unit: cached tiles [tile0, tile0 + ntile) of (sequence s, kv head h,
// row group rg).  `slot` < 0: the segment is the whole unit and its result goes to `out`,
// else to partial `slot` of the workspace.
template <int D>
__device__ void decode_segment(const Args &a, DecodeSmem<D> &sm, const Seq &sq, int s, int h, int rg, int tile0,
                               int ntile, int slot) {
  using C = Cfg<D>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, q = lane & 3;
  const int n_rows = min(kRows, sq.q_len * a.group - rg * kRows);

  // Visible tokens of each row; the fewest and the most of the unit's rows.
  if (threadIdx.x < kRows) {
    const int R = rg * kRows + min(static_cast<int>(threadIdx.x), n_rows - 1);
    sm.lim[threadIdx.x] = a.causal ? min(sq.kv_len, sq.kv_len - sq.q_len + R / a.group + 1) : sq.kv_len;
  }
  for (int i = threadIdx.x; i < D; i += kThreads) sm.nan_first[i] = 0x7fffffff;

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
  const int lim_min = sm.lim[0], lim_max = sm.lim[kRows - 1];  // rows are in token order
  const int kv_end = min(sq.kv_len, lim_max);

  float o[C::MB][4];
#pragma unroll
  for (int i = 0; i < C::MB; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) o[i][j] = 0.0f;
  float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.0f, l1 = 0.0f;

  int tok = (tile0 * kWarps + warp) * C::TS;
  const int tok_end = min((tile0 + ntile) * C::TILE, kv_end);
  KStage<D> ks;
  int64_t blk[C::NG];
#pragma unroll
  for (int n = 0; n < C::NG; ++n) {
    blk[n] = group_block<D>(a, s, h, tok + kGroup * n, min(kv_end, tok_end));
    load_k<D>(a, ks.r[n], blk[n], tok + kGroup * n, kv_end);
  }
  for (; tok < tok_end; tok += C::TILE) {
    VStage<D> vs;
    float sk[C::NG], sv[C::NG];
#pragma unroll
    for (int n = 0; n < C::NG; ++n) {
      load_v<D>(a, vs.r[n], blk[n], tok + kGroup * n, kv_end);
      sk[n] = blk[n] >= 0 ? __ldg(a.k_scales + blk[n]) : 0.0f;
      sv[n] = blk[n] >= 0 ? __ldg(a.v_scales + blk[n]) : 1.0f;
    }
    int64_t nblk[C::NG];
#pragma unroll
    for (int n = 0; n < C::NG; ++n) nblk[n] = group_block<D>(a, s, h, tok + C::TILE + kGroup * n, tok_end);

    float x[C::NG][4];
#pragma unroll
    for (int n = 0; n < C::NG; ++n) {
#pragma unroll
      for (int j = 0; j < 4; ++j) x[n][j] = 0.0f;
#pragma unroll
      for (int i = 0; i < C::SEGK; ++i) {
        const uint32_t ka[4] = {ks.r[n][0][i].x, ks.r[n][0][i].y, ks.r[n][0][i].z, ks.r[n][0][i].w};
        const uint32_t kb[4] = {ks.r[n][1][i].x, ks.r[n][1][i].y, ks.r[n][1][i].z, ks.r[n][1][i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          mma_f16(x[n], e4m3x2_to_f16x2(ka[j]), e4m3x2_to_f16x2(kb[j]), e4m3x2_to_f16x2(ka[j] >> 16),
                  e4m3x2_to_f16x2(kb[j] >> 16), qf[i][j][0], qf[i][j][1]);
      }
    }
#pragma unroll
    for (int n = 0; n < C::NG; ++n) load_k<D>(a, ks.r[n], nblk[n], tok + C::TILE + kGroup * n, kv_end);

    float mx0 = m0, mx1 = m1, inv[C::NG];
#pragma unroll
    for (int n = 0; n < C::NG; ++n) {
      const float e = log_scale(sv[n]);
      inv[n] = exp2f(-e);
      const float c0 = sk[n] * rc0, c1 = sk[n] * rc1;
      const int t0 = blk[n] >= 0 ? tok + kGroup * n + g : 0x7fffffff - 8;
      x[n][0] = t0 < lim0 ? fmaf(x[n][0], c0, e) : -INFINITY;
      x[n][1] = t0 < lim1 ? fmaf(x[n][1], c1, e) : -INFINITY;
      x[n][2] = t0 + 8 < lim0 ? fmaf(x[n][2], c0, e) : -INFINITY;
      x[n][3] = t0 + 8 < lim1 ? fmaf(x[n][3], c1, e) : -INFINITY;
      mx0 = fmaxf(mx0, fmaxf(x[n][0], x[n][2]));
      mx1 = fmaxf(mx1, fmaxf(x[n][1], x[n][3]));
    }
#pragma unroll
    for (int w = 4; w < 32; w <<= 1) {
      mx0 = fmaxf(mx0, __shfl_xor_sync(0xffffffffu, mx0, w));
      mx1 = fmaxf(mx1, __shfl_xor_sync(0xffffffffu, mx1, w));
    }
    if (__any_sync(0xffffffffu, mx0 > m0 || mx1 > m1)) {
      const float f0 = mx0 > m0 ? ex2(m0 - mx0) : 1.0f, f1 = mx1 > m1 ? ex2(m1 - mx1) : 1.0f;
      m0 = mx0, m1 = mx1;
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
      l0 = fmaf(p0 + p2, inv[n], l0);
      l1 = fmaf(p1 + p3, inv[n], l1);
      pf[n][0] = movmatrix_trans(pack_f16(p0, p1));
      pf[n][1] = movmatrix_trans(pack_f16(p2, p3));
    }
    // Tokens that only some of the rows see: a NaN value there must not reach the rows that
    // do not (their weight is 0, and 0 * NaN is NaN), so it is taken out of the product
    // and its place remembered.
    if (tok + C::TS > lim_min) {
#pragma unroll
      for (int n = 0; n < C::NG; ++n)
#pragma unroll
        for (int t = 0; t < 4; ++t)
#pragma unroll
          for (int i = 0; i < C::SEGV; ++i)
#pragma unroll
            for (int w = 0; w < C::VW; ++w) {
              uint32_t &word = vs.r[n][t][i][w];
              if ((((word & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) == 0) continue;
              const int tt = tok + kGroup * n + 2 * q + (t & 1) + 8 * (t >> 1);
              for (int b = 0; b < 4; ++b)
                if (((word >> (8 * b)) & 0x7f) == 0x7f) {
                  atomicMin(&sm.nan_first[i * 128 + 4 * C::VW * g + 4 * w + b], tt);
                  word &= ~(0xffu << (8 * b));
                }
            }
    }
#pragma unroll
    for (int n = 0; n < C::NG; ++n)
#pragma unroll
      for (int i = 0; i < C::SEGV; ++i)
#pragma unroll
        for (int w = 0; w < C::VW; ++w) {
          const uint32_t(&r)[4][C::SEGV][C::VW] = vs.r[n];
          const uint32_t lo01 = __byte_perm(r[0][i][w], r[1][i][w], 0x5140);
          const uint32_t lo23 = __byte_perm(r[2][i][w], r[3][i][w], 0x5140);
          const uint32_t hi01 = __byte_perm(r[0][i][w], r[1][i][w], 0x7362);
          const uint32_t hi23 = __byte_perm(r[2][i][w], r[3][i][w], 0x7362);
          float(&oa)[4] = o[(i * C::VW + w) * 2], (&ob)[4] = o[(i * C::VW + w) * 2 + 1];
          mma_f16(oa, e4m3x2_to_f16x2(lo01), e4m3x2_to_f16x2(lo01 >> 16), e4m3x2_to_f16x2(lo23),
                  e4m3x2_to_f16x2(lo23 >> 16), pf[n][0], pf[n][1]);
          mma_f16(ob, e4m3x2_to_f16x2(hi01), e4m3x2_to_f16x2(hi01 >> 16), e4m3x2_to_f16x2(hi23),
                  e4m3x2_to_f16x2(hi23 >> 16), pf[n][0], pf[n][1]);
        }
#pragma unroll
    for (int n = 0; n < C::NG; ++n) blk[n] = nblk[n];
  }

  // Join the warps: (O, M, l) of each through shared memory.
#pragma unroll
  for (int w = 4; w < 32; w <<= 1) {
    l0 += __shfl_xor_sync(0xffffffffu, l0, w);
    l1 += __shfl_xor_sync(0xffffffffu, l1, w);
  }
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
          sm.o[warp][2 * q + (j & 1)][i * 128 + 4 * C::VW * g + 4 * w + 2 * b + (j >> 1)] = o[(i * C::VW + w) * 2 + b][j];
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
      o0 = fmaf(sm.o[w][r][c], f, o0);
      o1 = fmaf(sm.o[w][r][c + 1], f, o1);
    }
    if (sm.nan_first[c] < sm.lim[r]) o0 = __int_as_float(0x7fffffff);
    if (sm.nan_first[c + 1] < sm.lim[r]) o1 = __int_as_float(0x7fffffff);
    if (slot >= 0) {
      *reinterpret_cast<float2 *>(a.part + (int64_t(slot) * kRows + r) * D + c) = make_float2(o0, o1);
      if (c == 0) a.part_ml[slot * kRows + r] = make_float2(M, l);
    } else {
      const float f = l == 0.0f ? 0.0f : 1.0f / l;  // no visible token: the row is 0
      const int R = rg * kRows + r;
      const int64_t at = (sq.start + R / a.group) * a.ld_out + int64_t(h * a.group + R % a.group) * D + c;
      if (a.out_fp32)
        *reinterpret_cast<float2 *>(static_cast<float *>(a.out) + at) = make_float2(o0 * f, o1 * f);
      else
        *reinterpret_cast<__nv_bfloat162 *>(static_cast<uint16_t *>(a.out) + at) = __floats2bfloat162_rn(o0 * f, o1 * f);
    }
  }
  __syncthreads();  // sm is used again by the next segment
}

template <int D>
__global__ void __launch_bounds__(kThreads) decode_kernel(const __grid_constant__ Args a) {
  __shared__ DecodeSmem<D> sm;
  grid_dep_wait();
  grid_dep_launch();

  // Total work.
  int64_t total = 0, total_u = 0;
  for (int s0 = 0; s0 < a.n_seqs; s0 += kThreads) {
    int tiles = 0, units = 0;
    const int s = s0 + threadIdx.x;
    if (s < a.n_seqs) {
      const Seq q = load_seq(a, s);
      if (!q.ok && blockIdx.x == 0) record_bad_index();
      seq_work<D>(a, q, tiles, units);
    }
    int64_t t = int64_t(tiles) * units, u = units;
    block_scan(t, u, sm.scan_t, sm.scan_u);
    if (threadIdx.x == kThreads - 1) {
      sm.base_t = t;
      sm.base_u = u;
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
  int64_t before_t = 0, before_u = 0;
  int seq = 0;
  for (int s0 = 0; s0 < a.n_seqs; s0 += kThreads) {
    int tiles = 0, units = 0;
    const int s = s0 + threadIdx.x;
    if (s < a.n_seqs) seq_work<D>(a, load_seq(a, s), tiles, units);
    const int64_t mine = int64_t(tiles) * units;
    int64_t t = mine, u = units;
    if (threadIdx.x == 0) sm.found = -1;
    block_scan(t, u, sm.scan_t, sm.scan_u);
    if (before_t + t > begin && before_t + t - mine <= begin) {
      sm.found = s;
      sm.base_t = before_t + t - mine;
      sm.base_u = before_u + u - units;
    }
    __syncthreads();
    if (sm.found >= 0) {
      seq = sm.found;
      before_t = sm.base_t;
      before_u = sm.base_u;
      break;
    }
    if (threadIdx.x == kThreads - 1) {
      sm.base_t = before_t + t;
      sm.base_u = before_u + u;
    }
    __syncthreads();
    before_t = sm.base_t;
    before_u = sm.base_u;
    __syncthreads();
  }
  __syncthreads();

  int64_t at = begin;
  Seq sq = load_seq(a, seq);
  int tiles, units;
  seq_work<D>(a, sq, tiles, units);
  while (at < end) {
    while (at >= before_t + int64_t(tiles) * units) {  // next sequence with work
      before_t += int64_t(tiles) * units;
      before_u += units;
      if (++seq >= a.n_seqs) return;
      sq = load_seq(a, seq);
      seq_work<D>(a, sq, tiles, units);
    }
    const int64_t local = at - before_t;
    const int unit = static_cast<int>(local / tiles), tile0 = static_cast<int>(local - int64_t(unit) * tiles);
    const int ntile = static_cast<int>(min(int64_t(tiles - tile0), end - at));
    const int h = unit % a.kv_heads, rg = unit / a.kv_heads;
    const bool whole = ntile == tiles;
    if (tile0 == 0 && threadIdx.x == 0) {
      const int64_t last = before_t + int64_t(unit + 1) * tiles - 1;
      a.desc[before_u + unit] = make_int4(seq, h, rg, 0);
      a.desc2[before_u + unit] = make_int2(blockIdx.x, static_cast<int>(((last + 1) * ctas - 1) / total));
    }
    decode_segment<D>(a, sm, sq, seq, h, rg, tile0, ntile, whole ? -1 : 2 * int(blockIdx.x) + (tile0 == 0));
    at += ntile;
  }
}

// Joins the partial results of the units that several CTAs share.  Grid (units, kRows),
// D / 2 threads: one query row, two values per thread.
template <int D>
__global__ void __launch_bounds__(D / 2) combine_kernel(const __grid_constant__ Args a) {
  grid_dep_wait();
  grid_dep_launch();
  if (int(blockIdx.x) >= *a.n_units) return;
  const int2 c = a.desc2[blockIdx.x];
  if (c.x == c.y) return;  // one CTA wrote the result
  const int4 u = a.desc[blockIdx.x];
  const Seq sq = load_seq(a, u.x);
  const int r = blockIdx.y, R = u.z * kRows + r;
  if (R >= sq.q_len * a.group) return;
  // the first CTA's partial is its last segment, the others' their first
  auto slot = [&](int i) { return int64_t(2 * i + (i == c.x)) * kRows + r; };
  float M = -INFINITY;
  for (int i = c.x; i <= c.y; ++i) M = fmaxf(M, a.part_ml[slot(i)].x);
  const float base = M == -INFINITY ? 0.0f : M;
  float l = 0.0f, o0 = 0.0f, o1 = 0.0f;
#pragma unroll 4
  for (int i = c.x; i <= c.y; ++i) {
    const int64_t at = slot(i);
    const float2 ml = a.part_ml[at];
    const float2 o = *reinterpret_cast<const float2 *>(a.part + at * D + 2 * threadIdx.x);
    const float f = ex2(ml.x - base);
    l = fmaf(ml.y, f, l);
    o0 = fmaf(o.x, f, o0);
    o1 = fmaf(o.y, f, o1);
  }
  const float f = l == 0.0f ? 0.0f : 1.0f / l;
  const int64_t at = (sq.start + R / a.group) * a.ld_out + int64_t(u.y * a.group + R % a.group) * D + 2 * threadIdx.x;
  if (a.out_fp32)
    *reinterpret_cast<float2 *>(static_cast<float *>(a.out) + at) = make_float2(o0 * f, o1 * f);
  else
    *reinterpret_cast<__nv_bfloat162 *>(static_cast<uint16_t *>(a.out) + at) = __floats2bfloat162_rn(o0 * f, o1 * f);
}

}  // namespace attn
}  // namespace nvfp4

// Attention over the block-scaled 8-bit cache for prompts: the mathematics of
// attn_decode.cuh on tcgen05 with tiles of 128 query rows.
//
// A query row is one head of one token; the rows of a kv head's group are numbered token by
// token, so 128 rows of a tile share every cached byte.  K and V codes are exact in FP16:
// converter warps turn a tile of codes into FP16 in shared memory (rows of tokens in panels of
// 64 values, 128-byte swizzle), where K is a K-major and V, in the same layout, an MN-major
// operand.  S = Q K^T accumulates in TMEM; a softmax warpgroup reads it one row per thread,
// writes P over it as FP16, and O += P V takes P from TMEM.  O stays in TMEM and is rescaled
// only when a row's maximum has grown by more than 2^kSlack since its reference was set
// (weights are at most 2^(kSlack + kBoost), within FP16).
//
// Two streams keep the tensor cores busy while the other's softmax runs.  Up to 128 values per
// head they are two tiles of query rows with their own O over the same K / V tiles of 128
// tokens; at 256 values TMEM holds one O, and the streams are the even and odd K / V tiles of
// 64 tokens, which hand the rows' reference maxima to each other.
//
// Warps (one CTA per SM): 0-3 and 4-7 softmax of stream 0 and 1, 8-11 K converters,
// 12-15 V converters, 16 MMA issuer.
#pragma once

#include "attn_decode.cuh"

namespace nvfp4 {
namespace attn {
namespace prompt {

constexpr int kThreads = 544;
constexpr int kTile = 128;      // query rows of a tile
constexpr float kSlack = 8.0f;
constexpr float kBoostP = 6.0f;

template <int D>
struct Cfg {
  static constexpr bool kSplitKV = D == 256;           // streams are K / V tiles, not row tiles
  static constexpr int NQ = kSplitKV ? 1 : 2;
  static constexpr int BN = kSplitKV ? 64 : 128;       // cached tokens of a tile
  static constexpr int PANELS = D / 64;
  static constexpr int Q_BYTES = NQ * kTile * D * 2;
  static constexpr int KV_BYTES = BN * D * 2;
  static constexpr int STAGES = 2;
  static constexpr int GROUPS = BN / kGroup;
  static constexpr int CPR = D / 16;                   // 16-byte pieces of a row of codes
  static constexpr int PIECES = BN * CPR / 128;        // per converter thread
  static constexpr int ROWS = NQ * kTile;
  static constexpr int S_COL = BN;                     // TMEM columns of one S
  static constexpr int O_COL0 = 256;
};

struct Scales {
  float k, log_v, inv_v, pad;
};

template <int D>
struct Control {
  uint64_t q_ready, k_full[2], k_empty[2], v_full[2], v_empty[2], s_ready[2], p_ready[2], o_done[2], m_ready[2], join, done;
  uint32_t tmem;
  int nan_any;
  // A tile's scales, written with its K.  Its slot comes up again four tiles later, when the
  // products with the earlier tile's weights have been issued: its readers are done.
  Scales ks[4][Cfg<D>::GROUPS];
  int nan_first[D];
  float m_ref[kTile];            // kSplitKV: reference maxima of the rows
  float l[2][kTile];
};

template <int D>
constexpr int smem_bytes() {
  return 1024 + Cfg<D>::Q_BYTES + 2 * Cfg<D>::STAGES * Cfg<D>::KV_BYTES + int(sizeof(Control<D>));
}

__host__ __device__ constexpr uint32_t idesc_f16(int m, int n, bool b_mn_major) {
  return (1u << 4) | (b_mn_major ? 1u << 16 : 0u) | (uint32_t(n >> 3) << 17) | (uint32_t(m >> 4) << 24);
}

// FP16 MMA with FP32 accumulation, A from shared memory / from TMEM.
__device__ __forceinline__ void mma_f16_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t a_tmem, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a_tmem), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}

// MN-major operand of 64-value panels (128-byte rows, one per contraction index, 128-byte
// swizzle): panels `panel_bytes` apart, 8-row groups 1024 bytes apart.
__device__ __forceinline__ uint64_t sdesc_sw128_mnmajor(uint32_t saddr, uint32_t panel_bytes) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr >> 4) & 0x3FFF);
  d |= (uint64_t)(panel_bytes >> 4) << 16;
  d |= (uint64_t)(1024 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

__device__ __forceinline__ void tmem_st_32x32b_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st_32x32b_x32(uint32_t taddr, const uint32_t (&r)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
      "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Generic-proxy writes to shared memory become visible to the tensor cores.
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// 16-byte piece `c` (of 8) of row `r` of panel `p`, a panel holding `rows` rows.
__device__ __forceinline__ uint32_t panel_offset(int rows, int p, int r, int c) {
  return (p * rows + r) * 128 + ((c ^ (r & 7)) << 4);
}

// What a CTA works on.
struct Item {
  Seq sq;
  int seq, h, row0;  // first query row of its tiles
  int kv_end;        // cached tokens that some row sees
  int lim_min;       // tokens that every row sees
};

// Finds the CTA's work: items of a sequence are (row block, kv head), the row blocks with
// the most visible tokens first.  Returns false when there is none.
template <int D>
__device__ bool find_item(const Args &a, Item &it) {
  using C = Cfg<D>;
  __shared__ int64_t s_sum[kThreads / 32], s_before;
  __shared__ int s_seq;
  int64_t base = 0;
  for (int s0 = 0; s0 < a.n_seqs; s0 += kThreads) {
    const int s = s0 + threadIdx.x;
    int64_t items = 0;
    if (s < a.n_seqs) {
      const Seq q = load_seq(a, s);
      const int64_t rows = int64_t(q.q_len) * a.group;
      if (rows > a.max_decode_rows) items = (rows + C::ROWS - 1) / C::ROWS * a.kv_heads;
    }
    int64_t sum = items;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(0xffffffffu, sum, o);
      if ((threadIdx.x & 31) >= o) sum += x;
    }
    if (threadIdx.x == 0) s_seq = -1;
    if ((threadIdx.x & 31) == 31) s_sum[threadIdx.x >> 5] = sum;
    __syncthreads();
    int64_t all = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < int(threadIdx.x >> 5)) sum += s_sum[w];
      all += s_sum[w];
    }
    if (int64_t(blockIdx.x) < base + sum && int64_t(blockIdx.x) >= base + sum - items) {
      s_seq = s;
      s_before = base + sum - items;
    }
    __syncthreads();
    if (s_seq >= 0) {
      const int local = static_cast<int>(blockIdx.x - s_before);
      it.seq = s_seq;
      it.sq = load_seq(a, it.seq);
      const int rows = it.sq.q_len * a.group;
      const int blocks = (rows + C::ROWS - 1) / C::ROWS;
      it.h = local % a.kv_heads;
      it.row0 = (blocks - 1 - local / a.kv_heads) * C::ROWS;
      const int last = min(it.row0 + C::ROWS, rows) - 1;
      const int off = it.sq.kv_len - it.sq.q_len + 1;
      it.kv_end = a.causal ? max(0, off + last / a.group) : it.sq.kv_len;
      it.lim_min = a.causal ? max(0, off + it.row0 / a.group) : it.sq.kv_len;
      return true;
    }
    base += all;
    __syncthreads();
  }
  return false;
}

// Converter warpgroup (tid 0..127) of K or of V.
template <int D, bool V>
__device__ void convert(const Args &a, Control<D> &c, unsigned char *buf, const Item &it, int n_tiles, int tid) {
  using C = Cfg<D>;
  const int lane = tid & 31;
  const uint8_t *src = V ? a.v : a.k;
  // lane i < GROUPS of every warp knows the (block, head) index of the tile's group i
  auto blocks_of = [&](int j) -> int64_t {
    if (j >= n_tiles || lane >= C::GROUPS) return -1;
    return group_block<D>(a, it.seq, it.h, j * C::BN + lane * kGroup, it.kv_end);
  };
  uint4 raw[C::PIECES];
  auto load = [&](int j, int64_t blk) {
#pragma unroll
    for (int i = 0; i < C::PIECES; ++i) {
      const int p = tid + 128 * i, row = p / C::CPR, col = p % C::CPR;
      const int64_t b = __shfl_sync(0xffffffffu, blk, row / kGroup);
      const int tok = j * C::BN + row;
      raw[i] = make_uint4(0, 0, 0, 0);
      if (b >= 0 && tok < it.kv_end)
        raw[i] = ld_stream(src + ((b << a.log_block) + (tok & ((1 << a.log_block) - 1))) * D + 16 * col);
    }
  };
  int64_t blk = blocks_of(0);
  load(0, blk);
  int64_t next = blocks_of(1);
  for (int j = 0; j < n_tiles; ++j) {
    const int st = j & 1;
    if (!mbar_wait(V ? &c.v_empty[st] : &c.k_empty[st], ((j >> 1) & 1) ^ 1)) return;
    if (!V && tid < C::GROUPS) {  // tid == lane here
      Scales s;
      s.k = blk >= 0 ? __ldg(a.k_scales + blk) : 0.0f;
      s.log_v = blk >= 0 ? log_scale(__ldg(a.v_scales + blk)) : -INFINITY;  // no such block: nothing to see
      s.inv_v = blk >= 0 ? exp2f(-s.log_v) : 0.0f;
      s.pad = 0.0f;
      c.ks[j & 3][tid] = s;
    }
    unsigned char *dst = buf + st * C::KV_BYTES;
    const bool partial = V && (j + 1) * C::BN > it.lim_min;
#pragma unroll
    for (int i = 0; i < C::PIECES; ++i) {
      const int p = tid + 128 * i, row = p / C::CPR, col = p % C::CPR;
      uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
      if (partial) {  // a NaN that some rows must not see: see decode_segment
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (((w[k] & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u)
            for (int b = 0; b < 4; ++b)
              if (((w[k] >> (8 * b)) & 0x7f) == 0x7f) {
                atomicMin(&c.nan_first[16 * col + 4 * k + b], j * C::BN + row);
                c.nan_any = 1;
                w[k] &= ~(0xffu << (8 * b));
              }
      }
      uint4 h[2];
      h[0] = make_uint4(e4m3x2_to_f16x2(w[0]), e4m3x2_to_f16x2(w[0] >> 16), e4m3x2_to_f16x2(w[1]), e4m3x2_to_f16x2(w[1] >> 16));
      h[1] = make_uint4(e4m3x2_to_f16x2(w[2]), e4m3x2_to_f16x2(w[2] >> 16), e4m3x2_to_f16x2(w[3]), e4m3x2_to_f16x2(w[3] >> 16));
      // the odd piece first in every other panel: eight lanes then hit distinct banks
      const int o = (col >> 2) & 1;
      *reinterpret_cast<uint4 *>(dst + panel_offset(C::BN, col >> 2, row, 2 * (col & 3) + o)) = o ? h[1] : h[0];
      *reinterpret_cast<uint4 *>(dst + panel_offset(C::BN, col >> 2, row, 2 * (col & 3) + (o ^ 1))) = o ? h[0] : h[1];
    }
    fence_async_smem();
    mbar_arrive(V ? &c.v_full[st] : &c.k_full[st]);
    blk = next;
    load(j + 1, blk);
    next = blocks_of(j + 2);
  }
}

// MMA issuer (one thread).
template <int D>
__device__ void issue(Control<D> &c, uint32_t tmem, uint32_t q, uint32_t k, uint32_t v, int n_tiles) {
  using C = Cfg<D>;
  constexpr uint32_t kIdescS = idesc_f16(kTile, C::BN, false), kIdescO = idesc_f16(kTile, D, true);
  auto qk = [&](int w, int j) {  // stream w's S = Q K_j^T
    const uint32_t qa = q + (C::kSplitKV ? 0 : w * kTile * D * 2), ka = k + (j & 1) * C::KV_BYTES;
#pragma unroll
    for (int p = 0; p < C::PANELS; ++p) {
      const uint64_t ad = sdesc_sw128_kmajor(qa + p * kTile * 128), bd = sdesc_sw128_kmajor(ka + p * C::BN * 128);
#pragma unroll
      for (int s = 0; s < 4; ++s) mma_f16_ss(tmem + w * C::S_COL, ad + 2 * s, bd + 2 * s, kIdescS, (p | s) != 0);
    }
    tc_commit(&c.s_ready[w]);
  };
  auto pv = [&](int w, int j) {  // O += P V_j
    const uint32_t va = v + (j & 1) * C::KV_BYTES;
    const uint32_t o = tmem + C::O_COL0 + (C::kSplitKV ? 0 : w * D);
#pragma unroll
    for (int s = 0; s < C::BN / 16; ++s)
      mma_f16_ts(o, tmem + w * C::S_COL + 8 * s, sdesc_sw128_mnmajor(va + s * 2048, C::BN * 128), kIdescO, (j | s) != 0);
    tc_commit(&c.o_done[w]);
  };
  auto full = [&](uint64_t *b, int j) { return mbar_wait(&b[j & 1], (j >> 1) & 1); };

  if (!mbar_wait(&c.q_ready, 0)) return;
  if constexpr (!C::kSplitKV) {
    if (!full(c.k_full, 0)) return;
    tc_fence_after();
    qk(0, 0);
    qk(1, 0);
    tc_commit(&c.k_empty[0]);
    for (int j = 0; j < n_tiles; ++j) {
      if (!full(c.v_full, j)) return;
#pragma unroll
      for (int w = 0; w < 2; ++w) {
        if (!mbar_wait(&c.p_ready[w], j & 1)) return;
        tc_fence_after();
        pv(w, j);
        if (w == 1) tc_commit(&c.v_empty[j & 1]);
        if (j + 1 < n_tiles) {
          if (w == 0 && !full(c.k_full, j + 1)) return;
          tc_fence_after();
          qk(w, j + 1);
          if (w == 1) tc_commit(&c.k_empty[(j + 1) & 1]);
        }
      }
    }
  } else {
    for (int j = 0; j < 2 && j < n_tiles; ++j) {
      if (!full(c.k_full, j)) return;
      tc_fence_after();
      qk(j, j);
      tc_commit(&c.k_empty[j]);
    }
    for (int j = 0; j < n_tiles; ++j) {
      const int w = j & 1;
      if (!full(c.v_full, j) || !mbar_wait(&c.p_ready[w], (j >> 1) & 1)) return;
      tc_fence_after();
      pv(w, j);
      tc_commit(&c.v_empty[w]);
      if (j + 2 < n_tiles) {
        if (!full(c.k_full, j + 2)) return;
        tc_fence_after();
        qk(w, j + 2);
        tc_commit(&c.k_empty[w]);
      }
    }
  }
}

// Multiplies columns [0, n) of the thread's O row by f.
template <int N>
__device__ __forceinline__ void scale_o(uint32_t o, float f) {
#pragma unroll 1
  for (int c0 = 0; c0 < N; c0 += 32) {
    uint32_t r[32];
    tmem_ld_32x32b_x32(o + c0, r);
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * f);
    tmem_st_32x32b_x32(o + c0, r);
  }
  tmem_st_wait();
}

// Softmax warpgroup of stream w; tid 0..127 is the row of its tile.
template <int D>
__device__ void softmax(const Args &a, Control<D> &c, uint32_t tmem, unsigned char *qbuf, const Item &it, int n_tiles,
                        int w, int tid) {
  using C = Cfg<D>;
  const int n_rows = it.sq.q_len * a.group;
  const int R = it.row0 + (C::kSplitKV ? 0 : w * kTile) + tid;
  const bool valid = R < n_rows;
  const int tok = valid ? R / a.group : 0, head = it.h * a.group + (valid ? R % a.group : 0);
  const int lim = !valid ? it.kv_end : a.causal ? it.sq.kv_len - it.sq.q_len + tok + 1 : it.sq.kv_len;
  const int warp_lim = __reduce_min_sync(0xffffffffu, lim);

  // This thread's Q row as FP16, scaled by 2^-e (both streams of kSplitKV need e; the second
  // writes half of the row).
  float rc;
  {
    const uint16_t *src = a.q + (it.sq.start + tok) * a.ld_q + int64_t(head) * D;
    float amax = 0.0f;
#pragma unroll 4
    for (int i = 0; i < D / 8; ++i) {
      const uint4 x = __ldg(reinterpret_cast<const uint4 *>(src) + i);
      const uint32_t v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int n = 0; n < 4; ++n)
        amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(v[n] << 16)), fabsf(__uint_as_float(v[n] & 0xFFFF0000u))));
    }
    const int e = valid ? row_exponent(amax) : 0;
    const float f0 = valid ? ldexpf(a.scale_log2 < 0.0f ? -1.0f : 1.0f, -(e / 2)) : 0.0f, f1 = ldexpf(1.0f, -(e - e / 2));
    rc = ldexpf(fabsf(a.scale_log2), e);
    unsigned char *q = qbuf + (C::kSplitKV ? 0 : w * kTile * D * 2);
    constexpr int kHalf = C::kSplitKV ? D / 16 : D / 8;
    const int first = C::kSplitKV ? w * kHalf : 0;
#pragma unroll 4
    for (int i = first; i < first + kHalf; ++i) {
      const uint4 x = valid ? __ldg(reinterpret_cast<const uint4 *>(src) + i) : make_uint4(0, 0, 0, 0);
      const uint32_t v[4] = {x.x, x.y, x.z, x.w};
      uint32_t o[4];
#pragma unroll
      for (int n = 0; n < 4; ++n)
        o[n] = pack_f16(__uint_as_float(v[n] << 16) * f0 * f1, __uint_as_float(v[n] & 0xFFFF0000u) * f0 * f1);
      *reinterpret_cast<uint4 *>(q + panel_offset(kTile, i >> 3, tid, i & 7)) = make_uint4(o[0], o[1], o[2], o[3]);
    }
    fence_async_smem();
    mbar_arrive(&c.q_ready);
  }

  const uint32_t lanes = (tid & ~31) << 16;  // TMEM lane quadrant of the warp
  const uint32_t s_tmem = tmem + lanes + w * C::S_COL, o_tmem = tmem + lanes + C::O_COL0 + (C::kSplitKV ? 0 : w * D);
  float m_ref = -INFINITY, l = 0.0f;
  const int steps = C::kSplitKV ? (n_tiles - w + 1) / 2 : n_tiles;
  for (int i = 0; i < steps; ++i) {
    const int j = C::kSplitKV ? 2 * i + w : i;
    if (!mbar_wait(&c.s_ready[w], i & 1)) return;
    tc_fence_after();
    const Scales *sc = c.ks[j & 3];
    const int vis = lim - j * C::BN;  // visible columns of this row
    const bool masked = warp_lim < (j + 1) * C::BN;

    // maximum of x = s c + e over the row
    float mt = -INFINITY;
#pragma unroll
    for (int c0 = 0; c0 < C::BN; c0 += 32) {
      uint32_t r[32];
      tmem_ld_32x32b_x32(s_tmem + c0, r);
      tmem_ld_wait();
      if (masked) {
#pragma unroll
        for (int n = 0; n < 32; ++n)
          if (c0 + n >= vis) r[n] = 0xff800000u;
      }
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        float x = -INFINITY;
#pragma unroll
        for (int n = 0; n < 16; ++n) x = fmaxf(x, __uint_as_float(r[16 * g + n]));
        const Scales s = sc[c0 / 16 + g];
        mt = fmaxf(mt, x == -INFINITY ? x : fmaf(x, s.k * rc, s.log_v));
      }
    }

    if constexpr (C::kSplitKV) {
      if (j > 0) {
        if (!mbar_wait(&c.m_ready[w ^ 1], w == 1 ? i & 1 : (i - 1) & 1)) return;
        const float m = c.m_ref[tid];
        if (m != m_ref) l *= m_ref == -INFINITY ? 0.0f : ex2(m_ref - m);
        m_ref = m;
      }
    }
    const bool grow = mt > m_ref + kSlack || (m_ref == -INFINITY && mt > m_ref);
    if (__any_sync(0xffffffffu, grow)) {
      const float f = grow ? ex2(m_ref - mt) : 1.0f;
      if (grow) {
        l *= f;
        m_ref = mt;
      }
      if (j > 0) {  // O holds the earlier tiles: it may be touched once their products are in
        // S_j was issued after the products of this stream's previous tile, so only the
        // latest phase can be open
        if (!mbar_wait(&c.o_done[C::kSplitKV ? w ^ 1 : w], (C::kSplitKV ? (j - 1) >> 1 : j - 1) & 1)) return;
        tc_fence_after();
        scale_o<D>(o_tmem, f);
      }
    }
    if constexpr (C::kSplitKV) {
      c.m_ref[tid] = m_ref;
      mbar_arrive(&c.m_ready[w]);
    }

    const float base = (m_ref == -INFINITY ? 0.0f : m_ref) - kBoostP;
#pragma unroll
    for (int c0 = 0; c0 < C::BN; c0 += 32) {
      uint32_t r[32], p[16];
      tmem_ld_32x32b_x32(s_tmem + c0, r);
      tmem_ld_wait();
#pragma unroll
      for (int g = 0; g < 2; ++g) {
        const Scales s = sc[c0 / 16 + g];
        const float ck = s.k * rc, ce = s.log_v - base;
        float sum = 0.0f;
#pragma unroll
        for (int n = 0; n < 16; n += 2) {
          float x0 = fmaf(__uint_as_float(r[16 * g + n]), ck, ce), x1 = fmaf(__uint_as_float(r[16 * g + n + 1]), ck, ce);
          if (masked) {
            if (c0 + 16 * g + n >= vis) x0 = -INFINITY;
            if (c0 + 16 * g + n + 1 >= vis) x1 = -INFINITY;
          }
          x0 = ex2(x0);
          x1 = ex2(x1);
          sum += x0 + x1;
          p[8 * g + n / 2] = pack_f16(x0, x1);
        }
        l = fmaf(sum, s.inv_v, l);
      }
      tmem_st_32x32b_x16(s_tmem + c0 / 2, p);
    }
    tmem_st_wait();
    tc_fence_before();
    __syncwarp();
    if ((tid & 31) == 0) mbar_arrive(&c.p_ready[w]);
  }

  // Epilogue: O / l.
  if constexpr (C::kSplitKV) {
    mbar_arrive(&c.join);
    if (!mbar_wait(&c.join, 0)) return;
    const float m = c.m_ref[tid];  // the last tile's reference; l is relative to the one seen last
    if (m != m_ref && m_ref != -INFINITY) l *= ex2(m_ref - m);
    c.l[w][tid] = l;
    mbar_arrive(&c.join);
    if (!mbar_wait(&c.join, 1)) return;
    l = c.l[0][tid] + c.l[1][tid];
  }
  // the last products of each stream that adds to this O
  if constexpr (C::kSplitKV) {
    if (!mbar_wait(&c.o_done[0], ((n_tiles - 1) >> 1) & 1)) return;
    if (n_tiles > 1 && !mbar_wait(&c.o_done[1], ((n_tiles >> 1) - 1) & 1)) return;
  } else {
    if (!mbar_wait(&c.o_done[w], (n_tiles - 1) & 1)) return;
  }
  tc_fence_after();
  const float f = l == 0.0f ? 0.0f : 1.0f / l;
  constexpr int kCols = C::kSplitKV ? D / 2 : D;
  const int col0 = C::kSplitKV ? w * kCols : 0;
  const int64_t at = (it.sq.start + tok) * a.ld_out + int64_t(head) * D;
  const bool nan_any = *const_cast<volatile int *>(&c.nan_any) != 0;
#pragma unroll 1
  for (int c0 = col0; c0 < col0 + kCols; c0 += 32) {
    uint32_t r[32];
    tmem_ld_32x32b_x32(o_tmem + c0, r);
    tmem_ld_wait();
#pragma unroll
    for (int n = 0; n < 32; ++n) {
      r[n] = __float_as_uint(l == 0.0f ? 0.0f : __uint_as_float(r[n]) * f);
      if (nan_any && c.nan_first[c0 + n] < lim) r[n] = 0x7fffffffu;
    }
    if (!valid) continue;
    if (a.out_fp32) {
      uint4 *dst = reinterpret_cast<uint4 *>(static_cast<float *>(a.out) + at + c0);
#pragma unroll
      for (int n = 0; n < 8; ++n) dst[n] = make_uint4(r[4 * n], r[4 * n + 1], r[4 * n + 2], r[4 * n + 3]);
    } else {
      uint4 *dst = reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out) + at + c0);
#pragma unroll
      for (int n = 0; n < 4; ++n) {
        uint32_t o[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const __nv_bfloat162 b = __floats2bfloat162_rn(__uint_as_float(r[8 * n + 2 * k]), __uint_as_float(r[8 * n + 2 * k + 1]));
          o[k] = *reinterpret_cast<const uint32_t *>(&b);
        }
        dst[n] = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  }
}

// Grid: an upper bound of the items; dynamic shared memory smem_bytes<D>().
template <int D>
__global__ void __launch_bounds__(kThreads, 1) prompt_kernel(const __grid_constant__ Args a) {
  using C = Cfg<D>;
  extern __shared__ unsigned char smem_raw[];
  grid_dep_wait();
  grid_dep_launch();
  Item it;
  if (!find_item<D>(a, it)) return;
  const int tid = threadIdx.x, warp = tid >> 5;
  if (it.kv_end == 0) {  // no row sees a token
    const int n_rows = it.sq.q_len * a.group;
    for (int r = it.row0 + warp; r < min(it.row0 + C::ROWS, n_rows); r += kThreads / 32) {
      const int64_t at = (it.sq.start + r / a.group) * a.ld_out + int64_t(it.h * a.group + r % a.group) * D;
      for (int i = tid & 31; i < D; i += 32) {
        if (a.out_fp32) static_cast<float *>(a.out)[at + i] = 0.0f;
        else static_cast<uint16_t *>(a.out)[at + i] = 0;
      }
    }
    return;
  }
  const int n_tiles = (it.kv_end + C::BN - 1) / C::BN;
  unsigned char *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  unsigned char *qbuf = smem, *kbuf = qbuf + C::Q_BYTES, *vbuf = kbuf + C::STAGES * C::KV_BYTES;
  Control<D> &c = *reinterpret_cast<Control<D> *>(vbuf + C::STAGES * C::KV_BYTES);
  if (tid == 0) {
    mbar_init(&c.q_ready, 256);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&c.k_full[i], 128);
      mbar_init(&c.v_full[i], 128);
      mbar_init(&c.k_empty[i], 1);
      mbar_init(&c.v_empty[i], 1);
      mbar_init(&c.s_ready[i], 1);
      mbar_init(&c.p_ready[i], 4);
      mbar_init(&c.o_done[i], 1);
      mbar_init(&c.m_ready[i], 128);
    }
    mbar_init(&c.join, 256);
    mbar_init(&c.done, 1);
    fence_barrier_init();
    c.nan_any = 0;
  }
  for (int i = tid; i < D; i += kThreads) c.nan_first[i] = 0x7fffffff;
  if (warp == 16) {
    tmem_alloc(&c.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = c.tmem;

  if (warp < 8) {
    softmax<D>(a, c, tmem, qbuf, it, n_tiles, warp >> 2, tid & 127);
  } else if (warp < 12) {
    convert<D, false>(a, c, kbuf, it, n_tiles, tid & 127);
  } else if (warp < 16) {
    convert<D, true>(a, c, vbuf, it, n_tiles, tid & 127);
  } else if ((tid & 31) == 0) {
    issue<D>(c, tmem, smem_u32(qbuf), smem_u32(kbuf), smem_u32(vbuf), n_tiles);
    tc_commit(&c.done);  // whatever was issued has to end before TMEM is given back
    mbar_wait(&c.done, 0);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 16) tmem_dealloc(tmem, 512);
}

}  // namespace prompt
}  // namespace attn
}  // namespace nvfp4

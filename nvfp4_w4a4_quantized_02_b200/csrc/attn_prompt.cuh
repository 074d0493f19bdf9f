// Attention over the block-scaled 8-bit cache for prompts: the mathematics of
// attn_decode.cuh on tcgen05 with tiles of 128 query rows.
//
// A query row is one head of one token; the rows of a kv head's group are numbered token by
// token, so 128 rows of a tile share every cached byte.
//  * S = Q K^T runs on the codes themselves: K goes by TMA straight into its operand layout,
//    and q, scaled by a power of two per row, is the sum of two E4M3 parts, hi = E4M3(q) and
//    lo = E4M3(q - hi).  A BF16 value has 8 significant bits and each part holds 4, so the sum is exact
//    down to 2^-10 of the row's largest value, and below within half of E4M3's smallest step, 2^-17 of it.
//    Two FP8 products cost what one in FP16 would, and K needs no conversion.
//  * O += P V runs in FP16, since P needs more than 8 bits of range and precision (11 bits down to 2^-20 of
//    the row's reference, below that to within 2^-31 of it): converter
//    warps load V codes (exact in FP16) and write panels of 64 values with 128-byte swizzle, token
//    rows, which the product reads as an MN-major operand.
// S accumulates in TMEM; a softmax thread reads a row of it and writes P over it as FP16, the A
// operand of O += P V.  Weights are taken relative to a reference per row, 2^kBoostP at the
// reference, which stays as it is while the weights fit FP16: a tile costs one pass over S, and the sum
// of its weights tells whether they did (a sum below FP16's largest value holds none above it).  When
// they did not (and at the first tile) the row's maximum becomes its reference, O, which stays in
// TMEM, is rescaled and the tile's weights are taken again.
//
// Two streams keep the tensor cores busy while the other's softmax runs.  Up to 128 values per
// head they are two tiles of query rows with their own O over the same K / V tiles; at 256 values TMEM
// holds one O, and the streams are the even and odd K / V tiles, which hand the rows' references to
// each other.
//
// Bounds.  Per tile of 128 tokens and stream, at 128 (256) values: the tensor cores 1024 (2048) cycles;
// shared memory, which an SM reads and writes at 128 bytes per cycle, 1024 (2304): the products read
// 64 (128) KB for S and 32 (64) KB for P V, the converters write 16 (64), the TMA 8 (32); the MUFU 1024
// (1024) for the exponentials.  A product of 128 x 128 x 32 bytes takes 64 cycles, and a warp needs about
// 55 to issue one with its descriptors ready (75 if it computes them).
//
// Measured (TFLOP/s at 4 D per visible pair).  8192 tokens, 48 + 8 heads of 128: 787 to 802 us, 1030 TFLOP/s
// (call after call, at the power cap, 890 us, 930), about 3600 cycles for a tile of both streams
// against the tensor cores' 2048; what is left is a stream's chain S -> exponentials -> P V, which one other
// stream does not cover.  1024 tokens on 32768, 24 + 4 heads of 256: 737 to 817 us, 990 to 1100 TFLOP/s
// (872 us, 930); there the products with K leave the converters little of shared memory (with time stamps
// in the kernel the MMA warp waits for V half of the time).
//
// Warps (one CTA per SM): 0 MMA issuer, 1 producer (block table, scales, K copies), 2-3 idle, 4-7 and
// 8-11 softmax of stream 0 and 1, 12-19 V converters.  Registers are handed from the others to the
// softmax.
#pragma once

#include "attn_decode.cuh"
#include "gdn.cuh"

namespace nvfp4 {
namespace attn {
namespace prompt {

constexpr int kThreads = 640;
constexpr int kSoftmax = 256;    // softmax threads
constexpr int kConverters = 256;
constexpr int kRegsLaunch = 65536 / kThreads / 8 * 8;  // registers per thread at launch
constexpr int kTile = 128;      // query rows of a tile
constexpr float kMostSum = 60000.0f;  // weights whose sum is below this are within FP16
constexpr float kBoostP = 6.0f;  // the sum may be 937 times the reference's weight; smallest normal weight 2^-20 of it

template <int D>
struct Cfg {
  static constexpr bool kSplitKV = D == 256;           // streams are K / V tiles, not row tiles
  static constexpr int NQ = kSplitKV ? 1 : 2;
  static constexpr int BN = 128;                       // cached tokens of a tile
  static constexpr int VT = kSplitKV ? 64 : 128;       // tokens of a V stage
  static constexpr int VSUB = BN / VT;
  static constexpr int ROWB = D < 128 ? D : 128;       // bytes of a row of a panel of codes
  static constexpr int PANELS8 = D / ROWB;             // panels of codes
  static constexpr int Q_PART = kTile * D;             // one part of one query tile
  static constexpr int Q_BYTES = NQ * 2 * Q_PART;
  static constexpr int K_BYTES = BN * D;
  static constexpr int V_BYTES = VT * D * 2;
  static constexpr int K_STAGES = kSplitKV ? 2 : 3;
  static constexpr int GROUPS = BN / kGroup;
  static constexpr int LOG_BOX = 7;                    // rows of a TMA box at most: a tile
  static constexpr int CPR = D / 16;                   // 16-byte pieces of a row of codes
  static constexpr int TURNS = kSplitKV ? 2 : 1;       // groups of converter warps that take V stages in turn
  static constexpr int PER_V = kConverters / TURNS;    // converter threads of a V stage
  static constexpr int PIECES = VT * CPR / PER_V;      // 16-byte pieces of each
  static constexpr int ROWS = NQ * kTile;
  static constexpr int O_COL0 = 256;
  // Registers per thread by role, after setmaxnreg: the softmax takes what the others do not need.
  static constexpr int REGS_SOFTMAX = kSplitKV ? 136 : 144, REGS_CONVERT = kSplitKV ? 80 : 64, REGS_OTHER = kSplitKV ? 48 : 64;
  static_assert(kSoftmax * REGS_SOFTMAX + kConverters * REGS_CONVERT + 128 * REGS_OTHER <= kThreads * kRegsLaunch &&
                    REGS_SOFTMAX >= kRegsLaunch && REGS_CONVERT <= kRegsLaunch && REGS_OTHER <= kRegsLaunch,
                "setmaxnreg shares out what the block was launched with; dec takes no more than that, inc no less");
  // shared memory: Q, K stages, V (FP16) x 2
  static constexpr int K_OFF = Q_BYTES, V_OFF = K_OFF + K_STAGES * K_BYTES, CTL_OFF = V_OFF + 2 * V_BYTES;
};

// Parity of the phase that a stream's barriers go through for its tile j.
template <int D>
__device__ __forceinline__ uint32_t phase(int j) { return (Cfg<D>::kSplitKV ? j >> 1 : j) & 1; }

struct Scales {
  float k, log_v, inv_v, pad;
};

template <int D>
struct Control {
  uint64_t q_ready, k_full[3], k_empty[3], ids_full[8], v_full[2], v_empty[2];
  uint64_t s_ready[2], p_ready[2], o_done[2], m_ready[2];  // by stream
  uint64_t join, done;
  uint32_t tmem;
  int nan_any;
  // Scales and (block, head) indexes (-1: no tokens) by tile.  A slot comes up again eight
  // tiles later; a tile's K is loaded at most three tiles ahead of the products with K, and those
  // are issued at most two tiles ahead of the last softmax that is not done.
  Scales ks[8][Cfg<D>::GROUPS];
  int blk[8][Cfg<D>::GROUPS];    // by 16-token group
  int nan_first[D];
  float rc[Cfg<D>::ROWS];        // score scale of each query row, times log2(e)
  float m_ref[2][kTile];         // kSplitKV: reference maxima of the rows, by parity of the tile
  float l[2][kTile];             // kSplitKV
};

template <int D>
constexpr int smem_bytes() {
  return 1024 + Cfg<D>::CTL_OFF + int(sizeof(Control<D>));
}

__host__ __device__ constexpr uint32_t make_idesc(int m, int n, bool b_mn_major) {
  return (1u << 4) | (b_mn_major ? 1u << 16 : 0u) | (uint32_t(n >> 3) << 17) | (uint32_t(m >> 4) << 24);
}

// 1 in one lane of the warp.  elect.sync and not a comparison of lane numbers: the compiler then
// knows that one lane issues and spends fewer instructions on each product (8192-token prompt
// 1073 -> 940 us).
__device__ __forceinline__ uint32_t elect_one() {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(r));
  return r;
}

// FP8 MMA, both operands E4M3 in shared memory, and FP16 MMA with A in TMEM; FP32 accumulation.
// (The E4M3 codes of the descriptor's type fields are 0, as are FP16's.)  Called by whole
// warps, so that operands stay warp-uniform; the lane with `elected` != 0 issues.
__device__ __forceinline__ void mma_f8_ss(uint32_t elected, uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(elected)
      : "memory");
}
__device__ __forceinline__ void mma_f16_ts(uint32_t elected, uint32_t d, uint32_t a_tmem, uint64_t b, uint32_t idesc,
                                           uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "setp.ne.b32 q, %5, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(a_tmem), "l"(b), "r"(idesc), "r"(accumulate), "r"(elected)
      : "memory");
}
__device__ __forceinline__ void commit(uint32_t elected, uint64_t *bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\t"
      "setp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar)),
      "r"(elected)
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

// K-major operand whose rows are 64 bytes, with the 64-byte swizzle; 8-row groups 512 bytes apart.
__device__ __forceinline__ uint64_t sdesc_sw64_kmajor(uint32_t saddr) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr >> 4) & 0x3FFF);
  d |= (uint64_t)1 << 16;
  d |= (uint64_t)(512 >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)4 << 61;
  return d;
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

__device__ __forceinline__ uint4 ld_stream(const void *p) {
  uint4 r;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w)
               : "l"(p));
  return r;
}

// Generic-proxy writes to shared memory become visible to the tensor cores.
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

// One arrival for the warp, after what all its lanes did.
__device__ __forceinline__ void warp_arrive(uint64_t *bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}

// 16-byte piece `c` (of 8) of row `r` of panel `p`, a panel holding `rows` rows.
__device__ __forceinline__ uint32_t panel_offset(int rows, int p, int r, int c) {
  return (p * rows + r) * 128 + ((c ^ (r & 7)) << 4);
}

// The same for rows of codes: panels of ROWB bytes.
template <int D>
__device__ __forceinline__ uint32_t code_offset(int rows, int r, int c) {
  if constexpr (D < 128) return r * 64 + ((c ^ ((r >> 1) & 3)) << 4);
  return ((c >> 3) * rows + r) * 128 + (((c & 7) ^ (r & 7)) << 4);
}

// What a CTA works on.
struct Item {
  Seq sq;
  int seq, h, row0;  // first query row of its tiles
  int kv_end;        // cached tokens that some row sees
  int lim_min;       // tokens that every row sees
  int parts;         // CTAs that share the item's K / V tiles
  int tok0, tiles;   // first token and number of tiles of this part
};

// Part `part` of item `index`: items of a sequence are (row block, kv head), the row blocks with
// the most visible tokens first.  Returns false when there is none.  An item is cut into up to
// a.splits parts of kMinTiles tiles at least.
constexpr int kMinTiles = 8;
template <int D, int THREADS>
__device__ bool find_item(const Args &a, Item &it, int index, int part) {
  using C = Cfg<D>;
  __shared__ int64_t s_sum[THREADS / 32], s_before;
  __shared__ int s_seq, s_bound[THREADS / 32];
  int64_t base = 0;
  int high = 0;
  bool odd = false;  // some sequence does not count by its own bounds or length; uniform
  constexpr int64_t kOdd = int64_t(1) << 48;  // more than THREADS sequences' items: marks one in the sums
  for (int s0 = 0; s0 < a.n_seqs; s0 += THREADS) {
    const int s = s0 + threadIdx.x;
    int64_t items, sum, all;
    for (;;) {
      Seq q{0, 0, 0, true};
      if (odd) q = scan_seq<THREADS>(a, s, high, s_bound);
      else if (s < a.n_seqs) q = load_seq(a, s);
      const int64_t rows = int64_t(q.q_len) * a.group;
      items = rows > a.max_decode_rows ? (rows + C::ROWS - 1) / C::ROWS * a.kv_heads : 0;
      sum = odd || q.ok ? items : kOdd;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, sum, o);
        if ((threadIdx.x & 31) >= o) sum += x;
      }
      if (threadIdx.x == 0) s_seq = -1;
      if ((threadIdx.x & 31) == 31) s_sum[threadIdx.x >> 5] = sum;
      __syncthreads();
      all = 0;
      for (int w = 0; w < THREADS / 32; ++w) {
        if (w < int(threadIdx.x >> 5)) sum += s_sum[w];
        all += s_sum[w];
      }
      if (all < kOdd) break;
      odd = true;  // again, with what the earlier sequences' bounds leave
      __syncthreads();
    }
    if (index < base + sum && index >= base + sum - items) {
      s_seq = s;
      s_before = base + sum - items;
    }
    __syncthreads();
    if (s_seq >= 0) {
      const int local = static_cast<int>(index - s_before);
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
      const int tiles = (it.kv_end + C::BN - 1) / C::BN;
      it.parts = min(max(tiles / kMinTiles, 1), a.splits);
      const int first = static_cast<int>(int64_t(tiles) * part / it.parts);
      it.tok0 = first * C::BN;
      it.tiles = static_cast<int>(int64_t(tiles) * (part + 1) / it.parts) - first;
      return part < it.parts;
    }
    base += all;
    __syncthreads();
  }
  return false;
}

// Producer warp.  A tile consists of BN / R boxes of R consecutive tokens of one cache block; lane i
// looks up box i, publishes where it is and its scales, and copies its K.
template <int D>
__device__ void produce(const Args &a, const CUtensorMap *k_map, Control<D> &c, unsigned char *kbuf, const Item &it,
                        int n_tiles) {
  using C = Cfg<D>;
  const int lane = threadIdx.x & 31;
  const int log_r = min(a.log_block, C::LOG_BOX), R = 1 << log_r, boxes = C::BN >> log_r;
  const int mask = (1 << a.log_block) - 1;
  const int32_t *row = a.table + it.seq * a.ld_table;
  auto token = [&](int j) { return it.tok0 + j * C::BN + (lane << log_r); };
  auto wanted = [&](int j) { return j < n_tiles && lane < boxes && token(j) < it.kv_end; };
  auto lookup = [&](int j) { return wanted(j) ? __ldg(row + (token(j) >> a.log_block)) : -1; };
  auto check = [&](int j, int id) -> int {  // (block, head) index, -1: nothing there
    if (!wanted(j)) return -1;
    if (id < 0 || id >= a.num_blocks) {
      record_bad_index();
      return -1;
    }
    return id * a.kv_heads + it.h;
  };
  int blk = check(0, lookup(0)), next_id = lookup(1);
  float sk = blk >= 0 ? __ldg(a.k_scales + blk) : 0.0f, sv = blk >= 0 ? __ldg(a.v_scales + blk) : 1.0f;
#pragma unroll 1
  for (int j = 0; j < n_tiles; ++j) {
    const int ks = j % C::K_STAGES;
    if (lane < boxes) {
      Scales s;
      s.k = sk;
      s.log_v = blk >= 0 ? log_scale(sv) : -INFINITY;  // no such block: nothing to see
      s.inv_v = blk >= 0 ? inverse_scale(sv) : 0.0f;
      s.pad = 0.0f;
      for (int g = 0; g < R / kGroup; ++g) {
        c.ks[j & 7][lane * (R / kGroup) + g] = s;
        c.blk[j & 7][lane * (R / kGroup) + g] = blk;
      }
    }
    warp_arrive(&c.ids_full[j & 7]);
    const uint32_t have = __ballot_sync(0xffffffffu, blk >= 0);
    if (!mbar_wait(&c.k_empty[ks], ((j / C::K_STAGES) & 1) ^ 1)) return;
    if (wanted(j) && blk < 0) {
      // no such block: what the stage held before may be NaN codes, whose scores no scale would mask
      for (int p = 0; p < C::PANELS8; ++p)
        for (int i = 0; i < R * C::ROWB; i += 16)
          *reinterpret_cast<uint4 *>(kbuf + ks * C::K_BYTES + (p * C::BN + lane * R) * C::ROWB + i) = make_uint4(0, 0, 0, 0);
      fence_async_smem();
    }
    __syncwarp();
    if (lane == 0) mbar_arrive_expect_tx(&c.k_full[ks], __popc(have) * (R * D));
    __syncwarp();
    if (blk >= 0) {
#pragma unroll
      for (int p = 0; p < C::PANELS8; ++p)
        tma_load_3d(kbuf + ks * C::K_BYTES + (p * C::BN + lane * R) * C::ROWB, k_map, &c.k_full[ks], p * 128, token(j) & mask, blk);
    }
    blk = check(j + 1, next_id);
    sk = blk >= 0 ? __ldg(a.k_scales + blk) : 0.0f;
    sv = blk >= 0 ? __ldg(a.v_scales + blk) : 1.0f;
    next_id = lookup(j + 2);
  }
}

// Converter threads: V stages of codes into FP16, a thread's next codes on their way to registers
// meanwhile.  At 256 values per head the products with K leave little of shared memory, a stage takes
// long, and two groups of four warps take stages in turn: one's loads and fence pass while the other
// stores (1024 tokens on 32768: 754 us, all eight on one stage 871).  At 128 values all warps take
// each stage (8192-token prompt 807 us; in turn 858; four warps in all 889).
template <int D>
struct Converter {
  using C = Cfg<D>;
  const Args &a;
  Control<D> &c;
  const Item &it;
  int n, turn, tid;  // stages in all

  // Piece k of a stage: 16 bytes of row tid / CPR + k STEP
  static constexpr int STEP = C::PER_V / C::CPR;
  static_assert(STEP % 8 == 0 && C::VT % STEP == 0, "the swizzle repeats every 8 rows");

  __device__ __forceinline__ bool load(int i, uint4 (&x)[C::PIECES]) const {
    if (i >= n) return true;
    const int j = i / C::VSUB;
    const bool ok = mbar_wait(&c.ids_full[j & 7], (j >> 3) & 1);
    const int row0 = (i % C::VSUB) * C::VT + tid / C::CPR, tok0 = it.tok0 + j * C::BN + row0;
    const int *blks = c.blk[j & 7];
    const unsigned char *v = reinterpret_cast<const unsigned char *>(a.v) + 16 * (tid % C::CPR);
#pragma unroll
    for (int k = 0; k < C::PIECES; ++k) {
      const int64_t blk = ok ? blks[(row0 + k * STEP) / kGroup] : -1;
      const int tok = tok0 + k * STEP;
      x[k] = make_uint4(0, 0, 0, 0);  // bytes that belong to no token never reach the product
      if (blk >= 0 && tok < it.kv_end) x[k] = ld_stream(v + ((blk << a.log_block) + (tok & ((1 << a.log_block) - 1))) * D);
    }
    return ok;
  }
  __device__ __forceinline__ bool store(int i, unsigned char *vbuf, uint4 (&x)[C::PIECES]) const {
    const int st = i & 1, row0 = tid / C::CPR, col = tid % C::CPR;
    if (!mbar_wait(&c.v_empty[st], ((i >> 1) & 1) ^ 1)) return false;
    if (it.tok0 + (i + 1) * C::VT > it.lim_min) {
#pragma unroll 1
      for (int m = 0; m < 4 * C::PIECES; ++m) {  // a NaN that some rows must not see: see decode_segment
        uint32_t w = 0;
#pragma unroll
        for (int k = 0; k < C::PIECES; ++k) {
          if (m == 4 * k) w = x[k].x;
          if (m == 4 * k + 1) w = x[k].y;
          if (m == 4 * k + 2) w = x[k].z;
          if (m == 4 * k + 3) w = x[k].w;
        }
        if ((((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u) == 0) continue;
        for (int b = 0; b < 4; ++b)
          if (((w >> (8 * b)) & 0x7f) == 0x7f) {
            atomicMin(&c.nan_first[16 * col + 4 * (m & 3) + b], it.tok0 + i * C::VT + row0 + (m >> 2) * STEP);
            c.nan_any = 1;
            w &= ~(0xffu << (8 * b));
          }
#pragma unroll
        for (int k = 0; k < C::PIECES; ++k) {
          if (m == 4 * k) x[k].x = w;
          if (m == 4 * k + 1) x[k].y = w;
          if (m == 4 * k + 2) x[k].z = w;
          if (m == 4 * k + 3) x[k].w = w;
        }
      }
    }
    // every other panel stores its odd piece first: eight lanes then hit distinct banks
    const int odd = (col >> 2) & 1;
    unsigned char *dst0 = vbuf + st * C::V_BYTES + panel_offset(C::VT, col >> 2, row0, 2 * (col & 3) + odd);
    unsigned char *dst1 = vbuf + st * C::V_BYTES + panel_offset(C::VT, col >> 2, row0, 2 * (col & 3) + (odd ^ 1));
#pragma unroll
    for (int k = 0; k < C::PIECES; ++k) {
      auto half = [](uint32_t lo, uint32_t hi) {
        uint4 h;
        e4m3x4_to_f16x4(lo, h.x, h.y);
        e4m3x4_to_f16x4(hi, h.z, h.w);
        return h;
      };
      *reinterpret_cast<uint4 *>(dst0 + k * STEP * 128) = odd ? half(x[k].z, x[k].w) : half(x[k].x, x[k].y);
      *reinterpret_cast<uint4 *>(dst1 + k * STEP * 128) = odd ? half(x[k].x, x[k].y) : half(x[k].z, x[k].w);
    }
    fence_async_smem();
    warp_arrive(&c.v_full[st]);
    return true;
  }
  __device__ void run(unsigned char *vbuf) const {
    uint4 x[C::PIECES];
    if (!load(turn, x)) return;
#pragma unroll 1
    for (int i = turn; i < n; i += C::TURNS)
      if (!store(i, vbuf, x) || !load(i + C::TURNS, x)) return;
  }
};

// MMA issuer (a whole warp).  All 512 TMEM columns are this CTA's: addresses start at 0.
// Descriptors are built once; within an operand they differ in the address field.
template <int D>
struct Issuer {
  using C = Cfg<D>;
  static constexpr uint32_t kIdescS = make_idesc(kTile, C::BN, false), kIdescO = make_idesc(kTile, D, true);
  Control<D> &c;
  uint32_t elected;
  uint64_t qd, kd, vd;

  __device__ Issuer(Control<D> &c, uint32_t q, uint32_t k, uint32_t v) : c(c), elected(elect_one()) {
    qd = D < 128 ? sdesc_sw64_kmajor(q) : sdesc_sw128_kmajor(q);
    kd = D < 128 ? sdesc_sw64_kmajor(k) : sdesc_sw128_kmajor(k);
    vd = sdesc_sw128_mnmajor(v, C::VT * 128);
  }

  // S = (hi + lo) K_j^T of stream w
  __device__ __forceinline__ void qk(int w, int j) const {
    const uint64_t a = qd + (C::kSplitKV ? 0 : w * (2 * C::Q_PART >> 4)), b = kd + (j % C::K_STAGES) * (C::K_BYTES >> 4);
    const uint32_t s_col = w * C::BN;
#pragma unroll
    for (int part = 0; part < 2; ++part)
#pragma unroll
      for (int p = 0; p < C::PANELS8; ++p)
#pragma unroll
        for (int s = 0; s < C::ROWB / 32; ++s)
          mma_f8_ss(elected, s_col, a + (part * C::Q_PART + p * kTile * 128 + 32 * s) / 16, b + (p * C::BN * 128 + 32 * s) / 16,
                    kIdescS, (part | p | s) != 0);
    commit(elected, &c.s_ready[w]);
  }
  // O += P V_j, by V stages; `last`: nobody else reads V_j
  __device__ __forceinline__ bool pv(int w, int j, bool last) const {
    const uint32_t p_col = w * C::BN, o_col = C::O_COL0 + (C::kSplitKV ? 0 : w * D);
#pragma unroll
    for (int h = 0; h < C::VSUB; ++h) {
      const int i = j * C::VSUB + h;
      bool ok = mbar_wait(&c.v_full[i & 1], (i >> 1) & 1);
      if (h == 0) ok = ok && mbar_wait(&c.p_ready[w], phase<D>(j));
      tc_fence_after();
      if (!__all_sync(0xffffffffu, ok)) return false;
      const uint64_t b = vd + (i & 1) * (C::V_BYTES >> 4);
#pragma unroll
      for (int s = 0; s < C::VT / 16; ++s)
        mma_f16_ts(elected, o_col, p_col + 8 * (h * (C::VT / 16) + s), b + s * (2048 / 16), kIdescO, (j | h | s) != 0);
      if (last) commit(elected, &c.v_empty[i & 1]);
    }
    commit(elected, &c.o_done[w]);
    return true;
  }
  __device__ __forceinline__ bool k_full(int j) const {
    const bool ok = mbar_wait(&c.k_full[j % C::K_STAGES], (j / C::K_STAGES) & 1);
    tc_fence_after();
    return __all_sync(0xffffffffu, ok);
  }
  __device__ __forceinline__ void k_done(int j) const { commit(elected, &c.k_empty[j % C::K_STAGES]); }

  // The streams in turn: each gets its products in one piece, which keeps the streams half a period
  // apart (with an issuer each they fell into step, and the tensor cores idled while both took
  // exponentials: 5040 cycles per tile against 4290).  A stream's next scores go over its P, right
  // behind the products with it: products of one issuer run in order.
  __device__ void run(int n_tiles) const {
    if (!__all_sync(0xffffffffu, mbar_wait(&c.q_ready, 0))) return;
    if constexpr (!C::kSplitKV) {
      if (!k_full(0)) return;
      qk(0, 0);
      qk(1, 0);
      k_done(0);
#pragma unroll 1
      for (int j = 0; j < n_tiles; ++j) {
        if (!pv(0, j, false)) return;
        if (j + 1 < n_tiles) {
          if (!k_full(j + 1)) return;
          qk(0, j + 1);
        }
        if (!pv(1, j, true)) return;
        if (j + 1 < n_tiles) {
          qk(1, j + 1);
          k_done(j + 1);
        }
      }
    } else {
      for (int j = 0; j < 2 && j < n_tiles; ++j) {
        if (!k_full(j)) return;
        qk(j, j);
        k_done(j);
      }
#pragma unroll 1
      for (int j = 0; j < n_tiles; ++j) {
        const int w = j & 1;
        if (!pv(w, j, true)) return;
        if (j + 2 < n_tiles) {
          if (!k_full(j + 2)) return;
          qk(w, j + 2);
          k_done(j + 2);
        }
      }
    }
  }
};

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

__device__ __forceinline__ float fmaxf_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// 2^x for two values on the FMA pipe: 2^n 2^f with n = round(x), f in [-1/2, 1/2], and a
// polynomial of degree 4 for 2^f (minimax in relative error by Remez' exchange, 2^-18.5, far
// below the FP16 rounding that follows).  x is clamped to [-126, 127]; a NaN becomes 2^127, which
// the check of the weights' sum catches.
__device__ __forceinline__ float2 exp2_poly(float2 x) {
  constexpr float kMagic = 12582912.0f;  // 1.5 * 2^23: adding it leaves round(x) in the low bits
  x.x = fminf(fmaxf_nan(x.x, -126.0f), 127.0f);
  x.y = fminf(fmaxf_nan(x.y, -126.0f), 127.0f);
  const float2 t = add_f32x2(x, make_float2(kMagic, kMagic));
  const float2 n = add_f32x2(t, make_float2(-kMagic, -kMagic));
  const float2 f = gdn::ffma2(n, make_float2(-1.0f, -1.0f), x);
  float2 p = gdn::ffma2(f, make_float2(0.009570102207362652f, 0.009570102207362652f),
                       make_float2(0.05591785907745361f, 0.05591785907745361f));
  p = gdn::ffma2(p, f, make_float2(0.240247443318367f, 0.240247443318367f));
  p = gdn::ffma2(p, f, make_float2(0.6931217908859253f, 0.6931217908859253f));
  p = gdn::ffma2(p, f, make_float2(0.9999992847442627f, 0.9999992847442627f));
  return make_float2(__uint_as_float(__float_as_uint(p.x) + (__float_as_uint(t.x) << 23)),
                     __uint_as_float(__float_as_uint(p.y) + (__float_as_uint(t.y) << 23)));
}

// Maximum of x = s c + e over the thread's row of S, NaN if there is one; MASK: only the
// first `vis` columns.
template <int D, bool MASK>
__device__ __forceinline__ float row_max(uint32_t s_tmem, const Scales *sc, float rc, int vis) {
  float mt = -INFINITY;
#pragma unroll
  for (int i = 0; i < Cfg<D>::BN / 32; ++i) {
    uint32_t v[32];
    tmem_ld_32x32b_x32(s_tmem + 32 * i, v);
    tmem_ld_wait();
    if constexpr (MASK) {
#pragma unroll
      for (int n = 0; n < 32; ++n)
        if (32 * i + n >= vis) v[n] = 0xff800000u;
    }
    float m[2][2];
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const uint32_t *u = v + 16 * g;
      m[g][0] = fmaxf_nan(__uint_as_float(u[0]), __uint_as_float(u[1]));
      m[g][1] = fmaxf_nan(__uint_as_float(u[2]), __uint_as_float(u[3]));
#pragma unroll
      for (int n = 4; n < 16; n += 4) {
        m[g][0] = max3(m[g][0], __uint_as_float(u[n]), __uint_as_float(u[n + 1]));
        m[g][1] = max3(m[g][1], __uint_as_float(u[n + 2]), __uint_as_float(u[n + 3]));
      }
      const float x = fmaxf_nan(m[g][0], m[g][1]);
      const Scales s = sc[2 * i + g];
      const float y = fmaf(x, s.k * rc, s.log_v);
      mt = fmaxf_nan(mt, x == -INFINITY ? x : y);
    }
  }
  return mt;
}

// P = 2^(x - base) over the row of S as FP16 in p, sum of P kSumUnit / sV in l; returns the sum of
// P (NaN if a score is).  MASK: only the first `vis` columns.
template <int D, bool MASK>
__device__ __forceinline__ float row_exp(uint32_t s_tmem, const Scales *sc, float rc, float base, int vis,
                                         uint32_t (&p)[Cfg<D>::BN / 2], float &l) {
  float all = 0.0f;
  l = 0.0f;
#pragma unroll
  for (int i = 0; i < Cfg<D>::BN / 32; ++i) {
    uint32_t v[32];
    tmem_ld_32x32b_x32(s_tmem + 32 * i, v);
    tmem_ld_wait();
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const Scales s = sc[2 * i + g];
      const float ck = s.k * rc, ce = s.log_v - base;
      float2 sum = make_float2(0.0f, 0.0f);
#pragma unroll
      for (int n = 0; n < 16; n += 2) {
        float2 x = gdn::ffma2(make_float2(__uint_as_float(v[16 * g + n]), __uint_as_float(v[16 * g + n + 1])),
                             make_float2(ck, ck), make_float2(ce, ce));
        if constexpr (MASK) {
          if (32 * i + 16 * g + n >= vis) x.x = -INFINITY;
          if (32 * i + 16 * g + n + 1 >= vis) x.y = -INFINITY;
        }
        // The MUFU's 16 exponentials per clock are one of the bounds where the streams are row
        // tiles: there one pair in eight goes to the FMA pipe (8192-token prompt 824 -> 806 us; one in
        // four 811, three in eight 825).  At 256 values it only costs issue slots (844 -> 850 us).
        if (!Cfg<D>::kSplitKV && n == 6) {
          x = exp2_poly(x);
        } else {
          x.x = ex2(x.x);
          x.y = ex2(x.y);
        }
        sum = add_f32x2(sum, x);
        p[16 * i + 8 * g + n / 2] = pack_f16(x.x, x.y);
      }
      all += sum.x + sum.y;
      l = fmaf(sum.x + sum.y, s.inv_v, l);
    }
  }
  return all;
}

// The CTA's query rows in two E4M3 parts, scaled by 2^-e.  A lane holds 16 consecutive values,
// one piece of each part, so D / 16 lanes take a row and a warp several rows at a time.
template <int D>
__device__ __forceinline__ void load_queries(const Args &a, Control<D> &c, unsigned char *qbuf, const Item &it, int warp) {
  using C = Cfg<D>;
  constexpr int kLanes = D / 16, kRowsAtOnce = 32 / kLanes;
  constexpr int kPer = C::ROWS / (kSoftmax / 32), kSteps = kPer / kRowsAtOnce;  // rows of a warp, in steps
  const int lane = threadIdx.x & 31, piece = lane % kLanes;
  const int n_rows = it.sq.q_len * a.group;
  const float sign = a.scale_log2 < 0.0f ? -1.0f : 1.0f;
  uint4 raw[kSteps][2];
#pragma unroll
  for (int u = 0; u < kSteps; ++u) {
    const int R = it.row0 + warp * kPer + u * kRowsAtOnce + lane / kLanes;
    raw[u][0] = raw[u][1] = make_uint4(0, 0, 0, 0);
    if (R < n_rows) {
      const int t = R / a.group;
      const uint4 *src = reinterpret_cast<const uint4 *>(
          a.q + (it.sq.start + t) * a.ld_q + int64_t(it.h * a.group + (R - t * a.group)) * D + 16 * piece);
      raw[u][0] = __ldg(src);
      raw[u][1] = __ldg(src + 1);
    }
  }
#pragma unroll
  for (int u = 0; u < kSteps; ++u) {
    const uint32_t v[8] = {raw[u][0].x, raw[u][0].y, raw[u][0].z, raw[u][0].w, raw[u][1].x, raw[u][1].y, raw[u][1].z, raw[u][1].w};
    uint32_t top = 0;  // BF16 magnitudes order as integers, two at a time
#pragma unroll
    for (int n = 0; n < 8; ++n) top = __vmaxu2(top, v[n] & 0x7fff7fffu);
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1) top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, o));
    const uint32_t bits = max(top & 0xffffu, top >> 16) << 16;  // the row's largest magnitude
    // 2^-e brings it into (224, 448], 448 = 1.75 * 2^8
    const int e = max(static_cast<int>(bits >> 23) - 127 - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0), -126);
    // an infinite value makes every score of the row infinite or NaN: the row is NaN
    const float f = bits < 0x7f800000u ? __uint_as_float(static_cast<uint32_t>(127 - e) << 23) * sign : __int_as_float(0x7fffffff);
    const int r = warp * kPer + u * kRowsAtOnce + lane / kLanes;
    if (piece == 0) c.rc[r] = fabsf(a.scale_log2) * __uint_as_float(static_cast<uint32_t>(min(e, 120) + 127) << 23);
    uint32_t hi[4], lo[4];
#pragma unroll
    for (int n = 0; n < 4; ++n) {
      hi[n] = lo[n] = 0;
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const uint32_t x = v[2 * n + m];
        const float x0 = __uint_as_float(x << 16) * f, x1 = __uint_as_float(x & 0xFFFF0000u) * f;
        const uint32_t c8 = cvt_e4m3x2(x1, x0), back = e4m3x2_to_f16x2(c8);
        const float2 h = __half22float2(*reinterpret_cast<const __half2 *>(&back));
        hi[n] |= c8 << (16 * m);
        lo[n] |= static_cast<uint32_t>(cvt_e4m3x2(x1 - h.y, x0 - h.x)) << (16 * m);
      }
    }
    unsigned char *dst = qbuf + (r / kTile) * 2 * C::Q_PART + code_offset<D>(kTile, r & (kTile - 1), piece);
    *reinterpret_cast<uint4 *>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4 *>(dst + C::Q_PART) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  }
  fence_async_smem();
  warp_arrive(&c.q_ready);
}

// Softmax warpgroup of stream w; tid 0..127 is the row of its tile.
template <int D>
__device__ void softmax(const Args &a, Control<D> &c, const Item &it, int n_tiles, int w, int tid) {
  using C = Cfg<D>;
  const int n_rows = it.sq.q_len * a.group;
  const int local = (C::kSplitKV ? 0 : w * kTile) + tid, R = it.row0 + local;
  const bool valid = R < n_rows;
  const int tok = valid ? R / a.group : 0, head = it.h * a.group + (valid ? R % a.group : 0);
  const int lim = !valid ? it.kv_end : a.causal ? it.sq.kv_len - it.sq.q_len + tok + 1 : it.sq.kv_len;
  const int warp_lim = __reduce_min_sync(0xffffffffu, lim);
  if (!__all_sync(0xffffffffu, mbar_wait(&c.q_ready, 0))) return;
  const float rc = c.rc[local];

  const uint32_t lanes = (tid & ~31) << 16;  // TMEM lane quadrant of the warp
  const uint32_t s_tmem = lanes + w * C::BN, o_tmem = lanes + C::O_COL0 + (C::kSplitKV ? 0 : w * D);
  float m_ref = -INFINITY, l = 0.0f;
  const int step = C::kSplitKV ? 2 : 1;
#pragma unroll 1
  for (int j = C::kSplitKV ? w : 0; j < n_tiles; j += step) {
    if (!__all_sync(0xffffffffu, mbar_wait(&c.s_ready[w], phase<D>(j)))) return;
    tc_fence_after();
    const Scales *sc = c.ks[j & 7];
    const int col0 = it.tok0 + j * C::BN, vis = lim - col0;  // visible columns of this row
    const bool masked = warp_lim < col0 + C::BN;
    uint32_t p[C::BN / 2];
    float add = 0.0f;
    // Takes up the reference that the other stream's tile j - 1 left (kSplitKV); 0: as it was, 1: moved, -1: failed.
    auto follow = [&] {
      if (!__all_sync(0xffffffffu, mbar_wait(&c.m_ready[w ^ 1], phase<D>(j - 1)))) return -1;
      const float m = c.m_ref[(j - 1) & 1][tid];
      const bool moved = m != m_ref;
      if (moved) l *= m_ref == -INFINITY ? 0.0f : ex2(m_ref - m);
      m_ref = m;
      return __any_sync(0xffffffffu, moved) ? 1 : 0;
    };
    if (C::kSplitKV && j == 1 && follow() < 0) return;
    bool over = j == 0;  // no reference yet: straight to the maximum
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
      if (pass == 1 || !over) {
        const float base = (m_ref == -INFINITY ? 0.0f : m_ref) - kBoostP;
        const float all = masked ? row_exp<D, true>(s_tmem, sc, rc, base, vis, p, add) : row_exp<D, false>(s_tmem, sc, rc, base, vis, p, add);
        if (pass == 1) break;
        over = __any_sync(0xffffffffu, !(all < kMostSum) || (m_ref == -INFINITY && all > 0.0f));
      }
      int moved = 0;
      if (C::kSplitKV && j > 1) moved = follow();
      if (moved < 0) return;
      if (over) {
        const float mt = masked ? row_max<D, true>(s_tmem, sc, rc, vis) : row_max<D, false>(s_tmem, sc, rc, vis);
        if (!(mt < INFINITY)) l = __int_as_float(0x7fffffff);  // a NaN or infinite score: so is the row
        const bool grow = mt > m_ref;
        const float f = grow ? ex2(m_ref - mt) : 1.0f;
        if (grow) {
          l *= f;
          m_ref = mt;
        }
        if (j > 0 && __any_sync(0xffffffffu, grow)) {
          // O holds the earlier tiles: it may be touched once their products are in
          if (!__all_sync(0xffffffffu, mbar_wait(&c.o_done[C::kSplitKV ? w ^ 1 : w], phase<D>(j - 1)))) return;
          tc_fence_after();
          scale_o<D>(o_tmem, f);
        }
      }
      if (!over && !moved) break;
    }
    l += add;
    if constexpr (C::kSplitKV) {
      c.m_ref[j & 1][tid] = m_ref;  // last read for tile j - 1, by the thread that let this one go on
      warp_arrive(&c.m_ready[w]);
    }
    uint32_t(*half)[32] = reinterpret_cast<uint32_t(*)[32]>(p);
    tmem_st_32x32b_x32(s_tmem, half[0]);
    tmem_st_32x32b_x32(s_tmem + 32, half[1]);
    tmem_st_wait();
    tc_fence_before();
    warp_arrive(&c.p_ready[w]);
  }

  if constexpr (C::kSplitKV) {  // join the streams' sums
    warp_arrive(&c.join);
    if (!__all_sync(0xffffffffu, mbar_wait(&c.join, 0))) return;
    const float m = c.m_ref[(n_tiles - 1) & 1][tid];  // the last reference; l is relative to the one seen last
    if (m != m_ref && m_ref != -INFINITY) l *= ex2(m_ref - m);
    m_ref = m;
    c.l[w][tid] = l;
    warp_arrive(&c.join);
    if (!__all_sync(0xffffffffu, mbar_wait(&c.join, 1))) return;
    l = c.l[0][tid] + c.l[1][tid];
  }
  // the last products, and all before
  if (!__all_sync(0xffffffffu, mbar_wait(&c.o_done[C::kSplitKV ? (n_tiles - 1) & 1 : w], phase<D>(n_tiles - 1)))) return;
  tc_fence_after();
  const bool empty = m_ref == -INFINITY && l == l;  // no visible token (a NaN score leaves m_ref, not l)
  const float f = kSumUnit / l;
  constexpr int kCols = C::kSplitKV ? D / 2 : D;
  const int col0 = C::kSplitKV ? w * kCols : 0;
  const int64_t at = (it.sq.start + tok) * a.ld_out + int64_t(head) * D;
  const bool nan_any = *const_cast<volatile int *>(&c.nan_any) != 0;
  const int64_t part_row = int64_t(blockIdx.x) * C::ROWS + local;  // of the partial results
  if (it.parts > 1 && col0 == 0) a.prompt_ml[part_row] = make_float2(m_ref, l);
#pragma unroll 1
  for (int c0 = col0; c0 < col0 + kCols; c0 += 32) {
    uint32_t r[32];
    tmem_ld_32x32b_x32(o_tmem + c0, r);
    tmem_ld_wait();
#pragma unroll
    for (int n = 0; n < 32; ++n) {
      if (it.parts == 1) r[n] = empty ? 0u : __float_as_uint(__uint_as_float(r[n]) * f);
      if (nan_any && c.nan_first[c0 + n] < lim) r[n] = 0x7fffffffu;
    }
    if (!valid) continue;
    if (it.parts > 1 || a.out_fp32) {
      uint4 *dst = reinterpret_cast<uint4 *>(it.parts > 1 ? a.prompt_part + part_row * D + c0 : static_cast<float *>(a.out) + at + c0);
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

// Grid: an upper bound of the items, times a.splits; dynamic shared memory smem_bytes<D>().
template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    prompt_kernel(const __grid_constant__ Args a, const __grid_constant__ CUtensorMap k_map) {
  using C = Cfg<D>;
  extern __shared__ unsigned char smem_raw[];
  grid_dep_wait();
  grid_dep_launch();
  Item it;
  const int index = blockIdx.x / a.splits;
  if (!find_item<D, kThreads>(a, it, index, static_cast<int>(blockIdx.x) - index * a.splits)) return;
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
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
  const int n_tiles = it.tiles;
  unsigned char *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
  unsigned char *qbuf = smem, *kbuf = smem + C::K_OFF, *vbuf = smem + C::V_OFF;
  Control<D> &c = *reinterpret_cast<Control<D> *>(smem + C::CTL_OFF);
  if (tid == 0) {
    mbar_init(&c.q_ready, kSoftmax / 32);
    for (int i = 0; i < 8; ++i) mbar_init(&c.ids_full[i], 1);
    for (int i = 0; i < 3; ++i) {
      mbar_init(&c.k_full[i], 1);
      mbar_init(&c.k_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&c.v_full[i], C::PER_V / 32);
      mbar_init(&c.v_empty[i], 1);
      mbar_init(&c.s_ready[i], 1);
      mbar_init(&c.p_ready[i], 4);
      mbar_init(&c.o_done[i], 1);
      mbar_init(&c.m_ready[i], 4);
    }
    mbar_init(&c.join, kSoftmax / 32);
    mbar_init(&c.done, 1);
    fence_barrier_init();
    c.nan_any = 0;
  }
  for (int i = tid; i < D; i += kThreads) c.nan_first[i] = 0x7fffffff;
  if (warp == 0) {
    tmem_alloc(&c.tmem, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  if (warp >= 4 && warp < 12) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::REGS_SOFTMAX));
    load_queries<D>(a, c, qbuf, it, warp - 4);
    softmax<D>(a, c, it, n_tiles, (warp - 4) >> 2, tid & 127);
  } else if (warp >= 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REGS_CONVERT));
    Converter<D>{a, c, it, n_tiles * C::VSUB, C::TURNS == 1 ? 0 : (tid - 12 * 32) / C::PER_V,
                 C::TURNS == 1 ? tid - 12 * 32 : (tid - 12 * 32) % C::PER_V}.run(vbuf);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REGS_OTHER));
    if (warp == 1) {
      produce<D>(a, &k_map, c, kbuf, it, n_tiles);
    } else if (warp == 0) {
      Issuer<D> mma(c, smem_u32(qbuf), smem_u32(kbuf), smem_u32(vbuf));
      mma.run(__reduce_max_sync(0xffffffffu, n_tiles));  // uniform for the compiler too
      commit(mma.elected, &c.done);  // whatever was issued has to end before TMEM is given back
      mbar_wait(&c.done, 0);
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 0) tmem_dealloc(c.tmem, 512);
}

// Joins the parts of the items that several CTAs share.  Grid (items, rows of an item / kJoinRows),
// 16 threads per row.
constexpr int kJoinRows = 16, kJoinThreads = 256;
template <int D>
__global__ void __launch_bounds__(kJoinThreads) join_kernel(const __grid_constant__ Args a) {
  using C = Cfg<D>;
  grid_dep_wait();
  grid_dep_launch();
  Item it;
  if (!find_item<D, kJoinThreads>(a, it, blockIdx.x, 0) || it.parts == 1) return;
  const int local = blockIdx.y * kJoinRows + threadIdx.x / 16, R = it.row0 + local;
  if (R >= it.sq.q_len * a.group) return;
  const int64_t first = int64_t(blockIdx.x) * a.splits * C::ROWS + local;
  float M = -INFINITY;
  for (int p = 0; p < it.parts; ++p) M = fmaxf(M, a.prompt_ml[first + int64_t(p) * C::ROWS].x);
  const float base = M == -INFINITY ? 0.0f : M;
  constexpr int N = D / 64;  // float4 per thread
  float l = 0.0f;
  float4 o[N];
#pragma unroll
  for (int n = 0; n < N; ++n) o[n] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 2
  for (int p = 0; p < it.parts; ++p) {
    const int64_t at = first + int64_t(p) * C::ROWS;
    const float2 ml = a.prompt_ml[at];
    const float f = ex2(ml.x - base);
    l = fmaf(ml.y, f, l);
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const float4 v = *reinterpret_cast<const float4 *>(a.prompt_part + at * D + 4 * (threadIdx.x % 16 + 16 * n));
      o[n].x = fmaf(v.x, f, o[n].x), o[n].y = fmaf(v.y, f, o[n].y), o[n].z = fmaf(v.z, f, o[n].z), o[n].w = fmaf(v.w, f, o[n].w);
    }
  }
  const float f = M == -INFINITY && l == l ? 0.0f : kSumUnit / l;  // no visible token, and no NaN score: 0
  const int64_t row = (it.sq.start + R / a.group) * a.ld_out + int64_t(it.h * a.group + R % a.group) * D;
#pragma unroll
  for (int n = 0; n < N; ++n) {
    const int64_t at = row + 4 * (threadIdx.x % 16 + 16 * n);
    if (a.out_fp32) {
      *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + at) = make_float4(o[n].x * f, o[n].y * f, o[n].z * f, o[n].w * f);
    } else {
      __nv_bfloat162 p[2] = {__floats2bfloat162_rn(o[n].x * f, o[n].y * f), __floats2bfloat162_rn(o[n].z * f, o[n].w * f)};
      *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.out) + at) = *reinterpret_cast<const uint2 *>(p);
    }
  }
}

}  // namespace prompt
}  // namespace attn
}  // namespace nvfp4

// Matrix-vector products with an NVFP4 weight and BF16 activations, for up to 16 tokens:
//     y[m, n] = sum_k x[m, k] e2m1(W[n, k]) e4m3(sf[n, k / 16]) / gs(seg(n)).
// Unlike the W4A4 linear nothing is quantised here: a code times its block scale has at
// most 6 significant bits and lies in FP16's range, so weights are exact FP16 operands of
// mma.m16n8k16; x is scaled by a power of two per (token, chunk of K) into FP16's range,
// which keeps all BF16 bits within 2^-29 of the chunk's largest value.  FP32 sums.
//
// Bound by HBM: 9/16 byte per weight, read once.  A CTA takes 128 weight rows (one atom row
// of the scale layout) and a K range, which a producer warp streams through a ring of stages
// of 256 columns (16 KB of codes by TMA, 2 KB of scales), so that up to 144 KB are on their way to an
// SM.  A lane reads 32 bytes, 64 consecutive columns, of two rows per stage, with their four scales in
// one word.  The contraction runs over columns in any order as long as W and x agree, so
// those 64 columns are the lane's values of 16 k-steps and need no shuffling.  The rows of a
// warp are 4 w + i + 32 j (i, j < 4), as the scale layout groups them; with the TMA's swizzle the
// reads of codes are free of bank conflicts.  x is converted once per CTA and chunk, into
// shared memory, the next chunk's loads in flight meanwhile.  When the row blocks alone do not
// fill the GPU, a cluster of CTAs splits K and adds its partial sums through distributed shared
// memory, in rank order.
//
// 34816 x 5120 at four tokens: 25.4 us, 3.9 TB/s; 5120 x 6144 at one token: 7.3 us, of which the weight's
// 17.7 MB take 2.7 us: launch, first loads and the cluster's sum are the rest.
#pragma once

#include "attn_decode.cuh"
#include "gemm.cuh"

namespace nvfp4 {
namespace matvec {

constexpr int kWarps = 8;                   // consumer warps
constexpr int kThreads = 32 * (kWarps + 1);  // and the producer
constexpr int kBN = 128;      // weight rows per CTA
constexpr int kChunk = 1024;  // columns of x staged at a time
constexpr int kStep = 256;    // columns of a stage
constexpr int kCodeBytes = kBN * kStep / 2, kScaleBytes = kBN * kStep / 16;

struct Args {
  const uint16_t *x;  // BF16 [M x ld_x]
  int64_t ld_x;
  int M;
  const uint8_t *scales;
  int64_t N, K;
  int64_t k_per_cta;  // multiple of kStep
  int nseg;
  gemm::Segment seg[16];
  void *out;
  int64_t ldo;
  int out_fp32;
};

// Eight codes of a word as four FP16 pairs.
__device__ __forceinline__ void e2m1x8_to_f16x8(uint32_t w, uint32_t (&v)[4]) {
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\t"
      "mov.b32 {b0, b1, b2, b3}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b0;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, b2;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, b3;\n\t}"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
      : "r"(w));
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

template <int NB>
struct Smem {
  static constexpr int kStages = NB == 1 ? 4 : 3;  // two CTAs fit an SM
  alignas(1024) unsigned char codes[kStages][kCodeBytes];
  alignas(128) unsigned char scales[kStages][kScaleBytes];
  // x chunk as FP16, token rows; the 16-byte pieces of lane q's 64 columns are permuted so
  // that the eight lanes of a quarter-warp hit distinct banks
  alignas(128) uint16_t x[8 * NB][kChunk];
  float scale[8 * NB];           // 2^e of each token's chunk
  float acc[kBN][8 * NB + 1];
  uint64_t full[kStages], empty[kStages];
};
template <int NB>
constexpr int smem_bytes() {
  return 1024 + int(sizeof(Smem<NB>));
}

// 16-byte piece p of a token's chunk.
__device__ __forceinline__ int piece(int tok, int p) {
  return (p & ~7) | ((p & 7) ^ (((p >> 3) & 3) | (tok & 1) << 2));
}

// One warp's tokens of an x chunk: loads, then conversion into shared memory.
template <int NB>
struct XChunk {
  static constexpr int T = NB;  // tokens per warp
  uint4 raw[T][4];

  __device__ __forceinline__ void load(const Args &a, int warp, int lane, int64_t k0, int64_t k_end) {
#pragma unroll
    for (int u = 0; u < T; ++u) {
      const int t = warp + kWarps * u;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t k = k0 + 8 * (lane + 32 * i);
        raw[u][i] = t < a.M && k < k_end ? __ldg(reinterpret_cast<const uint4 *>(a.x + t * a.ld_x + k)) : make_uint4(0, 0, 0, 0);
      }
    }
  }
  __device__ __forceinline__ void store(Smem<NB> &sm, int warp, int lane) const {
#pragma unroll
    for (int u = 0; u < T; ++u) {
      const int t = warp + kWarps * u;
      uint32_t top = 0;  // BF16 magnitudes order as integers, two at a time
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        top = __vmaxu2(__vmaxu2(top, raw[u][i].x & 0x7fff7fffu), raw[u][i].y & 0x7fff7fffu);
        top = __vmaxu2(__vmaxu2(top, raw[u][i].z & 0x7fff7fffu), raw[u][i].w & 0x7fff7fffu);
      }
      const uint32_t bits = __reduce_max_sync(0xffffffffu, max(top & 0xffffu, top >> 16)) << 16;
      // 2^-e brings the chunk's largest magnitude into [2^14, 2^15); an infinity counts as the
      // largest finite value, so that finite values stay finite next to it
      const int e = bits == 0 ? 0 : min(max(static_cast<int>(bits >> 23) - 127 - 14, -126), 113);
      const float f = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
      if (lane == 0) sm.scale[t] = __uint_as_float(static_cast<uint32_t>(127 + e) << 23);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t v[4] = {raw[u][i].x, raw[u][i].y, raw[u][i].z, raw[u][i].w};
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) o[j] = attn::pack_f16(__uint_as_float(v[j] << 16) * f, __uint_as_float(v[j] & 0xFFFF0000u) * f);
        *reinterpret_cast<uint4 *>(&sm.x[t][8 * piece(t, lane + 32 * i)]) = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
  }
};

// Grid: (row blocks * cluster size), cluster of CTAs along K.  NB: blocks of 8 tokens.
template <int NB>
__global__ void __launch_bounds__(kThreads, 2) matvec_kernel(const __grid_constant__ Args a, const __grid_constant__ CUtensorMap map) {
  constexpr int kStages = Smem<NB>::kStages;
  extern __shared__ unsigned char smem_raw[];
  Smem<NB> &sm = *reinterpret_cast<Smem<NB> *>(smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023));
  uint32_t nrank, rank = cluster_ctarank();
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(nrank));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int64_t n0 = int64_t(blockIdx.x / nrank) * kBN;
  const int64_t k_begin = rank * a.k_per_cta, k_end = min(a.K, k_begin + a.k_per_cta);
  const int steps = k_end > k_begin ? static_cast<int>((k_end - k_begin + kStep - 1) / kStep) : 0;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&sm.full[i], 1);
      mbar_init(&sm.empty[i], kWarps);
    }
    fence_barrier_init();
  }
  __syncthreads();
  grid_dep_wait();
  grid_dep_launch();

  bool ok = true;
  float acc[NB][4];
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[b][j] = 0.0f;

  if (warp == kWarps) {
    if (lane == 0) {
      const int64_t atoms = a.K / 64;
      const uint8_t *sf = a.scales + (n0 / 128) * atoms * 512;
      for (int i = 0; i < steps && ok; ++i) {
        const int st = i % kStages;
        ok = mbar_wait(&sm.empty[st], ((i / kStages) & 1) ^ 1);
        if (!ok) break;
        const int64_t k = k_begin + int64_t(i) * kStep;
        const uint32_t bytes = static_cast<uint32_t>(min(int64_t(4), atoms - k / 64)) * 512;
        mbar_arrive_expect_tx(&sm.full[st], kCodeBytes + bytes);
        tma_load_2d(sm.codes[st], &map, &sm.full[st], static_cast<int>(k / 2), static_cast<int>(n0));  // zeros outside W
        bulk_load(sm.scales[st], sf + (k / 64) * 512, bytes, &sm.full[st]);
      }
    }
  } else {
    // this lane's two weight rows: mma rows g and g + 8
    int row[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) row[r] = 4 * warp + (g & 3) + 32 * ((g >> 2) + 2 * r);
    const bool have[2] = {n0 + row[0] < a.N, n0 + row[1] < a.N};
    XChunk<NB> x;
    x.load(a, warp, lane, k_begin, k_end);
    constexpr int kPerChunk = kChunk / kStep;
    for (int i0 = 0; i0 < steps; i0 += kPerChunk) {  // to the end even if a wait ran out: others wait here
      x.store(sm, warp, lane);
      asm volatile("bar.sync 1, 256;" ::: "memory");  // consumer warps
      if (i0 + kPerChunk < steps) x.load(a, warp, lane, k_begin + int64_t(i0 + kPerChunk) * kStep, k_end);
      float c[NB][2][4];  // two chains: even and odd k-steps
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int j = 0; j < 8; ++j) c[b][j >> 2][j & 3] = 0.0f;
#pragma unroll 1
      for (int s = 0; s < kPerChunk && i0 + s < steps; ++s) {
        const int i = i0 + s, st = i % kStages;
        ok = ok && mbar_wait(&sm.full[st], (i / kStages) & 1);
        const bool inside = k_begin + int64_t(i) * kStep + 64 * q < k_end;
        uint32_t w[2][8], sc[2][4];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const unsigned char *src = sm.codes[st] + row[r] * 128;
          const uint4 lo = *reinterpret_cast<const uint4 *>(src + (((2 * q) ^ (row[r] & 7)) << 4));
          const uint4 hi = *reinterpret_cast<const uint4 *>(src + (((2 * q + 1) ^ (row[r] & 7)) << 4));
          w[r][0] = lo.x, w[r][1] = lo.y, w[r][2] = lo.z, w[r][3] = lo.w;
          w[r][4] = hi.x, w[r][5] = hi.y, w[r][6] = hi.z, w[r][7] = hi.w;
          uint32_t f = *reinterpret_cast<const uint32_t *>(sm.scales[st] + 512 * q + (row[r] & 31) * 16 + (row[r] >> 5) * 4);
          if (!(have[r] && inside)) f = 0;  // padding's scales may be anything
          uint32_t a0, a1;
          attn::e4m3x4_to_f16x4(f, a0, a1);
          sc[r][0] = __byte_perm(a0, a0, 0x1010);
          sc[r][1] = __byte_perm(a0, a0, 0x3232);
          sc[r][2] = __byte_perm(a1, a1, 0x1010);
          sc[r][3] = __byte_perm(a1, a1, 0x3232);
        }
#pragma unroll
        for (int n = 0; n < 8; ++n) {  // word n: k-steps 2 n, 2 n + 1, group n / 2
          uint4 xb[NB];
#pragma unroll
          for (int b = 0; b < NB; ++b)
            xb[b] = *reinterpret_cast<const uint4 *>(&sm.x[8 * b + g][8 * piece(g, s * 32 + q * 8 + n)]);
          uint32_t v[2][4];
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            e2m1x8_to_f16x8(w[r][n], v[r]);
#pragma unroll
            for (int j = 0; j < 4; ++j) v[r][j] = mul_f16x2(v[r][j], sc[r][n >> 1]);
          }
#pragma unroll
          for (int b = 0; b < NB; ++b) {
            attn::mma_f16(c[b][0], v[0][0], v[1][0], v[0][1], v[1][1], xb[b].x, xb[b].y);
            attn::mma_f16(c[b][1], v[0][2], v[1][2], v[0][3], v[1][3], xb[b].z, xb[b].w);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.empty[st]);
      }
      // accumulator j: row g + 8 (j / 2), token 2 q + j % 2
#pragma unroll
      for (int b = 0; b < NB; ++b)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          acc[b][j] = fmaf(c[b][0][j] + c[b][1][j], sm.scale[8 * b + 2 * q + (j & 1)], acc[b][j]);
      asm volatile("bar.sync 1, 256;" ::: "memory");  // x is staged again
    }
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        sm.acc[row[j >> 1]][8 * b + 2 * q + (j & 1)] = acc[b][j];
  }
  __syncwarp();
  cluster_sync();

  // rank r adds its share of the rows of all the cluster's partial sums
  const int per = (kBN + nrank - 1) / nrank;
  for (int idx = threadIdx.x; idx < per * a.M; idx += kThreads) {
    const int t = idx / per, local = static_cast<int>(rank) * per + idx % per;
    const int64_t n = n0 + local;
    if (local >= kBN || n >= a.N) continue;
    float y = 0.0f;
    for (uint32_t r = 0; r < nrank; ++r) {
      float v;
      asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(mapa_shared(smem_u32(&sm.acc[local][t]), r)));
      y += v;
    }
    const float *gs = a.seg[0].gs_w;
    for (int i = 1; i < a.nseg; ++i)
      if (n >= a.seg[i].n_begin) gs = a.seg[i].gs_w;
    y = __fdiv_rn(y, __ldg(gs));
    if (a.out_fp32)
      static_cast<float *>(a.out)[t * a.ldo + n] = y;
    else
      static_cast<__nv_bfloat16 *>(a.out)[t * a.ldo + n] = __float2bfloat16_rn(y);
  }
  cluster_sync();  // no CTA leaves while another reads its shared memory
}

}  // namespace matvec
}  // namespace nvfp4

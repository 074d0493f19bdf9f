// Matrix-vector products with an NVFP4 weight and BF16 activations, for up to 16 tokens:
//     y[m, n] = sum_k x[m, k] e2m1(W[n, k]) e4m3(sf[n, k / 16]) / gs(seg(n)).
// Unlike the W4A4 linear nothing is quantised here: a code times its block scale has at
// most 6 significant bits and lies in FP16's range, so weights are exact FP16 operands of
// mma.m16n8k16; x is scaled by a power of two per (token, chunk of K) into FP16's range,
// which keeps all BF16 bits within 2^-29 of the chunk's largest value.  FP32 sums.
//
// Bound by HBM: 9/16 byte per weight, read once.  A CTA takes 128 weight rows (one atom row
// of the scale layout) and a K range; a lane reads 32 bytes of two rows per step, 64
// consecutive columns, with their four scales in one word.  The contraction runs over
// columns in any order as long as W and x agree, so those 64 columns are the lane's values
// of 16 k-steps and need no shuffling.  The rows of a warp are 4 w + i + 32 j (i, j < 4): their
// scale words fill whole 16-byte pieces.  x is converted once per CTA and chunk, into
// shared memory.  When the row blocks alone do not fill the GPU, a cluster of CTAs splits K
// and adds its partial sums through distributed shared memory, in rank order.
#pragma once

#include "attn_decode.cuh"
#include "gemm.cuh"

namespace nvfp4 {
namespace matvec {

constexpr int kWarps = 8;
constexpr int kThreads = 32 * kWarps;
constexpr int kBN = 128;      // weight rows per CTA
constexpr int kChunk = 1024;  // columns of x staged at a time
constexpr int kStep = 256;    // columns of a warp's step

struct Args {
  const uint16_t *x;  // BF16 [M x ld_x]
  int64_t ld_x;
  int M;
  const uint8_t *codes, *scales;
  int64_t N, K;
  int64_t k_per_cta;  // multiple of kChunk
  int nseg;
  gemm::Segment seg[16];
  void *out;
  int64_t ldo;
  int out_fp32;
};

__device__ __forceinline__ uint32_t e2m1x2_to_f16x2(uint32_t byte) {
  uint32_t r;
  asm("{\n\t.reg .b8 b, z0, z1, z2;\n\t"
      "mov.b32 {b, z0, z1, z2}, %1;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, b;\n\t}"
      : "=r"(r)
      : "r"(byte));
  return r;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// 32 bytes through one load.
struct W32 {
  uint32_t w[8];
};
__device__ __forceinline__ W32 ld_w32(const uint8_t *p) {
  W32 r;
  asm volatile("ld.global.nc.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]), "=r"(r.w[4]), "=r"(r.w[5]), "=r"(r.w[6]),
                 "=r"(r.w[7])
               : "l"(p));
  return r;
}

template <int NB>
struct Smem {
  // x chunk as FP16, token rows; the 16-byte pieces of lane q's 64 columns are permuted so
  // that the eight lanes of a quarter-warp hit distinct banks
  alignas(128) uint16_t x[8 * NB][kChunk];
  float scale[8 * NB];           // 2^e of each token's chunk
  float acc[kBN][8 * NB + 1];
};

// 16-byte piece p of a token's chunk.
__device__ __forceinline__ int piece(int tok, int p) {
  return (p & ~7) | ((p & 7) ^ (((p >> 3) & 3) | (tok & 1) << 2));
}

// Grid: (row blocks * cluster size), cluster of CTAs along K.  NB: blocks of 8 tokens.
template <int NB>
__global__ void __launch_bounds__(kThreads) matvec_kernel(const __grid_constant__ Args a) {
  extern __shared__ __align__(128) unsigned char smem_raw[];
  Smem<NB> &sm = *reinterpret_cast<Smem<NB> *>(smem_raw);
  grid_dep_wait();
  grid_dep_launch();
  uint32_t nrank, rank = cluster_ctarank();
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(nrank));
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, q = lane & 3;
  const int64_t n0 = int64_t(blockIdx.x / nrank) * kBN;
  const int64_t k_begin = rank * a.k_per_cta, k_end = min(a.K, k_begin + a.k_per_cta);

  // this lane's two weight rows: mma rows g and g + 8
  int64_t row[2];
  const uint8_t *wp[2], *sp[2];
  const int64_t kb_atoms = a.K / 64;
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int local = 4 * warp + (g & 3) + 32 * ((g >> 2) + 2 * r);
    row[r] = n0 + local;
    wp[r] = a.codes + row[r] * (a.K / 2) + 32 * q;
    sp[r] = a.scales + scale_word_offset(row[r], q, kb_atoms);
  }
  float acc[NB][4];
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[b][j] = 0.0f;

  auto load_step = [&](int64_t k, W32 (&w)[2], uint32_t (&s)[2]) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const bool ok = row[r] < a.N && k + 64 * q < k_end;
      s[r] = ok ? __ldg(reinterpret_cast<const uint32_t *>(sp[r] + (k / 64) * 512)) : 0u;
      if (ok) {
        w[r] = ld_w32(wp[r] + k / 2);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[r].w[i] = 0;
      }
    }
  };

  W32 w[2];
  uint32_t s[2];
  load_step(k_begin, w, s);
  for (int64_t k0 = k_begin; k0 < k_end; k0 += kChunk) {
    // stage x: a warp takes whole tokens, 32 columns a lane
    for (int t = warp; t < 8 * NB; t += kWarps) {
      uint4 raw[4];
      float amax = 0.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t k = k0 + 8 * (lane + 32 * i);
        raw[i] = t < a.M && k < k_end ? __ldg(reinterpret_cast<const uint4 *>(a.x + t * a.ld_x + k)) : make_uint4(0, 0, 0, 0);
        const uint32_t v[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          amax = fmaxf(amax, fmaxf(fabsf(__uint_as_float(v[j] << 16)), fabsf(__uint_as_float(v[j] & 0xFFFF0000u))));
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
      const int e = attn::row_exponent(amax);
      const float f0 = ldexpf(1.0f, -(e / 2)), f1 = ldexpf(1.0f, -(e - e / 2));
      if (lane == 0) sm.scale[t] = ldexpf(1.0f, e);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t v[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
        uint32_t o[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          o[j] = attn::pack_f16(__uint_as_float(v[j] << 16) * f0 * f1, __uint_as_float(v[j] & 0xFFFF0000u) * f0 * f1);
        *reinterpret_cast<uint4 *>(&sm.x[t][8 * piece(t, lane + 32 * i)]) = make_uint4(o[0], o[1], o[2], o[3]);
      }
    }
    __syncthreads();
    float c[NB][2][4];  // two chains: even and odd k-steps
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int j = 0; j < 8; ++j) c[b][j >> 2][j & 3] = 0.0f;
#pragma unroll
    for (int st = 0; st < kChunk / kStep; ++st) {
      const int64_t k = k0 + st * kStep;
      if (k >= k_end) break;
      W32 nw[2];
      uint32_t ns[2];
      load_step(k + kStep, nw, ns);  // next step, possibly of the next chunk
      uint32_t sc[2][4];  // the four scales of each row, twice each
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const uint32_t lo = attn::e4m3x2_to_f16x2(s[r]), hi = attn::e4m3x2_to_f16x2(s[r] >> 16);
        sc[r][0] = __byte_perm(lo, lo, 0x1010);
        sc[r][1] = __byte_perm(lo, lo, 0x3232);
        sc[r][2] = __byte_perm(hi, hi, 0x1010);
        sc[r][3] = __byte_perm(hi, hi, 0x3232);
      }
#pragma unroll
      for (int i = 0; i < 8; ++i) {  // word i: k-steps 2 i, 2 i + 1, group i / 2
        uint4 xb[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b)
          xb[b] = *reinterpret_cast<const uint4 *>(&sm.x[8 * b + g][8 * piece(g, st * 32 + q * 8 + i)]);
        uint32_t v[2][4];
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
          for (int j = 0; j < 4; ++j) v[r][j] = mul_f16x2(e2m1x2_to_f16x2(w[r].w[i] >> (8 * j)), sc[r][i >> 1]);
#pragma unroll
        for (int b = 0; b < NB; ++b) {
          attn::mma_f16(c[b][0], v[0][0], v[1][0], v[0][1], v[1][1], xb[b].x, xb[b].y);
          attn::mma_f16(c[b][1], v[0][2], v[1][2], v[0][3], v[1][3], xb[b].z, xb[b].w);
        }
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        w[r] = nw[r];
        s[r] = ns[r];
      }
    }
    // accumulator j: row g + 8 (j / 2), token 2 q + j % 2
#pragma unroll
    for (int b = 0; b < NB; ++b)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        acc[b][j] = fmaf(c[b][0][j] + c[b][1][j], sm.scale[8 * b + 2 * q + (j & 1)], acc[b][j]);
    __syncthreads();  // x is staged again
  }
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      sm.acc[4 * warp + (g & 3) + 32 * ((g >> 2) + 2 * (j >> 1))][8 * b + 2 * q + (j & 1)] = acc[b][j];
  cluster_sync();

  // rank r adds rows [r, r + 1) * 128 / nrank of all the cluster's partial sums
  const int per = kBN / nrank;
  for (int idx = threadIdx.x; idx < per * a.M; idx += kThreads) {
    const int t = idx / per, local = static_cast<int>(rank) * per + idx % per;
    const int64_t n = n0 + local;
    if (n >= a.N) continue;
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

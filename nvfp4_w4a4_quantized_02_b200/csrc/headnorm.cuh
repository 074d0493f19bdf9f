// RMS norm of every query and key head with the position rotation, in one pass over the
// projection's output:
//     y = x / sqrt(mean(x^2) + eps) * (offset + w)          per head of D values
//     (y_a, y_b) <- (y_a c - y_b s, y_b c + y_a s)          for the first R values,
// with (a, b) = (i, i + R/2) or, interleaved, (2i, 2i + 1), and c, s the cosine and sine of
// the token's position from an FP32 table.  FP32 throughout, one rounding to BF16.
//
// HBM-bound: 2 bytes read and 2 written per element.  A lane holds 8 consecutive values
// (16 bytes), D / 8 lanes a head, a warp 256 / D heads at a time; sums and the halves of
// a rotated pair travel by shuffles (the raw BF16 words of the partner lane: four
// shuffles instead of eight).  A warp takes a run of one token's heads and forms the products of
// norm weight and rotation once, y = (x (w c) + x_partner (w_partner s)) / rms, which leaves three
// packed FP32 operations per pair of values; kDepth heads' loads are in flight.  32768 tokens of 48 + 8
// heads of 128 values, 64 rotated: 164 us, 5.8 TB/s (273 us with the rotation after the norm and one head at
// a time); 32 tokens: 3 us, the latency of one launch.
#pragma once

#include "gdn.cuh"

namespace nvfp4 {
namespace headnorm {

constexpr int kThreads = 128;
constexpr int kDepth = 4;  // head groups loaded before any is computed

struct Args {
  const uint16_t *q, *k;   // BF16 rows, head h at column h * D
  int64_t ld_q, ld_k;
  int64_t tokens;
  int heads, kv_heads;
  const uint16_t *w_q, *w_k;  // BF16 [D]
  float w_offset, eps;
  const int64_t *positions;   // [tokens]
  const float *table;         // [max_pos][R]: R/2 cosines, then R/2 sines
  int64_t max_pos;
  int rot;                    // R
  int interleaved;
  uint16_t *q_out, *k_out;
  int64_t ld_qo, ld_ko;
  int parts;                  // warps per token
  int per_part;               // head groups per warp
};

__device__ __forceinline__ void unpack8(const uint4 &w, float2 (&f)[4]) {
  const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) f[i] = make_float2(__uint_as_float(x[i] << 16), __uint_as_float(x[i] & 0xFFFF0000u));
}

template <int LANES>
__device__ __forceinline__ float group_sum(float x) {
#pragma unroll
  for (int o = 1; o < LANES; o <<= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}
template <int LANES>
__device__ __forceinline__ float group_max(float x) {
#pragma unroll
  for (int o = 1; o < LANES; o <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, o));
  return x;
}

// 1 / sqrt(x) to 2 ulp, for normal x.
__device__ __forceinline__ float rsqrt_approx(float x) {
  float r;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

template <int D>
__device__ __forceinline__ float sum_squares(const float2 (&x)[4]) {
  float2 s = make_float2(0.0f, 0.0f);
#pragma unroll
  for (int i = 0; i < 4; ++i) s = gdn::ffma2(x[i], x[i], s);
  return group_sum<D / 8>(s.x + s.y);
}

// Whether a sum of squares left FP32's range, or lost bits below it that eps does not outweigh.
__device__ __forceinline__ bool outside(float ss, float eps) { return !(ss <= 1e37f) || (ss < 1e-30f && eps < 1e-25f); }

// 1 / sqrt(mean(x^2) + eps) of such a head: of x scaled by a power of two, by which x and its
// partner's values p are then scaled too.
template <int D>
__device__ __forceinline__ float careful_inv_rms(float2 (&x)[4], float2 (&p)[4], float eps) {
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = fmaxf(m, fmaxf(fabsf(x[i].x), fabsf(x[i].y)));
  m = group_max<D / 8>(m);
  if (m > 0.0f && m <= 3.4e38f) {
    int e;
    frexpf(m, &e);
    e = max(e, -90);
    const float f = ldexpf(1.0f, -e);
    eps = ldexpf(eps, -2 * e);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = gdn::fmul2(x[i], make_float2(f, f));
      p[i] = gdn::fmul2(p[i], make_float2(f, f));
    }
  }
  return rsqrtf(sum_squares<D>(x) * (1.0f / D) + eps);
}

template <int D>
__global__ void __launch_bounds__(kThreads) head_norm_kernel(const __grid_constant__ Args a) {
  constexpr int LANES = D / 8, HPW = 32 / LANES;  // lanes per head, heads per warp
  grid_dep_wait();
  grid_dep_launch();
  const int64_t wid = (int64_t(blockIdx.x) * kThreads + threadIdx.x) >> 5;
  const int64_t tok = wid / a.parts;
  const int part = static_cast<int>(wid - tok * a.parts);
  if (tok >= a.tokens) return;  // whole warps
  const int lane = threadIdx.x & 31, sub = lane / LANES, l = lane % LANES;
  // head groups of this warp: [g_begin, g_end) of q's groups followed by k's
  const int q_groups = (a.heads + HPW - 1) / HPW, groups = q_groups + (a.kv_heads + HPW - 1) / HPW;
  const int g_begin = part * a.per_part, g_end = min(groups, g_begin + a.per_part);
  if (g_begin >= groups) return;

  const int64_t pos = a.rot ? __ldg(a.positions + tok) : 0;
  if (pos < 0 || pos >= a.max_pos) {  // no such row in the table: the token is left alone
    if (lane == 0) record_bad_index();
    return;
  }

  // The lane's 8 values: y = (x * A + p * B) / rms with A = w c, B = w_partner s, the sign in s.
  const int first = 8 * l, half = a.rot / 2;
  const bool rotated = first < a.rot;
  int partner = lane;
  if (rotated && !a.interleaved) partner = first >= half ? lane - half / 8 : lane + half / 8;
  float2 A[4], B[4];
  auto load_factors = [&](const uint16_t *src) {
    float2 w[4], wp[4];
    unpack8(__ldg(reinterpret_cast<const uint4 *>(src + first)), w);
    unpack8(__ldg(reinterpret_cast<const uint4 *>(src + 8 * (partner % LANES))), wp);
    const float2 off = make_float2(a.w_offset, a.w_offset);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      A[i] = add_f32x2(w[i], off);
      wp[i] = add_f32x2(wp[i], off);
      B[i] = make_float2(0.0f, 0.0f);
    }
    if (!rotated) return;
    const float *row = a.table + pos * a.rot;
    if (a.interleaved) {  // values 2 i and 2 i + 1 are a pair
      const float4 c4 = __ldg(reinterpret_cast<const float4 *>(row + first / 2));
      const float4 s4 = __ldg(reinterpret_cast<const float4 *>(row + half + first / 2));
      const float c[4] = {c4.x, c4.y, c4.z, c4.w}, s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        B[i] = make_float2(A[i].y * -s[i], A[i].x * s[i]);
        A[i] = make_float2(A[i].x * c[i], A[i].y * c[i]);
      }
    } else {
      const bool upper = first >= half;
      const float *at = row + (upper ? first - half : first);
      const float sg = upper ? 1.0f : -1.0f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 c = __ldg(reinterpret_cast<const float2 *>(at) + i), s = __ldg(reinterpret_cast<const float2 *>(at + half) + i);
        A[i] = gdn::fmul2(A[i], c);
        B[i] = gdn::fmul2(wp[i], make_float2(sg * s.x, sg * s.y));
      }
    }
  };
  auto expand = [&](const uint4 &raw, float2 (&x)[4], float2 (&p)[4]) {
    unpack8(raw, x);
    if (a.interleaved) {
#pragma unroll
      for (int i = 0; i < 4; ++i) p[i] = rotated ? make_float2(x[i].y, x[i].x) : x[i];  // no factor 0 on another value
    } else {
      uint4 o;
      o.x = __shfl_sync(0xffffffffu, raw.x, partner);
      o.y = __shfl_sync(0xffffffffu, raw.y, partner);
      o.z = __shfl_sync(0xffffffffu, raw.z, partner);
      o.w = __shfl_sync(0xffffffffu, raw.w, partner);
      unpack8(o, p);
    }
  };
  auto store = [&](uint16_t *to, const float2 (&x)[4], const float2 (&p)[4], float inv) {
    uint32_t out[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 y = gdn::fmul2(gdn::ffma2(x[i], A[i], gdn::fmul2(p[i], B[i])), make_float2(inv, inv));
      const __nv_bfloat162 b = __floats2bfloat162_rn(y.x, y.y);
      out[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
    *reinterpret_cast<uint4 *>(to) = make_uint4(out[0], out[1], out[2], out[3]);
  };
  // Groups [g0, g1) of one operand: head g * HPW + sub of `heads`, rows `from` / `to` at the lane's values.
  auto run = [&](const uint16_t *from, uint16_t *to, const uint16_t *w, int heads, int g0, int g1) {
    if (g0 >= g1) return;
    load_factors(w);
    from += (g0 * HPW + sub) * D;
    to += (g0 * HPW + sub) * D;
    const int count = g1 - g0, n = min(g1 * HPW, heads) - (g0 * HPW + sub);  // heads left, from this lane's first on
#pragma unroll 1
    for (int c0 = 0; c0 < count; c0 += 32) {
      uint32_t odd = 0;  // bit i: this lane's head of group c0 + i has squares outside FP32's range and is left as it was
#pragma unroll 1
      for (int g = c0; g < min(count, c0 + 32); g += kDepth) {
        const uint16_t *src = from + g * HPW * D;
        uint16_t *dst = to + g * HPW * D;
        uint4 raw[kDepth];
#pragma unroll
        for (int u = 0; u < kDepth; ++u) {  // `to` may be `from`: no read-only path
          raw[u] = make_uint4(0, 0, 0, 0);
          if ((g + u) * HPW < n) raw[u] = *reinterpret_cast<const uint4 *>(src + u * HPW * D);
        }
#pragma unroll
        for (int u = 0; u < kDepth; ++u) {
          float2 x[4], p[4];
          expand(raw[u], x, p);
          const float ss = sum_squares<D>(x);
          if ((g + u) * HPW < n) {
            if (outside(ss, a.eps)) odd |= 1u << (g - c0 + u);
            else store(dst + u * HPW * D, x, p, rsqrt_approx(ss * (1.0f / D) + a.eps));
          }
        }
      }
      if (!__any_sync(0xffffffffu, odd)) continue;
#pragma unroll 1
      for (int i = 0; i < 32; ++i) {
        const bool again = (odd >> i) & 1;
        if (!__any_sync(0xffffffffu, again)) continue;
        float2 x[4], p[4];
        expand(again ? *reinterpret_cast<const uint4 *>(from + (c0 + i) * HPW * D) : make_uint4(0, 0, 0, 0), x, p);
        const float inv = careful_inv_rms<D>(x, p, a.eps);
        if (again) store(to + (c0 + i) * HPW * D, x, p, inv);
      }
    }
  };
  run(a.q + tok * a.ld_q + first, a.q_out + tok * a.ld_qo + first, a.w_q, a.heads, g_begin, min(g_end, q_groups));
  run(a.k + tok * a.ld_k + first, a.k_out + tok * a.ld_ko + first, a.w_k, a.kv_heads, max(g_begin, q_groups) - q_groups, g_end - q_groups);
}

// table[p][i] = cos(p base^(-2i/R)), table[p][R/2 + i] = sin of the same, i < R/2.  FP64:
// an FP32 angle is off by 2^-24 of itself, radians at far positions.
constexpr int kTableThreads = 128;
__global__ void __launch_bounds__(kTableThreads) rope_table_kernel(float *table, int64_t max_pos, int rot, double base) {
  grid_dep_wait();
  grid_dep_launch();
  const int half = rot / 2;
  const int64_t n = max_pos * half;
  for (int64_t i = int64_t(blockIdx.x) * kTableThreads + threadIdx.x; i < n; i += int64_t(gridDim.x) * kTableThreads) {
    const int64_t p = i / half;
    const int j = static_cast<int>(i - p * half);
    double s, c;
    sincos(double(p) * pow(base, -2.0 * j / rot), &s, &c);
    table[p * rot + j] = static_cast<float>(c);
    table[p * rot + half + j] = static_cast<float>(s);
  }
}

}  // namespace headnorm
}  // namespace nvfp4

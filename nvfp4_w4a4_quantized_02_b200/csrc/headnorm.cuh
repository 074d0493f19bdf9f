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
// shuffles instead of eight).  A warp takes a run of one token's heads, so that the
// table row and the norm weights are loaded once, with four heads' loads in flight.
#pragma once

#include "ptx.cuh"

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

__device__ __forceinline__ void unpack8(const uint4 &w, float (&f)[8]) {
  const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(x[i] << 16);
    f[2 * i + 1] = __uint_as_float(x[i] & 0xFFFF0000u);
  }
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

// 1 / sqrt(mean(x^2) + eps) times 2^-e in `inv`, and 2^e's inverse already in x: squares
// that leave FP32's range are taken of x scaled by a power of two instead.
template <int D>
__device__ __forceinline__ float inv_rms(float (&x)[8], float (&p)[8], float eps) {
  constexpr int LANES = D / 8;
  float ss = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
  ss = group_sum<LANES>(ss);
  const bool odd = ss > 1e37f || ss < 1e-30f;
  if (__any_sync(0xffffffffu, odd)) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = fmaxf(m, fabsf(x[i]));
    m = group_max<LANES>(m);
    // with an eps that outweighs them, tiny squares need no care
    if (odd && m > 0.0f && m <= 3.4e38f && (m > 1.0f || eps < 1e-25f)) {
      int e;
      frexpf(m, &e);
      e = max(e, -90);
      const float f = ldexpf(1.0f, -e);
      float s2 = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[i] *= f;
        p[i] *= f;
        s2 = fmaf(x[i], x[i], s2);
      }
      ss = s2;
      eps = ldexpf(eps, -2 * e);
    } else if (odd) {
      ss = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
    }
    // every lane takes part; a group that was fine sums to what it had
    const float again = group_sum<LANES>(odd ? ss : 0.0f);
    if (odd) ss = again;
  }
  return 1.0f / sqrtf(ss * (1.0f / D) + eps);
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
  const int total = a.heads + a.kv_heads;
  const int h_begin = part * a.per_part * HPW, h_end = min(total, h_begin + a.per_part * HPW);
  if (h_begin >= total) return;

  const int64_t pos = a.rot ? __ldg(a.positions + tok) : 0;
  if (pos < 0 || pos >= a.max_pos) {  // no such row in the table: the token is left alone
    if (lane == 0) record_bad_index();
    return;
  }

  // Rotation of the lane's 8 values: y = n * c + n_partner * s, with the sign in s.
  float c[8], s[8];
  const int first = 8 * l, half = a.rot / 2;
  const bool rotated = first < a.rot;
  int partner = lane;
  if (rotated) {
    const float *row = a.table + pos * a.rot;
    if (a.interleaved) {
      const float4 cc = __ldg(reinterpret_cast<const float4 *>(row + first / 2));
      const float4 ss = __ldg(reinterpret_cast<const float4 *>(row + half + first / 2));
      const float c4[4] = {cc.x, cc.y, cc.z, cc.w}, s4[4] = {ss.x, ss.y, ss.z, ss.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        c[2 * i] = c[2 * i + 1] = c4[i];
        s[2 * i] = -s4[i];
        s[2 * i + 1] = s4[i];
      }
    } else {
      const bool upper = first >= half;
      const int at = upper ? first - half : first;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float4 cc = __ldg(reinterpret_cast<const float4 *>(row + at) + i);
        const float4 ss = __ldg(reinterpret_cast<const float4 *>(row + half + at) + i);
        const float sg = upper ? 1.0f : -1.0f;
        c[4 * i] = cc.x, c[4 * i + 1] = cc.y, c[4 * i + 2] = cc.z, c[4 * i + 3] = cc.w;
        s[4 * i] = sg * ss.x, s[4 * i + 1] = sg * ss.y, s[4 * i + 2] = sg * ss.z, s[4 * i + 3] = sg * ss.w;
      }
      partner = upper ? lane - half / 8 : lane + half / 8;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      c[i] = 1.0f;
      s[i] = 0.0f;
    }
  }
  const int pl = 8 * (partner % LANES);  // the partner's first value

  // The weights change once, between the last query head and the first key head.
  float w[8], wp[8];
  bool have_k = false;
  auto load_weights = [&](const uint16_t *src) {
    unpack8(__ldg(reinterpret_cast<const uint4 *>(src + first)), w);
    unpack8(__ldg(reinterpret_cast<const uint4 *>(src + pl)), wp);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      w[i] += a.w_offset;
      wp[i] += a.w_offset;
    }
  };
  load_weights(h_begin + sub < a.heads ? a.w_q : a.w_k);
  have_k = h_begin + sub >= a.heads;

  for (int h0 = h_begin; h0 < h_end; h0 += kDepth * HPW) {
    uint4 raw[kDepth];
#pragma unroll
    for (int u = 0; u < kDepth; ++u) {
      const int h = h0 + u * HPW + sub;
      raw[u] = make_uint4(0, 0, 0, 0);
      if (h < h_end) {
        const uint16_t *src = h < a.heads ? a.q + tok * a.ld_q + int64_t(h) * D : a.k + tok * a.ld_k + int64_t(h - a.heads) * D;
        raw[u] = *reinterpret_cast<const uint4 *>(src + first);  // q_out may be q itself: no read-only path
      }
    }
#pragma unroll
    for (int u = 0; u < kDepth; ++u) {
      if (h0 + u * HPW >= h_end) break;  // uniform over the warp
      const int h = h0 + u * HPW + sub;
      float x[8], p[8];
      unpack8(raw[u], x);
      if (a.interleaved) {
#pragma unroll
        for (int i = 0; i < 8; ++i) p[i] = x[i ^ 1];
      } else {
        uint4 o;
        o.x = __shfl_sync(0xffffffffu, raw[u].x, partner);
        o.y = __shfl_sync(0xffffffffu, raw[u].y, partner);
        o.z = __shfl_sync(0xffffffffu, raw[u].z, partner);
        o.w = __shfl_sync(0xffffffffu, raw[u].w, partner);
        unpack8(o, p);
      }
      const float inv = inv_rms<D>(x, p, a.eps);
      if (h >= a.heads && !have_k) {
        load_weights(a.w_k);
        have_k = true;
      }
      uint32_t out[4];
#pragma unroll
      for (int i = 0; i < 8; i += 2) {
        float y[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float n = x[i + j] * inv * w[i + j];
          if (rotated) {
            const float np = p[i + j] * inv * (a.interleaved ? w[(i + j) ^ 1] : wp[i + j]);
            y[j] = fmaf(n, c[i + j], np * s[i + j]);
          } else {
            y[j] = n;
          }
        }
        const __nv_bfloat162 b = __floats2bfloat162_rn(y[0], y[1]);
        out[i / 2] = *reinterpret_cast<const uint32_t *>(&b);
      }
      if (h < h_end) {
        uint16_t *dst = h < a.heads ? a.q_out + tok * a.ld_qo + int64_t(h) * D
                                    : a.k_out + tok * a.ld_ko + int64_t(h - a.heads) * D;
        *reinterpret_cast<uint4 *>(dst + first) = make_uint4(out[0], out[1], out[2], out[3]);
      }
    }
  }
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

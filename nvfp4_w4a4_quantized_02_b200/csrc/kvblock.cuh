// Append of new K and V rows to a paged 8-bit cache with one scale per (block of tokens,
// kv head).  The scale is the smallest power of two s with 448 s >= max|x| over the block's
// tokens: for a floating code a power of two costs no precision (only range below the
// block's maximum), quantising x / s rounds once, and when later tokens of a block need a
// larger scale, the earlier codes move by an exact factor: only values that become
// subnormal round again.
//
// HBM-bound: 2 bytes read and 1 written per new element.  A CTA owns one (touched block,
// kv head) of K or of V: it reads the block's new rows once into registers, takes their
// maximum, settles the scale and writes the codes; the codes of earlier tokens in the block
// are read and rewritten only when the scale grows.  The touched blocks are found on
// the device: sequence s gets the slots from cu[s] / B + 2 s on, at least as many as blocks
// that cu[s + 1] - cu[s] tokens can touch.  8 sequences of 4096 new tokens, 8 heads of 128 values: 38 us,
// 5.3 TB/s; one new token in each of 32 sequences: 4.6 us, latency.
#pragma once

#include "batch.cuh"
#include "ptx.cuh"

namespace nvfp4 {
namespace kvblock {

constexpr int kMinExp = -100;  // exponent of the smallest scale

struct Args {
  const uint16_t *k, *v;      // BF16 [tokens x ld], head h at column h * D
  int64_t ld_k, ld_v;
  const int32_t *cu_seqlens;  // [n_seqs + 1]
  const int32_t *kv_lens;     // [n_seqs], the new tokens included
  int64_t tokens;
  int n_seqs;
  int kv_heads, log_d;
  const int32_t *table;
  int64_t ld_table, max_kv;
  uint8_t *k_cache, *v_cache;  // [num_blocks][kv_heads][B][D]
  float *k_scales, *v_scales;  // [num_blocks][kv_heads]
  int64_t num_blocks;
  int log_block;
};

// Smallest power of two s >= 2^kMinExp with 448 s >= amax, for a finite FP32 amax >= 0 that
// is a BF16 value: 448 = 1.75 * 2^8.
__device__ __forceinline__ float pow2_scale(float amax) {
  const uint32_t b = __float_as_uint(amax);
  const int e = static_cast<int>(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
  return __uint_as_float(static_cast<uint32_t>(max(e, kMinExp) + 127) << 23);
}

// Whether `slot` is one of sequence s with the bounds c0, c1.
__device__ __forceinline__ bool holds(int64_t slot, int s, int64_t c0, int64_t c1, int log_block) {
  return (c0 >> log_block) + 2 * int64_t(s) <= slot && slot < (c1 >> log_block) + 2 * int64_t(s + 1);
}

// The sequence that has `slot`, where the bounds of some do not count: their slots may overlap others'.
template <int THREADS>
__device__ __noinline__ void find_slot(const Args &a, int64_t slot, int &s_seq) {
  __shared__ int s_bound[THREADS / 32];
  if (threadIdx.x == 0) s_seq = -1;
  int high = 0;
  for (int s0 = 0; s0 < a.n_seqs; s0 += THREADS) {
    const int s = s0 + threadIdx.x;
    const bool have = s < a.n_seqs;
    const int64_t c0 = have ? __ldg(a.cu_seqlens + s) : 0, c1 = have ? __ldg(a.cu_seqlens + s + 1) : 0;
    const int before = bound_scan<THREADS>(have, c0, a.tokens, high, s_bound);
    if (!bounds_ok(c0, c1, a.tokens) || c0 < before) {
      if (have && slot == 0) record_bad_index();
    } else if (have && holds(slot, s, c0, c1, a.log_block)) {
      s_seq = s;
    }
  }
  __syncthreads();
}

// Grid (slots, kv_heads, 2: K, V); CHUNKS 16-byte pieces of BF16 rows per thread.
template <int THREADS, int CHUNKS>
__global__ void __launch_bounds__(THREADS) append_kernel(const __grid_constant__ Args a) {
  __shared__ int s_seq, s_odd;  // s_odd: some sequence does not count by its own bounds
  __shared__ float s_max[THREADS / 32];
  grid_dep_wait();
  grid_dep_launch();
  const int tid = threadIdx.x;
  const int B = 1 << a.log_block;
  if (tid == 0) s_seq = -1, s_odd = 0;
  __syncthreads();
  // slots of sequence s: [cu[s] / B + 2 s, cu[s + 1] / B + 2 (s + 1))
  const int64_t slot = blockIdx.x;
  for (int s = tid; s < a.n_seqs; s += THREADS) {
    const int64_t c0 = __ldg(a.cu_seqlens + s), c1 = __ldg(a.cu_seqlens + s + 1);
    if (!bounds_ok(c0, c1, a.tokens)) s_odd = 1;
    else if (holds(slot, s, c0, c1, a.log_block)) s_seq = s;
  }
  __syncthreads();
  if (s_odd) find_slot<THREADS>(a, slot, s_seq);
  const int seq = s_seq;
  if (seq < 0) return;
  const int64_t start = __ldg(a.cu_seqlens + seq), n_new = __ldg(a.cu_seqlens + seq + 1) - start;
  const int64_t total = __ldg(a.kv_lens + seq), past = total - n_new;
  const int64_t first_slot = (start >> a.log_block) + 2 * int64_t(seq);
  if (past < 0 || total > a.max_kv) {
    if (tid == 0 && slot == first_slot) record_bad_index();
    return;
  }
  const int64_t n = (past >> a.log_block) + (slot - first_slot);  // the sequence's n-th block
  const int64_t lo = n << a.log_block;                            // its first position
  if (n_new == 0 || lo >= total) return;
  const int64_t id = __ldg(a.table + seq * a.ld_table + n);
  if (id < 0 || id >= a.num_blocks) {
    if (tid == 0) record_bad_index();
    return;
  }
  const int held = static_cast<int>(max(past - lo, int64_t(0)));      // earlier tokens in the block
  const int end = static_cast<int>(min(total - lo, int64_t(B)));     // tokens in the block after the call
  const int h = blockIdx.y;
  const bool is_v = blockIdx.z != 0;
  const int log_c = a.log_d - 3;  // 8-element pieces per row
  const int64_t ld = is_v ? a.ld_v : a.ld_k;
  const uint16_t *src = (is_v ? a.v : a.k) + (start + lo + held - past) * ld + (int64_t(h) << a.log_d);
  const int64_t at = id * a.kv_heads + h;
  uint8_t *dst = (is_v ? a.v_cache : a.k_cache) + (at << (a.log_block + a.log_d));
  float *scale = (is_v ? a.v_scales : a.k_scales) + at;

  const int pieces = (end - held) << log_c;
  uint4 x[CHUNKS];
#pragma unroll
  for (int i = 0; i < CHUNKS; ++i) {
    const int p = tid + i * THREADS;
    x[i] = make_uint4(0, 0, 0, 0);
    if (p < pieces) x[i] = __ldg(reinterpret_cast<const uint4 *>(src + (p >> log_c) * ld + ((p & ((1 << log_c) - 1)) << 3)));
  }
  // largest finite magnitude: BF16 magnitudes order as integers, two at a time
  uint32_t m2 = 0;
#pragma unroll
  for (int i = 0; i < CHUNKS; ++i) {
    m2 = __vmaxu2(__vmaxu2(m2, x[i].x & 0x7fff7fffu), x[i].y & 0x7fff7fffu);
    m2 = __vmaxu2(__vmaxu2(m2, x[i].z & 0x7fff7fffu), x[i].w & 0x7fff7fffu);
  }
  uint32_t m = max(m2 & 0xffffu, m2 >> 16);
  if (m >= 0x7f80u) {  // an infinity or NaN does not set the scale
    m = 0;
#pragma unroll
    for (int i = 0; i < CHUNKS; ++i) {
      const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t u0 = w[j] & 0x7fffu, u1 = (w[j] >> 16) & 0x7fffu;
        if (u0 < 0x7f80u) m = max(m, u0);
        if (u1 < 0x7f80u) m = max(m, u1);
      }
    }
  }
  m = __reduce_max_sync(0xffffffffu, m);
  if ((tid & 31) == 0) s_max[tid >> 5] = __uint_as_float(m << 16);
  const float old = held > 0 ? *scale : 0.0f;
  __syncthreads();
  float amax = 0.0f;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) amax = fmaxf(amax, s_max[w]);
  float s = pow2_scale(amax);
  if (held > 0) {
    if (old >= s) {
      s = old;
    } else {  // the scale grows: the earlier codes move onto it
      const float f = old / s;
      for (int p = tid; p < (held << log_c) / 2; p += THREADS) {
        uint4 *c = reinterpret_cast<uint4 *>(dst) + p;
        const uint4 w = *c;
        const uint32_t in[4] = {w.x, w.y, w.z, w.w};
        uint32_t out[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float v[4];
#pragma unroll
          for (int b = 0; b < 4; ++b) v[b] = e4m3_to_f32(in[j] >> (8 * b)) * f;
          out[j] = cvt_e4m3x2(v[1], v[0]) | static_cast<uint32_t>(cvt_e4m3x2(v[3], v[2])) << 16;
        }
        *c = make_uint4(out[0], out[1], out[2], out[3]);
      }
    }
  }
  if (tid == 0) *scale = s;
  const float inv = 1.0f / s;
#pragma unroll
  for (int i = 0; i < CHUNKS; ++i) {
    const int p = tid + i * THREADS;
    if (p >= pieces) continue;
    const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
    uint32_t c[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      c[j] = cvt_e4m3x2(__uint_as_float(w[j] & 0xFFFF0000u) * inv, __uint_as_float(w[j] << 16) * inv);
    *reinterpret_cast<uint2 *>(dst + ((int64_t(held) << a.log_d) + (int64_t(p) << 3))) =
        make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
  }
}

}  // namespace kvblock
}  // namespace nvfp4

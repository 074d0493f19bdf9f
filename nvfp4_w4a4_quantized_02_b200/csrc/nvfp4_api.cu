// C ABI of the NVFP4 W4A4 linear library (declared in include/nvfp4.h):
// argument validation, TMA descriptor creation and kernel launches.
// Everything runs asynchronously on the caller's stream; nothing is allocated.
#include <cuda.h>
#include <cuda_runtime.h>

#include <nvtx3/nvToolsExt.h>

#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>
#include <unordered_map>

#include "nvfp4.h"
#include "quantize.cuh"
#include "gemm.cuh"
#include "fold.cuh"
#include "kvcache.cuh"
#include "gdn.cuh"
#include "gdn_chunk.cuh"
#include "layout.cuh"
#include "attn_decode.cuh"
#include "attn_prompt.cuh"
#include "headnorm.cuh"
#include "kvblock.cuh"
#include "matvec.cuh"

using namespace nvfp4;

namespace {

constexpr int kMaxDevices = 64;

struct DeviceInfo {
  bool init = false;
  bool ok = false;
  int sms = 0;
  bool attrs = false;
  int quant_ctas_per_sm = 1;
  int gemm2_clusters = 1;  // co-resident 2-CTA clusters of gemm2_kernel
};
DeviceInfo g_dev[kMaxDevices];
std::mutex g_mu;

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// Current device, checked to be an sm_100 part; fills `info`.
nvfp4_status_t current_device(DeviceInfo **info) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return NVFP4_ERR_CUDA;
  if (dev < 0 || dev >= kMaxDevices) return NVFP4_ERR_UNSUPPORTED_DEVICE;
  std::lock_guard<std::mutex> lk(g_mu);
  DeviceInfo &d = g_dev[dev];
  if (!d.init) {
    int major = 0, minor = 0, sms = 0;
    if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
        cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
      return NVFP4_ERR_CUDA;
    d.ok = (major == 10 && minor == 0);
    d.sms = sms;
    d.init = true;
  }
  if (!d.ok) return NVFP4_ERR_UNSUPPORTED_DEVICE;
  if (!d.attrs) {
    if (cudaFuncSetAttribute(gemm::gemm_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             gemm::Plan1::BYTES) != cudaSuccess ||
        cudaFuncSetAttribute(gemm::gemm_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             gemm::Plan1::BYTES) != cudaSuccess ||
        cudaFuncSetAttribute(gemm::gemm_kernel<false, true>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             gemm::Plan1::BYTES) != cudaSuccess ||
        cudaFuncSetAttribute(gemm::gemm2_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             gemm::Plan2::BYTES) != cudaSuccess ||
        cudaFuncSetAttribute(gemm::decode_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             gemm::PlanD::BYTES) != cudaSuccess ||
        cudaFuncSetAttribute(gemm::gemm2_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 0) !=
            cudaSuccess ||
        cudaFuncSetAttribute(quantize_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kQSmemBytes) !=
            cudaSuccess ||
        cudaFuncSetAttribute(gdn::recurrence_kernel<32>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             int(sizeof(gdn::Smem<32>))) != cudaSuccess ||
        cudaFuncSetAttribute(gdn::recurrence_kernel<16>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             int(sizeof(gdn::Smem<16>))) != cudaSuccess ||
        cudaFuncSetAttribute(matvec::matvec_kernel<1>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             matvec::smem_bytes<1>()) != cudaSuccess ||
        cudaFuncSetAttribute(matvec::matvec_kernel<2>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             matvec::smem_bytes<2>()) != cudaSuccess ||
        cudaFuncSetAttribute(attn::decode_kernel<64>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             attn::decode_smem_bytes<64>()) != cudaSuccess ||
        cudaFuncSetAttribute(attn::decode_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             attn::decode_smem_bytes<128>()) != cudaSuccess ||
        cudaFuncSetAttribute(attn::decode_kernel<256>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             attn::decode_smem_bytes<256>()) != cudaSuccess ||
        cudaFuncSetAttribute(attn::prompt::prompt_kernel<64>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             attn::prompt::smem_bytes<64>()) != cudaSuccess ||
        cudaFuncSetAttribute(attn::prompt::prompt_kernel<128>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             attn::prompt::smem_bytes<128>()) != cudaSuccess ||
        cudaFuncSetAttribute(attn::prompt::prompt_kernel<256>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             attn::prompt::smem_bytes<256>()) != cudaSuccess ||
        cudaFuncSetAttribute(gdn::chunk_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             int(sizeof(gdn::ChunkSmem))) != cudaSuccess)
      return NVFP4_ERR_CUDA;
    {
      cudaLaunchConfig_t cfg = {};
      cudaLaunchAttribute attr[1];
      attr[0].id = cudaLaunchAttributeClusterDimension;
      attr[0].val.clusterDim.x = 2;
      attr[0].val.clusterDim.y = 1;
      attr[0].val.clusterDim.z = 1;
      cfg.gridDim = dim3(2 * d.sms, 1, 1);
      cfg.blockDim = dim3(gemm::NUM_THREADS, 1, 1);
      cfg.dynamicSmemBytes = gemm::Plan2::BYTES;
      cfg.attrs = attr;
      cfg.numAttrs = 1;
      int clusters = 0;
      if (cudaOccupancyMaxActiveClusters(&clusters, gemm::gemm2_kernel, &cfg) != cudaSuccess) return NVFP4_ERR_CUDA;
      d.gemm2_clusters = clusters < 1 ? 1 : clusters;
    }
    int occ = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, quantize_kernel, kQThreads, kQSmemBytes) != cudaSuccess)
      return NVFP4_ERR_CUDA;
    d.quant_ctas_per_sm = occ < 1 ? 1 : occ;
    d.attrs = true;
  }
  *info = &d;
  return NVFP4_OK;
}

// NVTX range around one C-ABI call, named after the entry point, so that profilers
// (Nsight Systems / Compute) show which call launched which kernels.  Without a tool
// attached each push / pop is a call through a no-op pointer.
struct NvtxRange {
  explicit NvtxRange(const char *name) { nvtxRangePushA(name); }
  ~NvtxRange() { nvtxRangePop(); }
  NvtxRange(const NvtxRange &) = delete;
  NvtxRange &operator=(const NvtxRange &) = delete;
};

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                   const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &p, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  });
  return fn;
}

// Cache of encoded tensor maps.  A map is a pure function of (kind, base address,
// sizes, box), so an entry can never go stale: a buffer freed and reallocated at the
// same address with the same sizes gets the same map.  Keyed also by device.  The
// cache is bounded: when full it is cleared and refilled.
struct MapKey {
  int dev, kind;
  const void *ptr;
  int64_t a, b, c;
  bool operator==(const MapKey &o) const {
    return dev == o.dev && kind == o.kind && ptr == o.ptr && a == o.a && b == o.b && c == o.c;
  }
};
struct MapKeyHash {
  size_t operator()(const MapKey &k) const {
    uint64_t h = reinterpret_cast<uintptr_t>(k.ptr) * 0x9E3779B97F4A7C15ull;
    for (uint64_t v : {uint64_t(k.dev), uint64_t(k.kind), uint64_t(k.a), uint64_t(k.b), uint64_t(k.c)})
      h = (h ^ v) * 0x100000001B3ull + (h >> 29);
    return static_cast<size_t>(h);
  }
};
constexpr size_t kMapCacheMax = 4096;
std::unordered_map<MapKey, CUtensorMap, MapKeyHash> g_maps;
std::mutex g_maps_mu;

enum MapKind : int { MAP_CODES = 0, MAP_BF16 = 1, MAP_SCALES = 2 };

// Looks `key` up; on a miss runs `encode(m)` and keeps its result.
template <typename F>
bool cached_map(CUtensorMap *m, MapKey key, F &&encode) {
  if (cudaGetDevice(&key.dev) != cudaSuccess) return false;
  {
    std::lock_guard<std::mutex> lk(g_maps_mu);
    auto it = g_maps.find(key);
    if (it != g_maps.end()) {
      std::memcpy(m, &it->second, sizeof(CUtensorMap));
      return true;
    }
  }
  if (!encode(m)) return false;
  std::lock_guard<std::mutex> lk(g_maps_mu);
  if (g_maps.size() >= kMapCacheMax) g_maps.clear();
  g_maps.emplace(key, *m);
  return true;
}

// Tensor map of packed codes [rows x K/2] bytes: 128-byte x box_rows boxes with the
// 128-byte swizzle (the smem layout the MMA descriptors describe); rows beyond
// `rows` read as zero.
bool encode_codes_map(CUtensorMap *m, const uint8_t *codes, int64_t rows, int64_t K, unsigned box_rows) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(K / 2), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(K / 2)};
  cuuint32_t box[2] = {128, box_rows};
  cuuint32_t estr[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t *>(codes), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool make_codes_map(CUtensorMap *m, const uint8_t *codes, int64_t rows, int64_t K, unsigned box_rows = 128) {
  return cached_map(m, MapKey{0, MAP_CODES, codes, rows, K, box_rows},
                    [&](CUtensorMap *mm) { return encode_codes_map(mm, codes, rows, K, box_rows); });
}

// Tensor map of a BF16 matrix [rows x cols] with row stride ld elements: 64-column x
// 128-row boxes (128 bytes per box row) with the 128-byte swizzle; coordinates
// outside the matrix read as zero.
bool encode_bf16_map(CUtensorMap *m, const void *x, int64_t rows, int64_t cols, int64_t ld) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(ld * 2)};
  cuuint32_t box[2] = {static_cast<cuuint32_t>(kQTileCols), static_cast<cuuint32_t>(kQTileRows)};
  cuuint32_t estr[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(x), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool make_bf16_map(CUtensorMap *m, const void *x, int64_t rows, int64_t cols, int64_t ld) {
  return cached_map(m, MapKey{0, MAP_BF16, x, rows, cols, ld},
                    [&](CUtensorMap *mm) { return encode_bf16_map(mm, x, rows, cols, ld); });
}

// Tensor map of a swizzled scale buffer of a [rows x K] operand, viewed as 8-byte
// elements: one row per 128-row group (K/64 atoms of 512 bytes), boxes of 256
// elements = the 4 atoms (2 KB) of one 256-wide K tile of one group.
bool encode_scales_map(CUtensorMap *m, const uint8_t *scales, int64_t rows, int64_t K) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  const int64_t groups = (rows + 127) / 128;
  cuuint64_t dims[2] = {static_cast<cuuint64_t>(K / 64 * 64), static_cast<cuuint64_t>(groups)};
  cuuint64_t strides[1] = {static_cast<cuuint64_t>(K / 64 * 512)};
  cuuint32_t box[2] = {256, 1};
  cuuint32_t estr[2] = {1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT64, 2, const_cast<uint8_t *>(scales), dims, strides, box, estr,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

bool make_scales_map(CUtensorMap *m, const uint8_t *scales, int64_t rows, int64_t K) {
  return cached_map(m, MapKey{0, MAP_SCALES, scales, rows, K, 0},
                    [&](CUtensorMap *mm) { return encode_scales_map(mm, scales, rows, K); });
}

// Launches `kernel` with programmatic stream serialization: it may begin (shared
// memory, barriers, TMEM) while the previous kernel on the stream finishes, and waits
// for it in griddepcontrol.wait before touching global memory (every kernel of the
// library does).  In a CUDA graph of many small launches (a decode step) this hides
// most of each launch's latency and prologue.  cluster_x > 1 adds a cluster shape.
template <typename... KArgs, typename... Args>
nvfp4_status_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                          unsigned cluster_x, Args &&...args) {
  cudaLaunchAttribute attr[2];
  unsigned n = 0;
  attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[n].val.programmaticStreamSerializationAllowed = 1;
  ++n;
  if (cluster_x > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = cluster_x;
    attr[n].val.clusterDim.y = 1;
    attr[n].val.clusterDim.z = 1;
    ++n;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = n;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Args &&>(args)...) == cudaSuccess ? NVFP4_OK : NVFP4_ERR_CUDA;
}

constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1;

// Argument checks shared by the entry points that work on a block-scaled cache.
nvfp4_status_t check_batch(const nvfp4_batch_t *b, const nvfp4_block_cache_t *c, int *log_block) {
  if (!b || !c || !b->cu_seqlens || !b->kv_lens || !b->block_table || !c->k || !c->v || !c->k_scales || !c->v_scales)
    return NVFP4_ERR_INVALID_ARG;
  if (b->n_seqs < 1 || b->tokens < 0 || b->max_blocks < 1 || b->ld_table < b->max_blocks || c->num_blocks < 1 ||
      c->n_kv_heads < 1)
    return NVFP4_ERR_INVALID_ARG;
  switch (c->block_size) {
    case 16: *log_block = 4; break;
    case 32: *log_block = 5; break;
    case 64: *log_block = 6; break;
    case 128: *log_block = 7; break;
    default: return NVFP4_ERR_UNSUPPORTED_SHAPE;
  }
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  // kernels count cached tokens in 32 bits, up to the end of a tile behind the last
  if (b->n_seqs > 65535 || b->tokens > kMaxDim || c->n_kv_heads > 65535 || c->num_blocks > kMaxDim ||
      b->max_blocks > (kMaxDim - 512) >> *log_block || c->num_blocks * c->n_kv_heads > kMaxDim)
    return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (!aligned(b->cu_seqlens, 4) || !aligned(b->kv_lens, 4) || !aligned(b->block_table, 4) || !aligned(c->k, 16) ||
      !aligned(c->v, 16) || !aligned(c->k_scales, 4) || !aligned(c->v_scales, 4))
    return NVFP4_ERR_MISALIGNED;
  return NVFP4_OK;
}

// Tensor map of the codes of K or V as [(block, head)][token][value], for boxes of 2^log_box of one
// head's rows, up to 128 bytes wide and with the swizzle of that width (the layout of a K-major MMA
// operand).  Encoded for every call: nothing is kept by a cache's address.
bool encode_cache_map(CUtensorMap *m, uint8_t *codes, const nvfp4_block_cache_t *c, int log_box) {
  EncodeTiledFn enc = encode_fn();
  if (!enc) return false;
  const int D = c->head_dim;
  cuuint64_t dims[3] = {cuuint64_t(D), cuuint64_t(c->block_size), cuuint64_t(c->num_blocks * c->n_kv_heads)};
  cuuint64_t strides[2] = {cuuint64_t(D), cuuint64_t(c->block_size) * D};
  cuuint32_t box[3] = {cuuint32_t(D < 128 ? D : 128), 1u << log_box, 1};
  cuuint32_t estr[3] = {1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, codes, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
             D < 128 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Workspace of nvfp4_attention: unit count, unit descriptors, partial results.
constexpr int kMaxAttnCtas = 640;
// Sequences with at most this many query rows per kv head (new tokens times heads of a
// group) go to the decode kernel, the others to the prompt kernel.
constexpr int kDecodeRows = 32;
// Few prompt items (row blocks times kv heads) for the SMs: each is cut into as many parts as make
// the CTAs fill whole waves best (1024 tokens on 32768 at four kv heads of 256 values: 192 items on
// 148 SMs, 955 us uncut), while the parts' results fit kMaxPromptParts places.
// The workspace's size is told without a device, so the rule takes a B200's count of SMs.
constexpr int kMaxPromptParts = 640, kMaxSplits = 8, kSmsAssumed = 148;
int prompt_splits(int64_t items, int most) {
  int best = 1;
  double best_cost = 1e300;
  for (int s = 1; s <= most && (s == 1 || items * s <= kMaxPromptParts); ++s) {
    const double cost = double((items * s + kSmsAssumed - 1) / kSmsAssumed) / s + 0.03 * (s - 1);
    if (cost < best_cost) best_cost = cost, best = s;
  }
  return best;
}

struct AttnWorkspace {
  int64_t units, items;  // bounds of the decode units and the prompt items of the call
  int splits;
  size_t desc, desc2, part_ml, part, prompt_ml, prompt_part, bytes;
  bool fits() const { return units <= kMaxDim && items * splits <= kMaxDim; }  // CTAs of the join and prompt kernels
};
AttnWorkspace attn_workspace(int64_t tokens, int64_t n_seqs, int n_heads, int n_kv_heads, int head_dim) {
  AttnWorkspace w;
  const int64_t group = n_heads / n_kv_heads;
  const int64_t most = n_seqs * (kDecodeRows / attn::kRows);
  w.units = (tokens * group + attn::kRows - 1) / attn::kRows + n_seqs;
  w.units = n_kv_heads * (w.units < most ? w.units : most);
  w.desc = 256;
  w.desc2 = w.desc + w.units * sizeof(int4);
  w.part_ml = (w.desc2 + w.units * sizeof(int2) + 255) / 256 * 256;
  w.part = w.part_ml + size_t(2) * kMaxAttnCtas * attn::kRows * sizeof(float2);
  w.prompt_ml = w.part + size_t(2) * kMaxAttnCtas * attn::kRows * head_dim * sizeof(float);
  // a prompt has more than kDecodeRows rows; its last row block may be short
  const int64_t rows = tokens * group, tile = head_dim == 256 ? 128 : 256;
  const int64_t prompts = rows / (kDecodeRows + 1) < n_seqs ? rows / (kDecodeRows + 1) : n_seqs;
  w.items = (rows / tile + prompts) * n_kv_heads;
  w.splits = prompt_splits(w.items, kMaxSplits);
  const size_t parts = w.splits > 1 ? size_t(w.items) * w.splits * tile : 0;
  w.prompt_part = w.prompt_ml + (parts * sizeof(float2) + 255) / 256 * 256;
  w.bytes = w.prompt_part + parts * head_dim * sizeof(float);
  return w;
}

// Validates the arguments of a linear and fills everything of Params but the tiling.
nvfp4_status_t prepare_linear(const nvfp4_operand_t *A, const float *gs_a, const nvfp4_operand_t *W,
                              const nvfp4_segment_t *segs, int nseg, int epilogue,
                              const nvfp4_epilogue_params_t *ep, void *out, int out_kind, int64_t ldo,
                              gemm::Params &p) {
  using namespace gemm;
  if (!A || !W || !gs_a || !segs || !out) return NVFP4_ERR_INVALID_ARG;
  if (!A->codes || !A->scales || !W->codes || !W->scales) return NVFP4_ERR_INVALID_ARG;
  if (A->rows < 1 || W->rows < 1 || A->K < 1 || A->K != W->K) return NVFP4_ERR_INVALID_ARG;
  if (epilogue < NVFP4_EPI_NONE || epilogue > NVFP4_EPI_GDN_GATES) return NVFP4_ERR_INVALID_ARG;
  if (out_kind < NVFP4_OUT_BF16 || out_kind > NVFP4_OUT_NVFP4) return NVFP4_ERR_INVALID_ARG;
  if (nseg < 1 || nseg > NVFP4_MAX_SEGMENTS) return NVFP4_ERR_INVALID_ARG;
  const int64_t M = A->rows, N = W->rows, K = A->K;
  if (M > kMaxDim || N > kMaxDim || K > kMaxDim) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (K % BK != 0 || N % 16 != 0) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  // segments: sorted, disjoint, 16-aligned, covering [0, N)
  int64_t expect = 0;
  for (int i = 0; i < nseg; ++i) {
    if (!segs[i].gs_w || !aligned(segs[i].gs_w, 4)) return NVFP4_ERR_INVALID_ARG;
    if (segs[i].n_begin != expect || segs[i].n_end <= segs[i].n_begin) return NVFP4_ERR_INVALID_ARG;
    if (segs[i].n_begin % 16 != 0 || segs[i].n_end % 16 != 0) return NVFP4_ERR_UNSUPPORTED_SHAPE;
    expect = segs[i].n_end;
  }
  if (expect != N) return NVFP4_ERR_INVALID_ARG;
  int64_t Nout = N;
  if (epilogue == NVFP4_EPI_SILU_MUL) {
    if (N % (2 * 128) != 0) return NVFP4_ERR_UNSUPPORTED_SHAPE;
    Nout = N / 2;
  }
  if (epilogue == NVFP4_EPI_GDN_GATES) {
    if (!ep || !ep->A_log || !ep->dt_bias || ep->n_heads < 1) return NVFP4_ERR_INVALID_ARG;
    const int64_t h = ep->n_heads;
    if (ep->beta_begin < 0 || ep->beta_begin + h > N || ep->alpha_begin < 0 || ep->alpha_begin + h > N)
      return NVFP4_ERR_INVALID_ARG;
    if (ep->beta_begin < ep->alpha_begin + h && ep->alpha_begin < ep->beta_begin + h) return NVFP4_ERR_INVALID_ARG;
    if (!aligned(ep->A_log, 4) || !aligned(ep->dt_bias, 4) || (ep->beta_out && !aligned(ep->beta_out, 4)) ||
        (ep->g_out && !aligned(ep->g_out, 4)))
      return NVFP4_ERR_MISALIGNED;
  }
  if (out_kind == NVFP4_OUT_NVFP4) {
    if (!ep || !ep->gs_out || !ep->out_scales) return NVFP4_ERR_INVALID_ARG;
    if (Nout % 64 != 0) return NVFP4_ERR_UNSUPPORTED_SHAPE;
    if (!aligned(out, 16) || !aligned(ep->out_scales, 16) || !aligned(ep->gs_out, 4)) return NVFP4_ERR_MISALIGNED;
  } else {
    const int64_t elem = out_kind == NVFP4_OUT_BF16 ? 2 : 4;
    if (ldo < Nout) return NVFP4_ERR_INVALID_ARG;
    if (!aligned(out, 16) || (ldo * elem) % 16 != 0) return NVFP4_ERR_MISALIGNED;
  }
  if (!aligned(A->codes, 16) || !aligned(W->codes, 16) || !aligned(A->scales, 16) || !aligned(W->scales, 16) ||
      !aligned(gs_a, 4))
    return NVFP4_ERR_MISALIGNED;

  p = Params{};
  p.M = static_cast<int>(M);
  p.N = static_cast<int>(N);
  p.K = static_cast<int>(K);
  p.Nout = static_cast<int>(Nout);
  p.mode = epilogue;
  p.tile_mode = epilogue;
  p.out_kind = out_kind;
  p.k_tiles = static_cast<int>(K / BK);
  p.splits = 1;
  p.kt_per_split = p.k_tiles;
  p.partial = nullptr;
  p.up_row0 = static_cast<int>(Nout);
  p.kb_atoms = K / 64;
  p.sfa = A->scales;
  p.sfb = W->scales;
  p.gs_a = gs_a;
  p.nseg = nseg;
  for (int i = 0; i < nseg; ++i) {
    p.seg[i].n_begin = static_cast<int>(segs[i].n_begin);
    p.seg[i].n_end = static_cast<int>(segs[i].n_end);
    p.seg[i].gs_w = segs[i].gs_w;
  }
  p.out = out;
  p.ldo = ldo;
  p.beta_begin = p.alpha_begin = -1;
  p.n_heads = 0;
  if (epilogue == NVFP4_EPI_GDN_GATES) {
    p.beta_begin = static_cast<int>(ep->beta_begin);
    p.alpha_begin = static_cast<int>(ep->alpha_begin);
    p.n_heads = static_cast<int>(ep->n_heads);
    p.A_log = ep->A_log;
    p.dt_bias = ep->dt_bias;
    p.beta_out = ep->beta_out;
    p.g_out = ep->g_out;
  }
  if (out_kind == NVFP4_OUT_NVFP4) {
    p.gs_out = ep->gs_out;
    p.out_scales = ep->out_scales;
    p.out_kb_atoms = Nout / 64;
  }
  // 32-byte epilogue stores when every row of the output starts 32-byte aligned (an
  // NVFP4 row is Nout / 2 bytes, a multiple of 32)
  const int64_t row_bytes = out_kind == NVFP4_OUT_NVFP4 ? Nout / 2 : ldo * (out_kind == NVFP4_OUT_BF16 ? 2 : 4);
  p.st32 = aligned(out, 32) && row_bytes % 32 == 0;
  p.group_m = GROUP_M;
  return NVFP4_OK;
}

// Split count of the split-K linear: as many splits as keep all work units in one
// wave on the SMs (SMs / tiles, rounded down), with at least 4 K tiles (1024 K) per
// split.  Tiles are 128 weight rows for the decode kernel (M <= 64), else 128 x 256.
// On the decode kernel at 32 rows the rule picks the fastest of splits 1, 2, 3, 4, 6
// for five of the six shapes of the 496-linear decode step; for the 12352-row GDN
// in-projection it picks 1 (13.2 us), where 3 measured 12.8 us.
int default_splits(int64_t M, int64_t N, int64_t K, int sms) {
  const int64_t tiles = M <= gemm::DEC_DN_MAX ? (N + gemm::DEC_BM - 1) / gemm::DEC_BM
                                               : (M + gemm::BM - 1) / gemm::BM * ((N + gemm::BN - 1) / gemm::BN);
  const int64_t k_tiles = K / gemm::BK;
  int64_t s = sms / tiles;
  if (s > k_tiles / 4) s = k_tiles / 4;
  return static_cast<int>(s < 1 ? 1 : s);
}

// Launches the 1-CTA GEMM in split-K mode and the epilogue kernel on `p` (prepared
// by prepare_linear); `splits` >= 1 and the workspace were checked by the caller.
nvfp4_status_t launch_splitk(gemm::Params p, const nvfp4_operand_t *A, const nvfp4_operand_t *W, int splits,
                             float *workspace, const DeviceInfo *dev, cudaStream_t st) {
  using namespace gemm;
  p.kt_per_split = (p.k_tiles + splits - 1) / splits;
  p.splits = (p.k_tiles + p.kt_per_split - 1) / p.kt_per_split;  // no empty split
  p.partial = workspace;
  p.tile_mode = MODE_NONE;
  CUtensorMap tmA, tmB;
  if (p.M <= DEC_DN_MAX) {  // decode size: weight rows are the MMA's M, tokens its N
    p.dn = p.M <= 32 ? 32 : DEC_DN_MAX;
    p.m_tiles = 1;
    p.n_tiles = (p.N + DEC_BM - 1) / DEC_BM;
    if (!make_codes_map(&tmB, W->codes, p.N, p.K) || !make_codes_map(&tmA, A->codes, p.M, p.K, p.dn))
      return NVFP4_ERR_CUDA;
    const int64_t units = int64_t(p.n_tiles) * p.splits;
    if (units > kMaxDim) return NVFP4_ERR_UNSUPPORTED_SHAPE;
    const int grid = static_cast<int>(units < dev->sms ? units : dev->sms);
    // One split, an element-wise epilogue and a BF16 / FP32 output: the kernel applies
    // the epilogue itself (no partials, no reduction kernel).  SiLU*mul pairs columns of
    // two tiles and an NVFP4 output needs 16 columns of a row; both keep the reduction.
    const bool direct = p.splits == 1 && p.mode != MODE_SILU_MUL && p.out_kind != OUT_NVFP4;
    if (direct) p.partial = nullptr;
    if (nvfp4_status_t e = launch_pdl(decode_kernel, dim3(grid), dim3(DEC_THREADS), PlanD::BYTES, st, 1, tmB, tmA, p))
      return e;
    if (direct) return NVFP4_OK;
  } else {
    if (!make_codes_map(&tmA, A->codes, p.M, p.K) || !make_codes_map(&tmB, W->codes, p.N, p.K)) return NVFP4_ERR_CUDA;
    p.m_tiles = (p.M + BM - 1) / BM;
    p.n_tiles = (p.N + BN - 1) / BN;
    const int64_t units = int64_t(p.m_tiles) * p.n_tiles * p.splits;
    if (units > kMaxDim) return NVFP4_ERR_UNSUPPORTED_SHAPE;
    const int grid = static_cast<int>(units < dev->sms ? units : dev->sms);
    if (nvfp4_status_t e =
            launch_pdl(gemm_kernel<true>, dim3(grid), dim3(NUM_THREADS), Plan1::BYTES, st, 1, tmA, tmB, p))
      return e;
  }
  // one thread per 16 columns (an E4M3 block) for an NVFP4 output, else per 4 columns
  const bool nvfp4_out = p.out_kind == OUT_NVFP4;
  const int64_t rows_cover = nvfp4_out ? (p.M + 127) / 128 * 128 : p.M;
  const int64_t threads = rows_cover * (p.Nout / (nvfp4_out ? 16 : 4));
  const int64_t blocks = (threads + REDUCE_THREADS - 1) / REDUCE_THREADS;
  if (blocks > kMaxDim) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  return launch_pdl(nvfp4_out ? splitk_epilogue_kernel<16> : splitk_epilogue_kernel<4>,
                    dim3(static_cast<unsigned>(blocks)), dim3(REDUCE_THREADS), 0, st, 1, p);
}

// ------------------------------------------------- scratch for callers that cannot allocate
// nvfp4_linear_splitk_noalloc keeps its split-K partial sums in this fixed array, so
// that callers which cannot allocate device memory (no workspace to hand in) can
// still run the decode-regime linear.  Every GPU that loads the library holds these
// NVFP4_NOALLOC_SCRATCH_BYTES until the process exits.
static __device__ __align__(256) float g_noalloc_scratch[NVFP4_NOALLOC_SCRATCH_BYTES / sizeof(float)];

// Device address of g_noalloc_scratch on each device, looked up once per device (the
// host-side name of the array is not a device address).
float *g_noalloc_ptr[kMaxDevices] = {};

nvfp4_status_t noalloc_scratch(float **ptr) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return NVFP4_ERR_CUDA;
  if (dev < 0 || dev >= kMaxDevices) return NVFP4_ERR_UNSUPPORTED_DEVICE;
  std::lock_guard<std::mutex> lk(g_mu);
  if (!g_noalloc_ptr[dev]) {
    void *p = nullptr;
    if (cudaGetSymbolAddress(&p, g_noalloc_scratch) != cudaSuccess || !p) return NVFP4_ERR_CUDA;
    g_noalloc_ptr[dev] = static_cast<float *>(p);
  }
  *ptr = g_noalloc_ptr[dev];
  return NVFP4_OK;
}

// max|x| of a BF16 matrix into *out (device FP32): zero it, then the amax kernel's
// atomicMax over the bit patterns (non-negative floats order as unsigned integers).
nvfp4_status_t launch_amax(const void *x_bf16, int64_t rows, int64_t cols, int64_t ld, float *out,
                           const DeviceInfo *dev, cudaStream_t s) {
  if (cudaMemsetAsync(out, 0, sizeof(float), s) != cudaSuccess) return NVFP4_ERR_CUDA;
  AmaxArgs a;
  a.x = static_cast<const uint16_t *>(x_bf16);
  a.rows = rows;
  a.cols = cols;
  a.ld = ld;
  a.amax_bits = reinterpret_cast<unsigned int *>(out);
  const int64_t vecs = rows * (cols / 8);
  const int64_t want = (vecs / 4 + kAmaxThreads - 1) / kAmaxThreads;
  const int64_t cap = int64_t(dev->sms) * 4;
  const int grid = static_cast<int>(want < 1 ? 1 : (want < cap ? want : cap));
  return launch_pdl(amax_kernel, dim3(grid), dim3(kAmaxThreads), 0, s, 1, a);
}

}  // namespace

extern "C" {

const char *nvfp4_status_string(int s) {
  switch (s) {
    case NVFP4_OK: return "NVFP4_OK";
    case NVFP4_ERR_INVALID_ARG: return "NVFP4_ERR_INVALID_ARG";
    case NVFP4_ERR_UNSUPPORTED_SHAPE: return "NVFP4_ERR_UNSUPPORTED_SHAPE";
    case NVFP4_ERR_MISALIGNED: return "NVFP4_ERR_MISALIGNED";
    case NVFP4_ERR_CUDA: return "NVFP4_ERR_CUDA";
    case NVFP4_ERR_DEVICE_TIMEOUT: return "NVFP4_ERR_DEVICE_TIMEOUT";
    case NVFP4_ERR_UNSUPPORTED_DEVICE: return "NVFP4_ERR_UNSUPPORTED_DEVICE";
    case NVFP4_ERR_DEVICE_INDEX: return "NVFP4_ERR_DEVICE_INDEX";
    default: return "NVFP4_ERR_UNKNOWN";
  }
}

size_t nvfp4_scale_bytes(int64_t rows, int64_t cols) {
  if (rows < 1 || cols < 16 || cols % 16 != 0 || rows > kMaxDim || cols > kMaxDim) return 0;
  const int64_t rows_pad = (rows + 127) / 128 * 128;
  const int64_t kb_pad = (cols / 16 + 3) / 4 * 4;
  return static_cast<size_t>(rows_pad * kb_pad);
}

nvfp4_status_t nvfp4_amax(const void *x_bf16, int64_t rows, int64_t cols, int64_t ld, float *amax_out,
                          nvfp4_stream_t stream) {
  NvtxRange nvtx("nvfp4_amax");
  if (!x_bf16 || !amax_out || rows < 1 || cols < 1 || ld < cols) return NVFP4_ERR_INVALID_ARG;
  if (cols % 16 != 0 || rows > kMaxDim || cols > kMaxDim) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (!aligned(x_bf16, 16) || ld % 8 != 0 || !aligned(amax_out, 4)) return NVFP4_ERR_MISALIGNED;
  DeviceInfo *dev = nullptr;
  if (nvfp4_status_t st = current_device(&dev)) return st;
  return launch_amax(x_bf16, rows, cols, ld, amax_out, dev, reinterpret_cast<cudaStream_t>(stream));
}

nvfp4_status_t nvfp4_global_scale(const void *x_bf16, int64_t rows, int64_t cols, int64_t ld, float *gs_out,
                                  nvfp4_stream_t stream) {
  NvtxRange nvtx("nvfp4_global_scale");
  if (!x_bf16 || !gs_out || rows < 1 || cols < 1 || ld < cols) return NVFP4_ERR_INVALID_ARG;
  if (cols % 16 != 0 || rows > kMaxDim || cols > kMaxDim) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (!aligned(x_bf16, 16) || ld % 8 != 0 || !aligned(gs_out, 4)) return NVFP4_ERR_MISALIGNED;
  DeviceInfo *dev = nullptr;
  if (nvfp4_status_t st = current_device(&dev)) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (nvfp4_status_t e = launch_amax(x_bf16, rows, cols, ld, gs_out, dev, s)) return e;
  return launch_pdl(global_scale_finalize_kernel, dim3(1), dim3(1), 0, s, 1, gs_out);
}

nvfp4_status_t nvfp4_quantize_rows(const void *x_bf16, int64_t rows, int64_t cols, int64_t ld, const float *gs,
                                   uint8_t *codes, uint8_t *scales, int64_t row_offset, int64_t total_rows,
                                   nvfp4_stream_t stream) {
  NvtxRange nvtx("nvfp4_quantize_rows");
  if (!x_bf16 || !gs || !codes || !scales || rows < 1 || cols < 1 || ld < cols) return NVFP4_ERR_INVALID_ARG;
  if (row_offset < 0 || total_rows < row_offset + rows) return NVFP4_ERR_INVALID_ARG;
  if (cols < 16 || cols % 16 != 0 || total_rows > kMaxDim || cols > kMaxDim) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (!aligned(x_bf16, 16) || ld % 8 != 0 || !aligned(codes, 16) || !aligned(scales, 16) || !aligned(gs, 4))
    return NVFP4_ERR_MISALIGNED;
  DeviceInfo *dev = nullptr;
  if (nvfp4_status_t st = current_device(&dev)) return st;
  QuantArgs a;
  a.gs = gs;
  a.codes = codes;
  a.scales = scales;
  a.rows = rows;
  a.cols = cols;
  a.row_offset = row_offset;
  const bool last = row_offset + rows == total_rows;
  a.own_end = last ? (total_rows + 127) / 128 * 128 : row_offset + rows;
  a.code_ld = cols / 2;
  a.kb_atoms = (cols + 63) / 64;
  a.tile_r0 = row_offset / 128;
  a.n_tiles = ((a.own_end + 127) / 128 - a.tile_r0) * a.kb_atoms;
  if (rows <= 64) {  // decode sizes: one thread per 16-element block, no TMA staging
    const int64_t threads = (a.own_end - row_offset) * 4 * a.kb_atoms;
    const int64_t blocks = (threads + kQSmallThreads - 1) / kQSmallThreads;
    if (blocks > kMaxDim) return NVFP4_ERR_UNSUPPORTED_SHAPE;
    return launch_pdl(quantize_small_kernel, dim3(static_cast<unsigned>(blocks)), dim3(kQSmallThreads), 0,
                      reinterpret_cast<cudaStream_t>(stream), 1, static_cast<const uint16_t *>(x_bf16), ld, a);
  }
  CUtensorMap tmX;
  if (!make_bf16_map(&tmX, x_bf16, rows, cols, ld)) return NVFP4_ERR_CUDA;
  const int64_t cap = int64_t(dev->sms) * dev->quant_ctas_per_sm;
  const int grid = static_cast<int>(a.n_tiles < cap ? a.n_tiles : cap);
  return launch_pdl(quantize_kernel, dim3(grid), dim3(kQThreads), kQSmemBytes, reinterpret_cast<cudaStream_t>(stream), 1,
                    tmX, a);
}

nvfp4_status_t nvfp4_quantize(const void *x_bf16, int64_t rows, int64_t cols, int64_t ld, const float *gs,
                              uint8_t *codes, uint8_t *scales, nvfp4_stream_t stream) {
  NvtxRange nvtx("nvfp4_quantize");
  return nvfp4_quantize_rows(x_bf16, rows, cols, ld, gs, codes, scales, 0, rows, stream);
}

nvfp4_status_t nvfp4_linear(const nvfp4_operand_t *A, const float *gs_a, const nvfp4_operand_t *W,
                            const nvfp4_segment_t *segs, int nseg, int epilogue, const nvfp4_epilogue_params_t *ep,
                            void *out, int out_kind, int64_t ldo, nvfp4_stream_t stream) {
  NvtxRange nvtx("nvfp4_linear");
  using namespace gemm;
  Params p;
  if (nvfp4_status_t st = prepare_linear(A, gs_a, W, segs, nseg, epilogue, ep, out, out_kind, ldo, p)) return st;
  DeviceInfo *dev = nullptr;
  if (nvfp4_status_t st = current_device(&dev)) return st;
  const int64_t M = p.M, N = p.N, K = p.K;

  const bool pair = M > BM;  // 2-CTA tiles of 256 rows; one CTA per tile for M <= 128
  CUtensorMap tmA, tmB, tmSFA, tmSFB;
  if (!make_codes_map(&tmA, A->codes, M, K) || !make_codes_map(&tmB, W->codes, N, K)) return NVFP4_ERR_CUDA;
  if (pair && (!make_scales_map(&tmSFA, A->scales, M, K) || !make_scales_map(&tmSFB, W->scales, N, K)))
    return NVFP4_ERR_CUDA;
  const int64_t tile_m = pair ? 2 * BM : BM;
  p.m_tiles = static_cast<int>((M + tile_m - 1) / tile_m);
  p.n_tiles = epilogue == NVFP4_EPI_SILU_MUL ? p.Nout / 128 : static_cast<int>((N + BN - 1) / BN);
  const int64_t tiles = int64_t(p.m_tiles) * p.n_tiles;
  if (tiles > kMaxDim) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (!pair) {
    const int grid = static_cast<int>(tiles < dev->sms ? tiles : dev->sms);
    return launch_pdl(gemm_kernel<false>, dim3(grid), dim3(NUM_THREADS), Plan1::BYTES, st, 1, tmA, tmB, p);
  }
  // A wide weight (64 N-tiles or more) is streamed from DRAM once per raster group:
  // groups of 32 M-tiles halve those re-reads while the group's A rows (codes and
  // scales) stay within 32 MB, a quarter of the B200's L2.  MLP gate|up at 32768
  // tokens: DRAM reads 895 -> 496 MB per launch, 1.6 % faster; a longer K (the down
  // projection) keeps 16.
  if (p.n_tiles >= 64 && int64_t(2 * GROUP_M) * (2 * BM) * (K / 2) * 9 / 8 <= (int64_t(32) << 20))
    p.group_m = 2 * GROUP_M;
  const int64_t clusters = tiles < dev->gemm2_clusters ? tiles : dev->gemm2_clusters;
  return launch_pdl(gemm2_kernel, dim3(static_cast<unsigned>(2 * clusters)), dim3(NUM_THREADS), Plan2::BYTES, st, 2, tmA,
                    tmB, tmSFA, tmSFB, p);
}

int nvfp4_splitk_default(int64_t M, int64_t N, int64_t K) {
  if (M < 1 || N < 16 || K < gemm::BK || K % gemm::BK != 0) return 0;
  DeviceInfo *dev = nullptr;
  if (current_device(&dev) != NVFP4_OK) return 0;
  return default_splits(M, N, K, dev->sms);
}

size_t nvfp4_splitk_workspace_bytes(int64_t M, int64_t N, int split_k) {
  if (M < 1 || N < 1 || split_k < 1 || M > kMaxDim || N > kMaxDim) return 0;
  return static_cast<size_t>(M) * static_cast<size_t>(N) * static_cast<size_t>(split_k) * sizeof(float);
}

nvfp4_status_t nvfp4_linear_splitk(const nvfp4_operand_t *A, const float *gs_a, const nvfp4_operand_t *W,
                                   const nvfp4_segment_t *segs, int nseg, int epilogue,
                                   const nvfp4_epilogue_params_t *ep, void *out, int out_kind, int64_t ldo,
                                   int split_k, void *workspace, size_t workspace_bytes, nvfp4_stream_t stream) {
  NvtxRange nvtx("nvfp4_linear_splitk");
  using namespace gemm;
  Params p;
  if (nvfp4_status_t st = prepare_linear(A, gs_a, W, segs, nseg, epilogue, ep, out, out_kind, ldo, p)) return st;
  if (split_k < 1 || split_k > p.k_tiles) return NVFP4_ERR_INVALID_ARG;
  if (!workspace) return NVFP4_ERR_INVALID_ARG;
  if (workspace_bytes < nvfp4_splitk_workspace_bytes(p.M, p.N, split_k)) return NVFP4_ERR_INVALID_ARG;
  if (!aligned(workspace, 16)) return NVFP4_ERR_MISALIGNED;
  // One split above decode size: the ordinary kernel, without partials or the second
  // kernel.  Up to 64 rows the decode kernel and the reduction beat it even unsplit
  // (a 496-linear decode step at 32 rows: 4.74 ms against 6.86 ms).
  if (split_k == 1 && p.M > DEC_DN_MAX)
    return nvfp4_linear(A, gs_a, W, segs, nseg, epilogue, ep, out, out_kind, ldo, stream);
  DeviceInfo *dev = nullptr;
  if (nvfp4_status_t st = current_device(&dev)) return st;
  return launch_splitk(p, A, W, split_k, static_cast<float *>(workspace), dev,
                       reinterpret_cast<cudaStream_t>(stream));
}

nvfp4_status_t nvfp4_linear_splitk_noalloc(const nvfp4_operand_t *A, const float *gs_a, const nvfp4_operand_t *W,
                                           const nvfp4_segment_t *segs, int nseg, int epilogue,
                                           const nvfp4_epilogue_params_t *ep, void *out, int out_kind, int64_t ldo,
                                           int split_k, nvfp4_stream_t stream) {
  NvtxRange nvtx("nvfp4_linear_splitk_noalloc");
  using namespace gemm;
  Params p;
  if (nvfp4_status_t st = prepare_linear(A, gs_a, W, segs, nseg, epilogue, ep, out, out_kind, ldo, p)) return st;
  if (split_k < 1 || split_k > p.k_tiles) return NVFP4_ERR_INVALID_ARG;
  // One split above decode size needs no partials: the ordinary kernel, which allocates
  // nothing either (as in nvfp4_linear_splitk).
  if (split_k == 1 && p.M > DEC_DN_MAX)
    return nvfp4_linear(A, gs_a, W, segs, nseg, epilogue, ep, out, out_kind, ldo, stream);
  if (nvfp4_splitk_workspace_bytes(p.M, p.N, split_k) > NVFP4_NOALLOC_SCRATCH_BYTES)
    return NVFP4_ERR_UNSUPPORTED_SHAPE;  // the partials do not fit the fixed scratch array
  DeviceInfo *dev = nullptr;
  if (nvfp4_status_t st = current_device(&dev)) return st;
  float *scratch = nullptr;
  if (nvfp4_status_t st = noalloc_scratch(&scratch)) return st;
  return launch_splitk(p, A, W, split_k, scratch, dev, reinterpret_cast<cudaStream_t>(stream));
}

nvfp4_status_t nvfp4_unswizzle_scales(const uint8_t *scales, int64_t rows, int64_t cols, uint8_t *out, int64_t ld,
                                      nvfp4_stream_t stream) {
  NvtxRange nvtx("nvfp4_unswizzle_scales");
  if (!scales || !out || rows < 1 || cols < 16 || ld < cols / 16) return NVFP4_ERR_INVALID_ARG;
  if (cols % 16 != 0 || rows > kMaxDim || cols > kMaxDim) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (!aligned(scales, 16)) return NVFP4_ERR_MISALIGNED;
  DeviceInfo *dev = nullptr;
  if (nvfp4_status_t st = current_device(&dev)) return st;
  UnswizzleArgs a;
  a.scales = scales;
  a.out = out;
  a.rows = rows;
  a.kb = cols / 16;
  a.kb_atoms = (a.kb + 3) / 4;
  a.ld = ld;
  const int64_t want = (rows * a.kb_atoms + kLayoutThreads - 1) / kLayoutThreads;
  const int64_t cap = int64_t(dev->sms) * 8;
  const int grid = static_cast<int>(want < cap ? want : cap);
  return launch_pdl(unswizzle_scales_kernel, dim3(grid), dim3(kLayoutThreads), 0,
                    reinterpret_cast<cudaStream_t>(stream), 1, a);
}

nvfp4_status_t nvfp4_pack_weight(const nvfp4_operand_t *parts, int nparts, uint8_t *codes, uint8_t *scales,
                                 int64_t rows_out, nvfp4_stream_t stream) {
  NvtxRange nvtx("nvfp4_pack_weight");
  if (!parts || !codes || !scales || nparts < 1 || nparts > NVFP4_MAX_SEGMENTS) return NVFP4_ERR_INVALID_ARG;
  PackArgs a{};
  const int64_t K = parts[0].K;
  int64_t row = 0;
  for (int i = 0; i < nparts; ++i) {
    const nvfp4_operand_t &q = parts[i];
    if (!q.codes || !q.scales || q.rows < 1 || q.K != K) return NVFP4_ERR_INVALID_ARG;
    if (!aligned(q.codes, 16) || !aligned(q.scales, 16)) return NVFP4_ERR_MISALIGNED;
    a.codes[i] = q.codes;
    a.scales[i] = q.scales;
    a.row0[i] = row;
    row += q.rows;
  }
  a.row0[nparts] = row;
  if (K < 64 || rows_out < row) return NVFP4_ERR_INVALID_ARG;
  if (K % 64 != 0 || rows_out > kMaxDim || K > kMaxDim) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (!aligned(codes, 16) || !aligned(scales, 16)) return NVFP4_ERR_MISALIGNED;
  DeviceInfo *dev = nullptr;
  if (nvfp4_status_t st = current_device(&dev)) return st;
  a.nparts = nparts;
  a.out_codes = codes;
  a.out_scales = scales;
  a.rows_out = rows_out;
  a.code_vecs = K / 32;
  a.kb_atoms = K / 64;
  const int64_t tasks = rows_out * a.code_vecs + (rows_out + 127) / 128 * 128 * a.kb_atoms;
  const int64_t want = (tasks + kLayoutThreads - 1) / kLayoutThreads;
  const int64_t cap = int64_t(dev->sms) * 8;
  const int grid = static_cast<int>(want < cap ? want : cap);
  return launch_pdl(pack_weight_kernel, dim3(grid), dim3(kLayoutThreads), 0, reinterpret_cast<cudaStream_t>(stream), 1,
                    a);
}

nvfp4_status_t nvfp4_fold_segments(uint8_t *scales, int64_t rows, int64_t cols, const nvfp4_segment_t *segs,
                                   int nseg, float *gs_common_out, nvfp4_stream_t stream) {
  NvtxRange nvtx("nvfp4_fold_segments");
  if (!scales || !segs || !gs_common_out || rows < 1 || cols < 1) return NVFP4_ERR_INVALID_ARG;
  if (nseg < 1 || nseg > NVFP4_MAX_SEGMENTS) return NVFP4_ERR_INVALID_ARG;
  if (cols % 16 != 0 || rows > kMaxDim || cols > kMaxDim) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (!aligned(scales, 16) || !aligned(gs_common_out, 4)) return NVFP4_ERR_MISALIGNED;
  FoldArgs a{};
  int64_t expect = 0;
  for (int i = 0; i < nseg; ++i) {
    if (!segs[i].gs_w || !aligned(segs[i].gs_w, 4)) return NVFP4_ERR_INVALID_ARG;
    if (segs[i].gs_w == gs_common_out) return NVFP4_ERR_INVALID_ARG;  // read while written
    if (segs[i].n_begin != expect || segs[i].n_end <= segs[i].n_begin) return NVFP4_ERR_INVALID_ARG;
    a.seg_begin[i] = static_cast<int>(segs[i].n_begin);
    a.seg_end[i] = static_cast<int>(segs[i].n_end);
    a.gs[i] = segs[i].gs_w;
    expect = segs[i].n_end;
  }
  if (expect != rows) return NVFP4_ERR_INVALID_ARG;
  DeviceInfo *dev = nullptr;
  if (nvfp4_status_t st = current_device(&dev)) return st;
  a.scales = scales;
  a.rows = rows;
  a.kb = cols / 16;
  a.kb_atoms = (a.kb + 3) / 4;
  a.bytes = static_cast<int64_t>(nvfp4_scale_bytes(rows, cols));
  a.nseg = nseg;
  a.gs_common = gs_common_out;
  const int64_t want = (a.bytes / 16 + kFoldThreads - 1) / kFoldThreads;
  const int64_t cap = int64_t(dev->sms) * 8;
  const int grid = static_cast<int>(want < cap ? want : cap);
  return launch_pdl(fold_scales_kernel, dim3(grid), dim3(kFoldThreads), 0, reinterpret_cast<cudaStream_t>(stream), 1,
                    a);
}

nvfp4_status_t nvfp4_fp8_scale(const void *x_bf16, int64_t rows, int64_t cols, int64_t ld, float *scale_out,
                               nvfp4_stream_t stream) {
  NvtxRange nvtx("nvfp4_fp8_scale");
  if (!x_bf16 || !scale_out || rows < 1 || cols < 1 || ld < cols) return NVFP4_ERR_INVALID_ARG;
  if (cols % 16 != 0 || rows > kMaxDim || cols > kMaxDim) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (!aligned(x_bf16, 16) || ld % 8 != 0 || !aligned(scale_out, 4)) return NVFP4_ERR_MISALIGNED;
  DeviceInfo *dev = nullptr;
  if (nvfp4_status_t st = current_device(&dev)) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (cudaMemsetAsync(scale_out, 0, sizeof(float), s) != cudaSuccess) return NVFP4_ERR_CUDA;
  AmaxArgs a;
  a.x = static_cast<const uint16_t *>(x_bf16);
  a.rows = rows;
  a.cols = cols;
  a.ld = ld;
  a.amax_bits = reinterpret_cast<unsigned int *>(scale_out);
  const int64_t vecs = rows * (cols / 8);
  const int64_t want = (vecs / 4 + kAmaxThreads - 1) / kAmaxThreads;
  const int64_t cap = int64_t(dev->sms) * 4;
  const int grid = static_cast<int>(want < 1 ? 1 : (want < cap ? want : cap));
  if (nvfp4_status_t e = launch_pdl(amax_kernel, dim3(grid), dim3(kAmaxThreads), 0, s, 1, a)) return e;
  return launch_pdl(fp8_scale_finalize_kernel, dim3(1), dim3(1), 0, s, 1, scale_out);
}

nvfp4_status_t nvfp4_kv_cache_fp8(const void *k_bf16, const void *v_bf16, int64_t tokens, int64_t width,
                                  int64_t ld, const float *k_scale, const float *v_scale, const int64_t *slots,
                                  uint8_t *k_cache, uint8_t *v_cache, int64_t num_slots, nvfp4_stream_t stream) {
  NvtxRange nvtx("nvfp4_kv_cache_fp8");
  if (!k_bf16 || !v_bf16 || !k_scale || !v_scale || !slots || !k_cache || !v_cache) return NVFP4_ERR_INVALID_ARG;
  if (tokens < 1 || width < 1 || ld < width || num_slots < 1) return NVFP4_ERR_INVALID_ARG;
  if (width % 16 != 0 || tokens > kMaxDim || width > kMaxDim) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (!aligned(k_bf16, 16) || !aligned(v_bf16, 16) || ld % 8 != 0 || !aligned(k_scale, 4) ||
      !aligned(v_scale, 4) || !aligned(slots, 8) || !aligned(k_cache, 16) || !aligned(v_cache, 16))
    return NVFP4_ERR_MISALIGNED;
  DeviceInfo *dev = nullptr;
  if (nvfp4_status_t st = current_device(&dev)) return st;
  KvArgs a;
  a.k = static_cast<const uint16_t *>(k_bf16);
  a.v = static_cast<const uint16_t *>(v_bf16);
  a.tokens = tokens;
  a.width = width;
  a.ld = ld;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.slots = slots;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.num_slots = num_slots;
  const int64_t chunks = tokens * (width / 16);
  const int64_t want = (chunks + kKvThreads - 1) / kKvThreads;
  const int64_t cap = int64_t(dev->sms) * 8;
  const int grid = static_cast<int>(want < cap ? want : cap);
  return launch_pdl(kv_cache_fp8_kernel, dim3(grid), dim3(kKvThreads), 0, reinterpret_cast<cudaStream_t>(stream), 1,
                    a);
}

nvfp4_status_t nvfp4_gdn_recurrence(const void *q_bf16, const void *k_bf16, int64_t ld_qk, const void *v_bf16,
                                    int64_t ld_v, const float *g, const float *beta, int64_t ld_gate,
                                    const int32_t *cu_seqlens, int64_t n_seqs, int64_t tokens, int n_key_heads,
                                    int n_value_heads, int head_dim, float *state, int initial_state, void *out,
                                    int64_t ld_out, int out_kind, nvfp4_stream_t stream) {
  NvtxRange nvtx("nvfp4_gdn_recurrence");
  if (!q_bf16 || !k_bf16 || !v_bf16 || !g || !beta || !cu_seqlens || !state || !out) return NVFP4_ERR_INVALID_ARG;
  if (n_seqs < 1 || tokens < 0 || n_key_heads < 1 || n_value_heads < 1 || n_value_heads % n_key_heads != 0)
    return NVFP4_ERR_INVALID_ARG;
  if (out_kind != NVFP4_OUT_BF16 && out_kind != NVFP4_OUT_F32) return NVFP4_ERR_INVALID_ARG;
  if (head_dim != gdn::kDim || n_seqs > 65535 || n_value_heads > 65535 || tokens > kMaxDim)
    return NVFP4_ERR_UNSUPPORTED_SHAPE;
  const int64_t wk = int64_t(n_key_heads) * gdn::kDim, wv = int64_t(n_value_heads) * gdn::kDim;
  if (ld_qk < wk || ld_v < wv || ld_gate < n_value_heads || ld_out < wv) return NVFP4_ERR_INVALID_ARG;
  if (!aligned(q_bf16, 16) || !aligned(k_bf16, 16) || !aligned(v_bf16, 16) || ld_qk % 8 != 0 || ld_v % 8 != 0 ||
      !aligned(g, 4) || !aligned(beta, 4) || !aligned(cu_seqlens, 4) || !aligned(state, 16) || !aligned(out, 16) ||
      ld_out % (out_kind == NVFP4_OUT_BF16 ? 8 : 4) != 0)
    return NVFP4_ERR_MISALIGNED;
  DeviceInfo *dev = nullptr;
  if (nvfp4_status_t st = current_device(&dev)) return st;
  gdn::Args a;
  a.q = static_cast<const uint16_t *>(q_bf16);
  a.k = static_cast<const uint16_t *>(k_bf16);
  a.v = static_cast<const uint16_t *>(v_bf16);
  a.ld_qk = ld_qk;
  a.ld_v = ld_v;
  a.g = g;
  a.beta = beta;
  a.ld_gate = ld_gate;
  a.cu_seqlens = cu_seqlens;
  a.tokens = tokens;
  a.heads_per_key = n_value_heads / n_key_heads;
  a.state = state;
  a.initial = initial_state != 0;
  a.out = out;
  a.ld_out = ld_out;
  a.out_fp32 = out_kind == NVFP4_OUT_F32;
  const dim3 grid(gdn::kColBlocks, n_value_heads, static_cast<unsigned>(n_seqs));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  // Long sequences (prefill): the chunked form on the tensor cores.
  if (tokens >= 64 * n_seqs)
    return launch_pdl(gdn::chunk_kernel, dim3(gdn::kChunkColBlocks, n_value_heads, static_cast<unsigned>(n_seqs)),
                      dim3(gdn::kChunkThreads), sizeof(gdn::ChunkSmem), s, 1, a);
  // Shorter sequences stage fewer tokens at a time: a smaller shared-memory footprint,
  // so more CTAs per SM in the state-bound case, and less staging work spent on the
  // empty slots of a chunk.
  if (tokens >= 16 * n_seqs)
    return launch_pdl(gdn::recurrence_kernel<32>, grid, dim3(gdn::kThreads), sizeof(gdn::Smem<32>), s, 1, a);
  if (tokens >= 4 * n_seqs)
    return launch_pdl(gdn::recurrence_kernel<16>, grid, dim3(gdn::kThreads), sizeof(gdn::Smem<16>), s, 1, a);
  // About one token per sequence (decode): one warp per four state columns.
  return launch_pdl(gdn::column_kernel, dim3(gdn::kColBlocksPerHead, n_value_heads, static_cast<unsigned>(n_seqs)),
                    dim3(gdn::kColThreads), 0, s, 1, a);
}

nvfp4_status_t nvfp4_rope_table(float *table, int64_t max_pos, int rot_dim, double base, nvfp4_stream_t stream) {
  NvtxRange nvtx("nvfp4_rope_table");
  if (!table || max_pos < 1 || rot_dim < 1 || !(base > 0.0) || !std::isfinite(base)) return NVFP4_ERR_INVALID_ARG;
  if (rot_dim % 16 != 0 || rot_dim > 256 || max_pos > kMaxDim) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (!aligned(table, 16)) return NVFP4_ERR_MISALIGNED;
  DeviceInfo *dev = nullptr;
  if (nvfp4_status_t st = current_device(&dev)) return st;
  const int64_t want = (max_pos * (rot_dim / 2) + headnorm::kTableThreads - 1) / headnorm::kTableThreads;
  const int64_t cap = int64_t(dev->sms) * 16;
  return launch_pdl(headnorm::rope_table_kernel, dim3(static_cast<unsigned>(want < cap ? want : cap)),
                    dim3(headnorm::kTableThreads), 0, reinterpret_cast<cudaStream_t>(stream), 1, table, max_pos,
                    rot_dim, base);
}

nvfp4_status_t nvfp4_qk_norm_rope(const void *q_bf16, int64_t ld_q, const void *k_bf16, int64_t ld_k, int64_t tokens,
                                  int n_heads, int n_kv_heads, int head_dim, const void *w_q_bf16,
                                  const void *w_k_bf16, float w_offset, float eps, const int64_t *positions,
                                  const float *table, int64_t max_pos, int rot_dim, int interleaved, void *q_out,
                                  int64_t ld_qo, void *k_out, int64_t ld_ko, nvfp4_stream_t stream) {
  NvtxRange nvtx("nvfp4_qk_norm_rope");
  if (!q_bf16 || !k_bf16 || !w_q_bf16 || !w_k_bf16 || !q_out || !k_out) return NVFP4_ERR_INVALID_ARG;
  if (tokens < 0 || n_heads < 1 || n_kv_heads < 1 || rot_dim < 0 || !(eps >= 0.0f) || !std::isfinite(eps) ||
      !std::isfinite(w_offset))
    return NVFP4_ERR_INVALID_ARG;
  if (rot_dim > 0 && (!positions || !table || max_pos < 1)) return NVFP4_ERR_INVALID_ARG;
  if ((head_dim != 64 && head_dim != 128 && head_dim != 256) || rot_dim % 16 != 0 || rot_dim > head_dim ||
      n_heads > 65535 || n_kv_heads > 65535 || tokens > kMaxDim)
    return NVFP4_ERR_UNSUPPORTED_SHAPE;
  const int64_t wq = int64_t(n_heads) * head_dim, wk = int64_t(n_kv_heads) * head_dim;
  if (ld_q < wq || ld_qo < wq || ld_k < wk || ld_ko < wk) return NVFP4_ERR_INVALID_ARG;
  if (!aligned(q_bf16, 16) || !aligned(k_bf16, 16) || !aligned(q_out, 16) || !aligned(k_out, 16) ||
      !aligned(w_q_bf16, 16) || !aligned(w_k_bf16, 16) || ld_q % 8 != 0 || ld_k % 8 != 0 || ld_qo % 8 != 0 ||
      ld_ko % 8 != 0 || (rot_dim > 0 && (!aligned(positions, 8) || !aligned(table, 16))))
    return NVFP4_ERR_MISALIGNED;
  DeviceInfo *dev = nullptr;
  if (nvfp4_status_t st = current_device(&dev)) return st;
  if (tokens == 0) return NVFP4_OK;
  headnorm::Args a;
  a.q = static_cast<const uint16_t *>(q_bf16);
  a.k = static_cast<const uint16_t *>(k_bf16);
  a.ld_q = ld_q;
  a.ld_k = ld_k;
  a.tokens = tokens;
  a.heads = n_heads;
  a.kv_heads = n_kv_heads;
  a.w_q = static_cast<const uint16_t *>(w_q_bf16);
  a.w_k = static_cast<const uint16_t *>(w_k_bf16);
  a.w_offset = w_offset;
  a.eps = eps;
  a.positions = positions;
  a.table = table;
  a.max_pos = rot_dim > 0 ? max_pos : 1;
  a.rot = rot_dim;
  a.interleaved = interleaved != 0;
  a.q_out = static_cast<uint16_t *>(q_out);
  a.k_out = static_cast<uint16_t *>(k_out);
  a.ld_qo = ld_qo;
  a.ld_ko = ld_ko;
  // Few tokens: a warp takes one head group, so that all SMs have work; many: whole
  // tokens, so that the table row and weights are read once.
  const int per_warp = 32 / (head_dim / 8);
  const int groups = (n_heads + per_warp - 1) / per_warp + (n_kv_heads + per_warp - 1) / per_warp;
  const int64_t warps = int64_t(dev->sms) * 32;
  int64_t parts = tokens >= warps ? 1 : (warps + tokens - 1) / tokens;
  if (parts > groups) parts = groups;
  a.per_part = static_cast<int>((groups + parts - 1) / parts);
  a.parts = (groups + a.per_part - 1) / a.per_part;
  const int64_t ctas = (tokens * a.parts * 32 + headnorm::kThreads - 1) / headnorm::kThreads;
  if (ctas > kMaxDim) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  auto kernel = head_dim == 64 ? headnorm::head_norm_kernel<64>
                : head_dim == 128 ? headnorm::head_norm_kernel<128> : headnorm::head_norm_kernel<256>;
  return launch_pdl(kernel, dim3(static_cast<unsigned>(ctas)), dim3(headnorm::kThreads), 0,
                    reinterpret_cast<cudaStream_t>(stream), 1, a);
}

nvfp4_status_t nvfp4_kv_append(const void *k_bf16, int64_t ld_k, const void *v_bf16, int64_t ld_v,
                               const nvfp4_batch_t *batch, const nvfp4_block_cache_t *cache, nvfp4_stream_t stream) {
  NvtxRange nvtx("nvfp4_kv_append");
  int log_block = 0;
  if (!k_bf16 || !v_bf16) return NVFP4_ERR_INVALID_ARG;
  if (nvfp4_status_t st = check_batch(batch, cache, &log_block)) return st;
  const int64_t width = int64_t(cache->n_kv_heads) * cache->head_dim;
  if (ld_k < width || ld_v < width) return NVFP4_ERR_INVALID_ARG;
  if (!aligned(k_bf16, 16) || !aligned(v_bf16, 16) || ld_k % 8 != 0 || ld_v % 8 != 0) return NVFP4_ERR_MISALIGNED;
  DeviceInfo *dev = nullptr;
  if (nvfp4_status_t st = current_device(&dev)) return st;
  if (batch->tokens == 0) return NVFP4_OK;
  kvblock::Args a;
  a.k = static_cast<const uint16_t *>(k_bf16);
  a.v = static_cast<const uint16_t *>(v_bf16);
  a.ld_k = ld_k;
  a.ld_v = ld_v;
  a.cu_seqlens = batch->cu_seqlens;
  a.kv_lens = batch->kv_lens;
  a.tokens = batch->tokens;
  a.n_seqs = static_cast<int>(batch->n_seqs);
  a.kv_heads = cache->n_kv_heads;
  a.log_d = cache->head_dim == 64 ? 6 : cache->head_dim == 128 ? 7 : 8;
  a.table = batch->block_table;
  a.ld_table = batch->ld_table;
  a.max_kv = batch->max_blocks << log_block;
  a.k_cache = cache->k;
  a.v_cache = cache->v;
  a.k_scales = cache->k_scales;
  a.v_scales = cache->v_scales;
  a.num_blocks = cache->num_blocks;
  a.log_block = log_block;
  const int64_t slots = (batch->tokens >> log_block) + 2 * batch->n_seqs;
  const dim3 grid(static_cast<unsigned>(slots), cache->n_kv_heads, 2);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  // Threads and 16-byte pieces per thread that hold one block of one head.
  const int pieces = cache->block_size * cache->head_dim / 8;
  if (pieces <= 256) return launch_pdl(kvblock::append_kernel<128, 2>, grid, dim3(128), 0, s, 1, a);
  if (pieces <= 1024) return launch_pdl(kvblock::append_kernel<256, 4>, grid, dim3(256), 0, s, 1, a);
  return launch_pdl(kvblock::append_kernel<512, 8>, grid, dim3(512), 0, s, 1, a);
}

size_t nvfp4_attention_workspace_bytes(int64_t tokens, int64_t n_seqs, int n_heads, int n_kv_heads, int head_dim) {
  if (tokens < 0 || n_seqs < 1 || n_heads < 1 || n_kv_heads < 1 || n_heads % n_kv_heads != 0 || head_dim < 1) return 0;
  if (tokens > kMaxDim || n_seqs > 65535 || n_heads > 65535 || head_dim > 256) return 0;
  const AttnWorkspace w = attn_workspace(tokens, n_seqs, n_heads, n_kv_heads, head_dim);
  return w.fits() ? w.bytes : 0;
}

nvfp4_status_t nvfp4_attention(const void *q_bf16, int64_t ld_q, int n_heads, const nvfp4_batch_t *batch,
                               const nvfp4_block_cache_t *cache, float softmax_scale, int causal, void *out,
                               int out_kind, int64_t ld_out, void *workspace, size_t workspace_bytes,
                               nvfp4_stream_t stream) {
  NvtxRange nvtx("nvfp4_attention");
  int log_block = 0;
  if (!q_bf16 || !out || !workspace) return NVFP4_ERR_INVALID_ARG;
  if (nvfp4_status_t st = check_batch(batch, cache, &log_block)) return st;
  if (n_heads < 1 || n_heads % cache->n_kv_heads != 0 || !std::isfinite(softmax_scale * 1.4426950408889634f))
    return NVFP4_ERR_INVALID_ARG;
  if (out_kind != NVFP4_OUT_BF16 && out_kind != NVFP4_OUT_F32) return NVFP4_ERR_INVALID_ARG;
  if (n_heads > 65535 || batch->tokens * (n_heads / cache->n_kv_heads) > kMaxDim / 2) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  const int64_t width = int64_t(n_heads) * cache->head_dim;
  if (ld_q < width || ld_out < width) return NVFP4_ERR_INVALID_ARG;
  if (!aligned(q_bf16, 16) || ld_q % 8 != 0 || !aligned(out, 16) || !aligned(workspace, 16) ||
      ld_out % (out_kind == NVFP4_OUT_BF16 ? 8 : 4) != 0)
    return NVFP4_ERR_MISALIGNED;
  const AttnWorkspace w = attn_workspace(batch->tokens, batch->n_seqs, n_heads, cache->n_kv_heads, cache->head_dim);
  if (!w.fits()) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (workspace_bytes < w.bytes) return NVFP4_ERR_INVALID_ARG;
  DeviceInfo *dev = nullptr;
  if (nvfp4_status_t st = current_device(&dev)) return st;
  if (batch->tokens == 0) return NVFP4_OK;
  attn::Args a;
  a.q = static_cast<const uint16_t *>(q_bf16);
  a.ld_q = ld_q;
  a.cu_seqlens = batch->cu_seqlens;
  a.kv_lens = batch->kv_lens;
  a.tokens = batch->tokens;
  a.n_seqs = static_cast<int>(batch->n_seqs);
  a.kv_heads = cache->n_kv_heads;
  a.group = n_heads / cache->n_kv_heads;
  a.table = batch->block_table;
  a.ld_table = batch->ld_table;
  a.max_kv = batch->max_blocks << log_block;
  a.k = cache->k;
  a.v = cache->v;
  a.k_scales = cache->k_scales;
  a.v_scales = cache->v_scales;
  a.num_blocks = cache->num_blocks;
  a.log_block = log_block;
  a.scale_log2 = softmax_scale * 1.4426950408889634f;
  a.causal = causal != 0;
  a.out = out;
  a.ld_out = ld_out;
  a.out_fp32 = out_kind == NVFP4_OUT_F32;
  char *base = static_cast<char *>(workspace);
  a.n_units = reinterpret_cast<int *>(base);
  a.desc = reinterpret_cast<int4 *>(base + w.desc);
  a.desc2 = reinterpret_cast<int2 *>(base + w.desc2);
  a.part_ml = reinterpret_cast<float2 *>(base + w.part_ml);
  a.part = reinterpret_cast<float *>(base + w.part);
  a.max_decode_rows = kDecodeRows;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const int i = cache->head_dim == 64 ? 0 : cache->head_dim == 128 ? 1 : 2;
  int ctas = dev->sms * (i == 0 ? attn::Cfg<64>::CTAS : i == 1 ? attn::Cfg<128>::CTAS : attn::Cfg<256>::CTAS);
  if (ctas > kMaxAttnCtas) ctas = kMaxAttnCtas;
  const int tile = i == 0 ? attn::Cfg<64>::TILE : i == 1 ? attn::Cfg<128>::TILE : attn::Cfg<256>::TILE;
  a.whole = a.max_kv <= int64_t(attn::kWholeTiles) * tile;
  CUtensorMap k_map, v_map;
  const int box = attn::box_log(log_block, cache->head_dim);
  if (!encode_cache_map(&k_map, cache->k, cache, box) || !encode_cache_map(&v_map, cache->v, cache, box))
    return NVFP4_ERR_CUDA;
  auto launch_decode = [&](auto kernel, auto combine, int smem) {
    if (nvfp4_status_t e = launch_pdl(kernel, dim3(ctas), dim3(attn::kThreads), smem, s, 1, a, k_map, v_map)) return e;
    if (a.whole) return NVFP4_OK;
    const int threads = i == 0 ? attn::Join<64>::THREADS : i == 1 ? attn::Join<128>::THREADS : attn::Join<256>::THREADS;
    return launch_pdl(combine, dim3(static_cast<unsigned>(w.units), attn::kRows / attn::Join<128>::ROWS), dim3(threads), 0, s, 1, a);
  };
  if (nvfp4_status_t e = i == 0 ? launch_decode(attn::decode_kernel<64>, attn::combine_kernel<64>, attn::decode_smem_bytes<64>())
                         : i == 1 ? launch_decode(attn::decode_kernel<128>, attn::combine_kernel<128>, attn::decode_smem_bytes<128>())
                                  : launch_decode(attn::decode_kernel<256>, attn::combine_kernel<256>, attn::decode_smem_bytes<256>()))
    return e;
  // Only the device knows the sequences' lengths; no prompt fits in few rows.
  const int64_t rows = batch->tokens * a.group;
  if (rows <= kDecodeRows || w.items == 0) return NVFP4_OK;
  const int most = i == 2 ? attn::prompt::Cfg<256>::LOG_BOX : attn::prompt::Cfg<128>::LOG_BOX;
  if (!encode_cache_map(&k_map, cache->k, cache, log_block < most ? log_block : most)) return NVFP4_ERR_CUDA;
  const int64_t prompt_tiles = a.max_kv / attn::prompt::Cfg<128>::BN;
  const int64_t most_splits = prompt_tiles / attn::prompt::kMinTiles;
  a.splits = prompt_splits(w.items, most_splits < 1 ? 1 : most_splits < w.splits ? static_cast<int>(most_splits) : w.splits);
  a.prompt_ml = reinterpret_cast<float2 *>(base + w.prompt_ml);
  a.prompt_part = reinterpret_cast<float *>(base + w.prompt_part);
  auto launch_prompt = [&](auto kernel, auto join, int tile_rows, int smem) {
    if (nvfp4_status_t e = launch_pdl(kernel, dim3(static_cast<unsigned>(w.items * a.splits)),
                                      dim3(attn::prompt::kThreads), smem, s, 1, a, k_map))
      return e;
    if (a.splits == 1) return NVFP4_OK;
    return launch_pdl(join, dim3(static_cast<unsigned>(w.items), tile_rows / attn::prompt::kJoinRows),
                      dim3(attn::prompt::kJoinThreads), 0, s, 1, a);
  };
  namespace ap = attn::prompt;
  if (i == 0) return launch_prompt(ap::prompt_kernel<64>, ap::join_kernel<64>, ap::Cfg<64>::ROWS, ap::smem_bytes<64>());
  if (i == 1) return launch_prompt(ap::prompt_kernel<128>, ap::join_kernel<128>, ap::Cfg<128>::ROWS, ap::smem_bytes<128>());
  return launch_prompt(ap::prompt_kernel<256>, ap::join_kernel<256>, ap::Cfg<256>::ROWS, ap::smem_bytes<256>());
}

nvfp4_status_t nvfp4_matvec(const void *x_bf16, int64_t ld_x, int64_t M, const nvfp4_operand_t *W,
                            const nvfp4_segment_t *segs, int nseg, void *out, int out_kind, int64_t ldo,
                            nvfp4_stream_t stream) {
  NvtxRange nvtx("nvfp4_matvec");
  if (!x_bf16 || !W || !segs || !out || !W->codes || !W->scales) return NVFP4_ERR_INVALID_ARG;
  if (M < 1 || W->rows < 1 || W->K < 1) return NVFP4_ERR_INVALID_ARG;
  if (out_kind != NVFP4_OUT_BF16 && out_kind != NVFP4_OUT_F32) return NVFP4_ERR_INVALID_ARG;
  if (nseg < 1 || nseg > NVFP4_MAX_SEGMENTS) return NVFP4_ERR_INVALID_ARG;
  const int64_t N = W->rows, K = W->K;
  if (M > 16 || N > kMaxDim || K > kMaxDim || K % 64 != 0) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  if (ld_x < K || ldo < N) return NVFP4_ERR_INVALID_ARG;
  matvec::Args a;
  int64_t expect = 0;
  for (int i = 0; i < nseg; ++i) {
    if (!segs[i].gs_w || !aligned(segs[i].gs_w, 4)) return NVFP4_ERR_INVALID_ARG;
    if (segs[i].n_begin != expect || segs[i].n_end <= segs[i].n_begin) return NVFP4_ERR_INVALID_ARG;
    a.seg[i].n_begin = static_cast<int>(segs[i].n_begin);
    a.seg[i].n_end = static_cast<int>(segs[i].n_end);
    a.seg[i].gs_w = segs[i].gs_w;
    expect = segs[i].n_end;
  }
  if (expect != N) return NVFP4_ERR_INVALID_ARG;
  if (!aligned(x_bf16, 16) || ld_x % 8 != 0 || !aligned(W->codes, 16) || !aligned(W->scales, 16) ||
      !aligned(out, out_kind == NVFP4_OUT_BF16 ? 2 : 4))
    return NVFP4_ERR_MISALIGNED;
  DeviceInfo *dev = nullptr;
  if (nvfp4_status_t st = current_device(&dev)) return st;
  a.x = static_cast<const uint16_t *>(x_bf16);
  a.ld_x = ld_x;
  a.M = static_cast<int>(M);
  a.scales = W->scales;
  a.N = N;
  a.K = K;
  a.nseg = nseg;
  a.out = out;
  a.ldo = ldo;
  a.out_fp32 = out_kind == NVFP4_OUT_F32;
  const int64_t blocks = (N + matvec::kBN - 1) / matvec::kBN;
  // K split over a cluster of up to 8 CTAs, as many as find a place at once (two per SM), then as
  // few as have the same number of steps each.
  const int64_t steps = (K + matvec::kStep - 1) / matvec::kStep;
  int64_t most = 2 * dev->sms / blocks;
  most = most < 1 ? 1 : most > 8 ? 8 : most;
  const int64_t each = (steps + most - 1) / most;
  const int cluster = static_cast<int>((steps + each - 1) / each);
  a.k_per_cta = (steps + cluster - 1) / cluster * matvec::kStep;
  if (blocks * cluster > kMaxDim) return NVFP4_ERR_UNSUPPORTED_SHAPE;
  CUtensorMap map;
  if (!encode_codes_map(&map, W->codes, N, K, matvec::kBN)) return NVFP4_ERR_CUDA;
  const dim3 grid(static_cast<unsigned>(blocks * cluster));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (M <= 8)
    return launch_pdl(matvec::matvec_kernel<1>, grid, dim3(matvec::kThreads), matvec::smem_bytes<1>(), s, cluster, a, map);
  return launch_pdl(matvec::matvec_kernel<2>, grid, dim3(matvec::kThreads), matvec::smem_bytes<2>(), s, cluster, a, map);
}

nvfp4_status_t nvfp4_selftest_stalled_linear(const nvfp4_operand_t *A, const float *gs_a, const nvfp4_operand_t *W,
                                             const nvfp4_segment_t *segs, int nseg, float *out, int64_t ldo,
                                             int stall_stage, nvfp4_stream_t stream) {
  NvtxRange nvtx("nvfp4_selftest_stalled_linear");
  using namespace gemm;
  Params p;
  if (nvfp4_status_t st = prepare_linear(A, gs_a, W, segs, nseg, NVFP4_EPI_NONE, nullptr, out, NVFP4_OUT_F32, ldo, p))
    return st;
  if (p.M > BM || p.N > BN) return NVFP4_ERR_UNSUPPORTED_SHAPE;  // one tile, one CTA
  if (stall_stage < 0 || stall_stage >= p.k_tiles) return NVFP4_ERR_INVALID_ARG;
  DeviceInfo *dev = nullptr;
  if (nvfp4_status_t st = current_device(&dev)) return st;
  CUtensorMap tmA, tmB;
  if (!make_codes_map(&tmA, A->codes, p.M, p.K) || !make_codes_map(&tmB, W->codes, p.N, p.K)) return NVFP4_ERR_CUDA;
  p.m_tiles = 1;
  p.n_tiles = 1;
  p.stall_stage = stall_stage;
  return launch_pdl(gemm_kernel<false, true>, dim3(1), dim3(NUM_THREADS), Plan1::BYTES,
                    reinterpret_cast<cudaStream_t>(stream), 1, tmA, tmB, p);
}

nvfp4_status_t nvfp4_get_device_status(int *code) {
  NvtxRange nvtx("nvfp4_get_device_status");
  if (!code) return NVFP4_ERR_INVALID_ARG;
  if (cudaDeviceSynchronize() != cudaSuccess) return NVFP4_ERR_CUDA;
  int v = 0, zero = 0;
  if (cudaMemcpyFromSymbol(&v, g_device_status, sizeof(int)) != cudaSuccess) return NVFP4_ERR_CUDA;
  if (cudaMemcpyToSymbol(g_device_status, &zero, sizeof(int)) != cudaSuccess) return NVFP4_ERR_CUDA;
  *code = v;
  return NVFP4_OK;
}

}  // extern "C"

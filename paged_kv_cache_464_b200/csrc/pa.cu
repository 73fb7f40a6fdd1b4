// pa.cu -- the C ABI of libpa_b200.so (declared in include/pa.h): host-side
// argument checks, TMA descriptor encoding and kernel launches.  The kernels
// themselves live in the pa_*.cuh headers, compiled here as one translation
// unit so that the per-device error word needs no separate device linking.
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdint>
#include <cstring>
#include <mutex>
#include <type_traits>
#include <utility>

#include "pa.h"
#include "pa_cache_ops.cuh"
#include "pa_decode.cuh"
#include "pa_prefill.cuh"
#include "pa_decode_fp8tc.cuh"
#include "pa_probe.cuh"
#include "pa_rope.cuh"
#include "pa_shared_prefix.cuh"
#include "pa_sparse.cuh"

#ifndef PA_PROGRAMMATIC_LAUNCH
#define PA_PROGRAMMATIC_LAUNCH 1
#endif
// Split sequences: 0 = a separate reduce kernel after the partition kernel
// (the default); 1 = the last partition CTA of each (sequence, KV head)
// combines the partials (one launch, plus a tiny counter-zeroing kernel).
// Measured on B200 the fused form is no faster on the GQA workload and ~5%
// slower on the long-context one: every split partition CTA then ends with a
// device-scope fence and an atomic round trip before it frees its SM slot.
#ifndef PA_FUSED_COMBINE
#define PA_FUSED_COMBINE 0
#endif

namespace {

using pa::kBlockSize;
using pa::kRowBytes;

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// Streaming multiprocessors of the current device, queried once per device
// (grids of the cache operations and the reduce are sized from it).  Falls
// back to 148 (a full B200) if the query fails.
constexpr int kMaxDevices = 128;
std::atomic<int> g_sm_count[kMaxDevices];

int sm_count() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 148;
  int n = g_sm_count[dev].load(std::memory_order_relaxed);
  if (n > 0) return n;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess || n <= 0) return 148;
  g_sm_count[dev].store(n, std::memory_order_relaxed);
  return n;
}

// Test hook (pa_test_stall_next_launch): armed by a test, consumed by the next
// decode or prefill launch of the armed kind; 0 = not armed.
std::atomic<int> g_stall_decode{0};
std::atomic<int> g_stall_prefill{0};
std::atomic<int> g_stall_prefix{0};

int elem_bytes(pa_dtype_t dt) {
  switch (dt) {
    case PA_F32: return 4;
    case PA_F16:
    case PA_BF16: return 2;
    case PA_FP8_E4M3: return 1;
  }
  return 0;
}

// Bytes of one (token, KV head) row: 256 for 16/32-bit caches, 128 for E4M3.
int row_bytes(pa_dtype_t dt) { return dt == PA_FP8_E4M3 ? 128 : kRowBytes; }

pa_status_t cache_shape_status(int64_t num_blocks, int block_size, int num_kv_heads, int head_dim,
                               pa_dtype_t dtype) {
  const int es = elem_bytes(dtype);
  if (es == 0) return PA_ERR_DTYPE;
  if (num_blocks <= 0 || num_blocks > INT32_MAX || block_size != kBlockSize || num_kv_heads <= 0 ||
      head_dim * es != row_bytes(dtype))
    return PA_ERR_SHAPE;
  return PA_OK;
}

// Every kernel is launched with programmatic stream serialisation: it may be
// scheduled while the previous kernel in the stream is still running, and it
// waits (griddepcontrol.wait) before touching global memory (but for the suffix
// walk of a shared prefix: pa_common.cuh, launch ordering), so stream order
// semantics are unchanged while the launch latency overlaps the previous tail.
template <typename... KArgs, typename... Args>
pa_status_t launch(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                   Args &&...args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = PA_PROGRAMMATIC_LAUNCH ? 1 : 0;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
  return e == cudaSuccess ? PA_OK : PA_ERR_CUDA;
}

// ---------------------------------------------------------------- TMA descriptors
PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static std::once_flag once;
  std::call_once(once, [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// The cache [NB][16][Hkv][R B] (R = 256 or 128) seen as a 5-D byte tensor
// {128 B, R/128 parts, Hkv, 16 tokens, NB}; the box is one 128-byte part of one
// (block, KV head) tile: {128, 1, 1, 16, 1} = 2 KiB (16 rows of 128 B),
// landing 128-byte swizzled.  R/128 boxes make the tile.
bool encode_cache_map(CUtensorMap *map, const void *cache, int64_t num_blocks, int num_kv_heads, int rb) {
  auto fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[5] = {128, (cuuint64_t)rb / 128, (cuuint64_t)num_kv_heads, (cuuint64_t)kBlockSize,
                              (cuuint64_t)num_blocks};
  const cuuint64_t strides[4] = {128, (cuuint64_t)rb, (cuuint64_t)num_kv_heads * rb,
                                 (cuuint64_t)kBlockSize * num_kv_heads * rb};
  const cuuint32_t box[5] = {128, 1, 1, kBlockSize, 1};
  const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  const CUresult r = fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 5, const_cast<void *>(cache), dims, strides, box,
                        estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS;
}

// ---------------------------------------------------------------- decode planning
// Library choice of the partition size: 1024 tokens for the tensor-core block
// math (16-bit caches, grouped heads), 512 for the CUDA-core one (measured best
// on B200 for the GQA and MHA workloads); one partition when the longest
// context fits.
int resolve_partition_size(int num_seqs, int num_heads, int num_kv_heads, int head_dim, int max_context_len,
                           int requested) {
  (void)num_seqs;
  if (max_context_len < 0 || requested < 0 || num_kv_heads <= 0) return -1;
  if (requested > 0) return requested % kBlockSize == 0 ? requested : -1;
  const bool tensor_core_math = head_dim == 128 && num_heads / num_kv_heads >= 2;
  const int P = tensor_core_math ? 1024 : 512;
  if (max_context_len <= P)
    return max_context_len <= kBlockSize ? kBlockSize : (max_context_len + kBlockSize - 1) / kBlockSize * kBlockSize;
  return P;
}

int max_partitions(int max_context_len, int partition_size) {
  const int np = (max_context_len + partition_size - 1) / partition_size;
  return np < 1 ? 1 : np;
}

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// Split-K workspace: m, l [S][Hq][NP] fp32, o [S][Hq][NP][D] fp32, then one
// counter per (sequence, KV head); each section 256-byte aligned.
struct WorkspaceLayout {
  size_t m_off, l_off, o_off, c_off, bytes;
};

WorkspaceLayout workspace_layout(int num_seqs, int num_heads, int num_kv_heads, int head_dim, int np) {
  WorkspaceLayout w{};
  if (np <= 1) return w;
  const size_t rows = (size_t)num_seqs * num_heads * np;
  w.m_off = 0;
  w.l_off = align256(rows * sizeof(float));
  w.o_off = w.l_off + align256(rows * sizeof(float));
  w.c_off = w.o_off + align256(rows * head_dim * sizeof(float));
  w.bytes = w.c_off + align256((size_t)num_seqs * num_kv_heads * sizeof(unsigned));
  return w;
}

template <typename T>
pa_status_t launch_reduce(const pa::DecodeParams &p, cudaStream_t stream);

template <typename T, int G, typename Math, int W = pa::kDecodeWarps>
pa_status_t launch_decode(const CUtensorMap &mk, const CUtensorMap &mv, const pa::DecodeParams &p,
                          cudaStream_t stream) {
  using SM = pa::DecodeSmem<T, G, Math, W>;
  auto kernel = pa::pa_decode_partition_kernel<T, G, Math, W>;
  // the attribute is per device; setting it on every call costs ~a microsecond of host time
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SM::kAlloc) != cudaSuccess)
    return PA_ERR_CUDA;
  const long long grid = (long long)p.num_seqs * p.num_kv_heads * p.max_partitions;
  if (grid == 0) return PA_OK;
  if (grid > INT32_MAX) return PA_ERR_SHAPE;
  if (p.ws_count != nullptr) {   // split call, combined in the partition kernel: counters start at 0
    const int n = p.num_seqs * p.num_kv_heads;
    const int ctas = (n + 255) / 256 < sm_count() ? (n + 255) / 256 : sm_count();
    pa_status_t st = launch(pa::zero_counts_kernel, dim3((unsigned)ctas), dim3(256), 0, stream, p.ws_count, n);
    if (st != PA_OK) return st;
  }
  pa_status_t st = launch(kernel, dim3((unsigned)grid), dim3(W * 32), SM::kAlloc, stream, mk, mv, p);
  if (st != PA_OK || p.max_partitions <= 1 || p.ws_count != nullptr) return st;
  return launch_reduce<T>(p, stream);
}

// Split-K reduce of a decode call's partials (after its partition kernel).
template <typename T>
pa_status_t launch_reduce(const pa::DecodeParams &p, cudaStream_t stream) {
  // warps per row: one per 8 partitions (at most kReduceWarps); a CTA takes
  // kReduceWarps / wpr rows at a time, the grid strides over the rest (at most
  // 8 CTAs of 8 warps per SM)
  int wpr = (p.max_partitions + pa::kReduceBatch - 1) / pa::kReduceBatch;
  wpr = wpr >= 8 ? 8 : wpr >= 4 ? 4 : wpr >= 2 ? 2 : 1;
  const long long rows = (long long)p.num_seqs * p.num_heads;
  const int rows_per_cta = pa::kReduceWarps / wpr;
  long long ctas = (rows + rows_per_cta - 1) / rows_per_cta;
  if (ctas > 8LL * sm_count()) ctas = 8LL * sm_count();
  return launch(pa::pa_decode_reduce_kernel<T>, dim3((unsigned)ctas), dim3(pa::kReduceWarps * 32), 0, stream, p,
                wpr);
}

// The tensor-core block math of a call that splits its sequences into
// partitions of at most 512 tokens runs as two-warp CTAs, six an SM (short
// CTAs: more of them resident hide more of each one's prologue and
// epilogue); every other call as four-warp CTAs, three an SM (see
// pa_decode.cuh).
template <typename T, int G, typename Math>
pa_status_t launch_mma(const CUtensorMap &mk, const CUtensorMap &mv, const pa::DecodeParams &p, cudaStream_t s) {
  if (p.max_partitions > 1 && p.partition_size <= 512) return launch_decode<T, G, Math, 2>(mk, mv, p, s);
  return launch_decode<T, G, Math>(mk, mv, p, s);
}

// fp32 caches and single-head groups run on the CUDA cores; 16-bit caches with
// grouped heads run the tensor-core block math.
template <typename T>
pa_status_t dispatch_group(int group, const CUtensorMap &mk, const CUtensorMap &mv, const pa::DecodeParams &p,
                           cudaStream_t s) {
  constexpr bool kMma = !std::is_same<T, float>::value;
  switch (group) {
    case 1: return launch_decode<T, 1, pa::FmaMath<T, 1>>(mk, mv, p, s);
    case 2:
      if constexpr (kMma) return launch_mma<T, 2, pa::MmaMath<T, 2>>(mk, mv, p, s);
      else return launch_decode<T, 2, pa::FmaMath<T, 2>>(mk, mv, p, s);
    case 4:
      if constexpr (kMma) return launch_mma<T, 4, pa::MmaMath<T, 4>>(mk, mv, p, s);
      else return launch_decode<T, 4, pa::FmaMath<T, 4>>(mk, mv, p, s);
    case 8:
      if constexpr (kMma) return launch_mma<T, 8, pa::MmaMath<T, 8>>(mk, mv, p, s);
      else return launch_decode<T, 8, pa::FmaMath<T, 8>>(mk, mv, p, s);
  }
  return PA_ERR_SHAPE;
}

// E4M3 caches on the tcgen05 path (pa_decode_fp8tc.cuh): the same grid and
// partials as launch_decode, combined by the same reduce.
template <typename T, int G>
pa_status_t launch_fp8tc(const CUtensorMap &mk, const CUtensorMap &mv, const pa::DecodeParams &p0,
                         cudaStream_t stream) {
  using SH = pa::Fp8TcShape<G>;
  auto kernel = pa::pa_decode_fp8tc_kernel<T, G>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SH::kAlloc) != cudaSuccess)
    return PA_ERR_CUDA;
  pa::DecodeParams p = p0;
  p.ws_count = nullptr;   // partials always combined by the reduce kernel
  const long long grid = (long long)p.num_seqs * p.num_kv_heads * p.max_partitions;
  if (grid == 0) return PA_OK;
  if (grid > INT32_MAX) return PA_ERR_SHAPE;
  pa_status_t st = launch(kernel, dim3((unsigned)grid), dim3(pa::kTcThreads), SH::kAlloc, stream, mk, mv, p);
  if (st != PA_OK || p.max_partitions <= 1) return st;
  return launch_reduce<T>(p, stream);
}

// 1-byte E4M3 caches: the mma.sync block math in fp16 with the codes
// converted on the CUDA cores (the default), or, built with PA_FP8_TC=1, the
// tcgen05 kernel whose tensor cores read the codes as they land (parity-green,
// measured 1.45x slower on B200: each 128-token tile waits on a serial chain of
// products, softmax and hand-overs, so too few tiles are in flight an SM)
#ifndef PA_FP8_TC
#define PA_FP8_TC 0
#endif
template <typename T>
pa_status_t dispatch_group_fp8(int group, const CUtensorMap &mk, const CUtensorMap &mv, const pa::DecodeParams &p,
                               cudaStream_t s) {
  if (PA_FP8_TC) {
    switch (group) {
      case 1: return launch_fp8tc<T, 1>(mk, mv, p, s);
      case 2: return launch_fp8tc<T, 2>(mk, mv, p, s);
      case 4: return launch_fp8tc<T, 4>(mk, mv, p, s);
      case 8: return launch_fp8tc<T, 8>(mk, mv, p, s);
    }
    return PA_ERR_SHAPE;
  }
  switch (group) {
    case 1: return launch_decode<T, 1, pa::Fp8MmaMath<T, 1>>(mk, mv, p, s);
    case 2: return launch_decode<T, 2, pa::Fp8MmaMath<T, 2>>(mk, mv, p, s);
    case 4: return launch_decode<T, 4, pa::Fp8MmaMath<T, 4>>(mk, mv, p, s);
    case 8: return launch_decode<T, 8, pa::Fp8MmaMath<T, 8>>(mk, mv, p, s);
  }
  return PA_ERR_SHAPE;
}

}  // namespace

extern "C" {

pa_status_t pa_reshape_and_cache(const void *key, const void *value, void *k_cache, void *v_cache,
                                 const int64_t *slot_mapping, int num_tokens, int64_t num_blocks,
                                 int block_size, int num_kv_heads, int head_dim, pa_dtype_t dtype,
                                 void *stream) {
  pa_status_t st = cache_shape_status(num_blocks, block_size, num_kv_heads, head_dim, dtype);
  if (st != PA_OK) return st;
  if (num_tokens < 0) return PA_ERR_SHAPE;
  if (num_tokens == 0) return PA_OK;
  if (!key || !value || !k_cache || !v_cache || !slot_mapping) return PA_ERR_NULL;
  if (!aligned(key, 16) || !aligned(value, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
      !aligned(slot_mapping, 8))
    return PA_ERR_ALIGN;
  const int chunks_per_slot = num_kv_heads * (row_bytes(dtype) / 16);
  const long long total = (long long)num_tokens * chunks_per_slot;
  long long blocks = (total + 255) / 256;
  if (blocks > 16LL * sm_count()) blocks = 16LL * sm_count();
  return launch(pa::reshape_and_cache_kernel, dim3((unsigned)blocks), dim3(256), 0, (cudaStream_t)stream,
                (const uint4 *)key, (const uint4 *)value, (uint4 *)k_cache, (uint4 *)v_cache, slot_mapping,
                num_tokens, chunks_per_slot, (long long)num_blocks * block_size);
}

int pa_decode_partition_size(int num_seqs, int num_heads, int num_kv_heads, int head_dim, int max_context_len,
                             int requested) {
  if (num_seqs < 0 || num_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0) return -1;
  return resolve_partition_size(num_seqs, num_heads, num_kv_heads, head_dim, max_context_len, requested);
}

size_t pa_decode_workspace_bytes(int num_seqs, int num_heads, int num_kv_heads, int head_dim, int max_context_len,
                                 int requested_partition_size) {
  const int P = pa_decode_partition_size(num_seqs, num_heads, num_kv_heads, head_dim, max_context_len,
                                         requested_partition_size);
  if (P <= 0) return 0;
  return workspace_layout(num_seqs, num_heads, num_kv_heads, head_dim, max_partitions(max_context_len, P)).bytes;
}

}  // extern "C"

namespace {

// A decode call's arguments, checked, with the partition plan derived from them.
struct DecodePlan {
  pa::DecodeParams p;
  CUtensorMap mk, mv;
  const void *k_cache, *v_cache;
  WorkspaceLayout ws;
  int group;
  pa_dtype_t dtype, q_dtype;
  bool empty;   // nothing to launch (no sequences)
};

// Every host-side check of a decode call, in order, except the workspace's:
// dtype: the cache dtype; q_dtype: q and out (equal to dtype except for E4M3 caches).
pa_status_t plan_decode(DecodePlan &d, void *out, const void *q, const void *new_k, const void *new_v,
                        const void *k_cache, const void *v_cache, const int32_t *block_tables, int max_blocks_per_seq,
                        const int32_t *context_lens, int num_seqs, int num_heads, int max_context_len, float scale,
                        int partition_size, int64_t num_blocks, int block_size, int num_kv_heads, int head_dim,
                        pa_dtype_t dtype, pa_dtype_t q_dtype, float k_scale, float v_scale) {
  pa_status_t st = cache_shape_status(num_blocks, block_size, num_kv_heads, head_dim, dtype);
  if (st != PA_OK) return st;
  if (dtype == PA_FP8_E4M3 ? (q_dtype != PA_F16 && q_dtype != PA_BF16) : q_dtype != dtype) return PA_ERR_DTYPE;
  if (!std::isfinite(k_scale) || !std::isfinite(v_scale) || k_scale <= 0.f || v_scale <= 0.f) return PA_ERR_SHAPE;
  if (num_seqs < 0 || num_heads <= 0 || max_context_len < 0 || max_blocks_per_seq < 0 ||
      num_heads % num_kv_heads != 0 || !std::isfinite(scale))
    return PA_ERR_SHAPE;
  const int group = num_heads / num_kv_heads;
  if (group != 1 && group != 2 && group != 4 && group != 8) return PA_ERR_SHAPE;
  if ((long long)max_blocks_per_seq * kBlockSize > INT32_MAX) return PA_ERR_SHAPE;
  const int P = resolve_partition_size(num_seqs, num_heads, num_kv_heads, head_dim, max_context_len,
                                       partition_size);
  if (P <= 0) return PA_ERR_SHAPE;
  d.empty = num_seqs == 0;
  if (d.empty) return PA_OK;
  if (!out || !q || !k_cache || !v_cache || !context_lens || (max_blocks_per_seq > 0 && !block_tables))
    return PA_ERR_NULL;
  if (!aligned(out, 16) || !aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
      !aligned(block_tables, 4) || !aligned(context_lens, 4))
    return PA_ERR_ALIGN;
  const int np = max_partitions(max_context_len, P);
  d.ws = workspace_layout(num_seqs, num_heads, num_kv_heads, head_dim, np);
  d.group = group;
  d.dtype = dtype;
  d.q_dtype = q_dtype;

  pa::DecodeParams &p = d.p;
  p = pa::DecodeParams{};
  p.out = out;
  p.q = q;
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.num_blocks = num_blocks;
  p.num_seqs = num_seqs;
  p.num_heads = num_heads;
  p.num_kv_heads = num_kv_heads;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.max_context_len = max_context_len;
  p.partition_size = P;
  p.max_partitions = np;
  p.scale_log2 = (float)((double)scale * 1.4426950408889634 * (double)k_scale);
  p.v_scale = v_scale;
  p.new_k = new_k;
  p.new_v = new_v;
  p.k_cache = new_k ? const_cast<void *>(k_cache) : nullptr;
  p.v_cache = new_k ? const_cast<void *>(v_cache) : nullptr;
  d.k_cache = k_cache;
  d.v_cache = v_cache;
  return PA_OK;
}

// Launch a planned decode with its split-K workspace (checked by the caller).
pa_status_t launch_planned(DecodePlan &d, void *workspace, void *stream) {
  if (d.empty) return PA_OK;
  pa::DecodeParams &p = d.p;
  const int rb = row_bytes(d.dtype);
  if (!encode_cache_map(&d.mk, d.k_cache, p.num_blocks, p.num_kv_heads, rb) ||
      !encode_cache_map(&d.mv, d.v_cache, p.num_blocks, p.num_kv_heads, rb))
    return PA_ERR_CUDA;
  char *w = static_cast<char *>(workspace);
  p.ws_m = d.ws.bytes ? reinterpret_cast<float *>(w + d.ws.m_off) : nullptr;
  p.ws_l = d.ws.bytes ? reinterpret_cast<float *>(w + d.ws.l_off) : nullptr;
  p.ws_o = d.ws.bytes ? reinterpret_cast<float *>(w + d.ws.o_off) : nullptr;
  p.ws_count = d.ws.bytes && PA_FUSED_COMBINE ? reinterpret_cast<unsigned *>(w + d.ws.c_off) : nullptr;
  p.stall_cta = g_stall_decode.exchange(0);
  cudaStream_t s = (cudaStream_t)stream;
  const int group = d.group;
  if (d.dtype == PA_FP8_E4M3)
    return d.q_dtype == PA_F16 ? dispatch_group_fp8<__half>(group, d.mk, d.mv, p, s)
                               : dispatch_group_fp8<__nv_bfloat16>(group, d.mk, d.mv, p, s);
  switch (d.dtype) {
    case PA_F32: return dispatch_group<float>(group, d.mk, d.mv, p, s);
    case PA_F16: return dispatch_group<__half>(group, d.mk, d.mv, p, s);
    case PA_BF16: return dispatch_group<__nv_bfloat16>(group, d.mk, d.mv, p, s);
    case PA_FP8_E4M3: break;
  }
  return PA_ERR_DTYPE;
}

pa_status_t decode_impl(void *out, const void *q, const void *new_k, const void *new_v, const void *k_cache,
                        const void *v_cache, const int32_t *block_tables, int max_blocks_per_seq,
                        const int32_t *context_lens, int num_seqs, int num_heads, int max_context_len, float scale,
                        int partition_size, void *workspace, size_t workspace_bytes, int64_t num_blocks,
                        int block_size, int num_kv_heads, int head_dim, pa_dtype_t dtype, void *stream,
                        pa_dtype_t q_dtype, float k_scale, float v_scale) {
  DecodePlan d;
  const pa_status_t st = plan_decode(d, out, q, new_k, new_v, k_cache, v_cache, block_tables, max_blocks_per_seq,
                                     context_lens, num_seqs, num_heads, max_context_len, scale, partition_size,
                                     num_blocks, block_size, num_kv_heads, head_dim, dtype, q_dtype, k_scale, v_scale);
  if (st != PA_OK || d.empty) return st;
  if (d.ws.bytes > 0) {
    if (!workspace || workspace_bytes < d.ws.bytes) return PA_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return PA_ERR_ALIGN;
  }
  return launch_planned(d, workspace, stream);
}

}  // namespace

extern "C" {

pa_status_t pa_decode(void *out, const void *q, const void *k_cache, const void *v_cache,
                      const int32_t *block_tables, int max_blocks_per_seq, const int32_t *context_lens,
                      int num_seqs, int num_heads, int max_context_len, float scale, int partition_size,
                      void *workspace, size_t workspace_bytes, int64_t num_blocks, int block_size,
                      int num_kv_heads, int head_dim, pa_dtype_t dtype, void *stream) {
  if (dtype == PA_FP8_E4M3) return PA_ERR_DTYPE;   // pa_decode_fp8
  return decode_impl(out, q, nullptr, nullptr, k_cache, v_cache, block_tables, max_blocks_per_seq, context_lens,
                     num_seqs, num_heads, max_context_len, scale, partition_size, workspace, workspace_bytes,
                     num_blocks, block_size, num_kv_heads, head_dim, dtype, stream, dtype, 1.f, 1.f);
}

pa_status_t pa_decode_fp8(void *out, const void *q, const void *k_cache, const void *v_cache, float k_scale,
                          float v_scale, const int32_t *block_tables, int max_blocks_per_seq,
                          const int32_t *context_lens, int num_seqs, int num_heads, int max_context_len,
                          float scale, int partition_size, void *workspace, size_t workspace_bytes,
                          int64_t num_blocks, int block_size, int num_kv_heads, int head_dim, pa_dtype_t q_dtype,
                          void *stream) {
  return decode_impl(out, q, nullptr, nullptr, k_cache, v_cache, block_tables, max_blocks_per_seq, context_lens,
                     num_seqs, num_heads, max_context_len, scale, partition_size, workspace, workspace_bytes,
                     num_blocks, block_size, num_kv_heads, head_dim, PA_FP8_E4M3, stream, q_dtype, k_scale, v_scale);
}

pa_status_t pa_reshape_and_cache_fp8(const void *key, const void *value, void *k_cache, void *v_cache,
                                     const int64_t *slot_mapping, int num_tokens, int64_t num_blocks,
                                     int block_size, int num_kv_heads, int head_dim, pa_dtype_t src_dtype,
                                     float k_scale, float v_scale, void *stream) {
  pa_status_t st = cache_shape_status(num_blocks, block_size, num_kv_heads, head_dim, PA_FP8_E4M3);
  if (st != PA_OK) return st;
  if (src_dtype != PA_F16 && src_dtype != PA_BF16) return PA_ERR_DTYPE;
  if (!std::isfinite(k_scale) || !std::isfinite(v_scale) || k_scale <= 0.f || v_scale <= 0.f) return PA_ERR_SHAPE;
  if (num_tokens < 0) return PA_ERR_SHAPE;
  if (num_tokens == 0) return PA_OK;
  if (!key || !value || !k_cache || !v_cache || !slot_mapping) return PA_ERR_NULL;
  if (!aligned(key, 16) || !aligned(value, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
      !aligned(slot_mapping, 8))
    return PA_ERR_ALIGN;
  const int chunks_per_slot = num_kv_heads * (head_dim / 8);   // 8 elements per thread
  const long long total = (long long)num_tokens * chunks_per_slot;
  long long blocks = (total + 255) / 256;
  if (blocks > 16LL * sm_count()) blocks = 16LL * sm_count();
  const long long slots = (long long)num_blocks * block_size;
  if (src_dtype == PA_F16)
    return launch(pa::reshape_and_cache_fp8_kernel<__half>, dim3((unsigned)blocks), dim3(256), 0,
                  (cudaStream_t)stream, (const uint4 *)key, (const uint4 *)value, (uint2 *)k_cache,
                  (uint2 *)v_cache, slot_mapping, num_tokens, chunks_per_slot, slots, k_scale, v_scale);
  return launch(pa::reshape_and_cache_fp8_kernel<__nv_bfloat16>, dim3((unsigned)blocks), dim3(256), 0,
                (cudaStream_t)stream, (const uint4 *)key, (const uint4 *)value, (uint2 *)k_cache, (uint2 *)v_cache,
                slot_mapping, num_tokens, chunks_per_slot, slots, k_scale, v_scale);
}

pa_status_t pa_decode_append(void *out, const void *q, const void *key, const void *value, void *k_cache,
                             void *v_cache, const int32_t *block_tables, int max_blocks_per_seq,
                             const int32_t *context_lens, int num_seqs, int num_heads, int max_context_len,
                             float scale, int partition_size, void *workspace, size_t workspace_bytes,
                             int64_t num_blocks, int block_size, int num_kv_heads, int head_dim, pa_dtype_t dtype,
                             void *stream) {
  if (num_seqs > 0 && (!key || !value)) return PA_ERR_NULL;
  if (!aligned(key, 16) || !aligned(value, 16)) return PA_ERR_ALIGN;
  if (dtype == PA_FP8_E4M3) return PA_ERR_DTYPE;
  return decode_impl(out, q, key, value, k_cache, v_cache, block_tables, max_blocks_per_seq, context_lens,
                     num_seqs, num_heads, max_context_len, scale, partition_size, workspace, workspace_bytes,
                     num_blocks, block_size, num_kv_heads, head_dim, dtype, stream, dtype, 1.f, 1.f);
}

pa_status_t pa_prefill(void *out, const void *q, const void *k_cache, const void *v_cache,
                       const int32_t *block_tables, int max_blocks_per_seq, const int32_t *context_lens,
                       const int32_t *query_start_loc, int num_seqs, int num_heads, int max_query_len,
                       float scale, int64_t num_blocks, int block_size, int num_kv_heads, int head_dim,
                       pa_dtype_t dtype, void *stream) {
  pa_status_t st = cache_shape_status(num_blocks, block_size, num_kv_heads, head_dim, dtype);
  if (st != PA_OK) return st;
  if (dtype != PA_F16 && dtype != PA_BF16) return PA_ERR_DTYPE;
  if (head_dim != 128 || num_seqs < 0 || num_seqs > 65535 || num_heads <= 0 || num_kv_heads > 65535 ||
      num_heads % num_kv_heads != 0 || max_query_len < 0 || max_blocks_per_seq < 0 || !std::isfinite(scale) ||
      !(scale > 0.f))
    return PA_ERR_SHAPE;
  const int group = num_heads / num_kv_heads;
  if (group != 1 && group != 2 && group != 4 && group != 8) return PA_ERR_SHAPE;
  if ((long long)max_blocks_per_seq * kBlockSize > INT32_MAX) return PA_ERR_SHAPE;
  if (num_seqs == 0 || max_query_len == 0) return PA_OK;
  if (!out || !q || !k_cache || !v_cache || !context_lens || !query_start_loc || (max_blocks_per_seq > 0 && !block_tables))
    return PA_ERR_NULL;
  if (!aligned(out, 16) || !aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
      !aligned(block_tables, 4) || !aligned(context_lens, 4) || !aligned(query_start_loc, 4))
    return PA_ERR_ALIGN;
  CUtensorMap mk, mv;
  if (!encode_cache_map(&mk, k_cache, num_blocks, num_kv_heads, kRowBytes) ||
      !encode_cache_map(&mv, v_cache, num_blocks, num_kv_heads, kRowBytes))
    return PA_ERR_CUDA;
  pa::PrefillParams p{};
  p.out = out;
  p.q = q;
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.query_start_loc = query_start_loc;
  p.num_blocks = num_blocks;
  p.num_seqs = num_seqs;
  p.num_heads = num_heads;
  p.num_kv_heads = num_kv_heads;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.max_query_len = max_query_len;
  p.scale_log2 = (float)((double)scale * 1.4426950408889634);
  p.stall_cta = g_stall_prefill.exchange(0);
  const int qt = pa::kPrefillTiles * pa::kPrefillRows / group;   // chunk queries per CTA
  const dim3 grid((unsigned)((max_query_len + qt - 1) / qt), (unsigned)num_kv_heads, (unsigned)num_seqs);
  auto go = [&](auto kernel) -> pa_status_t {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, pa::PrefillSmem::kAlloc) !=
        cudaSuccess)
      return PA_ERR_CUDA;
    return launch(kernel, grid, dim3(pa::kPrefillThreads), pa::PrefillSmem::kAlloc, (cudaStream_t)stream, mk, mv, p);
  };
  if (dtype == PA_BF16) {
    switch (group) {
      case 1: return go(pa::pa_prefill_kernel<__nv_bfloat16, 1>);
      case 2: return go(pa::pa_prefill_kernel<__nv_bfloat16, 2>);
      case 4: return go(pa::pa_prefill_kernel<__nv_bfloat16, 4>);
      case 8: return go(pa::pa_prefill_kernel<__nv_bfloat16, 8>);
    }
  } else {
    switch (group) {
      case 1: return go(pa::pa_prefill_kernel<__half, 1>);
      case 2: return go(pa::pa_prefill_kernel<__half, 2>);
      case 4: return go(pa::pa_prefill_kernel<__half, 4>);
      case 8: return go(pa::pa_prefill_kernel<__half, 8>);
    }
  }
  return PA_ERR_SHAPE;
}

pa_status_t pa_copy_blocks(void *k_cache, void *v_cache, const int64_t *block_mapping, int num_pairs,
                           int64_t num_blocks, int block_size, int num_kv_heads, int head_dim, pa_dtype_t dtype,
                           void *stream) {
  pa_status_t st = cache_shape_status(num_blocks, block_size, num_kv_heads, head_dim, dtype);
  if (st != PA_OK) return st;
  if (num_pairs < 0 || num_pairs > PA_MAX_COPY_PAIRS) return PA_ERR_SHAPE;
  if (num_pairs == 0) return PA_OK;
  if (!k_cache || !v_cache || !block_mapping) return PA_ERR_NULL;
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16) || !aligned(block_mapping, 8)) return PA_ERR_ALIGN;
  const int chunks_per_block = kBlockSize * num_kv_heads * (row_bytes(dtype) / 16);
  // one CTA per pair up to two per SM, then each CTA takes several pairs (at
  // most kCopyMaxPairsPerCta); blockIdx.y: 0 = K cache, 1 = V cache
  long long ctas = num_pairs < 2LL * sm_count() ? num_pairs : 2LL * sm_count();
  const long long min_ctas = (num_pairs + pa::kCopyMaxPairsPerCta - 1) / pa::kCopyMaxPairsPerCta;
  if (ctas < min_ctas) ctas = min_ctas;
  return launch(pa::copy_blocks_kernel, dim3((unsigned)ctas, 2), dim3(pa::kCopyThreads), 0, (cudaStream_t)stream,
                (uint4 *)k_cache, (uint4 *)v_cache, (const longlong2 *)block_mapping, num_pairs,
                (long long)num_blocks, chunks_per_block);
}

// ---------------------------------------------------------------- no-allocation decode
// Split-K scratch owned by the library, for callers that cannot allocate device
// memory themselves.  It lives in every device that loads this library, for
// the life of the process.  Host code must not use the array's name as a device
// address: the address is looked up per device with cudaGetSymbolAddress.
static __device__ __align__(256) unsigned char g_decode_scratch[PA_STATIC_WORKSPACE_BYTES];

namespace {
// Address of the current device's copy of g_decode_scratch, looked up on every
// call (cheap, allocates nothing), so that it is never stale -- e.g. after a
// cudaDeviceReset, which gives the device a new context and a new copy.  The
// first lookup on a device may load the library's device code there.
void *scratch_for_current_device() {
  void *ptr = nullptr;
  if (cudaGetSymbolAddress(&ptr, g_decode_scratch) != cudaSuccess) return nullptr;
  return ptr;
}
}  // namespace

pa_status_t pa_decode_static_workspace(void *out, const void *q, const void *k_cache, const void *v_cache,
                                       const int32_t *block_tables, int max_blocks_per_seq,
                                       const int32_t *context_lens, int num_seqs, int num_heads,
                                       int max_context_len, float scale, int partition_size, int64_t num_blocks,
                                       int block_size, int num_kv_heads, int head_dim, pa_dtype_t dtype,
                                       void *stream) {
  if (dtype == PA_FP8_E4M3) return PA_ERR_DTYPE;   // as pa_decode
  // every check of pa_decode first, in its order; then the size of the scratch
  DecodePlan d;
  const pa_status_t st = plan_decode(d, out, q, nullptr, nullptr, k_cache, v_cache, block_tables, max_blocks_per_seq,
                                     context_lens, num_seqs, num_heads, max_context_len, scale, partition_size,
                                     num_blocks, block_size, num_kv_heads, head_dim, dtype, dtype, 1.f, 1.f);
  if (st != PA_OK || d.empty) return st;
  void *scratch = nullptr;
  if (d.ws.bytes > 0) {
    if (d.ws.bytes > PA_STATIC_WORKSPACE_BYTES) return PA_ERR_WORKSPACE;
    scratch = scratch_for_current_device();
    if (!scratch) return PA_ERR_CUDA;
  }
  return launch_planned(d, scratch, stream);
}

// ---------------------------------------------------------------- rotate and append
pa_status_t pa_rope_table(float *cos_sin, int max_position, int rotary_dim, double base, void *stream) {
  if (max_position <= 0 || rotary_dim <= 0 || rotary_dim % 2 != 0 || !std::isfinite(base) || base <= 0.0)
    return PA_ERR_SHAPE;
  if (!cos_sin) return PA_ERR_NULL;
  if (!aligned(cos_sin, 16)) return PA_ERR_ALIGN;
  const long long total = (long long)max_position * (rotary_dim / 2);
  long long ctas = (total + 255) / 256;
  if (ctas > 32LL * sm_count()) ctas = 32LL * sm_count();
  return launch(pa::rope_table_kernel, dim3((unsigned)ctas), dim3(256), 0, (cudaStream_t)stream, cos_sin, max_position,
                rotary_dim / 2, base);
}

}  // extern "C"

namespace {

// Do two byte ranges overlap?
bool ranges_overlap(const void *a, size_t a_bytes, const void *b, size_t b_bytes) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return x < y + b_bytes && y < x + a_bytes;
}

// Do n rows of a_row bytes, a_stride apart, and n of b_row bytes overlap?  Rows as far
// apart as each other (columns of the same wider rows) are compared as such, others by
// the ranges they span.
bool rows_overlap(const void *a, size_t a_stride, size_t a_row, const void *b, size_t b_stride, size_t b_row, int n) {
  if (!ranges_overlap(a, (n - 1) * a_stride + a_row, b, (n - 1) * b_stride + b_row)) return false;
  if (a_stride != b_stride) return true;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  const size_t after = y >= x ? (y - x) % a_stride : (a_stride - (x - y) % a_stride) % a_stride;
  return after < a_row || after + b_row > a_stride;   // b's columns start within a's, or run into the next row's
}

// Heads a thread: three where that leaves a wave of CTAs (256 threads, up to eight an
// SM), one below that, where the number of CTAs counts more.
template <typename T>
pa_status_t launch_rope(const pa::RopeParams &p, bool interleaved, bool fp8, cudaStream_t stream) {
  const int rows = p.num_heads + 2 * p.num_kv_heads;
  const unsigned tokens = (unsigned)((p.num_tokens + pa::kRopeTokens - 1) / pa::kRopeTokens);
  const bool many = (long long)tokens * ((rows + 23) / 24) >= 8LL * sm_count();
  const int per_cta = pa::kRopeHeads * (many ? 3 : 1);
  const dim3 grid(tokens, (unsigned)((rows + per_cta - 1) / per_cta));
  auto go = [&](auto kernel) { return launch(kernel, grid, dim3(256), 0, stream, p); };
  auto pick = [&](auto inter, auto quant) {
    constexpr bool I = decltype(inter)::value, Q = decltype(quant)::value;
    return many ? go(pa::rope_and_cache_kernel<T, I, Q, 3>) : go(pa::rope_and_cache_kernel<T, I, Q, 1>);
  };
  if constexpr (!std::is_same<T, float>::value) {
    if (fp8) return interleaved ? pick(std::true_type{}, std::true_type{}) : pick(std::false_type{}, std::true_type{});
  }
  return interleaved ? pick(std::true_type{}, std::false_type{}) : pick(std::false_type{}, std::false_type{});
}

// cache_dtype: dtype, or PA_FP8_E4M3.
pa_status_t rope_impl(void *q_out, const void *q, const void *key, const void *value, void *k_cache, void *v_cache,
                      const int64_t *positions, const float *cos_sin, const int64_t *slot_mapping, int num_tokens,
                      int64_t q_out_stride, int64_t q_stride, int64_t k_stride, int64_t v_stride, int max_position,
                      int rotary_dim, int interleaved, int64_t num_blocks, int block_size, int num_heads,
                      int num_kv_heads, int head_dim, pa_dtype_t dtype, pa_dtype_t cache_dtype, float k_scale,
                      float v_scale, void *stream) {
  pa_status_t st = cache_shape_status(num_blocks, block_size, num_kv_heads, head_dim, cache_dtype);
  if (st != PA_OK) return st;
  const int es = elem_bytes(dtype), epc = 16 / es;
  if (num_tokens < 0 || num_heads <= 0 || num_heads > 65536 || num_kv_heads > 65536 || max_position <= 0 ||
      rotary_dim <= 0 || rotary_dim > head_dim || rotary_dim % (2 * epc) != 0)
    return PA_ERR_SHAPE;
  if (!std::isfinite(k_scale) || !std::isfinite(v_scale) || k_scale <= 0.f || v_scale <= 0.f) return PA_ERR_SHAPE;
  const int64_t q_row = (int64_t)num_heads * head_dim, kv_row = (int64_t)num_kv_heads * head_dim;
  if (q_stride < q_row || q_out_stride < q_row || k_stride < kv_row || v_stride < kv_row || q_stride > INT32_MAX ||
      q_out_stride > INT32_MAX || k_stride > INT32_MAX || v_stride > INT32_MAX)
    return PA_ERR_SHAPE;
  if (num_tokens == 0) return PA_OK;
  if (!q_out || !q || !key || !value || !k_cache || !v_cache || !positions || !cos_sin || !slot_mapping)
    return PA_ERR_NULL;
  if (!aligned(q_out, 16) || !aligned(q, 16) || !aligned(key, 16) || !aligned(value, 16) || !aligned(k_cache, 16) ||
      !aligned(v_cache, 16) || !aligned(cos_sin, 16) || !aligned(positions, 8) || !aligned(slot_mapping, 8) ||
      q_stride % epc != 0 || q_out_stride % epc != 0 || k_stride % epc != 0 || v_stride % epc != 0)
    return PA_ERR_ALIGN;
  auto meets = [&](const void *x, int64_t x_stride, int64_t x_row) {
    return rows_overlap(q_out, q_out_stride * es, q_row * es, x, x_stride * es, x_row * es, num_tokens);
  };
  if (!(q_out == q && q_out_stride == q_stride) &&
      (meets(q, q_stride, q_row) || meets(key, k_stride, kv_row) || meets(value, v_stride, kv_row)))
    return PA_ERR_SHAPE;
  pa::RopeParams p{};
  p.q_out = q_out;
  p.q = q;
  p.key = key;
  p.value = value;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.positions = positions;
  p.cos_sin = cos_sin;
  p.slot_mapping = slot_mapping;
  p.q_out_stride = q_out_stride;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.num_slots = num_blocks * block_size;
  p.max_position = max_position;
  p.num_tokens = num_tokens;
  p.num_heads = num_heads;
  p.num_kv_heads = num_kv_heads;
  p.rotary = rotary_dim;
  auto split = [](float scale) {
    const float unit = scale < 0x1p-60f ? 0x1p96f : scale > 0x1p60f ? 0x1p-64f : 1.f;
    const float s = scale * unit;   // exact
    return pa::E4m3Scale{s, 1.f / s, unit};
  };
  p.k_scale = split(k_scale);
  p.v_scale = split(v_scale);
  const bool fp8 = cache_dtype == PA_FP8_E4M3;
  cudaStream_t s = (cudaStream_t)stream;
  switch (dtype) {
    case PA_F32: return launch_rope<float>(p, interleaved != 0, fp8, s);
    case PA_F16: return launch_rope<__half>(p, interleaved != 0, fp8, s);
    case PA_BF16: return launch_rope<__nv_bfloat16>(p, interleaved != 0, fp8, s);
    case PA_FP8_E4M3: break;
  }
  return PA_ERR_DTYPE;
}

}  // namespace

extern "C" {

pa_status_t pa_rope_and_cache(void *q_out, const void *q, const void *key, const void *value, void *k_cache,
                              void *v_cache, const int64_t *positions, const float *cos_sin,
                              const int64_t *slot_mapping, int num_tokens, int64_t q_out_stride, int64_t q_stride,
                              int64_t k_stride, int64_t v_stride, int max_position, int rotary_dim, int interleaved,
                              int64_t num_blocks, int block_size, int num_heads, int num_kv_heads, int head_dim,
                              pa_dtype_t dtype, void *stream) {
  if (dtype == PA_FP8_E4M3) return PA_ERR_DTYPE;   // pa_rope_and_cache_fp8
  return rope_impl(q_out, q, key, value, k_cache, v_cache, positions, cos_sin, slot_mapping, num_tokens, q_out_stride,
                   q_stride, k_stride, v_stride, max_position, rotary_dim, interleaved, num_blocks, block_size,
                   num_heads, num_kv_heads, head_dim, dtype, dtype, 1.f, 1.f, stream);
}

pa_status_t pa_rope_and_cache_fp8(void *q_out, const void *q, const void *key, const void *value, void *k_cache,
                                  void *v_cache, const int64_t *positions, const float *cos_sin,
                                  const int64_t *slot_mapping, int num_tokens, int64_t q_out_stride, int64_t q_stride,
                                  int64_t k_stride, int64_t v_stride, int max_position, int rotary_dim,
                                  int interleaved, int64_t num_blocks, int block_size, int num_heads,
                                  int num_kv_heads, int head_dim, pa_dtype_t src_dtype, float k_scale, float v_scale,
                                  void *stream) {
  if (src_dtype != PA_F16 && src_dtype != PA_BF16) return PA_ERR_DTYPE;
  return rope_impl(q_out, q, key, value, k_cache, v_cache, positions, cos_sin, slot_mapping, num_tokens, q_out_stride,
                   q_stride, k_stride, v_stride, max_position, rotary_dim, interleaved, num_blocks, block_size,
                   num_heads, num_kv_heads, head_dim, src_dtype, PA_FP8_E4M3, k_scale, v_scale, stream);
}

}  // extern "C"

// ---------------------------------------------------------------- shared prefix
namespace {

// How pa_decode_shared_prefix cuts its work: partitions of the prefix (by the work that the
// device finds, pa::prefix_part_tiles), and the suffix's split-K; the workspace has `slots`
// partials a row, the suffix's from slot0 on.
struct PrefixPlan {
  int levels, most_row_ctas, part_tiles[pa::kPrefixLevels];
  double ctas;   // of the prefix kernel
  int suffix_partition, suffix_parts, slot0, slots;
  WorkspaceLayout ws;
};

// Tiles of a partition, for `ctas` (256 rows, KV head) pairs over `tiles` tiles: as many
// partitions as give the shortest run by this model, in us measured on B200.  A
// CTA (one an SM) takes 8.5 of set-up and epilogue and 2.9 a step; a step is a
// tile, or two where a CTA has at most 128 rows.  A last wave that is not full counts for
// at least half.  Each partition's partials cost 0.35 to combine and their
// bytes, written and read.  (47 sequences in three groups, 32 KV heads: 44.3 a call with
// the two partitions chosen, 55.6 with one, 53.9 with three; 128 sequences over 1024 tokens:
// 38.0 with four, 39.2 with three, 39.5 with eight; 5 over 4000: 15.8 with eight, 16.5 with
// sixteen, 24.6 with three.)
int plan_part_tiles(double ctas, int tiles, bool split, double partial_us) {
  const double sms = sm_count();
  double best = 1e300;
  int per = tiles, last = 0;
  for (int parts = 1; parts <= tiles && parts <= 64; ++parts) {
    const int t = (tiles + parts - 1) / parts;
    if (t == last) continue;
    last = t;
    const int steps = split ? (t + 1) / 2 : t;
    const double waves = ctas * parts / sms, full = std::floor(waves), rest = waves - full;
    const double runs = waves <= 1 ? 1 : full + (rest > 0 ? (rest > 0.5 ? rest : 0.5) : 0);
    const double cost = runs * (8.5 + 2.9 * steps) + parts * partial_us;
    if (cost < best) {
      best = cost;
      per = t;
    }
  }
  return per;
}

PrefixPlan plan_prefix(int num_seqs, int num_groups, int num_heads, int num_kv_heads, int head_dim, int max_prefix_len,
                       int max_suffix_len, int max_group_size) {
  PrefixPlan r{};
  const int group = num_heads / num_kv_heads;
  const int rows = max_group_size * group, cta_rows = 2 * pa::kPrefixRows;
  const int tiles = (max_prefix_len + pa::kPrefixKv - 1) / pa::kPrefixKv;
  int most_parts = 0;
  if (tiles > 0) {
    // 256 rows at a time: no group has more than the largest, and all of them no more than the batch and a rest each
    const double most = std::min((double)num_groups * ((rows + cta_rows - 1) / cta_rows),
                                 num_groups + std::floor((double)num_seqs * group / cta_rows));
    r.most_row_ctas = (int)std::min(most, (double)INT32_MAX);
    const double partial_us = 0.35 + (double)num_seqs * num_heads * 2 * head_dim * sizeof(float) / 6.5e6;
    // With one group its rows are the work; with more, the device says which of the levels it is
    // (in 32 bits, so beyond them it is taken to be all that the bounds allow).
    const int levels = num_groups == 1 || most * tiles >= 2147483648.0 ? 1 : pa::kPrefixLevels;
    for (int i = 0; i < levels; ++i) {
      const double live = (double)((r.most_row_ctas + (1ll << i) - 1) >> i);
      const int per = plan_part_tiles(live * num_kv_heads, tiles, rows <= pa::kPrefixRows, partial_us);
      const int parts = (tiles + per - 1) / per;
      r.part_tiles[i] = per;
      r.levels = i + 1;
      most_parts = std::max(most_parts, parts);
      // Each 256 rows' first partition may be as short as a tile; every further one takes a whole one before it.
      const double first = std::min(most, live * tiles);
      r.ctas = std::max(r.ctas, std::min(first + std::floor((live * tiles - first) / per), most * parts) * num_kv_heads);
      if (live <= 1) break;
    }
  }
  r.suffix_partition = resolve_partition_size(num_seqs, num_heads, num_kv_heads, head_dim, max_suffix_len, 0);
  r.suffix_parts = max_partitions(max_suffix_len, r.suffix_partition);
  r.slot0 = 2 * most_parts;
  r.slots = r.slot0 + r.suffix_parts;
  const size_t n = (size_t)num_seqs * num_heads * r.slots;
  r.ws.l_off = align256(n * sizeof(float));
  r.ws.o_off = 2 * r.ws.l_off;
  r.ws.bytes = r.ws.o_off + align256(n * head_dim * sizeof(float));
  return r;
}

pa_status_t prefix_shape_status(int num_seqs, int num_groups, int num_heads, int num_kv_heads, int max_prefix_len,
                                int max_suffix_len, int max_group_size) {
  if (num_seqs < 0 || num_groups < 0 || num_heads <= 0 || num_kv_heads <= 0 || num_heads % num_kv_heads != 0 ||
      max_prefix_len < 0 || max_prefix_len % kBlockSize != 0 || max_suffix_len < 0 || max_group_size < 0 ||
      max_prefix_len > (1 << 30) || max_suffix_len > (1 << 30) || max_group_size > (1 << 24) || num_groups > (1 << 24))
    return PA_ERR_SHAPE;
  const int group = num_heads / num_kv_heads;
  if (group != 1 && group != 2 && group != 4 && group != 8) return PA_ERR_SHAPE;
  if (num_seqs > 0 && (num_groups == 0 || max_group_size == 0)) return PA_ERR_SHAPE;
  return PA_OK;
}

template <typename T, int G, typename Math>
pa_status_t launch_prefix(const CUtensorMap &mk, const CUtensorMap &mv, const pa::SuffixParams &p, unsigned prefix_ctas,
                          cudaStream_t stream) {
  pa_status_t st;
  if (prefix_ctas > 0) {
    auto kernel = pa::pa_shared_prefix_kernel<T, G>;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, pa::PrefixSmem::kAlloc) != cudaSuccess)
      return PA_ERR_CUDA;
    st = launch(kernel, dim3(prefix_ctas), dim3(pa::kPrefixThreads), pa::PrefixSmem::kAlloc, stream, mk, mv, p);
    if (st != PA_OK) return st;
  }
  using SM = pa::DecodeSmem<T, G, Math>;
  auto suffix = pa::pa_decode_partition_kernel<T, G, Math, pa::kDecodeWarps, pa::kWalkSuffix>;
  if (cudaFuncSetAttribute(suffix, cudaFuncAttributeMaxDynamicSharedMemorySize, SM::kAlloc) != cudaSuccess)
    return PA_ERR_CUDA;
  const unsigned grid = (unsigned)(p.num_seqs * p.num_kv_heads * p.max_partitions);
  pa::SuffixParams sp = p;
  sp.stall_cta = 0;
  st = launch(suffix, dim3(grid), dim3(pa::kDecodeThreads), SM::kAlloc, stream, mk, mv, sp);
  if (st != PA_OK || p.max_partitions == 1) return st;
  const long long rows = (long long)p.num_seqs * p.num_heads;
  long long ctas = (rows + pa::kReduceWarps - 1) / pa::kReduceWarps;
  if (ctas > 8LL * sm_count()) ctas = 8LL * sm_count();
  return launch(pa::pa_join_shared_kernel<T, G>, dim3((unsigned)ctas), dim3(pa::kReduceWarps * 32), 0, stream, p);
}

template <typename T>
pa_status_t dispatch_prefix(int group, const CUtensorMap &mk, const CUtensorMap &mv, const pa::SuffixParams &p,
                            unsigned prefix_ctas, cudaStream_t s) {
  switch (group) {
    case 1: return launch_prefix<T, 1, pa::FmaMath<T, 1>>(mk, mv, p, prefix_ctas, s);
    case 2: return launch_prefix<T, 2, pa::MmaMath<T, 2>>(mk, mv, p, prefix_ctas, s);
    case 4: return launch_prefix<T, 4, pa::MmaMath<T, 4>>(mk, mv, p, prefix_ctas, s);
    case 8: return launch_prefix<T, 8, pa::MmaMath<T, 8>>(mk, mv, p, prefix_ctas, s);
  }
  return PA_ERR_SHAPE;
}

}  // namespace

extern "C" {

size_t pa_decode_shared_prefix_workspace_bytes(int num_seqs, int num_groups, int num_heads, int num_kv_heads,
                                               int head_dim, int max_prefix_len, int max_suffix_len,
                                               int max_group_size) {
  if (prefix_shape_status(num_seqs, num_groups, num_heads, num_kv_heads, max_prefix_len, max_suffix_len,
                          max_group_size) != PA_OK ||
      head_dim != 128 || num_seqs == 0)
    return 0;
  return plan_prefix(num_seqs, num_groups, num_heads, num_kv_heads, head_dim, max_prefix_len, max_suffix_len,
                     max_group_size).ws.bytes;
}

pa_status_t pa_decode_shared_prefix(void *out, const void *q, const void *k_cache, const void *v_cache,
                                    const int32_t *block_tables, int max_blocks_per_seq, const int32_t *context_lens,
                                    const int32_t *group_start, const int32_t *prefix_lens, int num_seqs,
                                    int num_groups, int num_heads, int max_prefix_len, int max_suffix_len,
                                    int max_group_size, float scale, void *workspace, size_t workspace_bytes,
                                    int64_t num_blocks, int block_size, int num_kv_heads, int head_dim,
                                    pa_dtype_t dtype, void *stream) {
  pa_status_t st = cache_shape_status(num_blocks, block_size, num_kv_heads, head_dim, dtype);
  if (st != PA_OK) return st;
  if (dtype != PA_F16 && dtype != PA_BF16) return PA_ERR_DTYPE;
  st = prefix_shape_status(num_seqs, num_groups, num_heads, num_kv_heads, max_prefix_len, max_suffix_len, max_group_size);
  if (st != PA_OK) return st;
  if (max_blocks_per_seq < 0 || (long long)max_blocks_per_seq * kBlockSize > INT32_MAX || !std::isfinite(scale) ||
      !(scale > 0.f))
    return PA_ERR_SHAPE;
  if (num_seqs == 0) return PA_OK;
  if (!out || !q || !k_cache || !v_cache || !context_lens || !group_start || !prefix_lens ||
      (max_blocks_per_seq > 0 && !block_tables))
    return PA_ERR_NULL;
  if (!aligned(out, 16) || !aligned(q, 16) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
      !aligned(block_tables, 4) || !aligned(context_lens, 4) || !aligned(group_start, 4) || !aligned(prefix_lens, 4))
    return PA_ERR_ALIGN;
  const PrefixPlan plan = plan_prefix(num_seqs, num_groups, num_heads, num_kv_heads, head_dim, max_prefix_len,
                                      max_suffix_len, max_group_size);
  // CTAs of the two launches (in floating point: a product of counts may pass 2^63)
  if (plan.ctas > INT32_MAX ||
      (double)num_seqs * num_kv_heads * plan.suffix_parts > INT32_MAX)
    return PA_ERR_SHAPE;
  if (!workspace || workspace_bytes < plan.ws.bytes) return PA_ERR_WORKSPACE;
  if (!aligned(workspace, 256)) return PA_ERR_ALIGN;
  CUtensorMap mk, mv;
  if (!encode_cache_map(&mk, k_cache, num_blocks, num_kv_heads, kRowBytes) ||
      !encode_cache_map(&mv, v_cache, num_blocks, num_kv_heads, kRowBytes))
    return PA_ERR_CUDA;
  char *w = static_cast<char *>(workspace);
  pa::SuffixParams p{};
  p.out = out;
  p.q = q;
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.ws_m = reinterpret_cast<float *>(w);
  p.ws_l = reinterpret_cast<float *>(w + plan.ws.l_off);
  p.ws_o = reinterpret_cast<float *>(w + plan.ws.o_off);
  p.num_blocks = num_blocks;
  p.num_seqs = num_seqs;
  p.num_heads = num_heads;
  p.num_kv_heads = num_kv_heads;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.max_context_len = max_suffix_len;
  p.partition_size = plan.suffix_partition;
  p.max_partitions = plan.suffix_parts;
  p.scale_log2 = (float)((double)scale * 1.4426950408889634);
  p.v_scale = 1.f;
  p.stall_cta = g_stall_prefix.exchange(0);
  p.group_start = group_start;
  p.prefix_lens = prefix_lens;
  p.num_groups = num_groups;
  p.max_prefix_len = max_prefix_len;
  p.max_group_size = max_group_size;
  p.slots = plan.slots;
  p.slot0 = plan.slot0;
  p.levels = plan.levels;
  p.most_row_ctas = plan.most_row_ctas;
  std::copy(plan.part_tiles, plan.part_tiles + pa::kPrefixLevels, p.part_tiles);
  const unsigned prefix_ctas = (unsigned)plan.ctas;
  const int group = num_heads / num_kv_heads;
  cudaStream_t s = (cudaStream_t)stream;
  return dtype == PA_F16 ? dispatch_prefix<__half>(group, mk, mv, p, prefix_ctas, s)
                         : dispatch_prefix<__nv_bfloat16>(group, mk, mv, p, prefix_ctas, s);
}

// ---------------------------------------------------------------- block-sparse decode
pa_status_t pa_update_block_bounds(const void *k_cache, void *block_bounds, const int32_t *block_tables,
                                   int max_blocks_per_seq, const int32_t *context_lens, const int32_t *new_lens,
                                   int num_seqs, int max_new_len, int64_t num_blocks, int block_size,
                                   int num_kv_heads, int head_dim, pa_dtype_t dtype, void *stream) {
  if (dtype == PA_FP8_E4M3) return PA_ERR_DTYPE;
  pa_status_t st = cache_shape_status(num_blocks, block_size, num_kv_heads, head_dim, dtype);
  if (st != PA_OK) return st;
  if (num_seqs < 0 || max_new_len < 0 || max_blocks_per_seq < 0 || num_kv_heads > 65536 ||
      (long long)max_blocks_per_seq * kBlockSize > INT32_MAX)
    return PA_ERR_SHAPE;
  if (num_seqs == 0 || max_new_len == 0) return PA_OK;
  if (!k_cache || !block_bounds || !context_lens || !new_lens || (max_blocks_per_seq > 0 && !block_tables))
    return PA_ERR_NULL;
  if (!aligned(k_cache, 16) || !aligned(block_bounds, 16) || !aligned(block_tables, 4) || !aligned(context_lens, 4) ||
      !aligned(new_lens, 4))
    return PA_ERR_ALIGN;
  pa::BoundsParams p{};
  p.k_cache = (const uint4 *)k_cache;
  p.bounds = (uint4 *)block_bounds;
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.new_lens = new_lens;
  p.num_blocks = num_blocks;
  p.num_seqs = num_seqs;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.chunks_per_token = num_kv_heads * pa::kChunksPerRow;
  p.max_new_len = max_new_len;
  // the new tokens may start anywhere in a block: n tokens touch at most ceil((n + 15) / 16) blocks
  p.blocks_per_seq = (int)(((long long)max_new_len + 2 * kBlockSize - 2) / kBlockSize);
  if (p.blocks_per_seq > max_blocks_per_seq) p.blocks_per_seq = max_blocks_per_seq > 0 ? max_blocks_per_seq : 1;
  const long long total = (long long)num_seqs * p.blocks_per_seq * p.chunks_per_token;
  long long ctas = (total + 255) / 256;
  if (ctas > 64LL * sm_count()) ctas = 64LL * sm_count();
  cudaStream_t s = (cudaStream_t)stream;
  switch (dtype) {
    case PA_F32: return launch(pa::block_bounds_kernel<float>, dim3((unsigned)ctas), dim3(256), 0, s, p);
    case PA_F16: return launch(pa::block_bounds_kernel<__half>, dim3((unsigned)ctas), dim3(256), 0, s, p);
    case PA_BF16: return launch(pa::block_bounds_kernel<__nv_bfloat16>, dim3((unsigned)ctas), dim3(256), 0, s, p);
    case PA_FP8_E4M3: break;
  }
  return PA_ERR_DTYPE;
}

}  // extern "C"

namespace {

constexpr int kMaxSelected = 1 << 26;   // blocks of a list: its tokens are counted in 32 bits

template <typename T, int G>
pa_status_t launch_choice(const pa::SelectParams &p, cudaStream_t s) {
  if (p.max_blocks > p.num_selected) {   // else no sequence has more blocks than are chosen
    const long long grid = (long long)p.num_seqs * p.num_kv_heads * p.chunks;
    if (grid > INT32_MAX) return PA_ERR_SHAPE;
    const pa_status_t st =
        launch(pa::block_score_kernel<T, G>, dim3((unsigned)grid), dim3(pa::kScoreWarps * 32), 0, s, p);
    if (st != PA_OK) return st;
  }
  const unsigned lists = (unsigned)(p.num_seqs * p.num_kv_heads);
  // Short lists, and more than two an SM, with half the threads: 8 lists of 256 blocks 8.5 us a call
  // against 9.0, 512 of 1024 blocks 66.0 against 70.3; but 8 lists of 2048 13.4 against 10.3.
  if (p.max_blocks <= 512 || lists > 2u * (unsigned)sm_count())
    return launch(pa::block_select_kernel<T, G, 256>, dim3(lists), dim3(256), 0, s, p);
  return launch(pa::block_select_kernel<T, G, 512>, dim3(lists), dim3(512), 0, s, p);
}

template <typename T>
pa_status_t dispatch_choice(int group, const pa::SelectParams &p, cudaStream_t s) {
  switch (group) {
    case 1: return launch_choice<T, 1>(p, s);
    case 2: return launch_choice<T, 2>(p, s);
    case 4: return launch_choice<T, 4>(p, s);
    case 8: return launch_choice<T, 8>(p, s);
  }
  return PA_ERR_SHAPE;
}

}  // namespace

extern "C" {

size_t pa_select_blocks_workspace_bytes(int num_seqs, int num_kv_heads, int max_context_len) {
  if (num_seqs <= 0 || num_kv_heads <= 0 || max_context_len <= 0) return 0;
  const size_t blocks = ((size_t)max_context_len + kBlockSize - 1) / kBlockSize;
  return 2 * align256((size_t)num_seqs * num_kv_heads * blocks * 8);   // fp32 scores with bounds, fp64 scores
}

pa_status_t pa_select_blocks(int32_t *selected, const void *q, const void *block_bounds, const int32_t *block_tables,
                             int max_blocks_per_seq, const int32_t *context_lens, int num_seqs, int num_heads,
                             int max_context_len, int num_selected, int sink_blocks, int recent_blocks,
                             void *workspace, size_t workspace_bytes, int64_t num_blocks, int block_size,
                             int num_kv_heads, int head_dim, pa_dtype_t dtype, void *stream) {
  if (dtype == PA_FP8_E4M3) return PA_ERR_DTYPE;
  pa_status_t st = cache_shape_status(num_blocks, block_size, num_kv_heads, head_dim, dtype);
  if (st != PA_OK) return st;
  if (num_seqs < 0 || num_heads <= 0 || num_heads % num_kv_heads != 0 || max_context_len < 0 ||
      max_blocks_per_seq < 0 || (long long)max_blocks_per_seq * kBlockSize > INT32_MAX || num_selected <= 0 ||
      sink_blocks < 0 || recent_blocks < 0 || (long long)sink_blocks + recent_blocks > num_selected ||
      num_selected > kMaxSelected)
    return PA_ERR_SHAPE;
  const int group = num_heads / num_kv_heads;
  if (group != 1 && group != 2 && group != 4 && group != 8) return PA_ERR_SHAPE;
  if ((long long)num_seqs * num_kv_heads > INT32_MAX) return PA_ERR_SHAPE;
  if (num_seqs == 0) return PA_OK;
  if (!selected || !q || !block_bounds || !context_lens || (max_blocks_per_seq > 0 && !block_tables)) return PA_ERR_NULL;
  if (!aligned(selected, 4) || !aligned(q, 16) || !aligned(block_bounds, 16) || !aligned(block_tables, 4) ||
      !aligned(context_lens, 4))
    return PA_ERR_ALIGN;
  const size_t need = pa_select_blocks_workspace_bytes(num_seqs, num_kv_heads, max_context_len);
  if (need > 0) {
    if (!workspace || workspace_bytes < need) return PA_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return PA_ERR_ALIGN;
  }
  pa::SelectParams p{};
  p.q = q;
  p.bounds = (const uint4 *)block_bounds;
  p.block_tables = block_tables;
  p.context_lens = context_lens;
  p.approx = (float2 *)workspace;
  p.keys = (unsigned long long *)(static_cast<char *>(workspace) + need / 2);
  p.selected = selected;
  p.num_blocks = num_blocks;
  p.num_seqs = num_seqs;
  p.num_heads = num_heads;
  p.num_kv_heads = num_kv_heads;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.max_context_len = max_context_len;
  p.max_blocks = (int)(((long long)max_context_len + kBlockSize - 1) / kBlockSize);
  p.num_selected = num_selected;
  p.sink = sink_blocks;
  p.recent = recent_blocks;
  p.chunks = (p.max_blocks + pa::kScoreBlocks - 1) / pa::kScoreBlocks;
  cudaStream_t s = (cudaStream_t)stream;
  switch (dtype) {
    case PA_F32: return dispatch_choice<float>(group, p, s);
    case PA_F16: return dispatch_choice<__half>(group, p, s);
    case PA_BF16: return dispatch_choice<__nv_bfloat16>(group, p, s);
    case PA_FP8_E4M3: break;
  }
  return PA_ERR_DTYPE;
}

}  // extern "C"

namespace {

// Tokens a partition of a selected-block decode: a multiple of 4 blocks (one a warp)
// that gives the shortest run, in units of a block a warp: a wave of three CTAs an SM
// takes its share of a partition's blocks plus about two blocks' time of set-up
// and merge, and every partition adds a partial to combine.
int selected_partition(int num_seqs, int num_kv_heads, int num_selected) {
  const long long pairs = (long long)num_seqs * num_kv_heads;
  const long long slots = 3LL * sm_count();
  double best = 1e300;
  int blocks = 4;
  for (int parts = 1; parts <= 64 && (parts == 1 || 4 * (parts - 1) < num_selected); ++parts) {
    const int per = ((num_selected + parts - 1) / parts + 3) / 4 * 4;
    const int n = (num_selected + per - 1) / per;
    // a last wave that is not full runs faster: it counts for at least half
    const double full = (double)(pairs * n / slots), rest = (double)(pairs * n % slots) / slots;
    const double waves = full + (rest > 0 ? (rest > 0.5 ? rest : 0.5) : 0.0);
    const double cost = (waves < 1 ? 1 : waves) * (per / 4 + 2) + 0.25 * n;
    if (cost < best) {
      best = cost;
      blocks = per;
    }
  }
  return blocks * kBlockSize;
}

template <typename T, int G, typename Math, int W = pa::kDecodeWarps>
pa_status_t launch_selected(const CUtensorMap &mk, const CUtensorMap &mv, const pa::SelectedParams &p,
                            cudaStream_t stream) {
  const long long grid = (long long)p.num_seqs * p.num_kv_heads * p.max_partitions;
  if (grid > INT32_MAX) return PA_ERR_SHAPE;
  // More CTAs than a wave of three an SM: two-warp CTAs, six an SM, where the block
  // math has them (640 CTAs of 16 blocks, G = 4: 19.5 us against 21.7 with four warps, 768 CTAs 17.6
  // against 19.2; within one wave four warps: 64 CTAs 7.6 against 8.8, 384 CTAs 17.1 against 17.7).
  if constexpr (W == pa::kDecodeWarps && !Math::kNeedsQInSmem) {
    if (grid > 3LL * sm_count()) return launch_selected<T, G, Math, 2>(mk, mv, p, stream);
  }
  using SM = pa::DecodeSmem<T, G, Math, W>;
  auto kernel = pa::pa_decode_partition_kernel<T, G, Math, W, pa::kWalkSelected>;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, SM::kAlloc) != cudaSuccess)
    return PA_ERR_CUDA;
  const pa_status_t st = launch(kernel, dim3((unsigned)grid), dim3(W * 32), SM::kAlloc, stream, mk, mv, p);
  if (st != PA_OK || p.max_partitions <= 1) return st;
  const long long rows = (long long)p.num_seqs * p.num_heads;
  long long ctas = (rows + pa::kReduceWarps - 1) / pa::kReduceWarps;
  if (ctas > 8LL * sm_count()) ctas = 8LL * sm_count();
  return launch(pa::pa_join_selected_kernel<T>, dim3((unsigned)ctas), dim3(pa::kReduceWarps * 32), 0, stream, p);
}

template <typename T>
pa_status_t dispatch_selected(int group, const CUtensorMap &mk, const CUtensorMap &mv, const pa::SelectedParams &p,
                              cudaStream_t s) {
  constexpr bool kMma = !std::is_same<T, float>::value;
  switch (group) {
    case 1: return launch_selected<T, 1, pa::FmaMath<T, 1>>(mk, mv, p, s);
    case 2:
      if constexpr (kMma) return launch_selected<T, 2, pa::MmaMath<T, 2>>(mk, mv, p, s);
      else return launch_selected<T, 2, pa::FmaMath<T, 2>>(mk, mv, p, s);
    case 4:
      if constexpr (kMma) return launch_selected<T, 4, pa::MmaMath<T, 4>>(mk, mv, p, s);
      else return launch_selected<T, 4, pa::FmaMath<T, 4>>(mk, mv, p, s);
    case 8:
      if constexpr (kMma) return launch_selected<T, 8, pa::MmaMath<T, 8>>(mk, mv, p, s);
      else return launch_selected<T, 8, pa::FmaMath<T, 8>>(mk, mv, p, s);
  }
  return PA_ERR_SHAPE;
}

WorkspaceLayout selected_workspace(int num_seqs, int num_heads, int num_kv_heads, int head_dim, int num_selected) {
  const int blocks = selected_partition(num_seqs, num_kv_heads, num_selected) / kBlockSize;
  return workspace_layout(num_seqs, num_heads, num_kv_heads, head_dim, (num_selected + blocks - 1) / blocks);
}

}  // namespace

extern "C" {

size_t pa_decode_selected_workspace_bytes(int num_seqs, int num_heads, int num_kv_heads, int head_dim,
                                          int num_selected) {
  if (num_seqs <= 0 || num_heads <= 0 || num_kv_heads <= 0 || head_dim <= 0 || num_selected <= 0 ||
      num_selected > kMaxSelected)
    return 0;
  return selected_workspace(num_seqs, num_heads, num_kv_heads, head_dim, num_selected).bytes;
}

pa_status_t pa_decode_selected(void *out, const void *q, const void *k_cache, const void *v_cache,
                               const int32_t *block_tables, int max_blocks_per_seq, const int32_t *context_lens,
                               const int32_t *selected, int num_seqs, int num_heads, int num_selected, float scale,
                               void *workspace, size_t workspace_bytes, int64_t num_blocks, int block_size,
                               int num_kv_heads, int head_dim, pa_dtype_t dtype, void *stream) {
  if (dtype == PA_FP8_E4M3) return PA_ERR_DTYPE;
  if (num_selected <= 0 || num_selected > kMaxSelected) return PA_ERR_SHAPE;
  if (num_seqs > 0 && !selected) return PA_ERR_NULL;
  if (!aligned(selected, 4)) return PA_ERR_ALIGN;
  // every other check is pa_decode's (one partition: the split is planned below)
  const long long capacity = (long long)max_blocks_per_seq * kBlockSize;
  DecodePlan d;
  const pa_status_t st = plan_decode(d, out, q, nullptr, nullptr, k_cache, v_cache, block_tables, max_blocks_per_seq,
                                     context_lens, num_seqs, num_heads,
                                     capacity < 0 || capacity > INT32_MAX ? 0 : (int)capacity, scale, 0, num_blocks,
                                     block_size, num_kv_heads, head_dim, dtype, dtype, 1.f, 1.f);
  if (st != PA_OK || d.empty) return st;
  const WorkspaceLayout ws = selected_workspace(num_seqs, num_heads, num_kv_heads, head_dim, num_selected);
  if (ws.bytes > 0) {
    if (!workspace || workspace_bytes < ws.bytes) return PA_ERR_WORKSPACE;
    if (!aligned(workspace, 256)) return PA_ERR_ALIGN;
  }
  if (!encode_cache_map(&d.mk, k_cache, num_blocks, num_kv_heads, kRowBytes) ||
      !encode_cache_map(&d.mv, v_cache, num_blocks, num_kv_heads, kRowBytes))
    return PA_ERR_CUDA;
  pa::SelectedParams p{};
  static_cast<pa::DecodeParams &>(p) = d.p;
  char *w = static_cast<char *>(workspace);
  if (ws.bytes > 0) {
    p.ws_m = reinterpret_cast<float *>(w + ws.m_off);
    p.ws_l = reinterpret_cast<float *>(w + ws.l_off);
    p.ws_o = reinterpret_cast<float *>(w + ws.o_off);
  }
  p.partition_size = selected_partition(num_seqs, num_kv_heads, num_selected);
  p.max_partitions = (num_selected + p.partition_size / kBlockSize - 1) / (p.partition_size / kBlockSize);
  p.selected = selected;
  p.num_selected = num_selected;
  cudaStream_t s = (cudaStream_t)stream;
  switch (dtype) {
    case PA_F32: return dispatch_selected<float>(d.group, d.mk, d.mv, p, s);
    case PA_F16: return dispatch_selected<__half>(d.group, d.mk, d.mv, p, s);
    case PA_BF16: return dispatch_selected<__nv_bfloat16>(d.group, d.mk, d.mv, p, s);
    case PA_FP8_E4M3: break;
  }
  return PA_ERR_DTYPE;
}

pa_status_t pa_stream_read(const void *buf, size_t bytes, uint64_t *sink, void *stream) {
  if (bytes % 16 != 0) return PA_ERR_SHAPE;
  if (bytes == 0) return PA_OK;
  if (!buf || !sink) return PA_ERR_NULL;
  if (!aligned(buf, 16) || !aligned(sink, 8)) return PA_ERR_ALIGN;
  // eight resident CTAs of 256 threads per SM: a full SM of threads
  const long long n16 = (long long)(bytes / 16);
  long long ctas = (n16 + pa::kProbeThreads - 1) / pa::kProbeThreads;
  if (ctas > 8LL * sm_count()) ctas = 8LL * sm_count();
  return launch(pa::stream_read_kernel, dim3((unsigned)ctas), dim3(pa::kProbeThreads), 0, (cudaStream_t)stream,
                (const uint4 *)buf, n16, (unsigned long long *)sink);
}

pa_status_t pa_test_stall_next_launch(int kernel, int64_t cta) {
  if (cta < -1 || cta >= INT32_MAX) return PA_ERR_SHAPE;
  const int armed = (int)cta + 1;   // cta -1: disarm
  switch (kernel) {
    case 0: g_stall_decode.store(armed); return PA_OK;
    case 1: g_stall_prefill.store(armed); return PA_OK;
    case 3: g_stall_prefix.store(armed); return PA_OK;
  }
  return PA_ERR_SHAPE;
}

int pa_get_device_error(void *stream, int64_t *detail, int clear) {
  if (cudaStreamSynchronize((cudaStream_t)stream) != cudaSuccess) return -1;
  int code = 0;
  long long d = 0;
  if (cudaMemcpyFromSymbol(&code, pa::g_error_code, sizeof(int)) != cudaSuccess) return -1;
  if (cudaMemcpyFromSymbol(&d, pa::g_error_detail, sizeof(long long)) != cudaSuccess) return -1;
  if (detail) *detail = d;
  if (clear) {
    const int zero = 0;
    const long long zd = 0;
    if (cudaMemcpyToSymbol(pa::g_error_code, &zero, sizeof(int)) != cudaSuccess) return -1;
    if (cudaMemcpyToSymbol(pa::g_error_detail, &zd, sizeof(long long)) != cudaSuccess) return -1;
  }
  return code;
}

const char *pa_status_string(pa_status_t status) {
  switch (status) {
    case PA_OK: return "PA_OK";
    case PA_ERR_NULL: return "PA_ERR_NULL: a required pointer is NULL";
    case PA_ERR_DTYPE: return "PA_ERR_DTYPE: unknown dtype";
    case PA_ERR_SHAPE: return "PA_ERR_SHAPE: unsupported or inconsistent sizes";
    case PA_ERR_WORKSPACE: return "PA_ERR_WORKSPACE: split-K workspace missing or too small";
    case PA_ERR_CUDA: return "PA_ERR_CUDA: a CUDA call or kernel launch failed";
    case PA_ERR_ALIGN: return "PA_ERR_ALIGN: a pointer is not aligned as required";
  }
  return "unknown status";
}

}  // extern "C"

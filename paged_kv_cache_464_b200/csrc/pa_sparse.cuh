// pa_sparse.cuh -- which blocks of a paged cache a query attends to: per-block
// key bounds, the score they give, and the choice of the best.  The attention
// over the chosen blocks is the partition kernel of pa_decode.cuh (kWalkSelected).
// Included only from pa.cu.
//
// For block j of KV head g, lo[d] and hi[d] are the smallest and largest key
// element d over the block's tokens.  For a query head h of the group,
//   s_h(j) = sum_d (q_d >= 0 ? q_d hi[d] : q_d lo[d])  >=  q . K_t  for every t in j,
// the largest product that any token within the bounds could have, and the
// block's score is max_h s_h(j).  The bounds are 1/16 of the keys and values.
#pragma once

#include <cuda_bf16.h>

#include "pa_common.cuh"
#include "pa_decode.cuh"

namespace pa {

// ---------------------------------------------------------------- bounds
struct BoundsParams {
  const uint4 *k_cache;           // [NB][16][Hkv][16 chunks]
  uint4 *bounds;                  // [NB][2][Hkv][16 chunks]: 0 = smallest, 1 = largest
  const int32_t *block_tables;    // [S][MBS]
  const int32_t *context_lens;    // [S]
  const int32_t *new_lens;        // [S]
  long long num_blocks;
  int num_seqs, max_blocks_per_seq, chunks_per_token, max_new_len, blocks_per_seq;
};

// Element-wise smaller / larger of two chunks; a NaN on either side stays (a
// block with a NaN key is then always chosen, as dense attention would meet it).
template <typename T, bool kMax>
__device__ __forceinline__ uint32_t bound_word(uint32_t a, uint32_t b) {
  uint32_t r;
  if constexpr (sizeof(T) == 4) {
    if (kMax) asm("max.NaN.f32 %0, %1, %2;" : "=f"(*reinterpret_cast<float *>(&r)) : "f"(__uint_as_float(a)), "f"(__uint_as_float(b)));
    else asm("min.NaN.f32 %0, %1, %2;" : "=f"(*reinterpret_cast<float *>(&r)) : "f"(__uint_as_float(a)), "f"(__uint_as_float(b)));
  } else if constexpr (std::is_same<T, __half>::value) {
    if (kMax) asm("max.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else asm("min.NaN.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  } else {
    if (kMax) asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    else asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  }
  return r;
}

template <typename T, bool kMax>
__device__ __forceinline__ void bound_chunk(uint4 &a, const uint4 &b) {
  a.x = bound_word<T, kMax>(a.x, b.x);
  a.y = bound_word<T, kMax>(a.y, b.y);
  a.z = bound_word<T, kMax>(a.z, b.z);
  a.w = bound_word<T, kMax>(a.w, b.w);
}

// The bounds of every block that holds one of a sequence's last new_lens[b]
// tokens, from all of the block's tokens (those before the new ones too, so
// the result does not depend on what the bounds held).  A thread owns one 16-byte
// chunk of one head's row and loads it for the block's 16 tokens at once.  528 blocks of
// 8 heads (19 MB) take 3.6 us, 256 blocks 2.8 (a launch and three dependent loads).
template <typename T>
__global__ void __launch_bounds__(256) block_bounds_kernel(const BoundsParams p) {
  pdl_wait();
  pdl_trigger();
  const long long per_seq = static_cast<long long>(p.blocks_per_seq) * p.chunks_per_token;
  const long long total = per_seq * p.num_seqs;
  const long long stride = static_cast<long long>(gridDim.x) * blockDim.x;
  for (long long k = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; k < total; k += stride) {
    const int b = static_cast<int>(k / per_seq);
    const long long rest = k - b * per_seq;
    const int i = static_cast<int>(rest / p.chunks_per_token);
    const int c = static_cast<int>(rest - static_cast<long long>(i) * p.chunks_per_token);
    const int L = p.context_lens[b], n = p.new_lens[b];
    if (L < 0 || n < 0 || n > L || n > p.max_new_len || L > p.max_blocks_per_seq * kBlockSize) {
      if (rest == 0) record_error(4 /*PA_DEV_BAD_CONTEXT_LEN*/, b);
      continue;
    }
    const int j = (L - n) / kBlockSize + i;
    if (n == 0 || j > (L - 1) / kBlockSize) continue;   // (j * 16 may pass 2^31)
    const int id = p.block_tables[static_cast<size_t>(b) * p.max_blocks_per_seq + j];
    if (id < 0 || id >= p.num_blocks) {
      if (c == 0) record_error(1 /*PA_DEV_BAD_BLOCK_ID*/, id);
      continue;
    }
    const int nvalid = min(kBlockSize, L - j * kBlockSize);
    const uint4 *src = p.k_cache + static_cast<size_t>(id) * kBlockSize * p.chunks_per_token + c;
    uint4 x[kBlockSize];
#pragma unroll
    for (int t = 0; t < kBlockSize; ++t)   // past the end: token 0 again, which changes nothing
      x[t] = src[static_cast<size_t>(t < nvalid ? t : 0) * p.chunks_per_token];
    uint4 lo = x[0], hi = x[0];
#pragma unroll
    for (int t = 1; t < kBlockSize; ++t) {
      bound_chunk<T, false>(lo, x[t]);
      bound_chunk<T, true>(hi, x[t]);
    }
    uint4 *dst = p.bounds + static_cast<size_t>(id) * 2 * p.chunks_per_token + c;
    dst[0] = lo;
    dst[p.chunks_per_token] = hi;
  }
}

// ---------------------------------------------------------------- scores
// Which blocks are chosen is decided by fp64 scores, but few of them are computed:
// block_score_kernel gives every block an fp32 score with a bound on its error, and
// block_select_kernel computes fp64 scores only for the blocks that the bound leaves in
// doubt.  fp64 scores of all blocks cost 80 us for 8 x 8 x 2048 blocks and 8 heads (two
// conversions to fp64 for each product, 16 a cycle and SM), the fp32 ones 13 (67 MB at
// 5 TB/s, 77% of the copy bandwidth: each warp's chain of length, block id and rows).
struct SelectParams {
  const void *q;                  // [S][Hq][D]
  const uint4 *bounds;            // [NB][2][Hkv][16 chunks]
  const int32_t *block_tables;    // [S][MBS]
  const int32_t *context_lens;    // [S]
  float2 *approx;                 // [S][Hkv][max_blocks] (score, error bound; an infinite bound: in doubt)
  unsigned long long *keys;       // [S][Hkv][max_blocks] fp64 scores in an order-preserving code
  int32_t *selected;              // [S][Hkv][K]
  long long num_blocks;
  int num_seqs, num_heads, num_kv_heads, max_blocks_per_seq, max_context_len;
  int max_blocks;                 // of a sequence: ceil(max_context_len / 16)
  int num_selected, sink, recent;
  int chunks;                     // CTAs a (sequence, KV head) in the score launch
};

// Doubles as unsigned integers in the same order (-0 as +0); NaN is largest.
__device__ __forceinline__ unsigned long long score_key(double s) {
  if (s != s) return ~0ull;
  const unsigned long long u = static_cast<unsigned long long>(__double_as_longlong(s + 0.0));
  return (u >> 63) ? ~u : u | (1ull << 63);
}

constexpr int kScoreWarps = 4;
constexpr int kScoreBlocks = 64;   // blocks a CTA scores: 16 a warp
// |fp32 score - score| <= kScoreError * sum_d |q_d| max(|lo_d|, |hi_d|).  The products of
// 16-bit values are exact; a sum of 256 of them in fp32, whatever its order and if each
// step drops bits below 2^-23 of the larger operand, is off by less than 2^-15 of
// the sum of magnitudes; 64 fp32 products and sums by less than 2^-17.
// Products and sums below the fp32 range lose at most 2^-126 each.
constexpr float kScoreError = 1.f / 16384, kScoreErrorMin = 0x1p-116f;

// 16-bit caches: s_h(j) = q+ . hi + q- . lo with q+ = max(q, 0), q- = min(q, 0), as
// warp-level matrix products (m16n8k16): 16 blocks by 8 heads, head_dim in any
// order as long as both operands agree -- so each lane loads 16-byte chunks (eight
// elements, the k slots of two products) of its rows straight from global memory, 256
// bytes a lane in flight.  A third product gives the error bound's sum.
template <typename T, int G>
__device__ __forceinline__ void score_tile(const SelectParams &p, int b, int g, int j0, int n) {
  const int lane = threadIdx.x & 31, gid = lane >> 2, tig = lane & 3;
  uint4 qv[4];   // head gid: elements 32 i + 8 tig ..
  const uint4 *qg = reinterpret_cast<const uint4 *>(static_cast<const T *>(p.q)) +
                    (static_cast<size_t>(b) * p.num_heads + g * G) * kChunksPerRow;
#pragma unroll
  for (int i = 0; i < 4; ++i) qv[i] = gid < G ? qg[gid * kChunksPerRow + 4 * i + tig] : make_uint4(0u, 0u, 0u, 0u);
  int id = -1;
  if (lane < 16 && j0 + lane < n) {
    id = p.block_tables[static_cast<size_t>(b) * p.max_blocks_per_seq + j0 + lane];
    if (id < 0 || id >= p.num_blocks) {
      record_error(1 /*PA_DEV_BAD_BLOCK_ID*/, id);
      id = -1;
    }
  }
  const size_t hi_off = static_cast<size_t>(p.num_kv_heads) * kChunksPerRow;
  uint4 lo[2][4], hi[2][4];
#pragma unroll
  for (int r = 0; r < 2; ++r) {   // rows gid, gid + 8
    const int rid = __shfl_sync(kFullMask, id, gid + 8 * r);
    const uint4 *src = p.bounds + (static_cast<size_t>(rid < 0 ? 0 : rid) * 2 * p.num_kv_heads + g) * kChunksPerRow + tig;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      lo[r][i] = src[4 * i];
      hi[r][i] = src[hi_off + 4 * i];
    }
  }
  float s[4] = {0.f, 0.f, 0.f, 0.f}, t[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t qw[4] = {qv[i].x, qv[i].y, qv[i].z, qv[i].w};
    const uint32_t l0[4] = {lo[0][i].x, lo[0][i].y, lo[0][i].z, lo[0][i].w};
    const uint32_t l1[4] = {lo[1][i].x, lo[1][i].y, lo[1][i].z, lo[1][i].w};
    const uint32_t h0[4] = {hi[0][i].x, hi[0][i].y, hi[0][i].z, hi[0][i].w};
    const uint32_t h1[4] = {hi[1][i].x, hi[1][i].y, hi[1][i].z, hi[1][i].w};
#pragma unroll
    for (int k = 0; k < 2; ++k) {   // words 2k, 2k + 1 are the k slots 2 tig .. and 2 tig + 8 ..
      const uint32_t q0 = qw[2 * k], q1 = qw[2 * k + 1];
      const uint32_t ah[4] = {h0[2 * k], h1[2 * k], h0[2 * k + 1], h1[2 * k + 1]};
      const uint32_t al[4] = {l0[2 * k], l1[2 * k], l0[2 * k + 1], l1[2 * k + 1]};
      uint32_t am[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) am[e] = bound_word<T, true>(ah[e] & 0x7fff7fffu, al[e] & 0x7fff7fffu);
      MmaType<T>::mma(s, ah, bound_word<T, true>(q0, 0u), bound_word<T, true>(q1, 0u));
      MmaType<T>::mma(s, al, bound_word<T, false>(q0, 0u), bound_word<T, false>(q1, 0u));
      MmaType<T>::mma(t, am, q0 & 0x7fff7fffu, q1 & 0x7fff7fffu);
    }
  }
  float2 *out = p.approx + (static_cast<size_t>(b) * p.num_kv_heads + g) * p.max_blocks;
#pragma unroll
  for (int r = 0; r < 2; ++r) {   // s[2r], s[2r + 1]: row gid + 8 r, heads 2 tig, 2 tig + 1
    float best = -INFINITY, most = 0.f;
    // no such block, or not finite: left to the fp64 score (the former's puts it last)
    bool odd = __shfl_sync(kFullMask, id, gid + 8 * r) < 0;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if (2 * tig + e >= G) continue;
      odd = odd || !(fabsf(s[2 * r + e]) < INFINITY) || !(t[2 * r + e] < INFINITY);
      best = fmaxf(best, s[2 * r + e]);
      most = fmaxf(most, t[2 * r + e]);
    }
#pragma unroll
    for (int off = 1; off < 4; off <<= 1) {
      best = fmaxf(best, __shfl_xor_sync(kFullMask, best, off));
      most = fmaxf(most, __shfl_xor_sync(kFullMask, most, off));
      odd = __shfl_xor_sync(kFullMask, odd ? 1 : 0, off) != 0 || odd;
    }
    const int j = j0 + gid + 8 * r;
    if (tig == 0 && j < n) out[j] = make_float2(best, odd ? INFINITY : fmaf(most, kScoreError, kScoreErrorMin));
  }
}

// fp32 caches: a half warp scores a block, lane c of it chunk c of every row.
template <int G>
__device__ __forceinline__ void score_tile_f32(const SelectParams &p, int b, int g, int j0, int n) {
  const int lane = threadIdx.x & 31, c = lane & 15;
  float q[G][4];
  const uint4 *qg = static_cast<const uint4 *>(p.q) + (static_cast<size_t>(b) * p.num_heads + g * G) * kChunksPerRow + c;
#pragma unroll
  for (int h = 0; h < G; ++h) Elem<float>::unpack(qg[h * kChunksPerRow], q[h]);
  float2 *out = p.approx + (static_cast<size_t>(b) * p.num_kv_heads + g) * p.max_blocks;
#pragma unroll 2
  for (int i = 0; i < 8; ++i) {
    const int j = j0 + 2 * i + (lane >> 4);
    int id = j < n ? p.block_tables[static_cast<size_t>(b) * p.max_blocks_per_seq + j] : 0;
    const bool bad = id < 0 || id >= p.num_blocks;   // left to the fp64 score, which puts it last
    if (bad) {
      if (c == 0) record_error(1 /*PA_DEV_BAD_BLOCK_ID*/, id);
      id = 0;
    }
    float lo[4], hi[4];
    const uint4 *src = p.bounds + (static_cast<size_t>(id) * 2 * p.num_kv_heads + g) * kChunksPerRow + c;
    Elem<float>::unpack(src[0], lo);
    Elem<float>::unpack(src[static_cast<size_t>(p.num_kv_heads) * kChunksPerRow], hi);
    float best = -INFINITY, most = 0.f;
    bool odd = bad;
#pragma unroll
    for (int h = 0; h < G; ++h) {
      float s = 0.f, t = 0.f;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        s = fmaf(q[h][e], q[h][e] >= 0.f ? hi[e] : lo[e], s);
        t = fmaf(fabsf(q[h][e]), fmaxf(fabsf(lo[e]), fabsf(hi[e])), t);
      }
#pragma unroll
      for (int off = 8; off > 0; off >>= 1) {
        s += __shfl_xor_sync(kFullMask, s, off);
        t += __shfl_xor_sync(kFullMask, t, off);
      }
      odd = odd || !(fabsf(s) < INFINITY) || !(t < INFINITY);
      best = fmaxf(best, s);
      most = fmaxf(most, t);
    }
    if (c == 0 && j < n) out[j] = make_float2(best, odd ? INFINITY : fmaf(most, kScoreError, kScoreErrorMin));
  }
}

// Six CTAs an SM: with the 80 registers a thread's 256 bytes are in flight at once (8 x 8 x
// 2048 blocks, a pass of choice and decode: 43.3 us; eight CTAs 45.6, seven 44.7, five 45.7;
// 64 x 8 x 2048, scores and choice: 119, 139, 131, 121).
template <typename T, int G>
__global__ void __launch_bounds__(kScoreWarps * 32, 6) block_score_kernel(const SelectParams p) {
  pdl_wait();
  pdl_trigger();
  int item = blockIdx.x;   // the heads of the same blocks side by side: their rows are neighbours in memory
  const int g = item % p.num_kv_heads;
  item /= p.num_kv_heads;
  const int chunk = item % p.chunks;
  const int b = item / p.chunks;
  const int L = p.context_lens[b];
  if (L < 0 || L > p.max_context_len || L > p.max_blocks_per_seq * kBlockSize) {
    if (chunk == 0 && g == 0 && threadIdx.x == 0) record_error(4 /*PA_DEV_BAD_CONTEXT_LEN*/, b);
    return;
  }
  const int n = (L + kBlockSize - 1) / kBlockSize;
  const int j0 = chunk * kScoreBlocks + (threadIdx.x >> 5) * 16;
  if (n <= p.num_selected || j0 >= n) return;   // every block is chosen, or none is left for this warp
  if constexpr (sizeof(T) == 4) score_tile_f32<G>(p, b, g, j0, n);
  else score_tile<T, G>(p, b, g, j0, n);
}

// ---------------------------------------------------------------- choice
constexpr int kSelectBins = 2048;
constexpr int kSelectCached = 4096;     // fp32 scores kept in shared memory (more are read again from L2)
constexpr int kSelectDoubt = 1024;      // blocks in doubt that the fast path takes
constexpr int kSelectMaxBlocks = 65536; // blocks that the fast path takes (a bit each)

// The fp64 score of block j, by a warp; every lane gets it.  Lane l holds elements
// E l .. of every row; all loads are in flight at once.
template <typename T, int G>
__device__ __noinline__ unsigned long long exact_key(const SelectParams &p, int b, int g, int j) {
  constexpr int D = kChunksPerRow * Elem<T>::kPerChunk;
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const int id = p.block_tables[static_cast<size_t>(b) * p.max_blocks_per_seq + j];
  if (id < 0 || id >= p.num_blocks) return 0ull;   // recorded by the score kernel
  struct alignas(8) Row {
    T x[E];
  };
  const Row *bounds = reinterpret_cast<const Row *>(p.bounds);
  const Row lo = bounds[(static_cast<size_t>(id) * 2 * p.num_kv_heads + g) * 32 + lane];
  const Row hi = bounds[(static_cast<size_t>(id) * 2 * p.num_kv_heads + p.num_kv_heads + g) * 32 + lane];
  const Row *qg = static_cast<const Row *>(p.q) + (static_cast<size_t>(b) * p.num_heads + g * G) * 32 + lane;
  Row q[G];
#pragma unroll
  for (int h = 0; h < G; ++h) q[h] = qg[h * 32];
  double s[G];
#pragma unroll
  for (int h = 0; h < G; ++h) {
    s[h] = 0.0;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const float x = Elem<T>::load(&q[h].x[e]);
      const float k = x >= 0.f ? Elem<T>::load(&hi.x[e]) : Elem<T>::load(&lo.x[e]);
      s[h] = fma(static_cast<double>(x), static_cast<double>(k), s[h]);
    }
  }
#pragma unroll
  for (int off = 16; off > 0; off >>= 1)
#pragma unroll
    for (int h = 0; h < G; ++h) s[h] += __shfl_xor_sync(kFullMask, s[h], off);
  unsigned long long best = score_key(s[0]);
#pragma unroll
  for (int h = 1; h < G; ++h) best = max(best, score_key(s[h]));
  return best;
}

// Exclusive sum of `x` over the CTA's threads, and the total.
template <int NT>
__device__ __forceinline__ int block_sum(int x, int *warp_s, int &total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int upto = x;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int y = __shfl_up_sync(kFullMask, upto, off);
    if (lane >= off) upto += y;
  }
  __syncthreads();   // warp_s of the previous call has been read
  if (lane == 31) warp_s[warp] = upto;
  __syncthreads();
  int before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < (NT / 32); ++w) {
    before += w < warp ? warp_s[w] : 0;
    total += warp_s[w];
  }
  return before + upto - x;
}

// Element-wise largest of `x` over the CTA's threads.
template <int NT>
__device__ __forceinline__ float4 block_max(float4 x, float4 *warp_f) {
  x = make_float4(warp_max(x.x), warp_max(x.y), warp_max(x.z), warp_max(x.w));
  __syncthreads();   // warp_f of the previous call has been read
  if ((threadIdx.x & 31) == 0) warp_f[threadIdx.x >> 5] = x;
  __syncthreads();
  const float4 y = warp_f[threadIdx.x & ((NT / 32) - 1)];
  return make_float4(warp_max(y.x), warp_max(y.y), warp_max(y.z), warp_max(y.w));
}

// The `need` largest fp64 scores of blocks j0 .. j1-1, ties to the lowest index, for lists
// that the fast path does not take: fp64 scores of all of them, then a radix select
// that narrows the smallest chosen key 8 bits at a time, then the list itself.
template <typename T, int G, int NT>
__device__ __noinline__ void select_all_exact(const SelectParams &p, int b, int g, int n, int j0, int j1, int need,
                                              unsigned long long *keys, int32_t *out, int *hist, int *warp_s,
                                              int *found) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll 1
  for (int j = j0 + warp; j < j1; j += (NT / 32)) {
    const unsigned long long key = exact_key<T, G>(p, b, g, j);
    if (lane == 0) keys[j] = key;
  }
  __syncthreads();
  unsigned long long prefix = 0;
  int shift = 64;
  while (shift > 0) {
#pragma unroll 1
    for (int i = threadIdx.x; i < 256; i += NT) hist[i] = 0;
    __syncthreads();
#pragma unroll 1
    for (int j = j0 + threadIdx.x; j < j1; j += NT) {
      const unsigned long long key = keys[j];
      if (shift == 64 || (key >> shift) == prefix) atomicAdd(&hist[(key >> (shift - 8)) & 255], 1);
    }
    __syncthreads();
    if (threadIdx.x == 0) {   // the digit that the need-th largest key has
      int d = 255, above = 0;
      while (above + hist[d] < need) above += hist[d--];
      found[0] = d;
      found[1] = above;
    }
    __syncthreads();
    need -= found[1];
    prefix = shift == 64 ? found[0] : (prefix << 8) | found[0];
    shift -= 8;
    __syncthreads();
  }
  int written = 0, equal_before = 0;
#pragma unroll 1
  for (int base = 0; base < n; base += NT) {
    const int j = base + threadIdx.x;
    bool take = j < n && (j < j0 || j >= j1), equal = false;
    if (j >= j0 && j < j1) {
      take = keys[j] > prefix;
      equal = keys[j] == prefix;
    }
    int total;
    const int rank = block_sum<NT>(equal ? 1 : 0, warp_s, total);
    if (equal && equal_before + rank < need) take = true;
    equal_before += total;
    const int at = block_sum<NT>(take ? 1 : 0, warp_s, total);
    if (take) out[written + at] = j;
    written += total;
  }
}

// A CTA per (sequence, KV head): the first `sink` and last `recent` blocks and,
// of the others, those of the largest scores, in ascending order; -1 behind them.
// With E the largest error bound and the need-th largest fp32 score within [t0, t1]
// (the scores of its bin of an even histogram), the need-th largest score is within
// [t0 - E, t1 + E]: an fp32 score above t1 + 2 E is chosen, one below t0 - 2 E is not,
// and only the rest is in doubt and ranked by fp64 scores (one to three blocks for N(0, 1)
// data; if more than kSelectDoubt, or more blocks than kSelectMaxBlocks, select_all_exact
// decides).  Its length, 8 us for 8 lists of 2048 blocks, is that of a dozen CTA-wide steps
// of 200 to 1300 cycles.  A thread keeps its first NT / 128 scores in registers (17.2 us a pass
// of choice and decode for one sequence; 18.5 with every score in shared memory).  Slower:
// bisection in the histogram's place; a first run through the code on a made-up
// list while the scores are computed, to have it in the instruction cache (19.7).
template <typename T, int G, int NT>
__global__ void __launch_bounds__(NT) block_select_kernel(const SelectParams p) {
  __shared__ union {
    int hist[kSelectBins];
    unsigned bits[kSelectMaxBlocks / 32];   // chosen blocks
  } u;
  __shared__ float score_s[kSelectCached];
  __shared__ unsigned long long doubt_key[kSelectDoubt];
  __shared__ int doubt_j[kSelectDoubt];
  __shared__ int warp_s[NT / 32];
  __shared__ float4 warp_f[NT / 32];
  __shared__ int found[2];
  __shared__ int num_doubt, num_in;
  static_assert(kSelectMaxBlocks / 32 <= kSelectBins, "the bits take the histogram's place");
  pdl_wait();
  pdl_trigger();
  const int g = blockIdx.x % p.num_kv_heads;
  const int b = blockIdx.x / p.num_kv_heads;
  const int K = p.num_selected;
  const int L = p.context_lens[b];
  int32_t *out = p.selected + static_cast<size_t>(blockIdx.x) * K;
  const bool bad = L < 0 || L > p.max_context_len || L > p.max_blocks_per_seq * kBlockSize;
  const int n = bad ? 0 : (L + kBlockSize - 1) / kBlockSize;   // a bad length: an empty list
  if (n <= K) {
    if (bad && threadIdx.x == 0) record_error(4 /*PA_DEV_BAD_CONTEXT_LEN*/, b);
#pragma unroll 1
    for (int i = threadIdx.x; i < K; i += NT) out[i] = i < n ? i : -1;
    return;
  }
  const float2 *approx = p.approx + static_cast<size_t>(blockIdx.x) * p.max_blocks;
  const int j0 = p.sink, j1 = n - p.recent;   // n > K >= sink + recent
  const int need = K - p.sink - p.recent;     // of the blocks j0 .. j1 - 1
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // ---- range and error of the fp32 scores; NaN marks the blocks that are in doubt anyway
  float top = -INFINITY, low = INFINITY, err = 0.f, odd = 0.f;
  constexpr int kReg = NT / 128;
  float2 ar[kReg];
#pragma unroll
  for (int k = 0; k < kReg; ++k) {
    const int j = j0 + threadIdx.x + k * NT;
    ar[k] = j < j1 ? approx[j] : make_float2(0.f, INFINITY);
  }
  float xr[kReg];
#pragma unroll
  for (int k = 0; k < kReg; ++k) {
    const bool fine = ar[k].y < INFINITY;
    xr[k] = fine ? ar[k].x : __int_as_float(0x7fffffff);
    if (fine) {
      top = fmaxf(top, ar[k].x);
      low = fminf(low, ar[k].x);
      err = fmaxf(err, ar[k].y);
    } else if (j0 + threadIdx.x + k * NT < j1) {
      odd = 1.f;
    }
  }
#pragma unroll 1
  for (int j = j0 + threadIdx.x + kReg * NT; j < j1; j += NT) {
    const float2 x = approx[j];
    const bool fine = x.y < INFINITY;
    if (j < kSelectCached) score_s[j] = fine ? x.x : __int_as_float(0x7fffffff);
    if (fine) {
      top = fmaxf(top, x.x);
      low = fminf(low, x.x);
      err = fmaxf(err, x.y);
    } else {
      odd = 1.f;
    }
  }
#pragma unroll 1
  for (int i = threadIdx.x; i < kSelectBins; i += NT) u.hist[i] = 0;
  if (threadIdx.x == 0) {
    num_doubt = num_in = 0;
    found[0] = -1;
  }
  const float4 range = block_max<NT>(make_float4(top, -low, err, odd), warp_f);
  top = range.x;
  low = -range.y;
  err = 2.f * range.z;
  const bool any_odd = range.w > 0.f;
  const float width = top - low;
  const float scale = width > 0.f && width < INFINITY ? (kSelectBins - 1) / width : 0.f;
  auto score = [&](int j) {
    if (j < kSelectCached) return score_s[j];
    const float2 x = approx[j];
    return x.y < INFINITY ? x.x : __int_as_float(0x7fffffff);
  };
  auto bin = [&](float x) { return min(kSelectBins - 1, static_cast<int>((x - low) * scale)); };   // grows with x
  float t0 = -INFINITY, t1 = INFINITY;   // no block with a finite score: all are in doubt
  if (need > 0) {
    int br[kReg];
#pragma unroll
    for (int k = 0; k < kReg; ++k) {
      br[k] = xr[k] == xr[k] ? bin(xr[k]) : -1;
      if (br[k] >= 0) atomicAdd(&u.hist[br[k]], 1);
    }
#pragma unroll 1
    for (int j = j0 + threadIdx.x + kReg * NT; j < j1; j += NT) {
      const float x = score(j);
      if (x == x) atomicAdd(&u.hist[bin(x)], 1);
    }
    __syncthreads();
    // the bin of the need-th largest (thread t: bins from the top down, 4 t .. 4 t + 3)
    constexpr int kPer = kSelectBins / NT;
    int mine = 0;
#pragma unroll
    for (int d = 0; d < kPer; ++d) mine += u.hist[kSelectBins - 1 - kPer * threadIdx.x - d];
    int total;
    int above = block_sum<NT>(mine, warp_s, total);
    if (above < need && above + mine >= need) {
      int d = kSelectBins - 1 - kPer * threadIdx.x;
      while (above + u.hist[d] < need) above += u.hist[d--];
      found[0] = d;
    }
    __syncthreads();
    const int at = found[0];
    float a = INFINITY, z = -INFINITY;
    if (at >= 0) {
#pragma unroll
      for (int k = 0; k < kReg; ++k)
        if (br[k] == at) {
          a = fminf(a, xr[k]);
          z = fmaxf(z, xr[k]);
        }
#pragma unroll 1
      for (int j = j0 + threadIdx.x + kReg * NT; j < j1; j += NT) {
        const float x = score(j);
        if (x == x && bin(x) == at) {
          a = fminf(a, x);
          z = fmaxf(z, x);
        }
      }
      const float4 edge = block_max<NT>(make_float4(-a, z, 0.f, 0.f), warp_f);
      t0 = -edge.x - err;
      t1 = edge.y + err;
    }
  }
  __syncthreads();
  // ---- chosen, not chosen, in doubt.  (Blocks without a finite fp32 score may be above any other
  // and take its place: with some, nothing is certain to be chosen; what is below t0 is still out.)
#pragma unroll 1
  for (int i = threadIdx.x; i < kSelectMaxBlocks / 32 && i * 32 < n; i += NT) u.bits[i] = 0u;
  __syncthreads();
  const bool fast = n <= kSelectMaxBlocks;
#pragma unroll
  for (int k = 0; k < kReg; ++k) {
    const int j = j0 + threadIdx.x + k * NT;
    const float x = xr[k];
    const bool live = j < j1 && need > 0 && fast;
    const bool in = live && !any_odd && x > t1;
    const bool doubt = live && !in && !(x < t0);
    if (in) {
      atomicAdd(&num_in, 1);
      atomicOr(&u.bits[j >> 5], 1u << (j & 31));
    }
    if (doubt) {
      const int at = atomicAdd(&num_doubt, 1);
      if (at < kSelectDoubt) doubt_j[at] = j;
    }
  }
#pragma unroll 1
  for (int base = j0 + kReg * NT; base < j1 && need > 0 && fast; base += NT) {
    const int j = base + threadIdx.x;
    const float x = j < j1 ? score(j) : -INFINITY;
    const bool in = j < j1 && !any_odd && x > t1;
    const bool doubt = j < j1 && !in && !(x < t0);
    if (in) {
      atomicAdd(&num_in, 1);
      atomicOr(&u.bits[j >> 5], 1u << (j & 31));
    }
    if (doubt) {
      const int at = atomicAdd(&num_doubt, 1);
      if (at < kSelectDoubt) doubt_j[at] = j;
    }
  }
  __syncthreads();
  const int m = num_doubt;
  const int left = need - num_in;   // how many of the blocks in doubt are chosen
  if (need > 0 && (!fast || m > kSelectDoubt || left < 0)) {
    __syncthreads();
    select_all_exact<T, G, NT>(p, b, g, n, j0, j1, need, p.keys + static_cast<size_t>(blockIdx.x) * p.max_blocks, out,
                           u.hist, warp_s, found);
    return;
  }
  if (!fast) {   // need == 0: the first and last blocks alone
#pragma unroll 1
    for (int i = threadIdx.x; i < K; i += NT) out[i] = i < j0 ? i : n - K + i;
    return;
  }
  if (m > left) {
#pragma unroll 1
    for (int i = warp; i < m; i += (NT / 32)) {
      const unsigned long long key = exact_key<T, G>(p, b, g, doubt_j[i]);
      if (lane == 0) doubt_key[i] = key;
    }
    __syncthreads();
  }
#pragma unroll 1
  for (int i = threadIdx.x; i < m; i += NT) {
    const int j = doubt_j[i];
    int before = 0;   // blocks in doubt that are chosen before this one
    if (m > left) {
      const unsigned long long key = doubt_key[i];
#pragma unroll 1
      for (int k = 0; k < m; ++k) before += doubt_key[k] > key || (doubt_key[k] == key && doubt_j[k] < j);
    }
    if (before < left) atomicOr(&u.bits[j >> 5], 1u << (j & 31));
  }
#pragma unroll 1
  for (int j = threadIdx.x; j < j0; j += NT) atomicOr(&u.bits[j >> 5], 1u << (j & 31));
#pragma unroll 1
  for (int j = j1 + threadIdx.x; j < n; j += NT) atomicOr(&u.bits[j >> 5], 1u << (j & 31));
  __syncthreads();
  // ---- the list
  int written = 0;
  const int words = (n + 31) / 32;
#pragma unroll 1
  for (int base = 0; base < words; base += NT) {
    unsigned w = base + threadIdx.x < words ? u.bits[base + threadIdx.x] : 0u;
    int total;
    int at = written + block_sum<NT>(__popc(w), warp_s, total);
    for (; w != 0u; w &= w - 1u) out[at++] = (base + threadIdx.x) * 32 + __ffs(w) - 1;
    written += total;
  }
}

}  // namespace pa

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
// chunk of one head's row and loads it for the block's 16 tokens at once.
template <typename T>
__global__ void __launch_bounds__(128) block_bounds_kernel(const BoundsParams p) {
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
    if (n == 0 || j * kBlockSize >= L) continue;
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
struct SelectParams {
  const void *q;                  // [S][Hq][D]
  const uint4 *bounds;            // [NB][2][Hkv][16 chunks]
  const int32_t *block_tables;    // [S][MBS]
  const int32_t *context_lens;    // [S]
  unsigned long long *keys;       // [S][Hkv][max_blocks] scores in an order-preserving code
  int32_t *selected;              // [S][Hkv][K]
  long long num_blocks;
  int num_seqs, num_heads, num_kv_heads, max_blocks_per_seq, max_context_len;
  int max_blocks;                 // of a sequence: ceil(max_context_len / 16)
  int num_selected, sink, recent;
  int chunks;                     // CTAs a (sequence, KV head) in the score launch
};

// Doubles as unsigned integers in the same order (-0 below +0, which add up
// equal only by a sum of all zeros: both are then mapped to +0); NaN is largest.
__device__ __forceinline__ unsigned long long score_key(double s) {
  if (s != s) return ~0ull;
  const unsigned long long u = static_cast<unsigned long long>(__double_as_longlong(s + 0.0));
  return (u >> 63) ? ~u : u | (1ull << 63);
}

constexpr int kScoreWarps = 4;
constexpr int kScoreBlocks = 64;   // blocks a CTA scores: 8 for each of its 8 half warps

// A half warp scores a block: lane c of it holds chunk c of the block's two
// rows and of the G query rows.  Sums are fp64 (the products of 16-bit values
// are exact in fp32, those of fp32 values in fp64), so that the order in which
// terms are added decides no near tie.
template <typename T, int G>
__global__ void __launch_bounds__(kScoreWarps * 32) block_score_kernel(const SelectParams p) {
  constexpr int EPC = Elem<T>::kPerChunk;
  pdl_wait();
  pdl_trigger();
  int item = blockIdx.x;
  const int chunk = item % p.chunks;
  item /= p.chunks;
  const int g = item % p.num_kv_heads;
  const int b = item / p.num_kv_heads;
  const int L = p.context_lens[b];
  if (L < 0 || L > p.max_context_len || L > p.max_blocks_per_seq * kBlockSize) {
    if (chunk == 0 && g == 0 && threadIdx.x == 0) record_error(4 /*PA_DEV_BAD_CONTEXT_LEN*/, b);
    return;
  }
  const int n = (L + kBlockSize - 1) / kBlockSize;
  if (n <= p.num_selected) return;   // every block is chosen
  const int lane = threadIdx.x & 31, c = lane & 15;
  const int half = (threadIdx.x >> 5) * 2 + (lane >> 4);
  float q[G][EPC];
  const uint4 *qg = reinterpret_cast<const uint4 *>(static_cast<const T *>(p.q)) +
                    (static_cast<size_t>(b) * p.num_heads + g * G) * kChunksPerRow + c;
#pragma unroll
  for (int h = 0; h < G; ++h) Elem<T>::unpack(qg[h * kChunksPerRow], q[h]);
  const int32_t *bt = p.block_tables + static_cast<size_t>(b) * p.max_blocks_per_seq;
  unsigned long long *keys = p.keys + (static_cast<size_t>(b) * p.num_kv_heads + g) * p.max_blocks;
  for (int i = 0; i < kScoreBlocks; i += 2 * kScoreWarps) {
    const int j = chunk * kScoreBlocks + i + half;
    const int id = j < n ? bt[j] : 0;
    const bool good = j < n && id >= 0 && id < p.num_blocks;
    if (j < n && !good && c == 0) record_error(1 /*PA_DEV_BAD_BLOCK_ID*/, id);
    float lo[EPC], hi[EPC];
    {
      const uint4 *src = p.bounds + (static_cast<size_t>(good ? id : 0) * 2 * p.num_kv_heads + g) * kChunksPerRow + c;
      Elem<T>::unpack(src[0], lo);
      Elem<T>::unpack(src[static_cast<size_t>(p.num_kv_heads) * kChunksPerRow], hi);
    }
    double best = 0.0;
#pragma unroll
    for (int h = 0; h < G; ++h) {
      double s = 0.0;
#pragma unroll
      for (int e = 0; e < EPC; ++e) {
        const float k = q[h][e] >= 0.f ? hi[e] : lo[e];
        s = fma(static_cast<double>(q[h][e]), static_cast<double>(k), s);
      }
#pragma unroll
      for (int off = 8; off > 0; off >>= 1) s += __shfl_xor_sync(kFullMask, s, off);
      best = h == 0 || s > best || s != s ? s : best;   // a NaN stays: no later score is larger than it
    }
    if (c == 0 && j < n) keys[j] = good ? score_key(best) : 0ull;
  }
}

// ---------------------------------------------------------------- choice
constexpr int kSelectThreads = 256;

// Exclusive sum of `flag` over the CTA's threads, and the total.
__device__ __forceinline__ int block_rank(bool flag, int *warp_s, int &total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const unsigned bits = __ballot_sync(kFullMask, flag);
  __syncthreads();   // warp_s of the previous call has been read
  if (lane == 0) warp_s[warp] = __popc(bits);
  __syncthreads();
  int before = 0;
  total = 0;
#pragma unroll
  for (int w = 0; w < kSelectThreads / 32; ++w) {
    before += w < warp ? warp_s[w] : 0;
    total += warp_s[w];
  }
  return before + __popc(bits & ((1u << lane) - 1u));
}

// A CTA per (sequence, KV head): the first `sink` and last `recent` blocks and,
// of the others, those of the largest keys -- a radix select that narrows the
// smallest chosen key 8 bits at a time -- written in ascending order, ties to the
// lowest index; -1 behind them.
__global__ void __launch_bounds__(kSelectThreads) block_select_kernel(const SelectParams p) {
  __shared__ int hist[256];
  __shared__ int warp_s[kSelectThreads / 32];
  __shared__ int found_digit, found_above;
  pdl_wait();
  pdl_trigger();
  const int b = blockIdx.x / p.num_kv_heads;
  const int K = p.num_selected;
  const int L = p.context_lens[b];
  int32_t *out = p.selected + static_cast<size_t>(blockIdx.x) * K;
  const unsigned long long *keys = p.keys + static_cast<size_t>(blockIdx.x) * p.max_blocks;
  const bool bad = L < 0 || L > p.max_context_len || L > p.max_blocks_per_seq * kBlockSize;
  const int n = bad ? 0 : (L + kBlockSize - 1) / kBlockSize;   // a bad length: an empty list
  if (n <= K) {
    if (bad && threadIdx.x == 0) record_error(4 /*PA_DEV_BAD_CONTEXT_LEN*/, b);
    for (int i = threadIdx.x; i < K; i += kSelectThreads) out[i] = i < n ? i : -1;
    return;
  }
  const int j0 = p.sink, j1 = n - p.recent;   // n > K >= sink + recent
  int need = K - p.sink - p.recent;           // of the blocks j0 .. j1 - 1
  // chosen: key >> shift above `prefix`, and the first `need` of those equal to it
  unsigned long long prefix = 0;
  int shift = 64;
  while (need > 0 && shift > 0) {
    for (int i = threadIdx.x; i < 256; i += kSelectThreads) hist[i] = 0;
    __syncthreads();
    for (int j = j0 + threadIdx.x; j < j1; j += kSelectThreads) {
      const unsigned long long key = keys[j];
      if (shift == 64 || (key >> shift) == prefix) atomicAdd(&hist[(key >> (shift - 8)) & 255], 1);
    }
    __syncthreads();
    if (threadIdx.x < 32) {   // the digit that the need-th largest key has
      const int lane = threadIdx.x;
      int mine = 0;   // lane l: digits 255 - 8 l down to 248 - 8 l
#pragma unroll
      for (int d = 0; d < 8; ++d) mine += hist[255 - 8 * lane - d];
      int upto = mine;
#pragma unroll
      for (int off = 1; off < 32; off <<= 1) {
        const int x = __shfl_up_sync(kFullMask, upto, off);
        if (lane >= off) upto += x;
      }
      int above = upto - mine;
      if (above < need && upto >= need) {
        int d = 255 - 8 * lane;
        while (above + hist[d] < need) above += hist[d--];
        found_digit = d;
        found_above = above;
      }
    }
    __syncthreads();
    need -= found_above;
    prefix = shift == 64 ? found_digit : (prefix << 8) | found_digit;
    shift -= 8;
    const bool whole = hist[found_digit] == need;   // every key with this prefix is chosen
    __syncthreads();
    if (whole) break;
  }
  int written = 0, equal_before = 0;
  for (int base = 0; base < n; base += kSelectThreads) {
    const int j = base + threadIdx.x;
    bool take = j < n && (j < j0 || j >= j1), equal = false;
    if (j >= j0 && j < j1 && K > p.sink + p.recent) {
      const unsigned long long high = keys[j] >> shift;
      take = high > prefix;
      equal = high == prefix;
    }
    int total;
    const int rank = block_rank(equal, warp_s, total);
    if (equal && equal_before + rank < need) take = true;
    equal_before += total;
    const int at = block_rank(take, warp_s, total);
    if (take) out[written + at] = j;
    written += total;
  }
}

}  // namespace pa

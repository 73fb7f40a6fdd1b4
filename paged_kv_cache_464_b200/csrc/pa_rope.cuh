// pa_rope.cuh -- rotary position embedding applied on the way into the paged
// cache, and the table of cosines and sines it reads.  Included only from pa.cu.
//
// With angle t(p, i) = p * base^(-2i/r) for position p and pair i < r/2 of the
// first r elements of a head row, the pair (a, b) becomes
//   a' = a cos t - b sin t,   b' = b cos t + a sin t.
// The pair is (x[i], x[i + r/2]) or, interleaved, (x[2i], x[2i + 1]); elements
// from r on are copied.  q rows go to q_out, K rows (rotated) and V rows (as
// they are) to the token's cache slot.
//
// Every product and sum is fp32, each rounded by itself (no contraction: the
// result does not depend on which of the two products the compiler would fuse),
// and the row is rounded once to its stored type.
//
// Bound by HBM: 8192 tokens of 32/8 bf16 heads (206 MB) take 32.5 to 33 us, 95 to 97% of the
// copy bandwidth.  E4M3 caches: 4093 tokens (92 MB) 19.2 to 19.6 us, 73%: half the time the SMs issue
// (rotation, quotients by the scale, conversions), and 3.5 waves of CTAs leave a tail.
#pragma once

#include "pa_common.cuh"

namespace pa {

// cos_sin[p][0 .. r/2) = cos t(p, i), cos_sin[p][r/2 .. r) = sin t(p, i).  The
// angle and its sine and cosine are fp64: at p = 10^6 an fp32 angle would be off
// by up to 2^-5.  Run once when a model is loaded; a thread per (p, i).
__global__ void __launch_bounds__(256) rope_table_kernel(float *__restrict__ cos_sin, int max_position, int half,
                                                         double base) {
  pdl_wait();
  pdl_trigger();
  const long long total = static_cast<long long>(max_position) * half;
  const long long stride = static_cast<long long>(gridDim.x) * blockDim.x;
  for (long long k = static_cast<long long>(blockIdx.x) * blockDim.x + threadIdx.x; k < total; k += stride) {
    const long long p = k / half;
    const int i = static_cast<int>(k - p * half);
    const double angle = static_cast<double>(p) * pow(base, -static_cast<double>(i) / half);
    double s, c;
    sincos(angle, &s, &c);
    cos_sin[p * 2 * half + i] = static_cast<float>(c);
    cos_sin[p * 2 * half + half + i] = static_cast<float>(s);
  }
}

// A 1-byte cache's scale as power * s with s in [2^-60, 2^64] and power a power of two, so that
// remainders of quotients by s are exact; inv = 1 / s rounded to nearest.
struct E4m3Scale {
  float s, inv, unit;   // unit = 1 / power
};

struct RopeParams {
  void *q_out;                      // [T] rows of Hq * D elements, q_out_stride apart
  const void *q, *key, *value;      // [T] rows, *_stride elements apart; heads contiguous in a row
  void *k_cache, *v_cache;
  const int64_t *positions;         // [T]
  const float *cos_sin;             // [max_position][rotary]
  const int64_t *slot_mapping;      // [T]
  long long q_out_stride, q_stride, k_stride, v_stride;   // in elements
  long long num_slots, max_position;
  int num_tokens, num_heads, num_kv_heads, rotary;
  E4m3Scale k_scale, v_scale;       // 1-byte caches
};

// Two 16-byte chunks of fp32 values -> where they go: T rows (16 bytes a chunk)
// or, for 1-byte caches, E4M3 codes (8 bytes a chunk; nearest even, saturating).
template <typename T>
__device__ __forceinline__ uint4 pack_chunk(const float *f);
template <>
__device__ __forceinline__ uint4 pack_chunk<float>(const float *f) {
  return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}
template <>
__device__ __forceinline__ uint4 pack_chunk<__nv_bfloat16>(const float *f) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<uint32_t *>(&v);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}
template <>
__device__ __forceinline__ uint4 pack_chunk<__half>(const float *f) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    __half2 v = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
    w[i] = *reinterpret_cast<uint32_t *>(&v);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The quotient by a scale, rounded to fp32, where it is between 2^-12 and 512; below and
// above, a number with the same E4M3 code.  Two corrections by the remainder: x * inv is
// off by up to 1.5 units of the last place, the first correction by less than one, and a
// quotient within one becomes the rounded quotient by another (Markstein, Computation of elementary
// functions on the IBM RISC System/6000 processor, IBM J. Res. Dev. 34, 1990).  x * unit is exact
// or too small or large to matter; the remainder's sign keeps -0.  19.4 us for the case above
// against 22.7 with IEEE divisions, whose branches cost more than their instructions.
__device__ __forceinline__ float e4m3_quotient(float x, const E4m3Scale &c) {
  x *= c.unit;
  const float q = x * c.inv;
  const float y = fmaf(-fmaf(q, c.s, -x), c.inv, q);
  const float z = fmaf(-fmaf(y, c.s, -x), c.inv, y);
  return fabsf(q) < 512.f ? z : q;   // q itself: saturates, infinity, NaN
}

__device__ __forceinline__ uint2 pack_e4m3(const float *f, const E4m3Scale &scale) {
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = e4m3_quotient(f[i], scale);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint16_t a;   // cvt packs its first source into the upper byte
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(a) : "f"(y[2 * i + 1]), "f"(y[2 * i]));
    w[i] = a;
  }
  return make_uint2(w[0] | (w[1] << 16), w[2] | (w[3] << 16));
}

// A head row is 16 chunks of 16 bytes, and an item of work is two of them: the
// two halves of a rotated pair (item c: chunks c and c + r/2 in chunks), two adjacent
// chunks of the interleaved form, or two adjacent chunks past r.  A CTA is 4 tokens x 8
// heads x 8 items, so a warp covers four heads of a token and its two loads four
// 128-byte lines each; a thread takes its item of NH heads, 8 apart, with every load in
// flight before the first use (they do not wait for the position) and its
// cosines and sines (2 * EPC fp32) in registers for all of them.
constexpr int kRopeTokens = 4, kRopeHeads = 8, kRopeItems = kChunksPerRow / 2;

template <typename T, bool kInterleaved, bool kFp8, int NH>
__global__ void __launch_bounds__(kRopeTokens * kRopeHeads * kRopeItems) rope_and_cache_kernel(const RopeParams p) {
  constexpr int EPC = Elem<T>::kPerChunk;
  pdl_wait();
  pdl_trigger();
  const int c = threadIdx.x % kRopeItems;
  const int tok = blockIdx.x * kRopeTokens + threadIdx.x / (kRopeItems * kRopeHeads);
  if (tok >= p.num_tokens) return;
  const int h0 = blockIdx.y * (kRopeHeads * NH) + threadIdx.x / kRopeItems % kRopeHeads;
  const int n_rows = p.num_heads + 2 * p.num_kv_heads;   // the token's q, K and V rows
  const long long pos = p.positions[tok];
  const long long slot = p.slot_mapping[tok];
  const int rc = p.rotary / (2 * EPC);   // items that rotate
  const bool turns = c < rc;
  // the item's two chunks of a row
  const int c0 = kInterleaved || !turns ? 2 * c : c;
  const int c1 = kInterleaved || !turns ? 2 * c + 1 : c + rc;
  uint4 x0[NH], x1[NH];
#pragma unroll
  for (int u = 0; u < NH; ++u) {
    const int h = h0 + u * kRopeHeads;
    x0[u] = x1[u] = make_uint4(0u, 0u, 0u, 0u);
    if (h < n_rows) {
      const bool is_q = h < p.num_heads;
      const bool is_k = h < p.num_heads + p.num_kv_heads;
      const int hl = h - (is_q ? 0 : is_k ? p.num_heads : p.num_heads + p.num_kv_heads);
      const T *base = static_cast<const T *>(is_q ? p.q : is_k ? p.key : p.value) +
                      tok * (is_q ? p.q_stride : is_k ? p.k_stride : p.v_stride);
      const uint4 *src = reinterpret_cast<const uint4 *>(base) + hl * kChunksPerRow;
      x0[u] = NH > 1 ? __ldcs(src + c0) : src[c0];
      x1[u] = NH > 1 ? __ldcs(src + c1) : src[c1];
    }
  }
  if (pos < 0) return;   // padding token: nothing is written
  const bool first = threadIdx.x % (kRopeItems * kRopeHeads) == 0 && blockIdx.y == 0;
  if (pos >= p.max_position) {
    if (first) record_error(7 /*PA_DEV_BAD_POSITION*/, pos);
    return;
  }
  if (slot >= p.num_slots && first) record_error(2 /*PA_DEV_BAD_SLOT*/, slot);
  const bool cached = slot >= 0 && slot < p.num_slots;
  float cs[EPC], sn[EPC];
  if (turns) {
    const float *row = p.cos_sin + pos * p.rotary + c * EPC;
#pragma unroll
    for (int e = 0; e < EPC; e += 4) {
      *reinterpret_cast<float4 *>(cs + e) = *reinterpret_cast<const float4 *>(row + e);
      *reinterpret_cast<float4 *>(sn + e) = *reinterpret_cast<const float4 *>(row + p.rotary / 2 + e);
    }
  }
#pragma unroll
  for (int u = 0; u < NH; ++u) {
    const int h = h0 + u * kRopeHeads;
    const bool is_q = h < p.num_heads;
    const bool is_k = !is_q && h < p.num_heads + p.num_kv_heads;
    const int hl = h - (is_q ? 0 : is_k ? p.num_heads : p.num_heads + p.num_kv_heads);
    if (h >= n_rows || (!is_q && !cached)) continue;
    const bool rotate = turns && (is_q || is_k);
    float f0[EPC], f1[EPC];
    if (rotate || (kFp8 && !is_q)) {
      Elem<T>::unpack(x0[u], f0);
      Elem<T>::unpack(x1[u], f1);
    }
    if (rotate) {
      if constexpr (kInterleaved) {
#pragma unroll
        for (int e = 0; e < EPC; e += 2) {   // chunk 0 holds pairs 0 .. EPC/2 - 1 of the item, chunk 1 the rest
          const float a0 = f0[e], b0 = f0[e + 1], a1 = f1[e], b1 = f1[e + 1];
          const float g0 = cs[e / 2], s0 = sn[e / 2], g1 = cs[EPC / 2 + e / 2], s1 = sn[EPC / 2 + e / 2];
          f0[e] = __fsub_rn(__fmul_rn(a0, g0), __fmul_rn(b0, s0));
          f0[e + 1] = __fadd_rn(__fmul_rn(b0, g0), __fmul_rn(a0, s0));
          f1[e] = __fsub_rn(__fmul_rn(a1, g1), __fmul_rn(b1, s1));
          f1[e + 1] = __fadd_rn(__fmul_rn(b1, g1), __fmul_rn(a1, s1));
        }
      } else {
#pragma unroll
        for (int e = 0; e < EPC; ++e) {
          const float a = f0[e], b = f1[e];
          f0[e] = __fsub_rn(__fmul_rn(a, cs[e]), __fmul_rn(b, sn[e]));
          f1[e] = __fadd_rn(__fmul_rn(b, cs[e]), __fmul_rn(a, sn[e]));
        }
      }
    }
    if (kFp8 && !is_q) {
      const E4m3Scale scale = is_k ? p.k_scale : p.v_scale;
      uint2 *dst = reinterpret_cast<uint2 *>(is_k ? p.k_cache : p.v_cache) +
                   (slot * p.num_kv_heads + hl) * kChunksPerRow;
      const uint2 y0 = pack_e4m3(f0, scale), y1 = pack_e4m3(f1, scale);
      if (c1 == c0 + 1 && (kInterleaved || !turns)) {   // c0 is even: 16 bytes at once
        *reinterpret_cast<uint4 *>(dst + c0) = make_uint4(y0.x, y0.y, y1.x, y1.y);
      } else {
        dst[c0] = y0;
        dst[c1] = y1;
      }
      continue;
    }
    if (rotate) {
      x0[u] = pack_chunk<T>(f0);
      x1[u] = pack_chunk<T>(f1);
    }
    uint4 *dst = is_q ? reinterpret_cast<uint4 *>(static_cast<T *>(p.q_out) + tok * p.q_out_stride) + hl * kChunksPerRow
                      : reinterpret_cast<uint4 *>(is_k ? p.k_cache : p.v_cache) +
                            (slot * p.num_kv_heads + hl) * kChunksPerRow;
    // Rows of a large batch are read and written with the streaming hint: 32.5 us against
    // 34.7 at 8192 tokens (97% of the copy bandwidth).  A small batch's stay in L2 for the attention.
    if (NH > 1) {
      __stcs(dst + c0, x0[u]);
      __stcs(dst + c1, x1[u]);
    } else {
      dst[c0] = x0[u];
      dst[c1] = x1[u];
    }
  }
}

}  // namespace pa

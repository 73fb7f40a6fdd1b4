// pa_shared_prefix.cuh -- decode attention of a group of sequences to the prefix
// they share, once for all of them, on the 5th-generation tensor cores.
// Included only from pa.cu.
//
// Sequences s0 .. s1-1 of a group have the same first `prefix` tokens (the same
// blocks in their tables).  Their rows -- (s1 - s0) sequences times the G query
// heads of a KV head -- all meet the same K and V, so the products are those of
// one matrix: S = Q K^T with a row for each (sequence, head), O = P V.  Each row
// keeps its own running maximum m and sum l (base 2); a partition of the prefix
// leaves (m, l, o) of every row in the workspace.  The walk over the sequences' own
// tokens (pa_decode.cuh, kWalkSuffix) combines them with its own, or, where some
// suffix is longer than a partition, pa_join_shared_kernel does.  Read once
// instead of (s1 - s0) times, the prefix costs 4 flops per row, token and head_dim
// element against 512 bytes a token.
//
// One CTA: a KV head, a partition of the prefix, up to 256 rows.  Two softmax
// warpgroups w = 0, 1 (thread = row) each own a 128-row tile of S and O in tensor
// memory (256 columns each).  With more than 128 rows ("pair"), they hold
// different rows and share every K/V tile; with at most 128 ("split"), they
// hold the same rows, tile w of every two, and leave a partial each.  K/V tiles are 128
// tokens (eight blocks), 32 KiB: a product is M=128 N=128 K=16 throughout, the
// widest form whose S (128 columns) and O (128 columns) fit twice.
// Warps (384 threads):
//   0-3, 4-7  softmax: tcgen05.ld of the row's 128 scores, maximum, O rescaled only
//             when a row's maximum grows by more than 2^8, exponentials, P written
//             over S, 32 scores' place at a time, as two parts in the cache's type (the
//             weight cut to its upper bits, and what they leave, rounded), so that V needs
//             no conversion and has no range limit and no weight is rounded to 16 bits:
//             twice the P V products, 5 us of 52 below; handed over in two halves of 64
//             tokens;
//   8, 9      tensor-core issue for w = 0, 1 (one thread each);
//   10, 11    TMA: pair: warp 10 fills one ring of 5 stages for both; split: warp 10 + w
//             fills w's own ring of 3.  Items alternate K(i), V(i): S has one
//             buffer, so QK(i+1) follows PV(i) and consumption alternates too.
// Barriers, per w: s_full (commit of QK(i)), p_half, p_full (4 warps each), o_done
// (commit of PV(i)); per stage: full, free (one arrival a consumer).  Each is
// waited on phase by phase by one role before that role enables the next phase,
// so parities never alias: QK(i+1) waits for o_done(i) (PV(i) reads P from S's
// columns), which needs p_full(i), which needs s_full(i) seen.  O may be
// rescaled once s_full(i) is seen, since QK(i) was issued after o_done(i-1).
// Every wait is bounded; a role that gives up raises the CTA's abort flag.
//
// Measured (64 sequences x 4 heads x 8 KV heads, 32768 tokens, bf16): 52 us, 656 TFLOP/s, 41% of
// the measured bf16 peak; prefix read at 2.6 TB/s.  A step of two tiles takes about 5400
// cycles, its products 3072 (48 of 64 cycles each).  The rest is each warpgroup's
// chain QK -> softmax (2300) -> PV -> QK: S has one buffer, since 512 columns hold no more.
// Without exponentials and low parts a step still takes 4300.  Set-up, the first
// tiles' latency and the epilogue take 8.5 us a CTA, most of it for short prefixes.
#pragma once

#include "pa_common.cuh"
#include "pa_decode.cuh"
#include "pa_prefill.cuh"
#include "pa_tcgen05.cuh"

namespace pa {

constexpr int kPrefixThreads = 384;
constexpr int kPrefixMmaWarp = 8;
constexpr int kPrefixLoadWarp = 10;
constexpr int kPrefixStagesPair = 5;      // one ring
constexpr int kPrefixStagesSplit = 3;     // each of two rings

// Which part of the batch's work CTA blockIdx.x has.  The items of a group, ((256 rows) x KV
// head) x partition with the partitions of the same rows side by side, follow those of
// the groups before it; groups without a prefix have none, so that idle CTAs come last.
// By whole warps.
struct PrefixItem {
  int s0, s1, prefix, part_tiles, row_cta, head, part;
  bool some;   // false: past the last item
};

template <int G>
__device__ __forceinline__ PrefixItem prefix_item(const SuffixParams &p) {
  PrefixItem r{};
  if (p.num_groups == 1) {   // the longest prefix's partitions, as the grid has them
    const int parts = p.slot0 / 2, rows = blockIdx.x / parts;
    r.part = blockIdx.x % parts;
    r.head = rows % p.num_kv_heads;
    r.row_cta = rows / p.num_kv_heads;
    r.part_tiles = p.part_tiles[0];
    const PrefixGroup e = prefix_group(p, 0);
    if (!e.ok && blockIdx.x == 0 && threadIdx.x == 0) record_error(8 /*PA_DEV_BAD_GROUP*/, 0);
    r.s0 = e.s0;
    r.s1 = e.s1;
    r.prefix = e.prefix;
    r.some = e.ok && r.row_cta * 2 * kPrefixRows < (e.s1 - e.s0) * G && r.part * r.part_tiles < e.tiles();
    return r;
  }
  const int lane = threadIdx.x & 31;
  PrefixGroup e = lane_group(p, 0);
  r.part_tiles = part_tiles_for(
      p, p.num_groups > 32 ? prefix_work<G>(p)
                           : __reduce_add_sync(kFullMask, static_cast<unsigned>(e.row_ctas<G>()) * e.tiles()));
  int at = blockIdx.x;   // counted from the items of these 32 groups
  for (int i0 = 0;;) {
    if (!e.ok && blockIdx.x == 0 && threadIdx.x < 32) record_error(8 /*PA_DEV_BAD_GROUP*/, e.index);
    const int row_ctas = e.row_ctas<G>();
    const int parts = e.ok ? (e.tiles() + r.part_tiles - 1) / r.part_tiles : 0;
    const int items = row_ctas * p.num_kv_heads * parts;
    int upto = items;   // of lanes 0 .. lane
    for (int off = 1; off < 32 && off < p.num_groups; off <<= 1) {
      const int y = __shfl_up_sync(kFullMask, upto, off);
      if (lane >= off) upto += y;
    }
    const unsigned here = __ballot_sync(kFullMask, at < upto);
    if (here != 0u && !r.some) {   // the first such lane's group has item `at`
      const int src = __ffs(here) - 1;
      const int k = __shfl_sync(kFullMask, at - (upto - items), src);
      const int n = __shfl_sync(kFullMask, parts, src);
      r.s0 = __shfl_sync(kFullMask, e.s0, src);
      r.s1 = __shfl_sync(kFullMask, e.s1, src);
      r.prefix = __shfl_sync(kFullMask, e.prefix, src);
      const int rows = k / max(n, 1);
      r.part = k % max(n, 1);
      r.head = rows % p.num_kv_heads;
      r.row_cta = rows / p.num_kv_heads;
      // (not so only where overlapping groups, which are reported, have more items than 32 bits count)
      r.some = k >= 0 && n > 0 && r.row_cta < __shfl_sync(kFullMask, row_ctas, src);
    }
    // CTA 0 looks at every group, to report bad ones
    if ((i0 += 32) >= p.num_groups || (r.some && blockIdx.x != 0)) return r;
    at -= __shfl_sync(kFullMask, upto, 31);
    e = lane_group(p, i0);
  }
}

struct PrefixSmem {
  static constexpr int kTile = 128 * 256;                  // [2 halves][128 rows][128 B]
  static constexpr int kHalf = 128 * 128;
  static constexpr int kTiles = 7;                         // pair: 2 Q + 5 stages; split: 1 Q + 2 x 3 stages
  static constexpr int kBar = kTiles * kTile;
  // full[6], free[6]; per w: s_full, p_half, p_full, o_done; drain; turn[2]
  static constexpr int kNumBars = 12 + 8 + 3;
  static constexpr int kTmemSlot = kBar + 8 * kNumBars;
  static constexpr int kFlag = kTmemSlot + 4;
  static constexpr int kBytes = kFlag + 4;
  static constexpr int kAlloc = kBytes + 1024;             // + alignment of the base to 1024 B (swizzle atoms)
};
static_assert(PrefixSmem::kAlloc <= 227 * 1024, "shared memory exceeds the per-CTA limit");
static_assert(2 * kPrefixRows * 512 <= PrefixSmem::kBar, "staged rows");
static_assert(2 + kPrefixStagesPair <= PrefixSmem::kTiles && 1 + 2 * kPrefixStagesSplit <= PrefixSmem::kTiles, "tiles");

// Bounded wait of the hand-overs between roles.  The timer is first read after 32
// polls (reading %globaltimer costs hundreds of cycles, which a wait that is about to
// end must not pay), and out of line: every wait's code counts (see the kernel).
// The start of the wait (t0, 0 at first), or 0 once it has to end.
__device__ __noinline__ unsigned long long wait_goes_on(unsigned long long t0, const volatile int *abort_flag,
                                                        int stall_cta) {
  const unsigned long long now = global_ns();
  if (t0 == 0) t0 = now;
  return *abort_flag || now - t0 > wait_limit_for(stall_cta, blockIdx.x) ? 0 : t0;
}

__device__ __forceinline__ bool role_wait(uint64_t *bar, uint32_t parity, const volatile int *abort_flag,
                                          int stall_cta) {
  unsigned long long t0 = 0;
  for (uint32_t it = 1; !mbar_try_wait(bar, parity); ++it) {
    if ((it & 31u) == 0) {
      t0 = wait_goes_on(t0, abort_flag, stall_cta);
      if (t0 == 0) return false;
    }
  }
  return true;
}

// A wait ran out: recorded, and the CTA's other roles are told.
__device__ __noinline__ void give_up(volatile int *abort_flag) {
  record_error(5 /*PA_DEV_WAIT_TIMEOUT*/, blockIdx.x);
  *abort_flag = 1;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}

// 16 consecutive 32-bit columns of this thread's lane from raw words.
__device__ __forceinline__ void tmem_st16u(uint32_t taddr, const uint32_t *v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
      "%15, %16};" ::"r"(taddr),
      "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]), "r"(v[9]),
      "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}

// AND of `pred` over the 256 softmax threads (named barrier 1).
__device__ __forceinline__ bool softmax_all(bool pred) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %1, 0;\n bar.red.and.pred p, 1, 256, p;\n selp.u32 %0, 1, 0, p;\n}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(pred))
      : "memory");
  return r != 0;
}

// Largest of N consecutive scores (N a multiple of 16).
template <int N>
__device__ __forceinline__ float row_max(const float *s) {
  float mx[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) mx[k] = fmaxf(s[k], s[8 + k]);
#pragma unroll
  for (int c = 16; c < N; c += 16)
#pragma unroll
    for (int k = 0; k < 8; ++k) mx[k] = max3(mx[k], s[c + k], s[c + 8 + k]);
  return max3(max3(mx[0], mx[1], mx[2]), max3(mx[3], mx[4], mx[5]), fmaxf(mx[6], mx[7]));
}

// Weights enter P V as hi + lo.  bf16: hi has the upper 8 of 24 bits, lo the next 8: off by
// less than 2^-15 of the weight.  fp16: 11 and 11 bits, 2^-20, as long as neither is
// subnormal (spaced 2^-24), and the largest row weights are 1 (up to 2^8 before a rescale).
// So fp16 weights are 2^7 times larger (2^15 at most, of 65504): what is lost of a small
// one is below 2^-24 of those units, 2^-31 of the row's largest weight.  The partial's
// maximum is stored 7 lower, which takes the factor out again.
template <typename T>
struct PrefixWeights;
template <>
struct PrefixWeights<__nv_bfloat16> {
  static constexpr float kBias = 0.f;
  static constexpr uint32_t kUpper = 0xffff0000u;   // the bits of fp32 that hi holds
  __device__ __forceinline__ static uint32_t pack_hi(uint32_t a, uint32_t b) { return __byte_perm(a, b, 0x7632); }
};
template <>
struct PrefixWeights<__half> {
  static constexpr float kBias = 7.f;
  static constexpr uint32_t kUpper = 0xffffe000u;
  __device__ __forceinline__ static uint32_t pack_hi(uint32_t a, uint32_t b) {   // exact but for subnormals
    return Pack16<__half>::pack(__uint_as_float(a & kUpper), __uint_as_float(b & kUpper));
  }
};

// P = 2^(s c2 + nmc) of the 32 scores in columns taddr .. taddr + 31, written over them: 16
// columns of pairs of upper parts, then 16 of lower ones.  Scores from `live` on
// count for nothing.  Adds the sums of even and odd columns to `sum`.
template <typename T>
__device__ __forceinline__ void exp_chunk(uint32_t taddr, int live, float2 cc2, float2 nmc, float2 &sum) {
  using W = PrefixWeights<T>;
  float s[32];
  tmem_ld32(taddr, s);
  if (live < 32) {
#pragma unroll
    for (int k = 0; k < 32; ++k) s[k] = k < live ? s[k] : -INFINITY;
  }
  uint32_t hi[16], lo[16];
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    const float2 x = __ffma2_rn(make_float2(s[2 * k], s[2 * k + 1]), cc2, nmc);
    const float2 e = make_float2(ex2(x.x), ex2(x.y));
    sum = __fadd2_rn(sum, e);
    const uint32_t ux = __float_as_uint(e.x), uy = __float_as_uint(e.y);
    hi[k] = W::pack_hi(ux, uy);
    lo[k] = Pack16<T>::pack(e.x - __uint_as_float(ux & W::kUpper), e.y - __uint_as_float(uy & W::kUpper));
  }
  tmem_st16u(taddr, hi);
  tmem_st16u(taddr + 16, lo);
}

template <typename T, int G>
__global__ void __launch_bounds__(kPrefixThreads, 1)
    pa_shared_prefix_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                            const SuffixParams p) {
  using SM = PrefixSmem;
  using PK = Pack16<T>;
  constexpr int D = 128;
  constexpr float kBias = PrefixWeights<T>::kBias;

  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + SM::kBar);
  uint64_t *free_ = full + 6;
  uint64_t *tile_bars = free_ + 6;   // w: s_full, p_half, p_full, o_done at 4 w
  uint64_t *drain = tile_bars + 8;
  uint64_t *turn = drain + 1;        // [w]: the PV of the other that w's next one follows is issued
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(smem + SM::kTmemSlot);
  volatile int *abort_s = reinterpret_cast<int *>(smem + SM::kFlag);

  const int tid = threadIdx.x;
  const int warp = tid >> 5;
  const int lane = tid & 31;
  const bool stall_here = p.stall_cta != 0 && static_cast<int>(blockIdx.x) == p.stall_cta - 1;
  if (warp == kPrefixLoadWarp && lane == 0) {
    prefetch_tensor_map(&tm_k);
    prefetch_tensor_map(&tm_v);
  }
  pdl_wait();
  pdl_trigger();

  const PrefixItem item = prefix_item<G>(p);
  if (!item.some) return;
  const int s0 = item.s0, s1 = item.s1, prefix = item.prefix;
  const int g = item.head, rc = item.row_cta, part = item.part;
  const int rows_group = (s1 - s0) * G;
  const int row0 = rc * 2 * kPrefixRows;
  const int part_tokens = item.part_tiles * kPrefixKv;
  const int tok0 = part * part_tokens;
  const int tokens = min(part_tokens, prefix - tok0);
  const int ntiles = (tokens + kPrefixKv - 1) / kPrefixKv;
  const int nblk = tokens / kBlockSize;
  const bool split = prefix_split(rows_group, rc);
  const int32_t *bt_row = p.block_tables + static_cast<size_t>(s0) * p.max_blocks_per_seq + tok0 / kBlockSize;
  // w's tiles: pair: 0 .. ntiles-1; split: w, w + 2, ...
  auto tiles_of = [&](int w) { return split ? (ntiles - w + 1) / 2 : ntiles; };
  // ring r: its first stage (barrier index, and tile of shared memory behind Q), and its length
  const int q_tiles = split ? 1 : 2;
  const int ring_len = split ? kPrefixStagesSplit : kPrefixStagesPair;
  auto ring_base = [&](int w) { return split ? w * kPrefixStagesSplit : 0; };
  auto stage_ptr = [&](int st) { return smem + (q_tiles + st) * SM::kTile; };

  if (warp == kPrefixLoadWarp && lane == 0) {
    for (int i = 0; i < 6; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&free_[i], split ? 1 : 2);   // one arrival per consuming issuer
    }
    for (int w = 0; w < 2; ++w) {
      uint64_t *tb = tile_bars + 4 * w;
      mbar_init(&tb[0], 1);   // s_full
      mbar_init(&tb[1], 4);   // p_half
      mbar_init(&tb[2], 4);   // p_full
      mbar_init(&tb[3], 1);   // o_done
    }
    mbar_init(drain, 2);
    mbar_init(&turn[0], 1);
    mbar_init(&turn[1], 1);

    fence_mbar_init();
    *abort_s = 0;
  }
  if (warp == kPrefixMmaWarp) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  // ---- the first 32 block ids (TMA warps), in flight while Q is put in place
  int my_id = static_cast<int>(p.num_blocks);   // past the end of the pool: the box reads zeros
  auto load_ids = [&](int grp) {
    const int lb = (grp << 5) + lane;
    my_id = static_cast<int>(p.num_blocks);
    if (lb < nblk) {
      const int v = bt_row[lb];
      if (v < 0 || v >= p.num_blocks) record_error(1 /*PA_DEV_BAD_BLOCK_ID*/, v);
      else my_id = v;
    }
  };
  if (warp >= kPrefixLoadWarp) load_ids(0);
  // the 16 boxes of an item: eight blocks (ids one a lane from `first`), two halves of their rows
  auto load_tile = [&](int st, const CUtensorMap *tm, int first) {
    uint8_t *dst = stage_ptr(st);
    if (lane == 0) mbar_arrive_expect_tx(&full[st], SM::kTile);
#pragma unroll 1
    for (int bi = 0; bi < 8; ++bi) {
      const int id = __shfl_sync(kFullMask, my_id, first + bi);
      if (lane == 0) {
        tma_load_5d(dst + bi * (kBlockSize * 128), tm, 0, 0, g, 0, id, &full[st]);
        tma_load_5d(dst + SM::kHalf + bi * (kBlockSize * 128), tm, 0, 1, g, 0, id, &full[st]);
      }
    }
  };
  // K tile 0 is on its way before Q is in place (this warp set the barriers up)
  if (warp == kPrefixLoadWarp && !stall_here) load_tile(0, &tm_k, 0);   // (test hook: left unissued)
  // ---- Q -> shared memory, K-major 128-byte swizzled: [d half][row][128 B]; warpgroup w its tile
  if (warp < kPrefixMmaWarp && (warp < 4 || !split)) {
    const int w = warp >> 2;
    uint8_t *q_s = smem + w * SM::kTile;
    const T *qg = reinterpret_cast<const T *>(p.q);
    const int c = tid & 15;
    uint4 x[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const int row = ((tid & 127) >> 4) + 8 * k;
      const int r = row0 + w * kPrefixRows + row;
      x[k] = make_uint4(0u, 0u, 0u, 0u);
      if (r < rows_group)
        x[k] = *reinterpret_cast<const uint4 *>(
            qg + (static_cast<size_t>(s0 + r / G) * p.num_heads + g * G + r % G) * D + c * 8);
    }
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const int row = ((tid & 127) >> 4) + 8 * k;
      *reinterpret_cast<uint4 *>(q_s + (c >> 3) * SM::kHalf + row * 128 + (((c & 7) ^ (row & 7)) << 4)) = x[k];
    }
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();   // barriers initialised, tensor memory allocated, Q in shared memory
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  int issued = 0;   // TMA warps: items taken (for the abort drain)
  if (warp >= kPrefixLoadWarp) {
    // ================================================================ TMA producers
    const int w = warp - kPrefixLoadWarp;
    if (w == 0 || split) {
      const int n = tiles_of(w);
      const int base = ring_base(w);
      int grp = 0;
      int st = 0, phase = 0;   // it % ring_len, it / ring_len & 1
      for (int it = 0; it < 2 * n; ++it) {   // item it: K (even) or V (odd) of this ring's tile it / 2
        if (it >= ring_len &&
            !__all_sync(kFullMask, role_wait(&free_[base + st], phase ^ 1, abort_s, p.stall_cta)))
          break;
        const int j = split ? 2 * (it >> 1) + w : it >> 1;
        if (((8 * j) >> 5) != grp) {
          grp = (8 * j) >> 5;
          load_ids(grp);
        }
        if (it > 0 || w > 0) load_tile(base + st, (it & 1) ? &tm_v : &tm_k, (8 * j) & 31);   // w = 0: K tile 0 above
        if (++st == ring_len) {
          st = 0;
          phase ^= 1;
        }
        issued = it + 1;
      }
    }
  } else if (warp >= kPrefixMmaWarp) {
    if (lane == 0) {
      // ================================================================ tensor-core issue for w
      const int w = warp - kPrefixMmaWarp;
      const int n = tiles_of(w);
      const int base = ring_base(w);
      uint64_t *tb = tile_bars + 4 * w;
      constexpr uint32_t kIdescQK = instr_desc_f16(PK::kFormat, false, kPrefixRows, kPrefixKv);
      constexpr uint32_t kIdescPV = instr_desc_f16(PK::kFormat, true, kPrefixRows, D);
      bool ok = true;
      auto wait = [&](uint64_t *bar, uint32_t parity) {
        if (!ok) return;
        ok = role_wait(bar, parity, abort_s, p.stall_cta);
        if (!ok) give_up(abort_s);
        tc_fence_after();
      };
      // an operand at byte offset `off` from a tile's base has the base's descriptor
      // with off / 16 added (the address field does not overflow: shared memory ends below 2^18)
      const uint64_t a0 = smem_desc_sw128(smem + (split ? 0 : w) * SM::kTile, 16, 1024);
      const uint64_t k_desc = smem_desc_sw128(stage_ptr(base), 16, 1024);
      const uint64_t v_desc = smem_desc_sw128(stage_ptr(base), SM::kHalf, 1024);
      const uint32_t s_tmem = tmem + w * 256, o_tmem = s_tmem + 128;
      // Stages and phases are counted along: a division by ring_len is a chain through the
      // exponent unit, behind the softmax's exponentials (several hundred cycles).
      int st = 0, phase = 0;
      auto next = [&]() {
        if (++st == ring_len) {
          st = 0;
          phase ^= 1;
        }
      };
      for (int i = 0; i < n && ok; ++i) {
        wait(&full[base + st], phase);
        if (i > 0) wait(&tb[3], (i - 1) & 1);   // PV(i-1) has read P from S's columns
        if (!ok) break;
        const uint64_t b0 = k_desc + ((st * SM::kTile) >> 4);
#pragma unroll 8
        for (int kk = 0; kk < D / 16; ++kk)
          umma_f16(s_tmem, a0 + (((kk >> 2) * SM::kHalf + (kk & 3) * 32) >> 4),
                   b0 + (((kk >> 2) * SM::kHalf + (kk & 3) * 32) >> 4), kIdescQK, kk > 0);
        umma_commit(&tb[0]);
        next();
        wait(&full[base + st], phase);
        if (i > 0 || w > 0) {   // PV_0(i) follows PV_1(i-1), PV_1(i) follows PV_0(i)
          const int before = w > 0 ? i : i - 1;
          if (before < tiles_of(1 - w)) wait(&turn[w], before & 1);
        }
        if (!ok) break;
        const uint64_t v0 = v_desc + ((st * SM::kTile) >> 4);
        next();
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          wait(&tb[1 + hf], i & 1);   // the half's P written
          if (!ok) break;
#pragma unroll
          for (int kk = 4 * hf; kk < 4 * hf + 4; ++kk) {   // 16 tokens = 8 columns of P a step
            const uint32_t p_tmem = s_tmem + 32 * (kk >> 1) + 8 * (kk & 1);   // 16 columns of P, 16 of its low parts
            umma_f16_ts(o_tmem, p_tmem, v0 + ((kk * 16 * 128) >> 4), kIdescPV, i > 0 || kk > 0);
            umma_f16_ts(o_tmem, p_tmem + 16, v0 + ((kk * 16 * 128) >> 4), kIdescPV, true);
          }
        }
        if (!ok) break;
        umma_commit(&tb[3]);
        mbar_arrive(&turn[1 - w]);
      }
    }
  } else if (warp < kPrefixMmaWarp) {
    // ================================================================ softmax warpgroup w
    const int w = warp >> 2;
    const int n = tiles_of(w);
    const int r = tid & 127;
    const uint32_t lane_base = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + w * 256 + lane_base;
    const uint32_t t_o = t_s + 128;
    uint64_t *tb = tile_bars + 4 * w;
    const float c2 = p.scale_log2;
    float m_run = -INFINITY;   // reference maximum of this row's raw scores
    float l_run = 0.f;         // sum of the weights, 2^((s - m_run) c2 + kBias)
    bool ok = true;
    auto wait = [&](uint64_t *bar, uint32_t parity) {
      if (!ok) return;
      ok = __all_sync(kFullMask, role_wait(bar, parity, abort_s, p.stall_cta));
      if (!ok && lane == 0) give_up(abort_s);
      tc_fence_after();
    };
    auto hand_over = [&](uint64_t *bar) {   // this warp's P is in tensor memory
      asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar);
    };
    const int base = ring_base(w);
    int st = 0;   // stage of the next item to free
    for (int i = 0; i < n && ok; ++i) {
      wait(&tb[0], i & 1);
      if (!ok) break;
      // QK(i) is complete, and so is PV(i-1), which it waited for: their stages are free
      if (i > 0) {
        if ((tid & 127) == 0) mbar_arrive(&free_[base + st]);   // item 2 i - 1
        st = st + 1 == ring_len ? 0 : st + 1;
      }
      if ((tid & 127) == 0) mbar_arrive(&free_[base + st]);     // item 2 i
      st = st + 1 == ring_len ? 0 : st + 1;
      const int live = tokens - (split ? 2 * i + w : i) * kPrefixKv;   // a multiple of 16
      float tmax;
      {
        float s[128];
        tmem_ld64(t_s, *reinterpret_cast<float (*)[64]>(s));
        tmem_ld64(t_s + 64, *reinterpret_cast<float (*)[64]>(s + 64));
        if (live < kPrefixKv) {
#pragma unroll
          for (int c = 0; c < 128; ++c) s[c] = c < live ? s[c] : -INFINITY;
        }
        tmax = row_max<128>(s);
      }
      // m_run, the reference of the exponentials, follows only a score that passes it by more than 2^8
      const bool need = i > 0 && (tmax - m_run) * c2 > kRescaleLog2;
      if (__any_sync(kFullMask, need)) {
        // O, complete up to tile i-1 (QK(i) was issued after PV(i-1)), follows
        const float f = need ? ex2((m_run - tmax) * c2) : 1.f;
        l_run *= f;
#pragma unroll 1
        for (int c = 0; c < D; c += 32) {
          float o[32];
          tmem_ld32(t_o + c, o);
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] *= f;
          tmem_st32(t_o + c, o);
        }
      }
      if (i == 0 || need) m_run = tmax;
      // The scores are read a second time, 32 a turn of a short loop: with all 128 in line the
      // kernel was 68 KB of instructions, which its roles (and the neighbouring SM's) evict
      // from the cache between them: 83.7 us a call against 75.2 (64 sequences x 32768 tokens).
      const float nm = fmaf(-m_run, c2, kBias);
      const float2 nmc = make_float2(nm, nm), cc2 = make_float2(c2, c2);
      float2 sum = make_float2(0.f, 0.f);
#pragma unroll 2
      for (int c = 0; c < 4; ++c) {
        exp_chunk<T>(t_s + 32 * c, live - 32 * c, cc2, nmc, sum);
        if (c & 1) hand_over(&tb[1 + (c >> 1)]);
      }
      l_run += sum.x + sum.y;
    }
    // ---- this warp's 32 rows of partials: m in base-2 units (less kBias), o and l relative to it.  In
    // the workspace they are consecutive, so o goes through shared memory (Q and the
    // K/V stages, free once both warpgroups' products are complete; 16-byte chunk c
    // of row r at c ^ (r & 31)) and out 512 consecutive bytes a warp store.  A thread
    // storing its own row, or one bulk copy a row, took 14000 and 8000 cycles.
    if (n > 0) wait(&tb[3], (n - 1) & 1);
    const int rw = row0 + (split ? 0 : w * kPrefixRows) + (r & ~31);   // the warp's first row
    const size_t at = prefix_slot(p, g, split ? 2 * part + w : part) + static_cast<size_t>(s0) * G + rw;
    if (ok && rw + lane < rows_group) {
      p.ws_m[at + lane] = n > 0 ? -fmaf(-m_run, c2, kBias) : -INFINITY;
      p.ws_l[at + lane] = l_run;
    }
    if (softmax_all(ok) && n > 0) {
      uint8_t *stage = smem + (warp * 32) * 512;
#pragma unroll 1
      for (int c = 0; c < D; c += 32) {
        float o[32];
        tmem_ld32(t_o + c, o);
#pragma unroll
        for (int k = 0; k < 32; k += 4)
          *reinterpret_cast<float4 *>(stage + lane * 512 + ((((c + k) >> 2) ^ lane) << 4)) =
              make_float4(o[k], o[k + 1], o[k + 2], o[k + 3]);
      }
      __syncwarp();
      float4 *dst = reinterpret_cast<float4 *>(p.ws_o) + at * (D / 4) + lane;
      const int rows = min(32, rows_group - rw);
#pragma unroll 8
      for (int k = 0; k < rows; ++k) dst[k * (D / 4)] = *reinterpret_cast<const float4 *>(stage + k * 512 + ((lane ^ k) << 4));
    }
    tc_fence_before();
  }

  // ---- all roles done: tensor-core operations, their barrier arrivals and (after an
  // abort) the copies in flight land before the memory is released, all bounded
  __syncthreads();
  if ((warp == kPrefixMmaWarp || warp == kPrefixMmaWarp + 1) && lane == 0) {
    umma_commit(drain);
    mbar_wait(drain, 0, wait_limit_for(p.stall_cta, blockIdx.x));
  }
  if (*abort_s && warp >= kPrefixLoadWarp && lane == 0) {
    // the last item issued into each stage (an earlier one's copy landed before its stage was reissued)
    const int w = warp - kPrefixLoadWarp;
    for (int it = max(0, issued - ring_len); it < issued; ++it)
      if (!(stall_here && it == 0 && w == 0)) mbar_wait(&full[ring_base(w) + it % ring_len], (it / ring_len) & 1,
                  wait_limit_for(p.stall_cta, blockIdx.x));
  }
  __syncthreads();
  if (warp == kPrefixMmaWarp) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Join of a row's prefix partials (slots 0 ..) and those of its own tokens (slot0 ..):
// only where the own tokens are more than one partition (else the suffix walk does it).
template <typename T, int G>
__global__ void __launch_bounds__(kReduceWarps * 32) pa_join_shared_kernel(const SuffixParams p) {
  pdl_wait();
  pdl_trigger();
  const long long rows = static_cast<long long>(p.num_seqs) * p.num_heads;
  const long long step = static_cast<long long>(gridDim.x) * kReduceWarps;
  const int part_tiles = p.slot0 > 0 ? part_tiles_for(p, prefix_work<G>(p)) : 1;
  for (long long row = static_cast<long long>(blockIdx.x) * kReduceWarps + (threadIdx.x >> 5); row < rows; row += step) {
    const int b = static_cast<int>(row / p.num_heads);
    const int h = static_cast<int>(row % p.num_heads);
    const int L = p.context_lens[b];
    const PrefixGroup group = group_of(p, b);
    if (!group.ok || L < group.prefix || L - group.prefix > p.max_context_len || L > p.max_blocks_per_seq * kBlockSize)
      continue;   // recorded by the partition kernel; the row is left as it was
    join_row<T>(p, row, prefix_slot(p, h / G, 0) + static_cast<size_t>(b) * G + h % G,
                static_cast<size_t>(p.num_seqs) * G, prefix_partials<G>(group, part_tiles, b, h % G), p.slot0,
                (L - group.prefix + p.partition_size - 1) / p.partition_size);
  }
}

}  // namespace pa

// hq_kv4_tree.cu -- attention of trees of drafted tokens over the 4-bit window
// cache with many query rows a KV head (include/hq_kv4.h; few rows, and short batches,
// go to hq_kv4_attn.cu, whose codes stay in registers).
//
// The formulas are those of hq_kv4_attn.cu: with q' = H D q / sqrt(128), z = q' . (c - 7.5)
// s_k, and the output's transform behind the sum of p s_v (c - 7.5).  A tile is 128
// rows (drafts x heads of the group) of one KV head.  A block streams its tokens 128 at a
// time: four warps unpack the codes to centred fp16 values in shared memory, exact, where
// the tensor cores take them as K and as V; the queries and the weights are two fp16
// parts each (weights one where the output is of 16 bits), products of their own into one sum:
//   S = (q' hi + q' lo) (c - 7.5)^T         queries and sums in tensor memory
//   z = S s_k, m, p = 2^(z - m), w = p s_v f   a row's 128 tokens by two threads; w's parts in S's place
//   O += (w hi + w lo) (c - 7.5)
// S has two places, so that the next tokens' scores are formed beside this block's
// softmax.  The queries are in tensor memory because shared memory is what all sides
// want: as an operand from there they take its whole rate while their products run, and the
// codes, scales and barriers of the other warps wait.
//
// 16 ragged sequences of up to 8192 tokens x 8 heads, 256 rows a head: 199 us, of which the products
// at the measured bf16 rate would take 50, and those of both parts of the queries 75.  128 tokens take
// 2600 cycles: unpacking 2500 (32 words of codes a thread, 10 instructions and 16 stored bytes each),
// softmax 2000, products 1600, all beside one another.  One sequence of 131072 tokens, 128 rows: 103 us, 9 of
// them the join.  Capped scores, 16 x 8192 tokens of 256 rows: 300 us while they stay below the cap, 430 where many pass it.
#include <cuda_runtime.h>

#include <cmath>

#include "hq_kv4.h"
#include "hq_kv4_walk.cuh"
#include "hq_launch.cuh"
#include "hq_umma.cuh"

namespace hq {

namespace {

constexpr int kRows = 128, kTokens = 128, kBlockUnits = kTokens / kUnit;
constexpr int kThreads = 512;                    // two threads a row, four warps to unpack, products (one warp)
constexpr int kUnpackThreads = 128, kPasses = 4 * kTokens / kUnpackThreads;    // 16 bytes of codes a thread and pass
constexpr int kLaunchRegs = 128, kRowRegs = 176, kUnpackRegs = 96, kOtherRegs = 64;
static_assert(2 * kRowRegs + kUnpackRegs + kOtherRegs <= 4 * kLaunchRegs, "no more than the block was launched with");
constexpr int kTileBytes = kRows * kTile * 2, kHalfBytes = kTileBytes / 2;      // 128 x 128 fp16, two halves of 64 columns
// Units that beginning and ending a segment takes as long as (13 us; 128 tokens take 1.3).  16 / 32 / 48 / 64 / 96:
// 16 ragged sequences of 8192, 256 rows 208 / 206 / 205 / 204 / 202 us (before the codes were read ahead, now 199); 64 of 2000, 64 rows 165 / 162 / 159 / 155 /
// 155; 24 very ragged of 4093, 64 rows 104 / 88 / 82 / 80 / 79; 16 of 1000, 128 rows 53 / 52 / 50 / 49 / 46.
constexpr int kSegmentCost = 96;
constexpr int kMaxBlocks = 160;                  // of a launch
constexpr int kScaleSlots = 4;                   // blocks of tokens whose scales are kept
// K's scales, below 2^122 as those of rows whose transform is finite, are brought down by this and a row's multiplier
// up, so that a product, below 2^16, times a scale stays within fp32.  (Scales below 2^-116 lose 2^-150 of 2^-10, a score
// less than 2^-23: |scale| |q| is below 2^110.)
constexpr float kKeyScale = 0x1p-10f;
constexpr int kSeenWords = HQ_KV4_MAX_DRAFTS / 32, kSeenRow = kSeenWords + 1;   // a word apart: no bank twice
constexpr uint32_t kIdesc = umma_idesc_f16(kRows, kTokens);
constexpr uint32_t kTmemS = 0, kTmemO = 256, kTmemQ = 384;       // columns: S twice, O, q' hi and lo

// Shared memory: K and V of even blocks of tokens, K and V of odd ones, and 64 KB through which
// query rows come in (64 at a time, with the transforms' tables behind them), then the codes
// of three blocks of tokens as they are in the pool, and at a segment's end its sums go
// out (then the tables lie in K and V).
constexpr int kRawStages = 3, kRawBytes = kBlockUnits * kUnitBytes;
static_assert(kRawStages * kRawBytes <= 2 * kTileBytes, "the codes fit");
struct Small {
  float sk[kScaleSlots][kTokens], sv[kScaleSlots][kTokens];
  float4 sv_top[kScaleSlots], sv_low[kScaleSlots];         // the largest and the least sv of 32 tokens each, of those that are there
  uint32_t valid[kScaleSlots];                   // units that have a page and belong to the segment
  uint32_t raw_valid[kRawStages];                // likewise, of the codes in the ring
  RowStat stat[kRows];
  float l[2][kRows];                             // sums of weights of a row's two threads
  float top[2][2][kRows], low[2][kRows];         // what these tell one another
  float mul[kRows];                              // multiplier of a row's scores
  uint32_t seen[kRows * kSeenRow];               // drafts that a row sees
  int parent[HQ_KV4_MAX_DRAFTS];
  uint32_t there[kSeenWords];
  Walk walk;                                     // over the block's piece, step by step
  int64_t piece;                                 // its length
  int more, b, pair, u_lo, u_hi, nu;             // the segment that it is at
  int len;                                       // tokens up to the last draft
  uint64_t k_full[2], k_empty[2], v_full[2], v_empty[2], s_full[2], p_full[2], o_full, o_empty, q_full, ready;
  uint64_t raw_full[kRawStages], raw_empty[kRawStages];
  uint32_t tmem;
  int abort;
};
constexpr int kSmem = 6 * kTileBytes + 1024 + (int)sizeof(Small);
static_assert(kSmem + 2048 <= 227 * 1024, "shared memory of a block, find_piece's beside it");
static_assert(kTileBytes + 8 * 4 * kTrTile * 4 <= 2 * kTileBytes, "64 rows of queries and the transforms' tables fit 64 KB");

__device__ __forceinline__ void rows_sync() { asm volatile("bar.sync 1, 256;" ::: "memory"); }
// The two warps that have the same rows.
__device__ __forceinline__ void pair_sync(int warp) { asm volatile("bar.sync %0, 64;" ::"r"(2 + (warp & 3)) : "memory"); }

__device__ __forceinline__ uint32_t centred(uint32_t c, uint32_t factor) {
  uint32_t y;                                    // -7.5 2^-9 twice
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(y) : "r"(c), "r"(factor), "r"(0xA380A380u));
  return y;
}
// 8 codes to centred fp16 values in units of 2^-9, exact: the bits of a code, or of 16 codes, are a
// subnormal number of units 2^-24.  Order: codes 0, 4, 1, 5, 2, 6, 3, 7.
__device__ __forceinline__ uint4 unpack_word(uint32_t x) {
  const uint32_t y = x >> 8;
  return make_uint4(centred(x & 0x000F000Fu, 0x78007800u), centred(x & 0x00F000F0u, 0x68006800u),
                    centred(y & 0x000F000Fu, 0x78007800u), centred(y & 0x00F000F0u, 0x68006800u));
}
// Where the 8 values of group g (of 16) of row r lie in a tile: 128-byte swizzle.
__device__ __forceinline__ uint32_t chunk_at(int r, int g) {
  return (uint32_t)((g >> 3) * kHalfBytes + r * 128 + (((g & 7) ^ (r & 7)) * 16));
}
__device__ __forceinline__ void st16(uint32_t at, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint4 ld16(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ void swap_if(bool c, uint32_t &a, uint32_t &b) {
  const uint32_t x = c ? b : a;
  b = c ? a : b;
  a = x;
}
// (x0, x1) = hi + lo as fp16 pairs, hi with 11 of their bits: x misses hi + lo by 2^-22 of it and
// 2^-25, which is up to 2^-31 of a row's largest weight times the largest of V's scales, as f holds that at 2^6 and more.
__device__ __forceinline__ void split_cut(float x0, float x1, uint32_t &hi, uint32_t &lo) {
  const float h0 = __uint_as_float(__float_as_uint(x0) & 0xFFFFE000u), h1 = __uint_as_float(__float_as_uint(x1) & 0xFFFFE000u);
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(h1), "f"(h0));
  float l0, l1;
  upk2(sub2(pk2(x0, x1), pk2(h0, h1)), l0, l1);
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(lo) : "f"(l1), "f"(l0));
}

// SPLIT: weights in two parts, for fp32 outputs; else rounded once to fp16, by at most 2^-11 of them and the same 2^-25.
template <bool CAP, bool SPLIT>
__global__ void __launch_bounds__(kThreads, 1) kv4_tree_kernel(Kv4AttnArgs a) {
  extern __shared__ unsigned char s_raw[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t raw = smem_addr(s_raw), base = (raw + 1023u) & ~1023u;
  const uint32_t kv_at = base, stage_at = base + 4 * kTileBytes;
  Small &S = *reinterpret_cast<Small *>(s_raw + (base - raw) + 6 * kTileBytes);
  volatile int *const abort = &S.abort;
  if (warp == 12) tmem_alloc(&S.tmem, 512);
  if (tid == 0) {
    S.abort = 0;
    for (int i = 0; i < 2; ++i) {
      mbar_init(&S.k_full[i], kUnpackThreads / 32);
      mbar_init(&S.k_empty[i], 1);
      mbar_init(&S.v_full[i], kUnpackThreads / 32);
      mbar_init(&S.v_empty[i], 1);
      mbar_init(&S.s_full[i], 1);
      mbar_init(&S.p_full[i], 8);
    }
    for (int i = 0; i < kRawStages; ++i) {
      mbar_init(&S.raw_full[i], 1);
      mbar_init(&S.raw_empty[i], kUnpackThreads / 32);
    }
    mbar_init(&S.o_full, 1);
    mbar_init(&S.o_empty, 8);
    mbar_init(&S.q_full, 8);
    mbar_init(&S.ready, 8);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  follow_launch();
  const uint32_t tmem = S.tmem;
  const Piece piece = find_piece<true, kThreads / 32, kSegmentCost>(a);
  if (tid == 0) {
    S.walk = Walk{piece.begin, piece.end, piece.b_begin, piece.b};
    S.piece = piece.size;
  }
  uint32_t segments = 0;
  if (warp >= 12) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kOtherRegs));
    if (warp == 12) {
      // -------------------------------------------------------------- products
      const bool leader = elect_one();
      uint32_t k_count[2] = {0, 0}, p_count[2] = {0, 0};
      const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0), kv_u = __shfl_sync(0xffffffffu, kv_at, 0);
      const auto scores = [&](int s) {
        wait(&S.k_full[s], k_count[s]++, abort);
        tc_fence_after();
        const uint64_t k = umma_desc_sw128(kv_u + s * 2 * kTileBytes, 16);
        if (leader) {
          fence_async_smem();                    // the writers' stores, in order before this by the barrier, to the tensor cores
#pragma unroll 1
          for (int part = 0; part < 2; ++part)   // the high parts, the low ones
#pragma unroll
            for (int e = 0; e < 8; ++e)
              umma_f16_ts(tm + kTmemS + s * 128, tm + kTmemQ + part * 64 + 8 * e,
                          k + (((e >> 2) * kHalfBytes + (e & 3) * 32) >> 4), kIdesc, part + e > 0);
          umma_commit(&S.s_full[s]);
          umma_commit(&S.k_empty[s]);
        }
      };
      while (true) {
        wait(&S.q_full, segments, abort);
        if (__shfl_sync(0xffffffffu, S.more, 0) == 0) break;
        const int n = __shfl_sync(0xffffffffu, (S.u_hi - S.u_lo + kBlockUnits - 1) / kBlockUnits, 0);
        tc_fence_after();
        scores(0);
        wait(&S.o_empty, segments + 1, abort);
        ++segments;
        for (int k = 0; k < n; ++k) {
          const int s = k & 1;
          if (k + 1 < n) scores(s ^ 1);          // in the place of weights whose product is asked for
          wait(&S.v_full[s], p_count[s], abort);
          wait(&S.p_full[s], p_count[s]++, abort);
          tc_fence_after();
          const uint64_t v = umma_desc_sw128(kv_u + (2 * s + 1) * kTileBytes, kHalfBytes);
          if (leader) {
            fence_async_smem();
#pragma unroll 1
            for (int part = 0; part < (SPLIT ? 2 : 1); ++part)     // the low parts 16 columns behind the high ones of 32 tokens
#pragma unroll
              for (int e = 0; e < 8; ++e)
                umma_f16_ts(tm + kTmemO, tm + kTmemS + s * 128 + 32 * (e >> 1) + 8 * (e & 1) + 16 * part,
                            v + ((e * 2048) >> 4), kIdesc | kUmmaBMnMajor, k > 0 || part + e > 0);
            umma_commit(&S.v_empty[s]);
            if (k + 1 == n) umma_commit(&S.o_full);
          }
        }
      }
      if (*abort) {                              // products in flight end before the block does
        if (leader) umma_commit(&S.o_full);
        for (uint32_t p = 0; p < 2; ++p) mbar_wait(&S.o_full, p, 1u << 16);
      }
    }
    if (warp == 13) {
      // -------------------------------------------------------------- pages
      // A lane a unit of a block of tokens: page numbers a block ahead, codes and scales as they are into the ring.
      uint32_t turn = 0;
      const int unit_shift = a.c.page_shift < 0 ? -1 : a.c.page_shift - 4;
      const uint32_t per_page = (uint32_t)a.c.page_units;
      int stage = 0;
      while (true) {
        wait(&S.ready, segments, abort);
        if (S.more == 0) break;
        const int u_lo = S.u_lo, b = S.b, h = S.pair / a.row_tiles, u_end = min(S.u_hi, (S.len + kUnit - 1) / kUnit);
        const int n = (S.u_hi - u_lo + kBlockUnits - 1) / kBlockUnits;
        const int32_t *const table = a.c.table + (int64_t)b * a.c.width;
        const auto in_page = [&](int u) { return unit_shift >= 0 ? (uint32_t)u >> unit_shift : (uint32_t)u / per_page; };
        const auto ask = [&](int u) { return lane < kBlockUnits && u < u_end ? table[in_page(u)] : -1; };
        int u = u_lo + lane, page = ask(u);
        bool bad = false;
        wait(&S.q_full, segments, abort);        // the queries are through what becomes the ring
        fence_async_smem();
        for (int k = 0; k < n; ++k, u += kBlockUnits) {
          const int next = ask(u + kBlockUnits);
          const bool in = lane < kBlockUnits && u < u_end, good = in && page >= 0 && page < a.c.n_pages;
          bad = bad || in != good;
          const uint32_t valid = __ballot_sync(0xffffffffu, good);
          wait(&S.raw_empty[stage], turn + 1, abort);
          if (lane == 0) {
            S.raw_valid[stage] = valid;
            mbar_expect(&S.raw_full[stage], __popc(valid) * kUnitBytes);
          }
          __syncwarp();
          if (good) {
            const uint32_t pool = (uint32_t)((page * a.c.n_kv + h) * per_page + u - in_page(u) * per_page);
            asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                             stage_at + stage * kRawBytes + lane * kUnitBytes),
                         "l"(a.c.pages + (uint64_t)pool * kUnitBytes), "n"(kUnitBytes), "r"(smem_addr(&S.raw_full[stage]))
                         : "memory");
          }
          page = next;
          if (++stage == kRawStages) {
            stage = 0;
            ++turn;
          }
        }
        if (bad) atomicOr(a.status, (uint32_t)HQ_ERR_PAGE);
        ++segments;
      }
      if (*abort) {                              // copies in flight end before the block does
        for (int i = 0; i < kRawStages; ++i)
          for (uint32_t p = 0; p < 2; ++p) mbar_wait(&S.raw_full[i], p, 1u << 16);
      }
    }
  } else if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kUnpackRegs));
    // ---------------------------------------------------------------- codes
    const int t = tid - 256;                     // 0 .. 127
    uint32_t count[2] = {0, 0}, turn = 0;
    int stage = 0;
    // K: 16 bytes are 32 dimensions of a token, four lanes a token; V: 16 dimensions of two tokens.  Half of the lanes
    // store their words in another order, so that 8 lanes meet all banks.
    const bool k_upper = (t & 2) != 0, v_upper = (t & 4) != 0;
    uint32_t k_to[4], v_to[4];                   // where a pass's words go, the rows of the first pass
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      k_to[e] = kv_at + chunk_at(t >> 2, 4 * (t & 3) + (e ^ (k_upper ? 2 : 0)));
      v_to[e] = kv_at + kTileBytes + chunk_at(16 * (t >> 6) + 2 * ((t & 63) >> 3) + (e >> 1), 2 * (t & 7) + ((e & 1) ^ (v_upper ? 1 : 0)));
    }
    constexpr uint32_t kPassRows = kTokens / kPasses * 128, kPassUnits = kBlockUnits / kPasses * kUnitBytes;
    static_assert(kTokens / kPasses % 8 == 0, "a pass's rows are swizzled alike");
    while (true) {
      wait(&S.ready, segments, abort);           // the segment and the drafts' masks are there, the sums before are out
      if (S.more == 0) break;
      const int u_lo = S.u_lo, n = (S.u_hi - u_lo + kBlockUnits - 1) / kBlockUnits, len = S.len;
      bool bad_len;
      const int committed = kv4_length(a.c, a.lengths, S.b, &bad_len);
      for (int k = 0; k < n; ++k) {
        const int s = k & 1, slot = k & (kScaleSlots - 1);
        const uint32_t set = s * 2 * kTileBytes, raw_at = stage_at + stage * kRawBytes;
        const uint32_t codes = raw_at + (t >> 6) * kUnitBytes + (t & 63) * 16;
        wait(&S.raw_full[stage], turn, abort);
        uint4 v[kPasses];                        // all on their way before the first is unpacked, and while the tile is in use
#pragma unroll
        for (int p = 0; p < kPasses; ++p) v[p] = ld16(codes + p * kPassUnits);
        const uint16_t *const sc =
            reinterpret_cast<const uint16_t *>(s_raw + (raw_at - raw) + (t >> 4) * kUnitBytes + kUnitKs) + (t & 15);
        const uint32_t valid = S.raw_valid[stage], sk_bits = sc[0], sv_bits = sc[16];
        wait(&S.k_empty[s], count[s] + 1, abort);
#pragma unroll
        for (int p = 0; p < kPasses; ++p) {
          uint32_t w[4] = {v[p].x, v[p].y, v[p].z, v[p].w};
          swap_if(k_upper, w[0], w[2]);
          swap_if(k_upper, w[1], w[3]);
#pragma unroll
          for (int e = 0; e < 4; ++e) st16(k_to[e] + set + p * kPassRows, unpack_word(w[e]));
        }
#pragma unroll
        for (int p = 0; p < kPasses; ++p) v[p] = ld16(codes + p * kPassUnits + kUnitV);
        {
          const int token = (u_lo + kBlockUnits * k) * kUnit + t, draft = token - committed;
          bool none = token >= len || !((valid >> (t >> 4)) & 1u);
          // what lies in the place of padding, or of a draft behind padding, may be no scale: those of rows that a row sees
          // are not negative, and finite.  A finite one is no matter, as its weights are 0
          if (!none && draft >= 0) none = !((S.there[draft >> 5] >> (draft & 31)) & 1u) || sv_bits >= 0x7F80u;
          const float sv = none ? 0.0f : bf16_to_f32((uint16_t)sv_bits);
          S.sk[slot][t] = none ? 0.0f : __fmul_rn(bf16_to_f32((uint16_t)sk_bits), kKeyScale);
          S.sv[slot][t] = sv;
          // bits of nonnegative floats order as they do
          const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(sv));
          const uint32_t low = __reduce_min_sync(0xffffffffu, none ? 0x7F800000u : __float_as_uint(sv));
          if (lane == 0) {
            reinterpret_cast<float *>(&S.sv_top[slot])[warp & 3] = __uint_as_float(top);
            reinterpret_cast<float *>(&S.sv_low[slot])[warp & 3] = __uint_as_float(low);
          }
          if (t == 0) S.valid[slot] = valid;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.k_full[s]);
        wait(&S.v_empty[s], count[s] + 1, abort);
        ++count[s];
#pragma unroll
        for (int p = 0; p < kPasses; ++p) {
          uint32_t w[4] = {v[p].x, v[p].y, v[p].z, v[p].w};
          swap_if(v_upper, w[0], w[1]);
          swap_if(v_upper, w[2], w[3]);
#pragma unroll
          for (int e = 0; e < 4; ++e) st16(v_to[e] + set + p * kPassRows, unpack_word(w[e]));
        }
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&S.v_full[s]);
          mbar_arrive(&S.raw_empty[stage]);
        }
        if (++stage == kRawStages) {
          stage = 0;
          ++turn;
        }
      }
      ++segments;
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRowRegs));
    // ---------------------------------------------------------------- rows
    const int half = warp >> 2, row = tid & 127;             // the thread's 64 tokens of a block, and its row
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;
    const uint32_t t_s = tmem + kTmemS + half * 64 + lanes, t_o = tmem + kTmemO + half * 64 + lanes;
    const int r8 = tid & 7;                      // lane of a row that 8 lanes have
    const uint32_t sign_bits = a.c.signs[r8 >> 1] >> (16 * (r8 & 1));
    int4 *const joins = reinterpret_cast<int4 *>(a.joins);
    uint32_t s_count[2] = {0, 0};
    if (tid == 0 && !a.by_pair) joins[blockIdx.x] = make_int4(0, 0, 0, 0);
    while (true) {
      if (tid == 0) {                            // one thread walks, as the walk's state takes registers
        Walk walk = S.walk;
        Segment seg;
        const bool more = walk.next<true, kSegmentCost>(a, &seg);
        S.walk = walk;
        S.more = more;
        if (more) {
          S.b = seg.b;
          S.pair = seg.pair;
          S.u_lo = seg.u_lo;
          S.u_hi = seg.u_hi;
          S.nu = seg.nu;
          const bool whole = seg.u_lo == 0 && seg.u_hi == seg.nu;
          if (seg.u_lo == 0 && (a.by_pair || !whole))      // begun here; ended by later blocks
            joins[a.by_pair ? seg.b * a.c.n_kv * a.row_tiles + seg.pair : blockIdx.x] =
                make_int4((int)(kv4_divide(seg.at_end - 1, S.piece) - blockIdx.x), blockIdx.x, seg.b, seg.pair);
        }
      }
      rows_sync();
      if (S.more == 0) {
        if (lane == 0) {
          mbar_arrive(&S.ready);
          mbar_arrive(&S.q_full);
        }
        break;
      }
      const int b = S.b, u_lo = S.u_lo, h = S.pair / a.row_tiles, row0 = (S.pair % a.row_tiles) * kRows;
      bool bad_len;
      const int committed = kv4_length(a.c, a.lengths, b, &bad_len);
      const int n = (S.u_hi - u_lo + kBlockUnits - 1) / kBlockUnits;
      // ---- the tree: which drafts there are, and which of them each row sees
      {
        const int p = tid < a.q_len ? a.parents[(int64_t)b * a.q_len + tid] : -2;
        const bool bad = p >= tid || p < -2;
        if (bad && tid < a.q_len) atomicOr(a.status, (uint32_t)HQ_ERR_PAGE);
        S.parent[tid] = bad ? -2 : p;
        const uint32_t bits = __ballot_sync(0xffffffffu, !bad && p >= -1);
        if (lane == 0) S.there[warp] = bits;
      }
      rows_sync();
      bool there = false;                        // the thread's row is a draft's, and its path leads to the committed tokens
      if (row0 + row < a.R) {
        uint32_t w[kSeenWords] = {};
        int j = (row0 + row) / a.G;
        const bool padding = S.parent[j] == -2;
        while (j >= 0) {                         // parents come first, so this ends
#pragma unroll
          for (int k = 0; k < kSeenWords; ++k)
            if (j >> 5 == k) w[k] |= 1u << (j & 31);
          j = S.parent[j];
        }
        there = j == -1;
        if (!there && !padding) atomicOr(a.status, (uint32_t)HQ_ERR_PAGE);      // a parent that is not there
        if (half == 0) {
#pragma unroll
          for (int k = 0; k < kSeenWords; ++k) S.seen[row * kSeenRow + k] = there ? w[k] : 0u;
        }
      }
      if (tid == 0) {
        int len = committed;
#pragma unroll
        for (int k = 0; k < kSeenWords; ++k)
          if (S.there[k] != 0u) len = committed + 32 * k + 32 - __clz(S.there[k]);
        if (len > (int)a.c.capacity()) {         // drafts behind the table's end
          atomicOr(a.status, (uint32_t)HQ_ERR_PAGE);
          len = (int)a.c.capacity();
        }
        S.len = len;
      }
      rows_sync();
      if (lane == 0) mbar_arrive(&S.ready);
      // ---- the query rows, 64 at a time: rotated, scaled by a power of two, split, 8 lanes a row; then, a lane a
      // row, into tensor memory, the high parts by one warp of a pair, the low ones by the other
      float ahead[16];                           // of the next pass
      const auto load = [&](int pass) {
        const int rw = row0 + 32 * pass + (tid >> 3);
#pragma unroll
        for (int i = 0; i < 16; ++i) ahead[i] = 0.0f;
        if (rw >= a.R) return;
        const int j = rw / a.G;
        const int64_t at = b * a.q_seq + j * a.q_token + (int64_t)(h * a.G + rw - j * a.G) * a.q_head;
        if (a.kind == HQ_T_F32) load_q16<HQ_T_F32>(a, at, r8, ahead);
        else if (a.kind == HQ_T_F16) load_q16<HQ_T_F16>(a, at, r8, ahead);
        else load_q16<HQ_T_BF16>(a, at, r8, ahead);
      };
      load(0);
#pragma unroll 1
      for (int pass = 0; pass < 4; ++pass) {
        float *const tr = reinterpret_cast<float *>(s_raw + (stage_at - raw) + kTileBytes) + warp * 4 * kTrTile;
        {
          const int rr = 32 * pass + (tid >> 3);
          float x[16];
#pragma unroll
          for (int i = 0; i < 16; ++i)
            x[i] = __fmul_rn(__uint_as_float(__float_as_uint(ahead[i]) ^ (((sign_bits >> i) & 1u) << 31)), kInvRoot128);
          if (pass < 3) load(pass + 1);
          fwht128_t8(x, tr + (lane >> 3) * kTrTile, r8);
          float top = 0.0f;
#pragma unroll
          for (int i = 0; i < 16; ++i) top = fmaxf(top, fabsf(x[i]));
#pragma unroll
          for (int d = 1; d < 8; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
          top = fmaxf(top, 0x1p-100f);
          // the largest value in 2^14 .. 2^15, so that the low parts keep their bits; the sign of scale beside it
          const float sc = scale_of(top), inv = inv_scale_of(top), up = copysignf(0x1p15f, a.scale);
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            uint32_t hi[4], lo[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
              split_f16x2(__fmul_rn(__fmul_rn(x[8 * g + i], sc), up), __fmul_rn(__fmul_rn(x[8 * g + i + 4], sc), up),
                          hi[i], lo[i]);
            const uint32_t to = stage_at + (rr & 63) * 512 + (((2 * r8 + g) ^ (rr & 7)) * 16);
            st16(to, make_uint4(hi[0], hi[1], hi[2], hi[3]));
            st16(to + 256, make_uint4(lo[0], lo[1], lo[2], lo[3]));
          }
          if (r8 == 0)
            S.mul[rr] = fmaxf(fabsf(__fmul_rn(__fmul_rn(CAP ? a.scale : __fmul_rn(a.scale, kLog2e), inv), 0x1p-6f / kKeyScale)), 0x1p-149f);   // not 0: -inf stays -inf
        }
        if (pass & 1) {
          rows_sync();
          if ((row >> 6) == (pass >> 1)) {
#pragma unroll 1
            for (int c = 0; c < 2; ++c) {
              uint32_t w[32];
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const uint4 v = ld16(stage_at + (row & 63) * 512 + half * 256 + (((8 * c + e) ^ (row & 7)) * 16));
                w[4 * e] = v.x;
                w[4 * e + 1] = v.y;
                w[4 * e + 2] = v.z;
                w[4 * e + 3] = v.w;
              }
              tmem_st32(tmem + kTmemQ + lanes + half * 64 + 32 * c, w);
            }
            tmem_wait_st();
          }
          rows_sync();
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.q_full);
      const float mul = S.mul[row];
      const uint64_t mul2x = pk2(mul, mul);
      // ---- the blocks of tokens: m and log2 f are whole numbers and apart, the same for a row's two threads
      float m = kNoMax, lf = 0.0f;
      uint64_t l2 = 0;
#pragma unroll 1
      for (int k = 0; k < n; ++k) {
        const int s = k & 1, slot = k & (kScaleSlots - 1), t0 = (u_lo + kBlockUnits * k) * kUnit + 64 * half;
        const uint32_t at = t_s + s * 128;
        wait(&S.s_full[s], s_count[s]++, abort);
        tc_fence_after();
        const uint32_t valid = S.valid[slot] >> (4 * half);
        const bool masked = t0 + 64 > committed || (valid & 0xFu) != 0xFu;
        const float4 *const sk = reinterpret_cast<const float4 *>(S.sk[slot]) + 16 * half;
        const float4 *const sv = reinterpret_cast<const float4 *>(S.sv[slot]) + 16 * half;
        // y, z without the row's multiplier (capped scores: z), and its maximum
        uint32_t y[2][32];
        float top = -INFINITY;
        if (CAP) {                               // capped in their place, by one body of code for both 32
#pragma unroll 1
          for (int c = 0; c < 2; ++c) {
            uint32_t z[32];
            tmem_ask32(at + 32 * c, z);
            tmem_wait32(z);
#pragma unroll
            for (int e = 0; e < 32; e += 4) {
              const float4 f = sk[8 * c + e / 4];
              put2(z + e, mul2(mul2(pk2(__uint_as_float(z[e]), __uint_as_float(z[e + 1])), pk2(f.x, f.y)), mul2x));
              put2(z + e + 2, mul2(mul2(pk2(__uint_as_float(z[e + 2]), __uint_as_float(z[e + 3])), pk2(f.z, f.w)), mul2x));
            }
            cap32(z, there, 1.0f, a.by_cap, kLog2e, a.by_cap, a.cap_l2);
            tmem_st32(at + 32 * c, z);
          }
          tmem_wait_st();
        }
        tmem_ask32(at, y[0]);
        tmem_ask32(at + 32, y[1]);
        tmem_wait32(y[0]);
        tmem_have32(y[1]);
#pragma unroll
        for (int c = 0; c < 2 && !CAP; ++c) {
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const float4 f = sk[8 * c + e / 4];
            put2(y[c] + e, mul2(pk2(__uint_as_float(y[c][e]), __uint_as_float(y[c][e + 1])), pk2(f.x, f.y)));
            put2(y[c] + e + 2, mul2(pk2(__uint_as_float(y[c][e + 2]), __uint_as_float(y[c][e + 3])), pk2(f.z, f.w)));
          }
        }
        if (masked) {
          // bits of 32 tokens that the row sees: all committed ones, then its path's
          const auto word = [&](int i) { return i < 0 ? 0xffffffffu : i >= kSeenWords ? 0u : S.seen[row * kSeenRow + i]; };
          const int d = t0 - committed, q = d >> 5;
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t sees = __funnelshift_r(word(q + c), word(q + c + 1), d & 31);
            if (!((valid >> (2 * c)) & 1u)) sees &= 0xFFFF0000u;
            if (!((valid >> (2 * c + 1)) & 1u)) sees &= 0x0000FFFFu;
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!(sees & (1u << e))) y[c][e] = 0xFF800000u;
          }
        }
#pragma unroll
        for (int e = 0; e < 32; ++e) top = max3(top, __uint_as_float(y[0][e]), __uint_as_float(y[1][e]));
        if (!CAP) top = __fmul_rn(top, mul);
        S.top[s][half][row] = top;
        pair_sync(warp);
        top = fmaxf(top, S.top[s][half ^ 1][row]);
        // The references move only when a weight 2^(z - m) s f might pass 2^15 by the block's largest s; f
        // then holds the row's largest weight so far near 2^7, or, where the block's scales are within 2^5 of one
        // another, no more than that below.  And they move before 2^(z - m), or that times s, leaves fp32: scales may
        // be 0, or far below those that f was taken from.
        {
          const float4 tops = S.sv_top[slot], lows = S.sv_low[slot];
          const float sv_top = fmaxf(fmaxf(tops.x, tops.y), fmaxf(tops.z, tops.w));
          const float lg_top = lg2(sv_top);
          const float up = __fsub_rn(top, m), up_s = __fadd_rn(up, lg_top);
          const bool need = k == 0 || __fadd_rn(up_s, lf) > 14.5f || up > 60.0f || up_s > 126.0f;
          if (__any_sync(0xffffffffu, need)) {
            const float sv_low = fminf(fminf(lows.x, lows.y), fminf(lows.z, lows.w));
            const float now = need ? fmaxf(m, ceilf(top)) : m;
            float ut = __fadd_rn(__fsub_rn(top, now), lg_top);   // the largest z + log2 s, beside the new m, or more
            if (!(sv_top <= __fmul_rn(sv_low, 32.0f))) {
              ut = kNoMax;
#pragma unroll
              for (int e = 0; e < 64; ++e) {
                const float z = CAP ? __uint_as_float(y[e >> 5][e & 31]) : __fmul_rn(__uint_as_float(y[e >> 5][e & 31]), mul);
                ut = fmaxf(ut, __fadd_rn(__fsub_rn(z, now), lg2(reinterpret_cast<const float *>(sv)[e])));
              }
              S.low[half][row] = ut;
              pair_sync(warp);
              ut = fmaxf(ut, S.low[half ^ 1][row]);
              pair_sync(warp);                   // read before it is written again
            }
            ut = fmaxf(ut, kNoMax);
            const float down = m == now ? 0.0f : __fsub_rn(m, now);
            // what was largest so far was near 2^7 / f; nothing was before the first block
            const float u2 = k == 0 ? ceilf(ut) : fmaxf(__fadd_rn(__fsub_rn(7.0f, lf), down), ceilf(ut));
            const float lf2 = need ? fminf(fmaxf(__fsub_rn(7.0f, u2), -120.0f), 120.0f) : lf;
            if (k > 0) {
              const float keep = ex2(down), by = ex2(__fadd_rn(down, __fsub_rn(lf2, lf)));
              l2 = mul2(l2, pk2(keep, keep));
              wait(&S.v_empty[s ^ 1], s_count[s ^ 1] - 1, abort);          // the product before is done
              tc_fence_after();
#pragma unroll
              for (int c = 0; c < 2; ++c) {
                uint32_t o[32];
                tmem_ask32(t_o + 32 * c, o);
                tmem_wait32(o);
#pragma unroll
                for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__fmul_rn(__uint_as_float(o[e]), by));
                tmem_st32(t_o + 32 * c, o);
              }
            }
            m = now;
            lf = lf2;
          }
        }
        // weights in two parts, in the place of their scores
        const uint64_t m2 = pk2(-m, -m);
        uint64_t by2 = CAP ? pk2(1.0f, 1.0f) : mul2x;
        // y times its multiplier less m in one step is off by the rounding of m's product, which is less than one
        // up to here; from there on the products are rounded alike first
        if (!CAP && __any_sync(0xffffffffu, fabsf(m) >= 0x1p20f && m > kNoMax)) {
#pragma unroll
          for (int e = 0; e < 64; ++e) y[e >> 5][e & 31] = __float_as_uint(__fmul_rn(__uint_as_float(y[e >> 5][e & 31]), mul));
          by2 = pk2(1.0f, 1.0f);
        }
        const float f1 = __uint_as_float((uint32_t)((int)lf + 127) << 23);
        const uint64_t f2 = pk2(f1, f1);
        uint64_t sum[2] = {0, 0};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t w[32];
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            const float4 f = sv[8 * c + e / 4];
            const uint64_t f4[2] = {pk2(f.x, f.y), pk2(f.z, f.w)};
#pragma unroll
            for (int g = 0; g < 2; ++g) {
              float p0, p1;
              upk2(fma2(pk2(__uint_as_float(y[c][e + 2 * g]), __uint_as_float(y[c][e + 2 * g + 1])), by2, m2), p0, p1);
              const uint64_t p = pk2(ex2(p0), ex2(p1));
              sum[g] = add2(sum[g], p);
              upk2(mul2(mul2(p, f4[g]), f2), p0, p1);
              if constexpr (SPLIT) split_cut(p0, p1, w[e / 2 + g], w[16 + e / 2 + g]);
              else w[e / 2 + g] = round_pair<HQ_T_F16>(p0, p1);
            }
          }
          if constexpr (SPLIT) tmem_st32(at + 32 * c, w);
          else tmem_st16(at + 32 * c, w);
        }
        l2 = add2(l2, add2(sum[0], sum[1]));
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&S.p_full[s]);
      }
      // ---- the sums: through shared memory, a row's 16-byte pieces permuted by the row
      wait(&S.o_full, segments++, abort);
      tc_fence_after();
#pragma unroll 1
      for (int c = 0; c < 2; ++c) {
        uint32_t o[32];
        tmem_ask32(t_o + 32 * c, o);
        tmem_wait32(o);
#pragma unroll
        for (int g = 0; g < 4; ++g) {            // positions 2 i + h of 8 are dimensions i + 4 h
          const int piece = 16 * half + 8 * c + 2 * g;
          st16(stage_at + row * 512 + ((piece ^ (row & 31)) * 16), make_uint4(o[8 * g], o[8 * g + 2], o[8 * g + 4], o[8 * g + 6]));
          st16(stage_at + row * 512 + (((piece + 1) ^ (row & 31)) * 16), make_uint4(o[8 * g + 1], o[8 * g + 3], o[8 * g + 5], o[8 * g + 7]));
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&S.o_empty);
      float l0, l1;
      upk2(l2, l0, l1);
      S.l[half][row] = __fadd_rn(l0, l1);
      // padding: zeros, whatever it added up
      if (half == 0) S.stat[row] = there ? RowStat{m, 1.0f, -lf, 0.0f} : RowStat{kNoMax, 0.0f, kNoMax, 0.0f};
      rows_sync();
      const bool whole = u_lo == 0 && S.u_hi == S.nu;
      {
        float *const tr = reinterpret_cast<float *>(s_raw + (kv_at - raw)) + warp * 4 * kTrTile;
#pragma unroll 1
        for (int pass = 0; pass < 4; ++pass) {
          const int rr = 32 * pass + (tid >> 3), rw = row0 + rr;
          const bool live = rw < a.R;
          const int j = live ? rw / a.G : 0, hq = h * a.G + rw - j * a.G;
          const RowStat st = S.stat[rr];
          const float M = st.m, E = st.e, L = st.l == 0.0f ? 0.0f : __fadd_rn(S.l[0][rr], S.l[1][rr]);
          float x[16];
#pragma unroll
          for (int i = 0; i < 4; ++i) {          // values are in units of 2^-9
            const uint4 v = ld16(stage_at + rr * 512 + (((4 * r8 + i) ^ (rr & 31)) * 16));
            x[4 * i] = L == 0.0f ? 0.0f : __fmul_rn(__uint_as_float(v.x), 512.0f);
            x[4 * i + 1] = L == 0.0f ? 0.0f : __fmul_rn(__uint_as_float(v.y), 512.0f);
            x[4 * i + 2] = L == 0.0f ? 0.0f : __fmul_rn(__uint_as_float(v.z), 512.0f);
            x[4 * i + 3] = L == 0.0f ? 0.0f : __fmul_rn(__uint_as_float(v.w), 512.0f);
          }
          if (whole) {
            normalize(x, E, L);
            finish_row(a, x, tr + (lane >> 3) * kTrTile, r8, sign_bits, live, ((int64_t)b * a.q_len + j) * a.Hq + hq);
            if (live && r8 == 0) finish_stats(a, b, h, rw, M, L);
          } else {
            const int64_t slot = 2 * (int64_t)blockIdx.x + (u_lo == 0 ? 1 : 0);
            float4 *dst = reinterpret_cast<float4 *>(a.part + (slot * kRows + rr) * kTile + 16 * r8);
#pragma unroll
            for (int c = 0; c < 4; ++c) dst[c] = make_float4(x[4 * c], x[4 * c + 1], x[4 * c + 2], x[4 * c + 3]);
            if (r8 == 0) reinterpret_cast<float4 *>(a.stat)[slot * kRows + rr] = make_float4(M, L, E, 0.0f);
          }
        }
      }
      rows_sync();                               // the sums are out, the statistics and masks used up
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  // rows of sequences without room for tokens, and lengths out of range
  for (int sb = blockIdx.x; sb < a.c.n_seqs; sb += gridDim.x) {
    bool bad_len;
    kv4_length(a.c, a.lengths, sb, &bad_len);
    if (bad_len && tid == 0) atomicOr(a.status, (uint32_t)HQ_ERR_PAGE);
    if (units_of<true>(a, sb) > 0) continue;
    if (a.by_pair)
      for (int i = tid; i < a.c.n_kv * a.row_tiles; i += kThreads)
        reinterpret_cast<int4 *>(a.joins)[sb * a.c.n_kv * a.row_tiles + i] = make_int4(0, 0, 0, 0);
    const int64_t at = (int64_t)sb * a.q_len * a.Hq;
    for (int64_t i = tid >> 3; i < (int64_t)a.q_len * a.Hq; i += kThreads / 8) {
      float zero[16] = {};
      if (a.out_kind == HQ_T_F32) store_row16<HQ_T_F32>(a.out, (at + i) * kTile, tid & 7, true, zero);
      else store_row16<HQ_T_BF16>(a.out, (at + i) * kTile, tid & 7, true, zero);   // the same in fp16
      if ((tid & 7) == 0 && a.lse != nullptr) a.lse[at + i] = -INFINITY;
    }
  }
  if (tid == 0 && S.abort) atomicOr(a.status, (uint32_t)HQ_ERR_TIMEOUT);
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <bool CAP, bool SPLIT>
int launch(const Kv4AttnArgs &a, cudaStream_t st) {
  static int blocks[64] = {};                    // asked once an instance and device
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 1;
  int grid = dev < 64 ? blocks[dev] : 0;
  if (grid == 0) {
    if (cudaFuncSetAttribute(kv4_tree_kernel<CAP, SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess ||
        cudaDeviceGetAttribute(&grid, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
      cudaGetLastError();
      return 1;
    }
    if (grid > kMaxBlocks) grid = kMaxBlocks;
    if (dev < 64) blocks[dev] = grid;
  }
  // no more blocks than pieces of the longest batch the table allows
  const int64_t pairs = (int64_t)a.c.n_seqs * a.c.n_kv * a.row_tiles;
  int64_t most = ((a.c.capacity() / kUnit + kSegmentCost) * pairs + kMinPiece - 1) / kMinPiece;
  if (most < pairs) most = pairs;
  if (most < grid) grid = (int)most;
  Kv4AttnArgs w = a;
  w.whole = 0;                                   // tables so short do not come here
  w.by_pair = pairs <= grid;
  if (launch_behind(kv4_tree_kernel<CAP, SPLIT>, dim3((unsigned)grid), kThreads, (size_t)kSmem, st, w) != 0) return 1;
  return launch_kv4_join(w, kRows, (w.by_pair ? (int)pairs : grid) * kRows, st);
}

}  // namespace

// 16 rows of a head at a time in registers (hq_kv4_attn.cu), or 128 through shared memory: the first streams and
// unpacks the tokens once for every 16 rows and begins as many tiles, the second takes 3 to 8 us more to begin and end.
// us, first / second, 8 heads: 36 rows over 1 x 65536 tokens 89 / 63, over 16 x 1000 40 / 43; 48 rows over 1 x 8192
// 25 / 29, 1 x 16384 34 / 34, 16 x 1000 42 / 43, 32 x 500 53 / 46; 64 rows over 1 x 8192 27 / 29, 16 x 500 40 / 40, 16 x 1000
// 52 / 45; 96 rows over 1 x 4000 26 / 28, 1 x 8192 37 / 30; 128 rows over 1 x 2000 25 / 28, 1 x 4000 31 / 29, 16 x 300
// 57 / 30; 256 rows over 1 x 1000 27 / 29, 1 x 2000 34 / 30, 1 x 8192 69 / 36; 512 rows over 1 x 500 20 / 30, 1 x 1000
// 36 / 31; 32 rows over 64 x 2000 136 / 150.  384: a tile of the first, in tokens (its kSegmentCost).  The lengths are on
// the device; the table's room stands for them.
bool kv4_tree_is_wide(int R, int64_t n_seqs, int n_kv, int64_t capacity) {
  return R > 32 && n_seqs * n_kv * ((R + 15) / 16) * (capacity + 384) > 280000;
}
int kv4_tree_row_tiles(int R) { return (R + kRows - 1) / kRows; }
size_t kv4_tree_part_bytes() { return (size_t)2 * kMaxBlocks * kRows * kTile * sizeof(float); }
size_t kv4_tree_stat_bytes() { return (size_t)2 * kMaxBlocks * kRows * sizeof(float4); }

int launch_kv4_tree(const Kv4AttnArgs &a, cudaStream_t st) {
  if (a.out_kind == HQ_T_F32) return a.cap > 0.0f ? launch<true, true>(a, st) : launch<false, true>(a, st);
  return a.cap > 0.0f ? launch<true, false>(a, st) : launch<false, false>(a, st);
}

}  // namespace hq

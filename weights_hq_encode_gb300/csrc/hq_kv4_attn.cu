// hq_kv4_attn.cu -- attention over the 4-bit window cache, read straight from
// the codes (include/hq_kv4.h).  The transform moves to the other operand:
// with q' = H D q / sqrt(128), q . Khat[t] = s_t sum_d q'_d (c_td - 7.5), and
// sum_t p_t Vhat[t] = D H (sum_t p_t s_t (c_t - 7.5)) / sqrt(128), one
// transform per query row and one per output row.
#include <cuda_runtime.h>

#include <cmath>

#include "hq_device.cuh"
#include "hq_kv4.h"
#include "hq_kv4_io.cuh"
#include "hq_launch.cuh"
#include "hq_umma.cuh"

namespace hq {

namespace {

constexpr float kInvRoot128 = 0.08838834764831845f;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kLoScale = 2048.0f;
constexpr float kNoMax = -3.0e38f;               // below every finite score

constexpr int kWarps = 4;                        // warps of a block
constexpr int kAttnThreads = 32 * kWarps;
constexpr int kUnits = 2;                        // units of a tile, a warp's step: 32 tokens
constexpr int kTileTokens = kUnits * kUnit, kStageBytes = kUnits * kUnitBytes;
constexpr int kStages = 3;                       // tiles a warp has in its ring
constexpr int kRingBytes = kWarps * kStages * kStageBytes;

// Blocks of 4, 8 or 16 query rows
template <int ROWS>
struct Shape {
  static constexpr int q_bytes = 2 * ROWS * kTile * 2;      // query fragments, high and low parts
  static constexpr int smem = kRingBytes + q_bytes + ROWS * kTrTile * 4;
  // Resident blocks a multiprocessor: 12 warps of 168 registers, or 8 of up to 255.  More warps of
  // fewer registers keep parts of a tile in local memory: 16 of 128 took 118 us instead of 110 for 16 x
  // 32768 tokens of 8 heads and 4 rows; 12 of 168 with 8 rows 46.6 instead of 45.5 for 16 x 8192.
  static constexpr int blocks = ROWS == 4 ? 3 : 2;
  static_assert(kWarps * ROWS * kTile * 4 <= kRingBytes, "the warps' sums fit the ring");
};

// Work of one (sequence, head, row tile) beyond its units, in units: the
// blocks split the batch into equal pieces of units + kSegmentCost.  Rotating
// its queries and adding up its sums takes a block 4 to 5 us, in which it streams
// 16 to 30 units.  Costs of 8 / 16 / 24 / 32 in us, without a cap: 24 ragged sessions of 4093 tokens 26.5 / 23.5 /
// 23.4 / 23.5 with 4 rows, 32.1 / 28.2 / 27.5 / 26.7 with 8, 43.4 / 39.5 / 38.8 / 38.0 with 16; one of 131072
// tokens 35.3 / 33.7 / 34.9 / 35.1 with 4 rows, 41.8 / 41.0 / 42.4 / 42.4 with 8, 63.0 / 61.6 / 62.8 / 63.0
// with 16; 16 of 32768 tokens 108.5 / 107.4 / 110 / 112 with 4 rows.
constexpr int kSegmentCost = 24, kMinPiece = 40;
// Where the table has room for no span (units + kSegmentCost) longer than this, and
// all (sequence, head, row tile) triples fit at once, each gets a block and nothing is joined: a join takes
// longer than the units it spreads.  The lengths are not known to the launch, so a wider table
// takes the other path, whatever the lengths (one session of 77 tokens: 5.5 us, and 7.1 to 7.4 with a table
// for more than 640 tokens).  On that path pieces are no shorter than the longest span
// up to this, so that a triple is cut once at most.
constexpr int kWholeSpan = 64;

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Codes as fp16 pairs.  The low bits of a half are a subnormal number of units
// 2^-24: pairs of a byte's low nibble, c_e, and of whole bytes, c_e + 16 c_o,
// take one instruction each, and one fused multiply-add more centres them, in
// units of 2^-9: c_e - 7.5 and (c_e - 7.5) + 16 (c_o - 7.5), exactly.  The other
// side sorts the bytes out: a score takes q_e - q_o / 16 with the even code
// and q_o / 16 with the byte, a value's odd dimension is (byte's sum - even
// sum) / 16.  Centred, because the adder of the tensor cores cuts small addends beside
// large ones: the scores of uncentred codes with the sum of -7.5 q as a start
// were 7 to 8 times further off, 6% faster.
// Pairs i = 0, 1 come from bytes 0 and 2 of x, i = 2, 3 from bytes 1 and 3.
__device__ __forceinline__ uint32_t centred(uint32_t c, uint32_t factor, uint32_t minus) {
  uint32_t y;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(y) : "r"(c), "r"(factor), "r"(minus));
  return y;
}
__device__ __forceinline__ void code_pairs(uint32_t x, uint32_t factor, uint32_t p[4]) {
  const uint32_t y = __byte_perm(x, 0u, 0x4341);
  p[0] = centred(x & 0x000F000Fu, factor, 0xA380A380u);   // -7.5 2^-9
  p[1] = centred(x & 0x00FF00FFu, factor, 0xB3F8B3F8u);   // -127.5 2^-9
  p[2] = centred(y & 0x000F000Fu, factor, 0xA380A380u);
  p[3] = centred(y, factor, 0xB3F8B3F8u);
}
// cap log2(e) tanh(y), y = z / cap, of two values: y's sign and 1 - 2 / (1 + e^2|y|) from 1/4 on; below,
// where that is off by 2^-23 beside a small value, y - y^3 / 3 + 2 y^5 / 15 - 17 y^7 / 315, whose rest
// is less than 3.4e-7 of it.  y is formed from z: with 1 / cap in the multipliers of a score's parts,
// small queries over large keys under a large cap left fp32's range on the way.
__device__ __forceinline__ uint64_t cap_tanh(float z0, float z1, const Kv4AttnArgs &a) {
  const uint64_t yy = pk2(__fmul_rn(z0, a.by_cap), __fmul_rn(z1, a.by_cap));
  const uint64_t y2 = mul2(yy, yy);
  uint64_t t = fma2(y2, pk2(-17.0f / 315.0f, -17.0f / 315.0f), pk2(2.0f / 15.0f, 2.0f / 15.0f));
  t = fma2(y2, t, pk2(-1.0f / 3.0f, -1.0f / 3.0f));
  t = fma2(mul2(yy, y2), t, yy);
  float y[2], p[2];
  upk2(yy, y[0], y[1]);
  upk2(t, p[0], p[1]);
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const float ey = ex2(__fmul_rn(fabsf(y[e]), 2.0f * kLog2e));
    const float far = copysignf(__fsub_rn(1.0f, __fdividef(2.0f, __fadd_rn(ey, 1.0f))), y[e]);
    p[e] = __fmul_rn(a.cap_l2, fabsf(y[e]) < 0.25f ? p[e] : far);
  }
  return pk2(p[0], p[1]);
}
__device__ __forceinline__ void mma16816(float d[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// Copies of the stream: read once, so they go first when L2 needs room, and
// the code, tables and queries of the next launches stay there (the first
// tile of a long batch's blocks begins after 5 us instead of 7).
__device__ __forceinline__ uint64_t stream_policy() {
  uint64_t p;
  asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, uint64_t policy) {
  asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "l"(policy)
               : "memory");
}
// A unit's codes, if its number is one: 16 bytes a lane and 512-byte quarter.
__device__ __forceinline__ void cp_async_codes(int unit, uint32_t k, uint32_t v, const void *src, uint64_t policy) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ge.s32 p, %0, 0;\n\t"
      "@p cp.async.cg.shared.global.L2::cache_hint [%1], [%3], 16, %4;\n\t"
      "@p cp.async.cg.shared.global.L2::cache_hint [%1 + 512], [%3 + 512], 16, %4;\n\t"
      "@p cp.async.cg.shared.global.L2::cache_hint [%2], [%3 + 1024], 16, %4;\n\t"
      "@p cp.async.cg.shared.global.L2::cache_hint [%2 + 512], [%3 + 1536], 16, %4;\n\t}" ::"r"(unit),
      "r"(k), "r"(v), "l"(src), "l"(policy)
      : "memory");
}
// The same from zero.
__device__ __forceinline__ void mma16816_first(float d[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                               uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ uint4 read16(const unsigned char *p) { return *reinterpret_cast<const uint4 *>(p); }
__device__ __forceinline__ float read_bf16(const unsigned char *p) {
  return bf16_to_f32(*reinterpret_cast<const uint16_t *>(p));
}
// An 8 x 8 matrix of 16-bit values, two a lane, transposed over the warp.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(v));
  return y;
}
// (lo, hi) -> hi parts and 2^11 times the rests, both fp16 pairs: the parts
// miss a value by 2^-22 of it, and by 2^-36 where it is below fp16's normal
// range, so that small values keep their bits beside large ones.
__device__ __forceinline__ void split2(float lo, float hi, uint32_t &h, uint32_t &rest) {
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(hi), "f"(lo));
  const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
  float r0, r1;                                  // exact: 2^11 x - 2^11 h
  upk2(fma2(pk2(f.x, f.y), pk2(-kLoScale, -kLoScale), mul2(pk2(lo, hi), pk2(kLoScale, kLoScale))), r0, r1);
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(rest) : "f"(r1), "f"(r0));
}

// The same with the rests as they are: the parts miss a value by 2^-22 of it and 2^-25, 2^-32
// of the largest weight.
__device__ __forceinline__ void split2_plain(float lo, float hi, uint32_t &h, uint32_t &rest) {
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(hi), "f"(lo));
  const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
  float r0, r1;
  upk2(sub2(pk2(lo, hi), pk2(f.x, f.y)), r0, r1);          // exact
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(rest) : "f"(r1), "f"(r0));
}

template <int KIND>
__device__ __forceinline__ void load_q16(const Kv4AttnArgs &a, int64_t at, int r, float x[16]) {
  load_row16<KIND>(a.q, at, r, a.q_vec != 0, x);
}

// 16 lanes of one row out, D H x / sqrt(128) applied: the last step of every
// row.  All 32 lanes of the warp must call it.
__device__ __forceinline__ void finish_row(const Kv4AttnArgs &a, float x[16], float *tile, int r,
                                           uint32_t mw, bool live, int64_t o) {
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = __fmul_rn(x[i], kInvRoot128);
  fwht128_t8(x, tile, r);
  if (!live) return;
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = __uint_as_float(__float_as_uint(x[i]) ^ (((mw >> i) & 1u) << 31));
  if (a.out_kind == HQ_T_F32) store_row16<HQ_T_F32>(a.out, o * kTile, r, true, x);
  else if (a.out_kind == HQ_T_F16) store_row16<HQ_T_F16>(a.out, o * kTile, r, true, x);
  else store_row16<HQ_T_BF16>(a.out, o * kTile, r, true, x);
}

// A row's sums over some of its tokens: l = sum 2^(z - m), and acc (kept
// beside it) = sum 2^(z - m - e) s (c - 7.5).  m and e are whole numbers and apart:
// from 2^24 on m has no bits left for e, which undoes the scaling of the
// weights and has to be exact whatever the scores.
struct RowStat {
  float m, l, e, pad;
};

// acc / l at its own references: x 2^e / l, zeros where there is no weight.
__device__ __forceinline__ void normalize(float x[16], float e, float l) {
  const float f = ex2(__fmul_rn(e, 0.5f));       // in two steps, each within range
  const float g = l == 0.0f ? 0.0f : __fmul_rn(__fdiv_rn(1.0f, l), f);
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = __fmul_rn(__fmul_rn(x[i], g), f);
}

__device__ __forceinline__ void finish_stats(const Kv4AttnArgs &a, int b, int h, int row, float M, float L) {
  const float l2 = L == 0.0f ? -INFINITY : log2f(L);
  const int j = row / a.G, hq = h * a.G + row % a.G;
  if (a.lse != nullptr) a.lse[((int64_t)b * a.q_len + j) * a.Hq + hq] = __fmul_rn(__fadd_rn(M, l2), kLn2);
  if (a.mass_out != nullptr) a.row_stat[((int64_t)b * a.c.n_kv + h) * a.R + row] = make_float2(M, l2);
}

// Where a block's piece of the batch begins, and the piece's length: the
// (sequence, head, row tile) triples laid end to end, each of its units +
// kSegmentCost, are cut into equal pieces.
struct Piece {
  int64_t begin, end;       // of the laid-out batch, this block's piece
  int64_t size;             // units + costs of a piece
  int b;                    // sequence at `begin` (n_seqs: nothing left)
  int64_t b_begin;          // where sequence b begins
};

__device__ __forceinline__ int units_of(const Kv4AttnArgs &a, int b) {
  bool bad;
  const int n = kv4_length(a.c, a.lengths, b, &bad);
  return (n + kUnit - 1) / kUnit;
}

__device__ __forceinline__ int64_t span_of(const Kv4AttnArgs &a, int b) {
  const int nu = units_of(a, b);
  return nu == 0 ? 0 : (int64_t)a.c.n_kv * a.row_tiles * (nu + kSegmentCost);
}

// The walk over a block's piece, segment by segment: the units of one
// (sequence, head, row tile) that lie in it.  Every warp walks alike.
struct Segment {
  int b, pair, u_lo, u_hi, nu;
  int64_t at_end;           // where the pair ends in the laid-out batch
};
struct Walk {
  int64_t cur, end, b_begin;
  int b;
  __device__ __forceinline__ bool next(const Kv4AttnArgs &a, Segment *s) {
    while (cur < end) {
      const int nu = units_of(a, b), span1 = nu + kSegmentCost;
      const int64_t b_end = b_begin + (nu == 0 ? 0 : (int64_t)a.c.n_kv * a.row_tiles * span1);
      if (cur >= b_end) {
        ++b;
        b_begin = b_end;
        continue;
      }
      const int pair = (int)kv4_divide(cur - b_begin, span1);       // head and row tile of sequence b
      const int64_t at = b_begin + (int64_t)pair * span1;    // where the pair begins
      s->b = b;
      s->pair = pair;
      s->nu = nu;
      s->u_lo = (int)max((int64_t)0, cur - at - kSegmentCost);
      s->u_hi = (int)min((int64_t)nu, end - at - kSegmentCost);
      s->at_end = at + span1;
      cur = min(at + span1, end);
      if (s->u_lo < s->u_hi) return true;
    }
    return false;
  }
};

__device__ Piece find_piece(const Kv4AttnArgs &a) {
  __shared__ int64_t s_sum[kWarps];
  __shared__ int s_top[kWarps];
  __shared__ int64_t s_begin;
  __shared__ int s_b;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int B = a.c.n_seqs;
  Piece p;
  if (a.whole) {                                 // block i takes the i-th (sequence, head, row tile)
    const int pairs = a.c.n_kv * a.row_tiles;
    p.b = blockIdx.x / pairs;
    const int units = units_of(a, p.b);
    p.size = units + kSegmentCost;
    p.b_begin = 0;                               // laid out from this sequence on
    p.begin = (int64_t)(blockIdx.x - p.b * pairs) * p.size;
    p.end = units == 0 ? p.begin : p.begin + p.size;
    return p;
  }
  if (B <= 32) {                                 // every warp by itself, a sequence a lane
    const int64_t span = lane < B ? span_of(a, lane) : 0;
    int top = lane < B ? units_of(a, lane) + kSegmentCost : 0;
    int64_t incl = span;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t o = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += o;
      top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
    }
    const int64_t total = __shfl_sync(0xffffffffu, incl, 31);
    const int64_t even = kv4_divide(total + gridDim.x - 1, gridDim.x), least = top <= kWholeSpan ? top : kMinPiece;
    p.size = even > least ? even : least;
    p.begin = (int64_t)blockIdx.x * p.size;
    p.end = p.begin + p.size < total ? p.begin + p.size : total;
    p.b = __popc(__ballot_sync(0xffffffffu, incl <= p.begin));   // sequences that end before
    if (p.b > 31) p.b = 31;
    p.b_begin = __shfl_sync(0xffffffffu, incl - span, p.b);
    return p;
  }
  int64_t total = 0;
  int top = 0;                                   // the longest sequence's span
  for (int b = tid; b < B; b += kAttnThreads) {
    total += span_of(a, b);
    top = max(top, units_of(a, b));
  }
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) {
    total += __shfl_xor_sync(0xffffffffu, total, d);
    top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
  }
  if (lane == 0) {
    s_sum[warp] = total;
    s_top[warp] = top;
  }
  if (tid == 0) s_b = B;
  __syncthreads();
  total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    total += s_sum[w];
    top = max(top, s_top[w]);
  }
  top += kSegmentCost;
  const int64_t even = kv4_divide(total + gridDim.x - 1, gridDim.x), least = top <= kWholeSpan ? top : kMinPiece;
  p.size = even > least ? even : least;
  p.begin = (int64_t)blockIdx.x * p.size;
  p.end = p.begin + p.size < total ? p.begin + p.size : total;
  int64_t base = 0;
  for (int b0 = 0; b0 < B && p.begin < p.end; b0 += kAttnThreads) {
    __syncthreads();
    const int b = b0 + tid;
    const int64_t span = b < B ? span_of(a, b) : 0;
    int64_t incl = span;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int64_t o = __shfl_up_sync(0xffffffffu, incl, d);
      if (lane >= d) incl += o;
    }
    if (lane == 31) s_sum[warp] = incl;
    __syncthreads();
    int64_t all = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) incl += s_sum[w];
      all += s_sum[w];
    }
    const int64_t e = base + incl;
    if (e - span <= p.begin && p.begin < e) {    // at most one thread of one step
      s_b = b;
      s_begin = e - span;
    }
    base += all;
    if (base > p.begin) break;                   // block-uniform
  }
  __syncthreads();
  p.b = s_b;
  p.b_begin = s_begin;
  return p;
}

// A block walks the segments of its piece.  Each of its warps takes every
// fourth tile of 32 tokens through a ring of its own in shared memory, filled
// by asynchronous copies, and keeps its own sums; at a segment's end the four
// are added.  A segment that is a whole (sequence, head, row tile) is finished
// here, the others leave their sums for kv4_join_kernel.
//
// The products run on mma.sync m16n8k16, tokens (scores) and dimensions
// (values) as the 16 rows and query rows as the 8 columns: with up to 4 rows
// columns 0 .. 3 are their high parts, columns 4 .. 7 their low parts, so that the
// fp32-level split of 4 rows fills one instruction; with more, 8 rows' high parts
// and 8 rows' low parts are products of their own, whose values share one sum (half
// the registers of sums of their own).  16 rows a block unpack the codes once (24
// ragged sessions of 4093 tokens, 16 rows a head, capped: 49 us; 56 with 8 a
// block and parts in columns).  The codes are unpacked in registers,
// straight into operand fragments; that is why these are not tcgen05
// products, whose operands would first have to be stored to shared memory as
// fp16, four times the bytes that were read: 512 bytes of K and V a token and head,
// written and read 1 KB, 8 cycles at the 128 bytes a cycle that shared memory takes.  Memory
// delivers a token in 6, and with 4 rows this kernel takes 8 (16 x 32768 tokens).  With 16 rows it takes 19,
// and there the choice is not shown to be the better one.
//
// Every 16 rows of a head stream and unpack all its tokens again, those that none of the rows sees among
// them: many new tokens at once are right but slow (512 over 32768 tokens, 8 heads x 4 rows: 1.59 ms).
//
// 16 sequences x 32768 tokens x 8 heads, 4 query rows a head: 109 us, 5.1 TB/s,
// 75% of the copy rate; the copies alone take 98 us, the rest is what instruction
// issue (about 293 a warp for 16 tokens, 54% of the cycles) does not hide.  One
// sequence of 131072 tokens: 34.8 us, of which 13 do not depend on its length (the
// first tile's way 4, the end and the join 5).  With 16 query rows a head, 24
// ragged sessions of 4093 tokens take 42 us (join included), bound by the latency of
// 8 warps a multiprocessor (issue 41%, tensor cores 49%).
template <int kRows, bool CAP, bool MASS>
__global__ void __launch_bounds__(kAttnThreads, Shape<kRows>::blocks) kv4_attn_kernel(Kv4AttnArgs a) {
  constexpr bool kWide = kRows > 4;              // high and low parts in products of their own
  constexpr int kGroups = kWide ? kRows / 8 : 1; // of 8 columns
  constexpr int kHalves = kWide ? 2 : 1;         // tokens of a unit that a lane goes on with
  constexpr int kApart = kWide ? 4 : 2;          // lanes this far and further apart share rows
  extern __shared__ __align__(128) unsigned char s_mem[];
  __shared__ RowStat s_stat[kWarps][kRows];
  __shared__ float s_mul[kRows];                 // multiplier of the scores
  __shared__ int s_seen[kRows];                  // tokens seen
  uint2 *const s_q = reinterpret_cast<uint2 *>(s_mem + kRingBytes);
  float *const s_acc = reinterpret_cast<float *>(s_mem);   // in the ring's place
  float *const s_tr = reinterpret_cast<float *>(s_mem + kRingBytes + Shape<kRows>::q_bytes);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  unsigned char *const ring = s_mem + warp * kStages * kStageBytes;
  const uint32_t ring_a = smem_addr(ring);
  // copies: 16 bytes a lane; V's 16-byte chunks are permuted inside their
  // 128-byte rows so that the reads of a warp touch all banks
  const uint32_t cp_v = kUnitV + (lane >> 3) * 128 + (((lane & 7) ^ (2 * (lane >> 3))) * 16);
  follow_launch();
  const uint32_t sign_bits = a.c.signs[(tid & 7) >> 1] >> (16 * (tid & 1));
  const Piece piece = find_piece(a);
  Walk walk{piece.begin, piece.end, piece.b_begin, piece.b};
  Segment seg;
  const int n8 = lane >> 2, c4 = lane & 3;       // fragment row group, and place in it
  const bool low = !kWide && c4 >= 2;            // this lane's columns are low parts
  const int e0 = kWide ? 2 * c4 : 2 * (c4 & 1);  // its rows of a group: e0, e0 + 1
  const int tok = n8 + (low ? 8 : 0);            // its token of a unit (8 or 16 rows: and the one 8 further on)
  const uint32_t ld_v = kUnitV + c4 * 128 + ((n8 ^ (2 * c4)) * 16);
  const uint64_t policy = stream_policy();
  uint32_t factor;                               // 2^15 twice, in a register that is not filled again
  asm volatile("mov.b32 %0, 0x78007800;" : "=r"(factor));
  const float k_own = low ? 0x1p-6f : 0x1p5f, k_other = low ? 0x1p5f : 0x1p-6f;
  int4 *const joins = reinterpret_cast<int4 *>(a.joins);
  if (tid == 0 && !a.whole && !a.by_pair) joins[blockIdx.x] = make_int4(0, 0, 0, 0);
  while (walk.next(a, &seg)) {
    const int h = seg.pair / a.row_tiles, row0 = (seg.pair % a.row_tiles) * kRows;
    bool bad_len;
    const int len = kv4_length(a.c, a.lengths, seg.b, &bad_len);
    // ---- the query rows' loads, then this warp's first tiles (warp, warp + 4, ..) into its ring
    const int rr = tid >> 3, r = tid & 7, row = row0 + rr;     // of the first 8 kRows threads
    const bool live = rr < kRows && row < a.R;
    const int row_j = live ? row / a.G : 0, row_hq = live ? h * a.G + row - row_j * a.G : 0;
    float x[16];
    if (live) {
      const int64_t qa = seg.b * a.q_seq + row_j * a.q_token + row_hq * a.q_head;
      if (a.kind == HQ_T_F32) load_q16<HQ_T_F32>(a, qa, r, x);
      else if (a.kind == HQ_T_F16) load_q16<HQ_T_F16>(a, qa, r, x);
      else load_q16<HQ_T_BF16>(a, qa, r, x);
    }
    const int mine = ((seg.u_hi - seg.u_lo + kUnits - 1) / kUnits - warp + kWarps - 1) / kWarps;
    int unit[kUnits];                            // unit numbers in the pool of 32 of this warp's tiles
    int issued = 0;                              // tiles asked for
    uint32_t put = 0;                            // byte offset of the next one's stage
    const auto issue = [&]() -> uint32_t {       // the next tile into its stage; one group, maybe empty
      uint32_t got = 0;                          // bit i: unit i has a page
      if (issued < mine) {
        if ((issued & 31) == 0) {                // the next 32 tiles' pages, a tile a lane
          bool bad = false;
#pragma unroll
          for (int k = 0; k < kUnits; ++k) {
            const int u = seg.u_lo + kUnits * (warp + kWarps * (issued + lane)) + k, pj = u / a.c.page_units;
            unit[k] = -1;
            if (u < seg.u_hi) {
              const int page = a.c.table[(int64_t)seg.b * a.c.width + pj];
              if (page >= 0 && page < a.c.n_pages)
                unit[k] = (page * a.c.n_kv + h) * a.c.page_units + u - pj * a.c.page_units;
              else bad = true;
            }
          }
          if (bad) atomicOr(a.status, (uint32_t)HQ_ERR_PAGE);
        }
        const unsigned char *base = a.c.pages + lane * 16;
        int us = -1;                             // scales: four lanes a unit
#pragma unroll
        for (int k = 0; k < kUnits; ++k) {
          const int uk = __shfl_sync(0xffffffffu, unit[k], issued & 31);
          const uint32_t dst = ring_a + put + k * kUnitBytes;
          cp_async_codes(uk, dst + lane * 16, dst + cp_v, base + (int64_t)uk * kUnitBytes, policy);
          if ((lane >> 2) == k) us = uk;
          got |= uk >= 0 ? 1u << k : 0u;
        }
        if (us >= 0)
          cp_async16(ring_a + put + kUnitKs + lane * 16 + (lane >> 2) * (kUnitBytes - 64),
                     base + (int64_t)us * kUnitBytes + kUnitKs - (lane >> 2) * 64, policy);
        ++issued;
        put += kStageBytes;
        if (put == kStages * kStageBytes) put = 0;
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
      return got;
    };
    uint32_t have = 0;                           // kUnits bits a tile in the ring, the oldest lowest
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) have |= issue() << (kUnits * i);
    // ---- the query rows: rotated, scaled by a power of two, split, as mma fragments
    if (tid < 8 * kRows) {
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float v = live ? x[i] : 0.0f;
        x[i] = __fmul_rn(__uint_as_float(__float_as_uint(v) ^ (((sign_bits >> i) & 1u) << 31)), kInvRoot128);
      }
      fwht128_t8(x, s_tr + rr * kTrTile, r);
      float top = 0.0f;
#pragma unroll
      for (int i = 0; i < 16; ++i) top = fmaxf(top, fabsf(x[i]));
#pragma unroll
      for (int d = 1; d < 8; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
      const float sc = scale_of(fmaxf(top, 0x1p-100f)), inv = inv_scale_of(fmaxf(top, 0x1p-100f));
      // 16 q_e - q_o beside an even dimension's code, q_o beside the byte of both
#pragma unroll
      for (int i = 0; i < 16; i += 2) {
        x[i + 1] = __fmul_rn(x[i + 1], sc);
        x[i] = __fmaf_rn(__fmul_rn(x[i], sc), 16.0f, -x[i + 1]);
      }
      // lane r holds words 2 (r & 1), 2 (r & 1) + 1 of the 32 dimensions of place r / 2; row rr is
      // column rr % 8 of group rr / 8, high and low parts side by side, or, with 4 rows, columns rr
      // (high) and rr + 4 (low)
#pragma unroll
      for (int w = 0; w < 2; ++w) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint2 hi, lo;
          split2(x[8 * w + 2 * i], x[8 * w + 2 * i + 4], hi.x, lo.x);
          split2(x[8 * w + 2 * i + 1], x[8 * w + 2 * i + 5], hi.y, lo.y);
          const int k = 2 * (2 * (r & 1) + w) + i;
          if constexpr (kWide) {
            reinterpret_cast<uint4 *>(s_q)[(k * kRows + rr) * 4 + (r >> 1)] = make_uint4(hi.x, hi.y, lo.x, lo.y);
          } else {
            uint2 *dst = s_q + k * 32 + rr * 4 + (r >> 1);
            dst[0] = hi;
            dst[16] = lo;
          }
        }
      }
      if (r == 0) {
        s_mul[rr] = __fmul_rn(CAP ? a.scale : __fmul_rn(a.scale, kLog2e), inv);
        s_seen[rr] = max(0, len - a.q_len + row_j + 1);
      }
    }
    __syncthreads();
    // query fragments: in registers with 4 rows, else read beside every use
    uint2 qr[8];
    if (!kWide) {
#pragma unroll
      for (int k = 0; k < 8; ++k) qr[k] = s_q[k * 32 + lane];
    }
    uint64_t m_own[kGroups], m_other[kGroups];   // multipliers of this lane's and the other part
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      const uint64_t mul = pk2(s_mul[8 * g + e0], s_mul[8 * g + e0 + 1]);
      m_own[g] = mul2(mul, pk2(k_own, k_own));
      m_other[g] = mul2(mul, pk2(k_other, k_other));
    }
    const int seen_all = len - a.q_len + row0 / a.G + 1;    // the least of any row here

    // sums: l of 2^(z - m), acc of w (c - 7.5) 2^-9, w = 2^(z - m) s f, f a power of two a row;
    // acc of odd dimensions with 16 times theirs and the even one's before them
    float acc[kGroups][8][4], l[kGroups][2], m[kGroups][2], f[kGroups][2];
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[g][i][e] = 0.0f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l[g][e] = 0.0f;
        m[g][e] = kNoMax;
        f[g][e] = 1.0f;
      }
    }
    // ---- the tiles
    uint32_t get = 0;                            // byte offset of the next tile's stage
    int t0 = (seg.u_lo + kUnits * warp) * kUnit;
    for (int i = 0; i < mine; ++i, t0 += kWarps * kTileTokens) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
      __syncwarp();                              // tile i has come, and tile i - 1 is used up
      have |= issue() << (kUnits * (kStages - 1));
      const unsigned char *const U = ring + get;
      const uint32_t got = have & ((1u << kUnits) - 1);
      have >>= kUnits;
      get += kStageBytes;
      if (get == kStages * kStageBytes) get = 0;
      // Scores: lane (n8, c4) gets tokens n8 and n8 + 8 of a unit, columns 2 c4, 2 c4 + 1.  With 8
      // or 16 rows these are the rows' high parts, the low parts come in a second result.  With 4 rows
      // lanes c4 and c4 ^ 2 hold the high and the low parts of the same rows: the first goes on with token
      // n8, the second with token n8 + 8, each with the other's part of its token's scores.
      float z[kUnits][kGroups][kHalves][2], sv[kUnits][kHalves];   // [unit][group][token][row], V's scales
#pragma unroll
      for (int un = 0; un < kUnits; ++un) {
        const unsigned char *const V = U + un * kUnitBytes;
        float s[kGroups][kHalves][4];            // [group][high, low]
        const uint4 k0 = read16(V + lane * 16), k1 = read16(V + lane * 16 + 512);
        const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t p0[4], p1[4];
          code_pairs(w0[j], factor, p0);
          code_pairs(w1[j], factor, p1);
#pragma unroll
          for (int g = 0; g < kGroups; ++g) {
            uint4 q0, q1;                        // high and low parts
            if constexpr (kWide) {
              q0 = reinterpret_cast<const uint4 *>(s_q)[(2 * j * kGroups + g) * 32 + lane];
              q1 = reinterpret_cast<const uint4 *>(s_q)[((2 * j + 1) * kGroups + g) * 32 + lane];
            } else {
              q0 = make_uint4(qr[2 * j].x, qr[2 * j].y, 0u, 0u);
              q1 = make_uint4(qr[2 * j + 1].x, qr[2 * j + 1].y, 0u, 0u);
            }
#pragma unroll
            for (int t = 0; t < kHalves; ++t) {
              const uint32_t b0 = t == 0 ? q0.x : q0.z, b1 = t == 0 ? q0.y : q0.w;
              if (j == 0) mma16816_first(s[g][t], p0[0], p1[0], p0[1], p1[1], b0, b1);
              else mma16816(s[g][t], p0[0], p1[0], p0[1], p1[1], b0, b1);
            }
#pragma unroll
            for (int t = 0; t < kHalves; ++t)
              mma16816(s[g][t], p0[2], p1[2], p0[3], p1[3], t == 0 ? q1.x : q1.z, t == 0 ? q1.y : q1.w);
          }
        }
#pragma unroll
        for (int t = 0; t < kHalves; ++t) {
          const float sk = read_bf16(V + kUnitKs + 2 * (tok + 8 * t));
          sv[un][t] = read_bf16(V + kUnitVs + 2 * (tok + 8 * t));
#pragma unroll
          for (int g = 0; g < kGroups; ++g) {
            uint64_t own, other;
            if constexpr (kWide) {
              own = pk2(s[g][0][2 * t], s[g][0][2 * t + 1]);
              other = pk2(s[g][kHalves - 1][2 * t], s[g][kHalves - 1][2 * t + 1]);
            } else {
              const float *const x4 = s[g][0];
              const float o0 = __shfl_xor_sync(0xffffffffu, low ? x4[0] : x4[2], 2);
              const float o1 = __shfl_xor_sync(0xffffffffu, low ? x4[1] : x4[3], 2);
              own = low ? pk2(x4[2], x4[3]) : pk2(x4[0], x4[1]);
              other = pk2(o0, o1);
            }
            float *const zz = z[un][g][t];
            uint64_t y = mul2(fma2(other, m_other[g], mul2(own, m_own[g])), pk2(sk, sk));
            upk2(y, zz[0], zz[1]);
            if (CAP) upk2(cap_tanh(zz[0], zz[1], a), zz[0], zz[1]);
          }
        }
      }
      // warp-uniform: not every row sees every token
      if (t0 + kTileTokens > seen_all || got != (1u << kUnits) - 1) {
#pragma unroll
        for (int un = 0; un < kUnits; ++un)
#pragma unroll
          for (int t = 0; t < kHalves; ++t) {
            const int at = t0 + kUnit * un + tok + 8 * t;
            const bool none = !((got >> un) & 1u) || at >= len;
            if (none) sv[un][t] = 0.0f;          // what lies there is no scale
#pragma unroll
            for (int g = 0; g < kGroups; ++g)
#pragma unroll
              for (int e = 0; e < 2; ++e)
                if (none || at >= s_seen[8 * g + e0 + e]) z[un][g][t][e] = -INFINITY;
          }
      }
      if (MASS) {
#pragma unroll
        for (int g = 0; g < kGroups; ++g)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int zr = row0 + 8 * g + e0 + e;
            if (zr >= a.R) continue;
            float *zrow = a.z + (((int64_t)seg.b * a.c.n_kv + h) * a.R + zr) * a.c.capacity() + t0 + tok;
#pragma unroll
            for (int un = 0; un < kUnits; ++un)
              if (t0 + kUnit * un < seg.u_hi * kUnit) {
#pragma unroll
                for (int t = 0; t < kHalves; ++t) zrow[kUnit * un + 8 * t] = z[un][g][t][e];
              }
          }
      }
      // The references m (a whole number) and f move only when a score is more than 4 above m, or a
      // weight 2^(z - m) s f could pass 2^15: f holds the row's largest weight so far near 2^7.
      float zt = kNoMax, ft = 0.0f, st = 0.0f;
#pragma unroll
      for (int un = 0; un < kUnits; ++un)
#pragma unroll
        for (int t = 0; t < kHalves; ++t) st = fmaxf(st, sv[un][t]);
#pragma unroll
      for (int g = 0; g < kGroups; ++g)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float top = kNoMax;
#pragma unroll
          for (int un = 0; un < kUnits; ++un)
#pragma unroll
            for (int t = 0; t < kHalves; ++t) top = fmaxf(top, z[un][g][t][e]);
          zt = fmaxf(zt, __fsub_rn(top, m[g][e]));
          ft = fmaxf(ft, f[g][e]);
        }
      if (__any_sync(0xffffffffu, zt > 4.0f || __fmul_rn(st, ft) > 2048.0f)) {
        // A row's first tokens, and a score 2^20 above all before it (whose weights are nothing beside it),
        // start the row anew from that score, so that z - m below has a fraction left.
        bool anew[kGroups][2] = {};
        if (__any_sync(0xffffffffu, zt > 0x1p20f)) {
#pragma unroll
          for (int g = 0; g < kGroups; ++g)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              float mt = kNoMax;
#pragma unroll
              for (int un = 0; un < kUnits; ++un)
#pragma unroll
                for (int t = 0; t < kHalves; ++t) mt = fmaxf(mt, z[un][g][t][e]);
#pragma unroll
              for (int d = kApart; d < 32; d <<= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, d));
              anew[g][e] = __fsub_rn(mt, m[g][e]) > 0x1p20f;
              if (anew[g][e]) {
                m[g][e] = ceilf(mt);
                l[g][e] = 0.0f;
                f[g][e] = 0x1p127f;              // no weight so far
              }
            }
        }
#pragma unroll
        for (int g = 0; g < kGroups; ++g)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            // The largest z and z + log2 s, both beside m: a large z has no room for log2 s.
            float mt = kNoMax, ut = kNoMax;
#pragma unroll
            for (int un = 0; un < kUnits; ++un)
#pragma unroll
              for (int t = 0; t < kHalves; ++t) {
                const float zm = __fsub_rn(z[un][g][t][e], m[g][e]);
                mt = fmaxf(mt, zm);
                ut = fmaxf(ut, __fadd_rn(zm, lg2(sv[un][t])));
              }
#pragma unroll
            for (int d = kApart; d < 32; d <<= 1) {
              mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, d));
              ut = fmaxf(ut, __shfl_xor_sync(0xffffffffu, ut, d));
            }
            // log2 f = 7 + m - the largest z + log2 s, that one rounded up
            const float lf = (float)((int)(__float_as_uint(f[g][e]) >> 23) - 127);
            const float m2 = __fadd_rn(m[g][e], fmaxf(0.0f, ceilf(mt))), down = __fsub_rn(m[g][e], m2);
            const float u2 = fmaxf(__fsub_rn(7.0f, lf), ceilf(ut));          // beside the old m
            const float l2 = fminf(fmaxf(__fsub_rn(7.0f, __fadd_rn(u2, down)), -120.0f), 120.0f);
            const float f2 = __uint_as_float((uint32_t)((int)l2 + 127) << 23);
            const float by = anew[g][e] ? 0.0f : ex2(__fadd_rn(down, __fsub_rn(l2, lf)));
            l[g][e] = __fmul_rn(l[g][e], ex2(down));
#pragma unroll
            for (int k = 0; k < 8; ++k) {
              acc[g][k][e] = __fmul_rn(acc[g][k][e], by);
              acc[g][k][2 + e] = __fmul_rn(acc[g][k][2 + e], by);
            }
            m[g][e] = m2;
            f[g][e] = f2;
          }
      }
      // Weights.  With 8 or 16 rows the low parts are the rests themselves and go into the same sums as
      // the high ones; with 4 rows they are 2^11 times the rests, in columns of their own, and a lane has
      // its token's parts and takes the other token's from its partner.
      uint32_t pb[kUnits][kGroups][kHalves][2];  // [unit][group][high, low][token n8, n8 + 8]
#pragma unroll
      for (int un = 0; un < kUnits; ++un)
#pragma unroll
        for (int g = 0; g < kGroups; ++g)
#pragma unroll
          for (int t = 0; t < kHalves; ++t) {
            float p0, p1, w0, w1;
            upk2(sub2(pk2(z[un][g][t][0], z[un][g][t][1]), pk2(m[g][0], m[g][1])), p0, p1);
            const uint64_t p = pk2(ex2(p0), ex2(p1));
            upk2(add2(pk2(l[g][0], l[g][1]), p), l[g][0], l[g][1]);
            upk2(mul2(mul2(p, pk2(sv[un][t], sv[un][t])), pk2(f[g][0], f[g][1])), w0, w1);
            uint32_t hi, lo;
            if constexpr (kWide) {
              split2_plain(w0, w1, hi, lo);
              pb[un][g][0][t] = transpose8(hi);
              pb[un][g][kHalves - 1][t] = transpose8(lo);
            } else {
              split2(w0, w1, hi, lo);
              const uint32_t from = __shfl_xor_sync(0xffffffffu, low ? hi : lo, 2);
              pb[un][g][0][0] = transpose8(low ? from : hi);
              pb[un][g][0][1] = transpose8(low ? lo : from);
            }
          }
      // lane (n8, c4) holds the 16 dimensions of chunk n8 of token pairs c4 and 4 + c4
      uint4 v[kUnits][2];
#pragma unroll
      for (int un = 0; un < kUnits; ++un) {
        v[un][0] = read16(U + un * kUnitBytes + ld_v);
        v[un][1] = read16(U + un * kUnitBytes + ld_v + 512);
      }
#pragma unroll
      for (int w = 0; w < 2; ++w) {
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          const uint32_t pick = hf ? 0x7632u : 0x5410u;
#pragma unroll
          for (int un = 0; un < kUnits; ++un) {
            const uint4 va = v[un][0], vb = v[un][1];
            uint32_t p0[4], p1[4];
            code_pairs(__byte_perm(w ? va.y : va.x, w ? va.w : va.z, pick), factor, p0);
            code_pairs(__byte_perm(w ? vb.y : vb.x, w ? vb.w : vb.z, pick), factor, p1);
#pragma unroll
            for (int t = kHalves - 1; t >= 0; --t)
#pragma unroll
              for (int g = 0; g < kGroups; ++g)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                  mma16816(acc[g][4 * w + 2 * hf + j], p0[2 * j], p0[2 * j + 1], p1[2 * j], p1[2 * j + 1],
                           pb[un][g][t][0], pb[un][g][t][1]);
          }
        }
      }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();                             // every warp's ring is free
    // ---- the block's sums: l over a row's lanes, then the warps
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int d = kApart; d < 32; d <<= 1) l[g][e] = __fadd_rn(l[g][e], __shfl_xor_sync(0xffffffffu, l[g][e], d));
        // dimensions 16 n8 .. + 15 of row e; with 4 rows both lanes of a (high, low) pair form the
        // sums, the high one stores row e0, the low one row e0 + 1
        float *dst = s_acc + (warp * kRows + 8 * g + e0 + e) * kTile + 16 * n8;
        const float f_own = low ? 0.25f : 512.0f, f_other = low ? 512.0f : 0.25f;
#pragma unroll
        for (int k = 0; k < 8; k += 2) {
          float v[4];
#pragma unroll
          for (int d = 0; d < 4; ++d) {
            const float own = acc[g][k + (d >> 1)][2 * (d & 1) + e];
            v[d] = __fmul_rn(own, f_own);
            if (!kWide) v[d] = __fmaf_rn(__shfl_xor_sync(0xffffffffu, own, 2), f_other, v[d]);
            if (d & 1) v[d] = __fmul_rn(__fsub_rn(v[d], v[d - 1]), 0.0625f);
          }
          if (kWide || low == (e == 1)) *reinterpret_cast<float4 *>(dst + 2 * k) = make_float4(v[0], v[1], v[2], v[3]);
        }
        if (n8 == 0 && !low)
          s_stat[warp][8 * g + e0 + e] =
              RowStat{m[g][e], l[g][e], (float)(127 - (int)(__float_as_uint(f[g][e]) >> 23)), 0.0f};
      }
    }
    __syncthreads();
    const bool whole = seg.u_lo == 0 && seg.u_hi == seg.nu;
    if (tid == 0 && seg.u_lo == 0 && !a.whole && (a.by_pair || !whole))      // begun here; ended by later blocks
      joins[a.by_pair ? seg.b * a.c.n_kv * a.row_tiles + seg.pair : blockIdx.x] =
          make_int4((int)(kv4_divide(seg.at_end - 1, piece.size) - blockIdx.x), blockIdx.x, seg.b, seg.pair);
    if (tid < 8 * kRows) {
      float M = kNoMax, E = kNoMax, L = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_stat[w][rr].m);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) E = fmaxf(E, __fadd_rn(__fsub_rn(s_stat[w][rr].m, M), s_stat[w][rr].e));
#pragma unroll
      for (int k = 0; k < 16; ++k) x[k] = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float down = __fsub_rn(s_stat[w][rr].m, M);
        L = __fmaf_rn(s_stat[w][rr].l, ex2(down), L);
        const float by = ex2(__fsub_rn(__fadd_rn(down, s_stat[w][rr].e), E));
        const float4 *src = reinterpret_cast<const float4 *>(s_acc + (w * kRows + rr) * kTile + 16 * r);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float4 v = src[k];
          x[4 * k] = __fmaf_rn(v.x, by, x[4 * k]);
          x[4 * k + 1] = __fmaf_rn(v.y, by, x[4 * k + 1]);
          x[4 * k + 2] = __fmaf_rn(v.z, by, x[4 * k + 2]);
          x[4 * k + 3] = __fmaf_rn(v.w, by, x[4 * k + 3]);
        }
      }
      if (whole) {
        normalize(x, E, L);
        finish_row(a, x, s_tr + rr * kTrTile, r, sign_bits, live,
                   ((int64_t)seg.b * a.q_len + row_j) * a.Hq + row_hq);
        if (live && r == 0) finish_stats(a, seg.b, h, row, M, L);
      } else {
        const int64_t slot = 2 * (int64_t)blockIdx.x + (seg.u_lo == 0 ? 1 : 0);
        float4 *dst = reinterpret_cast<float4 *>(a.part + (slot * kRows + rr) * kTile + 16 * r);
#pragma unroll
        for (int c = 0; c < 4; ++c) dst[c] = make_float4(x[4 * c], x[4 * c + 1], x[4 * c + 2], x[4 * c + 3]);
        if (r == 0) reinterpret_cast<float4 *>(a.stat)[slot * kRows + rr] = make_float4(M, L, E, 0.0f);
      }
    }
    __syncthreads();                             // the ring and the statistics are free
  }
  // rows of sequences without tokens, and lengths out of range
  for (int sb = blockIdx.x; sb < a.c.n_seqs; sb += gridDim.x) {
    bool bad_len;
    const int len = kv4_length(a.c, a.lengths, sb, &bad_len);
    if (bad_len && tid == 0) atomicOr(a.status, (uint32_t)HQ_ERR_PAGE);
    if (len > 0) continue;
    if (a.by_pair && !a.whole)
      for (int i = tid; i < a.c.n_kv * a.row_tiles; i += kAttnThreads)
        joins[sb * a.c.n_kv * a.row_tiles + i] = make_int4(0, 0, 0, 0);
    const int64_t first = (int64_t)sb * a.q_len * a.Hq;
    for (int64_t i = tid >> 3; i < (int64_t)a.q_len * a.Hq; i += kAttnThreads / 8) {
      float zero[16];
#pragma unroll
      for (int k = 0; k < 16; ++k) zero[k] = 0.0f;
      if (a.out_kind == HQ_T_F32) store_row16<HQ_T_F32>(a.out, (first + i) * kTile, tid & 7, true, zero);
      else store_row16<HQ_T_BF16>(a.out, (first + i) * kTile, tid & 7, true, zero);   // the same in fp16
      if ((tid & 7) == 0 && a.lse != nullptr) a.lse[first + i] = -INFINITY;
    }
  }
}

// The sums of a (sequence, head, row tile) that several blocks share, joined
// by WARPS warps a row: each adds every WARPS-th block's sums, in order, a lane four
// dimensions, and the warps' are added in order.  A chain of latencies: what to
// join, the sums, asked for before the largest references are known, the
// transform.  8 warps a row, and more of its sums asked for at once, while all
// rows' blocks fit at once, else one warp: 8 x 4 rows (one sequence of 131072 tokens,
// 57 blocks a row) with 8 sums ahead 34.5 us in all, with 4 36.9, with 32 warps
// 35.5; 128 x 4 rows with 4 ahead 42.7 (attention of 16 ragged sessions of 8192 tokens,
// with mass), with 8 (registers for half the blocks) 44.7, with one warp 44.9;
// 128 x 16 rows (16 x 4096 tokens) with one 40.3, with 8 44.9.  (References in one number then.)
constexpr int kJoinThreads = 256, kJoinWarps = kJoinThreads / 32;
template <int WARPS, int AHEAD>
__global__ void __launch_bounds__(kJoinThreads) kv4_join_kernel(Kv4AttnArgs a, int rows, int items) {
  __shared__ __align__(16) float s_tr[kJoinWarps / WARPS][4 * kTrTile];
  __shared__ __align__(16) float s_x[kJoinWarps][kTile];
  __shared__ float s_l[kJoinWarps];
  follow_launch();                               // launched while that kernel runs
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = warp % WARPS;
  const int item = blockIdx.x * (kJoinWarps / WARPS) + warp / WARPS;
  if (item >= items) return;                     // whole blocks, or warps by themselves
  const int4 job = reinterpret_cast<const int4 *>(a.joins)[item / rows];
  const int rr = item % rows, h = job.w / a.row_tiles, row = (job.w % a.row_tiles) * rows + rr;
  if (job.x == 0 || row >= a.R) return;
  const float4 *stat = reinterpret_cast<const float4 *>(a.stat);
  const auto slot_of = [&](int i) { return (2 * ((int64_t)job.y + i) + (i == 0 ? 1 : 0)) * rows + rr; };
  // A lane's first two references (the last ones again where there are fewer): asked for before the sums
  // by 8 warps, behind them by one (one sequence of 131072 tokens 34.7 us, 35.8 the other way round; 24
  // ragged sessions of 4093 tokens with 16 rows 41.6, 42.5).
  float4 near, far;
  const auto ask = [&] {
    near = stat[slot_of(min(lane, job.x))];
    far = stat[slot_of(min(lane + 32, job.x))];
  };
  if (WARPS > 1) ask();
  float4 s[AHEAD], v[AHEAD];
#pragma unroll
  for (int k = 0; k < AHEAD; ++k) {
    const int i = part + WARPS * k;
    if (i <= job.x) {
      s[k] = stat[slot_of(i)];
      v[k] = reinterpret_cast<const float4 *>(a.part + slot_of(i) * kTile)[lane];
    }
  }
  if (WARPS == 1) ask();
  // RowStat's m and e of the whole row, m first as e is taken beside it
  float M = fmaxf(near.x, far.x), L = 0.0f;
#pragma unroll 4
  for (int i = lane + 64; i <= job.x; i += 32) M = fmaxf(M, stat[slot_of(i)].x);
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
  const auto e_of = [&](const float4 &st) { return __fadd_rn(__fsub_rn(st.x, M), st.z); };
  float E = fmaxf(e_of(near), e_of(far));
#pragma unroll 4
  for (int i = lane + 64; i <= job.x; i += 32) E = fmaxf(E, e_of(stat[slot_of(i)]));
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) E = fmaxf(E, __shfl_xor_sync(0xffffffffu, E, d));
  float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  const auto add = [&](const float4 &st, const float4 &sums) {
    const float down = __fsub_rn(st.x, M);
    L = __fmaf_rn(st.y, ex2(down), L);
    const float f = ex2(__fsub_rn(__fadd_rn(down, st.z), E));
    x.x = __fmaf_rn(sums.x, f, x.x);
    x.y = __fmaf_rn(sums.y, f, x.y);
    x.z = __fmaf_rn(sums.z, f, x.z);
    x.w = __fmaf_rn(sums.w, f, x.w);
  };
#pragma unroll
  for (int k = 0; k < AHEAD; ++k)
    if (part + WARPS * k <= job.x) add(s[k], v[k]);
#pragma unroll 4
  for (int i = part + WARPS * AHEAD; i <= job.x; i += WARPS)
    add(stat[slot_of(i)], reinterpret_cast<const float4 *>(a.part + slot_of(i) * kTile)[lane]);
  reinterpret_cast<float4 *>(s_x[warp])[lane] = x;
  if (WARPS == 1) {
    __syncwarp();
  } else {
    if (lane == 0) s_l[warp] = L;
    __syncthreads();
    float y = 0.0f;
    if (threadIdx.x < kTile) {
#pragma unroll
      for (int w = 0; w < kJoinWarps; ++w) y = __fadd_rn(y, s_x[w][threadIdx.x]);
    }
    __syncthreads();
    if (threadIdx.x < kTile) s_x[0][threadIdx.x] = y;
    __syncthreads();
    if (warp != 0) return;
    L = 0.0f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) L = __fadd_rn(L, s_l[w]);
  }
  const int r = lane & 7;
  float y[16];
#pragma unroll
  for (int c = 0; c < 4; ++c) {
    const float4 q = reinterpret_cast<const float4 *>(s_x[warp] + 16 * r)[c];
    y[4 * c] = q.x; y[4 * c + 1] = q.y; y[4 * c + 2] = q.z; y[4 * c + 3] = q.w;
  }
  normalize(y, E, L);
  const int j = row / a.G, hq = h * a.G + row % a.G;
  const uint32_t sign_bits = a.c.signs[r >> 1] >> (16 * (r & 1));
  finish_row(a, y, s_tr[warp / WARPS] + (lane >> 3) * kTrTile, r, sign_bits, lane < 8,
             ((int64_t)job.z * a.q_len + j) * a.Hq + hq);
  if (lane == 0) finish_stats(a, job.z, h, row, M, L);
}

// mass_out = mass_in + sum over the head's rows of 2^((z - m) - log2 l), rows in order,
// four tokens a thread.  m and log2 l by themselves: in their sum large scores would
// take the bits of log2 l (up to 0.3% of a weight at scores of 10^5).
constexpr int kMassThreads = 256;
__global__ void __launch_bounds__(kMassThreads) kv4_mass_kernel(Kv4AttnArgs a) {
  follow_launch();
  const int h = blockIdx.y, b = blockIdx.z;
  const int64_t t = ((int64_t)blockIdx.x * kMassThreads + threadIdx.x) * 4;
  bool bad;
  const int len = kv4_length(a.c, a.lengths, b, &bad);
  if (t >= len) return;
  const int64_t head = (int64_t)b * a.c.n_kv + h, cap = a.c.capacity();   // a multiple of 16
  const float *z = a.z + head * a.R * cap + t;
  const float2 *stat = a.row_stat + head * a.R;
  float s[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 4
  for (int row = 0; row < a.R; ++row) {
    const float4 v = *reinterpret_cast<const float4 *>(z + row * cap);
    const float2 ml = stat[row];
    const float x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (x[k] > -INFINITY || x[k] != x[k]) s[k] = __fadd_rn(s[k], ex2(__fsub_rn(__fsub_rn(x[k], ml.x), ml.y)));
  }
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    if (t + k >= len) break;
    const int64_t at = head * cap + t + k;
    a.mass_out[at] = a.mass_in != nullptr ? __fadd_rn(a.mass_in[at], s[k]) : s[k];
  }
}

// Resident blocks of the attention kernel on the current device (asked once
// per instance and device).
template <int ROWS, bool CAP, bool MASS>
int resident_blocks() {
  static int cache[64] = {};
  int dev = 0, sms = 0, per_sm = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev >= 0 && dev < 64 && cache[dev] > 0) return cache[dev];
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (cudaFuncSetAttribute(kv4_attn_kernel<ROWS, CAP, MASS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           Shape<ROWS>::smem) != cudaSuccess)
    return 0;
  cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kv4_attn_kernel<ROWS, CAP, MASS>, kAttnThreads,
                                                Shape<ROWS>::smem);
  const int n = sms * per_sm;
  if (dev >= 0 && dev < 64) cache[dev] = n;
  return n;
}

template <int ROWS, bool CAP, bool MASS>
int launch_attn(const Kv4AttnArgs &a, cudaStream_t st) {
  int grid = resident_blocks<ROWS, CAP, MASS>();
  if (grid <= 0) return 1;
  if (grid > kKv4MaxBlocks) grid = kKv4MaxBlocks;
  // no more blocks than pieces of the longest batch the table allows
  const int64_t pairs = (int64_t)a.c.n_seqs * a.c.n_kv * a.row_tiles;
  int64_t most = ((a.c.capacity() / kUnit + kSegmentCost) * pairs + kMinPiece - 1) / kMinPiece;
  if (most < pairs) most = pairs;
  if (most < grid) grid = (int)most;
  Kv4AttnArgs w = a;
  w.whole = pairs <= grid && a.c.capacity() / kUnit + kSegmentCost <= kWholeSpan;
  if (w.whole) grid = (int)pairs;
  w.by_pair = pairs <= grid;
  if (launch_behind(kv4_attn_kernel<ROWS, CAP, MASS>, dim3((unsigned)grid), kAttnThreads, Shape<ROWS>::smem, st, w) != 0)
    return 1;
  if (w.whole) return 0;                         // nothing to join
  const int items = (w.by_pair ? (int)pairs : grid) * ROWS;
  const auto join = [&](auto kernel, int a_block) {
    return launch_behind(kernel, dim3((unsigned)((items + a_block - 1) / a_block)), kJoinThreads, 0, st, a, ROWS, items);
  };
  if (items <= 2 * 152) return join(kv4_join_kernel<8, 8>, 1);
  if (items <= 4 * 152) return join(kv4_join_kernel<8, 4>, 1);
  return join(kv4_join_kernel<1, 4>, kJoinWarps);
}

template <int ROWS>
int launch_rows(const Kv4AttnArgs &a, cudaStream_t st) {
  const bool mass = a.mass_out != nullptr;
  if (a.cap > 0.0f) return mass ? launch_attn<ROWS, true, true>(a, st) : launch_attn<ROWS, true, false>(a, st);
  return mass ? launch_attn<ROWS, false, true>(a, st) : launch_attn<ROWS, false, false>(a, st);
}

int rows_a_block(int R) { return R <= 4 ? 4 : R <= 8 ? 8 : 16; }

}  // namespace

int kv4_row_tiles(int R) { return (R + rows_a_block(R) - 1) / rows_a_block(R); }
size_t kv4_part_bytes(int R) { return (size_t)2 * kKv4MaxBlocks * rows_a_block(R) * kTile * sizeof(float); }
size_t kv4_stat_bytes(int R) { return (size_t)2 * kKv4MaxBlocks * rows_a_block(R) * sizeof(float4); }
size_t kv4_join_bytes() { return (size_t)kKv4MaxBlocks * sizeof(int4); }

int launch_kv4_attention(const Kv4AttnArgs &a, cudaStream_t st) {
  const int rows = rows_a_block(a.R);
  const int rc = rows == 4 ? launch_rows<4>(a, st) : rows == 8 ? launch_rows<8>(a, st) : launch_rows<16>(a, st);
  if (rc != 0) return rc;
  if (a.mass_out != nullptr && a.c.capacity() > 0)
    return launch_behind(kv4_mass_kernel,
                         dim3((unsigned)((a.c.capacity() + 4 * kMassThreads - 1) / (4 * kMassThreads)),
                              (unsigned)a.c.n_kv, (unsigned)a.c.n_seqs), kMassThreads, 0, st, a);
  return 0;
}

}  // namespace hq

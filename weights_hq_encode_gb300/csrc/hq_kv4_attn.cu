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
#include "hq_umma.cuh"

namespace hq {

namespace {

constexpr float kInvRoot128 = 0.08838834764831845f;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kLoScale = 2048.0f, kInvLoScale = 0x1p-11f;
constexpr float kNoMax = -3.0e38f;               // below every finite score

constexpr int kWarps = 4;                        // warps of a block
constexpr int kAttnThreads = 32 * kWarps;
constexpr int kStages = 4;                       // units a warp has in its ring
constexpr int kRingBytes = kWarps * kStages * kUnitBytes;
// NC column groups of 8: the high and the low parts of 4 query rows each
template <int NC>
struct Shape {
  static constexpr int rows = 4 * NC;            // query rows of a block
  static constexpr int q_bytes = 8 * NC * 32 * 8;   // query fragments: 8 K steps, 8 bytes a lane
  static constexpr int sum_bytes = kWarps * rows * kTile * 4;   // the warps' sums, in the ring's place
  static constexpr int ring = kRingBytes > sum_bytes ? kRingBytes : sum_bytes;
  static constexpr int smem = ring + q_bytes + rows * kTrTile * 4;
  static constexpr int blocks = NC == 1 ? 4 : 3; // resident blocks a multiprocessor
};

// Work of one (sequence, head, row tile) beyond its units, in units: the
// blocks split the batch into equal pieces of units + kSegmentCost.
constexpr int kSegmentCost = 8, kMinPiece = 16;

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
// The exponents under which a nibble becomes an fp16 value, in registers that
// the compiler does not fill again at every use.
struct Magic {
  uint32_t low, high;       // 1024 (nibble in bits 0-3), 64 (bits 4-7), twice each
};
__device__ __forceinline__ Magic make_magic() {
  Magic g;
  asm volatile("mov.b32 %0, 0x64006400;" : "=r"(g.low));
  asm volatile("mov.b32 %0, 0x54005400;" : "=r"(g.high));
  return g;
}
// (x & MASK) | bits as two fp16 values, less MINUS.
template <uint32_t MASK, uint32_t MINUS>
__device__ __forceinline__ uint32_t codes2(uint32_t x, uint32_t bits) {
  uint32_t y;
  asm("lop3.b32 %0, %1, %2, %3, 0xEA;" : "=r"(y) : "r"(x), "n"(MASK), "r"(bits));
  asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(y) : "r"(y), "r"(MINUS));
  return y;
}
// Four pairs of codes less 8 as fp16: pair i is nibble i of the low and of
// the high half of x.  Under the exponents above a nibble is 1024 + c or
// 64 + c exactly.
__device__ __forceinline__ void unpack_pairs(uint32_t x, const Magic &g, uint32_t p[4]) {
  const uint32_t y = x >> 8;
  p[0] = codes2<0x000F000Fu, 0x64086408u>(x, g.low);    // 1032
  p[1] = codes2<0x00F000F0u, 0x54805480u>(x, g.high);   // 72
  p[2] = codes2<0x000F000Fu, 0x64086408u>(y, g.low);
  p[3] = codes2<0x00F000F0u, 0x54805480u>(y, g.high);
}
__device__ __forceinline__ void mma16816(float d[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a));
  return v;
}
__device__ __forceinline__ float lds_bf16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
  return __uint_as_float((uint32_t)v << 16);
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
  const float r0 = __fmul_rn(__fsub_rn(lo, f.x), kLoScale), r1 = __fmul_rn(__fsub_rn(hi, f.y), kLoScale);
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(rest) : "f"(r1), "f"(r0));
}

template <int KIND>
__device__ __forceinline__ void load_q16(const Kv4AttnArgs &a, int64_t at, int r, float x[16]) {
  load_row16<KIND>(a.q, at, r, a.q_vec != 0, x);
}

// 16 lanes of one row out, D H x / sqrt(128) applied: the last step of every
// row.  All 32 lanes of the warp must call it.
__device__ __forceinline__ void finish_row(const Kv4AttnArgs &a, float x[16], float *tile, int r,
                                           bool live, int64_t o) {
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = __fmul_rn(x[i], kInvRoot128);
  fwht128_t8(x, tile, r);
  if (!live) return;
  const uint32_t mw = __ldg(a.c.signs + (r >> 1)) >> (16 * (r & 1));
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = __uint_as_float(__float_as_uint(x[i]) ^ (((mw >> i) & 1u) << 31));
  if (a.out_kind == HQ_T_F32) store_row16<HQ_T_F32>(a.out, o * kTile, r, true, x);
  else if (a.out_kind == HQ_T_F16) store_row16<HQ_T_F16>(a.out, o * kTile, r, true, x);
  else store_row16<HQ_T_BF16>(a.out, o * kTile, r, true, x);
}

// A row's sums over some of its tokens: l = sum 2^(z - m), and acc (kept
// beside it) = sum 2^(z + log2 s - mw) (c - 7.5).
struct RowStat {
  float m, l, mw, pad;
};

// acc / l at its own references: x 2^mw / (l 2^m), zeros where there is no weight.
__device__ __forceinline__ void normalize(float x[16], float m, float mw, float l) {
  const float f = ex2(__fmul_rn(__fsub_rn(mw, m), 0.5f));   // in two steps, each within range
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = l == 0.0f ? 0.0f : __fmul_rn(__fmul_rn(__fdiv_rn(x[i], l), f), f);
}

__device__ __forceinline__ void finish_stats(const Kv4AttnArgs &a, int b, int h, int row, float M, float L) {
  const float l2 = L == 0.0f ? -INFINITY : __fadd_rn(M, log2f(L));
  const int j = row / a.G, hq = h * a.G + row % a.G;
  if (a.lse != nullptr) a.lse[((int64_t)b * a.q_len + j) * a.Hq + hq] = __fmul_rn(l2, kLn2);
  if (a.mass_out != nullptr) a.row_lse[((int64_t)b * a.c.n_kv + h) * a.R + row] = l2;
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

__device__ Piece find_piece(const Kv4AttnArgs &a) {
  __shared__ int64_t s_sum[kWarps];
  __shared__ int64_t s_begin;
  __shared__ int s_b;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int B = a.c.n_seqs;
  Piece p;
  int64_t total = 0;
  for (int b = tid; b < B; b += kAttnThreads) total += span_of(a, b);
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) total += __shfl_xor_sync(0xffffffffu, total, d);
  if (lane == 0) s_sum[warp] = total;
  if (tid == 0) s_b = B;
  __syncthreads();
  total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) total += s_sum[w];
  const int64_t even = (total + gridDim.x - 1) / gridDim.x;
  p.size = even > kMinPiece ? even : kMinPiece;
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

// Each warp of a block takes every fourth unit of a segment (the units of one
// sequence and head that fall into the block's piece) through a ring of its
// own in shared memory, filled by asynchronous copies, and keeps its own sums;
// the four are added at the segment's end.  A segment that is a whole
// (sequence, head) is finished here, the others leave their sums for
// kv4_join_kernel.
//
// The products run on mma.sync m16n8k16, tokens (scores) and dimensions
// (values) as the 16 rows and query rows as the 8 columns: columns 0 .. 3 the
// high parts of 4 rows, columns 4 .. 7 their low parts, so that the fp32-level
// split of 4 rows fills one instruction.  The codes are unpacked in registers,
// straight into operand fragments; that is why these are not tcgen05
// products, whose operands would first have to be stored to shared memory as
// fp16, four times the bytes that were read.
template <int NC, bool CAP, bool MASS>
__global__ void __launch_bounds__(kAttnThreads, Shape<NC>::blocks) kv4_attn_kernel(Kv4AttnArgs a) {
  constexpr int kRows = Shape<NC>::rows;
  extern __shared__ __align__(128) unsigned char s_mem[];
  __shared__ RowStat s_stat[kWarps][kRows];
  __shared__ float s_mul[kRows], s_half[kRows];  // multiplier of the scores, sum q' / 2
  __shared__ int s_seen[kRows];                  // tokens seen
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int n8 = lane >> 2, c4 = lane & 3;       // fragment row group, and place in it
  const bool low = c4 >= 2;                      // this lane's columns are low parts
  const int e0 = 2 * (c4 & 1);                   // its rows of a column group: e0, e0 + 1
  uint2 *const s_q = reinterpret_cast<uint2 *>(s_mem + Shape<NC>::ring);
  float *const s_tr = reinterpret_cast<float *>(s_mem + Shape<NC>::ring + Shape<NC>::q_bytes);
  const uint32_t ring_a = smem_addr(s_mem) + warp * kStages * kUnitBytes;
  // copies: 16 bytes a lane and 512-byte quarter; V's chunks are permuted
  // inside their 128-byte rows so that the reads below touch all banks
  const uint32_t cp_k = lane * 16, cp_v = kUnitV + (lane >> 3) * 128 + (((lane & 7) ^ (2 * (lane >> 3))) * 16);
  const uint32_t ld_v = kUnitV + c4 * 128 + ((n8 ^ (2 * c4)) * 16);
  const Magic magic = make_magic();
  const float k_own = low ? kInvLoScale : 1.0f, k_other = low ? 1.0f : kInvLoScale;
  const Piece piece = find_piece(a);
  int join_b = 0, join_count = 0, join_pair = 0;
  int64_t cur = piece.begin;
  int b = piece.b;
  int64_t b_begin = piece.b_begin;
  while (cur < piece.end) {                      // block-uniform throughout
    const int nu = units_of(a, b), span1 = nu + kSegmentCost;
    const int64_t b_end = b_begin + (nu == 0 ? 0 : (int64_t)a.c.n_kv * a.row_tiles * span1);
    if (cur >= b_end) {
      ++b;
      b_begin = b_end;
      continue;
    }
    const int pair = (int)((cur - b_begin) / span1);        // head and row tile of sequence b
    const int64_t at = b_begin + (int64_t)pair * span1;     // where the pair begins
    const int u_lo = (int)max((int64_t)0, cur - at - kSegmentCost);
    const int u_hi = (int)min((int64_t)nu, piece.end - at - kSegmentCost);
    cur = min(at + span1, piece.end);
    if (u_lo >= u_hi) continue;
    const int h = pair / a.row_tiles, row0 = (pair % a.row_tiles) * kRows;
    bool bad_len;
    const int len = kv4_length(a.c, a.lengths, b, &bad_len);

    // ---- this warp's units u_lo + warp, u_lo + warp + 4, ..: the ring's first copies
    const int mine = (u_hi - u_lo - warp + kWarps - 1) / kWarps;
    int where_now = -1, where_next = -1;         // unit numbers in the pool of 32 of this warp's units
    const auto look_up = [&](int first) {
      const int i = first + lane;
      if (i >= mine) return -1;
      const int u = u_lo + warp + kWarps * i, pj = u / a.c.page_units;
      const int page = __ldg(a.c.table + (int64_t)b * a.c.width + pj);
      return page >= 0 && page < a.c.n_pages ? (page * a.c.n_kv + h) * a.c.page_units + u - pj * a.c.page_units
                                             : -1;
    };
    int issued = 0, put = 0;                     // units asked for, and the stage of the next
    uint32_t bad_stages = 0;                     // stages whose unit has no page
    const auto issue = [&]() {                   // the next unit into its stage; one group, maybe empty
      if (issued < mine) {
        if ((issued & 31) == 0) {
          where_now = issued == 0 ? look_up(0) : where_next;
          where_next = look_up(issued + 32);
        }
        const int unit = __shfl_sync(0xffffffffu, where_now, issued & 31);
        bad_stages &= ~(1u << put);
        if (unit >= 0) {
          const unsigned char *src = a.c.pages + (int64_t)unit * kUnitBytes + lane * 16;
          const uint32_t dst = ring_a + put * kUnitBytes;
          cp_async16(dst + cp_k, src);
          cp_async16(dst + cp_k + 512, src + 512);
          cp_async16(dst + cp_v, src + kUnitV);
          cp_async16(dst + cp_v + 512, src + kUnitV + 512);
          if (lane < 4) cp_async16(dst + kUnitKs + lane * 16, src + kUnitKs);
        } else {
          bad_stages |= 1u << put;
        }
        ++issued;
        put = put == kStages - 1 ? 0 : put + 1;
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) issue();

    // ---- the query rows: rotated, scaled by a power of two, split, as mma fragments
    if (tid < 8 * kRows) {
      const int rr = tid >> 3, r = tid & 7, row = row0 + rr;
      const bool live = row < a.R;
      const int j = live ? row / a.G : 0, hq = live ? h * a.G + row % a.G : 0;
      float x[16];
      if (live) {
        const int64_t qa = b * a.q_seq + j * a.q_token + hq * a.q_head;
        if (a.kind == HQ_T_F32) load_q16<HQ_T_F32>(a, qa, r, x);
        else if (a.kind == HQ_T_F16) load_q16<HQ_T_F16>(a, qa, r, x);
        else load_q16<HQ_T_BF16>(a, qa, r, x);
      }
      const uint32_t mw = __ldg(a.c.signs + (r >> 1)) >> (16 * (r & 1));
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float v = live ? x[i] : 0.0f;
        x[i] = __fmul_rn(__uint_as_float(__float_as_uint(v) ^ (((mw >> i) & 1u) << 31)), kInvRoot128);
      }
      fwht128_t8(x, s_tr + rr * kTrTile, r);
      float top = 0.0f, sum = 0.0f;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        top = fmaxf(top, fabsf(x[i]));
        sum = __fadd_rn(sum, x[i]);
      }
#pragma unroll
      for (int d = 1; d < 8; d <<= 1) {
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
        sum = __fadd_rn(sum, __shfl_xor_sync(0xffffffffu, sum, d));
      }
      const float sc = scale_of(top), inv = inv_scale_of(top);
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = __fmul_rn(x[i], sc);
      // lane r holds words 2 (r & 1), 2 (r & 1) + 1 of the 32 dimensions of place r / 2; row rr is
      // columns rr % 4 (high parts) and rr % 4 + 4 (low parts) of group rr / 4
#pragma unroll
      for (int w = 0; w < 2; ++w) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint2 hi, lo;
          split2(x[8 * w + 2 * i], x[8 * w + 2 * i + 4], hi.x, lo.x);
          split2(x[8 * w + 2 * i + 1], x[8 * w + 2 * i + 5], hi.y, lo.y);
          uint2 *dst = s_q + ((2 * (2 * (r & 1) + w) + i) * NC + (rr >> 2)) * 32 + (rr & 3) * 4 + (r >> 1);
          dst[0] = hi;
          dst[16] = lo;
        }
      }
      if (r == 0) {
        s_mul[rr] = CAP ? __fmul_rn(__fdiv_rn(a.scale, a.cap), inv) : __fmul_rn(__fmul_rn(a.scale, kLog2e), inv);
        s_half[rr] = __fmul_rn(__fmul_rn(sum, sc), 0.5f);
        s_seen[rr] = max(0, len - a.q_len + j + 1);
      }
    }
    __syncthreads();
    uint2 qb[8][NC];
    uint64_t zmul[NC];
    float q0[NC][2];
#pragma unroll
    for (int k = 0; k < 8; ++k)
#pragma unroll
      for (int g = 0; g < NC; ++g) qb[k][g] = s_q[(k * NC + g) * 32 + lane];
#pragma unroll
    for (int g = 0; g < NC; ++g) {
      zmul[g] = pk2(s_mul[4 * g + e0], s_mul[4 * g + e0 + 1]);
      q0[g][0] = low ? 0.0f : s_half[4 * g + e0];
      q0[g][1] = low ? 0.0f : s_half[4 * g + e0 + 1];
    }
    const int seen_all = len - a.q_len + row0 / a.G + 1;    // the least of any row here
    const float cap_l2 = CAP ? __fmul_rn(a.cap, kLog2e) : 0.0f;

    // ---- the units
    float acc[NC][8][4], l[NC][2], wsum[NC][2], m[NC][2], mw[NC][2];
#pragma unroll
    for (int g = 0; g < NC; ++g) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[g][i][e] = 0.0f;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        l[g][e] = wsum[g][e] = 0.0f;
        m[g][e] = mw[g][e] = kNoMax;
      }
    }
    int get = 0;                                 // stage of the next unit to use
    int t0 = (u_lo + warp) * kUnit;
    for (int it = 0; it < mine; ++it, t0 += kWarps * kUnit) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
      __syncwarp();                              // unit `it` has come, and unit `it` - 1 is used up
      issue();
      const uint32_t U = ring_a + get * kUnitBytes;
      const bool bad = (bad_stages >> get) & 1u;
      get = get == kStages - 1 ? 0 : get + 1;
      // scores: lane (n8, c4) gets tokens n8 and n8 + 8, columns 2 c4, 2 c4 + 1
      float s[NC][4];
#pragma unroll
      for (int g = 0; g < NC; ++g) {
        s[g][0] = s[g][2] = q0[g][0];
        s[g][1] = s[g][3] = q0[g][1];
      }
      {
        const uint4 k0 = lds128(U + cp_k), k1 = lds128(U + cp_k + 512);
        const uint32_t w0[4] = {k0.x, k0.y, k0.z, k0.w}, w1[4] = {k1.x, k1.y, k1.z, k1.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t p0[4], p1[4];
          unpack_pairs(w0[j], magic, p0);
          unpack_pairs(w1[j], magic, p1);
#pragma unroll
          for (int g = 0; g < NC; ++g) {
            mma16816(s[g], p0[0], p1[0], p0[1], p1[1], qb[2 * j][g].x, qb[2 * j][g].y);
            mma16816(s[g], p0[2], p1[2], p0[3], p1[3], qb[2 * j + 1][g].x, qb[2 * j + 1][g].y);
          }
        }
      }
      const float sk[2] = {lds_bf16(U + kUnitKs + 2 * n8), lds_bf16(U + kUnitKs + 2 * n8 + 16)};
      const float ls[2] = {lg2(lds_bf16(U + kUnitVs + 2 * n8)), lg2(lds_bf16(U + kUnitVs + 2 * n8 + 16))};
      float z[NC][2][2], u[NC][2][2];            // [group][token][row]
#pragma unroll
      for (int g = 0; g < NC; ++g)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const float o0 = __shfl_xor_sync(0xffffffffu, s[g][2 * t], 2);
          const float o1 = __shfl_xor_sync(0xffffffffu, s[g][2 * t + 1], 2);
          const uint64_t d = fma2(pk2(o0, o1), pk2(k_other, k_other),
                                  mul2(pk2(s[g][2 * t], s[g][2 * t + 1]), pk2(k_own, k_own)));
          upk2(mul2(mul2(d, pk2(sk[t], sk[t])), zmul[g]), z[g][t][0], z[g][t][1]);
          if (CAP) {                             // cap tanh(y) = cap (1 - 2 / (1 + e^2|y|)), y's sign
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const float y = z[g][t][e], x = ex2(__fmul_rn(fabsf(y), 2.0f * kLog2e));
              z[g][t][e] = copysignf(
                  __fmul_rn(cap_l2, __fsub_rn(1.0f, __fdividef(2.0f, __fadd_rn(x, 1.0f)))), y);
            }
          }
          upk2(add2(pk2(z[g][t][0], z[g][t][1]), pk2(ls[t], ls[t])), u[g][t][0], u[g][t][1]);
        }
      if (t0 + kUnit > seen_all || bad) {        // warp-uniform: some token is not seen by some row
#pragma unroll
        for (int g = 0; g < NC; ++g)
#pragma unroll
          for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int e = 0; e < 2; ++e)
              if (bad || t0 + 8 * t + n8 >= s_seen[4 * g + e0 + e]) z[g][t][e] = u[g][t][e] = -INFINITY;
        if (bad && lane == 0) atomicOr(a.status, (uint32_t)HQ_ERR_PAGE);
      }
      if (MASS && !low) {
#pragma unroll
        for (int g = 0; g < NC; ++g)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int row = row0 + 4 * g + e0 + e;
            if (row >= a.R) continue;
            float *zrow = a.z + (((int64_t)b * a.c.n_kv + h) * a.R + row) * a.c.capacity() + t0 + n8;
            zrow[0] = z[g][0][e];
            zrow[8] = z[g][1][e];
          }
      }
      // p = 2^(z - m) stays below 2^64 and a weight w = 2^(z + log2 s - mw) below 2^15 without
      // moving the references m and mw at every unit
      float pe[NC][2][2], we[NC][2][2];
#pragma unroll
      for (int pass = 0; pass < 2; ++pass) {
        float pt = kNoMax, wt = kNoMax;
#pragma unroll
        for (int g = 0; g < NC; ++g)
#pragma unroll
          for (int t = 0; t < 2; ++t) {
            upk2(sub2(pk2(z[g][t][0], z[g][t][1]), pk2(m[g][0], m[g][1])), pe[g][t][0], pe[g][t][1]);
            upk2(sub2(pk2(u[g][t][0], u[g][t][1]), pk2(mw[g][0], mw[g][1])), we[g][t][0], we[g][t][1]);
            pt = fmaxf(pt, fmaxf(pe[g][t][0], pe[g][t][1]));
            wt = fmaxf(wt, fmaxf(we[g][t][0], we[g][t][1]));
          }
        if (pass == 1 || !__any_sync(0xffffffffu, pt > 64.0f || wt > 15.0f)) break;
#pragma unroll
        for (int g = 0; g < NC; ++g) {
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float zt = fmaxf(z[g][0][e], z[g][1][e]), ut = fmaxf(u[g][0][e], u[g][1][e]);
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) {
              zt = fmaxf(zt, __shfl_xor_sync(0xffffffffu, zt, d));
              ut = fmaxf(ut, __shfl_xor_sync(0xffffffffu, ut, d));
            }
            const float m2 = fmaxf(m[g][e], zt), mw2 = fmaxf(mw[g][e], __fsub_rn(ut, 7.0f));
            const float f = ex2(__fsub_rn(mw[g][e], mw2));
            l[g][e] = __fmul_rn(l[g][e], ex2(__fsub_rn(m[g][e], m2)));
            wsum[g][e] = __fmul_rn(wsum[g][e], f);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              acc[g][i][e] = __fmul_rn(acc[g][i][e], f);
              acc[g][i][2 + e] = __fmul_rn(acc[g][i][2 + e], f);
            }
            m[g][e] = m2;
            mw[g][e] = mw2;
          }
        }
      }
      uint32_t pb[NC][2];
#pragma unroll
      for (int g = 0; g < NC; ++g)
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          const float w0 = ex2(we[g][t][0]), w1 = ex2(we[g][t][1]);
          uint32_t hi, lo;
          split2(w0, w1, hi, lo);
          pb[g][t] = transpose8(low ? lo : hi);
          upk2(add2(pk2(l[g][0], l[g][1]), pk2(ex2(pe[g][t][0]), ex2(pe[g][t][1]))), l[g][0], l[g][1]);
          upk2(add2(pk2(wsum[g][0], wsum[g][1]), pk2(w0, w1)), wsum[g][0], wsum[g][1]);
        }
      // values: lane (n8, c4) holds the 16 dimensions of chunk n8 of token pairs c4 and 4 + c4
      const uint4 v0 = lds128(U + ld_v), v1 = lds128(U + ld_v + 512);
      const uint32_t a0[2] = {v0.x, v0.y}, b0[2] = {v0.z, v0.w}, a1[2] = {v1.x, v1.y}, b1[2] = {v1.z, v1.w};
#pragma unroll
      for (int w = 0; w < 2; ++w) {
#pragma unroll
        for (int hf = 0; hf < 2; ++hf) {
          uint32_t p0[4], p1[4];
          unpack_pairs(__byte_perm(a0[w], b0[w], hf ? 0x7632 : 0x5410), magic, p0);
          unpack_pairs(__byte_perm(a1[w], b1[w], hf ? 0x7632 : 0x5410), magic, p1);
#pragma unroll
          for (int g = 0; g < NC; ++g) {
            mma16816(acc[g][4 * w + 2 * hf], p0[0], p0[1], p1[0], p1[1], pb[g][0], pb[g][1]);
            mma16816(acc[g][4 * w + 2 * hf + 1], p0[2], p0[3], p1[2], p1[3], pb[g][0], pb[g][1]);
          }
        }
      }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    // ---- the block's sums: l and the weights' sum over a row's lanes, then the four warps
    __syncthreads();                             // every warp's ring is free
    float *const s_acc = reinterpret_cast<float *>(s_mem);
#pragma unroll
    for (int g = 0; g < NC; ++g) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) {
          l[g][e] = __fadd_rn(l[g][e], __shfl_xor_sync(0xffffffffu, l[g][e], d));
          wsum[g][e] = __fadd_rn(wsum[g][e], __shfl_xor_sync(0xffffffffu, wsum[g][e], d));
        }
        // dimensions 16 n8 .. + 15 of row e: both lanes of a (high, low) pair form the sums, the
        // high one stores row e0, the low one row e0 + 1
        float *dst = s_acc + (warp * kRows + 4 * g + e0 + e) * kTile + 16 * n8;
        const float half = __fmul_rn(wsum[g][e], 0.5f);
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
          float v[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float own = acc[g][i + (k >> 1)][2 * (k & 1) + e];
            const float other = __shfl_xor_sync(0xffffffffu, own, 2);
            v[k] = __fadd_rn(__fmaf_rn(other, k_other, __fmul_rn(own, k_own)), half);
          }
          if (low == (e == 1)) *reinterpret_cast<float4 *>(dst + 2 * i) = make_float4(v[0], v[1], v[2], v[3]);
        }
        if (n8 == 0 && !low) s_stat[warp][4 * g + e0 + e] = RowStat{m[g][e], l[g][e], mw[g][e], 0.0f};
      }
    }
    __syncthreads();
    const bool whole = u_lo == 0 && u_hi == nu;
    if (!whole && u_lo == 0) {                   // begun here, ended by later blocks
      join_b = b;
      join_pair = pair;
      join_count = (int)((at + span1 - 1) / piece.size - blockIdx.x);
    }
    if (tid < 8 * kRows) {
      const int rr = tid >> 3, r = tid & 7, row = row0 + rr;
      float M = kNoMax, MW = kNoMax, L = 0.0f, x[16];
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        M = fmaxf(M, s_stat[w][rr].m);
        MW = fmaxf(MW, s_stat[w][rr].mw);
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = 0.0f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        L = __fmaf_rn(s_stat[w][rr].l, ex2(__fsub_rn(s_stat[w][rr].m, M)), L);
        const float f = ex2(__fsub_rn(s_stat[w][rr].mw, MW));
        const float *src = s_acc + (w * kRows + rr) * kTile + 16 * r;
#pragma unroll
        for (int i = 0; i < 16; ++i) x[i] = __fmaf_rn(src[i], f, x[i]);
      }
      if (whole) {
        const bool live = row < a.R;
        normalize(x, M, MW, L);
        const int j = row / a.G, hq = h * a.G + row % a.G;
        finish_row(a, x, s_tr + rr * kTrTile, r, live, ((int64_t)b * a.q_len + j) * a.Hq + hq);
        if (live && r == 0) finish_stats(a, b, h, row, M, L);
      } else {
        const int64_t slot = 2 * (int64_t)blockIdx.x + (u_lo == 0 ? 1 : 0);
        float4 *dst = reinterpret_cast<float4 *>(a.part + (slot * kRows + rr) * kTile + 16 * r);
#pragma unroll
        for (int c = 0; c < 4; ++c) dst[c] = make_float4(x[4 * c], x[4 * c + 1], x[4 * c + 2], x[4 * c + 3]);
        if (r == 0) reinterpret_cast<float4 *>(a.stat)[slot * kRows + rr] = make_float4(M, L, MW, 0.0f);
      }
    }
    __syncthreads();                             // the ring, the rows and the statistics are free
  }
  if (tid == 0) reinterpret_cast<int4 *>(a.joins)[blockIdx.x] = make_int4(join_count, join_b, join_pair, 0);
  // rows of sequences without tokens, and lengths out of range
  for (int64_t i = (int64_t)blockIdx.x * (kAttnThreads / 8) + (tid >> 3); i < (int64_t)a.c.n_seqs * a.q_len * a.Hq;
       i += (int64_t)gridDim.x * (kAttnThreads / 8)) {
    const int sb = (int)(i / ((int64_t)a.q_len * a.Hq));
    bool bad_len;
    const int len = kv4_length(a.c, a.lengths, sb, &bad_len);
    if (bad_len && (tid & 7) == 0) atomicOr(a.status, (uint32_t)HQ_ERR_PAGE);
    if (len > 0) continue;
    float x[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) x[k] = 0.0f;
    if (a.out_kind == HQ_T_F32) store_row16<HQ_T_F32>(a.out, i * kTile, tid & 7, true, x);
    else store_row16<HQ_T_BF16>(a.out, i * kTile, tid & 7, true, x);   // zeros are the same in fp16
    if ((tid & 7) == 0 && a.lse != nullptr) a.lse[i] = -INFINITY;
  }
}

// The sums of a (sequence, head, row tile) that several blocks share: block
// (i, row) joins that row of what block i of the attention kernel began.  Each
// of the four warps adds every fourth block's sums, in order, a lane four
// dimensions; the four are added in order.
constexpr int kJoinThreads = 128;
__global__ void __launch_bounds__(kJoinThreads) kv4_join_kernel(Kv4AttnArgs a, int rows) {
  __shared__ __align__(16) float s_tr[4 * kTrTile];
  __shared__ __align__(16) float s_x[kJoinThreads / 32][kTile];
  __shared__ float s_l[kJoinThreads / 32];
  const int4 job = reinterpret_cast<const int4 *>(a.joins)[blockIdx.x];
  const int rr = blockIdx.y, h = job.z / a.row_tiles, row = (job.z % a.row_tiles) * rows + rr;
  if (job.x == 0 || row >= a.R) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const float4 *stat = reinterpret_cast<const float4 *>(a.stat);
  const auto slot_of = [&](int i) { return 2 * ((int64_t)blockIdx.x + i) + (i == 0 ? 1 : 0); };
  float M = kNoMax, MW = kNoMax, L = 0.0f;
  for (int i = lane; i <= job.x; i += 32) {
    const float4 s = stat[slot_of(i) * rows + rr];
    M = fmaxf(M, s.x);
    MW = fmaxf(MW, s.z);
  }
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) {
    M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
    MW = fmaxf(MW, __shfl_xor_sync(0xffffffffu, MW, d));
  }
  float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int i = warp; i <= job.x; i += kJoinThreads / 32) {
    const float4 s = stat[slot_of(i) * rows + rr];
    const float4 v = reinterpret_cast<const float4 *>(a.part + (slot_of(i) * rows + rr) * kTile)[lane];
    L = __fmaf_rn(s.y, ex2(__fsub_rn(s.x, M)), L);
    const float f = ex2(__fsub_rn(s.z, MW));
    x.x = __fmaf_rn(v.x, f, x.x);
    x.y = __fmaf_rn(v.y, f, x.y);
    x.z = __fmaf_rn(v.z, f, x.z);
    x.w = __fmaf_rn(v.w, f, x.w);
  }
  reinterpret_cast<float4 *>(s_x[warp])[lane] = x;
  if (lane == 0) s_l[warp] = L;
  __syncthreads();
  if (warp != 0) return;
  const int r = lane & 7;
  float y[16];
  L = 0.0f;
#pragma unroll
  for (int i = 0; i < 16; ++i) y[i] = 0.0f;
#pragma unroll
  for (int w = 0; w < kJoinThreads / 32; ++w) {
    L = __fadd_rn(L, s_l[w]);
#pragma unroll
    for (int i = 0; i < 16; ++i) y[i] = __fadd_rn(y[i], s_x[w][16 * r + i]);
  }
  normalize(y, M, MW, L);
  const int j = row / a.G, hq = h * a.G + row % a.G;
  finish_row(a, y, s_tr + (lane >> 3) * kTrTile, r, lane < 8, ((int64_t)job.y * a.q_len + j) * a.Hq + hq);
  if (lane == 0) finish_stats(a, job.y, h, row, M, L);
}

// mass_out = mass_in + sum over the head's rows of 2^(z - log2 of the row's sum).
__global__ void __launch_bounds__(256) kv4_mass_kernel(Kv4AttnArgs a) {
  const int h = blockIdx.y, b = blockIdx.z;
  const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
  bool bad;
  const int len = kv4_length(a.c, a.lengths, b, &bad);
  if (t >= len) return;
  const int64_t head = (int64_t)b * a.c.n_kv + h, cap = a.c.capacity();
  float s = 0.0f;
  for (int row = 0; row < a.R; ++row) {
    const float z = a.z[(head * a.R + row) * cap + t];
    if (z > -INFINITY || z != z) s = __fadd_rn(s, ex2(__fsub_rn(z, a.row_lse[head * a.R + row])));
  }
  a.mass_out[head * cap + t] = a.mass_in != nullptr ? __fadd_rn(a.mass_in[head * cap + t], s) : s;
}

// Resident blocks of the attention kernel on the current device (asked once
// per instance and device).
template <int NC, bool CAP, bool MASS>
int resident_blocks() {
  static int cache[64] = {};
  int dev = 0, sms = 0, per_sm = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  if (dev >= 0 && dev < 64 && cache[dev] > 0) return cache[dev];
  cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (cudaFuncSetAttribute(kv4_attn_kernel<NC, CAP, MASS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           Shape<NC>::smem) != cudaSuccess)
    return 0;
  cudaOccupancyMaxActiveBlocksPerMultiprocessor(&per_sm, kv4_attn_kernel<NC, CAP, MASS>, kAttnThreads,
                                                Shape<NC>::smem);
  const int n = sms * per_sm;
  if (dev >= 0 && dev < 64) cache[dev] = n;
  return n;
}

template <int NC, bool CAP, bool MASS>
int launch_attn(const Kv4AttnArgs &a, cudaStream_t st) {
  int grid = resident_blocks<NC, CAP, MASS>();
  if (grid <= 0) return 1;
  if (grid > kKv4MaxBlocks) grid = kKv4MaxBlocks;
  // no more blocks than pieces of the longest batch the table allows
  const int64_t most = ((a.c.capacity() / kUnit + kSegmentCost) * a.c.n_seqs * a.c.n_kv * a.row_tiles +
                        kMinPiece - 1) / kMinPiece;
  if (most < grid) grid = (int)most;
  kv4_attn_kernel<NC, CAP, MASS><<<grid, kAttnThreads, Shape<NC>::smem, st>>>(a);
  if (cudaGetLastError() != cudaSuccess) return 1;
  kv4_join_kernel<<<dim3((unsigned)grid, Shape<NC>::rows), kJoinThreads, 0, st>>>(a, Shape<NC>::rows);
  return cudaGetLastError() == cudaSuccess ? 0 : 1;
}

template <int NC>
int launch_rows(const Kv4AttnArgs &a, cudaStream_t st) {
  const bool mass = a.mass_out != nullptr;
  if (a.cap > 0.0f) return mass ? launch_attn<NC, true, true>(a, st) : launch_attn<NC, true, false>(a, st);
  return mass ? launch_attn<NC, false, true>(a, st) : launch_attn<NC, false, false>(a, st);
}

int row_groups(int R) { return R <= 4 ? 1 : 2; }

}  // namespace

int kv4_row_tiles(int R) { return (R + 4 * row_groups(R) - 1) / (4 * row_groups(R)); }
size_t kv4_part_bytes(int R) { return (size_t)2 * kKv4MaxBlocks * 4 * row_groups(R) * kTile * sizeof(float); }
size_t kv4_stat_bytes(int R) { return (size_t)2 * kKv4MaxBlocks * 4 * row_groups(R) * sizeof(float4); }
size_t kv4_join_bytes() { return (size_t)kKv4MaxBlocks * sizeof(int4); }

int launch_kv4_attention(const Kv4AttnArgs &a, cudaStream_t st) {
  const int rc = row_groups(a.R) == 1 ? launch_rows<1>(a, st) : launch_rows<2>(a, st);
  if (rc != 0) return rc;
  if (a.mass_out != nullptr && a.c.capacity() > 0) {
    kv4_mass_kernel<<<dim3((unsigned)((a.c.capacity() + 255) / 256), (unsigned)a.c.n_kv,
                           (unsigned)a.c.n_seqs), 256, 0, st>>>(a);
    if (cudaGetLastError() != cudaSuccess) return 1;
  }
  return 0;
}

}  // namespace hq

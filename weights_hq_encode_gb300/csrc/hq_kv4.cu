// hq_kv4.cu -- the 4-bit window cache's writes, reads and evictions
// (include/hq_kv4.h states the format).  All of them move rows: a token of one
// head is 132 bytes in the cache and 2 x 128 values outside it.
#include <cuda_runtime.h>

#include <type_traits>

#include "hq_device.cuh"
#include "hq_kv4.h"
#include "hq_kv4_io.cuh"
#include "hq_launch.cuh"

namespace hq {

constexpr int kRowsThreads = 256;                // 32 rows a block
constexpr float kRoot128 = 11.313708498984761f, kInvRoot128 = 0.08838834764831845f;
constexpr float kAbsToScale = 0.011785113019775793f;   // 1 / (7.5 sqrt(128))

// Byte offset in its unit of the 8 bytes that hold dimensions 16 r .. 16 r + 15
// of token `tok`'s K (which = 0) or V row.
__device__ __forceinline__ int kv4_chunk(int which, int tok, int r) {
  return which == 0 ? tok * 64 + r * 8 : kUnitV + (tok >> 1) * 128 + r * 16 + (tok & 1) * 8;
}

// fwht128_t8_smem without its last step back to the lanes' own dimensions: y[m]
// is coordinate r + 8 m.  The caller orders calls on one table by __syncwarp.
__device__ __forceinline__ void fwht128_t8_columns(float x[16], float *tile, int r, float y[16]) {
#pragma unroll
  for (int h = 1; h < 8; h <<= 1) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (!(j & h)) bfly2(x[j], x[j + 8], x[j + h], x[j + h + 8]);
  }
  float2 *const out = reinterpret_cast<float2 *>(tile + 2 * r);
#pragma unroll
  for (int j = 0; j < 8; ++j)                    // coordinates 16 r + j, 16 r + j + 8
    out[j * (kTrRow / 2)] = make_float2(__fadd_rn(x[j], x[j + 8]), __fsub_rn(x[j], x[j + 8]));
  __syncwarp();
  const float4 *const in = reinterpret_cast<const float4 *>(tile + kTrRow * r);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const float4 v = in[q];
    y[4 * q] = v.x; y[4 * q + 1] = v.y; y[4 * q + 2] = v.z; y[4 * q + 3] = v.w;
  }
#pragma unroll
  for (int h = 1; h < 8; h <<= 1) {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (!(j & h)) bfly2(y[2 * j], y[2 * j + 1], y[2 * (j + h)], y[2 * (j + h) + 1]);
  }
}

// Two values' codes into field `at` of two words of 4-bit fields: floor(z inv + 8)
// exactly, by one fused multiply-add to 2^23 + 8 rounded towards zero.  |z| inv is
// at most 7.5 (1 + 2^-8) and a few units, so the codes are 0 .. 15 as they are;
// 2^23's own bits are taken out at the end.
__device__ __forceinline__ void add_codes(uint32_t &even, uint32_t &odd, float z0, float z1, uint64_t inv, int at) {
  uint64_t t;
  asm("fma.rz.f32x2 %0, %1, %2, %3;" : "=l"(t) : "l"(pk2(z0, z1)), "l"(inv), "l"(pk2(8388616.0f, 8388616.0f)));
  float a, b;
  upk2(t, a, b);
  even += __float_as_uint(a) << (4 * at);
  odd += __float_as_uint(b) << (4 * at);
}

// Codes of coordinates r + 8 m, fields i of even and odd for m = 2 i and 2 i + 1,
// to the row's words 2 r and 2 r + 1 (coordinates 16 r .. 16 r + 15): a
// transposition over the row's 8 lanes in four exchanges.  A lane first joins its
// nibbles with its neighbour's (even lanes take the even m) to bytes r / 2 of
// 8 words, then bytes go over by halves: words by distance 4, 2 and 1 lanes.
__device__ __forceinline__ uint2 words_of_columns(uint32_t even, uint32_t odd, int r) {
  const bool q = r & 1, b1 = r & 2, b2 = r & 4;
  const uint32_t got = __shfl_xor_sync(0xffffffffu, q ? even : odd, 1);
  const uint32_t lo = q ? got : even, hi = q ? odd : got;
  const uint32_t x = (lo & 0x0F0F0F0Fu) | ((hi & 0x0F0F0F0Fu) << 4);           // items 0, 2, 4, 6
  const uint32_t y = ((lo >> 4) & 0x0F0F0F0Fu) | (hi & 0xF0F0F0F0u);           // items 1, 3, 5, 7
  const uint32_t l = __byte_perm(x, y, 0x5410), h = __byte_perm(x, y, 0x7632);  // items 0 2 1 3, 4 6 5 7
  const uint32_t k1 = b2 ? h : l, g1 = __shfl_xor_sync(0xffffffffu, b2 ? l : h, 4);
  const uint32_t a = __byte_perm(k1, g1, 0x6240), c = __byte_perm(k1, g1, 0x7351);
  const uint32_t k2 = b1 ? c : a, g2 = __shfl_xor_sync(0xffffffffu, b1 ? a : c, 2);
  const uint32_t f = __byte_perm(k2, g2, 0x5410), g = __byte_perm(k2, g2, 0x7632);
  const uint32_t k3 = q ? g : f, g3 = __shfl_xor_sync(0xffffffffu, q ? f : g, 1);
  // byte k came from the lanes r / 2 ^ {0, 2, 1, 3}[k]
  const uint32_t p = r >> 1;
  const uint32_t order = p == 0 ? 0x3120u : p == 1 ? 0x1302u : p == 2 ? 0x2031u : 0x0213u;
  return make_uint2(__byte_perm(q ? g3 : k3, 0u, order), __byte_perm(q ? k3 : g3, 0u, order));
}

// Codes K and V rows, 8 lanes an entry as the codec's kernels hold a tile
// (lane r: dimensions 16 r .. 16 r + 15), so that the transform is the codec's,
// its stages in the codec's order.  It is not taken back to the lanes'
// dimensions in fp32: the codes are, 8 bytes a lane instead of 64.  Bound by
// instruction issue (72% of the cycles): 289000 entries in bf16 take 56 us where
// their 186 MB want 27.
template <int KIND>
__global__ void __launch_bounds__(kRowsThreads, 5) kv4_append_kernel(Kv4RowArgs a) {
  __shared__ __align__(16) float s_tr[(kRowsThreads / 8) * kTrTile];
  follow_launch();
  const int tl = threadIdx.x >> 3, r = threadIdx.x & 7;
  const int64_t entry = (int64_t)blockIdx.x * (kRowsThreads / 8) + tl;
  const int64_t i = kv4_divide(entry, a.c.n_kv, a.c.kv_shift);
  const int h = (int)(entry - i * a.c.n_kv);
  // K and V rows one after the other, or, in short calls, in blocks of their own (gridDim.y 2)
  const auto takes = [](int which) { return gridDim.y == 1 || (int)blockIdx.y == which; };
  Row16<KIND> rows[2];
  uint32_t place = kNoPlace;
  if (i < a.n_tokens) {                          // every lane stays for the transform
    if (takes(0)) rows[0].load(a.rows.k, i * a.rows.k_token + h * a.rows.k_head, r, a.rows.vec != 0);
    if (takes(1)) rows[1].load(a.rows.v, i * a.rows.v_token + h * a.rows.v_head, r, a.rows.vec != 0);
    const int seq = a.seq[i], pos = a.pos[i];
    if (seq >= 0) {
      place = kv4_place(a.c, seq, pos, h);
      if (place == kNoPlace && r == 0) atomicOr(a.status, (uint32_t)HQ_ERR_PAGE);
    }
  } else {
    rows[0].zero();
    rows[1].zero();
  }
  const uint32_t mw = (a.c.signs[r >> 1] >> (16 * (r & 1))) & 0xFFFFu;
  unsigned char *const unit = kv4_unit(a.c, place);
  const int tok = place % kUnit;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    if (!takes(which)) continue;
    float x[16], y[16];
    rows[which].get(mw, x);
    if (which == 1) __syncwarp();                // the table is free
    fwht128_t8_columns(x, s_tr + tl * kTrTile, r, y);
    float top = 0.0f;                            // the largest magnitude, NaN if there is one
#pragma unroll
    for (int j = 0; j < 16; j += 2)
      asm("max.NaN.abs.f32 %0, %0, %1, %2;" : "+f"(top) : "f"(y[j]), "f"(y[j + 1]));
#pragma unroll
    for (int d = 1; d < 8; d <<= 1)
      asm("max.NaN.f32 %0, %0, %1;" : "+f"(top) : "f"(__shfl_xor_sync(0xffffffffu, top, d)));
    const bool finite = top < INFINITY;
    float sf = finite ? __bfloat162float(__float2bfloat16_rn(__fmul_rn(top, kAbsToScale))) : 0.0f;
    if (sf < 0x1p-126f) sf = 0.0f;               // no subnormal scales: the row is zero
    const float inv = sf > 0.0f ? __fdiv_rn(1.0f, __fmul_rn(sf, kRoot128)) : 0.0f;
    const uint64_t inv2 = pk2(inv, inv);
    constexpr uint32_t kOnes = 0x4B000000u * 0x11111111u;      // 2^23's bits in every field
    uint32_t even = 0u - kOnes, odd = 0u - kOnes;
#pragma unroll
    for (int i = 0; i < 8; ++i) add_codes(even, odd, y[2 * i], y[2 * i + 1], inv2, i);
    uint2 w = words_of_columns(even, odd, r);
    if (place == kNoPlace) continue;
    if (sf == 0.0f) w.x = w.y = 0x88888888u;
    *reinterpret_cast<uint2 *>(unit + kv4_chunk(which, tok, r)) = w;
    if (r == 0) {
      if (!finite) atomicOr(a.status, (uint32_t)HQ_ERR_RANGE);
      reinterpret_cast<uint16_t *>(unit + (which == 0 ? kUnitKs : kUnitVs))[tok] =
          (uint16_t)(__float_as_uint(sf) >> 16);
    }
  }
}

// ---------------------------------------------------------------- reading
// +1 or -1 of the Hadamard matrix as fp16, entries (i, j) and (i, k).
__device__ __forceinline__ uint32_t signs_f16(int i, int j, int k) {
  return (0x3C00u | ((uint32_t)(__popc(i & j) & 1) << 15)) | (0x3C000000u | ((uint32_t)(__popc(i & k) & 1) << 31));
}

// Writes a row's 4 values of this lane, dimensions d, d + 1 and d + 64, d + 65; p: dimension d.
// VEC: the row starts on a 16-byte boundary.
template <int KIND, bool VEC>
__device__ __forceinline__ void store4(char *to, const float v[4], const uint32_t flip[4]) {
  if constexpr (KIND == HQ_T_F32) {
    float x[4], *p = reinterpret_cast<float *>(to);
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = __uint_as_float(__float_as_uint(v[j]) ^ flip[j]);
    if constexpr (VEC) {
      *reinterpret_cast<float2 *>(p) = make_float2(x[0], x[1]);
      *reinterpret_cast<float2 *>(p + 64) = make_float2(x[2], x[3]);
    } else {
      p[0] = x[0]; p[1] = x[1]; p[64] = x[2]; p[65] = x[3];
    }
  } else {
    uint16_t *p = reinterpret_cast<uint16_t *>(to);
    const uint32_t lo = round_pair<KIND>(v[0], v[1]) ^ (flip[0] >> 16 | flip[1]);
    const uint32_t hi = round_pair<KIND>(v[2], v[3]) ^ (flip[2] >> 16 | flip[3]);
    if constexpr (VEC) {
      *reinterpret_cast<uint32_t *>(p) = lo;
      *reinterpret_cast<uint32_t *>(p + 64) = hi;
    } else {
      p[0] = (uint16_t)lo; p[1] = (uint16_t)(lo >> 16); p[64] = (uint16_t)hi; p[65] = (uint16_t)(hi >> 16);
    }
  }
}

// Values of K and V rows, up to 32 (token, head) entries a warp.  With d = 8 a + b the
// matrix is H16 x H8, and a row's codes are a 16 x 8 matrix X: H16 X is one
// mma.sync m16n8k16, (H16 X) H8 one m16n8k8 of the first one's result.  All of it is
// exact (+-1 times half-integers, sums below 2^10 in fp16 and fp32), so the
// one rounding is that of the product with the scale; and a lane ends with
// dimensions 8 n8 + 2 c4 and the next, and the same + 64: whole 128-byte
// stores.  262144 entries to bf16: 37.5 us, 25 of them the memory's.  The first stall is
// the codes' loads, of which registers let a warp ask for four entries at a time (5.0
// cycles an instruction); 81 instructions an entry issue in 55% of the cycles.  The codec's transform
// in registers and shared memory instead takes 330 for 4 rows, 68 us.
constexpr int kReadBatch = 4;                    // entries of a warp at a time
template <int KIND, bool VEC>
__global__ void __launch_bounds__(kRowsThreads) kv4_read_kernel(Kv4RowArgs a, int per_warp) {
  follow_launch();
  const int lane = threadIdx.x & 31, n8 = lane >> 2, c4 = lane & 3;
  const int64_t first = ((int64_t)blockIdx.x * (kRowsThreads / 32) + (threadIdx.x >> 5)) * per_warp;
  const int64_t entries = a.n_tokens * a.c.n_kv;
  if (first >= entries) return;
  // an entry a lane: its place, its scales and where its rows go
  uint32_t place = 0;
  bool writes = false;
  constexpr int kSize = KIND == HQ_T_F32 ? 4 : 2;
  int64_t k_to = 0, v_to = 0;                    // addresses
  float ks = 0.0f, vs = 0.0f;
  if (lane < per_warp && first + lane < entries) {
    const int64_t i = kv4_divide(first + lane, a.c.n_kv, a.c.kv_shift);
    const int h = (int)(first + lane - i * a.c.n_kv);
    const int seq = a.seq[i], pos = a.pos[i];
    writes = seq >= 0;                           // no padding token
    if (writes) {
      place = kv4_place(a.c, seq, pos, h);
      k_to = reinterpret_cast<int64_t>(a.rows.k) + (i * a.rows.k_token + h * a.rows.k_head) * kSize;
      v_to = reinterpret_cast<int64_t>(a.rows.v) + (i * a.rows.v_token + h * a.rows.v_head) * kSize;
      if (place == kNoPlace) {
        atomicOr(a.status, (uint32_t)HQ_ERR_PAGE);
        place = 0;                               // the pool's first row, times a scale of 0
      } else {
        const unsigned char *unit = kv4_unit(a.c, place);
        ks = bf16_to_f32(reinterpret_cast<const uint16_t *>(unit + kUnitKs)[place % kUnit]);
        vs = bf16_to_f32(reinterpret_cast<const uint16_t *>(unit + kUnitVs)[place % kUnit]);
        ks = __fmul_rn(__fmul_rn(ks, kInvRoot128), 512.0f);    // codes come in units of 2^-9
        vs = __fmul_rn(__fmul_rn(vs, kInvRoot128), 512.0f);
      }
    }
  }
  const uint32_t live = __ballot_sync(0xffffffffu, writes);
  // rows n8 and n8 + 8 of H16 (its columns in the order of the words below), columns of H8
  const uint32_t h0 = signs_f16(n8, 4 * c4, 4 * c4 + 1), h1 = signs_f16(n8 + 8, 4 * c4, 4 * c4 + 1);
  const uint32_t h2 = signs_f16(n8, 4 * c4 + 2, 4 * c4 + 3), h3 = signs_f16(n8 + 8, 4 * c4 + 2, 4 * c4 + 3);
  const uint32_t g0 = signs_f16(n8, 2 * c4, 2 * c4 + 1);
  // nibble n8 of a word: byte n8 / 2, as a subnormal of 2^-24 or 2^-20, centred to (c - 7.5) 2^-9
  const uint32_t sel = (uint32_t)(n8 >> 1) | ((uint32_t)(n8 >> 1) + 4u) << 8;   // into bytes 0 and 2
  const uint32_t mask = (n8 & 1) ? 0x00F000F0u : 0x000F000Fu, factor = (n8 & 1) ? 0x68006800u : 0x78007800u;
  const int d = 8 * n8 + 2 * c4;
  uint32_t flip[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int dj = d + (j & 1) + 64 * (j >> 1);
    flip[j] = ((a.c.signs[dj >> 5] >> (dj & 31)) & 1u) << 31;
  }
  // V's rows lie where K's do, `apart` bytes further on, when the strides are the same
  const bool same = a.rows.k_token == a.rows.v_token && a.rows.k_head == a.rows.v_head;
  const int64_t apart = reinterpret_cast<int64_t>(a.rows.v) - reinterpret_cast<int64_t>(a.rows.k);
  const uint32_t k_off = 16 * c4, v_off = kUnitV + 32 * c4;
#pragma unroll 1
  for (int e0 = 0; e0 < 32 && (live >> e0) != 0; e0 += kReadBatch) {
    // words 4 c4 .. 4 c4 + 3 (8 dimensions each) of every entry's K and V
    uint4 k[kReadBatch];
    uint2 lo[kReadBatch], hi[kReadBatch];
#pragma unroll
    for (int e = 0; e < kReadBatch; ++e) {
      const uint32_t p = __shfl_sync(0xffffffffu, place, e0 + e), tok = p % kUnit;
      const unsigned char *unit = kv4_unit(a.c, p) + tok * 64;
      k[e] = *reinterpret_cast<const uint4 *>(unit + k_off);
      const uint2 *v = reinterpret_cast<const uint2 *>(unit + v_off - (tok & 1) * 56);   // pairs are 128 bytes apart
      lo[e] = v[0];
      hi[e] = v[2];
    }
#pragma unroll
    for (int e = 0; e < kReadBatch; ++e) {
      if (!((live >> (e0 + e)) & 1u)) continue;  // warp-uniform
      const int64_t to_k = __shfl_sync(0xffffffffu, k_to, e0 + e) + d * kSize;
      const int64_t to_v = same ? to_k + apart : __shfl_sync(0xffffffffu, v_to, e0 + e) + d * kSize;
#pragma unroll
      for (int which = 0; which < 2; ++which) {
        const uint4 w = which == 0 ? k[e] : make_uint4(lo[e].x, lo[e].y, hi[e].x, hi[e].y);
        const float s = __shfl_sync(0xffffffffu, which == 0 ? ks : vs, e0 + e);
        uint32_t b0 = __byte_perm(w.x, w.y, sel) & mask, b1 = __byte_perm(w.z, w.w, sel) & mask;
        asm("fma.rn.f16x2 %0, %0, %1, %2;" : "+r"(b0) : "r"(factor), "r"(0xA380A380u));
        asm("fma.rn.f16x2 %0, %0, %1, %2;" : "+r"(b1) : "r"(factor), "r"(0xA380A380u));
        float t[4], x[4];
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
            "{%8, %9}, {%10, %10, %10, %10};"
            : "=f"(t[0]), "=f"(t[1]), "=f"(t[2]), "=f"(t[3])
            : "r"(h0), "r"(h1), "r"(h2), "r"(h3), "r"(b0), "r"(b1), "f"(0.0f));
        const uint32_t t0 = round_pair<HQ_T_F16>(t[0], t[1]), t1 = round_pair<HQ_T_F16>(t[2], t[3]);   // exact
        asm("mma.sync.aligned.m16n8k8.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5}, {%6}, "
            "{%7, %7, %7, %7};"
            : "=f"(x[0]), "=f"(x[1]), "=f"(x[2]), "=f"(x[3])
            : "r"(t0), "r"(t1), "r"(g0), "f"(0.0f));
        upk2(mul2(pk2(x[0], x[1]), pk2(s, s)), x[0], x[1]);
        upk2(mul2(pk2(x[2], x[3]), pk2(s, s)), x[2], x[3]);
        store4<KIND, VEC>(reinterpret_cast<char *>(which == 0 ? to_k : to_v), x, flip);
      }
    }
  }
}

// ---------------------------------------------------------------- eviction
constexpr int kSelThreads = 1024, kSelBins = 2048;

// Masses in the order of eviction as unsigned integers: larger mass, larger
// key; -0 as 0; a NaN is the least.
__device__ __forceinline__ uint32_t mass_key(float m) {
  if (m != m) return 0u;
  const uint32_t b = __float_as_uint(__fadd_rn(m, 0.0f));
  return (b >> 31) ? ~b : b | 0x80000000u;
}

// The inclusive sum of v over the block's threads up to this one, and the
// block's total; s_w: 2 x 32 words, flip: alternates from call to call.
__device__ __forceinline__ uint32_t block_scan(uint32_t v, uint32_t *s_w, int flip, uint32_t *total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t o = __shfl_up_sync(0xffffffffu, v, d);
    if (lane >= d) v += o;
  }
  uint32_t *w = s_w + 32 * flip;
  if (lane == 31) w[warp] = v;
  __syncthreads();
  uint32_t t = w[lane];
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const uint32_t o = __shfl_up_sync(0xffffffffu, t, d);
    if (lane >= d) t += o;
  }
  *total = __shfl_sync(0xffffffffu, t, 31);
  const uint32_t before = __shfl_sync(0xffffffffu, t, warp > 0 ? warp - 1 : 0);
  return v + (warp > 0 ? before : 0u);
}

// The positions that one head of one sequence keeps.  The competing masses'
// keys are read once (the first `cached` into shared memory, four at a time from
// there on) for their least and largest; the threshold is found digit by digit
// of (key - least), 11 bits at a time from the top of that range, by
// histograms in shared memory, until all that share the digits are kept (one
// pass for a few hundred masses, two for 30000, where three are the most); a last
// pass in order compacts what lies above it
// and the first of what equals it.  Digits of the range and not of the key:
// masses of a few binary orders spread over all 2048 bins, where the key's own
// top bits are a handful of values and their atomics one behind another.
// cached: a multiple of 4.  16 x 32768 tokens of 8 heads: 128 blocks, one a
// multiprocessor, 19 us for 15 MB of masses (their loads 5, 7 in passes of 11 bits, 6 to compact).
__global__ void __launch_bounds__(kSelThreads) kv4_select_kernel(Kv4EvictArgs a, int cached) {
  extern __shared__ __align__(16) uint32_t s_keys[];
  __shared__ uint32_t s_hist[kSelBins];
  __shared__ uint32_t s_w[64];
  __shared__ uint32_t s_digit, s_above, s_there, s_least, s_most;
  follow_launch();
  const int h = blockIdx.x, b = blockIdx.y, tid = threadIdx.x;
  bool bad;
  const int n = kv4_length(a.src, a.lengths, b, &bad);
  if (bad && tid == 0 && h == 0) atomicOr(a.status, (uint32_t)HQ_ERR_PAGE);
  const int keep = min(n, a.budget);
  if (h == 0 && tid == 0) a.new_lengths[b] = keep;
  int32_t *kept = a.kept + ((int64_t)b * a.src.n_kv + h) * a.budget;
  const float *mass = a.mass + ((int64_t)b * a.src.n_kv + h) * a.src.capacity();
  const int old = n > a.budget ? n - a.recent : 0;        // tokens that compete
  const int need = n > a.budget ? a.budget - a.recent : 0;
  for (int i = need + tid; i < keep; i += kSelThreads) kept[i] = old + i - need;
  for (int i = keep + tid; i < a.budget; i += kSelThreads) kept[i] = -1;
  if (need == 0) return;
  if (tid == 0) {
    s_least = 0xFFFFFFFFu;
    s_most = 0u;
  }
  __syncthreads();
  const int near = min(old, cached);             // keys in shared memory; a few behind them fill up a four
  uint4 *const s_keys4 = reinterpret_cast<uint4 *>(s_keys);
  uint32_t least = 0xFFFFFFFFu, most = 0u;
  int from = 0;                                  // where the loads one by one begin
  if ((reinterpret_cast<uintptr_t>(mass) & 15) == 0) {
    from = near & ~3;
    for (int i0 = tid; 4 * i0 < from; i0 += 8 * kSelThreads) {   // 8 loads, then what they bring
      float4 m[8];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        if (4 * (i0 + u * kSelThreads) < from) m[u] = reinterpret_cast<const float4 *>(mass)[i0 + u * kSelThreads];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        if (4 * (i0 + u * kSelThreads) >= from) break;
        const uint4 k = make_uint4(mass_key(m[u].x), mass_key(m[u].y), mass_key(m[u].z), mass_key(m[u].w));
        s_keys4[i0 + u * kSelThreads] = k;
        least = min(least, min(min(k.x, k.y), min(k.z, k.w)));
        most = max(most, max(max(k.x, k.y), max(k.z, k.w)));
      }
    }
  }
#pragma unroll 8
  for (int i = from + tid; i < old; i += kSelThreads) {
    const uint32_t key = mass_key(mass[i]);
    if (i < cached) s_keys[i] = key;
    least = min(least, key);
    most = max(most, key);
  }
  least = __reduce_min_sync(0xffffffffu, least);
  most = __reduce_max_sync(0xffffffffu, most);
  if ((tid & 31) == 0) {
    atomicMin(&s_least, least);
    atomicMax(&s_most, most);
  }
  __syncthreads();
  least = s_least;
  // fillers are least keys behind all others: equals go to the lower position, so none is kept
  if (tid < 3 && near + tid < ((near + 3) & ~3)) s_keys[near + tid] = least;
  int shift = 32 - __clz((int)(s_most - least));  // bits of the range: those below `shift` are to be found
  uint32_t prefix = 0, want = (uint32_t)need;     // digits found; how many to keep among their equals
  int flip = 0;
  while (shift > 0) {
    const int bits = min(shift, 11);
    const uint32_t found = shift == 32 ? 0u : 0xFFFFFFFFu << shift;   // bits of the digits found
    shift -= bits;
    const uint32_t mask = (1u << bits) - 1;
    for (int i = tid; i < kSelBins; i += kSelThreads) s_hist[i] = 0;
    __syncthreads();
    const auto count = [&](uint32_t key) {
      key -= least;
      if ((key & found) == prefix) atomicAdd(&s_hist[(key >> shift) & mask], 1u);
    };
#pragma unroll 2
    for (int i = tid; 4 * i < near; i += kSelThreads) {
      const uint4 k = s_keys4[i];
      count(k.x);
      count(k.y);
      count(k.z);
      count(k.w);
    }
    for (int i = cached + tid; i < old; i += kSelThreads) count(mass_key(mass[i]));
    __syncthreads();
    // bins from the largest down, two a thread
    const uint32_t d0 = kSelBins - 1 - 2 * tid, c0 = s_hist[d0], c1 = s_hist[d0 - 1];
    uint32_t total;
    const uint32_t end = block_scan(c0 + c1, s_w, flip, &total), begin = end - c0 - c1;
    flip ^= 1;
    if (begin < want && want <= end) {            // exactly one thread
      const bool first = want <= begin + c0;
      s_digit = first ? d0 : d0 - 1;
      s_above = first ? begin : begin + c0;
      s_there = first ? c0 : c1;
    }
    __syncthreads();
    prefix |= s_digit << shift;
    want -= s_above;
    if (want == s_there && prefix + least != 0) { // all of them are kept: what is above the key before theirs
      --prefix;
      want = 0;
      break;
    }
  }
  __syncthreads();                                // the fillers, when no digit was to be found
  // The keys in order, 8 a thread in a step, or one where that is a step: those above the threshold
  // so far in the low half of a word, its equals in the high half.
  const uint32_t level = prefix + least;
  uint32_t gt_before = 0, eq_before = 0;
  const auto compact = [&](auto keys, int base) {
    constexpr int kKeys = decltype(keys)::value;
    const int at = base + kKeys * tid;
    uint32_t key[kKeys < 4 ? 4 : kKeys], c = 0;
    if (kKeys == 8 && at + 8 <= cached) {         // what lies behind `near` is not looked at
#pragma unroll
      for (int j = 0; j < kKeys; j += 4) {
        const uint4 x = s_keys4[(at + j) / 4];
        key[j] = x.x; key[j + 1] = x.y; key[j + 2] = x.z; key[j + 3] = x.w;
      }
    } else {
#pragma unroll
      for (int j = 0; j < kKeys; ++j) key[j] = at + j < near ? s_keys[at + j] : at + j < old ? mass_key(mass[at + j]) : 0u;
    }
#pragma unroll
    for (int j = 0; j < kKeys; ++j)
      if (at + j < old) c += key[j] > level ? 1u : key[j] == level ? 0x10000u : 0u;
    uint32_t total;
    const uint32_t incl = block_scan(c, s_w, flip, &total), excl = incl - c;
    flip ^= 1;
    if (c != 0) {
      uint32_t gt = gt_before + (excl & 0xFFFFu), eq = eq_before + (excl >> 16);
#pragma unroll
      for (int j = 0; j < kKeys; ++j) {
        if (at + j >= old) break;
        if (key[j] > level) {
          kept[gt + min(eq, want)] = at + j;
          ++gt;
        } else if (key[j] == level) {
          if (eq < want) kept[gt + eq] = at + j;
          ++eq;
        }
      }
    }
    gt_before += total & 0xFFFFu;
    eq_before += total >> 16;
  };
  if (old <= kSelThreads) compact(std::integral_constant<int, 1>{}, 0);
  else
    for (int base = 0; base < old; base += 8 * kSelThreads) compact(std::integral_constant<int, 8>{}, base);
}

// Rows and masses of the kept positions, up to 32 a warp: a lane looks one up,
// moves its scales and its mass; then 8 lanes a row move the codes, all rows'
// loads before the first store.  16 x 4096 of 32768 tokens, 8 heads: 40 us for 69 MB
// each way, 179 MB read: a kept V row's pieces lie in the 128 bytes of its token
// pair, and the memory delivers 64 at a time.
__global__ void __launch_bounds__(kRowsThreads) kv4_move_kernel(Kv4EvictArgs a, int per_warp) {
  follow_launch();
  const int lane = threadIdx.x & 31, r = lane & 7, h = blockIdx.y, b = blockIdx.z;
  const int first = (blockIdx.x * (kRowsThreads / 32) + (threadIdx.x >> 5)) * per_warp, i = first + lane;
  bool bad;
  const int n = min(kv4_length(a.src, a.lengths, b, &bad), a.budget);
  if (first >= n) return;
  const int64_t head = (int64_t)b * a.src.n_kv + h;
  uint32_t from = kNoPlace, to = kNoPlace;
  if (lane < per_warp && i < n) {
    const int t = a.kept[head * a.budget + i];
    from = kv4_place(a.src, b, t, h);
    to = kv4_place(a.dst, b, i, h);
    a.new_mass[head * a.dst.capacity() + i] = a.mass[head * a.src.capacity() + t];
    if (from == kNoPlace || to == kNoPlace) {
      atomicOr(a.status, (uint32_t)HQ_ERR_PAGE);
      from = to = kNoPlace;
    } else {
      const uint16_t *s = reinterpret_cast<const uint16_t *>(kv4_unit(a.src, from) + kUnitKs) + from % kUnit;
      uint16_t *d = reinterpret_cast<uint16_t *>(kv4_unit(a.dst, to) + kUnitKs) + to % kUnit;
      const uint16_t ks = s[0], vs = s[kUnit];
      d[0] = ks;
      d[kUnit] = vs;
    }
  }
  uint2 k[8], v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t p = __shfl_sync(0xffffffffu, from, 4 * e + (lane >> 3));
    if (p == kNoPlace) continue;
    const unsigned char *unit = kv4_unit(a.src, p);
    k[e] = *reinterpret_cast<const uint2 *>(unit + kv4_chunk(0, p % kUnit, r));
    v[e] = *reinterpret_cast<const uint2 *>(unit + kv4_chunk(1, p % kUnit, r));
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const uint32_t p = __shfl_sync(0xffffffffu, to, 4 * e + (lane >> 3));
    if (p == kNoPlace) continue;
    unsigned char *unit = kv4_unit(a.dst, p);
    *reinterpret_cast<uint2 *>(unit + kv4_chunk(0, p % kUnit, r)) = k[e];
    *reinterpret_cast<uint2 *>(unit + kv4_chunk(1, p % kUnit, r)) = v[e];
  }
}

// ---------------------------------------------------------------- launches
int launch_kv4_append(const Kv4RowArgs &a, cudaStream_t st) {
  const unsigned blocks = (unsigned)((a.n_tokens * a.c.n_kv + kRowsThreads / 8 - 1) / (kRowsThreads / 8));
  const dim3 grid(blocks, blocks <= 152 * 5 / 2 ? 2 : 1);      // twice the blocks while they fit at once
  switch (a.rows.kind) {
    case HQ_T_F32: return launch_behind(kv4_append_kernel<HQ_T_F32>, grid, kRowsThreads, 0, st, a);
    case HQ_T_F16: return launch_behind(kv4_append_kernel<HQ_T_F16>, grid, kRowsThreads, 0, st, a);
    default: return launch_behind(kv4_append_kernel<HQ_T_BF16>, grid, kRowsThreads, 0, st, a);
  }
}

// Rows a warp takes, a multiple of `step` (or 1) up to 32: as many as fill whole
// waves of the 4 blocks that a multiprocessor holds.  Short calls get few, as
// their time is that of one warp's chain of loads; long ones many, whose look-ups
// are then one a lane (262144 rows: 39 us with 32 a warp in 1.7 waves).
static int rows_a_warp(int64_t rows, int step) {
  constexpr int64_t kWave = 152 * 4 * (kRowsThreads / 32);
  const int64_t waves = (rows + 32 * kWave - 1) / (32 * kWave);
  const int64_t per = (rows + waves * kWave - 1) / (waves * kWave);
  return per <= 1 && step == 1 ? 1 : (int)((per + 3) / 4 * 4);
}

int launch_kv4_read(const Kv4RowArgs &a, cudaStream_t st) {
  const int64_t entries = a.n_tokens * a.c.n_kv;
  const int per = rows_a_warp(entries, 1), block = kRowsThreads / 32 * per;
  const dim3 grid((unsigned)((entries + block - 1) / block));
  const bool vec = a.rows.vec != 0;
  const auto go = [&](auto with, auto without) {
    return vec ? launch_behind(with, grid, kRowsThreads, 0, st, a, per)
               : launch_behind(without, grid, kRowsThreads, 0, st, a, per);
  };
  switch (a.rows.kind) {
    case HQ_T_F32: return go(kv4_read_kernel<HQ_T_F32, true>, kv4_read_kernel<HQ_T_F32, false>);
    case HQ_T_F16: return go(kv4_read_kernel<HQ_T_F16, true>, kv4_read_kernel<HQ_T_F16, false>);
    default: return go(kv4_read_kernel<HQ_T_BF16, true>, kv4_read_kernel<HQ_T_BF16, false>);
  }
}

int launch_kv4_evict(const Kv4EvictArgs &a, cudaStream_t st) {
  // keys in shared memory, as many as a block may have
  constexpr int kMostKeys = 48 * 1024;
  const int cached = a.src.capacity() < kMostKeys ? (int)a.src.capacity() : kMostKeys;
  if (cached > 8 * 1024 &&                       // with s_hist above what a block has unasked
      cudaFuncSetAttribute(kv4_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostKeys * 4) !=
          cudaSuccess)
    return 1;
  if (launch_behind(kv4_select_kernel, dim3((unsigned)a.src.n_kv, (unsigned)a.src.n_seqs), kSelThreads,
                    (size_t)cached * 4, st, a, cached) != 0)
    return 1;
  if (a.src.capacity() == 0) return 0;           // no tokens to move
  const int64_t most = a.budget < a.src.capacity() ? a.budget : a.src.capacity();
  const int per = rows_a_warp(most * a.src.n_kv * a.src.n_seqs, 4), block = kRowsThreads / 32 * per;
  return launch_behind(kv4_move_kernel, dim3((unsigned)((most + block - 1) / block), (unsigned)a.src.n_kv,
                                             (unsigned)a.src.n_seqs), kRowsThreads, 0, st, a, per);
}

}  // namespace hq

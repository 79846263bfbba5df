// hq_kv4.cu -- the 4-bit window cache's writes, reads and evictions
// (include/hq_kv4.h states the format).  All of them are bound by memory: a
// token of one head is 132 bytes in the cache and 2 x 128 values outside it.
// 8 lanes hold a row as the codec's kernels do (lane r: dimensions 16 r ..
// 16 r + 15), so that the transform is the codec's, its stages in the codec's
// order, and a lane's 16 codes are the 8 bytes it stores.
#include <cuda_runtime.h>

#include "hq_device.cuh"
#include "hq_kv4.h"
#include "hq_kv4_io.cuh"

namespace hq {

constexpr int kRowsThreads = 256;                // 32 rows a block
constexpr float kRoot128 = 11.313708498984761f, kInvRoot128 = 0.08838834764831845f;
constexpr float kAbsToScale = 0.011785113019775793f;   // 1 / (7.5 sqrt(128))

// Byte offset in its unit of the 8 bytes that hold dimensions 16 r .. 16 r + 15
// of token `tok`'s K (which = 0) or V row.
__device__ __forceinline__ int kv4_chunk(int which, int tok, int r) {
  return which == 0 ? tok * 64 + r * 8 : kUnitV + (tok >> 1) * 128 + r * 16 + (tok & 1) * 8;
}

// One row a group of 8 lanes: blockIdx.y 0 codes K, 1 codes V.
template <int KIND>
__global__ void __launch_bounds__(kRowsThreads) kv4_append_kernel(Kv4RowArgs a) {
  __shared__ __align__(16) float s_tr[(kRowsThreads / 8) * kTrTile];
  const int tl = threadIdx.x >> 3, r = threadIdx.x & 7, which = blockIdx.y;
  const int64_t row = (int64_t)blockIdx.x * (kRowsThreads / 8) + tl;
  const int64_t i = row / a.c.n_kv;
  const int h = (int)(row - i * a.c.n_kv);
  int64_t page = -1;
  int pos = 0;
  if (i < a.n_tokens) {                          // every lane stays for the transform
    const int seq = __ldg(a.seq + i);
    pos = __ldg(a.pos + i);
    if (seq >= 0) {
      if (seq < a.c.n_seqs && pos >= 0 && pos < a.c.capacity()) page = kv4_page(a.c, seq, pos);
      if (page < 0 && r == 0) atomicOr(a.status, (uint32_t)HQ_ERR_PAGE);
    }
  }
  float x[16];
  if (page >= 0) {
    const int64_t at = which == 0 ? i * a.rows.k_token + h * a.rows.k_head
                                  : i * a.rows.v_token + h * a.rows.v_head;
    load_row16<KIND>(which == 0 ? a.rows.k : a.rows.v, at, r, a.rows.vec != 0, x);
  } else {
#pragma unroll
    for (int j = 0; j < 16; ++j) x[j] = 0.0f;
  }
  const uint32_t mw = __ldg(a.c.signs + (r >> 1)) >> (16 * (r & 1));
#pragma unroll
  for (int j = 0; j < 16; ++j) x[j] = __uint_as_float(__float_as_uint(x[j]) ^ (((mw >> j) & 1u) << 31));
  fwht128_t8(x, s_tr + tl * kTrTile, r);
  // the largest magnitude as an integer: an infinity or a NaN is above every finite value
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < 16; ++j) top = max(top, __float_as_uint(x[j]) & 0x7FFFFFFFu);
#pragma unroll
  for (int d = 1; d < 8; d <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, d));
  if (page < 0) return;
  const bool finite = top < 0x7F800000u;
  if (!finite && r == 0) atomicOr(a.status, (uint32_t)HQ_ERR_RANGE);
  __nv_bfloat16 s = __float2bfloat16_rn(finite ? __fmul_rn(__uint_as_float(top), kAbsToScale) : 0.0f);
  float sf = __bfloat162float(s);
  if (sf < 0x1p-126f) sf = 0.0f;                 // no subnormal scales: the row is zero
  const float inv = sf > 0.0f ? __fdiv_rn(1.0f, __fmul_rn(sf, kRoot128)) : 0.0f;
  uint32_t w[2] = {0u, 0u};
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const float t = floorf(__fadd_rn(__fmul_rn(sf > 0.0f ? x[j] : 0.0f, inv), 8.0f));
    w[j >> 3] |= (uint32_t)fminf(fmaxf(t, 0.0f), 15.0f) << (4 * (j & 7));
  }
  unsigned char *unit = kv4_unit(a.c, page, h, pos);
  const int tok = pos % kUnit;
  *reinterpret_cast<uint2 *>(unit + kv4_chunk(which, tok, r)) = make_uint2(w[0], w[1]);
  if (r == 0)
    reinterpret_cast<uint16_t *>(unit + (which == 0 ? kUnitKs : kUnitVs))[tok] =
        (uint16_t)(__float_as_uint(sf) >> 16);
}

template <int KIND>
__global__ void __launch_bounds__(kRowsThreads) kv4_read_kernel(Kv4RowArgs a) {
  __shared__ __align__(16) float s_tr[(kRowsThreads / 8) * kTrTile];
  const int tl = threadIdx.x >> 3, r = threadIdx.x & 7, which = blockIdx.y;
  const int64_t row = (int64_t)blockIdx.x * (kRowsThreads / 8) + tl;
  const int64_t i = row / a.c.n_kv;
  const int h = (int)(row - i * a.c.n_kv);
  bool live = i < a.n_tokens;                    // every lane stays for the transform
  uint2 w = make_uint2(0x88888888u, 0x88888888u);
  float s = 0.0f;
  if (live) {
    const int seq = __ldg(a.seq + i), pos = __ldg(a.pos + i);
    live = seq >= 0;
    if (live) {
      int64_t page = -1;
      if (seq < a.c.n_seqs && pos >= 0 && pos < a.c.capacity()) page = kv4_page(a.c, seq, pos);
      if (page >= 0) {
        const unsigned char *unit = kv4_unit(a.c, page, h, pos);
        const int tok = pos % kUnit;
        w = *reinterpret_cast<const uint2 *>(unit + kv4_chunk(which, tok, r));
        s = bf16_to_f32(reinterpret_cast<const uint16_t *>(unit + (which == 0 ? kUnitKs : kUnitVs))[tok]);
      } else if (r == 0) {
        atomicOr(a.status, (uint32_t)HQ_ERR_PAGE);
      }
    }
  }
  s = __fmul_rn(s, kInvRoot128);                 // before the sums, so that they stay in range
  float x[16];
#pragma unroll
  for (int j = 0; j < 16; ++j)
    x[j] = __fmul_rn((float)(int)(((j < 8 ? w.x : w.y) >> (4 * (j & 7))) & 15u) - 7.5f, s);
  fwht128_t8(x, s_tr + tl * kTrTile, r);
  if (!live) return;
  const uint32_t mw = __ldg(a.c.signs + (r >> 1)) >> (16 * (r & 1));
#pragma unroll
  for (int j = 0; j < 16; ++j) x[j] = __uint_as_float(__float_as_uint(x[j]) ^ (((mw >> j) & 1u) << 31));
  const int64_t at = which == 0 ? i * a.rows.k_token + h * a.rows.k_head
                                : i * a.rows.v_token + h * a.rows.v_head;
  store_row16<KIND>(const_cast<void *>(which == 0 ? a.rows.k : a.rows.v), at, r, a.rows.vec != 0, x);
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

// The positions that one head of one sequence keeps.  The threshold mass is
// found digit by digit (11, 11 and 10 bits of the ordered key, most
// significant first) from histograms in shared memory; a last pass in order
// compacts what lies above it and the first of what equals it.
__global__ void __launch_bounds__(kSelThreads) kv4_select_kernel(Kv4EvictArgs a) {
  __shared__ uint32_t s_hist[kSelBins];
  __shared__ uint32_t s_w[64];
  __shared__ uint32_t s_digit, s_above;
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
  uint32_t prefix = 0, want = (uint32_t)need;    // digits found; how many to keep among their equals
  int flip = 0;
  for (int digit = 0; digit < 3; ++digit) {
    const int shift = digit == 0 ? 21 : digit == 1 ? 10 : 0;
    const uint32_t bins = digit == 2 ? 1024u : 2048u;
    const uint32_t above_mask = digit == 0 ? 0u : digit == 1 ? 0xFFE00000u : 0xFFFFFC00u;
    for (int i = tid; i < kSelBins; i += kSelThreads) s_hist[i] = 0;
    __syncthreads();
    for (int i = tid; i < old; i += kSelThreads) {
      const uint32_t key = mass_key(__ldg(mass + i));
      if ((key & above_mask) == prefix) atomicAdd(&s_hist[(key >> shift) & (bins - 1)], 1u);
    }
    __syncthreads();
    // bins from the largest down, two a thread
    const uint32_t d0 = kSelBins - 1 - 2 * tid, c0 = s_hist[d0], c1 = s_hist[d0 - 1];
    uint32_t total;
    const uint32_t end = block_scan(c0 + c1, s_w, flip, &total), begin = end - c0 - c1;
    flip ^= 1;
    if (begin < want && want <= end) {           // exactly one thread
      const bool first = want <= begin + c0;
      s_digit = first ? d0 : d0 - 1;
      s_above = first ? begin : begin + c0;
    }
    __syncthreads();
    prefix |= s_digit << shift;
    want -= s_above;
  }
  uint32_t gt_before = 0, eq_before = 0;
  for (int base = 0; base < old; base += 4 * kSelThreads) {
    uint32_t key[4], c = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = base + 4 * tid + j;
      key[j] = i < old ? mass_key(__ldg(mass + i)) : 0u;
      if (i < old) c += key[j] > prefix ? 1u : key[j] == prefix ? 0x10000u : 0u;
    }
    uint32_t total;
    const uint32_t incl = block_scan(c, s_w, flip, &total), excl = incl - c;
    flip ^= 1;
    uint32_t gt = gt_before + (excl & 0xFFFFu), eq = eq_before + (excl >> 16);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = base + 4 * tid + j;
      if (i >= old) break;
      if (key[j] > prefix) {
        kept[gt + min(eq, want)] = i;
        ++gt;
      } else if (key[j] == prefix) {
        if (eq < want) kept[gt + eq] = i;
        ++eq;
      }
    }
    gt_before += total & 0xFFFFu;
    eq_before += total >> 16;
  }
}

// Rows and masses of the kept positions: 8 lanes a row.
__global__ void __launch_bounds__(kRowsThreads) kv4_move_kernel(Kv4EvictArgs a) {
  const int r = threadIdx.x & 7, h = blockIdx.y, b = blockIdx.z;
  const int i = blockIdx.x * (kRowsThreads / 8) + (threadIdx.x >> 3);
  bool bad;
  const int n = kv4_length(a.src, a.lengths, b, &bad);
  if (i >= min(n, a.budget)) return;
  const int64_t head = (int64_t)b * a.src.n_kv + h;
  const int t = a.kept[head * a.budget + i];
  if (r == 0) a.new_mass[head * a.dst.capacity() + i] = __ldg(a.mass + head * a.src.capacity() + t);
  const int64_t from = kv4_page(a.src, b, t), to = kv4_page(a.dst, b, i);
  if (from < 0 || to < 0) {
    if (r == 0) atomicOr(a.status, (uint32_t)HQ_ERR_PAGE);
    return;
  }
  const unsigned char *su = kv4_unit(a.src, from, h, t);
  unsigned char *du = kv4_unit(a.dst, to, h, i);
  const int st = t % kUnit, dt = i % kUnit;
#pragma unroll
  for (int which = 0; which < 2; ++which)
    *reinterpret_cast<uint2 *>(du + kv4_chunk(which, dt, r)) =
        *reinterpret_cast<const uint2 *>(su + kv4_chunk(which, st, r));
  if (r < 2)
    reinterpret_cast<uint16_t *>(du + kUnitKs + 32 * r)[dt] =
        reinterpret_cast<const uint16_t *>(su + kUnitKs + 32 * r)[st];
}

// ---------------------------------------------------------------- launches
static dim3 rows_grid(const Kv4RowArgs &a) {
  return dim3((unsigned)((a.n_tokens * a.c.n_kv + kRowsThreads / 8 - 1) / (kRowsThreads / 8)), 2);
}

int launch_kv4_append(const Kv4RowArgs &a, cudaStream_t st) {
  const dim3 grid = rows_grid(a);
  switch (a.rows.kind) {
    case HQ_T_F32: kv4_append_kernel<HQ_T_F32><<<grid, kRowsThreads, 0, st>>>(a); break;
    case HQ_T_F16: kv4_append_kernel<HQ_T_F16><<<grid, kRowsThreads, 0, st>>>(a); break;
    default: kv4_append_kernel<HQ_T_BF16><<<grid, kRowsThreads, 0, st>>>(a); break;
  }
  return cudaGetLastError() == cudaSuccess ? 0 : 1;
}

int launch_kv4_read(const Kv4RowArgs &a, cudaStream_t st) {
  const dim3 grid = rows_grid(a);
  switch (a.rows.kind) {
    case HQ_T_F32: kv4_read_kernel<HQ_T_F32><<<grid, kRowsThreads, 0, st>>>(a); break;
    case HQ_T_F16: kv4_read_kernel<HQ_T_F16><<<grid, kRowsThreads, 0, st>>>(a); break;
    default: kv4_read_kernel<HQ_T_BF16><<<grid, kRowsThreads, 0, st>>>(a); break;
  }
  return cudaGetLastError() == cudaSuccess ? 0 : 1;
}

int launch_kv4_evict(const Kv4EvictArgs &a, cudaStream_t st) {
  kv4_select_kernel<<<dim3((unsigned)a.src.n_kv, (unsigned)a.src.n_seqs), kSelThreads, 0, st>>>(a);
  if (cudaGetLastError() != cudaSuccess) return 1;
  if (a.src.capacity() == 0) return 0;           // no tokens to move
  const int64_t most = a.budget < a.src.capacity() ? a.budget : a.src.capacity();
  kv4_move_kernel<<<dim3((unsigned)((most + kRowsThreads / 8 - 1) / (kRowsThreads / 8)),
                         (unsigned)a.src.n_kv, (unsigned)a.src.n_seqs), kRowsThreads, 0, st>>>(a);
  return cudaGetLastError() == cudaSuccess ? 0 : 1;
}

}  // namespace hq

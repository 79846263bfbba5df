// hq_kv4_attn.cu -- attention over the 4-bit window cache, read straight from
// the codes (include/hq_kv4.h).  The transform moves to the other operand:
// with y' = H D q / sqrt(128), q . Khat[t] = s_t sum_d y'_d (c_d - 7.5), and
// sum_t p_t Vhat[t] = D H (sum_t p_t s_t (c_t - 7.5)) / sqrt(128), one
// transform per output row.
#include <cuda_runtime.h>

#include <cmath>

#include "hq_device.cuh"
#include "hq_kv4.h"
#include "hq_kv4_io.cuh"

namespace hq {

constexpr float kInvRoot128 = 0.08838834764831845f;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kSimpleThreads = 128;

template <int KIND>
__device__ __forceinline__ void load_q16(const Kv4AttnArgs &a, int64_t at, int r, float x[16]) {
  load_row16<KIND>(a.q, at, r, a.q_vec != 0, x);
}

// One query row a block: every warp takes every fourth token, lane l of a
// warp the dimensions 4 l .. 4 l + 3.
__global__ void __launch_bounds__(kSimpleThreads) kv4_attn_kernel(Kv4AttnArgs a) {
  __shared__ __align__(16) float s_tr[4 * kTrTile];
  __shared__ __align__(16) float s_q[kTile];
  __shared__ float s_m[4], s_l[4], s_acc[4][kTile];
  const int hq = blockIdx.x, j = blockIdx.y, b = blockIdx.z, tid = threadIdx.x;
  const int h = hq / a.G, row = j * a.G + hq % a.G, lane = tid & 31, warp = tid >> 5;
  bool bad;
  const int len = kv4_length(a.c, a.lengths, b, &bad);
  if (bad && tid == 0) atomicOr(a.status, (uint32_t)HQ_ERR_PAGE);
  const int n = max(0, len - a.q_len + j + 1);
  const int r = tid & 7;
  const uint32_t mw = __ldg(a.c.signs + (r >> 1)) >> (16 * (r & 1));
  if (warp == 0) {
    float x[16];
    const int64_t at = b * a.q_seq + j * a.q_token + hq * a.q_head;
    if (a.kind == HQ_T_F32) load_q16<HQ_T_F32>(a, at, r, x);
    else if (a.kind == HQ_T_F16) load_q16<HQ_T_F16>(a, at, r, x);
    else load_q16<HQ_T_BF16>(a, at, r, x);
#pragma unroll
    for (int i = 0; i < 16; ++i)
      x[i] = __fmul_rn(__uint_as_float(__float_as_uint(x[i]) ^ (((mw >> i) & 1u) << 31)), kInvRoot128);
    fwht128_t8(x, s_tr + (lane >> 3) * kTrTile, r);
    if (lane < 8)
      for (int i = 0; i < 16; ++i) s_q[16 * r + i] = x[i];
  }
  __syncthreads();
  float q[4], acc[4] = {0.f, 0.f, 0.f, 0.f}, m = -3.0e38f, l = 0.0f;
  for (int i = 0; i < 4; ++i) q[i] = s_q[4 * lane + i];
  const int64_t head = (int64_t)b * a.c.n_kv + h;
  float *zrow = a.mass_out ? a.z + (head * a.R + row) * a.c.capacity() : nullptr;
  for (int t = warp; t < n; t += 4) {
    const int64_t page = kv4_page(a.c, b, t);
    float z = -INFINITY;
    if (page >= 0) {
      const unsigned char *u = kv4_unit(a.c, page, h, t);
      const int tok = t % kUnit;
      const uint32_t kw = *reinterpret_cast<const uint16_t *>(u + tok * 64 + 2 * lane);
      float s = 0.0f;
      for (int i = 0; i < 4; ++i) s = __fmaf_rn(q[i], (float)((kw >> (4 * i)) & 15u) - 7.5f, s);
      for (int d = 16; d >= 1; d >>= 1) s = __fadd_rn(s, __shfl_xor_sync(0xffffffffu, s, d));
      z = __fmul_rn(__fmul_rn(s, bf16_to_f32(reinterpret_cast<const uint16_t *>(u + kUnitKs)[tok])), a.scale);
      if (a.cap > 0.0f) z = __fmul_rn(a.cap, tanhf(__fdiv_rn(z, a.cap)));
      z = __fmul_rn(z, kLog2e);
      const uint32_t vw = *reinterpret_cast<const uint16_t *>(u + kUnitV + (tok >> 1) * 128 + (lane >> 2) * 16 +
                                                             (tok & 1) * 8 + 2 * (lane & 3));
      const float mm = fmaxf(m, z), f = exp2f(__fsub_rn(m, mm)), p = exp2f(__fsub_rn(z, mm));
      const float w = __fmul_rn(p, bf16_to_f32(reinterpret_cast<const uint16_t *>(u + kUnitVs)[tok]));
      m = mm;
      l = __fmaf_rn(l, f, p);
      for (int i = 0; i < 4; ++i)
        acc[i] = __fmaf_rn(w, (float)((vw >> (4 * i)) & 15u) - 7.5f, __fmul_rn(acc[i], f));
    } else if (lane == 0) {
      atomicOr(a.status, (uint32_t)HQ_ERR_PAGE);
    }
    if (zrow != nullptr && lane == 0) zrow[t] = z;
  }
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
  for (int i = 0; i < 4; ++i) s_acc[warp][4 * lane + i] = acc[i];
  __syncthreads();
  float M = fmaxf(fmaxf(s_m[0], s_m[1]), fmaxf(s_m[2], s_m[3])), L = 0.0f;
  for (int w = 0; w < 4; ++w) L = __fmaf_rn(s_l[w], exp2f(__fsub_rn(s_m[w], M)), L);
  if (warp == 0) {                               // D H (acc / L) / sqrt(128)
    float x[16];
    for (int i = 0; i < 16; ++i) {
      float v = 0.0f;
      for (int w = 0; w < 4; ++w)
        v = __fmaf_rn(s_acc[w][16 * r + i], exp2f(__fsub_rn(s_m[w], M)), v);
      x[i] = L == 0.0f ? 0.0f : __fmul_rn(__fdiv_rn(v, L), kInvRoot128);
    }
    fwht128_t8(x, s_tr + (lane >> 3) * kTrTile, r);
    for (int i = 0; i < 16; ++i) x[i] = __uint_as_float(__float_as_uint(x[i]) ^ (((mw >> i) & 1u) << 31));
    const int64_t o = ((int64_t)b * a.q_len + j) * a.Hq + hq;
    if (lane < 8) {
      if (a.out_kind == HQ_T_F32) store_row16<HQ_T_F32>(a.out, o * kTile, r, true, x);
      else if (a.out_kind == HQ_T_F16) store_row16<HQ_T_F16>(a.out, o * kTile, r, true, x);
      else store_row16<HQ_T_BF16>(a.out, o * kTile, r, true, x);
    }
    if (lane == 0) {
      const float l2 = L == 0.0f ? -INFINITY : __fadd_rn(M, log2f(L));
      if (a.lse != nullptr) a.lse[o] = __fmul_rn(l2, kLn2);
      if (a.mass_out != nullptr) a.row_lse[head * a.R + row] = l2;
    }
  }
}

// mass_out = mass_in + sum over the head's rows of exp2(z - lse).
__global__ void __launch_bounds__(256) kv4_mass_kernel(Kv4AttnArgs a) {
  const int h = blockIdx.y, b = blockIdx.z;
  const int64_t t = (int64_t)blockIdx.x * 256 + threadIdx.x;
  bool bad;
  const int len = kv4_length(a.c, a.lengths, b, &bad);
  if (t >= len) return;
  const int64_t head = (int64_t)b * a.c.n_kv + h, cap = a.c.capacity();
  float s = 0.0f;
  for (int row = 0; row < a.R; ++row) {
    if (t > len - a.q_len + row / a.G) continue;
    const float z = a.z[(head * a.R + row) * cap + t];
    if (z > -INFINITY || z != z) s = __fadd_rn(s, exp2f(__fsub_rn(z, a.row_lse[head * a.R + row])));
  }
  a.mass_out[head * cap + t] = a.mass_in != nullptr ? __fadd_rn(a.mass_in[head * cap + t], s) : s;
}

int launch_kv4_attention(const Kv4AttnArgs &a, cudaStream_t st) {
  kv4_attn_kernel<<<dim3((unsigned)a.Hq, (unsigned)a.q_len, (unsigned)a.c.n_seqs), kSimpleThreads, 0, st>>>(a);
  if (cudaGetLastError() != cudaSuccess) return 1;
  if (a.mass_out != nullptr) {
    kv4_mass_kernel<<<dim3((unsigned)((a.c.capacity() + 255) / 256), (unsigned)a.c.n_kv,
                           (unsigned)a.c.n_seqs), 256, 0, st>>>(a);
    if (cudaGetLastError() != cudaSuccess) return 1;
  }
  return 0;
}

}  // namespace hq

// hq_kv4_io.cuh -- rows of bf16, fp16 or fp32 values spread over 8 lanes
// (lane r holds dimensions 16 r .. 16 r + 15) and the roundings out of fp32.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/hq_kv4.h"

namespace hq {

__device__ __forceinline__ void unpack16(int kind, const uint4 &w, float *x) {
  const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (kind == HQ_T_BF16) {
      x[2 * i] = __uint_as_float(u[i] << 16);
      x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&u[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
}

// The lane's 16 values of a row that starts at element `at` of `base`;
// KIND is HQ_T_BF16, HQ_T_F16 or HQ_T_F32 (every conversion is exact).
template <int KIND>
__device__ __forceinline__ void load_row16(const void *base, int64_t at, int r, bool vec, float x[16]) {
  if constexpr (KIND == HQ_T_F32) {
    const float *p = static_cast<const float *>(base) + at + 16 * r;
    if (vec) {
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float4 v = __ldg(reinterpret_cast<const float4 *>(p) + c);
        x[4 * c] = v.x; x[4 * c + 1] = v.y; x[4 * c + 2] = v.z; x[4 * c + 3] = v.w;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = __ldg(p + i);
    }
  } else {
    const uint16_t *p = static_cast<const uint16_t *>(base) + at + 16 * r;
    uint4 w[2];
    if (vec) {
      w[0] = __ldg(reinterpret_cast<const uint4 *>(p));
      w[1] = __ldg(reinterpret_cast<const uint4 *>(p) + 1);
    } else {
      uint32_t u[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) u[i] = (uint32_t)__ldg(p + 2 * i) | ((uint32_t)__ldg(p + 2 * i + 1) << 16);
      w[0] = make_uint4(u[0], u[1], u[2], u[3]);
      w[1] = make_uint4(u[4], u[5], u[6], u[7]);
    }
    unpack16(KIND, w[0], x);
    unpack16(KIND, w[1], x + 8);
  }
}

// fp32 -> two 16-bit values in one word, each rounded to nearest even.
template <int KIND>
__device__ __forceinline__ uint32_t round_pair(float lo, float hi) {
  if constexpr (KIND == HQ_T_BF16) {
    const __nv_bfloat162 b = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&b);
  } else {
    const __half2 b = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&b);
  }
}

// The lane's 16 values into a row that starts at element `at` of `base`.
template <int KIND>
__device__ __forceinline__ void store_row16(void *base, int64_t at, int r, bool vec, const float x[16]) {
  if constexpr (KIND == HQ_T_F32) {
    float *p = static_cast<float *>(base) + at + 16 * r;
    if (vec) {
#pragma unroll
      for (int c = 0; c < 4; ++c)
        reinterpret_cast<float4 *>(p)[c] = make_float4(x[4 * c], x[4 * c + 1], x[4 * c + 2], x[4 * c + 3]);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) p[i] = x[i];
    }
  } else {
    uint16_t *p = static_cast<uint16_t *>(base) + at + 16 * r;
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = round_pair<KIND>(x[2 * i], x[2 * i + 1]);
    if (vec) {
      reinterpret_cast<uint4 *>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
      reinterpret_cast<uint4 *>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        p[2 * i] = (uint16_t)w[i];
        p[2 * i + 1] = (uint16_t)(w[i] >> 16);
      }
    }
  }
}

}  // namespace hq

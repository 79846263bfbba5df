// hq_kv4_io.cuh -- rows of bf16, fp16 or fp32 values spread over 8 lanes
// (lane r holds dimensions 16 r .. 16 r + 15) and the roundings out of fp32.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/hq_kv4.h"

namespace hq {

// 8 packed 16-bit values to fp32 (exact).
template <int KIND>
__device__ __forceinline__ void unpack8(const uint32_t u[4], float *x) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (KIND == HQ_T_BF16) {
      x[2 * i] = __uint_as_float(u[i] << 16);
      x[2 * i + 1] = __uint_as_float(u[i] & 0xFFFF0000u);
    } else {
      const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&u[i]));
      x[2 * i] = f.x;
      x[2 * i + 1] = f.y;
    }
  }
}

// The lane's 16 values of a row, as they are in memory: 8 words of 16-bit or
// 16 of 32-bit values, from element `at` of `base` on.
template <int KIND>
struct Row16 {
  static constexpr int words = KIND == HQ_T_F32 ? 16 : 8;
  uint32_t w[words];
  __device__ __forceinline__ void load(const void *base, int64_t at, int r, bool vec) {
    if constexpr (KIND == HQ_T_F32) {
      const uint32_t *p = static_cast<const uint32_t *>(base) + at + 16 * r;
      if (vec) {
#pragma unroll
        for (int c = 0; c < 4; ++c) put4(4 * c, reinterpret_cast<const uint4 *>(p)[c]);
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) w[i] = p[i];
      }
    } else {
      const uint16_t *p = static_cast<const uint16_t *>(base) + at + 16 * r;
      if (vec) {
        put4(0, reinterpret_cast<const uint4 *>(p)[0]);
        put4(4, reinterpret_cast<const uint4 *>(p)[1]);
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = (uint32_t)p[2 * i] | ((uint32_t)p[2 * i + 1] << 16);
      }
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < words; ++i) w[i] = 0u;
  }
  // The values in fp32, those whose bit of `flips` (bits 0-15) is set negated.
  __device__ __forceinline__ void get(uint32_t flips, float x[16]) const {
    if constexpr (KIND == HQ_T_F32) {
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = __uint_as_float(w[i] ^ ((flips << (31 - i)) & 0x80000000u));
    } else {
      uint32_t u[8];
      // bits 2 i and 2 i + 1 of flips at bits 15 and 31 of the 64-bit word shifted by 2 i
      const uint32_t low = (flips << 15) | (flips << 30 & 0x80000000u), high = flips >> 2;
#pragma unroll
      for (int i = 0; i < 8; ++i) u[i] = w[i] ^ (__funnelshift_r(low, high, 2 * i) & 0x80008000u);
      unpack8<KIND>(u, x);
      unpack8<KIND>(u + 4, x + 8);
    }
  }

 private:
  __device__ __forceinline__ void put4(int i, uint4 v) {
    w[i] = v.x; w[i + 1] = v.y; w[i + 2] = v.z; w[i + 3] = v.w;
  }
};

template <int KIND>
__device__ __forceinline__ void load_row16(const void *base, int64_t at, int r, bool vec, float x[16]) {
  Row16<KIND> row;
  row.load(base, at, r, vec);
  row.get(0u, x);
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

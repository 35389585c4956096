// Loads and stores of bf16 or fp32 values as fp32 registers.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace lq {

// VEC consecutive values as they lie in memory: 16 bytes, or one value.
template <bool BF16, int VEC>
struct Raw {
  uint4 v;
  __device__ __forceinline__ void load(const void *p, int64_t i) {
    v = *reinterpret_cast<const uint4 *>(static_cast<const char *>(p) + i * (BF16 ? 2 : 4));
  }
};
template <bool BF16>
struct Raw<BF16, 1> {
  uint32_t v;
  __device__ __forceinline__ void load(const void *p, int64_t i) {
    if constexpr (BF16)
      v = static_cast<uint32_t>(static_cast<const uint16_t *>(p)[i]) << 16;
    else
      v = static_cast<const uint32_t *>(p)[i];
  }
};

// The same as fp32.
template <bool BF16, int VEC>
struct Chunk {
  float x[VEC];
  __device__ __forceinline__ void set(const Raw<BF16, VEC> &r) {
    if constexpr (VEC == 1) {
      x[0] = __uint_as_float(r.v);
    } else {
      const uint32_t w[4] = {r.v.x, r.v.y, r.v.z, r.v.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if constexpr (BF16) {
          x[2 * j] = __uint_as_float(w[j] << 16);
          x[2 * j + 1] = __uint_as_float(w[j] & 0xffff0000u);
        } else {
          x[j] = __uint_as_float(w[j]);
        }
      }
    }
  }
  __device__ __forceinline__ void store(void *p, int64_t i) const { store_as<BF16>(p, i); }
  // As another type: VEC values, aligned to their size in it (16 bytes at most).
  template <bool OUT16>
  __device__ __forceinline__ void store_as(void *p, int64_t i) const {
    if constexpr (OUT16) {
      __nv_bfloat16 *o = reinterpret_cast<__nv_bfloat16 *>(p) + i;
      if constexpr (VEC == 1) {
        o[0] = __float2bfloat16_rn(x[0]);
      } else {
        uint32_t w[VEC / 2];
#pragma unroll
        for (int j = 0; j < VEC / 2; ++j) {
          const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * j], x[2 * j + 1]);
          w[j] = *reinterpret_cast<const uint32_t *>(&v);
        }
        if constexpr (VEC == 8)
          *reinterpret_cast<uint4 *>(o) = make_uint4(w[0], w[1], w[2], w[3]);
        else
          *reinterpret_cast<uint2 *>(o) = make_uint2(w[0], w[1]);
      }
    } else {
      float *o = reinterpret_cast<float *>(p) + i;
      if constexpr (VEC == 1) {
        o[0] = x[0];
      } else {
#pragma unroll
        for (int j = 0; j < VEC; j += 4)
          *reinterpret_cast<float4 *>(o + j) = make_float4(x[j], x[j + 1], x[j + 2], x[j + 3]);
      }
    }
  }
};

}  // namespace lq

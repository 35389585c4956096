// Device code that the kernels of the decayed linear attention share.
#pragma once

#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "lq_internal.h"
#include "lq_layer.h"

namespace lq {

constexpr unsigned kAllLanes = 0xffffffffu;

template <bool BF16>
__device__ __forceinline__ float load_value(const void *p, int64_t i) {
  if constexpr (BF16)
    return __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(p)[i]);
  else
    return reinterpret_cast<const float *>(p)[i];
}

// Four consecutive values (8- or 16-byte aligned).
template <bool BF16>
__device__ __forceinline__ float4 load_four(const void *p, int64_t i) {
  if constexpr (BF16) {
    const uint2 u = *reinterpret_cast<const uint2 *>(reinterpret_cast<const __nv_bfloat16 *>(p) + i);
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u),
                       __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
  } else {
    return *reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(p) + i);
  }
}

__device__ __forceinline__ void store_value(void *p, int64_t i, float x, int bf16) {
  if (bf16)
    reinterpret_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(x);
  else
    reinterpret_cast<float *>(p)[i] = x;
}

// The pool slot of sequence b, -1 if it has none that can be used.
__device__ __forceinline__ int slot_in_range(const LinParams &p, int b, bool report) {
  const int slot = p.slots != nullptr ? p.slots[b] : b;
  if (slot < 0) return -1;
  if (slot >= p.num_slots) {
    if (report && threadIdx.x == 0) atomicOr(p.err, kErrBadPhase);
    return -1;
  }
  return slot;
}

// Whether an earlier sequence of the call names the same slot (two sequences
// would race on its state).  Called by the whole block; it is one pass over
// the slots before b, which all blocks find in L2.
__device__ __forceinline__ bool slot_taken(const LinParams &p, int b, int slot, bool report) {
  if (p.slots == nullptr) return false;
  int hit = 0;
  for (int i = threadIdx.x; i < b; i += blockDim.x) hit |= p.slots[i] == slot;
  if (!__syncthreads_or(hit)) return false;
  if (report && threadIdx.x == 0) atomicOr(p.err, kErrBadPhase);
  return true;
}

// Sequence b's tokens: first and count; -1 if its offsets are not ascending
// within the call's rows.
struct Span {
  int first, count;
};
__device__ __forceinline__ Span sequence_span(const LinParams &p, int b) {
  const int lo = p.offsets[b], hi = p.offsets[b + 1];
  if (lo < 0 || hi < lo || hi > p.tokens) return {0, -1};
  return {lo, hi - lo};
}

// A warp's share of state rows: 8 rows of DK columns, 4 columns a lane, LPR
// lanes a row and NP passes.  Sums over a row leave pass (lane % LPR) / 4 of
// the lane's row group in every lane.
template <int DK>
struct RowMap {
  static constexpr int LPR = DK / 4;
  static constexpr int RPP = 32 / LPR;  // rows a pass
  static constexpr int NP = 8 / RPP;
  static __device__ __forceinline__ int col(int lane) { return lane % LPR * 4; }
  static __device__ __forceinline__ int row(int lane, int pass) { return pass * RPP + lane / LPR; }
  // NP row sums over LPR lanes, halving the values a lane holds at each step
  // while there are any: NP - 1 + 2 shuffles instead of NP log2(LPR).
  static __device__ __forceinline__ float reduce(float (&x)[NP], int lane) {
    int nv = NP;
#pragma unroll
    for (int off = LPR / 2; off >= 1; off >>= 1) {
      if (nv > 1) {
        nv >>= 1;
        const bool upper = (lane & off) != 0;
#pragma unroll
        for (int i = 0; i < NP / 2; ++i) {
          if (i >= nv) break;
          const float send = upper ? x[i] : x[i + nv];
          const float keep = upper ? x[i + nv] : x[i];
          x[i] = keep + __shfl_xor_sync(kAllLanes, send, off);
        }
      } else {
        x[0] += __shfl_xor_sync(kAllLanes, x[0], off);
      }
    }
    return x[0];
  }
  static __device__ __forceinline__ bool writes(int lane) { return (lane & 3) == 0; }
  static __device__ __forceinline__ int reduced_row(int lane) { return row(lane, (lane % LPR) >> 2); }
};

}  // namespace lq

// Group norm with an activation or a gate, channels last: each (token, group)
// row of `size` values is normalised by itself.
//
// Bound by the bytes of x, the gate and out: a row is read once into
// registers, its statistics are two reductions over the lanes that hold it
// (the variance from the centred values), and it is written once.  Rows of up
// to a warp's registers take 1 to 32 lanes, several rows a warp; longer rows
// take a block.  Blocks walk over the rows with a step that is a multiple of
// `groups`, so that a lane keeps the weights of its channels in registers.

#include "lq_chunk.cuh"
#include "lq_layer.h"

namespace lq {
namespace {

constexpr int kNT = 256;
constexpr unsigned kAllLanes = 0xffffffffu;

__device__ __forceinline__ float activate(int act, float x) {
  if (act == 0) return x;
  const float s = __fdividef(1.0f, 1.0f + expf(-x));
  return act == 1 ? x * s : s;
}

// Sum over the `lanes` lanes (a power of two) or the block that hold a row.
template <bool BLOCK>
__device__ __forceinline__ float row_sum(float x, int lanes, float *scratch) {
  for (int o = lanes >> 1; o > 0; o >>= 1) x += __shfl_xor_sync(kAllLanes, x, o);
  if constexpr (BLOCK) {
    __syncthreads();
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = x;
    __syncthreads();
    x = 0.0f;
#pragma unroll
    for (int i = 0; i < kNT / 32; ++i) x += scratch[i];
  }
  return x;
}

// `lanes` threads a row (kNT with BLOCK), CPL chunks of VEC values each.
// `blocks` is the grid; blocks * (kNT / lanes) % groups == 0 unless every row
// has threads of its own.
template <bool BF16, bool OUT16, int VEC, int CPL, bool BLOCK>
__global__ void __launch_bounds__(kNT) norm_kernel(const NormParams p, int lanes) {
  __shared__ float scratch[kNT / 32];
  const int per = BLOCK ? 1 : kNT / lanes;  // rows of a block at a time
  const int lane = BLOCK ? threadIdx.x : threadIdx.x % lanes;
  const int width = BLOCK ? kNT : lanes;
  const int64_t rows = static_cast<int64_t>(p.tokens) * p.groups;
  const int64_t step = static_cast<int64_t>(gridDim.x) * per;
  int64_t row = static_cast<int64_t>(blockIdx.x) * per + (BLOCK ? 0 : threadIdx.x / lanes);
  int64_t token = row / p.groups;
  const int group = static_cast<int>(row - token * p.groups);
  const int64_t token_step = step / p.groups;
  const float inv = 1.0f / p.size;
  float w[CPL][VEC], bias[CPL][VEC];
#pragma unroll
  for (int c = 0; c < CPL; ++c)
#pragma unroll
    for (int j = 0; j < VEC; ++j) {
      const int at = (c * width + lane) * VEC + j;
      const bool in = at < p.size;
      w[c][j] = in && p.weight ? p.weight[p.shared_weight ? at : group * p.size + at] : 1.0f;
      bias[c][j] = in && p.bias ? p.bias[group * p.size + at] : 0.0f;
    }
  // every lane of a warp takes part in the reductions until its warp is done
  const int64_t base = row - (BLOCK ? 0 : (threadIdx.x & 31) / lanes);
  for (int64_t first = base; first < rows; first += step, row += step, token += token_step) {
    const bool live = row < rows;
    const int64_t xat = token * p.x_stride + static_cast<int64_t>(group) * p.size;
    const int64_t zat = token * p.gate_stride + static_cast<int64_t>(group) * p.size;
    Chunk<BF16, VEC> x[CPL], z[CPL];
#pragma unroll
    for (int c = 0; c < CPL; ++c) {
      const int at = (c * width + lane) * VEC;
      const bool in = live && at < p.size;
#pragma unroll
      for (int j = 0; j < VEC; ++j) x[c].x[j] = z[c].x[j] = 0.0f;
      if (in) {
        x[c].load(p.x, xat + at);
        if (p.gate) z[c].load(p.gate, zat + at);
      }
    }
    float sum = 0.0f;
#pragma unroll
    for (int c = 0; c < CPL; ++c)
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        if (p.gate) {
          z[c].x[j] = activate(p.act, z[c].x[j]);
          if (p.gate_before) x[c].x[j] *= z[c].x[j];
        }
        sum += x[c].x[j];
      }
    const float mean = p.kind == 1 ? row_sum<BLOCK>(sum, BLOCK ? 32 : lanes, scratch) * inv : 0.0f;
    float sq = 0.0f;
#pragma unroll
    for (int c = 0; c < CPL; ++c) {
      if ((c * width + lane) * VEC >= p.size) continue;
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        x[c].x[j] -= mean;
        sq = fmaf(x[c].x[j], x[c].x[j], sq);
      }
    }
    const float var = row_sum<BLOCK>(sq, BLOCK ? 32 : lanes, scratch) * inv;
    const float scale = rsqrtf(var + p.eps);
    const int64_t oat = token * p.out_stride + static_cast<int64_t>(group) * p.size;
#pragma unroll
    for (int c = 0; c < CPL; ++c) {
      const int at = (c * width + lane) * VEC;
#pragma unroll
      for (int j = 0; j < VEC; ++j) {
        const float y = fmaf(x[c].x[j] * scale, w[c][j], bias[c][j]);
        x[c].x[j] = p.gate == nullptr ? activate(p.act, y) : p.gate_before ? y : y * z[c].x[j];
      }
      if (live && at < p.size) x[c].template store_as<OUT16>(p.out, oat + at);
    }
  }
}

template <bool BF16, bool OUT16, int VEC, int CPL, bool BLOCK>
cudaError_t norm_t(const NormParams &p, int lanes, cudaStream_t st) {
  const int64_t rows = static_cast<int64_t>(p.tokens) * p.groups;
  const int64_t per = BLOCK ? 1 : kNT / lanes;
  const int64_t all = (rows + per - 1) / per;
  // blocks that keep a lane on one group: a multiple of groups / gcd(groups, per)
  int64_t unit = p.groups;
  for (int64_t g = per; unit % 2 == 0 && g > 1; g /= 2) unit /= 2;
  const int64_t want = 148 * 16;
  int64_t grid = all;
  if (all > want && unit <= want) grid = want / unit * unit;
  if (grid > INT32_MAX) return cudaErrorInvalidConfiguration;
  norm_kernel<BF16, OUT16, VEC, CPL, BLOCK>
      <<<static_cast<unsigned>(grid), kNT, 0, st>>>(p, lanes);
  return cudaGetLastError();
}

template <bool BF16, bool OUT16, int VEC>
cudaError_t norm_v(const NormParams &p, cudaStream_t st) {
  const int chunks = (p.size + VEC - 1) / VEC;
  constexpr int kMost = VEC == 1 ? 16 : 4;  // chunks of a lane within a warp
  if (chunks > 32 * kMost) return norm_t<BF16, OUT16, VEC, 8192 / kNT / VEC, true>(p, kNT, st);
  int lanes = 1;
  while (lanes < 32 && lanes < chunks) lanes *= 2;
  const int cpl = (chunks + lanes - 1) / lanes;
  if (cpl <= 1) return norm_t<BF16, OUT16, VEC, 1, false>(p, lanes, st);
  if (cpl <= kMost / 2) return norm_t<BF16, OUT16, VEC, kMost / 2, false>(p, lanes, st);
  return norm_t<BF16, OUT16, VEC, kMost, false>(p, lanes, st);
}

template <bool BF16, bool OUT16>
cudaError_t norm_io(const NormParams &p, cudaStream_t st) {
  constexpr int VEC = BF16 ? 8 : 4;
  bool wide = p.size % VEC == 0 && p.x_stride % VEC == 0 && p.out_stride % VEC == 0 &&
              reinterpret_cast<uintptr_t>(p.x) % 16 == 0 &&
              reinterpret_cast<uintptr_t>(p.out) % 16 == 0;
  if (p.gate != nullptr)
    wide = wide && p.gate_stride % VEC == 0 && reinterpret_cast<uintptr_t>(p.gate) % 16 == 0;
  return wide ? norm_v<BF16, OUT16, VEC>(p, st) : norm_v<BF16, OUT16, 1>(p, st);
}

}  // namespace

cudaError_t launch_group_norm(const NormParams &p, cudaStream_t st) {
  if (p.in_bf16) return p.out_bf16 ? norm_io<true, true>(p, st) : norm_io<true, false>(p, st);
  return p.out_bf16 ? norm_io<false, true>(p, st) : norm_io<false, false>(p, st);
}

}  // namespace lq

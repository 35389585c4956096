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

__device__ __forceinline__ float exp2_of(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float inverse_of(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The activation of a row's values: one choice for all of them.  exp(-x) is
// 2^(-x log2 e) with the product rounded once, an error of |x| 2^-24 of the
// result; both approximations are good to 2^-22, and past 2^126 the inverse is
// a plain 0.
template <int N>
__device__ __forceinline__ void activate(int act, float (&x)[N]) {
  if (act == 0) return;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const float s = inverse_of(1.0f + exp2_of(x[j] * -1.4426950408889634f));
    x[j] = act == 1 ? x[j] * s : s;
  }
}

// Sums over the `lanes` lanes (a power of two) or the block that hold a row.
template <bool BLOCK, int U>
__device__ __forceinline__ void row_sums(float (&x)[U], int lanes, float *scratch) {
  for (int o = lanes >> 1; o > 0; o >>= 1)
#pragma unroll
    for (int u = 0; u < U; ++u) x[u] += __shfl_xor_sync(kAllLanes, x[u], o);
  if constexpr (BLOCK) {
    static_assert(U == 1, "a block holds one row");
    __syncthreads();
    if ((threadIdx.x & 31) == 0) scratch[threadIdx.x >> 5] = x[0];
    __syncthreads();
    x[0] = 0.0f;
#pragma unroll
    for (int i = 0; i < kNT / 32; ++i) x[0] += scratch[i];
  }
}

// `lanes` threads a row (kNT with BLOCK), CPL chunks of VEC values each, U rows
// at a time, all of their loads in flight.  Rows go round the blocks in steps
// of gridDim.x * (kNT / lanes), a multiple of `groups` unless every row has
// threads of its own.
template <bool BF16, bool OUT16, bool GATE, int VEC, int CPL, bool BLOCK, int U>
__global__ void __launch_bounds__(kNT, U > 1 ? 4 : 1) norm_kernel(const NormParams p, int lanes) {
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
  for (int64_t first = base; first < rows;
       first += U * step, row += U * step, token += U * token_step) {
    Raw<BF16, VEC> rx[U][CPL], rz[U][CPL];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t t = token + u * token_step;
      const int64_t at0 = static_cast<int64_t>(group) * p.size + lane * VEC;
      const int64_t xat = t * p.x_stride + at0, zat = t * p.gate_stride + at0;
#pragma unroll
      for (int c = 0; c < CPL; ++c) {
        rx[u][c] = {};
        if (GATE) rz[u][c] = {};
        if (row + u * step < rows && (c * width + lane) * VEC < p.size) {
          rx[u][c].load(p.x, xat + c * width * VEC);
          if (GATE) rz[u][c].load(p.gate, zat + c * width * VEC);
        }
      }
    }
    Chunk<BF16, VEC> x[U][CPL];
    float sum[U], sq[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      sum[u] = sq[u] = 0.0f;
#pragma unroll
      for (int c = 0; c < CPL; ++c) {
        x[u][c].set(rx[u][c]);
        if (GATE && p.gate_before) {
          Chunk<BF16, VEC> z;
          z.set(rz[u][c]);
          activate(p.act, z.x);
#pragma unroll
          for (int j = 0; j < VEC; ++j) x[u][c].x[j] *= z.x[j];
        }
#pragma unroll
        for (int j = 0; j < VEC; ++j) sum[u] += x[u][c].x[j];
      }
    }
    if (p.kind == 1) {
      row_sums<BLOCK, U>(sum, BLOCK ? 32 : lanes, scratch);
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int c = 0; c < CPL; ++c) {
          const float mean = (c * width + lane) * VEC < p.size ? sum[u] * inv : 0.0f;
#pragma unroll
          for (int j = 0; j < VEC; ++j) x[u][c].x[j] -= mean;
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int c = 0; c < CPL; ++c)
#pragma unroll
        for (int j = 0; j < VEC; ++j) sq[u] = fmaf(x[u][c].x[j], x[u][c].x[j], sq[u]);
    row_sums<BLOCK, U>(sq, BLOCK ? 32 : lanes, scratch);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const float scale = rsqrtf(fmaf(sq[u], inv, p.eps));
      const int64_t oat = (token + u * token_step) * p.out_stride +
                          static_cast<int64_t>(group) * p.size + lane * VEC;
#pragma unroll
      for (int c = 0; c < CPL; ++c) {
#pragma unroll
        for (int j = 0; j < VEC; ++j)
          x[u][c].x[j] = fmaf(x[u][c].x[j] * scale, w[c][j], bias[c][j]);
        if (!GATE) {
          activate(p.act, x[u][c].x);
        } else if (!p.gate_before) {
          Chunk<BF16, VEC> z;
          z.set(rz[u][c]);
          activate(p.act, z.x);
#pragma unroll
          for (int j = 0; j < VEC; ++j) x[u][c].x[j] *= z.x[j];
        }
        if (row + u * step < rows && (c * width + lane) * VEC < p.size)
          x[u][c].template store_as<OUT16>(p.out, oat + c * width * VEC);
      }
    }
  }
}

template <bool BF16, bool OUT16, bool GATE, int VEC, int CPL, bool BLOCK, int U>
cudaError_t norm_u(const NormParams &p, int lanes, int64_t grid, cudaStream_t st) {
  if (grid > INT32_MAX) return cudaErrorInvalidConfiguration;
  norm_kernel<BF16, OUT16, GATE, VEC, CPL, BLOCK, U>
      <<<static_cast<unsigned>(grid), kNT, 0, st>>>(p, lanes);
  return cudaGetLastError();
}

// One row a thread group where the rows do not fill the GPU twice; else blocks
// that all run at once and keep every lane on one group: a grid that is a
// multiple of groups / gcd(groups, rows of a block).  Then two rows at a time,
// but for fp32 with a gate, where a row's own loads are enough: 16,384 x 32 x
// 128, fp32 to bf16, 76 us with two and 90 with one (70 and 80 us with two by
// short bursts of calls and by long runs at the power cap); with a gate and fp32
// 130 and 105; bf16 throughout 63 and 72, with a gate 78 and 82.  Value by value
// (VEC = 1) neither side leads: 5,216 x 32 x 201, bf16, 92 with two and 105 with
// one, with a gate 155 and 139; 61,680 x 32 x 17, 124 and 120, 152 and 163.
template <bool BF16, bool OUT16, bool GATE, int VEC, int CPL, bool BLOCK>
cudaError_t norm_t(const NormParams &p, int lanes, cudaStream_t st) {
  const int64_t rows = static_cast<int64_t>(p.tokens) * p.groups;
  const int64_t per = BLOCK ? 1 : kNT / lanes;
  const int64_t all = (rows + per - 1) / per;
  int64_t unit = p.groups;
  for (int64_t g = per; unit % 2 == 0 && g > 1; g /= 2) unit /= 2;
  constexpr int kRows = BLOCK || CPL * VEC > 8 || (GATE && !BF16) ? 1 : 2;
  const int64_t want = 148 * 4;
  if (all <= 2 * want || unit > want)
    return norm_u<BF16, OUT16, GATE, VEC, CPL, BLOCK, 1>(p, lanes, all, st);
  return norm_u<BF16, OUT16, GATE, VEC, CPL, BLOCK, kRows>(p, lanes, want / unit * unit, st);
}

template <bool BF16, bool OUT16, bool GATE, int VEC>
cudaError_t norm_v(const NormParams &p, cudaStream_t st) {
  // Lanes of a row: 8 values a lane or so, which the reductions are shared by,
  // up to a warp; then up to kMost chunks a lane; then a block.
  const int chunks = (p.size + VEC - 1) / VEC;
  constexpr int kMost = VEC == 1 ? 16 : 4, kFew = VEC >= 8 ? 1 : VEC == 4 ? 2 : 8;
  if (chunks > 32 * kMost) return norm_t<BF16, OUT16, GATE, VEC, 8192 / kNT / VEC, true>(p, kNT, st);
  int lanes = 1;
  while (lanes < 32 && lanes * kFew < chunks) lanes *= 2;
  const int cpl = (chunks + lanes - 1) / lanes;
  if (cpl <= kFew) return norm_t<BF16, OUT16, GATE, VEC, kFew, false>(p, lanes, st);
  if (cpl <= kMost / 2 && kMost / 2 > kFew)
    return norm_t<BF16, OUT16, GATE, VEC, kMost / 2, false>(p, lanes, st);
  return norm_t<BF16, OUT16, GATE, VEC, kMost, false>(p, lanes, st);
}

template <bool BF16, bool OUT16>
cudaError_t norm_io(const NormParams &p, cudaStream_t st) {
  constexpr int VEC = BF16 ? 8 : 4;
  bool wide = p.size % VEC == 0 && p.x_stride % VEC == 0 && p.out_stride % VEC == 0 &&
              reinterpret_cast<uintptr_t>(p.x) % 16 == 0 &&
              reinterpret_cast<uintptr_t>(p.out) % 16 == 0;
  if (p.gate != nullptr)
    wide = wide && p.gate_stride % VEC == 0 && reinterpret_cast<uintptr_t>(p.gate) % 16 == 0;
  if (p.gate != nullptr)
    return wide ? norm_v<BF16, OUT16, true, VEC>(p, st) : norm_v<BF16, OUT16, true, 1>(p, st);
  return wide ? norm_v<BF16, OUT16, false, VEC>(p, st) : norm_v<BF16, OUT16, false, 1>(p, st);
}

}  // namespace

cudaError_t launch_group_norm(const NormParams &p, cudaStream_t st) {
  if (p.in_bf16) return p.out_bf16 ? norm_io<true, true>(p, st) : norm_io<true, false>(p, st);
  return p.out_bf16 ? norm_io<false, true>(p, st) : norm_io<false, false>(p, st);
}

}  // namespace lq

// Linear attention with a decay for each head,
//   S_t = a_t S_{t-1} + v_t k_t^T,   o_t = S_t q_t,
// one token for every sequence (linear_step_kernel) and token by token over
// packed prompts (linear_tokens_kernel).
//
// Rows of a state (value channels) are independent: row i needs v_i, the
// decay, k and q alone, and gives o_i.  Both kernels therefore take blocks of
// 32 rows, which is also what spreads a single sequence over the GPU.

#include "lq_linear_common.cuh"

namespace lq {
namespace {

constexpr int kRows = 32;  // state rows of a block: 8 a warp
constexpr int kNT = 128;

// One token.  Bound by the state's bytes: 16 KB read and written a block at
// dk = 128, all of its loads in flight before the first use.  The slots are
// compared with the earlier ones while the state is under way.
template <int DK, bool BF16>
__global__ void __launch_bounds__(kNT) linear_step_kernel(const LinParams p) {
  using M = RowMap<DK>;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int blocks = p.dv / kRows;
  const int tile = blockIdx.x / blocks, row0 = blockIdx.x % blocks * kRows + warp * 8;
  const int b = tile / p.Hv, h = tile - b * p.Hv, hk = h / (p.Hv / p.Hk);
  const bool report = blockIdx.x == b * p.Hv * blocks;
  const int slot = slot_in_range(p, b, report);
  if (slot < 0) return;
  float *S = p.S + ((static_cast<int64_t>(slot) * p.Hv + h) * p.dv + row0) * DK + M::col(lane);
  float4 s[M::NP];
#pragma unroll
  for (int i = 0; i < M::NP; ++i)
    s[i] = *reinterpret_cast<const float4 *>(S + M::row(lane, i) * DK);
  const float4 k = load_four<BF16>(p.k, b * p.k_stride + hk * DK + M::col(lane));
  const float4 q = load_four<BF16>(p.q, b * p.q_stride + hk * DK + M::col(lane));
  const float a = p.decay[p.decay_head ? h : tile];
  float v[M::NP];
#pragma unroll
  for (int i = 0; i < M::NP; ++i)
    v[i] = load_value<BF16>(p.v, b * p.v_stride + h * p.dv + row0 + M::row(lane, i));
  if (slot_taken(p, b, slot, report)) return;
  float o[M::NP];
#pragma unroll
  for (int i = 0; i < M::NP; ++i) {
    s[i].x = fmaf(a, s[i].x, v[i] * k.x);
    s[i].y = fmaf(a, s[i].y, v[i] * k.y);
    s[i].z = fmaf(a, s[i].z, v[i] * k.z);
    s[i].w = fmaf(a, s[i].w, v[i] * k.w);
    *reinterpret_cast<float4 *>(S + M::row(lane, i) * DK) = s[i];
    o[i] = fmaf(s[i].x, q.x, fmaf(s[i].y, q.y, fmaf(s[i].z, q.z, s[i].w * q.w)));
  }
  const float sum = M::reduce(o, lane);
  if (M::writes(lane))
    store_value(p.out, static_cast<int64_t>(tile) * p.dv + row0 + M::reduced_row(lane), sum,
                p.out_bf16);
}

// Packed prompts, one token after the other: the state rows stay in registers,
// kTok tokens of inputs at a time in shared memory.  Exact fp32 recurrence,
// any type and length.
constexpr int kTok = 32;

template <int DK>
struct TokensSmem {
  alignas(16) float q[kTok][DK];
  alignas(16) float k[kTok][DK];
  float v[kTok][kRows];
  float o[kTok][kRows];
  float a[kTok];
};

template <int DK, bool BF16>
__global__ void __launch_bounds__(kNT) linear_tokens_kernel(const LinParams p) {
  using M = RowMap<DK>;
  __shared__ TokensSmem<DK> sm;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int blocks = p.dv / kRows;
  const int tile = blockIdx.x / blocks, block0 = blockIdx.x % blocks * kRows;
  const int row0 = warp * 8;
  const int b = tile / p.Hv, h = tile - b * p.Hv, hk = h / (p.Hv / p.Hk);
  const bool report = blockIdx.x == b * p.Hv * blocks;
  const int slot = slot_in_range(p, b, report);
  if (slot < 0) return;
  if (slot_taken(p, b, slot, report)) return;
  const Span span = sequence_span(p, b);
  if (span.count < 0) {
    if (report && tid == 0) atomicOr(p.err, kErrBadPhase);
    return;
  }
  const bool fresh = p.fresh != nullptr && p.fresh[b] != 0;
  if (span.count == 0 && !fresh) return;
  float *S = p.S + ((static_cast<int64_t>(slot) * p.Hv + h) * p.dv + block0 + row0) * DK +
             M::col(lane);
  float4 s[M::NP];
#pragma unroll
  for (int i = 0; i < M::NP; ++i)
    s[i] = fresh ? make_float4(0.0f, 0.0f, 0.0f, 0.0f)
                 : *reinterpret_cast<const float4 *>(S + M::row(lane, i) * DK);
  for (int t0 = 0; t0 < span.count; t0 += kTok) {
    const int n = min(kTok, span.count - t0);
    const int64_t first = span.first + t0;
    for (int i = tid; i < n * (DK / 4); i += kNT) {
      const int t = i / (DK / 4), c = i % (DK / 4) * 4;
      *reinterpret_cast<float4 *>(&sm.q[t][c]) =
          load_four<BF16>(p.q, (first + t) * p.q_stride + hk * DK + c);
      *reinterpret_cast<float4 *>(&sm.k[t][c]) =
          load_four<BF16>(p.k, (first + t) * p.k_stride + hk * DK + c);
    }
    for (int i = tid; i < n * kRows; i += kNT)
      sm.v[i / kRows][i % kRows] =
          load_value<BF16>(p.v, (first + i / kRows) * p.v_stride + h * p.dv + block0 + i % kRows);
    if (tid < n) sm.a[tid] = p.decay[p.decay_head ? h : (first + tid) * p.Hv + h];
    __syncthreads();
#pragma unroll 2
    for (int t = 0; t < n; ++t) {
      const float4 q = *reinterpret_cast<const float4 *>(&sm.q[t][M::col(lane)]);
      const float4 k = *reinterpret_cast<const float4 *>(&sm.k[t][M::col(lane)]);
      const float a = sm.a[t];
      float o[M::NP];
#pragma unroll
      for (int i = 0; i < M::NP; ++i) {
        const float v = sm.v[t][row0 + M::row(lane, i)];
        s[i].x = fmaf(a, s[i].x, v * k.x);
        s[i].y = fmaf(a, s[i].y, v * k.y);
        s[i].z = fmaf(a, s[i].z, v * k.z);
        s[i].w = fmaf(a, s[i].w, v * k.w);
        o[i] = fmaf(s[i].x, q.x, fmaf(s[i].y, q.y, fmaf(s[i].z, q.z, s[i].w * q.w)));
      }
      const float sum = M::reduce(o, lane);
      if (M::writes(lane)) sm.o[t][row0 + M::reduced_row(lane)] = sum;
    }
    __syncthreads();
    if (p.out != nullptr)
      for (int i = tid; i < n * kRows; i += kNT)
        store_value(p.out,
                    ((first + i / kRows) * p.Hv + h) * p.dv + block0 + i % kRows,
                    sm.o[i / kRows][i % kRows], p.out_bf16);
  }
#pragma unroll
  for (int i = 0; i < M::NP; ++i)
    *reinterpret_cast<float4 *>(S + M::row(lane, i) * DK) = s[i];
}

template <int DK>
cudaError_t step_d(const LinParams &p, cudaStream_t st) {
  const int grid = p.B * p.Hv * (p.dv / kRows);
  if (p.in_bf16)
    linear_step_kernel<DK, true><<<grid, kNT, 0, st>>>(p);
  else
    linear_step_kernel<DK, false><<<grid, kNT, 0, st>>>(p);
  return cudaGetLastError();
}

template <int DK>
cudaError_t tokens_d(const LinParams &p, cudaStream_t st) {
  const int grid = p.B * p.Hv * (p.dv / kRows);
  if (p.in_bf16)
    linear_tokens_kernel<DK, true><<<grid, kNT, 0, st>>>(p);
  else
    linear_tokens_kernel<DK, false><<<grid, kNT, 0, st>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_linear_step(const LinParams &p, cudaStream_t st) {
  if (p.dk == 32) return step_d<32>(p, st);
  if (p.dk == 64) return step_d<64>(p, st);
  return step_d<128>(p, st);
}

cudaError_t launch_linear_tokens(const LinParams &p, cudaStream_t st) {
  if (p.dk == 32) return tokens_d<32>(p, st);
  if (p.dk == 64) return tokens_d<64>(p, st);
  return tokens_d<128>(p, st);
}

}  // namespace lq

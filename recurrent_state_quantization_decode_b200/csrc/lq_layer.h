// Internal interface between the layer operators' C ABI (lq_layer_capi.cu)
// and their kernels (lq_linear.cu, lq_rotary.cu, lq_norm.cu).  Not installed;
// callers use include/leapquant_layer.h.
#pragma once

#include <cstddef>
#include <cstdint>

#include <cuda_runtime.h>

namespace lq {

// Everything a launch of the decayed linear attention needs.
struct LinParams {
  int B, Hk, Hv, dk, dv, num_slots, tokens;
  int decay_head;  // decay is [Hv], else [tokens][Hv]
  int in_bf16, out_bf16;
  int64_t q_stride, k_stride, v_stride;  // elements from token to token
  const void *q, *k, *v;
  const float *decay;
  float *S;
  const int32_t *slots, *offsets, *fresh;
  void *out;
  int32_t *err;
};

struct RotaryParams {
  int tokens, Hq, Hk, d, rot, interleaved, bf16;
  float cos_mul, sin_mul;  // magnitude, and the magnitude with the direction's sign
  int64_t q_stride, k_stride, q_out_stride, k_out_stride;
  const void *q, *k;
  void *q_out, *k_out;
  const int32_t *positions;
  const uint64_t *table;
};

struct NormParams {
  int tokens, groups, size, kind, act, gate_before, shared_weight, in_bf16, out_bf16;
  float eps;
  int64_t x_stride, gate_stride, out_stride;
  const void *x, *gate;
  const float *weight, *bias;
  void *out;
};

cudaError_t launch_linear_step(const LinParams &p, cudaStream_t stream);
cudaError_t launch_linear_tokens(const LinParams &p, void *workspace, cudaStream_t stream);
cudaError_t launch_linear_chunks(const LinParams &p, void *workspace, cudaStream_t stream);
// What a prompt call needs, and the most that one of no more tokens and no more
// sequences does.
size_t linear_tokens_workspace(const LinParams &p);
size_t linear_chunks_workspace(const LinParams &p);
size_t linear_tokens_workspace_most(const LinParams &p);
size_t linear_chunks_workspace_most(const LinParams &p);
cudaError_t launch_rotary(const RotaryParams &p, cudaStream_t stream);
cudaError_t launch_group_norm(const NormParams &p, cudaStream_t stream);

}  // namespace lq

// C ABI of the layer operators (declared in include/leapquant_layer.h):
// argument validation on the host, then the call's launches.  No call here
// allocates memory or keeps global state.

#include <cmath>
#include <cstdint>
#include <cstring>

#include <cuda_runtime.h>

#include "../../include/leapquant_layer.h"
#include "lq_internal.h"
#include "lq_layer.h"

namespace {

bool aligned(const void *p, size_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }
bool is_dtype(int32_t t) { return t == LQ_DTYPE_F32 || t == LQ_DTYPE_BF16; }
size_t size_of(int32_t t) { return t == LQ_DTYPE_BF16 ? 2 : 4; }
lq_status from_cuda(cudaError_t e) { return e == cudaSuccess ? LQ_OK : LQ_ERR_CUDA; }

// A token stride: 0 means packed; below a token's row it would make tokens overlap.
bool resolve_stride(int64_t given, int64_t row, int64_t *out) {
  *out = given == 0 ? row : given;
  return given >= 0 && *out >= row;
}

lq_status check_linear(const lq_linear_config *c, lq::LinParams *p) {
  if (c == nullptr) return LQ_ERR_INVALID_ARG;
  if (c->batch < 0 || c->num_k_heads < 1 || c->num_v_heads < 1) return LQ_ERR_INVALID_ARG;
  if (c->num_v_heads % c->num_k_heads != 0) return LQ_ERR_INVALID_ARG;
  if (c->decay != LQ_DECAY_TOKEN && c->decay != LQ_DECAY_HEAD) return LQ_ERR_INVALID_ARG;
  if (!is_dtype(c->in_dtype) || !is_dtype(c->out_dtype)) return LQ_ERR_INVALID_ARG;
  for (const int32_t d : {c->dk, c->dv})
    if (d != 32 && d != 64 && d != 128) return LQ_ERR_UNSUPPORTED;
  // blocks (32 state rows each) and tiles are counted in 32 bits
  if (static_cast<int64_t>(c->batch) * c->num_v_heads * (c->dv / 32) > INT32_MAX)
    return LQ_ERR_UNSUPPORTED;
  // each block reads the earlier sequences' slots and lengths: a square of the batch
  if (c->batch > (1 << 16) || c->num_k_heads > 2048) return LQ_ERR_UNSUPPORTED;
  std::memset(p, 0, sizeof(*p));
  if (!resolve_stride(c->q_stride, static_cast<int64_t>(c->num_k_heads) * c->dk, &p->q_stride) ||
      !resolve_stride(c->k_stride, static_cast<int64_t>(c->num_k_heads) * c->dk, &p->k_stride) ||
      !resolve_stride(c->v_stride, static_cast<int64_t>(c->num_v_heads) * c->dv, &p->v_stride))
    return LQ_ERR_INVALID_ARG;
  const int64_t unit = 16 / static_cast<int64_t>(size_of(c->in_dtype));
  if (p->q_stride % unit != 0 || p->k_stride % unit != 0 || p->v_stride % unit != 0)
    return LQ_ERR_MISALIGNED;
  p->B = c->batch;
  p->Hk = c->num_k_heads;
  p->Hv = c->num_v_heads;
  p->dk = c->dk;
  p->dv = c->dv;
  p->decay_head = c->decay == LQ_DECAY_HEAD;
  p->in_bf16 = c->in_dtype == LQ_DTYPE_BF16;
  p->out_bf16 = c->out_dtype == LQ_DTYPE_BF16;
  return LQ_OK;
}

// What both forms take; `inputs`: whether there are tokens to read.
lq_status check_linear_io(const lq_linear_config *c, lq::LinParams *p, bool inputs, const void *q,
                          const void *k, const void *v, const float *decay, float *S,
                          int32_t num_slots, const int32_t *slots, void *out, int32_t *err) {
  if (inputs && (!q || !k || !v || !decay)) return LQ_ERR_INVALID_ARG;
  if (!S || !err || num_slots < 0) return LQ_ERR_INVALID_ARG;
  if (slots == nullptr && num_slots < c->batch) return LQ_ERR_INVALID_ARG;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(decay, 4) ||
      !aligned(S, 16) || !aligned(slots, 4) || !aligned(out, size_of(c->out_dtype)) ||
      !aligned(err, 4))
    return LQ_ERR_MISALIGNED;
  p->q = q;
  p->k = k;
  p->v = v;
  p->decay = decay;
  p->S = S;
  p->num_slots = num_slots;
  p->slots = slots;
  p->out = out;
  p->err = err;
  return LQ_OK;
}

// Which prompt kernel a call takes: bf16 inputs go to the tensor cores, unless
// sequences are so short on average that a chunk of 128 tokens would be mostly
// padding (64 sequences x 32 heads, d = 128: 16 tokens each 119 us token by
// token and 235 us in chunks, 32 each 198 and 240, 36 each 221 and 240, 48 each
// 279 and 243, 64 each 357 and 249).  The lengths themselves are on the device: a
// long sequence among many empty ones goes token by token by this rule, though
// chunks would be faster (7,900 tokens and 255 empty sequences, 32 heads: 1,154
// us; by itself, in chunks, 155).
bool by_chunks(const lq::LinParams &p) {
  return p.in_bf16 != 0 && p.tokens > 32 * static_cast<int64_t>(p.B);
}

}  // namespace

extern "C" {

lq_status lq_linear_decode_step(const lq_linear_config *cfg, const void *q, const void *k,
                                const void *v, const float *decay, float *S, int32_t num_slots,
                                const int32_t *slots, void *out, int32_t *err, void *stream) {
  lq::LinParams p;
  lq_status s = check_linear(cfg, &p);
  if (s != LQ_OK) return s;
  if (out == nullptr) return LQ_ERR_INVALID_ARG;
  if ((s = check_linear_io(cfg, &p, true, q, k, v, decay, S, num_slots, slots, out, err)) != LQ_OK)
    return s;
  if (cfg->batch == 0) return LQ_OK;
  p.tokens = cfg->batch;
  return from_cuda(lq::launch_linear_step(p, static_cast<cudaStream_t>(stream)));
}

size_t lq_linear_workspace_bytes(const lq_linear_config *cfg, int32_t tokens) {
  lq::LinParams p;
  if (check_linear(cfg, &p) != LQ_OK || tokens < 0) return 0;
  // the most of both kernels over the calls that each may get
  p.tokens = tokens;
  const size_t chunks = p.in_bf16 ? lq::linear_chunks_workspace_most(p) : 0;
  if (p.in_bf16 && tokens > 32 * static_cast<int64_t>(p.B)) p.tokens = 32 * p.B;
  const size_t others = lq::linear_tokens_workspace_most(p);
  return chunks > others ? chunks : others;
}

lq_status lq_linear_prefill(const lq_linear_config *cfg, const void *q, const void *k,
                            const void *v, const float *decay, int32_t tokens,
                            const int32_t *offsets, float *S, int32_t num_slots,
                            const int32_t *slots, const int32_t *fresh, void *out,
                            void *workspace, size_t workspace_bytes, int32_t *err, void *stream) {
  lq::LinParams p;
  lq_status s = check_linear(cfg, &p);
  if (s != LQ_OK) return s;
  if (tokens < 0 || offsets == nullptr) return LQ_ERR_INVALID_ARG;
  if ((s = check_linear_io(cfg, &p, tokens > 0, q, k, v, decay, S, num_slots, slots, out, err)) !=
      LQ_OK)
    return s;
  if (!aligned(offsets, 4) || !aligned(fresh, 4) || !aligned(workspace, 16))
    return LQ_ERR_MISALIGNED;
  p.tokens = tokens;
  const size_t need =
      by_chunks(p) ? lq::linear_chunks_workspace(p) : lq::linear_tokens_workspace(p);
  if (need > 0 && (workspace == nullptr || workspace_bytes < need)) return LQ_ERR_INVALID_ARG;
  if (cfg->batch == 0) return LQ_OK;
  p.offsets = offsets;
  p.fresh = fresh;
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  return from_cuda(by_chunks(p) ? lq::launch_linear_chunks(p, workspace, cs)
                                : lq::launch_linear_tokens(p, workspace, cs));
}

lq_status lq_rotary_table(int32_t rot, double theta, int32_t scaling, double factor,
                          double trained, double fast, double slow, uint64_t *table,
                          float *magnitude) {
  if (table == nullptr || rot < 2 || rot % 2 != 0) return LQ_ERR_INVALID_ARG;
  if (rot > 1024) return LQ_ERR_UNSUPPORTED;
  if (scaling < LQ_ROPE_NONE || scaling > LQ_ROPE_PARTS) return LQ_ERR_INVALID_ARG;
  if (!(theta >= 1.0) || !std::isfinite(theta)) return LQ_ERR_INVALID_ARG;
  if (scaling != LQ_ROPE_NONE && (!(factor >= 1.0) || !std::isfinite(factor)))
    return LQ_ERR_INVALID_ARG;
  if (scaling == LQ_ROPE_PARTS &&
      (!(trained > 0.0) || !std::isfinite(trained) || !(fast > slow) || !std::isfinite(fast) ||
       !std::isfinite(slow)))
    return LQ_ERR_INVALID_ARG;
  const double two_pi = 6.283185307179586476925286766559;
  if (scaling == LQ_ROPE_NTK && rot > 2)
    theta *= std::pow(factor, static_cast<double>(rot) / (rot - 2));
  for (int32_t i = 0; i < rot / 2; ++i) {
    double f = std::pow(theta, -2.0 * i / rot);
    if (scaling == LQ_ROPE_LINEAR) f /= factor;
    if (scaling == LQ_ROPE_PARTS) {
      const double keep =
          std::fmin(1.0, std::fmax(0.0, (trained * f / two_pi - slow) / (fast - slow)));
      f = f * keep + f / factor * (1.0 - keep);
    }
    // f <= 1 radian, below half a turn
    table[i] = static_cast<uint64_t>(std::ldexp(f / two_pi, 64) + 0.5);
  }
  if (magnitude != nullptr)
    *magnitude = scaling == LQ_ROPE_PARTS ? static_cast<float>(0.1 * std::log(factor) + 1.0) : 1.0f;
  return LQ_OK;
}

lq_status lq_rotary(const lq_rotary_config *cfg, int32_t tokens, const void *q, const void *k,
                    const int32_t *positions, const uint64_t *table, void *q_out, void *k_out,
                    void *stream) {
  if (cfg == nullptr || tokens < 0) return LQ_ERR_INVALID_ARG;
  const lq_rotary_config &c = *cfg;
  if (c.num_q_heads < 0 || c.num_k_heads < 0 || c.rot < 2 || c.rot % 2 != 0 || c.rot > c.d)
    return LQ_ERR_INVALID_ARG;
  if (c.layout != LQ_ROPE_HALF && c.layout != LQ_ROPE_INTERLEAVED) return LQ_ERR_INVALID_ARG;
  if (!is_dtype(c.dtype)) return LQ_ERR_INVALID_ARG;
  if (c.d > 1024 || static_cast<int64_t>(c.num_q_heads) + c.num_k_heads > 65535)
    return LQ_ERR_UNSUPPORTED;
  lq::RotaryParams p{};
  const int64_t q_row = static_cast<int64_t>(c.num_q_heads) * c.d;
  const int64_t k_row = static_cast<int64_t>(c.num_k_heads) * c.d;
  if (!resolve_stride(c.q_stride, q_row, &p.q_stride) ||
      !resolve_stride(c.k_stride, k_row, &p.k_stride) ||
      !resolve_stride(c.q_out_stride, q_row, &p.q_out_stride) ||
      !resolve_stride(c.k_out_stride, k_row, &p.k_out_stride))
    return LQ_ERR_INVALID_ARG;
  if (tokens == 0 || q_row + k_row == 0) return LQ_OK;
  if (positions == nullptr || table == nullptr || (q_row > 0 && (!q || !q_out)) ||
      (k_row > 0 && (!k || !k_out)))
    return LQ_ERR_INVALID_ARG;
  // in place, a token's row has to be read where it is written
  if ((q_row > 0 && q == q_out && p.q_stride != p.q_out_stride) ||
      (k_row > 0 && k == k_out && p.k_stride != p.k_out_stride))
    return LQ_ERR_INVALID_ARG;
  const size_t e = size_of(c.dtype);
  if ((q_row > 0 && (!aligned(q, e) || !aligned(q_out, e))) ||
      (k_row > 0 && (!aligned(k, e) || !aligned(k_out, e))) || !aligned(positions, 4) ||
      !aligned(table, 8))
    return LQ_ERR_MISALIGNED;
  p.tokens = tokens;
  p.Hq = c.num_q_heads;
  p.Hk = c.num_k_heads;
  p.d = c.d;
  p.rot = c.rot;
  p.interleaved = c.layout == LQ_ROPE_INTERLEAVED;
  p.bf16 = c.dtype == LQ_DTYPE_BF16;
  p.cos_mul = c.magnitude;
  p.sin_mul = c.inverse ? -c.magnitude : c.magnitude;
  p.q = q;
  p.k = k;
  p.q_out = q_out;
  p.k_out = k_out;
  p.positions = positions;
  p.table = table;
  return from_cuda(lq::launch_rotary(p, static_cast<cudaStream_t>(stream)));
}

lq_status lq_group_norm(const lq_norm_config *cfg, int32_t tokens, const void *x,
                        const void *gate, const float *weight, const float *bias, void *out,
                        void *stream) {
  if (cfg == nullptr || tokens < 0) return LQ_ERR_INVALID_ARG;
  const lq_norm_config &c = *cfg;
  if (c.groups < 1 || c.size < 1) return LQ_ERR_INVALID_ARG;
  if (c.kind != LQ_NORM_RMS && c.kind != LQ_NORM_MEAN) return LQ_ERR_INVALID_ARG;
  if (c.act < LQ_ACT_NONE || c.act > LQ_ACT_SIGMOID) return LQ_ERR_INVALID_ARG;
  if (!is_dtype(c.in_dtype) || !is_dtype(c.out_dtype)) return LQ_ERR_INVALID_ARG;
  if (!(c.eps >= 0.0f)) return LQ_ERR_INVALID_ARG;
  if (c.groups > 65535 || c.size > 8192) return LQ_ERR_UNSUPPORTED;
  if (static_cast<int64_t>(tokens) * c.groups > INT32_MAX) return LQ_ERR_UNSUPPORTED;
  lq::NormParams p{};
  const int64_t row = static_cast<int64_t>(c.groups) * c.size;
  if (!resolve_stride(c.x_stride, row, &p.x_stride) ||
      !resolve_stride(c.gate_stride, row, &p.gate_stride) ||
      !resolve_stride(c.out_stride, row, &p.out_stride))
    return LQ_ERR_INVALID_ARG;
  if (tokens == 0) return LQ_OK;
  if (x == nullptr || out == nullptr) return LQ_ERR_INVALID_ARG;
  if (gate == nullptr && c.gate_before) return LQ_ERR_INVALID_ARG;
  // in place, a row has to be read where it is written
  if ((out == x && (p.x_stride != p.out_stride || c.in_dtype != c.out_dtype)) ||
      (gate != nullptr && out == gate &&
       (p.gate_stride != p.out_stride || c.in_dtype != c.out_dtype)))
    return LQ_ERR_INVALID_ARG;
  if (!aligned(x, size_of(c.in_dtype)) || !aligned(gate, size_of(c.in_dtype)) ||
      !aligned(out, size_of(c.out_dtype)) || !aligned(weight, 4) || !aligned(bias, 4))
    return LQ_ERR_MISALIGNED;
  p.tokens = tokens;
  p.groups = c.groups;
  p.size = c.size;
  p.kind = c.kind;
  p.act = c.act;
  p.gate_before = c.gate_before != 0;
  p.shared_weight = c.shared_weight != 0;
  p.in_bf16 = c.in_dtype == LQ_DTYPE_BF16;
  p.out_bf16 = c.out_dtype == LQ_DTYPE_BF16;
  p.eps = c.eps;
  p.x = x;
  p.gate = gate;
  p.weight = weight;
  p.bias = bias;
  p.out = out;
  return from_cuda(lq::launch_group_norm(p, static_cast<cudaStream_t>(stream)));
}

lq_status lq_get_error_word(int32_t *err, void *stream) {
  lq_state st;
  std::memset(&st, 0, sizeof(st));
  st.err = err;
  return lq_get_last_error(&st, stream);
}

}  // extern "C"

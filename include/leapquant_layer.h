/*
 * leapquant_layer.h - C ABI of the operators around a linear-attention state
 * that libleapquant.so offers next to the int8 GDN / KDA decode path of
 * leapquant.h: linear attention with a decay for each head (prompt and
 * single-token forms), rotary positions, and group norm with an activation.
 *
 * Together they are what a decayed linear-attention layer computes between
 * its projections: rotary q and k, the recurrence, the normalised and gated
 * head outputs.  lq_group_norm equally takes the outputs of lq_decode_step,
 * lq_decode_tokens and lq_prefill.  All of it is inference: nothing here has
 * a gradient.
 *
 * Conventions (those of leapquant.h unless said otherwise):
 *  - Tensor arguments are device pointers of the current device; the library
 *    allocates nothing and keeps no global state; `stream` is a cudaStream_t
 *    (NULL = legacy default) and work is asynchronous on it.  Every call but
 *    lq_get_error_word, which waits, can be captured into a graph.
 *  - Argument errors are detected on the host before anything is launched:
 *    LQ_ERR_INVALID_ARG (null pointer, bad shape, stride or option),
 *    LQ_ERR_UNSUPPORTED (a size outside the stated range), LQ_ERR_MISALIGNED.
 *    A failed launch returns LQ_ERR_CUDA.
 *  - Device-side problems never trap: a kernel sets a bit in *err (int32,
 *    device, zeroed once by the caller), leaves out the sequence, and
 *    lq_get_error_word reports it.
 *  - Token-major: token t of a tensor with H heads of d values starts at
 *    t * stride; its heads lie back to back.  A stride counts elements from
 *    token to token; 0 means packed (H * d).  Strided inputs are slices of a
 *    fused projection's rows.
 *  - Rows behind the last sequence are neither read as tokens nor written.
 */
#ifndef LEAPQUANT_LAYER_H
#define LEAPQUANT_LAYER_H

#include "leapquant.h"

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------------
 * Linear attention with a decay for each head
 *
 *   S_t = a_t S_{t-1} + v_t k_t^T,   o_t = S_t q_t
 *
 * with one scalar decay a_t in [0, 1] per value head.  A state is
 * [dv][dk] fp32 (row = value channel), as lq_fp32_decode_step's; the pool S
 * is [num_slots][num_v_heads][dv][dk], 16-byte aligned.  Value head h reads
 * key / query head h / (num_v_heads / num_k_heads).  q is used as given.
 *
 * slots: nullable int32 [batch], the pool slot of each sequence (null: slot b
 * for sequence b).  A negative slot skips the sequence: its state and its
 * outputs stay as they are.  A slot >= num_slots, or one that an earlier
 * sequence of the call names already, is skipped too and sets
 * LQ_ERR_DEVICE_BOUNDS in the error word.
 * ---------------------------------------------------------------------- */

typedef enum {
  LQ_DECAY_TOKEN = 0, /* decay: fp32 [tokens][num_v_heads], one per token and head */
  LQ_DECAY_HEAD = 1   /* decay: fp32 [num_v_heads], fixed per head */
} lq_decay;

typedef struct {
  int32_t batch;       /* sequences, 0..65536.  Every block compares its slot with the earlier
                          ones: a step with slots (1 head, d = 32) takes 0.05 ms at 4,096
                          sequences, 1.2 ms at 65,536, a one-token prompt 0.09 and 11 */
  int32_t num_k_heads; /* key / query heads, 1..2048 */
  int32_t num_v_heads; /* value heads, a multiple of num_k_heads */
  int32_t dk;          /* key channels, one of 32, 64, 128 */
  int32_t dv;          /* value channels, one of 32, 64, 128 */
  int32_t decay;       /* lq_decay */
  int32_t in_dtype;    /* lq_dtype of q, k, v */
  int32_t out_dtype;   /* lq_dtype of out */
  int64_t q_stride, k_stride, v_stride; /* elements from token to token, 0 = packed */
} lq_linear_config;

/* One token for every sequence: token b is sequence b's.
 *  q, k [batch][Hk][dk], v [batch][Hv][dv] (16-byte aligned, strides whole
 *  16-byte units); decay as cfg says (tokens = batch); out [batch][Hv][dv]
 *  packed.  States are updated in place. */
lq_status lq_linear_decode_step(const lq_linear_config *cfg, const void *q, const void *k,
                                const void *v, const float *decay, float *S, int32_t num_slots,
                                const int32_t *slots, void *out, int32_t *err, void *stream);

/* Packed prompts of any lengths: sequence b owns tokens offsets[b] ..
 * offsets[b+1]-1 of `tokens` rows (offsets: int32 [batch+1], ascending, within
 * [0, tokens]; a sequence whose pair is not, and every one behind a pair that
 * descends, is left out and sets LQ_ERR_DEVICE_BOUNDS).  Runs the recurrence over each sequence from the
 * state in its slot, or from zeros where fresh[b] != 0 (fresh: nullable int32
 * [batch]), writes out [tokens][Hv][dv] (nullable: states only) and leaves the
 * last state in the slot.  An empty sequence leaves its state, or zeros if
 * fresh.  Arguments as for lq_linear_decode_step; decay per token is
 * [tokens][Hv].
 *  workspace: lq_linear_workspace_bytes(cfg, tokens) bytes, 16-byte aligned
 *  (nullable when that is 0).  That is enough for every call of no more tokens
 *  and no more sequences with cfg otherwise the same, so that a program can size
 *  one buffer for its largest call (78 MB at most up to 2^29 tokens, d = 128).
 *  Its contents matter during the call only; calls that may run at the same time,
 *  captured ones too, need one each.
 *  - bf16 prompts of more than 32 tokens a sequence on average (tokens > 32
 *    batch) are taken in chunks of 128 tokens whose products run on the tensor
 *    cores with fp32 accumulation; all others go token by token, which is slower
 *    for a long sequence: among 255 empty ones 7,900 tokens, 32 heads, take 1,154
 *    us and by themselves 155.  Such a sequence is better off in a call of its own.
 *  - In chunks, states and fp32 outputs are fp32 results (operands go in as exact
 *    sums of bf16 parts).  bf16 outputs see the state and the decayed scores to
 *    2^-16, well below their own rounding: 1.66e-3 against 64 bits (2-norm), as
 *    exact outputs have it.
 *  - In chunks, decays enter as products over ranges of tokens, never as
 *    quotients: a decay of 0 (a reset) and long chains of small ones give exact
 *    zeros.  An infinite or NaN v shows, as NaN, in its channel of its sequence's
 *    outputs from the start of its chunk on, where the recurrence has it from its
 *    token on; nothing else sees it.  Token by token it shows from its token on.
 *  - out may not overlap the inputs. */
size_t lq_linear_workspace_bytes(const lq_linear_config *cfg, int32_t tokens);
lq_status lq_linear_prefill(const lq_linear_config *cfg, const void *q, const void *k,
                            const void *v, const float *decay, int32_t tokens,
                            const int32_t *offsets, float *S, int32_t num_slots,
                            const int32_t *slots, const int32_t *fresh, void *out,
                            void *workspace, size_t workspace_bytes, int32_t *err, void *stream);

/* ------------------------------------------------------------------------
 * Rotary positions
 *
 * The first rot channels of a head are pairs (a, b); pair i of a token at
 * position p turns by p f_i:
 *   a' = m (a cos - b sin),   b' = m (b cos + a sin)
 * Half layout: pair i is channels (i, i + rot/2).  Interleaved: (2i, 2i + 1).
 * Channels from rot on are copied (left alone in place).
 * ---------------------------------------------------------------------- */

typedef enum { LQ_ROPE_HALF = 0, LQ_ROPE_INTERLEAVED = 1 } lq_rope_layout;

/* Scaling of the frequencies f_i = theta^(-2i/rot) for contexts `factor`
 * times the trained one. */
typedef enum {
  LQ_ROPE_NONE = 0,
  LQ_ROPE_LINEAR = 1, /* f_i / factor */
  LQ_ROPE_NTK = 2,    /* theta <- theta factor^(rot / (rot - 2)) */
  LQ_ROPE_PARTS = 3   /* by turns within the trained context: w_i f_i + (1 - w_i) f_i / factor,
                         w_i = clamp((trained f_i / 2 pi - slow) / (fast - slow), 0, 1);
                         magnitude m = 0.1 ln(factor) + 1 for factor > 1.  The ramp is linear in
                         turns.  Checkpoints whose code ramps over the pair's index i between two
                         bounds instead (often rounded to whole pairs) have other frequencies in
                         between: fill the table from those, entry by entry as lq_rotary_table
                         says */
} lq_rope_scaling;

typedef struct {
  int32_t num_q_heads;  /* >= 0 */
  int32_t num_k_heads;  /* >= 0: 0 = no k */
  int32_t d;            /* channels of a head, 2..1024 */
  int32_t rot;          /* rotated channels, even, 2..d */
  int32_t layout;       /* lq_rope_layout */
  int32_t dtype;        /* lq_dtype of q, k and the outputs */
  int32_t inverse;      /* nonzero: turn by -p f_i (undoes a rotation; m is applied as it is) */
  float magnitude;      /* m, the factor on cos and sin */
  int64_t q_stride, k_stride;         /* elements from token to token, 0 = packed */
  int64_t q_out_stride, k_out_stride;
} lq_rotary_config;

/* The table of a rotation, on the host: rot / 2 entries, entry i = f_i in
 * turns per position as a fraction of 2^64 (f_i / 2 pi 2^64, rounded; a
 * frequency is at most half a turn), and the magnitude m (nullable).  The
 * caller copies it to the device once.  A position's angle is its product with
 * the entry modulo 2^64, exact for every int32 position, so that far
 * positions lose nothing.  fast and slow: LQ_ROPE_PARTS only (fast > slow). */
lq_status lq_rotary_table(int32_t rot, double theta, int32_t scaling, double factor,
                          double trained, double fast, double slow, uint64_t *table,
                          float *magnitude);

/* Rotates q [tokens][Hq][d] and k [tokens][Hk][d] into q_out and k_out, which
 * may be q and k themselves (then with the same strides) but may not overlap
 * them otherwise.  positions: int32 [tokens].  table: device, 8-byte aligned.
 * k and k_out are ignored if num_k_heads is 0, q and q_out if num_q_heads is. */
lq_status lq_rotary(const lq_rotary_config *cfg, int32_t tokens, const void *q, const void *k,
                    const int32_t *positions, const uint64_t *table, void *q_out, void *k_out,
                    void *stream);

/* ------------------------------------------------------------------------
 * Group norm with an activation, channels last
 *
 * Each token's channels are `groups` groups of `size`; each group is
 * normalised by itself (for head outputs, a group is a head):
 *   n(x) = (x - mean) / sqrt(var + eps) w + b      LQ_NORM_MEAN
 *   n(x) = x / sqrt(mean(x^2) + eps) w + b         LQ_NORM_RMS
 *   y = act(n(x))            without a gate
 *   y = n(x) act(z)          with a gate z
 *   y = n(x act(z))          with a gate z and gate_before
 * Statistics are fp32 over the group's values held on chip, the variance from
 * the centred values (a group whose squares add up past fp32's range comes out
 * as zeros).  Rows move in pieces of 16 bytes where size, strides and addresses
 * are whole pieces, else value by value, at 2 to 20 times the time.
 * ---------------------------------------------------------------------- */

typedef enum { LQ_NORM_RMS = 0, LQ_NORM_MEAN = 1 } lq_norm_kind;
typedef enum { LQ_ACT_NONE = 0, LQ_ACT_SILU = 1, LQ_ACT_SIGMOID = 2 } lq_act;

typedef struct {
  int32_t groups;        /* 1..65535 */
  int32_t size;          /* channels of a group, 1..8192 */
  int32_t kind;          /* lq_norm_kind */
  int32_t act;           /* lq_act */
  int32_t gate_before;   /* nonzero: the gate multiplies x before the norm */
  int32_t shared_weight; /* nonzero: w is [size], shared by the groups; else [groups][size] */
  int32_t in_dtype;      /* lq_dtype of x and the gate */
  int32_t out_dtype;     /* lq_dtype of out */
  float eps;             /* >= 0 */
  int64_t x_stride, gate_stride, out_stride; /* elements from token to token, 0 = packed */
} lq_norm_config;

/* x [tokens][groups][size]; gate: nullable, as x; weight: nullable fp32;
 * bias: nullable fp32 [groups][size], also with a shared weight (a shared bias
 * is repeated there by the caller); out may be x or the gate itself (with the
 * same type and stride). */
lq_status lq_group_norm(const lq_norm_config *cfg, int32_t tokens, const void *x,
                        const void *gate, const float *weight, const float *bias, void *out,
                        void *stream);

/* Synchronize `stream`, read and clear *err: LQ_OK, LQ_ERR_DEVICE_BOUNDS (a
 * sequence was left out) or LQ_ERR_TIMEOUT (a kernel's bounded wait expired:
 * the outputs of the call are not to be used). */
lq_status lq_get_error_word(int32_t *err, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* LEAPQUANT_LAYER_H */

// Rotary positions on q and k.
//
// The angle of pair i at position p is p f_i.  With f_i held as a 64-bit
// fraction of a turn, the product modulo 2^64 is the angle modulo one turn,
// exact for every int32 position: no argument reduction and no 64-bit
// floating point, and the top 32 bits, read as signed, are the angle in
// [-1/2, 1/2) turns to 2^-32.
//
// Bound by the bytes of q and k.  A block computes the sines and cosines of
// its few tokens once (rot / 2 each) and applies them to all heads.

#include "lq_chunk.cuh"
#include "lq_layer.h"

namespace lq {
namespace {

constexpr int kNT = 128;
constexpr int kMaxTok = 8;  // tokens of a block

// A head is split into work items: `turned` ones (two chunks that pair up in
// the half layout, one chunk of pairs interleaved), then those that copy the
// channels behind rot (as many chunks an item, so that a warp's lanes all do
// the same).  A thread has kHeads heads in flight: 16,381 tokens x 64 heads x
// 128, bf16, half layout 88 us with two and 101 with four; interleaved, with
// half the loads a head, 98 and 89.
template <bool BF16, bool INTER, int VEC>
__global__ void __launch_bounds__(kNT, 8)
    rotary_kernel(const RotaryParams p, int tok, bool copy_q, bool copy_k) {
  constexpr bool kTwo = !INTER || VEC == 1;  // two chunks an item
  constexpr int kHeads = kTwo ? 2 : 4;
  constexpr int kPairs = kTwo ? VEC : VEC / 2;
  extern __shared__ float2 cs[];  // [tok][rot / 2] (cos, sin)
  const int half = p.rot / 2, heads = p.Hq + p.Hk;
  const int t0 = blockIdx.x * tok, nt = min(tok, p.tokens - t0);
  const int tid = threadIdx.y * blockDim.x + threadIdx.x;
  for (int i = tid; i < nt * half; i += blockDim.x * blockDim.y) {
    const int t = i / half;
    const uint64_t turn = p.table[i - t * half] *
                          static_cast<uint64_t>(static_cast<int64_t>(p.positions[t0 + t]));
    const float x = static_cast<float>(static_cast<int32_t>(turn >> 32)) * 0x1p-31f;  // half turns
    float s, c;
    sincospif(x, &s, &c);
    cs[i] = make_float2(c * p.cos_mul, s * p.sin_mul);
  }
  __syncthreads();
  const int turned = half / kPairs;
  const int copied = copy_q || copy_k ? (p.d - p.rot) / VEC : 0;
  const int items = turned + (kTwo ? (copied + 1) / 2 : copied);
  const int step = gridDim.y * blockDim.y;
  for (int t = 0; t < nt; ++t) {
    const float2 *row = cs + t * half;
    for (int h0 = blockIdx.y * blockDim.y + threadIdx.y; h0 < heads; h0 += kHeads * step) {
      for (int c = threadIdx.x; c < items; c += blockDim.x) {
        const bool turn = c < turned;
        const int k = c - turned;
        const int at = turn ? (INTER ? 2 * kPairs : VEC) * c : p.rot + (kTwo ? 2 : 1) * VEC * k;
        const int other = turn ? (INTER ? at + 1 : at + half) : at + VEC;
        const bool two = kTwo && (turn || 2 * k + 1 < copied);
        Raw<BF16, VEC> ra[kHeads], rb[kTwo ? kHeads : 1];
#pragma unroll
        for (int u = 0; u < kHeads; ++u) {
          const int hh = h0 + u * step;
          const bool is_q = hh < p.Hq;
          if (hh < heads) {
            const void *src = is_q ? p.q : p.k;
            const int64_t from = (t0 + t) * (is_q ? p.q_stride : p.k_stride) +
                                 (is_q ? hh : hh - p.Hq) * p.d;
            ra[u].load(src, from + at);
            if constexpr (kTwo) {
              if (two) rb[u].load(src, from + other);
            }
          }
        }
        float2 w[kPairs];
        if (turn) {
#pragma unroll
          for (int j = 0; j < kPairs; ++j) w[j] = row[c * kPairs + j];
        }
#pragma unroll
        for (int u = 0; u < kHeads; ++u) {
          const int hh = h0 + u * step;
          const bool is_q = hh < p.Hq;
          if (hh >= heads) break;
          void *dst = is_q ? p.q_out : p.k_out;
          const int64_t to = (t0 + t) * (is_q ? p.q_out_stride : p.k_out_stride) +
                             (is_q ? hh : hh - p.Hq) * p.d;
          Chunk<BF16, VEC> a, b;
          a.set(ra[u]);
          if constexpr (kTwo) b.set(rb[u]);
          if (turn) {
            if constexpr (kTwo) {
#pragma unroll
              for (int j = 0; j < VEC; ++j) {
                const float x = a.x[j], y = b.x[j];
                a.x[j] = x * w[j].x - y * w[j].y;
                b.x[j] = y * w[j].x + x * w[j].y;
              }
            } else {
#pragma unroll
              for (int j = 0; j < kPairs; ++j) {
                const float x = a.x[2 * j], y = a.x[2 * j + 1];
                a.x[2 * j] = x * w[j].x - y * w[j].y;
                a.x[2 * j + 1] = y * w[j].x + x * w[j].y;
              }
            }
          }
          if (turn || (is_q ? copy_q : copy_k)) {
            a.store(dst, to + at);
            if constexpr (kTwo) {
              if (two) b.store(dst, to + other);
            }
          }
        }
      }
    }
  }
}

template <bool BF16, bool INTER, int VEC>
cudaError_t rotary_t(const RotaryParams &p, cudaStream_t st) {
  const int half = p.rot / 2, heads = p.Hq + p.Hk;
  const int rest = (p.d - p.rot) / VEC;
  const int items = INTER && VEC > 1 ? p.rot / VEC + rest : half / VEC + (rest + 1) / 2;
  const int bx = items < kNT ? items : kNT;
  const dim3 block(bx, kNT / bx);
  // Several tokens share a block where that fills its threads with sines, but
  // only as long as the blocks still fill the GPU twice over; few tokens
  // instead split their heads over more blocks.
  int tok = 1;
  while (tok < kMaxTok && 2 * tok * half <= 2 * kNT && p.tokens / (2 * tok) >= 1184) tok *= 2;
  const int gx = (p.tokens - 1) / tok + 1;
  int gy = 1;
  while (gy * static_cast<int>(block.y) < heads && gx * gy < 296) gy *= 2;
  rotary_kernel<BF16, INTER, VEC><<<dim3(gx, gy), block, tok * half * sizeof(float2), st>>>(
      p, tok, p.q != p.q_out, p.k != p.k_out);
  return cudaGetLastError();
}

template <bool BF16, bool INTER>
cudaError_t rotary_v(const RotaryParams &p, cudaStream_t st) {
  constexpr int VEC = BF16 ? 8 : 4;
  bool wide = (INTER ? p.rot : p.rot / 2) % VEC == 0 && p.d % VEC == 0;
  const void *ptr[4] = {p.q, p.q_out, p.k, p.k_out};
  const int64_t stride[4] = {p.q_stride, p.q_out_stride, p.k_stride, p.k_out_stride};
  for (int i = 0; i < 4; ++i)
    if (i < 2 ? p.Hq > 0 : p.Hk > 0)
      wide = wide && reinterpret_cast<uintptr_t>(ptr[i]) % 16 == 0 && stride[i] % VEC == 0;
  return wide ? rotary_t<BF16, INTER, VEC>(p, st) : rotary_t<BF16, INTER, 1>(p, st);
}

}  // namespace

cudaError_t launch_rotary(const RotaryParams &p, cudaStream_t st) {
  if (p.bf16) return p.interleaved ? rotary_v<true, true>(p, st) : rotary_v<true, false>(p, st);
  return p.interleaved ? rotary_v<false, true>(p, st) : rotary_v<false, false>(p, st);
}

}  // namespace lq

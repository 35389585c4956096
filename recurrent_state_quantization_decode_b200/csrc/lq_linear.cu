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

// Packed prompts, token by token: the exact fp32 recurrence, any type and
// length.  The state rows stay in registers; inputs come in stages of kTok
// tokens, the next stage's copies under way while one is worked on; kGroup
// tokens' row sums are reduced together, since nothing waits for them.
//
// Bound by its instructions: 3 multiply-adds a state value and token, two
// values an instruction.  8 columns a lane and sums over 4 tokens at once leave
// 73 instructions a token of 8 rows at d = 64, where 4 columns and a sum for
// each token took 101: 8 x 512 tokens, 32 heads, d = 128, fp32, 328 us against
// 415 us.  What a single long sequence lacks is parallelism: such calls are cut
// into segments, whose own states a first launch computes (without outputs) and
// the second one starts from (5 prompts of 3,001 tokens, 8 heads, d = 64: 41 us,
// 17 of them the states).
constexpr int kTok = 16, kGroup = 4;

template <int DK, bool BF16>
struct TokensSmem {
  static constexpr int E = BF16 ? 2 : 4;  // bytes of a value
  alignas(16) uint8_t q[2][kTok][DK * E];
  alignas(16) uint8_t k[2][kTok][DK * E];
  alignas(16) uint8_t v[2][kTok][kRows * E];
  float a[2][kTok];
  int scratch[kPlaceInts<kNT>];
};

// A warp's 8 state rows in the kernel for prompts: W columns a lane in pieces
// of 4, LPR lanes a row, NP consecutive rows a lane.  kGroup tokens' sums are as
// many values as a row has lanes: summed by halving, one stays in each.  (With 8
// columns of 32 a lane would have one row, and load more than it computes.)
template <int DK, bool BF16>
struct TokensMap {
  static constexpr int W = DK == 32 ? 4 : 8, LPR = DK / W, NP = LPR / 4;
  static_assert(kGroup * NP == LPR, "a sum for each lane");
  static __device__ __forceinline__ int row(int lane) { return lane / LPR * NP; }
  // a lane's 16-byte pieces of an input row: next to each other in bf16 (one
  // load), and in fp32 where a quarter warp's loads meet different banks
  static __device__ __forceinline__ int col(int lane, int piece) {
    const int c = lane % LPR;
    return BF16 ? c * W + piece * 4 : (piece * LPR + c) * 4;
  }
  static __device__ __forceinline__ void load(const void *row, int lane, float2 (&x)[W / 2]) {
    if constexpr (W == 4) {
      const float4 v = load_four<BF16>(row, col(lane, 0));
      x[0] = make_float2(v.x, v.y), x[1] = make_float2(v.z, v.w);
    } else if constexpr (BF16) {
      const char *at = static_cast<const char *>(row) + lane % LPR * 16;
      const uint4 v = *reinterpret_cast<const uint4 *>(at);
      const uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i)
        x[i] = make_float2(__uint_as_float(u[i] << 16), __uint_as_float(u[i] & 0xffff0000u));
    } else {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const float4 v = load_four<false>(row, col(lane, i));
        x[2 * i] = make_float2(v.x, v.y), x[2 * i + 1] = make_float2(v.z, v.w);
      }
    }
  }
  // x[lane % LPR], summed over the row's lanes
  static __device__ __forceinline__ float reduce(float (&x)[LPR], int lane) {
#pragma unroll
    for (int off = LPR / 2; off >= 1; off >>= 1) {
      const bool upper = (lane & off) != 0;
#pragma unroll
      for (int i = 0; i < LPR / 2; ++i) {
        if (i >= off) break;
        const float send = upper ? x[i] : x[i + off];
        const float keep = upper ? x[i + off] : x[i];
        x[i] = keep + __shfl_xor_sync(kAllLanes, send, off);
      }
    }
    return x[0];
  }
};

__device__ __forceinline__ void copy16(void *dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                   static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
               "l"(src)
               : "memory");
}
__device__ __forceinline__ void copy4(void *dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(
                   static_cast<uint32_t>(__cvta_generic_to_shared(dst))),
               "l"(src)
               : "memory");
}

template <int DK, bool BF16, bool OUT>
__global__ void __launch_bounds__(kNT) linear_tokens_kernel(const LinParams p, const Segments sg) {
  using M = TokensMap<DK, BF16>;
  constexpr int E = BF16 ? 2 : 4;
  __shared__ TokensSmem<DK, BF16> sm;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int blocks = p.dv / kRows;
  const int tile = blockIdx.x / blocks, block0 = blockIdx.x % blocks * kRows;
  const int row0 = warp * 8;
  const int h = tile % p.Hv, hk = h / (p.Hv / p.Hk);
  Work pl;
  if (!locate<kNT, false>(p, sg, tile / p.Hv, !sg.partial && h == 0 && block0 == 0, sm.scratch, pl)) return;
  const int slot = pl.slot;
  const bool last = pl.index == pl.count - 1, fresh = pl.fresh;
  if (!OUT && !sg.partial && !last) return;  // no outputs asked for: the last state alone
  const int64_t begin = pl.first + pl.index * sg.tokens;
  const int rest = pl.length - pl.index * sg.tokens;
  const int count = pl.count > 1 ? min(sg.tokens, rest) : rest;
  if (count == 0 && !fresh) return;

  const int stages = (count + kTok - 1) / kTok;
  auto fetch = [&](int st) {
    const int n = min(kTok, count - st * kTok), b = st & 1;
    const int64_t first = begin + st * kTok;
    constexpr int kU = DK * E / 16, vU = kRows * E / 16;  // 16-byte units of a row
    const char *q = static_cast<const char *>(p.q), *k = static_cast<const char *>(p.k);
    const char *v = static_cast<const char *>(p.v);
    for (int i = tid; i < n * kU; i += kNT) {
      const int t = i / kU, u = i % kU * 16;
      copy16(&sm.q[b][t][u], q + ((first + t) * p.q_stride + hk * DK) * E + u);
      copy16(&sm.k[b][t][u], k + ((first + t) * p.k_stride + hk * DK) * E + u);
    }
    for (int i = tid; i < n * vU; i += kNT) {
      const int t = i / vU, u = i % vU * 16;
      copy16(&sm.v[b][t][u], v + ((first + t) * p.v_stride + h * p.dv + block0) * E + u);
    }
    if (tid < n) copy4(&sm.a[b][tid], p.decay + (p.decay_head ? h : (first + tid) * p.Hv + h));
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  if (sg.partial) let_next_start();
  if (stages > 0) fetch(0);

  const int64_t tile_size = static_cast<int64_t>(p.dv) * DK;
  const int64_t at = static_cast<int64_t>(block0 + row0 + M::row(lane)) * DK;
  float *S = p.S + (static_cast<int64_t>(slot) * p.Hv + h) * tile_size + at;
  float *entry = sg.states + (static_cast<int64_t>(pl.entry) * p.Hv + h) * tile_size + at;
  const int64_t entry_step = static_cast<int64_t>(p.Hv) * tile_size;
  float2 s[M::NP][M::W / 2];
  auto load = [&](const float *src) {
#pragma unroll
    for (int i = 0; i < M::NP; ++i)
#pragma unroll
      for (int c = 0; c < M::W / 4; ++c) {
        const float4 x = *reinterpret_cast<const float4 *>(src + i * DK + M::col(lane, c));
        s[i][2 * c] = make_float2(x.x, x.y), s[i][2 * c + 1] = make_float2(x.z, x.w);
      }
  };
  auto store = [&](float *dst) {
#pragma unroll
    for (int i = 0; i < M::NP; ++i)
#pragma unroll
      for (int c = 0; c < M::W / 4; ++c)
        *reinterpret_cast<float4 *>(dst + i * DK + M::col(lane, c)) =
            make_float4(s[i][2 * c].x, s[i][2 * c].y, s[i][2 * c + 1].x, s[i][2 * c + 1].y);
  };
  wait_for_states();
  if (!fresh && sg.partial && pl.index == 0) {
    // a split sequence's first state moves to the workspace: the last
    // segment's blocks write the pool while others still need it
    load(S);
    store(entry);
  }
  if (fresh || sg.partial) {
#pragma unroll
    for (int i = 0; i < M::NP; ++i)
#pragma unroll
      for (int c = 0; c < M::W / 2; ++c) s[i][c] = make_float2(0.0f, 0.0f);
  } else {
    load(pl.count > 1 ? entry : S);
  }
  if (!sg.partial) {
#pragma unroll 1
    for (int r = 0; r < pl.index; ++r) {
      const float d = sg.decays[static_cast<int64_t>(pl.entry + 1 + r) * p.Hv + h];
      const float *src = entry + (r + 1) * entry_step;
      const float2 dd = make_float2(d, d);
#pragma unroll
      for (int i = 0; i < M::NP; ++i)
#pragma unroll
        for (int c = 0; c < M::W / 4; ++c) {
          const float4 x = *reinterpret_cast<const float4 *>(src + i * DK + M::col(lane, c));
          s[i][2 * c] = __ffma2_rn(s[i][2 * c], dd, make_float2(x.x, x.y));
          s[i][2 * c + 1] = __ffma2_rn(s[i][2 * c + 1], dd, make_float2(x.z, x.w));
        }
    }
  }

  double total = 1.0;  // the segment's whole decay
  // the lane's output of a group: token mine / NP, row mine % NP of its rows
  const int mine = lane % M::LPR;
  int64_t to = ((begin + mine / M::NP) * p.Hv + h) * p.dv + block0 + row0 + M::row(lane) +
               mine % M::NP;
  const int64_t to_step = static_cast<int64_t>(kGroup) * p.Hv * p.dv;
#pragma unroll 1
  for (int st = 0; st < stages; ++st) {
    const int n = min(kTok, count - st * kTok), b = st & 1;
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();  // the stage is in; the other one is free
    if (st + 1 < stages) fetch(st + 1);
    if (sg.partial && warp == 0) {
      double x = lane < n ? sm.a[b][lane] : 1.0;
#pragma unroll
      for (int o = kTok / 2; o > 0; o >>= 1) x *= __shfl_xor_sync(kAllLanes, x, o);
      total *= x;
    }
#pragma unroll 1
    for (int t0 = 0; t0 < n; t0 += kGroup) {
      float o[M::LPR];
#pragma unroll
      for (int g = 0; g < kGroup; ++g) {
        const int t = t0 + g;
        if (t < n) {
          float2 k[M::W / 2], q[M::W / 2];
          M::load(sm.k[b][t], lane, k);
          if (OUT) M::load(sm.q[b][t], lane, q);
          const float2 a = make_float2(sm.a[b][t], sm.a[b][t]);
          float v[M::NP];
          load_rows<BF16, M::NP>(sm.v[b][t], row0 + M::row(lane), v);
#pragma unroll
          for (int i = 0; i < M::NP; ++i) {
            const float2 vv = make_float2(v[i], v[i]);
            float2 x;
#pragma unroll
            for (int c = 0; c < M::W / 2; ++c) {
              s[i][c] = __ffma2_rn(a, s[i][c], __fmul2_rn(vv, k[c]));
              if (OUT) x = c == 0 ? __fmul2_rn(s[i][c], q[c]) : __ffma2_rn(s[i][c], q[c], x);
            }
            if (OUT) o[g * M::NP + i] = x.x + x.y;
          }
        } else {
#pragma unroll
          for (int i = 0; i < M::NP; ++i) o[g * M::NP + i] = 0.0f;
        }
      }
      if constexpr (OUT) {
        const float sum = M::reduce(o, lane);
        if (t0 + mine / M::NP < n) store_value(p.out, to, sum, p.out_bf16);
        to += to_step;
      }
    }
  }
  if (sg.partial) {
    store(entry + (pl.index + 1) * entry_step);
    if (tid == 0 && block0 == 0)
      sg.decays[static_cast<int64_t>(pl.entry + 1 + pl.index) * p.Hv + h] =
          static_cast<float>(total);
  } else if (last) {
    store(S);
  }
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

constexpr int64_t kBlocks = 148 * 5;

// Tokens of a segment: so many that the segments' blocks fill the GPU about
// once (5 of them an SM), but a launch's worth at least.
int tokens_segment(const LinParams &p) {
  constexpr int64_t kLeast = 64;
  const int64_t each = static_cast<int64_t>(p.tokens) * p.Hv * (p.dv / kRows) / kBlocks;
  const int64_t n = (each + kTok - 1) / kTok * kTok;
  return static_cast<int>(n < kLeast ? kLeast : n);
}

template <int DK, bool BF16>
cudaError_t tokens_t(const LinParams &p, Segments sg, cudaStream_t st) {
  const int64_t split = split_segments(p, sg.tokens), each = static_cast<int64_t>(p.Hv) * (p.dv / kRows);
  if ((split + p.B) * each > INT32_MAX) return cudaErrorInvalidConfiguration;
  if (split > 0) {
    sg.partial = true;
    linear_tokens_kernel<DK, BF16, false>
        <<<static_cast<unsigned>(split * each), kNT, 0, st>>>(p, sg);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    sg.partial = false;
  }
  auto kernel = p.out != nullptr ? linear_tokens_kernel<DK, BF16, true>
                                 : linear_tokens_kernel<DK, BF16, false>;
  return launch_next(kernel, (split + p.B) * each, kNT, 0, split > 0, st, p, sg);
}

template <int DK>
cudaError_t tokens_d(const LinParams &p, const Segments &sg, cudaStream_t st) {
  return p.in_bf16 ? tokens_t<DK, true>(p, sg, st) : tokens_t<DK, false>(p, sg, st);
}

}  // namespace

cudaError_t launch_linear_step(const LinParams &p, cudaStream_t st) {
  if (p.dk == 32) return step_d<32>(p, st);
  if (p.dk == 64) return step_d<64>(p, st);
  return step_d<128>(p, st);
}

size_t linear_tokens_workspace(const LinParams &p) {
  return segments_workspace(p, split_segments(p, tokens_segment(p)));
}

// tokens_segment is 64 at least and more than x - 1 for x = tokens * blocks a
// token / kBlocks, so that a call of x >= 64 has fewer than kBlocks / blocks *
// 64 / 63 segments and any has at most tokens / 64.
size_t linear_tokens_workspace_most(const LinParams &p) {
  const int64_t some = p.tokens / 64;
  const int64_t most = kBlocks * 64 / (63 * static_cast<int64_t>(p.Hv) * (p.dv / kRows));
  return segments_workspace(p, some < most ? some : most);
}

cudaError_t launch_linear_tokens(const LinParams &p, void *workspace, cudaStream_t st) {
  const int segment = tokens_segment(p);
  const Segments sg = segments_in(p, segment, segment, workspace);
  if (p.dk == 32) return tokens_d<32>(p, sg, st);
  if (p.dk == 64) return tokens_d<64>(p, sg, st);
  return tokens_d<128>(p, sg, st);
}

}  // namespace lq

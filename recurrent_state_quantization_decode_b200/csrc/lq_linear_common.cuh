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

// N consecutive values (aligned to their size together, 16 bytes at most).
template <bool BF16, int N>
__device__ __forceinline__ void load_rows(const void *p, int i, float (&x)[N]) {
  if constexpr (N >= 4) {
#pragma unroll
    for (int j = 0; j < N; j += 4) {
      const float4 v = load_four<BF16>(p, i + j);
      x[j] = v.x, x[j + 1] = v.y, x[j + 2] = v.z, x[j + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) x[j] = load_value<BF16>(p, i + j);
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

struct Segments {
  int tokens;      // tokens of a segment
  int whole;       // a sequence of no more tokens than this is not cut
  bool partial;    // segments before a sequence's last: their own state, into the workspace
  float *states;   // workspace: per split sequence its first state, then each segment's state
  float *decays;   // workspace: [entry][Hv] the segments' whole decays

  __device__ __forceinline__ int pieces(int length) const {
    return length <= whole ? 1 : (length - 1) / tokens + 1;
  }
};

// Where sequences longer than a segment stay whole, blocks are numbered through
// the long sequences first: one that starts late adds its whole time to the
// call's.  Pass 0 takes those whole ones, 1 the cut ones and all of more than
// half a segment, 2 the rest.  24 prompts of 20,011 tokens, 32 heads, the longest
// 1.4 segments: in the call's order 268 us with it first and 417 us with it last,
// in passes 259 to 276 us in seven orders.
//
// A sequence's blocks count in its pass's 10 bits of a sum.  There are fewer than
// 1,024: with several sequences a segment is an SM's share of the call at least,
// so 148 cover it, cut or longer than half of one there are not more than twice
// that, and at most kRankedMost sequences are ranked.
constexpr int kRankedMost = 768;
struct Rank {
  int shift;
  __device__ __forceinline__ Rank(const Segments &sg, int length) {
    shift = length <= sg.tokens / 2 ? 20 : length <= sg.tokens || length > sg.whole ? 10 : 0;
  }
  // the blocks up to the sequence's last among those of its pass, and all of earlier passes
  __device__ __forceinline__ int upto(unsigned prefix, unsigned all) const {
    const int before = (shift > 0 ? all & 1023 : 0) + (shift > 10 ? all >> 10 & 1023 : 0);
    return before + static_cast<int>(prefix >> shift & 1023);
  }
};

// Where a block works.
struct Place {
  int b, index, count;  // sequence, its segment, its segments
  int entry;            // the sequence's first workspace entry
  int length;           // its tokens, -1 if it is left out
};

// From the first pair of offsets that descends, sequences could overlap and so
// need more workspace than the call has: that one and all behind it are left
// out, as one segment each.  Then the others' tokens are disjoint, and
// ceil(n / tokens) <= 2 n / tokens for n >= tokens keeps to the workspace.
constexpr int kNoDescent = 0x7fffffff;
template <int NT>
constexpr int kPlaceInts = 2 * (NT / 32) + 6;

// Segments are numbered through the sequences.  Whole block of NT threads;
// `scratch` is kPlaceInts<NT> ints of shared memory.  Returns false if there
// are fewer than `wanted` + 1.
template <int NT, bool RANKED>
__device__ __forceinline__ bool find_place(const LinParams &p, const Segments &sg, int wanted,
                                           int *scratch, Place &pl) {
  static_assert(!RANKED || NT >= kRankedMost, "ranked sequences are looked at together");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const bool ranked = RANKED && sg.whole > sg.tokens;
  int done = 0, entries = 0;
  int *found = scratch + 2 * (NT / 32);
  if (threadIdx.x == 0) found[0] = -1, found[5] = kNoDescent;
  __syncthreads();
  for (int b0 = 0; b0 < p.B; b0 += NT) {
    const int b = b0 + threadIdx.x;
    int segs = 0, cnt = 0, ent = 0;
    if (b < p.B && p.offsets[b + 1] < p.offsets[b]) atomicMin(&found[5], b);
    __syncthreads();
    const int length = b < p.B && b < found[5] ? sequence_span(p, b).count : -1;
    if (b < p.B) {
      segs = sg.pieces(length);
      cnt = sg.partial ? segs - 1 : segs;
      ent = segs > 1 ? segs : 0;
    }
    const Rank rank(sg, length);
    int c = ranked ? cnt << rank.shift : cnt, e = ent;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int c2 = __shfl_up_sync(kAllLanes, c, o), e2 = __shfl_up_sync(kAllLanes, e, o);
      if (lane >= o) c += c2, e += e2;
    }
    __syncthreads();
    if (lane == 31) scratch[warp] = c, scratch[(NT / 32) + warp] = e;
    __syncthreads();
    int before = done, ebefore = entries;
#pragma unroll
    for (int w = 0; w < (NT / 32); ++w) {
      if (w < warp) before += scratch[w], ebefore += scratch[(NT / 32) + w];
      done += scratch[w], entries += scratch[(NT / 32) + w];
    }
    const int first = (ranked ? rank.upto(before + c, done) : before + c) - cnt;
    if (wanted >= first && wanted < first + cnt) {
      found[0] = b;
      found[1] = wanted - first;
      found[2] = segs;
      found[3] = ebefore + e - ent;
      found[4] = length;
    }
    if (ranked || wanted < done) break;
  }
  __syncthreads();
  pl = {found[0], found[1], found[2], found[3], found[4]};
  return pl.b >= 0;
}

// What a block works on: a segment of a sequence.
struct Work {
  int b, index, count, entry;  // as in Place
  int slot;
  int first, length;  // of the sequence's tokens
  bool fresh;
};

// Segment `wanted` in the call's order, checked: false if there is none, or if
// its sequence is left out (no slot, a slot past the pool or an earlier
// sequence's, offsets that do not ascend).  With `reports`, a fault goes into
// the error word.  Up to 128 sequences every warp reads them all at once and
// keeps them in registers, one round trip to L2 in place of four.
template <int NT, bool RANKED>
__device__ __forceinline__ bool locate(const LinParams &p, const Segments &sg, int wanted,
                                       bool reports, int *scratch, Work &w) {
  const int lane = threadIdx.x & 31;
  bool fault = false, taken = false;
  if (p.B <= 128) {
    int lo[4], hi[4], slots[4], fresh[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int b = j * 32 + lane;
      lo[j] = hi[j] = fresh[j] = 0, slots[j] = -1;
      if (b < p.B) {
        lo[j] = p.offsets[b], hi[j] = p.offsets[b + 1];
        slots[j] = p.slots != nullptr ? p.slots[b] : b;
        if (p.fresh != nullptr) fresh[j] = p.fresh[b] != 0;
      }
    }
    int segs[4], c[4], e[4];  // segments; blocks through the sequence's last; entries before it
    int all = 0, entries = 0, descent = kNoDescent;
    const bool ranked = RANKED && sg.whole > sg.tokens;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      segs[j] = c[j] = e[j] = 0;
      if (j * 32 >= p.B) continue;
      const unsigned descends = __ballot_sync(kAllLanes, hi[j] < lo[j]);
      if (descends != 0 && descent == kNoDescent) descent = j * 32 + __ffs(descends) - 1;
      const bool bad = j * 32 + lane >= descent || lo[j] < 0 || hi[j] > p.tokens;
      hi[j] = bad ? -1 : hi[j] - lo[j];  // the length from here on
      if (j * 32 + lane < p.B) segs[j] = sg.pieces(hi[j]);
      const int cnt = sg.partial && segs[j] > 0 ? segs[j] - 1 : segs[j];
      const int ent = segs[j] > 1 ? segs[j] : 0;
      c[j] = ranked ? cnt << Rank(sg, hi[j]).shift : cnt, e[j] = ent;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int c2 = __shfl_up_sync(kAllLanes, c[j], o), e2 = __shfl_up_sync(kAllLanes, e[j], o);
        if (lane >= o) c[j] += c2, e[j] += e2;
      }
      const int more = __shfl_sync(kAllLanes, c[j], 31), more_e = __shfl_sync(kAllLanes, e[j], 31);
      c[j] += all, e[j] += entries - ent;
      all += more, entries += more_e;
    }
    unsigned hit = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (hit != 0 || j * 32 >= p.B) continue;
      const int cnt = sg.partial && segs[j] > 0 ? segs[j] - 1 : segs[j];
      const int first = (ranked ? Rank(sg, hi[j]).upto(c[j], all) : c[j]) - cnt;
      hit = __ballot_sync(kAllLanes, wanted >= first && wanted < first + cnt);
      if (hit != 0) {
        const int from = __ffs(hit) - 1;
        w.b = j * 32 + from;
        w.index = wanted - __shfl_sync(kAllLanes, first, from);
        w.count = __shfl_sync(kAllLanes, segs[j], from);
        w.entry = __shfl_sync(kAllLanes, e[j], from);
        w.slot = __shfl_sync(kAllLanes, slots[j], from);
        w.first = __shfl_sync(kAllLanes, lo[j], from);
        w.length = __shfl_sync(kAllLanes, hi[j], from);
        w.fresh = __shfl_sync(kAllLanes, fresh[j], from) != 0;
      }
    }
    if (hit == 0) return false;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      taken = taken || __any_sync(kAllLanes, j * 32 + lane < w.b && slots[j] == w.slot);
    taken = taken && p.slots != nullptr;
    if (w.slot < 0) return false;
    fault = w.slot >= p.num_slots || taken || w.length < 0;
  } else {
    Place pl;
    if (!find_place<NT, RANKED>(p, sg, wanted, scratch, pl)) return false;
    w.b = pl.b, w.index = pl.index, w.count = pl.count, w.entry = pl.entry;
    w.slot = p.slots != nullptr ? p.slots[w.b] : w.b;
    w.first = p.offsets[w.b], w.length = pl.length;
    w.fresh = p.fresh != nullptr && p.fresh[w.b] != 0;
    if (w.slot < 0) return false;
    int same = 0;
    if (p.slots != nullptr)
      for (int i = threadIdx.x; i < w.b; i += NT) same |= p.slots[i] == w.slot;
    taken = __syncthreads_or(same) != 0;
    fault = w.slot >= p.num_slots || taken || w.length < 0;
  }
  if (fault && reports && w.index == 0 && threadIdx.x == 0) atomicOr(p.err, kErrBadPhase);
  return !fault;
}

// The second launch of a call in segments may start while the first one's last
// blocks run (its blocks then find their places, fetch their first tokens and
// wait here before they touch a state): 8,192 tokens, 8 heads, d = 128, 91 -> 88
// us.  No effect in a launch of its own.
__device__ __forceinline__ void wait_for_states() {
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
__device__ __forceinline__ void let_next_start() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
template <class... Params, class... Args>
cudaError_t launch_next(void (*kernel)(Params...), int64_t grid, int threads, int smem, bool overlaps,
                        cudaStream_t st, const Args &...args) {
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = overlaps ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// At most how many segments come before a sequence's last one.
inline int64_t split_segments(const LinParams &p, int segment) {
  return p.tokens > segment ? p.tokens / segment : 0;
}

// Workspace of a call with so many segments before a last one: a sequence of
// s > 1 of them needs s entries, a state and a decay each for every value head.
inline size_t segments_workspace(const LinParams &p, int64_t split) {
  return static_cast<size_t>(2 * split * p.Hv * (static_cast<int64_t>(p.dk) * p.dv + 1) * 4);
}
inline Segments segments_in(const LinParams &p, int segment, int whole, void *workspace) {
  float *states = static_cast<float *>(workspace);
  return {segment, whole, false, states,
          states + 2 * split_segments(p, segment) * p.Hv * p.dk * p.dv};
}

// A warp's share of state rows: 8 rows of DK columns, 4 columns a lane, LPR
// lanes a row, NP consecutive rows a lane.  Sums over a row leave that of row
// (lane % LPR) / 4 of its rows in every lane.
template <int DK>
struct RowMap {
  static constexpr int LPR = DK / 4;
  static constexpr int NP = LPR / 4;
  static __device__ __forceinline__ int col(int lane) { return lane % LPR * 4; }
  static __device__ __forceinline__ int row(int lane, int i) { return lane / LPR * NP + i; }
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

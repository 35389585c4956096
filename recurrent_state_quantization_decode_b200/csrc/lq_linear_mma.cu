// Prompts of the decayed linear attention on the tensor cores: bf16 inputs,
// chunks of 128 tokens.
//
// Within a chunk write G_i = a_1 ... a_i, W_ij = a_{j+1} ... a_i (j <= i) and
// w_j = a_{j+1} ... a_128.  With S the state before the chunk,
//   P  = Q K^T,   O_i = sum_{j <= i} W_ij P_ij V_j + G_i (Q S^T)_i,
//   S' = G_128 S + (w V)^T K.
// Decays enter as products over ranges of tokens, never as quotients: a decay
// of zero and chains that underflow give exact zeros.
//
// One block walks over the chunks of one (sequence, value head), or of one
// segment of it, with everything between the tiles' loads and the outputs'
// stores on chip:
//   warps 0-7    the state, fp32 in registers (one value channel a lane): S'
//                from the increment, and its bf16 copy for Q S^T; by token,
//                G (Q S^T) in place, to which the product with V is added, and
//                the outputs
//   warps 8-15   by token: W o P back into tensor memory as the left operand of
//                the product with V
//   warps 16-19  (w V)^T, 32 tokens at a time, into tensor memory as the left
//                operand of the increment
//   warp 20      issues the products for the outputs
//   warp 21      loads Q, K, V tiles of the next chunks (bulk copies, 2 stages)
//   warp 22      issues the products for the increment
//   warp 23      products of decays; stores the outputs of a chunk (bf16; fp32
//                ones leave from registers, 32 bytes a lane)
// The operands that decays scale go through tensor memory and not through
// shared memory: written and read there, the three parts of w V alone cost 288
// KB a chunk of its bandwidth (128 bytes a cycle), half of all that the
// products read.
//
// Roundings.  P, O and the increment are fp32 sums of exact bf16 products.  w V
// is split into three bf16 parts, which hold all of its fp32 bits, so that the
// state is an fp32 result; S' = G S + increment is rounded once or twice in
// fp32 (G as a sum of two floats: an error in G would be the same in every
// chunk and add up).  W o P and S meet bf16 operands in the products for O.
// With fp32 outputs they go in as three exact parts, with bf16 outputs as two, to
// 2^-16, which leaves the rounding of O itself: 1.66e-3 against 64 bits on 24
// prompts and on 32,768 tokens, where S as one part (2^-8) gave 1.72e-3 and
// 2.0e-3, and more where q sees only a small difference of a large state.  The
// second part of S costs 9 % (24 prompts of 20,011 tokens, 32 heads, 260 -> 285
// us; 32,768 tokens 507 -> 554); a third one of W o P, which leaves the error as
// it is, would take 298 and 594.

#include <atomic>
#include <cstddef>
#include <type_traits>

#include "lq_linear_common.cuh"
#include "lq_tensor.cuh"

namespace lq {
namespace {

constexpr int kC = 128;        // tokens of a chunk
constexpr int kNT = 768;
constexpr uint32_t kPolls = 1u << 11;  // of 64 polls of at most 20 us each: a wait ends within 3 s

struct Decays {
  float a[kC];     // the tokens' decays, 1 behind the last token
  float rest[kC];  // a_{j+1} ... to the end of j's block of 32 tokens
};
// The block's barriers; those up to kStaged come in pairs, one a stage or slot.
// A single one's next phase needs what follows the wait for the last; outputs
// can be staged before the warp that stores them has seen the chunk before.
enum Barrier : uint32_t {
  kFullK = 0, kFullV = 2, kFullQ = 4, kEmptyQ = 6, kEmptyK = 8, kEmptyV = 10, kDecFull = 12,
  kDecEmpty = 14, kRingFull = 16, kRingEmpty = 18, kStaged = 20,
  kPFull = 22, kPDone, kSReady, kQSPart, kQSDone, kOScaled, kOFull, kOEmpty, kSFull, kGrownRead,
  kStored, kTail,
  kBarriers
};
struct Control {
  Decays dec[2];
  alignas(16) float block[2][4];  // products over the blocks of 32 tokens
  float whole[2][2];  // product over the chunk, as a sum of two floats
  uint64_t bar[kBarriers];
  uint32_t tmem;
  int dead;
};

template <int DKP, int DVP>
struct Tiles {
  static constexpr int kQ = kC * DKP * 2, kV = kC * DVP * 2, kS = DKP * DVP * 2;
  static constexpr int kStage = 2 * kQ + kV;
  // The outputs on their way to memory take the chunk's Q tile, which is not
  // needed any more, at 128 x 128, and a place of their own where there is one.
  static constexpr bool kOverQ = DKP == 128 && DVP == 128;
  static constexpr int kState = 2 * kStage, kOut = kState + kS;
  static constexpr int kControl = kOut + (kOverQ ? 0 : kV);
  static constexpr int kBytes = kControl + static_cast<int>(sizeof(Control));
  static_assert(kBytes <= 232448, "shared memory of a block");
};

__device__ __forceinline__ uint32_t bits(float x) { return __float_as_uint(x); }
__device__ __forceinline__ float2 floats(uint32_t x, uint32_t y) {
  return make_float2(__uint_as_float(x), __uint_as_float(y));
}
// Two floats rounded to bf16, the first in the low half; and back.
__device__ __forceinline__ uint32_t pack(float2 x) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(x.x, x.y);
  return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ float2 unpack(uint32_t v) { return floats(v << 16, v & 0xffff0000u); }
// x - v, exactly where v is x rounded.
__device__ __forceinline__ float2 remainder(float2 x, uint32_t v) {
  return __ffma2_rn(unpack(v), make_float2(-1.0f, -1.0f), x);
}
// Part 0, 1 or 2 of the split of fp32 into bf16: what the parts before leave,
// rounded.  Three parts hold 24 bits.
template <int PART>
__device__ __forceinline__ uint32_t part_of(float2 x) {
#pragma unroll
  for (int i = 0; i < PART; ++i) x = remainder(x, pack(x));
  return pack(x);
}
__device__ __forceinline__ void scale2(uint32_t &x, uint32_t &y, float2 f) {
  const float2 z = __fmul2_rn(floats(x, y), f);
  x = bits(z.x), y = bits(z.y);
}

__device__ __forceinline__ void store_shared16(uint32_t addr, uint32_t a, uint32_t b, uint32_t c,
                                               uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(a), "r"(b), "r"(c),
               "r"(d)
               : "memory");
}
// v[at ..] to 32 aligned bytes.
__device__ __forceinline__ void store_global32(void *p, const uint32_t (&v)[16], int at) {
  asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(v[at]),
               "r"(v[at + 1]), "r"(v[at + 2]), "r"(v[at + 3]), "r"(v[at + 4]), "r"(v[at + 5]),
               "r"(v[at + 6]), "r"(v[at + 7])
               : "memory");
}

// Bounded wait of one thread.  A wait that runs out marks the block and the
// error word; the other warps see the mark in their own waits.
__device__ __forceinline__ bool wait_one(uint32_t bar, uint32_t parity, volatile int *dead,
                                         int32_t *err) {
#pragma unroll 1
  for (uint32_t i = 0; i < kPolls; ++i) {
    if (tc::bar_try(bar, parity)) return true;
    if (*dead != 0) return false;
  }
  *dead = 1;
  atomicOr(err, kErrTimeout);
  return false;
}
// The same for a warp, all of whose lanes go on or give up together.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, volatile int *dead,
                                          int32_t *err) {
  return __all_sync(kAllLanes, wait_one(bar, parity, dead, err)) != 0;
}
__device__ __forceinline__ void arrive_warp(uint32_t bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) tc::bar_arrive(bar);
}

// A value that the compiler computes addresses from anew at each use, instead
// of keeping them all through a loop.
__device__ __forceinline__ uint32_t anew(uint32_t x) {
  asm volatile("" : "+r"(x));
  return x;
}

// Registers of a warpgroup, taken from and given back to what the block was
// launched with: kNT * 80 = 256 * 112 + 256 * 64 + 128 * 64 + 128 * 64.
template <int N>
__device__ __forceinline__ void set_registers_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void set_registers_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// The products of the decays from the start of 16 tokens through each lane's.
__device__ __forceinline__ float run_product(float a, int lane) {
#pragma unroll
  for (int o = 1; o < 16; o <<= 1) {
    const float x = __shfl_up_sync(kAllLanes, a, o, 16);
    if (lane % 16 >= o) a *= x;
  }
  return a;
}

// 16 value channels x 32 tokens of V, two tokens a register, times the tokens'
// weights, in three parts of 16 columns.
__device__ __forceinline__ void split_and_store(uint32_t to, uint32_t (&raw)[8],
                                                const float2 (&w)[4]) {
  uint32_t top[8], low[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    float2 x = __fmul2_rn(unpack(raw[i]), w[i / 2]);
    top[i] = pack(x);
    x = remainder(x, top[i]);
    raw[i] = pack(x);
    low[i] = pack(remainder(x, raw[i]));
  }
  tc::store_blocks(to, top);
  tc::store_blocks(to + 16, raw);
  tc::store_blocks(to + 32, low);
}

// Step i of 16 along a contraction, in an operand's units of 16 bytes: along
// the columns of a tile of `rows` rows, and along the rows.
__host__ __device__ constexpr uint32_t row_step(int i, int rows) {
  return (i / 4 * (rows * 128) + i % 4 * 32) / 16;
}
__host__ __device__ constexpr uint32_t column_step(int i) { return i * 2048 / 16; }

// Columns of tensor memory: the increment, P, O, and the ring of (w V)^T,
// 3 parts of 32 tokens (16 columns each) a slot.
constexpr uint32_t kGrown = 0, kP = 128, kO = 256, kRing = 384, kSlot = 48;
// Where part `part` of W o P lies for step i of 16 tokens: parts 0 and 1 over
// the step's own scores, part 2 behind the ring's first slot.
__host__ __device__ constexpr uint32_t weight_column(int part, int i) {
  return part < 2 ? kP + i * 16 + part * 8 : kRing + 64 + i * 8;
}

template <int DKP, int DVP, bool F32OUT, bool STATES>
__global__ void __launch_bounds__(kNT, 1)
    linear_chunks_kernel(const LinParams p, const Segments sg, const __grid_constant__ CUtensorMap mq,
                         const __grid_constant__ CUtensorMap mk,
                         const __grid_constant__ CUtensorMap mv,
                         const __grid_constant__ CUtensorMap mo) {
  using T = Tiles<DKP, DVP>;
  constexpr int PARTS = F32OUT ? 3 : 2;   // bf16 parts of W o P
  constexpr int SPARTS = F32OUT ? 3 : 2;  // and of the state in Q S^T
  constexpr int RING = F32OUT ? 1 : 2;    // slots of the ring
  constexpr int SWARPS = DVP / 16, VWARPS = DVP / 32;  // warps with the state, with w V
  extern __shared__ __align__(1024) uint8_t smem[];
  Control &ctl = *reinterpret_cast<Control *>(smem + T::kControl);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int h = blockIdx.x % p.Hv, hk = h / (p.Hv / p.Hk);
  Work pl;
  if (!locate<kNT, true>(p, sg, blockIdx.x / p.Hv, !sg.partial && h == 0,
                         reinterpret_cast<int *>(smem), pl))
    return;
  const int slot = pl.slot;
  const bool last = pl.index == pl.count - 1, fresh = pl.fresh;
  if (STATES && !sg.partial && !last) return;  // no outputs asked for: the last state alone
  const int first = pl.first + pl.index * sg.tokens;
  const int rest = pl.length - pl.index * sg.tokens;
  const int n = pl.count > 1 ? min(sg.tokens, rest) : rest;
  const int chunks = (n + kC - 1) / kC;
  if (chunks == 0 && !fresh) return;
  const int64_t tile = static_cast<int64_t>(p.dv) * p.dk;
  float *pool = p.S + (static_cast<int64_t>(slot) * p.Hv + h) * tile;
  float *entry = sg.states + (static_cast<int64_t>(pl.entry) * p.Hv + h) * tile;
  const int64_t entry_step = static_cast<int64_t>(p.Hv) * tile;

  if (sg.partial) let_next_start();
  const uint32_t base = tc::smem_addr(smem);
  volatile int *dead = &ctl.dead;
  const uint32_t bars = base + T::kControl + static_cast<uint32_t>(offsetof(Control, bar));
  auto at = [bars](uint32_t barrier) { return bars + 8 * barrier; };
  __syncthreads();  // what locate left in shared memory is read
  if (tid == 0) {
    for (int s = 0; s < 2; ++s) {
      tc::bar_init(at(kFullK + s), 1);
      tc::bar_init(at(kFullQ + s), 1);
      tc::bar_init(at(kStaged + s), 8);
      tc::bar_init(at(kFullV + s), 1);
      tc::bar_init(at(kEmptyQ + s), T::kOverQ && !F32OUT ? 2 : 1);
      tc::bar_init(at(kEmptyK + s), STATES ? 1 : 2);
      tc::bar_init(at(kEmptyV + s), STATES ? VWARPS : VWARPS + 1);
      tc::bar_init(at(kDecFull + s), 1);
      tc::bar_init(at(kDecEmpty + s), 8 + VWARPS + (STATES ? 0 : 8));
      tc::bar_init(at(kRingFull + s), VWARPS);
      tc::bar_init(at(kRingEmpty + s), 1);
    }
    tc::bar_init(at(kPFull), 1);
    tc::bar_init(at(kPDone), 8);
    tc::bar_init(at(kSReady), SWARPS);
    tc::bar_init(at(kQSPart), 1);
    tc::bar_init(at(kQSDone), 1);
    tc::bar_init(at(kOScaled), 8);
    tc::bar_init(at(kOFull), 1);
    tc::bar_init(at(kOEmpty), 8);
    tc::bar_init(at(kSFull), 1);
    tc::bar_init(at(kGrownRead), SWARPS);
    tc::bar_init(at(kStored), 1);
    tc::bar_init(at(kTail), SWARPS);
    ctl.dead = (base & 1023) != 0;  // never: the tiles' alignment
    if (ctl.dead) atomicOr(p.err, kErrTimeout);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 0) tc::tmem_alloc(tc::smem_addr(&ctl.tmem), 512);
  tc::fence_async();
  tc::before_sync();
  __syncthreads();
  tc::after_sync();
  const uint32_t tm = ctl.tmem;
  const bool sound = ctl.dead == 0;

  // Whether a chunk's outputs go through shared memory and a bulk store: whole
  // chunks do (the rows behind a last one are another sequence's), where the
  // outputs are aligned for it.
  auto staged = [&](int c) {
    return !F32OUT && n - c * kC >= kC && (reinterpret_cast<uintptr_t>(p.out) & 15) == 0;
  };
  if (!sound) {
  } else if (warp >= 20) {
    set_registers_down<64>();
    // The issuing warps run as a whole, which leaves their operands' addresses in
    // uniform registers, and one lane issues (by a single thread's code 32,768
    // tokens, 32 heads took 476 us where this took 451, with the state in one part
    // and in short bursts of calls; with two parts now 478, and 532 in long runs,
    // which the power cap slows down).
    const uint32_t lead = tc::elect();
    if (warp == 20) {
      constexpr uint32_t kShapeQK = tc::product_shape(kC, kC, false, false);
      constexpr uint32_t kShapeQS = tc::product_shape(kC, DVP, false, false);
      constexpr uint32_t kShapePV = tc::product_shape(kC, DVP, false, true);
      if constexpr (!STATES) {
        auto scores = [&](int c) {
          const uint32_t q = tc::operand(base + (c & 1) * T::kStage, 0);
#pragma unroll
          for (int i = 0; i < DKP / 16; ++i)
            tc::product_ss(lead, tm + kP, q + row_step(i, kC), q + T::kQ / 16 + row_step(i, kC),
                           kShapeQK, i > 0);
          tc::commit(lead, at(kPFull));
          tc::commit(lead, at(kEmptyK + (c & 1)));
        };
        bool ok = chunks > 0 && wait_warp(at(kFullK), 0, dead, p.err) &&
                  wait_warp(at(kFullQ), 0, dead, p.err);
        if (ok) scores(0);
#pragma unroll 1
        for (int c = 0; ok && c < chunks; ++c) {
          const int s = c & 1;
          const uint32_t stage = base + s * T::kStage;
          // Q S^T, part by part as the state's copies come
          ok = c == 0 || wait_warp(at(kOEmpty), (c - 1) & 1, dead, p.err);
#pragma unroll 1
          for (int part = 0; ok && part < SPARTS; ++part) {
            ok = wait_warp(at(kSReady), (c * SPARTS + part) & 1, dead, p.err);
            if (!ok) break;
            tc::after_sync();
            const uint32_t q = tc::operand(stage, 0);
            const uint32_t state = tc::operand(base + T::kState, 0);
#pragma unroll
            for (int i = 0; i < DKP / 16; ++i)
              tc::product_ss(lead, tm + kO, q + row_step(i, kC), state + row_step(i, DVP), kShapeQS,
                             i > 0 || part > 0);
            tc::commit(lead, part < SPARTS - 1 ? at(kQSPart) : at(kQSDone));
          }
          if (!ok) break;
          tc::commit(lead, at(kEmptyQ + s));
          // (W o P) V onto G (Q S^T), the small parts first
          ok = wait_warp(at(kFullV + s), (c >> 1) & 1, dead, p.err) &&
               (n - c * kC >= kC || wait_warp(at(kTail), 0, dead, p.err)) &&
               wait_warp(at(kPDone), c & 1, dead, p.err) &&
               wait_warp(at(kOScaled), c & 1, dead, p.err);
          if (!ok) break;
          tc::after_sync();
          const uint32_t v = tc::operand(stage + 2 * T::kQ, kC * 128);
#pragma unroll 1
          for (int part = PARTS - 1; part >= 0; --part)
#pragma unroll
            for (int i = 0; i < kC / 16; ++i)
              tc::product_ts(lead, tm + kO, tm + weight_column(part, i), v + column_step(i), kShapePV,
                             true);
          tc::commit(lead, at(kOFull));
          tc::commit(lead, at(kEmptyV + s));
          // the next scores, over W o P, which is read by then
          if (c + 1 < chunks) {
            ok = wait_warp(at(kFullK + (s ^ 1)), ((c + 1) >> 1) & 1, dead, p.err) &&
                 wait_warp(at(kFullQ + (s ^ 1)), ((c + 1) >> 1) & 1, dead, p.err) &&
                 wait_warp(at(kOFull), c & 1, dead, p.err);
            if (ok) scores(c + 1);
          }
        }
      }
    } else if (warp == 22) {
      // (w V)^T K, 32 tokens at a time, the small parts first.  The value
      // channels are padded to 128 rows, of which those behind DVP are never
      // read.
      constexpr uint32_t kShapeS = tc::product_shape(128, DKP, false, true);
      bool ok = true;
#pragma unroll 1
      for (int c = 0; ok && c < chunks; ++c) {
        const int s = c & 1;
        // the state's warps have taken the last increment
        ok = wait_warp(at(kFullK + s), (c >> 1) & 1, dead, p.err) &&
             (n - c * kC >= kC || wait_warp(at(kTail), 0, dead, p.err)) &&
             (c == 0 || wait_warp(at(kGrownRead), (c - 1) & 1, dead, p.err));
        uint32_t k = tc::operand(base + s * T::kStage + T::kQ, kC * 128);
#pragma unroll 1
        for (int r = 0; ok && r < 4; ++r) {
          const int fill = 4 * c + r, slot = fill % RING;
          ok = wait_warp(at(kRingFull + slot), (fill / RING) & 1, dead, p.err);
          if (!ok) break;
          tc::after_sync();
          const uint32_t a = tm + kRing + slot * kSlot;
#pragma unroll
          for (int part = 2; part >= 0; --part)
#pragma unroll
            for (int i = 0; i < 2; ++i)
              tc::product_ts(lead, tm + kGrown, a + part * 16 + i * 8, k + column_step(i), kShapeS,
                             r > 0 || i > 0 || part < 2);
          tc::commit(lead, at(kRingEmpty + slot));
          k = k + 2 * column_step(1);
        }
        if (!ok) break;
        tc::commit(lead, at(kSFull));
        tc::commit(lead, at(kEmptyK + s));
      }
    } else if (warp == 21) {
      if (lane == 0) {
#pragma unroll 1
        for (int c = 0; c < chunks; ++c) {
          const int s = c & 1, row = first + c * kC;
          const uint32_t before = ((c >> 1) - 1) & 1;
          const uint32_t q = base + s * T::kStage, k = q + T::kQ, v = k + T::kQ;
          // in the order in which the tiles before are done with, Q's last: its
          // place holds the outputs
          if (c >= 2 && !wait_one(at(kEmptyK + s), before, dead, p.err)) break;
          tc::bar_expect(at(kFullK + s), T::kQ);
#pragma unroll
          for (int x = 0; x < DKP; x += 64)
            tc::load_tile(k + x * (2 * kC), &mk, at(kFullK + s), x, hk, row);
          if (c >= 2 && !wait_one(at(kEmptyV + s), before, dead, p.err)) break;
          tc::bar_expect(at(kFullV + s), T::kV);
#pragma unroll
          for (int x = 0; x < DVP; x += 64)
            tc::load_tile(v + x * (2 * kC), &mv, at(kFullV + s), x, h, row);
          if constexpr (!STATES) {
            if (c >= 2 && !wait_one(at(kEmptyQ + s), before, dead, p.err)) break;
            tc::bar_expect(at(kFullQ + s), T::kQ);
#pragma unroll
            for (int x = 0; x < DKP; x += 64)
              tc::load_tile(q + x * (2 * kC), &mq, at(kFullQ + s), x, hk, row);
          }
        }
      }
    } else {
      // The products of a chunk's decays: 4 tokens a lane, 8 lanes a block of 32.
      float a[4];
      auto fetch = [&](int c) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int t = c * kC + 4 * lane + i;
          a[i] = t >= n ? 1.0f
                        : p.decay[p.decay_head ? h : static_cast<int64_t>(first + t) * p.Hv + h];
        }
      };
      double total = 1.0;
      auto decays = [&](int c) {
        const int s = c & 1;
        double r[4];  // products from behind token i to the lane's last
        r[3] = 1.0;
#pragma unroll
        for (int i = 2; i >= 0; --i) r[i] = r[i + 1] * a[i + 1];
        double run = r[0] * a[0];
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) {
          const double x = __shfl_down_sync(kAllLanes, run, o, 8);
          if (lane % 8 + o < 8) run *= x;
        }
        // run: from the lane's first token to the block's end; behind the lane:
        double behind = __shfl_down_sync(kAllLanes, run, 1, 8);
        if (lane % 8 == 7) behind = 1.0;
        const double whole = __shfl_sync(kAllLanes, run, 0) * __shfl_sync(kAllLanes, run, 8) *
                             __shfl_sync(kAllLanes, run, 16) * __shfl_sync(kAllLanes, run, 24);
        total *= whole;
        if (c >= 2 && !wait_warp(at(kDecEmpty + s), ((c >> 1) - 1) & 1, dead, p.err)) return false;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          ctl.dec[s].a[4 * lane + i] = a[i];
          ctl.dec[s].rest[4 * lane + i] = static_cast<float>(r[i] * behind);
        }
        if (lane % 8 == 0) ctl.block[s][lane / 8] = static_cast<float>(run);
        if (lane == 0) {
          const float hi = static_cast<float>(whole);
          ctl.whole[s][0] = hi;
          ctl.whole[s][1] = static_cast<float>(whole - hi);
        }
        arrive_warp(at(kDecFull + s));
        if (c + 1 < chunks) fetch(c + 1);
        return true;
      };
      bool ok = true;
      if (chunks > 0) {
        fetch(0);
        ok = decays(0);
      }
      if (ok && chunks > 1) ok = decays(1);
#pragma unroll 1
      for (int c = 0; ok && c < chunks; ++c) {
        // before the wait for the outputs: all other warps need the decays
        if (c + 2 < chunks && !(ok = decays(c + 2))) break;
        if constexpr (!STATES && !F32OUT) {
          // the chunk's outputs, unless they have left from registers
          const int s = c & 1;
          if (!(ok = wait_warp(at(kStaged + s), (c >> 1) & 1, dead, p.err))) break;
          if (lane == 0 && staged(c)) {
            const uint32_t from = base + (T::kOverQ ? s * T::kStage : T::kOut);
#pragma unroll
            for (int x = 0; x < DVP; x += 64)
              tc::store_tile(&mo, from + x * (2 * kC), x, h, first + c * kC);
            tc::store_done();
          }
          arrive_warp(at(kStored));
          if (T::kOverQ) arrive_warp(at(kEmptyQ + s));
        }
      }
      if (sg.partial && lane == 0)
        sg.decays[static_cast<int64_t>(pl.entry + 1 + pl.index) * p.Hv + h] =
            static_cast<float>(total);
    }
  } else if (warp >= 8 && warp < 16) {
    set_registers_down<64>();
    if constexpr (!STATES) {
      // Token 32 w + lane; the two warps of a quadrant share its columns.
      const int w = warp & 3, side = (warp - 8) >> 2;
      const uint32_t lanes = static_cast<uint32_t>(w * 32) << 16;
      // Products of decays through the row's token: from the start of its 16
      // tokens, and of its block.
      float near = 1.0f, grow = 1.0f;
      auto decays = [&](int c) {
        if (!wait_warp(at(kDecFull + (c & 1)), (c >> 1) & 1, dead, p.err)) return false;
        near = run_product(ctl.dec[c & 1].a[w * 32 + lane], lane);
        const float lower = __shfl_sync(kAllLanes, near, 15);
        grow = lane < 16 ? near : near * lower;
        return true;
      };
      bool ok = chunks == 0 || decays(0);
#pragma unroll 1
      for (int c = 0; ok && c < chunks; ++c) {
        const int s = c & 1;
        const Decays &dec = ctl.dec[s];
        if (!(ok = wait_warp(at(kPFull), c & 1, dead, p.err))) break;
        tc::after_sync();
        // 16 columns of each block of 32, in a loop (with all roles unrolled
        // their code does not fit the instruction caches); the next ones are
        // loaded meanwhile.
        uint32_t next[16];
        tc::load16(tm + kP + lanes + side * 16, next);
        float f = grow;  // from b's end through the row's token
        if (w > 1) f *= ctl.block[s][1];
        if (w > 2) f *= ctl.block[s][2];
#pragma unroll 1
        for (int b = 0; b < 4; ++b) {
          const int step = 2 * b + side;
          uint32_t y[16];
          if (b <= w) {
            tc::wait_loads(next);
#pragma unroll
            for (int j = 0; j < 16; ++j) y[j] = next[j];
            if (b < w) tc::load16(tm + kP + lanes + step * 16 + 32, next);
            const int j0 = side * 16;
            if (b == w) {
              float run = side == 0 && lane >= 16 ? near : 1.0f;
              const float *a = &dec.a[step * 16];
#pragma unroll
              for (int j = 15; j >= 0; --j) {
                if (j < 15 && j0 + j < lane) run *= a[j + 1];
                y[j] = j0 + j <= lane ? bits(__uint_as_float(y[j]) * run) : 0u;
              }
            } else {
              const float2 ff = make_float2(f, f);
#pragma unroll
              for (int j = 0; j < 16; j += 4) {
                const float4 r = *reinterpret_cast<const float4 *>(&dec.rest[step * 16 + j]);
                scale2(y[j], y[j + 1], __fmul2_rn(ff, make_float2(r.x, r.y)));
                scale2(y[j + 2], y[j + 3], __fmul2_rn(ff, make_float2(r.z, r.w)));
              }
              // without the next block
              f = grow;
              if (b == 0 && w > 2) f *= ctl.block[s][2];
            }
          } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) y[j] = 0u;
          }
          uint32_t z[16];  // the parts, 8 columns each
#pragma unroll
          for (int part = 0; part < 2; ++part)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float2 x = floats(y[2 * j], y[2 * j + 1]);
              z[part * 8 + j] = pack(x);
              if (part + 1 < PARTS) {
                const float2 left = remainder(x, z[part * 8 + j]);
                y[2 * j] = bits(left.x), y[2 * j + 1] = bits(left.y);
              }
            }
          tc::store16(tm + lanes + weight_column(0, step), z);
          if constexpr (PARTS == 3) {
            uint32_t u[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) u[j] = pack(floats(y[2 * j], y[2 * j + 1]));
            tc::store8(tm + lanes + weight_column(2, step), u);
          }
        }
        tc::wait_stores();
        tc::before_sync();
        arrive_warp(at(kPDone));
        arrive_warp(at(kDecEmpty + s));
        if (c + 1 < chunks) ok = decays(c + 1);
      }
    }
  } else if (warp >= 16) {
    set_registers_down<64>();
    const int quad = warp & 3;
    if (quad * 32 < DVP) {
      // (w V)^T in three parts: value channels 32 quad .. + 31
      const int e16 = quad * 32;
#pragma unroll 1
      for (int c = 0; c < chunks; ++c) {
        const int s = c & 1;
        bool ok = wait_warp(at(kFullV + s), (c >> 1) & 1, dead, p.err) &&
                  wait_warp(at(kDecFull + s), (c >> 1) & 1, dead, p.err);
        if (ok && n - c * kC < kC) ok = wait_warp(at(kTail), 0, dead, p.err);
        if (!ok) break;
        const float4 block = *reinterpret_cast<const float4 *>(ctl.block[s]);
        const uint32_t tile_v = base + s * T::kStage + 2 * T::kQ + e16 / 64 * (kC * 128) +
                                ((lane & 7) + (lane >> 4) * 8) * 128;
        // 16-byte units of the quadrant's two halves, swizzled by the row
        const int u = e16 % 64 / 8 + (lane >> 3 & 1);
        const uint32_t unit0 = (u ^ (lane & 7)) << 4, unit1 = ((u + 2) ^ (lane & 7)) << 4;
#pragma unroll 1
        for (int r = 0; r < 4; ++r) {
          const uint32_t from = tile_v + r * 32 * 128;
          uint32_t raw0[8], raw1[8];
          tc::load_transposed(from + unit0, raw0, 0);
          tc::load_transposed(from + unit0 + 16 * 128, raw0, 4);
          tc::load_transposed(from + unit1, raw1, 0);
          tc::load_transposed(from + unit1 + 16 * 128, raw1, 4);
          // the blocks of tokens behind this one
          const float behind = r == 0   ? block.y * block.z * block.w
                               : r == 1 ? block.z * block.w
                               : r == 2 ? block.w
                                        : 1.0f;
          float2 w[4];
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            w[g] = *reinterpret_cast<const float2 *>(
                &ctl.dec[s].rest[r * 32 + g * 8 + (lane & 3) * 2]);
            w[g] = __fmul2_rn(w[g], make_float2(behind, behind));
          }
          const int fill = 4 * c + r, slot = fill % RING;
          if (fill >= RING &&
              !(ok = wait_warp(at(kRingEmpty + slot), (fill / RING - 1) & 1, dead, p.err)))
            break;
          tc::after_sync();
          const uint32_t to = tm + kRing + slot * kSlot + (static_cast<uint32_t>(e16) << 16);
          split_and_store(to, raw0, w);
          split_and_store(to + (16u << 16), raw1, w);
          tc::wait_stores();
          tc::before_sync();
          arrive_warp(at(kRingFull + slot));
        }
        if (!ok) break;
        arrive_warp(at(kEmptyV + s));
        arrive_warp(at(kDecEmpty + s));
      }
    }
  } else {
    set_registers_up<112>();
    // Lane l of quadrant x holds value channel 32 x + l and kF key channels
    // from f0.
    constexpr int kF = DKP / 2;
    const int quad = warp & 3, half = warp >> 2;
    const int e = quad * 32 + lane, f0 = half * kF;
    const bool holds = quad * 32 < DVP;
    float S[kF];
    const bool mine = holds && e < p.dv && f0 < p.dk;
    auto load_state = [&](const float *src) {
      const float4 *row = reinterpret_cast<const float4 *>(src + e * p.dk + f0);
#pragma unroll
      for (int f = 0; f < kF; f += 4) {
        const float4 x = mine ? row[f / 4] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        S[f] = x.x, S[f + 1] = x.y, S[f + 2] = x.z, S[f + 3] = x.w;
      }
    };
    auto store_state = [&](float *dst) {
      float *row = dst + e * p.dk + f0;
      if (mine && (reinterpret_cast<uintptr_t>(dst) & 31) == 0) {
#pragma unroll
        for (int f = 0; f < kF; f += 8) {  // whole sectors
          uint32_t v[16];
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = bits(S[f + j]);
          store_global32(row + f, v, 0);
        }
      } else if (mine) {
#pragma unroll
        for (int f = 0; f < kF; f += 4)
          *reinterpret_cast<float4 *>(row + f) = make_float4(S[f], S[f + 1], S[f + 2], S[f + 3]);
      }
    };
    wait_for_states();
    if (!fresh && sg.partial && pl.index == 0) {
      // a split sequence's first state moves to the workspace: the block of
      // the last segment writes the pool while others still need it
      load_state(pool);
      store_state(entry);
    }
    if (fresh || sg.partial) {
#pragma unroll
      for (int f = 0; f < kF; ++f) S[f] = 0.0f;
    } else {
      load_state(pl.count > 1 ? entry : pool);
    }
    if (!sg.partial) {
#pragma unroll 1
      for (int r = 0; r < pl.index; ++r) {
        const float d = sg.decays[static_cast<int64_t>(pl.entry + 1 + r) * p.Hv + h];
        const float4 *row = reinterpret_cast<const float4 *>(entry + (r + 1) * entry_step +
                                                             e * p.dk + f0);
#pragma unroll
        for (int f = 0; f < kF; f += 4) {
          if (f % 16 == 0) asm volatile("" ::: "memory");
          if (mine) {
            const float4 x = row[f / 4];
            S[f] = fmaf(S[f], d, x.x), S[f + 1] = fmaf(S[f + 1], d, x.y);
            S[f + 2] = fmaf(S[f + 2], d, x.z), S[f + 3] = fmaf(S[f + 3], d, x.w);
          }
        }
      }
    }
    float g_hi = 0.0f, g_lo = 0.0f, row_scale = 1.0f;
    bool ok = true;
    // S' from the increment of chunk c
    auto advance = [&](int c) {
      const float2 hi = make_float2(g_hi, g_hi), lo = make_float2(g_lo, g_lo);
      if (!wait_warp(at(kSFull), c & 1, dead, p.err)) return false;
      tc::after_sync();
      const uint32_t from = tm + kGrown + (static_cast<uint32_t>(quad * 32) << 16) + f0;
#pragma unroll
      for (int f = 0; f < kF; f += 32) {
        uint32_t x[2][16];
        tc::load16(from + f, x[0]);
        tc::load16(from + f + 16, x[1]);
        tc::wait_loads(x[0], x[1]);
#pragma unroll
        for (int j = 0; j < 32; j += 2) {
          const float2 old = make_float2(S[f + j], S[f + j + 1]);
          float2 now = floats(x[j / 16][j % 16], x[j / 16][j % 16 + 1]);
          now = __ffma2_rn(old, lo, now);
          now = __ffma2_rn(old, hi, now);
          S[f + j] = now.x, S[f + j + 1] = now.y;
        }
      }
      tc::before_sync();
      arrive_warp(at(kGrownRead));
      return true;
    };
    // The state's bf16 copy, a part at a time: row e of [DVP][DKP].  S being the
    // same for all parts, the compiler would keep earlier ones and remainders across
    // the waits in between, and spill for it with DKP = 128 (fp32 outputs: 786 bytes
    // stored and 1,196 loaded a thread, bf16 350 and 700): there S is hidden from it,
    // which leaves 60 to 80 and 220 to 256.
    auto copy_state = [&](auto part) {
      constexpr int kPart = decltype(part)::value;
      if constexpr (kPart > 0 && DKP == 128) {
#pragma unroll
        for (int f = 0; f < kF; ++f) asm volatile("" : "+f"(S[f]));
      }
      const uint32_t row = anew(base) + T::kState + f0 / 64 * (DVP * 128) + e * 128;
#pragma unroll
      for (int f = 0; f < kF; f += 8) {
        uint32_t v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          v[j] = part_of<kPart>(make_float2(S[f + 2 * j], S[f + 2 * j + 1]));
        }
        const int u = (f0 % 64 + f) / 8;
        store_shared16(row + ((u ^ (e & 7)) << 4), v[0], v[1], v[2], v[3]);
      }
      tc::fence_async();
      arrive_warp(at(kSReady));
    };
    // The outputs of chunk c: token `row`, the value channels of its half.
    const int row = quad * 32 + lane, half_e = half * (DVP / 2);
    const uint32_t lanes = static_cast<uint32_t>(quad * 32) << 16;
    auto outputs = [&](int c) {
      if (!wait_warp(at(kOFull), c & 1, dead, p.err)) return false;
      tc::after_sync();
      const bool through = staged(c);
      if (!F32OUT && !T::kOverQ && c > 0 && !wait_warp(at(kStored), (c - 1) & 1, dead, p.err))
        return false;
      const uint32_t to_tile = base + (T::kOverQ ? (c & 1) * T::kStage : T::kOut) + row * 128;
      const bool live = c * kC + row < n;
      const bool wide = (reinterpret_cast<uintptr_t>(p.out) & 31) == 0;
      const int64_t to = (static_cast<int64_t>(first + c * kC + row) * p.Hv + h) * p.dv;
#pragma unroll 1
      for (int e = half_e; e < half_e + DVP / 2; e += 16) {
        uint32_t x[16];
        tc::load16(tm + kO + lanes + e, x);
        tc::wait_loads(x);
        if constexpr (!F32OUT) {
          uint32_t v[16];
#pragma unroll
          for (int j = 0; j < 8; ++j) v[j] = pack(floats(x[2 * j], x[2 * j + 1]));
          if (through) {
            const int u = e % 64 / 8;
            const uint32_t block = to_tile + e / 64 * (kC * 128);
            store_shared16(block + ((u ^ (row & 7)) << 4), v[0], v[1], v[2], v[3]);
            store_shared16(block + (((u + 1) ^ (row & 7)) << 4), v[4], v[5], v[6], v[7]);
          } else if (live && e < p.dv) {
            __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.out) + to + e;
            if (wide) {
              store_global32(dst, v, 0);
            } else {
#pragma unroll
              for (int j = 0; j < 16; ++j)
                reinterpret_cast<uint16_t *>(dst)[j] = static_cast<uint16_t>(v[j / 2] >> (j % 2 * 16));
            }
          }
        } else if (live && e < p.dv) {
          float *dst = static_cast<float *>(p.out) + to + e;
          if (wide) {
            store_global32(dst, x, 0);
            store_global32(dst + 8, x, 8);
          } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) dst[j] = __uint_as_float(x[j]);
          }
        }
        __syncwarp();
      }
      tc::before_sync();
      arrive_warp(at(kOEmpty));
      if constexpr (!F32OUT) {
        tc::fence_async();
        arrive_warp(at(kStaged + (c & 1)));
      }
      return true;
    };
#pragma unroll 1
    for (int c = 0; c < chunks; ++c) {
      const int s = c & 1;
      const uint32_t stage = anew(base) + s * T::kStage;
      const int live = n - c * kC;  // tokens of the chunk
      if (holds && live < kC) {
        // rows of other sequences behind the last token: nothing may come of them
        ok = wait_warp(at(kFullK + s), (c >> 1) & 1, dead, p.err) &&
             wait_warp(at(kFullV + s), (c >> 1) & 1, dead, p.err);
        if (!ok) break;
        const int bt = (half * (SWARPS / 2) + quad) * 32 + lane;
        for (int i = bt; i < T::kQ / 16; i += SWARPS * 32)
          if (i % (kC * 8) / 8 >= live) store_shared16(stage + T::kQ + i * 16, 0u, 0u, 0u, 0u);
        for (int i = bt; i < T::kV / 16; i += SWARPS * 32)
          if (i % (kC * 8) / 8 >= live) store_shared16(stage + 2 * T::kQ + i * 16, 0u, 0u, 0u, 0u);
        tc::fence_async();
        arrive_warp(at(kTail));
      }
      if (holds && c > 0 && !(ok = advance(c - 1))) break;
      if (!(ok = wait_warp(at(kDecFull + s), (c >> 1) & 1, dead, p.err))) break;
      g_hi = ctl.whole[s][0], g_lo = ctl.whole[s][1];
      if constexpr (!STATES) {
        const float near = run_product(ctl.dec[s].a[row], lane);
        const float lower = __shfl_sync(kAllLanes, near, 15);
        const float4 block = *reinterpret_cast<const float4 *>(ctl.block[s]);
        row_scale = (lane < 16 ? near : near * lower) * (quad > 0 ? block.x : 1.0f) *
                    (quad > 1 ? block.y : 1.0f) * (quad > 2 ? block.z : 1.0f);
      }
      arrive_warp(at(kDecEmpty + s));
      if constexpr (!STATES) {
        if (c > 0 && !(ok = wait_warp(at(kQSDone), (c - 1) & 1, dead, p.err))) break;
        if (holds) {
          copy_state(std::integral_constant<int, 0>());
          // its further parts once the products with the last one are done; those
          // need the last chunk's outputs out of the way
          if (c > 0 && !(ok = outputs(c - 1))) break;
          if (!(ok = wait_warp(at(kQSPart), F32OUT ? 0 : c & 1, dead, p.err))) break;
          copy_state(std::integral_constant<int, 1>());
          if constexpr (F32OUT) {
            if (!(ok = wait_warp(at(kQSPart), 1, dead, p.err))) break;
            copy_state(std::integral_constant<int, 2>());
          }
        }
        if (!holds && c > 0 && !(ok = outputs(c - 1))) break;
        // G (Q S^T)
        if (!(ok = wait_warp(at(kQSDone), c & 1, dead, p.err))) break;
        tc::after_sync();
        const float2 scale = make_float2(row_scale, row_scale);
#pragma unroll 1
        for (int e = half_e; e < half_e + DVP / 2; e += 32) {
          uint32_t x[16], y[16];
          tc::load16(tm + kO + lanes + e, x);
          tc::load16(tm + kO + lanes + e + 16, y);
          tc::wait_loads(x, y);
#pragma unroll
          for (int j = 0; j < 16; j += 2) {
            scale2(x[j], x[j + 1], scale);
            scale2(y[j], y[j + 1], scale);
          }
          tc::store16(tm + kO + lanes + e, x);
          tc::store16(tm + kO + lanes + e + 16, y);
        }
        tc::wait_stores();
        tc::before_sync();
        arrive_warp(at(kOScaled));
      }
    }
    if (ok && holds && chunks > 0) ok = advance(chunks - 1);
    if constexpr (!STATES) {
      if (ok && chunks > 0) ok = outputs(chunks - 1);
    }
    if (ok && holds) {
      if (sg.partial)
        store_state(entry + (pl.index + 1) * entry_step);
      else if (last)
        store_state(pool);
    }
  }
  __syncthreads();
  if (ctl.dead != 0 && tid == 0) {
    // A wait ran out: give the copies and products in flight time to land.
    for (int i = 0; i < 2000; ++i) __nanosleep(1000);
  }
  __syncthreads();
  if (warp == 0) tc::tmem_free(tm, 512);
}

// ---- launch --------------------------------------------------------------

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                                 const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                                 const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// The driver's encoder, looked up once.
EncodeTiled encoder() {
  static const EncodeTiled fn = [] {
    void *f = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                         &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      return static_cast<EncodeTiled>(nullptr);
    return reinterpret_cast<EncodeTiled>(f);
  }();
  return fn;
}

// [tokens][heads][d] with a token stride, in boxes of 128 tokens x 64 channels
// of one head.  Channels past d and tokens past the last row read as zeros.
bool encode(CUtensorMap *map, const void *p, int tokens, int heads, int d, int64_t stride) {
  const cuuint64_t dims[3] = {static_cast<cuuint64_t>(d), static_cast<cuuint64_t>(heads),
                              static_cast<cuuint64_t>(tokens)};
  const cuuint64_t strides[2] = {static_cast<cuuint64_t>(d) * 2,
                                 static_cast<cuuint64_t>(stride) * 2};
  const cuuint32_t box[3] = {64, 1, kC}, unit[3] = {1, 1, 1};
  return encoder()(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void *>(p), dims, strides,
                   box, unit, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                   CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                   CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DKP, int DVP, bool F32OUT, bool STATES>
cudaError_t launch_t(const LinParams &p, const Segments &sg, const CUtensorMap (&m)[4], int64_t grid,
                     bool overlaps, cudaStream_t st) {
  auto kernel = linear_chunks_kernel<DKP, DVP, F32OUT, STATES>;
  // once for each device
  static std::atomic<uint64_t> ready{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if ((ready.load(std::memory_order_acquire) & bit) == 0) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             Tiles<DKP, DVP>::kBytes);
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit, std::memory_order_release);
  }
  return launch_next(kernel, grid, kNT, Tiles<DKP, DVP>::kBytes, overlaps, st, p, sg, m[0], m[1], m[2],
                     m[3]);
}

template <int DKP, int DVP>
cudaError_t launch_d(const LinParams &p, Segments sg, const CUtensorMap (&m)[4], cudaStream_t st) {
  const int64_t split = split_segments(p, sg.tokens);
  if (split > 0) {
    sg.partial = true;
    const cudaError_t e = launch_t<DKP, DVP, false, true>(p, sg, m, split * p.Hv, false, st);
    if (e != cudaSuccess) return e;
    sg.partial = false;
  }
  const int64_t grid = (split + p.B) * p.Hv;
  const bool over = split > 0;
  if (p.out == nullptr) return launch_t<DKP, DVP, false, true>(p, sg, m, grid, over, st);
  if (p.out_bf16) return launch_t<DKP, DVP, false, false>(p, sg, m, grid, over, st);
  return launch_t<DKP, DVP, true, false>(p, sg, m, grid, over, st);
}

}  // namespace

constexpr int kSMs = 148, kMostWaves = 4;

// Tokens of a segment.  One block an SM walks over a segment, so that n
// segments of every head take `waves` rounds of n heads / SMs blocks; a round
// costs its chunks and about two more (its start and its end).  The segments'
// own states, which a second launch needs first, cost about half of that again:
// a call is split only where it gains more.  Several sequences keep the SMs
// busy side by side: pieces of one need not be shorter than an SM's share of
// the call.
int linear_segment(const LinParams &p) {
  const int64_t chunks = (static_cast<int64_t>(p.tokens) + kC - 1) / kC;
  int64_t best = chunks, cost = chunks + 2;
  for (int waves = 1; waves <= kMostWaves; ++waves) {
    const int64_t n = kSMs * waves / p.Hv;
    if (n < 2) continue;
    const int64_t each = (chunks + n - 1) / n;
    const int64_t c = waves * (each + 2) * 3 / 2;
    if (c < cost) best = each, cost = c;
  }
  const int64_t share = (chunks * p.Hv + kSMs - 1) / kSMs;
  if (p.B > 1 && best < share) best = share;
  if (p.B > 1 && best + best / 2 >= chunks) best = chunks;  // no sequence to cut, see below
  const int64_t tokens = (best < 1 ? 1 : best) * kC;
  return static_cast<int>(tokens > 1 << 29 ? 1 << 29 : tokens);
}

// The longest sequence that stays whole.  The states' pass makes a cut sequence
// cost half as much again, so among several, one of up to one and a half shares
// of an SM takes no longer whole if its blocks start first (Rank): 24 prompts of
// 20,011 tokens in all, 32 heads, the longest 1.4 shares, 271 us whole and 345 us
// cut (fp32 outputs 405 and 449); 9 prompts of 7,000 tokens, the longest 1.95
// shares, fp32 outputs, 217 us whole and 191 us cut (bf16 outputs 140 and 147).
static int longest_whole(const LinParams &p, int segment) {
  return p.B > 1 && p.B <= kRankedMost && segment < p.tokens ? segment + segment / 2 : segment;
}

size_t linear_chunks_workspace(const LinParams &p) {
  return segments_workspace(p, split_segments(p, linear_segment(p)));
}

// linear_segment covers a call's chunks at most kSMs * 4 / heads times (any
// number of sequences; a segment is one chunk at least), or by its limit of 2^29
// tokens.
size_t linear_chunks_workspace_most(const LinParams &p) {
  const int64_t some = p.tokens / kC, cut = kSMs * kMostWaves / p.Hv, limit = p.tokens >> 29;
  const int64_t most = cut > limit ? cut : limit;
  return segments_workspace(p, some < most ? some : most);
}

cudaError_t launch_linear_chunks(const LinParams &p, void *workspace, cudaStream_t st) {
  if (encoder() == nullptr) return cudaErrorNotSupported;
  CUtensorMap m[4] = {};
  if (p.tokens > 0) {
    if (!encode(&m[0], p.q, p.tokens, p.Hk, p.dk, p.q_stride) ||
        !encode(&m[1], p.k, p.tokens, p.Hk, p.dk, p.k_stride) ||
        !encode(&m[2], p.v, p.tokens, p.Hv, p.dv, p.v_stride))
      return cudaErrorInvalidValue;
    // an output that a bulk store could not reach goes out in single values
    if (p.out != nullptr && p.out_bf16 && reinterpret_cast<uintptr_t>(p.out) % 16 == 0 &&
        !encode(&m[3], p.out, p.tokens, p.Hv, p.dv, static_cast<int64_t>(p.Hv) * p.dv))
      return cudaErrorInvalidValue;
  }
  const int segment = linear_segment(p);
  const Segments sg = segments_in(p, segment, longest_whole(p, segment), workspace);
  if (p.dk <= 64) return p.dv <= 64 ? launch_d<64, 64>(p, sg, m, st) : launch_d<64, 128>(p, sg, m, st);
  return p.dv <= 64 ? launch_d<128, 64>(p, sg, m, st) : launch_d<128, 128>(p, sg, m, st);
}

}  // namespace lq

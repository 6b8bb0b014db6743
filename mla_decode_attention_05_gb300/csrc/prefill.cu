// Prefill attention: the queries of prompts, or of chunks of new tokens, over
// the expanded keys and values of their sequences.  For query row i of a
// sequence with n_q queries and n_k keys, and head h,
//   s_j = scale * (q[i][h][0:128] . k_nope[j][h] + q[i][h][128:192] . k_pe[j])
//   lse = ln sum_j exp(s_j),  out = sum_j exp(s_j - lse) v[j][h]
// over j < n_k, causal: j < n_k - n_q + i + 1 (the last query sees every key).
// A row without keys gets out = 0 and lse = -inf.
//
// 640 flops a pair and head against one exponential, so the tensor cores
// bound it (8192 tokens, 32 heads, causal: 440 us in a long run of calls, 401 us,
// 1.7 PFLOP/s, over fifty from rest; eight prompts of 136 to 1500 tokens, 128
// heads: 302 and 282 us); softmax has to stay in their shadow.  (Figures below
// that compare two forms were taken side by side when the choice was made.)  One
// pass over the keys with a running reference m and sum l per row:
//   p_j = 2^(s_j c - m c),  l += p_j,  O += p_j v_j        (c = scale log2 e)
// m is the row's maximum when it was last moved.  It moves, and O and l are
// scaled down, only when the maximum has grown by more than 8 in the exponent:
// until then p stays below 2^8, which costs fp32 sums and bf16 probabilities
// no precision (a rounding is relative), and O is rarely touched.
//
// Roundings: p to bf16 (the MMA's operand; l sums the fp32 values), out to
// bf16 once.  Scores, m, l and O are fp32.
//
// Values that a row does not see must not reach it, whatever they hold: 0 * inf
// and 0 * nan in P V would.  Such a row comes out as nan.  So a unit of work in
// which some row sees only a part of its keys, and some output is not finite, is
// done again: then a warp looks through the values of those steps in shared
// memory, replaces what is not finite by zero before the MMA reads it and notes
// the key, and rows that do see such a key add its non-finite values at the
// end.  (A weight is positive, so inf and nan reach the row's output as they
// are.)  Looking through all values the first time cost ragged prompts a third.
#include <cstddef>

#include "common.cuh"
#include "dependent.cuh"
#include "ptx.cuh"
#include "ptx_pair.cuh"
#include "tma_map.cuh"

namespace mla {
namespace {

using namespace ptx;

constexpr int kNope = 128;
constexpr int kHead = 192;
constexpr int kDv = 128;
constexpr int kRows = 128;     // query rows of one tile; a CTA has two
constexpr int kKeys = 128;     // keys of one step
constexpr int kCtaRows = 2 * kRows;

// Warps 0-3 and 4-7: softmax and output of tile 0 and 1 (one row a thread);
// warp 8 issues the MMAs, warp 9 the loads, warp 10 hands out the work, warp 11
// waits for warp 8.  Registers move between the three warpgroups, from 168 a
// thread at launch to 208 for the softmax and 88 for the rest (2 * 208 + 88 =
// 3 * 168).
constexpr int kThreads = 384;

// Shared memory: Q of both tiles as 2 x 3 blocks of 128 rows x 64 values; a
// ring of 16 KB units for keys (128 keys x 64 values: no-PE low, no-PE high,
// PE) and values (64 keys x 128 values, as two boxes of 64 values).
constexpr uint32_t kUnit = 16384;
constexpr int kUnits = 8;
constexpr int kUnitsPerStep = 5;
constexpr uint32_t OFF_RING = 6 * kUnit;
constexpr uint32_t OFF_BARS = OFF_RING + kUnits * kUnit;

// Tensor memory: S of both tiles (P, as bf16, over the S it came from), O of both.
constexpr uint32_t TM_S = 0;
constexpr uint32_t TM_O = 256;
constexpr uint32_t IDESC_QK = idesc_bf16_f32(128, 128, false, false);
constexpr uint32_t IDESC_PV = idesc_bf16_f32(128, 128, false, true);
constexpr float kMoveAt = 8.f;
constexpr int kMaxSplits = 32;  // parts of a unit's keys, a lane each in the join

struct PrefillParams {
  const int32_t *cu_q, *cu_k;
  const __nv_bfloat16 *v;
  __nv_bfloat16 *out;  // [Nq][H][128]
  float *lse;          // [H][Nq]
  float *part_o;       // splits > 1: [splits][Nq][H][128], normalised
  float *part_lse;     // splits > 1: [splits][H][Nq]
  unsigned int *status;
  long long v_tok, v_head;
  int B, H, Nq, Nk, tiles, splits;
  int causal;
  int out_v8;
  float scale, scale_log2;
  uint32_t wait_ns;  // limit of every wait
};
// The same for the kernel that is compiled for short limits (kPoll) or for others.
template <bool kPoll>
struct Limited : PrefillParams {
  static constexpr bool poll = kPoll;
};

// A CTA's unit of work: up to 256 query rows of one sequence, one head, a
// range of its keys.
struct Work {
  int q0, nq;  // first row in the packed queries, rows (<= 256); 0: no more work
  int k0, nk;  // first key, keys
  int diff;    // row i sees min(nk, max(0, diff + i + 1)) of them
  int h, split;
  int block;   // the block of the grid that it is
};

// Steps over its keys: n[t] of tile t, of which those from `masked` on hold
// keys that some row of a tile does not see.  The values of the steps from
// `look` on are looked through.
struct Steps {
  int n[2], most, masked, look;
};
constexpr int kNever = 1 << 30;
constexpr int kRedo = 64;

struct Bars {
  uint64_t k_full[2], v_full[2];  // the keys (values) of every second step have landed
  uint64_t empty[kUnits];         // all products with this part of the ring are done
  uint64_t work_full[2], work_empty[2];
  uint64_t taken;       // the load warp is about to end a unit of work
  uint64_t q_full[2], q_empty[2];
  uint64_t s_full[2];   // scores of a tile are in tensor memory
  uint64_t p_full[2][2];  // its probabilities are: of the first and the last 64 keys
  uint64_t o_done[2];   // its last P V of a unit of work has been added
  uint64_t o_free[2];   // its output has been read
  uint64_t v_look;      // the values of a step are there (told by the waiting warp: the ring's barriers
                        // can be a phase further than a warp that does not follow every unit)
  uint64_t v_ok;        // they have been looked through
  uint64_t next_full;   // the answer to a request for the next unit of work
  uint4 next;           // (16 bytes, 16-byte aligned)
  Work work[2];
  Steps steps[2];
  uint32_t bad_keys[2][16];  // keys with a non-finite value, from step `look` on
  uint32_t odd[2];           // the work's output is not finite
  uint32_t redo_count;       // works to be done again, so far
  int redo[kRedo];           // their blocks (a ring)
  uint32_t tmem_base;
  int abort;
};
constexpr uint32_t kSmem = OFF_BARS + sizeof(Bars) + 1024;
static_assert(kSmem <= 232448, "shared memory budget");
static_assert(OFF_BARS % 16 == 0 && offsetof(Bars, next) % 16 == 0, "the answer is 16 bytes");

__device__ __forceinline__ int visible(const Work &w, int i) { return min(w.nk, max(0, w.diff + i + 1)); }

// Where the last search ended: sequences b0 .. b0 + 31, the first of whose
// tiles is number `before`.
struct Place {
  int b0, before;
};

// Tiles are numbered through the sequences; the whole warp looks for tile t,
// from the last place on (units of work come in nearly falling order).
__device__ Work find_work(const PrefillParams &p, int t, int h, int lane, Place &at) {
  Work w = {};
  w.h = h;
  bool back = false;
  for (;;) {
    const int b = at.b0 + lane;
    int s = 0, e = 0, ck = 0, cke = 0;
    if (b < p.B) {
      const int cs = __ldg(p.cu_q + b), ce = __ldg(p.cu_q + b + 1);
      ck = __ldg(p.cu_k + b);
      cke = __ldg(p.cu_k + b + 1);
      s = min(max(cs, 0), p.Nq);
      e = min(max(ce, s), p.Nq);
      if (s != cs || e != ce) atomicOr(p.status, MLA_STATUS_BAD_SEQLEN);
    }
    const int mine = ceil_div(e - s, kCtaRows);
    int upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    const int total = __shfl_sync(0xffffffffu, upto, 31);
    if (back) at.before -= total;
    if (t < at.before) {  // (before > 0, so there are sequences before b0)
      at.b0 -= 32;
      back = true;
      continue;
    }
    if (t >= at.before + total) {
      if (at.b0 + 32 >= p.B) return w;
      at.b0 += 32;
      at.before += total;
      back = false;
      continue;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, t < at.before + upto);
    const int who = __ffs(hit) - 1;
    const int part = t - at.before - __shfl_sync(0xffffffffu, upto - mine, who);
    s = __shfl_sync(0xffffffffu, s, who);
    e = __shfl_sync(0xffffffffu, e, who);
    ck = __shfl_sync(0xffffffffu, ck, who);
    cke = __shfl_sync(0xffffffffu, cke, who);
    w.k0 = min(max(ck, 0), p.Nk);
    w.nk = min(max(cke, w.k0), p.Nk) - w.k0;
    if (lane == 0 && (w.k0 != ck || w.k0 + w.nk != cke)) atomicOr(p.status, MLA_STATUS_BAD_SEQLEN);
    // Of an odd number of tiles of 128 rows the first one is alone, not the last,
    // which sees the most keys: a step of one tile takes as long as one of two.
    const int odd = ceil_div(e - s, kRows) & 1, from = max(0, 2 * part - odd) * kRows;
    w.q0 = s + from;
    w.nq = min(part == 0 && odd ? kRows : kCtaRows, e - w.q0);
    w.diff = p.causal ? w.nk - (e - s) + from : p.Nk;
    return w;
  }
}

__device__ __forceinline__ Steps steps_of(const Work &w) {
  Steps s;
  s.masked = kNever;
  s.look = kNever;
#pragma unroll
  for (int t = 0; t < 2; t++) {
    const int first = t * kRows, last = min(w.nq, first + kRows) - 1;
    s.n[t] = last < first ? 0 : ceil_div(visible(w, last), kKeys);
    const int whole = visible(w, first) / kKeys;  // steps that every row of the tile sees whole
    if (whole < s.n[t]) s.masked = min(s.masked, whole);
  }
  s.most = max(s.n[0], s.n[1]);
  return s;
}

// The part of a work unit's steps that falls to split `i` of `splits`.
__device__ __forceinline__ void take_split(Work &w, int i, int splits) {
  const int most = steps_of(w).most;
  const int from = (int)((long long)most * i / splits), to = (int)((long long)most * (i + 1) / splits);
  w.split = i;
  w.k0 += from * kKeys;
  w.nk = max(0, min(w.nk - from * kKeys, (to - from) * kKeys));
  w.diff -= from * kKeys;
}

// A bounded wait; the kernel tells of one that gave up at its end.  (With the
// longer form of a wait in its twenty places: ragged prompts 304 us, not 296.)
template <class P>
__device__ __forceinline__ bool warp_wait_ok(const P &p, Bars *b, uint64_t *bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_wait_small<false, P::poll>(smem_u32(bar), parity, &b->abort, p.wait_ns));
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}

// Pairs of fp32 in one 64-bit register (fma and add of two at a time).
__device__ __forceinline__ uint64_t pack2(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float &a, float &b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Asks the hardware for a block of the grid that has not been launched yet:
// this CTA takes over its work.  The answer arrives at `next_full`.
__device__ __forceinline__ void ask_next(Bars *br) {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // the last answer has been read
  mbar_arrive_expect_tx(smem_u32(&br->next_full), 16);
  asm volatile(
      "clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(
          smem_u32(&br->next)),
      "r"(smem_u32(&br->next_full))
      : "memory");
}

// The block that was taken over, or -1 if there was none.
__device__ __forceinline__ int next_block(Bars *br) {
  int got, x;
  asm volatile(
      "{\n\t.reg .b128 h;\n\t.reg .pred p;\n\t.reg .b32 y, z, w;\n\t"
      "ld.shared.b128 h, [%2];\n\t"
      "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h;\n\t"
      "selp.s32 %0, 1, 0, p;\n\t"
      "mov.s32 %1, 0;\n\t"
      "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%1, y, z, w}, h;\n\t}"
      : "=r"(got), "=r"(x)
      : "r"(smem_u32(&br->next))
      : "memory");
  return got ? x : -1;
}

// Block -> work.  Heads go in groups of eight, so that several CTAs come by the
// same keys and values together (groups of 4, 8, 16, 32: 425, 409, 412 and
// 419 us for 8192 tokens and 32 heads); within a group the last tiles, which see
// the most keys, go first, so that the small ones fill the end.
constexpr int kHeadGroup = 8;
__device__ __forceinline__ Work block_work(const PrefillParams &p, int block, int lane, Place &at) {
  const int split = block % p.splits;
  const int i = block / p.splits;
  const int g = i / (p.tiles * kHeadGroup), in = i % (p.tiles * kHeadGroup);
  const int heads = min(kHeadGroup, p.H - g * kHeadGroup);
  Work w = find_work(p, p.tiles - 1 - in / heads, g * kHeadGroup + in % heads, lane, at);
  if (p.splits > 1 && w.nq > 0) take_split(w, split, p.splits);
  return w;
}

// The load warp asks for the units in their order, each as soon as its place in
// the ring is free.  That decides how early keys are there, and so the time: places
// are freed one by one (all keys, all values of a step at a time: 440 instead of
// 421 us for 8192 tokens), and the whole warp waits while one elected lane asks (a
// loop of one lane takes 500 cycles a unit: 421 instead of 409 us).
template <class P>
__device__ __forceinline__ void load_rows(const P &p, const CUtensorMap *q_map, const CUtensorMap *kn_map,
                                          const CUtensorMap *kp_map, const CUtensorMap *v_map, Bars *br,
                                          uint32_t smem, int lane) {
  const uint64_t pol = policy_evict_normal(), once = policy_evict_first();
  uint32_t u = 0, steps = 0, tiles0 = 0, tiles1 = 0;  // units, steps, tiles so far
  for (uint32_t count = 0;; count++) {
    const uint32_t slot = count & 1;
    if (!warp_wait_ok(p, br, &br->work_full[slot], (count >> 1) & 1)) return;
    const Work w = br->work[slot];
    const Steps st = br->steps[slot];
    __syncwarp();
    if (w.nq == 0) return;
    if (lane == 0) mbar_arrive(smem_u32(&br->work_empty[slot]));
    if (st.most == 0 && lane == 0) mbar_arrive(smem_u32(&br->taken));
#pragma unroll 1
    for (int j = 0; j < st.most; j++) {
      if (j == max(0, st.most - 3) && lane == 0) mbar_arrive(smem_u32(&br->taken));
      const int key = w.k0 + j * kKeys;
      const uint32_t g = steps + j, k_full = smem_u32(&br->k_full[g & 1]), v_full = smem_u32(&br->v_full[g & 1]);
#pragma unroll
      for (int c = 0; c < kUnitsPerStep; c++, u++) {
        if (c == 3 && j == 0) {  // Q, behind the first keys, whose places are free earlier
#pragma unroll 1
          for (int t = 0; t < 2; t++) {
            if ((t == 0 ? st.n[0] : st.n[1]) == 0) continue;
            const uint32_t full = smem_u32(&br->q_full[t]);
            if (!warp_wait_ok(p, br, &br->q_empty[t], ((t == 0 ? tiles0++ : tiles1++) & 1) ^ 1)) return;
            if (elect_one()) {
              mbar_arrive_expect_tx(full, 3 * kUnit);
#pragma unroll 1
              for (int c = 0; c < 3; c++)
                tma_load_3d(smem + (3 * t + c) * kUnit, q_map, full, 64 * c, w.q0 + t * kRows, w.h, once);
            }
            __syncwarp();
          }
        }
        const uint32_t s = u % kUnits, dst = smem + OFF_RING + s * kUnit;
        if (!warp_wait_ok(p, br, &br->empty[s], ((u / kUnits) & 1) ^ 1)) return;
        if (elect_one()) {
          if (c == 0) mbar_arrive_expect_tx(k_full, 3 * kUnit);
          if (c == 3) mbar_arrive_expect_tx(v_full, 2 * kUnit);
          if (c < 3) {
            tma_load_3d(dst, c < 2 ? kn_map : kp_map, k_full, c < 2 ? 64 * c : 0, key, c < 2 ? w.h : 0, pol);
          } else {
            tma_load_3d(dst, v_map, v_full, 0, key + 64 * (c - 3), w.h, pol);
            tma_load_3d(dst + kUnit / 2, v_map, v_full, 64, key + 64 * (c - 3), w.h, pol);
          }
        }
        __syncwarp();
      }
    }
    steps += st.most;
  }
}

// The MMA warp's order of work, gone through by two warps.  A wait on an
// mbarrier by the warp that issues MMAs returns only when its MMAs in flight
// are done (measured: about 130 cycles of idle tensor cores a wait, 4100
// instead of 2560 cycles a step of two tiles); a named barrier does not.  So
// warp 11 (kWaiter) makes the waits, meeting the MMA warp at a named barrier
// before each group of MMAs; the barrier also tells of a wait that gave up.
constexpr uint32_t kMmaBar = 1;

template <bool kWaiter, class P>
__device__ __forceinline__ void mma_sequence(const P &p, Bars *br, uint32_t smem, uint32_t tmem) {
  const int lane = threadIdx.x & 31;
  const uint64_t q_desc = smem_desc_sw128(smem, 16, 1024), k_desc = smem_desc_sw128(smem + OFF_RING, 16, 1024);
  const uint64_t v_desc = smem_desc_sw128(smem + OFF_RING, kUnit / 2, 1024);
  bool ok = true;
  uint32_t base = 0, masked = 0, steps0 = 0, steps1 = 0, works0 = 0, works1 = 0;  // units, masked steps, steps, works so far
  uint32_t steps = 0;  // of both tiles
  // (one wait after the other, each by the whole warp: side by side, a lane for
  // each, five waits took 400 cycles even where all were over)
  auto wait = [&](uint64_t *bar, uint32_t parity) {
    if (kWaiter) ok = ok && warp_wait_ok(p, br, bar, parity);
  };
  auto meet = [&](bool stop = false) { return !bar_red_or(kMmaBar, 64, !ok || stop); };
  // Scores of tile t for step j (units 5j .. 5j + 2).
  auto qk = [&](int t, int j, bool last, bool last_q) {
    if (kWaiter) return;
    tc_fence_after();
    if (elect_one()) {
#pragma unroll
      for (int c = 0; c < 3; c++) {
        const uint32_t s = (base + (uint32_t)j * kUnitsPerStep + c) % kUnits;
        const uint64_t a = q_desc + (uint32_t)(3 * t + c) * (kUnit >> 4), b = k_desc + s * (kUnit >> 4);
#pragma unroll
        for (int k = 0; k < 4; k++)
          mma_ss(tmem + TM_S + t * 128, a + 2 * k, b + 2 * k, IDESC_QK, (c | k) ? 1u : 0u);
        if (c == 2) mma_commit(smem_u32(&br->s_full[t]));
        if (last) mma_commit(smem_u32(&br->empty[s]));
      }
      if (last_q) mma_commit(smem_u32(&br->q_empty[t]));
    }
    __syncwarp();
  };
  // Half c of P V of tile t for step j (unit 5j + 3 + c: 64 keys).
  auto pv = [&](int t, int j, int c, bool last, bool last_o) {
    if (kWaiter) return;
    tc_fence_after();
    if (elect_one()) {
      const uint32_t s = (base + (uint32_t)j * kUnitsPerStep + 3 + c) % kUnits;
      const uint64_t b = v_desc + s * (kUnit >> 4);
#pragma unroll
      for (int k = 0; k < 4; k++)
        mma_ts(tmem + TM_O + t * 128, tmem + TM_S + t * 128 + c * 32 + k * 8, b + k * (2048 >> 4), IDESC_PV,
               (j | c | k) ? 1u : 0u);
      if (c == 1 && last_o) mma_commit(smem_u32(&br->o_done[t]));
      if (last) mma_commit(smem_u32(&br->empty[s]));
    }
    __syncwarp();
  };
  for (uint32_t count = 0;; count++) {
    const uint32_t slot = count & 1;
    wait(&br->work_full[slot], (count >> 1) & 1);
    const bool stop = kWaiter && ok && br->work[slot].nq == 0;
    if (!meet(stop)) return;
    const Steps st = br->steps[slot];
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&br->work_empty[slot]));
    __syncwarp();  // (the barrier below is the whole warp's)
    const int n0 = st.n[0], n1 = st.n[1];
    // While a tile's softmax runs, the tensor cores work on the other tile:
    // its P V, then its next scores (j = -1: the first ones).  One loop for both
    // tiles: the code of all roles has to stay in the instruction cache.
#pragma unroll 1
    for (int i = -2; i < 2 * st.most; i++) {
      const int j = i >> 1, t = i & 1;
      const uint32_t g = steps + (uint32_t)j;
      if (t == 0 && j >= st.look) {
        if (kWaiter) {
          wait(&br->v_full[g & 1], (g >> 1) & 1);
          if (ok && elect_one()) mbar_arrive(smem_u32(&br->v_look));
          wait(&br->v_ok, masked & 1);
        }
        masked++;
      }
      const int n = t == 0 ? n0 : n1, other = t == 0 ? n1 : n0;
      if (j >= n) continue;
      const uint32_t work_parity = (t == 0 ? works0 : works1) & 1, step = (t == 0 ? steps0 : steps1) + j;
      const bool first = t == 0 || j >= other, first_k = t == 0 || j + 1 >= other;
      const bool last = t == 1 || j >= other, last_k = t == 1 || j + 1 >= other;
      if (j >= 0) {
        if (first) wait(&br->v_full[g & 1], (g >> 1) & 1);
        if (j == 0) wait(&br->o_free[t], work_parity ^ 1);  // the output of the unit of work before has been read
#pragma unroll
        for (int c = 0; c < 2; c++) {
          wait(&br->p_full[t][c], step & 1);
          if (!meet()) return;
          pv(t, j, c, last, j + 1 == n);
        }
      }
      if (j + 1 < n) {
        if (first_k || j < 0) {
          if (first_k) wait(&br->k_full[(g + 1) & 1], ((g + 1) >> 1) & 1);
          if (j < 0) wait(&br->q_full[t], work_parity);
          if (!meet()) return;
        }
        qk(t, j + 1, last_k, j + 2 == n);
      }
    }
    base += (uint32_t)st.most * kUnitsPerStep;
    steps += st.most;
    steps0 += n0;
    steps1 += n1;
    works0 += n0 > 0 ? 1 : 0;
    works1 += n1 > 0 ? 1 : 0;
  }
}

// The whole warp looks through the values of one unit of work, from step `look`
// on; base: the unit of the ring that its first step begins with.
template <class P>
__device__ __forceinline__ bool check_values(const P &p, Bars *br, uint8_t *ring, const Steps &st,
                                             uint32_t slot, uint32_t base, uint32_t &looks, int lane) {
  for (int j = st.look; j < st.most; j++) {
    if (!warp_wait_ok(p, br, &br->v_look, looks++ & 1)) return false;
    bool patched = false;
    for (int c = 0; c < 2; c++) {
      const uint32_t u = base + (uint32_t)j * kUnitsPerStep + 3 + c, s = u % kUnits, g = u / kUnitsPerStep;
      if (!warp_wait_ok(p, br, &br->v_full[g & 1], (g >> 1) & 1)) return false;
      uint8_t *unit = ring + s * kUnit;
      // x * 0 summed up stays 0, unless some x is not finite: then it is nan
      uint32_t sum[4] = {0u, 0u, 0u, 0u};
#pragma unroll 1
      for (int i = lane; i < (int)(kUnit / 16); i += 32 * 8) {
        uint4 v[8];
#pragma unroll
        for (int k = 0; k < 8; k++) v[k] = *reinterpret_cast<const uint4 *>(unit + (i + 32 * k) * 16);
#pragma unroll
        for (int k = 0; k < 8; k++) {
          const uint32_t x[4] = {v[k].x, v[k].y, v[k].z, v[k].w};
#pragma unroll
          for (int e = 0; e < 4; e++) asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(sum[e]) : "r"(x[e]), "r"(0u));
        }
      }
      bool some = false;
#pragma unroll
      for (int e = 0; e < 4; e++) some |= (sum[e] & 0x7FFF7FFFu) != 0;
      if (!some) continue;
#pragma unroll 1
      for (int i = lane; i < (int)(kUnit / 16); i += 32) {  // (this lane's part again)
        uint32_t x[4];
        bool bad = false;
#pragma unroll
        for (int e = 0; e < 4; e++) {
          x[e] = reinterpret_cast<const uint32_t *>(unit + i * 16)[e];
          // a bf16 is not finite when its eight exponent bits are all set
          if ((x[e] & 0x7F80u) == 0x7F80u) {
            x[e] &= 0xFFFF0000u;
            bad = true;
          }
          if ((x[e] & 0x7F800000u) == 0x7F800000u) {
            x[e] &= 0x0000FFFFu;
            bad = true;
          }
        }
        if (!bad) continue;
        *reinterpret_cast<uint4 *>(unit + i * 16) = make_uint4(x[0], x[1], x[2], x[3]);
        const int key = (j - st.look) * kKeys + c * 64 + ((i * 16) % (int)(kUnit / 2)) / 128;
        if (key < 512) atomicOr(&br->bad_keys[slot][key >> 5], 1u << (key & 31));
        patched = true;
      }
    }
    if (patched) fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&br->v_ok));
  }
  return true;
}

// The scheduling warp: hands out the units of work.  Blocks of the grid come one
// after the other.  When there are no more, or many units wait to be done again
// (never more than their ring holds: two are under way beside this), all that
// is under way is let finish, and they are, with this warp looking through their
// values.
template <class P>
__device__ __forceinline__ void schedule(const P &p, Bars *br, uint8_t *ring, int lane) {
  uint32_t asked = 0, count = 0, redone = 0, base = 0, looks = 0;
  Place place = {0, 0};
  // the slot that unit of work number n gets is free
  auto slot_free = [&](uint32_t n) {
    return warp_wait_ok(p, br, &br->work_empty[n & 1], ((n >> 1) & 1) ^ 1);
  };
  auto tell = [&](const Work &w, const Steps &st) {
    const uint32_t slot = count & 1;
    if (!slot_free(count)) return false;
    if (lane < 16) br->bad_keys[slot][lane] = 0;
    if (lane == 0) {
      br->work[slot] = w;
      br->steps[slot] = st;
      br->odd[slot] = 0;
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&br->work_full[slot]));
    count++;
    return true;
  };
  int block = blockIdx.x;
  for (;;) {
    const uint32_t waiting = __shfl_sync(0xffffffffu, *(volatile uint32_t *)&br->redo_count, 0) - redone;
    const bool redo = block < 0 || waiting >= kRedo / 2;
    int now = block;
    if (redo) {
      if (!slot_free(count) || !slot_free(count + 1)) return;
      if (*(volatile uint32_t *)&br->redo_count == redone) break;
      now = *(volatile int *)&br->redo[redone++ % kRedo];
    }
    __syncwarp();
    Work w = block_work(p, now, lane, place);
    w.block = now;
    bool ok = true;
    if (w.nq > 0) {
      Steps st = steps_of(w);
      if (redo) st.look = st.masked;
      const uint32_t slot = count & 1;
      ok = tell(w, st);
      if (ok && redo) ok = check_values(p, br, ring, st, slot, base, looks, lane);
      base += (uint32_t)st.most * kUnitsPerStep;
      // The next block is taken over when this one's last loads begin: taken
      // earlier, blocks are shared out unevenly (8192 tokens, two units ahead:
      // 545 us).
      ok = ok && warp_wait_ok(p, br, &br->taken, (count - 1) & 1);
    }
    if (!redo && ok) {
      if (lane == 0) ask_next(br);
      // (also after a wait that gave up: the answer has to land before the CTA ends)
      const bool told = warp_wait_ok(p, br, &br->next_full, asked++ & 1);
      ok = ok && told;
      block = told ? next_block(br) : -1;
      __syncwarp();
    }
    if (!ok) return;
  }
  tell(Work{}, Steps{});
}

// One row a thread: the softmax of tile t over the steps of one unit of work,
// then its output.  done, works: the tile's steps and its units of work with
// steps before this one.
template <class P>
__device__ __forceinline__ bool softmax_work(const P &p, Bars *br, uint32_t tmem, int slot, int t,
                                             uint32_t done, uint32_t works) {
  const int warp = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
  const int i = t * kRows + warp * 32 + lane;  // the CTA's row
  const int seen = visible(br->work[slot], i);
  const uint32_t lanes = (uint32_t)(warp * 32) << 16;
  const uint32_t ts = tmem + TM_S + t * 128 + lanes, to = tmem + TM_O + t * 128 + lanes;
  const int n = br->steps[slot].n[t];
  float m = -INFINITY;  // reference, in score units
  uint64_t l0 = 0, l1 = 0;
  const uint64_t c2 = pack2(p.scale_log2, p.scale_log2);
  const int low = __shfl_sync(0xffffffffu, seen, 0);  // the fewest keys of the warp's rows
  for (int j = 0; j < n; j++) {
    if (!warp_wait_ok(p, br, &br->s_full[t], (done + j) & 1)) return false;
    tc_fence_after();
    uint32_t s[4][32];
#pragma unroll
    for (int c = 0; c < 4; c++) tmem_ld32(ts + 32 * c, s[c]);
    tmem_wait_ld();
    if (low < (j + 1) * kKeys) {  // some row sees only a part of these keys
#pragma unroll
      for (int c = 0; c < 4; c++) {
        const int here = seen - j * kKeys - 32 * c;
        if (low - j * kKeys - 32 * c < 32) {  // (the same for the whole warp)
          const uint32_t keep = here <= 0 ? 0u : here >= 32 ? 0xFFFFFFFFu : (1u << here) - 1u;
#pragma unroll
          for (int e = 0; e < 32; e++)
            if (!((keep >> e) & 1u)) s[c][e] = 0xFF800000u;
        }
      }
    }
    float mx[4];
#pragma unroll
    for (int c = 0; c < 4; c++) {
      mx[c] = __uint_as_float(s[c][0]);
#pragma unroll
      for (int e = 1; e < 31; e += 2) mx[c] = max3(mx[c], __uint_as_float(s[c][e]), __uint_as_float(s[c][e + 1]));
      mx[c] = fmaxf(mx[c], __uint_as_float(s[c][31]));
    }
    const float top = fmaxf(max3(mx[0], mx[1], mx[2]), mx[3]);
    const bool move = (top - m) * p.scale_log2 > kMoveAt;  // (-inf - -inf is nan: no move)
    if (__any_sync(0xffffffffu, move)) {
      const float alpha = move ? ex2((m - top) * p.scale_log2) : 1.f;
      if (move) m = top;
      if (j > 0) {  // (the P V before has been added: its MMAs came before this step's scores)
        __syncwarp();  // (as below)
        const uint64_t a2 = pack2(alpha, alpha);
        asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(l0) : "l"(a2));
        asm("mul.rn.f32x2 %0, %0, %1;" : "+l"(l1) : "l"(a2));
#pragma unroll 1
        for (int c = 0; c < 8; c++) {
          uint32_t o[16];
          asm volatile(
              "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
              "%14, %15}, [%16];"
              : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3]), "=r"(o[4]), "=r"(o[5]), "=r"(o[6]), "=r"(o[7]),
                "=r"(o[8]), "=r"(o[9]), "=r"(o[10]), "=r"(o[11]), "=r"(o[12]), "=r"(o[13]), "=r"(o[14]), "=r"(o[15])
              : "r"(to + 16 * c)
              : "memory");
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 16; e++) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
          asm volatile(
              "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
              "%14, %15, %16};" ::"r"(to + 16 * c),
              "r"(o[0]), "r"(o[1]), "r"(o[2]), "r"(o[3]), "r"(o[4]), "r"(o[5]), "r"(o[6]), "r"(o[7]), "r"(o[8]),
              "r"(o[9]), "r"(o[10]), "r"(o[11]), "r"(o[12]), "r"(o[13]), "r"(o[14]), "r"(o[15])
              : "memory");
        }
      }
    }
    const float mc = m == -INFINITY ? 0.f : m * p.scale_log2;
    const uint64_t nm2 = pack2(-mc, -mc);
#pragma unroll
    for (int half = 0; half < 2; half++) {
      uint32_t pw[32];
#pragma unroll
      for (int e = 0; e < 32; e++) {
        const int c = 2 * half + (e >> 4), x = 2 * (e & 15);
        const uint64_t y = fma2(pack2(__uint_as_float(s[c][x]), __uint_as_float(s[c][x + 1])), c2, nm2);
        float a, b;
        unpack2(y, a, b);
        a = ex2(a);
        b = ex2(b);
        if (e & 1) l1 = add2(l1, pack2(a, b)); else l0 = add2(l0, pack2(a, b));
        __nv_bfloat162 h2 = __floats2bfloat162_rn(a, b);
        pw[e] = *reinterpret_cast<uint32_t *>(&h2);
      }
      tmem_st32(ts + 32 * half, pw);
      tmem_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&br->p_full[t][half]));
      __syncwarp();  // (as below)
    }
  }

  float la, lb, lc, ld;
  unpack2(l0, la, lb);
  unpack2(l1, lc, ld);
  const float l = (la + lb) + (lc + ld);
  // (the work is read again here, and above only what the steps need: with 28
  // bytes spilled in the loop ragged prompts took 319 us instead of 303)
  const Work w = br->work[slot];
  const Steps st = br->steps[slot];
  const bool live = i < w.nq, none = seen == 0;
  if (n > 0) {
    if (!warp_wait_ok(p, br, &br->o_done[t], works & 1)) return false;
    tc_fence_after();
  }
  // l = 0: every score of the row is -inf (0 / 0: nan, unless another part of its keys has weight)
  const float inv = l != 0.f || p.splits == 1 ? 1.f / l : 0.f;
  // have the steps that were looked through non-finite values?
  const uint32_t *bad_keys = br->bad_keys[slot];
  bool bad = false;
  if (n > 0 && st.look < st.most)
    for (int k = 0; k < 16; k++) bad |= *(volatile const uint32_t *)&bad_keys[k] != 0;
  uint64_t zero = 0;  // (two fp32) becomes nan if an output is not finite
  const uint64_t inv2 = pack2(none ? 0.f : inv, none ? 0.f : inv);
  const size_t row = w.q0 + i;
  __nv_bfloat16 *dst = p.out + (row * p.H + w.h) * kDv;
  float *part = p.part_o + ((w.split * (size_t)p.Nq + row) * p.H + w.h) * kDv;
#pragma unroll 1
  for (int c = 0; c < 4; c++) {
    // Loads from and stores to tensor memory are the whole warp's: its lanes
    // have to meet again behind every branch that only some of them take.
    __syncwarp();
    uint32_t o[32];
    if (n > 0) {
      tmem_ld32(to + 32 * c, o);
      tmem_wait_ld();
    }
    if (!live) continue;
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
      const uint64_t x = pack2(__uint_as_float(o[e]), __uint_as_float(o[e + 1]));
      zero = fma2(x, 0ull, zero);
      uint64_t y;
      asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(y) : "l"(x), "l"(inv2));
      float a, b;
      unpack2(y, a, b);
      o[e] = none ? 0u : __float_as_uint(a);
      o[e + 1] = none ? 0u : __float_as_uint(b);
    }
    if (p.splits > 1) {
#pragma unroll
      for (int k = 0; k < 4; k++) {
        const uint32_t a8[8] = {o[8 * k],     o[8 * k + 1], o[8 * k + 2], o[8 * k + 3],
                                o[8 * k + 4], o[8 * k + 5], o[8 * k + 6], o[8 * k + 7]};
        st_global_v8(part + 32 * c + 8 * k, a8);
      }
      continue;
    }
    uint32_t r[16];
#pragma unroll
    for (int e = 0; e < 16; e++) {
      __nv_bfloat162 h2 = __floats2bfloat162_rn(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1]));
      r[e] = *reinterpret_cast<uint32_t *>(&h2);
    }
    if (p.out_v8) {
      const uint32_t a8[8] = {r[0], r[1], r[2], r[3], r[4], r[5], r[6], r[7]};
      const uint32_t b8[8] = {r[8], r[9], r[10], r[11], r[12], r[13], r[14], r[15]};
      st_global_v8(dst + 32 * c, a8);
      st_global_v8(dst + 32 * c + 16, b8);
    } else {
#pragma unroll
      for (int k = 0; k < 4; k++)
        reinterpret_cast<uint4 *>(dst + 32 * c)[k] = make_uint4(r[4 * k], r[4 * k + 1], r[4 * k + 2], r[4 * k + 3]);
    }
  }
  float zero0, zero1;
  unpack2(zero, zero0, zero1);
  if (n > 0) {  // the MMA warp may start the next unit's output
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(smem_u32(&br->o_free[t]));
  }
  // once more, with a look at the values
  if (st.masked < st.most && st.look == kNever && __any_sync(0xffffffffu, n > 0 && live && !none && (zero0 != 0.f || zero1 != 0.f))) {
    if (lane == 0 && atomicExch(&br->odd[slot], 1u) == 0) br->redo[atomicAdd(&br->redo_count, 1u) % kRedo] = w.block;
  }
  if (live && bad) {  // rare: add the non-finite values of the keys that this row sees
#pragma unroll 1
    for (int k = 0; k < 512; k++) {
      if (!((*(volatile const uint32_t *)&bad_keys[k >> 5] >> (k & 31)) & 1u)) continue;
      const int key = st.look * kKeys + k;
      if (key >= seen) continue;
      const __nv_bfloat16 *vr = p.v + (size_t)(w.k0 + key) * p.v_tok + (size_t)w.h * p.v_head;
#pragma unroll 1
      for (int d = 0; d < kDv; d++) {
        const float x = __bfloat162float(vr[d]);
        if (fabsf(x) < INFINITY) continue;
        if (p.splits > 1) part[d] += x;
        else dst[d] = __float2bfloat16_rn(__bfloat162float(dst[d]) + x);
      }
    }
  }
  if (live) {
    const float lse = none ? -INFINITY : m * p.scale + logf(l);
    if (p.splits > 1) p.part_lse[((size_t)w.split * p.H + w.h) * p.Nq + row] = lse;
    else p.lse[(size_t)w.h * p.Nq + row] = lse;
  }
  return true;
}

template <class P>
__device__ __forceinline__ void softmax_rows(const P &p, Bars *br, uint32_t tmem, int t) {
  uint32_t done = 0, works = 0;
  for (uint32_t count = 0;; count++) {
    const uint32_t slot = count & 1;
    if (!warp_wait_ok(p, br, &br->work_full[slot], (count >> 1) & 1)) return;
    if (br->work[slot].nq == 0) return;
    if (!softmax_work(p, br, tmem, (int)slot, t, done, works)) return;
    const int n = br->steps[slot].n[t];
    done += n;
    works += n > 0 ? 1 : 0;
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(smem_u32(&br->work_empty[slot]));
  }
}

// Splits joined: four warps a row and head, every fourth part each, four values
// a lane.  All loads go out at once (a warp that took eight parts at a time after
// it had found its row needed 11 us for 1600 rows of 19 parts).
constexpr int kJoinWarps = 4;
__global__ void __launch_bounds__(32 * kJoinWarps) prefill_join_kernel(PrefillParams p) {
  __shared__ float4 sums[kJoinWarps][32];
  grid_dep_trigger();
  grid_dep_wait();  // (a programmatic dependent of the kernel below)
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long i = blockIdx.x;
  const int row = (int)(i / p.H), h = (int)(i % p.H);
  const float *part = p.part_o + (size_t)i * kDv + 4 * lane;
  const size_t next = (size_t)p.Nq * p.H * kDv;
  float4 v[kMaxSplits / kJoinWarps];
#pragma unroll
  for (int k = 0; k < kMaxSplits / kJoinWarps; k++) {
    const int s = warp + kJoinWarps * k;
    v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
    if (s < p.splits) v[k] = *reinterpret_cast<const float4 *>(part + s * next);
  }
  const float mine = lane < p.splits ? p.part_lse[((size_t)lane * p.H + h) * p.Nq + row] : -INFINITY;
  int lo = 0, hi = p.B;  // the last sequence that starts at or before the row
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(p.cu_q + mid) <= row) lo = mid; else hi = mid;
  }
  const bool live = row >= __ldg(p.cu_q + lo) && row < __ldg(p.cu_q + lo + 1);  // else: of no sequence
  // (a nan among them has to stay one: not through fmaxf alone)
  float m = mine;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float weight = mine == -INFINITY ? 0.f : expf(mine - m);
  float sum = weight;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
  for (int k = 0; k < kMaxSplits / kJoinWarps; k++) {
    const int s = warp + kJoinWarps * k;
    const float ws = __shfl_sync(0xffffffffu, weight, s);
    if (s >= p.splits) continue;
    acc.x += ws * v[k].x;  // (a part without keys has weight 0 and finite values)
    acc.y += ws * v[k].y;
    acc.z += ws * v[k].z;
    acc.w += ws * v[k].w;
  }
  sums[warp][lane] = acc;
  __syncthreads();
  if (warp != 0 || !live) return;
#pragma unroll
  for (int k = 1; k < kJoinWarps; k++) {
    const float4 o = sums[k][lane];
    acc.x += o.x;
    acc.y += o.y;
    acc.z += o.z;
    acc.w += o.w;
  }
  const bool none = sum == 0.f;
  float inv = none ? 0.f : 1.f / sum;
  if (none) {  // no key, or all scores -inf?
    const int s = min(max(__ldg(p.cu_q + lo), 0), p.Nq), e = min(max(__ldg(p.cu_q + lo + 1), s), p.Nq);
    const int k0 = min(max(__ldg(p.cu_k + lo), 0), p.Nk), nk = min(max(__ldg(p.cu_k + lo + 1), k0), p.Nk) - k0;
    if ((p.causal ? min(nk, nk - (e - s) + row - s + 1) : nk) > 0) inv = INFINITY;  // 0 / 0
  }
  __nv_bfloat162 a = __floats2bfloat162_rn(acc.x * inv, acc.y * inv), b = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
  uint2 r = make_uint2(*reinterpret_cast<uint32_t *>(&a), *reinterpret_cast<uint32_t *>(&b));
  *reinterpret_cast<uint2 *>(p.out + (size_t)i * kDv + 4 * lane) = r;
  if (lane == 0) p.lse[(size_t)h * p.Nq + row] = none ? -INFINITY : m + logf(sum);
}

template <bool kPoll>
__global__ void __launch_bounds__(kThreads, 1)
    prefill_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap kn_map,
                   const __grid_constant__ CUtensorMap kp_map, const __grid_constant__ CUtensorMap v_map,
                   Limited<kPoll> p) {
  grid_dep_trigger();
  extern __shared__ uint8_t smem_raw[];
  uint8_t *base = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  Bars *br = reinterpret_cast<Bars *>(base + OFF_BARS);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (warp == 0) {
    tmem_alloc(smem_u32(&br->tmem_base), 512);
    tmem_relinquish();
  }
  if (threadIdx.x == 32) {
    for (int s = 0; s < kUnits; s++) mbar_init(smem_u32(&br->empty[s]), 1);
    for (int t = 0; t < 2; t++) {
      mbar_init(smem_u32(&br->k_full[t]), 1);
      mbar_init(smem_u32(&br->v_full[t]), 1);
      mbar_init(smem_u32(&br->q_empty[t]), 1);
      mbar_init(smem_u32(&br->work_full[t]), 1);
      mbar_init(smem_u32(&br->work_empty[t]), 11);  // softmax, MMA, waiting and load warps
      mbar_init(smem_u32(&br->q_full[t]), 1);
      mbar_init(smem_u32(&br->s_full[t]), 1);
      mbar_init(smem_u32(&br->p_full[t][0]), 4);
      mbar_init(smem_u32(&br->p_full[t][1]), 4);
      mbar_init(smem_u32(&br->o_done[t]), 1);
      mbar_init(smem_u32(&br->o_free[t]), 4);
    }
    mbar_init(smem_u32(&br->v_look), 1);
    mbar_init(smem_u32(&br->v_ok), 1);
    mbar_init(smem_u32(&br->next_full), 1);
    mbar_init(smem_u32(&br->taken), 1);
    br->redo_count = 0;
    br->abort = 0;
    fence_mbar_init_cluster();
  }
  if (threadIdx.x == 9 * 32) {
    prefetch_tensormap(&q_map);
    prefetch_tensormap(&kn_map);
    prefetch_tensormap(&kp_map);
    prefetch_tensormap(&v_map);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_dep_wait();  // nothing of the caller's is read or written before the kernel in front has ended
  const uint32_t tmem = br->tmem_base, smem = smem_u32(base);
  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    softmax_rows(p, br, tmem, warp >> 2);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == 8) {
      mma_sequence<false>(p, br, smem, tmem);
    } else if (warp == 9) {
      load_rows(p, &q_map, &kn_map, &kp_map, &v_map, br, smem, lane);
    } else if (warp == 10) {
      schedule(p, br, base + OFF_RING, lane);
    } else {
      mma_sequence<true>(p, br, smem, tmem);
    }
  }
  __syncthreads();
  if (threadIdx.x == 0 && *(volatile int *)&br->abort) atomicOr(p.status, MLA_STATUS_WAIT_TIMEOUT);
  if (*(volatile int *)&br->abort) {  // a wait gave up: let copies or MMAs still in flight land before the CTA exits
    const uint64_t t0 = globaltimer();
    while (globaltimer() - t0 < 2000000ull) {
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

int fail(int code, const char *msg) {
  set_last_error(msg);
  return code;
}

}  // namespace
}  // namespace mla

namespace mla {
namespace {

// 256 rows a tile: at most one tile that is not full for each sequence.
long long tiles_of(int B, int Nq) { return Nq < B ? Nq : (Nq - B) / kCtaRows + (long long)B; }

// Few tiles over long keys: each tile's keys are split into s parts, whose
// outputs are joined.  In steps of 128 keys (2 us), a part costs its steps and
// three more for its beginning and end, for every round of the 152 SMs, and the
// join one step and one for every 20000 rows of parts.  The s with the least cost
// is taken if it saves a tenth; a part has at least four steps (of a sequence of
// average length).  Split by it against whole: 20 queries on 8200 keys, 3
// sequences, 32 heads 78 / 98 us; 16 on 8000, 8 sequences, 20 heads 134 / 184 us.
constexpr int kSms = 152;
int splits_of(int B, int H, int Nq, int Nk) {
  const long long works = tiles_of(B, Nq) * H;
  if (B < 1 || works < 1 || works > 2 * kSms) return 1;
  const int steps = ceil_div(Nk / B, kKeys), most = steps / 4 < kMaxSplits ? steps / 4 : kMaxSplits;
  int best = 1;
  float least = 0.9f * (float)((works + kSms - 1) / kSms * (steps + 3));
  for (int s = 2; s <= most; s++) {
    const long long rounds = (works * s + kSms - 1) / kSms;
    const float cost = (float)(rounds * (ceil_div(steps, s) + 3)) + 1.f + (float)s * (float)Nq * (float)H / 20000.f;
    if (cost < least) {
      least = cost;
      best = s;
    }
  }
  return best;
}

size_t lse_bytes(int splits, int H, int Nq) { return ((size_t)splits * H * Nq * 4 + 255) / 256 * 256; }

}  // namespace
}  // namespace mla

size_t mla_prefill_workspace_bytes(int B, int H, int Nq, int Nk) {
  using namespace mla;
  if (B < 0 || H < 1 || H > MLA_MAX_HEADS || Nq < 0 || Nk < 0) return 0;
  const int s = splits_of(B, H, Nq, Nk);
  return s == 1 ? 0 : lse_bytes(s, H, Nq) + (size_t)s * Nq * H * kDv * 4;
}

int mla_prefill(const void *q, int64_t q_tok, int64_t q_head, const void *k_nope, int64_t k_tok, int64_t k_head,
                const void *k_pe, int64_t pe_tok, const void *v, int64_t v_tok, int64_t v_head,
                const int32_t *cu_seqlens_q, const int32_t *cu_seqlens_k, int B, int H, int Nq, int Nk,
                float softmax_scale, int causal, void *workspace, size_t workspace_bytes, void *out, float *lse,
                mla_stream_t stream) {
  using namespace mla;
  if (B < 0 || Nq < 0 || Nk < 0) return fail(MLA_ERR_INVALID_ARG, "B, Nq and Nk must be >= 0");
  // (2^26 keys are a second's work for one tile, under the limit of its waits)
  if (B > (1 << 20) || Nq > (1 << 30) || Nk > (1 << 26))
    return fail(MLA_ERR_UNSUPPORTED, "B must be at most 2^20, Nq at most 2^30, Nk at most 2^26");
  if (H < 1 || H > MLA_MAX_HEADS) return fail(MLA_ERR_INVALID_ARG, "H must be in [1, 128]");
  if (causal != 0 && causal != 1) return fail(MLA_ERR_INVALID_ARG, "causal must be 0 or 1");
  if (!(softmax_scale > 0.f) || softmax_scale > 2.0e38f)  // (log2 e times it is finite too)
    return fail(MLA_ERR_INVALID_ARG, "softmax_scale must be > 0 and at most 2e38");
  for (int64_t s : {q_tok, q_head, k_tok, k_head, pe_tok, v_tok, v_head})
    if (s % 8) return fail(MLA_ERR_INVALID_ARG, "strides must be multiples of 8 elements");
  if ((Nq > 1 && q_tok < kHead) || (H > 1 && q_head < kHead) || (Nk > 1 && (k_tok < kNope || v_tok < kDv || pe_tok < 64)) ||
      (H > 1 && (k_head < kNope || v_head < kDv)))
    return fail(MLA_ERR_INVALID_ARG, "strides must be at least a row's width");
  if (B == 0 || Nq == 0) {
    set_last_error("");
    return MLA_OK;
  }
  if (!q || !cu_seqlens_q || !cu_seqlens_k || !out || !lse || (Nk > 0 && (!k_nope || !k_pe || !v)))
    return fail(MLA_ERR_INVALID_ARG, "null pointer");
  auto al = [](const void *p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; };
  if (!al(q, 16) || !al(k_nope, 16) || !al(k_pe, 16) || !al(v, 16) || !al(out, 16))
    return fail(MLA_ERR_INVALID_ARG, "q, k_nope, k_pe, v and out must be 16-byte aligned");
  if (!al(cu_seqlens_q, 4) || !al(cu_seqlens_k, 4) || !al(lse, 4))
    return fail(MLA_ERR_INVALID_ARG, "int32 and fp32 arrays must be 4-byte aligned");
  const size_t need = mla_prefill_workspace_bytes(B, H, Nq, Nk);
  if (need > 0 && (!workspace || workspace_bytes < need))
    return fail(MLA_ERR_WORKSPACE, "workspace smaller than mla_prefill_workspace_bytes(B, H, Nq, Nk)");
  if (need > 0 && !al(workspace, 256)) return fail(MLA_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  const long long tiles = tiles_of(B, Nq);
  const int splits = splits_of(B, H, Nq, Nk);
  if (tiles * H * splits > 0x7FFFFFFFll) return fail(MLA_ERR_UNSUPPORTED, "too many query tiles");
  CUtensorMap q_map, kn_map, kp_map, v_map;
  bool ok = make_map_3d(&q_map, q, kHead, Nq, H, q_tok, q_head, kRows, 1);
  if (Nk > 0) {
    ok = ok && make_map_3d(&kn_map, k_nope, kNope, Nk, H, k_tok, k_head, kKeys, 1) &&
         make_map_3d(&kp_map, k_pe, 64, Nk, 1, pe_tok, 64, kKeys, 1) &&
         make_map_3d(&v_map, v, kDv, Nk, H, v_tok, v_head, kKeys / 2, 1);
  } else {
    kn_map = kp_map = v_map = q_map;  // no step reads them
  }
  if (!ok) return fail(MLA_ERR_CUDA, "cuTensorMapEncodeTiled failed");
  Limited<false> p;
  p.cu_q = cu_seqlens_q;
  p.cu_k = cu_seqlens_k;
  p.v = static_cast<const __nv_bfloat16 *>(v);
  p.out = static_cast<__nv_bfloat16 *>(out);
  p.lse = lse;
  if (status_word(&p.status) != MLA_OK) return MLA_ERR_CUDA;
  p.v_tok = v_tok;
  p.v_head = v_head;
  p.B = B;
  p.H = H;
  p.Nq = Nq;
  p.Nk = Nk;
  p.tiles = (int)tiles;
  p.splits = splits;
  p.part_lse = static_cast<float *>(workspace);
  p.part_o = splits > 1 ? p.part_lse + lse_bytes(splits, H, Nq) / 4 : nullptr;
  p.causal = causal;
  p.out_v8 = al(out, 32) ? 1 : 0;
  p.scale = softmax_scale;
  p.scale_log2 = softmax_scale * LOG2E;
  const unsigned long long limit = wait_limit_ns(), most = 4000000000ull;  // (a 32-bit clock)
  p.wait_ns = (uint32_t)(limit < most ? limit : most);
  auto launch = [&](auto *kernel, const auto &params) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
    return e != cudaSuccess ? e
                            : launch_dependent(kernel, (unsigned)(tiles * H * splits), kThreads, kSmem,
                                               (cudaStream_t)stream, q_map, kn_map, kp_map, v_map, params);
  };
  const PrefillParams &common = p;
  cudaError_t e = limit < ptx::kShortWaitNs ? launch(&prefill_kernel<true>, Limited<true>{common})
                                            : launch(&prefill_kernel<false>, p);
  if (e == cudaSuccess && splits > 1)
    e = launch_dependent(prefill_join_kernel, (unsigned)((long long)Nq * H), 32 * kJoinWarps, 0, (cudaStream_t)stream,
                         common);
  if (e != cudaSuccess) return fail(MLA_ERR_CUDA, cudaGetErrorString(e));
  set_last_error("");
  return MLA_OK;
}

// Attention of the items of a batch that shares prefixes (see SharedItem), on
// the tensor cores.
//
// A group's query rows are packed into MMA tiles of 128 whatever sequence they
// belong to, so that a tile of keys multiplies 128 rows also where a sequence has
// 16; own tokens have only their sequence's rows.  Both kinds of items lie on one
// line that is cut into equal parts, so the prefix's tiles, which L2 delivers and the tensor
// cores bound, and the own tokens', which come from HBM, share the workers.
//
// One worker is a cluster of two CTAs, split by stage as the decode kernel's (a
// 128 x 512 fp32 accumulator fills one SM's tensor memory): rank 0 computes S =
// Q K^T and the softmax, rank 1 accumulates O += P V; P goes from one to the
// other through a small ring in L2.  All results are fp32 partials, normalised,
// with a base-2 log-sum-exp: another kernel joins prefix and own parts.
//
// 64 sequences of 128 heads on 16384 shared tokens: 220 us in all for 301 GFLOP (154 us at the
// measured bf16 rate, which would keep both SMs' tensor cores busy).  A tile takes 0.78 us, bound by rank 0's MMAs
// (36 of 38 cycles, 0.7 us); the start and the end of an item of 128 rows take 5.8 us.
//
// FP8 rows are multiplied as bf16 values that the widening kernel has made.  With one
// scale the codes themselves (exact; the scale multiplies scores and results).  With a scale
// for each 128 values a product of code and scale does not fit 8 bits, and a log-sum-exp over few
// keys shows it: keys are sums of two bf16 values (16 bits), so rank 0 makes twice the products
// of a latent, from a second stage a tile: 117 us of 146 for 48 sequences of four tokens and 64 heads on three
// prefixes of up to 5000, where codes with one scale take 80 of 104.  (One bf16 value: log-sum-exps off by 1e-4 of
// themselves instead of 1e-6.)  Values are the first of the two: P is bf16 too, and its
// rounding of the same size.
//
// Rows behind an item's last key, in its last page, and pages outside the pool never
// reach a result: their scores are replaced by -inf, and rank 1 clears their
// values in shared memory before the MMA reads them (0 * nan is nan).  A query of nan or a score of
// +inf makes its row's sum nan, which no comparison may take for the 0 of a row without keys.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "dependent.cuh"
#include "pairs_f32.cuh"
#include "ptx.cuh"
#include "shared_prefix.cuh"
#include "tma_map.cuh"

namespace mla {
namespace {

using namespace ptx;

constexpr int kThreads = 384;
constexpr int kSoftWarps = 8;
constexpr int kStages = 3;
constexpr uint32_t kBlk = PAGE * 128;       // 64 tokens x 64 dims, 128-byte swizzle
constexpr uint32_t kStage0 = 9 * kBlk;      // rank 0: one page of keys
constexpr uint32_t kStage1 = 8 * kBlk;      // rank 1: one page of values
constexpr uint32_t kPBytes = M_TILE * 128;  // P tile: 128 rows x 64 tokens bf16
constexpr int kValidRing = 8;
constexpr int kPublishBatch = 4;
constexpr uint32_t kFreeBatch = 4;          // P slots that rank 0 waits for at once
constexpr int kSplit = 5;                   // rank 0: blocks of a page's first box
// The reference of a row moves when a maximum exceeds it by 2^32: a rescale of O takes
// longer than a tile, and what it guards against, fp32 and bf16 running out of range, is
// 2^64 further off (8 instead of 32: 238 against 227 us for 64 sequences of 128 heads on
// 16384 shared tokens).
constexpr float kRescale = 32.0f;           // log2 units

constexpr uint32_t OFF_RCV_P = kStages * kStage1;        // rank 1: two P tiles
constexpr uint32_t OFF_BARS = OFF_RCV_P + 2 * kPBytes;
constexpr uint32_t TM_Q = 0, TM_S = 320, TM_O = 0, TM_COLS = 512;
constexpr uint32_t IDESC_QK = idesc_bf16_f32(128, 64, false, false);
constexpr uint32_t IDESC_PV = idesc_bf16_f32(128, 256, false, true);

struct Bars {
  uint64_t kv_full[kStages], kv_empty[kStages];      // rank 0: blocks 0-4 of a stage; rank 1: whole stages
  uint64_t kv_full_b[kStages], kv_empty_b[kStages];  // rank 0: blocks 5-8
  uint64_t s_full[2], s_free[2];
  uint64_t gfree[P_RING], pwritten[P_RING];          // rank 0: ring slot copied out by rank 1; written
  uint64_t q_ready;
  uint64_t p_full[P_RING];                           // rank 1: ring slot published
  uint64_t p_land[2], p_empty[2], o_done[2], o_ready[2];
  uint64_t lsum[4][2];
  int valid[kValidRing];                             // rank 0: keys of a tile that count (seen through the tile's scores)
  uint32_t tmem_base;
  int abort;
};
constexpr uint32_t OFF_LPART = OFF_BARS + (sizeof(Bars) + 15) / 16 * 16;  // rank 0: float[2][2][128]
constexpr uint32_t kSmem = OFF_LPART + 4 * M_TILE * 4;
static_assert(kStages * kStage0 <= OFF_BARS && kSmem <= 232448, "shared memory budget");

// A message from rank 0 to rank 1 behind its P tile.
struct Meta {
  float alpha[M_TILE];
  float ell[M_TILE];
  uint32_t flags[kSoftWarps];  // of each warp: it has rescaled a row in this tile (else alpha is not written)
  int valid;                   // keys of the tile that count
};
static_assert(kPBytes + sizeof(Meta) <= P_SLOT_BYTES, "P ring slot");

struct Ctx {
  const SharedParams *p;
  uint8_t *base;
  Bars *bars;
  uint32_t rank;
  int part;
};

template <bool kCluster = false>
__device__ __forceinline__ bool wait_ok(const Ctx &c, uint64_t *bar, uint32_t parity) {
  if (mbar_wait<kCluster>(smem_u32(bar), parity, &c.bars->abort, c.p->wait_ns)) return true;
  atomicOr(c.p->status, MLA_STATUS_WAIT_TIMEOUT);
  *(volatile int *)&c.bars->abort = 1;
  return false;
}

// For a whole warp: its lanes go on, or give up, together.
template <bool kCluster = false>
__device__ __forceinline__ bool warp_wait(const Ctx &c, uint64_t *bar, uint32_t parity, bool need = true) {
  return __all_sync(0xffffffffu, !need || wait_ok<kCluster>(c, bar, parity));
}

__device__ __forceinline__ SharedItem item_of(const SharedParams &p, int i) {
  const int4 *src = reinterpret_cast<const int4 *>(p.items + i);
  const int4 a = __ldg(src), b = __ldg(src + 1);
  return SharedItem{a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
}

// The pieces of this worker: f(item, first tile, end tile, slot).
template <class F>
__device__ __forceinline__ bool for_each_piece(const SharedParams &p, int part, F &&f) {
  const int32_t *md = p.md + (size_t)part * MD_STRIDE;
  const int a = md[0], bt = md[1], z = md[2], et = md[3], fp = md[4];
  for (int i = a; i <= z; i++) {
    const SharedItem it = item_of(p, i);
    const int t0 = i == a ? bt : 0, t1 = i == z ? et : it.tiles;
    if (t1 <= t0) continue;
    if (!f(it, t0, t1, it.slot + (i == a ? fp : 0))) return false;
  }
  return true;
}

// Stages of rank 0 for a tile of keys.
template <bool kScaled>
constexpr uint32_t kTileStages = kScaled ? 2 : 1;

// rank 0's ring carries, per piece, the query rows (one stage for 64 rows) before the keys.
__device__ __forceinline__ int q_stages(const SharedItem &it) { return it.rows > 64 ? 2 : 1; }

// (Widened pages lie side by side, a table row's behind those of the rows before it.)
__device__ __forceinline__ int page_of(const SharedParams &p, const SharedItem &it, int tile) {
  const int width = it.own ? p.max_pages : p.max_prefix;
  const int page = __ldg((it.own ? p.block_table : p.prefix_table) + (size_t)it.src * width + tile);
  if (page < 0 || page >= p.num_pages) {
    atomicOr(p.status, MLA_STATUS_BAD_PAGE);
    return -1;
  }
  return p.format == MLA_KV_BF16 ? page : __ldg(p.first + (it.own ? p.G : 0) + it.src) + tile;
}

// ---- warp 0: loads --------------------------------------------------------------------
//
// The pool as [page][9 blocks][64 tokens][64 dims]: one box brings a page as
// column blocks, the K-major operand layout.  rank 0 takes two boxes with barriers of
// their own, so half a stage can be refilled earlier.
template <bool kScaled>
__device__ void load_role(const Ctx &c, const CUtensorMap *map, const CUtensorMap *map_b, const CUtensorMap *q_map, int lane) {
  const SharedParams &p = *c.p;
  Bars &br = *c.bars;
  const uint32_t stage_bytes = c.rank == 0 ? kStage0 : kStage1, kv0 = smem_u32(c.base);
  uint32_t g = 0, s = 0, ph = 1;
  auto next = [&] {
    if (++s == kStages) {
      s = 0;
      ph ^= 1;
    }
  };
  for_each_piece(p, c.part, [&](const SharedItem &it, int t0, int t1, int) {
    // rank 1 is the last to read an own page, unless the sequence has more tiles of rows
    const uint64_t pol = c.rank == 1 && it.own && p.n_mt == 1 ? policy_evict_first() : policy_evict_normal();
    if (c.rank == 0)
      for (int qh = 0; qh < q_stages(it); qh++) {
        bool ok = true;
        if (lane == 0) {
          ok = wait_ok(c, &br.kv_empty[s], ph) && wait_ok(c, &br.kv_empty_b[s], ph);
          if (ok) {
            const uint32_t bar = smem_u32(&br.kv_full[s]);
            mbar_arrive_expect_tx(bar, kStage0);
            tma_load_3d(kv0 + s * kStage0, q_map, bar, 0, it.q_row + 64 * qh, 0, policy_evict_normal());
            mbar_arrive(smem_u32(&br.kv_full_b[s]));
          }
        }
        if (!__shfl_sync(0xffffffffu, ok, 0)) return false;
        next();
      }
    for (int base = t0; base < t1; base += 32) {
      const int pg = base + lane < t1 ? page_of(p, it, base + lane) : -1;
      const int cnt = min(32, t1 - base);
      for (int i = 0; i < cnt; i++, g++) {
        const int page = __shfl_sync(0xffffffffu, pg, i);
        bool ok = true;
        if (lane == 0) {
          if (c.rank == 0) br.valid[g % kValidRing] = page < 0 ? 0 : min(PAGE, it.len - (base + i) * PAGE);
          ok = wait_ok(c, &br.kv_empty[s], ph);
          if (ok) {
            const uint32_t bar = smem_u32(&br.kv_full[s]);
            mbar_arrive_expect_tx(bar, c.rank == 0 ? kSplit * kBlk : kStage1);
            tma_load_4d(kv0 + s * stage_bytes, map, bar, 0, 0, 0, max(page, 0), pol);
          }
          auto upper = [&](int block) {
            ok = ok && wait_ok(c, &br.kv_empty_b[s], ph);
            if (!ok) return;
            const uint32_t bar = smem_u32(&br.kv_full_b[s]);
            mbar_arrive_expect_tx(bar, (9 - kSplit) * kBlk);
            tma_load_4d(kv0 + s * stage_bytes + kSplit * kBlk, map_b, bar, 0, 0, block, max(page, 0), pol);
          };
          if (c.rank == 0) upper(kSplit);
          if (kScaled && c.rank == 0 && ok) {  // the keys' second values (a last block of zeros)
            next();  // (lane 0 alone: the others count nothing)
            ok = wait_ok(c, &br.kv_empty[s], ph);
            if (ok) {
              const uint32_t bar = smem_u32(&br.kv_full[s]);
              mbar_arrive_expect_tx(bar, kSplit * kBlk);
              tma_load_4d(kv0 + s * stage_bytes, map, bar, 0, 0, 9, max(page, 0), pol);
            }
            upper(9 + kSplit);
          }
        }
        if (!__shfl_sync(0xffffffffu, ok, 0)) return false;
        next();
      }
    }
    return true;
  });
}

// ---- MMA warps and their waiters ------------------------------------------------------
//
// A wait in the warp that issues MMAs would hold up those in flight, so warp 3
// does the waiting and meets warp 1 at a named barrier, which also carries the
// decision to give up.
constexpr uint32_t kMmaBar = 1;

__device__ __forceinline__ bool waiter_meet(bool ok) {
  ok = __shfl_sync(0xffffffffu, ok, 0);
  return bar_red_or(kMmaBar, 64, !ok);
}

template <bool kScaled>
__device__ void qk_waiter(const Ctx &c, int lane) {
  Bars &br = *c.bars;
  uint32_t g = 0, qn = 0, sq = 0;
  for_each_piece(*c.p, c.part, [&](const SharedItem &it, int t0, int t1, int) {
    bool ok = true;
    if (lane == 0) ok = wait_ok(c, &br.q_ready, qn & 1);
    qn++;
    sq += q_stages(it);
    if (waiter_meet(ok)) return false;
    for (int t = t0; t < t1; t++, g++) {
      if (lane == 0) ok = wait_ok(c, &br.s_free[g & 1], ((g >> 1) & 1) ^ 1);
      for (uint32_t k = 0; k < kTileStages<kScaled>; k++, sq++) {
        const uint32_t s = sq % kStages, ph = (sq / kStages) & 1;
        if (lane == 0) ok = ok && wait_ok(c, &br.kv_full[s], ph);
        if (waiter_meet(ok)) return false;
        if (lane == 0) ok = wait_ok(c, &br.kv_full_b[s], ph);
        if (waiter_meet(ok)) return false;
      }
    }
    return true;
  });
}

// rank 0: S[g & 1] = Q K^T, A = Q from tensor memory, B = the key blocks.
template <bool kScaled>
__device__ void mma_qk(const Ctx &c, uint32_t tmem) {
  Bars &br = *c.bars;
  const uint32_t kv0 = smem_u32(c.base);
  uint32_t g = 0, sq = 0;
  for_each_piece(*c.p, c.part, [&](const SharedItem &it, int t0, int t1, int) {
    if (bar_red_or(kMmaBar, 64, false)) return false;  // Q is in tensor memory: its stages are free
    tc_fence_after();
    if (elect_one())
      for (int qh = 0; qh < q_stages(it); qh++) {
        mma_commit(smem_u32(&br.kv_empty[(sq + qh) % kStages]));
        mma_commit(smem_u32(&br.kv_empty_b[(sq + qh) % kStages]));
      }
    __syncwarp();
    sq += q_stages(it);
    for (int t = t0; t < t1; t++, g++) {
      const uint32_t b = g & 1, d = tmem + TM_S + b * 64;
#pragma unroll
      for (uint32_t k = 0; k < kTileStages<kScaled>; k++, sq++) {
        const uint32_t s = sq % kStages;
        const uint64_t kd = smem_desc_sw128(kv0 + s * kStage0, 16, 1024);
        if (bar_red_or(kMmaBar, 64, false)) return false;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int i = 0; i < 4 * kSplit; i++)
            mma_ts(d, tmem + TM_Q + i * 8, kd + (uint64_t)((i >> 2) * 512 + (i & 3) * 2), IDESC_QK, k || i ? 1u : 0u);
          mma_commit(smem_u32(&br.kv_empty[s]));
        }
        __syncwarp();
        if (bar_red_or(kMmaBar, 64, false)) return false;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int i = 4 * kSplit; i < (k ? 32 : 36); i++)
            mma_ts(d, tmem + TM_Q + i * 8, kd + (uint64_t)((i >> 2) * 512 + (i & 3) * 2), IDESC_QK, 1u);
          mma_commit(smem_u32(&br.kv_empty_b[s]));
          if (k + 1 == kTileStages<kScaled>) mma_commit(smem_u32(&br.s_full[b]));
        }
        __syncwarp();
      }
    }
    return true;
  });
}

__device__ void pv_waiter(const Ctx &c, int lane) {
  Bars &br = *c.bars;
  uint32_t g = 0;
  for_each_piece(*c.p, c.part, [&](const SharedItem &, int t0, int t1, int) {
    for (int t = t0; t < t1; t++, g++) {
      const uint32_t b = g & 1, u = g >> 1;
      bool ok = true;
      if (lane == 0) {
        ok = wait_ok(c, &br.kv_full[g % kStages], (g / kStages) & 1);
        if (ok) ok = wait_ok(c, &br.p_land[b], u & 1);
        if (ok) ok = wait_ok(c, &br.o_ready[b], u & 1);
      }
      if (waiter_meet(ok)) return false;
    }
    return true;
  });
}

// rank 1: O (+)= P V, A = P from shared memory, B = the value blocks read MN-major.
__device__ void mma_pv(const Ctx &c, uint32_t tmem) {
  Bars &br = *c.bars;
  const uint32_t kv0 = smem_u32(c.base), pbuf = smem_u32(c.base + OFF_RCV_P);
  uint32_t g = 0;
  for_each_piece(*c.p, c.part, [&](const SharedItem &, int t0, int t1, int) {
    for (int t = t0; t < t1; t++, g++) {
      const uint32_t s = g % kStages, b = g & 1;
      if (bar_red_or(kMmaBar, 64, false)) return false;
      tc_fence_after();
      if (elect_one()) {
#pragma unroll
        for (int kk = 0; kk < 4; kk++) {
          const uint64_t a = smem_desc_noswz(pbuf + b * kPBytes + kk * 2 * 2048, 2048, 128);
#pragma unroll
          for (int nh = 0; nh < 2; nh++)
            mma_ss(tmem + TM_O + nh * 256, a, smem_desc_sw128(kv0 + s * kStage1 + nh * 4 * kBlk + kk * 2048, kBlk, 1024),
                   IDESC_PV, t == t0 && kk == 0 ? 0u : 1u);
        }
        mma_commit(smem_u32(&br.kv_empty[s]));
        mma_commit(smem_u32(&br.p_empty[b]));
        mma_commit(smem_u32(&br.o_done[b]));
      }
      __syncwarp();
    }
    return true;
  });
}

// ---- rank 0: softmax ---------------------------------------------------------------------

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t *>(&v);
}

// Query row `row` of a stage of 64, blocks [kb0, kb1), into tensor memory; zeros
// for a row that the item has not.  (Not inlined: it runs once a piece, and its
// registers would crowd the softmax loop.)
__device__ __noinline__ void load_q(uint32_t lane_tmem, uint32_t stage, int row, bool ok, int kb0, int kb1) {
  for (int kb = kb0; kb < kb1; kb++) {
    uint32_t v[32];
#pragma unroll
    for (int j = 0; j < 8; j++) {
      uint4 x = make_uint4(0, 0, 0, 0);
      if (ok)
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                     : "r"(stage + kb * kBlk + row * 128 + ((j ^ (row & 7)) << 4)));
      v[4 * j] = x.x;
      v[4 * j + 1] = x.y;
      v[4 * j + 2] = x.z;
      v[4 * j + 3] = x.w;
    }
    __syncwarp();
    tmem_st32(lane_tmem + TM_Q + kb * 32, v);
  }
  tmem_wait_st();
}

// The largest of three (one instruction).
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

__device__ __forceinline__ float max32(const float (&v)[32]) {
  float m[4];
#pragma unroll
  for (int k = 0; k < 4; k++) {
    m[k] = max3(v[8 * k], v[8 * k + 1], v[8 * k + 2]);
    m[k] = max3(m[k], v[8 * k + 3], v[8 * k + 4]);
    m[k] = max3(m[k], v[8 * k + 5], v[8 * k + 6]);
  }
  return max3(max3(max3(m[0], v[7], v[15]), m[1], m[2]), max3(m[3], v[23], v[31]), m[0]);
}

// Scores from `lim` on become -inf.
__device__ __forceinline__ void cut32(float (&v)[32], int lim) {
  if (lim < 32) {
#pragma unroll
    for (int n = 0; n < 32; n++) v[n] = n < lim ? v[n] : -INFINITY;
  }
}

// Warps 4-11: thread (q, hf) has row 32 q + lane and keys [32 hf, 32 hf + 32) of
// each tile.  Both threads of a row read all 64 scores, so they agree on the
// running maximum without talking; the reference moves only when it grows by kRescale.
template <bool kScaled>
__device__ void softmax_role(const Ctx &c, uint32_t tmem, int w, int lane) {
  const SharedParams &p = *c.p;
  Bars &br = *c.bars;
  const int q = w & 3, hf = (w - 4) >> 2, r = q * 32 + lane;
  const uint32_t lt = tmem + ((uint32_t)(q * 32) << 16), kv0 = smem_u32(c.base);
  float *lpart = reinterpret_cast<float *>(c.base + OFF_LPART);
  // (not 0, so that -inf stays -inf: a scale of 0 is one of codes of 0)
  const float cs = p.format == MLA_KV_FP8_E4M3_TENSOR ? fmaxf(p.scale_log2 * __ldg(p.kv_scales), 1e-37f) : p.scale_log2;
  uint32_t g = 0, pc = 0, sq = 0;
  for_each_piece(p, c.part, [&](const SharedItem &it, int t0, int t1, int slot_out) {
    const bool live = r < it.rows;
    {
      const uint32_t qs = sq + (r >> 6);
      if (!warp_wait(c, &br.kv_full[qs % kStages], (qs / kStages) & 1, live)) return false;
      load_q(lt, kv0 + (qs % kStages) * kStage0, r & 63, live, hf ? 5 : 0, hf ? 9 : 5);
      sq += q_stages(it) + (t1 - t0) * kTileStages<kScaled>;
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&br.q_ready));
    }
    // keys that this row sees
    const int len = it.own ? row_kv_len(it.len, p.T, min(it.row0 + r, p.T * p.H - 1) / p.H, p.causal) : it.len;
    float m_ref = -INFINITY, l = 0.f, l_all = 0.f;
    int most = 0;  // keys of a tile that it has seen, at most
    for (int t = t0; t < t1; t++, g++) {
      const uint32_t b = g & 1, u = g >> 1;
      if (!warp_wait(c, &br.s_full[b], u & 1)) return false;
      const int valid = br.valid[g % kValidRing], lim = min(valid, len - t * PAGE);
      most = max(most, lim);
      tc_fence_after();
      float own[32], oth[32];
      tmem_ld32(lt + TM_S + b * 64 + hf * 32, *reinterpret_cast<uint32_t(*)[32]>(&own[0]));
      tmem_ld32(lt + TM_S + b * 64 + (hf ^ 1) * 32, *reinterpret_cast<uint32_t(*)[32]>(&oth[0]));
      tmem_wait_ld();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&br.s_free[b]));
      cut32(own, lim - 32 * hf);
      cut32(oth, lim - 32 * (hf ^ 1));
      const float mt = fmaxf(max32(own), max32(oth));
      float alpha = 1.f;
      bool resc = false;
      if ((mt - m_ref) * cs > kRescale) {
        if (m_ref != -INFINITY) {
          alpha = ex2((m_ref - mt) * cs);
          resc = true;
        }
        m_ref = mt;
        l *= alpha;
      }
      const float nb = m_ref == -INFINITY ? 0.f : -m_ref * cs;
      const uint32_t gs = g % P_RING;
      // (slots come back in order: one wait for the last of four)
      if (g % kFreeBatch == 0) {
        const uint32_t ahead = g | (kFreeBatch - 1);
        if (!warp_wait(c, &br.gfree[ahead % P_RING], ((ahead / P_RING) & 1) ^ 1)) return false;
      }
      uint8_t *slot = p.ring + ((size_t)c.part * P_RING + gs) * P_SLOT_BYTES;
      float2 psum = make_float2(0.f, 0.f);
#pragma unroll
      for (int cc = 0; cc < 4; cc++) {  // chunk-major: chunk ch of row r at ch * 2048 + r * 16
        uint32_t wv[4];
#pragma unroll
        for (int e = 0; e < 4; e++) {
          const float2 x = fma2(make_float2(own[cc * 8 + 2 * e], own[cc * 8 + 2 * e + 1]), make_float2(cs, cs), make_float2(nb, nb));
          const float2 pr = make_float2(ex2(x.x), ex2(x.y));
          psum = add2(psum, pr);
          wv[e] = pack_bf16(pr.x, pr.y);
        }
        *reinterpret_cast<uint4 *>(slot + (hf * 4 + cc) * 2048 + r * 16) = make_uint4(wv[0], wv[1], wv[2], wv[3]);
      }
      l += psum.x + psum.y;
      Meta *mo = reinterpret_cast<Meta *>(slot + kPBytes);
      const bool any = __any_sync(0xffffffffu, resc);
      if (any && hf == 0) mo->alpha[r] = alpha;
      if (lane == 0) mo->flags[w - 4] = any ? 1u : 0u;
      if (w == 4 && lane == 0) mo->valid = valid;
      if (t == t1 - 1) {  // the row's two halves meet
        float *lp = lpart + (pc & 1) * 2 * M_TILE;
        lp[hf * M_TILE + r] = l;
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&br.lsum[q][pc & 1]));
        if (!warp_wait(c, &br.lsum[q][pc & 1], (pc >> 1) & 1)) return false;
        l_all = lp[r] + lp[M_TILE + r];
        if (hf == 0) mo->ell[r] = l_all;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&br.pwritten[gs]));
    }
    pc++;
    // (the sum is 0 without keys and where all scores are -inf: the largest score's weight is 1 otherwise)
    if (live && hf == 0)
      p.lse_p[(size_t)slot_out * M_TILE + r] = l_all != 0.f ? m_ref * cs + __log2f(l_all) : most > 0 ? kAllLow : -INFINITY;
    return true;
  });
}

// rank 0, one thread: makes written messages visible to rank 1, up to four at once
// (a fence waits for the stores to reach L2, so it is off the softmax warps' path).
__device__ void publish_role(const Ctx &c) {
  Bars &br = *c.bars;
  const uint32_t pfull = mapa(smem_u32(&br.p_full[0]), 1);
  uint32_t total = 0;
  for_each_piece(*c.p, c.part, [&](const SharedItem &, int t0, int t1, int) {
    total += (uint32_t)(t1 - t0);
    return true;
  });
  for (uint32_t g = 0; g < total;) {
    if (!wait_ok(c, &br.pwritten[g % P_RING], (g / P_RING) & 1)) return;
    uint32_t n = 1;
    while (n < kPublishBatch && g + n < total &&
           mbar_test_wait(smem_u32(&br.pwritten[(g + n) % P_RING]), ((g + n) / P_RING) & 1))
      n++;
    fence_acq_rel_cluster();
    for (uint32_t i = 0; i < n; i++) mbar_arrive_remote_relaxed(pfull + ((g + i) % P_RING) * 8);
    g += n;
  }
}

// ---- rank 1: P into shared memory, rescales, results ---------------------------------------

__device__ __forceinline__ void st_shared_v4(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

__device__ void output_role(const Ctx &c, uint32_t tmem, int w, int lane) {
  const SharedParams &p = *c.p;
  Bars &br = *c.bars;
  const int q = w & 3, hf = (w - 4) >> 2, r = q * 32 + lane, e = (w - 4) * 32 + lane;
  const uint32_t lt = tmem + ((uint32_t)(q * 32) << 16) + TM_O + hf * 256;
  const uint32_t pbuf = smem_u32(c.base + OFF_RCV_P), gfree = mapa(smem_u32(&br.gfree[0]), 0);
  uint32_t g = 0;
  for_each_piece(p, c.part, [&](const SharedItem &it, int t0, int t1, int slot_out) {
    float ell = 0.f;
    for (int t = t0; t < t1; t++, g++) {
      const uint32_t b = g & 1, u = g >> 1, gs = g % P_RING;
      if (!warp_wait<true>(c, &br.p_full[gs], (g / P_RING) & 1)) return false;
      const uint8_t *slot = p.ring + ((size_t)c.part * P_RING + gs) * P_SLOT_BYTES;
      const uint4 *src = reinterpret_cast<const uint4 *>(slot);
      uint4 v[4];
#pragma unroll
      for (int k = 0; k < 4; k++) v[k] = __ldcg(src + e + 256 * k);
      const Meta *m = reinterpret_cast<const Meta *>(slot + kPBytes);
      const uint4 f0 = __ldcg(reinterpret_cast<const uint4 *>(m->flags));
      const uint4 f1 = __ldcg(reinterpret_cast<const uint4 *>(m->flags) + 1);
      const int valid = __ldcg(&m->valid);
      if (t == t1 - 1) ell = __ldcg(&m->ell[r]);
      if (!warp_wait(c, &br.p_empty[b], (u & 1) ^ 1)) return false;
#pragma unroll
      for (int k = 0; k < 4; k++) st_shared_v4(pbuf + b * kPBytes + (e + 256 * k) * 16, v[k]);
      if (valid < PAGE) {  // values that do not count become 0 (16 bytes of each block's row for a thread)
        if (!warp_wait(c, &br.kv_full[g % kStages], (g / kStages) & 1)) return false;
        const uint32_t stage = smem_u32(c.base) + (g % kStages) * kStage1;
        for (int i = valid * 64 + e; i < PAGE * 64; i += 256)
          st_shared_v4(stage + ((i >> 3) & 7) * kBlk + (i >> 6) * 128 + (i & 7) * 16, make_uint4(0, 0, 0, 0));
      }
      // (the rescales' factors are read from the slot only where there are any)
      const bool rescale = (f0.x | f0.y | f0.z | f0.w | f1.x | f1.y | f1.z | f1.w) != 0u;
      const bool mine = (q == 0 ? f0.x : q == 1 ? f0.y : q == 2 ? f0.z : f0.w) != 0u;  // this row group's
      float alpha = 1.f;
      if (mine) alpha = __ldcg(&m->alpha[r]);
      // the slot goes back once this warp's loads are done: the chunks are consumed
      // by the stores above, the rest by this (a release would wait for the stores too)
      {
        uint32_t dep;
        asm volatile("add.u32 %0, %1, %2;" : "=r"(dep) : "r"(__float_as_uint(alpha)), "r"(__float_as_uint(ell)));
        asm volatile("" ::"r"(dep), "r"(f0.x), "r"(f1.w), "r"(valid));
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(smem_u32(&br.p_land[b]));
        mbar_arrive_remote_relaxed(gfree + gs * 8);
      }
      if (rescale) {  // rare: O *= alpha between two products
        if (!warp_wait(c, &br.o_done[(g - 1) & 1], ((g - 1) >> 1) & 1)) return false;
        tc_fence_after();
        for (int cc = 0; cc < 8; cc++) {
          uint32_t o[32];
          tmem_ld32(lt + cc * 32, o);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 32; j++) o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha);
          tmem_st32(lt + cc * 32, o);
        }
        tmem_wait_st();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&br.o_ready[b]));
    }
    if (!warp_wait(c, &br.o_done[(g - 1) & 1], ((g - 1) >> 1) & 1)) return false;
    tc_fence_after();
    const float inv = (ell != 0.f ? 1.f / ell : 0.f) * (p.format == MLA_KV_FP8_E4M3_TENSOR ? __ldg(p.kv_scales) : 1.f);
    // chunk-major: the 32 rows of a warp store 8 columns as 1 KB side by side; the
    // next columns are on their way meanwhile
    float *dst = p.o_p + ((size_t)slot_out * 64 + hf * 32) * (M_TILE * 8) + (size_t)r * 8;
    uint32_t o[2][32];
    tmem_ld32(lt, o[0]);
#pragma unroll
    for (int cc = 0; cc < 8; cc++) {
      tmem_wait_ld();
      if (cc + 1 < 8) tmem_ld32(lt + (cc + 1) * 32, o[(cc + 1) & 1]);
      uint32_t(&v)[32] = o[cc & 1];
#pragma unroll
      for (int j = 0; j < 32; j++) v[j] = __float_as_uint(__uint_as_float(v[j]) * inv);
      if (r < it.rows)
#pragma unroll
        for (int j = 0; j < 4; j++)
          st_global_v8(dst + (size_t)(cc * 4 + j) * (M_TILE * 8), *reinterpret_cast<const uint32_t(*)[8]>(&v[8 * j]));
      __syncwarp();
    }
    return true;
  });
}

template <bool kScaled>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    shared_attention_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap kb_map,
                            const __grid_constant__ CUtensorMap v_map, const __grid_constant__ CUtensorMap q_map,
                            const SharedParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023u) {
    if (threadIdx.x == 0) atomicOr(p.status, MLA_STATUS_SMEM_ALIGN);
    return;
  }
  Bars &br = *reinterpret_cast<Bars *>(smem + OFF_BARS);
  const uint32_t rank = cluster_ctarank();
  const Ctx c{&p, smem, &br, rank, (int)cluster_id_x()};
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; s++) {
      mbar_init(smem_u32(&br.kv_full[s]), 1);
      mbar_init(smem_u32(&br.kv_empty[s]), 1);
      mbar_init(smem_u32(&br.kv_full_b[s]), 1);
      mbar_init(smem_u32(&br.kv_empty_b[s]), 1);
    }
    for (int i = 0; i < P_RING; i++) {
      mbar_init(smem_u32(&br.gfree[i]), kSoftWarps);
      mbar_init(smem_u32(&br.pwritten[i]), kSoftWarps);
      mbar_init(smem_u32(&br.p_full[i]), 1);
    }
    for (int b = 0; b < 2; b++) {
      mbar_init(smem_u32(&br.s_full[b]), 1);
      mbar_init(smem_u32(&br.s_free[b]), kSoftWarps);
      mbar_init(smem_u32(&br.p_land[b]), kSoftWarps);
      mbar_init(smem_u32(&br.p_empty[b]), 1);
      mbar_init(smem_u32(&br.o_ready[b]), kSoftWarps);
      mbar_init(smem_u32(&br.o_done[b]), 1);
    }
    mbar_init(smem_u32(&br.q_ready), kSoftWarps);
    for (int q = 0; q < 4; q++)
      for (int b = 0; b < 2; b++) mbar_init(smem_u32(&br.lsum[q][b]), 2);
    br.abort = 0;
    fence_mbar_init_cluster();
    prefetch_tensormap(rank == 0 ? (const void *)&k_map : (const void *)&v_map);
    prefetch_tensormap(&q_map);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&br.tmem_base), TM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  cluster_sync();
  const uint32_t tmem = br.tmem_base;
  grid_dep_wait();
  if (warp == 0) {
    load_role<kScaled>(c, rank == 0 ? &k_map : &v_map, &kb_map, &q_map, lane);
  } else if (warp == 1) {
    if (rank == 0) mma_qk<kScaled>(c, tmem);
    else mma_pv(c, tmem);
  } else if (warp == 3) {
    if (rank == 0) qk_waiter<kScaled>(c, lane);
    else pv_waiter(c, lane);
  } else if (warp == 2) {
    if (lane == 0 && rank == 0) publish_role(c);
  } else {
    if (rank == 0) softmax_role<kScaled>(c, tmem, warp, lane);
    else output_role(c, tmem, warp, lane);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  grid_dep_trigger();
  if (br.abort) {  // copies and MMAs in flight end
    const uint64_t t0 = globaltimer();
    while (globaltimer() - t0 < 2000000ull) {
    }
  }
  __syncwarp();
  cluster_sync();  // the peer no longer arrives on this CTA's barriers
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, TM_COLS);
  }
}

}  // namespace

cudaError_t launch_shared_attention(const SharedParams &p, cudaStream_t stream) {
  const auto fn = tensor_map_encoder();
  if (!fn) return cudaErrorNotSupported;
  // pages of 9 blocks, with scales 17; the first 8 are the values too
  const bool wide = p.format != MLA_KV_BF16, scaled = p.format == MLA_KV_FP8_E4M3;
  const uint8_t *pool = wide ? p.scratch : p.cache;
  const cuuint64_t pages = wide ? (cuuint64_t)p.scratch_pages : (cuuint64_t)p.num_pages;
  const cuuint64_t row = (scaled ? D_QK + D_V : D_QK) * 2;
  cuuint64_t dims[4] = {64, (cuuint64_t)PAGE, scaled ? 17u : 9u, pages}, strides[3] = {row, 128, row * PAGE};
  cuuint32_t estr[4] = {1, 1, 1, 1};
  CUtensorMap maps[4];
  const cuuint32_t blocks[3] = {kSplit, 9 - kSplit, 8};
  for (int m = 0; m < 3; m++) {
    cuuint32_t box[4] = {64, (cuuint32_t)PAGE, blocks[m], 1};
    if (fn(&maps[m], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<uint8_t *>(pool), dims, strides, box, estr,
           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
      return cudaErrorInvalidValue;
  }
  if (!make_map_3d(&maps[3], p.q, 64, (uint64_t)p.B * p.T * p.H, 9, D_QK, 64, 64, 9)) return cudaErrorInvalidValue;
  const auto kernel = scaled ? shared_attention_kernel<true> : shared_attention_kernel<false>;
  cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
  if (e != cudaSuccess) return e;
  return launch_dependent(kernel, 2 * p.parts, kThreads, kSmem, stream, maps[0], maps[1], maps[2], maps[3], p);
}

}  // namespace mla

// The attention weight of cached tokens: for each cached token n of a sequence
//   mass[n] = decay * mass[n] + sum_{t,h} exp(scale * q[t][h] . K_n - lse[h][t])
// over the query rows (t, h) that see it: the column sums of the softmax that a
// decode (or a prompt's attention) has made, from its log-sum-exp, without its
// product with the values.
//
// A pair of CTAs works as one: an MMA tile has 256 keys as its M rows, 128 of each
// CTA, and up to 256 query rows as its N columns, half of them from the shared
// memory of each.  A key's scores lie in one lane of tensor memory, so its sum is
// one thread's own: nothing crosses lanes, no atomics.  (Pairs halve what each SM
// holds and reads of the query rows: alone, an SM has room for 128 rows and 64 KB
// of keys on their way, and with many rows its shared memory is the limit: 8192
// rows on 12001 keys 101 us.)
//
// 64 sequences of up to 32768 tokens, 128 heads: 184 us, bound by HBM (6.6 TB/s of 6.7).
// The last 64 tokens of 12001, 128 heads: 67 us for 113 GFLOP, bound by the tensor cores (82 % of the
// cycles).  32 FP8 sequences of up to 8192 tokens, 2 x 64 rows: 41 us for 95 MB (one scale: 36 for 84), bound by the
// hand-overs between loads, widening, products and sums.
#include <atomic>
#include <cmath>
#include <cstdio>

#include "common.cuh"
#include "dependent.cuh"
#include "fp8.cuh"
#include "pairs_f32.cuh"
#include "ptx.cuh"
#include "ptx_pair.cuh"
#include "tma_map.cuh"

namespace mla {
namespace {

using namespace ptx;

constexpr int kKeys = 128;                     // keys of a CTA's half of a tile: two pages
constexpr int kTileKeys = 2 * kKeys;
constexpr int kBlocks = D_QK / 64;             // blocks of 64 of the 576 dims
constexpr uint32_t kBlock = kKeys * 128;       // 128 rows x 64 dims, 128-byte swizzle
constexpr uint32_t kHalf = kBlock / 2;
constexpr int kMostSlots = 9;                  // units of the streaming operand
constexpr int kMostRows = 256;                 // query rows of a tile

// What depends on the cache's format.  No rounding is made on the way to the scores:
// FP8 codes are exact in bf16, so a per-tensor scale multiplies the scores, and
// with a scale for each 128 latent values the product is made in five parts (four
// times 128 values, and the rotated 64), which the summing threads scale and add.
// Those hold a tile's scores in registers, so its tiles have half the query rows and
// two threads a key.  (Rows dequantised to bf16 would put the scores off by 3e-3.)
template <int kFormat>
struct Of {
  static constexpr bool fp8 = kFormat != MLA_KV_BF16, scaled = kFormat == MLA_KV_FP8_E4M3;
  static constexpr int rows = scaled ? 128 : kMostRows;        // query rows of a tile
  static constexpr int parts = scaled ? 5 : 1;                 // score tiles in tensor memory for one tile
  static constexpr int kd = 512 / rows;                        // score tiles that there is room for
  static constexpr int halves = scaled ? 2 : 1;                // threads of a key
  static constexpr int cols = rows / halves;                   // columns of a thread
  static constexpr int sum_warps = 4 * halves;
  static constexpr int wide_warps = fp8 ? 8 : 0;               // warps that widen cached rows
  static constexpr int threads = 32 * (4 + sum_warps + wide_warps);
  // Operands come in units: a block, or with FP8 two (a last one alone), so that a row of a
  // copy is 128 bytes (rows of 64 codes: 44.5 us instead of 38.8 for 32 sequences of up to 8192
  // tokens, two query tokens, 64 heads)
  static constexpr int unit = fp8 ? 2 : 1, units = fp8 ? 5 : kBlocks;
  __device__ static constexpr int blocks(int u) { return u < kBlocks / unit ? unit : kBlocks % unit; }
  // The score tile that unit u belongs to begins, or ends, with it.
  __device__ static constexpr bool begins(int u) { return parts > 1 || u == 0; }
  __device__ static constexpr bool ends(int u) { return parts > 1 || u == units - 1; }
};
// Two groups of four warps widen units in turn.  A barrier is always waited for by the same
// group (of an even number of slots, and of the units that stay): one that comes to it while
// the phase before is still open would take the one before that for its own.
constexpr int kGroups = 2, kGroupWarps = 4;
// With scales: registers of the threads that load, sum and widen (96 each would spill where
// scores are summed, 48.5 us instead of 44.6 for 32 sequences of up to 8192 tokens, two query
// tokens, 64 heads).
constexpr int kLoadRegs = 72, kSumRegs = 120, kWideRegs = 80;
constexpr uint32_t IDESC = idesc_bf16_f32(kTileKeys, 16, false, false) - (2u << 17);  // N is added

struct MassParams {
  const float *kv_scales;
  const int32_t *block_table, *seqlens;
  const float *lse;  // [B][H][T]
  float *mass;       // [B][cap]
  float *partial;    // [pairs][2][256]: sums of tiles that a pair has in part, its first and its last
  unsigned int *status;
  int num_pages, max_pages, B, T, H, cap, causal;
  int rows, n_qt, box;  // query rows of a sequence, their tiles, the columns of a tile (half of each CTA)
  int slots;
  float scale, decay;
  unsigned long long wait_ns;
};

struct Bars {
  uint64_t res_full[kBlocks], res_empty[kBlocks];        // full: rank 0, for both CTAs
  uint64_t slot_full[kMostSlots], slot_empty[kMostSlots];
  uint64_t raw_full[kMostSlots];  // FP8: a unit's codes are in place (of the resident ones, or of the slots)
  uint64_t wide_full[kMostSlots]; // FP8, rank 1: a unit is widened
  uint64_t d_full[4], d_empty[4];                        // empty: rank 0
  alignas(16) float nl[2][kMostRows];  // -lse of a tile's query rows
  alignas(16) int lim[2][kMostRows];   // keys that a row sees; 0 for one that is no row, or has no weight to give
  int least[2][kMostRows / 32];        // the smallest of each 32 rows
  float half[2][kKeys];                // sums of the columns' upper half
  int warp_sums[32];
  int start_b, start_t;
  uint32_t tmem_base;
  int abort;
};
// Shared memory: barriers, the resident operand's blocks, what streams.
constexpr uint32_t OFF_RES = 7 * 1024;
constexpr uint32_t kSmem = 232448 / 1024 * 1024;
static_assert(sizeof(Bars) <= OFF_RES, "shared memory map");
static_assert(OFF_RES + kBlocks * kBlock + 4 * kBlock <= kSmem, "shared memory map");

constexpr uint32_t kRoom = kSmem - OFF_RES;

// Tile loads into this CTA whose bytes a barrier of either CTA of the pair counts.
__device__ __forceinline__ void tma_load_4d_pair(uint32_t dst, const void *map, uint32_t cluster_bar, int c0, int c1, int c2,
                                                 int c3, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes.cta_group::2.L2::cache_hint"
      " [%0], [%1, {%2, %3, %4, %5}], [%6], %7;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(cluster_bar), "l"(policy)
      : "memory");
}

__device__ __forceinline__ int seq_len(const MassParams &p, int b) {
  const int most = (int)min((long long)p.max_pages * PAGE, (long long)p.cap);
  return min(max(__ldg(p.seqlens + b), 0), most);
}

// kCluster: acquire at the scope of the cluster, for what threads of the other CTA have written.
// The other waits are for copies and MMAs, or for writes of this CTA.
template <bool kPoll, bool kCluster = false>
__device__ __forceinline__ bool wait_ok(Bars *b, uint64_t *bar, uint32_t parity, const MassParams &p) {
  if (mbar_wait_limited<kCluster, kPoll>(smem_u32(bar), parity, &b->abort, p.wait_ns)) return true;
  atomicOr(p.status, MLA_STATUS_WAIT_TIMEOUT);
  *(volatile int *)&b->abort = 1;
  return false;
}

// The same for a whole warp: its lanes go on, or give up, together.
template <bool kPoll, bool kCluster = false>
__device__ __forceinline__ bool warp_wait(Bars *b, uint64_t *bar, uint32_t parity, const MassParams &p) {
  return __all_sync(0xffffffffu, wait_ok<kPoll, kCluster>(b, bar, parity, p));
}

// The work is a line of units (key tile, query tile), query tiles innermost, of
// which each pair has an equal part.  A phase: a resident operand and what
// streams past it.  kStreamKeys (one query tile): the query rows of sequence b stay
// and its key tiles [i0, i1) pass by, each one a sum of its own.  Otherwise key tile
// t stays and query tiles [i0, i1) pass by; whole: they are all of its query tiles,
// else their sum is one of several, kept in place `part` of the pair's two.
struct Phase {
  int b, t, i0, i1, len, part;
  bool whole;
};

struct Work {
  int b, t;          // sequence and key tile of the first unit
  long long u0, u1;  // units of this pair
};

template <bool kStreamKeys, int kRows, class F>
__device__ __forceinline__ bool for_each_phase(const MassParams &p, const Work &w, F &&f) {
  int b = w.b, t = w.t, len = w.u0 < w.u1 ? seq_len(p, b) : 0;
  for (long long u = w.u0; u < w.u1;) {
    while (t * kTileKeys >= len) {
      if (++b >= p.B) return true;
      t = 0;
      len = seq_len(p, b);
    }
    if (kStreamKeys) {
      const int n = (int)min(w.u1 - u, (long long)(ceil_div(len, kTileKeys) - t));
      if (!f(Phase{b, t, t, t + n, len, 0, true})) return false;
      t += n;
      u += n;
    } else {
      const int i0 = (int)(u % p.n_qt), i1 = (int)min((long long)p.n_qt, i0 + (w.u1 - u));
      Phase ph{b, t, i0, i1, len, i0 == 0 ? 1 : 0, i0 == 0 && i1 == p.n_qt};
      if (p.causal) {  // query rows before the first that sees any of these keys
        const int t_min = max(0, t * kTileKeys - len + p.T);
        ph.i0 = (int)min((long long)i1, max((long long)i0, (long long)t_min * p.H / kRows));
      }
      if (!f(ph)) return false;
      u += i1 - i0;
      t++;
    }
  }
  return true;
}

// The number of key tiles; with `b` and `at`, those of the sequences before this thread's.
struct Tiles {
  int mine, before, total, b0, b1;
};

__device__ Tiles count_tiles(const MassParams &p, int *warp_sums) {
  const int n = blockDim.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = ceil_div(p.B, n);
  Tiles t;
  t.b0 = min(p.B, tid * per);
  t.b1 = min(p.B, t.b0 + per);
  t.mine = 0;
  for (int b = t.b0; b < t.b1; b++) t.mine += ceil_div(seq_len(p, b), kTileKeys);
  int incl = t.mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  t.before = incl - t.mine;
  t.total = 0;
  for (int i = 0; i < n / 32; i++) {
    if (i < warp) t.before += warp_sums[i];
    t.total += warp_sums[i];
  }
  return t;
}

// Sequence and tile within it of tile `x` of all, told by the thread that has it.
__device__ __forceinline__ void find_tile(const MassParams &p, const Tiles &t, int x, int *b_out, int *t_out) {
  if (x < t.before || x >= t.before + t.mine) return;
  int at = t.before;
  for (int b = t.b0; b < t.b1; b++) {
    const int c = ceil_div(seq_len(p, b), kTileKeys);
    if (x < at + c) {
      *b_out = b;
      *t_out = x - at;
      return;
    }
    at += c;
  }
}

__device__ __forceinline__ long long first_unit(long long units, int pair, int pairs) { return units * pair / pairs; }

__device__ Work find_work(const MassParams &p, Bars &br, int pair, int pairs) {
  const Tiles t = count_tiles(p, br.warp_sums);
  if (blockIdx.x == 0)
    for (int b = t.b0; b < t.b1; b++)
      if (__ldg(p.seqlens + b) != seq_len(p, b)) atomicOr(p.status, MLA_STATUS_BAD_SEQLEN);
  const long long units = (long long)t.total * p.n_qt;
  Work w;
  w.u0 = first_unit(units, pair, pairs);
  w.u1 = first_unit(units, pair + 1, pairs);
  find_tile(p, t, (int)(w.u0 / p.n_qt), &br.start_b, &br.start_t);
  __syncthreads();
  w.b = br.start_b;
  w.t = br.start_t;
  return w;
}

// Where this CTA's operands lie.
struct Place {
  uint32_t res, res_block, slots, slot_block, slot, rank;  // slot: bytes of a unit
};

// ---- loads -------------------------------------------------------------------------

// Warps 0 and 3: cached rows, each one page of this CTA's two; warp 0 query rows too.
// (A warp's wait, arrival and copy take some 350 cycles together, whatever the copy's
// size: one warp alone would take longer over a block's two pages than HBM.)  The
// whole warp waits and looks pages up, one elected lane asks for the copies.  rank 0's
// barriers count the bytes of both CTAs.  A unit of FP8 rows lands as codes in the
// upper half of what it will fill, on a barrier of this CTA; the rotated part of rows
// with scales is bf16 and lands as it is used.
template <bool kStreamKeys, int kFormat, bool kPoll>
__device__ void load_role(const MassParams &p, Bars &br, const CUtensorMap *k_map, const CUtensorMap *pe_map,
                          const CUtensorMap *q_map, const Work &w, const Place &at, int which) {
  using C = Of<kFormat>;
  constexpr int kRows = C::rows;
  const uint64_t keep = policy_evict_normal(), key_pol = kStreamKeys ? policy_evict_first() : keep;
  int s = 0;
  uint32_t ph = 1, rph = 1;
  // This CTA's pages of a tile, and how many both CTAs have.  Lanes 0-3 look up the
  // tile's four pages; those of the next tile while this one is asked for.
  int pg[2] = {-1, -1}, pages = 0, entry = -1;
  bool listed = false;
  const int lane = threadIdx.x & 31;
  auto fetch = [&](int b, int t, int len) {
    listed = lane < 4 && (4ll * t + lane) * PAGE < len;
    if (listed) entry = __ldg(p.block_table + (size_t)b * p.max_pages + 4 * t + lane);
  };
  auto look = [&] {
    const bool good = listed && entry >= 0 && entry < p.num_pages;
    if (listed && !good) atomicOr(p.status, MLA_STATUS_BAD_PAGE);
    const uint32_t have = __ballot_sync(0xffffffffu, good);
    pages = __popc(have);
#pragma unroll
    for (int h = 0; h < 2; h++) {
      const int at_lane = 2 * at.rank + h, page = __shfl_sync(0xffffffffu, entry, at_lane);
      pg[h] = (have >> at_lane) & 1 ? page : -1;
    }
  };
  auto keys = [&](uint32_t dst, uint64_t *full, uint64_t *raw, int u) {
    if (!elect_one()) return;
    const int page = pg[which];
    if (!C::fp8) {
      if (which == 0 && at.rank == 0) mbar_arrive_expect_tx(smem_u32(full), pages * kHalf);
      if (page >= 0) tma_load_4d_pair(dst + which * kHalf, k_map, mapa(smem_u32(full), 0), 0, 0, u, page, key_pol);
      return;
    }
    const uint32_t bar = smem_u32(raw), n = (pg[0] >= 0) + (pg[1] >= 0);
    const bool last = u == C::units - 1;
    if (which == 0) mbar_arrive_expect_tx(bar, n * (last && !C::scaled ? kHalf / 2 : kHalf));
    if (page < 0) return;
    if (!last) tma_load_3d(dst + kBlock + which * kHalf, k_map, bar, u * 128, 0, page, key_pol);
    else if (C::scaled) tma_load_3d(dst + which * kHalf, pe_map, bar, 0, 0, page, key_pol);
    else tma_load_3d(dst + kHalf + which * (kHalf / 2), pe_map, bar, D_V, 0, page, key_pol);
  };
  const int half = p.box / 2;  // query rows of each CTA
  auto rows = [&](uint32_t dst, uint32_t block, uint64_t *full, int b, int qt, int u) {
    if (!elect_one()) return;
    const int n = C::blocks(u);
    if (at.rank == 0) mbar_arrive_expect_tx(smem_u32(full), n * p.box * 128);
    for (int j = 0; j < n; j++)
      tma_load_3d_pair(dst + j * block, q_map, mapa(smem_u32(full), 0), 0, b * p.rows + qt * kRows + (int)at.rank * half,
                       u * C::unit + j, keep);
  };
  for_each_phase<kStreamKeys, kRows>(p, w, [&](const Phase &f) {
    if (f.i0 >= f.i1) return true;
    // (the first of what streams is asked for along with the resident units, so that
    // both follow the last phase's MMAs unit by unit)
    fetch(f.b, f.t, f.len);
    if (!kStreamKeys) look();
    for (int i = f.i0; i < (kStreamKeys || which == 0 ? f.i1 : f.i0 + 1); i++) {
      if (kStreamKeys) {
        look();
        if (i + 1 < f.i1) fetch(f.b, i + 1, f.len);
      }
      for (int u = 0; u < C::units; u++) {
        if (i == f.i0 && (!kStreamKeys || which == 0)) {
          if (!warp_wait<kPoll>(&br, &br.res_empty[u], rph, p)) return false;
          const uint32_t dst = at.res + u * C::unit * at.res_block;
          if (kStreamKeys) rows(dst, at.res_block, &br.res_full[u], f.b, 0, u);
          else keys(dst, &br.res_full[u], &br.raw_full[u], u);
          __syncwarp();
        }
        if (!kStreamKeys && which == 1) continue;
        if (!warp_wait<kPoll>(&br, &br.slot_empty[s], ph, p)) return false;
        const uint32_t dst = at.slots + s * at.slot;
        if (kStreamKeys) keys(dst, &br.slot_full[s], &br.raw_full[s], u);
        else rows(dst, at.slot_block, &br.slot_full[s], f.b, i, u);
        __syncwarp();
        if (++s == p.slots) {
          s = 0;
          ph ^= 1;
        }
      }
    }
    rph ^= 1;
    return true;
  });
}

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ void st_shared_v4(uint32_t addr, const uint4 &v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// The last warps widen FP8 codes in place, in groups that take the units in turn.  All
// of a group read their codes before any writes bf16 values over them.  (The codes come
// by TMA: a load of its own in flight would hold up the thread's proxy fences.)
constexpr uint32_t kWideBar = 3, kGroupThreads = 32 * kGroupWarps;

// Rows of kChunks * 16 codes at `raw` to blocks from `dst` on: thread i has 16 codes of
// kChunks rows.
template <int kChunks>
__device__ __forceinline__ bool widen_unit(uint32_t dst, uint32_t raw, int i, int group, bool ok) {
  constexpr int kStep = kGroupThreads / kChunks, kMine = kKeys / kStep;
  static_assert(kStep % 8 == 0, "a thread's rows have one swizzle");
  const int r = i / kChunks, c = i % kChunks, x = r & 7;
  uint4 v[kMine];
#pragma unroll
  for (int j = 0; j < kMine; j++) v[j] = ld_shared_v4(raw + (r + kStep * j) * (kChunks * 16) + c * 16);
  if (bar_red_or(kWideBar + group, kGroupThreads, !ok)) return false;
#pragma unroll
  for (int j = 0; j < kMine; j++) {
    uint4 lo, hi;
    codes16(v[j], lo, hi);
    const uint32_t row = dst + (c >> 2) * kBlock + (r + kStep * j) * 128;
    st_shared_v4(row + (((2 * (c & 3)) ^ x) << 4), lo);
    st_shared_v4(row + (((2 * (c & 3) + 1) ^ x) << 4), hi);
  }
  fence_proxy_async_smem();
  return true;
}

template <bool kStreamKeys, int kFormat, bool kPoll>
__device__ void widen_role(const MassParams &p, Bars &br, const Work &w, const Place &at, int thread) {
  using C = Of<kFormat>;
  const int group = thread / kGroupThreads, i = thread % kGroupThreads;
  const bool first = (threadIdx.x & 31) == 0;
  static_assert(C::wide_warps == kGroups * kGroupWarps, "");
  int s = 0;
  uint32_t ph = 0, tile = 0;
  auto widen_tile = [&] {
    for (int u = 0; u < C::units; u++) {
      const int k = kStreamKeys ? s : u;
      if (k % kGroups == group) {
        const uint32_t dst = kStreamKeys ? at.slots + s * at.slot : at.res + u * C::unit * kBlock;
        const bool ok = warp_wait<kPoll>(&br, &br.raw_full[k], kStreamKeys ? ph : tile & 1, p);
        if (u < C::units - 1) {
          if (!widen_unit<8>(dst, dst + kBlock, i, group, ok)) return false;
        } else if (!C::scaled) {
          if (!widen_unit<4>(dst, dst + kHalf, i, group, ok)) return false;
        } else if (bar_red_or(kWideBar + group, kGroupThreads, !ok)) {
          return false;
        }
        __syncwarp();
        if (first) mbar_arrive(smem_u32(at.rank == 1 ? &br.wide_full[k] : kStreamKeys ? &br.slot_full[k] : &br.res_full[k]));
      }
      if (++s == p.slots) {
        s = 0;
        ph ^= 1;
      }
    }
    tile++;
    return true;
  };
  for_each_phase<kStreamKeys, C::rows>(p, w, [&](const Phase &f) {
    for (int t = f.i0; t < (kStreamKeys ? f.i1 : min(f.i0 + 1, f.i1)); t++)
      if (!widen_tile()) return false;
    return true;
  });
}

// rank 1, two warps in turn that write nothing themselves: they pass on to rank 0 that units are widened.  What the
// widening warps have written is ordered before them by a barrier of this CTA, and before rank 0's MMA, which reads
// it, by their release at cluster scope, which takes some thousand cycles whatever there is to wait for.  (32 sequences
// of up to 8192 tokens, two query tokens, 64 heads, one scale: 38.3 us, with one such warp 40.8, with the
// release in the four widening warps 44.4; 33.2 with a release at the scope of the CTA, which orders
// nothing for rank 0.  With a scale for each 128 values 41.4 and 37.3; both with the copy of the sums, 1.5.)
template <bool kStreamKeys, int kFormat, bool kPoll>
__device__ void forward_role(const MassParams &p, Bars &br, const Work &w, int which) {
  using C = Of<kFormat>;
  const uint32_t full = mapa(smem_u32(kStreamKeys ? &br.slot_full[0] : &br.res_full[0]), 0);
  const bool first = (threadIdx.x & 31) == 0;
  int s = 0;
  uint32_t ph = 0, tile = 0;
  for_each_phase<kStreamKeys, C::rows>(p, w, [&](const Phase &f) {
    for (int t = f.i0; t < (kStreamKeys ? f.i1 : min(f.i0 + 1, f.i1)); t++, tile++)
      for (int u = 0; u < C::units; u++) {
        const int k = kStreamKeys ? s : u;
        if (k % 2 == which) {
          if (!warp_wait<kPoll>(&br, &br.wide_full[k], kStreamKeys ? ph : tile & 1, p)) return false;
          if (first) mbar_arrive_remote(full + k * 8);
        }
        if (++s == p.slots) {
          s = 0;
          ph ^= 1;
        }
      }
    return true;
  });
}

// ---- scores ------------------------------------------------------------------------

constexpr uint32_t kMmaBar = 1, kSumBar = 2;

// rank 0, warp 2 waits for what the MMAs of warp 1 need and meets it at a named
// barrier (a wait in the issuing warp would hold up its MMAs in flight).
template <bool kStreamKeys, int kFormat, bool kPoll>
__device__ void wait_role(const MassParams &p, Bars &br, const Work &w) {
  using C = Of<kFormat>;
  int s = 0;
  uint32_t ph = 0, rph = 0, g = 0;
  for_each_phase<kStreamKeys, C::rows>(p, w, [&](const Phase &f) {
    if (f.i0 >= f.i1) return true;
    for (int i = f.i0; i < f.i1; i++) {
      for (int u = 0; u < C::units; u++) {
        bool ok = true;
        if (C::begins(u)) {
          ok = warp_wait<kPoll>(&br, &br.d_empty[g % C::kd], ((g / C::kd) & 1) ^ 1, p);
          g++;
        }
        // (keys widened by threads of both CTAs)
        if (ok && i == f.i0) ok = warp_wait<kPoll, C::fp8 && !kStreamKeys>(&br, &br.res_full[u], rph, p);
        if (ok) ok = warp_wait<kPoll, C::fp8 && kStreamKeys>(&br, &br.slot_full[s], ph, p);
        if (bar_red_or(kMmaBar, 64, !ok)) return false;
        if (++s == p.slots) {
          s = 0;
          ph ^= 1;
        }
      }
    }
    rph ^= 1;
    return true;
  });
}

template <bool kStreamKeys, int kFormat>
__device__ void mma_role(const MassParams &p, Bars &br, const Work &w, const Place &at, uint32_t tmem) {
  using C = Of<kFormat>;
  const uint32_t idesc = IDESC + ((uint32_t)(p.box >> 3) << 17);
  int s = 0;
  uint32_t g = 0;
  for_each_phase<kStreamKeys, C::rows>(p, w, [&](const Phase &f) {
    if (f.i0 >= f.i1) return true;
    for (int i = f.i0; i < f.i1; i++) {
      for (int u = 0; u < C::units; u++) {
        if (bar_red_or(kMmaBar, 64, false)) return false;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int j = 0; j < C::unit; j++) {
            if (j >= C::blocks(u)) break;
            const uint64_t stay = smem_desc_sw128(at.res + (u * C::unit + j) * at.res_block, 16, 1024);
            const uint64_t pass = smem_desc_sw128(at.slots + s * at.slot + j * at.slot_block, 16, 1024);
            const uint64_t a = kStreamKeys ? pass : stay, b = kStreamKeys ? stay : pass;
#pragma unroll
            for (int kk = 0; kk < 4; kk++)
              mma_pair_ss(tmem + (g % C::kd) * C::rows, a + kk * 2, b + kk * 2, idesc, !C::begins(u) || j || kk ? 1u : 0u);
          }
          mma_commit_pair(smem_u32(&br.slot_empty[s]));
          if (i == f.i1 - 1) mma_commit_pair(smem_u32(&br.res_empty[u]));
          if (C::ends(u)) mma_commit_pair(smem_u32(&br.d_full[g % C::kd]));
        }
        __syncwarp();
        if (C::ends(u)) g++;
        if (++s == p.slots) s = 0;
      }
    }
    return true;
  });
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The warps from 4 on that sum: thread = key of the tile = lane of tensor memory (and,
// with scales, half of the columns).
template <bool kStreamKeys, int kFormat, bool kPoll>
__device__ void sum_role(const MassParams &p, Bars &br, const Work &w, uint32_t tmem, uint32_t rank, int pair_index) {
  using C = Of<kFormat>;
  constexpr int kD = C::kd, kRows = C::rows, kThreads = 32 * C::sum_warps;
  const int me = threadIdx.x - 128, lane = threadIdx.x & 31, i = me % kKeys, first = me / kKeys * C::cols;
  const uint32_t lt = tmem + ((uint32_t)(i & 96) << 16) + first;
  const uint32_t d_empty = mapa(smem_u32(&br.d_empty[0]), 0);
  uint32_t g = 0, buf = 0, tile = 0;
  const float scale = kFormat == MLA_KV_FP8_E4M3_TENSOR ? p.scale * __ldg(p.kv_scales) : p.scale;
  const float2 cs = make_float2(scale, scale), log2e = make_float2(LOG2E, LOG2E);
  auto set_rows = [&](const Phase &f, int qt) {
    buf ^= 1;
#pragma unroll
    for (int k = 0; k < kRows; k += kThreads) {
      if (k + me >= kRows) break;  // (whole warps)
      const int R = qt * kRows + k + me;
      int lim = 0;
      float nl = 0.f;
      if (R < p.rows) {
        const int t = R / p.H, h = R % p.H;
        const float l = __ldg(p.lse + ((size_t)f.b * p.H + h) * p.T + t);
        lim = l == -INFINITY ? 0 : row_kv_len(f.len, p.T, t, p.causal);
        nl = -l;
      }
      br.nl[buf][k + me] = nl;
      br.lim[buf][k + me] = lim;
      const int least = __reduce_min_sync(0xffffffffu, lim);
      if (lane == 0) br.least[buf][(k + me) / 32] = least;
    }
  };
  // exp(score - lse), the difference made before it is taken to base 2: its rounding then goes with
  // the difference, which is small where the weight is not
  auto weights = [&](float2 x, float2 nl) {
    const float2 y = mul2(fma2(x, cs, nl), log2e);
    return make_float2(ex2(y.x), ex2(y.y));
  };
  // the weights of 32 rows, from column c0 of the thread's on
  float2 acc[2];
  auto add32 = [&](const float2 (&v)[16], int c0, int key, int end) {
    const float4 *nl = reinterpret_cast<const float4 *>(&br.nl[buf][first + c0]);
    if (end <= br.least[buf][(first + c0) / 32]) {  // these rows see all the tile's keys
#pragma unroll
      for (int j = 0; j < 8; j++) {
        const float4 n = nl[j];
        acc[0] = add2(acc[0], weights(v[2 * j], make_float2(n.x, n.y)));
        acc[1] = add2(acc[1], weights(v[2 * j + 1], make_float2(n.z, n.w)));
      }
    } else {
      const int4 *lims = reinterpret_cast<const int4 *>(&br.lim[buf][first + c0]);
#pragma unroll
      for (int j = 0; j < 8; j++) {
        const float4 n = nl[j];
        const int4 lim = lims[j];
        const float2 a = weights(v[2 * j], make_float2(n.x, n.y)), b = weights(v[2 * j + 1], make_float2(n.z, n.w));
        acc[0] = add2(acc[0], make_float2(key < lim.x ? a.x : 0.f, key < lim.y ? a.y : 0.f));
        acc[1] = add2(acc[1], make_float2(key < lim.z ? b.x : 0.f, key < lim.w ? b.y : 0.f));
      }
    }
  };
  for_each_phase<kStreamKeys, kRows>(p, w, [&](const Phase &f) {
    if (kStreamKeys) set_rows(f, 0);
    float sum = 0.f;
    auto key_of = [&](int t) { return t * kTileKeys + (int)rank * kKeys + i; };
    // what a key had before is fetched while its scores are made
    float before = 0.f;
    // A key's page is looked up two tiles ahead, its scales are fetched one ahead.  (By TMA along
    // with the keys they came 2400 cycles after the first scores: 35 instead of 33 us for 32 sequences of 4400
    // tokens, 64 heads.)
    const int end_t = kStreamKeys ? f.i1 : f.t + 1;
    auto page_at = [&](int t) {
      const int n = key_of(t), page = t < end_t && n < f.len ? __ldg(p.block_table + (size_t)f.b * p.max_pages + n / PAGE) : -1;
      return page;
    };
    auto scales_at = [&](int t, int page) {
      return C::scaled && page >= 0 && page < p.num_pages
                 ? __ldg(reinterpret_cast<const float4 *>(p.kv_scales) + (size_t)page * PAGE + key_of(t) % PAGE)
                 : make_float4(0.f, 0.f, 0.f, 0.f);
    };
    int page = page_at(kStreamKeys ? f.i0 : f.t), next_page = page_at(kStreamKeys ? f.i0 + 1 : f.t + 1);
    float4 sc = scales_at(kStreamKeys ? f.i0 : f.t, page);
    auto prepare = [&](int t) {
      const int n = key_of(t);
      if (first > 0) return;
      if (f.whole && p.decay != 0.f && n < f.len) before = p.mass[(size_t)f.b * p.cap + n];
    };
    auto store = [&](int t, float v) {
      const int n = key_of(t);
      if (first > 0 || n >= f.len) return;
      if (page < 0 || page >= p.num_pages) v = 0.f;  // (told by the warps that load)
      if (f.whole) p.mass[(size_t)f.b * p.cap + n] = p.decay != 0.f ? fmaf(p.decay, before, v) : v;
      else p.partial[((size_t)pair_index * 2 + f.part) * kTileKeys + rank * kKeys + i] = v;
    };
    // the halves of a key's sum meet
    auto finish = [&](int t, float v, bool ok) {
      if (C::halves > 1) {
        if (first > 0) br.half[tile & 1][i] = v;
        if (bar_red_or(kSumBar, kThreads, !ok)) return false;
        v += br.half[tile & 1][i];
      }
      store(t, v);
      tile++;
      return true;
    };
    if (!kStreamKeys) prepare(f.t);
    for (int k = f.i0; k < f.i1; k++) {
      if (kStreamKeys) prepare(k);
      else set_rows(f, k);
      const float4 next_sc = scales_at(k + 1, kStreamKeys ? next_page : -1);
      const int after = kStreamKeys ? page_at(k + 2) : -1;
      bool ok = warp_wait<kPoll>(&br, &br.d_full[g % kD], (g / kD) & 1, p);
      if (bar_red_or(kSumBar, kThreads, !ok)) return false;
      tc_fence_after();
      const int key = key_of(kStreamKeys ? k : f.t);
      const int cols = p.rows - (kStreamKeys ? 0 : k * kRows) - first;  // of the thread's columns (may be more, or none)
      const int end = min((kStreamKeys ? k + 1 : f.t + 1) * kTileKeys, f.len);
      acc[0] = acc[1] = make_float2(0.f, 0.f);
      if constexpr (!C::scaled) {
        for (int c0 = 0; c0 < min(C::cols, cols); c0 += 32) {
          float2 v[16];
          __syncwarp();
          tmem_ld32(lt + (g % kD) * kRows + c0, *reinterpret_cast<uint32_t(*)[32]>(&v[0]));
          tmem_wait_ld();
          add32(v, c0, key, end);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote_relaxed(d_empty + (g % kD) * 8);
        g++;
      } else {
        float2 x[2][16];
#pragma unroll
        for (int part = 0; part < C::parts; part++) {
          if (part > 0 && ok) ok = warp_wait<kPoll>(&br, &br.d_full[g % kD], (g / kD) & 1, p);
          tc_fence_after();
          const float factor = part == 0 ? sc.x : part == 1 ? sc.y : part == 2 ? sc.z : part == 3 ? sc.w : 1.f;
          const float2 f2 = make_float2(factor, factor);
#pragma unroll
          for (int q = 0; q < 2; q++) {
            if (q * 32 < cols) {
              float2 v[16];
              __syncwarp();
              tmem_ld32(lt + (g % kD) * kRows + q * 32, *reinterpret_cast<uint32_t(*)[32]>(&v[0]));
              tmem_wait_ld();
#pragma unroll
              for (int j = 0; j < 16; j++) {
                float2 &to = x[q][j];
                to = part == 0 ? mul2(v[j], f2) : fma2(v[j], f2, to);
              }
            }
          }
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_remote_relaxed(d_empty + (g % kD) * 8);
          g++;
        }
#pragma unroll
        for (int c = 0; c < 2; c++)
          if (c * 32 < cols) add32(x[c], c * 32, key, end);
      }
      const float got = (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y);
      if (kStreamKeys) {
        if (!finish(k, got, ok)) return false;
        page = next_page, next_page = after, sc = next_sc;
      } else {
        sum += got;
        if (bar_red_or(kSumBar, kThreads, !ok)) return false;
      }
    }
    if (kStreamKeys) return true;
    if (f.i0 < f.i1) return finish(f.t, sum, true);
    store(f.t, 0.f);  // no row sees these keys
    return true;
  });
}

template <bool kStreamKeys, int kFormat, bool kPoll>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(Of<kFormat>::threads, 1)
    attention_mass_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap pe_map,
                          const __grid_constant__ CUtensorMap q_map, const MassParams p) {
  using C = Of<kFormat>;
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023u) {
    if (threadIdx.x == 0) atomicOr(p.status, MLA_STATUS_SMEM_ALIGN);
    return;
  }
  Bars &br = *reinterpret_cast<Bars *>(smem);
  const int warp = threadIdx.x >> 5;
  const int pair_index = (int)cluster_id_x(), pairs = (int)gridDim.x / 2;
  Place at;
  at.rank = cluster_ctarank();
  at.res = smem_u32(smem + OFF_RES);
  at.res_block = kStreamKeys ? p.box / 2 * 128 : kBlock;
  at.slots = at.res + kBlocks * at.res_block;
  at.slot_block = kStreamKeys ? kBlock : p.box / 2 * 128;
  at.slot = C::unit * at.slot_block;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kBlocks; i++) {
      mbar_init(smem_u32(&br.res_full[i]), C::fp8 && !kStreamKeys ? kGroupWarps + 1 : 1);
      mbar_init(smem_u32(&br.res_empty[i]), 1);
    }
    for (int i = 0; i < kMostSlots; i++) {
      mbar_init(smem_u32(&br.slot_full[i]), C::fp8 && kStreamKeys ? kGroupWarps + 1 : 1);
      mbar_init(smem_u32(&br.slot_empty[i]), 1);
      mbar_init(smem_u32(&br.raw_full[i]), 1);
      mbar_init(smem_u32(&br.wide_full[i]), kGroupWarps);
    }
    for (int i = 0; i < C::kd; i++) {
      mbar_init(smem_u32(&br.d_full[i]), 1);
      mbar_init(smem_u32(&br.d_empty[i]), 2 * C::sum_warps);
    }
    br.abort = 0;
    br.start_b = br.start_t = 0;
    fence_mbar_init_cluster();
    prefetch_tensormap(&q_map);
    prefetch_tensormap(&k_map);
  }
  if (warp == 1) {
    tmem_alloc_pair(smem_u32(&br.tmem_base), 512);
    tmem_relinquish_pair();
  }
  grid_dep_trigger();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  cluster_sync();  // the peer's barriers exist before anything arrives on them
  const uint32_t tmem = br.tmem_base;
  grid_dep_wait();
  const Work w = find_work(p, br, pair_index, pairs);
  if (warp < 4) {
    if constexpr (C::scaled) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kLoadRegs));
    if (warp == 0 || warp == 3) load_role<kStreamKeys, kFormat, kPoll>(p, br, &k_map, &pe_map, &q_map, w, at, warp == 3);
    else if (at.rank == 0 && warp == 1) mma_role<kStreamKeys, kFormat>(p, br, w, at, tmem);
    else if (at.rank == 0 && warp == 2) wait_role<kStreamKeys, kFormat, kPoll>(p, br, w);
    else if (C::fp8 && (warp == 1 || warp == 2)) forward_role<kStreamKeys, kFormat, kPoll>(p, br, w, warp - 1);
  } else if (warp < 4 + C::sum_warps) {
    if constexpr (C::scaled) asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSumRegs));
    sum_role<kStreamKeys, kFormat, kPoll>(p, br, w, tmem, at.rank, pair_index);
  } else if constexpr (C::fp8) {
    if constexpr (C::scaled) asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kWideRegs));
    widen_role<kStreamKeys, kFormat, kPoll>(p, br, w, at, threadIdx.x - 32 * (4 + C::sum_warps));
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (br.abort) {  // copies and MMAs in flight end
    const uint64_t t0 = globaltimer();
    while (globaltimer() - t0 < 2000000ull) {
    }
  }
  __syncwarp();
  cluster_sync();  // nothing of the peer's reads or arrives here any more
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

// Sums of tiles that several pairs have a part of, in the order of the pairs.  Block
// p: the tile that begins in pair p and ends in another.
__global__ void __launch_bounds__(kTileKeys) mass_reduce_kernel(MassParams p, int pairs) {
  __shared__ int warp_sums[32], found[2];
  grid_dep_wait();
  const Tiles t = count_tiles(p, warp_sums);
  const long long units = (long long)t.total * p.n_qt;
  const int pair = blockIdx.x;
  const long long u0 = first_unit(units, pair, pairs), u1 = first_unit(units, pair + 1, pairs);
  if (u0 >= u1) return;
  const long long tile = (u1 - 1) / p.n_qt, first = tile * p.n_qt, end = first + p.n_qt;
  if (first < u0 || end <= u1) return;  // begins before this pair, or is whole
  find_tile(p, t, (int)tile, &found[0], &found[1]);
  __syncthreads();
  const int b = found[0], n = found[1] * kTileKeys + threadIdx.x;
  if (n >= seq_len(p, b)) return;
  float v = p.partial[((size_t)pair * 2 + 1) * kTileKeys + threadIdx.x];
  for (int q = pair + 1; q < pairs && first_unit(units, q, pairs) < end; q++)
    if (first_unit(units, q, pairs) < first_unit(units, q + 1, pairs)) v += p.partial[(size_t)q * 2 * kTileKeys + threadIdx.x];
  float *m = p.mass + (size_t)b * p.cap + n;
  *m = p.decay != 0.f ? fmaf(p.decay, *m, v) : v;
}

int fail(int code, const char *msg) {
  set_last_error(msg);
  return code;
}

bool aligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

int check_sizes(int B, int T, int H, int cap) {
  char msg[160];
  if (B < 1 || B > MLA_MAX_ITEMS || T < 1 || H < 1 || H > MLA_MAX_HEADS || cap < 1) {
    snprintf(msg, sizeof msg, "B = %d not in [1, %d], T = %d < 1, H = %d not in [1, %d] or mass_cap = %d < 1", B,
             MLA_MAX_ITEMS, T, H, MLA_MAX_HEADS, cap);
    return fail(MLA_ERR_INVALID_ARG, msg);
  }
  if ((long long)B * T * H > 0x7fffff00LL) return fail(MLA_ERR_UNSUPPORTED, "B * T * H exceeds 2^31 - 256 query rows");
  if (cap > (1 << 24)) return fail(MLA_ERR_UNSUPPORTED, "mass_cap exceeds 2^24");
  return MLA_OK;
}

int sm_pairs(int *pairs) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return fail(MLA_ERR_CUDA, cudaGetErrorString(e));
  *pairs = sms / 2 > 0 ? sms / 2 : 1;
  return MLA_OK;
}

// Room for the partial sums of twice as many pairs as any GPU of this kind has.
constexpr size_t kMostPairs = 160;

// Warpgroups that ask for more registers than the block was launched with wait for ever.
// Looked at once for each of the four kernels.
cudaError_t registers_suffice(const void *kernel, int threads, bool keys, bool poll) {
  static std::atomic<int> seen[4];
  std::atomic<int> &s = seen[2 * keys + poll];
  if (s.load(std::memory_order_relaxed)) return cudaSuccess;
  cudaFuncAttributes a;
  const cudaError_t e = cudaFuncGetAttributes(&a, kernel);
  if (e != cudaSuccess) return e;
  using C = Of<MLA_KV_FP8_E4M3>;
  if (a.numRegs * threads < 32 * (4 * kLoadRegs + C::sum_warps * kSumRegs + C::wide_warps * kWideRegs)) return cudaErrorLaunchOutOfResources;
  s.store(1, std::memory_order_relaxed);
  return cudaSuccess;
}

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" size_t mla_attention_mass_workspace_bytes(int B, int T, int H, int mass_cap) {
  if (check_sizes(B, T, H, mass_cap) != MLA_OK) return 0;
  // (a tile of query rows of the format with most tiles)
  return T * H <= Of<MLA_KV_FP8_E4M3>::rows ? 0 : kMostPairs * 2 * kTileKeys * sizeof(float);
}

extern "C" int mla_attention_mass(const void *q, const void *kv_cache, int kv_format, int num_pages, int page_size,
                                  const int32_t *block_table, int max_pages, const int32_t *cache_seqlens,
                                  const float *kv_scales, const float *lse, float softmax_scale, int causal, float decay,
                                  float *mass, int mass_cap, void *workspace, size_t workspace_bytes, int B, int T, int H,
                                  mla_stream_t stream) {
  int rc = check_sizes(B, T, H, mass_cap);
  if (rc != MLA_OK) return rc;
  if (!q || !kv_cache || !block_table || !cache_seqlens || !lse || !mass)
    return fail(MLA_ERR_INVALID_ARG, "null pointer argument");
  if (kv_format != MLA_KV_BF16 && kv_format != MLA_KV_FP8_E4M3 && kv_format != MLA_KV_FP8_E4M3_TENSOR)
    return fail(MLA_ERR_INVALID_ARG, "kv_format unknown");
  if (!aligned(q, 16) || !aligned(kv_cache, 16)) return fail(MLA_ERR_INVALID_ARG, "q and kv_cache must be 16-byte aligned");
  if (!aligned(block_table, 4) || !aligned(cache_seqlens, 4) || !aligned(lse, 4) || !aligned(mass, 4))
    return fail(MLA_ERR_INVALID_ARG, "int32/fp32 arrays must be 4-byte aligned");
  if (kv_format != MLA_KV_BF16 && (!kv_scales || !aligned(kv_scales, kv_format == MLA_KV_FP8_E4M3 ? 16 : 4)))
    return fail(MLA_ERR_INVALID_ARG, "an FP8 cache needs aligned kv_scales");
  if (page_size != MLA_PAGE_SIZE) return fail(MLA_ERR_UNSUPPORTED, "page_size must be 64");
  if (num_pages < 1 || max_pages < 1) return fail(MLA_ERR_INVALID_ARG, "num_pages/max_pages < 1");
  if (causal != 0 && causal != 1) return fail(MLA_ERR_INVALID_ARG, "causal must be 0 or 1");
  if (!(softmax_scale > 0.f) || !std::isfinite(softmax_scale))
    return fail(MLA_ERR_INVALID_ARG, "softmax_scale must be finite and > 0");
  if (!(decay >= 0.f) || !std::isfinite(decay)) return fail(MLA_ERR_INVALID_ARG, "decay must be finite and >= 0");
  const size_t need = mla_attention_mass_workspace_bytes(B, T, H, mass_cap);
  if (need && (!workspace || workspace_bytes < need)) {
    char msg[96];
    snprintf(msg, sizeof msg, "workspace needs %zu bytes, got %zu", need, workspace_bytes);
    return fail(MLA_ERR_WORKSPACE, msg);
  }
  if (need && !aligned(workspace, 256)) return fail(MLA_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  MassParams p{};
  if ((rc = status_word(&p.status)) != MLA_OK) return rc;
  int pairs = 0;
  if ((rc = sm_pairs(&pairs)) != MLA_OK) return rc;
  if (need && (size_t)pairs > kMostPairs) return fail(MLA_ERR_UNSUPPORTED, "more SMs than the workspace has room for");
  p.kv_scales = kv_scales;
  p.block_table = block_table;
  p.seqlens = cache_seqlens;
  p.lse = lse;
  p.mass = mass;
  p.partial = need ? static_cast<float *>(workspace) : nullptr;
  p.num_pages = num_pages;
  p.max_pages = max_pages;
  p.B = B;
  p.T = T;
  p.H = H;
  p.cap = mass_cap;
  p.causal = causal;
  p.rows = T * H;
  const int tile_rows = kv_format == MLA_KV_FP8_E4M3 ? Of<MLA_KV_FP8_E4M3>::rows : kMostRows;
  p.n_qt = ceil_div(p.rows, tile_rows);
  p.box = p.rows < tile_rows ? ceil_div(p.rows, 16) * 16 : tile_rows;
  p.scale = softmax_scale;
  p.decay = decay;
  p.wait_ns = wait_limit_ns();

  CUtensorMap k_map{}, pe_map{}, q_map{};
  auto fn = tensor_map_encoder();
  if (!fn) return fail(MLA_ERR_CUDA, "cuTensorMapEncodeTiled not found");
  bool ok = make_map_3d(&q_map, q, 64, (uint64_t)B * p.rows, kBlocks, D_QK, 64, p.box / 2, 1);
  if (ok && kv_format == MLA_KV_BF16) {
    cuuint64_t dims[4] = {64, (cuuint64_t)PAGE, kBlocks, (cuuint64_t)num_pages};
    cuuint64_t strides[3] = {(cuuint64_t)D_QK * 2, 128, (cuuint64_t)D_QK * 2 * PAGE};
    cuuint32_t box[4] = {64, (cuuint32_t)PAGE, 1, 1}, estr[4] = {1, 1, 1, 1};
    ok = fn(&k_map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(kv_cache), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  } else if (ok) {
    // codes, 128 of each row of a page at a time
    const cuuint64_t row = kv_format == MLA_KV_FP8_E4M3 ? FP8_ROW : D_QK;
    cuuint64_t dims[3] = {row, (cuuint64_t)PAGE, (cuuint64_t)num_pages}, strides[2] = {row, row * PAGE};
    cuuint32_t box[3] = {128, (cuuint32_t)PAGE, 1}, estr[3] = {1, 1, 1};
    auto codes = [&](CUtensorMap *map) {
      return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(kv_cache), dims, strides, box, estr,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
    };
    ok = codes(&k_map);
    // the rotated part: 64 codes, or 64 bf16 behind the codes
    box[0] = 64;
    if (ok && kv_format == MLA_KV_FP8_E4M3_TENSOR) ok = codes(&pe_map);
    if (ok && kv_format == MLA_KV_FP8_E4M3)
      ok = make_map_3d(&pe_map, static_cast<const uint8_t *>(kv_cache) + D_V, 64, PAGE, (uint64_t)num_pages, FP8_ROW / 2,
                       PAGE * FP8_ROW / 2, PAGE, 1);
  }
  if (!ok) return fail(MLA_ERR_CUDA, "a tensor map could not be made");
  const uint32_t q_block = p.box / 2 * 128, unit = kv_format == MLA_KV_BF16 ? 1 : 2;
  const uint32_t resident = kBlocks * (p.n_qt == 1 ? q_block : kBlock);
  p.slots = (int)((kRoom - resident) / (unit * (p.n_qt == 1 ? kBlock : q_block)));
  if (p.slots > kMostSlots) p.slots = kMostSlots;
  if (kv_format != MLA_KV_BF16) p.slots -= p.slots % kGroups;
  cudaError_t e = cudaSuccess;
  const bool keys = p.n_qt == 1, poll = p.wait_ns < kShortWaitNs;
  using Kernel = void (*)(CUtensorMap, CUtensorMap, CUtensorMap, MassParams);
  Kernel k = nullptr;
  int threads = 0;
#define PICK(format)                                                                                              \
  case format:                                                                                                    \
    k = keys ? (poll ? attention_mass_kernel<true, format, true> : attention_mass_kernel<true, format, false>)    \
             : (poll ? attention_mass_kernel<false, format, true> : attention_mass_kernel<false, format, false>); \
    threads = Of<format>::threads;                                                                                \
    break
  switch (kv_format) {
    PICK(MLA_KV_BF16);
    PICK(MLA_KV_FP8_E4M3);
    PICK(MLA_KV_FP8_E4M3_TENSOR);
  }
#undef PICK
  cudaStream_t s = (cudaStream_t)stream;
  if (e == cudaSuccess && kv_format == MLA_KV_FP8_E4M3) e = registers_suffice(reinterpret_cast<const void *>(k), threads, keys, poll);
  if (e == cudaSuccess) e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
  if (e == cudaSuccess) e = launch_dependent(k, 2 * pairs, threads, kSmem, s, k_map, pe_map, q_map, p);
  if (e == cudaSuccess && p.n_qt > 1) e = launch_dependent(mass_reduce_kernel, pairs, kTileKeys, 0, s, p, pairs);
  if (e != cudaSuccess) {
    char msg[128];
    snprintf(msg, sizeof msg, "attention mass: %s", cudaGetErrorString(e));
    return fail(MLA_ERR_CUDA, msg);
  }
  set_last_error("");
  return MLA_OK;
}

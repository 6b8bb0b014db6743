// KV expansion: cached latent rows to the keys and values of every head, for
// the attention of prompts (mla_prefill).  Packed output row r belongs to
// sequence b with cu[b] <= r < cu[b + 1] and holds token pos = r - cu[b],
// found at page block_table[b][pos / 64], slot pos % 64:
//   kv[r][h][0:128]   = bf16(W_UK[h] . c)       (128 no-PE key values)
//   kv[r][h][128:256] = bf16(W_UV[h] . c)       (128 values)
//   k_pe[r]           = the row's 64 rotated key values
// with c the row's 512 latent values.
//
// As one GEMM with gathered rows: M = rows of the packed output, N = 256 (one
// head: its W_UK rows, then its W_UV rows), K = 512.  2 * 512 flops per
// 2-byte output value are above the ridge, so with many rows it is bound by
// the tensor cores, with the output's write close behind; with few rows by
// the read of the weights (16384 rows, 128 heads: 364 us in a long run of calls, 325
// us, 1.7 PFLOP/s, over fifty from rest; 100 rows, 64 heads: 10.4 us with the
// weights in L2, 11.9 us without).  Figures below that compare two forms were
// taken side by side when the choice was made.
//
// Roundings: bf16 rows are used as they are.  A row with per-128 scales is
// dequantised to bf16 (one rounding, the one the decode makes too: the MMA's
// operands have one type, and four partial sums, which could take the row's four
// scales, would need four times the tensor memory and drain).
// The codes of a one-scale cache are exact in bf16, so there the scale
// multiplies the fp32 sum.  Sums are fp32 in tensor memory, rounded once.
#include <cuda_fp8.h>

#include "common.cuh"
#include "dependent.cuh"
#include "ptx.cuh"
#include "ptx_pair.cuh"
#include "tma_map.cuh"

namespace mla {
namespace {

using namespace ptx;

struct ExpandParams {
  const uint8_t *cache;
  const float *scales;
  const int32_t *block_table;
  const int32_t *cu;
  __nv_bfloat16 *kv;    // [total][H][256]
  __nv_bfloat16 *k_pe;  // [total][64]
  unsigned int *status;
  int format, num_pages, max_pages, B, H, total;
  unsigned long long wait_ns;  // limit of every wait
};

// A cluster of two CTAs works as one: M = 256 rows, 128 gathered by each CTA;
// of the N = 256 weight rows of a head rank 0 fetches W_UK[h] and rank 1
// W_UV[h], and each MMA reads both.  One CTA alone would take 32 KB of weights
// from L2 for every 64 latent values (64 bytes a cycle and SM at the tensor
// cores' pace, more than L2 gives); a pair takes half of that.
//
// Warps 0-7 gather the rows (A) and drain D, warp 8 loads the weights, warp 9
// of rank 0 issues the MMAs.  A pair walks over (row block, head) units, heads
// innermost, so A (128 rows x 512, 128 KB) stays in shared memory for all heads
// of a block while the weights stream through a ring; D is double buffered in
// tensor memory, so a unit is drained while the next one is computed.
constexpr int kRowWarps = 8;
constexpr int kThreads = 32 * (kRowWarps + 2);
constexpr int kM = 128;                       // rows of a CTA
constexpr int kPairRows = 2 * kM;
constexpr int kKBlocks = 8;
constexpr uint32_t kABlock = kM * 128;        // 64 latent values x 128 rows
constexpr uint32_t kWStage = 128 * 128;       // 64 latent values x this CTA's 128 weight rows
constexpr int kWStages = 4;
constexpr uint32_t kOutBytes = 32 * 128;      // 32 rows x 64 columns of the output, on their way out
constexpr uint32_t OFF_W = kKBlocks * kABlock;
constexpr uint32_t OFF_OUT = OFF_W + kWStages * kWStage;  // boxes of the draining warps
constexpr uint32_t OFF_BARS = OFF_OUT + kRowWarps * kOutBytes;
constexpr uint32_t IDESC = idesc_bf16_f32(256, 256, false, false);

struct Bars {
  uint64_t w_full[kWStages];   // rank 0: the stage of both CTAs
  uint64_t w_empty[kWStages];
  uint64_t a_full;             // rank 0: the rows of both CTAs
  uint64_t d_full[2];
  uint64_t d_empty[2];         // rank 0: drained by both CTAs
  int source[3][kM];           // the cache rows of three blocks of rows in turn (a warp may be two units behind)
  uint32_t tmem_base;
  int abort;
};
constexpr uint32_t kSmem = OFF_BARS + sizeof(Bars) + 1024;
static_assert(kSmem <= 232448, "shared memory budget");

template <bool kPoll>
__device__ __forceinline__ bool wait_ok(Bars *b, uint64_t *bar, uint32_t parity, const ExpandParams &p) {
  if (mbar_wait_limited<true, kPoll>(smem_u32(bar), parity, &b->abort, p.wait_ns)) return true;
  atomicOr(p.status, MLA_STATUS_WAIT_TIMEOUT);
  *(volatile int *)&b->abort = 1;
  return false;
}

// A pair's units, [u0, u1) of (row block, head) in rows of H heads, in the order
// it works through them: the last block's first heads, the first block's last
// heads, then the blocks between.  All pairs then come by the same heads at
// about the same time and find their weights in L2; the output's stream, which
// would push them out, is marked to leave first (16384 rows, 128 heads: 420 us
// in plain order with or without that mark, 427 us in this order without it,
// 335 us with it).
struct Order {
  int u0, u1, H;
  __device__ __forceinline__ int unit(int i) const {
    const int first = u0 / H, last = (u1 - 1) / H;
    if (first == last) return u0 + i;
    const int n_last = u1 - last * H, n_first = (first + 1) * H - u0;
    if (i < n_last) return last * H + i;
    if (i < n_last + n_first) return u0 + (i - n_last);
    return (first + 1) * H + (i - n_last - n_first);
  }
  // does unit i need other rows than the one before?
  __device__ __forceinline__ bool new_rows(int i) const { return i == 0 || unit(i) / H != unit(i - 1) / H; }
};

// The cache rows of the packed rows r0 + lane % 16: the row's index
// in the pool, -1 for one that cannot be read (written as zeros) and -2 for one
// that belongs to no sequence (left as it was).
__device__ int row_source(const ExpandParams &p, int r0, int lane) {
  const int r = r0 + (lane & 15);
  // the last sequence that starts at or before r0, by 32 probes at a time ...
  int lo = 0, hi = p.B;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32, at = lo + (lane + 1) * step;
    const bool before = at < hi && __ldg(p.cu + at) <= r0;
    lo += __popc(__ballot_sync(0xffffffffu, before)) * step;
    hi = min(hi, lo + step);
  }
  // ... and from there each lane's own
  int start = __ldg(p.cu + lo), end = __ldg(p.cu + lo + 1);
  if (lo + 1 < p.B && end <= r) {
    int top = p.B;
    while (top - lo > 1) {
      const int mid = (lo + top) >> 1;
      if (__ldg(p.cu + mid) <= r) lo = mid; else top = mid;
    }
    start = __ldg(p.cu + lo);
    end = __ldg(p.cu + lo + 1);
  }
  if (r >= p.total) return -2;
  if (start < 0 || end > p.total || end < start) atomicOr(p.status, MLA_STATUS_BAD_SEQLEN);
  if (start < 0 || r < start || r >= end) return -2;
  const int pos = r - start;
  if (pos / PAGE >= p.max_pages) {
    atomicOr(p.status, MLA_STATUS_BAD_SEQLEN);
    return -1;
  }
  const int page = __ldg(p.block_table + (size_t)lo * p.max_pages + pos / PAGE);
  if (page < 0 || page >= p.num_pages) {
    atomicOr(p.status, MLA_STATUS_BAD_PAGE);
    return -1;
  }
  return page * PAGE + pos % PAGE;  // (the host has checked that the pool's rows fit)
}

// 16 e4m3 codes times sc -> 16 bf16 (the products rounded once).
__device__ __forceinline__ void dequant(const uint4 &v, float sc, uint32_t (&o)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 8; i++) {
    const uint16_t two = (uint16_t)(w[i >> 1] >> (16 * (i & 1)));
    const __half2 h2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3));
    const float2 f = __half22float2(h2);
    __nv_bfloat162 b = __floats2bfloat162_rn(f.x * sc, f.y * sc);
    o[i] = *reinterpret_cast<uint32_t *>(&b);
  }
}

// Byte offset of 16-byte piece c (0..63) of row r in the swizzled A blocks.
__device__ __forceinline__ uint32_t a_off(int r, int c) {
  return (uint32_t)(c >> 3) * kABlock + (uint32_t)r * 128 + (uint32_t)(((c & 7) ^ (r & 7)) << 4);
}

// 16 bytes, or 16 zero bytes where `bytes` is 0 (nothing is read then).
__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, uint32_t bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(src)),
               "r"(bytes)
               : "memory");
}

// Warp w fetches rows 16w .. 16w + 15 of the block at row0 into A; src: row
// lane % 16's.  With `pe` it also writes the rows' k_pe.  All of the warp's
// rows are on their way at once (8 to 16 KB): fetched eight rows at a time a
// block took 16000 cycles, four memory latencies under load.
__device__ void gather_rows(const ExpandParams &p, uint8_t *a, int row0, int warp, int lane, int src, bool pe) {
  const uint32_t sa = smem_u32(a);
  const bool bf16 = p.format == MLA_KV_BF16, tile = p.format == MLA_KV_FP8_E4M3;
  const int row_bytes = bf16 ? 2 * D_QK : tile ? FP8_ROW : D_QK;
  // Latent values: bf16 rows straight to their place, codes into the upper
  // half of it (pieces 32..63), from where they are expanded below, and the
  // four scales of a row into its first piece.
#pragma unroll 4
  for (int i = 0; i < 16; i++) {  // (no branches: the addresses of four rows at a time)
    const int s = __shfl_sync(0xffffffffu, src, i);
    const int r = warp * 16 + i;
    const uint8_t *row = p.cache + (size_t)(s < 0 ? 0 : s) * row_bytes + lane * 16;
    const uint32_t bytes = s < 0 ? 0u : 16u;
    cp_async16(sa + a_off(r, 32 + lane), row + (bf16 ? 512 : 0), bytes);
    if (bf16) cp_async16(sa + a_off(r, lane), row, bytes);
    if (tile && lane == 0) cp_async16(sa + a_off(r, 0), p.scales + (size_t)(s < 0 ? 0 : s) * 4, bytes);
  }
  if (pe) {  // four rows at a time, eight lanes each
    const int sub = lane & 7;
    const float one = p.format == MLA_KV_FP8_E4M3_TENSOR ? __ldg(p.scales) : 1.f;
    uint4 q[4];
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const int s = __shfl_sync(0xffffffffu, src, 4 * i + (lane >> 3));
      const uint8_t *at = p.cache + (size_t)(s < 0 ? 0 : s) * row_bytes + (bf16 ? 2 * D_V : D_V);
      q[i] = make_uint4(0u, 0u, 0u, 0u);
      if (s >= 0) {
        if (bf16 || tile) {
          q[i] = __ldg(reinterpret_cast<const uint4 *>(at) + sub);
        } else {  // eight codes a lane
          const uint2 v = __ldg(reinterpret_cast<const uint2 *>(at) + sub);
          uint32_t o[8];
          dequant(make_uint4(v.x, v.y, 0u, 0u), one, o);
          q[i] = make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; i++) {
      const int s = __shfl_sync(0xffffffffu, src, 4 * i + (lane >> 3));
      if (s != -2)
        reinterpret_cast<uint4 *>(p.k_pe + (size_t)(row0 + warp * 16 + 4 * i + (lane >> 3)) * D_ROPE)[sub] = q[i];
    }
  }
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncwarp();
  if (bf16) return;
  // (little code: it runs once or twice a launch, and unrolled further it costs
  // more in instruction fetches than it hides)
  const int t = lane >> 3;
  uint4 next = *reinterpret_cast<const uint4 *>(a + a_off(warp * 16, 32 + lane));
  float next_scale = tile ? *reinterpret_cast<const float *>(a + a_off(warp * 16, 0) + 4 * t) : 1.f;
#pragma unroll 2
  for (int i = 0; i < 16; i++) {
    const int r = warp * 16 + i;
    const uint4 v = next;
    const float scale = next_scale;
    if (i < 15) {
      next = *reinterpret_cast<const uint4 *>(a + a_off(r + 1, 32 + lane));
      if (tile) next_scale = *reinterpret_cast<const float *>(a + a_off(r + 1, 0) + 4 * t);
    }
    uint32_t o[8];
    dequant(v, scale, o);
    __syncwarp();  // the row's codes are all read before its values are written
    *reinterpret_cast<uint4 *>(a + a_off(r, 2 * lane)) = make_uint4(o[0], o[1], o[2], o[3]);
    *reinterpret_cast<uint4 *>(a + a_off(r, 2 * lane + 1)) = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

template <bool kPoll>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    expand_kernel(const __grid_constant__ CUtensorMap uk_map, const __grid_constant__ CUtensorMap uv_map,
                  const __grid_constant__ CUtensorMap o_map, ExpandParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *base = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  Bars *br = reinterpret_cast<Bars *>(base + OFF_BARS);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  const long long units = (long long)ceil_div(p.total, kPairRows) * p.H;
  const Order order = {(int)(units * pair / pairs), (int)(units * (pair + 1) / pairs), p.H};
  const int n = order.u1 - order.u0;
  // With many units a pair, D is drained while the next unit is computed, by
  // four warps with two boxes each; with few it is waited for, and all eight
  // drain (100 rows, 64 heads: 10.6 us instead of 12.6; 16384 rows, 128 heads:
  // 338 instead of 322 us).
  const bool few = n <= 2;
  if (warp == 0) {
    tmem_alloc_pair(smem_u32(&br->tmem_base), 512);
    tmem_relinquish_pair();
  }
  if (threadIdx.x == 32) {
    for (int s = 0; s < kWStages; s++) {
      mbar_init(smem_u32(&br->w_full[s]), 1);
      mbar_init(smem_u32(&br->w_empty[s]), 1);
    }
    mbar_init(smem_u32(&br->a_full), 2 * kRowWarps);
    for (int s = 0; s < 2; s++) {
      mbar_init(smem_u32(&br->d_full[s]), 1);
      mbar_init(smem_u32(&br->d_empty[s]), 2 * kRowWarps);
    }
    br->abort = 0;
    fence_mbar_init_cluster();
  }
  if (threadIdx.x == kRowWarps * 32) {
    prefetch_tensormap(rank == 0 ? &uk_map : &uv_map);
    prefetch_tensormap(&o_map);
  }
  grid_dep_trigger();
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // both CTAs' barriers are there
  tc_fence_after();
  grid_dep_wait();  // nothing of the caller's is read or written before the kernel in front has ended
  const uint32_t tmem = br->tmem_base;
  const uint32_t sa = smem_u32(base), sw = sa + OFF_W;

  if (warp < kRowWarps) {
    const float out_scale = p.format == MLA_KV_FP8_E4M3_TENSOR ? __ldg(p.scales) : 1.f;
    const int quarter = warp & 3;  // of D: 32 rows
    const int c0 = few ? 2 * (warp >> 2) : 0, c1 = few ? c0 + 2 : warp < 4 ? 4 : 0;  // and 64 columns each
    const uint32_t lane_base = tmem + ((uint32_t)(quarter * 32) << 16);
    const uint64_t pol_out = policy_evict_first();
    uint32_t blocks = 0;
    // this block's rows
    auto gather = [&](int u) {
      const int row0 = u / p.H * kPairRows + (int)rank * kM;
      const int src = row_source(p, row0 + warp * 16, lane);
      if (lane < 16) br->source[blocks % 3][warp * 16 + lane] = src;
      gather_rows(p, base, row0, warp, lane, src, u % p.H == 0);
      blocks++;
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote(mapa(smem_u32(&br->a_full), 0));
    };
    if (n > 0) gather(order.unit(0));
    int mine = -2;
    for (int i = 0; i < n; i++) {
      const int u = order.unit(i), buf = i & 1;
      const bool ok = __all_sync(0xffffffffu, wait_ok<kPoll>(br, &br->d_full[buf], (i >> 1) & 1, p));
      if (!ok) break;
      tc_fence_after();
      if (order.new_rows(i)) mine = br->source[(blocks - 1) % 3][quarter * 32 + lane];
      const int row = u / p.H * kPairRows + (int)rank * kM + quarter * 32 + lane, h = u % p.H;
      // the next unit's rows first: every MMA that reads A has completed
      if (i + 1 < n && order.new_rows(i + 1)) gather(order.unit(i + 1));
      // Rows go out as boxes of 32 rows x 64 columns through shared memory, by
      // TMA (rows behind the last of the output are clipped): stores of a
      // lane's own row, 32 bytes at a time, took 6600 cycles a unit, longer
      // than its MMAs.  Where a row belongs to no sequence each lane stores its own.
      const bool whole = __all_sync(0xffffffffu, mine != -2 || row >= p.total);
      uint8_t *dst = reinterpret_cast<uint8_t *>(p.kv + ((size_t)row * p.H + h) * 256);
#pragma unroll 1
      for (int c = c0; c < c1; c++) {
        uint32_t v[2][32];
        __syncwarp();  // the loads are the whole warp's, and its lanes may have stored apart from each other
        tmem_ld32(lane_base + buf * 256 + 64 * c, v[0]);
        tmem_ld32(lane_base + buf * 256 + 64 * c + 32, v[1]);
        uint8_t *out = base + OFF_OUT + (few ? warp : 2 * warp + (c & 1)) * kOutBytes;
        if (lane == 0) {  // the last box from this place is out
          if (few) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
          else asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
        }
        __syncwarp();
        tmem_wait_ld();
        __syncwarp();
#pragma unroll
        for (int k = 0; k < 8; k++) {
          uint32_t w[4];
#pragma unroll
          for (int j = 0; j < 4; j++) {
            const uint32_t *x = &v[k >> 2][8 * (k & 3) + 2 * j];
            __nv_bfloat162 b2 = __floats2bfloat162_rn(__uint_as_float(x[0]) * out_scale, __uint_as_float(x[1]) * out_scale);
            w[j] = *reinterpret_cast<uint32_t *>(&b2);
          }
          const uint4 piece = make_uint4(w[0], w[1], w[2], w[3]);
          if (whole) {
            *reinterpret_cast<uint4 *>(out + lane * 128 + ((k ^ (lane & 7)) << 4)) = piece;
          } else if (mine != -2) {
            *reinterpret_cast<uint4 *>(dst + 128 * c + 16 * k) = piece;
          }
        }
        if (whole) {
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            const int first = row;  // lane 0's
            if (first < p.total)
              asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group.L2::cache_hint [%0, {%2, %3, %4}], [%1], %5;" ::"l"(
                               reinterpret_cast<uint64_t>(&o_map)),
                           "r"(smem_u32(out)), "r"(64 * c), "r"(h), "r"(first), "l"(pol_out)
                           : "memory");
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      // relaxed: nothing but tensor memory has been read, and the releasing
      // form would wait for the output's way to memory (3700 cycles a unit)
      // (also from a warp that drains nothing: d_full must not run a phase ahead of it)
      if (lane == 0) mbar_arrive_remote_relaxed(mapa(smem_u32(&br->d_empty[buf]), 0));
    }
    if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
  } else if (warp == kRowWarps) {
    const uint64_t pol = policy_evict_normal();
    const CUtensorMap *map = rank == 0 ? &uk_map : &uv_map;
    uint32_t k = 0;
    bool ok = true;
    for (int i = 0; i < n && ok; i++) {
      const int h = order.unit(i) % p.H;
      for (int kb = 0; kb < kKBlocks; kb++, k++) {
        const uint32_t s = k % kWStages, dst = sw + s * kWStage;
        ok = __all_sync(0xffffffffu, wait_ok<kPoll>(br, &br->w_empty[s], ((k / kWStages) & 1) ^ 1, p));
        if (!ok) break;
        if (elect_one()) {
          if (rank == 0) mbar_arrive_expect_tx(smem_u32(&br->w_full[s]), 2 * kWStage);
          tma_load_3d_pair(dst, map, mapa(smem_u32(&br->w_full[s]), 0), 64 * kb, 0, h, pol);
        }
        __syncwarp();
      }
    }
  } else if (rank == 0) {
    // The whole warp waits and one elected lane issues: with the loop in a
    // branch of one lane every wait drains the MMAs (4 MMAs of 256 columns and
    // a wait: 627 cycles, against 514 of the MMAs alone).
    uint32_t k = 0, na = 0;
    bool ok = true;
    auto wait = [&](uint64_t *bar, uint32_t parity) {
      ok = ok && __all_sync(0xffffffffu, wait_ok<kPoll>(br, bar, parity, p));
    };
    for (int i = 0; i < n && ok; i++) {
      const int buf = i & 1;
      if (order.new_rows(i)) wait(&br->a_full, na++ & 1);
      wait(&br->d_empty[buf], ((i >> 1) & 1) ^ 1);
      for (int kb = 0; kb < kKBlocks; kb++, k++) {
        const uint32_t s = k % kWStages;
        wait(&br->w_full[s], (k / kWStages) & 1);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 4; kk++)
            mma_pair_ss(tmem + buf * 256, smem_desc_sw128(sa + kb * kABlock + kk * 32, 16, 1024),
                        smem_desc_sw128(sw + s * kWStage + kk * 32, 16, 1024), IDESC, (kb | kk) ? 1u : 0u);
          mma_commit_pair(smem_u32(&br->w_empty[s]));
          if (kb == kKBlocks - 1) mma_commit_pair(smem_u32(&br->d_full[buf]));
        }
        __syncwarp();
      }
    }
  }
  __syncthreads();
  if (*(volatile int *)&br->abort) {  // a wait gave up: let copies or MMAs still in flight land before the CTA exits
    const uint64_t t0 = globaltimer();
    while (globaltimer() - t0 < 2000000ull) {
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync();  // neither CTA's memory is used by the other any more
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, 512);
  }
}

int fail(int code, const char *msg) {
  set_last_error(msg);
  return code;
}

}  // namespace
}  // namespace mla

int mla_kv_expand(const void *kv_cache, int kv_format, int num_pages, int page_size, const int32_t *block_table,
                  int max_pages, const int32_t *cu_seqlens, int B, int total, const float *kv_scales,
                  const void *w_uk, int64_t uk_row, int64_t uk_head, const void *w_uv, int64_t uv_row,
                  int64_t uv_head, int H, void *kv, void *k_pe, mla_stream_t stream) {
  using namespace mla;
  if (B < 0 || total < 0) return fail(MLA_ERR_INVALID_ARG, "B and total must be >= 0");
  if (total > (1 << 30)) return fail(MLA_ERR_UNSUPPORTED, "total must be at most 2^30 rows");
  if (H < 1 || H > MLA_MAX_HEADS) return fail(MLA_ERR_INVALID_ARG, "H must be in [1, 128]");
  if (kv_format != MLA_KV_BF16 && kv_format != MLA_KV_FP8_E4M3 && kv_format != MLA_KV_FP8_E4M3_TENSOR)
    return fail(MLA_ERR_INVALID_ARG, "kv_format unknown");
  if (page_size != MLA_PAGE_SIZE) return fail(MLA_ERR_UNSUPPORTED, "page_size must be 64");
  if (num_pages < 1 || max_pages < 1) return fail(MLA_ERR_INVALID_ARG, "num_pages and max_pages must be >= 1");
  if (num_pages > 0x7FFFFFFF / MLA_PAGE_SIZE) return fail(MLA_ERR_UNSUPPORTED, "num_pages must be below 2^25");
  if (uk_row % 8 || uk_head % 8 || uv_row % 8 || uv_head % 8)
    return fail(MLA_ERR_INVALID_ARG, "weight strides must be multiples of 8 elements");
  if (uk_row < D_V || uv_row < D_V || (H > 1 && (uk_head < D_V || uv_head < D_V)))
    return fail(MLA_ERR_INVALID_ARG, "weight strides must be at least 512 elements");
  if (B == 0 || total == 0) {
    set_last_error("");
    return MLA_OK;
  }
  if (!kv_cache || !block_table || !cu_seqlens || !w_uk || !w_uv || !kv || !k_pe)
    return fail(MLA_ERR_INVALID_ARG, "null pointer");
  auto al = [](const void *p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; };
  if (!al(kv_cache, 16) || !al(w_uk, 16) || !al(w_uv, 16) || !al(kv, 16) || !al(k_pe, 16))
    return fail(MLA_ERR_INVALID_ARG, "kv_cache, w_uk, w_uv, kv and k_pe must be 16-byte aligned");
  if (!al(block_table, 4) || !al(cu_seqlens, 4))
    return fail(MLA_ERR_INVALID_ARG, "int32 arrays must be 4-byte aligned");
  if (kv_format != MLA_KV_BF16 && (!kv_scales || !al(kv_scales, kv_format == MLA_KV_FP8_E4M3 ? 16 : 4)))
    return fail(MLA_ERR_INVALID_ARG, "an FP8 cache needs kv_scales (16-byte aligned per row, 4 for one scale)");
  CUtensorMap uk_map, uv_map, o_map;
  if (!make_map_3d(&uk_map, w_uk, D_V, 128, H, uk_row, uk_head, 128, 1) ||
      !make_map_3d(&uv_map, w_uv, D_V, 128, H, uv_row, uv_head, 128, 1) ||
      !make_map_3d(&o_map, kv, 256, H, total, 256, (int64_t)H * 256, 1, 32))
    return fail(MLA_ERR_CUDA, "cuTensorMapEncodeTiled failed");
  ExpandParams p;
  p.cache = static_cast<const uint8_t *>(kv_cache);
  p.scales = kv_scales;
  p.block_table = block_table;
  p.cu = cu_seqlens;
  p.kv = static_cast<__nv_bfloat16 *>(kv);
  p.k_pe = static_cast<__nv_bfloat16 *>(k_pe);
  if (status_word(&p.status) != MLA_OK) return MLA_ERR_CUDA;
  p.format = kv_format;
  p.num_pages = num_pages;
  p.max_pages = max_pages;
  p.B = B;
  p.H = H;
  p.total = total;
  p.wait_ns = wait_limit_ns();
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  auto *kernel = p.wait_ns < ptx::kShortWaitNs ? &expand_kernel<true> : &expand_kernel<false>;
  if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
  if (e != cudaSuccess) return fail(MLA_ERR_CUDA, cudaGetErrorString(e));
  const long long units = (long long)ceil_div(total, kPairRows) * H;
  // An equal share of the units for each pair; with few heads a block of rows for
  // each where that is at most one unit more, as most pairs of a share fetch the
  // rows of two blocks (64 blocks on 76 pairs, FP8 / bf16 rows: 2 heads 18.4 ->
  // 14.1 / 15.5 -> 12.6 us, 8 heads 31.3 -> 28.6 / 27.9 -> 27.2 us; 70 blocks, 16
  // heads 51 -> 48 / 49 -> 54 us; 40 blocks, 8 heads 25 -> 28 / 22 -> 27 us).
  const int blocks = ceil_div(total, kPairRows);
  int pairs = (int)(units < sms / 2 ? units : sms / 2);
  if (blocks < pairs && H <= 8 && H - (int)((units + pairs - 1) / pairs) <= 1) pairs = blocks;
  e = launch_dependent(kernel, 2 * pairs, kThreads, kSmem, (cudaStream_t)stream, uk_map, uv_map, o_map, p);
  if (e != cudaSuccess) return fail(MLA_ERR_CUDA, cudaGetErrorString(e));
  set_last_error("");
  return MLA_OK;
}

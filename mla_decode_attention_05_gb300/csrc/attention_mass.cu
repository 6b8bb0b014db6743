// The attention weight of cached tokens: for each cached token n of a sequence
//   mass[n] = decay * mass[n] + sum_{t,h} exp(scale * q[t][h] . K_n - lse[h][t])
// over the query rows (t, h) that see it: the column sums of the softmax that a
// decode (or a prompt's attention) has made, from its log-sum-exp, without its
// product with the values.
//
// One MMA tile has 128 keys as its M rows and up to 128 query rows as its N
// columns, so a key's scores lie in one lane of tensor memory and its sum is
// one thread's own: nothing crosses lanes, no atomics.
#include <cmath>
#include <cstdio>

#include "common.cuh"
#include "dependent.cuh"
#include "fp8.cuh"
#include "ptx.cuh"
#include "ptx_pair.cuh"
#include "tma_map.cuh"

namespace mla {
namespace {

using namespace ptx;

constexpr int kKeys = 128;                     // keys of a tile: two pages
constexpr int kRows = 128;                     // query rows of a tile
constexpr int kBlocks = D_QK / 64;             // blocks of 64 of the 576 dims
constexpr uint32_t kBlock = kKeys * 128;       // 128 rows x 64 dims, 128-byte swizzle
constexpr uint32_t kHalf = kBlock / 2;
constexpr int kD = 4;                          // score tiles in tensor memory
constexpr int kWideWarps = 8;                  // FP8: warps that widen cached rows
constexpr int kWideGroups = 2;
constexpr int kRaw = 5;                        // FP8: blocks as they lie in the cache, on their way or being widened
constexpr uint32_t kRawBlock = kKeys * 64;     // 128 rows x 64 bytes
constexpr uint32_t kRawHalf = kRawBlock / 2;
// The streaming operand's ring; FP8 gives half of it to the raw blocks.
__host__ __device__ constexpr int slots_of(bool fp8) { return fp8 ? 2 : 4; }
constexpr int kMostSlots = 4;
constexpr uint32_t OFF_SLOTS = kBlocks * kBlock;
constexpr uint32_t OFF_RAW = OFF_SLOTS + 2 * kBlock;
constexpr uint32_t OFF_SCALES = OFF_RAW + kRaw * kRawBlock;  // two tiles' scales, [128][4]
constexpr uint32_t kScaleBytes = kKeys * 16;
constexpr uint32_t OFF_BARS = OFF_SLOTS + 5 * kBlock;
static_assert(OFF_SCALES + 2 * kScaleBytes <= OFF_BARS, "shared memory map");
__host__ __device__ constexpr int threads_of(bool fp8) { return fp8 ? 256 + 32 * kWideWarps : 256; }

struct MassParams {
  const uint8_t *cache;
  const float *kv_scales;
  const int32_t *block_table, *seqlens;
  const float *lse;  // [B][H][T]
  float *mass;       // [B][cap]
  float *partial;    // [splits][B][cap], and before it the number of splits in use
  int32_t *splits;
  unsigned int *status;
  int format, num_pages, max_pages, B, T, H, cap, causal;
  int rows, n_qt, box;  // query rows of a sequence, their tiles, rows of a tile's box
  int max_splits;
  float scale_log2, decay;
  unsigned long long wait_ns;
};

struct Bars {
  uint64_t res_full[kBlocks], res_empty[kBlocks];
  uint64_t slot_full[kMostSlots], slot_empty[kMostSlots];
  uint64_t raw_full[kRaw], raw_empty[kRaw];
  uint64_t d_full[kD], d_empty[kD];
  float nl2[2][kRows];  // -lse * log2(e) of a tile's query rows
  int lim[2][kRows];    // keys that a row sees; 0 for one that is no row, or has no weight to give
  int warp_sums[32];
  int start_b, start_t, n_tiles;
  uint32_t tmem_base;
  int abort;
};
constexpr uint32_t kSmem = OFF_BARS + sizeof(Bars);
static_assert(kSmem <= 232448, "shared memory budget");

// `bytes` (a multiple of 16) side by side into shared memory.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
               "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
               : "memory");
}

__device__ __forceinline__ int seq_len(const MassParams &p, int b) {
  const int most = (int)min((long long)p.max_pages * PAGE, (long long)p.cap);
  return min(max(__ldg(p.seqlens + b), 0), most);
}

template <bool kPoll>
__device__ __forceinline__ bool wait_ok(Bars *b, uint64_t *bar, uint32_t parity, const MassParams &p) {
  if (mbar_wait_limited<false, kPoll>(smem_u32(bar), parity, &b->abort, p.wait_ns)) return true;
  atomicOr(p.status, MLA_STATUS_WAIT_TIMEOUT);
  *(volatile int *)&b->abort = 1;
  return false;
}

// The same for a whole warp: its lanes go on, or give up, together.
template <bool kPoll>
__device__ __forceinline__ bool warp_wait(Bars *b, uint64_t *bar, uint32_t parity, const MassParams &p) {
  return __all_sync(0xffffffffu, wait_ok<kPoll>(b, bar, parity, p));
}

// A phase: a resident operand and what streams past it.  kStreamKeys: the query
// rows of sequence b stay and its key tiles [i0, i1) pass by, each one a sum of its
// own.  Otherwise key tile t stays, query tiles [i0, i1) pass by, and their sum
// is part `split` of the tile's.
struct Phase {
  int b, t, i0, i1, split, len;
};

struct Work {
  int b, t;              // sequence and key tile of the first unit
  long long u0, u1;      // units
  int splits;
};

template <bool kStreamKeys, class F>
__device__ __forceinline__ bool for_each_phase(const MassParams &p, const Work &w, F &&f) {
  int b = w.b, t = w.t, len = w.u0 < w.u1 ? seq_len(p, b) : 0;
  for (long long u = w.u0; u < w.u1;) {
    while (t * kKeys >= len) {
      if (++b >= p.B) return true;
      t = 0;
      len = seq_len(p, b);
    }
    if (kStreamKeys) {
      const int n = (int)min(w.u1 - u, (long long)(ceil_div(len, kKeys) - t));
      if (!f(Phase{b, t, t, t + n, 0, len})) return false;
      t += n;
      u += n;
    } else {
      const int s = (int)(u % w.splits);
      int i0 = (int)((long long)p.n_qt * s / w.splits), i1 = (int)((long long)p.n_qt * (s + 1) / w.splits);
      if (p.causal) {  // query rows before the first that sees any of these keys
        const int t_min = max(0, t * kKeys - len + p.T);
        i0 = (int)min((long long)i1, max((long long)i0, (long long)t_min * p.H / kRows));
      }
      if (!f(Phase{b, t, i0, i1, s, len})) return false;
      u++;
      if (s == w.splits - 1) t++;
    }
  }
  return true;
}

// This CTA's units, found by all threads together.
template <bool kStreamKeys>
__device__ Work find_work(const MassParams &p, Bars &br) {
  const int n = blockDim.x, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = ceil_div(p.B, n), b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
  int mine = 0;
  for (int b = b0; b < b1; b++) {
    const int raw = __ldg(p.seqlens + b), len = seq_len(p, b);
    if (raw != len && blockIdx.x == 0) atomicOr(p.status, MLA_STATUS_BAD_SEQLEN);
    mine += ceil_div(len, kKeys);
  }
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) br.warp_sums[warp] = incl;
  __syncthreads();
  int before = 0, total = 0;
  for (int i = 0; i < n / 32; i++) {
    if (i < warp) before += br.warp_sums[i];
    total += br.warp_sums[i];
  }
  Work w;
  w.splits = 1;
  if (!kStreamKeys) w.splits = max(1, min(p.max_splits, ceil_div(2 * (int)gridDim.x, max(total, 1))));
  const long long units = (long long)total * w.splits;
  w.u0 = units * blockIdx.x / gridDim.x;
  w.u1 = units * (blockIdx.x + 1) / gridDim.x;
  const int first = (int)(w.u0 / w.splits);
  int at = before + incl - mine;
  if (first >= at && first < at + mine)
    for (int b = b0; b < b1; b++) {
      const int c = ceil_div(seq_len(p, b), kKeys);
      if (first < at + c) {
        br.start_b = b;
        br.start_t = first - at;
        break;
      }
      at += c;
    }
  if (blockIdx.x == 0 && tid == 0 && p.splits) *p.splits = w.splits;
  __syncthreads();
  w.b = br.start_b;
  w.t = br.start_t;
  return w;
}

__device__ __forceinline__ int page_of(const MassParams &p, int b, int j, int len) {
  if ((long long)j * PAGE >= len) return -1;
  const int page = __ldg(p.block_table + (size_t)b * p.max_pages + j);
  if (page < 0 || page >= p.num_pages) {
    atomicOr(p.status, MLA_STATUS_BAD_PAGE);
    return -1;
  }
  return page;
}

// ---- loads -------------------------------------------------------------------------

// Warp 0: query rows, the pages of a bf16 cache, and the raw blocks of an FP8 one
// (64 bytes of each row; ten of them where the rotated part is bf16).  The whole
// warp waits and looks pages up, one elected lane asks for the copies.
template <bool kStreamKeys, bool kFp8, bool kPoll>
__device__ void load_role(const MassParams &p, uint8_t *base, Bars &br, const CUtensorMap *k_map, const CUtensorMap *q_map,
                          const Work &w) {
  constexpr int kSlots = slots_of(kFp8);
  const uint32_t res = smem_u32(base), slots = smem_u32(base + OFF_SLOTS);
  const uint32_t raws = smem_u32(base + OFF_RAW), scales = smem_u32(base + OFF_SCALES);
  const uint64_t keep = policy_evict_normal(), pass = policy_evict_first();
  const uint64_t key_pol = kStreamKeys ? pass : keep;
  const bool scaled = p.format == MLA_KV_FP8_E4M3;
  const int n_raw = scaled ? 10 : 9;
  uint32_t s = 0, ph = 1, rph = 1, rs = 0, rawph = 1, tile = 0;
  auto keys = [&](uint32_t dst, uint64_t *full, int pg0, int pg1, int kb) {
    if (!elect_one()) return;
    const uint32_t bar = smem_u32(full);
    mbar_arrive_expect_tx(bar, (pg0 >= 0 ? kHalf : 0) + (pg1 >= 0 ? kHalf : 0));
    if (pg0 >= 0) tma_load_4d(dst, k_map, bar, 0, 0, kb, pg0, key_pol);
    if (pg1 >= 0) tma_load_4d(dst + kHalf, k_map, bar, 0, 0, kb, pg1, key_pol);
  };
  auto rows = [&](uint32_t dst, uint64_t *full, int b, int qt, int kb) {
    if (!elect_one()) return;
    const uint32_t bar = smem_u32(full);
    mbar_arrive_expect_tx(bar, p.box * 128);
    tma_load_3d(dst, q_map, bar, 0, b * p.rows + qt * kRows, kb, keep);
  };
  // an FP8 tile's raw blocks and, with the first, its scales
  auto raw_tile = [&](int pg0, int pg1) {
    const uint32_t n = (pg0 >= 0) + (pg1 >= 0);
    for (int k = 0; k < n_raw; k++) {
      if (!warp_wait<kPoll>(&br, &br.raw_empty[rs], rawph, p)) return false;
      if (elect_one()) {
        const uint32_t bar = smem_u32(&br.raw_full[rs]), dst = raws + rs * kRawBlock;
        const bool with = scaled && k == 0;
        mbar_arrive_expect_tx(bar, n * (kRawHalf + (with ? kScaleBytes / 2 : 0)));
#pragma unroll
        for (int h = 0; h < 2; h++) {
          const int pg = h ? pg1 : pg0;
          if (pg < 0) continue;
          tma_load_3d(dst + h * kRawHalf, k_map, bar, k * 64, 0, pg, key_pol);
          if (with)
            bulk_load(scales + (tile & 1) * kScaleBytes + h * (kScaleBytes / 2), p.kv_scales + (size_t)pg * PAGE * 4,
                      kScaleBytes / 2, bar);
        }
      }
      __syncwarp();
      if (++rs == kRaw) {
        rs = 0;
        rawph ^= 1;
      }
    }
    tile++;
    return true;
  };
  for_each_phase<kStreamKeys>(p, w, [&](const Phase &f) {
    if (f.i0 >= f.i1) return true;
    int pg0 = -1, pg1 = -1;
    if (!kStreamKeys) {
      pg0 = page_of(p, f.b, 2 * f.t, f.len);
      pg1 = page_of(p, f.b, 2 * f.t + 1, f.len);
    }
    if (kStreamKeys || !kFp8) {
      for (int kb = 0; kb < kBlocks; kb++) {
        if (!warp_wait<kPoll>(&br, &br.res_empty[kb], rph, p)) return false;
        if (kStreamKeys) rows(res + kb * kBlock, &br.res_full[kb], f.b, 0, kb);
        else keys(res + kb * kBlock, &br.res_full[kb], pg0, pg1, kb);
        __syncwarp();
      }
      rph ^= 1;
    } else if (!raw_tile(pg0, pg1)) {
      return false;
    }
    for (int i = f.i0; i < f.i1; i++) {
      if (kStreamKeys) {
        pg0 = page_of(p, f.b, 2 * i, f.len);
        pg1 = page_of(p, f.b, 2 * i + 1, f.len);
      }
      if constexpr (kStreamKeys && kFp8) {
        if (!raw_tile(pg0, pg1)) return false;
      } else {
        for (int kb = 0; kb < kBlocks; kb++) {
          if (!warp_wait<kPoll>(&br, &br.slot_empty[s], ph, p)) return false;
          if (kStreamKeys) keys(slots + s * kBlock, &br.slot_full[s], pg0, pg1, kb);
          else rows(slots + s * kBlock, &br.slot_full[s], f.b, i, kb);
          __syncwarp();
          if (++s == kSlots) {
            s = 0;
            ph ^= 1;
          }
        }
      }
    }
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

// Warps 8-15 widen FP8 rows, in two groups that take the blocks in turn: thread i of
// a group has 16 bytes of rows i / 4 + 32 k.  (The raw blocks come by TMA: a load of its own in flight
// would hold up the thread's proxy fences.)
template <bool kStreamKeys, bool kPoll>
__device__ void widen_role(const MassParams &p, uint8_t *base, Bars &br, const Work &w, int thread) {
  constexpr int kSlots = slots_of(true);
  static_assert(kSlots == kWideGroups, "a group has a slot of its own");
  const uint32_t res = smem_u32(base), slots = smem_u32(base + OFF_SLOTS), raws = smem_u32(base + OFF_RAW);
  const int group = thread / (32 * kWideWarps / kWideGroups), i = thread % (32 * kWideWarps / kWideGroups);
  const int r = i >> 2, c = i & 3, x = r & 7;
  const bool first = (threadIdx.x & 31) == 0, scaled = p.format == MLA_KV_FP8_E4M3;
  const float one = scaled ? 0.f : __ldg(p.kv_scales);
  uint32_t raw = 0, block = 0, phase = 0, tile = 0;  // raw blocks, blocks, phases and tiles so far
  uint4 v[4];
  // this thread's bytes of raw block `raw`, which is then free
  auto take = [&](uint32_t k) {
    if (!warp_wait<kPoll>(&br, &br.raw_full[k % kRaw], (k / kRaw) & 1, p)) return false;
#pragma unroll
    for (int j = 0; j < 4; j++) v[j] = ld_shared_v4(raws + (k % kRaw) * kRawBlock + (r + 32 * j) * 64 + c * 16);
    return true;
  };
  auto taken = [&](uint32_t k) {
    __syncwarp();
    if (first) mbar_arrive(smem_u32(&br.raw_empty[k % kRaw]));
  };
  auto widen_tile = [&] {
    const float *sc = reinterpret_cast<const float *>(base + OFF_SCALES + (tile & 1) * kScaleBytes) + r * 4;
    for (int kb = 0; kb < kBlocks; kb++, block++, raw++) {
      const bool two = kb == 8 && scaled;  // the rotated part, bf16: two raw blocks, chunks 0-3 and 4-7 of a row
      if ((int)(block % kWideGroups) != group) {
        raw += two;
        continue;
      }
      const uint32_t s = block % kSlots;
      if (!take(raw)) return false;
      if (!warp_wait<kPoll>(&br, kStreamKeys ? &br.slot_empty[s] : &br.res_empty[kb],
                            ((kStreamKeys ? block / kSlots : phase) & 1) ^ 1, p))
        return false;
      const uint32_t at = (kStreamKeys ? slots + s * kBlock : res + kb * kBlock) + r * 128;
      if (two) {
#pragma unroll
        for (int j = 0; j < 4; j++) st_shared_v4(at + 32 * j * 128 + ((c ^ x) << 4), v[j]);
        taken(raw);
        if (!take(++raw)) return false;
#pragma unroll
        for (int j = 0; j < 4; j++) st_shared_v4(at + 32 * j * 128 + (((4 + c) ^ x) << 4), v[j]);
      } else {
#pragma unroll
        for (int j = 0; j < 4; j++) {
          uint4 lo, hi;
          widen16(v[j], scaled ? sc[32 * j * 4 + (kb >> 1)] : one, lo, hi);
          st_shared_v4(at + 32 * j * 128 + (((2 * c) ^ x) << 4), lo);
          st_shared_v4(at + 32 * j * 128 + (((2 * c + 1) ^ x) << 4), hi);
        }
      }
      taken(raw);
      fence_proxy_async_smem();
      __syncwarp();
      if (first) mbar_arrive(smem_u32(kStreamKeys ? &br.slot_full[s] : &br.res_full[kb]));
    }
    phase++;
    tile++;
    return true;
  };
  for_each_phase<kStreamKeys>(p, w, [&](const Phase &f) {
    for (int t = f.i0; t < (kStreamKeys ? f.i1 : min(f.i0 + 1, f.i1)); t++)
      if (!widen_tile()) return false;
    return true;
  });
}

// ---- scores ------------------------------------------------------------------------

constexpr uint32_t kMmaBar = 1, kSumBar = 2;

// Warp 2 waits for what the MMAs of warp 1 need and meets it at a named barrier (a
// wait in the issuing warp would hold up its MMAs in flight).
template <bool kStreamKeys, bool kFp8, bool kPoll>
__device__ void wait_role(const MassParams &p, Bars &br, const Work &w) {
  constexpr int kSlots = slots_of(kFp8);
  uint32_t s = 0, ph = 0, rph = 0, g = 0;
  for_each_phase<kStreamKeys>(p, w, [&](const Phase &f) {
    if (f.i0 >= f.i1) return true;
    for (int i = f.i0; i < f.i1; i++, g++) {
      bool ok = warp_wait<kPoll>(&br, &br.d_empty[g % kD], ((g / kD) & 1) ^ 1, p);
      for (int kb = 0; kb < kBlocks; kb++) {
        if (ok && i == f.i0) ok = warp_wait<kPoll>(&br, &br.res_full[kb], rph, p);
        if (ok) ok = warp_wait<kPoll>(&br, &br.slot_full[s], ph, p);
        if (bar_red_or(kMmaBar, 64, !ok)) return false;
        if (++s == kSlots) {
          s = 0;
          ph ^= 1;
        }
      }
    }
    rph ^= 1;
    return true;
  });
}

template <bool kStreamKeys, bool kFp8>
__device__ void mma_role(const MassParams &p, uint8_t *base, Bars &br, const Work &w, uint32_t tmem) {
  constexpr int kSlots = slots_of(kFp8);
  const uint32_t res = smem_u32(base), slots = smem_u32(base + OFF_SLOTS);
  const uint32_t idesc = idesc_bf16_f32(kKeys, p.box, false, false);
  uint32_t s = 0, g = 0;
  for_each_phase<kStreamKeys>(p, w, [&](const Phase &f) {
    if (f.i0 >= f.i1) return true;
    for (int i = f.i0; i < f.i1; i++, g++) {
      for (int kb = 0; kb < kBlocks; kb++) {
        if (bar_red_or(kMmaBar, 64, false)) return false;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t stay = smem_desc_sw128(res + kb * kBlock, 16, 1024);
          const uint64_t pass = smem_desc_sw128(slots + s * kBlock, 16, 1024);
          const uint64_t a = kStreamKeys ? pass : stay, b = kStreamKeys ? stay : pass;
#pragma unroll
          for (int kk = 0; kk < 4; kk++)
            mma_ss(tmem + (g % kD) * kRows, a + kk * 2, b + kk * 2, idesc, kb || kk ? 1u : 0u);
          mma_commit(smem_u32(&br.slot_empty[s]));
          if (i == f.i1 - 1) mma_commit(smem_u32(&br.res_empty[kb]));
          if (kb == kBlocks - 1) mma_commit(smem_u32(&br.d_full[g % kD]));
        }
        __syncwarp();
        if (++s == kSlots) s = 0;
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

// Warps 4-7: thread = key of the tile = lane of tensor memory.
template <bool kStreamKeys, bool kPoll>
__device__ void sum_role(const MassParams &p, Bars &br, const Work &w, uint32_t tmem) {
  const int i = threadIdx.x - 128, lane = threadIdx.x & 31;
  const uint32_t lt = tmem + ((uint32_t)(i & 96) << 16);
  uint32_t g = 0, buf = 0;
  auto set_rows = [&](const Phase &f, int qt) {
    buf ^= 1;
    const int R = qt * kRows + i;
    int lim = 0;
    float nl = 0.f;
    if (R < p.rows) {
      const int t = R / p.H, h = R % p.H;
      const float l = __ldg(p.lse + ((size_t)f.b * p.H + h) * p.T + t);
      lim = l == -INFINITY ? 0 : row_kv_len(f.len, p.T, t, p.causal);
      nl = -l * LOG2E;
    }
    br.nl2[buf][i] = nl;
    br.lim[buf][i] = lim;
  };
  for_each_phase<kStreamKeys>(p, w, [&](const Phase &f) {
    if (kStreamKeys) set_rows(f, 0);
    float sum = 0.f;
    auto key_of = [&](int t) { return t * kKeys + i; };
    auto store = [&](int t, float v) {
      const int n = key_of(t);
      if (n >= f.len) return;
      if (page_of(p, f.b, n / PAGE, f.len) < 0) v = 0.f;
      if (!kStreamKeys && w.splits > 1) {
        p.partial[((size_t)f.split * p.B + f.b) * p.cap + n] = v;
      } else {
        float *m = p.mass + (size_t)f.b * p.cap + n;
        *m = p.decay != 0.f ? fmaf(p.decay, *m, v) : v;
      }
    };
    for (int k = f.i0; k < f.i1; k++, g++) {
      if (!kStreamKeys) set_rows(f, k);
      const bool ok = warp_wait<kPoll>(&br, &br.d_full[g % kD], (g / kD) & 1, p);
      if (bar_red_or(kSumBar, 128, !ok)) return false;
      tc_fence_after();
      const int key = key_of(kStreamKeys ? k : f.t);
      const int cols = min(kRows, p.rows - (kStreamKeys ? 0 : k * kRows));
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
      for (int c0 = 0; c0 < cols; c0 += 32) {
        uint32_t v[32];
        __syncwarp();
        tmem_ld32(lt + (g % kD) * kRows + c0, v);
        tmem_wait_ld();
#pragma unroll
        for (int j = 0; j < 32; j += 4) {
          const float4 nl = *reinterpret_cast<const float4 *>(&br.nl2[buf][c0 + j]);
          const int4 lim = *reinterpret_cast<const int4 *>(&br.lim[buf][c0 + j]);
          const float e0 = ex2(fmaf(__uint_as_float(v[j]), p.scale_log2, nl.x));
          const float e1 = ex2(fmaf(__uint_as_float(v[j + 1]), p.scale_log2, nl.y));
          const float e2 = ex2(fmaf(__uint_as_float(v[j + 2]), p.scale_log2, nl.z));
          const float e3 = ex2(fmaf(__uint_as_float(v[j + 3]), p.scale_log2, nl.w));
          if (key < lim.x) acc[0] += e0;
          if (key < lim.y) acc[1] += e1;
          if (key < lim.z) acc[2] += e2;
          if (key < lim.w) acc[3] += e3;
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&br.d_empty[g % kD]));
      const float got = (acc[0] + acc[1]) + (acc[2] + acc[3]);
      if (kStreamKeys) store(k, got);
      else sum += got;
    }
    if (!kStreamKeys) store(f.t, sum);
    return true;
  });
}

template <bool kStreamKeys, bool kFp8, bool kPoll>
__global__ void __launch_bounds__(threads_of(kFp8), 1)
    attention_mass_kernel(const __grid_constant__ CUtensorMap k_map, const __grid_constant__ CUtensorMap q_map,
                          const MassParams p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  if (smem_u32(smem) & 1023u) {
    if (threadIdx.x == 0) atomicOr(p.status, MLA_STATUS_SMEM_ALIGN);
    return;
  }
  Bars &br = *reinterpret_cast<Bars *>(smem + OFF_BARS);
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kBlocks; i++) {
      mbar_init(smem_u32(&br.res_full[i]), kFp8 && !kStreamKeys ? kWideWarps / kWideGroups : 1);
      mbar_init(smem_u32(&br.res_empty[i]), 1);
    }
    for (int i = 0; i < kMostSlots; i++) {
      mbar_init(smem_u32(&br.slot_full[i]), kFp8 && kStreamKeys ? kWideWarps / kWideGroups : 1);
      mbar_init(smem_u32(&br.slot_empty[i]), 1);
    }
    for (int i = 0; i < kRaw; i++) {
      mbar_init(smem_u32(&br.raw_full[i]), 1);
      mbar_init(smem_u32(&br.raw_empty[i]), kWideWarps / kWideGroups);
    }
    for (int i = 0; i < kD; i++) {
      mbar_init(smem_u32(&br.d_full[i]), 1);
      mbar_init(smem_u32(&br.d_empty[i]), 4);
    }
    br.abort = 0;
    br.start_b = br.start_t = 0;
    fence_mbar_init_cluster();
    prefetch_tensormap(&q_map);
    prefetch_tensormap(&k_map);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(&br.tmem_base), kD * kRows);
    tmem_relinquish();
  }
  grid_dep_trigger();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = br.tmem_base;
  grid_dep_wait();
  const Work w = find_work<kStreamKeys>(p, br);
  if (warp == 0) load_role<kStreamKeys, kFp8, kPoll>(p, smem, br, &k_map, &q_map, w);
  else if (warp == 1) mma_role<kStreamKeys, kFp8>(p, smem, br, w, tmem);
  else if (warp == 2) wait_role<kStreamKeys, kFp8, kPoll>(p, br, w);
  else if (warp >= 4 && warp < 8) sum_role<kStreamKeys, kPoll>(p, br, w, tmem);
  else if constexpr (kFp8) {
    if (warp >= 8) widen_role<kStreamKeys, kPoll>(p, smem, br, w, threadIdx.x - 256);
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (br.abort) {  // copies and MMAs in flight end
    const uint64_t t0 = globaltimer();
    while (globaltimer() - t0 < 2000000ull) {
    }
  }
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kD * kRows);
  }
}

// The parts of each key's sum, in their order.
__global__ void __launch_bounds__(256) mass_reduce_kernel(MassParams p) {
  grid_dep_wait();
  const int splits = *p.splits;
  if (splits <= 1) return;
  const int b = blockIdx.y, len = seq_len(p, b);
  for (int n = blockIdx.x * 256 + threadIdx.x; n < len; n += gridDim.x * 256) {
    float v = 0.f;
    for (int s = 0; s < splits; s++) v += p.partial[((size_t)s * p.B + b) * p.cap + n];
    float *m = p.mass + (size_t)b * p.cap + n;
    *m = p.decay != 0.f ? fmaf(p.decay, *m, v) : v;
  }
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

// Parts of a key's sum, at most: none where a sequence's query rows are one tile.
int most_splits(int B, int T, int H) {
  const int n_qt = ceil_div(T * H, kRows), want = ceil_div(304, B);
  return n_qt < want ? n_qt : want;
}

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" size_t mla_attention_mass_workspace_bytes(int B, int T, int H, int mass_cap) {
  if (check_sizes(B, T, H, mass_cap) != MLA_OK) return 0;
  const int s = most_splits(B, T, H);
  return s <= 1 ? 0 : 256 + ((size_t)s * B * mass_cap * sizeof(float) + 255) / 256 * 256;
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
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  p.cache = static_cast<const uint8_t *>(kv_cache);
  p.kv_scales = kv_scales;
  p.block_table = block_table;
  p.seqlens = cache_seqlens;
  p.lse = lse;
  p.mass = mass;
  p.splits = need ? static_cast<int32_t *>(workspace) : nullptr;
  p.partial = need ? reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + 256) : nullptr;
  p.format = kv_format;
  p.num_pages = num_pages;
  p.max_pages = max_pages;
  p.B = B;
  p.T = T;
  p.H = H;
  p.cap = mass_cap;
  p.causal = causal;
  p.rows = T * H;
  p.n_qt = ceil_div(p.rows, kRows);
  p.box = p.rows < kRows ? ceil_div(p.rows, 16) * 16 : kRows;
  p.max_splits = most_splits(B, T, H);
  p.scale_log2 = softmax_scale * LOG2E;
  p.decay = decay;
  p.wait_ns = wait_limit_ns();

  CUtensorMap k_map{}, q_map{};
  auto fn = tensor_map_encoder();
  if (!fn) return fail(MLA_ERR_CUDA, "cuTensorMapEncodeTiled not found");
  bool ok = make_map_3d(&q_map, q, 64, (uint64_t)B * p.rows, kBlocks, D_QK, 64, p.box, 1);
  if (ok && kv_format == MLA_KV_BF16) {
    cuuint64_t dims[4] = {64, (cuuint64_t)PAGE, kBlocks, (cuuint64_t)num_pages};
    cuuint64_t strides[3] = {(cuuint64_t)D_QK * 2, 128, (cuuint64_t)D_QK * 2 * PAGE};
    cuuint32_t box[4] = {64, (cuuint32_t)PAGE, 1, 1}, estr[4] = {1, 1, 1, 1};
    ok = fn(&k_map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(kv_cache), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  } else if (ok) {
    // bytes, 64 of each row of a page at a time
    const cuuint64_t row = kv_format == MLA_KV_FP8_E4M3 ? FP8_ROW : D_QK;
    cuuint64_t dims[3] = {row, (cuuint64_t)PAGE, (cuuint64_t)num_pages}, strides[2] = {row, row * PAGE};
    cuuint32_t box[3] = {64, (cuuint32_t)PAGE, 1}, estr[3] = {1, 1, 1};
    ok = fn(&k_map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void *>(kv_cache), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  }
  if (!ok) return fail(MLA_ERR_CUDA, "a tensor map could not be made");
  const bool keys = p.n_qt == 1, fp8 = kv_format != MLA_KV_BF16, poll = p.wait_ns < kShortWaitNs;
  using Kernel = void (*)(CUtensorMap, CUtensorMap, MassParams);
  Kernel k = nullptr;
#define PICK(a, b, c) \
  if (keys == a && fp8 == b && poll == c) k = attention_mass_kernel<a, b, c>
  PICK(false, false, false); PICK(false, false, true); PICK(false, true, false); PICK(false, true, true);
  PICK(true, false, false); PICK(true, false, true); PICK(true, true, false); PICK(true, true, true);
#undef PICK
  cudaStream_t s = (cudaStream_t)stream;
  if (e == cudaSuccess) e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
  if (e == cudaSuccess) e = launch_dependent(k, sms, threads_of(fp8), kSmem, s, k_map, q_map, p);
  if (e == cudaSuccess && need) {
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    const int blocks = ceil_div(mass_cap, 256);
    cfg.gridDim = dim3(blocks < 64 ? blocks : 64, B);
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, mass_reduce_kernel, p);
  }
  if (e != cudaSuccess) {
    char msg[128];
    snprintf(msg, sizeof msg, "attention mass: %s", cudaGetErrorString(e));
    return fail(MLA_ERR_CUDA, msg);
  }
  set_last_error("");
  return MLA_OK;
}

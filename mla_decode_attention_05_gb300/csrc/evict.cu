// Eviction from a paged latent cache by accumulated attention weight: of a
// sequence's n > keep cached tokens the first positions (sinks), the latest
// (recent) and the heaviest of the others stay, keep in all, ties in favour of
// the lower slot.  Attention does not depend on the order of slots, so nothing is
// compacted: the stayers behind slot `keep`, in order, move into the slots that
// empty before it, in order.  Sources and targets do not overlap, so all rows
// move at once, and no row moves that need not (sliding the stayers together
// would move nearly every row behind the first hole).
//
// Bound by the latency of dependent steps: 64 FP8 sequences of 4352 tokens cut to 4096 take
// 17 us (3.6 for the bytes at the copy rate), eight of up to 32768 cut to 4096 23 us (7.8), one of 1100
// 11.5 us; about 60 % of it is the selection.
#include <cstdio>

#include "common.cuh"
#include "dependent.cuh"
#include "ptx.cuh"

namespace mla {
namespace {

using namespace ptx;

constexpr int kSelectThreads = 1024;
constexpr int kWarps = kSelectThreads / 32;
constexpr int kMostCtas = 8;                 // CTAs of a cluster, one cluster a sequence
constexpr int kCtaTokens = 4096;             // tokens for which a cluster gets another CTA
constexpr int kHeld = kCtaTokens / kSelectThreads;  // tokens of a lane that stay in registers while the latest is found
constexpr int kKeyCache = 16384;             // sort keys that a CTA keeps in shared memory
constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 8;                 // rows that a warp looks up together
constexpr int kMoveFlight = 4;               // and of those, rows on their way together

struct EvictParams {
  uint8_t *cache;
  float *kv_scales;
  const int32_t *block_table, *seqlens;
  float *mass;
  int32_t *positions, *out_seqlens;
  int32_t *counts, *holes, *movers;  // workspace: [B], [B][room], [B][room]
  unsigned int *status;
  int format, num_pages, max_pages, cap, keep, sinks, recent, room;
};

struct SelectShared {
  uint32_t keys[kKeyCache];
  alignas(16) int hist[4][256];
  alignas(16) int total[256];
  int newest;
  int counts[4][kWarps];  // of a warp's keys: above the border and equal to it, in slots below `keep` and behind
  int before[4][kWarps], all[4];
  int digit, above;
  int warp_max[kWarps];
};

__device__ __forceinline__ int ld_cluster(const int *p, uint32_t rank) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(mapa(smem_u32(p), rank)) : "memory");
  return v;
}

// All threads that work on a sequence; the lanes of a warp meet first.
template <bool kAlone>
__device__ __forceinline__ void meet() {
  if (kAlone) {
    __syncthreads();
  } else {
    __syncwarp();
    cluster_sync();
  }
}

// A weight's place in the order: larger is heavier, -0 is 0, nan below everything.
__device__ __forceinline__ uint32_t order_key(float m) {
  if (m != m) return 0u;
  const uint32_t b = __float_as_uint(m == 0.f ? 0.f : m);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// The selection, a cluster (kAlone: a CTA) for each sequence.  Warp w of CTA r has
// the slots of segment r * kWarps + w, so what lies before a slot is counted by
// warps.  The keep-th key of the order, the border, is found by four passes over
// digits of 8 bits; the keys stay in shared memory, and lanes with equal digits
// count together (the first digits of weights are few: a lane each would queue up).
// A stayer has a key above the border, or is among the first `want` equal to it.
// Bound by the chain of its steps, not by what it reads: a cluster gets a CTA for
// each 4096 tokens.
template <bool kAlone>
__global__ void __launch_bounds__(kSelectThreads) evict_select_kernel(EvictParams p, int ctas) {
  extern __shared__ __align__(16) uint8_t smem[];
  SelectShared &sh = *reinterpret_cast<SelectShared *>(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = kAlone ? 0 : (int)cluster_ctarank();
  const int b = kAlone ? (int)blockIdx.x : (int)blockIdx.x / ctas;
  grid_dep_trigger();
  sh.hist[0][tid] = 0;  // (4 * 256 = kSelectThreads)
  static_assert(4 * 256 == kSelectThreads, "one bin a thread");
  grid_dep_wait();
  const long long most = min((long long)p.max_pages * PAGE, (long long)p.cap);
  const int raw = p.seqlens[b];
  const int n = (int)min((long long)max(raw, 0), most);
  if (n != raw && rank == 0 && tid == 0) atomicOr(p.status, MLA_STATUS_BAD_SEQLEN);
  if (n <= p.keep) {
    meet<kAlone>();  // (out_seqlens may be seqlens: everyone has read it)
    if (rank == 0 && tid == 0) {
      p.counts[b] = 0;
      p.out_seqlens[b] = n;
    }
    return;
  }
  float *mass = p.mass + (size_t)b * p.cap;
  int32_t *pos = p.positions + (size_t)b * p.cap;
  const int seg = ceil_div(ceil_div(n, ctas * kWarps), 32) * 32;
  const long long at = (long long)(rank * kWarps + warp) * seg;
  const int lo = (int)min(at, (long long)n), hi = (int)min(at + seg, (long long)n);

  int held_pos[kHeld];
  float held_mass[kHeld];
  int newest = INT32_MIN;
#pragma unroll
  for (int k = 0; k < kHeld; k++) {
    const int i = lo + 32 * k + lane;
    held_pos[k] = i < hi ? pos[i] : INT32_MIN;
    held_mass[k] = i < hi ? mass[i] : 0.f;
    newest = max(newest, held_pos[k]);
  }
  for (int i = lo + 32 * kHeld + lane; i < hi; i += 32) newest = max(newest, pos[i]);
  newest = __reduce_max_sync(0xffffffffu, newest);
  if (lane == 0) sh.warp_max[warp] = newest;
  __syncthreads();
  newest = __reduce_max_sync(0xffffffffu, sh.warp_max[lane]);
  static_assert(kWarps == 32, "a lane a warp");
  if (!kAlone) {
    if (tid == 0) sh.newest = newest;
    meet<kAlone>();
    newest = __reduce_max_sync(0xffffffffu, lane < ctas ? ld_cluster(&sh.newest, lane) : INT32_MIN);
  }

  auto key_of = [&](int at, float weight) {
    return at < p.sinks || (long long)at > (long long)newest - p.recent ? 0xffffffffu : order_key(weight);
  };
  uint32_t *mine = sh.keys + warp * (kKeyCache / kWarps);
  auto key = [&](int i) { return i - lo < kKeyCache / kWarps ? mine[i - lo] : key_of(pos[i], mass[i]); };
#pragma unroll
  for (int k = 0; k < kHeld; k++) {
    const int i = lo + 32 * k + lane;
    if (i < hi) mine[i - lo] = key_of(held_pos[k], held_mass[k]);
  }
  for (int i = lo + 32 * kHeld + lane; i < hi && i - lo < kKeyCache / kWarps; i += 32) mine[i - lo] = key_of(pos[i], mass[i]);

  uint32_t border = 0;  // its digits so far
  int want = p.keep;    // of the keys that have these digits
  for (int pass = 0; pass < 4; pass++) {
    const int shift = 24 - 8 * pass;
    for (int i0 = lo; i0 < hi; i0 += 32) {
      const int i = i0 + lane;
      const uint32_t k = i < hi ? key(i) : 0u;
      const bool counts = i < hi && (pass == 0 || (k >> (shift + 8)) == border);
      if (!__any_sync(0xffffffffu, counts)) continue;
      const int digit = counts ? (int)((k >> shift) & 255u) : 256;
      const uint32_t same = __match_any_sync(0xffffffffu, digit);
      if (counts && lane == __ffs(same) - 1) atomicAdd(&sh.hist[pass][digit], __popc(same));
    }
    meet<kAlone>();
    const int *bins = sh.hist[pass];
    if (!kAlone) {
      if (tid < 256) {
        int v[kMostCtas], sum = 0;
#pragma unroll
        for (int r = 0; r < kMostCtas; r++) v[r] = r < ctas ? ld_cluster(&sh.hist[pass][tid], r) : 0;
#pragma unroll
        for (int r = 0; r < kMostCtas; r++) sum += v[r];
        sh.total[tid] = sum;
      }
      bins = sh.total;
      __syncthreads();
    }
    if (warp == 0) {  // lane l: digits 255 - 8 l ... 248 - 8 l
      const int4 high = *reinterpret_cast<const int4 *>(bins + 252 - 8 * lane), low = *reinterpret_cast<const int4 *>(bins + 248 - 8 * lane);
      const int got[8] = {high.w, high.z, high.y, high.x, low.w, low.z, low.y, low.x};
      const int sum = (got[0] + got[1] + got[2] + got[3]) + (got[4] + got[5] + got[6] + got[7]);
      int above = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, above, o);
        if (lane >= o) above += v;
      }
      above -= sum;
      bool found = false;
#pragma unroll
      for (int j = 0; j < 8; j++) {
        if (!found && above < want && want <= above + got[j]) {
          sh.digit = 255 - 8 * lane - j;
          sh.above = above;
          found = true;
        }
        above += got[j];
      }
    }
    __syncthreads();
    border = (border << 8) | (uint32_t)sh.digit;
    want -= sh.above;
    __syncthreads();
  }

  int counts[4] = {0, 0, 0, 0};
  for (int i0 = lo; i0 < hi; i0 += 32) {
    const int i = i0 + lane;
    const uint32_t k = i < hi ? key(i) : 0u;
    const uint32_t above = __ballot_sync(0xffffffffu, i < hi && k > border);
    const uint32_t equal = __ballot_sync(0xffffffffu, i < hi && k == border);
    const int first = min(max(p.keep - i0, 0), 32);  // lanes whose slots lie below keep
    const uint32_t front = first == 32 ? 0xffffffffu : (1u << first) - 1u;
    counts[0] += __popc(above & front);
    counts[1] += __popc(equal & front);
    counts[2] += __popc(above & ~front);
    counts[3] += __popc(equal & ~front);
  }
  if (lane == 0)
#pragma unroll
    for (int k = 0; k < 4; k++) sh.counts[k][warp] = counts[k];
  meet<kAlone>();
  if (warp < 4) {  // warp k: what the warps before each of this CTA's have of counts[k], and all have
    int v[kMostCtas], earlier = 0, all = 0;
#pragma unroll
    for (int r = 0; r < kMostCtas; r++)
      v[r] = kAlone ? (r == 0 ? sh.counts[warp][lane] : 0) : (r < ctas ? ld_cluster(&sh.counts[warp][lane], r) : 0);
    int own = 0;
#pragma unroll
    for (int r = 0; r < kMostCtas; r++) {
      const int sum = __reduce_add_sync(0xffffffffu, v[r]);
      all += sum;
      if (r < rank) earlier += sum;
      if (r == rank) own = v[r];
    }
    int incl = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += u;
    }
    sh.before[warp][lane] = earlier + incl - own;
    if (lane == 0) sh.all[warp] = all;
  }
  __syncthreads();
  const int before[4] = {sh.before[0][warp], sh.before[1][warp], sh.before[2][warp], sh.before[3][warp]};
  const int total[4] = {sh.all[0], sh.all[1], sh.all[2], sh.all[3]};
  const uint32_t below = (1u << lane) - 1u;
  int32_t *holes = p.holes + (size_t)b * p.room, *movers = p.movers + (size_t)b * p.room;
  int tie_at = before[1] + before[3];
  int hole_at = min(lo, p.keep) - before[0] - min(want, before[1]);
  int mover_at = before[2] + min(want, before[1] + before[3]) - min(want, before[1]);
  for (int i0 = lo; i0 < hi; i0 += 32) {
    const int i = i0 + lane;
    const uint32_t k = i < hi ? key(i) : 0u;
    const bool tie = i < hi && k == border;
    const uint32_t tied = __ballot_sync(0xffffffffu, tie);
    const bool stays = i < hi && (k > border || (tie && tie_at + __popc(tied & below) < want));
    const bool hole = i < hi && i < p.keep && !stays, mover = i >= p.keep && stays;
    const uint32_t hs = __ballot_sync(0xffffffffu, hole), ms = __ballot_sync(0xffffffffu, mover);
    if (hole) holes[hole_at + __popc(hs & below)] = i;
    if (mover) movers[mover_at + __popc(ms & below)] = i;
    if (i < hi && i >= p.keep && !stays) {
      mass[i] = 0.f;
      pos[i] = -1;
    }
    tie_at += __popc(tied);
    hole_at += __popc(hs);
    mover_at += __popc(ms);
  }
  if (rank == 0 && tid == 0) {
    p.counts[b] = total[2] + want - min(want, total[1]);
    p.out_seqlens[b] = p.keep;
  }
  if (!kAlone) meet<kAlone>();  // the others have read this CTA's counts
}

// Blocks y: sequence; a warp looks up eight rows at once, a lane each, and copies
// four at a time with all its lanes.
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(EvictParams p) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, b = blockIdx.y;
  grid_dep_trigger();
  grid_dep_wait();
  const int count = p.counts[b];
  const int units = p.format == MLA_KV_BF16 ? 72 : p.format == MLA_KV_FP8_E4M3 ? 40 : 36;  // of 16 bytes
  float *mass = p.mass + (size_t)b * p.cap;
  int32_t *pos = p.positions + (size_t)b * p.cap;
  const int32_t *table = p.block_table + (size_t)b * p.max_pages;
  for (int j0 = (blockIdx.x * (kMoveThreads / 32) + warp) * kMoveRows; j0 < count;
       j0 += gridDim.x * (kMoveThreads / 32) * kMoveRows) {
    long long from = -1, to = -1;  // rows of the pool
    if (lane < kMoveRows && j0 + lane < count) {
      const int src = p.movers[(size_t)b * p.room + j0 + lane], dst = p.holes[(size_t)b * p.room + j0 + lane];
      const int ps = table[src / PAGE], pd = table[dst / PAGE];
      mass[dst] = mass[src];
      pos[dst] = pos[src];
      mass[src] = 0.f;
      pos[src] = -1;
      if (ps >= 0 && ps < p.num_pages && pd >= 0 && pd < p.num_pages) {
        from = (long long)ps * PAGE + src % PAGE;
        to = (long long)pd * PAGE + dst % PAGE;
      } else {
        atomicOr(p.status, MLA_STATUS_BAD_PAGE);
      }
    }
    __syncwarp();
#pragma unroll
    for (int j = 0; j < kMoveRows; j += kMoveFlight) {
      uint4 v[kMoveFlight][3];
      float sc[kMoveFlight];
#pragma unroll
      for (int r = 0; r < kMoveFlight; r++) {
        const long long row = __shfl_sync(0xffffffffu, from, j + r);
        if (row < 0) continue;
        const uint4 *s = reinterpret_cast<const uint4 *>(p.cache) + row * units;
#pragma unroll
        for (int k = 0; k < 3; k++)
          if (k * 32 + lane < units) v[r][k] = s[k * 32 + lane];
        if (p.format == MLA_KV_FP8_E4M3 && lane < 4) sc[r] = p.kv_scales[row * 4 + lane];
      }
#pragma unroll
      for (int r = 0; r < kMoveFlight; r++) {
        const long long row = __shfl_sync(0xffffffffu, to, j + r);
        if (row < 0) continue;
        uint4 *d = reinterpret_cast<uint4 *>(p.cache) + row * units;
#pragma unroll
        for (int k = 0; k < 3; k++)
          if (k * 32 + lane < units) d[k * 32 + lane] = v[r][k];
        if (p.format == MLA_KV_FP8_E4M3 && lane < 4) p.kv_scales[row * 4 + lane] = sc[r];
      }
    }
  }
}

int fail(int code, const char *msg) {
  set_last_error(msg);
  return code;
}

bool aligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

int check_sizes(int B, int cap, int keep) {
  char msg[160];
  if (B < 1 || B > MLA_MAX_ITEMS || cap < 1 || keep < 1) {
    snprintf(msg, sizeof msg, "B = %d not in [1, %d], mass_cap = %d < 1 or keep = %d < 1", B, MLA_MAX_ITEMS, cap, keep);
    return fail(MLA_ERR_INVALID_ARG, msg);
  }
  if (cap > (1 << 24)) return fail(MLA_ERR_UNSUPPORTED, "mass_cap exceeds 2^24");
  return MLA_OK;
}

// Rows of one sequence that move, at most.
int room_of(int cap, int keep) { return cap <= keep ? 0 : cap - keep < keep ? cap - keep : keep; }

size_t round256(size_t n) { return (n + 255) / 256 * 256; }

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" size_t mla_evict_workspace_bytes(int B, int mass_cap, int keep) {
  if (check_sizes(B, mass_cap, keep) != MLA_OK) return 0;
  return round256((size_t)B * 4) + 2 * round256((size_t)B * room_of(mass_cap, keep) * 4);
}

extern "C" int mla_evict(void *kv_cache, int kv_format, int num_pages, int page_size, const int32_t *block_table,
                         int max_pages, const int32_t *cache_seqlens, float *kv_scales, float *mass, int32_t *positions,
                         int mass_cap, int keep, int sinks, int recent, int32_t *out_seqlens, void *workspace,
                         size_t workspace_bytes, int B, mla_stream_t stream) {
  int rc = check_sizes(B, mass_cap, keep);
  if (rc != MLA_OK) return rc;
  char msg[160];
  if (sinks < 0 || recent < 0 || (long long)sinks + recent > keep) {
    snprintf(msg, sizeof msg, "sinks = %d and recent = %d must be >= 0 and at most keep = %d together", sinks, recent, keep);
    return fail(MLA_ERR_INVALID_ARG, msg);
  }
  if (!kv_cache || !block_table || !cache_seqlens || !mass || !positions || !out_seqlens)
    return fail(MLA_ERR_INVALID_ARG, "null pointer argument");
  if (kv_format != MLA_KV_BF16 && kv_format != MLA_KV_FP8_E4M3 && kv_format != MLA_KV_FP8_E4M3_TENSOR)
    return fail(MLA_ERR_INVALID_ARG, "kv_format unknown");
  if (!aligned(kv_cache, 16)) return fail(MLA_ERR_INVALID_ARG, "kv_cache must be 16-byte aligned");
  if (!aligned(block_table, 4) || !aligned(cache_seqlens, 4) || !aligned(mass, 4) || !aligned(positions, 4) ||
      !aligned(out_seqlens, 4))
    return fail(MLA_ERR_INVALID_ARG, "int32/fp32 arrays must be 4-byte aligned");
  if (kv_format == MLA_KV_FP8_E4M3 && (!kv_scales || !aligned(kv_scales, 16)))
    return fail(MLA_ERR_INVALID_ARG, "MLA_KV_FP8_E4M3 needs 16-byte aligned kv_scales");
  if (page_size != MLA_PAGE_SIZE) return fail(MLA_ERR_UNSUPPORTED, "page_size must be 64");
  if (num_pages < 1 || max_pages < 1) return fail(MLA_ERR_INVALID_ARG, "num_pages/max_pages < 1");
  const size_t need = mla_evict_workspace_bytes(B, mass_cap, keep);
  if (!workspace || workspace_bytes < need) {
    snprintf(msg, sizeof msg, "workspace needs %zu bytes, got %zu", need, workspace_bytes);
    return fail(MLA_ERR_WORKSPACE, msg);
  }
  if (!aligned(workspace, 256)) return fail(MLA_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  EvictParams p{};
  if ((rc = status_word(&p.status)) != MLA_OK) return rc;
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  p.cache = static_cast<uint8_t *>(kv_cache);
  p.kv_scales = kv_scales;
  p.block_table = block_table;
  p.seqlens = cache_seqlens;
  p.mass = mass;
  p.positions = positions;
  p.out_seqlens = out_seqlens;
  p.format = kv_format;
  p.num_pages = num_pages;
  p.max_pages = max_pages;
  p.cap = mass_cap;
  p.keep = keep;
  p.sinks = sinks;
  p.recent = recent;
  p.room = room_of(mass_cap, keep);
  p.counts = reinterpret_cast<int32_t *>(ws);
  p.holes = reinterpret_cast<int32_t *>(ws + round256((size_t)B * 4));
  p.movers = reinterpret_cast<int32_t *>(ws + round256((size_t)B * 4) + round256((size_t)B * p.room * 4));
  cudaStream_t s = (cudaStream_t)stream;
  int ctas = 1;
  while (ctas < kMostCtas && mass_cap > ctas * kCtaTokens) ctas *= 2;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(B * ctas));
  cfg.blockDim = dim3(kSelectThreads);
  cfg.dynamicSmemBytes = sizeof(SelectShared);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = ctas > 1 ? 2 : 1;
  const auto select = ctas > 1 ? evict_select_kernel<false> : evict_select_kernel<true>;
  cudaError_t e = cudaFuncSetAttribute(select, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)sizeof(SelectShared));
  if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, select, p, ctas);
  if (e == cudaSuccess && p.room > 0) {
    // eight warps of eight rows a block; blocks enough for the GPU, shared out among the sequences
    const int most = ceil_div(p.room, kMoveThreads / 32 * kMoveRows), share = ceil_div(1216, B);
    cfg.gridDim = dim3((unsigned)(most < share ? most : share), (unsigned)B);
    cfg.blockDim = dim3(kMoveThreads);
    cfg.dynamicSmemBytes = 0;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, evict_move_kernel, p);
  }
  if (e != cudaSuccess) {
    snprintf(msg, sizeof msg, "evict: %s", cudaGetErrorString(e));
    return fail(MLA_ERR_CUDA, msg);
  }
  set_last_error("");
  return MLA_OK;
}

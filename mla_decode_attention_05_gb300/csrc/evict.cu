// Eviction from a paged latent cache by accumulated attention weight: of a
// sequence's n > keep cached tokens the first positions (sinks), the latest
// (recent) and the heaviest of the others stay, keep in all, ties in favour of
// the lower slot.  Attention does not depend on the order of slots, so nothing is
// compacted: the stayers behind slot `keep`, in order, move into the slots that
// empty before it, in order.  Sources and targets do not overlap, so all rows
// move at once, and no row moves that need not (sliding the stayers together
// would move nearly every row behind the first hole).
#include <cstdio>

#include "common.cuh"
#include "dependent.cuh"
#include "ptx.cuh"

namespace mla {
namespace {

using namespace ptx;

constexpr int kSelectThreads = 512;
constexpr int kWarps = kSelectThreads / 32;
constexpr int kMostCtas = 8;                 // CTAs of a cluster, one cluster a sequence
constexpr int kKeyCache = 16384;             // sort keys that a CTA keeps in shared memory
constexpr int kMoveThreads = 256;

struct EvictParams {
  uint8_t *cache;
  float *kv_scales;
  const int32_t *block_table, *seqlens;
  float *mass;
  int32_t *positions, *out_seqlens;
  int32_t *counts, *holes, *movers;  // workspace: [B], [B][room], [B][room]
  unsigned int *status;
  int format, num_pages, max_pages, B, cap, keep, sinks, recent, room;
};

struct SelectShared {
  uint32_t keys[kKeyCache];
  int hist[4][256];
  int total[256];
  int newest;
  int ties[kWarps], holes[kWarps], movers[kWarps];
  int base[3][kWarps];
  int digit, above;
  int warp_max[kWarps];
};

__device__ __forceinline__ int ld_cluster(const int *p, uint32_t rank) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(mapa(smem_u32(p), rank)));
  return v;
}

// All threads of the cluster; the lanes of a warp meet first.
__device__ __forceinline__ void meet() {
  __syncwarp();
  cluster_sync();
}

// A weight's place in the order: larger is heavier, -0 is 0, nan below everything.
__device__ __forceinline__ uint32_t order_key(float m) {
  if (m != m) return 0u;
  const uint32_t b = __float_as_uint(m == 0.f ? 0.f : m);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// Cluster b: sequence b.  Warp w of CTA r owns the slots of segment r * kWarps + w.
// The order's keep-th key is found by four passes over its digits of 8 bits.
__global__ void __launch_bounds__(kSelectThreads) evict_select_kernel(EvictParams p, int ctas) {
  extern __shared__ __align__(16) uint8_t smem[];
  SelectShared &sh = *reinterpret_cast<SelectShared *>(smem);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t rank = cluster_ctarank();
  const int b = blockIdx.x / ctas;
  grid_dep_trigger();
  grid_dep_wait();
  const long long most = min((long long)p.max_pages * PAGE, (long long)p.cap);
  const int raw = p.seqlens[b];
  const int n = (int)min((long long)max(raw, 0), most);
  if (n != raw && rank == 0 && tid == 0) atomicOr(p.status, MLA_STATUS_BAD_SEQLEN);
  // (out_seqlens may be seqlens: everyone has read it before it is written)
  meet();
  if (n <= p.keep) {
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
  for (int i = tid; i < 4 * 256; i += kSelectThreads) sh.hist[0][i] = 0;

  int newest = INT32_MIN;
  for (int i = lo + lane; i < hi; i += 32) newest = max(newest, pos[i]);
  newest = __reduce_max_sync(0xffffffffu, newest);
  if (lane == 0) sh.warp_max[warp] = newest;
  __syncthreads();
  if (warp == 0) {
    int v = lane < kWarps ? sh.warp_max[lane] : INT32_MIN;
    v = __reduce_max_sync(0xffffffffu, v);
    if (lane == 0) sh.newest = v;
  }
  meet();
  newest = INT32_MIN;
  for (int r = 0; r < ctas; r++) newest = max(newest, ld_cluster(&sh.newest, r));

  auto fresh_key = [&](int i) {
    const int q = pos[i];
    if (q < p.sinks || (long long)q > (long long)newest - p.recent) return 0xffffffffu;
    return order_key(mass[i]);
  };
  uint32_t *mine = sh.keys + warp * (kKeyCache / kWarps);
  auto key = [&](int i) { return i - lo < kKeyCache / kWarps ? mine[i - lo] : fresh_key(i); };
  uint32_t prefix = 0;
  int want = p.keep;  // of the keys that share the prefix
  for (int pass = 0; pass < 4; pass++) {
    const int shift = 24 - 8 * pass;
    for (int i = lo + lane; i < hi; i += 32) {
      uint32_t k;
      if (pass == 0) {
        k = fresh_key(i);
        if (i - lo < kKeyCache / kWarps) mine[i - lo] = k;
      } else {
        k = key(i);
        if ((k >> (shift + 8)) != prefix) continue;
      }
      atomicAdd(&sh.hist[pass][(k >> shift) & 255], 1);
    }
    meet();
    if (tid < 256) {
      int v = 0;
      for (int r = 0; r < ctas; r++) v += ld_cluster(&sh.hist[pass][tid], r);
      sh.total[tid] = v;
    }
    __syncthreads();
    if (warp == 0) {  // lane l: digits 255 - 8 l ... 248 - 8 l
      int sum = 0;
      for (int j = 0; j < 8; j++) sum += sh.total[255 - 8 * lane - j];
      int incl = sum;
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      int above = incl - sum;
      if (above < want && want <= incl)
        for (int j = 0; j < 8; j++) {
          const int d = 255 - 8 * lane - j;
          if (want <= above + sh.total[d]) {
            sh.digit = d;
            sh.above = above;
            break;
          }
          above += sh.total[d];
        }
    }
    __syncthreads();
    prefix = (prefix << 8) | (uint32_t)sh.digit;
    want -= sh.above;
    __syncthreads();
  }
  // stays: every key above `prefix`, and the first `want` equal ones
  auto exchange = [&](int *counts, int *base) {  // base[w]: of the warps before, in the whole cluster
    meet();
    if (warp == 0) {
      int before = 0;
      for (int r = 0; r < (int)rank; r++) {
        const int v = lane < kWarps ? ld_cluster(&counts[lane], r) : 0;
        before += __reduce_add_sync(0xffffffffu, v);
      }
      int incl = lane < kWarps ? counts[lane] : 0;
      const int own = incl;
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += v;
      }
      if (lane < kWarps) base[lane] = before + incl - own;
    }
    __syncthreads();
  };
  int ties = 0;
  for (int i = lo + lane; i < hi; i += 32) ties += key(i) == prefix;
  ties = __reduce_add_sync(0xffffffffu, ties);
  if (lane == 0) sh.ties[warp] = ties;
  exchange(sh.ties, sh.base[0]);
  const uint32_t below = (1u << lane) - 1u;
  int holes = 0;
  for (int write = 0; write < 2; write++) {
    int tie_at = sh.base[0][warp];
    int hole_at = write ? sh.base[1][warp] : 0, mover_at = write ? sh.base[2][warp] : 0;
    for (int i0 = lo; i0 < hi; i0 += 32) {
      const int i = i0 + lane;
      const uint32_t k = i < hi ? key(i) : 0u;
      const bool tie = i < hi && k == prefix;
      const uint32_t tied = __ballot_sync(0xffffffffu, tie);
      const bool stays = i < hi && (k > prefix || (tie && tie_at + __popc(tied & below) < want));
      tie_at += __popc(tied);
      const bool hole = i < hi && i < p.keep && !stays, mover = i >= p.keep && stays;
      const uint32_t hs = __ballot_sync(0xffffffffu, hole), ms = __ballot_sync(0xffffffffu, mover);
      if (write) {
        if (hole) p.holes[(size_t)b * p.room + hole_at + __popc(hs & below)] = i;
        if (mover) p.movers[(size_t)b * p.room + mover_at + __popc(ms & below)] = i;
        if (i < hi && i >= p.keep && !stays) {
          mass[i] = 0.f;
          pos[i] = -1;
        }
      }
      hole_at += __popc(hs);
      mover_at += __popc(ms);
    }
    if (!write) {
      if (lane == 0) {
        sh.holes[warp] = hole_at;
        sh.movers[warp] = mover_at;
      }
      exchange(sh.holes, sh.base[1]);
      exchange(sh.movers, sh.base[2]);
    } else {
      holes = hole_at;
    }
  }
  if (rank == ctas - 1 && warp == kWarps - 1 && lane == 0) {
    p.counts[b] = holes;
    p.out_seqlens[b] = p.keep;
  }
  meet();  // the others have read this CTA's counts
}

// A warp a row.
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(EvictParams p) {
  extern __shared__ __align__(16) int starts[];  // [B + 1]
  __shared__ int warp_sums[kMoveThreads / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  grid_dep_trigger();
  grid_dep_wait();
  const int per = ceil_div(p.B, kMoveThreads), b0 = min(p.B, tid * per), b1 = min(p.B, b0 + per);
  int mine = 0;
  for (int b = b0; b < b1; b++) mine += p.counts[b];
  int incl = mine;
  for (int o = 1; o < 32; o <<= 1) {
    const int v = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += v;
  }
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  int before = incl - mine;
  for (int i = 0; i < warp; i++) before += warp_sums[i];
  for (int b = b0; b < b1; b++) {
    starts[b] = before;
    before += p.counts[b];
  }
  if (b1 == p.B) starts[p.B] = before;  // (every such thread has the same)
  __syncthreads();
  const int total = starts[p.B];
  const int units = p.format == MLA_KV_BF16 ? 72 : p.format == MLA_KV_FP8_E4M3 ? 40 : 36;  // of 16 bytes
  for (int r = blockIdx.x * (kMoveThreads / 32) + warp; r < total; r += gridDim.x * (kMoveThreads / 32)) {
    int lo = 0, hi = p.B;
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (starts[mid] <= r) lo = mid; else hi = mid;
    }
    const int b = lo, j = r - starts[b];
    const int src = p.movers[(size_t)b * p.room + j], dst = p.holes[(size_t)b * p.room + j];
    const int from = p.block_table[(size_t)b * p.max_pages + src / PAGE], to = p.block_table[(size_t)b * p.max_pages + dst / PAGE];
    if (from >= 0 && from < p.num_pages && to >= 0 && to < p.num_pages) {
      const size_t rs = (size_t)from * PAGE + src % PAGE, rd = (size_t)to * PAGE + dst % PAGE;
      const uint4 *s = reinterpret_cast<const uint4 *>(p.cache) + rs * units;
      uint4 *d = reinterpret_cast<uint4 *>(p.cache) + rd * units;
      uint4 v[3];
#pragma unroll
      for (int k = 0; k < 3; k++)
        if (k * 32 + lane < units) v[k] = s[k * 32 + lane];
      if (p.format == MLA_KV_FP8_E4M3 && lane < 4) p.kv_scales[rd * 4 + lane] = p.kv_scales[rs * 4 + lane];
#pragma unroll
      for (int k = 0; k < 3; k++)
        if (k * 32 + lane < units) d[k * 32 + lane] = v[k];
    } else if (lane == 0) {
      atomicOr(p.status, MLA_STATUS_BAD_PAGE);
    }
    if (lane == 0) {
      float *m = p.mass + (size_t)b * p.cap;
      int32_t *q = p.positions + (size_t)b * p.cap;
      m[dst] = m[src];
      q[dst] = q[src];
      m[src] = 0.f;
      q[src] = -1;
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
  p.B = B;
  p.cap = mass_cap;
  p.keep = keep;
  p.sinks = sinks;
  p.recent = recent;
  p.room = room_of(mass_cap, keep);
  p.counts = reinterpret_cast<int32_t *>(ws);
  p.holes = reinterpret_cast<int32_t *>(ws + round256((size_t)B * 4));
  p.movers = reinterpret_cast<int32_t *>(ws + round256((size_t)B * 4) + round256((size_t)B * p.room * 4));
  cudaStream_t s = (cudaStream_t)stream;
  const int ctas = mass_cap > 4096 ? kMostCtas : 1;
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
  cfg.numAttrs = 2;
  cudaError_t e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                       (int)sizeof(SelectShared));
  if (e == cudaSuccess) e = cudaLaunchKernelEx(&cfg, evict_select_kernel, p, ctas);
  if (e == cudaSuccess && p.room > 0) {
    const long long rows = (long long)B * p.room, blocks = (rows + 7) / 8;
    e = launch_dependent(evict_move_kernel, (unsigned)(blocks < 1216 ? blocks : 1216), kMoveThreads,
                         (unsigned)((B + 1) * sizeof(int)), s, p);
  }
  if (e != cudaSuccess) {
    snprintf(msg, sizeof msg, "evict: %s", cudaGetErrorString(e));
    return fail(MLA_ERR_CUDA, msg);
  }
  set_last_error("");
  return MLA_OK;
}

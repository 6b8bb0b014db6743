// Decode of a batch whose sequences share long prefixes: attention over a
// group's prefix for the query rows of all its sequences together, over each
// sequence's own cache, and the join of the two.
#include <cmath>
#include <cstdio>

#include "common.cuh"
#include "dependent.cuh"

namespace mla {
namespace {

constexpr int kSchedThreads = 1024;
constexpr int kMaxItems = MLA_MAX_ITEMS;

struct SharedParams {
  const __nv_bfloat16 *q;
  const uint8_t *cache;
  const float *kv_scales;
  const int32_t *prefix_table, *prefix_lens, *offsets;  // offsets null: one group of all sequences
  const int32_t *block_table, *seqlens;
  unsigned int *status;
  int format, num_pages, max_prefix, max_pages, G, B, T, H, causal;
  int n_pt;   // room for prefix tiles
  int n_mt;   // own M tiles of a sequence
  int parts;
  // workspace
  int32_t *md_p, *ns_p, *md_o, *ns_o;  // the two schedules
  int32_t *cnt_p, *cnt_o;              // pieces of each item (0: no keys)
  int32_t *lens_p;                     // [n_pt] keys of a prefix tile
  int4 *tile_p;                        // [n_pt] {group, first query row, rows, 0}
  int32_t *table_p;                    // [n_pt][max_prefix]
  int32_t *lens_o;                     // [B] clamped
  int2 *seq;                           // [B] {first prefix tile of its group or -1, its first row among the group's}
  uint8_t *q_p;                        // [n_pt * 128][576] bf16
  uint8_t *scratch;                    // FP8: [G * max_prefix][64][576] bf16
  float *lse_p, *o_p, *lse_o, *o_o;    // partials
  __nv_bfloat16 *out;
  float *lse;
};

template <class Op>
__device__ inline int block_scan(int v, int *warp_sums, int identity, Op op) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v = op(v, u);
  }
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  if (warp == 0) {
    int s = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s = op(s, u);
    }
    warp_sums[lane] = s;
  }
  __syncthreads();
  if (warp > 0) v = op(v, warp_sums[warp - 1]);
  __syncthreads();
  return v;
}

__device__ inline int last_le(const int *C, int n, int x) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (C[mid] <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// The decode kernel's schedule (mla_decode_metadata's rule) of n items with
// tiles(i) key tiles each, but with room for two pieces at least of every item:
// it then writes all its results as fp32 partials.
template <class Tiles>
__device__ void schedule(int n, int parts, int32_t *md_out, int32_t *ns_out, int32_t *cnt, int *C, int *warp_sums,
                         int *carry, Tiles tiles) {
  const int tid = threadIdx.x;
  auto add = [](int a, int b) { return a + b; };
  if (tid == 0) { *carry = 0; C[0] = 0; }
  __syncthreads();
  for (int base = 0; base < n; base += kSchedThreads) {
    const int i = base + tid;
    const int incl = block_scan(i < n ? FIXED_COST + tiles(i) : 0, warp_sums, 0, add);
    if (i < n) C[i + 1] = *carry + incl;
    __syncthreads();
    if (tid == kSchedThreads - 1) *carry += incl;
    __syncthreads();
  }
  const int W = C[n], L = max(ceil_div(W, parts), 1);
  for (int p = tid; p < parts; p += kSchedThreads) {
    int32_t *md = md_out + (size_t)p * MD_STRIDE;
    const long long at = (long long)p * L;
    if (at >= W) {
      md[0] = n; md[1] = 0; md[2] = n - 1; md[3] = 0; md[4] = 0; md[5] = 0; md[6] = 0; md[7] = 0;
      continue;
    }
    const int lo = (int)at, hi = min(lo + L, W);
    const int a = last_le(C, n, lo), z = last_le(C, n, hi - 1);
    const int na = C[a + 1] - C[a] - FIXED_COST, nz = C[z + 1] - C[z] - FIXED_COST;
    md[0] = a;
    md[1] = min(max(lo - C[a] - FIXED_COST, 0), na);
    md[2] = z;
    md[3] = min(max(hi - C[z] - FIXED_COST, 0), nz);
    md[4] = na > 0 ? max(p - (C[a] + FIXED_COST) / L, 0) : 0;
    md[5] = C[a] == lo ? 1 : 0;
    md[6] = 0; md[7] = 0;
  }
  if (tid == 0) *carry = 0;
  __syncthreads();
  for (int base = 0; base < n; base += kSchedThreads) {
    const int i = base + tid;
    int room = 0;
    if (i < n) {
      const int k = C[i + 1] - C[i] - FIXED_COST, first = C[i] + FIXED_COST;
      const int pieces = k == 0 ? 0 : (first + k - 1) / L - first / L + 1;
      cnt[i] = pieces;
      room = max(pieces, 2);
    }
    const int incl = block_scan(room, warp_sums, 0, add);
    if (i < n) ns_out[i + 1] = *carry + incl;
    __syncthreads();
    if (tid == kSchedThreads - 1) *carry += incl;
    __syncthreads();
  }
  if (tid == 0) ns_out[0] = 0;
}

// Block 0: the groups' tiles of 128 query rows and their schedule; block 1: the own caches'.
__global__ void __launch_bounds__(kSchedThreads) shared_schedule_kernel(SharedParams p) {
  __shared__ int C[kMaxItems + 1];
  __shared__ int warp_sums[32];
  __shared__ int carry, top;
  const int tid = threadIdx.x, TH = p.T * p.H;
  grid_dep_trigger();
  grid_dep_wait();
  if (blockIdx.x == 1) {
    const int most = p.max_pages > 0x7fffffff / PAGE ? 0x7fffffff : p.max_pages * PAGE;
    for (int b = tid; b < p.B; b += kSchedThreads) {
      const int n = p.seqlens[b];
      if (n < 0 || n > most) atomicOr(p.status, MLA_STATUS_BAD_SEQLEN);
      p.lens_o[b] = min(max(n, 0), most);
    }
    __syncthreads();
    schedule(p.B * p.n_mt, p.parts, p.md_o, p.ns_o, p.cnt_o, C, warp_sums, &carry, [&](int i) {
      return item_at(i, p.lens_o, p.B, p.H, p.T, 0, p.causal, p.status).ntiles;
    });
    return;
  }
  for (int b = tid; b < p.B; b += kSchedThreads) p.seq[b] = make_int2(-1, 0);
  if (tid == 0) { carry = 0; top = 0; }
  __syncthreads();
  const int most = p.max_prefix > 0x7fffffff / PAGE ? 0x7fffffff : p.max_prefix * PAGE;
  // (tiles are numbered among the groups that have any keys)
  for (int base = 0; base < p.G; base += kSchedThreads) {
    const int g = base + tid;
    int b0 = 0, b1 = 0, n = 0;
    bool bad = false;
    if (g < p.G) {
      b0 = p.offsets ? p.offsets[g] : 0;
      b1 = p.offsets ? p.offsets[g + 1] : p.B;
      bad = b0 < 0 || b0 > b1 || b1 > p.B;
      n = p.prefix_lens[g];
      bad = bad || n < 0 || n > most;
      n = min(max(n, 0), most);
      if (bad) atomicOr(p.status, MLA_STATUS_BAD_SEQLEN);
    }
    // offsets out of order are pulled up to the largest before them
    const int ceil1 = max(block_scan(min(max(max(b0, b1), 0), p.B), warp_sums, 0, [](int a, int b) { return max(a, b); }), top);
    int before = __shfl_up_sync(0xffffffffu, ceil1, 1);
    if ((tid & 31) == 31) warp_sums[tid >> 5] = ceil1;
    __syncthreads();
    if ((tid & 31) == 0) before = tid == 0 ? top : warp_sums[(tid >> 5) - 1];
    __syncthreads();
    b0 = min(max(max(b0, before), 0), p.B);
    b1 = max(min(max(b1, b0), p.B), b0);
    const int rows = (b1 - b0) * TH;
    const int tiles = g < p.G && n > 0 ? ceil_div(rows, M_TILE) : 0;
    const int incl = block_scan(tiles, warp_sums, 0, [](int a, int b) { return a + b; });
    const int first = carry + incl - tiles;
    for (int t = 0; t < tiles; t++) {
      p.tile_p[first + t] = make_int4(g, b0 * TH + t * M_TILE, min(M_TILE, rows - t * M_TILE), 0);
      p.lens_p[first + t] = n;
    }
    if (tiles > 0)
      for (int b = b0; b < b1; b++) p.seq[b] = make_int2(first, (b - b0) * TH);
    __syncthreads();
    if (tid == kSchedThreads - 1) { carry += incl; top = max(top, ceil1); }
    __syncthreads();
  }
  const int n_tiles = carry;
  __syncthreads();
  for (int t = n_tiles + tid; t < p.n_pt; t += kSchedThreads) {
    p.lens_p[t] = 0;
    p.tile_p[t] = make_int4(-1, 0, 0, 0);
  }
  schedule(n_tiles, p.parts, p.md_p, p.ns_p, p.cnt_p, C, warp_sums, &carry,
           [&](int i) { return ceil_div(p.lens_p[i], PAGE); });
}

// Block t: the query rows of prefix tile t side by side, and its group's pages.
__global__ void __launch_bounds__(256) shared_pack_kernel(SharedParams p) {
  grid_dep_trigger();
  grid_dep_wait();
  const int t = blockIdx.x;
  const int4 tile = p.tile_p[t];
  if (tile.x < 0) return;
  const uint4 *src = reinterpret_cast<const uint4 *>(p.q) + (size_t)tile.y * (D_QK / 8);
  uint4 *dst = reinterpret_cast<uint4 *>(p.q_p) + (size_t)t * M_TILE * (D_QK / 8);
  for (int i = threadIdx.x; i < tile.z * (D_QK / 8); i += blockDim.x) dst[i] = src[i];
  for (int j = threadIdx.x; j < p.max_prefix; j += blockDim.x) {
    int page = p.prefix_table[(size_t)tile.x * p.max_prefix + j];
    if (p.format != MLA_KV_BF16) {
      if (page >= 0 && page < p.num_pages) page = tile.x * p.max_prefix + j;
      else page = -1;
    }
    p.table_p[(size_t)t * p.max_prefix + j] = page;
  }
}

// FP8 prefixes: page j of group g as bf16 rows, once for all its tiles.
__global__ void __launch_bounds__(256) shared_widen_kernel(SharedParams p) {
  grid_dep_trigger();
  grid_dep_wait();
  const int g = blockIdx.y;
  const int n = min(p.prefix_lens[g], p.max_prefix * PAGE);
  for (int j = blockIdx.x; j * PAGE < n; j += gridDim.x) {
    const int page = p.prefix_table[(size_t)g * p.max_prefix + j];
    if (page < 0 || page >= p.num_pages) continue;
    __nv_bfloat16 *dst = reinterpret_cast<__nv_bfloat16 *>(p.scratch) + ((size_t)g * p.max_prefix + j) * PAGE * D_QK;
    const bool tensor = p.format == MLA_KV_FP8_E4M3_TENSOR;
    const int row_bytes = tensor ? D_QK : FP8_ROW;
    for (int i = threadIdx.x; i < PAGE * D_QK; i += blockDim.x) {
      const int r = i / D_QK, d = i % D_QK;
      const uint8_t *src = p.cache + ((size_t)page * PAGE + r) * row_bytes;
      float v = 0.f;
      if (j * PAGE + r < n) {
        if (d < D_V || tensor) {
          const float s = tensor ? p.kv_scales[0] : p.kv_scales[((size_t)page * PAGE + r) * 4 + d / 128];
          v = e4m3_to_float(src[d]) * s;
        } else {
          v = bf16_bits_to_float(reinterpret_cast<const uint16_t *>(src + D_V)[d - D_V]);
        }
      }
      dst[i] = __float2bfloat16_rn(v);
    }
  }
}

// ---- join ------------------------------------------------------------------------

constexpr int kWarps = 8, kChunks = 4;

__device__ __forceinline__ void ld_cg_v8(float (&v)[8], const float *ptr) {
  uint32_t u[8];
  asm volatile("ld.global.cg.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7])
               : "l"(ptr));
#pragma unroll
  for (int j = 0; j < 8; j++) v[j] = __uint_as_float(u[j]);
}

// Lane: one query row; warp: 32 of its columns; block: 32 rows x 256 columns.
__global__ void __launch_bounds__(kWarps * 32) shared_join_kernel(SharedParams p) {
  grid_dep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, TH = p.T * p.H;
  const long long R = (long long)blockIdx.x * 32 + lane;
  if (R >= (long long)p.B * TH) return;
  const int b = (int)(R / TH), r = (int)(R % TH);
  const int chunk0 = blockIdx.y * 32 + warp * kChunks;
  const float *lse_part[2] = {nullptr, nullptr};
  const float *o_part[2] = {nullptr, nullptr};
  int n[2] = {0, 0};
  const int2 s = p.seq[b];
  if (s.x >= 0) {
    const int row = s.y + r, i = s.x + row / M_TILE, at = row % M_TILE;
    n[0] = p.cnt_p[i];
    lse_part[0] = p.lse_p + (size_t)p.ns_p[i] * M_TILE + at;
    o_part[0] = p.o_p + (((size_t)p.ns_p[i] * 64 + chunk0) * M_TILE + at) * 8;
  }
  {
    const int i = (r / M_TILE) * p.B + b, at = r % M_TILE;
    n[1] = p.cnt_o[i];
    lse_part[1] = p.lse_o + (size_t)p.ns_o[i] * M_TILE + at;
    o_part[1] = p.o_o + (((size_t)p.ns_o[i] * 64 + chunk0) * M_TILE + at) * 8;
  }
  float m = -INFINITY;
  for (int k = 0; k < 2; k++)
    for (int j = 0; j < n[k]; j++) m = fmaxf(m, __ldcg(lse_part[k] + (size_t)j * M_TILE));
  float acc[kChunks * 8], sum = 0.f;
#pragma unroll
  for (int k = 0; k < kChunks * 8; k++) acc[k] = 0.f;
  if (m != -INFINITY)
    for (int k = 0; k < 2; k++)
      for (int j = 0; j < n[k]; j++) {
        const float l = __ldcg(lse_part[k] + (size_t)j * M_TILE);
        const float w = l == -INFINITY ? 0.f : exp2f(l - m);
        sum += w;
#pragma unroll
        for (int c = 0; c < kChunks; c++) {
          float v[8];
          ld_cg_v8(v, o_part[k] + ((size_t)j * 64 + c) * M_TILE * 8);
#pragma unroll
          for (int e = 0; e < 8; e++) acc[8 * c + e] = fmaf(w, v[e], acc[8 * c + e]);
        }
      }
  const float inv = sum > 0.f ? 1.f / sum : 0.f;
  uint4 *dst = reinterpret_cast<uint4 *>(p.out + R * D_V + chunk0 * 8);
#pragma unroll
  for (int c = 0; c < kChunks; c++) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; e++) {
      __nv_bfloat162 v = __floats2bfloat162_rn(acc[8 * c + 2 * e] * inv, acc[8 * c + 2 * e + 1] * inv);
      w[e] = *reinterpret_cast<uint32_t *>(&v);
    }
    dst[c] = make_uint4(w[0], w[1], w[2], w[3]);
  }
  if (warp == 0 && blockIdx.y == 0)
    p.lse[((size_t)b * p.H + r % p.H) * p.T + r / p.H] = sum > 0.f ? (m + log2f(sum)) * LN2 : -INFINITY;
}

// ---- host ------------------------------------------------------------------------

struct Layout {
  size_t md_p, ns_p, md_o, ns_o, cnt_p, cnt_o, lens_p, tile_p, table_p, lens_o, seq, q_p, scratch, lse_p, o_p, lse_o, o_o,
      ring, total;
  int n_pt, n_mt;
};

Layout layout(int B, int T, int H, int G, int format, int max_prefix, int parts) {
  Layout l;
  l.n_pt = (int)(((long long)B * T * H + M_TILE - 1) / M_TILE) + G;
  l.n_mt = ceil_div(T * H, M_TILE);
  const size_t n_ot = (size_t)B * l.n_mt;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at = (at + bytes + 255) / 256 * 256;
    return here;
  };
  const size_t slots_p = 2 * (size_t)l.n_pt + parts, slots_o = 2 * n_ot + parts, row = M_TILE * sizeof(float);
  l.md_p = take((size_t)parts * MD_STRIDE * 4);
  l.ns_p = take(((size_t)l.n_pt + 1) * 4);
  l.md_o = take((size_t)parts * MD_STRIDE * 4);
  l.ns_o = take((n_ot + 1) * 4);
  l.cnt_p = take((size_t)l.n_pt * 4);
  l.cnt_o = take(n_ot * 4);
  l.lens_p = take((size_t)l.n_pt * 4);
  l.tile_p = take((size_t)l.n_pt * sizeof(int4));
  l.table_p = take((size_t)l.n_pt * max_prefix * 4);
  l.lens_o = take((size_t)B * 4);
  l.seq = take((size_t)B * sizeof(int2));
  l.q_p = take((size_t)l.n_pt * M_TILE * D_QK * 2);
  l.scratch = take(format == MLA_KV_BF16 ? 0 : (size_t)G * max_prefix * PAGE * D_QK * 2);
  l.lse_p = take(slots_p * row);
  l.o_p = take(slots_p * row * D_V);
  l.lse_o = take(slots_o * row);
  l.o_o = take(slots_o * row * D_V);
  l.ring = take((size_t)parts * P_RING * P_SLOT_BYTES);
  l.total = at;
  return l;
}

int fail(int code, const char *msg) {
  set_last_error(msg);
  return code;
}

int check_sizes(int B, int T, int H, int G, int format, int max_prefix) {
  char msg[160];
  if (B < 1 || G < 1 || max_prefix < 1) {
    snprintf(msg, sizeof msg, "B = %d, G = %d and max_prefix_pages = %d must be >= 1", B, G, max_prefix);
    return fail(MLA_ERR_INVALID_ARG, msg);
  }
  if (H < 1 || H > MLA_MAX_HEADS || T < 1 || T > MLA_MAX_QUERY_TOKENS) {
    snprintf(msg, sizeof msg, "H = %d not in [1, %d] or T = %d not in [1, %d]", H, MLA_MAX_HEADS, T, MLA_MAX_QUERY_TOKENS);
    return fail(MLA_ERR_INVALID_ARG, msg);
  }
  if (format != MLA_KV_BF16 && format != MLA_KV_FP8_E4M3 && format != MLA_KV_FP8_E4M3_TENSOR)
    return fail(MLA_ERR_INVALID_ARG, "kv_format unknown");
  const long long own = (long long)B * ceil_div(T * H, M_TILE), shared = ((long long)B * T * H + M_TILE - 1) / M_TILE + G;
  if (own > kMaxItems || shared > kMaxItems) {
    snprintf(msg, sizeof msg, "%lld work items exceed the limit %d", own > shared ? own : shared, kMaxItems);
    return fail(MLA_ERR_UNSUPPORTED, msg);
  }
  if ((long long)G * max_prefix > 0x7fffffffLL) return fail(MLA_ERR_UNSUPPORTED, "G * max_prefix_pages exceeds 2^31 - 1");
  return MLA_OK;
}

int device_parts(int *parts) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return fail(MLA_ERR_CUDA, "cudaGetDevice failed");
  *parts = mla_default_num_parts(dev);
  return *parts > 0 ? MLA_OK : MLA_ERR_CUDA;
}

bool aligned(const void *p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

}  // namespace
}  // namespace mla

using namespace mla;

extern "C" size_t mla_decode_shared_workspace_bytes(int B, int T, int H, int G, int kv_format, int max_prefix_pages) {
  int parts = 0;
  if (check_sizes(B, T, H, G, kv_format, max_prefix_pages) != MLA_OK || device_parts(&parts) != MLA_OK) return 0;
  return layout(B, T, H, G, kv_format, max_prefix_pages, parts).total;
}

extern "C" int mla_decode_shared(const void *q, const void *kv_cache, int kv_format, int num_pages, int page_size,
                                 const int32_t *prefix_table, int max_prefix_pages, const int32_t *prefix_lens,
                                 const int32_t *group_offsets, int G, const int32_t *block_table, int max_pages,
                                 const int32_t *cache_seqlens, const float *kv_scales, float softmax_scale, int causal,
                                 void *workspace, size_t workspace_bytes, void *out, float *lse, int B, int T, int H,
                                 mla_stream_t stream) {
  int rc = check_sizes(B, T, H, G, kv_format, max_prefix_pages);
  if (rc != MLA_OK) return rc;
  if (!q || !kv_cache || !prefix_table || !prefix_lens || !block_table || !cache_seqlens || !out || !lse)
    return fail(MLA_ERR_INVALID_ARG, "null pointer argument");
  if (!group_offsets && G != 1) return fail(MLA_ERR_INVALID_ARG, "group_offsets may be null for one group only");
  if (!aligned(q, 16) || !aligned(kv_cache, 16) || !aligned(out, 16))
    return fail(MLA_ERR_INVALID_ARG, "q, kv_cache and out must be 16-byte aligned");
  if (!aligned(prefix_table, 4) || !aligned(prefix_lens, 4) || !aligned(group_offsets, 4) || !aligned(block_table, 4) ||
      !aligned(cache_seqlens, 4) || !aligned(lse, 4))
    return fail(MLA_ERR_INVALID_ARG, "int32/fp32 arrays must be 4-byte aligned");
  if (kv_format != MLA_KV_BF16 && (!kv_scales || !aligned(kv_scales, kv_format == MLA_KV_FP8_E4M3 ? 16 : 4)))
    return fail(MLA_ERR_INVALID_ARG, "an FP8 cache needs aligned kv_scales");
  if (page_size != MLA_PAGE_SIZE) return fail(MLA_ERR_UNSUPPORTED, "page_size must be 64");
  if (num_pages < 1 || max_pages < 1) return fail(MLA_ERR_INVALID_ARG, "num_pages/max_pages < 1");
  if (causal != 0 && causal != 1) return fail(MLA_ERR_INVALID_ARG, "causal must be 0 or 1");
  if (!(softmax_scale > 0.f) || !std::isfinite(softmax_scale))
    return fail(MLA_ERR_INVALID_ARG, "softmax_scale must be finite and > 0");
  int parts = 0;
  if ((rc = device_parts(&parts)) != MLA_OK) return rc;
  const Layout l = layout(B, T, H, G, kv_format, max_prefix_pages, parts);
  if (!workspace || workspace_bytes < l.total) {
    char msg[96];
    snprintf(msg, sizeof msg, "workspace needs %zu bytes, got %zu", l.total, workspace_bytes);
    return fail(MLA_ERR_WORKSPACE, msg);
  }
  if (!aligned(workspace, 256)) return fail(MLA_ERR_INVALID_ARG, "workspace must be 256-byte aligned");
  unsigned int *st = nullptr;
  if ((rc = status_word(&st)) != MLA_OK) return rc;

  uint8_t *ws = static_cast<uint8_t *>(workspace);
  auto at = [&](size_t off) { return ws + off; };
  SharedParams p{};
  p.q = static_cast<const __nv_bfloat16 *>(q);
  p.cache = static_cast<const uint8_t *>(kv_cache);
  p.kv_scales = kv_scales;
  p.prefix_table = prefix_table;
  p.prefix_lens = prefix_lens;
  p.offsets = group_offsets;
  p.block_table = block_table;
  p.seqlens = cache_seqlens;
  p.status = st;
  p.format = kv_format;
  p.num_pages = num_pages;
  p.max_prefix = max_prefix_pages;
  p.max_pages = max_pages;
  p.G = G;
  p.B = B;
  p.T = T;
  p.H = H;
  p.causal = causal;
  p.n_pt = l.n_pt;
  p.n_mt = l.n_mt;
  p.parts = parts;
  p.md_p = reinterpret_cast<int32_t *>(at(l.md_p));
  p.ns_p = reinterpret_cast<int32_t *>(at(l.ns_p));
  p.md_o = reinterpret_cast<int32_t *>(at(l.md_o));
  p.ns_o = reinterpret_cast<int32_t *>(at(l.ns_o));
  p.cnt_p = reinterpret_cast<int32_t *>(at(l.cnt_p));
  p.cnt_o = reinterpret_cast<int32_t *>(at(l.cnt_o));
  p.lens_p = reinterpret_cast<int32_t *>(at(l.lens_p));
  p.tile_p = reinterpret_cast<int4 *>(at(l.tile_p));
  p.table_p = reinterpret_cast<int32_t *>(at(l.table_p));
  p.lens_o = reinterpret_cast<int32_t *>(at(l.lens_o));
  p.seq = reinterpret_cast<int2 *>(at(l.seq));
  p.q_p = at(l.q_p);
  p.scratch = at(l.scratch);
  p.lse_p = reinterpret_cast<float *>(at(l.lse_p));
  p.o_p = reinterpret_cast<float *>(at(l.o_p));
  p.lse_o = reinterpret_cast<float *>(at(l.lse_o));
  p.o_o = reinterpret_cast<float *>(at(l.o_o));
  p.out = static_cast<__nv_bfloat16 *>(out);
  p.lse = lse;

  DecodeParams own{};
  own.q = p.q;
  own.kv = p.cache;
  own.kv_scales = kv_scales;
  own.block_table = block_table;
  own.seqlens = p.lens_o;
  own.tile_md = p.md_o;
  own.num_splits = p.ns_o;
  own.ws_lse = p.lse_o;
  own.ws_o = p.o_o;
  own.ws_p = at(l.ring);
  own.out = p.out;
  own.lse = p.lse;
  own.status = st;
  own.kv_format = kv_format;
  own.num_pages = num_pages;
  own.max_pages = max_pages;
  own.causal = causal;
  own.B = B;
  own.T = T;
  own.H = H;
  own.n_mt = l.n_mt;
  own.n_items = B * l.n_mt;
  own.num_parts = parts;
  own.out_v8 = 0;
  own.scale_log2 = softmax_scale * LOG2E;
  own.wait_ns = wait_limit_ns();
  own.help = kv_format != MLA_KV_BF16 && T * H <= 64 ? 1 : 0;

  // (a tile of prefix rows is a sequence of one token and 128 heads)
  DecodeParams pre = own;
  pre.q = reinterpret_cast<const __nv_bfloat16 *>(p.q_p);
  pre.kv = kv_format == MLA_KV_BF16 ? p.cache : p.scratch;
  pre.block_table = p.table_p;
  pre.seqlens = p.lens_p;
  pre.tile_md = p.md_p;
  pre.num_splits = p.ns_p;
  pre.ws_lse = p.lse_p;
  pre.ws_o = p.o_p;
  pre.kv_format = MLA_KV_BF16;
  pre.num_pages = kv_format == MLA_KV_BF16 ? num_pages : G * max_prefix_pages;
  pre.max_pages = max_prefix_pages;
  pre.causal = 0;
  pre.B = l.n_pt;
  pre.T = 1;
  pre.H = M_TILE;
  pre.n_mt = 1;
  pre.n_items = l.n_pt;
  pre.help = 0;

  cudaStream_t s = (cudaStream_t)stream;
  cudaError_t e = launch_dependent(shared_schedule_kernel, 2, kSchedThreads, 0, s, p);
  if (e == cudaSuccess && kv_format != MLA_KV_BF16) {
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(max_prefix_pages < 1024 ? max_prefix_pages : 1024, G);
    cfg.blockDim = dim3(256);
    cfg.stream = s;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, shared_widen_kernel, p);
  }
  if (e == cudaSuccess) e = launch_dependent(shared_pack_kernel, l.n_pt, 256, 0, s, p);
  if (e == cudaSuccess) e = launch_decode(pre, s, nullptr, nullptr);
  if (e == cudaSuccess) e = launch_decode(own, s, nullptr, nullptr);
  if (e == cudaSuccess) {
    cudaLaunchAttribute pdl[1];
    pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    pdl[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(((long long)B * T * H + 31) / 32), 2);
    cfg.blockDim = dim3(kWarps * 32);
    cfg.stream = s;
    cfg.attrs = pdl;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, shared_join_kernel, p);
  }
  if (e != cudaSuccess) {
    char msg[128];
    snprintf(msg, sizeof msg, "decode over shared prefixes: %s", cudaGetErrorString(e));
    return fail(MLA_ERR_CUDA, msg);
  }
  set_last_error("");
  return MLA_OK;
}

// Decode of a batch whose sequences share long prefixes: the schedule, the
// widening of FP8 prefixes, the join of prefix and own parts, and the C entry.
//
// For a query row with parts s over disjoint keys (its group's prefix and its own
// tokens, each perhaps split over several workers), L_s = log2 sum 2^score and
// O_s = sum 2^(score - L_s) v:
//   L = log2 sum_s 2^L_s,  O = sum_s 2^(L_s - L) O_s
// and a part without keys has L_s = -inf and weight 0 (see also kAllLow).
#include <cmath>
#include <cstdio>

#include "dependent.cuh"
#include "fp8.cuh"
#include "shared_prefix.cuh"

namespace mla {
namespace {

constexpr int kMaxItems = MLA_MAX_ITEMS;

template <int kSchedThreads, class Op>
__device__ inline int block_scan(int v, int *warp_sums, Op op) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v = op(v, u);
  }
  if (lane == 31) warp_sums[warp] = v;
  __syncthreads();
  if (warp == 0) {
    int s = lane < kSchedThreads / 32 ? warp_sums[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s = op(s, u);
    }
    if (lane < kSchedThreads / 32) warp_sums[lane] = s;
  }
  __syncthreads();
  if (warp > 0) v = op(v, warp_sums[warp - 1]);
  __syncthreads();
  return v;
}

struct Add {
  __device__ int operator()(int a, int b) const { return a + b; }
};
struct Max {
  __device__ int operator()(int a, int b) const { return max(a, b); }
};

// The largest i in [0, n) with at(i) <= x (at(0) <= x, nondecreasing).
template <class At>
__device__ inline int last_le(int n, int x, At at) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (at(mid) <= x) lo = mid; else hi = mid - 1;
  }
  return lo;
}

constexpr int kGroupCache = 256;  // groups that are kept in shared memory
constexpr int kMostParts = 511;

constexpr int kFewThreads = 256;  // of the schedule's block where that is enough for items, sequences, groups and workers

struct SchedShared {
  int C[kMaxItems + 1];
  int cuts[kMostParts + 1];  // where each worker's segment of the line begins, and the end
  uint8_t head[kMaxItems];
  int4 groups[kGroupCache];
  int lens[kFewThreads];  // own tokens, where there are no more sequences
  int warp_sums[32];
  int carry, top;
};

struct Cost {
  int head, tiles;
};

// Two kinds of items lie on one line, those from `from` on of the second kind.  A worker that
// begins within an item has that item's head to do again, which is not on the line.
struct Kinds {
  int from, head1, head2;  // heads of a usual item of each
};

// How much of the line a worker gets of each kind, c1 and c2, so that all have the same to do:
//   c1 + head1 = c2 + head2 = L,  W1 / c1 + W2 / c2 = parts
// which is a quadratic equation for L (its larger root).
__device__ __forceinline__ float2 shares(const Kinds &k, int W1, int W2, int parts) {
  const float n = (float)parts, w1 = (float)W1, w2 = (float)W2;
  const float h1 = W1 > 0 ? (float)k.head1 : 0.f, h2 = W2 > 0 ? (float)k.head2 : 0.f;
  const float b = n * (h1 + h2) + w1 + w2, c = n * h1 * h2 + w1 * h2 + w2 * h1;
  const float L = (b + sqrtf(fmaxf(b * b - 4.f * n * c, 0.f))) / (2.f * n);
  return make_float2(fmaxf(L - h1, 1.f), fmaxf(L - h2, 1.f));
}

// The schedule of n items: item i costs head + tiles, as item(i) says, on a
// line that is cut into `parts` segments (mla_decode_metadata's form).  Writes the segments, the pieces
// of each item and its first slot of results; `least`: slots that every item has
// at least.
template <int kSchedThreads, class Item, class Slot>
__device__ void schedule(SchedShared &sh, int n, int parts, int least, int32_t *md_out, int32_t *pieces, const Kinds &kinds,
                         Item item, Slot slot) {
  const int tid = threadIdx.x;
  if (tid == 0) { sh.carry = 0; sh.C[0] = 0; }
  __syncthreads();
  for (int base = 0; base < n; base += kSchedThreads) {
    const int i = base + tid;
    Cost cost = {0, 0};
    if (i < n) {
      cost = item(i);
      sh.head[i] = (uint8_t)cost.head;
    }
    const int incl = block_scan<kSchedThreads>(cost.head + cost.tiles, sh.warp_sums, Add()) + sh.carry;
    if (i < n) sh.C[i + 1] = incl;
    __syncthreads();
    if (tid == kSchedThreads - 1) sh.carry = incl;
    __syncthreads();
  }
  const int W = sh.C[n], W1 = sh.C[min(kinds.from, n)];
  const float2 c = shares(kinds, W1, W - W1, parts);
  const float border = (float)W1 / c.x;
  {
    // no two cuts at one place before the end: every segment has a tile or a head
    const float at = (float)tid <= border ? tid * c.x : W1 + (tid - border) * c.y;
    const int cut = block_scan<kSchedThreads>(tid < parts ? (int)fminf(at, (float)W) - tid : INT32_MIN, sh.warp_sums, Max());
    if (tid <= parts) sh.cuts[tid] = tid < parts ? min(cut + tid, W) : W;
    __syncthreads();
  }
  const float per1 = 1.f / c.x, per2 = 1.f / c.y;
  auto worker = [&](int x) {  // the last whose segment begins at x or before: near where the shares put it
    int p = min(max((int)(x < W1 ? x * per1 : border + (x - W1) * per2), 0), parts - 1);
    while (p > 0 && sh.cuts[p] > x) p--;
    while (p + 1 < parts && sh.cuts[p + 1] <= x) p++;
    return p;
  };
  for (int p = tid; p < parts; p += kSchedThreads) {
    const int lo = sh.cuts[p], hi = sh.cuts[p + 1];
    int4 lo4 = make_int4(n, 0, n - 1, 0), hi4 = make_int4(0, 0, 0, 0);
    if (lo < W) {
      auto C = [&](int i) { return sh.C[i]; };
      const int a = last_le(n, lo, C), z = last_le(n, hi - 1, C);
      const int fa = sh.C[a] + sh.head[a], fz = sh.C[z] + sh.head[z];  // where their first tiles lie
      const int na = sh.C[a + 1] - fa, nz = sh.C[z + 1] - fz;
      lo4 = make_int4(a, min(max(lo - fa, 0), na), z, min(max(hi - fz, 0), nz));
      hi4 = make_int4(na > 0 ? max(p - worker(fa), 0) : 0, sh.C[a] == lo ? 1 : 0, 0, 0);
    }
    reinterpret_cast<int4 *>(md_out)[2 * p] = lo4;
    reinterpret_cast<int4 *>(md_out)[2 * p + 1] = hi4;
  }
  if (tid == 0) sh.carry = 0;
  __syncthreads();
  for (int base = 0; base < n; base += kSchedThreads) {
    const int i = base + tid;
    int room = 0;
    if (i < n) {
      const int first = sh.C[i] + sh.head[i], k = sh.C[i + 1] - first;
      const int got = k == 0 ? 0 : worker(first + k - 1) - worker(first) + 1;
      pieces[i] = got;
      room = max(got, least);
    }
    const int incl = block_scan<kSchedThreads>(room, sh.warp_sums, Add()) + sh.carry;
    if (i < n) slot(i, incl - room, incl);
    __syncthreads();
    if (tid == kSchedThreads - 1) sh.carry = incl;
    __syncthreads();
  }
}

// An item's head, in tiles: its queries' way into tensor memory and its results' way out.  On 80
// workers' times over eight batches (bf16, one scale): 6.7 us + 0.78 a tile of a prefix + 0.85 of own
// tokens + 1.1 an item + 1.2 for each 32 of its rows; with a scale for each 128 values a tile takes 1.4 us and an item
// of 128 rows 4.2.  (Heads of 2 + rows / 32 for all, and equal parts of the line: 228 instead of 221 us for 64
// sequences of 128 heads on 16384 shared tokens, FP8 groups 163 instead of 155.)
__device__ __forceinline__ int head_of(const SharedParams &p, int rows) {
  const int r = ceil_div(rows, 32);
  return p.format == MLA_KV_FP8_E4M3 ? 1 + (r + 1) / 2 : (3 + 3 * r) / 2;
}

// Keys of the last row of own tile mt of a sequence of n tokens.
__device__ __forceinline__ int own_keys(const SharedParams &p, int n, int mt) {
  const int last = min((mt + 1) * M_TILE, p.T * p.H) - 1;
  return row_kv_len(n, p.T, last / p.H, p.causal);
}

// Block 0: the items of shared_attention_kernel, prefixes first, and their
// schedule.  Block 1 (FP8): where widened pages lie.  Block 2 (FP8, where own pages in use may be more
// than there is room for): the decode kernel's schedule of the own tokens, with room for two pieces
// of every item, so that it writes all its results as partials; an empty one where there is room.
template <int kSchedThreads>
__global__ void __launch_bounds__(kSchedThreads) shared_schedule_kernel(SharedParams p) {
  __shared__ SchedShared sh;
  const int tid = threadIdx.x, TH = p.T * p.H;
  grid_dep_trigger();
  grid_dep_wait();
  auto length = [&](int n, int pages) {
    const int most = pages > 0x7fffffff / PAGE ? 0x7fffffff : pages * PAGE;
    if (n < 0 || n > most) atomicOr(p.status, MLA_STATUS_BAD_SEQLEN);
    return min(max(n, 0), most);
  };
  const bool near_by = p.B <= kFewThreads;
  if (near_by && tid < p.B) sh.lens[tid] = p.seqlens[tid];  // (seen behind the groups' barriers)
  bool apart = false;  // own tokens go another way: their pages in use are more than there is room for
  if (p.md_o) {
    int pages = 0;
    for (int b = tid; b < p.B; b += kSchedThreads) pages += ceil_div(length(p.seqlens[b], p.max_pages), PAGE);
    pages = block_scan<kSchedThreads>(pages, sh.warp_sums, Add());
    if (tid == kSchedThreads - 1) sh.top = pages;
    __syncthreads();
    apart = sh.top > p.own_room;
    __syncthreads();
  }
  if (blockIdx.x == 1) {
    if (tid == 0) {
      sh.carry = 0;
      p.first[0] = 0;
    }
    __syncthreads();
    for (int base = 0; base < p.G + p.B; base += kSchedThreads) {
      const int y = base + tid;
      int pages = 0;
      if (y < p.G) pages = ceil_div(length(p.prefix_lens[y], p.max_prefix), PAGE);
      else if (y < p.G + p.B && !apart) pages = ceil_div(length(p.seqlens[y - p.G], p.max_pages), PAGE);
      const int incl = block_scan<kSchedThreads>(pages, sh.warp_sums, Add()) + sh.carry;
      if (y < p.G + p.B) p.first[y + 1] = incl;
      __syncthreads();
      if (tid == kSchedThreads - 1) sh.carry = incl;
      __syncthreads();
    }
    return;
  }
  if (blockIdx.x == 2) {
    if (!apart) {
      for (int w = tid; w < p.parts; w += kSchedThreads) {
        reinterpret_cast<int4 *>(p.md_o)[2 * w] = make_int4(p.B * p.n_mt, 0, p.B * p.n_mt - 1, 0);
        reinterpret_cast<int4 *>(p.md_o)[2 * w + 1] = make_int4(0, 0, 0, 0);
      }
      return;
    }
    for (int b = tid; b < p.B; b += kSchedThreads) p.lens_o[b] = length(p.seqlens[b], p.max_pages);
    __syncthreads();
    schedule<kSchedThreads>(sh, p.B * p.n_mt, p.parts, 2, p.md_o, p.cnt_o, Kinds{0, 0, 0},
             [&](int i) { return Cost{FIXED_COST, ceil_div(own_keys(p, p.lens_o[i % p.B], i / p.B), PAGE)}; },
             [&](int i, int at, int end) {
               if (i == 0) p.ns_o[0] = 0;
               p.ns_o[i + 1] = end;
             });
    return;
  }
  // groups: {first sequence, end, first item, keys}; items are numbered among the
  // groups that have keys and sequences
  int4 *groups = p.G <= kGroupCache ? sh.groups : p.groups;
  if (tid == 0) { sh.carry = 0; sh.top = 0; }
  __syncthreads();
  for (int base = 0; base < p.G; base += kSchedThreads) {
    const int g = base + tid;
    int b0 = 0, b1 = 0, n = 0;
    if (g < p.G) {
      b0 = p.offsets ? p.offsets[g] : 0;
      b1 = p.offsets ? p.offsets[g + 1] : p.B;
      if (b0 < 0 || b0 > b1 || b1 > p.B) atomicOr(p.status, MLA_STATUS_BAD_SEQLEN);
      n = length(p.prefix_lens[g], p.max_prefix);
    }
    // a group that begins before the end of an earlier one begins there
    const int reach = max(block_scan<kSchedThreads>(min(max(max(b0, b1), 0), p.B), sh.warp_sums, Max()), sh.top);
    int before = __shfl_up_sync(0xffffffffu, reach, 1);
    if ((tid & 31) == 31) sh.warp_sums[tid >> 5] = reach;
    __syncthreads();
    if ((tid & 31) == 0) before = tid == 0 ? sh.top : sh.warp_sums[(tid >> 5) - 1];
    __syncthreads();
    b0 = min(max(b0, before), p.B);
    b1 = max(min(b1, p.B), b0);
    const int tiles = g < p.G && n > 0 ? ceil_div((b1 - b0) * TH, M_TILE) : 0;
    const int incl = block_scan<kSchedThreads>(tiles, sh.warp_sums, Add());
    if (g < p.G) groups[g] = make_int4(b0, b1, sh.carry + incl - tiles, n);
    __syncthreads();
    if (tid == kSchedThreads - 1) {
      sh.carry += incl;
      sh.top = reach;
    }
    __syncthreads();
  }
  const int n_prefix = sh.carry, n_items = n_prefix + (apart ? 0 : p.B * p.n_mt);
  if (tid == 0) {
    *p.n_prefix = n_prefix;
    if (p.md_o) *p.apart = apart;
  }
  __syncthreads();
  for (int b = tid; b < p.B; b += kSchedThreads) {
    const int4 g = groups[last_le(p.G, b, [&](int i) { return i == 0 ? 0 : groups[i].x; })];
    p.seq[b] = g.w > 0 && b >= g.x && b < g.y ? make_int2(g.z, (b - g.x) * TH) : make_int2(-1, 0);
  }
  const Kinds kinds{n_prefix, head_of(p, min(M_TILE, p.B * TH)), head_of(p, min(M_TILE, TH))};
  schedule<kSchedThreads>(sh, n_items, p.parts, 0, p.md, p.pieces, kinds,
           [&](int i) {
             SharedItem it;
             if (i < n_prefix) {
               const int g = last_le(p.G, i, [&](int k) { return groups[k].z; });
               const int4 at = groups[g];
               const int row = (i - at.z) * M_TILE;
               it = SharedItem{at.x * TH + row, min(M_TILE, (at.y - at.x) * TH - row), at.w, ceil_div(at.w, PAGE), g, 0, 0, 0};
             } else {
               const int k = i - n_prefix, mt = p.n_mt == 1 ? 0 : k / p.B, b = k - mt * p.B;
               const int n = length(near_by ? sh.lens[b] : p.seqlens[b], p.max_pages);
               it = SharedItem{b * TH + mt * M_TILE, min(M_TILE, TH - mt * M_TILE), n, ceil_div(own_keys(p, n, mt), PAGE), b,
                               1, mt * M_TILE, 0};
             }
             p.items[i] = it;
             return Cost{head_of(p, it.rows), it.tiles};
           },
           [&](int i, int at, int) { p.items[i].slot = at; });
}

// Bytes of a page as bf16 rows.
__host__ __device__ constexpr size_t wide_page_bytes(int format) {
  return (size_t)PAGE * 2 * (format == MLA_KV_FP8_E4M3 ? D_QK + D_V : D_QK);
}

constexpr int kWidenParts = 2;

// The last i in [0, n) with first[i] <= x (first[0] <= x, nondecreasing), found by a whole warp,
// 256 entries at once.
__device__ __forceinline__ int warp_last_le(const int32_t *first, int n, int x) {
  const int lane = threadIdx.x & 31;
  int lo = 0;
  while (n > 1) {
    const int step = ceil_div(n, 256);
    int count = 0;
#pragma unroll
    for (int k = 0; k < 8; k++) {
      const int i = (32 * k + lane) * step;
      count += __popc(__ballot_sync(0xffffffffu, i < n && first[lo + i] <= x));
    }
    lo += (count - 1) * step;
    n = min(step, n - (count - 1) * step);
  }
  return lo;
}

// FP8: the pages in use as bf16 rows (zeros behind the last token), once for all the
// tiles that read them: prefixes first, then own pages where there is room for them.  A block takes
// one of kWidenParts parts of a page's rows at a time (FP8 groups of 48 sequences, 477 pages on 152 SMs:
// 170.4 us with halves, 174.5 with whole pages, 172.1 with quarters).  A warp a row: lane l widens 16 of its
// values, and lanes 0-3 or 0-7 the rotated part.  With one scale the codes as they are; with a
// scale for each 128 values as sums of two values, the second ones behind the row's first.
template <bool kScaled>
__global__ void __launch_bounds__(256) shared_widen_kernel(SharedParams p) {
  grid_dep_trigger();
  grid_dep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const long long units = (long long)p.first[p.G + p.B] * kWidenParts;
  constexpr int kRowBytes = kScaled ? FP8_ROW : D_QK, kRows = PAGE / 8 / kWidenParts;
  constexpr int kPieces = (kScaled ? D_QK + D_V : D_QK) / 8;  // 16-byte pieces of a widened row
  const uint4 zero = make_uint4(0, 0, 0, 0);
  for (long long u = blockIdx.x; u < units; u += gridDim.x) {
    const int at_page = (int)(u / kWidenParts), y = warp_last_le(p.first, p.G + p.B, at_page), j = at_page - p.first[y];
    const bool own = y >= p.G;
    const int row = own ? y - p.G : y, width = own ? p.max_pages : p.max_prefix;
    const int page = (own ? p.block_table : p.prefix_table)[(size_t)row * width + j];
    if (page < 0 || page >= p.num_pages) continue;
    const int tokens = (int)min((long long)PAGE, (long long)(own ? p.seqlens : p.prefix_lens)[row] - (long long)j * PAGE);
    uint4 *to = reinterpret_cast<uint4 *>(p.scratch + (size_t)at_page * wide_page_bytes(p.format));
#pragma unroll
    for (int i = 0; i < kRows; i++) {
      const int r = (int)(u % kWidenParts) * (PAGE / kWidenParts) + warp + 8 * i;
      const size_t at = (size_t)page * PAGE + r;
      const uint4 *src = reinterpret_cast<const uint4 *>(p.cache + at * kRowBytes);
      uint4 *dst = to + r * kPieces;
      const bool live = r < tokens;
      const uint4 codes = live ? __ldg(src + lane) : zero;
      if constexpr (kScaled) {
        uint4 v[2] = {zero, zero}, rest[2] = {zero, zero};
        if (live) widen16_twice(codes, __ldg(p.kv_scales + at * 4 + lane / 8), v, rest);
#pragma unroll
        for (int e = 0; e < 2; e++) {
          dst[2 * lane + e] = v[e];
          dst[D_QK / 8 + 2 * lane + e] = rest[e];
        }
        if (lane < 8) dst[64 + lane] = live ? __ldg(src + 32 + lane) : zero;
      } else {
        uint4 lo, hi;
        codes16(codes, lo, hi);
        dst[2 * lane] = lo;
        dst[2 * lane + 1] = hi;
        if (lane < 4) {
          codes16(live ? __ldg(src + 32 + lane) : zero, lo, hi);
          dst[64 + 2 * lane] = lo;
          dst[65 + 2 * lane] = hi;
        }
      }
    }
  }
}

// ---- join ------------------------------------------------------------------------

constexpr int kJoinWarps = 8;

__device__ __forceinline__ void ld_cg_v8(float (&v)[8], const float *ptr) {
  uint32_t u[8];
  asm volatile("ld.global.cg.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7])
               : "l"(ptr));
#pragma unroll
  for (int j = 0; j < 8; j++) v[j] = __uint_as_float(u[j]);
}

// Lane: a query row; warp: kChunks * 8 of its columns; block: 32 rows and the columns
// of its eight warps.  Rows side by side lie side by side in the partials, so a warp
// reads 1 KB at once.  The first part of each side is asked for with the first
// log-sum-exps, before its weight is known.
template <int kChunks>
__global__ void __launch_bounds__(kJoinWarps * 32) shared_join_kernel(SharedParams p) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, TH = p.T * p.H;
  const int R = blockIdx.x * 32 + lane, chunk = (blockIdx.y * kJoinWarps + warp) * kChunks;
  const bool live = R < p.B * TH, apart = p.md_o && *p.apart;
  const int b = live ? R / TH : 0, r = live ? R % TH : 0;
  const float *lse[2] = {p.lse_p, p.lse_p}, *o[2] = {p.o_p, p.o_p};
  int n[2] = {0, 0};
  // (the schedule was complete before the kernel before this one began its work)
  if (live) {
    const int2 s = p.seq[b];
    if (s.x >= 0) {
      const int row = s.y + r, i = s.x + row / M_TILE, slot = p.items[i].slot, at = row % M_TILE;
      n[0] = p.pieces[i];
      lse[0] += (size_t)slot * M_TILE + at;
      o[0] += (((size_t)slot * 64 + chunk) * M_TILE + at) * 8;
    }
    const int k = (r / M_TILE) * p.B + b, at = r % M_TILE;
    const int i = apart ? k : *p.n_prefix + k, slot = apart ? p.ns_o[i] : p.items[i].slot;
    n[1] = apart ? p.cnt_o[i] : p.pieces[i];
    lse[1] = (apart ? p.lse_o : p.lse_p) + (size_t)slot * M_TILE + at;
    o[1] = (apart ? p.o_o : p.o_p) + (((size_t)slot * 64 + chunk) * M_TILE + at) * 8;
  }
  grid_dep_wait();
  if (!live) return;
  constexpr size_t kNext = (size_t)64 * M_TILE * 8, kChunk = (size_t)M_TILE * 8;
  float v[2][kChunks][8], first[2];
#pragma unroll
  for (int k = 0; k < 2; k++) {
    first[k] = -INFINITY;
    if (n[k] > 0) {
      first[k] = __ldcg(lse[k]);
#pragma unroll
      for (int c = 0; c < kChunks; c++) ld_cg_v8(v[k][c], o[k] + c * kChunk);
    }
  }
  float m = fmaxf(first[0], first[1]);
#pragma unroll
  for (int k = 0; k < 2; k++)
#pragma unroll 4
    for (int j = 1; j < n[k]; j++) m = fmaxf(m, __ldcg(lse[k] + (size_t)j * M_TILE));
  float acc[kChunks][8], sum = 0.f;
#pragma unroll
  for (int c = 0; c < kChunks; c++)
#pragma unroll
    for (int e = 0; e < 8; e++) acc[c][e] = 0.f;
  auto add = [&](float l, const float(&part)[kChunks][8]) {
    if (l == -INFINITY) return;
    const float w = exp2f(l - m);
    sum += w;
#pragma unroll
    for (int c = 0; c < kChunks; c++)
#pragma unroll
      for (int e = 0; e < 8; e++) acc[c][e] = fmaf(w, part[c][e], acc[c][e]);
  };
#pragma unroll
  for (int k = 0; k < 2; k++) {
    add(first[k], v[k]);
    constexpr int kDeep = kChunks == 1 ? 4 : 1;  // parts on their way together
    for (int j0 = 1; j0 < n[k]; j0 += kDeep) {
      float w[kDeep][kChunks][8], l[kDeep];
#pragma unroll
      for (int j = 0; j < kDeep; j++) {
        l[j] = -INFINITY;
        if (j0 + j < n[k]) {
          l[j] = __ldcg(lse[k] + (size_t)(j0 + j) * M_TILE);
#pragma unroll
          for (int c = 0; c < kChunks; c++) ld_cg_v8(w[j][c], o[k] + (j0 + j) * kNext + c * kChunk);
        }
      }
#pragma unroll
      for (int j = 0; j < kDeep; j++) add(l[j], w[j]);
    }
  }
  // nan in any part is nan here (m leaves it out, the sum does not)
  const bool low = m == kAllLow && sum == sum;
  const float inv = low ? __uint_as_float(0x7FC00000u) : sum != 0.f ? 1.f / sum : 0.f;
#pragma unroll
  for (int c = 0; c < kChunks; c++) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; e++) {
      const __nv_bfloat162 x = __floats2bfloat162_rn(acc[c][2 * e] * inv, acc[c][2 * e + 1] * inv);
      w[e] = *reinterpret_cast<const uint32_t *>(&x);
    }
    reinterpret_cast<uint4 *>(p.out + (size_t)R * D_V)[chunk + c] = make_uint4(w[0], w[1], w[2], w[3]);
  }
  if (chunk == 0)
    p.lse[((size_t)b * p.H + r % p.H) * p.T + r / p.H] = sum != 0.f && !low ? (m + log2f(sum)) * LN2 : -INFINITY;
}

// ---- host ------------------------------------------------------------------------

struct Layout {
  size_t items, md, pieces, n_prefix, groups, lens_o, seq, md_o, ns_o, cnt_o, apart, first, scratch, lse_p, o_p, lse_o, o_o, ring, total;
  size_t pages;
  int room, own_room, n_mt;
  bool maybe_apart;  // own FP8 tokens go through the decode kernel where their pages in use exceed own_room
};

// Room for widened own FP8 pages where the caller gives no bound (151 MB of workspace, 285 MB with
// scales).  Own tokens of more pages go through the decode kernel's gather, which needs no room but
// rounds rows to bf16 and takes longer: 48 sequences of up to 300 tokens, four query tokens, 64 heads
// 135 us that way and 105 this way with one scale, 175 and 147 with a scale for each 128 values; 16 of up to
// 8000 tokens, one query token, 128 heads 142 and 81, 152 and 121.  (Where a table is wider than the room, the decode
// kernel is launched with nothing to do, which takes 6 to 8 us.)
constexpr long long kMostOwnPages = 2048;

// Room for B * max_pages = `entries` own pages at most.  Without a bound (-1) rows with a scale for each 128
// values have room for a whole table or none: their results with a wide table are those of rounded rows.
int own_room_of(int format, long long entries, int bound) {
  if (format == MLA_KV_BF16) return 0;
  if (bound >= 0) return (int)(bound < entries ? bound : entries);
  if (entries <= kMostOwnPages) return (int)entries;
  return format == MLA_KV_FP8_E4M3_TENSOR ? (int)kMostOwnPages : 0;
}

Layout layout(int B, int T, int H, int G, int format, int max_prefix, int max_pages, int bound, int parts) {
  const bool wide = format != MLA_KV_BF16;
  const long long entries = (long long)B * max_pages;
  Layout l;
  l.n_mt = ceil_div(T * H, M_TILE);
  l.own_room = own_room_of(format, entries, bound);
  const bool apart = l.maybe_apart = wide && l.own_room < entries;
  const size_t own = (size_t)B * l.n_mt, prefix = ((size_t)B * T * H + M_TILE - 1) / M_TILE + G;
  l.room = (int)(prefix + own);
  l.pages = wide ? (size_t)G * max_prefix + l.own_room : 0;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at = (at + bytes + 255) / 256 * 256;
    return here;
  };
  // slots of results: one for each item, and one for each cut.  Those of the decode kernel lie behind the
  // prefixes', where the own tokens' are otherwise.
  const size_t slots_p = prefix + parts, slots = slots_p + (apart ? 2 * own + parts : own), row = M_TILE * sizeof(float);
  l.items = take((size_t)l.room * sizeof(SharedItem));
  l.md = take((size_t)parts * MD_STRIDE * 4);
  l.pieces = take((size_t)l.room * 4);
  l.n_prefix = take(4);
  l.groups = take((size_t)G * sizeof(int4));
  l.seq = take((size_t)B * sizeof(int2));
  l.lens_o = take(apart ? (size_t)B * 4 : 0);
  l.md_o = take(apart ? (size_t)parts * MD_STRIDE * 4 : 0);
  l.ns_o = take(apart ? (own + 1) * 4 : 0);
  l.cnt_o = take(apart ? own * 4 : 0);
  l.apart = take(apart ? 4 : 0);
  l.first = take(wide ? ((size_t)G + B + 1) * 4 : 0);
  l.scratch = take(l.pages * wide_page_bytes(format));
  l.lse_p = take(slots * row);
  l.o_p = take(slots * row * D_V);
  l.lse_o = l.lse_p + slots_p * row;
  l.o_o = l.o_p + slots_p * row * D_V;
  l.ring = take((size_t)parts * P_RING * P_SLOT_BYTES);
  l.total = at;
  return l;
}

int fail(int code, const char *msg) {
  set_last_error(msg);
  return code;
}

int check_sizes(int B, int T, int H, int G, int format, int max_prefix, int max_pages, int bound) {
  char msg[160];
  if (B < 1 || G < 1 || max_prefix < 1 || max_pages < 1) {
    snprintf(msg, sizeof msg, "B = %d, G = %d, max_prefix_pages = %d and max_pages = %d must be >= 1", B, G, max_prefix, max_pages);
    return fail(MLA_ERR_INVALID_ARG, msg);
  }
  if (H < 1 || H > MLA_MAX_HEADS || T < 1 || T > MLA_MAX_QUERY_TOKENS) {
    snprintf(msg, sizeof msg, "H = %d not in [1, %d] or T = %d not in [1, %d]", H, MLA_MAX_HEADS, T, MLA_MAX_QUERY_TOKENS);
    return fail(MLA_ERR_INVALID_ARG, msg);
  }
  if (format != MLA_KV_BF16 && format != MLA_KV_FP8_E4M3 && format != MLA_KV_FP8_E4M3_TENSOR)
    return fail(MLA_ERR_INVALID_ARG, "kv_format unknown");
  if (bound < -1) return fail(MLA_ERR_INVALID_ARG, "own_pages must be >= 0, or -1 for no bound");
  const long long items = (long long)B * ceil_div(T * H, M_TILE) + ((long long)B * T * H + M_TILE - 1) / M_TILE + G;
  if (items > kMaxItems) {
    snprintf(msg, sizeof msg, "%lld work items exceed the limit %d", items, kMaxItems);
    return fail(MLA_ERR_UNSUPPORTED, msg);
  }
  // (the schedule counts tiles in 32 bits, and so are widened pages, of which there are no more)
  const long long tiles = (long long)B * ceil_div(T * H, M_TILE) * max_pages + (((long long)B * T * H + M_TILE - 1) / M_TILE + G) * max_prefix;
  if (tiles > 0x3fffffffLL) return fail(MLA_ERR_UNSUPPORTED, "more than 2^30 tiles of 64 keys in max_pages and max_prefix_pages");
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

extern "C" size_t mla_decode_shared_workspace_bytes(int B, int T, int H, int G, int kv_format, int max_prefix_pages,
                                                    int max_pages) {
  return mla_decode_shared_bounded_workspace_bytes(B, T, H, G, kv_format, max_prefix_pages, max_pages, -1);
}

extern "C" int mla_decode_shared(const void *q, const void *kv_cache, int kv_format, int num_pages, int page_size,
                                 const int32_t *prefix_table, int max_prefix_pages, const int32_t *prefix_lens,
                                 const int32_t *group_offsets, int G, const int32_t *block_table, int max_pages,
                                 const int32_t *cache_seqlens, const float *kv_scales, float softmax_scale, int causal,
                                 void *workspace, size_t workspace_bytes, void *out, float *lse, int B, int T, int H,
                                 mla_stream_t stream) {
  return mla_decode_shared_bounded(q, kv_cache, kv_format, num_pages, page_size, prefix_table, max_prefix_pages, prefix_lens,
                                   group_offsets, G, block_table, max_pages, cache_seqlens, -1, kv_scales, softmax_scale,
                                   causal, workspace, workspace_bytes, out, lse, B, T, H, stream);
}

extern "C" size_t mla_decode_shared_bounded_workspace_bytes(int B, int T, int H, int G, int kv_format, int max_prefix_pages,
                                                            int max_pages, int own_pages) {
  int parts = 0;
  if (check_sizes(B, T, H, G, kv_format, max_prefix_pages, max_pages, own_pages) != MLA_OK || device_parts(&parts) != MLA_OK)
    return 0;
  return layout(B, T, H, G, kv_format, max_prefix_pages, max_pages, own_pages, parts).total;
}

extern "C" int mla_decode_shared_bounded(const void *q, const void *kv_cache, int kv_format, int num_pages, int page_size,
                                         const int32_t *prefix_table, int max_prefix_pages, const int32_t *prefix_lens,
                                         const int32_t *group_offsets, int G, const int32_t *block_table, int max_pages,
                                         const int32_t *cache_seqlens, int own_pages, const float *kv_scales,
                                         float softmax_scale, int causal, void *workspace, size_t workspace_bytes, void *out,
                                         float *lse, int B, int T, int H, mla_stream_t stream) {
  int rc = check_sizes(B, T, H, G, kv_format, max_prefix_pages, max_pages, own_pages);
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
  if (num_pages < 1) return fail(MLA_ERR_INVALID_ARG, "num_pages must be >= 1");
  if (causal != 0 && causal != 1) return fail(MLA_ERR_INVALID_ARG, "causal must be 0 or 1");
  if (!(softmax_scale > 0.f) || !std::isfinite(softmax_scale))
    return fail(MLA_ERR_INVALID_ARG, "softmax_scale must be finite and > 0");
  int parts = 0;
  if ((rc = device_parts(&parts)) != MLA_OK) return rc;
  if (parts > kMostParts) return fail(MLA_ERR_UNSUPPORTED, "more SMs than the schedule has room for");
  const Layout l = layout(B, T, H, G, kv_format, max_prefix_pages, max_pages, own_pages, parts);
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
  p.own_room = l.own_room;
  p.n_mt = l.n_mt;
  p.parts = parts;
  p.scale_log2 = softmax_scale * LOG2E;
  p.wait_ns = wait_limit_ns();
  p.items = reinterpret_cast<SharedItem *>(at(l.items));
  p.md = reinterpret_cast<int32_t *>(at(l.md));
  p.pieces = reinterpret_cast<int32_t *>(at(l.pieces));
  p.n_prefix = reinterpret_cast<int32_t *>(at(l.n_prefix));
  p.groups = reinterpret_cast<int4 *>(at(l.groups));
  p.lens_o = reinterpret_cast<int32_t *>(at(l.lens_o));
  p.seq = reinterpret_cast<int2 *>(at(l.seq));
  p.md_o = l.maybe_apart ? reinterpret_cast<int32_t *>(at(l.md_o)) : nullptr;
  p.ns_o = reinterpret_cast<int32_t *>(at(l.ns_o));
  p.cnt_o = reinterpret_cast<int32_t *>(at(l.cnt_o));
  p.apart = reinterpret_cast<int32_t *>(at(l.apart));
  p.first = reinterpret_cast<int32_t *>(at(l.first));
  p.scratch = at(l.scratch);
  p.lse_p = reinterpret_cast<float *>(at(l.lse_p));
  p.o_p = reinterpret_cast<float *>(at(l.o_p));
  p.lse_o = reinterpret_cast<float *>(at(l.lse_o));
  p.o_o = reinterpret_cast<float *>(at(l.o_o));
  p.ring = at(l.ring);
  p.out = static_cast<__nv_bfloat16 *>(out);
  p.lse = lse;
  p.scratch_pages = l.pages;
  const bool wide = kv_format != MLA_KV_BF16;

  cudaStream_t s = (cudaStream_t)stream;
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  // (few threads meet sooner)
  const bool small = l.room <= kFewThreads && B <= kFewThreads && G <= kFewThreads && parts < kFewThreads;
  const unsigned blocks_s = !wide ? 1 : l.maybe_apart ? 3 : 2;
  cudaError_t e = small ? launch_dependent(shared_schedule_kernel<kFewThreads>, blocks_s, kFewThreads, 0, s, p)
                        : launch_dependent(shared_schedule_kernel<1024>, blocks_s, 1024, 0, s, p);
  if (e == cudaSuccess && wide) {
    // as many blocks as the SMs hold (six each, of 40 registers a thread), or as there can be parts of pages
    const long long most = (long long)l.pages * kWidenParts, held = 2ll * parts * 6;
    cfg.gridDim = dim3((unsigned)(most < held ? most : held));
    e = cudaLaunchKernelEx(&cfg, kv_format == MLA_KV_FP8_E4M3 ? shared_widen_kernel<true> : shared_widen_kernel<false>, p);
  }
  if (e == cudaSuccess) e = launch_shared_attention(p, s);
  if (e == cudaSuccess && l.maybe_apart) {
    // own FP8 rows that there is no room for go through the decode kernel, which gathers and widens them
    DecodeParams d{};
    d.q = p.q;
    d.kv = p.cache;
    d.kv_scales = kv_scales;
    d.block_table = block_table;
    d.seqlens = p.lens_o;
    d.tile_md = p.md_o;
    d.num_splits = p.ns_o;
    d.ws_lse = p.lse_o;
    d.ws_o = p.o_o;
    d.ws_p = p.ring;
    d.out = p.out;  // (it writes the zeros of empty sequences; the join writes every row after it)
    d.lse = p.lse;
    d.status = st;
    d.kv_format = kv_format;
    d.num_pages = num_pages;
    d.max_pages = max_pages;
    d.causal = causal;
    d.B = B;
    d.T = T;
    d.H = H;
    d.n_mt = l.n_mt;
    d.n_items = B * l.n_mt;
    d.num_parts = parts;
    d.scale_log2 = p.scale_log2;
    d.wait_ns = p.wait_ns;
    d.help = T * H <= 64 ? 1 : 0;
    e = launch_decode(d, s, nullptr, nullptr);
  }
  if (e == cudaSuccess) {
    // Few rows: a warp has 8 columns, so that there are warps enough; many: 32, as finding a row's
    // parts takes longer than reading 8 columns of them.
    const unsigned blocks = (unsigned)(((long long)B * T * H + 31) / 32);
    const bool few = blocks < 128;
    cfg.gridDim = dim3(blocks, 64 / kJoinWarps / (few ? 1 : 4));
    e = cudaLaunchKernelEx(&cfg, few ? shared_join_kernel<1> : shared_join_kernel<4>, p);
  }
  if (e != cudaSuccess) {
    char msg[128];
    snprintf(msg, sizeof msg, "decode over shared prefixes: %s", cudaGetErrorString(e));
    return fail(MLA_ERR_CUDA, msg);
  }
  set_last_error("");
  return MLA_OK;
}

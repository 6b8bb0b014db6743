// Value projection: what follows the decode.  The decode's output row of a
// head is a mix of latent rows (512 values); the head's W_UV takes it to the
// 128 values the output projection reads:
//   o[n][h][v] = bf16(sum_{l<512} attn[n][h][l] * W_UV[h][v][l])     v < 128
// with fp32 accumulation in tensor memory, rounded to bf16 once.
//
// Bytes bound it: 2 * 128 * 512 flops per 1280 bytes of a row are about 100
// flops a byte, a third of what the tensor cores can take (4095 tokens, 64 heads:
// 60 us, 5.7 TB/s, where outputs cannot stay in L2; 64 tokens, 128 heads: 4.6 us
// with the weights in L2, 7.4 us without).
#include "common.cuh"
#include "dependent.cuh"
#include "ptx.cuh"
#include "ptx_pair.cuh"
#include "tma_map.cuh"

namespace mla {
namespace {

using namespace ptx;

// D[v][n] is computed with the 128 weight rows as the MMA's M and up to 64
// tokens as its N, so that a decode batch of any size fills M.  A persistent
// CTA takes an equal share of the (head, token tile) items, heads outermost:
// W_UV[h] (128 KB) stays in shared memory for all its tiles of a head while
// the tokens' rows stream through a ring.  D is double buffered in tensor
// memory; four warps drain it through shared memory, from where TMA stores
// whole lines (and clips the tokens behind the last).
//
// Warps 0-3 drain D, warp 4 loads, warp 5 issues the MMAs.
constexpr int kThreads = 192;
constexpr int kDv = 128;
constexpr int kKBlocks = D_V / 64;            // 8 blocks of 64 latent values
constexpr uint32_t kWBytes = 128 * 128;       // one block of 128 weight rows
constexpr int kMaxTile = 64;
constexpr uint32_t kUnit = 2 * kMaxTile * 128;  // 128 latent values of a tile's tokens, as two boxes of 64
constexpr int kUnits = 5;
constexpr uint32_t OFF_RING = kKBlocks * kWBytes;
constexpr uint32_t OFF_OUT = OFF_RING + kUnits * kUnit;
constexpr uint32_t OFF_BARS = OFF_OUT + kMaxTile * kDv * 2;

struct Bars {
  uint64_t w_full[kKBlocks / 2], w_empty;
  uint64_t full[kUnits], empty[kUnits];
  uint64_t d_full[2], d_empty[2];
  uint32_t tmem_base;
  int abort;
};
constexpr uint32_t kSmem = OFF_BARS + sizeof(Bars) + 1024;
static_assert(kSmem <= 232448, "shared memory budget");

template <bool kPoll>
__device__ __forceinline__ bool wait_ok(Bars *b, uint64_t *bar, uint32_t parity, unsigned int *status,
                                        unsigned long long wait_ns) {
  if (mbar_wait_limited<false, kPoll>(smem_u32(bar), parity, &b->abort, wait_ns)) return true;
  atomicOr(status, MLA_STATUS_WAIT_TIMEOUT);
  *(volatile int *)&b->abort = 1;
  return false;
}

template <bool kPoll>
__global__ void __launch_bounds__(kThreads, 1)
    value_kernel(const __grid_constant__ CUtensorMap w_map, const __grid_constant__ CUtensorMap x_map,
                 const __grid_constant__ CUtensorMap o_map, int tiles, int items, int ntile, unsigned int *status,
                 unsigned long long wait_ns) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *base = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  Bars *br = reinterpret_cast<Bars *>(base + OFF_BARS);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int i0 = (int)((long long)items * blockIdx.x / gridDim.x);
  const int i1 = (int)((long long)items * (blockIdx.x + 1) / gridDim.x);
  if (warp == 0) {
    tmem_alloc(smem_u32(&br->tmem_base), 128);
    tmem_relinquish();
  }
  if (threadIdx.x == 32) {
    for (int k = 0; k < kKBlocks / 2; k++) mbar_init(smem_u32(&br->w_full[k]), 1);
    mbar_init(smem_u32(&br->w_empty), 1);
    for (int s = 0; s < kUnits; s++) {
      mbar_init(smem_u32(&br->full[s]), 1);
      mbar_init(smem_u32(&br->empty[s]), 1);
    }
    for (int s = 0; s < 2; s++) {
      mbar_init(smem_u32(&br->d_full[s]), 1);
      mbar_init(smem_u32(&br->d_empty[s]), 4);
    }
    br->abort = 0;
    fence_mbar_init_cluster();
  }
  if (threadIdx.x == 4 * 32) {
    prefetch_tensormap(&w_map);
    prefetch_tensormap(&x_map);
    prefetch_tensormap(&o_map);
  }
  grid_dep_trigger();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  grid_dep_wait();  // nothing of the caller's is read or written before the kernel in front has ended
  const uint32_t tmem = br->tmem_base, smem = smem_u32(base);
  const uint32_t box = (uint32_t)ntile * 128;

  if (warp == 4) {
    // the whole warp waits, one elected lane asks
    const uint64_t pol_w = policy_evict_normal(), pol_x = policy_evict_first();
    uint32_t u = 0, heads = 0;
    bool ok = true;
    for (int i = i0; i < i1 && ok; i++) {
      const int h = i / tiles, n0 = i % tiles * ntile;
      const bool new_head = i == i0 || n0 == 0;
      if (new_head) ok = __all_sync(0xffffffffu, wait_ok<kPoll>(br, &br->w_empty, (heads++ & 1) ^ 1, status, wait_ns));
      for (int k = 0; k < kKBlocks / 2 && ok; k++, u++) {
        const uint32_t s = u % kUnits, dst = smem + OFF_RING + s * kUnit;
        if (new_head && elect_one()) {
          mbar_arrive_expect_tx(smem_u32(&br->w_full[k]), 2 * kWBytes);
          tma_load_3d(smem + 2 * k * kWBytes, &w_map, smem_u32(&br->w_full[k]), 128 * k, 0, h, pol_w);
          tma_load_3d(smem + (2 * k + 1) * kWBytes, &w_map, smem_u32(&br->w_full[k]), 128 * k + 64, 0, h, pol_w);
        }
        __syncwarp();
        ok = __all_sync(0xffffffffu, wait_ok<kPoll>(br, &br->empty[s], ((u / kUnits) & 1) ^ 1, status, wait_ns));
        if (!ok) break;
        if (elect_one()) {
          mbar_arrive_expect_tx(smem_u32(&br->full[s]), 2 * box);
          tma_load_3d(dst, &x_map, smem_u32(&br->full[s]), 128 * k, h, n0, pol_x);
          tma_load_3d(dst + box, &x_map, smem_u32(&br->full[s]), 128 * k + 64, h, n0, pol_x);
        }
        __syncwarp();
      }
    }
  } else if (warp == 5) {
    // the whole warp waits, one elected lane issues
    const uint32_t idesc = idesc_bf16_f32(128, ntile, false, false);
    uint32_t u = 0, heads = 0;
    bool ok = true;
    auto wait = [&](uint64_t *bar, uint32_t parity) {
      ok = ok && __all_sync(0xffffffffu, wait_ok<kPoll>(br, bar, parity, status, wait_ns));
    };
    for (int i = i0; i < i1 && ok; i++) {
      const int j = i - i0, buf = j & 1;
      const bool new_head = i == i0 || i % tiles == 0;
      heads += new_head ? 1 : 0;
      wait(&br->d_empty[buf], ((j >> 1) & 1) ^ 1);
      for (int k = 0; k < kKBlocks / 2; k++, u++) {
        const uint32_t s = u % kUnits;
        if (new_head) wait(&br->w_full[k], (heads - 1) & 1);
        wait(&br->full[s], (u / kUnits) & 1);
        if (!ok) break;
        tc_fence_after();
        if (elect_one()) {
#pragma unroll
          for (int kk = 0; kk < 8; kk++)
            mma_ss(tmem + buf * 64, smem_desc_sw128(smem + (2 * k + (kk >> 2)) * kWBytes + (kk & 3) * 32, 16, 1024),
                   smem_desc_sw128(smem + OFF_RING + s * kUnit + (kk >> 2) * box + (kk & 3) * 32, 16, 1024), idesc,
                   (k | kk) ? 1u : 0u);
          mma_commit(smem_u32(&br->empty[s]));
          if (k == kKBlocks / 2 - 1) {
            mma_commit(smem_u32(&br->d_full[buf]));
            if (i + 1 == i1 || (i + 1) % tiles == 0) mma_commit(smem_u32(&br->w_empty));
          }
        }
        __syncwarp();
      }
    }
  } else {
    uint8_t *out = base + OFF_OUT;
    const int r = warp * 32 + lane;
    for (int i = i0; i < i1; i++) {
      const int j = i - i0, buf = j & 1;
      // a wait that gives up lets all four warps go on to the barriers below, which they pass together
      const bool ok = __all_sync(0xffffffffu, wait_ok<kPoll>(br, &br->d_full[buf], (j >> 1) & 1, status, wait_ns));
      tc_fence_after();
      if (threadIdx.x == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");  // the tile before is out
      __syncwarp();  // (the barriers are the whole warp's)
      named_bar_sync(1, 128);
      if (ok) {
        // D (lane = value row, column = token) -> bf16 [token][128]
        for (int c = 0; c < ntile; c += 32) {
          uint32_t v[32];
          tmem_ld32(tmem + ((uint32_t)(warp * 32) << 16) + buf * 64 + c, v);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; e++)
            if (c + e < ntile)
              *reinterpret_cast<__nv_bfloat16 *>(out + (c + e) * 256 + r * 2) =
                  __float2bfloat16_rn(__uint_as_float(v[e]));
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&br->d_empty[buf]));
      __syncwarp();
      fence_proxy_async_smem();
      // all four warps stop together, at the barrier (abort alone may be set
      // by another role between their looks at it); nothing of this tile is stored then
      if (bar_red_or(1, 128, !ok || *(volatile int *)&br->abort)) break;
      if (threadIdx.x == 0) {
        asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                         reinterpret_cast<uint64_t>(&o_map)),
                     "r"(smem + OFF_OUT), "r"(0), "r"(i / tiles), "r"(i % tiles * ntile)
                     : "memory");
        asm volatile("cp.async.bulk.commit_group;" ::: "memory");
      }
    }
    if (threadIdx.x == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
  }
  __syncthreads();
  if (*(volatile int *)&br->abort) {  // a wait gave up: let copies or MMAs still in flight land before the CTA exits
    const uint64_t t0 = globaltimer();
    while (globaltimer() - t0 < 2000000ull) {
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 128);
  }
}

int fail(int code, const char *msg) {
  set_last_error(msg);
  return code;
}

}  // namespace
}  // namespace mla

int mla_value_project(const void *attn, int64_t ld_token, int64_t ld_head, const void *w_uv, int64_t w_row,
                      int64_t w_head, int N, int H, void *out, mla_stream_t stream) {
  using namespace mla;
  if (N < 0) return fail(MLA_ERR_INVALID_ARG, "N must be >= 0");
  if (H < 1 || H > MLA_MAX_HEADS) return fail(MLA_ERR_INVALID_ARG, "H must be in [1, 128]");
  if (ld_token % 8 || ld_head % 8 || w_row % 8 || w_head % 8)
    return fail(MLA_ERR_INVALID_ARG, "strides must be multiples of 8 elements");
  if ((N > 1 && ld_token < D_V) || (H > 1 && ld_head < D_V) || w_row < D_V || (H > 1 && w_head < D_V))
    return fail(MLA_ERR_INVALID_ARG, "strides of attn and w_uv rows must be at least 512 elements");
  if (N == 0) {
    set_last_error("");
    return MLA_OK;
  }
  if (!attn || !w_uv || !out) return fail(MLA_ERR_INVALID_ARG, "null pointer");
  auto a16 = [](const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; };
  if (!a16(attn) || !a16(w_uv) || !a16(out))
    return fail(MLA_ERR_INVALID_ARG, "attn, w_uv and out must be 16-byte aligned");
  const int ntile = N >= kMaxTile ? kMaxTile : (N + 15) / 16 * 16;
  CUtensorMap w_map, x_map, o_map;
  if (!make_map_3d(&w_map, w_uv, D_V, kDv, H, w_row, w_head, 128, 1) ||
      !make_map_3d(&x_map, attn, D_V, H, N, ld_head, ld_token, 1, ntile) ||
      !make_map_3d(&o_map, out, kDv, H, N, kDv, (int64_t)H * kDv, 1, ntile, kDv, false))
    return fail(MLA_ERR_CUDA, "cuTensorMapEncodeTiled failed");
  const int tiles = (N + ntile - 1) / ntile;
  if ((long long)tiles * H > 0x7FFFFFFFll) return fail(MLA_ERR_UNSUPPORTED, "too many tokens");
  unsigned int *st = nullptr;
  if (status_word(&st) != MLA_OK) return MLA_ERR_CUDA;
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  const unsigned long long limit = wait_limit_ns();
  auto *kernel = limit < ptx::kShortWaitNs ? &value_kernel<true> : &value_kernel<false>;
  if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
  if (e != cudaSuccess) return fail(MLA_ERR_CUDA, cudaGetErrorString(e));
  const int items = tiles * H;
  e = launch_dependent(kernel, items < sms ? items : sms, kThreads, kSmem, (cudaStream_t)stream, w_map, x_map,
                       o_map, tiles, items, ntile, st, limit);
  if (e != cudaSuccess) return fail(MLA_ERR_CUDA, cudaGetErrorString(e));
  set_last_error("");
  return MLA_OK;
}

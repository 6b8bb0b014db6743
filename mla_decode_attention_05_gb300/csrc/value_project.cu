// Value projection: what follows the decode.  The decode's output row of a
// head is a mix of latent rows (512 values); the head's W_UV takes it to the
// 128 values the output projection reads:
//   o[n][h][v] = bf16(sum_{l<512} attn[n][h][l] * W_UV[h][v][l])     v < 128
// with fp32 accumulation in tensor memory, rounded to bf16 once.
//
// Bytes bound it: 2 * 128 * 512 flops per 1280 bytes of a row are about 100
// flops a byte, a third of what the tensor cores can take.
#include "common.cuh"
#include "ptx.cuh"
#include "tma_map.cuh"

namespace mla {
namespace {

using namespace ptx;

// One CTA per (block of up to 64 tokens, head).  D[v][n] is computed with the
// 128 weight rows as the MMA's M and the tokens as its N, so that a decode
// batch of any size fills M.
constexpr int kThreads = 128;
constexpr int kDv = 128;
constexpr int kKBlocks = D_V / 64;            // 8 blocks of 64 latent values
constexpr uint32_t kWBytes = 128 * 128;       // one block of 128 weight rows
constexpr int kMaxTile = 64;
constexpr uint32_t kSmem = kKBlocks * (kWBytes + kMaxTile * 128) + 256 + 1024;

__global__ void __launch_bounds__(kThreads, 1)
    value_kernel(const __grid_constant__ CUtensorMap w_map, const __grid_constant__ CUtensorMap x_map,
                 __nv_bfloat16 *out, int N, int H, int ntile, unsigned int *status) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t *base = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  uint64_t *full = reinterpret_cast<uint64_t *>(base + kKBlocks * (kWBytes + kMaxTile * 128));
  uint64_t *done = full + kKBlocks;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(done + 1);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int h = blockIdx.y, n0 = blockIdx.x * ntile;
  int abort_flag = 0;  // the waits below give up only on their time limit
  if (warp == 0) {
    tmem_alloc(smem_u32(tmem_slot), 64);
    tmem_relinquish();
  }
  if (threadIdx.x == 32) {
    for (int k = 0; k < kKBlocks; k++) mbar_init(smem_u32(&full[k]), 1);
    mbar_init(smem_u32(done), 1);
    fence_mbar_init_cluster();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t sw = smem_u32(base), sx = sw + kKBlocks * kWBytes;
  if (threadIdx.x == 0) {
    const uint64_t pol_w = policy_evict_normal(), pol_x = policy_evict_first();
    for (int k = 0; k < kKBlocks; k++) {
      mbar_arrive_expect_tx(smem_u32(&full[k]), kWBytes + ntile * 128);
      tma_load_3d(sw + k * kWBytes, &w_map, smem_u32(&full[k]), 64 * k, 0, h, pol_w);
      tma_load_3d(sx + k * (uint32_t)ntile * 128, &x_map, smem_u32(&full[k]), 64 * k, h, n0, pol_x);
    }
    const uint32_t idesc = idesc_bf16_f32(128, ntile, false, false);
    bool ok = true;
    for (int k = 0; k < kKBlocks && ok; k++) {
      ok = mbar_wait<false>(smem_u32(&full[k]), 0, &abort_flag, kDefaultWaitNs);
      if (!ok) break;
      tc_fence_after();
#pragma unroll
      for (int kk = 0; kk < 4; kk++)
        mma_ss(tmem, smem_desc_sw128(sw + k * kWBytes + kk * 32, 16, 1024),
               smem_desc_sw128(sx + k * (uint32_t)ntile * 128 + kk * 32, 16, 1024), idesc, (k | kk) ? 1u : 0u);
    }
    if (ok) {
      mma_commit(smem_u32(done));
    } else {
      atomicOr(status, MLA_STATUS_WAIT_TIMEOUT);
    }
  }
  const bool ok = __syncthreads_and(mbar_wait<false>(smem_u32(done), 0, &abort_flag, kDefaultWaitNs));
  if (ok) {
    tc_fence_after();
    // D (lane = value row, column = token) -> bf16 [token][128] in the
    // weights' place, which every MMA has finished reading
    const int r = warp * 32 + lane;
    for (int c = 0; c < ntile; c += 32) {
      uint32_t v[32];
      tmem_ld32(tmem + ((uint32_t)(warp * 32) << 16) + c, v);
      tmem_wait_ld();
#pragma unroll
      for (int j = 0; j < 32; j++)
        if (c + j < ntile)
          *reinterpret_cast<__nv_bfloat16 *>(base + (c + j) * 256 + r * 2) =
              __float2bfloat16_rn(__uint_as_float(v[j]));
    }
  } else {  // a wait gave up: let copies or MMAs still in flight land before the CTA exits
    if (lane == 0) atomicOr(status, MLA_STATUS_WAIT_TIMEOUT);
    const uint64_t t0 = globaltimer();
    while (globaltimer() - t0 < 2000000ull) {
    }
  }
  tc_fence_before();
  __syncthreads();
  if (ok) {
    const int rows = min(ntile, N - n0);
    for (int i = threadIdx.x; i < rows * 16; i += kThreads) {
      const int n = i >> 4, c = i & 15;
      reinterpret_cast<uint4 *>(out + ((size_t)(n0 + n) * H + h) * kDv)[c] =
          *reinterpret_cast<const uint4 *>(base + n * 256 + c * 16);
    }
  }
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem, 64);
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
  CUtensorMap w_map, x_map;
  if (!make_map_3d(&w_map, w_uv, D_V, kDv, H, w_row, w_head, 128, 1) ||
      !make_map_3d(&x_map, attn, D_V, H, N, ld_head, ld_token, 1, ntile))
    return fail(MLA_ERR_CUDA, "cuTensorMapEncodeTiled failed");
  unsigned int *st = nullptr;
  if (status_word(&st) != MLA_OK) return MLA_ERR_CUDA;
  cudaError_t e = cudaFuncSetAttribute(value_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
  if (e != cudaSuccess) return fail(MLA_ERR_CUDA, cudaGetErrorString(e));
  value_kernel<<<dim3((N + ntile - 1) / ntile, H), kThreads, kSmem, (cudaStream_t)stream>>>(
      w_map, x_map, static_cast<__nv_bfloat16 *>(out), N, H, ntile, st);
  e = cudaGetLastError();
  if (e != cudaSuccess) return fail(MLA_ERR_CUDA, cudaGetErrorString(e));
  set_last_error("");
  return MLA_OK;
}

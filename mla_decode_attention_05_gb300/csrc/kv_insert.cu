// KV insert: RMSNorm of each new token's latent row, then the write of the
// normalised row and its RoPE'd key into the paged cache (vLLM kimi_k3
// specialized-decode "mla.query" page, MlaQuery.insert: page and offset are
// slot // page_size and slot % page_size; k_pe follows the 512 latent values).
//
// Arithmetic, per token with a live slot (every step after S is one IEEE
// fp32 operation, round to nearest even):
//   S    = sum x_i^2, exact, then rounded once to fp32
//   mean = fp32(fp32(S * 2^-9) + eps)
//   r    = fp32(1 / fp32(sqrt(mean)))         (0 when mean == 0)
//   n_i  = bf16(fp32(fp32(x_i * w_i) * r))
// S is exact because a bf16 square is an 8-bit integer squared times a power
// of two: the 512 squares are added as integers in a fixed-point frame
// aligned to the largest one (exact_sum.cuh), so the sum does not depend on
// the order of additions and every code below is a function of the inputs.
//
// One warp per token, a persistent grid of warps striding over the tokens.
// Each warp keeps its next kStages - 1 tokens (latent row, k_pe, slot) in
// flight into a ring in shared memory with cp.async while it processes the
// current one.
// Lane l holds latent values 16l .. 16l + 15, so the 8 lanes 8t .. 8t+7 hold
// FP8 scale tile t (values 128t .. 128t + 127) and every lane stores one
// 16-byte piece of the latent part of the row.
//
// With rotation (mla_kv_insert_rope) the pair (a, b) of a key or query row
// and its angle's cosine c and sine s at the token's position become
//   a' = bf16(fp32(fp32(a c) - fp32(b s)))
//   b' = bf16(fp32(fp32(a s) + fp32(b c)))
// from a table of fp32 cosines and sines (angles of far positions need more
// than 32 bits, so they are the caller's, taken once).  The key is rotated in
// the lanes that hold it before the row is written, so a row is bit for bit
// what the plain insert writes for the rotated bf16 key.  The query rows are
// rotated by further blocks of the same launch: rows of 128 bytes, eight
// lanes a row, so a warp moves four rows at a time; that part is bound by HBM
// (256 bytes a row) and shares nothing with the insert but the launch (8191
// tokens, 64 heads, FP8 rows: 27 us, 5.6 TB/s where outputs cannot stay in L2;
// 64 tokens, 128 heads: 3.1 us).
#include <cuda_fp8.h>

#include "common.cuh"
#include "dependent.cuh"
#include "exact_sum.cuh"

namespace mla {
namespace {

constexpr int kWarps = 8;
constexpr int kBlocksPerSm = 4;

template <int N>
__device__ __forceinline__ void unpack8(const uint4 &u, float (&f)[N], int at) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int k = 0; k < 4; k++) {
    f[at + 2 * k] = __uint_as_float(w[k] << 16);
    f[at + 2 * k + 1] = __uint_as_float(w[k] & 0xFFFF0000u);
  }
}

// Two values -> two e4m3 codes (first value in the low byte), saturating.
__device__ __forceinline__ uint32_t e4m3x2(float a, float b) {
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  return e4m3x2(a, b) | (e4m3x2(c, d) << 16);
}

constexpr int kStages = 4;
constexpr int kStageBytes = 1024 + 128 + 16;  // latent row, k_pe, slot (8 bytes, padded)
constexpr int kSmemBytes = kWarps * kStages * kStageBytes;

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(src))
               : "memory");
}
__device__ __forceinline__ void cp_async8(uint32_t dst, const void *src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(src))
               : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Start the copies of token j into a stage (nothing past the last token);
// every call commits one group, so the group count per stage stays fixed.
template <bool kRope>
__device__ __forceinline__ void issue_token(const KvInsertParams &p, const int64_t *positions, int j, int lane,
                                            uint32_t stage) {
  if (j < p.N) {
    if (kRope && lane == 1) cp_async8(stage + 1160, positions + j);
    const uint8_t *x = reinterpret_cast<const uint8_t *>(p.kv_c + (size_t)j * p.ld_kv) + 32 * lane;
    cp_async16(stage + 32 * lane, x);
    cp_async16(stage + 32 * lane + 16, x + 16);
    if (lane < 8) cp_async16(stage + 1024 + 16 * lane, p.k_pe + (size_t)j * p.ld_pe + 8 * lane);
    if (lane == 0) cp_async8(stage + 1152, p.slots + j);
  }
  cp_async_commit();
}

// Tile scale s = max(fp32(amax / 448), 2^-126) and inv = fp32(1 / s) for a
// bf16 amax > 0.  amax = m * 2^E with m its 8-bit significand (1..255), and
// scaling by a power of two commutes with rounding while the result stays
// normal, so s and inv are fp32(m / 448) and fp32(1 / fp32(m / 448)) (tables
// built at kernel start with those same divisions) with E added to, or taken
// from, the exponent.  A quotient below 2^-126 is the floor, whose
// reciprocal is 2^126.
__device__ __forceinline__ void tile_scale(float amax, const uint32_t *sc_tab, const uint32_t *inv_tab, float &sc,
                                           float &inv) {
  const uint32_t a = __float_as_uint(amax);
  const int e = (int)((a >> 23) & 0xFFu);
  const uint32_t m = ((a >> 16) & 0x7Fu) | (e ? 0x80u : 0u);
  const int E = e ? e - 134 : -133;
  const uint32_t sb = sc_tab[m];
  if ((int)(sb >> 23) + E >= 1) {
    sc = __uint_as_float(sb + ((uint32_t)E << 23));
    inv = __uint_as_float(inv_tab[m] - ((uint32_t)E << 23));
  } else {
    sc = 0x1p-126f;
    inv = 0x1p126f;
  }
}

struct Token {
  uint4 xa, xb, pe;
  long long slot;
};

__device__ __forceinline__ void insert_token(const KvInsertParams &p, const Token &tk, const float (&w)[16],
                                             int lane, const uint32_t *sc_tab, const uint32_t *inv_tab) {
  const long long slot = tk.slot;
  if (slot < 0 || slot >= p.n_slots) {
    if (slot != -1 && lane == 0) atomicOr(p.status, MLA_STATUS_BAD_PAGE);
    return;
  }
  const LaneBf16<8> xr = {{tk.xa.x, tk.xa.y, tk.xa.z, tk.xa.w, tk.xb.x, tk.xb.y, tk.xb.z, tk.xb.w}};
  const uint32_t *xw = xr.w;
  const float S = sum_sq_rn<8>(xr);
  const float mean = __fadd_rn(__fmul_rn(S, 1.f / 512.f), p.eps);
  const float r = mean > 0.f ? __frcp_rn(__fsqrt_rn(mean)) : 0.f;

  // n_i = bf16(fp32(fp32(x_i * w_i) * r)), kept as packed bf16 pairs
  uint32_t nb[8];
#pragma unroll
  for (int k = 0; k < 8; k++) {
    const float x0 = __uint_as_float(xw[k] << 16), x1 = __uint_as_float(xw[k] & 0xFFFF0000u);
    __nv_bfloat162 b2 = __floats2bfloat162_rn(__fmul_rn(__fmul_rn(x0, w[2 * k]), r),
                                              __fmul_rn(__fmul_rn(x1, w[2 * k + 1]), r));
    nb[k] = *reinterpret_cast<uint32_t *>(&b2);
  }

  if (p.kv_format == MLA_KV_BF16) {
    uint8_t *row = p.cache + (size_t)slot * (D_QK * 2);
    uint4 *dst = reinterpret_cast<uint4 *>(row) + 2 * lane;
    dst[0] = make_uint4(nb[0], nb[1], nb[2], nb[3]);
    dst[1] = make_uint4(nb[4], nb[5], nb[6], nb[7]);
    if (lane < 8) reinterpret_cast<uint4 *>(row + D_V * 2)[lane] = tk.pe;
    return;
  }
  float n[16];
#pragma unroll
  for (int k = 0; k < 8; k++) {
    n[2 * k] = __uint_as_float(nb[k] << 16);
    n[2 * k + 1] = __uint_as_float(nb[k] & 0xFFFF0000u);
  }
  if (p.kv_format == MLA_KV_FP8_E4M3) {
    uint8_t *row = p.cache + (size_t)slot * FP8_ROW;
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < 16; i++) amax = fmaxf(amax, fabsf(n[i]));
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    // s = fp32(amax / 448), at least the smallest normal 2^-126 (so 1 / s
    // stays finite); 1 for an all-zero tile
    float sc = 1.f, inv = 1.f;
    if (amax > 0.f) tile_scale(amax, sc_tab, inv_tab, sc, inv);
    uint32_t c[4];
#pragma unroll
    for (int k = 0; k < 4; k++)
      c[k] = e4m3x4(__fmul_rn(n[4 * k], inv), __fmul_rn(n[4 * k + 1], inv), __fmul_rn(n[4 * k + 2], inv),
                    __fmul_rn(n[4 * k + 3], inv));
    reinterpret_cast<uint4 *>(row)[lane] = make_uint4(c[0], c[1], c[2], c[3]);
    if (lane < 8) reinterpret_cast<uint4 *>(row + D_V)[lane] = tk.pe;
    const float s1 = __shfl_sync(0xffffffffu, sc, 8);
    const float s2 = __shfl_sync(0xffffffffu, sc, 16);
    const float s3 = __shfl_sync(0xffffffffu, sc, 24);
    if (lane == 0) reinterpret_cast<float4 *>(p.kv_scales)[slot] = make_float4(sc, s1, s2, s3);
  } else {  // MLA_KV_FP8_E4M3_TENSOR
    uint8_t *row = p.cache + (size_t)slot * D_QK;
    const float ksi = __ldg(p.k_scale_inv);
    uint32_t c[4];
#pragma unroll
    for (int k = 0; k < 4; k++)
      c[k] = e4m3x4(__fmul_rn(n[4 * k], ksi), __fmul_rn(n[4 * k + 1], ksi), __fmul_rn(n[4 * k + 2], ksi),
                    __fmul_rn(n[4 * k + 3], ksi));
    reinterpret_cast<uint4 *>(row)[lane] = make_uint4(c[0], c[1], c[2], c[3]);
    if (lane < 8) {
      float f[8];
      unpack8(tk.pe, f, 0);
      reinterpret_cast<uint2 *>(row + D_V)[lane] =
          make_uint2(e4m3x4(__fmul_rn(f[0], ksi), __fmul_rn(f[1], ksi), __fmul_rn(f[2], ksi), __fmul_rn(f[3], ksi)),
                     e4m3x4(__fmul_rn(f[4], ksi), __fmul_rn(f[5], ksi), __fmul_rn(f[6], ksi), __fmul_rn(f[7], ksi)));
    }
  }
}

// The rotation of one 16-byte piece (values 8 * sub .. 8 * sub + 7) of a row
// of 64, held by eight neighbouring lanes.  cs: the position's 32 cosines and
// 32 sines.  Pairs are (2i, 2i + 1), within a piece, or (i, i + 32), whose
// halves are four lanes apart; every lane of the warp takes part.
__device__ __forceinline__ uint4 rotate8(uint4 x, int sub, const float *cs, int interleaved) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t o[4];
  if (interleaved) {
    const float4 c = __ldg(reinterpret_cast<const float4 *>(cs) + sub);
    const float4 s = __ldg(reinterpret_cast<const float4 *>(cs) + 8 + sub);
    const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int k = 0; k < 4; k++) {
      const float a = __uint_as_float(w[k] << 16), b = __uint_as_float(w[k] & 0xFFFF0000u);
      __nv_bfloat162 r = __floats2bfloat162_rn(__fsub_rn(__fmul_rn(a, cc[k]), __fmul_rn(b, ss[k])),
                                               __fadd_rn(__fmul_rn(a, ss[k]), __fmul_rn(b, cc[k])));
      o[k] = *reinterpret_cast<uint32_t *>(&r);
    }
  } else {
    const float4 *cp = reinterpret_cast<const float4 *>(cs) + 2 * (sub & 3);
    const float4 c0 = __ldg(cp), c1 = __ldg(cp + 1), s0 = __ldg(cp + 8), s1 = __ldg(cp + 9);
    const float cc[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
    const float ss[8] = {s0.x, s0.y, s0.z, s0.w, s1.x, s1.y, s1.z, s1.w};
#pragma unroll
    for (int k = 0; k < 4; k++) {
      const uint32_t u = __shfl_xor_sync(0xffffffffu, w[k], 4);  // the other half of each pair
      float r[2];
#pragma unroll
      for (int e = 0; e < 2; e++) {
        const float own = __uint_as_float(e ? w[k] & 0xFFFF0000u : w[k] << 16);
        const float far = __uint_as_float(e ? u & 0xFFFF0000u : u << 16);
        const float c = cc[2 * k + e], s = ss[2 * k + e];
        r[e] = sub < 4 ? __fsub_rn(__fmul_rn(own, c), __fmul_rn(far, s))
                       : __fadd_rn(__fmul_rn(far, s), __fmul_rn(own, c));
      }
      __nv_bfloat162 r2 = __floats2bfloat162_rn(r[0], r[1]);
      o[k] = *reinterpret_cast<uint32_t *>(&r2);
    }
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// A token's position: false for a token that is skipped (-1), and for one
// outside the table, which also sets the status bit.
__device__ __forceinline__ bool position_ok(long long pos, int max_pos, unsigned int *status, bool tell) {
  if (pos >= 0 && pos < max_pos) return true;
  if (pos != -1 && tell) atomicOr(status, MLA_STATUS_BAD_POSITION);
  return false;
}

// Query rows: each warp takes sixteen heads of one token at a time, as groups
// of four rows (2 KB on their way for each warp).
constexpr int kQHeads = 16;
__device__ void rotate_queries(const KvInsertParams &p, const RopeParams &r, int unit, int stride) {
  const int lane = threadIdx.x & 31, sub = lane & 7;
  const int groups = (r.H + kQHeads - 1) / kQHeads;
  const long long units = (long long)p.N * groups;
  for (long long u = unit; u < units; u += stride) {
    const int n = (int)(u / groups), h0 = (int)(u % groups) * kQHeads;
    const long long pos = __ldg(reinterpret_cast<const long long *>(r.positions) + n);
    if (!position_ok(pos, r.max_pos, p.status, lane == 0)) continue;
    const float *cs = r.cos_sin + pos * 64;
    uint4 x[kQHeads / 4];
#pragma unroll
    for (int i = 0; i < kQHeads / 4; i++) {
      const int h = h0 + 4 * i + (lane >> 3);
      x[i] = make_uint4(0u, 0u, 0u, 0u);
      if (h < r.H) x[i] = *reinterpret_cast<const uint4 *>(r.q_pe + n * r.q_tok + h * r.q_head + 8 * sub);
    }
#pragma unroll
    for (int i = 0; i < kQHeads / 4; i++) {
      const int h = h0 + 4 * i + (lane >> 3);
      if (h0 + 4 * i >= r.H) break;  // (the same for the whole warp)
      const uint4 y = rotate8(x[i], sub, cs, r.interleaved);
      if (h < r.H) *reinterpret_cast<uint4 *>(r.q_out + n * r.o_tok + h * r.o_head + 8 * sub) = y;
    }
  }
}

template <bool kRope>
__global__ void __launch_bounds__(kWarps * 32, kBlocksPerSm)
    kv_insert_kernel(KvInsertParams p, RopeParams r, int insert_blocks) {
  if (kRope) {
    grid_dep_trigger();
    grid_dep_wait();  // nothing of the caller's is read or written before the kernel in front has ended
  }
  // Blocks of both kinds are spread evenly over the grid, so that the queries'
  // stream runs beside the inserts' arithmetic on every SM.
  int block = blockIdx.x;
  if (kRope) {
    const int grid = gridDim.x, before = (int)((long long)block * insert_blocks / grid);
    if ((int)((long long)(block + 1) * insert_blocks / grid) == before) {
      rotate_queries(p, r, (block - before) * kWarps + ((int)threadIdx.x >> 5), (grid - insert_blocks) * kWarps);
      return;
    }
    block = before;
  }
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ uint32_t sc_tab[256], inv_tab[256];  // fp32(m / 448), fp32(1 / that), m = 0..255
  static_assert(kWarps * 32 == 256, "one table entry per thread");
  {
    const float q = __fdiv_rn((float)threadIdx.x, 448.f);
    sc_tab[threadIdx.x] = __float_as_uint(q);
    inv_tab[threadIdx.x] = __float_as_uint(__fdiv_rn(1.f, q));  // m = 0: unused
  }
  __syncthreads();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int first = block * kWarps + warp;
  const int stride = insert_blocks * kWarps;
  if (first >= p.N) return;
  uint8_t *ring = smem + warp * kStages * kStageBytes;
  const uint32_t ring_s = (uint32_t)__cvta_generic_to_shared(ring);
  float w[16];
  const uint4 *wr = reinterpret_cast<const uint4 *>(p.w_kva) + 2 * lane;
  unpack8(__ldg(wr), w, 0);
  unpack8(__ldg(wr + 1), w, 8);
#pragma unroll
  for (int s = 0; s < kStages - 1; s++) issue_token<kRope>(p, r.positions, first + s * stride, lane, ring_s + s * kStageBytes);
  int st = 0;
  for (int j = first; j < p.N; j += stride) {
    const int ahead = st == 0 ? kStages - 1 : st - 1;  // the stage freed last iteration
    issue_token<kRope>(p, r.positions, j + (kStages - 1) * stride, lane, ring_s + ahead * kStageBytes);
    cp_async_wait<kStages - 1>();  // this token's group has landed (for this lane's copies)
    __syncwarp();                  // ... and lane 0's slot copy is visible to all lanes
    const uint8_t *cur = ring + st * kStageBytes;
    Token tk;
    tk.xa = *reinterpret_cast<const uint4 *>(cur + 32 * lane);
    tk.xb = *reinterpret_cast<const uint4 *>(cur + 32 * lane + 16);
    tk.pe = lane < 8 ? *reinterpret_cast<const uint4 *>(cur + 1024 + 16 * lane) : make_uint4(0u, 0u, 0u, 0u);
    tk.slot = *reinterpret_cast<const long long *>(cur + 1152);
    if (kRope) {
      const long long pos = *reinterpret_cast<const long long *>(cur + 1160);
      __syncwarp();  // every lane has read the stage before it is refilled
      if (!position_ok(pos, r.max_pos, p.status, lane == 0)) {
        st = st + 1 == kStages ? 0 : st + 1;
        continue;
      }
      tk.pe = rotate8(tk.pe, lane & 7, r.cos_sin + pos * 64, r.interleaved);  // (lanes 8.. rotate zeros)
    } else {
      __syncwarp();  // every lane has read the stage before it is refilled
    }
    insert_token(p, tk, w, lane, sc_tab, inv_tab);
    st = st + 1 == kStages ? 0 : st + 1;
  }
  cp_async_wait<0>();
}

}  // namespace

cudaError_t launch_kv_insert(const KvInsertParams &p, cudaStream_t stream) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int need = (p.N + kWarps - 1) / kWarps;
  const int blocks = need < sms * kBlocksPerSm ? need : sms * kBlocksPerSm;
  static_assert(kSmemBytes <= 48 * 1024, "dynamic shared memory above the default limit");
  kv_insert_kernel<false><<<blocks, kWarps * 32, kSmemBytes, stream>>>(p, RopeParams{}, blocks);
  return cudaGetLastError();
}

cudaError_t launch_kv_insert_rope(const KvInsertParams &p, const RopeParams &r, cudaStream_t stream) {
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const long long most = (long long)sms * kBlocksPerSm;
  const long long need = ((long long)p.N + kWarps - 1) / kWarps;
  const long long q_units = r.q_pe ? (long long)p.N * ((r.H + kQHeads - 1) / kQHeads) : 0;
  const long long q_need = (q_units + kWarps - 1) / kWarps;
  // All blocks run at once.  With queries, which are most of the bytes, the
  // inserts get what those leave, at least a block (8 tokens at a time) on each SM.
  const long long rest = q_need + sms < most ? most - q_need : sms;
  const int blocks = (int)(need < rest ? need : rest);
  const int q_blocks = (int)(q_need < most - blocks ? q_need : most - blocks);
  return launch_dependent(kv_insert_kernel<true>, blocks + q_blocks, kWarps * 32, kSmemBytes, stream, p, r, blocks);
}

}  // namespace mla

// What the operators around the decode share: their launches as programmatic
// dependents, the limit of their waits, and the rotating insert's parameters.
// (Apart from common.cuh and ptx.cuh, which the decode kernel is compiled from: a
// measurement of that kernel holds as long as its sources stay as they are.)
#pragma once

#include "common.cuh"

namespace mla {

// Launches a kernel as a programmatic dependent of the one before it in the
// stream (see grid_dep_wait): it sets itself up while that one ends.
template <typename... P, typename... A>
inline cudaError_t launch_dependent(void (*kernel)(P...), unsigned grid, unsigned block, unsigned smem,
                                    cudaStream_t stream, A... args) {
  cudaLaunchAttribute pdl[1];
  pdl[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(block);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = pdl;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// What mla_kv_insert_rope adds to an insert: the angle table, the tokens'
// positions and the query rows that are rotated with the keys.
struct RopeParams {
  const int64_t *positions;
  const float *cos_sin;  // [max_pos][64]: 32 cosines, 32 sines
  const __nv_bfloat16 *q_pe;  // rows of 64 values, null without queries
  __nv_bfloat16 *q_out;
  long long q_tok, q_head, o_tok, o_head;  // element strides
  int max_pos;
  int interleaved;
  int H;
};
cudaError_t launch_kv_insert_rope(const KvInsertParams &p, const RopeParams &r, cudaStream_t stream);

// The calling thread's limit of bounded waits (mla_set_wait_limit_ns).
unsigned long long wait_limit_ns();

}  // namespace mla

// What the parts of the decode over shared prefixes have in common.
#pragma once

#include "common.cuh"

namespace mla {

// One item of work: up to 128 query rows that lie side by side, and the keys that
// all of them attend to: a group's rows and its prefix, or the rows of one sequence
// and its own tokens.
struct SharedItem {
  int q_row;   // first of its rows among all B * T * H
  int rows;
  int len;     // its keys; with `own`, the sequence's tokens, of which a row may see fewer
  int tiles;   // 64-key tiles
  int src;     // group (prefix) or sequence (own): the row of the page table
  int own;
  int row0;    // own: its first row within the sequence
  int slot;    // its first slot of partial results
};
static_assert(sizeof(SharedItem) == 32, "read as two 16-byte words");

struct SharedParams {
  const __nv_bfloat16 *q;
  const uint8_t *cache;
  const float *kv_scales;
  const int32_t *prefix_table, *prefix_lens, *offsets;  // offsets null: one group of all sequences
  const int32_t *block_table, *seqlens;
  unsigned int *status;
  int format, num_pages, max_prefix, max_pages, G, B, T, H, causal;
  int own_room;   // FP8: room for widened own pages
  int n_mt;       // own tiles of query rows of a sequence
  int parts;
  float scale_log2;
  unsigned long long wait_ns;
  // workspace
  SharedItem *items;
  int32_t *md;         // [parts][8], as mla_decode_metadata's
  int32_t *pieces;     // [room] slots of an item that hold results
  int32_t *n_prefix;   // items that are prefixes: they come first
  int4 *groups;        // [G] {first sequence, end, first item, keys}
  int2 *seq;           // [B] {first prefix item of its group or -1, its first row among the group's}
  int32_t *lens_o;     // [B] own tokens, clamped, where they
  int32_t *md_o, *ns_o, *cnt_o;  // may go through the decode kernel: its schedule (else null)
  int32_t *apart;      // with md_o: whether they do
  int32_t *first;      // FP8: [G + B + 1] widened pages of the prefixes and sequences before each
  uint8_t *scratch;    // FP8: pages as bf16, those in use side by side: [64][576], with scales [64][1088]
  size_t scratch_pages;
  float *lse_p, *o_p;  // partial results: base-2 log-sum-exp [slots][128] and output [slots][64][128][8]
  float *lse_o, *o_o;  // those of the decode kernel
  uint8_t *ring;       // [parts][P_RING][P_SLOT_BYTES]
  __nv_bfloat16 *out;
  float *lse;
};

cudaError_t launch_shared_attention(const SharedParams &p, cudaStream_t stream);

}  // namespace mla

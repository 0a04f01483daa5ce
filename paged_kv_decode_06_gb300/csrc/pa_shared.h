// Layout of the shared-prefix part of a decode call: what the plan kernel writes, and
// how the prefix and merge kernels number its work and its partial rows.
//
// The rows of one (group, KV head), G query heads of every query token of the group's
// sequences, are cut into pairs of 128-row tiles, one tile a slot; a last pair of at most
// 128 rows has one tile, which both slots take, each a half of every block of keys.  A step
// is one block of 128 keys for both tiles, or two blocks for the single tile.  Steps stand
// end to end in (group, head, pair, block) order, X in all; CTA c of the NG in use takes
// [c X / NG, (c + 1) X / NG).
//
// The sequences' own pages are attended beside the shared ones, by the split kernel on the
// SMs that the prefix kernel leaves: the plan cuts the SMs in two by the work of each.
//
// A CTA leaves partial rows for each piece it holds: piece (pair, CTA c) at rows row0 +
// 256 c of the pair's row0 = the padded rows of all pairs before it, so that no two pieces
// meet: a next pair starts at least its predecessor's rows, a next CTA 256 rows further.  A
// slot's tile of R rows holds chunk d / 4 of all R rows, then the next chunk.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace pa {

constexpr int kSharedTile = 128;
constexpr int kSharedPair = 2 * kSharedTile;
constexpr int kSharedBlockPages = 8;

struct SharedGroup {
  int32_t seq;          // the sequence whose block-table row names the pages
  int32_t pages;        // shared pages; 0: nothing shared
  int32_t t0, rows;     // first query token, rows (query tokens x G) a KV head
  int32_t pairs;        // tile pairs a head
  int32_t last_rows;    // rows of the last pair
  int32_t blocks;       // blocks of keys
  int32_t steps_head;   // steps a head
  int32_t rows_head;    // padded rows a head
  int32_t reserved;
  int64_t step0;        // steps of the groups before
  int64_t row0;         // padded rows of the groups before
};

struct SharedTotals {
  int64_t steps;
  int32_t ctas;         // CTAs that take the steps
};

__host__ __device__ inline bool shared_single(const SharedGroup& g, int pair) {
  return pair == g.pairs - 1 && g.last_rows <= kSharedTile;
}
__host__ __device__ inline int shared_steps(const SharedGroup& g, int pair) {
  return shared_single(g, pair) ? (g.blocks + 1) / 2 : g.blocks;
}
// Rows of a slot's tile.
__host__ __device__ inline int shared_tile_rows(const SharedGroup& g, int pair, int slot) {
  const int rows = pair == g.pairs - 1 ? g.last_rows : kSharedPair;
  if (rows <= kSharedTile) return rows;
  return slot == 0 ? kSharedTile : rows - kSharedTile;
}
// The CTA of ng that holds step x (64-bit divisions only where they are needed).
__host__ __device__ inline int shared_cta_of(int64_t x, int64_t steps, int ng) {
  const int64_t y = (x + 1) * ng - 1;
  if (y < (int64_t(1) << 32) && steps < (int64_t(1) << 32))
    return static_cast<int>(static_cast<uint32_t>(y) / static_cast<uint32_t>(steps));
  return static_cast<int>(y / steps);
}

struct SharedParams {
  const uint16_t* q;          // bf16 [T, Hq, D], head stride D
  int64_t q_stride_t;
  const int32_t* block_tables;
  int64_t bt_stride;
  const int32_t* seq_lens;
  const int32_t* qsl;         // [B + 1] or nullptr
  const int32_t* group_start; // [groups + 1]
  const int32_t* shared_lens; // [groups]
  int32_t num_seqs, num_tokens, num_groups, max_qlen, max_blocks, num_pages, G, Hkv;
  int32_t min_pages;          // fewer shared pages are left to the sequences
  int32_t ctas;               // CTAs of the prefix kernel
  int32_t own_ctas;           // CTAs of the split kernel
  int32_t beside;             // they run side by side on `ctas` SMs
  int32_t step_cost, page_cost, unit_cost;   // time of a step, a sequence's page and a sequence, for one head on one SM
  int32_t alone_cost;         // nothing is shared that takes less on an SM
  int32_t split_boxes;        // 128 features, bf16, bit 0 for K, 1 for V: heads are not contiguous, pages come in four boxes
  float scale_log2;
  uint64_t wait_ns;
  int32_t give_up_cta;        // testing aid: the softmax of this CTA's first slot gives up at once (-1 = off)
  uint32_t* err;
  // workspace: written by the plan kernel ...
  int32_t* skip;              // [B] pages that the group attends for the sequence
  int32_t* seq_group;         // [B] its group, -1: none
  SharedGroup* groups;
  SharedTotals* totals;
  uint64_t* ready;
  uint64_t call;              // number of this call, never 0
  // ... and by the prefix kernel: partial rows
  float2* ws_ml;
  float* ws_o;
};

cudaError_t launch_shared_plan(const SharedParams& p, bool pdl, cudaStream_t stream);
cudaError_t launch_shared_prefix(int head_dim, bool fp8, const CUtensorMap& tk, const CUtensorMap& tv,
                                 const SharedParams& p, int grid, bool pdl, cudaStream_t stream);
cudaError_t set_shared_smem_limits();

}  // namespace pa

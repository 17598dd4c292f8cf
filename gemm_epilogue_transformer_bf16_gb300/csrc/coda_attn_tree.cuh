// Attention of drafted trees over the 4-bit cache: arguments and launcher.
#pragma once
#include <cuda.h>

#include "coda_kvcache.cuh"

namespace coda {

constexpr int TREE_MAX_NODES = 256;  // of a tree given by parents
constexpr int TREE_ROWS = 128;       // query rows (nodes times heads of a group) of a tile
constexpr int TREE_MAX_CTAS = 160;   // partial results reserved for this many CTAs

struct TreeArgs {
  KvCache c;
  const __nv_bfloat16* Q;  // [T, n_q * 128]
  int64_t ldq;
  const int32_t* table;    // [B, max_pages]
  int max_pages;
  const int32_t* seq_lens;
  const int32_t* cu;       // [B + 1]
  const int32_t* parents;  // [T] within the tree, or null: chains
  int T, B, n_q, group;
  float scale_log2;
  __nv_bfloat16* O;        // [T, n_q * 128]
  float* lse;              // [T, n_q]
  int64_t* places;         // [B + 2]: places on the line of work before each sequence, their total, places per CTA
  uint32_t* seen;          // [TREE_MAX_CTAS, TREE_ROWS / 32, TREE_MAX_NODES] rows of a CTA's tile that see a node, by warpgroup
  float* part;             // [2 * TREE_MAX_CTAS, part_rows, 128] normalised partial outputs
  float* part_lse;         // [2 * TREE_MAX_CTAS, part_rows] log2 domain
  int part_rows;
  int* status;
};
// maps: codes, block scales, row scales (see cache_maps).
cudaError_t launch_attn_tree(const TreeArgs& a, const CUtensorMap* maps, int sms, cudaStream_t s);

// The cache's arrays as tensors whose boxes are one head's rows of a page, at
// most 128 of them, keys and values together.
bool cache_maps(CUtensorMap* maps, const KvCache& c);

}  // namespace coda

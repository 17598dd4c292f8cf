// Attention of drafted trees over the 4-bit cache: arguments and launcher.
#pragma once
#include "coda_kvcache.cuh"

namespace coda {

constexpr int TREE_MAX_NODES = 256;  // of a tree given by parents

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
  int* status;
};
cudaError_t launch_attn_tree(const TreeArgs& a, int sms, cudaStream_t s);

}  // namespace coda

// Verification of drafted tokens: arguments and launcher.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

namespace coda {

constexpr int VERIFY_MAX_NODES = 1024;  // of one tree: what a CTA keeps in shared memory

struct VerifyArgs {
  const void* P;            // [T, V] probabilities of the target after every node
  const void* Q;            // [T, V] those that the node's children were drawn from, or null
  const int32_t* tokens;    // [T]
  const int32_t* cu;        // [B + 1]
  const int32_t* parents;   // [T] within the tree, or null: chains
  const float* u;           // [T]
  const float* u_next;      // [B]
  int32_t* count;           // [B]
  int32_t* nodes;           // [B, width]
  int32_t* out;             // [B, width]
  int64_t V;
  int T, B, width;
  int ctas;                 // of a request, set at the launch
  int* status;
};
cudaError_t launch_verify(VerifyArgs a, bool f32, cudaStream_t s);

}  // namespace coda

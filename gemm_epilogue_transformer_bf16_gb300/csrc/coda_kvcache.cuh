// The 4-bit key/value cache: layout and launchers.
//
// Slot s = page * page_size + offset holds, for each plane (0 keys, 1
// values) and key/value head h, one NVFP4 row of 128 elements: 64 bytes of
// e2m1 codes, 8 e4m3 block scales and an fp32 row scale, at row index
// ((page * 2 + plane) * n_kv + h) * page_size + offset of three arrays, so
// the rows of one head within a page are contiguous.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace coda {

struct KvCache {
  uint8_t* codes;  // [pages, 2, n_kv, page, 64]
  uint8_t* sf;     // [pages, 2, n_kv, page, 8]
  float* scale;    // [pages, 2, n_kv, page]
  int num_pages;
  int page_shift;  // page size = 1 << page_shift, >= 16
  int n_kv;
};

// rows: 2 * n_kv per token.
cudaError_t launch_kv_append(const KvCache& c, const __nv_bfloat16* K, int64_t ldk, const __nv_bfloat16* V,
                             int64_t ldv, const int32_t* slots, int rows, int* status, cudaStream_t s);
// f32: outputs are fp32, else bf16; both [T, n_kv * 128].
cudaError_t launch_kv_read(const KvCache& c, const int32_t* slots, int rows, void* K, void* V, bool f32, int* status,
                           cudaStream_t s);

struct AcceptArgs {
  KvCache c;
  const int32_t* table;  // [B, max_pages]
  int max_pages;
  const int32_t *seq_lens, *cu, *nodes, *count;  // [B], [B + 1], [B, width], [B]
  int B, width;
  int32_t* out_lens;     // [B]
  int* status;
};
cudaError_t launch_kv_accept(const AcceptArgs& a, cudaStream_t s);

constexpr int DEC_MAX_CTAS = 3 * 160;  // partial results reserved for this many CTAs
constexpr int DEC_HEADS = 16;          // query heads of one pass over a key/value head's rows

struct DecodeArgs {
  KvCache c;
  const __nv_bfloat16* Q;
  int64_t ldq;
  const int32_t* table;  // [B, max_pages]
  int max_pages;
  const int32_t* seq_lens;
  int B, n_q, group, splits;  // splits: passes a group of more than DEC_HEADS heads is cut into
  float scale_log2;
  __nv_bfloat16* O;  // [B, n_q * 128]
  float* lse;        // [B, n_q]
  int* units;        // [B + 2]: places on the line of units before each sequence, their total, places per CTA
  float* part;       // [2 * DEC_MAX_CTAS, heads, 128] normalised partial outputs
  float* part_lse;   // [2 * DEC_MAX_CTAS, heads] log2 domain
  int part_heads;    // min(group, DEC_HEADS)
  int* status;
};
cudaError_t launch_attn_decode(const DecodeArgs& a, int sms, cudaStream_t s);

}  // namespace coda

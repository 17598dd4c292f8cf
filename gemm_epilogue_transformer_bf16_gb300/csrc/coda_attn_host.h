// Host helpers that the attention, cache and drafting entry points share:
// argument checks and the layout of workspaces.
#pragma once
#include <cmath>
#include <cstdint>
#include <algorithm>

#include "coda.h"
#include "coda_attn.cuh"
#include "coda_kvcache.cuh"

namespace {

constexpr size_t HEADER = 256;
constexpr double LOG2E = 1.4426950408889634074;

inline bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
inline bool al4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
inline size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

// Lays out (base == nullptr: only sizes) consecutive 256-byte aligned arrays.
struct Cursor {
  uint8_t* base;
  size_t off = HEADER;
  template <class T>
  T* take(int64_t count) {
    T* p = base ? reinterpret_cast<T*>(base + off) : nullptr;
    off = up256(off + static_cast<size_t>(count) * sizeof(T));
    return p;
  }
};

// Shapes both directions share.  CODA_OK, or the error to return.
inline int check_shape(int64_t Tq, int64_t Tk, int64_t n_seq, int32_t n_q, int32_t n_kv, int32_t head_dim, float scale) {
  if (Tq < 0 || Tk < 0 || n_seq < 0 || n_q <= 0 || n_kv <= 0) return CODA_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !std::isfinite(scale)) return CODA_ERR_INVALID_ARG;
  if (head_dim != coda::ATTN_D || n_q % n_kv != 0) return CODA_ERR_UNSUPPORTED;
  // rows and work items are counted in 32 bits on the device
  constexpr int64_t LIM = int64_t(1) << 30;
  if (Tq >= LIM || Tk >= LIM || n_seq >= LIM / 4 || n_q >= 65536) return CODA_ERR_UNSUPPORTED;
  if ((std::max(Tq / 32, Tk / coda::ATTN_BLK) + n_seq + 1) * n_q >= (int64_t(1) << 31)) return CODA_ERR_UNSUPPORTED;
  return CODA_OK;
}

#define CK(x)                     \
  do {                            \
    int _r = (x);                 \
    if (_r != CODA_OK) return _r; \
  } while (0)
#define CU(x) \
  do { if ((x) != cudaSuccess) return CODA_ERR_CUDA; } while (0)

// The cache's shape; CODA_OK or the error to return.
inline int check_cache(coda::KvCache& c, const uint8_t* codes, const uint8_t* sf, const float* scale, int64_t num_pages,
                int32_t page_size, int32_t n_kv, int32_t head_dim) {
  if (num_pages < 0 || page_size <= 0 || n_kv <= 0) return CODA_ERR_INVALID_ARG;
  if (head_dim != coda::ATTN_D || page_size < 16 || (page_size & (page_size - 1)) || n_kv >= 65536)
    return CODA_ERR_UNSUPPORTED;
  if (num_pages * page_size >= (int64_t(1) << 31)) return CODA_ERR_UNSUPPORTED;  // slots are 32-bit
  if (num_pages > 0 && (!codes || !sf || !scale)) return CODA_ERR_INVALID_ARG;
  if (!al16(codes) || !al16(sf) || !al16(scale)) return CODA_ERR_ALIGNMENT;
  c.codes = const_cast<uint8_t*>(codes);
  c.sf = const_cast<uint8_t*>(sf);
  c.scale = const_cast<float*>(scale);
  c.num_pages = static_cast<int>(num_pages);
  c.page_shift = 0;
  while ((1 << c.page_shift) < page_size) ++c.page_shift;
  c.n_kv = n_kv;
  return CODA_OK;
}

inline int check_ws(const void* ws, size_t have, size_t need) {
  if (!ws || have < need) return CODA_ERR_WORKSPACE;
  return al16(ws) ? CODA_OK : CODA_ERR_ALIGNMENT;
}

inline const __nv_bfloat16* B(const coda_bf16* p) { return reinterpret_cast<const __nv_bfloat16*>(p); }
inline __nv_bfloat16* B(coda_bf16* p) { return reinterpret_cast<__nv_bfloat16*>(p); }

}  // namespace

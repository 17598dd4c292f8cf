// Host side of the attention operators declared in include/coda.h: argument
// checks, tensor maps, workspace layout and launch sequences.
#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstdlib>
#include <cstring>
#include <mutex>

#include "coda.h"
#include "coda_attn.cuh"
#include "coda_internal.h"
#include "coda_status.h"

namespace coda {

bool attn_programmatic_launch() {
  static const bool v = [] {
    const char* e = std::getenv("CODA_PDL");
    return e ? e[0] != '0' : true;
  }();
  return v;
}

cudaError_t attn_smem_attribute(const void* kernel, int id, uint32_t bytes) {
  static std::mutex init;
  static std::atomic<bool> done[8][64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64 || id < 0 || id >= 8) return cudaErrorInvalidDevice;
  if (done[id][dev].load(std::memory_order_acquire)) return cudaSuccess;
  std::lock_guard<std::mutex> lock(init);
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
  if (e == cudaSuccess) done[id][dev].store(true, std::memory_order_release);
  return e;
}

}  // namespace coda

namespace {

constexpr size_t HEADER = 256;
constexpr uint64_t WAIT_LIMIT_NS = 2000000000ull;  // 2 s per pipeline wait
constexpr double LOG2E = 1.4426950408889634074;

bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool al4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }
size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

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
int check_shape(int64_t Tq, int64_t Tk, int64_t n_seq, int32_t n_q, int32_t n_kv, int32_t head_dim, float scale) {
  if (Tq < 0 || Tk < 0 || n_seq < 0 || n_q <= 0 || n_kv <= 0) return CODA_ERR_INVALID_ARG;
  if (!(scale > 0.f) || !std::isfinite(scale)) return CODA_ERR_INVALID_ARG;
  if (head_dim != coda::ATTN_D || n_q % n_kv != 0) return CODA_ERR_UNSUPPORTED;
  // rows and work items are counted in 32 bits on the device
  constexpr int64_t LIM = int64_t(1) << 30;
  if (Tq >= LIM || Tk >= LIM || n_seq >= LIM / 4 || n_q >= 65536) return CODA_ERR_UNSUPPORTED;
  if ((Tq / 32 + n_seq + 1) * n_q >= (int64_t(1) << 31)) return CODA_ERR_UNSUPPORTED;
  return CODA_OK;
}

// Heads that share a 128-row tile (a power of two dividing the group).  With
// one head a tile covers 128 tokens, so sequences of a few tokens would leave
// most rows empty: tiles then take several heads of fewer tokens each.  Rule:
// as many as keep a tile at least as long as the mean sequence.
int head_shift(int64_t Tq, int64_t n_seq, int group) {
  const int64_t mean = n_seq > 0 ? (Tq + n_seq - 1) / n_seq : Tq;
  int s = 0;
  while (s < 4 && group % (2 << s) == 0 && (coda::ATTN_BLK >> (s + 1)) >= mean) ++s;
  return s;
}

struct PlanLayout {
  coda::AttnPlanArgs a;
  int64_t max_q_tiles, max_k_tiles;
};

void lay_plan(Cursor& c, PlanLayout& l, int64_t Tq, int64_t Tk, int64_t n_seq, int q_span, bool keys) {
  l.max_q_tiles = Tq / q_span + n_seq;
  l.max_k_tiles = keys ? Tk / coda::ATTN_BLK + n_seq : 0;
  l.a.plan.counts = c.take<int>(2);
  l.a.prefix_q = c.take<int>(n_seq + 1);
  l.a.prefix_k = keys ? c.take<int>(n_seq + 1) : nullptr;
  l.a.plan.q_tiles = c.take<coda::AttnTile>(l.max_q_tiles);
  l.a.plan.k_tiles = keys ? c.take<coda::AttnTile>(l.max_k_tiles) : nullptr;
  l.a.q_span = q_span;
}

bool map_rows(CUtensorMap* m, const void* p, int64_t rows, int64_t cols, int64_t ld) {
  const uint64_t dims[2] = {static_cast<uint64_t>(cols), static_cast<uint64_t>(rows)};
  const uint64_t st[1] = {static_cast<uint64_t>(ld) * 2};
  const uint32_t box[2] = {64, static_cast<uint32_t>(coda::ATTN_BLK)};
  return coda::encode_bf16_map(m, p, 2, dims, st, box);
}

#define CK(x)                     \
  do {                            \
    int _r = (x);                 \
    if (_r != CODA_OK) return _r; \
  } while (0)
#define CU(x) \
  do { if ((x) != cudaSuccess) return CODA_ERR_CUDA; } while (0)

const __nv_bfloat16* B(const coda_bf16* p) { return reinterpret_cast<const __nv_bfloat16*>(p); }
__nv_bfloat16* B(coda_bf16* p) { return reinterpret_cast<__nv_bfloat16*>(p); }

}  // namespace

extern "C" {

size_t coda_attention_workspace_size(int64_t Tq, int64_t Tk, int64_t n_seq, int32_t n_q, int32_t n_kv,
                                     int32_t head_dim) {
  if (check_shape(Tq, Tk, n_seq, n_q, n_kv, head_dim, 1.f) != CODA_OK) return HEADER;
  Cursor c{nullptr};
  PlanLayout l{};
  // the shortest entry a call can take, so the size depends on the shape alone
  lay_plan(c, l, Tq, Tk, n_seq, coda::ATTN_BLK >> head_shift(Tq, n_seq, n_q / n_kv), false);
  return c.off;
}

int coda_attention(const coda_bf16* Q, int64_t ldq, const coda_bf16* K, int64_t ldk, const coda_bf16* V, int64_t ldv,
                   const int32_t* cu_q, const int32_t* cu_k, int64_t n_seq, int32_t n_q, int32_t n_kv,
                   int32_t head_dim, float scale, coda_bf16* O, float* lse, int64_t Tq, int64_t Tk, void* ws,
                   size_t ws_bytes, coda_stream stream) {
  CK(check_shape(Tq, Tk, n_seq, n_q, n_kv, head_dim, scale));
  if (Tq == 0 || n_seq == 0) return CODA_OK;
  if (!Q || !cu_q || !O || !lse || (Tk > 0 && (!K || !V))) return CODA_ERR_INVALID_ARG;
  if (!cu_k) cu_k = cu_q;
  if (cu_k == cu_q && Tk != Tq) return CODA_ERR_INVALID_ARG;
  const int64_t wq = int64_t(n_q) * head_dim, wk = int64_t(n_kv) * head_dim;
  if (ldq < wq || ldk < wk || ldv < wk) return CODA_ERR_INVALID_ARG;
  if (!al16(Q) || !al16(K) || !al16(V) || !al16(O) || !al4(lse) || !al4(cu_q) || !al4(cu_k) || ldq % 8 || ldk % 8 ||
      ldv % 8)
    return CODA_ERR_ALIGNMENT;
  if (!ws || ws_bytes < coda_attention_workspace_size(Tq, Tk, n_seq, n_q, n_kv, head_dim)) return CODA_ERR_WORKSPACE;
  if (!al16(ws)) return CODA_ERR_ALIGNMENT;
  const int sms = coda::device_sms();
  if (sms <= 0 || !coda::tensor_map_encoder()) return CODA_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int group = n_q / n_kv;
  const int hs = head_shift(Tq, n_seq, group);
  const int pair_heads = (group >> hs) % 2 == 0 ? 1 : 0;
  const int span = coda::ATTN_BLK >> hs;
  Cursor c{static_cast<uint8_t*>(ws)};
  PlanLayout l{};
  lay_plan(c, l, Tq, Tk, n_seq, pair_heads ? span : 2 * span, false);
  l.a.cu_q = cu_q;
  l.a.cu_k = cu_k;
  l.a.n_seq = static_cast<int>(n_seq);
  l.a.Tq = Tq;
  l.a.Tk = Tk;
  l.a.status = static_cast<int*>(ws);
  CUtensorMap maps[3];
  const uint64_t dims[3] = {static_cast<uint64_t>(head_dim), static_cast<uint64_t>(n_q), static_cast<uint64_t>(Tq)};
  const uint64_t st[2] = {static_cast<uint64_t>(head_dim) * 2, static_cast<uint64_t>(ldq) * 2};
  const uint32_t box[3] = {64, 1u << hs, static_cast<uint32_t>(span)};
  if (!coda::encode_bf16_map(&maps[0], Q, 3, dims, st, box)) return CODA_ERR_CUDA;
  if (Tk > 0) {
    if (!map_rows(&maps[1], K, Tk, wk, ldk) || !map_rows(&maps[2], V, Tk, wk, ldv)) return CODA_ERR_CUDA;
  } else {
    maps[1] = maps[2] = maps[0];  // no key is ever loaded
  }
  coda::AttnFwdArgs a{};
  a.counts = l.a.plan.counts;
  a.tiles = l.a.plan.q_tiles;
  a.O = B(O);
  a.lse = lse;
  a.Tq = Tq;
  a.n_q = n_q;
  a.group = group;
  a.head_shift = hs;
  a.pair_heads = pair_heads;
  a.scale = scale;
  a.scale_log2 = static_cast<float>(scale * LOG2E);
  a.status = static_cast<int*>(ws);
  a.timeout_ns = WAIT_LIMIT_NS;
  CU(coda::launch_attn_plan(l.a, s));
  CU(coda::launch_attn_fwd(a, maps, l.max_q_tiles * (n_q >> (hs + pair_heads)), sms, s));
  return CODA_OK;
}

}  // extern "C"

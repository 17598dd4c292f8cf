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
#include "coda_kvcache.cuh"
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
  if ((std::max(Tq / 32, Tk / coda::ATTN_BLK) + n_seq + 1) * n_q >= (int64_t(1) << 31)) return CODA_ERR_UNSUPPORTED;
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

// parts: room for the parts of cut runs, in the key list if there is one (see
// bwd_max_parts), else in the query list (fwd_max_parts).
void lay_plan(Cursor& c, PlanLayout& l, int64_t Tq, int64_t Tk, int64_t n_seq, int q_span, bool keys, int64_t parts) {
  l.max_q_tiles = Tq / q_span + n_seq;
  l.max_k_tiles = keys ? Tk / coda::ATTN_BLK + n_seq : 0;
  l.a.plan.counts = c.take<int>(4);
  l.a.prefix_q = c.take<int>(n_seq + 1);
  l.a.prefix_k = keys ? c.take<int>(n_seq + 1) : nullptr;
  l.a.plan.q_tiles = c.take<coda::AttnTile>(l.max_q_tiles + (keys ? 0 : parts));
  l.a.plan.k_tiles = keys ? c.take<coda::AttnTile>(l.max_k_tiles + parts) : nullptr;
  l.a.plan.cuts = c.take<coda::AttnTile>(parts);
  l.a.q_span = q_span;
}

constexpr int64_t PART_FLOATS = 2 * coda::ATTN_BLK * coda::ATTN_D;

// Forward: how a shape is cut into items.
struct FwdShape {
  int head_shift, pair_heads, span, q_span, per;  // rows per tile, per list entry; items per entry
};
FwdShape fwd_shape(int64_t Tq, int64_t n_seq, int n_q, int group) {
  FwdShape f;
  f.head_shift = head_shift(Tq, n_seq, group);
  f.pair_heads = (group >> f.head_shift) % 2 == 0 ? 1 : 0;
  f.span = coda::ATTN_BLK >> f.head_shift;
  f.q_span = f.pair_heads ? f.span : 2 * f.span;
  f.per = n_q >> (f.head_shift + f.pair_heads);
  return f;
}
// Bound on the parts (of 128 KB) that the forward's items may be cut into along
// the keys: 0 where the items may occupy the SMs twice already (304: two for each
// of this chip's 152, as a number since sizes are asked for without a device
// too), or where the keys are too few to gain more than the second kernel costs.
int fwd_max_parts(const FwdShape& f, int64_t Tq, int64_t Tk, int64_t n_seq) {
  constexpr int64_t PARTS = 512, LEAST = 14 * coda::ATTN_BLK;
  return Tk < LEAST || (Tq / f.q_span + n_seq) * f.per > 304 ? 0 : PARTS;
}

// Padded rows of the backward's per-row values (see AttnBwdArgs).
int64_t padded_rows(int64_t Tq, int64_t n_seq) { return (Tq / coda::ATTN_BLK + n_seq + 1) * coda::ATTN_BLK; }

// Bound on the parts (of 128 KB) that the backward's key-tile items may be cut
// into: 0 where the tiles alone already occupy the SMs more than once.
int bwd_max_parts(int64_t Tk, int64_t n_seq, int n_q, int n_kv) {
  constexpr int64_t PARTS = 512;
  const int64_t least = Tk / coda::ATTN_BLK * n_kv, most = (Tk / coda::ATTN_BLK + n_seq) * n_kv * (n_q / n_kv);
  return n_q == n_kv || least * 2 > PARTS ? 0 : static_cast<int>(std::min(PARTS, most));
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

// The cache's shape; CODA_OK or the error to return.
int check_cache(coda::KvCache& c, const uint8_t* codes, const uint8_t* sf, const float* scale, int64_t num_pages,
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

int check_ws(const void* ws, size_t have, size_t need) {
  if (!ws || have < need) return CODA_ERR_WORKSPACE;
  return al16(ws) ? CODA_OK : CODA_ERR_ALIGNMENT;
}

struct DecodeLayout {
  int* units;
  float* part;
  float* part_lse;
};
void lay_decode(Cursor& c, DecodeLayout& l, int64_t batch, int group) {
  const int heads = std::min(group, coda::DEC_HEADS);
  l.units = c.take<int>(batch + 2);
  l.part = c.take<float>(int64_t(2) * coda::DEC_MAX_CTAS * heads * coda::ATTN_D);
  l.part_lse = c.take<float>(int64_t(2) * coda::DEC_MAX_CTAS * heads);
}

const __nv_bfloat16* B(const coda_bf16* p) { return reinterpret_cast<const __nv_bfloat16*>(p); }
__nv_bfloat16* B(coda_bf16* p) { return reinterpret_cast<__nv_bfloat16*>(p); }

}  // namespace

extern "C" {

size_t coda_attention_workspace_size(int64_t Tq, int64_t Tk, int64_t n_seq, int32_t n_q, int32_t n_kv,
                                     int32_t head_dim) {
  if (check_shape(Tq, Tk, n_seq, n_q, n_kv, head_dim, 1.f) != CODA_OK) return HEADER;
  Cursor c{nullptr};
  PlanLayout l{};
  const FwdShape f = fwd_shape(Tq, n_seq, n_q, n_q / n_kv);
  const int parts = fwd_max_parts(f, Tq, Tk, n_seq);
  lay_plan(c, l, Tq, Tk, n_seq, f.q_span, false, parts / f.per);
  c.take<float>(parts * PART_FLOATS);
  c.take<float>(parts * 2 * coda::ATTN_BLK);
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
  const FwdShape f = fwd_shape(Tq, n_seq, n_q, n_q / n_kv);
  const int parts = fwd_max_parts(f, Tq, Tk, n_seq);
  Cursor c{static_cast<uint8_t*>(ws)};
  PlanLayout l{};
  lay_plan(c, l, Tq, Tk, n_seq, f.q_span, false, parts / f.per);
  l.a.max_q_parts = parts;
  l.a.q_items = f.per;
  l.a.sms = sms;
  l.a.cu_q = cu_q;
  l.a.cu_k = cu_k;
  l.a.n_seq = static_cast<int>(n_seq);
  l.a.Tq = Tq;
  l.a.Tk = Tk;
  l.a.status = static_cast<int*>(ws);
  CUtensorMap maps[3];
  const uint64_t dims[3] = {static_cast<uint64_t>(head_dim), static_cast<uint64_t>(n_q), static_cast<uint64_t>(Tq)};
  const uint64_t st[2] = {static_cast<uint64_t>(head_dim) * 2, static_cast<uint64_t>(ldq) * 2};
  const uint32_t box[3] = {64, 1u << f.head_shift, static_cast<uint32_t>(f.span)};
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
  a.group = n_q / n_kv;
  a.head_shift = f.head_shift;
  a.pair_heads = f.pair_heads;
  a.part = parts ? c.take<float>(parts * PART_FLOATS) : nullptr;
  a.part_lse = parts ? c.take<float>(parts * 2 * coda::ATTN_BLK) : nullptr;
  a.cuts = l.a.plan.cuts;
  a.scale = scale;
  a.scale_log2 = static_cast<float>(scale * LOG2E);
  a.status = static_cast<int*>(ws);
  a.timeout_ns = WAIT_LIMIT_NS;
  CU(coda::launch_attn_plan(l.a, s));
  CU(coda::launch_attn_fwd(a, maps, l.max_q_tiles * f.per + parts, sms, s));
  return CODA_OK;
}

size_t coda_attention_bwd_workspace_size(int64_t Tq, int64_t Tk, int64_t n_seq, int32_t n_q, int32_t n_kv,
                                         int32_t head_dim) {
  if (check_shape(Tq, Tk, n_seq, n_q, n_kv, head_dim, 1.f) != CODA_OK) return HEADER;
  Cursor c{nullptr};
  PlanLayout l{};
  lay_plan(c, l, Tq, Tk, n_seq, coda::ATTN_BLK, true, bwd_max_parts(Tk, n_seq, n_q, n_kv) / n_kv);
  c.take<float>(2 * n_q * padded_rows(Tq, n_seq));
  c.take<float>(bwd_max_parts(Tk, n_seq, n_q, n_kv) * PART_FLOATS);
  return c.off;
}

int coda_attention_bwd(const coda_bf16* dO, const coda_bf16* Q, int64_t ldq, const coda_bf16* K, int64_t ldk,
                       const coda_bf16* V, int64_t ldv, const coda_bf16* O, const float* lse, const int32_t* cu_q,
                       const int32_t* cu_k, int64_t n_seq, int32_t n_q, int32_t n_kv, int32_t head_dim, float scale,
                       coda_bf16* dQ, coda_bf16* dK, coda_bf16* dV, int64_t Tq, int64_t Tk, void* ws, size_t ws_bytes,
                       coda_stream stream) {
  CK(check_shape(Tq, Tk, n_seq, n_q, n_kv, head_dim, scale));
  if ((Tq == 0 && Tk == 0) || n_seq == 0) return CODA_OK;
  if (!cu_q || (Tq > 0 && (!Q || !dO || !O || !lse || !dQ)) || (Tk > 0 && (!K || !V || !dK || !dV)))
    return CODA_ERR_INVALID_ARG;
  if (!cu_k) cu_k = cu_q;
  if (cu_k == cu_q && Tk != Tq) return CODA_ERR_INVALID_ARG;
  const int64_t wq = int64_t(n_q) * head_dim, wk = int64_t(n_kv) * head_dim;
  if (ldq < wq || ldk < wk || ldv < wk) return CODA_ERR_INVALID_ARG;
  if (!al16(Q) || !al16(K) || !al16(V) || !al16(O) || !al16(dO) || !al16(dQ) || !al16(dK) || !al16(dV) || !al4(lse) ||
      !al4(cu_q) || !al4(cu_k) || ldq % 8 || ldk % 8 || ldv % 8)
    return CODA_ERR_ALIGNMENT;
  CK(check_ws(ws, ws_bytes, coda_attention_bwd_workspace_size(Tq, Tk, n_seq, n_q, n_kv, head_dim)));
  const int sms = coda::device_sms();
  if (sms <= 0 || !coda::tensor_map_encoder()) return CODA_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  Cursor c{static_cast<uint8_t*>(ws)};
  PlanLayout l{};
  lay_plan(c, l, Tq, Tk, n_seq, coda::ATTN_BLK, true, bwd_max_parts(Tk, n_seq, n_q, n_kv) / n_kv);
  l.a.cu_q = cu_q;
  l.a.cu_k = cu_k;
  l.a.n_seq = static_cast<int>(n_seq);
  l.a.Tq = Tq;
  l.a.Tk = Tk;
  l.a.status = static_cast<int*>(ws);
  coda::AttnBwdArgs a{};
  a.Tp = padded_rows(Tq, n_seq);
  a.nlse2 = c.take<float>(2 * n_q * a.Tp);
  a.ndelta = a.nlse2 + n_q * a.Tp;
  a.max_parts = bwd_max_parts(Tk, n_seq, n_q, n_kv);
  a.part = c.take<float>(a.max_parts * PART_FLOATS);
  l.a.n_kv = n_kv;
  l.a.group = n_q / n_kv;
  l.a.max_parts = a.max_parts;
  for (int p = 2; p <= std::min(l.a.group, 32); ++p)
    if (l.a.group % p == 0) l.a.divisors |= 1u << (p - 1);
  l.a.sms = sms;
  a.counts = l.a.plan.counts;
  a.q_tiles = l.a.plan.q_tiles;
  a.k_tiles = l.a.plan.k_tiles;
  a.cuts = l.a.plan.cuts;
  a.lse = lse;
  a.dQ = B(dQ);
  a.dK = B(dK);
  a.dV = B(dV);
  a.Tq = Tq;
  a.Tk = Tk;
  a.n_q = n_q;
  a.n_kv = n_kv;
  a.group = n_q / n_kv;
  a.scale = scale;
  a.scale_log2 = static_cast<float>(scale * LOG2E);
  a.status = static_cast<int*>(ws);
  a.timeout_ns = WAIT_LIMIT_NS;
  CUtensorMap maps[5];
  if (Tq > 0 && (!map_rows(&maps[0], Q, Tq, wq, ldq) || !map_rows(&maps[3], dO, Tq, wq, wq) ||
                 !map_rows(&maps[4], O, Tq, wq, wq)))
    return CODA_ERR_CUDA;
  if (Tk > 0 && (!map_rows(&maps[1], K, Tk, wk, ldk) || !map_rows(&maps[2], V, Tk, wk, ldv))) return CODA_ERR_CUDA;
  // without queries (keys) no tile of them is ever loaded
  if (Tq == 0) maps[0] = maps[3] = maps[4] = maps[1];
  if (Tk == 0) maps[1] = maps[2] = maps[0];
  CU(coda::launch_attn_plan(l.a, s));
  CU(coda::launch_attn_bwd(a, maps, Tq > 0 ? l.max_q_tiles : 0, Tk > 0 ? l.max_k_tiles : 0, sms, s));
  return CODA_OK;
}

int coda_kv_append_nvfp4(const coda_bf16* K, int64_t ldk, const coda_bf16* V, int64_t ldv, const int32_t* slots,
                         int64_t T, uint8_t* codes, uint8_t* sf, float* scale, int64_t num_pages, int32_t page_size,
                         int32_t n_kv, int32_t head_dim, void* ws, size_t ws_bytes, coda_stream stream) {
  if (T < 0) return CODA_ERR_INVALID_ARG;
  coda::KvCache c{};
  CK(check_cache(c, codes, sf, scale, num_pages, page_size, n_kv, head_dim));
  if (T >= (int64_t(1) << 30) / n_kv) return CODA_ERR_UNSUPPORTED;  // rows are counted in 32 bits
  if (T == 0) return CODA_OK;
  if (!K || !V || !slots || ldk < int64_t(n_kv) * head_dim || ldv < int64_t(n_kv) * head_dim)
    return CODA_ERR_INVALID_ARG;
  if (!al16(K) || !al16(V) || !al4(slots) || ldk % 8 || ldv % 8) return CODA_ERR_ALIGNMENT;
  CK(check_ws(ws, ws_bytes, HEADER));
  CU(coda::launch_kv_append(c, B(K), ldk, B(V), ldv, slots, static_cast<int>(T * 2 * n_kv), static_cast<int*>(ws),
                            static_cast<cudaStream_t>(stream)));
  return CODA_OK;
}

int coda_kv_read_nvfp4(const uint8_t* codes, const uint8_t* sf, const float* scale, int64_t num_pages,
                       int32_t page_size, const int32_t* slots, int64_t T, int32_t n_kv, int32_t head_dim, void* K,
                       void* V, int dtype, void* ws, size_t ws_bytes, coda_stream stream) {
  if (T < 0 || (dtype != CODA_BF16 && dtype != CODA_F32)) return CODA_ERR_INVALID_ARG;
  coda::KvCache c{};
  CK(check_cache(c, codes, sf, scale, num_pages, page_size, n_kv, head_dim));
  if (T >= (int64_t(1) << 30) / n_kv) return CODA_ERR_UNSUPPORTED;  // rows are counted in 32 bits
  if (T == 0) return CODA_OK;
  if (!K || !V || !slots) return CODA_ERR_INVALID_ARG;
  if (!al16(K) || !al16(V) || !al4(slots)) return CODA_ERR_ALIGNMENT;
  CK(check_ws(ws, ws_bytes, HEADER));
  CU(coda::launch_kv_read(c, slots, static_cast<int>(T * 2 * n_kv), K, V, dtype == CODA_F32, static_cast<int*>(ws),
                          static_cast<cudaStream_t>(stream)));
  return CODA_OK;
}

size_t coda_attention_decode_nvfp4_workspace_size(int64_t batch, int32_t n_q, int32_t n_kv, int32_t head_dim) {
  if (check_shape(batch, batch, batch, n_q, n_kv, head_dim, 1.f) != CODA_OK) return HEADER;
  Cursor c{nullptr};
  DecodeLayout l{};
  lay_decode(c, l, batch, n_q / n_kv);
  return c.off;
}

int coda_attention_decode_nvfp4(const coda_bf16* Q, int64_t ldq, const uint8_t* codes, const uint8_t* sf,
                                const float* scale, int64_t num_pages, int32_t page_size, const int32_t* block_table,
                                int64_t max_pages, const int32_t* seq_lens, int64_t batch, int32_t n_q, int32_t n_kv,
                                int32_t head_dim, float softmax_scale, coda_bf16* O, float* lse, void* ws,
                                size_t ws_bytes, coda_stream stream) {
  CK(check_shape(batch, batch, batch, n_q, n_kv, head_dim, softmax_scale));
  if (max_pages < 0) return CODA_ERR_INVALID_ARG;
  coda::DecodeArgs a{};
  CK(check_cache(a.c, codes, sf, scale, num_pages, page_size, n_kv, head_dim));
  if (batch == 0) return CODA_OK;
  if (!Q || !seq_lens || !O || !lse || (max_pages > 0 && !block_table) || ldq < int64_t(n_q) * head_dim)
    return CODA_ERR_INVALID_ARG;
  if (!al16(Q) || !al16(O) || !al4(lse) || !al4(block_table) || !al4(seq_lens) || ldq % 8) return CODA_ERR_ALIGNMENT;
  a.group = n_q / n_kv;
  a.splits = (a.group + coda::DEC_HEADS - 1) / coda::DEC_HEADS;
  // key positions and work units are 32-bit on the device
  const int64_t longest = max_pages * page_size;
  if (max_pages >= (int64_t(1) << 31) || longest >= (int64_t(1) << 31) - 256 ||
      batch * ((longest + 383) / 128) * n_kv * a.splits >= (int64_t(1) << 31) - 65536)
    return CODA_ERR_UNSUPPORTED;
  CK(check_ws(ws, ws_bytes, coda_attention_decode_nvfp4_workspace_size(batch, n_q, n_kv, head_dim)));
  const int sms = coda::device_sms();
  if (sms <= 0) return CODA_ERR_CUDA;
  Cursor cur{static_cast<uint8_t*>(ws)};
  DecodeLayout l{};
  lay_decode(cur, l, batch, a.group);
  a.Q = B(Q);
  a.ldq = ldq;
  a.table = block_table;
  a.max_pages = static_cast<int>(max_pages);
  a.seq_lens = seq_lens;
  a.B = static_cast<int>(batch);
  a.n_q = n_q;
  a.scale_log2 = static_cast<float>(softmax_scale * LOG2E);
  a.O = B(O);
  a.lse = lse;
  a.units = l.units;
  a.part = l.part;
  a.part_lse = l.part_lse;
  a.part_heads = std::min(a.group, coda::DEC_HEADS);
  a.status = static_cast<int*>(ws);
  CU(coda::launch_attn_decode(a, sms, static_cast<cudaStream_t>(stream)));
  return CODA_OK;
}

}  // extern "C"

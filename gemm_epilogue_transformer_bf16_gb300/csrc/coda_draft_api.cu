// Host side of the rotary and drafting operators declared in include/coda.h:
// argument checks and launches.
#include "coda_attn_host.h"
#include "coda_attn_tree.cuh"
#include "coda_internal.h"
#include "coda_rope.cuh"
#include "coda_verify.cuh"

namespace {

// Table and heads of a rotation; CODA_OK or the error to return.
int check_rope(const int32_t* pos, const float* cs, int32_t max_pos, int32_t rotary_dim, int32_t head_dim, int pairing) {
  if (max_pos <= 0 || rotary_dim <= 0 || (pairing != CODA_ROPE_INTERLEAVED && pairing != CODA_ROPE_HALF))
    return CODA_ERR_INVALID_ARG;
  if (head_dim != coda::ATTN_D || rotary_dim > head_dim || rotary_dim % 16) return CODA_ERR_UNSUPPORTED;
  if (!pos || !cs) return CODA_ERR_INVALID_ARG;
  return al16(cs) && al4(pos) ? CODA_OK : CODA_ERR_ALIGNMENT;
}

int rope(const coda_bf16* X, int64_t ldx, const int32_t* pos, const float* cs, int32_t max_pos, int32_t rotary_dim,
         int pairing, bool back, coda_bf16* Y, int64_t ldy, int64_t T, int32_t n_heads, int32_t head_dim, void* ws,
         size_t ws_bytes, coda_stream stream) {
  if (T < 0 || n_heads <= 0) return CODA_ERR_INVALID_ARG;
  if (T >= (int64_t(1) << 30) / n_heads) return CODA_ERR_UNSUPPORTED;  // heads are counted in 32 bits
  if (T == 0) return CODA_OK;
  CK(check_rope(pos, cs, max_pos, rotary_dim, head_dim, pairing));
  const int64_t w = int64_t(n_heads) * head_dim;
  if (!X || !Y || ldx < w || ldy < w || (X == Y && ldx != ldy)) return CODA_ERR_INVALID_ARG;
  if (!al16(X) || !al16(Y) || ldx % 8 || ldy % 8) return CODA_ERR_ALIGNMENT;
  CK(check_ws(ws, ws_bytes, HEADER));
  const coda::RopeArgs a{B(X), ldx, B(Y), ldy, pos, cs, max_pos, rotary_dim, static_cast<int>(T), n_heads,
                         static_cast<int*>(ws)};
  CU(coda::launch_rope(a, pairing == CODA_ROPE_HALF, back, static_cast<cudaStream_t>(stream)));
  return CODA_OK;
}

// A row for each node and head of a group, up to a tile's.
void lay_tree(Cursor& c, coda::TreeArgs& a, int64_t T, int64_t batch, int group) {
  a.part_rows = static_cast<int>(std::min<int64_t>(coda::TREE_ROWS, T * group));
  a.places = c.take<int64_t>(batch + 2);
  a.seen = c.take<uint32_t>(int64_t(coda::TREE_MAX_CTAS) * coda::TREE_MAX_NODES * (coda::TREE_ROWS / 32));
  a.part = c.take<float>(int64_t(2) * coda::TREE_MAX_CTAS * a.part_rows * coda::ATTN_D);
  a.part_lse = c.take<float>(int64_t(2) * coda::TREE_MAX_CTAS * a.part_rows);
}

}  // namespace

extern "C" {

int coda_rope_table_scaled(float theta, int32_t rotary_dim, int32_t max_pos, int kind, float factor, float original,
                           float low, float high, float amplitude, float* cos_sin, coda_stream stream) {
  if (rotary_dim <= 0 || rotary_dim % 2 || max_pos <= 0 || !(theta > 0.f) || !std::isfinite(theta)) return CODA_ERR_INVALID_ARG;
  if (kind < CODA_ROPE_PLAIN || kind > CODA_ROPE_RAMP || !std::isfinite(amplitude)) return CODA_ERR_INVALID_ARG;
  if (kind != CODA_ROPE_PLAIN && (!(factor > 0.f) || !std::isfinite(factor))) return CODA_ERR_INVALID_ARG;
  if (kind >= CODA_ROPE_BANDS &&
      (!(original > 0.f) || !std::isfinite(original) || !(low > 0.f) || !(high > low) || !std::isfinite(high)))
    return CODA_ERR_INVALID_ARG;
  if (kind == CODA_ROPE_RAMP && !(theta > 1.f)) return CODA_ERR_INVALID_ARG;
  if (!cos_sin) return CODA_ERR_INVALID_ARG;
  if (!al16(cos_sin)) return CODA_ERR_ALIGNMENT;
  const coda::RopeTableArgs a{theta, factor, low, high, amplitude, original, rotary_dim, max_pos, kind,
                              reinterpret_cast<float2*>(cos_sin)};
  CU(coda::launch_rope_table_scaled(a, static_cast<cudaStream_t>(stream)));
  return CODA_OK;
}

int coda_rope(const coda_bf16* X, int64_t ldx, const int32_t* pos, const float* cos_sin, int32_t max_pos,
              int32_t rotary_dim, int pairing, coda_bf16* Y, int64_t ldy, int64_t T, int32_t n_heads, int32_t head_dim,
              void* ws, size_t ws_bytes, coda_stream stream) {
  return rope(X, ldx, pos, cos_sin, max_pos, rotary_dim, pairing, false, Y, ldy, T, n_heads, head_dim, ws, ws_bytes, stream);
}

int coda_rope_bwd(const coda_bf16* dY, int64_t lddy, const int32_t* pos, const float* cos_sin, int32_t max_pos,
                  int32_t rotary_dim, int pairing, coda_bf16* dX, int64_t lddx, int64_t T, int32_t n_heads,
                  int32_t head_dim, void* ws, size_t ws_bytes, coda_stream stream) {
  return rope(dY, lddy, pos, cos_sin, max_pos, rotary_dim, pairing, true, dX, lddx, T, n_heads, head_dim, ws, ws_bytes,
              stream);
}

int coda_kv_append_rope_nvfp4(const coda_bf16* Q, int64_t ldq, const coda_bf16* K, int64_t ldk, const coda_bf16* V,
                              int64_t ldv, const int32_t* slots, const int32_t* pos, const float* cos_sin,
                              int32_t max_pos, int32_t rotary_dim, int pairing, coda_bf16* Q_out, coda_bf16* K_out,
                              int64_t T, uint8_t* codes, uint8_t* sf, float* scale, int64_t num_pages, int32_t page_size,
                              int32_t n_q, int32_t n_kv, int32_t head_dim, void* ws, size_t ws_bytes,
                              coda_stream stream) {
  if (T < 0 || n_q < 0) return CODA_ERR_INVALID_ARG;
  coda::AppendRopeArgs a{};
  CK(check_cache(a.c, codes, sf, scale, num_pages, page_size, n_kv, head_dim));
  if (n_q >= 65536 || T >= (int64_t(1) << 30) / std::max(n_q, n_kv)) return CODA_ERR_UNSUPPORTED;  // 32-bit counts
  if (T == 0) return CODA_OK;
  CK(check_rope(pos, cos_sin, max_pos, rotary_dim, head_dim, pairing));
  const int64_t wq = int64_t(n_q) * head_dim, wk = int64_t(n_kv) * head_dim;
  if (!K || !V || !slots || ldk < wk || ldv < wk || (n_q > 0 && (!Q || !Q_out || ldq < wq))) return CODA_ERR_INVALID_ARG;
  if (!al16(Q) || !al16(K) || !al16(V) || !al16(Q_out) || !al16(K_out) || !al4(slots) || ldk % 8 || ldv % 8 ||
      (n_q > 0 && ldq % 8))
    return CODA_ERR_ALIGNMENT;
  CK(check_ws(ws, ws_bytes, HEADER));
  a.K = B(K);
  a.V = B(V);
  a.ldk = ldk;
  a.ldv = ldv;
  a.slots = slots;
  a.K_out = B(K_out);
  a.q = coda::RopeArgs{B(Q), ldq, B(Q_out), wq, pos, cos_sin, max_pos, rotary_dim, static_cast<int>(T), n_q,
                       static_cast<int*>(ws)};
  CU(coda::launch_kv_append_rope(a, pairing == CODA_ROPE_HALF, static_cast<cudaStream_t>(stream)));
  return CODA_OK;
}

int coda_kv_accept_nvfp4(uint8_t* codes, uint8_t* sf, float* scale, int64_t num_pages, int32_t page_size,
                         const int32_t* block_table, int64_t max_pages, const int32_t* seq_lens, const int32_t* cu,
                         const int32_t* nodes, int64_t width, const int32_t* count, int64_t batch,
                         int32_t n_kv, int32_t head_dim, int32_t* new_lens, void* ws, size_t ws_bytes,
                         coda_stream stream) {
  if (batch < 0 || width < 1 || max_pages < 0) return CODA_ERR_INVALID_ARG;
  coda::AcceptArgs a{};
  CK(check_cache(a.c, codes, sf, scale, num_pages, page_size, n_kv, head_dim));
  if (batch >= (int64_t(1) << 29) / n_kv || width >= (int64_t(1) << 30) ||
      max_pages >= (int64_t(1) << 31) || max_pages * page_size >= (int64_t(1) << 31))
    return CODA_ERR_UNSUPPORTED;
  if (batch == 0) return CODA_OK;
  if (!seq_lens || !cu || !nodes || !count || !new_lens || (max_pages > 0 && !block_table)) return CODA_ERR_INVALID_ARG;
  if (new_lens == seq_lens) return CODA_ERR_INVALID_ARG;  // other heads still read the old lengths
  if (!al4(block_table) || !al4(seq_lens) || !al4(cu) || !al4(nodes) || !al4(count) || !al4(new_lens))
    return CODA_ERR_ALIGNMENT;
  CK(check_ws(ws, ws_bytes, HEADER));
  a.table = block_table;
  a.max_pages = static_cast<int>(max_pages);
  a.seq_lens = seq_lens;
  a.cu = cu;
  a.nodes = nodes;
  a.count = count;
  a.B = static_cast<int>(batch);
  a.width = static_cast<int>(width);
  a.out_lens = new_lens;
  a.status = static_cast<int*>(ws);
  CU(coda::launch_kv_accept(a, static_cast<cudaStream_t>(stream)));
  return CODA_OK;
}

size_t coda_attention_tree_nvfp4_workspace_size(int64_t T, int64_t batch, int32_t n_q, int32_t n_kv, int32_t head_dim) {
  if (check_shape(T, T, batch, n_q, n_kv, head_dim, 1.f) != CODA_OK) return HEADER;
  Cursor c{nullptr};
  coda::TreeArgs a{};
  lay_tree(c, a, T, batch, n_q / n_kv);
  return c.off;
}

int coda_attention_tree_nvfp4(const coda_bf16* Q, int64_t ldq, const uint8_t* codes, const uint8_t* sf,
                              const float* scale, int64_t num_pages, int32_t page_size, const int32_t* block_table,
                              int64_t max_pages, const int32_t* seq_lens, const int32_t* cu, const int32_t* parents,
                              int64_t T, int64_t batch, int32_t n_q, int32_t n_kv, int32_t head_dim, float softmax_scale,
                              coda_bf16* O, float* lse, void* ws, size_t ws_bytes, coda_stream stream) {
  CK(check_shape(T, T, batch, n_q, n_kv, head_dim, softmax_scale));
  if (max_pages < 0) return CODA_ERR_INVALID_ARG;
  coda::TreeArgs a{};
  CK(check_cache(a.c, codes, sf, scale, num_pages, page_size, n_kv, head_dim));
  if (T == 0 || batch == 0) return CODA_OK;
  if (!Q || !seq_lens || !cu || !O || !lse || (max_pages > 0 && !block_table) || ldq < int64_t(n_q) * head_dim)
    return CODA_ERR_INVALID_ARG;
  if (!al16(Q) || !al16(O) || !al4(lse) || !al4(block_table) || !al4(seq_lens) || !al4(cu) || !al4(parents) || ldq % 8)
    return CODA_ERR_ALIGNMENT;
  if (max_pages >= (int64_t(1) << 31) || max_pages * page_size >= (int64_t(1) << 31) - 256) return CODA_ERR_UNSUPPORTED;
  CK(check_ws(ws, ws_bytes, coda_attention_tree_nvfp4_workspace_size(T, batch, n_q, n_kv, head_dim)));
  const int sms = coda::device_sms();
  if (sms <= 0 || !coda::tensor_map_encoder()) return CODA_ERR_CUDA;
  CUtensorMap maps[3] = {};
  if (num_pages > 0 && !coda::cache_maps(maps, a.c)) return CODA_ERR_CUDA;  // without pages nothing is ever loaded
  Cursor cur{static_cast<uint8_t*>(ws)};
  lay_tree(cur, a, T, batch, n_q / n_kv);
  a.Q = B(Q);
  a.ldq = ldq;
  a.table = block_table;
  a.max_pages = static_cast<int>(max_pages);
  a.seq_lens = seq_lens;
  a.cu = cu;
  a.parents = parents;
  a.T = static_cast<int>(T);
  a.B = static_cast<int>(batch);
  a.n_q = n_q;
  a.group = n_q / n_kv;
  a.scale_log2 = static_cast<float>(softmax_scale * LOG2E);
  a.O = B(O);
  a.lse = lse;
  a.status = static_cast<int*>(ws);
  CU(coda::launch_attn_tree(a, maps, sms, static_cast<cudaStream_t>(stream)));
  return CODA_OK;
}

size_t coda_verify_drafts_workspace_size(int64_t, int64_t, int64_t) { return HEADER; }

int coda_verify_drafts(const void* probs, const void* draft_probs, int dtype, int64_t V, const int32_t* tokens,
                       const int32_t* cu, const int32_t* parents, const float* u, const float* u_next, int64_t T,
                       int64_t batch, int64_t width, int32_t* count, int32_t* nodes, int32_t* out_tokens, void* ws,
                       size_t ws_bytes, coda_stream stream) {
  if (T < 0 || batch < 0 || V < 1 || width < 1 || (dtype != CODA_BF16 && dtype != CODA_F32)) return CODA_ERR_INVALID_ARG;
  if (V >= (int64_t(1) << 30) || T >= (int64_t(1) << 30) || batch >= (int64_t(1) << 27) || width >= (int64_t(1) << 30))
    return CODA_ERR_UNSUPPORTED;
  if (batch == 0) return CODA_OK;
  if (!cu || !u_next || !count || !nodes || !out_tokens || (T > 0 && (!probs || !tokens || !u)))
    return CODA_ERR_INVALID_ARG;
  if (!al16(probs) || !al16(draft_probs) || !al4(tokens) || !al4(cu) || !al4(parents) || !al4(u) || !al4(u_next) ||
      !al4(count) || !al4(nodes) || !al4(out_tokens))
    return CODA_ERR_ALIGNMENT;
  CK(check_ws(ws, ws_bytes, coda_verify_drafts_workspace_size(T, batch, V)));
  coda::VerifyArgs a{probs, draft_probs, tokens, cu, parents, u, u_next, count, nodes, out_tokens, V,
                     static_cast<int>(T), static_cast<int>(batch), static_cast<int>(width), 0, static_cast<int*>(ws)};
  CU(coda::launch_verify(a, dtype == CODA_F32, static_cast<cudaStream_t>(stream)));
  return CODA_OK;
}

}  // extern "C"

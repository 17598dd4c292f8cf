// Rotary positions: the pieces that the rotation of whole tensors and the append
// to the cache share, and the launchers.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "coda_kvcache.cuh"
#include "coda_ptx.cuh"

namespace coda {

struct RopeArgs {
  const __nv_bfloat16* X;
  int64_t ldx;
  __nv_bfloat16* Y;
  int64_t ldy;
  const int32_t* pos;
  const float* cs;  // [max_pos, rotary / 2, 2]
  int max_pos, rotary;
  int tokens, heads;
  int* status;
};
// back: the transposed rotation.  half: pairs (j, j + rotary / 2).
cudaError_t launch_rope(const RopeArgs& a, bool half, bool back, cudaStream_t s);

struct AppendRopeArgs {
  KvCache c;
  const __nv_bfloat16 *K, *V;
  int64_t ldk, ldv;
  const int32_t* slots;
  RopeArgs q;             // the query heads (heads 0: none) and what they share with the keys
  __nv_bfloat16* K_out;   // [tokens, n_kv * 128] rotated keys, or null
};
cudaError_t launch_kv_append_rope(const AppendRopeArgs& a, bool half, cudaStream_t s);

// A table whose frequencies are scaled for longer contexts: f_j = theta^(-2j / d)
// becomes f_j (g_j + (1 - g_j) / factor).
struct RopeTableArgs {
  double theta, factor, low, high, amplitude, original;
  int rotary, max_pos, kind;  // kind: CODA_ROPE_PLAIN ...
  float2* cs;
};
cudaError_t launch_rope_table_scaled(const RopeTableArgs& a, cudaStream_t s);

#ifdef __CUDACC__
// Position of token t, clamped to the table (the status tells).
__device__ __forceinline__ int rope_position(const RopeArgs& a, int t, bool tell) {
  int p = a.pos[t];
  if (p < 0 || p >= a.max_pos) {
    if (tell) atomicOr(a.status, CODA_DEV_POSITION_RANGE);
    p = p < 0 ? 0 : a.max_pos - 1;
  }
  return p;
}

// y1 = x1 c - x2 s, y2 = x2 c + x1 s: two products and a sum, each rounded to
// fp32 on its own, so that keys quantised here agree bit for bit with any other
// evaluation in that order.
__device__ __forceinline__ void rope_pair(float& x1, float& x2, float c, float s) {
  const float y1 = __fsub_rn(__fmul_rn(x1, c), __fmul_rn(x2, s));
  x2 = __fadd_rn(__fmul_rn(x2, c), __fmul_rn(x1, s));
  x1 = y1;
}

// A warp's share of one token: HEADS heads from h0 on.  Eight lanes per head,
// sixteen elements each: two runs of eight (16 bytes) that hold eight whole
// pairs, the same ones in every head, so that a lane reads its cosines and
// sines once.  Rows may be rotated in place: a lane writes what it has read.
template <bool HALF, bool BACK, int HEADS>
__device__ __forceinline__ void rope_heads(const RopeArgs& a, int t, int h0, int lane) {
  const int u = lane & 7, n = a.rotary >> 4;
  const bool turn = u < n;
  const int lo = HALF && turn ? 8 * u : 16 * u, hi = HALF && turn ? a.rotary / 2 + 8 * u : 16 * u + 8;
  const __nv_bfloat16* x = a.X + t * a.ldx;
  __nv_bfloat16* y = a.Y + t * a.ldy;
  constexpr int N = HEADS / 4;
  uint4 v[N][2];
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int h = h0 + 4 * i + (lane >> 3);
    if (h < a.heads) {
      v[i][0] = *reinterpret_cast<const uint4*>(x + h * 128 + lo);
      v[i][1] = *reinterpret_cast<const uint4*>(x + h * 128 + hi);
    }
  }
  float4 cs[4];
  const int p = rope_position(a, t, h0 == 0 && lane == 0);
#pragma unroll
  for (int i = 0; i < 4; ++i) cs[i] = make_float4(1.f, 0.f, 1.f, 0.f);
  if (turn) {
    const float4* at = reinterpret_cast<const float4*>(a.cs + static_cast<int64_t>(p) * a.rotary) + 4 * u;
#pragma unroll
    for (int i = 0; i < 4; ++i) cs[i] = at[i];
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int h = h0 + 4 * i + (lane >> 3);
    if (h >= a.heads) continue;
    if (turn) {
      float f[16];
      bf16x8_to_f32(v[i][0], f);
      bf16x8_to_f32(v[i][1], f + 8);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float c = j & 1 ? cs[j >> 1].z : cs[j >> 1].x;
        float s = j & 1 ? cs[j >> 1].w : cs[j >> 1].y;
        if (BACK) s = -s;
        if (HALF)
          rope_pair(f[j], f[j + 8], c, s);
        else
          rope_pair(f[2 * j], f[2 * j + 1], c, s);
      }
      store_bf16x8(y + h * 128 + lo, f);
      store_bf16x8(y + h * 128 + hi, f + 8);
    } else {
      *reinterpret_cast<uint4*>(y + h * 128 + lo) = v[i][0];
      *reinterpret_cast<uint4*>(y + h * 128 + hi) = v[i][1];
    }
  }
}
#endif

}  // namespace coda

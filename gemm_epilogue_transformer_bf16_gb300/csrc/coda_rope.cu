// Rotary positions of whole tensors (forward and gradient), tables scaled for
// long contexts, and the append to the 4-bit cache that rotates on the way.
#include <algorithm>

#include "coda.h"
#include "coda_attn.cuh"
#include "coda_internal.h"
#include "coda_kvrow.cuh"
#include "coda_status.h"
#include "coda_rope.cuh"

namespace coda {
namespace {

constexpr int ROPE_HEADS = 12;  // heads per warp

// Y = R(pos) X per head (BACK: the transposed rotation, which is the gradient).
// HBM-bound: 4 bytes per element.
template <bool HALF, bool BACK>
__global__ void __launch_bounds__(256) rope_kernel(const RopeArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const int groups = (a.heads + ROPE_HEADS - 1) / ROPE_HEADS;
  const int w = static_cast<int>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  const int t = w / groups;
  if (t >= a.tokens) return;
  rope_heads<HALF, BACK, ROPE_HEADS>(a, t, (w - t * groups) * ROPE_HEADS, threadIdx.x & 31);
}

// Keys rotated, keys and values quantised as kv_append_kernel does (the
// rotated keys in fp32, not rounded to bf16 in between), queries rotated:
// the first blocks take the cache rows, eight lanes each, the others the
// queries.  A lane's sixteen elements of a key are one block of the cache's
// format, so in the half-split pairing the other element of each pair is read
// a second time.
template <bool HALF>
__global__ void __launch_bounds__(256) kv_append_rope_kernel(const AppendRopeArgs a, int kv_blocks) {
  griddep_wait();
  griddep_launch_dependents();
  const KvCache& c = a.c;
  if (static_cast<int>(blockIdx.x) >= kv_blocks) {
    const int groups = (a.q.heads + ROPE_HEADS - 1) / ROPE_HEADS;
    const int w = (static_cast<int>(blockIdx.x) - kv_blocks) * 8 + (threadIdx.x >> 5);
    const int t = w / groups;
    if (t < a.q.tokens)
      rope_heads<HALF, false, ROPE_HEADS>(a.q, t, (w - t * groups) * ROPE_HEADS, threadIdx.x & 31);
    return;
  }
  const int sub = threadIdx.x & 7;
  const int row = blockIdx.x * 32 + (threadIdx.x >> 3);
  float x[16];
  int64_t at = -1;  // cache row, -1: none
  if (row < a.q.tokens * 2 * c.n_kv) {
    const int t = row / (2 * c.n_kv), rest = row - t * 2 * c.n_kv;
    const int plane = rest >= c.n_kv, h = rest - plane * c.n_kv;
    const __nv_bfloat16* src = (plane ? a.V + t * a.ldv : a.K + t * a.ldk) + h * 128;
    load_bf16x8(src + sub * 16, x);
    load_bf16x8(src + sub * 16 + 8, x + 8);
    const int slot = a.slots[t];
    if (slot >= 0) {
      if ((slot >> c.page_shift) < c.num_pages)
        at = cache_row(c, slot >> c.page_shift, plane, h, slot & ((1 << c.page_shift) - 1));
      else if (rest == 0 && sub == 0)
        atomicOr(a.q.status, CODA_DEV_PAGE_RANGE);
    }
    if (plane == 0) {
      const int p = rope_position(a.q, t, rest == 0 && sub == 0);
      const float* cs = a.q.cs + static_cast<int64_t>(p) * a.q.rotary;
      const int halfr = a.q.rotary / 2;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int e = sub * 16 + 8 * i;  // elements e .. e + 7 of the head
        float* y = x + 8 * i;
        if (e >= a.q.rotary) continue;
        if constexpr (HALF) {
          const bool first = e < halfr;
          float z[8];
          load_bf16x8(src + (first ? e + halfr : e - halfr), z);
          const float4* at4 = reinterpret_cast<const float4*>(cs + 2 * (first ? e : e - halfr));
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float4 f = at4[j];
            const float s0 = first ? -f.y : f.y, s1 = first ? -f.w : f.w;
            y[2 * j] = __fadd_rn(__fmul_rn(y[2 * j], f.x), __fmul_rn(z[2 * j], s0));
            y[2 * j + 1] = __fadd_rn(__fmul_rn(y[2 * j + 1], f.z), __fmul_rn(z[2 * j + 1], s1));
          }
        } else {
          const float4* at4 = reinterpret_cast<const float4*>(cs + e);
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const float4 f = at4[j];
            rope_pair(y[4 * j], y[4 * j + 1], f.x, f.y);
            rope_pair(y[4 * j + 2], y[4 * j + 3], f.z, f.w);
          }
        }
      }
      if (a.K_out) {
        __nv_bfloat16* to = a.K_out + (static_cast<int64_t>(t) * c.n_kv + h) * 128 + sub * 16;
        store_bf16x8(to, x);
        store_bf16x8(to + 8, x + 8);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = 0.f;
  }
  uint32_t w[2], sfb;
  float s;
  quantise_row16(x, w, sfb, s);
  if (at >= 0) {
    *reinterpret_cast<uint2*>(c.codes + at * 64 + sub * 8) = make_uint2(w[0], w[1]);
    c.sf[at * 8 + sub] = static_cast<uint8_t>(sfb);
    if (sub == 0) c.scale[at] = s;
  }
}

// Angles in fp64, stored fp32: an angle of a far position loses its fraction in
// fp32.  g_j by the frequency's rotations over the original context (bands) or
// by the pair's number between those of `high` and `low` rotations (ramp).
__global__ void rope_table_scaled_kernel(const RopeTableArgs a) {
  griddep_launch_dependents();
  constexpr double TWO_PI = 6.283185307179586476925286766559;
  const int half = a.rotary / 2;
  const int64_t total = static_cast<int64_t>(a.max_pos) * half;
  double first = 0.0, last = 1.0;
  if (a.kind == CODA_ROPE_RAMP) {
    // the pair number whose frequency makes r rotations over the original context
    const double per = a.rotary / (2.0 * log(a.theta));
    first = fmax(0.0, floor(per * log(a.original / (a.high * TWO_PI))));
    last = fmin(a.rotary - 1.0, ceil(per * log(a.original / (a.low * TWO_PI))));
    if (first == last) last += 0.001;
  }
  for (int64_t i = blockIdx.x * static_cast<int64_t>(blockDim.x) + threadIdx.x; i < total;
       i += static_cast<int64_t>(gridDim.x) * blockDim.x) {
    const int64_t p = i / half;
    const int j = static_cast<int>(i - p * half);
    double f = pow(a.theta, -2.0 * j / a.rotary);
    double g = 1.0;
    if (a.kind == CODA_ROPE_LINEAR) g = 0.0;
    if (a.kind == CODA_ROPE_BANDS) g = (a.original * f / TWO_PI - a.low) / (a.high - a.low);
    if (a.kind == CODA_ROPE_RAMP) g = 1.0 - (j - first) / (last - first);
    g = fmin(1.0, fmax(0.0, g));
    if (a.kind != CODA_ROPE_PLAIN) f = f * (g + (1.0 - g) / a.factor);
    double sn, cn;
    sincos(static_cast<double>(p) * f, &sn, &cn);
    a.cs[i] = make_float2(static_cast<float>(cn * a.amplitude), static_cast<float>(sn * a.amplitude));
  }
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, bool half, bool back, cudaStream_t s) {
  const int64_t warps = static_cast<int64_t>(a.tokens) * ((a.heads + ROPE_HEADS - 1) / ROPE_HEADS);
  const int64_t grid = (warps + 7) / 8;
  if (half)
    return back ? attn_launch(rope_kernel<true, true>, grid, 256, 0, s, a)
                : attn_launch(rope_kernel<true, false>, grid, 256, 0, s, a);
  return back ? attn_launch(rope_kernel<false, true>, grid, 256, 0, s, a)
              : attn_launch(rope_kernel<false, false>, grid, 256, 0, s, a);
}

cudaError_t launch_kv_append_rope(const AppendRopeArgs& a, bool half, cudaStream_t s) {
  const int64_t kv = (static_cast<int64_t>(a.q.tokens) * 2 * a.c.n_kv + 31) / 32;
  const int64_t warps = static_cast<int64_t>(a.q.tokens) * ((a.q.heads + ROPE_HEADS - 1) / ROPE_HEADS);
  const int64_t grid = kv + (warps + 7) / 8;
  return half ? attn_launch(kv_append_rope_kernel<true>, grid, 256, 0, s, a, static_cast<int>(kv))
              : attn_launch(kv_append_rope_kernel<false>, grid, 256, 0, s, a, static_cast<int>(kv));
}

cudaError_t launch_rope_table_scaled(const RopeTableArgs& a, cudaStream_t s) {
  const int64_t total = static_cast<int64_t>(a.max_pos) * (a.rotary / 2);
  const int64_t blocks = std::min<int64_t>((total + 255) / 256, 4096);
  note_launch();
  rope_table_scaled_kernel<<<static_cast<unsigned>(std::max<int64_t>(blocks, 1)), 256, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace coda

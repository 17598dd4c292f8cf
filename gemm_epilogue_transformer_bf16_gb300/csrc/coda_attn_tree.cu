// Attention of drafted tokens over the 4-bit cache: node i of a sequence's tree
// sees the committed prefix, its ancestors and itself,
//   s_ij = scale q_i . k_j,  O_i = sum_j exp(s_ij - lse_i) v_j.
#include <algorithm>

#include "coda_attn.cuh"
#include "coda_attn_tree.cuh"
#include "coda_internal.h"
#include "coda_kvrow.cuh"
#include "coda_status.h"

namespace coda {
namespace {

// The plainest form: a warp per node and query head, one key at a time, four
// elements per lane.
__global__ void __launch_bounds__(128) attn_tree_kernel(const TreeArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const int64_t w = static_cast<int64_t>(blockIdx.x) * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  const int t = static_cast<int>(w / a.n_q), head = static_cast<int>(w % a.n_q);
  if (blockIdx.x == 0)
    for (int x = threadIdx.x; x < a.B; x += 128)
      if (a.cu[x] < 0 || a.cu[x + 1] < a.cu[x] || a.cu[x + 1] > a.T) atomicOr(a.status, CODA_DEV_SEQLEN_RANGE);
  if (t >= a.T) return;
  int b = 0;
  while (b < a.B && !(t >= a.cu[b] && t < a.cu[b + 1])) ++b;
  if (b == a.B) return;
  const int q0 = a.cu[b], q1 = a.cu[b + 1], n = q1 - q0, i = t - q0;
  const int len = a.seq_lens[b];
  const bool off = q0 < 0 || q1 > a.T || len < n || len > (static_cast<int64_t>(a.max_pages) << a.c.page_shift);
  const bool big = !off && a.parents && n > TREE_MAX_NODES;
  if (off && lane == 0) atomicOr(a.status, CODA_DEV_SEQLEN_RANGE);
  if (big && lane == 0) atomicOr(a.status, CODA_DEV_TREE_RANGE);
  uint32_t seen[TREE_MAX_NODES / 32] = {};
  if (!off && !big && a.parents) {
    int j = i;
    while (j >= 0) {
      seen[j >> 5] |= 1u << (j & 31);
      const int up = a.parents[q0 + j];
      if (up < -1 || up >= j) {
        if (lane == 0) atomicOr(a.status, CODA_DEV_TREE_RANGE);
        break;
      }
      j = up;
    }
  }
  const int kvh = head / a.group;
  const __nv_bfloat16* q = a.Q + t * a.ldq + head * 128 + lane * 4;
  float qf[4], o[4] = {0.f, 0.f, 0.f, 0.f}, m = -INFINITY, l = 0.f;
  for (int k = 0; k < 4; ++k) qf[k] = __bfloat162float(q[k]);
  for (int j = 0; j < (off || big ? 0 : len); ++j) {
    const int d = j - (len - n);
    if (d >= 0 && (a.parents ? !((seen[d >> 5] >> (d & 31)) & 1u) : d > i)) continue;
    const int page = a.table[static_cast<int64_t>(b) * a.max_pages + (j >> a.c.page_shift)];
    if (page < 0 || page >= a.c.num_pages) {
      if (lane == 0) atomicOr(a.status, CODA_DEV_PAGE_RANGE);
      continue;
    }
    float kv[2][4];
    for (int p = 0; p < 2; ++p) {
      const int64_t r = cache_row(a.c, page, p, kvh, j & ((1 << a.c.page_shift) - 1));
      const uint32_t codes = *reinterpret_cast<const uint16_t*>(a.c.codes + r * 64 + lane * 2);
      uint32_t f[4];
      e2m1x8_f16(codes, f);
      const float sf = e4m3_f32(a.c.sf[r * 8 + lane / 4]) * a.c.scale[r];
      kv[p][0] = f16_lo(f[0]) * sf, kv[p][1] = f16_hi(f[0]) * sf;
      kv[p][2] = f16_lo(f[1]) * sf, kv[p][3] = f16_hi(f[1]) * sf;
    }
    float s = 0.f;
    for (int k = 0; k < 4; ++k) s += qf[k] * kv[0][k];
    for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
    s *= a.scale_log2;
    const float nm = fmaxf(m, s), by = m == -INFINITY ? 0.f : exp2f(m - nm), p = exp2f(s - nm);
    l = l * by + p;
    for (int k = 0; k < 4; ++k) o[k] = o[k] * by + p * kv[1][k];
    m = nm;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  for (int k = 0; k < 4; ++k) a.O[static_cast<int64_t>(t) * a.n_q * 128 + head * 128 + lane * 4 + k] = __float2bfloat16(o[k] * inv);
  if (lane == 0) a.lse[static_cast<int64_t>(t) * a.n_q + head] = l == 0.f ? -INFINITY : m * 0.69314718056f + logf(l);
}

}  // namespace

cudaError_t launch_attn_tree(const TreeArgs& a, int sms, cudaStream_t s) {
  return attn_launch(attn_tree_kernel, (static_cast<int64_t>(a.T) * a.n_q + 3) / 4, 128, 0, s, a);
}

}  // namespace coda

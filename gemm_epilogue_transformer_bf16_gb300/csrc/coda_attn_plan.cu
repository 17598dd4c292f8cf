// Work lists of the attention kernels.  The sequence lengths live on the
// device, so one small block cuts the sequences into runs of rows and orders
// the runs by the number of 128-key blocks (or query blocks) they meet,
// longest first: the persistent kernels deal the list out round robin, and
// the long runs must not start last.
#include "coda_attn.cuh"
#include "coda_internal.h"
#include "coda_status.h"

namespace coda {
namespace {

constexpr int PLAN_THREADS = 1024;
constexpr int PLAN_BINS = 2048;
constexpr int PLAN_SMALL = 1024;  // sequences whose offsets fit in shared memory

// Inclusive scan over the block (1024 threads).
__device__ int block_scan(int v, int* warp_sums) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int n = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += n;
  }
  if (lane == 31) warp_sums[w] = v;
  __syncthreads();
  if (w == 0) {
    int s = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int n = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += n;
    }
    warp_sums[lane] = s;
  }
  __syncthreads();
  if (w > 0) v += warp_sums[w - 1];
  __syncthreads();
  return v;
}

struct Side {
  const int32_t* cu_q;  // the offsets (shared memory when there are few sequences)
  const int32_t* cu_k;
  int span;
  int* prefix;          // runs before each sequence, likewise
  AttnTile* out;
  int* count;
  bool keys;            // the list of key runs
};

// Entry t of a list and its bin (longest first).
__device__ __forceinline__ AttnTile make_entry(const AttnPlanArgs& a, const Side& sd, int t, int shift, int& bin, int& w) {
  int lo = 0, hi = a.n_seq;  // prefix[lo] <= t < prefix[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (sd.prefix[mid] <= t) lo = mid; else hi = mid;
  }
  AttnTile e;
  e.q0 = sd.cu_q[lo];
  e.lq = sd.cu_q[lo + 1] - e.q0;
  e.k0 = sd.cu_k[lo];
  e.lk = sd.cu_k[lo + 1] - e.k0;
  e.t0 = (t - sd.prefix[lo]) * sd.span;
  e.seq = lo;
  e.pad1 = e.pad2 = 0;
  if (sd.keys) {
    const int first = max(0, e.t0 - (e.lk - e.lq)) / ATTN_BLK;  // first query block that sees the run
    w = max(0, (e.lq + ATTN_BLK - 1) / ATTN_BLK - first);
  } else {
    w = key_blocks(e, min(e.t0 + sd.span, e.lq) - 1);
  }
  bin = PLAN_BINS - 1 - min(w >> shift, PLAN_BINS - 1);
  return e;
}
__device__ __forceinline__ void put_entry(AttnTile* out, const AttnTile& e) {
  int4* o = reinterpret_cast<int4*>(out);
  o[0] = make_int4(e.q0, e.lq, e.k0, e.lk);
  o[1] = make_int4(e.t0, e.seq, 0, 0);
}

// weights (key list): each warp's largest and total weight of its entries.
__device__ void build_side(const AttnPlanArgs& a, const Side& sd, int* hist, int* warp_sums, float2* weights) {
  const int32_t* cu = sd.keys ? sd.cu_k : sd.cu_q;
  const int64_t other = (sd.keys ? a.Tq : a.Tk) / ATTN_BLK + 2;
  int shift = 0;  // weights beyond the bins share bins
  while ((other >> shift) >= PLAN_BINS) ++shift;
  for (int i = threadIdx.x; i < PLAN_BINS; i += PLAN_THREADS) hist[i] = 0;
  // runs before each sequence
  int total = 0;
  if (threadIdx.x == 0) sd.prefix[0] = 0;
  for (int b0 = 0; b0 < a.n_seq; b0 += PLAN_THREADS) {
    const int b = b0 + static_cast<int>(threadIdx.x);
    const int runs = b < a.n_seq ? (cu[b + 1] - cu[b] + sd.span - 1) / sd.span : 0;
    const int incl = block_scan(runs, warp_sums) + total;
    if (b < a.n_seq) sd.prefix[b + 1] = incl;
    if (threadIdx.x == PLAN_THREADS - 1) warp_sums[32] = incl;
    __syncthreads();
    total = warp_sums[32];
  }
  // counts per bin -> first positions -> entries.  A thread's first entry
  // stays in registers between the two passes.
  const int t0 = static_cast<int>(threadIdx.x);
  int bin0 = 0, bin, w, top = 0;
  float sum = 0.f;
  AttnTile e0;
  if (t0 < total) {
    e0 = make_entry(a, sd, t0, shift, bin0, top);
    sum = static_cast<float>(top);
    atomicAdd(&hist[bin0], 1);
  }
  for (int t = t0 + PLAN_THREADS; t < total; t += PLAN_THREADS) {
    make_entry(a, sd, t, shift, bin, w);
    top = max(top, w);
    sum += static_cast<float>(w);
    atomicAdd(&hist[bin], 1);
  }
  if (sd.keys) {
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
      sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    if ((threadIdx.x & 31) == 0) weights[threadIdx.x >> 5] = make_float2(static_cast<float>(top), sum);
  }
  __syncthreads();
  const int i = 2 * t0, c0 = hist[i], c1 = hist[i + 1];
  const int incl = block_scan(c0 + c1, warp_sums);
  hist[i] = incl - c0 - c1;
  hist[i + 1] = incl - c1;
  __syncthreads();
  if (t0 < total) put_entry(sd.out + atomicAdd(&hist[bin0], 1), e0);
  for (int t = t0 + PLAN_THREADS; t < total; t += PLAN_THREADS) {
    const AttnTile e = make_entry(a, sd, t, shift, bin, w);
    put_entry(sd.out + atomicAdd(&hist[bin], 1), e);
  }
  if (threadIdx.x == 0) *sd.count = total;
  __syncthreads();
}

__global__ void __launch_bounds__(PLAN_THREADS) attn_plan_kernel(const AttnPlanArgs a) {
  __shared__ int hist[PLAN_BINS];
  __shared__ int warp_sums[33];
  __shared__ int32_t small_q[PLAN_SMALL + 1], small_k[PLAN_SMALL + 1];
  __shared__ int small_prefix[PLAN_SMALL + 1];
  __shared__ int bad;
  __shared__ float2 weights[PLAN_THREADS / 32];
  if (threadIdx.x == 0) bad = 0;
  __syncthreads();
  griddep_wait();
  // the next kernel's prologue may start now: it waits for this grid's end in
  // griddep_wait before it reads the lists
  griddep_launch_dependents();
  const bool small = a.n_seq <= PLAN_SMALL;
  // offsets must rise from >= 0 to at most the row counts
  for (int b = threadIdx.x; b < a.n_seq; b += PLAN_THREADS) {
    const int q0 = a.cu_q[b], q1 = a.cu_q[b + 1], k0 = a.cu_k[b], k1 = a.cu_k[b + 1];
    if (q0 < 0 || q1 < q0 || q1 > a.Tq || k0 < 0 || k1 < k0 || k1 > a.Tk) bad = 1;
    if (small) {
      small_q[b] = q0;
      small_k[b] = k0;
      if (b == a.n_seq - 1) {
        small_q[b + 1] = q1;
        small_k[b + 1] = k1;
      }
    }
  }
  __syncthreads();
  if (bad) {
    if (threadIdx.x == 0) {
      atomicOr(a.status, CODA_DEV_SEQLEN_RANGE);
      a.plan.counts[0] = 0;
      a.plan.counts[1] = 0;
      a.plan.counts[2] = 1;
    }
    return;
  }
  const int32_t* cq = small ? small_q : a.cu_q;
  const int32_t* ck = small ? small_k : a.cu_k;
  build_side(a, Side{cq, ck, a.q_span, small ? small_prefix : a.prefix_q, a.plan.q_tiles, a.plan.counts, false}, hist,
             warp_sums, weights);
  if (!a.plan.k_tiles) return;
  build_side(a, Side{cq, ck, ATTN_BLK, small ? small_prefix : a.prefix_k, a.plan.k_tiles, a.plan.counts + 1, true}, hist,
             warp_sums, weights);
  // Parts of a group (a divisor of it).  An item of the key list meets all
  // query tiles of its part's heads, so with few key tiles the longest item
  // (whole group, whole sequence) runs on while most SMs are idle; each part
  // costs a write and a read of 128 KB.  The choice minimises the kernel's
  // estimated time: ITER us per block pair of the longest item or of an SM's
  // share, JOIN us for the joining kernel, PART us for each part (one sequence
  // of 1024 tokens, 64 + 8 heads: 135 -> 82 us with four parts).  One warp
  // looks at a divisor per lane.
  if (threadIdx.x >= 32) return;
  constexpr float ITER = 1.2f, JOIN = 3.f, PART = 0.06f;
  const float heads = static_cast<float>(a.plan.counts[1]) * a.n_kv;  // items of whole groups
  float longest = weights[threadIdx.x].x, pairs = weights[threadIdx.x].y;
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    longest = fmaxf(longest, __shfl_xor_sync(0xffffffffu, longest, o));
    pairs += __shfl_xor_sync(0xffffffffu, pairs, o);
  }
  const float share = pairs * a.n_kv * a.group / a.sms;
  int best = 1;
  float least = ITER * fmaxf(static_cast<float>(a.group) * longest, share);
  if (a.max_parts > 0) {
    for (int s = 2 + static_cast<int>(threadIdx.x); s <= a.group; s += 32) {
      if (heads * s > a.max_parts || a.group % s) continue;
      const float t = ITER * fmaxf(static_cast<float>(a.group / s) * longest, share) + JOIN + PART * heads * s;
      if (t < least) {
        best = s;
        least = t;
      }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      const float t = __shfl_xor_sync(0xffffffffu, least, o);
      const int s = __shfl_xor_sync(0xffffffffu, best, o);
      if (t < least || (t == least && s < best)) {
        best = s;
        least = t;
      }
    }
  }
  if (threadIdx.x == 0) a.plan.counts[2] = best;
}

}  // namespace

cudaError_t launch_attn_plan(const AttnPlanArgs& a, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(1);
  cfg.blockDim = dim3(PLAN_THREADS);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = attn_programmatic_launch() ? 1 : 0;
  note_launch();
  const cudaError_t e = cudaLaunchKernelEx(&cfg, attn_plan_kernel, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace coda

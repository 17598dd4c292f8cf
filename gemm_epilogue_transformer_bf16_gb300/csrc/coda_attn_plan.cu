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
  const int32_t* cu;   // lengths that are cut
  int span;
  int* prefix;
  AttnTile* out;
  int* count;
  bool keys;           // the list of key runs
};

__device__ void build_side(const AttnPlanArgs& a, const Side& sd, int* hist, int* warp_sums) {
  // runs before each sequence
  __shared__ int carry;
  if (threadIdx.x == 0) {
    carry = 0;
    sd.prefix[0] = 0;
  }
  __syncthreads();
  for (int b0 = 0; b0 < a.n_seq; b0 += PLAN_THREADS) {
    const int b = b0 + static_cast<int>(threadIdx.x);
    const int runs = b < a.n_seq ? (sd.cu[b + 1] - sd.cu[b] + sd.span - 1) / sd.span : 0;
    const int incl = block_scan(runs, warp_sums);
    if (b < a.n_seq) sd.prefix[b + 1] = carry + incl;
    __syncthreads();
    if (threadIdx.x == PLAN_THREADS - 1) carry += incl;
    __syncthreads();
  }
  const int total = carry;
  const int64_t other = (sd.keys ? a.Tq : a.Tk) / ATTN_BLK + 2;
  int shift = 0;  // weights beyond the bins share bins
  while ((other >> shift) >= PLAN_BINS) ++shift;
  for (int i = threadIdx.x; i < PLAN_BINS; i += PLAN_THREADS) hist[i] = 0;
  __syncthreads();
  for (int pass = 0; pass < 2; ++pass) {
    for (int t = threadIdx.x; t < total; t += PLAN_THREADS) {
      int lo = 0, hi = a.n_seq;  // prefix[lo] <= t < prefix[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (sd.prefix[mid] <= t) lo = mid; else hi = mid;
      }
      AttnTile e;
      e.q0 = a.cu_q[lo];
      e.lq = a.cu_q[lo + 1] - e.q0;
      e.k0 = a.cu_k[lo];
      e.lk = a.cu_k[lo + 1] - e.k0;
      e.t0 = (t - sd.prefix[lo]) * sd.span;
      e.seq = lo;
      e.pad1 = e.pad2 = 0;
      int w;
      if (sd.keys) {
        const int first = max(0, e.t0 - (e.lk - e.lq)) / ATTN_BLK;   // first query block that sees the run
        w = max(0, (e.lq + ATTN_BLK - 1) / ATTN_BLK - first);
      } else {
        w = key_blocks(e, min(e.t0 + sd.span, e.lq) - 1);
      }
      const int bin = PLAN_BINS - 1 - min(w >> shift, PLAN_BINS - 1);
      if (pass == 0) {
        atomicAdd(&hist[bin], 1);
      } else {
        const int at = atomicAdd(&hist[bin], 1);
        int4* o = reinterpret_cast<int4*>(sd.out + at);
        o[0] = make_int4(e.q0, e.lq, e.k0, e.lk);
        o[1] = make_int4(e.t0, e.seq, 0, 0);
      }
    }
    __syncthreads();
    if (pass == 0) {
      // counts -> first positions, two bins a thread
      const int i = 2 * static_cast<int>(threadIdx.x);
      const int c0 = hist[i], c1 = hist[i + 1];
      const int incl = block_scan(c0 + c1, warp_sums);
      hist[i] = incl - c0 - c1;
      hist[i + 1] = incl - c1;
      __syncthreads();
    }
  }
  if (threadIdx.x == 0) *sd.count = total;
  __syncthreads();
}

__global__ void __launch_bounds__(PLAN_THREADS) attn_plan_kernel(const AttnPlanArgs a) {
  __shared__ int hist[PLAN_BINS];
  __shared__ int warp_sums[32];
  __shared__ int bad;
  if (threadIdx.x == 0) bad = 0;
  __syncthreads();
  griddep_wait();
  // offsets must rise from >= 0 to at most the row counts
  for (int b = threadIdx.x; b < a.n_seq; b += PLAN_THREADS) {
    const int q0 = a.cu_q[b], q1 = a.cu_q[b + 1], k0 = a.cu_k[b], k1 = a.cu_k[b + 1];
    if (q0 < 0 || q1 < q0 || q1 > a.Tq || k0 < 0 || k1 < k0 || k1 > a.Tk) bad = 1;
  }
  __syncthreads();
  if (bad) {
    if (threadIdx.x == 0) {
      atomicOr(a.status, CODA_DEV_SEQLEN_RANGE);
      a.plan.counts[0] = 0;
      a.plan.counts[1] = 0;
    }
    __syncthreads();
  } else {
    build_side(a, Side{a.cu_q, a.q_span, a.prefix_q, a.plan.q_tiles, a.plan.counts, false}, hist, warp_sums);
    if (a.plan.k_tiles)
      build_side(a, Side{a.cu_k, ATTN_BLK, a.prefix_k, a.plan.k_tiles, a.plan.counts + 1, true}, hist, warp_sums);
  }
  // the lists are complete: the next kernel waits for this grid's end in
  // griddep_wait, so its prologue may start now
  griddep_launch_dependents();
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

// Work lists of the attention kernels.  The sequence lengths live on the
// device, so one small block per list cuts the sequences into runs of rows and orders
// the runs by the number of 128-key blocks (or query blocks) they meet,
// longest first: the persistent kernels deal the list out round robin, and
// the long runs must not start last.  The backward's key tiles may be cut by
// query heads as well, where whole groups would make too long an item.
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

// Run t of a list and the blocks it meets.
__device__ __forceinline__ AttnTile make_entry(const AttnPlanArgs& a, const Side& sd, int t, int& w) {
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
  e.slot = -1;
  e.block = 0;
  if (sd.keys) {
    const int first = max(0, e.t0 - (e.lk - e.lq)) / ATTN_BLK;  // first query block that sees the run
    w = max(0, (e.lq + ATTN_BLK - 1) / ATTN_BLK - first);
  } else {
    w = key_blocks(e, min(e.t0 + sd.span, e.lq) - 1);
  }
  return e;
}
__device__ __forceinline__ void put_entry(AttnTile* out, const AttnTile& e) {
  int4* o = reinterpret_cast<int4*>(out);
  o[0] = make_int4(e.q0, e.lq, e.k0, e.lk);
  o[1] = make_int4(e.t0, e.seq, e.slot, e.block);
}

// Longest first.
__device__ __forceinline__ int bin_of(int64_t w, int shift) {
  return PLAN_BINS - 1 - static_cast<int>(min(w >> shift, static_cast<int64_t>(PLAN_BINS - 1)));
}
__device__ __forceinline__ int bin_shift(int64_t most) {  // weights beyond the bins share bins
  int shift = 0;
  while ((most >> shift) >= PLAN_BINS) ++shift;
  return shift;
}
// Counts per bin -> first positions.
__device__ void scan_bins(int* hist, int* warp_sums) {
  __syncthreads();
  const int i = 2 * static_cast<int>(threadIdx.x), c0 = hist[i], c1 = hist[i + 1];
  const int incl = block_scan(c0 + c1, warp_sums);
  hist[i] = incl - c0 - c1;
  hist[i + 1] = incl - c1;
  __syncthreads();
}

constexpr int LENS = 4;  // lengths of parts that are weighed (query list)

// How the groups of the key list are cut: tiles that meet more than `above`
// query blocks into `parts`; `cuts` of them.
struct Cut {
  int parts, above, cuts;
};

// An item of the key list meets all query tiles of its heads, so the longest
// one (whole group, whole sequence) may run on while most SMs are idle; each
// part costs a write and a read of 128 KB.  For each number of parts (a divisor
// of the group) either all tiles are cut, or those longer than NEAR of an SM's
// share or of the longest tile's part.  The choice minimises the kernels'
// estimated time: ITER us per block pair of the longest item or of a share,
// JOIN us for the joining kernel, PART us for each part, and MIXED on the pairs
// where only some are cut (items of many heads and few blocks hold more of the
// dearer blocks on the diagonal than the estimate says).
// Backward in us, all tiles cut alike where room allows -> this rule: 12 + 4
// heads, sequences of 1911, 700, 480, 255, 128, 33, 1: 88 -> 77; 28 + 4 heads,
// 2000 and 20 of 150: 246 -> 182; 16 + 2 heads, 4000 and 100 of 30: 462 -> 267;
// one of 1024, 64 + 8 heads: 82 either way, 135 without a cut.
// longest, pairs: largest and total weight of the runs; count(w): runs above w.
template <class F>
__device__ Cut choose_cut(const AttnPlanArgs& a, int total, float longest, float pairs, F count) {
  constexpr float ITER = 1.2f, JOIN = 3.f, PART = 0.04f, NEAR = 0.7f, MIXED = 1.12f;
  const float share = pairs * a.n_kv * a.group / a.sms;
  Cut best{1, 0, 0};
  float least = ITER * fmaxf(a.group * longest, share);
  for (uint32_t left = a.divisors; left; left &= left - 1) {
    const int s = __ffs(left);  // bit s - 1: a divisor
    const float time = fmaxf(a.group / s * longest, share);
    const int some = static_cast<int>(NEAR * time / a.group);
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int above = k == 0 ? -1 : some;
      const int n = k == 0 ? total : count(above);
      if (n == 0 || static_cast<int64_t>(n) * a.n_kv * s > a.max_parts) continue;
      const float t = ITER * time * (k == 0 ? 1.f : MIXED) + JOIN + PART * static_cast<float>(n * a.n_kv * s);
      if (t < least) {
        best = Cut{s, above, n};
        least = t;
      }
    }
  }
  return best;
}

// Few rows over many keys: the runs of a query list longer than `len` key blocks
// are cut into parts of `len`, whose outputs a second kernel joins.  Of an SM's
// share, its half, third and quarter, and no cut, the one with the least
// estimated time: ITER us for each key block of the longest item, or, where
// there are more items than SMs, of the share and half an item (they are dealt
// whole); JOIN us for the parts' own work and PART us for each.  Forward in us,
// whole runs -> parts: 16 rows over 100000 keys, 64 + 8 heads 989 -> 84; 128
// over 32768 357 -> 102; one row over 65536, 8 + 1 heads 648 -> 53; 5000 tokens,
// 2 + 1 heads 62 -> 28; 2000 tokens, 8 + 2 heads 31 -> 27.  Weighing it costs 4
// us where nothing is cut (1024 rows over 9000, 32 + 8 heads 106 -> 110).
// count(lens, parts, runs): for each length the parts of the longer runs, and
// those runs' number.
template <class F>
__device__ int choose_len(const AttnPlanArgs& a, int total, float longest, float blocks, F count) {
  constexpr float ITER = 1.4f, JOIN = 7.f, PART = 0.04f;
  const float share = blocks * a.q_items / a.sms;
  auto time = [&](float item, int entries) {
    return ITER * (static_cast<int64_t>(entries) * a.q_items <= a.sms ? item : fmaxf(item, share + 0.5f * item));
  };
  float least = time(longest, total);
  int best = 0;
  if (least <= ITER * share + JOIN) return 0;
  int lens[LENS], parts[LENS], runs[LENS];
#pragma unroll
  for (int k = 0; k < LENS; ++k) lens[k] = max(4, static_cast<int>(ceilf(share / static_cast<float>(k + 1))));
  count(lens, parts, runs);
#pragma unroll
  for (int k = 0; k < LENS; ++k) {
    if (parts[k] == 0 || static_cast<int64_t>(parts[k]) * a.q_items > a.max_q_parts) continue;
    const float t = time(static_cast<float>(lens[k]), total - runs[k] + parts[k]) + JOIN +
                    PART * static_cast<float>(parts[k] * a.q_items);
    if (t < least) {
      best = lens[k];
      least = t;
    }
  }
  return best;
}

// CUT: runs may be cut.
template <bool CUT>
__device__ void build_side(const AttnPlanArgs& a, const Side& sd, int* hist, int* warp_sums, float2* weights) {
  const int32_t* cu = sd.keys ? sd.cu_k : sd.cu_q;
  const int64_t most = (sd.keys ? a.Tq : a.Tk) / ATTN_BLK + 2;
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
  // A thread's first run stays in registers between the passes.
  const int t0 = static_cast<int>(threadIdx.x);
  int w0 = 0, w;
  AttnTile e0;
  if (t0 < total) e0 = make_entry(a, sd, t0, w0);

  const bool may_cut = CUT && (sd.keys ? a.max_parts : a.max_q_parts) > 0;
  Cut cut{1, 0, 0};
  int len = 0;  // query list: key blocks of a part
  if (may_cut) {
    int top = w0;
    float pairs = static_cast<float>(w0);
    for (int t = t0 + PLAN_THREADS; t < total; t += PLAN_THREADS) {
      make_entry(a, sd, t, w);
      top = max(top, w);
      pairs += static_cast<float>(w);
    }
    top = __reduce_max_sync(0xffffffffu, top);
#pragma unroll
    for (int o = 16; o; o >>= 1) pairs += __shfl_xor_sync(0xffffffffu, pairs, o);
    if ((t0 & 31) == 0) weights[t0 >> 5] = make_float2(static_cast<float>(top), pairs);
    __syncthreads();
    float longest = weights[t0 & 31].x;
    pairs = weights[t0 & 31].y;
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      longest = fmaxf(longest, __shfl_xor_sync(0xffffffffu, longest, o));
      pairs += __shfl_xor_sync(0xffffffffu, pairs, o);
    }
    // every thread chooses for itself, on the same numbers
    if (sd.keys) {
      cut = choose_cut(a, total, longest, pairs, [&](int above) {
        int n = __syncthreads_count(w0 > above);
        for (int t = PLAN_THREADS; t < total; t += PLAN_THREADS) {
          int v = 0;
          if (t + t0 < total) make_entry(a, sd, t + t0, v);
          n += __syncthreads_count(v > above);
        }
        return n;
      });
    } else {
      len = choose_len(a, total, longest, pairs, [&](const int(&lens)[LENS], int(&parts)[LENS], int(&runs)[LENS]) {
#pragma unroll
        for (int k = 0; k < LENS; ++k) {
          runs[k] = w0 > lens[k];
          parts[k] = runs[k] ? (w0 + lens[k] - 1) / lens[k] : 0;
        }
        for (int t = t0 + PLAN_THREADS; t < total; t += PLAN_THREADS) {
          make_entry(a, sd, t, w);
#pragma unroll
          for (int k = 0; k < LENS; ++k) {
            if (w <= lens[k]) continue;
            ++runs[k];
            parts[k] += (w + lens[k] - 1) / lens[k];
          }
        }
        __shared__ int sums[PLAN_THREADS / 32][2 * LENS];
#pragma unroll
        for (int k = 0; k < LENS; ++k) {
          parts[k] = __reduce_add_sync(0xffffffffu, parts[k]);
          runs[k] = __reduce_add_sync(0xffffffffu, runs[k]);
          if ((t0 & 31) == 0) {
            sums[t0 >> 5][k] = parts[k];
            sums[t0 >> 5][LENS + k] = runs[k];
          }
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < LENS; ++k) {
          parts[k] = __reduce_add_sync(0xffffffffu, sums[t0 & 31][k]);
          runs[k] = __reduce_add_sync(0xffffffffu, sums[t0 & 31][LENS + k]);
        }
      });
    }
  }
  const int heads = sd.keys && may_cut ? a.group : 1;
  const int shift = bin_shift(most * heads);
  __shared__ int ranks, runs_cut;  // parts of cut runs, cut runs
  if (t0 == 0) ranks = runs_cut = 0;
  __syncthreads();
  // parts of a run of this weight, and the weight of its part p
  auto parts_of = [&](int weight) {
    if (!CUT) return 1;
    if (sd.keys) return weight > cut.above ? cut.parts : 1;
    return len > 0 && weight > len ? (weight + len - 1) / len : 1;
  };
  auto bin = [&](int weight, int parts, int p) {
    if (sd.keys) return bin_of(static_cast<int64_t>(weight) * (heads / parts), shift);
    return bin_of(parts == 1 ? weight : min(len, weight - p * len), shift);
  };
  // counts per bin -> first positions -> entries.  The parts of a key tile
  // stand together: they lie in one bin.
  auto count = [&](int weight) {
    const int parts = parts_of(weight);
    if (sd.keys) {
      atomicAdd(&hist[bin(weight, parts, 0)], parts);
    } else {
      for (int p = 0; p < parts; ++p) atomicAdd(&hist[bin(weight, parts, p)], 1);
    }
  };
  auto put = [&](AttnTile e, int weight) {
    const int parts = parts_of(weight);
    if (parts == 1) {
      put_entry(sd.out + atomicAdd(&hist[bin(weight, 1, 0)], 1), e);
      return;
    }
    const int first = atomicAdd(&ranks, parts), rank = atomicAdd(&runs_cut, 1);
    const int at = sd.keys ? atomicAdd(&hist[bin(weight, parts, 0)], parts) : 0;
    for (int p = 0; p < parts; ++p) {
      e.slot = first + p;
      e.block = p * len;
      put_entry(sd.out + (sd.keys ? at + p : atomicAdd(&hist[bin(weight, parts, p)], 1)), e);
    }
    e.slot = first;
    e.block = parts;
    put_entry(a.plan.cuts + (sd.keys ? first / parts : rank), e);
  };
  if (t0 < total) count(w0);
  for (int t = t0 + PLAN_THREADS; t < total; t += PLAN_THREADS) {
    make_entry(a, sd, t, w);
    count(w);
  }
  scan_bins(hist, warp_sums);
  if (t0 < total) put(e0, w0);
  for (int t = t0 + PLAN_THREADS; t < total; t += PLAN_THREADS) {
    const AttnTile e = make_entry(a, sd, t, w);
    put(e, w);
  }
  __syncthreads();
  if (t0 == 0) {
    *sd.count = total + ranks - runs_cut;
    if (may_cut) {
      a.plan.counts[2] = sd.keys ? cut.parts : len;
      a.plan.counts[3] = runs_cut;
    }
  }
  __syncthreads();
}

template <bool CUT>
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
  const bool keys = blockIdx.x != 0;
  if (bad) {
    if (threadIdx.x == 0) {
      atomicOr(a.status, CODA_DEV_SEQLEN_RANGE);
      a.plan.counts[keys] = 0;
      if ((keys ? a.max_parts : a.max_q_parts) > 0) {
        a.plan.counts[2] = keys;
        a.plan.counts[3] = 0;
      }
    }
    return;
  }
  const int32_t* cq = small ? small_q : a.cu_q;
  const int32_t* ck = small ? small_k : a.cu_k;
  const Side sd = keys ? Side{cq, ck, ATTN_BLK, small ? small_prefix : a.prefix_k, a.plan.k_tiles, a.plan.counts + 1, true}
                       : Side{cq, ck, a.q_span, small ? small_prefix : a.prefix_q, a.plan.q_tiles, a.plan.counts, false};
  build_side<CUT>(a, sd, hist, warp_sums, weights);
}

}  // namespace

cudaError_t launch_attn_plan(const AttnPlanArgs& a, cudaStream_t s) {
  const int lists = a.plan.k_tiles ? 2 : 1;
  return a.max_parts > 0 || a.max_q_parts > 0 ? attn_launch(attn_plan_kernel<true>, lists, PLAN_THREADS, 0, s, a)
                                              : attn_launch(attn_plan_kernel<false>, lists, PLAN_THREADS, 0, s, a);
}

}  // namespace coda

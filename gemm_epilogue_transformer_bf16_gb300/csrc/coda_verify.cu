// Verification of drafted tokens against the target's probabilities, from given
// random numbers.
//
// The walk begins at node 0 with w = p_0, Z = 1.  A child i of the node where it
// stands, in order of their numbers, with token x:
//   u_i q(x) Z < w(x): accepted, the walk goes on there with w = p_i, Z = 1;
//   else               w <- max(w - Z q, 0), Z <- sum w
// (q: the probabilities the node's children were drawn from; without them, drafts
// that were not drawn, q is 1 at x and 0 elsewhere: w(x) <- 0, Z <- Z - w(x)).
// Where no child is left the next token is the first x with
//   sum_{y <= x} w(y) > u sum w,
// so that the tokens together are distributed as the target's own.
//
// A decision at the edge of a step of a sum over 10^5 tokens must not depend on
// the order of the sum: fp32 sums of a vocabulary are off by more than many
// tokens' probability.  The weights are therefore integers in units of 2^-60
// (the probabilities' own bits down to there, smaller ones are dropped), and
// their sums are exact in any order.
//
// HBM-bound: one row of p and q per request (the walk before it reads two values
// per node), and bound by latency when there are few.  A cluster of up to eight
// CTAs per request: in every CTA one warp walks on the nodes' values in shared
// memory (the same walk in all of them), sums over the vocabulary are split
// between the CTAs and meet by distributed shared memory.  128 requests of 5
// drawn tokens over 128256 probabilities in fp32 (131 MB at most, 19 us): 32 us
// in a graph; one request of 7 11 us; 48 trees of 1 to 40 nodes over 50257
// probabilities in bf16 19 us.  With eight CTAs to every request, each thread
// walking and sums by conversions to 64 bits it was 128, 33 and 61 us.
#include <algorithm>
#include <cuda_bf16.h>

#include "coda_attn.cuh"
#include "coda_internal.h"
#include "coda_status.h"
#include "coda_verify.cuh"

namespace coda {
namespace {

constexpr int VF_CTAS = 8;  // of a cluster, at most
constexpr int VF_THREADS = 512;
constexpr int VF_WARPS = VF_THREADS / 32;
typedef unsigned long long u64;

__device__ __forceinline__ ulonglong2 ld_cluster_2u64(const void* p, uint32_t rank) {
  ulonglong2 v;
  asm volatile("ld.shared::cluster.v2.u64 {%0, %1}, [%2];" : "=l"(v.x), "=l"(v.y) : "r"(mapa_shared(p, rank)) : "memory");
  return v;
}

// A probability in units of 2^-60; NaN and negative values count as 0, values
// above 1 as 1.
__device__ __forceinline__ u64 fixed60(float p) {
  return p > 0.f ? __float2ull_rz(fminf(p, 1.f) * 0x1p60f) : 0ull;
}
// Z q, both in units of 2^-60.
__device__ __forceinline__ u64 scaled60(u64 Z, u64 q) { return __umul64hi(Z, q) << 4 | Z * q >> 60; }

template <bool F32>
__device__ __forceinline__ float value(const void* base, int64_t at) {
  if constexpr (F32) return static_cast<const float*>(base)[at];
  return __bfloat162float(static_cast<const __nv_bfloat16*>(base)[at]);
}

__device__ __forceinline__ u64 warp_sum(u64 v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}
__device__ __forceinline__ u64 warp_scan(u64 v, int lane) {
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const u64 n = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += n;
  }
  return v;
}

// Sums of probabilities in units of 2^-60, with no conversion (F2I of 64 bits
// runs at an eighth of the rate of an addition): the bits of a probability above
// 2^-22, the next 22 and the 16 after them are each read off an addition, rounded
// to zero, to a number whose last place is that unit.  Sums of the three in 32
// bits hold for 511 values.
struct Sum60 {
  int hi = 0, mid = 0, lo = 0;
  static __device__ __forceinline__ void cut(float p, int& a, int& b, int& c) {
    const float t = __fadd_rz(p, 2.f), r = p - (t - 2.f);              // exact
    const float t2 = __fadd_rz(r, 0x1p-21f), r2 = r - (t2 - 0x1p-21f);  // exact
    a = __float_as_int(t);
    b = __float_as_int(t2);
    c = __float_as_int(__fadd_rz(r2, 0x1p-37f));
  }
  // p in [0, 1]
  __device__ __forceinline__ void add(float p) {
    int a, b, c;
    cut(p, a, b, c);
    hi += a - 0x40000000;   // the bits of 2
    mid += b - 0x35000000;  // 2^-21
    lo += c - 0x2d000000;   // 2^-37
  }
  // max(p - q, 0), each cut to its units
  __device__ __forceinline__ void add_above(float p, float q) {
    int a, b, c, d, e, f;
    cut(p, a, b, c);
    cut(fminf(p, q), d, e, f);
    hi += a - d;
    mid += b - e;
    lo += c - f;
  }
};

// A thread's sum in units of 2^-60, modulo 16, and the whole of it in units of 2^-22,
// 16 at most: sums of the latter over all threads are too low by less than 2^-10,
// which tells whether those of the former have passed 16.
struct Sum {
  u64 fine;
  uint32_t coarse;
};
constexpr uint32_t COARSE_16 = 16u << 22, COARSE_LOW = 1u << 12;

struct VerifyShared {
  u64 Z[VERIFY_MAX_NODES];  // Z after each refusal at the node (Z[0] = 1)
  ulonglong2 warp[VF_WARPS];  // fine and coarse sums
  ulonglong2 total;           // of this CTA, read by the others
  u64 fine[VF_WARPS];
  int here, count, ngone, refused, more;  // where the walk stands; more: it wants a sum
  float p[VERIFY_MAX_NODES], q[VERIFY_MAX_NODES], u[VERIFY_MAX_NODES];
  int token[VERIFY_MAX_NODES], parent[VERIFY_MAX_NODES];
  int gone[VERIFY_MAX_NODES];  // tokens refused at the node, each once (drafts not drawn)
};

// Weights of the row where the walk stands.  A row is read in aligned pieces
// of 16 bytes, numbered from the one that holds its first element: E elements,
// the first `lead` elements of piece 0 belong to the row before.
template <bool F32>
struct Row {
  static constexpr int E = F32 ? 4 : 8;
  const void *p, *q;  // row starts; q null: drafts not drawn
  int lead, V;
  int refused;        // refusals that w has gone through
  __device__ __forceinline__ int pieces() const { return (V + lead + E - 1) / E; }

  // A piece as it lies in memory, zeros outside the row.
  __device__ __forceinline__ uint4 load(const void* base, int piece) const {
    const int e0 = piece * E - lead;
    if (e0 >= 0 && e0 + E <= V)
      return *reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(base) + static_cast<int64_t>(e0) * (16 / E));
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < E; ++i)
      if (e0 + i >= 0 && e0 + i < V) {
        const uint32_t bits = __float_as_uint(value<F32>(base, e0 + i));
        w[F32 ? i : i >> 1] |= F32 ? bits : (i & 1) ? bits : bits >> 16;
      }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
  static __device__ __forceinline__ float element(const uint4& v, int i) {
    const uint32_t w = (F32 ? i : i >> 1) == 0 ? v.x : (F32 ? i : i >> 1) == 1 ? v.y : (F32 ? i : i >> 1) == 2 ? v.z : v.w;
    return F32 ? __uint_as_float(w) : (i & 1) ? bf16_hi(w) : bf16_lo(w);
  }
  __device__ __forceinline__ u64 weight(float pv, float qv, const u64* Z) const {
    u64 w = fixed60(pv);
    if (q == nullptr) return w;
    const u64 fq = fixed60(qv);
    for (int k = 0; k < refused; ++k) {
      const u64 d = k == 0 ? fq : scaled60(Z[k], fq);
      w = w > d ? w - d : 0;
    }
    return w;
  }
  __device__ __forceinline__ bool need_q() const { return q != nullptr && refused > 0; }
};

// Sum of this lane's share of the weights of pieces [piece, stop); tokens
// refused where nothing was drawn are left out by the caller.  (One copy of the
// code for all of a kernel's sums: the registers of a second one are spilled.)
template <bool F32>
__device__ __noinline__ Sum sum_pieces(const Row<F32> r, int piece, int stop, const u64* Z) {
  int64_t hi = 0, lo = 0;  // in units of 2^-22 and 2^-60
  constexpr int N = 4;  // pieces in flight
  if (!r.need_q()) {
    for (; piece < stop; piece += N * 32) {
      uint4 vp[N];
#pragma unroll
      for (int n = 0; n < N; ++n)
        vp[n] = piece + n * 32 < stop ? r.load(r.p, piece + n * 32) : make_uint4(0, 0, 0, 0);
      Sum60 c;
#pragma unroll
      for (int n = 0; n < N; ++n)
#pragma unroll
        for (int i = 0; i < Row<F32>::E; ++i) c.add(__saturatef(r.element(vp[n], i)));  // NaN: 0
      hi += c.hi;
      lo += (static_cast<int64_t>(c.mid) << 16) + c.lo;
    }
  } else if (r.refused == 1) {
    for (; piece < stop; piece += N * 32) {
      uint4 vp[N], vq[N];
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const bool in = piece + n * 32 < stop;
        vp[n] = in ? r.load(r.p, piece + n * 32) : make_uint4(0, 0, 0, 0);
        vq[n] = in ? r.load(r.q, piece + n * 32) : make_uint4(0, 0, 0, 0);
      }
      Sum60 c;
#pragma unroll
      for (int n = 0; n < N; ++n)
#pragma unroll
        for (int i = 0; i < Row<F32>::E; ++i)
          c.add_above(__saturatef(r.element(vp[n], i)), __saturatef(r.element(vq[n], i)));
      hi += c.hi;
      lo += (static_cast<int64_t>(c.mid) << 16) + c.lo;
    }
  } else {
    for (; piece < stop; piece += 32) {
      const uint4 vp = r.load(r.p, piece), vq = r.load(r.q, piece);
#pragma unroll 1
      for (int i = 0; i < Row<F32>::E; ++i) {
        const u64 w = r.weight(r.element(vp, i), r.element(vq, i), Z);
        hi += static_cast<int64_t>(w >> 38);
        lo += static_cast<int64_t>(w & ((u64(1) << 38) - 1));
      }
    }
  }
  return {(static_cast<u64>(hi) << 38) + static_cast<u64>(lo),
          static_cast<uint32_t>(min(hi + (lo >> 38), static_cast<int64_t>(COARSE_16)))};
}

template <bool F32>
__global__ void __launch_bounds__(VF_THREADS, 2) verify_kernel(const VerifyArgs a) {
  __shared__ VerifyShared sh;
  griddep_wait();
  griddep_launch_dependents();
  constexpr int E = Row<F32>::E;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_ctarank();
  const int ctas = a.ctas, b = static_cast<int>(blockIdx.x) / ctas;
  const int t0 = a.cu[b], t1 = a.cu[b + 1];
  const int n = t1 - t0;
  int32_t* nodes = a.nodes + static_cast<int64_t>(b) * a.width;
  int32_t* out = a.out + static_cast<int64_t>(b) * a.width;
  const bool off = t0 < 0 || n < 0 || t1 > a.T;
  if (off || n == 0 || n > VERIFY_MAX_NODES) {
    if (rank == 0) {
      if (tid == 0) {
        a.count[b] = 0;
        if (off) atomicOr(a.status, CODA_DEV_SEQLEN_RANGE);
        else if (n > 0) atomicOr(a.status, CODA_DEV_TREE_RANGE);
      }
      for (int i = tid; i < a.width; i += VF_THREADS) nodes[i] = out[i] = -1;
    }
    return;  // the whole cluster
  }
  // what the walk looks at
  for (int i = tid; i < n; i += VF_THREADS) {
    int up = i - 1, x = a.tokens[t0 + i];
    if (a.parents) up = a.parents[t0 + i];
    bool bad = up < -1 || up >= i;
    if (bad && rank == 0) atomicOr(a.status, CODA_DEV_TREE_RANGE);
    if (bad) up = -1;
    if (i > 0 && up >= 0 && (x < 0 || x >= a.V)) {
      if (rank == 0) atomicOr(a.status, CODA_DEV_LABEL_RANGE);
      up = -1;  // never a child
    }
    const int64_t at = static_cast<int64_t>(t0 + max(up, 0)) * a.V + x;
    sh.parent[i] = up;
    sh.token[i] = x;
    sh.u[i] = a.u[t0 + i];
    // negative or NaN: 0, above 1: 1, as in the sums
    sh.p[i] = up >= 0 ? __saturatef(value<F32>(a.P, at)) : 0.f;
    sh.q[i] = up >= 0 && a.Q ? __saturatef(value<F32>(a.Q, at)) : 1.f;
  }
  __syncthreads();

  Row<F32> r;
  auto stand = [&](int node) {
    const int64_t at = static_cast<int64_t>(t0 + node) * a.V;
    r.p = F32 ? static_cast<const void*>(static_cast<const float*>(a.P) + at)
              : static_cast<const void*>(static_cast<const __nv_bfloat16*>(a.P) + at);
    r.q = !a.Q ? nullptr
               : F32 ? static_cast<const void*>(static_cast<const float*>(a.Q) + at)
                     : static_cast<const void*>(static_cast<const __nv_bfloat16*>(a.Q) + at);
    r.V = static_cast<int>(a.V);
    r.lead = static_cast<int>(at % E);
    r.refused = 0;
  };
  // this CTA's and this warp's pieces
  int c0 = 0, c1 = 0, w0 = 0, w1 = 0;
  auto share = [&]() {
    const int all = r.pieces(), per = (all + ctas - 1) / ctas;
    c0 = min(all, static_cast<int>(rank) * per);
    c1 = min(all, c0 + per);
    const int pw = (c1 - c0 + VF_WARPS - 1) / VF_WARPS;
    w0 = min(c1, c0 + warp * pw);
    w1 = min(c1, w0 + pw);
  };
  // Weights that the refused tokens of a draft not drawn still have in [w0, w1).
  auto refused_in = [&](int gone, int from, int to) {
    u64 s = 0;
    if (r.q == nullptr)
      for (int k = lane; k < gone; k += 32) {
        const int x = sh.gone[k], at = (x + r.lead) / E;
        if (at >= from && at < to) s += fixed60(value<F32>(r.p, x));
      }
    return warp_sum(s);
  };
  // Sum over the vocabulary; sh.warp holds the warps' parts of this CTA, and
  // `before` what the CTAs in front of it have.  A row of 16 or more is `excess`.
  bool excess = false;
  auto total = [&](int gone, u64& before) {
    share();
    const Sum part = sum_pieces<F32>(r, w0 + lane, w1, sh.Z);
    const u64 s = warp_sum(part.fine) - refused_in(gone, w0, w1);
    const uint32_t high = __reduce_add_sync(0xffffffffu, part.coarse);
    if (lane == 0) sh.warp[warp] = make_ulonglong2(s, min(high, COARSE_16));
    __syncthreads();
    u64 c = 0, all = 0;
    uint32_t coarse = 0;
    before = 0;
#pragma unroll
    for (int i = 0; i < VF_WARPS; ++i) {
      const ulonglong2 v = sh.warp[i];
      c += v.x;
      coarse += static_cast<uint32_t>(v.y);
    }
    all = c;
    if (ctas > 1) {
      if (tid == 0) sh.total = make_ulonglong2(c, min(coarse, COARSE_16));
      cluster_sync();
      all = 0;
      coarse = 0;
#pragma unroll
      for (uint32_t i = 0; i < VF_CTAS; ++i)
        if (i < ctas) {
          const ulonglong2 v = ld_cluster_2u64(&sh.total, i);
          if (i < rank) before += v.x;
          all += v.x;
          coarse += static_cast<uint32_t>(v.y);
        }
      cluster_sync();  // read by all before it is written again, or its CTA ends
    }
    excess = coarse >= COARSE_16 ||
             (coarse >= COARSE_16 - COARSE_LOW && all >> 63 == 0);
    return all;
  };

  // Warp 0 walks (the comparisons are in 64 bits, of which an SM does few), up
  // to a child whose decision needs a sum over the vocabulary, or to the end.
  int here = 0, count = 0, gone = 0, refused = 0, next = 1;
  bool summed = true;  // Z is that of the refusals so far
  double Z = 1.0;
  u64 before = 0;
  if (rank == 0 && tid == 0) nodes[0] = 0;
  if (tid == 0) sh.Z[0] = 1ull << 60;
  for (;;) {
    if (warp == 0) {
      bool more = false;
      while (count + 1 < a.width && next < n) {
        const int seen = next & ~31;
        const uint32_t kids = __ballot_sync(0xffffffffu, seen + lane < n && sh.parent[seen + lane] == here) &
                              (0xffffffffu << (next & 31));
        if (kids == 0) {
          next = seen + 32;
          continue;
        }
        const int i = seen + __ffs(kids) - 1;
        if (!summed) {
          next = i;
          more = true;
          break;
        }
        next = i + 1;
        const int x = sh.token[i];
        double wx = sh.p[i];
        bool again = false;  // refused here before: nothing is left of it
        if (a.Q) {
          r.q = a.Q;  // (only whether there is one)
          r.refused = refused;
          if (refused > 0) wx = static_cast<double>(r.weight(sh.p[i], sh.q[i], sh.Z)) * 0x1p-60;
        } else {
          again = false;
          for (int k = lane; k < gone; k += 32) again |= sh.gone[k] == x;
          again = __any_sync(0xffffffffu, again);
          if (again) wx = 0.0;
        }
        if (static_cast<double>(sh.u[i]) * (static_cast<double>(sh.q[i]) * Z) < wx) {
          if (rank == 0 && lane == 0) {
            out[count] = x;
            nodes[count + 1] = i;
          }
          ++count;
          here = i;
          Z = 1.0;
          gone = refused = 0;
        } else if (a.Q) {
          ++refused;
          summed = false;
        } else if (!again) {
          Z -= wx;
          if (lane == 0) sh.gone[gone] = x;
          __syncwarp();
          ++gone;
        }
      }
      if (lane == 0) {
        sh.here = here;
        sh.count = count;
        sh.ngone = gone;
        sh.refused = refused;
        sh.more = more;
      }
    }
    __syncthreads();
    stand(sh.here);
    r.refused = sh.refused;
    count = sh.count;
    gone = sh.ngone;
    if (!sh.more) break;
    const u64 z = total(0, before);
    if (excess) break;
    if (tid == 0) sh.Z[r.refused] = z;
    __syncthreads();
    summed = true;
    Z = static_cast<double>(z) * 0x1p-60;
  }

  // The next token.  Nothing left (probabilities that do not sum to 1): the
  // row's own probabilities; none there either: -1.
  u64 all = excess ? 0 : total(gone, before);
  if (all == 0 && !excess && (r.refused > 0 || gone > 0)) {
    r.refused = 0;
    gone = 0;
    __syncthreads();  // the warps' parts have been read
    all = total(0, before);
  }
  if (excess) {
    all = 0;
    if (rank == 0 && tid == 0) atomicOr(a.status, CODA_DEV_PROB_RANGE);
  }
  const float un = a.u_next[b];
  u64 tau = 0;  // floor(un all): a sum in whole units that passes it passes un all
  if (un > 0.f) {
    const uint32_t bits = __float_as_uint(un), e = bits >> 23;
    const u64 m = (bits & 0x7FFFFFu) | (e ? 0x800000u : 0u);  // un = m 2^(e - 150)
    tau = e > 126 ? all : e < 63 ? 0 : __umul64hi(all, m << 40) >> (126 - e);  // of all < 2^64
  }
  if (tau >= all && all > 0) tau = all - 1;
  if (rank == 0) {
    if (tid == 0) {
      a.count[b] = count;
      if (all == 0) out[count] = -1;
    }
    for (int i = count + 1 + tid; i < a.width; i += VF_THREADS) nodes[i] = out[i] = -1;
  }
  u64 mine = 0;
#pragma unroll
  for (int i = 0; i < VF_WARPS; ++i) mine += sh.warp[i].x;
  if (all == 0 || tau < before || tau - before >= mine) return;
  // In this CTA.  The warp's share that holds it, cut into pieces of 32 ...
  u64 left = tau - before;  // the token's weight passes this
  int at = 0;
#pragma unroll
  for (int i = 0; i < VF_WARPS; ++i) {
    const u64 s = sh.warp[i].x;
    if (at == i && left >= s && i + 1 < VF_WARPS) {
      left -= s;
      ++at;
    }
  }
  const int pw = (c1 - c0 + VF_WARPS - 1) / VF_WARPS;
  const int s0 = min(c1, c0 + at * pw), s1 = min(c1, s0 + pw);
  const int run = ((s1 - s0 + VF_WARPS - 1) / VF_WARPS + 31) & ~31;  // pieces per warp
  const int f0 = min(s1, s0 + warp * run), f1 = min(s1, f0 + run);
  const u64 s = warp_sum(sum_pieces<F32>(r, f0 + lane, f1, sh.Z).fine) - refused_in(gone, f0, f1);
  if (lane == 0) sh.fine[warp] = s;
  __syncthreads();
  at = 0;
#pragma unroll
  for (int i = 0; i < VF_WARPS; ++i) {
    const u64 c = sh.fine[i];
    if (at == i && left >= c && i + 1 < VF_WARPS) {
      left -= c;
      ++at;
    }
  }
  if (warp != at) return;
  // ... and the warp that holds it goes through them in order
  for (int p0 = f0; p0 < f1; p0 += 32) {
    const bool in = p0 + lane < f1;
    const uint4 vp = in ? r.load(r.p, p0 + lane) : make_uint4(0, 0, 0, 0);
    const uint4 vq = in && r.need_q() ? r.load(r.q, p0 + lane) : make_uint4(0, 0, 0, 0);
    u64 w[E];
#pragma unroll
    for (int i = 0; i < E; ++i) w[i] = r.weight(r.element(vp, i), r.element(vq, i), sh.Z);
    const int e0 = (p0 + lane) * E - r.lead;
    if (r.q == nullptr)
      for (int k = 0; k < gone; ++k) {
        const int o = sh.gone[k] - e0;
#pragma unroll
        for (int i = 0; i < E; ++i)
          if (o == i) w[i] = 0;
      }
    u64 sum = 0;
#pragma unroll
    for (int i = 0; i < E; ++i) sum += w[i];
    const u64 incl = warp_scan(sum, lane), excl = incl - sum;
    const u64 step = __shfl_sync(0xffffffffu, incl, 31);
    if (left < step) {
      if (left >= excl && left < incl) {
        u64 c = excl;
        int x = -1;
#pragma unroll
        for (int i = 0; i < E; ++i) {
          c += w[i];
          if (x < 0 && c > left) x = e0 + i;
        }
        out[count] = x;
      }
      return;
    }
    left -= step;
  }
}

}  // namespace

cudaError_t launch_verify(VerifyArgs a, bool f32, cudaStream_t s) {
  // As many CTAs to a request as are resident at once, two to an SM; a second
  // wave would walk its trees while the memory has nothing to do.  (Shares are not
  // even then: 128 requests have two each, so that of 152 SMs 104 have two of 256
  // and the others one.)
  const int64_t slots = 2 * static_cast<int64_t>(device_sms());
  a.ctas = VF_CTAS;
  while (a.ctas > 1 && static_cast<int64_t>(a.B) * a.ctas > slots) a.ctas >>= 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.B) * a.ctas);
  cfg.blockDim = dim3(VF_THREADS);
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = a.ctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = attn_programmatic_launch() ? 2 : 1;
  note_launch();
  const cudaError_t e = f32 ? cudaLaunchKernelEx(&cfg, verify_kernel<true>, a)
                            : cudaLaunchKernelEx(&cfg, verify_kernel<false>, a);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace coda

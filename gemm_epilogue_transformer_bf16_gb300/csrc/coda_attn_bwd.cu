// Causal attention over packed sequences, backward.
//
//   p_ij = exp(s_ij - lse_i),  D_i = dO_i . O_i,  ds_ij = p_ij (dO_i . v_j - D_i)
//   dv_j = sum_i p_ij dO_i,  dk_j = scale sum_i ds_ij q_i,  dq_i = scale sum_j ds_ij k_j
//
// Two persistent kernels, each owning its outputs, so nothing is summed
// through memory and the gradients do not depend on the order of anything:
// one walks key tiles (dK, dV in TMEM, four products per block pair), one
// walks query tiles (dQ, three products).  S and dO V^T are formed twice: 7
// products where a single pass has 5, against fp32 sums of dQ over the key
// tiles in global memory (64 KB per block pair and head, in an order that
// changes from run to run).  The products bound the key-tile kernel, the waits
// between arithmetic and products the query-tile kernel.
//
// The query-tile kernel runs first: it has the rows of dO at hand, forms D, and
// leaves -lse * log2(e) and -D per row and head for the key-tile kernel.
//
// One item of the key-tile kernel holds all query heads of its group, so few
// sequences, or one long one among short ones, give it items longer than an
// SM's share.  Such tiles' groups are cut into parts, whose fp32 partial dK and
// dV a third kernel adds in fixed order.
//
// Roundings: P and dS to bf16 before their products; dQ, dK, dV to bf16 once.
// D = dO . O inherits O's rounding to bf16, which weighs where a row sees few
// keys (|O| is then as large as the values); rows of a tile with one key block
// take D = sum_j p_ij dP_ij instead, which is the same number.
#include <algorithm>

#include "coda_attn.cuh"
#include "coda_internal.h"
#include "coda_status.h"

namespace coda {
namespace {

constexpr int BWD_THREADS = 384;
constexpr uint32_t TILE_BYTES = ATTN_BLK * ATTN_D * 2;  // 32 KB
constexpr uint32_t HALF_BYTES = TILE_BYTES / 2;
constexpr int KV_STAGES = 5;  // key-tile kernel: ring of Q and dO tiles beside K and V
constexpr int Q_STAGES = 6;   // query-tile kernel: ring of K, V, dO and O tiles beside Q
constexpr uint32_t ROW_BYTES = 2 * ATTN_BLK * 4;  // -lse2 and -D of a tile
constexpr uint32_t KV_SMEM = (2 + KV_STAGES) * TILE_BYTES + 2 * ROW_BYTES + 512;
constexpr uint32_t Q_SMEM = (1 + Q_STAGES) * TILE_BYTES + 512 + 3 * ATTN_BLK * 4;
static_assert(KV_SMEM <= 232448 && Q_SMEM <= 232448, "shared memory per CTA");

__device__ __forceinline__ int64_t padded_row(const AttnTile& t) {
  return (static_cast<int64_t>(t.q0 / ATTN_BLK) + t.seq) * ATTN_BLK;
}

// Barrier waits of one role; `ok` latches the first failure.
struct Waiter {
  volatile int* abort_flag;
  int* status;
  uint64_t limit;
  bool ok = true;
  __device__ __forceinline__ bool operator()(uint64_t* bar, uint32_t parity) {
    if (ok) ok = mbar_wait_bounded(bar, parity, abort_flag, status, limit);
    return ok;
  }
  // the same for a whole warp that stays converged
  __device__ __forceinline__ bool warp(uint64_t* bar, uint32_t parity) {
    ok = __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity, abort_flag, status, limit)) && ok;
    return ok;
  }
};

__device__ __forceinline__ void let_copies_land() {
  const uint64_t t0 = globaltimer_ns();
  while (globaltimer_ns() - t0 < 2000000ull) {
  }
}

// C (+)= A B^T, 128 x 128 x 128: A, B in shared memory, K-major.
__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t sa, uint32_t sb, bool acc, uint32_t el) {
  constexpr uint32_t ID = idesc_bf16(128, 128, 0, 0);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t o = (i >> 2) * HALF_BYTES + (i & 3) * 32;
    umma_bf16(d, sdesc_sw128(sa + o, 16, 1024), sdesc_sw128(sb + o, 16, 1024), ID, acc || i > 0, el);
  }
}
// A in TMEM (64 columns, contiguous), B in shared memory, K-major.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t ta, uint32_t sb, bool acc, uint32_t el) {
  constexpr uint32_t ID = idesc_bf16(128, 128, 0, 0);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const uint32_t o = (i >> 2) * HALF_BYTES + (i & 3) * 32;
    umma_bf16_ts(d, ta + i * 8, sdesc_sw128(sb + o, 16, 1024), ID, acc || i > 0, el);
  }
}
// C (+)= A B: A in TMEM, 64 of the contraction's columns in each half of a
// 128-column region; B [contraction, 128] in shared memory (MN-major).
__device__ __forceinline__ void mma_tn(uint32_t d, uint32_t ta, uint32_t sb, bool acc, uint32_t el) {
  constexpr uint32_t ID = idesc_bf16(128, 128, 0, 1);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    umma_bf16_ts(d, ta + (i >> 2) * 64 + (i & 3) * 8, sdesc_sw128(sb + i * 2048, HALF_BYTES, 1024), ID, acc || i > 0,
                 el);
}

__device__ __forceinline__ void load_pair(uint8_t* dst, const CUtensorMap* m, uint64_t* bar, int col, int row,
                                          uint32_t el) {
  tma_load_2d(dst, m, bar, col, row, el);
  tma_load_2d(dst + HALF_BYTES, m, bar, col + 64, row, el);
}

// 64 bf16 (as fp32 pairs) of a row, scaled, from 64 TMEM columns.
__device__ __forceinline__ void store_row64(uint32_t taddr, __nv_bfloat16* dst, float scale, bool write) {
#pragma unroll 1
  for (int q = 0; q < 2; ++q) {
    float v[32];
    __syncwarp();
    tmem_ld32(taddr + q * 32, v);
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] *= scale;
    if (write) {
#pragma unroll
      for (int i = 0; i < 4; ++i) store_bf16x8(dst + q * 32 + i * 8, v + i * 8);
    }
  }
}

// ------------------------------------------------------------------ dK, dV
// Item: a tile of 128 keys of one key/value head and a part of its query
// heads; it meets the query tiles that see it, head by head (iterations).
//
//   warps 0-7   thread = key row, warpgroup = half of the 128 queries:
//               P^T = exp2(S^T c - lse2) and dS^T = P^T (dP^T - D), bf16,
//               back into TMEM over their sources (each half its own).
//   warp 8      UMMA: dV += P^T dO | S^T = K Q'^T | dK += dS^T Q | dP^T = V dO'^T
//               (primes: the next iteration), so the exponentials run beside
//               dK and dP^T, and dS^T beside dV and S^T.
//   warp 9      TMA: K and V, a ring of Q and dO tiles, the rows' -lse2 and -D.
//   warp 10     zeroes Q and dO rows behind the sequence.
//
// Measured: 4 sequences of 2048 tokens, 64 + 8 heads (four products, 550 GFLOP)
// 330 us, 1670 TFLOP/s, the tensor pipe active 76 %: bound by the products (620
// to 700 clocks each for 128^3).
struct KvItem {
  AttnTile t;
  int kv, first, n;  // first query tile, query tiles
  int h0, nh;        // query heads
  int64_t part;      // place of the partial results; -1: the whole group
};
// The entries of a cut tile stand together, and so do the parts of a head: in
// the order of the items and in memory.
__device__ __forceinline__ KvItem kv_item(const AttnBwdArgs& a, int w, int splits) {
  KvItem it;
  const int ti = w / a.n_kv;
  it.t = load_tile(a.k_tiles + ti);
  it.kv = w - ti * a.n_kv;
  it.nh = a.group;
  it.h0 = it.kv * a.group;
  it.part = -1;
  if (it.t.slot >= 0) {
    const int rank = it.t.slot / splits;
    const int rest = w - (ti - (it.t.slot - rank * splits)) * a.n_kv;
    it.kv = rest / splits;
    it.nh = a.group / splits;
    it.h0 = it.kv * a.group + (rest - it.kv * splits) * it.nh;
    it.part = static_cast<int64_t>(rank) * a.n_kv * splits + rest;
  }
  it.first = max(0, it.t.t0 - (it.t.lk - it.t.lq)) / ATTN_BLK;
  it.n = max(0, (it.t.lq + ATTN_BLK - 1) / ATTN_BLK - it.first);
  return it;
}

__global__ void __launch_bounds__(BWD_THREADS, 1)
    attn_bwd_kv_kernel(const __grid_constant__ CUtensorMap mQ, const __grid_constant__ CUtensorMap mK,
                       const __grid_constant__ CUtensorMap mV, const __grid_constant__ CUtensorMap mG,
                       const AttnBwdArgs a) {
  extern __shared__ __align__(1024) uint8_t bwd_smem[];
  uint8_t* sK = bwd_smem;
  uint8_t* sV = sK + TILE_BYTES;
  uint8_t* ring = sV + TILE_BYTES;
  float* rows = reinterpret_cast<float*>(ring + KV_STAGES * TILE_BYTES);  // two buffers of -lse2 | -D
  uint64_t* full = reinterpret_cast<uint64_t*>(reinterpret_cast<uint8_t*>(rows) + 2 * ROW_BYTES);
  uint64_t* empty = full + KV_STAGES;
  uint64_t* raw = empty + KV_STAGES;
  uint64_t* row_full = raw + KV_STAGES;
  uint64_t* row_empty = row_full + 2;
  uint64_t* kv_full = row_empty + 2;
  uint64_t* kv_empty = kv_full + 1;
  uint64_t* s_full = kv_empty + 1;
  uint64_t* dp_full = s_full + 1;
  uint64_t* p_ready = dp_full + 1;
  uint64_t* ds_ready = p_ready + 1;
  uint64_t* acc_full = ds_ready + 1;
  uint64_t* drain = acc_full + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  static_assert((3 * KV_STAGES + 12) * 8 + 8 <= 512, "barrier area");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < KV_STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
      mbar_init(&raw[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&row_full[b], 1);
      mbar_init(&row_empty[b], 8);
    }
    mbar_init(kv_full, 1);
    mbar_init(kv_empty, 1);
    mbar_init(s_full, 1);
    mbar_init(dp_full, 1);
    mbar_init(p_ready, 8);
    mbar_init(ds_ready, 8);
    mbar_init(acc_full, 1);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 9 && lane == 0) {
    tma_prefetch_desc(&mQ);
    tma_prefetch_desc(&mK);
    tma_prefetch_desc(&mV);
    tma_prefetch_desc(&mG);
  }
  if (warp == 8) {
    tmem_alloc<false>(tmem_slot, 512);
    tmem_relinquish<false>();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t tS = tmem, tP = tmem + 128, tDV = tmem + 256, tDK = tmem + 384;
  griddep_wait();
  griddep_launch_dependents();
  const int splits = reinterpret_cast<const volatile int*>(a.counts)[2];
  const int items = reinterpret_cast<const volatile int*>(a.counts)[1] * a.n_kv;
  const int step = static_cast<int>(gridDim.x), first = static_cast<int>(blockIdx.x);
  Waiter wait{abort_flag, a.status, a.timeout_ns};

  // Registers: 384 threads x 168 at launch = 256 x 216 + 128 x 72
  if (warp >= 8) {
    reg_dec<72>();
    if (warp == 9) {
      // ---------------------------------------------------------- producer
      const uint32_t el = elect_one();
      uint32_t pos = 0, iter = 0, kvn = 0;
      auto put = [&](const CUtensorMap& m, int col, int row, bool ragged) {
        const uint32_t s = pos % KV_STAGES;
        if (!wait(&empty[s], ((pos / KV_STAGES) & 1) ^ 1)) return;
        uint64_t* bar = ragged ? &raw[s] : &full[s];
        mbar_arrive_expect_tx(bar, TILE_BYTES, el);
        load_pair(ring + s * TILE_BYTES, &m, bar, col, row, el);
        ++pos;
      };
      for (int k = 0, w = first; w < items && wait.ok; w = snake_item(first, step, ++k)) {
        const KvItem it = kv_item(a, w, splits);
        if (it.n == 0) continue;
        if (!wait(kv_empty, (kvn & 1) ^ 1)) break;
        ++kvn;
        mbar_arrive_expect_tx(kv_full, 2 * TILE_BYTES, el);
        load_pair(sK, &mK, kv_full, it.kv * ATTN_D, it.t.k0 + it.t.t0, el);
        load_pair(sV, &mV, kv_full, it.kv * ATTN_D, it.t.k0 + it.t.t0, el);
        const int64_t pad = padded_row(it.t);
        for (int h = it.h0; h < it.h0 + it.nh && wait.ok; ++h) {
          for (int j = 0; j < it.n && wait.ok; ++j, ++iter) {
            const int row = (it.first + j) * ATTN_BLK;
            const bool ragged = row + ATTN_BLK > it.t.lq;
            put(mQ, h * ATTN_D, it.t.q0 + row, ragged);
            const uint32_t b = iter & 1;
            if (!wait(&row_empty[b], ((iter >> 1) & 1) ^ 1)) break;
            float* dst = rows + b * 2 * ATTN_BLK;
            mbar_arrive_expect_tx(&row_full[b], ROW_BYTES, el);
            bulk_load(dst, a.nlse2 + h * a.Tp + pad + row, ATTN_BLK * 4, &row_full[b], el);
            bulk_load(dst + ATTN_BLK, a.ndelta + h * a.Tp + pad + row, ATTN_BLK * 4, &row_full[b], el);
            put(mG, h * ATTN_D, it.t.q0 + row, ragged);
          }
        }
      }
      if (!wait.ok) let_copies_land();
    } else if (warp == 10) {
      // ---------------------------------------------------------- rows behind the sequence
      uint32_t pos = 0, seen = 0;
      for (int k = 0, w = first; w < items && wait.ok; w = snake_item(first, step, ++k)) {
        const KvItem it = kv_item(a, w, splits);
        const int last = (it.first + it.n - 1) * ATTN_BLK;
        for (int h = 0; h < it.nh && it.n > 0 && wait.ok; ++h) {
          pos += 2 * it.n;
          if (last + ATTN_BLK <= it.t.lq) continue;
          for (int x = 2; x >= 1; --x) {  // the head's last Q tile, then its dO tile
            const uint32_t s = (pos - x) % KV_STAGES;
            if (!wait.warp(&raw[s], (seen >> s) & 1)) break;
            seen ^= 1u << s;
            zero_tile_rows(ring + s * TILE_BYTES, it.t.lq - last);
            if (lane == 0) mbar_arrive(&full[s]);
          }
        }
      }
    } else if (warp == 8) {
      // ---------------------------------------------------------- UMMA issuer
      const uint32_t el = elect_one();
      uint32_t pos = 0, iter = 0, kvn = 0;
      bool issued = false;
      const uint32_t k_s = smem_u32(sK), v_s = smem_u32(sV), r_s = smem_u32(ring);
      auto stage = [&](uint32_t p) { return r_s + (p % KV_STAGES) * TILE_BYTES; };
      auto ready = [&](uint32_t p) {
        const bool ok = wait(&full[p % KV_STAGES], (p / KV_STAGES) & 1);
        tc_fence_after();
        return ok;
      };
      for (int k = 0, w = first; w < items && wait.ok; w = snake_item(first, step, ++k)) {
        const KvItem it = kv_item(a, w, splits);
        if (it.n == 0) continue;
        const int n = it.n * it.nh;
        if (!wait(kv_full, kvn & 1)) break;
        ++kvn;
        if (!ready(pos)) break;
        mma_ss(tS, k_s, stage(pos), false, el);
        issued = true;
        umma_commit(s_full, el);
        if (!ready(pos + 1)) break;
        mma_ss(tP, v_s, stage(pos + 1), false, el);
        umma_commit(dp_full, el);
        for (int i = 0; i < n; ++i, ++iter, pos += 2) {
          if (!wait(p_ready, iter & 1)) break;
          tc_fence_after();
          mma_tn(tDV, tS, stage(pos + 1), i > 0, el);
          umma_commit(&empty[(pos + 1) % KV_STAGES], el);
          if (i + 1 < n) {
            if (!ready(pos + 2)) break;
            mma_ss(tS, k_s, stage(pos + 2), false, el);
            umma_commit(s_full, el);
          }
          if (!wait(ds_ready, iter & 1)) break;
          tc_fence_after();
          mma_tn(tDK, tP, stage(pos), i > 0, el);
          umma_commit(&empty[pos % KV_STAGES], el);
          if (i + 1 < n) {
            if (!ready(pos + 3)) break;
            mma_ss(tP, v_s, stage(pos + 3), false, el);
            umma_commit(dp_full, el);
          }
          if (i + 1 == n) umma_commit(acc_full, el);
          if (i + 2 == n || n == 1) umma_commit(kv_empty, el);  // K and V have been read for the last time
        }
      }
      if (!wait.ok && issued) {
        umma_commit(drain, el);
        mbar_wait_drain(drain, 0, 200000000ull);
      }
    }
  } else {
    // ------------------------------------------------------------ P^T, dS^T
    reg_inc<216>();
    const int half = warp >> 2;
    const int r = (warp & 3) * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t mS = tS + lanes + half * 64, mP = tP + lanes + half * 64;
    const uint64_t c2 = f2_pack(a.scale_log2, a.scale_log2);
    uint32_t iter = 0, done = 0;
    for (int k = 0, w = first; w < items && wait.ok; w = snake_item(first, step, ++k)) {
      const KvItem it = kv_item(a, w, splits);
      const int off = it.t.lk - it.t.lq;
      for (int h = 0; h < it.nh && wait.ok; ++h) {
        for (int j = 0; j < it.n; ++j, ++iter) {
          const int q0 = (it.first + j) * ATTN_BLK;
          const bool diag = it.t.t0 + ATTN_BLK - 1 > q0 + off;          // some key is later than some query
          const int from = it.t.t0 + r - off - q0 - half * 64;          // first query column that sees this key
          const float* nl = rows + (iter & 1) * 2 * ATTN_BLK + half * 64;
          const float* nd = nl + ATTN_BLK;
          if (!wait.warp(&row_full[iter & 1], (iter >> 1) & 1)) break;
          if (!wait.warp(s_full, iter & 1)) break;
          tc_fence_after();
          float p[64];
          {
            uint32_t s[64];
            tmem_ld64(mS, s);
#pragma unroll
            for (int i = 0; i < 64; i += 4) {
              const float4 l4 = *reinterpret_cast<const float4*>(nl + i);
              float z0, z1, z2, z3;
              f2_unpack(f2_fma(f2_pack(__uint_as_float(s[i]), __uint_as_float(s[i + 1])), c2, f2_pack(l4.x, l4.y)), z0, z1);
              f2_unpack(f2_fma(f2_pack(__uint_as_float(s[i + 2]), __uint_as_float(s[i + 3])), c2, f2_pack(l4.z, l4.w)), z2,
                        z3);
              p[i] = exp2_sfu(z0);
              p[i + 1] = exp2_sfu(z1);
              p[i + 2] = exp2_sfu(z2);
              p[i + 3] = exp2_sfu(z3);
            }
          }
          if (diag) {
            keep_branch();
#pragma unroll
            for (int i = 0; i < 64; ++i) p[i] = i >= from ? p[i] : 0.f;
          }
          {
            uint32_t u[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) u[i] = pack_bf16x2(p[2 * i], p[2 * i + 1]);
            tmem_st32(mS, u);
          }
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(p_ready);
          if (!wait.warp(dp_full, iter & 1)) break;
          tc_fence_after();
          {
            uint32_t d[64], u[32];
            tmem_ld64(mP, d);
#pragma unroll
            for (int i = 0; i < 64; i += 4) {
              const float4 d4 = *reinterpret_cast<const float4*>(nd + i);
              const uint64_t x0 = f2_mul(f2_pack(p[i], p[i + 1]),
                                         f2_add(f2_pack(__uint_as_float(d[i]), __uint_as_float(d[i + 1])),
                                                f2_pack(d4.x, d4.y)));
              const uint64_t x1 = f2_mul(f2_pack(p[i + 2], p[i + 3]),
                                         f2_add(f2_pack(__uint_as_float(d[i + 2]), __uint_as_float(d[i + 3])),
                                                f2_pack(d4.z, d4.w)));
              float e0, e1, e2, e3;
              f2_unpack(x0, e0, e1);
              f2_unpack(x1, e2, e3);
              u[i / 2] = pack_bf16x2(e0, e1);
              u[i / 2 + 1] = pack_bf16x2(e2, e3);
            }
            tmem_st32(mP, u);
          }
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(ds_ready);
            mbar_arrive(&row_empty[iter & 1]);
          }
        }
      }
      if (!wait.ok) break;
      // warpgroup 0 writes dV, warpgroup 1 dK
      const int key = it.t.t0 + r;
      const bool valid = key < it.t.lk;
      const float f = half ? a.scale : 1.f;
      const uint32_t src = (half ? tDK : tDV) + lanes;
      if (it.n > 0) {
        if (!wait.warp(acc_full, done & 1)) break;
        ++done;
        tc_fence_after();
      }
      if (it.part >= 0) {
        // column by column of four, rows side by side
        float4* dst = reinterpret_cast<float4*>(a.part + (it.part * 2 + half) * ATTN_BLK * ATTN_D) + r;
#pragma unroll 1
        for (int q = 0; q < 4; ++q) {
          float v[32];
          if (it.n > 0) {
            __syncwarp();
            tmem_ld32(src + q * 32, v);
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = 0.f;
          }
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (valid) dst[(q * 8 + i) * ATTN_BLK] = make_float4(v[4 * i] * f, v[4 * i + 1] * f, v[4 * i + 2] * f, v[4 * i + 3] * f);
        }
      } else {
        __nv_bfloat16* dst = (half ? a.dK : a.dV) + ((static_cast<int64_t>(it.t.k0) + key) * a.n_kv + it.kv) * ATTN_D;
        if (it.n > 0) {
          store_row64(src, dst, f, valid);
          store_row64(src + 64, dst + 64, f, valid);
        } else if (valid) {
#pragma unroll
          for (int i = 0; i < 16; ++i) *reinterpret_cast<uint4*>(dst + i * 8) = make_uint4(0, 0, 0, 0);
        }
      }
      tc_fence_before();
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 8) {
    __syncwarp();
    tmem_dealloc<false>(tmem, 512);
  }
}

// Adds the parts of a key tile's dV and dK: a thread takes one row and eight
// columns, a block 256 of the 2 * 2048 such pieces of a (key tile, head) at a
// time, so the loads of all parts are in flight at once.
__global__ void __launch_bounds__(256) attn_bwd_join_kernel(const AttnBwdArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const int splits = reinterpret_cast<const volatile int*>(a.counts)[2];
  const int cuts = reinterpret_cast<const volatile int*>(a.counts)[3];
  for (int w = blockIdx.x; w < cuts * a.n_kv * 16; w += gridDim.x) {
    const int which = (w >> 3) & 1;  // 0: dV
    const int at = w >> 4;           // key tile, head
    const int ti = at / a.n_kv, kv = at - ti * a.n_kv;
    const AttnTile t = load_tile(a.cuts + ti);
    const int u = (w & 7) * 256 + static_cast<int>(threadIdx.x);
    const int row = u & (ATTN_BLK - 1), c8 = u >> 7;
    if (t.t0 + row >= t.lk) continue;
    const int64_t part = static_cast<int64_t>(at) * splits;  // t.slot is ti * splits
    const float4* src =
        reinterpret_cast<const float4*>(a.part + (part * 2 + which) * ATTN_BLK * ATTN_D) + 2 * c8 * ATTN_BLK + row;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int p = 0; p < splits; ++p) {
      const float4* s = src + static_cast<int64_t>(p) * 2 * ATTN_BLK * ATTN_D / 4;
      const float4 x = s[0], y = s[ATTN_BLK];
      v[0] += x.x; v[1] += x.y; v[2] += x.z; v[3] += x.w;
      v[4] += y.x; v[5] += y.y; v[6] += y.z; v[7] += y.w;
    }
    store_bf16x8((which ? a.dK : a.dV) + ((static_cast<int64_t>(t.k0) + t.t0 + row) * a.n_kv + kv) * ATTN_D + c8 * 8, v);
  }
}

// ------------------------------------------------------------------ dQ
// Item: a tile of 128 queries of one head; it meets the key blocks it sees.
//
//   TMEM  S 128 | dP 128 | dQ 128 | dS 64 | dO 64 (the A operand of dP)
//   UMMA  S = Q K^T | dP = dO V^T | dQ += dS K of the block before
//
// The three products of a block have places of their own, so the tensor core
// always has work that does not wait for the arithmetic in front of it, and
// the blocks of all items form one stream: the first scores of the next item
// are under way while the last dQ product of this one runs, and dQ leaves
// between the two arithmetic steps of the next item's first block.
//
//   warps 0-7   thread = query row, warpgroup = half of the 128 keys:
//               E1 p = exp2(S c - lse2);  E2 dS = p (dP - D), bf16.
//               Warpgroup 1 also moves the next dO to TMEM and forms D.
//   warp 8      UMMA issuer      warp 9  TMA      warp 10  K rows behind the sequence
//
// Ring order of an item: dO, O, K0, V0, K1, V1, ...; Q has a buffer.  A block's
// K stays until its dQ product, which runs behind the next block's dP: that
// one's V lies three places on, within the ring.  The next item's first V lies
// five places behind this item's last K, so there the dQ product runs first.
//
// Measured: 4 sequences of 2048 tokens, 64 + 8 heads (three products, 413 GFLOP)
// 361 us, 1140 TFLOP/s, the tensor pipe active 50 %.  A block takes about 3000
// clocks, more than its arithmetic (2000 in two warpgroups) or its three products
// (2100): one 128-row tile is in flight, so E1, E2 and the products wait for one
// another in turn.  A form of 370 us took 367 without the exponentials, 357
// without the loads, 321 without the products.
struct QItem {
  AttnTile t;
  int head, n;
};
__device__ __forceinline__ QItem q_item(const AttnBwdArgs& a, int w) {
  QItem it;
  const int ti = w / a.n_q;
  it.head = w - ti * a.n_q;
  it.t = load_tile(a.q_tiles + ti);
  it.n = key_blocks(it.t, min(it.t.t0 + ATTN_BLK, it.t.lq) - 1);
  return it;
}
__device__ __forceinline__ uint32_t ring_k(uint32_t pos, int j) { return pos + 2 + 2 * j; }
__device__ __forceinline__ uint32_t ring_v(uint32_t pos, int j) { return pos + 3 + 2 * j; }

__global__ void __launch_bounds__(BWD_THREADS, 1)
    attn_bwd_q_kernel(const __grid_constant__ CUtensorMap mQ, const __grid_constant__ CUtensorMap mK,
                      const __grid_constant__ CUtensorMap mV, const __grid_constant__ CUtensorMap mG,
                      const __grid_constant__ CUtensorMap mO, const AttnBwdArgs a) {
  extern __shared__ __align__(1024) uint8_t bwd_smem[];
  uint8_t* sQ = bwd_smem;
  uint8_t* ring = sQ + TILE_BYTES;
  uint64_t* full = reinterpret_cast<uint64_t*>(ring + Q_STAGES * TILE_BYTES);
  uint64_t* empty = full + Q_STAGES;
  uint64_t* raw = empty + Q_STAGES;
  uint64_t* q_full = raw + Q_STAGES;
  uint64_t* q_empty = q_full + 1;
  uint64_t* g_ready = q_empty + 1;   // dO is in TMEM
  uint64_t* s_full = g_ready + 1;
  uint64_t* s_read = s_full + 1;
  uint64_t* dp_full = s_read + 1;
  uint64_t* dp_read = dp_full + 1;
  uint64_t* ds_ready = dp_read + 1;
  uint64_t* dq_done = ds_ready + 1;  // the block's dQ product has read dS
  uint64_t* d_ready = dq_done + 1;
  uint64_t* x_ready = d_ready + 1;
  uint64_t* drain = x_ready + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  static_assert((3 * Q_STAGES + 12) * 8 + 8 <= 512, "barrier area");
  float* row_d = reinterpret_cast<float*>(ring + Q_STAGES * TILE_BYTES + 512);  // D of the item's rows
  float* row_x = row_d + ATTN_BLK;                                   // two half sums of p dP

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < Q_STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
      mbar_init(&raw[s], 1);
    }
    mbar_init(q_full, 1);
    mbar_init(q_empty, 1);
    mbar_init(g_ready, 4);
    mbar_init(s_full, 1);
    mbar_init(s_read, 8);
    mbar_init(dp_full, 1);
    mbar_init(dp_read, 8);
    mbar_init(ds_ready, 8);
    mbar_init(dq_done, 1);
    mbar_init(d_ready, 4);
    mbar_init(x_ready, 8);
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 9 && lane == 0) {
    tma_prefetch_desc(&mQ);
    tma_prefetch_desc(&mK);
    tma_prefetch_desc(&mV);
    tma_prefetch_desc(&mG);
    tma_prefetch_desc(&mO);
  }
  if (warp == 8) {
    tmem_alloc<false>(tmem_slot, 512);
    tmem_relinquish<false>();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t tS = tmem, tP = tmem + 128, tDQ = tmem + 256, tDS = tmem + 384, tG = tmem + 448;
  griddep_wait();
  griddep_launch_dependents();
  const int items = *reinterpret_cast<const volatile int*>(a.counts) * a.n_q;
  const int step = static_cast<int>(gridDim.x), first = static_cast<int>(blockIdx.x);
  Waiter wait{abort_flag, a.status, a.timeout_ns};

  if (warp >= 8) {
    reg_dec<72>();
    if (warp == 9) {
      // ---------------------------------------------------------- producer
      const uint32_t el = elect_one();
      uint32_t pos = 0, qn = 0;
      auto put = [&](const CUtensorMap& m, int col, int row, bool ragged) {
        const uint32_t s = pos % Q_STAGES;
        if (!wait(&empty[s], ((pos / Q_STAGES) & 1) ^ 1)) return;
        uint64_t* bar = ragged ? &raw[s] : &full[s];
        mbar_arrive_expect_tx(bar, TILE_BYTES, el);
        load_pair(ring + s * TILE_BYTES, &m, bar, col, row, el);
        ++pos;
      };
      for (int k = 0, w = first; w < items && wait.ok; w = snake_item(first, step, ++k)) {
        const QItem it = q_item(a, w);
        if (it.n == 0) continue;
        const int col = it.head / a.group * ATTN_D, qcol = it.head * ATTN_D, qrow = it.t.q0 + it.t.t0;
        put(mG, qcol, qrow, false);
        if (wait.ok) put(mO, qcol, qrow, false);
        if (!wait(q_empty, (qn & 1) ^ 1)) break;
        ++qn;
        mbar_arrive_expect_tx(q_full, TILE_BYTES, el);
        load_pair(sQ, &mQ, q_full, qcol, qrow, el);
        for (int j = 0; j < it.n && wait.ok; ++j) {
          const int row = j * ATTN_BLK;
          put(mK, col, it.t.k0 + row, row + ATTN_BLK > it.t.lk);
          if (wait.ok) put(mV, col, it.t.k0 + row, false);
        }
      }
      if (!wait.ok) let_copies_land();
    } else if (warp == 10) {
      // ---------------------------------------------------------- K rows behind the sequence
      uint32_t pos = 0, seen = 0;
      for (int k = 0, w = first; w < items && wait.ok; w = snake_item(first, step, ++k)) {
        const QItem it = q_item(a, w);
        if (it.n == 0) continue;
        const uint32_t s = ring_k(pos, it.n - 1) % Q_STAGES;
        pos += 2 + 2 * it.n;
        if (it.n * ATTN_BLK <= it.t.lk) continue;
        if (!wait.warp(&raw[s], (seen >> s) & 1)) break;
        seen ^= 1u << s;
        zero_tile_rows(ring + s * TILE_BYTES, it.t.lk - (it.n - 1) * ATTN_BLK);
        if (lane == 0) mbar_arrive(&full[s]);
      }
    } else if (warp == 8) {
      // ---------------------------------------------------------- UMMA issuer
      const uint32_t el = elect_one();
      uint32_t pos = 0, iter = 0, itn = 0, k_before = 0;
      bool acc = false;  // of the dQ product that is due
      const uint32_t q_s = smem_u32(sQ), r_s = smem_u32(ring);
      auto stage = [&](uint32_t p) { return r_s + (p % Q_STAGES) * TILE_BYTES; };
      auto ready = [&](uint32_t p) {
        const bool ok = wait(&full[p % Q_STAGES], (p / Q_STAGES) & 1);
        tc_fence_after();
        return ok;
      };
      auto before = [&](uint64_t* bar) {  // the previous block's arrival on `bar` (none for the first)
        const bool ok = iter == 0 || wait(bar, (iter - 1) & 1);
        tc_fence_after();
        return ok;
      };
      auto product_dq = [&] {
        constexpr uint32_t ID = idesc_bf16(128, 128, 0, 1);
        const uint32_t b = stage(k_before);
#pragma unroll
        for (int i = 0; i < 8; ++i)
          umma_bf16_ts(tDQ, tDS + i * 8, sdesc_sw128(b + i * 2048, HALF_BYTES, 1024), ID, acc || i > 0, el);
        umma_commit(&empty[k_before % Q_STAGES], el);
        umma_commit(dq_done, el);
      };
      for (int k = 0, w = first; w < items && wait.ok; w = snake_item(first, step, ++k)) {
        const QItem it = q_item(a, w);
        if (it.n == 0) continue;
        for (int j = 0; j < it.n; ++j) {
          const uint32_t kp = ring_k(pos, j), vp = ring_v(pos, j);
          if (!ready(kp) || (j == 0 && !wait(q_full, itn & 1)) || !before(s_read)) break;
          mma_ss(tS, q_s, stage(kp), false, el);
          umma_commit(s_full, el);
          if (j + 1 == it.n) umma_commit(q_empty, el);
          if (j == 0) {
            if (!wait(g_ready, itn & 1)) break;
            tc_fence_after();
            if (el) {  // dO and O have left the ring
              mbar_arrive(&empty[pos % Q_STAGES]);
              mbar_arrive(&empty[(pos + 1) % Q_STAGES]);
            }
            __syncwarp();
            if (iter > 0) {
              if (!before(ds_ready)) break;
              product_dq();
            }
          }
          if (!ready(vp) || !before(dp_read)) break;
          mma_ts(tP, tG, stage(vp), false, el);
          umma_commit(dp_full, el);
          umma_commit(&empty[vp % Q_STAGES], el);
          if (j > 0) {
            if (!before(ds_ready)) break;
            product_dq();
          }
          k_before = kp;
          acc = j > 0;
          ++iter;
        }
        pos += 2 + 2 * it.n;
        ++itn;
      }
      if (wait.ok && iter > 0 && before(ds_ready)) product_dq();
      if (!wait.ok) {
        umma_commit(drain, el);
        mbar_wait_drain(drain, 0, 200000000ull);
      }
    }
  } else {
    // ------------------------------------------------------------ P, dS, dO and D
    reg_inc<216>();
    const int half = warp >> 2;
    const int r = (warp & 3) * 32 + lane;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t mS = tS + lanes + half * 64, mP = tP + lanes + half * 64, mDS = tDS + lanes + half * 32;
    const uint64_t c2 = f2_pack(a.scale_log2, a.scale_log2);
    uint32_t iter = 0, itn = 0, xn = 0, pos = 0;

    // dQ of a finished item, this warpgroup's 64 columns.  (Through boxes in
    // shared memory the stores would cover whole lines; a sixth ring stage is
    // worth more.)
    auto leave = [&](const QItem& y) {
      __nv_bfloat16* dst = a.dQ + ((static_cast<int64_t>(y.t.q0) + y.t.t0 + r) * a.n_q + y.head) * ATTN_D + half * 64;
      store_row64(tDQ + lanes + half * 64, dst, a.scale, y.t.t0 + r < y.t.lq);
      tc_fence_before();
    };

    QItem was;  // the item whose dQ is still in TMEM
    was.n = 0;
    for (int k = 0, w = first; w < items && wait.ok; w = snake_item(first, step, ++k)) {
      const QItem it = q_item(a, w);
      const int row = it.t.t0 + r;
      const int vis = min(it.t.lk, row + 1 + it.t.lk - it.t.lq);
      const int all = it.t.t0 + 1 + it.t.lk - it.t.lq;  // keys every row sees
      // the row's -lse2 and -D (0 weight: behind the sequence, or no key)
      const int64_t pr = it.head * a.Tp + padded_row(it.t) + row;
      const bool seen = row < it.t.lq && vis > 0;
      const float nl = seen ? -__ldcg(a.lse + static_cast<int64_t>(it.head) * a.Tq + it.t.q0 + row) * 1.4426950408889634f
                            : -INFINITY;
      if (it.n == 0) {
        if (half == 0) {
          a.nlse2[pr] = nl;
          a.ndelta[pr] = 0.f;
        }
        if (row < it.t.lq) {
          __nv_bfloat16* dst = a.dQ + ((static_cast<int64_t>(it.t.q0) + row) * a.n_q + it.head) * ATTN_D + half * 64;
#pragma unroll
          for (int i = 0; i < 8; ++i) *reinterpret_cast<uint4*>(dst + i * 8) = make_uint4(0, 0, 0, 0);
        }
        continue;
      }
      if (half) {
        // dO to TMEM (dP of the item before is complete: E2 has waited for
        // it), and D = dO . O for both warpgroups
        const uint32_t at = pos;
        auto piece = [&](uint32_t p, int i) {
          return *reinterpret_cast<const uint4*>(ring + (p % Q_STAGES) * TILE_BYTES + (i >> 3) * HALF_BYTES + r * 128 +
                                                 (((i & 7) ^ (r & 7)) << 4));
        };
        if (!wait.warp(&full[at % Q_STAGES], (at / Q_STAGES) & 1)) break;
        if (!wait.warp(&full[(at + 1) % Q_STAGES], ((at + 1) / Q_STAGES) & 1)) break;
        float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t v[32];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const uint4 g = piece(at, 8 * h + i);
            float x[8], y[8];
            bf16x8_to_f32(piece(at + 1, 8 * h + i), x);
            bf16x8_to_f32(g, y);
#pragma unroll
            for (int e = 0; e < 8; ++e) d[e & 3] = fmaf(x[e], y[e], d[e & 3]);
            v[4 * i] = g.x;
            v[4 * i + 1] = g.y;
            v[4 * i + 2] = g.z;
            v[4 * i + 3] = g.w;
          }
          tmem_st32(tG + lanes + 32 * h, v);
        }
        row_d[r] = (d[0] + d[1]) + (d[2] + d[3]);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(g_ready);
          mbar_arrive(d_ready);
        }
      }
      pos += 2 + 2 * it.n;
      if (!wait.warp(d_ready, itn & 1)) break;
      ++itn;
      float nd = seen ? -row_d[r] : 0.f;
      if (half == 0) {
        a.nlse2[pr] = nl;
        if (it.n != 1) a.ndelta[pr] = nd;
      }
      const uint64_t nl2 = f2_pack(nl, nl);
      for (int j = 0; j < it.n; ++j, ++iter) {
        const bool diag = (j + 1) * ATTN_BLK > all;
        const int lim = vis - j * ATTN_BLK - half * 64;
        if (!wait.warp(s_full, iter & 1)) break;
        tc_fence_after();
        float p[64];
        {
          uint32_t s[64];
          tmem_ld64(mS, s);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(s_read);
#pragma unroll
          for (int i = 0; i < 64; i += 2) {
            float z0, z1;
            f2_unpack(f2_fma(f2_pack(__uint_as_float(s[i]), __uint_as_float(s[i + 1])), c2, nl2), z0, z1);
            p[i] = exp2_sfu(z0);
            p[i + 1] = exp2_sfu(z1);
          }
        }
        const bool flush = j == 0 && was.n > 0;
        if (flush) {
          if (!wait.warp(dq_done, (iter - 1) & 1)) break;
          tc_fence_after();
          leave(was);
        }
        if (!wait.warp(dp_full, iter & 1)) break;
        tc_fence_after();
        uint32_t u[32];
        {
          uint32_t d[64];
          tmem_ld64(mP, d);
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(dp_read);
          if (it.n == 1) {
            keep_branch();
            float t[2] = {0.f, 0.f};
#pragma unroll
            for (int i = 0; i < 64; ++i) t[i & 1] += i < lim ? p[i] * __uint_as_float(d[i]) : 0.f;
            row_x[half * ATTN_BLK + r] = t[0] + t[1];
            __syncwarp();
            if (lane == 0) mbar_arrive(x_ready);
            if (!wait.warp(x_ready, xn & 1)) break;
            ++xn;
            nd = seen ? -(row_x[r] + row_x[ATTN_BLK + r]) : 0.f;
            if (half == 0) a.ndelta[pr] = nd;
          }
          if (diag) {
            // masked keys: weight 0 and a dP that cannot make it NaN
            keep_branch();
#pragma unroll
            for (int i = 0; i < 64; ++i) {
              p[i] = i < lim ? p[i] : 0.f;
              d[i] = i < lim ? d[i] : 0u;
            }
          }
          const uint64_t nd2 = f2_pack(nd, nd);
#pragma unroll
          for (int i = 0; i < 64; i += 2) {
            float e0, e1;
            f2_unpack(f2_mul(f2_pack(p[i], p[i + 1]),
                             f2_add(f2_pack(__uint_as_float(d[i]), __uint_as_float(d[i + 1])), nd2)),
                      e0, e1);
            u[i / 2] = pack_bf16x2(e0, e1);
          }
        }
        if (iter > 0 && !flush && !wait.warp(dq_done, (iter - 1) & 1)) break;  // dS may be replaced
        tmem_st32(mDS, u);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(ds_ready);
      }
      was = it;
    }
    if (wait.ok && was.n > 0 && wait.warp(dq_done, (iter - 1) & 1)) {
      tc_fence_after();
      leave(was);
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 8) {
    __syncwarp();
    tmem_dealloc<false>(tmem, 512);
  }
}

}  // namespace

cudaError_t launch_attn_bwd(const AttnBwdArgs& a, const CUtensorMap* maps, int64_t max_q_tiles, int64_t max_k_tiles,
                            int sms, cudaStream_t s) {
  cudaError_t e = attn_smem_attribute(reinterpret_cast<const void*>(attn_bwd_kv_kernel), 3, KV_SMEM);
  if (e != cudaSuccess) return e;
  e = attn_smem_attribute(reinterpret_cast<const void*>(attn_bwd_q_kernel), 4, Q_SMEM);
  if (e != cudaSuccess) return e;
  if (max_q_tiles > 0) {
    e = attn_launch(attn_bwd_q_kernel, std::min<int64_t>(sms, max_q_tiles * a.n_q), BWD_THREADS, Q_SMEM, s, maps[0], maps[1],
               maps[2], maps[3], maps[4], a);
    if (e != cudaSuccess) return e;
  }
  if (max_k_tiles == 0) return cudaSuccess;
  e = attn_launch(attn_bwd_kv_kernel, std::min<int64_t>(sms, max_k_tiles * a.n_kv * (a.max_parts ? a.group : 1)), BWD_THREADS,
             KV_SMEM, s, maps[0], maps[1], maps[2], maps[3], a);
  if (e != cudaSuccess || a.max_parts == 0) return e;
  return attn_launch(attn_bwd_join_kernel, std::min<int64_t>(max_k_tiles * a.n_kv * 16, 8 * sms), 256, 0, s, a);
}

}  // namespace coda

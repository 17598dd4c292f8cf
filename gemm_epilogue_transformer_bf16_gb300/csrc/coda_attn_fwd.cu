// Causal attention over packed sequences, forward.
//
//   s_ij = scale q_i . k_j  (j <= i + lk - lq),  lse_i = log sum_j exp s_ij,
//   o_i  = sum_j exp(s_ij - lse_i) v_j
//
// in one pass over the keys with the running maximum m and sum l of each row
// (the attention core between the QKV projection and the output projection
// of the block).  Tensor bound: 2 * 128 multiply-adds (4 * 128 operations) per
// visible pair and head against 512 bytes of K and V per key, shared by a
// 256-row item.
//
// One persistent CTA per SM walks the work list.  An item is two 128-row
// query tiles of one key/value head -- two sets of query heads on the same
// tokens when the group is even, else consecutive tokens -- so every K and V
// block in shared memory feeds two tiles:
//
//   warps 0-3    softmax of tile 0: thread = row.  128 scores come from TMEM
//   warps 4-7    softmax of tile 1  into registers, the weights go back as
//                                   bf16 over the scores, and are the A
//                                   operand of the P V product from there.
//   warp 8       UMMA issuer: S0 S1 | P0V S0' | P1V S1' ...  While one tile's
//                softmax runs, the tensor core works for the other tile.
//   warp 9       TMA producer: Q tiles, and a ring of K and V blocks.
//   warp 10      zeroes the rows of a V block that lie behind the sequence.
//
// TMEM: S0 S1 (128 fp32 columns each, P in the lower 64) and O0 O1.  The
// accumulator O is rescaled only when a row's maximum has risen by more than
// 2^8 over the one its weights refer to (weights stay below 256, which bf16
// and the fp32 sums hold without loss); the tile's P V product of the
// previous block is complete by then, since S of this block was issued
// behind it.
//
// Measured: 4 sequences of 2048 tokens, 64 + 8 heads (275 GFLOP over the visible
// pairs) 209 us, 1320 TFLOP/s; one of 16384 tokens, 32 + 8 heads 1280 us, 1720.
// The long one is bound by the products: the two of a 128 x 128 block take 1250
// to 1400 clocks with N = 128 and one CTA (1024 at the pipe's rate).  The first,
// with the masked halves of its diagonal blocks, would take 169 us at that rate;
// the other 40 are 3 us at the ends of each of an SM's 13.5 items, the first
// softmax and O leaving without products beside them (O alone 20 us; four warps
// of their own for it took registers from the others: 226 to 270 us).  The tensor
// pipe is active 59 % of the first.
//
// Few rows over many keys leave most SMs without an item: then the keys of the
// longer runs are cut into parts (attn_plan_kernel), which leave normalised
// fp32 outputs and log-sum-exps that a second kernel joins in fixed order.
// 16 rows over 100000 keys, 64 + 8 heads: 989 -> 84 us.
//
// Roundings: P to bf16 before the second product (the sum l adds the fp32
// weights), O to bf16 once at the end.
#include <algorithm>

#include "coda_attn.cuh"
#include "coda_internal.h"
#include "coda_status.h"

namespace coda {
namespace {

constexpr int FWD_THREADS = 384;
constexpr int FWD_STAGES = 4;
constexpr uint32_t TILE_BYTES = ATTN_BLK * ATTN_D * 2;  // 32 KB
constexpr uint32_t HALF_BYTES = TILE_BYTES / 2;         // 64 columns
constexpr uint32_t FWD_OUT = 8 * 4096;  // 32 rows x 64 columns of O per softmax warp, on their way to memory
constexpr uint32_t FWD_SMEM = 1024 + (2 + FWD_STAGES) * TILE_BYTES + FWD_OUT + 512;
static_assert(FWD_SMEM <= 232448, "shared memory per CTA");

struct FwdItem {
  AttnTile t;
  int head[2], row[2], n[2];  // per tile: first head, first row of the sequence, key blocks (0: none)
  int kv;
};

// The softmax warps load the next item's entry before O leaves, when no scores
// are held (4 x 2048 tokens 214 -> 210 us); one whole item ahead the registers
// cost more than the latency (16384 tokens 1295 -> 1375 us).
__device__ __forceinline__ FwdItem fwd_item(const AttnFwdArgs& a, int w) {
  FwdItem it;
  const int hp = 1 << a.head_shift;
  const int per = a.n_q >> (a.head_shift + a.pair_heads);
  const int ti = w / per, hi = w - ti * per;
  it.t = load_tile(a.tiles + ti);
  const int span = ATTN_BLK >> a.head_shift;  // tokens of a tile
  it.head[0] = hi << (a.head_shift + a.pair_heads);
  it.head[1] = a.pair_heads ? it.head[0] + hp : it.head[0];
  it.row[0] = it.t.t0;
  it.row[1] = a.pair_heads ? it.t.t0 : it.t.t0 + span;
  it.kv = it.head[0] / a.group;
#pragma unroll
  for (int x = 0; x < 2; ++x)
    it.n[x] = it.row[x] < it.t.lq ? key_blocks(it.t, min(it.row[x] + span, it.t.lq) - 1) : 0;
  if (it.t.slot >= 0) {  // a part of the keys
    const int len = __ldcg(a.counts + 2);
#pragma unroll
    for (int x = 0; x < 2; ++x) it.n[x] = max(0, min(it.n[x] - it.t.block, len));
  }
  return it;
}

__global__ void __launch_bounds__(FWD_THREADS, 1)
    attn_fwd_kernel(const __grid_constant__ CUtensorMap mQ, const __grid_constant__ CUtensorMap mK,
                    const __grid_constant__ CUtensorMap mV, const AttnFwdArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* sQ = smem;
  uint8_t* sKV = smem + 2 * TILE_BYTES;
  uint8_t* sO = sKV + FWD_STAGES * TILE_BYTES;
  uint64_t* kv_full = reinterpret_cast<uint64_t*>(sO + FWD_OUT);
  uint64_t* kv_empty = kv_full + FWD_STAGES;
  uint64_t* kv_raw = kv_empty + FWD_STAGES;  // a V block that still has to be cleared behind the sequence
  uint64_t* q_full = kv_raw + FWD_STAGES;
  uint64_t* q_empty = q_full + 2;
  uint64_t* s_full = q_empty + 2;
  uint64_t* p_full = s_full + 2;
  uint64_t* o_full = p_full + 2;
  uint64_t* drain = o_full + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  static_assert((3 * FWD_STAGES + 11) * 8 + 8 <= 512, "barrier area");

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < FWD_STAGES; ++s) {
      mbar_init(&kv_full[s], 1);
      mbar_init(&kv_empty[s], 1);
      mbar_init(&kv_raw[s], 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&q_full[x], 1);
      mbar_init(&q_empty[x], 1);
      mbar_init(&s_full[x], 1);
      mbar_init(&p_full[x], 4);
      mbar_init(&o_full[x], 1);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 9 && lane == 0) {
    tma_prefetch_desc(&mQ);
    tma_prefetch_desc(&mK);
    tma_prefetch_desc(&mV);
  }
  if (warp == 8) {
    tmem_alloc<false>(tmem_slot, 512);
    tmem_relinquish<false>();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  griddep_wait();
  griddep_launch_dependents();
  const int items = __ldcg(a.counts) * (a.n_q >> (a.head_shift + a.pair_heads));
  const int step = static_cast<int>(gridDim.x), first = static_cast<int>(blockIdx.x);
  bool ok = true;

  // Registers: 384 threads x 168 at launch = 256 x 200 + 128 x 104.  Each
  // branch below begins with its own share, so the compiler sees it.
  if (warp >= 8) {
  reg_dec<104>();
  if (warp == 9) {
    // ------------------------------------------------------------ producer
    const uint32_t el = elect_one();
    uint32_t pos = 0, qn[2] = {0, 0};
    auto put = [&](const CUtensorMap& m, int col, int row, bool ragged) {
      const uint32_t s = pos % FWD_STAGES, ph = (pos / FWD_STAGES) & 1;
      if (!mbar_wait_bounded(&kv_empty[s], ph ^ 1, abort_flag, a.status, a.timeout_ns)) return false;
      uint64_t* bar = ragged ? &kv_raw[s] : &kv_full[s];
      mbar_arrive_expect_tx(bar, TILE_BYTES, el);
      tma_load_2d(sKV + s * TILE_BYTES, &m, bar, col, row, el);
      tma_load_2d(sKV + s * TILE_BYTES + HALF_BYTES, &m, bar, col + 64, row, el);
      ++pos;
      return true;
    };
    for (int k = 0, w = first; w < items && ok; w = snake_item(first, step, ++k)) {
      const FwdItem it = fwd_item(a, w);
      const int n = max(it.n[0], it.n[1]);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (!ok) break;
        if (it.n[x] > 0) {
          ok = mbar_wait_bounded(&q_empty[x], (qn[x] & 1) ^ 1, abort_flag, a.status, a.timeout_ns);
          if (!ok) break;
          ++qn[x];
          uint8_t* q = sQ + x * TILE_BYTES;
          mbar_arrive_expect_tx(&q_full[x], TILE_BYTES, el);
          tma_load_3d(q, &mQ, &q_full[x], 0, it.head[x], it.t.q0 + it.row[x], el);
          tma_load_3d(q + HALF_BYTES, &mQ, &q_full[x], 64, it.head[x], it.t.q0 + it.row[x], el);
        }
        if (x == 0 && n > 0) ok = put(mK, it.kv * ATTN_D, it.t.k0 + it.t.block * ATTN_BLK, false);
      }
      for (int j = 0; j < n && ok; ++j) {
        const int row = (it.t.block + j) * ATTN_BLK;
        ok = put(mV, it.kv * ATTN_D, it.t.k0 + row, row + ATTN_BLK > it.t.lk);
        if (ok && j + 1 < n) ok = put(mK, it.kv * ATTN_D, it.t.k0 + row + ATTN_BLK, false);
      }
    }
    if (!ok) {
      // let every copy already issued land before the CTA's memory is reused
      const uint64_t t0 = globaltimer_ns();
      while (globaltimer_ns() - t0 < 2000000ull) {
      }
    }
  } else if (warp == 10) {
    // ------------------------------------------------------------ rows behind the sequence
    uint32_t pos = 0, seen = 0;  // seen: bit s = parity of kv_raw[s]'s next phase
    for (int k = 0, w = first; w < items && ok; w = snake_item(first, step, ++k)) {
      const FwdItem it = fwd_item(a, w);
      const int n = max(it.n[0], it.n[1]);
      const int end = it.t.block + n;
      if (n > 0 && end * ATTN_BLK > it.t.lk) {
        const uint32_t s = (pos + 2 * n - 1) % FWD_STAGES;  // the item's last V block
        ok = mbar_wait_bounded(&kv_raw[s], (seen >> s) & 1, abort_flag, a.status, a.timeout_ns);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        seen ^= 1u << s;
        zero_tile_rows(sKV + s * TILE_BYTES, it.t.lk - (end - 1) * ATTN_BLK);
        if (lane == 0) mbar_arrive(&kv_full[s]);
      }
      pos += 2 * n;
    }
  } else if (warp == 8) {
    // ------------------------------------------------------------ UMMA issuer
    const uint32_t el = elect_one();
    constexpr uint32_t ID_S = idesc_bf16(128, 128, 0, 0);
    constexpr uint32_t ID_O = idesc_bf16(128, 128, 0, 1);
    uint32_t pos = 0, qn[2] = {0, 0}, pn[2] = {0, 0};
    bool issued = false;
    auto wait = [&](uint64_t* bar, uint32_t parity) {
      ok = mbar_wait_bounded(bar, parity, abort_flag, a.status, a.timeout_ns);
      tc_fence_after();
      return ok;
    };
    auto score = [&](int x, uint32_t kpos) {  // S_x = Q_x K^T
      const uint32_t q = smem_u32(sQ + x * TILE_BYTES), k = smem_u32(sKV + (kpos % FWD_STAGES) * TILE_BYTES);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t o = (i >> 2) * HALF_BYTES + (i & 3) * 32;
        umma_bf16(tmem + x * 128, sdesc_sw128(q + o, 16, 1024), sdesc_sw128(k + o, 16, 1024), ID_S, i > 0, el);
      }
      umma_commit(&s_full[x], el);
      issued = true;
    };
    for (int k = 0, w = first; w < items && ok; w = snake_item(first, step, ++k)) {
      const FwdItem it = fwd_item(a, w);
      const int n = max(it.n[0], it.n[1]);
      if (n == 0) continue;
      if (!wait(&kv_full[pos % FWD_STAGES], (pos / FWD_STAGES) & 1)) break;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (!ok || it.n[x] == 0) continue;
        if (!wait(&q_full[x], qn[x] & 1)) break;
        ++qn[x];
        score(x, pos);
        if (it.n[x] == 1) umma_commit(&q_empty[x], el);
      }
      if (!ok) break;
      umma_commit(&kv_empty[pos % FWD_STAGES], el);
      for (int j = 0; j < n && ok; ++j) {
        const uint32_t vpos = pos + 2 * j + 1, kpos = vpos + 1, vs = vpos % FWD_STAGES;
        if (!wait(&kv_full[vs], (vpos / FWD_STAGES) & 1)) break;
        const uint32_t v = smem_u32(sKV + vs * TILE_BYTES);
        bool k_here = false;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          if (j < it.n[x]) {
            if (!wait(&p_full[x], pn[x] & 1)) break;
            ++pn[x];
#pragma unroll
            for (int i = 0; i < 8; ++i)  // O_x += P_x V, 16 keys a step
              umma_bf16_ts(tmem + 256 + x * 128, tmem + x * 128 + i * 8, sdesc_sw128(v + i * 2048, HALF_BYTES, 1024),
                           ID_O, (j | i) > 0, el);
            if (j + 1 == it.n[x]) umma_commit(&o_full[x], el);
          }
          if (x == 1) umma_commit(&kv_empty[vs], el);
          if (j + 1 < it.n[x]) {
            if (!k_here && !wait(&kv_full[kpos % FWD_STAGES], (kpos / FWD_STAGES) & 1)) break;
            k_here = true;
            score(x, kpos);
            if (j + 2 == it.n[x]) umma_commit(&q_empty[x], el);
          }
        }
        if (ok && j + 1 < n) umma_commit(&kv_empty[kpos % FWD_STAGES], el);
      }
      pos += 2 * n;
    }
    if (!ok && issued) {
      umma_commit(drain, el);
      mbar_wait_drain(drain, 0, 200000000ull);
    }
  }
  } else {
    // ------------------------------------------------------------ softmax
    reg_inc<200>();
    const int x = warp >> 2;
    const int r = (warp & 3) * 32 + lane;  // row of the tile
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lanes + x * 128, tO = tmem + lanes + 256 + x * 128;
    const int tok = r >> a.head_shift, hd = r & ((1 << a.head_shift) - 1);
    const float c = a.scale_log2;
    uint32_t sn = 0, on = 0;
    FwdItem it = first < items ? fwd_item(a, first) : FwdItem{};
    for (int k = 0, w = first; w < items && ok;) {
      const int n = x ? it.n[1] : it.n[0];
      const int row0 = x ? it.row[1] : it.row[0];
      const int row = row0 + tok;
      // keys this row sees, keys every row of the tile sees, from the item's first on
      const int vis = max(0, min(it.t.lk, row + 1 + it.t.lk - it.t.lq) - it.t.block * ATTN_BLK);
      const int all = row0 + 1 + it.t.lk - it.t.lq - it.t.block * ATTN_BLK;
      float m = -INFINITY, l = 0.f;
      for (int j = 0; j < n; ++j) {
        ok = mbar_wait_bounded(&s_full[x], sn & 1, abort_flag, a.status, a.timeout_ns);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        ++sn;
        tc_fence_after();
        uint32_t s[128];
        tmem_ld128(tS, s);
        if ((j + 1) * ATTN_BLK > all) {
          keep_branch();
          const int lim = vis - j * ATTN_BLK;
#pragma unroll
          for (int i = 0; i < 128; ++i) s[i] = i < lim ? s[i] : 0xFF800000u;
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int i = 0; i < 128; i += 8)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mx[k] = fmaxf(mx[k], fmaxf(__uint_as_float(s[i + 2 * k]), __uint_as_float(s[i + 2 * k + 1])));
        const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        const bool raise = j == 0 || (top - m) * c > 8.f;
        if (j == 0) {
          m = top;
        } else if (__any_sync(0xffffffffu, raise)) {
          const float f = raise ? exp2_sfu((m - top) * c) : 1.f;
          if (raise) m = top;
          l *= f;
#pragma unroll 1
          for (int q = 0; q < 4; ++q) {
            float o[32];
            tmem_ld32(tO + q * 32, o);
            uint32_t u[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) u[i] = __float_as_uint(o[i] * f);
            tmem_st32(tO + q * 32, u);
          }
          tmem_st_wait();
        }
        // a row without any key keeps m = -inf: its weights are 2^-inf = 0
        const float mc = m == -INFINITY ? 0.f : m * c;
        const uint64_t c2 = f2_pack(c, c), mc2 = f2_pack(-mc, -mc);
        uint64_t sum[2] = {0ull, 0ull};
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t p[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            const int e = h * 64 + 2 * i;
            uint64_t z = f2_fma(f2_pack(__uint_as_float(s[e]), __uint_as_float(s[e + 1])), c2, mc2);
            float z0, z1;
            f2_unpack(z, z0, z1);
            z0 = exp2_sfu(z0);
            z1 = exp2_sfu(z1);
            sum[i & 1] = f2_add(sum[i & 1], f2_pack(z0, z1));
            p[i] = pack_bf16x2(z0, z1);
          }
          tmem_st32(tS + h * 32, p);
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[x]);
        float s0, s1;
        f2_unpack(f2_add(sum[0], sum[1]), s0, s1);
        l += s0 + s1;
      }
      if (!ok) break;
      w = snake_item(first, step, ++k);
      FwdItem nx = it;
      if (w < items) nx = fwd_item(a, w);
      const bool valid = row < it.t.lq;
      const int head = (x ? it.head[1] : it.head[0]) + hd;
      const int64_t grow = static_cast<int64_t>(it.t.q0) + row;
      __nv_bfloat16* dst = a.O + grow * a.n_q * ATTN_D + head * ATTN_D;
      if (n > 0) {
        ok = mbar_wait_bounded(&o_full[x], on & 1, abort_flag, a.status, a.timeout_ns);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        ++on;
        tc_fence_after();
      }
      const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);  // NaN stays NaN
      if (it.t.slot >= 0) {
        // column by column of four, rows side by side
        const int shift = a.head_shift + a.pair_heads;
        const int64_t at = (static_cast<int64_t>(it.t.slot) * (a.n_q >> shift) + (it.head[0] >> shift)) * 2 + x;
        if (n > 0) {
          float4* dst = reinterpret_cast<float4*>(a.part + at * ATTN_BLK * ATTN_D) + r;
#pragma unroll 1
          for (int q = 0; q < 4; ++q) {
            float o[32];
            __syncwarp();
            tmem_ld32(tO + q * 32, o);
#pragma unroll
            for (int i = 0; i < 8; ++i)
              if (valid)
                dst[(q * 8 + i) * ATTN_BLK] =
                    make_float4(o[4 * i] * inv, o[4 * i + 1] * inv, o[4 * i + 2] * inv, o[4 * i + 3] * inv);
          }
          tc_fence_before();
        }
        // -inf: no key of this part, and no output read
        a.part_lse[at * ATTN_BLK + r] = n == 0 || vis == 0 ? -INFINITY : m * c + log2f(l);
        it = nx;
        continue;
      }
      if (n > 0) {
        // through shared memory, so that a warp's store covers whole 128-byte
        // lines: rows of 64 columns, 16-byte piece p of row r at p ^ (r & 7)
        uint8_t* box = sO + warp * 4096;
        const int64_t rows = static_cast<int64_t>(it.t.q0) + row0;
        const int heads0 = x ? it.head[1] : it.head[0];
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            float o[32];
            tmem_ld32(tO + h * 64 + q * 32, o);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              float v[8];
#pragma unroll
              for (int k2 = 0; k2 < 8; ++k2) v[k2] = vis > 0 ? o[8 * i + k2] * inv : 0.f;
              store_bf16x8(reinterpret_cast<__nv_bfloat16*>(box + lane * 128 + (((4 * q + i) ^ (lane & 7)) << 4)), v);
            }
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int br = 4 * i + (lane >> 3), tr = (warp & 3) * 32 + br;  // row of the box, of the tile
            const int trow = row0 + (tr >> a.head_shift);
            const uint4 v = *reinterpret_cast<const uint4*>(box + br * 128 + (((lane & 7) ^ (br & 7)) << 4));
            if (trow < it.t.lq)
              *reinterpret_cast<uint4*>(a.O + ((rows + (tr >> a.head_shift)) * a.n_q + heads0 +
                                               (tr & ((1 << a.head_shift) - 1))) * ATTN_D + h * 64 + (lane & 7) * 8) = v;
          }
          __syncwarp();
        }
        tc_fence_before();
      }
      if (valid) {
        if (n == 0) {
#pragma unroll
          for (int i = 0; i < 16; ++i) *reinterpret_cast<uint4*>(dst + i * 8) = make_uint4(0, 0, 0, 0);
        }
        a.lse[static_cast<int64_t>(head) * a.Tq + grow] = vis == 0 ? -INFINITY : m * a.scale + logf(l);
      }
      it = nx;
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

// Joins the parts of a run's keys: O = sum_p 2^(lse_p - W) O_p / sum_p 2^(lse_p - W).
// A thread takes one row and eight columns, a block 256 of the 2 * 2048 such
// pieces of an item at a time.
__global__ void __launch_bounds__(256) attn_fwd_join_kernel(const AttnFwdArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const int cuts = __ldcg(a.counts + 3);
  const int per = a.n_q >> (a.head_shift + a.pair_heads);
  const int span = ATTN_BLK >> a.head_shift, hp = 1 << a.head_shift;
  for (int w = blockIdx.x; w < cuts * per * 16; w += gridDim.x) {
    const int x = (w >> 3) & 1, at = w >> 4;  // tile; run, item
    const int ti = at / per, hi = at - ti * per;
    const AttnTile t = load_tile(a.cuts + ti);
    const int u = (w & 7) * 256 + static_cast<int>(threadIdx.x);
    const int r = u & (ATTN_BLK - 1), c8 = u >> 7;
    const int row = t.t0 + (a.pair_heads ? 0 : x * span) + (r >> a.head_shift);
    if (row >= t.lq) continue;
    const int head = (hi << (a.head_shift + a.pair_heads)) + (a.pair_heads ? x * hp : 0) + (r & (hp - 1));
    const int parts = t.block;
    const int64_t step = static_cast<int64_t>(per) * 2 * ATTN_BLK;  // rows from part to part
    const int64_t first = ((static_cast<int64_t>(t.slot) * per + hi) * 2 + x) * ATTN_BLK;
    float top = -INFINITY;
    for (int p = 0; p < parts; ++p) top = fmaxf(top, a.part_lse[first + p * step + r]);
    const float base = top == -INFINITY ? 0.f : top;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, sum = 0.f;
#pragma unroll 4
    for (int p = 0; p < parts; ++p) {
      const float lse = a.part_lse[first + p * step + r];
      if (lse == -INFINITY) continue;  // nothing was left there
      const float4* s = reinterpret_cast<const float4*>(a.part + (first + p * step) * ATTN_D) + 2 * c8 * ATTN_BLK + r;
      const float4 lo = s[0], hi4 = s[ATTN_BLK];
      const float wgt = exp2_sfu(lse - base);
      sum += wgt;
      v[0] += wgt * lo.x; v[1] += wgt * lo.y; v[2] += wgt * lo.z; v[3] += wgt * lo.w;
      v[4] += wgt * hi4.x; v[5] += wgt * hi4.y; v[6] += wgt * hi4.z; v[7] += wgt * hi4.w;
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= inv;
    const int64_t grow = static_cast<int64_t>(t.q0) + row;
    store_bf16x8(a.O + (grow * a.n_q + head) * ATTN_D + c8 * 8, v);
    if (c8 == 0)
      a.lse[static_cast<int64_t>(head) * a.Tq + grow] = sum == 0.f ? -INFINITY : top * 0.69314718056f + logf(sum);
  }
}

}  // namespace

cudaError_t launch_attn_fwd(const AttnFwdArgs& a, const CUtensorMap* maps, int64_t max_items, int sms,
                            cudaStream_t s) {
  cudaError_t e = attn_smem_attribute(reinterpret_cast<const void*>(attn_fwd_kernel), 0, FWD_SMEM);
  if (e != cudaSuccess) return e;
  e = attn_launch(attn_fwd_kernel, std::min<int64_t>(sms, max_items), FWD_THREADS, FWD_SMEM, s, maps[0], maps[1], maps[2], a);
  if (e != cudaSuccess || !a.part) return e;
  return attn_launch(attn_fwd_join_kernel, 4 * sms, 256, 0, s, a);
}

}  // namespace coda

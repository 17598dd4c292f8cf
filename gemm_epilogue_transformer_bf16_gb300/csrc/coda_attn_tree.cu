// Attention of drafted tokens over the 4-bit cache: node i of a sequence's tree
// sees the committed prefix, its ancestors and itself,
//   s_ij = scale q_i . k_j,  O_i = sum_j exp(s_ij - lse_i) v_j.
//
// Bounds: 152 bytes per cached token and key/value head feed 2 * 128
// multiply-adds for each row, a row being a node and a query head of the
// group.  Up to about 80 rows the bytes take longer at this chip's rates, then the
// products.
//
// Work: the rows of a sequence and key/value head are cut into tiles of up to
// 128, and the keys of a tile into units of 128.  The units of the whole batch
// form one line, each as many places as it costs, that the CTAs (one per SM)
// divide evenly.  A CTA whose stretch covers all keys of a tile writes the
// output; the others leave normalised partial outputs that a second kernel
// joins.
//
// Scores and outputs are transposed, keys and elements along the 128 lanes of
// TMEM and rows along its columns:
//   S^T [128 keys x rows]      = K' Q^T    K' = e2m1 * e4m3, exact in f16, is the
//                                          A operand in TMEM, a thread per key
//   O^T [128 elements x rows] += V'^T P'^T V' in shared memory, elements
//                                          contiguous; P' too, rows contiguous
// so that few rows make a narrow product instead of an empty one, and a
// softmax thread has one key: its scales are two registers, sums over keys stay
// in the thread until the end, and no maximum is exchanged unless a weight passes
// its bound.
//
// A weight carries its value's row scale rs:
//   P' = 2^t,  t = scale log2(e) rs_k (q . k') + log2 rs_v - r,  l = sum P' / rs_v
// with a reference r per row, raised when some t passes 10 (f16 holds 2^15),
// so P' is rounded by 2^-11 of itself or 2^-25 of the largest weighted row
// scale.  Rows of zeros take the smallest row scale of their neighbours: their
// own says nothing.  l, r and O are fp32.
#include <algorithm>

#include "coda_attn.cuh"
#include "coda_attn_tree.cuh"
#include "coda_internal.h"
#include "coda_kvrow.cuh"
#include "coda_status.h"

namespace coda {
namespace {

constexpr int TR_GROUPS = 4;                          // warpgroups that unpack and weigh
constexpr int TR_THREADS = TR_GROUPS * 128 + 64;      // and two warps: copies, products
constexpr int TR_UNIT = 128;
constexpr int TR_STAGES = 3;
// a stage of the cache's rows as they lie in memory
constexpr int RW_K = 0, RW_V = 8192, RW_SFK = 16384, RW_SFV = 17408, RW_RSK = 18432, RW_RSV = 18944;
constexpr int TR_RAW = 19456;
constexpr uint32_t TILE = 32768, HALF_TILE = 16384;  // 128 x 128 f16, as two halves of 64 columns
constexpr uint32_t OFF_Q = 0, OFF_P = TILE, OFF_V = 3 * TILE, OFF_RAW = 5 * TILE;
constexpr uint32_t OFF_ROW = OFF_RAW + TR_STAGES * TR_RAW;  // [2][64] pairs of rows, by item: factors, -r
constexpr uint32_t OFF_KEY = OFF_ROW + 2048;                // [4][128] row scale of the key, log2 of the value's
constexpr uint32_t OFF_RED = OFF_KEY + 4096;                // [4][4][32] exchange of a warpgroup
constexpr uint32_t OFF_BAR = OFF_RED + 2048;
constexpr uint32_t TR_SMEM = 1024 + OFF_BAR + 256;
static_assert(TR_SMEM <= 232448, "shared memory per CTA");
constexpr uint32_t COL_S = 0, COL_O = 256, COL_K = 384;  // TMEM columns: S twice, O, K' twice (64 each)
constexpr float TR_RAISE = 10.f;
constexpr uint32_t TR_NO_MORE = 1u << 31;
constexpr uint64_t TR_WAIT_NS = 2000000000ull;

// Places of a unit, by the rows of its tile, and of a stretch's ends.
constexpr int TR_COST_FEW = 4, TR_COST_MANY = 6, TR_END = 12;

__device__ __forceinline__ constexpr uint32_t idesc_f16(int M, int N, int a_mn, int b_mn) {
  return (1u << 4) | (static_cast<uint32_t>(a_mn) << 15) | (static_cast<uint32_t>(b_mn) << 16) |
         (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ void fence_async_smem() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }
// Barrier of a warpgroup that tells whether any thread's predicate holds.
__device__ __forceinline__ bool group_any(int id, bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred P, R;\n\tsetp.ne.b32 P, %1, 0;\n\t"
      "barrier.cta.red.or.pred R, %2, 128, P;\n\tselp.u32 %0, 1, 0, R;\n\t}"
      : "=r"(r)
      : "r"(static_cast<uint32_t>(p)), "r"(id)
      : "memory");
  return r != 0;
}
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : CODA_R8(r, 0), CODA_R8(r, 8)
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ldn(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : CODA_R8(r, 0)
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void tmem_ldn(uint32_t taddr, uint32_t (&r)[16]) { tmem_ld16(taddr, r); }
__device__ __forceinline__ void tmem_ldn(uint32_t taddr, uint32_t (&r)[32]) {
  float v[32];
  tmem_ld32(taddr, v);
#pragma unroll
  for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(v[i]);
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), CODA_W8(r, 0)
               : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      CODA_W8(r, 0), CODA_W8(r, 8)
      : "memory");
}

// A sequence's work.
struct TreeSeq {
  int q0, n, len;     // first token, nodes, cached tokens; n = 0: no work
  int units, tiles;
  int64_t place_kv;   // places per key/value head
  __device__ __forceinline__ int rows(int tile, int group) const { return min(TREE_ROWS, n * group - tile * TREE_ROWS); }
};
__device__ __forceinline__ int tree_cost(int rows) { return rows <= 64 ? TR_COST_FEW : TR_COST_MANY; }
__device__ __forceinline__ TreeSeq tree_seq(const TreeArgs& a, int b, bool tell) {
  TreeSeq s;
  s.q0 = a.cu[b];
  s.n = a.cu[b + 1] - s.q0;
  s.len = a.seq_lens[b];
  const bool off = s.q0 < 0 || s.n < 0 || s.q0 + s.n > a.T;
  if (off || (s.n > 0 && (s.len < s.n || s.len > (static_cast<int64_t>(a.max_pages) << a.c.page_shift)))) {
    if (tell) atomicOr(a.status, CODA_DEV_SEQLEN_RANGE);
    s.n = 0;
  } else if (a.parents && s.n > TREE_MAX_NODES) {
    if (tell) atomicOr(a.status, CODA_DEV_TREE_RANGE);
    s.n = 0;
  }
  s.units = (s.len + TR_UNIT - 1) / TR_UNIT;
  s.tiles = (s.n * a.group + TREE_ROWS - 1) / TREE_ROWS;
  s.place_kv = 0;
  if (s.n > 0)
    s.place_kv = static_cast<int64_t>(s.tiles - 1) * (static_cast<int64_t>(s.units) * TR_COST_MANY + TR_END) +
                 static_cast<int64_t>(s.units) * tree_cost(s.rows(s.tiles - 1, a.group)) + TR_END;
  return s;
}
// First unit that starts at `place` or behind it, of an item at `base`.
__device__ __forceinline__ int unit_at(int64_t place, int64_t base, int cost, int units) {
  const int64_t d = place - base - TR_END;
  return d <= 0 ? 0 : static_cast<int>(min(static_cast<int64_t>(units), (d + cost - 1) / cost));
}

// A CTA's way along the line: items (sequence, key/value head, tile) with the
// units [u0, u1) that it takes of each.  Every warp walks it for itself.
struct TreeWalk {
  int b, item;            // sequence, next item of it
  int64_t base;           // place of that item
  TreeSeq s;
  // current
  int kvh, tile, rows, u0, u1;
  __device__ __forceinline__ bool next(const TreeArgs& a, int64_t first, int64_t last) {
    while (base < last) {
      if (s.n == 0 || item == a.c.n_kv * s.tiles) {
        if (++b >= a.B) return false;
        s = tree_seq(a, b, false);
        item = 0;
        continue;
      }
      kvh = item / s.tiles;
      tile = item - kvh * s.tiles;
      rows = s.rows(tile, a.group);
      const int cost = tree_cost(rows);
      u0 = unit_at(first, base, cost, s.units);
      u1 = unit_at(last, base, cost, s.units);
      base += static_cast<int64_t>(s.units) * cost + TR_END;
      ++item;
      if (u0 < u1) return true;
    }
    return false;
  }
};

// Maximum (or sum) over the warp's lanes of N columns, N a power of two: lane i
// gets column i % N.
template <int N, bool SUM>
__device__ __forceinline__ float warp_columns(float (&v)[N], int lane) {
#pragma unroll
  for (int o = 16; o >= N; o >>= 1)
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float x = __shfl_xor_sync(0xffffffffu, v[i], o);
      v[i] = SUM ? v[i] + x : fmaxf(v[i], x);
    }
#pragma unroll
  for (int o = N / 2; o; o >>= 1)
#pragma unroll
    for (int i = 0; i < o; ++i) {
      const bool up = lane & o;
      const float give = up ? v[i] : v[i + o], keep = up ? v[i + o] : v[i];
      const float x = __shfl_xor_sync(0xffffffffu, give, o);
      v[i] = SUM ? keep + x : fmaxf(keep, x);
    }
  return v[0];
}

struct TreeBars {
  uint64_t raw_full[TR_STAGES], raw_empty[TR_STAGES];
  uint64_t k_full[2], v_full[2], s_full[2], s_empty[2], p_full[2], o_done[2];
  uint64_t q_full, o_empty, drain;
  uint32_t keys_in[TR_STAGES];  // bit i: keys 16 i .. 16 i + 15 of the stage are there; TR_NO_MORE: no unit, nor behind it
  int left[TR_STAGES];          // keys of the sequence from the stage's first on
  uint32_t tmem;
  int abort;
};
static_assert(sizeof(TreeBars) <= 256, "barrier area");

__device__ __forceinline__ bool tree_wait(uint64_t* bar, uint32_t parity, TreeBars* s, int* status, uint32_t sleep_ns = 0) {
  return mbar_wait_bounded(bar, parity, &s->abort, status, TR_WAIT_NS, sleep_ns);
}

// What a warp of the unpacking has in hand between the keys of a unit and its
// values.
struct Unpack {
  uint32_t it;      // number of the unit
  bool more;        // there is one
  uint32_t on;      // its groups of 16 keys
  int left;
  uint32_t rs_zero;  // row scale that rows of zeros take
};

// K' of unit x.it: thread (wg, key) takes elements 32 wg .. 32 wg + 31 of its
// key's row, to TMEM.  Its place was read by the scores of two units ago, which
// every warp has seen.
__device__ __forceinline__ bool unpack_keys(const TreeArgs& a, uint8_t* smem, TreeBars* bar, uint32_t tmem, int wg, int warp4,
                                            int lane, Unpack& x) {
  const uint32_t st = x.it % TR_STAGES, buf = x.it & 1;
  if (!__all_sync(0xffffffffu, tree_wait(&bar->raw_full[st], (x.it / TR_STAGES) & 1, bar, a.status))) return false;
  x.on = bar->keys_in[st];
  x.left = bar->left[st];
  x.more = x.on != TR_NO_MORE;
  if (!x.more) return true;
  tc_fence_after();
  const uint8_t* raw = smem + OFF_RAW + st * TR_RAW;
  const int key = warp4 * 32 + lane;
  const bool in = ((x.on >> (key >> 4)) & 1u) && key < x.left;
  const uint32_t two =
      e4m3x2_f16(in ? *reinterpret_cast<const uint16_t*>(raw + RW_SFK + key * 8 + wg * 2) : 0);
  const uint32_t s0 = __byte_perm(two, two, 0x1010), s1 = __byte_perm(two, two, 0x3232);
  const uint4 v = *reinterpret_cast<const uint4*>(raw + RW_K + key * 64 + wg * 16);
  uint32_t o[16];
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    uint32_t f[4];
    e2m1x8_f16(w == 0 ? v.x : w == 1 ? v.y : w == 2 ? v.z : v.w, f);
#pragma unroll
    for (int i = 0; i < 4; ++i) o[w * 4 + i] = hmul2(f[i], w < 2 ? s0 : s1);
  }
  tmem_st16(tmem + (static_cast<uint32_t>(warp4 * 32) << 16) + COL_K + buf * 64 + wg * 16, o);
  if (wg == 0) {  // the key's scales
    const uint2 sfv = *reinterpret_cast<const uint2*>(raw + RW_SFV + key * 8);
    const float rsk = *reinterpret_cast<const float*>(raw + RW_RSK + key * 4);
    const float rsv = *reinterpret_cast<const float*>(raw + RW_RSV + key * 4);
    const bool sick = (((sfv.x & 0x7F7F7F7Fu) + 0x01010101u) | ((sfv.y & 0x7F7F7F7Fu) + 0x01010101u)) & 0x80808080u;
    const bool zeros = ((sfv.x | sfv.y) & 0x7F7F7F7Fu) == 0;
    const uint32_t least = __reduce_min_sync(0xffffffffu, in && !zeros && !sick ? __float_as_uint(rsv) : 0x7F7FFFFFu);
    if (least < 0x7F7FFFFFu) x.rs_zero = least;
    const float rs = zeros ? __uint_as_float(x.rs_zero) : rsv;
    float2 meta;
    meta.x = in ? rsk : 0.f;
    // below 2^-100 the sum l would pass fp32's end: unpack_values takes the rest
    meta.y = !in ? -INFINITY : sick ? __uint_as_float(0x7FC00000u) : rs < 0x1p-100f ? -100.f : log2f(rs);
    *reinterpret_cast<float2*>(smem + OFF_KEY + (x.it & 3) * 1024 + key * 8) = meta;
  }
  tmem_st_wait();
  tc_fence_before();
  __syncwarp();
  if (lane == 0) mbar_arrive(&bar->k_full[buf]);
  return true;
}

// V' of the unit: a warp takes eight keys, a lane sixteen elements of two of
// them.  A block scale that is NaN leaves zeros (the key's weights are NaN).
__device__ __forceinline__ bool unpack_values(const TreeArgs& a, uint8_t* smem, TreeBars* bar, int wwarp, int lane, Unpack& x) {
  const uint32_t st = x.it % TR_STAGES, buf = x.it & 1;
  if (!__all_sync(0xffffffffu, tree_wait(&bar->o_done[buf], ((x.it >> 1) & 1) ^ 1, bar, a.status))) return false;
  const uint8_t* raw = smem + OFF_RAW + st * TR_RAW;
  uint8_t* to = smem + OFF_V + buf * TILE;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int k = wwarp * 8 + i * 4 + (lane >> 3), piece = lane & 7;  // key, elements 16 piece ..
    const uint2 c = *reinterpret_cast<const uint2*>(raw + RW_V + k * 64 + piece * 8);
    uint32_t sf = raw[RW_SFV + k * 8 + piece];
    const bool in = ((x.on >> (k >> 4)) & 1u) && k < x.left;  // else whatever the stage held before
    const float rv = in ? *reinterpret_cast<const float*>(raw + RW_RSV + k * 4) : 1.f;
    if (!in || (sf & 0x7Fu) == 0x7Fu) sf = 0;
    uint32_t s = e4m3x2_f16(sf * 0x101u);
    if (__any_sync(0xffffffffu, rv < 0x1p-100f)) {
      keep_branch();
      const float by = rv < 0x1p-100f ? rv * 0x1p100f : 1.f;
      s = pack_f16(f16_lo(s) * by, f16_hi(s) * by);
    }
    uint32_t f[4], h[4];
    e2m1x8_f16(c.x, f);
    e2m1x8_f16(c.y, h);
    uint8_t* row = to + (piece >> 2) * HALF_TILE + k * 128;
    const int p = 2 * (piece & 3);
    *reinterpret_cast<uint4*>(row + ((p ^ (k & 7)) << 4)) =
        make_uint4(hmul2(f[0], s), hmul2(f[1], s), hmul2(f[2], s), hmul2(f[3], s));
    *reinterpret_cast<uint4*>(row + (((p + 1) ^ (k & 7)) << 4)) =
        make_uint4(hmul2(h[0], s), hmul2(h[1], s), hmul2(h[2], s), hmul2(h[3], s));
  }
  fence_async_smem();
  __syncwarp();
  if (lane == 0) {
    mbar_arrive(&bar->v_full[buf]);
    mbar_arrive(&bar->raw_empty[st]);
  }
  ++x.it;
  return true;
}

// A warpgroup's part of one stretch: the weights of columns wg * NC .. of the
// tile, and between them its share of unpacking the next unit.  `it` counts the
// CTA's units.  False: a wait ran out.
template <int NC>
__device__ __forceinline__ bool tree_softmax(const TreeArgs& a, const TreeWalk& w, uint8_t* smem, TreeBars* bar, uint32_t tmem,
                                             int wg, uint32_t& it, uint32_t item, Unpack& x) {
  const int tid = threadIdx.x & 127, warp = tid >> 5, lane = tid & 31;
  const int id = 1 + wg;                 // named barrier
  const int row0 = w.tile * TREE_ROWS;   // of the tile, among the sequence's rows
  const int col0 = wg * NC;
  float* red = reinterpret_cast<float*>(smem + OFF_RED) + wg * 128;  // [4][32]
  float* rowtab = reinterpret_cast<float*>(smem + OFF_ROW + (item & 1) * 1024);  // per pair of columns: f, f, -r, -r
  const int64_t q0 = w.s.q0;
  bool ok = true;

  // ---- Q: rows scaled by a power of two to a maximum in [1, 2), f16; rows
  // behind the tile's are zeros.  Sixteen lanes per row.
  for (int i = tid >> 4; i < NC; i += 8) {
    const int c = col0 + i, row = row0 + c, piece = tid & 15;
    float y[8];
    const bool there = c < w.rows;
    if (there) {
      const int node = row / a.group, head = w.kvh * a.group + row - node * a.group;
      load_bf16x8(a.Q + (q0 + node) * a.ldq + head * 128 + piece * 8, y);
    } else {
#pragma unroll
      for (int k = 0; k < 8; ++k) y[k] = 0.f;
    }
    float mx = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) mx = fmaxf(mx, fabsf(y[k]) <= 3.4e38f ? fabsf(y[k]) : 0.f);
#pragma unroll
    for (int o = 8; o; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    int e = static_cast<int>(__float_as_uint(mx) >> 23) - 127;
    e = mx == 0.f ? 0 : max(-126, min(126, e));
    const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
    uint4 v;
    v.x = pack_f16(y[0] * down, y[1] * down);
    v.y = pack_f16(y[2] * down, y[3] * down);
    v.z = pack_f16(y[4] * down, y[5] * down);
    v.w = pack_f16(y[6] * down, y[7] * down);
    *reinterpret_cast<uint4*>(smem + OFF_Q + (piece >> 3) * HALF_TILE + c * 128 + (((piece & 7) ^ (c & 7)) << 4)) = v;
    if (piece == 0) {
      float* at = rowtab + (c >> 1) * 4 + (c & 1);
      at[0] = __uint_as_float(static_cast<uint32_t>(127 + e) << 23) * a.scale_log2;
      at[2] = 0.f;  // no reference yet
    }
  }
  fence_async_smem();
  __syncwarp();
  if (lane == 0) mbar_arrive(&bar->q_full);

  // ---- what each row sees of its tree
  const int prefix = w.s.len - w.s.n;  // keys that every row sees
  uint32_t* seen = a.seen + (static_cast<int64_t>(blockIdx.x) * TREE_ROWS + col0) * (TREE_MAX_NODES / 32);
  if (a.parents && min(w.u1 * TR_UNIT, w.s.len) > prefix) {
    int16_t* up = reinterpret_cast<int16_t*>(red);  // 256 of them fit
    for (int i = tid; i < w.s.n; i += 128) {
      const int p = a.parents[q0 + i];
      const bool bad = p < -1 || p >= i;
      if (bad) atomicOr(a.status, CODA_DEV_TREE_RANGE);
      up[i] = static_cast<int16_t>(bad ? -1 : p);
    }
    group_any(id, false);
    if (tid < NC && col0 + tid < w.rows) {
      uint32_t m[TREE_MAX_NODES / 32];
#pragma unroll
      for (int k = 0; k < TREE_MAX_NODES / 32; ++k) m[k] = 0;
      for (int j = (row0 + col0 + tid) / a.group; j >= 0; j = up[j])
#pragma unroll
        for (int k = 0; k < TREE_MAX_NODES / 32; ++k) m[k] |= (j >> 5) == k ? 1u << (j & 31) : 0u;
#pragma unroll
      for (int k = 0; k < TREE_MAX_NODES / 32; ++k) seen[tid * (TREE_MAX_NODES / 32) + k] = m[k];
    }
  }
  group_any(id, false);

  const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
  float l[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) l[c] = 0.f;
  bool unset = true;        // some column has no reference
  bool mine_unset = true;   // column col0 + tid (tid < NC)
  const float4* tab4 = reinterpret_cast<const float4*>(rowtab) + (col0 >> 1);
  uint8_t* pbase = smem + OFF_P + ((col0 >> 6) * HALF_TILE) + tid * 128;
  const int chunk0 = (col0 & 63) >> 3;

  for (int u = w.u0; u < w.u1; ++u, ++it) {
    const uint32_t buf = it & 1, ph = (it >> 1) & 1;
    ok = ok && (!x.more || unpack_keys(a, smem, bar, tmem, wg, warp, lane, x));
    ok = ok && tree_wait(&bar->k_full[buf], ph, bar, a.status) && tree_wait(&bar->s_full[buf], ph, bar, a.status);
    ok = __all_sync(0xffffffffu, ok);
    float t[NC];
    float mx = -INFINITY;
    float inv = 0.f;
    if (ok) {
      tc_fence_after();
      const float2 key = *reinterpret_cast<const float2*>(smem + OFF_KEY + (it & 3) * 1024 + tid * 8);
      uint32_t s[NC];
      tmem_ldn(tmem + lanes + COL_S + buf * 128 + col0, s);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar->s_empty[buf]);
      inv = fabsf(key.y) < 1e30f ? exp2_sfu(-key.y) : 0.f;  // finite: it meets zero weights too
      const uint64_t rk = f2_pack(key.x, key.x), lr = f2_pack(key.y, key.y);
#pragma unroll
      for (int c = 0; c < NC; c += 2) {
        const float4 f = tab4[c >> 1];
        const uint64_t z = f2_mul(f2_pack(__uint_as_float(s[c]), __uint_as_float(s[c + 1])), rk);
        f2_unpack(f2_fma(z, f2_pack(f.x, f.y), f2_add(lr, f2_pack(f.z, f.w))), t[c], t[c + 1]);
      }
      const int d = u * TR_UNIT + tid - prefix;  // this key's node, if it is one
      if ((u + 1) * TR_UNIT > prefix) {
        keep_branch();
        if (a.parents) {
          const uint32_t* at = seen + (max(d, 0) >> 5);
#pragma unroll
          for (int c = 0; c < NC; ++c)
            if (d >= 0 && (d >= w.s.n || !((__ldcg(at + c * (TREE_MAX_NODES / 32)) >> (d & 31)) & 1u))) t[c] = -INFINITY;
        } else {
#pragma unroll
          for (int c = 0; c < NC; ++c)
            if (d >= 0 && (d >= w.s.n || d * a.group > row0 + col0 + c)) t[c] = -INFINITY;
        }
      }
#pragma unroll
      for (int c = 0; c < NC; c += 2) mx = fmaxf(mx, fmaxf(t[c], t[c + 1]));
    }
    if (group_any(id, !ok || unset || mx > TR_RAISE)) {
      // a reference rises, or is not there yet
      if (group_any(id, !ok)) return false;
      float v[NC];
#pragma unroll
      for (int i = 0; i < NC; ++i) v[i] = t[i];
      const float most = warp_columns<NC, false>(v, lane);
      if (lane < NC) red[warp * 32 + lane] = most;
      group_any(id, false);
      float step = 0.f, shrink = 1.f;
      if (tid < NC) {
        const float m = fmaxf(fmaxf(red[tid], red[32 + tid]), fmaxf(red[64 + tid], red[96 + tid]));
        if (m > (mine_unset ? -INFINITY : TR_RAISE)) {  // whatever the other rows do
          step = m;
          shrink = mine_unset ? 1.f : exp2_sfu(-m);
          mine_unset = false;
          const int c = col0 + tid;
          rowtab[(c >> 1) * 4 + (c & 1) + 2] -= m;
        }
      }
      group_any(id, false);  // the maxima are read
      if (tid < NC) {
        red[tid] = step;
        red[32 + tid] = shrink;
      }
      unset = group_any(id, tid < NC && mine_unset);
      const bool before = u > w.u0;  // O holds something
      if (before) {
        const uint32_t p = it - 1;
        ok = tree_wait(&bar->o_done[p & 1], (p >> 1) & 1, bar, a.status);
        ok = __all_sync(0xffffffffu, ok);
        tc_fence_after();
      }
#pragma unroll
      for (int c0 = 0; c0 < NC; c0 += 8) {
        float by[8];
        bool any = false;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          t[c0 + i] -= red[c0 + i];
          by[i] = red[32 + c0 + i];
          l[c0 + i] *= by[i];
          any |= by[i] != 1.f;
        }
        if (before && any && ok) {
          uint32_t o[8];
          tmem_ldn(tmem + lanes + COL_O + col0 + c0, o);
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * by[i]);
          tmem_st8(tmem + lanes + COL_O + col0 + c0, o);
          tmem_st_wait();
        }
      }
      tc_fence_before();
      group_any(id, false);  // red is read
    }
    // ---- P', into the place that the product of two units ago has read
    ok = ok && tree_wait(&bar->o_done[buf], ph ^ 1, bar, a.status);
    ok = __all_sync(0xffffffffu, ok);
    if (ok) {
      const uint64_t in2 = f2_pack(inv, inv);
      uint8_t* at = pbase + buf * TILE;
#pragma unroll
      for (int c = 0; c < NC; c += 8) {
        uint32_t p[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float x = exp2_sfu(t[c + 2 * k]), y = exp2_sfu(t[c + 2 * k + 1]);
          f2_unpack(f2_fma(f2_pack(x, y), in2, f2_pack(l[c + 2 * k], l[c + 2 * k + 1])), l[c + 2 * k], l[c + 2 * k + 1]);
          p[k] = pack_f16(x, y);
        }
        *reinterpret_cast<uint4*>(at + (((chunk0 + (c >> 3)) ^ (tid & 7)) << 4)) = make_uint4(p[0], p[1], p[2], p[3]);
      }
      fence_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bar->p_full[buf]);
      if (x.more) ok = unpack_values(a, smem, bar, wg * 4 + warp, lane, x);
    }
  }

  // ---- the end: l over the keys, O out of TMEM
  {
    const uint32_t p = it - 1;
    ok = ok && tree_wait(&bar->o_done[p & 1], (p >> 1) & 1, bar, a.status);
    ok = __all_sync(0xffffffffu, ok);
    const float sum = warp_columns<NC, true>(l, lane);
    if (lane < NC) red[warp * 32 + lane] = sum;
    if (group_any(id, !ok)) return false;
    const bool alone = w.u0 == 0 && w.u1 == w.s.units;
    const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (w.u0 > 0 ? 0 : 1);
    float total = 0.f;
    if (tid < NC) total = (red[tid] + red[32 + tid]) + (red[64 + tid] + red[96 + tid]);
    group_any(id, false);
    if (tid < NC) {
      red[tid] = total > 0.f ? 1.f / total : (total == 0.f ? 0.f : total);  // NaN stays NaN
      const int c = col0 + tid;
      if (c < w.rows) {
        const float r = -rowtab[(c >> 1) * 4 + (c & 1) + 2];
        const int row = row0 + c, node = row / a.group, head = w.kvh * a.group + row - node * a.group;
        if (alone)
          a.lse[(q0 + node) * a.n_q + head] = total == 0.f ? -INFINITY : r * 0.69314718056f + logf(total);
        else
          a.part_lse[slot * a.part_rows + c] = total == 0.f ? -INFINITY : r + log2f(total);
      }
    }
    group_any(id, false);
    tc_fence_after();
    const int d = warp * 32 + lane;  // element
#pragma unroll 1
    for (int c0 = 0; c0 < NC && col0 + c0 < w.rows; c0 += 8) {
      uint32_t o[8];
      tmem_ldn(tmem + lanes + COL_O + col0 + c0, o);
      if (alone) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int c = col0 + c0 + i, row = row0 + c;
          if (c < w.rows) {
            const int node = row / a.group, head = w.kvh * a.group + row - node * a.group;
            a.O[((q0 + node) * a.n_q + head) * 128 + d] = __float2bfloat16(__uint_as_float(o[i]) * red[c0 + i]);
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int c = col0 + c0 + i;
          if (c < w.rows) a.part[(slot * a.part_rows + c) * 128 + d] = __uint_as_float(o[i]) * red[c0 + i];
        }
      }
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&bar->o_empty);
    group_any(id, false);  // red is read
  }
  return true;
}

__global__ void __launch_bounds__(TR_THREADS, 1) attn_tree_kernel(const TreeArgs a) {
  extern __shared__ uint8_t tree_smem[];
  __shared__ int64_t sh_warp[TR_THREADS / 32], sh_before;
  __shared__ int sh_seq;
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(tree_smem) + 1023) & ~uintptr_t(1023));
  TreeBars* bar = reinterpret_cast<TreeBars*>(smem + OFF_BAR);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int s = 0; s < TR_STAGES; ++s) {
      mbar_init(&bar->raw_full[s], 1);
      mbar_init(&bar->raw_empty[s], TR_GROUPS * 4);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bar->k_full[s], TR_GROUPS * 4);
      mbar_init(&bar->v_full[s], TR_GROUPS * 4);
      mbar_init(&bar->s_full[s], 1);
      mbar_init(&bar->s_empty[s], TR_GROUPS * 4);
      mbar_init(&bar->p_full[s], TR_GROUPS * 4);
      mbar_init(&bar->o_done[s], 1);
    }
    mbar_init(&bar->q_full, TR_GROUPS * 4);
    mbar_init(&bar->o_empty, TR_GROUPS * 4);
    mbar_init(&bar->drain, 1);
    bar->abort = 0;
    sh_seq = a.B;
    sh_before = 0;
    fence_mbar_init();
  }
  if (warp == TR_GROUPS * 4 + 1) {
    tmem_alloc<false>(&bar->tmem, 512);
    tmem_relinquish<false>();
  }
  griddep_wait();
  griddep_launch_dependents();

  // places before each sequence: a contiguous run of sequences per thread,
  // scanned over the block
  const int chunk = (a.B + TR_THREADS - 1) / TR_THREADS;
  const int b0 = min(a.B, tid * chunk), b1 = min(a.B, b0 + chunk);
  int64_t mine = 0;
  for (int b = b0; b < b1; ++b) mine += tree_seq(a, b, blockIdx.x == 0).place_kv * a.c.n_kv;
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t n = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += n;
  }
  if (lane == 31) sh_warp[warp] = incl;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bar->tmem;
  int64_t total = 0;
#pragma unroll
  for (int w = 0; w < TR_THREADS / 32; ++w) {
    if (w < warp) incl += sh_warp[w];
    total += sh_warp[w];
  }
  // no CTA between two others of an item is left without a unit
  const int64_t per = max(static_cast<int64_t>(TR_COST_MANY), (total + gridDim.x - 1) / gridDim.x);
  const int64_t first = blockIdx.x * per, last = min(total, first + per);
  {
    int64_t before = incl - mine;
    for (int b = b0; b < b1; ++b) {
      const int64_t n = tree_seq(a, b, false).place_kv * a.c.n_kv;
      if (blockIdx.x == 0) a.places[b] = before;
      if (first >= before && first < before + n) {
        sh_seq = b;
        sh_before = before;
      }
      before += n;
    }
    if (blockIdx.x == 0 && tid == 0) {
      a.places[a.B] = total;
      a.places[a.B + 1] = per;
    }
  }
  __syncthreads();

  TreeWalk w;
  w.b = sh_seq;
  w.base = sh_before;
  w.item = 0;
  bool ok = true;
  if (first < last) {
    w.s = tree_seq(a, w.b, false);
    // to the item that holds `first`
    const int64_t d = first - w.base, kv = d / w.s.place_kv;
    const int64_t tile = (d - kv * w.s.place_kv) / (static_cast<int64_t>(w.s.units) * TR_COST_MANY + TR_END);
    const int64_t tl = min(tile, static_cast<int64_t>(w.s.tiles - 1));
    w.item = static_cast<int>(kv * w.s.tiles + tl);
    w.base += kv * w.s.place_kv + tl * (static_cast<int64_t>(w.s.units) * TR_COST_MANY + TR_END);

    if (warp < TR_GROUPS * 4) {
      const int wg = warp >> 2;
      uint32_t it = 0, item = 0;
      Unpack x;
      x.it = 0;
      x.more = true;
      x.rs_zero = __float_as_uint(0x1p-12f);
      ok = unpack_keys(a, smem, bar, tmem, wg, warp & 3, lane, x);
      if (ok && x.more) ok = unpack_values(a, smem, bar, warp, lane, x);
      for (; ok && w.next(a, first, last); ++item) {
        if (w.rows <= 32)
          ok = tree_softmax<8>(a, w, smem, bar, tmem, wg, it, item, x);
        else if (w.rows <= 64)
          ok = tree_softmax<16>(a, w, smem, bar, tmem, wg, it, item, x);
        else
          ok = tree_softmax<32>(a, w, smem, bar, tmem, wg, it, item, x);
      }
    } else {
      if (warp == TR_GROUPS * 4) {
        // ------------------------------------------------------------ copies
        // Lane i of each group of eight takes part i of a unit (a page, or 128
        // keys of one): group 0 the codes, 1 the block scales, 2 the row scales,
        // keys and values each.
        const KvCache& kc = a.c;
        const int part = lane & 7, arr = lane >> 3;
        const int part_shift = min(kc.page_shift, 7);
        const uint32_t row_bytes = arr == 0 ? 64 : arr == 1 ? 8 : 4;
        const uint32_t to_k = arr == 0 ? RW_K : arr == 1 ? RW_SFK : RW_RSK, to_v = arr == 0 ? RW_V : arr == 1 ? RW_SFV : RW_RSV;
        const uint8_t* src = arr == 0 ? kc.codes : arr == 1 ? kc.sf : reinterpret_cast<const uint8_t*>(kc.scale);
        const int64_t plane = static_cast<int64_t>(kc.n_kv) << kc.page_shift;
        uint32_t it = 0;
        while (ok && w.next(a, first, last)) {
          const int32_t* table = a.table + static_cast<int64_t>(w.b) * a.max_pages;
          auto page_of = [&](int u) {  // of this lane's part of unit u; -1: nothing there
            const int k = u * TR_UNIT + (part << part_shift);
            return u < w.u1 && (part << part_shift) < TR_UNIT && k < w.s.len ? table[k >> kc.page_shift] : -1;
          };
          int page = page_of(w.u0);
          for (int u = w.u0; u < w.u1; ++u, ++it) {
            const int nextp = page_of(u + 1);
            const int k = u * TR_UNIT + (part << part_shift);
            const bool named = (part << part_shift) < TR_UNIT && k < w.s.len;
            const bool in = named && page >= 0 && page < kc.num_pages;
            if (named && !in && arr == 0) atomicOr(a.status, CODA_DEV_PAGE_RANGE);
            // whole groups of 16 keys: rows behind the length exist within the page
            const int n = in ? min(1 << part_shift, (w.s.len - k + 15) & ~15) : 0;
            const uint32_t bytes = arr < 3 ? n * row_bytes : 0;
            const uint32_t st = it % TR_STAGES;
            ok = tree_wait(&bar->raw_empty[st], ((it / TR_STAGES) & 1) ^ 1, bar, a.status, 100);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            const uint32_t sum = __reduce_add_sync(0xffffffffu, 2 * bytes);
            const uint32_t mask =
                __reduce_or_sync(0xffffffffu, arr == 0 && n ? ((1u << (n / 16)) - 1) << (part << part_shift >> 4) : 0);
            if (lane == 0) {
              bar->keys_in[st] = mask;
              bar->left[st] = w.s.len - u * TR_UNIT;
              if (sum == 0) mbar_arrive(&bar->raw_full[st]);
            }
            mbar_arrive_expect_tx(&bar->raw_full[st], sum, lane == 0 && sum != 0);
            __syncwarp();
            if (bytes) {
              const int64_t row = cache_row(kc, page, 0, w.kvh, k & ((1 << kc.page_shift) - 1));
              uint8_t* to = smem + OFF_RAW + st * TR_RAW + (part << part_shift) * row_bytes;
              bulk_load(to + to_k, src + row * row_bytes, bytes, &bar->raw_full[st], 1);
              bulk_load(to + to_v, src + (row + plane) * row_bytes, bytes, &bar->raw_full[st], 1);
            }
            page = nextp;
          }
        }
        if (ok) {  // nothing more
          const uint32_t st = it % TR_STAGES;
          ok = tree_wait(&bar->raw_empty[st], ((it / TR_STAGES) & 1) ^ 1, bar, a.status, 100);
          ok = __all_sync(0xffffffffu, ok);
          if (ok && lane == 0) {
            bar->keys_in[st] = TR_NO_MORE;
            mbar_arrive(&bar->raw_full[st]);
          }
        }
        if (!ok) {
          // let every copy already issued land before the CTA's memory is reused
          const uint64_t t0 = globaltimer_ns();
          while (globaltimer_ns() - t0 < 2000000ull) {
          }
        }
      } else {
        // ------------------------------------------------------------ products
        const uint32_t el = elect_one();
        uint32_t it = 0, items = 0;
        bool issued = false;
        const uint32_t q = smem_u32(smem + OFF_Q);
        auto wait = [&](uint64_t* b, uint32_t parity) {
          ok = ok && tree_wait(b, parity, bar, a.status);
          ok = __all_sync(0xffffffffu, ok);
          tc_fence_after();
          return ok;
        };
        while (ok && w.next(a, first, last)) {
          const int n = w.u1 - w.u0;
          const uint32_t id_s = idesc_f16(128, w.rows <= 32 ? 32 : w.rows <= 64 ? 64 : 128, 0, 0);
          const uint32_t id_o = idesc_f16(128, w.rows <= 64 ? 64 : 128, 1, 1);
          auto scores = [&](uint32_t i) {
            const uint32_t buf = i & 1, ph = (i >> 1) & 1;
            if (!wait(&bar->k_full[buf], ph) || !wait(&bar->s_empty[buf], ph ^ 1)) return;
#pragma unroll
            for (int x = 0; x < 8; ++x)
              umma_bf16_ts(tmem + COL_S + buf * 128, tmem + COL_K + buf * 64 + x * 8,
                           sdesc_sw128(q + (x >> 2) * HALF_TILE + (x & 3) * 32, 16, 1024), id_s, x > 0, el);
            umma_commit(&bar->s_full[buf], el);
            issued = true;
          };
          if (!wait(&bar->q_full, items & 1)) break;
          scores(it);
          for (int j = 0; j < n && ok; ++j, ++it) {
            if (j + 1 < n) scores(it + 1);
            if (!ok || (j == 0 && !wait(&bar->o_empty, (items & 1) ^ 1))) break;
            const uint32_t buf = it & 1, ph = (it >> 1) & 1;
            if (!wait(&bar->v_full[buf], ph) || !wait(&bar->p_full[buf], ph)) break;
            const uint32_t v = smem_u32(smem + OFF_V + buf * TILE), p = smem_u32(smem + OFF_P + buf * TILE);
#pragma unroll
            for (int x = 0; x < 8; ++x)  // 16 keys a step
              umma_bf16(tmem + COL_O, sdesc_sw128(v + x * 2048, HALF_TILE, 1024), sdesc_sw128(p + x * 2048, HALF_TILE, 1024),
                        id_o, (j | x) > 0, el);
            umma_commit(&bar->o_done[buf], el);
          }
          ++items;
        }
        if (!ok && issued) {
          umma_commit(&bar->drain, el);
          mbar_wait_drain(&bar->drain, 0, 200000000ull);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == TR_GROUPS * 4 + 1) {
    __syncwarp();
    tmem_dealloc<false>(tmem, 512);
  }
}

// Joins the partial outputs of a row: with W the largest partial log-sum-exp,
// O = sum 2^(lse_i - W) O_i / sum 2^(lse_i - W).  A warp per node and query
// head; zeros for a sequence that is left out.
__global__ void __launch_bounds__(256) attn_tree_join_kernel(const TreeArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t at = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (at >= static_cast<int64_t>(a.T) * a.n_q) return;
  const int t = static_cast<int>(at / a.n_q), head = static_cast<int>(at - static_cast<int64_t>(t) * a.n_q);
  int b = -1;
  for (int x = 0; x < a.B && b < 0; x += 32) {
    const bool here = x + lane < a.B && t >= a.cu[x + lane] && t < a.cu[x + lane + 1];
    const uint32_t m = __ballot_sync(0xffffffffu, here);
    if (m) b = x + __ffs(m) - 1;
  }
  if (b < 0) return;
  const TreeSeq s = tree_seq(a, b, false);
  uint2* out = reinterpret_cast<uint2*>(a.O + at * 128 + lane * 4);
  if (s.n == 0) {
    *out = make_uint2(0, 0);
    if (lane == 0) a.lse[at] = -INFINITY;
    return;
  }
  const int kvh = head / a.group, row = (t - s.q0) * a.group + head - kvh * a.group;
  const int tile = row / TREE_ROWS, c = row - tile * TREE_ROWS;
  const int cost = tree_cost(s.rows(tile, a.group));
  const int64_t per = a.places[a.B + 1];
  const int64_t u0 = a.places[b] + kvh * s.place_kv + tile * (static_cast<int64_t>(s.units) * TR_COST_MANY + TR_END) + TR_END;
  const int c0 = static_cast<int>(u0 / per), c1 = static_cast<int>((u0 + static_cast<int64_t>(s.units - 1) * cost) / per);
  if (c0 == c1) return;  // that CTA wrote the output
  float W = -INFINITY;
  for (int x = c0; x <= c1; ++x) W = fmaxf(W, a.part_lse[(2ll * x + (x == c0 ? 1 : 0)) * a.part_rows + c]);
  const float W0 = W == -INFINITY ? 0.f : W;
  float acc[4] = {0.f, 0.f, 0.f, 0.f}, sum = 0.f;
  for (int x = c0; x <= c1; ++x) {
    const int64_t p = (2ll * x + (x == c0 ? 1 : 0)) * a.part_rows + c;
    const float wgt = exp2_sfu(a.part_lse[p] - W0);
    const float4 v = *reinterpret_cast<const float4*>(a.part + p * 128 + lane * 4);
    sum += wgt;
    acc[0] += wgt * v.x;
    acc[1] += wgt * v.y;
    acc[2] += wgt * v.z;
    acc[3] += wgt * v.w;
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  *out = make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv));
  if (lane == 0) a.lse[at] = sum == 0.f ? -INFINITY : W * 0.69314718056f + logf(sum);
}

}  // namespace

cudaError_t launch_attn_tree(const TreeArgs& a, int sms, cudaStream_t s) {
  cudaError_t e = attn_smem_attribute(reinterpret_cast<const void*>(attn_tree_kernel), 7, TR_SMEM);
  if (e != cudaSuccess) return e;
  e = attn_launch(attn_tree_kernel, std::min(sms, TREE_MAX_CTAS), TR_THREADS, TR_SMEM, s, a);
  if (e != cudaSuccess) return e;
  return attn_launch(attn_tree_join_kernel, (static_cast<int64_t>(a.T) * a.n_q + 7) / 8, 256, 0, s, a);
}

}  // namespace coda

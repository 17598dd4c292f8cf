// Attention of drafted tokens over the 4-bit cache: node i of a sequence's tree
// sees the committed prefix, its ancestors and itself,
//   s_ij = scale q_i . k_j,  O_i = sum_j exp(s_ij - lse_i) v_j.
//
// Floor: 152 bytes per cached token and key/value head feed 2 * 128
// multiply-adds for each row, a row being a node and a query head of the
// group.  Up to about 80 rows the bytes take longer at this chip's rates, then the
// products.
//
// Work: the rows of a sequence and key/value head are cut into tiles of up to
// 128, and the keys of a tile into units of 128.  The units of the whole batch
// form one line, with places for the ends of every tile, that the CTAs (one per SM)
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
// thread of the weights has one key: its scales are two registers, sums over
// keys stay in the thread until the end, and no maximum is exchanged unless a
// weight passes its bound.  (K' from shared memory would take the whole of its
// bandwidth with 128 rows; from TMEM the product runs at its own rate.)
//
// A weight carries its value's row scale rs:
//   P' = 2^t,  t = scale log2(e) rs_k (q . k') + log2 rs_v - r,  l = sum P' / rs_v
// with a reference r per row that rises when some t passes 10 (f16 holds 2^15),
// so P' is rounded by 2^-11 of itself or 2^-25 of the largest weighted row
// scale.  l, r and O are fp32.  Weights are computed and summed in one
// pass over the scores; where one turns out to pass the bound the pass is taken
// back (the sums with a minus), the reference rises and a second pass follows.
// A 2^t below fp32's least, 2^-126, may count in l where its value is much smaller
// than others.  With row scales of 2^-90 to 1 it is 2^-36 of l at most; from a key
// with a larger one on (values beyond 2688) units are treated as those that pass
// the bound, and what was lost is added in a third pass.  (l itself is 2^-117 or
// more: values beyond 1e33 leave its smaller terms no room.)
//
// Roles: four warpgroups of weights with a quarter of the tile's rows each (their
// sums fit the 72 registers that 28 warps leave), two of them with half each for
// up to 64 rows; four warps each for K' and V', one that copies by tensor maps,
// one that issues the products, two idle.  Stages of the cache, scores, K', V'
// and P' are double or triple, so that all roles work on different units.
//
// What bounds it: instructions, and fetching them.  A unit of 128 keys takes 1900
// to 2900 clocks (at 32 to 128 rows) for 850 of copies and 130 to 510 of
// products, and 5500 to 8600 warp instructions (2.95 a clock and SM at 128 rows).
// Weights, four per score, and unpacking, two per element, are 2600 to 4100 of them;
// the others (waits, barriers, votes, addresses of 26 warps) have not been taken
// apart.  The roles' loops take turns in the four schedulers and evict each other
// from the instruction caches.  So code that is run in every unit counts, and how
// often:
//   waits without a clock and a flag in their loops   192 -> 150 us (64 chains)
//   one copy of what sets and raises a reference      150 -> 140
//   columns in sixteens (a branch for four)           184 -> 178 (8 trees)
//   one barrier for scores and scales, one for scores
//   read and weights written                          190 -> 184
//   unpacking rolled, its waits' loads ahead          268 -> 218 (8 trees)
//   one copy of the weights' code                     299 -> 268
//   no register spilled                               580 -> 321
// Two teams of warpgroups for alternate units (126 for 139 us at two long
// documents) and 32 warps with eight for V' cost more elsewhere than they gained;
// the next item's Q in front of an item's end gained nothing.
//
// Now, in a graph: 64 + 8 heads, 64 chains of 4 over up to 8192 keys 136 us
// (floor 45), 24 trees of 1 to 64 nodes over 60 to 6000 keys 191 us (44), a chain
// of 6 over 777 keys 18 us; 32 + 8 heads, 8 trees of 64 nodes over 16384 keys
// 180 us (71), trees of 16 and 11 nodes over 131055 and 100001 keys 128 us (42).
#include <algorithm>

#include "coda_attn.cuh"
#include "coda_attn_tree.cuh"
#include "coda_internal.h"
#include "coda_kvrow.cuh"
#include "coda_status.h"

namespace coda {
namespace {

constexpr int TR_THREADS = 896;
constexpr int TR_GROUPS = 4;  // warpgroups of weights: warps 0-15
constexpr int TR_KEYS = 16, TR_VALUES = 20, TR_COPY_WARP = 24, TR_MMA_WARP = 25;  // first warps of the other roles
constexpr int TR_UNIT = 128;
constexpr int TR_STAGES = 3;
// A stage holds a unit's rows of the cache part by part (a page, or 128 keys of
// one), each part as the copies leave it: keys, then values.  16-byte pieces of
// the codes are exchanged by the 64-byte swizzle.
constexpr int RW_CODES = 0, RW_SF = 16384, RW_RS = 18432;
constexpr int TR_RAW = 19456;
// Row of a key's codes (and of its value's, 1 << shift rows on) in a stage;
// likewise of its block scales and row scales.
__device__ __forceinline__ int raw_row(int key, int shift) { return ((key >> shift) << (shift + 1)) + (key & ((1 << shift) - 1)); }
constexpr uint32_t TILE = 32768, HALF_TILE = 16384;  // 128 x 128 f16, as two halves of 64 columns
constexpr uint32_t OFF_Q = 0, OFF_P = TILE, OFF_V = 3 * TILE, OFF_RAW = 5 * TILE;
constexpr uint32_t OFF_ROW = OFF_RAW + TR_STAGES * TR_RAW;  // [2][128] minus the rows' references, by item
constexpr uint32_t OFF_KEY = OFF_ROW + 1024;                // [4][128] row scale of the key, log2 of the value's
constexpr uint32_t OFF_RED = OFF_KEY + 4096;                // [4][192] exchange of a warpgroup
constexpr uint32_t OFF_BAR = OFF_RED + TR_GROUPS * 192 * 4;
constexpr uint32_t TR_SMEM = 896 + OFF_BAR + 1152;
static_assert(TR_SMEM <= 232448, "shared memory per CTA");
constexpr uint32_t COL_S = 0, COL_O = 256, COL_K = 384;  // TMEM columns: S twice, O, K' twice (64 each)
constexpr int TR_HALF_ROWS = 64;               // up to here two warpgroups: 64 chains 140 us for 152, long documents 138 for 140
constexpr float TR_RAISE = 10.f;               // a weight may pass 2^10 ...
constexpr uint32_t TR_RAISE_F16 = 0x6400;      // ... 1024 in f16
constexpr uint32_t TR_NO_MORE = 1u << 31;
// The least row scale of a weight, in log2: smaller ones take it (V' the rest), and
// rows of zeros, whose own says nothing.
constexpr float TR_LEAST = -90.f;

// Places of a stretch's ends on the line, a unit having one: their loads, sums and
// stores take as long as four to seven units.  Geometric mean over 80 batches drawn
// at random (1 to 64 sequences of up to 131072 keys, 1 to 64 nodes, all groups):
// 3 22.6 us, 4 22.5, 5 22.5, 6 22.4, 7 22.5; with a unit of more than 64 rows a fifth
// dearer (5, 6, ends 24) 23.0.
constexpr int TR_END = 5;

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
__device__ __forceinline__ void mbar_arrive_n(uint64_t* bar, uint32_t n) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(n) : "memory");
}
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
__device__ __forceinline__ void tmem_ldn(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : CODA_R8(r, 0)
      : "r"(taddr)
      : "memory");
}
__device__ __forceinline__ uint32_t hmax2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// The larger one, NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
      CODA_W8(r, 0), CODA_W8(r, 8)
      : "memory");
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), CODA_W8(r, 0)
               : "memory");
}

// A sequence's work.
struct TreeSeq {
  int q0, n, len;     // first token, nodes, cached tokens; n = 0: no work
  int units, tiles;
  int64_t place_kv;   // places per key/value head: of each tile, its ends' and units'
  __device__ __forceinline__ int rows(int tile, int group) const { return min(TREE_ROWS, n * group - tile * TREE_ROWS); }
};
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
  s.place_kv = s.n > 0 ? static_cast<int64_t>(s.tiles) * (s.units + TR_END) : 0;
  return s;
}
// First unit at `place` or behind it, of an item at `base`.
__device__ __forceinline__ int unit_at(int64_t place, int64_t base, int units) {
  return static_cast<int>(max(static_cast<int64_t>(0), min(static_cast<int64_t>(units), place - base - TR_END)));
}

// A CTA's way along the line: items (sequence, key/value head, tile) with the
// units [u0, u1) that it takes of each.  Every warp walks it for itself.
struct TreeWalk {
  int b, item;            // sequence, next item of it
  int64_t base;           // place of that item
  int64_t first, last;    // the CTA's places
  TreeSeq s;
  // current
  int kvh, tile, rows, u0, u1;
  __device__ __forceinline__ bool next(const TreeArgs& a) {
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
      u0 = unit_at(first, base, s.units);
      u1 = unit_at(last, base, s.units);
      base += s.units + TR_END;
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

extern __shared__ __align__(128) uint8_t tree_smem[];
// Aligned, and known to the compiler as shared memory.
__device__ __forceinline__ uint8_t* tree_shared() { return tree_smem + (-smem_u32(tree_smem) & 1023u); }

// What a CTA does of an item; the copying warp walks the line and leaves it in
// shared memory, ahead of the item's first unit.
struct TreeItem {
  int q0, n, len, kvh;
  int row0, rows;      // of the tile, among the sequence's rows
  int u0, u1, units;
};
constexpr int TR_ITEMS = 8;  // the copies are at most five units ahead

// Where the copies are on the line.
struct TreeCopies {
  TreeWalk w;
  int u;               // next unit of the walk's item
  uint32_t it, items;  // units and items so far
  int done;            // the end has been told
};

struct TreeBars {
  TreeItem item[TR_ITEMS];
  TreeCopies copies;
  uint64_t raw_full[TR_STAGES], raw_empty[TR_STAGES];
  uint64_t k_full[2], s_full[2], p_full[2], o_done[2];
  uint64_t q_full, o_empty, drain;
  uint64_t item_full[TR_ITEMS];
  uint32_t keys_in[TR_STAGES];  // bit i: keys 16 i .. 16 i + 15 of the stage are there; TR_NO_MORE: no unit, nor behind it
  int left[TR_STAGES];          // keys of the sequence from the stage's first on
  int64_t scan[TR_THREADS / 32], before;  // of the places, and the sequence that the CTA begins with
  int seq;
  uint32_t tmem;
};
static_assert(sizeof(TreeBars) <= 1152, "barrier area");

// A wait that gives up after 2^19 tries, for each of which the hardware may suspend
// the warp for about 2 us: a second in all.  As short as can be: every role waits
// in every unit.
__device__ __forceinline__ bool tree_wait(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .u32 n;\n\t"
      "mov.u32 n, 0;\n\t"
      "again_%=:\n\t"
      "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, 2000;\n\t"
      "@p bra done_%=;\n\t"
      "add.u32 n, n, 1;\n\t"
      "setp.ge.u32 p, n, 524288;\n\t"
      "@!p bra again_%=;\n\t"
      "setp.ne.u32 p, n, n;\n\t"
      "done_%=:\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

__device__ __forceinline__ void tma_load_5d(void* dst, const CUtensorMap* m, uint64_t* bar, int x, int y, int z, int v, int w,
                                            uint32_t p) {
  asm volatile(
      "{\n\t.reg .pred P;\n\tsetp.ne.b32 P, %8, 0;\n\t"
      "@P cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6, %7}], [%2];\n\t}" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(v), "r"(w), "r"(p)
      : "memory");
}
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* m, uint64_t* bar, int x, int y, int z, int v,
                                            uint32_t p) {
  asm volatile(
      "{\n\t.reg .pred P;\n\tsetp.ne.b32 P, %7, 0;\n\t"
      "@P cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];\n\t}" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(v), "r"(p)
      : "memory");
}

// Copies of the next unit of the line into its stage, by one warp: three per
// part, keys and values together.  Lane i holds the page of part i, read a unit
// ahead (`page`).
__device__ __forceinline__ bool copy_unit(const TreeArgs& a, const CUtensorMap* codes, const CUtensorMap* sf,
                                          const CUtensorMap* scale, uint8_t* smem, TreeBars* bar, int lane, uint32_t el,
                                          int& page) {
  TreeCopies& c = bar->copies;
  const KvCache& kc = a.c;
  const int shift = min(kc.page_shift, 7);  // keys of a part
  const uint32_t st = c.it % TR_STAGES;
  bool ok = tree_wait(&bar->raw_empty[st], ((c.it / TR_STAGES) & 1) ^ 1);
  if (!__all_sync(0xffffffffu, ok)) return false;
  auto page_of = [&](int u) {  // of this lane's part of unit u; -1: nothing there
    const int k = u * TR_UNIT + (lane << shift);
    return u < c.w.u1 && (lane << shift) < TR_UNIT && k < c.w.s.len
               ? a.table[static_cast<int64_t>(c.w.b) * a.max_pages + (k >> kc.page_shift)]
               : -1;
  };
  if (c.u == c.w.u1) {  // the next item
    int more = 0;
    if (lane == 0) {
      TreeWalk w = c.w;
      more = w.next(a);
      c.w = w;
      c.u = w.u0;
      TreeItem& to = bar->item[c.items % TR_ITEMS];
      to.rows = 0;
      if (more) {
        to.q0 = w.s.q0;
        to.n = w.s.n;
        to.len = w.s.len;
        to.kvh = w.kvh;
        to.row0 = w.tile * TREE_ROWS;
        to.rows = w.rows;
        to.u0 = w.u0;
        to.u1 = w.u1;
        to.units = w.s.units;
      } else {
        c.done = 1;
        bar->keys_in[st] = TR_NO_MORE;
        mbar_arrive(&bar->raw_full[st]);
      }
      mbar_arrive(&bar->item_full[c.items++ % TR_ITEMS]);
    }
    __syncwarp();
    if (!__shfl_sync(0xffffffffu, more, 0)) return true;
    page = page_of(c.u);
  }
  const int u = c.u, len = c.w.s.len;
  const int k = u * TR_UNIT + (lane << shift);
  const bool named = (lane << shift) < TR_UNIT && k < len;
  const bool in = named && page >= 0 && page < kc.num_pages;
  if (named && !in) atomicOr(a.status, CODA_DEV_PAGE_RANGE);
  const uint32_t parts = __ballot_sync(0xffffffffu, in);
  const int groups = 1 << (shift - 4);  // of 16 keys in a part
  const uint32_t mask = __reduce_or_sync(0xffffffffu, in ? ((1u << groups) - 1) << (lane * groups) : 0);
  if (lane == 0) {
    bar->keys_in[st] = mask;
    bar->left[st] = len - u * TR_UNIT;
    if (parts == 0) mbar_arrive(&bar->raw_full[st]);
  }
  mbar_arrive_expect_tx(&bar->raw_full[st], __popc(parts) * (152u << shift), lane == 0 && parts != 0);
  __syncwarp();
  uint8_t* to = smem + OFF_RAW + st * TR_RAW;
  const int row = (u * TR_UNIT) & ((1 << kc.page_shift) - 1);  // of the page, where it holds more than a unit
  for (uint32_t left = parts; left; left &= left - 1) {
    const int p = __ffs(left) - 1;
    const int pg = __shfl_sync(0xffffffffu, page, p);
    tma_load_5d(to + RW_CODES + (p << (shift + 7)), codes, &bar->raw_full[st], 0, row, c.w.kvh, 0, pg, el);
    tma_load_4d(to + RW_SF + (p << (shift + 4)), sf, &bar->raw_full[st], row * 2, c.w.kvh, 0, pg, el);
    tma_load_4d(to + RW_RS + (p << (shift + 3)), scale, &bar->raw_full[st], row, c.w.kvh, 0, pg, el);
  }
  page = page_of(u + 1);
  __syncwarp();
  if (lane == 0) {
    c.u = u + 1;
    ++c.it;
  }
  __syncwarp();
  return true;
}

// The scores of unit i, once its keys are unpacked (those of two units ago have
// been read: the outputs of that unit, issued before, have waited for its weights).
// The places are constants
// (BUF is i's parity), so that descriptors stay in uniform registers: with
// computed ones eight products took twice the time to issue that they run.
template <int BUF>
__device__ __forceinline__ bool issue_scores(uint8_t* smem, TreeBars* bar, uint32_t tmem, uint32_t i, uint32_t id,
                                             uint32_t el) {
  const uint32_t ph = (i >> 1) & 1;
  const bool ok = tree_wait(&bar->k_full[BUF], ph);
  if (!__all_sync(0xffffffffu, ok)) return false;
  tc_fence_after();
  const uint32_t q = smem_u32(smem + OFF_Q);
#pragma unroll
  for (int x = 0; x < 8; ++x)
    umma_bf16_ts(tmem + COL_S + BUF * 128, tmem + COL_K + BUF * 64 + x * 8,
                 sdesc_sw128(q + (x >> 2) * HALF_TILE + (x & 3) * 32, 16, 1024), id, x > 0, el);
  umma_commit(&bar->s_full[BUF], el);
  if (el) mbar_arrive(&bar->s_full[BUF]);
  return true;
}
// O^T += V'^T P'^T of unit i; first: of an item, whose predecessor's O has left.
template <int BUF>
__device__ __forceinline__ bool issue_outputs(uint8_t* smem, TreeBars* bar, uint32_t tmem, uint32_t i, uint32_t id,
                                              bool first, uint32_t item, uint32_t el) {
  const uint32_t ph = (i >> 1) & 1;
  const bool ok = tree_wait(&bar->p_full[BUF], ph) && (!first || tree_wait(&bar->o_empty, (item & 1) ^ 1));
  if (!__all_sync(0xffffffffu, ok)) return false;
  tc_fence_after();
  const uint32_t v = smem_u32(smem + OFF_V + BUF * TILE), p = smem_u32(smem + OFF_P + BUF * TILE);
  const uint32_t more = !first;
#pragma unroll
  for (int x = 0; x < 8; ++x)  // 16 keys a step
    umma_bf16(tmem + COL_O, sdesc_sw128(v + x * 2048, HALF_TILE, 1024), sdesc_sw128(p + x * 2048, HALF_TILE, 1024), id,
              x > 0 ? 1u : more, el);
  umma_commit(&bar->o_done[BUF], el);
  return true;
}
// After a wait that ran out: let what was issued land before the CTA's memory
// is used again.
__device__ __forceinline__ void tree_drain(TreeBars* bar, int warp, int lane) {
  if (warp == TR_MMA_WARP) {
    umma_commit(&bar->drain, lane == 0);
    mbar_wait_drain(&bar->drain, 0, 200000000ull);
  } else if (warp == TR_COPY_WARP) {
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 2000000ull) {
    }
  }
}

// Unit `it` of the stage ring, or none: its groups of 16 keys, and the keys of the
// sequence from the warp's first (32 g) on.
struct UnitIn {
  uint32_t on;
  int left;
};
__device__ __forceinline__ bool unit_in(TreeBars* bar, uint32_t it, int g, UnitIn& x, bool& more) {
  const uint32_t st = it % TR_STAGES;
  const bool ok = tree_wait(&bar->raw_full[st], (it / TR_STAGES) & 1);
  x.on = bar->keys_in[st];
  x.left = bar->left[st] - 32 * g;
  more = __all_sync(0xffffffffu, ok && x.on != TR_NO_MORE);
  return ok;
}

// K' of unit `it` by four warps, a thread per key, to the lane of TMEM that is
// its row, and the key's scales.  False: a wait ran out; without `more`, no unit was
// left.  (Rolled, as below: warps of all roles share a scheduler, and their
// straight-line code does not fit its instruction cache together.)
__device__ __forceinline__ bool unpack_keys(uint8_t* smem, TreeBars* bar, uint32_t tmem, int g, int lane,
                                            uint32_t it, int shift, int krow, bool& more) {
  const uint32_t st = it % TR_STAGES, buf = it & 1, ph = (it >> 1) & 1;
  UnitIn x;
  const bool here = unit_in(bar, it, g, x, more);
  const uint8_t* raw = smem + OFF_RAW + st * TR_RAW;
  const bool in = ((x.on >> (2 * g + (lane >> 4))) & 1u) && lane < x.left;  // else whatever the stage held before
  const uint2 sfk = *reinterpret_cast<const uint2*>(raw + RW_SF + krow * 8);
  const uint2 sfv = *reinterpret_cast<const uint2*>(raw + RW_SF + (krow + (1 << shift)) * 8);
  const float rsk = *reinterpret_cast<const float*>(raw + RW_RS + krow * 4);
  const float rsv = *reinterpret_cast<const float*>(raw + RW_RS + (krow + (1 << shift)) * 4);
  const uint8_t* kc = raw + RW_CODES + krow * 64;
  uint4 v = *reinterpret_cast<const uint4*>(kc + (((krow >> 1) & 3) << 4));
  if (!more) return here;
  const bool ok = tree_wait(&bar->s_full[buf], ph ^ 1);  // the scores of two units ago have read K'
  if (!__all_sync(0xffffffffu, ok)) return false;
  tc_fence_after();
  uint64_t sf8 = in ? static_cast<uint64_t>(sfk.y) << 32 | sfk.x : 0;
  const uint32_t to = tmem + (static_cast<uint32_t>(g * 32) << 16) + COL_K + buf * 64;
#pragma unroll 1
  for (int q = 0; q < 4; ++q, sf8 >>= 16) {
    const uint4 now = v;
    v = *reinterpret_cast<const uint4*>(kc + (((q + 1) ^ (krow >> 1)) & 3) * 16);
    const uint32_t two = e4m3x2_f16(static_cast<uint32_t>(sf8) & 0xFFFFu);
    const uint32_t s0 = __byte_perm(two, two, 0x1010), s1 = __byte_perm(two, two, 0x3232);
    uint32_t o[16];
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      uint32_t f[4];
      e2m1x8_f16(w == 0 ? now.x : w == 1 ? now.y : w == 2 ? now.z : now.w, f);
#pragma unroll
      for (int i = 0; i < 4; ++i) o[w * 4 + i] = hmul2(f[i], w < 2 ? s0 : s1);
    }
    tmem_st16(to + q * 16, o);
  }
  const bool sick = (((sfv.x & 0x7F7F7F7Fu) + 0x01010101u) | ((sfv.y & 0x7F7F7F7Fu) + 0x01010101u)) & 0x80808080u;
  const bool zeros = ((sfv.x | sfv.y) & 0x7F7F7F7Fu) == 0;
  // a key that is not finite somewhere: NaN, and finite codes, so that rows that
  // do not see it stay clear of it
  const bool poison = sick || !(fabsf(rsk) <= 3.4e38f) || !(fabsf(rsv) <= 3.4e38f);
  float2 meta;
  meta.x = !in ? 0.f : poison ? 1.f : rsk;
  // below 2^-90 the sum l would pass fp32's end (2^10 / 2^-90 for a key, room for
  // 2^26 of them): V' takes the rest
  meta.y = !in ? -INFINITY : poison ? __uint_as_float(0x7FC00000u) : zeros || rsv < 0x1p-90f ? TR_LEAST : log2f(rsv);
  *reinterpret_cast<float2*>(smem + OFF_KEY + (it & 3) * 1024 + (g * 32 + lane) * 8) = meta;
  tmem_st_wait();
  tc_fence_before();
  __syncwarp();
  if (lane == 0) {
    mbar_arrive(&bar->k_full[buf]);
    mbar_arrive(&bar->raw_empty[st]);
  }
  return true;
}

// V' of unit `it` by four warps: a lane takes sixteen elements (piece p of eight)
// of keys k0 + 4 j of the warp's 32.  Eight lanes write four pieces of two
// neighbouring keys, which the swizzle sends to different banks.
struct ValueLane {
  uint32_t v[2];    // codes of the values: first 16 keys, the others
  uint32_t sf[2];   // their block scales
  uint32_t to;      // where V' goes; even and odd j differ in one bit of the swizzled places
  int k0, row;      // and the row of key `lane`
  __device__ __forceinline__ ValueLane(int g, int lane, int shift) {
    const int piece = ((lane >> 1) & 4) | (lane & 3);
    k0 = ((lane >> 2) & 1) | ((lane >> 3) & 2);
    row = raw_row(g * 32 + lane, shift) + (1 << shift);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = raw_row(g * 32 + 16 * h + k0, shift) + (1 << shift);
      sf[h] = RW_SF + r * 8 + piece;
      v[h] = RW_CODES + r * 64 + ((((piece >> 1) ^ (r >> 1)) & 3) << 4) + (piece & 1) * 8;
    }
    to = (piece >> 2) * HALF_TILE + (g * 32 + k0) * 128 + (((2 * (piece & 3)) ^ k0) << 4);
  }
};
__device__ __forceinline__ void value_out(uint8_t* a0, uint8_t* a1, uint2 c, uint32_t s) {
  uint32_t f[4], e[4];
  e2m1x8_f16(c.x, f);
  e2m1x8_f16(c.y, e);
  *reinterpret_cast<uint4*>(a0) = make_uint4(hmul2(f[0], s), hmul2(f[1], s), hmul2(f[2], s), hmul2(f[3], s));
  *reinterpret_cast<uint4*>(a1) = make_uint4(hmul2(e[0], s), hmul2(e[1], s), hmul2(e[2], s), hmul2(e[3], s));
}
__device__ __forceinline__ bool unpack_values(uint8_t* smem, TreeBars* bar, int g, int lane, uint32_t it, int shift,
                                              const ValueLane& x, bool& more) {
  const uint32_t st = it % TR_STAGES, buf = it & 1, ph = (it >> 1) & 1;
  UnitIn u;
  const bool here = unit_in(bar, it, g, u, more);
  uint8_t* raw = smem + OFF_RAW + st * TR_RAW;
  // a row scale below 2^-90 (unpack_keys): what it is of that
  const float rsv = *reinterpret_cast<const float*>(raw + RW_RS + x.row * 4);
  const uint2 sfv = *reinterpret_cast<const uint2*>(raw + RW_SF + x.row * 8);
  const bool in = ((u.on >> (2 * g + (lane >> 4))) & 1u) && lane < u.left;
  const float less = in && rsv < 0x1p-90f ? rsv * 0x1p90f : 1.f;
  const bool sick = (((sfv.x & 0x7F7F7F7Fu) + 0x01010101u) | ((sfv.y & 0x7F7F7F7Fu) + 0x01010101u)) & 0x80808080u;
  const bool odd = __any_sync(0xffffffffu, !in || less != 1.f || sick);
  if (!more) return here;
  const bool ok = tree_wait(&bar->o_done[buf], ph ^ 1);
  if (!__all_sync(0xffffffffu, ok)) return false;
  uint8_t* out = smem + OFF_V + buf * TILE;
#pragma unroll 1
  for (int h2 = 0; h2 < 4; ++h2) {
    const int h = h2 >> 1;
    const uint32_t v = (h ? x.v[1] : x.v[0]) + (h2 & 1) * 512, sf = (h ? x.sf[1] : x.sf[0]) + (h2 & 1) * 64;
    uint2 c[2];
    uint32_t s[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      c[j] = *reinterpret_cast<const uint2*>(raw + (v ^ ((j & 1) * 32)) + j * 256);
      s[j] = raw[sf + j * 32] * 0x101u;
    }
    if (odd) {
      keep_branch();
      // zeros outside the sequence, and for a scale that is NaN (the key's weights
      // are NaN then)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int k = 8 * h2 + 4 * j + x.k0;
        const float by = __shfl_sync(0xffffffffu, less, k);
        const uint32_t t = e4m3x2_f16((s[j] & 0x7Fu) != 0x7Fu ? s[j] : 0u);
        s[j] = ((u.on >> (2 * g + h)) & 1u) && k < u.left ? pack_f16(f16_lo(t) * by, f16_hi(t) * by) : 0u;
      }
    } else {
#pragma unroll
      for (int j = 0; j < 2; ++j) s[j] = e4m3x2_f16(s[j]);
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint32_t turn = j * 64, by = h2 * 1024 + j * 512;  // of the swizzle
      value_out(out + (x.to ^ turn) + by, out + (x.to ^ turn ^ 16) + by, c[j], s[j]);
    }
  }
  fence_async_smem();
  __syncwarp();
  if (lane == 0) {
    mbar_arrive(&bar->p_full[buf]);
    mbar_arrive(&bar->raw_empty[st]);
  }
  return true;
}

// Warpgroups that share a tile's rows, and the columns that each takes, in
// sixteens: 16 or 32.
__device__ __forceinline__ int tree_groups(int rows) { return rows <= TR_HALF_ROWS ? 2 : TR_GROUPS; }
__device__ __forceinline__ int tree_columns(int rows) {
  const int per = 16 * tree_groups(rows);
  return (rows + per - 1) / per * 16;
}

// A warpgroup's part of one stretch: the weights of nc columns of the tile, in
// chunks of 8.  `it` counts the CTA's units.  False: a wait ran out.
__device__ __forceinline__ bool tree_softmax(const TreeArgs& a, uint8_t* smem, TreeBars* bar, uint32_t tmem, uint32_t item,
                                             uint32_t& it) {
  const int wg = threadIdx.x >> 7;
  const int tid = threadIdx.x & 127, warp = tid >> 5, lane = tid & 31;
  const int id = 1 + wg;                 // named barrier
  const TreeItem& w = bar->item[item % TR_ITEMS];
  const int row0 = w.row0;
  const int nc = tree_columns(w.rows), col0 = wg * nc;
  const uint32_t arrive = TR_GROUPS / tree_groups(w.rows);  // for the warps without rows too
  constexpr int NC = TREE_ROWS / TR_GROUPS;  // the most there may be
  float* red = reinterpret_cast<float*>(smem + OFF_RED) + wg * 192;                           // [4][32] and more
  float* nref = reinterpret_cast<float*>(smem + OFF_ROW) + (item & 1) * TREE_ROWS + col0;  // -r per column
  bool ok = true;

  // ---- Q in f16: the warpgroup's rows scaled by one power of two, to a maximum
  // in [2^14, 2^15) (an element below 2^-39 of it is rounded by 2^-39: scores are
  // exponents, their absolute error counts); rows behind the tile's are zeros.
  // Sixteen lanes per row.
  float factor;  // of the scores
  {
    uint4 v[NC / 8];
    const int piece = tid & 15;
    float mx = 0.f;
#pragma unroll
    for (int i = 0; i < NC / 8; ++i) {
      const int c = col0 + 8 * i + (tid >> 4), row = row0 + c;
      v[i] = make_uint4(0, 0, 0, 0);
      if (8 * i < nc && c < w.rows) {
        const int node = row / a.group, head = w.kvh * a.group + row - node * a.group;
        v[i] = *reinterpret_cast<const uint4*>(a.Q + (static_cast<int64_t>(w.q0) + node) * a.ldq + head * 128 + piece * 8);
      }
    }
#pragma unroll
    for (int i = 0; i < NC / 8; ++i) {
      float y[8];
      bf16x8_to_f32(v[i], y);
#pragma unroll
      for (int k = 0; k < 8; ++k) mx = fmaxf(mx, fabsf(y[k]) <= 3.4e38f ? fabsf(y[k]) : 0.f);
    }
    mx = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(mx)));
    if (lane == 0) red[warp] = mx;
    group_any(id, false);
    mx = fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3]));
    // 2^-e scales the maximum to [2^14, 2^15), as two factors within fp32's range
    const int e = mx == 0.f ? 0 : max(static_cast<int>(__float_as_uint(mx) >> 23) - 127, -126) - 14;
    const int e0 = max(-126, min(126, e)), e1 = e - e0;
    const float down0 = __uint_as_float(static_cast<uint32_t>(127 - e0) << 23);
    const float down1 = __uint_as_float(static_cast<uint32_t>(127 - e1) << 23);
    factor = fmaxf(a.scale_log2 / down0 / down1, 1.2e-38f);
#pragma unroll
    for (int i = 0; i < NC / 8; ++i) {
      if (8 * i >= nc) break;
      const int c = col0 + 8 * i + (tid >> 4);
      float y[8];
      bf16x8_to_f32(v[i], y);
#pragma unroll
      for (int k = 0; k < 8; ++k) y[k] = y[k] * down0 * down1;
      *reinterpret_cast<uint4*>(smem + OFF_Q + (piece >> 3) * HALF_TILE + c * 128 + (((piece & 7) ^ (c & 7)) << 4)) =
          make_uint4(pack_f16(y[0], y[1]), pack_f16(y[2], y[3]), pack_f16(y[4], y[5]), pack_f16(y[6], y[7]));
    }
  }
  if (tid < nc) nref[tid] = 0.f;  // no reference yet
  fence_async_smem();
  __syncwarp();
  if (lane == 0) mbar_arrive(&bar->q_full);  // (and that the item before is read: its end's place is P' now)

  // ---- what each row sees of its tree
  const int prefix = w.len - w.n;  // keys that every row sees
  // For each node the rows that see it, a bit each: a thread of the last
  // units has one key.
  uint32_t* seen = a.seen + (static_cast<int64_t>(blockIdx.x) * TR_GROUPS + wg) * TREE_MAX_NODES;
  const bool tree = a.parents != nullptr;
  group_any(id, false);  // red is read
  if (tree && min(w.u1 * TR_UNIT, w.len) > prefix) {
    int16_t* up = reinterpret_cast<int16_t*>(red);
    for (int i = tid; i < w.n; i += 128) {
      const int p = a.parents[w.q0 + i];
      const bool bad = p < -1 || p >= i;
      if (bad) atomicOr(a.status, CODA_DEV_TREE_RANGE);
      up[i] = static_cast<int16_t>(bad ? -1 : p);
      seen[i] = 0;
    }
    group_any(id, false);
    if (tid < nc && col0 + tid < w.rows)
      for (int j = (row0 + col0 + tid) / a.group; j >= 0; j = up[j]) atomicOr(seen + j, 1u << tid);
    group_any(id, false);
  }

  const uint32_t lanes = static_cast<uint32_t>(warp * 32) << 16;
  float l[NC];
#pragma unroll
  for (int c = 0; c < NC; ++c) l[c] = 0.f;
  bool unset = true;        // some column has no reference
  bool mine_unset = tid < nc;  // column tid
  bool large = false;       // a key of this thread had a row scale above 1
  const int u0 = w.u0, u1 = w.u1, nodes = w.n, group = a.group;

  for (int u = u0; u < u1; ++u, ++it) {
    const uint32_t buf = it & 1, ph = (it >> 1) & 1;
    // rows that see this key, where it is a node (or none of the sequence)
    const int d = u * TR_UNIT + tid - prefix;
    uint32_t sees = ~0u;
    if (d >= 0) {
      keep_branch();
      if (d >= nodes) {
        sees = 0;
      } else if (tree) {
        sees = __ldcg(seen + d);
      } else {
        const int64_t from = static_cast<int64_t>(d) * group - row0 - col0;  // rows from the node's own on
        sees = from <= 0 ? ~0u : from >= 32 ? 0 : ~0u << from;
      }
    }
    // the scores, and through the warp that issued them the keys' scales (the
    // unpacking is at most three units ahead: none of four places is lost)
    ok = ok && tree_wait(&bar->s_full[buf], ph);
    ok = __all_sync(0xffffffffu, ok);
    tc_fence_after();
    const float2 key = *reinterpret_cast<const float2*>(smem + OFF_KEY + (it & 3) * 1024 + tid * 8);
    const bool there = key.y != -INFINITY;
    float lr = key.y;
    float inv = there ? exp2_sfu(-lr) : 0.f;  // finite: it meets zero weights too
    const float rk = there ? fmaxf(key.x * factor, 1.2e-38f) : 0.f;  // not 0, so that -inf below stays what it is
    const uint32_t tS = tmem + lanes + COL_S + buf * 128 + col0, tO = tmem + lanes + COL_O + col0;
    bool odd = false;
    if (__any_sync(0xffffffffu, sees != ~0u || !(lr <= 0.f))) {  // scores that do not count become -inf where they lie
      keep_branch();
      const bool poison = lr != lr;
      if (poison) {
        lr = 0.f;
        inv = 1.f;
      } else if (lr > 0.f) {
        // A key whose row scale is above 1 is left out of the first weights, which
        // are taken back: 2^t might be infinite although 2^t / rs_v, without which it
        // cannot be, is no more than l.
        odd = true;
        lr = -INFINITY;
        inv = 0.f;
      }
#pragma unroll 1
      for (int q = 0; q < nc; q += 8) {
        uint32_t s[8];
        tmem_ldn(tS + q, s);
        const uint32_t m = sees >> q;
#pragma unroll
        for (int c = 0; c < 8; ++c) s[c] = !((m >> c) & 1) ? there ? 0xFF800000u : 0u : poison ? 0x7FC00000u : s[c];
        tmem_st8(tS + q, s);
      }
      tmem_st_wait();
    }
    bool lost = false;  // some weights may be below 2^-126 and count in the sum all the same
    // The largest exponent of each row over this unit's keys, to column tid.
    auto row_max = [&]() {
#pragma unroll 1
      for (int q = 0; q < nc; q += 8) {
        uint32_t s[8];
        tmem_ldn(tS + q, s);
        float v[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) v[c] = fmaf(__uint_as_float(s[c]), rk, lr + nref[q + c]);
        const float most = warp_columns<8, false>(v, lane);
        if (lane < 8) red[warp * 32 + q + lane] = most;
      }
      lost = group_any(id, odd || large);
      float m = -INFINITY;
      if (tid < nc) m = fmaxf(fmaxf(red[tid], red[32 + tid]), fmaxf(red[64 + tid], red[96 + tid]));
      group_any(id, false);
      return m;
    };
    // ---- P', into the place that the product of two units ago has read: it was
    // issued before these scores, so it is done.  Where some weight passes its
    // bound the round is taken back, the reference of that row rises, and a third
    // one follows.
    uint8_t* at = smem + OFF_P + buf * TILE + tid * 128;
    const uint64_t rk2 = f2_pack(rk, rk);
    float add = inv;
    // Round 0 (an item's first unit, a reference is missing): it is set.  1: the
    // weights.  2: they are taken back, the reference rises.  3: again.
#pragma unroll 1
    for (int round = unset ? 0 : 1;; ++round) {
      asm volatile("" : "+r"(round));  // one copy of the code: what misses the instruction cache costs most here
      uint32_t top = 0;  // the largest weight, as f16 pairs
      if (round != 0) {
        const uint64_t in2 = f2_pack(add, add), lr2 = f2_pack(lr, lr);
#pragma unroll
        for (int q = 0; q < NC; q += 8) {
          if (q == 16 && nc == 16) break;
          uint32_t s[8];
          tmem_ldn(tS + q, s);
          uint32_t p[4];
#pragma unroll
          for (int k = 0; k < 8; k += 4) {
            const float4 n = *reinterpret_cast<const float4*>(nref + q + k);
            float x[4];
            f2_unpack(f2_fma(f2_pack(__uint_as_float(s[k]), __uint_as_float(s[k + 1])), rk2, f2_add(lr2, f2_pack(n.x, n.y))), x[0],
                      x[1]);
            f2_unpack(f2_fma(f2_pack(__uint_as_float(s[k + 2]), __uint_as_float(s[k + 3])), rk2, f2_add(lr2, f2_pack(n.z, n.w))),
                      x[2], x[3]);
#pragma unroll
            for (int h = 0; h < 4; ++h) x[h] = exp2_sfu(x[h]);
            f2_unpack(f2_fma(f2_pack(x[0], x[1]), in2, f2_pack(l[q + k], l[q + k + 1])), l[q + k], l[q + k + 1]);
            f2_unpack(f2_fma(f2_pack(x[2], x[3]), in2, f2_pack(l[q + k + 2], l[q + k + 3])), l[q + k + 2], l[q + k + 3]);
            p[k / 2] = pack_f16(x[0], x[1]);
            p[k / 2 + 1] = pack_f16(x[2], x[3]);
          }
          top = hmax2(top, hmax2(hmax2(p[0], p[1]), hmax2(p[2], p[3])));
          const int to = (col0 + q) >> 3;  // piece of eight rows
          *reinterpret_cast<uint4*>(at + (to >> 3) * HALF_TILE + (((to ^ tid) & 7) << 4)) = make_uint4(p[0], p[1], p[2], p[3]);
        }
      }
      if (round == 3) {
        if (!lost) break;
        keep_branch();
        // 2^t / rs_v = 2^(s - r), where 2^t was nothing.  (Rolled, l turning by eight
        // columns: little code, and nothing spilled.)
#pragma unroll 1
        for (int q = 0; q < NC; q += 8) {
          uint32_t s[8];
          tmem_ldn(tS + q, s);
          float next[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float n = nref[q + k], z = __uint_as_float(s[k]);  // the weight to the bit as above
            next[k] = l[k] + (there && exp2_sfu(fmaf(z, rk, lr + n)) == 0.f ? exp2_sfu(fmaf(z, rk, n)) : 0.f);
          }
#pragma unroll
          for (int k = 0; k < NC - 8; ++k) l[k] = l[k + 8];
#pragma unroll
          for (int k = 0; k < 8; ++k) l[NC - 8 + k] = next[k];
        }
        break;
      }
      // (as numbers: f16 of one sign are ordered as their bits)
      if (round == 1 && !group_any(id, !ok || odd || large || max(top & 0xFFFFu, top >> 16) > TR_RAISE_F16)) break;
      keep_branch();
      if (round < 2 && group_any(id, !ok)) return false;
      if (round == 1) {
        add = -inv;
        // A sum that passed fp32 cannot be taken back: it is marked.
#pragma unroll
        for (int c = 0; c < NC; ++c) l[c] = l[c] == INFINITY ? -INFINITY : l[c];
        continue;
      }
      // l is what it was, to a rounding of what this unit adds.  Where that passed
      // fp32, 2^t / rs_v >= 2^128, the old l is dropped: a unit left it 2^10 / 2^-90 at
      // most, 2^-28 of what this one leaves once r has risen by t or more.  Elsewhere
      // it falls by 2^-rise in two steps: values much smaller than the ones that raise
      // r make it so large that one step would leave nothing.  NaN stays NaN.
      const float size = reinterpret_cast<const float2*>(smem + OFF_KEY + (it & 3) * 1024)[tid].y;
      if (size > 0.f) {
        large = true;  // the reference may be its value's from now on
        lr = size;
        inv = exp2_sfu(-lr);
      }
      const float m = row_max();
      const bool first = mine_unset && m > -INFINITY;
      const float rise = first || (!mine_unset && m > TR_RAISE) ? m : 0.f;  // whatever the other rows do
      if (tid < nc) {
        red[tid] = first ? 1.f : exp2_sfu(-0.5f * rise);
        nref[tid] -= rise;
      }
      if (u > u0) {  // O holds something
        const uint32_t p = it - 1;
        ok = tree_wait(&bar->o_done[p & 1], (p >> 1) & 1);
        ok = __all_sync(0xffffffffu, ok);
        tc_fence_after();
      }
      group_any(id, false);
#pragma unroll
      for (int c = 0; c < NC; ++c)
        if (c < nc) l[c] = max_nan(l[c], 0.f) * red[c] * red[c];
      if (u > u0 && ok) {
#pragma unroll 1
        for (int q = 0; q < nc; q += 8) {
          uint32_t o[8];
          tmem_ldn(tO + q, o);
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * red[q + i] * red[q + i]);
          tmem_st8(tO + q, o);
        }
        tmem_st_wait();
      }
      if (first) mine_unset = false;
      unset = group_any(id, mine_unset);  // (red is read)
      add = inv;
      if (round == 0) round = 2;  // nothing passes its bound now
    }
    tc_fence_before();
    fence_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive_n(&bar->p_full[buf], arrive);
  }

  // ---- the end: l over the keys, O out of TMEM
  const uint32_t p = it - 1;
  ok = ok && tree_wait(&bar->o_done[p & 1], (p >> 1) & 1);
  ok = __all_sync(0xffffffffu, ok);
  if (group_any(id, !ok)) return false;
  // The sums meet in shared memory (a place of P': no score of the next item is
  // issued, so no weight written, before all sixteen warps have arrived there, with
  // rows or without): thread t's, 16 bytes at piece c / 4 ^ (t & 7).
  float* box = reinterpret_cast<float*>(smem + OFF_P + wg * HALF_TILE);
#pragma unroll
  for (int c = 0; c < NC; c += 4)
    if (c < nc)
      *reinterpret_cast<float4*>(box + tid * 32 + (((c >> 2) ^ (tid & 7)) << 2)) = make_float4(l[c], l[c + 1], l[c + 2], l[c + 3]);
  group_any(id, false);
  {
    float sum = 0.f;
    if (lane < nc)
#pragma unroll 8
      for (int t = warp * 32; t < warp * 32 + 32; ++t) sum += box[t * 32 + (((lane >> 2) ^ (t & 7)) << 2) + (lane & 3)];
    red[tid] = sum;
  }
  group_any(id, false);
  const bool alone = u0 == 0 && u1 == w.units;
  const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (u0 > 0 ? 0 : 1);
  int64_t* to = reinterpret_cast<int64_t*>(red + 128);  // where each row goes
  if (tid < nc) {
    const float total = (red[tid] + red[32 + tid]) + (red[64 + tid] + red[96 + tid]);
    const int c = col0 + tid, row = row0 + c, node = row / group, head = w.kvh * group + row - node * group;
    red[tid] = total > 0.f ? 1.f / total : (total == 0.f ? 0.f : total);  // NaN stays NaN
    to[tid] = alone ? (static_cast<int64_t>(w.q0) + node) * a.n_q + head : slot * a.part_rows + c;
    if (c < w.rows) {
      const float r = -nref[tid];
      if (alone)
        a.lse[to[tid]] = total == 0.f ? -INFINITY : r * 0.69314718056f + logf(total);
      else
        a.part_lse[to[tid]] = total == 0.f ? -INFINITY : r + log2f(total);
    }
  }
  group_any(id, false);
  tc_fence_after();
#pragma unroll 1
  for (int c0 = 0; c0 < nc && col0 + c0 < w.rows; c0 += 8) {
    uint32_t o[8];
    tmem_ldn(tmem + lanes + COL_O + col0 + c0, o);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (col0 + c0 + i >= w.rows) break;
      const float x = __uint_as_float(o[i]) * red[c0 + i];
      if (alone)
        a.O[to[c0 + i] * 128 + tid] = __float2bfloat16(x);
      else
        a.part[to[c0 + i] * 128 + tid] = x;
    }
  }
  tc_fence_before();
  __syncwarp();
  if (lane == 0) mbar_arrive(&bar->o_empty);
  group_any(id, false);  // red is read
  return true;
}

__global__ void __launch_bounds__(TR_THREADS, 1)
    attn_tree_kernel(const __grid_constant__ CUtensorMap codes, const __grid_constant__ CUtensorMap sf,
                     const __grid_constant__ CUtensorMap scale, const TreeArgs a) {
  uint8_t* smem = tree_shared();
  TreeBars* bar = reinterpret_cast<TreeBars*>(smem + OFF_BAR);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int s = 0; s < TR_STAGES; ++s) {
      mbar_init(&bar->raw_full[s], 1);
      mbar_init(&bar->raw_empty[s], 8);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&bar->k_full[s], 4);
      mbar_init(&bar->s_full[s], 2);  // the products, and who issued them having seen the keys' scales
      mbar_init(&bar->p_full[s], TR_GROUPS * 4 + 4);  // weights and values
      mbar_init(&bar->o_done[s], 1);
    }
    mbar_init(&bar->q_full, TR_GROUPS * 4);
    mbar_init(&bar->o_empty, TR_GROUPS * 4);
    for (int i = 0; i < TR_ITEMS; ++i) mbar_init(&bar->item_full[i], 1);
    mbar_init(&bar->drain, 1);
    bar->seq = a.B;
    bar->before = 0;
    fence_mbar_init();
  }
  if (warp == TR_MMA_WARP) {
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
#pragma unroll 1
  for (int b = b0; b < b1; ++b) mine += tree_seq(a, b, blockIdx.x == 0).place_kv * a.c.n_kv;
  int64_t incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t n = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += n;
  }
  if (lane == 31) bar->scan[warp] = incl;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = bar->tmem;
  int64_t total = 0;
#pragma unroll
  for (int w = 0; w < TR_THREADS / 32; ++w) {
    if (w < warp) incl += bar->scan[w];
    total += bar->scan[w];
  }
  const int64_t per = max(static_cast<int64_t>(1), (total + gridDim.x - 1) / gridDim.x);
  const int64_t first = blockIdx.x * per, last = min(total, first + per);
  {
    int64_t before = incl - mine;
#pragma unroll 1
    for (int b = b0; b < b1; ++b) {
      const int64_t n = tree_seq(a, b, false).place_kv * a.c.n_kv;
      if (blockIdx.x == 0) a.places[b] = before;
      if (first >= before && first < before + n) {
        bar->seq = b;
        bar->before = before;
      }
      before += n;
    }
    if (blockIdx.x == 0 && tid == 0) {
      a.places[a.B] = total;
      a.places[a.B + 1] = per;
    }
  }
  __syncthreads();

  bool ok = true;
  if (first < last) {
    if (tid == TR_COPY_WARP * 32) {
      // to the item that holds `first`
      TreeCopies c;
      TreeWalk& w = c.w;
      w.b = bar->seq;
      w.base = bar->before;
      w.first = first;
      w.last = last;
      w.s = tree_seq(a, w.b, false);
      const int64_t each = w.s.units + TR_END, item = (first - w.base) / each;
      w.item = static_cast<int>(item);
      w.base += item * each;
      w.u0 = w.u1 = 0;
      c.u = 0;
      c.it = c.items = 0;
      c.done = 0;
      bar->copies = c;
    }
    __syncwarp();
    // Registers: 896 threads x 72 at launch = 512 x 88 + 128 x 56 + 128 x 48 + 128 x 48
    if (warp < TR_KEYS) {
      reg_inc<88>();
      uint32_t it = 0;
      bool behind = false;
      for (uint32_t item = 0; ok; ++item) {
        ok = tree_wait(&bar->item_full[item % TR_ITEMS], (item / TR_ITEMS) & 1);
        ok = !group_any(1 + (warp >> 2), !ok);
        const TreeItem& w = bar->item[item % TR_ITEMS];
        if (!ok || w.rows == 0) break;
        const bool idle = warp >= 4 * tree_groups(w.rows);  // few rows: the other warpgroups have them
        // The item before is done: its products have read Q, every warpgroup has
        // read what its end left in P', and one that has no rows is at most one item
        // away from the others.
        if (item > 0 && (idle || behind)) ok = tree_wait(&bar->o_empty, (item - 1) & 1);
        ok = !group_any(1 + (warp >> 2), !ok);
        if (!ok) break;
        behind = idle;
        if (idle) {
          it += w.u1 - w.u0;
          if (lane == 0) {
            mbar_arrive(&bar->q_full);
            mbar_arrive(&bar->o_empty);
          }
          continue;
        }
        ok = tree_softmax(a, smem, bar, tmem, item, it);
      }
    } else if (warp < TR_VALUES) {
      reg_dec<56>();
      bool more = true;
      const int shift = min(a.c.page_shift, 7), krow = raw_row((warp - TR_KEYS) * 32 + lane, shift);
      for (uint32_t it = 0; ok && more; ++it)
        ok = unpack_keys(smem, bar, tmem, warp - TR_KEYS, lane, it, shift, krow, more);
    } else if (warp < TR_COPY_WARP) {
      reg_dec<48>();
      bool more = true;
      const int shift = min(a.c.page_shift, 7);
      const ValueLane x(warp - TR_VALUES, lane, shift);
      for (uint32_t it = 0; ok && more; ++it) ok = unpack_values(smem, bar, warp - TR_VALUES, lane, it, shift, x, more);
    } else {
      reg_dec<48>();
      if (warp == TR_COPY_WARP) {
        int page = -1;  // of the lane's part of the next unit
        const uint32_t el = elect_one();
        while (ok && !bar->copies.done) ok = copy_unit(a, &codes, &sf, &scale, smem, bar, lane, el, page);
      } else if (warp == TR_MMA_WARP) {
        const uint32_t el = elect_one();
        uint32_t it = 0;
        for (uint32_t item = 0; ok; ++item) {
          ok = tree_wait(&bar->item_full[item % TR_ITEMS], (item / TR_ITEMS) & 1);
          ok = __all_sync(0xffffffffu, ok);
          const TreeItem& w = bar->item[item % TR_ITEMS];
          const int rows = w.rows, n = w.u1 - w.u0;
          if (!ok || rows == 0) break;
          const int ns = tree_groups(rows) * tree_columns(rows);
          const uint32_t id_s = idesc_f16(128, ns, 0, 0), id_o = idesc_f16(128, (ns + 63) & ~63, 1, 1);
          auto scores = [&](uint32_t i) {
            return i & 1 ? issue_scores<1>(smem, bar, tmem, i, id_s, el)
                         : issue_scores<0>(smem, bar, tmem, i, id_s, el);
          };
          auto outputs = [&](uint32_t i, bool head) {
            return i & 1 ? issue_outputs<1>(smem, bar, tmem, i, id_o, head, item, el)
                         : issue_outputs<0>(smem, bar, tmem, i, id_o, head, item, el);
          };
          ok = tree_wait(&bar->q_full, item & 1);
          ok = __all_sync(0xffffffffu, ok) && scores(it);
          for (int j = 0; j < n && ok; ++j, ++it) {
            if (j + 1 < n) ok = scores(it + 1);
            ok = ok && outputs(it, j == 0);
          }
        }
      }
    }
    if (!ok) {
      if (lane == 0) atomicOr(a.status, CODA_DEV_TIMEOUT);
      tree_drain(bar, warp, lane);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == TR_MMA_WARP) {
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
  const int64_t per = a.places[a.B + 1];
  const int64_t u0 = a.places[b] + kvh * s.place_kv + tile * static_cast<int64_t>(s.units + TR_END) + TR_END;
  const int c0 = static_cast<int>(u0 / per), c1 = static_cast<int>((u0 + s.units - 1) / per);
  if (c0 == c1) return;  // that CTA wrote the output
  // The weights a lane each, then the parts in order with four loads in flight:
  // two long documents (up to 76 parts a row) 138 -> 134 us, a chain of 6 over 777
  // keys 21 -> 19, 8 trees of 64 nodes 189 -> 190.
  auto part_of = [&](int x) { return (2ll * x + (x == c0 ? 1 : 0)) * a.part_rows + c; };
  float W = -INFINITY;
  for (int x = c0 + lane; x <= c1; x += 32) W = fmaxf(W, a.part_lse[part_of(x)]);
#pragma unroll
  for (int o = 16; o; o >>= 1) W = fmaxf(W, __shfl_xor_sync(0xffffffffu, W, o));
  const float W0 = W == -INFINITY ? 0.f : W;
  float acc[4] = {0.f, 0.f, 0.f, 0.f}, sum = 0.f;
  for (int x0 = c0; x0 <= c1; x0 += 32) {
    const int n = min(32, c1 - x0 + 1);
    // halves of the exponent: a large value counts at a probability below 2^-126 too
    const float mine = lane < n ? exp2_sfu(0.5f * (a.part_lse[part_of(x0 + lane)] - W0)) : 0.f;
#pragma unroll 4
    for (int i = 0; i < n; ++i) {
      const float wgt = __shfl_sync(0xffffffffu, mine, i);
      const float4 v = *reinterpret_cast<const float4*>(a.part + part_of(x0 + i) * 128 + lane * 4);
      sum += wgt * wgt;
      acc[0] += wgt * v.x * wgt;
      acc[1] += wgt * v.y * wgt;
      acc[2] += wgt * v.z * wgt;
      acc[3] += wgt * v.w * wgt;
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  *out = make_uint2(pack_bf16x2(acc[0] * inv, acc[1] * inv), pack_bf16x2(acc[2] * inv, acc[3] * inv));
  if (lane == 0) a.lse[at] = sum == 0.f ? -INFINITY : W * 0.69314718056f + logf(sum);
}

}  // namespace

bool cache_maps(CUtensorMap* m, const KvCache& c) {
  const uint64_t page = uint64_t(1) << c.page_shift, kv = c.n_kv, pages = c.num_pages;
  const uint32_t part = static_cast<uint32_t>(std::min<uint64_t>(page, TR_UNIT));
  {
    const uint64_t dims[5] = {64, page, kv, 2, pages}, st[4] = {64, page * 64, kv * page * 64, 2 * kv * page * 64};
    const uint32_t box[5] = {64, part, 1, 2, 1};
    if (!encode_cache_map(&m[0], c.codes, 1, 5, dims, st, box, true)) return false;
  }
  for (int i = 1; i < 3; ++i) {  // words of a page's rows: two of block scales each, one row scale
    const uint64_t row = page * (i == 1 ? 2 : 1);
    const uint64_t dims[4] = {row, kv, 2, pages}, st[3] = {row * 4, kv * row * 4, 2 * kv * row * 4};
    const uint32_t box[4] = {part * (i == 1 ? 2 : 1), 1, 2, 1};
    if (!encode_cache_map(&m[i], i == 1 ? static_cast<const void*>(c.sf) : c.scale, 4, 4, dims, st, box, false)) return false;
  }
  return true;
}

cudaError_t launch_attn_tree(const TreeArgs& a, const CUtensorMap* maps, int sms, cudaStream_t s) {
  cudaError_t e = attn_smem_attribute(reinterpret_cast<const void*>(attn_tree_kernel), 7, TR_SMEM);
  if (e != cudaSuccess) return e;
  e = attn_launch(attn_tree_kernel, std::min(sms, TREE_MAX_CTAS), TR_THREADS, TR_SMEM, s, maps[0], maps[1], maps[2],
                  a);
  if (e != cudaSuccess) return e;
  return attn_launch(attn_tree_join_kernel, (static_cast<int64_t>(a.T) * a.n_q + 7) / 8, 256, 0, s, a);
}

}  // namespace coda

// The 4-bit key/value cache (NVFP4 rows): append, read back, and attention of
// one new token per sequence over it.
#include <algorithm>

#include "coda_attn.cuh"
#include "coda_internal.h"
#include "coda_kvrow.cuh"
#include "coda_status.h"

namespace coda {
namespace {

// ------------------------------------------------------------------ append
// Eight lanes per row of 128, one 16-element block each (quantise_row16).  HBM-bound: 512 bytes in and
// 152 out per token and head, 11.6 us for 8192 tokens and 8 heads (44 MB; 12.3
// with the 36 registers that six blocks per SM leave).
// One row per lane group, many blocks: with four rows per group in flight
// instead it took 21.5 us (6.6 instead of 3.7 us for 61 tokens).
__global__ void __launch_bounds__(256, 8)
    kv_append_kernel(const KvCache c, const __nv_bfloat16* __restrict__ K, int64_t ldk,
                     const __nv_bfloat16* __restrict__ V, int64_t ldv, const int32_t* __restrict__ slots, int rows,
                     int* status) {
  griddep_wait();
  griddep_launch_dependents();
  const int sub = threadIdx.x & 7;
  const int row = blockIdx.x * 32 + (threadIdx.x >> 3);
  float x[16];
  int64_t at = -1;  // cache row, -1: none
  if (row < rows) {
    const int t = row / (2 * c.n_kv), rest = row - t * 2 * c.n_kv;
    const int plane = rest >= c.n_kv, h = rest - plane * c.n_kv;
    const __nv_bfloat16* src = (plane ? V + t * ldv : K + t * ldk) + h * 128 + sub * 16;
    load_bf16x8(src, x);
    load_bf16x8(src + 8, x + 8);
    const int slot = slots[t];
    if (slot >= 0) {
      if ((slot >> c.page_shift) < c.num_pages)
        at = cache_row(c, slot >> c.page_shift, plane, h, slot & ((1 << c.page_shift) - 1));
      else if (rest == 0 && sub == 0)
        atomicOr(status, CODA_DEV_PAGE_RANGE);
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

// -------------------------------------------------------------------- read
// The rows back: (e2m1 * e4m3, exact in f16) * scale, one fp32 rounding; then
// bf16 for the bf16 form.  Sixteen lanes per row, eight elements each; in fp32
// four of each half, so that every store of a warp covers whole lines.  Bound by
// the writes and the start: 67 MB in fp32 for 8192 tokens and 8 heads, 15.8 us
// (22.3 with 32 lanes per row and the products in fp32, where the instructions
// were the limit; two and four rows per lane group in turn 15.8 and 16.4, and
// 4.4 and 6.0 instead of 3.7 us for 61 tokens).  In bf16, 34 MB: 12.4 us against
// 14.4 in fp32, both back to back.
template <bool F32>
__global__ void __launch_bounds__(256)
    kv_read_kernel(const KvCache c, const int32_t* __restrict__ slots, int rows, void* __restrict__ K,
                   void* __restrict__ V, int* status) {
  griddep_wait();
  griddep_launch_dependents();
  const int sub = threadIdx.x & 15;
  const int row = blockIdx.x * 16 + (threadIdx.x >> 4);
  if (row >= rows) return;
  const int t = row / (2 * c.n_kv), rest = row - t * 2 * c.n_kv;
  const int plane = rest >= c.n_kv, h = rest - plane * c.n_kv;
  const int slot = slots[t];
  uint32_t codes = 0, sfs = 0;
  float sc = 0.f;
  if (slot >= 0) {
    if ((slot >> c.page_shift) < c.num_pages) {
      const int64_t r = cache_row(c, slot >> c.page_shift, plane, h, slot & ((1 << c.page_shift) - 1));
      const uint8_t* q = c.codes + r * 64;
      const uint8_t* f = c.sf + r * 8;
      if constexpr (F32) {
        codes = *reinterpret_cast<const uint16_t*>(q + sub * 2) |
                static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(q + 32 + sub * 2)) << 16;
        sfs = f[sub >> 2] | static_cast<uint32_t>(f[4 + (sub >> 2)]) << 8;
      } else {
        codes = *reinterpret_cast<const uint32_t*>(q + sub * 4);
        sfs = f[sub >> 1] * 0x101u;
      }
      sc = c.scale[r];
    } else if (rest == 0 && sub == 0) {
      atomicOr(status, CODA_DEV_PAGE_RANGE);
    }
  }
  const uint32_t sf = e4m3x2_f16(sfs);
  uint32_t f[4];
  e2m1x8_f16(codes, f);
  float v[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t x = hmul2(f[i], __byte_perm(sf, sf, i < 2 ? 0x1010 : 0x3232));
    v[2 * i] = __fmul_rn(f16_lo(x), sc);
    v[2 * i + 1] = __fmul_rn(f16_hi(x), sc);
  }
  const int64_t at = (static_cast<int64_t>(t) * c.n_kv + h) * 128;
  if constexpr (F32) {
    float4* dst = reinterpret_cast<float4*>(static_cast<float*>(plane ? V : K) + at) + sub;
    dst[0] = make_float4(v[0], v[1], v[2], v[3]);
    dst[16] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    store_bf16x8(static_cast<__nv_bfloat16*>(plane ? V : K) + at + sub * 8, v);
  }
}

// ------------------------------------------------------------------ accept
// The rows of a tree's accepted nodes move to the places behind the prefix, in
// the order of the path: place d takes node path[d] >= d.  A warp per sequence,
// plane and head, four lanes per row; eight rows are read, then written, and
// the rows of later steps lie behind every place written so far.
__global__ void __launch_bounds__(256) kv_accept_kernel(const AcceptArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const KvCache& c = a.c;
  const int w = static_cast<int>(blockIdx.x) * 8 + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int b = w / (2 * c.n_kv), rest = w - b * 2 * c.n_kv;
  if (b >= a.B) return;
  const int plane = rest >= c.n_kv, h = rest - plane * c.n_kv;
  const bool tell = rest == 0 && lane == 0;
  const int q0 = a.cu[b], q1 = a.cu[b + 1], len = a.seq_lens[b];
  const int n = q1 - q0;
  if (q0 < 0 || n < 0 || len < n || len > (static_cast<int64_t>(a.max_pages) << c.page_shift)) {
    if (tell) {
      atomicOr(a.status, CODA_DEV_SEQLEN_RANGE);
      a.out_lens[b] = 0;
    }
    return;
  }
  int count = n > 0 ? a.count[b] : 0;
  const int32_t* path = a.nodes + static_cast<int64_t>(b) * a.width;
  bool bad = count < 0 || (n > 0 && (count >= n || count >= a.width));
  // a path rises from node 0: then no row is overwritten before it is read
  for (int d = lane; !bad && d <= count && n > 0; d += 32) {
    const int at = path[d];
    bad = at >= n || (d == 0 ? at != 0 : at <= path[d - 1]);
  }
  if (__any_sync(0xffffffffu, bad)) {
    if (tell) {
      atomicOr(a.status, CODA_DEV_TREE_RANGE);
      a.out_lens[b] = len - n;
    }
    return;
  }
  if (tell) a.out_lens[b] = n > 0 ? len - n + count + 1 : len;
  const int32_t* table = a.table + static_cast<int64_t>(b) * a.max_pages;
  const int part = lane & 3;
  auto row_of = [&](int node) {
    const int k = len - n + node, page = table[k >> c.page_shift];
    if (page < 0 || page >= c.num_pages) {
      if (rest == 0 && part == 0) atomicOr(a.status, CODA_DEV_PAGE_RANGE);
      return static_cast<int64_t>(-1);
    }
    return cache_row(c, page, plane, h, k & ((1 << c.page_shift) - 1));
  };
  for (int d0 = 1; d0 <= count; d0 += 8) {
    const int d = d0 + (lane >> 2);
    int64_t to = -1;
    uint4 codes = make_uint4(0, 0, 0, 0);
    uint16_t sf = 0;
    float scale = 0.f;
    if (d <= count) {
      const int node = path[d];
      const int64_t from = node != d ? row_of(node) : -1;
      to = from >= 0 ? row_of(d) : -1;
      if (to >= 0) {
        codes = reinterpret_cast<const uint4*>(c.codes + from * 64)[part];
        sf = reinterpret_cast<const uint16_t*>(c.sf + from * 8)[part];
        if (part == 0) scale = c.scale[from];
      }
    }
    __syncwarp();
    if (to >= 0) {
      reinterpret_cast<uint4*>(c.codes + to * 64)[part] = codes;
      reinterpret_cast<uint16_t*>(c.sf + to * 8)[part] = sf;
      if (part == 0) c.scale[to] = scale;
    }
    __syncwarp();
  }
}

// ------------------------------------------------------------------ decode
// One query token per sequence over its cached keys and values:
//   s_j = scale q . k_j,  O = sum_j exp(s_j - lse) v_j,
// HBM-bound: 152 bytes per cached token and key/value head feed 2 * 128
// multiply-adds (4 * 128 operations) per query head.  The cost beside the bytes
// is unpacking: 256 codes per token and head.
//
// Work: every (sequence, key/value head) is cut into units of 128 keys; the
// units of the whole batch form one line that the CTAs divide evenly, so a
// batch of mixed lengths, or one long sequence, keeps every SM busy.  Each
// (sequence, head) has DEC_END places more on that line than it has units,
// for the work at its end.  A CTA whose stretch covers a whole (sequence,
// head) writes the output itself; the others leave normalised partial outputs, merged by a second kernel.
//
// A fifth warp copies units into a shared-memory ring by bulk copies (one per
// page and array), ahead of the four that compute and across the ends of
// stretches; each of the four takes 32 keys of a unit.  Products are m16n8k16
// on f16:
//   S^T [16 keys x 8 heads] = K Q^T:  e2m1 * e4m3 has at most 6 significant
//     bits, so K' = code * sf is exact in f16; the row scale multiplies S.
//     A lane's 16 bytes of a key row are 32 neighbouring elements, two blocks
//     with one scale each: the k index of the product is a permutation of
//     the head's elements, the same for Q.
//   O^T [16 elements x 8 heads] += V'^T P'^T with the row scale of V in
//     P' = exp2(z - m) * rs * f, where f (per head) sets the largest P' of a row
//     that is not all zeros to 1 and is renewed before one would pass 2^14 (f16
//     ends at 2^16): P' is rounded to f16 (2^-11, or 2^-25 of that largest one),
//     O accumulates in fp32.
// The keys of a tile are read in the order 0 4 1 5 2 6 3 7: then the lanes'
// shared-memory reads of both K and V are contiguous, and movmatrix turns
// the S^T fragment into the P operand.
//
// Measured: 127 sequences of 1 to 8192 keys, 64 + 8 heads (616 MB) 132 us, 4.6
// TB/s; four of 98304 to 131072 keys, 32 + 8 heads (560 MB) 115 us, 4.9 TB/s.
// The first with 32 heads for each of 4 key/value heads (two passes of 16) 213 us,
// with 16 heads 115 (cold).
// Without any arithmetic an earlier form's copies and stretch ends took 119 and
// 94 us, so these come first (with pages of 64 a unit is 12 bulk copies, eight of
// them of 512 or 256 bytes; which of the two it is was not measured apart); the
// unpacking (309 instructions per 16 keys and warp) fills 55 % of the issue slots
// beside them.
constexpr int DEC_WARPS = 4;  // computing warps
constexpr int DEC_THREADS = (DEC_WARPS + 1) * 32;
constexpr int DEC_STAGES = 3;
constexpr int DEC_UNIT = 128;
constexpr int ST_K = 0, ST_V = 8192, ST_SFK = 16384, ST_SFV = 17408, ST_RSK = 18432, ST_RSV = 18944;
constexpr int DEC_STAGE_BYTES = 19456;
// ring, merge buffer (two warps' fragments), barriers and page masks
constexpr uint32_t dec_smem_bytes(int nt) { return DEC_STAGES * DEC_STAGE_BYTES + 2 * nt * (4096 + 256) + 128; }

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t movmatrix_t(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// Length of sequence b; 0 (and the status bit, if `tell`) when it is negative
// or longer than its page table.
__device__ __forceinline__ int decode_len(const DecodeArgs& a, int b, bool tell) {
  const int n = a.seq_lens[b];
  if (n < 0 || n > (static_cast<int64_t>(a.max_pages) << a.c.page_shift)) {
    if (tell) atomicOr(a.status, CODA_DEV_SEQLEN_RANGE);
    return 0;
  }
  return n;
}

// Measured with 64 + 8 heads, 0 against 1, 2 and 3 places: 128 sequences of 1 to
// 8192 keys 153, 137, 132 and 131 us; 512 of 512 keys with 64 of 4096 167, 164,
// 158 and 166 us; 128 of 4096 keys 132, 135, 134 and 134 us.
constexpr int DEC_END = 2;

// Places on the line of units that each head of a sequence of `len` keys takes.
__device__ __forceinline__ int decode_places(int len) { return len > 0 ? (len + DEC_UNIT - 1) / DEC_UNIT + DEC_END : 0; }

// A CTA's way along the line: stretches of one (sequence, virtual head).
// Every warp walks it for itself.
struct Stretch {
  int b, before;        // sequence, places before it
  int u;                // next place of the line
  // current stretch
  int first, nu, stop;  // the place of its first unit, its units, where this CTA stops in it
  int vh, len;
  // false: no unit before `last`
  __device__ __forceinline__ bool next(const DecodeArgs& a, int vheads, int last) {
    if (u >= last) return false;
    len = decode_len(a, b, false);
    int places = decode_places(len);
    while (u >= before + places * vheads) {
      before += places * vheads;
      len = decode_len(a, ++b, false);
      places = decode_places(len);
    }
    vh = (u - before) / places;
    nu = places - DEC_END;
    first = before + vh * places + DEC_END;  // the places in front stand for its end
    u = max(u, first);
    stop = min(last, first + nu);
    return u < last;
  }
};

template <int NT>
__global__ void __launch_bounds__(DEC_THREADS, NT == 1 ? 3 : 2) attn_decode_kernel(const DecodeArgs a) {
  extern __shared__ __align__(128) uint8_t dec_smem[];
  __shared__ int sh_warp[DEC_WARPS + 1], sh_seq, sh_before;
  float* merge = reinterpret_cast<float*>(dec_smem + DEC_STAGES * DEC_STAGE_BYTES);
  uint64_t* full = reinterpret_cast<uint64_t*>(dec_smem + DEC_STAGES * DEC_STAGE_BYTES + 2 * NT * (4096 + 256));
  uint64_t* empty = full + DEC_STAGES;
  uint32_t* pages_in = reinterpret_cast<uint32_t*>(empty + DEC_STAGES);  // per stage: bit i = keys 16 i .. 16 i + 15 are there
  volatile int* abort_flag = reinterpret_cast<volatile int*>(pages_in + DEC_STAGES);
  static_assert(2 * DEC_STAGES * 8 + DEC_STAGES * 4 + 4 <= 128, "barrier area");
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, c = lane & 3;
  const int vheads = a.c.n_kv * a.splits;
  if (tid == 0) {
    for (int s = 0; s < DEC_STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], DEC_WARPS);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  griddep_wait();
  griddep_launch_dependents();

  // places before each sequence: a contiguous run of sequences per thread,
  // scanned over the block
  const int chunk = (a.B + DEC_THREADS - 1) / DEC_THREADS;
  const int s0 = min(a.B, tid * chunk), s1 = min(a.B, s0 + chunk);
  int mine = 0;
  for (int b = s0; b < s1; ++b) mine += decode_places(decode_len(a, b, blockIdx.x == 0)) * vheads;
  int incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int n = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += n;
  }
  if (lane == 31) sh_warp[warp] = incl;
  __syncthreads();
  int total = 0;
#pragma unroll
  for (int w = 0; w <= DEC_WARPS; ++w) {
    if (w < warp) incl += sh_warp[w];
    total += sh_warp[w];
  }
  const int per = max(1, (total + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x));
  const int first = static_cast<int>(blockIdx.x) * per, last = min(total, first + per);
  {
    int before = incl - mine;
    for (int b = s0; b < s1; ++b) {
      const int n = decode_places(decode_len(a, b, false)) * vheads;
      if (blockIdx.x == 0) a.units[b] = before;
      if (first >= before && first < before + n) {
        sh_seq = b;
        sh_before = before;
      }
      before += n;
    }
    if (blockIdx.x == 0 && tid == 0) {
      a.units[a.B] = total;
      a.units[a.B + 1] = per;
    }
  }
  __syncthreads();
  if (first >= last) return;

  Stretch x;
  x.b = sh_seq;
  x.before = sh_before;
  x.u = first;
  uint32_t it = 0;  // units so far: stage it % DEC_STAGES
  bool ok = true;

  if (warp == DEC_WARPS) {
    // ------------------------------------------------------------ copies
    // Lane i of each group of eight takes part i of a unit (a page, or 128
    // keys of one): group 0 the codes, 1 the block scales, 2 the row scales,
    // keys and values each.
    const KvCache& kc = a.c;
    const int part = lane & 7, arr = lane >> 3;
    const int part_shift = min(kc.page_shift, 7);
    const uint32_t row_bytes = arr == 0 ? 64 : arr == 1 ? 8 : 4;
    const uint32_t to_k = arr == 0 ? ST_K : arr == 1 ? ST_SFK : ST_RSK, to_v = arr == 0 ? ST_V : arr == 1 ? ST_SFV : ST_RSV;
    const uint8_t* src = arr == 0 ? kc.codes : arr == 1 ? kc.sf : reinterpret_cast<const uint8_t*>(kc.scale);
    const int64_t plane = static_cast<int64_t>(kc.n_kv) << kc.page_shift;
    while (ok && x.next(a, vheads, last)) {
      const int kvh = x.vh / a.splits;
      const int32_t* table = a.table + static_cast<int64_t>(x.b) * a.max_pages;
      auto page_of = [&](int u) {  // of this lane's part of unit u; -1: nothing there
        const int k = (u - x.first) * DEC_UNIT + (part << part_shift);
        return u < x.stop && (part << part_shift) < DEC_UNIT && k < x.len ? table[k >> kc.page_shift] : -1;
      };
      int page = page_of(x.u);
      for (; x.u < x.stop; ++x.u, ++it) {
        const int nextp = page_of(x.u + 1);
        const int k = (x.u - x.first) * DEC_UNIT + (part << part_shift);
        const bool named = (part << part_shift) < DEC_UNIT && k < x.len;
        const bool in = named && page >= 0 && page < kc.num_pages;
        if (named && !in && arr == 0) atomicOr(a.status, CODA_DEV_PAGE_RANGE);
        // whole groups of 16 keys: rows behind the length exist within the page
        const int n = in ? min(1 << part_shift, (x.len - k + 15) & ~15) : 0;
        const uint32_t bytes = arr < 3 ? n * row_bytes : 0;
        const uint32_t s = it % DEC_STAGES;
        ok = mbar_wait_bounded(&empty[s], ((it / DEC_STAGES) & 1) ^ 1, abort_flag, a.status, 2000000000ull, 100);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const uint32_t sum = __reduce_add_sync(0xffffffffu, 2 * bytes);
        const uint32_t mask = __reduce_or_sync(0xffffffffu, arr == 0 && n ? ((1u << (n / 16)) - 1) << (part << part_shift >> 4) : 0);
        if (lane == 0) {
          pages_in[s] = mask;
          if (sum == 0) mbar_arrive(&full[s]);
        }
        mbar_arrive_expect_tx(&full[s], sum, lane == 0 && sum != 0);
        __syncwarp();
        if (bytes) {
          const int64_t row = cache_row(kc, page, 0, kvh, k & ((1 << kc.page_shift) - 1));
          uint8_t* st = dec_smem + s * DEC_STAGE_BYTES + (part << part_shift) * row_bytes;
          bulk_load(st + to_k, src + row * row_bytes, bytes, &full[s], 1);
          bulk_load(st + to_v, src + (row + plane) * row_bytes, bytes, &full[s], 1);
        }
        page = nextp;
      }
    }
    if (!ok) {
      // let every copy already issued land before the CTA's memory is reused
      const uint64_t t0 = globaltimer_ns();
      while (globaltimer_ns() - t0 < 2000000ull) {
      }
    }
    return;
  }

  const int pi = (g >> 1) + (g & 1) * 4;  // key of fragment row g; row g + 8 is 8 keys on
  // this lane's places in a stage, of the warp's 32 keys
  const uint8_t* k_at = dec_smem + ST_K + (warp * 32 + pi) * 64 + c * 16;
  const uint8_t* sfk_at = dec_smem + ST_SFK + (warp * 32 + pi) * 8 + 2 * c;
  const uint8_t* rsk_at = dec_smem + ST_RSK + (warp * 32 + pi) * 4;
  const uint8_t* v_at = dec_smem + ST_V + (warp * 32 + c) * 64 + g * 8;
  const uint8_t* sfv_at = dec_smem + ST_SFV + (warp * 32 + c) * 8 + g;
  const uint8_t* rsv_at = dec_smem + ST_RSV + (warp * 32 + pi) * 4;
  while (x.next(a, vheads, last)) {
    const int u0 = x.u;
    const int kvh = x.vh / a.splits;
    const int head0 = kvh * a.group + (x.vh - kvh * a.splits) * DEC_HEADS;
    const int heads = min(DEC_HEADS, (kvh + 1) * a.group - head0);

    // Q of head g (+ 8 per n tile), elements 32c .. 32c + 31, scaled by a
    // power of two to a maximum in [1, 2) so that f16 holds it
    uint32_t q[NT][16];
    float hf[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float y[32];
      const int h = t * 8 + g;
      if (h < heads) {
        const __nv_bfloat16* src = a.Q + x.b * a.ldq + (head0 + h) * 128 + c * 32;
#pragma unroll
        for (int i = 0; i < 4; ++i) load_bf16x8(src + 8 * i, y + 8 * i);
      } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) y[i] = 0.f;
      }
      float mx = 0.f;
#pragma unroll
      for (int i = 0; i < 32; ++i) mx = fmaxf(mx, fabsf(y[i]));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      int e = static_cast<int>(__float_as_uint(mx) >> 23) - 127;
      e = mx == 0.f ? 0 : max(-126, min(126, e));
      const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
      for (int i = 0; i < 16; ++i) q[t][i] = pack_f16(y[2 * i] * down, y[2 * i + 1] * down);
      const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23) * a.scale_log2;
      hf[t][0] = __shfl_sync(0xffffffffu, up, (2 * c) * 4);
      hf[t][1] = __shfl_sync(0xffffffffu, up, (2 * c + 1) * 4);
    }

    float m[NT][2], l[NT][2], f[NT][2], o[NT][8][4];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        m[t][k] = 0.f;
        l[t][k] = 0.f;
        f[t][k] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[t][i][k] = 0.f;
    }
    bool fresh = true, unset = true;  // no key yet (m is a placeholder); a head without units of O (f = 0)

    for (; x.u < x.stop; ++x.u, ++it) {
      const uint32_t s = it % DEC_STAGES;
      ok = ok && mbar_wait_bounded(&full[s], (it / DEC_STAGES) & 1, abort_flag, a.status, 2000000000ull);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) {  // the status word tells; the warp still meets the others at the merges
        x.u = x.stop;
        break;
      }
      const uint32_t so = s * DEC_STAGE_BYTES;
      const uint32_t on = (pages_in[s] >> (2 * warp)) & 3u;
      const int left = x.len - (x.u - x.first) * DEC_UNIT - 32 * warp;  // of the warp's 32 keys
      if (left > 0 && on) {
        const bool whole = on == 3u && left >= 32;
        // S^T: z = s * scale * log2(e); the two groups of 16 keys side by side
        // (each a chain of eight dependent products)
        float z[NT][2][4];
        uint4 w0[2], w1[2];
        uint32_t f0[2], f1[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int k = 0; k < 4; ++k) z[t][h][k] = 0.f;
          w0[h] = *reinterpret_cast<const uint4*>(k_at + so + h * 1024);
          w1[h] = *reinterpret_cast<const uint4*>(k_at + so + h * 1024 + 512);
          f0[h] = e4m3x2_f16(*reinterpret_cast<const uint16_t*>(sfk_at + so + h * 128));
          f1[h] = e4m3x2_f16(*reinterpret_cast<const uint16_t*>(sfk_at + so + h * 128 + 64));
        }
#pragma unroll
        for (int k = 0; k < 8; k += 2) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t xa[4], ya[4];
            e2m1x8_f16(k == 0 ? w0[h].x : k == 2 ? w0[h].y : k == 4 ? w0[h].z : w0[h].w, xa);
            e2m1x8_f16(k == 0 ? w1[h].x : k == 2 ? w1[h].y : k == 4 ? w1[h].z : w1[h].w, ya);
            // both halves of the scale register: block 2c for the first 16 elements, 2c + 1 for the others
            const uint32_t g0 = __byte_perm(f0[h], f0[h], k < 4 ? 0x1010 : 0x3232);
            const uint32_t g1 = __byte_perm(f1[h], f1[h], k < 4 ? 0x1010 : 0x3232);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const uint32_t a0 = hmul2(xa[2 * i], g0), a1 = hmul2(ya[2 * i], g1);
              const uint32_t a2 = hmul2(xa[2 * i + 1], g0), a3 = hmul2(ya[2 * i + 1], g1);
#pragma unroll
              for (int t = 0; t < NT; ++t) mma_f16(z[t][h], a0, a1, a2, a3, q[t][2 * (k + i)], q[t][2 * (k + i) + 1]);
            }
          }
        }
        // z = s * scale * log2(e) - m, the exponent of the weight
        float rv[4], top[NT][2];
        bool up = false;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const float r0 = *reinterpret_cast<const float*>(rsk_at + so + h * 64);
          const float r1 = *reinterpret_cast<const float*>(rsk_at + so + h * 64 + 32);
          rv[2 * h] = *reinterpret_cast<const float*>(rsv_at + so + h * 64);
          rv[2 * h + 1] = *reinterpret_cast<const float*>(rsv_at + so + h * 64 + 32);
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int k = 0; k < 4; ++k) z[t][h][k] = fmaf(z[t][h][k] * (k < 2 ? r0 : r1), hf[t][k & 1], -m[t][k & 1]);
          if (!whole) {
            const bool in0 = ((on >> h) & 1) && 16 * h + pi < left, in1 = ((on >> h) & 1) && 16 * h + pi + 8 < left;
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
              for (int k = 0; k < 4; ++k) z[t][h][k] = (k < 2 ? in0 : in1) ? z[t][h][k] : -INFINITY;
            rv[2 * h] = in0 ? rv[2 * h] : 0.f;
            rv[2 * h + 1] = in1 ? rv[2 * h + 1] : 0.f;
          }
        }
        // raise m only when a weight passes 2^8: l and f have room, and rows that rise slowly rarely come here
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            top[t][k] = fmaxf(fmaxf(z[t][0][k], z[t][0][k + 2]), fmaxf(z[t][1][k], z[t][1][k + 2]));
            up |= top[t][k] > 8.f;
          }
        up |= fresh;
        if (__any_sync(0xffffffffu, up)) {
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              float y = top[t][k];
#pragma unroll
              for (int d = 4; d < 32; d <<= 1) y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, d));
              if ((fresh && y > -INFINITY) || y > 0.f) {
                l[t][k] = fresh ? 0.f : l[t][k] * exp2_sfu(-y);
                // O is in units of f * 2^m and keeps its value; where f ends (values
                // below about 1e-32), O takes the rest of the step
                float nf = f[t][k] == 0.f ? 0.f : f[t][k] * exp2_sfu(y);
                if (nf > 0x1p127f) {
                  const float by = exp2_sfu(127.f - __log2f(f[t][k]) - y);
                  nf = 0x1p127f;
#pragma unroll
                  for (int i = 0; i < 8; ++i) {
                    o[t][i][k] *= by;
                    o[t][i][k + 2] *= by;
                  }
                }
                f[t][k] = nf;
                m[t][k] += y;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  z[t][h][k] -= y;
                  z[t][h][k + 2] -= y;
                }
              }
            }
        }
        // the weights, times the row scales of V, in units of O
        float pf[NT][2][4], big = 0.f;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float e = exp2_sfu(z[t][h][k]);
              l[t][k & 1] += e;
              z[t][h][k] = e * rv[2 * h + (k >> 1)];
              pf[t][h][k] = z[t][h][k] * f[t][k & 1];
              big = fmaxf(big, pf[t][h][k]);
            }
        // new units when P' would pass 2^14, or a head has none yet
        if (__any_sync(0xffffffffu, unset || big > 16384.f)) {
          unset = false;
          // A row of zeros has the row scale 1 and adds nothing: it has no say
          // in the units (a row scale that is not finite keeps its own)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint2 b = *reinterpret_cast<const uint2*>(dec_smem + ST_SFV + (warp * 32 + pi) * 8 + so + i * 64);
            if (((b.x | b.y) & 0x7F7F7F7Fu) == 0) {
#pragma unroll
              for (int t = 0; t < NT; ++t) {
                z[t][i >> 1][2 * (i & 1)] *= 0.f;
                z[t][i >> 1][2 * (i & 1) + 1] *= 0.f;
              }
            }
          }
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              float y = fmaxf(fmaxf(z[t][0][k], z[t][0][k + 2]), fmaxf(z[t][1][k], z[t][1][k + 2]));
#pragma unroll
              for (int d = 4; d < 32; d <<= 1) y = fmaxf(y, __shfl_xor_sync(0xffffffffu, y, d));
              if (y * f[t][k] > 1.f || (f[t][k] == 0.f && y > 0.f)) {
                const float nf = fminf(1.f / y, 3e38f);
                const float by = f[t][k] == 0.f ? 0.f : nf / f[t][k];
                f[t][k] = nf;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                  o[t][i][k] *= by;
                  o[t][i][k + 2] *= by;
                }
              }
              unset |= f[t][k] == 0.f;
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                pf[t][h][k] = z[t][h][k] * f[t][k];
                pf[t][h][k + 2] = z[t][h][k + 2] * f[t][k];
              }
            }
        }
        fresh = false;
        // O^T += V'^T P'^T
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t p[NT][2];
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            p[t][0] = movmatrix_t(pack_f16(pf[t][h][0], pf[t][h][1]));
            p[t][1] = movmatrix_t(pack_f16(pf[t][h][2], pf[t][h][3]));
          }
          // keys c, c + 4, c + 8, c + 12; elements 16 g .. 16 g + 15: one block
          uint2 w[4];
          uint32_t sf[4];
#pragma unroll
          for (int y = 0; y < 4; ++y) {
            w[y] = *reinterpret_cast<const uint2*>(v_at + so + h * 1024 + y * 256);
            sf[y] = sfv_at[so + h * 128 + y * 32];
          }
          if (!whole) {
#pragma unroll
            for (int y = 0; y < 4; ++y)  // an unwritten row's scale may be NaN
              if (!(((on >> h) & 1) && 16 * h + c + 4 * y < left)) sf[y] = 0;
          }
          const uint32_t g0 = e4m3x2_f16(sf[0] | (sf[1] << 8)), g1 = e4m3x2_f16(sf[2] | (sf[3] << 8));
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const uint32_t x0 = half ? w[0].y : w[0].x, x1 = half ? w[1].y : w[1].x;
            const uint32_t x2 = half ? w[2].y : w[2].x, x3 = half ? w[3].y : w[3].x;
            // the same element of two keys in one byte: even elements, odd elements
            uint32_t e0[4], o0[4], e1[4], o1[4];
            e2m1x8_f16((x0 & 0x0F0F0F0Fu) | ((x1 << 4) & 0xF0F0F0F0u), e0);
            e2m1x8_f16(((x0 >> 4) & 0x0F0F0F0Fu) | (x1 & 0xF0F0F0F0u), o0);
            e2m1x8_f16((x2 & 0x0F0F0F0Fu) | ((x3 << 4) & 0xF0F0F0F0u), e1);
            e2m1x8_f16(((x2 >> 4) & 0x0F0F0F0Fu) | (x3 & 0xF0F0F0F0u), o1);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const uint32_t a0 = hmul2(e0[j], g0), a1 = hmul2(o0[j], g0), a2 = hmul2(e1[j], g1), a3 = hmul2(o1[j], g1);
#pragma unroll
              for (int t = 0; t < NT; ++t) mma_f16(o[t][half * 4 + j], a0, a1, a2, a3, p[t][0], p[t][1]);
            }
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[s]);
    }

    // merge the four warps, pairs first: the fragments lie alike, so a lane
    // adds what the same lane of the other warp left
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[t][k] += __shfl_xor_sync(0xffffffffu, l[t][k], d);
        if (l[t][k] == 0.f) m[t][k] = -INFINITY;  // no key
        // O in units of 2^m
        const float by = f[t][k] > 0.f ? 1.f / f[t][k] : 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          o[t][i][k] = f[t][k] > 0.f ? o[t][i][k] * by : o[t][i][k];
          o[t][i][k + 2] = f[t][k] > 0.f ? o[t][i][k + 2] * by : o[t][i][k + 2];
        }
      }
#pragma unroll 1
    for (int pair = DEC_WARPS / 2; pair >= 1; pair >>= 1) {
      float4* box = reinterpret_cast<float4*>(merge + (warp % pair) * NT * (1024 + 64));
      if (warp >= pair && warp < 2 * pair) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
#pragma unroll
          for (int i = 0; i < 8; ++i) box[(t * 8 + i) * 32 + lane] = make_float4(o[t][i][0], o[t][i][1], o[t][i][2], o[t][i][3]);
          if (g == 0) box[NT * 256 + t * 4 + c] = make_float4(m[t][0], m[t][1], l[t][0], l[t][1]);
        }
      }
      asm volatile("bar.sync 1, %0;" ::"n"(DEC_WARPS * 32) : "memory");
      if (warp < pair) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const float4 st = box[NT * 256 + t * 4 + c];
          float by[2], of[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float om = k ? st.y : st.x, ol = k ? st.w : st.z;
            const float M = fmaxf(m[t][k], om), M0 = fmaxf(M, -3e38f);
            by[k] = exp2_sfu(m[t][k] - M0);
            of[k] = exp2_sfu(om - M0);
            l[t][k] = l[t][k] * by[k] + ol * of[k];
            m[t][k] = M;
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float4 v = box[(t * 8 + i) * 32 + lane];
            o[t][i][0] = o[t][i][0] * by[0] + v.x * of[0];
            o[t][i][1] = o[t][i][1] * by[1] + v.y * of[1];
            o[t][i][2] = o[t][i][2] * by[0] + v.z * of[0];
            o[t][i][3] = o[t][i][3] * by[1] + v.w * of[1];
          }
        }
      }
      asm volatile("bar.sync 1, %0;" ::"n"(DEC_WARPS * 32) : "memory");
    }
    if (warp == 0) {
      const bool alone = u0 == x.first && x.stop == x.first + x.nu;
      const int slot = 2 * static_cast<int>(blockIdx.x) + (u0 == first ? 0 : 1);
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const int h = t * 8 + 2 * c + k;
          if (h >= heads) continue;
          const float inv = l[t][k] == 0.f ? 0.f : 1.f / l[t][k];
          float v[16];  // elements 16 g .. 16 g + 15
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            v[2 * i] = o[t][i][k] * inv;
            v[2 * i + 1] = o[t][i][k + 2] * inv;
          }
          if (alone) {
            const int64_t at = static_cast<int64_t>(x.b) * a.n_q + head0 + h;
            store_bf16x8(a.O + at * 128 + 16 * g, v);
            store_bf16x8(a.O + at * 128 + 16 * g + 8, v + 8);
            if (g == 0) a.lse[at] = l[t][k] == 0.f ? -INFINITY : m[t][k] * 0.69314718056f + logf(l[t][k]);
          } else {
            const int64_t at = static_cast<int64_t>(slot) * a.part_heads + h;
#pragma unroll
            for (int i = 0; i < 4; ++i)
              *reinterpret_cast<float4*>(a.part + at * 128 + 16 * g + 4 * i) =
                  make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
            if (g == 0) a.part_lse[at] = l[t][k] == 0.f ? -INFINITY : m[t][k] + log2f(l[t][k]);
          }
        }
    }
  }
}

// Joins the partial outputs of a (sequence, virtual head): with W the largest
// partial log-sum-exp, O = sum 2^(lse_i - W) O_i / sum 2^(lse_i - W).  A warp
// per query head; writes zeros for an empty sequence.
__global__ void __launch_bounds__(256) attn_decode_join_kernel(const DecodeArgs a) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int vheads = a.c.n_kv * a.splits;
  const int64_t at = static_cast<int64_t>(blockIdx.x) * 8 + (threadIdx.x >> 5);
  if (at >= static_cast<int64_t>(a.B) * a.n_q) return;
  const int b = static_cast<int>(at / a.n_q), head = static_cast<int>(at - static_cast<int64_t>(b) * a.n_q);
  const int before = a.units[b], places = (a.units[b + 1] - before) / vheads, per = a.units[a.B + 1];
  uint2* out = reinterpret_cast<uint2*>(a.O + at * 128 + lane * 4);
  if (places == 0) {
    *out = make_uint2(0, 0);
    if (lane == 0) a.lse[at] = -INFINITY;
    return;
  }
  const int kvh = head / a.group, in = head - kvh * a.group;
  const int vh = kvh * a.splits + in / DEC_HEADS, h = in % DEC_HEADS;
  const int u0 = before + vh * places + DEC_END, u1 = before + (vh + 1) * places - 1;  // places of its units
  const int c0 = u0 / per, c1 = u1 / per;
  if (c0 == c1) return;  // the stretch's CTA wrote the output
  float W = -INFINITY;
  for (int x = c0; x <= c1; ++x)
    W = fmaxf(W, a.part_lse[static_cast<int64_t>(2 * x + (max(u0, x * per) == x * per ? 0 : 1)) * a.part_heads + h]);
  const float W0 = W == -INFINITY ? 0.f : W;
  float acc[4] = {0.f, 0.f, 0.f, 0.f}, sum = 0.f;
  for (int x = c0; x <= c1; ++x) {
    const int64_t p = static_cast<int64_t>(2 * x + (max(u0, x * per) == x * per ? 0 : 1)) * a.part_heads + h;
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

cudaError_t launch_kv_append(const KvCache& c, const __nv_bfloat16* K, int64_t ldk, const __nv_bfloat16* V,
                             int64_t ldv, const int32_t* slots, int rows, int* status, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>((rows - 1) / 32 + 1);
  return attn_launch(kv_append_kernel, grid, 256, 0, s, c, K, ldk, V, ldv, slots, rows, status);
}

cudaError_t launch_kv_read(const KvCache& c, const int32_t* slots, int rows, void* K, void* V, bool f32, int* status,
                           cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>((rows - 1) / 16 + 1);
  return f32 ? attn_launch(kv_read_kernel<true>, grid, 256, 0, s, c, slots, rows, K, V, status)
             : attn_launch(kv_read_kernel<false>, grid, 256, 0, s, c, slots, rows, K, V, status);
}

cudaError_t launch_kv_accept(const AcceptArgs& a, cudaStream_t s) {
  return attn_launch(kv_accept_kernel, (static_cast<int64_t>(a.B) * 2 * a.c.n_kv + 7) / 8, 256, 0, s, a);
}

cudaError_t launch_attn_decode(const DecodeArgs& a, int sms, cudaStream_t s) {
  const unsigned ctas = a.part_heads <= 8 ? 3 : 2;  // per SM: registers
  const unsigned grid = std::min<unsigned>(DEC_MAX_CTAS, ctas * static_cast<unsigned>(sms));
  cudaError_t e;
  if (a.part_heads <= 8) {
    e = attn_smem_attribute(reinterpret_cast<const void*>(attn_decode_kernel<1>), 1, dec_smem_bytes(1));
    if (e == cudaSuccess) e = attn_launch(attn_decode_kernel<1>, grid, DEC_THREADS, dec_smem_bytes(1), s, a);
  } else {
    e = attn_smem_attribute(reinterpret_cast<const void*>(attn_decode_kernel<2>), 2, dec_smem_bytes(2));
    if (e == cudaSuccess) e = attn_launch(attn_decode_kernel<2>, grid, DEC_THREADS, dec_smem_bytes(2), s, a);
  }
  if (e != cudaSuccess) return e;
  return attn_launch(attn_decode_join_kernel, static_cast<unsigned>((static_cast<int64_t>(a.B) * a.n_q + 7) / 8), 256, 0, s,
                a);
}

}  // namespace coda

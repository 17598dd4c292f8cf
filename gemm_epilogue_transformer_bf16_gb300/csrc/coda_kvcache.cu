// The 4-bit key/value cache (NVFP4 rows): append, read back, and attention of
// one new token per sequence over it.
#include <algorithm>
#include <cuda_fp16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include "coda_attn.cuh"
#include "coda_internal.h"
#include "coda_kvcache.cuh"
#include "coda_status.h"

namespace coda {
namespace {

__device__ __forceinline__ int64_t cache_row(const KvCache& c, int page, int plane, int h, int off) {
  return ((static_cast<int64_t>(page) * 2 + plane) * c.n_kv + h << c.page_shift) + off;
}

// Two e2m1 codes of a byte as f16 (low nibble first), exact.
__device__ __forceinline__ uint32_t e2m1x2_f16(uint32_t byte) {
  const __half2_raw h = __nv_cvt_fp4x2_to_halfraw2(static_cast<__nv_fp4x2_storage_t>(byte), __NV_E2M1);
  return static_cast<uint32_t>(h.x) | (static_cast<uint32_t>(h.y) << 16);
}
// The eight codes of a word as four f16 pairs (byte by byte, low nibble
// first), exact: the conversion takes its byte from the register, without
// shifts and masks.
__device__ __forceinline__ void e2m1x8_f16(uint32_t w, uint32_t (&o)[4]) {
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(o[0]), "=r"(o[1]), "=r"(o[2]), "=r"(o[3])
      : "r"(w));
}
__device__ __forceinline__ uint32_t e4m3x2_f16(uint32_t two) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(two), __NV_E4M3);
  return static_cast<uint32_t>(h.x) | (static_cast<uint32_t>(h.y) << 16);
}
__device__ __forceinline__ float e4m3_f32(uint32_t b) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw(static_cast<__nv_fp8_storage_t>(b), __NV_E4M3);
  return __half2float(__half(h));
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ float f16_lo(uint32_t v) { return __half2float(__ushort_as_half(v & 0xFFFFu)); }
__device__ __forceinline__ float f16_hi(uint32_t v) { return __half2float(__ushort_as_half(v >> 16)); }

// ------------------------------------------------------------------ append
// Eight lanes per row of 128, one 16-element block each; every arithmetic
// step is one fp32 operation, the same steps as quantize_nvfp4_rows, so the
// codes and scales agree with it bit for bit.  HBM-bound: 512 bytes in and
// 152 out per token and head.
__global__ void __launch_bounds__(256)
    kv_append_kernel(const KvCache c, const __nv_bfloat16* __restrict__ K, int64_t ldk,
                     const __nv_bfloat16* __restrict__ V, int64_t ldv, const int32_t* __restrict__ slots, int64_t T,
                     int* status) {
  griddep_wait();
  griddep_launch_dependents();
  const int sub = threadIdx.x & 7;
  const int64_t rows = T * 2 * c.n_kv;
  const int64_t step = static_cast<int64_t>(gridDim.x) * 32;
  // whole warps stay in the loop: the shuffles below need all lanes
  for (int64_t base = static_cast<int64_t>(blockIdx.x) * 32 + (threadIdx.x >> 5) * 4; base < rows; base += step) {
    const int64_t row = base + ((threadIdx.x & 31) >> 3);
    bool live = row < rows;
    const int64_t t = live ? row / (2 * c.n_kv) : 0;
    const int rest = live ? static_cast<int>(row - t * 2 * c.n_kv) : 0;
    const int plane = rest / c.n_kv, h = rest - plane * c.n_kv;
    const int slot = live ? slots[t] : -1;
    if (slot < 0) {
      live = false;
    } else if ((slot >> c.page_shift) >= c.num_pages) {
      live = false;
      if (rest == 0 && sub == 0) atomicOr(status, CODA_DEV_PAGE_RANGE);
    }
    float x[16];
    if (live) {
      const __nv_bfloat16* src = (plane ? V + t * ldv : K + t * ldk) + h * 128 + sub * 16;
      load_bf16x8(src, x);
      load_bf16x8(src + 8, x + 8);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = 0.f;
    }
    float bmax = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) bmax = fmaxf(bmax, fabsf(x[i]));
    float amax = bmax;
#pragma unroll
    for (int o = 4; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    const float s = amax > 0.f ? __fdiv_rn(amax, 2688.0f) : 1.0f;
    const float sf_f = fminf(__fdiv_rn(bmax, __fmul_rn(6.0f, s)), 448.0f);
    const uint32_t sfb = __nv_cvt_float_to_fp8(sf_f, __NV_SATFINITE, __NV_E4M3);
    const float denom = __fmul_rn(e4m3_f32(sfb), s);
    uint32_t w[2] = {0, 0};
    if (denom > 0.f) {
      const float inv = fminf(__fdiv_rn(1.0f, denom), 3.40282347e38f);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t c2 = __nv_cvt_float2_to_fp4x2(
            make_float2(__fmul_rn(x[2 * i], inv), __fmul_rn(x[2 * i + 1], inv)), __NV_E2M1, cudaRoundNearest);
        w[i >> 2] |= (c2 & 0xFFu) << (8 * (i & 3));
      }
      // no negative zero: clear the sign of codes whose magnitude bits are 0
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t mag = w[i] & 0x77777777u;
        const uint32_t any = (mag | (mag << 1) | (mag << 2)) & 0x44444444u;
        w[i] &= 0x77777777u | (any << 1);
      }
    }
    if (live) {
      const int64_t r = cache_row(c, slot >> c.page_shift, plane, h, slot & ((1 << c.page_shift) - 1));
      *reinterpret_cast<uint2*>(c.codes + r * 64 + sub * 8) = make_uint2(w[0], w[1]);
      c.sf[r * 8 + sub] = static_cast<uint8_t>(sfb);
      if (sub == 0) c.scale[r] = s;
    }
  }
}

// -------------------------------------------------------------------- read
// The rows back: (e2m1 * e4m3, exact) * scale, one fp32 rounding; then bf16
// for the bf16 form.  Eight lanes per row as above.
template <bool F32>
__global__ void __launch_bounds__(256)
    kv_read_kernel(const KvCache c, const int32_t* __restrict__ slots, int64_t T, void* __restrict__ K,
                   void* __restrict__ V, int* status) {
  griddep_wait();
  griddep_launch_dependents();
  const int sub = threadIdx.x & 7;
  const int64_t rows = T * 2 * c.n_kv;
  for (int64_t row = static_cast<int64_t>(blockIdx.x) * 32 + (threadIdx.x >> 3); row < rows;
       row += static_cast<int64_t>(gridDim.x) * 32) {
    const int64_t t = row / (2 * c.n_kv);
    const int rest = static_cast<int>(row - t * 2 * c.n_kv);
    const int plane = rest / c.n_kv, h = rest - plane * c.n_kv;
    const int slot = slots[t];
    float v[16];
    const bool inside = slot >= 0 && (slot >> c.page_shift) < c.num_pages;
    if (slot >= 0 && !inside && rest == 0 && sub == 0) atomicOr(status, CODA_DEV_PAGE_RANGE);
    if (inside) {
      const int64_t r = cache_row(c, slot >> c.page_shift, plane, h, slot & ((1 << c.page_shift) - 1));
      const uint2 w = *reinterpret_cast<const uint2*>(c.codes + r * 64 + sub * 8);
      const float sf = e4m3_f32(c.sf[r * 8 + sub]), sc = c.scale[r];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t p = e2m1x2_f16(((i < 4 ? w.x : w.y) >> (8 * (i & 3))) & 0xFFu);
        v[2 * i] = __fmul_rn(f16_lo(p) * sf, sc);
        v[2 * i + 1] = __fmul_rn(f16_hi(p) * sf, sc);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = 0.f;
    }
    const int64_t at = (t * c.n_kv + h) * 128 + sub * 16;
    if constexpr (F32) {
      float4* o = reinterpret_cast<float4*>(static_cast<float*>(plane ? V : K) + at);
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
    } else {
      __nv_bfloat16* o = static_cast<__nv_bfloat16*>(plane ? V : K) + at;
      store_bf16x8(o, v);
      store_bf16x8(o + 8, v + 8);
    }
  }
}

// ------------------------------------------------------------------ decode
// One query token per sequence over its cached keys and values:
//   s_j = scale q . k_j,  O = sum_j exp(s_j - lse) v_j,
// HBM-bound: 152 bytes per cached token and key/value head feed 4 * 128
// multiply-adds per query head.  The cost beside the bytes is unpacking: 256
// codes per token and head.
//
// Work: every (sequence, key/value head) is cut into units of 128 keys; the
// units of the whole batch form one line that the CTAs divide evenly, so a
// batch of mixed lengths, or one long sequence, keeps every SM busy.  A CTA
// whose stretch covers a whole (sequence, head) writes the output itself;
// the others leave normalised partial outputs, merged by a second kernel.
//
// A warp takes tiles of 32 keys, copied to its own shared-memory ring by
// cp.async two tiles ahead.  Products are m16n8k16 on f16:
//   S^T [16 keys x 8 heads] = K Q^T:  e2m1 * e4m3 has at most 6 significant
//     bits, so K' = code * sf is exact in f16; the row scale multiplies S.
//     A lane's 16 bytes of a key row are 32 neighbouring elements, two blocks
//     with one scale each: the k index of the product is a permutation of
//     the head's elements, the same for Q.
//   O^T [16 elements x 8 heads] += V'^T P'^T with the row scale of V in
//     P' = exp2(z - m) * rs * f, where f (per head) keeps P' <= 2^8: P' is
//     rounded to f16 (2^-11), O accumulates in fp32.
// The keys of a tile are read in the order 0 4 1 5 2 6 3 7: then the lanes'
// shared-memory reads of both K and V are contiguous, and movmatrix turns
// the S^T fragment into the P operand.
constexpr int DEC_WARPS = 4;
constexpr int DEC_STAGES = 3;
constexpr int DEC_TILE = 32;
constexpr int DEC_UNIT = 128;
constexpr int ST_K = 0, ST_V = 2048, ST_SFK = 4096, ST_SFV = 4352, ST_RSK = 4608, ST_RSV = 4736;
constexpr int DEC_STAGE_BYTES = 4864;
constexpr int DEC_SMEM = DEC_WARPS * DEC_STAGES * DEC_STAGE_BYTES;
static_assert(DEC_SMEM >= DEC_WARPS * DEC_HEADS * (128 + 4) * 4, "merge buffer");

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool fill) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(fill ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t movmatrix_t(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
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

// Copies keys [key, key + 32) of the sequence, those below `len` whose pages
// are in the cache; returns one bit per 16-key half that has such keys.
__device__ __forceinline__ uint32_t decode_fetch(const DecodeArgs& a, const int32_t* table, int kvh, int key, int len,
                                                 uint32_t stage) {
  const int lane = threadIdx.x & 31;
  const KvCache& c = a.c;
  uint32_t halves = 0;
  int64_t row[2];  // of the keys plane
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int k = key + 16 * h;
    row[h] = 0;
    if (k < len) {
      const int page = table[k >> c.page_shift];
      if (page >= 0 && page < c.num_pages) {
        halves |= 1u << h;
        row[h] = cache_row(c, page, 0, kvh, k & ((1 << c.page_shift) - 1));
      } else if (lane == 0) {
        atomicOr(a.status, CODA_DEV_PAGE_RANGE);
      }
    }
  }
  const int64_t plane = static_cast<int64_t>(c.n_kv) << c.page_shift;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int h = i >> 1;
    const uint32_t o = i * 512 + lane * 16;
    const uint8_t* src = c.codes + row[h] * 64 + (o & 1023);
    const bool on = (halves >> h) & 1;
    cp_async16(stage + ST_K + o, src, on);
    cp_async16(stage + ST_V + o, on ? src + plane * 64 : src, on);
  }
  {
    const int h = (lane >> 3) & 1;  // 8 lanes cover 16 keys of one plane
    const bool on = (halves >> h) & 1;
    const int64_t r = row[h] + (on && lane >= 16 ? plane : 0);
    cp_async16(stage + ST_SFK + lane * 16, c.sf + r * 8 + (lane & 7) * 16, on);
    if (lane < 16) {
      const int h2 = (lane >> 2) & 1;  // 4 lanes cover 16 keys
      const bool on2 = (halves >> h2) & 1;
      const int64_t r2 = row[h2] + (on2 && lane >= 8 ? plane : 0);
      cp_async16(stage + ST_RSK + lane * 16, c.scale + r2 + (lane & 3) * 4, on2);
    }
  }
  return halves;
}

template <int NT>
__global__ void __launch_bounds__(DEC_WARPS * 32, 3) attn_decode_kernel(const DecodeArgs a) {
  extern __shared__ __align__(128) uint8_t dec_smem[];
  __shared__ int sh_warp[DEC_WARPS], sh_seq, sh_before;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, c = lane & 3;
  const int vheads = a.c.n_kv * a.splits;
  griddep_wait();
  griddep_launch_dependents();

  // units before each sequence: a contiguous run of sequences per thread,
  // scanned over the block
  const int chunk = (a.B + DEC_WARPS * 32 - 1) / (DEC_WARPS * 32);
  const int s0 = min(a.B, tid * chunk), s1 = min(a.B, s0 + chunk);
  int mine = 0;
  for (int b = s0; b < s1; ++b) mine += (decode_len(a, b, blockIdx.x == 0) + DEC_UNIT - 1) / DEC_UNIT * vheads;
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
  for (int w = 0; w < DEC_WARPS; ++w) {
    if (w < warp) incl += sh_warp[w];
    total += sh_warp[w];
  }
  const int per = max(1, (total + static_cast<int>(gridDim.x) - 1) / static_cast<int>(gridDim.x));
  const int first = static_cast<int>(blockIdx.x) * per, last = min(total, first + per);
  {
    int before = incl - mine;
    for (int b = s0; b < s1; ++b) {
      const int n = (decode_len(a, b, false) + DEC_UNIT - 1) / DEC_UNIT * vheads;
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

  uint8_t* ring = dec_smem + warp * DEC_STAGES * DEC_STAGE_BYTES;
  const uint32_t ring_u = smem_u32(ring);
  int b = sh_seq, before = sh_before;
  int u = first;
  while (u < last) {
    // next (sequence, virtual head) stretch
    int len = decode_len(a, b, false);
    int nu = (len + DEC_UNIT - 1) / DEC_UNIT;
    while (u >= before + nu * vheads) {
      before += nu * vheads;
      len = decode_len(a, ++b, false);
      nu = (len + DEC_UNIT - 1) / DEC_UNIT;
    }
    const int vh = (u - before) / nu;
    const int h_first = before + vh * nu;               // the stretch's units are [h_first, h_first + nu)
    const int stop = min(last, h_first + nu);
    const int key0 = (u - h_first) * DEC_UNIT, key1 = min(len, (stop - h_first) * DEC_UNIT);
    const int kvh = vh / a.splits;
    const int head0 = kvh * a.group + (vh - kvh * a.splits) * DEC_HEADS;
    const int heads = min(DEC_HEADS, (kvh + 1) * a.group - head0);
    const int32_t* table = a.table + static_cast<int64_t>(b) * a.max_pages;

    // Q of head g (+ 8 per n tile), elements 32c .. 32c + 31, scaled by a
    // power of two to a maximum in [1, 2) so that f16 holds it
    uint32_t q[NT][16];
    float hf[NT][2];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      float x[32];
      const int h = t * 8 + g;
      if (h < heads) {
        const __nv_bfloat16* src = a.Q + b * a.ldq + (head0 + h) * 128 + c * 32;
#pragma unroll
        for (int i = 0; i < 4; ++i) load_bf16x8(src + 8 * i, x + 8 * i);
      } else {
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] = 0.f;
      }
      float mx = 0.f;
#pragma unroll
      for (int i = 0; i < 32; ++i) mx = fmaxf(mx, fabsf(x[i]));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      int e = static_cast<int>(__float_as_uint(mx) >> 23) - 127;
      e = mx == 0.f ? 0 : max(-126, min(126, e));
      const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
      for (int i = 0; i < 16; ++i) q[t][i] = pack_f16(x[2 * i] * down, x[2 * i + 1] * down);
      const float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23) * a.scale_log2;
      hf[t][0] = __shfl_sync(0xffffffffu, up, (2 * c) * 4);
      hf[t][1] = __shfl_sync(0xffffffffu, up, (2 * c + 1) * 4);
    }

    float m[NT][2], l[NT][2], f[NT][2], o[NT][8][4];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        m[t][k] = -INFINITY;
        l[t][k] = 0.f;
        f[t][k] = 0.f;
      }
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[t][i][k] = 0.f;
    }

    // this warp's tiles: key0 + 32 * (warp + 4 i)
    const int tiles = (key1 - key0 + DEC_TILE - 1) / DEC_TILE;
    const int count = tiles > warp ? (tiles - warp + DEC_WARPS - 1) / DEC_WARPS : 0;
    uint32_t have = 0;  // two bits per stage
    auto fetch = [&](int i) {
      if (i < count) {
        const uint32_t s = i % DEC_STAGES;
        const uint32_t h = decode_fetch(a, table, kvh, key0 + DEC_TILE * (warp + DEC_WARPS * i), key1,
                                        ring_u + s * DEC_STAGE_BYTES);
        have = (have & ~(3u << (2 * s))) | (h << (2 * s));
      }
      cp_commit();
    };
#pragma unroll
    for (int i = 0; i < DEC_STAGES - 1; ++i) fetch(i);
    for (int i = 0; i < count; ++i) {
      fetch(i + DEC_STAGES - 1);
      cp_wait<DEC_STAGES - 1>();
      __syncwarp();
      const int s = i % DEC_STAGES;
      const uint8_t* st = ring + s * DEC_STAGE_BYTES;
      const int key = key0 + DEC_TILE * (warp + DEC_WARPS * i);
      const uint32_t on = (have >> (2 * s)) & 3u;
      const int left = key1 - key;  // keys of the tile that exist
      const bool whole = on == 3u && left >= DEC_TILE;
      const int pi = (g >> 1) + (g & 1) * 4;  // key of fragment row g; row g + 8 is 8 keys on

      // S^T and the weights
      float z[NT][2][4];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int k = 0; k < 4; ++k) z[t][h][k] = 0.f;
        const uint8_t* kp = st + ST_K + (16 * h + pi) * 64 + c * 16;
        const uint4 w0 = *reinterpret_cast<const uint4*>(kp), w1 = *reinterpret_cast<const uint4*>(kp + 512);
        const uint32_t f0 = e4m3x2_f16(*reinterpret_cast<const uint16_t*>(st + ST_SFK + (16 * h + pi) * 8 + 2 * c));
        const uint32_t f1 = e4m3x2_f16(*reinterpret_cast<const uint16_t*>(st + ST_SFK + (16 * h + pi + 8) * 8 + 2 * c));
        // both halves of the scale register: block 2c for the first 16 elements, 2c + 1 for the others
        const uint32_t g00 = __byte_perm(f0, f0, 0x1010), g01 = __byte_perm(f0, f0, 0x3232);
        const uint32_t g10 = __byte_perm(f1, f1, 0x1010), g11 = __byte_perm(f1, f1, 0x3232);
#pragma unroll
        for (int k = 0; k < 8; k += 2) {
          uint32_t x[4], y[4];
          e2m1x8_f16(k == 0 ? w0.x : k == 2 ? w0.y : k == 4 ? w0.z : w0.w, x);
          e2m1x8_f16(k == 0 ? w1.x : k == 2 ? w1.y : k == 4 ? w1.z : w1.w, y);
          const uint32_t g0 = k < 4 ? g00 : g01, g1 = k < 4 ? g10 : g11;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t a0 = hmul2(x[2 * i], g0), a1 = hmul2(y[2 * i], g1);
            const uint32_t a2 = hmul2(x[2 * i + 1], g0), a3 = hmul2(y[2 * i + 1], g1);
#pragma unroll
            for (int t = 0; t < NT; ++t) mma_f16(z[t][h], a0, a1, a2, a3, q[t][2 * (k + i)], q[t][2 * (k + i) + 1]);
          }
        }
        const float* rk = reinterpret_cast<const float*>(st + ST_RSK) + 16 * h + pi;
        const float r0 = rk[0], r1 = rk[8];
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int k = 0; k < 4; ++k) z[t][h][k] = z[t][h][k] * (k < 2 ? r0 : r1) * hf[t][k & 1];
        if (!whole) {
          const bool in0 = ((on >> h) & 1) && 16 * h + pi < left, in1 = ((on >> h) & 1) && 16 * h + pi + 8 < left;
#pragma unroll
          for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int k = 0; k < 4; ++k) z[t][h][k] = (k < 2 ? in0 : in1) ? z[t][h][k] : -INFINITY;
        }
      }
      // raise the reference maximum when a score lies more than 2^8 above it
      float top[NT][2];
      bool up = false;
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          top[t][k] = fmaxf(fmaxf(z[t][0][k], z[t][0][k + 2]), fmaxf(z[t][1][k], z[t][1][k + 2]));
          up |= top[t][k] > m[t][k] + 8.f;
        }
      if (__any_sync(0xffffffffu, up)) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float x = top[t][k];
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
            if (x > m[t][k]) {
              const float by = x - m[t][k];
              l[t][k] *= exp2_sfu(-by);   // m = -inf: l is 0 and stays 0
              // O is in units of f * 2^m and keeps its value
              f[t][k] = f[t][k] == 0.f ? 0.f : fminf(f[t][k] * exp2_sfu(by), 3e38f);
              m[t][k] = x;
            }
          }
      }
      const float* rv = reinterpret_cast<const float*>(st + ST_RSV);
      float big[NT][2];
#pragma unroll
      for (int t = 0; t < NT; ++t) big[t][0] = big[t][1] = 0.f;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float r0 = rv[16 * h + pi], r1 = rv[16 * h + pi + 8];
        if (!whole) {
          r0 = ((on >> h) & 1) && 16 * h + pi < left ? r0 : 0.f;
          r1 = ((on >> h) & 1) && 16 * h + pi + 8 < left ? r1 : 0.f;
        }
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float mm = m[t][k & 1];
            const float e = exp2_sfu(z[t][h][k] - (mm == -INFINITY ? 0.f : mm));
            l[t][k & 1] += e;
            z[t][h][k] = e * (k < 2 ? r0 : r1);
            big[t][k & 1] = fmaxf(big[t][k & 1], z[t][h][k]);
          }
      }
      up = false;
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int k = 0; k < 2; ++k) up |= big[t][k] * f[t][k] > 256.f || (f[t][k] == 0.f && big[t][k] > 0.f);
      if (__any_sync(0xffffffffu, up)) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float x = big[t][k];
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
            if (x * f[t][k] > 1.f || (f[t][k] == 0.f && x > 0.f)) {
              const float nf = fminf(1.f / x, 3e38f);
              const float by = f[t][k] == 0.f ? 0.f : nf / f[t][k];
              f[t][k] = nf;
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                o[t][i][k] *= by;
                o[t][i][k + 2] *= by;
              }
            }
          }
      }
      // O^T += V'^T P'^T
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t p[NT][2];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          p[t][0] = movmatrix_t(pack_f16(z[t][h][0] * f[t][0], z[t][h][1] * f[t][1]));
          p[t][1] = movmatrix_t(pack_f16(z[t][h][2] * f[t][0], z[t][h][3] * f[t][1]));
        }
        // keys c, c + 4, c + 8, c + 12; elements 16 g .. 16 g + 15: one block
        uint2 w[4];
        uint32_t sf[4];
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int kk = 16 * h + c + 4 * x;
          w[x] = *reinterpret_cast<const uint2*>(st + ST_V + kk * 64 + g * 8);
          sf[x] = st[ST_SFV + kk * 8 + g];
          if (!whole && !(((on >> h) & 1) && kk < left)) sf[x] = 0;  // an unwritten row's scale may be NaN
        }
        const uint32_t g0 = e4m3x2_f16(sf[0] | (sf[1] << 8)), g1 = e4m3x2_f16(sf[2] | (sf[3] << 8));
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const uint32_t x0 = half ? w[0].y : w[0].x, x1 = half ? w[1].y : w[1].x;
          const uint32_t x2 = half ? w[2].y : w[2].x, x3 = half ? w[3].y : w[3].x;
          // the same element of two keys in one byte: even elements, odd elements
          const uint32_t ev0 = (x0 & 0x0F0F0F0Fu) | ((x1 << 4) & 0xF0F0F0F0u);
          const uint32_t od0 = ((x0 >> 4) & 0x0F0F0F0Fu) | (x1 & 0xF0F0F0F0u);
          const uint32_t ev1 = (x2 & 0x0F0F0F0Fu) | ((x3 << 4) & 0xF0F0F0F0u);
          const uint32_t od1 = ((x2 >> 4) & 0x0F0F0F0Fu) | (x3 & 0xF0F0F0F0u);
          uint32_t e0[4], o0[4], e1[4], o1[4];
          e2m1x8_f16(ev0, e0);
          e2m1x8_f16(od0, o0);
          e2m1x8_f16(ev1, e1);
          e2m1x8_f16(od1, o1);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t a0 = hmul2(e0[j], g0), a1 = hmul2(o0[j], g0), a2 = hmul2(e1[j], g1), a3 = hmul2(o1[j], g1);
#pragma unroll
            for (int t = 0; t < NT; ++t) mma_f16(o[t][half * 4 + j], a0, a1, a2, a3, p[t][0], p[t][1]);
          }
        }
      }
      __syncwarp();  // the stage may be refilled
    }
    cp_wait<0>();
    __syncthreads();

    // merge the warps: row w * 16 + head of 132 floats (128 outputs, m, l, f)
    float* mg = reinterpret_cast<float*>(dec_smem);
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float x = l[t][k];
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
        float* row = mg + (warp * DEC_HEADS + t * 8 + 2 * c + k) * 132;
#pragma unroll
        for (int i = 0; i < 8; ++i) *reinterpret_cast<float2*>(row + 16 * g + 2 * i) = make_float2(o[t][i][k], o[t][i][k + 2]);
        if (g == 0) {
          row[128] = m[t][k];
          row[129] = x;
          row[130] = f[t][k];
        }
      }
    __syncthreads();
    const bool alone = u == h_first && stop == h_first + nu;
    const int slot = 2 * static_cast<int>(blockIdx.x) + (u == first ? 0 : 1);
    for (int h = warp; h < heads; h += DEC_WARPS) {
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < DEC_WARPS; ++w) M = fmaxf(M, mg[(w * DEC_HEADS + h) * 132 + 128]);
      const float M0 = M == -INFINITY ? 0.f : M;
      float L = 0.f, acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = 0; w < DEC_WARPS; ++w) {
        const float* row = mg + (w * DEC_HEADS + h) * 132;
        const float e = exp2_sfu(row[128] - M0);
        L += row[129] * e;
        const float by = row[130] > 0.f ? e / row[130] : 0.f;
        const float4 v = *reinterpret_cast<const float4*>(row + lane * 4);
        if (row[130] != 0.f) {
          acc[0] += v.x * by;
          acc[1] += v.y * by;
          acc[2] += v.z * by;
          acc[3] += v.w * by;
        }
      }
      const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[i] *= inv;
      if (alone) {
        uint2 v;
        v.x = pack_bf16x2(acc[0], acc[1]);
        v.y = pack_bf16x2(acc[2], acc[3]);
        *reinterpret_cast<uint2*>(a.O + (static_cast<int64_t>(b) * a.n_q + head0 + h) * 128 + lane * 4) = v;
        if (lane == 0)
          a.lse[static_cast<int64_t>(b) * a.n_q + head0 + h] = L == 0.f ? -INFINITY : M * 0.69314718056f + logf(L);
      } else {
        const int64_t at = static_cast<int64_t>(slot) * a.part_heads + h;
        *reinterpret_cast<float4*>(a.part + at * 128 + lane * 4) = make_float4(acc[0], acc[1], acc[2], acc[3]);
        if (lane == 0) a.part_lse[at] = L == 0.f ? -INFINITY : M + log2f(L);
      }
    }
    __syncthreads();  // the merge buffer is the next stretch's ring
    u = stop;
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
  const int before = a.units[b], nu = (a.units[b + 1] - before) / vheads, per = a.units[a.B + 1];
  uint2* out = reinterpret_cast<uint2*>(a.O + at * 128 + lane * 4);
  if (nu == 0) {
    *out = make_uint2(0, 0);
    if (lane == 0) a.lse[at] = -INFINITY;
    return;
  }
  const int kvh = head / a.group, in = head - kvh * a.group;
  const int vh = kvh * a.splits + in / DEC_HEADS, h = in % DEC_HEADS;
  const int u0 = before + vh * nu, u1 = u0 + nu - 1;
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

template <class... Exp, class... Act>
cudaError_t launch(void (*kern)(Exp...), unsigned grid, unsigned threads, uint32_t smem, cudaStream_t s,
                   Act&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = attn_programmatic_launch() ? 1 : 0;
  note_launch();
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, static_cast<Exp>(args)...);
  return e != cudaSuccess ? e : cudaGetLastError();
}

unsigned row_grid(int64_t rows, int sms) {
  return static_cast<unsigned>(std::max<int64_t>(1, std::min<int64_t>((rows + 31) / 32, static_cast<int64_t>(sms) * 8)));
}

}  // namespace

cudaError_t launch_kv_append(const KvCache& c, const __nv_bfloat16* K, int64_t ldk, const __nv_bfloat16* V,
                             int64_t ldv, const int32_t* slots, int64_t T, int* status, int sms, cudaStream_t s) {
  return launch(kv_append_kernel, row_grid(T * 2 * c.n_kv, sms), 256, 0, s, c, K, ldk, V, ldv, slots, T, status);
}

cudaError_t launch_kv_read(const KvCache& c, const int32_t* slots, int64_t T, void* K, void* V, bool f32, int* status,
                           int sms, cudaStream_t s) {
  const unsigned grid = row_grid(T * 2 * c.n_kv, sms);
  return f32 ? launch(kv_read_kernel<true>, grid, 256, 0, s, c, slots, T, K, V, status)
             : launch(kv_read_kernel<false>, grid, 256, 0, s, c, slots, T, K, V, status);
}

cudaError_t launch_attn_decode(const DecodeArgs& a, int sms, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>(std::min(DEC_MAX_CTAS, 3 * sms));
  cudaError_t e;
  if (a.part_heads <= 8) {
    e = attn_smem_attribute(reinterpret_cast<const void*>(attn_decode_kernel<1>), 1, DEC_SMEM);
    if (e == cudaSuccess) e = launch(attn_decode_kernel<1>, grid, DEC_WARPS * 32, DEC_SMEM, s, a);
  } else {
    e = attn_smem_attribute(reinterpret_cast<const void*>(attn_decode_kernel<2>), 2, DEC_SMEM);
    if (e == cudaSuccess) e = launch(attn_decode_kernel<2>, grid, DEC_WARPS * 32, DEC_SMEM, s, a);
  }
  if (e != cudaSuccess) return e;
  return launch(attn_decode_join_kernel, static_cast<unsigned>((static_cast<int64_t>(a.B) * a.n_q + 7) / 8), 256, 0, s,
                a);
}

}  // namespace coda

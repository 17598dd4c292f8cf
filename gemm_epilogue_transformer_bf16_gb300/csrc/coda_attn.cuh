// Shared pieces of the attention kernels: the work list that the packed
// sequences are cut into, PTX wrappers the GEMM does not need (3-D TMA,
// UMMA with the A operand in TMEM, TMEM stores, packed fp32 arithmetic), and
// the launchers' declarations.
#pragma once
#include <cstdint>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "coda_internal.h"
#include "coda_ptx.cuh"

namespace coda {

constexpr int ATTN_D = 128;    // head width
constexpr int ATTN_BLK = 128;  // keys per block, rows per tile

// One entry of a work list: a run of query (or key) rows of one sequence.
// The sequence has queries [q0, q0 + lq) and keys [k0, k0 + lk) of the packed
// tensors; t0 is the run's first row within the sequence.
struct AttnTile {
  int q0, lq, k0, lk;
  int t0, seq;
  int slot;   // number of the part among all parts of cut runs; -1: a whole run
  int block;  // query list: the part's first key block
};
static_assert(sizeof(AttnTile) == 32, "two 16-byte loads");

// Work lists in the caller's workspace, written by attn_plan_kernel before
// the kernels that walk them.  counts[0]: entries of the query list;
// counts[1]: entries of the key list.  Runs may be cut (see attn_plan_kernel):
// counts[2] is the number of parts that the query heads of a group are cut into
// (key list), or the key blocks of a part (query list); counts[3] the number of
// runs cut, whose first parts stand in `cuts`.  A call cuts one of its lists.
struct AttnPlan {
  int* counts;
  AttnTile* q_tiles;
  AttnTile* k_tiles;  // null: no key list
  AttnTile* cuts;
};

struct AttnPlanArgs {
  const int32_t* cu_q;
  const int32_t* cu_k;
  int n_seq;
  int64_t Tq, Tk;
  int q_span;        // query rows per q_tiles entry
  int* prefix_q;     // [n_seq + 1] scratch
  int* prefix_k;
  AttnPlan plan;
  int n_kv, group;   // key list: heads
  int max_parts;     // key list: bound on the parts of all key tiles and heads (0: never cut)
  int max_q_parts;   // query list: bound on the parts of all runs (0: never cut)
  int q_items;       // items per entry of the query list
  uint32_t divisors;  // bit s - 1: a group may be cut into s parts (2 <= s <= 32)
  int sms;
  int* status;
};
// Programmatic dependent launch of the attention kernels (CODA_PDL=0: off).
bool attn_programmatic_launch();
// Raises a kernel's dynamic shared-memory limit, once per device and kernel id.
cudaError_t attn_smem_attribute(const void* kernel, int id, uint32_t bytes);

// Launch with the programmatic attribute: the kernel's prologue may run while
// the kernel before it ends (griddep_wait orders the rest).
template <class... Exp, class... Act>
cudaError_t attn_launch(void (*kern)(Exp...), int64_t grid, unsigned threads, uint32_t smem, cudaStream_t s,
                        Act&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(grid < 1 ? 1 : grid));
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

cudaError_t launch_attn_plan(const AttnPlanArgs& a, cudaStream_t s);

struct AttnFwdArgs {
  const int* counts;
  const AttnTile* tiles;
  __nv_bfloat16* O;  // [Tq, n_q * 128]
  float* lse;        // [n_q, Tq]
  int64_t Tq;
  int n_q, group;    // query heads; query heads per key/value head
  int head_shift;    // log2 of the heads that share a 128-row tile
  float* part;       // [part, item of the entry, 2, 32, 128, 4] partial O where the keys of a run are cut; null: never
  float* part_lse;   // [part, item of the entry, 2, 128] their log2-sum-exp
  const AttnTile* cuts;
  int pair_heads;    // 1: an item's two tiles are two head sets on the same tokens; 0: consecutive tokens
  float scale_log2;  // scale * log2(e)
  float scale;
  int* status;
  uint64_t timeout_ns;
};
cudaError_t launch_attn_fwd(const AttnFwdArgs& a, const CUtensorMap* maps, int64_t max_items, int sms,
                            cudaStream_t s);

// Per-row values of the backward live in padded rows: sequence b's queries
// start at row (q0 / 128 + b) * 128, so every 128-row tile is aligned and its
// rows behind the sequence exist.
struct AttnBwdArgs {
  const int* counts;
  const AttnTile* q_tiles;
  const AttnTile* k_tiles;
  const AttnTile* cuts;
  const float* lse;         // [n_q, Tq]
  float* nlse2;             // [n_q, Tp]: -lse * log2(e); -inf where the row has no weight
  float* ndelta;            // [n_q, Tp]: -rowsum(dO * O)
  __nv_bfloat16* dQ;       // [Tq, n_q * 128]
  __nv_bfloat16* dK;       // [Tk, n_kv * 128]
  __nv_bfloat16* dV;
  int64_t Tq, Tk, Tp;
  int n_q, n_kv, group;
  float* part;             // [cut tile, n_kv, part, 2, 32, 128, 4] partial dV | dK
  int max_parts;
  float scale_log2, scale;
  int* status;
  uint64_t timeout_ns;
};
// maps: Q, K, V, dO, O (boxes of 64 columns x 128 rows)
cudaError_t launch_attn_bwd(const AttnBwdArgs& a, const CUtensorMap* maps, int64_t max_q_tiles, int64_t max_k_tiles,
                            int sms, cudaStream_t s);

// --------------------------------------------------------------------- PTX
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* m, uint64_t* bar, int x, int y, int z,
                                            uint32_t p) {
  asm volatile(
      "{\n\t.reg .pred P;\n\tsetp.ne.b32 P, %6, 0;\n\t"
      "@P cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];\n\t}" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(p)
      : "memory");
}

// D[tmem] (+)= A[tmem] * B[smem]^T: A is bf16, two elements per 32-bit TMEM
// column, row = lane.
__device__ __forceinline__ void umma_bf16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc, uint32_t idesc,
                                             uint32_t accumulate, uint32_t p) {
  asm volatile(
      "{\n\t.reg .pred A, P;\n\t"
      "setp.ne.b32 A, %4, 0;\n\t"
      "setp.ne.b32 P, %5, 0;\n\t"
      "@P tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, A;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate), "r"(p)
      : "memory");
}

#define CODA_R8(a, i) "=r"(a[i]), "=r"(a[i + 1]), "=r"(a[i + 2]), "=r"(a[i + 3]), "=r"(a[i + 4]), "=r"(a[i + 5]), \
                      "=r"(a[i + 6]), "=r"(a[i + 7])
#define CODA_R32(a, i) CODA_R8(a, i), CODA_R8(a, i + 8), CODA_R8(a, i + 16), CODA_R8(a, i + 24)
#define CODA_W8(a, i) "r"(a[i]), "r"(a[i + 1]), "r"(a[i + 2]), "r"(a[i + 3]), "r"(a[i + 4]), "r"(a[i + 5]), \
                      "r"(a[i + 6]), "r"(a[i + 7])
#define CODA_W32(a, i) CODA_W8(a, i), CODA_W8(a, i + 8), CODA_W8(a, i + 16), CODA_W8(a, i + 24)

// 128 (64) consecutive fp32 columns of one TMEM lane per thread, wait
// included: loads of 32 columns each, so the registers need not be one
// consecutive run.
__device__ __forceinline__ void tmem_ld128(uint32_t taddr, uint32_t (&r)[128]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%128];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, %48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%129];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%64, %65, %66, %67, %68, %69, %70, %71, %72, %73, %74, %75, %76, %77, %78, %79, %80, %81, %82, %83, %84, %85, %86, %87, %88, %89, %90, %91, %92, %93, %94, %95}, [%130];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%96, %97, %98, %99, %100, %101, %102, %103, %104, %105, %106, %107, %108, %109, %110, %111, %112, %113, %114, %115, %116, %117, %118, %119, %120, %121, %122, %123, %124, %125, %126, %127}, [%131];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : CODA_R32(r, 0), CODA_R32(r, 32), CODA_R32(r, 64), CODA_R32(r, 96)
      : "r"(taddr + 0), "r"(taddr + 32), "r"(taddr + 64), "r"(taddr + 96)
      : "memory");
}
__device__ __forceinline__ void tmem_ld64(uint32_t taddr, uint32_t (&r)[64]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%64];\n\t"
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%32, %33, %34, %35, %36, %37, %38, %39, %40, %41, %42, %43, %44, %45, %46, %47, %48, %49, %50, %51, %52, %53, %54, %55, %56, %57, %58, %59, %60, %61, %62, %63}, [%65];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : CODA_R32(r, 0), CODA_R32(r, 32)
      : "r"(taddr + 0), "r"(taddr + 32)
      : "memory");
}
// 32 TMEM columns of one lane per thread, written; tmem_st_wait makes them
// complete.
__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
      CODA_W32(r, 0)
      : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 2^x (approximate to about 2 ulp, denormal results flushed), one
// instruction of the special-function unit.
__device__ __forceinline__ float exp2_sfu(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Packed pairs of fp32 (one instruction for two lanes of arithmetic).
__device__ __forceinline__ uint64_t f2_pack(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void f2_unpack(uint64_t v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t f2_mul(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Keeps the code of a rare, warp-uniform case behind a branch: without it the
// compiler turns the masks of diagonal blocks into selects that every block
// executes.
__device__ __forceinline__ void keep_branch() { asm volatile("" ::: "memory"); }

template <int N>
__device__ __forceinline__ void reg_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void reg_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Zero rows [first, 128) of a 128-row x 128-column bf16 tile held as two
// 128-byte-wide halves of 16 KB, then order the writes before the tensor
// core's reads.  Called by a whole warp.  Rows behind a sequence's end hold
// the next sequence (or whatever lies behind the last one); their products
// carry a zero weight, and 0 * inf must not reach the sum.
__device__ __forceinline__ void zero_tile_rows(uint8_t* tile, int first) {
  const int lane = threadIdx.x & 31;
  for (int r = first + (lane >> 3); r < 128; r += 4) {
    uint4* a = reinterpret_cast<uint4*>(tile + r * 128) + (lane & 7);
    *a = make_uint4(0, 0, 0, 0);
    *reinterpret_cast<uint4*>(reinterpret_cast<uint8_t*>(a) + 16384) = make_uint4(0, 0, 0, 0);
  }
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
  __syncwarp();
}

__device__ __forceinline__ AttnTile load_tile(const AttnTile* p) {
  const int4 a = __ldcg(reinterpret_cast<const int4*>(p));
  const int4 b = __ldcg(reinterpret_cast<const int4*>(p) + 1);
  AttnTile t;
  t.q0 = a.x; t.lq = a.y; t.k0 = a.z; t.lk = a.w;
  t.t0 = b.x; t.seq = b.y; t.slot = b.z; t.block = b.w;
  return t;
}

// Item that CTA `c` of `n` takes in round `k`: odd rounds run backwards, so
// with items sorted longest first every CTA gets about the same total.
__device__ __forceinline__ int snake_item(int c, int n, int k) { return k * n + ((k & 1) ? n - 1 - c : c); }

// Blocks of 128 keys that queries up to `last` (within the sequence) see.
__device__ __forceinline__ int key_blocks(const AttnTile& t, int last) {
  int vis = last + 1 + t.lk - t.lq;
  vis = vis < t.lk ? vis : t.lk;
  return vis <= 0 ? 0 : (vis + ATTN_BLK - 1) / ATTN_BLK;
}

}  // namespace coda

// Device pieces of the 4-bit key/value cache that several kernels share: where a
// row lies, its values, and the quantiser.
#pragma once
#include <cuda_fp16.h>
#include <cuda_fp4.h>
#include <cuda_fp8.h>

#include "coda_kvcache.cuh"
#include "coda_ptx.cuh"

namespace coda {

__device__ __forceinline__ int64_t cache_row(const KvCache& c, int page, int plane, int h, int off) {
  return ((static_cast<int64_t>(page) * 2 + plane) * c.n_kv + h << c.page_shift) + off;
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

// Sixteen elements of a row of 128, eight neighbouring lanes per row: codes
// (w), the block's e4m3 scale and the row's fp32 scale.  Every arithmetic step
// is one fp32 operation, the same steps as quantize_nvfp4_rows, so the codes
// and scales agree with it bit for bit.  All lanes of the warp take part.
__device__ __forceinline__ void quantise_row16(const float (&x)[16], uint32_t (&w)[2], uint32_t& sfb, float& s) {
  float bmax = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) bmax = fmaxf(bmax, fabsf(x[i]));
  float amax = bmax;
#pragma unroll
  for (int o = 4; o; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, o));
  s = amax > 0.f ? __fdiv_rn(amax, 2688.0f) : 1.0f;
  const float sf_f = fminf(__fdiv_rn(bmax, __fmul_rn(6.0f, s)), 448.0f);
  sfb = __nv_cvt_float_to_fp8(sf_f, __NV_SATFINITE, __NV_E4M3);
  const float denom = __fmul_rn(e4m3_f32(sfb), s);
  w[0] = w[1] = 0;
  if (denom > 0.f) {
    const float inv = fminf(__fdiv_rn(1.0f, denom), 3.40282347e38f);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t c2 = __nv_cvt_float2_to_fp4x2(make_float2(__fmul_rn(x[2 * i], inv), __fmul_rn(x[2 * i + 1], inv)),
                                                   __NV_E2M1, cudaRoundNearest);
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
}

}  // namespace coda

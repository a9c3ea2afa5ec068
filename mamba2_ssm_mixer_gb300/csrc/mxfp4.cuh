// Arithmetic of the microscaled 4-bit format that its kernels share (the format
// itself: mxfp4.cu).
#pragma once
#include <cuda_bf16.h>
#include <stdint.h>

namespace m2 {

// 128-value groups of a row.
__host__ __device__ inline int mx_kb(int K) { return (K + 127) / 128; }

// Scale code of a block from its largest |x| (bf16 bits): exponent field less 2,
// 0 at least (subnormals and zeros included), 255 for infinities and NaN.
__device__ __forceinline__ uint32_t scale_code(uint32_t amax) {
  const uint32_t e = amax >> 7;
  return amax >= 0x7F80u ? 255u : e > 2u ? e - 2u : 0u;
}

__device__ __forceinline__ __nv_bfloat162 as_bf16x2(uint32_t v) { return *reinterpret_cast<__nv_bfloat162*>(&v); }
__device__ __forceinline__ uint32_t bits_of(__nv_bfloat162 v) { return *reinterpret_cast<uint32_t*>(&v); }
// The larger magnitudes of two pairs, NaN if there is one.
__device__ __forceinline__ __nv_bfloat162 max_abs(__nv_bfloat162 a, __nv_bfloat162 b) {
  return __hmax2_nan(__habs2(a), __habs2(b));
}
__device__ __forceinline__ __nv_bfloat162 max_abs(const uint4& v) {
  return max_abs(max_abs(as_bf16x2(v.x), as_bf16x2(v.y)), max_abs(as_bf16x2(v.z), as_bf16x2(v.w)));
}

// e2m1 codes of eight bf16 times f (a power of two: exact, but for products
// below bf16's range, whose code is 0 either way).
__device__ __forceinline__ uint32_t quant8(const uint4& v, __nv_bfloat162 f) {
  const uint32_t w[4] = {bits_of(__hmul2(as_bf16x2(v.x), f)), bits_of(__hmul2(as_bf16x2(v.y), f)),
                         bits_of(__hmul2(as_bf16x2(v.z), f)), bits_of(__hmul2(as_bf16x2(v.w), f))};
  uint32_t q;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}\n"
      : "=r"(q)
      : "r"(w[0] << 16), "r"(w[0] & 0xFFFF0000u), "r"(w[1] << 16), "r"(w[1] & 0xFFFF0000u), "r"(w[2] << 16),
        "r"(w[2] & 0xFFFF0000u), "r"(w[3] << 16), "r"(w[3] & 0xFFFF0000u));
  return q;
}

// 2^(127 - code) twice, for code <= 252: the exact factor of x / 2^(code - 127).
__device__ __forceinline__ __nv_bfloat162 inverse_scale(uint32_t code) {
  return as_bf16x2(((254u - code) << 7) * 0x10001u);
}
// A thread's 16 values of a block, whose other half the next or the previous
// lane has: the block's scale code and the values' codes (all lanes of the warp
// together).
__device__ __forceinline__ uint2 quant16(const uint4 (&v)[2], uint32_t* scale) {
  const uint32_t two = bits_of(max_abs(max_abs(v[0]), max_abs(v[1])));
  uint32_t m = max(two & 0xFFFFu, two >> 16);   // (no sign: magnitudes order like their bits)
  m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
  const uint32_t code = scale_code(m);
  *scale = code;
  if (code == 255u) return make_uint2(0u, 0u);
  const __nv_bfloat162 f = inverse_scale(code);
  return make_uint2(quant8(v[0], f), quant8(v[1], f));
}

}  // namespace m2

// Microscaled 4-bit floating point (OCP MX, MXFP4): blocks of 32 values along K
// share one power-of-two scale, elements are e2m1 (1 sign, 2 exponent and 1
// mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6).  For a block with largest
// magnitude a,
//   e = max(floor(log2 a) - 2, -127),  scale code e + 127,
//   code_k = e2m1(x_k / 2^e), nearest even, 6 past the end;
// a block with an infinity or a NaN gets scale code 255 (NaN) and zero codes.
// x / 2^e is exact in f32, so the codes are bit-exact.
//
// Codes are row-major, two to a byte, the even k in the low half.  Scales are
// laid out in the order in which the tensor cores take them from shared
// memory: tiles of 128 rows x 4 blocks (128 values of K), 512 bytes, byte
// (r % 32) 16 + (r / 32) 4 + b of a tile for row r and block b; tiles
// [ceil(rows / 128)][ceil(K / 128)], zero past the rows and past K.
#include <cuda_fp4.h>

#include "launch_util.h"
#include "m2_kernels.h"

namespace m2 {

namespace {

constexpr int kMxThreads = 256;
constexpr int kMxUnroll = 4;

__host__ __device__ inline int mx_kb(int K) { return (K + 127) / 128; }
// Bytes offset of the four scale codes of row r's 128-value group kb.
__device__ __forceinline__ size_t scale_word(int r, int kb, int KB) {
  return ((size_t)(r >> 7) * KB + kb) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4;
}

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) { return __vmaxu2(a, b); }

// Scale code of a block from the largest |x| bits (bf16): exponent field less
// 2, 0 at least (subnormals and zeros included), 255 for infinities and NaN.
__device__ __forceinline__ uint32_t scale_code(uint32_t amax) {
  const uint32_t e = amax >> 7;
  return amax >= 0x7F80u ? 255u : e > 2u ? e - 2u : 0u;
}

// e2m1 codes of two floats, a in the low half of the byte.
__device__ __forceinline__ uint32_t e2m1x2(float a, float b) {
  return (uint32_t)__nv_cvt_float2_to_fp4x2(make_float2(a, b), __NV_E2M1, cudaRoundNearest);
}

// 2^(127 - code) for code <= 254: the exact factor of x / 2^(code - 127).
__device__ __forceinline__ float inverse_scale(uint32_t code) { return __uint_as_float((254u - code) << 23); }
// 2^(code - 127), NaN for 255.
__device__ __forceinline__ float scale_value(uint32_t code) {
  return __uint_as_float(code == 255u ? 0x7FC00000u : code ? code << 23 : 0x00400000u);
}

__device__ __forceinline__ uint32_t quant8(const uint4& v, uint32_t code) {
  if (code == 255u) return 0u;
  const float f = inverse_scale(code);
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t q = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    q |= e2m1x2(__uint_as_float(w[i] << 16) * f, __uint_as_float(w[i] & 0xFFFF0000u) * f) << (8 * i);
  return q;
}

}  // namespace

// A half-warp takes 128 values of one row (16 lanes x 8 values: 256 bytes in,
// 64 bytes of codes and one word of four scale codes out), kMxUnroll of them
// with their loads under way together.
__global__ void __launch_bounds__(kMxThreads) k_mx_quant(const uint16_t* __restrict__ x, size_t stride, int rows, int K,
                                                         int rows_pad, uint8_t* __restrict__ codes,
                                                         uint8_t* __restrict__ scales) {
  pdl_wait();
  pdl_trigger();
  const int KB = mx_kb(K), lane16 = threadIdx.x & 15;
  const uint32_t units = (uint32_t)rows_pad * (uint32_t)KB;   // (below 2^32: rows K <= 2^38)
  const uint32_t u0 = blockIdx.x * (kMxUnroll * kMxThreads / 16) + threadIdx.x / 16;
  uint4 v[kMxUnroll];
  int row[kMxUnroll], kb[kMxUnroll];
#pragma unroll
  for (int i = 0; i < kMxUnroll; ++i) {
    const uint32_t u = u0 + i * (kMxThreads / 16);
    row[i] = u < units ? (int)(u / (uint32_t)KB) : rows_pad;
    kb[i] = (int)(u % (uint32_t)KB);
    v[i] = make_uint4(0u, 0u, 0u, 0u);
    if (row[i] < rows && kb[i] * 128 + lane16 * 8 < K)
      v[i] = *reinterpret_cast<const uint4*>(x + (size_t)row[i] * stride + kb[i] * 128 + lane16 * 8);
  }
#pragma unroll
  for (int i = 0; i < kMxUnroll; ++i) {
    // the block's largest |x| as bf16 bits, over four lanes
    uint32_t m = max_u16x2(max_u16x2(v[i].x & 0x7FFF7FFFu, v[i].y & 0x7FFF7FFFu),
                           max_u16x2(v[i].z & 0x7FFF7FFFu, v[i].w & 0x7FFF7FFFu));
    m = max(m & 0xFFFFu, m >> 16);
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 1));
    m = max(m, __shfl_xor_sync(0xffffffffu, m, 2));
    const uint32_t code = scale_code(m);
    uint32_t word = code << (8 * (lane16 >> 2));
    word |= __shfl_xor_sync(0xffffffffu, word, 4);
    word |= __shfl_xor_sync(0xffffffffu, word, 8);
    if (row[i] >= rows_pad) continue;
    if (lane16 == 0) *reinterpret_cast<uint32_t*>(scales + scale_word(row[i], kb[i], KB)) = word;
    if (row[i] < rows && kb[i] * 128 + lane16 * 8 < K)
      *reinterpret_cast<uint32_t*>(codes + ((size_t)row[i] * K + kb[i] * 128 + lane16 * 8) / 2) = quant8(v[i], code);
  }
}

// The reverse: bf16(e2m1 x 2^(code - 127)), exact except for scale codes that
// pass bf16's range (254 with magnitude 4 and 6: infinity).
__global__ void __launch_bounds__(kMxThreads) k_mx_dequant(const uint8_t* __restrict__ codes,
                                                           const uint8_t* __restrict__ scales, int rows, int K,
                                                           uint16_t* __restrict__ out) {
  pdl_wait();
  pdl_trigger();
  const int KB = mx_kb(K), lane16 = threadIdx.x & 15;
  const uint32_t units = (uint32_t)rows * (uint32_t)KB;
  const uint32_t u0 = blockIdx.x * (kMxUnroll * kMxThreads / 16) + threadIdx.x / 16;
  uint32_t q[kMxUnroll], s[kMxUnroll];
  size_t at[kMxUnroll];
#pragma unroll
  for (int i = 0; i < kMxUnroll; ++i) {
    const uint32_t u = u0 + i * (kMxThreads / 16);
    const int row = (int)(u / (uint32_t)KB), kb = (int)(u % (uint32_t)KB), k = kb * 128 + lane16 * 8;
    const bool in = u < units && k < K;
    at[i] = in ? (size_t)row * K + k : ~(size_t)0;
    q[i] = in ? *reinterpret_cast<const uint32_t*>(codes + at[i] / 2) : 0u;
    s[i] = in ? scales[scale_word(row, kb, KB) + (lane16 >> 2)] : 0u;
  }
#pragma unroll
  for (int i = 0; i < kMxUnroll; ++i) {
    if (at[i] == ~(size_t)0) continue;
    const float f = scale_value(s[i]);
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float e[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint32_t c = q[i] >> (8 * j + 4 * h);
        // exponent field 0 is 0 or 0.5; else (1 + m / 2) 2^(field - 1)
        const uint32_t mag = c & 7u;
        const float v = mag < 2u ? 0.5f * (float)mag : __uint_as_float((126u + (mag >> 1)) << 23 | (mag & 1u) << 22);
        e[h] = __uint_as_float(__float_as_uint(v) | (c & 8u) << 28) * f;
      }
      o[j] = pack_bf16x2(e[0], e[1]);
    }
    *reinterpret_cast<uint4*>(out + at[i]) = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

// Row-major scale codes [rows, K / 32] to tiles; one word (four blocks of a
// row) per thread.
__global__ void __launch_bounds__(kMxThreads) k_mx_pack(const uint8_t* __restrict__ s, int rows, int K, int rows_pad,
                                                        uint8_t* __restrict__ tiles) {
  pdl_wait();
  pdl_trigger();
  const int KB = mx_kb(K), blocks = K / 32;
  const size_t n = (size_t)rows_pad * KB;
  for (size_t i = (size_t)blockIdx.x * kMxThreads + threadIdx.x; i < n; i += (size_t)gridDim.x * kMxThreads) {
    // consecutive threads write consecutive words: (r % 32, r / 32 % 4) fastest
    const size_t tile = i / 128;
    const int w = (int)(i % 128), kb = (int)(tile % KB);
    const int r = (int)(tile / KB) * 128 + (w & 3) * 32 + (w >> 2);
    uint32_t word = 0;
    if (r < rows)
      for (int j = 0; j < 4 && kb * 4 + j < blocks; ++j)
        word |= (uint32_t)s[(size_t)r * blocks + kb * 4 + j] << (8 * j);
    reinterpret_cast<uint32_t*>(tiles)[i] = word;
  }
}

size_t mx_scale_bytes(int rows, int K) { return (size_t)((rows + 127) / 128) * mx_kb(K) * 512; }

cudaError_t launch_mx_quant(const uint16_t* x, size_t stride, int rows, int K, uint8_t* codes, uint8_t* scales,
                            cudaStream_t st) {
  if (rows == 0) return cudaSuccess;
  const int rows_pad = (rows + 127) / 128 * 128;
  const size_t units = (size_t)rows_pad * mx_kb(K), per = (size_t)kMxUnroll * kMxThreads / 16;
  return launch_pdl(k_mx_quant, dim3((unsigned)((units + per - 1) / per)), dim3(kMxThreads), 0, st, x, stride, rows, K,
                    rows_pad, codes, scales);
}

cudaError_t launch_mx_dequant(const uint8_t* codes, const uint8_t* scales, int rows, int K, uint16_t* out,
                              cudaStream_t st) {
  if (rows == 0) return cudaSuccess;
  const size_t units = (size_t)rows * mx_kb(K), per = (size_t)kMxUnroll * kMxThreads / 16;
  return launch_pdl(k_mx_dequant, dim3((unsigned)((units + per - 1) / per)), dim3(kMxThreads), 0, st, codes, scales, rows,
                    K, out);
}

cudaError_t launch_mx_pack(const uint8_t* scales, int rows, int K, uint8_t* tiles, cudaStream_t st) {
  if (rows == 0) return cudaSuccess;
  const int rows_pad = (rows + 127) / 128 * 128;
  size_t blocks = ((size_t)rows_pad * mx_kb(K) + kMxThreads - 1) / kMxThreads;
  const size_t cap = (size_t)16 * device_sm_count();
  if (blocks > cap) blocks = cap;
  return launch_pdl(k_mx_pack, dim3((unsigned)blocks), dim3(kMxThreads), 0, st, scales, rows, K, rows_pad, tiles);
}

}  // namespace m2

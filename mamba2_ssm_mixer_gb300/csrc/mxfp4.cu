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
#include "launch_util.h"
#include "m2_kernels.h"
#include "mxfp4.cuh"

namespace m2 {

namespace {

constexpr int kMxThreads = 256;
constexpr int kMxUnroll = 2;

// Bytes offset of the four scale codes of row r's 128-value group kb.
__device__ __forceinline__ size_t scale_word(int r, int kb, int KB) {
  return ((size_t)(r >> 7) * KB + kb) * 512 + (r & 31) * 16 + ((r >> 5) & 3) * 4;
}

// bf16 values of eight e2m1 codes times f.  A magnitude's two bytes come from
// tables of eight, picked by the code's nibble.
__device__ __forceinline__ uint4 dequant8(uint32_t q, __nv_bfloat162 f) {
  uint32_t o[4];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t c = q >> (16 * h), sel = c & 0x7777u;
    const uint32_t hi = __byte_perm(0x3F3F3F00u, 0x40404040u, sel);   // 0, 0.5, 1, 1.5 | 2, 3, 4, 6
    const uint32_t lo = __byte_perm(0xC0800000u, 0xC0804000u, sel);
    const uint32_t s0 = ((c << 12) & 0x8000u) | ((c << 24) & 0x80000000u);
    const uint32_t s1 = ((c << 4) & 0x8000u) | ((c << 16) & 0x80000000u);
    o[2 * h] = bits_of(__hmul2(as_bf16x2(__byte_perm(lo, hi, 0x5140) | s0), f));
    o[2 * h + 1] = bits_of(__hmul2(as_bf16x2(__byte_perm(lo, hi, 0x7362) | s1), f));
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}

// 2^(code - 127) twice, NaN for 255.
__device__ __forceinline__ __nv_bfloat162 scale_value(uint32_t code) {
  return as_bf16x2((code == 255u ? 0x7FC0u : code ? code << 7 : 0x0040u) * 0x10001u);
}

// A unit is 128 values of one row, taken by 8 lanes of 16 values; a thread has
// kMxUnroll of them, kMxThreads / 8 units apart, under way together.  The
// first one's place takes a division, the others steps.
struct Units {
  int row, kb, KB, dr, dk;
  __device__ Units(int K) : KB(mx_kb(K)) {
    const uint32_t u = blockIdx.x * (kMxUnroll * kMxThreads / 8) + threadIdx.x / 8;   // (below 2^32: rows K <= 2^38)
    row = (int)(u / (uint32_t)KB);
    kb = (int)(u % (uint32_t)KB);
    dr = (kMxThreads / 8) / KB;
    dk = (kMxThreads / 8) % KB;
  }
  __device__ void step() {
    row += dr;
    kb += dk;
    if (kb >= KB) kb -= KB, ++row;
  }
};

}  // namespace

// 16 values of a thread are 32 bytes in and 8 bytes of codes out; a block's
// largest magnitude takes one exchange, a unit's word of scale codes two.
// Bound by the instructions: with 8 values a thread, an index division per 8
// and f32 products 8192 x 2688 took 15.3 us.
__global__ void __launch_bounds__(kMxThreads) k_mx_quant(const uint16_t* __restrict__ x, size_t stride, int rows, int K,
                                                         int rows_pad, uint8_t* __restrict__ codes,
                                                         uint8_t* __restrict__ scales) {
  pdl_wait();
  pdl_trigger();
  const int lane8 = threadIdx.x & 7;
  uint4 v[kMxUnroll][2];
  Units at(K);
#pragma unroll
  for (int i = 0; i < kMxUnroll; ++i, at.step()) {
    const int k = at.kb * 128 + lane8 * 16;
    const bool in = at.row < rows && k < K;
    const uint4* p = reinterpret_cast<const uint4*>(x + (size_t)at.row * stride + k);
    v[i][0] = in ? __ldg(p) : make_uint4(0u, 0u, 0u, 0u);
    v[i][1] = in ? __ldg(p + 1) : make_uint4(0u, 0u, 0u, 0u);
  }
  at = Units(K);
#pragma unroll
  for (int i = 0; i < kMxUnroll; ++i, at.step()) {
    uint32_t code;
    const uint2 q = quant16(v[i], &code);
    uint32_t word = code << (8 * (lane8 >> 1));
    word |= __shfl_xor_sync(0xffffffffu, word, 2);
    word |= __shfl_xor_sync(0xffffffffu, word, 4);
    if (lane8 == 0 && at.row < rows_pad)
      *reinterpret_cast<uint32_t*>(scales + scale_word(at.row, at.kb, at.KB)) = word;
    const int k = at.kb * 128 + lane8 * 16;
    if (at.row < rows && k < K) *reinterpret_cast<uint2*>(codes + ((size_t)at.row * K + k) / 2) = q;
  }
}

// The reverse: bf16(e2m1 x 2^(code - 127)), exact except for scale codes that
// pass bf16's range (254 with magnitude 4 and 6: infinity).
__global__ void __launch_bounds__(kMxThreads) k_mx_dequant(const uint8_t* __restrict__ codes,
                                                           const uint8_t* __restrict__ scales, int rows, int K,
                                                           uint16_t* __restrict__ out) {
  pdl_wait();
  pdl_trigger();
  const int lane8 = threadIdx.x & 7;
  uint2 q[kMxUnroll];
  uint32_t s[kMxUnroll];
  Units at(K);
#pragma unroll
  for (int i = 0; i < kMxUnroll; ++i, at.step()) {
    const int k = at.kb * 128 + lane8 * 16;
    const bool in = at.row < rows && k < K;
    q[i] = in ? __ldg(reinterpret_cast<const uint2*>(codes + ((size_t)at.row * K + k) / 2)) : make_uint2(0u, 0u);
    s[i] = in ? __ldg(scales + scale_word(at.row, at.kb, at.KB) + (lane8 >> 1)) : 0u;
  }
  at = Units(K);
#pragma unroll
  for (int i = 0; i < kMxUnroll; ++i, at.step()) {
    const int k = at.kb * 128 + lane8 * 16;
    if (at.row < rows && k < K) {
      const __nv_bfloat162 f = scale_value(s[i]);
      uint4* o = reinterpret_cast<uint4*>(out + (size_t)at.row * K + k);
      o[0] = dequant8(q[i].x, f);
      o[1] = dequant8(q[i].y, f);
    }
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
  const size_t units = (size_t)rows_pad * mx_kb(K), per = (size_t)kMxUnroll * kMxThreads / 8;
  return launch_pdl(k_mx_quant, dim3((unsigned)((units + per - 1) / per)), dim3(kMxThreads), 0, st, x, stride, rows, K,
                    rows_pad, codes, scales);
}

cudaError_t launch_mx_dequant(const uint8_t* codes, const uint8_t* scales, int rows, int K, uint16_t* out,
                              cudaStream_t st) {
  if (rows == 0) return cudaSuccess;
  const size_t units = (size_t)rows * mx_kb(K), per = (size_t)kMxUnroll * kMxThreads / 8;
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

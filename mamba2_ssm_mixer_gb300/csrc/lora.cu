// Low-rank adapters of many requests beside a shared projection: row m of a
// batch names adapter a = row_adapter[m] (or none, -1) and
//   out[m] = bf16( y[m] + s_a B_a (A_a x[m]) ),     A_a [rank, K], B_a [N, rank]
// with y the shared projection's bf16 rows.  A_a x and the sum over the rank
// are held in f32; out is rounded once.
#include "launch_util.h"
#include "m2_kernels.h"

namespace m2 {

namespace {
constexpr int kLoThreads = 256;
}

// t[m][j] = A_a[j] . x[m]: one warp per (row, rank index).
__global__ void __launch_bounds__(kLoThreads) k_lora_down(const uint16_t* __restrict__ x, const uint16_t* __restrict__ a,
                                                          const int32_t* __restrict__ ids, int n_adapters, int rank,
                                                          int M, int K, float* __restrict__ t, int* err) {
  pdl_wait();
  pdl_trigger();
  const size_t w = ((size_t)blockIdx.x * kLoThreads + threadIdx.x) >> 5;
  const int lane = threadIdx.x & 31;
  if (w >= (size_t)M * rank) return;
  const int m = (int)(w / rank), j = (int)(w % rank);
  const int id = ids[m];
  if (id < -1 || id >= n_adapters) {
    if (lane == 0 && j == 0) atomicOr(err, kErrAdapter);
    return;
  }
  if (id < 0) return;
  const uint4* xp = reinterpret_cast<const uint4*>(x + (size_t)m * K);
  const uint4* ap = reinterpret_cast<const uint4*>(a + ((size_t)id * rank + j) * K);
  float acc = 0.f;
  for (int v = lane; v < K / 8; v += 32) {
    const uint4 xv = xp[v], av = ap[v];
    const uint32_t xb[4] = {xv.x, xv.y, xv.z, xv.w}, ab[4] = {av.x, av.y, av.z, av.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      acc = fmaf(__uint_as_float(xb[e] << 16), __uint_as_float(ab[e] << 16), acc);
      acc = fmaf(__uint_as_float(xb[e] & 0xFFFF0000u), __uint_as_float(ab[e] & 0xFFFF0000u), acc);
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, o);
  if (lane == 0) t[w] = acc;
}

// out[m][n] = bf16(y[m][n] + s_a sum_j t[m][j] B_a[n][j]): one thread per element.
__global__ void __launch_bounds__(kLoThreads) k_lora_up(const uint16_t* y, const float* __restrict__ t,
                                                        const uint16_t* __restrict__ b, const float* __restrict__ scale,
                                                        const int32_t* __restrict__ ids, int n_adapters, int rank, int N,
                                                        uint16_t* out) {
  pdl_wait();
  pdl_trigger();
  const int m = blockIdx.x, n = blockIdx.y * kLoThreads + threadIdx.x;
  if (n >= N) return;
  const int id = ids[m];
  const size_t at = (size_t)m * N + n;
  if (id < 0 || id >= n_adapters) {
    if (out != y) out[at] = y[at];
    return;
  }
  const uint4* bp = reinterpret_cast<const uint4*>(b + ((size_t)id * N + n) * rank);
  const float* tp = t + (size_t)m * rank;
  float acc = 0.f;
  for (int v = 0; v < rank / 8; ++v) {
    const uint4 bv = bp[v];
    const uint32_t bb[4] = {bv.x, bv.y, bv.z, bv.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      acc = fmaf(tp[8 * v + 2 * e], __uint_as_float(bb[e] << 16), acc);
      acc = fmaf(tp[8 * v + 2 * e + 1], __uint_as_float(bb[e] & 0xFFFF0000u), acc);
    }
  }
  out[at] = f2bfbits(fmaf(scale ? scale[id] : 1.f, acc, bfbits2f(y[at])));
}

size_t lora_workspace_bytes(int M, int N, int K, int rank, int n_adapters) {
  (void)N, (void)K, (void)n_adapters;
  return (size_t)M * rank * 4;
}

cudaError_t launch_lora_add(const uint16_t* y, const uint16_t* x, const LoraWeights& w, const int32_t* ids, uint16_t* out,
                            int M, int N, int K, void* ws, int* err, cudaStream_t st, int* launches) {
  if (M == 0) return cudaSuccess;
  float* t = static_cast<float*>(ws);
  const unsigned blocks = (unsigned)(((size_t)M * w.rank * 32 + kLoThreads - 1) / kLoThreads);
  cudaError_t e = launch_pdl(k_lora_down, dim3(blocks), dim3(kLoThreads), 0, st, x, w.a, ids, w.n_adapters, w.rank, M, K,
                             t, err);
  if (e != cudaSuccess) return e;
  *launches = 2;
  return launch_pdl(k_lora_up, dim3(M, (N + kLoThreads - 1) / kLoThreads), dim3(kLoThreads), 0, st, y, t, w.b, w.scale,
                    ids, w.n_adapters, w.rank, N, out);
}

// Adapter of every row of a packed call: the decode rows' own, then each
// sequence's for all of its tokens.
__global__ void __launch_bounds__(kLoThreads) k_lora_row_ids(const int32_t* __restrict__ dec_ids, int Bt,
                                                             const SeqInfo si, const SeqAdapters sa,
                                                             int32_t* __restrict__ ids) {
  pdl_wait();
  pdl_trigger();
  const int r = blockIdx.x * kLoThreads + threadIdx.x;
  if (r < Bt)
    ids[r] = dec_ids[r];
  else if (r < Bt + si.total_tokens)
    ids[r] = sa.id[seq_of_token(si, r - Bt)];
}

cudaError_t launch_lora_row_ids(const int32_t* dec_ids, int Bt, const SeqInfo& si, const SeqAdapters& sa, int32_t* ids,
                                cudaStream_t st) {
  const int rows = Bt + si.total_tokens;
  return launch_pdl(k_lora_row_ids, dim3((rows + kLoThreads - 1) / kLoThreads), dim3(kLoThreads), 0, st, dec_ids, Bt, si,
                    sa, ids);
}

}  // namespace m2

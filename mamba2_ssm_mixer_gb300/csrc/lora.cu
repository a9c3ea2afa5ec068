// Low-rank adapters of many requests beside a shared projection: row m of a
// batch names adapter a = row_adapter[m] (or none, -1) and
//   out[m] = bf16( y[m] + s_a B_a t ),   t = A_a x[m],   A_a [rank, K], B_a [N, rank]
// with y the shared projection's bf16 rows.  At these ranks the products are
// small change (2 rank (K + N) operations per row); what bounds the call is
// reading y and writing out once, or, in a decode batch, reading each named
// adapter once.  Two forms:
//  - few rows (see few_rows): one kernel, one 4-CTA cluster per (up to kUnit rows
//    of one adapter, slice of N).  Which rows share an adapter is found by
//    each cluster itself from the batch's ids (a ballot), so there is no
//    sorting launch and no workspace, and a shared adapter is read once per
//    kUnit rows.
//  - more rows: k_lora_group deals the rows out to tiles of 64 of one adapter
//    (while the next kernel's CTAs bring x to L2), k_lora_down forms t on the
//    tensor cores, K split over a cluster, and k_lora_up streams y past B t;
//    or, up to rank 32 and a middling batch, k_lora_tile does both.
// t is summed in f32 and enters the second product as two bf16 parts, 2^-16 of
// it in all (an f32 operand would keep 2^-24; out keeps 2^-9 of the sum): the
// 16-bit tensor rate, at twice the operations.  mma.sync: up to rank 32 the tensor work hides behind
// the stream of y (8192 rows, 2688 -> 10304: rank 16 70 us, floor 57; rank 32
// 77); at rank 64 and 128 its two passes show (98 and 200).
#include <algorithm>
#include <type_traits>

#include "launch_util.h"
#include "m2_kernels.h"
#include "tc_ptx.cuh"

namespace m2 {

using tc::smem_u32;

namespace {

constexpr int kLoThreads = 256;
constexpr int kLoWarps = kLoThreads / 32;

__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// a, b as two bf16 pairs: their first 8 bits and the remainder, 2^-16 of them
// in all.  Cut, not rounded, and with the least normal value for a remainder
// of 0, so that the parts of what is not 0 have one sign and neither is 0: an
// infinite weight then makes the same infinity of both, as the formula does
// (0 x inf or inf - inf would be NaN).  2^-126 of a weight is past the last
// digit of the first part's product, and of no account where that is not.
__device__ __forceinline__ void split_bf16x2(float a, float b, uint32_t* hi, uint32_t* lo) {
  const uint32_t h = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
  // (an infinite value has no remainder, a NaN is one in both parts)
  const uint32_t r = pack_bf16x2(isinf(a) ? 0.f : a - lo_f(h), isinf(b) ? 0.f : b - hi_f(h));
  const uint32_t la = (r & 0x7FFFu) || !(h & 0x7FFFu) ? 0u : (h & 0x8000u) | 0x0080u;
  const uint32_t lb = (r & 0x7FFF0000u) || !(h & 0x7FFF0000u) ? 0u : (h & 0x80000000u) | 0x00800000u;
  *hi = h;
  *lo = r | la | lb;
}

__device__ __forceinline__ uint32_t lo_cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void lo_cluster_arrive() { asm volatile("barrier.cluster.arrive.aligned;" ::: "memory"); }
__device__ __forceinline__ void lo_cluster_wait() { asm volatile("barrier.cluster.wait.aligned;" ::: "memory"); }
// Another CTA's copy of this CTA's shared float.
__device__ __forceinline__ float ld_cluster_f32(uint32_t addr, uint32_t rank) {
  float v;
  asm volatile(
      "{\n\t.reg .b32 ra;\n\t"
      "mapa.shared::cluster.u32 ra, %1, %2;\n\t"
      "ld.shared::cluster.f32 %0, [ra];\n\t}"
      : "=f"(v)
      : "r"(addr), "r"(rank)
      : "memory");
  return v;
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// y's 8 columns, as words of MMAs 0 to 3, plus accumulator row h (0, or 1: + 8)
__device__ __forceinline__ void add_pairs(uint4* y, const float (&acc)[4][4], int h) {
  y->x = pack_bf16x2(lo_f(y->x) + acc[0][2 * h], hi_f(y->x) + acc[0][2 * h + 1]);
  y->y = pack_bf16x2(lo_f(y->y) + acc[1][2 * h], hi_f(y->y) + acc[1][2 * h + 1]);
  y->z = pack_bf16x2(lo_f(y->z) + acc[2][2 * h], hi_f(y->z) + acc[2][2 * h + 1]);
  y->w = pack_bf16x2(lo_f(y->w) + acc[3][2 * h], hi_f(y->w) + acc[3][2 * h + 1]);
}
__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

}  // namespace

// ---------------------------------------------------------------------------
// Few rows.  Grid (4 x slices of N, M), clusters of 4 along x; the
// cluster of row m goes on if m is the first of a run of 8 among the rows of
// its adapter in its window of 256 rows (a ballot in every warp, no barrier).
// Both products put the adapter's matrix on the 16-wide side of m16n8k16 and
// the rows (up to 8) on the other, and take their operands straight from
// global memory: the order of the summed index inside an MMA is free, so each
// lane loads whole 8- or 16-byte pieces.  A x: K in 32-wide blocks over the
// cluster's 32 warps, the parts summed in shared memory, then over the CTAs'
// shared memories.  B t: 16 columns per warp and step, the first steps' B and
// y on their way before t is known.
// A decode batch is bound by reading each adapter once and, more, by latency
// (ids, operands, the cluster's sum, the columns: each a trip).  Adapters of
// rank 16, 2688 -> 10304: 1 to 8 rows 4.6 us, 64 rows with 64 adapters 10.9
// (floor 4.4); a form on FMA units, with ten times the instructions for
// unpacking, took 16.8 for those, clusters of 8 and of 2 13.2 and 11.3, 32
// columns per step 10.7 (but 0.7 more at rank 64), bringing B's slice to L2
// ahead 0.3 to 1.2 more.
// ---------------------------------------------------------------------------
namespace {
constexpr int kFewRows = 320, kFewMost = 1024;   // see few_rows
constexpr int kWindow = 256;
constexpr int kFewCluster = 4;
constexpr int kUnit = 8;   // rows that share the reads of an adapter
}  // namespace

// NT: rank / 16 rounded up to a power of two.  kPair: y and out move two
// columns at a time (N even, 4-byte aligned).
template <int NT, bool kPair>
__global__ void __launch_bounds__(kLoThreads, NT <= 4 ? 2 : 1) k_lora_few(
    const uint16_t* y, const uint16_t* __restrict__ x, const uint16_t* __restrict__ a, const uint16_t* __restrict__ b,
    const float* __restrict__ scale, const int32_t* __restrict__ ids, int n_adapters, int rank, uint16_t* out, int M,
    int N, int K, int* err) {
  constexpr int kAheadF = NT == 1 ? 8 : NT == 2 ? 4 : 1;   // steps of B and y under way
  __shared__ int rows_s[kUnit];
  __shared__ __align__(16) float red[kLoWarps][NT * 128];
  __shared__ float part[NT * 128];
  __shared__ __align__(16) uint16_t t_s[2][kUnit][NT * 16 + 8];   // t's two bf16 parts
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, g = lane >> 2, q = lane & 3;
  const int crank = (int)lo_cluster_rank();
  const int m = blockIdx.y;
  const int cols16 = (N + 15) / 16;
  const int n_lo = 16 * (int)((long long)cols16 * blockIdx.x / gridDim.x);
  const int n_hi = min(N, 16 * (int)((long long)cols16 * (blockIdx.x + 1) / gridDim.x));
  pdl_wait();
  pdl_trigger();
  const int id = ids[m], w0 = m - m % kWindow;
  int other[kWindow / 32];
#pragma unroll
  for (int i = 0; i < kWindow / 32; ++i) other[i] = w0 + 32 * i + lane < M ? ids[w0 + 32 * i + lane] : -1;
  if (id < 0 || id >= n_adapters) {   // the same for the whole cluster
    if (id != -1 && blockIdx.x == 0 && tid == 0) atomicOr(err, kErrAdapter);
    if (out != y) {   // (loads ahead of the stores: y and out may be one buffer for all the compiler knows)
      constexpr int kCopies = 4;
      using E = typename std::conditional<kPair, uint32_t, uint16_t>::type;
      constexpr int kE = sizeof(E) / 2;
      const E* from = reinterpret_cast<const E*>(y + (size_t)m * N);
      E* to = reinterpret_cast<E*>(out + (size_t)m * N);
      for (int n0 = n_lo / kE + tid; n0 < n_hi / kE; n0 += kCopies * kLoThreads) {
        E v[kCopies];
#pragma unroll
        for (int i = 0; i < kCopies; ++i) v[i] = from[min(n0 + i * kLoThreads, n_hi / kE - 1)];
#pragma unroll
        for (int i = 0; i < kCopies; ++i)
          if (n0 + i * kLoThreads < n_hi / kE) to[n0 + i * kLoThreads] = v[i];
      }
    }
    return;
  }
  uint32_t same[kWindow / 32];
  int before = 0;   // rows of this adapter in the window before m
#pragma unroll
  for (int i = 0; i < kWindow / 32; ++i) {
    same[i] = __ballot_sync(0xffffffffu, other[i] == id);
    const int k = m - w0 - 32 * i;
    before += __popc(same[i] & (k >= 32 ? 0xffffffffu : k > 0 ? (1u << k) - 1u : 0u));
  }
  if (before % kUnit) return;   // an earlier row's cluster takes this row along
  if (warp == 0) {   // the unit's rows: places `before` .. of the adapter's
    if (lane < kUnit) rows_s[lane] = -1;
    __syncwarp();
    int base = 0;
#pragma unroll
    for (int i = 0; i < kWindow / 32; ++i) {
      const int place = base + __popc(same[i] & ((1u << lane) - 1u)) - before;
      if (((same[i] >> lane) & 1u) && place >= 0 && place < kUnit) rows_s[place] = w0 + 32 * i + lane;
      base += __popc(same[i]);
    }
  }
  __syncthreads();
  const int xrow = rows_s[g], row0 = rows_s[2 * q], row1 = rows_s[2 * q + 1];

  // the first steps of B and y: step i of this warp holds columns n, n + 1
  const uint16_t* bp = b + (size_t)id * N * rank + 4 * q;
  uint2 bv[kAheadF][NT][2];
  uint32_t yv[kAheadF][2];
  // (loads are unconditional, from a valid place instead where there is none:
  // a condition around them costs the overlap)
  const size_t ybase0 = (size_t)(row0 < 0 ? m : row0) * N, ybase1 = (size_t)(row1 < 0 ? m : row1) * N;
  auto fetch = [&](int u, int n) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint16_t* bn = bp + (size_t)(n + h < n_hi ? n + h : n_lo) * rank;
#pragma unroll
      for (int s = 0; s < NT; ++s) {
        const bool in = 16 * s + 4 * q < rank;
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(bn + (in ? 16 * s : -4 * q)));
        bv[u][s][h] = in ? v : make_uint2(0u, 0u);
      }
    }
    const int nc = n < n_hi ? n : n_lo;
    if constexpr (kPair) {
      yv[u][0] = *reinterpret_cast<const uint32_t*>(y + ybase0 + nc);
      yv[u][1] = *reinterpret_cast<const uint32_t*>(y + ybase1 + nc);
    } else {
      const int nd = nc + 1 < n_hi ? nc + 1 : nc;
      yv[u][0] = (uint32_t)y[ybase0 + nc] | ((uint32_t)y[ybase0 + nd] << 16);
      yv[u][1] = (uint32_t)y[ybase1 + nc] | ((uint32_t)y[ybase1 + nd] << 16);
    }
  };
  const int n_first = n_lo + warp * 16 + 2 * g;
#pragma unroll
  for (int u = 0; u < kAheadF; ++u) fetch(u, n_first + u * (16 * kLoWarps));

  // t = A x: 32-wide K blocks over the cluster's warps
  float acc[NT][4];
#pragma unroll
  for (int i = 0; i < NT; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
  const uint16_t* ap = a + ((size_t)id * rank + g) * K;
  const uint16_t* xp = x + (size_t)(xrow < 0 ? m : xrow) * K;
  constexpr int kStep = kFewCluster * kLoWarps, kBlocks = NT == 1 ? 4 : NT == 2 ? 2 : 1;
  for (int kb = crank * kLoWarps + warp; kb * 32 < K; kb += kBlocks * kStep) {
    uint4 xv[kBlocks], av[kBlocks][2 * NT];
    bool in[kBlocks];
#pragma unroll
    for (int u = 0; u < kBlocks; ++u) {
      const int k = (kb + u * kStep) * 32 + 8 * q;
      in[u] = k < K;
      const int o = in[u] ? k : 0;
      xv[u] = __ldg(reinterpret_cast<const uint4*>(xp + o));
#pragma unroll
      for (int i = 0; i < 2 * NT; ++i)
        av[u][i] = __ldg(reinterpret_cast<const uint4*>(ap + (size_t)(8 * i < rank ? 8 * i : 0) * K + o));
    }
#pragma unroll
    for (int u = 0; u < kBlocks; ++u) {
      if (!in[u]) {   // past K: zeros on both sides
        xv[u] = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int i = 0; i < 2 * NT; ++i) av[u][i] = make_uint4(0u, 0u, 0u, 0u);
      }
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const uint4 a0 = av[u][2 * i], a1 = av[u][2 * i + 1];
        mma16816(acc[i], {a0.x, a1.x, a0.y, a1.y}, xv[u].x, xv[u].y);
        mma16816(acc[i], {a0.z, a1.z, a0.w, a1.w}, xv[u].z, xv[u].w);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NT; ++i)
    *reinterpret_cast<float4*>(&red[warp][i * 128 + lane * 4]) = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
  __syncthreads();
  for (int i = tid; i < NT * 128; i += kLoThreads) {
    float t = red[0][i];
#pragma unroll
    for (int w = 1; w < kLoWarps; ++w) t += red[w][i];
    part[i] = t;
  }
  const float sc = scale ? scale[id] : 1.f;
  lo_cluster_arrive();
  lo_cluster_wait();
  for (int i = tid; i < NT * 128; i += kLoThreads) {
    float v[kFewCluster];
#pragma unroll
    for (int r = 0; r < kFewCluster; ++r) v[r] = ld_cluster_f32(smem_u32(&part[i]), (uint32_t)r);
    float t = v[0];
#pragma unroll
    for (int r = 1; r < kFewCluster; ++r) t += v[r];
    const int l = (i >> 2) & 31, e = i & 3;   // fragment entry: rank index l / 4 (+ 8), row 2 (l % 4) (+ 1)
    const int j = (i >> 7) * 16 + (l >> 2) + 8 * (e >> 1);
    uint32_t hi, lo;
    split_bf16x2(j < rank ? t * sc : 0.f, 0.f, &hi, &lo);
    t_s[0][2 * (l & 3) + (e & 1)][j] = (uint16_t)hi;
    t_s[1][2 * (l & 3) + (e & 1)][j] = (uint16_t)lo;
  }
  lo_cluster_arrive();   // (waited for at the end: no CTA leaves while its part is read)
  __syncthreads();

  // t of row g, in the order of B's pieces
  uint2 th[NT], tl[NT];
#pragma unroll
  for (int s = 0; s < NT; ++s) {
    th[s] = *reinterpret_cast<const uint2*>(&t_s[0][g][16 * s + 4 * q]);
    tl[s] = *reinterpret_cast<const uint2*>(&t_s[1][g][16 * s + 4 * q]);
  }
  for (int n0 = n_first; n0 - 2 * g < n_hi; n0 += kAheadF * (16 * kLoWarps)) {
#pragma unroll
    for (int u = 0; u < kAheadF; ++u) {
      const int n = n0 + u * (16 * kLoWarps);
      float d[4] = {0.f, 0.f, 0.f, 0.f};   // (n, row0), (n, row1), (n + 1, row0), (n + 1, row1)
#pragma unroll
      for (int s = 0; s < NT; ++s) {
        const uint32_t(&bf)[4] = {bv[u][s][0].x, bv[u][s][1].x, bv[u][s][0].y, bv[u][s][1].y};
        mma16816(d, bf, tl[s].x, tl[s].y);
        mma16816(d, bf, th[s].x, th[s].y);
      }
      const uint32_t y0 = yv[u][0], y1 = yv[u][1];
      fetch(u, n + kAheadF * (16 * kLoWarps));
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = r ? row1 : row0;
        if (row < 0 || n >= n_hi) continue;
        const uint32_t w = r ? y1 : y0, o = pack_bf16x2(lo_f(w) + d[r], hi_f(w) + d[2 + r]);
        uint16_t* op = out + (size_t)row * N + n;
        if constexpr (kPair) {
          *reinterpret_cast<uint32_t*>(op) = o;
        } else {
          op[0] = (uint16_t)o;
          if (n + 1 < n_hi) op[1] = (uint16_t)(o >> 16);
        }
      }
    }
  }
  lo_cluster_wait();
}

// ---------------------------------------------------------------------------
// More rows: grouping by adapter.  One CTA counts the rows of each adapter
// (bucket n_adapters: rows without one) and deals them out to tiles of up to
// 64 rows of one bucket: tile i holds rows row_of[64 i] .. of info[i].adapter.
// The order of rows inside a bucket varies with the atomics' order; each
// row's result does not depend on it.
// ---------------------------------------------------------------------------
namespace {
constexpr int kTile = 64;
constexpr int kGroupThreads = 1024;
constexpr int kRun = 8;   // consecutive rows per thread

struct TileInfo {
  int adapter, rows;   // adapter -1: rows without one
};
}  // namespace

__global__ void __launch_bounds__(kGroupThreads) k_lora_group(const int32_t* __restrict__ ids, int n_adapters, int M,
                                                              int32_t* __restrict__ row_of, TileInfo* __restrict__ info,
                                                              int* __restrict__ n_tiles, int* err) {
  extern __shared__ int lg_smem[];
  int* cnt = lg_smem;                       // rows of each bucket
  int* tstart = cnt + n_adapters + 1;       // its first tile
  int* cur = tstart + n_adapters + 1;       // rows placed so far
  __shared__ int wsum[32];
  __shared__ int carry;
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  bool bad = false;
  const bool vec = ((uintptr_t)ids & 15u) == 0;
  // A thread takes kRun consecutive rows, a warp kRun * 32: rows in runs of one
  // adapter (the tokens of a sequence) are dealt with kRun at a time.
  int first[kRun];   // the buckets of the first rows, kept for the placing (-1: no row)
  auto load = [&](int r0, int (&v)[kRun]) {
    static_assert(kRun == 8, "two 16-byte loads");
    if (r0 + kRun <= M && vec) {
      const int4 p = *reinterpret_cast<const int4*>(ids + r0), w = *reinterpret_cast<const int4*>(ids + r0 + 4);
      v[0] = p.x, v[1] = p.y, v[2] = p.z, v[3] = p.w, v[4] = w.x, v[5] = w.y, v[6] = w.z, v[7] = w.w;
    } else {
#pragma unroll
      for (int i = 0; i < kRun; ++i) v[i] = r0 + i < M ? ids[r0 + i] : -2;
    }
#pragma unroll
    for (int i = 0; i < kRun; ++i) {
      const bool in = r0 + i < M, named = v[i] >= 0 && v[i] < n_adapters;
      bad |= in && !named && v[i] != -1;
      v[i] = !in ? -1 : named ? v[i] : n_adapters;
    }
  };
  auto one_run = [&](const int (&v)[kRun]) {
    bool same = true;
#pragma unroll
    for (int i = 1; i < kRun; ++i) same &= v[i] == v[0];
    return __all_sync(0xffffffffu, same);
  };
  load(tid * kRun, first);
  for (int i = tid; i <= n_adapters; i += kGroupThreads) cnt[i] = cur[i] = 0;
  if (tid == 0) carry = 0;
  __syncthreads();
  auto count = [&](int bkt, int weight) {
    const uint32_t same = __match_any_sync(0xffffffffu, bkt);
    if (bkt >= 0 && __ffs(same) - 1 == lane) atomicAdd(&cnt[bkt], weight * __popc(same));
  };
  for (int r0 = tid * kRun; r0 - lane * kRun < M; r0 += kGroupThreads * kRun) {
    int v[kRun];
    if (r0 == tid * kRun) {
#pragma unroll
      for (int i = 0; i < kRun; ++i) v[i] = first[i];
    } else {
      load(r0, v);
    }
    if (one_run(v)) {
      count(v[0], kRun);
    } else {
#pragma unroll
      for (int i = 0; i < kRun; ++i) count(v[i], 1);
    }
  }
  if (bad) atomicOr(err, kErrAdapter);
  __syncthreads();
  for (int i0 = 0; i0 <= n_adapters; i0 += kGroupThreads) {   // exclusive sum of the buckets' tiles
    const int i = i0 + tid;
    const int v = i <= n_adapters ? (cnt[i] + kTile - 1) / kTile : 0;
    int s = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int t = __shfl_up_sync(0xffffffffu, s, o);
      if (lane >= o) s += t;
    }
    if (lane == 31) wsum[warp] = s;
    __syncthreads();
    if (warp == 0) {
      int w = wsum[lane];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += t;
      }
      wsum[lane] = w;
    }
    __syncthreads();
    if (i <= n_adapters) tstart[i] = carry + (warp ? wsum[warp - 1] : 0) + s - v;
    __syncthreads();
    if (tid == 0) carry += wsum[31];
    __syncthreads();
  }
  if (tid == 0) *n_tiles = carry;
  auto place = [&](int bkt, int r, auto weight) {
    constexpr int kW = decltype(weight)::value;
    const uint32_t same = __match_any_sync(0xffffffffu, bkt);
    const int lead = __ffs(same) - 1;
    int at = 0;
    if (bkt >= 0 && lead == lane) at = atomicAdd(&cur[bkt], kW * __popc(same));
    at = __shfl_sync(0xffffffffu, at, lead) + kW * __popc(same & ((1u << lane) - 1u));
    if (bkt < 0) return;
    if (kW == 8 && at % 8 == 0) {   // the run lies in one tile
      const int tile = tstart[bkt] + at / kTile;
      int4* to = reinterpret_cast<int4*>(row_of + (size_t)tile * kTile + at % kTile);
      to[0] = make_int4(r, r + 1, r + 2, r + 3), to[1] = make_int4(r + 4, r + 5, r + 6, r + 7);
      if (at % kTile == 0) info[tile] = TileInfo{bkt == n_adapters ? -1 : bkt, min(kTile, cnt[bkt] - at)};
    } else {
#pragma unroll 1
      for (int i = 0; i < kW; ++i, ++at) {
        const int tile = tstart[bkt] + at / kTile;
        row_of[(size_t)tile * kTile + at % kTile] = r + i;
        if (at % kTile == 0) info[tile] = TileInfo{bkt == n_adapters ? -1 : bkt, min(kTile, cnt[bkt] - at)};
      }
    }
  };
  for (int r0 = tid * kRun; r0 - lane * kRun < M; r0 += kGroupThreads * kRun) {
    int v[kRun];
    if (r0 == tid * kRun) {
#pragma unroll
      for (int i = 0; i < kRun; ++i) v[i] = first[i];
    } else {
      load(r0, v);
    }
    if (one_run(v)) {
      place(v[0], r0, std::integral_constant<int, kRun>());
    } else {
#pragma unroll 1
      for (int i = 0; i < kRun; ++i) {
        int bkt = v[0];
#pragma unroll
        for (int j = 1; j < kRun; ++j) bkt = i == j ? v[j] : bkt;
        place(bkt, r0 + i, std::integral_constant<int, 1>());
      }
    }
  }
}

// ---------------------------------------------------------------------------
// t of a tile: 64 rows x K by the adapter's A^T; a cluster of `splits` CTAs
// shares a tile, each a part of K.  Four 16-row warps x two halves of each
// 64-wide K block; operands by cp.async into 128-byte-swizzled stages.  The
// parts are added in order (halves, then CTAs, through distributed shared
// memory), scaled, and stored as the two bf16 parts of k_lora_up's operand
// fragments: frag[tile][16-row group][16-wide step][part][lane].  (Loading
// fragments straight from global memory, without stages, was a third slower;
// handing f32 parts on to k_lora_up to add saves 3 us here and costs it more
// from rank 32 on.)
// ---------------------------------------------------------------------------
namespace {
constexpr int kDownStages = 4;
constexpr int kDownK = 64;

// Bytes from one column of B to the next in shared memory: whole 16-wide steps
// and 16 more, so that the 8 columns of a fragment lie in different banks.
__host__ __device__ __forceinline__ int b_pitch(int rank) { return ((rank + 15) & ~15) * 2 + 16; }

// How a thread's 8 columns of a 32-column group lie, in pieces of kW columns
// that every row of y and out is aligned to: piece p at column 4 kW p + kW q of
// the group, so that four lanes touch 8 kW bytes of a row at once.  Their words
// are, in order, the accumulator pairs of MMAs 0 to 3.
template <int kW>
struct Cols {
  static constexpr int kPieces = 8 / kW;
  __device__ static int at(int p, int q) { return 4 * kW * p + kW * q; }
  // where column n of B lies among the operands: MMA j, its column 2 q + n % 2
  __device__ static uint32_t place(uint32_t n) {
    const uint32_t j = (n & 31) / (4 * kW) * (kW / 2) + (n % kW) / 2, q = (n & 31) % (4 * kW) / kW;
    return (n & ~31u) | (j << 3) | (q << 1) | (n & 1);
  }
  // y's pieces into a 16-byte slot; c: the group's first column
  __device__ static void fetch(uint32_t slot, const uint16_t* row, int c, int q, int c_hi) {
#pragma unroll
    for (int p = 0; p < kPieces; ++p) {
      const int n = c + at(p, q);
      if (n >= c_hi) continue;
      if constexpr (kW == 8)
        cp16(slot, row + n, true);
      else if constexpr (kW == 4)
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(slot + p * 8), "l"(row + n) : "memory");
      else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(slot + p * 4), "l"(row + n) : "memory");
    }
  }
  __device__ static void store(uint16_t* row, int c, int q, int c_hi, const uint4& v) {
    if constexpr (kW == 8) {
      if (c + at(0, q) < c_hi) *reinterpret_cast<uint4*>(row + c + at(0, q)) = v;
    } else if constexpr (kW == 4) {
      if (c + at(0, q) < c_hi) *reinterpret_cast<uint2*>(row + c + at(0, q)) = make_uint2(v.x, v.y);
      if (c + at(1, q) < c_hi) *reinterpret_cast<uint2*>(row + c + at(1, q)) = make_uint2(v.z, v.w);
    } else {
      const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int p = 0; p < 4; ++p)
        if (c + at(p, q) < c_hi) *reinterpret_cast<uint32_t*>(row + c + at(p, q)) = w[p];
    }
  }
};

// 16-byte piece `c` (0..7) of 128-byte row r of a swizzled tile.
__device__ __forceinline__ uint32_t swz(int r, int c) { return (uint32_t)(r * 128 + ((c ^ (r & 7)) << 4)); }

__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr, uint32_t rank) {
  float4 v;
  asm volatile(
      "{\n\t.reg .b32 ra;\n\t"
      "mapa.shared::cluster.u32 ra, %4, %5;\n\t"
      "ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [ra];\n\t}"
      : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
      : "r"(addr), "r"(rank)
      : "memory");
  return v;
}

// NK: 16-wide steps of the rank (rank / 16 rounded up to a power of two).
template <int NK>
struct Down {
  static constexpr int kItems = 4 * NK * 32;
};

// The part of a tile's A x that K block range `split` of `splits` makes, in
// shared memory as [K half][8-wide half of the step][16-row group][step][lane].
// src: the rows of this thread's pieces.  after(i), i < kDownStages - 1, may
// issue copies in place of the last blocks' (one group each, not waited for).
template <int NK, typename F>
__device__ __forceinline__ float4* down_part(const uint16_t* __restrict__ x, const uint16_t* __restrict__ a, int rank,
                                             int K, int split, int splits, const TileInfo& tile, const int (&src)[2],
                                             uint8_t* smem, F after) {
  constexpr int kItems = Down<NK>::kItems;
  const int arows = (rank + 15) & ~15;                       // rows of an A stage (the last 8 may be unused)
  const uint32_t stage = (uint32_t)(kTile + arows) * 128;
  const uint32_t s0 = smem_u32(smem);
  const int kblocks = (K + kDownK - 1) / kDownK;
  const int kb0 = kblocks * split / splits, nk = kblocks * (split + 1) / splits - kb0;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int piece = tid & 7, r0 = tid >> 3;   // this thread's pieces: rows r0 + 32 i
  const uint16_t* xr[2];
  bool xin[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    xin[i] = r0 + 32 * i < tile.rows;
    xr[i] = x + (size_t)(xin[i] ? src[i] : 0) * K + piece * 8;
  }
  const uint16_t* ar = a + ((size_t)tile.adapter * rank + r0) * K + piece * 8;
  const size_t anext = (size_t)32 * K;
  const uint32_t xdst = swz(r0, piece);   // (rows 32 apart swizzle alike)
  auto load = [&](int kb, int s) {
    const int k = (kb0 + kb) * kDownK;
    const bool kin = k + piece * 8 < K;
    const uint32_t base = s0 + s * stage;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const bool in = kin && xin[i];
      cp16(base + xdst + 32 * 128 * i, in ? xr[i] + k : x, in);
    }
    const uint16_t* ap = ar + k;
    uint32_t adst = base + kTile * 128 + xdst;
    for (int r = r0; r < rank; r += 32, ap += anext, adst += 32 * 128) cp16(adst, kin ? ap : a, kin);
  };
#pragma unroll
  for (int s = 0; s < kDownStages - 1; ++s) {
    if (s < nk) load(s, s);
    else after(s - nk);
    cp_commit();
  }
  const int mg = warp & 3, kh = warp >> 2;
  float acc[2 * NK][4];
#pragma unroll
  for (int i = 0; i < 2 * NK; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
  const int am = mg * 16 + (lane & 7) + ((lane >> 3) & 1) * 8, ac = lane >> 4;     // x fragment: row, piece
  const int bm = (lane & 7) + (lane >> 4) * 8, bc = (lane >> 3) & 1;               // A fragment: rank row, piece
  uint32_t xoff[2], aoff[2];   // of the block's two 16-wide steps (rank rows 16 apart swizzle alike)
#pragma unroll
  for (int k16 = 0; k16 < 2; ++k16) {
    const int c = kh * 4 + k16 * 2;
    xoff[k16] = swz(am, c + ac), aoff[k16] = kTile * 128 + swz(bm, c + bc);
  }
  for (int kb = 0; kb < nk; ++kb) {
    cp_wait<kDownStages - 2>();
    __syncthreads();
    const int s = kb % kDownStages;
    if (kb + kDownStages - 1 < nk) load(kb + kDownStages - 1, (kb + kDownStages - 1) % kDownStages);
    else after(kb + kDownStages - 1 - nk);
    cp_commit();
    if (mg * 16 >= tile.rows) continue;   // no rows for this warp
    const uint32_t xs = s0 + s * stage;
    if constexpr (NK <= 2) {   // the block's operands ahead of its MMAs (at NK 4 and 8 this took 5 to 10% more)
      uint32_t af[2][4], bf[2][NK][4];
#pragma unroll
      for (int k16 = 0; k16 < 2; ++k16) {
        ldsm4(af[k16], xs + xoff[k16]);
#pragma unroll
        for (int p = 0; p < NK; ++p) ldsm4(bf[k16][p], xs + aoff[k16] + p * 16 * 128);
      }
#pragma unroll
      for (int k16 = 0; k16 < 2; ++k16)
#pragma unroll
        for (int p = 0; p < NK; ++p) {
          mma16816(acc[2 * p], af[k16], bf[k16][p][0], bf[k16][p][1]);
          if (p * 16 + 8 < rank) mma16816(acc[2 * p + 1], af[k16], bf[k16][p][2], bf[k16][p][3]);
        }
    } else {
#pragma unroll
      for (int k16 = 0; k16 < 2; ++k16) {
        uint32_t af[4];
        ldsm4(af, xs + xoff[k16]);
#pragma unroll
        for (int p = 0; p < NK; ++p)
          if (p * 16 < rank) {
            uint32_t bf[4];
            ldsm4(bf, xs + aoff[k16] + p * 16 * 128);
            mma16816(acc[2 * p], af, bf[0], bf[1]);
            if (p * 16 + 8 < rank) mma16816(acc[2 * p + 1], af, bf[2], bf[3]);
          }
      }
    }
  }
  __syncthreads();
  float4* part = reinterpret_cast<float4*>(smem);
#pragma unroll
  for (int i = 0; i < 2 * NK; ++i)
    part[(kh * 2 + (i & 1)) * kItems + (mg * NK + i / 2) * 32 + lane] = make_float4(acc[i][0], acc[i][1], acc[i][2], acc[i][3]);
  return part;
}

__device__ __forceinline__ void st_cluster_u4(uint32_t addr, uint32_t rank, const uint4& v) {
  asm volatile(
      "{\n\t.reg .b32 ra;\n\t"
      "mapa.shared::cluster.u32 ra, %0, %1;\n\t"
      "st.shared::cluster.v4.u32 [ra], {%2, %3, %4, %5};\n\t}" ::"r"(addr),
      "r"(rank), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
      : "memory");
}

// t of item i of a tile (see k_lora_down) from the cluster's parts.
template <int NK>
__device__ __forceinline__ void gather_t(const float4* part, int i, int splits, float sc, uint4* hi, uint4* lo) {
  float4 v[2] = {make_float4(0.f, 0.f, 0.f, 0.f), make_float4(0.f, 0.f, 0.f, 0.f)};
  for (int c = 0; c < splits; ++c)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float4* p = part + e * Down<NK>::kItems + i;
      const float4 w = splits > 1 ? ld_cluster_f32x4(smem_u32(p), (uint32_t)c) : *p;
      float4& t = v[e & 1];
      t.x += w.x, t.y += w.y, t.z += w.z, t.w += w.w;
    }
  // rows g, g + 8 of entries 2 q, + 1; the same of 8 + 2 q, + 1
  split_bf16x2(v[0].x * sc, v[0].y * sc, &hi->x, &lo->x);
  split_bf16x2(v[0].z * sc, v[0].w * sc, &hi->y, &lo->y);
  split_bf16x2(v[1].x * sc, v[1].y * sc, &hi->z, &lo->z);
  split_bf16x2(v[1].z * sc, v[1].w * sc, &hi->w, &lo->w);
}

// While one CTA groups the rows the next kernel's bring x to L2, each a share
// (x is older than the grouping kernel, which waited for it before letting
// this one start).
__device__ __forceinline__ void x_to_l2(const uint16_t* x, size_t bytes) {
  if (threadIdx.x >= 32) return;
  const size_t share = (bytes / gridDim.x / 32) & ~(size_t)15;
  if (share)
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(
                     reinterpret_cast<uint64_t>(x) + ((size_t)blockIdx.x * 32 + threadIdx.x) * share),
                 "r"((uint32_t)share)
                 : "memory");
}

}  // namespace

template <int NK>
__global__ void __launch_bounds__(kLoThreads) k_lora_down(const uint16_t* __restrict__ x, const uint16_t* __restrict__ a,
                                                          const float* __restrict__ scale,
                                                          const int32_t* __restrict__ row_of,
                                                          const TileInfo* __restrict__ info,
                                                          const int* __restrict__ n_tiles, int rank, int K, int splits,
                                                          size_t x_ahead, uint4* __restrict__ frag) {
  extern __shared__ __align__(128) uint8_t ld_smem[];
  constexpr int kItems = Down<NK>::kItems;
  const int tid = threadIdx.x;
  const int at = blockIdx.x / splits, split = blockIdx.x - at * splits;
  x_to_l2(x, x_ahead);
  pdl_wait();
  pdl_trigger();
  const int have = *n_tiles;
  const TileInfo tile = info[at];
  int src[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) src[i] = row_of[(size_t)at * kTile + (tid >> 3) + 32 * i];
  if (at >= have || tile.adapter < 0) return;   // (what was read past the last tile is not used)
  const float4* part = down_part<NK>(x, a, rank, K, split, splits, tile, src, ld_smem, [](int) {});
  const float sc = scale ? scale[tile.adapter] : 1.f;
  if (splits > 1) {
    lo_cluster_arrive();
    lo_cluster_wait();
  } else {
    __syncthreads();
  }
  uint4* out = frag + (size_t)at * kItems * 2;
  for (int i = split * kLoThreads + tid; i < kItems; i += splits * kLoThreads) {
    uint4 hi, lo;
    gather_t<NK>(part, i, splits, sc, &hi, &lo);
    uint4* o = out + (size_t)(i >> 5) * 64 + (i & 31);
    o[0] = hi;
    o[32] = lo;
  }
  if (splits > 1) {   // no CTA leaves while its part is read
    lo_cluster_arrive();
    lo_cluster_wait();
  }
}

// ---------------------------------------------------------------------------
// Both products of a tile in one kernel, where the tiles' clusters fit on the
// GPU at once (see lora_one_kernel): the CTAs that shared K share the columns,
// in 64-wide steps through a ring of stages.  The first steps' y and B are under
// way while t is joined.  No launch and no tail between the products: 5669 rows
// 4096 -> 2688 in 30.5 us at rank 32, 28.0 at rank 16 (with the two kernels 34.0
// and 32.4; floor 16.3).  Bringing each row's y to L2 further ahead took 3 more.
// kW: columns per piece of y and out (8, or 4 or 2 where rows of N % 4 or N % 2
// columns start on no more: 1336 x 2498 of 63 adapters, rank 24, in 23.3 us, with
// the two kernels 26).
// ---------------------------------------------------------------------------
namespace {
constexpr int kStepCols = 64;
constexpr int kStepStages = kDownStages;   // (the first kDownStages - 1 go out in down_part's last groups)

template <int NK>
struct Step {
  static constexpr int kY = 2 * kLoThreads * 16;
  static constexpr int kBytes = kY + kStepCols * (32 * NK + 16);
};
}  // namespace

template <int NK, int kW>
__global__ void __launch_bounds__(kLoThreads, 2) k_lora_tile(
    const uint16_t* y, const uint16_t* __restrict__ x, const uint16_t* __restrict__ a, const uint16_t* __restrict__ b,
    const float* __restrict__ scale, const int32_t* __restrict__ row_of, const TileInfo* __restrict__ info,
    const int* __restrict__ n_tiles, int rank, int N, int K, int splits, size_t x_ahead, uint16_t* out) {
  extern __shared__ __align__(128) uint8_t lt_smem[];
  constexpr int kItems = Down<NK>::kItems;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, q = lane & 3, mg = warp & 3;
  const int at = blockIdx.x / splits, split = blockIdx.x - at * splits;
  x_to_l2(x, x_ahead);
  pdl_wait();
  pdl_trigger();
  const int have = *n_tiles;
  const TileInfo tile = info[at];
  int src[2], row[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    src[i] = row_of[(size_t)at * kTile + (tid >> 3) + 32 * i];
    row[i] = row_of[(size_t)at * kTile + mg * 16 + g + 8 * i];
  }
  if (at >= have) return;   // (what was read past the last tile is not used)
  const int units = (N + kStepCols - 1) / kStepCols;
  const int u0 = (int)((long long)units * split / splits), nu = (int)((long long)units * (split + 1) / splits) - u0;
  const bool bare = tile.adapter < 0;   // rows without an adapter: y moves as it is
  if (bare && out == y) return;
#pragma unroll
  for (int h = 0; h < 2; ++h)
    if (mg * 16 + g + 8 * h >= tile.rows) row[h] = -1;
  // a step: y into slots of each thread's own, B in the order of the MMAs
  const int arows = (rank + 15) & ~15, pitch = b_pitch(rank), rv = rank / 8;
  uint8_t* steps = lt_smem + kDownStages * (kTile + arows) * 128;
  const int bn = tid / rv, bv = tid - bn * rv;   // this thread's piece of B
  const int bpos = Cols<kW>::place(bn);
  const uint16_t* bt = b + (size_t)(bare ? 0 : tile.adapter) * N * rank + bv * 8;
  const int cw = (warp >> 2) * 32;               // this warp's columns of a step
  auto load = [&](int u) {
    if (u >= nu) return;
    uint8_t* st = steps + (u % kStepStages) * Step<NK>::kBytes;
    const int c0 = (u0 + u) * kStepCols;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      if (row[h] >= 0) Cols<kW>::fetch(smem_u32(st + (h * kLoThreads + tid) * 16), y + (size_t)row[h] * N, c0 + cw, q, N);
    if (bn < kStepCols && !bare) {
      const bool in = c0 + bn < N;
      cp16(smem_u32(st + Step<NK>::kY + bpos * pitch + bv * 16), in ? bt + (size_t)(c0 + bn) * rank : b, in);
    }
  };
  if (rank & 8)   // the last 16-wide step reads 8 entries past the rank: zeros
    for (int i = tid; i < kStepStages * kStepCols; i += kLoThreads)
      *reinterpret_cast<uint4*>(steps + i / kStepCols * Step<NK>::kBytes + Step<NK>::kY + i % kStepCols * pitch + rank * 2) =
          make_uint4(0u, 0u, 0u, 0u);
  uint4 th[NK], tl[NK];   // t of the warp's 16 rows
  if (bare) {
#pragma unroll
    for (int u = 0; u < kStepStages - 1; ++u) load(u), cp_commit();
  } else {
    const float4* part = down_part<NK>(x, a, rank, K, split, splits, tile, src, lt_smem, load);
    const float sc = scale ? scale[tile.adapter] : 1.f;
    lo_cluster_arrive();
    lo_cluster_wait();
    // each CTA joins its share of the items and hands them to all (every CTA
    // joining all of them took 3 to 20 us more)
    uint4* tf = reinterpret_cast<uint4*>(lt_smem + 4 * kItems * 16);
    for (int i = kItems * split / splits + tid; i < kItems * (split + 1) / splits; i += kLoThreads) {
      uint4 hi, lo;
      gather_t<NK>(part, i, splits, sc, &hi, &lo);
      for (int c = 0; c < splits; ++c) {
        st_cluster_u4(smem_u32(tf + i), (uint32_t)c, hi);
        st_cluster_u4(smem_u32(tf + kItems + i), (uint32_t)c, lo);
      }
    }
    lo_cluster_arrive();
    lo_cluster_wait();
#pragma unroll
    for (int s = 0; s < NK; ++s) th[s] = tf[(mg * NK + s) * 32 + lane], tl[s] = tf[kItems + (mg * NK + s) * 32 + lane];
  }
  const uint32_t boff = Step<NK>::kY + (uint32_t)((warp >> 2) * 32 + (lane & 7) + (lane >> 4) * 8) * pitch +
                        (uint32_t)((lane >> 3) & 1) * 16;
  for (int u = 0; u < nu; ++u) {
    cp_wait<kStepStages - 2>();
    __syncthreads();
    load(u + kStepStages - 1);
    cp_commit();
    if (mg * 16 >= tile.rows) continue;   // no rows for this warp
    const uint8_t* st = steps + (u % kStepStages) * Step<NK>::kBytes;
    const uint32_t bs = smem_u32(st) + boff;
    float acc[4][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
#pragma unroll
    for (int s = 0; s < NK; ++s)
      if (s * 16 < rank && !bare) {
        const uint32_t lo[4] = {tl[s].x, tl[s].y, tl[s].z, tl[s].w}, hi[4] = {th[s].x, th[s].y, th[s].z, th[s].w};
        uint32_t bf[2][4];
#pragma unroll
        for (int jp = 0; jp < 2; ++jp) ldsm4(bf[jp], bs + (uint32_t)(jp * 16) * pitch + s * 32);
#pragma unroll
        for (int j = 0; j < 4; ++j) mma16816(acc[j], lo, bf[j / 2][j % 2 * 2], bf[j / 2][j % 2 * 2 + 1]);
#pragma unroll
        for (int j = 0; j < 4; ++j) mma16816(acc[j], hi, bf[j / 2][j % 2 * 2], bf[j / 2][j % 2 * 2 + 1]);
      }
    const int c = (u0 + u) * kStepCols + cw;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (row[h] < 0) continue;
      uint4 v = *reinterpret_cast<const uint4*>(st + (h * kLoThreads + tid) * 16);
      if (!bare) add_pairs(&v, acc, h);
      Cols<kW>::store(out + (size_t)row[h] * N, c, q, N, v);
    }
  }
  cp_wait<0>();
}

// ---------------------------------------------------------------------------
// out of a tile and Up::kCols columns: y + B t.  The columns of B are dealt out
// to the MMAs so that a thread's accumulators are 8 consecutive columns: y and
// out move in 16-byte pieces, 64 bytes of a row per four lanes, or, where rows
// start on less (!kVec), through rows in shared memory (44 us against 27.5 for
// 6614 x 5020 and x 5024, rank 24; in 8-byte pieces straight 45: their stores
// end inside sectors).  Many small CTAs: the stream runs at the copy rate when its tail is short (a pure copy in this
// pattern: 41 CTAs per tile 6580 GB/s, 3 to 6 of them 5200 to 5600), so what a
// CTA needs before its first load of y is two dependent reads deep.
// ---------------------------------------------------------------------------
namespace {
template <int NK>
struct Up {
  static constexpr int kCols = NK <= 4 ? 256 : 128;
  static constexpr int kRowBytes = kCols * 2 + 64;   // of an unaligned row in shared memory (pieces, and no bank conflicts)
};
}  // namespace

template <int NK, bool kVec>
__global__ void __launch_bounds__(kLoThreads, NK <= 2 ? 4 : NK == 4 ? 3 : 2) k_lora_up(
    const uint16_t* y, const uint4* __restrict__ frag, const uint16_t* __restrict__ b,
    const int32_t* __restrict__ row_of, const TileInfo* __restrict__ info, const int* __restrict__ n_tiles, int rank,
    int N, int chunks, uint16_t* out) {
  extern __shared__ __align__(128) uint8_t lu_smem[];
  constexpr int kCols = Up<NK>::kCols, kGroups = kCols / 64;   // 32-column groups per warp
  const int at = blockIdx.x / chunks, c0 = (blockIdx.x - at * chunks) * kCols, c_hi = min(N, c0 + kCols);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int g = lane >> 2, q = lane & 3, mg = warp & 3;
  // What k_lora_group wrote, y and B are read ahead of the wait: the kernel
  // waited for (k_lora_down, which writes none of them) itself waited for
  // everything before it prior to letting this one start.
  const int have = *n_tiles;
  const TileInfo tile = info[at];
  int row[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) row[h] = row_of[(size_t)at * kTile + mg * 16 + g + 8 * h];
  // (unaligned: the warp moves rows warp + 8 i of the tile, known to lane i)
  int moved = 0;
  if constexpr (!kVec) moved = row_of[(size_t)at * kTile + warp + kLoWarps * (lane & 7)];
  if (at >= have) {   // (what was read past the last tile is not used)
    pdl_wait();
    return;
  }
#pragma unroll
  for (int h = 0; h < 2; ++h)
    if (mg * 16 + g + 8 * h >= tile.rows) row[h] = -1;
  const int cw = c0 + (warp >> 2) * (kCols / 2);
  uint4* ys = reinterpret_cast<uint4*>(lu_smem) + tid;   // [group][half][thread]
  if (tile.adapter < 0 && (kVec || out == y)) {   // rows without an adapter: y moves as it is
    pdl_wait();
    pdl_trigger();
    if (out == y) return;
    uint4 v[kGroups][2];
#pragma unroll
    for (int i = 0; i < 2 * kGroups; ++i)
      v[i / 2][i % 2] = row[i % 2] >= 0 && cw + i / 2 * 32 + q * 8 < c_hi
                            ? *reinterpret_cast<const uint4*>(y + (size_t)row[i % 2] * N + cw + i / 2 * 32 + q * 8)
                            : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int i = 0; i < 2 * kGroups; ++i)
      if (row[i % 2] >= 0 && cw + i / 2 * 32 + q * 8 < c_hi)
        *reinterpret_cast<uint4*>(out + (size_t)row[i % 2] * N + cw + i / 2 * 32 + q * 8) = v[i / 2][i % 2];
    return;
  }
  const bool bare = !kVec && tile.adapter < 0;
  // y, asked for at once and held by no registers.  Aligned: each thread's
  // pieces into slots of its own.  Otherwise each row's aligned 16-byte pieces
  // (all of which hold bytes of the row's columns) into a row of shared memory,
  // shifted there by the warp that fetched them, and back on the way out.
  if constexpr (kVec) {
#pragma unroll
    for (int u = 0; u < kGroups; ++u)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int n = cw + u * 32 + q * 8;
        if (row[h] >= 0 && n < c_hi) cp16(smem_u32(ys + (u * 2 + h) * kLoThreads), y + (size_t)row[h] * N + n, true);
      }
  } else {
#pragma unroll
    for (int i = 0; i < kTile / kLoWarps; ++i) {
      const int r = warp + kLoWarps * i;
      if (r >= tile.rows) break;
      const uintptr_t p = (uintptr_t)(y + (size_t)__shfl_sync(0xffffffffu, moved, i) * N + c0), first = p & ~(uintptr_t)15;
      const int pieces = (int)((p + (size_t)(c_hi - c0) * 2 - first + 15) / 16);
      for (int j = lane; j < pieces; j += 32)
        cp16(smem_u32(lu_smem + r * Up<NK>::kRowBytes + j * 16), (const void*)(first + j * 16), true);
    }
  }
  const int pitch = b_pitch(rank), rv = rank / 8;
  uint8_t* bsm = lu_smem + (kVec ? kGroups * 2 * kLoThreads * 16 : kTile * Up<NK>::kRowBytes);
  const uint32_t s0 = smem_u32(bsm);
  if (!bare) {
    const uint16_t* bt = b + ((size_t)tile.adapter * N + c0) * rank;
    const int n_step = kLoThreads / rv, v_step = kLoThreads - n_step * rv;
    int n = tid / rv, v = tid - n * rv;   // (stepped, not divided, from piece to piece)
    for (int i = tid; i < kCols * rv; i += kLoThreads) {
      const int pos = Cols<8>::place(n);
      const bool in = c0 + n < c_hi;
      cp16(s0 + (uint32_t)(pos * pitch + v * 16), in ? bt + (size_t)i * 8 : b, in);
      n += n_step, v += v_step;
      if (v >= rv) v -= rv, ++n;
    }
    if (rank & 8)   // the last 16-wide step reads 8 entries past the rank: zeros
      for (int n = tid; n < kCols; n += kLoThreads)
        *reinterpret_cast<uint4*>(bsm + n * pitch + rank * 2) = make_uint4(0u, 0u, 0u, 0u);
  }
  cp_commit();
  pdl_wait();
  pdl_trigger();
  uint4 th[NK], tl[NK];   // t of the warp's 16 rows (a bare tile's is not written, and not used)
  const uint4* fp = frag + ((size_t)at * 4 + mg) * NK * 64 + lane;
#pragma unroll
  for (int s = 0; s < NK; ++s) th[s] = __ldg(fp + s * 64), tl[s] = __ldg(fp + s * 64 + 32);
  cp_wait<0>();
  if constexpr (!kVec) {
    __syncwarp();   // (the row's pieces came through all lanes)
    uint4 v[kTile / kLoWarps];
#pragma unroll
    for (int i = 0; i < kTile / kLoWarps; ++i) {
      const uint32_t mis = (uint32_t)((uintptr_t)(y + (size_t)__shfl_sync(0xffffffffu, moved, i) * N + c0) & 15u);
      const uint4* rp = reinterpret_cast<const uint4*>(lu_smem + (warp + kLoWarps * i) * Up<NK>::kRowBytes);
      if (lane < kCols / 8) v[i] = bytes16_at(rp[lane], rp[lane + 1], mis);
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < kTile / kLoWarps; ++i)
      if (lane < kCols / 8) reinterpret_cast<uint4*>(lu_smem + (warp + kLoWarps * i) * Up<NK>::kRowBytes)[lane] = v[i];
  }
  __syncthreads();
  if (kVec && mg * 16 >= tile.rows) return;   // no rows for this warp
  const uint32_t bs = s0 + (uint32_t)((warp >> 2) * (kCols / 2) + (lane & 7) + (lane >> 4) * 8) * pitch +
                      (uint32_t)((lane >> 3) & 1) * 16;
  if (kVec || !bare)
#pragma unroll
  for (int u = 0; u < kGroups; ++u) {
    float acc[4][4];
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j][0] = acc[j][1] = acc[j][2] = acc[j][3] = 0.f;
#pragma unroll
    for (int s = 0; s < NK; ++s)
      if (s * 16 < rank) {
        const uint32_t lo[4] = {tl[s].x, tl[s].y, tl[s].z, tl[s].w}, hi[4] = {th[s].x, th[s].y, th[s].z, th[s].w};
        uint32_t bf[2][4];
#pragma unroll
        for (int jp = 0; jp < 2; ++jp) ldsm4(bf[jp], bs + (uint32_t)(u * 32 + jp * 16) * pitch + s * 32);
#pragma unroll
        for (int j = 0; j < 4; ++j) mma16816(acc[j], lo, bf[j / 2][j % 2 * 2], bf[j / 2][j % 2 * 2 + 1]);
#pragma unroll
        for (int j = 0; j < 4; ++j) mma16816(acc[j], hi, bf[j / 2][j % 2 * 2], bf[j / 2][j % 2 * 2 + 1]);
      }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (row[h] < 0) continue;
      if constexpr (kVec) {
        const int n = cw + u * 32 + q * 8;
        if (n >= c_hi) continue;
        uint4 v = ys[(u * 2 + h) * kLoThreads];
        add_pairs(&v, acc, h);
        *reinterpret_cast<uint4*>(out + (size_t)row[h] * N + n) = v;
      } else {
        // (columns past the last are computed in place too, and not stored)
        uint4* rp = reinterpret_cast<uint4*>(lu_smem + (mg * 16 + g + 8 * h) * Up<NK>::kRowBytes) + (cw - c0 + u * 32) / 8 + q;
        uint4 v = *rp;
        add_pairs(&v, acc, h);
        *rp = v;
      }
    }
  }
  if constexpr (!kVec) {   // rows out, by out's aligned pieces; the ends by element
    __syncthreads();
    const int bytes = (c_hi - c0) * 2;
#pragma unroll
    for (int i = 0; i < kTile / kLoWarps; ++i) {
      const int r = warp + kLoWarps * i;
      if (r >= tile.rows) break;
      uint8_t* o = reinterpret_cast<uint8_t*>(out + (size_t)__shfl_sync(0xffffffffu, moved, i) * N + c0);
      const int mis = (int)((uintptr_t)o & 15u);
      const uint4* rp = reinterpret_cast<const uint4*>(lu_smem + r * Up<NK>::kRowBytes);
      // whole pieces: j = 1 .. (or 0, aligned) up to the last that ends inside
      const int whole = (mis + bytes) / 16;
      for (int j = lane + (mis ? 1 : 0); j < whole; j += 32)
        *reinterpret_cast<uint4*>(o - mis + j * 16) = mis ? bytes16_at(rp[j - 1], rp[j], 16 - mis) : rp[j];
      // the ends: lanes 0..7 the first piece's elements, 8..15 the last one's
      const int e = lane < 8 ? 2 * lane : whole * 16 - mis + 2 * (lane - 8);
      if (lane < 16 && e >= 0 && e < bytes && (lane < 8 ? mis && e < 16 - mis : whole > 0 || !mis))
        *reinterpret_cast<uint16_t*>(o + e) = *reinterpret_cast<const uint16_t*>(reinterpret_cast<const uint8_t*>(rp) + e);
    }
  }
}

namespace {

size_t lo_align256(size_t v) { return (v + 255) & ~(size_t)255; }

// No more tiles than the full ones and one partial per bucket.
int lora_max_tiles(int M, int n_adapters) { return M / kTile + (n_adapters < M ? n_adapters + 1 : M); }

int lora_steps(int rank) { return rank <= 16 ? 1 : rank <= 32 ? 2 : rank <= 64 ? 4 : 8; }

struct LoraWs {
  int32_t* row_of;
  TileInfo* info;
  int* n_tiles;
  uint4* frag;
  size_t total;
};

// CTAs sharing a tile's K: two per SM for the fewest tiles the rows can make.
int lora_splits(int M, int K) {
  const int tiles = (M + kTile - 1) / kTile, kblocks = (K + kDownK - 1) / kDownK;
  const int s = (2 * device_sm_count() + tiles - 1) / tiles;
  return std::max(1, std::min({s, 8, kblocks / 4}));   // (four blocks each at least: the stages)
}

// CTAs per tile of the one-kernel form (0: the two-kernel form).  It wins
// where the tiles' clusters fit on the GPU at once, two CTAs per SM, with two
// CTAs a tile at least; a CTA's columns are a loop, so not where few CTAs have
// many steps; and a long stream of y runs better with many small CTAs.  us, one
// kernel / two, 4096 -> 2688 rank 32: 600 rows 15.3 / 16.9, 2048 17.1 / 21.7,
// 5669 30.5 / 34.0, 9600 (more tiles than that) 64 / 48; 2688 -> 10304 rank 16:
// 1024 rows (128 CTAs of 20 steps) 21.5 / 19.2, 2048 24.3 / 27.5, 5669 53.6 /
// 54.5, 8192 73.5 / 70.6.
int lora_one_kernel(int M, int N, int K, int max_tiles) {
  const int sms = device_sm_count(), kblocks = (K + kDownK - 1) / kDownK;
  const int splits = std::min({2 * sms / max_tiles, 8, kblocks / 4});
  if (splits < 2 || (long long)M * N > 1ll << 26) return 0;
  const int steps = (N + kStepCols * splits - 1) / (kStepCols * splits);
  const int tiles = (M + kTile - 1) / kTile;   // the fewest; there may be as many as max_tiles
  return (tiles + max_tiles) / 2 * splits >= sms || steps <= 8 ? splits : 0;
}

LoraWs carve_lora(void* base, int M, int rank, int n_adapters) {
  char* p = static_cast<char*>(base);
  const size_t tiles = (size_t)lora_max_tiles(M, n_adapters);
  LoraWs w;
  size_t off = 0;
  w.row_of = reinterpret_cast<int32_t*>(p + off), off += lo_align256(tiles * kTile * 4);
  w.info = reinterpret_cast<TileInfo*>(p + off), off += lo_align256(tiles * sizeof(TileInfo));
  w.n_tiles = reinterpret_cast<int*>(p + off), off += 256;
  w.frag = reinterpret_cast<uint4*>(p + off), off += tiles * lora_steps(rank) * 4 * 64 * sizeof(uint4);
  w.total = off;
  return w;
}

template <int NT, bool kPair>
cudaError_t launch_few(const uint16_t* y, const uint16_t* x, const LoraWeights& w, const int32_t* ids, uint16_t* out,
                       int M, int N, int K, int* err, cudaStream_t st) {
  // slices of N: clusters for most SMs, one CTA each (a second on some SMs
  // holds up its cluster: 152 CTAs took 5.8 us where 128 took 5.1), but no
  // less than a step of each warp
  const int sms = device_sm_count(), least = kFewCluster * kLoWarps * 16;
  int slices = sms * 27 / 32 / (kFewCluster * M);
  const int most = (N + least - 1) / least;
  if (slices > most) slices = most;
  if (slices < 1) slices = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(kFewCluster * slices), (unsigned)M);
  cfg.blockDim = dim3(kLoThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kFewCluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, k_lora_few<NT, kPair>, y, x, w.a, w.b, w.scale, ids, w.n_adapters, w.rank, out, M, N, K,
                            err);
}

template <int NK>
cudaError_t launch_many(const uint16_t* y, const uint16_t* x, const LoraWeights& w, uint16_t* out, int M, int N, int K,
                        const LoraWs& ws, int max_tiles, cudaStream_t st, int* launches) {
  // columns per piece of y and out: every row starts on such a piece
  const uintptr_t where = (uintptr_t)y | (uintptr_t)out;
  const int width = N % 8 == 0 && where % 16 == 0  ? 8
                    : N % 4 == 0 && where % 8 == 0 ? 4
                    : N % 2 == 0 && where % 4 == 0 ? 2
                                                   : 0;
  const int one = NK <= 2 && width ? lora_one_kernel(M, N, K, max_tiles) : 0;
  const int splits = one ? one : lora_splits(M, K);
  const size_t dsm = (size_t)kDownStages * (kTile + ((w.rank + 15) & ~15)) * 128;
  static_assert(kDownStages * (kTile + 8) * 128 >= 4 * 4 * 32 * 16, "the parts fit where the stages were");
  cudaError_t e = ensure_smem_optin((const void*)k_lora_down<NK>, kDownStages * (kTile + 16 * NK) * 128);
  if (e != cudaSuccess) return e;
  constexpr size_t kXAhead = (size_t)64 << 20;   // half of L2: a larger x would push itself out
  const size_t x_bytes = (size_t)M * K * 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)splits * (unsigned)max_tiles);
  cfg.blockDim = dim3(kLoThreads);
  cfg.dynamicSmemBytes = dsm;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)splits;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  if constexpr (NK <= 2) {
    if (one) {
      *launches = 2;
      const auto kernel = width == 8 ? k_lora_tile<NK, 8> : width == 4 ? k_lora_tile<NK, 4> : k_lora_tile<NK, 2>;
      if ((e = ensure_smem_optin((const void*)kernel,
                                 kDownStages * (kTile + 16 * NK) * 128 + kStepStages * Step<NK>::kBytes)) != cudaSuccess)
        return e;
      cfg.dynamicSmemBytes = dsm + kStepStages * Step<NK>::kBytes;
      return cudaLaunchKernelEx(&cfg, kernel, y, x, w.a, w.b, w.scale, (const int32_t*)ws.row_of,
                                (const TileInfo*)ws.info, (const int*)ws.n_tiles, w.rank, N, K, splits,
                                x_bytes <= kXAhead ? x_bytes : 0, out);
    }
  }
  e = cudaLaunchKernelEx(&cfg, k_lora_down<NK>, x, w.a, w.scale, (const int32_t*)ws.row_of, (const TileInfo*)ws.info,
                         (const int*)ws.n_tiles, w.rank, K, splits, x_bytes <= kXAhead ? x_bytes : 0, ws.frag);
  if (e != cudaSuccess) return e;
  constexpr int kCols = Up<NK>::kCols;
  const int chunks = (N + kCols - 1) / kCols;
  if ((long long)chunks * max_tiles > 0x7fffffffll) return cudaErrorInvalidValue;
  constexpr int kRows = kTile * Up<NK>::kRowBytes;   // (more than the aligned form's kCols / 32 slots per thread)
  static_assert(kRows >= kCols / 32 * kLoThreads * 16, "");
  const size_t usm = (size_t)kCols * b_pitch(w.rank) + (width == 8 ? kCols / 32 * kLoThreads * 16 : kRows);
  const dim3 grid((unsigned)(chunks * max_tiles));
  const auto kernel = width == 8 ? k_lora_up<NK, true> : k_lora_up<NK, false>;
  if ((e = ensure_smem_optin((const void*)kernel, kCols * (32 * NK + 16) + kRows)) != cudaSuccess)
    return e;
  return launch_pdl(kernel, grid, dim3(kLoThreads), usm, st, y, ws.frag, w.b, ws.row_of, ws.info, ws.n_tiles, w.rank, N,
                    chunks, out);
}

}  // namespace

// Which form: units of an adapter's rows up to kFewRows rows; beyond, up to
// kFewMost, while the adapters are so many that 64-row tiles would be nearly
// empty if the rows named them all, which the host does not know: 1000 rows
// that name 1 or 4 of 256 adapters take 36 us, of 64 adapters (tiles) 19 to 21
// (2688 -> 10304 rank 16).  The tile form's grids follow the adapters there are
// as well: 5669 rows that name 4 of 4, 512 and 4096 take 54, 62 and 165 us.
// Measured with all adapters named (us, units / tiles): 2688 -> 10304 rank 16, 1
// adapter: 256 rows 13 / 13, 320 14.5 / 12.9, 384 16.4 / 13.7; 64 adapters: 256
// rows 17 / 29, 384 21 / 30, 512 23 / 25, 640 31 / 31; 256 adapters: 1024 rows
// 52 / 82.  4096 -> 2688 rank 32, 1 adapter: 320 rows 12.0 / 13.3, 384 13.9 /
// 13.3; 64 adapters: 384 rows 17 / 23, 640 26 / 23; 128: 896 rows 30.5 / 32,
// 1024 32 / 28.
static bool few_rows(int M, int n_adapters) { return M <= kFewRows || (M <= kFewMost && M <= 7 * n_adapters); }

size_t lora_workspace_bytes(int M, int N, int K, int rank, int n_adapters) {
  (void)N, (void)K;
  return few_rows(M, n_adapters) ? 0 : carve_lora(nullptr, M, rank, n_adapters).total;
}

cudaError_t launch_lora_add(const uint16_t* y, const uint16_t* x, const LoraWeights& w, const int32_t* ids, uint16_t* out,
                            int M, int N, int K, void* ws, int* err, cudaStream_t st, int* launches) {
  if (M == 0) return cudaSuccess;
  if (few_rows(M, w.n_adapters)) {
    *launches = 1;
    const bool pair = N % 2 == 0 && (uintptr_t)y % 4 == 0 && (uintptr_t)out % 4 == 0;
#define M2_LORA_FEW(NT)                                                            \
  return pair ? launch_few<NT, true>(y, x, w, ids, out, M, N, K, err, st)           \
              : launch_few<NT, false>(y, x, w, ids, out, M, N, K, err, st)
    if (w.rank <= 16) M2_LORA_FEW(1);
    if (w.rank <= 32) M2_LORA_FEW(2);
    if (w.rank <= 64) M2_LORA_FEW(4);
    M2_LORA_FEW(8);
#undef M2_LORA_FEW
  }
  *launches = 3;
  const LoraWs lw = carve_lora(ws, M, w.rank, w.n_adapters);
  const size_t gsm = (size_t)3 * (w.n_adapters + 1) * 4;
  cudaError_t e = ensure_smem_optin((const void*)k_lora_group, 3 * (kLoraMaxAdapters + 1) * 4);
  if (e != cudaSuccess) return e;
  e = launch_pdl(k_lora_group, dim3(1), dim3(kGroupThreads), gsm, st, ids, w.n_adapters, M, lw.row_of, lw.info,
                 lw.n_tiles, err);
  if (e != cudaSuccess) return e;
  const int max_tiles = lora_max_tiles(M, w.n_adapters);
  if (w.rank <= 16) return launch_many<1>(y, x, w, out, M, N, K, lw, max_tiles, st, launches);
  if (w.rank <= 32) return launch_many<2>(y, x, w, out, M, N, K, lw, max_tiles, st, launches);
  if (w.rank <= 64) return launch_many<4>(y, x, w, out, M, N, K, lw, max_tiles, st, launches);
  return launch_many<8>(y, x, w, out, M, N, K, lw, max_tiles, st, launches);
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

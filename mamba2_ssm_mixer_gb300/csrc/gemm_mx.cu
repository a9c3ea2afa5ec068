// Tensor-core GEMMs on microscaled 4-bit operands: y = A . B^T with A [M, K]
// and B [N, K] in MXFP4 (e2m1 codes K-major, two to a byte; scale tiles as
// mxfp4.cu lays them out), f32 accumulation in TMEM, y bf16 or f32.
// tcgen05.mma kind::mxf4 takes 64 values (32 bytes) of K per instruction and
// the blocks' scales from TMEM, where tcgen05.cp puts them from shared memory:
// a stage of 256 values (128 swizzled bytes a row) is 4 MMAs and one 512-byte
// copy per 128 rows of each operand and 128 values.  Copies and MMAs of one
// thread run in the order issued, so one set of scale columns serves every
// stage.
//
// k_mx_pair (more than 64 rows): persistent two-CTA clusters on 256-row output
//   tiles, as the e4m3 kernel of gemm_tc.cu; each CTA keeps the scales of its
//   own 128 rows of A and of all of the tile's columns.
// k_mx_fewrow (up to 64 rows): the weights are the MMA's 128-row operand, K
//   is split over the CTAs of a cluster and the partial sums meet in
//   distributed shared memory.
// k_mx_stream (up to 64 rows, many columns): the same tiles, unsplit, on
//   persistent CTAs.
// Waits are bounded as in gemm_tc.cu.
#include <cudaTypedefs.h>

#include <map>
#include <mutex>
#include <tuple>
#include <type_traits>

#include "gemm.h"
#include "launch_util.h"
#include "m2_common.cuh"
#include "mxfp4.cuh"
#include "tc_ptx.cuh"

namespace m2 {

using namespace tc;

namespace {

constexpr int kBM = 128;         // MMA rows per CTA
constexpr int kRowBytes = 128;   // bytes of K per stage and row
constexpr int kBK = 256;         // values of K per stage
constexpr int kThreads = 192;    // 6 warps: producer, MMA, 4 x epilogue
constexpr uint32_t kSfTile = 512;
constexpr int kInsideStages = 12, kInsideThreads = kThreads + 128;   // (the form that quantises X itself)

// Tiles of 128 rows of scales that a tile of `width` columns lies in: it starts
// on a multiple of 64, tiles of 128 on their own width.
__host__ __device__ constexpr int sb_tiles(int width) { return width == 128 ? 1 : (width + 64 + 127) / 128; }

struct __align__(8) Ctl {
  uint64_t full[8];
  uint64_t empty[8];
  uint64_t tfull[2];
  uint64_t tempty[2];
  uint64_t drain;
  uint64_t xfull[kInsideStages];   // the stages of X that the kernel quantises itself
  uint32_t tmem_base;
  int abort;
};

__device__ __forceinline__ void raise_abort(Ctl* ctl, int* err) {
  *reinterpret_cast<volatile int*>(&ctl->abort) = 1;
  if (err) atomicOr(err, kErrTimeout);
}

// go(steps) with as many 64-value steps (at most 4) as `left` values of K take.
// The choice is made outside the issuing lane's code: conditions in there keep
// its operands out of uniform registers (4 MMAs of N = 192: 474 clocks
// instead of 384).
template <class Go>
__device__ __forceinline__ void by_steps(int left, Go& go) {
  if (left > 192)
    go(std::integral_constant<int, 4>());
  else if (left > 128)
    go(std::integral_constant<int, 3>());
  else if (left > 64)
    go(std::integral_constant<int, 2>());
  else
    go(std::integral_constant<int, 1>());
}

// Output staging: two buffers per epilogue warp, 32 rows of 128 bytes each in
// the 128-byte swizzle of the output tensor map.
constexpr uint32_t kEpiBuf = 32 * 128;
constexpr uint32_t kEpiBytes = 4 * 2 * kEpiBuf;

template <bool kF32>
struct Out;
template <>
struct Out<false> {
  using T = uint16_t;
  static constexpr int kCols = 64;   // columns of a 128-byte slice
  __device__ static T one(uint32_t v) { return f2bfbits(__uint_as_float(v)); }
};
template <>
struct Out<true> {
  using T = float;
  static constexpr int kCols = 32;
  __device__ static T one(uint32_t v) { return __uint_as_float(v); }
};

// One epilogue warp: 32 accumulator lanes (output rows row0 ..) over the
// tile's BN columns from TMEM column `tcol`, output column n0.  With a store
// map, 128-byte slices go through shared memory and TMA stores; else 32 x 32
// pieces do, transposed, so that a warp writes a row's consecutive elements
// (517 x 5003 x 1056 f32: 11.5 us, rows written by a thread each 35.5).
template <bool kF32>
__device__ __forceinline__ void epilogue_rows(int BN, uint32_t tcol, uint8_t* bufs, int& buf, const CUtensorMap* tmC,
                                              bool tma_store, typename Out<kF32>::T* __restrict__ C, int M, int N,
                                              int row0, int n0, int lane) {
  using O = Out<kF32>;
  if (tma_store) {
#pragma unroll 1
    for (int c = 0; c < BN; c += O::kCols) {
      // slices outside the output are neither staged nor stored: each staged
      // buffer is followed by its store, which the read wait below counts on
      // (warp-uniform)
      if (row0 >= M || n0 + c >= N) break;
      uint32_t r[O::kCols];
#pragma unroll
      for (int h = 0; h < O::kCols; h += 32)
        tmem_ld_32x32b_x32(tcol + (uint32_t)(c + h), *reinterpret_cast<uint32_t(*)[32]>(&r[h]));
      tmem_ld_wait();
      uint8_t* b = bufs + buf * kEpiBuf;
      if (lane == 0) bulk_wait_read<1>();
      __syncwarp();
      const uint32_t row_addr = smem_u32(b) + (uint32_t)lane * 128u;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t at = row_addr + (uint32_t)((j ^ (lane & 7)) << 4);
        if constexpr (kF32) {
          st_shared_v4(at, r[4 * j], r[4 * j + 1], r[4 * j + 2], r[4 * j + 3]);
        } else {
          const uint32_t* v = &r[8 * j];
          st_shared_v4(at, pack_bf16x2(__uint_as_float(v[0]), __uint_as_float(v[1])),
                       pack_bf16x2(__uint_as_float(v[2]), __uint_as_float(v[3])),
                       pack_bf16x2(__uint_as_float(v[4]), __uint_as_float(v[5])),
                       pack_bf16x2(__uint_as_float(v[6]), __uint_as_float(v[7])));
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        tma_store_2d(tmC, b, n0 + c, row0);
        bulk_commit();
      }
      buf ^= 1;
    }
    return;
  }
  uint32_t* piece = reinterpret_cast<uint32_t*>(bufs);   // word (row, column) at row 32 + (column ^ row)
#pragma unroll 1
  for (int c = 0; c < BN; c += 32) {
    if (row0 >= M || n0 + c >= N) break;
    uint32_t r[32];
    tmem_ld_32x32b_x32(tcol + (uint32_t)c, r);
    tmem_ld_wait();
#pragma unroll
    for (int j = 0; j < 32; ++j) piece[lane * 32 + (j ^ lane)] = r[j];
    __syncwarp();
    const int n = n0 + c + lane, rows = min(32, M - row0);
    if (n < N) {
      typename O::T* col = C + (size_t)row0 * N + n;
#pragma unroll 8
      for (int j = 0; j < rows; ++j) col[(size_t)j * N] = O::one(piece[j * 32 + (lane ^ j)]);
    }
    __syncwarp();
  }
}

}  // namespace

// ---------------------------------------------------------------------------
// Tiles of 256 rows on CTA pairs.  CTA r of a pair stages rows [128 r, ..) of A
// with their scales, half of the tile's columns of B and the scales of all of
// them (sb_tiles of 128 rows: a tile may start in the middle of one, and the MMA
// then reads from its third column on).  The two accumulators may differ in
// width (W0, W1): a pair's unit is then a tile of each, side by side; 256 + 192
// columns and the scales are what TMEM holds.  The rest as k_gemm_pair.
// Bound by the bytes into an SM: 8192 x 10304 x 2688 takes 82 us (5.5 PFLOP/s), at
// 55 bytes a clock and SM for operands and output; the MMAs alone take 48 at
// their 128 and 96 clocks, with the loads but no stores 68.  192 columns in both
// accumulators: 84 (5669 x 2688 x 4096: 24.4 us, 22.3 with 256 + 192).  256 in
// both, sharing 24 columns: 88, a bubble of 2000 clocks a tile.  Clusters of two
// pairs that share A or B by multicast: 85 (fewer bytes out of L2, the same into
// an SM, and only 36 such clusters fit).  256-bit stores from the registers
// instead of staged ones: 85.
// ---------------------------------------------------------------------------
template <int W0, int W1, int STAGES, bool kF32>
__global__ void __launch_bounds__(kThreads, 1)
    k_mx_pair(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB0,
              const __grid_constant__ CUtensorMap tmB1,
              const __grid_constant__ CUtensorMap tmSA, const __grid_constant__ CUtensorMap tmSB,
              const __grid_constant__ CUtensorMap tmC, int tma_store, typename Out<kF32>::T* __restrict__ C, int M, int N,
              int K, int* err) {
  static_assert(STAGES <= 8, "STAGES");
  constexpr int kPM = 2 * kBM;
  constexpr int kSub = W0 == W1 ? 1 : 2, kSpan = W0 == W1 ? W0 : W0 + W1;   // tiles and columns of a unit
  constexpr uint32_t A_BYTES = kBM * kRowBytes;
  constexpr uint32_t B_BYTES = (W0 / 2) * kRowBytes;
  constexpr uint32_t SA_BYTES = 2 * kSfTile;          // 128 rows x 256 values
  constexpr int kSbTiles = sb_tiles(W0);
  constexpr uint32_t SB_BYTES = kSbTiles * 2 * kSfTile;
  constexpr uint32_t STAGE_BYTES = A_BYTES + B_BYTES + SA_BYTES + SB_BYTES;
  static_assert(W0 >= W1 && kSpan % 64 == 0 && W0 % 64 == 0, "a tile's columns start on half a scale tile");
  static_assert(STAGE_BYTES % 1024 == 0 && B_BYTES % 1024 == 0, "operand tiles on 1024-byte boundaries");
  constexpr uint32_t TMEM_COLS = 512;
  constexpr uint32_t SFA_COL = W0 + W1, SFB_COL = SFA_COL + 8;   // 2 x 4 and 2 x 4 kSbTiles columns
  static_assert(SFB_COL + 8 * kSbTiles <= TMEM_COLS, "scale columns");
  constexpr uint16_t kPair = 0x3;

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_align<1024>(smem_raw);
  uint8_t* epi = smem + STAGES * STAGE_BYTES;
  Ctl* ctl = reinterpret_cast<Ctl*>(epi + kEpiBytes);
  volatile int* abort = &ctl->abort;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  const int tiles_m = (M + kPM - 1) / kPM, tiles_n = (N + kSpan - 1) / kSpan;
  const int num_units = tiles_m * tiles_n;
  const int kblocks = (K + kBK - 1) / kBK;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&ctl->full[s], 1);
      mbar_init(&ctl->empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl->tfull[i], 1);
      mbar_init(&ctl->tempty[i], 2 * 4);
    }
    mbar_init(&ctl->drain, 1);
    ctl->abort = 0;
    fence_mbar_init();
    tma_prefetch(&tmA);
    tma_prefetch(&tmB0);
    if (kSub == 2) tma_prefetch(&tmB1);
    tma_prefetch(&tmSA);
    tma_prefetch(&tmSB);
    if (tma_store) tma_prefetch(&tmC);
  }
  if (warp == 1) {
    tmem_alloc_pair(&ctl->tmem_base, TMEM_COLS);
    tc_fence_before();
  }
  __syncwarp();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem_base = ctl->tmem_base;
  pdl_wait();
  pdl_trigger();

  if (warp == 0) {
    // ---------------- TMA producer (both CTAs): the warp loops, one lane issues
    const bool lead = elect_one();
    int stage = 0;
    uint32_t phase = 0;
    int issued = 0;   // stages requested
    bool ok = true;
    for (int unit = pair; unit < num_units && ok; unit += npairs) {
      const int m0 = (unit % tiles_m) * kPM + (int)rank * kBM;
      for (int sub = 0; sub < kSub && ok; ++sub) {
        const int width = sub ? W1 : W0;
        const int nt = (unit / tiles_m) * kSpan + sub * W0, n0 = nt + (int)rank * (width / 2);
        for (int kb = 0; kb < kblocks; ++kb) {
          if (!__all_sync(0xffffffffu, mbar_wait(&ctl->empty[stage], phase ^ 1u, abort))) {
            if (lead) raise_abort(ctl, err);
            ok = false;
            break;
          }
          if (lead) {
            uint8_t* sA = smem + stage * STAGE_BYTES;
            const uint32_t full0 = cluster_map(smem_u32(&ctl->full[stage]), 0);
            if (rank == 0)
              mbar_expect_tx(&ctl->full[stage], 2 * (STAGE_BYTES - (uint32_t)(W0 - width) / 2 * kRowBytes));
            tma_load_2d_pair(sA, &tmA, full0, kb * kRowBytes, m0);
            tma_load_2d_pair(sA + A_BYTES, sub ? &tmB1 : &tmB0, full0, kb * kRowBytes, n0);
            // (the maps of the scales are in 4-byte words: 256 words = two tiles)
            tma_load_2d_pair(sA + A_BYTES + B_BYTES, &tmSA, full0, kb * 256, m0 / 128);
            tma_load_2d_pair(sA + A_BYTES + B_BYTES + SA_BYTES, &tmSB, full0, kb * 256, nt / 128);
          }
          __syncwarp();
          ++issued;
          if (++stage == STAGES) stage = 0, phase ^= 1u;
        }
      }
    }
    // before the CTA may exit: every stage's last MMA commit has arrived on
    // its empty barrier; after an abort, the copies in flight have landed (the
    // even CTA's full barriers count both CTAs')
    for (int i = issued > STAGES ? issued - STAGES : 0; i < issued; ++i) {
      const int s = i % STAGES;
      const uint32_t ph = (uint32_t)(i / STAGES) & 1u;
      if (!*abort) {
        if (!mbar_wait(&ctl->empty[s], ph, abort) && lead) raise_abort(ctl, err);
      } else if (rank == 0) {
        mbar_wait(&ctl->full[s], ph, nullptr, 100000000ull);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (rank == 0) {
      // ---------------- MMA issuer (even CTA only): the warp loops, one lane issues
      const bool lead = elect_one();
      int stage = 0;
      uint32_t phase = 0;
      int acc = 0;
      uint32_t acc_phase = 0;
      // one tile of `width` columns
      auto tile = [&](auto width, int nt) {
        constexpr int kW = decltype(width)::value;
        if (!__all_sync(0xffffffffu, mbar_wait_cluster(&ctl->tempty[acc], acc_phase ^ 1u, abort))) {
          if (lead) raise_abort(ctl, err);
          return false;
        }
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + (uint32_t)acc * W0;
        const uint32_t sfb0 = tmem_base + SFB_COL + (uint32_t)(nt % 128) / 32;
        for (int kb = 0; kb < kblocks; ++kb) {
          if (!__all_sync(0xffffffffu, mbar_wait(&ctl->full[stage], phase, abort))) {
            if (lead) raise_abort(ctl, err);
            return false;
          }
          tc_fence_after();
          const uint32_t a_addr = smem_u32(smem + stage * STAGE_BYTES);
          const uint32_t sf_addr = a_addr + A_BYTES + B_BYTES;
          const uint64_t adesc = desc_kmajor_sw128(a_addr);
          const uint64_t bdesc = desc_kmajor_sw128(a_addr + A_BYTES);
          // the stage's first n MMAs and their scales
          auto issue = [&](auto n) {
            if (lead) {
              constexpr int kN = decltype(n)::value;
#pragma unroll
              for (int t = 0; t < (kN + 1) / 2; ++t) {   // the scales of 128 values each
                tmem_cp_32x128b_pair(tmem_base + SFA_COL + 4 * t, desc_scale_tile(sf_addr + t * kSfTile));
#pragma unroll
                for (int q = 0; q < sb_tiles(kW); ++q)
                  tmem_cp_32x128b_pair(tmem_base + SFB_COL + 4 * (kSbTiles * t + q),
                                       desc_scale_tile(sf_addr + SA_BYTES + (2 * q + t) * kSfTile));
              }
#pragma unroll
              for (int i = 0; i < kN; ++i)
                mma_mxf4_pair(d_tmem, adesc + 2 * i, bdesc + 2 * i, idesc_mxf4(kPM, kW, 2 * (i % 2)),
                              tmem_base + SFA_COL + 4 * (i / 2), sfb0 + 4 * kSbTiles * (i / 2), (kb | i) != 0);
              mma_commit_pair(&ctl->empty[stage], kPair);
            }
          };
          by_steps(K - kb * kBK, issue);
          __syncwarp();
          if (++stage == STAGES) stage = 0, phase ^= 1u;
        }
        if (lead) mma_commit_pair(&ctl->tfull[acc], kPair);
        __syncwarp();
        if (++acc == 2) acc = 0, acc_phase ^= 1u;
        return true;
      };
      for (int unit = pair; unit < num_units; unit += npairs) {
        const int nt = (unit / tiles_m) * kSpan;
        if (!tile(std::integral_constant<int, W0>(), nt)) break;
        if constexpr (kSub == 2)
          if (!tile(std::integral_constant<int, W1>(), nt + W0)) break;
      }
      if (*abort && lead) {
        mma_commit_pair(&ctl->drain, kPair);
        mbar_wait(&ctl->drain, 0, nullptr, 100000000ull);
      }
      __syncwarp();
    }
  } else {
    // ---------------- epilogue (both CTAs): warps 2..5 own TMEM lane quarters (warp % 4)
    const int quarter = warp & 3;
    const uint32_t tempty0[2] = {cluster_map(smem_u32(&ctl->tempty[0]), 0),
                                 cluster_map(smem_u32(&ctl->tempty[1]), 0)};
    uint8_t* bufs = epi + quarter * 2 * kEpiBuf;
    int buf = 0;
    int acc = 0;
    uint32_t acc_phase = 0;
    bool ok = true;
    for (int unit = pair; unit < num_units && ok; unit += npairs)
      for (int sub = 0; sub < kSub; ++sub) {
        const int m0 = (unit % tiles_m) * kPM + (int)rank * kBM, n0 = (unit / tiles_m) * kSpan + sub * W0;
        if (!__all_sync(0xffffffffu, mbar_wait(&ctl->tfull[acc], acc_phase, abort))) {
          raise_abort(ctl, err);
          ok = false;
          break;
        }
        tc_fence_after();
        epilogue_rows<kF32>(sub ? W1 : W0, tmem_base + ((uint32_t)(quarter * 32) << 16) + (uint32_t)acc * W0, bufs, buf, &tmC,
                            tma_store != 0, C, M, N, m0 + quarter * 32, n0, lane);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(tempty0[acc]);
        if (++acc == 2) acc = 0, acc_phase ^= 1u;
      }
    if (lane == 0) bulk_wait<0>();
  }
  __syncwarp();
  __syncthreads();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, TMEM_COLS);
  }
}

// ---------------------------------------------------------------------------
// Few rows: D^T[n, m] = W X^T for one 128-row block of W per cluster, K split
// over its CTAs, as k_gemm_fewrow.  w_early: W and its scales are not written
// by the kernel before this one in the stream, so the first stages of them are
// requested before waiting for it.  kInside: X is bf16 and the epilogue's warps
// quantise the CTA's part of it into shared memory first, while W arrives (one
// launch and no workspace).  2688 -> 10304, 1 row: 5.25 us, the quantisation by
// itself before it 5.7; 4096 -> 2688, 64 rows: 9.1 and 7.8, but an eager call
// takes 9 us instead of 16, and the calls are the host's.
// ---------------------------------------------------------------------------
template <int BNT, int STAGES, bool kF32, bool kInside>
__global__ void __launch_bounds__(kInside ? kInsideThreads : kThreads, 1)
    k_mx_fewrow(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                const __grid_constant__ CUtensorMap tmSW, const __grid_constant__ CUtensorMap tmSX,
                const uint16_t* __restrict__ x, size_t x_stride, typename Out<kF32>::T* __restrict__ y, int Mtok, int N,
                int K, int S, int w_early, int* err) {
  static_assert(BNT % 16 == 0 && BNT >= 16 && BNT <= 64, "BNT");
  using O = Out<kF32>;
  constexpr uint32_t A_BYTES = kBM * kRowBytes;
  constexpr uint32_t B_BYTES = BNT * kRowBytes;
  constexpr uint32_t SF_BYTES = 2 * kSfTile;
  constexpr uint32_t X_BYTES = B_BYTES + SF_BYTES;                   // a stage of X with its scales
  constexpr uint32_t STAGE_BYTES = A_BYTES + SF_BYTES + (kInside ? 0u : X_BYTES);   // W, its scales, X, its scales
  static_assert(STAGE_BYTES % 1024 == 0, "operand tiles on 1024-byte boundaries");
  constexpr uint32_t ACC_COLS = BNT < 32 ? 32 : BNT;
  constexpr uint32_t SFA_COL = ACC_COLS, SFB_COL = ACC_COLS + 8;
  constexpr uint32_t TMEM_COLS = BNT <= 32 ? 64 : 128;
  static_assert(SFB_COL + 8 <= TMEM_COLS, "scale columns");
  constexpr int RED_LD = BNT + 4;
  static_assert(kBM * RED_LD * 4 <= (int)(STAGES * STAGE_BYTES), "the exchange buffer fits in the ring");

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_align<1024>(smem_raw);
  const int kblocks = (K + kBK - 1) / kBK;
  uint8_t* xs = smem + STAGES * STAGE_BYTES;          // kInside: this CTA's stages of X
  Ctl* ctl = reinterpret_cast<Ctl*>(xs + (kInside ? (kblocks + S - 1) / S : 0) * X_BYTES);
  float* red = reinterpret_cast<float*>(smem);
  volatile int* abort = &ctl->abort;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = (int)cluster_ctarank();            // of the S CTAs of a weight block
  const int n0 = (int)(blockIdx.x / (unsigned)S) * kBM;
  const int kb0 = rank * kblocks / S;
  const int nk = (rank + 1) * kblocks / S - kb0;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&ctl->full[s], 1);
      mbar_init(&ctl->empty[s], 1);
    }
    mbar_init(&ctl->tfull[0], 1);
    mbar_init(&ctl->drain, 1);
    if (kInside)
      for (int i = 0; i < kInsideStages; ++i) mbar_init(&ctl->xfull[i], (kInsideThreads - 64) / 32);
    ctl->abort = 0;
    fence_mbar_init();
    tma_prefetch(&tmW);
    tma_prefetch(&tmSW);
    if (!kInside) {
      tma_prefetch(&tmX);
      tma_prefetch(&tmSX);
    }
  }
  if (warp == 1) {
    tmem_alloc(&ctl->tmem_base, TMEM_COLS);
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = ctl->tmem_base;

  if (warp == 0) {
    if (lane == 0) {
      // ---------------- TMA producer: ring slot i holds k-block kb0 + i
      const int npre = nk < STAGES ? nk : STAGES;
      auto load_w = [&](int i) {
        uint8_t* s = smem + (i % STAGES) * STAGE_BYTES;
        uint64_t* bar = &ctl->full[i % STAGES];
        mbar_expect_tx(bar, STAGE_BYTES);
        tma_load_2d(s, &tmW, bar, (kb0 + i) * kRowBytes, n0);
        tma_load_2d(s + A_BYTES, &tmSW, bar, (kb0 + i) * 256, n0 / 128);
      };
      auto load_x = [&](int i) {
        if (kInside) return;
        uint8_t* s = smem + (i % STAGES) * STAGE_BYTES;
        uint64_t* bar = &ctl->full[i % STAGES];
        tma_load_2d(s + A_BYTES + SF_BYTES, &tmX, bar, (kb0 + i) * kRowBytes, 0);
        tma_load_2d(s + A_BYTES + SF_BYTES + B_BYTES, &tmSX, bar, (kb0 + i) * 256, 0);
      };
      if (w_early)
        for (int i = 0; i < npre; ++i) load_w(i);
      pdl_wait();
      pdl_trigger();
      for (int i = 0; i < npre; ++i) {
        if (!w_early) load_w(i);
        load_x(i);
      }
      int issued = npre;
      for (int i = npre; i < nk; ++i) {
        if (!mbar_wait(&ctl->empty[i % STAGES], ((uint32_t)(i / STAGES) & 1u) ^ 1u, abort)) {
          raise_abort(ctl, err);
          break;
        }
        load_w(i);
        load_x(i);
        issued = i + 1;
      }
      if (*abort)   // let the copies in flight land before the CTA can exit
        for (int j = issued > STAGES ? issued - STAGES : 0; j < issued; ++j)
          mbar_wait(&ctl->full[j % STAGES], (uint32_t)(j / STAGES) & 1u, nullptr, 100000000ull);
    }
  } else {
    pdl_wait();
    pdl_trigger();
    if (warp == 1) {
      // ---------------- MMA issuer: the warp loops, one lane issues
      const bool lead = elect_one();
      bool ok = true;
      int stg = 0;
      uint32_t phase = 0;
      for (int i = 0; i < nk; ++i) {
        if (!__all_sync(0xffffffffu, (!kInside || mbar_wait(&ctl->xfull[i], 0, abort)) &&
                                         mbar_wait(&ctl->full[stg], phase, abort))) {
          if (lead) raise_abort(ctl, err);
          ok = false;
          break;
        }
        tc_fence_after();
        const uint32_t a_addr = smem_u32(smem + stg * STAGE_BYTES);
        const uint32_t sf_addr = a_addr + A_BYTES;
        const uint32_t x_addr = kInside ? smem_u32(xs + i * X_BYTES) : sf_addr + SF_BYTES;
        const uint64_t adesc = desc_kmajor_sw128(a_addr);
        const uint64_t bdesc = desc_kmajor_sw128(x_addr);
        auto issue = [&](auto n) {
          if (lead) {
            constexpr int kN = decltype(n)::value;
#pragma unroll
            for (int t = 0; t < (kN + 1) / 2; ++t) {
              tmem_cp_32x128b(tmem_base + SFA_COL + 4 * t, desc_scale_tile(sf_addr + t * kSfTile));
              tmem_cp_32x128b(tmem_base + SFB_COL + 4 * t, desc_scale_tile(x_addr + B_BYTES + t * kSfTile));
            }
#pragma unroll
            for (int j = 0; j < kN; ++j)
              mma_mxf4(tmem_base, adesc + 2 * j, bdesc + 2 * j, idesc_mxf4(kBM, BNT, 2 * (j % 2)),
                       tmem_base + SFA_COL + 4 * (j / 2), tmem_base + SFB_COL + 4 * (j / 2), (i | j) != 0);
            mma_commit(&ctl->empty[stg]);
          }
        };
        by_steps(K - (kb0 + i) * kBK, issue);
        __syncwarp();
        if (++stg == STAGES) stg = 0, phase ^= 1u;
      }
      if (lead) {
        if (ok && nk > 0) {
          mma_commit(&ctl->tfull[0]);
        } else {
          mma_commit(&ctl->drain);
          mbar_wait(&ctl->drain, 0, nullptr, 100000000ull);
        }
      }
      __syncwarp();
    } else {
      if constexpr (kInside) {
        // ---------------- warps 2..9 quantise: 16 values a thread, 16 rows of a stage at a time
        constexpr int kRows = (kInsideThreads - 64) / 16, kSub = BNT / kRows, kBatch = 8;   // (a batch's loads under way together)
        const int t = threadIdx.x - 64, c = t & 15;
        for (int j0 = 0; j0 < nk * kSub; j0 += kBatch) {
          uint4 v[kBatch][2];
#pragma unroll
          for (int b = 0; b < kBatch; ++b) {
            const int j = j0 + b, row = j % kSub * kRows + (t >> 4), k = (kb0 + j / kSub) * kBK + c * 16;
            v[b][0] = v[b][1] = make_uint4(0u, 0u, 0u, 0u);
            if (j < nk * kSub && row < Mtok && k < K) {
              const uint4* p = reinterpret_cast<const uint4*>(x + (size_t)row * x_stride + k);
              v[b][0] = __ldg(p);
              v[b][1] = __ldg(p + 1);
            }
          }
#pragma unroll
          for (int b = 0; b < kBatch; ++b) {
            const int j = j0 + b, row = j % kSub * kRows + (t >> 4);
            if (j >= nk * kSub) break;
            uint32_t code;
            const uint2 q = quant16(v[b], &code);
            uint8_t* st = xs + j / kSub * X_BYTES;
            // as TMA writes 128-byte rows in the 128-byte swizzle
            *reinterpret_cast<uint2*>(st + row * 128 + (((c >> 1) ^ (row & 7)) << 4) + (c & 1) * 8) = q;
            if (!(c & 1)) st[B_BYTES + (c >> 3) * kSfTile + (row & 31) * 16 + (row >> 5) * 4 + ((c & 7) >> 1)] = (uint8_t)code;
            if ((j + 1) % kSub == 0) {
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) mbar_arrive(&ctl->xfull[j / kSub]);
            }
          }
        }
      }
      // ---------------- epilogue warps 2..5: accumulator rows -> own exchange buffer
      if (!kInside || warp < 6) {
        const int quarter = warp & 3;
        float* dst = red + (quarter * 32 + lane) * RED_LD;
        if (__all_sync(0xffffffffu, nk > 0 && mbar_wait(&ctl->tfull[0], 0, abort))) {
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < BNT; c += 16) {
            uint32_t r[16];
            tmem_ld_32x32b_x16(tmem_base + ((uint32_t)(quarter * 32) << 16) + (uint32_t)c, r);
            tmem_ld_wait();
#pragma unroll
            for (int q = 0; q < 4; ++q)
              *reinterpret_cast<float4*>(dst + c + 4 * q) =
                  make_float4(__uint_as_float(r[4 * q]), __uint_as_float(r[4 * q + 1]), __uint_as_float(r[4 * q + 2]),
                              __uint_as_float(r[4 * q + 3]));
          }
          tc_fence_before();
        } else {
          if (nk > 0) raise_abort(ctl, err);
          for (int c = 0; c < BNT; c += 4) *reinterpret_cast<float4*>(dst + c) = make_float4(0.f, 0.f, 0.f, 0.f);
        }
      }
    }
  }
  __syncwarp();
  cluster_sync();   // every CTA's partial sits in its exchange buffer
  {
    const int r0 = rank * kBM / S, rows = (rank + 1) * kBM / S - r0;
    const int quads = (Mtok + 3) >> 2;
    const uint32_t red_s = smem_u32(red);
    for (int idx = threadIdx.x; idx < rows * quads; idx += kInside ? kInsideThreads : kThreads) {
      const int nl = r0 + idx % rows, m = 4 * (idx / rows);
      const uint32_t off = red_s + (uint32_t)((nl * RED_LD + m) * 4);
      float4 v[8];
#pragma unroll
      for (int r = 0; r < 8; ++r)
        if (r < S) v[r] = ld_dsmem_f32x4(cluster_map(off, (uint32_t)r));
      float4 acc = v[0];
#pragma unroll
      for (int r = 1; r < 8; ++r)
        if (r < S) acc.x += v[r].x, acc.y += v[r].y, acc.z += v[r].z, acc.w += v[r].w;
      const int n = n0 + nl;
      if (n < N) {
        typename O::T* yc = y + (size_t)m * N + n;
        yc[0] = O::one(__float_as_uint(acc.x));
        if (m + 1 < Mtok) yc[N] = O::one(__float_as_uint(acc.y));
        if (m + 2 < Mtok) yc[2 * (size_t)N] = O::one(__float_as_uint(acc.z));
        if (m + 3 < Mtok) yc[3 * (size_t)N] = O::one(__float_as_uint(acc.w));
      }
    }
  }
  cluster_sync();   // no CTA leaves while another still reads its buffer
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, TMEM_COLS);
  }
}

// ---------------------------------------------------------------------------
// Few rows against many weights (a head): persistent CTAs walk the 128-row
// blocks of W, D^T = W X^T as above with all of K, the ring running on from
// block to block and two accumulators, so that W streams without a pause.  A
// thread of the epilogue holds one column n of y: a warp writes 32 consecutive
// elements of a row.
// ---------------------------------------------------------------------------
template <int BNT, int STAGES, bool kF32>
__global__ void __launch_bounds__(kThreads, 1)
    k_mx_stream(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                const __grid_constant__ CUtensorMap tmSW, const __grid_constant__ CUtensorMap tmSX,
                typename Out<kF32>::T* __restrict__ y, int Mtok, int N, int K, int w_early, int* err) {
  static_assert(BNT % 16 == 0 && BNT >= 16 && BNT <= 64 && STAGES <= 8, "BNT, STAGES");
  using O = Out<kF32>;
  constexpr uint32_t A_BYTES = kBM * kRowBytes;
  constexpr uint32_t B_BYTES = BNT * kRowBytes;
  constexpr uint32_t SF_BYTES = 2 * kSfTile;
  constexpr uint32_t STAGE_BYTES = A_BYTES + B_BYTES + 2 * SF_BYTES;
  static_assert(STAGE_BYTES % 1024 == 0, "operand tiles on 1024-byte boundaries");
  constexpr uint32_t ACC_COLS = BNT < 32 ? 32 : BNT;
  constexpr uint32_t SFA_COL = 2 * ACC_COLS, SFB_COL = SFA_COL + 8;
  constexpr uint32_t TMEM_COLS = BNT <= 32 ? 128 : 256;
  static_assert(SFB_COL + 8 <= TMEM_COLS, "scale columns");

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_align<1024>(smem_raw);
  Ctl* ctl = reinterpret_cast<Ctl*>(smem + STAGES * STAGE_BYTES);
  volatile int* abort = &ctl->abort;

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int blocks = (N + kBM - 1) / kBM;
  const int kblocks = (K + kBK - 1) / kBK;

  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&ctl->full[s], 1);
      mbar_init(&ctl->empty[s], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&ctl->tfull[i], 1);
      mbar_init(&ctl->tempty[i], 4);
    }
    mbar_init(&ctl->drain, 1);
    ctl->abort = 0;
    fence_mbar_init();
    tma_prefetch(&tmW);
    tma_prefetch(&tmX);
    tma_prefetch(&tmSW);
    tma_prefetch(&tmSX);
  }
  if (warp == 1) {
    tmem_alloc(&ctl->tmem_base, TMEM_COLS);
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = ctl->tmem_base;

  if (warp == 0) {
    // ---------------- TMA producer: the warp loops, one lane issues
    const bool lead = elect_one();
    auto load_w = [&](int stg, int kb, int n0) {
      uint8_t* s = smem + stg * STAGE_BYTES;
      mbar_expect_tx(&ctl->full[stg], STAGE_BYTES);
      tma_load_2d(s, &tmW, &ctl->full[stg], kb * kRowBytes, n0);
      tma_load_2d(s + A_BYTES + B_BYTES, &tmSW, &ctl->full[stg], kb * 256, n0 / 128);
    };
    auto load_x = [&](int stg, int kb) {
      uint8_t* s = smem + stg * STAGE_BYTES;
      tma_load_2d(s + A_BYTES, &tmX, &ctl->full[stg], kb * kRowBytes, 0);
      tma_load_2d(s + A_BYTES + B_BYTES + SF_BYTES, &tmSX, &ctl->full[stg], kb * 256, 0);
    };
    // the first block's first stages of W, before the wait
    const int npre = w_early ? (kblocks < STAGES ? kblocks : STAGES) : 0;
    if (lead)
      for (int i = 0; i < npre; ++i) load_w(i, i, (int)blockIdx.x * kBM);
    __syncwarp();
    pdl_wait();
    pdl_trigger();
    int stage = 0, issued = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int blk = blockIdx.x; blk < blocks && ok; blk += gridDim.x)
      for (int kb = 0; kb < kblocks; ++kb) {
        if (!__all_sync(0xffffffffu, mbar_wait(&ctl->empty[stage], phase ^ 1u, abort))) {
          if (lead) raise_abort(ctl, err);
          ok = false;
          break;
        }
        if (lead) {
          if (issued >= npre) load_w(stage, kb, blk * kBM);
          load_x(stage, kb);
        }
        __syncwarp();
        ++issued;
        if (++stage == STAGES) stage = 0, phase ^= 1u;
      }
    // after an abort, the copies in flight land before the CTA can exit
    if (*abort && lead) {
      for (int i = issued; i < npre; ++i) load_x(i, i);   // (stages whose W went out alone)
      const int last = issued > npre ? issued : npre;
      for (int i = last > STAGES ? last - STAGES : 0; i < last; ++i)
        mbar_wait(&ctl->full[i % STAGES], (uint32_t)(i / STAGES) & 1u, nullptr, 100000000ull);
    }
    __syncwarp();
  } else {
    pdl_wait();
    pdl_trigger();
    if (warp == 1) {
      // ---------------- MMA issuer: the warp loops, one lane issues
      const bool lead = elect_one();
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      for (int blk = blockIdx.x; blk < blocks && ok; blk += gridDim.x) {
        if (!__all_sync(0xffffffffu, mbar_wait(&ctl->tempty[acc], acc_phase ^ 1u, abort))) {
          if (lead) raise_abort(ctl, err);
          break;
        }
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + (uint32_t)acc * ACC_COLS;
        for (int kb = 0; kb < kblocks; ++kb) {
          if (!__all_sync(0xffffffffu, mbar_wait(&ctl->full[stage], phase, abort))) {
            if (lead) raise_abort(ctl, err);
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t a_addr = smem_u32(smem + stage * STAGE_BYTES);
          const uint32_t sf_addr = a_addr + A_BYTES + B_BYTES;
          const uint64_t adesc = desc_kmajor_sw128(a_addr);
          const uint64_t bdesc = desc_kmajor_sw128(a_addr + A_BYTES);
          auto issue = [&](auto n) {
            if (lead) {
              constexpr int kN = decltype(n)::value;
#pragma unroll
              for (int t = 0; t < (kN + 1) / 2; ++t) {
                tmem_cp_32x128b(tmem_base + SFA_COL + 4 * t, desc_scale_tile(sf_addr + t * kSfTile));
                tmem_cp_32x128b(tmem_base + SFB_COL + 4 * t, desc_scale_tile(sf_addr + SF_BYTES + t * kSfTile));
              }
#pragma unroll
              for (int j = 0; j < kN; ++j)
                mma_mxf4(d_tmem, adesc + 2 * j, bdesc + 2 * j, idesc_mxf4(kBM, BNT, 2 * (j % 2)),
                         tmem_base + SFA_COL + 4 * (j / 2), tmem_base + SFB_COL + 4 * (j / 2), (kb | j) != 0);
              mma_commit(&ctl->empty[stage]);
            }
          };
          by_steps(K - kb * kBK, issue);
          __syncwarp();
          if (++stage == STAGES) stage = 0, phase ^= 1u;
        }
        if (!ok) break;
        if (lead) mma_commit(&ctl->tfull[acc]);
        __syncwarp();
        if (++acc == 2) acc = 0, acc_phase ^= 1u;
      }
      if (*abort && lead) {
        mma_commit(&ctl->drain);
        mbar_wait(&ctl->drain, 0, nullptr, 100000000ull);
      }
      __syncwarp();
    } else {
      // ---------------- epilogue warps 2..5
      const int quarter = warp & 3;
      int acc = 0;
      uint32_t acc_phase = 0;
      for (int blk = blockIdx.x; blk < blocks; blk += gridDim.x) {
        if (!__all_sync(0xffffffffu, mbar_wait(&ctl->tfull[acc], acc_phase, abort))) {
          if (lane == 0) raise_abort(ctl, err);
          break;
        }
        tc_fence_after();
        constexpr int kStep = BNT < 32 ? 16 : 32;
        const int n = blk * kBM + quarter * 32 + lane;
        const uint32_t col = tmem_base + ((uint32_t)(quarter * 32) << 16) + (uint32_t)acc * ACC_COLS;
#pragma unroll 1
        for (int c = 0; c < Mtok; c += kStep) {
          uint32_t r[kStep];
          if constexpr (kStep == 16)
            tmem_ld_32x32b_x16(col + (uint32_t)c, r);
          else
            tmem_ld_32x32b_x32(col + (uint32_t)c, r);
          tmem_ld_wait();
          if (n < N) {
            typename O::T* yc = y + (size_t)c * N + n;
#pragma unroll
            for (int j = 0; j < kStep; ++j)
              if (c + j < Mtok) yc[(size_t)j * N] = O::one(r[j]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->tempty[acc]);
        if (++acc == 2) acc = 0, acc_phase ^= 1u;
      }
    }
  }
  __syncwarp();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, TMEM_COLS);
  }
}

// ---------------------------------------------------------------------------
// host side
// ---------------------------------------------------------------------------
namespace {

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }();
  return fn;
}

cudaError_t encode(CUtensorMap* map, CUtensorMapDataType dt, const void* base, uint64_t inner, uint64_t rows,
                   uint64_t row_bytes, uint32_t box_inner, uint32_t box_rows, CUtensorMapSwizzle swizzle,
                   CUtensorMapL2promotion promo) {
  auto fn = encode_fn();
  if (!fn) return cudaErrorNotSupported;
  cuuint64_t dims[2] = {inner, rows};
  cuuint64_t strides[1] = {row_bytes};
  cuuint32_t box[2] = {box_inner, box_rows};
  cuuint32_t estr[2] = {1, 1};
  return fn(map, dt, 2, const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, promo,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
             ? cudaSuccess
             : cudaErrorInvalidValue;
}

// Codes [rows, K / 2] bytes: boxes of box_rows x 128 bytes, 128-byte swizzle.
cudaError_t map_codes(CUtensorMap* map, const uint8_t* p, int rows, int K, int box_rows) {
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, p, (uint64_t)K / 2, rows, (uint64_t)K / 2, kRowBytes, box_rows,
                CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}
// Scale tiles as words [ceil(rows / 128), ceil(K / 128) x 128]: boxes of two
// tiles (256 values of K) by box_rows rows of tiles.
cudaError_t map_scales(CUtensorMap* map, const uint8_t* p, int rows, int K, int box_rows) {
  const uint64_t words = (uint64_t)((K + 127) / 128) * 128;
  return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT32, p, words, (rows + 127) / 128, words * 4, 256, box_rows,
                CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B);
}
// Output map: boxes of 128 bytes x 32 rows.  False when rows are not 16-byte
// aligned; the kernels then store per thread.
template <bool kF32>
bool map_out(CUtensorMap* map, void* y, int M, int N) {
  constexpr int es = kF32 ? 4 : 2;
  if (((size_t)N * es) % 16 != 0 || (reinterpret_cast<uintptr_t>(y) & 15) != 0) return false;
  return encode(map, kF32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, y, N, M, (uint64_t)N * es,
                128 / es, 32, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE) == cudaSuccess;
}

// Clusters of `size` CTAs of a kernel that fit on the device at once (found
// once per device, kernel and size).
int max_clusters(const void* kernel, int size, size_t smem, int threads = kThreads) {
  static std::mutex mu;
  static std::map<std::tuple<int, const void*, int, size_t>, int> known;
  int dev = 0;
  cudaGetDevice(&dev);
  std::lock_guard<std::mutex> lock(mu);
  auto it = known.find({dev, kernel, size, smem});
  if (it != known.end()) return it->second;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(size * device_sm_count()));
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = size;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1) {
    cudaGetLastError();
    n = device_sm_count() / size > 1 ? device_sm_count() / size : 1;
  }
  try {
    known[{dev, kernel, size, smem}] = n;
  } catch (...) {   // (no memory: asked again the next time)
  }
  return n;
}

template <int W0, int W1, int STAGES, bool kF32>
cudaError_t launch_pair(const MxOperand& a, const MxOperand& b, void* y, int M, int N, int K, int* err,
                        cudaStream_t st) {
  constexpr int kSpan = W0 == W1 ? W0 : W0 + W1;
  CUtensorMap ta, tb0, tb1, tsa, tsb, tc = {};
  cudaError_t e;
  if ((e = map_codes(&ta, a.codes, M, K, kBM)) != cudaSuccess) return e;
  if ((e = map_codes(&tb0, b.codes, N, K, W0 / 2)) != cudaSuccess) return e;
  if ((e = map_codes(&tb1, b.codes, N, K, W1 / 2)) != cudaSuccess) return e;
  if ((e = map_scales(&tsa, a.scales, M, K, 1)) != cudaSuccess) return e;
  if ((e = map_scales(&tsb, b.scales, N, K, sb_tiles(W0))) != cudaSuccess) return e;
  const int tma_store = map_out<kF32>(&tc, y, M, N) ? 1 : 0;
  const size_t smem = 1024 + (size_t)STAGES * ((kBM + W0 / 2) * kRowBytes + (2 + 2 * sb_tiles(W0)) * kSfTile) + kEpiBytes +
                      sizeof(Ctl);
  auto k = k_mx_pair<W0, W1, STAGES, kF32>;
  if ((e = ensure_smem_optin(reinterpret_cast<const void*>(k), (int)smem)) != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  const int cap = max_clusters(reinterpret_cast<const void*>(k), 2, smem);
  const long long units = (long long)((M + 2 * kBM - 1) / (2 * kBM)) * ((N + kSpan - 1) / kSpan);
  cfg.gridDim = dim3(2 * (unsigned)(units < cap ? units : cap));
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, k, ta, tb0, tb1, tsa, tsb, tc, tma_store, static_cast<typename Out<kF32>::T*>(y), M, N, K,
                            err);
}

// Over how many CTAs K is split for few rows: as many as let the clusters of
// all nb blocks of W run at once with a CTA on an SM, at most 8, with two
// stages of K each at least.  (64 rows, 4096 -> 2688, 21 blocks: 6 splits 6.0
// us, 8 splits 8.7, since 16 clusters of 8 fit.  2688 -> 10304, 81 blocks: 1
// split 7.6, 2 splits 7.9.)  Up to 16 rows a second CTA fits beside the first
// and costs nothing more: 2 splits at least (1 row, 2688 -> 10304: 4.65 us,
// unsplit 5.35).
int fewrow_splits(const void* kernel, size_t smem, int nb, int kblocks, int bnt) {
  const int sms = device_sm_count();
  int s = sms / nb;
  if (s > 8) s = 8;
  if (s > kblocks / 2) s = kblocks / 2;
  while (s > 1 && max_clusters(kernel, s, smem) < nb) --s;
  if (s < 2 && bnt <= 16 && nb < sms && kblocks >= 4) s = 2;
  return s < 1 ? 1 : s;
}

template <int BNT, int STAGES, int STREAM_STAGES, bool kF32>
cudaError_t launch_fewrow(const MxOperand& x, const MxOperand& w, void* y, int Mtok, int N, int K, bool w_early, int* err,
                          cudaStream_t st) {
  CUtensorMap tw, tx, tsw, tsx;
  cudaError_t e;
  if ((e = map_codes(&tw, w.codes, N, K, kBM)) != cudaSuccess) return e;
  if ((e = map_codes(&tx, x.codes, Mtok, K, BNT)) != cudaSuccess) return e;
  if ((e = map_scales(&tsw, w.scales, N, K, 1)) != cudaSuccess) return e;
  if ((e = map_scales(&tsx, x.scales, Mtok, K, 1)) != cudaSuccess) return e;
  const size_t smem = 1024 + (size_t)STAGES * ((kBM + BNT) * kRowBytes + 4 * kSfTile) + sizeof(Ctl);
  auto k = k_mx_fewrow<BNT, STAGES, kF32, false>;
  if ((e = ensure_smem_optin(reinterpret_cast<const void*>(k), (int)smem)) != cudaSuccess) return e;
  const int nb = (N + kBM - 1) / kBM;
  const int S = fewrow_splits(reinterpret_cast<const void*>(k), smem, nb, (K + kBK - 1) / kBK, BNT);
  if (S == 1) {
    const size_t bytes = 1024 + (size_t)STREAM_STAGES * ((kBM + BNT) * kRowBytes + 4 * kSfTile) + sizeof(Ctl);
    auto stream = k_mx_stream<BNT, STREAM_STAGES, kF32>;
    if ((e = ensure_smem_optin(reinterpret_cast<const void*>(stream), (int)bytes)) != cudaSuccess) return e;
    const int sms = device_sm_count();
    return launch_pdl(stream, dim3(nb < sms ? nb : sms), dim3(kThreads), bytes, st, tw, tx, tsw, tsx,
                      static_cast<typename Out<kF32>::T*>(y), Mtok, N, K, (int)w_early, err);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(S * nb));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = S;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, k, tw, tx, tsw, tsx, (const uint16_t*)nullptr, (size_t)0,
                            static_cast<typename Out<kF32>::T*>(y), Mtok, N, K, S, (int)w_early, err);
}

// The few-row kernel that quantises X itself: over how many CTAs K is split, 0
// where that form is not for the shape.  A CTA's quantising warps take up to 12
// pieces of 16 values a thread (beyond that the quantisation by itself, spread
// over the GPU, is faster); the clusters of all blocks of W run at once.
constexpr int kInsideRing = 4;
constexpr int inside_stages(int bnt) { return 12 * 16 / bnt < kInsideStages ? 12 * 16 / bnt : kInsideStages; }
size_t inside_smem(int bnt, int stages) {
  return 1024 + (size_t)kInsideRing * (kBM * kRowBytes + 2 * kSfTile) +
         (size_t)stages * (bnt * kRowBytes + 2 * kSfTile) + sizeof(Ctl);
}
template <int BNT>
int inside_splits(int N, int K) {
  const void* k = reinterpret_cast<const void*>(k_mx_fewrow<BNT, kInsideRing, false, true>);   // (f32's takes as much)
  const int kblocks = (K + kBK - 1) / kBK, nb = (N + kBM - 1) / kBM, sms = device_sm_count();
  if (nb >= sms) return 0;
  int s = sms / nb;
  if (s < 2 && BNT <= 16) s = 2;
  if (s > 8) s = 8;
  if (s > kblocks / 2) s = kblocks / 2 > 1 ? kblocks / 2 : 1;
  for (; s >= 1; --s) {
    const int stages = (kblocks + s - 1) / s;
    if (stages > inside_stages(BNT)) return 0;   // (fewer splits only mean more)
    const size_t smem = inside_smem(BNT, stages);
    if (ensure_smem_optin(k, (int)inside_smem(BNT, inside_stages(BNT))) != cudaSuccess) {
      cudaGetLastError();
      return 0;
    }
    if (s == 1 || (s == 2 && sms / nb < 2) || max_clusters(k, s, smem, kInsideThreads) >= nb)
      return s;
  }
  return 0;
}

template <int BNT, bool kF32>
cudaError_t launch_inside(const uint16_t* x, size_t x_stride, const MxOperand& w, void* y, int Mtok, int N, int K, int S,
                          int* err, cudaStream_t st) {
  CUtensorMap tw, tsw;
  cudaError_t e;
  if ((e = map_codes(&tw, w.codes, N, K, kBM)) != cudaSuccess) return e;
  if ((e = map_scales(&tsw, w.scales, N, K, 1)) != cudaSuccess) return e;
  auto k = k_mx_fewrow<BNT, kInsideRing, kF32, true>;
  if ((e = ensure_smem_optin(reinterpret_cast<const void*>(k), (int)inside_smem(BNT, inside_stages(BNT)))) != cudaSuccess)
    return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(S * ((N + kBM - 1) / kBM)));
  cfg.blockDim = dim3(kInsideThreads);
  cfg.dynamicSmemBytes = inside_smem(BNT, ((K + kBK - 1) / kBK + S - 1) / S);
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = S;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, k, tw, tw, tsw, tsw, x, x_stride,
                            static_cast<typename Out<kF32>::T*>(y), Mtok, N, K, S, 0, err);
}

template <bool kF32>
cudaError_t gemm_t(const MxOperand& a, const MxOperand& w, void* y, int M, int N, int K, bool w_early, int* err,
                   cudaStream_t st) {
  if (M <= 16) return launch_fewrow<16, 4, 8, kF32>(a, w, y, M, N, K, w_early, err, st);
  if (M <= 32) return launch_fewrow<32, 4, 8, kF32>(a, w, y, M, N, K, w_early, err, st);
  if (M <= 64) return launch_fewrow<64, 4, 8, kF32>(a, w, y, M, N, K, w_early, err, st);
  // (from 65 rows on, with the weights as N operand: 128 rows 2688 -> 10304 in 6.7 us, as few rows 9.1)
  // The tile widths with the shortest waves: a stage of a tile takes as long as
  // its bytes into an SM (36 + 32, 31, 26 and 22 KB).  517 x 5003 x 1056 f32: 81
  // tiles of 192 columns, two waves of 76 pairs.
  const long long tiles_m = (M + 2 * kBM - 1) / (2 * kBM), pairs = device_sm_count() / 2;
  auto cost = [&](int span, int kb) { return ((tiles_m * ((N + span - 1) / span) + pairs - 1) / pairs) * kb; };
  const long long c448 = cost(448, 68), c192 = cost(192, 31), c128 = cost(128, 26), c64 = cost(64, 22);
  if (c448 < c192 && c448 < c128 && c448 < c64) return launch_pair<256, 192, 5, kF32>(a, w, y, M, N, K, err, st);
  if (c64 < c192 && c64 < c128) return launch_pair<64, 64, 8, kF32>(a, w, y, M, N, K, err, st);
  if (c128 < c192) return launch_pair<128, 128, 7, kF32>(a, w, y, M, N, K, err, st);
  return launch_pair<192, 192, 6, kF32>(a, w, y, M, N, K, err, st);
}

}  // namespace

cudaError_t gemm_mx(const MxOperand& a, const MxOperand& w, void* y, bool f32, int M, int N, int K, bool w_early, int* err,
                    cudaStream_t st) {
  if (M <= 0) return cudaSuccess;
  return f32 ? gemm_t<true>(a, w, y, M, N, K, w_early, err, st) : gemm_t<false>(a, w, y, M, N, K, w_early, err, st);
}

int mx_inside_splits(int M, int N, int K) {
  if (M < 1 || M > 64) return 0;
  return M <= 16 ? inside_splits<16>(N, K) : M <= 32 ? inside_splits<32>(N, K) : inside_splits<64>(N, K);
}

cudaError_t gemm_mx_inside(const uint16_t* x, size_t x_stride, const MxOperand& w, void* y, bool f32, int M, int N, int K,
                           int splits, int* err, cudaStream_t st) {
  auto go = [&](auto bnt) {
    constexpr int kB = decltype(bnt)::value;
    return f32 ? launch_inside<kB, true>(x, x_stride, w, y, M, N, K, splits, err, st)
               : launch_inside<kB, false>(x, x_stride, w, y, M, N, K, splits, err, st);
  };
  if (M <= 16) return go(std::integral_constant<int, 16>());
  if (M <= 32) return go(std::integral_constant<int, 32>());
  return go(std::integral_constant<int, 64>());
}

}  // namespace m2

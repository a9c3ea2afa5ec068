// Reordering of the paged recurrent states after a beam selection.
// Row (i, j) of a batch of requests goes on from beam p = parents[i][j] of the
// same request, so its state has to be the one in slot_idx[i][p].  A gather of
// every row would read and write all of them; here the slots are renamed and
// only what cannot be renamed moves: the first row that names a beam takes
// over that beam's slot as it is, and each further one gets the slot of a beam
// that no row names, with a copy of the parent's state.  Copied-to slots are
// never copied from, so the copies are independent of each other and need no
// second buffer.  One launch does the plan and the copies of every layer's
// pools: the plan (a few integers per row) is computed by every CTA for
// itself in shared memory, which costs less than a second launch.
// Bound by moving the bytes: 23 layers x 32 copies of bf16 rows (1.6 GB) in
// 238 to 246 us, 0.97 to 1.01 of the copy rate; 32 copies of f32 rows (137 MB) in 23 us, 0.87;
// two copies 3.9 us.  Four CTAs per SM with eight loads each under way: 2, 3, 5
// and 6 CTAs took 9 to 30 us more on the first.
#include "launch_util.h"
#include "m2_kernels.h"

namespace m2 {

namespace {

constexpr int kRoThreads = 256;
constexpr int kPiece = kRoThreads * 16;             // bytes a CTA moves with one load per thread
constexpr int kAheadRo = 8;                         // pieces under way per CTA
constexpr int kConvRow = kConv * (kW - 1) * 2;      // 36864 bytes of a conv window
constexpr int kConvPieces = kConvRow / kPiece;
static_assert(kConvRow % kPiece == 0, "conv windows move in whole pieces");

struct Pools {
  uint4* conv[kReorderMaxLayers];
  uint4* ssm[kReorderMaxLayers];
};

// Position of the r-th (from 0) set bit of m; r < popc(m).
__device__ __forceinline__ int nth_bit(uint32_t m, int r) {
  for (; r > 0; --r) m &= m - 1;
  return __ffs(m) - 1;
}

__device__ __forceinline__ uint32_t slot_hash(int slot) { return (uint32_t)slot * 2654435761u; }

}  // namespace

// Shared memory: [rows] src, dst, rank of a row's copy in its request (-1:
// none), [rows] requests' first copy, and the table of named slots (keys and
// the first row naming each; 2^bits >= 2 rows entries).
__global__ void __launch_bounds__(kRoThreads) k_state_reorder(const Pools pools, int layers, int ssm_row, int n_slots,
                                                              const int32_t* __restrict__ slot_idx,
                                                              const int32_t* __restrict__ parents,
                                                              int32_t* __restrict__ new_slot, int batch, int beams,
                                                              int bits, int* err) {
  extern __shared__ int ro_smem[];
  const int rows = batch * beams, size = 1 << bits;
  int* src = ro_smem;
  int* dst = src + rows;
  int* rank = dst + rows;
  int* first_copy = rank + rows;   // [batch], then the exclusive sum
  int* key = first_copy + rows;
  int* key_row = key + size;
  __shared__ int total;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();

  // which row names each slot first
  for (int i = tid; i < size; i += kRoThreads) key[i] = -1, key_row[i] = 0x7fffffff;
  __syncthreads();
  for (int r = tid; r < rows; r += kRoThreads) {
    const int s = slot_idx[r];
    if (s < 0 || s >= n_slots) continue;
    uint32_t at = slot_hash(s) >> (32 - bits);
    for (;;) {   // at most half of the entries are taken, so a free one is met
      const int was = atomicCAS(&key[at], -1, s);
      if (was == -1 || was == s) break;
      at = (at + 1) & (size - 1);
    }
    atomicMin(&key_row[at], r);
  }
  __syncthreads();

  // one warp per request, one lane per beam
  for (int q = warp; q < batch; q += kRoThreads / 32) {
    const bool in = lane < beams;
    const int row = q * beams + lane;
    const int slot = in ? slot_idx[row] : -1;
    const int par = in ? parents[row] : -1;
    int wrong = 0;
    if (in) {
      if (slot < -1 || slot >= n_slots) wrong = kErrSlot;
      if (slot >= 0 && slot < n_slots) {
        uint32_t at = slot_hash(slot) >> (32 - bits);
        while (key[at] != slot) at = (at + 1) & (size - 1);
        if (key_row[at] < row) wrong = kErrDupSlot;
      }
      if (par < -1 || par >= beams) wrong |= kErrBeam;
    }
    const int pslot = __shfl_sync(0xffffffffu, slot, par < 0 || par >= beams ? 0 : par);
    const bool live = in && par >= 0 && par < beams;
    if (live && pslot < 0) wrong |= kErrBeam;
    const uint32_t same = __match_any_sync(0xffffffffu, live ? par : -1 - lane);
    const bool first = live && __ffs(same) - 1 == lane;
    const uint32_t named = __reduce_or_sync(0xffffffffu, live ? 1u << par : 0u);
    const uint32_t spare = __ballot_sync(0xffffffffu, in && slot >= 0 && !((named >> lane) & 1u));
    const uint32_t extra = __ballot_sync(0xffffffffu, live && !first);
    const uint32_t dead = __ballot_sync(0xffffffffu, in && !live);
    if (__popc(extra) > __popc(spare)) wrong |= kErrBeam;   // more rows than slots
    const int all_wrong = (int)__reduce_or_sync(0xffffffffu, (unsigned)wrong);
    const uint32_t below = (1u << lane) - 1u;
    // spare slots in order: to the further rows of a beam, then to rows without a beam
    const int want = live ? __popc(extra & below) : __popc(extra) + __popc(dead & below);
    const bool given = in && !first && want < __popc(spare);
    const int gslot = __shfl_sync(0xffffffffu, slot, given ? nth_bit(spare, want) : 0);
    const bool copy = live && !first && !all_wrong;
    if (in) {
      src[row] = pslot;
      dst[row] = gslot;
      rank[row] = copy ? want : -1;
      if (blockIdx.x == 0) new_slot[row] = all_wrong ? slot : first ? pslot : given ? gslot : -1;
    }
    if (lane == 0) {
      first_copy[q] = all_wrong ? 0 : __popc(extra);
      if (all_wrong && blockIdx.x == 0) atomicOr(err, all_wrong);
    }
  }
  __syncthreads();
  if (warp == 0) {   // exclusive sum over the requests
    int run = 0;
    for (int q0 = 0; q0 < batch; q0 += 32) {
      const int v = q0 + lane < batch ? first_copy[q0 + lane] : 0;
      int sum = v;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += t;
      }
      if (q0 + lane < batch) first_copy[q0 + lane] = run + sum - v;
      run += __shfl_sync(0xffffffffu, sum, 31);
    }
    if (lane == 0) total = run;
  }
  __syncthreads();
  // the list of copies, over the table of slots: (from, to)
  int2* list = reinterpret_cast<int2*>(key);
  for (int r = tid; r < rows; r += kRoThreads)
    if (rank[r] >= 0) list[first_copy[r / beams] + rank[r]] = make_int2(src[r], dst[r]);
  __syncthreads();

  // All copies' pieces in one row (a copy, its layers, in each the state row
  // then the conv window), cut into even stretches: every CTA moves the same
  // bytes to within a piece.
  const int spieces = ssm_row / kPiece, per = spieces + kConvPieces;
  static_assert((long long)kReorderMaxRows * kReorderMaxLayers * (kNH * kP * kN * 4 / kPiece + kConvPieces) < (1ll << 31),
                "pieces are counted in 32 bits");
  const uint32_t work = (uint32_t)total * layers * per;
  const uint32_t each = work / gridDim.x, more = work % gridDim.x;
  const uint32_t lo = blockIdx.x * each + min(blockIdx.x, more), hi = lo + each + (blockIdx.x < more);
  if (lo >= hi) return;
  const uint32_t row = lo / per;   // of the copies' layers
  int piece = (int)(lo - row * per), copy = (int)(row / (uint32_t)layers), layer = (int)(row - copy * layers);
  for (uint32_t w = lo; w < hi; w += kAheadRo) {
    uint4 v[kAheadRo];
    uint4* to[kAheadRo];
#pragma unroll
    for (int i = 0; i < kAheadRo; ++i) {
      if (w + i >= hi) break;
      const int2 c = list[copy];
      const bool st = piece < spieces;
      uint4* base = (st ? pools.ssm[layer] : pools.conv[layer]) + (size_t)(st ? piece : piece - spieces) * kRoThreads + tid;
      const size_t row16 = (st ? ssm_row : kConvRow) / 16;
      v[i] = base[(size_t)c.x * row16];
      to[i] = base + (size_t)c.y * row16;
      if (++piece == per) {
        piece = 0;
        if (++layer == layers) layer = 0, ++copy;
      }
    }
#pragma unroll
    for (int i = 0; i < kAheadRo; ++i)
      if (w + i < hi) *to[i] = v[i];
  }
}

cudaError_t launch_state_reorder(uint16_t* const* conv_pools, void* const* ssm_pools, int layers, bool bf16_state,
                                 int n_slots, const int32_t* slot_idx, const int32_t* parents, int32_t* new_slot,
                                 int batch, int beams, int* err, cudaStream_t st) {
  Pools p;
  for (int l = 0; l < layers; ++l) {
    p.conv[l] = reinterpret_cast<uint4*>(conv_pools[l]);
    p.ssm[l] = reinterpret_cast<uint4*>(ssm_pools[l]);
  }
  const int rows = batch * beams;
  int bits = 1;
  while ((1 << bits) < 2 * rows) ++bits;
  const int ssm_row = kNH * kP * kN * (bf16_state ? 2 : 4);
  const size_t smem = (size_t)(4 * rows + 2 * (1 << bits)) * 4;
  // the plan of the most rows (kReorderMaxRows) takes 128 KB
  cudaError_t e = ensure_smem_optin((const void*)k_state_reorder, 4 * kReorderMaxRows * 4 + 4 * kReorderMaxRows * 4);
  if (e != cudaSuccess) return e;
  const long long most = (long long)batch * (beams - 1) * layers * (ssm_row / kPiece + kConvPieces);
  long long grid = 4ll * device_sm_count();
  if (grid > most) grid = most;
  if (grid < 1) grid = 1;
  return launch_pdl(k_state_reorder, dim3((unsigned)grid), dim3(kRoThreads), smem, st, p, layers, ssm_row, n_slots,
                    slot_idx, parents, new_slot, batch, beams, bits, err);
}

}  // namespace m2

// Beam selection: for each request the k best of beams x vocabulary by
//   value(b, v) = score_b + x_bv - lse_b,   lse_b = log sum_u exp(x_bu)
// in one pass over the logits x.
//
// k_beam_rows: a CTA takes one chunk of one row, held in registers: each warp's
// maximum and sum of exponentials (online softmax, joined later), and the
// chunk's k best tokens.  The k best need no sort: if every one of the 8 warps
// has ceil(k / 8) threads whose own maximum is at least tau, then at least k
// elements of the chunk are >= tau, so only those are looked at further (for
// unordered logits a small multiple of k).  tau is the least, over the warps,
// of the warp's ceil(k / 8)-th largest thread maximum: a few warp reductions.
// The survivors are ranked by counting.  Where equal values leave more
// survivors than fit, the k best are taken one after another instead.
// k_beam_merge: a CTA per request joins the chunks' sums to lse_b, and selects
// among the chunks' survivors by the 64-bit value in the same way.
//
// Order: greater value first, then the lower beam * vocab + token.  Within a
// row the logits themselves are compared; rows are compared in 64 bits with
// lse from f32 sums in an order that depends on the token's index alone (not
// on the row's address), so equal rows get equal values and a true tie stays
// one.
#include "launch_util.h"
#include "m2_kernels.h"

namespace m2 {

namespace {

constexpr int kBeThreads = 256;
constexpr int kBeWarps = kBeThreads / 32;
constexpr int kCap = 1024;   // survivors ranked by counting

struct ChunkSum {
  float m, s;   // maximum and sum of exp(x - m) of one chunk
};

// Order-preserving map of floats to unsigned; no value maps to 0.
__device__ __forceinline__ uint32_t ord32(float f) {
  const uint32_t u = __float_as_uint(f);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unord32(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? o ^ 0x80000000u : ~o);
}
__device__ __forceinline__ uint64_t ord64(double d) {
  const uint64_t u = (uint64_t)__double_as_longlong(d);
  return u ^ ((uint64_t)((int64_t)u >> 63) | 0x8000000000000000ull);
}
__device__ __forceinline__ double unord64(uint64_t o) {
  return __longlong_as_double((long long)((o & 0x8000000000000000ull) ? o ^ 0x8000000000000000ull : ~o));
}
constexpr uint32_t kOrdNegInf = 0x007fffffu;   // ord32(-inf)

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

template <typename T>
struct Elem;   // logits: vector width and widening; + 0 makes -0 a +0 (equal logits)
template <>
struct Elem<uint16_t> {
  static constexpr int kVec = 8;
  __device__ static float load(const uint16_t* p) { return bfbits2f(*p); }
};
template <>
struct Elem<float> {
  static constexpr int kVec = 4;
  __device__ static float load(const float* p) { return *p; }
};

// 16 bytes from p, whose address may sit `off` bytes past a 16-byte boundary
// (off uniform over the row): two aligned loads and byte shifts.  Both loads
// hold at least one byte of the 16.
__device__ __forceinline__ uint4 load16(const void* p, uint32_t off) {
  const uint4* q = reinterpret_cast<const uint4*>((const char*)p - off);
  const uint4 a = __ldg(q);
  if (off == 0) return a;
  const uint4 b = __ldg(q + 1);
  const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
  const uint32_t words = off >> 2, sh = (off & 3) * 8;
  uint32_t r[5];
#pragma unroll
  for (int i = 0; i < 5; ++i) {
    r[i] = words == 0 ? w[i] : words == 1 ? w[i + 1] : words == 2 ? w[i + 2] : w[i + 3];
  }
  return make_uint4(__funnelshift_r(r[0], r[1], sh), __funnelshift_r(r[1], r[2], sh),
                    __funnelshift_r(r[2], r[3], sh), __funnelshift_r(r[3], r[4], sh));
}

__device__ __forceinline__ uint64_t warp_max64(uint64_t v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const uint64_t t = __shfl_xor_sync(0xffffffffu, v, o);
    v = t > v ? t : v;
  }
  return v;
}

}  // namespace

// VPT 16-byte vectors per thread; element e of vector j of thread t is token
// chunk * 256 VPT kVec + (256 j + t) kVec + e.
template <typename T, int VPT>
__global__ void __launch_bounds__(kBeThreads) k_beam_rows(const T* __restrict__ logits, size_t stride, int vocab,
                                                          const float* __restrict__ scores,
                                                          const uint8_t* __restrict__ done, int k, int splits,
                                                          uint64_t* __restrict__ keys, ChunkSum* __restrict__ sums) {
  constexpr int V = Elem<T>::kVec, kEl = V * VPT;
  __shared__ uint64_t cand[kCap];
  __shared__ float wm[kBeWarps], ws[kBeWarps];
  __shared__ uint32_t wtau[kBeWarps];
  __shared__ int n_cand;
  pdl_wait();
  pdl_trigger();
  const int row = blockIdx.x / splits, split = blockIdx.x % splits;
  if (!isfinite(scores[row]) || (done && done[row])) return;   // no candidates here (the merge reads nothing either)
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const T* base = logits + (size_t)row * stride;
  const uint32_t off = (uint32_t)((uintptr_t)base & 15u);
  const int first = split * (kBeThreads * kEl);
  if (tid == 0) n_cand = 0;

  float x[kEl];
  float mx = -INFINITY;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int at = first + (j * kBeThreads + tid) * V;
    if (at + V <= vocab) {
      const uint4 q = load16(base + at, off);
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if constexpr (V == 8) {
          x[j * V + 2 * e] = __uint_as_float(w[e] << 16);
          x[j * V + 2 * e + 1] = __uint_as_float(w[e] & 0xFFFF0000u);
        } else {
          x[j * V + e] = __uint_as_float(w[e]);
        }
      }
    } else {
#pragma unroll
      for (int e = 0; e < V; ++e) x[j * V + e] = at + e < vocab ? Elem<T>::load(base + at + e) : -INFINITY;
    }
#pragma unroll
    for (int e = 0; e < V; ++e) mx = fmaxf(mx, x[j * V + e]);   // a NaN never is the maximum
  }
  const uint32_t om = ord32(mx + 0.f);
  const uint32_t owm = __reduce_max_sync(0xffffffffu, om);
  const float m = unord32(owm);
  float s = 0.f;
  constexpr float kLog2e = 1.4426950408889634f;
#pragma unroll
  for (int i = 0; i < kEl; ++i) s += exp2_fast((x[i] - m) * kLog2e);
  if (isnan(s)) {   // a NaN (no candidate), a row of -inf, or +inf (takes all the probability)
    s = 0.f;
#pragma unroll
    for (int i = 0; i < kEl; ++i)
      if (x[i] > -INFINITY) s += x[i] == m ? 1.f : exp2_fast((x[i] - m) * kLog2e);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  // the warp's ceil(k / 8)-th largest thread maximum
  uint32_t tau = owm, left = om;
  for (int r = (k + kBeWarps - 1) / kBeWarps; r > 1; --r) {
    const uint32_t who = __ballot_sync(0xffffffffu, left == tau);
    if (lane == __ffs(who) - 1) left = 0;
    tau = __reduce_max_sync(0xffffffffu, left);
  }
  if (lane == 0) wm[warp] = m, ws[warp] = s, wtau[warp] = tau;
  __syncthreads();
  uint32_t t = wtau[0];
#pragma unroll
  for (int i = 1; i < kBeWarps; ++i) t = min(t, wtau[i]);
  if (tid == 0) {
    float M = wm[0];
#pragma unroll
    for (int i = 1; i < kBeWarps; ++i) M = fmaxf(M, wm[i]);
    double S = 0.;
    for (int i = 0; i < kBeWarps; ++i)
      if (ws[i] > 0.f) S += (double)ws[i] * (wm[i] == M ? 1. : (double)expf(wm[i] - M));
    sums[blockIdx.x] = ChunkSum{M, (float)S};
  }
  // survivors: >= tau and above -inf
  const float low = unord32(max(t, kOrdNegInf));
  if (mx >= low && mx > -INFINITY) {
#pragma unroll
    for (int i = 0; i < kEl; ++i)
      if (x[i] >= low && x[i] > -INFINITY) {
        const int at = atomicAdd(&n_cand, 1);
        const uint32_t token = (uint32_t)(first + ((i / V) * kBeThreads + tid) * V + i % V);
        if (at < kCap) cand[at] = ((uint64_t)ord32(x[i] + 0.f) << 32) | (0xffffffffu - token);
      }
  }
  __syncthreads();
  const int n = n_cand;
  uint64_t* out = keys + (size_t)blockIdx.x * k;
  if (n <= kCap) {
    for (int i = tid; i < n; i += kBeThreads) {
      const uint64_t mine = cand[i];
      int rank = 0;
      for (int j = 0; j < n; ++j) rank += cand[j] > mine;
      if (rank < k) out[rank] = mine;
    }
    for (int i = n + tid; i < k; i += kBeThreads) out[i] = 0;
  } else {   // many equal values: the greatest key below the last one, k times
    uint64_t last = ~0ull;
    for (int r = 0; r < k; ++r) {
      uint64_t best = 0;
#pragma unroll
      for (int i = 0; i < kEl; ++i)
        if (x[i] > -INFINITY) {
          const uint32_t token = (uint32_t)(first + ((i / V) * kBeThreads + tid) * V + i % V);
          const uint64_t key = ((uint64_t)ord32(x[i] + 0.f) << 32) | (0xffffffffu - token);
          if (key < last && key > best) best = key;
        }
      best = warp_max64(best);
      __syncthreads();
      if (lane == 0) cand[warp] = best;
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kBeWarps; ++i) best = cand[i] > best ? cand[i] : best;
      if (tid == 0) out[r] = best;
      last = best;
    }
  }
}

// One request.  offs[b] = score_b - lse_b; a finished beam has one candidate.
__global__ void __launch_bounds__(1024) k_beam_merge(const uint64_t* __restrict__ keys,
                                                     const ChunkSum* __restrict__ sums, const float* scores,
                                                     const uint8_t* done, int beams, int vocab, int eos, int k,
                                                     int splits, int32_t* __restrict__ tokens,
                                                     int32_t* __restrict__ parents, float* out_scores,
                                                     uint8_t* out_done) {
  __shared__ double score[kBeamMaxBeams], lse[kBeamMaxBeams];
  __shared__ float top[kBeamMaxBeams];      // the row's maximum (+inf: lse holds the log of their count)
  __shared__ int kind[kBeamMaxBeams];       // 0: no candidates, 1: live, 2: finished
  __shared__ uint64_t wtau[32], cval[kCap], cflat[kCap];
  __shared__ int n_cand;
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = blockDim.x >> 5;
  const int row0 = blockIdx.x * beams;
  if (tid == 0) n_cand = 0;
  for (int b = warp; b < beams; b += nw) {
    const float sc = scores[row0 + b];
    const bool fin = done && done[row0 + b];
    if (!isfinite(sc) || fin) {
      if (lane == 0) kind[b] = isfinite(sc) ? 2 : 0, score[b] = (double)sc;
      continue;
    }
    const ChunkSum* cs = sums + (size_t)(row0 + b) * splits;
    float m = -INFINITY;
    for (int i = lane; i < splits; i += 32) m = fmaxf(m, cs[i].m);
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    double s = 0.;
    for (int i = lane; i < splits; i += 32) {
      const ChunkSum c = cs[i];
      if (c.s > 0.f) s += c.m == m ? (double)c.s : (double)c.s * exp((double)c.m - (double)m);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) {
      kind[b] = s > 0. ? 1 : 0;
      top[b] = m;
      score[b] = (double)sc;
      lse[b] = isinf(m) ? log(s) : (double)m + log(s);
    }
  }
  __syncthreads();

  const int per = splits * k, total = beams * per;
  // candidate i: its ordered 64-bit value (0: none) and beam * vocab + token
  auto candidate = [&](int i, uint64_t* flat) -> uint64_t {
    const int b = i / per, j = i - b * per;
    if (kind[b] == 0) return 0;
    if (kind[b] == 2) {
      *flat = (uint64_t)b * vocab + eos;
      return j == 0 ? ord64(score[b]) : 0;
    }
    const uint64_t key = keys[(size_t)(row0 + b) * per + j];
    if (key == 0) return 0;
    const float x = unord32((uint32_t)(key >> 32));
    *flat = (uint64_t)b * vocab + (0xffffffffu - (uint32_t)key);
    if (isinf(top[b])) return x == top[b] ? ord64(score[b] - lse[b]) : 0;
    return ord64(score[b] + ((double)x - lse[b]));
  };
  uint64_t mine = 0, f = 0;
  for (int i = tid; i < total; i += blockDim.x) {
    const uint64_t v = candidate(i, &f);
    mine = v > mine ? v : mine;
  }
  uint64_t tau = warp_max64(mine);
  for (int r = (k + nw - 1) / nw; r > 1; --r) {
    const uint32_t who = __ballot_sync(0xffffffffu, mine == tau);
    if (lane == __ffs(who) - 1) mine = 0;
    tau = warp_max64(mine);
  }
  if (lane == 0) wtau[warp] = tau;
  __syncthreads();
  for (int i = 0; i < nw; ++i) tau = wtau[i] < tau ? wtau[i] : tau;
  if (tau == 0) tau = 1;
  for (int i = tid; i < total; i += blockDim.x) {
    const uint64_t v = candidate(i, &f);
    if (v >= tau) {
      const int at = atomicAdd(&n_cand, 1);
      if (at < kCap) cval[at] = v, cflat[at] = f;
    }
  }
  __syncthreads();
  const int n = n_cand;
  const size_t o0 = (size_t)blockIdx.x * k;
  auto put = [&](int rank, uint64_t v, uint64_t flat) {
    const int b = (int)(flat / vocab), token = (int)(flat % vocab);
    tokens[o0 + rank] = token;
    parents[o0 + rank] = b;
    out_scores[o0 + rank] = (float)unord64(v);
    if (out_done) out_done[o0 + rank] = (uint8_t)(kind[b] == 2 || token == eos);
  };
  auto none = [&](int rank) {
    tokens[o0 + rank] = -1;
    parents[o0 + rank] = -1;
    out_scores[o0 + rank] = -INFINITY;
    if (out_done) out_done[o0 + rank] = 0;
  };
  if (n <= kCap) {
    for (int i = tid; i < n; i += blockDim.x) {
      const uint64_t v = cval[i], fl = cflat[i];
      int rank = 0;
      for (int j = 0; j < n; ++j) rank += cval[j] > v || (cval[j] == v && cflat[j] < fl);
      if (rank < k) put(rank, v, fl);
    }
    for (int i = n + tid; i < k; i += blockDim.x) none(i);
  } else {   // many equal values: the best after the last one, k times
    uint64_t lv = ~0ull, lf = 0;
    for (int r = 0; r < k; ++r) {
      uint64_t bv = 0, bf = ~0ull;
      for (int i = tid; i < total; i += blockDim.x) {
        const uint64_t v = candidate(i, &f);
        if (v == 0 || v > lv || (v == lv && f <= lf)) continue;
        if (v > bv || (v == bv && f < bf)) bv = v, bf = f;
      }
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        const uint64_t tv = __shfl_xor_sync(0xffffffffu, bv, o), tf = __shfl_xor_sync(0xffffffffu, bf, o);
        if (tv > bv || (tv == bv && tf < bf)) bv = tv, bf = tf;
      }
      __syncthreads();
      if (lane == 0) cval[warp] = bv, cflat[warp] = bf;
      __syncthreads();
      for (int i = 0; i < nw; ++i)
        if (cval[i] > bv || (cval[i] == bv && cflat[i] < bf)) bv = cval[i], bf = cflat[i];
      if (tid == 0) {
        if (bv) put(r, bv, bf);
        else none(r);
      }
      lv = bv, lf = bf;
    }
  }
}

namespace {

// Tokens per chunk (a CTA's work): 8192, or fewer where that leaves SMs idle.
int beam_chunk(int rows, int vocab, int sms) {
  int chunk = 8192;
  while (chunk > 2048 && (long long)rows * ((vocab + chunk - 1) / chunk) < 2ll * sms) chunk /= 2;
  return chunk;
}

template <typename T, int VPT>
cudaError_t launch_rows(const void* logits, size_t stride, int rows, int vocab, const float* scores, const uint8_t* done,
                        int k, int splits, uint64_t* keys, ChunkSum* sums, cudaStream_t st) {
  return launch_pdl(k_beam_rows<T, VPT>, dim3((unsigned)(rows * splits)), dim3(kBeThreads), 0, st,
                    static_cast<const T*>(logits), stride, vocab, scores, done, k, splits, keys, sums);
}

size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

}  // namespace

size_t beam_workspace_bytes(int batch, int beams, int vocab, int k) {
  const size_t parts = (size_t)batch * beams * ((vocab + 2047) / 2048);   // the most chunks any device's rule makes
  return align256(parts * k * sizeof(uint64_t)) + align256(parts * sizeof(ChunkSum));
}

cudaError_t launch_beam_select(const void* logits, bool bf16, size_t stride, int batch, int beams, int vocab,
                               const float* scores, const uint8_t* done, int eos, int k, int32_t* tokens,
                               int32_t* parents, float* out_scores, uint8_t* out_done, void* ws, cudaStream_t st) {
  const int rows = batch * beams, chunk = beam_chunk(rows, vocab, device_sm_count());
  const int splits = (vocab + chunk - 1) / chunk;
  uint64_t* keys = static_cast<uint64_t*>(ws);
  ChunkSum* sums = reinterpret_cast<ChunkSum*>(static_cast<char*>(ws) + align256((size_t)rows * splits * k * sizeof(uint64_t)));
  cudaError_t e;
#define M2_BEAM_ROWS(T, VPT) launch_rows<T, VPT>(logits, stride, rows, vocab, scores, done, k, splits, keys, sums, st)
  if (bf16)
    e = chunk == 8192 ? M2_BEAM_ROWS(uint16_t, 4) : chunk == 4096 ? M2_BEAM_ROWS(uint16_t, 2) : M2_BEAM_ROWS(uint16_t, 1);
  else
    e = chunk == 8192 ? M2_BEAM_ROWS(float, 8) : chunk == 4096 ? M2_BEAM_ROWS(float, 4) : M2_BEAM_ROWS(float, 2);
#undef M2_BEAM_ROWS
  if (e != cudaSuccess) return e;
  const int threads = beams * splits * k > 2048 ? 1024 : 256;
  return launch_pdl(k_beam_merge, dim3((unsigned)batch), dim3(threads), 0, st, keys, sums, scores, done, beams, vocab,
                    eos, k, splits, tokens, parents, out_scores, out_done);
}

}  // namespace m2

// Beam selection: for each request the k best of beams x vocabulary by
//   value(b, v) = score_b + x_bv - lse_b,   lse_b = log sum_u exp(x_bu)
// in one pass over the logits x.
//
// k_beam_rows: a CTA takes one chunk of one row, held packed in registers: each
// warp's maximum and sum of exponentials (online softmax, joined later), and
// the chunk's k best tokens.  The k best need no sort: if every one of the 8
// warps has ceil(k / 8) threads whose own maximum is at least tau, then at
// least k elements of the chunk are >= tau, so only those are looked at further
// (for unordered logits a small multiple of k).  tau is the least, over the
// warps, of the warp's ceil(k / 8)-th largest thread maximum: a few warp
// reductions.  The survivors are ranked by counting.  Where equal values leave
// more survivors than fit, the k best are taken one after another instead.
// Bound by a chunk's way through the CTA (load, sum, select: the sums alone take
// 25 us of the 33 below, issue and exp2 unit half used): 64 x 8 rows of 131072
// bf16 tokens, with the merge, in 33 us (floor 18.5); 16 KB chunks instead of
// 32 take 36 (more selections), three and six CTAs per SM instead of four 37
// and 43.  A CTA over several chunks that keeps its list from one to the next
// took 47 to 64, a first form that kept the row unpacked in registers and
// summed in f64 181.
// k_beam_merge: a CTA per request joins the chunks' sums of a row, and selects
// among the chunks' survivors by the 64-bit value in the same way.
//
// Order: greater value first, then the lower beam * vocab + token.  Within a
// row the logits themselves are compared; rows are compared in 64 bits with
// lse from f32 sums in an order that depends on the token's index alone (not
// on the row's address), so equal rows get equal values and a true tie stays
// one.
#include <type_traits>

#include "launch_util.h"
#include "m2_kernels.h"

namespace m2 {

namespace {

constexpr int kBeThreads = 256;
constexpr int kBeWarps = kBeThreads / 32;
constexpr int kCap = 1024;   // survivors ranked by counting
constexpr int kCapV = 64;    // a warp's vectors with survivors among their elements
constexpr int kRankStep = 8; // keys a ranking thread compares per step

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

// f32 pairs in one 64-bit register: one instruction for two lanes' worth.
__device__ __forceinline__ uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float2 unpair(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma_pair(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t mul_pair(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t add_pair(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

// Logits in 16-byte vectors, kept packed in registers.  Maxima ignore NaN.
template <typename T>
struct Elem;
template <>
struct Elem<uint16_t> {
  static constexpr int kVec = 8;
  static constexpr uint32_t kNegInf = 0xFF80FF80u;
  __device__ static float load(const uint16_t* p) { return bfbits2f(*p); }
  __device__ static float at(const uint4& q, int e) {
    const uint32_t w = e < 2 ? q.x : e < 4 ? q.y : e < 6 ? q.z : q.w;
    return __uint_as_float(e & 1 ? w & 0xFFFF0000u : w << 16);
  }
  __device__ static uint32_t max2(uint32_t a, uint32_t b) {
    uint32_t d;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
  }
  __device__ static float max(const uint4& q) {
    const uint32_t m = max2(max2(q.x, q.y), max2(q.z, q.w));
    return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u));
  }
  __device__ static void put(uint4* q, int e, uint16_t v) {
    uint32_t* w = reinterpret_cast<uint32_t*>(q) + e / 2;
    *w = e & 1 ? (*w & 0xFFFFu) | ((uint32_t)v << 16) : (*w & 0xFFFF0000u) | v;
  }
};
template <>
struct Elem<float> {
  static constexpr int kVec = 4;
  static constexpr uint32_t kNegInf = 0xFF800000u;
  __device__ static float load(const float* p) { return *p; }
  __device__ static float at(const uint4& q, int e) {
    return __uint_as_float(e == 0 ? q.x : e == 1 ? q.y : e == 2 ? q.z : q.w);
  }
  __device__ static float max(const uint4& q) {
    return fmaxf(fmaxf(__uint_as_float(q.x), __uint_as_float(q.y)), fmaxf(__uint_as_float(q.z), __uint_as_float(q.w)));
  }
  __device__ static void put(uint4* q, int e, float v) { reinterpret_cast<float*>(q)[e] = v; }
};

// Keeps the vectors packed: without it the compiler holds every unpacked
// element from the sum to the selection.
template <int VPT>
__device__ __forceinline__ void repack(uint4 (&q)[VPT]) {
#pragma unroll
  for (int j = 0; j < VPT; ++j) asm volatile("" : "+r"(q[j].x), "+r"(q[j].y), "+r"(q[j].z), "+r"(q[j].w));
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
// split * chunk + (256 j + t) kVec + e.  kAligned: every row starts on a
// 16-byte boundary.  Keys go to [request][rank][split][beam], the order in
// which the merge's warps each meet every beam and every rank.
template <typename T, int VPT, bool kAligned>
__global__ void __launch_bounds__(kBeThreads, VPT == 8 ? 4 : 6) k_beam_rows(const T* __restrict__ logits, size_t stride, int vocab,
                                                          const float* __restrict__ scores,
                                                          const uint8_t* __restrict__ done, int k, int beams,
                                                          int chunk, uint64_t* __restrict__ keys,
                                                          ChunkSum* __restrict__ sums) {
  using E = Elem<T>;
  constexpr int V = E::kVec;
  __shared__ __align__(16) uint64_t cand[kCap + kRankStep];
  __shared__ uint4 vecs[kBeWarps][kCapV];
  __shared__ int vec_at[kBeWarps][kCapV];
  __shared__ float wm[kBeWarps], ws[kBeWarps];
  __shared__ __align__(16) uint32_t wtau[kBeWarps];
  __shared__ int n_cand;
  pdl_wait();
  pdl_trigger();
  const int row = blockIdx.z * beams + blockIdx.y, split = blockIdx.x, splits = gridDim.x;
  const float score = scores[row];
  const bool ended = done && done[row];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const T* base = logits + (size_t)row * stride;
  const uint32_t off = kAligned ? 0u : (uint32_t)((uintptr_t)base & 15u);
  const int first = split * chunk, end = min(vocab, first + chunk);
  if (tid == 0) n_cand = 0;
  if (!isfinite(score) || ended) return;   // no candidates here (the merge reads nothing either)

  uint4 q[VPT];
  float vm[VPT], mx = -INFINITY;
  const bool full = first + kBeThreads * V * VPT <= end;
  const int whole = (end - first) / V;   // vectors that lie in the chunk
  if (whole > 0) {
    // loads without conditions, past the chunk from its last vector instead,
    // and a few ahead of their shifts: else each waits for the one before
    const uint4* p = reinterpret_cast<const uint4*>((const char*)(base + first) - off);
    const int more = off != 0;
    constexpr int kBatch = kAligned || VPT < 4 ? VPT : 4;
#pragma unroll
    for (int j0 = 0; j0 < VPT; j0 += kBatch) {
      uint4 next[kBatch];
#pragma unroll
      for (int j = 0; j < kBatch; ++j) {
        const int at = full ? (j0 + j) * kBeThreads + tid : min((j0 + j) * kBeThreads + tid, whole - 1);
        q[j0 + j] = __ldg(p + at);
        if constexpr (!kAligned) next[j] = __ldg(p + at + more);
      }
      if constexpr (!kAligned)
#pragma unroll
        for (int j = 0; j < kBatch; ++j) q[j0 + j] = bytes16_at(q[j0 + j], next[j], off);
    }
  }
  if (!full) {
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int i = j * kBeThreads + tid;
      if (i >= whole) {
        q[j] = make_uint4(E::kNegInf, E::kNegInf, E::kNegInf, E::kNegInf);
#pragma unroll
        for (int e = 0; e < V; ++e)
          if (first + i * V + e < end) E::put(&q[j], e, base[first + i * V + e]);
      }
    }
  }
#pragma unroll
  for (int j = 0; j < VPT; ++j) vm[j] = E::max(q[j]), mx = fmaxf(mx, vm[j]);
  const uint32_t om = ord32(mx + 0.f);   // + 0: -0 and +0 are equal logits
  const uint32_t owm = __reduce_max_sync(0xffffffffu, om);
  const float m = unord32(owm);
  // sum of exp(x - m) = 2^-r sum 2^(c x - cm), cm = c m rounded, r = c m - cm:
  // one multiply-add per element, and the error of c scales x - m only.  2^-r
  // is taken to first order, which is right to 2^-24 while |r| <= 2^-11: always
  // up to |m| = 2^14 / c.  Past that x - m comes first, in one instruction more
  // (half a us of 35 for 64 x 8 x 131072).
  constexpr float kLog2e = 1.4426950408889634f;
  const float cm = m * kLog2e, r = fmaf(m, kLog2e, -cm);
  auto sum = [&](auto shifted) {
    constexpr bool kShifted = decltype(shifted)::value;
    uint64_t acc = pair(0.f, 0.f);
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const uint32_t w[4] = {q[j].x, q[j].y, q[j].z, q[j].w};
#pragma unroll
      for (int e = 0; e < V / 2; ++e) {
        uint64_t x;
        if constexpr (V == 8)
          x = pair(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xFFFF0000u));
        else
          x = pair(__uint_as_float(w[2 * e]), __uint_as_float(w[2 * e + 1]));
        const float2 t = unpair(kShifted ? mul_pair(add_pair(x, pair(-m, -m)), pair(kLog2e, kLog2e))
                                         : fma_pair(x, pair(kLog2e, kLog2e), pair(-cm, -cm)));
        acc = add_pair(acc, pair(exp2_fast(t.x), exp2_fast(t.y)));
      }
    }
    const float2 acc2 = unpair(acc);
    return acc2.x + acc2.y;
  };
  float s;
  if (fabsf(r) <= 0x1p-11f) {   // (the same for the warp)
    s = sum(std::false_type());
    s = fmaf(s, -0.6931471805599453f * r, s);
  } else {
    s = sum(std::true_type());
  }
  repack(q);
  if (isnan(s)) {   // a NaN (no candidate), a warp of -inf, +inf (takes all the probability)
    s = 0.f;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      float sj = 0.f;   // (a vector's sum of its own: as few additions in a row as above)
#pragma unroll 1
      for (int e = 0; e < V; ++e) {
        const float x = E::at(q[j], e);
        if (x > -INFINITY) sj += x == m ? 1.f : exp2_fast((x - m) * kLog2e);
      }
      s += sj;
    }
  }
  repack(q);
#pragma unroll
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  // the warp's j-th largest thread maximum (0: it has not as many threads)
  auto nth_max = [&](int j) {
    uint32_t left = om, v = owm;
    for (; j > 1; --j) {
      const uint32_t who = __ballot_sync(0xffffffffu, left == v);
      if (lane == __ffs(who) - 1) left = 0;
      v = __reduce_max_sync(0xffffffffu, left);
    }
    return v;
  };
  const uint32_t tau = nth_max((k + kBeWarps - 1) / kBeWarps);
  if (lane == 0) wm[warp] = m, ws[warp] = s, wtau[warp] = tau;
  __syncthreads();
  const uint4 t0 = reinterpret_cast<const uint4*>(wtau)[0], t1 = reinterpret_cast<const uint4*>(wtau)[1];
  static_assert(kBeWarps == 8, "one threshold per warp, in two vectors");
  uint32_t t = min(min(min(t0.x, t0.y), min(t0.z, t0.w)), min(min(t1.x, t1.y), min(t1.z, t1.w)));
  if (warp == 0) {
    const float wmi = wm[lane & 7];
    float M = wmi;
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float wsi = ws[lane & 7];
    float S = wsi > 0.f ? wsi * (wmi == M ? 1.f : expf(wmi - M)) : 0.f;
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) S += __shfl_xor_sync(0xffffffffu, S, o);
    if (lane == 0) sums[row * splits + split] = ChunkSum{M, S};
  }
  if (t <= kOrdNegInf) {   // some warps have no unmasked token: the same over those that have
    int active = 0;
#pragma unroll
    for (int i = 0; i < kBeWarps; ++i) active += wm[i] > -INFINITY;
    const int j = active ? (k + active - 1) / active : 33;
    const uint32_t again = j <= 32 && m > -INFINITY ? nth_max(j) : 0xffffffffu;
    __syncthreads();
    if (lane == 0) wtau[warp] = again;
    __syncthreads();
    t = j <= 32 ? 0xffffffffu : 0u;
#pragma unroll
    for (int i = 0; i < kBeWarps; ++i) t = min(t, wtau[i]);
    // (still none: too few threads have any, and all their tokens survive)
  }
  // survivors: >= tau and above -inf.  First the few vectors that hold some
  // are put side by side, then their elements are looked at, one a lane (in
  // place, the warp would step through all elements of a vector for one
  // lane's sake).
  const float low = unord32(max(t, kOrdNegInf + 1u));
  int nv = 0;
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const uint32_t hit = __ballot_sync(0xffffffffu, vm[j] >= low);
    if (hit) {
      const int at = nv + __popc(hit & ((1u << lane) - 1u));
      if (vm[j] >= low && at < kCapV) vecs[warp][at] = q[j], vec_at[warp][at] = first + (j * kBeThreads + tid) * V;
      nv += __popc(hit);
    }
  }
  __syncwarp();
  if (nv > kCapV) {
    if (lane == 0) atomicAdd(&n_cand, kCap + 1);
  } else {
    for (int i = lane; i < nv * V; i += 32) {
      const float x = E::load(reinterpret_cast<const T*>(vecs[warp]) + i);
      if (x >= low) {
        const int at = atomicAdd(&n_cand, 1);
        const uint32_t token = (uint32_t)(vec_at[warp][i / V] + i % V);
        if (at < kCap) cand[at] = ((uint64_t)ord32(x + 0.f) << 32) | (0xffffffffu - token);
      }
    }
  }
  __syncthreads();
  const int n = n_cand;
  uint64_t* out = keys + (size_t)blockIdx.z * beams * splits * k + split * beams + blockIdx.y;
  const int next = splits * beams;   // from one rank to the next
  if (n <= kCap) {
    // a thread counts the betters of its candidate, a few keys at a time
    // (zeros past the last: each warp that counts puts them there itself)
    for (int i0 = warp * 32; i0 < n; i0 += kBeThreads) {
      if (lane < kRankStep) cand[n + lane] = 0;
      __syncwarp();
      const uint64_t mine = i0 + lane < n ? cand[i0 + lane] : ~0ull;
      int rank = 0;
      for (int j = 0; j < n; j += kRankStep) {
#pragma unroll
        for (int e = 0; e < kRankStep; e += 2) {
          const ulonglong2 w = *reinterpret_cast<const ulonglong2*>(&cand[j + e]);
          rank += w.x > mine;
          rank += w.y > mine;
        }
      }
      if (i0 + lane < n && rank < k) out[rank * next] = mine;
    }
    for (int i = n + tid; i < k; i += kBeThreads) out[i * next] = 0;
  } else {   // many equal values: the greatest key below the last one, k times
    uint64_t last = ~0ull;
    for (int i = 0; i < k; ++i) {
      repack(q);
      uint64_t best = 0;
#pragma unroll
      for (int j = 0; j < VPT; ++j)
#pragma unroll 1
        for (int e = 0; e < V; ++e) {
          const float x = E::at(q[j], e);
          if (x > -INFINITY) {
            const uint32_t token = (uint32_t)(first + (j * kBeThreads + tid) * V + e);
            const uint64_t key = ((uint64_t)ord32(x + 0.f) << 32) | (0xffffffffu - token);
            if (key < last && key > best) best = key;
          }
        }
      best = warp_max64(best);
      __syncthreads();
      if (lane == 0) cand[warp] = best;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kBeWarps; ++w) best = cand[w] > best ? cand[w] : best;
      if (tid == 0) out[i * next] = best;
      last = best;
    }
  }
}

// One request.  With m the row's maximum and l = lse - m, value(b, v) is
// score + ((x - m) - l): l keeps its digits whatever the size of m, where a
// 64-bit lse of a row near 1e12 or more would have none for it.  (A row whose
// maximum is at the bottom of f32, below -2^127, holds nothing but the lowest
// values that masks are filled with: l is 0 there, as in a 64-bit lse.)
// The chunks' keys are first bounded in f32: value(b, v) lies within 2^-22
// (|score - l| + |x - m|) of its f32 sum (f64 runs at a small fraction of the
// f32 rate); tau is taken over the lower bounds, and only the few whose upper
// bound reaches it are valued in 64 bits and ranked.
constexpr int kKeep = 4;   // keys a thread holds in registers between the two looks at them
__global__ void __launch_bounds__(1024) k_beam_merge(const uint64_t* __restrict__ keys,
                                                     const ChunkSum* __restrict__ sums, const float* scores,
                                                     const uint8_t* done, int beams, int eos, int k, int splits, int32_t* __restrict__ tokens,
                                                     int32_t* __restrict__ parents, float* out_scores,
                                                     uint8_t* out_done) {
  __shared__ double score[kBeamMaxBeams], lsum[kBeamMaxBeams];   // l: log of sum exp(x - m)
  __shared__ float offs[kBeamMaxBeams];     // f32 of score - l
  __shared__ float top[kBeamMaxBeams];      // m (+inf: l is the log of their count)
  __shared__ int kind[kBeamMaxBeams];       // 0: no candidates, 1: live, 2: finished
  __shared__ uint32_t wtau[32];
  __shared__ uint64_t cval[kCap], cflat[kCap];
  __shared__ int n_cand;
  pdl_wait();
  pdl_trigger();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = blockDim.x >> 5;
  const int row0 = blockIdx.x * beams;
  const int per = splits * k, total = beams * per;
  const uint64_t* mykeys = keys + (size_t)row0 * per;
  // (rows without candidates have no keys: what is read there is not used)
  uint64_t held[kKeep];
#pragma unroll
  for (int i = 0; i < kKeep; ++i) {
    const int c = tid + i * blockDim.x;
    held[i] = c < total ? mykeys[c] : 0;
  }
  if (tid == 0) n_cand = 0;
  for (int b = warp; b < beams; b += nw) {
    const float sc = scores[row0 + b];
    const bool fin = done && done[row0 + b];
    if (!isfinite(sc) || fin) {
      if (lane == 0) kind[b] = isfinite(sc) ? 2 : 0, score[b] = (double)sc, offs[b] = sc;
      continue;
    }
    const ChunkSum* cs = sums + (size_t)(row0 + b) * splits;
    float m = -INFINITY;
    for (int i = lane; i < splits; i += 32) m = fmaxf(m, cs[i].m);
#pragma unroll
    for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    float s = 0.f;
    for (int i = lane; i < splits; i += 32) {
      const ChunkSum c = cs[i];
      if (c.s > 0.f) s += c.m == m ? c.s : c.s * expf(c.m - m);
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
    if (lane == 0) {
      // log s = e log 2 + log f, f near 1: the f32 log's error stays below 2^-25
      int e;
      float f = frexpf(s, &e);
      if (f < 0.70710678f) f *= 2.f, --e;
      const double l = m > -0x1p127f ? (double)e * 0.693147180559945309 + (double)logf(f) : 0.;
      kind[b] = s > 0.f ? 1 : 0;
      top[b] = m;
      score[b] = (double)sc;
      lsum[b] = l;
      offs[b] = (float)((double)sc - l);
    }
  }
  __syncthreads();

  // candidate c with key `key`, of beam b = c % beams: lower and upper bound
  // of its value as ordered f32 (0: no candidate)
  auto bounds = [&](int c, int b, uint64_t key, uint32_t* hi) -> uint32_t {
    *hi = 0;
    const int kd = kind[b];
    const float off = offs[b];
    if (kd != 1) return kd == 2 && c < beams ? *hi = ord32(off + 0.f) : 0;
    if (key == 0) return 0;
    const float x = unord32((uint32_t)(key >> 32)), m = top[b];
    if (isinf(m) && x != m) return 0;
    const float d = isinf(m) ? 0.f : x - m;
    const float v = d + off, err = 0x1p-22f * (fabsf(d) + fabsf(off));
    if (!(fabsf(v) + err < 3.0e38f)) {   // past f32: bounded by nothing
      *hi = ord32(INFINITY);
      return kOrdNegInf;
    }
    *hi = ord32(v + err + 0.f);
    return ord32(v - err + 0.f);
  };
  // its 64-bit value and place (beam, token), which orders like beam * vocab + token
  auto value = [&](int b, uint64_t key, uint64_t* flat) -> uint64_t {
    if (kind[b] == 2) {
      *flat = ((uint64_t)b << 32) | (uint32_t)eos;
      return ord64(score[b] + 0.);
    }
    *flat = ((uint64_t)b << 32) | (0xffffffffu - (uint32_t)key);
    const double d = isinf(top[b]) ? 0. : (double)unord32((uint32_t)(key >> 32)) - (double)top[b];
    return ord64(score[b] + (d - lsum[b]) + 0.);
  };
  uint32_t mine = 0, hi, hi_held[kKeep];
  int b_held[kKeep];
  {
    const int step = blockDim.x % beams;
    int b = tid % beams;
#pragma unroll
    for (int i = 0; i < kKeep; ++i) {
      const int c = tid + i * blockDim.x;
      b_held[i] = b;
      hi_held[i] = 0;
      if (c < total) mine = max(mine, bounds(c, b, held[i], &hi_held[i]));
      b += step;
      b -= b >= beams ? beams : 0;
    }
  }
  for (int c = tid + kKeep * blockDim.x; c < total; c += blockDim.x) mine = max(mine, bounds(c, c % beams, mykeys[c], &hi));
  // (tau from the first 8 warps, theirs are the chunks' best, or from those
  // whose lanes all have a key: an empty warp would leave no threshold)
  const int tw = min(8, max(1, min(nw, total / 32)));
  uint32_t tau = __reduce_max_sync(0xffffffffu, mine);
  for (int i = (k + tw - 1) / tw; i > 1; --i) {
    const uint32_t who = __ballot_sync(0xffffffffu, mine == tau);
    if (lane == __ffs(who) - 1) mine = 0;
    tau = __reduce_max_sync(0xffffffffu, mine);
  }
  if (lane == 0) wtau[warp] = tau;
  __syncthreads();
  tau = __reduce_min_sync(0xffffffffu, lane < tw ? wtau[lane] : 0xffffffffu);
  if (tau == 0) tau = 1;
  auto keep = [&](int b, uint64_t key) {
    const int at = atomicAdd(&n_cand, 1);
    uint64_t f;
    if (at < kCap) cval[at] = value(b, key, &f), cflat[at] = f;
  };
#pragma unroll
  for (int i = 0; i < kKeep; ++i)
    if (hi_held[i] >= tau) keep(b_held[i], held[i]);
  for (int c = tid + kKeep * blockDim.x; c < total; c += blockDim.x) {
    const uint64_t key = mykeys[c];
    bounds(c, c % beams, key, &hi);
    if (hi >= tau) keep(c % beams, key);
  }
  __syncthreads();
  const int n = n_cand;
  const size_t o0 = (size_t)blockIdx.x * k;
  auto put = [&](int rank, uint64_t v, uint64_t flat) {
    const int b = (int)(flat >> 32), token = (int)(uint32_t)flat;
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
    for (int i0 = 0; i0 < n; i0 += blockDim.x / 8) {   // eight threads count a candidate's betters
      const int i = i0 + tid / 8;
      const uint64_t v = i < n ? cval[i] : ~0ull, fl = i < n ? cflat[i] : 0;
      int rank = 0;
      for (int j = tid % 8; j < n; j += 8) {
        const uint64_t w = cval[j];
        rank += w > v;
        if (w == v) rank += cflat[j] < fl;
      }
#pragma unroll
      for (int o = 1; o < 8; o <<= 1) rank += __shfl_xor_sync(0xffffffffu, rank, o);
      if (i < n && tid % 8 == 0 && rank < k) put(rank, v, fl);
    }
    for (int i = n + tid; i < k; i += blockDim.x) none(i);
  } else {   // many equal values: the best after the last one, k times
    uint64_t lv = ~0ull, lf = 0;
    for (int i = 0; i < k; ++i) {
      uint64_t bv = 0, bf = ~0ull;
      for (int c = tid; c < total; c += blockDim.x) {
        const uint64_t key = mykeys[c];
        bounds(c, c % beams, key, &hi);
        if (hi < tau) continue;
        uint64_t f;
        const uint64_t v = value(c % beams, key, &f);
        if (v > lv || (v == lv && f <= lf)) continue;
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
      for (int w = 0; w < nw; ++w)
        if (cval[w] > bv || (cval[w] == bv && cflat[w] < bf)) bv = cval[w], bf = cflat[w];
      if (tid == 0) {
        if (bv) put(i, bv, bf);
        else none(i);
      }
      lv = bv, lf = bf;
    }
  }
}

namespace {

// 16-byte vectors per thread and chunk: 8 (32 KB), or fewer where that leaves
// SMs idle.
int beam_vectors(int rows, int vocab, int vec, int sms) {
  int vpt = 8;
  while (vpt > 1 && (long long)rows * ((vocab + kBeThreads * vec * vpt - 1) / (kBeThreads * vec * vpt)) < 2ll * sms)
    vpt /= 2;
  return vpt;
}

template <typename T, int VPT, bool kAligned>
cudaError_t launch_rows(const void* logits, size_t stride, int rows, int vocab, const float* scores, const uint8_t* done,
                        int k, int beams, int splits, uint64_t* keys, ChunkSum* sums, cudaStream_t st) {
  const int vec = Elem<T>::kVec, chunk = ((vocab + splits - 1) / splits + vec - 1) / vec * vec;   // even parts
  return launch_pdl(k_beam_rows<T, VPT, kAligned>, dim3((unsigned)splits, (unsigned)beams, (unsigned)(rows / beams)), dim3(kBeThreads), 0, st,
                    static_cast<const T*>(logits), stride, vocab, scores, done, k, beams, chunk, keys, sums);
}

template <typename T>
cudaError_t launch_rows(int vpt, bool aligned, const void* logits, size_t stride, int rows, int vocab,
                        const float* scores, const uint8_t* done, int k, int beams, int splits, uint64_t* keys,
                        ChunkSum* sums, cudaStream_t st) {
#define M2_BEAM_ROWS(VPT)                                                                                           \
  return aligned ? launch_rows<T, VPT, true>(logits, stride, rows, vocab, scores, done, k, beams, splits, keys, sums, st)   \
                 : launch_rows<T, VPT, false>(logits, stride, rows, vocab, scores, done, k, beams, splits, keys, sums, st)
  if (vpt == 8) M2_BEAM_ROWS(8);
  if (vpt == 4) M2_BEAM_ROWS(4);
  if (vpt == 2) M2_BEAM_ROWS(2);
  M2_BEAM_ROWS(1);
#undef M2_BEAM_ROWS
}

size_t align256(size_t v) { return (v + 255) & ~(size_t)255; }

}  // namespace

size_t beam_workspace_bytes(int batch, int beams, int vocab, int k) {
  constexpr int kLeast = kBeThreads * Elem<float>::kVec;   // the smallest chunk: the most parts
  const size_t parts = (size_t)batch * beams * ((vocab + kLeast - 1) / kLeast);
  return align256(parts * k * sizeof(uint64_t)) + align256(parts * sizeof(ChunkSum));
}

cudaError_t launch_beam_select(const void* logits, bool bf16, size_t stride, int batch, int beams, int vocab,
                               const float* scores, const uint8_t* done, int eos, int k, int32_t* tokens,
                               int32_t* parents, float* out_scores, uint8_t* out_done, void* ws, cudaStream_t st) {
  const int rows = batch * beams, vec = bf16 ? 8 : 4, vpt = beam_vectors(rows, vocab, vec, device_sm_count());
  const int chunk = kBeThreads * vec * vpt, splits = (vocab + chunk - 1) / chunk;
  const bool aligned = (uintptr_t)logits % 16 == 0 && (rows == 1 || stride % vec == 0);
  uint64_t* keys = static_cast<uint64_t*>(ws);
  ChunkSum* sums = reinterpret_cast<ChunkSum*>(static_cast<char*>(ws) + align256((size_t)rows * splits * k * sizeof(uint64_t)));
  cudaError_t e = bf16 ? launch_rows<uint16_t>(vpt, aligned, logits, stride, rows, vocab, scores, done, k, beams, splits, keys, sums, st)
                       : launch_rows<float>(vpt, aligned, logits, stride, rows, vocab, scores, done, k, beams, splits, keys, sums, st);
  if (e != cudaSuccess) return e;
  const int threads = beams * splits * k > 1024 ? 1024 : 256;
  return launch_pdl(k_beam_merge, dim3((unsigned)batch), dim3(threads), 0, st, keys, sums, scores, done, beams, eos, k,
                    splits, tokens, parents, out_scores, out_done);
}

}  // namespace m2

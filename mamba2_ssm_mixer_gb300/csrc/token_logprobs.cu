// Log probabilities of given tokens, their ranks, the rows' entropy and the
// largest tokens, in one pass over the logits x:
//   m = max x, S = sum exp(x - m), E = sum exp(x - m) x / S
//   logprob(t) = (x_t - m) - log S, entropy = m + log S - E,
//   rank(t) = 1 + the tokens before t in the order (greater logit, lower token).
//
// k_token_logprobs: a CTA takes a row, or a slice of one where rows are few (the
// slices' CTAs form a cluster and the first of them joins the parts through
// distributed shared memory).  Warp 8 streams 16 KB chunks into a ring with
// bulk copies, across rows, so that the stream does not wait for a row's
// end; warps 0 to 7 keep per thread
//  - sums in base 2 with a whole number c as reference: u = fma(x, L, -c) with
//    L = f32(log2 e) is rounded once, S += 2^u, U += 2^u u.  c moves only when
//    a chunk's maximum passes it by 16 (no rescaling in most chunks), and what
//    L lacks of log2 e is put back at the end: lse = ln 2 (c + m (log2 e - L)) +
//    log S.  Rows whose maximum is beyond +-2^16 (or +inf) are summed again
//    as x - m (row_again);
//  - the number of logits greater than the given token's;
//  - the maxima of up to kGroups groups of its vectors.
// The k largest need no sort and no list while streaming: if each of w warps has
// ceil(k / w) threads whose maximum is at least tau, at least k tokens are >=
// tau; only groups whose maximum reaches tau are read again (a few KB of the
// row, from L2), and the survivors are ranked by counting.  Where equal values
// leave more survivors than fit, the row is read once more against a running
// k-th best (top_again).
#include <cuda_bf16.h>

#include "launch_util.h"
#include "m2_kernels.h"
#include "tc_ptx.cuh"

namespace m2 {

using namespace tc;

namespace {

constexpr int kLpWarps = 8;
constexpr int kLpThreads = kLpWarps * 32;           // consumers
constexpr int kVpt = 4;                             // 16-byte vectors per thread and chunk
constexpr int kChunkVecs = kLpThreads * kVpt;
constexpr int kChunkBytes = kChunkVecs * 16;
constexpr int kStages = 4;
constexpr int kGroups = 16;                         // groups of vectors per thread
constexpr int kLpCap = 2048;                        // survivors ranked by counting
constexpr int kLpHits = 1024;                       // groups they may lie in
constexpr int kStep = kLpCap / 2 / kLpThreads;      // tokens a thread takes per step of top_again
constexpr float kL = 1.4426950408889634f;           // log2 e, rounded to f32
constexpr double kLn2 = 0.6931471805599453094;
constexpr double kLRest = 1.4426950408889634074 - (double)1.4426950408889634f;   // log2 e - L
constexpr float kNone = -0x1p18f;                   // reference c before any unmasked logit
constexpr float kPlain = 0x1p16f;                   // |m| up to which c is exact enough

struct __align__(16) LpPart {
  float c, s, u, m;   // reference, sums, maximum
  int greater;        // logits before the given token's
};

struct __align__(16) LpShared {
  uint64_t full[kStages], empty[kStages];
  uint64_t cand[kLpCap];
  uint64_t best[kLpMaxTop];          // the slice's largest keys, in order
  uint32_t gmax[kGroups][kLpThreads];
  LpPart warp[kLpWarps];
  LpPart part;                       // the slice's
  uint32_t tau[kLpWarps];
  double z;                          // log S of the whole row (relative to its maximum m)
  float m;
  int n_cand, n_hit, abort;
  uint16_t hits[kLpHits];            // groups whose maximum reaches the threshold
};

// Order-preserving map of floats to unsigned (no NaN).
__device__ __forceinline__ uint32_t ord32(float f) {
  const uint32_t u = __float_as_uint(f);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unord32(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? o ^ 0x80000000u : ~o);
}
constexpr uint32_t kOrdNegInf = 0x007fffffu;
// Greater for a greater logit, then for the lower token; +0: -0 and +0 are equal.
__device__ __forceinline__ uint64_t key_of(float x, int token) {
  return (uint64_t)ord32(x + 0.f) << 32 | (uint32_t)~token;
}
__device__ __forceinline__ float key_logit(uint64_t k) { return unord32((uint32_t)(k >> 32)); }
__device__ __forceinline__ int key_token(uint64_t k) { return (int)~(uint32_t)k; }

// The next value below x, `ulp` the last place of its type in f32 bits: what is
// greater than that is x or greater.
__device__ __forceinline__ float next_below(float x, uint32_t ulp) {
  const uint32_t b = __float_as_uint(x);
  return __uint_as_float(x == 0.f ? 0x80000000u + ulp : x > 0.f ? b - ulp : b + ulp);
}
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// f32 pairs in one 64-bit register
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
__device__ __forceinline__ uint64_t add_pair(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

__device__ __forceinline__ void consumers_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kLpThreads) : "memory"); }

// 16-byte vectors of logits.  Maxima ignore NaN.
template <typename T>
struct Vec;
template <>
struct Vec<uint16_t> {
  static constexpr int kN = 8;
  static constexpr uint32_t kNegInf = 0xFF80FF80u;
  __device__ static float load(const uint16_t* p) { return bfbits2f(*p); }
  __device__ static float at(const uint4& q, int e) {
    const uint32_t w = e < 2 ? q.x : e < 4 ? q.y : e < 6 ? q.z : q.w;
    return __uint_as_float(e & 1 ? w & 0xFFFF0000u : w << 16);
  }
  __device__ static void mask(uint4& q, int e) {
    uint32_t* w = reinterpret_cast<uint32_t*>(&q) + e / 2;
    *w = e & 1 ? (*w & 0xFFFFu) | 0xFF800000u : (*w & 0xFFFF0000u) | 0xFF80u;
  }
  __device__ static float max(const uint4 (&q)[kVpt]) {
    uint32_t m = max_bf16x2(max_bf16x2(q[0].x, q[0].y), max_bf16x2(q[0].z, q[0].w));
#pragma unroll
    for (int j = 1; j < kVpt; ++j)
      m = max_bf16x2(m, max_bf16x2(max_bf16x2(q[j].x, q[j].y), max_bf16x2(q[j].z, q[j].w)));
    return fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u));
  }
  // logits greater than the bf16 value thr
  __device__ static int greater(const uint4& q, float thr) {
    const __nv_bfloat162 t = __float2bfloat162_rn(thr);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    __nv_bfloat162 n = __hgt2(*reinterpret_cast<const __nv_bfloat162*>(&w[0]), t);
#pragma unroll
    for (int i = 1; i < 4; ++i) n = __hadd2(n, __hgt2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]), t));
    return (int)(__low2float(n) + __high2float(n));
  }
  __device__ static float below(float x) { return next_below(x, 0x10000u); }
  struct Low {
    uint32_t v;
    __device__ explicit Low(float low) { v = pack_bf16x2(low, low); }
  };
  __device__ static void sums(const uint4& q, const Low& low, uint64_t cc, uint64_t& s, uint64_t& u) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t x = max_bf16x2(w[i], low.v);
      const uint64_t d = fma_pair(pair(__uint_as_float(x << 16), __uint_as_float(x & 0xFFFF0000u)), pair(kL, kL), cc);
      const float2 t = unpair(d);
      const uint64_t p = pair(exp2_fast(t.x), exp2_fast(t.y));
      s = add_pair(s, p);
      u = fma_pair(p, d, u);
    }
  }
};
template <>
struct Vec<float> {
  static constexpr int kN = 4;
  static constexpr uint32_t kNegInf = 0xFF800000u;
  __device__ static float load(const float* p) { return *p; }
  __device__ static float at(const uint4& q, int e) {
    return __uint_as_float(e == 0 ? q.x : e == 1 ? q.y : e == 2 ? q.z : q.w);
  }
  __device__ static void mask(uint4& q, int e) { reinterpret_cast<uint32_t*>(&q)[e] = kNegInf; }
  __device__ static float max(const uint4 (&q)[kVpt]) {
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < kVpt; ++j)
      m = fmaxf(m, fmaxf(fmaxf(at(q[j], 0), at(q[j], 1)), fmaxf(at(q[j], 2), at(q[j], 3))));
    return m;
  }
  __device__ static int greater(const uint4& q, float thr) {
    int n = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) n += at(q, e) > thr;
    return n;
  }
  __device__ static float below(float x) { return next_below(x, 1u); }
  struct Low {
    float v;
    __device__ explicit Low(float low) : v(low) {}
  };
  __device__ static void sums(const uint4& q, const Low& low, uint64_t cc, uint64_t& s, uint64_t& u) {
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      const uint64_t d = fma_pair(pair(fmaxf(at(q, i), low.v), fmaxf(at(q, i + 1), low.v)), pair(kL, kL), cc);
      const float2 t = unpair(d);
      const uint64_t p = pair(exp2_fast(t.x), exp2_fast(t.y));
      s = add_pair(s, p);
      u = fma_pair(p, d, u);
    }
  }
};

// Where a row's vectors lie: token i is element (i + off) % kN of vector
// (i + off) / kN, counted from the 16-byte boundary at or below the row.
template <typename T>
struct RowAt {
  const T* base;     // token 0
  const uint4* vec;  // vector 0
  int off;           // elements of vector 0 before token 0
  int nv;            // vectors that hold tokens
  int vocab;
  __device__ RowAt(const T* logits, size_t stride, int row, int n) : base(logits + (size_t)row * stride), vocab(n) {
    const uint32_t b = (uint32_t)((uintptr_t)base & 15u);
    vec = reinterpret_cast<const uint4*>(reinterpret_cast<const char*>(base) - b);
    off = (int)(b / sizeof(T));
    nv = (off + n + Vec<T>::kN - 1) / Vec<T>::kN;
  }
  // q is vector v: elements that are no tokens become -inf
  __device__ void edges(uint4& q, int v) const {
#pragma unroll
    for (int e = 0; e < Vec<T>::kN; ++e) {
      const int t = v * Vec<T>::kN + e - off;
      if (t < 0 || t >= vocab) Vec<T>::mask(q, e);
    }
  }
  __device__ bool edge(int v) const { return v == 0 || v == nv - 1; }
};

// Two parts of a row as one, in the larger of their references.
__device__ __forceinline__ LpPart join(const LpPart& a, const LpPart& b) {
  const float c = fmaxf(a.c, b.c), da = a.c - c, db = b.c - c;
  const float fa = exp2_fast(da), fb = exp2_fast(db);
  return {c, a.s * fa + b.s * fb, fmaf(a.s, da, a.u) * fa + fmaf(b.s, db, b.u) * fb, fmaxf(a.m, b.m),
          a.greater + b.greater};
}

// The k largest of cand[0, n) by counting, in order, to best[0, k) (n < k: the
// rest are 0).
__device__ __forceinline__ void rank_candidates(const uint64_t* cand, int n, int k, uint64_t* best) {
  for (int i = threadIdx.x; i < n; i += kLpThreads) {
    const uint64_t mine = cand[i];
    int r = 0;
    for (int j = 0; j < n; ++j) r += cand[j] > mine;
    if (r < k) best[r] = mine;
  }
  for (int i = n + (int)threadIdx.x; i < k; i += kLpThreads) best[i] = 0;
}

// The k largest keys of tokens [t0, t1) of a row, by a pass in order against
// the k-th best so far: equal logits never pass it later.  All consumers.
template <typename T>
__device__ __noinline__ void top_again(LpShared* sh, const T* base, int t0, int t1, int k) {
  uint64_t floor = 0;
  consumers_sync();
  if (threadIdx.x == 0) sh->n_cand = 0;
  consumers_sync();
  int held = 0;
  for (int t = t0; t < t1; t += kStep * kLpThreads) {
    for (int e = 0; e < kStep; ++e) {
      const int i = t + e * kLpThreads + (int)threadIdx.x;
      if (i < t1) {
        const float x = Vec<T>::load(base + i);
        const uint64_t key = key_of(x, i);
        if (x > -INFINITY && key > floor) sh->cand[atomicAdd(&sh->n_cand, 1)] = key;
      }
    }
    consumers_sync();
    const int n = sh->n_cand;
    consumers_sync();   // all have read it before any appends again
    if (n == held) continue;
    rank_candidates(sh->cand, n, k, sh->best);
    consumers_sync();
    held = n < k ? n : k;
    if ((int)threadIdx.x < held) sh->cand[threadIdx.x] = sh->best[threadIdx.x];
    if (n >= k) floor = sh->best[k - 1];
    if (threadIdx.x == 0) sh->n_cand = held;
    consumers_sync();
  }
  if (held == 0)
    for (int i = threadIdx.x; i < k; i += kLpThreads) sh->best[i] = 0;
  consumers_sync();
}

// log S and the entropy of a row whose maximum m is finite and large, or +inf
// (then the +inf tokens share the probability).  All consumers.
template <typename T>
__device__ __noinline__ float2 row_again(LpShared* sh, const T* base, int vocab, float m) {
  float s = 0.f, u = 0.f;
  for (int i = threadIdx.x; i < vocab; i += kLpThreads) {
    const float x = Vec<T>::load(base + i);
    if (m == INFINITY) {
      s += x == INFINITY ? 1.f : 0.f;
    } else {
      const float d = x - m, p = expf(d);
      if (p > 0.f) s += p, u = fmaf(p, d, u);
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o), u += __shfl_xor_sync(0xffffffffu, u, o);
  consumers_sync();
  if ((threadIdx.x & 31) == 0) sh->warp[threadIdx.x >> 5].s = s, sh->warp[threadIdx.x >> 5].u = u;
  consumers_sync();
  s = u = 0.f;
  for (int w = 0; w < kLpWarps; ++w) s += sh->warp[w].s, u += sh->warp[w].u;
  consumers_sync();
  const float z = logf(s);
  return make_float2(z, z - u / s);
}

}  // namespace

template <typename T>
__global__ void __launch_bounds__(kLpThreads + 32, 2)
    k_token_logprobs(const T* __restrict__ logits, size_t stride, int rows, int vocab, const int32_t* __restrict__ tokens,
                     int top, LpOut out, int* err) {
  using V = Vec<T>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = smem_align<128>(smem_raw);
  LpShared* sh = reinterpret_cast<LpShared*>(ring + kStages * kChunkBytes);
  volatile int* abort = &sh->abort;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // slices of a row: the CTAs of a cluster (grid x), one row each; else CTAs walk rows
  const int S = (int)gridDim.x, slice = (int)blockIdx.x;
  const int row0 = blockIdx.y, row_step = gridDim.y;

  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&sh->full[s], 1);
      mbar_init(&sh->empty[s], kLpWarps);
    }
    sh->abort = 0;
    fence_mbar_init();
  }
  __syncthreads();
  pdl_wait();
  pdl_trigger();

  auto slice_of = [&](const RowAt<T>& r, int& v0, int& v1) {
    v0 = (int)((long long)r.nv * slice / S);
    v1 = (int)((long long)r.nv * (slice + 1) / S);
  };

  if (warp == kLpWarps) {
    if (lane == 0) {
      // ---------------- producer
      int stage = 0, issued = 0;
      uint32_t phase = 0;
      for (int row = row0; row < rows && !*abort; row += row_step) {
        const RowAt<T> r(logits, stride, row, vocab);
        int v0, v1;
        slice_of(r, v0, v1);
        for (int v = v0; v < v1; v += kChunkVecs) {
          if (!mbar_wait_sleep(&sh->empty[stage], phase ^ 1u, abort)) {
            *abort = 1;
            if (err) atomicOr(err, kErrTimeout);
            break;
          }
          const uint32_t bytes = (uint32_t)(min(kChunkVecs, v1 - v) * 16);
          mbar_expect_tx(&sh->full[stage], bytes);
          bulk_g2s(ring + stage * kChunkBytes, r.vec + v, bytes, &sh->full[stage]);
          ++issued;
          if (++stage == kStages) stage = 0, phase ^= 1u;
        }
      }
      if (*abort)   // let the copies in flight land before the CTA can exit
        for (int i = issued > kStages ? issued - kStages : 0; i < issued; ++i)
          mbar_wait(&sh->full[i % kStages], (uint32_t)(i / kStages) & 1u, nullptr, 100000000ull);
    }
    __syncwarp();
  } else {
    // ---------------- consumers
    int stage = 0;
    uint32_t phase = 0;
    auto token_of = [&](int row) { return tokens && row < rows ? tokens[row] : -1; };
    auto valid = [&](int t) { return t >= 0 && t < vocab; };
    auto logit_of = [&](int row, int t) { return valid(t) ? V::load(logits + (size_t)row * stride + t) : 0.f; };
    int token = token_of(row0);
    float xt = logit_of(row0, token);
    for (int row = row0; row < rows; row += row_step) {
      const RowAt<T> r(logits, stride, row, vocab);
      int v0, v1;
      slice_of(r, v0, v1);
      const int chunks = (v1 - v0 + kChunkVecs - 1) / kChunkVecs;
      const int per_group = (chunks + kGroups - 1) / kGroups;   // chunks of a group
      const int next_token = token_of(row + row_step);
      const bool masked = !(xt > -INFINITY);                    // (NaN too)
      // before the given token's vector equal logits count as greater
      const int vt = valid(token) && !masked ? (token + r.off) / V::kN : -1;
      const float thr = masked ? -INFINITY : xt, thr_eq = masked ? -INFINITY : V::below(xt);

      float c = kNone, m = -INFINITY, gm = -INFINITY;
      uint64_t s2 = pair(0.f, 0.f), u2 = pair(0.f, 0.f);
      int greater = 0;
      for (int ch = 0; ch < chunks; ++ch) {
        const bool there = *abort ? false : mbar_wait(&sh->full[stage], phase, abort);
        if (!__all_sync(0xffffffffu, there)) {   // (the rows left go through without data)
          *abort = 1;
          if (err && lane == 0) atomicOr(err, kErrTimeout);
        }
        const int va = v0 + ch * kChunkVecs + tid;
        const uint4* p = reinterpret_cast<const uint4*>(ring + stage * kChunkBytes) + tid;
        uint4 q[kVpt];
        if (ch > 0 && ch + 1 < chunks) {
#pragma unroll
          for (int j = 0; j < kVpt; ++j) q[j] = p[j * kLpThreads];
        } else {
#pragma unroll
          for (int j = 0; j < kVpt; ++j) {
            const int v = va + j * kLpThreads;
            q[j] = v < v1 ? p[j * kLpThreads] : make_uint4(V::kNegInf, V::kNegInf, V::kNegInf, V::kNegInf);
            if (v < v1 && r.edge(v)) r.edges(q[j], v);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&sh->empty[stage]);
        if (++stage == kStages) stage = 0, phase ^= 1u;

        const float mx = V::max(q);
        gm = fmaxf(gm, mx);
        if (top && ((ch + 1) % per_group == 0 || ch + 1 == chunks)) {
          sh->gmax[ch / per_group][tid] = ord32(gm + 0.f);
          m = fmaxf(m, gm);
          gm = -INFINITY;
        }
        if (mx * kL > c + 16.f) {
          const float cn = rintf(mx * kL), d = fmaxf(c - cn, -1e30f), f = exp2_fast(d);
          u2 = fma_pair(s2, pair(d, d), u2);
          s2 = fma_pair(s2, pair(f, f), pair(0.f, 0.f));
          u2 = fma_pair(u2, pair(f, f), pair(0.f, 0.f));
          c = cn;
        }
        if (c > kNone) {
          // masked logits and NaN take a value whose exponential is 0 (-160 in base 2 at least, finite)
          float low = (c - 160.f) / kL;
          low -= fabsf(low) * 0.01f;
          const typename V::Low lo(low);
          const uint64_t cc = pair(-c, -c);
#pragma unroll
          for (int j = 0; j < kVpt; ++j) V::sums(q[j], lo, cc, s2, u2);
        }
#pragma unroll
        for (int j = 0; j < kVpt; ++j) {
          const int v = va + j * kLpThreads;
          if (v != vt) {
            greater += V::greater(q[j], v < vt ? thr_eq : thr);
          } else {
#pragma unroll
            for (int e = 0; e < V::kN; ++e) {
              const float x = V::at(q[j], e);
              greater += x > xt || (x == xt && v * V::kN + e - r.off < token);
            }
          }
        }
      }
      const float next_xt = logit_of(row + row_step, next_token);
      m = fmaxf(m, gm);

      // ---------------- the slice's sums
      const float2 ss = unpair(s2), uu = unpair(u2);
      LpPart a{c, ss.x + ss.y, uu.x + uu.y, m, greater};
#pragma unroll
      for (int o = 16; o; o >>= 1) {
        LpPart b;
        b.c = __shfl_xor_sync(0xffffffffu, a.c, o);
        b.s = __shfl_xor_sync(0xffffffffu, a.s, o);
        b.u = __shfl_xor_sync(0xffffffffu, a.u, o);
        b.m = __shfl_xor_sync(0xffffffffu, a.m, o);
        b.greater = __shfl_xor_sync(0xffffffffu, a.greater, o);
        a = join(a, b);
      }
      if (lane == 0) sh->warp[warp] = a;
      if (tid == 0) sh->n_cand = 0, sh->n_hit = 0;
      if (top) {
        // this warp's ceil(k / w)-th largest thread maximum, w the warps whose
        // threads all have a vector (none: every token is a candidate)
        const int full = min(kLpWarps, (v1 - v0) / 32);
        const int need = full ? (top + full - 1) / full : 33;
        uint32_t mine = ord32(m + 0.f), t = 0;
        if (need <= 32)
          for (int i = 0; i < need; ++i) {
            t = __reduce_max_sync(0xffffffffu, mine);
            if (__ffs(__ballot_sync(0xffffffffu, mine == t)) - 1 == lane) mine = 0;
          }
        if (lane == 0) sh->tau[warp] = warp < full ? t : 0xffffffffu;
      }
      consumers_sync();
      // what the given token and the entropy get from a row's whole part
      auto finish = [&](const LpPart& b, float2 again, bool odd) {
        double z = again.x, h = again.y;
        if (!odd && b.m > -INFINITY) {
          // S = 2^e f with f near 1: its logarithm without a double's
          const int e = (int)((__float_as_uint(b.s) + 0x4AFB0Du) >> 23) - 127;
          const double ln = kLn2 * (double)e + (double)logf(__uint_as_float(__float_as_uint(b.s) - ((uint32_t)e << 23)));
          const double shift = kLn2 * ((double)b.c + (double)b.m * kLRest);
          const float q = b.u / b.s;
          const double mean = (double)q + (double)(fmaf(-q, b.s, b.u) / b.s);   // u / s past f32
          z = ln + (shift - (double)b.m);
          h = ln + (shift - (mean + (double)b.c) * (1.0 / (double)kL));
        }
        sh->z = z;
        sh->m = b.m;
        if (!(b.m > -INFINITY)) h = 0.0;
        if (out.entropy) out.entropy[row] = fmaxf((float)h, 0.f);
        float lp = 0.f;
        int rank = 0;
        if (valid(token)) {
          lp = masked ? -INFINITY : b.m == INFINITY ? (xt == INFINITY ? (float)-z : -INFINITY)
                                                     : (float)((double)xt - (double)b.m - z);
          rank = 1 + b.greater;
        } else if (token != -1 && err) {
          atomicOr(err, kErrToken);
        }
        if (tokens) out.logprobs[row] = lp, out.ranks[row] = rank;
      };
      auto is_odd = [](float m) { return m > -INFINITY && !(fabsf(m) <= kPlain); };
      if (warp == 0) {
        LpPart b = sh->warp[lane & (kLpWarps - 1)];
#pragma unroll
        for (int o = kLpWarps / 2; o; o >>= 1) {
          LpPart d;
          d.c = __shfl_xor_sync(0xffffffffu, b.c, o);
          d.s = __shfl_xor_sync(0xffffffffu, b.s, o);
          d.u = __shfl_xor_sync(0xffffffffu, b.u, o);
          d.m = __shfl_xor_sync(0xffffffffu, b.m, o);
          d.greater = __shfl_xor_sync(0xffffffffu, b.greater, o);
          b = join(b, d);
        }
        if (lane == 0) {
          sh->part = b;
          if (S == 1 && !is_odd(b.m)) finish(b, make_float2(0.f, 0.f), false);
        }
        __syncwarp();
      }
      // ---------------- the slice's largest tokens
      if (top) {
        uint32_t tau = 0xffffffffu;
        for (int w = 0; w < kLpWarps; ++w) tau = min(tau, sh->tau[w]);
        if (tau == 0xffffffffu || (v1 - v0) / 32 * 32 < top) tau = 0;
        tau = max(tau, kOrdNegInf + 1);
        // the groups with a token that reaches tau, then their vectors, one per
        // thread: read where they are found, a warp takes its groups' loads one
        // after another (4096 x 131072: 519 us)
        const int groups = chunks ? (chunks + per_group - 1) / per_group : 0;
        for (int g = 0; g < groups; ++g)
          if (sh->gmax[g][tid] >= tau) {
            const int at = atomicAdd(&sh->n_hit, 1);
            if (at < kLpHits) sh->hits[at] = (uint16_t)(g * kLpThreads + tid);
          }
        consumers_sync();
        const int hits = sh->n_hit, per_hit = per_group * kVpt;
        if (hits <= kLpHits)
          for (int i = tid; i < hits * per_hit; i += kLpThreads) {
            const int hit = sh->hits[i / per_hit], j = i % per_hit;
            const int v = v0 + (hit / kLpThreads * per_hit + j) * kLpThreads + hit % kLpThreads;
            if (v >= v1) continue;
            uint4 q = __ldg(r.vec + v);
            if (r.edge(v)) r.edges(q, v);
#pragma unroll
            for (int e = 0; e < V::kN; ++e) {
              const float x = V::at(q, e);
              if (x > -INFINITY && ord32(x + 0.f) >= tau) {
                const int at = atomicAdd(&sh->n_cand, 1);
                if (at < kLpCap) sh->cand[at] = key_of(x, v * V::kN + e - r.off);
              }
            }
          }
        consumers_sync();
        const int n = sh->n_cand;
        if (hits <= kLpHits && n <= kLpCap)
          rank_candidates(sh->cand, n, top, sh->best);
        else
          top_again(sh, r.base, max(0, v0 * V::kN - r.off), min(vocab, v1 * V::kN - r.off), top);
      }
      consumers_sync();

      // ---------------- the row's results, from its slices' parts
      if (S > 1) {
        cluster_sync();   // (the producer's warp arrives too, below)
        if (slice == 0) {
          LpPart b = sh->part;
          for (int o = 1; o < S; ++o) {
            const uint32_t at = cluster_map(smem_u32(&sh->part), (uint32_t)o);
            const float4 d = ld_dsmem_f32x4(at);
            LpPart p{d.x, d.y, d.z, d.w, ld_dsmem_s32(at + 16)};
            b = join(b, p);
          }
          consumers_sync();
          if (tid == 0) {
            sh->part = b;
            if (!is_odd(b.m)) finish(b, make_float2(0.f, 0.f), false);
          }
          if (top) {
            for (int i = tid; i < S * top; i += kLpThreads)
              sh->cand[i] = ld_dsmem_u64(cluster_map(smem_u32(&sh->best[i % top]), (uint32_t)(i / top)));
            consumers_sync();
            // (empty places hold 0 and may be many: they stay behind every key)
            for (int i = tid; i < S * top; i += kLpThreads) {
              const uint64_t mine = sh->cand[i];
              int n = 0;
              for (int j = 0; j < S * top; ++j) n += sh->cand[j] > mine || (sh->cand[j] == mine && j < i);
              if (n < top) sh->best[n] = mine;
            }
          }
          consumers_sync();
        }
      }
      if (slice == 0) {
        const LpPart b = sh->part;
        if (is_odd(b.m)) {   // (the same for all)
          const float2 again = row_again(sh, r.base, vocab, b.m);
          if (tid == 0) finish(b, again, true);
          consumers_sync();
        }
        for (int i = tid; i < top; i += kLpThreads) {
          const uint64_t key = sh->best[i];
          const float x = key_logit(key);
          const bool any = key != 0 && (sh->m < INFINITY || x == INFINITY);
          out.top_tokens[(size_t)row * top + i] = any ? key_token(key) : -1;
          out.top_logprobs[(size_t)row * top + i] =
              !any ? -INFINITY : sh->m == INFINITY ? (float)-sh->z : (float)((double)x - (double)sh->m - sh->z);
        }
      }
      consumers_sync();   // the shared parts are free for the next row
      token = next_token;
      xt = next_xt;
    }
  }
  if (S > 1) {
    if (warp == kLpWarps) cluster_sync();   // (the consumers' first one)
    cluster_sync();                         // no CTA leaves while another reads its parts
  }
}

size_t lp_smem_bytes() { return 128 + (size_t)kStages * kChunkBytes + sizeof(LpShared); }

template <typename T>
static cudaError_t launch_t(const T* logits, size_t stride, int rows, int vocab, const int32_t* tokens, int top,
                            const LpOut& out, int* err, cudaStream_t st) {
  auto k = k_token_logprobs<T>;
  const size_t smem = lp_smem_bytes();
  cudaError_t e = ensure_smem_optin(reinterpret_cast<const void*>(k), (int)smem);
  if (e != cudaSuccess) return e;
  // few rows: slices of at least one chunk, as many as CTAs fit beside one another
  const int resident = 2 * device_sm_count();
  const long long chunks = ((long long)vocab * (long long)sizeof(T) + kChunkBytes - 1) / kChunkBytes;
  int S = 1;
  while (S < 8 && (long long)2 * S * rows <= resident && 2 * S <= chunks) S *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(S, S > 1 ? rows : (rows < resident ? rows : resident));
  cfg.blockDim = dim3(kLpThreads + 32);
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
  return cudaLaunchKernelEx(&cfg, k, logits, stride, rows, vocab, tokens, top, out, err);
}

cudaError_t launch_token_logprobs(const void* logits, bool bf16, size_t stride, int rows, int vocab,
                                  const int32_t* tokens, int top, const LpOut& out, int* err, cudaStream_t st) {
  if (rows == 0) return cudaSuccess;
  return bf16 ? launch_t(static_cast<const uint16_t*>(logits), stride, rows, vocab, tokens, top, out, err, st)
              : launch_t(static_cast<const float*>(logits), stride, rows, vocab, tokens, top, out, err, st);
}

}  // namespace m2

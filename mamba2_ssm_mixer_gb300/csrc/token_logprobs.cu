// Log probabilities of given tokens, their ranks, the rows' entropy and the
// largest tokens, in one pass over the logits x:
//   m = max x, S = sum exp(x - m), E = sum exp(x - m) x / S
//   logprob(t) = (x_t - m) - log S, entropy = m + log S - E,
//   rank(t) = 1 + the tokens before t in the order (greater logit, lower token).
// Threads keep
//  - sums in base 2 with a whole number c as reference: u = fma(x, L, -c) with
//    L = f32(log2 e) is rounded once, S += 2^u, U += 2^u u.  What L lacks of
//    log2 e is put back at the end: lse = ln 2 (c + m (log2 e - L)) + log S.
//    Rows whose maximum is beyond +-2^16 (or +inf) are summed again as x - m
//    (row_again);
//  - the number of logits greater than the given token's;
//  - maxima of groups of their vectors.
// The k largest need no sort and no list on the way: if each of w warps has
// ceil(k / w) threads whose maximum is at least tau, at least k tokens are >=
// tau; only groups whose maximum reaches tau are looked at again, and the
// survivors are ranked by counting.  Where they are many, a sample of them
// gives the next tau; where many are equal, the first of those join the greater
// ones (survivors).
//
// k_lp_held (few rows, or short ones): a CTA, or each of a cluster's, holds its
// slice of one row in registers; the first CTA joins the slices' parts through
// distributed shared memory.  A row's latency is what counts: 1 x 131072 bf16
// takes 8.3 us of which 0.04 are its bytes', 64 x 65536 f32 8.9 (2.5).
// k_lp_stream (many long rows): two persistent CTAs per SM.  One warp copies
// chunks into a ring, from row to row without a pause; eight warps (the readers)
// sum; three warps (the selectors) find a row's largest tokens and write its
// results while the readers are at the next row.  2048 x 131072 f32 with 20
// tokens: 172 us (0.93 of the copy rate); 4096 x 131072 bf16: 201 (0.80), where
// the readers' latency counts (as many elements for half the bytes).  Shorter
// rows are bound by the selection of one, 12000 clocks beside the readers: 4096
// x 32000 bf16 takes 65 us without tokens to select, with 20 108.
#include <cuda_bf16.h>

#include "launch_util.h"
#include "m2_kernels.h"
#include "tc_ptx.cuh"

namespace m2 {

using namespace tc;

namespace {

constexpr int kReaders = 256;                       // threads of k_lp_stream's warps 0 .. 7
constexpr int kSelectors = 96;                      // of warps 8 .. 10; warp 11 copies
constexpr int kReadWarps = kReaders / 32, kSelWarps = kSelectors / 32;
constexpr int kStreamThreads = kReaders + kSelectors + 32;
constexpr int kVpt = 4;                             // 16-byte vectors per reader and chunk, at most
constexpr int kChunkVecs = kReaders * kVpt;
constexpr int kChunkBytes = kChunkVecs * 16;
constexpr int kStages = 3;
constexpr int kGroups = 16;                         // groups of vectors per reader
constexpr int kHeldThreads = 256;                   // of k_lp_held
constexpr int kHeldWarps = kHeldThreads / 32;
constexpr int kLpMaxSlices = 8;
constexpr float kL = 1.4426950408889634f;           // log2 e, rounded to f32
constexpr float kLn2 = 0.693147180559945309f, kLn2Lo = (float)(0.693147180559945309 - (double)kLn2);   // ln 2
constexpr double kLRest = 1.4426950408889634074 - (double)1.4426950408889634f;                         // log2 e - L
constexpr double kInvL = 1.0 / (double)1.4426950408889634f;
constexpr float kNone = -0x1p18f;                   // reference c before any unmasked logit
constexpr float kPlain = 0x1p16f;                   // |m| up to which c is exact enough

struct __align__(16) LpPart {
  float c, s, u, m;   // reference, sums, maximum
  int greater;        // logits before the given token's
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
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t d;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
  return d;
}

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
  // The elements that are at least lo, a bit each.
  __device__ static uint32_t reach(const uint4& q, float lo) {
    uint32_t which = 0;
#pragma unroll
    for (int e = 0; e < kN; ++e) which |= at(q, e) >= lo ? 1u << e : 0u;
    return which;
  }
  __device__ static void mask(uint4& q, int e) {
    uint32_t* w = reinterpret_cast<uint32_t*>(&q) + e / 2;
    *w = e & 1 ? (*w & 0xFFFFu) | 0xFF800000u : (*w & 0xFFFF0000u) | 0xFF80u;
  }
  using Max = uint32_t;   // of the even and of the odd elements
  __device__ static Max max(const uint4& q) { return max_bf16x2(max_bf16x2(q.x, q.y), max_bf16x2(q.z, q.w)); }
  __device__ static Max max(Max a, Max b) { return max_bf16x2(a, b); }
  __device__ static float whole(Max m) {
    return fmaxf(fmaxf(__uint_as_float(m << 16), __uint_as_float(m & 0xFFFF0000u)), -INFINITY);   // (NaN: -inf)
  }
  // Counts of logits greater than a bf16 value: the comparisons' masks (0xFFFF
  // a half) are summed as whole words, two per addition.  H and L of them:
  // sum = 65536 (L - H) - L modulo 2^32.
  struct Thr {
    __nv_bfloat162 v;
    __device__ explicit Thr(float thr) : v(__float2bfloat162_rn(thr)) {}
  };
  struct Count {
    uint32_t n = 0;
    __device__ void add(const uint4& q, const Thr& t) {
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) n += __hgt2_mask(*reinterpret_cast<const __nv_bfloat162*>(&w[i]), t.v);
    }
    __device__ int total() const {
      const uint32_t l = (0u - n) & 0xFFFFu, d = (n + l) >> 16;   // d = L - H modulo 2^16
      return (int)(2 * l - (uint32_t)(int)(int16_t)d);
    }
  };
  __device__ static float below(float x) { return next_below(x, 0x10000u); }
  struct Low {
    uint32_t v;
    __device__ explicit Low(float low) { v = pack_bf16x2(low, low); }
  };
  template <bool kFirst>   // (s and u begin here)
  __device__ static void sums(const uint4& q, const Low& low, uint64_t cc, uint64_t& s, uint64_t& u) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t x = max_bf16x2(w[i], low.v);
      const uint64_t d = fma_pair(pair(__uint_as_float(x << 16), __uint_as_float(x & 0xFFFF0000u)), pair(kL, kL), cc);
      const float2 t = unpair(d);
      const uint64_t p = pair(exp2_fast(t.x), exp2_fast(t.y));
      s = kFirst && i == 0 ? p : add_pair(s, p);
      u = kFirst && i == 0 ? mul_pair(p, d) : fma_pair(p, d, u);
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
  // The elements that are at least lo, a bit each.
  __device__ static uint32_t reach(const uint4& q, float lo) {
    uint32_t which = 0;
#pragma unroll
    for (int e = 0; e < kN; ++e) which |= at(q, e) >= lo ? 1u << e : 0u;
    return which;
  }
  __device__ static void mask(uint4& q, int e) { reinterpret_cast<uint32_t*>(&q)[e] = kNegInf; }
  using Max = float;
  __device__ static Max max(const uint4& q) { return fmaxf(fmaxf(at(q, 0), at(q, 1)), fmaxf(at(q, 2), at(q, 3))); }
  __device__ static Max max(Max a, Max b) { return fmaxf(a, b); }
  __device__ static float whole(Max m) { return fmaxf(m, -INFINITY); }
  struct Thr {
    float v;
    __device__ explicit Thr(float thr) : v(thr) {}
  };
  struct Count {
    int n = 0;
    __device__ void add(const uint4& q, const Thr& t) {
#pragma unroll
      for (int e = 0; e < 4; ++e) n += at(q, e) > t.v;
    }
    __device__ int total() const { return n; }
  };
  __device__ static float below(float x) { return next_below(x, 1u); }
  struct Low {
    float v;
    __device__ explicit Low(float low) : v(low) {}
  };
  template <bool kFirst>   // (s and u begin here)
  __device__ static void sums(const uint4& q, const Low& low, uint64_t cc, uint64_t& s, uint64_t& u) {
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
      const float a = at(q, i), b = at(q, i + 1);
      const uint64_t d = fma_pair(pair(fmaxf(a, low.v), fmaxf(b, low.v)), pair(kL, kL), cc);
      const float2 t = unpair(d);
      const uint64_t p = pair(exp2_fast(t.x), exp2_fast(t.y));
      s = kFirst && i == 0 ? p : add_pair(s, p);
      u = kFirst && i == 0 ? mul_pair(p, d) : fma_pair(p, d, u);
    }
  }
};

// Maximum of a thread's vectors.
template <typename T, int N>
__device__ __forceinline__ float max_of(const uint4 (&q)[N]) {
  using V = Vec<T>;
  typename V::Max m[N];
#pragma unroll
  for (int j = 0; j < N; ++j) m[j] = V::max(q[j]);
#pragma unroll
  for (int o = N / 2; o; o /= 2)
#pragma unroll
    for (int j = 0; j < o; ++j) m[j] = V::max(m[j], m[j + o]);
  return V::whole(m[0]);
}

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
// The parts of `n` neighbouring lanes (a power of two) as one.
__device__ __forceinline__ LpPart join_lanes(LpPart a, int n) {
  for (int o = n / 2; o; o >>= 1) {
    LpPart b;
    b.c = __shfl_xor_sync(0xffffffffu, a.c, o);
    b.s = __shfl_xor_sync(0xffffffffu, a.s, o);
    b.u = __shfl_xor_sync(0xffffffffu, a.u, o);
    b.m = __shfl_xor_sync(0xffffffffu, a.m, o);
    b.greater = __shfl_xor_sync(0xffffffffu, a.greater, o);
    a = join(a, b);
  }
  return a;
}
// A row that is summed again as x - m.
__device__ __forceinline__ bool is_odd(float m) { return m > -INFINITY && !(fabsf(m) <= kPlain); }

// A warp's n-th largest key (n <= 32).
__device__ __forceinline__ uint32_t nth_largest(uint32_t mine, int n, int lane) {
  uint32_t t = 0;
  for (int i = 0; i < n; ++i) {
    t = __reduce_max_sync(0xffffffffu, mine);
    if (__ffs(__ballot_sync(0xffffffffu, mine == t)) - 1 == lane) mine = 0;
  }
  return t;
}
// What one of `full` warps whose threads all have a vector gives to the bound
// that k tokens reach: its ceil(k / full)-th largest thread maximum; 0 (every
// token is looked at) where there are too few threads, all ones from a warp
// that does not count.
__device__ __forceinline__ uint32_t warp_tau(float thread_max, int k, int full, int warp, int lane) {
  const int need = full ? (k + full - 1) / full : 33;
  if (need > 32) return 0u;
  const uint32_t t = nth_largest(ord32(thread_max + 0.f), need, lane);
  return warp < full ? t : 0xffffffffu;
}

// The threads that select for a row.
struct SelectorGroup {
  static constexpr int kSize = kSelectors;
  int at;
  __device__ void sync() const { asm volatile("bar.sync 1, %0;" ::"n"(kSelectors) : "memory"); }
};
struct BlockGroup {
  static constexpr int kSize = kHeldThreads;
  int at;
  __device__ void sync() const { __syncthreads(); }
};

// Their shared state.
template <class G>
struct __align__(16) LpSelect {
  static constexpr int kCap = 512;     // survivors ranked by counting, at most
  uint64_t cand[kCap];
  uint64_t best[kLpMaxTop];            // the slice's largest keys, in order
  uint64_t merged[kLpMaxTop];          // the row's, from several slices'
  LpPart part, whole;                  // the slice's, the row's
  float z, z_lo, m;                    // log S of the row, relative to its maximum m, in two parts
  float h;                             // the entropy of one that was summed again
  int n_cand, n_hit, n_over;
  float sum[G::kSize / 32][2];
  int equal[G::kSize / 32];
};

// The k largest of cand[0, n) by counting, in order, to best[0, k) (n < k: the
// rest are 0).
template <class G>
__device__ __forceinline__ void rank_candidates(LpSelect<G>* sh, const G& g, int n, int k) {
  if (n <= 48) {
    if (g.at < n) {
      const uint64_t mine = sh->cand[g.at];
      int r = 0;
#pragma unroll 4
      for (int j = 0; j < n; ++j) r += sh->cand[j] > mine;
      if (r < k) sh->best[r] = mine;
    }
  } else {
    // two threads for each, on every other one (64 x 131072 bf16, 20 tokens: 11.7
    // us, by one thread each 12.1; with few survivors the exchange costs more than
    // it saves: 4096 x 1000 bf16, 20 tokens: 29.7, by two 31.4)
    for (int i0 = 0; i0 < n; i0 += G::kSize / 2) {
      const int i = i0 + g.at / 2;
      const uint64_t mine = sh->cand[min(i, n - 1)];
      int r = 0;
#pragma unroll 8
      for (int j = g.at & 1; j < n; j += 2) r += sh->cand[j] > mine;
      r += __shfl_xor_sync(0xffffffffu, r, 1);
      if (i < n && r < k) sh->best[r] = mine;
    }
  }
  for (int i = n + g.at; i < k; i += G::kSize) sh->best[i] = 0;
  g.sync();
}

// The elements of a vector per thread that equal x join the n survivors, the
// first ones in order of the threads until there are k; how many there are then.
template <typename T, class G>
__device__ __forceinline__ int append_equal(LpSelect<G>* sh, const G& g, const uint4& q, float x, int token, int n, int k) {
  using V = Vec<T>;
  const int lane = g.at & 31, warp = g.at >> 5;
  int at = 0, all = 0;
#pragma unroll
  for (int e = 0; e < V::kN; ++e) {
    const uint32_t who = __ballot_sync(0xffffffffu, V::at(q, e) == x);
    at += __popc(who & ((1u << lane) - 1u));
    all += __popc(who);
  }
  if (lane == 0) sh->equal[warp] = all;
  g.sync();
  all = 0;
#pragma unroll
  for (int w = 0; w < G::kSize / 32; ++w) {
    at += w < warp ? sh->equal[w] : 0;
    all += sh->equal[w];
  }
  at += n;
#pragma unroll
  for (int e = 0; e < V::kN; ++e)
    if (V::at(q, e) == x) {
      if (at < k) sh->cand[at] = key_of(x, token + e);
      ++at;
    }
  g.sync();
  return min(n + all, k);
}

// Those of a row's vectors [v0, v1).
template <typename T, class G>
__device__ __noinline__ int first_equal(LpSelect<G>* sh, const G g, const RowAt<T> r, int v0, int v1, float x, int n, int k) {
  using V = Vec<T>;
  constexpr int kAhead = 4;
  for (int v = v0; v < v1 && n < k; v += G::kSize * kAhead) {
    uint4 q[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      const int at = v + G::kSize * j + g.at;
      q[j] = at < v1 ? __ldg(r.vec + at) : make_uint4(V::kNegInf, V::kNegInf, V::kNegInf, V::kNegInf);
      if (at < v1 && r.edge(at)) r.edges(q[j], at);
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (n >= k) break;   // (the same for all)
      n = append_equal<T>(sh, g, q[j], x, (v + G::kSize * j + g.at) * V::kN - r.off, n, k);
    }
  }
  return n;
}

// The k largest keys to best[0, k), given a bound that k tokens reach (or
// every token above -inf does).  gather(lo) appends the tokens >= lo and
// returns how many there are, at least that there are more than kCap; where
// there are, the k-th largest of a sample of them is the next bound, and where
// the sample shows nothing but the bound itself, only what is greater is
// gathered and equal(x, n) adds the first tokens that equal it, in order, until
// there are k.  (512 rows of 131072 bf16 logits, 10 of them above a finite
// mask, 20 asked for: 79 us; another pass over the row against a running k-th
// best 594.)
template <typename T, class G, class Gather, class Equal>
__device__ __forceinline__ int survivors(LpSelect<G>* sh, const G& g, int k, float lo, Gather gather, Equal equal) {
  using V = Vec<T>;
  constexpr int kSample = 256;
  bool ties = false;   // tokens that equal `tie` are left out
  float tie = lo;
  int n;
  for (;;) {
    n = gather(lo);
    if (n <= LpSelect<G>::kCap) break;
    rank_candidates(sh, g, kSample, k);
    const float x = key_logit(sh->best[k - 1]);
    ties = x == lo;
    tie = lo;
    lo = ties ? -V::below(-lo) : x;
    g.sync();   // (all have read it)
    if (g.at == 0) sh->n_cand = 0, sh->n_hit = 0;
    g.sync();
  }
  return ties && n < k ? equal(tie, n) : n;
}

// a + b exactly, as a rounded sum and its error.
struct Two {
  float hi, lo;
};
__device__ __forceinline__ Two two_sum(float a, float b) {
  const float s = a + b, t = s - a;
  return {s, (a - (s - t)) + (b - t)};
}
// a + b for a in two parts.
__device__ __forceinline__ Two add(const Two& a, float b) {
  const Two s = two_sum(a.hi, b);
  return {s.hi, s.lo + a.lo};
}
// log s in two parts: s = 2^e f with f near 1, log s = e ln 2 + log f.
__device__ __forceinline__ Two log_parts(float s) {
  const int e = (int)((__float_as_uint(s) + 0x4AFB0Du) >> 23) - 127;
  const float lf = logf(__uint_as_float(__float_as_uint(s) - ((uint32_t)e << 23))), ef = (float)e;
  const float el = ef * kLn2;
  return add(add({el, fmaf(ef, kLn2, -el) + ef * kLn2Lo}, lf), 0.f);
}

// log S and the entropy of a row whose maximum m is finite and large, or +inf
// (then the +inf tokens share the probability), left in sh by the first thread.
// A thread adds up to 2^24 / 96 terms, which among equal logits err to the same
// side (as in Sums::carry): a vector's at first, these sums then with what is
// rounded off beside them.
template <typename T, class G>
__device__ __noinline__ void row_again(LpSelect<G>* sh, const G g, const RowAt<T> r, float m) {
  using V = Vec<T>;
  Two s = {0.f, 0.f}, u = {0.f, 0.f};
#pragma unroll 4
  for (int v = g.at; v < r.nv; v += G::kSize) {
    uint4 q = __ldg(r.vec + v);
    if (r.edge(v)) r.edges(q, v);
    float sv = 0.f, uv = 0.f;
#pragma unroll
    for (int e = 0; e < V::kN; ++e) {
      const float x = V::at(q, e);
      if (m == INFINITY) {
        sv += x == INFINITY ? 1.f : 0.f;
      } else {
        const float d = x - m, p = expf(d);
        if (p > 0.f) sv += p, uv = fmaf(p, d, uv);
      }
    }
    s = add(s, sv);
    u = add(u, uv);
  }
  float a = s.hi + s.lo, b = u.hi + u.lo;
#pragma unroll
  for (int o = 16; o; o >>= 1) a += __shfl_xor_sync(0xffffffffu, a, o), b += __shfl_xor_sync(0xffffffffu, b, o);
  g.sync();
  if ((g.at & 31) == 0) sh->sum[g.at >> 5][0] = a, sh->sum[g.at >> 5][1] = b;
  g.sync();
  a = b = 0.f;
#pragma unroll
  for (int w = 0; w < G::kSize / 32; ++w) a += sh->sum[w][0], b += sh->sum[w][1];
  if (g.at == 0) {
    const Two z = log_parts(a);
    sh->z = z.hi;
    sh->z_lo = z.lo;
    sh->h = z.hi - (b / a - z.lo);
  }
}

// A row and the token to score in it.
template <typename T>
struct LpJob {
  RowAt<T> r;
  int row, vocab, token;
  float xt;   // its logit
  __device__ bool valid() const { return token >= 0 && token < vocab; }
};

// x - m - z, rounded once but for the errors' errors.
__device__ __forceinline__ float minus_z(float x, float m, float z, float z_lo) {
  const Two d = two_sum(x, -m);
  if (!(fabsf(d.hi) < 0x1p100f)) return d.hi;   // (past what z can change, or infinite)
  const Two e = two_sum(d.hi, -z);
  return e.hi + (e.lo + (d.lo - z_lo));
}

// What the given token and the entropy get from the whole row's part b (one
// thread; an odd row's log S and entropy are in sh).  In pairs of f32 values: a
// double's operations take this one thread longer than the rest of a short
// row's.
template <typename T, class G>
__device__ __forceinline__ void finish(LpSelect<G>* sh, const LpJob<T>& job, const LpPart& b, const LpOut& out,
                                       bool scored, int* err) {
  float z = 0.f, z_lo = 0.f, h = 0.f;
  if (is_odd(b.m)) {
    z = sh->z, z_lo = sh->z_lo, h = sh->h;
  } else if (b.m > -INFINITY) {
    const Two ln = log_parts(b.s);
    // z = log S + (c ln 2 - m) + m (log2 e - L) ln 2
    const float rest = b.m * (float)(kLRest * 0.693147180559945309), cl = b.c * kLn2;
    const Two dc = two_sum(cl, -b.m);
    Two t = add(ln, dc.hi);
    t.lo += dc.lo + (fmaf(b.c, kLn2, -cl) + b.c * kLn2Lo) + rest;
    z = t.hi + t.lo;
    z_lo = t.lo - (z - t.hi);
    // h = log S - (U / S) / L + c (ln 2 - 1 / L) + m (log2 e - L) ln 2
    const float q = __fdividef(b.u, b.s), ql = __fdividef(fmaf(-q, b.s, b.u), b.s), qi = q * (float)kInvL;   // U / S in two parts
    const Two g = add(ln, -qi);
    h = g.hi + (g.lo - (fmaf(q, (float)kInvL, -qi) + q * (float)(kInvL - (double)(float)kInvL) + ql * (float)kInvL) +
                (b.c * (float)(0.693147180559945309 - kInvL) + rest));
  }
  sh->z = z;
  sh->z_lo = z_lo;
  sh->m = b.m;
  if (out.entropy) out.entropy[job.row] = fmaxf(h, 0.f);
  if (!scored) return;
  float lp = 0.f;
  int rank = 0;
  if (job.valid()) {
    lp = !(job.xt > -INFINITY) ? -INFINITY
         : b.m == INFINITY     ? (job.xt == INFINITY ? -z : -INFINITY)
                               : minus_z(job.xt, b.m, z, z_lo);
    rank = 1 + b.greater;
  } else if (job.token != -1 && err) {
    atomicOr(err, kErrToken);
  }
  out.logprobs[job.row] = lp;
  out.ranks[job.row] = rank;
}

// From the slice's part and largest keys (sh->part, sh->best; S = 1: the whole
// row's, finished unless it is odd) to the row's results.  S > 1: by the first
// slice's CTA, between the cluster's two barriers, the second of which it
// passes itself when it has read the others' parts; sh->merged is 0.
template <typename T, class G>
__device__ __forceinline__ void row_results(LpSelect<G>* sh, const G& g, const LpJob<T>& job, int S, int top,
                                            const LpOut& out, bool scored, int* err) {
  const uint64_t* best = sh->best;
  if (S > 1) {
    const bool last = g.at >= G::kSize - 32;   // (a warp whose keys, if any, are few)
    LpPart mine;
    if (last) {   // a lane per slice
      const uint32_t at = cluster_map(smem_u32(&sh->part), (uint32_t)(g.at & (S - 1)));
      const float4 d = ld_dsmem_f32x4(at);
      mine = {d.x, d.y, d.z, d.w, __float_as_int(ld_dsmem_f32(at + 16))};
    }
    for (int i = g.at; i < S * top; i += G::kSize)
      sh->cand[i] = ld_dsmem_u64(cluster_map(smem_u32(&sh->best[i % top]), (uint32_t)(i / top)));
    g.sync();
    cluster_sync();
    // a key's place: its own slice's keys before it, and those of the other
    // slices that are greater (each list is in order, empty places hold 0)
    for (int i = g.at; i < S * top; i += G::kSize) {
      const uint64_t key = sh->cand[i];
      if (key == 0) continue;
      int lo[kLpMaxSlices], hi[kLpMaxSlices];   // the first that is not greater lies in [lo, hi]
#pragma unroll
      for (int o = 0; o < kLpMaxSlices; ++o) lo[o] = 0, hi[o] = o < S && o != i / top ? top : 0;
      for (int width = top; width; width >>= 1)
#pragma unroll
        for (int o = 0; o < kLpMaxSlices; ++o)
          if (lo[o] < hi[o]) {
            const int mid = (lo[o] + hi[o]) >> 1;
            if (sh->cand[o * top + mid] > key) lo[o] = mid + 1; else hi[o] = mid;
          }
      int n = i % top;
#pragma unroll
      for (int o = 0; o < kLpMaxSlices; ++o) n += lo[o];
      if (n < top) sh->merged[n] = key;
    }
    __syncwarp();
    if (last) {
      const LpPart b = join_lanes(mine, S);
      if (g.at == G::kSize - 32) {
        sh->whole = b;
        if (!is_odd(b.m)) finish(sh, job, b, out, scored, err);
      }
      __syncwarp();
    }
    g.sync();
    best = sh->merged;
  }
  const LpPart b = S > 1 ? sh->whole : sh->part;
  if (is_odd(b.m)) {   // (the same for all)
    row_again<T, G>(sh, g, job.r, b.m);
    if (g.at == 0) finish(sh, job, b, out, scored, err);
    g.sync();
  }
  for (int i = g.at; i < top; i += G::kSize) {
    const uint64_t key = best[i];
    const float x = key_logit(key);
    const bool any = key != 0 && (sh->m < INFINITY || x == INFINITY);
    out.top_tokens[(size_t)job.row * top + i] = any ? key_token(key) : -1;
    out.top_logprobs[(size_t)job.row * top + i] =
        !any ? -INFINITY : sh->m == INFINITY ? -sh->z : minus_z(x, sh->m, sh->z, sh->z_lo);
  }
}

// A thread's sums s and u relative to its reference c, in pairs.
template <typename T>
struct Sums {
  using V = Vec<T>;
  float c = kNone;
  uint64_t s = pair(0.f, 0.f), u = pair(0.f, 0.f);

  // The reference moves where a maximum passes it by 16.
  __device__ bool passes(float mx) const { return mx * kL > c + 16.f; }
  __device__ void reach(float mx) {
    if (passes(mx)) {
      const float cn = rintf(mx * kL), d = fmaxf(c - cn, -1e30f), f = exp2_fast(d);
      u = fma_pair(fma_pair(s, pair(d, d), u), pair(f, f), pair(0.f, 0.f));
      s = fma_pair(s, pair(f, f), pair(0.f, 0.f));
      c = cn;
    }
  }
  // Masked logits and NaN take a value whose exponential is 0 (-160 in base 2
  // at least, finite: 0 times it is 0).
  __device__ typename V::Low low() const {
    const float l = (c - 160.f) * 0.6931472f;
    return typename V::Low(fmaf(fabsf(l), -0.01f, l));
  }
  __device__ LpPart part(float m, int greater) const {
    const float2 a = unpair(s), b = unpair(u);
    return {c, a.x + a.y, b.x + b.y, m, greater};
  }
};

// What a reader of a long row has put by of its sums (in shared memory: it has
// no registers left).  Among equal logits each addition errs to the same side, and
// n terms one after another by up to n / 2 of the last place (in a row of 2^24
// tokens 2^-13 of S).  So a chunk is summed by itself, its sum joins the thread's,
// and after kCarry chunks that is put by: what this addition rounds off stays
// behind as the next sum's first term.
constexpr int kCarry = 16;
struct LpCarried {
  float c, s, u;
};
template <typename T>
__device__ __forceinline__ void carry(LpCarried& to, Sums<T>& sums, bool first) {
  const float2 a = unpair(sums.s), b = unpair(sums.u);
  const float x = a.x + a.y, y = b.x + b.y;
  float s0 = 0.f, u0 = 0.f;
  if (!first) {
    const float d = to.c - sums.c, f = exp2_fast(d);   // (a reference only grows)
    s0 = to.s * f, u0 = fmaf(to.s, d, to.u) * f;
  }
  const float s = s0 + x, u = u0 + y;
  to = {sums.c, s, u};
  sums.s = pair(x - (s - s0), 0.f);
  sums.u = pair(y - (u - u0), 0.f);
}

}  // namespace

template <typename T, int VPT>
__global__ void __launch_bounds__(kHeldThreads, VPT == 16 ? 2 : VPT == 8 ? 3 : 5)
    k_lp_held(const T* __restrict__ logits, size_t stride, int vocab, const int32_t* __restrict__ tokens, int top,
              LpOut out, int S, int* err) {
  using V = Vec<T>;
  constexpr int kLists = 512;   // vectors with a token that reaches the bound
  __shared__ LpSelect<BlockGroup> sel;
  __shared__ uint4 vecs[kLists];
  __shared__ int vec_at[kLists];
  __shared__ LpPart parts[kHeldWarps];
  __shared__ uint32_t taus[kHeldWarps];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int row = (int)(blockIdx.x / (unsigned)S), slice = (int)(blockIdx.x % (unsigned)S);
  const RowAt<T> r(logits, stride, row, vocab);
  const BlockGroup g{tid};
  const int v0 = (int)((long long)r.nv * slice / S), v1 = (int)((long long)r.nv * (slice + 1) / S);
  if (tid == 0) sel.n_cand = 0, sel.n_hit = 0;
  if (tid < kLpMaxTop) sel.merged[tid] = 0;
  pdl_wait();
  pdl_trigger();

  uint4 q[VPT];
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int v = v0 + j * kHeldThreads + tid;
    q[j] = v < v1 ? __ldg(r.vec + v) : make_uint4(V::kNegInf, V::kNegInf, V::kNegInf, V::kNegInf);
  }
  LpJob<T> job{r, row, vocab, tokens ? tokens[row] : -1, 0.f};
  if (job.valid()) job.xt = V::load(r.base + job.token);
#pragma unroll
  for (int j = 0; j < VPT; ++j) {
    const int v = v0 + j * kHeldThreads + tid;
    if (v < v1 && r.edge(v)) r.edges(q[j], v);
  }
  const float mx = max_of<T>(q);
  Sums<T> sums;
  if (sums.passes(mx)) {
    sums.c = rintf(mx * kL);
    const typename V::Low low = sums.low();
    const uint64_t cc = pair(-sums.c, -sums.c);
    uint64_t s[2], u[2];   // (of every other vector: up to 32 terms one after another)
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      if (j < 2)
        V::template sums<true>(q[j], low, cc, s[j], u[j]);
      else
        V::template sums<false>(q[j], low, cc, s[j & 1], u[j & 1]);
    }
    sums.s = VPT > 1 ? add_pair(s[0], s[VPT > 1]) : s[0];
    sums.u = VPT > 1 ? add_pair(u[0], u[VPT > 1]) : u[0];
  }
  int greater = 0;
  if (job.valid()) {   // before the given token's vector equal logits count as greater
    const bool masked = !(job.xt > -INFINITY);
    const int vt = masked ? -1 : (job.token + r.off) / V::kN;
    const typename V::Thr above(masked ? -INFINITY : job.xt), from(masked ? -INFINITY : V::below(job.xt));
    typename V::Count count;
#pragma unroll
    for (int j = 0; j < VPT; ++j) {
      const int v = v0 + j * kHeldThreads + tid;
      if (v != vt) {
        count.add(q[j], v < vt ? from : above);
      } else {
#pragma unroll
        for (int e = 0; e < V::kN; ++e) {
          const float x = V::at(q[j], e);
          greater += x > job.xt || (x == job.xt && v * V::kN + e - r.off < job.token);
        }
      }
    }
    greater += count.total();
  }
  const LpPart a = join_lanes(sums.part(mx, greater), 32);
  if (lane == 0) parts[warp] = a;
  if (top) {
    const uint32_t t = warp_tau(mx, top, min(kHeldWarps, (v1 - v0) / 32), warp, lane);
    if (lane == 0) taus[warp] = t;
  }
  __syncthreads();
  if (warp == 0) {
    const LpPart b = join_lanes(parts[lane & (kHeldWarps - 1)], kHeldWarps);
    if (lane == 0) sel.part = b;
  }
  if (top) {
    uint32_t tau = kOrdNegInf + 1, t = taus[0];
#pragma unroll
    for (int w = 1; w < kHeldWarps; ++w) t = min(t, taus[w]);
    tau = max(tau, t);
    const float bound = unord32(tau);
    // vectors that reach the bound, then their tokens, one per thread
    bool first = true;
    auto gather = [&](float lo) {
      if (mx >= lo) {
#pragma unroll
        for (int j = 0; j < VPT; ++j)
          if (V::whole(V::max(q[j])) >= lo) {
            const int at = atomicAdd(&sel.n_hit, 1);
            if (at < kLists) vecs[at] = q[j], vec_at[at] = v0 + j * kHeldThreads + tid;
          }
      }
      __syncthreads();
      const int hits = min(sel.n_hit, kLists);   // (each has a token: beyond kLists there are too many)
      for (int i = tid; i < hits * V::kN; i += kHeldThreads) {
        const float x = V::load(reinterpret_cast<const T*>(vecs) + i);
        if (x >= lo) {
          const int at = atomicAdd(&sel.n_cand, 1);
          if (at < sel.kCap) sel.cand[at] = key_of(x, vec_at[i / V::kN] * V::kN + i % V::kN - r.off);
        }
      }
      if (first && S == 1 && tid == 32 * (kHeldWarps - 1) && !is_odd(sel.part.m))   // (beside the others' search)
        finish(&sel, job, sel.part, out, tokens != nullptr, err);
      first = false;
      __syncthreads();
      return max(sel.n_cand, sel.n_hit);
    };
    auto equal = [&](float x, int n) {
#pragma unroll
      for (int j = 0; j < VPT; ++j) {
        if (n >= top) break;   // (the same for all)
        n = append_equal<T>(&sel, g, q[j], x, (v0 + j * kHeldThreads + tid) * V::kN - r.off, n, top);
      }
      return n;
    };
    rank_candidates(&sel, g, survivors<T>(&sel, g, top, bound, gather, equal), top);
  } else {
    __syncthreads();
    if (S == 1 && tid == 0 && !is_odd(sel.part.m))
      finish(&sel, job, sel.part, out, tokens != nullptr, err);
  }
  if (S > 1) {
    cluster_sync();
    if (slice != 0) {
      cluster_sync();   // (no CTA leaves while another reads its parts)
      return;
    }
  }
  row_results(&sel, g, job, S, top, out, tokens != nullptr, err);
}

namespace {

// What the readers hand over of a row.
struct __align__(16) LpRow {
  uint32_t gmax[kGroups][kReaders];   // maxima of a reader's groups
  uint32_t tmax[kReaders];            // and of all of them
  LpPart warp[kReadWarps];
  uint32_t tau[kReadWarps];
};

struct __align__(16) LpShared {
  uint64_t full[kStages], empty[kStages];        // the ring's
  uint64_t read[2], taken[2];                    // the two rows'
  LpRow row[2];
  LpCarried carried[kReaders];
  LpSelect<SelectorGroup> sel;
  uint16_t over[kReaders];                       // readers whose maximum reaches the bound
  uint16_t hits[kGroups * kReaders];             // and their groups
  int abort;
};

// How a slice of nv vectors is cut: chunks, and chunks of a group.
struct Cut {
  int chunks, group;
  __device__ explicit Cut(int nv) : chunks((nv + kChunkVecs - 1) / kChunkVecs), group((chunks + kGroups - 1) / kGroups) {}
};

}  // namespace

// kLong: slices of more than 2^17 tokens, whose sums are put by on the way.  Up to
// there a thread's sums are 32 chunks' of 8 terms (bf16: 16 of 16) one after
// another.  2000 x 151937 bf16: 129 us, without it 126; 4096 x 131072 with it
// 204, without it 201.
template <typename T, bool kLong>
__global__ void __launch_bounds__(kStreamThreads, 2)
    k_lp_stream(const T* __restrict__ logits, size_t stride, int rows, int vocab, const int32_t* __restrict__ tokens,
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
      mbar_init(&sh->empty[s], kReadWarps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sh->read[i], kReadWarps);
      mbar_init(&sh->taken[i], kSelWarps);
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
  // a warp's wait (asleep: polling warps would take issue slots from the
  // others); after one that ran out the rows left go through without data
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return;
    const bool there = *abort ? false : mbar_wait_sleep(bar, parity, abort);
    if (!__all_sync(0xffffffffu, there)) {
      *abort = 1;
      if (err && lane == 0) atomicOr(err, kErrTimeout);
    }
  };
  auto token_of = [&](int row) { return tokens && row < rows ? tokens[row] : -1; };
  auto valid = [&](int t) { return t >= 0 && t < vocab; };
  auto logit_of = [&](int row, int t) { return valid(t) ? V::load(logits + (size_t)row * stride + t) : 0.f; };

  if (warp == kReadWarps + kSelWarps) {
    if (lane == 0) {
      // ---------------- copies
      int stage = 0, issued = 0;
      uint32_t phase = 0;
      for (int row = row0; row < rows && !*abort; row += row_step) {
        const RowAt<T> r(logits, stride, row, vocab);
        int v0, v1;
        slice_of(r, v0, v1);
        const Cut cut(v1 - v0);
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
  } else if (warp < kReadWarps) {
    // ---------------- readers
    int stage = 0, turn = 0;
    uint32_t phase = 0, turn_phase = 0;
    // the tokens to score and their logits are asked for a row ahead of their use
    int token = token_of(row0), token1 = token_of(row0 + row_step);
    float xt = logit_of(row0, token);
    for (int row = row0; row < rows; row += row_step) {
      const RowAt<T> r(logits, stride, row, vocab);
      int v0, v1;
      slice_of(r, v0, v1);
      const Cut cut(v1 - v0);
      const float xt1 = logit_of(row + row_step, token1);
      const int token2 = token_of(row + 2 * row_step);
      const bool masked = !(xt > -INFINITY);                    // (NaN too)
      // before the given token's vector equal logits count as greater
      const int vt = valid(token) && !masked ? (token + r.off) / V::kN : -1;
      const typename V::Thr above(masked ? -INFINITY : xt), from(masked ? -INFINITY : V::below(xt));
      LpRow& hand = sh->row[turn];
      wait(&sh->taken[turn], turn_phase ^ 1u);

      Sums<T> sums;
      float m = -INFINITY, gm = -INFINITY;
      int greater = 0, group = 0, left = cut.group;
      auto chunks = [&](int ch, int to) {
        for (; ch < to; ++ch) {
          wait(&sh->full[stage], phase);
          const int vc = v0 + ch * kChunkVecs;
          const uint4* p = reinterpret_cast<const uint4*>(ring + stage * kChunkBytes) + tid;
          uint4 q[kVpt];
          if (ch > 0 && ch + 1 < cut.chunks) {
#pragma unroll
            for (int j = 0; j < kVpt; ++j) q[j] = p[j * kReaders];
          } else {
#pragma unroll
            for (int j = 0; j < kVpt; ++j) {
              const int v = vc + j * kReaders + tid;
              q[j] = v < v1 ? p[j * kReaders] : make_uint4(V::kNegInf, V::kNegInf, V::kNegInf, V::kNegInf);
              if (v < v1 && r.edge(v)) r.edges(q[j], v);
            }
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&sh->empty[stage]);
          if (++stage == kStages) stage = 0, phase ^= 1u;

          const float mx = max_of<T>(q);
          gm = fmaxf(gm, mx);
          if (--left == 0 || ch + 1 == cut.chunks) {
            if (top) hand.gmax[group][tid] = ord32(gm + 0.f);
            m = fmaxf(m, gm);
            gm = -INFINITY;
            ++group;
            left = cut.group;
          }
          sums.reach(mx);
          // (while everything is masked the reference is kNone and what is added 0)
          const uint64_t cc = pair(-sums.c, -sums.c);
          const typename V::Low low = sums.low();
          uint64_t s, u;
          V::template sums<true>(q[0], low, cc, s, u);
#pragma unroll
          for (int j = 1; j < kVpt; ++j) V::template sums<false>(q[j], low, cc, s, u);
          sums.s = add_pair(sums.s, s);
          sums.u = add_pair(sums.u, u);
          typename V::Count count;
          if (vt < vc || vt >= vc + kChunkVecs) {   // (the same for all)
            const typename V::Thr t = vt < vc ? above : from;
#pragma unroll
            for (int j = 0; j < kVpt; ++j)
              count.add(q[j], t);
          } else {
#pragma unroll
            for (int j = 0; j < kVpt; ++j) {
              const int v = vc + j * kReaders + tid;
              if (v != vt) {
                count.add(q[j], v < vt ? from : above);
              } else {
#pragma unroll
                for (int e = 0; e < V::kN; ++e) {
                  const float x = V::at(q[j], e);
                  greater += x > xt || (x == xt && v * V::kN + e - r.off < token);
                }
              }
            }
          }
          greater += count.total();
        }
      };
      if constexpr (kLong) {
#pragma unroll 1
        for (int ch = 0; ch < cut.chunks; ch += kCarry) {
          if (ch > 0) carry(sh->carried[tid], sums, ch == kCarry);
          chunks(ch, min(ch + kCarry, cut.chunks));
        }
      } else {
        chunks(0, cut.chunks);
      }
      // ---------------- the warp's part to the selectors
      LpPart a = sums.part(m, greater);
      if (kLong && cut.chunks > kCarry) {
        const LpCarried& b = sh->carried[tid];
        a = join(a, {b.c, b.s, b.u, -INFINITY, 0});
      }
      a = join_lanes(a, 32);
      if (lane == 0) hand.warp[warp] = a;
      if (top) {
        hand.tmax[tid] = ord32(m + 0.f);
        const uint32_t t = warp_tau(m, top, min(kReadWarps, (v1 - v0) / 32), warp, lane);
        if (lane == 0) hand.tau[warp] = t;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->read[turn]);
      if (++turn == 2) turn = 0, turn_phase ^= 1u;
      token = token1, token1 = token2;
      xt = xt1;
    }
  } else {
    // ---------------- selectors
    LpSelect<SelectorGroup>* sel = &sh->sel;
    const SelectorGroup g{tid - kReaders};
    int turn = 0;
    uint32_t turn_phase = 0;
    for (int row = row0; row < rows; row += row_step) {
      LpJob<T> job{RowAt<T>(logits, stride, row, vocab), row, vocab, token_of(row), 0.f};
      const RowAt<T>& r = job.r;
      int v0, v1;
      slice_of(r, v0, v1);
      const Cut cut(v1 - v0);
      job.xt = logit_of(row, job.token);
      if (g.at == 0) sel->n_cand = 0, sel->n_hit = 0, sel->n_over = 0;
      g.sync();
      wait(&sh->read[turn], turn_phase);
      const LpRow& hand = sh->row[turn];
      if (warp == kReadWarps + kSelWarps - 1) {   // (beside the others' search)
        const LpPart b = join_lanes(lane < kReadWarps ? hand.warp[lane] : LpPart{kNone, 0.f, 0.f, -INFINITY, 0}, 16);
        if (lane == 0) {
          sel->part = b;
          if (S == 1 && !is_odd(b.m)) finish(sel, job, b, out, tokens != nullptr, err);
        }
        __syncwarp();
      }
      int found = 0;
      if (top) {
        const uint32_t tau = max(kOrdNegInf + 1, __reduce_min_sync(0xffffffffu, lane < kReadWarps ? hand.tau[lane] : 0xffffffffu));
        const float bound = unord32(tau);
        // the readers and their groups with a token that reaches the bound, then
        // the groups' vectors, one per thread, a few loads under way
        const int groups = cut.chunks ? (cut.chunks + cut.group - 1) / cut.group : 0;
        const int per_hit = cut.group * kVpt;
        constexpr int kAhead = 4;
        for (int i = g.at; i < kReaders; i += kSelectors)
          if (hand.tmax[i] >= tau) sh->over[atomicAdd(&sel->n_over, 1)] = (uint16_t)i;
        g.sync();
        const int pairs = sel->n_over * groups;
        auto gather = [&](float lo) {
          const uint32_t key = ord32(lo);
          for (int i = g.at; i < pairs; i += kSelectors) {
            const int j = i % groups, who = sh->over[i / groups];
            if (hand.gmax[j][who] >= key) sh->hits[atomicAdd(&sel->n_hit, 1)] = (uint16_t)(j * kReaders + who);
          }
          g.sync();
          const int total = sel->n_hit * per_hit;
          volatile int* n_cand = &sel->n_cand;
#pragma unroll 1
          for (int i0 = g.at; i0 < total && *n_cand <= sel->kCap; i0 += kSelectors * kAhead) {
            uint4 q[kAhead];
            int v[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
              const int i = i0 + kSelectors * k;
              v[k] = v1;
              if (i < total) {
                const int hit = sh->hits[i / per_hit], j = i % per_hit;
                v[k] = v0 + (hit / kReaders * per_hit + j) * kReaders + hit % kReaders;
              }
              if (v[k] < v1) q[k] = __ldg(r.vec + v[k]);
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
              if (v[k] >= v1) continue;
              if (r.edge(v[k])) r.edges(q[k], v[k]);
              for (uint32_t which = V::reach(q[k], lo); which; which &= which - 1) {
                const int e = __ffs(which) - 1, n = atomicAdd(&sel->n_cand, 1);
                if (n < sel->kCap) sel->cand[n] = key_of(V::at(q[k], e), v[k] * V::kN + e - r.off);
              }
            }
          }
          g.sync();
          return sel->n_cand;
        };
        auto equal = [&](float x, int n) { return first_equal<T>(sel, g, r, v0, v1, x, n, top); };
        found = survivors<T>(sel, g, top, bound, gather, equal);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->taken[turn]);   // what the readers handed over is read
      if (++turn == 2) turn = 0, turn_phase ^= 1u;
      if (top)
        rank_candidates(sel, g, found, top);
      else
        g.sync();
      if (S > 1) {   // (the other warps arrive too, below)
        for (int i = g.at; i < kLpMaxTop; i += kSelectors) sel->merged[i] = 0;
        cluster_sync();
        if (slice != 0) cluster_sync();
      }
      if (slice == 0) row_results(sel, g, job, S, top, out, tokens != nullptr, err);
      g.sync();   // the shared results are free for the next row
    }
  }
  if (S > 1 && (warp < kReadWarps || warp == kReadWarps + kSelWarps)) {
    // one row: the selectors' two, between which another CTA reads this one's parts
    cluster_sync();
    cluster_sync();
  }
}

namespace {

template <typename K, typename... A>
cudaError_t launch_cluster(K kernel, dim3 grid, int threads, size_t smem, int cluster, cudaStream_t st, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename T>
cudaError_t launch_t(const T* logits, size_t stride, int rows, int vocab, const int32_t* tokens, int top,
                     const LpOut& out, int* err, cudaStream_t st) {
  const int sms = device_sm_count();
  // vectors of a row (one more where rows start on different places of theirs)
  const bool aligned = (uintptr_t)logits % 16 == 0 && (rows == 1 || stride * sizeof(T) % 16 == 0);
  const int nv = (int)(((long long)vocab + (aligned ? 1 : 2) * (Vec<T>::kN - 1)) / Vec<T>::kN);
  // The fewest slices that registers hold, then more while CTAs fit beside one
  // another and have a vector per thread.  A thread holds up to 8 vectors, or 16
  // where all rows run at once, two CTAs on an SM (200 x 16000 f32: 7.5 us,
  // streamed 9.6; 4096 x 16000: 91, streamed 79, and of 8 vectors 4096 x 8000: 51,
  // streamed 77).  Rows in several slices only where all run at once (64 x 131072
  // bf16, 4 slices of 16 vectors: 12.0 us, streamed 16.3; 8 slices of 8, two
  // waves: 21.5).
  const int held = kHeldThreads * (rows <= 2 * sms ? 16 : 8);
  int S = 1;
  while (S < kLpMaxSlices && (nv + S - 1) / S > held) S *= 2;
  if ((nv + S - 1) / S <= held && (S == 1 || (long long)S * rows <= 2 * sms)) {
    while (S < kLpMaxSlices && (long long)2 * S * rows <= 2 * sms && nv / (2 * S) >= kHeldThreads) S *= 2;
    const int per = ((nv + S - 1) / S + kHeldThreads - 1) / kHeldThreads;
    auto go = [&](auto k) {
      return launch_cluster(k, dim3((unsigned)S * (unsigned)rows), kHeldThreads, 0, S, st, logits, stride, vocab, tokens,
                            top, out, S, err);
    };
    if (per <= 1) return go(k_lp_held<T, 1>);
    if (per <= 2) return go(k_lp_held<T, 2>);
    if (per <= 4) return go(k_lp_held<T, 4>);
    if (per <= 8) return go(k_lp_held<T, 8>);
    return go(k_lp_held<T, 16>);
  }
  const size_t smem = 128 + (size_t)kStages * kChunkBytes + sizeof(LpShared);
  S = 1;
  while (S < kLpMaxSlices && (long long)2 * S * rows <= 2 * sms && 2ll * S * kChunkVecs <= nv) S *= 2;
  const auto k = vocab > S << 17 ? k_lp_stream<T, true> : k_lp_stream<T, false>;
  const cudaError_t e = ensure_smem_optin(reinterpret_cast<const void*>(k), (int)smem);
  if (e != cudaSuccess) return e;
  return launch_cluster(k, dim3(S, S > 1 ? rows : (rows < 2 * sms ? rows : 2 * sms)), kStreamThreads, smem, S, st, logits,
                        stride, rows, vocab, tokens, top, out, err);
}

}  // namespace

cudaError_t launch_token_logprobs(const void* logits, bool bf16, size_t stride, int rows, int vocab,
                                  const int32_t* tokens, int top, const LpOut& out, int* err, cudaStream_t st) {
  if (rows == 0) return cudaSuccess;
  return bf16 ? launch_t(static_cast<const uint16_t*>(logits), stride, rows, vocab, tokens, top, out, err, st)
              : launch_t(static_cast<const float*>(logits), stride, rows, vocab, tokens, top, out, err, st);
}

}  // namespace m2

// Log probabilities of given tokens, their ranks, the rows' entropy and the
// largest tokens, in one pass over the logits x:
//   m = max x, S = sum exp(x - m), E = sum exp(x - m) x / S
//   logprob(t) = (x_t - m) - log S, entropy = m + log S - E,
//   rank(t) = 1 + the tokens before t in the order (greater logit, lower token).
//
// k_token_logprobs: a CTA takes a row, or a slice of one where rows are few (the
// slices' CTAs form a cluster and the first of them joins the parts through
// distributed shared memory).  One warp streams 16 KB chunks into a ring with
// bulk copies, from row to row without a pause.  Eight warps (the readers) keep
// per thread
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
// k-th best (top_again).  Three warps (the selectors) do that and write a row's
// results while the readers are at the next row.
#include <cuda_bf16.h>

#include "launch_util.h"
#include "m2_kernels.h"
#include "tc_ptx.cuh"

namespace m2 {

using namespace tc;

namespace {

constexpr int kReaders = 256;                       // threads of warps 0 .. 7
constexpr int kSelectors = 96;                      // of warps 8 .. 10; warp 11 copies
constexpr int kReadWarps = kReaders / 32, kSelWarps = kSelectors / 32;
constexpr int kLpThreads = kReaders + kSelectors + 32;
constexpr int kVpt = 4;                             // 16-byte vectors per reader and chunk
constexpr int kChunkVecs = kReaders * kVpt;
constexpr int kChunkBytes = kChunkVecs * 16;
constexpr int kStages = 3;                          // with two CTAs per SM
constexpr int kGroups = 16;                         // groups of vectors per reader
constexpr int kLpCap = 1024;                        // survivors ranked by counting
constexpr float kL = 1.4426950408889634f;           // log2 e, rounded to f32
constexpr double kLn2 = 0.6931471805599453094;
constexpr double kLRest = 1.4426950408889634074 - (double)1.4426950408889634f;   // log2 e - L
constexpr float kNone = -0x1p18f;                   // reference c before any unmasked logit
constexpr float kPlain = 0x1p16f;                   // |m| up to which c is exact enough

struct __align__(16) LpPart {
  float c, s, u, m;   // reference, sums, maximum
  float greater;      // logits before the given token's (below 2^24: exact)
};

// What the readers hand over of a row.
struct __align__(16) LpRow {
  uint32_t gmax[kGroups][kReaders];
  LpPart warp[kReadWarps];
  uint32_t tau[kReadWarps];
};

struct __align__(16) LpShared {
  uint64_t full[kStages], empty[kStages];   // the ring's
  uint64_t read[2], taken[2];               // the two LpRow's
  uint64_t cand[kLpCap];
  uint64_t best[kLpMaxTop];                 // the slice's largest keys, in order
  LpRow row[2];
  LpPart part;                              // the slice's
  double z;                                 // log S of the whole row (relative to its maximum m)
  float m;
  int n_cand, n_hit, abort;
  float sum[kSelWarps][2];
  uint32_t step_tau[kSelWarps];
  uint16_t hits[kGroups * kReaders];        // groups whose maximum reaches the threshold
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

// Barrier of the selectors; sel_any: whether `p` holds for one of them.
__device__ __forceinline__ void sel_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kSelectors) : "memory"); }
__device__ __forceinline__ bool sel_any(bool p) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.red.or.pred q, 1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}\n"
      : "=r"(r)
      : "r"((uint32_t)p), "n"(kSelectors)
      : "memory");
  return r != 0;
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
  __device__ static void mask(uint4& q, int e) {
    uint32_t* w = reinterpret_cast<uint32_t*>(&q) + e / 2;
    *w = e & 1 ? (*w & 0xFFFFu) | 0xFF800000u : (*w & 0xFFFF0000u) | 0xFF80u;
  }
  __device__ static float max(const uint4 (&q)[kVpt]) {
    uint32_t m[kVpt];
#pragma unroll
    for (int j = 0; j < kVpt; ++j) m[j] = max_bf16x2(max_bf16x2(q[j].x, q[j].y), max_bf16x2(q[j].z, q[j].w));
#pragma unroll
    for (int o = kVpt / 2; o; o /= 2)
#pragma unroll
      for (int j = 0; j < o; ++j) m[j] = max_bf16x2(m[j], m[j + o]);
    return fmaxf(__uint_as_float(m[0] << 16), __uint_as_float(m[0] & 0xFFFF0000u));
  }
  // Counts of logits greater than a bf16 value, in bf16 pairs: exact up to 256
  // a half, of which a chunk's vectors give 32.
  struct Thr {
    __nv_bfloat162 v;
    __device__ explicit Thr(float thr) : v(__float2bfloat162_rn(thr)) {}
  };
  struct Count {
    __nv_bfloat162 n = __float2bfloat162_rn(0.f);
    __device__ void add(const uint4& q, const Thr& t) {
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) n = __hadd2(n, __hgt2(*reinterpret_cast<const __nv_bfloat162*>(&w[i]), t.v));
    }
    __device__ float total() const {
      const uint32_t b = *reinterpret_cast<const uint32_t*>(&n);
      return __uint_as_float(b << 16) + __uint_as_float(b & 0xFFFF0000u);
    }
  };
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
    __device__ float total() const { return (float)n; }
  };
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
// rest are 0).  All selectors, `sel` their index.
__device__ __forceinline__ void rank_candidates(const uint64_t* cand, int n, int k, uint64_t* best, int sel) {
  for (int i = sel; i < n; i += kSelectors) {
    const uint64_t mine = cand[i];
    int r = 0;
#pragma unroll 4
    for (int j = 0; j < n; ++j) r += cand[j] > mine;
    if (r < k) best[r] = mine;
  }
  for (int i = n + sel; i < k; i += kSelectors) best[i] = 0;
}

// A warp's n-th largest key (n <= 32).
__device__ __forceinline__ uint32_t nth_largest(uint32_t mine, int n, int lane) {
  uint32_t t = 0;
  for (int i = 0; i < n; ++i) {
    t = __reduce_max_sync(0xffffffffu, mine);
    if (__ffs(__ballot_sync(0xffffffffu, mine == t)) - 1 == lane) mine = 0;
  }
  return t;
}

// The k largest keys of vectors [v0, v1) of a row, by a pass in order against
// the k-th best so far: once k are held, equal logits (of later tokens) never
// pass, so that a step whose maximum is not greater is done with.  In a step
// the selectors' maxima bound what has to be looked at, as for a row; where
// equal values leave more than fits, its vectors are taken one by one.  All
// selectors.
template <typename T>
__device__ __noinline__ void top_again(LpShared* sh, const RowAt<T>& r, int v0, int v1, int k, int sel) {
  using V = Vec<T>;
  static_assert(kSelectors * V::kN + kLpMaxTop <= kLpCap, "a vector of each selector fits beside the best");
  float floor = -INFINITY;
  int held = 0;
  sel_sync();
  if (sel == 0) sh->n_cand = 0;
  sel_sync();
  // what has been appended joins the best
  auto join_best = [&](int n) {
    rank_candidates(sh->cand, n, k, sh->best, sel);
    sel_sync();
    held = n < k ? n : k;
    for (int i = sel; i < held; i += kSelectors) sh->cand[i] = sh->best[i];
    if (n >= k) floor = key_logit(sh->best[k - 1]);
    if (sel == 0) sh->n_cand = held;
    sel_sync();
  };
  for (int v = v0; v < v1; v += kVpt * kSelectors) {
    uint4 q[kVpt];
#pragma unroll
    for (int j = 0; j < kVpt; ++j) {
      const int at = v + j * kSelectors + sel;
      q[j] = at < v1 ? __ldg(r.vec + at) : make_uint4(V::kNegInf, V::kNegInf, V::kNegInf, V::kNegInf);
      if (at < v1 && r.edge(at)) r.edges(q[j], at);
    }
    const float mx = V::max(q);
    if (!sel_any(mx > floor)) continue;
    const uint32_t w = nth_largest(ord32(fmaxf(mx, -INFINITY) + 0.f), (k + kSelWarps - 1) / kSelWarps, sel & 31);
    if ((sel & 31) == 0) sh->step_tau[sel >> 5] = w;
    sel_sync();
    uint32_t tau = sh->step_tau[0];
    for (int i = 1; i < kSelWarps; ++i) tau = min(tau, sh->step_tau[i]);
    auto append = [&](const uint4& vec, int j) {
#pragma unroll
      for (int e = 0; e < V::kN; ++e) {
        const float x = V::at(vec, e);
        if (x > floor && ord32(x + 0.f) >= tau) {
          const int at = atomicAdd(&sh->n_cand, 1);
          if (at < kLpCap) sh->cand[at] = key_of(x, (v + j * kSelectors + sel) * V::kN + e - r.off);
        }
      }
    };
#pragma unroll
    for (int j = 0; j < kVpt; ++j) append(q[j], j);
    sel_sync();
    const int n = sh->n_cand;
    sel_sync();   // all have read it before any appends again
    if (n <= kLpCap) {
      if (n != held) join_best(n);
      continue;
    }
    if (sel == 0) sh->n_cand = held;   // (the best are still in the first places)
    sel_sync();
#pragma unroll 1
    for (int j = 0; j < kVpt; ++j) {
      uint4 mine = q[0];   // (q[j] without an index into registers)
#pragma unroll
      for (int i = 1; i < kVpt; ++i)
        if (i == j) mine = q[i];
      append(mine, j);
      sel_sync();
      const int some = sh->n_cand;
      sel_sync();
      if (some != held) join_best(some);
    }
  }
  if (held == 0)
    for (int i = sel; i < k; i += kSelectors) sh->best[i] = 0;
  sel_sync();
}

// log S and the entropy of a row whose maximum m is finite and large, or +inf
// (then the +inf tokens share the probability).  All selectors.
template <typename T>
__device__ __noinline__ float2 row_again(LpShared* sh, const RowAt<T>& r, float m, int sel) {
  using V = Vec<T>;
  float s = 0.f, u = 0.f;
#pragma unroll 4
  for (int v = sel; v < r.nv; v += kSelectors) {
    uint4 q = __ldg(r.vec + v);
    if (r.edge(v)) r.edges(q, v);
#pragma unroll
    for (int e = 0; e < V::kN; ++e) {
      const float x = V::at(q, e);
      if (m == INFINITY) {
        s += x == INFINITY ? 1.f : 0.f;
      } else {
        const float d = x - m, p = expf(d);
        if (p > 0.f) s += p, u = fmaf(p, d, u);
      }
    }
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o), u += __shfl_xor_sync(0xffffffffu, u, o);
  sel_sync();
  if ((sel & 31) == 0) sh->sum[sel >> 5][0] = s, sh->sum[sel >> 5][1] = u;
  sel_sync();
  s = u = 0.f;
  for (int w = 0; w < kSelWarps; ++w) s += sh->sum[w][0], u += sh->sum[w][1];
  const float z = logf(s);
  return make_float2(z, z - u / s);
}

}  // namespace

template <typename T>
__global__ void __launch_bounds__(kLpThreads, 2)
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
  // a warp's wait; after one that ran out the rows left go through without data
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    const bool there = *abort ? false : mbar_wait(bar, parity, abort);
    if (!__all_sync(0xffffffffu, there)) {
      *abort = 1;
      if (err && lane == 0) atomicOr(err, kErrTimeout);
    }
  };
  auto token_of = [&](int row) { return tokens && row < rows ? tokens[row] : -1; };
  auto valid = [&](int t) { return t >= 0 && t < vocab; };
  auto logit_of = [&](int row, int t) { return valid(t) ? V::load(logits + (size_t)row * stride + t) : 0.f; };
  // chunks of a group of vectors
  auto group_of = [](int chunks) { return (chunks + kGroups - 1) / kGroups; };

  if (warp == kReadWarps + kSelWarps) {
    if (lane == 0) {
      // ---------------- copies
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
  } else if (warp < kReadWarps) {
    // ---------------- readers
    int stage = 0, it = 0;
    uint32_t phase = 0;
    int token = token_of(row0);
    float xt = logit_of(row0, token);
    for (int row = row0; row < rows; row += row_step, ++it) {
      const RowAt<T> r(logits, stride, row, vocab);
      int v0, v1;
      slice_of(r, v0, v1);
      const int chunks = (v1 - v0 + kChunkVecs - 1) / kChunkVecs;
      const int per_group = group_of(chunks);
      const int next_token = token_of(row + row_step);
      const bool masked = !(xt > -INFINITY);                    // (NaN too)
      // before the given token's vector equal logits count as greater
      const int vt = valid(token) && !masked ? (token + r.off) / V::kN : -1;
      const typename V::Thr above(masked ? -INFINITY : xt), from(masked ? -INFINITY : V::below(xt));
      LpRow& hand = sh->row[it & 1];
      wait(&sh->taken[it & 1], ((uint32_t)(it >> 1) & 1u) ^ 1u);

      float c = kNone, m = -INFINITY, gm = -INFINITY, greater = 0.f;
      uint64_t s2[2] = {pair(0.f, 0.f), pair(0.f, 0.f)}, u2[2] = {pair(0.f, 0.f), pair(0.f, 0.f)};
      int group = 0, left = per_group;
      for (int ch = 0; ch < chunks; ++ch) {
        wait(&sh->full[stage], phase);
        const int vc = v0 + ch * kChunkVecs;
        const uint4* p = reinterpret_cast<const uint4*>(ring + stage * kChunkBytes) + tid;
        uint4 q[kVpt];
        if (ch > 0 && ch + 1 < chunks) {
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

        const float mx = V::max(q);
        gm = fmaxf(gm, mx);
        if (--left == 0 || ch + 1 == chunks) {
          if (top) hand.gmax[group][tid] = ord32(gm + 0.f);
          m = fmaxf(m, gm);
          gm = -INFINITY;
          ++group;
          left = per_group;
        }
        if (mx * kL > c + 16.f) {
          const float cn = rintf(mx * kL), d = fmaxf(c - cn, -1e30f), f = exp2_fast(d);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            u2[i] = fma_pair(s2[i], pair(d, d), u2[i]);
            s2[i] = fma_pair(s2[i], pair(f, f), pair(0.f, 0.f));
            u2[i] = fma_pair(u2[i], pair(f, f), pair(0.f, 0.f));
          }
          c = cn;
        }
        if (c > kNone) {
          // masked logits and NaN take a value whose exponential is 0 (-160 in base 2 at least, finite)
          const float low = (c - 160.f) * 0.6931472f;
          const typename V::Low lo(fmaf(fabsf(low), -0.01f, low));
          const uint64_t cc = pair(-c, -c);
#pragma unroll
          for (int j = 0; j < kVpt; ++j) V::sums(q[j], lo, cc, s2[j & 1], u2[j & 1]);
        }
        typename V::Count count;
        if (vt < vc || vt >= vc + kChunkVecs) {   // (the same for all)
          const typename V::Thr t = vt < vc ? above : from;
#pragma unroll
          for (int j = 0; j < kVpt; ++j) count.add(q[j], t);
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
                greater += x > xt || (x == xt && v * V::kN + e - r.off < token) ? 1.f : 0.f;
              }
            }
          }
        }
        greater += count.total();
      }
      const float next_xt = logit_of(row + row_step, next_token);

      // ---------------- the warp's part to the selectors
      const float2 ss = unpair(add_pair(s2[0], s2[1])), uu = unpair(add_pair(u2[0], u2[1]));
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
      if (lane == 0) hand.warp[warp] = a;
      if (top) {
        // this warp's ceil(k / w)-th largest thread maximum, w the warps whose
        // threads all have a vector (none, or too few threads: every token is a
        // candidate)
        const int full = min(kReadWarps, (v1 - v0) / 32);
        const int need = full ? (top + full - 1) / full : 33;
        const uint32_t t = need <= 32 ? nth_largest(ord32(m + 0.f), need, lane) : 0u;
        if (lane == 0) hand.tau[warp] = warp < full ? t : full ? 0xffffffffu : 0u;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->read[it & 1]);
      token = next_token;
      xt = next_xt;
    }
  } else {
    // ---------------- selectors
    const int sel = tid - kReaders;
    int it = 0;
    for (int row = row0; row < rows; row += row_step, ++it) {
      const RowAt<T> r(logits, stride, row, vocab);
      int v0, v1;
      slice_of(r, v0, v1);
      const int chunks = (v1 - v0 + kChunkVecs - 1) / kChunkVecs;
      const int per_group = group_of(chunks);
      const int token = token_of(row);
      const float xt = logit_of(row, token);
      if (sel == 0) sh->n_cand = 0, sh->n_hit = 0;
      sel_sync();
      wait(&sh->read[it & 1], (uint32_t)(it >> 1) & 1u);
      const LpRow& hand = sh->row[it & 1];

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
        const bool masked = !(xt > -INFINITY);
        float lp = 0.f;
        int rank = 0;
        if (valid(token)) {
          lp = masked ? -INFINITY : b.m == INFINITY ? (xt == INFINITY ? (float)-z : -INFINITY)
                                                     : (float)((double)xt - (double)b.m - z);
          rank = 1 + (int)b.greater;
        } else if (token != -1 && err) {
          atomicOr(err, kErrToken);
        }
        if (tokens) out.logprobs[row] = lp, out.ranks[row] = rank;
      };
      auto is_odd = [](float m) { return m > -INFINITY && !(fabsf(m) <= kPlain); };
      if (sel == 0) {
        LpPart b = hand.warp[0];
        for (int w = 1; w < kReadWarps; ++w) b = join(b, hand.warp[w]);
        sh->part = b;
        if (S == 1 && !is_odd(b.m)) finish(b, make_float2(0.f, 0.f), false);
      }
      __syncwarp();
      // ---------------- the slice's largest tokens
      if (top) {
        uint32_t tau = 0xffffffffu;
        for (int w = 0; w < kReadWarps; ++w) tau = min(tau, hand.tau[w]);
        tau = max(tau, kOrdNegInf + 1);
        // the groups with a token that reaches tau, then their vectors, one per
        // thread: read where they are found, a warp takes its groups' loads one
        // after another
        const int groups = chunks ? (chunks + per_group - 1) / per_group : 0;
        const uint4* gmax = reinterpret_cast<const uint4*>(hand.gmax);
        for (int i = sel; i < groups * (kReaders / 4); i += kSelectors) {
          const uint4 g = gmax[i];
          const uint32_t w[4] = {g.x, g.y, g.z, g.w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (w[e] >= tau) sh->hits[atomicAdd(&sh->n_hit, 1)] = (uint16_t)(4 * i + e);
        }
        sel_sync();
        const int hits = sh->n_hit, per_hit = per_group * kVpt;
        for (int i = sel; i < hits * per_hit; i += kSelectors) {
          const int hit = sh->hits[i / per_hit], j = i % per_hit;
          const int v = v0 + (hit / kReaders * per_hit + j) * kReaders + hit % kReaders;
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
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&sh->taken[it & 1]);   // (the parts and tau are read; the hits are this side's)
      sel_sync();
      if (top) {
        const int n = sh->n_cand;
        if (n <= kLpCap)
          rank_candidates(sh->cand, n, top, sh->best, sel);
        else
          top_again<T>(sh, r, v0, v1, top, sel);
        sel_sync();
      }

      // ---------------- the row's results, from its slices' parts
      if (S > 1) {
        cluster_sync();   // (the other warps arrive too, below)
        if (slice == 0) {
          LpPart b = sh->part;
          for (int o = 1; o < S; ++o) {
            const uint32_t at = cluster_map(smem_u32(&sh->part), (uint32_t)o);
            const float4 d = ld_dsmem_f32x4(at);
            const LpPart p{d.x, d.y, d.z, d.w, ld_dsmem_f32(at + 16)};
            b = join(b, p);
          }
          sel_sync();
          if (sel == 0) {
            sh->part = b;
            if (!is_odd(b.m)) finish(b, make_float2(0.f, 0.f), false);
          }
          if (top) {
            for (int i = sel; i < S * top; i += kSelectors)
              sh->cand[i] = ld_dsmem_u64(cluster_map(smem_u32(&sh->best[i % top]), (uint32_t)(i / top)));
            sel_sync();
            // a key's place: its own slice's keys before it, and those of the
            // other slices that are greater (each list is in order, empty
            // places hold 0)
            for (int i = sel; i < top; i += kSelectors) sh->best[i] = 0;
            sel_sync();
            for (int i = sel; i < S * top; i += kSelectors) {
              const uint64_t mine = sh->cand[i];
              if (mine == 0) continue;
              int n = i % top;
              for (int o = 0; o < S && n < top; ++o) {
                if (o == i / top) continue;
                int lo = 0, hi = top;   // the first that is not greater lies in [lo, hi]
                while (lo < hi) {
                  const int mid = (lo + hi) / 2;
                  if (sh->cand[o * top + mid] > mine) lo = mid + 1; else hi = mid;
                }
                n += lo;
              }
              if (n < top) sh->best[n] = mine;
            }
          }
          sel_sync();
        }
      }
      if (slice == 0) {
        const LpPart b = sh->part;
        if (is_odd(b.m)) {   // (the same for all)
          const float2 again = row_again<T>(sh, r, b.m, sel);
          if (sel == 0) finish(b, again, true);
          sel_sync();
        }
        for (int i = sel; i < top; i += kSelectors) {
          const uint64_t key = sh->best[i];
          const float x = key_logit(key);
          const bool any = key != 0 && (sh->m < INFINITY || x == INFINITY);
          out.top_tokens[(size_t)row * top + i] = any ? key_token(key) : -1;
          out.top_logprobs[(size_t)row * top + i] =
              !any ? -INFINITY : sh->m == INFINITY ? (float)-sh->z : (float)((double)x - (double)sh->m - sh->z);
        }
      }
      sel_sync();   // the shared results are free for the next row
    }
  }
  if (S > 1) {
    if (warp < kReadWarps || warp == kReadWarps + kSelWarps) cluster_sync();   // (the selectors' first one)
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
  cfg.blockDim = dim3(kLpThreads);
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

// ssd_logprob.cu -- log probabilities of given tokens with entropy, rank and
// the best alternatives, in one pass over the rows.
//
// With a reference m, c = log2(e) / T and x = (z - m) c,
//     S = sum 2^x,  U = sum 2^x x:
//     log p(v) = ln 2 (x_v - log2 S),   H = ln 2 (log2 S - U / S).
// A thread's m is the maximum of its first elements and moves only when an
// element's 2^x exceeds 2^16 (S and U then scale: S' = 2^d S, U' = 2^d (U + d S),
// d = (m - m') c); threads, and CTAs that share a row, are joined by the same
// rule in a fixed order.  The pass computes z c - round(m c) with one fused
// multiply-add an element and takes the rounding error of m c out of S and U
// afterwards (the same rule again); rows whose m c is beyond 2^24 or whose T is
// below 1e-7 or above 7e22 are summed by a plain second loop.  The rank is a count of the
// elements that come before the token's logit, known before the pass.
//
// Best alternatives: the K-th largest of the warps' first maxima bounds the K-th
// largest of all from below; elements that reach the bound go to a list in
// shared memory, a part of it for each warp, and the bound rises after 4, 16,
// ... rounds to about the K-th largest of the lists (found by counting at three
// values at a time), which drops the others.  The pass compares one maximum of
// a thread and round with it.  A row with more such elements than the lists hold
// (hundreds of equal logits, or of -inf) is searched K times instead.
//
// A warp copies its slices of the row into a ring of its own (bulk copies, two
// rounds of 2 KB ahead: 96 KB in flight on an SM; with three the fp32
// pass of K = 0 falls from 6.6 to 5.0 TB/s).  One CTA per row, or per part of a row,
// whose last CTA to finish joins the parts.
//
// Bound: HBM for fp32 (4096 x 151936, K = 8: 386 us, 6.5 TB/s; 2048 rows, K = 0:
// 189 us, 6.6 TB/s); 384 rows of bf16 are one wave, which begins and ends together
// (384 x 151936: K = 0 26 us, 4.5 TB/s) and whose candidates' steps, two raised
// bounds and the selection leave the memory idle (K = 20 43 us); a few rows, and
// short ones, are steps one after another (8 x 128256 bf16: K = 0 6.5 us, K = 5 9.5
// us; 4096 x 4096 bf16: K = 0 43 us, K = 8 67 us, of 5 us of bytes).
#include <math.h>

#include <algorithm>

#include "ssd_async.cuh"
#include "ssd_device.cuh"
#include "ssd_kv.cuh"

namespace ssd {
namespace {

constexpr int kLpThreads = 256;
// CTAs of an SM.  Four (64 registers a thread) hide more of the candidates'
// steps where fp32 rows ask for the best (1000 x 128256, K = 8: 99 us, three: 108;
// 4096 x 151936: 386, three: 405); elsewhere long rows are faster with three (bf16,
// 384 x 151936, K = 20: 43 us, four: 46; fp32, 2048 x 151936, K = 0: 189, four: 212),
// short ones with four (bf16, 4096 x 4096, K = 0: 43, four: 36; K = 8: 67, four: 60).
template <class Tag, bool TOP>
constexpr int kLpCtas = TOP && Tag::kVec == 4 ? 4 : 3;
constexpr int kFlight = 4;        // vectors of a thread and round
constexpr int kStages = 2;        // rounds on their way into shared memory
constexpr int kSlice = 32 * kFlight;  // a warp's vectors of a round
constexpr int kLpWarps = kLpThreads / 32;
constexpr int kList = 896;        // elements of the list, a part of it for each warp (one counter
                                  // for all of them, with its atomics, cost more than the pass)
constexpr int kOwn = kList / kLpWarps;
constexpr int kMaxSplit = 31;     // parts of a row (of whose lists each thread takes kHold keys)
constexpr int kCounters = 1024;   // most rows that are split
constexpr int kHold = 4;          // most keys of a thread where the best are selected
constexpr int kFirst = 5;         // most of each warp's maxima of the first round
constexpr int kRaise = 4;         // rounds before the bound first rises, and the factor to the next time
constexpr int kLpTop = 32;        // SSD_MAX_TOP
constexpr float kStep = 16.f;     // excess of an element over m that moves it
constexpr float kLowest = -3.0e38f;
constexpr float kLeast = 2e-23f;   // least c of the pass: below it -1e30 c, its floor, is not far below m c
constexpr float kMost = 3.402823466e38f;  // c where log2(e) / T is more
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLog2e = 1.4426950408889634f;

using Part = LogprobPart;

struct LpSmem {
  uint4 ring[kLpWarps][kStages][kSlice];  // each warp's own
  uint64_t bar[kLpWarps][kStages];
  alignas(16) unsigned long long key[kList];  // candidates: order of the value, then of the index
  unsigned long long best[kLpTop];
  float m[kLpWarps], S[kLpWarps], U[kLpWarps];
  int count[kLpWarps];
  alignas(16) float top[kLpWarps * kFirst];
  uint4 range[kLpWarps];
  alignas(16) uint32_t above[2][kLpWarps];
  unsigned long long wkey[kLpWarps];
  int n[kLpWarps], last;
  float tau;
  alignas(8) volatile uint8_t lost[kLpWarps];  // a copy of this warp did not come
  volatile int gone;                           // of some warp: the others need not wait as long
};

// Values as numbers above 0 of the same order, and back; -0 counts as 0.
__device__ __forceinline__ uint32_t order_of(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float order_value(uint32_t u) {
  return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u);
}
// A (value, index) pair as one number that orders by value, then by lower
// index.
__device__ __forceinline__ unsigned long long key_of(float v, int i) {
  return (static_cast<unsigned long long>(order_of(v)) << 32) | (0x7fffffffu - static_cast<uint32_t>(i));
}
__device__ __forceinline__ float key_value(unsigned long long k) {
  return order_value(static_cast<uint32_t>(k >> 32));
}
__device__ __forceinline__ int key_index(unsigned long long k) {
  return static_cast<int>(0x7fffffffu - static_cast<uint32_t>(k));
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ float min3(float a, float b, float c) {
  float r;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t max_nan_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// The largest value below v (v finite): v > below(w) where v >= w.
__device__ __forceinline__ uint32_t below_bits(uint32_t b, uint32_t sign) {
  return (b & ~sign) == 0 ? sign | 1 : b & sign ? b + 1 : b - 1;
}

// Vector v of a row of V elements as it lies in memory, -inf behind the row's
// end (`whole`: the row is 16-byte aligned), and what the pass asks of it.
template <class Tag>
struct Raw;
template <>
struct Raw<F32Tag> {
  float4 r;
  struct Count {
    int n = 0;
    __device__ __forceinline__ int take() {
      const int k = n;
      n = 0;
      return k;
    }
  };
  typedef float Bound;
  __device__ __forceinline__ static Bound bound(float z) { return z; }
  __device__ __forceinline__ static Bound below(float z) {
    return __uint_as_float(below_bits(__float_as_uint(z), 0x80000000u));
  }
  __device__ __forceinline__ void load(const float* z, int v, int V, bool whole) {
    const int i = v * 4;
    if (whole && i + 4 <= V) {
      r = F32Tag::loadraw(z + i);
    } else {
      float x[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) x[k] = i + k < V ? F32Tag::load1(z + i + k) : -INFINITY;
      r = make_float4(x[0], x[1], x[2], x[3]);
    }
  }
  __device__ __forceinline__ void raw(const uint4& w) {
    r = make_float4(__uint_as_float(w.x), __uint_as_float(w.y), __uint_as_float(w.z), __uint_as_float(w.w));
  }
  __device__ __forceinline__ void none() { r = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY); }
  __device__ __forceinline__ float top() const { return max3(fmaxf(r.x, r.y), r.z, r.w); }
  // largest of a round's elements
  __device__ __forceinline__ static float top(const Raw (&w)[kFlight]) {
    float t = w[0].top();
#pragma unroll
    for (int u = 1; u < kFlight; ++u) t = max3(max3(t, w[u].r.x, w[u].r.y), w[u].r.z, w[u].r.w);
    return t;
  }
  // The logits with a floor of -1e30 under them (c is at most 1.5e7, and where
  // a logit is -inf 2^x x has to be 0), checked a round at a time.
  __device__ __forceinline__ static void floor(Raw (&w)[kFlight]) {
    float t = INFINITY;
#pragma unroll
    for (int u = 0; u < kFlight; ++u) t = min3(min3(t, w[u].r.x, w[u].r.y), w[u].r.z, w[u].r.w);
    if (t < -1e30f) {
#pragma unroll
      for (int u = 0; u < kFlight; ++u)
        w[u].r = make_float4(max_nan(w[u].r.x, -1e30f), max_nan(w[u].r.y, -1e30f), max_nan(w[u].r.z, -1e30f),
                             max_nan(w[u].r.w, -1e30f));
    }
  }
  // z c - mc
  __device__ __forceinline__ void scaled(f32x2 c, f32x2 m, f32x2 (&x)[4]) const {
    x[0] = fma2(pk2(r.x, r.y), c, m);
    x[1] = fma2(pk2(r.z, r.w), c, m);
  }
  __device__ __forceinline__ void count(Bound t, Count& n) const {
    n.n += (r.x > t) + (r.y > t) + (r.z > t) + (r.w > t);
  }
};
template <>
struct Raw<BF16Tag> {
  uint4 r;
  struct Count {  // of whole numbers in bf16, exact to 256
    __nv_bfloat162 n = __floats2bfloat162_rn(0.f, 0.f);
    __device__ __forceinline__ int take() {
      const int k = static_cast<int>(__low2float(n) + __high2float(n));
      n = __floats2bfloat162_rn(0.f, 0.f);
      return k;
    }
  };
  typedef __nv_bfloat162 Bound;
  __device__ __forceinline__ static Bound two(uint32_t bits) {
    const uint32_t w = bits | (bits << 16);
    return *reinterpret_cast<const __nv_bfloat162*>(&w);
  }
  __device__ __forceinline__ static Bound bound(float z) { return two(__float_as_uint(z) >> 16); }
  __device__ __forceinline__ static Bound below(float z) {
    return two(below_bits(__float_as_uint(z) >> 16, 0x8000u) & 0xffffu);
  }
  __device__ __forceinline__ void load(const uint16_t* z, int v, int V, bool whole) {
    const int i = v * 8;
    if (whole && i + 8 <= V) {
      r = BF16Tag::loadraw(z + i);
    } else {
      uint32_t w[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t lo = i + 2 * k < V ? z[i + 2 * k] : 0xff80u, hi = i + 2 * k + 1 < V ? z[i + 2 * k + 1] : 0xff80u;
        w[k] = lo | (hi << 16);
      }
      r = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  __device__ __forceinline__ void raw(const uint4& w) { r = w; }
  __device__ __forceinline__ void none() { r = make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u); }
  __device__ __forceinline__ float top() const {
    const uint32_t w = max_bf16x2(max_bf16x2(r.x, r.y), max_bf16x2(r.z, r.w));
    return fmaxf(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
  }
  __device__ __forceinline__ static float top(const Raw (&w)[kFlight]) {
    uint32_t t = max_bf16x2(max_bf16x2(w[0].r.x, w[0].r.y), max_bf16x2(w[0].r.z, w[0].r.w));
#pragma unroll
    for (int u = 1; u < kFlight; ++u)
      t = max_bf16x2(max_bf16x2(t, max_bf16x2(w[u].r.x, w[u].r.y)), max_bf16x2(w[u].r.z, w[u].r.w));
    return fmaxf(__uint_as_float(t << 16), __uint_as_float(t & 0xffff0000u));
  }
  __device__ __forceinline__ static void floor(Raw (&w)[kFlight]) {
#pragma unroll
    for (int u = 0; u < kFlight; ++u)
      w[u].r = make_uint4(max_nan_bf16x2(w[u].r.x, 0xf149f149u), max_nan_bf16x2(w[u].r.y, 0xf149f149u),
                          max_nan_bf16x2(w[u].r.z, 0xf149f149u), max_nan_bf16x2(w[u].r.w, 0xf149f149u));
  }
  __device__ __forceinline__ void scaled(f32x2 c, f32x2 m, f32x2 (&x)[4]) const {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int k = 0; k < 4; ++k)
      x[k] = fma2(pk2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xffff0000u)), c, m);
  }
  __device__ __forceinline__ void count(Bound t, Count& n) const {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int k = 0; k < 4; ++k)
      n.n = __hadd2(n.n, __hgt2(*reinterpret_cast<const __nv_bfloat162*>(&w[k]), t));
  }
};

// (z - m) c, also where z - m or c exceeds 32 bits.
__device__ __noinline__ float far_scaled(float z, float m, float c, float T) {
  const float d = z - m;
  return d > -INFINITY ? d / T * kLog2e : 2.f * ((0.5f * z - 0.5f * m) * c);
}
__device__ __forceinline__ float scaled(float z, float m, float c, float T) {
  const float d = z - m;
  return d > -INFINITY && c < kMost ? d * c : far_scaled(z, m, c, T);
}

// What two lanes or parts hold, joined over the warp in a fixed order: m first,
// then sums of scaled S and U.  FAR: where m may differ by more than 32 bits hold
// and c be so small that this counts (the lanes of a CTA share m then).
template <bool FAR = false>
__device__ __forceinline__ void join_warp(float c, float T, float& m, float& S, float& U) {
  float M = m;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
  const float d0 = fmaxf(FAR ? scaled(m, M, c, T) : (m - M) * c, -1e4f), f = exp2f(d0);  // 2^-1e4 = 0
  U = f * fmaf(S, d0, U);
  S *= f;
  m = M;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    S += __shfl_xor_sync(0xffffffffu, S, d);
    U += __shfl_xor_sync(0xffffffffu, U, d);
  }
}

// Maximum m, S and U of a part of a row by two plain loops, for every thread of
// the CTA: rows whose m c is too large to be rounded once for all elements,
// temperatures below 1e-7 or above 7e22, and rows that never moved a reference
// (all logits at or below kLowest; m = -inf and S = 0 where none is finite).
template <class Tag>
__device__ __noinline__ void sum_plain(LpSmem& sm, const typename Tag::Elem* z, int i0, int i1, float c, float T,
                                       float& m, float& S, float& U) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  float top = -INFINITY;
  for (int i = i0 + tid; i < i1; i += kLpThreads) top = fmaxf(top, Tag::load1(z + i));
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
  __syncthreads();
  if (lane == 0) sm.m[warp] = top;
  __syncthreads();
  m = -INFINITY;
  for (int w = 0; w < kLpWarps; ++w) m = fmaxf(m, sm.m[w]);
  S = 0.f;
  U = 0.f;
  for (int i = i0 + tid; i < i1; i += kLpThreads) {
    const float v = Tag::load1(z + i);
    if (v == -INFINITY) continue;  // (c = 0 at an infinite T)
    const float x = max_nan(scaled(v, m, c, T), -1000.f), e = exp2f(x);
    S += e;
    U = fmaf(e, x, U);
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    S += __shfl_xor_sync(0xffffffffu, S, d);
    U += __shfl_xor_sync(0xffffffffu, U, d);
  }
  if (lane == 0) {
    sm.S[warp] = S;
    sm.U[warp] = U;
  }
  __syncthreads();
  S = U = 0.f;
  for (int w = 0; w < kLpWarps; ++w) {
    S += sm.S[w];
    U += sm.U[w];
  }
  __syncthreads();
}

// Log probability of a logit z under a reference m and ls = log2 S: in units of
// log 2, or in nats, with the difference halved, where 32 bits do not hold those
// or their factor.  S is off by a few units of its last place, which may leave a
// probability just above 1, as an entropy just below 0: both are cut to the bound.
// (S and U moved to the row's maximum before the answer instead: 391 us for 386,
// 4096 x 151936 fp32, and errors as before, 5e-8 of a log probability and 3.5e-7 of
// an entropy, whose terms are summed around a reference up to 16 lower.)
__device__ __noinline__ float far_log_prob(float z, float m, float T, float ls) {
  if (z == -INFINITY) return z;
  return (z - m > -INFINITY ? (z - m) / T : 2.f * ((0.5f * z - 0.5f * m) / T)) - ls * kLn2;
}
__device__ __forceinline__ float log_prob(float z, float m, float c, float T, float ls) {
  const float x = (z - m) * c;
  return x > -1e30f && c < kMost ? fminf((x - ls) * kLn2, 0.f) : far_log_prob(z, m, T, ls);
}

// A bound on the K-th largest of the CTA's orders (a thread's v, 0: none) from
// below that most of them reach at most, or the K-th largest itself; 1 where
// there are fewer than K.  Counts at three places of the range that is left, in
// 10 bits each, until it is found.  Every thread of the CTA calls it.
__device__ __noinline__ uint32_t bound_of(LpSmem& sm, uint32_t v0, uint32_t v1, uint32_t v2, uint32_t v3, int K,
                                          int most) {
  const uint32_t v[kHold] = {v0, v1, v2, v3};
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint32_t hi = 0, lo = ~0u, n = 0;
#pragma unroll
  for (int k = 0; k < kHold; ++k) {
    hi = max(hi, v[k]);
    lo = min(lo, v[k] - 1);  // (0 is the largest of these)
    n += v[k] != 0;
  }
  hi = __reduce_max_sync(0xffffffffu, hi);
  lo = __reduce_min_sync(0xffffffffu, lo);
  n = __reduce_add_sync(0xffffffffu, n);
  if (lane == 0) sm.range[warp] = make_uint4(hi, lo, n, 0);
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kLpWarps; ++w) {
    const uint4 q = sm.range[w];
    hi = max(hi, q.x);
    lo = min(lo, q.y);
    n = w == 0 ? q.z : n + q.z;
  }
  ++lo;
  ++hi;
  if (n <= static_cast<uint32_t>(most)) __syncthreads();  // (before the next call)
  if (n < static_cast<uint32_t>(K)) return 1;
  // n >= K reach lo, fewer reach hi
#pragma unroll 1
  for (int turn = 0; n > static_cast<uint32_t>(most) && hi - lo > 1; turn ^= 1) {
    const uint32_t q = max(1u, (hi - lo) >> 2);
    uint32_t c = 0;
#pragma unroll
    for (int k = 0; k < kHold; ++k)
      c += (v[k] >= lo + q) + (v[k] >= lo + 2 * q) * (1u << 10) + (v[k] >= lo + 3 * q) * (1u << 20);
    c = __reduce_add_sync(0xffffffffu, c);
    if (lane == 0) sm.above[turn][warp] = c;
    __syncthreads();
    c = 0;
#pragma unroll
    for (int w = 0; w < kLpWarps; w += 4) {
      const uint4 a = *reinterpret_cast<const uint4*>(&sm.above[turn][w]);
      c += a.x + a.y + a.z + a.w;
    }
    uint32_t at = 0;  // the highest place that K reach
#pragma unroll
    for (int k = 0; k < 3; ++k) {
      const uint32_t a = (c >> (10 * k)) & 1023u;
      if (a >= static_cast<uint32_t>(K)) {
        at = k + 1;
        n = a;
      }
    }
    if (at < 3) hi = lo + (at + 1) * q;
    lo += at * q;
  }
  if (n > static_cast<uint32_t>(most)) __syncthreads();  // (n is the same for all: every path has one)
  return lo;
}

// The K first of the CTA's different keys (a thread's, 0: none), in order, into
// best, which holds zeros: those that reach a bound, moved to `found`, each
// ranked by four threads.  `part`: in any order, with others where they fit.
__device__ __noinline__ void select_best(LpSmem& sm, unsigned long long k0, unsigned long long k1,
                                         unsigned long long k2, unsigned long long k3, int K,
                                         unsigned long long* found, bool part) {
  const unsigned long long key[kHold] = {k0, k1, k2, k3};
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t least =
      bound_of(sm, static_cast<uint32_t>(k0 >> 32), static_cast<uint32_t>(k1 >> 32), static_cast<uint32_t>(k2 >> 32),
               static_cast<uint32_t>(k3 >> 32), K, part ? kLpTop : kLpThreads / 4);
  unsigned in[kHold];
  int n = 0;
#pragma unroll
  for (int k = 0; k < kHold; ++k) {
    in[k] = __ballot_sync(0xffffffffu, static_cast<uint32_t>(key[k] >> 32) >= least);
    n += __popc(in[k]);
  }
  if (lane == 0) sm.n[warp] = n;
  __syncthreads();
  int at = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kLpWarps; ++w) {
    const int m = sm.n[w];
    at += w < warp ? m : 0;
    all += m;
  }
#pragma unroll
  for (int k = 0; k < kHold; ++k) {
    if ((in[k] >> lane) & 1) found[at + __popc(in[k] & ((1u << lane) - 1))] = key[k];
    at += __popc(in[k]);
  }
  __syncthreads();
  if (part && all <= kLpTop) {
    if (tid < all) sm.best[tid] = found[tid];
    return;
  }
#pragma unroll 1
  for (int b = 0; b < all; b += kLpThreads / 4) {
    const int j = b + (tid >> 2);
    const unsigned long long mine = j < all ? found[j] : 0;
    int rank = 0;
#pragma unroll 4
    for (int k = tid & 3; k < all; k += 4) rank += found[k] > mine;
    rank += __shfl_xor_sync(0xffffffffu, rank, 1);
    rank += __shfl_xor_sync(0xffffffffu, rank, 2);
    if ((tid & 3) == 0 && mine && rank < K) sm.best[rank] = mine;
  }
}

// ---------------------------------------------------------------------------
// Bulk copies of a warp's slices into its ring, one mbarrier a stage.
// ---------------------------------------------------------------------------
__device__ __forceinline__ void lp_copy(uint4* dst, const void* src, int bytes, uint64_t* bar, int withheld) {
  bar_expect(bar, bytes + withheld);
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   sptr(dst)),
               "l"(src), "r"(bytes), "r"(sptr(bar))
               : "memory");
}
// Bounded wait: after `us` microseconds (or once another wait of the CTA gave up)
// the row counts as lost, and the CTA runs on to its end.
__device__ __forceinline__ bool lp_wait(uint64_t* bar, uint32_t parity, unsigned us, LpSmem& sm, int* err) {
  unsigned long long t0 = 0;
  for (unsigned i = 1;; ++i) {
    if (bar_try(bar, parity)) return true;
    const bool other = sm.gone;
    if (other || (i & 31) == 0) {  // the global timer is slow to read
      const unsigned long long t = now_ns();
      if (t0 == 0) t0 = t;
      if (other || t - t0 > us * 1000ull) {
        sm.lost[threadIdx.x >> 5] = 1;
        sm.gone = 1;
        atomicOr(err, kErrTimeout);
        return false;
      }
    }
  }
}

// The K first elements of a part of a row, one search each (rows whose
// candidates do not fit the list).
template <class Tag>
__device__ __noinline__ void search_best(LpSmem& sm, const typename Tag::Elem* z, int i0, int i1, int K) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  __syncthreads();
  if (tid < kLpTop) sm.best[tid] = 0;
  unsigned long long last = ~0ull;
#pragma unroll 1
  for (int k = 0; k < K; ++k) {
    unsigned long long mine = 0;
#pragma unroll 4
    for (int j = i0 + tid; j < i1; j += kLpThreads) {
      const unsigned long long x = key_of(Tag::load1(z + j), j);
      if (x < last && x > mine) mine = x;
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      const unsigned long long o = __shfl_xor_sync(0xffffffffu, mine, d);
      if (o > mine) mine = o;
    }
    __syncthreads();
    if (lane == 0) sm.wkey[warp] = mine;
    __syncthreads();
    last = sm.wkey[0];
    for (int w = 1; w < kLpWarps; ++w)
      if (sm.wkey[w] > last) last = sm.wkey[w];
    if (tid == 0) sm.best[k] = last;
  }
}

template <class Tag, bool TOP>
__global__ void __launch_bounds__(kLpThreads, kLpCtas<Tag, TOP>) logprob_kernel(const __grid_constant__ LogprobParams p) {
  constexpr int N = Tag::kVec;
  constexpr int U = kFlight;
  extern __shared__ __align__(16) char lp_raw[];
  LpSmem& sm = *reinterpret_cast<LpSmem*>(lp_raw);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int r = blockIdx.x / p.split, part = blockIdx.x % p.split;
  const int row = p.rows ? p.rows[r] : r;
  const int tok = p.tok[r];
  const float T = p.T ? p.T[r] : 1.f;
  int bits = 0;
  bool fail = row < 0 || row >= p.n_rows || !(T >= 0.f);
  if (row >= p.n_rows) bits |= kErrBadLength;
  if (!(T >= 0.f)) bits |= kErrBadTemperature;
  const bool tok_ok = tok >= 0 && tok < p.V;
  if (!tok_ok && tok != -1) bits |= kErrBadToken;
  const int K = TOP ? p.K : 0;
  const float c = T > 0.f ? fminf(kLog2e / T, kMost) : kLog2e;
  const typename Tag::Elem* z =
      static_cast<const typename Tag::Elem*>(p.logits) + static_cast<long long>(fail ? 0 : row) * p.row_stride;
  const int nv = (p.V + N - 1) / N;  // vectors of a row
  const int per = (nv + p.split - 1) / p.split;
  const int v0 = min(nv, part * per), v1 = min(nv, v0 + per);
  float m = kLowest, S = 0.f, E = 0.f, zt = INFINITY;
  f32x2 S2 = pk2(0.f, 0.f), E2 = S2;  // of even and odd elements
  int count = 0;
  bool gone = false;  // a copy did not come: no answer
  if (TOP && tid < kLpTop) sm.best[tid] = 0;
  if (!fail) {
    if (tok_ok) zt = Tag::load1(z + tok);
    const typename Raw<Tag>::Bound after = Raw<Tag>::bound(zt),
                                   ahead = zt > -INFINITY && zt < INFINITY ? Raw<Tag>::below(zt) : after;
    float tau = -INFINITY, mc = 0.f;
    bool plain = !(c > kLeast && c < 1e7f);
    bool over = false;  // more than its list holds
    // a thread's keys of the list
    auto keys = [&](unsigned long long (&key)[kHold]) {
      static_assert(kOwn <= 32 * kHold, "a warp's list");
      __syncwarp();
      const int own = sm.n[warp];
      over |= own > kOwn;
#pragma unroll
      for (int k = 0; k < kHold; ++k)
        key[k] = lane + 32 * k < min(own, kOwn) ? sm.key[warp * kOwn + lane + 32 * k] : 0;
    };
    const f32x2 c2 = pk2(c, c);
    // S and U for a reference that lies d (in units of x) lower
    auto shift = [&](float d) {
      const float f = exp2f(d);
      const f32x2 f2 = pk2(f, f);
      E2 = mul2(f2, fma2(S2, pk2(d, d), E2));
      S2 = mul2(f2, S2);
    };
    // the rounding error of m c out of the sums
    auto exact = [&]() {
      if (m != kLowest) shift(-fmaf(m, c, -mc));
    };
    int round = 0, raise_at = kRaise;
    Raw<Tag> now[U];
    // aligned rows come by bulk copies, a warp's slices on its own ring
    // (a lane for which a copy did not come waits for none and starts none any more:
    // its barrier's phase is still open)
    int vfull = p.whole ? min(v1, p.V / N) : v0;
    uint64_t* bar = sm.bar[warp];
    auto slice = [&](int k) { return v0 + k * (kLpThreads * U) + warp * kSlice; };
    int stage = 0;
    uint32_t phase = 0;
    auto fetch = [&](int k, int stage) {
      const int v = slice(k), n = min(kSlice, vfull - v);
      if (n > 0 && lane == 0)
        lp_copy(sm.ring[warp][stage], z + static_cast<long long>(v) * N, n * 16, bar + stage, p.withheld);
    };
    if (lane == 0) {
      sm.n[warp] = 0;
      sm.lost[warp] = 0;
      sm.gone = 0;  // (by each warp before it looks there)
#pragma unroll
      for (int k = 0; k < kStages; ++k) bar_init(bar + k, 1);
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncwarp();
#pragma unroll
    for (int k = 0; k < kStages; ++k) fetch(k, k);
#pragma unroll 1
    for (int b = v0; b < v1; b += kLpThreads * U, ++round) {
      const int first = slice(round), n = min(kSlice, vfull - first);
      if (n > 0 && !lp_wait(bar + stage, phase, p.wait_us, sm, p.err)) vfull = v0;
      const uint4* ring = sm.ring[warp][stage] + lane;
      if (n >= kSlice) {
#pragma unroll
        for (int u = 0; u < U; ++u) now[u].raw(ring[u * 32]);
      } else {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int k = u * 32 + lane;
          if (k < n) now[u].raw(ring[u * 32]);
          else if (first + k < v1) now[u].load(z, first + k, p.V, p.whole);
          else now[u].none();
        }
      }
      __syncwarp();
      fetch(round + kStages, stage);
      if (++stage == kStages) {
        stage = 0;
        phase ^= 1;
      }
      const float top = Raw<Tag>::top(now);
      if (TOP && round == 0) {
        // of every warp the largest of its threads' maxima: the K-th largest
        // of those different elements is the first bound
        uint32_t v = order_of(top);
        const int take = (K + kLpWarps - 1) / kLpWarps + 1;
        static_assert((kLpTop + kLpWarps - 1) / kLpWarps + 1 <= kFirst, "the warps' maxima");
#pragma unroll 1
        for (int k = 0; k < take; ++k) {
          const uint32_t w = __reduce_max_sync(0xffffffffu, v);
          if (lane == 0) sm.top[warp * take + k] = order_value(w);
          const unsigned who = __ballot_sync(0xffffffffu, v == w);
          if (lane == __ffs(who) - 1) v = 0;
        }
        __syncthreads();
        if (tid < kLpWarps * take) {
          const float mine = sm.top[tid];
          int rank = 0;
#pragma unroll 4
          for (int k = 0; k < kLpWarps * take; k += 4) {
            const float4 o = *reinterpret_cast<const float4*>(&sm.top[k]);
            rank += (o.x > mine || (o.x == mine && k < tid)) + (o.y > mine || (o.y == mine && k + 1 < tid)) +
                    (o.z > mine || (o.z == mine && k + 2 < tid)) + (o.w > mine || (o.w == mine && k + 3 < tid));
          }
          if (rank == K - 1) sm.tau = mine;
        }
        __syncthreads();
        tau = sm.tau;
      }
      // the rank, where an element may come before the token's: a slice before
      // its logit, behind it, its own
      if (top >= zt) {
        const int i0 = first * N, i1 = i0 + kSlice * N;
        if (i1 <= tok || i0 > tok) {
          const typename Raw<Tag>::Bound t = i0 > tok ? after : ahead;
          typename Raw<Tag>::Count cnt;
#pragma unroll
          for (int u = 0; u < U; ++u) now[u].count(t, cnt);
          count += cnt.take();
        } else {
#pragma unroll
          for (int u = 0; u < U; ++u) {
            float y[8];
            Tag::unpackraw(now[u].r, y);
            const int i = (first + u * 32 + lane) * N;
#pragma unroll
            for (int k = 0; k < N; ++k) count += y[k] > zt || (y[k] == zt && zt > -INFINITY && i + k < tok);
          }
        }
      }
      if (TOP && top >= tau) {
        // candidates, a vector and an element at a time
        uint32_t vectors = 0;
#pragma unroll
        for (int u = 0; u < U; ++u) vectors |= now[u].top() >= tau ? 1u << u : 0u;
#pragma unroll 1
        for (; vectors; vectors &= vectors - 1) {
          const int u = __ffs(vectors) - 1;
          Raw<Tag> w = now[0];
#pragma unroll
          for (int k = 1; k < U; ++k)
            if (u == k) w = now[k];
          float y[8];
          Tag::unpackraw(w.r, y);
          uint32_t hits = 0;
#pragma unroll
          for (int k = 0; k < N; ++k) hits |= y[k] >= tau ? 1u << k : 0u;
#pragma unroll 1
          for (; hits; hits &= hits - 1) {
            const int k = __ffs(hits) - 1, i = (first + u * 32 + lane) * N + k;
            float v = y[0];
#pragma unroll
            for (int j = 1; j < N; ++j)
              if (k == j) v = y[j];
            if (i >= p.V) break;
            const int at = atomicAdd(&sm.n[warp], 1);
            if (at < kOwn) sm.key[warp * kOwn + at] = key_of(v, i);
          }
        }
      }
      // the reference
      if ((top - m) * c > kStep) {  // (the first round's from kLowest, S = 0)
        exact();
        shift(fmaxf((m - top) * c, -1e4f));
        m = top;
        mc = m * c;
        plain |= !(fabsf(mc) < 16777216.f);
      }
      Raw<Tag>::floor(now);
      const f32x2 m2 = pk2(-mc, -mc);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        f32x2 x[4];
        now[u].scaled(c2, m2, x);
#pragma unroll
        for (int k = 0; k < N / 2; ++k) {
          float a, d;
          up2(x[k], a, d);
          const f32x2 e = pk2(ex2_fast(a), ex2_fast(d));
          S2 = add2(S2, e);
          E2 = fma2(e, x[k], E2);
        }
      }
      if (TOP) {
        if (round + 1 == raise_at && b + kLpThreads * U < v1) {
          raise_at *= kRaise;
          // a bound from the candidates, of which those below it go
          unsigned long long key[kHold];
          keys(key);
          const uint32_t least = bound_of(
              sm, static_cast<uint32_t>(key[0] >> 32), static_cast<uint32_t>(key[1] >> 32),
              static_cast<uint32_t>(key[2] >> 32), static_cast<uint32_t>(key[3] >> 32), K, K + K / 4);
          tau = fmaxf(tau, order_value(least));
          int own = 0;
#pragma unroll
          for (int k = 0; k < kHold; ++k) {
            const bool in = static_cast<uint32_t>(key[k] >> 32) >= least;
            const unsigned who = __ballot_sync(0xffffffffu, in);
            if (in) sm.key[warp * kOwn + own + __popc(who & ((1u << lane) - 1))] = key[k];
            own += __popc(who);
          }
          if (lane == 0) sm.n[warp] = own;
          __syncwarp();
        }
      }
    }
    exact();
    {
      float a, d;
      up2(S2, a, d);
      S = a + d;
      up2(E2, a, d);
      E = a + d;
    }
    // a masked token: the masked ones before it
    if (tok_ok && zt == -INFINITY)
      for (int i = v0 * N + tid; i < min(tok, v1 * N); i += kLpThreads) count += Tag::load1(z + i) == -INFINITY;
    const bool again = __syncthreads_or(plain);
    gone = *reinterpret_cast<const volatile unsigned long long*>(sm.lost) != 0;
    if (gone)  // copies land before the shared memory is used for something else
      for (int k = 0; k < 200; ++k) __nanosleep(100000);
    if (again) {
      sum_plain<Tag>(sm, z, v0 * N, min(p.V, v1 * N), c, T, m, S, E);
      if (tid > 0) S = E = 0.f;
    }
    // lanes of a warp, warps of the CTA
    join_warp(c, T, m, S, E);
    count = __reduce_add_sync(0xffffffffu, count);
    if (lane == 0) {
      sm.m[warp] = m;
      sm.S[warp] = S;
      sm.U[warp] = E;
      sm.count[warp] = count;
    }
    bool full = false;
    if (TOP) {
      unsigned long long key[kHold];
      keys(key);
      full = __syncthreads_or(over);
      select_best(sm, key[0], key[1], key[2], key[3], K, reinterpret_cast<unsigned long long*>(sm.ring),
                  p.split > 1);
      if (full) search_best<Tag>(sm, z, v0 * N, min(p.V, v1 * N), K);
    } else {
      __syncthreads();
    }
    // (by every warp: shuffles where only some warps run cost 250 clocks each)
    const bool in = lane < kLpWarps;
    m = sm.m[lane % kLpWarps];
    S = in ? sm.S[lane] : 0.f;
    E = in ? sm.U[lane] : 0.f;
    join_warp(c, T, m, S, E);
    count = __reduce_add_sync(0xffffffffu, in ? sm.count[lane] : 0);
    __syncthreads();
  }
  bool last = true;
  if (p.split > 1) {
    Part* parts = p.parts + static_cast<long long>(r) * p.split;
    unsigned long long* tk = p.part_key + static_cast<long long>(r) * p.split * kLpTop;
    if (!fail) {
      if (TOP && tid < kLpTop) {
        tk[part * kLpTop + tid] = sm.best[tid];
      }
      if (tid == 0) {
        Part q;
        q.m = m; q.S = S; q.U = E; q.count = gone ? -1 : count;
        parts[part] = q;
      }
    }
    __threadfence();
    __syncthreads();
    if (tid == 0) {
      const int n = atomicAdd(p.counter + r, 1);
      sm.last = n == p.split - 1;
      if (sm.last) p.counter[r] = 0;  // for the next call
    }
    __syncthreads();
    last = sm.last;
    if (!last) return;
    __threadfence();
    if (!fail) {
      const bool in = lane < p.split;  // lane k holds part k
      m = __ldcg(&parts[in ? lane : 0].m);
      S = in ? __ldcg(&parts[lane].S) : 0.f;
      E = in ? __ldcg(&parts[lane].U) : 0.f;
      join_warp<true>(c, T, m, S, E);
      count = in ? __ldcg(&parts[lane].count) : 0;
      gone = __any_sync(0xffffffffu, count < 0);
      count = __reduce_add_sync(0xffffffffu, count);
      if constexpr (TOP) {
        const int n = p.split * kLpTop;
        if (tid < kLpTop) sm.best[tid] = 0;
        unsigned long long key[kHold];
        static_assert(kMaxSplit * kLpTop <= kHold * kLpThreads && sizeof(sm.ring) >= sizeof(key) * kLpThreads,
                      "the parts' lists");
#pragma unroll
        for (int k = 0; k < kHold; ++k) {
          const int j = tid + kLpThreads * k;
          key[k] = j < n ? __ldcg(tk + j) : 0ull;
        }
        select_best(sm, key[0], key[1], key[2], key[3], K, reinterpret_cast<unsigned long long*>(sm.ring), false);
        __syncthreads();
      }
    }
  }
  fail |= gone;
  if (!fail && S == 0.f) sum_plain<Tag>(sm, z, 0, p.V, c, T, m, S, E);  // (no logit above kLowest)
  // the answer
  if (tid == 0) {
    if (!fail && !(S > 0.f && S < INFINITY)) {  // NaN, +inf or nothing but -inf
      fail = true;
      bits |= kErrBadLogits;
    }
    const float ls = log2f(S);
    float lp = NAN, H = NAN;
    if (!fail) {
      H = T == 0.f ? 0.f : fmaxf(kLn2 * (ls - E / S), 0.f);
      if (tok_ok) lp = T == 0.f ? (count == 0 ? 0.f : -INFINITY) : log_prob(zt, m, c, T, ls);
    }
    p.logprob[r] = lp;
    if (p.entropy) p.entropy[r] = H;
    if (p.rank) p.rank[r] = !fail && tok_ok ? count + 1 : -1;
    if (bits) atomicOr(p.err, bits);
    sm.m[0] = m;
    sm.S[0] = fail ? NAN : ls;
  }
  if (TOP) {
    __syncthreads();
    if (tid < K) {
      const float ls = sm.S[0];
      const bool ok = ls == ls;  // the row is valid
      float lp = NAN;
      int i = -1;
      if (ok) {
        const unsigned long long k = sm.best[tid];
        const float v = key_value(k);
        i = k ? key_index(k) : -1;
        lp = i < 0 ? -INFINITY : T == 0.f ? (tid == 0 ? 0.f : -INFINITY) : log_prob(v, sm.m[0], c, T, ls);
      }
      p.top_tok[static_cast<long long>(r) * K + tid] = i;
      p.top_logprob[static_cast<long long>(r) * K + tid] = lp;
    }
  }
}

// Parts of a row: as many as make the whole shortest, in elements' time on a
// full SM (24 K bf16 or 12 K fp32 elements a microsecond).  n CTAs of an SM take
// turns (one alone reaches 7/8 of the rate) and begin and end in 4 us, or 8 us and
// 0.1 us K where the best are asked for; the join of the parts costs 1.3 us.
// (8 rows of 128256 bf16 logits: K = 0 12.2 us whole, 8.1, 7.0, 6.8 in 4, 8, 31
// parts, 6.5 as chosen; K = 5 18.5, 11.8, 10.3, 10.1, 9.6; 384 rows of 151936, K = 20:
// 43 us whole, 54 in two.)
int split_of(int R, int V, int K, bool half) {
  const long long us = half ? 24000 : 12000, sms = 152, ctas = K > 0 && !half ? 4 : 3;
  const long long fixed = K > 0 ? 8 * us + us * K / 10 : 4 * us;
  const int most = K > 0 && half ? 14 : 10;  // tenths of an element's time
  const auto wave = [&](long long n, long long v) {
    return n == 0 ? 0 : fixed + us * (n - 1) / 2 + (n == 1 ? v * 8 / 7 : v * n) * most / 10;
  };
  long long least = 0;
  int best = 1;
  const int parts = R <= kCounters ? kMaxSplit : 1;
  for (int s = 1; s <= parts && (s == 1 || V / s >= 4096); ++s) {
    const long long all = static_cast<long long>(R) * s, v = V / s;
    const long long cost = all / (sms * ctas) * wave(ctas, v) + wave((all % (sms * ctas) + sms - 1) / sms, v) +
                           (s > 1 ? us * 13 / 10 + us * s / 50 : 0);
    if (s == 1 || cost < least) {
      least = cost;
      best = s;
    }
  }
  return best;
}

template <class Tag>
cudaError_t launch_t(const LogprobParams& p, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>(p.R) * p.split;
  const auto kernel = p.K > 0 ? logprob_kernel<Tag, true> : logprob_kernel<Tag, false>;
  const cudaError_t e =
      cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(sizeof(LpSmem)));
  if (e != cudaSuccess) return e;
  kernel<<<grid, kLpThreads, sizeof(LpSmem), s>>>(p);
  return cudaGetLastError();
}

// The counters have a place of their own in front, so that calls of different
// sizes may take turns with a workspace.
constexpr size_t kPartsAt = 256 + 4 * kCounters;
size_t part_keys_at(size_t n) { return kPartsAt + sizeof(Part) * n; }

}  // namespace

size_t logprobs_bytes(int R, int V, int K) {
  size_t most = 256;
  for (const bool half : {false, true}) {
    const int split = split_of(R, V, K, half);
    const size_t n = static_cast<size_t>(R) * split;
    if (split > 1) most = std::max(most, part_keys_at(n) + 8 * kLpTop * n);
  }
  return most;
}

cudaError_t launch_logprobs(const LogprobParams& p0, int dtype, bool vec, cudaStream_t s) {
  LogprobParams p = p0;
  p.split = split_of(p.R, p.V, p.K, dtype == 1);
  char* ws = reinterpret_cast<char*>(p.err);
  p.counter = reinterpret_cast<int*>(ws + 256);
  p.parts = reinterpret_cast<Part*>(ws + kPartsAt);
  p.part_key = reinterpret_cast<unsigned long long*>(ws + part_keys_at(static_cast<size_t>(p.R) * p.split));
  p.whole = vec;
  return dtype == 1 ? launch_t<BF16Tag>(p, s) : launch_t<F32Tag>(p, s);
}

}  // namespace ssd

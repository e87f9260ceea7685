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
// below 1e-7 are summed by a plain second loop.  The rank is a count of the
// elements that come before the token's logit, known before the pass.
//
// Best alternatives: the K-th largest of a few of the first elements bounds the
// K-th largest of all from below; elements that reach the bound go to a list in
// shared memory, and the bound rises a few times as the list grows.  The pass
// compares one maximum per vector with it.  A row with more such elements than
// the list holds (thousands of equal logits, or of -inf) is searched K times
// instead.
//
// Bound: HBM for fp32; for bf16 also the instructions (about 8 an element; the
// largest element, the floor under -inf and the count for the rank are packed
// 16-bit operations).  One CTA per row, or per part of a row, whose last CTA to
// finish joins the parts.
#include <math.h>

#include "ssd_device.cuh"
#include "ssd_kv.cuh"

namespace ssd {
namespace {

constexpr int kLpThreads = 256;
constexpr int kLpCtas = 4;        // per SM
constexpr int kFlight = 4;        // vectors of a thread and round
constexpr int kStages = 3;        // rounds on their way into shared memory
constexpr int kSlice = 32 * kFlight;  // a warp's vectors of a round
constexpr int kLpWarps = kLpThreads / 32;
constexpr int kList = 1024;       // elements of the list, a part of it for each warp (one counter
                                  // for all of them, with its atomics, cost more than the pass)
constexpr int kOwn = kList / kLpWarps;
constexpr int kMaxSplit = 32;     // parts of a row
constexpr int kLpTop = 32;        // SSD_MAX_TOP
constexpr float kStep = 16.f;     // excess of an element over m that moves it
constexpr float kLowest = -3.0e38f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLog2e = 1.4426950408889634f;

using Part = LogprobPart;

constexpr int kRaise = 16;   // candidates of a warp that raise the bound
constexpr int kFirst = 6;  // most of each warp's maxima of the first round

struct LpSmem {
  uint4 ring[kLpWarps][kStages][kSlice];  // each warp's own
  unsigned long long bar[kLpWarps][kStages];
  alignas(16) unsigned long long key[kList];  // candidates: order of the value, then of the index
  unsigned long long best[kLpTop];
  float m[kLpWarps], S[kLpWarps], U[kLpWarps];
  int count[kLpWarps];
  float top[kLpWarps * kFirst];
  unsigned long long wkey[kLpWarps];
  int n[kLpWarps], last;
  float tau;
};

// A (value, index) pair as one number that orders by value, then by lower
// index; -0 counts as 0.
__device__ __forceinline__ unsigned long long key_of(float v, int i) {
  const uint32_t b = __float_as_uint(v + 0.f);
  const uint32_t u = b & 0x80000000u ? ~b : b | 0x80000000u;
  return (static_cast<unsigned long long>(u) << 32) | (0x7fffffffu - static_cast<uint32_t>(i));
}
__device__ __forceinline__ float key_value(unsigned long long k) {
  const uint32_t u = static_cast<uint32_t>(k >> 32);
  return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u);
}
__device__ __forceinline__ int key_index(unsigned long long k) {
  return static_cast<int>(0x7fffffffu - static_cast<uint32_t>(k));
}
__device__ __forceinline__ float redux_max(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
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
  // z c - mc, at least about -1000 (2^-1000 (-1000) = 0 where the logit is -inf)
  __device__ __forceinline__ void scaled(f32x2 c, f32x2 m, f32x2 (&x)[4]) const {
    float a, b;
    up2(fma2(pk2(r.x, r.y), c, m), a, b);
    x[0] = pk2(max_nan(a, -1000.f), max_nan(b, -1000.f));
    up2(fma2(pk2(r.z, r.w), c, m), a, b);
    x[1] = pk2(max_nan(a, -1000.f), max_nan(b, -1000.f));
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
  // the floor, -1e30, under the logits themselves: c is at most 1.5e7
  __device__ __forceinline__ void scaled(f32x2 c, f32x2 m, f32x2 (&x)[4]) const {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t f = max_nan_bf16x2(w[k], 0xf149f149u);
      x[k] = fma2(pk2(__uint_as_float(f << 16), __uint_as_float(f & 0xffff0000u)), c, m);
    }
  }
  __device__ __forceinline__ void count(Bound t, Count& n) const {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int k = 0; k < 4; ++k)
      n.n = __hadd2(n.n, __hgt2(*reinterpret_cast<const __nv_bfloat162*>(&w[k]), t));
  }
};

// S and U of a part of a row by a plain second loop around its maximum m:
// rows whose m c is too large to be rounded once for all elements, and
// temperatures below 1e-7.
template <class Tag>
__device__ __noinline__ void sum_plain(const typename Tag::Elem* z, int i0, int i1, float c, float& m, float& S,
                                       float& E) {
  S = 0.f;
  E = 0.f;
  for (int i = i0 + threadIdx.x; i < i1; i += kLpThreads) {
    const float x = max_nan((Tag::load1(z + i) - m) * c, -1000.f), e = exp2f(x);
    S += e;
    E = fmaf(e, x, E);
  }
}

// What two lanes or parts hold, joined over the warp in a fixed order: m first,
// then sums of scaled S and U.
__device__ __forceinline__ void join_warp(float c, float& m, float& S, float& U) {
  float M = m;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
  const float d0 = fmaxf((m - M) * c, -1e4f), f = exp2f(d0);  // 2^-1e4 = 0
  U = f * fmaf(S, d0, U);
  S *= f;
  m = M;
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) {
    S += __shfl_xor_sync(0xffffffffu, S, d);
    U += __shfl_xor_sync(0xffffffffu, U, d);
  }
}

// Keys that come before one, of the first n (an even number) of `parts` lists
// kOwn apart.
__device__ __forceinline__ int rank_of(const unsigned long long* key, int parts, int n, unsigned long long mine) {
  int rank = 0;
#pragma unroll 1
  for (int w = 0; w < parts; ++w) {
#pragma unroll 4
    for (int k = 0; k < n; k += 2) {
      const ulonglong2 two = *reinterpret_cast<const ulonglong2*>(key + w * kOwn + k);
      rank += (two.x > mine) + (two.y > mine);
    }
  }
  return rank;
}

// The K first of different keys (0: none), in order, into best, which holds
// zeros: every thread counts the keys before its own.
__device__ __forceinline__ void select_best(const unsigned long long* key, int parts, int n, int K,
                                            unsigned long long* best) {
#pragma unroll 1
  for (int j = threadIdx.x; j < parts * n; j += kLpThreads) {
    const unsigned long long mine = key[(j / n) * kOwn + j % n];
    if (mine == 0) continue;
    const int rank = rank_of(key, parts, n, mine);
    if (rank < K) best[rank] = mine;
  }
}

// ---------------------------------------------------------------------------
// Bulk copies of a warp's slices into its ring, one mbarrier a stage.
// ---------------------------------------------------------------------------
__device__ __forceinline__ uint32_t lp_ptr(const void* p) {
  return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}
__device__ __forceinline__ void lp_copy(uint4* dst, const void* src, int bytes, unsigned long long* bar) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(lp_ptr(bar)), "r"(bytes) : "memory");
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(
                   lp_ptr(dst)),
               "l"(src), "r"(bytes), "r"(lp_ptr(bar))
               : "memory");
}
// Bounded wait: false after a second.
__device__ __forceinline__ bool lp_wait(unsigned long long* bar, uint32_t parity) {
  unsigned long long t0 = 0;
  for (unsigned i = 1;; ++i) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.b32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(lp_ptr(bar)), "r"(parity), "r"(20000)
        : "memory");
    if (ok) return true;
    if ((i & 31) == 0) {
      unsigned long long t;
      asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
      if (t0 == 0) t0 = t;
      if (t - t0 > 1000000000ull) return false;
    }
  }
}

// The K first elements of a part of a row, one search each (rows whose
// candidates do not fit the list).
template <class Tag>
__device__ __noinline__ void search_best(LpSmem& sm, const typename Tag::Elem* z, int i0, int i1, int K) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
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
__global__ void __launch_bounds__(kLpThreads, kLpCtas) logprob_kernel(const __grid_constant__ LogprobParams p) {
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
  const float c = T > 0.f ? kLog2e / T : kLog2e;
  const typename Tag::Elem* z =
      static_cast<const typename Tag::Elem*>(p.logits) + static_cast<long long>(fail ? 0 : row) * p.row_stride;
  const int nv = (p.V + N - 1) / N;  // vectors of a row
  const int per = (nv + p.split - 1) / p.split;
  const int v0 = min(nv, part * per), v1 = min(nv, v0 + per);
  float m = kLowest, S = 0.f, E = 0.f, zt = INFINITY;
  int count = 0;
  if (TOP && tid < kLpTop) sm.best[tid] = 0;
  if (!fail) {
    if (tok_ok) zt = Tag::load1(z + tok);
    const typename Raw<Tag>::Bound after = Raw<Tag>::bound(zt),
                                   ahead = zt > -INFINITY && zt < INFINITY ? Raw<Tag>::below(zt) : after;
    typename Raw<Tag>::Count cnt;
    float tau = -INFINITY, mc = 0.f;
    bool plain = c > 1e7f;
    int own = 0;  // candidates of the warp
    // the longest of the warps' lists, an even number; the others filled up
    // with zeros
    auto longest = [&](int most) {
      if (lane == 0) sm.n[warp] = own;
      __syncthreads();
      int n = 0;
#pragma unroll
      for (int w = 0; w < kLpWarps; ++w) n = max(n, sm.n[w]);
      n = min((n + 1) & ~1, most);
      for (int k = own + lane; k < n; k += 32) sm.key[warp * kOwn + k] = 0;
      __syncthreads();
      return n;
    };
    const f32x2 c2 = pk2(c, c);
    // the rounding error of m c out of the sums
    auto exact = [&]() {
      if (m == kLowest) return;  // nothing yet
      const float d = -fmaf(m, c, -mc), f = exp2f(d);
      E = f * fmaf(S, d, E);
      S *= f;
    };
    int round = 0, raise_at = 4;
    Raw<Tag> now[U];
    // aligned rows come by bulk copies, a warp's slices on its own ring
    const int vfull = p.whole ? min(v1, p.V / N) : v0;
    unsigned long long* bar = sm.bar[warp];
    auto slice = [&](int k) { return v0 + k * (kLpThreads * U) + warp * kSlice; };
    auto fetch = [&](int k, int stage) {
      const int v = slice(k), n = min(kSlice, vfull - v);
      if (n > 0 && lane == 0) lp_copy(sm.ring[warp][stage], z + static_cast<long long>(v) * N, n * 16, bar + stage);
    };
    if (lane == 0) {
#pragma unroll
      for (int k = 0; k < kStages; ++k)
        asm volatile("mbarrier.init.shared::cta.b64 [%0], 1;" ::"r"(lp_ptr(bar + k)) : "memory");
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncwarp();
#pragma unroll
    for (int k = 0; k < kStages; ++k) fetch(k, k);
    int stage = 0;
    uint32_t phase = 0;
#pragma unroll 1
    for (int b = v0; b < v1; b += kLpThreads * U, ++round) {
      const int first = slice(round), n = min(kSlice, vfull - first);
      if (n > 0 && !lp_wait(bar + stage, phase)) bits |= kErrTimeout;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int k = u * 32 + lane;
        if (k < n) now[u].raw(sm.ring[warp][stage][k]);
        else if (first + k < v1) now[u].load(z, first + k, p.V, p.whole);
        else now[u].none();
      }
      __syncwarp();
      fetch(round + kStages, stage);
      if (++stage == kStages) {
        stage = 0;
        phase ^= 1;
      }
      if (TOP && round == 0) {
        // of every warp the largest of its threads' maxima: the K-th largest
        // of those different elements is the first bound
        float v = now[0].top();
#pragma unroll
        for (int u = 1; u < U; ++u) v = fmaxf(v, now[u].top());
        const int take = min((K + kLpWarps - 1) / kLpWarps + 1, kFirst);
#pragma unroll 1
        for (int k = 0; k < take; ++k) {
          const float w = redux_max(v);
          if (lane == 0) sm.top[warp * take + k] = w;
          const unsigned who = __ballot_sync(0xffffffffu, v == w);
          if (lane == __ffs(who) - 1) v = -INFINITY;
        }
        __syncthreads();
        if (tid < kLpWarps * take) {
          const float mine = sm.top[tid];
          int rank = 0;
#pragma unroll 8
          for (int k = 0; k < kLpWarps * take; ++k) {
            const float o = sm.top[k];
            rank += o > mine || (o == mine && k < tid);
          }
          if (rank == K - 1) sm.tau = mine;
        }
        __syncthreads();
        tau = sm.tau;
      }
      unsigned hit = 0;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (first + u * 32 >= v1) break;
        const Raw<Tag>& w = now[u];
        const int i = (first + u * 32 + lane) * N;
        const float top = w.top();
        // the reference
        if ((top - m) * c > kStep) {  // (the first vector's from kLowest, S = 0)
          exact();
          const float d = fmaxf((m - top) * c, -1e4f), f = exp2f(d);
          E = f * fmaf(S, d, E);
          S *= f;
          m = top;
          mc = m * c;
          plain |= !(fabsf(mc) < 16777216.f);
        }
        f32x2 x[4], s2 = pk2(0.f, 0.f), e2 = pk2(0.f, 0.f);
        w.scaled(c2, pk2(-mc, -mc), x);
#pragma unroll
        for (int k = 0; k < N / 2; ++k) {
          float a, d;
          up2(x[k], a, d);
          const f32x2 e = pk2(ex2_fast(a), ex2_fast(d));
          s2 = add2(s2, e);
          e2 = fma2(e, x[k], e2);
        }
        float a, d;
        up2(s2, a, d);
        S += a + d;
        up2(e2, a, d);
        E += a + d;
        // the rank: vectors before the token's, behind it, its own
        if (i > tok || i + N <= tok) {
          w.count(i > tok ? after : ahead, cnt);
        } else {
          float y[8];
          Tag::unpackraw(w.r, y);
#pragma unroll
          for (int k = 0; k < N; ++k) count += y[k] > zt || (y[k] == zt && i + k < tok);
        }
        if (TOP) hit |= static_cast<unsigned>(__any_sync(0xffffffffu, top >= tau)) << u;
      }
      if (TOP) {
        // the warp's candidates (one copy of this code for all vectors)
#pragma unroll 1
        while (hit) {
          const int u = __ffs(hit) - 1;
          hit &= hit - 1;
          Raw<Tag> w = now[0];
#pragma unroll
          for (int k = 1; k < U; ++k)
            if (u == k) w = now[k];
          const int i = (first + u * 32 + lane) * N;
          float y[8];
          Tag::unpackraw(w.r, y);
          unsigned hits = 0;
#pragma unroll
          for (int k = 0; k < N; ++k) hits |= (y[k] >= tau && i + k < p.V) ? 1u << k : 0u;
          const int mine = __popc(hits);
          int at = mine;
#pragma unroll
          for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, at, d);
            if (lane >= d) at += o;
          }
          const int sum = __shfl_sync(0xffffffffu, at, 31);
          at += own - mine;
          own += sum;
#pragma unroll
          for (int k = 0; k < N; ++k) {
            if ((hits >> k) & 1) {
              if (at < kOwn) sm.key[warp * kOwn + at] = key_of(y[k], i + k);
              ++at;
            }
          }
        }
      }
      count += cnt.take();
      if (TOP) {
        if (round + 1 == raise_at && b + kLpThreads * U < v1) {
          raise_at *= 8;
          // a bound from the first candidates of every warp
          const int n = longest(kRaise);
          if (tid < kLpWarps * kRaise && tid % kRaise < n) {
            const unsigned long long mine = sm.key[tid / kRaise * kOwn + tid % kRaise];
            if (mine && rank_of(sm.key, kLpWarps, n, mine) == K - 1) sm.tau = fmaxf(tau, key_value(mine));
          }
          __syncthreads();
          tau = sm.tau;
        }
      }
    }
    exact();
    // a masked token: the masked ones before it
    if (tok_ok && zt == -INFINITY)
      for (int i = v0 * N + tid; i < min(tok, v1 * N); i += kLpThreads) count += Tag::load1(z + i) == -INFINITY;
    if (__syncthreads_or(plain)) {
      float top = -INFINITY;
      for (int i = v0 * N + tid; i < min(p.V, v1 * N); i += kLpThreads) top = fmaxf(top, Tag::load1(z + i));
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
      if (lane == 0) sm.m[warp] = top;
      __syncthreads();
      m = kLowest;
      for (int w = 0; w < kLpWarps; ++w) m = fmaxf(m, sm.m[w]);
      __syncthreads();
      sum_plain<Tag>(z, v0 * N, min(p.V, v1 * N), c, m, S, E);
    }
    // lanes of a warp, warps of the CTA
    join_warp(c, m, S, E);
    count = __reduce_add_sync(0xffffffffu, count);
    if (lane == 0) {
      sm.m[warp] = m;
      sm.S[warp] = S;
      sm.U[warp] = E;
      sm.count[warp] = count;
    }
    const int n = TOP ? longest(kOwn) : 0;  // (and the barrier)
    if (!TOP) __syncthreads();
    if (TOP) {
      bool full = false;
#pragma unroll
      for (int w = 0; w < kLpWarps; ++w) full |= sm.n[w] > kOwn;
      if (full) search_best<Tag>(sm, z, v0 * N, min(p.V, v1 * N), K);
      else select_best(sm.key, kLpWarps, n, K, sm.best);
    }
    if (warp == 0) {
      const bool in = lane < kLpWarps;
      m = in ? sm.m[lane] : kLowest;
      S = in ? sm.S[lane] : 0.f;
      E = in ? sm.U[lane] : 0.f;
      join_warp(c, m, S, E);
      count = __reduce_add_sync(0xffffffffu, in ? sm.count[lane] : 0);
    }
    __syncthreads();
  }
  bool last = true;
  if (p.split > 1) {
    Part* parts = p.parts + static_cast<long long>(r) * p.split;
    unsigned long long* tk = p.part_key + static_cast<long long>(r) * p.split * kLpTop;
    if (!fail) {
      if (TOP && tid < K) {
        tk[part * kLpTop + tid] = sm.best[tid];
      }
      if (tid == 0) {
        Part q;
        q.m = m; q.S = S; q.U = E; q.count = count;
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
      if (warp == 0) {  // lane k holds part k
        const bool in = lane < p.split;
        m = in ? __ldcg(&parts[lane].m) : kLowest;
        S = in ? __ldcg(&parts[lane].S) : 0.f;
        E = in ? __ldcg(&parts[lane].U) : 0.f;
        join_warp(c, m, S, E);
        count = __reduce_add_sync(0xffffffffu, in ? __ldcg(&parts[lane].count) : 0);
      }
      if constexpr (TOP) {
        const int n = p.split * K;
        if (tid < kLpTop) sm.best[tid] = 0;
        for (int j = tid; j < n + (n & 1); j += kLpThreads)
          sm.key[j] = j < n ? __ldcg(tk + (j / K) * kLpTop + j % K) : 0ull;
        __syncthreads();
        select_best(sm.key, 1, n + (n & 1), K, sm.best);
        __syncthreads();
      }
    }
  }
  // the answer
  if (tid == 0) {
    if (!fail && !(S > 0.f && S < INFINITY)) {  // NaN, +inf or nothing but -inf
      fail = true;
      bits |= kErrBadLogits;
    }
    const float ls = log2f(S);
    float lp = NAN, H = NAN;
    if (!fail) {
      H = T == 0.f ? 0.f : kLn2 * (ls - E / S);
      if (tok_ok) lp = T == 0.f ? (count == 0 ? 0.f : -INFINITY) : ((zt - m) * c - ls) * kLn2;
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
        lp = i < 0 ? -INFINITY : T == 0.f ? (tid == 0 ? 0.f : -INFINITY) : ((v - sm.m[0]) * c - ls) * kLn2;
      }
      p.top_tok[static_cast<long long>(r) * K + tid] = i;
      p.top_logprob[static_cast<long long>(r) * K + tid] = lp;
    }
  }
}

// Parts of a row: as many as make the work of the longest place shortest, in
// elements: what a CTA reads; its start and end, and its list of K; and the
// join of the parts' lists (measured at R = 8 .. 4096: 16 K, 1.5 K and 0.2 K
// elements' time).
int split_of(int R, int V, int K) {
  const long long places = 152 * kLpCtas;
  long long least = 0;
  int best = 1;
  for (int s = 1; s <= kMaxSplit && (s == 1 || V / s >= 4096); ++s) {
    const long long waves = (static_cast<long long>(R) * s + places - 1) / places;
    const long long cost = waves * (V / s + 16384 + 1536 * K) + (s > 1 ? 16384 + 200ll * s * K : 0);
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

struct LpLayout {
  size_t counter, parts, key, total;
};
LpLayout lp_layout(int R, int V, int K) {
  const size_t n = static_cast<size_t>(R) * split_of(R, V, K);
  LpLayout L;
  L.counter = 256;
  L.parts = (L.counter + 4ull * R + 255) / 256 * 256;
  L.key = L.parts + sizeof(Part) * n;
  L.total = L.key + 8 * kLpTop * n;
  return L;
}

}  // namespace

size_t logprobs_bytes(int R, int V, int K) { return split_of(R, V, K) > 1 ? lp_layout(R, V, K).total : 256; }

cudaError_t launch_logprobs(const LogprobParams& p0, int dtype, bool vec, cudaStream_t s) {
  LogprobParams p = p0;
  p.split = split_of(p.R, p.V, p.K);
  const LpLayout L = lp_layout(p.R, p.V, p.K);
  char* ws = reinterpret_cast<char*>(p.err);
  p.counter = reinterpret_cast<int*>(ws + L.counter);
  p.parts = reinterpret_cast<Part*>(ws + L.parts);
  p.part_key = reinterpret_cast<unsigned long long*>(ws + L.key);
  p.whole = vec;
  return dtype == 1 ? launch_t<BF16Tag>(p, s) : launch_t<F32Tag>(p, s);
}

}  // namespace ssd

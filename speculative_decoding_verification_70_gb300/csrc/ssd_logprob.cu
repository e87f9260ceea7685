// ssd_logprob.cu -- log probabilities of given tokens with entropy, rank and
// the best alternatives, in one pass over the rows.
//
// With a reference m and x = (z - m) c, c = log2(e) / T (the difference first:
// it is exact where it matters),
//     S = sum 2^x,  U = sum 2^x x:
//     log p(v) = ln 2 (x_v - log2 S),   H = ln 2 (log2 S - U / S).
// A thread's m is the maximum of its first elements and moves only when an
// element's 2^x exceeds 2^16 (S and U then scale: S' = 2^d S, U' = 2^d (U + d S),
// d = (m - m') c); threads, and CTAs that share a row, are joined by the same rule
// in a fixed order.  The rank is a count of the elements that come before the
// token's logit, known before the pass.
//
// Best alternatives: the K-th largest of a few of the first elements bounds the
// K-th largest of all from below; elements that reach the bound go to a list in
// shared memory, and the bound rises a few times as the list grows.  The pass
// compares one maximum per vector with it.  A row with more such elements than
// the list holds (thousands of equal logits, or of -inf) is searched K times
// instead.
//
// Bound: HBM, about 7 operations an element.  One CTA per row, or (fewer rows
// than fill the GPU four times over) per part of a row, whose last CTA to finish
// joins the parts.
#include <math.h>

#include "ssd_device.cuh"
#include "ssd_kv.cuh"

namespace ssd {
namespace {

constexpr int kLpThreads = 256;
constexpr int kLpCtas = 3;        // per SM
constexpr int kFlight = 4;        // vectors of a thread on their way while four others are worked on
constexpr int kLpWarps = kLpThreads / 32;
constexpr int kList = 1024;       // elements of the list
constexpr int kMaxSplit = 32;     // parts of a row
constexpr int kLpTop = 32;        // SSD_MAX_TOP
constexpr float kStep = 16.f;     // excess of an element over m that moves it
constexpr float kLowest = -3.0e38f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLog2e = 1.4426950408889634f;

using Part = LogprobPart;

constexpr int kRaise = 256;  // candidates that raise the bound
constexpr int kFirst = 8;  // of each warp's maxima of the first round

struct LpSmem {
  unsigned long long key[kList];  // candidates: order of the value, then of the index
  unsigned long long best[kLpTop];
  float m[kLpWarps], S[kLpWarps], U[kLpWarps];
  int count[kLpWarps];
  float top[kLpWarps * kFirst];
  unsigned long long wkey[kLpWarps];
  int n, last;
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

// (m, S, U) joined with another part's.
__device__ __forceinline__ void join(float c, float& m, float& S, float& U, float m2, float S2, float U2) {
  const float M = fmaxf(m, m2);
  const float d = fmaxf((m - M) * c, -1e4f), d2 = fmaxf((m2 - M) * c, -1e4f);  // 2^-1e4 = 0
  const float f = exp2f(d), f2 = exp2f(d2);
  U = f * fmaf(S, d, U) + f2 * fmaf(S2, d2, U2);
  S = f * S + f2 * S2;
  m = M;
}

// Vector v of a row of V elements as it lies in memory, -inf behind the row's
// end (`whole`: the row is 16-byte aligned).
template <class Tag>
struct Raw;
template <>
struct Raw<F32Tag> {
  float4 r;
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
  __device__ __forceinline__ void none() { r = make_float4(-INFINITY, -INFINITY, -INFINITY, -INFINITY); }
};
template <>
struct Raw<BF16Tag> {
  uint4 r;
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
  __device__ __forceinline__ void none() { r = make_uint4(0xff80ff80u, 0xff80ff80u, 0xff80ff80u, 0xff80ff80u); }
};

template <int N>
__device__ __forceinline__ float largest(const float (&x)[8]) {
  float t = x[0];
#pragma unroll
  for (int k = 1; k < N; ++k) t = fmaxf(t, x[k]);
  return t;
}

// The K first of n different keys, in order, into best (0 where there are
// fewer): every thread counts the keys before its own.
__device__ __forceinline__ void select_best(const unsigned long long* key, int n, int K, unsigned long long* best) {
  if (threadIdx.x >= n && threadIdx.x < K) best[threadIdx.x] = 0;
#pragma unroll 1
  for (int j = threadIdx.x; j < n; j += kLpThreads) {
    const unsigned long long mine = key[j];
    int rank = 0;
#pragma unroll 4
    for (int k = 0; k < n; ++k) rank += key[k] > mine;
    if (rank < K) best[rank] = mine;
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
  __shared__ LpSmem sm;
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
  bool full = false;  // more candidates than the list holds
  if (!fail) {
    if (tok_ok) zt = Tag::load1(z + tok);
    float tau = -INFINITY;
    if (TOP && tid == 0) sm.n = 0;
    const f32x2 c2 = pk2(c, c);
    int round = 0, raise_at = 2;
    Raw<Tag> now[U], next[U];
    auto load = [&](Raw<Tag>(&to)[U], int b) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int v = b + u * kLpThreads + tid;
        if (v < v1) to[u].load(z, v, p.V, p.whole);
        else to[u].none();
      }
    };
    load(now, v0);
#pragma unroll 1
    for (int b = v0; b < v1; b += kLpThreads * U, ++round) {
      load(next, b + kLpThreads * U);
      if (TOP && round == 0) {
        // of every warp the largest of its threads' maxima: the K-th largest
        // of those different elements is the first bound
        float v = -INFINITY;
#pragma unroll
        for (int u = 0; u < U; ++u) {
          float x[8];
          Tag::unpackraw(now[u].r, x);
          v = fmaxf(v, largest<N>(x));
        }
#pragma unroll 1
        for (int k = 0; k < kFirst; ++k) {
          const float w = redux_max(v);
          if (lane == 0) sm.top[warp * kFirst + k] = w;
          const unsigned who = __ballot_sync(0xffffffffu, v == w);
          if (lane == __ffs(who) - 1) v = -INFINITY;
        }
        __syncthreads();
        if (tid < kLpWarps * kFirst) {
          const float mine = sm.top[tid];
          int rank = 0;
#pragma unroll 8
          for (int k = 0; k < kLpWarps * kFirst; ++k) {
            const float o = sm.top[k];
            rank += o > mine || (o == mine && k < tid);
          }
          if (rank == K - 1) sm.tau = mine;
        }
        __syncthreads();
        tau = sm.tau;
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        float x[8];
        Tag::unpackraw(now[u].r, x);
        const int i = (b + u * kLpThreads + tid) * N;
        const float top = largest<N>(x);
        // the reference
        if ((top - m) * c > kStep) {  // (the first vector's from kLowest, S = 0)
          const float d = fmaxf((m - top) * c, -1e4f), f = exp2f(d);
          E = f * fmaf(S, d, E);
          S *= f;
          m = top;
        }
        const f32x2 m2 = pk2(-m, -m);
        f32x2 s2 = pk2(0.f, 0.f), e2 = pk2(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < N; k += 2) {
          float a, d;
          up2(mul2(add2(pk2(x[k], x[k + 1]), m2), c2), a, d);
          a = max_nan(a, -1000.f);  // 2^-1000 (-1000) = 0 where the logit is -inf
          d = max_nan(d, -1000.f);
          const f32x2 e = pk2(ex2_fast(a), ex2_fast(d));
          s2 = add2(s2, e);
          e2 = fma2(e, pk2(a, d), e2);
        }
        float a, d;
        up2(s2, a, d);
        S += a + d;
        up2(e2, a, d);
        E += a + d;
        // the rank: vectors before the token's, behind it, its own
        if (i + N <= tok) {
#pragma unroll
          for (int k = 0; k < N; ++k) count += x[k] >= zt;
        } else if (i > tok) {
#pragma unroll
          for (int k = 0; k < N; ++k) count += x[k] > zt;
        } else {
#pragma unroll
          for (int k = 0; k < N; ++k) count += x[k] > zt || (x[k] == zt && i + k < tok);
        }
        if (TOP && top >= tau) {
#pragma unroll
          for (int k = 0; k < N; ++k) {
            if (x[k] >= tau && i + k < p.V) {
              const int at = atomicAdd(&sm.n, 1);
              if (at < kList) sm.key[at] = key_of(x[k], i + k);
            }
          }
        }
      }
      if (TOP) {
        if (round + 1 == raise_at && b + kLpThreads * U < v1) {
          raise_at *= 4;
          __syncthreads();
          const int n = min(sm.n, kRaise);  // of the first of them: a bound, too
          if (tid < n) {
            const unsigned long long mine = sm.key[tid];
            int rank = 0;
#pragma unroll 4
            for (int k = 0; k < n; ++k) rank += sm.key[k] > mine;
            if (rank == K - 1) sm.tau = fmaxf(tau, key_value(mine));
          }
          __syncthreads();
          tau = sm.tau;
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) now[u] = next[u];
    }
    // threads of a warp, warps of the CTA
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
      const float m2 = __shfl_xor_sync(0xffffffffu, m, d), S2 = __shfl_xor_sync(0xffffffffu, S, d),
                  E2 = __shfl_xor_sync(0xffffffffu, E, d);
      // the same order on both sides: bits do not depend on the lane
      if (lane & d) {
        float mm = m2, ss = S2, ee = E2;
        join(c, mm, ss, ee, m, S, E);
        m = mm; S = ss; E = ee;
      } else {
        join(c, m, S, E, m2, S2, E2);
      }
      count += __shfl_xor_sync(0xffffffffu, count, d);
    }
    if (lane == 0) {
      sm.m[warp] = m;
      sm.S[warp] = S;
      sm.U[warp] = E;
      sm.count[warp] = count;
    }
    __syncthreads();
    if (TOP) {
      full = sm.n > kList;
      if (full) {
        search_best<Tag>(sm, z, v0 * N, min(p.V, v1 * N), K);
      } else {
        select_best(sm.key, sm.n, K, sm.best);
      }
    }
    if (tid == 0) {
      for (int w = 1; w < kLpWarps; ++w) {
        join(c, m, S, E, sm.m[w], sm.S[w], sm.U[w]);
        count += sm.count[w];
      }
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
      if (tid == 0) {
        m = __ldcg(&parts[0].m);
        S = __ldcg(&parts[0].S);
        E = __ldcg(&parts[0].U);
        count = __ldcg(&parts[0].count);
      }
      if (warp == 0) {
        // lane k holds part k; joined in order by lane 0
        const bool in = lane < p.split;
        const float pm = in ? __ldcg(&parts[lane].m) : 0.f, pS = in ? __ldcg(&parts[lane].S) : 0.f,
                    pU = in ? __ldcg(&parts[lane].U) : 0.f;
        const int pc = in ? __ldcg(&parts[lane].count) : 0;
        for (int k = 1; k < p.split; ++k) {
          const float a = __shfl_sync(0xffffffffu, pm, k), b = __shfl_sync(0xffffffffu, pS, k),
                      e = __shfl_sync(0xffffffffu, pU, k);
          const int n = __shfl_sync(0xffffffffu, pc, k);
          if (lane == 0) {
            join(c, m, S, E, a, b, e);
            count += n;
          }
        }
      }
      if (TOP) {
        if (tid == 0) sm.n = 0;
        __syncthreads();
        for (int j = tid; j < p.split * kLpTop; j += kLpThreads) {
          const unsigned long long k = j % kLpTop < K ? __ldcg(tk + j) : 0ull;
          if (k) sm.key[atomicAdd(&sm.n, 1)] = k;
        }
        __syncthreads();
        select_best(sm.key, sm.n, K, sm.best);
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

// Parts of a row: as many as make the waves of CTAs shortest, a CTA costing
// what it reads and about 4096 elements for its start and end.  (384 rows of
// 151936 as 384 CTAs on 456 places, or in 4 parts in 3.4 waves, leave a fifth
// of the GPU idle; in 7 parts it is a fiftieth.)
int split_of(int R, int V) {
  const long long places = 152 * kLpCtas;
  long long least = 0;
  int best = 1;
  for (int s = 1; s <= kMaxSplit && (s == 1 || V / s >= 4096); ++s) {
    const long long waves = (static_cast<long long>(R) * s + places - 1) / places;
    const long long cost = waves * (V / s + 4096);
    if (s == 1 || cost < least) {
      least = cost;
      best = s;
    }
  }
  return best;
}

template <class Tag>
void launch_t(const LogprobParams& p, cudaStream_t s) {
  const unsigned grid = static_cast<unsigned>(p.R) * p.split;
  if (p.K > 0) logprob_kernel<Tag, true><<<grid, kLpThreads, 0, s>>>(p);
  else logprob_kernel<Tag, false><<<grid, kLpThreads, 0, s>>>(p);
}

struct LpLayout {
  size_t counter, parts, key, total;
};
LpLayout lp_layout(int R, int V) {
  const size_t n = static_cast<size_t>(R) * split_of(R, V);
  LpLayout L;
  L.counter = 256;
  L.parts = (L.counter + 4ull * R + 255) / 256 * 256;
  L.key = L.parts + sizeof(Part) * n;
  L.total = L.key + 8 * kLpTop * n;
  return L;
}

}  // namespace

size_t logprobs_bytes(int R, int V) { return split_of(R, V) > 1 ? lp_layout(R, V).total : 256; }

cudaError_t launch_logprobs(const LogprobParams& p0, int dtype, bool vec, cudaStream_t s) {
  LogprobParams p = p0;
  p.split = split_of(p.R, p.V);
  const LpLayout L = lp_layout(p.R, p.V);
  char* ws = reinterpret_cast<char*>(p.err);
  p.counter = reinterpret_cast<int*>(ws + L.counter);
  p.parts = reinterpret_cast<Part*>(ws + L.parts);
  p.part_key = reinterpret_cast<unsigned long long*>(ws + L.key);
  p.whole = vec;
  if (dtype == 1) launch_t<BF16Tag>(p, s);
  else launch_t<F32Tag>(p, s);
  return cudaGetLastError();
}

}  // namespace ssd

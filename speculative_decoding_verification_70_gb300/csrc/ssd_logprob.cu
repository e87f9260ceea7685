// ssd_logprob.cu -- log probabilities of given tokens with entropy, rank and
// the best alternatives.
//
// One CTA per answer.  With x = (z - m) log2(e) / T, S = sum 2^x, U = sum 2^x x:
//     log p(v) = ln 2 (x_v - log2 S),   H = ln 2 (log2 S - U / S).
// The first pass finds the maximum, the second the sums and the rank, and
// each of K more the next token in the order (logit descending, index
// ascending).
#include <math.h>

#include "ssd_device.cuh"
#include "ssd_kv.cuh"

namespace ssd {
namespace {

constexpr int kLpThreads = 512;

struct LpSmem {
  float a[16], b[16];
  int i[16], n[16];
  float fa, fb;
  int fi, fn;
};

__device__ __forceinline__ bool before(float a, int ai, float b, int bi) {
  return a > b || (a == b && ai < bi);
}

// The first (value, index) pair of the CTA, by (value desc, index asc).
__device__ __forceinline__ void block_best(LpSmem& sm, float& v, int& i) {
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  for (int d = 16; d > 0; d >>= 1) {
    const float ov = __shfl_xor_sync(0xffffffffu, v, d);
    const int oi = __shfl_xor_sync(0xffffffffu, i, d);
    if (before(ov, oi, v, i)) { v = ov; i = oi; }
  }
  __syncthreads();
  if (lane == 0) { sm.a[w] = v; sm.i[w] = i; }
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int k = 1; k < kLpThreads / 32; ++k)
      if (before(sm.a[k], sm.i[k], v, i)) { v = sm.a[k]; i = sm.i[k]; }
    sm.fa = v; sm.fi = i;
  }
  __syncthreads();
  v = sm.fa; i = sm.fi;
}

template <class Tag>
__global__ void __launch_bounds__(kLpThreads) logprob_kernel(const LogprobParams p) {
  __shared__ LpSmem sm;
  const int r = blockIdx.x, tid = threadIdx.x, w = tid >> 5, lane = tid & 31;
  const int row = p.rows ? p.rows[r] : r;
  const int tok = p.tok[r];
  const float T = p.T ? p.T[r] : 1.f;
  int bits = 0;
  bool fail = false;
  if (row < 0) fail = true;
  if (row >= p.n_rows) { fail = true; bits |= kErrBadLength; }
  if (!(T >= 0.f)) { fail = true; bits |= kErrBadTemperature; }
  const bool tok_ok = tok >= 0 && tok < p.V;
  if (!tok_ok && tok != -1) bits |= kErrBadToken;
  const typename Tag::Elem* z = static_cast<const typename Tag::Elem*>(p.logits) +
                                static_cast<long long>(fail ? 0 : row) * p.row_stride;
  float m = -INFINITY, S = 0.f, U = 0.f, zt = 0.f;
  int am = 0x7fffffff, cnt = 0;
  const float c = T > 0.f ? 1.4426950408889634f / T : 0.f;
  if (!fail) {
    bool nan = false;
    for (int v = tid; v < p.V; v += kLpThreads) {
      const float x = Tag::load1(z + v);
      nan |= !(x < INFINITY);
      if (before(x, v, m, am)) { m = x; am = v; }
    }
    nan = __syncthreads_or(nan);
    block_best(sm, m, am);
    if (nan || m == -INFINITY) { fail = true; bits |= kErrBadLogits; }
  }
  if (!fail) {
    zt = tok_ok ? Tag::load1(z + tok) : 0.f;
    for (int v = tid; v < p.V; v += kLpThreads) {
      const float x = Tag::load1(z + v);
      const float y = fmaxf((x - m) * c, -1000.f), e = exp2f(y);
      S += e;
      U = fmaf(e, y, U);
      cnt += before(x, v, zt, tok) ? 1 : 0;
    }
    for (int d = 16; d > 0; d >>= 1) {
      S += __shfl_xor_sync(0xffffffffu, S, d);
      U += __shfl_xor_sync(0xffffffffu, U, d);
      cnt += __shfl_xor_sync(0xffffffffu, cnt, d);
    }
    __syncthreads();
    if (lane == 0) { sm.a[w] = S; sm.b[w] = U; sm.n[w] = cnt; }
    __syncthreads();
    if (tid == 0) {
      for (int k = 1; k < kLpThreads / 32; ++k) { S += sm.a[k]; U += sm.b[k]; cnt += sm.n[k]; }
      sm.fa = S; sm.fb = U; sm.fn = cnt;
    }
    __syncthreads();
    S = sm.fa; U = sm.fb; cnt = sm.fn;
  }
  const float ls = fail ? 0.f : log2f(S);
  const float ln2 = 0.6931471805599453f;
  if (tid == 0) {
    const float bad = NAN;
    float lp = bad, H = bad;
    if (!fail) {
      H = T == 0.f ? 0.f : ln2 * (ls - U / S);
      if (tok_ok) lp = T == 0.f ? (tok == am ? 0.f : -INFINITY) : ((zt - m) * c - ls) * ln2;
    }
    p.logprob[r] = lp;
    if (p.entropy) p.entropy[r] = H;
    if (p.rank) p.rank[r] = !fail && tok_ok ? cnt + 1 : -1;
    if (bits) atomicOr(p.err, bits);
  }
  float lv = INFINITY;
  int li = -1;
  for (int k = 0; k < p.K; ++k) {
    float bv = -INFINITY;
    int bi = 0x7fffffff;
    if (!fail) {
      for (int v = tid; v < p.V; v += kLpThreads) {
        const float x = Tag::load1(z + v);
        if (before(lv, li, x, v) && before(x, v, bv, bi)) { bv = x; bi = v; }
      }
      block_best(sm, bv, bi);
    }
    if (tid == 0) {
      const bool ok = !fail && bi < p.V;
      float lp = fail ? NAN : -INFINITY;
      if (ok) lp = T == 0.f ? (k == 0 ? 0.f : -INFINITY) : ((bv - m) * c - ls) * ln2;
      p.top_tok[static_cast<long long>(r) * p.K + k] = ok ? bi : -1;
      p.top_logprob[static_cast<long long>(r) * p.K + k] = lp;
    }
    lv = bv;
    li = bi;
  }
}

}  // namespace

cudaError_t launch_logprobs(const LogprobParams& p, int dtype, bool, cudaStream_t s) {
  if (dtype == 1) logprob_kernel<BF16Tag><<<p.R, kLpThreads, 0, s>>>(p);
  else logprob_kernel<F32Tag><<<p.R, kLpThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace ssd

// ssd_attn.cu -- attention of the drafted nodes over the paged cache.
//
// A warp per (node, query head): 32 slots at a time, one slot's score per
// lane, an online softmax (running maximum m, sum l, output o):
//     m' = max(m, max_s x_s),  o' = o 2^(m - m') + sum_s 2^(x_s - m') v_s.
// Slots a node does not see are skipped, so what they hold cannot matter.
#include <math.h>

#include "ssd_device.cuh"
#include "ssd_kv.cuh"

namespace ssd {
namespace {

constexpr int kRows = 4;  // warps per CTA

template <class T, int D>
__global__ void __launch_bounds__(32 * kRows) attn_kernel(const AttnParams p) {
  constexpr int E = D / 32;  // output columns per lane
  __shared__ float qs[kRows][D];
  const int w = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int N = p.nodes.N;
  const long long row = static_cast<long long>(blockIdx.x) * kRows + w;
  if (row >= static_cast<long long>(p.nodes.B) * N * p.Hq) return;
  const int h = static_cast<int>(row % p.Hq);
  const long long bj = row / p.Hq;
  const int j = static_cast<int>(bj % N), b = static_cast<int>(bj / N);
  const int hk = h / p.G;
  const int ctx = p.nodes.ctx_len[b];
  bool bad_len, broken;
  const int n = seq_nodes(ctx, p.nodes.n_nodes ? p.nodes.n_nodes[b] : N, N, p.kv.width, p.kv.ps, bad_len);
  uint64_t mask;
  int depth;
  const bool there = node_way(p.nodes.parent ? p.nodes.parent + static_cast<long long>(b) * N : nullptr,
                              n, j, mask, depth, broken);
  int bits = (bad_len ? kErrBadLength : 0) | (broken ? kErrBadTree : 0);
  const char* q = p.q + 2 * (b * p.q_b + j * p.q_n + h * p.q_h);
  for (int e = lane * 2; e < D; e += 64) {
    const uint32_t x = *reinterpret_cast<const uint32_t*>(q + 2 * e);
    qs[w][e] = T::lo(x);
    qs[w][e + 1] = T::hi(x);
  }
  __syncwarp();
  const float c = p.scale * 1.4426950408889634f;
  float m = -INFINITY, l = 0.f, o[E];
#pragma unroll
  for (int e = 0; e < E; ++e) o[e] = 0.f;
  const int tot = there ? ctx + n : 0;
  for (int s0 = 0; s0 < tot; s0 += 32) {
    const int s = s0 + lane;
    const bool seen = s < tot && (s < ctx || ((mask >> (s - ctx)) & 1));
    float x = -INFINITY;
    const char* vrow = nullptr;
    if (seen) {
      int page, off;
      float acc = 0.f;
      if (kv_slot(p.kv.table + b * p.kv.table_stride, p.kv.width, p.kv.pages, p.kv.ps, s, page, off)) {
        const char* k = p.kv.k + 2 * (page * p.kv.k_page + off * p.kv.k_slot + hk * p.kv.k_head);
        vrow = p.kv.v + 2 * (page * p.kv.v_page + off * p.kv.v_slot + hk * p.kv.v_head);
        for (int e = 0; e < D; e += 8) {
          float f[8];
          unpack8<T>(*reinterpret_cast<const uint4*>(k + 2 * e), f);
#pragma unroll
          for (int t = 0; t < 8; ++t) acc = fmaf(f[t], qs[w][e + t], acc);
        }
      } else {
        bits |= kErrBadPage;
      }
      x = acc * c;
    }
    float mx = x;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
    const float mn = fmaxf(m, mx);
    const float ref = mn == -INFINITY ? 0.f : mn;
    const float f = exp2f(m - ref);
    const float pr = seen ? exp2f(x - ref) : 0.f;
    m = mn;
    l = l * f + pr;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] *= f;
    for (int t = 0; t < 32; ++t) {
      const float pt = __shfl_sync(0xffffffffu, pr, t);
      const char* vt = reinterpret_cast<const char*>(
          __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(vrow), t));
      if (!vt || pt == 0.f) continue;
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const uint32_t x2 = *reinterpret_cast<const uint32_t*>(vt + 2 * (lane * E + e));
        o[e] = fmaf(pt, T::lo(x2), o[e]);
        o[e + 1] = fmaf(pt, T::hi(x2), o[e + 1]);
      }
    }
  }
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
  const bool any = !(l <= 0.f);
  const float inv = any ? 1.f / l : 0.f;
  char* out = p.out + 2 * (row * D + lane * E);
#pragma unroll
  for (int e = 0; e < E; e += 2)
    *reinterpret_cast<uint32_t*>(out + 2 * e) =
        any ? T::pack(o[e] * inv, o[e + 1] * inv) : 0u;
  if (p.lse && lane == 0)
    p.lse[row] = any ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
  bits = __reduce_or_sync(0xffffffffu, bits);
  if (bits && lane == 0) atomicOr(p.err, bits);
}

template <class T>
cudaError_t attn_t(const AttnParams& p, int D, cudaStream_t s) {
  const long long rows = static_cast<long long>(p.nodes.B) * p.nodes.N * p.Hq;
  const unsigned grid = static_cast<unsigned>((rows + kRows - 1) / kRows);
  if (D == 128) attn_kernel<T, 128><<<grid, 32 * kRows, 0, s>>>(p);
  else attn_kernel<T, 64><<<grid, 32 * kRows, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_tree_attention(const AttnParams& p, int dtype, int D, cudaStream_t s) {
  return dtype == Bf16::kId ? attn_t<Bf16>(p, D, s) : attn_t<F16>(p, D, s);
}

}  // namespace ssd

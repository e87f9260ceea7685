// ssd_chunk.cu -- attention of chunks of new tokens over the paged cache.
//
// Token i of a sequence lies in slot p = ctx + i and sees the slots s <= p with
// s > p - window (window 0: all of them) or s < sinks:
//     out = sum_s softmax_s(c q k_s) v_s,   lse = log sum_s exp(c q k_s).
// A warp per (token, query head), a slot at a time, lanes over the head's entries.
#include <math.h>

#include "ssd_device.cuh"
#include "ssd_kv.cuh"

namespace ssd {
namespace {

constexpr int kWarps = 8;

template <class T, int D>
__global__ void __launch_bounds__(32 * kWarps) chunk_kernel(const __grid_constant__ ChunkParams p) {
  constexpr int E = D / 64;  // pairs of entries a lane
  const int lane = threadIdx.x & 31;
  const long long at = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const int N = p.nodes.N, Hq = p.Hq;
  if (at >= static_cast<long long>(p.nodes.B) * N * Hq) return;
  const int hq = static_cast<int>(at % Hq), i = static_cast<int>(at / Hq % N), b = static_cast<int>(at / Hq / N);
  const int h = hq / p.G;
  const int ctx = p.nodes.ctx_len[b], nn = p.nodes.n_nodes ? p.nodes.n_nodes[b] : N;
  bool bad;
  const int n = seq_nodes(ctx, nn, N, p.kv.width, p.kv.ps, bad);
  if (bad && lane == 0) atomicOr(p.err, kErrBadLength);
  float o[2 * E], m = -INFINITY, l = 0.f;
#pragma unroll
  for (int e = 0; e < 2 * E; ++e) o[e] = 0.f;
  if (i < n) {
    const int pos = ctx + i;
    const uint32_t* qr =
        reinterpret_cast<const uint32_t*>(p.q + 2 * (b * p.q_b + i * p.q_n + hq * p.q_h)) + lane * E;
    float q[2 * E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      q[2 * e] = T::lo(qr[e]);
      q[2 * e + 1] = T::hi(qr[e]);
    }
    const int* row = p.kv.table + b * p.kv.table_stride;
    for (int s = 0; s <= pos; ++s) {
      if (p.window && s >= p.sinks && s <= pos - p.window) {
        s = pos - p.window;
        continue;
      }
      int page, off;
      const bool ok = kv_slot(row, p.kv.width, p.kv.pages, p.kv.ps, s, page, off);
      if (!ok && lane == 0) atomicOr(p.err, kErrBadPage);
      float x = 0.f, v[2 * E];
      const uint32_t* kr = reinterpret_cast<const uint32_t*>(
                               p.kv.k + 2 * (page * p.kv.k_page + off * p.kv.k_slot + h * p.kv.k_head)) + lane * E;
      const uint32_t* vr = reinterpret_cast<const uint32_t*>(
                               p.kv.v + 2 * (page * p.kv.v_page + off * p.kv.v_slot + h * p.kv.v_head)) + lane * E;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        const uint32_t k = ok ? kr[e] : 0u, w = ok ? vr[e] : 0u;
        x = fmaf(q[2 * e], T::lo(k), x);
        x = fmaf(q[2 * e + 1], T::hi(k), x);
        v[2 * e] = T::lo(w);
        v[2 * e + 1] = T::hi(w);
      }
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
      x = p.scale == 0.f ? 0.f : x * p.scale;
      const float mn = fmaxf(m, x);
      if (x == -INFINITY) continue;
      // (2^-40: sums of values near the largest stay finite)
      const float f = m == mn ? 1.f : expf(m - mn), w = 0x1p-40f * (x == mn ? 1.f : expf(x - mn));
      l = l * f + w;
#pragma unroll
      for (int e = 0; e < 2 * E; ++e) o[e] = fmaf(w, v[e], o[e] * f);
      m = mn;
    }
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const long long r = (static_cast<long long>(b) * N + i) * Hq + hq;
  uint32_t* out = reinterpret_cast<uint32_t*>(p.out + 2 * r * D) + lane * E;
#pragma unroll
  for (int e = 0; e < E; ++e) out[e] = T::pack(o[2 * e] * inv, o[2 * e + 1] * inv);
  if (p.lse && lane == 0) p.lse[r] = l == 0.f ? -INFINITY : m + logf(l * 0x1p40f);
}

template <class T>
cudaError_t launch_t(const ChunkParams& p, int D, cudaStream_t s) {
  const long long rows = static_cast<long long>(p.nodes.B) * p.nodes.N * p.Hq;
  const unsigned grid = static_cast<unsigned>((rows + kWarps - 1) / kWarps);
  if (D == 128) chunk_kernel<T, 128><<<grid, 32 * kWarps, 0, s>>>(p);
  else chunk_kernel<T, 64><<<grid, 32 * kWarps, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

size_t chunk_attention_bytes(int, int, int) { return 256; }

cudaError_t launch_chunk_attention(const ChunkParams& p, int dtype, int D, cudaStream_t s) {
  return dtype == Bf16::kId ? launch_t<Bf16>(p, D, s) : launch_t<F16>(p, D, s);
}

}  // namespace ssd

// ssd_weights.cu -- attention weights added up for every slot of the paged cache:
//     w[h, s] = decay w[h, s] + sum over (token, query head of the group) that see s
//               of exp(c q k_s - lse).
// A warp per (sequence, head, slot), a token at a time, lanes over the head's entries.
#include <math.h>

#include "ssd_device.cuh"
#include "ssd_kv.cuh"

namespace ssd {
namespace {

constexpr int kWarps = 8;

template <class T, int D>
__global__ void __launch_bounds__(32 * kWarps) weights_kernel(const __grid_constant__ WeightsParams p) {
  constexpr int E = D / 64;
  const int lane = threadIdx.x & 31;
  const int s = blockIdx.x * kWarps + (threadIdx.x >> 5), h = blockIdx.y, N = p.nodes.N;
  for (int b = blockIdx.z; b < p.nodes.B; b += gridDim.z) {
    const int ctx = p.nodes.ctx_len[b], nn = p.nodes.n_nodes ? p.nodes.n_nodes[b] : N;
    bool bad;
    int n = seq_nodes(ctx, nn, N, p.kv.width, p.kv.ps, bad);
    if (!bad && n > 0 && ctx + n > p.w_len) {
      bad = true;
      n = 0;
    }
    if (bad && s == 0 && h == 0 && lane == 0) atomicOr(p.err, kErrBadLength);
    if (n == 0 || s >= ctx + n) continue;
    int page, off;
    const bool ok = kv_slot(p.kv.table + b * p.kv.table_stride, p.kv.width, p.kv.pages, p.kv.ps, s, page, off);
    if (!ok && lane == 0) atomicOr(p.err, kErrBadPage);
    const uint32_t* kr = reinterpret_cast<const uint32_t*>(
                             p.kv.k + 2 * (page * p.kv.k_page + off * p.kv.k_slot + h * p.kv.k_head)) + lane * E;
    float k[2 * E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const uint32_t w = ok ? kr[e] : 0u;
      k[2 * e] = T::lo(w);
      k[2 * e + 1] = T::hi(w);
    }
    float sum = 0.f;
    for (int i = max(0, s - ctx); i < n; ++i) {
      if (p.window && s >= p.sinks && s <= ctx + i - p.window) break;
      for (int g = 0; g < p.G; ++g) {
        const int hq = h * p.G + g;
        const uint32_t* qr =
            reinterpret_cast<const uint32_t*>(p.q + 2 * (b * p.q_b + i * p.q_n + hq * p.q_h)) + lane * E;
        float x = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
          x = fmaf(T::lo(qr[e]), k[2 * e], x);
          x = fmaf(T::hi(qr[e]), k[2 * e + 1], x);
        }
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
        const float lse = p.lse[(static_cast<long long>(b) * N + i) * p.Hq + hq];
        if (lse != -INFINITY) sum += expf((p.scale == 0.f ? 0.f : x * p.scale) - lse);
      }
    }
    if (lane == 0) {
      float* w = p.weights + b * p.w_b + h * p.w_h + s;
      *w = p.decay == 0.f ? sum : fmaf(p.decay, *w, sum);
    }
  }
}

template <class T>
cudaError_t launch_t(const WeightsParams& p, int D, cudaStream_t s) {
  const dim3 grid((p.w_len + kWarps - 1) / kWarps, p.kv.Hkv, p.nodes.B < 65535 ? p.nodes.B : 65535);
  if (D == 128) weights_kernel<T, 128><<<grid, 32 * kWarps, 0, s>>>(p);
  else weights_kernel<T, 64><<<grid, 32 * kWarps, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv_weights(const WeightsParams& p, int dtype, int D, cudaStream_t s) {
  return dtype == Bf16::kId ? launch_t<Bf16>(p, D, s) : launch_t<F16>(p, D, s);
}

}  // namespace ssd

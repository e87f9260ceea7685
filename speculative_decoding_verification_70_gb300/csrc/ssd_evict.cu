// ssd_evict.cu -- a paged cache cut down to a budget of slots a sequence, each
// key/value head keeping its heaviest ones.
//
// evict_pick_kernel, a CTA per (layer, sequence, head): the first `sinks` slots
// and the last `recent` stay; of those between, the weight of the last one that
// stays is found by its bits (histograms of 8 bits a pass), then one pass in slot
// order writes the list of the kept slots and their weights.
// evict_move_kernel moves the rows: row r of the list goes to slot r.  A source
// lies at or behind its target, so that blocks of rows taken in order, all of a
// block's loads before its stores, read every row before it is overwritten.
#include "ssd_device.cuh"
#include "ssd_kv.cuh"

namespace ssd {
namespace {

constexpr int kPickThreads = 512;
constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 8;  // rows in flight a thread

// Ordered as the weights are; NaN below all of them.
__device__ __forceinline__ uint32_t key_of(float w) {
  if (w != w) return 0;
  const int b = __float_as_int(w + 0.f);  // (-0 counts as 0)
  return static_cast<uint32_t>(b) ^ (b < 0 ? 0xffffffffu : 0x80000000u);
}

struct PickSmem {
  int hist[256];
  int warp[kPickThreads / 32];
  int bin, above;
};

// Exclusive sum of v over the CTA; all: the total.
__device__ __forceinline__ int block_before(int v, int* warp, int& all) {
  const int lane = threadIdx.x & 31;
  int inc = v;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, inc, d);
    if (lane >= d) inc += o;
  }
  __syncthreads();
  if (lane == 31) warp[threadIdx.x >> 5] = inc;
  __syncthreads();
  int before = inc - v;
  all = 0;
#pragma unroll
  for (int i = 0; i < kPickThreads / 32; ++i) {
    if (i < static_cast<int>(threadIdx.x >> 5)) before += warp[i];
    all += warp[i];
  }
  return before;
}

__global__ void __launch_bounds__(kPickThreads) evict_pick_kernel(const __grid_constant__ EvictParams p) {
  __shared__ PickSmem sm;
  const int tid = threadIdx.x;
  const int H = p.kv.Hkv, h = blockIdx.x % H, b = blockIdx.x / H % p.B, layer = blockIdx.x / H / p.B;
  const int ctx = p.ctx_len[b], C = p.budget;
  const bool bad = ctx < 0 || ctx > p.w_len || ctx > static_cast<long long>(p.kv.width) * p.kv.ps;
  int* kept = p.kept + static_cast<long long>(blockIdx.x) * C;
  if (tid == 0 && h == 0 && layer == 0) {
    p.new_len[b] = bad || ctx < C ? ctx : C;
    if (bad) atomicOr(p.err, kErrBadLength);
  }
  if (bad) {
    for (int r = tid; r < C; r += kPickThreads) kept[r] = -1;
    return;
  }
  const float* w = p.weights + layer * p.w_layer + b * p.w_b + h * p.w_h;
  float* wo = p.w_out ? p.w_out + layer * p.wo_layer + b * p.wo_b + h * p.wo_h : nullptr;
  // the slots that compete, and how many of them stay
  const int lo = ctx <= C ? ctx : p.sinks, hi = ctx <= C ? ctx : ctx - p.recent;
  uint32_t want = 0, known = 0;  // the last one's key as far as it is known
  int need = ctx <= C ? 0 : C - p.sinks - p.recent;
  bool none = need == 0;
  for (int shift = 24; shift >= 0 && !none; shift -= 8) {
    if (tid < 256) sm.hist[tid] = 0;
    __syncthreads();
    for (int s = lo + tid; s < hi; s += kPickThreads) {
      const uint32_t k = key_of(w[s]);
      if ((k & known) == want) atomicAdd(&sm.hist[(k >> shift) & 255], 1);
    }
    __syncthreads();
    const int mine = tid < 256 ? sm.hist[255 - tid] : 0;
    int all;
    const int before = block_before(mine, sm.warp, all);
    if (tid < 256 && before < need && need <= before + mine) {
      sm.bin = 255 - tid;
      sm.above = before;
    }
    __syncthreads();
    want |= static_cast<uint32_t>(sm.bin) << shift;
    known |= 255u << shift;
    need -= sm.above;  // those of the bin that stay
  }
  int out = 0, equal = 0;
  for (int s0 = 0; s0 < ctx; s0 += kPickThreads) {
    const int s = s0 + tid;
    const float v = s < ctx ? w[s] : 0.f;
    const bool middle = s >= lo && s < hi;
    const uint32_t k = key_of(v);
    const bool eq = middle && !none && k == want;
    int all;
    const int rank = equal + block_before(eq, sm.warp, all);
    equal += all;
    const bool stay = s < ctx && (!middle || (!none && (k > want || (eq && rank < need))));
    const int at = out + block_before(stay, sm.warp, all);
    if (stay) {
      kept[at] = s;
      if (wo) wo[at] = v;  // (at <= s, and every slot up to this block's end has been read)
    }
    out += all;
  }
  for (int r = out + tid; r < C; r += kPickThreads) kept[r] = -1;
  if (wo)
    for (int r = out + tid; r < p.w_len; r += kPickThreads) wo[r] = 0.f;
}

__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const __grid_constant__ EvictParams p) {
  const int tid = threadIdx.x;
  const int H = p.kv.Hkv, h = blockIdx.x % H, b = blockIdx.x / H % p.B, layer = blockIdx.x / H / p.B;
  const int ctx = p.ctx_len[b], C = p.budget;
  if (ctx <= C || ctx > p.w_len || ctx > static_cast<long long>(p.kv.width) * p.kv.ps) return;
  const int* kept = p.kept + static_cast<long long>(blockIdx.x) * C;
  const int* table = p.kv.table + b * p.kv.table_stride;
  const int per = p.D / 8, side = kMoveThreads / per;  // rows side by side
  const int col = tid % per, r0 = tid / per;
  char* base = blockIdx.y ? p.kv.v + 2 * (layer * p.v_layer + h * p.kv.v_head + col * 8)
                          : p.kv.k + 2 * (layer * p.k_layer + h * p.kv.k_head + col * 8);
  const long long pg = blockIdx.y ? p.kv.v_page : p.kv.k_page, sl = blockIdx.y ? p.kv.v_slot : p.kv.k_slot;
  for (int at = 0; at < C; at += side * kMoveRows) {
    uint4 x[kMoveRows];
    char* to[kMoveRows];
#pragma unroll
    for (int u = 0; u < kMoveRows; ++u) {
      const int r = at + u * side + r0;
      to[u] = nullptr;
      if (r >= C) continue;
      const int s = kept[r];
      if (s == r) continue;
      int sp, so, dp, d_o;
      const bool a = kv_slot(table, p.kv.width, p.kv.pages, p.kv.ps, s, sp, so);
      const bool c = kv_slot(table, p.kv.width, p.kv.pages, p.kv.ps, r, dp, d_o);
      if (!a || !c) {
        atomicOr(p.err, kErrBadPage);
        continue;
      }
      x[u] = *reinterpret_cast<const uint4*>(base + 2 * (sp * pg + so * sl));
      to[u] = base + 2 * (dp * pg + d_o * sl);
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kMoveRows; ++u)
      if (to[u]) *reinterpret_cast<uint4*>(to[u]) = x[u];
  }
}

}  // namespace

cudaError_t launch_kv_evict(const EvictParams& p, cudaStream_t s) {
  const unsigned units = static_cast<unsigned>(p.layers) * p.B * p.kv.Hkv;
  evict_pick_kernel<<<units, kPickThreads, 0, s>>>(p);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  evict_move_kernel<<<dim3(units, 2), kMoveThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace ssd

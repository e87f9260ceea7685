// ssd_evict.cu -- a paged cache cut down to a budget of slots a sequence, each
// key/value head keeping its heaviest ones.
//
// evict_pick_kernel, a cluster of CTAs per (layer, sequence, head), a segment of the slots
// each: the first `sinks` slots and the last `recent` stay; of those between, the weight
// of the last one that stays is found by its bits (11 a pass, a histogram of them summed
// over the cluster; done as soon as all of a bin stay), then the stays of the segments
// before are added up and the list of the kept slots is written in slot order.
// evict_move_kernel moves rows and weights: entry r of the list goes to slot r.  A source
// lies at or behind its target, so that blocks of rows taken in order, all of a block's
// loads before its stores, read every row before it is overwritten.
#include "ssd_device.cuh"
#include "ssd_kv.cuh"

namespace ssd {
namespace {

constexpr int kPickThreads = 512;
constexpr int kPickWarps = kPickThreads / 32;
constexpr int kPerLane = 16;                              // slots of a lane
constexpr int kChunk = kPickThreads * kPerLane;           // slots of a CTA at a time
constexpr int kBins = 2048;
constexpr int kMaxCluster = 8;

// Ordered as the weights are; NaN below all of them.
__device__ __forceinline__ uint32_t key_of(float w) {
  if (w != w) return 0;
  const int b = __float_as_int(w + 0.f);  // (-0 counts as 0)
  return static_cast<uint32_t>(b) ^ (b < 0 ? 0xffffffffu : 0x80000000u);
}

struct PickSmem {
  alignas(16) int hist[kBins];
  int warp[2][kPickWarps];
  int count[2];       // of the segment: those that stay whatever equal ones do, and equal ones
  int bin, above, in_bin;
};

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// The same variable of another CTA of the cluster.
__device__ __forceinline__ uint32_t of_rank(const void* p, int rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(p))), "r"(rank));
  return r;
}
__device__ __forceinline__ int4 far_int4(uint32_t at) {
  int4 v;
  asm volatile("ld.shared::cluster.v4.s32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at));
  return v;
}
__device__ __forceinline__ int far_int(uint32_t at) {
  int v;
  asm volatile("ld.shared::cluster.s32 %0, [%1];" : "=r"(v) : "r"(at));
  return v;
}

// Exclusive sums of a and b over the CTA's warps (each given by its warp), and the totals.
__device__ __forceinline__ void warps_before(PickSmem& sm, int& a, int& b, int& all_a, int& all_b) {
  const int warp = threadIdx.x >> 5;
  __syncthreads();
  if ((threadIdx.x & 31) == 0) {
    sm.warp[0][warp] = a;
    sm.warp[1][warp] = b;
  }
  __syncthreads();
  a = b = all_a = all_b = 0;
#pragma unroll
  for (int i = 0; i < kPickWarps; ++i) {
    const int x = sm.warp[0][i], y = sm.warp[1][i];
    if (i < warp) {
      a += x;
      b += y;
    }
    all_a += x;
    all_b += y;
  }
}

__global__ void __launch_bounds__(kPickThreads) evict_pick_kernel(const __grid_constant__ EvictParams p, int cluster) {
  __shared__ PickSmem sm;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = blockIdx.x % cluster, unit = blockIdx.x / cluster;
  const int H = p.kv.Hkv, h = unit % H, b = unit / H % p.B, layer = unit / H / p.B;
  const int ctx = p.ctx_len[b], C = p.budget;
  const bool bad = ctx < 0 || ctx > p.w_len || ctx > static_cast<long long>(p.kv.width) * p.kv.ps;
  int* kept = p.kept + static_cast<long long>(unit) * C;
  if (tid == 0 && h == 0 && layer == 0 && rank == 0) {
    p.new_len[b] = bad || ctx < C ? ctx : C;
    if (bad) atomicOr(p.err, kErrBadLength);
  }
  // (all CTAs of a cluster take the same way)
  if (bad || ctx <= C) {
    for (int r = rank * kPickThreads + tid; r < C; r += cluster * kPickThreads) kept[r] = !bad && r < ctx ? r : -1;
    return;
  }
  const float* w = p.weights + layer * p.w_layer + b * p.w_b + h * p.w_h;
  // the slots that compete, how many of them stay, and this CTA's segment
  const int lo = p.sinks, hi = ctx - p.recent;
  int need = C - p.sinks - p.recent;
  const int seg = ((ctx + cluster - 1) / cluster + 511) / 512 * 512;
  const int s0 = min(ctx, rank * seg), s1 = min(ctx, s0 + seg);
  const int chunks = max(1, (s1 - s0 + kChunk - 1) / kChunk);
  // a warp's 512 slots of a chunk, 32 side by side
  uint32_t key[kPerLane];
  auto slot_of = [&](int chunk, int k) { return s0 + chunk * kChunk + warp * (32 * kPerLane) + k * 32 + lane; };
  auto load = [&](int chunk) {
#pragma unroll
    for (int k = 0; k < kPerLane; ++k) {
      const int s = slot_of(chunk, k);
      key[k] = s < s1 ? key_of(w[s]) : 0u;
    }
  };
  auto competes = [&](int s) { return s >= lo && s < hi && s < s1; };
  load(0);
  uint32_t want = 0, known = 0;  // the last one's key as far as it is known
  if (need > 0) {  // (fewer than compete)
#pragma unroll 1
    for (int pass = 0; pass < 3; ++pass) {
      const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bits = pass == 2 ? 10 : 11;
      *reinterpret_cast<int4*>(&sm.hist[4 * tid]) = make_int4(0, 0, 0, 0);
      __syncthreads();
#pragma unroll 1
      for (int c = 0; c < chunks; ++c) {
        if (chunks > 1) load(c);
#pragma unroll
        for (int k = 0; k < kPerLane; ++k)
          if (competes(slot_of(c, k)) && (key[k] & known) == want)
            atomicAdd(&sm.hist[(key[k] >> shift) & ((1 << bits) - 1)], 1);
      }
      if (cluster > 1) cluster_sync();
      else __syncthreads();
      // bins from the heaviest on, four a thread
      const int at = kBins - 4 - 4 * tid;
      int4 v = make_int4(0, 0, 0, 0);
      if (cluster > 1) {
        for (int r = 0; r < cluster; ++r) {
          const int4 x = far_int4(of_rank(&sm.hist[at], r));
          v.x += x.x;
          v.y += x.y;
          v.z += x.z;
          v.w += x.w;
        }
      } else {
        v = *reinterpret_cast<const int4*>(&sm.hist[at]);
      }
      const int mine = v.x + v.y + v.z + v.w;
      int inc = mine;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += o;
      }
      int wa = __shfl_sync(0xffffffffu, inc, 31), wb = 0, x, y;
      warps_before(sm, wa, wb, x, y);
      int before = wa + inc - mine;
      if (before < need && need <= before + mine) {
        const int c4[4] = {v.w, v.z, v.y, v.x};
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          if (before < need && need <= before + c4[q]) {
            sm.bin = at + 3 - q;
            sm.above = before;
            sm.in_bin = c4[q];
          }
          before += c4[q];
        }
      }
      __syncthreads();
      want |= static_cast<uint32_t>(sm.bin) << shift;
      known |= ((1u << bits) - 1) << shift;
      need -= sm.above;  // those of the bin that stay
      const bool done = need == sm.in_bin;
      if (cluster > 1) cluster_sync();  // (the histograms have been read)
      else __syncthreads();
      if (done) break;
    }
  }
  const bool none = need == 0;
  // what stays: outside the middle, above the last one's key, or equal and early enough
  auto classes = [&](int c, int k, bool& stay, bool& equal) {
    const int s = slot_of(c, k);
    const bool middle = s >= lo && s < hi;
    const uint32_t x = key[k] & known;
    stay = s < s1 && (!middle || (!none && x > want));
    equal = s < s1 && middle && !none && x == want;
  };
  int gt = 0, eq = 0;  // of the segment, by warp
#pragma unroll 1
  for (int c = 0; c < chunks; ++c) {
    if (chunks > 1) load(c);
#pragma unroll
    for (int k = 0; k < kPerLane; ++k) {
      bool stay, equal;
      classes(c, k, stay, equal);
      gt += __popc(__ballot_sync(0xffffffffu, stay));
      eq += __popc(__ballot_sync(0xffffffffu, equal));
    }
  }
  int all_gt, all_eq, a = gt, e = eq;
  warps_before(sm, a, e, all_gt, all_eq);
  int out = 0, equal_before = 0;
  if (cluster > 1) {
    if (tid == 0) {
      sm.count[0] = all_gt;
      sm.count[1] = all_eq;
    }
    cluster_sync();
    for (int r = 0; r < rank; ++r) {
      const int g = far_int(of_rank(&sm.count[0], r)), q = far_int(of_rank(&sm.count[1], r));
      out += g + min(max(need - equal_before, 0), q);
      equal_before += q;
    }
    cluster_sync();  // (read before a CTA ends)
  }
#pragma unroll 1
  for (int c = 0; c < chunks; ++c) {
    if (chunks > 1) {  // this chunk's counts of the warps before
      load(c);
      gt = eq = 0;
#pragma unroll
      for (int k = 0; k < kPerLane; ++k) {
        bool stay, equal;
        classes(c, k, stay, equal);
        gt += __popc(__ballot_sync(0xffffffffu, stay));
        eq += __popc(__ballot_sync(0xffffffffu, equal));
      }
      a = gt;
      e = eq;
      warps_before(sm, a, e, all_gt, all_eq);
    }
    // equal ones before this warp, and where it writes
    int eb = equal_before + e;
    int at = out + a + min(max(need - equal_before, 0), e);
    const unsigned under = (1u << lane) - 1;
#pragma unroll
    for (int k = 0; k < kPerLane; ++k) {
      bool stay, equal;
      classes(c, k, stay, equal);
      const unsigned em = __ballot_sync(0xffffffffu, equal);
      if (equal && eb + __popc(em & under) < need) stay = true;
      eb += __popc(em);
      const unsigned m = __ballot_sync(0xffffffffu, stay);
      if (stay) kept[at + __popc(m & under)] = slot_of(c, k);
      at += __popc(m);
    }
    out += all_gt + min(max(need - equal_before, 0), all_eq);
    equal_before += all_eq;
  }
}

// ---------------------------------------------------------------------------
// moves
// ---------------------------------------------------------------------------
constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 512;  // most rows of a block

struct MoveSmem {
  long long src[2][kMoveRows], dst[2][kMoveRows];  // bytes from the head's first entry; -1: nothing to move
};

// blockIdx.y: a group of K's columns, of V's, or the weights.  L lanes a row of 16 bytes
// each, U rows in flight a thread.
template <int U>
__global__ void __launch_bounds__(kMoveThreads) evict_move_kernel(const __grid_constant__ EvictParams p, int groups,
                                                                  int L) {
  __shared__ MoveSmem sm;
  const int tid = threadIdx.x, unit = blockIdx.x;
  const int H = p.kv.Hkv, h = unit % H, b = unit / H % p.B, layer = unit / H / p.B;
  const int C = p.budget;
  pdl_wait();
  const int ctx = p.ctx_len[b];
  if (ctx < 0 || ctx > p.w_len || ctx > static_cast<long long>(p.kv.width) * p.kv.ps) return;
  const int* kept = p.kept + static_cast<long long>(unit) * C;
  if (static_cast<int>(blockIdx.y) == 2 * groups) {
    // ---- weights ----
    const float* w = p.weights + layer * p.w_layer + b * p.w_b + h * p.w_h;
    float* wo = p.w_out + layer * p.wo_layer + b * p.wo_b + h * p.wo_h;
    const int n = min(ctx, C);
    constexpr int V = 8;
    for (int at = 0; at < n; at += V * kMoveThreads) {
      float x[V];
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const int r = at + k * kMoveThreads + tid;
        x[k] = r < n ? w[kept[r]] : 0.f;
      }
      __syncthreads();
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const int r = at + k * kMoveThreads + tid;
        if (r < n) wo[r] = x[k];
      }
    }
    for (int r = n + tid; r < p.w_len; r += kMoveThreads) wo[r] = 0.f;
    return;
  }
  if (ctx <= C) return;
  const bool isv = static_cast<int>(blockIdx.y) >= groups;
  const int group = isv ? blockIdx.y - groups : blockIdx.y;
  const int side = kMoveThreads / L, R = side * U;  // rows side by side, of a block
  const int* table = p.kv.table + b * p.kv.table_stride;
  char* base = (isv ? p.kv.v + 2 * (layer * p.v_layer + h * p.kv.v_head)
                    : p.kv.k + 2 * (layer * p.k_layer + h * p.kv.k_head)) + (group * L + tid % L) * 16;
  const long long pg = 2 * (isv ? p.kv.v_page : p.kv.k_page), sl = 2 * (isv ? p.kv.v_slot : p.kv.k_slot);
  auto places = [&](int at, int buf) {
    for (int i = tid; i < R; i += kMoveThreads) {
      const int r = at + i;
      long long from = -1, to = -1;
      if (r < C) {
        const int s = kept[r];
        if (s != r) {
          int sp, so, dp, d_o;
          const bool x = kv_slot(table, p.kv.width, p.kv.pages, p.kv.ps, s, sp, so);
          const bool y = kv_slot(table, p.kv.width, p.kv.pages, p.kv.ps, r, dp, d_o);
          if (x && y) {
            from = sp * pg + so * sl;
            to = dp * pg + d_o * sl;
          } else {
            atomicOr(p.err, kErrBadPage);
          }
        }
      }
      sm.src[buf][i] = from;
      sm.dst[buf][i] = to;
    }
  };
  const int row = tid / L;
  uint4 x[2][U];
  auto load = [&](int buf) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long from = sm.src[buf][u * side + row];
      if (from >= 0) x[buf][u] = *reinterpret_cast<const uint4*>(base + from);
    }
  };
  auto store = [&](int buf) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long to = sm.dst[buf][u * side + row];
      if (to >= 0) *reinterpret_cast<uint4*>(base + to) = x[buf][u];
    }
  };
  // (a block's sources lie behind the targets of the one before, so its loads may pass
  // that one's stores)
  places(0, 0);
  __syncthreads();
  load(0);
#pragma unroll 1
  for (int at = 0; at < C; at += 2 * R) {
    places(at + R, 1);
    __syncthreads();
    load(1);
    store(0);
    if (at + R >= C) break;
    __syncthreads();  // (the places have been read)
    places(at + 2 * R, 0);
    __syncthreads();
    load(0);
    store(1);
    __syncthreads();
  }
}

}  // namespace

cudaError_t launch_kv_evict(const EvictParams& p, cudaStream_t s) {
  const unsigned units = static_cast<unsigned>(p.layers) * p.B * p.kv.Hkv;
  // a cluster as large as gives each SM two CTAs, with at least 2048 slots each
  int cluster = 1;
  while (cluster < kMaxCluster && units * cluster * 2 <= 2 * 152 && p.w_len / (2 * cluster) >= 2048) cluster *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(units * cluster);
  cfg.blockDim = dim3(kPickThreads);
  cfg.stream = s;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeClusterDimension;
  at.val.clusterDim.x = cluster;
  at.val.clusterDim.y = at.val.clusterDim.z = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, evict_pick_kernel, p, cluster);
  if (e != cudaSuccess) return e;
  // groups of columns (64 bytes at least) as give each SM two CTAs
  int groups = 1;
  while (units * 2 * groups < 2 * 152 && p.D * 2 / (2 * groups) >= 64) groups *= 2;
  const int L = p.D / 8 / groups;
  cfg.gridDim = dim3(units, 2 * groups + (p.w_out ? 1 : 0));
  cfg.blockDim = dim3(kMoveThreads);
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  // (256 / L * U rows a block: 512 at most)
  return L >= 4 ? cudaLaunchKernelEx(&cfg, evict_move_kernel<8>, p, groups, L)
                : cudaLaunchKernelEx(&cfg, evict_move_kernel<4>, p, groups, L);
}

}  // namespace ssd

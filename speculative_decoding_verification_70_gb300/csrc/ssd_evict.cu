// ssd_evict.cu -- a paged cache cut down to a budget of slots a sequence, each
// key/value head keeping its heaviest ones.
//
// pick(), a CTA or a cluster of them per (layer, sequence, head), a segment of the slots
// each: the first `sinks` slots and the last `recent` stay; of those between, the weight
// of the last one that stays is found by its bits (11 a pass, a histogram of them summed
// over the cluster; done as soon as all of a bin stay), then the stays of the segments
// before are added up and the list of the kept slots is written in slot order.
// move_rows() and move_weights(): entry r of the list goes to slot r.  A source lies at or
// behind its target, so that blocks of rows taken in order, all of a block's loads before
// its stores, read every row before it is overwritten.
// Nothing is computed in floating point: weights are compared by their bits.
//
// What bounds it: many heads, the bytes moved, read and written (80 layers, 1024 of 4096
// slots kept, 133 us, 5.2 TB/s); few, the passes over the weights, which wait for one
// another (2 layers, 8192 of 100003 slots: 56 us, half of them the choice; 69 with 16 slots
// a lane, read again in every pass, and releasing barriers between the rounds of rows).
#include "ssd_device.cuh"
#include "ssd_kv.cuh"

namespace ssd {
namespace {

constexpr int kEvictThreads = 512;
constexpr int kWarps = kEvictThreads / 32;
constexpr int kBins = 2048;
constexpr int kMaxCluster = 8;

// Ordered as the weights are; NaN below all of them.
__device__ __forceinline__ uint32_t key_of(float w) {
  if (w != w) return 0;
  const int b = __float_as_int(w + 0.f);  // (-0 counts as 0)
  return static_cast<uint32_t>(b) ^ (b < 0 ? 0xffffffffu : 0x80000000u);
}

// Bits 0 .. n - 1, n up to 32.
__device__ __forceinline__ uint32_t first_bits(int n) { return n < 32 ? (1u << n) - 1 : ~0u; }

struct PickSmem {
  alignas(16) int hist[kBins], tot[kBins];  // of the CTA; of the cluster (a share of the bins a CTA)
  int warp[2][kWarps];
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
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  __syncthreads();
  if (lane == 0) {
    sm.warp[0][warp] = a;
    sm.warp[1][warp] = b;
  }
  __syncthreads();
  int x = lane < kWarps ? sm.warp[0][lane] : 0, y = lane < kWarps ? sm.warp[1][lane] : 0;
#pragma unroll
  for (int d = 1; d < kWarps; d <<= 1) {
    const int ox = __shfl_up_sync(0xffffffffu, x, d), oy = __shfl_up_sync(0xffffffffu, y, d);
    if (lane >= d) {
      x += ox;
      y += oy;
    }
  }
  all_a = __shfl_sync(0xffffffffu, x, kWarps - 1);
  all_b = __shfl_sync(0xffffffffu, y, kWarps - 1);
  a = __shfl_sync(0xffffffffu, x, (warp + 31) & 31);
  b = __shfl_sync(0xffffffffu, y, (warp + 31) & 31);
  if (warp == 0) a = b = 0;
}

// By all threads of a cluster; the CTA is number `rank` of it.  PER: most slots of a lane at
// a time (a segment above 512 of them is read again for every pass).
template <int PER>
__device__ __forceinline__ void pick(const EvictParams& p, PickSmem& sm, int unit, int rank, int cluster) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
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
    for (int r = rank * kEvictThreads + tid; r < C; r += cluster * kEvictThreads) kept[r] = !bad && r < ctx ? r : -1;
    return;
  }
  const float* w = p.weights + layer * p.w_layer + b * p.w_b + h * p.w_h;
  // the slots that compete, how many of them stay, and this CTA's segment
  const int lo = p.sinks, hi = ctx - p.recent;
  int need = C - p.sinks - p.recent;
  const int seg = ((ctx + cluster - 1) / cluster + 31) / 32 * 32;
  const int s0 = min(ctx, rank * seg), s1 = min(ctx, s0 + seg);
  // slots of a lane at a time: all, or PER.  A warp's lie 32 side by side.
  const int pl = min(PER, max(1, (s1 - s0 + kEvictThreads - 1) / kEvictThreads));
  const int chunk = pl * kEvictThreads, chunks = max(1, (s1 - s0 + chunk - 1) / chunk);
  uint32_t key[PER], comp = 0;  // keys, and which of them compete
  auto slot_of = [&](int c, int k) { return s0 + c * chunk + (warp * pl + k) * 32 + lane; };
  auto load = [&](int c) {
    // (without a branch, so that all loads are on their way at once)
    const int first = slot_of(c, 0), count = min(pl, (s1 - first + 31) / 32);
    float x[PER];
#pragma unroll
    for (int k = 0; k < PER; ++k) x[k] = k < count ? w[first + 32 * k] : 0.f;
#pragma unroll
    for (int k = 0; k < PER; ++k) key[k] = key_of(x[k]);
    // those from lo to hi - 1
    const int from = min(max((lo - first + 31) >> 5, 0), 32), to = min(max((min(hi, s1) - first + 31) >> 5, 0), pl);
    comp = first_bits(to) & ~first_bits(from);
  };
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
        for (int k = 0; k < PER; ++k) {
          if (k >= pl) break;
          if (((comp >> k) & 1) && (key[k] & known) == want)
            atomicAdd(&sm.hist[(key[k] >> shift) & ((1 << bits) - 1)], 1);
        }
      }
      if (cluster > 1) cluster_sync();
      else __syncthreads();
      // bins from the heaviest on, four a thread.  (A cluster's CTAs add up a share of the
      // bins each: with every CTA reading all histograms, 16 of 8 KB took 13 us.)
      const int at = kBins - 4 - 4 * tid;
      int4 v;
      if (cluster > 1) {
        const int share = kBins / cluster;
        for (int i = rank * share + tid; i < (rank + 1) * share; i += kEvictThreads) {
          int x = 0;
#pragma unroll
          for (int r = 0; r < kMaxCluster; ++r)
            if (r < cluster) x += far_int(of_rank(&sm.hist[i], r));
          sm.tot[i] = x;
        }
        cluster_sync();
        v = far_int4(of_rank(&sm.tot[at], at / share));
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
      __syncthreads();
      if (done) break;
    }
  }
  const bool none = need == 0;
  // what stays of a lane's slots: outside the middle, or above the last one's key; and
  // what is equal to it
  uint32_t stays = 0, equals = 0;
  auto classes = [&](int c) {
    stays = equals = 0;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      if (k >= pl) break;
      const uint32_t x = key[k] & known;
      stays |= static_cast<uint32_t>(x > want) << k;
      equals |= static_cast<uint32_t>(x == want) << k;
    }
    if (none) stays = equals = 0;
    // slots of the segment that do not compete
    const int there = min(pl, max(0, (s1 - slot_of(c, 0) + 31) / 32));
    stays = (stays & comp) | (first_bits(there) & ~comp);
    equals &= comp;
  };
  int gt = 0, eq = 0;  // of the segment, by warp
#pragma unroll 1
  for (int c = 0; c < chunks; ++c) {
    if (chunks > 1) load(c);
    classes(c);
    gt += __reduce_add_sync(0xffffffffu, __popc(stays));
    eq += __reduce_add_sync(0xffffffffu, __popc(equals));
  }
  int all_gt, all_eq, a = gt, e = eq;
  warps_before(sm, a, e, all_gt, all_eq);
  int out = 0, equal_before = 0;
  if (cluster > 1) {
    if (tid == 0) {
      sm.count[0] = all_gt;
      sm.count[1] = all_eq;
    }
    cluster_sync();  // (and the histograms' sums have been read)
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
      classes(c);
      a = __reduce_add_sync(0xffffffffu, __popc(stays));
      e = __reduce_add_sync(0xffffffffu, __popc(equals));
      warps_before(sm, a, e, all_gt, all_eq);
    }
    // equal ones before this warp, and where it writes
    int eb = equal_before + e;
    int at = out + a + min(max(need - equal_before, 0), e);
    const unsigned under = (1u << lane) - 1;
#pragma unroll
    for (int k = 0; k < PER; ++k) {
      if (k >= pl) break;
      const bool equal = (equals >> k) & 1;
      bool stay = (stays >> k) & 1;
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
constexpr int kMoveBytes = 32768;                // of a CTA's rows at a time
constexpr int kMoveRows = kMoveBytes / 128;      // at most

struct MoveSmem {
  uint4 rows[2][kMoveBytes / 16];
  long long src[2][kMoveRows], dst[2][kMoveRows];  // bytes from the head's first entry; -1: nothing to move
};

// A cluster per (unit, K or V; or the weights), which takes its rows in rounds, a CTA
// kMoveBytes of them: on their way into shared memory while the places of the next round
// are found, and out again once every CTA of the cluster has its own, beside the next
// round's loads (whose sources lie behind this round's targets).
// (The cluster's barrier is relaxed: it orders copies that have ended before other CTAs'
// writes, and no values pass between CTAs.  The places of the next round pass between a
// CTA's threads, by its own barrier.)
__device__ __forceinline__ void round_sync(int cluster) {
  __syncthreads();
  if (cluster > 1)
    asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

__device__ __forceinline__ bool in_range(const EvictParams& p, int ctx) {
  return ctx >= 0 && ctx <= p.w_len && ctx <= static_cast<long long>(p.kv.width) * p.kv.ps;
}

__device__ __forceinline__ void move_weights(const EvictParams& p, int unit, int rank, int cluster) {
  const int tid = threadIdx.x, H = p.kv.Hkv, h = unit % H, b = unit / H % p.B, layer = unit / H / p.B, C = p.budget;
  const int ctx = p.ctx_len[b];
  if (!in_range(p, ctx)) return;
  const int* kept = p.kept + static_cast<long long>(unit) * C;
  {
    const float* w = p.weights + layer * p.w_layer + b * p.w_b + h * p.w_h;
    float* wo = p.w_out + layer * p.wo_layer + b * p.wo_b + h * p.wo_h;
    const int n = min(ctx, C);
    constexpr int V = 4;
#pragma unroll 1
    for (int at = rank * V * kEvictThreads; at - rank * V * kEvictThreads < n; at += cluster * V * kEvictThreads) {
      float x[V];
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const int r = at + k * kEvictThreads + tid;
        x[k] = r < n ? w[kept[r]] : 0.f;
      }
      if (cluster > 1) cluster_sync();  // (released: loads to registers may still be on their way)
      else __syncthreads();
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const int r = at + k * kEvictThreads + tid;
        if (r < n) wo[r] = x[k];
      }
    }
    for (int r = n + rank * kEvictThreads + tid; r < p.w_len; r += cluster * kEvictThreads) wo[r] = 0.f;
  }
}

__device__ __forceinline__ void move_rows(const EvictParams& p, MoveSmem& sm, int unit, int rank, int cluster, bool isv) {
  constexpr int U = kMoveBytes / 16 / kEvictThreads;
  const int tid = threadIdx.x, H = p.kv.Hkv, h = unit % H, b = unit / H % p.B, layer = unit / H / p.B, C = p.budget;
  const int ctx = p.ctx_len[b];
  if (!in_range(p, ctx) || ctx <= C) return;
  const int* kept = p.kept + static_cast<long long>(unit) * C;
  const int per = p.D / 8, rows = kEvictThreads * U / per;  // 16-byte pieces of a row; rows of a CTA and round
  const int* table = p.kv.table + b * p.kv.table_stride;
  char* base = isv ? p.kv.v + 2 * (layer * p.v_layer + h * p.kv.v_head) : p.kv.k + 2 * (layer * p.k_layer + h * p.kv.k_head);
  const long long pg = 2 * (isv ? p.kv.v_page : p.kv.k_page), sl = 2 * (isv ? p.kv.v_slot : p.kv.k_slot);
  auto places = [&](int round, int buf) {
    if (tid >= rows) return;
    const int r = (round * cluster + rank) * rows + tid;
    long long from = -1, to = -1;
    const int s = r < C ? kept[r] : r;
    if (s != r) {
      const int fp = table[s / p.kv.ps], tp = table[r / p.kv.ps];
      if (static_cast<unsigned>(fp) < static_cast<unsigned>(p.kv.pages) &&
          static_cast<unsigned>(tp) < static_cast<unsigned>(p.kv.pages)) {
        from = fp * pg + s % p.kv.ps * sl;
        to = tp * pg + r % p.kv.ps * sl;
      } else {
        atomicOr(p.err, kErrBadPage);
      }
    }
    sm.src[buf][tid] = from;
    sm.dst[buf][tid] = to;
  };
  const int col = tid % per, row = tid / per, side = kEvictThreads / per;
  auto load = [&](int buf) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const long long from = sm.src[buf][u * side + row];
      if (from >= 0)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(static_cast<uint32_t>(
                         __cvta_generic_to_shared(&sm.rows[buf][u * kEvictThreads + tid]))),
                     "l"(base + from + col * 16)
                     : "memory");
    }
  };
  const int rounds = (C + cluster * rows - 1) / (cluster * rows);
  __syncthreads();
  places(0, 0);
  __syncthreads();
  load(0);
#pragma unroll 1
  for (int i = 0; i < rounds; ++i) {
    const int buf = i & 1;
    if (i + 1 < rounds) places(i + 1, buf ^ 1);
    asm volatile("cp.async.wait_all;" ::: "memory");
    round_sync(cluster);
    if (i + 1 < rounds) load(buf ^ 1);
#pragma unroll
    for (int u = 0; u < U; ++u) {  // (what this thread has brought)
      const long long to = sm.dst[buf][u * side + row];
      if (to >= 0) *reinterpret_cast<uint4*>(base + to + col * 16) = sm.rows[buf][u * kEvictThreads + tid];
    }
    __syncthreads();  // (the places have been read)
  }
}

// Few units: clusters that pick, then clusters that move (blockIdx.y: K, V, the weights).
__global__ void __launch_bounds__(kEvictThreads) evict_pick_kernel(const __grid_constant__ EvictParams p, int cluster) {
  __shared__ PickSmem sm;
  pick<32>(p, sm, blockIdx.x / cluster, blockIdx.x % cluster, cluster);
}
__global__ void __launch_bounds__(kEvictThreads) evict_move_kernel(const __grid_constant__ EvictParams p, int cluster) {
  extern __shared__ __align__(16) char dyn[];
  const int unit = blockIdx.x / cluster, rank = blockIdx.x % cluster;
  pdl_wait();
  if (blockIdx.y == 2) move_weights(p, unit, rank, cluster);
  else move_rows(p, *reinterpret_cast<MoveSmem*>(dyn), unit, rank, cluster, blockIdx.y == 1);
}
// Many units: a CTA each, so that one's choice runs beside others' moves.
__global__ void __launch_bounds__(kEvictThreads, 3) evict_kernel(const __grid_constant__ EvictParams p) {
  extern __shared__ __align__(16) char dyn[];
  MoveSmem& sm = *reinterpret_cast<MoveSmem*>(dyn);
  pick<16>(p, *reinterpret_cast<PickSmem*>(dyn), blockIdx.x, 0, 1);
  __syncthreads();
  move_rows(p, sm, blockIdx.x, 0, 1, false);
  move_rows(p, sm, blockIdx.x, 0, 1, true);
  if (p.w_out) move_weights(p, blockIdx.x, 0, 1);
}

}  // namespace

cudaError_t launch_kv_evict(const EvictParams& p, cudaStream_t s) {
  const unsigned units = static_cast<unsigned>(p.layers) * p.B * p.kv.Hkv;
  // (one kernel against two, budget 1024 of 4096 slots: 128 units 41 us against 34, 304
  // units 65 against 67, 640 units 132 against 130; 16 units of 100000 slots 327 against 69)
  const bool many = units > 152;
  const void* big = many ? reinterpret_cast<const void*>(evict_kernel) : reinterpret_cast<const void*>(evict_move_kernel);
  cudaError_t e = cudaFuncSetAttribute(big, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(MoveSmem));
  if (e != cudaSuccess) return e;
  if (many) {
    evict_kernel<<<units, kEvictThreads, sizeof(MoveSmem), s>>>(p);
    return cudaGetLastError();
  }
  // clusters as large as find an SM a CTA, with at least 2048 slots each (16 units of 100000
  // slots 69 us, without 136; pairs for 128 units of 4096 slots 40 us, without 34)
  int cluster = 1;
  while (cluster < kMaxCluster && units * cluster * 2 <= 152 && p.w_len / (2 * cluster) >= 2048) cluster *= 2;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(units * cluster);
  cfg.blockDim = dim3(kEvictThreads);
  cfg.stream = s;
  cudaLaunchAttribute at[2];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = cluster;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, evict_pick_kernel, p, cluster);
  if (e != cudaSuccess) return e;
  // and as give each SM two of those that move (the 16 units 69 us, without clusters 137)
  int wide = 1;
  while (wide < kMaxCluster && units * 2 * wide * 2 <= 2 * 152) wide *= 2;
  cfg.gridDim = dim3(units * wide, p.w_out ? 3 : 2);
  cfg.dynamicSmemBytes = sizeof(MoveSmem);
  at[0].val.clusterDim.x = wide;
  at[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, evict_move_kernel, p, wide);
}

}  // namespace ssd

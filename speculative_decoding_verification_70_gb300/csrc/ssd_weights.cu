// ssd_weights.cu -- attention weights added up for every slot of the paged cache:
//     w[h, s] = decay w[h, s] + sum over (token, query head of the group) that see s
//               of exp(c q k_s - lse).
//
// With slots on the tensor cores' M axis and the group's (token, head) rows as columns,
//     S^T = K Q^T   [128 slots, up to 128 rows]
// a thread owns a slot: it reads its scores from tensor memory, adds 2^(c' s - lse') over
// the columns in registers, and no sum crosses threads.  An item is two tiles of slots of
// a (sequence, key/value head), kept in shared memory while the blocks of rows that see
// them pass.  One persistent CTA per SM; the batch's blocks are
// numbered and cut into equal ranges by the lengths on the device; an item that is cut
// leaves its sums in the workspace, and weights_join_kernel adds them in range order.
//
// Warps of a CTA: 0 copies the blocks of Q, 2 and 20 the tiles of K, by TMA into rings; 1
// issues the products; 3 brings the columns' -lse; 4..19 four warpgroups for the sums, two
// a tile, which take its blocks in turn.
//
// Scores, exponentials and sums are held in 32 bits; nothing is rounded to fewer.  What
// bounds it: few rows, the bytes of K and of the weights (64 single tokens at 200..8000,
// 64 / 8 heads of 128: 64 us, 4.6 TB/s); many, the exponentials and what stands before and
// behind them in a warp (4 prompts of up to 5500 slots, 32 / 8 heads of 64: 108 us, of which
// the exponentials' pipe alone would want 50).
#include <math.h>

#include "ssd_device.cuh"
#include "ssd_kv.cuh"
#include "ssd_tiles.cuh"

namespace ssd {
namespace {

constexpr int kSumThreads = 672;
constexpr int kMaxCtas = 160;
constexpr int kMaxKeys = 4, kMaxQueries = 4, kBias = 4;  // slots of the rings (of K two, for the tiles of an item)
constexpr float kLog2e = 1.4426950408889634f;

// A CTA's range of blocks, for the joining kernel.
struct alignas(16) Range {
  long long lo;      // first block (its position in cost)
  int t0, used;      // its place in its item; 0: a range without blocks, 2: one that was given up
  int b, p, h, T;    // its item, the item's blocks
};

struct Args : PageTiles {
  NodesView nodes;
  int Hq, Hkv, G;
  int tq, cols;            // tokens and columns of a block
  int NP;                  // pairs of tiles of the longest sequence
  int window, sinks;
  int item_cost;           // what an item's start and end cost, in blocks
  int nk, nq;              // slots of the rings
  float c;                 // |scale| * log2(e)
  int negate, zero;
  const float* lse;
  float decay;
  float* weights;
  long long w_b, w_h;
  int w_len;
  float* part;             // [2 ctas][256]
  Range* ranges;
  unsigned long long per_cta;  // 2^64 / ctas, rounded up
  int* err;
  unsigned wait_us;
  int withheld;
};

struct alignas(16) Misc {
  alignas(16) float bias[kBias][kTile];  // -lse of the columns, in units of log 2
  uint4 none[kBias];                     // columns whose lse is -inf: they add nothing, whatever they score
  uint64_t kfull[2][kMaxKeys], kempty[2][kMaxKeys], qfull[kMaxQueries], qempty[kMaxQueries], bfull[kBias], bempty[kBias];
  uint64_t sfull[2][2], sempty[2][2], done;
  long long left;
  int b0, p0, h0, t0, cost;
  unsigned tmem;
  int abort;
  unsigned wait_us;
  long long scan[2][kSumThreads / 32];
  float other[2][kTile];      // sums of the warpgroups that do not lead
};
static_assert(sizeof(Misc) <= 4 * 1024, "shared memory beside the rings");

__device__ __forceinline__ int tokens_of(const Args& a, int b, int& ctx, bool& bad) {
  const int n = seq_tokens(a, a.nodes, b, ctx, bad);
  if (n > 0 && ctx > a.w_len - n) bad = true;
  return bad ? 0 : n;
}

// A pair of tiles: its slots, and the tokens ia .. ib - 1 that see some of them, in T
// blocks.
struct Item {
  int tiles, first, last, ia, ib, T;
};
__device__ __forceinline__ Item item_of(const Args& a, int ctx, int n, int p) {
  Item x;
  int count;
  tile_slots(a, 2 * p, x.first, count);
  x.last = x.first + count - 1;
  x.tiles = 1;
  if (x.last < ctx + n - 1) {
    int f;
    tile_slots(a, 2 * p + 1, f, count);
    x.last = f + count - 1;
    x.tiles = 2;
  }
  x.last = min(x.last, ctx + n - 1);
  x.ia = max(0, x.first - ctx);
  x.ib = n;
  if (a.window && x.first >= a.sinks)
    x.ib = static_cast<int>(max(0ll, min(static_cast<long long>(n), static_cast<long long>(x.last) + a.window - ctx)));
  x.T = x.ib > x.ia ? (x.ib - x.ia + a.tq - 1) / a.tq : 0;
  return x;
}
// The pair behind p; behind one that nobody sees, the first that the window reaches.
__device__ __forceinline__ int pair_after(const Args& a, int ctx, int p, int T) {
  return T > 0 ? p + 1 : max(p + 1, tile_of(a, max(0, ctx - a.window + 1)) / 2);
}
__device__ __forceinline__ int pairs_of(const Args& a, int ctx, int n) {
  return n > 0 ? tile_of(a, ctx + n - 1) / 2 + 1 : 0;
}

// The pieces of a CTA's range, one item after another.
struct Pieces {
  long long left;
  int w, b, p, h, ctx, n, pairs;
  Item k;
  int t0, end;     // blocks t0 .. end - 1
  bool fresh;
  __device__ __forceinline__ void start(const Args& a, const Misc& sm) {
    left = sm.left;
    w = sm.cost;
    b = sm.b0;
    p = sm.p0;
    h = sm.h0;
    t0 = sm.t0;
    fresh = true;
    if (left > 0) {
      bool bad;
      n = tokens_of(a, b, ctx, bad);
      pairs = pairs_of(a, ctx, n);
      k = item_of(a, ctx, n, p);
    }
  }
  __device__ __forceinline__ bool direct() const { return t0 == 0 && end == k.T; }
  __device__ __forceinline__ bool next(const Args& a) {
    if (!fresh) {
      left -= end - t0 + (end == k.T ? w : 0);
      t0 = 0;
      if (left > 0 && ++h == a.Hkv) {
        h = 0;
        do {
          p = pair_after(a, ctx, p, k.T);
          while (p >= pairs) {
            if (++b >= a.nodes.B) {
              left = 0;
              return false;
            }
            bool bad;
            n = tokens_of(a, b, ctx, bad);
            pairs = pairs_of(a, ctx, n);
            p = 0;
          }
          k = item_of(a, ctx, n, p);
        } while (k.T == 0);
      }
    }
    fresh = false;
    if (left <= 0) return false;
    end = static_cast<int>(min(static_cast<long long>(k.T), t0 + left));
    return true;
  }
};

// The (sequence, pair)s from number `at` on, up to number e; f(pair's item).
template <class F>
__device__ __forceinline__ void each_pair(const Args& a, long long at, long long e, F&& f) {
  int ctx = 0, n = 0, pairs = 0, had = -1;
#pragma unroll 1
  while (at < e) {
    const int b = static_cast<int>(at / a.NP), p = static_cast<int>(at - static_cast<long long>(b) * a.NP);
    if (b != had) {
      bool bad;
      n = tokens_of(a, b, ctx, bad);
      if (bad && p == 0 && blockIdx.x == 0) atomicOr(a.err, kErrBadLength);
      pairs = pairs_of(a, ctx, n);
      had = b;
    }
    if (p >= pairs) {  // the next sequence
      at += a.NP - p;
      continue;
    }
    const Item k = item_of(a, ctx, n, p);
    if (k.T > 0 && !f(b, p, k)) return;
    at += min(pair_after(a, ctx, p, k.T), a.NP) - p;
  }
}

__device__ __forceinline__ uint32_t below(int x) { return x <= 0 ? 0u : x >= 32 ? ~0u : (1u << x) - 1; }

// ---------------------------------------------------------------------------
// sums: a warpgroup a tile, a thread a slot
// ---------------------------------------------------------------------------
// 16 columns' sum.  (A column that the slot does not see is left out behind its bias, which
// may be NaN.)
template <bool MASKED>
__device__ __forceinline__ void add_columns(f32x2 c2, uint32_t (&s)[16], const float* bias, uint32_t seen, f32x2 (&sum)[2]) {
#pragma unroll
  for (int e = 0; e < 16; e += 4) {
    const float4 m = *reinterpret_cast<const float4*>(bias + e);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      float y0, y1;
      up2(fma2(pk2(__uint_as_float(s[e + 2 * q]), __uint_as_float(s[e + 2 * q + 1])), c2, q ? pk2(m.z, m.w) : pk2(m.x, m.y)),
          y0, y1);
      if (MASKED) {
        if (!(seen & (1u << (e + 2 * q)))) y0 = -INFINITY;
        if (!(seen & (2u << (e + 2 * q)))) y1 = -INFINITY;
      }
      sum[q] = add2(sum[q], pk2(ex2_fast(y0), ex2_fast(y1)));
    }
  }
}

// A block's columns, 16 at a time, the next ones on their way meanwhile.
template <bool MASKED, class Read>
__device__ __forceinline__ float block_sum(const Args& a, uint32_t tS, const float* bias, const uint32_t* none, int lo,
                                           int hi, Read&& read) {
  const f32x2 c2 = pk2(a.c, a.c);
  f32x2 sum[2] = {0ull, 0ull};
  uint32_t s0[16], s1[16];
  tm_get16(tS, s0);
#pragma unroll 1
  for (int j = 0; j < a.cols; j += 32) {
    tm_wait_loads();
    tm_tie16(s0);
    tm_get16(tS + j + 16, s1);
    const uint32_t seen = MASKED ? below(hi - j) & ~below(lo - j) & ~none[j / 32] : 0u;
    add_columns<MASKED>(c2, s0, bias + j, seen, sum);
    tm_wait_loads();
    tm_tie16(s1);
    if (j + 32 < a.cols) tm_get16(tS + j + 32, s0);
    else read();
    add_columns<MASKED>(c2, s1, bias + j + 16, seen >> 16, sum);
  }
  float x, y;
  up2(add2(sum[0], sum[1]), x, y);
  return x + y;
}

// Warpgroup `half` of the two of tile w of each item takes every second block.
__device__ __forceinline__ void sum_role(const Args& a, Misc& sm, uint32_t tmem, int w, int half) {
  const int wt = threadIdx.x & 127;
  const uint32_t tS = tmem + (static_cast<uint32_t>(wt & 96) << 16) + (2 * half + w) * 128;
  const int off = row_offset(a, wt);
  int block = 0, item = -1;
  uint32_t ph = 0;  // phase of sfull
  Pieces pc;
  pc.start(a, sm);
#pragma unroll 1
  while (pc.next(a)) {
    ++item;
    const bool mine = w < pc.k.tiles;
    int first = 0, count = 0;
    if (mine) tile_slots(a, 2 * pc.p + w, first, count);
    const int slot = first + off;
    const bool there = mine && off < count && slot < pc.ctx + pc.n;
    // the sums of two warpgroups are joined by the one with the item's first block
    const bool two = pc.end - pc.t0 > 1, leads = (block & 1) == half;
    float* at = a.weights + pc.b * a.w_b + pc.h * a.w_h + slot;
    float old = 0.f;
    if (leads && there && pc.direct() && a.decay != 0.f) old = *at;  // (on its way during the sums)
    // tokens that see the slot: from ts to te - 1
    const int ts = slot - pc.ctx;
    const int te = a.window && slot >= a.sinks
                       ? static_cast<int>(min(static_cast<long long>(pc.k.ib), static_cast<long long>(ts) + a.window))
                       : pc.k.ib;
    float acc = 0.f;
#pragma unroll 1
    for (int t = pc.t0; t < pc.end; ++t, ++block) {
      if ((block & 1) != half) continue;
      const int bs = block % kBias;
      if (mine) bar_wait(&sm.sfull[w][half], ph, sm, a.err);
      bar_wait(&sm.bfull[bs], (block / kBias) & 1, sm, a.err);
      if (mine) {
        ph ^= 1;
        tc_after();
        const int i0 = pc.k.ia + t * a.tq, used = min(a.tq, pc.k.ib - i0);
        int lo = min(max(ts - i0, 0), a.tq), hi = min(max(te - i0, 0), used);
        if (!there) hi = 0;
        auto read = [&]() {
          tc_before();
          bar_arrive(&sm.sempty[w][half]);
        };
        // (columns that are no row, behind the block's, are masked like those that do not see it)
        const uint4 none = sm.none[bs];
        const bool whole = lo == 0 && hi * a.G == a.cols && (none.x | none.y | none.z | none.w) == 0;
        const uint32_t* out = reinterpret_cast<const uint32_t*>(&sm.none[bs]);
        if (__all_sync(0xffffffffu, whole)) acc += block_sum<false>(a, tS, sm.bias[bs], out, 0, 0, read);
        else acc += block_sum<true>(a, tS, sm.bias[bs], out, lo * a.G, hi * a.G, read);
      }
      bar_arrive(&sm.bempty[bs]);
    }
    if (mine && two) {
      if (!leads) sm.other[w][wt] = acc;
      named_sync(1 + w, 256);
      if (leads) acc += sm.other[w][wt];
      named_sync(1 + w, 256);
    }
    // (a wait that gave up: what is there stays)
    if (!there || !leads || *reinterpret_cast<volatile int*>(&sm.abort)) continue;
    if (pc.direct()) *at = a.decay == 0.f ? acc : fmaf(a.decay, old, acc);
    else a.part[(2 * blockIdx.x + (item == 0 ? 0 : 1)) * 256 + w * 128 + wt] = acc;
  }
}

// ---------------------------------------------------------------------------
// copies of K: first (w = 0) or second tiles of items
// ---------------------------------------------------------------------------
template <int D, bool GATHER>
__device__ __forceinline__ void keys_role(const Args& a, Misc& sm, const CUtensorMap& map, uint32_t ring, int w) {
  constexpr int kSlotBytes = D / 64 * kHalf;
  const int lane = threadIdx.x & 31;
  Pieces pc;
  pc.start(a, sm);
  Ring rk = {&map, sm.kfull[w], sm.kempty[w], ring + w * a.nk * kSlotBytes, a.nk, -1, 0};
  bool bad_page = false;
  // an item's tile: the boxes that hold slots, and this lane's page id, on its way
  // while the tile of the item before is copied
  struct Tile {
    int t, h, pl;
    Place id;
  };
  auto lookup = [&](Tile& x) {
    x.t = -1;
    do {
      if (!pc.next(a)) return;
    } while (w >= pc.k.tiles);
    x.t = 2 * pc.p + w;
    x.h = pc.h;
    int first, count;
    tile_slots(a, x.t, first, count);
    x.pl = a.uneven ? 0 : min(a.boxes - 1, (pc.ctx + pc.n - 1 - first) / a.step);
    x.id = box_place<GATHER>(a, a.table + pc.b * a.table_stride, x.t, pc.ctx + pc.n - 1, lane <= x.pl);
  };
  Tile cur, nxt;
  lookup(nxt);
#pragma unroll 1
  while (nxt.t >= 0) {
    cur = nxt;
    lookup(nxt);
    bad_page |= !load_tile<D, GATHER>(a, sm, rk, 0, cur.pl, cur.id, cur.h, a.err, a.withheld);
  }
  // whether somebody sees them
  if (__any_sync(0xffffffffu, bad_page)) {
    bad_page = false;
    pc.start(a, sm);
#pragma unroll 1
    while (pc.next(a)) {
      const int lo = a.window ? max(0, pc.ctx - a.window + 1) : 0;
      if (w < pc.k.tiles)
        bad_page |= bad_box<GATHER>(a, a.table + pc.b * a.table_stride, 2 * pc.p + w, pc.ctx + pc.n - 1, lo, min(a.sinks, lo));
    }
    if (bad_page) atomicOr(a.err, kErrBadPage);
  }
}

// ---------------------------------------------------------------------------
// the kernel
// ---------------------------------------------------------------------------
template <class T, int D, bool GATHER>
__global__ void __launch_bounds__(kSumThreads, 1)
    weights_kernel(const __grid_constant__ CUtensorMap mapq, const __grid_constant__ CUtensorMap mapk,
                   const __grid_constant__ Args a) {
  extern __shared__ __align__(1024) char base[];
  constexpr int HALVES = D / 64;
  constexpr int kSlotBytes = HALVES * kHalf;
  char* ring = base;
  char* Q = ring + 2 * a.nk * kSlotBytes;
  const int qhalf = a.cols * 128, qbytes = qhalf * HALVES;
  Misc& sm = *reinterpret_cast<Misc*>(Q + a.nq * qbytes);
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int C = gridDim.x, B = a.nodes.B;

  if (tid == 0) {
    for (int i = 0; i < 2 * kMaxKeys; ++i) {
      bar_init(&sm.kfull[i / kMaxKeys][i % kMaxKeys], 1);
      bar_init(&sm.kempty[i / kMaxKeys][i % kMaxKeys], 1);
    }
    for (int i = 0; i < kMaxQueries; ++i) {
      bar_init(&sm.qfull[i], 1);
      bar_init(&sm.qempty[i], 1);
    }
    for (int i = 0; i < kBias; ++i) {
      bar_init(&sm.bfull[i], 1);
      bar_init(&sm.bempty[i], 256);
    }
    for (int i = 0; i < 4; ++i) {
      bar_init(&sm.sfull[i >> 1][i & 1], 1);
      bar_init(&sm.sempty[i >> 1][i & 1], 128);
    }
    bar_init(&sm.done, 1);
    sm.abort = 0;
    sm.wait_us = a.wait_us;
    sm.left = 0;
    sm.b0 = sm.p0 = sm.h0 = sm.t0 = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(sptr(&sm.tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (warp == 0 && lane == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(&mapq));
    asm volatile("prefetch.tensormap [%0];" ::"l"(&mapk));
  }
  // ---- this CTA's range ----
  {
    const long long all = static_cast<long long>(B) * a.NP, per = (all + kSumThreads - 1) / kSumThreads;
    const long long f = tid * per, e = min(all, f + per);
    long long mine = 0, pairs = 0;  // blocks of a head, and pairs that have some
    each_pair(a, f, e, [&](int, int, const Item& k) {
      mine += k.T;
      ++pairs;
      return true;
    });
    long long inc = mine, incp = pairs;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long o = __shfl_up_sync(0xffffffffu, inc, d), op = __shfl_up_sync(0xffffffffu, incp, d);
      if (lane >= d) {
        inc += o;
        incp += op;
      }
    }
    if (lane == 31) {
      sm.scan[0][warp] = inc;
      sm.scan[1][warp] = incp;
    }
    __syncthreads();
    long long before = inc - mine, beforep = incp - pairs, blocks = 0, items = 0;
#pragma unroll
    for (int i = 0; i < kSumThreads / 32; ++i) {
      if (i < warp) {
        before += sm.scan[0][i];
        beforep += sm.scan[1][i];
      }
      blocks += sm.scan[0][i];
      items += sm.scan[1][i];
    }
    const long long w = a.item_cost, W = (blocks + w * items) * a.Hkv;
    const long long me = blockIdx.x, lo = __umul64hi(W * me, a.per_cta),
                    hi = me + 1 == C ? W : static_cast<long long>(__umul64hi(W * (me + 1), a.per_cta));
    long long p = (before + w * beforep) * a.Hkv;
    const long long mine_cost = (mine + w * pairs) * a.Hkv;
    if (tid == 0) {
      a.ranges[me].used = 0;
      sm.cost = static_cast<int>(w);
    }
    __syncthreads();
    // the thread whose pairs hold the range's first block (lo may lie behind the blocks of
    // the last item before them)
    if (lo < p + mine_cost && hi > p && p - lo <= w) {
      each_pair(a, f, e, [&](int b, int pair, const Item& k) {
        const long long one = k.T + w, end = p + one * a.Hkv;
        if (lo < end) {
          const unsigned long long d = lo > p ? lo - p : 0;
          int h = static_cast<int>(d / one);
          int t0 = static_cast<int>(d - h * one);
          if (t0 >= k.T) {  // behind the item's blocks: the next item
            ++h;
            t0 = 0;
          }
          const long long from = p + h * one + t0;  // cost position of the first block
          if (h < a.Hkv) {
            if (from < hi) {
              Range r;
              r.lo = from;
              r.t0 = sm.t0 = t0;
              r.used = 1;
              r.b = sm.b0 = b;
              r.p = sm.p0 = pair;
              r.h = sm.h0 = h;
              r.T = k.T;
              a.ranges[me] = r;
              sm.left = hi - from;
            }
            return false;
          }
        }
        p = end;
        return true;
      });
    }
  }
  tc_before();
  __syncthreads();
  tc_after();
  pdl_trigger();
  const uint32_t tmem = __shfl_sync(0xffffffffu, sm.tmem, 0);

  if (warp >= 4 && warp < 20) {
    sum_role(a, sm, tmem, ((warp - 4) >> 2) & 1, (warp - 4) >> 3);
  } else {
    Pieces pc;
    pc.start(a, sm);
    if (warp == 0) {
      // ---- blocks of Q ----
      int slot = -1;
      uint32_t phase = 0;
#pragma unroll 1
      while (pc.next(a)) {
#pragma unroll 1
        for (int t = pc.t0; t < pc.end; ++t) {
          if (++slot == a.nq) {
            slot = 0;
            phase ^= 1;
          }
          const bool ok = bar_await(&sm.qempty[slot], phase ^ 1, sm, a.err) &&
                          !*reinterpret_cast<volatile int*>(&sm.abort);
          if (__all_sync(0xffffffffu, ok) && elect_one()) {
            bar_expect(&sm.qfull[slot], HALVES * a.tq * a.G * 128 + a.withheld);
            // (scale 0: behind the last token, zeros)
            const int i0 = a.zero ? a.nodes.N : pc.k.ia + t * a.tq;
            for (int d = 0; d < HALVES; ++d)
              tma_rows(sptr(Q) + slot * qbytes + d * qhalf, &mapq, d * 64, pc.h * a.G, i0, pc.b, &sm.qfull[slot]);
          }
          __syncwarp();
        }
      }
    } else if (warp == 2 || warp == 20) {
      // ---- first (2) or second (20) tiles of K ----
      const int w = warp == 20;
      keys_role<D, GATHER>(a, sm, mapk, sptr(ring), w);
    } else if (warp == 3) {
      int place[kTile / 32];  // of a column's lse behind the block's first
#pragma unroll
      for (int k = 0; k < kTile / 32; ++k) {
        const int r = lane + 32 * k;
        place[k] = r / a.G * a.Hq + r % a.G;
      }
      // ---- the columns' -lse, loaded two blocks ahead ----
      int t = 0, end = 0, block = 0;
      struct Lse {
        int there;
        float x[kTile / 32];
      };
      auto load = [&](Lse& l) {
        l.there = 0;
        if (++t >= end) {
          if (end < 0 || !pc.next(a)) {
            end = -1;
            t = 0;
            return;
          }
          t = pc.t0;
          end = pc.end;
        }
        l.there = 1;
        const int i0 = pc.k.ia + t * a.tq, rows = min(a.tq, pc.k.ib - i0) * a.G;
        const float* lse = a.lse + (static_cast<long long>(pc.b) * a.nodes.N + i0) * a.Hq + pc.h * a.G;
#pragma unroll
        for (int k = 0; k < kTile / 32; ++k)
          l.x[k] = lane + 32 * k < rows ? __ldg(lse + place[k]) : 0.f;
      };
      Lse l0, l1, l2;
      load(l0);
      load(l1);
#pragma unroll 1
      while (l0.there) {
        load(l2);
        const int bs = block % kBias;
        bar_await(&sm.bempty[bs], ((block / kBias) & 1) ^ 1, sm, a.err);
        uint32_t none[kTile / 32];
#pragma unroll
        for (int k = 0; k < kTile / 32; ++k) {
          none[k] = __ballot_sync(0xffffffffu, l0.x[k] == -INFINITY);
          sm.bias[bs][lane + 32 * k] = -l0.x[k] * kLog2e;
        }
        if (lane == 0) sm.none[bs] = make_uint4(none[0], none[1], none[2], none[3]);
        __syncwarp();
        if (lane == 0) bar_arrive(&sm.bfull[bs]);
        ++block;
        l0 = l1;
        l1 = l2;
      }
    } else if (warp == 1) {
      // ---- products ----
      const uint32_t khalf = a.half / 16, id = instr<T>(a.cols, false, false, a.negate);
      const uint64_t kd0 = operand(sptr(ring), 16, a.group), qd0 = operand(sptr(Q), 16, 1024);
      int qslot = -1, kslot[2] = {-1, -1}, block = 0;
      uint32_t qphase = 0, kphase[2] = {0, 0}, sph = 0;  // (sph: of sempty)
#pragma unroll 1
      while (pc.next(a)) {
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          if (w >= pc.k.tiles) continue;
          if (++kslot[w] == a.nk) {
            kslot[w] = 0;
            kphase[w] ^= 1;
          }
          bar_await(&sm.kfull[w][kslot[w]], kphase[w], sm, a.err);
        }
#pragma unroll 1
        for (int t = pc.t0; t < pc.end; ++t, ++block) {
          if (++qslot == a.nq) {
            qslot = 0;
            qphase ^= 1;
          }
          bar_await(&sm.qfull[qslot], qphase, sm, a.err);
          const uint64_t qd = qd0 + qslot * (qbytes / 16);
#pragma unroll
          for (int w = 0; w < 2; ++w) {
            if (w >= pc.k.tiles) continue;
            const int buf = block & 1, bit = 2 * w + buf;
            bar_await(&sm.sempty[w][buf], ((sph >> bit) & 1) ^ 1, sm, a.err);
            sph ^= 1u << bit;
            tc_after();
            const uint64_t kd = kd0 + (w * a.nk + kslot[w]) * (kSlotBytes / 16);
            if (elect_one()) {
#pragma unroll
              for (int k = 0; k < D / 16; ++k)
                tc_mma(tmem + (2 * buf + w) * 128, kd + (k / 4) * khalf + (k & 3) * 2,
                       qd + (k / 4) * (qhalf / 16) + (k & 3) * 2, id, k > 0);
              tc_commit(&sm.sfull[w][buf]);
              if (w == pc.k.tiles - 1) tc_commit(&sm.qempty[qslot]);
              if (t + 1 == pc.end) tc_commit(&sm.kempty[w][kslot[w]]);
            }
            __syncwarp();
          }
        }
      }
      if (elect_one()) tc_commit(&sm.done);
      __syncwarp();
      bar_await(&sm.done, 0, sm, a.err);
    }
  }
  // ---- pairs of tiles that no token sees: their weights fade ----
  if (a.decay != 1.f && a.window) {
#pragma unroll 1
    for (int b0 = 0; b0 < B; b0 += 32) {
      int n = 0, ctx = 0;
      bool bad;
      if (b0 + lane < B) n = tokens_of(a, b0 + lane, ctx, bad);
      unsigned some = __ballot_sync(0xffffffffu, n > 0 && ctx >= a.window);
#pragma unroll 1
      for (; some; some &= some - 1) {
        const int j = __ffs(some) - 1, c = __shfl_sync(0xffffffffu, ctx, j);
        // (a pair of which the window or the first tokens reach a part is an item)
        const int p0 = a.sinks > 0 ? tile_of(a, min(a.sinks - 1, c)) / 2 + 1 : 0, p1 = tile_of(a, c - a.window + 1) / 2;
        if (p0 >= p1) continue;
        int from, to, count;
        tile_slots(a, 2 * p0, from, count);
        tile_slots(a, 2 * p1, to, count);
        const long long m = static_cast<long long>(to - from) * a.Hkv;
        for (long long i = blockIdx.x * static_cast<long long>(kSumThreads) + tid; i < m;
             i += static_cast<long long>(C) * kSumThreads) {
          const int h = static_cast<int>(i / (to - from));
          float* at = a.weights + (b0 + j) * a.w_b + h * a.w_h + from + (i - static_cast<long long>(h) * (to - from));
          *at = a.decay == 0.f ? 0.f : a.decay * *at;
        }
      }
    }
  }
  tc_before();
  __syncthreads();
  if (warp == 0 && *reinterpret_cast<volatile int*>(&sm.abort)) {
    if (lane == 0 && a.ranges[blockIdx.x].used) a.ranges[blockIdx.x].used = 2;
    // given up: let copies in flight land before the shared memory is freed
    const unsigned long long t0 = now_ns();
    while (now_ns() - t0 < 20000000ull) __nanosleep(100000);
  }
  __syncthreads();
  if (warp == 1) {
    tc_after();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
  }
}

// Adds the parts of the items that range borders cut, in range order (not where a part's CTA
// gave up).  blockIdx.x: a range
// that starts inside an item; the first such range of an item does its work, a thread a slot.
__global__ void __launch_bounds__(256) weights_join_kernel(const __grid_constant__ Args a, int C) {
  const int c = blockIdx.x + 1, w = threadIdx.x >> 7, wt = threadIdx.x & 127;
  pdl_wait();
  const Range me = a.ranges[c];
  if (!me.used || me.t0 == 0) return;
  const long long s = me.lo - me.t0, e = s + me.T;
  int pk = c - 1;
  while (pk > 0 && !a.ranges[pk].used) --pk;
  const long long before = a.ranges[pk].lo;
  if (before > s) return;  // an earlier range's item
  int ctx, first, count;
  bool bad;
  const int n = tokens_of(a, me.b, ctx, bad);
  if (w >= item_of(a, ctx, n, me.p).tiles) return;
  tile_slots(a, 2 * me.p + w, first, count);
  const int off = row_offset(a, wt), slot = first + off;
  if (off >= count || slot >= ctx + n) return;
  float sum = 0.f;
#pragma unroll 1
  for (int k = pk; k < C; ++k) {
    if (k > pk) {
      if (!a.ranges[k].used) continue;
      if (a.ranges[k].lo >= e) break;
    }
    if (a.ranges[k].used == 2) return;
    sum += a.part[(2 * k + (k == pk && before < s ? 1 : 0)) * 256 + threadIdx.x];
  }
  float* at = a.weights + me.b * a.w_b + me.h * a.w_h + slot;
  *at = a.decay == 0.f ? sum : fmaf(a.decay, *at, sum);
}

struct Layout {
  size_t ranges, part, total;
};
Layout layout() {
  Layout L;
  L.ranges = 256;
  L.part = (L.ranges + sizeof(Range) * kMaxCtas + 255) / 256 * 256;
  L.total = L.part + 4ull * 2 * kMaxCtas * 256;
  return L;
}

template <class T, int D, bool GATHER>
cudaError_t launch_g(const CUtensorMap& mq, const CUtensorMap& mk, const Args& a, int C, size_t smem, cudaStream_t s) {
  cudaError_t e = cudaFuncSetAttribute(weights_kernel<T, D, GATHER>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
  if (e != cudaSuccess) return e;
  weights_kernel<T, D, GATHER><<<C, kSumThreads, smem, s>>>(mq, mk, a);
  e = cudaGetLastError();
  if (e != cudaSuccess || C < 2) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(C - 1);
  cfg.blockDim = dim3(256);
  cfg.stream = s;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, weights_join_kernel, a, C);
}

template <class T, int D>
cudaError_t launch_t(const CUtensorMap& mq, const CUtensorMap& mk, const Args& a, int C, size_t smem, cudaStream_t s) {
  return a.gather ? launch_g<T, D, true>(mq, mk, a, C, smem, s) : launch_g<T, D, false>(mq, mk, a, C, smem, s);
}

}  // namespace

size_t kv_weights_bytes() { return layout().total; }

cudaError_t launch_kv_weights(const WeightsParams& p, int dtype, int D, cudaStream_t s) {
  Args a;
  a.nodes = p.nodes;
  a.Hq = p.Hq; a.Hkv = p.kv.Hkv; a.G = p.G;
  a.tq = kTile / p.G < p.nodes.N ? kTile / p.G : p.nodes.N;
  a.cols = (a.tq * p.G + 31) / 32 * 32;
  const long long most = static_cast<long long>(p.kv.width) * p.kv.ps;
  a.window = p.window < most ? p.window : 0;  // (a window that no sequence exceeds is none)
  a.sinks = a.window ? p.sinks : 0;
  a.item_cost = 1;  // (an item's tiles of K, its first block and its sums)
  a.zero = p.scale == 0.f;
  a.c = a.zero ? 1.f : fabsf(p.scale) * kLog2e;
  a.negate = p.scale < 0.f;
  a.lse = p.lse; a.decay = p.decay;
  a.weights = p.weights; a.w_b = p.w_b; a.w_h = p.w_h; a.w_len = p.w_len;
  a.err = p.err;
  a.wait_us = p.wait_us; a.withheld = p.withheld;
  const Layout L = layout();
  char* ws = reinterpret_cast<char*>(p.err);
  a.ranges = reinterpret_cast<Range*>(ws + L.ranges);
  a.part = reinterpret_cast<float*>(ws + L.part);
  CUtensorMap mq, mk;
  if (!page_tiles(a, p.kv, dtype, D, &mk, nullptr) ||
      !encode_queries(&mq, p.q, p.q_b, p.q_n, p.q_h, p.Hq, p.nodes, p.G, dtype, D, a.tq))
    return cudaErrorInvalidValue;
  const long long slots = most < p.w_len ? most : p.w_len;
  const long long tiles = !a.uneven ? (slots + a.tk - 1) / a.tk : (slots / a.ps + 1) * a.tpp;
  a.NP = static_cast<int>((tiles + 1) / 2);
  // as many tiles of K as fit beside the blocks of Q (two of 32 KB: a third would leave one
  // slot a ring of K, and an item's tiles would wait for the last item's sums)
  const size_t slot = static_cast<size_t>(D) * 2 * kTile, qslot = static_cast<size_t>(D) * 2 * a.cols;
  a.nq = qslot > 16384 ? 2 : kMaxQueries;
  const size_t left = kSmemMax - sizeof(Misc) - a.nq * qslot;
  a.nk = static_cast<int>(left / (2 * slot) < kMaxKeys ? left / (2 * slot) : kMaxKeys);
  const size_t smem = 2 * a.nk * slot + a.nq * qslot + sizeof(Misc);
  int C = sm_count();
  if (C < 1) return cudaErrorInvalidDevice;
  C = C < kMaxCtas ? C : kMaxCtas;
  a.per_cta = C > 1 ? ~0ull / C + 1 : 0;
  const auto launch = dtype == Bf16::kId ? (D == 128 ? launch_t<Bf16, 128> : launch_t<Bf16, 64>)
                                         : (D == 128 ? launch_t<F16, 128> : launch_t<F16, 64>);
  return launch(mq, mk, a, C, smem, s);
}

}  // namespace ssd

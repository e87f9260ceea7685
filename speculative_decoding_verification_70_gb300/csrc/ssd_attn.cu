// ssd_attn.cu -- attention of the drafted nodes over the paged cache.
//
// For one key/value head the query rows are the R = N * G (node, query head of
// the group) pairs.  Over tiles of 128 cache slots,
//     S^T = K Q^T          [128 slots, R]    (scores, slots on the M axis)
//     P^T = 2^(c S^T - m)  masked            (c = scale log2 e, m per row)
//     O^T += V^T P^T       [D, R],  l += column sums of P^T
// and at the end O / l.  Slots lie on the tensor cores' M axis and rows on
// their N axis, so that few rows cost few columns (16 at least) instead of
// most of a 128-row tile, and one kernel serves one token, chains and wide
// trees.
//
// One persistent CTA per SM.  The batch's tiles (every sequence's, for every
// key/value head) are numbered and cut into equal ranges, one per CTA, by the
// lengths on the device: ragged batches and long single sequences are
// balanced alike.  A (sequence, head) whose tiles lie in one range is
// finished there; one that is cut leaves its parts (m, l, O in 32 bits) in
// the workspace, and attn_combine_kernel joins them in range order.
//
// Warps of a CTA:
//   0, 2   copy K and V tiles, page by page, by TMA into rings of slots
//          (128-byte swizzle; a page id out of range is a coordinate out of
//          bounds, which TMA fills with zeros)
//   1, 3   issue tcgen05.mma: S^T (K, Q from shared memory), and O^T (V^T read
//          transposed from the same row-major tile, P^T from shared memory)
//   4..15  three warpgroups for the softmax, which also fetch the rows of Q,
//          clear what must not be multiplied in tiles that hold drafted nodes
//          (V rows behind the sequence's end; NaN or infinite entries of
//          nodes, which are added at the end for the rows that see them) and
//          write the results.  Up to 64 rows: the warpgroups take tiles in
//          turn and keep their own m, l, O; more: the same tiles, a third of
//          the rows each.  (Two warpgroups with half of the rows each left
//          the pass over the scores waiting for its own latencies: 96 rows a
//          tile took 1680 cycles, three times 64 take 1200.)
//
// m follows the running maximum lazily: P and l come out of one pass over the
// scores, and only where a row's l grew by more than 2^12 (fp16: 2^8) of what the
// maximum adds the warpgroup finds the tile's row maxima, rescales l and O and
// repeats the pass.  P at a row's maximum is 2^-40 in bf16 (m is the maximum and 40):
// of 2^28 slots with P up to 2^-28 the sum P V stays within 32 bits whatever V holds,
// and down to V of 1e-21 their product does not fall below them.  In fp16, whose V
// ends at 65504 and whose range is short, it is 2^7, so that entries down to 2^-21 of
// the largest keep their precision.  (q k c - m is rounded once, but m itself is a
// number of 32 bits: scores beyond 2^24 differ by what their own roundings weigh,
// and beyond 2^27 the rounding of m alone exceeds what P holds.)
//
// Bound: HBM for up to 64 rows of a key/value head where the work is long (64
// contexts of 6800 slots, 32 + 8 heads, N = 1: D = 128 277 us, 6.4 TB/s; D = 64 178
// us, 5.0 TB/s).  With more rows the bytes in flight: Q and P leave four (168 rows)
// or three (256 rows) slots of 32 KB for the rings, which come round once in 5 us: 64
// trees of 21 nodes over 500..8000 slots in 197 us, 3.9 TB/s, two trees of 64 nodes
// over 60000 and 130000 slots in 235 us, 3.3 TB/s.  Beyond 256 rows every row block
// reads K and V (8 trees of 64 nodes, 8 heads a group, 500..8000 slots: 97 us).
// Short items: an item's start and end cost 5 us of a CTA (64 single tokens over
// 200..6000 slots: D = 64 63 us, 3.6 TB/s, D = 128 86 us, 5.3 TB/s).  One short
// sequence: the chain of set-up, first copies, one tile, results and join (8 nodes
// over 4096 slots: 20 us).
#include <cuda.h>
#include <math.h>

#include "ssd_async.cuh"
#include "ssd_device.cuh"
#include "ssd_kv.cuh"

namespace ssd {
namespace {

constexpr int kGroups = 3;           // warpgroups of the softmax
constexpr int kSoft = 128 * kGroups; // their threads
constexpr int kAttnThreads = 128 + kSoft;
constexpr int kTile = 128;           // slots of a tile (rows of the ring's tiles)
constexpr int kHalf = kTile * 128;   // bytes of a tile's 64-column half
constexpr int kPBlock = kTile * 32;  // bytes of P of 16 rows
constexpr int kPMin = 8192;          // least bytes of a warpgroup's P buffer
constexpr int kMaxRing = 4;           // slots of each ring
constexpr int kMaxRows = 256;        // rows of a row block
constexpr int kAlternate = 64;       // most rows whose tiles the warpgroups take in turn
constexpr int kMaxJob = 96;          // most rows of a warpgroup
constexpr int kTailBars = 8;
constexpr int kMaxCtas = 160;
constexpr int kNoRow = 0x7fffffff;   // a column without a row (rows of zeros: ~row)
constexpr float kNoScore = -1e30f;   // m of a row that has seen nothing
constexpr int kSmemMax = 227 * 1024;
template <class T>
constexpr float kLift = T::kId == Bf16::kId ? -40.f : 7.f;  // log2 of P at a row's maximum

// A CTA's range of tiles, for the joining kernel.
struct alignas(16) Range {
  long long lo;          // first tile (its position in cost)
  int t0;                // its place in its item
  int used;              // 0: a range without tiles
  int b, h, rb, T;       // its item, the item's tiles
};
static_assert(sizeof(Range) == 32, "read as two vectors");

struct Args {
  NodesView nodes;
  const int* table;
  long long table_stride;
  int width, pages, ps;
  int Hq, Hkv, G, R;
  int RB, rows_per_block;   // row blocks of a key/value head
  int split;                // the warpgroups split the rows
  int item_cost;            // what an item's start and end cost, in tiles
  int cols;                 // columns of S^T: the rows, rounded up to 16
  int wcols[kGroups], off[kGroups];  // a warpgroup's columns
  int poff[kGroups], pbytes;         // its P buffer; all of them
  int nk, nv;               // slots of the K and V rings
  int box, ppt, tk, tpp;    // rows of a TMA box, pages a tile, slots a tile, tiles a page
  int ragged;               // tiles have rows that are no slot
  int fold;                 // copies of whole groups of 8 slots: groups a page (0: rows of 64-column halves)
  int group, half;          // bytes from 8 slots of a tile to the next, from half to half
  int cover;                // rows of a tile that TMA writes
  const char* q;
  long long q_b, q_n, q_h;
  float c;                  // scale * log2(e)
  int zero;                 // scale 0: Q counts as zeros (and c as 1)
  char* out;
  float* lse;
  const char* vcache;       // for the rows that see a node with NaN or infinities
  long long v_page, v_slot, v_head;
  float* part_o;            // [2 ctas][cols][D]
  float2* part_ml;          // [2 ctas][cols]
  struct Range* ranges;     // [ctas]
  unsigned long long per_cta;  // 2^64 / ctas, rounded up
  int* err;
  unsigned wait_us;         // a wait that takes longer has failed
  int withheld;             // bytes that are waited for beside the copied ones (self-test)
};

// Shared memory behind the ring, Q and P (256 rows leave 3 KB for it).
struct alignas(16) Misc {
  uint64_t kfull[kMaxRing], kempty[kMaxRing], vfull[kMaxRing], vempty[kMaxRing];
  uint64_t qfull[2], sfull[kGroups], pfull[kGroups], pvdone[kGroups], vready[kTailBars], done;
  uint64_t anc[2][kMaxNodes + 1];   // nodes' ancestors (0: absent); the last: no row
  long long left;
  alignas(16) float nm[kMaxRows];   // -m, of each warpgroup's columns
  uint8_t node[2][kMaxRows];        // rows' nodes
  unsigned nf[2][2];                // nodes with NaN or infinite values
  int b0, h0, rb0, t0;              // first piece, its sequence's
  int T0, ctx0, tot0, tail0;        // tiles and lengths
  int cost;                         // of an item beside its tiles
  unsigned tmem;
  int abort;
  unsigned wait_us;
};
static_assert(sizeof(Misc) <= 3 * 1024, "shared memory of 256 rows");

// What a warpgroup keeps in its P buffer while that holds no P: between the
// product of one tile and the P of the next, and at the end of a piece.
struct Scratch {
  float fac[kMaxJob];
  int row[kMaxJob];  // node * Hq + head of the group, its complement, or kNoRow
  union {
    struct {
      float red[4][kMaxJob];
      uint4 seen[kMaxJob];  // rows' masks, for a tile with drafted nodes
    };
    char stage[4][1024];    // results on their way out, a part per warp
  };
};
static_assert(sizeof(Scratch) <= kPMin, "the smallest P buffer");

// ---------------------------------------------------------------------------
// mbarriers, TMA, tcgen05
// ---------------------------------------------------------------------------
__device__ __forceinline__ void bar_arrive(uint64_t* b) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(sptr(b)) : "memory");
}
// Bounded wait: after wait_us (or once another wait of the CTA gave up) the CTA
// runs on without waiting, to its end; the error word says so.
__device__ __forceinline__ bool bar_wait(uint64_t* b, uint32_t parity, Misc& sm, int* err) {
  unsigned long long t0 = 0;
  for (unsigned i = 1;; ++i) {
    if (bar_try(b, parity)) return true;
    if (*reinterpret_cast<volatile int*>(&sm.abort)) return false;
    if ((i & 31) == 0) {  // the global timer is slow to read
      const unsigned long long t = now_ns();
      if (t0 == 0) t0 = t;
      if (t - t0 > sm.wait_us * 1000ull) {
        *reinterpret_cast<volatile int*>(&sm.abort) = 1;
        atomicOr(err, kErrTimeout);
        return false;
      }
    }
  }
}

__device__ __forceinline__ void named_sync(int id, int n) {
  asm volatile("barrier.cta.sync %0, %1;" ::"r"(id), "r"(n) : "memory");
}
__device__ __forceinline__ bool named_or(int id, int n, bool v) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 q, %3, 0;\n\t"
      "barrier.cta.red.or.pred p, %1, %2, q;\n\t"
      "selp.b32 %0, 1, 0, p;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(n), "r"(static_cast<uint32_t>(v))
      : "memory");
  return r != 0;
}

__device__ __forceinline__ void tma_rows(uint32_t dst, const CUtensorMap* map, int d, int slot, int head,
                                         int page, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(map), "r"(sptr(bar)), "r"(d), "r"(slot), "r"(head), "r"(page)
      : "memory");
}

// As tma_rows for whole groups of 8 slots, both 64-column halves in one copy.
__device__ __forceinline__ void tma_groups(uint32_t dst, const CUtensorMap* map, int group, int head,
                                           uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%3, %3, %3, %4, %5}], [%2];" ::"r"(dst),
      "l"(map), "r"(sptr(bar)), "r"(0), "r"(group), "r"(head)
      : "memory");
}

__device__ __forceinline__ void fence_async() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}
__device__ __forceinline__ void tc_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tc_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.b32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ void tc_commit(uint64_t* b) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(
                   sptr(b))
               : "memory");
}
__device__ __forceinline__ void tc_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.u32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(static_cast<uint32_t>(acc))
      : "memory");
}

// Shared-memory operand descriptor: strides in bytes; swizzle 2: 128 bytes,
// 6: 32 bytes.
__device__ __forceinline__ uint64_t operand(uint32_t addr, uint32_t lead, uint32_t stride, uint64_t swizzle = 2) {
  return static_cast<uint64_t>((addr >> 4) & 0x3fff) | (static_cast<uint64_t>(lead >> 4) << 16) |
         (static_cast<uint64_t>(stride >> 4) << 32) | (1ull << 46) | (swizzle << 61);
}
// Instruction descriptor: 32-bit accumulator, 128 x n, 16-bit operands.
template <class T>
__device__ __forceinline__ uint32_t instr(int n, bool a_mn, bool b_mn) {
  const uint32_t f = T::kId == Bf16::kId ? 1u : 0u;
  return (1u << 4) | (f << 7) | (f << 10) | (static_cast<uint32_t>(a_mn) << 15) |
         (static_cast<uint32_t>(b_mn) << 16) | (static_cast<uint32_t>(n >> 3) << 17) | (8u << 24);
}

#define SSD_TM16(r)                                                                              \
  "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), \
      "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),   \
      "=r"(r[15])

__device__ __forceinline__ void tm_ld16(uint32_t addr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : SSD_TM16(r)
      : "r"(addr));
}
__device__ __forceinline__ void tm_st16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(addr));
}
// Waits for this thread's tcgen05.ld; the registers are tied to the wait so
// that no use moves before it.
__device__ __forceinline__ void tm_wait_ld(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
                 "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]),
                 "+r"(r[13]), "+r"(r[14]), "+r"(r[15]));
}
// 32 lanes x 16 columns as fragments: register [half][4 g + 2 r + i] of lane
// 4 y + x is lane 16 half + 8 r + y, column 8 g + 2 x + i.
__device__ __forceinline__ void tm_ld_frag(uint32_t addr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
      : "r"(addr));
  asm volatile(
      "tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
      : "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
        "=r"(r[15])
      : "r"(addr + (16u << 16)));
}
__device__ __forceinline__ void tm_st_frag(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile("tcgen05.st.sync.aligned.16x256b.x2.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::"r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(addr));
  asm volatile("tcgen05.st.sync.aligned.16x256b.x2.b32 [%8], {%0,%1,%2,%3,%4,%5,%6,%7};" ::"r"(r[8]), "r"(r[9]),
               "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(addr + (16u << 16)));
}
__device__ __forceinline__ void tm_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// ---------------------------------------------------------------------------
// the tiles of the batch
// ---------------------------------------------------------------------------
// n / tk (most pages fill tiles: a shift instead of a division)
__device__ __forceinline__ int by_tile(const Args& a, int n) { return a.tk == kTile ? n / kTile : n / a.tk; }
__device__ __forceinline__ int tiles_of(const Args& a, int tot) {
  if (a.ps <= kTile) return by_tile(a, tot + a.tk - 1);
  return (tot / a.ps) * a.tpp + (tot % a.ps + kTile - 1) / kTile;
}
// First slot of tile t, and how many it holds.
__device__ __forceinline__ void tile_slots(const Args& a, int t, int& first, int& count) {
  if (a.ps <= kTile) {
    first = t * a.tk;
    count = a.tk;
  } else {
    const int r = (t % a.tpp) * kTile;
    first = (t / a.tpp) * a.ps + r;
    count = min(kTile, a.ps - r);
  }
}
// Offset of a tile's row from its first slot, -1 for a row that is no slot.
__device__ __forceinline__ int row_slot(const Args& a, int row, int count) {
  if (a.ps > kTile) return row < count ? row : -1;
  const int p = row / a.box, r = row - p * a.box;
  return p < a.ppt && r < a.ps ? p * a.ps + r : -1;
}

__device__ __forceinline__ int seq_len(const Args& a, int b, int& ctx, bool& bad) {
  ctx = __ldg(a.nodes.ctx_len + b);
  const int nn = a.nodes.n_nodes ? __ldg(a.nodes.n_nodes + b) : a.nodes.N;
  const int n = seq_nodes(ctx, nn, a.nodes.N, a.width, a.ps, bad);
  return n == 0 ? 0 : ctx + n;  // a sequence without nodes has no tiles
}

struct SeqTiles {
  int T, ctx, tot, tail;  // tiles; lengths; the first tile with slots behind the context
};
__device__ __noinline__ SeqTiles seq_tiles(const Args& a, int b) {
  SeqTiles q;
  bool bad;
  q.tot = seq_len(a, b, q.ctx, bad);
  q.T = tiles_of(a, q.tot);
  q.tail = a.ps <= kTile ? by_tile(a, q.ctx) : (q.ctx / a.ps) * a.tpp + (q.ctx % a.ps) / kTile;
  return q;
}

// The pieces of a CTA's range, one (sequence, head, row block) after another.
// Only the first may start behind tile 0.
struct Pieces {
  long long left;     // cost from t0 to the range's end: a tile 1, an item's end w
  int w;
  int b, h, rb;
  int T, ctx, tot;    // of sequence b
  int t0, end, tail;  // tiles t0 .. end - 1; the first with slots behind the context
  bool fresh;
  __device__ __forceinline__ void start(const Misc& sm) {
    left = sm.left;
    w = sm.cost;
    b = sm.b0;
    h = sm.h0;
    rb = sm.rb0;
    t0 = sm.t0;
    T = sm.T0;
    ctx = sm.ctx0;
    tot = sm.tot0;
    tail = sm.tail0;
    fresh = true;
  }
  __device__ __forceinline__ bool direct() const { return t0 == 0 && end == T; }
  __device__ __forceinline__ void load(const Args& a) {
    const SeqTiles q = seq_tiles(a, b);
    T = q.T;
    ctx = q.ctx;
    tot = q.tot;
    tail = q.tail;
  }
  __device__ __forceinline__ bool next(const Args& a) {
    bool reload = false;
    if (!fresh) {
      left -= end - t0 + (end == T ? w : 0);
      t0 = 0;
      if (++rb == a.RB) {
        rb = 0;
        if (++h == a.Hkv) {
          h = 0;
          ++b;
          reload = true;
        }
      }
    }
    fresh = false;
    if (left <= 0) return false;
    if (reload) {
#pragma unroll 1
      for (;; ++b) {
        if (b >= a.nodes.B) {
          left = 0;
          return false;
        }
        load(a);
        if (T > 0) break;
      }
    }
    end = static_cast<int>(min(static_cast<long long>(T), t0 + left));
    return true;
  }
};

// ---------------------------------------------------------------------------
// softmax: one tile for one warpgroup
// ---------------------------------------------------------------------------
// A thread works on fragments: of every 16 rows (columns of S^T) it holds the
// four 2 x + {0, 1}, 8 + 2 x + {0, 1} for the four slots y + {0, 8, 16, 24} of
// its warp's 32 (lane 4 y + x), so a row's sum needs one register of four
// threads' columns and m one load per two rows.

// A row's mask as four words: ~0 for the 32 slots before the first node, the
// 64 nodes, 0 behind them.  32 bits of it from slot j (relative to the first
// node) on, j >= -32:
__device__ __forceinline__ uint32_t seen_from(const uint4* row, int word, int shift) {
  const uint32_t* w = reinterpret_cast<const uint32_t*>(row);
  return __funnelshift_r(w[word], word < 3 ? w[word + 1] : 0u, shift);
}

// Scores that are not seen become `none` (-inf once scaled), in place.  mask:
// the rows' masks, from the thread's first row.
template <bool PLAIN>
__device__ __noinline__ void mask_tile(const Args& a, int t, int ctx, int tot, uint32_t tS, int nch,
                                       const uint4* mask, float none) {
  const int row0 = ((threadIdx.x >> 5) & 3) * 32, y = (threadIdx.x & 31) >> 2;
  int first, count;
  tile_slots(a, t, first, count);
  if (PLAIN && first + row0 + 32 <= ctx) return;
  int word[4], shift[4];
#pragma unroll
  for (int q = 0; q < (PLAIN ? 1 : 4); ++q) {
    // plain: row r of the tile is slot first + r, and bits 8 q of a word from
    // the first of the thread's slots on are the four
    const int r = PLAIN ? row0 + y : row_slot(a, row0 + y + 8 * q, count);
    int j = first + r - ctx;
    if (r < 0 || first + r >= tot) j = kMaxNodes;
    j = min(max(j, -32), kMaxNodes) + 32;
    word[q] = j >> 5;
    shift[q] = j & 31;
  }
#pragma unroll 1
  for (int k = 0; k < nch; ++k) {
    uint32_t s[16], w[4];
    tm_ld_frag(tS + k * 16, s);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4* m = mask + k * 16 + (i >> 1) * 8 + (i & 1);
      w[i] = seen_from(m, word[0], shift[0]);
      if (!PLAIN) {
        w[i] &= 1;
#pragma unroll
        for (int q = 1; q < 4; ++q) w[i] |= (seen_from(m, word[q], shift[q]) & 1) << (8 * q);
      }
    }
    tm_wait_ld(s);
#pragma unroll
    for (int g = 0; g < 2; ++g) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int i = (q >> 1) * 8 + g * 4 + (q & 1) * 2;
        if (!(w[g * 2] & (1u << (8 * q)))) s[i] = __float_as_uint(none);
        if (!(w[g * 2 + 1] & (1u << (8 * q)))) s[i + 1] = __float_as_uint(none);
      }
    }
    tm_st_frag(tS + k * 16, s);
  }
  tm_wait_st();
}

// Four 8 x 8 matrices of 16-bit entries from fragments into shared memory;
// lane 8 i + j gives the address of row j of matrix i.  (Ordered among the
// volatile statements; the fence before the consumers orders the memory.)
__device__ __forceinline__ void st_matrices(uint32_t at, const uint32_t (&w)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(w[0]), "r"(w[1]),
               "r"(w[2]), "r"(w[3]));
}
// The same with each matrix transposed.
__device__ __forceinline__ void st_matrices_t(uint32_t at, const uint32_t (&w)[4]) {
  asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(w[0]),
               "r"(w[1]), "r"(w[2]), "r"(w[3]));
}

// P^T of the tile into shared memory (rows contiguous, 16 of them and 128
// slots a block, 32-byte swizzle), l += P.  prow: this lane's slot's line of
// the first block.  The matrices of 16 rows are stored while the next rows'
// exponentials are on their way; `ready` is called before the first store.
template <class T, int NC, class Ready>
__device__ __forceinline__ void tile_pass(uint32_t tS, int nch, f32x2 c2, const float* nm, int x2, uint32_t prow,
                                          int slot, f32x2 (&l)[NC / 8], Ready&& ready) {
  uint32_t s[2][16], w[2][4];
  const uint32_t a0 = prow + (((slot >> 2) & 1) << 4), a1 = a0 ^ 16;
  tm_ld_frag(tS, s[0]);
  const float* m = nm + x2;
  f32x2 m0 = *reinterpret_cast<const f32x2*>(m), m1 = *reinterpret_cast<const f32x2*>(m + 8);
#pragma unroll
  for (int k = 0; k < NC / 16; ++k) {
    if (k < nch) {
      tm_wait_ld(s[k & 1]);
      f32x2 n0 = 0ull, n1 = 0ull;
      if (k + 1 < nch) {
        tm_ld_frag(tS + (k + 1) * 16, s[(k + 1) & 1]);
        n0 = *reinterpret_cast<const f32x2*>(m + (k + 1) * 16);
        n1 = *reinterpret_cast<const f32x2*>(m + (k + 1) * 16 + 8);
      }
      const uint32_t(&x)[16] = s[k & 1];
      uint32_t v[2][4];
#pragma unroll
      for (int g = 0; g < 2; ++g) {
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int i = (q >> 1) * 8 + g * 4 + (q & 1) * 2;
          float t0, t1;
          up2(fma2(pk2(__uint_as_float(x[i]), __uint_as_float(x[i + 1])), c2, g ? m1 : m0), t0, t1);
          const float e0 = ex2_fast(t0), e1 = ex2_fast(t1);
          l[k * 2 + g] = add2(l[k * 2 + g], pk2(e0, e1));
          v[g][q] = T::pack(e0, e1);
        }
      }
      if (k > 0) {
        st_matrices(a0 + (k - 1) * kPBlock, w[0]);
        st_matrices(a1 + (k - 1) * kPBlock, w[1]);
      } else {
        ready();
      }
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        w[0][q] = v[0][q];
        w[1][q] = v[1][q];
      }
      m0 = n0;
      m1 = n1;
    }
  }
  st_matrices(a0 + (nch - 1) * kPBlock, w[0]);
  st_matrices(a1 + (nch - 1) * kPBlock, w[1]);
}

// ln(2^m l).  (m goes back to the maximum first, which is exact, so that no digits
// are lost to the distance.)
template <class T>
__device__ __forceinline__ float log_sum(float m, float l) {
  constexpr float far = kLift<T> < 0.f ? kLift<T> : 0.f, back = kLift<T> < 0.f ? 0x1p40f : 1.f;
  return (m + far + log2f(l * back)) * 0.6931471805599453f;
}

// The largest growth of a row sum.
template <int N>
__device__ __forceinline__ float growth(const f32x2 (&l)[N], const f32x2 (&old)[N]) {
  float ex = 0.f;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    float a, b;
    up2(sub2(l[i], old[i]), a, b);
    ex = max3(ex, a, b);
  }
  return ex;
}

// Joins v over the eight lanes that hold the same rows, each lane giving half
// of its rows away at a step, and stores the results: v[2 i + h] belongs to
// row 8 i + x2 + h.
template <int NC, bool MAX>
__device__ __forceinline__ void join_rows(float (&v)[NC / 4], float* red, int lane, int ncj) {
  int base = 0, n = NC / 8;  // groups of 8 rows: base .. base + n - 1 are in v
#pragma unroll
  for (int d = 16; d >= 4; d >>= 1) {
    const bool up = lane & d;
    if (n % 2 == 0) {
      n >>= 1;
      if (up) base += n;
#pragma unroll
      for (int i = 0; i < NC / 8; ++i) {
        if (i < 2 * n && i + 2 * n < NC / 4) {
          const float give = up ? v[i] : v[i + 2 * n];
          const float mine = up ? v[i + 2 * n] : v[i];
          const float got = __shfl_xor_sync(0xffffffffu, give, d);
          v[i] = MAX ? fmaxf(mine, got) : mine + got;
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < NC / 4; ++i) {
        if (i < 2 * n) {
          const float got = __shfl_xor_sync(0xffffffffu, v[i], d);
          v[i] = MAX ? fmaxf(v[i], got) : v[i] + got;
        }
      }
    }
  }
#pragma unroll
  for (int i = 0; i < NC / 8; ++i) {
    if (i < n && (base + i) * 8 < ncj)
      *reinterpret_cast<float2*>(red + (base + i) * 8 + (lane & 3) * 2) = make_float2(v[2 * i], v[2 * i + 1]);
  }
}

// Row maxima of c s over the warp's 32 slots, into red.
template <int NC>
__device__ __noinline__ void tile_maxima(uint32_t tS, int ncj, float c, float* red) {
  const int lane = threadIdx.x & 31;
  float v[NC / 4];
#pragma unroll
  for (int k = 0; k < NC / 16; ++k) {
    if (k * 16 < ncj) {
      uint32_t s[16];
      tm_ld_frag(tS + k * 16, s);
      tm_wait_ld(s);
#pragma unroll
      for (int g = 0; g < 2; ++g) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const float a = __uint_as_float(s[g * 4 + i]) * c, b = __uint_as_float(s[g * 4 + 2 + i]) * c;
          const float d = __uint_as_float(s[8 + g * 4 + i]) * c, e = __uint_as_float(s[8 + g * 4 + 2 + i]) * c;
          v[k * 4 + g * 2 + i] = fmaxf(fmaxf(a, b), fmaxf(d, e));
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) v[k * 4 + i] = 0.f;
    }
  }
  join_rows<NC, true>(v, red, lane, ncj);
}

// O of the warpgroup times the factors of its rows.
__device__ __noinline__ void rescale(uint32_t tO, int nch, const float* fac) {
#pragma unroll 1
  for (int k = 0; k < nch; ++k) {
    uint32_t o[16];
    tm_ld16(tO + k * 16, o);
    tm_wait_ld(o);
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * fac[k * 16 + i]);
    tm_st16(tO + k * 16, o);
  }
  tm_wait_st();
}

// Adds the NaN or infinite values of nodes (nf: the nodes that hold some) to
// the written rows that see them: column d of the job's rows, in `out`
// (row numbers in `row`) or in the parts.
template <class T, int D>
__device__ __noinline__ void add_nonfinite(const Args& a, int b, int h, int ctx, unsigned long long nf, int d,
                                           const uint64_t* anc, const uint8_t* node, const int* row, int c0, int c1,
                                           char* out, float* part) {
#pragma unroll 1
  for (int j = 0; j < a.nodes.N; ++j) {
    if (!((nf >> j) & 1)) continue;
    int page, off;
    if (!kv_slot(a.table + b * a.table_stride, a.width, a.pages, a.ps, static_cast<long long>(ctx) + j, page, off))
      continue;
    const unsigned short raw = *reinterpret_cast<const unsigned short*>(
        a.vcache + 2 * (page * a.v_page + off * a.v_slot + h * a.v_head + d));
    const float v = T::lo(raw);
    if (fabsf(v) < INFINITY) continue;
#pragma unroll 1
    for (int c = c0; c < c1; ++c) {
      if (row[c] < 0 || row[c] == kNoRow || !((anc[node[c]] >> j) & 1)) continue;
      if (part) {
        part[static_cast<long long>(c) * D + d] += v;
      } else {
        unsigned short* o = reinterpret_cast<unsigned short*>(out) + static_cast<long long>(row[c]) * D + d;
        *o = static_cast<unsigned short>(T::pack(T::lo(*o) + v, 0.f));
      }
    }
  }
}

// The nodes of a piece's rows and the nodes' masks (by all threads of the
// warpgroups).
__device__ __noinline__ void row_tables(const Args& a, Misc& sm, int b, int rb, int n, int tb) {
  const int at = threadIdx.x - 128;
  const int r0 = rb * a.rows_per_block;
  const int rows = min(a.rows_per_block, a.R - r0);
  if (at < a.cols) sm.node[tb][at] = static_cast<uint8_t>(at < rows ? (r0 + at) / a.G : kMaxNodes);
  if (at >= kMaxRows && at < kMaxRows + kMaxNodes) {
    const int j = at - kMaxRows;
    const int* parent = a.nodes.parent ? a.nodes.parent + static_cast<long long>(b) * a.nodes.N : nullptr;
    uint64_t m = 0;
    int depth;
    bool broken = false;
    if (j < n) node_way(parent, n, j, m, depth, broken);
    if (broken) atomicOr(a.err, kErrBadTree);
    sm.anc[tb][j] = m;
    if (j < 2) sm.nf[tb][j] = 0;
    if (j == 0) sm.anc[tb][kMaxNodes] = 0;
  }
}

// Columns c0 .. c1 - 1 of Q of a piece on their way into shared memory, by
// `threads` threads, of which this is number `at`.
template <int D>
__device__ __noinline__ void fetch_rows(const Args& a, int b, int h, int rb, int n, char* Q, int c0, int c1, int at,
                                        int threads) {
  const int r0 = rb * a.rows_per_block;
  const int rows = min(a.rows_per_block, a.R - r0);
  constexpr int PER = D / 8;         // 16-byte vectors of a row
  const int step = threads / PER;    // rows side by side
  const int v = at % PER;
  const char* base = a.q + 2 * (b * a.q_b + static_cast<long long>(h) * a.G * a.q_h + v * 8);
  const uint32_t dst = sptr(Q) + (v / 8) * (a.cols * 128);
  int r = c0 + at / PER;
  int i = (r0 + r) / a.G, g = r0 + r - i * a.G;
#pragma unroll 1
  for (; r < c1; r += step) {
    const bool real = r < rows && i < n && !a.zero;
    const char* src = real ? base + 2 * (i * a.q_n + g * a.q_h) : a.q;
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst + r * 128 + (((v ^ r) & 7) << 4)), "l"(src),
                 "r"(real ? 16 : 0)
                 : "memory");
    g += step;
    while (g >= a.G) {
      g -= a.G;
      ++i;
    }
  }
}
__device__ __forceinline__ void rows_ready(Misc& sm, int qb) {
  asm volatile("cp.async.wait_all;" ::: "memory");
  fence_async();
  bar_arrive(&sm.qfull[qb]);
}

// Clears V rows that are no slot of the sequence and the NaN or infinite
// entries of its nodes (whose bits go to nf).  One warpgroup, a row a thread.
template <class T, int D>
__device__ __noinline__ void clean_tile(const Args& a, Misc& sm, int t, int ctx, int tot, char* V, int tb, int r) {
  int first, count;
  tile_slots(a, t, first, count);
  const int rs = row_slot(a, r, count);
  const int slot = rs < 0 ? 0x7fffffff : first + rs;
  if (slot < ctx) return;
  uint4* line = reinterpret_cast<uint4*>(V + (r >> 3) * a.group + (r & 7) * 128);
  const int half = a.half / 16;
  if (slot >= tot) {
#pragma unroll
    for (int v = 0; v < D / 8; ++v) line[(v / 8) * half + ((v ^ r) & 7)] = make_uint4(0, 0, 0, 0);
    return;
  }
  // an exponent of all ones carries into the sign's place
  constexpr uint32_t kExp = T::kId == Bf16::kId ? 0x7f807f80u : 0x7c007c00u;
  constexpr uint32_t kOne = T::kId == Bf16::kId ? 0x00800080u : 0x04000400u;
  uint32_t carry = 0;
#pragma unroll
  for (int v = 0; v < D / 8; ++v) {
    const uint4 x = line[(v / 8) * half + ((v ^ r) & 7)];
    carry |= ((x.x & kExp) + kOne) | ((x.y & kExp) + kOne) | ((x.z & kExp) + kOne) | ((x.w & kExp) + kOne);
  }
  const bool bad = carry & 0x80008000u;
  if (bad) {
#pragma unroll 1
    for (int v = 0; v < D / 8; ++v) {
      uint32_t* p = reinterpret_cast<uint32_t*>(line + (v / 8) * half + ((v ^ r) & 7));
#pragma unroll 1
      for (int i = 0; i < 4; ++i) {
        const uint32_t c = ((p[i] & kExp) + kOne) & 0x80008000u;
        if (c) p[i] &= (c & 0x8000u ? 0u : 0xffffu) | (c >> 31 ? 0u : 0xffff0000u);
      }
    }
  }
  if (bad) {
    const int j = slot - ctx;
    atomicOr(&sm.nf[tb][j >> 5], 1u << (j & 31));
  }
}

template <class T, int D, int NC>
__device__ __forceinline__ void softmax_role(const Args& a, Misc& sm, uint32_t tmem, char* Q, int qbytes, char* V,
                                             char* P0, int wg) {
  constexpr float kGrow = T::kId == Bf16::kId ? 0x1p-28f : 0x1p15f;
  const bool split = a.split;
  char* P = P0 + a.poff[wg];
  Scratch& sc = *reinterpret_cast<Scratch*>(P);
  const int wt = threadIdx.x - 128 - wg * 128;  // thread of the warpgroup = TMEM lane
  const int warp = __shfl_sync(0xffffffffu, wt >> 5, 0), lane = wt & 31;
  const int x2 = (lane & 3) * 2;  // first of the thread's rows in a group of 8
  const int ncj = a.wcols[wg], nch = ncj / 16, colbase = a.off[wg];
  const int tcol = split ? colbase : wg * kAlternate;  // its columns of TMEM and of nm
  const uint32_t lane_base = static_cast<uint32_t>(warp * 32) << 16;
  const uint32_t tS = tmem + lane_base + tcol;
  const uint32_t tO0 = tmem + lane_base + kMaxRows;
  const uint32_t tO = tO0 + tcol;
  const uint32_t prow = sptr(P) + wt * 32;
  const f32x2 c2 = pk2(a.c, a.c);
  float* nm = sm.nm + tcol;
  const int bar = 1 + wg;
  const float none = a.c < 0.f ? INFINITY : -INFINITY;
  uint32_t ps = 0, ppv = 0;  // phases of sfull, pvdone
  int item_no = 0;
  const int at = threadIdx.x - 128;
  int g0 = 0, tails0 = 0;  // tiles (with drafted nodes) before this piece
  Pieces pn;               // one piece ahead
  pn.start(sm);
  bool more = pn.next(a);
  if (more) {
    fetch_rows<D>(a, pn.b, pn.h, pn.rb, pn.tot - pn.ctx, Q, 0, a.cols, at, kSoft);
    row_tables(a, sm, pn.b, pn.rb, pn.tot - pn.ctx, 0);
    rows_ready(sm, 0);
  }
  while (more) {
    const int b = pn.b, h = pn.h, t0 = pn.t0, end = pn.end, ctx = pn.ctx, tot = pn.tot;
    const int tail = max(pn.tail, t0), mask_from = a.ragged ? 0 : tail;
    const bool direct = pn.direct();
    const int r0 = pn.rb * a.rows_per_block + colbase;
    const int rows = min(a.rows_per_block - colbase, a.R - r0);  // of this job's columns
    const int tb = item_no & 1;                                  // tables
    more = pn.next(a);
    // The next piece's tables and rows, while this piece's first product
    // runs: the rows go into the other buffer, or (one buffer) later into
    // this warpgroup's part, once its last scores are there.
    bool todo = more, pending = false;
    auto prefetch = [&]() {
      row_tables(a, sm, pn.b, pn.rb, pn.tot - pn.ctx, tb ^ 1);
      if (!split) {
        fetch_rows<D>(a, pn.b, pn.h, pn.rb, pn.tot - pn.ctx, Q + (tb ^ 1) * qbytes, 0, a.cols, at, kSoft);
        pending = true;
      }
      todo = false;
    };
    const uint64_t* anc = sm.anc[tb];
    const uint8_t* node = sm.node[tb] + colbase;
    if (wt < ncj) nm[wt] = -kNoScore;
    f32x2 l[NC / 8];
#pragma unroll
    for (int i = 0; i < NC / 8; ++i) l[i] = 0ull;
    named_sync(kGroups + 1, kSoft);
    int jobs = 0;
    const int turn = split ? 0 : (wg + kGroups - g0 % kGroups) % kGroups, step = split ? 1 : kGroups;
#pragma unroll 1
    for (int t = t0 + turn; t < end; t += step) {
      bar_wait(&sm.sfull[wg], ps, sm, a.err);
      ps ^= 1;
      bool fresh = jobs > 0;  // the last tile's product is to be waited for
      auto ready = [&]() {
        if (fresh) {
          bar_wait(&sm.pvdone[wg], ppv, sm, a.err);
          ppv ^= 1;
          fresh = false;
          tc_after();
        }
      };
      tc_after();
      if (t >= mask_from) {
        ready();
        if (wt < ncj) {
          const uint64_t m = anc[node[wt]];
          sc.seen[wt] = make_uint4(~0u, static_cast<uint32_t>(m), static_cast<uint32_t>(m >> 32), 0u);
        }
        named_sync(bar, 128);
        if (a.ragged) mask_tile<false>(a, t, ctx, tot, tS, nch, sc.seen + x2, none);
        else mask_tile<true>(a, t, ctx, tot, tS, nch, sc.seen + x2, none);
        named_sync(bar, 128);  // the masks lie where P goes
      }
      bool raise = jobs == 0;
#pragma unroll 1
      while (true) {
        if (raise) {
          ready();
          tile_maxima<NC>(tS, ncj, a.c, sc.red[warp]);
          named_sync(bar, 128);
          if (wt < ncj) {
            const float mx = fmaxf(fmaxf(sc.red[0][wt], sc.red[1][wt]), fmaxf(sc.red[2][wt], sc.red[3][wt]));
            const float mo = -nm[wt];
            const float mn = fmaxf(mo, mx - kLift<T>);
            sc.fac[wt] = mn == mo ? 1.f : exp2f(mo - mn);
            nm[wt] = -mn;
          }
          named_sync(bar, 128);
          if (jobs > 0) {
#pragma unroll
            for (int i = 0; i < NC / 8; ++i)
              if (8 * i < ncj) l[i] = mul2(l[i], *reinterpret_cast<const f32x2*>(sc.fac + 8 * i + x2));
            rescale(tO, nch, sc.fac);
            named_sync(bar, 128);  // the factors lie where P goes
          }
        }
        f32x2 old[NC / 8];
#pragma unroll
        for (int i = 0; i < NC / 8; ++i) old[i] = l[i];
        tile_pass<T, NC>(tS, nch, c2, nm, x2, prow, wt, l, ready);
        if (!named_or(bar, 128, growth(l, old) > kGrow) || raise) break;
        raise = true;
#pragma unroll
        for (int i = 0; i < NC / 8; ++i) l[i] = old[i];
      }
      if (t >= tail && (!split || wg == 0)) {
        const int n = tails0 + t - tail, slot = (g0 + t - t0) % a.nv;
        bar_wait(&sm.vready[n % kTailBars], (n / kTailBars) & 1, sm, a.err);
        clean_tile<T, D>(a, sm, t, ctx, tot, V + slot * (kTile * D * 2), tb, wt);
      }
      tc_before();
      fence_async();
      bar_arrive(&sm.pfull[wg]);
      ++jobs;
      if (pending) {
        rows_ready(sm, tb ^ 1);
        pending = false;
      }
      if (todo) prefetch();
    }

    // ---- end of the piece: l over the slots, then O ----
    if (todo) prefetch();
    if (pending) rows_ready(sm, tb ^ 1);
    if (split && more) fetch_rows<D>(a, pn.b, pn.h, pn.rb, pn.tot - pn.ctx, Q, colbase, colbase + ncj, wt, 128);
    if (jobs > 0) {
      bar_wait(&sm.pvdone[wg], ppv, sm, a.err);
      ppv ^= 1;
      tc_after();
    }
    {
      float v[NC / 4];
#pragma unroll
      for (int i = 0; i < NC / 8; ++i) up2(l[i], v[2 * i], v[2 * i + 1]);
      join_rows<NC, false>(v, sc.red[warp], lane, ncj);
    }
    if (split) named_sync(bar, 128);
    else named_sync(kGroups + 1, kSoft);
    const int tiles = end - t0;
    const long long pslot = (2ll * blockIdx.x + (item_no == 0 ? 0 : 1)) * a.cols + colbase;
    const long long orow = static_cast<long long>(b) * a.nodes.N * a.Hq + h * a.G;
    // tiles in turn: the warpgroups that took part, of which each writes a
    // share of the rows
    const int w0 = split ? wg : 0, w1 = split ? wg + 1 : kGroups;
    auto used = [&](int w) { return split || (w + kGroups - g0 % kGroups) % kGroups < tiles; };
    auto scratch = [&](int w) -> Scratch& { return *reinterpret_cast<Scratch*>(P0 + a.poff[w]); };
    Scratch& so = scratch(w0);
    if (wt < ncj && wg == w0) {
      // factors of the warpgroups' O, and where the rows go
      const int cc = wt;
      float M = kNoScore, L = 0.f;
#pragma unroll 1
      for (int w = w0; w < w1; ++w)
        if (used(w)) M = fmaxf(M, -sm.nm[(split ? tcol : w * kAlternate) + cc]);
#pragma unroll 1
      for (int w = w0; w < w1; ++w) {
        Scratch& x = scratch(w);
        float f = 0.f;
        if (used(w)) {
          const float m = -sm.nm[(split ? tcol : w * kAlternate) + cc];
          f = m == M ? 1.f : exp2f(m - M);
          L += f * ((x.red[0][cc] + x.red[1][cc]) + (x.red[2][cc] + x.red[3][cc]));
        }
        x.fac[cc] = f;
      }
      int row = kNoRow;
      if (cc < rows) {
        const int i = (r0 + cc) / a.G;
        row = i * a.Hq + (r0 + cc - i * a.G);
        const bool absent = anc[node[cc]] == 0, empty = absent || L == 0.f;
        if (direct) {
          const float inv = empty ? 0.f : 1.f / L;
#pragma unroll 1
          for (int w = w0; w < w1; ++w) scratch(w).fac[cc] *= inv;
          if (a.lse) a.lse[orow + row] = empty ? -INFINITY : log_sum<T>(M, L);
          if (empty) row = ~row;
        } else {
          a.part_ml[pslot + cc] = make_float2(M, absent ? 0.f : L);  // (0: an empty row)
        }
      }
      so.row[cc] = row;
    }
    if (split && more) rows_ready(sm, 0);  // (its first scores are made while this piece's results go out)
    if (split) named_sync(bar, 128);
    else named_sync(kGroups + 1, kSoft);
    {
      // 16 rows (columns of O^T) at a time, a warp per 32 output columns;
      // shared out over the warpgroups (tiles in turn) and, where O^T repeats
      // itself (D = 64), over the two copies.  Finished rows go through
      // shared memory, transposed, to 64-byte stores.
      constexpr int WD = D / 32;
      const int groups = (split ? 1 : kGroups) * (4 / WD), me = (split ? 0 : wg) * (4 / WD) + warp / WD;
      const int d0 = (warp % WD) * 32;
      char* obase = a.out + 2 * orow * D + 2 * (d0 + (lane & 3) * 8);
      float* pbase = a.part_o + pslot * D + d0 + (lane >> 2);
      char* stage = sc.stage[warp];
      const uint32_t st_at = sptr(stage) + (lane & 7) * 64 + (((lane >> 3) ^ ((lane >> 1) & 3)) << 4);
      const char* ld_at = stage + (lane >> 2) * 64 + (((lane & 3) ^ ((lane >> 3) & 3)) << 4);
#pragma unroll 1
      for (int k = me * 16; k < ncj; k += groups * 16) {
        f32x2 o[2][4];
#pragma unroll
        for (int g = 0; g < 2; ++g)
#pragma unroll
          for (int q = 0; q < 4; ++q) o[g][q] = 0ull;
#pragma unroll 1
        for (int w = w0; w < w1; ++w) {
          if (!used(w)) continue;
          uint32_t u[16];
          tm_ld_frag((split ? tO : tO0 + w * kAlternate) + k, u);
          const float* f = scratch(w).fac + k + x2;
          const f32x2 f0 = *reinterpret_cast<const f32x2*>(f), f1 = *reinterpret_cast<const f32x2*>(f + 8);
          tm_wait_ld(u);
#pragma unroll
          for (int g = 0; g < 2; ++g) {
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              const int i = (q >> 1) * 8 + g * 4 + (q & 1) * 2;
              o[g][q] = fma2(pk2(__uint_as_float(u[i]), __uint_as_float(u[i + 1])), g ? f1 : f0, o[g][q]);
            }
          }
        }
        if (direct) {
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            uint32_t w[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              float x, y;
              up2(o[g][q], x, y);
              w[q] = T::pack(x, y);
            }
            st_matrices_t(st_at + g * 512, w);
          }
          asm volatile("" ::: "memory");
          __syncwarp();
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            int r = so.row[k + g * 8 + (lane >> 2)];
            uint4 w = *reinterpret_cast<const uint4*>(ld_at + g * 512);
            if (r < 0) {  // a row of zeros
              r = ~r;
              w = make_uint4(0, 0, 0, 0);
            }
            if (r != kNoRow) *reinterpret_cast<uint4*>(obase + static_cast<long long>(r) * (2 * D)) = w;
          }
          __syncwarp();
        } else {
#pragma unroll
          for (int g = 0; g < 2; ++g) {
            const int c = k + g * 8 + x2;
            float* at0 = pbase + c * D;
            const bool ok0 = so.row[c] != kNoRow, ok1 = so.row[c + 1] != kNoRow;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              float x, y;
              up2(o[g][q], x, y);
              if (ok0) at0[8 * q] = x;
              if (ok1) at0[D + 8 * q] = y;
            }
          }
        }
      }
      const unsigned long long nf = sm.nf[tb][0] | (static_cast<unsigned long long>(sm.nf[tb][1]) << 32);
      if (nf) {
        if (split) named_sync(bar, 128);
        else named_sync(kGroups + 1, kSoft);
        if (wt < D && wg == w0)
          add_nonfinite<T, D>(a, b, h, ctx, nf, wt, anc, node, so.row, 0, ncj, a.out + 2 * orow * D,
                              direct ? nullptr : a.part_o + pslot * D);
      }
    }
    tc_before();
    named_sync(kGroups + 1, kSoft);  // P and the tables may be written again
    g0 += tiles;
    tails0 += max(end - tail, 0);
    ++item_no;
  }
}

template <class T, int D, int NC>
__global__ void __launch_bounds__(kAttnThreads, 1)
    attn_kernel(const __grid_constant__ CUtensorMap mapk, const __grid_constant__ CUtensorMap mapv,
                const __grid_constant__ Args a) {
  extern __shared__ __align__(1024) char base[];
  constexpr int HALVES = D / 64;
  constexpr int kSlotBytes = HALVES * kHalf;
  char* ring = base;
  char* ringv = ring + a.nk * kSlotBytes;
  char* Q = ringv + a.nv * kSlotBytes;
  const int qbytes = a.cols * D * 2;
  char* P = Q + (a.split ? 1 : 2) * qbytes;
  Misc& sm = *reinterpret_cast<Misc*>(P + a.pbytes);
  const int tid = threadIdx.x, lane = tid & 31;
  // (known to be the same for the warp, so that its role runs with uniform registers)
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int C = gridDim.x, B = a.nodes.B;
  const int per = (B + kAttnThreads - 1) / kAttnThreads;
  if (tid * per < B) asm volatile("prefetch.global.L1 [%0];" ::"l"(a.nodes.ctx_len + tid * per));

  if (tid == 0) {
    for (int i = 0; i < kMaxRing; ++i) {
      bar_init(&sm.kfull[i], 1);
      bar_init(&sm.kempty[i], 1);
      bar_init(&sm.vfull[i], 1);
      bar_init(&sm.vempty[i], 1);
    }
    for (int i = 0; i < 2; ++i) bar_init(&sm.qfull[i], kSoft);
    for (int i = 0; i < kGroups; ++i) {
      bar_init(&sm.sfull[i], 1);
      bar_init(&sm.pfull[i], 128);
      bar_init(&sm.pvdone[i], 1);
    }
    for (int i = 0; i < kTailBars; ++i) bar_init(&sm.vready[i], 1);
    bar_init(&sm.done, 2);
    sm.abort = 0;
    sm.wait_us = a.wait_us;
    sm.b0 = sm.h0 = sm.rb0 = sm.t0 = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(sptr(&sm.tmem))
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  if (warp == 0 && lane == 0) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(&mapk));
    asm volatile("prefetch.tensormap [%0];" ::"l"(&mapv));
  }
  // rows of the ring that no copy writes are zeros (they meet P = 0, and
  // must not be NaN)
  if (a.cover < kTile) {
    for (int i = tid; i < (a.nk + a.nv) * kSlotBytes / 16; i += kAttnThreads)
      reinterpret_cast<uint4*>(ring)[i] = make_uint4(0, 0, 0, 0);
    fence_async();
  }

  // ---- this CTA's range: tiles before each sequence (a block scan over the
  // batch), and where the range starts ----
  {
    const int f = tid * per, e = min(B, f + per);
    const int items = a.Hkv * a.RB;
    long long mine = 0;  // tiles
    int seqs = 0;        // sequences with tiles
    bool any_bad = false;
#pragma unroll 1
    for (int b = f; b < e; ++b) {
      int ctx;
      bool bad;
      const int Tb = tiles_of(a, seq_len(a, b, ctx, bad));
      mine += Tb;
      seqs += Tb > 0;
      any_bad |= bad;
    }
    if (any_bad && blockIdx.x == 0) atomicOr(a.err, kErrBadLength);
    long long inc = mine;
    int inc_seqs = seqs;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long o = __shfl_up_sync(0xffffffffu, inc, d);
      const int os = __shfl_up_sync(0xffffffffu, inc_seqs, d);
      if (lane >= d) {
        inc += o;
        inc_seqs += os;
      }
    }
    constexpr int kWarps = kAttnThreads / 32;
    long long* pre = reinterpret_cast<long long*>(Q);  // not in use yet
    int* pre_seqs = reinterpret_cast<int*>(pre + kWarps);
    if (lane == 31) {
      pre[warp] = inc;
      pre_seqs[warp] = inc_seqs;
    }
    __syncthreads();
    long long before = inc - mine, all = 0;
    int before_seqs = inc_seqs - seqs, all_seqs = 0;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) {
      if (i < warp) {
        before += pre[i];
        before_seqs += pre_seqs[i];
      }
      all += pre[i];
      all_seqs += pre_seqs[i];
    }
    const long long tiles = all * items, n_items = static_cast<long long>(all_seqs) * items;
    // What an item costs beside its tiles (first and last tile, results), in
    // tiles, less where a range is of a few tiles only.
    long long w = 0;  // min(item_cost, tiles / (4 C))
#pragma unroll 1
    for (int k = 1; k <= a.item_cost; ++k) w += tiles >= 4ll * k * C;
    const long long W = tiles + w * n_items;
    // The range's ends in cost: [lo, hi); an item's tiles come first in its
    // T + w.  A range may hold no tile.
    const long long me = blockIdx.x, lo = __umul64hi(W * me, a.per_cta), hi = me + 1 == C ? W : static_cast<long long>(__umul64hi(W * (me + 1), a.per_cta));
    long long p = (before + w * before_seqs) * items;
    const long long mine_cost = (mine + w * seqs) * items;
    if (tid == 0) {
      sm.left = 0;
      a.ranges[me].used = 0;
    }
    __syncthreads();
    // the thread whose sequences hold the range's first tile (lo may lie behind
    // the tiles of the last item before them)
    const bool mine_here = lo < p + mine_cost && hi > p && p - lo <= w;
#pragma unroll 1
    for (int b = f; b < e && mine_here; ++b) {
      const SeqTiles q = seq_tiles(a, b);
      if (q.T == 0) continue;
      const long long one = q.T + w, end = p + one * items;
      if (lo < end) {
        const unsigned long long d = lo > p ? lo - p : 0;
        int item = static_cast<int>((d | one) >> 32 ? d / one : static_cast<unsigned>(d) / static_cast<unsigned>(one));
        int t0 = lo > p ? static_cast<int>(lo - p - item * one) : 0;
        if (t0 >= q.T) {  // behind the item's tiles: the next item
          ++item;
          t0 = 0;
        }
        const long long from = p + item * one + t0;  // cost position of the first tile
        if (item < items) {
          if (from < hi) {
            Range r;
            r.lo = from;
            r.b = sm.b0 = b;
            r.h = sm.h0 = a.RB == 1 ? item : item / a.RB;
            r.rb = sm.rb0 = item - r.h * a.RB;
            r.t0 = sm.t0 = t0;
            r.T = sm.T0 = q.T;
            sm.ctx0 = q.ctx;
            sm.tot0 = q.tot;
            sm.tail0 = q.tail;
            r.used = 1;
            asm volatile("prefetch.global.L1 [%0];" ::"l"(a.table + b * a.table_stride +
                                                           (a.ps <= kTile ? t0 * a.ppt : t0 / a.tpp)));
            a.ranges[me] = r;
            sm.left = hi - from;
          }
          break;
        }
      }
      p = end;
    }
    if (tid == 0) sm.cost = static_cast<int>(w);
  }
  tc_before();
  __syncthreads();
  tc_after();
  pdl_trigger();
  const uint32_t tmem = __shfl_sync(0xffffffffu, sm.tmem, 0);  // (uniform)

  if (warp == 0 || warp == 2) {
    // ---- K (warp 0) or V (warp 2) tiles ----
    const CUtensorMap* map = warp == 0 ? &mapk : &mapv;
    Pieces pc;
    pc.start(sm);
    uint64_t* full = warp == 0 ? sm.kfull : sm.vfull;
    uint64_t* empty = warp == 0 ? sm.kempty : sm.vempty;
    const uint32_t ring0 = sptr(warp == 0 ? ring : ringv);
    const int slots = warp == 0 ? a.nk : a.nv;
    int slot = -1;
    uint32_t phase = 0;
    bool bad_page = false;
#pragma unroll 1
    while (pc.next(a)) {
      const int* trow = a.table + pc.b * a.table_stride;
      const int npages = (pc.tot + a.ps - 1) / a.ps;
      auto lookup = [&](int t) {
        const int p = a.ps <= kTile ? t * a.ppt + lane : t / a.tpp;
        int id = 0;
        if ((a.ps > kTile || lane < a.ppt) && p < npages) {
          id = __ldg(trow + p);
          if (static_cast<unsigned>(id) >= static_cast<unsigned>(a.pages)) {
            bad_page = true;
            id = a.pages;  // out of bounds: zeros
          }
        }
        return id;
      };
      int id = lookup(pc.t0);
#pragma unroll 1
      for (int t = pc.t0; t < pc.end; ++t) {
        const int cur = id;
        if (t + 1 < pc.end) id = lookup(t + 1);
        const int boxes = a.ps <= kTile ? min(a.ppt, npages - t * a.ppt) : 1;
        const int s0 = a.ps <= kTile ? 0 : (t % a.tpp) * kTile;
        // (a page id out of range: a coordinate behind the last)
        const int unit = a.fold ? cur * a.fold + s0 / 8 : cur;
        if (++slot == slots) {
          slot = 0;
          phase ^= 1;
        }
        const bool ok = bar_wait(&empty[slot], phase ^ 1, sm, a.err) &&
                        !*reinterpret_cast<volatile int*>(&sm.abort);
        if (__all_sync(0xffffffffu, ok)) {
          if (lane == 0) bar_expect(&full[slot], boxes * a.box * 128 * HALVES + a.withheld);
          __syncwarp();
          const uint32_t dst = ring0 + slot * kSlotBytes;
#pragma unroll 1
          for (int p0 = 0; p0 < boxes; p0 += 8) {
            int pg[8];
#pragma unroll
            for (int p = 0; p < 8; ++p) pg[p] = __shfl_sync(0xffffffffu, unit, p0 + p);
            if (elect_one()) {
              if (D == 128 && a.fold) {
#pragma unroll
                for (int p = 0; p < 8; ++p)
                  if (p0 + p < boxes) tma_groups(dst + (p0 + p) * a.box * 256, map, pg[p], pc.h, &full[slot]);
              } else {
#pragma unroll
                for (int p = 0; p < 8; ++p) {
                  if (p0 + p < boxes) {
#pragma unroll
                    for (int d = 0; d < HALVES; ++d)
                      tma_rows(dst + (p0 + p) * a.box * 128 + d * kHalf, map, d * 64, s0, pc.h, pg[p], &full[slot]);
                  }
                }
              }
            }
            __syncwarp();
          }
          __syncwarp();
        }
      }
    }
    if (bad_page) atomicOr(a.err, kErrBadPage);
  } else if (warp == 1) {
    // ---- scores (the warp runs as one; one lane issues) ----
    const uint32_t khalf = a.half / 16;
    const uint64_t kd0 = operand(sptr(ring), 16, a.group), qd0 = operand(sptr(Q), 16, 1024);
    const uint32_t qhalf = a.cols * 8;
    Pieces pc;
    pc.start(sm);
    int slot = -1, item = 0, turn = 0;
    uint32_t phase = 0, done = 0;  // done: parity of each warpgroup's jobs; bit 8 + w: it has had one
#pragma unroll 1
    while (pc.next(a)) {
      const int qb = a.split ? 0 : item & 1;
      bar_wait(&sm.qfull[qb], (a.split ? item : item >> 1) & 1, sm, a.err);
      const uint64_t qd = qd0 + qb * (qbytes / 16);
      ++item;
#pragma unroll 1
      for (int t = pc.t0; t < pc.end; ++t) {
        if (++slot == a.nk) {
          slot = 0;
          phase ^= 1;
        }
        bar_wait(&sm.kfull[slot], phase, sm, a.err);
        const uint64_t kd = kd0 + slot * (kSlotBytes / 16);
        const int w0 = a.split ? 0 : turn, w1 = a.split ? kGroups : turn + 1;
#pragma unroll 1
        for (int w = w0; w < w1; ++w) {
          // S of this warpgroup is free once it has made its P of the last one
          if ((done >> (8 + w)) & 1) bar_wait(&sm.pfull[w], ((done >> w) & 1) ^ 1, sm, a.err);
          done = (done ^ (1u << w)) | (256u << w);
          tc_after();
          const uint64_t q = qd + a.off[w] * 8;
          const uint32_t d = tmem + (a.split ? a.off[w] : w * kAlternate);
          const uint32_t id = instr<T>(a.wcols[w], false, false);
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < D / 16; ++k)
              tc_mma(d, kd + (k / 4) * khalf + (k & 3) * 2, q + (k / 4) * qhalf + (k & 3) * 2, id, k > 0);
            tc_commit(&sm.sfull[w]);
            if (w == w1 - 1) tc_commit(&sm.kempty[slot]);
          }
          __syncwarp();
        }
        if (++turn == kGroups) turn = 0;
      }
    }
    if (elect_one()) tc_commit(&sm.done);
    __syncwarp();
    bar_wait(&sm.done, 0, sm, a.err);
  } else if (warp == 3) {
    // ---- values ----
    const uint32_t vstep = a.group / 8;  // 16 slots
    const uint64_t vd0 = operand(sptr(ringv), D == 128 ? a.half : 0, a.group), pd0 = operand(sptr(P), kPBlock, 256, 6);
    Pieces pc;
    pc.start(sm);
    int slot = -1, turn = 0, tails = 0;
    uint32_t phase = 0, ppf = 0;
#pragma unroll 1
    while (pc.next(a)) {
#pragma unroll 1
      for (int t = pc.t0; t < pc.end; ++t) {
        if (++slot == a.nv) {
          slot = 0;
          phase ^= 1;
        }
        bar_wait(&sm.vfull[slot], phase, sm, a.err);
        if (t >= pc.tail) {  // for the warpgroup that clears what must not be multiplied
          if (lane == 0) bar_arrive(&sm.vready[tails % kTailBars]);
          ++tails;
        }
        const uint64_t vd = vd0 + slot * (kSlotBytes / 16);
        const bool add = t - pc.t0 >= (a.split ? 1 : kGroups);  // not the warpgroup's first tile of the piece
        const int w0 = a.split ? 0 : turn, w1 = a.split ? kGroups : turn + 1;
#pragma unroll 1
        for (int w = w0; w < w1; ++w) {
          bar_wait(&sm.pfull[w], (ppf >> w) & 1, sm, a.err);
          ppf ^= 1u << w;
          tc_after();
          const uint64_t pd = pd0 + a.poff[w] / 16;
          const uint32_t d =
              tmem + kMaxRows + (a.split ? a.off[w] : w * kAlternate);
          const uint32_t id = instr<T>(a.wcols[w], true, true);
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < kTile / 16; ++k) tc_mma(d, vd + k * vstep, pd + k * 32, id, add || k > 0);
            tc_commit(&sm.pvdone[w]);
            if (w == w1 - 1) tc_commit(&sm.vempty[slot]);
          }
          __syncwarp();
        }
        if (++turn == kGroups) turn = 0;
      }
    }
    if (elect_one()) tc_commit(&sm.done);
    __syncwarp();
    bar_wait(&sm.done, 0, sm, a.err);
    // sequences without tiles: their rows are empty
#pragma unroll 1
    for (int b = blockIdx.x; b < B; b += C) {
      int ctx;
      bool bad;
      if (seq_len(a, b, ctx, bad) != 0) continue;
      const long long n = static_cast<long long>(a.nodes.N) * a.Hq;
      uint4* o = reinterpret_cast<uint4*>(a.out + 2 * (b * n * D));
      for (long long i = lane; i < n * D / 8; i += 32) o[i] = make_uint4(0, 0, 0, 0);
      if (a.lse)
        for (long long i = lane; i < n; i += 32) a.lse[b * n + i] = -INFINITY;
    }
  } else {
    const int wg = (warp - 4) >> 2;
    softmax_role<T, D, NC>(a, sm, tmem, Q, qbytes, ringv, P, wg);
  }
  tc_before();
  __syncthreads();
  if (warp == 0 && *reinterpret_cast<volatile int*>(&sm.abort)) {
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

// ---------------------------------------------------------------------------
// Joins the parts of the (sequence, head, row block)s that range borders cut:
//     M = max m_i,  w_i = 2^(m_i - M),  o = sum w_i O_i / sum w_i l_i
// in range order.  blockIdx.x: a range that starts inside an item; the first
// such range of an item does its work, a warp per row, four parts' loads on
// their way at a time.  One round trip finds the ranges around it.  (With a
// branch per part, which kept the loads apart, 19 parts took 5.4 us, now 2 us;
// batches of ten took registers from the many short joins of a large batch.)
// ---------------------------------------------------------------------------
constexpr int kJoinWarps = 8;
template <int N>
struct Size {
  static constexpr int value = N;
};

template <class T_, int D>
__global__ void __launch_bounds__(32 * kJoinWarps, 6) attn_combine_kernel(const __grid_constant__ Args a, int C) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const int c = blockIdx.x + 1;
  pdl_wait();
  // ranges c - 1 .. c + 30, a lane each; this one's item
  union {
    uint4 v;
    struct {
      long long lo;
      int t0, used;
    };
  } head;
  head.v = make_uint4(0, 0, 0, 0);
  if (c - 1 + lane < C) head.v = *reinterpret_cast<const uint4*>(a.ranges + c - 1 + lane);
  const int4 item = *(reinterpret_cast<const int4*>(a.ranges + c) + 1);
  const int t0 = __shfl_sync(0xffffffffu, head.t0, 1);
  if (!__shfl_sync(0xffffffffu, head.used, 1) || t0 == 0) return;
  const int b = item.x, h = item.y, rb = item.z, T = item.w;
  const long long s = __shfl_sync(0xffffffffu, head.lo, 1) - t0, e = s + T;
  // the range before, which holds the item's tile t0 - 1
  int pk = c - 1;
  long long before = __shfl_sync(0xffffffffu, head.lo, 0);
  if (!__shfl_sync(0xffffffffu, head.used, 0) && pk > 0) {
    while (--pk > 0 && !a.ranges[pk].used) {}
    before = a.ranges[pk].lo;
  }
  if (before > s) return;  // an earlier range's item
  const int r0 = rb * a.rows_per_block, rows = min(a.rows_per_block, a.R - r0);
  const int r = blockIdx.y * kJoinWarps + (threadIdx.x >> 5);
  if (r >= rows) return;
  // the part of range pk + k; only the first can be its CTA's last
  auto part = [&](int k) { return (2ll * (pk + k) + (k == 0 && before < s ? 1 : 0)) * a.cols + r; };
  const float* const first = a.part_o + part(0) * D + lane * E;
  const float* const rest = a.part_o + 2ll * pk * a.cols * D + r * D + lane * E;  // of range pk + k: + 2 k cols D
  const int step = 2 * a.cols * D;
  float M = kNoScore, L = 0.f, o[E];
#pragma unroll
  for (int q = 0; q < E; ++q) o[q] = 0.f;
#pragma unroll 1
  for (int k0 = 0;; k0 += 32) {
    const int k = k0 + lane, at = pk + k;
    bool in = k == 0, past = at >= C;
    int used;
    long long lo;
    if (k0 > 0 || pk != c - 1) {
      used = !past && a.ranges[at].used;
      lo = used ? a.ranges[at].lo : 0;
    } else {
      used = head.used;
      lo = head.lo;
    }
    if (!in && !past && used) {
      in = lo < e;
      past = !in;
    }
    const float2 ml = in ? a.part_ml[part(k)] : make_float2(kNoScore, 0.f);
    const unsigned parts = __ballot_sync(0xffffffffu, in);
    const int n = parts ? 32 - __clz(parts) : 0;
    float w = 0.f;
    const auto weights = [&]() {
      float m = ml.x;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
      const float Mn = fmaxf(M, m);
      w = in ? (ml.x == Mn ? 1.f : exp2f(ml.x - Mn)) : 0.f;
      float l = w * ml.y;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
      const float old = M == Mn ? 1.f : exp2f(M - Mn);
      L = L * old + l;
      M = Mn;
#pragma unroll
      for (int q = 0; q < E; ++q) o[q] *= old;
    };
    // kBatch parts' loads on their way at a time
    const auto batch = [&](int t, auto size) {
      constexpr int kBatch = decltype(size)::value;
      float v[kBatch][E];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const bool have = t + i < 32 && (parts >> ((t + i) & 31)) & 1;
        const float* src = i == 0 && k0 + t == 0 ? first : rest + (k0 + t + i) * step;
#pragma unroll
        for (int q = 0; q < E; q += 2) {
          const float2 x = have ? *reinterpret_cast<const float2*>(src + q) : make_float2(0.f, 0.f);
          v[i][q] = x.x;
          v[i][q + 1] = x.y;
        }
      }
      if (t == 0) weights();  // (the loads of both are on their way)
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const float wt = __shfl_sync(0xffffffffu, w, (t + i) & 31);
#pragma unroll
        for (int q = 0; q < E; ++q) o[q] = fmaf(wt, v[i][q], o[q]);
      }
    };
    if (n <= 2) {
      batch(0, Size<2>{});
    } else {
#pragma unroll 1
      for (int t = 0; t < n; t += 4) batch(t, Size<4>{});
    }
    if (__any_sync(0xffffffffu, past)) break;
  }
  const int i = (r0 + r) / a.G, g = r0 + r - i * a.G;
  const bool empty = L == 0.f;
  const float inv = empty ? 0.f : 1.f / L;
  const long long row = (static_cast<long long>(b) * a.nodes.N + i) * a.Hq + h * a.G + g;
  char* out = a.out + 2 * (row * D + lane * E);
#pragma unroll
  for (int q = 0; q < E; q += 2)
    *reinterpret_cast<uint32_t*>(out + 2 * q) = empty ? 0u : T_::pack(o[q] * inv, o[q + 1] * inv);
  if (a.lse && lane == 0) a.lse[row] = empty ? -INFINITY : log_sum<T_>(M, L);
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
typedef CUresult (*EncodeFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                             const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                             CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
  static const EncodeFn fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &r) !=
            cudaSuccess ||
        r != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeFn>(p);
  }();
  return fn;
}

CUtensorMapDataType map_type(int dtype) {
  return dtype == Bf16::kId ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
}

// {D, page_size, Hkv, pages}; boxes of 64 columns and `box` slots of one head
// of one page.
bool encode_rows(CUtensorMap* m, void* base, int dtype, int D, int ps, int H, int pages, long long slot,
                 long long head, long long page, int box) {
  const EncodeFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(ps),
                              static_cast<cuuint64_t>(H), static_cast<cuuint64_t>(pages)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(slot) * 2, static_cast<cuuint64_t>(head) * 2,
                                 static_cast<cuuint64_t>(page) * 2};
  const cuuint32_t bx[4] = {64, static_cast<cuuint32_t>(box), 1, 1};
  const cuuint32_t one[4] = {1, 1, 1, 1};
  return fn(m, map_type(dtype), 4, base, dims, strides, bx, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Groups of 8 slots a page apart, where the cache's strides make the slots of
// all pages one sequence of such groups; 0 where they don't, or where a tile
// could run over a page's end.
long long page_groups(int ps, int pages, long long slot, long long page) {
  if (ps % 8 != 0 || (ps > kTile && ps % kTile != 0) || (ps < kTile && kTile % ps != 0)) return 0;
  if (page % (8 * slot) != 0) return 0;
  const long long g = page / (8 * slot);
  return g >= ps / 8 && g * (pages + 1ll) < (1ll << 31) ? g : 0;
}

// {64, 8 slots, 2 halves, groups, Hkv}; boxes of `box` slots.
bool encode_groups(CUtensorMap* m, void* base, int dtype, int ps, int H, int pages, long long slot, long long head,
                   long long groups, int box) {
  const EncodeFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[5] = {64, 8, 2, static_cast<cuuint64_t>(groups * (pages - 1) + ps / 8),
                              static_cast<cuuint64_t>(H)};
  const cuuint64_t strides[4] = {static_cast<cuuint64_t>(slot) * 2, 128, static_cast<cuuint64_t>(slot) * 16,
                                 static_cast<cuuint64_t>(head) * 2};
  const cuuint32_t bx[5] = {64, 8, 2, static_cast<cuuint32_t>(box / 8), 1};
  const cuuint32_t one[5] = {1, 1, 1, 1, 1};
  return fn(m, map_type(dtype), 5, base, dims, strides, bx, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Shape {
  int RB, rows, split, cols, width[kGroups], off[kGroups], poff[kGroups], pbytes;
};
Shape shape_of(int R) {
  Shape s;
  s.RB = (R + kMaxRows - 1) / kMaxRows;
  s.rows = (R + s.RB - 1) / s.RB;
  s.split = s.rows > kAlternate;
  const int units = (s.rows + 15) / 16;
  s.cols = units * 16;
  s.pbytes = 0;
  int off = 0;
  for (int w = 0; w < kGroups; ++w) {
    const int mine = s.split ? units / kGroups + (w < units % kGroups) : units;
    s.width[w] = mine * 16;
    s.off[w] = off;
    if (s.split) off += mine * 16;
    s.poff[w] = s.pbytes;
    const int p = mine * kPBlock;
    s.pbytes += p > kPMin ? p : kPMin;
  }
  return s;
}

struct Layout {
  size_t ranges, ml, o, total;
};
Layout layout_of(int R, int D) {
  const Shape s = shape_of(R);
  Layout L;
  L.ranges = 256;
  L.ml = (L.ranges + sizeof(Range) * kMaxCtas + 255) / 256 * 256;
  L.o = (L.ml + 8ull * 2 * kMaxCtas * s.cols + 255) / 256 * 256;
  L.total = L.o + 4ull * 2 * kMaxCtas * s.cols * D;
  return L;
}

int sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess ||
      cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
    return 0;
  return n;
}

template <class T, int D, int NC>
cudaError_t launch_t(const CUtensorMap& mk, const CUtensorMap& mv, const Args& a, int C, size_t smem,
                     cudaStream_t s) {
  cudaError_t e = cudaFuncSetAttribute(attn_kernel<T, D, NC>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
  if (e != cudaSuccess) return e;
  attn_kernel<T, D, NC><<<C, kAttnThreads, smem, s>>>(mk, mv, a);
  e = cudaGetLastError();
  if (e != cudaSuccess || C < 2) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(C - 1, (a.rows_per_block + kJoinWarps - 1) / kJoinWarps);
  cfg.blockDim = dim3(32 * kJoinWarps);
  cfg.stream = s;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attn_combine_kernel<T, D>, a, C);
}

template <class T, int D>
cudaError_t launch_d(const CUtensorMap& mk, const CUtensorMap& mv, const Args& a, int C, size_t smem,
                     cudaStream_t s) {
  if (a.wcols[0] <= 32) return launch_t<T, D, 32>(mk, mv, a, C, smem, s);
  if (a.wcols[0] <= 64) return launch_t<T, D, 64>(mk, mv, a, C, smem, s);
  return launch_t<T, D, 96>(mk, mv, a, C, smem, s);
}

}  // namespace

size_t tree_attention_bytes(int N, int G, int D) { return layout_of(N * G, D).total; }

cudaError_t launch_tree_attention(const AttnParams& p, int dtype, int D, cudaStream_t s) {
  Args a;
  a.nodes = p.nodes;
  a.table = p.kv.table;
  a.table_stride = p.kv.table_stride;
  a.width = p.kv.width; a.pages = p.kv.pages; a.ps = p.kv.ps;
  a.Hq = p.Hq; a.Hkv = p.kv.Hkv; a.G = p.G; a.R = p.nodes.N * p.G;
  const Shape sh = shape_of(a.R);
  a.RB = sh.RB; a.rows_per_block = sh.rows; a.split = sh.split; a.cols = sh.cols;
  for (int w = 0; w < kGroups; ++w) {
    a.wcols[w] = sh.width[w];
    a.off[w] = sh.off[w];
    a.poff[w] = sh.poff[w];
  }
  a.pbytes = sh.pbytes;
  // About 5 us of the pass's time.  Measured at 4, 6, 8, 10 tiles: 64 single tokens
  // over 200..6000 slots, D = 64, 73.0, 66.3, 63.4, 65.5 us, D = 128, 83.6, 85.4,
  // 86.8, 88.0; 64 chains of 32 rows, D = 128, 89.6, 90.3, 93.1, 95.9; 32 trees of 64
  // rows, D = 128, 72.2, 63.3, 63.3, 63.4; 64 trees of 168 rows, D = 128, 208.6, 197.0,
  // 202.1, 209.4, D = 64, 195.5, 189.1, 193.5, 202.1; 32 trees of 128 rows, D = 64, 79.4,
  // 78.7, 78.7, 78.7; 32 trees of 256 rows, D = 128, 164.5, 162.3, 170.7, 172.8.
  a.item_cost = D == 64 && !a.split ? 8 : 6;
  a.q = p.q; a.q_b = p.q_b; a.q_n = p.q_n; a.q_h = p.q_h;
  a.zero = p.scale == 0.f;
  a.c = a.zero ? 1.f : p.scale * 1.4426950408889634f;
  a.out = p.out; a.lse = p.lse;
  a.vcache = p.kv.v; a.v_page = p.kv.v_page; a.v_slot = p.kv.v_slot; a.v_head = p.kv.v_head;
  a.err = p.err;
  a.wait_us = p.wait_us; a.withheld = p.withheld;
  const Layout L = layout_of(a.R, D);
  char* ws = reinterpret_cast<char*>(p.err);
  a.ranges = reinterpret_cast<Range*>(ws + L.ranges);
  a.part_ml = reinterpret_cast<float2*>(ws + L.ml);
  a.part_o = reinterpret_cast<float*>(ws + L.o);
  // tiles: whole pages up to 128 slots; boxes of a multiple of 8 rows (the
  // swizzle's period), what exceeds the page filled with zeros
  if (a.ps <= kTile) {
    a.box = (a.ps + 7) / 8 * 8;
    a.ppt = kTile / a.box;
    if (a.ppt > 32) a.ppt = 32;
    a.tk = a.ppt * a.ps;
    a.tpp = 1;
    a.cover = a.ppt * a.box;
    a.ragged = a.tk != kTile;
  } else {
    a.box = kTile;
    a.ppt = 1;
    a.tk = kTile;
    a.tpp = (a.ps + kTile - 1) / kTile;
    a.cover = kTile;
    a.ragged = a.ps % kTile != 0;
  }
  const int slot = D * 2 * kTile;
  const size_t qb = static_cast<size_t>(a.cols) * D * 2;
  const size_t fixed = (a.split ? 1 : 2) * qb + a.pbytes + sizeof(Misc);
  int slots = static_cast<int>((kSmemMax - fixed) / slot);
  if (slots > 2 * kMaxRing) slots = 2 * kMaxRing;
  if (slots < 3) return cudaErrorInvalidConfiguration;
  // (an odd slot to K: a product of scores frees its K tile at once, but the next
  // one is wanted a softmax earlier than the next V tile.  Two wide trees, three
  // slots: 235 us, with two for V 244)
  a.nk = (slots + 1) / 2;
  a.nv = slots - a.nk;
  const size_t smem = fixed + static_cast<size_t>(slots) * slot;
  CUtensorMap mk, mv;
  const KvView& kv = p.kv;
  const long long gk = page_groups(a.ps, a.pages, kv.k_slot, kv.k_page);
  const long long gv = page_groups(a.ps, a.pages, kv.v_slot, kv.v_page);
  // One copy per page brings both halves of D = 128 (two copies of 2 KB of a
  // page of 16 took the loader 80 cycles each, more than the copies' share of
  // the memory's time).
  a.fold = D == 128 && gk == gv ? static_cast<int>(gk) : 0;
  a.group = a.fold ? 2048 : 1024;
  a.half = a.fold ? 1024 : kHalf;
  const bool ok =
      a.fold ? encode_groups(&mk, kv.k, dtype, a.ps, a.Hkv, a.pages, kv.k_slot, kv.k_head, gk, a.box) &&
                   encode_groups(&mv, kv.v, dtype, a.ps, a.Hkv, a.pages, kv.v_slot, kv.v_head, gv, a.box)
             : encode_rows(&mk, kv.k, dtype, D, a.ps, a.Hkv, a.pages, kv.k_slot, kv.k_head, kv.k_page, a.box) &&
                   encode_rows(&mv, kv.v, dtype, D, a.ps, a.Hkv, a.pages, kv.v_slot, kv.v_head, kv.v_page, a.box);
  if (!ok) return cudaErrorInvalidValue;
  int C = sm_count();
  if (C < 1) return cudaErrorInvalidDevice;
  C = C < kMaxCtas ? C : kMaxCtas;
  a.per_cta = C > 1 ? ~0ull / C + 1 : 0;
  if (dtype == Bf16::kId)
    return D == 128 ? launch_d<Bf16, 128>(mk, mv, a, C, smem, s) : launch_d<Bf16, 64>(mk, mv, a, C, smem, s);
  return D == 128 ? launch_d<F16, 128>(mk, mv, a, C, smem, s) : launch_d<F16, 64>(mk, mv, a, C, smem, s);
}

}  // namespace ssd

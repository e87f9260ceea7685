// ssd_tiles.cuh -- a paged cache as tiles of up to 128 slots for the tensor cores: where a
// slot lies, copies of a tile, and the queries' copies.
#pragma once

#include "ssd_tc.cuh"

namespace ssd {

struct PageTiles {
  const int* table;
  long long table_stride;
  int width, pages, ps;
  int box, boxes;          // rows of a TMA box, boxes of a tile
  int step, tk;            // slots of a box, of a tile
  int tpp;                 // (uneven) tiles a page
  int fold;                // copies of whole groups of 8 slots: groups a page (0: rows of 64-column halves)
  int group, half;         // bytes from 8 slots of a tile to the next, from half to half
  int holes;               // tiles have rows that are no slot, the same in each
  int uneven;              // tiles that differ: a page's tiles of 128 slots and a rest
  int gather;              // boxes of four slots by their rows' numbers (0, or the rows there are)
  int g_page, g_head, g_x; // rows a page, rows a head, columns a head
};

constexpr int kFar = 1 << 30;  // offset of a row that is no slot

__device__ __forceinline__ int tile_of(const PageTiles& a, int slot) {
  if (a.uneven) return (slot / a.ps) * a.tpp + (slot % a.ps) / kTile;
  return a.tk == kTile ? slot / kTile : slot / a.tk;
}
// First slot of tile t, and how many it holds.
__device__ __forceinline__ void tile_slots(const PageTiles& a, int t, int& first, int& count) {
  if (!a.uneven) {
    first = t * a.tk;
    count = a.tk;
  } else {
    const int r = (t % a.tpp) * kTile;
    first = (t / a.tpp) * a.ps + r;
    count = min(kTile, a.ps - r);
  }
}

// Offset of a tile's row from its first slot (uneven: a slot's below the tile's count).
__device__ __forceinline__ int row_offset(const PageTiles& a, int row) {
  if (!a.holes) return row;
  const int p = row / a.box, r = row - p * a.box;
  return p < a.boxes && r < a.ps ? p * a.ps + r : kFar;
}

// This lane's box of a tile: its page (gather: its four slots' pages) and first slot there.
struct Place {
  int id[4], s0;
};
// Of tile t, where the box is wanted; `last` is the sequence's last slot (or the item's).
// (GATHER: kernels of their own, as the other copies slow down by up to a tenth beside it.)
template <bool GATHER>
__device__ __forceinline__ Place box_place(const PageTiles& a, const int* trow, int t, int last, bool wanted) {
  Place x = {};
  if (a.uneven) {
    x.s0 = (t % a.tpp) * kTile;
    if (wanted) x.id[0] = __ldg(trow + t / a.tpp);
    return x;
  }
  const unsigned slot = static_cast<unsigned>(t) * a.tk + (threadIdx.x & 31) * a.step, p = slot / a.ps;
  x.s0 = slot - p * a.ps;
  if (wanted) {
    x.id[0] = __ldg(trow + p);
    if (GATHER) {  // (behind the last slot: its page again)
#pragma unroll
      for (int i = 1; i < 4; ++i) x.id[i] = __ldg(trow + min(slot + i, static_cast<unsigned>(last)) / a.ps);
    }
  }
  return x;
}

// Whether this lane's box of tile t has a page id out of range at a slot that somebody sees: of
// those up to `last` the ones before sk and from lo on (other entries of a table may be
// anything).
template <bool GATHER>
__device__ __forceinline__ bool bad_box(const PageTiles& a, const int* trow, int t, int last, int lo, int sk) {
  const int lane = threadIdx.x & 31;
  int first, count;
  tile_slots(a, t, first, count);
  if (!a.uneven) {
    first += lane * a.step;
    count = a.step;
  }
  if (lane >= a.boxes || first > last) return false;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < (GATHER ? 4 : 1); ++i) {
    const int s = min(first + i, last), end = GATHER ? s + 1 : first + count;  // (in one page)
    bad |= (s < sk || end > lo) && static_cast<unsigned>(__ldg(trow + s / a.ps)) >= static_cast<unsigned>(a.pages);
  }
  return bad;
}

__device__ __forceinline__ int seq_tokens(const PageTiles& a, const NodesView& nodes, int b, int& ctx, bool& bad) {
  ctx = __ldg(nodes.ctx_len + b);
  const int nn = nodes.n_nodes ? __ldg(nodes.n_nodes + b) : nodes.N;
  return seq_nodes(ctx, nn, nodes.N, a.width, a.ps, bad);
}

// ---------------------------------------------------------------------------
// copies
// ---------------------------------------------------------------------------
// A ring's next tile: boxes p0 .. p1.  False where this lane's has a page id out of range.
struct Ring {
  const CUtensorMap* map;
  uint64_t *full, *empty;
  uint32_t base;
  int slots, slot;
  uint32_t phase;
};
template <int D, bool GATHER, class Misc>
__device__ __forceinline__ bool load_tile(const PageTiles& a, Misc& sm, Ring& r, int p0, int p1, const Place& x, int h,
                                          int* err, int withheld) {
  constexpr int HALVES = D / 64, kSlotBytes = HALVES * kHalf;
  const int lane = threadIdx.x & 31;
  bool good = static_cast<unsigned>(x.id[0]) < static_cast<unsigned>(a.pages);
  const int id = good ? x.id[0] : a.pages;  // out of bounds: zeros
  const int s0 = x.s0, unit = a.fold ? id * a.fold + s0 / 8 : id;
  if (GATHER) {
#pragma unroll
    for (int i = 1; i < 4; ++i) good = good && static_cast<unsigned>(x.id[i]) < static_cast<unsigned>(a.pages);
  }
  if (++r.slot == r.slots) {
    r.slot = 0;
    r.phase ^= 1;
  }
  uint64_t* full = r.full + r.slot;
  const bool ok = bar_await(r.empty + r.slot, r.phase ^ 1, sm, err) && !*reinterpret_cast<volatile int*>(&sm.abort);
  if (!__all_sync(0xffffffffu, ok)) return true;
  if (lane == 0) bar_expect(full, (p1 - p0 + 1) * a.box * 128 * HALVES + withheld);
  __syncwarp();
  const uint32_t dst = r.base + r.slot * kSlotBytes;
  // a lane a box
  if (lane >= p0 && lane <= p1) {
    if constexpr (GATHER) {
      int row[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        row[i] = static_cast<unsigned>(x.id[i]) < static_cast<unsigned>(a.pages)
                     ? x.id[i] * a.g_page + (s0 + i) % a.ps + h * a.g_head
                     : a.gather;
#pragma unroll
      for (int d = 0; d < HALVES; ++d)
        tma_gather(dst + lane * 512 + d * kHalf, r.map, h * a.g_x + d * 64, row, full);
    } else if (D == 128 && a.fold) {
      tma_groups(dst + lane * a.box * 256, r.map, unit, h, full);
    } else {
#pragma unroll
      for (int d = 0; d < HALVES; ++d)
        tma_rows(dst + lane * a.box * 128 + d * kHalf, r.map, d * 64, s0, h, unit, full);
    }
  }
  __syncwarp();
  return good || lane < p0 || lane > p1;
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
// Where slots of any pages are rows of one matrix, `slot` elements apart: rows a page, rows
// and columns a head, the matrix's size.
struct RowsOf {
  long long page, head, x, columns, rows;
};
inline bool rows_of(RowsOf& g, int ps, int H, int pages, int D, long long slot, long long head, long long page) {
  if (page % slot != 0) return false;
  g.page = page / slot;
  g.head = g.x = 0;
  if (H > 1) {
    if (head % slot == 0) g.head = head / slot;
    else if (head * (H - 1) + D <= slot) g.x = head;
    else return false;
  }
  g.columns = g.x * (H - 1) + D;
  g.rows = g.page * (pages - 1ll) + g.head * (H - 1ll) + ps;
  return g.page < (1ll << 31) && g.head < (1ll << 31) && g.rows < (1ll << 31) - 1;
}

// The cache's tiles and its maps (mv may be null).
inline bool page_tiles(PageTiles& a, const KvView& kv, int dtype, int D, CUtensorMap* mk, CUtensorMap* mv) {
  a.table = kv.table;
  a.table_stride = kv.table_stride;
  a.width = kv.width; a.pages = kv.pages; a.ps = kv.ps;
  // Tiles of 128 slots from boxes that lie in one page: of the largest power of two that
  // divides the page, at least 8 (the swizzle's period).  Other pages (1, 5, 201): up to 128
  // slots whole pages, what a box of a multiple of 8 rows exceeds them by filled with zeros;
  // above that a page's tiles of 128 and a rest.  Pages of up to 3 slots, which would leave a
  // tile more than half empty: four slots at a time by their rows' numbers, where the cache's
  // strides make all slots rows of one matrix.  (Boxes of parts of pages against
  // whole pages, 4096 tokens at 4000, 32 / 8 heads of 64: pages of 24 336 us against 342,
  // of 48 260 against 409, of 200 336 against 434; 64 single tokens at 4000: 178 us against
  // 186, 198, 234.  Rows by their numbers against whole pages: pages of 1 685 us against 2550
  // and 335 against 1278; of 5 686 against 546 and 334 against 281.)
  a.box = kTile;
  while (a.ps % a.box != 0) a.box /= 2;
  a.holes = a.uneven = a.gather = a.g_page = a.g_head = a.g_x = 0;
  a.step = a.box;
  a.boxes = kTile / a.box;
  a.tk = kTile;
  a.tpp = 1;
  RowsOf gk_rows, gv_rows;
  if (a.ps <= 3 && rows_of(gk_rows, a.ps, kv.Hkv, a.pages, D, kv.k_slot, kv.k_head, kv.k_page) &&
      (!mv || (rows_of(gv_rows, a.ps, kv.Hkv, a.pages, D, kv.v_slot, kv.v_head, kv.v_page) &&
               gv_rows.page == gk_rows.page && gv_rows.head == gk_rows.head && gv_rows.x == gk_rows.x))) {
    a.box = a.step = 4;
    a.boxes = kTile / 4;
    a.gather = static_cast<int>(gk_rows.rows);
    a.g_page = static_cast<int>(gk_rows.page);
    a.g_head = static_cast<int>(gk_rows.head);
    a.g_x = static_cast<int>(gk_rows.x);
    a.fold = 0;
    a.group = 1024;
    a.half = kHalf;
    return encode_gather(mk, kv.k, dtype, gk_rows.columns, gk_rows.rows, kv.k_slot) &&
           (!mv || encode_gather(mv, kv.v, dtype, gv_rows.columns, gv_rows.rows, kv.v_slot));
  }
  if (a.box < 8) {
    a.uneven = a.ps > kTile;
    a.holes = !a.uneven;
    a.box = a.uneven ? kTile : (a.ps + 7) / 8 * 8;
    a.boxes = kTile / a.box;
    a.step = a.uneven ? kTile : a.ps;
    a.tk = a.boxes * a.step;
    a.tpp = (a.ps + kTile - 1) / kTile;
  }
  const int whole = a.holes || a.uneven ? 0 : a.box;
  const long long gk = page_groups(a.ps, a.pages, kv.k_slot, kv.k_page, whole);
  const long long gv = mv ? page_groups(a.ps, a.pages, kv.v_slot, kv.v_page, whole) : gk;
  a.fold = D == 128 && gk == gv ? static_cast<int>(gk) : 0;
  a.group = a.fold ? 2048 : 1024;
  a.half = a.fold ? 1024 : kHalf;
  const auto encode = [&](CUtensorMap* m, void* base, long long slot, long long head, long long page, long long groups) {
    return a.fold ? encode_groups(m, base, dtype, a.ps, kv.Hkv, a.pages, slot, head, groups, a.box)
                  : encode_rows(m, base, dtype, D, a.ps, kv.Hkv, a.pages, slot, head, page, a.box);
  };
  return encode(mk, kv.k, kv.k_slot, kv.k_head, kv.k_page, gk) &&
         (!mv || encode(mv, kv.v, kv.v_slot, kv.v_head, kv.v_page, gv));
}

// {D, Hq, N, B}; boxes of 64 columns, G heads and tq tokens.
inline bool encode_queries(CUtensorMap* m, const char* q, long long q_b, long long q_n, long long q_h, int Hq,
                           const NodesView& nodes, int G, int dtype, int D, int tq) {
  const EncodeFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(D), static_cast<cuuint64_t>(Hq),
                              static_cast<cuuint64_t>(nodes.N), static_cast<cuuint64_t>(nodes.B)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(q_h) * 2, static_cast<cuuint64_t>(q_n) * 2,
                                 static_cast<cuuint64_t>(q_b) * 2};
  const cuuint32_t bx[4] = {64, static_cast<cuuint32_t>(G), static_cast<cuuint32_t>(tq), 1};
  const cuuint32_t one[4] = {1, 1, 1, 1};
  return fn(m, map_type(dtype), 4, const_cast<char*>(q), dims, strides, bx, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace ssd

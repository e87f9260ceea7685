// ssd_chunk.cu -- attention of chunks of new tokens over the paged cache.
//
// Token i of a sequence lies in slot p = ctx + i and sees the slots s <= p with
// s > p - window (window 0: all of them) or s < sinks:
//     out = sum_s softmax_s(c q k_s) v_s,   lse = log sum_s exp(c q k_s).
//
// For one key/value head the rows are the (token, query head of the group) pairs, G
// heads a token.  A row tile is 128 / G whole tokens, 128 rows at most, on the tensor
// cores' M axis; over tiles of 128 slots
//     S = Q K^T  [rows, slots],   P = 2^(c S - m) masked,   O += P V  [rows, D]
// with Q, K and V in shared memory and S, P and O in tensor memory: a thread of the
// softmax owns a row, reads its scores, and writes P over them as the next product's
// operand, so that nothing of S or P passes shared memory and no row needs another
// thread.
//
// An item is a (sequence, block of tokens, key/value head): two row tiles side by side
// (chunks of more than one row tile), whose softmax and products alternate, or one
// (short chunks), whose tiles alternate between two score buffers, or the few rows of
// short chunks of heads of 64 as copies.  Of the slots it takes the tiles that hold first
// tokens, then those from the window's begin to the block's last token.  One persistent
// CTA per SM: the batch's tiles are numbered and cut into equal ranges by the lengths on
// the device, an item's start and end counted as some tiles; an item that is cut leaves
// its parts (m, l, O in 32 bits) in the workspace, and chunk_join_kernel joins them in
// range order (the same bits every call).
//
// Warps of a CTA:
//   0      copies K and V tiles, a lane a box, by TMA into rings of slots (one row tile: K,
//          and warp 2 V)
//   1, 2   issue the products, of a row tile each (one row tile: warp 1)
//   3      copies Q, and clears what must not be multiplied in V tiles at the edges of
//          what is seen: rows that no row of the item sees, and NaN or infinite entries
//          of slots that only some see (added at the end for the rows that see them)
//   4..11  two warpgroups for the softmax: one for each row tile; or (one row tile) one for
//          every second item, so that an item's end runs beside the next one's begin; or
//          (copies) one for every second tile
//
// m follows the running maximum lazily: only where a row's maximum in units of log 2
// grew by more than 8 are l and O rescaled.  P at m is 2^-40 in bf16, so that sums of
// finite values stay finite, and 2^7 in fp16, whose V ends at 65504 and whose P at
// 2^16.  P is rounded to the cache's type, which the product's operands share; scores, m,
// l and O are held in 32 bits, and l adds the weights before they are rounded.
//
// What bounds it: long chunks, the chain of a row tile's scores, softmax (1400 cycles),
// weights and products, of which the two row tiles overlap 2800 cycles a pair of tiles
// (products of heads of 128: 2048): a prompt of 8192 tokens, 64 / 8 heads of 128, 840 us
// (1310 TFLOP/s, at the GPU's power limit).  Single tokens, the copies: 64 at 6800 slots,
// 64 / 8 heads of 128, 279 us (6.4 TB/s).  Few slots, latency: a chain of 8 under a window
// of 4096 24 us, of which 7 until the first scores, 3 to end an item and 6 to join parts.
#include <math.h>

#include "ssd_device.cuh"
#include "ssd_kv.cuh"
#include "ssd_tiles.cuh"

namespace ssd {
namespace {

// One row tile, two, or one with copies of its rows.
enum { kOne, kTwo, kCopies };
constexpr int kThreads = 384;
constexpr int kRegsCopy = 88, kRegsSoft = 208;  // 128 x 88 + 256 x 208 = 384 x 168
constexpr int kMaxRing = 6;
constexpr int kMaxCtas = 160;
constexpr int kEdgeBars = 8;   // edge tiles whose clearing may lie ahead of their products
constexpr int kFlagSets = 8;   // items whose flags live side by side
constexpr int kStage = 2 * kTile * 128;  // 32 columns of O of the copies
constexpr float kNoScore = -1e30f;  // m of a row that has seen nothing
constexpr float kGrow = 8.f;
template <class T>
constexpr float kLift = T::kId == Bf16::kId ? -40.f : 7.f;  // log2 of P at m

// A CTA's range of tiles, for the joining kernel.
struct alignas(16) Range {
  long long lo;       // first tile (its position in cost)
  int t0, used;       // its place in its item; 0: a range without tiles
  int b, blk, h, T;   // its item, the item's tiles
};

struct Args : PageTiles {
  NodesView nodes;
  int Hq, Hkv, G;
  int tq, tpi;             // tokens of a row tile, of an item
  int copies;              // of the rows in a row tile (1, 2, 4)
  int NB;                  // blocks of the longest chunk
  int window, sinks;
  int item_cost;           // what an item's start and end cost, in tiles
  int nk, nv;              // slots of the K and V rings
  float c;                 // |scale| * log2(e)
  int negate;              // scale < 0: the scores' products are negated
  int zero;                // scale 0: Q counts as zeros (and c as 1)
  char* out;
  float* lse;
  const char* vcache;      // for the rows that see a slot with NaN or infinities
  long long v_page, v_slot, v_head;
  float* part_o;           // [2 ctas][tpi * G][D]
  float2* part_ml;         // [2 ctas][tpi * G]
  Range* ranges;           // [ctas]
  unsigned long long per_cta;  // 2^64 / ctas, rounded up
  int* err;
  unsigned wait_us;
  int withheld;
};

// What tokens p0 .. p1 (slots) see together: slots < sk and lo .. p1.
struct Seen {
  int p0, p1, lo, sk;
};
// The tiles of a block: nsk of first tokens, then those from ft on; T in all.  Each of
// its tokens sees every slot of tiles f0 .. f1 - 1; the others are its edges.
struct Block {
  int T, nsk, ft, f0, f1;
  __device__ __forceinline__ bool edge(int t) const { return t < f0 || t >= f1; }
};
struct alignas(16) Misc {
  uint64_t kfull[kMaxRing], kempty[kMaxRing], vfull[kMaxRing], vempty[kMaxRing];
  uint64_t turn[2], qfull[2], qempty[2], sfull[2][2], pfull[2][2], pvdone[2], ofree[2], vready[kEdgeBars], done;
  long long left;
  int b0, blk0, h0, t0;       // first piece
  int ctx0, n0;
  Seen s0;
  Block k0;
  int cost;                   // of an item beside its tiles
  int pad;                    // some sequence has fewer tokens than N
  unsigned tmem;
  int abort;
  unsigned wait_us;
  float sums[kTile / 2];   // l of an item's rows (copies)
  unsigned flags[kFlagSets][16];  // slots with NaN or infinite values that some rows see
  alignas(16) int off[kTile]; // offset of a tile's row from its first slot; far: no slot
  unsigned plain[4];          // rows of a tile that are slots (pages of up to 128)
  long long scan[2][kThreads / 32];
};
static_assert(sizeof(Misc) <= 3 * 1024, "shared memory beside rings and Q");

// ---------------------------------------------------------------------------
// tiles, blocks, pieces
// ---------------------------------------------------------------------------
__device__ __forceinline__ Seen seen_by(const Args& a, int p0, int p1) {
  Seen s;
  s.p0 = p0;
  s.p1 = p1;
  s.lo = a.window ? max(0, p0 - a.window + 1) : 0;
  s.sk = min(a.sinks, s.lo);
  return s;
}
// Whether they see some of the slots first .. last, and whether each sees all.
__device__ __forceinline__ bool some(const Seen& s, int first, int last) {
  return first <= s.p1 && (last >= s.lo || first < s.sk);
}
__device__ __forceinline__ bool all(const Args& a, const Seen& s, int first, int last) {
  return last <= s.p0 && (a.window == 0 || first > s.p1 - a.window || last < a.sinks);
}

__device__ __forceinline__ Block block_of(const Args& a, const Seen& s) {
  Block k;
  k.ft = s.lo > 0 ? tile_of(a, s.lo) : 0;
  k.nsk = s.sk > 0 ? min(tile_of(a, s.sk - 1) + 1, k.ft) : 0;
  k.T = k.nsk + tile_of(a, s.p1) - k.ft + 1;
  const int low = a.window ? max(0, s.p1 - a.window + 1) : 0;
  k.f0 = low > 0 ? tile_of(a, low - 1) + 1 : 0;
  k.f1 = a.uneven ? 0 : tile_of(a, s.p0 + 1);
  return k;
}
__device__ __forceinline__ Seen block_seen(const Args& a, int ctx, int n, int blk) {
  const int i0 = blk * a.tpi;
  return seen_by(a, ctx + i0, ctx + min(n, i0 + a.tpi) - 1);
}

// The pieces of a CTA's range, one item after another.  Only the first may start
// behind its item's tile 0.
struct Pieces {
  long long left;  // cost from t0 to the range's end: a tile 1, an item's end w
  int w, b, blk, h, ctx, n;
  Seen s;
  Block k;
  int t0, end;     // tiles t0 .. end - 1
  bool fresh;
  __device__ __forceinline__ void load(const Args& a) {
    s = block_seen(a, ctx, n, blk);
    k = block_of(a, s);
  }
  __device__ __forceinline__ void start(const Misc& sm) {
    left = sm.left;
    w = sm.cost;
    b = sm.b0;
    blk = sm.blk0;
    h = sm.h0;
    t0 = sm.t0;
    fresh = true;
    ctx = sm.ctx0;
    n = sm.n0;
    s = sm.s0;
    k = sm.k0;
  }
  __device__ __forceinline__ bool direct() const { return t0 == 0 && end == k.T; }
  __device__ __forceinline__ int tile(int i) const { return i < k.nsk ? i : k.ft + i - k.nsk; }
  __device__ __forceinline__ bool next(const Args& a) {
    if (!fresh) {
      left -= end - t0 + (end == k.T ? w : 0);
      t0 = 0;
      if (left > 0 && ++h == a.Hkv) {
        h = 0;
        ++blk;
        if (blk * static_cast<long long>(a.tpi) >= n) {
          blk = 0;
          do {
            if (++b >= a.nodes.B) {
              left = 0;
              return false;
            }
            bool bad;
            n = seq_tokens(a, a.nodes, b, ctx, bad);
          } while (n == 0);
        }
        load(a);
      }
    }
    fresh = false;
    if (left <= 0) return false;
    end = static_cast<int>(min(static_cast<long long>(k.T), t0 + left));
    return true;
  }
};

// ---------------------------------------------------------------------------
// softmax
// ---------------------------------------------------------------------------
// Bits 0 .. x - 1 of a word.
__device__ __forceinline__ uint32_t below(int x) { return x <= 0 ? 0u : x >= 32 ? ~0u : (1u << x) - 1; }

// Rows of a tile that lie before its slot c (0 .. its slots).
__device__ __forceinline__ int rows_before(const Args& a, int c) {
  if (!a.holes || c <= 0) return c;
  const int p = c / a.ps;
  return c >= a.tk ? kTile : p * a.box + c - p * a.ps;
}

// A score becomes -inf where `seen` is 0.
__device__ __forceinline__ void hide(uint32_t& s, uint32_t seen) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.eq.u32 p, %1, 0;\n\t@p mov.b32 %0, 0xff800000;\n\t}" : "+r"(s) : "r"(seen));
}

// ln(2^m l), m in units of log 2 with P's lift in it.
template <class T>
__device__ __forceinline__ float log_sum(float m, float l) {
  constexpr float far = kLift<T> < 0.f ? kLift<T> : 0.f, back = kLift<T> < 0.f ? 0x1p40f : 1.f;
  return (m + far + log2f(l * back)) * 0.6931471805599453f;
}

template <class T>
__device__ __forceinline__ bool has_nonfinite(const uint4& x) {
  // an exponent of all ones carries into the sign's place
  constexpr uint32_t kExp = T::kId == Bf16::kId ? 0x7f807f80u : 0x7c007c00u;
  constexpr uint32_t kOne = T::kId == Bf16::kId ? 0x00800080u : 0x04000400u;
  return (((x.x & kExp) + kOne) | ((x.y & kExp) + kOne) | ((x.z & kExp) + kOne) | ((x.w & kExp) + kOne)) & 0x80008000u;
}
template <class T>
__device__ __forceinline__ uint32_t only_finite(uint32_t x) {
  constexpr uint32_t kExp = T::kId == Bf16::kId ? 0x7f807f80u : 0x7c007c00u;
  constexpr uint32_t kOne = T::kId == Bf16::kId ? 0x00800080u : 0x04000400u;
  const uint32_t c = ((x & kExp) + kOne) & 0x80008000u;
  return x & (c & 0x8000u ? 0xffff0000u : ~0u) & (c >> 31 ? 0xffffu : ~0u);
}

// The slot that bit i of an item's flags stands for.
__device__ __forceinline__ int flag_slot(const Args& a, const Seen& s, int i) {
  return i < 256 ? s.p0 + i : s.p0 - a.window + 1 + (i - 256);
}

// N entries from k on of the values that are not finite, for a row that sees them.
template <class T, int N>
__device__ __forceinline__ void add_nonfinite(const Args& a, int b, int h, const Seen& s, int pos, const unsigned* fl, int k,
                                              uint32_t (&o)[N]) {
#pragma unroll 1
  for (int q = 0; q < 16; ++q) {
#pragma unroll 1
    for (unsigned bits = fl[q]; bits; bits &= bits - 1) {
      const int slot = flag_slot(a, s, 32 * q + __ffs(bits) - 1);
      int page, off;
      if (slot > pos || (a.window && slot <= pos - a.window && slot >= a.sinks)) continue;
      if (!kv_slot(a.table + b * a.table_stride, a.width, a.pages, a.ps, slot, page, off)) continue;
      const uint32_t* v =
          reinterpret_cast<const uint32_t*>(a.vcache + 2 * (page * a.v_page + off * a.v_slot + h * a.v_head + k));
#pragma unroll
      for (int e = 0; e < N / 2; ++e) {
        const uint32_t x = v[e];
        const float lo = T::lo(x), hi = T::hi(x);
        if (!(fabsf(lo) < INFINITY)) o[2 * e] = __float_as_uint(__uint_as_float(o[2 * e]) + lo);
        if (!(fabsf(hi) < INFINITY)) o[2 * e + 1] = __float_as_uint(__uint_as_float(o[2 * e + 1]) + hi);
      }
    }
  }
}

__device__ __forceinline__ float row_max(const uint32_t (&s)[4][32]) {
  float m[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) m[j] = max3(__uint_as_float(s[j][0]), __uint_as_float(s[j][1]), __uint_as_float(s[j][2]));
#pragma unroll
  for (int e = 3; e < 31; e += 2) {
#pragma unroll
    for (int j = 0; j < 4; ++j) m[j] = max3(m[j], __uint_as_float(s[j][e]), __uint_as_float(s[j][e + 1]));
  }
  return fmaxf(max3(m[0], m[1], m[2]), max3(m[3], __uint_as_float(s[0][31]), max3(__uint_as_float(s[1][31]), __uint_as_float(s[2][31]), __uint_as_float(s[3][31]))));
}

// A row of D columns of tensor memory times f.
template <int D>
__device__ __forceinline__ void scale_columns(uint32_t at, float f) {
#pragma unroll 1
  for (int k = 0; k < D; k += 32) {
    uint32_t o[32];
    tm_ld32(at + k, o);
    tm_wait_loads();
    tm_tie32(o);
#pragma unroll
    for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
    tm_st32(at + k, o);
  }
}

// N columns of a row from k on: results, or a part.
template <class T, int D, int N>
__device__ __forceinline__ void write_columns(const Args& a, const uint32_t (&o)[N], long long row, int k, bool direct,
                                              bool empty, float inv) {
  if (direct) {
    uint2* out = reinterpret_cast<uint2*>(a.out + 2 * (row * D + k));
    uint32_t y[N / 2];
#pragma unroll
    for (int e = 0; e < N / 2; ++e)
      y[e] = empty ? 0u : T::pack(__uint_as_float(o[2 * e]) * inv, __uint_as_float(o[2 * e + 1]) * inv);
    if (N % 8 == 0) {
#pragma unroll
      for (int q = 0; q < N / 8; ++q)
        reinterpret_cast<uint4*>(out)[q] = make_uint4(y[4 * q], y[4 * q + 1], y[4 * q + 2], y[4 * q + 3]);
    } else {
#pragma unroll
      for (int q = 0; q < N / 4; ++q) out[q] = make_uint2(y[2 * q], y[2 * q + 1]);
    }
  } else {
    uint4* out = reinterpret_cast<uint4*>(a.part_o + row * D + k);
#pragma unroll
    for (int q = 0; q < N / 4; ++q) out[q] = make_uint4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
  }
}

template <bool V>
struct Flag {
  static constexpr bool value = V;
};

template <class T, int D, bool WIDE>
__device__ __forceinline__ void softmax_role(const Args& a, Misc& sm, uint32_t tmem, int w) {
  const int wt = threadIdx.x & 127;  // row of the row tile = lane of tensor memory
  const uint32_t lanes = static_cast<uint32_t>(wt & 96) << 16;
  const int tok = wt / a.G, g = wt - tok * a.G;
  const bool in_tile = tok < a.tq;
  const f32x2 c2 = pk2(a.c, a.c);
  const uint32_t tO = tmem + lanes + 256 + w * D;
  uint32_t ppv = 0;    // phase of pvdone[w]
  uint32_t sph = 0;    // phases of sfull[w][.]
  int tiles = 0, item = -1;
  Pieces pc;
  pc.start(sm);
#pragma unroll 1
  while (pc.next(a)) {
    ++item;
    if (!WIDE && (item & 1) != w) {
      tiles += pc.end - pc.t0;
      continue;
    }
    // this row tile's tokens
    const int i0 = pc.blk * a.tpi + (WIDE ? w * a.tq : 0), i1 = min(pc.n, i0 + a.tq) - 1;
    if (WIDE && i1 < i0) continue;
    const Seen mine = seen_by(a, pc.ctx + i0, pc.ctx + i1);
    const int i = i0 + tok, pos = pc.ctx + i;
    const bool valid = in_tile && i <= i1;
    const bool busy = __any_sync(0xffffffffu, valid);
    float m = kNoScore, l = 0.f;
    int jobs = 0;
    bool edges = false;  // tiles that the clearing warp has looked at
#pragma unroll 1
    for (int at = pc.t0; at < pc.end; ++at, ++tiles) {
      const int t = pc.tile(at);
      const bool edge = pc.k.edge(t);
      int first = 0, count = kTile;
      if (edge) {
        tile_slots(a, t, first, count);
        if (WIDE && !some(mine, first, first + count - 1)) continue;
        edges = true;
      }
      const int buf = WIDE ? w : tiles & 1;
      bar_wait(&sm.sfull[w][buf], (sph >> buf) & 1, sm, a.err);
      sph ^= 1u << buf;
      // The last tile's product: with two row tiles it was issued before these scores, and
      // so has been made.
      bool waited = WIDE || jobs == 0;
      auto last_done = [&]() {
        if (!waited) {
          bar_wait(&sm.pvdone[w], ppv, sm, a.err);
          ppv ^= 1;
          tc_after();
          waited = true;
        }
      };
      tc_after();
      // (a copy of its own for tiles with masks: with one body for both, what the scheduler
      // made of it changed by 1.15 times with the mask's code)
      auto softmax = [&](auto masked) {
        constexpr bool MASKED = decltype(masked)::value;
        const uint32_t tS = tmem + lanes + buf * 128;
        uint32_t s[4][32];
#pragma unroll
        for (int j = 0; j < 4; ++j) tm_ld32(tS + 32 * j, s[j]);
        tm_wait_loads();
#pragma unroll
        for (int j = 0; j < 4; ++j) tm_tie32(s[j]);
        if (MASKED) {
          // rows from lo, or before sk, to hi - 1
          int hi = kTile, lo = 0, sk = 0;
          if (edge) {
            hi = rows_before(a, min(pos - first + 1, count));
            lo = a.window ? rows_before(a, pos - a.window - first + 1) : 0;
            sk = rows_before(a, a.sinks - first);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t v = sm.plain[j] & below(hi - 32 * j) & (~below(lo - 32 * j) | below(sk - 32 * j));
#pragma unroll
            for (int e = 0; e < 32; ++e) hide(s[j][e], v & (1u << e));
          }
        }
        const float top = a.c * row_max(s) - kLift<T>;
        const bool raise = top > (m == kNoScore ? m : m + kGrow);
        if (__builtin_expect(__any_sync(0xffffffffu, raise), 0)) {
          const float f = raise ? ex2_fast(m - top) : 1.f;
          if (raise) m = top;
          l *= f;
          if (jobs > 0) {
            last_done();
            scale_columns<D>(tO, f);
          }
        }
        // P a quarter at a time (all four at once want 255 registers), the sums and
        // stores of one beside the exponentials of the next
        const f32x2 nm = pk2(-m, -m);
        f32x2 sum[2] = {0ull, 0ull};
        auto exps = [&](uint32_t (&x)[32]) {
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            float y0, y1;
            up2(fma2(pk2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])), c2, nm), y0, y1);
            x[e] = __float_as_uint(ex2_fast(y0));
            x[e + 1] = __float_as_uint(ex2_fast(y1));
          }
        };
        exps(s[0]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (j < 3) exps(s[j < 3 ? j + 1 : 3]);
          if (j == 2) {  // (their stores end beside the last exponentials)
            tm_tie32(s[3]);
            tm_wait_stores();
            tc_before();
            bar_arrive(&sm.pfull[buf][0]);
          }
          uint32_t p[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const float y0 = __uint_as_float(s[j][2 * e]), y1 = __uint_as_float(s[j][2 * e + 1]);
            sum[e & 1] = add2(sum[e & 1], pk2(y0, y1));
            p[e] = T::pack(y0, y1);
          }
          tm_put16(tS + 16 * j, p);
          if (j < 2) tm_tie32(s[j < 2 ? j + 2 : 3]);
        }
        float a0, a1;
        up2(add2(sum[0], sum[1]), a0, a1);
        l += a0 + a1;
        tm_wait_stores();
      };
      if (busy) {
        if (edge || a.holes) softmax(Flag<true>{});
        else softmax(Flag<false>{});
      } else {
        tc_before();
        bar_arrive(&sm.pfull[buf][0]);
      }
      last_done();
      tc_before();
      bar_arrive(&sm.pfull[buf][1]);
      ++jobs;
    }

    // ---- end of the piece ----
    if (jobs > 0) {
      bar_wait(&sm.pvdone[w], ppv, sm, a.err);
      ppv ^= 1;
      tc_after();
    }
    // (a warp's rows go out 32 columns at a time)
    const bool direct = pc.direct(), empty = l == 0.f;
    const float inv = !direct ? 1.f : empty ? 0.f : 1.f / l;
    const long long row = direct ? (static_cast<long long>(pc.b) * a.nodes.N + i) * a.Hq + pc.h * a.G + g
                                 : (2ll * blockIdx.x + (item == 0 ? 0 : 1)) * a.tpi * a.G + (WIDE ? w * a.tq * a.G : 0) + wt;
    const unsigned* fl = sm.flags[item % kFlagSets];
    unsigned any = 0;
    if (busy && jobs > 0) {
      if (edges) {
#pragma unroll
        for (int q = 0; q < 16; ++q) any |= fl[q];
      }
#pragma unroll 1
      for (int k = 0; k < D; k += 32) {
        uint32_t o[32];
        tm_ld32(tO + k, o);
        tm_wait_loads();
        tm_tie32(o);
        if (any && valid) add_nonfinite<T>(a, pc.b, pc.h, pc.s, pos, fl, k, o);
        if (valid) write_columns<T, D>(a, o, row, k, direct, empty, inv);
      }
    }
    if (jobs > 0) {
      tc_before();
      bar_arrive(&sm.ofree[w]);
    }
    if (valid && direct && a.lse) a.lse[row] = empty ? -INFINITY : log_sum<T>(m, l);
    if (valid && !direct) a.part_ml[row] = make_float2(m, l);
  }
}

// ---------------------------------------------------------------------------
// softmax of copies
// ---------------------------------------------------------------------------
// Four entries from k on of a row that came out NaN or infinite because a slot that every row
// sees holds such a value, which met other copies' weights of 0 as well: what the values
// alone make of them.  By the lanes of a warp that write results, which share the piece's
// slots (alone, each took 29 ms for 20000; the CTA's other warps give up waiting after a
// second).
template <class T>
__device__ __forceinline__ void seen_nonfinite(const Args& a, const Pieces& pc, int k, uint32_t (&o)[4]) {
  const unsigned here = __activemask();
  const int n = __popc(here), me = __popc(here & ((1u << (threadIdx.x & 31)) - 1));
  unsigned odd[3][2] = {};  // columns with NaN, inf, -inf
#pragma unroll 1
  for (int at = pc.t0; at < pc.end; ++at) {
    int first, count;
    tile_slots(a, pc.tile(at), first, count);
#pragma unroll 1
    for (int s = first + me; s < first + count; s += n) {
      int page, off;
      if (!all(a, pc.s, s, s)) continue;  // (cleared)
      if (!kv_slot(a.table + pc.b * a.table_stride, a.width, a.pages, a.ps, s, page, off)) continue;
      const uint4* v = reinterpret_cast<const uint4*>(a.vcache + 2 * (page * a.v_page + off * a.v_slot + pc.h * a.v_head));
      uint4 x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = v[i];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        if (!has_nonfinite<T>(x[i])) continue;
        const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll 1
        for (int e = 0; e < 8; ++e) {
          const uint32_t y = e < 2 ? w[0] : e < 4 ? w[1] : e < 6 ? w[2] : w[3];
          const float f = e & 1 ? T::hi(y) : T::lo(y);
          const unsigned bit = 1u << (8 * (i & 3) + e);
          if (f != f) odd[0][i >> 2] |= bit;
          else if (f == INFINITY) odd[1][i >> 2] |= bit;
          else if (f == -INFINITY) odd[2][i >> 2] |= bit;
        }
      }
    }
  }
  __syncwarp(here);
#pragma unroll
  for (int q = 0; q < 6; ++q) odd[q >> 1][q & 1] = __reduce_or_sync(here, odd[q >> 1][q & 1]);
  const bool second = k >= 32;
  const unsigned nan = (second ? odd[0][1] : odd[0][0]) >> (k & 31), up = (second ? odd[1][1] : odd[1][0]) >> (k & 31),
                 down = (second ? odd[2][1] : odd[2][0]) >> (k & 31);
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const unsigned bit = 1u << e;
    if (!(fabsf(__uint_as_float(o[e])) < INFINITY) && ((nan | up | down) & bit))
      o[e] = (nan | (up & down)) & bit ? 0x7fc00000u : up & bit ? 0x7f800000u : 0xff800000u;
  }
}

// The same (not if it is only rows whose l, the row's `sum`, is NaN as well: scores that are
// not finite need no more), and the values that only some rows see, for a token in slot `pos`.
// Out of line: few calls come here, and its instructions would stand between those of every
// item (64 single tokens under a window took 1 to 5 of 72 us more with it in line).
template <class T>
__device__ __noinline__ uint4 mend_copies(const Args& a, const Pieces pc, const unsigned* fl, int pos, float sum, int k, uint4 x) {
  uint32_t z[4] = {x.x, x.y, x.z, x.w};
  bool finite = true;
#pragma unroll
  for (int e = 0; e < 4; ++e) finite = finite && fabsf(__uint_as_float(z[e])) < INFINITY;
  if (__any_sync(__activemask(), !finite && sum > 0.f)) seen_nonfinite<T>(a, pc, k, z);
  add_nonfinite<T>(a, pc.b, pc.h, pc.s, pos, fl, k, z);
  return make_uint4(z[0], z[1], z[2], z[3]);
}

// Few rows (64 at most) of heads of 64, whose tiles come in half the time of heads of 128:
// they lie in the row tile two or four times, and a copy takes its part of a tile's slots
// alone, so that a thread has 64 or 32 scores instead of 128; and the warpgroups take turns
// within an item, as copies of each other.  The copies have their own m, l and O, which
// are joined at the item's end; the O's of two items lie side by side in tensor memory.
// (64 single tokens under a window of 2048, 32 / 8 heads: 71 us, with rows once and a
// warpgroup an item 95.  Heads of 128 are as fast without: 64 / 8 heads, 64 single tokens
// at 6800 279 us both ways, a chain of 8 under a window 27 us with copies and 24 without.)
template <class T>
__device__ __forceinline__ void share_role(const Args& a, Misc& sm, uint32_t tmem, char* stage, int w) {
  const int wt = threadIdx.x & 127, span = kTile / a.copies;
  const uint32_t lanes = static_cast<uint32_t>(wt & 96) << 16;
  const int copy = wt / span, r = wt - copy * span, nq = span / 32, q0 = copy * nq;  // its quarters of the slots
  const int tok = r / a.G, g = r - tok * a.G;
  const f32x2 c2 = pk2(a.c, a.c);
  constexpr int D = 64, kLines = 256;  // (threads that work on an item)
  uint32_t ppv = 0;    // phase of pvdone[w]
  uint32_t sph = 0;    // phases of sfull[w][.]
  int tiles = 0, item = -1;
  Pieces pc;
  pc.start(sm);
#pragma unroll 1
  while (pc.next(a)) {
    ++item;
    const uint32_t tO = tmem + lanes + 256 + ((item & 1) * 2 + w) * D;
    const int i = pc.blk * a.tpi + tok, pos = pc.ctx + i;
    const bool valid = tok < a.tq && i < pc.n;
    float m = kNoScore, l = 0.f;
    int jobs = 0;
    bool edges = false;
#pragma unroll 1
    for (int at = pc.t0; at < pc.end; ++at, ++tiles) {
      const int t = pc.tile(at);
      const bool edge = pc.k.edge(t);
      edges |= edge;
      if ((tiles & 1) != w) continue;
      const int buf = w;
      bar_wait(&sm.sfull[w][buf], (sph >> buf) & 1, sm, a.err);
      sph ^= 1u << buf;
      bool waited = jobs == 0;  // for the last tile's product
      auto last_done = [&]() {
        if (!waited) {
          bar_wait(&sm.pvdone[w], ppv, sm, a.err);
          ppv ^= 1;
          tc_after();
          waited = true;
        }
      };
      tc_after();
      const uint32_t tS = tmem + lanes + buf * 128;
      uint32_t s[2][32];
      tm_ld32(tS + 32 * q0, s[0]);
      if (nq == 2) tm_ld32(tS + 32 * q0 + 32, s[1]);
      tm_wait_loads();
      tm_tie32(s[0]);
      tm_tie32(s[1]);
      if (edge || a.holes) {
        int hi = kTile, lo = 0, sk = 0;
        if (edge) {
          int first, count;
          tile_slots(a, t, first, count);
          hi = rows_before(a, min(pos - first + 1, count));
          lo = a.window ? rows_before(a, pos - a.window - first + 1) : 0;
          sk = rows_before(a, a.sinks - first);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const int e0 = 32 * (q0 + j);
          const uint32_t v = j < nq ? sm.plain[q0 + j] & below(hi - e0) & (~below(lo - e0) | below(sk - e0)) : 0u;
#pragma unroll
          for (int e = 0; e < 32; ++e) hide(s[j][e], v & (1u << e));
        }
      }
      float mx[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        mx[j] = max3(__uint_as_float(s[j][0]), __uint_as_float(s[j][1]), __uint_as_float(s[j][2]));
#pragma unroll
        for (int e = 3; e < 31; e += 2) mx[j] = max3(mx[j], __uint_as_float(s[j][e]), __uint_as_float(s[j][e + 1]));
        mx[j] = fmaxf(mx[j], __uint_as_float(s[j][31]));
      }
      const float top = a.c * (nq == 2 ? fmaxf(mx[0], mx[1]) : mx[0]) - kLift<T>;
      const bool raise = top > (m == kNoScore ? m : m + kGrow);
      if (__any_sync(0xffffffffu, raise)) {
        const float f = raise ? ex2_fast(m - top) : 1.f;
        if (raise) m = top;
        l *= f;
        if (jobs > 0) {
          last_done();
          scale_columns<D>(tO, f);
        }
      }
      const f32x2 nm = pk2(-m, -m);
      f32x2 sum[2] = {0ull, 0ull};
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        if (j >= nq) break;
        uint32_t p[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          float y0, y1;
          up2(fma2(pk2(__uint_as_float(s[j][2 * e]), __uint_as_float(s[j][2 * e + 1])), c2, nm), y0, y1);
          y0 = ex2_fast(y0);
          y1 = ex2_fast(y1);
          sum[e & 1] = add2(sum[e & 1], pk2(y0, y1));
          p[e] = T::pack(y0, y1);
        }
        tm_put16(tS + 16 * (q0 + j), p);
      }
      // no weight for the other copies' slots
      uint32_t zero[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) zero[e] = 0;
#pragma unroll
      for (int q = 0; q < 4; ++q)
        if (q < q0 || q >= q0 + nq) tm_put16(tS + 16 * q, zero);
      float a0, a1;
      up2(add2(sum[0], sum[1]), a0, a1);
      l += a0 + a1;
      tm_wait_stores();
      last_done();
      tc_before();
      bar_arrive(&sm.pfull[buf][0]);
      bar_arrive(&sm.pfull[buf][1]);
      ++jobs;
    }

    // ---- end of the piece: the copies joined ----
    if (jobs > 0) {
      bar_wait(&sm.pvdone[w], ppv, sm, a.err);
      ppv ^= 1;
      tc_after();
    }
    const int id = w * 128 + wt;
    float2* ml = reinterpret_cast<float2*>(stage);
    ml[id] = make_float2(m, l);
    named_sync(1, kLines);
    float M = kNoScore, L = 0.f;
    for (int k = r; k < kLines; k += span) M = fmaxf(M, ml[k].x);
    for (int k = r; k < kLines; k += span) {
      const float2 x = ml[k];
      L += x.x == M ? x.y : x.y * ex2_fast(x.x - M);
    }
    const bool direct = pc.direct();
    auto place = [&](int token, int head) {
      return direct ? (static_cast<long long>(pc.b) * a.nodes.N + pc.blk * a.tpi + token) * a.Hq + pc.h * a.G + head
                    : (2ll * blockIdx.x + (item == 0 ? 0 : 1)) * a.tpi * a.G + token * a.G + head;
    };
    if (valid && id < span) {
      sm.sums[r] = L;
      const long long row = place(tok, g);
      if (!direct) a.part_ml[row] = make_float2(M, L);
      else if (a.lse) a.lse[row] = L == 0.f ? -INFINITY : log_sum<T>(M, L);
    }
    named_sync(1, kLines);
    const float f = m == M ? 1.f : ex2_fast(m - M);
    const unsigned* fl = sm.flags[item % kFlagSets];
    unsigned any = 0;
    if (edges) {
#pragma unroll
      for (int q = 0; q < 16; ++q) any |= fl[q];
    }
    uint4* line = reinterpret_cast<uint4*>(stage + id * 128);
    const int quads = min(a.tq, pc.n - pc.blk * a.tpi) * a.G * 8;
#pragma unroll 1
    for (int k = 0; k < D; k += 32) {
      uint32_t o[32];
      tm_ld32(tO + k, o);
      tm_wait_loads();
      tm_tie32(o);
#pragma unroll
      for (int e = 0; e < 32; ++e) o[e] = jobs > 0 ? __float_as_uint(__uint_as_float(o[e]) * f) : 0u;
#pragma unroll
      for (int q = 0; q < 8; ++q) line[q ^ (wt & 7)] = make_uint4(o[4 * q], o[4 * q + 1], o[4 * q + 2], o[4 * q + 3]);
      named_sync(1, kLines);
      // four columns of a row a thread
#pragma unroll 1
      for (int i = id; i < quads; i += kLines) {
        const int rr = i >> 3, q = i & 7, token = rr / a.G;
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int c = rr; c < kLines; c += span) {
          // (copies lie multiples of 8 rows apart)
          const float4 y = *reinterpret_cast<const float4*>(stage + c * 128 + (q ^ (rr & 7)) * 16);
          x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
        }
        const float sum = sm.sums[rr];
        uint4 y = make_uint4(__float_as_uint(x.x), __float_as_uint(x.y), __float_as_uint(x.z), __float_as_uint(x.w));
        const bool finite = fabsf(x.x) < INFINITY && fabsf(x.y) < INFINITY && fabsf(x.z) < INFINITY && fabsf(x.w) < INFINITY;
        if (__builtin_expect(__any_sync(__activemask(), !finite || any), 0))
          y = mend_copies<T>(a, pc, fl, pc.ctx + pc.blk * a.tpi + token, sum, k + 4 * q, y);
        const uint32_t z[4] = {y.x, y.y, y.z, y.w};
        write_columns<T, D>(a, z, place(token, rr - token * a.G), k + 4 * q, direct, sum == 0.f,
                            !direct ? 1.f : sum == 0.f ? 0.f : 1.f / sum);
      }
      named_sync(1, kLines);
    }
    tc_before();
    bar_arrive(&sm.ofree[item & 1]);
  }
}

// ---------------------------------------------------------------------------
// copies of K and V
// ---------------------------------------------------------------------------
// K, V or both: K a tile ahead, as the products take them.
template <int D, bool KEYS, bool VALUES, bool GATHER>
__device__ __forceinline__ void load_role(const Args& a, Misc& sm, const CUtensorMap& mapk, const CUtensorMap& mapv,
                                          uint32_t ring, uint32_t ringv) {
  const int lane = threadIdx.x & 31;
  Ring rk = {&mapk, sm.kfull, sm.kempty, ring, a.nk, -1, 0}, rv = {&mapv, sm.vfull, sm.vempty, ringv, a.nv, -1, 0};
  Pieces pc;
  pc.start(sm);
  bool bad_page = false;
  Place idv = {};
  int p0v = 0, p1v = 0, hv = 0;  // the tile whose values are to come
  bool pending = false;
#pragma unroll 1
  while (pc.next(a)) {
    const int* trow = a.table + pc.b * a.table_stride;
    // boxes of a tile that hold something seen, and this lane's page ids
    auto lookup = [&](int t, int& p0, int& p1) {
      p0 = p1 = 0;
      if (!a.uneven) {
        p1 = a.boxes - 1;
        if (pc.k.edge(t)) {
          const int first = t * a.tk, end = first + a.tk;
          const int last = min(end - 1, end > pc.s.lo ? pc.s.p1 : pc.s.sk - 1);
          p0 = first < pc.s.sk ? 0 : max(0, pc.s.lo - first) / a.step;
          p1 = (last - first) / a.step;
        }
      }
      // (not looked at before its tile's turn: the load is on its way meanwhile)
      return box_place<GATHER>(a, trow, t, pc.s.p1, lane >= p0 && lane <= p1);
    };
    int p0n, p1n;
    Place idn = lookup(pc.tile(pc.t0), p0n, p1n);
#pragma unroll 1
    for (int at = pc.t0; at < pc.end; ++at) {
      const Place id = idn;
      const int p0 = p0n, p1 = p1n;
      if (at + 1 < pc.end) idn = lookup(pc.tile(at + 1), p0n, p1n);
      if (KEYS) bad_page |= !load_tile<D, GATHER>(a, sm, rk, p0, p1, id, pc.h, a.err, a.withheld);
      if (VALUES && !KEYS) bad_page |= !load_tile<D, GATHER>(a, sm, rv, p0, p1, id, pc.h, a.err, a.withheld);
      if (VALUES && KEYS) {
        if (pending) load_tile<D, GATHER>(a, sm, rv, p0v, p1v, idv, hv, a.err, a.withheld);
        p0v = p0;
        p1v = p1;
        idv = id;
        hv = pc.h;
        pending = true;
      }
    }
  }
  if (pending) load_tile<D, GATHER>(a, sm, rv, p0v, p1v, idv, hv, a.err, a.withheld);
  // whether somebody sees them (looked up once more: the copies' loop has no time for it)
  if (__any_sync(0xffffffffu, bad_page)) {
    bad_page = false;
    pc.start(sm);
#pragma unroll 1
    while (pc.next(a)) {
#pragma unroll 4
      for (int at = pc.t0; at < pc.end; ++at)
        bad_page |= bad_box<GATHER>(a, a.table + pc.b * a.table_stride, pc.tile(at), pc.s.p1, pc.s.lo, pc.s.sk);
    }
    if (bad_page) atomicOr(a.err, kErrBadPage);
  }
}

// ---------------------------------------------------------------------------
// products (the warp runs as one; one lane issues)
// ---------------------------------------------------------------------------
// Two row tiles: a warp each, so that one's waits pass beside the other's products (a
// wait costs 100 cycles at least, and few products queue up).  One row tile: one warp.
template <class T, int D, int MODE>
__device__ __forceinline__ void product_role(const Args& a, Misc& sm, uint32_t tmem, uint32_t ring, uint32_t ringv,
                                             uint32_t Q, int w) {
  constexpr bool WIDE = MODE == kTwo, ALT = MODE == kCopies;
  constexpr int kSlotBytes = D / 64 * kHalf;
  const uint32_t khalf = a.half / 16, vstep = a.group / 8;
  const uint64_t kd0 = operand(ring, 16, a.group), qd0 = operand(Q, 16, 1024);
  const uint64_t vd0 = operand(ringv, D == 128 ? a.half : 0, a.group);
  const uint32_t ids = instr<T>(kTile, false, false, a.negate), ido = instr<T>(D, false, true);
  struct Step {
    bool valid, newq, last, edge, act, begin, fresh, final;  // (fresh: O's first product)
    int item, no;  // the item; the tile's number in the CTA
  };
  Pieces pc;
  pc.start(sm);
  int item = -1, at = 0, no = -1, lasting = 0;
  bool started = false, inside = false, some_rows = true;
  // whether this row tile sees some of tile t
  Seen mine;
  auto acting = [&](int t) {
    if (!WIDE) return true;
    if (!some_rows) return false;
    if (!pc.k.edge(t)) return true;
    int first, count;
    tile_slots(a, t, first, count);
    return some(mine, first, first + count - 1);
  };
  auto gen = [&](Step& st) {
    st.newq = false;
    if (!inside || ++at == pc.end) {
      if (!pc.next(a)) {
        st.valid = false;
        return;
      }
      inside = true;
      ++item;
      at = pc.t0;
      started = false;
      st.newq = true;
      if (WIDE) {
        const int i0 = pc.s.p0 + w * a.tq;
        some_rows = i0 <= pc.s.p1;
        if (some_rows) mine = seen_by(a, i0, min(pc.s.p1, i0 + a.tq - 1));
        lasting = pc.end - 1;
        while (lasting >= pc.t0 && !acting(pc.tile(lasting))) --lasting;
      }
    }
    const int t = pc.tile(at);
    st.valid = true;
    st.last = at + 1 == pc.end;
    st.item = item;
    st.no = ++no;
    st.edge = pc.k.edge(t);
    st.act = acting(t);
    st.final = !WIDE || at == lasting;
    st.begin = st.act && !started;
    st.fresh = ALT ? at < pc.t0 + 2 : st.begin;
    started |= st.act;
  };
  int kslot = -1, vslot = -1, edges = 0;
  uint32_t kphase = 0, vphase = 0;
  uint32_t pph = 0, oph = 0;  // phases of pfull (two row tiles) and ofree
  // what scores and values wait for beside the turn
  auto before_scores = [&](const Step& st) {
    if (st.newq) bar_await(&sm.qfull[WIDE ? 0 : st.item & 1], (WIDE ? st.item : st.item >> 1) & 1, sm, a.err);
    if (++kslot == a.nk) {
      kslot = 0;
      kphase ^= 1;
    }
    bar_await(&sm.kfull[kslot], kphase, sm, a.err);
  };
  auto scores = [&](const Step& st) {
    const int buf = WIDE ? w : st.no & 1, qb = WIDE ? w : st.item & 1;
    uint64_t* qempty = &sm.qempty[WIDE ? 0 : qb];
    if (st.act) {
      tc_after();
      const uint64_t qd = qd0 + qb * (kSlotBytes / 16), kd = kd0 + kslot * (kSlotBytes / 16);
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < D / 16; ++k)
          tc_mma(tmem + buf * 128, qd + (k / 4) * (kHalf / 16) + (k & 3) * 2, kd + (k / 4) * khalf + (k & 3) * 2, ids,
                 k > 0);
        tc_commit(&sm.sfull[WIDE ? w : ALT ? buf : st.item & 1][buf]);  // (each warpgroup has its own: it skips items)
        tc_commit(&sm.kempty[kslot]);
        if (st.last) tc_commit(qempty);
      }
    } else if (elect_one()) {
      bar_arrive(&sm.kempty[kslot]);
      if (st.last) tc_commit(qempty);  // (behind this warp's earlier products)
    }
    __syncwarp();
  };
  uint32_t ph = 0;
  auto before_values = [&](const Step& st) {
    if (++vslot == a.nv) {
      vslot = 0;
      vphase ^= 1;
    }
    bar_await(&sm.vfull[vslot], vphase, sm, a.err);
    if (st.edge) {
      bar_await(&sm.vready[edges % kEdgeBars], (edges / kEdgeBars) & 1, sm, a.err);
      ++edges;
    }
    if (!st.act) return;
    const int ob = WIDE ? w : st.item & 1;
    if (st.begin) {  // the results of the last item in these columns have been read
      bar_await(&sm.ofree[ob], ((oph >> ob) & 1) ^ 1, sm, a.err);
      oph ^= 1u << ob;
    }
    ph = WIDE ? pph : (st.no >> 1) & 1;
    pph ^= 1;
    bar_await(&sm.pfull[WIDE ? w : st.no & 1][0], ph, sm, a.err);
  };
  auto values = [&](const Step& st) {
    const int buf = WIDE ? w : st.no & 1, ob = WIDE ? w : st.item & 1;
    const uint32_t tO = tmem + 256 + (ALT ? ob * 2 + buf : ob) * D;
    if (st.act) {
      const uint64_t vd = vd0 + vslot * (kSlotBytes / 16);
      tc_after();
      if (elect_one()) {
#pragma unroll
        for (int k = 0; k < kTile / 32; ++k)
          tc_mma_ta(tO, tmem + buf * 128 + k * 8, vd + k * vstep, ido, !st.fresh || k > 0);
      }
      __syncwarp();
      bar_await(&sm.pfull[buf][1], ph, sm, a.err);
      tc_after();
      if (elect_one()) {
#pragma unroll
        for (int k = kTile / 32; k < kTile / 16; ++k)
          tc_mma_ta(tO, tmem + buf * 128 + k * 8, vd + k * vstep, ido, true);
        if (st.final) tc_commit(&sm.pvdone[ALT ? buf : ob]);
        tc_commit(&sm.vempty[vslot]);
      }
    } else if (elect_one()) {
      bar_arrive(&sm.vempty[vslot]);
    }
    __syncwarp();
  };
  // Two row tiles: the warps take turns, so that the row tiles' softmax run apart (side
  // by side they share the exponentials' pipe, and then the products': 4200 cycles a tile
  // instead of 2800).
  uint32_t tph = w ^ 1;
  auto take = [&]() {
    if (WIDE) bar_await(&sm.turn[w], tph, sm, a.err);
    tph ^= 1;
  };
  auto pass = [&]() {
    if (WIDE && elect_one()) bar_arrive(&sm.turn[w ^ 1]);
    __syncwarp();
  };
  Step cur, nxt;
  if (WIDE || w == 0) {
    gen(nxt);
    if (nxt.valid) {
      before_scores(nxt);
      take();
      scores(nxt);
      pass();
    }
#pragma unroll 1
    while (nxt.valid) {
      cur = nxt;
      gen(nxt);
      if (!WIDE) {  // the next scores go to the other buffer
        if (nxt.valid) {
          before_scores(nxt);
          scores(nxt);
        }
        before_values(cur);
        values(cur);
        continue;
      }
      const bool together = nxt.valid && !nxt.newq;  // (a new item's rows come late)
      if (together) before_scores(nxt);
      before_values(cur);
      take();
      values(cur);
      if (together) scores(nxt);
      pass();
      if (nxt.valid && !together) {
        before_scores(nxt);
        take();
        scores(nxt);
        pass();
      }
    }
    if (elect_one()) tc_commit(&sm.done);
    __syncwarp();
    bar_await(&sm.done, 0, sm, a.err);
  }
}

// ---------------------------------------------------------------------------
// the kernel
// ---------------------------------------------------------------------------
template <class T, int D, int MODE, bool GATHER>
__global__ void __launch_bounds__(kThreads, 1)
    chunk_kernel(const __grid_constant__ CUtensorMap mapq, const __grid_constant__ CUtensorMap mapk,
                 const __grid_constant__ CUtensorMap mapv, const __grid_constant__ Args a) {
  extern __shared__ __align__(1024) char base[];
  constexpr bool WIDE = MODE == kTwo;
  constexpr int HALVES = D / 64;
  constexpr int kSlotBytes = HALVES * kHalf;
  char* ring = base;
  char* ringv = ring + a.nk * kSlotBytes;
  char* Q = ringv + a.nv * kSlotBytes;
  char* stage = Q + 2 * kSlotBytes;  // (copies)
  Misc& sm = *reinterpret_cast<Misc*>(stage + (MODE == kCopies ? kStage : 0));
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int C = gridDim.x, B = a.nodes.B;

  if (tid == 0) {
    for (int i = 0; i < kMaxRing; ++i) {
      bar_init(&sm.kfull[i], 1);
      bar_init(&sm.kempty[i], WIDE ? 2 : 1);  // the warps that issue products
      bar_init(&sm.vfull[i], 1);
      bar_init(&sm.vempty[i], WIDE ? 3 : 2);  // and the clearing one
    }
    for (int i = 0; i < 2; ++i) {
      bar_init(&sm.turn[i], 1);
      bar_init(&sm.qfull[i], 1);
      bar_init(&sm.qempty[i], WIDE ? 2 : 1);
      bar_init(&sm.sfull[i][0], 1);
      bar_init(&sm.sfull[i][1], 1);
      bar_init(&sm.pfull[i][0], 128);  // (halves of the slots)
      bar_init(&sm.pfull[i][1], 128);
      bar_init(&sm.pvdone[i], 1);
      bar_init(&sm.ofree[i], MODE == kCopies ? 256 : 128);
    }
    for (int i = 0; i < kEdgeBars; ++i) bar_init(&sm.vready[i], 1);
    bar_init(&sm.done, WIDE ? 2 : 1);
    sm.abort = 0;
    sm.wait_us = a.wait_us;
    sm.left = 0;
    sm.b0 = sm.blk0 = sm.h0 = sm.t0 = 0;
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
    asm volatile("prefetch.tensormap [%0];" ::"l"(&mapv));
  }
  if (tid < kTile) {
    const int o = row_offset(a, tid);
    sm.off[tid] = o;
    const unsigned there = __ballot_sync(0xffffffffu, o != kFar);
    if (lane == 0) sm.plain[tid >> 5] = there;
  }
  // Rows between pages are zeros (they meet P = 0, and must not be NaN): in an edge tile the
  // pages that nobody sees are not copied, and nothing clears their rows that are no slot.
  if (a.holes) {
    for (int i = tid; i < (a.nk + a.nv) * kSlotBytes / 16; i += kThreads)
      reinterpret_cast<uint4*>(ring)[i] = make_uint4(0, 0, 0, 0);
    fence_async();
  }

  // ---- this CTA's range: the cost of the (sequence, block)s before each thread's (a
  // block scan), and where the range starts ----
  {
    const long long pairs = static_cast<long long>(B) * a.NB, per = (pairs + kThreads - 1) / kThreads;
    const long long f = tid * per, e = min(pairs, f + per);
    long long mine = 0;  // tiles of a head
    long long blocks = 0;
    bool any_bad = false, any_pad = false;
    int b = -1, ctx = 0, n = 0, blk = 0;
    auto load = [&](long long at) {
      if (b < 0) {
        b = static_cast<int>(at / a.NB);
        blk = static_cast<int>(at - static_cast<long long>(b) * a.NB);
      } else if (++blk == a.NB) {
        blk = 0;
        ++b;
      } else {
        return;
      }
      bool bad;
      n = seq_tokens(a, a.nodes, b, ctx, bad);
      any_bad |= bad;
      any_pad |= n < a.nodes.N;
    };
#pragma unroll 1
    for (long long at = f; at < e; ++at) {
      load(at);
      if (blk * static_cast<long long>(a.tpi) >= n) continue;
      mine += block_of(a, block_seen(a, ctx, n, blk)).T;
      ++blocks;
    }
    if (any_bad && blockIdx.x == 0) atomicOr(a.err, kErrBadLength);
    long long inc = mine, incb = blocks;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long o = __shfl_up_sync(0xffffffffu, inc, d), ob = __shfl_up_sync(0xffffffffu, incb, d);
      if (lane >= d) {
        inc += o;
        incb += ob;
      }
    }
    if (lane == 31) {
      sm.scan[0][warp] = inc;
      sm.scan[1][warp] = incb;
    }
    const bool pad = __syncthreads_or(any_pad);
    long long before = inc - mine, beforeb = incb - blocks, tiles = 0, nblocks = 0;
#pragma unroll
    for (int i = 0; i < kThreads / 32; ++i) {
      if (i < warp) {
        before += sm.scan[0][i];
        beforeb += sm.scan[1][i];
      }
      tiles += sm.scan[0][i];
      nblocks += sm.scan[1][i];
    }
    tiles *= a.Hkv;
    nblocks *= a.Hkv;
    // What an item costs beside its tiles, less where a range is of a few tiles only.
    long long w = 0;  // min(item_cost, tiles / (4 C))
#pragma unroll 1
    for (int k = 1; k <= a.item_cost; ++k) w += tiles >= 4ll * k * C;
    const long long W = tiles + w * nblocks;
    // The range's ends in cost: [lo, hi); an item's tiles come first in its T + w.  A
    // range may hold no tile.
    const long long me = blockIdx.x, lo = __umul64hi(W * me, a.per_cta),
                    hi = me + 1 == C ? W : static_cast<long long>(__umul64hi(W * (me + 1), a.per_cta));
    long long p = (before + w * beforeb) * a.Hkv;
    const long long mine_cost = (mine + w * blocks) * a.Hkv;
    if (tid == 0) {
      a.ranges[me].used = 0;
      sm.cost = static_cast<int>(w);
      sm.pad = pad;
    }
    __syncthreads();
    // the thread whose blocks hold the range's first tile (lo may lie behind the tiles
    // of the last item before them)
    if (lo < p + mine_cost && hi > p && p - lo <= w) {
      b = -1;
#pragma unroll 1
      for (long long at = f; at < e; ++at) {
        load(at);
        if (blk * static_cast<long long>(a.tpi) >= n) continue;
        const Seen seen = block_seen(a, ctx, n, blk);
        const Block k = block_of(a, seen);
        const int all_t = k.T;
        const long long one = all_t + w, end = p + one * a.Hkv;
        if (lo < end) {
          const unsigned long long d = lo > p ? lo - p : 0;
          int h = static_cast<int>(d / one);
          int t0 = static_cast<int>(d - h * one);
          if (t0 >= all_t) {  // behind the item's tiles: the next item
            ++h;
            t0 = 0;
          }
          const long long from = p + h * one + t0;  // cost position of the first tile
          if (h < a.Hkv) {
            if (from < hi) {
              Range r;
              r.lo = from;
              r.t0 = sm.t0 = t0;
              r.used = 1;
              r.b = sm.b0 = b;
              r.blk = sm.blk0 = blk;
              r.h = sm.h0 = h;
              r.T = all_t;
              a.ranges[me] = r;
              sm.left = hi - from;
              sm.ctx0 = ctx;
              sm.n0 = n;
              sm.s0 = seen;
              sm.k0 = k;
            }
            break;
          }
        }
        p = end;
      }
    }
  }
  tc_before();
  __syncthreads();
  tc_after();
  pdl_trigger();
  const uint32_t tmem = __shfl_sync(0xffffffffu, sm.tmem, 0);

  if (warp >= 4) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoft));
    const int w = (warp - 4) >> 2;
    if constexpr (MODE == kCopies) share_role<T>(a, sm, tmem, stage, w);
    else softmax_role<T, D, WIDE>(a, sm, tmem, w);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsCopy));
    if (warp == 0) {
      load_role<D, true, WIDE, GATHER>(a, sm, mapk, mapv, sptr(ring), sptr(ringv));
    } else if (!WIDE && warp == 2) {
      load_role<D, false, true, GATHER>(a, sm, mapk, mapv, sptr(ring), sptr(ringv));
    } else if (warp == 1 || warp == 2) {
      product_role<T, D, MODE>(a, sm, tmem, sptr(ring), sptr(ringv), sptr(Q), warp - 1);
    } else {
      // ---- Q, and what must not be multiplied ----
      Pieces pq, pc;
      pq.start(sm);
      pc.start(sm);
      int nq = 0;
      // the rows of the next item, once the scores of the one before are made
      auto fetch = [&]() {
        if (!pq.next(a)) return;
        const int qb = WIDE ? 0 : nq & 1;
        const uint32_t ph = (WIDE ? nq : nq >> 1) & 1;
        ++nq;
        const bool ok = bar_await(&sm.qempty[qb], ph ^ 1, sm, a.err) && !*reinterpret_cast<volatile int*>(&sm.abort);
        if (__all_sync(0xffffffffu, ok)) {
          // boxes of rows: of one row tile, of two, or the same for every copy
          const int boxes = MODE == kCopies ? a.copies : WIDE && pq.s.p1 - pq.s.p0 >= a.tq ? 2 : 1;
          if (lane == 0) bar_expect(&sm.qfull[qb], boxes * HALVES * a.tq * a.G * 128 + a.withheld);
          __syncwarp();
          if (elect_one()) {
            for (int w = 0; w < boxes; ++w)
              for (int d = 0; d < HALVES; ++d)
                tma_rows(sptr(Q) + (MODE == kCopies ? qb * kSlotBytes + w * (kTile / a.copies) * 128 : (qb + w) * kSlotBytes) +
                             d * kHalf,
                         &mapq, d * 64, pq.h * a.G,
                         a.zero ? a.nodes.N : pq.blk * a.tpi + (WIDE ? w * a.tq : 0),  // (behind the last: zeros)
                         pq.b, &sm.qfull[qb]);
          }
          __syncwarp();
        }
      };
      fetch();
      int slot = -1, edges = 0, item = -1;
      uint32_t phase = 0;
#pragma unroll 1
      while (pc.next(a)) {
        ++item;
        if (!WIDE) fetch();
        unsigned* fl = sm.flags[item % kFlagSets];
        if (lane < 16) fl[lane] = 0;
        __syncwarp();
#pragma unroll 1
        for (int at = pc.t0; at < pc.end; ++at) {
          const int t = pc.tile(at);
          if (++slot == a.nv) {
            slot = 0;
            phase ^= 1;
          }
          bar_await(&sm.vfull[slot], phase, sm, a.err);
          if (pc.k.edge(t)) {
            int first, count;
            tile_slots(a, t, first, count);
            char* V = ringv + slot * kSlotBytes;
#pragma unroll 1
            for (int r = lane; r < kTile; r += 32) {
              const int o = sm.off[r], s = first + o;
              if (o >= count) continue;  // zeros
              if (all(a, pc.s, s, s)) continue;
              uint4* line = reinterpret_cast<uint4*>(V + (r >> 3) * a.group + (r & 7) * 128);
              const int half = a.half / 16;
              if (!some(pc.s, s, s)) {
#pragma unroll
                for (int v = 0; v < D / 8; ++v) line[(v / 8) * half + ((v ^ r) & 7)] = make_uint4(0, 0, 0, 0);
                continue;
              }
              bool bad = false;
#pragma unroll
              for (int v = 0; v < D / 8; ++v) bad |= has_nonfinite<T>(line[(v / 8) * half + ((v ^ r) & 7)]);
              if (bad) {
#pragma unroll 1
                for (int v = 0; v < D / 8; ++v) {
                  uint4& x = line[(v / 8) * half + (v & 7)];
                  x = make_uint4(only_finite<T>(x.x), only_finite<T>(x.y), only_finite<T>(x.z), only_finite<T>(x.w));
                }
                const int i = s > pc.s.p0 ? s - pc.s.p0 : 256 + s - (pc.s.p0 - a.window + 1);
                atomicOr(&fl[i >> 5], 1u << (i & 31));
              }
            }
            fence_async();
            __syncwarp();
            if (lane == 0) bar_arrive(&sm.vready[edges % kEdgeBars]);
            ++edges;
          }
          __syncwarp();
          if (lane == 0) bar_arrive(&sm.vempty[slot]);
        }
        if (WIDE) fetch();
      }
    }
  }
  // ---- tokens that are not there: zeros ----
  if (sm.pad) {
#pragma unroll 1
    for (int b0 = 0; b0 < B; b0 += 32) {
      int n = a.nodes.N, ctx;
      bool bad;
      if (b0 + lane < B) n = seq_tokens(a, a.nodes, b0 + lane, ctx, bad);
      unsigned some = __ballot_sync(0xffffffffu, n < a.nodes.N);
#pragma unroll 1
      for (; some; some &= some - 1) {
        const int j = __ffs(some) - 1, nb = __shfl_sync(0xffffffffu, n, j);
        const long long rows = static_cast<long long>(a.nodes.N - nb) * a.Hq;
        const long long r0 = (static_cast<long long>(b0 + j) * a.nodes.N + nb) * a.Hq;
        const long long from = rows * blockIdx.x / C, to = rows * (blockIdx.x + 1) / C;
        uint4* o = reinterpret_cast<uint4*>(a.out + 2 * (r0 + from) * D);
        for (long long i = tid; i < (to - from) * (D / 8); i += kThreads) o[i] = make_uint4(0, 0, 0, 0);
        if (a.lse)
          for (long long i = r0 + from + tid; i < r0 + to; i += kThreads) a.lse[i] = -INFINITY;
      }
    }
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
// Joins the parts of the items that range borders cut:
//     M = max m_i,  w_i = 2^(m_i - M),  o = sum w_i O_i / sum w_i l_i
// in range order.  blockIdx.x: a range that starts inside an item; the first such range
// of an item does its work, a warp per row.
// ---------------------------------------------------------------------------
constexpr int kJoinWarps = 8;

template <class T, int D>
__global__ void __launch_bounds__(32 * kJoinWarps) chunk_join_kernel(const __grid_constant__ Args a, int C) {
  constexpr int E = D / 32;
  const int lane = threadIdx.x & 31;
  const int c = blockIdx.x + 1;
  pdl_wait();
  const Range me = a.ranges[c];
  if (!me.used || me.t0 == 0) return;
  const long long s = me.lo - me.t0, e = s + me.T;
  // the range before, which holds the item's tile t0 - 1
  int pk = c - 1;
  while (pk > 0 && !a.ranges[pk].used) --pk;
  const long long before = a.ranges[pk].lo;
  if (before > s) return;  // an earlier range's item
  bool bad;
  int ctx;
  const int n = seq_tokens(a, a.nodes, me.b, ctx, bad);
  const int i0 = me.blk * a.tpi, rows = (min(n, i0 + a.tpi) - i0) * a.G, cap = a.tpi * a.G;
  const int r = blockIdx.y * kJoinWarps + (threadIdx.x >> 5);
  if (r >= rows) return;
  float M = kNoScore, L = 0.f, o[E];
#pragma unroll
  for (int q = 0; q < E; ++q) o[q] = 0.f;
  // a lane a range, so that few loads wait for one another (8 items in 19 parts each)
#pragma unroll 1
  for (int k0 = pk; k0 < C; k0 += 32) {
    const int k = k0 + lane;
    const int used = k < C ? a.ranges[k].used : 0;
    const long long lo = k < C ? a.ranges[k].lo : 0;
    const bool in = used && (k == pk || lo < e);
    // only the first can be its CTA's last piece
    const long long at = (2ll * k + (k == pk && before < s ? 1 : 0)) * cap + r;
    const float2 ml = in ? a.part_ml[at] : make_float2(kNoScore, 0.f);
    unsigned parts = __ballot_sync(0xffffffffu, ml.y != 0.f);
    const bool last = __any_sync(0xffffffffu, used && !in);
    if (parts) {
      float m = ml.y != 0.f ? fmaxf(M, ml.x) : M;
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
      // (at least the smallest number: an infinite value stays infinite)
      const float x = ml.x == m ? 1.f : fmaxf(exp2f(ml.x - m), 0x1p-126f);
      const float y = L == 0.f ? 0.f : M == m ? 1.f : fmaxf(exp2f(M - m), 0x1p-126f);
      L *= y;
#pragma unroll
      for (int q = 0; q < E; ++q) o[q] *= y;
      M = m;
      while (parts) {
        float w[4], v[4][E];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int from = __ffs(parts) - 1;
          const float wu = __shfl_sync(0xffffffffu, x, from & 31), lu = __shfl_sync(0xffffffffu, ml.y, from & 31);
          const long long place = __shfl_sync(0xffffffffu, at, from & 31);
          w[u] = 0.f;
#pragma unroll
          for (int q = 0; q < E; ++q) v[u][q] = 0.f;
          if (from >= 0) {
            w[u] = wu;
            L = fmaf(lu, wu, L);
#pragma unroll
            for (int q = 0; q < E; q += 2) {
              const float2 z = *reinterpret_cast<const float2*>(a.part_o + place * D + lane * E + q);
              v[u][q] = z.x;
              v[u][q + 1] = z.y;
            }
          }
          parts &= parts - 1;
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
          for (int q = 0; q < E; ++q) o[q] = fmaf(v[u][q], w[u], o[q]);
      }
    }
    if (last) break;
  }
  const int tok = r / a.G, g = r - tok * a.G;
  const bool empty = L == 0.f;
  const float inv = empty ? 0.f : 1.f / L;
  const long long row = (static_cast<long long>(me.b) * a.nodes.N + i0 + tok) * a.Hq + me.h * a.G + g;
  char* out = a.out + 2 * (row * D + lane * E);
#pragma unroll
  for (int q = 0; q < E; q += 2)
    *reinterpret_cast<uint32_t*>(out + 2 * q) = empty ? 0u : T::pack(o[q] * inv, o[q + 1] * inv);
  if (a.lse && lane == 0) a.lse[row] = empty ? -INFINITY : log_sum<T>(M, L);
}

// ---------------------------------------------------------------------------
// host
// ---------------------------------------------------------------------------
// Tokens of an item: all where copies of them fit a row tile, one row tile of them where
// every chunk fits it, else two (with one: 8192 tokens, 64 / 8 heads 1343 us against 831;
// 16 chunks of 40 at 4000, 32 / 8 heads of 128 108 us against 83).
int item_tokens(int N, int G, int D) {
  const int tq = kTile / G;
  return D == 64 && N * static_cast<long long>(G) <= kTile / 2 ? N : N <= tq ? tq : 2 * tq;
}

struct Layout {
  size_t ranges, ml, o, total;
};
Layout layout_of(int N, int G, int D) {
  const size_t rows = static_cast<size_t>(item_tokens(N, G, D)) * G;
  Layout L;
  L.ranges = 256;
  L.ml = (L.ranges + sizeof(Range) * kMaxCtas + 255) / 256 * 256;
  L.o = (L.ml + 8ull * 2 * kMaxCtas * rows + 255) / 256 * 256;
  L.total = L.o + 4ull * 2 * kMaxCtas * rows * D;
  return L;
}

template <class T_, int D, int MODE, bool GATHER>
cudaError_t launch_g(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const Args& a, int C,
                     size_t smem, cudaStream_t s) {
  cudaError_t e = cudaFuncSetAttribute(chunk_kernel<T_, D, MODE, GATHER>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMax);
  if (e != cudaSuccess) return e;
  chunk_kernel<T_, D, MODE, GATHER><<<C, kThreads, smem, s>>>(mq, mk, mv, a);
  e = cudaGetLastError();
  if (e != cudaSuccess || C < 2) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(C - 1, (a.tpi * a.G + kJoinWarps - 1) / kJoinWarps);
  cfg.blockDim = dim3(32 * kJoinWarps);
  cfg.stream = s;
  cudaLaunchAttribute at;
  at.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, chunk_join_kernel<T_, D>, a, C);
}

template <class T_, int D, int MODE>
cudaError_t launch_t(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const Args& a, int C,
                     size_t smem, cudaStream_t s) {
  return a.gather ? launch_g<T_, D, MODE, true>(mq, mk, mv, a, C, smem, s)
                  : launch_g<T_, D, MODE, false>(mq, mk, mv, a, C, smem, s);
}

template <class T_, int D>
cudaError_t launch_m(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const Args& a, int C, int mode,
                     size_t smem, cudaStream_t s) {
  if constexpr (D == 64) {
    if (mode == kCopies) return launch_t<T_, D, kCopies>(mq, mk, mv, a, C, smem, s);
  }
  return mode == kTwo ? launch_t<T_, D, kTwo>(mq, mk, mv, a, C, smem, s) : launch_t<T_, D, kOne>(mq, mk, mv, a, C, smem, s);
}

}  // namespace

size_t chunk_attention_bytes(int N, int G, int D) { return layout_of(N, G, D).total; }

cudaError_t launch_chunk_attention(const ChunkParams& p, int dtype, int D, cudaStream_t s) {
  Args a;
  const KvView& kv = p.kv;
  a.nodes = p.nodes;
  a.Hq = p.Hq; a.Hkv = kv.Hkv; a.G = p.G;
  a.tpi = item_tokens(p.nodes.N, p.G, D);
  const int rows = a.tpi * p.G;
  a.copies = D == 128 ? 1 : rows <= kTile / 4 ? 4 : rows <= kTile / 2 ? 2 : 1;
  a.tq = a.copies > 1 ? a.tpi : kTile / p.G;
  const int mode = a.copies > 1 ? kCopies : a.tpi > a.tq ? kTwo : kOne;
  a.NB = (p.nodes.N + a.tpi - 1) / a.tpi;
  // (a window that no sequence exceeds is none)
  a.window = p.window < static_cast<long long>(kv.width) * kv.ps ? p.window : 0;
  a.sinks = a.window ? p.sinks : 0;
  // (2, 4, 7: a prompt of 8192 964, 826, 847 us; a ragged batch under a window 280, 264, 294)
  a.item_cost = 4;
  a.zero = p.scale == 0.f;
  a.c = a.zero ? 1.f : fabsf(p.scale) * 1.4426950408889634f;
  a.negate = p.scale < 0.f;
  a.out = p.out; a.lse = p.lse;
  a.vcache = kv.v; a.v_page = kv.v_page; a.v_slot = kv.v_slot; a.v_head = kv.v_head;
  a.err = p.err;
  a.wait_us = p.wait_us; a.withheld = p.withheld;
  const Layout L = layout_of(p.nodes.N, p.G, D);
  char* ws = reinterpret_cast<char*>(p.err);
  a.ranges = reinterpret_cast<Range*>(ws + L.ranges);
  a.part_ml = reinterpret_cast<float2*>(ws + L.ml);
  a.part_o = reinterpret_cast<float*>(ws + L.o);
  const int slot = D * 2 * kTile;
  const size_t beside = 2 * slot + (mode == kCopies ? kStage : 0) + sizeof(Misc);
  const int slots = static_cast<int>((kSmemMax - beside) / slot);
  a.nk = (slots + 1) / 2 < kMaxRing ? (slots + 1) / 2 : kMaxRing;
  a.nv = slots - a.nk < kMaxRing ? slots - a.nk : kMaxRing;
  const size_t smem = static_cast<size_t>(a.nk + a.nv) * slot + beside;
  CUtensorMap mq, mk, mv;
  if (!page_tiles(a, kv, dtype, D, &mk, &mv) || !encode_queries(&mq, p.q, p.q_b, p.q_n, p.q_h, p.Hq, p.nodes, p.G, dtype, D, a.tq))
    return cudaErrorInvalidValue;
  int C = sm_count();
  if (C < 1) return cudaErrorInvalidDevice;
  C = C < kMaxCtas ? C : kMaxCtas;
  a.per_cta = C > 1 ? ~0ull / C + 1 : 0;
  const auto launch = dtype == Bf16::kId ? (D == 128 ? launch_m<Bf16, 128> : launch_m<Bf16, 64>)
                                         : (D == 128 ? launch_m<F16, 128> : launch_m<F16, 64>);
  return launch(mq, mk, mv, a, C, mode, smem, s);
}

}  // namespace ssd

// ssd_kv.cu -- the paged cache of the target pass: storing the drafted nodes
// (with per-head norms and position rotation on the way) and moving the
// accepted path behind the context.
//
// kv_append_kernel: per head vector x of D entries,
//     y = x / sqrt(mean(x^2) + eps) * w,
//     z = (y_a c - y_b s, y_b c + y_a s) for each rotated pair (a, b),
// in fp32, rounded once.  It reads q, k, v and one row of the cosine/sine
// table a token and writes as much: bound by HBM for a batch, by the chain
// of loads (length -> way to the root -> table row and page id) for a few
// tokens.  The grid is one wave, so that the chain is waited for once, and its
// places are found once a token, by one lane; a lane holds 16 entries of a
// head, which halves the address arithmetic of eight.  64 trees of 21 tokens,
// 64 + 16 heads of 128 (56 MB): 15.1 us, 3.7 TB/s (a CTA per token, 8 entries a
// lane: 24.6 us); 512 chains of 8, 32 + 16 heads of 64 (51 MB): 13.1 us, 3.9 TB/s
// (26.8); one chain of 8: 3.7 us.
// kv_commit_kernel: a copy of the accepted rows, bound by HBM (or by its two
// chained round trips).  64 paths of up to 12 nodes, 32 layers (118 MB): 23.4 us,
// 5.0 TB/s, of which launch and look-up are 3.6; 64 to 512 threads a CTA, 4 to 12
// rows in flight and one to four waves of CTAs gave 23.4 to 25.4.
#include <algorithm>

#include "ssd_device.cuh"
#include "ssd_kv.cuh"

namespace ssd {
namespace {

constexpr int kAppThreads = 128;
constexpr int kAppUnroll = 2;   // head vectors in flight per thread
constexpr int kAppCtas = 7;     // per SM
constexpr int kAppTokens = 32;  // most tokens of a CTA (a lane finds each one's place)

// Eight entries of a head vector.
template <bool VEC>
__device__ __forceinline__ uint4 load8(const char* p) {
  if (VEC) return *reinterpret_cast<const uint4*>(p);
  const unsigned short* h = reinterpret_cast<const unsigned short*>(p);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = static_cast<uint32_t>(h[2 * i]) | (static_cast<uint32_t>(h[2 * i + 1]) << 16);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

struct AppSmem {
  // of each token: where its heads lie and go to, heads numbered through q, k
  // and v (0: nowhere); its row of the table, or null
  uint64_t src[kAppTokens][4], dst[kAppTokens][4];
  const float* turn[kAppTokens];
  int there[kAppTokens];
  alignas(16) float w[2][4][8][4];  // weights of q's and k's norm: a lane's a, b, a, b, four each
};

// A CTA takes a range of (token, head) pairs; lanes of its first warp find the
// places of the range's tokens side by side, while the first head vectors are
// on their way.  A head vector is spread over D / 16 lanes, which hold the pairs
// of a rotation whole: eight entries (a) and their eight partners (b).
template <class T, int D, bool VEC, bool NEIGHBOURS>
__global__ void __launch_bounds__(kAppThreads, kAppCtas) kv_append_kernel(const __grid_constant__ AppendParams p) {
  constexpr int LP = D / 16;                // lanes per head vector
  constexpr int GROUPS = kAppThreads / LP;  // head vectors side by side
  constexpr int U = kAppUnroll;
  __shared__ AppSmem sm;
  const int tid = threadIdx.x, g = tid / LP, l = tid % LP;
  const int Hq = p.Hq, Hkv = p.kv.Hkv, Htot = Hq + 2 * Hkv, N = p.nodes.N;
  const long long i0 = static_cast<long long>(blockIdx.x) * p.items;
  const int items = static_cast<int>(min(static_cast<long long>(p.items), p.all - i0));
  const bool small = p.all <= INT32_MAX;
  const int t0 = small ? static_cast<int>(i0) / Htot : static_cast<int>(i0 / Htot);
  const int h0 = static_cast<int>(i0 - static_cast<long long>(t0) * Htot);
  // this lane's columns: ea.. and eb.., partners where they turn
  const int half = p.rot / 2;
  const bool turns = 16 * l < p.rot;
  const int ea = NEIGHBOURS || !turns ? 16 * l : 8 * l;
  const int eb = NEIGHBOURS || !turns ? 16 * l + 8 : half + 8 * l;

  auto kind = [&](int h) { return (h >= Hq) + (h >= Hq + Hkv); };
  // where head 0 of q, k or v would lie, counted on to k's and v's heads
  auto source = [&](int t, int kind) {
    const int b = t / N, j = t % N;
    return kind == 0   ? reinterpret_cast<uint64_t>(p.q) + 2 * (b * p.q_b + j * p.q_n)
           : kind == 1 ? reinterpret_cast<uint64_t>(p.k) + 2 * (b * p.kv_b + j * p.kv_n - Hq * p.kv_h)
                       : reinterpret_cast<uint64_t>(p.v) + 2 * (b * p.kv_b + j * p.kv_n - (Hq + Hkv) * p.kv_h);
  };
  const uint64_t q_h = 2 * p.q_h, kv_h = 2 * p.kv_h;
  struct Vec {
    uint4 a, b;
  };
  auto load = [&](uint64_t base, int h) {
    const char* r = reinterpret_cast<const char*>(base + (h < Hq ? q_h : kv_h) * static_cast<uint32_t>(h));
    return Vec{load8<VEC>(r + 2 * ea), load8<VEC>(r + 2 * eb)};
  };
  const int tokens = (h0 + items + Htot - 1) / Htot;
  if (tid < tokens) {
#pragma unroll
    for (int k = 0; k < 3; ++k) sm.src[tid][k] = source(t0 + tid, k);
  }
  __syncthreads();
  // the thread's pairs, GROUPS apart: token and head of each in flight, and of
  // the next to load
  Vec raw[U];
  int tag[U];
  const int dt = GROUPS / Htot, dh = GROUPS % Htot;
  int lt = (h0 + g) / Htot, lh = (h0 + g) % Htot, li = g;
  auto next = [&]() {
    lh += dh;
    lt += dt;
    if (lh >= Htot) {
      lh -= Htot;
      ++lt;
    }
    li += GROUPS;
  };
  constexpr int kTag = 20;  // bits of a head's number
#pragma unroll
  for (int u = 0; u < U; ++u) {
    if (li < items) raw[u] = load(sm.src[lt][kind(lh)], lh);
    tag[u] = (lt << kTag) | lh;
    next();
  }

  // the tokens' places
  if (tid < tokens) {
    const int b = (t0 + tid) / N, j = (t0 + tid) % N;
    const int ctx = p.nodes.ctx_len[b];
    const int nn = p.nodes.n_nodes ? p.nodes.n_nodes[b] : N;
    bool bad_len, broken;
    const int n = seq_nodes(ctx, nn, N, p.kv.width, p.kv.ps, bad_len);
    uint64_t mask;
    int depth;
    bool there = node_way(p.nodes.parent ? p.nodes.parent + static_cast<long long>(b) * N : nullptr, n, j, mask, depth,
                          broken);
    const long long pos = static_cast<long long>(ctx) + depth;
    if (there && p.rot > 0 && pos >= p.max_pos) {
      there = false;
      bad_len = true;
    }
    int page = -1, off = 0;
    bool store = false;
    if (there)
      store = kv_slot(p.kv.table + b * p.kv.table_stride, p.kv.width, p.kv.pages, p.kv.ps,
                      static_cast<long long>(ctx) + j, page, off);
    const int bits = (bad_len ? kErrBadLength : 0) | (broken ? kErrBadTree : 0) | (there && !store ? kErrBadPage : 0);
    if (bits) atomicOr(p.err, bits);
    sm.dst[tid][0] = reinterpret_cast<uint64_t>(p.q_out) + 2 * (static_cast<long long>(t0 + tid) * Hq * D);
    sm.dst[tid][1] = store ? reinterpret_cast<uint64_t>(p.kv.k) +
                                 2 * (page * p.kv.k_page + off * p.kv.k_slot - Hq * p.kv.k_head)
                           : 0;
    sm.dst[tid][2] = store ? reinterpret_cast<uint64_t>(p.kv.v) +
                                 2 * (page * p.kv.v_page + off * p.kv.v_slot - (Hq + Hkv) * p.kv.v_head)
                           : 0;
    sm.turn[tid] = there && p.rot > 0 ? p.cos_sin + pos * p.rot : nullptr;
    sm.there[tid] = there;
  }
  const bool norm = p.q_norm != nullptr;
  if (norm && tid < 4 * LP) {  // eight of a lane's weights each
    const bool second = tid & 1, isk = tid >= 2 * LP;
    const int lane = tid / 2 % LP;
    const bool turn = 16 * lane < p.rot;
    const unsigned short* w = reinterpret_cast<const unsigned short*>(isk ? p.k_norm : p.q_norm);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int i = NEIGHBOURS ? 16 * lane + 2 * k + second
                               : !turn ? 16 * lane + 8 * second + k : half * second + 8 * lane + k;
      sm.w[isk][2 * (k / 4) + second][lane][k % 4] = T::lo(w[i]);
    }
  }
  __syncthreads();

  const uint64_t k_head = 2 * p.kv.k_head, v_head = 2 * p.kv.v_head;
#pragma unroll 1
  for (int b = 0; b < items; b += U * GROUPS) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (b + u * GROUPS >= items) break;  // uniform over the CTA
      const bool act = b + u * GROUPS + g < items;
      const int h = tag[u] & ((1 << kTag) - 1), t = act ? tag[u] >> kTag : 0;
      const bool isq = h < Hq, isv = h >= Hq + Hkv;
      Vec o = raw[u];
      if ((norm || p.rot > 0) && __any_sync(0xffffffffu, act && !isv)) {
        const uint32_t w[8] = {o.a.x, o.a.y, o.a.z, o.a.w, o.b.x, o.b.y, o.b.z, o.b.w};
        f32x2 xa[4], xb[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          if (NEIGHBOURS) {
            xa[k] = pk2(T::lo(w[2 * k]), T::lo(w[2 * k + 1]));
            xb[k] = pk2(T::hi(w[2 * k]), T::hi(w[2 * k + 1]));
          } else {
            xa[k] = pk2(T::lo(w[k]), T::hi(w[k]));
            xb[k] = pk2(T::lo(w[k + 4]), T::hi(w[k + 4]));
          }
        }
        f32x2 inv2 = pk2(1.f, 1.f);
        if (norm) {
          f32x2 q = mul2(xa[0], xa[0]);
#pragma unroll
          for (int k = 1; k < 4; ++k) q = fma2(xa[k], xa[k], q);
#pragma unroll
          for (int k = 0; k < 4; ++k) q = fma2(xb[k], xb[k], q);
          float s0, s1;
          up2(q, s0, s1);
          float ss = s0 + s1;
#pragma unroll
          for (int m = LP / 2; m > 0; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
          const float inv = rsqrtf(fmaf(ss, 1.0f / D, p.eps));  // (2 units of the last place of fp32)
          inv2 = pk2(inv, inv);
        }
        const float* turn = sm.turn[t];
        const bool rotate = turn && turns;
#pragma unroll
        for (int k = 0; k < 4; k += 2) {  // four of a, four of b
          if (norm) {
            const float4 wa = *reinterpret_cast<const float4*>(sm.w[!isq][k][l]),
                         wb = *reinterpret_cast<const float4*>(sm.w[!isq][k + 1][l]);
            xa[k] = mul2(mul2(xa[k], inv2), pk2(wa.x, wa.y));
            xa[k + 1] = mul2(mul2(xa[k + 1], inv2), pk2(wa.z, wa.w));
            xb[k] = mul2(mul2(xb[k], inv2), pk2(wb.x, wb.y));
            xb[k + 1] = mul2(mul2(xb[k + 1], inv2), pk2(wb.z, wb.w));
          }
          if (rotate) {
            const float4 c = *reinterpret_cast<const float4*>(turn + 8 * l + 2 * k);
            const float4 s = *reinterpret_cast<const float4*>(turn + half + 8 * l + 2 * k);
            const f32x2 cc[2] = {pk2(c.x, c.y), pk2(c.z, c.w)}, sn[2] = {pk2(s.x, s.y), pk2(s.z, s.w)};
            const f32x2 neg[2] = {pk2(-s.x, -s.y), pk2(-s.z, -s.w)};
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const f32x2 y = xa[k + i], z = xb[k + i];
              xa[k + i] = fma2(z, neg[i], mul2(y, cc[i]));
              xb[k + i] = fma2(y, sn[i], mul2(z, cc[i]));
            }
          }
        }
        if (!isv) {
          uint32_t r[8];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float a0, a1, b0, b1;
            up2(xa[k], a0, a1);
            up2(xb[k], b0, b1);
            r[NEIGHBOURS ? 2 * k : k] = NEIGHBOURS ? T::pack(a0, b0) : T::pack(a0, a1);
            r[NEIGHBOURS ? 2 * k + 1 : k + 4] = NEIGHBOURS ? T::pack(a1, b1) : T::pack(b0, b1);
          }
          o.a = make_uint4(r[0], r[1], r[2], r[3]);
          o.b = make_uint4(r[4], r[5], r[6], r[7]);
        }
      }
      const uint64_t base = sm.dst[t][kind(h)];
      if (act && base) {
        if (isq && !sm.there[t]) o.a = o.b = make_uint4(0, 0, 0, 0);
        char* d = reinterpret_cast<char*>(base + (isq ? 2 * D : isv ? v_head : k_head) * static_cast<uint32_t>(h));
        *reinterpret_cast<uint4*>(d + 2 * ea) = o.a;
        *reinterpret_cast<uint4*>(d + 2 * eb) = o.b;
      }
      if (li < items) raw[u] = load(sm.src[lt][kind(lh)], lh);
      tag[u] = (lt << kTag) | lh;
      next();
    }
  }
}

template <class T, int D>
cudaError_t append_t(const AppendParams& p, bool vec, unsigned grid, cudaStream_t s) {
  const auto kernel = vec ? (p.interleaved ? kv_append_kernel<T, D, true, true> : kv_append_kernel<T, D, true, false>)
                          : (p.interleaved ? kv_append_kernel<T, D, false, true> : kv_append_kernel<T, D, false, false>);
  kernel<<<grid, kAppThreads, 0, s>>>(p);
  return cudaGetLastError();
}

// ---------------------------------------------------------------------------
// commit
// ---------------------------------------------------------------------------
constexpr int kComThreads = 256;
constexpr int kComBatch = 8;  // rows in flight per thread

struct ComSmem {
  long long ksrc[kMaxNodes], kdst[kMaxNodes], vsrc[kMaxNodes], vdst[kMaxNodes];
  int count;
};

// One CTA per (sequence, range of layers).  Move i reads slot ctx + node_i and
// writes slot ctx + 1 + i with node_i >= 1 + i increasing, so a slot is read
// (by move i) before it is written (by a later one): a thread that owns
// 16 bytes of every row makes the moves in order, loads of up to eight moves
// ahead of their stores (a later move's source lies behind every earlier
// target), and no two threads share a byte.
__global__ void __launch_bounds__(kComThreads) kv_commit_kernel(const CommitParams p) {
  __shared__ ComSmem sm;
  const int b = blockIdx.x, tid = threadIdx.x;
  const int ctx = p.ctx_len[b], acc = p.accept_len[b];
  const bool first = blockIdx.y == 0;
  if (tid < 32) {
    bool bad_len = false, bad_tree = false;
    int n = acc < 0 ? -1 : acc;
    if (ctx < 0 || (n >= 0 && ctx + 1LL + n > static_cast<long long>(p.kv.width) * p.kv.ps)) {
      bad_len = true;
    }
    if (n > p.N - 1) bad_tree = true;
    int node[2] = {0, 0};
    if (p.out_node && !bad_len && !bad_tree && n > 0) {
      bool bad = false;
      int last = 0;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int i = r * 32 + tid;
        if (i < n) node[r] = p.out_node[static_cast<long long>(b) * p.N + i];
        int prev = __shfl_up_sync(0xffffffffu, node[r], 1);
        if (tid == 0) prev = last;
        if (i < n && (node[r] <= prev || node[r] < 1 || node[r] >= p.N)) bad = true;
        last = __shfl_sync(0xffffffffu, node[r], 31);
      }
      bad_tree = __any_sync(0xffffffffu, bad);
      const int top = max(node[0], node[1]);
      const int far = __reduce_max_sync(0xffffffffu, top);
      if (!bad_tree && ctx + 1LL + far > static_cast<long long>(p.kv.width) * p.kv.ps) bad_len = true;
    }
    const bool none = n < 0 || bad_len || bad_tree;
    bool bad_page = false;
    const int* row = p.kv.table + b * p.kv.table_stride;
    int count = 0;
    if (p.out_node && !none) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int i = r * 32 + tid;
        bool go = i < n && node[r] != i + 1;
        if (go) {
          int sp, so, dp, d_o;
          const bool a = kv_slot(row, p.kv.width, p.kv.pages, p.kv.ps, ctx + (long long)node[r], sp, so);
          const bool c = kv_slot(row, p.kv.width, p.kv.pages, p.kv.ps, ctx + 1LL + i, dp, d_o);
          if (!a || !c) {
            bad_page = true;
            go = false;
          }
          if (go) {
            sm.ksrc[i] = sp * p.kv.k_page + so * p.kv.k_slot;
            sm.kdst[i] = dp * p.kv.k_page + d_o * p.kv.k_slot;
            sm.vsrc[i] = sp * p.kv.v_page + so * p.kv.v_slot;
            sm.vdst[i] = dp * p.kv.v_page + d_o * p.kv.v_slot;
          }
        }
        if (i < n && !go) sm.ksrc[i] = -1;  // nothing to move
      }
      count = n;
    }
    bad_page = __any_sync(0xffffffffu, bad_page);
    if (tid == 0) {
      sm.count = count;
      if (first) {
        p.new_len[b] = none ? ctx : ctx + 1 + n;
        const int bits = (bad_len ? kErrBadLength : 0) | (bad_tree ? kErrBadTree : 0) |
                         (bad_page ? kErrBadPage : 0);
        if (bits) atomicOr(p.err, bits);
      }
    }
  }
  __syncthreads();
  const int n = sm.count;
  if (n == 0) return;
  const int per_head = p.D / 8;
  const int cols = p.kv.Hkv * per_head;  // 16-byte columns of one row
  const int l0 = blockIdx.y * p.layers_per_cta;
  const int l1 = min(p.layers, l0 + p.layers_per_cta);
  const int total = (l1 - l0) * 2 * cols;
  for (int c = tid; c < total; c += kComThreads) {
    const int col = c % cols, lv = c / cols;
    const bool isv = lv & 1;
    const int layer = l0 + lv / 2;
    const int h = col / per_head, e = (col % per_head) * 8;
    char* base = isv ? p.kv.v + 2 * (layer * p.v_layer + h * p.kv.v_head + e)
                     : p.kv.k + 2 * (layer * p.k_layer + h * p.kv.k_head + e);
    const long long* src = isv ? sm.vsrc : sm.ksrc;
    const long long* dst = isv ? sm.vdst : sm.kdst;
    for (int i0 = 0; i0 < n; i0 += kComBatch) {
      uint4 x[kComBatch];
#pragma unroll
      for (int u = 0; u < kComBatch; ++u)
        if (i0 + u < n && sm.ksrc[i0 + u] >= 0)
          x[u] = *reinterpret_cast<const uint4*>(base + 2 * src[i0 + u]);
#pragma unroll
      for (int u = 0; u < kComBatch; ++u)
        if (i0 + u < n && sm.ksrc[i0 + u] >= 0)
          *reinterpret_cast<uint4*>(base + 2 * dst[i0 + u]) = x[u];
    }
  }
}

}  // namespace

cudaError_t launch_kv_append(const AppendParams& p0, int dtype, int D, bool vec, cudaStream_t s) {
  AppendParams p = p0;
  const int Htot = p.Hq + 2 * p.kv.Hkv, groups = kAppThreads / (D / 16);
  p.all = static_cast<long long>(p.nodes.B) * p.nodes.N * Htot;
  // pairs of a CTA: one wave of CTAs, at least a head vector a thread, at most
  // as many as kAppTokens tokens surely hold
  const long long places = 152 * kAppCtas;
  const long long each = (p.all + places - 1) / places, most = static_cast<long long>(kAppTokens - 2) * Htot;
  p.items = static_cast<int>(std::min((each + groups - 1) / groups * groups, most));
  const unsigned grid = static_cast<unsigned>((p.all + p.items - 1) / p.items);
  if (dtype == Bf16::kId) return D == 128 ? append_t<Bf16, 128>(p, vec, grid, s) : append_t<Bf16, 64>(p, vec, grid, s);
  return D == 128 ? append_t<F16, 128>(p, vec, grid, s) : append_t<F16, 64>(p, vec, grid, s);
}

cudaError_t launch_kv_commit(const CommitParams& p0, cudaStream_t s) {
  CommitParams p = p0;
  // layers per CTA: as few as give the GPU about four waves of CTAs
  const long long want = 4 * 152 * 4;
  long long per = (static_cast<long long>(p.B) * p.layers + want - 1) / want;
  if (!p.out_node) per = p.layers;  // nothing moves: lengths only
  p.layers_per_cta = static_cast<int>(per);
  while ((p.layers + p.layers_per_cta - 1) / p.layers_per_cta > 65535) ++p.layers_per_cta;
  const dim3 grid(p.B, (p.layers + p.layers_per_cta - 1) / p.layers_per_cta);
  kv_commit_kernel<<<grid, kComThreads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace ssd

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
// tokens.
// kv_commit_kernel: a copy of the accepted rows, bound by HBM (or by its two
// chained round trips).
#include "ssd_kv.cuh"

namespace ssd {
namespace {

constexpr int kAppThreads = 256;
constexpr int kAppUnroll = 4;  // head vectors in flight per thread

template <bool VEC>
__device__ __forceinline__ uint4 load8(const char* p) {
  if (VEC) {
    uint4 v;
    asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
  }
  const unsigned short* h = reinterpret_cast<const unsigned short*>(p);
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w[i] = static_cast<uint32_t>(h[2 * i]) | (static_cast<uint32_t>(h[2 * i + 1]) << 16);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// One CTA per (token, range of heads).  A head vector is spread over D / 8
// lanes, 16 bytes each; a thread keeps its eight columns for every head it
// handles, so the cosines, sines and weights are loaded once.  The raw head
// vectors are loaded before the token's length, tree and page are known:
// the two latencies overlap.
template <class T, int D, bool VEC>
__global__ void __launch_bounds__(kAppThreads) kv_append_kernel(const AppendParams p) {
  constexpr int LP = D / 8;                    // lanes per head vector
  constexpr int GROUPS = kAppThreads / LP;     // head vectors side by side
  const int tid = threadIdx.x;
  const int g = tid / LP, e = (tid % LP) * 8;  // group; first column
  const int N = p.nodes.N;
  const int b = static_cast<int>(blockIdx.x / N), j = static_cast<int>(blockIdx.x % N);
  const int Hkv = p.kv.Hkv, Hq = p.Hq, Htot = Hq + 2 * Hkv;
  const int h0 = blockIdx.y * p.heads_per_cta;
  const int h1 = min(Htot, h0 + p.heads_per_cta);

  const char* qrow = p.q + 2 * (b * p.q_b + j * p.q_n);
  const char* krow = p.k + 2 * (b * p.kv_b + j * p.kv_n);
  const char* vrow = p.v + 2 * (b * p.kv_b + j * p.kv_n);
  auto src = [&](int h) -> const char* {
    if (h < Hq) return qrow + 2 * (h * p.q_h + e);
    if (h < Hq + Hkv) return krow + 2 * ((h - Hq) * p.kv_h + e);
    return vrow + 2 * ((h - Hq - Hkv) * p.kv_h + e);
  };
  uint4 raw[kAppUnroll];
#pragma unroll
  for (int u = 0; u < kAppUnroll; ++u) {
    const int h = h0 + u * GROUPS + g;
    if (h < h1) raw[u] = load8<VEC>(src(h));
  }

  // the token's place
  const int ctx = p.nodes.ctx_len[b];
  const int nn = p.nodes.n_nodes ? p.nodes.n_nodes[b] : N;
  bool bad_len, broken;
  const int n = seq_nodes(ctx, nn, N, p.kv.width, p.kv.ps, bad_len);
  uint64_t mask;
  int depth;
  bool there = node_way(p.nodes.parent ? p.nodes.parent + static_cast<long long>(b) * N : nullptr,
                        n, j, mask, depth, broken);
  const long long pos = static_cast<long long>(ctx) + depth;
  if (there && p.rot > 0 && pos >= p.max_pos) {
    there = false;
    bad_len = true;
  }
  int page = -1, off = 0;
  bool store = false;
  if (there) {
    store = kv_slot(p.kv.table + b * p.kv.table_stride, p.kv.width, p.kv.pages, p.kv.ps,
                    static_cast<long long>(ctx) + j, page, off);
  }
  if (tid == 0 && blockIdx.y == 0) {
    const int bits = (bad_len ? kErrBadLength : 0) | (broken ? kErrBadTree : 0) |
                     (there && !store ? kErrBadPage : 0);
    if (bits) atomicOr(p.err, bits);
  }

  // this thread's columns of the rotation and the weights
  float cs[8], sn[8], wq[8], wk[8];
  const int half = p.rot / 2;
  const bool turns = there && e < p.rot;
  const bool upper = e >= half;
  if (turns) {
    const float* row = p.cos_sin + pos * p.rot;
    if (p.interleaved) {
      const float4 c = *reinterpret_cast<const float4*>(row + e / 2);
      const float4 s = *reinterpret_cast<const float4*>(row + half + e / 2);
      cs[0] = cs[1] = c.x; cs[2] = cs[3] = c.y; cs[4] = cs[5] = c.z; cs[6] = cs[7] = c.w;
      sn[0] = sn[1] = s.x; sn[2] = sn[3] = s.y; sn[4] = sn[5] = s.z; sn[6] = sn[7] = s.w;
    } else {
      const int i = upper ? e - half : e;
#pragma unroll
      for (int t = 0; t < 8; t += 4) {
        *reinterpret_cast<float4*>(cs + t) = *reinterpret_cast<const float4*>(row + i + t);
        *reinterpret_cast<float4*>(sn + t) = *reinterpret_cast<const float4*>(row + half + i + t);
      }
    }
  }
  const bool norm = p.q_norm != nullptr;
  if (norm) {
    unpack8<T>(load8<false>(p.q_norm + 2 * e), wq);
    unpack8<T>(load8<false>(p.k_norm + 2 * e), wk);
  }
  const int lane = tid & 31;
  const int partner = upper ? lane - half / 8 : lane + half / 8;  // neighbour pairs: unused

  for (int base = h0; base < h1; base += kAppUnroll * GROUPS) {
    if (base != h0) {
#pragma unroll
      for (int u = 0; u < kAppUnroll; ++u) {
        const int h = base + u * GROUPS + g;
        if (h < h1) raw[u] = load8<VEC>(src(h));
      }
    }
#pragma unroll
    for (int u = 0; u < kAppUnroll; ++u) {
      const int h = base + u * GROUPS + g;
      if (base + u * GROUPS >= h1) break;  // uniform over the CTA
      const bool act = h < h1;
      const bool isq = h < Hq, isv = h >= Hq + Hkv;
      uint4 o = act ? raw[u] : make_uint4(0, 0, 0, 0);
      float x[8];
      unpack8<T>(o, x);
      if (norm) {
        float ss = 0.f;
#pragma unroll
        for (int t = 0; t < 8; ++t) ss = fmaf(x[t], x[t], ss);
#pragma unroll
        for (int m = LP / 2; m > 0; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
        const float inv = 1.0f / sqrtf(ss * (1.0f / D) + p.eps);
#pragma unroll
        for (int t = 0; t < 8; ++t) x[t] = x[t] * inv * (isq ? wq[t] : wk[t]);
      }
      if (p.rot > 0) {
        float y[8];
        if (p.interleaved) {
#pragma unroll
          for (int t = 0; t < 8; ++t) y[t] = x[t ^ 1];
        } else {
#pragma unroll
          for (int t = 0; t < 8; ++t) y[t] = __shfl_sync(0xffffffffu, x[t], partner & 31);
        }
        if (turns) {
#pragma unroll
          for (int t = 0; t < 8; ++t) {
            const bool second = p.interleaved ? (t & 1) : upper;
            const float c = x[t] * cs[t], s = y[t] * sn[t];
            x[t] = second ? c + s : c - s;
          }
        }
      }
      if (!isv && (norm || p.rot > 0)) o = pack8<T>(x);
      if (!act) continue;
      if (isq) {
        if (!there) o = make_uint4(0, 0, 0, 0);
        char* d = p.q_out + 2 * ((static_cast<long long>(blockIdx.x) * Hq + h) * D + e);
        *reinterpret_cast<uint4*>(d) = o;
      } else if (store) {
        char* d = isv ? p.kv.v + 2 * (page * p.kv.v_page + off * p.kv.v_slot +
                                      (h - Hq - Hkv) * p.kv.v_head + e)
                      : p.kv.k + 2 * (page * p.kv.k_page + off * p.kv.k_slot +
                                      (h - Hq) * p.kv.k_head + e);
        *reinterpret_cast<uint4*>(d) = o;
      }
    }
  }
}

template <class T>
cudaError_t append_t(const AppendParams& p, int D, bool vec, dim3 grid, cudaStream_t s) {
  if (D == 128) {
    if (vec) kv_append_kernel<T, 128, true><<<grid, kAppThreads, 0, s>>>(p);
    else kv_append_kernel<T, 128, false><<<grid, kAppThreads, 0, s>>>(p);
  } else {
    if (vec) kv_append_kernel<T, 64, true><<<grid, kAppThreads, 0, s>>>(p);
    else kv_append_kernel<T, 64, false><<<grid, kAppThreads, 0, s>>>(p);
  }
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
  const long long tokens = static_cast<long long>(p.nodes.B) * p.nodes.N;
  const int Htot = p.Hq + 2 * p.kv.Hkv;
  const int groups = kAppThreads / (D / 8);
  // few tokens: the heads over more CTAs, up to one round of loads each
  const int most = (Htot + groups - 1) / groups;
  int split = static_cast<int>(tokens >= 608 ? 1 : (608 + tokens - 1) / tokens);
  split = split < most ? split : most;
  const int rounds = (most + split - 1) / split;
  p.heads_per_cta = rounds * groups;
  const dim3 grid(static_cast<unsigned>(tokens), (Htot + p.heads_per_cta - 1) / p.heads_per_cta);
  return dtype == Bf16::kId ? append_t<Bf16>(p, D, vec, grid, s) : append_t<F16>(p, D, vec, grid, s);
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

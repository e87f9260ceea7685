// ssd_target_api.cu -- the C-ABI entry points (include/ssd.h) of the target
// pass's operators: paged cache, tree attention, token log probabilities.
// Host-side argument checks and launches.
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>

#include "../../include/ssd.h"
#include "ssd_host.h"
#include "ssd_kv.cuh"

using namespace ssd;

static_assert(SSD_MAX_TREE_NODES == kMaxNodes, "a node's ancestors are one 64-bit mask");
static_assert(SSD_DEVERR_BAD_TREE == kErrBadTree && SSD_DEVERR_BAD_LENGTH == kErrBadLength &&
                  SSD_DEVERR_BAD_PAGE == kErrBadPage && SSD_DEVERR_BAD_LOGITS == kErrBadLogits &&
                  SSD_DEVERR_BAD_TOKEN == kErrBadToken && SSD_DEVERR_TIMEOUT == kErrTimeout &&
                  SSD_DEVERR_BAD_TEMPERATURE == kErrBadTemperature,
              "device error bits");

namespace {

// How long kernels wait for a copy, and (self-test) bytes that never come.
unsigned g_wait_us = 1000000;
int g_withheld = 0;

constexpr int64_t kMaxStride = 1ll << 38;

bool stride_ok(int64_t s) { return s > 0 && s % 8 == 0 && s < kMaxStride; }

ssd_status check_kv(const ssd_paged_kv* kv) {
  if (!kv) return SSD_ERR_INVALID_ARG;
  if (kv->dtype != SSD_BF16 && kv->dtype != SSD_F16) return SSD_ERR_UNSUPPORTED_DTYPE;
  if (!kv->k || !kv->v || !kv->page_table) return SSD_ERR_INVALID_ARG;
  if (kv->num_pages < 1 || kv->page_size < 1 || kv->Hkv < 1 || kv->max_pages < 1)
    return SSD_ERR_INVALID_ARG;
  if (kv->page_size > (1 << 20) || kv->Hkv > 1024) return SSD_ERR_INVALID_ARG;
  if (kv->D != 64 && kv->D != 128) return SSD_ERR_INVALID_ARG;
  if (kv->table_stride < kv->max_pages) return SSD_ERR_INVALID_ARG;
  // (slots are counted in 32 bits, rounded up to whole pages and tiles)
  if ((kv->max_pages + 1ll) * kv->page_size > INT32_MAX - 256) return SSD_ERR_INVALID_ARG;
  const int64_t s[6] = {kv->k_page, kv->k_slot, kv->k_head, kv->v_page, kv->v_slot, kv->v_head};
  for (int64_t x : s)
    if (!stride_ok(x) || x < kv->D) return SSD_ERR_INVALID_ARG;
  if (!aligned(kv->k, 16) || !aligned(kv->v, 16) || !aligned(kv->page_table, 4))
    return SSD_ERR_INVALID_ARG;
  return SSD_OK;
}

ssd_status check_nodes(const ssd_draft_nodes* n) {
  if (!n || !n->ctx_len) return SSD_ERR_INVALID_ARG;
  if (n->B < 1 || n->N < 1 || n->N > SSD_MAX_TREE_NODES) return SSD_ERR_INVALID_ARG;
  // (sequences and nodes are counted in 32 bits, rounded up to a block's threads)
  if (static_cast<int64_t>(n->B) * n->N > INT32_MAX - 1024) return SSD_ERR_INVALID_ARG;
  if (!aligned(n->ctx_len, 4) || !aligned(n->parent, 4) || !aligned(n->n_nodes, 4))
    return SSD_ERR_INVALID_ARG;
  return SSD_OK;
}

KvView view_of(const ssd_paged_kv& kv) {
  KvView v;
  v.k = static_cast<char*>(kv.k);
  v.v = static_cast<char*>(kv.v);
  v.k_page = kv.k_page; v.k_slot = kv.k_slot; v.k_head = kv.k_head;
  v.v_page = kv.v_page; v.v_slot = kv.v_slot; v.v_head = kv.v_head;
  v.pages = kv.num_pages; v.ps = kv.page_size; v.Hkv = kv.Hkv;
  v.table = kv.page_table; v.table_stride = kv.table_stride; v.width = kv.max_pages;
  return v;
}

NodesView view_of(const ssd_draft_nodes& n) {
  NodesView v;
  v.B = n.B; v.N = n.N;
  v.ctx_len = n.ctx_len; v.parent = n.parent; v.n_nodes = n.n_nodes;
  return v;
}

// n words at a and at b share some.
bool overlap(const int32_t* a, const int32_t* b, int n) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return (x > y ? x - y : y - x) < 4ull * n;
}

bool rows16(const void* p, int64_t a, int64_t b, int64_t c) {
  return aligned(p, 16) && a % 8 == 0 && b % 8 == 0 && c % 8 == 0;
}

}  // namespace

extern "C" {

ssd_status ssd_kv_append(const ssd_paged_kv* kv, const ssd_draft_nodes* nodes, int Hq, const void* q,
                         int64_t q_b, int64_t q_n, int64_t q_h, const void* k, const void* v,
                         int64_t kv_b, int64_t kv_n, int64_t kv_h, void* q_out, const float* cos_sin,
                         int max_pos, int rot, int interleaved, const void* q_norm,
                         const void* k_norm, float eps, void* ws, size_t ws_bytes,
                         ssd_stream_t stream) {
  CallRange nvtx_range("ssd_kv_append");
  ssd_status st = check_kv(kv);
  if (st == SSD_OK) st = check_nodes(nodes);
  if (st != SSD_OK) return st;
  if (!q || !k || !v || !q_out || !ws || Hq < 1 || Hq > 65536) return SSD_ERR_INVALID_ARG;
  if (q_b < 0 || q_n < 0 || q_h < 0 || kv_b < 0 || kv_n < 0 || kv_h < 0) return SSD_ERR_INVALID_ARG;
  if (!aligned(q, 2) || !aligned(k, 2) || !aligned(v, 2) || !aligned(q_out, 16) || !aligned(ws, 256))
    return SSD_ERR_INVALID_ARG;
  if (rot < 0 || rot > kv->D || rot % 16 != 0 || (rot > 0) != (cos_sin != nullptr))
    return SSD_ERR_INVALID_ARG;
  if (rot > 0 && (max_pos < 1 || !aligned(cos_sin, 16))) return SSD_ERR_INVALID_ARG;
  if ((q_norm == nullptr) != (k_norm == nullptr) || !aligned(q_norm, 2) || !aligned(k_norm, 2))
    return SSD_ERR_INVALID_ARG;
  if (q_norm && !(eps >= 0.f && eps < INFINITY)) return SSD_ERR_INVALID_ARG;
  if (ws_bytes < SSD_ERRWORD_BYTES) return SSD_ERR_WORKSPACE;
  AppendParams p;
  p.kv = view_of(*kv);
  p.nodes = view_of(*nodes);
  p.Hq = Hq; p.rot = rot; p.max_pos = max_pos; p.interleaved = interleaved != 0;
  p.q = static_cast<const char*>(q);
  p.k = static_cast<const char*>(k);
  p.v = static_cast<const char*>(v);
  p.q_b = q_b; p.q_n = q_n; p.q_h = q_h;
  p.kv_b = kv_b; p.kv_n = kv_n; p.kv_h = kv_h;
  p.q_out = static_cast<char*>(q_out);
  p.cos_sin = cos_sin;
  p.q_norm = static_cast<const char*>(q_norm);
  p.k_norm = static_cast<const char*>(k_norm);
  p.eps = eps;
  p.items = 0;
  p.all = 0;
  p.err = static_cast<int*>(ws);
  const bool vec = rows16(q, q_b, q_n, q_h) && rows16(k, kv_b, kv_n, kv_h) && aligned(v, 16);
  ProfScope ps("kv_append", S(stream));
  return cuda_status(launch_kv_append(p, kv->dtype, kv->D, vec, S(stream)));
}

size_t ssd_tree_attention_workspace_bytes(int B, int N, int Hq, int Hkv, int D) {
  if (B < 1 || N < 1 || N > SSD_MAX_TREE_NODES || Hkv < 1 || Hq < Hkv || Hq % Hkv != 0 ||
      Hq / Hkv > 64 || (D != 64 && D != 128))
    return 0;
  return tree_attention_bytes(N, Hq / Hkv, D);
}

ssd_status ssd_tree_attention(const ssd_paged_kv* kv, const ssd_draft_nodes* nodes, int Hq,
                              const void* q, int64_t q_b, int64_t q_n, int64_t q_h, float scale,
                              void* out, float* lse, void* ws, size_t ws_bytes,
                              ssd_stream_t stream) {
  CallRange nvtx_range("ssd_tree_attention");
  ssd_status st = check_kv(kv);
  if (st == SSD_OK) st = check_nodes(nodes);
  if (st != SSD_OK) return st;
  // (scores are counted in units of log 2)
  if (!q || !out || !ws || !isfinite(scale) || fabsf(scale) > 2e38f) return SSD_ERR_INVALID_ARG;
  if (Hq < kv->Hkv || Hq % kv->Hkv != 0 || Hq / kv->Hkv > 64) return SSD_ERR_INVALID_ARG;
  if (q_b < 0 || q_n < 0 || q_h < 0 || !rows16(q, q_b, q_n, q_h)) return SSD_ERR_INVALID_ARG;
  if (!aligned(out, 16) || !aligned(lse, 4) || !aligned(ws, 256)) return SSD_ERR_INVALID_ARG;
  if (ws_bytes < ssd_tree_attention_workspace_bytes(nodes->B, nodes->N, Hq, kv->Hkv, kv->D))
    return SSD_ERR_WORKSPACE;
  AttnParams p;
  p.kv = view_of(*kv);
  p.nodes = view_of(*nodes);
  p.Hq = Hq; p.G = Hq / kv->Hkv;
  p.q = static_cast<const char*>(q);
  p.q_b = q_b; p.q_n = q_n; p.q_h = q_h;
  p.scale = scale;
  p.out = static_cast<char*>(out);
  p.lse = lse;
  p.err = static_cast<int*>(ws);
  p.wait_us = g_wait_us;
  p.withheld = g_withheld;
  ProfScope ps("tree_attention", S(stream));
  return cuda_status(launch_tree_attention(p, kv->dtype, kv->D, S(stream)));
}

ssd_status ssd_kv_commit(const ssd_paged_kv* kv, int layers, int64_t k_layer, int64_t v_layer, int B,
                         int N, const int32_t* ctx_len, const int32_t* accept_len,
                         const int32_t* out_node, int32_t* new_len, void* ws, size_t ws_bytes,
                         ssd_stream_t stream) {
  CallRange nvtx_range("ssd_kv_commit");
  const ssd_status st = check_kv(kv);
  if (st != SSD_OK) return st;
  if (!ctx_len || !accept_len || !new_len || !ws) return SSD_ERR_INVALID_ARG;
  if (B < 1 || N < 1 || N > SSD_MAX_TREE_NODES || layers < 1) return SSD_ERR_INVALID_ARG;
  if (layers > 1 && (!stride_ok(k_layer) || !stride_ok(v_layer))) return SSD_ERR_INVALID_ARG;
  if (overlap(new_len, ctx_len, B) || overlap(new_len, accept_len, B)) return SSD_ERR_INVALID_ARG;
  if (!aligned(ctx_len, 4) || !aligned(accept_len, 4) || !aligned(out_node, 4) ||
      !aligned(new_len, 4) || !aligned(ws, 256))
    return SSD_ERR_INVALID_ARG;
  if (ws_bytes < SSD_ERRWORD_BYTES) return SSD_ERR_WORKSPACE;
  CommitParams p;
  p.kv = view_of(*kv);
  p.layers = layers; p.B = B; p.N = N; p.D = kv->D;
  p.k_layer = k_layer; p.v_layer = v_layer;
  p.ctx_len = ctx_len; p.accept_len = accept_len; p.out_node = out_node; p.new_len = new_len;
  p.layers_per_cta = 0;
  p.err = static_cast<int*>(ws);
  ProfScope ps("kv_commit", S(stream));
  return cuda_status(launch_kv_commit(p, S(stream)));
}

size_t ssd_logprobs_workspace_bytes(int R, int V, int K) {
  if (R < 1 || V < 1 || V > (1 << 28) || K < 0 || K > SSD_MAX_TOP) return 0;
  return logprobs_bytes(R, V, K);
}

ssd_status ssd_logprobs(const void* logits, ssd_dtype dtype, int64_t row_stride, int n_rows, int V,
                        const int32_t* rows, int R, const int32_t* tok, const float* T, int K,
                        float* logprob, float* entropy, int32_t* rank, int32_t* top_tok,
                        float* top_logprob, void* ws, size_t ws_bytes, ssd_stream_t stream) {
  CallRange nvtx_range("ssd_logprobs");
  if (!dtype_ok(dtype)) return SSD_ERR_UNSUPPORTED_DTYPE;
  if (!logits || !tok || !logprob || !ws) return SSD_ERR_INVALID_ARG;
  if (R > (1 << 26)) return SSD_ERR_INVALID_ARG;
  if (n_rows < 1 || V < 1 || V > (1 << 28) || row_stride < V || R < 1 || (!rows && R > n_rows))
    return SSD_ERR_INVALID_ARG;
  if (K < 0 || K > SSD_MAX_TOP || (K > 0 && (!top_tok || !top_logprob))) return SSD_ERR_INVALID_ARG;
  if (!aligned(logits, esize(dtype)) || !aligned(rows, 4) || !aligned(tok, 4) || !aligned(T, 4) ||
      !aligned(logprob, 4) || !aligned(entropy, 4) || !aligned(rank, 4) || !aligned(top_tok, 4) ||
      !aligned(top_logprob, 4) || !aligned(ws, 256))
    return SSD_ERR_INVALID_ARG;
  if (ws_bytes < ssd_logprobs_workspace_bytes(R, V, K)) return SSD_ERR_WORKSPACE;
  LogprobParams p = {};
  p.logits = logits; p.row_stride = row_stride; p.n_rows = n_rows; p.V = V; p.R = R; p.K = K;
  p.rows = rows; p.tok = tok; p.T = T;
  p.logprob = logprob; p.entropy = entropy; p.rank = rank;
  p.top_tok = top_tok; p.top_logprob = top_logprob;
  p.err = static_cast<int*>(ws);
  p.wait_us = g_wait_us;
  p.withheld = g_withheld;
  const bool vec = aligned(logits, 16) && (static_cast<size_t>(row_stride) * esize(dtype)) % 16 == 0;
  ProfScope ps("logprobs", S(stream));
  return cuda_status(launch_logprobs(p, dtype == SSD_BF16 ? 1 : 0, vec, S(stream)));
}

ssd_status ssd_selftest_copy_wait(int limit_us, int withhold) {
  if (limit_us < 0 || limit_us > 1000000) return SSD_ERR_INVALID_ARG;
  g_wait_us = limit_us ? limit_us : 1000000;
  g_withheld = withhold ? 16 : 0;
  return SSD_OK;
}

int ssd_selftest_kv_slot(const int32_t* table_row, int max_pages, int num_pages, int page_size,
                         int64_t slot, int32_t* page, int32_t* off) {
  if (!table_row || !page || !off || page_size < 1) return 0;
  int pg, of;
  const bool ok = kv_slot(table_row, max_pages, num_pages, page_size, slot, pg, of);
  *page = pg;
  *off = of;
  return ok;
}

int ssd_selftest_node(const int32_t* parent, int n, int j, uint64_t* mask, int32_t* depth) {
  if (!mask || !depth || n > kMaxNodes) return 0;
  uint64_t m;
  int d;
  bool broken;
  const bool ok = node_way(parent, n, j, m, d, broken);
  *mask = m;
  *depth = d;
  return ok;
}

}  // extern "C"

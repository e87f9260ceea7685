// ssd_kv.cuh -- the paged cache and the drafted nodes as the kernels see them:
// page lookup, the walk from a node to its root, 16-bit element types.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace ssd {

constexpr int kMaxNodes = 64;  // SSD_MAX_TREE_NODES: a node's ancestors are one 64-bit mask

struct KvView {
  char* k;
  char* v;
  long long k_page, k_slot, k_head;  // elements
  long long v_page, v_slot, v_head;
  int pages, ps, Hkv;
  const int* table;
  long long table_stride;
  int width;  // pages of a sequence's table row
};

struct NodesView {
  int B, N;
  const int* ctx_len;
  const int* parent;   // null: a chain
  const int* n_nodes;  // null: N
};

// The number of nodes of a sequence (0 when its lengths are out of range,
// with bad = true).
__host__ __device__ inline int seq_nodes(int ctx, int n, int N, int width, int ps, bool& bad) {
  bad = ctx < 0 || n < 0 || n > N ||
        static_cast<long long>(ctx) + n > static_cast<long long>(width) * ps;
  return bad ? 0 : n;
}

// Page and entry of a slot; false where the table row has no such page.
__host__ __device__ inline bool kv_slot(const int* row, int width, int pages, int ps,
                                        long long slot, int& page, int& off) {
  const long long p = slot / ps;
  page = -1;
  off = static_cast<int>(slot - p * ps);
  if (slot < 0 || p >= width) return false;
  page = row[p];
  return static_cast<unsigned>(page) < static_cast<unsigned>(pages);
}

// Node j of a sequence of n nodes: the mask of its ancestors and itself and
// its depth; false for an absent node.  The walk is strictly decreasing, so
// it ends.  (A node >= n is absent without an error; broken = true marks a
// broken way.)
__host__ __device__ inline bool node_way(const int* parent, int n, int j, uint64_t& mask,
                                         int& depth, bool& broken) {
  broken = false;
  mask = 0;
  depth = 0;
  if (j < 0 || j >= n) return false;
  if (!parent) {
    mask = j == 63 ? ~0ull : (2ull << j) - 1;
    depth = j;
    return true;
  }
  uint64_t m = 1ull << j;
  int i = j, d = 0;
#ifdef __CUDA_ARCH__
#pragma unroll 1
#endif
  while (i > 0) {
    const int p = parent[i];
    if (p < 0 || p >= i) {
      broken = true;
      return false;
    }
    m |= 1ull << p;
    i = p;
    ++d;
  }
  if (parent[0] != -1) {
    broken = true;
    return false;
  }
  mask = m;
  depth = d;
  return true;
}

// ---------------------------------------------------------------------------
// 16-bit element types
// ---------------------------------------------------------------------------
struct Bf16 {
  static constexpr int kId = 1;  // SSD_BF16
  __device__ __forceinline__ static float lo(uint32_t w) { return __uint_as_float(w << 16); }
  __device__ __forceinline__ static float hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
  // two floats rounded to nearest even, lo in the low half
  __device__ __forceinline__ static uint32_t pack(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
};

struct F16 {
  static constexpr int kId = 2;  // SSD_F16
  __device__ __forceinline__ static float lo(uint32_t w) {
    return __half2float(__ushort_as_half(static_cast<unsigned short>(w)));
  }
  __device__ __forceinline__ static float hi(uint32_t w) {
    return __half2float(__ushort_as_half(static_cast<unsigned short>(w >> 16)));
  }
  __device__ __forceinline__ static uint32_t pack(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
};

// ---------------------------------------------------------------------------
// kernel arguments
// ---------------------------------------------------------------------------
struct AppendParams {
  KvView kv;
  NodesView nodes;
  int Hq, rot, max_pos, interleaved;
  const char* q;
  const char* k;
  const char* v;
  long long q_b, q_n, q_h, kv_b, kv_n, kv_h;
  char* q_out;
  const float* cos_sin;
  const char* q_norm;
  const char* k_norm;
  float eps;
  int items;      // (token, head) pairs of a CTA
  long long all;  // of the call
  int* err;
};

struct CommitParams {
  KvView kv;
  int layers, B, N, D;
  long long k_layer, v_layer;
  const int* ctx_len;
  const int* accept_len;
  const int* out_node;
  int* new_len;
  int layers_per_cta;
  int* err;
};

struct AttnParams {
  KvView kv;
  NodesView nodes;
  int Hq, G;
  const char* q;
  long long q_b, q_n, q_h;
  float scale;
  char* out;
  float* lse;
  int* err;
  unsigned wait_us;      // a copy that takes longer has failed
  int withheld;          // bytes that are waited for beside the copied ones (self-test)
};

// A part of a row, as its CTA leaves it.
struct LogprobPart {
  float m, S, U;
  int count;
};

struct LogprobParams {
  const void* logits;
  long long row_stride;
  int n_rows, V, R, K;
  const int* rows;
  const int* tok;
  const float* T;
  float* logprob;
  float* entropy;
  int* rank;
  int* top_tok;
  float* top_logprob;
  bool whole;            // rows are 16-byte aligned
  int split;             // parts of a row
  int* counter;          // [R] parts done (0 between calls)
  LogprobPart* parts;    // [R, split]
  unsigned long long* part_key;  // [R, split, 32] the parts' best
  int* err;
  unsigned wait_us;      // a copy that takes longer has failed
  int withheld;          // bytes that are waited for beside the copied ones (self-test)
};

constexpr int kErrBadTemperature = 0x1, kErrBadLogits = 0x2, kErrBadToken = 0x4, kErrTimeout = 0x10,
              kErrBadTree = 0x40, kErrBadLength = 0x80, kErrBadPage = 0x100;

cudaError_t launch_kv_append(const AppendParams& p, int dtype, int D, bool vec, cudaStream_t s);
cudaError_t launch_kv_commit(const CommitParams& p, cudaStream_t s);
cudaError_t launch_tree_attention(const AttnParams& p, int dtype, int D, cudaStream_t s);
size_t tree_attention_bytes(int N, int G, int D);
size_t logprobs_bytes(int R, int V, int K);
cudaError_t launch_logprobs(const LogprobParams& p, int dtype, bool vec, cudaStream_t s);

}  // namespace ssd

/*
 * ssd.h -- C ABI of the GB300 verify-and-recover library for speculative
 * decoding (SD) and Speculative Speculative Decoding (SSD).
 *
 * Sources (page title, section):
 *   [SUM]  "tanishqkumar/ssd" repository summary (thehardwarestore.ai),
 *          module notes: the sampler mixes greedy and stochastic sampling by
 *          temperature; get_forked_recovery_tokens_from_logits picks tokens by
 *          top-k over logits with masking for cache hits and misses.
 *   [SSD]  "SSD: drafting and verification on separate GPUs, in parallel"
 *          (hysenlabs.com), "What changes in SSD": the target verifies the
 *          draft in one forward pass; the method is exact; the drafter
 *          pre-speculates likely outcomes and a correct guess is returned at
 *          once; the roadmap's speculation cache.
 *   [SPS]  speculative-sampling project summary (sourcepulse.org 1842340),
 *          "How It Works": accept correct tokens, regenerate from the point of
 *          divergence; Google's and DeepMind's algorithms.
 *   [LKM]  the rule those algorithms share (Leviathan et al. 2023, Chen et
 *          al. 2023): accept x_i with probability min(1, p_i(x_i)/q_i(x_i));
 *          at the first rejection n draw from norm(max(0, p_n - q_n)); after
 *          k accepts draw the bonus token from p_k.
 *
 * Conventions shared by every call:
 *   - Tensor arguments are DEVICE pointers owned by the caller, unless a
 *     parameter says "host".  Nothing is allocated per call; scratch comes
 *     from a caller-supplied workspace (ssd_workspace_bytes) or from a
 *     speculation cache made once by ssd_spec_cache_create.
 *   - All work is enqueued on `stream` (a cudaStream_t; NULL = legacy
 *     default stream) and the call returns after enqueueing.
 *   - Logits are row-major: row (b, i) of a [B, P, V] tensor starts at
 *     element b*bstride + i*V.  dtype is SSD_F32 or SSD_BF16; bf16 is widened
 *     to fp32 exactly before any arithmetic.
 *   - Every call returns an ssd_status; no call aborts or throws.  Argument
 *     errors are found on the host before anything is enqueued.  Errors in
 *     the DATA (invalid temperature, NaN logits, out-of-range tokens, a full
 *     cache) become per-row sentinels plus bits in a device error word, read
 *     by ssd_get_device_error.
 *   - Pointers need 4-byte alignment; logits, when the base pointer, V and
 *     bstride all give 16-byte aligned rows, are read with 16-byte vector
 *     loads, otherwise with scalar loads.
 *   - A workspace must be zero-filled once before its first use (cudaMemset
 *     or ssd_workspace_init); the calls keep it consistent afterwards.
 *   - Calls that share a workspace must not overlap on the GPU.
 */
#ifndef SSD_GB300_H
#define SSD_GB300_H

#include <stddef.h>
#include <stdint.h>

#if defined(__GNUC__)
#define SSD_API __attribute__((visibility("default")))
#else
#define SSD_API
#endif

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st *ssd_stream_t; /* same type as cudaStream_t */

typedef enum {
    SSD_OK = 0,
    SSD_ERR_INVALID_ARG = 1,
    SSD_ERR_UNSUPPORTED_DTYPE = 2,
    SSD_ERR_CUDA = 3,
    SSD_ERR_CACHE_FULL = 4,
    SSD_ERR_TIMEOUT = 5,
    SSD_ERR_WORKSPACE = 6
} ssd_status;

/* SSD_F16 is a type of the paged-cache calls only; logits are SSD_F32 or
 * SSD_BF16. */
typedef enum { SSD_F32 = 0, SSD_BF16 = 1, SSD_F16 = 2 } ssd_dtype;

/* Bits of the device error word (ssd_get_device_error). */
#define SSD_DEVERR_BAD_TEMPERATURE 0x1 /* T < 0 or NaN: row sentinel -1   */
#define SSD_DEVERR_BAD_LOGITS 0x2      /* NaN (or +inf / all -inf at T>0) */
#define SSD_DEVERR_BAD_TOKEN 0x4       /* draft token outside [0, V): -2  */
#define SSD_DEVERR_CACHE_FULL 0x8      /* insert found no free slot       */
#define SSD_DEVERR_TIMEOUT 0x10        /* a bounded device wait ran out   */
#define SSD_DEVERR_FILTER_BAND 0x20    /* a filtered row's cut fell outside its collected
                                          bins; it was cut by bisection (results exact) */
#define SSD_DEVERR_BAD_TREE 0x40       /* a node whose way to the root is broken, or an
                                          accepted path that is none: left out */
#define SSD_DEVERR_BAD_LENGTH 0x80     /* a length, node count or position out of range:
                                          the sequence (or node) is left out */
#define SSD_DEVERR_BAD_PAGE 0x100      /* a page id outside [0, num_pages)  */

/* Sentinels written to accept_len. */
#define SSD_ROW_INVALID (-1)
#define SSD_ROW_BAD_TOKEN (-2)

/* Limits checked on the host. */
#define SSD_MAX_K 31   /* draft length: one warp ballot holds k flags */
#define SSD_MAX_F 16   /* forked recovery fan-out                    */
#define SSD_MAX_M 64   /* masked tokens per (b, position)            */
#define SSD_MAX_TREE_NODES 64  /* nodes of one draft tree              */

SSD_API const char *ssd_status_string(ssd_status s);

/* Library version (major*10000 + minor*100 + patch). */
SSD_API int ssd_version(void);

/*
 * Streams, graphs, batch size.  Every call enqueues work on the caller's
 * stream and returns: no device allocation, no host synchronisation (except
 * the error-word reads, which say so).  The verify calls (all but
 * ssd_verify_noalloc) run the target-row and draft-row statistics on two
 * internal streams forked from and joined back to the caller's stream by
 * events (the draft-row stream at the device's greatest priority), and the
 * SSD round step inserts the forks into the cache on a third one, also at
 * the greatest priority, beside the draw; the streams and events are
 * created on the first such call on a device.  Calls can therefore be captured into a CUDA
 * graph (make one verify call on the device before capturing).  B may exceed
 * 65535: kernels launch in grids of 65535 batch rows.
 */

/*
 * Workspace bytes for ssd_verify / ssd_verify_fork / ssd_sample_residual /
 * ssd_forked_recovery on batch B, draft length k, vocabulary V and fan-out
 * f (0 if no forked recovery).  Returns 0 for invalid sizes.
 */
SSD_API size_t ssd_workspace_bytes(int B, int k, int V, int f);

/* Workspace bytes for ssd_softmax_temp on `rows` rows of V logits. */
SSD_API size_t ssd_softmax_workspace_bytes(int rows, int V);

/* Zero-fill `bytes` of workspace `ws` on `stream` (one cudaMemsetAsync). */
SSD_API ssd_status ssd_workspace_init(void *ws, size_t bytes, ssd_stream_t stream);

/*
 * Read (and, if clear != 0, reset) the device error word of a workspace or
 * of a speculation cache workspace.  Synchronises `stream`.  *out is a host
 * int32 receiving an OR of SSD_DEVERR_* bits.
 */
SSD_API ssd_status ssd_get_device_error(void *ws, ssd_stream_t stream, int32_t *out,
                                int clear);

/*
 * ssd_softmax_temp -- temperature softmax per row ([SUM] sampler: greedy at
 * temperature 0, stochastic otherwise).
 *   logits : [rows, V] (dtype)
 *   T      : [rows] fp32 temperatures.  T == 0 rows give the greedy
 *            distribution: a one-hot at the argmax (lowest index on ties),
 *            row_sum = 1.  T < 0 / NaN or an invalid row give m = S = NaN,
 *            argmax = -1, probs = NaN and set the error word.
 *   probs  : [rows, V] fp32 or NULL.  p_v = exp((z_v - m)/T) / S.
 *   row_max, row_sum : [rows] fp32, m = max z, S = sum exp((z - m)/T).
 *   row_argmax : [rows] int32.
 *   ws     : ssd_softmax_workspace_bytes(rows, V) bytes.
 */
SSD_API ssd_status ssd_softmax_temp(const void *logits, ssd_dtype dtype, int rows, int V,
                            const float *T, float *probs, float *row_max,
                            float *row_sum, int32_t *row_argmax, void *ws,
                            size_t ws_bytes, ssd_stream_t stream);

/*
 * ssd_verify -- acceptance, first-reject prefix and (optionally) the
 * recovery/bonus draw, in one call ([SSD] verify in one pass; [SPS] point of
 * divergence; [LKM] the rule).
 *   Z        : target logits [B, k+1, V], batch stride z_bstride elements.
 *   D        : draft logits [B, >=k, V], batch stride d_bstride; rows
 *              0..k-1 are read.
 *   x        : [B, k] int32 draft tokens.   T : [B] fp32 temperatures, used
 *              for target and draft rows alike; T == 0 is greedy.
 *   u_acc    : [B, k] fp32 uniforms in [0, 1).  Draft token i is accepted
 *              iff u_acc[b,i] < p_i(x_i) / q_i(x_i) (q == 0: iff p > 0);
 *              greedy rows accept iff x_i == argmax Z[b,i].
 *   accept_len : [B] int32 out: n in 0..k, or SSD_ROW_INVALID /
 *              SSD_ROW_BAD_TOKEN.
 *   p_at_x, q_at_x : [B, k] fp32 out or NULL: p_i(x_i), q_i(x_i) (greedy:
 *              1 if x_i is the argmax of that row, else 0).
 *   u_smp    : [B] fp32 uniforms, or NULL to skip the draw.
 *   out_tok  : [B, k+1] int32 out, required when u_smp is given: the n
 *              accepted tokens, then the drawn token, then -1.  The draw is
 *              the smallest j with C_j > u_smp * C_{V-1}, C the prefix sum of
 *              w = max(0, p_n - q_n) (n < k; if w is all zero, w = p_n) or of
 *              w = p_k (n == k); greedy rows take argmax Z[b,n].
 *   ws       : ssd_workspace_bytes(B, k, V, 0) bytes (or more).
 */
SSD_API ssd_status ssd_verify(const void *Z, int64_t z_bstride, const void *D,
                      int64_t d_bstride, ssd_dtype dtype, int B, int k, int V,
                      const int32_t *x, const float *T, const float *u_acc,
                      int32_t *accept_len, float *p_at_x, float *q_at_x,
                      const float *u_smp, int32_t *out_tok, void *ws,
                      size_t ws_bytes, ssd_stream_t stream);

/*
 * ssd_verify_noalloc -- ssd_verify for callers that cannot allocate device
 * memory (the pages have no counterpart; this is a deployment aid).  Some
 * callers cannot call cudaMalloc or an allocating library routine: code that
 * runs inside a framework that owns every allocation, or a process whose
 * device memory is fully pre-reserved.  This call takes no workspace: its
 * scratch is a file-scope device array of SSD_NOALLOC_SCRATCH_BYTES (8 MiB)
 * that every GPU which loads the library holds until exit.
 *   - Arguments and results are those of ssd_verify without ws/ws_bytes.
 *   - Sizes whose workspace (ssd_workspace_bytes(B, k, V, 0)) exceeds the
 *     array return SSD_ERR_WORKSPACE before anything is enqueued.
 *   - The first call on a device looks up the array's device address
 *     (cudaGetSymbolAddress) with that device current; make that first call
 *     before any stream capture.
 *   - Every call shares the one array, which keeps the last call's contents;
 *     each call writes every part it reads, so nothing needs clearing.  Calls
 *     that overlap on the GPU (other streams, other host threads) race.
 *   - The array's device error word is not exposed: data errors show as the
 *     accept_len sentinels.
 *   - u_smp may be NULL (out_tok then too): acceptance only.  T > 0 rows then
 *     get no recovery / bonus token (out_tok[b][n] = -1, if out_tok is
 *     given), and no later call can draw it, because ssd_sample_residual
 *     needs the statistics in a workspace this call does not expose.
 *   - Argument checks run before the array is touched: invalid sizes return
 *     SSD_ERR_INVALID_ARG, sizes beyond the array SSD_ERR_WORKSPACE, then
 *     null or misaligned pointers SSD_ERR_INVALID_ARG.
 */
#define SSD_NOALLOC_SCRATCH_BYTES (8u << 20)
SSD_API ssd_status ssd_verify_noalloc(const void *Z, int64_t z_bstride, const void *D,
                                      int64_t d_bstride, ssd_dtype dtype, int B, int k, int V,
                                      const int32_t *x, const float *T, const float *u_acc,
                                      int32_t *accept_len, float *p_at_x, float *q_at_x,
                                      const float *u_smp, int32_t *out_tok,
                                      ssd_stream_t stream);

/*
 * ssd_sample_residual -- the recovery/bonus draw alone, after an ssd_verify
 * call on the same workspace, inputs and sizes that was given u_smp = NULL.
 * accept_len may be that call's output or any values in 0..k (negative
 * entries are skipped).  Writes out_tok [B, k+1] as ssd_verify does.
 */
SSD_API ssd_status ssd_sample_residual(const void *Z, int64_t z_bstride, const void *D,
                               int64_t d_bstride, ssd_dtype dtype, int B, int k,
                               int V, const int32_t *x, const float *T,
                               const int32_t *accept_len, const float *u_smp,
                               int32_t *out_tok, void *ws, size_t ws_bytes,
                               ssd_stream_t stream);

/*
 * ssd_forked_recovery -- SSD's forked recovery tokens ([SUM]
 * get_forked_recovery_tokens_from_logits: top-k over logits with masking).
 *   L        : [B, P, V] logits, batch stride l_bstride.
 *   mask     : [B, P, M] int32 tokens to skip at each (b, j) (entries
 *              outside [0, V) skip nothing); may be NULL when M == 0.
 *   fork_tok : [B, P, f] int32 out, fork_logit : [B, P, f] fp32 out: the f
 *              largest unmasked logits of each row, logit descending then
 *              index ascending.  Missing candidates are (-1, -inf); a row
 *              holding a NaN gives (-1, NaN) and sets the error word.
 *   ws       : ssd_workspace_bytes(B, P-1, V, f) bytes (or more).
 */
SSD_API ssd_status ssd_forked_recovery(const void *L, int64_t l_bstride, ssd_dtype dtype,
                               int B, int P, int V, int f, const int32_t *mask,
                               int M, int32_t *fork_tok, float *fork_logit,
                               void *ws, size_t ws_bytes, ssd_stream_t stream);

/*
 * ssd_verify_fork -- ssd_verify and ssd_forked_recovery over the draft
 * buffer in one pass over the logits.  D must hold P = k+1 rows per batch
 * row (the SSD draft: rows 0..k-1 feed acceptance, rows 0..k the forked
 * recovery).  Arguments as in the two calls; ws: ssd_workspace_bytes(B, k,
 * V, f).
 */
SSD_API ssd_status ssd_verify_fork(const void *Z, int64_t z_bstride, const void *D,
                           int64_t d_bstride, ssd_dtype dtype, int B, int k,
                           int V, const int32_t *x, const float *T,
                           const float *u_acc, int32_t *accept_len,
                           float *p_at_x, float *q_at_x, const float *u_smp,
                           int32_t *out_tok, int f, const int32_t *mask, int M,
                           int32_t *fork_tok, float *fork_logit, void *ws,
                           size_t ws_bytes, ssd_stream_t stream);

/*
 * Variable fan-out ([SUM] get_forked_recovery_tokens_from_logits: selection
 * by fan-out strategy).  As ssd_forked_recovery / ssd_verify_fork with
 * F (<= SSD_MAX_F) in place of f, plus
 *   fanout   : [P] int32 device array, f_j tokens kept at position j
 *              (clamped to [0, F]).  fork_tok / fork_logit stay [B, P, F]:
 *              slots f_j .. F-1 of position j hold (-1, -inf), which the
 *              cache insert skips.  NULL keeps F everywhere.
 *   ws       : sized with f = F.
 */
SSD_API ssd_status ssd_forked_recovery_fanout(const void *L, int64_t l_bstride,
                                      ssd_dtype dtype, int B, int P, int V, int F,
                                      const int32_t *fanout, const int32_t *mask,
                                      int M, int32_t *fork_tok, float *fork_logit,
                                      void *ws, size_t ws_bytes, ssd_stream_t stream);
SSD_API ssd_status ssd_verify_fork_fanout(const void *Z, int64_t z_bstride,
                                  const void *D, int64_t d_bstride, ssd_dtype dtype,
                                  int B, int k, int V, const int32_t *x,
                                  const float *T, const float *u_acc,
                                  int32_t *accept_len, float *p_at_x, float *q_at_x,
                                  const float *u_smp, int32_t *out_tok, int F,
                                  const int32_t *fanout, const int32_t *mask, int M,
                                  int32_t *fork_tok, float *fork_logit, void *ws,
                                  size_t ws_bytes, ssd_stream_t stream);

/*
 * ssd_draft_sample -- the drafter's tokens, drawn on the GPU ([SUM] sampler:
 * greedy at temperature 0, stochastic otherwise; [SPS] the small model
 * proposes the draft), fused with the draft rows' statistics so that a later
 * ssd_verify_drafted reads only the target rows.
 *   D        : draft logits [B, >= row0+rows, V], batch stride d_bstride.
 *   k        : the verify call's draft length (sizes and places the
 *              statistics in ws); rows [row0, row0+rows) with
 *              row0 + rows <= k + 1 (row k: SSD's next-round token).
 *   T        : [B] fp32; the verify call must use the same temperatures.
 *   seed, offset : the draw of element v of row i of batch row b uses word
 *              v mod 4 of Philox4x32-10 (Salmon et al. 2011) at counter
 *              (v / 4, i, b, offset) under key (seed low, seed high 32 bits)
 *              and u = ((w >> 9) + 1/2) / 2^23.
 *   x_out    : x_out[b * x_bstride + (i - row0)] = the token: T > 0 the
 *              Gumbel-max draw argmax_v (z_v / T - ln(-ln u_v)) (an exact
 *              draw from softmax(z / T); ties to the lowest index); T == 0
 *              the argmax; -1 for T < 0 / NaN or an invalid row (device
 *              error word set).
 *   f, fork_tok, fork_logit : f >= 1 also writes [B, rows, f] forks: the f
 *              largest logits of each row other than its drafted token (SSD
 *              forked recovery with the drafter's token masked); f == 0
 *              writes none (pointers may be NULL).  f + 1 <= SSD_MAX_F.
 *   ws       : ssd_workspace_bytes(B, k, V, f > 0 ? f + 1 : 0) bytes; the
 *              same workspace goes to ssd_verify_drafted.
 */
SSD_API ssd_status ssd_draft_sample(const void *D, int64_t d_bstride, ssd_dtype dtype, int B,
                            int k, int V, int row0, int rows, const float *T,
                            uint64_t seed, uint32_t offset, int32_t *x_out,
                            int64_t x_bstride, int f, int32_t *fork_tok,
                            float *fork_logit, void *ws, size_t ws_bytes,
                            ssd_stream_t stream);

/*
 * ssd_verify_drafted -- ssd_verify whose draft rows 0..k-1 were already
 * summarised into ws by ssd_draft_sample calls (same B, k, V, T and ws):
 * the streaming pass reads only the k+1 target rows; D is still read at the
 * draft tokens and, for the recovery draw, at row n.  Arguments and results
 * as ssd_verify.
 */
SSD_API ssd_status ssd_verify_drafted(const void *Z, int64_t z_bstride, const void *D,
                              int64_t d_bstride, ssd_dtype dtype, int B, int k, int V,
                              const int32_t *x, const float *T, const float *u_acc,
                              int32_t *accept_len, float *p_at_x, float *q_at_x,
                              const float *u_smp, int32_t *out_tok, void *ws,
                              size_t ws_bytes, ssd_stream_t stream);

/*
 * ssd_verify_topk -- ssd_verify over top-k / top-p filtered distributions:
 * the target rows and the draft rows are filtered alike (order the tokens by
 * logit descending, index ascending; keep the first K; keep the shortest
 * prefix of those holding >= top_p[b] of their probability mass;
 * renormalise), and acceptance, the residual and the bonus draw use the
 * filtered p and q.  Greedy rows (T == 0) are unaffected.
 *   K        : K >= 1; K >= V keeps every token (top-p over the whole
 *              vocabulary).  min(K, V) <= 32: one pass over the 2k+1 rows
 *              keeps per-chunk top-K lists (no exponentials) and the rest
 *              works on at most K candidates per row.  Larger K: each row's
 *              kept set is found as a threshold on the token order (a row
 *              maximum pass, a histogram pass of x = (m - z) log2(e) / T in
 *              1/16 steps, a pass that sums the exact mass above the bins
 *              holding the cuts and collects those bins' tokens, an exact
 *              cut on them; see ssd_filter.cu), three reads of the rows in
 *              all.  A row whose cut bins hold more than 2048 tokens (e.g.
 *              thousands of equal logits) is cut by bisection on the token
 *              order, slower but exact.  V <= 2^21 on this path.
 *   top_p    : [B] fp32 device array, or NULL for 1 (no cut).  Values >= 1
 *              or NaN cut nothing.
 *   other arguments and results as ssd_verify (the draft tokens x must have
 *   been drawn from the filtered draft distribution for exactness).
 *   ws       : ssd_topk_workspace_bytes(B, k, V, K) bytes (0 for invalid
 *              sizes).
 * Mass sums and the top-p cut are exact to ~1e-12 relative (extended
 * precision exponentials, fixed-point sums), so a cut differs from an exact
 * computation only when the cumulative mass at the cut lies that close to
 * top_p times the kept tokens' mass.
 */
SSD_API size_t ssd_topk_workspace_bytes(int B, int k, int V, int K);
SSD_API ssd_status ssd_verify_topk(const void *Z, int64_t z_bstride, const void *D,
                           int64_t d_bstride, ssd_dtype dtype, int B, int k, int V,
                           const int32_t *x, const float *T, int K, const float *top_p,
                           const float *u_acc, int32_t *accept_len, float *p_at_x,
                           float *q_at_x, const float *u_smp, int32_t *out_tok, void *ws,
                           size_t ws_bytes, ssd_stream_t stream);

/*
 * ssd_verify_tree -- verification of a draft token tree per batch row (the
 * "tanishqkumar/ssd" summary's tree decoding), by the multi-step speculative
 * sampling of SpecInfer (Miao et al. 2024), which keeps the target's output
 * law when the children of a node were drawn independently from the
 * draft's q at that node:
 *   start at the root with r = p(root); try the children of the current
 *   node in increasing node index; child x is accepted when
 *   u_acc[b, child] < r(x) / q(x) (q(x) == 0: accepted iff r(x) > 0); an
 *   accepted child becomes the current node with r = its p; a rejection
 *   replaces r by norm(max(0, r - q)) (unchanged if that is all zero); when
 *   the children are exhausted the final token is drawn from r by inverse
 *   CDF with u_smp[b] (smallest v whose prefix sum exceeds u times the
 *   total).  T == 0 rows accept the first child whose token is the argmax
 *   (lowest index) of the current node's target row and end with that
 *   argmax.
 * One streaming pass over the N target rows and the inner nodes' draft rows
 * gives each row's maximum, argmax and sum; then a thread-block cluster per
 * batch row walks the tree, with one pass over the current node's two rows
 * per rejection (the next residual mass) and one for the final draw when it
 * is not already known.
 *   Z        : target logits at the nodes, row (b, j) at Z + b*z_bstride +
 *              j*V (the target's logits after node j's path; node 0 is the
 *              last committed position).  z_bstride >= N*V.
 *   D        : draft logits at the nodes, same layout (q of node j's
 *              children).  Only the rows of nodes that have children are
 *              read and checked: a leaf's q is never used.
 *   N        : nodes per tree, 1 <= N <= SSD_MAX_TREE_NODES.
 *   parent   : [B, N] int32 device: parent[b, 0] == -1, 0 <= parent[b, j] < j.
 *   tok      : [B, N] int32 device: node j's token (entry 0 unused).
 *   T        : [B] temperatures; u_acc: [B, N] uniforms in [0, 1), entry
 *              (b, j) tests node j (entry 0 unused); u_smp: [B].
 *   accept_len : [B] accepted nodes (path depth), or a sentinel: -1 for
 *              T < 0 or NaN or an invalid row (as ssd_verify), -2 for an
 *              invalid tree (parent or token out of range).
 *   out_tok  : [B, N]: the accepted tokens in path order, the final token,
 *              then -1 (all -1 on a sentinel).
 *   out_node : [B, N] or NULL: the accepted node ids, then -1.
 *   ws       : ssd_tree_workspace_bytes(B, N, V) bytes (its first word is
 *              the device error word, as for ssd_verify).  For V >= 32768
 *              it includes a cache of 16 (V + 32768) bytes per tree, where a
 *              node's first residual pass keeps each element's two
 *              exponentials for the later passes at that node.
 * Errors: SSD_ERR_INVALID_ARG for null required pointers, sizes out of
 * range, strides below N*V or misaligned pointers; SSD_ERR_WORKSPACE when
 * ws_bytes is too small; SSD_ERR_CUDA when a launch fails.
 */
SSD_API size_t ssd_tree_workspace_bytes(int B, int N, int V);
SSD_API ssd_status ssd_verify_tree(const void *Z, int64_t z_bstride, const void *D,
                           int64_t d_bstride, ssd_dtype dtype, int B, int N, int V,
                           const int32_t *parent, const int32_t *tok, const float *T,
                           const float *u_acc, const float *u_smp, int32_t *accept_len,
                           int32_t *out_tok, int32_t *out_node, void *ws, size_t ws_bytes,
                           ssd_stream_t stream);

/*
 * Speculation cache ([SSD] roadmap: the speculation cache; [SUM] cache
 * hits and misses).  An open-addressing table on the device mapping the key
 * (b, position, token) to `depth` draft tokens.  Keys compare exactly, so the
 * hash only decides slots, never results.  Inserts apply in input order (the
 * last duplicate wins, also across calls).  The call order is counted on the
 * device, so inserts into one cache must be ordered on one stream (or joined
 * by events); an insert captured in a CUDA graph keeps the rule on every
 * replay.  Probing is bounded by the capacity: an insert that finds no slot
 * is dropped and sets SSD_DEVERR_CACHE_FULL.  Limits: b < 2^24,
 * position < 256, token >= 0.
 */
typedef struct ssd_spec_cache ssd_spec_cache;

/* capacity: power of two >= 2; depth >= 1.  Allocates device memory once
 * (on the current device). */
SSD_API ssd_status ssd_spec_cache_create(int capacity, int depth, ssd_spec_cache **out);
SSD_API void ssd_spec_cache_destroy(ssd_spec_cache *cache);
SSD_API ssd_status ssd_spec_cache_clear(ssd_spec_cache *cache, ssd_stream_t stream);

/*
 * ssd_verify_fork_cache -- one SSD round step ([SSD] the drafter keeps
 * speculations for the likely verification outcomes; a correct guess is
 * returned at once): ssd_verify_fork, then (after clearing the cache when
 * clear != 0) the forks go into `cache` keyed (b, position, fork token) with
 * payload rows payload[((b*(k+1) + j)*f + r) * depth ..], and each row's
 * realised outcome (accept_len[b], out_tok[b, accept_len[b]]) is looked up:
 * hit[b] in {0, 1}, tok_out[b, 0..depth) (-1 on a miss).  With B >= 32 the
 * clear and the insert run on an internal stream while the recovery draw
 * runs.  Arguments otherwise as ssd_verify_fork (out_tok required); the
 * cache must live on the current device.
 */
SSD_API ssd_status ssd_verify_fork_cache(const void *Z, int64_t z_bstride, const void *D,
                                 int64_t d_bstride, ssd_dtype dtype, int B, int k, int V,
                                 const int32_t *x, const float *T, const float *u_acc,
                                 int32_t *accept_len, float *p_at_x, float *q_at_x,
                                 const float *u_smp, int32_t *out_tok, int f,
                                 const int32_t *mask, int M, int32_t *fork_tok,
                                 float *fork_logit, ssd_spec_cache *cache, int clear,
                                 const int32_t *payload, int32_t *hit, int32_t *tok_out,
                                 void *ws, size_t ws_bytes, ssd_stream_t stream);

/* n keys (b[i], pos[i], tok[i]) -> payload[i*depth .. +depth). */
SSD_API ssd_status ssd_spec_cache_insert(ssd_spec_cache *cache, const int32_t *b,
                                 const int32_t *pos, const int32_t *tok,
                                 const int32_t *payload, int n,
                                 ssd_stream_t stream);

/* hit[i] = 1 and tok_out[i*depth..] = payload on a hit; 0 and -1 on a miss
 * (keys with a negative token or out-of-range b/pos always miss). */
SSD_API ssd_status ssd_spec_cache_lookup(const ssd_spec_cache *cache, const int32_t *b,
                                 const int32_t *pos, const int32_t *tok, int n,
                                 int32_t *hit, int32_t *tok_out,
                                 ssd_stream_t stream);

/* Insert the forked recovery tokens directly: key (b, j, fork_tok[b,j,r])
 * -> payload[((b*P + j)*f + r)*depth ..] for every fork_tok >= 0. */
SSD_API ssd_status ssd_spec_cache_insert_forks(ssd_spec_cache *cache,
                                       const int32_t *fork_tok, int B, int P,
                                       int f, const int32_t *payload,
                                       ssd_stream_t stream);

/* Look up each row's realised outcome: key (b, n_b, out_tok[b, n_b]) with
 * n_b = accept_len[b] (rows with n_b < 0 miss).  hit [B], tok_out [B,depth]. */
SSD_API ssd_status ssd_spec_cache_lookup_outcome(const ssd_spec_cache *cache,
                                         const int32_t *accept_len,
                                         const int32_t *out_tok, int B, int k,
                                         int32_t *hit, int32_t *tok_out,
                                         ssd_stream_t stream);

/* Read (and optionally clear) the cache's device error word; syncs stream. */
SSD_API ssd_status ssd_spec_cache_get_error(ssd_spec_cache *cache, ssd_stream_t stream,
                                    int32_t *out, int clear);

SSD_API int ssd_spec_cache_capacity(const ssd_spec_cache *cache);
SSD_API int ssd_spec_cache_depth(const ssd_spec_cache *cache);

/*
 * ---------------------------------------------------------------------------
 * The target pass around a verification: a paged cache of keys and values,
 * filled with a batch of drafted nodes (ssd_kv_append), attended by them
 * (ssd_tree_attention), and cut down to the accepted path afterwards
 * (ssd_kv_commit).  The nodes of a sequence are those of ssd_verify_tree:
 * node 0 is the last committed token, whose key and value are not cached
 * yet; a chain of k drafted tokens (ssd_verify) is the tree parent[j] = j-1
 * with N = k + 1; plain decoding is N = 1.
 *   - Slots 0 .. ctx_len[b]-1 of sequence b hold its committed context.  Node
 *     j is stored in slot ctx_len[b] + j; its position (for the rotation) is
 *     ctx_len[b] + depth(j).
 *   - Slot s of sequence b is entry s % page_size of page
 *     page_table[b*table_stride + s / page_size].
 * ---------------------------------------------------------------------------
 */

/* A paged cache of one layer: a HOST struct of device pointers and sizes,
 * read during the call only.  Entry d of head h of slot `off` of page `p`
 * is k[p*k_page + off*k_slot + h*k_head + d] (all strides in elements, so
 * token-major and head-major pages are both served).  k and v need 16-byte
 * alignment and strides that are positive multiples of 8 elements, below
 * 2^38 elements, and rows must not overlap. */
typedef struct {
    void *k, *v;
    int64_t k_page, k_slot, k_head;
    int64_t v_page, v_slot, v_head;
    ssd_dtype dtype;        /* SSD_BF16 or SSD_F16 */
    int num_pages, page_size;
    int Hkv, D;             /* key/value heads; head size 64 or 128 */
    const int32_t *page_table; /* device, [B, max_pages] */
    int64_t table_stride;
    int max_pages;          /* a sequence holds at most max_pages*page_size slots;
                               (max_pages+1)*page_size <= 2^31 - 257 */
} ssd_paged_kv;

/* The drafted nodes of a batch (HOST struct).  Every node's way to the root
 * has to satisfy parent[b, 0] == -1 and 0 <= parent[b, j] < j; a node whose
 * way does not (SSD_DEVERR_BAD_TREE) or with j >= n_nodes[b] is absent: it is
 * not stored, sees nothing and is seen by none.  A sequence with
 * ctx_len < 0, n_nodes outside [0, N] or ctx_len + n_nodes beyond its table
 * (SSD_DEVERR_BAD_LENGTH) has no nodes. */
typedef struct {
    int B, N;               /* 1 <= N <= SSD_MAX_TREE_NODES; B*N < 2^31 - 1024 */
    const int32_t *ctx_len; /* device, [B] */
    const int32_t *parent;  /* device, [B, N]; NULL: a chain */
    const int32_t *n_nodes; /* device, [B]; NULL: N everywhere */
} ssd_draft_nodes;

/* Bytes of the workspace of ssd_kv_append and ssd_kv_commit (its first word is
 * the device error word). */
#define SSD_ERRWORD_BYTES 256

/*
 * ssd_kv_append -- the queries, keys and values of the drafted nodes on their
 * way from the projections to the attention: per head x (q and k alike, each
 * with its own weights)
 *     y = x / sqrt(mean(x^2) + eps) * w        (q_norm / k_norm given)
 *     z = y with its first rot entries rotated by the node's position
 * computed in fp32 and rounded once; z_q goes to q_out, z_k and v to the
 * node's slot of the cache.
 *   q        : [B, N, Hq, D], element strides q_b, q_n, q_h (D contiguous);
 *              k, v: [B, N, Hkv, D] with one set of strides kv_b, kv_n, kv_h
 *              (views into a packed projection).  Type kv->dtype, 2-byte
 *              alignment; 16-byte aligned rows are read with vector loads.
 *   q_out    : [B, N, Hq, D] contiguous, 16-byte aligned; may be q itself when
 *              that is contiguous.  Absent nodes get zeros.
 *   cos_sin  : [max_pos, rot] fp32, 16-byte aligned: rot/2 cosines, then rot/2
 *              sines, of each position; NULL (rot = 0): no rotation.
 *              rot % 16 == 0, rot <= D.  A position >= max_pos makes its node
 *              absent (SSD_DEVERR_BAD_LENGTH).
 *   interleaved : 0 rotates pairs (i, i + rot/2), else pairs (2i, 2i+1).
 *   q_norm, k_norm : [D] weights of kv->dtype, both or neither.
 * A node whose page id is out of range is not stored (SSD_DEVERR_BAD_PAGE).
 */
SSD_API ssd_status ssd_kv_append(const ssd_paged_kv *kv, const ssd_draft_nodes *nodes, int Hq,
                         const void *q, int64_t q_b, int64_t q_n, int64_t q_h, const void *k,
                         const void *v, int64_t kv_b, int64_t kv_n, int64_t kv_h, void *q_out,
                         const float *cos_sin, int max_pos, int rot, int interleaved,
                         const void *q_norm, const void *k_norm, float eps, void *ws,
                         size_t ws_bytes, ssd_stream_t stream);

/*
 * ssd_tree_attention -- attention of the drafted nodes over the cache: query
 * head h of node i sees the context slots and the slots of node i and its
 * ancestors, of key/value head h / (Hq / Hkv);
 *     out = sum_s p_s v_s,  p = softmax over the seen slots of scale * q.k_s.
 *   q        : [B, N, Hq, D] with element strides q_b, q_n, q_h, type
 *              kv->dtype, 16-byte aligned rows; Hq a multiple of Hkv, at most
 *              64 heads a group.
 *   out      : [B, N, Hq, D] contiguous, kv->dtype, 16-byte aligned.
 *   lse      : [B, N, Hq] fp32 or NULL: log sum exp(scale * q.k) of the seen
 *              slots.
 *   scale    : finite, up to 2e38.
 *   ws       : ssd_tree_attention_workspace_bytes(B, N, Hq, Hkv, D) bytes.
 * Scores are held in 32 bits: where scale * q.k exceeds 2^24 their roundings decide
 * between slots, and beyond 2^26 a row may come out empty or NaN.
 * An absent node, or one whose seen slots all score -inf, gets out 0 and
 * lse -inf.  Slots that a node does not see never reach its output, whatever
 * they hold (NaN and infinities included).  A page id out of range reads as a
 * page of zeros (SSD_DEVERR_BAD_PAGE).  A tile that does not arrive within a
 * second ends the call (SSD_DEVERR_TIMEOUT); what out and lse hold is undefined
 * then.
 */
SSD_API size_t ssd_tree_attention_workspace_bytes(int B, int N, int Hq, int Hkv, int D);
SSD_API ssd_status ssd_tree_attention(const ssd_paged_kv *kv, const ssd_draft_nodes *nodes, int Hq,
                              const void *q, int64_t q_b, int64_t q_n, int64_t q_h, float scale,
                              void *out, float *lse, void *ws, size_t ws_bytes,
                              ssd_stream_t stream);

/*
 * ssd_kv_commit -- after a verification: the keys and values of the accepted
 * path move to the slots right behind the context, in `layers` caches that
 * share one page table (layer l starts at k + l*k_layer, v + l*v_layer).
 *   accept_len, out_node : ssd_verify_tree's outputs ([B], and [B, N] with row
 *              stride N): slot ctx + out_node[b, i] moves to slot ctx + 1 + i
 *              for i < accept_len[b].  out_node NULL: a chain, whose nodes
 *              already lie there.
 *   new_len  : [B] int32: ctx_len + 1 + accept_len.  Must not overlap ctx_len or
 *              accept_len.
 * A negative accept_len commits nothing (new_len = ctx_len), and so does a
 * path that is not increasing within 1 .. N-1 (SSD_DEVERR_BAD_TREE) or a
 * length out of range (SSD_DEVERR_BAD_LENGTH).  A move from or to a page id
 * out of range is left out (SSD_DEVERR_BAD_PAGE).
 */
SSD_API ssd_status ssd_kv_commit(const ssd_paged_kv *kv, int layers, int64_t k_layer, int64_t v_layer,
                         int B, int N, const int32_t *ctx_len, const int32_t *accept_len,
                         const int32_t *out_node, int32_t *new_len, void *ws, size_t ws_bytes,
                         ssd_stream_t stream);

/* Most new tokens of a sequence in one call of the operators for chunks. */
#define SSD_MAX_CHUNK (1 << 20)

/*
 * ssd_kv_append_at -- ssd_kv_append for chunks and for cut caches: a chain
 * (parent NULL) may have up to SSD_MAX_CHUNK tokens, and pos0 ([B] int32 or NULL:
 * ctx_len) gives the position of node 0, which after an eviction is not its slot:
 * node j has position pos0[b] + depth(j).  (A position < 0 or >= max_pos makes
 * its node absent where rot > 0.)
 */
SSD_API ssd_status ssd_kv_append_at(const ssd_paged_kv *kv, const ssd_draft_nodes *nodes, const int32_t *pos0,
                         int Hq, const void *q, int64_t q_b, int64_t q_n, int64_t q_h, const void *k,
                         const void *v, int64_t kv_b, int64_t kv_n, int64_t kv_h, void *q_out,
                         const float *cos_sin, int max_pos, int rot, int interleaved,
                         const void *q_norm, const void *k_norm, float eps, void *ws,
                         size_t ws_bytes, ssd_stream_t stream);

/*
 * ssd_chunk_attention -- attention of chunks of new tokens over the cache that
 * already holds them: prompts, parts of prompts, drafted chains, single tokens,
 * in one ragged batch.  tokens: chains (parent NULL) of up to SSD_MAX_CHUNK
 * tokens; sequence b has n_nodes[b] (or N) of them, in slots ctx_len[b] ...
 * The token in slot p sees the slots s <= p with s > p - window (window 0: all
 * of them) or s < sinks, of key/value head h / (Hq / Hkv);
 *     out = sum_s p_s v_s,  p = softmax over the seen slots of scale * q.k_s.
 * (window and sinks count slots, which after ssd_kv_evict are no positions.)
 *   q        : [B, N, Hq, D] with element strides q_b, q_n, q_h, positive
 *              multiples of 8 (those of a dimension of one entry too), type
 *              kv->dtype, 16-byte aligned; Hq a multiple of Hkv, at most 64
 *              heads a group.
 *   out      : [B, N, Hq, D] contiguous, kv->dtype, 16-byte aligned.
 *   lse      : [B, N, Hq] fp32 or NULL: log sum exp(scale * q.k) of the seen
 *              slots.
 *   ws       : ssd_chunk_attention_workspace_bytes(B, N, Hq, Hkv, D) bytes.
 * scale, empty rows, tokens that are not there, slots that are not seen, page
 * ids out of range, scores beyond 2^24 and tiles that do not arrive: as in
 * ssd_tree_attention.  Table entries of pages of which no token sees a slot
 * (between the first tokens and the window) may hold anything.
 */
SSD_API size_t ssd_chunk_attention_workspace_bytes(int B, int N, int Hq, int Hkv, int D);
SSD_API ssd_status ssd_chunk_attention(const ssd_paged_kv *kv, const ssd_draft_nodes *tokens, int Hq,
                              const void *q, int64_t q_b, int64_t q_n, int64_t q_h, int window,
                              int sinks, float scale, void *out, float *lse, void *ws, size_t ws_bytes,
                              ssd_stream_t stream);

/*
 * ssd_kv_weights -- what attention each slot received: for every slot s below
 * ctx_len[b] + n_nodes[b] of a sequence with new tokens
 *     w[b, h, s] = decay * w[b, h, s]
 *                + sum over the tokens i and query heads g of head h's group that
 *                  see s of exp(scale * q_ig.k_s - lse_ig),
 * with the slots that ssd_chunk_attention's token sees and the lse it wrote
 * (rows of lse -inf add nothing, whatever they score; those of lse NaN make the
 * slots that they see NaN, and no others).
 *   lse      : [B, N, Hq] fp32.
 *   weights  : fp32, row (b, h) at b*w_b + h*w_h (elements), w_len entries; decay 0
 *              writes without reading.  Slots behind a sequence's end stay as
 *              they are.
 *   kv, tokens, q, window, sinks, scale, page ids : as in ssd_chunk_attention;
 *              the values (v) are not read.
 *   ws       : ssd_kv_weights_workspace_bytes() bytes, of any sizes.
 * A sequence with ctx_len + n_nodes > w_len sets SSD_DEVERR_BAD_LENGTH and adds
 * nothing.  Sums are made in an order that the sizes and lengths alone decide.
 * After a call that was given up (SSD_DEVERR_TIMEOUT) each weight is as it was or
 * as the call was to make it.
 */
SSD_API size_t ssd_kv_weights_workspace_bytes(void);
SSD_API ssd_status ssd_kv_weights(const ssd_paged_kv *kv, const ssd_draft_nodes *tokens, int Hq, const void *q,
                         int64_t q_b, int64_t q_n, int64_t q_h, const float *lse, int window, int sinks,
                         float scale, float decay, float *weights, int64_t w_b, int64_t w_h, int w_len,
                         void *ws, size_t ws_bytes, ssd_stream_t stream);

/*
 * ssd_kv_evict -- every sequence longer than `budget` slots cut down to it, in
 * `layers` caches that share one page table (layer l starts at k + l*k_layer, v +
 * l*v_layer), every head of every layer by its own weights: the first `sinks`
 * slots stay, the last `recent`, and of those between the heaviest budget - sinks
 * - recent (of equal weights the lower slot; -0 equals 0, NaN is below all).
 * The kept slots' keys and values move to slots 0 .. budget-1 in slot order.
 *   weights  : fp32, row (l, b, h) at l*w_layer + b*w_b + h*w_h, w_len entries, of
 *              which the first ctx_len[b] count.
 *   budget   : >= 1 and >= sinks + recent; like w_len below 2^31 - 2^16.
 *   new_len  : [B] int32: min(ctx_len, budget).  Must not overlap ctx_len.
 *   kept     : [layers, B, Hkv, budget] int32: the slot that each slot's entry
 *              came from, -1 behind new_len.
 *   w_out    : the kept slots' weights, then zeros, w_len entries a row, with its
 *              own strides; weights itself (with its strides), memory apart from
 *              it, or NULL.
 *   ws       : SSD_ERRWORD_BYTES.
 * A sequence with ctx_len < 0, beyond its table or beyond w_len
 * (SSD_DEVERR_BAD_LENGTH) stays as it is: new_len = ctx_len, kept = -1, w_out not
 * written.  A move from or to a page id out of range is left out
 * (SSD_DEVERR_BAD_PAGE).  Sequences must not share pages.
 */
SSD_API ssd_status ssd_kv_evict(const ssd_paged_kv *kv, int layers, int64_t k_layer, int64_t v_layer, int B,
                         const int32_t *ctx_len, const float *weights, int64_t w_layer, int64_t w_b,
                         int64_t w_h, int w_len, int budget, int sinks, int recent, int32_t *new_len,
                         int32_t *kept, float *w_out, int64_t wo_layer, int64_t wo_b, int64_t wo_h,
                         void *ws, size_t ws_bytes, ssd_stream_t stream);

/*
 * ssd_logprobs -- what a server answers about emitted tokens, in one pass over
 * their rows: log p(tok), the entropy of p in nats, the token's rank and the
 * K best tokens with their log probabilities; p = softmax(z / T).
 *   logits   : rows of V logits, row_stride elements apart (>= V).
 *   rows     : [R] int32 or NULL: answer r is about row rows[r] of n_rows
 *              (a row id < 0: no answer, NaN and -1); NULL: row r, R <= n_rows.
 *   tok      : [R] int32; a token outside [0, V) gets logprob NaN, rank -1
 *              (SSD_DEVERR_BAD_TOKEN unless it is -1).
 *   T        : [R] fp32 or NULL (1).  T == 0: the one-hot at the lowest
 *              argmax (logprob 0 or -inf, entropy 0); T < 0 or NaN:
 *              SSD_DEVERR_BAD_TEMPERATURE, an answer of NaN and -1.
 *   logprob, entropy : [R] fp32; rank: [R] int32, 1 for the best token (larger
 *              logit first, then lower index).  entropy, rank may be NULL.
 *   K, top_tok, top_logprob : 0 <= K <= SSD_MAX_TOP; [R, K], best first.
 *   ws       : ssd_logprobs_workspace_bytes(R, V, K) bytes, for calls of any size
 *              that it is large enough for; entry points that keep more than the
 *              error word in their workspace need another.  R <= 2^26.
 * A row with a NaN or +inf logit, or only -inf, sets SSD_DEVERR_BAD_LOGITS and
 * gives NaN and -1.  A row id >= n_rows sets SSD_DEVERR_BAD_LENGTH.  A row of
 * which a part does not arrive within a second sets SSD_DEVERR_TIMEOUT and gives
 * NaN and -1.
 */
#define SSD_MAX_TOP 32
SSD_API size_t ssd_logprobs_workspace_bytes(int R, int V, int K);
SSD_API ssd_status ssd_logprobs(const void *logits, ssd_dtype dtype, int64_t row_stride, int n_rows,
                        int V, const int32_t *rows, int R, const int32_t *tok, const float *T,
                        int K, float *logprob, float *entropy, int32_t *rank, int32_t *top_tok,
                        float *top_logprob, void *ws, size_t ws_bytes, ssd_stream_t stream);

/*
 * Self-test hooks (HOST pointers, no GPU): the page lookup and the node walk
 * that the kernels above use.  ssd_selftest_kv_slot returns 1 and the page
 * and the entry within it, or 0 for a slot that the table does not hold.
 * ssd_selftest_node returns 1 and the node's ancestors-or-self as a bit mask
 * and its depth, or 0 for an absent node; parent NULL: a chain.
 */
SSD_API int ssd_selftest_kv_slot(const int32_t *table_row, int max_pages, int num_pages, int page_size,
                         int64_t slot, int32_t *page, int32_t *off);
SSD_API int ssd_selftest_node(const int32_t *parent, int n, int j, uint64_t *mask, int32_t *depth);

/*
 * Self-test hook of the bounded waits, process-wide for later calls of
 * ssd_tree_attention, ssd_chunk_attention, ssd_kv_weights and ssd_logprobs: a copy
 * into shared memory that takes longer than limit_us (1 .. 1000000; 0: the default
 * of a second) has failed;
 * withhold != 0: each waits for 16 bytes more than its copy brings, so that every
 * wait runs out.
 */
SSD_API ssd_status ssd_selftest_copy_wait(int limit_us, int withhold);

/*
 * Launch profiler (observability, not part of the method).  Between
 * ssd_profile_begin and ssd_profile_end every kernel the library launches
 * from this process is bracketed by a pair of CUDA events recorded on the
 * launch stream (at most max_launches launches; later ones go unrecorded but
 * are still counted).  ssd_profile_end waits for the recorded events and
 * fills out[0 .. *n_out) with one entry per kernel name: launches and total
 * device time.  Entries with launches == 0 are phases that span several
 * launches: "stats_pass" is the statistics pass of a batched verify, whose
 * target-row and draft-row kernels run concurrently on two internal streams,
 * from the fork to the join on the caller's stream; "stats_span" is the same
 * pass without the fork and join: from the earlier of its two launches'
 * begin events to the later of their end events.  Events are created at
 * begin and destroyed at end.
 */
typedef struct {
    char name[40];
    int launches;
    int timed;          /* launches with recorded events */
    double total_ms;    /* sum of event-measured durations of timed launches */
} ssd_profile_entry;

SSD_API ssd_status ssd_profile_begin(int max_launches);
SSD_API ssd_status ssd_profile_end(ssd_profile_entry *out, int cap, int *n_out);

/*
 * Vocabulary split override (tuning and tests; not part of the method).
 * Every logit row is split into chunks ("split-V") that CTAs stream and
 * whose partial statistics are merged in chunk order.  chunk_elems > 0 fixes
 * the chunk length (rounded up to a multiple of 8 and clamped to
 * [ceil(V / 256), 32 KB of logits]); chunks_per_cta > 0 fixes how many
 * consecutive chunks one statistics CTA streams (at most the chunk count).
 * 0 restores the built-in policy.  The setting is process-wide and read when
 * a call (or a workspace-size query) lays out its workspace, so query the
 * workspace size after setting it.  Integer results (accept lengths, tokens,
 * forks, cache lookups) do not depend on it; float outputs (p_at_x, q_at_x,
 * softmax sums) can differ in the last bits, because the chunk sums round
 * differently.  Returns SSD_ERR_INVALID_ARG for negative values.
 */
SSD_API ssd_status ssd_set_split(int chunk_elems, int chunks_per_cta);

/*
 * Small-batch schedule override (tuning and tests; not part of the method).
 * After the statistics pass, a verify call of at most max_b batch rows
 * (default 16) runs its finalisation, recovery / bonus draw and, in
 * ssd_verify_fork_cache, the cache insert and outcome lookup as one
 * cluster kernel: one thread-block cluster of up to 8 CTAs per batch row,
 * the row merges and the draw's pass over the vocabulary split over the
 * cluster, partial sums exchanged through distributed shared memory.
 * Larger batches launch the finalisation, draw and cache kernels
 * separately.  max_b = 0 disables the cluster kernel; negative restores the
 * default.  Process-wide, read at each call.  Accept lengths, p_at_x,
 * q_at_x and forks are the same bits on both schedules; a drawn token is
 * the same except where u falls within ~1e-12 relative of a boundary of the
 * inverse CDF (the two schedules round their fixed-point partial masses
 * over different ranges).  Returns SSD_OK.
 */
SSD_API ssd_status ssd_set_chain_batch(int max_b);

/*
 * Whole-call schedule override for the smallest batches (tuning and tests;
 * not part of the method).  A verify call of at most max_b batch rows
 * (default 4, at most 8) runs as one cooperative kernel: the statistics
 * pass, row merges and forks, acceptance, the draw's two exact passes over
 * rows n and the select, separated by grid-wide barriers among CTAs that
 * are all resident; in ssd_verify_fork_cache also the cache clear, insert
 * and outcome lookup.  max_b = 0 disables it, negative restores the default;
 * max_grid > 0 caps the CTAs of that kernel (0: as many as the GPU holds at
 * once).  If the launch is refused the call takes the launch-by-launch
 * schedule.  Every barrier wait is bounded: one that runs out sets
 * SSD_DEVERR_TIMEOUT and the kernel returns without finishing the call.
 * Accept lengths, p_at_x, q_at_x and forks are the same bits on every
 * schedule; a drawn token is the same except where u falls within ~1e-12
 * relative of a boundary of the inverse CDF.  Returns SSD_ERR_INVALID_ARG
 * for max_grid < 0, else SSD_OK.  Process-wide, read at each call.
 */
SSD_API ssd_status ssd_set_step_schedule(int max_b, int max_grid);

/*
 * Self-test hook for the library's extended-precision exponential (used by
 * the recovery draw): out[i] = 2^(x_hi[i] + x_lo[i]) in double, for
 * x_hi <= 0.  Device pointers, n >= 0.  Not part of the verify path.
 */
SSD_API ssd_status ssd_selftest_exp2(const float *x_hi, const float *x_lo, double *out,
                             int n, ssd_stream_t stream);

#ifdef __cplusplus
}
#endif
#endif /* SSD_GB300_H */

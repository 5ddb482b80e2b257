/*
 * spec_verify.h -- C ABI of libspecverify: batched draft-token verification
 * for speculative decoding on one NVIDIA GB300 (sm_103a).
 *
 * What is computed (sources are web pages, cited by title and section):
 *   [REVIEW] "EAGLE-3 speculative decoding review" (6unoyunr.github.io)
 *   [MATH]   "EAGLE math" (aicassindra.com, tm_eagle_math)
 *   [WIKI]   "Speculative decoding" (addictedtoai.net wiki)
 *
 * Conventions shared by every entry point
 *   - All array arguments are DEVICE pointers (cudaMalloc / torch CUDA
 *     memory), row-major and contiguous.  The caller owns all memory; the
 *     library allocates nothing.  State kept across calls: the launch counter
 *     read by spec_verify_launch_count(); per device context, the kernels'
 *     shared-memory opt-ins and launch shapes; and the fixed scratch array of
 *     spec_verify_greedy_noalloc (resident on every device that loads the
 *     library) with its device address.  Each per-context entry records the
 *     context's unique id and is redone when it changes (after
 *     cudaDeviceReset, for example).
 *   - `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *     stream).  Every call only enqueues work on that stream and returns; it
 *     never synchronises.  Outputs are valid once the stream reaches them.
 *   - Logits are fp32 (SPEC_DTYPE_F32) or bf16 (SPEC_DTYPE_BF16, raw 16-bit
 *     patterns).  Logit pointers must be aligned to the element size; rows
 *     whose byte length is a multiple of 16 starting at a 16-byte aligned base
 *     take the vectorised path, others a scalar path with identical results.
 *   - Logits must be finite with |logit / T| < 2^23; other values give
 *     unspecified (but memory-safe) outputs.  spec_verify_tree_sample also
 *     takes -inf, a token of probability 0.
 *   - `workspace`: device scratch of at least spec_verify_workspace_bytes()
 *     bytes, 256-byte aligned.  Its contents on entry do not matter: every
 *     record a kernel reads is written earlier in the same call, so one
 *     workspace serves calls of any shape.  Its first 4 bytes hold the sticky
 *     flag word (see spec_verify_read_flags): zero the workspace once, or
 *     read the flags with clear != 0, before relying on them.  Two calls that
 *     share a workspace must not run concurrently (issue them on one stream,
 *     or order them with events).
 *   - Errors found on the host (NULL pointer, bad size, bad temperature,
 *     misalignment, workspace too small) return before anything is enqueued.
 *     A failed kernel launch returns SPEC_ERR_CUDA.  Bad DEVICE data (a token
 *     id outside [0, V), a malformed tree) is never trapped: the kernels clamp
 *     every access, treat the item as not matching, and set a bit of the
 *     workspace's flag word (spec_verify_read_flags).
 *   - B = 0 is a no-op that returns SPEC_OK.
 *   - Every call's kernels are programmatic dependent launches:
 *     the first kernel of a call waits for the kernel before it in the
 *     stream to finish (and its writes to be visible) before it writes
 *     memory or reads anything but its logits, and the last kernel of a call
 *     lets the next kernel in the stream be scheduled early.  The streaming
 *     kernels of spec_verify_greedy (and its _noalloc form),
 *     spec_verify_tree_greedy and (for short per-CTA ranges)
 *     spec_verify_sample start reading their logits (and
 *     sampling its draft tokens) before that wait, while the call before
 *     them on the stream is finishing.  So the logits and draft tokens of
 *     these three must not be written by the library call issued just before
 *     them on the same stream (a kernel of the caller's own, issued between
 *     two calls, has always finished before the next call's kernels start).
 *     All other calls read nothing before that wait, and may take what the
 *     call before them writes: spec_tree_grow, spec_tree_attention_mask,
 *     spec_tree_qkv_rope, spec_tree_attention, spec_verify_tree_sample and
 *     spec_kv_commit_path can be issued one after the other, and so can the
 *     calls on the 4-bit cache, on pages and on beams.
 */
#ifndef SPEC_VERIFY_H_
#define SPEC_VERIFY_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define SPEC_VERIFY_ABI_VERSION 1

#if defined(__GNUC__)
#define SPEC_API __attribute__((visibility("default")))
#else
#define SPEC_API
#endif

typedef enum {
  SPEC_OK = 0,
  SPEC_ERR_INVALID_ARG = 1, /* NULL pointer, size out of range, T <= 0 or NaN */
  SPEC_ERR_ALIGNMENT = 2,   /* pointer not aligned as documented */
  SPEC_ERR_WORKSPACE = 3,   /* workspace NULL or smaller than required */
  SPEC_ERR_CUDA = 4,        /* a CUDA runtime call or kernel launch failed */
  SPEC_ERR_TOO_LARGE = 5    /* the call needs more scratch than the fixed
                               array of spec_verify_greedy_noalloc holds */
} spec_status_t;

typedef enum { SPEC_DTYPE_F32 = 0, SPEC_DTYPE_BF16 = 1 } spec_dtype_t;

typedef enum {
  SPEC_MODE_SAMPLE = 0,
  SPEC_MODE_GREEDY = 1,
  SPEC_MODE_TREE_GREEDY = 2,
  SPEC_MODE_TREE_MASK = 3, /* spec_tree_attention_mask: the flag header only */
  SPEC_MODE_KV_COMMIT = 4, /* spec_kv_commit_path: the flag header only */
  SPEC_MODE_LM_HEAD_GREEDY = 5, /* spec_lm_head_verify_greedy (k_or_N = k) */
  SPEC_MODE_TREE_GROW = 6,      /* spec_tree_grow (k_or_N = K children per node) */
  SPEC_MODE_LM_HEAD_SAMPLE = 7, /* spec_lm_head_verify_sample (k_or_N = k, d <= SPEC_LM_MAX_D) */
  SPEC_MODE_TREE_SAMPLE = 8,    /* spec_verify_tree_sample: the flag header only */
  SPEC_MODE_TREE_QKV = 10,      /* spec_tree_qkv_rope: the flag header only */
  SPEC_MODE_KV4 = 11            /* spec_kv4_commit_path, spec_kv4_read: the flag header only */
} spec_mode_t;

/* Bits of the workspace flag word (sticky until read with clear != 0). */
#define SPEC_FLAG_TOKEN_RANGE 1u       /* a draft/node token was outside [0, V) */
#define SPEC_FLAG_BAD_PARENT 2u        /* parents[v] outside [0, v) for some v >= 1 */
#define SPEC_FLAG_DEPTH 4u             /* a node deeper than max_depth */
#define SPEC_FLAG_RESIDUAL_FALLBACK 8u /* residual mass was 0 after a rejection;
                                          that position was sampled from p */
#define SPEC_FLAG_TIMEOUT 16u          /* a kernel gave up waiting for its own
                                          bulk copies or matrix products, or one
                                          of its roles for another (outputs of
                                          that call are unspecified); never
                                          expected */
#define SPEC_FLAG_BAD_PATH 32u         /* spec_kv_commit_path: a path that does
                                          not start at node 0, names a node
                                          outside [1, N), is longer than
                                          max_depth, or a tree that does not fit
                                          the cache; that sequence is untouched.
                                          spec_tree_qkv_rope, spec_tree_attention:
                                          a tree that does not fit the cache;
                                          the calls on pages: a length outside
                                          the table (see each call) */
#define SPEC_FLAG_EMPTY_ROW 64u        /* spec_verify_tree_sample: a row on the walk
                                          without a finite logit; no token drawn */
#define SPEC_FLAG_BAD_PAGE 128u        /* an entry of a page table that is needed names no page */
#define SPEC_FLAG_NO_PAGE 256u         /* spec_kv_pages_fork: no free page left */

/* Limits checked on the host. */
#define SPEC_MAX_V (1 << 26)
#define SPEC_MAX_K 256
#define SPEC_MAX_TREE_NODES 65536
#define SPEC_MAX_TREE_DEPTH 1024

/*
 * Bytes of workspace needed by one call.  mode: spec_mode_t; k_or_N: k draft
 * tokens (chain modes) or N tree nodes (tree mode).  Returns 0 for arguments
 * outside the limits above or whose scratch index space exceeds 2^31 records.
 */
SPEC_API size_t spec_verify_workspace_bytes(int mode, int B, int k_or_N, int V, int dtype);

/*
 * Rejection-sampling verification of B chains of k draft tokens.
 *
 * Computes, per sequence b ([REVIEW] "Speculative Decoding" step 3 "Accept or
 * Reject"; "Does Using a Small Model's Answer Reduce Quality?", eqs. A(x) and
 * p_residual; [MATH] "Vanilla speculative decoding"; [WIKI] "The mechanism"):
 *   p_i = softmax(target[b,i,:] / T),  q_i = softmax(draft[b,i,:] / T)
 *   accept draft i iff u_accept[b,i] * q_i(x_i) < p_i(x_i)  (strict; left to
 *   right); n = index of the first rejection, or k if none;
 *   if n < k: token ~ norm(max(0, p_n - q_n)) by inverse CDF with u_sample[b]
 *   else:     bonus token ~ p_k by inverse CDF with u_sample[b].
 * Inverse CDF: the smallest vocabulary index j with u * R < C_j, C_j the
 * inclusive prefix sum of the weights and R their total.
 *
 *   target_logits [B, k+1, V]  row i scores draft position i; row k = bonus row
 *   draft_logits  [B, k, V]    row i = the distribution draft i was drawn from
 *   draft_tokens  int32 [B, k]
 *   u_accept      float [B, k] in [0, 1);   u_sample float [B] in [0, 1)
 *   temperature   > 0, finite; the same T scales target and draft rows
 * Outputs (device, written in full):
 *   accepted_len  int32 [B]       n in [0, k]
 *   out_tokens    int32 [B, k+1]  x_0..x_{n-1}, the resampled/bonus token, then -1
 *   p_out, q_out  float [B, k]    p_i(x_i), q_i(x_i) for EVERY i (also i > n)
 *   resid_mass    float [B]       R = sum_j max(0, p_n - q_n) when n < k, else 0
 * With k = 0, draft_logits, draft_tokens, u_accept, p_out and q_out may be
 * NULL and the call samples one token from softmax(target[b,0,:] / T).
 * Launches two kernels: the softmax statistics, then one thread-block cluster
 * per sequence for row merge, accept test, residual/bonus prefix sums and the
 * inverse-CDF walk (three kernels when a row spans more than 16 32-KB chunks:
 * V > 262144 bf16 or 131072 fp32).
 */
SPEC_API spec_status_t spec_verify_sample(const void* target_logits, const void* draft_logits,
                                 int dtype, const int32_t* draft_tokens,
                                 const float* u_accept, const float* u_sample,
                                 float temperature, int B, int k, int V,
                                 int32_t* accepted_len, int32_t* out_tokens,
                                 float* p_out, float* q_out, float* resid_mass,
                                 void* workspace, size_t workspace_bytes, void* stream);

/*
 * Greedy verification ([REVIEW] "Does Using a Small Model's Answer Reduce
 * Quality?", greedy bullets): g_i = argmax_j target[b,i,j] on raw logits,
 * lowest index among ties; n = first i < k with draft_tokens[b,i] != g_i, or
 * k; emits x_0..x_{n-1}, g_n.  Temperature plays no part.
 *   target_logits [B, k+1, V]; draft_tokens int32 [B, k] (NULL allowed if k = 0)
 *   accepted_len  int32 [B];   out_tokens int32 [B, k+1] (unused slots -1)
 * Launches two kernels (argmax partials; row merge + accept).
 */
SPEC_API spec_status_t spec_verify_greedy(const void* target_logits, int dtype,
                                 const int32_t* draft_tokens, int B, int k, int V,
                                 int32_t* accepted_len, int32_t* out_tokens,
                                 void* workspace, size_t workspace_bytes, void* stream);

/*
 * Draft-tree greedy verification (EAGLE-2 style trees; [REVIEW] "EAGLE-2",
 * "The Complete EAGLE-3 Inference Process" steps 3-4; [MATH] "EAGLE-2:
 * dynamic draft trees").  Node 0 is the root (the last committed token); row v
 * of target_logits is the target's next-token logits after the path root..v.
 * Node v >= 1 is accepted iff every node w on the path root..v has
 * node_tokens[w] == argmax(target row of parent(w)).  The deepest accepted
 * node v* wins (lowest node index among equally deep ones); the bonus token
 * is argmax(target row v*).
 *   target_logits [B, N, V]
 *   node_tokens   int32 [B, N]   (node 0's entry is ignored)
 *   parents       int32 [B, N]   parents[b,0] ignored; 0 <= parents[b,v] < v
 *   max_depth     depth limit of the trees, 0..SPEC_MAX_TREE_DEPTH
 * Outputs:
 *   accepted_len  int32 [B]                depth of v*
 *   path_nodes    int32 [B, max_depth+1]   0, ..., v*, then -1
 *   out_tokens    int32 [B, max_depth+1]   tokens of path nodes 1..depth, the
 *                                          bonus token, then -1
 * Launches two kernels (argmax partials; row merge + tree walk).
 */
SPEC_API spec_status_t spec_verify_tree_greedy(const void* target_logits, int dtype,
                                      const int32_t* node_tokens, const int32_t* parents,
                                      int B, int N, int V, int max_depth,
                                      int32_t* accepted_len, int32_t* path_nodes,
                                      int32_t* out_tokens, void* workspace,
                                      size_t workspace_bytes, void* stream);

/*
 * Sampling verification of B draft trees ("EAGLE-3 speculative decoding
 * review", "Does Using a Small Model's Answer Reduce Quality?", with drafts
 * that are points: the children that spec_tree_grow picks are the draft's most
 * probable tokens, not draws from it, so a child x is taken with probability
 * p(x) and a miss leaves p without the children).  The walk starts at the root.
 * At a node of depth d with target row z it draws
 *   x = the smallest j with u_sample[b, d] * R < C_j,
 * C_j the inclusive prefix sum and R the total of the weights exp(z_j / T),
 * moves to the lowest-numbered child whose token is x, or ends there.  The
 * emitted tokens are those that drawing one at a time from softmax(z / T)
 * with the same uniforms gives, whatever the tree; the tree decides only how
 * many of them one call emits.
 *   target_logits [B, N, V]   row v: the target's logits after the path root..v;
 *                             -inf is a token of probability 0
 *   node_tokens   int32 [B, N] (node 0's entry is ignored)
 *   parents       int32 [B, N]  as spec_verify_tree_greedy
 *   u_sample      float [B, max_depth + 1] in [0, 1)
 *   temperature   > 0, finite
 *   max_depth     0..SPEC_MAX_TREE_DEPTH; deeper nodes are not taken
 * Outputs (device, written in full):
 *   accepted_len  int32 [B]              depth of the last node of the walk
 *   path_nodes    int32 [B, max_depth+1] 0, ..., that node, then -1
 *   out_tokens    int32 [B, max_depth+1] the tokens drawn at those nodes (the
 *                                        last one is the new token), then -1
 *   out_probs     float [B, max_depth+1] their probabilities, then 0
 * so that spec_kv_commit_path takes accepted_len and path_nodes as they are.
 * Draws are decided by float32 sums with a bounded error and, next to a border
 * C_j, by integer sums of weights rounded to 2^-50 of the largest, each off by
 * 2^-40 of itself and another |z_j / T| 2^-46 of itself: a border of such sums
 * is off by less than V 2^-51 + 2^-28 of R (2^-24 at the largest V; a token
 * below 2^-51 of the largest is never drawn) where all |z_j / T| < 2^16;
 * out_probs is within 2e-5 of its value.  A row without a finite logit draws
 * nothing (token -1, probability 0, SPEC_FLAG_EMPTY_ROW) and ends the walk.
 * Malformed nodes are never taken
 * (SPEC_FLAG_BAD_PARENT, SPEC_FLAG_TOKEN_RANGE); SPEC_FLAG_DEPTH is set when
 * the walk would have gone below max_depth.  Only the rows on the walk are
 * read.  One launch of a cluster of up to 16 CTAs per sequence.  Workspace:
 * spec_verify_workspace_bytes(SPEC_MODE_TREE_SAMPLE, ...) bytes (the flag
 * header).
 */
SPEC_API spec_status_t spec_verify_tree_sample(const void* target_logits, int dtype,
                                               const int32_t* node_tokens, const int32_t* parents,
                                               const float* u_sample, float temperature, int B,
                                               int N, int V, int max_depth, int32_t* accepted_len,
                                               int32_t* path_nodes, int32_t* out_tokens,
                                               float* out_probs, void* workspace,
                                               size_t workspace_bytes, void* stream);

/*
 * Tree attention mask of B draft trees ("EAGLE-3 speculative decoding
 * review", "EAGLE-2: Does Every Context Need the Same Draft Tree?" and "Must
 * the Feature Be Predicted Exactly?": each node sees the shared prefix and
 * only its own ancestors; "The Complete EAGLE-3 Inference Process" step 3).
 * The prefix columns are visible to every node and are not written; this
 * call writes the tree block.
 *   parents  int32 [B, N]  parents[b,0] ignored (node 0 is the root, the
 *                          last committed token); 0 <= parents[b,v] < v
 * Outputs:
 *   mask     uint32 [B, N, W], W = (N + 31) / 32: bit (u % 32) of word u / 32
 *            of row (b, v) is set iff u == v or u is an ancestor of v; the
 *            bits past N in the last word are 0
 *   depth    int32 [B, N] or NULL: edges from v to the root
 * A node whose ancestor chain meets a parent outside [0, child) keeps the
 * nodes walked so far, gets depth -1 and raises SPEC_FLAG_BAD_PARENT.
 * Pointers: device memory, 4-byte aligned; workspace of at least
 * spec_verify_workspace_bytes(SPEC_MODE_TREE_MASK, ...) bytes (the flag
 * header), 256-byte aligned.  One kernel launch; N <= SPEC_MAX_TREE_NODES.
 */
SPEC_API spec_status_t spec_tree_attention_mask(const int32_t* parents, int B, int N,
                                                uint32_t* mask, int32_t* depth, void* workspace,
                                                size_t workspace_bytes, void* stream);

/*
 * Query, key and value heads of the tree's nodes, ready for spec_tree_attention
 * ("EAGLE-3 speculative decoding review", "The Complete EAGLE-3 Inference
 * Process" step 3: the target scores all nodes in one pass).  Node v of
 * sequence b stands at position pos_offset + base_len[b] - 1 + depth[b, v] (the
 * root is the last committed token).  Query and key heads are normalised,
 *   y = x / sqrt(mean(x^2) + eps) * w   (a null w: no norm),
 * and their first rot_dim elements rotated in pairs by position * inv_freq[i],
 *   (a, b) -> (a cos - b sin, b cos + a sin),
 * in float32, rounded once (angles are reduced to one turn in 64-bit integers:
 * an angle of A turns is off by less than A 2^-47 + 2^-24 of a turn, which at
 * position 2^31 is 3e-6 for a frequency of 1).  Queries go to
 * q_out; keys and values go to cache position base_len[b] - 1 + v, where
 * spec_kv_commit_path expects them.
 *   qkv           bf16 [B, N, Hq + 2 Hkv, D]: query, key, value heads
 *   q_norm,k_norm bf16 [D] or NULL
 *   inv_freq      float [rot_dim / 2] (NULL when rot_dim = 0), finite
 *   rot_dim       even, 0..D;  interleaved: 0 pairs (i, i + rot_dim / 2),
 *                 else (2i, 2i + 1)
 *   pos_offset    0..2^31 - 1 (the length of a prefix shared by the batch)
 *   base_len      int32 [B]; depth int32 [B, N] or NULL (a chain: node v at
 *                 depth v); a negative depth counts as 0 and raises
 *                 SPEC_FLAG_BAD_PARENT
 *   q_out         bf16 [B, N, Hq, D]; outputs must not overlap inputs
 *   k_cache, v_cache bf16: sequence b's position t starts seq_stride * b +
 *                 t * Hkv * D * 2 bytes in; L positions per sequence
 * D is 64 or 128; qkv, q_out, the norms and the caches 16-byte aligned,
 * seq_stride a multiple of 16.  A sequence whose tree does not fit the cache
 * (base_len < 1 or base_len + N - 1 > L) writes no key or value, gets queries
 * of 0 and raises SPEC_FLAG_BAD_PATH.  One launch.  Workspace:
 * spec_verify_workspace_bytes(SPEC_MODE_TREE_QKV, ...) bytes (the flag header).
 */
SPEC_API spec_status_t spec_tree_qkv_rope(const void* qkv, const void* q_norm, const void* k_norm,
                                          float eps, const float* inv_freq, int rot_dim,
                                          int interleaved, long long pos_offset,
                                          const int32_t* base_len, const int32_t* depth, int B,
                                          int N, int Hq, int Hkv, int D, int L,
                                          long long seq_stride, void* q_out, void* k_cache,
                                          void* v_cache, void* workspace, size_t workspace_bytes,
                                          void* stream);

/*
 * Attention of the tree's nodes over the KV cache ("EAGLE-3 speculative
 * decoding review", "EAGLE-2: Does Every Context Need the Same Draft Tree?":
 * a node sees the committed prefix and its own ancestors).  Query head
 * h G + g (G = Hq / Hkv) reads key-value head h:
 *   out = sum_j softmax_j(scale q . k_j) v_j
 * over j in
 *   - the shared prefix: prefix_k/v entries [0, P), one copy for the batch;
 *   - the sequence's own positions [0, base_len[b] - 1);
 *   - the tree's entries base_len[b] - 1 + u for the set bits u < N of the
 *     node's mask row (spec_tree_attention_mask; NULL: u <= v, a chain).
 * Entries that a node does not see are never used, whatever they hold.  A
 * node that sees nothing gets out = 0 and lse = -inf.
 *   q          bf16 [B, N, Hq, D]
 *   k_cache, v_cache bf16, layout as in spec_tree_qkv_rope
 *   prefix_k, prefix_v bf16 [P, Hkv, D] (NULL when P = 0)
 *   mask       uint32 [B, N, ceil(N/32)] or NULL
 *   base_len   int32 [B]; scale > 0, below 2^127, scores |scale q . k| below 2^24
 *   out        bf16 [B, N, Hq, D]
 *   lse        float [B, N, Hq] or NULL: ln sum_j exp(scale q . k_j)
 * N = 1 without a mask is plain decoding.  D is 64 or 128, Hq a multiple of
 * Hkv, G at most 128, N at most SPEC_ATTN_MAX_NODES, L and P at most
 * 2^31 - 257; q, out, the caches and prefixes 16-byte aligned, seq_stride a
 * multiple of 16.  A sequence whose
 * tree does not fit the cache (base_len < 1 or base_len + N - 1 > L) gets out
 * = 0, lse = -inf and raises SPEC_FLAG_BAD_PATH.  Values that are not finite:
 * an element of a tree entry (the root's or a node's) makes all of out NaN for
 * the query heads that read it, of the nodes that see the entry alone; an
 * element of the prefix or of the committed positions, which all nodes see,
 * makes its own column of out infinite or NaN, as in the sum.  lse does not
 * depend on values.  Outputs must not overlap inputs.
 * Two launches: the attention of equal runs of 128-entry tiles, one run per
 * SM, on the tensor cores (weights rounded to bf16, sums in float32), which
 * takes most of each SM's shared and tensor memory until it ends, and the join
 * of items that were cut; the cut, and so the last bits, depend on base_len and
 * the number of SMs alone.  Workspace: at least
 * spec_tree_attention_workspace_bytes() bytes (float32 partials: of cut items,
 * two per SM at most, or of every item behind a shared prefix).
 */
#define SPEC_ATTN_MAX_NODES 4096
SPEC_API size_t spec_tree_attention_workspace_bytes(int B, int N, int Hq, int Hkv, int D, int P);
SPEC_API spec_status_t spec_tree_attention(const void* q, const void* k_cache, const void* v_cache,
                                           long long seq_stride, int L, const void* prefix_k,
                                           const void* prefix_v, int P, const uint32_t* mask,
                                           const int32_t* base_len, int B, int N, int Hq, int Hkv,
                                           int D, float scale, void* out, float* lse,
                                           void* workspace, size_t workspace_bytes, void* stream);

/*
 * KV commit of the accepted path ("EAGLE-3 speculative decoding review",
 * "The Complete EAGLE-3 Inference Process" step 5: keep only the accepted
 * path's cache entries, discard the rejected branches, resume drafting from
 * the committed prefix).  Tree node v >= 1 of sequence b holds its entries at
 * cache position base_len[b] + v - 1 (the tree follows the committed prefix,
 * whose last token is the root).  For the path 0, v_1, ..., v_d written by
 * spec_verify_tree_greedy (d = accepted_len[b]), node v_i's entry moves to
 * position base_len[b] + i - 1 in every plane, in place; every other
 * position keeps its contents; new_len[b] = base_len[b] + d (the bonus token
 * has no cache entry yet).
 *   cache        device bytes; entry (plane p, sequence b, position t) starts
 *                at p * plane_stride + b * seq_stride + t * entry_bytes (a
 *                plane is one layer's K or V); 16-byte aligned, entry_bytes
 *                and both strides multiples of 16; entries must not overlap
 *   L            positions per sequence; N tree nodes; base_len[b] >= 1 and
 *                base_len[b] + N - 1 <= L
 *   base_len, accepted_len  int32 [B]; path_nodes int32 [B, max_depth + 1]
 *   new_len      int32 [B] out
 * A malformed sequence (see SPEC_FLAG_BAD_PATH) is left untouched with
 * new_len = base_len.  Workspace: spec_verify_workspace_bytes(
 * SPEC_MODE_KV_COMMIT, ...) bytes (the flag header).  One kernel launch (one
 * CTA per sequence and plane; the moved entries are staged in shared memory
 * before any is stored); planes <= 65535.
 */
SPEC_API spec_status_t spec_kv_commit_path(void* cache, int B, int planes, long long plane_stride,
                                           long long seq_stride, int entry_bytes, int L, int N,
                                           const int32_t* base_len, const int32_t* accepted_len,
                                           const int32_t* path_nodes, int max_depth,
                                           int32_t* new_len, void* workspace,
                                           size_t workspace_bytes, void* stream);

/*
 * The target's LM head fused with greedy verification ("EAGLE math", "Why
 * feature drafting lands a higher acceptance rate": the target's logits are
 * its LM head applied to the hidden state, z = W_LM h; "EAGLE-3 speculative
 * decoding review", "Does Using a Small Model's Answer Reduce Quality?"
 * greedy bullets).  Computes every target row's argmax of z = W_LM h on the
 * tensor cores without writing the logits, then the same acceptance as
 * spec_verify_greedy.
 *   hidden       bf16 [B*(k+1), d]  row b*(k+1)+i: the target's hidden state
 *                                   at draft position i of sequence b
 *   w_lm         bf16 [V, d]        the LM head, row j = vocabulary entry j
 *   draft_tokens int32 [B, k]
 *   d            multiple of 8; hidden and w_lm 16-byte aligned
 * Outputs as spec_verify_greedy.  The argmax is of the float32-accumulated
 * products (lowest index among equal values); rows whose top two logits lie
 * closer than the accumulation error may pick either.  Two kernel launches
 * (tcgen05 GEMM with an argmax epilogue; record merge + chain resolve).  The
 * GEMM runs on clusters of two CTAs, one per SM, that share each 256-entry
 * vocabulary tile through two-CTA MMAs; it occupies every SM it can hold a
 * pair on (most of each SM's shared and tensor memory) until it ends.
 * Workspace: spec_verify_workspace_bytes(SPEC_MODE_LM_HEAD_GREEDY, B, k, V,
 * SPEC_DTYPE_BF16).
 */
SPEC_API spec_status_t spec_lm_head_verify_greedy(const void* hidden, const void* w_lm,
                                                  const int32_t* draft_tokens, int B, int k,
                                                  int d, int V, int32_t* accepted_len,
                                                  int32_t* out_tokens, void* workspace,
                                                  size_t workspace_bytes, void* stream);

/*
 * The target's LM head fused with sampling verification ("EAGLE math",
 * "EAGLE's move": p = softmax(LM_head(f)), the drafted features going through
 * the target's own LM head; "EAGLE-3 speculative decoding review", "Does
 * Using a Small Model's Answer Reduce Quality?" eqs. A(x), p_residual).
 * The target rows' logits W_LM h_t and the draft rows' logits W_LM h_d are
 * reduced on the tensor cores to their softmax statistics and draft-token
 * logits without being written; the accept test follows, and only the rows
 * a sequence draws from (the target and draft rows of its first rejection,
 * or its bonus row) are recomputed as fp32 logits in the workspace for the
 * residual or bonus draw.  Same decisions and outputs as spec_verify_sample
 * on the float32-accumulated logits.
 *   hidden_target bf16 [B*(k+1), d]  row b*(k+1)+i: the target's hidden state
 *                                    at position i of sequence b
 *   hidden_draft  bf16 [B*k, d]      row b*k+i: the drafted feature of
 *                                    position i (NULL when k = 0)
 *   w_lm          bf16 [V, d]        the LM head, row j = vocabulary entry j
 *   draft_tokens, u_accept, u_sample, temperature, outputs: as
 *                 spec_verify_sample
 *   d             multiple of 8, at most SPEC_LM_MAX_D; the matrices 16-byte
 *                 aligned
 * Four kernel launches: the statistics GEMM (tcgen05, softmax epilogue), the
 * accept test with the gather of the drawn rows' hidden states, the GEMM
 * that writes those rows' logits, and the draw (as spec_verify_sample's).
 * Workspace: spec_verify_workspace_bytes(SPEC_MODE_LM_HEAD_SAMPLE, B, k, V,
 * SPEC_DTYPE_BF16).
 */
#define SPEC_LM_MAX_D 8192
SPEC_API spec_status_t spec_lm_head_verify_sample(
    const void* hidden_target, const void* hidden_draft, const void* w_lm,
    const int32_t* draft_tokens, const float* u_accept, const float* u_sample, float temperature,
    int B, int k, int d, int V, int32_t* accepted_len, int32_t* out_tokens, float* p_out,
    float* q_out, float* resid_mass, void* workspace, size_t workspace_bytes, void* stream);

/*
 * EAGLE-2 dynamic draft-tree growth ("EAGLE math", "EAGLE-2: dynamic draft
 * trees": expand the nodes with the highest cumulative draft probability,
 * prune low-probability paths, re-rank under an unchanged node budget;
 * "EAGLE-3 speculative decoding review", "EAGLE-2: Does Every Context Need
 * the Same Draft Tree?").  Layer l expands the frontier (slot j holds a node;
 * layer 0: the root in slot 0) with the draft row draft_logits[b, l, j]:
 * q = softmax(z / T); the node's children are its K most probable tokens
 * (ties: lower token), valued parent + ln q(token) (root 0); the next
 * frontier is the layer's K best children (ties: creation order).  After D
 * layers the tree is the root plus the M best nodes (ties: creation order),
 * listed in creation order (parents before children) with parents
 * renumbered, ready for spec_verify_tree_greedy and spec_tree_attention_mask.
 *   draft_logits  [B, D, K, V] dtype (slot j of layer 0 is read for j = 0 only)
 *   K             1..16 children per node and frontier size; D 1..16 layers
 *   M             node budget, 0 <= M <= K + (D-1) K^2
 * Outputs [B, M+1]: tokens (root -1), parents (root -1), depth, values
 * (float32 cumulative ln probability; computed in float64).  Token choices
 * compare raw logits (exact); node values near a selection boundary may
 * order differently from a float64 reference when within ~1e-12.
 * Workspace: spec_verify_workspace_bytes(SPEC_MODE_TREE_GROW, B, K, V, dtype)
 * (sized for up to 16 layers); requires ceil(V / chunk) * K <= 2048 (chunk =
 * 16384 bf16 / 8192 fp32 elements).  Two kernel launches: the K best tokens
 * and softmax normaliser of every draft row read (B (1 + (D-1) K) rows, one
 * streaming pass), then a cluster of two CTAs per tree for the rows' merge,
 * the layer-by-layer expansion and the selection of the M best nodes.
 */
SPEC_API spec_status_t spec_tree_grow(const void* draft_logits, int dtype, float temperature,
                                      int B, int D, int K, int V, int M, int32_t* tokens,
                                      int32_t* parents, int32_t* depth, float* values,
                                      void* workspace, size_t workspace_bytes, void* stream);

/*
 * spec_tree_qkv_rope for a cache in pages: the same norms, rotation and
 * queries, but node v's key and value go to place v of k_out and v_out
 * (bf16 [B, N, Hkv, D], 16-byte aligned), where spec_tree_attention_kv4 and
 * spec_kv4_commit_path take them.  A sequence with base_len < 1 gets queries of
 * 0, writes no key or value and raises SPEC_FLAG_BAD_PATH.  One launch;
 * workspace as spec_tree_qkv_rope.
 */
SPEC_API spec_status_t spec_tree_qkv_rope_nodes(const void* qkv, const void* q_norm,
                                                const void* k_norm, float eps,
                                                const float* inv_freq, int rot_dim,
                                                int interleaved, long long pos_offset,
                                                const int32_t* base_len, const int32_t* depth,
                                                int B, int N, int Hq, int Hkv, int D, void* q_out,
                                                void* k_out, void* v_out, void* workspace,
                                                size_t workspace_bytes, void* stream);

/*
 * A key-value cache in pages of 4-bit values (a deployment format: the pages
 * cited above fix only which entries a node sees and which are kept, "The
 * Complete EAGLE-3 Inference Process" steps 3 and 5).
 *
 *   pages       uint8 [layers, n_pages, Hkv, block], 16-byte aligned: a page
 *               holds page_size positions (16, 32, 64 or 128) of one layer.  The
 *               block of a head is 9 page_size D / 8 bytes: for each 16
 *               positions key codes [16, D/2], key scales [16, D/16], value
 *               codes, value scales
 *   page_table  int32 [B, W]: position t of sequence b stands in page
 *               page_table[b, t / page_size], at place t % page_size, in every
 *               layer; sequences may share pages
 *   kv_exp      int32 [layers, 2] or NULL (all 0): exponents e of a layer's keys
 *               and values (beyond +-64 taken as that)
 * 16 channels of a head share a scale: with a = max |x|,
 *   s = e4m3(min(448, a / 6 * 2^-e)),  code = e2m1(x / (s 2^e)),
 *   value = code * s * 2^e,
 * both to nearest even, codes saturating at 6 (all codes 0 where s is 0), the
 * even channel in a byte's low half.  Values are exact in bf16.  A good e keeps
 * s between 2^-6 and 448: a between 0.1 * 2^e and 2688 * 2^e.
 *
 * spec_kv4_commit_path writes the accepted path of B sequences into the pages
 * of all layers.  For the path 0, v_1, ..., v_d (d = accepted_len[b]) node
 * v_i's key and value go to position base_len[b] - 1 + i (the root, node 0, is
 * the last committed token: its entry is written too), and new_len[b] =
 * base_len[b] + d, the number of positions that hold entries.
 *   node_k, node_v  bf16 [layers, B, N, Hkv, D], finite
 *   base_len        int32 [B], at least 1
 *   accepted_len    int32 [B], 0..min(max_depth, N - 1); NULL: N - 1
 *   path_nodes      int32 [B, max_depth + 1], needs accepted_len; or NULL: a
 *                   chain, v_i = i (max_depth is not looked at).  With neither,
 *                   all N nodes are written: a prompt, or a part of one
 * All positions' table entries must name pages that no other sequence reads
 * there (spec_kv_pages_fork sees to that).  A sequence with a malformed path
 * (SPEC_FLAG_BAD_PATH) or a needed table entry that names no page
 * (SPEC_FLAG_BAD_PAGE) is left untouched, with new_len = max(base_len - 1, 0).
 * Elements that are not finite give unspecified values of their scale's 16.
 * new_len must not overlap the inputs (SPEC_ERR_INVALID_ARG).
 * One launch.  Workspace: spec_verify_workspace_bytes(SPEC_MODE_KV4, ...) bytes
 * (the flag header).  D is 64 or 128, N at most SPEC_MAX_TREE_NODES, W at most
 * SPEC_KV_MAX_TABLE.
 */
#define SPEC_KV_MAX_TABLE (1 << 20)
#define SPEC_KV_MAX_PAGES (1 << 24) /* of spec_kv_pages_fork and _compact */
SPEC_API spec_status_t spec_kv4_commit_path(void* pages, int layers, long long n_pages,
                                            int page_size, int Hkv, int D,
                                            const int32_t* page_table, int W, const void* node_k,
                                            const void* node_v, const int32_t* base_len,
                                            const int32_t* accepted_len, const int32_t* path_nodes,
                                            int max_depth, const int32_t* kv_exp, int B, int N,
                                            int32_t* new_len, void* workspace,
                                            size_t workspace_bytes, void* stream);

/*
 * The first length[b] positions of B sequences, all layers, back in bf16 (a
 * prefix for spec_tree_attention, or another consumer's cache).
 *   length        int32 [B], 0..L (others are cut to that and raise
 *                 SPEC_FLAG_BAD_PATH)
 *   k_out, v_out  bf16: position t of sequence b and layer l starts l *
 *                 layer_stride + b * seq_stride + t * Hkv * D * 2 bytes in; both
 *                 strides multiples of 16, the arrays 16-byte aligned.  Positions
 *                 from length[b] on keep their contents
 * Positions whose table entry names no page read as 0 (SPEC_FLAG_BAD_PAGE).
 * One launch; workspace as spec_kv4_commit_path.
 */
SPEC_API spec_status_t spec_kv4_read(const void* pages, int layers, long long n_pages,
                                     int page_size, int Hkv, int D, const int32_t* page_table,
                                     int W, const int32_t* length, const int32_t* kv_exp, int B,
                                     int L, void* k_out, void* v_out, long long layer_stride,
                                     long long seq_stride, void* workspace, size_t workspace_bytes,
                                     void* stream);

/*
 * spec_tree_attention over one layer of a 4-bit cache in pages: query head
 * h G + g of node v of sequence b attends to
 *   - the committed positions [0, base_len[b] - 1), in the pages;
 *   - the tree's nodes u < N of the node's mask row (NULL: u <= v, a chain),
 *     whose keys and values are still bf16.
 *   q, out          bf16 [B, N, Hq, D];  lse float [B, N, Hq] or NULL
 *   pages           uint8 [n_pages, Hkv, block] (one layer, see above)
 *   node_k, node_v  bf16 [B, N, Hkv, D], taken as fp16 in units of 2^e (kv_exp's of
 *                   keys, of values): exact from 2^-17 * 2^e to 65504 * 2^e,
 *                   larger magnitudes count as that, smaller ones are rounded
 *                   to multiples of 2^-24 * 2^e (the cache itself holds up to
 *                   2688 * 2^e, in steps of 2^-10 * 2^e at least)
 *   mask, base_len, scale  as spec_tree_attention;  kv_exp int32 [2] or NULL
 * N = 1 without a mask is plain decoding.  A node that sees nothing gets out = 0
 * and lse = -inf.  Entries that a node does not see are never used, whatever
 * they hold; a node's entry with an element that is not finite makes out and
 * lse NaN for the query heads that see it, and so does a query element that is
 * not finite for its own head.  Positions whose table entry names no page are
 * not seen (SPEC_FLAG_BAD_PAGE); a sequence with base_len < 1 or more than W *
 * page_size committed positions gets out = 0, lse = -inf and raises
 * SPEC_FLAG_BAD_PATH.
 * Queries and weights are rounded to fp16 (queries at a power of two that
 * brings a head's largest element to 2^14, weights at 2^7: both have at least
 * bf16's 8 bits down to 2^-24 of the largest), the cached values are exact in
 * fp16, sums are float32.  out and lse must not overlap the inputs
 * (SPEC_ERR_INVALID_ARG).  Limits as spec_tree_attention (D 64 or 128, G at most
 * 128, N at most SPEC_ATTN_MAX_NODES); W * page_size + N at most 2^31 - 257.  Two
 * launches; the cut of the work, and so the last bits, depend on base_len and
 * the number of SMs alone.  Workspace: at least
 * spec_tree_attention_kv4_workspace_bytes() bytes.
 */
SPEC_API size_t spec_tree_attention_kv4_workspace_bytes(int B, int N, int Hq, int Hkv, int D);
SPEC_API spec_status_t spec_tree_attention_kv4(const void* q, const void* pages, long long n_pages,
                                               int page_size, const int32_t* page_table, int W,
                                               const void* node_k, const void* node_v,
                                               const uint32_t* mask, const int32_t* base_len,
                                               const int32_t* kv_exp, int B, int N, int Hq,
                                               int Hkv, int D, float scale, void* out, float* lse,
                                               void* workspace, size_t workspace_bytes,
                                               void* stream);

/*
 * Forks of sequences whose pages a table names (any cache in pages: a page is
 * page_bytes bytes in each of `planes` planes).  New sequence j goes on from
 * old sequence parent[j], several from one if need be (beams, samples of one
 * prompt), or is empty (parent[j] = -1):
 *   - new_len[j] = length[parent[j]]; the pages that are full up to there are
 *     shared;
 *   - the unfinished page is taken over by the lowest j that has it, unless a
 *     sequence holds it as a full one; the others get a copy of it (all planes);
 *   - fresh pages follow up to need[j] positions (at least new_len[j]), the free
 *     pages with the lowest ids first, in the order of j and of places; pages
 *     that no new sequence holds are free (entries of page_table behind a
 *     sequence's length are not looked at).
 * So every position from new_len[j] on stands in a page that j alone holds.
 *   pages       planes plane_stride bytes apart, each n_pages * page_bytes;
 *               16-byte aligned, strides and page_bytes multiples of 16
 *   page_table  int32 [B, W]; length int32 [B], 0..W page_size
 *   parent      int32 [B2], or NULL (j's own, B2 <= B: growth alone)
 *   need        int32 [B2], or NULL (new_len)
 * Outputs: new_table int32 [B2, W] (-1 behind a sequence's pages), new_len
 * int32 [B2], used int32 [1] (pages held).  Outputs must not overlap the inputs
 * (SPEC_ERR_INVALID_ARG).  No page left: -1 (SPEC_FLAG_NO_PAGE).  A needed entry
 * that names no page stays -1, an unfinished one gets a fresh page without a
 * copy (SPEC_FLAG_BAD_PAGE); a parent outside [-1, B) counts as -1
 * (SPEC_FLAG_BAD_PARENT); a length outside its range counts as 0, a need beyond
 * W page_size as that (SPEC_FLAG_BAD_PATH).
 * B2 = 0 frees all pages (used = 0).  Two launches.  Workspace:
 * spec_kv_pages_workspace_bytes(n_pages, B2) bytes.
 */
SPEC_API size_t spec_kv_pages_workspace_bytes(long long n_pages, int rows);
SPEC_API spec_status_t spec_kv_pages_fork(void* pages, int planes, long long plane_stride,
                                          long long n_pages, long long page_bytes, int page_size,
                                          const int32_t* page_table, const int32_t* length, int B,
                                          const int32_t* parent, const int32_t* need, int B2,
                                          int W, int32_t* new_table, int32_t* new_len,
                                          int32_t* used, void* workspace, size_t workspace_bytes,
                                          void* stream);

/*
 * Compaction: the n pages that a table names move to the places [0, n), so that
 * the pages from n on can be given back.  A page below n stays; those from n on
 * move to the free places below n, in ascending order both.
 *   page_table  int32 [B, W], negative: no page (others outside [0, n_pages)
 *               become -1, SPEC_FLAG_BAD_PAGE)
 * Outputs: new_table int32 [B, W] (may be page_table itself, not a part of it),
 * used int32 [1] (n).
 * Two launches.  Other arguments as spec_kv_pages_fork; workspace:
 * spec_kv_pages_workspace_bytes(n_pages, B) bytes.
 */
SPEC_API spec_status_t spec_kv_pages_compact(void* pages, int planes, long long plane_stride,
                                             long long n_pages, long long page_bytes,
                                             const int32_t* page_table, int B, int W,
                                             int32_t* new_table, int32_t* used, void* workspace,
                                             size_t workspace_bytes, void* stream);

/*
 * Beam search's selection (no counterpart in the pages: a decoder beside the
 * draft trees): the M best continuations of each request over its K beams and
 * V tokens,
 *   total[b, k, v] = scores[b, k] + z_v / T - ln sum_j exp(z_j / T),
 * z = logits[b, k, :]; a finished beam has the single candidate (eos, its
 * score).  Larger totals first, then lower beams, then lower tokens (logits -0 and
 * +0 are the same).
 *   logits    [B, K, V] dtype, of any magnitude; -inf is a token of probability 0
 *             (a row of the type's lowest value alone is a flat one)
 *   scores    float [B, K]; -inf (or NaN): the beam has no candidate
 *   finished  int32 [B, K] (not 0: finished) or NULL
 *   eos       the token that ends a beam, or -1
 *   K         1..64;  M 1..16;  B K ceil(V / chunk) < 2^25 (chunk = 16384 bf16 /
 *             8192 fp32 elements)
 * Outputs [B, M]: out_scores float (the totals), out_parents int32 (rows b K +
 * k: what spec_kv_pages_fork takes), out_tokens int32, out_finished int32 (the
 * parent was finished, or the token is eos).  Places without a candidate:
 * -inf, -1, -1, 1.
 * Totals are ordered in float64 from float32 exponentials: they are off by less
 * than 2^-18 + 2^-24 (z_max - z_v) / T, z_max the row's largest logit (and
 * out_scores rounds them to float); within a beam the order is that of the
 * logits, and beams with the same logits and scores tie.  A logit that is NaN
 * or +inf makes what its request gets unspecified.  Outputs must not overlap
 * the inputs (SPEC_ERR_INVALID_ARG).
 * Two launches.  Workspace: spec_beam_select_workspace_bytes() bytes.
 */
SPEC_API size_t spec_beam_select_workspace_bytes(int B, int K, int V, int M, int dtype);
SPEC_API spec_status_t spec_beam_select(const void* logits, int dtype, const float* scores,
                                        const int32_t* finished, int eos, float temperature, int B,
                                        int K, int V, int M, float* out_scores,
                                        int32_t* out_parents, int32_t* out_tokens,
                                        int32_t* out_finished, void* workspace,
                                        size_t workspace_bytes, void* stream);

/*
 * Copy the workspace's flag word to *host_flags (synchronises `stream`); with
 * clear != 0 the word is then reset to 0 on the stream.
 */
SPEC_API spec_status_t spec_verify_read_flags(void* workspace, uint32_t* host_flags, int clear,
                                     void* stream);

/*
 * Self-test of the two 2^x evaluations the kernels use (no counterpart in the
 * pages): y_fma[i] = the FMA-pipe polynomial (Cody-Waite reduction, degree-5
 * minimax; relative error below 2e-7 for -126 <= x <= 0.5), y_sfu[i] = the
 * special-function unit's ex2.approx.ftz.  x, y_fma, y_sfu: device float [n].
 */
SPEC_API spec_status_t spec_verify_selftest_exp2(const float* x, float* y_fma, float* y_sfu,
                                                 int n, void* stream);

/* Number of kernels this library has launched in this process. */
SPEC_API uint64_t spec_verify_launch_count(void);

/*
 * Diagnostic control of the bounded waits (no counterpart in the pages).
 *
 * Every wait of the verification kernels on their own bulk copies, and every
 * wait between the roles of a CTA of spec_tree_attention and of
 * spec_tree_attention_kv4 (copies, products, softmax), gives up after a limit
 * (0.2 s by default; the one role that lists a CTA's work ahead may wait 20 us
 * longer for each tile of it): the CTA then sets SPEC_FLAG_TIMEOUT, stops
 * copying, waits (with the default limit) for the copies and products it has
 * in flight and finishes its control flow, so the call completes with
 * unspecified outputs and the flag raised instead of hanging.  This sets the
 * limit used by calls of spec_verify_sample, spec_verify_greedy,
 * spec_verify_tree_greedy, spec_verify_greedy_noalloc, spec_tree_attention and
 * spec_tree_attention_kv4 enqueued afterwards, process-wide; limit_ns = 0
 * restores the default.  limit_ns = 1 gives up whenever a copy has not landed
 * (a role has not answered) at the first look, which is how a test exercises
 * that path.  Between two looks at the GPU's clock a wait sleeps for about 4 us
 * at least (shorter limits are rounded up) and 1 ms at most.  Not for
 * production use.
 */
SPEC_API void spec_verify_set_wait_limit_ns(uint64_t limit_ns);

/*
 * Greedy verification without any allocation (no counterpart in the pages:
 * this is a deployment convenience, not part of the method).
 *
 * Same computation, arguments and outputs as spec_verify_greedy, minus the
 * workspace: its scratch is a fixed array of SPEC_NOALLOC_SCRATCH_BYTES in
 * the library's own device memory, resident on every GPU that loads the
 * library until the process exits.  It is for callers that cannot allocate
 * device memory at the point of the call: for example a plugin inside a
 * serving framework that owns every device allocation, or a decode loop that
 * must not allocate once it is running.  The library itself calls no
 * cudaMalloc, cudaFree or other allocating routine on this path.
 *
 *   - The first call on each device looks up the array's device address
 *     (cudaGetSymbolAddress, with that device current) and caches it for the
 *     device's current context; make that first call before any stream
 *     capture begins on the device, and again after a cudaDeviceReset.
 *   - Calls whose scratch would exceed SPEC_NOALLOC_SCRATCH_BYTES return
 *     SPEC_ERR_TOO_LARGE before anything is enqueued (B=64 sequences of k=4
 *     drafts over V=128256 bf16 need about 0.66 MB).
 *   - Every call uses the same array, which keeps what the previous call left
 *     there.  Nothing the kernels read needs to start at zero; the flag word is
 *     cleared on entry and device-side input errors are not reported.  Calls
 *     that overlap on the GPU (different streams without ordering, or
 *     concurrent host threads) race on the array: serialise them.
 */
#define SPEC_NOALLOC_SCRATCH_BYTES (4u << 20)
SPEC_API spec_status_t spec_verify_greedy_noalloc(const void* target_logits, int dtype,
                                                  const int32_t* draft_tokens, int B, int k, int V,
                                                  int32_t* accepted_len, int32_t* out_tokens,
                                                  void* stream);

/* Static description of a status code. */
SPEC_API const char* spec_status_string(int status);

/* SPEC_VERIFY_ABI_VERSION of the loaded library. */
SPEC_API int spec_verify_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_VERIFY_H_ */

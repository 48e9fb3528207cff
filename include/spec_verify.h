/*
 * spec_verify.h - C ABI of libspecverify, the GB300 (sm_103a) implementation
 * of the target-model verification step of speculative decoding.
 *
 * The method is the one stated on these pages:
 *   "【大模型基础设施工程】15：推测解码与 MTP" (juejin.cn), §2.1 "算法骨架":
 *     accept draft x_i with probability min(1, p_i(x_i) / q_i(x_i)); at the
 *     first rejection draw one token from norm(max(0, p_i - q_i)) and stop;
 *     if all K drafts are accepted draw one extra token from p_{K+1}.
 *   the same page, "1.2 正确性保证" (inside part 2): the emitted tokens are
 *     distributed exactly as sampling from the target;
 *   the same page, §2.3: 1 <= accept length <= K+1;
 *   the same page, §3.3 "Tree Attention": candidate trees, each node sees only
 *     its ancestors, the longest accepted root path wins;
 *   the same page, §11: greedy (do_sample=False) output equals plain decoding;
 *   "投机解码" (FastDeploy docs), "高效投机解码框架设计": per-sample parallel
 *     sampling+verification; output tokens located by batch id through
 *     padding-free indexing instead of copies and slices.
 *
 * Conventions shared by every entry point
 *   - Tensor pointers are DEVICE pointers to caller-owned, contiguous,
 *     row-major memory.  The library never allocates, frees or retains them;
 *     it reads inputs and writes outputs on `stream`.
 *   - Calls are asynchronous and stream-ordered: they return after queueing
 *     the kernels; nothing is synchronised.  `stream` is a cudaStream_t
 *     (NULL = the legacy default stream).
 *   - The return value reports ARGUMENT errors found on the host before any
 *     launch (nothing is queued then), or SV_ERR_CUDA if a launch failed.
 *   - DATA errors found on the device never trap or hang: they set bits in
 *     the request's status word (SV_REQ_*), and that request emits nothing
 *     (accept_len 0, all token slots -1).
 *   - Token ids are int32.  Unused output token slots hold -1.
 *   - Logits are bfloat16 or IEEE fp32 (sv_dtype).  Every logit must be finite
 *     or -inf (masking); each row that the rule needs must hold at least one
 *     finite logit.  NaN or +inf in a needed row is a data error.  |logit / T|
 *     must be representable in fp32.
 *   - A workspace (device memory, >= spec_verify_workspace_size bytes,
 *     256-byte aligned) holds per-call scratch: chunk records, row summaries
 *     and arrival counters.  Zero-fill a newly allocated workspace once with
 *     spec_verify_workspace_init.  The counters must be zero when a call
 *     starts; every call leaves them zero, and when a workspace is used with a
 *     different (B, K, mode) than on its previous call, the library first
 *     zero-fills the counter region on the call's stream (one small
 *     cudaMemsetAsync).  Calls that share a workspace must be ordered on one
 *     stream: concurrent calls need separate workspaces.
 */
#ifndef SPEC_VERIFY_H_
#define SPEC_VERIFY_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct CUstream_st* sv_stream_t;

typedef enum sv_status {
  SV_OK = 0,
  SV_ERR_NULL = 1,        /* a required pointer is NULL */
  SV_ERR_SHAPE = 2,       /* B, K, V, N or max_depth outside the supported range */
  SV_ERR_DTYPE = 3,       /* unknown sv_dtype */
  SV_ERR_TEMPERATURE = 4, /* temperature negative, NaN or infinite */
  SV_ERR_TREE = 5,        /* tree parent stride neither 0 nor N */
  SV_ERR_WORKSPACE = 6,   /* workspace NULL, not 256-byte aligned, or too small */
  SV_ERR_CUDA = 7,        /* a CUDA runtime call or kernel launch failed */
  SV_ERR_FILTER = 8,      /* top_k negative, top_p outside (0, 1], or eps / delta negative */
  SV_ERR_ALIAS = 9,       /* an output overlaps an input that it must not overlap */
  SV_ERR_SCORE = 10       /* attention scale not finite, softcap outside [0, 1e30], window negative */
} sv_status;

typedef enum sv_dtype { SV_F32 = 0, SV_BF16 = 1 } sv_dtype;

/* Per-request device status bits (out_status). */
#define SV_REQ_BAD_TOKEN 1     /* a draft / tree token outside [0, V) */
#define SV_REQ_BAD_LOGITS 2    /* a needed row has NaN or +inf, or no finite logit */
#define SV_REQ_BAD_DRAFT_LEN 4 /* draft_lens[b] outside [0, K] */
#define SV_REQ_TIMEOUT 8       /* a bounded wait for staged logits gave up (device fault, or
                                  the limit of spec_verify_set_wait_limit_ns ran out) */
#define SV_REQ_BAD_TREE 16     /* the request's parent array is not a tree of depth <= max_depth */
#define SV_REQ_BAD_PAGE 32     /* a page that the request needs is not one of the cache's */

/* Limits. */
#define SV_MAX_K 31             /* draft positions per request */
#define SV_MAX_B 65536          /* requests per call */
#define SV_MAX_V (1 << 24)      /* vocabulary size */
#define SV_MAX_TREE_NODES 256   /* candidate nodes per tree (root excluded) */
#define SV_MAX_NGRAM 32         /* longest n-gram the proposer matches */
#define SV_MAX_TOP 128          /* logits of a top-logits record, candidates a beam selection keeps */
#define SV_MAX_BEAMS 64         /* beams per request */
#define SV_MAX_ROWS (1 << 27)   /* rows (B * P) of a top-logits or distillation call */
#define SV_MAX_DISTILL_ROW 1572864 /* bytes of a student row (V * sizeof(logit)) */
#define SV_MAX_STEP 257         /* tokens of a verification step: a tree's nodes and its root */
#define SV_MAX_HEADS 1024       /* heads of a layer */
#define SV_MAX_SLOTS (1 << 27)  /* tokens a request's page table can hold */

/* Bytes of workspace that spec_verify_sample / _greedy need for B requests
 * of K draft positions over a vocabulary of V (the dense-draft sampling case,
 * the largest).  spec_verify_tree needs none.  Returns 0 if out of range. */
size_t spec_verify_workspace_size(int B, int K, int V);

/* Zero-fill a workspace on `stream` (one cudaMemsetAsync).  Needed once per
 * workspace before its first use. */
sv_status spec_verify_workspace_init(void* workspace, size_t ws_bytes, sv_stream_t stream);

/* Rejection-sampling verification ("推测解码与 MTP" §2.1).
 *
 *   target_logits  [B, K+1, V] dtype: row i < K scores draft position i,
 *                  row K is the extra (bonus) position.
 *   draft_logits   [B, K, V] dtype, or NULL.  Given: q_i = softmax(d_i / T),
 *                  the same temperature as the target (the drafts are assumed
 *                  sampled from exactly that q).  NULL: one-hot drafts from a
 *                  deterministic proposer (n-gram / prompt lookup), q_i is the
 *                  point mass at x_i: acceptance probability p_i(x_i), residual
 *                  p_i with x_i removed and renormalised.
 *   draft_tokens   [B, K] int32, the drafts x_i.  May be NULL when K == 0.
 *   uniforms       [B, K+1] fp32 in [0, 1): column i < K drives the test at
 *                  position i (accept iff u_i * q_i(x_i) < p_i(x_i)); column K
 *                  drives the residual or bonus draw: the emitted token is the
 *                  smallest j whose cumulative weight exceeds u_K times the total.
 *   temperature    T > 0: p_i = softmax(target_i / T).  T == 0 selects the greedy
 *                  rule of spec_verify_greedy (draft_logits and uniforms unused;
 *                  out_accept_prob reports 1 for a match and 0 for a mismatch).
 *   out_tokens     [B, K+1] int32: x_0 .. x_{n-1}, then the drawn token, then -1.
 *   out_accept_len [B] int32: n + 1 emitted tokens (1 <= n+1 <= K_b+1), or 0 for
 *                  a request with a data error.
 *   dtype, B, K, V 1 <= B <= SV_MAX_B, 0 <= K <= SV_MAX_K, 1 <= V <= SV_MAX_V.
 *   draft_lens     [B] int32 or NULL: per-request draft count K_b <= K (ragged
 *                  drafts).  Rows beyond K_b are never read; the bonus position
 *                  of request b is row K_b; the draw still uses column K.
 *   out_cu_accept  [B+1] int32 or NULL: exclusive prefix sum of out_accept_len.
 *   out_packed     [B*(K+1)] int32 or NULL: the emitted tokens of all requests
 *                  back to back (request b at out_cu_accept[b]..), then -1.
 *   out_batch_id   [B*(K+1)] int32 or NULL: the request of each packed token, -1
 *                  past the end.  (Any of the three packed outputs may be given
 *                  alone; out_cu_accept is computed either way.)
 *   out_accept_prob [B, K] fp32 or NULL: min(1, p_i(x_i)/q_i(x_i)) at each
 *                  tested position (i <= n, i < K_b), -1 elsewhere.
 *   out_status     [B] int32 or NULL: SV_REQ_* bits per request.
 *   workspace, ws_bytes  see the conventions above.
 */
sv_status spec_verify_sample(const void* target_logits, const void* draft_logits,
                             const int32_t* draft_tokens, const float* uniforms,
                             float temperature, int32_t* out_tokens, int32_t* out_accept_len,
                             sv_dtype dtype, int B, int K, int V, const int32_t* draft_lens,
                             int32_t* out_cu_accept, int32_t* out_packed,
                             int32_t* out_batch_id, float* out_accept_prob,
                             int32_t* out_status, void* workspace, size_t ws_bytes,
                             sv_stream_t stream);

/* Greedy verification ("推测解码与 MTP" §11, temperature 0): x_i is accepted
 * while it equals the argmax of target row i (lowest index among equal
 * maxima; -0.0 == +0.0); the first mismatch emits that argmax; if all K_b
 * match, the argmax of row K_b is the extra token.  Arguments as in
 * spec_verify_sample.  Bit-exact: the argmax is taken on the stored values. */
sv_status spec_verify_greedy(const void* target_logits, const int32_t* draft_tokens,
                             int32_t* out_tokens, int32_t* out_accept_len, sv_dtype dtype,
                             int B, int K, int V, const int32_t* draft_lens,
                             int32_t* out_cu_accept, int32_t* out_packed,
                             int32_t* out_batch_id, int32_t* out_status, void* workspace,
                             size_t ws_bytes, sv_stream_t stream);

/* Grammar-constrained verification ("Speculative Decoding" (LMDeploy docs),
 * "投机解码与结构化输出" / "工作原理"): with structured output (a JSON schema, a
 * regular expression) each position may only emit the tokens its grammar
 * state allows.  The mask of position i is applied to target row i - and to
 * draft row i, since the draft was proposed under the same mask - before the
 * rule runs: a ruled-out token has probability 0, so it is never accepted,
 * drawn or taken as the argmax.  The masks of positions 1..K depend on the
 * drafts before them; the caller's grammar matcher computes them all (on a
 * fork advanced through the drafts) before the call.
 *
 *   token_mask  [B, K+1, ceil(V/32)] 32-bit words, 4-byte aligned: request b,
 *               position i allows token j iff bit j % 32 of word j / 32 of row
 *               (b, i) is set.  Bits at j >= V are ignored.  When the rows are
 *               16-byte aligned (16-byte aligned base and ceil(V/32) a multiple
 *               of 4) the words travel with the logits in the same bulk copies;
 *               otherwise they are read word by word.
 * A needed position whose mask leaves no finite logit is a data error
 * (SV_REQ_BAD_LOGITS).  NULL or misaligned token_mask: SV_ERR_NULL.  All other
 * arguments, results and the workspace size are those of spec_verify_sample
 * and spec_verify_greedy. */
sv_status spec_verify_sample_masked(const void* target_logits, const void* draft_logits,
                                    const int32_t* draft_tokens, const float* uniforms,
                                    float temperature, const uint32_t* token_mask,
                                    int32_t* out_tokens, int32_t* out_accept_len, sv_dtype dtype,
                                    int B, int K, int V, const int32_t* draft_lens,
                                    int32_t* out_cu_accept, int32_t* out_packed,
                                    int32_t* out_batch_id, float* out_accept_prob,
                                    int32_t* out_status, void* workspace, size_t ws_bytes,
                                    sv_stream_t stream);
sv_status spec_verify_greedy_masked(const void* target_logits, const int32_t* draft_tokens,
                                    const uint32_t* token_mask, int32_t* out_tokens,
                                    int32_t* out_accept_len, sv_dtype dtype, int B, int K, int V,
                                    const int32_t* draft_lens, int32_t* out_cu_accept,
                                    int32_t* out_packed, int32_t* out_batch_id,
                                    int32_t* out_status, void* workspace, size_t ws_bytes,
                                    sv_stream_t stream);

/* Verification of top-k / top-p filtered sampling (the vLLM Ascend guide's
 * examples sample with SamplingParams(temperature=0.8, top_p=0.95); "推测解码与
 * MTP" §8.3 non-greedy decoding with wide top-p).  Every sampled
 * distribution - target rows and, with dense drafts, draft rows - is the
 * tempered softmax of the (grammar-masked) logits filtered as follows, and
 * the drafts are assumed drawn from the filtered draft distributions:
 *   top_k > 0 keeps the tokens whose logit is >= the k-th largest logit of
 *     the row (counted with multiplicity, so ties at the cut are all kept),
 *     then renormalises; top_k = 0 (or >= V) switches it off;
 *   top_p < 1 then keeps a token when the probability mass of the tokens
 *     with a strictly larger logit is below top_p (the smallest set of
 *     leading logit values whose mass reaches top_p, ties kept together),
 *     then renormalises; top_p = 1 switches it off.
 * The acceptance test, the residual norm(max(0, p' - q')) and the bonus draw
 * use the filtered p', q'.  temperature == 0 is the greedy rule (filters do
 * not change the argmax).  token_mask: as in spec_verify_sample_masked, or
 * NULL.  Each row of a filtered call is taken by one CTA: V * sizeof(logit)
 * must not exceed 512 KB (V <= 262144 for bf16, 131072 for fp32), else
 * SV_ERR_SHAPE.  SV_ERR_FILTER for a negative top_k or
 * top_p outside (0, 1].
 *   out_cut   [B, R] fp32 or NULL, R = K+1 (one-hot drafts) or 2K+1 (draft
 *             logits): the lowest logit each filtered distribution keeps -
 *             row i <= K target position i, row K+1+i the draft of position
 *             i; NaN for rows the request does not need (beyond K_b, or a
 *             request with a bad draft length); -inf for a row without a
 *             finite max.  Written only when a filter is active (top_k in
 *             (0, V) or top_p < 1).  With top-p the cut is where the fp32
 *             mass of the leading value classes reaches top_p; it tells a
 *             caller (or a test) which value classes were kept.
 * All other arguments, results and the workspace size are those of
 * spec_verify_sample. */
sv_status spec_verify_sample_filtered(const void* target_logits, const void* draft_logits,
                                      const int32_t* draft_tokens, const float* uniforms,
                                      float temperature, int top_k, float top_p,
                                      const uint32_t* token_mask, int32_t* out_tokens,
                                      int32_t* out_accept_len, sv_dtype dtype, int B, int K, int V,
                                      const int32_t* draft_lens, int32_t* out_cu_accept,
                                      int32_t* out_packed, int32_t* out_batch_id,
                                      float* out_accept_prob, float* out_cut,
                                      int32_t* out_status, void* workspace, size_t ws_bytes,
                                      sv_stream_t stream);

/* Typical acceptance ("推测解码与 MTP" §10.4: the rule of the original Medusa,
 * an approximation that is not exactly lossless, also offered by EAGLE).
 * Draft x_i passes when p_i(x_i) > min(eps, delta * exp(-H(p_i))), with p_i
 * the tempered target distribution of position i and H its entropy in nats;
 * positions are tested in order, and at the first failure n (or at K_b when
 * all pass) one token is drawn from p_n itself with uniforms[b, K] (inverse
 * CDF: the smallest j whose cumulative probability exceeds u).  There is no
 * residual: the output follows the rule, not the target distribution.
 *   eps, delta      the rule's two thresholds (Medusa's defaults are 0.09 and
 *                   0.3), finite and >= 0, else SV_ERR_FILTER.
 *   temperature     T > 0; T == 0 applies the greedy rule instead.
 *   out_accept_prob p_i(x_i) at each tested position, -1 elsewhere.
 * Drafts are one-hot (no draft logits).  uniforms [B, K+1], of which only
 * column K is used.  All other arguments, results and the workspace size are
 * those of spec_verify_sample. */
sv_status spec_verify_typical(const void* target_logits, const int32_t* draft_tokens,
                              const float* uniforms, float temperature, float eps, float delta,
                              int32_t* out_tokens, int32_t* out_accept_len, sv_dtype dtype, int B,
                              int K, int V, const int32_t* draft_lens, int32_t* out_cu_accept,
                              int32_t* out_packed, int32_t* out_batch_id, float* out_accept_prob,
                              int32_t* out_status, void* workspace, size_t ws_bytes,
                              sv_stream_t stream);

/* Typical acceptance on a candidate tree (§10.4 with §3.3).  Node n passes
 * when its parent passed (the root always does) and its token passes the
 * typical test under its parent's distribution; the result is the deepest
 * passing node (the lowest id among equally deep ones): the tokens of its
 * root path, then one token drawn from its own distribution with
 * uniforms[b].  Rows of passing nodes must be valid (SV_REQ_BAD_LOGITS).
 *   target_logits, tree_parent, parent_stride, tree_tokens, out_tokens,
 *   out_path, out_accept_len, out_status, max_depth: as in spec_verify_tree.
 *   uniforms [B] fp32 in [0, 1).  temperature > 0; eps, delta as in
 *   spec_verify_typical.  workspace: >= spec_verify_tree_workspace_size(B, N,
 *   V) bytes, 256-byte aligned, zero-filled once (spec_verify_workspace_init).
 * Every row of the tree is read once (all candidate rows are reduced in
 * parallel). */
size_t spec_verify_tree_workspace_size(int B, int N, int V);
sv_status spec_verify_tree_typical(const void* target_logits, const int32_t* tree_parent,
                                   int parent_stride, const int32_t* tree_tokens,
                                   const float* uniforms, float temperature, float eps,
                                   float delta, int32_t* out_tokens, int32_t* out_accept_len,
                                   sv_dtype dtype, int B, int N, int V, int max_depth,
                                   int32_t* out_path, int32_t* out_status, void* workspace,
                                   size_t ws_bytes, sv_stream_t stream);

/* Lossless tree verification by rejection sampling ("推测解码与 MTP" §10.4:
 * the methods that verify by rejection sampling, EAGLE among them, are
 * lossless; the candidate trees of §3.3 "Tree Attention" and §4.2, whose
 * nodes are each head's top-k candidates).  Every candidate is a
 * deterministic (one-hot) draft of the distribution at its parent.  From the
 * root: with p the tempered target distribution at the current node and w = p,
 * the node's children are tested in increasing id - child c with token x_c
 * is accepted iff u_c < w(x_c) / sum(w), and a rejected child's token leaves
 * w (w(x_c) = 0); the first accepted child's token is emitted and the walk
 * moves to it; when no child is accepted (or at a leaf) one token is drawn
 * from w / sum(w) with u_0 (the smallest j whose cumulative weight exceeds
 * u_0 times the total) and the walk ends.  Each emitted token is distributed
 * exactly as the target's distribution at its node; a token repeated among
 * siblings has no mass left when its turn comes and is rejected.
 *   uniforms  [B, N+1] fp32 in [0, 1): column c (1..N) drives the test of
 *             node c, column 0 the final draw.
 *   temperature  T > 0; T == 0 runs the greedy walk of spec_verify_tree
 *             (uniforms and workspace unused).
 *   target_logits, tree_parent, parent_stride, tree_tokens, out_tokens,
 *   out_path, out_accept_len, out_status, max_depth: as in spec_verify_tree
 *   (out_tokens: the accepted candidates' tokens, then the drawn token).
 *   workspace: >= spec_verify_tree_workspace_size(B, N, V) bytes, as for
 *   spec_verify_tree_typical.
 * Every row of the tree is read once (all candidate rows are reduced in
 * parallel, each row's sums leaving out its children's tokens); only the
 * walked rows must be valid (SV_REQ_BAD_LOGITS). */
sv_status spec_verify_tree_sample(const void* target_logits, const int32_t* tree_parent,
                                  int parent_stride, const int32_t* tree_tokens,
                                  const float* uniforms, float temperature, int32_t* out_tokens,
                                  int32_t* out_accept_len, sv_dtype dtype, int B, int N, int V,
                                  int max_depth, int32_t* out_path, int32_t* out_status,
                                  void* workspace, size_t ws_bytes, sv_stream_t stream);

/* Greedy tree verification (Medusa / EAGLE; "推测解码与 MTP" §3.3).
 *
 *   target_logits  [B, N+1, V] dtype: row 0 is the root (the last committed
 *                  token), row n the target's logits after candidate node n.
 *   tree_parent    [N] or [B, N] int32 (device): parent of node n (n = 1..N)
 *                  at index n-1; a tree needs 0 <= parent < n (an earlier
 *                  node; breadth-first order qualifies) and no node deeper
 *                  than max_depth - a request whose array breaks this gets
 *                  SV_REQ_BAD_TREE and emits nothing.
 *   parent_stride  0: every request shares the one [N] tree; N: request b's
 *                  tree is tree_parent[b*N .. b*N+N) (EAGLE-2's dynamic trees,
 *                  built per request on the device, §4.3).  Other values:
 *                  SV_ERR_TREE.
 *   tree_tokens    [B, N] int32: the candidate token of node n at index n-1.
 *   out_tokens     [B, max_depth+1] int32: the target argmax at each node of the
 *                  accepted path (root first): the accepted node tokens followed
 *                  by the extra token; -1 after.
 *   out_accept_len [B] int32: accepted nodes + 1, or 0 on a data error.
 *   N, max_depth   0 <= N <= SV_MAX_TREE_NODES; max_depth >= the tree's depth.
 *   out_path       [B, max_depth+1] int32 or NULL: node ids of the path from the
 *                  root (0) on, -1 after.
 *   out_status     [B] int32 or NULL: SV_REQ_* bits.
 * A node is accepted when its token equals the argmax at its parent and its
 * parent is accepted.  With distinct sibling tokens (top-k candidates) the
 * accepted nodes form one chain and the walk returns the longest accepted
 * path; if a caller repeats a token among siblings, the lowest node id wins.
 * Only the rows on the accepted path are read. */
sv_status spec_verify_tree(const void* target_logits, const int32_t* tree_parent,
                           int parent_stride, const int32_t* tree_tokens, int32_t* out_tokens,
                           int32_t* out_accept_len, sv_dtype dtype, int B, int N, int V,
                           int max_depth, int32_t* out_path, int32_t* out_status,
                           sv_stream_t stream);

/* The longest time a kernel waits for logits it staged in shared memory (in
 * spec_top_logits and spec_beam_select, for what CTAs send each other or ask
 * of the launch) before it gives up: the call then marks every request
 * SV_REQ_TIMEOUT, calls of rows or beams those whose wait ran out (the
 * workspace stays usable; the next call starts clean).  Default 2 s, which
 * only a device fault can exhaust; a serving loop with a watchdog may set
 * less.  0 makes the waits give up at once, without polling - every call
 * that waits then reports SV_REQ_TIMEOUT, which is how the timeout path is
 * tested.
 * Process-wide; applies to the calls queued after it.  Always SV_OK. */
sv_status spec_verify_set_wait_limit_ns(uint64_t limit_ns);
uint64_t spec_verify_wait_limit_ns(void);

/* n-gram (prompt-lookup) proposer: the step before verification that makes
 * the one-hot drafts ("投机解码" (FastDeploy docs), "使用 Ngram 解码": drafts
 * come from matching an n-gram window against the prompt and the generated
 * tokens; the vLLM Ascend guide's n-gram example, prompt_lookup_max = 4 and 5
 * speculative tokens; "推测解码与 MTP" §9.1 prompt lookup).
 *
 * For n = n_max down to n_min, the last n tokens of request b's context
 * c = tokens[b, 0 .. lens[b]) are looked up earlier in c: the match is the
 * EARLIEST start s with c[s .. s+n) equal to them and at least one token
 * after it (s + n < lens[b]).  The first n that matches decides; the drafts
 * are the tokens after the match, c[s+n .. min(s+n+K, lens[b])).
 *
 *   tokens          [B, L] int32: request b's context in its first lens[b]
 *                   entries (prompt then generated tokens); the rest is never
 *                   read.  Any int32 values (they are only compared).
 *   lens            [B] int32, 0 <= lens[b] <= L; outside that range the
 *                   request gets no drafts and SV_REQ_BAD_DRAFT_LEN.
 *   n_min, n_max    1 <= n_min <= n_max <= SV_MAX_NGRAM.
 *   K               0 <= K <= SV_MAX_K drafts per request.
 *   out_drafts      [B, K] int32: the drafts, -1 after them.
 *   out_draft_lens  [B] int32: how many (0..K); pass it as draft_lens to
 *                   spec_verify_sample with draft_logits = NULL.
 *   out_match       [B] int32 or NULL: the start s, or -1 without a match.
 *   out_status      [B] int32 or NULL: SV_REQ_* bits.
 * B * L < 2^31.  One pass over each context; no workspace. */
sv_status spec_ngram_propose(const int32_t* tokens, const int32_t* lens, int B, int L,
                             int n_min, int n_max, int K, int32_t* out_drafts,
                             int32_t* out_draft_lens, int32_t* out_match, int32_t* out_status,
                             sv_stream_t stream);

/* The record of a teacher's rows: each row's k largest logits and its
 * log-sum-exp.  The verification step has the target's logits at hand at
 * every position; with lens = out_accept_len the rows on the accepted path
 * are recorded, and spec_distill trains a draft model on the records.
 *
 *   logits      [B, P, V] dtype (P = K+1 for the rows of a verify call).
 *   k           1 <= k <= SV_MAX_TOP logits kept per row.
 *   temperature T > 0, finite: out_lse is of the tempered logits.
 *   lens        [B] int32 or NULL: rows i < lens[b] of request b are recorded,
 *               the others are not read.  lens[b] outside [0, P] gives every
 *               row of the request SV_REQ_BAD_DRAFT_LEN and no record.
 *   out_ids     [B, P, k] int32: the tokens of the k largest logits, in
 *               descending order, equal logits (-0.0 == +0.0) by ascending
 *               token; only finite logits are kept, -1 past the last of them.
 *   out_logits  [B, P, k] fp32: their logits (exact), -inf past the last.
 *   out_lse     [B, P] fp32: log sum_j exp(l_j / T); -inf for a row that is
 *               not read or has no finite logit.
 *   out_status  [B, P] int32 or NULL: SV_REQ_* bits per row.  A row with NaN or
 *               +inf (SV_REQ_BAD_LOGITS), or with a wait that ran out
 *               (SV_REQ_TIMEOUT), has no record (-1, -inf) and lse NaN.
 *   B, P, V     0 <= B <= SV_MAX_B, P >= 1, B * P <= SV_MAX_ROWS, 1 <= V <= SV_MAX_V.
 * No workspace: a call keeps nothing, so calls may overlap on any streams. */
sv_status spec_top_logits(const void* logits, int k, float temperature, const int32_t* lens,
                          int32_t* out_ids, float* out_logits, float* out_lse,
                          int32_t* out_status, sv_dtype dtype, int B, int P, int V,
                          sv_stream_t stream);

/* Distillation of a draft model from a teacher's top logits: the divergence
 * KL(p || q) of each row, and its gradient by the student's logits.
 *
 * With a record (ids, t_j) of a row, T the temperature, x = s / T the
 * student's tempered logits and q = softmax(x):
 *   top_lse given (L, the teacher's log-sum-exp at the same T): p_j =
 *     exp(t_j / T - L) on the recorded tokens, and every other token in one
 *     bucket of p_rest = max(0, 1 - sum p_j) against q_rest, the student's mass
 *     outside the record:
 *       loss = sum_j p_j (log p_j - log q_j) + p_rest (log p_rest - log q_rest)
 *     (a record of all V tokens has no rest);
 *   top_lse NULL: p is the softmax of t / T over the record alone and
 *       loss = sum_j p_j (log p_j - log q_j).
 *   gradient by s_i: (P q_i - p_i) / T on recorded tokens, elsewhere
 *     (P q_i - p_rest q_i / q_rest) / T, each times grad_loss of the row, where
 *     P = sum_j p_j + p_rest: 1, or the record's own mass where that is more than
 *     top_lse leaves room for or the record holds all V tokens.
 * A term with p = 0 is 0.  A recorded token with p_j > 0 whose student logit is
 * -inf gives loss +inf (the gradient stays finite), and so does p_rest > 0 where
 * the student is -inf on every token outside the record; there a p_rest of up to
 * 2^-20 + 2^-23 |top_lse|, the rounding of a record that holds all of the
 * teacher's mass (rows masked to fewer tokens than k), counts as 0.
 *
 *   student_logits [B, P, V] dtype, V * sizeof(logit) <= SV_MAX_DISTILL_ROW.
 *   top_ids     [B, P, k] int32: distinct tokens in [0, V); -1 marks an unused
 *               entry.  A row without a used entry has loss 0 and gradient 0.
 *   top_logits  [B, P, k] fp32: finite, or -inf (p_j = 0).
 *   top_lse     [B, P] fp32 or NULL.
 *   lens        [B] int32 or NULL: rows i >= lens[b] are not read; their loss and
 *               gradient are 0.  lens[b] outside [0, P]: SV_REQ_BAD_DRAFT_LEN.
 *   grad_loss   [B, P] fp32 or NULL: with it the call also writes out_grad, the
 *               gradient of sum(grad_loss * loss), reading the student once.
 *   out_loss    [B, P] fp32.
 *   out_stats   [B, P, 4] fp32 (16-byte aligned) or NULL: what spec_distill_grad
 *               needs of this call.
 *   out_grad    [B, P, V] dtype: written when grad_loss is given (every row).
 *               It may be student_logits itself, and overlap it in no other way;
 *               the other outputs must not overlap grad_loss (SV_ERR_ALIAS), and no
 *               output any other input.
 *   out_status  [B, P] int32 or NULL: SV_REQ_BAD_LOGITS (student NaN, +inf or no
 *               finite logit; a used entry's logit NaN or +inf, or a top_lse beside
 *               it that is not finite or so far below them that sum_j p_j is not,
 *               or without one no finite logit),
 *               SV_REQ_BAD_TOKEN (a token outside [-1, V) or
 *               given twice), SV_REQ_BAD_DRAFT_LEN, SV_REQ_TIMEOUT.  Such a row has
 *               loss NaN and gradient 0.
 *   k, B, P, V, temperature: as in spec_top_logits.  No workspace. */
sv_status spec_distill(const void* student_logits, const int32_t* top_ids,
                       const float* top_logits, const float* top_lse, const int32_t* lens,
                       const float* grad_loss, float temperature, float* out_loss,
                       float* out_stats, void* out_grad, int32_t* out_status, sv_dtype dtype,
                       int B, int P, int V, int k, sv_stream_t stream);

/* The backward pass of spec_distill alone: out_grad [B, P, V] = the gradient
 * of sum(grad_loss * loss), from the out_stats of a spec_distill call with the
 * same student_logits, record, lens and temperature.  Rows with a data error
 * there have gradient 0; a part of a row whose wait for staged logits ran out
 * here has gradient NaN. */
sv_status spec_distill_grad(const void* student_logits, const int32_t* top_ids,
                            const float* top_logits, const float* top_lse, const int32_t* lens,
                            const float* stats, const float* grad_loss, float temperature,
                            void* out_grad, sv_dtype dtype, int B, int P, int V, int k,
                            sv_stream_t stream);

/* One step of beam selection: of all continuations (beam w, token v) of a
 * request, the n of largest score
 *     scores[b, w] + l[b, w, v] - log sum_j exp(l[b, w, j]),
 * in descending order.  Equal scores go by ascending beam; a beam's tokens whose
 * scores are equal (by rounding: a score of -1e30 swallows every difference of
 * logits) by descending logit, and of equal logits by ascending token.  With a
 * draft model's logits each call is one level of a candidate tree (the kept
 * (parent, token) pairs are its nodes) for spec_verify_tree and its kin.
 *
 *   logits      [B, W, V] dtype.
 *   scores      [B, W] fp32: each beam's score so far; -inf marks a finished
 *               beam, whose row is not read.  At the first step all beams but one
 *               are -inf.
 *   out_tokens, out_parents [B, n] int32: token v and beam w of each kept
 *               candidate; out_scores [B, n] fp32.  Candidates have finite logits; past
 *               the last one the slots hold -1, -1 and -inf.
 *   out_status  [B] int32 or NULL: SV_REQ_BAD_LOGITS when a live beam's row has NaN
 *               or +inf, or a score is NaN or +inf, SV_REQ_TIMEOUT when a wait of
 *               its rows ran out; nothing is kept then.
 *   1 <= W <= SV_MAX_BEAMS, 1 <= n <= SV_MAX_TOP, 0 <= B <= SV_MAX_B, and
 *   ceil(W / 8) * ceil(V / 8192) <= 256 (V <= 2097152 up to 8 beams, 262144 with
 *   64).  Scores are compared in 64 bits (their row sums are of 32-bit terms).
 *   workspace   >= spec_beam_workspace_size(dtype, B, W, V, n) bytes (0 for small
 *               calls), 16-byte aligned; SV_ERR_WORKSPACE otherwise.  It needs no
 *               preparation and holds nothing between calls; calls that may
 *               overlap need one each. */
size_t spec_beam_workspace_size(sv_dtype dtype, int B, int W, int V, int n);
sv_status spec_beam_select(const void* logits, const float* scores, int32_t* out_tokens,
                           int32_t* out_parents, float* out_scores, int32_t* out_status,
                           sv_dtype dtype, int B, int W, int V, int n, void* workspace,
                           size_t ws_bytes, sv_stream_t stream);

/* Reordering of per-beam states: out[g, b, w, h, l] = state[g, b, parents[b, w],
 * h, l] for l < lens[b], each entry a run of row_bytes contiguous bytes.  It
 * moves a draft model's states (hidden states, keys and values, block tables)
 * along a beam selection's parents, and gathers the accepted path's entries out
 * of a candidate tree's (parents = out_path of a tree call, which names node ids).
 *
 *   state       G x B x W x H x L entries at byte strides state_strides[5].
 *   out         G x B x W_out x H x L entries at byte strides out_strides[5].
 *               Strides are >= 0 and may come in any order (heads before or after
 *               beams); entries of `out` must not overlap each other, nor entries
 *               of state (SV_ERR_ALIAS); the two may be interleaved parts of one
 *               allocation.
 *   parents     [B, W_out] int32: -1 leaves the slot as it is.
 *   lens        [B] int32 or NULL (all L): entries l >= lens[b] of out are left as
 *               they are.
 *   out_status  [B] int32 or NULL: SV_REQ_BAD_TREE for a parent outside [-1, W)
 *               (its slot is left as it is), SV_REQ_BAD_DRAFT_LEN for lens[b] outside
 *               [0, L] (nothing is moved).
 * Every extent but row_bytes may be 0.  B <= SV_MAX_B, W and W_out < 65536; G,
 * H, L and row_bytes < 2^31.  No workspace. */
sv_status spec_beam_reorder(const void* state, const int64_t* state_strides,
                            const int32_t* parents, const int32_t* lens, void* out,
                            const int64_t* out_strides, int32_t* out_status, int G, int B, int W,
                            int W_out, int H, int L, int row_bytes, sv_stream_t stream);

/* A key/value cache held in 4 bits, for the layer that scores a step's tokens.
 *
 * The cache is `pages` pages of page_size tokens, each token's keys and values of
 * every head quantised in groups of 32 values: a scale byte c stands for
 *     s = (1 + (c mod 8) / 8) * 2^(floor(c / 8) - 20),   c = 0..238 (s up to 896),
 * the least with 7 s >= the group's largest magnitude, and each value for the nearest
 * whole multiple q of s, ties to even, q = -7..7 (magnitudes above 7 * 896 = 6272
 * become 6272).  A token of which a head's keys or values hold NaN or infinity reads
 * back as NaN throughout that head, and attention rows that see it are NaN there.
 *
 *   cache       `pages` pages, page_stride bytes apart (a multiple of 16 below
 *               2^32; the layers of a model may be interleaved), 16-byte aligned.  A page is
 *               [kv_heads, 2 (keys, values), spec_cache_page_bytes]: for each
 *               head, page_size rows of head_dim / 2 code bytes, then scale bytes
 *               [page_size / 16, head_dim / 32, 16 (tokens)].  A row is
 *               little-endian words of 8 values, value i's q + 8 in bits
 *               4 (i / 2 + 4 (i mod 2)) onwards.
 *   table       [B, M] int32: the pages of request b's slots 0 .. M * page_size - 1.
 *               A page that is written belongs to one request; pages that are
 *               only read (a shared prefix) may occur in any number of rows.
 *               Entries whose slots a call does not touch are not read.
 *   start       [B] int32: the first slot of the request that the call touches.
 *   page_size   16, 32, 64, 128 or 256; head_dim 64, 128 or 256; M * page_size <=
 *               SV_MAX_SLOTS, kv_heads <= SV_MAX_HEADS, 0 <= B <= SV_MAX_B.
 *   out_status  [B] int32 or NULL: SV_REQ_BAD_DRAFT_LEN (slots or lengths out of
 *               range: nothing is done for the request), SV_REQ_BAD_PAGE (tokens
 *               on such pages are skipped; attention rows that would see them are NaN).
 * Calls need no workspace unless they name one, and no result depends on what the cache
 * holds beyond the slots in use. */

/* Bytes of a page of one head's keys (or values); 0 when not supported. */
size_t spec_cache_page_bytes(int page_size, int head_dim);

/* Writes tokens: request b's token i < lens[b] (NULL: N) goes to slot start[b] + i.
 *
 *   k, v        [B, N, kv_heads, head_dim] dtype at byte strides k_strides[3],
 *               v_strides[3] of b, n and h (>= 0, multiples of 16, 16-byte aligned; each
 *               row of head_dim values contiguous).
 * 0 <= N <= SV_MAX_SLOTS, B * N * kv_heads < 2^31. */
sv_status spec_cache_write(void* cache, int64_t page_stride, const void* k,
                           const int64_t* k_strides, const void* v, const int64_t* v_strides,
                           const int32_t* table, const int32_t* start, const int32_t* lens,
                           int32_t* out_status, sv_dtype dtype, int pages, int page_size, int B,
                           int N, int M, int kv_heads, int head_dim, sv_stream_t stream);

/* Reads tokens back: k[b, i] and v[b, i] of slot start[b] + i (NULL: slot i) for
 * i < lens[b] (NULL: N); the other rows are left as they are, or with fill != 0 set to 0.
 * Every value is exact in either type.  k and v as in spec_cache_write; rows of one must not overlap each
 * other (SV_ERR_ALIAS), nor the other's or the cache. */
sv_status spec_cache_read(const void* cache, int64_t page_stride, void* k,
                          const int64_t* k_strides, void* v, const int64_t* v_strides,
                          const int32_t* table, const int32_t* start, const int32_t* lens,
                          int fill, int32_t* out_status, sv_dtype dtype, int pages, int page_size,
                          int B, int N, int M, int kv_heads, int head_dim, sv_stream_t stream);

/* Keeps the accepted path of a tree whose nodes lie in slots start[b] + node: slot
 * start[b] + path[b, i] moves to start[b] + i, for the entries before the first -1
 * (path = out_path of a tree call).  The request then has start[b] + accept_len
 * tokens.  Entries must ascend from 0 or above: SV_REQ_BAD_TREE otherwise, and nothing is
 * moved for the request.  0 <= P <= SV_MAX_STEP. */
sv_status spec_cache_keep(void* cache, int64_t page_stride, const int32_t* table,
                          const int32_t* start, const int32_t* path, int32_t* out_status,
                          int pages, int page_size, int B, int P, int M, int kv_heads,
                          int head_dim, sv_stream_t stream);

/* Attention of a step's tokens over the cache, which holds them already ("推测解码与
 * MTP" §3.3 "Tree Attention": a node sees its ancestors only).  Request b's token i < n
 * (n = q_lens[b], NULL: N) is in slot base + i, base = lens[b] - n, and
 *     out[b, i, h] = sum_j w_j v_j / sum_j w_j,  w_j = exp(x_j),
 *     x_j = c(scale * q . k_j) - slopes[h] * (at_i - at_j),
 * over the slots j that it sees, c(x) = softcap * tanh(x / softcap) or x itself.  It sees
 * every slot before base; of the step's own, those up to itself, or in a tree
 * its ancestors and itself.  A slot's position at_j is j before base, base + i for
 * the i-th token of a chain, base + depth for a tree's node.  With a window, only
 * slots with at_i - at_j < window are seen.
 *
 *   q           [B, N, q_heads, head_dim] dtype at byte strides q_strides[3] as of
 *               k; q_heads a multiple of kv_heads, heads in groups of q_heads /
 *               kv_heads to a key/value head; 0 <= N <= SV_MAX_STEP.
 *   lens        [B] int32: slots in use, the step's own among them.  lens[b]
 *               outside [n, M * page_size] or q_lens[b] outside [0, N]:
 *               SV_REQ_BAD_DRAFT_LEN, and the request's rows are 0.
 *   tree_parent, parent_stride (0 or N - 1): as in spec_verify_tree for a tree of
 *               N - 1 candidate nodes, n - 1 of them in use; NULL: a chain.  No tree:
 *               SV_REQ_BAD_TREE, and the request's rows are 0.
 *   slopes      [q_heads] fp32 or NULL (no bias).
 *   scale       finite.  softcap up to 1e30, 0: none.  window 0: none.
 *               Scores and the parts that they are made of, |scale| max |q| of a row among
 *               them, are to stay below 2^127: other rows have no defined values.
 *   out         [B, N, q_heads, head_dim] dtype, contiguous, 16-byte aligned; rows
 *               behind q_lens[b] are left as they are.  It must not reach into the bytes
 *               from q's first to its last (SV_ERR_ALIAS), nor into other inputs.
 *   out_lse     [B, N, q_heads] fp32 or NULL: log sum_j exp(x_j).
 *   workspace   >= spec_cache_attention_workspace_size bytes (of the current
 *               device), 16-byte aligned.  It needs no preparation and holds nothing
 *               between calls; calls that may overlap need one each.
 * Sums are of 32-bit terms; weights are rounded to 11 bits before they meet the
 * values (22 bits in fp32).  The tensor cores cut the sums of weighted values off, by about
 * 2^-24 of them for every 16 slots that a warp (more than 16 query rows: a block) adds up: up to
 * 2^-10 of a bf16 result over 2^17 slots that one block has for itself, 2^-8 over 2^19; some 2^-17 in
 * fp32, whatever the length.  Results do not vary between calls of the same lengths.
 * There is no backward pass.
 * bf16 calls of more than 16 query rows a key/value head (N * q_heads / kv_heads) and a
 * head_dim of 64 or 128 wait for the tensor cores, each time no longer than the limit of
 * spec_verify_set_wait_limit_ns: a wait that ran out makes rows NaN and sets SV_REQ_TIMEOUT
 * in every request's status. */
size_t spec_cache_attention_workspace_size(sv_dtype dtype, int N, int q_heads, int kv_heads,
                                           int head_dim);
sv_status spec_cache_attention(const void* q, const int64_t* q_strides, const void* cache,
                               int64_t page_stride, const int32_t* table, const int32_t* lens,
                               const int32_t* q_lens, const int32_t* tree_parent,
                               int parent_stride, const float* slopes, float scale, float softcap,
                               int window, void* out, float* out_lse, int32_t* out_status,
                               sv_dtype dtype, int pages, int page_size, int B, int N, int M,
                               int q_heads, int kv_heads, int head_dim, void* workspace,
                               size_t ws_bytes, sv_stream_t stream);

/* Allocation-free variant of spec_verify_sample.  The pages have no
 * counterpart to this entry point; it exists for callers that cannot
 * allocate device memory - for example an inference runtime that reserves the
 * whole device for its own pool and hands a plugin only its input and output
 * buffers, or a path on which a cudaMalloc (which may synchronise the device)
 * is not allowed.
 *
 * Arguments and results are those of spec_verify_sample, without the
 * workspace.  Its scratch is one fixed device array of
 * SV_NOALLOC_SCRATCH_BYTES inside the library, held by every GPU that loads
 * the library until the process exits; the call itself allocates nothing.
 *   - Limit: spec_verify_workspace_size(B, K, V) must not exceed
 *     SV_NOALLOC_SCRATCH_BYTES; larger problems return SV_ERR_WORKSPACE with
 *     nothing queued.  (B = 256, K = 5, V = 152064 needs about 3.4 MB.)
 *   - Each call looks up the array's device address on the current device
 *     (cudaGetSymbolAddress; it queues no work, and a device reset that
 *     reloads the module cannot leave a stale address behind).  The first
 *     call on a device may load the library's module there: make that first
 *     call before any stream capture.
 *   - Every call on a device uses the same array, which keeps the previous
 *     call's contents; each call first clears, on its stream, the counters
 *     that must start at zero.  Calls that overlap on the GPU (different
 *     streams, or different host threads without ordering) race on the
 *     array and give wrong results: order them on one stream. */
#define SV_NOALLOC_SCRATCH_BYTES (8u << 20)
sv_status spec_verify_sample_noalloc(const void* target_logits, const void* draft_logits,
                                     const int32_t* draft_tokens, const float* uniforms,
                                     float temperature, int32_t* out_tokens,
                                     int32_t* out_accept_len, sv_dtype dtype, int B, int K, int V,
                                     const int32_t* draft_lens, int32_t* out_cu_accept,
                                     int32_t* out_packed, int32_t* out_batch_id,
                                     float* out_accept_prob, int32_t* out_status,
                                     sv_stream_t stream);

/* Human-readable name of a status code (static storage). */
const char* spec_verify_status_string(sv_status status);

/* Library ABI version: 100 * major + minor. */
int spec_verify_version(void);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_VERIFY_H_ */

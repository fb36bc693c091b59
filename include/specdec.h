/*
 * specdec.h -- C ABI of the GB300 (sm_103a) speculative-decoding verification library.
 *
 * The library implements the verification step of speculative decoding: it turns
 * the target model's logits and the drafter's distributions into accepted tokens.
 * Sources, cited by page title and section:
 *   "Speculative decoding" (zerotofrontier.app, Chapter 20, Section 20.5)      -- SD 20.5
 *   "Speculative-Decoding / Medusa" (s1mplewind.github.io)                    -- Medusa notes
 *   "Speculative Decoding: The Art of Guessing Well" (astralord.github.io)    -- Art of Guessing
 *
 * Conventions shared by every entry point
 *   - Array arguments are caller-owned DEVICE pointers to contiguous row-major arrays;
 *     the library never allocates, frees or retains them.  Sizes are element counts.
 *   - `stream` is a cudaStream_t passed as void* (NULL = the legacy default stream).
 *     Every call is asynchronous on `stream`; the caller synchronises before reading
 *     outputs.  Work is launched only on `stream`.
 *   - The return code covers host-side validation and launch errors only:
 *       SPECDEC_OK, SPECDEC_ERR_INVALID_ARG (a null required pointer, a non-positive
 *       size, an unknown dtype, misaligned workspace), SPECDEC_ERR_UNSUPPORTED (sizes the
 *       kernels do not handle), SPECDEC_ERR_CUDA (a launch failed), SPECDEC_ERR_WORKSPACE
 *       (workspace smaller than the matching *_workspace_bytes()).  On a non-OK return
 *       nothing was launched, except for SPECDEC_ERR_CUDA.
 *   - Problems in the DATA are reported per sequence in `out_status` (bit flags below).
 *     A sequence with any error bit set gets num_accepted = -1 and all its tokens -1.
 *     Warning bits leave the outputs valid.
 *   - Temperatures below SPECDEC_GREEDY_TEMPERATURE (including 0 and negatives) select
 *     greedy verification for that sequence (SD 20.5, "A round of greedy speculative
 *     decoding"; the special case "A greedy target" of the sampling rule).
 *   - Deterministic: the same inputs give bit-identical outputs on every call.
 *   - Workspaces: a call's workspace must hold at least the size the matching
 *     *_workspace_bytes() returns and be 256-byte aligned.  Its contents need no
 *     preparation: each call clears the counters it uses on its stream first.  One
 *     workspace can serve calls of any shape that fits, one call at a time; calls that
 *     overlap on the GPU must not share a workspace.
 */
#ifndef SPECDEC_H
#define SPECDEC_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  SPECDEC_F32 = 0,
  SPECDEC_BF16 = 1,
  SPECDEC_F16 = 2, /* the cache calls: queries, keys, values and 16-bit pages */
  SPECDEC_KV4 = 3, /* the cache calls: pages held in 4 bits                    */
  SPECDEC_KV8 = 4  /* the cache calls: pages held in 8 bits                    */
} specdec_dtype;

/* return codes */
#define SPECDEC_OK 0
#define SPECDEC_ERR_INVALID_ARG 1
#define SPECDEC_ERR_UNSUPPORTED 2
#define SPECDEC_ERR_CUDA 3
#define SPECDEC_ERR_WORKSPACE 4
#define SPECDEC_ERR_TOO_LARGE 5   /* the shape needs more scratch than the built-in array */

/* per-sequence status bits (errors: low byte; warnings: above) */
#define SPECDEC_STATUS_BAD_LOGIT 1          /* NaN or +inf logit in a row the call reads      */
#define SPECDEC_STATUS_EMPTY_ROW 2          /* a row whose logits are all -inf                */
#define SPECDEC_STATUS_BAD_TOKEN 4          /* draft / node token outside [0, V)              */
#define SPECDEC_STATUS_BAD_PROB 8           /* draft probability NaN, inf or negative         */
#define SPECDEC_STATUS_BAD_UNIFORM 16       /* uniform outside [0, 1) on a sampled sequence   */
#define SPECDEC_STATUS_BAD_TREE 32          /* parent not in [-1, i), or tree deeper than D   */
#define SPECDEC_STATUS_BAD_TEMPERATURE 64   /* temperature NaN or infinite                    */
#define SPECDEC_STATUS_TIMEOUT 128          /* a bounded wait inside a kernel gave up: not finished */
#define SPECDEC_STATUS_BAD_CACHE 32         /* cache calls: a length or page out of range (the bit
                                               with which a path that leaves the cache is reported) */
#define SPECDEC_STATUS_BAD_PENALTY 64       /* logits processing: a penalty that is not a number it takes */
#define SPECDEC_STATUS_ERROR_MASK 0xFF
#define SPECDEC_STATUS_ZERO_Q 256           /* warning: q_i(x_i) == 0; accepted iff p_i(x_i) > 0 */
#define SPECDEC_STATUS_ZERO_RESIDUAL 512    /* warning: residual mass 0 after rounding; drew from p */

#define SPECDEC_GREEDY_TEMPERATURE 1e-3f

/* ------------------------------------------------------------------------------------
 * Chain verification: one round of speculative sampling per sequence.
 *
 * SD 20.5, "A round of speculative sampling" (Leviathan et al. Alg. 1) and the exercise
 * "Verify one round of speculative sampling"; Art of Guessing, "Speculative sampling".
 * For sequence b with temperature T = temperatures[b] >= SPECDEC_GREEDY_TEMPERATURE:
 *   p_i = softmax(logits[b, i, :] / T), i = 0..g
 *   draft i is accepted iff uniforms[b, i] * q_i(x_i) < p_i(x_i)   (u < p/q, min(1, .) implicit)
 *   J = number of leading accepted drafts
 *   the extra token y is the inverse-CDF draw with u = uniforms[b, g] from
 *   (p_J - q_J)+ (normalised), where q_g == 0 so that J == g draws the bonus from p_g:
 *   y = smallest k with C_k > u * S, C the running sum and S the total of the weights.
 * Greedy sequences accept while x_i == argmax_k logits[b, i, k] (lowest index on ties)
 * and emit the argmax of row J; draft_probs and uniforms are not read for them.
 *
 * logits          [B, g+1, V]  fp32 or bf16 (ldt)          row i: target after x_0..x_{i-1}
 * draft_probs     [B, g, V]    fp32, the distribution each draft was sampled from, as given
 * draft_tokens    [B, g]       int32
 * temperatures    [B]          fp32
 * uniforms        [B, g+1]     fp32 in [0, 1): slot i tests draft i, slot g drives y
 * out_tokens      [B, g+1]     int32: x_0..x_{J-1}, y, then -1
 * out_num_accepted[B]          int32: J (or -1 on a data error)
 * out_p_draft     [B, g]       fp32, optional (NULL): p_i(x_i) for i <= J; NaN after J,
 *                              for greedy sequences and on a data error
 * out_status      [B]          int32, optional (NULL): status bits
 * Positions are evaluated left to right, as the round itself runs: row i (its logits,
 * draft token, q_i(x_i) and uniform) counts only if drafts 0..i-1 were all accepted,
 * and the first data error or rejection ends the scan.  Rows after J therefore neither
 * change the outputs nor are validated (the default kernel does not read them at all),
 * and status bits describe rows 0..J plus uniforms[b, g] and q row J where the draw
 * uses them.  A non-finite temperature is an error whatever the rows hold.
 * Sizes: B >= 1, g >= 1, V >= 1, V < 2^31.
 * Host-resident rows: logits and draft_probs may be pinned host memory (cudaHostAlloc, or
 * registered with cudaHostRegister, mapped at its own address).  The left-to-right kernel
 * then reads only the rows the round needs, straight over the host link (no copy of the
 * whole batch); this needs 16-byte aligned rows, g + 1 <= 32 and V <= 1,048,576 (bf16) or
 * 786,432 (fp32), else SPECDEC_ERR_UNSUPPORTED.  Pageable host memory gives
 * SPECDEC_ERR_INVALID_ARG, and so does a device pointer on a device other than the current
 * one.  The other inputs, the outputs and the workspace are device memory.  The same holds
 * for specdec_verify_greedy and specdec_verify_chain_varlen.
 * Bounded waits: the left-to-right kernel's waits on its queues and copies give up after a
 * bound (one second); a sequence the kernel could not finish then comes back with
 * SPECDEC_STATUS_TIMEOUT, num_accepted -1 and tokens -1 (out_p_draft NaN).  The kernel
 * does not need its whole grid resident at once: while kernels on other streams hold SMs,
 * the part that is running takes every sequence in turn, and no running part waits on one
 * that has not started, so sharing the GPU slows a call but does not time it out.
 */
size_t specdec_chain_workspace_bytes(int B, int g, int V, specdec_dtype ldt);

/* Workspace for host-resident logits: specdec_chain_workspace_bytes plus room for one
 * device copy of a logits row per sequence (B * V * element size, rounded up to 256
 * bytes).  Given a workspace at least this large, with logits in pinned host memory, the
 * left-to-right kernel also writes each row it streams for a sequence's chain into that
 * sequence's copy, and a draw from that row (the residual at a rejection, or the bonus
 * row) reads the copy from device memory instead of reading the row a second time over
 * the host link.  A smaller workspace (at least specdec_chain_workspace_bytes) gives the
 * same results and reads drawn rows from the host again.  Device-resident logits, and
 * greedy-only calls, never use the copy.  The same sizes serve
 * specdec_verify_chain_varlen.  Returns 0 for invalid sizes or dtype. */
size_t specdec_chain_host_workspace_bytes(int B, int g, int V, specdec_dtype ldt);

int specdec_verify_chain(const void* logits, specdec_dtype ldt, const float* draft_probs,
                         const int32_t* draft_tokens, const float* temperatures,
                         const float* uniforms, int B, int g, int V, int32_t* out_tokens,
                         int32_t* out_num_accepted, float* out_p_draft, int32_t* out_status,
                         void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------------------
 * Chain verification with a per-request number of verified drafts (SD 20.5, "Choosing how
 * much to verify at every step": adaptive verification verifies l_r drafts of request r).
 *
 * The arguments of specdec_verify_chain, padded to g drafts, plus gammas [B] int32 with
 * 0 <= gammas[b] <= g: sequence b's round is the chain round on its first gammas[b] + 1
 * rows -- drafts 0..gammas[b]-1 tested with uniforms[b, 0..gammas[b]-1], the extra token
 * from row J (a rejection's residual, or the bonus row gammas[b]) with uniforms[b,
 * gammas[b]].  Rows, q rows and uniforms past gammas[b] are not read; out_tokens are -1
 * past J, out_p_draft NaN past J.  A count outside [0, g] gives SPECDEC_STATUS_BAD_TOKEN.
 * Exactness needs each count chosen without looking at the drafts it decides on (the
 * page's non-anticipating requirement, box "Trimming a draft can break exactness"); the
 * verifier cannot check it.  Needs 16-byte aligned rows, g + 1 <= 32 and V <= 1,048,576 (bf16)
 * or 786,432 (fp32) (the left-to-right kernel), else SPECDEC_ERR_UNSUPPORTED.  Workspace:
 * specdec_chain_workspace_bytes.
 */
int specdec_verify_chain_varlen(const void* logits, specdec_dtype ldt, const float* draft_probs,
                                const int32_t* draft_tokens, const float* temperatures,
                                const float* uniforms, const int32_t* gammas, int B, int g, int V,
                                int32_t* out_tokens, int32_t* out_num_accepted, float* out_p_draft,
                                int32_t* out_status, void* workspace, size_t workspace_bytes,
                                void* stream);

/* ------------------------------------------------------------------------------------
 * Block verification: one round per sequence, the draft judged jointly.
 *
 * Art of Guessing, "Block verification" (Sun et al.).  Same inputs, outputs and shapes as
 * specdec_verify_chain.  For a sampled sequence (T >= SPECDEC_GREEDY_TEMPERATURE), with
 * p_k = softmax(logits[b, k, :] / T) and q_k = draft_probs[b, k, :]:
 *   w_0 = 1, w_{k+1} = min(1, w_k * p_k(x_k) / q_k(x_k))       (q(x) = 0: ratio +inf, or 0
 *                                                              when p(x) = 0; 0 * inf = 0)
 *   mass_k = sum_v (w_k p_k(v) - q_k(v))+ (k < g), mass_g = w_g
 *   survival_k = mass_k / (mass_k + 1 - w_k) if w_k < 1, else 1
 *   prefix length k (1..g) survives iff uniforms[b, k-1] <= survival_k
 *   n = the longest surviving prefix (0 if none): out_num_accepted[b]
 *   the extra token is the inverse-CDF draw with uniforms[b, g] from (w_n p_n - q_n)+
 *   (q_g == 0): y = smallest v with C_v > u * S.  out_tokens = x_0..x_{n-1}, y, -1...
 * Greedy sequences are verified exactly as by specdec_verify_greedy (a one-hot target
 * reduces the rule to argmax matching).  The rule reads every row, every draft, every
 * q row and every uniform, so all are validated and every error found is reported
 * (status bits OR'd); an error gives J = -1, tokens -1 and p_draft NaN.  out_p_draft[b, k]
 * = p_k(x_k) for every k of a clean sampled sequence.  Warnings: SPECDEC_STATUS_ZERO_Q
 * (some q_k(x_k) == 0), SPECDEC_STATUS_ZERO_RESIDUAL (the residual of row n summed to 0
 * after rounding; the token is drawn from p_n).
 * Layout requirement: every logits row and q row starts on a 16-byte boundary (V * elem
 * size and V * 4 multiples of 16, bases aligned) and g + 1 <= 32; other shapes return
 * SPECDEC_ERR_UNSUPPORTED.  Sizes: B >= 1, g >= 1, V >= 1.
 */
size_t specdec_block_workspace_bytes(int B, int g, int V, specdec_dtype ldt);

int specdec_verify_block(const void* logits, specdec_dtype ldt, const float* draft_probs,
                         const int32_t* draft_tokens, const float* temperatures,
                         const float* uniforms, int B, int g, int V, int32_t* out_tokens,
                         int32_t* out_num_accepted, float* out_p_draft, int32_t* out_status,
                         void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------------------
 * Greedy verification (SD 20.5, "A round of greedy speculative decoding"; Art of
 * Guessing, "Draft and verify"): z_i = argmax logits[b, i, :] (lowest index on ties),
 * J = longest prefix with x_i == z_i, emit x_0..x_{J-1}, z_J.  Shapes as for the chain
 * call.  Every sequence is greedy whatever its temperature would be.
 */
size_t specdec_greedy_workspace_bytes(int B, int g, int V, specdec_dtype ldt);

int specdec_verify_greedy(const void* logits, specdec_dtype ldt, const int32_t* draft_tokens,
                          int B, int g, int V, int32_t* out_tokens, int32_t* out_num_accepted,
                          int32_t* out_status, void* workspace, size_t workspace_bytes,
                          void* stream);

/* ------------------------------------------------------------------------------------
 * Medusa tree verification: a walk of a candidate tree per sequence.
 *
 * Medusa notes, section "Attention Tree": at the current node the target draws a token
 * (inverse CDF of softmax(logits / T) with uniforms[b, d] at depth d, or the argmax for a
 * greedy sequence); if a child of the node carries that token the walk appends it and
 * descends, otherwise it emits the token and stops.  SD 20.5 gives the greedy walk after
 * the exercise "The tree attention mask".  Among children carrying the same token the
 * lowest node index is taken.
 *
 * logits        [B, N+1, V]  row 0: after the committed prefix (the root); row 1+i: after node i
 * node_tokens   [B, N]       int32
 * parents       [N]          int32, shared by the batch, parents[i] in [-1, i)
 * temperatures  [B]          fp32
 * uniforms      [B, D+1]     fp32 in [0, 1), D = max_depth
 * out_tokens    [B, D+1]     int32: the accepted node tokens then the final draw, -1 padded
 * out_path      [B, D]       int32: node ids of the accepted path, -1 padded
 * out_num_accepted [B]       int32: accepted nodes (or -1 on a data error)
 * out_status    [B]          int32, optional
 * max_depth D bounds the number of nodes on any root path (SPECDEC_STATUS_BAD_TREE if a
 * path is longer).  Only the rows the walk visits are read.  N >= 0, 1 <= D <= 64.
 */
size_t specdec_tree_workspace_bytes(int B, int N, int V, int max_depth, specdec_dtype ldt);

int specdec_verify_tree(const void* logits, specdec_dtype ldt, const int32_t* node_tokens,
                        const int32_t* parents, const float* temperatures, const float* uniforms,
                        int B, int N, int V, int max_depth, int32_t* out_tokens,
                        int32_t* out_path, int32_t* out_num_accepted, int32_t* out_status,
                        void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------------------
 * Sampled tree verification by recursive rejection (SD 20.5, box "Recursive rejection at
 * a node with several children"; the multi-step speculative sampling of SpecInfer).
 *
 * At the current node, whose children s_1..s_k were drafted independently from q, start
 * from R_1 = p = softmax(logits / T) at the node; try the children in node-index order:
 * accept s_i when uniforms[b, 1 + s_i's node id] * q(s_i) < R_i(s_i) and move to it;
 * otherwise R_{i+1} = (R_i - q)+ normalised and try the next child.  When every child is
 * rejected (or the node is a leaf) the extra token is the inverse-CDF draw of
 * uniforms[b, 0] from the last R (smallest v with C_v > u * S) and the walk ends.  The
 * emitted tokens follow the target exactly when every node's children are independent
 * draws from that node's q.  A greedy sequence descends into the lowest-index child
 * carrying the argmax and emits the argmax where none does.
 *
 * logits        [B, N+1, V]  row 0: after the committed prefix (the root); row 1+i: after node i
 * draft_probs   [B, N+1, V]  fp32: row 0: the distribution the root's children were drafted
 *                            from; row 1+i: node i's children's (leaf rows are not read)
 * node_tokens   [B, N]       int32
 * parents       [N]          int32, shared by the batch, parents[i] in [-1, i)
 * temperatures  [B]          fp32
 * uniforms      [B, N+1]     fp32 in [0, 1): slot 1+j tests node j, slot 0 the final draw
 * out_tokens    [B, D+1]     int32: the accepted node tokens then the final draw, -1 padded
 * out_path      [B, D]       int32: node ids of the accepted path, -1 padded
 * out_num_accepted [B]       int32: accepted nodes (or -1 on a data error)
 * out_status    [B]          int32, optional: the tree, every token, T and (sampled) every
 *                            uniform are checked first; then, along the walk, each visited
 *                            row (BAD_LOGIT, EMPTY_ROW), q(s) of each tried child and a q
 *                            row read whole at its node's first rejection (BAD_PROB).  An
 *                            error reports error bits only.  Warnings: ZERO_Q (a tried
 *                            child with q(s) = 0: accepted iff R(s) > 0), ZERO_RESIDUAL
 *                            (a residual summed to 0 after rounding; R_i is kept).
 * max_depth D bounds the number of nodes on any root path.  N >= 0, 1 <= D <= 64.  No
 * workspace is needed (specdec_tree_workspace_bytes applies and returns 0).
 *
 * flags: 0, or SPECDEC_TREE_WITHOUT_REPLACEMENT -- the children of every node were drawn
 * without replacement (Sequoia, Chen et al.; SD 20.5, the paragraph after the box's
 * proof): try i uses q_i, q with the tokens of the children already rejected at the node
 * set to zero and renormalised by Z_i = 1 - (q at those tokens), in the test
 * (u * q_i(s_i) < R_i(s_i)) and in the residual (R_{i+1} = (R_i - q_i)+ normalised).
 * When Z_i <= 0 (q's mass is used up) q_i is zero: the try follows the ZERO_Q rule and a
 * rejection leaves R_i.  Children drawn without replacement carry distinct tokens, so
 * two children of one node with the same token are an input error (BAD_TREE).  Other
 * flag bits: SPECDEC_ERR_INVALID_ARG.
 */
#define SPECDEC_TREE_WITHOUT_REPLACEMENT 1
int specdec_verify_tree_recursive(const void* logits, specdec_dtype ldt, const float* draft_probs,
                                  const int32_t* node_tokens, const int32_t* parents,
                                  const float* temperatures, const float* uniforms, int B, int N, int V,
                                  int max_depth, int flags, int32_t* out_tokens, int32_t* out_path,
                                  int32_t* out_num_accepted, int32_t* out_status, void* stream);

/* ------------------------------------------------------------------------------------
 * Gumbel-coupled verification (Art of Guessing, "Gumbel coupling", Daliri et al.).
 *
 * The drafter and the target use the same noise g_k at position k: the drafter proposed
 * x_k = argmax_i (log q_k(i) + g_k,i) (specdec_gumbel_draft below), the target samples
 * t_k = argmax_i (log p_k(i) + g_k,i) with p_k = softmax(logits[b, k, :] / T); the round keeps
 * x_0..x_{n-1} for the first n with x_n != t_n (n = g if none) and appends t_n.  The emitted
 * tokens are what the target alone samples with that noise, whatever the drafter.
 *
 * Noise: Philox4x32-10 (Salmon et al., SC 2011).  Entries 4j..4j+3 of row k of sequence b
 * use the outputs of counter (j, k, b, 0) under key (seed & 0xffffffff, seed >> 32); an
 * output x gives u = ((x >> 9) + 0.5) / 2^23.  Race in log2 units, float32:
 * score_i = a_i - log2(xi_i), xi_i = -log1p(u_i - 1), a_i = logit_i * log2(e) / T (target) or
 * log2(q_i) (drafter); ties go to the lowest index.  A greedy sequence (T < 1e-3) uses the
 * plain argmax of the logits.
 *
 * logits [B, g+1, V] (bf16/fp32), draft_tokens [B, g] int32, temperatures [B] fp32.
 * out_tokens [B, g+1] int32 (-1 padded), out_num_accepted [B] int32 (n, or -1 on an error),
 * out_status [B] int32 (optional).  Rows are evaluated left to right and the round stops at
 * n: rows after n are neither read nor validated.  Errors: BAD_TEMPERATURE (non-finite T),
 * then in row order BAD_LOGIT / EMPTY_ROW (row k) and BAD_TOKEN (draft k).
 * Sizes: B >= 1, g >= 1, V >= 1, B <= 65535; 16-byte aligned rows (V * element size a
 * multiple of 16, aligned base) take 16-byte loads, others scalar loads.  Workspace:
 * specdec_gumbel_workspace_bytes(B, g) bytes, 256-byte aligned, device memory (rows are
 * evaluated in waves of two across the GPU; the workspace holds each wave's partial races
 * and which rounds are still open).
 */
size_t specdec_gumbel_workspace_bytes(int B, int g);

int specdec_verify_gumbel(const void* logits, specdec_dtype ldt, const int32_t* draft_tokens,
                          const float* temperatures, uint64_t seed, int B, int g, int V,
                          int32_t* out_tokens, int32_t* out_num_accepted, int32_t* out_status,
                          void* workspace, size_t workspace_bytes, void* stream);

/* The drafter's side of Gumbel coupling: out_draft_tokens[b, k] = argmax_i (log q[b, k, i]
 * + g_{k,i}) with the noise above (same seed, counter (j, k, b, 0)).  draft_probs [B, g, V]
 * fp32; entries that are 0 are never chosen, nor are NaN or negative ones (-1 if no entry
 * qualifies). */
int specdec_gumbel_draft(const float* draft_probs, uint64_t seed, int B, int g, int V,
                         int32_t* out_draft_tokens, void* stream);

/* The shared noise itself, for a drafter that runs its race elsewhere:
 * out_noise[(b * rows + k) * V + i] = G = -log2(xi), xi = -ln(u), of entry i at row k of
 * sequence b (the race adds it to a_i).  out_noise [B, rows, V] fp32.  The library evaluates
 * G with its own approximation (absolute error below 4e-6 against the float64 definition). */
int specdec_gumbel_noise(uint64_t seed, int B, int rows, int V, float* out_noise, void* stream);

/* ------------------------------------------------------------------------------------
 * Accepted-branch KV compaction (SD 20.5, "Keeping the caches consistent after a
 * rejection": after a tree round the accepted branch's cache entries, scattered among
 * discarded siblings, are gathered into consecutive slots; a chain only moves a length).
 *
 * Node i of sequence b's candidates sits at logical slot prefix_len[b] + i; for
 * d < num_accepted[b] the entry of node path[b, d] moves to slot prefix_len[b] + d, in place.
 * A slot is row_bytes bytes:
 *   contiguous (block_table == NULL): slot s of sequence b at cache + b * seq_stride +
 *     s * slot_stride, num_slots slots per sequence;
 *   paged: at cache + block_table[b * max_blocks + s / block_size] * block_stride +
 *     (s % block_size) * slot_stride (num_slots = max_blocks * block_size).
 * Call it once per cache tensor (per layer, keys and values, or one call for a fused
 * layout).  path [B, max_depth] int32 (the tree verifier's out_path), num_accepted [B]
 * (its out_num_accepted; a negative count leaves the sequence alone).
 * out_new_len [B] int32 (optional): prefix_len + num_accepted, the entries to keep (the
 * extra token has no entry yet).  out_status [B] (optional): SPECDEC_STATUS_BAD_TREE when
 * a path does not climb the tree (path[d] >= d, strictly increasing) or leaves the cache;
 * that sequence is left alone.  Freeing emptied pages is the allocator's business.
 * 16-byte aligned layouts move 16-byte words, others bytes.  All pointers are device
 * pointers; strides and sizes in bytes.
 * Slots move as the bytes they are and hold their values whole.  SPECDEC_KV8 pages are not such a cache: a code's scale is
 * its block's and stays where it is (specdec_append_kv8 appends their accepted tokens again).
 */
int specdec_compact_kv(void* cache, int64_t row_bytes, int64_t slot_stride, int64_t seq_stride,
                       int64_t num_slots, const int32_t* block_table, int block_size, int max_blocks,
                       int64_t block_stride, int B, const int32_t* prefix_len, const int32_t* path,
                       int max_depth, const int32_t* num_accepted, int32_t* out_new_len,
                       int32_t* out_status, void* stream);

/* ------------------------------------------------------------------------------------
 * The paged cache of the target's attention (SD 20.5, "Keeping the caches consistent after a
 * rejection"): the calls that write it and attend over it, before the logits are verified.
 *
 * A sequence's tokens sit at logical slots 0, 1, ...; slot s of sequence b is entry
 * s % page_size of page block_table[b * max_pages + s / page_size].  A slot holds kv_heads
 * rows of head_dim values for keys and as many for values, at
 *   k + page * page_stride + (s % page_size) * slot_stride + head * head_stride   (bytes),
 * the same strides for v.  specdec_compact_kv moves slots of the same pages.
 *   SPECDEC_BF16, SPECDEC_F16: a row is head_dim 16-bit values.
 *   SPECDEC_KV4: a row is head_dim / 2 bytes of E2M1 codes, the even value in the low nibble;
 *     k_scales / v_scales hold head_dim / 16 E4M3 bytes per row at their own strides, one for
 *     each 16 values.  A value is code * scale * k_scale (v_scale for values).  k_scale and
 *     v_scale are positive and finite; they are not read for 16-bit pages.
 *   SPECDEC_KV8: a row is head_dim E4M3 codes.  The scale_block slots of a block share a scale for each
 *     head, a power of two between 2^-15 and 2^7 held as its E8M0 byte (the exponent plus 127): k_scales /
 *     v_scales hold it at page * scale_page_stride + (s % page_size / scale_block) * scale_slot_stride +
 *     head * scale_head_stride (bytes, any).  A value is code * scale * k_scale (v_scale); before k_scale it is exact
 *     in fp16.  page_size is a multiple of scale_block, that a multiple of 16; the pages' strides are below 2^40, that of
 *     slots positive; k_scale and v_scale have finite reciprocals.  specdec_compact_kv does not
 *     know the scales: after a tree's round the accepted tokens are appended again at their slots.
 * Pointers and strides are multiples of 16 bytes (4-bit pages' scales: of head_dim / 16 bytes); head_dim is
 * 64 or 128; max_pages * page_size < 2^31 - 256.
 *
 * Lengths, for each call below: context_len[b] counts sequence b's tokens including the new
 * ones of this call, query_len[b] <= n the new ones (NULL: n for every sequence); new token i
 * is slot context_len[b] - query_len[b] + i.  Outputs for i >= query_len[b] are zeros.
 * out_status[b] (optional) is SPECDEC_STATUS_BAD_CACHE for a length that does not fit (negative,
 * query_len above n or above context_len, slots past max_pages) or a page outside
 * [0, num_pages) among those the call uses for the sequence, else 0.
 */
typedef struct specdec_kv_pages {
  void* k;
  void* v;
  void* k_scales; /* SPECDEC_KV4 and SPECDEC_KV8 */
  void* v_scales;
  const int32_t* block_table; /* [B, max_pages], device */
  int64_t page_stride, slot_stride, head_stride;
  int64_t scale_page_stride, scale_slot_stride, scale_head_stride; /* SPECDEC_KV4 and SPECDEC_KV8 */
  int32_t num_pages, page_size, max_pages, kv_heads, head_dim;
  int32_t format; /* SPECDEC_BF16, SPECDEC_F16, SPECDEC_KV4 or SPECDEC_KV8 */
  float k_scale, v_scale;
  int32_t scale_block; /* SPECDEC_KV8 only: slots that share a scale */
} specdec_kv_pages;

/* Norms of queries and keys for each head, the position rotation, and the write of keys and
 * values to 16-bit pages, in one pass.
 *
 * For each head vector x of D = head_dim values:
 *   y = x * weight / sqrt(mean(x^2) + eps)      (weight NULL: y = x)
 *   (y_a, y_b) <- (y_a cos t - y_b sin t, y_b cos t + y_a sin t),  t = position * f_j,
 * for the pairs (a, b) = (j, j + rot/2), or (2j, 2j + 1) with interleaved != 0, j < rot/2; values
 * from rot on are not rotated.  The position is context_len[b] - query_len[b] + i, or + depth[i]
 * for tree nodes (depth [n] int32, specdec_build_tree_mask's out_depth; NULL: i).
 * turns [rot/2] uint64: f_j in 2^-64 turns for a position (f_j / (2 pi) * 2^64 for f_j in
 * radians), so that position * f_j is exact modulo a turn at every position.
 * Statistics, angles and products are fp32; every value is rounded once, at the end.
 *
 * q, k, v         [B, n, heads, D] of dtype (SPECDEC_BF16 or SPECDEC_F16); strides in elements
 *                 of sequence, token and head in q_strides[3], k_strides[3], v_strides[3] (host
 *                 arrays), the last dimension contiguous: views of a fused projection's output
 * q_weight, k_weight [D] of dtype, or NULL
 * out_q           [B, n, q_heads, D] contiguous
 * out_k           [B, n, kv_heads, D] contiguous when pages is NULL (v is not used then); else
 *                 NULL, and keys and values go to the pages, whose format is dtype
 * A sequence in error leaves its pages alone; its out_q (and out_k) rows are NaN.
 * 16 <= rot <= D, a multiple of 16; D is 64 or 128; B <= 65535; pointers and strides multiples of
 * 16 bytes.  Two sequences must not write the same slot. */
int specdec_rotate_qk(const void* q, const int64_t* q_strides, const void* k, const int64_t* k_strides,
                      const void* v, const int64_t* v_strides, specdec_dtype dtype, const void* q_weight,
                      const void* k_weight, float eps, const uint64_t* turns, int rot, int interleaved,
                      const int32_t* context_len, const int32_t* query_len, const int32_t* depth, int B, int n,
                      int q_heads, int kv_heads, int head_dim, void* out_q, void* out_k,
                      const specdec_kv_pages* pages, int32_t* out_status, void* stream);

/* Keys and values [B, n, kv_heads, D] (strides as above) written to 4-bit pages.
 * For each 16 values x, with y = x * (1 / k_scale) in fp32: scale = E4M3(max|y| / 6) (nearest
 * even, saturated at 448), code = the E2M1 number nearest to y / scale (ties to the even
 * code); a zero scale gives zeros.  A group with a value that is not finite stores the scale
 * NaN and reads back as NaN.  A sequence in error is left alone.  B <= 65535. */
int specdec_append_kv4(const void* k, const int64_t* k_strides, const void* v, const int64_t* v_strides,
                       specdec_dtype dtype, const int32_t* context_len, const int32_t* query_len, int B, int n,
                       const specdec_kv_pages* pages, int32_t* out_status, void* stream);

/* The values that 4-bit pages hold for the last query_len[b] tokens of each sequence:
 * out_k, out_v [B, n, kv_heads, D] of dtype, contiguous, each rounded once.  A sequence in
 * error gives NaN.  B <= 65535. */
int specdec_read_kv4(const int32_t* context_len, const int32_t* query_len, int B, int n,
                     const specdec_kv_pages* pages, specdec_dtype dtype, void* out_k, void* out_v,
                     int32_t* out_status, void* stream);

/* Keys and values [B, n, kv_heads, D] (strides as above) written to 8-bit pages.
 * With y = x * (1 / k_scale) in fp32: a block's scale is the smallest 2^e, e in [-15, 7], with max|y| <= 448 * 2^e
 * over the new tokens that fall into it, and never below its scale of before when the block holds earlier tokens of
 * the sequence (slots before the first new one); code = the E4M3 number nearest to y / 2^e (ties to the even code,
 * saturated at 448).  Where a block's scale grows, the codes of its earlier tokens are rounded to the new scale: exact but
 * for codes that become subnormal.  A value that is not finite is stored as NaN and does not count for the scale.
 * Slots from a block's new tokens on are not looked at: rejected drafts are overwritten by appending again with the
 * shorter context_len (a block keeps its scale then).  So a rejected draft leaves a mark: the scale s that it raised stays until
 * the block is begun again, and accepted tokens of the block, those before it and those after, are off by up to 2^-9 s (times k_scale)
 * from what they would be without it, where they are below 2^-6 s.  A caller whose accepted tokens must not depend on rejected ones
 * keeps the codes and scale bytes of the block of slot context_len[b] - query_len[b] before drafts are appended, puts them back once the drafts
 * are verified, and appends the accepted ones again at their slots.  A sequence in error is left alone.  Two sequences must not write the
 * same block; strides of zero (of more than one page, block or head) are refused here.  B <= 65535. */
int specdec_append_kv8(const void* k, const int64_t* k_strides, const void* v, const int64_t* v_strides,
                       specdec_dtype dtype, const int32_t* context_len, const int32_t* query_len, int B, int n,
                       const specdec_kv_pages* pages, int32_t* out_status, void* stream);

/* The values that 8-bit pages hold for the last query_len[b] tokens of each sequence, as
 * specdec_read_kv4 gives them. */
int specdec_read_kv8(const int32_t* context_len, const int32_t* query_len, int B, int n,
                     const specdec_kv_pages* pages, specdec_dtype dtype, void* out_k, void* out_v,
                     int32_t* out_status, void* stream);

/* Attention of the new tokens over the cache, which holds their keys and values already
 * (specdec_rotate_qk, specdec_append_kv4, specdec_append_kv8).
 *
 * With P = context_len[b] - query_len[b], query i sees slot s when
 *   chain (tree_mask NULL):  s <= P + i
 *   tree: s < P, or tree_mask[i * n + (s - P)] != 0 and s < context_len[b]
 * and, with window > 0, pos(i) - pos(s) < window or pos(s) < sinks: the last `window` positions,
 * itself among them, and the first `sinks`.  pos(s) = s before P, P + i for new token i, or
 * P + depth[i] in a tree (depth in [0, n)).  tree_mask [n, n] uint8 and depth [n] int32 are
 * shared by the batch: specdec_build_tree_mask's out_mask and out_depth for prefix_len 0.
 *   out[b, i, h] = sum_s p_s v_s,  p = softmax over the visible s of scale * q . k_s,
 * query head h with key head h / (q_heads / kv_heads).  Values and keys of slots that a query
 * does not see do not touch its output, whatever they hold (NaN, infinities, stale pages); an
 * output that does depend on a value that is not finite is not finite (an infinity or NaN).  A
 * visible score of -inf (an infinite key) has the weight 0; a row whose visible scores are all -inf, or
 * one of them +inf, gives NaN and lse NaN.
 *
 * q            [B, n, q_heads, D] of dtype (SPECDEC_BF16 or SPECDEC_F16), q_strides as above
 * pages        16-bit pages of the same dtype, SPECDEC_KV4 or SPECDEC_KV8
 * out          [B, n, q_heads, D] contiguous
 * out_lse      [B, n, q_heads] fp32, optional: log of the sum of exp(scale * q . k_s)
 * A query that sees nothing gives zeros and lse -inf; one that sees a slot on a page outside
 * [0, num_pages) gives NaN, as does every query of a sequence whose lengths do not fit.  Pages
 * that no query sees (behind a window) are not read, and their entries are not looked at.
 * Scores, statistics and sums are fp32; the weights p are rounded to 16 bits (dtype, or fp16 for
 * 4-bit and 8-bit pages; in fp16 to 2^-32 of the row's largest where that is more) for the matrix products,
 * the output once at the end.  Over 8-bit and 4-bit pages bf16 queries are held in fp16, to 2^-25 of a row's largest value;
 * over 8-bit pages with 17 to 32 query rows to a key head queries of either type are held to 2^-17 of a
 * row's largest value (values from 2^-9 of it up in bf16, and from 2^-6 up in fp16, are exact).
 * Every wait inside the kernels is bounded (one second); a call in which one runs out reports
 * SPECDEC_STATUS_TIMEOUT for every sequence, and its outputs do not count.
 * The workspace (specdec_attend_workspace_bytes) follows the rules at the top.  The split of the
 * work follows the lengths on the device: the host reads none of them.
 * window, sinks >= 0 (window 0: no window, sinks then has no effect); q_heads a multiple of
 * kv_heads, at most 65535 times; n * (q_heads / kv_heads) < 2^24; B < 2^24. */
size_t specdec_attend_workspace_bytes(int B, int n, int q_heads, int kv_heads, int head_dim);

int specdec_attend(const void* q, const int64_t* q_strides, specdec_dtype dtype, const specdec_kv_pages* pages,
                   const int32_t* context_len, const int32_t* query_len, const uint8_t* tree_mask,
                   const int32_t* depth, int B, int n, int q_heads, int window, int sinks, float scale, void* out,
                   float* out_lse, int32_t* out_status, void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------------------
 * What is done to the target's logits before they are verified (SD 20.5, "Four ways to lose exactness": p is the
 * distribution the target samples from, after its processing; every row of a round has its own history).
 *
 * Row i of a sequence follows the tokens generated so far and the drafts before it: tokens[b, 0 .. i-1] of a chain
 * (parents NULL), or row 0 the root and row 1 + i node i with the tokens on the path from the root to node i,
 * itself included.  With c the number of times t occurs among those (its entry of `counts` and the row's drafts),
 * for each token t of the vocabulary:
 *   x  = logits[b, i, t];  if c > 0 or t is in the prompt:  x = x > 0 ? x / repetition[b] : x * repetition[b]
 *   x  = x - frequency[b] * c - (c > 0 ? presence[b] : 0) + the bias listed for t
 *   out[b, i, t] = x, or -inf where the row's mask has no bit for t.
 * Computed in fp32, each step rounded to nearest: the quotient or product; the penalties (frequency * c + presence once); the bias
 * less them; the sum.  A bf16 result is rounded once more.  A masked token is -inf whatever its logit holds (NaN too); a row whose mask leaves nothing
 * is all -inf, which the verification calls report (SPECDEC_STATUS_EMPTY_ROW).
 *
 * logits       [B, rows, V] of dtype (SPECDEC_F32 or SPECDEC_BF16); out the same, or logits itself: in place (one that overlaps
 *              it otherwise is refused)
 * tokens       [B, rows - 1] int32: drafts or node tokens; may be NULL (then they do not count, whatever rows is)
 * parents      [rows - 1] int32, parent in [-1, i): a tree; NULL: a chain
 * gammas       [B] int32 in [0, rows - 1], optional, chains only: the drafts that specdec_verify_chain_varlen verifies;
 *              rows past gammas[b] are neither read nor written, and tokens from gammas[b] on may hold anything
 * counts       [B, V] int32, optional: the low 31 bits are c without drafts, the sign bit says that t is in the prompt
 *              (specdec_count_tokens)
 * repetition, presence, frequency [B] fp32, each optional (NULL: 1, 0, 0); repetition is positive
 * bias_tokens, bias_values [B, num_bias] int32 and fp32, optional (num_bias 0): negative tokens are skipped; of a token
 *              that is listed twice the last entry counts
 * mask         [B, rows, (V + 31) / 32] uint32, optional: bit t % 32 of word t / 32 is set where t is allowed
 * out_status   [B] int32, optional: SPECDEC_STATUS_BAD_TOKEN (a token outside [0, V) that a row counts, a bias token
 *              of V or more, gammas[b] out of range), SPECDEC_STATUS_BAD_TREE (a parent out of range), SPECDEC_STATUS_BAD_PENALTY (a repetition that is not
 *              positive and finite, a presence or frequency that is not finite), else 0.  The rows of a sequence in error are NaN.
 * rows <= 8192, B <= 65535, num_bias < 2^24, V < 2^31 - 65536.  Meant for a round's tens of rows: a draft's token is counted
 * along the path of each row, so that thousands of different drafts take tens of milliseconds; every few thousand tokens
 * of the vocabulary the list of biases is read once. */
int specdec_process_logits(const void* logits, specdec_dtype dtype, const int32_t* tokens, const int32_t* parents,
                           const int32_t* gammas, const int32_t* counts, const float* repetition,
                           const float* presence, const float* frequency, const int32_t* bias_tokens,
                           const float* bias_values, int num_bias, const uint32_t* mask, int B, int rows, int V,
                           void* out, int32_t* out_status, void* stream);

/* The table of token counts that specdec_process_logits reads: for each of the first num_tokens[b] <= n tokens of
 * sequence b (NULL: n), counts[b, t] grows by one, or, with prompt != 0, its sign bit is set.  Negative tokens are skipped, so a
 * verification call's out_tokens can be counted as they are; so are tokens of V or more, which out_status reports
 * (SPECDEC_STATUS_BAD_TOKEN), as num_tokens[b] outside [0, n] is clamped.  reset != 0: the sequence's entries are set to zero before.
 * tokens [B, n] int32, rows token_stride elements apart; counts [B, V] int32, in place.
 * n may be 0.  B <= 65535, V and n < 2^31 - 65536. */
int specdec_count_tokens(int32_t* counts, const int32_t* tokens, int64_t token_stride, const int32_t* num_tokens, int B,
                         int n, int V, int prompt, int reset, int32_t* out_status, void* stream);

/* ------------------------------------------------------------------------------------
 * Tree-attention mask and position ids (SD 20.5, box "Token tree and tree attention").
 *   out_mask          [N, P+N] uint8: row i is 1 on every prefix column j < P, on column
 *                     P+i and on column P+a for every ancestor a of node i; 0 elsewhere
 *   out_position_ids  [N] int64: P + depth(i), depth = number of ancestors
 *   out_depth         [N] int32, optional
 *   out_status        [1] int32: SPECDEC_STATUS_BAD_TREE if some parents[i] is not in
 *                     [-1, i); the other outputs are then unspecified
 * N >= 1, P >= 0, (P + N) * N < 2^31.
 */
int specdec_build_tree_mask(const int32_t* parents, int N, int prefix_len, uint8_t* out_mask,
                            int64_t* out_position_ids, int32_t* out_depth, int32_t* out_status,
                            void* stream);

/* ------------------------------------------------------------------------------------
 * Kernel timing for benchmarks.  While enabled, every kernel the library launches is
 * bracketed by a pair of CUDA events recorded on the launching stream.  The state is
 * process-global and not thread-safe; enable it only around single-threaded timing.
 *   specdec_profile_start(max_launches): creates the event pool; returns SPECDEC_OK.
 *   specdec_profile_read(total_ms, launches, n): synchronises the recorded events and
 *     writes per-kernel totals for kernel ids 0..n-1 (ids: SPECDEC_KERNEL_*); resets.
 *   specdec_profile_stop(): disables timing and destroys the events.
 */
#define SPECDEC_KERNEL_CHAIN_STATS 0   /* row statistics over every logits row      */
#define SPECDEC_KERNEL_CHAIN_SAMPLE 1  /* residual / bonus masses of the drawn rows */
#define SPECDEC_KERNEL_TREE_WALK 2
#define SPECDEC_KERNEL_TREE_MASK 3
#define SPECDEC_KERNEL_CHAIN_DECIDE 4  /* accept tests and first rejection          */
#define SPECDEC_KERNEL_CHAIN_FINISH 5  /* inverse-CDF search of the drawn rows      */
#define SPECDEC_KERNEL_CHAIN_SEQ 6     /* left-to-right chain verification          */
#define SPECDEC_KERNEL_BLOCK_DECIDE 7  /* block verification: weights per prefix    */
#define SPECDEC_KERNEL_BLOCK_FINISH 8  /* block verification: survival and the draw */
#define SPECDEC_KERNEL_BLOCK_FUSED 9   /* block verification in one launch           */
#define SPECDEC_KERNEL_TREE_RR 10      /* tree verification by recursive rejection   */
#define SPECDEC_KERNEL_GUMBEL 11       /* Gumbel-coupled verification                */
#define SPECDEC_KERNEL_GUMBEL_DRAFT 12 /* the drafter's shared-noise sampler          */
#define SPECDEC_KERNEL_KV_COMPACT 13   /* accepted-branch KV compaction              */
#define SPECDEC_KERNEL_ROTATE_QK 14        /* norms, rotation and the page write          */
#define SPECDEC_KERNEL_APPEND_KV4 15       /* the 4-bit page write                       */
#define SPECDEC_KERNEL_READ_KV4 16         /* 4-bit pages read back                      */
#define SPECDEC_KERNEL_ATTEND 17           /* attention over pages, its join included    */
#define SPECDEC_KERNEL_APPEND_KV8 18       /* the 8-bit page write                       */
#define SPECDEC_KERNEL_READ_KV8 19         /* 8-bit pages read back                      */
#define SPECDEC_KERNEL_PROCESS_LOGITS 20   /* penalties, biases and masks                */
#define SPECDEC_KERNEL_COUNT_TOKENS 21     /* the table of token counts                  */
#define SPECDEC_NUM_KERNELS 22

int specdec_profile_start(int max_launches);
int specdec_profile_read(double* total_ms, int* launches, int n);
int specdec_profile_stop(void);

/* ------------------------------------------------------------------------------------
 * Chain verification without any allocation (no counterpart in the source pages; this is
 * a deployment convenience).
 *
 * Some callers cannot allocate device memory, or must not: code running under an
 * inference server's fixed memory plan that forbids allocations after start-up, plain C
 * hosts that link only this library and receive their tensors from elsewhere, and
 * latency-critical paths where cudaMalloc/cudaFree would synchronise the device.  This
 * entry point takes the same arguments as specdec_verify_chain minus the workspace and
 * uses scratch memory built into the library instead: one array of
 * SPECDEC_NOALLOC_SCRATCH_BYTES in device memory, which every GPU that loads the library
 * holds until the process exits.  It allocates nothing and calls no allocating routine.
 *
 *   - Set-up: the first call on each device (with that device current) looks up the
 *     array's device address; make that first call before any stream capture begins.
 *     The address is kept per device and primary context: after a device reset
 *     (cudaDeviceReset) the next call looks it up again.
 *   - Limit: a shape whose specdec_chain_workspace_bytes() exceeds
 *     SPECDEC_NOALLOC_SCRATCH_BYTES is rejected with SPECDEC_ERR_TOO_LARGE (nothing is
 *     launched; specdec_last_error() gives the sizes).  16 MiB covers, e.g., B=512, g=8,
 *     V=152064 fp32.
 *   - Sharing: every call on a device uses the same array and it keeps the last call's
 *     contents; each call clears the counters it needs on its own stream first.  Calls
 *     that overlap on the GPU (different streams, or host threads) race on the array and
 *     must be serialised by the caller.
 *   - Results are the same as specdec_verify_chain's for the same inputs.
 */
#define SPECDEC_NOALLOC_SCRATCH_BYTES ((size_t)16 << 20)

int specdec_verify_chain_noalloc(const void* logits, specdec_dtype ldt, const float* draft_probs,
                                 const int32_t* draft_tokens, const float* temperatures,
                                 const float* uniforms, int B, int g, int V, int32_t* out_tokens,
                                 int32_t* out_num_accepted, float* out_p_draft, int32_t* out_status,
                                 void* stream);

/* ------------------------------------------------------------------------------------
 * Test hooks (the library's own tests and sweeps; not for production use).
 *
 * Process-global settings read by the calls issued after them (not thread-safe; set them
 * while no call is being issued).  Every hook defaults to 0, the production behaviour.
 *   SPECDEC_HOOK_CHAIN_ALL_ROWS    1: chain and greedy calls whose rows the left-to-right
 *                                  kernel takes run the all-rows streaming kernels instead
 *   SPECDEC_HOOK_BLOCK_TWO_PASS    1: block verification runs the statistics and mass
 *                                  kernels instead of the one-launch kernel
 *   SPECDEC_HOOK_TREE_CLUSTER      1, 2, 4 or 8: the tree walks' cluster size (where it fits)
 *   SPECDEC_HOOK_CHAIN_DROP_DRAWS  1: the left-to-right kernel never marks a queued draw
 *                                  as published, so the teams that take its ticket wait
 *                                  until the queue wait gives up (the sequences it belongs
 *                                  to come back with SPECDEC_STATUS_TIMEOUT)
 *   SPECDEC_HOOK_QUEUE_WAIT_US     >= 1: the left-to-right kernel's bound on waits for
 *                                  queued work, in microseconds (0: one second)
 *   SPECDEC_HOOK_ATTEND_KERNEL     1 or 2: attention over pages takes the kernel on warp-level
 *                                  matrix instructions, or the tensor-memory kernel, whatever
 *                                  the number of rows
 * Returns SPECDEC_OK, or SPECDEC_ERR_INVALID_ARG for an unknown hook or value.
 */
#define SPECDEC_HOOK_CHAIN_ALL_ROWS 0
#define SPECDEC_HOOK_BLOCK_TWO_PASS 1
#define SPECDEC_HOOK_TREE_CLUSTER 2
#define SPECDEC_HOOK_CHAIN_DROP_DRAWS 3
#define SPECDEC_HOOK_QUEUE_WAIT_US 4
#define SPECDEC_HOOK_ATTEND_KERNEL 5
#define SPECDEC_NUM_HOOKS 6

int specdec_set_test_hook(int hook, int value);
int specdec_get_test_hook(int hook);

/* Library version string, e.g. "0.1.0". */
const char* specdec_version(void);

/* Description of the last SPECDEC_ERR_CUDA returned on the calling host thread: the step
 * that failed and the CUDA error.  The string stays valid until the thread's next call. */
const char* specdec_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* SPECDEC_H */

/*
 * spec_verify.h -- C ABI of the speculative-sampling verify library for
 * NVIDIA GB300 (sm_103a).
 *
 * One vocabulary sweep per (batch row, drafted position) computes the
 * temperature softmax of target and draft logits, the overlap
 * alpha = sum_v min(p, q) = 1 - d_TV(p, q), the min(1, p/q) acceptance, the
 * residual max(0, p - q) correction and the bonus draw; the E2E-TV entry
 * point turns the same sweep into a loss and its draft-logit gradient.
 *
 * Citations name the page and the section that defines each operation:
 *   "Speculative Decoding 与 MTP：先猜多个 token，再让大模型一次验完"
 *   "读 Qwen Bebop 与 DeepSeek DSpark：Speculative Decoding 正在从技巧变成系统工程"
 *   "SpecOPD: Branch-Parallel On-Policy Distillation for Speculative Decoding"
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - Every buffer argument is a DEVICE pointer owned by the caller.  The
 *    library allocates no device memory; scratch space is the caller's
 *    `workspace` (size from the matching *_workspace_bytes function).
 *  - Logit tensors are row-major and contiguous: element v of position k of
 *    batch row b sits at base + ((b * P + k) * V + v) * elem_size, where P is
 *    the number of positions stored per batch row.  Bulk (TMA) loads are used
 *    when V * elem_size is a multiple of 16 bytes and the base is 16-byte
 *    aligned; other shapes take a slower element-wise staging path.
 *  - Work is enqueued asynchronously on `stream` (a cudaStream_t; NULL is the
 *    legacy default stream).  The host return value covers argument checks
 *    and the launch only.  Problems found in the data are OR-ed into the
 *    caller's 32-bit device word `dev_status` (may be NULL) and become visible
 *    once the caller synchronises the stream; kernels never trap.
 *  - The workspace must be zero-filled before its first use (for instance by
 *    cudaMemsetAsync); every call that completes leaves it zero-filled again.
 *    Two calls that may run at the same time on the GPU must not share a
 *    workspace.
 *  - Temperatures are float32; T == 0 selects greedy decoding where allowed.
 *  - Limits: B >= 0, 0 <= K <= 64, 1 <= V, and 2 * V * elem_size may not
 *    exceed 16 CTAs' worth of shared memory (V up to about 900k for bf16).
 */
#ifndef SPEC_VERIFY_H_
#define SPEC_VERIFY_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  SPEC_OK = 0,
  SPEC_ERR_INVALID_ARG = 1, /* a pointer, size, dtype or temperature is invalid */
  SPEC_ERR_UNSUPPORTED = 2, /* valid request beyond the library's limits */
  SPEC_ERR_CUDA = 3         /* the CUDA runtime reported an error */
} spec_status_t;

/* SPEC_F16: the drafter-training losses, and keys and values. */
typedef enum { SPEC_F32 = 0, SPEC_BF16 = 1, SPEC_F16 = 2 } spec_dtype_t;

/* Bits OR-ed into *dev_status by the kernels. */
#define SPEC_DEV_BAD_TOKEN 1u      /* a drafted token outside [0, V) (treated as rejected) */
#define SPEC_DEV_BAD_LOGITS 2u     /* NaN or +inf logit, or no finite logit in a row */
#define SPEC_DEV_BAD_UNIFORM 4u    /* a uniform outside [0, 1) */
#define SPEC_DEV_TIMEOUT 8u        /* a bounded wait inside a kernel gave up */
#define SPEC_DEV_EMPTY_RESIDUAL 16u /* rejection with zero residual mass: drawn from p */
#define SPEC_DEV_BAD_OFFSETS 32u   /* ragged row offsets rejected (nothing computed), or a tree parent outside [-1, i) */
#define SPEC_DEV_BAD_PAGE 64u      /* a page or slot outside the cache */
#define SPEC_DEV_NO_PAGES 128u     /* too few free pages for the tokens that a step commits */

/* Version of this ABI (bumped on any signature change). */
int spec_abi_version(void);

/* Human-readable name of a status code (static string). */
const char* spec_status_string(spec_status_t status);

/* Number of kernels this library has launched in this process, over every
 * device and stream: counted on the host when a launch is enqueued without
 * error (library memsets are not counted).  For measurement: read it before
 * and after a timed region.  Never fails. */
unsigned long long spec_kernel_launches(void);

/* ------------------------------------------------------------------------ */
/* Batched verify step.
 *
 * Defined by "Speculative Decoding 与 MTP", section 2 (draft/verify loop: K
 * candidates, target distributions p_1..p_K plus the bonus distribution, the
 * first rejection ends the block), section 3 (accept with min(1, p/q); after
 * a rejection draw from the residual max(0, p - q), never from the full p)
 * and section 4 (greedy T == 0 compares with the target argmax; p and q use
 * the same temperature).  The overlap written to alpha_out is alpha_RS of
 * "读 Qwen Bebop 与 DeepSeek DSpark", section "用公式看".
 *
 * target_logits  [B, K+1, V] dtype: p_k = softmax(target[b,k] / T); row K is
 *                the bonus distribution.
 * draft_logits   [B, K, V] dtype: q_k = softmax(draft[b,k] / T).  May be NULL
 *                only when T == 0 and alpha_out == NULL.
 * draft_tokens   [B, K] int32: the drafted tokens y_k (sampled by the caller).
 * u_accept       [B, K] float32 in [0, 1): draft k is accepted iff
 *                u_accept <= p_k(y_k) / q_k(y_k).  Unused when T == 0.
 * u_final        [B] float32 in [0, 1): inverse-CDF uniform for the one
 *                correction or bonus token of the row.  Unused when T == 0.
 * out_tokens     [B, K+1] int32 (written): the n accepted drafts, then the
 *                correction (n < K) or bonus (n == K) token, then -1.
 * n_accepted     [B] int32 (written): n in [0, K]; tokens emitted = n + 1.
 * alpha_out      [B, K] float32 or NULL: per-position overlap alpha_k
 *                (at T == 0 the indicator [argmax p_k == argmax q_k]).
 * Inverse CDF: the smallest token v whose running sum in vocabulary order
 * exceeds u_final times the total mass.
 */
size_t spec_verify_workspace_bytes(int B, int K, int V);

spec_status_t spec_verify(const void* target_logits, const void* draft_logits,
                          spec_dtype_t dtype, int B, int K, int V,
                          float temperature, const int32_t* draft_tokens,
                          const float* u_accept, const float* u_final,
                          int32_t* out_tokens, int32_t* n_accepted,
                          float* alpha_out, uint32_t* dev_status,
                          void* workspace, size_t workspace_bytes,
                          void* stream);

/* ------------------------------------------------------------------------ */
/* Relaxed verify -- LOSSY: the output no longer follows the target
 * distribution.
 *
 * "Speculative Decoding 与 MTP", section 4: accepting a candidate because it
 * lies in the target's top-k, or because its logprob is close, raises the
 * acceptance rate but gives up the lossless guarantee; results must be
 * labelled lossy.  Draft k is accepted, in prefix order, when its drafted
 * token ranks among the target's top_k tokens (by logit, ties to the smaller
 * index; top_k <= 0: no rank condition) and
 * log p_k(y) >= max_v log p_k(v) - delta (delta = +inf: no gap condition).
 * The first rejected position emits a draw from the full p_k with u_final
 * (no residual); a block with every draft accepted emits the bonus from
 * p_{K+1}, as spec_verify does.  alpha_out reports the exact overlap.
 *
 * Arguments as spec_verify (same workspace size), without u_accept;
 * temperature T > 0; delta >= 0.
 */
spec_status_t spec_verify_relaxed(const void* target_logits,
                                  const void* draft_logits, spec_dtype_t dtype,
                                  int B, int K, int V, float temperature,
                                  int top_k, float delta,
                                  const int32_t* draft_tokens,
                                  const float* u_final, int32_t* out_tokens,
                                  int32_t* n_accepted, float* alpha_out,
                                  uint32_t* dev_status, void* workspace,
                                  size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------ */
/* Candidate trees.
 *
 * A tree of N candidate nodes per row is given by parent[b][i] < i (-1: the
 * node hangs on the committed prefix).  "SpecOPD", section "树注意力(Tree
 * Attention)": node u may attend to v iff v is u or an ancestor of u, so one
 * batched target pass scores every node without leaking sibling branches.
 *
 * spec_tree_mask: mask [B, N, N] uint8 (written): 1 iff v is u or an
 * ancestor of u; depth [B, N] int32 or NULL: the number of strict ancestors
 * (the node's offset past the prefix).  A parent outside [-1, i) sets
 * SPEC_DEV_BAD_OFFSETS and stops that node's walk.
 */
spec_status_t spec_tree_mask(const int32_t* parent, int B, int N,
                             uint8_t* mask, int32_t* depth,
                             uint32_t* dev_status, void* stream);

/* Greedy (T = 0) verify of a candidate tree, committing one path per row:
 * "Speculative Decoding 与 MTP", section 4 (keep a candidate equal to the
 * target argmax; the first mismatch emits the target's token) and section 11
 * (a tree commits a single path).
 *
 * target_logits [B, N + 1, V] dtype: slot 0 after the committed prefix, slot
 *               i + 1 after node i (one target pass over the tree, masked as
 *               spec_tree_mask gives).
 * parent, node_tokens [B, N] int32.
 * From the prefix, the walk moves to the first child (node order) whose token
 * is the current slot's argmax (smallest index on ties), and emits that argmax
 * where no child matches.
 * path        [B, N] int32 (written): accepted nodes, prefix side first, -1 after.
 * out_tokens  [B, N + 1] int32 (written): their tokens, then the emitted
 *             target token, then -1.
 * n_accepted  [B] int32 (written): accepted nodes (-1 for a bad parent map).
 * Sampling (T > 0) over trees needs a multi-candidate acceptance rule that
 * the cited pages do not give; it is not provided.
 */
size_t spec_tree_verify_workspace_bytes(int B, int N, int V);

spec_status_t spec_tree_verify_greedy(const void* target_logits,
                                      spec_dtype_t dtype, int B, int N, int V,
                                      const int32_t* parent,
                                      const int32_t* node_tokens,
                                      int32_t* path, int32_t* out_tokens,
                                      int32_t* n_accepted,
                                      uint32_t* dev_status, void* workspace,
                                      size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------ */
/* Ragged verify: every row verifies its own number of drafted tokens, in
 * flattened tensors.
 *
 * "读 Qwen Bebop 与 DeepSeek DSpark", section "DSpark 真正厉害的地方：它为生产系统
 * 做了让步" (variable-length verification tokens of all requests are
 * flattened, and a marker tensor carries which request each belongs to) and
 * section "DSpark 的第二块拼图" (per-request verify lengths l_r); the
 * acceptance, correction and bonus rules are those of spec_verify.
 *
 * row_offsets  [B + 1] int32, device: row r owns flattened target rows
 *              [row_offsets[r], row_offsets[r+1]) = its l_r drafted positions
 *              then its bonus position; row_offsets[0] = 0,
 *              row_offsets[B] = units, 0 <= l_r <= 64.  Offsets that break
 *              this set SPEC_DEV_BAD_OFFSETS and nothing is computed.
 * units        the number of flattened target rows (host value).
 * target_logits [units, V] dtype; draft_logits [units - B, V] dtype, drafted
 *              row of (r, j) at row_offsets[r] - r + j (NULL if units == B).
 * draft_tokens, u_accept [units - B]: same flattened order as the drafts.
 * u_final      [B].  temperature T > 0.
 * out_tokens   [units] int32: row r's n accepted drafts, then the correction
 *              or bonus token, then -1, at row_offsets[r] ...
 * n_accepted   [B]; alpha_out [units - B] float32 or NULL.
 * The workspace follows the common rules (zero before first use, zero
 * after every call).  The per-unit marker (row, position, bonus) is built in
 * the workspace by the call.
 */
size_t spec_verify_ragged_workspace_bytes(int B, int units, int V);

spec_status_t spec_verify_ragged(const void* target_logits,
                                 const void* draft_logits, spec_dtype_t dtype,
                                 int B, const int32_t* row_offsets, int units,
                                 int V, float temperature,
                                 const int32_t* draft_tokens,
                                 const float* u_accept, const float* u_final,
                                 int32_t* out_tokens, int32_t* n_accepted,
                                 float* alpha_out, uint32_t* dev_status,
                                 void* workspace, size_t workspace_bytes,
                                 void* stream);

/* ------------------------------------------------------------------------ */
/* Allocation-free verify.  The pages have no counterpart: this entry point
 * exists for callers that cannot allocate device memory when they run a
 * verify step -- runtimes whose pool owns all device memory from start-up,
 * plugin hosts that provide buffers but no allocator, and latency-critical
 * decode loops that cannot take the device-wide synchronisation of
 * cudaMalloc / cudaFree.
 *
 * Same arguments and results as spec_verify, without the workspace: the
 * scratch is a fixed device array of SPEC_NOALLOC_SCRATCH_BYTES inside the
 * library, held by every GPU that loads the library until the process exits.
 * Sizes whose spec_verify_workspace_bytes(B, K, V) exceeds it are rejected with
 * SPEC_ERR_UNSUPPORTED (at K = 4 that is 393 rows, at K = 7 245 rows).  No call
 * allocates or frees memory; each clears the part of the array it uses with
 * cudaMemsetAsync on `stream`.
 *  - The first call on a device looks up the array's device address (once per
 *    device, with that device current; a failed lookup is retried by the next
 *    call); make that first call before any stream capture.
 *  - Every call on a device shares the one array: calls that may overlap on
 *    the GPU (different streams without ordering between them) race and give
 *    wrong results.  Serialise them. */
#define SPEC_NOALLOC_SCRATCH_BYTES (4u << 20)

spec_status_t spec_verify_noalloc(const void* target_logits,
                                  const void* draft_logits, spec_dtype_t dtype,
                                  int B, int K, int V, float temperature,
                                  const int32_t* draft_tokens,
                                  const float* u_accept, const float* u_final,
                                  int32_t* out_tokens, int32_t* n_accepted,
                                  float* alpha_out, uint32_t* dev_status,
                                  void* stream);

/* ------------------------------------------------------------------------ */
/* Overlap statistics of K drafted positions.
 *
 * alpha_k = sum_v min(p_k, q_k) = 1 - d_TV(p_k, q_k), prefix survival
 * a_j = prod_{k<=j} alpha_k and E[tau] = sum_j a_j: "读 Qwen Bebop 与
 * DeepSeek DSpark", section "用公式看" (alpha_RS, d_TV, P(tau >= j), E[tau])
 * and section "DSpark 的第二块拼图" (soft label c*_k = 1 - d_TV, a_j).
 *
 * target_logits  [B, KT, V] dtype, KT >= K: position k < K of each row is used
 *                (pass KT = K + 1 to reuse a verify batch's target tensor).
 * draft_logits   [B, K, V] dtype.
 * temperature    T >= 0 (T == 0: alpha_k = [argmax p_k == argmax q_k]).
 * alpha          [B, K] float32 (written, required).
 * tv             [B, K] float32 or NULL: 1 - alpha_k.
 * prefix_survival [B, K] float32 or NULL.
 * expected_accepted [B] float32 or NULL: E[tau] (add 1 for emitted tokens).
 */
size_t spec_overlap_workspace_bytes(int B, int K, int V);

spec_status_t spec_overlap(const void* target_logits, const void* draft_logits,
                           spec_dtype_t dtype, int B, int K, int KT, int V,
                           float temperature, float* alpha, float* tv,
                           float* prefix_survival, float* expected_accepted,
                           uint32_t* dev_status, void* workspace,
                           size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------ */
/* E2E-TV loss and its gradient with respect to the draft logits.
 *
 * L = (1/B) sum_b sum_{j=1..K} prod_{k<=j} alpha_{b,k}: "读 Qwen Bebop 与
 * DeepSeek DSpark", section "Bebop 的解法" (E[tau] written with
 * 1 - d_TV(p_k, q_k)); "SpecOPD", method step (6): prefix products of the
 * per-position overlap, only the draft probabilities are differentiated and
 * the target is a constant.  The loss is the expected accepted length (to be
 * maximised); pass grad_scale = -1 to get the gradient of -L.
 *
 * grad[b,k,v] = grad_scale * dL/dalpha_{b,k} * (q_v / T) * (1[q_v < p_v] - S),
 * S = sum_{u: q_u < p_u} q_u, with
 * dL/dalpha_k = (1/B) prod_{i<k} alpha_i (1 + alpha_{k+1} + alpha_{k+1} alpha_{k+2} + ...).
 *
 * target_logits  [B, KT, V] dtype, KT >= K (first K positions used).
 * draft_logits   [B, K, V] dtype.
 * temperature    T > 0.
 * loss_out       [1] float32 (written).
 * alpha_out      [B, K] float32 or NULL.
 * grad_draft_logits [B, K, V] float32 (overwritten).
 */
size_t spec_e2e_tv_workspace_bytes(int B, int K, int V);

spec_status_t spec_e2e_tv_fwd_bwd(const void* target_logits,
                                  const void* draft_logits, spec_dtype_t dtype,
                                  int B, int K, int KT, int V,
                                  float temperature, float grad_scale,
                                  float* loss_out, float* alpha_out,
                                  float* grad_draft_logits,
                                  uint32_t* dev_status, void* workspace,
                                  size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------ */
/* Per-position distribution diagnostics of K drafted positions.
 *
 * "读 Qwen Bebop 与 DeepSeek DSpark", section "Qwen Bebop：RL 里的瓶颈不是 MTP
 * 不会猜，而是策略熵在变" (acceptance falls as the target's entropy rises; a
 * point-mass drafter is accepted with probability p(argmax q)) and section
 * "Bebop 的解法" (cross-entropy or KL training of the drafter against
 * training for the acceptance itself).  With p = softmax(target / T) and
 * q = softmax(draft / T), natural logarithms, 0 log 0 = 0:
 *   alpha   = sum_v min(p_v, q_v)
 *   entropy = -sum_v p_v log p_v
 *   kl      = sum_v p_v (log p_v - log q_v)   (+inf if some q_v = 0 < p_v)
 *   cross_entropy = entropy + kl = -sum_v p_v log q_v
 *   alpha_target_only = p(y_hat), y_hat = argmax_v q_v (smallest index on ties)
 *
 * target_logits  [B, KT, V] dtype, KT >= K (first K positions used).
 * draft_logits   [B, K, V] dtype.
 * temperature    T > 0.
 * alpha, entropy, cross_entropy, kl, alpha_target_only
 *                [B, K] float32 each, or NULL (not written).
 * A row with NaN or +inf logits, or no finite logit, gets NaN in every output
 * and SPEC_DEV_BAD_LOGITS.
 */
size_t spec_diagnostics_workspace_bytes(int B, int K, int V);

spec_status_t spec_diagnostics(const void* target_logits,
                               const void* draft_logits, spec_dtype_t dtype,
                               int B, int K, int KT, int V, float temperature,
                               float* alpha, float* entropy,
                               float* cross_entropy, float* kl,
                               float* alpha_target_only, uint32_t* dev_status,
                               void* workspace, size_t workspace_bytes,
                               void* stream);

/* ------------------------------------------------------------------------ */
/* Top-k / top-p truncation of logit rows, to be applied with the same
 * arguments to the target and the draft logits before a verify step.
 *
 * "Speculative Decoding 与 MTP", section 4 (p and q are both computed after the
 * agreed temperature and top-k / top-p transforms) and section 23 (a mask that
 * only one side applies breaks correctness).  Tokens are ranked by logit,
 * larger first, ties to the smaller index.  Top-k (0 < top_k < V) keeps the
 * first top_k.  Top-p (top_p < 1) then renormalises softmax(z / T) over the
 * kept tokens and keeps the shortest ranked prefix whose mass reaches top_p.
 * Dropped logits become -inf; kept logits are copied unchanged.
 *
 * logits       [rows, V] dtype, device.
 * out          [rows, V] dtype, device; may be `logits` itself (in place) but
 *              may not overlap it otherwise.
 * temperature  T > 0 when top_p < 1 (unused otherwise).
 * top_k        >= 0; 0 or >= V disables top-k.
 * top_p        in (0, 1]; 1 disables top-p.
 * A row holding a NaN or +inf logit, or no finite logit, is copied unchanged
 * and sets SPEC_DEV_BAD_LOGITS.  Top-p masses are fixed point with 2^-44 of
 * the row maximum's mass as unit; a cut whose preceding mass lies within
 * about 1e-6 of top_p may move by one token against exact arithmetic.
 */
spec_status_t spec_truncate_logits(const void* logits, void* out,
                                   spec_dtype_t dtype, int rows, int V,
                                   float temperature, int top_k, float top_p,
                                   uint32_t* dev_status, void* stream);

/* ------------------------------------------------------------------------ */
/* Verify-length scheduling.
 *
 * "读 Qwen Bebop 与 DeepSeek DSpark", section "DSpark 的第二块拼图：置信度调度验证
 * 长度": request r verifying l_r drafted tokens adds 1 + l_r tokens to the
 * target batch, B = sum_r (1 + l_r), and produces tau_r = 1 +
 * sum_{j<=l_r} a_{r,j} tokens in expectation; the lengths maximise
 * Theta = (sum_r tau_r) * SPS(B), SPS(B) the engine's decode steps per second
 * at batch B.  For a fixed B the best choice takes the B - R largest
 * survivals; equal survivals are taken in (row, position) order and equal
 * Theta keeps the smaller B.
 *
 * survival   [R, L] float32: a_{r,j}, j = 1..L, non-increasing in j (the
 *            prefix_survival output of spec_overlap is such a table); the
 *            running minimum along j is used; NaN counts as 0 and sets
 *            SPEC_DEV_BAD_LOGITS.
 * sps        [sps_len] float32 >= 0: SPS(B) for B = 0 .. sps_len - 1,
 *            sps_len >= R * (1 + L) + 1.
 * lengths    [R] int32 (written): l_r in [0, L].
 * objective  [2] float32 or NULL: {Theta, tau} at the choice.
 * Limits: 1 <= L <= 64 and R * L <= 16384 (SPEC_ERR_UNSUPPORTED beyond).
 * One cluster of 16 CTAs (distributed shared memory; no workspace).
 * Survivals are summed exactly as integers in units of 2^-48 (one
 * rounding each, so sums of n of them are within n * 2^-49 of the real sum);
 * Theta is formed in fp64.  A choice whose Theta lies within about 1e-10
 * relative of another B's may therefore differ from exact arithmetic.
 */
spec_status_t spec_schedule_lengths(const float* survival, int R, int L,
                                    const float* sps, int sps_len,
                                    int32_t* lengths, float* objective,
                                    uint32_t* dev_status, void* stream);

/* ------------------------------------------------------------------------ */
/* Losses for training a drafter.
 *
 * "读 Qwen Bebop 与 DeepSeek DSpark", section "Bebop 的解法" (drafters are trained
 * with cross entropy or KL; the E2E-TV loss above is the alternative that
 * targets acceptance); "SpecOPD", method step (6) (only the draft side is
 * differentiated, the target is a constant).
 *
 * Rules shared by these entry points
 *  - reduction: loss = (1 / count) sum_n w_n L_n (SPEC_MEAN, count = the rows
 *    that count, 0 if there are none) or sum_n w_n L_n (SPEC_SUM); w_n =
 *    row_weight[n], or 1 where row_weight is NULL.  Gradients are those of
 *    grad_scale * loss.
 *  - A row that is left out has row_loss 0 and no part in loss, count or any
 *    gradient, whatever its logits or hidden states hold (also NaN).
 *  - A row that counts and whose logits hold NaN or +inf, or no finite value,
 *    sets SPEC_DEV_BAD_LOGITS; its results are NaN.
 *  - Results do not depend on timing: the same inputs give the same bits.
 *  - The workspace needs NO initial contents and holds none to rely on
 *    afterwards: unlike the other entry points' workspaces it is not
 *    zero-filled by the call, so it must not be shared with them.
 *    It must lie on a 256-byte boundary.
 *  - N == 0 gives loss 0 and a zero head gradient.
 *  - Listed teacher tokens: teacher_ids [N, k] int32, 1 <= k <= 256, -1 marks
 *    an unused slot; teacher_logits [N, k] float32.  A row without a used
 *    slot is left out.  An id outside [-1, V) or listed twice sets
 *    SPEC_DEV_BAD_TOKEN, and teacher values that cannot be normalised (NaN,
 *    +inf, nothing but -inf) set SPEC_DEV_BAD_LOGITS; both leave the row out.
 */
typedef enum { SPEC_MEAN = 0, SPEC_SUM = 1 } spec_reduction_t;

/* Cross entropy of a vocabulary head from its hidden states, z_n = hidden_n .
 * weight^T / T, without storing the logits (of a call with gradients see
 * the workspace):
 *   L_n = logsumexp(z_n) - z_n[label_n]
 *
 * hidden     [N, H], weight [V, H]: dtype SPEC_BF16 or SPEC_F16, contiguous,
 *            16-byte aligned, H a multiple of 8 (N <= 2^20, V < 2^24, H <= 2^16;
 *            SPEC_ERR_UNSUPPORTED beyond).  Products are exact and summed
 *            in fp32 by the tensor cores, 16 at a time: a logit is within about
 *            2.5e-6 of its size at H = 2048, growing with H (the label's and the listed tokens'
 *            logits come from the same sums, so that confident rows keep
 *            their digits).
 * labels     [N] int32; a row whose label is ignore_index is left out, and so
 *            is one whose label is otherwise outside [0, V), which also sets
 *            SPEC_DEV_BAD_TOKEN.
 * loss_out   [1], row_loss [N] or NULL, lse_out [N] or NULL (natural log of
 *            the normaliser, of every row): float32.
 * grad_hidden [N, H], grad_weight [V, H] or NULL (not computed), of
 *            grad_dtype = dtype or SPEC_F32, 16-byte aligned.  The gradient of
 *            the logits is rounded once to dtype on its way into the products.
 *
 * Workspace: spec_linear_loss_workspace_bytes gives the preferred size,
 * spec_linear_loss_workspace_least the least; a call takes what it is given,
 * in between too.  Both cover the gradients that are asked for:
 *  - a call of any kind holds the rows' statistics of every 256 tokens (8 bytes
 *    each), its lists, and up to one copy of the hidden states;
 *  - one with grad_hidden adds fp32 partials of it (4 N H bytes each, up to 32 where
 *    few rows would leave the GPU idle);
 *  - one with a gradient adds N values for each token of the vocabulary, or of a
 *    piece of it.  A batch whose N V values fit 4 GB prefers the whole
 *    vocabulary, and the normaliser's pass then leaves its unnormalised
 *    probabilities there: 2 bytes a value for SPEC_BF16 and 6 for SPEC_F16, so
 *    up to as much as the logits in 16 bits, or three times that.  Longer
 *    batches, and calls with less room, go in pieces of 2 bytes a value
 *    (preferred 256 MB, least 4 KB a row) and compute the logits a second
 *    time: one product more than the three with both gradients, or the two
 *    with one.
 * The same workspace size gives the same bits; another one may cut the sums
 * elsewhere and agrees within rounding.
 */
size_t spec_linear_loss_workspace_bytes(spec_dtype_t dtype, int N, int V, int H, int k, int want_grad_hidden,
                                        int want_grad_weight);
size_t spec_linear_loss_workspace_least(spec_dtype_t dtype, int N, int V, int H, int k, int want_grad_hidden,
                                        int want_grad_weight);

spec_status_t spec_linear_cross_entropy(const void* hidden, const void* weight, spec_dtype_t dtype, int N, int V,
                                        int H, float temperature, const int32_t* labels, int ignore_index,
                                        const float* row_weight, spec_reduction_t reduction, float* loss_out,
                                        float* row_loss, float* lse_out, uint32_t* dev_status, void* workspace,
                                        size_t workspace_bytes, void* stream);

spec_status_t spec_linear_cross_entropy_fwd_bwd(const void* hidden, const void* weight, spec_dtype_t dtype, int N,
                                                int V, int H, float temperature, float grad_scale,
                                                const int32_t* labels, int ignore_index, const float* row_weight,
                                                spec_reduction_t reduction, float* loss_out, float* row_loss,
                                                float* lse_out, void* grad_hidden, void* grad_weight,
                                                spec_dtype_t grad_dtype, uint32_t* dev_status, void* workspace,
                                                size_t workspace_bytes, void* stream);

/* Distillation from a teacher's top logits through the head: with t =
 * softmax(teacher_logits / T) over the row's used slots and q = softmax(z),
 *   L_n = sum_i t_i (log t_i - log q_i)
 * Other arguments as above (workspace with this call's k). */
spec_status_t spec_linear_topk_distill(const void* hidden, const void* weight, spec_dtype_t dtype, int N, int V, int H,
                                       int k, float temperature, const int32_t* teacher_ids,
                                       const float* teacher_logits, const float* row_weight,
                                       spec_reduction_t reduction, float* loss_out, float* row_loss, float* lse_out,
                                       uint32_t* dev_status, void* workspace, size_t workspace_bytes, void* stream);

spec_status_t spec_linear_topk_distill_fwd_bwd(const void* hidden, const void* weight, spec_dtype_t dtype, int N,
                                               int V, int H, int k, float temperature, float grad_scale,
                                               const int32_t* teacher_ids, const float* teacher_logits,
                                               const float* row_weight, spec_reduction_t reduction, float* loss_out,
                                               float* row_loss, float* lse_out, void* grad_hidden, void* grad_weight,
                                               spec_dtype_t grad_dtype, uint32_t* dev_status, void* workspace,
                                               size_t workspace_bytes, void* stream);

/* Distillation of given student logits from a teacher's top logits.
 *
 * student [N, V] dtype (SPEC_F32, SPEC_BF16 or SPEC_F16), row-contiguous, any
 * alignment of the element's size; -inf marks dropped tokens.
 * q = softmax(student / T) over the whole vocabulary.
 * teacher_lse NULL: t = softmax(teacher_logits / T) over the used slots, and
 *   L_n = sum_i t_i (log t_i - log q_i)
 * teacher_lse [N] float32 (logsumexp of the teacher's whole row / T): t_i =
 * exp(teacher_logits_i / T - teacher_lse), and what both sides leave over
 * counts as one more token,
 *   L_n = sum_i t_i (log t_i - log q_i) + t_r (log t_r - log q_r),
 * t_r = 1 - sum_i t_i (0 where that is below 1e-6, the rounding of the sum),
 * q_r = 1 - sum_i q_i.
 * With M = sum_i t_i + t_r the gradient is (M q_i - t_i) / T on the listed
 * tokens and q_v (M - t_r / q_r) / T on the others.
 * loss_out [1], row_loss [N] or NULL: float32.  grad [N, V] of grad_dtype =
 * dtype or SPEC_F32.
 * Limits: N <= 2^30; a row of at most 16 x 208 KiB (what 16 CTAs hold): V up to
 * 1703936 16-bit or 851968 fp32 logits.
 */
size_t spec_topk_distill_workspace_bytes(int N, int V, int k);

spec_status_t spec_topk_distill(const void* student, spec_dtype_t dtype, int N, int V, int k, float temperature,
                                const int32_t* teacher_ids, const float* teacher_logits, const float* teacher_lse,
                                const float* row_weight, spec_reduction_t reduction, float* loss_out, float* row_loss,
                                uint32_t* dev_status, void* workspace, size_t workspace_bytes, void* stream);

spec_status_t spec_topk_distill_fwd_bwd(const void* student, spec_dtype_t dtype, int N, int V, int k,
                                        float temperature, float grad_scale, const int32_t* teacher_ids,
                                        const float* teacher_logits, const float* teacher_lse,
                                        const float* row_weight, spec_reduction_t reduction, float* loss_out,
                                        float* row_loss, void* grad, spec_dtype_t grad_dtype, uint32_t* dev_status,
                                        void* workspace, size_t workspace_bytes, void* stream);

/* ------------------------------------------------------------------------ */
/* One decoding step around the verify: attention over a paged cache, the
 * cache's tables, and the sampling rules on the logits.
 *
 * A pass holds, for every request b, T_b rows: row 0 is the last committed
 * token, the others are drafted tokens (a chain, or a tree's nodes), as the
 * target slots of spec_verify, spec_verify_ragged and spec_tree_verify_greedy
 * follow them.  Rows are laid out [B, T, ...] (row_offsets NULL, T_b = T) or
 * flattened with row_offsets [B + 1] int32 (request b owns the rows
 * [row_offsets[b], row_offsets[b + 1]), at most T of them).  A request whose
 * offsets decrease, leave [0, rows] or hold more than T rows is left out
 * (nothing of it is written) and sets SPEC_DEV_BAD_OFFSETS.  Rows that no
 * request owns are left as they were.
 * mask [B, T, T] uint8: row i sees row j of its pass iff mask[b][i][j] != 0
 * (spec_tree_mask of the rows' parent map); NULL: a chain, i sees 0 .. i.
 *
 * The cache holds, page by page, the keys and values of committed tokens:
 * token n of request b lies at place n % page_size of the page
 * block_table[b][n / page_size]. */

typedef struct {
  const void* q;       /* [rows, Hq, D] dtype, strides below */
  const void* k_new;   /* [rows, Hkv, D]: keys of the pass's own rows */
  const void* v_new;   /* [rows, Hkv, D] */
  const void* k_cache; /* [pages, page_size, Hkv, D] */
  const void* v_cache; /* [pages, page_size, Hkv, D] */
  void* out;           /* [rows, Hq, D] dtype, contiguous (written) */
  float* lse;          /* [rows, Hq] contiguous (written) or NULL */
  const int32_t* block_table;  /* [B, table_width], rows table_stride apart */
  const int32_t* context_lens; /* [B]: cached tokens of each request */
  const int32_t* row_offsets;  /* [B + 1] or NULL */
  const uint8_t* mask;         /* [B, T, T] or NULL */
  long long q_stride[2];       /* elements between rows, heads */
  long long k_new_stride[2], v_new_stride[2];
  long long k_stride[3], v_stride[3]; /* elements between pages, tokens, heads */
  long long table_stride;
  int B, T, rows, Hq, Hkv, D, pages, page_size, table_width;
  spec_dtype_t dtype;  /* SPEC_BF16 or SPEC_F16 */
  float scale;         /* of the scores; log2(e) of it finite */
} spec_attention_t;

/* Attention of a pass's rows over the cache and the pass itself.
 *
 * "SpecOPD", section "树注意力(Tree Attention)": a node sees the committed
 * prefix, itself and its ancestors, so that one target pass scores every node;
 * "Speculative Decoding 与 MTP", section 2 (a chain); T = 1 is plain decoding.
 * For row i of request b and head h, over the cached tokens n <
 * context_lens[b] and the rows j that row i sees:
 *   s = scale q . k,  out = sum exp(s) v / sum exp(s),  lse = log sum exp(s)
 * with the keys and values of head h / (Hq / Hkv).  A row that sees nothing,
 * or only scores of -inf, gets out = 0 and lse = -inf.  Keys and values that a
 * row does not see do not enter it, whatever they hold.  Scores and sums are
 * fp32; the weights exp(s - max) are rounded once for the product with v, to
 * dtype's precision (in fp16 with 2^11 times their size: weights below 2^-25 of
 * the largest are off by up to 2^-36 of it).
 *
 * No gradients.  T decides how the work is laid out: beyond 128 / (Hq / Hkv)
 * (rounded down) requests of few rows take up to a third longer, so that a batch of
 * single tokens and a few large trees is better off in two calls.
 *
 * Limits: D a multiple of 8, at most 256; Hq a multiple of Hkv, at most 128
 * times it; page_size a multiple of 8; T <= 1024; table_width * page_size below
 * 2^31; strides multiples of 8 and below 2^39; tensors on 16-byte boundaries,
 * the workspace on a 256-byte one.
 * A context length outside [0, table_width * page_size] counts as the nearer
 * bound and sets SPEC_DEV_BAD_OFFSETS.  A page outside [0, pages) reads as
 * zeros and sets SPEC_DEV_BAD_PAGE.
 * out and lse overlap nothing that is read.
 * The workspace need not be zeroed, and is not left zero. */
size_t spec_tree_attention_workspace_bytes(int B, int T, int Hq, int Hkv, int D);

spec_status_t spec_tree_attention(const spec_attention_t* args, uint32_t* dev_status, void* workspace,
                                  size_t workspace_bytes, void* stream);

/* Tables of the cache for the tokens that a step commits.
 *
 * Request b holds ceil(context_lens[b] / page_size) pages, the first entries
 * of its row of the block table.  new_lens[b] >= 0 tokens are appended to it,
 * or its last -new_lens[b] are taken back (-context_lens[b]: the request is
 * done).  free_pages[0 .. free_count) is a stack of unused pages.  First all
 * pages that are given back are pushed, in the order of the requests and, in
 * each, of its table; then the pages that are needed are popped in the same
 * order.  From the first request on that finds too few pages left, requests
 * that need pages are left as they were (their slots -1, their length
 * unchanged) and SPEC_DEV_NO_PAGES is set.
 *
 * context_lens, new_lens [B] int32; block_table [B, table_width] int32;
 * free_pages [capacity] int32; free_count [1] int32.
 * out_table, out_free: as block_table and free_pages, and may be them (in
 *   place); they may not overlap them otherwise.  Entries of the table behind
 *   a request's pages, and of the stack above its new count, keep what they
 *   held: the pages given back were pushed before any was popped.
 * out_count [1], out_lens [B] int32 (written): the new count and lengths; not
 *   the inputs.
 * slots [B, T] int32 (written): page * page_size + place of the appended
 *   tokens, then -1.  A page below 0, or one whose slot is beyond 2^31 - 1, gives its
 *   tokens the slot 2^31 - 1, which no cache has (spec_commit_cache refuses it), and sets
 *   SPEC_DEV_BAD_PAGE.
 * A request with context_lens or the new length outside [0, table_width *
 * page_size], or with new_lens > T, is left as it was and sets
 * SPEC_DEV_BAD_OFFSETS.  A free_count outside [0, capacity], or pages given
 * back beyond the capacity, leave every request as it was and set that bit. */
spec_status_t spec_plan_cache(const int32_t* context_lens, const int32_t* new_lens, const int32_t* block_table,
                              const int32_t* free_pages, const int32_t* free_count, int B, int T, int table_width,
                              int capacity, int page_size, int32_t* out_table, int32_t* out_free, int32_t* out_count,
                              int32_t* out_lens, int32_t* slots, uint32_t* dev_status, void* stream);

typedef struct {
  const void* k_new;    /* [layers, rows, Hkv, D], strides below */
  const void* v_new;
  void* k_cache;        /* [layers, pages, page_size, Hkv, D] (written) */
  void* v_cache;
  const int32_t* slots; /* [B, S]: spec_plan_cache's; -1: none */
  const int32_t* path;  /* [B, S - 1], rows path_stride apart: accepted nodes, or NULL */
  const int32_t* row_offsets;                   /* [B + 1] or NULL */
  long long k_new_stride[3], v_new_stride[3];   /* elements between layers, rows, heads */
  long long k_stride[4], v_stride[4];           /* elements between layers, pages, tokens, heads */
  long long path_stride;
  int layers, B, T, rows, S, Hkv, D, pages, page_size;
  spec_dtype_t dtype;   /* SPEC_BF16 or SPEC_F16 */
} spec_commit_t;

/* Copies the keys and values of the committed rows of a pass into the cache,
 * all layers at once ("Speculative Decoding 与 MTP", section 11: a tree commits
 * a single path).  Place i of request b takes row 0 for i = 0, then row i
 * (path NULL) or path[b][i - 1] + 1 (spec_tree_verify_greedy's path, whose
 * node n is the pass's row n + 1).  Slots below 0 take nothing.  A slot beyond
 * the cache sets SPEC_DEV_BAD_PAGE, a node below 0 or a row that the request does
 * not have SPEC_DEV_BAD_OFFSETS; neither writes anything.  Slots have to be distinct:
 * of one that occurs twice, what its token holds afterwards may come from
 * either row.
 * k_new and v_new may not lie in the cache's own slots.
 * Limits: D a multiple of 8; strides multiples of 8; tensors on 16-byte boundaries;
 * pages * page_size below 2^31. */
spec_status_t spec_commit_cache(const spec_commit_t* args, uint32_t* dev_status, void* stream);

typedef struct {
  const void* logits;          /* [rows, V] dtype, contiguous */
  void* out;                   /* as logits (written); may be logits */
  const int32_t* tokens;       /* [rows]: the pass's row tokens; -1: not counted (a root that the history holds) */
  const int32_t* history;      /* [B, history_width]: tokens before the pass */
  const int32_t* history_lens; /* [B] */
  const int32_t* prompt_lens;  /* [B] or NULL (0): the history's first tokens that were given, not generated */
  const float* repetition;     /* [B] or NULL (1) */
  const float* frequency;      /* [B] or NULL (0) */
  const float* presence;       /* [B] or NULL (0) */
  const int32_t* bias_ids;     /* [B, biases]; -1: none */
  const float* bias;           /* [B, biases] */
  const uint32_t* allowed;     /* [rows, ceil(V / 32)] or NULL: bit v % 32 of word v / 32 */
  const int32_t* row_offsets;  /* [B + 1] or NULL */
  const uint8_t* mask;         /* [B, T, T] or NULL */
  int B, T, rows, V, history_width, biases;
  spec_dtype_t dtype;          /* SPEC_F32 or SPEC_BF16 */
} spec_adjust_t;

/* Sampling rules on the logits of a pass, before spec_truncate_logits and the
 * verify; apply them to the target and the draft logits alike
 * ("Speculative Decoding 与 MTP", sections 4 and 23: p and q after the same
 * transforms, and a mask that only one side applies breaks correctness).
 *
 * For token v at row i of request b, c(v) counts v in the history behind the
 * prompt and among the tokens of the rows that row i sees (itself included):
 *   z  = z > 0 ? z / repetition : z * repetition   where c(v) > 0 or the prompt holds v
 *   z += the biases listed for v, less frequency * c(v) + presence where c(v) > 0
 *   z  = -inf                                      where v is not allowed
 * in fp32 (the biases added up in their order), rounded once to dtype.  Untouched logits are copied bit by bit.
 * No gradients.
 * Tokens, history and bias ids outside [0, V) count for nothing and set
 * SPEC_DEV_BAD_TOKEN (-1 as a row's token or a bias id does not); history or
 * prompt lengths beyond the history count as the nearer bound and set
 * SPEC_DEV_BAD_OFFSETS.  Rows that nothing is allowed for become -inf
 * throughout.
 * Limits: B <= 65535, T <= 1024, biases <= 1024, history_width < 2^19, V <= 2^24. */
spec_status_t spec_adjust_logits(const spec_adjust_t* args, uint32_t* dev_status, void* stream);

/* ------------------------------------------------------------------------ */
/* Failure-path self-test of the bounded wait.
 *
 * Launches two warps.  The second one waits, with the same bounded mbarrier
 * wait the sweep uses on its bulk copies, for a phase of a fresh shared-memory
 * mbarrier that nothing ever completes; the first one's wait ends at once.  No
 * copy is in flight.  After limit_ns nanoseconds of wall time the wait gives
 * up; the block's first thread learns of it as in the logit rules, ORs
 * SPEC_DEV_TIMEOUT into *dev_status, and the kernel returns.  Tests use it to check that
 * a wait that runs out is reported on the status word and that the context
 * stays usable afterwards.
 * limit_ns   in [1, 10^10] (10 s).
 * dev_status [1] uint32, device (required).
 * Returns SPEC_ERR_INVALID_ARG for a limit out of range or a NULL status.
 */
spec_status_t spec_selftest_bounded_wait(uint64_t limit_ns, uint32_t* dev_status, void* stream);

/* ------------------------------------------------------------------------ */
/* Launch shape the library picks for a sampling verify sweep over `units`
 * (row, position) pairs of V logits with rows on 16-byte boundaries (for
 * benchmarks and diagnostics; the two-pass sweep when units x 2 rows reach
 * 200 MB, as in spec_set_kernel_override): CTAs per cluster, threads per CTA (608 for
 * the two-pass sweep: sixteen consumer warps, a copy warp, a decision warp
 * and a completion warp; 256 for the single-read sweep), dynamic shared memory
 * per CTA, the number of persistent clusters launched and the shared-memory
 * stages per CTA.  Needs a current CUDA device.  Returns
 * SPEC_ERR_UNSUPPORTED if V does not fit.  Any output pointer may be NULL. */
spec_status_t spec_launch_shape(spec_dtype_t dtype, int units, int V,
                                int* cluster_ctas, int* threads,
                                int* smem_bytes, int* clusters, int* stages);

/* Forces the CTAs per cluster (1..16) and caps the shared-memory stages per
 * CTA (the two-pass sweep's ring stages, at least 1; the single-read sweep's
 * 1 or 2) of later launches in this process, for launch-shape sweeps in
 * benchmarks; 0 restores the automatic choice of either.  Process-wide; not
 * synchronised with launches in flight. */
void spec_set_launch_override(int cluster_ctas, int stages);

/* Selects the vocabulary-sweep kernel of later verify, overlap and E2E-TV
 * calls in this process: 0 automatic (the two-pass sweep for calls that read
 * at least 200 MB of logits, where rows start on 16-byte boundaries and the
 * mode has it; else the single-read sweep),
 * 1 the single-read sweep (rows resident in cluster shared memory between
 * passes), 2 the two-pass sweep where it applies (pass A from HBM, pass C
 * from L2).  Any other value means 0.  For tests and benchmarks; both give
 * the same results within the parity bar.  Process-wide; not synchronised
 * with launches in flight. */
void spec_set_kernel_override(int kernel);

#ifdef __cplusplus
}
#endif

#endif /* SPEC_VERIFY_H_ */

/*
 * smcsd.h -- C ABI of the GB300 library for the speculative-decoding verify step over
 * vocabulary-wide logits: temperature / power-target logsumexp, SD rejection sampling,
 * SMC-SD importance reweighting, effective sample size, systematic resampling, the paged-KV
 * page-table remap, and the PACER blockwise stop rule with ragged verify.
 *
 * Sources (gist.science summary pages; the pages print no formulas, so where a step is only
 * named the textbook rule is used and stated below):
 *   [SMC]   "Faster LLM Inference via Sequential Monte Carlo": sec. 1 (SD verifies by rejection
 *           sampling, the block is discarded after the first rejection), sec. 2 steps 1-4
 *           (N particles, K drafts each, one target scoring pass, reweighting by the
 *           target/draft probability ratio, resampling when the effective sample size falls
 *           below a threshold, exactly K+1 tokens per particle and step), sec. 3 (page-based
 *           KV: resampling is a metadata update; power sampling and reward-weighted decoding as
 *           modified targets; error bounds in N), sec. 5 (reward optimisation and hard
 *           constraints through the same importance weights).
 *   [PACER] "PACER: Blockwise Pre-verification for Speculative Decoding with Adaptive Length",
 *           Methodik 1-3 (blocks of b drafts whose hidden states, with position embeddings, give
 *           an estimated acceptance; the block mean against a threshold t that is multiplied by
 *           rho after each block that passes).
 *   [UAG]   "Cross-Family Speculative Decoding for Polish Language Models on Apple Silicon",
 *           sec. 1 (the target verifies k candidates in one pass).
 *
 * Conventions for every entry point
 *   - Every pointer argument is a DEVICE pointer owned by the caller, except where noted. The
 *     library allocates nothing and keeps no state between calls outside the caller's buffers;
 *     the one exception is smc_step_static, whose scratch is a device area of the library's own.
 *   - `stream` is a cudaStream_t passed as void* (NULL = the legacy default stream). Every call
 *     only enqueues work on it and returns; results are valid once the stream has reached them.
 *   - Logits are row-major [rows, V] with V contiguous; dtype SMCSD_F32 (float32) or SMCSD_BF16.
 *     -inf marks a masked token. NaN or +inf, or a row with nothing but -inf, is an error
 *     detected on the device (SMCSD_ERR_NONFINITE).
 *   - Uniforms are float32 in [0,1), supplied by the caller (one per random decision), so that a
 *     run is reproducible and its randomness can be shared with a checker.
 *   - `ws` is a scratch buffer of at least smcsd_workspace_size(op, ...) bytes, 256-byte aligned,
 *     which must be zero-filled once before its first use (smcsd_workspace_init). Every call that
 *     returns SMCSD_OK leaves the buffer's counters at zero again, at one place for all operators
 *     and sizes, so a buffer of the largest size needed can be reused by calls of any of them in
 *     stream order without clearing. Calls that may overlap on the GPU need separate buffers.
 *   - Return value: SMCSD_OK, or a negative status for errors found on the host before anything
 *     is enqueued (bad argument, dtype, workspace size) or at launch (CUDA error). Errors that
 *     depend on device data (non-finite logits, token ids or offsets out of range) are recorded
 *     in `ws` and read with smcsd_check_status(). The kernels never trap. The waits inside a block
 *     (the copy pipelines of the streaming pass and of the attention) and those of the steps and of
 *     distill_loss for another block of their cluster give up after a few seconds at most and record
 *     SMCSD_ERR_TIMEOUT. The counters that such a call leaves behind are cleared by
 *     smcsd_check_status; calls that use the buffer before that are unspecified. Two kinds of waits have
 *     no limit of their own: the cluster barriers of kv_slot_map, kv_pagetable_remap, kv_fork, kv_free,
 *     kv_compact and distill_loss (a cluster's blocks run at the same time), and those of tree_attention in bf16
 *     for its SM's tensor memory, as long as another kernel holds some of it. So a bad input cannot fault or hang the GPU; outputs are unspecified
 *     after such an error.
 */
#ifndef SMCSD_H
#define SMCSD_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* status codes */
#define SMCSD_OK 0
#define SMCSD_ERR_INVALID_ARG (-1) /* null pointer, non-positive size, T <= 0, alpha <= 0, ... */
#define SMCSD_ERR_DTYPE (-2)       /* dtype other than SMCSD_F32 / SMCSD_BF16 */
#define SMCSD_ERR_WORKSPACE (-3)   /* ws_bytes smaller than smcsd_workspace_size() or ws misaligned */
#define SMCSD_ERR_CUDA (-4)        /* a CUDA call or kernel launch failed */
#define SMCSD_ERR_NONFINITE (-5)   /* device: NaN/+inf logit or weight, or an all-masked row */
#define SMCSD_ERR_RANGE (-6)       /* device: token id, offset, ancestor or page id out of range */
#define SMCSD_ERR_TIMEOUT (-7)     /* device: a bounded wait inside a kernel ran out (a few seconds) */
#define SMCSD_ERR_PAGES (-8)       /* device: kv_slot_map found fewer free pages than it needs */

/* logit element types */
#define SMCSD_F32 0
#define SMCSD_BF16 1

/* targets of the tilted SMC reweight (smc_reweight_tilted, smc_step_tilted) */
#define SMCSD_TARGET_TOKEN 0    /* per position: pi = softmax(alpha z / T), as smc_reweight */
#define SMCSD_TARGET_SEQUENCE 1 /* whole sequence: prod_t p_t(x_t)^alpha, p = softmax(z / T) */

/* operation ids for smcsd_workspace_size */
#define SMCSD_OP_SD_VERIFY 0
#define SMCSD_OP_SMC_REWEIGHT 1
#define SMCSD_OP_SMC_STEP 2
#define SMCSD_OP_ESS_RESAMPLE 3
#define SMCSD_OP_PAGETABLE_REMAP 4
#define SMCSD_OP_PACER_BLOCK_STOP 5
#define SMCSD_OP_DRAFT_SAMPLE 6 /* S = number of rows R; K is ignored */
#define SMCSD_OP_KV_SLOT_MAP 7    /* S sequences, V = number of pages; K is ignored */
#define SMCSD_OP_KV_APPEND 8      /* any S > 0; K and V are ignored */
#define SMCSD_OP_TREE_MASK 9      /* any S > 0; K and V are ignored */
#define SMCSD_OP_LOGITS_PROCESS 10 /* any S > 0; K and V are ignored */
#define SMCSD_OP_BEAM_SELECT 11    /* S = rows of logits (G*N), V; K is ignored */
#define SMCSD_OP_STATE_REORDER 12  /* any S > 0; K and V are ignored */
#define SMCSD_OP_KV_FORK 13        /* kv_fork, kv_free and kv_copy_pages: any S > 0; K and V are ignored */
#define SMCSD_OP_KV_COMPACT 14     /* any S > 0, V = number of pages; K is ignored (serves kv_fork's calls too) */
#define SMCSD_OP_DISTILL_LOSS 15   /* any S > 0; K and V are ignored */

/*
 * Scratch bytes that `op` needs for S sequences (or particles; for the resampling ops S is the
 * number of groups G), at most K draft positions and vocabulary V.
 */
size_t smcsd_workspace_size(int op, int S, int K, int V);

/* Zero-fill `ws` on `stream` (needed once before a buffer's first use). */
int smcsd_workspace_init(void* ws, size_t ws_bytes, void* stream);

/*
 * Wait for `stream`, then return the first device-side error recorded in `ws` since the last
 * check (SMCSD_OK if none) and clear it.
 */
int smcsd_check_status(void* ws, void* stream);

/* Static text for a status code. */
const char* smcsd_status_string(int code);

/*
 * Diagnostic for the failure path of the bounded waits (no counterpart on the pages): one warp
 * runs the streaming pass's two pipeline waits against a barrier and a slot tag that nothing
 * completes, each giving up after limit_us microseconds (1 .. 2000000) and recording
 * SMCSD_ERR_TIMEOUT in `ws` as a stalled pipeline would. Read it with smcsd_check_status; the
 * context stays usable. ws: any workspace of at least 8 bytes (zero-filled once, as always).
 */
int smcsd_selftest_wait(unsigned int limit_us, void* ws, size_t ws_bytes, void* stream);

/*
 * Speculative-decoding verify ([SMC] sec. 1; [UAG] sec. 1; ragged lengths from [PACER]
 * Methodik 2). For every sequence s, with p = softmax(z_t / T) and q = softmax(z_d / T):
 *   accept draft x_k iff u[s*(K+1)+k] < min(1, p_k(x_k) / q_k(x_k)), k = 0, 1, ... in order;
 *   accept_len[s] = index of the first rejection, or K_s if all pass;
 *   out_token[s]  = draw from normalise(max(0, p_acc - q_acc)) if a draft was rejected, else
 *                   the bonus draw from p at target row K_s; both by inverse CDF with
 *                   u[s*(K+1)+K]: the first token whose cumulative weight exceeds u * total.
 *                   A residual with zero mass (only reachable through rounding) falls back to p.
 * Layout, fixed (tgt_offsets == drf_offsets == NULL): target [S*(K+1), V] (row s*(K+1)+k),
 *   draft [S*K, V] (row s*K+k), draft_tokens [S*K].
 * Layout, ragged (both offsets given, int32 [S+1] device arrays): sequence s has
 *   K_s = drf_offsets[s+1]-drf_offsets[s] <= K drafts, target rows tgt_offsets[s] ..
 *   tgt_offsets[s+1]-1 (K_s+1 rows), draft rows and draft tokens drf_offsets[s] .. +K_s-1.
 *   Inconsistent offsets are reported as SMCSD_ERR_RANGE through smcsd_check_status.
 * uniforms: [S*(K+1)] (positions k >= K_s of a ragged sequence are unused).
 * accept_len, out_token: int32 [S]. lse_tgt / lse_drf: optional float [rows] (NULL to skip),
 *   the natural-log normaliser of each scaled row, log sum_i exp(z_i / T).
 */
int sd_verify(const void* tgt_logits, const void* drf_logits, int dtype,
              const int32_t* draft_tokens, const int32_t* tgt_offsets, const int32_t* drf_offsets,
              int S, int K, int V, float temperature, const float* uniforms,
              int32_t* accept_len, int32_t* out_token, float* lse_tgt, float* lse_drf,
              void* ws, size_t ws_bytes, void* stream);

/*
 * SMC-SD reweight and bonus token ([SMC] sec. 2 steps 3-4; power target from [SMC] sec. 3).
 * Target pi = softmax(alpha * z_t / T) (alpha = 1 is plain p; alpha != 1 is the power target
 * p^alpha renormalised), draft q = softmax(z_d / T). For each particle s:
 *   logw[s] += sum_{k<K} ( log pi_k(x_k) - log q_k(x_k) )   (float in/out)
 *   bonus_token[s] = inverse-CDF draw from pi at target row K with uniforms[s]
 *   (the (K+1)-th token; its weight factor is pi/pi = 1).
 * Layout: target [S*(K+1), V], draft [S*K, V], draft_tokens [S*K], uniforms [S].
 * lse_tgt [S*(K+1)] / lse_drf [S*K]: optional normalisers (NULL to skip).
 */
int smc_reweight(const void* tgt_logits, const void* drf_logits, int dtype,
                 const int32_t* draft_tokens, int S, int K, int V, float temperature, float alpha,
                 const float* uniforms, float* logw, int32_t* bonus_token,
                 float* lse_tgt, float* lse_drf, void* ws, size_t ws_bytes, void* stream);

/*
 * SMC-SD reweight toward a tilted target ([SMC] sec. 3 "flexibility": modified targets such as
 * power sampling and reward-weighted decoding; sec. 5: reward optimisation and hard
 * constraints through the same importance weights). Arguments and layout as smc_reweight, plus:
 *   target = SMCSD_TARGET_TOKEN: smc_reweight's per-position target pi = softmax(alpha z_t / T).
 *   target = SMCSD_TARGET_SEQUENCE: the unnormalised power of the sequence probability,
 *     prod_t p_t(x_t)^alpha with p = softmax(z_t / T). The draft tokens are proposed by q and
 *     the (K+1)-th token b_s is drawn from p at target row K (with uniforms[s]), so
 *       logw[s] += sum_{k<K} ( alpha log p_k(x_k) - log q_k(x_k) ) + (alpha - 1) log p_K(b_s).
 *     alpha = 1 gives smc_reweight's result. lse_tgt then holds the normalisers at 1/T.
 *   log_reward: optional float [S] (NULL for none); logw[s] += reward_scale * log_reward[s].
 *     A NaN or infinite reward is SMCSD_ERR_NONFINITE (device side, smcsd_check_status);
 *     reward_scale must be finite when log_reward is given.
 * target other than the two values above: SMCSD_ERR_INVALID_ARG.
 */
int smc_reweight_tilted(const void* tgt_logits, const void* drf_logits, int dtype,
                        const int32_t* draft_tokens, int S, int K, int V, float temperature,
                        float alpha, int target, const float* log_reward, float reward_scale,
                        const float* uniforms, float* logw, int32_t* bonus_token,
                        float* lse_tgt, float* lse_drf, void* ws, size_t ws_bytes, void* stream);

/*
 * Draft-token sampling ([SMC] sec. 2 step 1: the draft model proposes K tokens per particle,
 * each drawn from its tempered distribution). For each of R rows of `logits` ([R, V], dtype as
 * above), with q_r = softmax(z_r / T):
 *   tokens[r] = the first token whose cumulative q_r exceeds uniforms[r] (inverse CDF, the same
 *               draw as the verify's final token);
 *   logq[r]   = log q_r(tokens[r]) (optional, NULL to skip), what a verify needs from the draft;
 *   lse[r]    = log sum_i exp(z_{r,i} / T) (optional).
 * uniforms: float [R]; tokens: int32 [R]; logq, lse: float [R]. ws: see
 * smcsd_workspace_size(SMCSD_OP_DRAFT_SAMPLE, R, 0, V). An all-masked or non-finite row is
 * SMCSD_ERR_NONFINITE (device side) and its token is reported as 0.
 */
int draft_sample(const void* logits, int dtype, int R, int V, float temperature,
                 const float* uniforms, int32_t* tokens, float* logq, float* lse,
                 void* ws, size_t ws_bytes, void* stream);

/*
 * Effective sample size and systematic resampling per group of N particles ([SMC] sec. 2
 * step 4; the textbook forms, in double precision):
 *   w_i = exp(logw_i - max logw), ess[g] = (sum w)^2 / sum w^2;
 *   resampled[g] = ess[g] < ess_threshold (strict);
 *   if resampled: C_i = (sum_{j<=i} w_j)/W with C_{N-1} = 1, v_j = (j + uniforms[g]) / N,
 *                 ancestors[g*N+j] = min{ i : C_i > v_j }, and logw of the group is set to 0;
 *   else ancestors[g*N+j] = j and logw is unchanged.
 * logw [G*N] float in/out; uniforms [G]; ancestors [G*N] (group-local indices); ess [G] and
 * resampled [G] may be NULL. ws: see smcsd_workspace_size(SMCSD_OP_ESS_RESAMPLE, G, 0, 0).
 */
int smc_ess_resample(float* logw, int G, int N, float ess_threshold, const float* uniforms,
                     int32_t* ancestors, float* ess, int32_t* resampled,
                     void* ws, size_t ws_bytes, void* stream);

/*
 * Paged-KV page-table remap ([SMC] sec. 3: resampling moves no KV data, only metadata).
 *   table_out[g*N+j][:] = table_in[g*N+a][:], a = ancestors[g*N+j] if resampled[g] (or if
 *   resampled == NULL), else a = j;
 *   refcount (optional, int32 [num_pages]) is rebuilt: refcount[p] = entries of table_out == p.
 * Tables are int32 [G*N, pages_per_seq]; table_out must not alias table_in. -1 marks an empty
 * slot (copied, not counted). Other ids outside [0, num_pages) or ancestors outside [0, N) are
 * reported as SMCSD_ERR_RANGE through smcsd_check_status (the entry is then not counted).
 */
int kv_pagetable_remap(const int32_t* ancestors, const int32_t* resampled, int G, int N,
                       const int32_t* table_in, int32_t* table_out, int pages_per_seq,
                       int32_t* refcount, int num_pages, void* ws, size_t ws_bytes, void* stream);

/*
 * pacer_block_stop with position embeddings ([PACER] Methodik 1: the pre-verification layer
 * reads the block's hidden states together with position embeddings; the ablation under
 * "Ergebnisse" finds them essential). pos_emb: bf16 [max_blocks*b, d], row j for draft position
 * j, shared by all sequences (NULL: pacer_block_stop). The score of position j is
 *   score_j = sigmoid(w . (h_j + pos_emb_j) + c);
 * everything else is as in pacer_block_stop below.
 */
int pacer_block_stop_pos(const void* hidden, const void* w, const void* pos_emb, float c, int S,
                         int b, int max_blocks, int d, float t0, float rho, int32_t* lengths,
                         float* block_scores, int32_t* tgt_offsets, int32_t* drf_offsets,
                         void* ws, size_t ws_bytes, void* stream);

/*
 * PACER blockwise stop ([PACER] Methodik 1-3), with the pre-verification layer modelled as
 * score_j = sigmoid(w . h_j + c) over hidden states h (bf16 [S, max_blocks*b, d]) and a head
 * w (bf16 [d]):
 *   t = t0; for block i: m_i = mean of the b scores; if m_i < t: length = (i+1)*b, stop;
 *   else t = t * rho. No stop: length = max_blocks*b.
 * Only the blocks up to the stop are read. lengths: int32 [S]. block_scores: optional float
 * [S*max_blocks] (m_i of scored blocks, -1 after the stop). tgt_offsets / drf_offsets: optional
 * int32 [S+1], filled with the ragged layout that sd_verify takes for these lengths
 * (prefix sums of length+1 and of length).
 */
int pacer_block_stop(const void* hidden, const void* w, float c, int S, int b, int max_blocks,
                     int d, float t0, float rho, int32_t* lengths, float* block_scores,
                     int32_t* tgt_offsets, int32_t* drf_offsets,
                     void* ws, size_t ws_bytes, void* stream);

/*
 * One whole SMC-SD step in one pass over the logits ([SMC] sec. 2 steps 3-4 and sec. 3):
 * smc_reweight for S = G*N particles, then per group the effective sample size, systematic
 * resampling and the page-table remap, with the same semantics as the three calls above
 * (bonus_uniforms [G*N], resample_uniforms [G]). table_in / table_out / refcount may all be
 * NULL to skip the remap (pages_per_seq and num_pages are then ignored). ess and resampled
 * may be NULL.
 */
int smc_step(const void* tgt_logits, const void* drf_logits, int dtype,
             const int32_t* draft_tokens, int G, int N, int K, int V, float temperature,
             float alpha, const float* bonus_uniforms, float* logw, int32_t* bonus_token,
             float ess_threshold, const float* resample_uniforms, int32_t* ancestors,
             float* ess, int32_t* resampled, const int32_t* table_in, int32_t* table_out,
             int pages_per_seq, int32_t* refcount, int num_pages,
             void* ws, size_t ws_bytes, void* stream);

/*
 * smc_step with the draft's log-probabilities in place of its logits ([SMC] sec. 2 steps 1 and 3:
 * the draft proposes each token from its own distribution, and the weight needs only the
 * probability the draft gave the proposed token). drf_logq: float [G*N*K], log q_k(x_k) of draft
 * token draft_tokens[s*K+k] under the draft's tempered distribution at `temperature`, as
 * draft_sample returns it when it draws the tokens. The step then reads only the target logits
 * (target [G*N*(K+1), V]); its results are those of smc_step on draft logits whose normalised
 * log-probabilities at the draft tokens equal drf_logq:
 *   logw[s] += sum_{k<K} ( log pi_k(x_k) - drf_logq[s*K+k] ),
 * with pi = softmax(alpha z_t / T), then the bonus token, ESS, resampling and remap as smc_step.
 * The values of drf_logq are taken as given (non-positive and finite for a real distribution; a
 * NaN makes the particle's weight NaN, reported as SMCSD_ERR_NONFINITE by the group's ESS).
 * Arguments otherwise as smc_step; ws: smcsd_workspace_size(SMCSD_OP_SMC_STEP, G*N, K, V).
 */
int smc_step_logq(const void* tgt_logits, int dtype, const int32_t* draft_tokens,
                  const float* drf_logq, int G, int N, int K, int V, float temperature, float alpha,
                  const float* bonus_uniforms, float* logw, int32_t* bonus_token,
                  float ess_threshold, const float* resample_uniforms, int32_t* ancestors,
                  float* ess, int32_t* resampled, const int32_t* table_in, int32_t* table_out,
                  int pages_per_seq, int32_t* refcount, int num_pages, void* ws, size_t ws_bytes,
                  void* stream);

/*
 * smc_step toward a tilted target: target, log_reward and reward_scale as in
 * smc_reweight_tilted; everything else as in smc_step. The reward enters the log-weights
 * before the group's ESS and resampling.
 */
int smc_step_tilted(const void* tgt_logits, const void* drf_logits, int dtype,
                    const int32_t* draft_tokens, int G, int N, int K, int V, float temperature,
                    float alpha, int target, const float* log_reward, float reward_scale,
                    const float* bonus_uniforms, float* logw, int32_t* bonus_token,
                    float ess_threshold, const float* resample_uniforms, int32_t* ancestors,
                    float* ess, int32_t* resampled, const int32_t* table_in, int32_t* table_out,
                    int pages_per_seq, int32_t* refcount, int num_pages,
                    void* ws, size_t ws_bytes, void* stream);

/*
 * smc_step without a workspace argument. None of the pages has a counterpart: this is an
 * interface variant of smc_step (same step, same arguments and results, minus ws / ws_bytes)
 * for callers that cannot allocate device memory for a workspace, such as a host program with no
 * device allocator or a plugin that must not use its host's allocator. The call allocates
 * nothing: its scratch is a device area of a little over 32 MiB owned by this library (SMCSD_STATIC_SCRATCH_BYTES),
 * set aside when the library's device code is loaded.
 *   status: optional int32 device pointer; receives this call's device-side status (SMCSD_OK or
 *     a negative SMCSD_* code, as smcsd_check_status would report), written in stream order.
 *     Without it, device-side errors of the call are not reported.
 * Returns SMCSD_ERR_WORKSPACE, before any device work, when the shape needs more scratch than the
 * area holds (smcsd_workspace_size(SMCSD_OP_SMC_STEP, G*N, K, V) > SMCSD_STATIC_SCRATCH_BYTES),
 * and the host-side errors of smc_step otherwise.
 * Each call clears, on the stream, the part of the scratch that must start at zero. All calls on
 * one device share the one area: calls whose device work may overlap (different streams, or
 * several host threads without ordering between them) race on it and give wrong results, so
 * order them, for instance on one stream. The first call on a device looks the area's address up
 * with that device current; make that first call before any stream capture begins.
 */
#define SMCSD_STATIC_SCRATCH_BYTES ((32u << 20) + (32u << 10))
int smc_step_static(const void* tgt_logits, const void* drf_logits, int dtype,
                    const int32_t* draft_tokens, int G, int N, int K, int V, float temperature,
                    float alpha, const float* bonus_uniforms, float* logw, int32_t* bonus_token,
                    float ess_threshold, const float* resample_uniforms, int32_t* ancestors,
                    float* ess, int32_t* resampled, const int32_t* table_in, int32_t* table_out,
                    int pages_per_seq, int32_t* refcount, int num_pages, int32_t* status,
                    void* stream);

/* ---------------------------------------------------------------------------------------------
 * The rest of a speculative step on the device: page tables and slots for the step's tokens, their
 * keys and values in the paged cache, attention of the drafted tokens over it, and the logits
 * before sampling or verify. The pages describe these steps ([SMC] sec. 2 step 2: one target pass
 * scores every particle's drafts; sec. 3: page-based KV with metadata-only resampling; sec. 5:
 * hard constraints) without formulas; the rules are stated here.
 *
 * Shared conventions
 *   - S sequences; sequence s has n_s new tokens, its NODES: the last committed token and the
 *     drafts after it, as a chain or a tree. Fixed layout (node_offsets == NULL): n_s = T, node t of
 *     sequence s is row s*T+t. Ragged: node_offsets int32 [S+1] (ascending from 0), rows
 *     node_offsets[s] .. node_offsets[s+1]-1, n_s <= T. R is the number of rows (S*T if fixed);
 *     offsets that do not fit R or T are SMCSD_ERR_RANGE (device side). Rows that no sequence has (before
 *     node_offsets[0] or from node_offsets[S] on, as where R is padded for a captured graph) get the
 *     slot -1 from kv_slot_map; the other operators leave their outputs as they are.
 *   - Paged cache: K and V each [num_pages, Hkv, page_size, D], contiguous, 16-byte aligned;
 *     page_size a power of two of 8 .. 256. Tables int32 [S, pages_per_seq], -1 = no page. Position x
 *     of a sequence is in page table[s][x / page_size] at offset x % page_size; its SLOT is
 *     page * page_size + offset (int64: a cache may have more than 2^31 slots).
 *   - Node j of sequence s is at position ctx_len[s] + j, ctx_len int32 [S] being the tokens already
 *     in the cache.
 *   - A node mask is uint32 [R, (T+31)/32]: bit j of row r says that the row's node sees node j of
 *     its own sequence (bits past n_s are ignored). NULL is a chain: node t sees nodes 0 .. t.
 * ------------------------------------------------------------------------------------------- */

/*
 * Page tables and slots for the new tokens of every sequence, with copy-on-write of shared pages
 * ([SMC] sec. 3: after a resampling several particles hold the same pages). For s = 0, 1, ... and
 * every page index j that the sequence writes, ctx_len[s]/page_size <= j <
 * ceil((ctx_len[s]+n_s)/page_size) (none if n_s = 0), with id = table_in[s][j]:
 *   id == -1               a free page is taken;
 *   refcount_in[id] > 1    a free page is taken in its place and refcount_out[id] drops by one; if j
 *                          is the first of them and ctx_len[s] % page_size > 0, its filled part has
 *                          to be copied: copy_src[s] = id, copy_dst[s] = the new page;
 *   otherwise              the page is kept.
 * Free pages are those with refcount_in == 0, taken in ascending order; a taken page's
 * refcount_out is 1. Everything else is copied from table_in / refcount_in (the outputs must not
 * alias them). slots int64 [R], -1 for every row of a sequence that is refused; copy_src, copy_dst int32 [S] (-1: no copy). The result does not
 * depend on the order of execution.
 * Device-side errors: SMCSD_ERR_RANGE (a negative length, more positions than the table has, ids or
 * offsets out of range), SMCSD_ERR_PAGES (too few free pages; the pages that are missing read -1 and
 * so do their slots).
 */
int kv_slot_map(const int32_t* ctx_len, const int32_t* node_offsets, int S, int T, int R,
                const int32_t* table_in, int32_t* table_out, int pages_per_seq, int page_size,
                const int32_t* refcount_in, int32_t* refcount_out, int num_pages, int64_t* slots,
                int32_t* copy_src, int32_t* copy_dst, void* ws, size_t ws_bytes, void* stream);

/*
 * Writes the new tokens' keys and values into the paged cache, and the copies that kv_slot_map
 * asked for. k_new / v_new: R tokens of [Hkv, D] each, token_stride elements from one token to the
 * next (both may be slices of one projection's output), 16-byte aligned, token_stride * element
 * size and D * element size multiples of 16. slots int64 [R]; a negative slot writes nothing.
 * copy_src / copy_dst int32 [S] with ctx_len int32 [S] (all three or none): where copy_src[s] >= 0
 * the first ctx_len[s] % page_size positions of that page go to copy_dst[s], for every head. Slots
 * must be distinct, and no slot or destination page lie in a page that is copied from.
 * Slots or pages outside the cache are SMCSD_ERR_RANGE (device side) and write nothing.
 */
int kv_append(const void* k_new, const void* v_new, int dtype, int R, int Hkv, int D,
              long long token_stride, const int64_t* slots, const int32_t* copy_src,
              const int32_t* copy_dst, const int32_t* ctx_len, int S, void* k_cache, void* v_cache,
              int page_size, int num_pages, void* ws, size_t ws_bytes, void* stream);

/*
 * Node mask of trees given by parents: parents int32 [R], the index within its own sequence of the
 * node that a node follows (smaller than its own), -1 for a first node. mask uint32
 * [R, (T+31)/32]: bit j is set for the node itself and for its ancestors. A parent out of range is
 * SMCSD_ERR_RANGE (device side).
 */
int tree_mask(const int32_t* parents, const int32_t* node_offsets, int S, int T, int R,
              uint32_t* mask, void* ws, size_t ws_bytes, void* stream);

/* Scratch bytes of tree_attention for these sizes (0 if they are not supported). */
size_t tree_attention_workspace_size(int S, int N, int T, int Hq, int Hkv, int D);

/*
 * Attention of every sequence's nodes over its cached tokens and over the nodes that they see
 * ([SMC] sec. 2 step 2: the target scores all drafted tokens of all particles in one pass). For row
 * r (node t of sequence s) and query head h, which reads the keys of head h / (Hq/Hkv):
 *   z_x = scale * q[r,h] . K_x   for x < ctx_len[s] and for x = ctx_len[s]+j with bit j of the mask,
 *   out[r,h] = sum_x softmax(z)_x V_x,   lse[r,h] = log sum_x exp(z_x).
 * The nodes' own keys and values are already in the cache (kv_append). A row that sees nothing gives
 * out = 0 and lse = -inf. What the cache holds at positions that no row sees (unwritten slots,
 * pages past the end) may be anything, NaN included; a NaN or infinity in a node reaches only the
 * rows that see that node.
 * Sequences come in groups of N (S a multiple of N; N = 1: none): pages that all sequences of a group
 * have in common at the start of their tables (the prompt, common ancestors) are read once for the
 * group. N changes no result beyond the order of the sums.
 * q: R rows of [Hq, D], q_stride elements apart (16-byte aligned, q_stride * element size a multiple
 * of 16); out [R, Hq, D] in the same type; lse float [R, Hq] (NULL to skip). D is 64 or 128, Hq a
 * multiple of Hkv. dtype is that of q, the caches and out. Products are accumulated in float32;
 * for bf16 the weights exp(z - max) are rounded to bf16 for the product with V.
 * Device-side errors: SMCSD_ERR_RANGE (lengths, offsets or page ids out of range).
 */
int tree_attention(const void* q, long long q_stride, const void* k_cache, const void* v_cache,
                   int dtype, int num_pages, int page_size, const int32_t* table, int pages_per_seq,
                   const int32_t* ctx_len, const int32_t* node_offsets, int S, int N, int T, int R,
                   const uint32_t* mask, int Hq, int Hkv, int D, float scale, void* out, float* lse,
                   void* ws, size_t ws_bytes, void* stream);

/*
 * Penalties, biases and grammar masks on logits, before draft_sample or a verify ([SMC] sec. 5:
 * constraints). Row r (node t of sequence s) predicts the token after that node. count_r(v) is the
 * number of times that token v stands in the sequence's history, hist_tokens[hist_offsets[s] ..
 * hist_offsets[s+1]-1], and among the node_tokens of the nodes that the row sees. In float32, rounded
 * once:
 *   z = logits[r, v];  if count > 0: z = z > 0 ? z / repetition[s] : z * repetition[s];
 *   z -= frequency[s] * count;  if count > 0: z -= presence[s];
 *   z += bias_values[i] for the last i of bias_offsets[s] .. bias_offsets[s+1]-1 with
 *        bias_tokens[i] == v;
 *   z = -inf if bit v of allowed[r] is clear.
 * logits, out [R, V] of dtype; out may be logits itself (nothing but changed values is then written
 * back). Each of these may be NULL to leave its part out: node_tokens int32 [R], mask (with
 * node_tokens: chain), hist_tokens int32 [n_hist] with hist_offsets int32 [S+1] (one history for
 * all three penalties), repetition (> 0), presence, frequency float [S] (1, 0, 0), bias_tokens int32 /
 * bias_values float [n_bias] with bias_offsets int32 [S+1], allowed uint32 [R, (V+31)/32]. A token
 * of -1 in hist_tokens, node_tokens or bias_tokens counts for nothing; others outside [0, V) are
 * SMCSD_ERR_RANGE (device side), as are offsets that descend, are negative or pass n_hist or n_bias.
 * S is at most 65535. A row whose mask allows nothing is -inf throughout, which the verify then
 * reports.
 */
int logits_process(const void* logits, void* out, int dtype, int R, int V, int S, int T,
                   const int32_t* node_offsets, const int32_t* node_tokens, const uint32_t* mask,
                   const int32_t* hist_tokens, const int32_t* hist_offsets, int n_hist,
                   const float* repetition, const float* presence, const float* frequency,
                   const int32_t* bias_tokens, const float* bias_values, const int32_t* bias_offsets,
                   int n_bias, const uint32_t* allowed, void* ws, size_t ws_bytes, void* stream);

/* ---------------------------------------------------------------------------------------------
 * Beam search, the pages' housekeeping, and what a draft learns from. None of the pages has these steps; they
 * stand beside the ones above: a beam search (or the growing of a draft tree) over the same logits, with
 * its sequences' pages and states following their ancestors as after a resampling; requests that come, fork and
 * end in the same cache; and the loss that draws the draft's distribution to the target's, on which the
 * acceptance rate rests.
 *
 * Shared conventions
 *   - G groups of N sequences (beams); sequence i of group g is row g*N+i. Ancestors are group-local, as
 *     smc_ess_resample's, and go to kv_pagetable_remap (with resampled == NULL) as they are.
 *   - Tables int32 [S, pages_per_seq] and refcounts int32 [num_pages] as above; -1 = no page. Tables and refcounts are
 *     written anew: outputs must not overlap inputs.
 * ------------------------------------------------------------------------------------------- */

/*
 * The M best continuations of each group's beams. With L_i = log sum_v exp(z_iv / T) of row i of `logits`,
 * candidate (i, v) has the score scores[i] + z_iv / T - L_i. A beam with finished[i] != 0 has one
 * candidate in place of V: the token pad_token, with the score scores[i] as it is; its logits are not
 * read. A beam with a score of -inf has none, and its logits are not read. For m = 0 .. M-1, the m-th
 * best candidate of group g in the order of score (falling), beam, token:
 *   tokens[g*M+m] = v;  ancestors[g*M+m] = i (group-local);  out_scores[g*M+m] = its score;
 *   out_finished[g*M+m] = 1 if the beam was finished or v == eos_token, else 0.
 * Where there are fewer than M candidates, the remaining places get pad_token, 0, -inf and 1. Masked tokens of -inf
 * are none, nor are those whose score (or z less the row's largest) lies below float32's range: a token masked with the
 * type's lowest value is a candidate with T >= 1, and none with T < 1. A row with nothing but -inf has no candidate; that is not an error here.
 * out_scores are good to 6e-6 (2e-7 as a rule: the sum's hardware exponentials) and half a step of float32, and carry the error of the
 * scores that came in: over a search it adds up by the step.
 * The order is that of the scores' real values, up to 1e-9 or so: candidates of one beam are ordered by their logits
 * exactly, those of two beams by sums that are computed again, to 2e-10, where hardware exponentials could
 * not tell them apart (a slower path: some 30 us for each such row of 128256). Beams with equal scores and
 * equal rows are exactly equal.
 * N = 1 and scores == NULL gives the M largest log-probabilities of each row: a teacher's top logits, or the children
 * of a draft tree's node.
 * logits [G*N rows, row_stride elements apart, V used], aligned to their type; scores float [G*N] (NULL: 0);
 * finished int32 [G*N] (NULL: none); eos_token < 0: none; tokens, ancestors int32, out_scores float,
 * out_finished int32 (NULL to skip) [G*M]; outputs must not overlap scores and finished. N and
 * M are at most 256, and a group's N rows of V logits at most 160 MB. ws: smcsd_workspace_size(SMCSD_OP_BEAM_SELECT, G*N, 0, V).
 * Device-side errors: SMCSD_ERR_NONFINITE (NaN or +inf in logits that are read, or in scores; such a beam has no candidate).
 */
int beam_select(const void* logits, long long row_stride, int dtype, int G, int N, int V, int M,
                float temperature, const float* scores, const int32_t* finished, int pad_token,
                int eos_token, int32_t* tokens, int32_t* ancestors, float* out_scores,
                int32_t* out_finished, void* ws, size_t ws_bytes, void* stream);

/*
 * Rows of per-sequence states by ancestors: for each of `count` tensors, row g*M+m of dst = row
 * g*N + ancestors[g*M+m] of src (M = N after a resampling or a step of beam search; N = 1: copies for M beams).
 * src, dst and row_bytes are HOST arrays of `count` (at most 64) device pointers and sizes; a source of G*N and a
 * destination of G*M rows of row_bytes each, contiguous, of any type. No destination may overlap a source (its own or another
 * tensor's), another destination or the ancestors. An ancestor outside [0, N) is SMCSD_ERR_RANGE (device side) and leaves its rows as they are.
 */
int state_reorder(const void* const* src, void* const* dst, const long long* row_bytes, int count,
                  const int32_t* ancestors, int G, int N, int M, void* ws, size_t ws_bytes, void* stream);

/*
 * Forks: every sequence s becomes a copy of sequence parents[s] as table_in holds it, of its first
 * ceil(lengths[s] / page_size) pages (lengths == NULL, or a length of INT32_MAX: all of them; pages past the
 * end of the table: none); parents[s] == s keeps it (cut to its length), -1 frees it. Pages are shared, not copied:
 *   refcount_out[id] = refcount_in[id] + (entries of table_out == id) - (entries of table_in == id),
 * so holders other than the table (a prefix cache) keep their share. A partly filled last page is shared too:
 * kv_slot_map copies it when one of its holders writes. parents, lengths int32 [S].
 * Device-side errors: SMCSD_ERR_RANGE for a parent outside [-1, S) or a negative length (the sequence is kept as it is), for page
 * ids outside [-1, num_pages) (copied, not counted), and for a page whose count ends below zero, or falls below it on the way (counts
 * change in any order: where an id is both let go and taken and its count was too small, the error may be reported or not).
 */
int kv_fork(const int32_t* parents, const int32_t* lengths, int S, const int32_t* table_in,
            int32_t* table_out, int pages_per_seq, int page_size, const int32_t* refcount_in,
            int32_t* refcount_out, int num_pages, void* ws, size_t ws_bytes, void* stream);

/*
 * Lets go of every sequence's pages past its length: kv_fork with every sequence its own parent (0: all of
 * them, as for a sequence that has ended; the accepted length: those of rejected drafts).
 */
int kv_free(const int32_t* lengths, int S, const int32_t* table_in, int32_t* table_out,
            int pages_per_seq, int page_size, const int32_t* refcount_in, int32_t* refcount_out,
            int num_pages, void* ws, size_t ws_bytes, void* stream);

/*
 * Moves the pages in use (refcount_in > 0) to the front of the cache with as few moves as there can be: with U pages in
 * use, the k-th (ascending) page in use from page U on takes the k-th free page below U.
 *   src[k], dst[k], k < counts[0]: the moves, for kv_copy_pages (-1 behind them); counts[1] = U;
 *   table_out, refcount_out: table_in and refcount_in with the pages' new ids; pages from U on are free.
 * src, dst int32 [num_pages / 2] (NULL for one page), counts int32 [2]; no output may overlap another. Nothing but counts and tables is touched: the caller
 * copies the pages of every layer. ws: smcsd_workspace_size(SMCSD_OP_KV_COMPACT, 1, 0, num_pages).
 * Device-side errors: SMCSD_ERR_RANGE (a negative refcount, taken as free; table entries outside [-1, num_pages) or of free pages,
 * left as they are).
 */
int kv_compact(int S, const int32_t* table_in, int32_t* table_out, int pages_per_seq,
               const int32_t* refcount_in, int32_t* refcount_out, int num_pages, int32_t* src,
               int32_t* dst, int32_t* counts, void* ws, size_t ws_bytes, void* stream);

/*
 * Copies whole pages within each of n_caches caches: page src[i] to page dst[i] for i < n, or i < *count (int32, device,
 * NULL: n). caches: HOST array of at most 256 device pointers (every layer's keys and values), 16-byte aligned, each
 * num_pages pages of page_bytes (a multiple of 16). An entry with src and dst both negative is passed over. Destinations must be distinct,
 * and none of them a source of the same call. Pages out of range are SMCSD_ERR_RANGE (device side) and copy
 * nothing, as does a count outside [0, n].
 */
int kv_copy_pages(void* const* caches, int n_caches, long long page_bytes, int num_pages,
                  const int32_t* src, const int32_t* dst, int n, const int32_t* count, void* ws,
                  size_t ws_bytes, void* stream);

/*
 * Distillation from a teacher's top logits: for each of R rows, q = softmax(z / T) of the draft's logits, and the
 * teacher's probabilities p_k of the row's listed tokens top_tokens[r*K+k] (-1: none), from top_values:
 *   rest == 0: p = softmax of the row's values (log-probabilities or logits): the list stands for everything, p_r = 0;
 *   rest == 1: p_k = exp(value), log-probabilities over the whole vocabulary; p_r = 1 - sum_k p_k is
 *              the share of all tokens that are not listed, as one event of probability q_r = 1 - sum of the listed q.
 *              p_r < 2^-21, which roundings of the values may make of 0, is taken as 0.
 *   loss[r] = sum_k p_k (log p_k - log q_k) + p_r (log p_r - log q_r)             (terms with p = 0 are 0)
 *   dlogits[r, v] = weight[r] * dloss[r] / dz_v
 *                 = weight[r] / T * (P q_v - p_v) for a listed v, weight[r] / T * q_v (P - p_r / q_r) for others,
 * P = sum_k p_k + p_r. weight is the gradient that comes to loss[r] (NULL: 1); it does not scale the loss. A token that is listed
 * several times has the sum of its entries' p in the gradient. A row whose list is empty, or holds nothing but values of -inf, has
 * a loss and a gradient of 0, whatever its logits are (padding). q_v = 0 for a masked token; a loss is +inf where p > 0 meets q = 0.
 * Either output may be NULL, loss for the backward pass alone and dlogits for the forward one; both together read the logits once,
 * as each alone does. logits, dlogits: rows row_stride and dlogits_stride elements apart, V used, of dtype, aligned to
 * it; dlogits may be logits (with one stride), else they must not overlap (rows may lie
 * between one another's); nor may either output overlap the lists, weight or the other output, nor loss the logits. top_tokens int32, top_values float [R, K], K at most 256;
 * weight, loss float [R]. V times the element size is at most 1638368 bytes. Sums are float32, the gradient is rounded once. (In torch the
 * call takes no part in autograd: the loss has no graph, and the gradient goes on by logits.backward(dlogits).)
 * Device-side errors: SMCSD_ERR_NONFINITE (NaN or +inf in logits or values, a row of -inf), SMCSD_ERR_RANGE (a token outside
 * [-1, V), taken as none).
 */
int distill_loss(const void* logits, long long row_stride, int dtype, int R, int V,
                 const int32_t* top_tokens, const float* top_values, int K, float temperature,
                 int rest, const float* weight, float* loss, void* dlogits, long long dlogits_stride,
                 void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* SMCSD_H */

/*
 * tsr.h - C ABI of the batched logits-to-token sampler for AMD Instinct MI355X
 * (gfx950): temperature, softmax, top-k, top-p, min-p, renormalisation and a
 * Philox draw per row, and the speculative-decoding verify step.
 *
 * Pages this interface implements:
 *  [P1] fareedkhan-dev.github.io "Inference: Sampling, the KV Cache,
 *       Speculative Decoding and int8" - "Picking the next token" (the knobs
 *       and their order, the min-p rule), "Speculative decoding".
 *  [P2] gowda.ai "Chapter 39 Decoding & Speculative Sampling" - 39.1 (greedy),
 *       39.2 (filters as transforms, eq. 39.2, Listing 39.2), 39.3 (an empty
 *       allowed set is an invalid state), 39.4 (eqs. 39.3-39.4, Listing 39.4).
 *  [P3] brentwoodlivery.com "Speculative decoding - Hinglish notes" - "The
 *       Algorithm (Step-by-Step)", "Batching Speculation", "Temperature and
 *       Sampling".
 *  [P4] scratchllm.com "Efficient Inference & Compression" - "Speculative
 *       decoding".
 *  [P5] legost.in "Choosing the next word" - "Temperature", "Cutting off the
 *       tail: top-k and top-p", "Where the randomness comes from".
 *
 * Conventions shared by every call
 *  - All tensors are caller-owned DEVICE memory on the handle's device. The
 *    library never allocates, frees or retains them.
 *  - Calls enqueue work on `hip_stream` (a hipStream_t; NULL = the default
 *    stream) and return without waiting. Outputs are valid once the stream
 *    has reached that point.
 *  - Argument errors are returned synchronously and nothing is enqueued.
 *    Per-row data errors (NaN/+inf logits, an all -inf row, a draft token out
 *    of range) are reported per row through a status array, with token -1.
 *    A failed launch returns TSR_EDEVICE. No C++ exception crosses this ABI.
 *  - Logits are float32 or bfloat16, row-major; each row holds `vocab`
 *    elements. Pointers must be aligned to the element size. Rows may start
 *    at any element boundary (a contiguous batch of an odd vocab too): they
 *    are read in 16-byte loads at whatever alignment they have, under the
 *    unaligned access mode the HSA runtime sets, and no byte outside a row
 *    is read.
 *  - A handle is not thread-safe. Two calls on one handle may run on different
 *    streams at the same time unless they use the same workspace of it:
 *    spec_verify and tree_verify share one, beam_step and verify_probs have
 *    one each.
 */
#ifndef TSR_H_
#define TSR_H_

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct tsr_ctx* tsr_handle;

/* Return codes. */
enum {
  TSR_OK = 0,
  TSR_EINVAL = 1,        /* bad argument: null pointer, size or parameter out of range */
  TSR_ENOMEM = 2,        /* workspace allocation failed in sampler_init */
  TSR_EDEVICE = 3,       /* HIP runtime error (device selection, launch) */
  TSR_EUNSUPPORTED = 4   /* a size this build has no kernel for */
};

/* Element types of the logits. */
enum { TSR_F32 = 0, TSR_BF16 = 1 };

/* How top-p combines with top-k [P2 Listing 39.2 vs P5's generation loop].
 * JOINT: every filter reads the same post-temperature p; the kept set is the
 *   intersection of the filters' sets and is renormalised once (eq. 39.2).
 * SEQUENTIAL: top-p measures mass relative to the tokens top-k kept. */
enum { TSR_JOINT = 0, TSR_SEQUENTIAL = 1 };

/* Per-row status. */
enum {
  TSR_ROW_OK = 0,
  TSR_ROW_NONFINITE = 1, /* the row holds NaN or +inf */
  TSR_ROW_EMPTY = 2,     /* every logit is -inf: the kept set is empty [P2 39.3] */
  TSR_ROW_BADTOKEN = 3,  /* verify only: a draft token outside [0, vocab) */
  TSR_ROW_BADPARAM = 4   /* the row's own parameters (tsr_constraints.row_params) are invalid */
};

/* Sampling parameters, one set per call [P1 "Picking the next token"].
 *  temperature: 0 = greedy (the lowest token id among the maximal logits);
 *               otherwise >= 1e-30, and p = softmax(logits / temperature).
 *               Not clamped. Negative or non-finite values are TSR_EINVAL.
 *  top_k:       keep every token with fewer than top_k strictly larger
 *               logits (ties with the k-th value stay); <= 0 or >= vocab: off.
 *  top_p:       keep the tie groups, in descending logit order, whose mass
 *               strictly above them is below top_p (times the top-k kept mass
 *               in SEQUENTIAL mode); the top group always stays. >= 1: off;
 *               < 0 or non-finite: TSR_EINVAL.
 *  min_p:       keep p_i >= min_p * max_j p_j; active iff 0 < min_p < 1.
 *  filter_mode: TSR_JOINT or TSR_SEQUENTIAL.
 * The kept set S always has the form {i : logit_i >= tau} and excludes -inf
 * logits; the draw renormalises over S (eq. 39.2). */
typedef struct {
  double temperature;
  int32_t top_k;
  double top_p;
  double min_p;
  int32_t filter_mode;
} tsr_params;

/* Optional per-row diagnostics for sample_rows; every pointer may be NULL.
 *  status      [rows]        TSR_ROW_* per row.
 *  kept_count  [rows]        |S| (0 on bad rows).
 *  threshold   [rows]        the smallest kept logit (as float32).
 *  kept_mass   [rows]        sum over S of softmax(logits / T), in (0, 1].
 *  probs       [rows][vocab] the renormalised distribution p~ (eq. 39.2),
 *                            0 outside S (all 0 on bad rows). Written by an
 *                            extra pass: meant for validation, not for the
 *                            timed hot path.
 * A greedy row (temperature 0) reports p~ as the point mass at its token:
 * kept_count 1, threshold the row's largest logit, kept_mass 1, probs one-hot. */
typedef struct {
  int32_t* status;
  int32_t* kept_count;
  float* threshold;
  double* kept_mass;
  float* probs;
} tsr_diag;

/* Create a handle on `device` and allocate its workspace once.
 *  max_rows, max_vocab, max_k bound later calls (max_k: the largest draft
 *  length K of spec_verify). The Philox4x32-10 key is `seed` (low word first);
 *  the counter of each draw is (row, position | domain << 16, step low, step
 *  high), so a token depends only on (seed, row, position, step) and the
 *  parameters [P5 "Where the randomness comes from"].
 *  Returns TSR_OK and writes *out, or an error code with *out = NULL. */
int sampler_init(tsr_handle* out, int device, int max_rows, int max_vocab, int max_k,
                 uint64_t seed);

/* Free the handle and its workspace. NULL is accepted. Waits for the device. */
int sampler_destroy(tsr_handle h);

/* Greedy decoding [P2 39.1]: out_tokens[r] = the lowest id among the maximal
 * logits of row r. logits[r] starts at logits + r * row_stride elements.
 * out_status (nullable, [rows]) gets TSR_ROW_*; bad rows get token -1. */
int greedy_argmax(tsr_handle h, const void* logits, int dtype, int rows, int vocab,
                  int64_t row_stride, int32_t* out_tokens, int32_t* out_status,
                  void* hip_stream);

/* The sampler [P1 "Picking the next token"; P2 39.2; P5]. For each row r:
 * z = logits[r] / T, p = softmax(z), the kept set S by top-k, top-p and
 * min-p (see tsr_params), p~ = p 1{S} / sum_S p (eq. 39.2), then one draw by
 * inverse CDF: u = w0 * 2^-32 with w0 the first Philox word of counter
 * (r, 0, step), and the token is the first kept id, in ascending id order,
 * whose running total of p~ exceeds u. temperature 0 gives greedy_argmax.
 * logits[r] starts at logits + r * row_stride elements (row_stride >= vocab).
 * diag may be NULL. */
int sample_rows(tsr_handle h, const void* logits, int dtype, int rows, int vocab,
                int64_t row_stride, const tsr_params* params, uint64_t step,
                int32_t* out_tokens, const tsr_diag* diag, void* hip_stream);

/* The sampler restricted to an allowed-token set (constrained decoding)
 * [P2 39.3: the disallowed logits become -inf before the softmax, every step;
 * an empty allowed set is an invalid state], with the log-probability of each
 * drawn token [P1 "Picking the next token": generation can return it].
 *  allowed [rows][allowed_stride] uint32 words (nullable: every token is
 *      allowed, and the call equals sample_rows): token i of row r is allowed
 *      iff bit (i % 32) of allowed[r * allowed_stride + i / 32] is set; bits
 *      of ids >= vocab are ignored. allowed_stride >= ceil(vocab / 32); the
 *      pointer is 4-byte aligned. Disallowed logits are replaced by -inf
 *      before any other step, so a NaN or +inf there does not make the row
 *      TSR_ROW_NONFINITE, and a row with no allowed finite logit is
 *      TSR_ROW_EMPTY (token -1).
 *  out_logprob [rows] float32 (nullable): log p~(token) of eq. 39.2 over the
 *      masked and filtered distribution, i.e. (z_tok - M) / T minus the log
 *      of sum over S of exp((z - M) / T); 0 for greedy rows (temperature 0)
 *      and NaN for rows whose status is not TSR_ROW_OK.
 * Every other argument, and the draw itself (the same uniform of counter
 * (r, 0, step)), is as in sample_rows: the call computes what sample_rows
 * computes for logits whose disallowed entries are -inf. */
int sample_rows_masked(tsr_handle h, const void* logits, int dtype, int rows, int vocab,
                       int64_t row_stride, const uint32_t* allowed, int64_t allowed_stride,
                       const tsr_params* params, uint64_t step, int32_t* out_tokens,
                       float* out_logprob, const tsr_diag* diag, void* hip_stream);

/* Per-row inputs applied to the logits before temperature and the filters
 * (device memory; every pointer may be NULL, a NULL struct means none).
 *  allowed, allowed_stride: the allowed-token bitmask, laid out and applied
 *      as in sample_rows_masked [P2 39.3].
 *  history [rows][history_stride] int32: the look-back window of each row,
 *      its last history_len token ids (0 <= history_len <= 64,
 *      history_stride >= history_len); ids outside [0, vocab) are padding.
 *  repetition_penalty: r, finite and >= 1 (TSR_EINVAL otherwise when a
 *      window is given). Every distinct id of the window has its logit
 *      rescaled once, z / r if z > 0, z * r otherwise, before anything else
 *      [P5 "The repetition penalty"]; the rescaled logit is rounded to the
 *      logits' element type (float32; bf16 to nearest even from that float32).
 *      r = 1 or history_len 0: no penalty. history NULL with history_len > 0
      is TSR_EINVAL.
 *  row_params [rows] tsr_params (device memory): each row's own sampling
 *      parameters in place of the call's `params` (which may then be NULL);
 *      a row whose parameters tsr_params would reject gets
 *      TSR_ROW_BADPARAM and token -1 (checked on the device, per row). */
typedef struct {
  const uint32_t* allowed;
  int64_t allowed_stride;
  const int32_t* history;
  int32_t history_len;
  int64_t history_stride;
  double repetition_penalty;
  const tsr_params* row_params;
} tsr_constraints;

/* sample_rows with the per-row inputs of `cons` (nullable) and log p~ of each
 * drawn token (out_logprob, nullable, as in sample_rows_masked). The penalty
 * applies first, then the mask; everything after is sample_rows.
 * sample_rows_masked(..., allowed, allowed_stride, ...) is this call with a
 * constraint holding the mask only. */
int sample_rows_ex(tsr_handle h, const void* logits, int dtype, int rows, int vocab,
                   int64_t row_stride, const tsr_constraints* cons, const tsr_params* params,
                   uint64_t step, int32_t* out_tokens, float* out_logprob,
                   const tsr_diag* diag, void* hip_stream);

/* The speculative verify step [P3 "The Algorithm"; P1, P4 "Speculative
 * decoding"; P2 39.4] for `rows` sequences with K drafted tokens each.
 *  target_logits [rows][K+1][vocab]: the target's logits at the K draft
 *      positions and at the position after them.
 *  draft_logits  [rows][K][vocab]:   the draft's logits (not read when the
 *      temperature is 0).
 *  draft_tokens  [rows][K] int32:    the drafted ids.
 * Both distributions go through the same chain (temperature and filters),
 * p~ and q~. For j = 0..K-1 in order, with (w0, w1) the Philox words of
 * counter (row, j | 1 << 16, step): keep x_j iff w0 * 2^-32 <
 * min(1, p~(x_j) / max(q~(x_j), 1e-300)) (eq. 39.3); at the first rejection
 * emit a draw from max(0, p~ - q~) / Z with w1 (eq. 39.4) and stop; if every
 * draft is kept emit a bonus draw from the target's row K with w0 of
 * position K. Greedy (temperature 0): keep x_j iff it is the target's argmax,
 * emit the argmax at the first mismatch, the bonus is row K's argmax.
 *  out_tokens   [rows][K+1]: emitted ids, -1 after the last one.
 *  out_accepted [rows]:      number of drafts kept (0..K).
 *  out_status   [rows] (nullable): TSR_ROW_*; a bad sequence gets all -1 and 0.
 * 1 <= K <= max_k (set by sampler_init) and K <= 32. vocab <= 155,648 bf16
 * or 77,824 float32 logits (TSR_EUNSUPPORTED beyond). Up to 65,536 bf16 or
 * 32,768 float32 logits each position's two rows are held in one workgroup's
 * registers; wider rows take one workgroup per row, then one per sequence,
 * which re-reads the rejecting position's rows for the residual draw. */
int spec_verify(tsr_handle h, const void* target_logits, const void* draft_logits,
                int dtype, const int32_t* draft_tokens, int rows, int K, int vocab,
                const tsr_params* params, uint64_t step, int32_t* out_tokens,
                int32_t* out_accepted, int32_t* out_status, void* hip_stream);

/* spec_verify for callers that cannot allocate device memory: code under
 * HIP graph capture, tight serving loops, harnesses that forbid hipMalloc.
 * No handle: the Philox key is `seed` (as sampler_init's), and the call runs
 * on `device` (made current for the call, the caller's restored after). The
 * verify workspace is a static device array in the library, 1 MiB, one
 * copy per device, held until the process ends; the call allocates nothing
 * and calls no allocating routine. Limits of that array: rows <= 16384 and
 * rows * (K + 1) <= 65536 (TSR_EINVAL beyond); 1 <= K <= 32; vocab <= 65,536
 * bf16 or 32,768 float32 logits (TSR_EUNSUPPORTED beyond: the array holds no
 * per-row records for spec_verify's wider-row path). Every call on a device shares that device's array: calls that overlap on
 * one device (on different streams, or from several threads) race and give
 * undefined results. Arguments, outputs and results are spec_verify's. */
int spec_verify_noalloc(int device, uint64_t seed, const void* target_logits,
                        const void* draft_logits, int dtype, const int32_t* draft_tokens,
                        int rows, int K, int vocab, const tsr_params* params, uint64_t step,
                        int32_t* out_tokens, int32_t* out_accepted, int32_t* out_status,
                        void* hip_stream);

/* Tree (multi-candidate) verify [P3 "Extensions and Variants": the draft
 * proposes a tree of candidates with several branches and the target
 * verifies every path; P2 39.4 for the rule at one candidate] for `rows`
 * sequences of `nodes` tree nodes each (1 <= nodes <= 32 and <= max_k + 1).
 *  parent [rows][nodes] int32: node 0 is the current context (parent -1);
 *      node n > 0 extends node parent[n] < n (else the sequence gets status 5).
 *  tokens [rows][nodes] int32: the token node n appends (tokens[0] unused).
 *  target_logits, draft_logits [rows][nodes][vocab]: the target's and the
 *      draft's logits for the token after node n's path (the draft's only read
 *      for nodes with children, and not at all at temperature 0).
 * The children of a node (in node order) are its candidates, taken as
 * independent draws from the draft's distribution q~ there. From the root:
 * child c of the current node v is kept iff w0 * 2^-32 < min(1, p_c(x) /
 * q~(x)), p_1 = p~_v and p_{c+1} = max(0, p_c - q~) normalised after each
 * rejection (w0 of the Philox counter (row, v * 32 + c | 2 << 16, step)); a
 * kept child becomes v; when every child of v is rejected, or v has none, one
 * token is drawn from the current p with w1 of (row, v * 32 | 2 << 16, step)
 * and the step ends. Temperature and filters shape p~ and q~ as in
 * spec_verify. Greedy (temperature 0): the first child holding the target's
 * argmax is kept, else the argmax is emitted.
 *  out_tokens [rows][nodes]: the kept children's tokens then the drawn one,
 *      -1 after; out_path [rows][nodes]: the kept nodes, -1 after;
 *  out_accepted [rows]: how many nodes were kept; out_status [rows]
 *      (nullable): TSR_ROW_* (NONFINITE/EMPTY for a bad target row or a bad
 *      draft row of a node with children, BADTOKEN for a token outside
 *      [0, vocab), 5 for a parent that is not an earlier node).
 * vocab limits as spec_verify's (above 65,536 bf16 or 32,768 float32 logits,
 * one workgroup per row, then one per sequence that follows the tree and
 * streams the rows of the nodes where candidates were rejected).
 * Shares the verify workspace: not concurrent with spec_verify on the handle. */
int tree_verify(tsr_handle h, const void* target_logits, const void* draft_logits, int dtype,
                const int32_t* parent, const int32_t* tokens, int rows, int nodes, int vocab,
                const tsr_params* params, uint64_t step, int32_t* out_tokens, int32_t* out_path,
                int32_t* out_accepted, int32_t* out_status, void* hip_stream);

/* One beam-search step [P2 39.1: eq. 39.1, Listing 39.1; P4 "Beam search"]
 * for `groups` independent searches of `beam` beams each (no length penalty
 * or end token, as in the listing).
 *  logits [groups * beam][vocab]: row g * beam + b holds beam b of group g,
 *      row_stride elements apart (vocab beyond 155,648 bf16 or 77,824
 *      float32 logits: TSR_EUNSUPPORTED).
 *  beam_scores [groups * beam] double: each beam's running score s_b, the sum
 *      of its tokens' log-probabilities (eq. 39.1); -inf marks a dead beam.
 * Every candidate (b, i) scores s_b + log softmax(logits_b)_i (temperature
 * 1, the row's own normalisation, so a row without a finite logit adds
 * nothing); the `beam` best of the group's beam * vocab candidates are kept,
 * best first, equal scores in the order (b, then i) ascending.
 *  out_parent [groups * beam] int32: the beam (0..beam-1) each kept candidate
 *      extends; out_token the token; out_score (double) its score. Positions
 *      past the group's finite candidates hold -1, -1, -inf.
 *  out_status [groups] (nullable): TSR_ROW_OK; TSR_ROW_NONFINITE when a NaN or
 *      +inf logit or score is in the group (outputs -1, -1, NaN);
 *      TSR_ROW_EMPTY when no candidate is finite.
 * 1 <= beam <= 16 and groups * beam <= max_rows (TSR_EINVAL otherwise). Uses
 * per-handle workspace: not concurrent with another beam_step on the handle. */
int beam_step(tsr_handle h, const void* logits, int dtype, int groups, int beam, int vocab,
              int64_t row_stride, const double* beam_scores, int32_t* out_parent,
              int32_t* out_token, double* out_score, int32_t* out_status, void* hip_stream);

/* 8-bit codes of float rows, one scale per row: the form int8_logits takes
 * its operands in (hidden states per token, a weight per output channel)
 * [P1 "int8 weights": per-row absmax].
 *  x [rows][width] float32 or bfloat16 (dtype), row_stride elements apart.
 *  out_scale [rows] float32: s = max |x| of the row times 1/127, in float32.
 *  out_codes [rows][width] int8, codes_stride bytes apart: x / s rounded to
 *      the nearest whole number, ties to even, decided on the exact quotient,
 *      and held to [-127, 127].
 * A row of zeros gets scale 0 and codes 0. A row that holds NaN or an
 * infinity gets scale NaN and codes 0, so its logits are NaN and the sampler
 * reports it as TSR_ROW_NONFINITE. Bytes of out_codes between width and
 * codes_stride are left as they are.
 * rows is not bound by the handle's max_rows (a weight has vocab rows); rows <
 * 2^24 and width <= 2^30 (TSR_EUNSUPPORTED beyond). Uses no workspace. */
int quantize_rows(tsr_handle h, const void* x, int dtype, int rows, int width, int64_t row_stride,
                  int8_t* out_codes, int64_t codes_stride, float* out_scale, void* hip_stream);

/* An output projection held in 8 bits (device memory, the caller's).
 *  weight [vocab][width] int8, weight_stride bytes apart (any alignment).
 *  scale [vocab] float32: the value of one step of each channel's codes.
 *  bias [vocab] float32, or NULL. */
typedef struct {
  const int8_t* weight;
  int64_t weight_stride;
  const float* scale;
  const float* bias;
  int32_t vocab;
  int32_t width;
} tsr_head;

/* Logits of `rows` hidden states against an 8-bit output projection:
 *   out[r][n] = (sum_k codes[r][k] * weight[n][k]) * code_scale[r] * scale[n]
 *               + bias[n].
 * The sum is exact, in 32-bit integers; it is then scaled in float32 (the sum
 * rounded, times code_scale, times scale and plus bias in one fma) and
 * rounded once more where the logits are bfloat16. A NaN scale makes its row's
 * (or channel's) logits NaN.
 *  codes [rows][width] int8, codes_stride bytes apart (any alignment).
 *  out_logits [rows][vocab] of type dtype, out_stride elements apart; what
 *      lies between vocab and out_stride is left as it is.
 * width <= 131071 (the sum fits 32 bits), vocab <= 2^29 and both operands'
 * strides < 2^22 (TSR_EUNSUPPORTED beyond; the stride of a single row is not
 * used). Rows that start at 4-byte words are read fastest, those at multiples
 * of 128 bytes most of all; other rows are read in whole 4-byte words, so up to
 * three bytes on either side of a row, in words that also hold bytes of it.
 * Uses no workspace. */
int int8_logits(tsr_handle h, const int8_t* codes, int64_t codes_stride, const float* code_scale,
                int rows, const tsr_head* head, void* out_logits, int dtype, int64_t out_stride,
                void* hip_stream);

/* From hidden states to tokens: quantize_rows, int8_logits and sample_rows
 * enqueued one after the other.
 *  hidden [rows][head->width] of type hidden_dtype, hidden_stride elements
 *      apart.
 *  codes [rows][width] (codes_stride bytes apart), code_scale [rows] and logits
 *      [rows][vocab] (of type dtype) are workspace of the caller's and hold the
 *      codes, the scales and the logits afterwards.
 * params, step, out_tokens and diag are sample_rows'; so are the limits on
 * vocab. */
int sample_hidden(tsr_handle h, const void* hidden, int hidden_dtype, int rows,
                  int64_t hidden_stride, const tsr_head* head, int8_t* codes,
                  int64_t codes_stride, float* code_scale, void* logits, int dtype,
                  const tsr_params* params, uint64_t step, int32_t* out_tokens,
                  const tsr_diag* diag, void* hip_stream);

/* The verify step from probabilities and the caller's random numbers
 * [P2 39.4, Listing 39.4; P3 "The Algorithm", "Batching Speculation"], for
 * `rows` sequences with up to K drafted tokens each.
 *  target_probs: p, K + 1 rows of `vocab` per sequence (float32 or bfloat16,
 *      dtype): position j of sequence b starts at b * target_seq_stride +
 *      j * target_row_stride elements.
 *  draft_probs: q, K rows per sequence, laid out by its own strides; NULL:
 *      each draft token was proposed with certainty (q is 1 at the token).
 *  draft_tokens [rows][K]; draft_lens [rows] (nullable: K each): how many of
 *      them sequence b has, 0..K. Positions past that many drafts are not
 *      read (the rows of p: past draft_lens[b]).
 *  accept_u [rows][K], draw_u [rows] float32, each in [0, 1).
 * For j = 0, 1, ...: draft x_j is kept iff accept_u[b][j] < min(1, p(x_j) /
 * q(x_j)) (eq. 39.3; with q = 0, iff p > 0). At the first refusal the step
 * ends with a draw from max(0, p - q) (eq. 39.4), or from p where that is
 * zero everywhere; with every draft kept it ends with a draw from the row of
 * p after them. The draw is the first id, in ascending order, whose running
 * total of the weights exceeds draw_u[b] times their sum (the last id with a
 * weight where rounding leaves none): the weights need not sum to 1. Tests,
 * weights and sums are formed in 64 bits.
 *  out_tokens   [rows][K+1]: the kept drafts, the drawn id, then -1.
 *  out_accepted [rows]: number of drafts kept.
 *  out_status   [rows] (nullable): TSR_ROW_OK; else the tokens are all -1 and
 *      the count is 0. The first that holds of: TSR_ROW_BADPARAM (draft_lens
 *      outside 0..K), TSR_ROW_BADTOKEN (one of the sequence's draft tokens
 *      outside [0, vocab)), TSR_ROW_NONFINITE (a probability of a tested
 *      draft is negative, infinite or NaN), TSR_ROW_BADPARAM (accept_u of a
 *      tested draft, or draw_u, outside [0, 1)), TSR_ROW_NONFINITE (such a
 *      value in the rows drawn from), TSR_ROW_EMPTY (they are all zero).
 *      Rows and positions that the step does not come to are not checked.
 * 1 <= K <= max_k and K <= 32; vocab <= 2^30 and rows < 2^22
 * (TSR_EUNSUPPORTED beyond). Strides are not negative; rows may overlap or
 * repeat (stride 0). Up to 512 sequences of many ids are summed by several
 * workgroups each, through per-handle workspace of its own: not concurrent
 * with another verify_probs on the handle (verify_probs_ex may be). */
int verify_probs(tsr_handle h, const void* target_probs, int64_t target_seq_stride,
                 int64_t target_row_stride, const void* draft_probs, int64_t draft_seq_stride,
                 int64_t draft_row_stride, int dtype, const int32_t* draft_tokens,
                 const int32_t* draft_lens, const float* accept_u, const float* draw_u, int rows,
                 int K, int vocab, int32_t* out_tokens, int32_t* out_accepted,
                 int32_t* out_status, void* hip_stream);

/* verify_probs with the caller's workspace in place of the handle's: calls with
 * workspaces of their own may run at the same time on one handle (graphs that
 * were captured with them as well).
 *  workspace: device memory, 16-byte aligned, workspace_bytes long; at least
 *      verify_probs_workspace's bytes (TSR_EINVAL otherwise). Its contents do
 *      not matter before the call or after it. NULL: the handle's. */
int verify_probs_ex(tsr_handle h, const void* target_probs, int64_t target_seq_stride,
                    int64_t target_row_stride, const void* draft_probs, int64_t draft_seq_stride,
                    int64_t draft_row_stride, int dtype, const int32_t* draft_tokens,
                    const int32_t* draft_lens, const float* accept_u, const float* draw_u, int rows,
                    int K, int vocab, int32_t* out_tokens, int32_t* out_accepted,
                    int32_t* out_status, void* workspace, int64_t workspace_bytes,
                    void* hip_stream);

/* Bytes of workspace that verify_probs_ex takes for these sizes (under 2^23); 0
 * where it takes none: one workgroup sums a sequence, or there is nothing to do. */
int verify_probs_workspace(int dtype, int rows, int vocab);

/* 8-bit codes of rows that are first added to a residual and normed by their root
 * mean square: quantize_rows for the hidden states that a model's last block
 * leaves, before int8_logits.
 *   h = x + residual, rounded once to their type (h = x without a residual)
 *   n_i = h_i weight_i / sqrt(mean(h^2) + eps)
 *  x, residual [rows][width] of type dtype, x_stride and residual_stride
 *      elements apart; residual NULL: none.
 *  weight [width] of type weight_dtype; NULL: ones. For a weight that is held
 *      less one, add the one when it is loaded.
 *  out_residual [rows][width] of type dtype, out_residual_stride elements apart:
 *      h. NULL: not kept; it has to be NULL without a residual. It may be x or
 *      residual itself, with the same stride.
 *  out_scale [rows] float32: s = max |n| of the row / 127.
 *  out_codes [rows][width] int8, codes_stride bytes apart: n / s = 127 h_i w_i /
 *      max |h w|, rounded to the nearest whole number, ties to even, decided on
 *      that exact quotient.
 * A row whose h w is zero everywhere gets scale 0 and codes 0. A row in which h or
 * h w holds NaN or an infinity (h rounded to its type, h w in 64 bits) gets scale
 * NaN and codes 0, as in quantize_rows. eps is finite and >= 0. Bytes between
 * the rows are left as they are. Outputs that overlap inputs or each other in any
 * other way are TSR_EINVAL (rows of the same stride may lie between each other's).
 * rows is not bound by the handle's max_rows; rows < 2^24, width <= 2^30 and
 * strides < 2^36 (TSR_EUNSUPPORTED beyond). Uses no workspace. */
int norm_quantize_rows(tsr_handle h, const void* x, int64_t x_stride, const void* residual,
                       int64_t residual_stride, int dtype, const void* weight, int weight_dtype,
                       double eps, int rows, int width, void* out_residual,
                       int64_t out_residual_stride, int8_t* out_codes, int64_t codes_stride,
                       float* out_scale, void* hip_stream);

/* Outputs of token_logprobs (device memory); NULL: not wanted.
 *  logprob [rows][n_tokens] float32: log p of each given token.
 *  entropy [rows] float32: -sum_j p_j log p_j.
 *  top_ids, top_logprob [rows][top_k]: the top_k ids of the largest logits, largest
 *      first, equal ones by the lower id, and their log p. Positions past the
 *      row's finite logits hold -1 and -inf.
 *  norm [rows][2] float32: the largest logit M and Z = sum_j exp((z_j - M) / T):
 *      what token_logprobs_grad takes; M / T + log Z is the log of the sum of all
 *      exp(z_j / T).
 *  status [rows]: TSR_ROW_NONFINITE (a NaN or +inf logit) or TSR_ROW_EMPTY (every
 *      logit is -inf), with NaN in the row's outputs and -1 in its ids; else
 *      TSR_ROW_BADTOKEN (a token that is neither -1 nor in [0, vocab): NaN for it
 *      alone); else TSR_ROW_OK. */
typedef struct {
  float* logprob;
  float* entropy;
  int32_t* top_ids;
  float* top_logprob;
  float* norm;
  int32_t* status;
} tsr_logprobs;

/* Log probabilities of given tokens under p = softmax(logits / temperature), with
 * the entropy and the likeliest alternatives: scores of prompts, drafts and choices,
 * and a teacher's top tokens for distill_topk.
 *  logits [rows][vocab] of type dtype, row_stride elements apart. Logits of -inf
 *      (tokens that are not allowed) have p = 0 and log p = -inf.
 *  temperature: 1e-30 .. 1e30.
 *  tokens [rows][n_tokens] int32 (NULL with n_tokens 0); -1 is padding, as the
 *      verify steps leave behind the last token: its log p is 0.
 *  workspace: 16-byte aligned device memory of at least token_logprobs_workspace
 *      bytes, the call's own until it is done (NULL where that is 0). Its
 *      contents do not matter before the call or after it.
 * Neither outputs nor the workspace lie over inputs or each other (TSR_EINVAL).
 * rows and vocab are not bound by the handle's. n_tokens <= 1024, top_k <= 64,
 * rows < 2^22, vocab <= 2^30, row_stride < 2^36 (TSR_EUNSUPPORTED beyond). */
int token_logprobs(tsr_handle h, const void* logits, int dtype, int rows, int vocab,
                   int64_t row_stride, double temperature, const int32_t* tokens, int n_tokens,
                   int top_k, const tsr_logprobs* out, void* workspace, int64_t workspace_bytes,
                   void* hip_stream);

/* Bytes of workspace that token_logprobs takes for these sizes; 0: none (or sizes
 * that it does not take). */
int token_logprobs_workspace(int dtype, int rows, int vocab, int top_k);

/* The gradient of token_logprobs' log p and entropy by the logits:
 *   out[r][j] = (sum_i g[r][i] [tokens[r][i] = j]
 *                - p_j (sum_i g[r][i] + ge[r] (log p_j + H[r]))) / temperature
 * with g = grad_logprob, ge = grad_entropy and H = entropy.
 *  logits, temperature, tokens: as given to token_logprobs; norm and entropy [rows]:
 *      as it left them. Tokens of -1 and their g do not count; one that is neither
 *      -1 nor in [0, vocab) makes its row NaN, as norm does in the rows that
 *      token_logprobs marked NONFINITE or EMPTY.
 *  grad_logprob [rows][n_tokens] (NULL with n_tokens 0); grad_entropy [rows], or
 *      NULL: no gradient comes back to the entropy (entropy may then be NULL).
 *  out_grad [rows][vocab] of type dtype, grad_stride elements apart, none of it in
 *      an input's memory (TSR_EINVAL). What lies between vocab and grad_stride is
 *      left as it is. Each element is rounded once.
 * A row to which only zeros come back gets zeros, and its logits are not looked at.
 * Where a row's gradients over the temperature pass float32's range, its elements are
 * not finite, those of weight 0 among them.
 * Limits as token_logprobs'. Uses no workspace. */
int token_logprobs_grad(tsr_handle h, const void* logits, int dtype, int rows, int vocab,
                        int64_t row_stride, double temperature, const int32_t* tokens,
                        int n_tokens, const float* norm, const float* grad_logprob,
                        const float* entropy, const float* grad_entropy, void* out_grad,
                        int64_t grad_stride, void* hip_stream);

/* Distillation of a draft model from a teacher's top tokens, loss and gradient: per
 * row the divergence of p = softmax(logits / temperature) from the teacher's q, which
 * is given by k entries.
 *  ids, teacher_logprob [rows][k]: token ids and the teacher's log probabilities at the
 *      same temperature, as token_logprobs' top_ids and top_logprob. An id of -1 is no
 *      entry, a log probability of -inf one with q = 0. An id that comes twice
 *      counts with both its q.
 *  tail 0: q is the entries' exp over their sum (any constant may be added to a row's
 *      values): L = sum_i q_i (log q_i - log p_i).
 *  tail 1: q_i = exp(teacher_logprob), and what they leave of 1 (0 where that is at
 *      most 2^-20, the rounding of the log probabilities) is the teacher's mass q_r of all
 *      ids that are no entry: L = sum_i q_i (log q_i - log p_i) + q_r (log q_r -
 *      log p_r), with p_r the sum of p over those ids.
 *  row_weight [rows] float32 (NULL: 1 each), for instance 1 / rows and 0 for
 *      padding: out_loss = row_weight * L, and rows of weight 0 get loss and gradient 0,
 *      their logits and entries not looked at.
 *  out_loss [rows] float32. +inf where p is 0 at an entry whose q is not.
 *  out_grad [rows][vocab] of type dtype, grad_stride elements apart: the gradient of the
 *      sum of out_loss by the logits, (row_weight / temperature) times Q p_j - q_j at
 *      entries and p_j (Q - q_r / p_r) elsewhere, Q = sum q + q_r; each rounded once.
 *      NULL: the loss alone. For a loss over temperatures the usual factor temperature^2
 *      goes into row_weight. row_weight / temperature within float32's range.
 *  out_status [rows] (nullable): TSR_ROW_OK, else loss and gradient are NaN: the first
 *      that holds of TSR_ROW_BADTOKEN (an id neither -1 nor in [0, vocab)),
 *      TSR_ROW_NONFINITE (a NaN or +inf log probability), TSR_ROW_EMPTY (no entry with
 *      q > 0), TSR_ROW_NONFINITE, TSR_ROW_EMPTY (the logits, as in token_logprobs).
 *  workspace: as token_logprobs', of distill_topk_workspace bytes.
 * Neither outputs nor the workspace lie over inputs or each other (TSR_EINVAL).
 * 1 <= k; k <= 64 and the limits of token_logprobs (TSR_EUNSUPPORTED beyond). */
int distill_topk(tsr_handle h, const void* logits, int dtype, int rows, int vocab,
                 int64_t row_stride, double temperature, const int32_t* ids,
                 const float* teacher_logprob, int k, int tail, const float* row_weight,
                 float* out_loss, void* out_grad, int64_t grad_stride, int32_t* out_status,
                 void* workspace, int64_t workspace_bytes, void* hip_stream);

/* Bytes of workspace that distill_topk takes for these sizes, with a gradient
 * (want_grad 1) or without one; 0: none. */
int distill_topk_workspace(int dtype, int rows, int vocab, int want_grad);

/* Test hook: out_words[i][0..3] = Philox4x32-10(counters[i][0..3], key = the
 * handle's seed) for i < n, computed on the device by the same function the
 * sampler uses. counters and out_words are device memory. */
int sampler_philox(tsr_handle h, const uint32_t* counters, int n, uint32_t* out_words,
                   void* hip_stream);

/* Static description of a return code. */
const char* sampler_strerror(int code);

#ifdef __cplusplus
}
#endif

#endif /* TSR_H_ */

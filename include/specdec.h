/*
 * specdec.h -- C ABI of libspecdec.so: batched speculative-decoding verification on
 * one GB300 (sm_103a).
 *
 * One call verifies a ragged batch of draft tokens against the target model's logits:
 * it applies each position's packed grammar bitmask, takes the temperature softmax,
 * accepts each draft with probability min(1, p/q) (or by argmax equality for greedy
 * requests), stops at the first rejection, draws the recovered token there from the
 * residual distribution, emits a bonus token when every draft is accepted, and
 * accumulates the raw / grammar-invalidated / eligible / accepted counters.
 *
 * Sources for the operation:
 *   - "vLLM tour part 2" (pyshine.com/vllm-2), section "Verification: rejection sampling
 *     on the GPU": target logits for every draft position plus one bonus position, cast
 *     to float32, temperature applied; acceptance where the target probability of the
 *     draft token beats a uniform draw; recovered token from the target probabilities
 *     minus the draft probabilities clamped at zero; greedy variant for temperature 0.
 *   - same page, section "Grammar gates: structured output": one bitmask row per request
 *     and per speculative position; masked tokens cannot be produced.
 *   - "5.2 Draft models and model-free methods" (infra-guide), section 4.3: a draft with
 *     no probabilities is a one-hot q -- accept with probability p(x), residual = p with x
 *     removed, renormalised.
 *   - "Structured output speculative decoding acceptance" (fanout.sh), section "Name the
 *     three counters": R raw drafts, I grammar-invalidated, D = R - I eligible, A accepted.
 *
 * Layout conventions (all calls):
 *   B requests; cu_num_draft[B+1] is an exclusive prefix sum, cu[0] = 0, non-decreasing;
 *   request b has k_b = cu[b+1] - cu[b] drafts; N = cu[B].
 *   Draft slot d(b,j) = cu[b] + j, j in [0, k_b).
 *   Logit row t(b,j) = cu[b] + b + j, j in [0, k_b]; row j = k_b is the bonus row;
 *   T = N + B rows.  W = ceil(V / 32) mask words per row.
 *   A request is greedy iff temperature[b] == 0. It is a draft-model request iff
 *   draft_probs != NULL and (has_q == NULL or has_q[b] != 0); otherwise model-free.
 */
#ifndef SPECDEC_H
#define SPECDEC_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define SPECDEC_KMAX 32           /* largest supported max_k (drafts per request) */
#define SPECDEC_TELEMETRY_ROW (SPECDEC_KMAX + 1)   /* entries per telemetry row */

typedef enum {
    SPECDEC_OK = 0,
    SPECDEC_ERR_INVALID_ARG = 1,   /* a NULL required pointer, a bad size or a misaligned pointer */
    SPECDEC_ERR_UNSUPPORTED = 2,   /* dtype unknown, or a row too wide for on-chip staging */
    SPECDEC_ERR_CUDA = 3,          /* a CUDA runtime error at launch (or from specdec_wait) */
    SPECDEC_ERR_TIMEOUT = 4        /* specdec_wait gave up */
} specdec_status_t;

/* The verify takes F32 and BF16 logits; the cache operators below also take F16, and E4M3 (8-bit
 * floating point, 4 exponent and 3 mantissa bits, no infinity) as a cache's type. */
typedef enum { SPECDEC_F32 = 0, SPECDEC_BF16 = 1, SPECDEC_F16 = 2, SPECDEC_E4M3 = 3 } specdec_dtype_t;

/* Per-request status bits written to status[b] (0 = clean). The kernel never traps. */
#define SPECDEC_ST_BAD_DRAFT_ID    1u   /* a draft id outside [0, V): counted invalid, never accepted */
#define SPECDEC_ST_EMPTY_MASK_ROW  2u   /* a row read allows no finite logit: -1 emitted there, request stops */
#define SPECDEC_ST_BAD_TEMPERATURE 4u   /* not 0 and not a positive normal finite float: verified greedily */
#define SPECDEC_ST_K_TOO_LARGE     8u   /* k_b > max_k: skipped, -1 in its rows, no counters */
#define SPECDEC_ST_BAD_OFFSETS    16u   /* cu[0] != 0 or cu[b] > cu[b+1] or cu[b+1] > cu[B]: skipped */
#define SPECDEC_ST_DEVICE_TIMEOUT 32u   /* an on-chip copy did not land within its time limit */
#define SPECDEC_ST_BAD_TOP_P      64u   /* top_p not a number in (0, 1]: no top-p filter */
/* Set by the cache operators (with K_TOO_LARGE, BAD_OFFSETS and DEVICE_TIMEOUT above). */
#define SPECDEC_ST_BAD_LENGTH    128u   /* a negative length, or one past the request's row of block_table: skipped */
#define SPECDEC_ST_BAD_PAGE      256u   /* a page id outside [0, num_pages): nothing written there, zeros read */
/* Set by the operators on rows of logits beside the verify (with EMPTY_MASK_ROW above, here also a row without
 * any logit above -infinity). */
#define SPECDEC_ST_BAD_SCORE     512u   /* a beam's score, or a logit of its row, is NaN or +infinity: no candidates */
#define SPECDEC_ST_BAD_TARGET   1024u   /* a listed id outside [-1, V) or listed before, or no log-probability: not counted */

/*
 * specdec_verify -- verify one batch (stream-ordered, asynchronous).
 *
 * Pointers are device pointers to caller-owned memory on the current device; the
 * library allocates nothing and keeps no state between calls.
 *
 *   target_logits  [T, V] row-major, fp32 or bf16 (logits_dtype); 4- resp. 2-byte aligned.
 *   draft_ids      [N] int32; may be NULL when N = 0 (a request that does have drafts then
 *                  gets SPECDEC_ST_BAD_DRAFT_ID and all its drafts count as invalid).
 *   draft_probs    [N, V] fp32 draft distributions q, or NULL (every request model-free).
 *                  Only q(x) of each tested draft and the q row of a rejected position are read.
 *   has_q          [B] uint8 or NULL (NULL: every request is a draft-model request iff
 *                  draft_probs != NULL).
 *   cu_num_draft   [B+1] int32 exclusive prefix of draft counts.
 *   B, V, max_k    B >= 0, V >= 1, 0 <= max_k <= SPECDEC_KMAX (every k_b must be <= max_k).
 *   bitmask        [T, W] int32 or NULL (unconstrained). Bit (i & 31) of word i >> 5 is 1
 *                  when token i is allowed; bits at or above V are ignored.
 *   temperature    [B] fp32; 0 means greedy.
 *   top_k          [B] int32 or NULL: top-k per request (<= 0: off). The target distribution of a
 *                  sampled request keeps every allowed id whose logit is at least the k-th largest
 *                  allowed logit (ties at the boundary kept) before acceptance, residual and bonus
 *                  ("vLLM tour part 2", section "Verification: rejection sampling on the GPU":
 *                  temperature and top-k/top-p are applied to the target tensor). Greedy requests
 *                  ignore it (the argmax is always kept).
 *   top_p          [B] fp32 or NULL: top-p per request (>= 1: off), applied after top-k: the kept
 *                  ids are those whose (top-k renormalised) mass of strictly larger logits is
 *                  below top_p (ties kept); p is renormalised over the kept ids. A value that is
 *                  not a number in (0, 1] sets SPECDEC_ST_BAD_TOP_P and is ignored. With top_k or
 *                  top_p given, the streaming kernel runs one CTA per request. A draft that is
 *                  surely kept and whose uniform lies below e_x / (S q(x)) (S the row's whole
 *                  softmax sum, a lower bound of the filtered ratio) is accepted without a
 *                  threshold search, unless diag_accept_prob is given (every filtered row then
 *                  searches, so that the exact filtered alpha can be reported). A top-k search
 *                  (k <= 1927) first streams a filtered row once more to take its top slice of
 *                  logits (the elements carrying at least 1.0625 S / 2048 of the mass, or 16x less
 *                  on a retry); when that holds k elements the top-k search, and a top-p search
 *                  after it, run on chip. Otherwise a search streams the row to bin its logits by
 *                  mass (an accepted top-p row may be settled there) and once more to collect the
 *                  chosen bin (on chip when it holds at most 2048 elements, else one more pass per
 *                  8-bit digit of its keys: at most 2 for bf16 logits, 4 for fp32). A stop row
 *                  with few kept ids draws from those ids only. The outputs do not depend on the
 *                  route. V > 2^20, or the slice-resident cluster kernel
 *                  (specdec_set_launch_options), with either of them: SPECDEC_ERR_UNSUPPORTED.
 *   uniforms       [T] fp32 in [0, 1); draft j of request b is accepted iff
 *                  uniforms[t(b,j)] < alpha (strict). Entries at bonus rows are unused.
 *   exp_noise      [T, V] fp32 Exp(1) samples > 0; the token drawn from weights w at row t
 *                  is argmax_i w_i / exp_noise[t, i] (lowest index on ties). Read only at
 *                  the one row per random request that draws a token.
 *   out_tokens     [T] int32: the accepted drafts, then the recovered or bonus token,
 *                  then -1 for every later position of the request.
 *   out_num_accepted [B] int32: accepted drafts a_b per request.
 *   counters       [4] uint64 (R, I, D, A), ADDED to (never cleared by the library).
 *   status         [B] uint32 per-request status bits (written, not accumulated), or NULL.
 *   diag_accept_prob [N] fp32 or NULL: alpha of every draft that was tested, NaN otherwise.
 *   diag_row_stats [T, 2] fp32 or NULL: for every row read, (m, S) with m = max_i z_i / T
 *                  and S = sum_i exp(z_i / T - m) on random requests, (max_i z_i, NaN) on
 *                  greedy ones; (NaN, NaN) for rows not read. Entries of a request skipped
 *                  for SPECDEC_ST_BAD_OFFSETS are left untouched (its rows are unknown).
 *   telemetry      [4 * SPECDEC_TELEMETRY_ROW] uint64 or NULL, ADDED to (never cleared), 8-byte
 *                  aligned: per position j, row 0 counts drafts (k_b > j), row 1 grammar-eligible
 *                  drafts (g_b > j, g_b the grammar-valid prefix behind I and D), row 2 drafts
 *                  accepted all the way through position j (a_b > j); row 3 [a] counts requests
 *                  that accepted exactly a drafts. Requests skipped for K_TOO_LARGE or BAD_OFFSETS
 *                  are not counted. Rows 0..2 sum to R, D and A. ("vLLM tour part 2", section
 *                  "Telemetry and tuning": per-position draft / accepted counts and the histogram
 *                  of accepted lengths; "5.2 Draft models and model-free methods", section 7.2:
 *                  a position counts drafts accepted through it.)
 *   workspace      device scratch of at least specdec_workspace_size(B, V) bytes, 16-byte
 *                  aligned, caller-owned, or NULL. With a workspace a one-CTA kernel first orders
 *                  the requests by an estimate of their work, heaviest first, and the verify
 *                  kernel takes them in that order (list scheduling by the longest-processing-
 *                  time rule: a long request that sits late in the batch no longer runs on alone
 *                  after the rest have finished). The schedule runs only when the batch needs more
 *                  than one wave of resident CTAs (two per SM); the verify kernel then starts as a
 *                  programmatic dependent of it. A batch that exceeds that wave additionally splits
 *                  its heaviest requests (a sixth of a wave) over clusters of 2 CTAs (their chains
 *                  of row passes are what set the launch's length) and runs the others two per
 *                  cluster, one per CTA. Without a workspace, requests start in index order, one
 *                  CTA each.
 *                  Results are identical either way; only the timing differs. The workspace
 *                  needs no initialisation and holds nothing between calls; calls that share one
 *                  workspace must not overlap in time (use one per stream).
 *   workspace_bytes its size in bytes.
 *   stream         a cudaStream_t (NULL = legacy default stream).
 *
 * Rows after a request's stop row a_b (its first rejection, or the bonus row) are never used: no
 * output depends on them. At the byte level, a request whose bitmask is absent or dense may read
 * the first two ring chunks (at most 2 x 32 KB) of row a_b + 1, queued before the decision on
 * row a_b and discarded unused; a request with a sparse bitmask prefetches the mask words of all
 * its rows into L2 when it starts. Nothing else of a later row is read.
 * Returns SPECDEC_OK once the kernel is queued; data errors land in status[].
 * Errors: SPECDEC_ERR_INVALID_ARG (nothing launched, nothing written) for a NULL required
 * pointer (draft_ids may be NULL), B < 0, V < 1, max_k outside [0, SPECDEC_KMAX], or a pointer not aligned to its
 * element (telemetry: 8 bytes); SPECDEC_ERR_UNSUPPORTED for an unknown dtype, for top_k or top_p with V > 2^20
 * (or with the cluster kernel), or, with the cluster kernel that keeps each row slice on chip, a row wider than
 * 3 MiB; SPECDEC_ERR_CUDA if the launch fails.
 *
 * Kernels: by default each request is verified by a cluster of G CTAs (G = 1 for large
 * batches, up to 4 for small ones), each streaming its slice of every row through a ring of
 * 32 KB shared-memory stages filled by bulk async copies; requests whose bitmask allows few ids
 * gather only the allowed 16-byte groups instead. specdec_set_launch_options (below) selects the
 * alternative kernel that keeps a slice of every row resident in shared memory, forces G, or
 * forces the request schedule on or off. All shapes compute identical results.
 */
specdec_status_t specdec_verify(
    const void* target_logits, specdec_dtype_t logits_dtype,
    const int32_t* draft_ids,
    const float* draft_probs,
    const uint8_t* has_q,
    const int32_t* cu_num_draft,
    int32_t B, int32_t V, int32_t max_k,
    const int32_t* bitmask,
    const float* temperature,
    const int32_t* top_k,
    const float* top_p,
    const float* uniforms,
    const float* exp_noise,
    int32_t* out_tokens,
    int32_t* out_num_accepted,
    unsigned long long* counters,
    uint32_t* status,
    float* diag_accept_prob,
    float* diag_row_stats,
    unsigned long long* telemetry,
    void* workspace,
    size_t workspace_bytes,
    void* stream);

/*
 * specdec_verify_noalloc -- specdec_verify for callers that cannot hand the library scratch
 * memory. The pages have no counterpart to this: it is a calling convention of this library,
 * not a step of the method.
 *
 * Same arguments, semantics and results as specdec_verify, without workspace / workspace_bytes:
 * the request schedule's scratch (an int32 order and a cost byte per request) is a fixed array
 * inside the library, file-scope device memory of 80 KiB per device holding up to
 * SPECDEC_NOALLOC_MAX_REQUESTS requests. The call allocates nothing (no cudaMalloc, no
 * allocating library routine) and needs no memory from the caller beyond the batch itself.
 * It serves callers that have no device allocator of their own (a plain C or C++ host program
 * that links this library directly) and serving loops that must not allocate inside a decode
 * step (cudaMalloc synchronises the device; a caching allocator may have to grow its pool).
 *
 *   B > SPECDEC_NOALLOC_MAX_REQUESTS: SPECDEC_ERR_UNSUPPORTED, checked before any CUDA call;
 *   nothing is launched or written. Every other error is specdec_verify's.
 *   Zeroing: nothing in the scratch has to start at zero; each call writes every entry it reads.
 *   Set-up: the first call with B > 0 on a device looks the array's address up with
 *   cudaGetSymbolAddress (once per device, then cached; SPECDEC_ERR_CUDA if that fails). Make
 *   that first call on each device before any stream capture begins on it. The cache is keyed
 *   on the current context's unique id as well: after cudaDeviceReset, or in a context the
 *   caller created with the driver API, the next call looks the address up again (so make that
 *   call outside stream capture too).
 *   Concurrency: all calls on a device share the one array. Two calls that overlap in time (on
 *   different streams, or from host threads whose calls are not stream-ordered) race on it, and
 *   the outputs and counters of both are then undefined. Queue such calls on one stream, or use
 *   specdec_verify with one workspace per stream.
 */
#define SPECDEC_NOALLOC_MAX_REQUESTS 16384
specdec_status_t specdec_verify_noalloc(
    const void* target_logits, specdec_dtype_t logits_dtype,
    const int32_t* draft_ids,
    const float* draft_probs,
    const uint8_t* has_q,
    const int32_t* cu_num_draft,
    int32_t B, int32_t V, int32_t max_k,
    const int32_t* bitmask,
    const float* temperature,
    const int32_t* top_k,
    const float* top_p,
    const float* uniforms,
    const float* exp_noise,
    int32_t* out_tokens,
    int32_t* out_num_accepted,
    unsigned long long* counters,
    uint32_t* status,
    float* diag_accept_prob,
    float* diag_row_stats,
    unsigned long long* telemetry,
    void* stream);

/*
 * specdec_ngram_propose -- model-free drafts for a batch: the n-gram proposer of "5.2 Draft
 * models and model-free methods" (infra-guide), sections 4.1 and 6 (stream-ordered,
 * asynchronous). For request b with history h = tokens[cu_hist[b] .. cu_hist[b+1]) of length L,
 * the window length is the longest n in [min_n, min(max_n, L - 1)] such that the last n tokens of
 * h also occur earlier in h (the tail itself excluded), taking the earliest such occurrence; the
 * proposal is the (up to) k tokens that follow it, cut at the end of h. The drafts go to the
 * verify as model-free drafts (no q): accepted with probability p(x).
 *
 *   tokens         [cu_hist[B]] int32 token ids, the histories back to back (device).
 *   cu_hist        [B+1] int64 offsets; a request with cu_hist[b+1] < cu_hist[b] or a negative
 *                  offset counts as an empty history (a miss).
 *   B              requests (>= 0).
 *   min_n, max_n   window lengths tried, 1 <= min_n; max_n <= SPECDEC_NGRAM_MAX_N (64);
 *                  max_n < min_n means no window is tried.
 *   k              proposal length, 0 <= k <= SPECDEC_KMAX.
 *   out_drafts     [B, k] int32: the proposal, then -1.
 *   out_num        [B] int32 proposal lengths (0 on a miss).
 *   out_match      [B] int32 window length of the match (0 on a miss).
 * Returns SPECDEC_OK once queued; SPECDEC_ERR_INVALID_ARG for a bad size, a NULL required pointer
 * or a misaligned one (nothing launched); SPECDEC_ERR_UNSUPPORTED for max_n > 64;
 * SPECDEC_ERR_CUDA if the launch fails.
 */
#define SPECDEC_NGRAM_MAX_N 64
specdec_status_t specdec_ngram_propose(const int32_t* tokens, const int64_t* cu_hist, int32_t B,
                                       int32_t min_n, int32_t max_n, int32_t k, int32_t* out_drafts,
                                       int32_t* out_num, int32_t* out_match, void* stream);

/*
 * specdec_bitmask_scatter -- the grammar bitmask of one verify step in batch order, from the
 * compacted masks in scheduler order ("vLLM tour part 2", section "Grammar gates: structured
 * output": masks arrive compacted to the constrained requests in scheduler order, while the batch
 * has its own order and per-request speculative offsets). Stream-ordered, asynchronous.
 *
 *   compact        [compact_rows, W] int32, W = ceil(V / 32): for each constrained request in
 *                  scheduler order, its k_b + 1 rows (draft positions, then the bonus position).
 *   constrained    [n] int32: the batch index b of each constrained request, scheduler order.
 *   cu_num_draft   [B+1] int32 batch-order draft offsets (the verify's layout: row t(b, j) =
 *                  cu[b] + b + j, j in [0, k_b]).
 *   bitmask        [T, W] int32 output, T = cu[B] + B: the rows of each constrained request take
 *                  its compact rows; rows of every other request are all ones (-1: all allowed).
 * Readings for malformed input: an id outside [0, B) owns no compact rows; a request listed twice
 * takes the rows of its first listing (the second listing's rows are skipped over); a row past the
 * end of `compact` gets zeros (nothing allowed; the verify then reports an empty mask row); a
 * request with malformed offsets (as SPECDEC_ST_BAD_OFFSETS) owns no rows and its rows are not
 * written. Returns SPECDEC_OK once queued; SPECDEC_ERR_INVALID_ARG for a bad size, a NULL
 * required pointer or a misaligned one; SPECDEC_ERR_UNSUPPORTED for V > 2^26; SPECDEC_ERR_CUDA if
 * the launch fails.
 */
specdec_status_t specdec_bitmask_scatter(const int32_t* compact, int64_t compact_rows,
                                         const int32_t* constrained, int32_t n,
                                         const int32_t* cu_num_draft, int32_t B, int32_t V,
                                         int32_t* bitmask, void* stream);

/* ------------------------------------------------------------------------------------------
 * The forward step whose logits specdec_verify reads: rotary positions, the paged key-value
 * cache (written as the step's rows arrive, optionally quantised, and read back), and the
 * attention of the step's rows over it. The pages describe the step only from outside ("vLLM
 * tour part 2": the target model runs over all draft positions and the bonus position of every
 * request); the operators are this library's, from their formulas.
 *
 * Rows. The layout is the verify's: request b owns the k_b + 1 rows t(b, j) = cu[b] + b + j, and
 * cached_len[b] tokens of it were in the cache before the step. Row j is the request's token
 * number cached_len[b] + j: its default rotary position, its place in the cache, and the last
 * token that its attention sees. After the verify the next step's cached_len[b] is
 * cached_len[b] + out_num_accepted[b] + 1; the cache entries of rejected drafts lie behind it and
 * are written over. A prompt is a request whose k_b + 1 rows are its tokens (the cache write and
 * the rotation take any k_b; the attention takes k_b <= max_k <= SPECDEC_KMAX). A request with
 * cached_len[b] < 0 is skipped (the attention fills its rows with zeros). Rows at and behind cu[B] + B are
 * neither read nor written. A request whose offsets name a row at or behind the `rows` of a call is malformed
 * (BAD_OFFSETS): nothing of it is written.
 *
 * status[b], where a call takes it (NULL: not reported), has bits OR-ed in and is never cleared,
 * so that one array can collect a step's calls. All pointers are device pointers on the current
 * device unless said otherwise; nothing is allocated; every call is asynchronous on `stream`
 * and may be captured into a graph (lengths, offsets and block tables are read on the device, so a
 * replay uses their values at that time). The kernels are launched as programmatic dependents: set up
 * while the work before them in the stream still runs, they wait for its end before they read or write.
 * ------------------------------------------------------------------------------------------ */

/* A rotary embedding. freq[i] (device) is how far the i-th pair turns per position, in units of
 * 2^-64 turn (specdec_rope_frequencies): the angle of position p is p * freq[i] modulo 2^64, exact
 * however far the position. rot_dim (even, 2 <= rot_dim <= head_dim) leading elements of each head
 * are rotated, the others copied. interleaved = 0: element i pairs with i + rot_dim / 2; 1: 2 i
 * with 2 i + 1. cosine and sine are multiplied by amplitude. */
typedef struct {
    const uint64_t* freq;       /* [rot_dim / 2], device */
    int32_t rot_dim;
    int32_t interleaved;
    float amplitude;
} specdec_rope_t;

typedef enum { SPECDEC_ROPE_PLAIN = 0, SPECDEC_ROPE_LINEAR = 1, SPECDEC_ROPE_BY_PARTS = 2 } specdec_rope_scaling_t;

/*
 * specdec_rope_frequencies -- the frequency table of a rotary embedding (host arithmetic in 64
 * bits; freq is HOST memory: copy it to the device once). Pair i of rot_dim / 2 turns by
 * f_i = theta^(-2 i / rot_dim) radians per position;
 *   LINEAR     f_i / factor (position interpolation);
 *   BY_PARTS   f_i (w + (1 - w) / factor), w = (original_len f_i / 2 pi - beta_slow) /
 *              (beta_fast - beta_slow) clamped to [0, 1]: pairs that turn more than beta_fast times
 *              over original_len positions are kept, those under beta_slow are interpolated; and
 *              *amplitude = 0.1 ln(factor) + 1 (factor > 1).
 * PLAIN and LINEAR give amplitude 1. amplitude may be NULL. factor is ignored by PLAIN;
 * original_len, beta_fast and beta_slow matter to BY_PARTS alone.
 * Errors: INVALID_ARG for rot_dim odd, < 2 or > 256, freq NULL, theta < 1 or not finite, factor
 * not in (0, inf) or so small that a frequency is infinite, an unknown scaling, original_len < 1 or
 * beta_fast <= beta_slow where they matter.
 */
specdec_status_t specdec_rope_frequencies(int32_t rot_dim, double theta, specdec_rope_scaling_t scaling,
                                          double factor, int64_t original_len, double beta_fast,
                                          double beta_slow, uint64_t* freq, float* amplitude);

/*
 * specdec_rope -- rotates the heads of `rows` rows: (a, b) -> (a c - b s, b c + a s) for every
 * pair, c = amplitude cos(angle), s = amplitude sin(angle). inverse != 0 turns the other way
 * (s -> -s), which is also the gradient: dx = rope(dout) with inverse = 1.
 *
 *   x, out     [rows, heads, head_dim] of dtype (F32, BF16 or F16), row and head strides in elements,
 *              the elements of a head contiguous. out may be x itself (with x's strides: rotation
 *              in place); any other overlap is undefined. Arithmetic is fp32, rounded once.
 *   positions  [rows] int32: the position of every row (may be negative); or NULL: row j of request
 *              b has position cached_len[b] + j, and rows of skipped or malformed requests and
 *              behind the last request are left as they were.
 *   cu_num_draft [B+1], cached_len [B] int32: used (and required) when positions is NULL.
 * Errors: INVALID_ARG for a NULL required pointer, rows or B < 0, heads < 1, a negative stride or a
 * misaligned pointer; UNSUPPORTED for another dtype, or head_dim odd, < 2 or > 256; CUDA.
 */
specdec_status_t specdec_rope(const void* x, void* out, specdec_dtype_t dtype, int32_t rows, int32_t heads,
                              int32_t head_dim, int64_t x_row_stride, int64_t x_head_stride,
                              int64_t out_row_stride, int64_t out_head_stride, const specdec_rope_t* rope,
                              int32_t inverse, const int32_t* positions, const int32_t* cu_num_draft,
                              const int32_t* cached_len, int32_t B, void* stream);

/* A paged key-value cache. Element (page, head, slot, d) of k and of v lies at
 * page * page_stride + head * head_stride + slot * slot_stride + d (strides in elements, so heads
 * and slots may lie in either order). Token i of request b lives in page block_table[b][i / page_size]
 * at slot i % page_size.
 * dtype BF16, F16 or E4M3. An E4M3 cache has one power-of-two scale for each token and head in
 * k_exp and v_exp, [num_pages, num_kv_heads, page_size] contiguous bytes, 16-byte aligned: the element stands for
 * e4m3 * 2^(byte - 127); 255 stands for NaN. Bytes the library writes are in [1, 254]. */
typedef struct {
    void* k;
    void* v;
    uint8_t* k_exp;             /* E4M3 only, else NULL */
    uint8_t* v_exp;
    specdec_dtype_t dtype;
    int32_t num_pages;
    int32_t page_size;          /* 16, 32, 64, 128 or 256 */
    int32_t num_kv_heads;
    int32_t head_dim;           /* a multiple of 16, at most 128 */
    int64_t page_stride;
    int64_t head_stride;
    int64_t slot_stride;
} specdec_kv_cache_t;

/*
 * specdec_kv_write -- puts the keys and values of a step's rows into the cache: row j of request b
 * as token cached_len[b] + j. With `rope` the keys are rotated on the way, in fp32.
 *
 *   k, v         [rows, num_kv_heads, head_dim] of dtype F32, BF16 or F16; row and head strides in
 *                elements, the same for both (slices of one projection's output, for instance).
 *   rope         NULL: keys are stored as given. positions [rows] int32 or NULL (NULL:
 *                cached_len[b] + j); it moves the rotation only, never the place in the cache.
 *   block_table  [B, max_blocks] int32 with block_stride elements between rows; only entries of
 *                pages that receive a token are read.
 * A stored value is the (rotated) value rounded once, to nearest, ties to even. For an E4M3 cache
 * the scale is the smallest power of two 2^e, e >= -126, with max |finite x| <= 448 * 2^e over the
 * head's elements (2^0 for a head of zeros): a power of two moves no mantissa bit, so the only
 * rounding is that to e4m3. Infinities and NaN are stored as NaN.
 * Two requests of one call that write the same page slot: one of them wins, element by element.
 * status: BAD_LENGTH (cached_len[b] < 0, or a token past max_blocks pages: none of the request's rows
 * are written), BAD_PAGE, BAD_OFFSETS.
 * Errors: INVALID_ARG for a NULL required pointer, a bad size or stride, or a misaligned pointer (k,
 * v of the cache: 16 bytes, and strides of a multiple of 16 bytes); UNSUPPORTED for a dtype,
 * page_size or head_dim outside those above; CUDA.
 */
specdec_status_t specdec_kv_write(const void* k, const void* v, specdec_dtype_t dtype, int32_t rows,
                                  int64_t row_stride, int64_t head_stride, const specdec_rope_t* rope,
                                  const int32_t* positions, const specdec_kv_cache_t* cache,
                                  const int32_t* block_table, int32_t max_blocks, int64_t block_stride,
                                  const int32_t* cached_len, const int32_t* cu_num_draft, int32_t B,
                                  uint32_t* status, void* stream);

/*
 * specdec_kv_read -- reads tokens back into dense rows: out row cu_len[b] + i takes token
 * first[b] + i of request b, i in [0, cu_len[b+1] - cu_len[b]), as the value that the cache holds
 * for it, rounded to out's type (exact where the type holds it).
 *
 *   cu_len       [B+1] int64 offsets, cu_len[0] = 0; rows at and behind cu_len[B] are left as they
 *                were, rows = the row capacity of the outputs.
 *   first        [B] int32 or NULL (0).
 *   out_k, out_v [rows, num_kv_heads, head_dim], F32, BF16 or F16; either may be NULL.
 * status: BAD_LENGTH (first[b] < 0, or a token past max_blocks pages: none of its rows are written),
 * BAD_PAGE (zeros), BAD_OFFSETS (also for rows at or behind `rows`). Errors as specdec_kv_write's.
 */
specdec_status_t specdec_kv_read(const specdec_kv_cache_t* cache, const int32_t* block_table,
                                 int32_t max_blocks, int64_t block_stride, const int32_t* first,
                                 const int64_t* cu_len, int32_t B, int64_t rows, void* out_k, void* out_v,
                                 specdec_dtype_t out_dtype, int64_t out_row_stride, int64_t out_head_stride,
                                 uint32_t* status, void* stream);

/*
 * specdec_paged_attention -- softmax(scale q K^T) V of a step's rows over the paged cache. Row j of
 * request b sees tokens 0 .. cached_len[b] + j of its request (the step's own rows must be in the
 * cache: specdec_kv_write first), or the last `window` of them when window > 0. One row a request
 * (k_b = 0) is plain decoding. Query head h reads key-value head h / (num_heads / num_kv_heads).
 *
 *   q, out       [rows, num_heads, head_dim] of dtype BF16 or F16, each with row and head strides in
 *                elements (multiples of 8; pointers 16-byte aligned). The cache has dtype's own type or
 *                E4M3. out must not overlap q.
 *   lse          [rows, num_heads] fp32 contiguous or NULL: ln(sum exp(scale q k)) of every row and
 *                head, by which partial results over other keys can be joined.
 *   max_k        every k_b must be <= max_k <= SPECDEC_KMAX; it chooses the kernel's row tile.
 *   scale        finite.  window >= 0.
 *   workspace    specdec_paged_attention_workspace_size(...) bytes (0 for sizes that the call refuses),
 *                16-byte aligned, no initialisation; it holds nothing between calls, and calls (or
 *                captured graphs) that share one must not overlap in time.
 *   wait_limit_us -1: 2 s; 0..2000000: the limit of every wait inside the kernel, after which the
 *                requests concerned get SPECDEC_ST_DEVICE_TIMEOUT and undefined outputs; nothing
 *                hangs or traps.
 * Equal calls give equal bits; where the batch's work is cut among the SMs (which depends on all of its
 * lengths) a request's result may differ in its last bits. Scores, maxima, sums and the output are
 * accumulated in fp32. The weights exp(s - m) are rounded to the cache's 16-bit type before their product
 * with V; over an E4M3 cache to F16, times their token's scale relative to the largest scale so far of tokens
 * that all rows computed together see (a head of zeros has 2^0), so a weight whose product falls 2^24 below that
 * is lost; values that only some of those rows see, of a scale 2^100 above it or more, may come out infinite.
 * There Q is taken as a sum of two (BF16) or three (F16) e4m3 numbers an element, exact but for elements under
 * 2^-9 (BF16) or 2^-6 (F16) of the row's largest, which are off by at most 2^-17 of it; an infinity in Q counts
 * as NaN there.
 * Keys and values that a row does not see do not reach it, whatever they hold (infinities, NaN, pages
 * never written; with a window, block_table entries of pages that lie wholly before it are not read).
 * A row that sees no finite score gets zeros and lse = -inf.
 * status: K_TOO_LARGE, BAD_OFFSETS (rows unknown: not written), BAD_LENGTH (both others: zeros, lse -inf in
 * its rows; also 2^31 - 128 tokens or more),
 * BAD_PAGE (its tokens read as zeros), DEVICE_TIMEOUT.
 * Errors: INVALID_ARG for a NULL required pointer, a bad size or stride, num_heads not a multiple of
 * num_kv_heads, a workspace too small or misaligned; UNSUPPORTED for types, page_size or head_dim
 * outside those above; CUDA.
 */
size_t specdec_paged_attention_workspace_size(int32_t B, int32_t max_k, int32_t num_heads,
                                              int32_t num_kv_heads, int32_t head_dim);
specdec_status_t specdec_paged_attention(const void* q, specdec_dtype_t dtype, int32_t rows, int32_t num_heads,
                                         int64_t q_row_stride, int64_t q_head_stride,
                                         const specdec_kv_cache_t* cache, const int32_t* block_table,
                                         int32_t max_blocks, int64_t block_stride, const int32_t* cached_len,
                                         const int32_t* cu_num_draft, int32_t B, int32_t max_k, float scale,
                                         int32_t window, void* out, int64_t out_row_stride,
                                         int64_t out_head_stride, float* lse, uint32_t* status,
                                         void* workspace, size_t workspace_bytes, int32_t wait_limit_us,
                                         void* stream);

/*
 * specdec_kv_fork -- new rows of block tables whose requests go on from other rows' tokens: the paged cache's part of a
 * beam step (specdec_beam_select's out_rows are the parents), or of a prompt that several requests share. Row i
 * takes over the lengths[parent[i]] tokens of its parent. Pages that those fill are shared: their ids are copied. The page that the
 * next token goes to becomes fresh[i], and the tokens that the parent already has there (length modulo page_size of them) are
 * copied into it, keys, values and scales as they are held.
 *
 *   block_table  [sources, max_blocks] of the parents, rows block_stride apart;  lengths [sources].
 *   parent       [n]: 0 .. sources - 1, or -1: an empty row (no pages, length 0).
 *   fresh        [n] or NULL: a page that no row reads or writes and that no other entry names. -1 (NULL: every row): the
 *                parent's page goes on being used, as it does, uncopied, where fresh[i] is that page itself. What is
 *                read of a page that another entry writes is undefined.
 *   out_table    [n, max_blocks] rows out_stride apart, -1 behind each row's last page; it must not overlap block_table.
 *                NULL: not written (the other layers of a model whose caches share one table: with fresh given, only
 *                the tokens are copied).
 *   out_lengths  [n] or NULL; it must not overlap lengths.
 * status, [n] here: BAD_OFFSETS (a parent outside [-1, sources)) and BAD_LENGTH (a negative length, or one past
 * max_blocks pages): an empty row; BAD_PAGE (fresh[i], or the page to be copied, outside [0, num_pages)): nothing is
 * copied and the parent's page stays (-1 where it has none). A length that fills all max_blocks pages leaves no place for fresh[i].
 * Errors: INVALID_ARG for a NULL required pointer (block_table, lengths, parent; one of out_table and fresh), a bad size or
 * stride; UNSUPPORTED for types, page_size or head_dim outside those above; CUDA.
 */
specdec_status_t specdec_kv_fork(const specdec_kv_cache_t* cache, const int32_t* block_table, int32_t max_blocks,
                                 int64_t block_stride, const int32_t* lengths, int32_t sources, const int32_t* parent,
                                 const int32_t* fresh, int32_t n, int32_t* out_table, int64_t out_stride,
                                 int32_t* out_lengths, uint32_t* status, void* stream);

/* ------------------------------------------------------------------------------------------
 * Rows of logits beside the verify: the best ids of every row, the distillation of a drafter from such a record of
 * its target, and a beam step's selection. The operators are this library's, from their formulas.
 *
 * Rows are [rows, V] of dtype F32, BF16 or F16, row_stride elements apart (at least V; any alignment of an element's), V
 * up to 2^30. Pointers, status bits (OR-ed in, never cleared) and streams are as the cache operators', and calls may
 * be captured: everything but sizes is read on the device. temperature (host) is in [1e-4, 1e4]; sums of exponentials
 * are of z / temperature, of which what lies beyond 2 10^38 either way counts as infinite (the lowest finite logit of
 * a masked place as -infinity; ids are still ordered by the logits themselves).
 * ------------------------------------------------------------------------------------------ */
#define SPECDEC_TOP_MAX 128       /* largest n, and the most beams of a request */

/*
 * specdec_top_logits -- the n largest logits of every row: their ids, and their log-probabilities in the softmax of
 * z / temperature over all allowed ids.
 *
 *   bitmask      [rows, W] as the verify's, or NULL (all ids allowed).
 *   out_ids      [rows, n]: largest logit first, the lower id first among equals. -infinity and NaN are never listed;
 *                behind the last id come -1, with log-probability -infinity.
 *   out_logprobs [rows, n] fp32.
 *   lse          [rows] fp32 or NULL: ln(sum exp(z / temperature)) over the allowed ids (-infinity for none). A NaN or
 *                +infinity among them makes it and the row's log-probabilities NaN; the ids stand.
 *   workspace    specdec_top_logits_workspace_size(...) bytes (0 for sizes that the call refuses), 16-byte aligned,
 *                no initialisation; it holds nothing between calls, and calls (or captured graphs) that share one must not overlap in time.
 * status, [rows] here: EMPTY_MASK_ROW where nothing is listed. Equal rows of one alignment give equal bits wherever they stand.
 * Sums are held in fp32 over 4 KB of a row, by a warp, and in pairs of fp32 numbers (some 46 bits) from there on.
 * Errors: INVALID_ARG for a NULL required pointer, n outside [1, SPECDEC_TOP_MAX], a bad size, stride or temperature, a
 * workspace too small or misaligned; UNSUPPORTED for a type or V outside those above, or more than 2^31 units of 4 KB; CUDA.
 */
size_t specdec_top_logits_workspace_size(int32_t rows, int32_t V, specdec_dtype_t dtype);
specdec_status_t specdec_top_logits(const void* logits, specdec_dtype_t dtype, int32_t rows, int32_t V, int64_t row_stride,
                                    const int32_t* bitmask, double temperature, int32_t n, int32_t* out_ids,
                                    float* out_logprobs, float* lse, uint32_t* status, void* workspace,
                                    size_t workspace_bytes, void* stream);

/*
 * specdec_distill -- the loss of a drafter's rows of logits against the top log-probabilities of its target, and its
 * gradient. With s = softmax(z / temperature), t_i = exp(top_logprobs_i) for the ids listed and w = weight[row]:
 *
 *   rest = 1   r = max(0, 1 - sum t) is left to all other ids together, one more category, of which the drafter
 *              gives rho = the sum of s outside the list:
 *              loss = w (sum t_i (ln t_i - ln s_i) + r (ln r - ln rho))
 *              grad_j = w / temperature (M s_j - t_j) on the list, w / temperature (M s_j - r s_j / rho) outside, M = sum t + r
 *   rest = 0   the t_i are divided by their sum, and r = 0.
 * One listed id of log-probability 0 makes it the cross entropy of a label.
 *
 *   top_ids      [rows, n] contiguous, 1 <= n <= SPECDEC_TOP_MAX, in any order; -1 is no entry.
 *   top_logprobs [rows, n] contiguous fp32: at the same temperature as the loss (specdec_top_logits').
 *   weight       [rows] fp32 or NULL (1): a row's factor. A row of weight 0 is not read: its loss and stats are 0, its gradient zeros.
 *   loss         [rows] fp32.
 *   stats        [rows, 2] fp32 contiguous or NULL: ln(sum exp(z / temperature)) over all ids and over those not listed,
 *                which specdec_distill_backward takes.
 *   grad         [rows, V] of the logits' type, rows grad_row_stride elements apart, or NULL (the loss alone). It may be
 *                logits itself (with its stride), and must not overlap it otherwise.
 * Where the drafter leaves nothing to the other ids (none is there, or all are -infinity), r does not count (it is taken as 0).
 * A row without a finite logit: loss +infinity, gradient zeros. A row whose list asks for nothing (rest = 0 and no entry): zeros. NaN or
 * +infinity in a row makes its loss and gradient NaN.
 * status, [rows] here: BAD_TARGET (an id outside [-1, V), one listed before, a log-probability that is NaN, +infinity or, with rest = 1, above
 * 0.5: that entry does not count); EMPTY_MASK_ROW (no finite logit).
 * Sums over the row are held in fp32 by a warp, and in pairs of fp32 numbers (some 46 bits) across them, as are targets, listed
 * exponentials and the loss; an element of the gradient is one fp32 exponential times one factor, rounded once to its type. Equal
 * calls give equal bits.
 * Errors: INVALID_ARG for a NULL required pointer, n, a size, a stride or a temperature outside those above, rest not 0 or 1;
 * UNSUPPORTED for a type or V outside those above, a row of more than 3,276,784 bytes (it is held on chip; the backward call
 * has no such limit, but one of 2^31 CTAs of 32 KB each); CUDA.
 */
specdec_status_t specdec_distill(const void* logits, specdec_dtype_t dtype, int32_t rows, int32_t V, int64_t row_stride,
                                 const int32_t* top_ids, const float* top_logprobs, int32_t n, double temperature,
                                 int32_t rest, const float* weight, float* loss, float* stats, void* grad,
                                 int64_t grad_row_stride, uint32_t* status, void* stream);

/*
 * specdec_distill_backward -- the gradient alone, where the loss's own gradient is known only after the forward pass:
 * grad as above with w = grad_loss[row] (times the forward call's weight, if it had one), from the stats that
 * specdec_distill kept for the same rows, list, temperature and rest. grad may be logits itself. grad_loss NULL: 1.
 * status: BAD_TARGET. Errors as specdec_distill's.
 */
specdec_status_t specdec_distill_backward(const void* logits, specdec_dtype_t dtype, int32_t rows, int32_t V,
                                          int64_t row_stride, const int32_t* top_ids, const float* top_logprobs, int32_t n,
                                          double temperature, int32_t rest, const float* stats, const float* grad_loss,
                                          void* grad, int64_t grad_row_stride, uint32_t* status, void* stream);

/*
 * specdec_beam_select -- the n best continuations of each of B requests with `beams` beams: of beam w (row b * beams + w) and
 * every allowed id v, score = scores[b, w] + ln softmax(z)[v] (over the allowed ids). A finished beam has one
 * continuation, end_token at its own score, and its row is not read; a beam of score -infinity (not begun yet) has none.
 *
 *   bitmask      [B * beams, W] or NULL.   scores [B, beams] fp32.   finished [B, beams] uint8 or NULL (none).
 *   end_token    the id that ends a beam, -1: none (finished must be NULL then).
 *   out_rows     [B, n] int32: the row b * beams + w that each continuation goes on from (specdec_kv_fork's parent), best score
 *                first, the lower row and then the lower id first among equals; behind the last, -1.
 *   out_tokens   [B, n] int32: its id (-1).   out_scores [B, n] fp32 (-infinity).
 *   out_finished [B, n] uint8 or NULL: whether it is finished now (it was, or its id is end_token).
 *   n            1 .. SPECDEC_TOP_MAX, beams up to SPECDEC_TOP_MAX, beams * n <= 4096.
 *   workspace    specdec_beam_select_workspace_size(...) bytes, as specdec_top_logits'.
 * scores may be out_scores and finished out_finished where n = beams. Scores compete in 64 bits (the row's sum of exponentials is held
 * as specdec_top_logits holds it: differences under 10^-6 may fall either way); out_scores is their value in fp32. Of a row, no more
 * than its n best ids are ever candidates; equal logits rank by id.
 * status, [B] here: BAD_SCORE (a score, or a row's logit, that is NaN or +infinity: that beam has no continuation), EMPTY_MASK_ROW (a
 * beam whose row allows nothing). Equal calls give equal bits.
 * Errors: INVALID_ARG for a NULL required pointer, a bad size or stride, end_token outside [-1, V) or -1 with finished, a
 * workspace too small or misaligned; UNSUPPORTED for a type or V outside those above or beams * n > 4096; CUDA.
 */
size_t specdec_beam_select_workspace_size(int32_t B, int32_t beams, int32_t V, specdec_dtype_t dtype, int32_t n);
specdec_status_t specdec_beam_select(const void* logits, specdec_dtype_t dtype, int32_t B, int32_t beams, int32_t V,
                                     int64_t row_stride, const int32_t* bitmask, const float* scores, const uint8_t* finished,
                                     int32_t end_token, int32_t n, int32_t* out_rows, int32_t* out_tokens, float* out_scores,
                                     uint8_t* out_finished, uint32_t* status, void* workspace, size_t workspace_bytes,
                                     void* stream);

/*
 * specdec_wait -- block the calling host thread until all work queued on `stream` has
 * finished, or until timeout_ms milliseconds have passed (polling; timeout_ms < 0 waits
 * without limit). Returns SPECDEC_OK, SPECDEC_ERR_TIMEOUT, or SPECDEC_ERR_CUDA when the
 * stream reports an error.
 */
specdec_status_t specdec_wait(void* stream, int32_t timeout_ms);

/*
 * specdec_set_launch_options -- for comparison and test runs: override the launch choices the
 * library otherwise makes by itself. No step of the method depends on them; every choice
 * computes identical results. Process-wide; set it between calls (a call in flight on another
 * host thread may see either setting). The initial values come once per process from the
 * environment (SPECDEC_KERNEL=cluster|stream, SPECDEC_CTAS_PER_REQUEST=G,
 * SPECDEC_SCHEDULE=1|0); no call reads the environment after that.
 *   kernel            -1: automatic (the streaming kernel); 0: streaming kernel; 1: the
 *                     slice-resident cluster kernel (a slice of every row kept in shared memory
 *                     by a cluster of CTAs per request; slower, kept as an independent
 *                     decomposition of the same computation for cross-checks).
 *   ctas_per_request  -1: automatic; 1..16: CTAs per request (the cluster size).
 *   schedule          -1: automatic (when the batch exceeds one wave of resident CTAs);
 *                     0: never; 1: always, whenever a workspace is given.
 *   wait_limit_us     -1: 2 s; 0..2000000: the limit, in microseconds, of every wait of the
 *                     streaming kernel on one of its barriers (a test sets 0 to make the waits
 *                     expire). When a wait expires the CTA issues no more copies, its other waits
 *                     give up at once, it waits (at most 1 s more) for the copies already in
 *                     flight, and the request gets SPECDEC_ST_DEVICE_TIMEOUT; its other outputs
 *                     are then undefined. Nothing traps or hangs, and later calls are unaffected.
 *   split_requests    -1: automatic; 0: none; n > 0: n. How many of the heaviest requests a
 *                     scheduled launch of one CTA per request (a workspace, no top-k / top-p)
 *                     splits over a cluster of 2 CTAs, the other requests then running two per
 *                     cluster, one per CTA. Automatic: when the batch has more requests than one
 *                     wave of resident CTAs (two per SM), the heaviest sixth of a wave of them.
 * Returns SPECDEC_ERR_INVALID_ARG (nothing changed) for a value outside those ranges.
 */
specdec_status_t specdec_set_launch_options(int32_t kernel, int32_t ctas_per_request, int32_t schedule,
                                            int32_t wait_limit_us, int32_t split_requests);

/* Bytes of workspace specdec_verify uses for B requests of vocabulary size V (0 if B or V <= 0):
 * the request order (int32 per request) and one cost byte per request. */
size_t specdec_workspace_size(int32_t B, int32_t V);

/* Human-readable name of a status code (static storage). */
const char* specdec_status_string(specdec_status_t status);

/*
 * specdec_launch_config -- the launch shape specdec_verify uses for a batch of B requests of
 * vocabulary size V (host arithmetic; the SM count comes from the current device, 152 when none
 * is visible): CTAs per request (a thread-block cluster that splits every vocabulary row into
 * contiguous slices), threads per CTA, dynamic shared memory per CTA in bytes, vocabulary ids
 * per slice, the number of kernels one call launches when given a workspace (2 when the
 * request schedule runs, else 1; without a workspace it is always 1), and how many requests a
 * call with a workspace and without top-k / top-p splits over clusters of 2 CTAs (0: none; the
 * others then run two per cluster, one per CTA, and the grid has 2 * (n + ceil((B - n) / 2))
 * CTAs). Any output pointer may be NULL. Returns SPECDEC_ERR_INVALID_ARG /
 * SPECDEC_ERR_UNSUPPORTED like specdec_verify.
 */
specdec_status_t specdec_launch_config(int32_t B, int32_t V, specdec_dtype_t logits_dtype,
                                       int32_t* ctas_per_request, int32_t* threads_per_cta,
                                       int32_t* smem_bytes, int32_t* slice_ids,
                                       int32_t* kernels_with_workspace, int32_t* split_requests);

#ifdef __cplusplus
}
#endif

#endif /* SPECDEC_H */

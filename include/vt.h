/*
 * vt.h — C ABI of the frequency-ranked trimmed drafter head (GB300, sm_103a).
 *
 * The library implements the data-parallel hot path of vocabulary trimming
 * for speculative-decoding drafters:
 *   offline build : token histogram -> top-V_high selection -> the two index
 *                   maps -> row gather of the kept lm_head rows;
 *   runtime head  : logits over the V_high kept rows only, fused with the
 *                   softmax over that subset, top-k, and the remap of the
 *                   chosen trimmed indices back to full-vocabulary ids.
 *
 * Sources (page title, then section):
 *   [VT] "VocabTrim: Memory-Efficient Vocabulary Pruning for Speculative
 *        Decoding" (skill page, English and Japanese copies), Architecture
 *        Overview and Implementation Steps 1-4.
 *   [FR] "FR-Spec: Accelerating Large-Vocabulary Language Models via
 *        Frequency-Ranked Speculative Sampling" (ACL 2025 paper notes),
 *        Method > Key design "frequency-ranked vocabulary compression".
 *
 * Conventions for every call
 *   - Pointers marked (device) must be device memory of the current CUDA
 *     device (or managed memory); (host) pointers are host memory.
 *   - bf16 tensors are passed as `const uint16_t*` holding the bf16 bit
 *     patterns; all matrices are row-major and densely packed.
 *   - `stream` is a cudaStream_t (NULL = the legacy default stream).  Every
 *     call is asynchronous and stream-ordered; none synchronises, allocates
 *     or frees.  The caller owns every buffer.
 *   - Argument errors are detected on the host before anything is launched
 *     and are returned synchronously (VT_ERR_INVALID_ARG, VT_ERR_WORKSPACE,
 *     VT_ERR_UNSUPPORTED); nothing is written in that case.  A failed launch
 *     returns VT_ERR_CUDA.  vt_last_error() gives a one-line reason for the
 *     latest non-OK status returned on the calling thread.
 *   - Data errors inside buffers (ids outside the vocabulary) never trap:
 *     they are counted into an optional device counter and skipped.
 *   - Calls that take a workspace (`ws`) need one of at least the size the
 *     matching *_workspace_size function returns, 256-byte aligned.  Calls
 *     running concurrently (other streams) need distinct workspaces.
 *   - Error words.  Kernels that wait on other CTAs or on their own copies
 *     (vt_select_vocab's look-back, the head's merges and tensor-core
 *     pipeline) bound every wait (about a second).  A wait that gives up
 *     writes VT_ERR_TIMEOUT to the 32-bit word at byte 128 of the call's
 *     workspace and the kernel returns; the call's outputs are then
 *     incomplete.  The call itself has returned VT_OK by then (it is
 *     asynchronous): read the word after synchronising the stream.
 *     vt_host_step_run reads it for you and returns VT_ERR_TIMEOUT.  After a
 *     timeout the head's counters may be left set: zero-fill its workspace
 *     again before the next call.
 */
#ifndef VT_H_
#define VT_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum vt_status {
  VT_OK = 0,
  VT_ERR_INVALID_ARG = 1, /* null pointer, bad size or alignment */
  VT_ERR_CUDA = 2,        /* a CUDA runtime call or launch failed */
  VT_ERR_UNSUPPORTED = 3, /* valid but outside what this build supports */
  VT_ERR_WORKSPACE = 4,   /* workspace missing, too small or misaligned */
  VT_ERR_TIMEOUT = 5      /* a bounded device wait gave up (see error words) */
} vt_status;

/* Static string naming a status code. */
const char* vt_status_string(int status);

/* One-line reason for the latest non-OK status returned on this thread
 * ("" if none).  The pointer stays valid until the next call on the thread. */
const char* vt_last_error(void);

/* Library ABI version (major * 100 + minor). */
int vt_version(void);

/* ------------------------------------------------------------------------
 * Debug builds.  The library can be compiled with VT_CHECKS defined (the
 * build script's checked variant, libvt_gb300_checks.so): every kernel then
 * tests the indices of its index-computed global accesses, skips an access
 * that would fall outside its buffer and records the source line of the
 * first such check.  Nothing traps.  The release build has no checks.
 *
 *   vt_debug_build   1 in a checked build, 0 otherwise.
 *   vt_debug_checks  after the work has finished (it reads device memory
 *                    synchronously): 0 if no check failed since the last
 *                    call, else the source line of a failed check (then
 *                    cleared); -1 if the words could not be read.  Always 0
 *                    in a release build.
 * ------------------------------------------------------------------------ */
int vt_debug_build(void);
int vt_debug_checks(void);

/* vt_selftest_check — one kernel whose bounds check fails by design, to see
 * the debug build's reporting work: it writes buf[i] = i for i = 0 .. n with
 * each write guarded by a check that allows only i < n.  buf (device,
 * uint32[n + 1], 4-byte aligned) holds every index, so nothing lands outside
 * it in either build; a release build writes all n + 1 values, a checked
 * build skips buf[n] and vt_debug_checks() then reports the check's line.
 * 1 <= n <= 2^30.  Argument errors return VT_ERR_INVALID_ARG with nothing
 * launched. */
vt_status vt_selftest_check(uint32_t* buf, int32_t n, void* stream);

/* ------------------------------------------------------------------------
 * vt_workspace_size — workspace bytes of one operation, in one call; the
 * same numbers as the per-operation *_workspace_size functions below.
 *
 *   op  VT_OP_COUNT  (vt_count_tokens):  n = V, the vocabulary size;
 *       VT_OP_SELECT (vt_select_vocab):  n = V;
 *       VT_OP_HEAD   (vt_draft_head, vt_draft_head_ex): M, n = V_high, k;
 *       VT_OP_Q      (vt_draft_q):       M.
 *   Arguments an operation does not use are ignored.  Returns 0 for an
 *   unknown op or sizes out of range.  (vt_draft_head_sets takes per-set
 *   sizes: use vt_draft_head_sets_workspace_size.)
 * ------------------------------------------------------------------------ */
typedef enum {
  VT_OP_COUNT = 0,
  VT_OP_SELECT = 1,
  VT_OP_HEAD = 2,
  VT_OP_Q = 3
} vt_op;
size_t vt_workspace_size(int32_t op, int32_t M, int32_t n, int32_t k);

/* ------------------------------------------------------------------------
 * vt_count_tokens — token-frequency histogram.
 * [VT] Step 1 counts every sampled id into a dict; [FR] Key design counts
 * corpus tokens.  Here the stream is counted into a dense array.
 *
 *   tokens    (device) int32[n], any values; 16-byte aligned.
 *   n         number of tokens, 0 <= n < 2^40.
 *   V         vocabulary size, 1 <= V <= 2^30.
 *   counts    (device) uint32[V]; ACCUMULATED INTO (counts[id] += hits), so
 *             a long stream may be counted in pieces.  Zero it before the
 *             first piece.  Arithmetic is modulo 2^32 per id.
 *   n_invalid (device, nullable) uint64[1]; accumulated: the number of
 *             tokens outside [0, V), which are not counted anywhere.
 *   ws        (device) workspace of vt_count_tokens_workspace_size(V) bytes.
 * ------------------------------------------------------------------------ */
size_t vt_count_tokens_workspace_size(int32_t V);
vt_status vt_count_tokens(const int32_t* tokens, int64_t n, int32_t V,
                          uint32_t* counts, uint64_t* n_invalid, void* ws,
                          size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------
 * vt_select_vocab — top-V_high selection and the two index maps.
 * [VT] Step 2: sort ids by count descending, keep the first V_high; the
 * trimmed index of an id is its rank; coverage = selected / total.
 * Tie rule (the pages leave it to dict order): lower id first, so the
 * result is unique.  Ids with count 0 take part, so exactly V_high ids are
 * always kept.
 *
 *   counts    (device) uint32[V].
 *   V_high    1 <= V_high <= V.
 *   t2f       (device) int32[V_high]: trimmed index -> full id, rank order
 *             (t2f[0] is the most frequent id).
 *   f2t       (device) int32[V]: full id -> trimmed index, -1 if dropped.
 *   sums      (device) uint64[2]: OVERWRITTEN with {kept, total}: the sum of
 *             the kept ids' counts and of all counts.  Coverage is
 *             (double)kept / (double)total, computed by the caller after
 *             the stream is synchronised (NaN when total == 0).
 *   ws        (device) workspace of vt_select_vocab_workspace_size(V) bytes;
 *             no zero-fill needed.  Its 32-bit word at byte 128 is the
 *             call's error word: cleared when the call starts, then 0, or
 *             VT_ERR_TIMEOUT if a look-back wait gave up (t2f, f2t and sums
 *             are then incomplete).
 * ------------------------------------------------------------------------ */
size_t vt_select_vocab_workspace_size(int32_t V);
vt_status vt_select_vocab(const uint32_t* counts, int32_t V, int32_t V_high,
                          int32_t* t2f, int32_t* f2t, uint64_t* sums,
                          void* ws, size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------
 * vt_gather_rows — reconstruct the trimmed lm_head.
 * [VT] Step 3: W_high = W[trimmed_to_full, :], W stored [vocab, hidden].
 * A bit-exact copy of V_high rows of d bf16 values.
 *
 *   W         (device) bf16[V, d], 16-byte aligned.
 *   d         hidden size, d > 0 and d % 8 == 0.
 *   t2f       (device) int32[V_high].
 *   W_high    (device) bf16[V_high, d], 16-byte aligned, must not overlap W.
 *   n_invalid (device, nullable) uint64[1]; accumulated: rows whose t2f
 *             entry lies outside [0, V); such rows are written as zeros.
 * ------------------------------------------------------------------------ */
vt_status vt_gather_rows(const uint16_t* W, int64_t V, int32_t d,
                         const int32_t* t2f, int32_t V_high, uint16_t* W_high,
                         uint64_t* n_invalid, void* stream);

/* ------------------------------------------------------------------------
 * vt_gather_bias — the kept rows' bias.  [VT] Step 3 copies the old head's
 * bias with the kept ids when the head has one: b_high[i] = b[t2f[i]].
 *
 *   b         (device) float[V], 4-byte aligned.
 *   t2f       (device) int32[V_high].
 *   b_high    (device) float[V_high], must not overlap b.
 *   n_invalid (device, nullable) uint64[1]; accumulated: entries whose t2f
 *             id lies outside [0, V); they are written as 0.
 * ------------------------------------------------------------------------ */
vt_status vt_gather_bias(const float* b, int64_t V, const int32_t* t2f,
                         int32_t V_high, float* b_high, uint64_t* n_invalid,
                         void* stream);

/* ------------------------------------------------------------------------
 * vt_draft_head — one draft step of the trimmed head for M hidden states.
 * [FR] Key design: the draft lm_head projects onto the V_high kept rows only
 * and the softmax is taken over that subset; [VT] Step 4: softmax of the
 * drafter logits, then the chosen trimmed index is mapped back to the full
 * vocabulary through trimmed_to_full before verification.
 *
 *   logit[m][i] = sum_j H[m][j] * W_high[i][j]   (bf16 inputs, fp32 sums)
 *   p[m][i]     = exp(logit[m][i] - max_i) / sum_i exp(logit[m][i] - max_i)
 *   out         = the k largest logits of row m, in descending order;
 *                 out_ids = t2f[i] (full-vocabulary ids), out_probs = p.
 *   Equal logits are ordered by lower full-vocabulary id.
 *
 *   H         (device) bf16, M rows of d values, row stride ldh elements
 *             (ldh >= d, ldh % 8 == 0), 16-byte aligned.
 *   M         number of hidden states (draft-tree nodes), 1 <= M <= 256.
 *   d         hidden size, d % 8 == 0, 8 <= d <= 16384.
 *   W_high    (device) bf16[V_high, d], 16-byte aligned.
 *   V_high    1 <= V_high < 2^31.
 *   t2f       (device, nullable) int32[V_high]; NULL means the identity,
 *             i.e. the untrimmed head over a full vocabulary of V_high rows.
 *   k         1 <= k <= 32 and k <= V_high.  k = 1 is the greedy argmax.
 *   out_ids   (device) int32[M, k].
 *   out_probs (device) float[M, k].
 *   out_logits(device, nullable) float[M, V_high]: every trimmed logit, for
 *             verification; costs an extra write of M*V_high*4 bytes.
 *   ws        (device) workspace of vt_draft_head_workspace_size(M, V_high,
 *             k) bytes.  It must be zero-filled once before its first use;
 *             the counters it holds are left zero by every call.  For
 *             M >= 2 it also holds the [M, V_high] fp32 logits (when
 *             out_logits is NULL).  On every path the 32-bit word at byte
 *             128 is a device error word: 0, or VT_ERR_TIMEOUT if a bounded
 *             wait inside the kernel gave up (readable after a synchronise;
 *             the outputs of that call are then incomplete).  The head never
 *             clears it: a caller that reads a non-zero word writes 0 back.
 *
 * Paths: M = 1 runs a split-V GEMV (CUDA cores, one launch); M >= 2 runs a
 * tcgen05 tensor-core GEMM over all M rows at once plus a per-row softmax
 * and top-k kernel.  One workspace can serve calls of any M.
 * The head's kernels are launched as programmatic dependents of the work
 * ahead of them in the stream: they may become resident while the previous
 * kernel finishes and ask L2 for their first W_high rows meanwhile (a
 * prefetch hint), but read H, t2f, the bias and the workspace, and write
 * anything, only after that kernel has completed; stream order is kept.
 * ------------------------------------------------------------------------ */
size_t vt_draft_head_workspace_size(int32_t M, int32_t V_high, int32_t k);
vt_status vt_draft_head(const uint16_t* H, int32_t M, int32_t d, int64_t ldh,
                        const uint16_t* W_high, int32_t V_high,
                        const int32_t* t2f, int32_t k, int32_t* out_ids,
                        float* out_probs, float* out_logits, void* ws,
                        size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------
 * vt_draft_head_ex — vt_draft_head with options: a bias on the kept rows,
 * a temperature, and drawing from the trimmed distribution instead of
 * taking its top-k.  [VT] Step 3 copies the optional bias of the kept rows
 * with the weight rows (b_high = b[t2f], gathered by the caller); [VT] Step 4
 * draws the draft token from the trimmed softmax with multinomial.  Draws
 * here use the Gumbel-max rule, which draws from the same distribution:
 *
 *   logit[m][i] = sum_j H[m][j] * W_high[i][j] + bias_high[i]
 *   s[m][i]     = logit[m][i] / temperature
 *   p[m][i]     = exp(s[m][i] - max_i s) / sum_i exp(s[m][i] - max_i s)
 *   score       = s                         (VT_HEAD_TOPK)
 *               = s + g(seed, offset, m, t2f[i])   (VT_HEAD_SAMPLE)
 *   out         = the k largest scores of row m, descending (ties: lower
 *                 full id); out_ids = full ids, out_probs = their p,
 *                 out_logits = logit (bias included, before temperature).
 *
 * In VT_HEAD_SAMPLE mode, k = 1 is one draw from p and k > 1 is k draws
 * without replacement.  g is Gumbel noise from the counter-based generator
 * Philox4x32-10 (Salmon et al., SC 2011): x = word 0 of the block at counter
 * (full id, m, offset low 32 bits, offset high 32 bits) and key (seed low,
 * seed high); u = ((x >> 9) + 0.5) / 2^23; g = -log(-log(u)).  Noise is
 * keyed by the full-vocabulary id, so it does not depend on which tokens
 * were kept: whenever the untrimmed head's draw (same seed, offset, m) is a
 * kept token, the trimmed head draws that same token.  Callers advance
 * `offset` once per draft step; m is the hidden state's row in this call.
 *
 *   opts      (host, nullable) options; NULL means no bias, temperature 1,
 *             VT_HEAD_TOPK (exactly vt_draft_head).
 *             bias_high   (device, nullable) float[V_high], 4-byte aligned.
 *             temperature finite and > 0.
 *             mode        VT_HEAD_TOPK or VT_HEAD_SAMPLE.
 *             seed, offset generator key and step counter (sampling only).
 *   Other arguments, the workspace (same size function) and the error word
 *   are those of vt_draft_head; invalid options return VT_ERR_INVALID_ARG.
 * ------------------------------------------------------------------------ */
typedef enum { VT_HEAD_TOPK = 0, VT_HEAD_SAMPLE = 1 } vt_head_mode;

typedef struct {
  const float* bias_high;
  float temperature;
  int32_t mode;
  uint64_t seed;
  uint64_t offset;
} vt_head_options;

vt_status vt_draft_head_ex(const uint16_t* H, int32_t M, int32_t d,
                           int64_t ldh, const uint16_t* W_high,
                           int32_t V_high, const int32_t* t2f, int32_t k,
                           const vt_head_options* opts, int32_t* out_ids,
                           float* out_probs, float* out_logits, void* ws,
                           size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------
 * vt_draft_noise — the Gumbel noise g(seed, offset, m, id) that
 * vt_draft_head_ex adds in VT_HEAD_SAMPLE mode, for n full-vocabulary ids;
 * for verifying draws.  The pages have no counterpart; it is the same
 * device function the sampling kernels call.
 *
 *   full_ids  (device) int32[n];  out (device) float[n];  n >= 0, m >= 0.
 *   Stream-ordered and asynchronous.
 * ------------------------------------------------------------------------ */
vt_status vt_draft_noise(uint64_t seed, uint64_t offset, int32_t m,
                         const int32_t* full_ids, int64_t n, float* out,
                         void* stream);

/* ------------------------------------------------------------------------
 * vt_draft_head_sets — one draft step for hidden states that use different
 * kept vocabularies.  [FR] Limitations: the kept set is one static,
 * corpus-wide vocabulary; vocabularies chosen per domain or per request are
 * future work.  Each set s has its own W_high_sets[s] [V_high_sets[s], d],
 * t2f_sets[s] and optional bias_sets[s], built by the same offline calls
 * from its own token stream; hidden state m is scored against set
 * set_of_row[m] exactly as vt_draft_head_ex would score it alone, and when
 * drawing its noise index is its row m in this call.
 *
 *   H, M (1..256), d, ldh, k, opts, out_ids, out_probs: as vt_draft_head_ex
 *             (opts->bias_high must be NULL: biases are per set).
 *   set_of_row  (host) int32[M], 0 <= set_of_row[m] < S.
 *   W_high_sets (host) array of S device pointers, 16-byte aligned.
 *   V_high_sets (host) int32[S], each >= k.
 *   t2f_sets    (host, nullable) array of S device pointers (entries may
 *               be NULL: identity).
 *   bias_sets   (host, nullable) array of S device pointers (nullable
 *               entries), fp32 [V_high_sets[s]], 4-byte aligned.
 *   ws          (device) vt_draft_head_sets_workspace_size(M, d, k, S,
 *               V_high_sets) bytes, 256-byte aligned, zero-filled once
 *               before its first use.  It begins with the head's workspace,
 *               so its error word is the head's (byte 128).
 * For each set in use: one gather of its rows' hidden states, the head
 * (GEMV for one row, tensor cores for more), one scatter of its outputs.
 * All sets are checked before anything is launched.
 * ------------------------------------------------------------------------ */
size_t vt_draft_head_sets_workspace_size(int32_t M, int32_t d, int32_t k,
                                         int32_t S, const int32_t* V_high_sets);
vt_status vt_draft_head_sets(const uint16_t* H, int32_t M, int32_t d,
                             int64_t ldh, const int32_t* set_of_row, int32_t S,
                             const uint16_t* const* W_high_sets,
                             const int32_t* V_high_sets,
                             const int32_t* const* t2f_sets,
                             const float* const* bias_sets, int32_t k,
                             const vt_head_options* opts, int32_t* out_ids,
                             float* out_probs, void* ws, size_t ws_bytes,
                             void* stream);

/* ------------------------------------------------------------------------
 * vt_draft_q — the full-vocabulary draft distribution of a draft step, for
 * verification.  [FR] Method > Key design: only the draft step is trimmed;
 * the target model verifies with its accept/reject test (rejection
 * sampling), which keeps the output exactly the target's distribution and
 * compares target and draft probabilities over the whole vocabulary, where
 * the trimmed draft gives every dropped id probability 0:
 *
 *   q[m][f] = exp(logits[m][f2t[f]] / T - max) / sum   if f2t[f] >= 0
 *           = 0                                        otherwise,
 *   max, sum over the V_high kept logits of row m (softmax of logit / T).
 *
 *   logits    (device) float[M, V_high], 4-byte aligned: the head's logits
 *             (vt_draft_head / _ex out_logits, bias included).
 *   f2t       (device, nullable) int32[V] from vt_select_vocab; NULL means
 *             the identity (requires V == V_high).
 *   V         full vocabulary size, V >= V_high; 1 <= M <= 65535.
 *   temperature  finite and > 0 (the head's T).
 *   q         (device) float[M, V], 4-byte aligned (16-byte aligned rows
 *             and V % 4 == 0 take the vector path), must not overlap logits.
 *   ws        (device) vt_draft_q_workspace_size(M) bytes, 8-byte aligned;
 *             holds per-row (max, sum); no zero-fill needed.
 * ------------------------------------------------------------------------ */
size_t vt_draft_q_workspace_size(int32_t M);
vt_status vt_draft_q(const float* logits, int32_t M, int32_t V_high,
                     const int32_t* f2t, int32_t V, float temperature,
                     float* q, void* ws, size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------
 * vt_selftest_wait_timeout — runs the library's bounded device wait until it
 * gives up, to check the failure path.  The pages have no counterpart.
 *
 * Every wait of the library's kernels on an mbarrier is bounded by a cycle
 * budget (about a second); when it runs out the kernel writes
 * VT_ERR_TIMEOUT to its error word (byte 128 of the head workspace), stops
 * issuing work and returns, and the context stays usable.  This call
 * launches one 32-thread CTA that waits on an mbarrier nothing arrives on,
 * with the given budget, then writes VT_ERR_TIMEOUT to *err_word.
 *
 *   err_word      (device) uint32, 4-byte aligned; set to VT_ERR_TIMEOUT.
 *   budget_cycles 1 .. 2^31 SM clock cycles (2e6 is about a millisecond).
 * Argument errors return VT_ERR_INVALID_ARG with nothing launched.
 * ------------------------------------------------------------------------ */
vt_status vt_selftest_wait_timeout(uint32_t* err_word, int64_t budget_cycles,
                                   void* stream);

/* ------------------------------------------------------------------------
 * vt_host_step_* — draft steps from host memory, each one CUDA-graph launch.
 * The pages have no counterpart; this serves callers whose hidden states
 * live on the host.  The handle owns a stream, pinned staging buffers,
 * device buffers, a zero-filled head workspace and a CUDA graph of: copy of
 * the staged H [M, d] to the device, then vt_draft_head_ex writing the ids
 * and probabilities straight into a pinned host buffer (device-addressable;
 * no copy node follows).
 *
 *   vt_host_step_create: W_high, V_high, d, t2f, M (1..256), k and opts are
 *     fixed for the handle's life (W_high and t2f must stay valid); opts may
 *     set a bias and a temperature, not VT_HEAD_SAMPLE (a replayed graph
 *     would repeat its step counter).  Runs one step eagerly, then captures.
 *     This call allocates and synchronises; the run call does neither.
 *   vt_host_step_run: copies H_host (host, bf16 [M, d]; skipped when it is
 *     the staging buffer) into the staging buffer, launches the graph,
 *     waits for the step and writes ids_host [M, k] and probs_host [M, k]
 *     (host).  The graph ends with a small kernel that moves the head's
 *     error word (byte 128 of the handle's workspace) into the pinned output
 *     buffer, clears it, and then publishes the step's sequence number there
 *     behind a system-scope fence; the call waits by polling that number
 *     (a stream synchronise takes over after ~10-50 ms, and its error, if
 *     any, is returned as VT_ERR_CUDA).  The graph's last kernel may still
 *     be exiting when the call returns; the next run queues behind it.  If a
 *     bounded wait inside the head gave up, the call returns VT_ERR_TIMEOUT
 *     and writes nothing.  Not thread-safe per handle.
 *   vt_host_step_staging: the pinned [M, d] staging buffer (write H there to
 *     skip the host copy).
 *   vt_host_step_error_word: the device address of the handle's error word
 *     (uint32), for tools and tests of the failure path.
 *   vt_host_step_destroy: synchronises and frees everything (NULL is a no-op).
 * ------------------------------------------------------------------------ */
typedef struct vt_host_step vt_host_step;
vt_status vt_host_step_create(const uint16_t* W_high, int32_t V_high, int32_t d,
                              const int32_t* t2f, int32_t M, int32_t k,
                              const vt_head_options* opts, vt_host_step** out);
vt_status vt_host_step_run(vt_host_step* h, const uint16_t* H_host,
                           int32_t* ids_host, float* probs_host);
uint16_t* vt_host_step_staging(vt_host_step* h);
uint32_t* vt_host_step_error_word(vt_host_step* h);
void vt_host_step_destroy(vt_host_step* h);

/* ------------------------------------------------------------------------
 * vt_draft_head_noalloc — vt_draft_head for callers that cannot allocate.
 * The pages have no counterpart to this call; it exists for integration.
 *
 * Some callers cannot allocate device memory where they run a draft step
 * (inside a CUDA stream capture that must not gain allocation nodes, on
 * hosts that forbid allocation after start-up, or as a plugin confined to
 * another framework's memory pool), so they cannot provide the workspace
 * vt_draft_head needs.  This call computes what vt_draft_head computes,
 * with the same arguments minus the workspace, and allocates nothing: its
 * scratch is one fixed 1 MiB array in device memory that the library
 * defines and every GPU that loads the library keeps until exit.
 * It always runs the GEMV kernel, four hidden states at a time.  For M = 1
 * that is vt_draft_head's own kernel.  For M >= 2 vt_draft_head uses the
 * tensor-core path, which sums in another order, so the two calls agree
 * within the head's tolerances (logits within 1e-3 * (1 + |logit|),
 * probabilities within 1e-4), and their ids agree except where two
 * candidates' logits are closer than that.
 *
 *   Limit     the GEMV scratch, 2048 + 4096 * min(M, 4) * P bytes with
 *             P = 4 + 2k rounded up to a multiple of 4, must fit in 1 MiB:
 *             any k <= 32 for M <= 3, k <= 28 for M >= 4; larger requests
 *             return VT_ERR_UNSUPPORTED.
 *   Set-up    the first call on each device looks up the array's device
 *             address and zero-fills its counters with a synchronous
 *             cudaMemset; make that first call before any stream capture.
 *   Sharing   all calls on a device share the one array; calls that overlap
 *             on the GPU (unordered streams) race on it and give wrong
 *             results.  Calls on one stream are safe.
 *   Timeouts  the kernel's one bounded wait (the final merge's copy of the
 *             partial results, about a second) cannot be reported by this
 *             call: its error word lies inside the private array and no
 *             call returns it, nor clears it.  When that wait gives up the
 *             call leaves the out_ids rows from the one it failed on
 *             unwritten.  A caller that must detect this fills out_ids with
 *             -1 before the call (no full-vocabulary id is negative) and
 *             checks for -1 after synchronising.
 * ------------------------------------------------------------------------ */
vt_status vt_draft_head_noalloc(const uint16_t* H, int32_t M, int32_t d,
                                int64_t ldh, const uint16_t* W_high,
                                int32_t V_high, const int32_t* t2f, int32_t k,
                                int32_t* out_ids, float* out_probs,
                                float* out_logits, void* stream);

/* ------------------------------------------------------------------------
 * Element types of the calls below (they take `void*` and one of these).
 * ------------------------------------------------------------------------ */
typedef enum { VT_BF16 = 0, VT_FP16 = 1, VT_FP32 = 2 } vt_dtype;

/* ------------------------------------------------------------------------
 * vt_quantize_rows — rows as 8-bit integers with one scale a row: the kept
 * lm_head rows (gathered through t2f, as vt_gather_rows does) or the hidden
 * states of a draft step, for vt_matmul_i8.  The pages have no counterpart;
 * the head is bound by its weights' bytes, which this halves.
 *
 *   x        = row ids[r] of X (row r without ids)
 *   scale[r] = max(max_j |x_j| * (1/127), 2^-126)   (fp32 product, 1/127 in
 *              fp32)
 *   Q[r][j]  = the integer nearest to x_j / scale[r] (the quotient itself,
 *              not a rounded one; ties to even), within [-127, 127]
 *   A row with an infinity or a NaN gets integers 0 and scale NaN, so that
 *   products with it are NaN.
 *
 *   X         (device) dtype[V, d], row stride ldx elements, ldx >= d when
 *             V > 1, ldx * element size % 16 == 0; 16-byte aligned.
 *   d         16 <= d <= 16384, d % 16 == 0.
 *   ids       (device, nullable) int32[R], 4-byte aligned; NULL means the
 *             rows of X in order (R == V).  The same id may come twice.
 *   Q         (device) int8[R, d], 16-byte aligned.
 *   scale     (device) float[R], 4-byte aligned.
 *   n_invalid (device, nullable) uint64[1]; accumulated: rows whose id lies
 *             outside [0, V); their integers and their scale are 0.
 *   R == 0 is a valid no-op.
 * ------------------------------------------------------------------------ */
vt_status vt_quantize_rows(const void* X, int32_t dtype, int64_t V, int32_t d,
                           int64_t ldx, const int32_t* ids, int32_t R,
                           int8_t* Q, float* scale, uint64_t* n_invalid,
                           void* stream);

/* ------------------------------------------------------------------------
 * vt_matmul_i8 — product of 8-bit rows with a scale for each row of both
 * operands (token and channel): the logits of a head quantised with
 * vt_quantize_rows.
 *
 *   out[m][n] = float(sum_k X[m][k] * W[n][k]) * (x_scale[m] * w_scale[n])
 *               + bias[n]
 *   The sum is exact (32-bit integers; any int8 values, -128 included); each
 *   of the other operations rounds to fp32 once, bf16 outputs once more.
 *
 *   X         (device) int8[M, d], 16-byte aligned; 0 <= M <= 65535.
 *   W         (device) int8[N, d], 16-byte aligned; 0 <= N <= 2^30.
 *   d         16 <= d <= 16384, d % 16 == 0.
 *   x_scale, w_scale  (device) float[M], float[N].
 *   bias      (device, nullable) float[N].
 *   out       (device) out_dtype[M, N] with row stride ldo >= N (any when
 *             M == 1); VT_FP32 or VT_BF16.  Must not overlap an input;
 *             elements of a row past N are left as they were.
 *   ws        (device) vt_matmul_i8_workspace_size() bytes, 256-byte aligned,
 *             zero-filled once before its first use.  It holds nothing but
 *             the error word (byte 128), so calls may share it, concurrent
 *             ones and captured ones too; which of them it speaks of is then
 *             not known.  The call never clears the word.
 *   M == 0 or N == 0 is a valid no-op.
 * ------------------------------------------------------------------------ */
size_t vt_matmul_i8_workspace_size(void);
vt_status vt_matmul_i8(const int8_t* X, const float* x_scale, int32_t M,
                       const int8_t* W, const float* w_scale, int32_t N,
                       int32_t d, const float* bias, void* out,
                       int32_t out_dtype, int64_t ldo, void* ws,
                       size_t ws_bytes, void* stream);

/* vt_selftest_matmul_i8 — vt_matmul_i8 with waits of budget_cycles SM clock
 * cycles at the most (1 .. 2^31) in place of about a second, to see its failure
 * path work: a wait that runs out writes VT_ERR_TIMEOUT to the error word, the
 * loads and products under way are waited for, and out is incomplete; where the
 * word stays 0 out is the product.  For sizes whose kernel has such waits
 * (more than 16 rows of X, or more than 4 with many rows of W); others are
 * VT_ERR_UNSUPPORTED. */
vt_status vt_selftest_matmul_i8(const int8_t* X, const float* x_scale, int32_t M,
                                const int8_t* W, const float* w_scale, int32_t N,
                                int32_t d, const float* bias, void* out,
                                int32_t out_dtype, int64_t ldo, void* ws,
                                size_t ws_bytes, int64_t budget_cycles, void* stream);

/* ------------------------------------------------------------------------
 * vt_sample_logits — sampling with temperature, top-k, top-p and min-p from
 * given random numbers, and the distribution that is sampled from.  [VT]
 * Step 4 draws the draft token from the softmax; serving filters that
 * distribution first, and the acceptance test has to see the filtered one.
 *
 *   w_i = exp((x_i - max x) / T).  Sorted by x descending, equal logits by
 *   lower index, the filters apply in this order, each to what the one
 *   before it left:
 *     top_k  the first top_k logits (0, or >= n: all);
 *     top_p  the shortest prefix whose mass is at least top_p of the mass
 *            (>= 1: all; the first logit always stays);
 *     min_p  the logits with w_i >= min_p (<= 0: all; > 1 counts as 1).
 *   S = sum of the kept w, p_i = w_i / S (0 where dropped).
 *   The draw is the first index i in the order of the logits with
 *   (sum of kept w_j over j <= i) > u * S; out_ids = t2f[i], or i;
 *   out_probs = p_i.  out_dist[m][i] = p_i.
 *
 *   Temperatures between 0 and 1e-30 count as 1e-30 in the weights.
 *   T == 0 is greedy: the first maximum, with probability 1.  Logits of -inf
 *   are never drawn; +inf logits share the mass equally.  A row that is all
 *   -inf gives id -1 and probability 0 (and a distribution of zeros); a row
 *   with a NaN logit, a negative or non-finite temperature, a NaN or negative
 *   setting where that has no meaning (top_p, min_p NaN; top_k < 0) or a u
 *   outside [0, 1] gives id -1 and NaN.  u == 1 draws the last kept token
 *   of positive weight.
 *   Weights are summed exactly in fixed point (largest 2^42, each within
 *   2^-28 of its value), so results do not depend on the launch.
 *
 *   logits    (device) dtype[M, n], row stride ld >= n (any when M == 1),
 *             aligned to the element; 0 <= M <= 65535, 1 <= n <= 2^19
 *             (beyond either: VT_ERR_UNSUPPORTED).
 *   opts      (host, nullable) settings; NULL means T = 1 and no filter.  A
 *             device array [M], where given, replaces the value for all rows.
 *   u         (device) float[M] uniforms in [0, 1), with out_ids int32[M]
 *             and out_probs float[M]: all three or none.
 *   t2f       (device, nullable) int32[n].
 *   out_dist  (device, nullable) float[M, n], row stride ld_dist >= n.
 *             Elements of a row past n are left as they were.  Required when
 *             u is NULL.
 *   Outputs must not overlap an input or each other.
 *   No workspace.  M == 0 is a valid no-op.
 * ------------------------------------------------------------------------ */
typedef struct {
  float temperature;
  int32_t top_k;
  float top_p;
  float min_p;
  const float* temperature_rows; /* (device, nullable) float[M] */
  const int32_t* top_k_rows;     /* (device, nullable) int32[M] */
  const float* top_p_rows;       /* (device, nullable) float[M] */
  const float* min_p_rows;       /* (device, nullable) float[M] */
} vt_sample_options;

vt_status vt_sample_logits(const void* logits, int32_t dtype, int32_t M,
                           int32_t n, int64_t ld,
                           const vt_sample_options* opts, const float* u,
                           const int32_t* t2f, int32_t* out_ids,
                           float* out_probs, float* out_dist, int64_t ld_dist,
                           void* stream);

/* ------------------------------------------------------------------------
 * vt_verify_draft — the acceptance test over a chain of drafted tokens.
 * [FR] Method > Key design: verification by rejection sampling keeps the
 * output exactly the target's distribution.  For sequence b:
 *
 *   position j = 0, 1, .. is accepted while u[b][j] * q[b][j][x_j] <
 *   p[b][j][x_j] (fp64), x_j = draft_ids[b][j], j < n_draft[b];
 *   n_accepted[b] = a, the number accepted;
 *   r_i = max(p[b][a][i] - q[b][a][i], 0) if a < n_draft[b], else p[b][a][i];
 *   next = the first id i with (sum of r_j over j <= i) > u[b][K] * sum r;
 *   out_ids[b] = the a accepted tokens, next, then -1.
 *
 *   If r is zero everywhere (p nowhere above q) next is drawn from p; if p
 *   is zero too, or u[b][K] is outside [0, 1], next is -1.  A drafted id
 *   outside [0, V) is rejected.  Probabilities count as 0 when negative or
 *   NaN and as 1 when above 1 in r, whose terms are summed in fixed point
 *   (2^-44).
 *
 *   draft_ids (device) int32[B, K]; n_draft (device, nullable) int32[B],
 *             clamped to [0, K]; NULL means K for every sequence.
 *   p         (device) float, row of V at p + b * p_seq + j * p_pos, j = 0 .. K
 *             (vt_sample_logits' out_dist of the target's logits).
 *   q         (device) float, row of Vq at q + b * q_seq + j * q_pos, j < K.
 *   f2t       (device, nullable) int32[V]: column of q of each id, -1 (or
 *             any value outside [0, Vq)) where q is 0.  NULL: Vq == V.
 *   u         (device) float[B, K + 1].
 *   n_accepted (device) int32[B]; out_ids (device) int32[B, K + 1].  Neither
 *             may overlap an input or the other.
 *   0 <= B, K <= 65535 and 1 <= V <= 2^19 (beyond: VT_ERR_UNSUPPORTED).
 *   K == 0 draws from p[b][0].  No workspace.  B == 0 is a valid no-op.
 * ------------------------------------------------------------------------ */
vt_status vt_verify_draft(const int32_t* draft_ids, const int32_t* n_draft,
                          int32_t B, int32_t K, int32_t V, const float* p,
                          int64_t p_seq, int64_t p_pos, const float* q,
                          int64_t q_seq, int64_t q_pos, int32_t Vq,
                          const int32_t* f2t, const float* u,
                          int32_t* n_accepted, int32_t* out_ids, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* VT_H_ */

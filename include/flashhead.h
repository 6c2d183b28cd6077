/*
 * flashhead.h — C ABI of libflashhead, an MI355X (gfx950) implementation of
 * FlashHead inference: a drop-in replacement for a language model's dense
 * output head z = E h by two-stage retrieval over a balanced clustering of
 * E's rows.
 *
 * Sources, cited by page title and section:
 *   [X]  FlashHead technical explainer (framerc.cn), §1.1 dense head cost,
 *        §1.2.1 balanced clustering and the dense C2T table, §1.2.2 multi-probe
 *        top-p retrieval, §1.2.3 multinomial probe sampling with temperature,
 *        §1.2.4 selective (INT4 stage-1) quantisation, §2.2.2 the computation
 *        graph h -> centroid scores -> top-p clusters -> token scores,
 *        §2.3 the quantisation config (centroid int4, token bf16).
 *   [A]  "FlashHead: Efficient Drop-In Replacement for the Classification Head
 *        in Language Model Inference" (arXiv 2603.14591), abstract,
 *        innovations (1)-(4).
 *
 * Conventions for every entry point:
 *   - Tensors are dense and row-major.  "Device" pointers address GPU memory
 *     on the engine's device; "host" pointers address CPU memory.
 *   - Work is enqueued on the HIP stream passed as `stream` (NULL = the
 *     default stream) and the call returns without waiting for it, except
 *     fh_create, which waits for its own set-up work.  Outputs are valid once
 *     that stream has reached the call.
 *   - Argument errors are detected before anything is enqueued: the call
 *     returns FH_EINVAL or FH_EUNSUPPORTED, writes nothing, and
 *     fh_last_error() describes the problem.  A failing HIP call returns
 *     FH_EHIP; allocation failure returns FH_ENOMEM.
 *   - Results are deterministic: the same inputs, p, mode, temperature and
 *     seed give bit-identical outputs on the same device.
 *   - One engine may be used from several threads only if the calls do not
 *     overlap: calls share the engine's workspace.
 */
#ifndef FLASHHEAD_H
#define FLASHHEAD_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct fh_engine fh_engine; /* opaque */

typedef enum {
  FH_OK = 0,
  FH_EINVAL = -1,       /* invalid argument                                 */
  FH_ENOMEM = -2,       /* device or host allocation failed                 */
  FH_EHIP = -3,         /* a HIP runtime call or kernel launch failed       */
  FH_EUNSUPPORTED = -4  /* valid, but outside what this library implements  */
} fh_status;

/* Storage type shared by E, C and h. */
typedef enum { FH_F32 = 0, FH_BF16 = 1 } fh_dtype;

/* Stage-1 centroid storage ([X] §1.2.4, §2.3; the W4A16 and W8A16 rows of
 * the tuning table, [X] §5.2).  Both integer forms are symmetric with one
 * fp16 scale per 32 consecutive elements of a centroid row:
 * sigma = fp16_rne(amax / qmax) (fp32 division), q = clamp(rint(x / sigma),
 * -qmax, qmax) with ties to even, q = 0 where sigma = 0; the score is
 * sum_g sigma_g sum_{i in g} q_i h_i.  Queries and token embeddings stay in
 * the engine's dtype. */
typedef enum {
  FH_QUANT_NONE = 0,      /* centroids used as given                         */
  FH_QUANT_INT4_G32 = 1,  /* qmax 7, two's-complement nibbles                */
  FH_QUANT_INT8_G32 = 2   /* qmax 127, int8                                  */
} fh_quant;

/* `mode` is the OR of one probe flag and one token flag. */
enum {
  FH_PROBE_TOPK = 0,   /* the p highest-scoring clusters ([X] §1.2.2)       */
  FH_PROBE_SAMPLE = 1, /* p distinct clusters drawn from softmax(s/T)
                          without replacement ([X] §1.2.3)                  */
  FH_TOKEN_ARGMAX = 0, /* highest logit among retrieved tokens              */
  FH_TOKEN_SAMPLE = 2, /* one draw from softmax(z/T) over retrieved tokens  */
  FH_PROBE_SHARED = 4  /* one probe set for the whole batch: the p clusters
                          with the largest summed score sum_b s[b, k]
                          (ties to the smaller id) -- [X] §4.2's shared
                          selection across samples, read this way; changes
                          results for B > 1, equals FH_PROBE_TOPK at B = 1;
                          not combinable with FH_PROBE_SAMPLE               */
};

/*
 * fh_create — build an engine over one output head.
 *
 *   E        device, [v x d] of `dtype`: output embeddings, one row per token
 *            ([X] §1.1).  BORROWED: not copied; keep it alive and unchanged
 *            until fh_destroy.
 *   C        device, [c x d] of `dtype`: cluster centroids ([X] §1.2.1).
 *            Borrowed for FH_QUANT_NONE.  For FH_QUANT_INT4_G32 and
 *            FH_QUANT_INT8_G32 it is read once here and may be freed after
 *            the call returns.
 *   C2T      HOST, [c x b] int32 with b = v / c: C2T[k*b + j] is the token in
 *            slot j of cluster k ([X] §1.2.1, [A] (1)).  Copied.  Must hold
 *            every token of [0, v) exactly once (balanced clustering).
 *   v, d, c  vocabulary size, hidden size, cluster count; v % c == 0.
 *            d % 4 == 0 for FH_F32, d % 8 == 0 for FH_BF16, and
 *            d % 32 == 0 with a quantised stage 1.  c <= 16384; d <= 4096
 *            for FH_BF16, d <= 2048 for FH_F32 (else FH_EUNSUPPORTED).
 *   quant    FH_QUANT_INT4_G32 / FH_QUANT_INT8_G32 quantise C here (the
 *            scheme above, qmax 7 or 127).  A scale that overflows fp16
 *            gives FH_EINVAL.
 *   max_batch largest B any later call will use (sizes the workspace).
 *            Besides the workspace, the engine keeps a cluster-contiguous
 *            copy of E (v x d of `dtype`, row f = E[C2T[f]]) so that each
 *            probe's b rows are read as one block ([X] §1.2.1); FH_ENOMEM if
 *            it does not fit.
 *   stream   stream for the set-up work; fh_create waits for it.
 *   out      receives the engine (set only on FH_OK).
 */
fh_status fh_create(const void* E, const void* C, const int32_t* C2T, fh_dtype dtype,
                    int64_t v, int64_t d, int64_t c, fh_quant quant, int64_t max_batch,
                    void* stream, fh_engine** out);

/* fh_destroy — release everything the engine owns (NULL is a no-op).  Waits
 * for the device to finish work that may still use it. */
void fh_destroy(fh_engine* e);

/*
 * fh_forward — one FlashHead call over B hidden states ([X] §2.2.2).
 *
 *   h        device, [B x d] of the engine's dtype.
 *   B        1 <= B <= max_batch.
 *   p        probes per query, 1 <= p <= c ([X] §1.2.2).
 *   mode     FH_PROBE_* | FH_TOKEN_*.
 *   temperature  > 0 when either stage samples ([X] §1.2.3); otherwise
 *            ignored.  One temperature serves both stages.
 *   seed     keys the Philox4x32-10 stream of every draw: probe k of row b
 *            uses counter (k/4, b, 0, 0), token t uses (t/4, b, 1, 0), key
 *            (seed mod 2^32, seed >> 32), word k mod 4 (resp. t mod 4),
 *            u = ((w >> 9) + 1/2) 2^-23, Gumbel noise -ln(-ln u).
 *
 * Outputs (device; any of the last four may be NULL to skip it):
 *   out_token        [B] int32: the chosen token id.
 *   out_token_logit  [B] float: its logit z = E[token] . h.
 *   out_lse          [B] float: log sum exp(z / T') over the retrieved
 *                    tokens, T' = temperature if tokens are sampled, else 1.
 *   out_clusters     [B x p] int32: the probed clusters, ascending id.
 *   out_ids          [B x p*b] int32: retrieved token ids, in cluster order
 *                    (ascending id) then slot order.
 *   out_logits       [B x p*b] float: their logits z = E[t] . h (float32
 *                    accumulation of the stored values).
 * Selection keys are compared in float32; equal keys go to the smaller
 * cluster / token id.
 */
fh_status fh_forward(fh_engine* e, const void* h, int64_t B, int64_t p, int mode,
                     float temperature, uint64_t seed, int32_t* out_token,
                     float* out_token_logit, float* out_lse, int32_t* out_clusters,
                     int32_t* out_ids, float* out_logits, void* stream);

/*
 * fh_forward_adaptive — fh_forward with a probe count per query ([X] §1.2.2:
 * the number of probes adapts to the distribution of h; §4.2: fewer probes
 * for confident queries, such as frequent tokens).  The pages give no
 * formula; this library's reading: the clusters are taken in the order of the
 * selection keys (by score, or with FH_PROBE_SAMPLE the draws without
 * replacement from softmax(s/T)), and query b stops at the first count n whose
 * clusters hold at least tau of softmax(s/T) over all c clusters; n is then
 * clamped to [p_min, p_max].  The mass is accumulated in float32.
 *   p_min, p_max  1 <= p_min <= p_max <= min(c, 1024).
 *   tau           in (0, 1].
 *   mode          FH_PROBE_TOPK or FH_PROBE_SAMPLE | FH_TOKEN_*; not
 *                 FH_PROBE_SHARED (FH_EINVAL).  temperature > 0 always (it
 *                 sets the mass even for greedy calls).
 *   out_nprobe    device [B] int32: n per query, or NULL.
 *   out_clusters  device [B x p_max] int32 or NULL: the n probes ascending,
 *                 then -1.
 *   out_ids, out_logits  device [B x p_max b] or NULL: the n b retrieved
 *                 tokens (cluster ascending, slot order), then id -1 and
 *                 logit -inf.
 *   out_token, out_token_logit, out_lse: as for fh_forward, over the n b
 *                 retrieved tokens.
 * B = 1 runs the single launch of fh_forward (its selector takes the count
 * and publishes only the kept probes); larger batches, stream capture and
 * FH_PATH_MULTI run per-stage launches (stage 1, selection of p_max, the
 * count, stage 2 over the kept probes, finish).  Stream-ordered, no host
 * synchronisation.
 */
fh_status fh_forward_adaptive(fh_engine* e, const void* h, int64_t B, int64_t p_max,
                              int64_t p_min, float tau, int mode, float temperature,
                              uint64_t seed, int32_t* out_nprobe, int32_t* out_token,
                              float* out_token_logit, float* out_lse, int32_t* out_clusters,
                              int32_t* out_ids, float* out_logits, void* stream);

/*
 * fh_probs_fp8 — the candidates' probabilities in fp8 ([X] §2.3: the
 * quantisation config keeps the probability intermediate as fp8).  Per row
 * q, p = exp(logits[q*n + i] / T' - lse[q]) (a -inf logit, an empty adaptive
 * slot, gives 0).  The pages do not say how the fp8 tensor is scaled; here a
 * power of two per row: k = 8 - e for the row's largest p = f 2^e, f in
 * [1/2, 1), which puts it in [128, 256) (no saturation, exact scaling, 17
 * binades below it).  out_probs[q*n + i] = E4M3(p 2^k), the OCP E4M3 byte
 * (sign, 4 exponent bits with bias 7, 3 mantissa bits, no infinities, 0x7F
 * NaN) rounded to nearest even; out_scale_exp[q] = k, so p = value(byte)
 * 2^-k.  Engine-free; stream-ordered.
 *   logits     device [B x n] float, e.g. fh_forward's out_logits (n = p b)
 *              or fh_forward_adaptive's (n = p_max b).
 *   lse        device [B] float: each row's log-sum-exp taken at T'
 *              (fh_forward's out_lse).
 *   temperature  T' > 0, the temperature of that LSE: the call's temperature
 *              when tokens were sampled, else 1.
 *   out_probs  device [B x n] uint8; out_scale_exp device [B] int32.
 * FH_EINVAL for NULL pointers, B outside [1, 65535], n outside [1, 2^31] or
 * a temperature that is not finite and > 0.
 */
fh_status fh_probs_fp8(const float* logits, const float* lse, int64_t B, int64_t n,
                       float temperature, uint8_t* out_probs, int32_t* out_scale_exp,
                       void* stream);

/*
 * fh_forward_noalloc — fh_forward without an engine and without allocating:
 * for callers that cannot call hipMalloc (code under HIP graph capture,
 * tight serving loops, harnesses that forbid it).  It runs the per-stage
 * launches (stage-1 scores, selection, stage 2, finish) on caller-owned
 * tables and keeps its workspace (scores, probe lists, stage-2 partials) in
 * a fixed 8 MiB device array of the library, one per GPU, held until the
 * process ends; it calls no hipMalloc, hipFree or allocating routine.
 *
 *   E, C     device [v x d] and [c x d] of dtype, 16-byte aligned (as for
 *            fh_create; C as stored, no quantisation).
 *   c2t      device int32 [c x b], b = v / c: a permutation of [0, v) (the
 *            caller's responsibility; fh_create checks it, this does not).
 *   h        device [B x d] of dtype, 16-byte aligned; 1 <= B <= 65535.
 *   p, mode, temperature, seed, outputs: as for fh_forward, except that
 *            FH_PROBE_SHARED is not offered (FH_EUNSUPPORTED).
 * Results equal fh_forward's per-stage path (fh_set_path FH_PATH_MULTI)
 * bit for bit.  FH_EINVAL, before anything is launched, when the call's
 * workspace, 4 B c + 4 B p + 20 B ceil(p b / 8) bytes (each term rounded up
 * to 256), exceeds 8 MiB, and for the argument errors of fh_create and
 * fh_forward.  Every call on a GPU shares that GPU's array, and the array
 * keeps the last call's contents (each call writes all it reads, so nothing
 * needs clearing): calls that overlap on one GPU (other streams, other
 * threads) race and must be serialised by the caller.
 */
fh_status fh_forward_noalloc(const void* E, const void* C, const int32_t* c2t, fh_dtype dtype,
                             int64_t v, int64_t d, int64_t c, const void* h, int64_t B, int64_t p,
                             int mode, float temperature, uint64_t seed, int32_t* out_token,
                             float* out_token_logit, float* out_lse, int32_t* out_clusters,
                             int32_t* out_ids, float* out_logits, void* stream);

/*
 * fh_score — stage 1 alone: out_scores[b*c + k] = C_hat[k] . h[b] in float32
 * accumulation, with C_hat the centroids as stored (INT4: sigma * q)
 * ([X] §1.2.4 stage 1).
 *   h device [B x d]; out_scores device [B x c] float.  1 <= B <= max_batch.
 */
fh_status fh_score(fh_engine* e, const void* h, int64_t B, float* out_scores, void* stream);

/*
 * fh_dense_forward — the dense head z = E h over all v tokens ([X] §1.1),
 * finished exactly like fh_forward (argmax or one draw from softmax(z/T), the
 * same Philox stream for tokens, LSE over all v).  The comparison baseline.
 *   out_logits may be NULL; otherwise device [B x v] float.
 */
fh_status fh_dense_forward(fh_engine* e, const void* h, int64_t B, int mode,
                           float temperature, uint64_t seed, int32_t* out_token,
                           float* out_token_logit, float* out_lse, float* out_logits,
                           void* stream);

/*
 * fh_get_int4 — copy the engine's quantised centroids out (FH_QUANT_INT4_G32
 * only, else FH_EINVAL).
 *   packed  device [c x d/2] uint8: two's-complement nibbles, element 2m in
 *           the low nibble of byte m.
 *   scales  device [c x d/32] uint16: fp16 bit patterns of sigma.
 */
fh_status fh_get_int4(fh_engine* e, uint8_t* packed, uint16_t* scales, void* stream);

/*
 * fh_get_int8 — copy the engine's INT8 centroids out (FH_QUANT_INT8_G32
 * only, else FH_EINVAL).
 *   codes   device [c x d] int8, row-major.
 *   scales  device [c x d/32] uint16: fp16 bit patterns of sigma.
 */
fh_status fh_get_int8(fh_engine* e, int8_t* codes, uint16_t* scales, void* stream);

/*
 * fh_spec_verify — verify B FlashHead draft tokens against the dense head
 * with the standard speculative-sampling rule ([X] §4.2 speculative
 * decoding: a FlashHead draft, the original head's probabilities, accept or
 * reject; the rule is Leviathan et al. 2023 / Chen et al. 2023).  Query q
 * is one position with hidden state h[q]:
 *   p(t) = softmax(E h / T) over all v tokens;
 *   q(t) = softmax(E_t h / T) over the retrieved tokens of the draft's
 *          probes, 0 elsewhere (what the draft sampled from);
 *   the draft token x is kept when u < min(1, p(x) / q(x)) with
 *   u = Philox uniform (seed, q, 0, stage 2); otherwise the output is a draw
 *   from max(0, p - q), i.e. from p over the tokens outside the probes
 *   (Gumbel-max with Philox (seed, q, t, stage 3)).
 * The output token is distributed exactly as p.  As both heads score a
 * retrieved token with the same E_t . h, p(x) / q(x) = exp(draft_lse -
 * LSE_full) for x inside the probes.
 *   h               device [B x d] of the engine's dtype, 16-byte aligned.
 *   p               probes per draft, 1 <= p <= c.
 *   draft_clusters  device [B x p] int32: the draft's probes (out_clusters
 *                   of fh_forward); ids outside [0, c) are ignored.
 *   draft_token     device [B] int32: the draft's tokens (out_token of
 *                   fh_forward with FH_TOKEN_SAMPLE at this temperature); a
 *                   token outside [0, v) is rejected, one outside its own
 *                   probes (q = 0) is kept.
 *   draft_lse       device [B] float: the draft's out_lse (log sum exp(z/T)
 *                   over its retrieved tokens).
 *   temperature     T > 0, the draft's temperature.
 *   out_token       device [B] int32: the verified token.
 *   out_accepted    device [B] int32, may be NULL: 1 where the draft was kept.
 *   out_lse         device [B] float, may be NULL: log sum exp(z/T) over all v.
 * Uses the engine's workspace like the other calls (B <= max_batch).
 */
fh_status fh_spec_verify(fh_engine* e, const void* h, int64_t B, int64_t p,
                         const int32_t* draft_clusters, const int32_t* draft_token,
                         const float* draft_lse, float temperature, uint64_t seed,
                         int32_t* out_token, int32_t* out_accepted, float* out_lse,
                         void* stream);

/*
 * Per-kernel timing.  fh_profile_begin(e, n) makes the engine record a HIP
 * event pair on the launch stream around each of its next n kernel launches.
 * fh_profile_end waits for those events and fills up to `max` records
 * (kernel name, launches, total milliseconds) aggregated by kernel, returning
 * how many it wrote in *count.  Names point to static strings.
 */
typedef struct {
  const char* name;
  int64_t launches;
  double total_ms;
} fh_kernel_time;

fh_status fh_profile_begin(fh_engine* e, int64_t max_launches);
fh_status fh_profile_end(fh_engine* e, fh_kernel_time* out, int max, int* count);

/*
 * fh_set_path — choose how fh_forward runs a batch-1 call.
 *   FH_PATH_AUTO  (default) one launch for the whole call when p probes fit
 *                 it: stage-1 workgroups, a selecting workgroup, stage-2
 *                 workgroups and a finishing workgroup hand over through
 *                 device memory.  Batches of B > 1 use one launch per stage.
 *   FH_PATH_MULTI always one launch per stage.
 * Both paths return the same ids and logits; the LSE may differ in the last
 * bits (a different merge order).  While `stream` is being captured into a
 * graph, fh_forward uses the per-stage launches whatever the path: they keep
 * no state between calls, so the graph can be replayed (the single launch
 * tells calls apart by a counter kept on the host).
 */
enum { FH_PATH_AUTO = 0, FH_PATH_MULTI = 1 };
fh_status fh_set_path(fh_engine* e, int path);

/*
 * fh_sync_status — wait for `stream`, then report FH_OK, or FH_EHIP if a
 * bounded wait inside a batch-1 call ever gave up (that call's outputs are
 * invalid; the flag stays set).  Calls that overlap on one engine (see
 * above) are what can cause it.
 */
fh_status fh_sync_status(fh_engine* e, void* stream);

/*
 * Offline clustering: the step that produces C and C2T for fh_create
 * ([X] §1.2.1 balanced clustering, §2.1 offline clustering; [A] abstract,
 * innovation (1)).  Balanced spherical k-means: rows are L2-normalised; c
 * centres are seeded with k-means++; every iteration computes the cosine
 * similarity of every token to every centre, assigns tokens so that every
 * cluster holds exactly b = v / c of them, and moves every centre to the
 * normalised mean of its tokens.  The pages leave these steps open; this
 * library reads them as:
 *   - k-means++ on the sphere: D(t) = 1 - max_j cos(t, C_j); centre 0 is
 *     token floor(u[0] v); centre i is the first token, in id order, whose
 *     running sum of D^2 exceeds u[i] * sum(D^2) (token floor(u[i] v) if
 *     every D is 0).  The uniforms u are inputs, so a run is repeatable.
 *   - balanced assignment by rounds: each unassigned token proposes to its
 *     most similar cluster that is not yet full (ties: smaller cluster id);
 *     each cluster accepts, up to its remaining room, the proposals with the
 *     highest similarity (ties: smaller token id); accepted tokens are final
 *     and the rest propose again.
 *   - update: C_k = normalise(sum of its tokens' unit rows); C2T[k] lists
 *     cluster k's tokens in ascending id.
 * Both calls allocate their own device workspace, run on `stream`, and
 * return after waiting for it (the rounds need the host).
 */

/*
 * fh_balanced_assign — the balanced assignment alone.
 *   sims        device [v x c] float: similarity of token t to cluster k at
 *               sims[t * c + k]; compared as given (no NaN).
 *   v, c        v a positive multiple of c; b = v / c tokens per cluster.
 *   out_assign  device [v] int32: the cluster of every token.
 *   out_rounds  host, may be NULL: the number of rounds taken.
 */
fh_status fh_balanced_assign(const float* sims, int64_t v, int64_t c, int32_t* out_assign,
                             int* out_rounds, void* stream);

typedef struct {
  float init_ms;  /* normalisation and k-means++ seeding                    */
  float sims_ms;  /* the similarity products, summed over iterations        */
  float total_ms; /* the whole call                                         */
  float pp_step_us; /* average duration of the k-means++ distance refresh
                       (one pass over the table), from HIP events around
                       every 16th launch                                    */
  int rounds;     /* balanced-assignment rounds, summed over iterations     */
} fh_cluster_times;

/*
 * fh_cluster — the whole offline clustering.
 *   E           device [v x d] of `dtype` (rows need not be unit length).
 *   v, d, c     v a positive multiple of c, c <= 65536; d as for fh_create
 *               (a multiple of 8 for bf16, of 4 for f32; at most 4096 bf16
 *               or 2048 f32 elements).
 *   iters       >= 1 iterations of (similarities, assignment, update).
 *   u           host [c] double, each in [0, 1): the k-means++ uniforms.
 *   out_C       device [c x d] float: unit centres after the last update.
 *   out_c2t     device [c x b] int32: C2T from the last assignment.
 *   out_init    device [c] int32, may be NULL: the k-means++ token ids.
 *   out_assign  device [v] int32, may be NULL: the last assignment.
 *   out_times   host, may be NULL.
 * out_C and out_c2t are what fh_create takes (after a cast of C to `dtype`
 * for bf16 engines).
 */
fh_status fh_cluster(const void* E, fh_dtype dtype, int64_t v, int64_t d, int64_t c, int iters,
                     const double* u, float* out_C, int32_t* out_c2t, int32_t* out_init,
                     int32_t* out_assign, fh_cluster_times* out_times, void* stream);

/*
 * Around the dense head: the final norm that makes its input, a dense head
 * whose operands are both int8 (W8A8), and the rules a server applies to
 * logits before a token is chosen.  These calls need no fh_engine.  They run
 * on the current device (fh_w8a8_*: the handle's device) and keep no state
 * between calls: scratch memory is the caller's (`workspace`, of the size
 * that the matching *_workspace call returns, 16-byte aligned, read and
 * written only by the call it is given to), so calls on different streams or
 * captured graphs overlap freely if their workspaces and outputs differ.
 * Row strides (ld_*) are in elements.
 */

/*
 * fh_rmsnorm — root-mean-square norm of B rows with the residual's addition,
 * and an int8 output with a scale per row.  Per row, in float32:
 *   s = x + residual;  y = s / sqrt(mean(s^2) + eps) * (weight_offset + weight)
 *   out = y rounded to dtype;  out_residual = s rounded to dtype
 *   out_scale = max |y| / 127;  out_q = rint(y / out_scale) (ties to even,
 *   within [-127, 127]; 0 where out_scale is 0)
 * The norm and the codes are taken from the unrounded s and y.  A row that
 * holds an infinity or NaN, or whose sum of squares exceeds float32, has an
 * out_scale or out that says so (NaN, or 0 from the infinite norm) and codes
 * that mean nothing; so does a row of zeros with eps = 0, and without eps a row
 * whose mean square is below float32's normal range (2^-126) loses precision.
 *   x             device [B x d] of dtype, row stride ld_x >= d.
 *   residual      the same, row stride ld_residual; NULL: s = x.
 *   weight        device [d] of dtype; NULL: the factor is 1.
 *   weight_offset 0, or 1 for norms stored as (1 + w); unused without weight.
 *   eps           >= 0.
 *   out, out_residual  device [B x d] of dtype, out_q device [B x d] int8, with
 *                 their row strides, out_scale device [B] float.  Any of out,
 *                 out_residual and the pair (out_q, out_scale) may be NULL,
 *                 not all.  out or out_residual may be x or residual itself
 *                 (same address and stride); no other overlap.
 * 1 <= B < 2^31, 1 <= d < 2^31.  Any alignment of the elements' own size.
 */
fh_status fh_rmsnorm(const void* x, int64_t ld_x, const void* residual, int64_t ld_residual,
                     const void* weight, fh_dtype dtype, int64_t B, int64_t d, float eps,
                     float weight_offset, void* out, int64_t ld_out, void* out_residual,
                     int64_t ld_out_residual, int8_t* out_q, int64_t ld_q, float* out_scale,
                     void* stream);

/* An int8 weight matrix [n x k] with a float scale per row (output channel). */
typedef struct fh_w8a8 fh_w8a8; /* opaque */

/*
 * fh_w8a8_create — quantise W, device [n x k] of dtype, dense: per row
 * scale = max |W| / 127 (float32 division), code = rint(W / scale) (ties to
 * even, within [-127, 127]; 0 where scale is 0).  A row that holds an infinity
 * or NaN gives FH_EINVAL.
 * fh_w8a8_create_codes — take codes [n x k] int8 (-128 included) and scales
 * [n] float as they are, both device and dense.
 * Both copy into the handle's own layout (n k bytes, n rounded up to 16 and k
 * to 128, plus 4 n), wait for `stream`, and keep nothing of their arguments.
 * 1 <= n <= 2^27, 1 <= k < 131072 (the int32 sums of the product are exact).
 * Not while `stream` is being captured.
 */
fh_status fh_w8a8_create(const void* W, fh_dtype dtype, int64_t n, int64_t k, void* stream,
                         fh_w8a8** out);
fh_status fh_w8a8_create_codes(const int8_t* codes, const float* scales, int64_t n, int64_t k,
                               void* stream, fh_w8a8** out);

/* fh_w8a8_destroy — release the handle (NULL is a no-op), after waiting for
 * the device to finish work that may still read it (so not while a stream is
 * being captured).  Captured graphs that use it end with it. */
void fh_w8a8_destroy(fh_w8a8* w);

/* fh_w8a8_get — copy the codes [n x k] and scales [n] out (device). */
fh_status fh_w8a8_get(const fh_w8a8* w, int8_t* codes, float* scales, void* stream);

/*
 * fh_w8a8_workspace — bytes of workspace that a fh_w8a8_matmul (forward = 0)
 * or fh_w8a8_forward (forward = 1) call with these q, ld_q and B needs, or a
 * negative fh_status.  0 for a product whose rows are aligned to 16 bytes.
 */
int64_t fh_w8a8_workspace(const fh_w8a8* w, const int8_t* q, int64_t ld_q, int64_t B, int forward);

/*
 * fh_w8a8_matmul — out[b, j] = (sum_i q[b, i] code[j, i]) (q_scale[b] scale[j]),
 * the sum exact in int32, the two products rounded to float32, then to bf16
 * for out_dtype FH_BF16.
 *   q        device [B x k] int8, row stride ld_q >= k.
 *   q_scale  device [B] float.
 *   out      device [B x n] of out_dtype, row stride ld_out >= n.
 *   workspace, workspace_bytes  see fh_w8a8_workspace (NULL, 0 if that is 0).
 * 1 <= B <= 65535, and ceil(n / 256) ceil(B / 128) < 2^23 for B > 64 (a launch's
 * threads).  q and out may have any alignment of their elements' size.
 */
fh_status fh_w8a8_matmul(const fh_w8a8* w, const int8_t* q, int64_t ld_q, const float* q_scale,
                         int64_t B, void* out, int64_t ld_out, fh_dtype out_dtype, void* workspace,
                         int64_t workspace_bytes, void* stream);

/*
 * fh_w8a8_forward — the dense head on that product: fh_dense_forward's
 * choice over the n logits of each row (argmax or one draw from softmax(z / T)
 * with the same Philox stream, LSE over all n; z / T is z times 1 / T rounded, so
 * a draw between keys that differ by a float32 rounding may fall otherwise).
 * +inf is drawn before any finite logit, the smallest token of several.
 *   mode, temperature, seed   as for fh_dense_forward.
 *   out_token  [B] int32: the token, -1 where no logit of the row is above
 *              -inf (NaN is never chosen).
 *   out_token_logit, out_lse  [B] float or NULL; out_logits [B x n] float,
 *              row stride ld_logits, or NULL.
 */
fh_status fh_w8a8_forward(const fh_w8a8* w, const int8_t* q, int64_t ld_q, const float* q_scale,
                          int64_t B, int mode, float temperature, uint64_t seed,
                          int32_t* out_token, float* out_token_logit, float* out_lse,
                          float* out_logits, int64_t ld_logits, void* workspace,
                          int64_t workspace_bytes, void* stream);

/*
 * fh_logit_rules — what a server lays on the logits of each row before it
 * chooses a token.  All pointers are device memory; a NULL one leaves its rule
 * out; penalties without a history do nothing.  Token ids outside [0, v) in
 * history and bias_ids are skipped.
 */
typedef struct {
  const int32_t* history;     /* [B x history_len] token ids, row stride ld_history */
  int64_t ld_history;
  int64_t history_len;
  const int32_t* n_prompt;    /* [B] ids at the row's start that are its prompt; NULL: 0 */
  const int32_t* n_history;   /* [B] ids of the row that count, clamped to
                                 [0, history_len]; NULL: history_len */
  const float* repetition;    /* [B] > 0: ids in prompt or output, z > 0 ? z (1 / r) : z r */
  const float* frequency;     /* [B]: z -= f times its count in the output */
  const float* presence;      /* [B]: z -= p if it is in the output */
  const int32_t* bias_ids;    /* [B x bias_len] ids, row stride ld_bias */
  const float* bias;          /* [B x bias_len], the same stride: z += each listed
                                 bias; an id listed several times takes their sum,
                                 added up in the list's order */
  int64_t ld_bias;
  int64_t bias_len;
  const int32_t* n_bias;      /* [B] entries that count, clamped; NULL: bias_len */
  const uint32_t* mask;       /* [mask_rows x ceil(v / 32)] words, row stride ld_mask:
                                 token t is allowed where bit t % 32 of word t / 32 is set */
  int64_t ld_mask;
  int64_t mask_rows;
  const int32_t* mask_row;    /* [B] the mask row of each row, outside [0, mask_rows):
                                 all allowed; NULL: row b takes mask row b */
} fh_logit_rules;

/*
 * fh_logits_workspace — bytes of workspace that are enough for a
 * fh_logits_apply call over [B x n] logits that asks for tokens or LSEs (0 for
 * short rows, and for a call that does not), or FH_EINVAL.
 */
int64_t fh_logits_workspace(int64_t B, int64_t n);

/*
 * fh_logits_apply — the rules, then the choice of the token.  Per row b and
 * token t with logit z, in float32 and in this order: the repetition, the
 * frequency and the presence penalty, the bias, and -inf where the mask does
 * not allow t (whatever z was, NaN too).  Then the choice over the row as
 * fh_w8a8_forward's: argmax or a draw from softmax(z / T), the same Philox
 * stream, LSE.
 *   logits   device [B x n] float, row stride ld_logits: of all tokens (ids
 *            NULL, n = v), e.g. fh_dense_forward's or fh_w8a8_matmul's, or of
 *            the tokens in ids, e.g. fh_forward's out_logits and out_ids.
 *   ids      device [B x n] int32, row stride ld_ids, or NULL.  An id outside
 *            [0, v) is no token: its logit becomes -inf.  Every place of an id
 *            listed several times gets the same rules.
 *   rules    host, the struct of device pointers; NULL: no rules.
 *   mode     FH_TOKEN_ARGMAX or FH_TOKEN_SAMPLE; temperature > 0 to sample.
 *   out_logits  device [B x n] float, row stride ld_out, or NULL; may be
 *            logits itself (same address and stride).
 *   out_token   [B] int32 or NULL: the token; ties go to the smaller id; -1
 *            where no logit is above -inf (NaN is never chosen).
 *   out_token_logit, out_lse  [B] float or NULL: its logit after the rules
 *            (-inf for token -1); log sum exp(z / T') over the row (-inf where
 *            nothing is left, NaN where an allowed logit is NaN).
 * 1 <= B <= 65535, 1 <= n, v <= 2^30, lists of at most 2^30 places.  At least
 * one output.
 */
fh_status fh_logits_apply(const float* logits, int64_t ld_logits, const int32_t* ids,
                          int64_t ld_ids, int64_t B, int64_t n, int64_t v,
                          const fh_logit_rules* rules, int mode, float temperature, uint64_t seed,
                          float* out_logits, int64_t ld_out, int32_t* out_token,
                          float* out_token_logit, float* out_lse, void* workspace,
                          int64_t workspace_bytes, void* stream);

/*
 * Around an fp8 head: hidden states in 8-bit floating point (OCP E4M3: bias 7,
 * finite to 448, no infinities, NaN 0x7F and 0xFF) with a float scale per 128
 * elements of a row (the last group of a row may be shorter), a weight with a
 * scale per block of 128 x 128, their product and the dense head on it.
 */

/*
 * fh_rmsnorm_fp8 — fh_rmsnorm with an fp8 output: s and y as there, and of every
 * 128 elements of a row, in float32,
 *   out_scale = max |y| / 448;  out_q = y / out_scale rounded to E4M3 (ties to
 *   even, within [-448, 448]; 0 where out_scale is 0)
 * A group that holds an infinity or NaN has an out_scale that says so (infinity
 * or NaN) and codes that mean nothing.
 *   out_q      device [B x d], row stride ld_q >= d.
 *   out_scale  device [B x ceil(d / 128)] float, row stride ld_scale.
 *   out, out_residual  as for fh_rmsnorm, either may be NULL.
 * The other arguments as for fh_rmsnorm.
 */
fh_status fh_rmsnorm_fp8(const void* x, int64_t ld_x, const void* residual, int64_t ld_residual,
                         const void* weight, fh_dtype dtype, int64_t B, int64_t d, float eps,
                         float weight_offset, void* out, int64_t ld_out, void* out_residual,
                         int64_t ld_out_residual, uint8_t* out_q, int64_t ld_q, float* out_scale,
                         int64_t ld_scale, void* stream);

/* fh_fp8_quant — the same codes and scales of x [B x d] as it is (y = x). */
fh_status fh_fp8_quant(const void* x, int64_t ld_x, fh_dtype dtype, int64_t B, int64_t d,
                       uint8_t* out_q, int64_t ld_q, float* out_scale, int64_t ld_scale,
                       void* stream);

/* An fp8 weight matrix [n x k] with a float scale per block of 128 x 128. */
typedef struct fh_fp8 fh_fp8; /* opaque */

/*
 * fh_fp8_create — quantise W, device [n x k] of dtype, dense: per block
 * scale = max |W| / 448, codes as fh_fp8_quant's.  A block that holds an infinity
 * or NaN gives FH_EINVAL.
 * fh_fp8_create_codes — take codes [n x k] and scales [ceil(n / 128) x
 * ceil(k / 128)] float as they are, both device and dense.
 * Both copy into the handle's own layout (n k bytes, n rounded up to 16 and k to
 * 128, plus the scales), wait for `stream`, and keep nothing of their arguments.
 * 1 <= n <= 2^27, 1 <= k < 131072.  Not while `stream` is being captured.
 */
fh_status fh_fp8_create(const void* W, fh_dtype dtype, int64_t n, int64_t k, void* stream,
                        fh_fp8** out);
fh_status fh_fp8_create_codes(const uint8_t* codes, const float* scales, int64_t n, int64_t k,
                              void* stream, fh_fp8** out);

/* fh_fp8_destroy — as fh_w8a8_destroy. */
void fh_fp8_destroy(fh_fp8* w);

/* fh_fp8_get — copy the codes [n x k] and scales out (device). */
fh_status fh_fp8_get(const fh_fp8* w, uint8_t* codes, float* scales, void* stream);

/* fh_fp8_workspace — as fh_w8a8_workspace. */
int64_t fh_fp8_workspace(const fh_fp8* w, const uint8_t* q, int64_t ld_q, int64_t B, int forward);

/*
 * fh_fp8_matmul — out[b, j] = sum over groups g of 128 of k of
 *   (sum_{i in g} q[b, i] code[j, i]) (q_scale[b, g] scale[j / 128, g]),
 * the products exact, the sums and the scales' product in float32, rounded to
 * bf16 at the end for out_dtype FH_BF16.  How the sum over g is cut up depends on
 * n, k and B, never on the values: equal calls give equal bits.
 *   q        device [B x k] E4M3 codes, row stride ld_q >= k.
 *   q_scale  device [B x ceil(k / 128)] float, row stride ld_scale.
 *   out, workspace, B   as for fh_w8a8_matmul (fh_fp8_workspace).
 */
fh_status fh_fp8_matmul(const fh_fp8* w, const uint8_t* q, int64_t ld_q, const float* q_scale,
                        int64_t ld_scale, int64_t B, void* out, int64_t ld_out,
                        fh_dtype out_dtype, void* workspace, int64_t workspace_bytes,
                        void* stream);

/*
 * fh_fp8_matmul_native — fh_fp8_matmul with bfloat16 results, by the matrix cores'
 * own fp8 product where n, k and B make it pay (4096 x 10240 x 2560: 103 us for 190;
 * small calls are fh_fp8_matmul's).  It adds up each eight neighbouring products (k
 * 8 i .. 8 i + 7) in fewer bits than float32: of the others it drops what lies below
 * 2^-13 of the largest one's power of two, where a code below 2^-6 but 0 counts as
 * 2^-6.  So a result may be off by 2^-10 of the sum of its products' magnitudes, such
 * codes counted so, besides its rounding: 1.5e-5 of the results of normally
 * distributed codes (2-norm), 5e-5 of codes of all sizes, but all of a result whose
 * products cancel.  A token's results may differ by as much with the batch that it
 * is in.
 */
fh_status fh_fp8_matmul_native(const fh_fp8* w, const uint8_t* q, int64_t ld_q, const float* q_scale,
                               int64_t ld_scale, int64_t B, void* out, int64_t ld_out,
                               void* workspace, int64_t workspace_bytes, void* stream);

/* fh_fp8_forward — the dense head on fh_fp8_matmul's product; fh_w8a8_forward's
 * arguments and choice. */
fh_status fh_fp8_forward(const fh_fp8* w, const uint8_t* q, int64_t ld_q, const float* q_scale,
                         int64_t ld_scale, int64_t B, int mode, float temperature, uint64_t seed,
                         int32_t* out_token, float* out_token_logit, float* out_lse,
                         float* out_logits, int64_t ld_logits, void* workspace,
                         int64_t workspace_bytes, void* stream);

/*
 * Decoding by beams: `sequences` of `beams` rows each, row s * beams + w being
 * beam w of sequence s.  As above these calls run on the current device, keep no
 * state, and use the caller's workspace.
 */

/* fh_beam_workspace — bytes of workspace of a fh_beam_select call, or FH_EINVAL. */
int64_t fh_beam_workspace(int64_t sequences, int64_t beams, int64_t n);

/*
 * fh_beam_select — of each sequence the `keep` continuations with the largest
 * total t = score + (z - lse), best first, in float64 and rounded to float32 at
 * the end; ties go to the smaller beam, then to the earlier place of its row.
 * An lse that is given is taken as it is.  One that the call computes sums float32
 * exponentials in float32, 1024 at a time, and those sums in float64: it is within
 * (42 + 8 ln n) 2^-24 of itself (8e-6 of 128256 logits; some 1e-7 in earnest),
 * by the same amount for all of a beam's continuations.  So their order within a
 * beam is that of their logits, and between beams whose totals are nearer to each
 * other than that it may go either way, the same in equal calls.
 *   logits   device [sequences beams x n] float, row stride ld_logits: after the
 *            rules, of all tokens (ids NULL, n = v) or of the tokens in ids.
 *            -inf and NaN are no continuation.
 *   ids      device, the same shape, int32, row stride ld_ids, or NULL.  An id
 *            outside [0, v) is no continuation; an id listed twice is two.
 *   lse      device [sequences beams] float: the log-sum-exp to take (a head's
 *            out_lse at T = 1, which knows more tokens than ids lists); NULL: that of
 *            the row's logits, as above (a row that holds NaN or +inf then has none, and
 *            no continuation).
 *   scores   device [sequences x beams] float: the beams' totals so far.  A beam
 *            of -inf or NaN has no continuation (a first step gives all but
 *            beam 0 -inf).
 *   finished device [sequences x beams] int32 or NULL: a beam where it is not 0
 *            has one continuation, eos with its score as it is, whatever its
 *            logits.
 *   eos      the token that finishes a beam, or -1 (finished is NULL then).
 *   out_score, out_token, out_parent  device [sequences x keep], dense: the total,
 *            the token and the beam that it continues; -inf, -1 and -1 where a
 *            sequence has fewer continuations.
 *   out_finished  the same, int32 or NULL: 1 where the token is eos.
 * out_score may be scores itself and out_finished finished itself where
 * keep = beams; no other overlap.
 * 1 <= beams, keep <= 64, sequences beams <= 65535, 1 <= n, v <= 2^30.
 */
fh_status fh_beam_select(const float* logits, int64_t ld_logits, const int32_t* ids, int64_t ld_ids,
                         int64_t sequences, int64_t beams, int64_t n, int64_t v, const float* lse,
                         const float* scores, const int32_t* finished, int32_t eos, int64_t keep,
                         float* out_score, int32_t* out_token, int32_t* out_parent,
                         int32_t* out_finished, void* workspace, int64_t workspace_bytes,
                         void* stream);

/*
 * How a state holds what belongs to the rows, in bytes: `outer` blocks (layers)
 * of rows of `mid` parts (heads) of `positions` of `run` contiguous bytes, each
 * level with its stride; a level of one has any.  No byte belongs to two places.
 */
typedef struct {
  int64_t outer, mid, positions, run;
  int64_t ld_outer, ld_row, ld_mid, ld_position;
} fh_beam_layout;

/*
 * fh_beam_reorder — states[i][s, w] = states[i][s, parent[s, w]] for all w at
 * once, in place; only rows that continue another are written.
 *   states   host array of `count` device pointers to states of one layout, which
 *            do not overlap; it is read before the call returns.
 *   parent   device [sequences x beams] int32; outside [0, beams) leaves the row
 *            as it is.
 *   lengths  device [sequences x beams] int32 or NULL (all): positions of each
 *            row that count, clamped to [0, positions].  A row takes its parent's;
 *            what lies behind them is left as it is.
 * parent and lengths must not lie among a state's bytes, from its first to its last,
 * not in part either, and no state is listed twice.  Any
 * alignment.  Positions that do not follow each other directly, and their runs,
 * are fewer than 2^31.
 */
fh_status fh_beam_reorder(void* const* states, int64_t count, const fh_beam_layout* layout,
                          int64_t sequences, int64_t beams, const int32_t* parent,
                          const int32_t* lengths, void* stream);

/* fh_beam_reorder_check — what fh_beam_reorder would refuse of these arguments, with
 * nothing moved: for states of several layouts, all of which are checked before the
 * first is reordered. */
fh_status fh_beam_reorder_check(void* const* states, int64_t count, const fh_beam_layout* layout,
                                int64_t sequences, int64_t beams, const int32_t* parent,
                                const int32_t* lengths);

/* Thread-local description of the last error on this thread ("" if none). */
const char* fh_last_error(void);

/* Library version string. */
const char* fh_version(void);

#ifdef __cplusplus
}
#endif

#endif /* FLASHHEAD_H */

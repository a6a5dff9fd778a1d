/*
 * semicrf.h — C ABI of the MI355X (gfx950) streaming semi-Markov CRF library.
 *
 * Method: "Streaming Structured Inference with Flash-SemiCRF" (pages: thelatestinai
 * abstract card; gist.science explainers in English, Dutch and Chinese).  A semi-CRF
 * labels whole segments [s, s+k), 1 <= k <= K, with one of C labels.  The potential
 * of a segment of label c that follows a segment of label c' is
 *
 *     S[s+k, c] - S[s, c] + dur[k-1, c] + trans[c', c]
 *
 * where S is the prefix sum of the emissions after subtracting their per-sequence,
 * per-label mean (EN explainer, "2. Methodology": "On-the-Fly Edge Computation via
 * Prefix Sums" and "Emission Baseline Centering").  The first segment of a sequence
 * pays no transition score and nothing is paid after the last one.  The library
 * evaluates every potential on the fly from S; the T*K*C^2 edge tensor is never
 * stored (EN explainer, "1. Problem Statement").
 *
 * Conventions shared by every entry point
 *  - All array arguments are DEVICE pointers to dense row-major arrays with the
 *    label index innermost:
 *        emissions [B, T, C] float32     lengths [B] int32 (1 <= lengths[b] <= T)
 *        trans     [C, C]    float32     (row = previous label, column = next label)
 *        dur       [K, C]    float32     (row k-1 scores a segment of length k)
 *    Emissions at t >= lengths[b] are ignored.  -inf in trans or dur forbids the
 *    transition / duration.
 *  - Ownership: the caller allocates and frees every input, output and the
 *    workspace.  The library allocates no device memory and keeps no pointer or
 *    other state after a call returns.  Calls on different streams with distinct
 *    workspaces may run concurrently.
 *  - Execution: all work is enqueued on `stream`; no call synchronises the host.  The
 *    arrays and `stream` belong to the current device (NULL is its default stream).
 *    Outputs are valid once the stream reaches that point.  Results are bitwise
 *    reproducible for the same inputs, shapes and checkpoint interval (fixed-order
 *    reductions, no floating-point atomics).
 *  - Errors: every call returns a semicrf_status and never aborts.  Host-side
 *    checks: B, T, C, K >= 1, required pointers non-NULL, workspace large enough,
 *    shape supported (SEMICRF_ERR_UNSUPPORTED: C > 128; K above 8193 when C <= 7,
 *    2049 when C <= 16, 513 when C <= 64, and for 64 < C <= 128 whatever the 160 KB
 *    of LDS of a compute unit holds: 129 down to 97 at C = 128; semicrf_workspace_bytes
 *    returns 0 for such shapes).  A failed
 *    kernel launch returns SEMICRF_ERR_DEVICE.  A length outside [1, T] is only
 *    visible on the device: that sequence is processed as if clamped to [1, T],
 *    its log Z / Viterbi score is set to NaN, and a flag is raised in the
 *    workspace that semicrf_read_status() returns.
 *  - Workspace: at least semicrf_workspace_bytes(op, ...) bytes of device memory,
 *    256-byte aligned, passed to the call of that op.  Its contents on entry do not
 *    matter and are overwritten.
 */
#ifndef SEMICRF_H
#define SEMICRF_H

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    SEMICRF_OK = 0,
    SEMICRF_ERR_INVALID = 1,      /* bad scalar argument or NULL pointer, or a device-flagged length */
    SEMICRF_ERR_WORKSPACE = 2,    /* workspace NULL, too small or misaligned */
    SEMICRF_ERR_UNSUPPORTED = 3,  /* shape outside the supported range */
    SEMICRF_ERR_DEVICE = 4,       /* a HIP launch or copy failed */
    SEMICRF_ERR_UNIMPLEMENTED = 5 /* reserved: no entry point of this library returns it */
} semicrf_status;

typedef enum {
    SEMICRF_OP_LOGZ = 0,
    SEMICRF_OP_BACKWARD = 1,
    SEMICRF_OP_VITERBI = 2,
    SEMICRF_OP_PREFIX = 3
} semicrf_op;

/* Human-readable name of a status code (static string, never NULL). */
const char* semicrf_status_string(int status);

/* Checkpoint interval for a padded length T and maximum duration K: delta if delta > 0,
 * else ceil(sqrt(T*K)) (EN explainer, "2. Methodology", "Checkpointing": an interval of
 * about sqrt(TK)); clamped to [1, T].  0 on bad input. */
int semicrf_checkpoint_interval(int T, int K, int delta);


/* The checkpoint interval `op` uses for delta = 0 (semicrf_viterbi takes none and always
 * uses it).  Every span is swept at once, so where the round kernels run (C <= 16,
 * K <= 1025) and for log Z and the backward everywhere, the interval is the one, over
 * every span count n (interval ceil(T/n)), that minimises
 * (interval + burn-in 3K) * ceil(workgroups / share): workgroups = B * spans for log Z, the
 * decode and a backward whose two directions share a workgroup (small label counts), else
 * twice that; share = 224 workgroups (7/8 of the MI355X's 256 compute units, leaving room
 * for a concurrent call) where the round kernels run, else 256.  Intervals shorter than
 * the burn-in are not taken (unless T is); ties go to the longer interval.  The decode
 * outside the round kernels takes ceil(sqrt(T*K)), halved when the batch holds at most
 * 128 spans of that length and each is at least four burn-ins (12 K) long.  0 on bad or
 * unsupported input. */
int semicrf_default_interval(semicrf_op op, int B, int T, int C, int K);

/* Bytes of workspace that `op` needs for these shapes (delta as the call takes it: > 0 an
 * explicit interval, 0 the default above).  0 if the arguments are invalid or
 * unsupported. */
size_t semicrf_workspace_bytes(semicrf_op op, int B, int T, int C, int K, int delta);

/* Centred prefix sums alone (EN explainer, "2. Methodology": "Emission Baseline
 * Centering" then "On-the-Fly Edge Computation via Prefix Sums"):
 *   S[b, 0, c] = 0,  S[b, t, c] = sum_{u < t} (em[b, u, c] - nu[b, c])  for t <= L_b,
 * nu[b, c] = mean of em[b, :L_b, c]; S[b, t, c] = S[b, L_b, c] for t > L_b.
 * Output: S [B, T+1, C] float64 (device).  Workspace: semicrf_workspace_bytes(
 * SEMICRF_OP_PREFIX, ...).  The other calls compute the same S internally. */
int semicrf_prefix(const float* emissions, const int32_t* lengths, int B, int T, int C,
                   hipStream_t stream, void* workspace, size_t workspace_bytes, double* S);

/* ------------------------------------------------------------------ the three calls
 * Each takes (emissions, lengths, trans, dur, sizes, stream) as the problem statement
 * gives them, plus a caller-owned workspace and the outputs. */

/* log Z for every sequence: the log-sum-exp of the scores of all segmentations
 * (EN explainer, "2. Methodology", "Streaming Forward-Backward with Ring Buffers",
 * forward pass).  delta: checkpoint interval (0 = semicrf_default_interval(SEMICRF_OP_LOGZ,
 * B, T, C, K)), the
 * same value as given to semicrf_workspace_bytes.  Output: log_z [B] float32. */
int semicrf_logz(const float* emissions, const int32_t* lengths, const float* trans,
                 const float* dur, int B, int T, int C, int K, int delta, hipStream_t stream,
                 void* workspace, size_t workspace_bytes, float* log_z);

/* Exact gradients of sum_b grad_log_z[b] * log Z_b (EN explainer, "2. Methodology",
 * backward pass with recomputation from checkpoints every `delta` positions;
 * "4. Results and Benchmarks": exact gradients).  Inputs as above plus
 *   grad_log_z [B] float32, or NULL for all ones.
 * Outputs (all overwritten; padding positions t >= lengths[b] are set to 0):
 *   grad_emissions [B, T, C] float32  d/d emissions, including the centring mean
 *   grad_trans     [C, C]    float32  summed over the batch
 *   grad_dur       [K, C]    float32  summed over the batch
 *   marginals      [B, T, C] float32  or NULL: posterior probability that position t
 *                                     lies in a segment of label c (sums to 1 over c)
 *   log_z          [B]       float32  or NULL
 * delta: checkpoint interval (0 = semicrf_default_interval(SEMICRF_OP_BACKWARD, B, T, C,
 * K)); results do not
 * depend on it beyond rounding. */
int semicrf_backward(const float* emissions, const int32_t* lengths, const float* trans,
                     const float* dur, int B, int T, int C, int K, int delta,
                     hipStream_t stream, void* workspace, size_t workspace_bytes,
                     const float* grad_log_z, float* grad_emissions, float* grad_trans,
                     float* grad_dur, float* marginals, float* log_z);

/* Max-plus decode of the best segmentation (the Viterbi counterpart of the forward
 * pass).  Every max-plus step keeps the shortest segment, then the lowest previous
 * label, among equal candidates, and the decode ends at the lowest best final label.
 * When several segmentations share the best score (to fp32 rounding), the one returned
 * may differ from the one these rules give in exact arithmetic; a decision that beats
 * every alternative by more than rounding is always taken as in exact arithmetic.
 * Outputs:
 *   best_score [B]    float32  score of the best segmentation
 *   labels     [B, T] int32    label of every position, -1 at t >= lengths[b]
 *   seg_start  [B, T] uint8    1 where a segment starts, else 0 */
int semicrf_viterbi(const float* emissions, const int32_t* lengths, const float* trans,
                    const float* dur, int B, int T, int C, int K, hipStream_t stream,
                    void* workspace, size_t workspace_bytes, float* best_score,
                    int32_t* labels, uint8_t* seg_start);

/* ------------------------------------------------------------------ extended calls
 * The same three calls (and the training loss) with optional extras.  A NULL options
 * pointer, or a zero-initialised struct, gives exactly the plain call. */
typedef struct semicrf_options {
    /* Boundary projections (EN explainer, "2. Methodology", "Boundary Projections": start
     * and end features computed apart and added to the edge potential), inputs of every
     * call:
     *   proj_start [B, T, C] or NULL: score of a segment of label c that starts at t
     *   proj_end   [B, T, C] or NULL: score of a segment of label c whose last position is t
     * so a segment [s, e) of label c gains proj_start[b, s, c] + proj_end[b, e-1, c].  NULL
     * means zeros; values at t >= lengths[b] are ignored; the values must be finite (a
     * large negative value, e.g. -1e4, effectively forbids a start or end); not centred. */
    const float* proj_start;
    const float* proj_end;
    /* Backward and training-loss outputs, each optional (NULL):
     *   grad_proj_start [B, T, C]  g_b times the probability that a segment of label c
     *                              starts at t (d/d proj_start)
     *   grad_proj_end   [B, T, C]  g_b times the probability that a segment of label c has
     *                              its last position at t (d/d proj_end) */
    float* grad_proj_start;
    float* grad_proj_end;
    /* Backward outputs, each optional (NULL):
     *   boundary  [B, T]  probability that a segment starts at t (1 at t = 0; EN explainer,
     *                     "4. Results and Benchmarks": boundary probabilities)
     *   node_mass [B, T]  the sum over labels of the node marginals as the forward and
     *                     backward values give them, before the marginals are divided by
     *                     it: 1 in exact arithmetic, so |node_mass - 1| measures the
     *                     rounding of the streamed recurrences (0 at padding) */
    float* boundary;
    float* node_mass;
    /* Stage timing: NULL, or events created by the caller (hipEventCreate), one more than
     * the call's stage count; events[i] is recorded on `stream` when stage i begins and
     * the last when the call's work ends.  No synchronisation.
     *   logz:     0 centring + prefix scan, 1 forward sweep
     *   backward: 0 centring + prefix scan, 1 the checkpoint spans of both directions
     *             with their per-position values, 2 seam check and repair, 3 segment
     *             posteriors, 4 node marginals and gradient reductions
     *   viterbi:  0 centring + prefix scan, 1 max-plus checkpoint spans with the seam
     *             check, repair and final label, 2 backtrace */
    hipEvent_t* events;
    /* Checkpoint spans swept at once.  The sweeps are sequential in the position; every
     * span of delta positions is swept at the same time instead, starting 3K positions
     * early (at least 64) from a ring in which every entry is equal.  The values a span
     * then reaches equal the exact ones plus one constant, to within rounding; at each
     * checkpoint the library compares the two spans' ring values over the K positions
     * before it, takes the constant from them and accepts the seam when every entry is
     * within seam_tolerance of it (natural-log units; 0 = the default, 1e-4).  From the
     * first seam that is not accepted the sequence is swept again in order, exactly as a
     * single sweep would.
     *   seam_bound   [B] float32 or NULL: per sequence, the sum over both directions'
     *                accepted seams of the largest deviation from the constant; no value
     *                of the call moves by more than it (beyond rounding) from the values
     *                of sweeps run in order
     *   seam_repairs [B] int32 or NULL: the number of directions (0..2) swept again in
     *                order from a seam that was not accepted
     * A negative seam_tolerance accepts no seam (every sequence is swept in order after
     * its first span: the exact fallback, for testing). */
    float* seam_bound;
    int32_t* seam_repairs;
    double seam_tolerance;
} semicrf_options;

#define SEMICRF_LOGZ_STAGES 2
#define SEMICRF_BACKWARD_STAGES 5
#define SEMICRF_VITERBI_STAGES 3

int semicrf_logz_ex(const float* emissions, const int32_t* lengths, const float* trans,
                    const float* dur, int B, int T, int C, int K, int delta,
                    hipStream_t stream, void* workspace, size_t workspace_bytes, float* log_z,
                    const semicrf_options* options);
int semicrf_backward_ex(const float* emissions, const int32_t* lengths, const float* trans,
                        const float* dur, int B, int T, int C, int K, int delta,
                        hipStream_t stream, void* workspace, size_t workspace_bytes,
                        const float* grad_log_z, float* grad_emissions, float* grad_trans,
                        float* grad_dur, float* marginals, float* log_z,
                        const semicrf_options* options);
int semicrf_viterbi_ex(const float* emissions, const int32_t* lengths, const float* trans,
                       const float* dur, int B, int T, int C, int K, hipStream_t stream,
                       void* workspace, size_t workspace_bytes, float* best_score,
                       int32_t* labels, uint8_t* seg_start, const semicrf_options* options);

/* Training loss of gold segmentations and its gradients.  nll[b] = log Z_b - score_b(y*),
 * the negative log-probability of the gold segmentation y* (the training loss of the
 * pages' convergence check, EN explainer, "4. Results and Benchmarks"); score sums, over
 * the gold segments [s, e) of label c, S[e,c] - S[s,c] + dur[e-s-1, c] (+ the
 * projections) and, between consecutive segments, trans[c', c] (the same centred
 * potential as log Z, "2. Methodology").  Inputs as semicrf_backward plus
 *   gold_labels    [B, T] int32  label of every position t < lengths[b]
 *   gold_seg_start [B, T] uint8  1 at each gold segment's first position (t = 0 must be 1)
 *   grad_nll       [B] float32 or NULL for all ones
 * Outputs: nll [B] float32, and the gradients of sum_b grad_nll[b] * nll[b] in
 * grad_emissions [B, T, C], grad_trans [C, C], grad_dur [K, C] and, through the options,
 * grad_proj_start / grad_proj_end [B, T, C] (expected minus gold feature counts; the
 * emission gradient includes the centring; 0 at padding).  Options: projections and
 * their gradients only (the other fields must be NULL).  A gold segmentation with a
 * segment longer than K, a label outside [0, C), a label change inside a segment or no
 * start at t = 0 gives NaN for that sequence and raises the status flag, like an invalid
 * length; its gold counts are then left out of the gradients, which keep only its log Z
 * half.  Workspace: semicrf_workspace_bytes(SEMICRF_OP_BACKWARD, ...). */
int semicrf_nll(const float* emissions, const int32_t* lengths, const float* trans,
                const float* dur, const int32_t* gold_labels, const uint8_t* gold_seg_start,
                int B, int T, int C, int K, int delta, hipStream_t stream, void* workspace,
                size_t workspace_bytes, const float* grad_nll, float* nll,
                float* grad_emissions, float* grad_trans, float* grad_dur,
                const semicrf_options* options);

/* ------------------------------------------------------------------ no allocation
 * For callers that cannot allocate device memory at all: code under HIP graph capture,
 * tight serving loops, harnesses that forbid hipMalloc.  semicrf_logz without a
 * workspace argument: the workspace is a static device array of
 * SEMICRF_STATIC_SCRATCH_BYTES inside the library, one per GPU, held from the first
 * call on that GPU until the process ends.  The call allocates nothing (no hipMalloc,
 * no allocating library routine).  Shapes whose semicrf_workspace_bytes(
 * SEMICRF_OP_LOGZ, ...) exceeds the array return SEMICRF_ERR_WORKSPACE before any
 * launch.  Every call on one GPU shares that GPU's array, so calls that overlap on one
 * GPU (on different streams, or from different threads) race and must be serialised
 * by the caller.  An invalid length gives NaN in log_z as for semicrf_logz; its status
 * flag is not readable.  The array lives on the device of `stream` (the current
 * device for the NULL stream). */
#define SEMICRF_STATIC_SCRATCH_BYTES ((size_t)32 << 20)
int semicrf_logz_static(const float* emissions, const int32_t* lengths, const float* trans,
                        const float* dur, int B, int T, int C, int K, int delta,
                        hipStream_t stream, float* log_z);

/* Synchronously reads the device status flag left in `workspace` by the last call
 * that used it (after waiting for `stream`).  SEMICRF_OK, SEMICRF_ERR_INVALID if a
 * length was outside [1, T], or SEMICRF_ERR_DEVICE if the copy failed. */
int semicrf_read_status(const void* workspace, hipStream_t stream);

/* ------------------------------------------------------------------ encoder operators
 * What makes the emissions: an embedding of tokens, layer norm, and linear attention with a
 * decay for each head, whose cost is linear in T like the CRF's.  Conventions as above
 * (device pointers, work enqueued on `stream`, no allocation, status codes, fixed-order
 * sums), and:
 *  - dtype is the type of the arrays given as void*: SEMICRF_F32 or SEMICRF_BF16.  Sums,
 *    statistics and states are held in float32; an output is rounded once.
 *  - lengths [B] int32 may be NULL (every length is T), and here a length may be 0.  A
 *    length outside [0, T] is taken as clamped.  What lies at t >= lengths[b] is not read,
 *    whatever it holds, and outputs are 0 there.
 *  - status: NULL, or a device word the caller has cleared; the call sets bit 0 in it when a
 *    length, or a token, was out of range.
 *  - B * T, V and the N of embed are below 2^30, B below 2^16 and Hq below 2^15 for the
 *    attention calls (else SEMICRF_ERR_UNSUPPORTED).  Arrays need the alignment of their elements only. */
typedef enum { SEMICRF_F32 = 0, SEMICRF_BF16 = 1 } semicrf_dtype;

/* out[b, t, :] = scale * table[tokens[b, t], :].  tokens [B, T] int32 or int64 (token_bits 32
 * or 64), table [V, N], out [B, T, N].  A token outside [0, V) gives a row of NaN. */
int semicrf_embed(const void* tokens, int token_bits, const int32_t* lengths, const void* table,
                  int dtype, int B, int T, int V, int N, float scale, hipStream_t stream,
                  void* out, int32_t* status);

/* grad_table[v, :] = scale * sum of grad_out[b, t, :] over the positions with token v (0 for a
 * token that does not appear; a token outside [0, V) counts for nothing).  Positions are
 * sorted by token and each row's sum has a fixed order.  N <= 2^23.  Workspace:
 * semicrf_embed_grad_bytes, 256-byte aligned. */
size_t semicrf_embed_grad_bytes(int dtype, int B, int T, int V, int N);
int semicrf_embed_grad(const void* tokens, int token_bits, const int32_t* lengths,
                       const void* grad_out, int dtype, int B, int T, int V, int N, float scale,
                       hipStream_t stream, void* workspace, size_t workspace_bytes,
                       void* grad_table, int32_t* status);

/* Layer norm of each row of x [B, T, N]: y = (x - mean) * rstd * weight + bias with rstd =
 * 1 / sqrt(variance + eps).  weight, bias [N] of type wdtype (dtype or SEMICRF_F32), or NULL
 * for ones and zeros.  mean, rstd [B, T] float32 (0 at padding), or NULL.  N <= 32768. */
int semicrf_layer_norm(const void* x, int dtype, const void* weight, const void* bias, int wdtype,
                       const int32_t* lengths, int B, int T, int N, float eps, hipStream_t stream,
                       void* y, float* mean, float* rstd, int32_t* status);

/* Its gradients from the mean and rstd the forward call left: grad_x [B, T, N] and, summed over
 * all rows, grad_weight and grad_bias [N] of type wdtype (each may be NULL).  Workspace:
 * semicrf_layer_norm_grad_bytes, 256-byte aligned. */
size_t semicrf_layer_norm_grad_bytes(int dtype, int B, int T, int N);
int semicrf_layer_norm_grad(const void* grad_out, const void* x, int dtype, const void* weight,
                            int wdtype, const float* mean, const float* rstd,
                            const int32_t* lengths, int B, int T, int N, hipStream_t stream,
                            void* workspace, size_t workspace_bytes, void* grad_x,
                            void* grad_weight, void* grad_bias, int32_t* status);

/* Linear attention with a decay for each head:
 *   S_t = gamma_h S_{t-1} + k_t v_t^T,   o_t = scale * q_t^T S_t,   gamma_h = exp(log_decay[h]),
 * S [Dk, Dv] for every sequence and query head, starting from `state` or 0.  Query head h reads
 * key / value head h / (Hq / Hk).  log_decay [Hq] is meant to be <= 0 (-inf forgets everything
 * but the position itself).  A value that is not finite, at a position before the length, may
 * spoil the outputs of up to 63 positions before it, and all after it. */
typedef struct semicrf_attention {
    const void* q;               /* [B, T, Hq, Dk] */
    const void* k;               /* [B, T, Hk, Dk] */
    const void* v;               /* [B, T, Hk, Dv] */
    int64_t q_stride[3];         /* elements between sequences, positions, heads; the last */
    int64_t k_stride[3];         /* axis is dense */
    int64_t v_stride[3];
    const int32_t* lengths;      /* [B] or NULL */
    const float* log_decay;      /* [Hq] */
    const float* state;          /* [B, Hq, Dk, Dv] before the first position, or NULL for 0 */
    float scale;
    int dtype;                   /* of q, k, v and the outputs shaped like them */
    int B, T, Hq, Hk, Dk, Dv;    /* Hq a multiple of Hk; Dk, Dv <= 128 */
} semicrf_attention;

/* Whole sequences.  out [B, T, Hq, Dv] dense; state_out [B, Hq, Dk, Dv] float32 after position
 * lengths[b] - 1, or NULL (it may be the array `state` points to).  Workspace:
 * semicrf_decay_attention_bytes(attention, 0), 256-byte aligned. */
size_t semicrf_decay_attention_bytes(const semicrf_attention* attention, int grad);
int semicrf_decay_attention(const semicrf_attention* attention, hipStream_t stream,
                            void* workspace, size_t workspace_bytes, void* out,
                            float* state_out, int32_t* status);

/* Gradients: of out (grad_out [B, T, Hq, Dv], dense) and of state_out (grad_state_out [B, Hq,
 * Dk, Dv] float32, or NULL for 0).  grad_q [B, T, Hq, Dk], grad_k [B, T, Hk, Dk], grad_v [B, T,
 * Hk, Dv], dense, shared heads summed; grad_state [B, Hq, Dk, Dv] float32 or NULL.  The decay
 * is a constant of the head: it has no gradient.  Workspace:
 * semicrf_decay_attention_bytes(attention, 1). */
int semicrf_decay_attention_grad(const semicrf_attention* attention, const void* grad_out,
                                 const float* grad_state_out, hipStream_t stream, void* workspace,
                                 size_t workspace_bytes, void* grad_q, void* grad_k, void* grad_v,
                                 float* grad_state, int32_t* status);

/* One token of B streams (attention->T is 1, lengths NULL): the recurrence once, on states
 * kept in a pool.  attention->state and state_out are [pool, Hq, Dk, Dv] float32 and may be the
 * same array; stream b uses row slots[b] (b itself where slots is NULL, then pool >= B).  A
 * slot outside [0, pool) marks an idle row: its output is 0 and no state is touched.  The
 * slots in [0, pool) must be distinct.  Rows of state_out that no slot names are left alone.
 * out [B, Hq, Dv].  Each token rounds the float32 state once, so a decay weaker than 2^-24 a token
 * may be lost in the rounding. */
int semicrf_decay_attention_step(const semicrf_attention* attention, const int32_t* slots,
                                 int pool, hipStream_t stream, void* out, float* state_out);

/* ------------------------------------------------------------------ blocks and pretraining
 * What an encoder block needs beside attention, and what it is trained on before there are
 * segments.  Conventions as for the encoder operators.  A workspace serves one call at a time: calls,
 * and replays of captured calls, that may overlap need one each. */

/* Gated linear recurrence, a decay of its own for each position and channel:
 *   s_t = log_decay[n] sig(r_t),  a_t = exp(s_t),  h_t = a_t h_{t-1} + sqrt(1 - a_t^2) sig(i_t) x_t,
 * sig(z) = 1 / (1 + exp(-z)), r the decay gate and i the input gate before their sigmoid, h_0 = `state`
 * or 0.  log_decay [N] is meant to be finite and <= 0: above 0, 1 - a^2 is negative and outputs are NaN.
 * A value that is not finite spoils its channel from its position on, and no other. */
typedef struct semicrf_recurrence {
    const void* x;               /* [B, T, N], as decay_gate and input_gate */
    const void* decay_gate;
    const void* input_gate;
    int64_t x_stride[2];         /* elements between sequences and positions (the second from 0 */
    int64_t decay_stride[2];     /* to 2^25 - 1 where T > 1); the last axis is dense */
    int64_t input_stride[2];
    const int32_t* lengths;      /* [B] or NULL */
    const float* log_decay;      /* [N] */
    const float* state;          /* [B, N] before the first position, or NULL for 0 */
    int dtype;                   /* of x, the gates and the outputs shaped like them */
    int B, T, N;                 /* B < 2^16, N <= 2^20, B * (N / 64, rounded up) < 2^22 */
} semicrf_recurrence;

/* Whole sequences.  out [B, T, N] dense, 0 at padding; state_out [B, N] float32 after position
 * lengths[b] - 1 (the state before the first where that is 0), or NULL; it may be the array `state`
 * points to.  starts [B, ceil(T / SEMICRF_RECURRENCE_SPAN), N] float32, or NULL: the state before
 * each span of positions, for the gradient (spans past the length are left as they are).
 * Workspace: semicrf_gated_recurrence_bytes(recurrence, 0), 256-byte aligned. */
#define SEMICRF_RECURRENCE_SPAN 16
size_t semicrf_gated_recurrence_bytes(const semicrf_recurrence* recurrence, int grad);
int semicrf_gated_recurrence(const semicrf_recurrence* recurrence, hipStream_t stream,
                             void* workspace, size_t workspace_bytes, void* out, float* state_out,
                             float* starts, int32_t* status);

/* Gradients, of out (grad_out [B, T, N] dense) and of state_out (grad_state_out [B, N] float32, or
 * NULL for 0), from the `starts` the forward call left.  grad_x, grad_decay_gate, grad_input_gate
 * [B, T, N] dense, 0 at padding; grad_log_decay [N] float32, summed over all positions in a fixed
 * order; grad_state [B, N] float32; the last two may be NULL.  A decay gate so far closed that 1 - a^2
 * is below 2^-123 counts sqrt(1 - a^2) as a constant.  Workspace:
 * semicrf_gated_recurrence_bytes(recurrence, 1). */
int semicrf_gated_recurrence_grad(const semicrf_recurrence* recurrence, const float* starts,
                                  const void* grad_out, const float* grad_state_out,
                                  hipStream_t stream, void* workspace, size_t workspace_bytes,
                                  void* grad_x, void* grad_decay_gate, void* grad_input_gate,
                                  float* grad_log_decay, float* grad_state, int32_t* status);

/* One token of B streams (recurrence->T is 1, lengths NULL, inputs [B, N]: the strides between
 * positions are not looked at), on states kept in a pool: recurrence->state and state_out are [pool,
 * N] float32 and may be the same array.  slots as in semicrf_decay_attention_step.  out [B, N]. */
int semicrf_gated_recurrence_step(const semicrf_recurrence* recurrence, const int32_t* slots,
                                  int pool, hipStream_t stream, void* out, float* state_out);

/* The end of one block and the start of the next, on the residual stream x:
 *   r = x + scale sig(gate) f(branch),   y = norm(r) weight + bias,
 * f(o) = o, or norm(o) branch_weight + branch_bias where norm_branch is set.  norm(z) = (z - mean) rstd
 * over the last axis with rstd = 1 / sqrt(mean (z - mean)^2 + eps); center = 0 takes mean as 0 (the
 * root-mean-square norm), in both norms.  A NULL gate or scale is a factor of 1, a NULL weight ones,
 * a NULL bias zeros. */
typedef struct semicrf_residual {
    const void* x;               /* [B, T, N] dense */
    const void* branch;          /* [B, T, N] */
    const void* gate;            /* [B, T, N] before its sigmoid, or NULL */
    int64_t branch_stride[2];    /* elements between sequences and positions; the last axis */
    int64_t gate_stride[2];      /* is dense */
    const void* scale;           /* [N] of type wdtype, as the four below; each may be NULL */
    const void* weight;
    const void* bias;
    const void* branch_weight;   /* looked at where norm_branch is set */
    const void* branch_bias;
    const int32_t* lengths;      /* [B] or NULL */
    float eps;
    int dtype, wdtype;           /* wdtype: dtype or SEMICRF_F32 */
    int norm_branch, center;
    int B, T, N;                 /* N <= 16384 */
} semicrf_residual;

/* r, y [B, T, N] dense, 0 at padding; y is the norm of r before its rounding.  stats [B, T, 4]
 * float32 (mean and rstd of r, mean and rstd of the branch; 0 where there is none), or NULL.  Outputs
 * may not overlap inputs. */
int semicrf_residual_norm(const semicrf_residual* residual, hipStream_t stream, void* r, void* y,
                          float* stats, int32_t* status);

/* Gradients of r and y (grad_r, grad_y [B, T, N] dense; NULL for 0) from the stats of the forward
 * call.  grad_x, grad_branch and, where there is a gate, grad_gate [B, T, N] dense; grad_params
 * [5][N] of type wdtype, or NULL: the gradients of weight, bias, scale, branch_weight and
 * branch_bias, summed over all rows in a fixed order (of those that are not there, as if they were).
 * Workspace: semicrf_residual_norm_grad_bytes, 256-byte aligned. */
size_t semicrf_residual_norm_grad_bytes(int dtype, int B, int T, int N);
int semicrf_residual_norm_grad(const semicrf_residual* residual, const float* stats,
                               const void* grad_r, const void* grad_y, hipStream_t stream,
                               void* workspace, size_t workspace_bytes, void* grad_x,
                               void* grad_branch, void* grad_gate, void* grad_params,
                               int32_t* status);

/* Negative log-likelihood of tokens over a vocabulary: with z_v = scale x[b, t] . table[v],
 *   loss[b, t] = log sum_v exp(z_v) - z_target,
 * x [B, T, N], table [V, N] (it may be the one semicrf_embed reads), targets [B, T] int32 or int64
 * (target_bits 32 or 64), loss [B, T] float32.  A negative target marks a position with nothing to
 * predict: its x is not read and its loss is 0.  A target of V or more gives NaN and the status bit.
 * lse [B, T] float32, or NULL: the log sum, for the gradient (0 where there is nothing to predict).
 * The scores are formed in pieces and never kept.  B * T and V up to 2^22, N <= 32768, (B * T + V + 2^17)
 * * N below 2^36.  Workspace: semicrf_token_nll_bytes(..., 0), 256-byte aligned, is enough for any table;
 * semicrf_token_nll_table_bytes is what a call with this table needs, which leaves out a copy of it where N
 * is a multiple of 64 and the table 16-byte aligned (but in the float32 gradient).  Both are for B * T
 * listed positions, whose number is known on the GPU only. */
size_t semicrf_token_nll_bytes(int dtype, int B, int T, int V, int N, int grad);
size_t semicrf_token_nll_table_bytes(int dtype, int B, int T, int V, int N, const void* table, int grad);
int semicrf_token_nll(const void* x, const void* table, int dtype, const void* targets,
                      int target_bits, const int32_t* lengths, int B, int T, int V, int N,
                      float scale, hipStream_t stream, void* workspace, size_t workspace_bytes,
                      float* loss, float* lse, int32_t* status);

/* Its gradients from those of loss (grad_loss [B, T] float32) and the lse of the forward call:
 * grad_x [B, T, N] (0 where there is nothing to predict) and grad_table [V, N], both of type dtype; either
 * may be NULL.  A target of V or more counts for nothing.  In bfloat16 the numbers that are multiplied are held
 * in fp16, scaled to the top of its range, and summed in float32: softmax less target (11 bits down to 2^-29, 0
 * below 2^-40, so that a word that is nowhere likelier has no gradient), the table (as it is down to 2^-28 of its
 * largest value) and x times the row's grad_loss (11 bits down to 2^-28 of the largest |x| times the largest
 * |grad_loss|, 0 from 2^-39 on; for grad_table only).  Workspace: semicrf_token_nll_bytes(..., 1), or
 * _table_bytes: two copies of x, one of the table, and softmaxes less targets for a piece of the vocabulary at a
 * time, of up to 2 GB or, where that is more, 256 words (4 GB for 2^22 positions in float32); with several
 * pieces also a float32 array shaped like x. */
int semicrf_token_nll_grad(const float* grad_loss, const void* x, const void* table, int dtype,
                           const void* targets, int target_bits, const int32_t* lengths,
                           const float* lse, int B, int T, int V, int N, float scale,
                           hipStream_t stream, void* workspace, size_t workspace_bytes,
                           void* grad_x, void* grad_table, int32_t* status);

#ifdef __cplusplus
}
#endif

#endif /* SEMICRF_H */

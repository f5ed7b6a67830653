/*
 * kda.h -- C ABI of the GB300 (sm_103a) KDA decode / speculative-verify step,
 * its record replay (kda_recover), the output-projection consumer epilogue
 * that follows the attention layer (kda_oproj), linear attention with one
 * decay per head (kda_lin_prompt, kda_lin_step), snapshots of state pages
 * in 8 or 4 bits (kda_snapshot_save, kda_snapshot_load), and the operators of a
 * selective-state-space layer: its short convolution (kda_conv_prompt,
 * kda_conv_step), its scan (kda_ssm_prompt, kda_ssm_step) and its projections
 * (kda_linear).
 *
 * The operation is the one defined by the vLLM API page
 *   "vllm.models.kimi_k3.nvidia.specialized_decode.cutedsl.kda.wide"
 * (class KdaWide: the constructor's validation, `kernel`, and the helpers
 * `silu`, `decay`, `quad_sum`).  For every (request r, head h) item one call:
 *
 *   1. resolves the item's slots (decode: slot = conv slot = slots[r], window
 *      offset 0; verify: slot = slots[r, accepted[r]-1], conv slot =
 *      slots[r, 0], window offset accepted[r]-1); slot <= 0 marks padding:
 *      the item's output rows are BF16 zeros and nothing else is written;
 *   2. runs the 4-tap causal depthwise convolution over the three cached taps
 *      and the new inputs (plus optional bias), SiLU, BF16 rounding (q, k, v);
 *   3. computes the low-rank gate raw_g = BF16(f_b[h] . f_a[row]) and the decay
 *      exp(lower_bound * sigmoid(exp(A_log[h]) * (raw_g + dt_bias)));
 *   4. beta = sigmoid(beta_raw); L2-normalises q (times scale) and k;
 *   5. applies the per-key-decayed delta rule to the 128x128 FP32 state page
 *      [value row i][key j]:  S *= d (per key);  u = (v - S k) * beta;
 *      S += u k^T;  o = BF16(S q);  and writes the page after every token to
 *      slot (decode) or slots[r, t] when > 0 (verify), or, in record mode,
 *      writes the records instead of any state;
 *   6. writes the new conv window [tap1, tap2, x_0 .. x_{T-1}];
 *   7. out = BF16(((o * rsqrt(mean(o^2) + eps)) * norm_weight) * sigmoid(gate)).
 *
 * Sizes fixed by the method: dk = dv = 128 and gate rank 128, conv kernel 4.
 * Arithmetic: FP32 with BF16 rounding of q, k, v, raw_g and o; exp is
 * 2^(x*log2 e) on the hardware's approximate exp2, division / square root /
 * reciprocal are the hardware's approximate (full-range) instructions, the
 * gate projection runs on tensor cores with FP32 accumulation.  Only FP32
 * reduction order differs from a sequential evaluation.
 *
 * Ownership and threading: the caller owns every buffer; every pointer is a
 * DEVICE pointer of the current device.  The library allocates nothing,
 * never synchronises, and enqueues exactly one kernel on `stream` per call
 * (kda_lin_prompt: up to three, kda_ssm_prompt: up to two).
 * The kernels of kda_conv_*, kda_ssm_step, kda_linear and, where no sequence
 * is longer than 64, kda_ssm_prompt are launched so that they may start while
 * the kernel before them on the stream ends; they read and write nothing
 * before it has.
 * Calls are reentrant and may come from several host threads at once (the
 * first call on a device reads its attributes and configures the kernel
 * under a lock); two calls that write the same pool regions must be ordered
 * by the caller (same stream or events).
 *
 * Aliasing contract: within one call, the state pages and conv rows touched
 * by different requests must be distinct (distinct slots per request).  An
 * item may write the page it read (same slot): its read completes first.
 */
#ifndef KDA_GB300_H
#define KDA_GB300_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define KDA_ABI_VERSION 7
#define KDA_DK 128
#define KDA_MAX_TOKENS 8

/* Host-side return codes (nothing is launched unless KDA_SUCCESS). */
enum {
  KDA_SUCCESS = 0,
  KDA_ERR_NULL_ARGS = 1,      /* args == NULL                                  */
  KDA_ERR_TOKENS = 2,         /* tokens outside 1..8 (KdaWide.__init__), or    */
                              /* kda_decode with tokens != 1, kda_verify == 1  */
  KDA_ERR_GATE_MODE = 3,      /* gate_mode not 0|1 (KdaWide.__init__)          */
  KDA_ERR_RECORD = 4,         /* record with tokens == 1 (KdaWide.__init__)    */
  KDA_ERR_NULL_POINTER = 5,   /* a required pointer is NULL                    */
  KDA_ERR_CONV_WIDTH = 6,     /* conv_width < tokens + 2, or too wide to stage */
                              /* (kda_conv_*: width < taps - 1)                */
  KDA_ERR_ALIGNMENT = 7,      /* a pointer breaks its alignment rule (below)   */
  KDA_ERR_SHAPE = 8,          /* negative sizes, num_slots < 1, slot_cols <    */
                              /* tokens, or an item count beyond 2^31-1        */
  KDA_ERR_DEVICE = 9,         /* no usable device, or not an sm_103 device     */
  KDA_ERR_LAUNCH = 10,        /* the kernel launch failed (CUDA error)         */
  KDA_ERR_PATH = 11,          /* path outside 0..2                             */
  KDA_ERR_WORKSPACE = 12,     /* kda_lin_prompt, kda_ssm_prompt: workspace     */
                              /* missing or too small                          */
  KDA_ERR_ACTIVATION = 13     /* kda_linear: activation not a KDA_ACT_*        */
};

/* Device-side error flags, OR-ed into *err when err != NULL.  An item that
 * raises one is handled like padding (zero output rows, nothing written). */
enum {
  KDA_DEVERR_SLOT = 1,        /* slot, conv slot or a write target >= num_slots,
                                 or a conv slot <= 0 on a live verify item     */
  KDA_DEVERR_ACCEPTED = 2,    /* accepted[r] outside 1..tokens                 */
  KDA_DEVERR_TIMEOUT = 4,     /* an on-chip copy wait ran out (the kernel      */
                              /* stopped early; outputs are incomplete)        */
  KDA_DEVERR_SEQ = 8          /* prompt calls: seq_starts out of order or       */
                              /* outside 0..tokens, or a sequence longer than  */
                              /* max_seq                                       */
};

/* Arguments of one step.  Layouts are row-major; dim = heads * 128.
 * Alignment: state, f_a, f_b, x, gate and conv_state 16 bytes; the other BF16
 * arrays 2 bytes, FP32/int32 arrays 4 bytes. */
typedef struct kda_args {
  int32_t batch;       /* B requests (0 is a no-op)                          */
  int32_t heads;       /* H heads (0 is a no-op)                             */
  int32_t tokens;      /* T: 1 = decode, 2..8 = verify                       */
  int32_t num_slots;   /* slots in both pools; slot 0 is the null slot       */
  int32_t conv_width;  /* W columns per conv channel row, >= T + 2           */
  int32_t slot_cols;   /* row stride of `slots` in verify, >= T (decode: 1)  */
  int32_t gate_mode;   /* 0: one FP32 chain over the rank; 1: four chains    */
                       /* over rank quarters, then 0 + (((c0+c1)+c2)+c3)     */
  int32_t has_bias;    /* conv bias present                                  */
  int32_t record;      /* record ("RecoverSSM verify") mode, T > 1 only      */
  int32_t use_pdl;     /* launch with programmatic dependent launch (the     */
                       /* page's griddepcontrol ordering): the kernel may    */
                       /* start before the preceding kernel on the stream    */
                       /* ends.  It reads the state pages, slots and         */
                       /* accepted BEFORE waiting for that kernel; every     */
                       /* other input (x, gate, f_a, beta, the conv pool,    */
                       /* the weights) and all of its writes come after.  So */
                       /* the preceding kernel must not write the state      */
                       /* pool, slots or accepted: two steps chained with    */
                       /* PDL must use disjoint state pages.  Ignored by the */
                       /* cluster-split path (path 2).                       */

  const void *x;            /* bf16 [B*T, 3*dim]  q | k | v column blocks    */
  const void *conv_weight;  /* bf16 [3, 4, dim]   (part, tap, channel)       */
  const void *conv_bias;    /* bf16 [3*dim] (has_bias) else ignored          */
  const void *f_a;          /* bf16 [B*T, 128]                               */
  const void *f_b;          /* bf16 [dim, 128]    (feature, rank)            */
  const void *beta;         /* bf16 [B*T, H]      raw logits                 */
  const void *gate;         /* bf16 [B*T, dim]    output gate logits         */
  const void *norm_weight;  /* bf16 [128]         shared by all heads        */
  const float *a_log;       /* f32  [H]                                      */
  const float *dt_bias;     /* f32  [dim]                                    */
  const int32_t *slots;     /* i32  [B] (decode) or [B, slot_cols] (verify)  */
  const int32_t *accepted;  /* i32  [B] (verify), ignored by decode          */

  void *conv_state;         /* bf16 (or f32, conv_f32) [num_slots, 3*dim, W] */
  float *state;             /* f32  [num_slots, H, 128, 128]     in/out      */
  void *output;             /* bf16 [B*T, dim]                   out         */
  float *rec_u;             /* f32  [B, H, T, 128]  record only, else NULL   */
  void *rec_kg;             /* bf16 [B, H, T, 256]  record only: k | raw_g   */

  float lower_bound;        /* decay lower bound (e.g. -5)                   */
  float scale;              /* q scale (e.g. 128^-0.5)                       */
  float eps;                /* RMSNorm epsilon (the L2 norms use 1e-6)       */

  int32_t *err;             /* optional device word for KDA_DEVERR_* flags   */
  void *dbg;                /* optional bf16 [B, H, T, 4, 128]: q, k, v      */
                            /* (after SiLU, before the norm) and raw_g, as   */
                            /* this call rounded them; for parity checks     */
  int32_t path;             /* kernel: 0 = automatic; 1 = persistent, one    */
                            /* CTA per SM walking a range of items (for many */
                            /* items); 2 = one item per cluster of 4 CTAs,   */
                            /* each owning 32 value rows (for few items;     */
                            /* ignores use_pdl).  Both give the same bits.   */
  int32_t conv_f32;         /* conv_state holds FP32 instead of BF16: taps   */
                            /* are read as stored and the new window is      */
                            /* written as FP32 (the page's conv_type is the  */
                            /* pool's element type)                          */
  int32_t *sched;           /* optional i32 [2] device scheduler words, zero */
                            /* before first use; the kernel leaves them zero */
                            /* when it ends.  With them the persistent path  */
                            /* hands the items past the CTAs' contiguous     */
                            /* ranges out one at a time to whichever CTA is  */
                            /* free (an eighth of the items for decode with  */
                            /* >= 32 items per SM and for record steps, else */
                            /* the remainder of an even split; same bits as  */
                            /* without); NULL = fixed contiguous ranges.     */
                            /* Launches that may run at the same time (other */
                            /* streams, other threads) need separate words;  */
                            /* launches in order on one stream, PDL-chained  */
                            /* or captured in a graph, may share them.       */
                            /* Ignored by the cluster-split path (path 2).   */
} kda_args;

/* One decode step (tokens == 1) on `stream` (a cudaStream_t; NULL = the
 * legacy default stream).  Returns KDA_SUCCESS or a KDA_ERR_* code. */
int kda_decode(const kda_args *args, void *stream);

/* One speculative-verify step (tokens 2..8, record optional) on `stream`. */
int kda_verify(const kda_args *args, void *stream);

/* kda_decode (tokens == 1) or kda_verify (tokens > 1) with no caller
 * allocation: args->sched is ignored and the library's own scheduler words
 * (a static, zero-initialised device array per GPU, left zero by every
 * launch) are used instead.  Every launch through this entry on one GPU
 * shares those words, so such launches must not run at the same time: issue
 * them in order on one stream (PDL chaining and graph capture are fine);
 * concurrent streams or threads pass their own words to kda_decode /
 * kda_verify.  Same return codes and bits as those calls. */
int kda_step_noalloc(const kda_args *args, void *stream);

/* Arguments of one record replay (kda_recover). */
typedef struct kda_recover_args {
  int32_t batch;            /* B requests (0 is a no-op)                       */
  int32_t heads;            /* H heads (0 is a no-op)                          */
  int32_t tokens;           /* T of the records, 1..8                          */
  int32_t num_slots;        /* slots in the state pool                         */
  const int32_t *src_slots; /* i32 [B]: checkpoint page; <= 0 = padding        */
  const int32_t *dst_slots; /* i32 [B]: page to write; <= 0 = padding; may     */
                            /* equal src_slots[r]                              */
  const int32_t *accepted;  /* i32 [B]: tokens to replay, 0..T (0 = copy)      */
  const float *rec_u;       /* f32 [B, H, T, 128] from a record-mode verify    */
  const void *rec_kg;       /* bf16 [B, H, T, 256]: k (pre-norm) | raw_g       */
  const float *a_log;       /* f32 [H]                                         */
  const float *dt_bias;     /* f32 [H*128]                                     */
  float lower_bound;        /* as in the step that wrote the records           */
  float *state;             /* f32 [num_slots, H, 128, 128]       in/out       */
  int32_t *err;             /* optional device word for KDA_DEVERR_* flags     */
  int32_t *sched;           /* optional i32 [2] scheduler words, as in         */
                            /* kda_args (zero before first use, left zero;     */
                            /* concurrent launches need their own); NULL =     */
                            /* contiguous item ranges only.  Same bits.        */
} kda_recover_args;

/* Record replay ("RecoverSSM" on the page, referenced but not shown there).
 * A record-mode kda_verify writes no state; it leaves per token the BF16 k
 * before the L2 norm, the BF16 raw gate and the FP32 u of every value row.
 * For each (request r, head h): start from state[src_slots[r], h], for the
 * first accepted[r] tokens decay every key column by the decay of the
 * recorded raw gate and add k_hat u^T (k_hat: L2-normalised recorded k), and
 * write the page to state[dst_slots[r], h].  The arithmetic is the step's, so
 * replaying the records of a record-mode verify reproduces bit for bit the
 * page a non-record verify writes after token accepted[r]-1.
 * Pointers are device pointers; state, rec_u and rec_kg need 16-byte
 * alignment.  Slot >= num_slots or accepted outside 0..T raise
 * KDA_DEVERR_SLOT / KDA_DEVERR_ACCEPTED and the item writes nothing.  Pages
 * of different requests must be distinct.  One kernel on `stream`. */
int kda_recover(const kda_recover_args *args, void *stream);

/* Arguments of one output-projection consumer epilogue (kda_oproj). */
typedef struct kda_oproj_args {
  int32_t tp;               /* partial outputs per token (TP ranks), 1..64     */
  int32_t tokens;           /* rows (0 is a no-op)                             */
  int32_t hidden;           /* features per row: a multiple of 256, <= 7168    */
  int32_t nb;               /* earlier block outputs per token, 0..8           */
  int32_t has_delta;        /* nonzero: new prefix = BF16(prefix + BF16(sum)); */
                            /* zero: new prefix = BF16(sum)                    */
  const void *partials;     /* bf16 [tp, tokens, hidden]: the partial sums     */
  const void *blocks;       /* bf16 [tokens, nb, hidden]; NULL when nb == 0    */
  const void *norm;         /* bf16 [hidden] (nb > 0): block RMSNorm weight    */
  const void *query;        /* bf16 [hidden] (nb > 0): block query             */
  const void *out_norm;     /* bf16 [hidden]: output RMSNorm weight            */
  void *prefix;             /* bf16 [tokens, hidden], in/out: the residual     */
                            /* stream, replaced by the new prefix              */
  void *output;             /* bf16 [tokens, hidden], out                      */
  float eps;                /* epsilon of the block (and prefix) RMS           */
  float out_eps;            /* epsilon of the output RMSNorm                   */
} kda_oproj_args;

/* Output-projection consumer epilogue on one GPU: the per-token arithmetic
 * of class OprojConsumer on the vLLM API page
 *   "vllm.models.kimi_k3.nvidia.specialized_decode.cutedsl.oproj.consumer"
 * (poll_sum, combined_weight, pre, post), with the tensor-parallel partial
 * outputs read from `partials` instead of remote mailboxes and the whole
 * hidden vector of a token in one CTA instead of a cluster.  Per token:
 *   1. sum = the tp partials, summed in FP32 in four rank groups of
 *      S = max(4, ceil(tp/4)) (each in rank order, then the groups in order);
 *      p = BF16(sum), or BF16(prefix + BF16(sum)) with has_delta; p is
 *      written back to `prefix`;
 *   2. with nb > 0: w = norm * query; logit_b = (v_b . w) * rstd(v_b . v_b,
 *      eps) for every block and likewise for p; a softmax over the blocks and
 *      p weights y = sum_b e_b v_b + e_p p;
 *   3. output = BF16(out_norm * y * rstd(y . y, out_eps)) (y = p when nb == 0),
 * where rstd(s, e) = 1 / sqrt(s / hidden + e) (a reading: the page uses rstd
 * without defining it).  FP32 arithmetic; exp and the reciprocal square root
 * on the hardware's approximate instructions; only the FP32 reduction order
 * over features differs from a sequential evaluation.  The MoE "latent"
 * copies and hints of the page's publish step are multi-GPU plumbing and are
 * not produced.  All pointers are device pointers of the current device with
 * 16-byte alignment; partials, blocks and prefix must not overlap output.
 * Errors: KDA_ERR_NULL_ARGS, KDA_ERR_NULL_POINTER, KDA_ERR_SHAPE (sizes
 * outside the ranges above), KDA_ERR_ALIGNMENT, KDA_ERR_DEVICE,
 * KDA_ERR_LAUNCH; nothing is launched on error.  One kernel on `stream`. */
int kda_oproj(const kda_oproj_args *args, void *stream);

/* ---- Linear attention with one decay per head -------------------------------
 *
 * The companion of the KDA step for layers whose state decays by one factor
 * per head instead of one per key and takes no delta correction.  Per head,
 * on the same 128x128 FP32 page [value row i][key j]:
 *     S_t = exp(g_t) S_{t-1} + v_t k_t^T,      o_t = scale * S_t q_t.
 * q and k have qk_heads heads, v and o heads; value head h reads query and key
 * head h / (heads / qk_heads).  g (`decay`) is the logarithm of the decay, <= 0:
 * f32 [heads] (decay_rows 0) or one per token, f32 [rows, heads] contiguous
 * (decay_rows 1); -inf is a reset (the factor 0).  Rows of q, k, v and output
 * are BF16 [head][128] and may be slices of wider rows: row t starts at
 * t * stride elements, strides are multiples of 8 and at least the row's own
 * width; q, k, v, output and state are 16-byte aligned, the other arrays 4. */

/* Arguments of one prompt call (kda_lin_prompt). */
typedef struct kda_lin_prompt_args {
  int32_t seqs;             /* sequences (0 is a no-op)                        */
  int32_t heads;            /* value heads H, <= 65536 (0 is a no-op)          */
  int32_t qk_heads;         /* query / key heads, a divisor of heads           */
  int32_t tokens;           /* rows of q, k, v and output                      */
  int32_t max_seq;          /* no sequence is longer than this                 */
  int32_t num_slots;        /* slots of `state` (ignored without slots)        */
  int32_t decay_rows;       /* 0: decay is [heads]; 1: [tokens, heads]         */
  int32_t path;             /* 0 = automatic; 1 = recurrent (token by token);  */
                            /* 2 = chunked (128 tokens at a time)              */
  int64_t q_stride, k_stride, v_stride, o_stride;   /* elements between rows   */
  const void *q;            /* bf16 [tokens, qk_heads * 128]                   */
  const void *k;            /* bf16 [tokens, qk_heads * 128]                   */
  const void *v;            /* bf16 [tokens, heads * 128]                      */
  const float *decay;       /* f32: see decay_rows                             */
  const int32_t *seq_starts;/* i32 [seqs + 1]: sequence r is rows              */
                            /* seq_starts[r] .. seq_starts[r + 1] - 1          */
  const int32_t *src_slots; /* i32 [seqs] or NULL: page a sequence starts from;*/
                            /* <= 0 (or NULL): from zeros.  May be shared      */
  const int32_t *dst_slots; /* i32 [seqs] or NULL: page its last state goes to;*/
                            /* <= 0 (or NULL): dropped.  Distinct, and no      */
                            /* other sequence's src; may be its own src        */
  float *state;             /* f32 [num_slots, heads, 128, 128] (with slots)   */
  void *output;             /* bf16 [tokens, heads * 128]                      */
  float scale;              /* of the output                                   */
  int32_t *err;             /* optional device word for KDA_DEVERR_* flags     */
  void *workspace;          /* 256-byte aligned; NULL when none is needed      */
  int64_t workspace_bytes;  /* at least kda_lin_prompt_workspace(args)         */
} kda_lin_prompt_args;

/* Bytes of workspace that kda_lin_prompt needs for args' sizes and strides (no
 * pointer is followed), 0 for none or for sizes that it refuses; -1 when args is
 * NULL.  The workspace holds nothing between
 * calls; calls that may run at the same time need their own. */
int64_t kda_lin_prompt_workspace(const kda_lin_prompt_args *args);

/* Prompt form over ragged sequences, chunked: a sequence's outputs and last
 * state from its first state.  Rows that no sequence covers are left as they
 * are; a sequence without tokens copies its first state.  A sequence with a
 * flagged slot (KDA_DEVERR_SLOT) or range (KDA_DEVERR_SEQ) writes nothing; starts
 * out of order can make other sequences share rows, whose outputs are then any
 * of theirs, and flag (KDA_DEVERR_SEQ) every sequence that the call would have
 * split.  An infinity or NaN in a live row reaches what the formulas send it to,
 * its own and later tokens of its sequence and head, as an infinity or NaN; rows
 * outside the sequence reach nothing.  The output must not overlap the inputs.
 *
 * The page is held and updated in FP32; products that only feed the BF16 output
 * are rounded to BF16 once.  The chunked form takes factors of up to 2^64 both
 * ways on the way to an output: q k and the page's elements keep their digits
 * from 2^-62 on (what is smaller is off by up to 2^-62 times v or q), the sums of
 * |q k v| and |S q| have to be below 2^62 and the scale within 2^-62 and 2^62, and
 * factors under 2^-126 are 0; path 1 has no such limits.
 *
 * Errors: KDA_ERR_NULL_ARGS, KDA_ERR_NULL_POINTER, KDA_ERR_SHAPE (sizes and
 * strides outside the rules above), KDA_ERR_PATH, KDA_ERR_ALIGNMENT,
 * KDA_ERR_WORKSPACE, KDA_ERR_DEVICE, KDA_ERR_LAUNCH; nothing is launched on error.
 * Up to three kernels on `stream`, in order. */
int kda_lin_prompt(const kda_lin_prompt_args *args, void *stream);

/* Arguments of one single-token step (kda_lin_step). */
typedef struct kda_lin_step_args {
  int32_t batch;            /* requests, one row each (0 is a no-op)           */
  int32_t heads;            /* value heads H (0 is a no-op)                    */
  int32_t qk_heads;         /* query / key heads, a divisor of heads           */
  int32_t num_slots;
  int32_t decay_rows;       /* 0: decay is [heads]; 1: [batch, heads]          */
  int64_t q_stride, k_stride, v_stride, o_stride;   /* elements between rows   */
  const void *q, *k, *v;    /* bf16 [batch, qk_heads (v: heads) * 128]         */
  const float *decay;
  const int32_t *slots;     /* i32 [batch]: the page, updated in place; <= 0 = */
                            /* padding (a row of zeros, nothing else written)  */
  float *state;             /* f32 [num_slots, heads, 128, 128]       in/out   */
  void *output;             /* bf16 [batch, heads * 128]                       */
  float scale;
  int32_t *err;             /* optional device word for KDA_DEVERR_* flags     */
} kda_lin_step_args;

/* Recurrent form, one token per request.  Live requests have distinct slots; the
 * output must not overlap the inputs.
 * A slot >= num_slots raises KDA_DEVERR_SLOT and is handled as padding.  One
 * kernel on `stream`. */
int kda_lin_step(const kda_lin_step_args *args, void *stream);

/* ---- Snapshots: state pages kept in 8 or 4 bits ------------------------------
 *
 * A snapshot keeps one slot's pages (of the KDA step or of the linear
 * attention above) for later: a prefix cache, a request to fork.  It holds the
 * state pages only: the KDA step's convolution window of the slot (conv_state[slot])
 * is the caller's to copy beside it.  Codes are
 * whole numbers -L .. L, L = 127 (bits 8) or 7 (bits 4), with one FP32 scale
 * for a group of keys of one value row (bits 8: the row's 128 keys; bits 4: 32
 * keys).  With m the group's largest magnitude: scale = m / L rounded to FP32
 * and code = x / scale to the nearest whole number, ties to even, decided as
 * in exact arithmetic.  Groups with m < 2^-118 are kept as zeros (scale 0);
 * groups with an infinity or NaN are kept as NaN (scale NaN, codes 0).  Reading
 * gives code * scale in FP32.  Two 4-bit codes share a byte: key 2j in the low
 * half, 2j + 1 in the high half, in two's complement. */
typedef struct kda_snapshot_args {
  int32_t count;            /* entries (0 is a no-op)                          */
  int32_t heads;            /* H heads (0 is a no-op)                          */
  int32_t num_slots;        /* slots of `state`                                */
  int32_t num_snaps;        /* rows of `codes` and `scales`                    */
  int32_t bits;             /* 8 or 4                                          */
  const int32_t *slots;     /* i32 [count]: pool slot; <= 0 = padding          */
  const int32_t *snaps;     /* i32 [count]: snapshot; <= 0 = padding           */
  float *state;             /* f32 [num_slots, heads, 128, 128]                */
  void *codes;              /* bits 8: i8 [num_snaps, heads, 128, 128];        */
                            /* bits 4: u8 [num_snaps, heads, 128, 64]          */
  float *scales;            /* f32 [num_snaps, heads, 128 (bits 4: , 4)]       */
  int32_t *err;             /* optional device word for KDA_DEVERR_* flags     */
} kda_snapshot_args;

/* Quantises state[slots[i]] into snapshot snaps[i], all heads.  The snapshots
 * written are distinct.  Pointers to state, codes and scales are 16-byte
 * aligned.  A slot or snapshot past its pool raises KDA_DEVERR_SLOT and the
 * entry writes nothing.  One kernel on `stream`. */
int kda_snapshot_save(const kda_snapshot_args *args, void *stream);

/* Reads snapshot snaps[i] back into state[slots[i]], all heads; the slots
 * written are distinct, a snapshot may be read into several.  Rules as above. */
int kda_snapshot_load(const kda_snapshot_args *args, void *stream);

/* ---- Short causal convolution ------------------------------------------------
 *
 * The depthwise convolution in front of a recurrent layer, for prompts and for
 * single tokens.  Per channel c, over a sequence's inputs x and the taps - 1
 * inputs before it:
 *     y_t = bias_c + sum_j weight[j, c] x[t - taps + 1 + j, c],
 *     output = BF16(silu(y)) or BF16(y),
 * summed in FP32 from the bias on, oldest input first, with the KDA step's
 * arithmetic: on a KDA layer's q, k and v (parts 3, taps 4, conv_state as the
 * window) a prompt leaves the bits that decoding it token by token would (but
 * values below 2^-118 may be zeros).
 * A window pool [num_slots, channels, width] keeps a slot's last inputs, oldest
 * first, in columns 0 .. taps - 2; other columns are left alone.  Rows of x and
 * output are BF16 [channels] and may be slices of wider rows: strides are
 * multiples of 8 elements and at least the row's width.  x, output, weight, bias and
 * window are 16-byte aligned, the index arrays 4.  The output must not overlap
 * the inputs.  (Rows and sequences of this call and of those below: up
 * to 2^31 - 256.) */

/* Arguments of one prompt call (kda_conv_prompt). */
typedef struct kda_conv_prompt_args {
  int32_t seqs;             /* sequences (0 is a no-op)                        */
  int32_t channels;         /* a multiple of 8 * parts (0 is a no-op)          */
  int32_t parts;            /* blocks of channels that `weight` is stored in   */
  int32_t taps;             /* 2..4                                            */
  int32_t tokens;           /* rows of x and output                            */
  int32_t num_slots;        /* slots of `window` (ignored without slots)       */
  int32_t width;            /* columns of `window`, >= taps - 1                */
  int32_t window_f32;       /* window holds FP32 instead of BF16               */
  int32_t silu;             /* nonzero: SiLU on the output                     */
  int64_t x_stride, o_stride;               /* elements between rows           */
  const void *x;            /* bf16 [tokens, channels]                         */
  const void *weight;       /* bf16 [parts, taps, channels / parts]            */
  const void *bias;         /* bf16 [channels] or NULL                         */
  const int32_t *seq_starts;/* i32 [seqs + 1]: sequence r is rows              */
                            /* seq_starts[r] .. seq_starts[r + 1] - 1          */
  const int32_t *src_slots; /* i32 [seqs] or NULL: window a sequence continues */
                            /* from; <= 0 (or NULL): zeros.  May be shared     */
  const int32_t *dst_slots; /* i32 [seqs] or NULL: window its last inputs go   */
                            /* to; <= 0 (or NULL): dropped.  Distinct, and no  */
                            /* other sequence's src; may be its own src        */
  void *window;             /* [num_slots, channels, width] (with slots)       */
  void *output;             /* bf16 [tokens, channels]                         */
  int32_t *err;             /* optional device word for KDA_DEVERR_* flags     */
} kda_conv_prompt_args;

/* Rows that no sequence covers are left as they are; a sequence shorter than
 * taps - 1 keeps the newest of its first window.  A sequence with a flagged slot
 * (KDA_DEVERR_SLOT) or range (KDA_DEVERR_SEQ) writes nothing; where starts are out
 * of order, the call's other sequences may be incomplete.  Errors: KDA_ERR_NULL_ARGS,
 * KDA_ERR_SHAPE, KDA_ERR_CONV_WIDTH, KDA_ERR_NULL_POINTER, KDA_ERR_ALIGNMENT,
 * KDA_ERR_DEVICE, KDA_ERR_LAUNCH; nothing is launched on error.  One kernel on
 * `stream`. */
int kda_conv_prompt(const kda_conv_prompt_args *args, void *stream);

/* Arguments of one single-token call (kda_conv_step). */
typedef struct kda_conv_step_args {
  int32_t batch;            /* requests, one row each (0 is a no-op)           */
  int32_t channels, parts, taps;
  int32_t num_slots, width, window_f32, silu;
  int64_t x_stride, o_stride;               /* elements between rows           */
  const void *x;            /* bf16 [batch, channels]                          */
  const void *weight;       /* bf16 [parts, taps, channels / parts]            */
  const void *bias;         /* bf16 [channels] or NULL                         */
  const int32_t *slots;     /* i32 [batch]: the window, shifted in place;      */
                            /* <= 0 = padding (a row of zeros, nothing else    */
                            /* written)                                        */
  void *window;             /* [num_slots, channels, width]           in/out   */
  void *output;             /* bf16 [batch, channels]                          */
  int32_t *err;             /* optional device word for KDA_DEVERR_* flags     */
} kda_conv_step_args;

/* One token per request.  Live requests have distinct slots.  A slot >= num_slots
 * raises KDA_DEVERR_SLOT and is handled as padding.  One kernel on `stream`. */
int kda_conv_step(const kda_conv_step_args *args, void *stream);

/* ---- Selective state-space scan ----------------------------------------------
 *
 * Per channel c with `states` states h_n, B and C shared by the channels of a
 * group (channel c reads group c / (channels / groups)):
 *     s_t = dt[t, c] + dt_bias[c], then softplus(s) = log(1 + exp(s)) if asked,
 *     h_n <- exp(s_t a[c, n]) h_n + s_t x[t, c] b[t, n],
 *     y_t = sum_n c[t, n] h_n + d[c] x[t, c],     output = BF16(y silu(z)),
 * in FP32, with the state in FP32 [num_slots, channels, states].  a is the decays'
 * rate, < 0 in use (-exp of a stored logarithm).  dt_bias, d and z may be NULL (0, 0,
 * no gate).  Rows of x, dt, b, c, z and output are BF16 and may be slices of wider
 * rows: strides are multiples of 8 elements and at least the row's own width.  They,
 * a and state are 16-byte aligned, the other arrays 4.  The output must not overlap
 * the inputs.  A slot has up to 2^31 - 256 states (channels * states).  a is finite;
 * where it grows (s a > 0), it has to stay below 2^64 over a sequence.  An infinity or NaN
 * reaches later tokens of its sequence and channel as an infinity or NaN; an infinite
 * state stays as it is while the decays since then are above 2^-126. */

/* Arguments of one prompt call (kda_ssm_prompt). */
typedef struct kda_ssm_prompt_args {
  int32_t seqs;             /* sequences (0 is a no-op)                        */
  int32_t channels;         /* a multiple of 8 * groups (0 is a no-op)         */
  int32_t states;           /* 16, 32 or 64                                    */
  int32_t groups;           /* of channels that share b and c                  */
  int32_t tokens;           /* rows                                            */
  int32_t max_seq;          /* no sequence is longer than this                 */
  int32_t num_slots;        /* slots of `state` (ignored without slots)        */
  int32_t softplus;         /* nonzero: softplus on dt + dt_bias               */
  int32_t path;             /* 0 = automatic; 1 = sequences whole; 2 = long    */
                            /* ones in segments                                */
  int64_t x_stride, dt_stride, b_stride, c_stride, z_stride, o_stride;
  const void *x, *dt;       /* bf16 [tokens, channels]                         */
  const float *a;           /* f32 [channels, states]                          */
  const void *b, *c;        /* bf16 [tokens, groups * states]                  */
  const float *d;           /* f32 [channels] or NULL                          */
  const void *z;            /* bf16 [tokens, channels] or NULL                 */
  const float *dt_bias;     /* f32 [channels] or NULL                          */
  const int32_t *seq_starts;/* i32 [seqs + 1]: sequence r is rows              */
                            /* seq_starts[r] .. seq_starts[r + 1] - 1          */
  const int32_t *src_slots; /* i32 [seqs] or NULL: state a sequence starts     */
                            /* from; <= 0 (or NULL): zeros.  May be shared     */
  const int32_t *dst_slots; /* i32 [seqs] or NULL: where its last state goes;  */
                            /* <= 0 (or NULL): dropped.  Distinct, and no      */
                            /* other sequence's src; may be its own src        */
  float *state;             /* f32 [num_slots, channels, states] (with slots)  */
  void *output;             /* bf16 [tokens, channels]                         */
  int32_t *err;             /* optional device word for KDA_DEVERR_* flags     */
  void *workspace;          /* 256-byte aligned; NULL when none is needed      */
  int64_t workspace_bytes;  /* at least kda_ssm_prompt_workspace(args)         */
} kda_ssm_prompt_args;

/* Bytes of workspace that kda_ssm_prompt needs for args' sizes and strides (no
 * pointer is followed), 0 for none or for sizes that it refuses; -1 when args is
 * NULL.  The workspace holds nothing between calls; calls that may run at the same
 * time need their own. */
int64_t kda_ssm_prompt_workspace(const kda_ssm_prompt_args *args);

/* Rows that no sequence covers are left as they are; a sequence without tokens
 * copies its first state.  A sequence with a flagged slot (KDA_DEVERR_SLOT) or range
 * (KDA_DEVERR_SEQ) writes nothing; where starts are out of order, the call's other
 * sequences may be incomplete.  Errors: KDA_ERR_NULL_ARGS, KDA_ERR_SHAPE,
 * KDA_ERR_PATH, KDA_ERR_NULL_POINTER, KDA_ERR_ALIGNMENT, KDA_ERR_WORKSPACE,
 * KDA_ERR_DEVICE, KDA_ERR_LAUNCH; nothing is launched on error.  Up to two
 * kernels on `stream`, in order. */
int kda_ssm_prompt(const kda_ssm_prompt_args *args, void *stream);

/* Arguments of one single-token step (kda_ssm_step). */
typedef struct kda_ssm_step_args {
  int32_t batch;            /* requests, one row each (0 is a no-op)           */
  int32_t channels, states, groups;
  int32_t num_slots, softplus;
  int64_t x_stride, dt_stride, b_stride, c_stride, z_stride, o_stride;
  const void *x, *dt;       /* bf16 [batch, channels]                          */
  const float *a;           /* f32 [channels, states]                          */
  const void *b, *c;        /* bf16 [batch, groups * states]                   */
  const float *d;           /* f32 [channels] or NULL                          */
  const void *z;            /* bf16 [batch, channels] or NULL                  */
  const float *dt_bias;     /* f32 [channels] or NULL                          */
  const int32_t *slots;     /* i32 [batch]: the state, updated in place; <= 0  */
                            /* = padding (a row of zeros, nothing else written) */
  float *state;             /* f32 [num_slots, channels, states]      in/out   */
  void *output;             /* bf16 [batch, channels]                          */
  int32_t *err;             /* optional device word for KDA_DEVERR_* flags     */
} kda_ssm_step_args;

/* One token per request.  Live requests have distinct slots.  A slot >= num_slots
 * raises KDA_DEVERR_SLOT and is handled as padding.  One kernel on `stream`. */
int kda_ssm_step(const kda_ssm_step_args *args, void *stream);

/* ---- Projections ---------------------------------------------------------------
 *
 *     output = BF16(act(x W^T + bias) + residual),
 * x [rows, inner] and W [outer, inner] (a linear layer's weight) BF16, products
 * summed in FP32 on the tensor cores, the epilogue in FP32, one rounding. */
enum { KDA_ACT_NONE = 0, KDA_ACT_SILU = 1, KDA_ACT_GELU = 2 /* with erf */,
       KDA_ACT_SOFTPLUS = 3 };

/* Arguments of one product (kda_linear).  All rows may be slices of wider rows:
 * strides are multiples of 8 elements and at least the row's own width, which may
 * be odd.  All pointers but err (4) are 16-byte aligned. */
typedef struct kda_linear_args {
  int32_t rows;             /* of x and output (0 is a no-op)                  */
  int32_t inner;            /* length of the sums, >= 1                        */
  int32_t outer;            /* columns of output (0 is a no-op)                */
  int32_t activation;       /* a KDA_ACT_*                                     */
  int64_t x_stride, w_stride, r_stride, o_stride;   /* elements between rows   */
  const void *x;            /* bf16 [rows, inner]                              */
  const void *weight;       /* bf16 [outer, inner]                             */
  const void *bias;         /* bf16 [outer] or NULL                            */
  const void *residual;     /* bf16 [rows, outer] or NULL; may be the output   */
                            /* itself (same address and stride)                */
  void *output;             /* bf16 [rows, outer]; overlaps no other input     */
  int32_t *err;             /* optional device word for KDA_DEVERR_* flags     */
} kda_linear_args;

/* Columns behind `outer` in a wider row are left as they are.  An infinity or NaN
 * reaches the sums that it is part of only.  Where a wait on the chip runs out (2 s each;
 * kda_linear has none for one row of up to 32768), KDA_DEVERR_TIMEOUT is set and the
 * output is incomplete: without `err` nobody learns of it, as the call has returned by
 * then.  Errors: KDA_ERR_NULL_ARGS,
 * KDA_ERR_SHAPE, KDA_ERR_ACTIVATION, KDA_ERR_NULL_POINTER, KDA_ERR_ALIGNMENT,
 * KDA_ERR_DEVICE, KDA_ERR_LAUNCH; nothing is launched on error.  One kernel on
 * `stream`. */
int kda_linear(const kda_linear_args *args, void *stream);

/* The same in a form of the caller's choice.  path 0: kda_linear's own; 1: 128 columns of
 * output and up to 256 rows to a block of threads or a cluster of them (few tiles); 2:
 * 256 x 256 to a pair of them, which takes several in turn (many tiles; outer >= 8).
 * Further errors: KDA_ERR_PATH, and KDA_ERR_SHAPE where a form does not take the sizes. */
int kda_linear_path(const kda_linear_args *args, int32_t path, void *stream);

/* Self-test of the bounded on-chip wait of the KDA step, the replay and the
 * output projection: one CTA waits on an mbarrier that nothing completes; the
 * wait gives up after its wall-clock limit (2 s), KDA_DEVERR_TIMEOUT is OR-ed
 * into *err (a device word, 4-byte aligned) and the kernel returns -- no trap, no
 * fault, the context stays usable.  For failure-detection tests.  Returns
 * KDA_ERR_NULL_POINTER / KDA_ERR_ALIGNMENT / KDA_ERR_LAUNCH or KDA_SUCCESS;
 * one kernel on `stream`. */
int kda_selftest_wait_timeout(int32_t *err, void *stream);

/* The same for the wait of kda_lin_prompt's chunked form (the other kernels of
 * the linear attention and the snapshots wait for nothing on the chip): a CTA of
 * that form's size takes TMEM, passes a completed phase, waits for one that
 * nothing completes until the same limit, and leaves as that form leaves. */
int kda_selftest_lin_wait_timeout(int32_t *err, void *stream);

/* Static description of a return code (never NULL). */
const char *kda_strerror(int code);

/* KDA_ABI_VERSION of the loaded library. */
int kda_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* KDA_GB300_H */

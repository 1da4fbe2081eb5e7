/*
 * gdn2.h -- C ABI of the Gated DeltaNet-2 operator library (libgdn2.so).
 *
 * The operator is the gated delta rule with decoupled erase and write gates
 * ("Gated DeltaNet-2: Decoupling Erase and Write in Linear Attention").  Per
 * (batch, head) it keeps a dk x dv state S and, for each token t,
 *
 *     Sbar = Diag(alpha_t) S_{t-1}          alpha_t = exp(log_alpha_t), per key channel
 *     e_t  = b_t (*) k_t                    erase gate b_t on the key axis
 *     z_t  = w_t (*) v_t                    write gate w_t on the value axis
 *     r_t  = Sbar^T e_t
 *     S_t  = Sbar + k_t (z_t - r_t)^T
 *     o_t  = S_t^T q_t                      the query reads the updated state
 *
 * as stated on the iplexlaw.co.kr page, section "Decisiones independientes en
 * dos ejes", and in product form S_t = (I - k_t (b_t (*) k_t)^T) D_t S_{t-1}
 * + k_t (w_t (*) v_t)^T in the zubnet.ai news item and the gist.science
 * summary (section 1, "Gated Delta Rule-2").  No scale is applied to q.
 *
 * Conventions shared by every entry point:
 *   - All tensor arguments are DEVICE pointers owned by the caller.  The
 *     library keeps no per-call state and never synchronises the stream; work
 *     is queued on `stream` (NULL = the legacy default stream) and the call
 *     returns once it is queued.  The bf16 paths of gdn2_fwd_chunked,
 *     gdn2_fwd_chunked_gates and gdn2_layer_fwd, and gdn2_bwd_chunked,
 *     gdn2_swa_bwd and gdn2_block_norm_bwd, need a workspace, which they take
 *     from a stream-ordered pool owned by the library (allocated and released
 *     on `stream`; the pool keeps freed blocks for reuse).  Nothing else
 *     allocates.
 *   - Layouts are dense row-major: q, k, b, log_alpha are [B][T][H][dk];
 *     v, w, o are [B][T][H][dv]; states are [B][H][dk][dv].  (The decode entry
 *     point drops the T axis.)
 *   - `dtype` is the element type of q, k, v, b, w and o.  log_alpha and
 *     every state are always fp32.  bf16 outputs are rounded to nearest even.
 *   - Every pointer must be 16-byte aligned.
 *   - Supported head sizes: dk and dv each 64 or 128.
 *   - The returned status covers argument checks and launch errors only.
 *     A condition found while the kernels run (a bounded wait that gave up) is
 *     recorded in a device-side error word and reported by
 *     gdn2_check_device_error().
 *   - Gates are used as given: values outside [0, 1] (the pages' ablation
 *     widens the erase range to [0, 2]) are not clamped.
 */
#ifndef GDN2_H
#define GDN2_H

#ifdef __cplusplus
extern "C" {
#endif

typedef enum gdn2_status {
    GDN2_OK = 0,
    GDN2_ERR_NULL = 1,           /* a required pointer is NULL                        */
    GDN2_ERR_SHAPE = 2,          /* a size is out of range (negative, zero, too big)  */
    GDN2_ERR_DTYPE = 3,          /* unknown gdn2_dtype code                           */
    GDN2_ERR_ALIGN = 4,          /* a pointer is not 16-byte aligned                  */
    GDN2_ERR_UNSUPPORTED = 5,    /* valid request outside the implemented set         */
    GDN2_ERR_CUDA = 6,           /* a CUDA runtime call or launch failed              */
    GDN2_ERR_DEVICE_TIMEOUT = 7, /* a device-side bounded wait gave up                */
    GDN2_ERR_RANGE = 8,          /* reserved: no longer reported (every decay is computed) */
    GDN2_ERR_SCRATCH_LIMIT = 9   /* needs more than gdn2_fwd_chunked_noalloc's fixed buffer */
} gdn2_status;

typedef enum gdn2_dtype {
    GDN2_F32 = 0,
    GDN2_BF16 = 1
} gdn2_dtype;

/*
 * Gate layouts: which of b, w and log_alpha hold one value per (token, head)
 * instead of one per channel.  Bits of the `layout` argument of
 * gdn2_fwd_chunked_gates and gdn2_decode_tokens; 0 is the per-channel layout of
 * every other entry point.
 *
 * The pages derive the special cases of the operator from these shapes
 * (iplexlaw.co.kr, section "Decisiones independientes en dos ejes"; gist.science,
 * section 1): b = w = beta with beta a scalar per token gives Kimi Delta
 * Attention (pass the same pointer for b and w with GDN2_ERASE_SCALAR |
 * GDN2_WRITE_SCALAR); a scalar decay as well gives Gated DeltaNet (add
 * GDN2_DECAY_SCALAR).  A channel-averaged erase or write gate alone is
 * GDN2_ERASE_SCALAR or GDN2_WRITE_SCALAR.  A scalar tensor is [B][T][H]
 * ([B][H] for gdn2_decode_step's T-less layout), same dtype as the per-channel
 * one; it reads fewer bytes, which is what the bandwidth-bound kernels spend
 * their time on.
 */
typedef enum gdn2_gate_layout {
    GDN2_GATES_PER_CHANNEL = 0,  /* b [..][dk], w [..][dv], log_alpha [..][dk]     */
    GDN2_ERASE_SCALAR = 1,       /* b is [B][T][H]: one erase gate per token, head  */
    GDN2_WRITE_SCALAR = 2,       /* w is [B][T][H]: one write gate per token, head  */
    GDN2_DECAY_SCALAR = 4        /* log_alpha is [B][T][H]: one decay per token, head */
} gdn2_gate_layout;

/* Same type as cudaStream_t; declared here so this header needs no CUDA header. */
typedef struct CUstream_st *gdn2_stream_t;

/*
 * gdn2_fwd_chunked -- prefill / training forward over a whole sequence.
 *
 * Computes o_t for t = 0..T-1 and the final state S_T of the recurrence above,
 * chunkwise with chunks of 64 tokens: the per-channel decay is cumulated in
 * fp32 inside each chunk and folded into asymmetric decayed erase/key factors,
 * the strictly lower triangular 64 x 64 system is solved per chunk, and the
 * state is passed from chunk to chunk (iplexlaw.co.kr, section "Procesamiento
 * del token y entrenamiento paralelo"; gist.science, section 3 "Efficient
 * chunkwise parallel training").  The result equals the token recurrence up
 * to rounding.
 *
 *   q, k, b     [B][T][H][dk]  dtype   query, key, erase gate
 *   v, w        [B][T][H][dv]  dtype   value, write gate
 *   log_alpha   [B][T][H][dk]  fp32    log of the per-key-channel decay (<= 0)
 *   S0          [B][H][dk][dv] fp32    initial state; NULL means zero
 *   o           [B][T][H][dv]  dtype   output, written (never read)
 *   S_T         [B][H][dk][dv] fp32    final state; NULL means not written.
 *                                      May alias S0 (in-place advance).
 *   B, H >= 1; T >= 0 (T = 0 only copies S0, or zeros, into S_T).
 *
 * Decay: any log_alpha <= 0 is accepted, -inf included (alpha = 0: the
 * channel forgets everything before that token).  A chunk whose cumulative
 * decay is mild splits it into growing and shrinking factors around the chunk
 * midpoint; a chunk where that split would leave the fp32 range (strong
 * decay, e.g. log_alpha below about -2.5 held for 32 tokens) is computed in a
 * form whose factors are all decays, at a higher cost for that chunk.
 *
 * Execution (bf16, dk = 128): when the sequences' state chains take at most a
 * quarter of the SMs (see gdn2_fwd_chunked_launches) the call is one
 * cooperative kernel with one CTA on every SM, whose CTAs hand work to one
 * another (each such wait gives up after one second and reports
 * GDN2_ERR_DEVICE_TIMEOUT); it starts once every SM is free, so kernels of
 * other streams delay it or wait for it.  If the device cannot hold that grid
 * the call falls back to the windowed schedule.  There, when the chains take
 * more than half of the SMs, each window of chunks is two kernels on `stream`:
 * the prep, then the chains, which also compute the outputs.  Otherwise it is
 * three kernels per window, with the output kernels on a library-owned side
 * stream that forks from and joins back into `stream`.
 */
gdn2_status gdn2_fwd_chunked(const void *q, const void *k, const void *v,
                             const void *b, const void *w, const float *log_alpha,
                             const float *S0, void *o, float *S_T,
                             int B, int T, int H, int dk, int dv,
                             gdn2_dtype dtype, gdn2_stream_t stream);

/*
 * gdn2_fwd_chunked_noalloc -- gdn2_fwd_chunked without any device allocation.
 *
 * The pages have no counterpart to this entry point; it serves callers that
 * cannot let a library allocate device memory: a runtime that hands out all
 * device memory itself, a hot loop that must never enter the driver's
 * allocator (an allocation can block, or fail on a fragmented heap), or a
 * process that must know its whole device footprint before it starts.
 *
 * Same arguments, layouts, dtypes and results as gdn2_fwd_chunked.  Instead of
 * drawing its workspace from a memory pool, it uses one fixed 32 MiB buffer in
 * the library's device image (held on every GPU that loads the library, until
 * the process exits) and processes the sequence in as many windows as needed
 * to fit it.  A problem whose single chunk of records does not fit (about
 * 185 KiB per (batch, head) pair for dv = 128, so B*H up to 177) returns
 * GDN2_ERR_SCRATCH_LIMIT and launches nothing.
 *
 * The first call on a device looks the buffer's device address up
 * (cudaGetSymbolAddress) with that device current; make that first call
 * before any stream capture.  All calls on one device share that device's
 * buffer: calls whose work overlaps on the GPU (for instance on two streams of
 * the same device) race and corrupt each other's results, so serialize them.
 * Each device has its own copy of the buffer; calls on different devices do
 * not share it.
 * Every byte of the buffer that a call reads, that call writes first, so its
 * leftover contents from earlier calls do not matter.
 */
gdn2_status gdn2_fwd_chunked_noalloc(const void *q, const void *k, const void *v,
                                     const void *b, const void *w, const float *log_alpha,
                                     const float *S0, void *o, float *S_T,
                                     int B, int T, int H, int dk, int dv,
                                     gdn2_dtype dtype, gdn2_stream_t stream);

/*
 * gdn2_decode_step -- one token of the recurrence with the state resident in
 * device memory (recurrent decoding with a fixed-size state instead of a
 * growing cache: gist.science, "Problem Statement"; iplexlaw.co.kr, "De una
 * caché creciente a un estado fijo").
 *
 *   q, k, b     [B][H][dk]      dtype
 *   v, w        [B][H][dv]      dtype
 *   log_alpha   [B][H][dk]      fp32
 *   S           [B][H][dk][dv]  fp32   read and updated in place
 *   o           [B][H][dv]      dtype  written
 *   B, H >= 1.
 *
 * Each state is streamed through the GPU once: read once, written once.
 */
gdn2_status gdn2_decode_step(const void *q, const void *k, const void *v,
                             const void *b, const void *w, const float *log_alpha,
                             float *S, void *o, int B, int H, int dk, int dv,
                             gdn2_dtype dtype, gdn2_stream_t stream);

/*
 * gdn2_decode_tokens -- T consecutive tokens of the recurrence on a state
 * resident in device memory (multi-token decode, or a short prefill into a
 * cached state: the recurrent form with a fixed-size state of gist.science,
 * "Problem Statement").  Equivalent to T calls of gdn2_decode_step, but each
 * state is read and written once per call instead of once per token; meant for
 * T up to a few dozen (longer sequences: gdn2_fwd_chunked).
 *
 *   q, k        [B][T][H][dk]  dtype
 *   v           [B][T][H][dv]  dtype
 *   b           [B][T][H][dk], or [B][T][H] with GDN2_ERASE_SCALAR   dtype
 *   w           [B][T][H][dv], or [B][T][H] with GDN2_WRITE_SCALAR   dtype
 *   log_alpha   [B][T][H][dk], or [B][T][H] with GDN2_DECAY_SCALAR   fp32
 *   S           [B][H][dk][dv] fp32   read and updated in place
 *   o           [B][T][H][dv]  dtype  written
 *   B, H, T >= 1; layout: a combination of gdn2_gate_layout bits.
 */
gdn2_status gdn2_decode_tokens(const void *q, const void *k, const void *v,
                               const void *b, const void *w, const float *log_alpha,
                               float *S, void *o, int B, int T, int H, int dk, int dv,
                               gdn2_dtype dtype, unsigned int layout, gdn2_stream_t stream);

/*
 * gdn2_fwd_chunked_gates -- gdn2_fwd_chunked with a gate layout: b, w and/or
 * log_alpha may be one value per (token, head) ([B][T][H]) as `layout` says.
 * Everything else (arguments, results, execution) is as for gdn2_fwd_chunked,
 * which is this function with layout 0.
 */
gdn2_status gdn2_fwd_chunked_gates(const void *q, const void *k, const void *v,
                                   const void *b, const void *w, const float *log_alpha,
                                   const float *S0, void *o, float *S_T,
                                   int B, int T, int H, int dk, int dv,
                                   gdn2_dtype dtype, unsigned int layout, gdn2_stream_t stream);

/*
 * gdn2_layer_fwd -- the chunked forward with the layer's processing around the
 * operator fused into its kernels ("Gated DeltaNet-2", iplexlaw.co.kr, section
 * "Procesamiento del token y entrenamiento paralelo": queries and keys are
 * L2-normalised, the gates come through sigmoids, and the recurrent output
 * receives RMS normalisation and an independent output gate before the output
 * projection).  The projections, the short convolution and the SiLU stay with
 * the caller.  Per (batch, token, head):
 *
 *     q_hat = q / sqrt(|q|^2 + 1e-6),  k_hat = k / sqrt(|k|^2 + 1e-6)
 *     b = sigmoid(b_logit),  w = sigmoid(w_logit),  log_alpha = log sigmoid(decay_logit)
 *     o, S_T = the operator of gdn2_fwd_chunked on (q_hat, k_hat, v, b, w, log_alpha, S0)
 *     y = o / sqrt(mean_j o_j^2 + eps) * norm_weight * sigmoid(g_logit)
 *
 * The pages name neither the decay's activation nor the output gate's, nor the
 * epsilons: this library reads both activations as the sigmoid the pages give
 * for the erase and write gates.  o never reaches device memory: y is formed
 * from the fp32 accumulators (bf16 inputs, dk = 128) or by a row kernel after
 * the operator (other inputs).
 *
 *   q, k                 [B][T][H][dk]  dtype   before the L2 norm
 *   v                    [B][T][H][dv]  dtype
 *   b_logit              [B][T][H][dk]  dtype
 *   w_logit, g_logit     [B][T][H][dv]  dtype
 *   decay_logit          [B][T][H][dk]  fp32
 *   norm_weight          [dv]           fp32   RMS-norm weight
 *   eps                  >= 0                  RMS-norm epsilon
 *   S0, S_T, B, T, H, dk, dv, dtype, stream    as for gdn2_fwd_chunked
 *   y                    [B][T][H][dv]  dtype   written
 */
gdn2_status gdn2_layer_fwd(const void *q, const void *k, const void *v,
                           const void *b_logit, const void *w_logit, const float *decay_logit,
                           const void *g_logit, const float *norm_weight, float eps,
                           const float *S0, void *y, float *S_T,
                           int B, int T, int H, int dk, int dv,
                           gdn2_dtype dtype, gdn2_stream_t stream);

/*
 * gdn2_bwd_chunked -- the backward of gdn2_fwd_chunked: gradients of
 * L = sum(o * dO) + sum(S_T * dS_T) with respect to every input, chunkwise
 * over 64-token chunks in reverse ("Gated DeltaNet-2", iplexlaw.co.kr, section
 * "Procesamiento del token y entrenamiento paralelo": the WY form's backward
 * must use the modulated keys and values, the per-channel gates staying inside
 * the gradient aggregation).  b and w get gradients of their own, per channel.
 * The forward is recomputed first (its chunk-entry states are the backward's
 * checkpoints, held in a workspace from the library's pool), then the gradient
 * of every chunk's exit state by a reverse pass over the chunks, then the
 * gradients of each chunk, all chunks at once.  Any log_alpha <= 0 is handled:
 * pairwise decays that a split around the chunk midpoint cannot hold are
 * running products of alpha.
 *   bf16 inputs with dk = 128: tensor cores (bf16 operands, fp32 accumulation
 *     and state), within the bf16 tolerance of the forward.  A chunk whose
 *     T = (I + A)^{-1} has an entry off the identity by more than 0.5 (nearly
 *     collinear keys with erase gates near 2) is computed a second time by the
 *     same CTA, with T and X = Z - Ebar S (the chunk's written values less what
 *     its erases read from the entry state) as bf16 pairs (hi + lo), over its
 *     plain gradients; three launches a call;
 *   fp32 inputs, and dk = 64: fp32 on the CUDA cores.
 *
 *   q, k, v, b, w, log_alpha, S0, B, T, H, dk, dv, dtype   as for gdn2_fwd_chunked
 *   dO          [B][T][H][dv]  dtype   incoming gradient of o
 *   dS_T        [B][H][dk][dv] fp32    incoming gradient of S_T; NULL means zero
 *   dq, dk, db, dlog_alpha  [B][T][H][dk]  fp32   written
 *   dv, dw                  [B][T][H][dv]  fp32   written
 *   dS0         [B][H][dk][dv] fp32    written; NULL means not wanted
 *
 * The key-axis gradients are sums over the value columns; one CTA per chunk and
 * head forms each of them in a fixed order, without atomics, so repeated calls
 * give identical bits.
 */
gdn2_status gdn2_bwd_chunked(const void *q, const void *k, const void *v,
                             const void *b, const void *w, const float *log_alpha,
                             const float *S0, const void *dO, const float *dS_T,
                             float *dq, float *dk, float *dv, float *db, float *dw,
                             float *dlog_alpha, float *dS0,
                             int B, int T, int H, int dk_, int dv_,
                             gdn2_dtype dtype, gdn2_stream_t stream);

/*
 * ======================================================================
 * The other operators of a hybrid block: windowed attention with sinks, a
 * diagonal gated linear recurrence, and the norms around a block.  The pages'
 * hybrid model interleaves the operator above with attention over a window of
 * 2K tokens (iplexlaw.co.kr, section "Condiciones de comparacion"; gist.science,
 * architecture).  The recurrence and the norms with their gate and residual
 * scale are not on the pages; they are what else a block of this kind is made
 * of.  All follow the conventions at the top of this header, with one addition:
 * the gradient of an input has the input's own type.
 * ======================================================================
 */

/*
 * gdn2_swa_fwd -- causal attention over a sliding window and a few first tokens
 * that stay visible (sinks), forward over T query tokens.
 *
 * The T queries are the last T of Tk positions: query i stands at position
 * p = Tk - T + i (Tk = T for a whole sequence; Tk > T continues a sequence whose
 * earlier keys are at the front of k and v).  Key j is visible to position p iff
 *     j <= p   and   (p - j < window   or   j < sinks)
 * and, over the visible keys of row i,
 *     o_i = sum_j softmax_j(scale * q_i . k_j) v_j,
 *     lse_i = log sum_j exp(scale * q_i . k_j).
 * Query head h reads key/value head h / (Hq / Hk).
 *
 *   q           [B][T][Hq][d]   dtype
 *   k, v        [B][Tk][Hk][d]  dtype
 *   lens        [B]             int32, device; NULL means T everywhere.  Sequence b
 *               has lens[b] query rows (cut to 0..T); the rows behind them are
 *               padding: o = 0, lse = -infinity.
 *   o           [B][T][Hq][d]   dtype  written
 *   lse         [B][Hq][T]      fp32   written; NULL means not wanted (the backward
 *               needs it)
 *   strides     host array of 9 element strides, {batch, token, head} of q, then of
 *               k, then of v; NULL means dense.  The d elements of a row are always
 *               contiguous; a stride is a multiple of 16 bytes and at least d
 *               (an axis cannot be broadcast).  Strides of an axis of size 1 are
 *               ignored.  Rows of a view may share memory otherwise (windows that
 *               slide over one buffer): each is read as a row of its own, and its
 *               gradient is its own as well.
 *   d 64 or 128; Hq a multiple of Hk; 0 <= T <= Tk <= GDN2_SWA_MAX_TOKENS;
 *   window >= 1; 0 <= sinks; 1e-30 <= scale <= 1e30.
 *
 * A row whose visible scores are all -infinity gives o = 0 and lse = -infinity.
 * What stands in places that a row does not see (keys behind the window or ahead
 * of the row, padding) never reaches that row, infinities and NaN included.
 * bf16 inputs run on the tensor cores (fp32 scores, statistics and sums; the
 * probabilities rounded to bf16 for the product with v); fp32 inputs in fp32 on
 * the CUDA cores.
 */
#define GDN2_SWA_MAX_TOKENS 4194304
gdn2_status gdn2_swa_fwd(const void *q, const void *k, const void *v, const int *lens, void *o, float *lse,
                         int B, int T, int Tk, int Hq, int Hk, int d, int window, int sinks, float scale,
                         const long long *strides, gdn2_dtype dtype, gdn2_stream_t stream);

/*
 * gdn2_swa_bwd -- gradients of sum(o * dO) with respect to q, k and v, from the
 * forward's o and lse.  With P the probabilities and D_i = dO_i . o_i,
 *     dv_j = sum_i P_ij dO_i,   dS_ij = P_ij (dO_i . v_j - D_i),
 *     dq_i = scale * sum_j dS_ij k_j,   dk_j = scale * sum_i dS_ij q_i,
 * sums over i running over the query heads of the group too.
 *
 *   q, k, v, lens, strides, sizes   as for gdn2_swa_fwd
 *   o, dO       [B][T][Hq][d]   dtype  dense
 *   lse         [B][Hq][T]      fp32   of the forward
 *   dq          [B][T][Hq][d]   dtype  written (0 in padding rows)
 *   dk, dv      [B][Tk][Hk][d]  dtype  written (0 where no row sees the key)
 *
 * No atomics: repeated calls give identical bits.  Takes its workspace (D, and
 * the partial sums of the keys that all rows see) from the library's pool.
 */
gdn2_status gdn2_swa_bwd(const void *q, const void *k, const void *v, const void *o, const float *lse,
                         const void *dO, const int *lens, void *dq, void *dk, void *dv,
                         int B, int T, int Tk, int Hq, int Hk, int d, int window, int sinks, float scale,
                         const long long *strides, gdn2_dtype dtype, gdn2_stream_t stream);

/*
 * gdn2_swa_decode -- one token of the windowed attention per sequence, against a
 * cache of fixed size: `sinks` slots for the first tokens, then a ring for the
 * window.  Position p lives in slot p if p < sinks, else in slot
 * sinks + (p - sinks) % (slots - sinks).
 *
 * The call puts k and v into the cache at position pos[b] (as gdn2_decode_step
 * advances its state in place) and then attends from that position.  pos is not
 * advanced.  pos[b] < 0 marks a row of the batch without a sequence: its o is 0
 * and its cache is left as it is.
 *
 *   q, o        [B][Hq][d]           dtype  (o written)
 *   k, v        [B][Hk][d]           dtype  the new token's
 *   k_cache, v_cache  [B][slots][Hk][d]  dtype  updated in place
 *   pos         [B]                  int32, device
 *   strides     host array of 6 element strides, {batch, head} of q, k and v; NULL
 *               means dense.
 *   slots >= sinks + window; the rest as for gdn2_swa_fwd.
 */
gdn2_status gdn2_swa_decode(const void *q, const void *k, const void *v, void *k_cache, void *v_cache,
                            const int *pos, void *o, int B, int slots, int Hq, int Hk, int d, int window, int sinks,
                            float scale, const long long *strides, gdn2_dtype dtype, gdn2_stream_t stream);

/*
 * gdn2_scan_fwd -- the gated linear recurrence: the state update of the gated
 * delta rule without its erase, one value per channel,
 *     h_t = alpha_t h_{t-1} + w_t x_t,   alpha_t = exp(log_alpha_t),   y_t = h_t.
 *
 *   x, w        [B][T][C]  dtype   input and write gate
 *   log_alpha   [B][T][C]  fp32    log of the decay (<= 0; -infinity forgets the state
 *               before that token, if it is finite: 0 times infinity or NaN is NaN)
 *   h0          [B][C]     fp32    initial state; NULL means zero
 *   y           [B][T][C]  dtype   written
 *   h_T         [B][C]     fp32    final state; NULL means not written.  May alias h0.
 *   ckpt        [B][ceil(T / GDN2_SCAN_BLOCK)][C]  fp32  the state entering every
 *               block of GDN2_SCAN_BLOCK tokens, for gdn2_scan_bwd; NULL means not
 *               written.
 *   B, C >= 1; T >= 0 (T = 0 only copies h0, or zeros, into h_T).
 *
 * The state is fp32 throughout.
 */
#define GDN2_SCAN_BLOCK 16
gdn2_status gdn2_scan_fwd(const void *x, const void *w, const float *log_alpha, const float *h0, void *y,
                          float *h_T, float *ckpt, int B, int T, int C, gdn2_dtype dtype, gdn2_stream_t stream);

/*
 * gdn2_scan_bwd -- gradients of sum(y * dy) + sum(h_T * dh_T): with
 * g_t = dy_t + alpha_{t+1} g_{t+1} (and dh_T added at the last token),
 *     dx_t = w_t g_t,   dw_t = x_t g_t,   dlog_alpha_t = g_t alpha_t h_{t-1},
 *     dh0 = alpha_1 g_1.
 *
 *   x, w, log_alpha, B, T, C, dtype   as for gdn2_scan_fwd
 *   ckpt        written by gdn2_scan_fwd on the same inputs; h_{t-1} is recomputed
 *               from it in fp32
 *   dy          [B][T][C]  dtype   incoming gradient of y
 *   dh_T        [B][C]     fp32    incoming gradient of h_T; NULL means zero
 *   dx, dw      [B][T][C]  dtype   written
 *   dlog_alpha  [B][T][C]  fp32    written
 *   dh0         [B][C]     fp32    written; NULL means not wanted
 */
gdn2_status gdn2_scan_bwd(const void *x, const void *w, const float *log_alpha, const float *ckpt, const void *dy,
                          const float *dh_T, void *dx, void *dw, float *dlog_alpha, float *dh0,
                          int B, int T, int C, gdn2_dtype dtype, gdn2_stream_t stream);

/*
 * gdn2_scan_step -- one token of the recurrence, the state updated in place.
 *   x, w, y [B][C] dtype; log_alpha, h [B][C] fp32; y and h written.
 */
gdn2_status gdn2_scan_step(const void *x, const void *w, const float *log_alpha, float *h, void *y,
                           int B, int C, gdn2_dtype dtype, gdn2_stream_t stream);

/*
 * gdn2_block_norm_fwd -- the norms around a block, fused with the block's gate and
 * residual scale: the block's output y is normalised, gated and added to the
 * residual stream r, and the sum is normalised for the next block.  Per row:
 *     r_out = r + res_scale (*) sigmoid(g_logit) (*) (y / rms(y)) (*) w_post
 *     x_out = (r_out / rms(r_out)) (*) w_pre          rms(a) = sqrt(mean(a^2) + eps)
 * x_out is formed from r_out before its rounding.  Sums of squares are fp32: they hold
 * for rows whose elements stay below about 1e17.
 *
 *   r, y        [N][D]  dtype   residual stream, block output
 *   g_logit     [N][D]  dtype   gate logits; NULL means no gate (sigmoid -> 1)
 *   w_post, res_scale, w_pre  [D]  fp32
 *   eps         >= 0, finite
 *   r_out, x_out  [N][D]  dtype  written; r_out may alias r
 *   N >= 0; 1 <= D <= 16384.
 */
gdn2_status gdn2_block_norm_fwd(const void *r, const void *y, const void *g_logit, const float *w_post,
                                const float *res_scale, const float *w_pre, float eps, void *r_out, void *x_out,
                                long long N, int D, gdn2_dtype dtype, gdn2_stream_t stream);

/*
 * gdn2_block_norm_bwd -- gradients of sum(r_out * dr_out) + sum(x_out * dx_out).  The
 * forward's inputs are read again and its rows recomputed (as many bytes as reading
 * r_out instead, and no rounding between).
 *
 *   r .. eps, N, D, dtype   as for gdn2_block_norm_fwd
 *   dr_out, dx_out          [N][D]  dtype  incoming gradients
 *   dr, dy, dg_logit        [N][D]  dtype  written; dr may alias dr_out; dg_logit is NULL
 *                           exactly when g_logit is
 *   dw_post, dres_scale, dw_pre  [D]  fp32  written: sums over the rows, in a fixed order
 *                           (no atomics: repeated calls give identical bits)
 * Takes its workspace (partial sums) from the library's pool.
 */
gdn2_status gdn2_block_norm_bwd(const void *r, const void *y, const void *g_logit, const float *w_post,
                                const float *res_scale, const float *w_pre, float eps, const void *dr_out,
                                const void *dx_out, void *dr, void *dy, void *dg_logit, float *dw_post,
                                float *dres_scale, float *dw_pre, long long N, int D, gdn2_dtype dtype,
                                gdn2_stream_t stream);

/*
 * gdn2_check_device_error -- wait for `stream`, then read and clear the
 * device error word of the current device.  Returns GDN2_OK,
 * GDN2_ERR_DEVICE_TIMEOUT or GDN2_ERR_CUDA.
 */
gdn2_status gdn2_check_device_error(gdn2_stream_t stream);

/*
 * gdn2_fwd_chunked_launches -- number of kernel launches one gdn2_fwd_chunked
 * call on the current device makes for this problem (-1 for arguments
 * gdn2_fwd_chunked would reject).  The bf16 path launches one persistent
 * kernel when the sequences' chains (batch * heads * dv / 64 CTAs) take at
 * most a quarter of the SMs, else
 * per window of chunks two kernels (chains on more than half of the SMs) or
 * three, the window size depending on the device's SM count, which is the only thing this
 * queries (without a device it plans for 148 SMs); the fp32 path launches one
 * kernel.  A zeroing memset of a few kilobytes of flags precedes the persistent
 * kernel and is not counted.
 */
int gdn2_fwd_chunked_launches(int B, int T, int H, int dk, int dv, gdn2_dtype dtype);

/*
 * gdn2_selftest_bounded_wait -- queue on `stream` a one-warp kernel that waits
 * for a device flag nothing sets, with the bounded wait the persistent forward
 * uses between its CTAs.  The wait gives up after one second and records
 * GDN2_ERR_DEVICE_TIMEOUT in the device error word, so the next
 * gdn2_check_device_error(stream) returns it, and the context stays usable.
 * Returns GDN2_OK once queued (GDN2_ERR_CUDA if queuing failed).
 */
gdn2_status gdn2_selftest_bounded_wait(gdn2_stream_t stream);

/* Human-readable name of a status code (static storage, never NULL). */
const char *gdn2_status_string(gdn2_status status);

#ifdef __cplusplus
}
#endif

#endif /* GDN2_H */

/*
 * tfl.h -- C ABI of the GB300 (sm_103a) Transformer-stack forward.
 *
 * What it computes (the forward pass of a fixed L-layer Transformer block
 * stack, "TikTok TechJam 2026 -- Problem 3: GPU Transformer Optimization",
 * section 1.A and section 2):
 *
 *   h = x
 *   for each layer l:
 *     a = LN1_l(h)                                   (pre-LN, the default)
 *     [q | k | v] = a [Wq; Wk; Wv]^T + [bq; bk; bv]  (fused QKV, section 2.2)
 *     o = softmax(q k^T / sqrt(hd) + mask) v         (per head, section 2.1)
 *     h = h + o Wo^T + bo ;  a2 = LN2_l(h)
 *     h = h + GELU(a2 W1^T + b1) W2^T + b2           (exact erf GELU, 2.3)
 *   out = LN_f(h), rows at padded positions set to 0 (section 1.A tail)
 *
 * mask: right-padded keys, key j of sequence b is valid iff j < len_b
 * (section 2.1, "the mask trick"); with causal, key j is visible to query i
 * iff j <= i, and the key mask is then redundant for every valid query.
 * With norm_placement = 1 (post-LN): h = LN1(h + attn(h)),
 * h = LN2(h + FFN(h)), out = LN_f(h) masked.
 *
 * Numerics: fp16 tensor-core operands with fp32 accumulation; residual
 * stream, LayerNorm statistics and softmax in fp32 ("Transformerkernel",
 * How we built it).  Output is fp32.
 *
 * Threading: a handle is not thread-safe; distinct handles are independent.
 * All device pointers must belong to the device that was current when the
 * handle was created.
 */
#ifndef TFL_H_
#define TFL_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Return codes.  Every int-returning entry point returns one of these. */
#define TFL_OK                   0
#define TFL_ERR_INVALID_ARG     -1  /* null pointer, non-positive size, aliasing */
#define TFL_ERR_UNSUPPORTED     -2  /* not sm_103, or a shape the kernels do not cover */
#define TFL_ERR_OOM             -3  /* device allocation failed or exceeds max_workspace_bytes */
#define TFL_ERR_CUDA            -4  /* a CUDA runtime call failed (see tfl_last_error) */
#define TFL_ERR_DEVICE_TIMEOUT  -5  /* a kernel's bounded wait ran out; its outputs are invalid */
#define TFL_ERR_BAD_LENGTHS     -6  /* a length was outside [0, S]; it was clamped */

/* Opaque handle: packed weights, workspace, captured graphs. */
typedef struct tfl_handle tfl_handle;

/* A cudaStream_t passed as an opaque pointer (NULL = legacy default stream). */
typedef void* tfl_stream;

/*
 * Shape of the stack (the dispatch key of "Shape-specialized Transformer
 * Inference on Commodity GPUs", What it does: batch, seq_len, d_model,
 * n_heads, d_ff, n_layers).
 * Supported: B, S >= 1; d_model and d_ff multiples of 128; head_dim =
 * d_model / n_heads in {32, 64, 256}; n_layers >= 1; B*S*max(3*d_model,
 * d_ff) < 2^31.  norm_placement: 0 = pre-LN (default), 1 = post-LN.
 */
typedef struct {
    int32_t B, S, d_model, n_heads, d_ff, n_layers;
    int32_t norm_placement;
} tfl_shape;

/*
 * One layer's parameters: float32, nn.Linear layout ([out, in], row-major,
 * "in" contiguous).  wq, wk, wv, wo: [d_model, d_model]; w1: [d_ff, d_model];
 * w2: [d_model, d_ff]; bq, bk, bv, bo, b2, ln*_g, ln*_b: [d_model]; b1: [d_ff].
 * Pointers may be host or device memory (read once by tfl_create).
 */
typedef struct {
    const float *wq, *bq, *wk, *bk, *wv, *bv, *wo, *bo;
    const float *ln1_g, *ln1_b, *ln2_g, *ln2_b;
    const float *w1, *b1, *w2, *b2;
} tfl_layer_weights;

typedef struct {
    const tfl_layer_weights* layers;   /* n_layers entries */
    int32_t n_layers;                  /* must equal shape->n_layers */
    const float *lnf_g, *lnf_b;        /* final LayerNorm, [d_model] */
} tfl_weights;

/*
 * precision: how GEMM operands are carried into the fp16 tensor cores (fp32
 * accumulation always).  x = hi + lo with lo = fp16(x - hi) is a "split":
 *   0  every operand rounded once to fp16 (fastest; too coarse for the graded
 *      rule over many seeds)
 *   1  weights split (two MMAs per k-step)
 *   2  weights split, and the GEMM activations (normed rows, GELU output)
 *      split too (three MMAs per k-step; the default)
 * fp8_corrections (precision 2, d_model > 128): the two correction terms of a
 *   split product, A_lo W_hi and A_hi W_lo, run as e4m3 MMAs (kind::f8f6f4,
 *   twice the fp16 rate) on e4m3 copies of the hi parts and of the lo parts
 *   times 2^11, beside the fp16 A_hi W_hi; a k-step then costs two fp16 MMAs'
 *   time instead of three.  1 (default) on, 0: fp16 lo planes as at d_model 128.
 */
typedef struct {
    int32_t precision;            /* 0, 1 or 2 (default 2), see above */
    float ln_eps;                 /* LayerNorm eps, default 1e-5 */
    int64_t wait_timeout_ns;      /* bound on every device-side wait, default 2e9 */
    int64_t max_workspace_bytes;  /* 0 = unlimited */
    int32_t use_graph;            /* 1 (default): replay the forward as one CUDA graph */
    int32_t whole_stack;          /* 1 (default): run every layer in one kernel where the
                                     shape allows it (d_model 128, head_dim 32, S <= 128,
                                     precision 2, d_ff <= 2048, n_layers <= 8); 0: per-layer kernels */
    int32_t fp8_corrections;      /* 1 (default) or 0, see above */
} tfl_options;

/* Fill *opt with the defaults above.  Returns TFL_OK or TFL_ERR_INVALID_ARG. */
int tfl_default_options(tfl_options* opt);

/* Bytes of device workspace tfl_create will allocate for this shape at the
 * default precision (0 if the shape is invalid). */
size_t tfl_workspace_bytes(const tfl_shape* shape);

/*
 * Validate the shape, check the current device is sm_103, allocate the
 * workspace (one allocation), pack the weights to fp16 K-major (W_qkv =
 * [Wq; Wk; Wv] rows, "TikTok TechJam 2026 -- Problem 3", section 2.2) and
 * build the TMA descriptors.  The caller may free its weights afterwards.
 * opt may be NULL (defaults).  On success *out owns all of that.
 * Synchronous.  Errors: INVALID_ARG, UNSUPPORTED, OOM, CUDA.
 */
int tfl_create(const tfl_shape* shape, const tfl_weights* w,
               const tfl_options* opt, tfl_handle** out);

/*
 * Run the forward on `stream`, asynchronously.
 *   x:       device float32 [B, S, d_model], read only (padded rows are never read).
 *   lengths: device int32 [B] or NULL (every sequence has length S); values
 *            are clamped to [0, S] on the device, and an out-of-range value
 *            makes the next tfl_status return TFL_ERR_BAD_LENGTHS.
 *   causal:  0 or 1.
 *   out:     device float32 [B, S, d_model], written in full (padded rows = 0);
 *            must not overlap x.
 * The first call for a given (causal, x, lengths, out) captures the launch
 * sequence as a CUDA graph (not allowed while `stream` is itself capturing
 * unless use_graph = 0); later calls replay it.
 * Errors: INVALID_ARG, CUDA.  Device-side errors surface via tfl_status.
 */
int tfl_forward(tfl_handle* h, const float* x, const int32_t* lengths,
                int causal, float* out, tfl_stream stream);

/*
 * The same forward with the model's inputs and outputs in bf16 (the model
 * dtype of a bf16 checkpoint): x and out are device bf16 [B, S, d_model]
 * (2 bytes per value, 16-byte aligned, not overlapping).  x is widened to fp32
 * as it is read; the residual stream, LayerNorms, softmax and accumulation stay
 * fp32 exactly as in tfl_forward; the final LayerNorm's output is rounded to
 * bf16 (nearest even) as it is written, padded rows as +0.
 * ("TikTok TechJam 2026 -- Problem 3", section 2.3, falls back to its baseline
 * at bf16.)
 * Graphs are cached per (causal, x, lengths, out) as for tfl_forward.
 * Errors: INVALID_ARG, CUDA.  Device-side errors surface via tfl_status.
 */
int tfl_forward_bf16(tfl_handle* h, const void* x, const int32_t* lengths,
                     int causal, void* out, tfl_stream stream);

/*
 * The same forward from host buffers, synchronizing `stream` before it returns.
 * If x and out are pinned host memory the device can address (cudaHostAlloc /
 * cudaHostRegister, mapped), 16-byte aligned and not overlapping, the kernels
 * read x and write out across the host link directly (the input row kernel
 * keeps a device copy of x as the first residual) and only the lengths are
 * copied.  Otherwise (pageable buffers) x and lengths are copied to
 * handle-owned device buffers, tfl_forward runs and out is copied back.
 * Allocates its device buffers on the first call.
 * Returns what tfl_status returns after the run.
 */
int tfl_forward_host(tfl_handle* h, const float* x_host, const int32_t* lengths_host,
                     int causal, float* out_host, tfl_stream stream);

/*
 * The forward of a batch held in host memory, streamed through the device in
 * slices of the handle's batch size B ("Shape-specialized Transformer
 * Inference on Commodity GPUs", How we built it: the S = 100000 case runs with
 * its input in host RAM, batch slices streaming through the device and the
 * outputs streaming back; its stream loop ran copies and compute one after
 * the other, here they overlap).
 *   x_host:       pinned host float32 [n_seq, S, d_model] (cudaHostAlloc /
 *                 cudaHostRegister; pageable memory is rejected)
 *   lengths_host: host int32 [n_seq] or NULL (every sequence has length S);
 *                 read during the call; a value outside [0, S] is rejected
 *   n_seq:        any number >= 1 of sequences; the last slice may be partial
 *   out_host:     pinned host float32 [n_seq, S, d_model], written in full
 *                 (padded rows = 0); must not overlap x_host
 * Slice k (sequences k*B .. k*B+B-1) is copied in while slice k-1 computes and
 * slice k-2's output is copied back, through two device buffers each for x
 * and out, so the device holds B sequences' workspace and four slice buffers
 * whatever n_seq is.  Asynchronous on `stream` (its earlier work runs first;
 * its later work waits for the whole batch); synchronize or call tfl_status
 * before reading out_host.  Allocates its device buffers (and a pinned
 * lengths staging area) on the first call, and again when n_seq grows; a call
 * first waits for the previous streamed call of the handle to finish with that
 * staging area.  Errors: INVALID_ARG, OOM, CUDA; device-side errors surface
 * via tfl_status.
 */
int tfl_forward_streamed(tfl_handle* h, const float* x_host, const int32_t* lengths_host, int64_t n_seq,
                         int causal, float* out_host, tfl_stream stream);

/*
 * Synchronize `stream` and read (then clear) the device status word.
 * Returns TFL_OK, TFL_ERR_DEVICE_TIMEOUT or TFL_ERR_BAD_LENGTHS (timeout
 * wins), or TFL_ERR_CUDA.
 */
int tfl_status(tfl_handle* h, tfl_stream stream);

/* Free everything the handle owns.  Synchronizes the device.  NULL is a no-op. */
void tfl_destroy(tfl_handle* h);

/* Message of the last error on this thread ("" if none).  Valid until the next call. */
const char* tfl_last_error(void);

/*
 * Eager forward (no graph) with a CUDA event around every launch, for
 * profiling.  Writes up to `cap` entries: kernel_ms[i] = device time of
 * launch i, kernel_kind[i] = TFL_KIND_* of that launch; *n = the timed launches: all of
 * tfl_forward's launches but the length check of the per-layer path (the whole-stack
 * kernel checks the lengths itself and is the one launch).  Synchronizes `stream`.
 */
#define TFL_KIND_ROWNORM   1
#define TFL_KIND_GEMM_QKV  2
#define TFL_KIND_ATTENTION 3
#define TFL_KIND_GEMM_OPROJ 4
#define TFL_KIND_GEMM_FFN1 5
#define TFL_KIND_GEMM_FFN2 6
#define TFL_KIND_POSTCHAIN 7   /* d_model 128: o_proj .. FFN-out .. next LayerNorm fused */
#define TFL_KIND_STACK     8   /* whole_stack: every layer of the forward in one kernel */
int tfl_profile_forward(tfl_handle* h, const float* x, const int32_t* lengths,
                        int causal, float* out, tfl_stream stream,
                        float* kernel_ms, int32_t* kernel_kind, int32_t cap, int32_t* n);

/*
 * Self-test of the epilogues' GELU (exact-erf form evaluated with erf from
 * Abramowitz & Stegun 7.1.26), both the scalar form and the packed fp32-pair
 * form: writes the largest |difference| from a GELU built on CUDA's erff over
 * n >= 2 points evenly spaced on [-12, 12].
 * Synchronizes `stream`.  Errors: INVALID_ARG, CUDA.
 */
int tfl_selftest_gelu(int32_t n, float* max_abs_diff, tfl_stream stream);

/*
 * Which kernel a launch of the gated feed-forward (below) takes, by the rule the
 * calls themselves use, so that tests can show that they reach each one.  Host
 * only.
 *   part   0 the forward; 1, 2, 3 the backward's slopes, dx and weight gradients
 *   units  what the device runs at once: CTAs with all of an SM's shared memory,
 *          pairs of them, clusters of 2, 4 and 8; NULL: asked of the current device
 *   out    a TFL_GLU_FORM_*, output columns of a tile, tiles, tiles at once (0s
 *          after the form for the few-token kernel)
 * Errors: INVALID_ARG, and without `units` UNSUPPORTED, CUDA.
 */
#define TFL_GLU_FORM_FEW    0   /* a few tokens, weights straight into MMA fragments */
#define TFL_GLU_FORM_LONE   1   /* lone CTAs */
#define TFL_GLU_FORM_SHARED 2   /* clusters of lone CTAs that share a tile's sum */
#define TFL_GLU_FORM_PAIR   3   /* CTA pairs, tiles narrower than the accumulator */
#define TFL_GLU_FORM_WIDE   4   /* CTA pairs, tiles as wide as it */
int tfl_selftest_glu_plan(int32_t d_model, int32_t d_ff, int32_t in_type, int32_t part, int64_t tokens,
                          const int32_t* units, int32_t* out);

/* Number of kernel launches one tfl_forward makes for this handle and causal flag. */
int tfl_launch_count(const tfl_handle* h, int causal);

/*
 * Self-test of the device-side bounded wait: launches one block that waits
 * on an mbarrier nothing will complete, with the given bound.  Returns
 * TFL_ERR_DEVICE_TIMEOUT when the bound ran out as it should (the context
 * stays usable), TFL_ERR_CUDA on a launch error.  Synchronizes `stream`.
 */
int tfl_probe_wait_timeout(int64_t timeout_ns, tfl_stream stream);

/*
 * tfl_forward_noalloc -- the forward for callers that cannot allocate device
 * memory when they run it.
 *
 * Who needs it: code that runs the forward where cudaMalloc is off limits --
 * for instance inside another component's CUDA-graph capture (allocation and
 * graph instantiation are not allowed while a capture is open), under a host
 * framework whose memory pool owns the device budget, or in a latency-critical
 * loop that must never hit the allocator's implicit synchronisation.
 * tfl_forward needs no allocation once warm, but its first call per buffer set
 * instantiates a CUDA graph; tfl_forward_host allocates staging buffers.  This
 * entry point does neither: it enqueues the same kernels eagerly on `stream`.
 *
 * This is an addition of this library; the pages describe no counterpart.
 *
 * Arguments, layouts and errors are those of tfl_forward (the handle supplies
 * the packed weights and the status word read by tfl_status).  Every
 * intermediate of the forward -- residual stream, normed rows, qkv, attention
 * output, FFN activations, attention work counters -- lives in one fixed
 * device array inside the library, TFL_NOALLOC_SCRATCH_BYTES (32 MiB) on each
 * GPU that loads the library, held until the process exits.  A shape whose
 * intermediates do not fit is rejected with TFL_ERR_UNSUPPORTED and a message
 * naming both sizes.  The intermediates take the handle's workspace layout:
 * per token 4 d_model (residual) + 2 d_model (normed rows) + 6 d_model (q, k, v)
 * + 2 d_model (attention output) + 2 d_ff (FFN activations) bytes, plus 2
 * d_model + 2 d_ff more at precision 2 (the lo planes), plus a few KiB; at
 * d_model 128, d_ff 512, precision 2 that is 4 KiB per token, so at most about
 * 8190 tokens (B * S) fit.  tfl_workspace_bytes(shape) gives that size at
 * precision 2.
 *
 * The first call on a device looks up the array's device address (one
 * cudaGetSymbolAddress with that device current); make that first call before
 * any stream capture.  All calls, on every handle and stream of a device,
 * share the array and it keeps the last call's contents: calls that overlap
 * on the GPU race and corrupt each other, so serialize them (one stream, or
 * events).  Each call clears the part of the array it uses (a memset on
 * `stream`) before its kernels run.  The handle is used only on the host
 * during the call (not thread-safe with other calls on the same handle).
 */
#define TFL_NOALLOC_SCRATCH_BYTES ((size_t)32 << 20)
int tfl_forward_noalloc(tfl_handle* h, const float* x, const int32_t* lengths,
                        int causal, float* out, tfl_stream stream);

/*
 * Attention on its own, forward and backward, for training use ("Training
 * throughput baseline", Fused attention: the forward keeps the row
 * log-sum-exp; the backward rebuilds the probabilities from it and takes the
 * softmax row sum from the output gradient and the output, in one kernel per
 * query tile (dQ) and one per key tile (dK, dV), without atomics).
 *
 * Per sequence b and head h (columns h*hd .. h*hd+hd-1 of q, k and v):
 *   O = softmax(Q K^T / sqrt(hd) + mask) V, key j visible to query i iff
 *   j < len_b and (not causal or j <= i).
 * Layouts (device memory, row-major):
 *   qkv   fp16 [B, S, 3 H hd]: q | k | v, as the fused QKV projection writes it;
 *         rows at or past len_b must hold finite values (masked keys are
 *         multiplied by a zero probability)
 *   o     fp16 [B, S, H hd]          lse  fp32 [B, H, S], log2 units:
 *         lse = log2 sum_j 2^(q.k_j log2(e) / sqrt(hd)) (natural LSE * log2(e))
 *   dout  fp16 [B, S, H hd]          dqkv fp32 [B, S, 3 H hd]: dq | dk | dv
 * Query rows at or past len_b are padding: their o and lse are unspecified,
 * their dout is ignored, their dq is 0 and they add nothing to dk and dv.
 * All buffers 16-byte aligned.  Asynchronous on `stream`; device-side errors
 * (a bounded wait that ran out, a length outside [0, S]) surface through
 * tfl_attn_status.  A handle is not thread-safe.
 */
typedef struct tfl_attn tfl_attn;

/* head_dim 32 or 64 (the backward's range; the forward also takes 256);
 * B, S, n_heads >= 1.  Allocates the handle's status word, work counter and
 * the backward's row-sum scratch (B * n_heads * S floats).
 * Errors: INVALID_ARG, UNSUPPORTED, OOM, CUDA. */
int tfl_attn_create(int32_t B, int32_t S, int32_t n_heads, int32_t head_dim, tfl_attn** out);

/* o and lse from qkv (lengths: device int32 [B] or NULL = all S). */
int tfl_attn_forward(tfl_attn* a, const void* qkv, const int32_t* lengths, int causal, void* o, float* lse,
                     tfl_stream stream);

/* dqkv from qkv, the forward's o and lse, and dout.  dqkv is cleared first, so
 * padding rows read 0. */
int tfl_attn_backward(tfl_attn* a, const void* qkv, const void* o, const void* dout, const float* lse,
                      const int32_t* lengths, int causal, float* dqkv, tfl_stream stream);

/* Synchronize `stream`, read and clear the status word: TFL_OK,
 * TFL_ERR_DEVICE_TIMEOUT or TFL_ERR_BAD_LENGTHS. */
int tfl_attn_status(tfl_attn* a, tfl_stream stream);

void tfl_attn_destroy(tfl_attn* a);

/*
 * The rest of a block on its own, beside the attention above: the
 * root-mean-square norm in front of a sublayer and the gated feed-forward
 * ("Training throughput baseline" trains a model of such blocks).
 *
 * Element types of these operators.
 */
#define TFL_F32  0
#define TFL_F16  1
#define TFL_BF16 2
#define TFL_E4M3 3   /* 8 bits: 4 exponent, 3 mantissa, largest value 448 */

/*
 * Root-mean-square norm with the residual's addition:
 *   s = x + res,   r = 1 / sqrt(mean(s^2) + eps),   y = s r gamma   (per row)
 * s, the sums and y are fp32 inside; res_out is s and y is y, each rounded once
 * to its type (y is taken from the unrounded s).  mean(s^2) + eps has to lie
 * within fp32's normal range, 1.2e-38 to 3.4e38: with eps 0, rows of an rms
 * between 1.1e-19 and 1.8e19 (a row of zeros has no norm then).
 *
 * e4m3 output: y_scale[row] = max(max|y|, 2^-100) / 448 and y holds
 * e4m3(y / y_scale[row]), so y_scale[row] times the stored value is the norm's
 * output; a row with a NaN has a NaN scale.
 *
 * Types: x fp32, fp16 or bf16; the residual fp32 or x's type; y x's type or
 * e4m3, and for fp32 x also fp16 or bf16.  gamma is fp32.
 */
typedef struct tfl_rmsnorm tfl_rmsnorm;

/* d_model in 1 .. 2^24, eps >= 0 and finite.  Where y is of x's type the handle also holds the
 * backward's scratch (at most max(64 MiB, 4 d_model bytes)).
 * Errors: INVALID_ARG, UNSUPPORTED (types, device), OOM, CUDA. */
int tfl_rmsnorm_create(int32_t d_model, int32_t x_type, int32_t res_type, int32_t y_type, float eps,
                       tfl_rmsnorm** out);

/*
 * Asynchronous on `stream`.  Device pointers, rows of d_model values one after
 * the other, 0 <= rows < 2^31 (0: nothing is done):
 *   x        [rows, d_model]
 *   res      [rows, d_model] of the residual's type, or NULL (s = x)
 *   gamma    fp32 [d_model]
 *   res_out  [rows, d_model] of the residual's type, or NULL (s is not stored);
 *            may be res, or x when the types are the same
 *   y        [rows, d_model]; may be x when the types are the same (and res_out is not x)
 *   y_scale  fp32 [rows] for an e4m3 y, else NULL
 * Other overlaps of an output are refused.  Any element-aligned buffers and
 * widths; 16-byte aligned buffers (y: 8 bytes for e4m3) and a d_model that is a
 * multiple of 8 up to 32768 take the kernels that keep a row in registers.
 * Calls on one handle may overlap.
 * Errors: INVALID_ARG (also when the current device is not the handle's), CUDA.
 */
int tfl_rmsnorm_forward(tfl_rmsnorm* n, int64_t rows, const void* x, const void* res, const float* gamma,
                        void* res_out, void* y, float* y_scale, tfl_stream stream);

/*
 * The gradients, with a = dy gamma and r as above (recomputed from s):
 *   ds = dres + r a - s r^3 mean(a s),   dgamma = sum over rows of dy s r
 *   sum     [rows, d_model] of the residual's type: the forward's res_out (x if it had no residual)
 *   dy      [rows, d_model] of y's type (which must be x's type)
 *   dres    [rows, d_model] of the residual's type: the gradient that reaches s past the norm, or NULL
 *   dx      ds in x's type, or NULL;  dsum  ds in the residual's type, or NULL
 *           (s = x + res, so ds is the gradient of both; at least one is given)
 *   dgamma  fp32 [d_model], written in full (zeros for rows = 0)
 * dx or dsum may be dy, dres or sum where the types are the same; other overlaps
 * are refused.  No atomics: the same inputs give the same bits.  Calls on one
 * handle share its scratch and must not overlap on the GPU (graphs that hold such
 * calls included).  Errors: INVALID_ARG, UNSUPPORTED (y is not of x's type), CUDA.
 */
int tfl_rmsnorm_backward(tfl_rmsnorm* n, int64_t rows, const void* sum, const float* gamma, const void* dy,
                         const void* dres, void* dx, void* dsum, float* dgamma, tfl_stream stream);

/* Free what the handle owns.  Synchronizes the device.  NULL is a no-op. */
void tfl_rmsnorm_destroy(tfl_rmsnorm* n);

/*
 * Layer norm with the residual's addition, the norm of the stack above on its own:
 *   s = x + res,  m = mean(s),  r = 1 / sqrt(mean((s - m)^2) + eps),
 *   t = (s - m) r,  y = t gamma + beta   (per row)
 * s, the sums and y are fp32 inside; res_out is s and y is y, each rounded once
 * to its type (y is taken from the unrounded s).  The variance is the centred
 * values' own, so a large mean costs only what fp32 loses of s - m.
 * var + eps has to lie within fp32's normal range (with eps 0 a constant row has
 * no norm), and the sum of a row's |s| below its largest value.  e4m3 output and
 * types: as for the root-mean-square norm above.
 */
typedef struct tfl_layernorm tfl_layernorm;

/* d_model in 1 .. 2^24, eps >= 0 and finite.  Where y is of x's type the handle also holds the
 * backward's scratch (at most max(64 MiB, 8 d_model bytes)).
 * Errors: INVALID_ARG, UNSUPPORTED (types, device), OOM, CUDA. */
int tfl_layernorm_create(int32_t d_model, int32_t x_type, int32_t res_type, int32_t y_type, float eps,
                         tfl_layernorm** out);

/*
 * Asynchronous on `stream`.  Device pointers, rows of d_model values one after
 * the other, 0 <= rows < 2^31 (0: nothing is done):
 *   x        [rows, d_model]
 *   res      [rows, d_model] of the residual's type, or NULL (s = x)
 *   gamma    fp32 [d_model];  beta  fp32 [d_model], or NULL (0)
 *   res_out  [rows, d_model] of the residual's type, or NULL (s is not stored);
 *            may be res, or x when the types are the same
 *   y        [rows, d_model]; may be x when the types are the same (and res_out is not x)
 *   y_scale  fp32 [rows] for an e4m3 y, else NULL
 *   stats    fp32 [rows, 2], 8-byte aligned: m and r of each row, which the
 *            backward takes; or NULL (not stored)
 * Other overlaps of an output are refused.  Any element-aligned buffers and
 * widths; 16-byte aligned buffers (y: 8 bytes for e4m3) and a d_model that is a
 * multiple of 8 up to 32768, or many rows of any other up to 8178, take the kernels
 * that move a row in 16-byte vectors.
 * Calls on one handle may overlap.
 * Errors: INVALID_ARG (also when the current device is not the handle's), CUDA.
 */
int tfl_layernorm_forward(tfl_layernorm* n, int64_t rows, const void* x, const void* res, const float* gamma,
                          const float* beta, void* res_out, void* y, float* y_scale, float* stats, tfl_stream stream);

/*
 * The gradients, with a = dy gamma and t = (s - m) r from the forward's m and r:
 *   ds = dres + r (a - mean(a) - t mean(a t)),   dgamma = sum over rows of dy t,   dbeta = sum over rows of dy
 *   sum     [rows, d_model] of the residual's type: the forward's res_out (x if it had no residual)
 *   stats   fp32 [rows, 2], 8-byte aligned: as the forward stored them
 *   dy      [rows, d_model] of y's type (which must be x's type)
 *   dres    [rows, d_model] of the residual's type: the gradient that reaches s past the norm, or NULL
 *   dx      ds in x's type, or NULL;  dsum  ds in the residual's type, or NULL
 *           (s = x + res, so ds is the gradient of both; at least one is given)
 *   dgamma  fp32 [d_model], written in full (zeros for rows = 0);  dbeta  the same, or NULL
 * dx or dsum may be dy, dres or sum where the types are the same; other overlaps
 * are refused.  No atomics: the same inputs give the same bits.  Calls on one
 * handle share its scratch and must not overlap on the GPU (graphs that hold such
 * calls included).  Errors: INVALID_ARG, UNSUPPORTED (y is not of x's type), CUDA.
 */
int tfl_layernorm_backward(tfl_layernorm* n, int64_t rows, const void* sum, const float* stats, const float* gamma,
                           const void* dy, const void* dres, void* dx, void* dsum, float* dgamma, float* dbeta,
                           tfl_stream stream);

/* Free what the handle owns.  Synchronizes the device.  NULL is a no-op. */
void tfl_layernorm_destroy(tfl_layernorm* n);

/*
 * Which kernel a call of the layer norm takes, by the rule the calls themselves use,
 * so that tests can show that they reach each one.  Host only.
 *   part     0 the forward, 1 the backward
 *   aligned  whether every buffer is 16-byte aligned, else none is
 *   sms      of the device; 0: asked of the current one
 *   out      a TFL_LN_FORM_*, and for the forms in vectors the threads of a block (at
 *            most) and a thread's vectors of a row (else 0s)
 * Errors: INVALID_ARG, and without `sms` UNSUPPORTED, CUDA.
 */
#define TFL_LN_FORM_VECTORS  0   /* rows that are whole 16-byte vectors */
#define TFL_LN_FORM_STRADDLE 1   /* rows that begin inside one, in vectors all the same */
#define TFL_LN_FORM_VALUES   2   /* a value at a time, a row in registers */
#define TFL_LN_FORM_ANY      3   /* a value at a time, a row read several times */
int tfl_selftest_layernorm_plan(int32_t d_model, int32_t res_type, int32_t part, int64_t rows, int32_t aligned,
                                int32_t sms, int32_t* out);

/*
 * Gated feed-forward block: both projections, the activation and the product
 *   h = act(x Wg^T) * (x Wu^T)
 * with Wg, Wu in nn.Linear layout [d_ff, d_model] (one packed [2 d_ff, d_model]
 * weight is passed as its two halves).  Products accumulate in fp32 and h is
 * rounded once.
 *
 * Operands (x, Wg, Wu): fp16 or bf16, the output's type; or e4m3 with one fp32
 * scale a row (the stored value times its row's scale is the operand's value,
 * as tfl_rmsnorm_forward writes x), and an fp16 or bf16 output.
 */
#define TFL_ACT_SILU 0   /* z / (1 + e^-z) */
#define TFL_ACT_GELU 1   /* z Phi(z), the exact erf form (Phi to 7.5e-8 absolute) */
#define TFL_ACT_NONE 2   /* z: the linear layer below only */
typedef struct tfl_glu tfl_glu;

/* d_model and d_ff: multiples of 8 (16 for e4m3 operands) up to 2^24.
 * max_grad_tokens: the most tokens tfl_glu_backward will be given (0: no
 * backward; e4m3 operands have none); the handle holds 4 max_grad_tokens d_ff
 * bytes of scratch for it (d_ff to the next multiple of 64).  Errors: INVALID_ARG, UNSUPPORTED, OOM, CUDA. */
int tfl_glu_create(int32_t d_model, int32_t d_ff, int32_t in_type, int32_t out_type, int32_t act,
                   int64_t max_grad_tokens, tfl_glu** out);

/*
 * Asynchronous on `stream`.  Device pointers, 16-byte aligned, row-major and
 * contiguous; any number of tokens from 0 (nothing is done):
 *   x [tokens, d_model], wg and wu [d_ff, d_model], h [tokens, d_ff]
 *   x_scale fp32 [tokens] (4-byte aligned), wg_scale and wu_scale fp32 [d_ff]
 *   for e4m3 operands, else NULL
 * h must not overlap an input.  Rows do not affect one another.  Calls on one
 * handle may overlap.  Errors: INVALID_ARG (also when the current device is not
 * the handle's), UNSUPPORTED, CUDA; a device-side wait that ran out surfaces
 * through tfl_glu_status.
 */
int tfl_glu_forward(tfl_glu* g, int64_t tokens, const void* x, const float* x_scale, const void* wg,
                    const float* wg_scale, const void* wu, const float* wu_scale, void* h, tfl_stream stream);

/*
 * The gradients, from the forward's inputs (its products are computed again, so
 * nothing is kept between the two calls) and dh [tokens, d_ff]:
 *   dg = dh u act'(g),  du = dh act(g),  g = x Wg^T,  u = x Wu^T
 *   dx = dg Wg + du Wu  [tokens, d_model],  dwg = dg^T x,  dwu = du^T x  [d_ff, d_model]
 * All of the operands' 16-bit type; dg and du are rounded to it once (in fp16
 * they overflow past 65504: scale the loss), sums are fp32, each gradient is
 * rounded once.  Outputs are written in full (dwg, dwu:
 * zeros for 0 tokens) and must not overlap anything.  No atomics: the same
 * inputs give the same bits.  Calls on one handle share its scratch and must not
 * overlap on the GPU (graphs that hold such calls included).
 * Errors: INVALID_ARG (also for more than max_grad_tokens), UNSUPPORTED, CUDA.
 */
int tfl_glu_backward(tfl_glu* g, int64_t tokens, const void* x, const void* wg, const void* wu, const void* dh,
                     void* dx, void* dwg, void* dwu, tfl_stream stream);

/* Synchronize `stream`, read and clear the status word: TFL_OK or TFL_ERR_DEVICE_TIMEOUT. */
int tfl_glu_status(tfl_glu* g, tfl_stream stream);

void tfl_glu_destroy(tfl_glu* g);

/*
 * Linear layer with its epilogue, the projections and the feed-forward halves of the
 * stack above on their own:
 *   z = x W^T + bias,   y = act(z) + res
 * with W in nn.Linear layout [d_out, d_in].  Products accumulate in fp32; bias,
 * activation and residual are applied to the fp32 sums and y is rounded once.
 * The sums are the tensor cores': an fp32 y of 4096 products is off by about 2e-6 of
 * its size (sums rounded to nearest: 3e-7); 16-bit outputs do not show it.
 * An infinite z gives act(inf) = inf and, as the product -inf times 0, no number
 * for act(-inf).
 *
 * Operands (x, W): fp16 or bf16; or e4m3 with one fp32 scale a row (the stored
 * value times its row's scale is the operand's value, as the norms above write x).
 * y and res: fp32, or 16 bits, the operands' type where they have 16.  bias is fp32.
 */
typedef struct tfl_linear tfl_linear;

/* d_in and d_out: multiples of 8 (16 for e4m3 operands) up to 2^24.  act: TFL_ACT_NONE,
 * TFL_ACT_SILU or TFL_ACT_GELU.
 * max_grad_tokens: the most tokens tfl_linear_backward will be given (0: no
 * backward; e4m3 operands have none), and dy_type the type of its dy, fp32 or the
 * operands' (not looked at without a backward).  The handle holds partial sums for it, at
 * most max(64 MiB, 4 d_out bytes) for db and, for small weights and many tokens, at most 24 MiB for
 * dw; with an activation or an fp32 dy 2 max_grad_tokens d_out bytes more (d_out to the next
 * multiple of 64).
 * Errors: INVALID_ARG, UNSUPPORTED, OOM, CUDA. */
int tfl_linear_create(int32_t d_in, int32_t d_out, int32_t in_type, int32_t out_type, int32_t act, int32_t dy_type,
                      int64_t max_grad_tokens, tfl_linear** out);

/*
 * Asynchronous on `stream`.  Device pointers, 16-byte aligned, row-major and
 * contiguous; any number of tokens from 0 (nothing is done):
 *   x [tokens, d_in], w [d_out, d_in], bias fp32 [d_out] or NULL
 *   x_scale fp32 [tokens] (4-byte aligned), w_scale fp32 [d_out] for e4m3
 *   operands, else NULL
 *   res  [tokens, d_out] of y's type, or NULL; may be y
 *   z    [tokens, d_out] of the operands' type, which the backward of a layer
 *        with an activation takes; or NULL (not stored; always so without an
 *        activation and for e4m3 operands)
 *   y    [tokens, d_out]
 * Other overlaps of an output are refused.  Rows do not affect one another.
 * Calls on one handle may overlap.  Errors: INVALID_ARG (also when the current
 * device is not the handle's), UNSUPPORTED, CUDA; a device-side wait that ran out
 * surfaces through tfl_linear_status.
 */
int tfl_linear_forward(tfl_linear* l, int64_t tokens, const void* x, const float* x_scale, const void* w,
                       const float* w_scale, const float* bias, const void* res, void* z, void* y, tfl_stream stream);

/*
 * The gradients, with dz = dy act'(z) (dy without an activation; res's gradient is dy):
 *   dx = dz W  [tokens, d_in],   dw = dz^T x  [d_out, d_in],   db = sum over tokens of dz  fp32 [d_out]
 *   x, w  as in the forward;  z  as it stored it, NULL without an activation
 *   dy    [tokens, d_out] of the handle's dy_type
 * dx, dw and db may each be NULL (not computed; w is then not read for dx, nor x for
 * dw, and may be NULL too); one at least is given.
 * dx and dw are of the operands' type.  dz is rounded to it once for the products, so
 * that their error is 1.4 times that of one rounding (in fp16 dz overflows past 65504,
 * loses bits below 6.1e-5 and is 0 below 3e-8, an fp32 dy's too: scale the loss); db
 * sums dz unrounded; sums are fp32, each gradient is rounded once.  Outputs are
 * written in full (dw, db: zeros for 0 tokens) and must not overlap anything.  No
 * atomics: the same inputs give the same bits, in any handle.  Calls on one handle
 * share its scratch and must not overlap on the GPU (graphs that hold such calls
 * included).
 * Errors: INVALID_ARG (also for more than max_grad_tokens), UNSUPPORTED, CUDA.
 */
int tfl_linear_backward(tfl_linear* l, int64_t tokens, const void* x, const void* w, const void* z, const void* dy,
                        void* dx, void* dw, float* db, tfl_stream stream);

/* Synchronize `stream`, read and clear the status word: TFL_OK or TFL_ERR_DEVICE_TIMEOUT. */
int tfl_linear_status(tfl_linear* l, tfl_stream stream);

/* Free what the handle owns.  Synchronizes the device.  NULL is a no-op. */
void tfl_linear_destroy(tfl_linear* l);

/* Which kernel a launch of the linear layer takes, as tfl_selftest_glu_plan tells it of
 * the feed-forward; part 0 the forward, 1 and 2 the backward's dx and dw. */
int tfl_selftest_linear_plan(int32_t d_in, int32_t d_out, int32_t in_type, int32_t part, int64_t tokens,
                             const int32_t* units, int32_t* out);

#ifdef __cplusplus
}
#endif
#endif /* TFL_H_ */

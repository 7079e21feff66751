/*
 * dg.h -- C ABI of the GB300 (sm_103a) decode-step skinny GEMV library (libdg.so).
 *
 * What it computes: the weight-streaming matrix-vector product of single-request
 * LLM decoding, y = x * W^T with x holding M = 1 token (or a few draft/verify
 * tokens), in three forms:
 *   - FP16 / BF16 weights                 (dg_gemv_f16)
 *   - a very wide lm_head + greedy argmax (dg_lm_head_argmax)
 *   - weight-quantized: W8A8 per-channel int8 (dg_gemv_w8a8) and groupwise
 *     int4 with fp16 or int8 activations (dg_gemv_w4), dequantized in registers.
 * and what a decoder runs between those products for a step's new tokens: norms
 * with the residual add (dg_norm_residual), rotary positions and the cache
 * append (dg_kv_append), attention over a paged cache (dg_attn_decode) and an
 * expert layer (dg_moe_forward); and what a serving step runs around them: pages
 * for the tokens to come (dg_assign_pages), head norms with the append, also to a
 * cache held in 4 bits (dg_qkv_append, dg_kv4_read), attention over that cache
 * (dg_attn4_decode) and log probabilities of tokens (dg_token_logprobs).
 * Sources: the M=1 custom cube matmul, the 16-slice lm_head with a host reduce
 * and the weight-bandwidth floor of "MiniCPM-V on Orange Pi AIPro (Ascend 310B)";
 * single-request decode and graph-replayed decode steps of "EdgeFM: Efficient
 * Edge Inference for Vision-Language Models" (sections 2.B and 2.C); W8A8 and
 * W4A8 of "vLLM Arm CPU optimizations" (sections "INT8 W8A8", "INT8 W4A8").
 * The pages give no formulas: the definitions below are the plain readings.
 *
 * Conventions (every entry point):
 *  - Layout.  W is [N][K] row-major (output features x input features, K
 *    contiguous).  x is [M][K] and y is [M][N], row-major.
 *    y[m][n] = sum_k W[n][k] * x[m][k].
 *  - Pointers.  All tensor pointers are DEVICE pointers owned by the caller.
 *    The library allocates and frees nothing; scratch comes from the caller's
 *    workspace (ws, ws_bytes), sized by dg_workspace_bytes.
 *  - Streams.  Work is enqueued on `stream` (NULL = legacy default stream);
 *    calls never synchronize and can be captured into a CUDA graph.  Kernels
 *    are launched with programmatic dependent launch: a kernel may prefetch its
 *    weights into L2 while the previous kernel on the stream finishes, and
 *    touches activations, outputs and workspace only after it completed.
 *  - Errors.  Arguments are validated on the host before anything is launched;
 *    on failure nothing is enqueued and a dg_status other than DG_OK returns.
 *    A failed launch returns DG_ERR_CUDA.  No C++ exception crosses the ABI.
 *  - Determinism.  Each output is summed in a fixed order that depends only on
 *    K and the element format (never on N, M, the row offset or the launch
 *    grid), so repeated calls are bitwise identical and a row slice of W gives
 *    bitwise the same rows as the whole matrix.  One exception, opt-in: a
 *    per-op call (dg_gemv_*) with few rows (its row groups would fill fewer
 *    than half the SMs) that is given workspace splits K across CTAs (split-K:
 *    S fixed K ranges, partial sums in ws, a second kernel adding them in range
 *    order); its order then also depends on N, M and the SM count, and is still
 *    the same on every call.  Integer (W8A8) sums are exact either way.  The
 *    second exception: fp16 / bf16 calls with 8 <= M <= 16 and no epilogue run
 *    on the tcgen05 tensor cores with the work split stream-K over all SMs (the
 *    launch's 128-row x 64-k weight blocks cut into one equal range per SM; a
 *    row tile cut between CTAs is summed in fp32 piece by piece in CTA order),
 *    so their order depends on K, on the rows of the whole launch and on the
 *    SM count, and is still the same on every call.  The same holds for int4
 *    calls on the int8 / int4 tcgen05 tile (by default 8+ tokens with K >
 *    8192; one fp32 accumulator per group, scaled as in the scalar
 *    definition); W8A8 calls with 8+ tokens also run there by default and
 *    keep exact int32 sums.  Such a call keeps a small
 *    fixup scratch per (device, stream) (about 4.3 MB, allocated on the
 *    stream's first such call); a stream first used inside graph capture runs
 *    the mma.sync tile instead (K split by a rule on K alone).
 *  - Alignment.  W, x, xq and y must be 16-byte aligned; K must be a multiple
 *    of 8 (fp16/bf16), 16 (int8) or 32 (int4).
 *  - Tuning.  The environment variable DG_TUNE (comma-separated KEY=value,
 *    read once per process) overrides launch choices for configuration
 *    sweeps; unset, the defaults above hold.  Every setting stays within the
 *    parity bound; KS (warps per row), KP (split-K ranges), MMA (tensor-core
 *    tiles off / int8 tile), TC (fewest tokens on the fp16 / bf16 tcgen05
 *    tile, 0 = off), TQ (fewest tokens on the int8 / int4 tcgen05 tile, 0 =
 *    off; by default W8A8 with 8+ tokens and int4 with 8+ tokens and K > 8192
 *    go there) and TG
 *    (the tcgen05 tiles' CTA count) change a row's summation order, the others
 *    (TK: 64-k boxes per stage of the fp16 tile, 1 or 2; TS: its ring stages,
 *    6 / 8 / 12 with one box, 3 / 4 / 6 with two; TP: stages it prefetches to
 *    L2 before the dependency wait) only the schedule.
 */
#ifndef DG_H_
#define DG_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

struct CUstream_st;
typedef struct CUstream_st* dg_stream; /* same type as cudaStream_t */

typedef enum {
    DG_OK = 0,
    DG_ERR_INVALID_ARG = 1, /* null pointer, non-positive size, bad enum */
    DG_ERR_UNSUPPORTED = 2, /* shape or option outside what the kernels handle */
    DG_ERR_MISALIGNED = 3,  /* a pointer or K breaks the alignment rules */
    DG_ERR_WORKSPACE = 4,   /* ws smaller than dg_workspace_bytes asks for */
    DG_ERR_CUDA = 5,        /* a CUDA call or launch failed */
    DG_ERR_TIMEOUT = 6      /* a bounded device-side wait gave up */
} dg_status;

typedef enum { DG_F16 = 0, DG_BF16 = 1 } dg_ftype;

/* Kind of one linear op in a decode step (dg_linear.kind). */
typedef enum {
    DG_LINEAR_F16 = 0,   /* W fp16 [N][K], x fp16 [M][K], y fp16 */
    DG_LINEAR_BF16 = 1,  /* W bf16, x bf16, y bf16 */
    DG_LINEAR_W8A8 = 2,  /* W int8 [N][K] + float w_scale[N]; x_i8 + x_scale; y fp16 */
    DG_LINEAR_W4A16 = 3, /* W packed int4 [N][K/2] + half w_scale[N][K/group]; x fp16; y fp16 */
    DG_LINEAR_W4A8 = 4   /* as W4A16 but x_i8 + x_scale; y fp16 */
} dg_kind;

/* Epilogue applied to an op's fp32 result before it is rounded to y
 * (dg_linear.epilogue); the pages motivate only removing the launches around
 * the weight stream (EdgeFM, section 2.C, graph-accelerated decode), so these
 * are the plain decoder definitions:
 *   DG_EPI_RESIDUAL: y = x * W^T + residual     (residual [M][N], y's type)
 *   DG_EPI_SWIGLU:   y = silu(x * W^T) * (x * W2^T),  silu(v) = v / (1 + e^-v)
 *                    (W the gate projection, W2 the up projection: same kind,
 *                    shape and group; w2_scale their scales for int4 kinds).
 * Both are evaluated in fp32 on the sums and rounded once into y; y may be
 * the residual itself (an in-place add: each element is read, then written,
 * by the same thread).  Not for
 * lm_heads (token != NULL), nor with acc_out; SwiGLU is not offered for
 * DG_LINEAR_W8A8 (DG_ERR_UNSUPPORTED). */
typedef enum { DG_EPI_NONE = 0, DG_EPI_RESIDUAL = 1, DG_EPI_SWIGLU = 2 } dg_epilogue;

/* One linear op: y = x * W^T in the format `kind`.
 * For the quantized-activation kinds (W8A8, W4A8), x_i8 [M][K] and x_scale[M]
 * are read; if `x` (fp16 [M][K]) is also given, dg_decode_step_weights first
 * quantizes x into x_i8 / x_scale (see dg_quantize_act_i8).
 * An op with token != NULL is an lm_head: M must be 1, logits (fp32 [N]) and
 * the greedy token are written and y may be NULL. */
typedef struct {
    int32_t kind;
    int32_t M, N, K;
    int32_t group_size;    /* int4 kinds: multiple of 32 dividing K (32 in the workloads) */
    const void* W;
    const void* w_scale;
    const void* x;
    const int8_t* x_i8;
    const float* x_scale;
    void* y;
    float* logits;
    int32_t* token;
    int32_t* acc_out;      /* W8A8 only, optional: exact int32 accumulators [M][N] */
    int32_t epilogue;      /* dg_epilogue (0 = none) */
    int32_t reserved;      /* must be 0 */
    const void* residual;  /* DG_EPI_RESIDUAL */
    const void* W2;        /* DG_EPI_SWIGLU: up-projection weights */
    const void* w2_scale;  /* DG_EPI_SWIGLU: their scales (int4 kinds) */
} dg_linear;

/* FP16 / BF16 weights (paragraph on the custom M=1 cube matmul of the Orange
 * Pi AIPro post; the vector-matrix product at M=1).
 * W [N][K], x [M][K], y [M][N], all of type t; 1 <= M <= 16 and M * K * 4
 * bytes within the shared memory of one CTA (DG_ERR_UNSUPPORTED otherwise).
 * Products are exact in fp32 and summed in fp32; y = round-to-nearest-even of
 * the fp32 sum.  ws may be NULL.  With ws (16-byte aligned) of at least
 * dg_workspace_bytes(&op, 1) bytes for the equivalent dg_linear, a call with
 * few rows may split K across CTAs (see Determinism above); with less, or
 * NULL, it does not.  The same holds for dg_gemv_w8a8 and dg_gemv_w4. */
dg_status dg_gemv_f16(const void* W, const void* x, void* y, dg_ftype t, int M, int N, int K,
                      void* ws, size_t ws_bytes, dg_stream stream);

/* W8A8 ("vLLM Arm CPU optimizations", section "INT8 W8A8").
 * W int8 [N][K], w_scale float [N] (per output channel), x int8 [M][K],
 * x_scale float [M] (per token), 1 <= M <= 16.
 * acc[m][n] = sum_k W[n][k] x[m][k] exactly in int32 (|acc| <= K*128*128
 * must fit: K <= 131072); y[m][n] = fp16(float(acc) * w_scale[n] * x_scale[m]).
 * acc_out (int32 [M][N]) receives acc when non-NULL. */
dg_status dg_gemv_w8a8(const int8_t* W, const float* w_scale, const int8_t* x,
                       const float* x_scale, void* y, int32_t* acc_out, int M, int N, int K,
                       void* ws, size_t ws_bytes, dg_stream stream);

/* Groupwise int4 weights ("vLLM Arm CPU optimizations", section "INT8 W4A8";
 * fused INT4 dequantization of the Orange Pi AIPro post's closing paragraph).
 * Wq uint8 [N][K/2]: byte j of a row holds k = 2j in bits 0-3 and k = 2j+1 in
 * bits 4-7 as 4-bit two's complement (codes -8..7).  scales fp16
 * [N][K/group_size]; group_size a multiple of 32 that divides K.
 * W4A16 when x_i8 == NULL:  y = fp16( sum_g s[n][g] * P_g ),
 *                           P_g = sum_{k in g} q[n][k] * x[m][k]   (fp32)
 * W4A8 when x_i8 != NULL:   acc_g = sum_{k in g} q * x_i8 (exact int32),
 *                           y = fp16( x_scale[m] * sum_g s[n][g] * acc_g ).
 * x_f16 [M][K] is read for W4A16 and ignored for W4A8.  1 <= M <= 16, and the
 * staged activations (2 bytes per element for W4A16, about 1 for W4A8) must
 * fit one CTA's shared memory (DG_ERR_UNSUPPORTED otherwise). */
dg_status dg_gemv_w4(const uint8_t* Wq, const void* scales, int group_size, const void* x_f16,
                     const int8_t* x_i8, const float* x_scale, void* y, int M, int N, int K,
                     void* ws, size_t ws_bytes, dg_stream stream);

/* One op described by a dg_linear (any kind except an lm_head; any epilogue),
 * M <= 16, as one launch (two with split-K).  Same arithmetic as the
 * dg_gemv_* entry points of its kind; ws as for them (may be NULL; an op
 * with an epilogue never splits K).  W8A8 / W4A8 ops read x_i8 / x_scale
 * and must not carry fp16 x here (quantize first with dg_quantize_act_i8). */
dg_status dg_linear_forward(const dg_linear* op, void* ws, size_t ws_bytes, dg_stream stream);

/* Elementwise fp16 epilogues as separate launches (what a decoder runs when
 * they are not fused into the weight stream; same fp32 arithmetic):
 *   dg_swiglu:       h[i] = fp16( silu(g[i]) * u[i] )
 *   dg_residual_add: out[i] = fp16( a[i] + b[i] )
 * n elements; pointers 16-byte aligned, n a multiple of 8; out may alias a
 * or b (elementwise), h may alias g or u. */
dg_status dg_swiglu(const void* g, const void* u, void* h, int n, dg_stream stream);
dg_status dg_residual_add(const void* a, const void* b, void* out, int n, dg_stream stream);

/* One decode step of a depthwise causal 1-D convolution (the causal-conv1d
 * step kernel of "MiniCPM-V on Orange Pi AIPro (Ascend 310B)"; the page gives
 * no formula, this is the plain definition).  For token m and channel c, with
 * u = state[m][c][0 .. width-2] (oldest first) followed by x[m][c]:
 *   v = bias[c] + sum_{j < width} w[c][j] * u[j]     (fp32: exact products,
 *       one rounding per term, j ascending after the bias)
 *   y[m][c] = fp16(act == DG_ACT_SILU ? silu(v) : v)
 * then state[m][c] becomes u[1 .. width-1] (the oldest input drops out).
 * x, y fp16 [M][C]; state fp16 [M][C][width-1] (read and rewritten in place);
 * w fp16 [C][width]; bias fp16 [C] or NULL.  2 <= width <= 8, C a multiple
 * of 8, pointers 16-byte aligned; y must not overlap state. */
typedef enum { DG_ACT_NONE = 0, DG_ACT_SILU = 1 } dg_act;
dg_status dg_causal_conv1d_update(const void* x, void* state, const void* w, const void* bias,
                                  void* y, int M, int C, int width, int act, dg_stream stream);

/* Load-time weight quantizers and packers ("vLLM Arm CPU optimizations",
 * section "Dense layer weight prepacking": weights are put in the kernels'
 * format once, at warm-up).  Decided in IEEE fp32, as the library's kernels
 * expect them; W fp16 [N][K] (16-byte aligned, K a multiple of 16 / of
 * group_size).
 *   dg_quantize_weights_i8: s[n] = max_k |W[n][k]| / 127 (1 for an all-zero
 *     row), Wq[n][k] = clamp(rne(W / s), -127, 127)  -> DG_LINEAR_W8A8 input.
 *   dg_quantize_weights_w4: per group of group_size k, s = fp16(amax / 7)
 *     raised to the smallest fp16 subnormal if it rounds to 0 (1 for an
 *     all-zero group), code = clamp(rne(W / s), -7, 7), packed two per byte
 *     (k = 2j in bits 0-3 of byte j, k = 2j+1 in bits 4-7); scales fp16
 *     [N][K/group_size]  -> DG_LINEAR_W4A16 / W4A8 input. */
dg_status dg_quantize_weights_i8(const void* W, int8_t* Wq, float* w_scale, int N, int K,
                                 dg_stream stream);
dg_status dg_quantize_weights_w4(const void* W, uint8_t* Wq, void* scales, int N, int K,
                                 int group_size, dg_stream stream);

/* Per-token symmetric int8 activations for W8A8 / W4A8 (same page, same
 * sections).  x fp16 [M][K] -> xq int8 [M][K], x_scale float [M]:
 *   amax = max_k |x[m][k]|,  s = amax / 127 (IEEE fp32 division),
 *   q = clamp(round-half-even(x / s), -127, 127);  s = 1, q = 0 if amax = 0. */
dg_status dg_quantize_act_i8(const void* x, int8_t* xq, float* x_scale, int M, int K,
                             dg_stream stream);

/* Wide lm_head with fused greedy argmax (paragraph on the ~248k-vocabulary
 * lm_head of the Orange Pi AIPro post, which splits it into 16 slices and
 * reduces on the host; here one launch plus a tiny second pass).
 * head->kind is DG_LINEAR_F16, DG_LINEAR_BF16, DG_LINEAR_W4A16 or
 * DG_LINEAR_W4A8; head->M must be 1.  Writes fp32 logits[N] and
 * token = the index of the largest logit, the lowest index on exact ties
 * (+0 equals -0); a NaN logit never wins.  Needs dg_workspace_bytes(head, 1)
 * bytes of workspace (per-CTA (value, index) partials). */
dg_status dg_lm_head_argmax(const dg_linear* head, void* ws, size_t ws_bytes, dg_stream stream);

/* dg_lm_head_argmax without a workspace argument, for callers that cannot
 * allocate device memory: a decode loop that must not allocate once running,
 * a plugin whose host runtime owns all device memory through its own pool, or
 * code whose memory plan was fixed ahead of time.  (The pages have no
 * counterpart to this entry point.)  Same inputs, outputs and results as
 * dg_lm_head_argmax (the same kernels and launch configuration, so the same
 * bits); the per-CTA partials live in a fixed 16 KB array inside the library
 * (2048 partials; every GPU that loads the library keeps it until the
 * process exits).  A head launches at most SMs x 8 CTAs (1216 on a 152-SM
 * GB300), so every head fits there.
 *  - The first call on a device looks up that array's address (with the
 *    device current) and caches it: make that first call before any stream
 *    capture.  The cached address belongs to the device's primary context:
 *    do not keep using the library across a cudaDeviceReset of that device.
 *    No call allocates or frees memory.
 *  - A head that would need more than 2048 partials (a GPU with more than 256
 *    SMs) returns DG_ERR_WORKSPACE and launches nothing.
 *  - Every call shares the array; nothing in it needs to start at zero (each
 *    call writes every partial it reads).  Calls that can overlap on the GPU
 *    (different streams, or different host threads on one device) race on the
 *    array: serialize them. */
dg_status dg_lm_head_argmax_noalloc(const dg_linear* head, dg_stream stream);

/* One decode step's weight stream (graph-accelerated decode of EdgeFM,
 * section 2.C): runs ops[0..n_ops) in order.  Consecutive ops of the same
 * kind that read the same activations (same x / x_i8 / x_scale pointers,
 * same M, K and group) and are not lm_heads are fused (q|k|v, gate|up); every
 * other boundary is a dependency: an op reads its activations only after
 * every earlier op finished.
 * Runs of single-token ops (M = 1, no acc_out) of one kind execute as ONE
 * persistent cooperative launch: one CTA per SM takes a contiguous row slice
 * of every fused group, groups meet at a grid-wide barrier, and each CTA
 * prefetches its upcoming weight rows into L2 ahead of use, across group
 * boundaries.  Other ops run as one launch per fused group.  Both give the
 * same bits as calling dg_gemv_* / dg_lm_head_argmax op by op.
 * For W8A8 / W4A8 ops that carry fp16 `x`, the step quantizes x exactly as
 * dg_quantize_act_i8 does and also writes the codes / scale to x_i8 / x_scale.
 * Ops may carry epilogues (dg_epilogue): a SwiGLU op streams W and W2 row by
 * row in pairs, and an op reading another op's output (the down projection
 * reading the SwiGLU result) waits for it like any other dependency.
 * Weights and scales must stay unchanged during the step (they are read
 * early).  ws: dg_workspace_bytes(ops, n_ops) bytes, 16-byte aligned, owned
 * by the caller; the step overwrites it (nothing needs to be zeroed first).
 * A barrier wait that exceeds its bound (about a second) makes the launch
 * end early; dg_check_device_status then reports DG_ERR_TIMEOUT. */
dg_status dg_decode_step_weights(const dg_linear* ops, int n_ops, void* ws, size_t ws_bytes,
                                 dg_stream stream);

/* Workspace bytes that dg_decode_step_weights needs for these ops (256 for
 * the persistent kernel's barrier, plus 32 KB of argmax partials when an op is
 * an lm_head, plus, per int4 op at M = 1, its activations in the kernel's
 * layout: DG_LINEAR_W4A8 ceil(K/1024)*1024 + K/8 bytes, DG_LINEAR_W4A16
 * ceil(K/1024)*2048 bytes, each rounded up to 256); for a
 * single lm_head this also covers dg_lm_head_argmax; for a single op of at
 * most 65536 outputs (M * N) it also covers split-K partials of a dg_gemv_*
 * call (8 ranges x M x N x 4 bytes).
 * 0 for n_ops <= 0.  Host-only; touches no device. */
size_t dg_workspace_bytes(const dg_linear* ops, int n_ops);

/* ---- the rest of a decoder layer -------------------------------------------------
 * What a decoder runs between its weight products, for the 1..16 new tokens per
 * sequence of a decode or verify step: norms, rotary positions and the cache
 * append, attention over the cache, and (sparse decoders) an expert layer.
 * The pages name these steps without formulas (single-request decode over a
 * KV cache and draft / verify tokens: EdgeFM, sections 2.B and 2.C); each
 * declaration states the definition.  All arithmetic is fp32 or wider, but for
 * what a declaration says of its weights or its hidden values; each 16-bit output
 * is rounded to nearest even once. */

/* A paged key / value cache of `batch` sequences.  Sequence b's position j lies
 * in page block_table[b * table_stride + j / page_size], slot j % page_size;
 * its key of head g starts at
 *   k + page * page_stride + slot * token_stride + g * head_stride
 * (strides in elements, the same for k and v; the head_dim values of one head
 * are contiguous), so [page][slot][head][dim] and [page][head][slot][dim] both
 * fit.  seq_lens[b] counts the step's new tokens too.  Positions from
 * max_pages * page_size on and positions whose page id is outside
 * [0, num_pages) do not exist: the append writes nothing there and no token
 * sees them.  The table and the lengths are device memory, read when the
 * kernels run, so a captured graph follows them.  Up to 2^20 sequences and 1024
 * heads; more return DG_ERR_UNSUPPORTED. */
typedef struct {
    int32_t type;      /* dg_ftype of the cache and of q, k, v, out */
    int32_t batch;
    int32_t kv_heads;
    int32_t head_dim;  /* multiple of 8, at most 256 */
    int32_t page_size;
    int32_t num_pages;
    int32_t max_pages; /* pages per sequence in block_table */
    int32_t reserved;  /* must be 0 */
    void* k;
    void* v;
    int64_t page_stride;
    int64_t token_stride;
    int64_t head_stride;
    const int32_t* block_table;
    int64_t table_stride;    /* at least max_pages, or batch 1 */
    const int32_t* seq_lens; /* [batch] */
} dg_paged_kv;

/* Rotary positions on a step's q and k, and k and v into their cache slots.
 * Token t = b * q_len + i (i < q_len) has position p = seq_lens[b] - q_len + i.
 * With half = rot_dim / 2, c = cos[p][j], s = sin[p][j] (fp32 [max_pos][half])
 * and the pair (x, y) at dims (j, j + half), or (2j, 2j + 1) if interleaved:
 *   (x, y) -> (x c - y s, y c + x s)           fp32, one rounding
 * dims from rot_dim on are copied.  q [batch * q_len][heads][head_dim] goes to
 * q_out (which may be q), k and v [batch * q_len][kv_heads][head_dim] to the
 * cache; *_stride are the elements from one token to the next, so q, k and v
 * may be columns of one q|k|v result.  A token with p < 0 (a sequence shorter
 * than the step) or, when rotating, p >= max_pos writes zeros to q_out and
 * nothing to the cache.  q may be NULL (heads 0): no q to rotate; rot_dim 0:
 * cos and sin are not read.  Two sequences must not share the page that they
 * append to.  Any 2-byte alignment works; 16-byte aligned pointers and strides
 * and rot_dim a multiple of 16 take the vector path. */
typedef struct {
    dg_paged_kv kv;
    int32_t q_len;       /* 1..16 */
    int32_t heads;
    int32_t rot_dim;     /* even, at most head_dim */
    int32_t interleaved; /* 0 or 1 */
    int32_t max_pos;
    int32_t reserved;    /* must be 0 */
    const void* q;
    const void* k;
    const void* v;
    void* q_out;
    int64_t q_stride, k_stride, v_stride, q_out_stride;
    const float* cos;
    const float* sin;
} dg_append;
dg_status dg_kv_append(const dg_append* op, dg_stream stream);

/* Attention of a step's new tokens over the paged cache (which already holds
 * their keys and values).  Query head h reads key / value head
 * h / (heads / kv_heads).  Token i of sequence b stands at
 * p = seq_lens[b] - q_len + i and sees the existing positions j with
 *   j <= p  and  (window == 0  or  j > p - window  or  j < sinks):
 * all of the past, or the last `window` positions plus the first `sinks` ones.
 *   z_j = scale * (q . k_j),  out = sum_j e^(z_j) v_j / sum_j e^(z_j),
 *   lse = log sum_j e^(z_j)                       (lse may be NULL)
 * A token that sees nothing (p < 0, no existing page), or whose visible scores
 * are all -infinity, gets out = 0 and lse = -infinity.  Values at positions a
 * token does not see never reach it, whatever they hold (NaN and infinity
 * too); visible ones follow IEEE.  scale is any number with a finite
 * scale * log2(e), zero and negative ones too.  Scores and sums are fp32; e^(z_j) meets v_j as
 * the sum of two 16-bit numbers, 2^-21 (fp16) or 2^-16 (bf16) of itself off, and in
 * fp16 up to 2^-32 of the strongest key's.  q [batch * q_len][heads][head_dim] with
 * q_stride elements between tokens, out likewise; lse fp32
 * [batch * q_len][heads].  heads is a multiple of kv_heads, 1 <= q_len <= 16.
 * q, out, k, v 16-byte aligned, strides multiples of 8.  The result does not
 * depend on the order in which CTAs run.  ws: dg_attn_workspace_bytes(op) bytes, 16-byte
 * aligned, overwritten (nothing needs to be zeroed); a call that may overlap
 * another needs its own. */
typedef struct {
    dg_paged_kv kv;
    int32_t q_len;
    int32_t heads;
    int32_t window; /* 0: no window */
    int32_t sinks;
    float scale;
    int32_t reserved; /* must be 0 */
    const void* q;
    void* out;
    float* lse;
    int64_t q_stride, out_stride;
} dg_attn;
dg_status dg_attn_decode(const dg_attn* op, void* ws, size_t ws_bytes, dg_stream stream);
/* Workspace of dg_attn_decode; 0 for an op that it would refuse. */
size_t dg_attn_workspace_bytes(const dg_attn* op);

/* The norms around a block, with its gate and residual scale.  Per row:
 *   r  = y, then (w_post) norm(r; w_post, b_post), then (gate) r * gate
 *   h' = alpha * h + beta * r             -> h_out    (r absent without y)
 *   x  = norm(h'; w_pre, b_pre)           -> x_out    (h' before its rounding)
 * with norm(v; w, b) = u / sqrt(mean(u^2) + eps) * (w_offset + w) + b, where
 * u = v (DG_NORM_RMS) or v - mean(v) (DG_NORM_LAYER), evaluated in fp32.
 * y, x_out, gate and the weights have type `type`; h and h_out have type
 * `type`, or are fp32 with h_f32.  All [rows][N] row-major; gate is [rows][N],
 * or one row [N] for all with gate_rows = 1.  May be NULL: y (with w_post and
 * gate), w_post, b_post, gate, b_pre, h (alpha * h is then absent; y must be
 * given), h_out or x_out (not both; w_pre is needed only with x_out).  h_out
 * may be h or (same type) y, x_out may be y or (same type) h; other overlaps
 * are not allowed.  1 <= N <= 32768; any 2-byte (fp32: 4-byte) alignment
 * works; the fastest path wants the row tensors 16-byte aligned (any N), for a
 * few rows the weights too and N a multiple of 8. */
typedef enum { DG_NORM_RMS = 0, DG_NORM_LAYER = 1 } dg_norm_kind;
typedef struct {
    int32_t type; /* dg_ftype */
    int32_t kind; /* dg_norm_kind */
    int32_t rows, N;
    int32_t h_f32;
    int32_t gate_rows; /* 0 without gate, else 1 or rows */
    float alpha, beta, eps, w_offset;
    const void* y;
    const void* w_post;
    const void* b_post;
    const void* gate;
    const void* h;
    const void* w_pre;
    const void* b_pre;
    void* h_out;
    void* x_out;
} dg_norm;
dg_status dg_norm_residual(const dg_norm* op, dg_stream stream);

/* A mixture-of-experts layer for a few tokens, 1 <= M <= 16.
 *   z = x * router^T;  prob = softmax(z) (or sigmoid(z) with DG_MOE_SIGMOID)
 *   the top_k experts of each token by prob, the lowest index on ties; a NaN
 *   counts below every number; weight = prob, divided by the chosen ones' sum
 *   with renormalize; times route_scale
 *   h_e = silu(x * W_gate[e]^T) * (x * W_up[e]^T)
 *   y = sum over the chosen e of weight_e * (h_e * W_down[e]^T)   (+ residual)
 * x, y, residual [M][K]; router [E][K] in x's type; W_gate, W_up [E][I][K] and
 * W_down [E][K][I] in the format `kind`: DG_LINEAR_F16, DG_LINEAR_BF16, or
 * DG_LINEAR_W4A16 (packed int4 [E][rows][cols / 2], fp16 scales
 * [E][rows][cols / group_size], x and y fp16).  All sums are fp32.  h_e is held
 * as the sum of two 16-bit numbers: 22 significant bits from |h_e| = 2^-6 up and
 * steps of 2^-27 below (fp16 x, int4; from about 2^24 on it becomes infinite), or
 * 16 significant bits (bf16 x).  ids int32 [M][top_k] and
 * weights fp32 [M][top_k], both optional, receive the routing in descending
 * order of prob.  Each expert's weights are read once for up to eight of its
 * tokens, mostly for all sixteen.  A token's result does not depend on the order
 * in which CTAs run.  K and I multiples of 8 (fp16,
 * bf16) or of group_size, itself a multiple of 32 (int4), up to 65536; 1 <= E <= 1024,
 * 1 <= top_k <= min(E, 16); pointers 16-byte aligned (scales 2, residual 2,
 * ids and weights 4).  y may be residual or x.  ws: dg_moe_workspace_bytes(op)
 * bytes, 16-byte aligned, overwritten; a call that may overlap another needs
 * its own. */
typedef enum { DG_MOE_SOFTMAX = 0, DG_MOE_SIGMOID = 1 } dg_moe_score;
typedef struct {
    int32_t kind; /* dg_kind */
    int32_t M, K, I, E, top_k;
    int32_t group_size; /* int4 only */
    int32_t score;      /* dg_moe_score */
    int32_t renormalize;
    float route_scale;
    const void* x;
    const void* router;
    const void* W_gate;
    const void* W_up;
    const void* W_down;
    const void* gate_scale; /* int4 only */
    const void* up_scale;
    const void* down_scale;
    const void* residual; /* optional */
    void* y;
    int32_t* ids;   /* optional */
    float* weights; /* optional */
} dg_moe;
dg_status dg_moe_forward(const dg_moe* op, void* ws, size_t ws_bytes, dg_stream stream);
/* Workspace of dg_moe_forward; 0 for an op that it would refuse. */
size_t dg_moe_workspace_bytes(const dg_moe* op);

/* ---- a serving step ------------------------------------------------------------------
 * Pages for the tokens to come, head norms with the append, a cache held in 4 bits
 * with the attention that reads it, and log probabilities of the answer.  The pages
 * name none of these; each declaration states the definition.  Lengths, tables, maps
 * and pools are device memory, read when the kernels run, so a captured graph follows
 * them.  All arithmetic on values is fp32 or wider, and each 16-bit output is rounded to
 * nearest even once. */

/* A paged cache as dg_paged_kv, held in 4 bits: each 16 consecutive dims of a head
 * are 16 codes c, 4-bit two's complement with dims 2j and 2j + 1 in bits 0-3 and 4-7
 * of byte j, and one scale byte s, an e4m3 number (fn: 0x7F and 0xFF are NaN).  A
 * value is factor * s * c, its factor k_factor or v_factor: 4.5 bits a value.  The
 * codes of sequence b's position j, head g start at
 *   k + page * page_stride + slot * token_stride + g * head_stride      (bytes)
 * and its head_dim / 16 scales at k_scale with the scale_* strides; v and v_scale
 * likewise.  [page][head][slot][..] reads each head's rows in one piece and is the
 * faster order.  Codes of -8 are read as such (the append writes none).  k, v and
 * the strides of codes are multiples of 8 bytes; scales may lie anywhere.  Strides of
 * 2^32 bytes or more return DG_ERR_UNSUPPORTED. */
typedef struct {
    int32_t type;      /* dg_ftype of q, k, v, out beside the cache */
    int32_t batch;
    int32_t kv_heads;
    int32_t head_dim;  /* multiple of 16, at most 256 */
    int32_t page_size;
    int32_t num_pages;
    int32_t max_pages; /* pages per sequence in block_table */
    int32_t reserved;  /* must be 0 */
    uint8_t* k;
    uint8_t* v;
    uint8_t* k_scale;
    uint8_t* v_scale;
    int64_t page_stride, token_stride, head_stride;                   /* of codes */
    int64_t scale_page_stride, scale_token_stride, scale_head_stride; /* of scales */
    float k_factor;    /* above 0, finite; 1 / 7 of a group's largest value over it */
    float v_factor;    /* should lie in 2^-6..448, where e4m3 has all of its bits */
    const int32_t* block_table;
    int64_t table_stride;    /* at least max_pages, or batch 1 */
    const int32_t* seq_lens; /* [batch] */
} dg_paged_kv4;

/* Norms of queries and keys for each head, rotary positions, and the append, in one
 * pass.  For a head's values x of one token (q with w_q, k with w_k; not normed
 * where that is NULL, and v never):
 *   x = u / sqrt(mean(u^2) + eps) * (w_offset + w),   u = x (DG_NORM_RMS) or
 *       x - mean(x) (DG_NORM_LAYER), over the head's head_dim values
 * then the rotation of dg_kv_append (pairs, dims from rot_dim on and tables as
 * there), all in fp32.  q goes to q_out (which may be q), k and v to the cache:
 *   bits 16 (kv):  rounded once
 *   bits 4 (kv4):  per 16 dims s = e4m3(max |x| / (7 factor)), to nearest even and at
 *       most 448, c = min(max(rne(x / (s factor)), -7), 7), 0 where s is 0 (products and
 *       quotients each rounded to fp32); a group that holds an infinity or a NaN gets s = NaN and c = 0.
 * Without slots: token t = b * q_len + i of batch * q_len, 1 <= q_len <= 16, has
 * position p = seq_lens[b] - q_len + i and its place by the block table.  With slots
 * (int64 [tokens]; positions int32 [tokens], both needed): token t has position
 * positions[t] and lies in slot slots[t] = page * page_size + place, wherever that
 * is: prompts of any lengths in one call (the table and the lengths are not read, q_len is 0).
 * A token with p < 0 or, when rotating, p >= max_pos writes zeros to q_out and
 * nothing to the cache; one whose page or slot does not exist writes nothing to the
 * cache.  Two tokens must not share a slot.  Any 2-byte alignment of q, k, v, q_out and
 * a 16-bit cache works; 16-byte aligned pointers and strides, head_dim a
 * multiple of 8 and rot_dim of 16 take the vector path.  q may be NULL (heads 0). */
typedef struct {
    dg_paged_kv kv;      /* bits 16 */
    dg_paged_kv4 kv4;    /* bits 4 */
    int32_t bits;        /* 16 or 4: which of the two is meant; the other is not read */
    int32_t q_len;
    int32_t tokens;      /* with slots, else 0 */
    int32_t heads;
    int32_t rot_dim;     /* even, at most head_dim */
    int32_t interleaved; /* 0 or 1 */
    int32_t max_pos;
    int32_t norm;        /* dg_norm_kind */
    float eps, w_offset;
    const void* q;
    const void* k;
    const void* v;
    void* q_out;
    int64_t q_stride, k_stride, v_stride, q_out_stride;
    const float* cos;
    const float* sin;
    const void* w_q;     /* [head_dim], the type of q */
    const void* w_k;
    const int64_t* slots;
    const int32_t* positions;
} dg_head_append;
dg_status dg_qkv_append(const dg_head_append* op, dg_stream stream);

/* Keys and values of a 4-bit cache back in 16 bits: k and v [tokens][kv_heads]
 * [head_dim] of type kv.type, *_stride elements from one token to the next, rounded
 * once; either may be NULL.  Without slots: the last q_len positions of each
 * sequence, any q_len >= 1, tokens = batch * q_len; with slots (int64 [tokens],
 * q_len 0): what lies there.  Zeros for what does not exist.  Any 2-byte alignment. */
typedef struct {
    dg_paged_kv4 kv;
    int32_t q_len;
    int32_t tokens;
    void* k;
    void* v;
    int64_t k_stride, v_stride;
    const int64_t* slots;
} dg_kv4_rows;
dg_status dg_kv4_read(const dg_kv4_rows* op, dg_stream stream);

/* dg_attn_decode over a cache held in 4 bits: the same definition, masks, outputs
 * and refusals, with the cache's values as dg_paged_kv4 states them.  They meet the
 * matrix instruction as they are (a code times an e4m3 number is exact in fp16); scores and
 * sums are fp32; e^(z_j) is the sum of two fp16 numbers, 2^-21 of itself off and up
 * to 2^-32 of the strongest key's, for both types; a bf16 query is taken in fp16 times a power of two,
 * exact but for values below 2^-30 of its row's largest.  A group whose scale is NaN makes
 * the scores (k) or its 16 dims of the output (v) NaN for those that see it, and for
 * nobody else.  scale * k_factor * log2(e) and 16 * v_factor must be finite.  q and out
 * 16-byte aligned, strides multiples of 8.  ws: dg_attn4_workspace_bytes(op) bytes,
 * 16-byte aligned, overwritten; a call that may overlap another needs its own. */
typedef struct {
    dg_paged_kv4 kv;
    int32_t q_len;
    int32_t heads;
    int32_t window;
    int32_t sinks;
    float scale;
    int32_t reserved; /* must be 0 */
    const void* q;
    void* out;
    float* lse;
    int64_t q_stride, out_stride;
} dg_attn4;
dg_status dg_attn4_decode(const dg_attn4* op, void* ws, size_t ws_bytes, dg_stream stream);
/* Workspace of dg_attn4_decode; 0 for an op that it would refuse. */
size_t dg_attn4_workspace_bytes(const dg_attn4* op);

/* Pages for a step's tokens, and where each token goes.  Sequence b holds lens[b]
 * tokens (below zero: none) in its first ceil(lens[b] / page_size) table entries and
 * asks for n = new_lens[b] more (new_len for all where new_lens is NULL); n < 0: it
 * ends.  Free pages wait in a queue, pool[(first + i) mod pool_size] for i < count,
 * with pool_state = {first, count}.  In order of b:
 *   - one that ends gives its pages back, behind the queue's end, to be taken by later
 *     calls; its length becomes 0 and its table row stays as it is;
 *   - one fits if its pages then fit the table (max_pages) and, with slots, its tokens
 *     the map (max_tokens); of those that fit, `asked` is the running sum of pages
 *     that they need beyond those held, and one is served if it needs none or
 *     asked <= count.  Served: the next pages of the queue go into its row, its
 *     length grows by n.  Not served: nothing of it changes.
 * Token i of sequence b is number starts[b] + i of the map, starts the running sum of
 * all n >= 0 (served or not; at most 2^31 - 1): slots[.] = page * page_size + place and
 * positions[.] = lens[b] + i, both -1 for tokens that are not served and in the rest
 * of the map (max_tokens); a slot whose table entry is below 0 is -1 too.  lens_out,
 * pool_state_out may be lens, pool_state; other overlaps are not allowed.  Table
 * entries and pool entries that no rule above names stay as they are.  May be NULL:
 * new_lens, starts [batch + 1], slots (int64, max_tokens 0 without), positions.
 * pool_size must be at least the number of pages there are.  ws:
 * dg_pages_workspace_bytes(op) bytes (0 for small calls: ws may be NULL then), 16-byte
 * aligned, overwritten; a call that may overlap another needs its own. */
typedef struct {
    int32_t batch;      /* up to 2^20 */
    int32_t page_size;
    int32_t max_pages;
    int32_t pool_size;
    int32_t new_len;
    int32_t max_tokens;
    int64_t table_stride; /* at least max_pages, or batch 1 */
    const int32_t* lens;
    const int32_t* new_lens;
    int32_t* lens_out;
    int32_t* block_table;
    int32_t* pool;
    const int32_t* pool_state;
    int32_t* pool_state_out;
    int32_t* starts;
    int64_t* slots;
    int32_t* positions;
} dg_page_plan;
dg_status dg_assign_pages(const dg_page_plan* op, void* ws, size_t ws_bytes, dg_stream stream);
/* Workspace of dg_assign_pages; 0 where it needs none, or would refuse the op. */
size_t dg_pages_workspace_bytes(const dg_page_plan* op);

/* Log probabilities of given tokens, entropy and the best alternatives, from logits
 * [rows][V] (type, or fp32 with logits_f32; `stride` elements between rows), with
 * z = scale * logit (scale, 1 / temperature, above 0):
 *   lse = log sum e^z,   logprob = z_token - lse,   entropy = lse - sum e^(z - lse) z
 *   rank = how many tokens come before the given one
 *   top_ids, top_logprobs [rows][top_k]: the first top_k tokens and their z - lse
 * in the order of larger logit, then lower index; a NaN counts below every number.
 * Logits of -infinity have no part in the sums; a row of nothing else has lse
 * and logprobs of -infinity and entropy 0.  A row that holds NaN or +infinity has
 * NaN for its numbers; order and ranks stay.  A token outside [0, V) has logprob
 * -infinity (NaN in such a row) and rank V.  0 <= top_k <= min(V, 32); up to 2^22 rows and
 * V up to 2^30.  May be NULL: tokens (with logprob and rank), logprob, rank, entropy,
 * lse, and with top_k 0 top_ids and top_logprobs (else one of the two); one output at
 * least.  Any alignment of the logits' own size works; 16 bytes and strides of
 * whole 16 bytes take wider loads.  Results do not depend on the order in which CTAs run.  ws:
 * dg_logprobs_workspace_bytes(op) bytes, 16-byte aligned, overwritten; a call that may overlap
 * another needs its own. */
typedef struct {
    int32_t type;       /* dg_ftype of the logits, where logits_f32 is 0 */
    int32_t logits_f32; /* 0 or 1 */
    int32_t rows;
    int32_t V;
    int32_t top_k;
    float scale;
    int64_t stride;
    const void* logits;
    const int32_t* tokens;
    float* logprob;
    int32_t* rank;
    float* entropy;
    float* lse;
    int32_t* top_ids;
    float* top_logprobs;
} dg_logprobs;
dg_status dg_token_logprobs(const dg_logprobs* op, void* ws, size_t ws_bytes, dg_stream stream);
/* Workspace of dg_token_logprobs (0 where it needs none); 0 for an op that it would refuse. */
size_t dg_logprobs_workspace_bytes(const dg_logprobs* op);

/* Synchronizes `stream`, then reports DG_ERR_CUDA for a sticky CUDA error or
 * DG_ERR_TIMEOUT if a bounded device-side wait gave up on the current device
 * since the last call (clearing that flag).  DG_OK otherwise. */
dg_status dg_check_device_status(dg_stream stream);

/* Diagnostic (not part of the method): launches one tiny kernel that waits on
 * a device word nothing ever sets, with the same bounded wait the step
 * kernel's barriers use, giving up after `spin_limit` polls (1..10^7, ~100 ns
 * each).  The following dg_check_device_status reports DG_ERR_TIMEOUT: the
 * failure path can be exercised without hanging or faulting anything. */
dg_status dg_selftest_wait_timeout(unsigned spin_limit, dg_stream stream);

/* Static, human-readable name of a status. */
const char* dg_status_string(dg_status s);

/* Measurement probes (not part of the method): stream `bytes` through HBM.
 * dg_probe_copy copies src to dst (bytes read + bytes written);
 * dg_probe_read reads src and writes one word per CTA to sink[0..1023].
 * bytes must be a multiple of 16; pointers 16-byte aligned. */
dg_status dg_probe_copy(const void* src, void* dst, size_t bytes, dg_stream stream);
dg_status dg_probe_read(const void* src, size_t bytes, uint32_t* sink, dg_stream stream);

/* Library version string. */
const char* dg_version(void);

#ifdef __cplusplus
}
#endif

#endif /* DG_H_ */

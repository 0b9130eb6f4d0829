/*
 * exl3.h -- C ABI of the GB300 (sm_103a) library for one routed-expert MoE
 * layer whose expert weights are EXL3 K-bit trellis codes.
 *
 * Sources (web pages, cited by title and section):
 *   [p1] "GLM-5.3-Flash EXL3 (~2.1 bpw, SM70 tile order)"
 *   [p2] "GLM-5.3 Flash EXL3 for 2x DGX Sparks"
 *   [p3] "GLM-5.3-Flash EXL3 K2"
 *   [p4] "GLM-5.3-Flash · exlr8 (K2/K3/K4)"
 *
 * Conventions for every entry point:
 *   - Tensors are caller-owned memory; "device" pointers must be CUDA device
 *     (or managed) memory of the current device, "host" pointers host memory.
 *     The library never frees them.  A layer handle borrows the weight
 *     pointers given to exl3_layer_create and must not outlive them.
 *   - `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *     stream).  Work is enqueued asynchronously; nothing synchronises the host
 *     unless stated.  exl3_moe_route and exl3_moe_forward never allocate and
 *     never read device data on the host, so they can be captured in a CUDA
 *     graph (the pages capture decode steps in graphs: [p2] What runs, Graphs).
 *   - Errors: argument, shape and width errors are returned before any launch
 *     and leave outputs untouched.  A failed launch returns EXL3_ERR_CUDA.
 *     Inconsistencies found on the device (bad expert id in a table, a wait
 *     that timed out) set a status word in the workspace, read back with
 *     exl3_get_device_status.
 *   - Layouts are row-major and densely packed unless stated.
 *
 * Format v1 (the library's reading of the pages, which name the format but
 * do not define its bits): codes of one projection of one expert are uint16 [in/16][out/16][16*K]
 * ([p1] intro: packed int16 words holding 16/K weights; [p4] Loading: 16x16
 * tiles, a 4096x128 half at width K is 65,536*K bytes); suh is fp16 [in],
 * svh fp16 [out] ([p2] What runs: trellis + suh + svh + mcg).
 */
#ifndef EXL3_H
#define EXL3_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct exl3_layer exl3_layer_t; /* opaque, immutable after create */

typedef enum {
    EXL3_OK = 0,
    EXL3_ERR_ARG = 1,       /* null pointer, bad enum, top_k out of range */
    EXL3_ERR_SHAPE = 2,     /* dimensions not multiples of 128, T < 0, ... */
    EXL3_ERR_K = 3,         /* code width not in {2, 3, 4} */
    EXL3_ERR_WORKSPACE = 4, /* workspace null or smaller than required */
    EXL3_ERR_CUDA = 5,      /* a CUDA call or launch failed */
    EXL3_ERR_DEVICE = 6     /* no sm_100-family device / device status set */
} exl3_status;

/* EXL3_E4M3 is a type of a key/value cache only (exl3_kv_cache). */
typedef enum { EXL3_F16 = 0, EXL3_BF16 = 1, EXL3_E4M3 = 2 } exl3_dtype;

/* Kernel path for the expert GEMMs.  AUTO picks the grouped GEMV for
 * decode-sized steps (few tokens per expert) and the tcgen05 grouped GEMM
 * for prefill-sized steps. */
typedef enum { EXL3_PATH_AUTO = 0, EXL3_PATH_GEMV = 1, EXL3_PATH_GEMM = 2 } exl3_path;

/* Projection index: 0 = gate, 1 = up, 2 = down. */
typedef struct {
    int num_experts;             /* E, 1..1024 */
    int hidden;                  /* H, multiple of 128 */
    int inter;                   /* I, multiple of 128 */
    int K[3];                    /* code width per projection, 2..4 */
    int fp8_round;               /* 1 = round codebook outputs to FP8 E4M3 before the side
                                    vectors ([p4] intro, the exlr8 rule) */
    uint32_t mcg_mult;           /* mcg multiplier (odd); 0 = 0x9E3779B1 */
    const uint16_t *codes[3];    /* device, [E][in/16][out/16][16*K[p]] */
    const uint16_t *suh[3];      /* device fp16 bits, [E][in] */
    const uint16_t *svh[3];      /* device fp16 bits, [E][out] */
    const uint16_t *shared_w[3]; /* device fp16 bits, dense [in][out], or all NULL: one
                                    unquantized shared expert added with weight 1
                                    ([p4] intro: one shared expert per MoE layer) */
    int hadamard;                /* 0 = format v1; 1 = format v2: the routed projections
                                    carry the 128-point Hadamard rotation on both sides,
                                    W_eff = diag(suh) Hb V Hb diag(svh), Hb block diagonal
                                    with copies of the normalized 128x128 Sylvester matrix,
                                    entries (-1)^popcount(i & j) / sqrt(128) ([p4]
                                    Calibration names the 128x128 Hadamard matrix as a
                                    format primitive).  Other values: EXL3_ERR_ARG */
    int shared_coded;            /* 1: the code, suh and svh arrays hold num_experts + 1
                                    experts, the last one a trellis-coded shared expert
                                    that every token uses with weight 1, after its routed
                                    pairs ([p4] Loading: the shared expert is stored as
                                    expert 288, after the routed experts, at their width).
                                    Requires shared_w all NULL and num_experts + 1 <= 1024.
                                    num_experts stays the router's width (logit columns). */
    const uint8_t *expert_K;     /* host, optional: [num_experts + shared_coded][3] code width
                                    (2..4) of every expert and projection ([p4] Loading: the
                                    bit201 and bit349 manifests give some experts or
                                    projections another width; [p5] Rates: every routed
                                    tensor K3 or K4).  With it K[] is ignored and codes[p]
                                    holds the experts' codes back to back: expert e at word
                                    offset sum over f < e of (in/16)(out/16)*16*expert_K[f][p].
                                    Copied at create (which then allocates two small device
                                    tables, freed by exl3_layer_destroy).  NULL: K[p] for
                                    every expert. */
    int act_fp8;                 /* 1: FP8 x FP8 products.  The activation operand of
                                    every routed projection (x * suh for gate and up,
                                    h * suh for down, after the rotation in format v2) is
                                    quantised per row to E4M3: s = amax / 448 and
                                    q = E4M3_RNE_sat(a / s), both divisions in IEEE fp32,
                                    and the product is s * sum q * v; the tensor-core
                                    path then multiplies E4M3 by E4M3 (tcgen05
                                    kind::f8f6f4).  Requires fp8_round = 1 (the weight
                                    operand is the E4M3 codebook value) ([p4] Widths: with
                                    the E4M3 codebook the prefill runs on FP8 tensor
                                    cores; the pages give no activation recipe, this is
                                    the library's reading).  The dense shared expert is
                                    not affected.  0: fp16 operands.  Other values, or 1
                                    without fp8_round: EXL3_ERR_ARG. */
} exl3_layer_desc;

/* Validate `desc` and build a handle.  codes, suh, svh and shared_w must be
 * 16-byte aligned.  Gate and up may differ in width (K[0] != K[1]): such a
 * layer, like one with expert_K, runs its expert kernels once per width over
 * device-built work lists.  A layer with a dense shared expert also
 * creates one CUDA stream and two events on the current device (released by
 * exl3_layer_destroy); the shared expert of every forward runs on that stream,
 * forked from the caller's stream after routing and joined before the
 * combine, so forwards on one handle must be issued by one host thread at a
 * time.  Errors:
 * EXL3_ERR_ARG (null pointers, shared_w partly NULL), EXL3_ERR_SHAPE,
 * EXL3_ERR_K, EXL3_ERR_DEVICE (current device is not compute capability
 * 10.x), EXL3_ERR_CUDA (stream or event creation failed). */
exl3_status exl3_layer_create(const exl3_layer_desc *desc, exl3_layer_t **out);
void exl3_layer_destroy(exl3_layer_t *layer);

/* Decode projection `proj` of `expert` (0 .. num_experts - 1 + shared_coded)
 * to a dense fp16 matrix out[in][out] (device).  apply_side = 0: the codebook values (after the E4M3 rule when the
 * layer has fp8_round); apply_side = 1: fp16(fp32(fp32(v*suh[i])*svh[o])).
 * The Hadamard rotation of format v2 is never applied here: this is the
 * element-wise, bit-exact check path for the codes ([p2] Cold prefill: the
 * dense "LinearEXL3 reference").  Errors: EXL3_ERR_ARG for bad expert/proj/null. */
exl3_status exl3_decode_dense(const exl3_layer_t *layer, int expert, int proj, int apply_side,
                              uint16_t *out, void *stream);

/* Bytes of workspace exl3_moe_route needs for T tokens, E experts, top_k. */
size_t exl3_route_workspace_size(int T, int E, int top_k);

/* Top-k routing and segment tables ([p4] intro: 288 experts, top-8; [p2] Cold
 * prefill (E3): device-side segment tables, no host sync).
 *   logits      device fp32 [T][E]
 *   ids         device int32 [T][top_k]  experts by descending logit, ties to
 *               the lower index, NaN as -inf
 *   w           device fp32 [T][top_k]   softmax over the k selected logits
 *   seg_offsets device int32 [E+1]       pairs with expert < e
 *   seg_pairs   device int32 [T*top_k]   pair ids t*top_k+j, expert-major,
 *               ascending inside an expert
 *   ws          device, >= exl3_route_workspace_size bytes
 * T = 0 is valid (offsets all zero).  1 <= top_k <= min(E, 16). */
exl3_status exl3_moe_route(const float *logits, int T, int E, int top_k, int32_t *ids, float *w,
                           int32_t *seg_offsets, int32_t *seg_pairs, void *ws, size_t ws_bytes,
                           void *stream);

/* Size of the device array behind exl3_moe_route_static: 1 MiB, held on every
 * device that loads this library until the process exits. */
#define EXL3_ROUTE_STATIC_SCRATCH_BYTES (1u << 20)

/* exl3_moe_route without a workspace argument.  The pages have no counterpart:
 * it exists for callers that cannot allocate device memory themselves, such
 * as a plugin whose host framework owns every device allocation and hands out
 * only the tensors of the call, or a loop that must not call cudaMalloc
 * because cudaMalloc can synchronise the device.  The caller still provides
 * logits and the four outputs, with the layouts, rules and errors of
 * exl3_moe_route; the routing scratch is instead a library-owned device array
 * of EXL3_ROUTE_STATIC_SCRATCH_BYTES.  No call allocates or frees memory.
 *   - Sizes whose exl3_route_workspace_size(T, E, top_k) exceeds
 *     EXL3_ROUTE_STATIC_SCRATCH_BYTES return EXL3_ERR_SHAPE before any launch;
 *     any T <= 4096 with E <= 1024 and top_k <= 16 fits.
 *   - The first call on a device looks up the array's device address
 *     (once per device, with that device current); make that first call
 *     before any stream capture begins.  The address is kept for the life
 *     of the process, so every call must run in the device's primary
 *     context (the CUDA runtime's default): not after cudaDeviceReset, and
 *     not under a context the caller created and made current.
 *   - Every call on a device shares the one array, and it keeps the last
 *     call's contents.  Each call clears what has to start at zero, but calls
 *     whose work overlaps on the GPU (different streams without ordering,
 *     several host threads) race on it: order them on one stream.
 *   - The device status word lives in that array, so exl3_get_device_status
 *     cannot read it. */
exl3_status exl3_moe_route_static(const float *logits, int T, int E, int top_k, int32_t *ids,
                                  float *w, int32_t *seg_offsets, int32_t *seg_pairs,
                                  void *stream);

/* Bytes of workspace exl3_moe_forward needs for T tokens and top_k (all
 * paths).  Deterministic in (layer shape, T, top_k). */
size_t exl3_moe_workspace_size(const exl3_layer_t *layer, int T, int top_k);

/* One MoE layer forward ([p2] Cold prefill (E3): gather, gate/up + SwiGLU,
 * down + scatter; [p1] Running it: decodes the trellis inside the matmul):
 *   x      device [T][H] in dtype dt (fp16 or bf16)
 *   logits device fp32 [T][E], E = num_experts (routed experts)
 *   out    device [T][H] in dtype dt; y_t = sum_j w_tj * expert_{id_tj}(x_t)
 *          (+ shared(x_t)), summed over j in order, no atomics; a coded
 *          shared expert is the last term, a dense one is added after it
 *   ws     device workspace of >= exl3_moe_workspace_size(layer, T, top_k)
 * out may not alias x. */
exl3_status exl3_moe_forward(const exl3_layer_t *layer, const void *x, exl3_dtype dt,
                             const float *logits, int T, int top_k, void *out, void *ws,
                             size_t ws_bytes, void *stream);

/* As exl3_moe_forward, plus an optional residual (device [T][H] in dt, may
 * be NULL; out = round(residual + y)) and an explicit kernel path.
 * Both return EXL3_ERR_SHAPE for T > 262,136 on a layer with a dense shared
 * expert (its launches cover 8 tokens per grid slice), and for more than 2^29
 * (token, expert) pairs (2^26 on the decode-sized GEMV path; exl3_moe_route
 * takes 2^29 too). */
exl3_status exl3_moe_forward_ex(const exl3_layer_t *layer, const void *x, exl3_dtype dt,
                                const float *logits, int T, int top_k, const void *residual,
                                void *out, int path, void *ws, size_t ws_bytes, void *stream);

/* One layer forward over a range of experts, for expert parallelism
 * (expert-parallel sharding of the routed experts over N ranks; the pages
 * split the layer over GPUs and sum the partial outputs with one
 * all-reduce per layer: [p2] Why the overlay exists).  Routing covers every
 * token and expert as in exl3_moe_forward; only the (token, expert) pairs
 * whose expert e has expert_begin <= e < expert_end are computed (with a
 * coded shared expert, its index is num_experts, the last one), plus the
 * dense shared expert when with_shared = 1.  out (device fp32 [T][H]) gets
 * their unrounded sum, summed in pair order, so the ranks' outputs summed
 * over a partition of [0, num_experts + shared_coded) with the shared expert
 * on exactly one rank give the layer before its final rounding (finish with
 * exl3_round_output).  The workspace and path are as for
 * exl3_moe_forward_ex.  Errors: those of exl3_moe_forward_ex, and
 * EXL3_ERR_ARG for a range outside [0, num_experts + shared_coded] or
 * with_shared not 0 / 1. */
exl3_status exl3_moe_forward_experts(const exl3_layer_t *layer, const void *x, exl3_dtype dt,
                                     const float *logits, int T, int top_k, int expert_begin,
                                     int expert_end, int with_shared, float *out, int path,
                                     void *ws, size_t ws_bytes, void *stream);

/* out = round(y + residual) to dt: the last step of a layer whose partial
 * sums were reduced outside the library.  y device fp32 [T][H], residual
 * device [T][H] in dt or NULL, out device [T][H] in dt; all 16-byte aligned,
 * H a multiple of 4. */
exl3_status exl3_round_output(const float *y, int T, int H, const void *residual, exl3_dtype dt,
                              void *out, void *stream);

/* Unweighted RMSNorm of each row: out = round(x / sqrt(mean(x^2) + eps)),
 * fp32 arithmetic, x and out device [T][H] in dt (out may alias x).  Used
 * between layers of a stacked prefill. */
exl3_status exl3_rmsnorm(const void *x, exl3_dtype dt, int T, int H, float eps, void *out,
                         void *stream);

/* Synchronise `stream` and read the device status word of a forward/route
 * workspace (0 = fine). */
exl3_status exl3_get_device_status(const void *ws, void *stream, int32_t *status);

/* Stage-boundary profiling.  When set, every forward on this layer records
 * events[i] (cudaEvent_t, created by the caller) on its stream at these
 * boundaries: 0 start, 1 routing done, 2 gather done, 3 gate/up done,
 * 4 down input prepared, 5 down done, 6 joined with the shared expert's
 * stream, 7 combine done.
 * n_events must be EXL3_NUM_STAGE_EVENTS; events = NULL clears the hook.
 * For measurement only: not safe while another thread runs a forward on the
 * same layer. */
#define EXL3_NUM_STAGE_EVENTS 8
exl3_status exl3_layer_set_stage_events(exl3_layer_t *layer, void *const *events, int n_events);

/* Number of kernels this library has launched in the process so far (a
 * host-side counter; launches captured into a CUDA graph count once, at
 * capture). */
uint64_t exl3_launch_count(void);

/* The per-row E4M3 quantisation of a layer with act_fp8 = 1, on its own:
 * for each of `rows` rows of `n` fp32 values a (device, row-major), the row
 * scale s = fp32(amax / 448) (0 for an all-zero row) and the E4M3 bytes
 * q_i = E4M3_RNE_sat(fp32(a_i / s)) (0 when s = 0), the decisions the
 * activation passes of the FP8 path take ([p4] Widths: FP8 tensor cores; the
 * recipe is the library's reading).  q: device uint8 [rows][n]; s: device
 * fp32 [rows].  Errors: EXL3_ERR_SHAPE for negative sizes, EXL3_ERR_ARG for
 * null pointers, EXL3_ERR_CUDA for a failed launch. */
exl3_status exl3_quantize_rows_e4m3(const float *a, int rows, int n, uint8_t *q, float *s,
                                    void *stream);

/* Test hook for the bounded waits of the tensor-core kernels (the pages have
 * no counterpart).  Every wait inside those kernels has a clock budget; when
 * one runs out, the kernel sets bit 4 (value 4) of the device status word,
 * every CTA of the grid stops issuing work, drains the copies and tensor-core
 * operations it already issued, frees its TMEM and returns, and
 * exl3_get_device_status then reports EXL3_ERR_DEVICE with that bit.  This
 * hook makes such a wait run out on purpose, without any fault: in the
 * gate/up launch of the chosen kernel (1 = big tiles of more than 128
 * tokens, 2 = small tiles of at most 128 tokens) the thread that loads the
 * activation operands skips K step `ks` (64 inputs per step; a step past the
 * end has no effect), so the MMA issuer waits on a barrier that nothing
 * completes, and every wait of that launch gets `budget_cycles` SM clock
 * cycles (100,000 .. 1,000,000,000) instead of the default 1,000,000,000.
 * kernel = 0 clears the hook.  It stays set for every later forward of the
 * process; a forward run with it gives an unspecified output.  Not thread
 * safe.  Errors: EXL3_ERR_ARG for values outside these ranges. */
exl3_status exl3_test_set_wait_fault(int kernel, int ks, long long budget_cycles);

/* ------------------------------------------------------------------------
 * Attention over a paged key/value cache: the other half of the decoder layer
 * that the MoE layer belongs to.  The pages have no counterpart; the three
 * operators follow their formulas below.
 *
 * The device status word of these calls is sticky: kernels only set bits in
 * it, so one word can serve every layer of a step.  The caller zeroes it once
 * (it is the first word of the attention workspace's head, see below, and the
 * word given to exl3_kv_append) and reads it with exl3_get_device_status.  Bits:
 *   1  a page id outside [0, num_pages): the page's keys count as absent, an
 *      append to it is skipped
 *   2  an inconsistent batch: cu_q not ascending or past T, a length outside
 *      [0, max_pages * page_size] or past 2^30, an append before position 0.
 *      A sequence whose cu_q is inconsistent is left out; a length is clamped
 *   4  a bounded wait ran out: outputs are unspecified, those of later calls
 *      too until the caller clears the bit
 */

/* The head of an attention workspace: the status word, and counters that every
 * call expects at zero and leaves at zero.  The caller zeroes these bytes once,
 * before the workspace's first call; what the rest holds does not matter.  A
 * workspace serves one call at a time: calls that may run at once (on other
 * streams, in replayed graphs) need one each. */
#define EXL3_ATTENTION_HEAD_BYTES 4096

/* A paged cache: channel c of kv head h of the token in place i of page p is
 * element p*page_stride + i*token_stride + h*head_stride + c of k and of v. */
typedef struct {
    void *k, *v;            /* device, 16-byte aligned */
    int dtype;              /* exl3_dtype: the activations' type, or EXL3_E4M3 */
    int num_pages;
    int page_size;          /* tokens per page, a multiple of 16, at most 4096 */
    int kv_heads;
    int head_dim;
    int64_t page_stride, token_stride, head_stride; /* elements, multiples of 16 bytes */
    const float *k_scale;   /* device fp32 [kv_heads] or NULL (1): with EXL3_E4M3 a stored */
    const float *v_scale;   /*   value x stands for x * scale (a scale may be 0 or negative);
                                 NULL with the other types */
} exl3_kv_cache;

/* The sequences of one step.  Sequence b has the new tokens cu_q[b] ..
 * cu_q[b+1]-1 of the step (rows of q, k, v, out) and seq_lens[b] tokens in
 * all, the new ones last: new token i of q_len stands at position
 * seq_len - q_len + i.  Position p is in place p % page_size of page
 * block_table[b*table_stride + p / page_size].  Table entries past a
 * sequence's length are never used.  Rows past cu_q[num_seqs] are left alone
 * (padding of a captured graph). */
typedef struct {
    int num_seqs;               /* 0 .. 65535 */
    int max_q;                  /* the most new tokens of a sequence (a hint: it only picks
                                   the kernel, results do not depend on it) */
    int max_pages;              /* entries per row of the table */
    int64_t table_stride;       /* elements */
    const int32_t *cu_q;        /* device [num_seqs + 1] */
    const int32_t *seq_lens;    /* device [num_seqs] */
    const int32_t *block_table; /* device [num_seqs][max_pages] */
} exl3_kv_batch;

/* Head vectors of T tokens: channel c of head h of token t is element
 * t*token_stride + h*head_stride + c of x and, where there is an out, element
 * t*out_token_stride + h*out_head_stride + c of out.  out may be x itself
 * (same strides), and may not overlap it otherwise. */
typedef struct {
    const void *x;              /* device, 16-byte aligned */
    void *out;                  /* device, 16-byte aligned; unused where the cache takes them */
    const void *weight;         /* device [head_dim], activations' type, 16-byte aligned: RMS
                                   norm of every head vector times this; NULL: no norm */
    int heads;
    int64_t token_stride, head_stride;         /* elements, multiples of 8 */
    int64_t out_token_stride, out_head_stride; /* elements, multiples of 8 */
} exl3_heads;

/* Rotary positions: pair i of the first rotary_dim channels turns by
 * position * inv_freq[i] radians, (a, b) -> (a cos - b sin, a sin + b cos).
 * Pair i is (i, i + rotary_dim/2), or (2i, 2i + 1) when interleaved.  The
 * angle is kept as a 64-bit fraction of a turn, so far positions lose
 * nothing.  0 <= inv_freq < 64 (radians per position). */
typedef struct {
    const double *inv_freq;     /* device [rotary_dim / 2] */
    int rotary_dim;             /* a multiple of 16, at most head_dim */
    int interleaved;            /* 0 or 1 */
} exl3_rope;

/* y = rotate(x / sqrt(mean(x^2) + eps) * weight), fp32 arithmetic, rounded
 * once, for every query head and (k not NULL) every key head of T tokens.
 *   positions  device int32 [T], may be negative
 *   rope       NULL: no rotation (positions unused)
 * head_dim a multiple of 8, at most 256.  Errors: EXL3_ERR_ARG (null or
 * misaligned pointers, strides not multiples of 8, bad enum), EXL3_ERR_SHAPE
 * (T < 0, heads < 1, head_dim or rotary_dim outside the above). */
exl3_status exl3_qk_norm_rope(const exl3_heads *q, const exl3_heads *k, exl3_dtype dt, int T,
                              int head_dim, const int32_t *positions, const exl3_rope *rope,
                              float eps, void *stream);

/* The new tokens' keys and values go to the cache: keys normed (k->weight)
 * and rotated as in exl3_qk_norm_rope on the way, values as they are.  With
 * q, the query heads are normed and rotated to q->out in the same launch.
 * Everything is rounded once, from fp32; to E4M3 as
 * E4M3_RNE(clamp(x / scale, -448, 448)), or 0 where the scale is 0, NaN
 * staying NaN.
 *   positions  device int32 [T] of the rotation, or NULL: the positions in the
 *              sequence (where the token is stored never depends on it)
 *   status     device int32, sticky (see above)
 * k->out, v->out, v->weight are not used.  k and v have cache->kv_heads heads.
 * Appending a token again overwrites it.  Errors: those of exl3_qk_norm_rope
 * and, for cache and batch, EXL3_ERR_ARG (null or misaligned pointers,
 * strides, a dtype neither dt nor EXL3_E4M3, scales without EXL3_E4M3) and
 * EXL3_ERR_SHAPE (sizes outside the ranges stated there). */
exl3_status exl3_kv_append(const exl3_kv_cache *cache, const exl3_kv_batch *batch,
                           const exl3_heads *q, const exl3_heads *k, const exl3_heads *v,
                           exl3_dtype dt, int T, const exl3_rope *rope, const int32_t *positions,
                           float eps, int32_t *status, void *stream);

/* Bytes of workspace exl3_paged_attention needs for T new tokens of up to
 * num_seqs sequences. */
size_t exl3_paged_attention_workspace_size(int T, int heads, int kv_heads, int head_dim,
                                           int num_seqs);

/* Attention of the new tokens over the cache, which already holds them:
 *   out_t = sum_p softmax_p(scale * q_t . k_p) v_p
 * over the positions p of t's sequence that t at position P sees: p <= P
 * when causal (every p otherwise), p < seq_len, and p > P - window when
 * window > 0 (requires causal).  Query head h reads kv head
 * h / (heads / kv_heads).  A token that sees nothing gets out = 0 and
 * lse = -inf.  What a token does not see (later tokens, keys before its
 * window, places past the sequence's length) has no effect on it, NaN
 * included.
 *   q      device, element t*q_token_stride + h*q_head_stride + c, strides
 *          multiples of 8
 *   out    device [T][heads][head_dim] in dt, 32-byte aligned; may not
 *          overlap q
 *   lse    device fp32 [T][heads] or NULL: natural log of the sum of
 *          exp(scale * q . k)
 *   path   EXL3_PATH_AUTO, or a fixed kernel: 1 warp-level MMA (few rows),
 *          2 tcgen05 (many rows)
 *   ws     device, 16-byte aligned, its first EXL3_ATTENTION_HEAD_BYTES zeroed
 *          once before its first call (see there)
 * head_dim 64 or 128, heads a multiple of kv_heads.  Scores, the running
 * maximum and sum and the output are fp32; softmax terms are rounded to the
 * 16-bit type of the products (dt; fp16 with an E4M3 cache) before they meet
 * the values; bf16 queries meet an E4M3 cache as fp16, times a power of two per
 * query head that brings its largest channel to 2^14: channels below 2^-31 of
 * that one lose bits, those below 2^-39 count as 0.  Errors: as exl3_kv_append, EXL3_ERR_ARG for scale not finite
 * and positive, window < 0 or without causal, and EXL3_ERR_WORKSPACE. */
exl3_status exl3_paged_attention(const exl3_kv_cache *cache, const exl3_kv_batch *batch,
                                 const void *q, int64_t q_token_stride, int64_t q_head_stride,
                                 exl3_dtype dt, int T, int heads, float scale, int causal,
                                 int window, void *out, float *lse, int path, void *ws,
                                 size_t ws_bytes, void *stream);

/* Test hook of the bounded waits of exl3_paged_attention's tcgen05 kernel, as
 * exl3_test_set_wait_fault is of the MoE kernels': in every CTA, barrier number
 * `barrier` (0 ..; a number past the last has no effect) never completes, so
 * that the waits on it, where the call has any, run out: after `budget_cycles`
 * SM clock cycles (1,000,000 .. 1,000,000,000, the default) in the warp that
 * issues the products, after at most the default in the others.  The call then
 * sets status bit 4, issues nothing more, drains its copies and products, frees
 * its TMEM and returns.  barrier = -1 clears the hook.  It stays set for every
 * later call of the process.  Not thread safe.  Errors: EXL3_ERR_ARG for values
 * outside these ranges. */
exl3_status exl3_test_set_attention_wait_fault(int barrier, long long budget_cycles);

const char *exl3_status_string(exl3_status s);

#ifdef __cplusplus
}
#endif

#endif /* EXL3_H */
